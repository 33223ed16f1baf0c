"""CPU-side checks of the rollout operators' C ABI: include/rlrollout.h's functions
are exported, and bad arguments are refused on the host before anything is
launched (fake device addresses are never dereferenced on these paths)."""
import ctypes
import os
import re
import shutil
import subprocess
import tempfile

import numpy as np
import pytest

import ppo_policy_loss_gb300 as rl
from tests._rollout import quantize_ref, verify_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rlrollout.h")
FAKE = 0x7F0000000000

needs_nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="no CUDA toolkit")


@pytest.fixture(scope="module")
def lib():
    rl.build()
    return rl.load()


def at(i):
    return FAKE + i * 0x40000000000


@needs_nvcc
def test_declared_functions_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(rl_[a-z0-9_]+)\s*\(", text))
    assert {"rl_quantize_rows_int8", "rl_lmhead_logits_int8", "rl_verify_drafts"} <= names
    out = subprocess.run(["nm", "-D", "--defined-only", rl.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT\s+(\w+)", out))
    for n in names:
        assert n in rl.__all__ and hasattr(rl, n)


@needs_nvcc
def test_header_compiles_as_c():
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", HEADER], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def call_quantize(lib, **over):
    a = dict(x=FAKE, dtype=rl.RL_BF16, R=8, D=1000, ld_x=1000, codes=at(1), ld_c=1008, scale=at(2))
    a.update(over)
    return lib.rl_quantize_rows_int8(a["x"], a["dtype"], a["R"], a["D"], a["ld_x"], a["codes"], a["ld_c"], a["scale"], None)


@needs_nvcc
@pytest.mark.parametrize("over,expect", [
    (dict(dtype=3), rl.RL_ERR_DTYPE),
    (dict(R=-1), rl.RL_ERR_SHAPE),
    (dict(R=1 << 31), rl.RL_ERR_SHAPE),
    (dict(D=0), rl.RL_ERR_SHAPE),
    (dict(D=1 << 31, ld_x=1 << 31, ld_c=1 << 31), rl.RL_ERR_SHAPE),
    (dict(ld_x=992), rl.RL_ERR_SHAPE),
    (dict(ld_c=992), rl.RL_ERR_SHAPE),
    (dict(ld_x=1 << 60), rl.RL_ERR_SHAPE),
    (dict(x=None), rl.RL_ERR_NULL),
    (dict(codes=None), rl.RL_ERR_NULL),
    (dict(scale=None), rl.RL_ERR_NULL),
    (dict(x=FAKE + 8), rl.RL_ERR_ALIGN),
    (dict(ld_x=1004), rl.RL_ERR_ALIGN),
    (dict(codes=at(1) + 8), rl.RL_ERR_ALIGN),
    (dict(ld_c=1000), rl.RL_ERR_ALIGN),
    (dict(scale=at(2) + 2), rl.RL_ERR_ALIGN),
    (dict(codes=FAKE), rl.RL_ERR_ALIAS),
    (dict(codes=FAKE + 7 * 2000 + 1984), rl.RL_ERR_ALIAS),
    (dict(R=0, x=None, codes=None, scale=None), rl.RL_OK),
])
def test_quantize_refusals(lib, over, expect):
    assert call_quantize(lib, **over) == expect


def call_logits(lib, **over):
    a = dict(h=FAKE, ld_h=1008, sh=at(1), w=at(2), ld_w=1008, sw=at(3), R=8, D=1000, V=5000, dtype=rl.RL_BF16, out=at(4), ld=5000, status=None,
             ws=at(5), ws_bytes=None)
    a.update(over)
    if a["ws_bytes"] is None:
        a["ws_bytes"] = 1 << 40
    return lib.rl_lmhead_logits_int8(a["h"], a["ld_h"], a["sh"], a["w"], a["ld_w"], a["sw"], a["R"], a["D"], a["V"], a["dtype"], a["out"], a["ld"],
                                     a["status"], a["ws"], a["ws_bytes"], None)


@needs_nvcc
@pytest.mark.parametrize("over,expect", [
    (dict(dtype=5), rl.RL_ERR_DTYPE),
    (dict(R=-1), rl.RL_ERR_SHAPE),
    (dict(R=1 << 31), rl.RL_ERR_SHAPE),
    (dict(D=0), rl.RL_ERR_SHAPE),
    (dict(D=131072, ld_h=131072, ld_w=131072), rl.RL_ERR_SHAPE),
    (dict(V=0), rl.RL_ERR_SHAPE),
    (dict(V=1 << 31, ld=1 << 31), rl.RL_ERR_SHAPE),
    (dict(ld_h=992), rl.RL_ERR_SHAPE),
    (dict(ld_w=992), rl.RL_ERR_SHAPE),
    (dict(ld=4992), rl.RL_ERR_SHAPE),
    (dict(h=None), rl.RL_ERR_NULL),
    (dict(w=None), rl.RL_ERR_NULL),
    (dict(sh=None), rl.RL_ERR_NULL),
    (dict(sw=None), rl.RL_ERR_NULL),
    (dict(out=None), rl.RL_ERR_NULL),
    (dict(h=FAKE + 1), rl.RL_ERR_ALIGN),
    (dict(w=at(2) + 8), rl.RL_ERR_ALIGN),
    (dict(ld_h=1000), rl.RL_ERR_ALIGN),
    (dict(ld_w=1001), rl.RL_ERR_ALIGN),
    (dict(ld=5001), rl.RL_ERR_ALIGN),
    (dict(out=at(4) + 2), rl.RL_ERR_ALIGN),
    (dict(ws=at(5) + 4), rl.RL_ERR_ALIGN),
    (dict(sw=at(3) + 1), rl.RL_ERR_ALIGN),
    (dict(out=FAKE), rl.RL_ERR_ALIAS),
    (dict(out=at(2) + 4096), rl.RL_ERR_ALIAS),
    (dict(ws=None), rl.RL_ERR_WORKSPACE),
    (dict(ws_bytes=8 * 1000 * 2 - 1), rl.RL_ERR_WORKSPACE),
    (dict(R=0, h=None, w=None, sh=None, sw=None, out=None, ws=None), rl.RL_OK),
])
def test_logits_refusals(lib, over, expect):
    assert call_logits(lib, **over) == expect


@needs_nvcc
def test_workspace_size(lib):
    assert rl.rl_lmhead_int8_workspace_size(-1, 64) == 0 and rl.rl_lmhead_int8_workspace_size(8, 131072) == 0
    assert rl.rl_lmhead_int8_workspace_size(8, 0) == 0 and rl.rl_lmhead_int8_workspace_size(1 << 31, 64) == 0
    sizes = [rl.rl_lmhead_int8_workspace_size(r, 1024) for r in (1, 16, 100, 4096)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    call = dict(R=8, ws_bytes=rl.rl_lmhead_int8_workspace_size(8, 1000) - 1)
    assert call_logits(lib, **call) == rl.RL_ERR_WORKSPACE


@needs_nvcc
@pytest.mark.parametrize("over", [
    dict(ws=FAKE + 1024), dict(ws=at(2) + 16), dict(ws=at(4) + 16), dict(ws=at(1) + 16, sh=at(1) + 16), dict(ws=at(3), sw=at(3) + 8),
    dict(out=at(4), sh=at(4) + 64), dict(out=at(4), sw=at(4) + 4096), dict(out=at(4) + 16 * 1000, ws=at(4)),
])
def test_logits_shared_memory(lib, over):
    """Neither the logits nor the scratch may lie in what is read, nor in one another."""
    assert call_logits(lib, **over) == rl.RL_ERR_ALIAS


@needs_nvcc
@pytest.mark.parametrize("over", [dict(codes=FAKE + 1024), dict(scale=FAKE + 64), dict(scale=at(1) + 1008 * 7), dict(codes=at(2), scale=at(2) + 16)])
def test_codes_shared_memory(lib, over):
    assert call_quantize(lib, **over) == rl.RL_ERR_ALIAS


def verify_desc(**over):
    d = rl.rl_verify_drafts_desc_init()
    d.target_logits, d.B, d.G, d.V, d.ld = FAKE, 8, 3, 1000, 1000
    d.draft_logits, d.ld_draft, d.draft_lse, d.draft_ids = at(1), 1000, at(2), at(3)
    d.uniforms, d.tokens = at(4), at(5)
    for k, v in over.items():
        setattr(d, k, v)
    return d


@needs_nvcc
def test_verify_desc_defaults(lib):
    d = rl.rl_verify_drafts_desc_init()
    assert (d.dtype, d.temperature, d.B, d.G) == (rl.RL_BF16, 1.0, 0, 0) and not d.target_logits and not d.n_draft and not d.status_dev
    lib.rl_verify_drafts_desc_init(None)


@needs_nvcc
@pytest.mark.parametrize("over,expect", [
    (dict(dtype=9), rl.RL_ERR_DTYPE),
    (dict(B=-1), rl.RL_ERR_SHAPE),
    (dict(B=1 << 31), rl.RL_ERR_SHAPE),
    (dict(B=1 << 29), rl.RL_ERR_SHAPE),                      # times four rows
    (dict(G=-1), rl.RL_ERR_SHAPE),
    (dict(G=129), rl.RL_ERR_SHAPE),
    (dict(V=0), rl.RL_ERR_SHAPE),
    (dict(V=(1 << 26) + 1, ld=(1 << 26) + 8, ld_draft=(1 << 26) + 8), rl.RL_ERR_SHAPE),
    (dict(ld=992), rl.RL_ERR_SHAPE),
    (dict(ld_draft=992), rl.RL_ERR_SHAPE),
    (dict(ld=1 << 60), rl.RL_ERR_SHAPE),
    (dict(temperature=0.0), rl.RL_ERR_ARG),
    (dict(temperature=float("nan")), rl.RL_ERR_ARG),
    (dict(temperature=0.0099), rl.RL_ERR_ARG),
    (dict(temperature=100.5), rl.RL_ERR_ARG),
    (dict(target_logits=None), rl.RL_ERR_NULL),
    (dict(draft_lse=None), rl.RL_ERR_NULL),
    (dict(draft_ids=None), rl.RL_ERR_NULL),
    (dict(uniforms=None), rl.RL_ERR_NULL),
    (dict(tokens=None), rl.RL_ERR_NULL),
    (dict(target_logits=FAKE + 2), rl.RL_ERR_ALIGN),
    (dict(draft_logits=at(1) + 8), rl.RL_ERR_ALIGN),
    (dict(V=999, ld=1001), rl.RL_ERR_ALIGN),
    (dict(ld_draft=1001), rl.RL_ERR_ALIGN),
    (dict(uniforms=at(4) + 4), rl.RL_ERR_ALIGN),
    (dict(tokens=at(5) + 4), rl.RL_ERR_ALIGN),
    (dict(B=0), rl.RL_OK),
    (dict(B=0, target_logits=None, uniforms=None, tokens=None), rl.RL_OK),
])
def test_verify_refusals(lib, over, expect):
    assert lib.rl_verify_drafts(ctypes.byref(verify_desc(**over)), None) == expect


@needs_nvcc
@pytest.mark.parametrize("over", [
    dict(tokens=at(3)), dict(tokens=at(3) + 8 * 23), dict(tokens=at(4) + 8), dict(tokens=FAKE + 16), dict(tokens=at(1) + 16), dict(tokens=at(2)),
    dict(n_draft=at(6), tokens=at(6) - 8), dict(n_accepted=at(5) + 8 * 31), dict(n_accepted=at(3)), dict(logp_out=at(2) + 4), dict(lse_out=at(2)),
    dict(logp_out=at(7), lse_out=at(7)), dict(logp_out=at(7), lse_out=at(7) + 4 * 31), dict(logp_out=at(5)), dict(lse_out=at(4)),
])
def test_verify_shared_memory(lib, over):
    """No output may lie in an input or in another output."""
    assert lib.rl_verify_drafts(ctypes.byref(verify_desc(**over)), None) == rl.RL_ERR_ALIAS


@needs_nvcc
def test_verify_rows_that_64_bits_do_not_address(lib):
    assert lib.rl_verify_drafts(ctypes.byref(verify_desc(B=1 << 24, ld=1 << 39)), None) == rl.RL_ERR_SHAPE
    assert lib.rl_verify_drafts(ctypes.byref(verify_desc(B=1 << 24, ld_draft=1 << 39)), None) == rl.RL_ERR_SHAPE


@needs_nvcc
def test_verify_without_a_descriptor(lib):
    assert lib.rl_verify_drafts(None, None) == rl.RL_ERR_NULL


# ------------------------------------------------------------------ the plain forms themselves
def test_codes_reference():
    q, s = quantize_ref(np.array([[127.0, -63.5, 63.5, 0.5, 1.5, -127.0], [0] * 6, [np.nan, 1, 2, 3, 4, 5]]))
    assert s[0] == 1 and q[0].tolist() == [127, -64, 64, 0, 2, -127]
    assert s[1] == 0 and not q[1].any() and np.isnan(s[2]) and not q[2].any()


def test_verification_reference_keeps_the_targets_distribution():
    """Over a grid of uniforms and all drafts, weighted by q, the first token's distribution is p."""
    gen = np.random.default_rng(3)
    V, n = 5, 60
    zt, zq = gen.normal(size=V), gen.normal(size=V)
    p, q = np.exp(zt) / np.exp(zt).sum(), np.exp(zq) / np.exp(zq).sum()
    lq = np.log(np.exp(zq).sum())
    g = (np.arange(n) + 0.5) / n
    u = np.stack(np.meshgrid(g, g, indexing="ij"), -1).reshape(-1, 2)
    got = np.zeros(V)
    for d in range(V):
        out = verify_ref(np.broadcast_to(zt, (n * n, 2, V)), np.full((n * n, 1), d), u, np.broadcast_to(zq, (n * n, 1, V)), np.full((n * n, 1), lq))
        got += q[d] * np.bincount(out["tokens"][:, 0], minlength=V) / (n * n)
    assert np.abs(got - p).max() < 3 / n


@needs_nvcc
def test_strides_beyond_the_address_space(lib):
    """Row spans of more than 2^60 bytes are refused before their product is formed."""
    big = 1 << 39
    assert call_quantize(lib, R=(1 << 31) - 1, ld_x=big) == rl.RL_ERR_SHAPE
    assert call_quantize(lib, R=(1 << 31) - 1, ld_c=big) == rl.RL_ERR_SHAPE
    assert call_logits(lib, R=(1 << 31) - 1, ld=big) == rl.RL_ERR_SHAPE
    assert call_logits(lib, R=(1 << 31) - 1, ld_h=big) == rl.RL_ERR_SHAPE
    assert call_logits(lib, V=(1 << 31) - 1, ld=1 << 32, ld_w=big) == rl.RL_ERR_SHAPE
    # more tiles than a launch counts
    assert call_logits(lib, R=1 << 24, V=(1 << 31) - 8, D=64, ld_h=64, ld_w=64, ld=1 << 31, w=at(2) + (1 << 56), out=at(4) + (1 << 57),
                       ws_bytes=1 << 50) == rl.RL_ERR_SHAPE


@needs_nvcc
def test_verify_record_matches_the_header(lib):
    """The ctypes record has the C struct's size and offsets."""
    t = rl.rl_verify_drafts_desc
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"rlrollout.h\"\nint main(void) {\n"
    src += 'printf("%zu", sizeof(rl_verify_drafts_desc));\n'
    for f, _ in t._fields_:
        src += f'printf(" %zu", offsetof(rl_verify_drafts_desc, {f}));\n'
    src += "return 0; }\n"
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "t.c"), "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), os.path.join(d, "t.c"), "-o", os.path.join(d, "t")], check=True)
        got = subprocess.run([os.path.join(d, "t")], capture_output=True, text=True, check=True).stdout
    assert [int(x) for x in got.split()] == [ctypes.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]
