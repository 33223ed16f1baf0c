"""CPU-side checks of the token operators' C ABI: include/rltoken.h's functions
are exported, and bad arguments are refused on the host before anything is
launched (fake device addresses are never dereferenced on these paths)."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import oracle
import ppo_policy_loss_gb300 as rl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "rltoken.h")
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
    assert {"rl_token_logprobs", "rl_token_logprobs_bwd", "rl_topk_distill_fwd_bwd"} <= names
    out = subprocess.run(["nm", "-D", "--defined-only", rl.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT\s+(\w+)", out))


@needs_nvcc
def test_header_compiles_as_c():
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", HEADER], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def call_fwd(lib, **over):
    a = dict(logits=FAKE, dtype=rl.RL_BF16, R=8, V=1000, ld=1000, ids=at(1), n_ids=1, mask=None, temperature=1.0, k=4,
             logp=at(2), entropy=None, lse=None, top=at(3), top_lp=at(4), status=None)
    a.update(over)
    return lib.rl_token_logprobs(a["logits"], a["dtype"], a["R"], a["V"], a["ld"], a["ids"], a["n_ids"], a["mask"],
                                 a["temperature"], a["k"], a["logp"], a["entropy"], a["lse"], a["top"], a["top_lp"],
                                 a["status"], None)


@needs_nvcc
@pytest.mark.parametrize("over,expect", [
    (dict(dtype=7), rl.RL_ERR_DTYPE),
    (dict(R=-1), rl.RL_ERR_SHAPE),
    (dict(R=1 << 31), rl.RL_ERR_SHAPE),
    (dict(V=0), rl.RL_ERR_SHAPE),
    (dict(V=(1 << 26) + 1, ld=(1 << 26) + 8, k=0), rl.RL_ERR_SHAPE),
    (dict(ld=992), rl.RL_ERR_SHAPE),
    (dict(V=3, k=4), rl.RL_ERR_SHAPE),                       # fewer tokens than alternatives
    (dict(V=(1 << 21) + 8, ld=(1 << 21) + 8), rl.RL_ERR_SHAPE),          # row too long to search
    (dict(k=-1), rl.RL_ERR_ARG),
    (dict(k=129), rl.RL_ERR_ARG),
    (dict(n_ids=-1), rl.RL_ERR_ARG),
    (dict(n_ids=129), rl.RL_ERR_ARG),
    (dict(temperature=0.0), rl.RL_ERR_ARG),
    (dict(temperature=-1.0), rl.RL_ERR_ARG),
    (dict(temperature=float("nan")), rl.RL_ERR_ARG),
    (dict(temperature=float("inf")), rl.RL_ERR_ARG),
    (dict(temperature=0.009), rl.RL_ERR_ARG),
    (dict(temperature=101.0), rl.RL_ERR_ARG),
    (dict(logits=None), rl.RL_ERR_NULL),
    (dict(ids=None), rl.RL_ERR_NULL),
    (dict(logp=None), rl.RL_ERR_NULL),
    (dict(top=None), rl.RL_ERR_NULL),
    (dict(top_lp=None), rl.RL_ERR_NULL),
    (dict(logits=FAKE + 8), rl.RL_ERR_ALIGN),
    (dict(V=1001, ld=1001), rl.RL_ERR_ALIGN),
    (dict(R=0), rl.RL_OK),
    (dict(R=0, logits=None, ids=None, logp=None, top=None, top_lp=None), rl.RL_OK),
])
def test_forward_refusals(lib, over, expect):
    assert call_fwd(lib, **over) == expect


def call_bwd(lib, **over):
    a = dict(logits=FAKE, dtype=rl.RL_BF16, R=8, V=1000, ld=1000, ids=at(1), n_ids=1, mask=None, temperature=1.0,
             lse=at(2), entropy=at(3), dlogp=at(4), dentropy=at(5), dlogits=at(6), status=None)
    a.update(over)
    return lib.rl_token_logprobs_bwd(a["logits"], a["dtype"], a["R"], a["V"], a["ld"], a["ids"], a["n_ids"], a["mask"],
                                     a["temperature"], a["lse"], a["entropy"], a["dlogp"], a["dentropy"], a["dlogits"],
                                     a["status"], None)


@needs_nvcc
@pytest.mark.parametrize("over,expect", [
    (dict(dtype=-1), rl.RL_ERR_DTYPE),
    (dict(V=0), rl.RL_ERR_SHAPE),
    (dict(ld=999), rl.RL_ERR_SHAPE),
    (dict(n_ids=129), rl.RL_ERR_ARG),
    (dict(temperature=0.0), rl.RL_ERR_ARG),
    (dict(lse=None), rl.RL_ERR_NULL),
    (dict(dlogits=None), rl.RL_ERR_NULL),
    (dict(dlogp=None), rl.RL_ERR_NULL),
    (dict(ids=None), rl.RL_ERR_NULL),
    (dict(entropy=None), rl.RL_ERR_NULL),
    (dict(dentropy=None), rl.RL_ERR_NULL),
    (dict(n_ids=0, entropy=None, dentropy=None), rl.RL_ERR_NULL),         # no gradient at all
    (dict(dlogits=at(6) + 8), rl.RL_ERR_ALIGN),
    (dict(dlogits=FAKE + 16), rl.RL_ERR_ALIAS),
    (dict(R=0), rl.RL_OK),
])
def test_backward_refusals(lib, over, expect):
    assert call_bwd(lib, **over) == expect


def distill_desc(**over):
    d = rl.rl_topk_distill_desc_init()
    d.logits, d.R, d.V, d.ld = FAKE, 8, 1000, 1000
    d.teacher_ids, d.teacher_logp, d.K = at(1), at(2), 16
    d.dlogits, d.stats_dev, d.workspace = at(3), at(4), at(5)
    d.workspace_bytes = rl.rl_topk_distill_workspace_size()
    for k, v in over.items():
        setattr(d, k, v)
    return d


@needs_nvcc
def test_distill_desc_defaults(lib):
    d = rl.rl_topk_distill_desc_init()
    assert (d.dtype, d.tail, d.reverse, d.temperature, d.grad_scale, d.norm) == (rl.RL_BF16, 0, 0.0, 1.0, 1.0, 0.0)
    assert not d.logits and not d.mask and not d.workspace


@needs_nvcc
@pytest.mark.parametrize("over,expect", [
    (dict(dtype=9), rl.RL_ERR_DTYPE),
    (dict(tail=2), rl.RL_ERR_DTYPE),
    (dict(R=-1), rl.RL_ERR_SHAPE),
    (dict(V=0), rl.RL_ERR_SHAPE),
    (dict(ld=992), rl.RL_ERR_SHAPE),
    (dict(K=0), rl.RL_ERR_ARG),
    (dict(K=129), rl.RL_ERR_ARG),
    (dict(reverse=-0.1), rl.RL_ERR_ARG),
    (dict(reverse=1.1), rl.RL_ERR_ARG),
    (dict(reverse=float("nan")), rl.RL_ERR_ARG),
    (dict(reverse=0.5, tail=rl.RL_DISTILL_TAIL_RENORM), rl.RL_ERR_ARG),
    (dict(temperature=0.0), rl.RL_ERR_ARG),
    (dict(temperature=1e3), rl.RL_ERR_ARG),
    (dict(grad_scale=float("inf")), rl.RL_ERR_ARG),
    (dict(norm=-1.0), rl.RL_ERR_ARG),
    (dict(norm=float("nan")), rl.RL_ERR_ARG),
    (dict(stats_dev=None), rl.RL_ERR_NULL),
    (dict(logits=None), rl.RL_ERR_NULL),
    (dict(teacher_ids=None), rl.RL_ERR_NULL),
    (dict(teacher_logp=None), rl.RL_ERR_NULL),
    (dict(workspace=None), rl.RL_ERR_WORKSPACE),
    (dict(workspace_bytes=64), rl.RL_ERR_WORKSPACE),
    (dict(logits=FAKE + 2), rl.RL_ERR_ALIGN),
    (dict(dlogits=at(3) + 8), rl.RL_ERR_ALIGN),
    (dict(workspace=at(5) + 8), rl.RL_ERR_ALIGN),
    (dict(V=1001, ld=1001), rl.RL_ERR_ALIGN),
    (dict(dlogits=FAKE + 32), rl.RL_ERR_ALIAS),
])
def test_distill_refusals(lib, over, expect):
    import ctypes
    assert lib.rl_topk_distill_fwd_bwd(ctypes.byref(distill_desc(**over)), None) == expect
    assert lib.rl_topk_distill_fwd_bwd(None, None) == rl.RL_ERR_NULL


@needs_nvcc
def test_distill_records_match_the_header(lib):
    """The ctypes records have the C structs' sizes and offsets."""
    import ctypes
    names = {"rl_topk_distill_desc": rl.rl_topk_distill_desc, "rl_distill_stats": rl.rl_distill_stats}
    src = "#include <stdio.h>\n#include <stddef.h>\n#include \"rltoken.h\"\nint main(void) {\n"
    for n, t in names.items():
        src += f'printf("%zu", sizeof({n}));\n'
        for f, _ in t._fields_:
            src += f'printf(" %zu", offsetof({n}, {f}));\n'
        src += 'printf("\\n");\n'
    src += "return 0; }\n"
    import tempfile
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "t.c"), "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), os.path.join(d, "t.c"), "-o", os.path.join(d, "t")], check=True)
        got = subprocess.run([os.path.join(d, "t")], capture_output=True, text=True, check=True).stdout.splitlines()
    for line, t in zip(got, names.values()):
        assert [int(x) for x in line.split()] == [ctypes.sizeof(t)] + [getattr(t, f).offset for f, _ in t._fields_]


# ------------------------------------------------------------------ the oracle against closed forms
def test_oracle_distill_closed_forms():
    V = 6
    z = np.log(np.array([[0.5, 0.2, 0.1, 0.1, 0.06, 0.04]]))
    ids, q = np.array([[0, 2]]), np.array([[0.7, 0.2]])
    o = oracle.topk_distill(z, "f64", V, ids, np.log(q))
    want = 0.7 * np.log(0.7 / 0.5) + 0.2 * np.log(0.2 / 0.1) + 0.1 * np.log(0.1 / 0.4)
    assert np.isclose(o["loss"], want, rtol=1e-12) and np.isclose(o["student_tail"], 0.4) and np.isclose(o["teacher_tail"], 0.1)
    assert np.isclose(o["reverse_kl"], 0.5 * np.log(0.5 / 0.7) + 0.1 * np.log(0.1 / 0.2) + 0.4 * np.log(0.4 / 0.1))
    assert np.allclose(o["dlogits"][0], [0.5 - 0.7, 0.2 * (1 - 0.25), 0.1 - 0.2, 0.1 * 0.75, 0.06 * 0.75, 0.04 * 0.75])
    same = oracle.topk_distill(z, "f64", V, ids, z[:, [0, 2]], reverse=0.5)   # the student's own probabilities
    assert abs(same["loss"]) < 1e-15 and np.abs(same["dlogits"]).max() < 1e-15
    r = oracle.topk_distill(z, "f64", V, ids, np.log(q), tail="renormalise")
    assert np.isclose(r["loss"], 7 / 9 * np.log(7 / 9 / 0.5) + 2 / 9 * np.log(2 / 9 / 0.1))
    assert np.allclose(r["dlogits"][0], [0.5 - 7 / 9, 0.2, 0.1 - 2 / 9, 0.1, 0.06, 0.04])


def test_oracle_distill_gradient_against_differences():
    g = np.random.default_rng(5)
    R, V, K, h = 3, 10, 4, 1e-5
    z = g.normal(0, 1.5, (R, V))
    ids = np.stack([g.permutation(V)[:K] for _ in range(R)])
    ids[1, 3] = -1
    lq = np.log(g.dirichlet(np.ones(K + 1), R))[:, :K]
    for kw in (dict(), dict(reverse=1.0), dict(reverse=0.3, temperature=1.7, weight=np.array([1.0, 2.0, 0.5]), norm=4.0),
               dict(tail="renormalise", mask=np.array([1, 1, 0]))):
        d = oracle.topk_distill(z, "f64", V, ids, lq, **kw)["dlogits"]
        for r in range(R):
            for v in range(V):
                a, b = z.copy(), z.copy()
                a[r, v] += h
                b[r, v] -= h
                num = (oracle.topk_distill(a, "f64", V, ids, lq, **kw)["loss"] - oracle.topk_distill(b, "f64", V, ids, lq, **kw)["loss"]) / (2 * h)
                assert abs(num - d[r, v]) < 1e-8, (kw, r, v)


def test_oracle_logprobs_closed_forms():
    V = 50
    z = np.zeros((3, V), np.float32)
    z[1, 7] = 3.0
    z[2, 10:] = -np.inf
    o = oracle.token_logprobs(z, "f32", V, np.array([[0], [7], [3]]), None, 3, 2.0)
    assert np.allclose(o["logp"][:, 0], [-np.log(50), 1.5 - np.log(np.exp(1.5) + 49), -np.log(10)], rtol=1e-14)
    assert np.allclose(o["entropy"][[0, 2]], [np.log(50), np.log(10)], rtol=1e-14)
    assert o["topk_ids"].tolist() == [[0, 1, 2], [7, 0, 1], [0, 1, 2]]
    p = np.exp(o["topk_logp"][1])
    assert np.isclose(p[0] + 49 * p[1], 1.0, rtol=1e-14)
    m = oracle.token_logprobs(z, "f32", V, np.array([[0], [7], [3]]), np.array([1, 0, 1]), 3, 2.0)
    assert m["topk_ids"][1].tolist() == [-1] * 3 and m["logp"][1, 0] == 0 and m["lse"][1] == 0


def test_oracle_gradient_against_differences():
    g = np.random.default_rng(3)
    R, V, h = 3, 11, 1e-5
    z = g.normal(0, 2, (R, V))
    ids = np.array([[1, 1], [0, 5], [10, 2]])
    dl, de = g.normal(size=(R, 2)), g.normal(size=R)
    o = oracle.token_logprobs(z, "f64", V, ids, None, 0, 0.7)
    d, _, _ = oracle.token_logprobs_bwd(z, "f64", V, ids, dl, o["lse"], o["entropy"], de, None, 0.7)

    def f(x):
        q = oracle.token_logprobs(x, "f64", V, ids, None, 0, 0.7)
        return (q["logp"] * dl).sum() + (q["entropy"] * de).sum()

    for r in range(R):
        for v in range(V):
            a, b = z.copy(), z.copy()
            a[r, v] += h
            b[r, v] -= h
            assert abs((f(a) - f(b)) / (2 * h) - d[r, v]) < 1e-7


@needs_nvcc
def test_distill_refuses_a_record_off_its_boundary(lib):
    import ctypes
    assert lib.rl_topk_distill_fwd_bwd(ctypes.byref(distill_desc(stats_dev=at(4) + 4)), None) == rl.RL_ERR_ALIGN
