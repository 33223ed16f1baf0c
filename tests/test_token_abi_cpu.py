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
    assert {"rl_token_logprobs", "rl_token_logprobs_bwd"} <= names
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
    (dict(V=(1 << 30) + 1, ld=(1 << 30) + 8, k=0), rl.RL_ERR_SHAPE),
    (dict(ld=992), rl.RL_ERR_SHAPE),
    (dict(V=3, k=4), rl.RL_ERR_SHAPE),                       # fewer tokens than alternatives
    (dict(V=(1 << 18) + 8, ld=(1 << 18) + 8), rl.RL_ERR_SHAPE),          # row too long to search
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


# ------------------------------------------------------------------ the oracle against closed forms
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
