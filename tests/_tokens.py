"""Shared helpers of the token log-probability and distillation tests: inputs,
the oracle's view of them, and rounding bounds.

Bounds.  u = 2^-24 is half a step of fp32.  The kernels form x = (z - m) c
with three roundings (the difference, c itself, the product), so 2^x carries
|ln p| 3 u relative error plus the hardware exponential's 2^-22 = 4 u.  A row's
sum runs over V / 512 terms in each of 512 chains (256 threads, two chains
each) and is then joined in 8 + 8 steps, each rounding at most u of the partial
sum: sum_steps(V) = V / 512 + 64 covers those, the exponentials' own errors
(weighted by p, |ln p| averages to the entropy, at most ln V < 13) and the
logarithm's.  Everything below is that many u, times the size of what is
rounded.
"""
import numpy as np
import torch

import oracle

U = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}  # half the last subnormal, or what is flushed


def storage(t):
    t = t.detach().cpu()
    if t.dtype in (torch.bfloat16, torch.float16):
        return t.contiguous().view(torch.int16).numpy().view(np.uint16)
    return t.contiguous().numpy()


def sum_steps(V):
    return V / 512 + 64


def logits(R, V, dtype, seed, ld=None, sd=3.0, sure=True):
    """[R, V] view of a [R, ld] tensor; columns past V hold NaN."""
    per = 4 if dtype == "f32" else 8
    ld = -(-V // per) * per if ld is None else ld
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn((R, ld), generator=gen) * sd
    if sure and R > 2:
        z[::3, V // 2] += 20.0  # rows with one token far above the others
    z[:, V:] = float("nan")
    return z.to(TORCH[dtype])[:, :V]


def check_close(name, got, ref, tol):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (name, "NaN places differ")
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), (name, "infinities differ")
    fine = np.isfinite(ref)
    tol = np.broadcast_to(tol, ref.shape)[fine]
    err = np.abs(got[fine] - ref[fine])
    if err.size:
        i = int(np.argmax(err - tol))
        assert (err <= tol).all(), (name, float(err[i]), float(tol[i]), float(got[fine][i]), float(ref[fine][i]))


def check_logprobs(out, ref, V, temperature=1.0):
    """The forward outputs against the oracle's."""
    n = sum_steps(V)
    for key in ("logp", "topk_logp"):
        if out.get(key) is not None and ref[key] is not None:
            r = ref[key].reshape(tuple(out[key].shape))
            # small log-probabilities keep relative precision: log1p(r) <= e^logp-weighted sums
            with np.errstate(invalid="ignore"):
                small = np.minimum(1.0, np.where(np.isfinite(r), np.abs(r), 1.0))
            # a row's log-probability next to 0 is log1p of a small sum; any other carries its row's
            # (each of V terms below 2^-126 may be flushed: V 2^-126 of the sum r)
            check_close(key, out[key].cpu(), r, n * U * np.where(small < 0.5, 2 * small, 1.0) + 4 * U * np.abs(
                np.where(np.isfinite(r), r, 0.0)) + V * TINY["f32"])
    if out.get("lse") is not None:
        check_close("lse", out["lse"].cpu(), ref["lse"], n * U + 4 * U * np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0)))
    if out.get("entropy") is not None:
        # (a flushed term p < 2^-126 takes p |ln p| < 90 2^-126 along)
        H = ref["entropy"]
        small = np.where(np.isfinite(H), np.minimum(1.0, np.abs(H)), 1.0)
        check_close("entropy", out["entropy"].cpu(), H, n * U * 3 * (small + np.where(np.isfinite(H), H, 0.0)) + 90 * V * TINY["f32"])
    if out.get("topk_ids") is not None:
        got = out["topk_ids"].cpu().numpy()
        assert np.array_equal(got, ref["topk_ids"]), np.argwhere(got != ref["topk_ids"])[:4]


def check_gradient(got, dtype, d, size, lp, temperature=1.0):
    """One rounding to the output's type, p's relative error on each part, and
    the sum of the ids' gradients (at most 128 terms: 2^7 u)."""
    with np.errstate(invalid="ignore", over="ignore"):
        rel = (4 * np.where(np.isfinite(lp), np.abs(lp), 0.0) + 16 + 128) * U
        tol = HALF_STEP[dtype] * np.abs(d) * (1 + 2 * rel) + rel * np.where(np.isfinite(size), size, 0.0) + TINY[dtype]
    check_close("dlogits", oracle.decode(storage(got), dtype), d, np.where(np.isfinite(tol), tol, 0.0))
