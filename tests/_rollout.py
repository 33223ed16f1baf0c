"""Plain fp64 forms of the rollout's operators, for the tests."""
import math

import numpy as np
import torch

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24  # half a step of fp32
RESOLUTION = 2.0 ** -34  # of a drawn token's border (include/rlrollout.h)


def quantize_ref(x):
    """(codes, scale) of float64 rows x that are numbers of a storage type."""
    a = np.abs(x).max(1)
    with np.errstate(invalid="ignore", over="ignore"):
        s = (a / 127.0).astype(np.float32)
        s = np.where(np.isfinite(a), s, np.float32(np.nan))
        held = np.where(s > 0, s, 1.0).astype(np.float64)
        q = np.clip(np.rint(x / held[:, None]), -127, 127)
    q = np.where((s > 0)[:, None], q, 0.0)
    return q.astype(np.int8), s


def logits_ref(h, sh, w, sw, dtype):
    """Logits with every rounding of the definition, as a torch tensor of the type."""
    acc = h.astype(np.int64) @ w.astype(np.int64).T
    with np.errstate(over="ignore", invalid="ignore"):
        z = acc.astype(np.float32) * sh[:, None] * sw[None, :]
    assert z.dtype == np.float32
    return torch.from_numpy(z).to(TORCH[dtype])


def verify_ref(target, ids, u, draft=None, draft_lse=None, n_draft=None, temperature=1.0):
    """The definition, one sequence after the other; target [B, G + 1, V] float64.
    The wording of the refusals is the header's: ids or counts out of range,
    rows without a distribution."""
    B, rows, V = target.shape
    G = rows - 1
    out = dict(tokens=np.full((B, rows), -1, np.int64), n_accepted=np.zeros(B, np.int64), logp=np.zeros((B, rows)),
               lse=np.zeros((B, rows)), status=0, near={})
    for b in range(B):
        n = G if n_draft is None else int(n_draft[b])
        if n < -1 or n > G or any(not 0 <= int(ids[b, i]) < V for i in range(max(n, 0))):
            out["logp"][b] = out["lse"][b] = np.nan
            out["status"] |= 1
            continue
        for i in range(n + 1):
            z = target[b, i] / temperature
            if np.isnan(z).any() or z.max() == np.inf or z.max() == -np.inf:
                out["logp"][b, i] = out["lse"][b, i] = np.nan
                break
            m = z.max()
            e = np.exp(z - m)
            S = e.sum()
            top = int(np.argmax(z))
            rest = np.delete(e, top).sum()
            out["lse"][b, i] = m + math.log1p(rest)
            p = e / S
            w = p
            if i < n:
                d = int(ids[b, i])
                if draft is None:
                    q = np.zeros(V)
                    q[d] = 1.0
                else:
                    zq, lq = draft[b, i] / temperature, float(draft_lse[b, i])
                    if not (zq[d] < np.inf) or not np.isfinite(lq):
                        out["logp"][b, i] = np.nan
                        break
                    with np.errstate(over="ignore", invalid="ignore"):
                        q = np.exp(zq - lq)
                if u[b, i] * q[d] < p[d]:
                    out["tokens"][b, i], out["logp"][b, i] = d, (z[d] - m) - math.log1p(rest)
                    out["n_accepted"][b] = i + 1
                    continue
                if draft is not None and not (draft[b, i] < np.inf).all():
                    out["logp"][b, i] = np.nan
                    break
                r = np.maximum(p - q, 0.0)
                w = r if r.sum() > 0 else p
            x = u[b, G]
            x = 0.0 if not x > 0 else min(x, 1 - 2.0 ** -53)
            edges = np.cumsum(w)
            over = np.nonzero((edges > x * edges[-1]) & (w > 0))[0]
            t = int(over[0]) if over.size else int(np.nonzero(w)[0][-1])
            out["tokens"][b, i], out["logp"][b, i] = t, (z[t] - m) - math.log1p(rest)
            # A border of the token within RESOLUTION of the row's total (1, p being normalised): the
            # kernel holds u and the sums in 48 bits and its terms to 2^-41, so which side of such a
            # border u lies on is not decided, and the neighbour with a weight is as right.
            weighty = np.nonzero(w > 0)[0]
            k = int(np.searchsorted(weighty, t))
            if k > 0 and x * edges[-1] - edges[weighty[k - 1]] <= RESOLUTION:
                out["near"][b, i] = int(weighty[k - 1])
            if k + 1 < weighty.size and edges[t] - x * edges[-1] <= RESOLUTION:
                out["near"][b, i] = int(weighty[k + 1])
            if (b, i) in out["near"]:
                out["near"][b, i] = (out["near"][b, i], (z[out["near"][b, i]] - m) - math.log1p(rest))
            break
    return out


def sum_steps(V):
    """How often a row's fp32 sum is rounded: V / 512 terms a thread in the
    narrowest CTA's chains, then 5 + 4 + 4 joins; each term carries the
    hardware exponential's 2^-22 = 4 u and |x| 3 u of its argument, |x| weighted
    by p at most ln V + 1 < 19."""
    return V / 512 + 13 + 4 + 3 * 19


def check_verify(out, ref, V):
    tokens = out["tokens"].cpu().numpy()
    ref = dict(ref, tokens=ref["tokens"].copy(), logp=ref["logp"].copy())
    for place, (token, logp) in ref["near"].items():
        if tokens[place] == token:
            ref["tokens"][place], ref["logp"][place] = token, logp
    for k in ("tokens", "n_accepted"):
        got = out[k].cpu().numpy()
        assert np.array_equal(got, ref[k]), (k, np.argwhere(got != ref[k])[:4], got[got != ref[k]][:4], ref[k][got != ref[k]][:4])
    n = sum_steps(V)
    for k in ("logp", "lse"):
        got, want = out[k].cpu().numpy().astype(np.float64), ref[k]
        assert np.array_equal(np.isnan(got), np.isnan(want)), k
        fine = np.isfinite(want)
        assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), k
        # the sum's relative error is an absolute one of its logarithm; next to 0 a log-probability
        # is log1p of a small sum and keeps its relative precision; then one rounding
        size = np.minimum(1.0, np.abs(want)) if k == "logp" else 1.0
        tol = n * U * size + 4 * U * np.abs(want) + 2.0 ** -126 * V
        err = np.abs(got - want)
        assert (err[fine] <= np.broadcast_to(tol, err.shape)[fine]).all(), (k, err[fine].max(), np.argwhere(fine & (err > tol))[:4])


def make_logits(shape, V, dtype, seed, ld=None, sd=3.0, sure=True):
    """[..., V] view of a [..., ld] tensor; columns past V hold NaN."""
    per = 4 if dtype == "f32" else 8
    ld = -(-V // per) * per if ld is None else ld
    gen = torch.Generator().manual_seed(seed)
    z = torch.randn((*shape, ld), generator=gen) * sd
    if sure:
        z.view(-1, ld)[::3, V // 2] += 18.0
    z[..., V:] = float("nan")
    return z.to(TORCH[dtype])[..., :V]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()
