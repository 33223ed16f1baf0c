"""Verification and sampling where rows, numbers and shares of the work lie at an edge: draft rows that nearly
equal the target's, low temperatures, log-sum-exps of any size, tokens of almost no probability, numbers next to
a draft's own border, maxima that rise all along a row, and the same sequences by clusters of every size."""
import math

import numpy as np
import pytest
import torch

import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api
from tests._rollout import RESOLUTION, TORCH, U, f64, make_logits

pytestmark = pytest.mark.gpu
DEV = "cuda"
BATCHES = (3, 30, 70, 110, 250, 400)   # clusters of 16, 10, 5, 4, 2 and 1 CTAs on 152 SMs (V = 33,000)


@pytest.fixture(scope="module", autouse=True)
def built():
    rl.build()
    rl.load()


def rows(t, B, n=1):
    """[B, n, V] on the GPU, every row the 1-D ``t``, 16-byte aligned."""
    V, per = t.shape[0], 16 // t.element_size()
    return torch.nn.functional.pad(t, (0, -V % per)).to(DEV).expand(B, n, -1).contiguous()[..., :V]


def softmax(z, T=1.0):
    e = np.exp(z / T - (z / T).max())
    return e / e.sum(), (z / T).max() + math.log(e.sum())


def check_draws(tokens, w, x):
    """The drawn tokens of weights w (of p's total of 1) with uniforms x: the border x W lies in the token's
    interval, to the resolution of its ends (include/rlrollout.h), and the token has a weight."""
    resolution = max(RESOLUTION, w.size * 2.0 ** -52)
    edges = np.cumsum(w)
    at = x * edges[-1]
    assert (tokens >= 0).all()
    assert (w[tokens] > 0).all(), (tokens[w[tokens] <= 0][:4], w[tokens][w[tokens] <= 0][:4])
    off = np.maximum(edges[tokens] - w[tokens] - at, at - edges[tokens])
    assert (off <= resolution).all(), (math.log2(off.max()), tokens[off > resolution][:4])


# ------------------------------------------------------------------ max(p - q, 0)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("beside", [-1e-7, -3e-8, -1e-8, 1e-8, 3e-8, 1e-7])
@pytest.mark.parametrize("B", BATCHES)
def test_draft_that_nearly_equals_the_target(dtype, beside, B):
    """The draft's row is the target's but for a masked tail of mass 2e-7 and one token that it has 300 times as
    often, and everywhere else p / q = 1 + beside: which tokens have p > q is known only once the row's sum is known
    to more than fp32 gives."""
    V = 33000
    z = make_logits((1,), V, dtype, 3, sure=False)[0]
    # without the one token that brings the row's log-sum-exp nearest to `beside` below a float
    e = np.exp(f64(z))
    lq = np.float32(math.log(e.sum()))
    if float(lq) > math.log(e.sum()) + beside:
        lq = np.nextafter(lq, np.float32(-np.inf))
    z[int(np.argmin(np.abs(np.log(e.sum() - e) - (float(lq) - beside))))] = -math.inf
    p, lse = softmax(f64(z))
    assert abs(float(lq) - lse - beside) < 2e-9
    order = np.argsort(p)
    tail = order[:int(np.searchsorted(np.cumsum(p[order]), 2e-7))]
    d = int(order[np.searchsorted(p[order], 1e-9)])
    y = z.clone()
    y[tail] = -math.inf
    y[d] = z[d].float() + math.log(300.0)
    w = np.maximum(p - np.exp(f64(y) - np.float64(lq)), 0.0)
    assert w[d] == 0 and w.sum() > 1e-7
    x = np.random.default_rng(B).random(B)
    u = torch.from_numpy(np.stack([np.full(B, 0.999), x], 1)).to(DEV)
    out = torch_api.verify_drafts(rows(z, B, 2), torch.full((B, 1), d, device=DEV), u, draft_logits=rows(y, B),
                                  draft_lse=torch.full((B, 1), float(lq), device=DEV))
    assert (out["n_accepted"] == 0).all()
    check_draws(out["tokens"][:, 0].cpu().numpy(), w, x)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature,shift", [(1.0, 0.0), (0.7, 0.0), (0.7, 20.0), (0.1, 0.0), (0.1, 3.0), (0.03, 1.0), (0.01, 0.0), (0.01, 0.5), (30.0, 0.0), (100.0, 700.0)])
def test_refused_drafts_next_to_a_border_at_any_temperature(dtype, temperature, shift):
    """Numbers 1.1 to 4 resolutions of p's total to either side of a border of max(p - q, 0), in rows whose
    log-sum-exps lie anywhere."""
    V, T, n, each = 4000, temperature, 24, 20
    gen, rng = torch.Generator().manual_seed(7), np.random.default_rng(1)
    z = (torch.randn((n, V), generator=gen) * 3 * T + shift).to(TORCH[dtype])
    y = (z.float() + torch.randn((n, V), generator=gen) * T).to(TORCH[dtype])
    weights, lqs, xs, ids = [], [], [], []
    for i in range(n):
        p, _ = softmax(f64(z[i]), T)
        q, lse = softmax(f64(y[i]), T)
        lqs.append(np.float32(lse))
        w = np.maximum(p - np.exp(f64(y[i]) / T - np.float64(lqs[-1])), 0.0)
        edges = np.cumsum(w)
        some = rng.choice(np.nonzero(w > 64 * RESOLUTION)[0][:-1], each, replace=False)
        xs.append((edges[some] + rng.uniform(1.1, 4.0, each) * rng.choice([-1.0, 1.0], each) * RESOLUTION) / edges[-1])
        weights.append(w)
        ids.append(int(np.argmax(q - p)))
    u = np.stack([np.full(n * each, 1 - 2.0 ** -53), np.concatenate(xs)], 1)
    spread = lambda t: t.to(DEV)[:, None].expand(n, each, V).reshape(n * each, 1, V)  # noqa: E731
    out = torch_api.verify_drafts(spread(z).expand(-1, 2, V).contiguous(), torch.tensor(ids, device=DEV).repeat_interleave(each)[:, None],
                                  torch.from_numpy(u).to(DEV), draft_logits=spread(y).contiguous(),
                                  draft_lse=torch.tensor(np.array(lqs), device=DEV).repeat_interleave(each)[:, None].contiguous(), temperature=T)
    assert (out["n_accepted"] == 0).all()
    tokens = out["tokens"][:, 0].cpu().numpy().reshape(n, each)
    for i in range(n):
        check_draws(tokens[i], weights[i], xs[i])


@pytest.mark.parametrize("dtype,size,temperature", [
    (dtype, size, T) for dtype, sizes in (("f32", (3e4, 1e6, 1e9, 1e15, 1e36, 3e38)), ("bf16", (3e4, 1e6, 1e15, 1e36)), ("f16", (6e4,))) for size in sizes
    for T in (1.0, 0.5, 2.0 ** -6, 64.0, 0.7, 0.01) if size / T < 3.3e38 and (size < 1e5 or math.log2(T) % 1 == 0)])
@pytest.mark.parametrize("B", [3, 250])
def test_draft_logits_of_any_size(dtype, size, temperature, B):
    """A draft's row of which one token has all: it is refused, and another one is drawn.  The same with every token at
    a very low number: q is 1 everywhere, nothing is left of max(p - q, 0), and the token is drawn from p."""
    V, T = 33000, temperature
    z = make_logits((1,), V, dtype, 11, sure=False)[0]
    z = (z.float() * min(T, 1.0)).to(TORCH[dtype])
    p, _ = softmax(f64(z), T)
    rng = np.random.default_rng(5)
    d, x = int(np.argmax(p)), rng.random(B)
    high, low = torch.zeros(V).to(TORCH[dtype]), torch.full((V,), -size).to(TORCH[dtype])
    high[d] = size
    for row in (high, low):
        lse = np.float32(f64(row)[d] / T)
        with np.errstate(over="ignore"):
            q = np.exp(f64(row) / T - np.float64(lse))
        assert (q[0] < 1e-30 or q[0] > 0.9) and q[d] > 0.9
        w = np.maximum(p - q, 0.0)
        w = w if w.any() else p
        u = torch.from_numpy(np.stack([np.full(B, 1 - 2.0 ** -53), x], 1)).to(DEV)
        out = torch_api.verify_drafts(rows(z, B, 2), torch.full((B, 1), d, device=DEV), u, draft_logits=rows(row, B),
                                      draft_lse=torch.full((B, 1), float(lse), device=DEV), temperature=T)
        assert (out["n_accepted"] == 0).all()
        check_draws(out["tokens"][:, 0].cpu().numpy(), w, x)


@pytest.mark.parametrize("dtype,at", [("f32", 5.0e3), ("f32", -2.0e4), ("f32", 3.0e7), ("f32", 1.0e9), ("f32", -1.0e9), ("bf16", 3.0e4), ("bf16", -3.0e4), ("bf16", 1.0e9), ("f16", 6.0e4), ("f16", -6.0e4)])
@pytest.mark.parametrize("temperature", [1.0, 64.0])
@pytest.mark.parametrize("B", [3, 70, 400])
def test_refused_drafts_of_rows_of_large_numbers(dtype, at, temperature, B):
    """Both rows far from 0, their numbers some steps of the type apart (a temperature that is a power of two: the fp64 form is
    exact); the draft's log-sum-exp is what fp32 holds of it."""
    V, T = 33000, temperature
    base = torch.tensor(at).to(TORCH[dtype])
    step = abs(float(torch.nextafter(base, torch.zeros_like(base)).double() - base.double()))
    gen = torch.Generator().manual_seed(37)
    levels = max(2, int(8 * T / step))
    k = torch.randint(0, levels, (V,), generator=gen)
    far = -1.0 if at > 0 else 1.0     # towards 0 steps do not grow
    z = (base.double() + far * k * step).to(TORCH[dtype])
    y = (base.double() + far * ((k + torch.randint(0, max(2, levels // 6), (V,), generator=gen)) % levels) * step).to(TORCH[dtype])
    p, _ = softmax(f64(z), T)
    lq = np.float32(softmax(f64(y), T)[1])
    with np.errstate(over="ignore"):
        q = np.exp(f64(y) / T - np.float64(lq))
    w = np.maximum(p - q, 0.0)
    w = w if w.any() else p
    d = int(np.argmax(q - p))
    x = np.random.default_rng(B).random(B)
    u = torch.from_numpy(np.stack([np.full(B, 1 - 2.0 ** -53), x], 1)).to(DEV)
    out = torch_api.verify_drafts(rows(z, B, 2), torch.full((B, 1), d, device=DEV), u, draft_logits=rows(y, B),
                                  draft_lse=torch.full((B, 1), float(lq), device=DEV), temperature=T)
    if q[d] * (1 - 2.0 ** -53) < p[d]:
        assert (out["n_accepted"] == 1).all() and (out["tokens"][:, 0] == d).all()
    else:
        assert (out["n_accepted"] == 0).all()
        check_draws(out["tokens"][:, 0].cpu().numpy(), w, x)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 0.1])
@pytest.mark.parametrize("top", [64.0, 64.1234567, 70.0001])
@pytest.mark.parametrize("B", BATCHES)
def test_draft_with_nothing_but_roundings_below_the_target(dtype, temperature, top, B):
    """One token has all but e^-60; the draft's row is the target's but for the refused token, of which it has more: p is
    nowhere above q, but equal to it in every digit, and the token is drawn from p."""
    V, T = 33000, temperature
    z = (make_logits((1,), V, dtype, 51, sure=False)[0].float() * T).clamp(max=10.0 * T).to(TORCH[dtype])
    z[V // 5] = top * T
    y = z.clone()
    y[17] += 0.5 * T
    lq = f64(z)[V // 5] / T
    if float(np.float32(lq)) != lq:
        lq = np.nextafter(np.float32(lq), np.float32(-np.inf)) if float(np.float32(lq)) > lq else np.float32(lq)   # q > p everywhere
    u = torch.from_numpy(np.stack([np.full(B, 0.99), np.random.default_rng(B).random(B)], 1)).to(DEV)
    out = torch_api.verify_drafts(rows(z, B, 2), torch.full((B, 1), 17, device=DEV), u, draft_logits=rows(y, B),
                                  draft_lse=torch.full((B, 1), float(lq), device=DEV), temperature=T)
    assert (out["n_accepted"] == 0).all() and (out["tokens"][:, 0] == V // 5).all()


# ------------------------------------------------------------------ numbers that are none
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("V,B", [(33000, 3), (33000, 70), (33000, 250), (33000, 400), (200000, 3)])
def test_a_row_with_one_number_that_is_none(dtype, value, V, B):
    """Wherever it stands in the row, and whatever stands behind it: no token, no log-probability; in a draft's row the same."""
    z = rows(make_logits((1,), V, dtype, 31)[0], B).clone()
    at = torch.from_numpy(np.random.default_rng(B).integers(0, V, B)).to(DEV)
    at[0], at[1], at[2] = 0, V - 1, V // 2
    one = torch.arange(B, device=DEV)
    clean = z.clone()
    z[one, 0, at] = value
    u = torch.full((B, 1), 0.4, dtype=torch.float64, device=DEV)
    out = torch_api.verify_drafts(z, None, u)
    assert (out["tokens"] == -1).all() and out["logp"].isnan().all() and out["lse"].isnan().all() and (out["n_accepted"] == 0).all()
    # a draft's row with it, where the draft is refused and its row asked
    ids = torch.full((B, 1), 17, device=DEV)
    at[at == 17] = 18
    y = clean.clone()
    y[one, 0, 17] += 9.0
    lse = y[:, 0].double().logsumexp(-1).float()[:, None].contiguous()
    y[one, 0, at] = value
    u2 = torch.full((B, 2), 0.9, dtype=torch.float64, device=DEV)
    out = torch_api.verify_drafts(rows(clean[0, 0], B, 2), ids, u2, draft_logits=y, draft_lse=lse)
    assert (out["tokens"] == -1).all() and out["logp"][:, 0].isnan().all() and (out["n_accepted"] == 0).all()


# ------------------------------------------------------------------ a draft's own test
@pytest.mark.parametrize("temperature,gap", [(1.0, 100.0), (1.0, 700.0), (1.0, 2000.0), (0.1, 9.0), (0.1, 300.0), (0.01, 0.9), (0.01, 5.0), (0.01, 100.0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("numbers", [torch.float32, torch.float64])
def test_drafts_of_almost_no_probability(dtype, temperature, gap, numbers):
    """A draft stays iff u q < p, however small p is: with u = 0 and with q = 0 always."""
    V, T, B = 1000, temperature, 6
    z = (torch.randn(V, generator=torch.Generator().manual_seed(9)) * 0.1 * T).to(TORCH[dtype])
    z[3] = 0.5 * T
    z[7] = 0.5 * T - gap
    y = torch.zeros(V).to(TORCH[dtype])
    y[7] = -math.inf
    log_p = (f64(z)[7] - f64(z).max()) / T - math.log(softmax(f64(z), T)[0].max() ** -1)
    ids = torch.full((B, 1), 7, device=DEV)
    u = torch.full((B, 2), 0.5, dtype=torch.float64)
    u[:, 0] = torch.tensor([0.0, math.exp(max(log_p - 2, -740)), math.exp(max(log_p - 0.01, -740)), math.exp(max(log_p + 0.01, -740)), 1e-3, 1 - 2.0 ** -53],
                           dtype=numbers).clamp(max=1 - 2.0 ** -53)
    x = u[:, 0].numpy()
    stays = (x == 0) | (np.log(np.maximum(x, 5e-324)) < log_p)
    out = torch_api.verify_drafts(rows(z, B, 2), ids, u.to(DEV), temperature=T)
    assert np.array_equal(out["n_accepted"].cpu().numpy(), stays.astype(int))
    logp = out["logp"][:, 0].cpu().numpy()
    assert np.abs(logp[stays] / log_p - 1).max() < 2.0 ** -20
    # q = 0 at the draft
    out = torch_api.verify_drafts(rows(z, B, 2), ids, u.to(DEV), draft_logits=rows(y, B), draft_lse=torch.full((B, 1), math.log(V - 1.0), device=DEV), temperature=T)
    assert (out["n_accepted"] == 1).all()
    # p = 0: refused, whatever u and q
    z[7] = -math.inf
    for kw in (dict(), dict(draft_logits=rows(y, B), draft_lse=torch.full((B, 1), math.log(V - 1.0), device=DEV))):
        out = torch_api.verify_drafts(rows(z, B, 2), ids, u.to(DEV), temperature=T, **kw)
        assert (out["n_accepted"] == 0).all() and (out["tokens"][:, 0] != 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 0.05])
@pytest.mark.parametrize("kind", ["model", "lookup"])
@pytest.mark.parametrize("B", BATCHES)
def test_drafts_next_to_their_own_border(dtype, temperature, kind, B):
    """u within 2^-32 of p / q to either side, by clusters of every size: what stays does not depend on the batch."""
    V, T = 33000, temperature
    z = make_logits((1,), V, dtype, 13, sure=False)[0]
    z = (z.float() * T).to(TORCH[dtype])
    z[100] = 9.0 * T
    p, _ = softmax(f64(z), T)
    y = z.clone()
    y[100] = z[100].float() + 0.75 * T
    q, lse = softmax(f64(y), T)
    lq = np.float32(lse)
    border = p[100] / (math.exp(f64(y)[100] / T - float(lq)) if kind == "model" else 1.0)
    u = np.full((B, 2), 0.3)
    sign = np.where(np.arange(B) % 2 == 0, 1.0, -1.0)
    u[:, 0] = border * (1 + sign * 2.0 ** -32 * (1 + np.arange(B) % 7))
    kw = dict(draft_logits=rows(y, B), draft_lse=torch.full((B, 1), float(lq), device=DEV)) if kind == "model" else {}
    out = torch_api.verify_drafts(rows(z, B, 2), torch.full((B, 1), 100, device=DEV), torch.from_numpy(u).to(DEV), temperature=T, **kw)
    assert np.array_equal(out["n_accepted"].cpu().numpy(), (sign < 0).astype(int))


# ------------------------------------------------------------------ the row's sum
def sum_bound(V):
    """Of a row's fp32 sum, relative, in units of 2^-24, whatever V: a term carries 4 of the hardware exponential and
    2 ln 2 |x| of its argument (the FMA's rounding and c's), |x| weighted by p at most log2 V; 9 additions in a chunk's
    chains, its frame's end and the frame's correction 10 each, 5 joins of lanes, 7 of a part's frame, 9 joins of parts."""
    return 4 + 2 * math.log(2) * math.log2(V) + 9 + 20 + 5 + 7 + 9


def check_sums(z, T=1.0):
    """lse of rows z [n, V] and the log-probabilities of drawn tokens."""
    n, V = z.shape
    per = 16 // z.element_size()
    zd = torch.nn.functional.pad(z, (0, -V % per)).to(DEV)[:, :V]
    out = torch_api.sample_tokens(zd, torch.full((n,), 0.37, dtype=torch.float64, device=DEV), temperature=T)
    x = f64(z) / T
    m = x.max(1)
    e = np.exp(x - m[:, None])
    top = e == 1.0
    log_s = np.log1p(top.sum(1) - 1 + np.where(top, 0.0, e).sum(1))
    tol = (sum_bound(V) + 4 * np.abs(log_s)) * U
    lse, logp = (out[k].cpu().numpy().astype(np.float64) for k in ("lse", "logp"))
    err = np.abs(lse - (m + log_s))
    assert (err <= tol + U * np.abs(m + log_s)).all(), (err / U, sum_bound(V))
    want = x[np.arange(n), out["tokens"].cpu().numpy()] - m - log_s
    err = np.abs(logp - want)
    assert (err <= tol + 2 * U * np.abs(want)).all(), (err / U, sum_bound(V))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,n", [(5, 3), (1000, 3), (33000, 3), (33000, 400), (151936, 4), (151936, 200), (1 << 20, 2), (1 << 22, 1)])
def test_sums_of_long_rows(dtype, V, n):
    check_sums(make_logits((n,), V, dtype, V + n))
    check_sums(make_logits((n,), V, dtype, V + n, sure=False), 0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,n", [(33000, 400), (1 << 20, 2), (1 << 23, 1)])
@pytest.mark.parametrize("rise", [1e-3, 0.01, 0.1, 1.0, 5.0])
@pytest.mark.parametrize("way", [1, -1])
def test_sums_of_rows_that_rise(dtype, V, n, rise, way):
    """The maximum rises by a little from one part of the row to the next."""
    z = torch.linspace(0, rise, V, dtype=torch.float64)
    z = (z if way > 0 else z.flip(0)).to(TORCH[dtype])
    check_sums(z.expand(n, V).contiguous())


@pytest.mark.parametrize("rise", [0.01, 0.5])
def test_sums_of_the_longest_rows_that_rise(rise):
    check_sums(torch.linspace(0, rise, 1 << 26)[None])


@pytest.mark.parametrize("V", [33000, 1 << 20, 1 << 25])
@pytest.mark.parametrize("at", [3.0e7, -2.0e4, 1.0e9])
@pytest.mark.parametrize("T", [1.0, 100.0])
def test_sums_of_rows_taken_by_differences(V, at, T):
    """Rows of large or very low numbers, their sums as those of any other row."""
    step = float(np.spacing(np.float32(abs(at))))
    k = torch.randint(0, max(1, int(8 * T / step)) + 2, (2, V), generator=torch.Generator().manual_seed(1))
    check_sums((at - k.double() * step).float(), T)
    k = torch.arange(V).expand(2, V) * (max(1, int(8 * T / step)) + 2) // V
    check_sums((at + k.double() * step).float(), T)


@pytest.mark.parametrize("dtype,V", [("f32", 1 << 20), ("bf16", 1 << 20), ("f32", 1 << 26)])
@pytest.mark.parametrize("rise", [0.01, 0.5, 2.0])
def test_draws_of_rows_that_rise(dtype, V, rise):
    """Numbers some 2^-22 to 2^-16 of the total to either side of a border, in rows whose maximum rises all along."""
    z = torch.linspace(0, rise, V, dtype=torch.float64).to(TORCH[dtype])
    p, _ = softmax(f64(z))
    n = 200 if V <= 1 << 20 else 12
    edges, rng = np.cumsum(p), np.random.default_rng(3)
    at = rng.integers(0, V - 1, n)
    x = np.clip(edges[at] + 2.0 ** rng.uniform(-22, -16, n) * rng.choice([-1.0, 1.0], n), 0.0, 1 - 2.0 ** -53)
    out = torch_api.verify_drafts(rows(z, n), None, torch.from_numpy(x)[:, None].to(DEV))
    check_draws(out["tokens"][:, 0].cpu().numpy(), p, x)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,B,low", [(V, B, low) for V, B in ((60000, 400), (60000, 70), (151936, 400), (151936, 30)) for low in (-4.7, -9.3, -11.8, -13.1)] +
                         [(1 << 21, 100, -14.1), (1 << 24, 3, -16.3)])
@pytest.mark.parametrize("kind", ["none", "model"])
def test_borders_of_rows_of_equal_numbers(dtype, V, B, low, kind):
    """One token, and all others alike: every addition to the fine sums rounds to the same side.  Numbers 1.1 to 4
    resolutions to either side of a border."""
    z = torch.full((V,), low).to(TORCH[dtype])
    z[V // 3] = 0.0
    p, _ = softmax(f64(z))
    w = p
    if kind == "model":
        y = torch.full((V,), low).to(TORCH[dtype])
        y[V // 2] = max(low + math.log(V), 0.0)     # half of the draft's mass, or more
        lq = np.float32(softmax(f64(y))[1])
        w = np.maximum(p - np.exp(f64(y) - np.float64(lq)), 0.0)
    edges, rng = np.cumsum(w), np.random.default_rng(B)
    # (where the draft has more of every token than the target, all but one: nothing but that one token is drawn)
    some = rng.choice(np.nonzero(w > min(64 * RESOLUTION, w.max()) / 2)[0], B)
    x = np.clip((edges[some] + rng.uniform(1.1, 4.0, B) * rng.choice([-1.0, 1.0], B) * RESOLUTION) / edges[-1], 0, 1 - 2.0 ** -53)
    if kind == "none":
        out = torch_api.verify_drafts(rows(z, B), None, torch.from_numpy(x)[:, None].to(DEV))
    else:
        u = torch.from_numpy(np.stack([np.full(B, 1 - 2.0 ** -53), x], 1)).to(DEV)
        out = torch_api.verify_drafts(rows(z, B, 2), torch.full((B, 1), V // 2, device=DEV), u, draft_logits=rows(y, B),
                                      draft_lse=torch.full((B, 1), float(lq), device=DEV))
        assert (out["n_accepted"] == 0).all()
    check_draws(out["tokens"][:, 0].cpu().numpy(), w, x)


# ------------------------------------------------------------------ clusters of every size
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["none", "model", "lookup"])
def test_the_same_sequences_by_clusters_of_every_size(dtype, kind):
    """Tokens of the same sequences in batches that clusters of 16, 10, 5, 4, 2 and 1 CTAs take, bit for bit, their
    drawn tokens' numbers 2^-32 to 2^-17 of the total from a border of the last row."""
    V, B, G = 33000, max(BATCHES), 0 if kind == "none" else 1
    gen = torch.Generator().manual_seed(17)
    z = make_logits((1,), V, dtype, 19, sure=False)[0]
    p, _ = softmax(f64(z))
    edges, rng = np.cumsum(p), np.random.default_rng(23)
    u = np.random.default_rng(29).random((B, G + 1))
    u[:, G] = np.clip(edges[rng.integers(1, V - 1, B)] + 2.0 ** rng.uniform(-32, -17, B) * rng.choice([-1.0, 1.0], B), 0, 1 - 2.0 ** -53)
    a = dict(target_logits=rows(z, B, G + 1), draft_ids=None, uniforms=torch.from_numpy(u).to(DEV))
    if G:
        y = (z.float() + torch.randn(V, generator=gen) * 0.7).to(z.dtype)
        q, lse = softmax(f64(y))
        a["draft_ids"] = torch.from_numpy(rng.choice(V, (B, 1), p=q)).to(DEV)
        if kind == "model":
            a.update(draft_logits=rows(y, B), draft_lse=torch.full((B, 1), float(np.float32(lse)), device=DEV))
    whole = torch_api.verify_drafts(**a)
    for n in BATCHES:
        for lo in range(0, B - n + 1, max(n, 80)):
            part = torch_api.verify_drafts(**{k: v if v is None else v[lo:lo + n] for k, v in a.items()})
            for k in ("tokens", "n_accepted"):
                assert torch.equal(part[k], whole[k][lo:lo + n]), (n, lo, k)
