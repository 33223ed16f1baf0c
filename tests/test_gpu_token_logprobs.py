"""rl_token_logprobs and rl_token_logprobs_bwd on the GPU against the fp64
oracle: every row and element, at the sizes, masks and values where the
kernels take another path; the bounds are derived in _tokens.py."""
import numpy as np
import pytest
import torch

import oracle
import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api
from _tokens import TORCH, check_close, check_gradient, check_logprobs, logits, storage

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    rl.build()
    rl.load()


def ref_of(z, dtype, ids=None, mask=None, k=0, temperature=1.0):
    i = None if ids is None else ids.cpu().numpy().reshape(z.shape[0], -1)
    return oracle.token_logprobs(storage(z), dtype, z.shape[1], i, None if mask is None else mask.cpu().numpy(), k,
                                 temperature)


def run(z, ids=None, mask=None, k=0, temperature=1.0, **kw):
    # the padding columns go along: to() of a view would pack the rows
    full = torch.empty((z.shape[0], z.stride(0)), dtype=z.dtype).fill_(float("nan"))
    full[:, :z.shape[1]] = z
    zd = full.to(DEV)[:, :z.shape[1]]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch_api.token_logprobs(zd, None if ids is None else ids.to(DEV), mask=None if mask is None else mask.to(DEV),
                                   k=k, temperature=temperature, want_lse=True, status=st, **kw)
    torch.cuda.synchronize()
    return zd, out, int(st.item())


CASES = [
    # R, V, dtype, k, n_ids, temperature
    (1, 1, "f32", 1, 1, 1.0),
    (3, 2, "bf16", 2, 1, 1.0),
    (5, 33, "f16", 5, 3, 1.0),            # one piece and one element
    (7, 1000, "bf16", 20, 1, 1.0),
    (4, 1023, "f32", 128, 2, 0.7),
    (9, 8192, "f16", 64, 1, 1.0),         # the last size whose elements are searched directly
    (6, 8193, "bf16", 64, 1, 1.0),        # the first that searches pieces first
    (3, 8193, "f32", 17, 1, 2.0),
    (5, 32001, "f16", 128, 16, 1.0),
    (300, 4099, "bf16", 8, 1, 1.0),
    (2, 50257, "f32", 33, 4, 1.0),
    (3, 151936, "bf16", 20, 1, 1.0),
    (2, 151936, "f16", 0, 128, 0.5),
    (700, 500, "f32", 3, 1, 1.0),         # more rows than CTAs
    (2, 262144, "bf16", 128, 1, 1.0),
    (2, 300007, "bf16", 50, 1, 1.0),
    (1, 1 << 20, "f32", 20, 1, 1.0),      # the longest row that can be searched
    (160, 300000, "bf16", 20, 1, 1.0),    # rows that need two CTAs, more of them than clusters
    (70, 40000, "f16", 9, 2, 1.0),        # clusters of 4
    (39, 20000, "f32", 100, 2, 1.0),
    (20, 9000, "bf16", 30, 1, 1.0),       # fewer chunks than CTAs of the largest cluster
    (310, 70000, "bf16", 0, 1, 1.0),
]


@pytest.mark.parametrize("R,V,dtype,k,n,temp", CASES)
def test_forward(R, V, dtype, k, n, temp):
    z = logits(R, V, dtype, 100 + R + V)
    ids = torch.from_numpy(np.random.default_rng(V + R).integers(0, V, (R, n)))
    ids[:, 0] = z.float().argmax(1)
    if n == 1:
        ids = ids[:, 0].contiguous()
    _, out, st = run(z, ids, None, k, temp)
    assert st == 0
    check_logprobs(out, ref_of(z, dtype, ids, None, k, temp), V, temp)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,k", [(700, 9), (20000, 100)])
def test_ties_go_to_the_lower_id(dtype, V, k):
    """Few distinct values, a constant row, sorted rows, and large values packed
    where one thread's keys are."""
    g = np.random.default_rng(V)
    z = torch.from_numpy(g.integers(-3, 4, (6, V + (-V % 8))).astype(np.float32)).to(TORCH[dtype])[:, :V]
    z[1] = 0.25
    z[2] = torch.linspace(-20, 20, V)
    z[3] = torch.linspace(20, -20, V)
    z[4] = -1.0
    z[4, :: 512] = 2.0  # one thread in 16 holds them all
    z[5] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)  # -0 = +0
    _, out, st = run(z, None, None, k)
    assert st == 0
    check_logprobs(out, ref_of(z, dtype, None, None, k), V)


@pytest.mark.parametrize("dtype,V,per", [("bf16", 200000, 32), ("f16", 260000, 32), ("f32", 130000, 16)])
def test_large_values_on_few_threads(dtype, V, per):
    """Every large value lies in the pieces of 20 of the 256 threads, so that
    the bound taken from the threads' maxima lets hundreds of pieces through
    and has to be raised."""
    z = logits(3, V, dtype, 77, sure=False)
    piece = torch.arange(V) // per
    z += torch.where(piece % 256 < 20, 10.0, 0.0).to(z.dtype)
    z[2] = torch.where(piece % 256 < 20, 1.0, 0.0)      # all of them tied
    _, out, st = run(z, None, None, 60)
    assert st == 0
    check_logprobs(out, ref_of(z, dtype, None, None, 60), V)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_banned_tokens_and_rows_with_nothing_left(dtype):
    """-inf and the type's lowest value in part of a row and in all of it; rows
    with fewer possible tokens than alternatives asked for."""
    V, k = 9000, 12
    low = torch.finfo(TORCH[dtype]).min
    z = logits(8, V, dtype, 5, sure=False)
    z[0, 100:] = -torch.inf            # 100 tokens left
    z[1, :] = -torch.inf
    z[1, 4000] = 1.5                   # one token left: probability 1
    z[2, :] = -torch.inf               # nothing left
    z[3, :] = low                      # the type's lowest everywhere: uniform
    z[4, 5:] = low
    z[5, :] = -torch.inf
    z[5, [7, 70]] = low                # two tokens left, at the lowest value
    z[6, ::2] = -torch.inf
    ids = torch.tensor([[0, 8000]] * 8)
    ids[1, 0] = 4000
    ids[5, 0] = 70
    _, out, st = run(z, ids, None, k)
    assert st == 0
    ref = ref_of(z, dtype, ids, None, k)
    check_logprobs(out, ref, V)
    assert out["logp"][1, 0].item() == 0.0 and out["entropy"][1].item() == 0.0
    assert abs(out["logp"][3, 0].item() + np.log(V)) < 1e-5
    assert np.isnan(out["entropy"][2].item()) and out["lse"][2].item() == -np.inf
    assert out["topk_ids"][2].tolist() == list(range(k))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_infinity_stay_in_their_row(dtype):
    V = 3000
    z = logits(6, V, dtype, 6)
    z[1, 17] = torch.nan
    z[1, 2999] = torch.nan
    z[3, 5] = torch.inf
    ids = torch.tensor([3, 3, 3, 5, 3, 3])
    _, out, st = run(z, ids, None, 4)
    assert st == 0
    ref = ref_of(z, dtype, ids, None, 4)
    good = [0, 2, 4, 5]
    check_logprobs({n: out[n][good] for n in ("logp", "entropy", "lse", "topk_ids", "topk_logp")},
                   {n: ref[n][good] for n in ref}, V)
    for r in (1, 3):
        assert torch.isnan(out["logp"][r]).all() and torch.isnan(out["entropy"][r])
    assert out["topk_ids"][1].tolist()[:2] == [17, 2999] and out["topk_ids"][3, 0].item() == 5


def test_masked_rows_are_not_read():
    V = 5000
    z = logits(40, V, "bf16", 8)
    mask = torch.from_numpy((np.arange(40) % 3 != 1).astype(np.uint8))
    z[mask == 0] = torch.nan
    ids = torch.randint(0, V, (40, 2), generator=torch.Generator().manual_seed(1))
    ids[mask == 0] = 10 ** 12
    for m in (mask, mask.bool(), torch.zeros(40, dtype=torch.uint8)):
        _, out, st = run(z, ids, m, 7)
        assert st == 0
        check_logprobs(out, ref_of(z, "bf16", ids, m, 7), V)


def test_id_out_of_range():
    V = 640
    z = logits(5, V, "f32", 9)
    ids = torch.tensor([[1, 2], [V, 3], [-1, 4], [5, 2 ** 40], [0, V - 1]])
    _, out, st = run(z, ids)
    assert st == rl.RL_DEVERR_ID_RANGE
    ref = ref_of(z, "f32", ids)
    check_logprobs(out, ref, V)
    assert np.isnan(out["logp"].cpu().numpy()[[1, 2, 3], [0, 0, 1]]).all()


def test_certain_rows_keep_relative_precision():
    """Log-probabilities next to 0 (one token 8 to 40 above the others)."""
    V = 32000
    z = torch.randn((33, V), generator=torch.Generator().manual_seed(3))
    top = torch.randint(0, V, (33,), generator=torch.Generator().manual_seed(4))
    z[torch.arange(33), top] = torch.arange(33).float() + 14.0
    _, out, _ = run(z, top, None, 1)
    ref = ref_of(z, "f32", top, None, 1)
    rel = np.abs(out["logp"].cpu().numpy() / ref["logp"][:, 0] - 1)
    assert rel.max() < (V / 512 + 64) * 2.0 ** -24
    rel = np.abs(out["entropy"].cpu().numpy() / ref["entropy"] - 1)
    assert rel.max() < 3 * (V / 512 + 64) * 2.0 ** -24


def bwd(z, dtype, ids, dlogp, dent, mask=None, temperature=1.0, inplace=False):
    zd, out, _ = run(z, ids, mask, 0, temperature)
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    src = zd.clone() if not inplace else zd
    got = torch_api.token_logprobs_backward(zd, to(ids), to(dlogp), out["lse"], out["entropy"] if dent is not None else None,
                                            to(dent), mask=to(mask), temperature=temperature,
                                            dlogits=zd if inplace else "new", status=st)
    torch.cuda.synchronize()
    if not inplace:
        assert torch.equal(zd.nan_to_num(7.0), src.nan_to_num(7.0))
    i = None if ids is None else ids.numpy().reshape(z.shape[0], -1)
    g = None if dlogp is None else dlogp.numpy().reshape(z.shape[0], -1)
    ref = oracle.token_logprobs_bwd(storage(z), dtype, z.shape[1], i, g, out["lse"].cpu().numpy(),
                                    out["entropy"].cpu().numpy() if dent is not None else None,
                                    None if dent is None else dent.numpy(), None if mask is None else mask.numpy(), temperature)
    return got, ref, int(st.item())


@pytest.mark.parametrize("R,V,dtype,n,ent,temp,inplace", [
    (1, 1, "f32", 1, True, 1.0, False),
    (1, 9, "bf16", 0, True, 1.0, False),
    (5, 1000, "f32", 1, True, 0.7, False),
    (7, 1001, "bf16", 1, False, 1.0, True),
    (3, 32001, "f16", 16, True, 1.0, False),
    (2, 151936, "bf16", 1, True, 1.0, False),
    (900, 300, "f16", 3, True, 2.0, True),
    (2, 70001, "f32", 128, True, 1.0, False),
])
def test_backward(R, V, dtype, n, ent, temp, inplace):
    z = logits(R, V, dtype, 7 * R + V)
    gen = torch.Generator().manual_seed(R + V)
    ids = torch.randint(0, V, (R, n), generator=gen) if n else None
    if n > 2:
        ids[:, 1] = ids[:, 0]      # the same token twice: its gradients add up
    dlogp = torch.randn((R, n), generator=gen) if n else None
    dent = torch.randn(R, generator=gen) if ent else None
    mask = (torch.arange(R) % 4 != 2).to(torch.uint8) if R > 4 else None
    got, (d, size, lp), st = bwd(z, dtype, ids, dlogp, dent, mask, temp, inplace)
    assert st == 0
    check_gradient(got, dtype, d, size, lp, temp)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
def test_backward_with_banned_tokens(dtype):
    z = logits(6, 2000, dtype, 21, sure=False)
    z[:, 100:1500] = -torch.inf
    z[4, :] = torch.finfo(TORCH[dtype]).min
    z[5, :] = -torch.inf
    ids = torch.tensor([[1, 200]] * 6)
    gen = torch.Generator().manual_seed(2)
    got, (d, size, lp), st = bwd(z, dtype, ids, torch.randn((6, 2), generator=gen), torch.randn(6, generator=gen))
    assert st == 0 and torch.isnan(got[5]).all()
    check_gradient(got[:5], dtype, d[:5], size[:5], lp[:5])
    assert (got[:4, 300:1500] == 0).all()


def test_backward_id_out_of_range_makes_its_row_nan():
    z = logits(3, 640, "f32", 9)
    ids = torch.tensor([[1], [640], [3]])
    zd, out, _ = run(z, ids)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = torch_api.token_logprobs_backward(zd, ids.to(DEV), torch.ones((3, 1), device=DEV), out["lse"], status=st)
    assert int(st.item()) == rl.RL_DEVERR_ID_RANGE
    assert torch.isnan(got[1]).all() and torch.isfinite(got[[0, 2]]).all()


def test_autograd_against_differences():
    """The wrapper's gradient against central differences of the oracle's
    log-probabilities and entropy: truncation is h^2 / 6 times a third
    derivative of at most 1 + 6 ln V, rounding 2^-52 / h."""
    R, V, h = 4, 37, 1e-4
    z = logits(R, 40, "f32", 31, sure=False)[:, :V]
    ids = torch.randint(0, V, (R, 3), generator=torch.Generator().manual_seed(5))
    gl, ge = torch.randn((R, 3)), torch.randn(R)
    leaf = z.to(DEV).contiguous()
    leaf = torch.empty((R, 40), device=DEV)[:, :V].copy_(z.to(DEV)).requires_grad_()
    logp, ent = torch_api.TokenLogprobs.apply(leaf, ids.to(DEV), None, 0.8)
    ((logp * gl.to(DEV)).sum() + (ent * ge.to(DEV)).sum()).backward()
    got = leaf.grad.cpu().numpy().astype(np.float64)
    x = z.numpy().astype(np.float64)

    def f(a):
        o = oracle.token_logprobs(a, "f64", V, ids.numpy(), None, 0, 0.8)
        return (o["logp"] * gl.numpy()).sum() + (o["entropy"] * ge.numpy()).sum()

    for r in range(R):
        for v in range(V):
            a, b = x.copy(), x.copy()
            a[r, v] += h
            b[r, v] -= h
            num = (f(a) - f(b)) / (2 * h)
            assert abs(num - got[r, v]) < 1e-5 * (1 + abs(num)), (r, v, num, got[r, v])


def test_autograd_one_output_used_and_expanded_gradient():
    z = logits(6, 512, "bf16", 33)
    ids = torch.randint(0, 512, (6,), generator=torch.Generator().manual_seed(5)).to(DEV)
    leaf = z.to(DEV).contiguous().requires_grad_()
    logp, _ = torch_api.TokenLogprobs.apply(leaf, ids)
    logp.sum().backward()      # the incoming gradient is an expanded scalar
    a = leaf.grad.clone()
    leaf.grad = None
    _, ent = torch_api.TokenLogprobs.apply(leaf, ids)
    ent.sum().backward()
    b = leaf.grad
    out = torch_api.token_logprobs(leaf.detach(), ids, want_lse=True)
    one = torch.ones(6, device=DEV)
    assert torch.equal(a, torch_api.token_logprobs_backward(leaf.detach(), ids, one, out["lse"]))
    assert torch.equal(b, torch_api.token_logprobs_backward(leaf.detach(), None, None, out["lse"], out["entropy"], one))


def test_two_streams_and_a_captured_graph():
    """Calls on two streams at once and a replayed graph give the bits of a plain call."""
    V, k = 40000, 20
    z = [logits(64, V, "bf16", 40 + i).to(DEV).contiguous() for i in range(2)]
    ids = torch.randint(0, V, (64,), generator=torch.Generator().manual_seed(5)).to(DEV)
    ref = [torch_api.token_logprobs(x, ids, k=k, want_lse=True) for x in z]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    outs = [[torch_api.token_logprobs(z[i], ids, k=k, want_lse=True, stream=streams[i]) for i in range(2)] for _ in range(4)]
    torch.cuda.synchronize()
    for o in outs:
        for i in range(2):
            for n in ref[i]:
                assert torch.equal(o[i][n], ref[i][n]), n
    buf = z[0].clone()
    dl = torch.randn(64, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = torch_api.token_logprobs(buf, ids, k=k, want_lse=True)
        d = torch_api.token_logprobs_backward(buf, ids, dl, o["lse"])
    for i in (1, 0):
        buf.copy_(z[i])
        g.replay()
        torch.cuda.synchronize()
        for n in ref[i]:
            assert torch.equal(o[n], ref[i][n]), n
        assert torch.equal(d, torch_api.token_logprobs_backward(z[i], ids, dl, ref[i]["lse"]))


def test_agrees_with_the_policy_loss_kernel():
    """The fused loss's log-probability and entropy of the same logits, within
    both kernels' bounds (the loss kernel's is 2e-3 absolute)."""
    R, V = 24, 32000
    z = logits(R, V, "f16", 50).to(DEV).contiguous()
    ids = torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(5)).to(DEV)
    loss = torch_api.policy_loss(z, ids, torch.ones(R, dtype=torch.uint8, device=DEV), torch.ones(1, device=DEV), 1, R)
    out = torch_api.token_logprobs(z, ids)
    assert (out["logp"] - loss["logp"]).abs().max() < 2.1e-3
    assert (out["entropy"] - loss["entropy"]).abs().max() < 2.1e-3


def test_empty():
    z = torch.empty((0, 64), device=DEV)
    out = torch_api.token_logprobs(z, torch.empty(0, dtype=torch.int64, device=DEV), k=3, want_lse=True)
    assert out["logp"].shape == (0,) and out["topk_ids"].shape == (0, 3)
    assert torch_api.token_logprobs_backward(z, torch.empty(0, dtype=torch.int64, device=DEV),
                                             torch.empty(0, device=DEV), out["lse"]).shape == (0, 64)


def test_wrapper_refusals():
    z = logits(4, 64, "f32", 1).to(DEV).contiguous()
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    bad = [dict(logits=z.double()), dict(logits=z.cpu()), dict(logits=z.t()), dict(logits=z[0]), dict(ids=ids.int()),
           dict(ids=ids[:3]), dict(ids=ids.cpu()), dict(ids=ids.repeat(2)[::2]), dict(mask=torch.ones(3, dtype=torch.bool, device=DEV)),
           dict(mask=torch.ones(4, device=DEV)), dict(ids=ids[:, None, None])]
    for b in bad:
        with pytest.raises(ValueError):
            torch_api.token_logprobs(**{**dict(logits=z, ids=ids), **b})
    with pytest.raises(rl.RlLossError):
        torch_api.token_logprobs(z, ids, k=65)
    with pytest.raises(rl.RlLossError):
        torch_api.token_logprobs(z, ids, temperature=0.0)
    lse = torch.zeros(4, device=DEV)
    for b in (dict(dlogp=None), dict(dlogp=torch.zeros(4, device=DEV).half()), dict(lse=lse[:2]), dict(dlogits=z.half()),
              dict(entropy=lse.double()), dict(dlogits=torch.empty((4, 72), device=DEV)[:, :64])):
        with pytest.raises(ValueError):
            torch_api.token_logprobs_backward(**{**dict(logits=z, ids=ids, dlogp=lse, lse=lse), **b})
    with pytest.raises(rl.RlLossError):
        torch_api.token_logprobs_backward(z, ids, lse, lse, entropy=lse)


@pytest.mark.parametrize("dtype,low", [("bf16", -1e30), ("f32", -1e9), ("bf16", -1e4), ("f32", -20000.0), ("f16", -60000.0)])
@pytest.mark.parametrize("entropy", [True, False])
def test_masks_of_large_negative_numbers(dtype, low, entropy):
    """Tokens ruled out by a large finite number: in whole pieces at the start,
    scattered, everywhere but one token, everywhere."""
    V, k = 6000, 9
    z = logits(5, V, dtype, 51, sure=False)
    z[0, :3000] = low
    z[1, ::3] = low
    z[2, :] = low
    z[2, 4567] = -3.0
    z[3, :] = low
    z[4, 100:] = low
    ids = torch.tensor([[5, 5000], [0, 1], [4567, 1], [0, 1], [0, 5999]])
    for temp in (1.0, 0.01, 100.0):
        _, out, st = run(z, ids, None, k, temp, want_entropy=entropy)
        assert st == 0
        check_logprobs(out, ref_of(z, dtype, ids, None, k, temp), V, temp)


def test_logits_of_large_size():
    """Maxima up to the type's largest: log-probabilities are differences."""
    z = logits(6, 3000, "f32", 52, sure=False)
    for r, c in enumerate((1e4, -1e5, 1e7, -1e8, 1e30, 3e38)):
        z[r] = c + torch.zeros(3000)
        z[r, 11] = c * (1 - 2 ** -20) if c > 0 else c * (1 + 2 ** -20)
        z[r, 1000:1010] = torch.nextafter(torch.tensor(c), torch.tensor(-3e38))
    ids = torch.tensor([[11, 1000]] * 6)
    _, out, st = run(z, ids, None, 5)
    assert st == 0
    check_logprobs(out, ref_of(z, "f32", ids, None, 5), 3000)


@pytest.mark.parametrize("V,dtype,k,n", [
    (1, "bf16", 1, 1), (9, "f32", 9, 1), (31, "f16", 16, 64), (1000, "bf16", 17, 1), (2047, "f16", 64, 2),
    (2049, "f32", 33, 1), (4100, "bf16", 1, 1), (20000, "f16", 16, 1), (20001, "bf16", 0, 3),
    (2500, "bf16", 65, 1), (2500, "bf16", 8, 65)])
def test_many_short_rows(V, dtype, k, n):
    """Enough short rows for the smaller CTAs, on both sides of their limits on
    alternatives and ids (64 threads: V / 256 terms a chain, within sum_steps
    up to V = 24,000)."""
    R = 1300
    z = logits(R, V, dtype, 9 * V + k)
    g = np.random.default_rng(V)
    ids = torch.from_numpy(g.integers(0, V, (R, n)))
    mask = torch.from_numpy((g.random(R) < 0.8).astype(np.uint8))
    z[mask == 0] = float("nan")
    if V > 100:
        z[5, 3:] = -torch.inf  # fewer tokens than alternatives
        z[6] = 0.5             # ties everywhere
    mask[5] = mask[6] = 1
    z[mask == 0] = float("nan")
    _, out, st = run(z, ids, mask, k)
    assert st == 0
    ref = ref_of(z, dtype, ids, mask, k)
    ref = {key: None if v is None else np.asarray(v) for key, v in ref.items()}
    check_logprobs({key: v.reshape(R, n) if key == "logp" else v for key, v in out.items()}, ref, V)


def test_a_minus_infinity_after_rows_without():
    """The first -inf a CTA meets is in its second row or later, in one warp's
    share of it."""
    V = 9000
    for R in (1300, 4000):  # CTAs of 64 threads; rows of several rounds
        z = logits(R, V, "bf16", 11, sure=False)
        z[R // 2::3, 4000] = -torch.inf
        z[-1, ::2] = -torch.inf
        _, out, st = run(z, None, None, 3)
        assert st == 0
        check_logprobs(out, ref_of(z, "bf16", None, None, 3), V)
