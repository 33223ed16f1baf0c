"""The token operators on rows and in calls where one of their steps had gone
wrong or was run by no other test.

Bounds.  u = 2^-24 is half a step of fp32.  A term is 2^x with x = z c + nm, one
fused multiply-add (|x| ln 2 u), or x = (z - m) c where a row is taken by
differences (c, the difference and the product: 3 |x| ln 2 u); the hardware
exponential adds 4 u.  A CTA's T threads each add V / T terms in at most four
chains, then join lanes (5 steps), warps (4) and CTAs (7).  steps(V, T) counts
V / T + 64 roundings, which is what T = 128 threads with one chain need, and
more than four chains of T = 64 do."""
import numpy as np
import pytest
import torch

import oracle
import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api
from _tokens import TORCH, U, check_close, logits, storage
from test_gpu_topk_distill import check, teacher, to_dev

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    rl.build()
    rl.load()


def steps(V, threads=128):
    return V / threads + 64


@pytest.mark.parametrize("R,V", [(40, 60001), (40, 20000), (3, 151936), (2200, 1024)])  # 512, 128, 8 x 128 and 32 threads
@pytest.mark.parametrize("base,temp", [(1e3, 1.0), (1e4, 1.0), (1e3, 0.1), (1e4, 0.1), (1e3, 0.01), (1e4, 0.01), (6e4, 0.01)])
def test_tail_sum_whose_frame_moves(R, V, base, temp):
    """Rows of large logits whose first chunk lies 12 to 14 nats below the
    rest: each warp's sum of the tail passes 2^24 after a few chunks and goes on
    in the frame of a larger maximum, which rounds m c to another number."""
    gen = torch.Generator().manual_seed(int(base) + V)
    first = 16 * (512 if V == 60001 else 32 if V == 1024 else 128)
    per = -(-(-(-V // 16)) // 8) * 16 if R == 3 else V  # a slice of the row
    low = (torch.arange(V) % per) < first
    rows = 11 if R > 1000 else R
    down = 12.0 + 0.25 * (torch.arange(rows) % 9).float()
    z = base + temp * (0.1 * torch.randn((rows, V), generator=gen) - low * down[:, None])
    z = z.float().repeat(-(-R // rows), 1)[:R]
    z = torch.nn.functional.pad(z, (0, -V % 4), value=float("nan"))[:, :V]
    ids, lq = teacher(z[:rows], 8, 3, noise=temp, temperature=temp)
    ids, lq = (t.repeat(-(-R // rows), 1)[:R].contiguous() for t in (ids, lq))
    check(z, "f32", ids, lq, temperature=temp, reverse=0.5)
    check(z, "f32", ids, lq, temperature=temp, tail="renormalise")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,V", [(9, 704), (9, 50000), (60, 60000), (2200, 1000)])
def test_nan_and_infinity_make_their_row_nan_in_the_distillation(dtype, R, V):
    """NaN or +inf at a given token, also one of teacher probability 0, or in
    the tail: that row's loss and gradient are NaN, the others keep their bits."""
    z = to_dev(logits(R, V, dtype, 3 + V))
    ids, lq = (t.to(DEV) for t in teacher(z.cpu(), 6, 3))
    lq[:, 2] = -torch.inf
    lq[:, 3] = -90.0
    bad = z.clone()
    where = {1: ids[1, 0], 2: ids[2, 2], 3: ids[3, 3], 5: (ids[5].max() + 1) % V, 6: ids[6, 2], 7: ids[7, 0]}
    while int(where[5]) in ids[5].tolist():
        where[5] = (where[5] + 1) % V
    for r, e in where.items():
        bad[r, e] = torch.nan if r > 5 else torch.inf
    for kw in (dict(), dict(reverse=1.0), dict(reverse=0.5, temperature=0.7), dict(tail="renormalise")):
        ref, out = (torch_api.topk_distill(x, ids, lq, **kw) for x in (z, bad))
        rows = torch.tensor(sorted(where), device=DEV)
        assert torch.isnan(out["row_loss"][rows]).all() and torch.isnan(out["dlogits"][rows]).all(), kw
        assert torch.isnan(out["loss"])
        rest = torch.ones(R, dtype=torch.bool, device=DEV)
        rest[rows] = False
        assert torch.equal(out["row_loss"][rest], ref["row_loss"][rest])
        assert torch.equal(out["dlogits"][rest], ref["dlogits"][rest])
        assert torch.isfinite(ref["dlogits"].float()).all()


@pytest.mark.parametrize("R", [33, 700, 1300])  # clusters, CTAs of 128 threads, of 64
@pytest.mark.parametrize("base,step", [(-20000.0, 2.0 ** -8), (2.0e7, 2.0)])
def test_certain_rows_taken_by_differences_keep_relative_precision(R, base, step):
    """Log-probabilities next to 0 in rows so far down, or of such large
    logits, that their statistics are taken by differences to the maximum.  The
    terms are at least e^-70: 3 x 70 u each, and the sum's steps."""
    V, rows = 20000, 33
    gen = torch.Generator().manual_seed(3)
    z = torch.round(torch.randn((rows, V), generator=gen) / step) * step
    top = torch.randint(0, V, (rows,), generator=gen)
    z[torch.arange(rows), top] = torch.round((torch.arange(rows).float() + 16.0) / step) * step
    z = (z + base).repeat(-(-R // rows), 1)[:R]
    top = top.repeat(-(-R // rows))[:R]
    out = torch_api.token_logprobs(z.to(DEV), top.to(DEV), want_lse=True)
    ref = oracle.token_logprobs(z[:rows].numpy(), "f32", V, top[:rows, None].numpy())
    bound = (steps(V, 64) + 3 * 70) * U
    rel = np.abs(out["logp"].cpu().numpy()[:rows] / ref["logp"][:, 0] - 1)
    assert rel.max() < bound, rel.max()
    rel = np.abs(out["entropy"].cpu().numpy()[:rows] / ref["entropy"] - 1)
    assert rel.max() < 3 * bound, rel.max()
    for n in ("logp", "entropy", "lse"):
        assert torch.equal(out[n][rows:2 * rows], out[n][:rows][:max(0, R - rows)]), n


@pytest.mark.parametrize("R,V,dtype", [
    (4000, 60000, "bf16"),   # rows dealt out, against CTAs of a fixed share
    (3000, 9000, "f16"),     # CTAs of 64 threads
    (700, 30000, "f32"),
    (74, 40000, "bf16")])    # clusters
def test_rows_with_banned_tokens_keep_their_bits_wherever_they_stand(R, V, dtype):
    """A row with -inf gives the same bits first or last in the batch, after
    rows with -inf or without, in every call."""
    gen = torch.Generator(device=DEV).manual_seed(R)
    z = torch.empty((R, V), dtype=torch.float32, device=DEV).normal_(0.0, 2.0, generator=gen).to(TORCH[dtype])
    some = torch.rand(R, device=DEV, generator=gen)
    at = torch.randint(0, V, (R,), device=DEV, generator=gen)
    one = (some < 0.2).nonzero()[:, 0]
    z[one, at[one]] = -torch.inf
    z[(some > 0.9).nonzero()[:, 0], V // 3:] = -torch.inf
    z[((some > 0.5) & (some < 0.52)).nonzero()[:, 0], 1::2] = -torch.inf
    z[(some > 0.97).nonzero()[:, 0], 7] = torch.nan
    ids = torch.randint(0, V // 3, (R,), device=DEV, generator=gen)
    ref = torch_api.token_logprobs(z, ids, k=5, want_lse=True)
    bits = lambda t: t.view(torch.int32) if t.dtype == torch.float32 else t  # noqa: E731
    for _ in range(3):
        out = torch_api.token_logprobs(z, ids, k=5, want_lse=True)
        for n in ref:
            assert torch.equal(bits(out[n]), bits(ref[n])), n
    back = torch_api.token_logprobs(z.flip(0).contiguous(), ids.flip(0).contiguous(), k=5, want_lse=True)
    for n in ref:
        assert torch.equal(bits(back[n].flip(0)), bits(ref[n])), n
    cut = {4000: 800, 3000: 1500, 700: 350, 74: 74}[R]
    for a in range(0, R, cut):
        part = torch_api.token_logprobs(z[a:a + cut], ids[a:a + cut], k=5, want_lse=True)
        for n in ref:
            assert torch.equal(bits(part[n]), bits(ref[n][a:a + cut])), (n, a)


@pytest.mark.parametrize("R", [20, 700, 1300])
def test_certain_rows_with_banned_tokens_keep_relative_precision(R):
    """One token far above the others, and tokens that cannot occur, in rows
    after rows without.  Terms of at least e^-60."""
    V, rows = 20000, 20
    gen = torch.Generator().manual_seed(3)
    z = torch.randn((rows, V), generator=gen)
    top = torch.randint(0, V // 2, (rows,), generator=gen)
    z[torch.arange(rows), top] = torch.arange(rows).float() + 16.0
    z = z.repeat(-(-R // rows), 1)[:R]
    top = top.repeat(-(-R // rows))[:R]
    z[R - rows:, V - 1 - 700 * (torch.arange(rows) % 3)] = -torch.inf
    out = torch_api.token_logprobs(z.to(DEV), top.to(DEV))
    ref = oracle.token_logprobs(z[R - rows:].numpy(), "f32", V, top[R - rows:, None].numpy())
    bound = (steps(V, 64) + 60) * U
    assert np.abs(out["logp"].cpu().numpy()[R - rows:] / ref["logp"][:, 0] - 1).max() < bound
    assert np.abs(out["entropy"].cpu().numpy()[R - rows:] / ref["entropy"] - 1).max() < 3 * bound


@pytest.mark.parametrize("R,V,K", [(60, 1000, 2), (60, 1000, 5), (48, 70000, 64), (3, 140000, 128), (2200, 700, 33)])
def test_teacher_whose_tail_is_the_rest_of_a_sum_next_to_one(R, V, K):
    """Given probabilities of ordinary size that leave a tail of 2^-22 to 2^-12,
    under a student who gives the tail half: ln q_t, in the reverse divergence
    and its gradient, has the relative error of 1 - sum q.  Each q is formed to
    2^-34 of itself and the sum in fp64, so that error is 2^-34 / q_t."""
    g = np.random.default_rng(R + K)
    tail = 2.0 ** -(12.0 + np.arange(R) % 11)
    q = g.dirichlet(np.full(K, 2.0), R) * (1.0 - tail[:, None])
    lq = torch.from_numpy(np.log(q).astype(np.float32))
    ids = torch.from_numpy(np.stack([g.permutation(V)[:K] for _ in range(R)]))
    z = torch.from_numpy(g.normal(0, 1, (R, V)).astype(np.float32))
    z.scatter_add_(1, ids, torch.full((R, K), float(np.log(V / K))))
    qt = 1.0 - np.exp(lq.double().numpy()).sum(1)
    assert 2.0 ** -24 < qt.min() and qt.max() < 2.0 ** -11
    zd = torch.nn.functional.pad(z, (0, -V % 4)).to(DEV)[:, :V]
    for reverse in (1.0, 0.5):
        out = torch_api.topk_distill(zd, ids.to(DEV), lq.to(DEV), reverse=reverse, norm=1.0)
        ref = oracle.topk_distill(z.numpy(), "f32", V, ids.numpy(), lq.numpy(), reverse=reverse, norm=1.0)
        n = 3 * (steps(V) + 64) * U
        check_close("row_loss", out["row_loss"].cpu(), ref["row_loss"], 2.0 ** -34 / qt + n * ref["size_row"])
        lp = np.abs(ref["lp"])
        check_close("dlogits", out["dlogits"].cpu(), ref["dlogits"],
                    2 * 2.0 ** -34 / qt[:, None] * np.exp(-lp) + (n + 4 * lp * U) * ref["size"])


def test_distill_wrapper_under_another_stream():
    """Forward and backward under a busy side stream: the bits of the current
    stream's gradient, read there after the side stream has been waited for."""
    z = logits(64, 32000, "bf16", 12, sure=False).to(DEV).contiguous()
    ids, lq = (t.to(DEV) for t in teacher(z.cpu(), 8, 3))
    ref = torch_api.topk_distill(z, ids, lq)["dlogits"]
    side = torch.cuda.Stream(DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        leaf = z.clone().requires_grad_()
        torch.cuda._sleep(20_000_000)
        grad = torch.autograd.grad(torch_api.FusedTopkDistill.apply(leaf, ids, lq), leaf)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(grad, ref)


def half_step(x, dtype):
    """Half a step of the 16-bit type at x (normal numbers)."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -14)))
    return 2.0 ** (e - (11 if dtype == "f16" else 8))


def test_gradient_factor_in_the_exponent_at_its_limit():
    """Logits near -706 and tail gradients up to 2^15: the exponent's offset passes
    1024, where it would keep 13 bits after the point.  Beside the output's own
    rounding, p_v's error: at most 20 u for x and its exponential, the offset's
    rounding (2^-15 ln 2 = 363 u) and the row's sum."""
    R, V = 1500, 504  # 13 values a row
    gen = torch.Generator().manual_seed(5)
    z = (-708.5 + 0.5 * torch.randint(-6, 7, (R, V), generator=gen)).half()
    ids = teacher(z, 4, 3)[0]
    lq = torch.log(torch.tensor([0.3, 0.25, 0.25, 0.16])).repeat(R, 1)   # q_t / p_t is small: no cancellation
    weight = torch.rand(R, generator=gen) * 0.5 + 0.5
    kw = dict(grad_scale=2.0 ** 21, norm=1.0)
    out = torch_api.topk_distill(to_dev(z), ids.to(DEV), lq.to(DEV), weight=weight.to(DEV), **kw)
    ref = oracle.topk_distill(storage(z), "f16", V, ids.numpy(), lq.numpy(), weight=weight.numpy(), **kw)
    tail = np.ones((R, V), bool)
    np.put_along_axis(tail, ids.numpy(), False, 1)   # the given tokens' gradients do not fit fp16
    d, size = ref["dlogits"][tail], ref["size"][tail]
    assert 2.0 ** 8 < np.median(np.abs(d)) and 2.0 ** 14 < np.abs(d).max() < 60000
    tol = half_step(d, "f16") * (1 + 2.0 ** -9) + (363 + 20 + 3 * steps(V)) * U * size
    check_close("dlogits", out["dlogits"].cpu().numpy()[tail], d, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,V", [(5, 100), (45, 70000), (3, 140000), (2200, 1000)])
def test_tails_of_almost_no_mass_under_a_large_loss_scale(dtype, R, V):
    """The student's tail holds e^-60 to e^-100 of its mass, the gradient is
    scaled by 65536: s q_t / p_t passes what fp32 holds, the tail's gradients s
    q_t p_v / max(p_t, 2^-126) do not.  Relative errors: x = (z - m) c of up to
    160 ln 2, three roundings, two exponentials, and the row's sum."""
    z = torch.zeros((R, V))
    gap = torch.tensor([60.0, 85.0, 87.5, 90.0, 100.0]).repeat(-(-R // 5))[:R]
    given = torch.arange(R) % V
    z[torch.arange(R), given] = gap + float(np.log(V))
    z = z + torch.randint(-2, 3, (R, V), generator=torch.Generator().manual_seed(1)) * 0.25
    z = z.to(TORCH[dtype])
    ids = torch.stack([given, (given + 3) % V], 1)
    lq = torch.log(torch.tensor([[0.5, 0.2]])).repeat(R, 1)
    kw = dict(grad_scale=65536.0, norm=1.0)
    out = torch_api.topk_distill(to_dev(torch.nn.functional.pad(z, (0, -V % 8))[:, :V]), ids.to(DEV), lq.to(DEV), **kw)
    ref = oracle.topk_distill(storage(z), dtype, V, ids.numpy(), lq.numpy(), **kw)
    d, got = ref["dlogits"], oracle.decode(storage(out["dlogits"]), dtype)
    tail = np.ones((R, V), bool)
    np.put_along_axis(tail, ids.numpy(), False, 1)
    assert np.abs(d[tail]).max() < 60000
    half = {"f32": 1.0, "bf16": 2.0 ** 16, "f16": 2.0 ** 13}[dtype] * U
    rel = half + (3 * 160 + 16 + 3 * steps(V)) * U
    tol = rel * np.abs(d[tail]) + {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}[dtype]
    check_close("tail", got[tail], d[tail], tol)
    check_close("row_loss", out["row_loss"].cpu(), ref["row_loss"], (3 * 160 + 16 + 3 * steps(V)) * U * ref["size_row"])


def test_gradients_beside_the_logits_in_one_buffer():
    """dlogits may begin where the logits' last row ends, and may lie in the
    columns beside them; tensors that share elements are refused."""
    R, V, ld = 6, 992, 1000
    buf = torch.randn(2 * R * ld, device=DEV).bfloat16()
    z = torch.as_strided(buf, (R, V), (ld, 1), 8)
    after = torch.as_strided(buf, (R, V), (ld, 1), R * ld)
    before = torch.as_strided(buf, (R, V), (ld, 1), R * ld + 8)  # z0 follows it
    ids = torch.randint(0, V, (R,), device=DEV)
    one = torch.ones(R, device=DEV)
    tid, tlq = (t.to(DEV) for t in teacher(z.cpu(), 4, 3))
    wide = torch.empty((R, 2 * 1024), dtype=torch.bfloat16, device=DEV)
    wide[:, :V] = z

    def both(x, d):
        lse = torch_api.token_logprobs(x, ids, want_lse=True)["lse"]
        a = torch_api.token_logprobs_backward(x, ids, one, lse, dlogits=d).clone()
        return a, torch_api.topk_distill(x, tid, tlq, dlogits=d)["dlogits"].clone()

    ref = both(z, "new")
    for x, d in ((z, after), (wide[:, :V], wide[:, 1024:1024 + V])):
        for a, b in zip(both(x, d), ref):
            assert torch.equal(a, b)
    wide[:, 1024:1024 + V] = z
    for a, b in zip(both(wide[:, 1024:1024 + V], wide[:, :V]), ref):
        assert torch.equal(a, b)
    lse = torch_api.token_logprobs(z, want_lse=True)["lse"]
    for off in (0, 16, 16 + ld, 8 + 2 * ld, R * ld - 8):
        d = torch.as_strided(buf, (R, V), (ld, 1), off)
        with pytest.raises(rl.RlLossError):
            torch_api.token_logprobs_backward(z, ids, one, lse, dlogits=d)
        with pytest.raises(rl.RlLossError):
            torch_api.topk_distill(z, tid, tlq, dlogits=d)
    d = torch.as_strided(buf, (R, V), (ld, 1), 0)
    with pytest.raises(rl.RlLossError):
        torch_api.topk_distill(before, tid, tlq, dlogits=torch.as_strided(buf, (R, V), (ld, 1), R * ld))


def test_gradient_of_no_given_tokens():
    """ids of shape [R, 0] have log-probabilities of shape [R, 0], whose
    gradient is zero; the entropy's stays."""
    z = logits(5, 512, "bf16", 33, sure=False).to(DEV).contiguous()
    none = torch.empty((5, 0), dtype=torch.int64, device=DEV)
    leaf = z.clone().requires_grad_()
    logp, ent = torch_api.TokenLogprobs.apply(leaf, none)
    assert logp.shape == (5, 0)
    logp.sum().backward()
    assert leaf.grad is not None and (leaf.grad == 0).all()
    leaf.grad = None
    logp, ent = torch_api.TokenLogprobs.apply(leaf, none)
    (logp.sum() + ent.sum()).backward()
    out = torch_api.token_logprobs(z, want_lse=True)
    one = torch.ones(5, device=DEV)
    assert torch.equal(leaf.grad, torch_api.token_logprobs_backward(z, None, None, out["lse"], out["entropy"], one))
    got = torch_api.token_logprobs_backward(z, none, torch.empty((5, 0), device=DEV), out["lse"], dlogits=z)
    assert got.data_ptr() == z.data_ptr() and (z == 0).all()
    with pytest.raises(rl.RlLossError):
        torch_api.token_logprobs_backward(z, None, None, out["lse"])


def test_overwritten_logits_are_not_used_by_an_earlier_backward():
    """A gradient written over the logits counts as a change in place: an
    autograd graph that has kept them refuses its backward pass."""
    z = logits(6, 512, "bf16", 33, sure=False).to(DEV).contiguous()
    ids = torch.randint(0, 512, (6,), device=DEV)
    tid, tlq = (t.to(DEV) for t in teacher(z.cpu(), 4, 3))
    one = torch.ones(6, device=DEV)
    lse = torch_api.token_logprobs(z, want_lse=True)["lse"]
    for over in (lambda x: torch_api.topk_distill(x, tid, tlq, dlogits=x),
                 lambda x: torch_api.token_logprobs_backward(x, ids, one, lse, dlogits=x)):
        leaf = z.clone().requires_grad_()
        logp, _ = torch_api.TokenLogprobs.apply(leaf, ids)
        over(leaf.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            logp.sum().backward()
    with torch.inference_mode():
        x = z.clone()
        assert torch.equal(torch_api.topk_distill(x, tid, tlq, dlogits=x)["dlogits"], torch_api.topk_distill(z, tid, tlq)["dlogits"])


@pytest.mark.parametrize("R,V,dtype,K", [
    (1, 1, "f32", 1), (40, 60001, "bf16", 20), (70, 20000, "f32", 9), (5, 100000, "f16", 64), (2300, 1000, "bf16", 16),
    (700, 300, "f16", 8)])
@pytest.mark.parametrize("kw", [dict(reverse=0.5, temperature=0.8), dict(tail="renormalise")], ids=["bucket", "renormalise"])
def test_loss_without_gradient(R, V, dtype, K, kw):
    """dlogits=None: the same losses and record, bit for bit, as with the
    gradient, within the oracle's bounds; row_loss=None leaves them as well."""
    z = logits(R, V, dtype, R + V)
    ids, lq = teacher(z, K, 3)
    gen = torch.Generator().manual_seed(9)
    if R > 4:
        kw = dict(kw, mask=(torch.arange(R) % 5 != 3).to(torch.uint8), weight=torch.rand(R, generator=gen) + 0.5)
    with_grad, _, _ = check(z, dtype, ids, lq, grad_scale=float(R) if dtype == "f16" else 1.0, **kw)
    kw = {n: t.to(DEV) if torch.is_tensor(t) else t for n, t in kw.items()}
    zd = to_dev(z)
    keep = zd.clone()
    ws = torch_api.new_distill_workspace(DEV)
    for row in ("new", None):
        out = torch_api.topk_distill(zd, ids.to(DEV), lq.to(DEV), dlogits=None, row_loss=row, workspace=ws, **kw)
        assert out["dlogits"] is None and torch.equal(out["loss"], with_grad["loss"])
        assert torch.equal(out["stats"], with_grad["stats"])
        if row:
            assert torch.equal(out["row_loss"], with_grad["row_loss"])
        else:
            assert out["row_loss"] is None
    assert torch.equal(zd.nan_to_num(7.0), keep.nan_to_num(7.0))


def reach(keys, k, threads):
    """How many keys (unique, larger wins) reach the bound of the exact search:
    the k-th largest of its buckets' maxima.  Key i is thread i % threads', in
    its even or odd block; below 2 threads buckets, neighbouring lanes share one."""
    nb = 32 if k <= 16 else 64 if k <= 32 else 128 if k <= 64 else 256
    i = np.arange(keys.size)
    thread, odd = i % threads, (i // threads) & 1
    bucket = 2 * thread + odd if nb == 2 * threads else thread // (threads // nb)
    best = np.full(nb, -1, np.int64)
    np.maximum.at(best, bucket, keys)
    bound = np.sort(best)[-k]
    return int((keys >= max(bound, 0)).sum())


def place_keys(values):
    """Unique keys in the order of (value, lower place first)."""
    order = np.lexsort((-np.arange(values.size), values))
    keys = np.empty(values.size, np.int64)
    keys[order] = np.arange(values.size)
    return keys


@pytest.mark.parametrize("dtype,R,V,k,threads,lanes", [
    ("bf16", 20, 1000, 32, 128, 48), ("f16", 20, 1000, 64, 128, 40), ("f32", 20, 1000, 64, 128, 40),
    ("bf16", 20, 4000, 128, 128, 50), ("f32", 20, 2040, 128, 128, 50),
    ("bf16", 1300, 1000, 32, 64, 24), ("f32", 1300, 1000, 64, 64, 20), ("f16", 1300, 2000, 64, 64, 20)])
def test_exact_search_over_elements_that_raises_its_bound(dtype, R, V, k, threads, lanes):
    """No more pieces than alternatives, the large values on few threads: more
    than 256 elements reach the search's first bound."""
    assert -(-V // (16 if dtype == "f32" else 32)) <= k
    at = torch.arange(V)
    z = logits(8, V, dtype, V + k, sure=False)
    z += torch.where(at % threads < lanes, 20.0, 0.0).to(z.dtype)
    z[1] = torch.where(at % threads < lanes, 1.0, 0.0)    # all of them tied
    z[2, V // 2:] = -torch.inf
    for r in (0, 1, 3, 7):
        assert reach(place_keys(z[r].double().numpy()), k, threads) > 256
    rows = torch.arange(R) % 8
    out = torch_api.token_logprobs(to_dev(torch.nn.functional.pad(z, (0, -V % 8))[:, :V])[rows.to(DEV)].contiguous(), k=k)
    ref = oracle.token_logprobs(storage(z), dtype, V, None, None, k)
    ids, lp = out["topk_ids"].cpu().numpy(), out["topk_logp"].cpu().numpy()
    assert np.array_equal(ids, ref["topk_ids"][rows.numpy()])
    want = ref["topk_logp"][rows.numpy()]
    check_close("topk_logp", lp, want, (steps(V, 64) + 3 * 40) * U * (1 + np.abs(np.where(np.isfinite(want), want, 0))))


@pytest.mark.parametrize("dtype,V,k", [("bf16", 200000, 60), ("f16", 150000, 16), ("f32", 100000, 100)])
def test_exact_search_over_pieces_that_raises_its_bound(dtype, V, k):
    """Long rows, one CTA each, with hundreds of tied pieces on 10 threads: the
    lists of the fast search overflow, and so does the exact search's first."""
    R, per = 320, 16 if dtype == "f32" else 32
    piece = torch.arange(V) // per
    z = logits(4, V, dtype, 77, sure=False).clamp_(-9.0, 9.0)
    z = torch.where(piece % 128 < 10, torch.full((), 10.0, dtype=z.dtype), z)
    z[1] = torch.where(piece % 128 < 10, 1.0, 0.0).to(z.dtype)
    z[2] = torch.where(piece % 128 < 10, z[2] + at_random(V, z.dtype), z[2])
    tops = torch.nn.functional.pad(z.float(), (0, -V % per), value=-99.0).view(4, -1, per).amax(2)
    for r in (0, 1):
        assert reach(place_keys(tops[r].double().numpy()), k, 128) > 256
    rows = torch.arange(R) % 4
    out = torch_api.token_logprobs(to_dev(z)[rows.to(DEV)].contiguous(), k=k)
    ref = oracle.token_logprobs(storage(z), dtype, V, None, None, k)
    assert np.array_equal(out["topk_ids"].cpu().numpy(), ref["topk_ids"][rows.numpy()])
    want = ref["topk_logp"][rows.numpy()]
    check_close("topk_logp", out["topk_logp"].cpu(), want, (steps(V) + 3 * 40) * U * (1 + np.abs(want)))


def at_random(V, dtype):
    return (torch.rand(V, generator=torch.Generator().manual_seed(2)) * 8.0).to(dtype)


def test_bindings_of_the_c_entry_points():
    """The functions that forward to the C entry points, with tensors and with
    addresses, give the bits of the torch layer."""
    R, V, k = 7, 1000, 5
    z = logits(R, V, "bf16", 3, sure=False).to(DEV).contiguous()
    ids = torch.randint(0, V, (R, 2), device=DEV)
    mask = (torch.arange(R, device=DEV) != 3).to(torch.uint8)
    ref = torch_api.token_logprobs(z, ids, mask=mask, k=k, temperature=0.9, want_lse=True)
    f32 = lambda *s: torch.empty(s, device=DEV)  # noqa: E731
    logp, ent, lse, top, top_lp = f32(R, 2), f32(R), f32(R), torch.empty((R, k), dtype=torch.int64, device=DEV), f32(R, k)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    rl.rl_token_logprobs(z, "bf16", R, V, V, ids, 2, mask, 0.9, k, logp, ent, lse.data_ptr(), top, top_lp, st)
    for n, t in dict(logp=logp, entropy=ent, lse=lse, topk_ids=top, topk_logp=top_lp).items():
        assert torch.equal(t, ref[n]), n
    g, h, dz = torch.randn((R, 2), device=DEV), torch.randn(R, device=DEV), torch.empty_like(z)
    rl.rl_token_logprobs_bwd(z, rl.RL_BF16, R, V, V, ids, 2, mask, 0.9, lse, ent, g, h, dz, st, torch.cuda.current_stream())
    assert torch.equal(dz, torch_api.token_logprobs_backward(z, ids, g, lse, ent, h, mask, 0.9))
    tid, tlq = (t.to(DEV) for t in teacher(z.cpu(), 4, 3))
    out = torch_api.topk_distill(z, tid, tlq, mask=mask)
    d = rl.rl_topk_distill_desc_init()
    ws, stats = torch_api.new_distill_workspace(DEV), torch.empty(rl.DISTILL_STATS_BYTES, dtype=torch.uint8, device=DEV)
    d.logits, d.R, d.V, d.ld, d.K = z.data_ptr(), R, V, V, 4
    d.teacher_ids, d.teacher_logp, d.mask = tid.data_ptr(), tlq.data_ptr(), mask.data_ptr()
    d.dlogits, d.stats_dev, d.workspace, d.workspace_bytes = dz.data_ptr(), stats.data_ptr(), ws.data_ptr(), ws.numel()
    rl.rl_topk_distill_fwd_bwd(d)
    assert torch.equal(dz, out["dlogits"]) and torch.equal(stats, out["stats"])
    assert rl.distill_stats_from_bytes(stats.cpu().numpy().tobytes())["n_rows"] == R - 1 and int(st.item()) == 0
    for call in (lambda: rl.rl_token_logprobs(z, "bf16", R, V, V, None, 1, None, 1.0, 0, None, ent, None, None, None),
                 lambda: rl.rl_token_logprobs_bwd(z, "bf16", R, V, V, None, 0, None, 1.0, lse, None, None, None, dz)):
        with pytest.raises(rl.RlLossError):
            call()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_longest_rows(dtype):
    """Rows of 2^26 - 3 logits, in clusters: log-probabilities, entropy, their
    gradient, and the distillation, against fp64 sums.  An element's term is
    added in one of 8 x 512 chains (8 x 128 x 4), 2^14 roundings, and a given
    token's log-probability carries the sum's error."""
    V, R, K = 2 ** 26 - 3, 2, 6
    gen = torch.Generator(device=DEV).manual_seed(4)
    full = torch.empty((R, 2 ** 26), dtype=torch.float32, device=DEV).normal_(0.0, 2.0, generator=gen).to(TORCH[dtype])
    z = full[:, :V]
    ids = torch.tensor([[0, V - 1, 12345678], [V - 1, 1, 40000000]], device=DEV)
    out = torch_api.token_logprobs(z, ids, want_lse=True)
    x = z.double()
    m = x.amax(1, keepdim=True)
    lse = m[:, 0] + (x - m).exp_().sum(1).log()
    lp = x.sub_(lse[:, None])
    p = lp.exp()
    H = -(p * lp).sum(1)
    bound = (2 ** 14 + 64 + 3 * 40) * U
    check_close("lse", out["lse"].cpu(), lse.cpu(), bound + 2 * U * np.abs(lse.cpu().numpy()))
    check_close("logp", out["logp"].cpu(), lp.gather(1, ids).cpu(), bound + 4 * U * 40)
    check_close("entropy", out["entropy"].cpu(), H.cpu(), 3 * bound * (1 + H.cpu().numpy()))
    g, h = torch.randn((R, 3), device=DEV, generator=gen), torch.randn(R, device=DEV, generator=gen)
    got = torch_api.token_logprobs_backward(z, ids, g, out["lse"], out["entropy"], h)
    off = (out["lse"].double() - lse)[:, None]            # the gradient is formed with the rounded lse and entropy
    want = -(p * torch.exp(-off)) * (g.double().sum(1, keepdim=True) + h.double()[:, None] * (lp - off + out["entropy"].double()[:, None]))
    size = (p * (g.abs().double().sum(1, keepdim=True) + h.abs().double()[:, None] * (lp.abs() + 40))).scatter_add_(1, ids, g.abs().double())
    want.scatter_add_(1, ids, g.double())
    half = 2.0 ** -8 if dtype == "bf16" else U
    err = (got.double() - want).abs()
    assert bool((err <= half * want.abs() * 1.001 + (4 * 40 + 144) * U * size + 2.0 ** -126).all())
    del got, want, size, err
    tid = torch.tensor([[5, V - 1, 77, 1 << 20, 1 << 25, -1], [0, 31, 32, 33, V - 2, V - 1]], device=DEV)
    tlq = torch.log_softmax(torch.randn((R, K + 1), device=DEV, generator=gen), 1)[:, :K].contiguous()
    q = torch.where(tid >= 0, tlq.double().exp(), 0.0)
    at = tid.clamp(min=0)
    pt = 1.0 - torch.where(tid >= 0, p.gather(1, at), 0.0).sum(1)
    qt = 1.0 - q.sum(1)
    F = torch.where(tid >= 0, q * (tlq.double() - lp.gather(1, at)), 0.0).sum(1) + qt * (qt.log() - pt.log())
    d = torch_api.topk_distill(z, tid, tlq, norm=1.0)
    check_close("row_loss", d["row_loss"].cpu(), F.cpu(), 3 * bound * (1 + 40))
    slope = (1.0 - qt / pt)[:, None]
    want = p * slope
    for r in range(R):
        for j in range(K):
            if tid[r, j] >= 0:
                want[r, tid[r, j]] = p[r, tid[r, j]] - q[r, j]
    size = (p * (1.0 + qt / pt)[:, None]).scatter_add_(1, at, q)
    err = (d["dlogits"].double() - want).abs_()
    assert bool((err <= half * want.abs() * 1.001 + 3 * bound * size + 2.0 ** -126).all())
