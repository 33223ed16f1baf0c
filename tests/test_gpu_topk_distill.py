"""rl_topk_distill_fwd_bwd on the GPU against the fp64 oracle: the loss, its
means, every row's loss and every gradient element, and the operators together
as a training step uses them.  Bounds are those of _tokens.py; a row's loss is
a sum of terms of sizes (size_row), each with its log-probability's error."""
import numpy as np
import pytest
import torch

import oracle
import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api
from _tokens import HALF_STEP, TINY, TORCH, U, check_close, logits, storage, sum_steps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    rl.build()
    rl.load()


def to_dev(z):
    full = torch.empty((z.shape[0], z.stride(0)), dtype=z.dtype).fill_(float("nan"))
    full[:, :z.shape[1]] = z
    return full.to(DEV)[:, :z.shape[1]]


def teacher(z, K, seed, noise=1.0, temperature=1.0):
    """The top K of a noisy copy of the logits."""
    gen = torch.Generator().manual_seed(seed)
    t = (z.float() + noise * torch.randn(z.shape, generator=gen)) / temperature
    lp = torch.log_softmax(t.double(), 1)
    top, ids = lp.topk(K, 1)
    return ids, top.float()


def tolerances(ref, dtype, V):
    """A gradient element is p_v times the row's slope (or a given token's sum
    of such terms), rounded once.  The hardware exponential flushes results
    below 2^-126 to 0, so p_v also has an absolute error of up to 2^-126 (its
    argument is that of a maximum-1 scale): slope * 2^-126, which is seen only
    where the tail's mass is itself near 2^-126 and the slope q_t / p_t is large."""
    n = sum_steps(V) + 64
    with np.errstate(invalid="ignore"):
        lp = np.where(np.isfinite(ref["lp"]), np.abs(ref["lp"]), 0.0)
        rel = (4 * lp + 3 * n) * U
        grad = HALF_STEP[dtype] * np.abs(ref["dlogits"]) * 1.01 + rel * np.where(np.isfinite(ref["size"]), ref["size"], 0) + TINY[dtype]
        grad = grad + 2.0 ** -126 * ref["slope"][:, None]
    row = 3 * n * U * np.where(np.isfinite(ref["size_row"]), ref["size_row"], 0) + U * np.abs(ref["row_loss"])
    return row, np.where(np.isfinite(grad), grad, 0)


def check(z, dtype, ids, lq, inplace=False, **kw):
    zd = to_dev(z)
    host = {n: t.cpu().numpy() if torch.is_tensor(t) else t for n, t in kw.items()}
    ref = oracle.topk_distill(storage(z), dtype, z.shape[1], ids.numpy(), lq.numpy(), **host)
    dev = {n: t.to(DEV) if torch.is_tensor(t) else t for n, t in kw.items()}
    out = torch_api.topk_distill(zd, ids.to(DEV), lq.to(DEV), dlogits=zd if inplace else "new", **dev)
    torch.cuda.synchronize()
    st = torch_api.read_distill_stats(out["stats"])
    row_tol, grad_tol = tolerances(ref, dtype, z.shape[1])
    check_close("row_loss", out["row_loss"].cpu(), ref["row_loss"], row_tol)
    check_close("dlogits", oracle.decode(storage(out["dlogits"]), dtype), ref["dlogits"], grad_tol)
    if np.isfinite(ref["loss"]):
        n = max(1.0, kw.get("norm", 0.0) or ref["n_rows"])
        assert abs(st["loss"] - ref["loss"]) <= row_tol.sum() / n + 1e-15
        assert abs(out["loss"].item() - ref["loss"]) <= row_tol.sum() / n + 2 * U * abs(ref["loss"])
        # a row's divergence is a mean of |ln p| + |ln q| + 1 < 100 here
        lim = 3 * (sum_steps(z.shape[1]) + 64) * U * 100
        for name in ("forward_kl", "reverse_kl", "teacher_tail", "student_tail"):
            same = st[name] == ref[name]  # two infinities have no difference
            assert same or abs(st[name] - ref[name]) <= lim * max(1.0, abs(ref[name])), (name, st[name], ref[name])
    assert st["n_rows"] == ref["n_rows"] and st["device_error"] == 0
    return out, ref, st


@pytest.mark.parametrize("R,V,dtype,K,reverse,temp,tail", [
    (1, 2, "f32", 1, 0.0, 1.0, "bucket"),
    (1, 1, "bf16", 1, 0.5, 1.0, "bucket"),           # every token given: no tail
    (3, 24, "f32", 24, 0.5, 1.0, "bucket"),
    (5, 33, "f16", 5, 1.0, 1.0, "bucket"),
    (7, 1000, "bf16", 20, 0.0, 1.0, "bucket"),
    (9, 1023, "f32", 128, 0.3, 0.7, "bucket"),
    (6, 4097, "f16", 64, 0.0, 2.0, "renormalise"),
    (4, 32001, "bf16", 33, 0.5, 2.0, "bucket"),
    (2, 151936, "bf16", 64, 0.0, 1.0, "bucket"),
    (2, 151936, "f16", 127, 1.0, 1.0, "bucket"),
    (2, 140003, "f32", 100, 0.5, 1.0, "bucket"),     # pieces that share a place of the table
    (700, 300, "bf16", 8, 0.0, 1.0, "bucket"),       # more rows than CTAs
    (650, 777, "f32", 3, 0.5, 1.0, "bucket"),
])
def test_against_the_oracle(R, V, dtype, K, reverse, temp, tail):
    z = logits(R, V, dtype, 300 + R + V, sd=2.0)
    ids, lq = teacher(z, K, R + V, temperature=temp)
    gen = torch.Generator().manual_seed(9)
    kw = {}
    if R > 4:
        kw["mask"] = (torch.arange(R) % 5 != 3).to(torch.uint8)
        kw["weight"] = torch.rand(R, generator=gen) + 0.5
    check(z, dtype, ids, lq, reverse=reverse, temperature=temp, tail=tail, grad_scale=float(R) if dtype == "f16" else 1.0, **kw)


def test_in_place_with_norm_and_bool_mask():
    z = logits(30, 5000, "bf16", 4)
    ids, lq = teacher(z, 16, 3)
    check(z, "bf16", ids, lq, inplace=True, mask=torch.arange(30) % 2 == 0, norm=7.5, grad_scale=3.0)


def test_every_given_token_in_one_piece():
    """All entries in the same 64 bytes, on a row's last piece, and in an order that is not sorted."""
    V = 2000 + 17
    z = logits(4, V, "bf16", 8)
    ids = torch.stack([torch.arange(16) + 64, torch.arange(V - 16, V), torch.arange(63, 47, -1), torch.arange(16) * 125 + 1])
    lq = torch.log_softmax(torch.randn((4, 17), generator=torch.Generator().manual_seed(1)), 1)[:, :16].contiguous()
    check(z, "bf16", ids, lq, reverse=0.5)


def test_empty_entries_and_teachers_of_zero_mass():
    z = logits(5, 600, "f32", 10)
    ids, lq = teacher(z, 6, 3)
    ids[1, 2:] = -1
    lq[1, 2:] = float("nan")       # what an empty entry holds is not read into anything
    ids[2] = -1
    lq[3, 4] = -torch.inf          # a given token of probability 0
    for tail in ("bucket", "renormalise"):
        out, ref, _ = check(z, "f32", ids, lq, tail=tail)
        assert out["row_loss"][2].item() == 0.0 and (out["dlogits"][2] == 0).all()
    check(z, "f32", ids, lq, reverse=1.0)


def test_teacher_that_is_sure_and_student_that_is_sure():
    """1 - sum q below what fp32 log-probabilities can hold, and a tail of the
    student far below its top token."""
    V = 3000
    z = torch.zeros((4, V))
    z[0, 5] = 60.0
    z[1, 5] = 100.0
    z[2, 9] = 30.0
    ids = torch.tensor([[5, 7], [5, 7], [5, 9], [5, 7]])
    lq = torch.tensor([[-1e-7, -17.0], [0.0, -30.0], [-1e-3, -8.0], [-0.6931472, -0.6931472]])
    for reverse in (0.0, 0.5, 1.0):
        check(z, "f32", ids, lq, reverse=reverse)


def test_logits_as_teacher_values_when_renormalised():
    z = logits(6, 900, "bf16", 12)
    gen = torch.Generator().manual_seed(8)
    ids = torch.stack([torch.randperm(900, generator=gen)[:40] for _ in range(6)])
    check(z, "bf16", ids, 200.0 * torch.rand((6, 40), generator=gen), tail="renormalise")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_banned_student_tokens(dtype):
    """-inf logits in the tail and at given tokens; all of the tail; all of a row."""
    V = 1500
    z = logits(6, V, dtype, 14, sd=1.0, sure=False)
    z[:, 700:] = -torch.inf
    ids, lq = teacher(torch.nan_to_num(z.float(), neginf=-30.0), 8, 3)
    z[1, :] = -torch.inf
    z[1, ids[1]] = torch.arange(8).to(z.dtype)       # nothing left in the tail
    check(z[:2], dtype, ids[:2], lq[:2], reverse=0.5)
    # a given token that the student cannot produce: infinite forward divergence, finite gradient
    z[2, ids[2, 0]] = -torch.inf
    out, ref, _ = check(z[2:3], dtype, ids[2:3], lq[2:3])
    assert out["row_loss"].item() == np.inf and torch.isfinite(out["dlogits"]).all()
    check(z[2:3], dtype, ids[2:3], lq[2:3], reverse=1.0)
    z[3, :] = torch.finfo(TORCH[dtype]).min          # the type's lowest everywhere: uniform
    check(z[3:4], dtype, ids[3:4], lq[3:4], reverse=0.5)
    z[4, :] = -torch.inf                              # no distribution
    out = torch_api.topk_distill(to_dev(z[4:]), ids[4:].to(DEV), lq[4:].to(DEV))
    assert torch.isnan(out["row_loss"][0]) and torch.isnan(out["dlogits"][0]).all()
    assert torch.isfinite(out["row_loss"][1]) and torch.isfinite(out["dlogits"][1].float()).all()


def test_bad_entries_make_their_row_nan():
    z = logits(5, 640, "f32", 9)
    ids, lq = teacher(z, 4, 3)
    good = ids.clone()
    ids[1, 2] = 640
    ids[2, 0] = -2
    ids[3, 3] = ids[3, 1]
    out = torch_api.topk_distill(to_dev(z), ids.to(DEV), lq.to(DEV))
    st = torch_api.read_distill_stats(out["stats"])
    assert st["device_error"] == rl.RL_DEVERR_ID_RANGE | rl.RL_DEVERR_ID_REPEAT and np.isnan(st["loss"])
    assert torch.isnan(out["row_loss"][1:4]).all() and torch.isnan(out["dlogits"][1:4]).all()
    ref = torch_api.topk_distill(to_dev(z), good.to(DEV), lq.to(DEV), workspace=out["workspace"])
    for r in (0, 4):
        assert torch.equal(out["dlogits"][r], ref["dlogits"][r]) and out["row_loss"][r] == ref["row_loss"][r]
    assert torch_api.read_distill_stats(ref["stats"])["device_error"] == 0   # the workspace was left ready


def test_masked_rows_are_not_read_and_no_valid_row():
    z = logits(20, 1000, "bf16", 2)
    ids, lq = teacher(z, 5, 3)
    mask = (torch.arange(20) % 3 == 0).to(torch.uint8)
    z[mask == 0] = torch.nan
    ids[mask == 0] = 10 ** 12
    check(z, "bf16", ids, lq, mask=mask)
    out = torch_api.topk_distill(to_dev(z), ids.to(DEV), lq.to(DEV), mask=torch.zeros(20, dtype=torch.uint8, device=DEV))
    st = torch_api.read_distill_stats(out["stats"])
    assert st["loss"] == 0 and st["n_rows"] == 0 and (out["dlogits"] == 0).all() and (out["row_loss"] == 0).all()


def test_columns_past_v_are_left_alone():
    z = to_dev(logits(9, 1001, "bf16", 2, ld=1024))
    ids, lq = teacher(z.cpu(), 5, 3)
    d = torch.full((9, 1024), 7.0, dtype=torch.bfloat16, device=DEV)
    torch_api.topk_distill(z, ids.to(DEV), lq.to(DEV), dlogits=d[:, :1001], mask=(torch.arange(9, device=DEV) != 4))
    assert (d[:, 1001:] == 7).all() and not (d[:, :1001] == 7).any()
    d.fill_(7.0)
    i = torch.zeros(9, dtype=torch.int64, device=DEV)
    out = torch_api.token_logprobs(z, i, want_lse=True)
    torch_api.token_logprobs_backward(z, i, torch.ones(9, device=DEV), out["lse"], dlogits=d[:, :1001],
                                      mask=(torch.arange(9, device=DEV) != 4))
    assert (d[:, 1001:] == 7).all() and not (d[:, :1001] == 7).any()


def test_gradient_against_differences():
    """The kernel's fp32 gradient against central differences of the oracle's loss."""
    R, V, h = 3, 29, 1e-5
    z = logits(R, 32, "f32", 31, sd=1.5, sure=False)[:, :V]
    for kw in (dict(reverse=0.0), dict(reverse=0.6, temperature=1.5), dict(tail="renormalise")):
        ids, lq = teacher(z, 7, 5)
        full = torch.empty((R, 32), device=DEV)[:, :V].copy_(z.to(DEV))
        got = torch_api.topk_distill(full, ids.to(DEV), lq.to(DEV), **kw)["dlogits"].cpu().numpy()
        x = z.numpy().astype(np.float64)
        for r in range(R):
            for v in range(V):
                a, b = x.copy(), x.copy()
                a[r, v] += h
                b[r, v] -= h
                f = [oracle.topk_distill(y, "f64", V, ids.numpy(), lq.numpy(), **kw)["loss"] for y in (a, b)]
                assert abs((f[0] - f[1]) / (2 * h) - got[r, v]) < 2e-6, (kw, r, v)


def test_autograd_wrapper():
    z = logits(12, 2000, "bf16", 12)
    ids, lq = (t.to(DEV) for t in teacher(z, 8, 3))
    leaf = to_dev(z).contiguous().requires_grad_()
    loss = torch_api.FusedTopkDistill.apply(leaf, ids, lq, None, dict(reverse=0.25))
    loss.backward()
    ref = torch_api.topk_distill(leaf.detach(), ids, lq, reverse=0.25)
    assert torch.equal(leaf.grad, ref["dlogits"]) and loss.item() == ref["loss"].item()
    leaf.grad = None
    (2.0 * torch_api.FusedTopkDistill.apply(leaf, ids, lq, None, dict(reverse=0.25))).backward()
    assert torch.equal(leaf.grad, 2 * ref["dlogits"])
    half = leaf.detach().half().requires_grad_()     # a loss scale that does not fit fp16
    (2.0 ** 17 * torch_api.FusedTopkDistill.apply(half, ids, lq, None, dict(grad_scale=2.0 ** -7))).backward()
    ref = torch_api.topk_distill(half.detach(), ids, lq, grad_scale=2.0 ** -7)
    assert torch.equal(half.grad, (ref["dlogits"].float() * 2.0 ** 17).half())


def test_teacher_scoring_then_student_step_as_a_loop_runs_them():
    """token_logprobs of the teacher, topk_distill of the student beside the
    policy loss on the same logits, its gradients added: one captured graph,
    replayed on new logits, gives the bits of the plain calls."""
    B, T, V, K = 2, 16, 8000, 32
    R = B * T
    t_logits, s_logits = (logits(R, V, "bf16", i).to(DEV).contiguous() for i in (60, 61))
    ids = torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(5)).to(DEV)
    mask = (torch.arange(R) % 7 != 2).to(torch.uint8).to(DEV)
    adv = torch.tensor([0.5, -1.0], device=DEV)
    ws, lws = torch_api.new_distill_workspace(DEV), torch_api.new_workspace(R, DEV)

    def step(t, s):
        top = torch_api.token_logprobs(t, ids, mask=mask, k=K)
        old = torch_api.token_logprobs(s, ids, mask=mask, want_entropy=False, want_lse=True)
        dist = torch_api.topk_distill(s, top["topk_ids"], top["topk_logp"], mask=mask, workspace=ws)
        pg = torch_api.policy_loss(s, ids, mask, adv, B, T, logp_old=old["logp"], workspace=lws)
        more = torch_api.token_logprobs_backward(s, ids, old["logp"], old["lse"], mask=mask)
        return dist["dlogits"] + pg["dlogits"] + more, dist["loss"], top["topk_ids"]

    ref = [[x.clone() for x in step(t_logits, s_logits)], [x.clone() for x in step(s_logits, t_logits)]]
    # the parts are the oracle's
    host = oracle.token_logprobs(storage(t_logits), "bf16", V, None, mask.cpu().numpy(), K)
    assert np.array_equal(ref[0][2].cpu().numpy(), host["topk_ids"])
    o = oracle.topk_distill(storage(s_logits), "bf16", V, host["topk_ids"], host["topk_logp"].astype(np.float32), mask=mask.cpu().numpy())
    assert abs(ref[0][1].item() - o["loss"]) < 1e-5 * abs(o["loss"])
    a, b = t_logits.clone(), s_logits.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(a, b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(a, b)
    for i in (1, 0):
        a.copy_((s_logits if i else t_logits))
        b.copy_((t_logits if i else s_logits))
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, ref[i]):
            assert torch.equal(x, y)


def test_repeated_calls_are_bitwise_equal():
    z = to_dev(logits(400, 3333, "bf16", 2))
    ids, lq = (t.to(DEV) for t in teacher(z.cpu(), 16, 3))
    a = torch_api.topk_distill(z, ids, lq, reverse=0.5)
    for _ in range(3):
        b = torch_api.topk_distill(z, ids, lq, reverse=0.5, workspace=a["workspace"])
        assert torch.equal(a["dlogits"].nan_to_num(), b["dlogits"].nan_to_num()) and torch.equal(a["stats"], b["stats"])


def test_wrapper_refusals_and_empty():
    z = logits(4, 64, "f32", 1).to(DEV).contiguous()
    ids = torch.tensor([[0, 1]] * 4, device=DEV)
    lq = torch.full((4, 2), -1.0, device=DEV)
    for b in (dict(teacher_ids=ids.int()), dict(teacher_ids=ids[:3]), dict(teacher_logp=lq.double()), dict(teacher_ids=ids[0]),
              dict(tail="none"), dict(mask=torch.ones(5, dtype=torch.uint8, device=DEV)), dict(weight=torch.ones(4, device=DEV).half()),
              dict(row_loss=torch.ones(3, device=DEV)), dict(dlogits=z.double()), dict(stats=torch.zeros(8, device=DEV)),
              dict(workspace=torch.zeros(1 << 18, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            torch_api.topk_distill(**{**dict(logits=z, teacher_ids=ids, teacher_logp=lq), **b})
    for b in (dict(reverse=1.5), dict(temperature=0.0), dict(reverse=0.5, tail="renormalise"), dict(norm=-1.0),
              dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(rl.RlLossError):
            torch_api.topk_distill(z, ids, lq, **b)
    out = torch_api.topk_distill(z[:0], ids[:0], lq[:0])
    assert torch_api.read_distill_stats(out["stats"])["loss"] == 0 and out["loss"].item() == 0


@pytest.mark.parametrize("dtype,low", [("bf16", -1e30), ("f32", -1e9), ("f32", -20000.0), ("f16", -60000.0)])
def test_masks_of_large_negative_numbers(dtype, low):
    """Student tokens ruled out by a large finite number: half of the tail, all
    of it, the whole row."""
    V = 4000
    z = logits(4, V, dtype, 15, sd=1.0, sure=False)
    ids, lq = teacher(z, 8, 3)
    z[0, :2000] = low
    z[1, :] = low
    z[1, ids[1]] = torch.arange(8).to(z.dtype)
    z[2, :] = low
    z[3, ids[3, :4]] = low
    check(z, dtype, ids, lq, reverse=1.0)
    check(z[:3], dtype, ids[:3], lq[:3], tail="renormalise")


def test_more_rows_than_one_round_of_ctas_long_rows():
    """Long rows (one a SM), masked in runs, more of them than SMs."""
    R, V = 400, 60001
    z = logits(R, V, "bf16", 16, sd=2.0)
    ids, lq = teacher(z, 20, 3)
    mask = ((torch.arange(R) // 37) % 3 != 1).to(torch.uint8)
    zd = to_dev(z)
    out = torch_api.topk_distill(zd, ids.to(DEV), lq.to(DEV), mask=mask.to(DEV), norm=1.0)
    rows = torch.tensor([0, 36, 37, 73, 74, 152, 153, 304, 399])
    ref = oracle.topk_distill(storage(z[rows]), "bf16", V, ids[rows].numpy(), lq[rows].numpy(), mask=mask[rows].numpy(), norm=1.0)
    row_tol, grad_tol = tolerances(ref, "bf16", V)
    check_close("row_loss", out["row_loss"].cpu()[rows], ref["row_loss"], row_tol)
    check_close("dlogits", oracle.decode(storage(out["dlogits"].cpu()[rows]), "bf16"), ref["dlogits"], grad_tol)
    masked = mask == 0
    assert (out["dlogits"].cpu()[masked] == 0).all() and (out["row_loss"].cpu()[masked] == 0).all()
    st = torch_api.read_distill_stats(out["stats"])
    assert st["n_rows"] == int(mask.sum()) and st["device_error"] == 0
    assert abs(st["loss"] - out["row_loss"].double().sum().item()) < 1e-6 * R


@pytest.mark.parametrize("R,V,dtype,K,reverse,inplace", [
    (1, 151936, "bf16", 64, 0.0, False), (3, 70001, "f16", 16, 0.5, True), (17, 40000, "f32", 128, 1.0, True),
    (38, 65537, "bf16", 33, 0.5, False), (75, 33000, "f16", 5, 0.0, True), (130, 20000, "f32", 9, 0.5, False),
    (304, 16400, "bf16", 12, 0.5, True)])
def test_few_rows_share_their_ctas(R, V, dtype, K, reverse, inplace):
    """Clusters of up to 8 CTAs a row, and numbers of rows on both sides of what
    gets clusters; entries at the slices' edges."""
    z = logits(R, V, dtype, R + V)
    ids, lq = teacher(z, K, 3)
    per = 16 if dtype == "f32" else 32
    pieces = -(-V // per)
    edges = [0, V - 1] + [min(V - 1, e) for c in (2, 4, 8) for e in (-(-pieces // c) * per - 1, -(-pieces // c) * per)]
    edges = [e for e in dict.fromkeys(edges) if e not in ids[0].tolist()][:K]
    ids[0, K - len(edges):] = torch.tensor(edges)
    mask = (torch.arange(R) % 6 != 4).to(torch.uint8) if R > 4 else None
    check(z, dtype, ids, lq, inplace=inplace, mask=mask, reverse=reverse)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_few_rows_taken_again(dtype):
    """Rows whose statistics are taken by differences (all tokens at or below
    the floor, or far above the frame) with their gradient written in place of
    the logits, in clusters, between rows that are not."""
    V, R = 40003, 12
    z = logits(R, V, dtype, 8, sure=False)
    low = torch.finfo(TORCH[dtype]).min
    z[1] = low
    z[2, 100:] = -torch.inf
    z[4, :] = -60000.0 if dtype == "f16" else -1e30
    z[4, 39000] = low if dtype == "f16" else -0.99e30
    z[5, :30000] = -torch.inf          # whole slices with nothing
    z[7, 1:] = low
    ids, lq = teacher(z, 6, 3)
    ids[4], ids[1] = torch.arange(6) * 7000, torch.arange(6) * 6000 + 5
    lq = torch.log_softmax(torch.randn(R, 6, generator=torch.Generator().manual_seed(4)), 1) - 0.3
    ids[7], ids[2] = torch.arange(6), torch.arange(6) + 90
    a, _, _ = check(z, dtype, ids, lq)
    b, _, _ = check(z, dtype, ids, lq, inplace=True)
    assert np.array_equal(storage(a["dlogits"]), storage(b["dlogits"]))


@pytest.mark.parametrize("R,V,dtype,K,reverse", [
    (2300, 1, "bf16", 1, 0.0), (2300, 37, "f32", 8, 0.5), (2200, 1000, "bf16", 128, 0.5), (4000, 2048, "f16", 16, 0.0),
    (2200, 1024, "f32", 5, 1.0), (2200, 2049, "bf16", 16, 0.0)])
def test_many_tiny_rows(R, V, dtype, K, reverse):
    """Many rows of at most 4 KB, and one element more."""
    z = logits(R, V, dtype, V)
    ids, lq = teacher(z, K, 3)
    check(z, dtype, ids, lq, mask=(torch.arange(R) % 5 != 2).to(torch.uint8), reverse=reverse)
