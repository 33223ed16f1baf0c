"""The rollout's operators on the GPU against plain fp64 forms of their definitions."""
import math

import numpy as np
import pytest
import torch

import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api
from tests._rollout import RESOLUTION, TORCH, check_verify, f64, logits_ref, make_logits, quantize_ref, verify_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    rl.build()
    rl.load()


# ------------------------------------------------------------------ 8-bit codes
def check_codes(x):
    codes, scale = torch_api.quantize_rows(x)
    want, s = quantize_ref(f64(x))
    got_s = scale.cpu().numpy()
    assert np.array_equal(got_s, s, equal_nan=True), np.argwhere(got_s != s)[:4]
    got = codes.cpu().numpy()
    assert np.array_equal(got, want), (np.argwhere(got != want)[:4], got[got != want][:4], want[got != want][:4])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,D", [(1, 1), (1, 7), (3, 16), (5, 100), (33, 1001), (7, 1024), (4, 2049), (3, 5000), (2, 8193), (2, 40000)])
def test_codes(dtype, R, D):
    x = make_logits((R,), D, dtype, R * 1000 + D, sure=False) * torch.exp(torch.randn(R, 1)).to(TORCH[dtype])
    per = 4 if dtype == "f32" else 8
    room = torch.full((R, -(-D // per) * per + per), float("nan"), dtype=TORCH[dtype])
    room[:, :D] = x
    check_codes(room.to(DEV)[:, :D])


def test_codes_next_to_a_half():
    """Quotients at, and one step from, every half: the exact quotient decides."""
    for top in (127.0, 100.0, 1.0, 3.7e-3, 8.9e5, 2.0 ** -120, 1.3e38):
        s = np.float32(np.float64(np.float32(top)) / 127.0)
        k = np.arange(-127, 127) + 0.5
        near = (k * np.float64(s)).astype(np.float32)
        x = np.concatenate([near, np.nextafter(near, np.float32(np.inf)), np.nextafter(near, np.float32(-np.inf)), [np.float32(top)]])
        x = np.clip(x, -np.float32(top), np.float32(top)).astype(np.float32)
        x = np.pad(x, (0, -x.size % 4))
        check_codes(torch.from_numpy(x)[None].to(DEV))


def test_codes_of_small_rows():
    """Rows of subnormal numbers: scales of few digits, or 0."""
    tiny = 2.0 ** -149
    rows = [[0, 0, 0, 0], [-0.0, 0, -0.0, 0], [tiny, -tiny, 0, 0], [63 * tiny, 5 * tiny, 0, 1 * tiny], [64 * tiny, -64 * tiny, 32 * tiny, 1 * tiny],
            [190 * tiny, -190 * tiny, 120 * tiny, tiny], [2.0 ** -126, 2.0 ** -130, -2.0 ** -140, 0], [2.0 ** -110, 1.5 * 2.0 ** -118, -2.0 ** -117, 0]]
    check_codes(torch.tensor(rows, dtype=torch.float64).float().to(DEV))


def test_codes_of_rows_with_nan_or_infinity():
    x = torch.randn(6, 304)
    x[1, 299] = float("nan")
    x[2, 0] = float("inf")
    x[4, 17] = -float("inf")
    for dtype in ("f32", "bf16", "f16"):
        check_codes(x.to(TORCH[dtype]).to(DEV))


def test_codes_are_written_inside_their_columns():
    x = torch.randn(5, 37, device=DEV)
    x = torch.nn.functional.pad(x, (0, 3))[:, :37]
    room = torch.full((5, 64), 99, dtype=torch.int8, device=DEV)
    scale = torch.full((5,), -1.0, device=DEV)
    codes, s = torch_api.quantize_rows(x, codes=room[:, :37], scale=scale)
    assert codes.data_ptr() == room.data_ptr() and s is scale
    want, ws = quantize_ref(f64(x))
    assert np.array_equal(room[:, :37].cpu().numpy(), want) and np.array_equal(scale.cpu().numpy(), ws)
    assert (room[:, 37:] == 99).all()


# ------------------------------------------------------------------ logits
def int8_inputs(R, D, V, seed, extreme=False):
    gen = np.random.default_rng(seed)
    if extreme:
        h, w = gen.choice(np.array([-128, 127], np.int8), (R, D)), gen.choice(np.array([-128, 127], np.int8), (V, D))
    else:
        h, w = gen.integers(-128, 128, (R, D), dtype=np.int8), gen.integers(-128, 128, (V, D), dtype=np.int8)
    return h, (gen.random(R).astype(np.float32) + 0.1) * 0.01, w, (gen.random(V).astype(np.float32) + 0.1) * 0.01


def to_dev(codes):
    """Codes in rows of a multiple of 16 bytes; what lies behind a row is no zero."""
    R, D = codes.shape
    room = torch.full((R, -(-D // 16) * 16 + 16), 77, dtype=torch.int8)
    room[:, :D] = torch.from_numpy(codes)
    return room.to(DEV)[:, :D]


def check_logits(h, sh, w, sw, dtype, pad=0):
    R, V = h.shape[0], w.shape[0]
    per = 4 if dtype == "f32" else 8
    room = torch.full((R, -(-V // per) * per + pad * per), 7.0, dtype=TORCH[dtype], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.full((rl.rl_lmhead_int8_workspace_size(R, h.shape[1]),), 0xff, dtype=torch.uint8, device=DEV)  # NaN as 16-bit numbers
    out = torch_api.lmhead_logits_int8(to_dev(h), torch.from_numpy(sh).to(DEV), to_dev(w), torch.from_numpy(sw).to(DEV), out=room[:, :V],
                                       status=status, workspace=ws)
    assert status.item() == 0
    want = logits_ref(h, sh, w, sw, dtype)
    got = out.cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    assert same.all(), (torch.nonzero(~same)[:4], got[~same][:4], want[~same][:4])
    assert (room[:, V:] == 7.0).all()
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("R,D,V", [(1, 1, 1), (1, 16, 129), (2, 100, 300), (16, 64, 128), (17, 65, 257), (33, 1024, 1000), (64, 1000, 513), (100, 127, 2000),
                                   (161, 640, 700), (192, 256, 384), (193, 256, 130), (400, 320, 1001), (1000, 96, 257)])
def test_logits(dtype, R, D, V):
    check_logits(*int8_inputs(R, D, V, R + 7 * D + V), dtype, pad=R % 3)


@pytest.mark.parametrize("R,D,V", [(5, 1025, 200), (20, 2048, 300), (130, 2500, 257), (200, 1151, 129), (3, 8192, 140), (2, 131071, 9), (300, 4100, 513)])
def test_logits_of_many_columns(R, D, V):
    """Sums beyond 24 bits are exact too."""
    check_logits(*int8_inputs(R, D, V, D), "f32")
    check_logits(*int8_inputs(R, D, V, D + 1, extreme=True), "f32")


@pytest.mark.parametrize("D", [1023, 1024, 1025, 2048, 4096])
def test_logits_of_the_largest_sums(D):
    h, w = np.full((40, D), -128, np.int8), np.full((150, D), -128, np.int8)
    w[1::2] = 127
    h[3, D // 2:] = 127      # halves that cancel
    h[5, 1::2] = 127
    check_logits(h, np.ones(40, np.float32), w, np.ones(150, np.float32), "f32")


def test_logits_do_not_depend_on_the_batch():
    h, sh, w, sw = int8_inputs(700, 512, 900, 3)
    whole = check_logits(h, sh, w, sw, "f32")
    for lo, n in ((0, 1), (5, 3), (100, 64), (128, 200)):
        assert torch.equal(check_logits(h[lo:lo + n], sh[lo:lo + n], w, sw, "f32"), whole[lo:lo + n])


@pytest.mark.parametrize("R", [1, 16, 50, 64, 90, 100, 128, 150, 160, 176, 192, 300])
def test_logits_of_many_calls_on_end(R):
    """Weights that L2 does not hold, so that tiles land late and in any order: the rings' every
    depth, each call's every bit."""
    D, V, calls = 1024, 151_936, 200
    g = torch.Generator(device=DEV).manual_seed(R)
    h = torch.randint(-128, 128, (R, D), generator=g, dtype=torch.int8, device=DEV)
    w = torch.randint(-128, 128, (V, D), generator=g, dtype=torch.int8, device=DEV)
    sh, sw = (torch.rand(n, generator=g, device=DEV) + 0.5 for n in (R, V))
    want = (h.double() @ w.double().T).float().mul_(sh[:, None]).mul_(sw).bfloat16()  # (sums below 2^24: exact in both)
    status, work = torch.zeros(1, dtype=torch.int32, device=DEV), torch_api.new_int8_workspace(R, D, device=DEV)
    out, wrong = torch.empty_like(want), torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(calls):
        for _ in range(4):
            torch_api.lmhead_logits_int8(h, sh, w, sw, out=out, workspace=work, status=status)
        wrong += (out.view(torch.int16) != want.view(torch.int16)).sum()
        out.zero_()
    assert wrong.item() == 0 and status.item() == 0


def test_logits_scales_that_are_not_numbers():
    h, sh, w, sw = int8_inputs(20, 64, 200, 5)
    sh[3], sh[4], sw[7], sw[9] = np.nan, 0.0, np.inf, np.nan
    h[6] = 0
    check_logits(h, sh, w, sw, "bf16")
    sh[:], sw[:] = 1e30, 1e30     # beyond fp32
    check_logits(h, sh, w, sw, "f16")


# ------------------------------------------------------------------ verification
def run_verify(target, ids, u, draft=None, draft_lse=None, n_draft=None, temperature=1.0):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731

    def strided(t):  # rows stay as far apart as they are
        if t is None:
            return None
        ld = t.stride(1) if t.shape[1] > 1 or t.shape[0] == 1 else t.stride(0)
        whole = torch.as_strided(t, (t.shape[0], t.shape[1], ld), (t.shape[1] * ld, ld, 1)) if ld > t.shape[2] else t
        return whole.to(DEV)[..., :t.shape[2]]

    out = torch_api.verify_drafts(strided(target), dev(ids), dev(u), draft_logits=strided(draft), draft_lse=dev(draft_lse), n_draft=dev(n_draft),
                                  temperature=temperature, status=status)
    ref = verify_ref(f64(target), None if ids is None else ids.numpy(), u.numpy(), None if draft is None else f64(draft),
                     None if draft_lse is None else draft_lse.numpy(), None if n_draft is None else n_draft.numpy(), temperature)
    assert status.item() == ref["status"]
    check_verify(out, ref, target.shape[2])
    return out, ref


def verify_inputs(B, G, V, dtype, seed, kind="model", temperature=1.0, noise=0.7, pad=1):
    per = 4 if dtype == "f32" else 8
    ld = -(-V // per) * per + pad * per
    target = make_logits((B, G + 1), V, dtype, seed, ld)
    gen = torch.Generator().manual_seed(seed + 1)
    u = torch.rand((B, G + 1), generator=gen, dtype=torch.float64)
    if G == 0:
        return dict(target=target, ids=None, u=u, temperature=temperature)
    room = torch.full((B, G, ld), float("nan")).to(TORCH[dtype])
    room[..., :V] = (target[:, :G].float() + torch.randn((B, G, V), generator=gen) * noise).to(TORCH[dtype])
    draft = room[..., :V]
    gumbel = -(-torch.rand((B, G, V), generator=gen).clamp_(min=1e-20).log()).log()
    ids = (draft.float() / temperature + gumbel).argmax(-1)
    lse = (draft.double() / temperature).logsumexp(-1).float()
    if kind == "lookup":
        draft = lse = None
    return dict(target=target, ids=ids, u=u, draft=draft, draft_lse=lse, temperature=temperature)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,V", [(1, 1), (3, 2), (2, 7), (5, 8), (5, 9), (9, 31), (4, 257), (70, 1000), (6, 4097), (5, 32001), (3, 50257), (4, 151936), (2, 262144)])
def test_sampling(dtype, B, V):
    run_verify(**verify_inputs(B, 0, V, dtype, B + V))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["model", "lookup"])
@pytest.mark.parametrize("B,G,V,temperature", [(1, 1, 1, 1.0), (6, 2, 2, 1.0), (8, 1, 9, 0.7), (40, 3, 257, 1.0), (30, 8, 1000, 1.5), (200, 4, 600, 1.0), (7, 4, 5001, 0.7),
                                              (6, 3, 32000, 1.0), (3, 4, 50257, 2.0), (4, 2, 151936, 1.0), (2, 128, 300, 1.0), (3, 2, 4000, 0.01), (3, 2, 4000, 100.0)])
def test_verification(dtype, kind, B, G, V, temperature):
    run_verify(**verify_inputs(B, G, V, dtype, 3 * B + G + V, kind, temperature))


@pytest.mark.parametrize("kind", ["model", "lookup"])
def test_ragged_drafts(kind):
    a = verify_inputs(60, 5, 800, "bf16", 11, kind)
    n = torch.randint(-1, 6, (60,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    # ids behind a sequence's drafts, and whole sequences that are left out, are not read
    for b in range(60):
        a["ids"][b, max(0, int(n[b])):] = -7
    run_verify(**a, n_draft=n)


def test_counts_and_ids_out_of_range():
    a = verify_inputs(8, 3, 500, "f32", 13)
    n = torch.tensor([3, 4, -2, 3, 3, 1, -1, 2], dtype=torch.int32)
    a["ids"][3, 2] = 500
    a["ids"][4, 0] = -1
    a["ids"][5, 1] = 1 << 40     # behind its drafts
    out, ref = run_verify(**a, n_draft=n)
    assert ref["status"] == 1


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_tokens(dtype):
    """-inf, the type's lowest number, one token left, none left."""
    V, low = 700, torch.finfo(TORCH[dtype]).min
    a = verify_inputs(12, 2, V, dtype, 17)
    z = a["target"]
    z[0, :, 1:] = -math.inf
    z[1, :, :-1] = -math.inf
    z[2, :, 5:690] = -math.inf
    z[3, :, 1:] = low
    z[4] = low
    z[5, 1] = -math.inf          # no distribution behind a kept draft
    z[6, 0] = -math.inf
    z[7, 0, ::2] = -math.inf
    z[8, :, 100] = torch.finfo(TORCH[dtype]).max
    a["u"][5, 0] = 0.0
    for b in range(9):
        a["ids"][b] = z[b, :2].float().argmax(-1)
    run_verify(**a)
    a["draft"] = a["draft_lse"] = None
    run_verify(**a)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_without_a_distribution(dtype):
    a = verify_inputs(10, 2, 900, dtype, 19)
    z, d, lq = a["target"], a["draft"], a["draft_lse"]
    a["u"][:, 0] = 0.999         # mostly refused at once
    a["u"][:3, :2] = 0.0         # kept
    z[0, 2, 899] = math.nan
    z[1, 0, 3] = math.inf
    z[2, 1, 0] = math.nan
    z[3, 2] = math.nan           # behind the refusal: decides nothing
    d[4, 0, 890] = math.nan
    d[5, 0, 1] = math.inf
    d[6, 0, a["ids"][6, 0]] = math.nan
    lq[7, 0] = math.nan
    lq[8, 0] = -math.inf
    d[9, 1] = math.nan
    for b in (4, 5):             # refused for certain: the draft is ten times too sure of it
        lq[b, 0] = lq[b, 0] - 5.0
    run_verify(**a)


def test_draft_that_is_never_below_the_target():
    """A refused draft with nothing left of max(p - q, 0): the token is drawn from p."""
    a = verify_inputs(40, 1, 304, "bf16", 23)
    a["draft"] = a["target"][:, :1].clone()
    a["draft_lse"] = (a["draft"].double().logsumexp(-1) - 1.0).float()
    a["u"][:, 0] = torch.linspace(0, 0.999, 40, dtype=torch.float64)
    out, ref = run_verify(**a)
    assert 0 < ref["n_accepted"].sum() < 40


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [301, 304, 5000])
@pytest.mark.parametrize("temperature", [1.0, 0.7, 0.01])
def test_masked_draft_that_is_never_below_the_target(dtype, V, temperature):
    """The same with tokens that neither distribution has: their p - q is 0 as well."""
    a = verify_inputs(40, 1, V, dtype, 24, temperature=temperature)
    a["target"][:, :, 5:V:3] = -math.inf
    a["target"][:, :, V - 1] = -math.inf
    a["ids"][:] = torch.arange(40)[:, None] % 5
    a["draft"] = torch.nn.functional.pad(a["target"][:, :1], (0, -V % 8))[..., :V]
    a["draft_lse"] = ((a["draft"].double() / temperature).logsumexp(-1) - 1.0).float()
    a["u"][:, 0] = 1.0 - 2.0 ** -20
    out, ref = run_verify(**a)
    assert ref["n_accepted"].sum() == 0


def test_draft_logits_of_minus_infinity():
    """q = 0 at the draft: kept wherever p > 0."""
    a = verify_inputs(20, 2, 300, "f16", 29)
    for b in range(20):
        a["draft"][b, 0, a["ids"][b, 0]] = -math.inf
    a["target"][3, 0, a["ids"][3, 0]] = -math.inf     # p = 0 too: refused
    run_verify(**a)


def test_uniforms_at_and_outside_their_ends():
    V = 515
    z = make_logits((1, 1), V, "f32", 31)
    z = z.expand(9, 1, V).contiguous()
    z = torch.nn.functional.pad(z, (0, 1))[..., :V]
    z[:, :, 0] = z[:, :, V - 1] = -math.inf
    u = torch.tensor([0.0, -0.0, 1 - 2.0 ** -53, 1.0, 2.0, -3.0, math.nan, math.inf, 2.0 ** -1074], dtype=torch.float64)[:, None]
    out, ref = run_verify(z, None, u)
    assert out["tokens"].view(-1).tolist() == [1, 1, V - 2, V - 2, V - 2, 1, 1, V - 2, 1]


@pytest.mark.parametrize("dtype,V", [("f32", 1000), ("bf16", 20000), ("f16", 151936)])
def test_uniforms_next_to_a_border(dtype, V):
    """Numbers 2^-33 of the total to either side of a token's border (its sums are good to 2^-36)."""
    z = make_logits((1, 1), V, dtype, 37)
    p = np.exp(f64(z)[0, 0] - f64(z).max())
    edges = np.cumsum(p) / p.sum()
    heavy = np.nonzero((p[:-1] / p.sum() > 2.0 ** -30) & (p[1:] / p.sum() > 2.0 ** -30))[0]
    at = heavy[np.linspace(0, heavy.size - 1, 100).astype(int)]
    u = np.concatenate([edges[at] - 2.0 ** -33, edges[at] + 2.0 ** -33])
    per = 4 if dtype == "f32" else 8
    whole = torch.nn.functional.pad(z, (0, -V % per)).expand(u.size, 1, -1).contiguous().to(DEV)[..., :V]
    got = torch_api.verify_drafts(whole, None, torch.from_numpy(u)[:, None].to(DEV))["tokens"].view(-1).cpu().numpy()
    assert np.array_equal(got, np.concatenate([at, at + 1]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["random", "rising", "falling", "two values"])
@pytest.mark.parametrize("B", [200, 1000])
def test_uniforms_some_way_from_a_border(dtype, order, B):
    """Numbers 2^-20 to 2^-17 of the total to either side of a border: around the distance at
    which fp32 sums are no longer asked."""
    V = 40000
    z = make_logits((1,), V, dtype, 39, sd=2.0, sure=False)[0]
    if order == "two values":
        z = torch.where(torch.arange(V) % 3 == 0, 0.0, -1.3).to(TORCH[dtype])
    elif order != "random":
        z = z.sort(descending=order == "falling").values
    p = np.exp(f64(z) - f64(z).max())
    p /= p.sum()
    edges = np.cumsum(p)
    gen = np.random.default_rng(B)
    at = gen.integers(1, V - 1, B)
    u = np.clip(edges[at] + 2.0 ** gen.uniform(-20, -17, B) * gen.choice([-1.0, 1.0], B), 0.0, 1 - 2.0 ** -53)
    got = torch_api.verify_drafts(z.expand(B, 1, V).contiguous().to(DEV), None, torch.from_numpy(u)[:, None].to(DEV))["tokens"]
    got = got[:, 0].cpu().numpy()
    # u lies in the token's interval, to the resolution of its borders
    assert (u < edges[got] + RESOLUTION).all() and (u >= edges[got] - p[got] - RESOLUTION).all()


def test_refused_drafts_next_to_a_border():
    """The same for max(p - q, 0) (terms of two rows: 2^-32)."""
    V = 30000
    a = verify_inputs(1, 1, V, "bf16", 41)
    z, d = f64(a["target"])[0, 0], f64(a["draft"])[0, 0]
    p = np.exp(z - z.max())
    r = np.maximum(p / p.sum() - np.exp(d - float(a["draft_lse"][0, 0])), 0)
    some = np.nonzero(r / r.sum() > 2.0 ** -28)[0]
    some = some[np.linspace(0, some.size - 2, 60).astype(int)]
    edges = np.cumsum(r) / r.sum()
    following = np.array([np.nonzero(r[i + 1:] > 0)[0][0] + i + 1 for i in some])
    big = r[following] / r.sum() > 2.0 ** -31
    some, following = some[big], following[big]
    last = np.concatenate([edges[some] - 2.0 ** -32, edges[some] + 2.0 ** -32])
    n = last.size
    u = torch.from_numpy(np.stack([np.ones(n), last], 1))     # 1: never below p / q of a token that stands out in q
    ids = torch.full((n, 1), int(np.argmax(np.exp(d - float(a["draft_lse"][0, 0])) - p / p.sum())))
    out = torch_api.verify_drafts(a["target"].expand(n, 2, V).contiguous().to(DEV), ids.to(DEV), u.to(DEV), draft_logits=a["draft"].expand(n, 1, V).contiguous().to(DEV),
                                  draft_lse=a["draft_lse"].expand(n, 1).contiguous().to(DEV))
    assert (out["n_accepted"] == 0).all()
    assert np.array_equal(out["tokens"][:, 0].cpu().numpy(), np.concatenate([some, following]))


def test_log_probabilities_next_to_zero():
    V = 2000
    z = torch.zeros(6, 1, V)
    for b, gap in enumerate((5.0, 15.0, 20.0, 25.0, 40.0, 80.0)):
        z[b, 0, 77 + b] = gap
    run_verify(z, None, torch.full((6, 1), 0.5, dtype=torch.float64))


@pytest.mark.parametrize("kind", ["model", "lookup"])
def test_the_same_row_in_any_batch(kind):
    """Tokens and log-probabilities of sequences alone and in batches of several sizes."""
    a = verify_inputs(300, 2, 2000, "bf16", 43, kind)
    whole, _ = run_verify(**a)
    for lo, n in ((0, 1), (7, 20), (100, 90)):
        part = {k: (v[lo:lo + n] if isinstance(v, torch.Tensor) else v) for k, v in a.items()}
        out, _ = run_verify(**part)
        assert torch.equal(out["tokens"], whole["tokens"][lo:lo + n])


def test_tokens_follow_the_target():
    """Whatever the drafts, the first token is distributed as the target's row says: expected
    counts of 16 tokens over 40,000 sequences, within 5 standard deviations."""
    V, B = 16, 40000
    gen = torch.Generator(device=DEV).manual_seed(5)
    zt, zq = torch.randn(V, generator=gen, device=DEV) * 1.5, torch.randn(V, generator=gen, device=DEV) * 1.5
    lq = zq.double().logsumexp(0)
    ids = torch.multinomial((zq.double() - lq).exp(), B, replacement=True, generator=gen)[:, None]
    u = torch.rand((B, 2), generator=gen, device=DEV, dtype=torch.float64)
    target = zt.expand(B, 2, V).contiguous()
    for draft in (True, False):
        out = torch_api.verify_drafts(target, ids, u, draft_logits=zq.expand(B, 1, V).contiguous() if draft else None,
                                      draft_lse=lq.float().expand(B, 1).contiguous() if draft else None)
        first = out["tokens"][:, 0]
        counts = torch.bincount(first, minlength=V).double()
        p = zt.double().softmax(0)
        sd = (B * p * (1 - p)).sqrt()
        assert ((counts - B * p).abs() <= 5 * sd + 1).all(), (draft, ((counts - B * p) / sd).tolist())


def test_offsets_beyond_32_bits():
    """More than 2^32 bytes and 2^31 elements before the last rows."""
    B, V = 14300, 151936
    target = torch.zeros((B, 1, V), dtype=torch.bfloat16, device=DEV)
    last = make_logits((3, 1), V, "bf16", 47).to(DEV)
    target[-3:] = last
    u = torch.rand((B, 1), dtype=torch.float64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    out = torch_api.verify_drafts(target, None, u)
    ref = verify_ref(f64(last), None, u[-3:].cpu().numpy())
    check_verify({k: v[-3:] for k, v in out.items()}, ref, V)
    flat = (u[:-3, 0] * V).floor().long()
    assert (out["tokens"][:-3, 0] - flat).abs().max() <= 1


@pytest.mark.parametrize("dtype,V", [("bf16", 1 << 22), ("f32", (1 << 21) + 5)])
def test_very_long_rows(dtype, V):
    """Rows whose parts are searched in several rounds."""
    run_verify(**verify_inputs(2, 0, V, dtype, 61))
    run_verify(**verify_inputs(1, 1, V, dtype, 67))
    run_verify(**verify_inputs(1, 1, V, dtype, 71, "lookup"))


@pytest.mark.parametrize("kind", ["model", "lookup"])
@pytest.mark.parametrize("B", [1, 14, 15, 28, 29, 114, 115, 500])
def test_every_size_of_cluster(B, kind):
    """The batch decides how many CTAs share a row."""
    run_verify(**verify_inputs(B, 1, 33000, "bf16", B, kind))


@pytest.mark.parametrize("kind", ["model", "lookup"])
@pytest.mark.parametrize("B,V", [(4, 66000), (5, 66000), (44, 66000), (45, 66000), (88, 66000), (89, 66000), (342, 66000), (343, 66000),
                                 (114, 40000), (115, 40000), (304, 40000), (5, 20479), (5, 18433), (45, 8193), (3, 6145)])
def test_every_share_of_a_row(B, V, kind):
    """Shares that are no powers of two; fewer where rows are short."""
    run_verify(**verify_inputs(B, 1, V, "bf16", B + V, kind))


def test_equal_logits():
    """Rows of one value, and of two: sums of equal terms, borders at multiples of them."""
    V = 50000
    z = torch.full((6, 1, V), 1.5)
    z[1] = -3.0e38
    z[2, :, V // 2:] = 0.75
    z[3, :, ::2] = -1.0e4
    z[4] = 6.0e4
    z[5] = -2.0e4
    u = torch.tensor([0.123456789, 0.5000001, 0.77, 0.9, 0.31, 0.999999], dtype=torch.float64)[:, None]
    run_verify(z, None, u)
    run_verify(z.clamp(min=-6.0e4).half(), None, u)


# ------------------------------------------------------------------ streams, graphs, a rollout's step
def step_inputs(seed, B=12, G=3, V=1200, D=256):
    gen = torch.Generator().manual_seed(seed)
    hidden = torch.randn((B * (G + 1), D), generator=gen).to(torch.bfloat16)
    weight = (torch.randn((V, D), generator=gen) * 3 / math.sqrt(D)).to(torch.bfloat16)
    ids = torch.randint(0, V, (B, G), generator=gen)
    u = torch.rand((B, G + 1), generator=gen, dtype=torch.float64)
    return hidden.to(DEV), weight.to(DEV), ids.to(DEV), u.to(DEV)


def rollout_step(hidden, weight, ids, u, **kw):
    B, rows = u.shape
    h, sh = torch_api.quantize_rows(hidden, **kw)
    w, sw = torch_api.quantize_rows(weight, **kw)
    logits = torch_api.lmhead_logits_int8(h, sh, w, sw, **kw)
    out = torch_api.verify_drafts(logits.view(B, rows, -1), ids, u, **kw)
    return logits, out


def test_a_rollouts_step():
    """Codes, logits, verification, and the loss of the tokens: with the target's own
    log-probabilities as the old ones every ratio is 1."""
    hidden, weight, ids, u = step_inputs(1)
    (B, G), rows = ids.shape, ids.shape[1] + 1
    logits, out = rollout_step(hidden, weight, ids, u)
    V = weight.shape[0]
    qh, sh = quantize_ref(f64(hidden))
    qw, sw = quantize_ref(f64(weight))
    want = logits_ref(qh, sh, qw, sw, "bf16")
    assert torch.equal(logits.cpu(), want)
    check_verify(out, verify_ref(f64(want).reshape(B, rows, V), ids.cpu().numpy(), u.cpu().numpy()), V)
    mask = (out["tokens"] >= 0).to(torch.uint8).view(-1)
    tokens = out["tokens"].clamp(min=0).view(-1)
    lp = torch_api.token_logprobs(logits, tokens, mask=mask)["logp"]
    assert torch.allclose(lp, out["logp"].view(-1), rtol=0, atol=2e-5)
    loss = torch_api.policy_loss(logits, tokens, mask, torch.randn(B, device=DEV), B, rows, logp_old=out["logp"].view(-1))
    st = torch_api.read_stats(loss["stats"])
    assert st["n_tokens"] == int(mask.sum()) and st["n_clipped"] == 0 and st["device_error"] == 0


def test_samples_serve_as_drafts():
    """sample_tokens' lse is the draft_lse of the next verification."""
    V = 900
    draft = make_logits((30,), V, "f32", 53).to(DEV)
    target = make_logits((30, 2), V, "f32", 53).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(2)
    u = torch.rand((30, 3), dtype=torch.float64, device=DEV, generator=gen)
    s = torch_api.sample_tokens(draft, u[:, 2].contiguous())
    args = dict(draft=draft.cpu()[:, None], draft_lse=s["lse"].cpu()[:, None])
    run_verify(target.cpu(), s["tokens"].cpu()[:, None], u[:, :2].contiguous().cpu(), **args)


def test_another_stream():
    want = rollout_step(*step_inputs(2))
    side = torch.cuda.Stream()
    inputs = step_inputs(2)
    side.wait_stream(torch.cuda.current_stream())
    got = rollout_step(*inputs, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1]["tokens"], want[1]["tokens"]) and torch.equal(got[1]["logp"], want[1]["logp"])


def test_captured_and_replayed():
    """One graph of the whole step, replayed on new inputs; two graphs with a workspace each, in turn."""
    inputs = step_inputs(3)
    rollout_step(*inputs)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = rollout_step(*inputs)
        graphs.append((g, out))
    for seed in (4, 5):
        for x, y in zip(inputs, step_inputs(seed)):
            x.copy_(y)
        want = rollout_step(*step_inputs(seed))
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1]["tokens"], want[1]["tokens"]) and torch.equal(out[1]["lse"], want[1]["lse"])


def test_behind_other_work():
    """Calls whose inputs the launch, copy or fill right before them writes, in part on a stream that is joined there: one after
    another, and captured.  (Each call's launch may begin before that work has ended.)"""
    sets = [step_inputs(seed) for seed in (6, 7)]
    wants = [rollout_step(*s) for s in sets]
    source, here = [x.clone() for x in sets[0]], [x.clone() for x in sets[0]]
    z, side = torch.empty_like(wants[0][0]), torch.cuda.Stream()
    (B, G), V = here[2].shape, z.shape[1]

    def step():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            here[1].copy_(source[1])                       # a copy, joined right before the step
        here[2].copy_(source[2])
        here[3].zero_()
        here[3].add_(source[3])
        here[0].copy_(source[0])
        torch.cuda.current_stream().wait_stream(side)
        logits, out = rollout_step(*here)
        z.fill_(-1.0)
        z.copy_(logits)                                    # a copy right before a verification
        again = torch_api.verify_drafts(z.view(B, G + 1, V), here[2], here[3])
        here[3].zero_()                                    # a fill: every draft stays that can, the first token is drawn
        first = torch_api.verify_drafts(z.view(B, G + 1, V), here[2], here[3])
        return logits, out, again, first

    def check(got, want):
        assert torch.equal(got[0], want[0])
        for k in ("tokens", "n_accepted", "logp", "lse"):
            assert torch.equal(got[1][k], want[1][k]) and torch.equal(got[2][k], want[1][k])
        possible = want[0].view(B, G + 1, V).gather(2, here[2].clamp(0, V - 1)[..., None].expand(B, G, 1)) > -math.inf
        assert torch.equal(got[3]["n_accepted"], possible[..., 0].long().cumprod(1).sum(1))

    for k in range(40):
        for x, y in zip(source, sets[k % 2]):
            x.copy_(y)
        check(step(), wants[k % 2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(10):
        for x, y in zip(source, sets[k % 2]):
            x.copy_(y)
        g.replay()
        check(got, wants[k % 2])


def test_the_c_names():
    """The bindings that forward to the C entry points, with their defaults."""
    hidden, weight, ids, u = step_inputs(7)
    (B, G), (V, D), R = ids.shape, weight.shape, hidden.shape[0]
    want_logits, want = rollout_step(hidden, weight, ids, u)
    h, w = torch.empty((R, D), dtype=torch.int8, device=DEV), torch.empty((V, D), dtype=torch.int8, device=DEV)
    sh, sw = torch.empty(R, device=DEV), torch.empty(V, device=DEV)
    rl.rl_quantize_rows_int8(hidden, "bf16", R, D, D, h, D, sh)
    rl.rl_quantize_rows_int8(weight, "bf16", V, D, D, w, D, sw)
    logits = torch.empty((R, V), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(rl.rl_lmhead_int8_workspace_size(R, D), dtype=torch.uint8, device=DEV)
    rl.rl_lmhead_logits_int8(h, D, sh, w, D, sw, R, D, V, "bf16", logits, V, workspace=ws)
    assert torch.equal(logits, want_logits)
    tokens = torch.empty((B, G + 1), dtype=torch.int64, device=DEV)
    d = rl.rl_verify_drafts_desc_init()
    d.target_logits, d.B, d.G, d.V, d.ld = logits.data_ptr(), B, G, V, V
    d.draft_ids, d.uniforms, d.tokens = ids.data_ptr(), u.data_ptr(), tokens.data_ptr()
    rl.rl_verify_drafts(d)      # the other outputs are not asked for
    assert torch.equal(tokens, want["tokens"])
    with pytest.raises(rl.RlLossError, match="rl_lmhead_logits_int8"):
        rl.rl_lmhead_logits_int8(h, D, sh, w, D, sw, R, D, V, "bf16", logits, V)


def test_nothing_to_do():
    assert torch_api.quantize_rows(torch.zeros((0, 64), device=DEV))[0].shape == (0, 64)
    w, sw = torch_api.quantize_rows(torch.randn((100, 64), device=DEV))
    out = torch_api.lmhead_logits_int8(torch.zeros((0, 64), dtype=torch.int8, device=DEV), torch.zeros(0, device=DEV), w, sw)
    assert out.shape == (0, 100)
    z = torch.zeros((0, 3, 64), device=DEV)
    got = torch_api.verify_drafts(z, torch.zeros((0, 2), dtype=torch.int64, device=DEV), torch.zeros((0, 3), dtype=torch.float64, device=DEV))
    assert got["tokens"].shape == (0, 3)
    left_out = torch_api.verify_drafts(torch.full((2, 2, 64), math.nan, device=DEV), torch.full((2, 1), -5, device=DEV), torch.zeros((2, 2), dtype=torch.float64, device=DEV),
                                       n_draft=torch.tensor([-1, -1], dtype=torch.int32, device=DEV))
    assert (left_out["tokens"] == -1).all() and (left_out["logp"] == 0).all() and (left_out["lse"] == 0).all()


@pytest.mark.parametrize("wrong", [
    lambda a: a.update(uniforms=a["uniforms"].float()),
    lambda a: a.update(draft_ids=a["draft_ids"].int()),
    lambda a: a.update(draft_ids=None),
    lambda a: a.update(draft_ids=a["draft_ids"][:, :1]),
    lambda a: a.update(draft_lse=None),
    lambda a: a.update(draft_logits=a["draft_logits"].float()),
    lambda a: a.update(n_draft=torch.zeros(4, dtype=torch.int64, device=DEV)),
    lambda a: a.update(target_logits=a["target_logits"].transpose(0, 1)),
    lambda a: a.update(target_logits=a["target_logits"][..., ::2]),
    lambda a: a.update(target_logits=a["target_logits"].cpu()),
    lambda a: a.update(uniforms=a["uniforms"].cpu()),
    lambda a: a.update(status=torch.zeros(2, dtype=torch.int32, device=DEV)),
])
def test_tensors_that_are_refused(wrong):
    a = dict(target_logits=torch.zeros((4, 3, 64), dtype=torch.bfloat16, device=DEV), draft_ids=torch.zeros((4, 2), dtype=torch.int64, device=DEV),
             uniforms=torch.zeros((4, 3), dtype=torch.float64, device=DEV), draft_logits=torch.zeros((4, 2, 64), dtype=torch.bfloat16, device=DEV),
             draft_lse=torch.zeros((4, 2), device=DEV))
    torch_api.verify_drafts(**a)
    wrong(a)
    with pytest.raises(ValueError):
        torch_api.verify_drafts(**a)


def test_a_stride_that_no_vector_load_takes():
    with pytest.raises(rl.RlLossError):
        torch_api.verify_drafts(torch.zeros((4, 3, 63), device=DEV), torch.zeros((4, 2), dtype=torch.int64, device=DEV), torch.zeros((4, 3), dtype=torch.float64, device=DEV))
    with pytest.raises(rl.RlLossError):
        torch_api.quantize_rows(torch.zeros((4, 63), device=DEV))
