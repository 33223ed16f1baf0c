"""The token operators at the edges of what a caller may do: offsets past 32
bits, inputs freed while another stream reads them, two host threads, captured
autograd wrappers, and the refusals that need a GPU tensor."""
import threading

import numpy as np
import pytest
import torch

import oracle
import ppo_policy_loss_gb300 as rl
from ppo_policy_loss_gb300 import torch_api
from _tokens import check_close, check_gradient, check_logprobs, logits, storage
from test_gpu_topk_distill import teacher, tolerances

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    rl.build()
    rl.load()


def test_offsets_past_32_bits():
    """More than 2^31 elements and 2^32 bytes of logits: the rows around the
    limit and the last one against the oracle, in all three operators."""
    R, V, k = 14200, 151936, 16
    gen = torch.Generator(device=DEV).manual_seed(3)
    z = torch.empty((R, V), dtype=torch.bfloat16, device=DEV).normal_(0.0, 3.0, generator=gen)
    ids = torch.randint(0, V, (R, 2), device=DEV, generator=gen)
    rows = [0, 14133, 14134, 14135, R - 1]  # 2^31 / V = 14134.2
    assert 2 ** 31 < R * V and 2 ** 32 < R * V * 2
    sub, sub_ids = z[rows].cpu(), ids[rows].cpu().numpy()
    out = torch_api.token_logprobs(z, ids, k=k, want_lse=True)
    ref = oracle.token_logprobs(storage(sub), "bf16", V, sub_ids, None, k, 1.0)
    check_logprobs({n: t[rows] for n, t in out.items()}, ref, V)
    dlogp = torch.randn((R, 2), device=DEV, generator=gen)
    dent = torch.randn(R, device=DEV, generator=gen)
    got = torch_api.token_logprobs_backward(z, ids, dlogp, out["lse"], out["entropy"], dent)[rows]
    host = [t[rows].cpu().numpy() for t in (dlogp, out["lse"], out["entropy"], dent)]
    d, size, lp = oracle.token_logprobs_bwd(storage(sub), "bf16", V, sub_ids, *host, None, 1.0)
    check_gradient(got, "bf16", d, size, lp)
    del got
    t = torch_api.topk_distill(z, out["topk_ids"], out["topk_logp"], reverse=0.5, norm=5.0)
    tid, tlq = out["topk_ids"][rows].cpu().numpy(), out["topk_logp"][rows].cpu().numpy()
    ref = oracle.topk_distill(storage(sub), "bf16", V, tid, tlq, reverse=0.5, norm=5.0)
    row_tol, grad_tol = tolerances(ref, "bf16", V)
    check_close("row_loss", t["row_loss"][rows].cpu(), ref["row_loss"], row_tol)
    check_close("dlogits", oracle.decode(storage(t["dlogits"][rows]), "bf16"), ref["dlogits"], grad_tol)


def test_inputs_freed_while_another_stream_reads_them():
    """The caller drops its tensors right after a call on a stream that is still
    busy, and memory of the same size is written on the current stream."""
    R, V = 256, 32000
    side = torch.cuda.Stream(DEV)
    z = logits(R, V, "bf16", 4).to(DEV).contiguous()
    ids = torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(5)).to(DEV)
    tid, tlq = (t.to(DEV) for t in teacher(z.cpu(), 8, 3))
    lse = torch_api.token_logprobs(z, ids, want_lse=True)["lse"]
    one = torch.ones(R, device=DEV)
    calls = [lambda x, s: torch_api.token_logprobs(x, ids, k=4, stream=s)["topk_logp"],
             lambda x, s: torch_api.token_logprobs_backward(x, ids, one, lse, stream=s),
             lambda x, s: torch_api.topk_distill(x, tid, tlq, stream=s)["dlogits"]]
    for call in calls:
        ref = call(z, None)
        x = z.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        out = call(x, side)
        del x
        junk = [torch.full((R, V), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        del junk


def test_two_host_threads():
    """Calls from two threads, each on its own stream with its own workspace."""
    V = 20000
    z = [logits(96, V, "f16", 70 + i).to(DEV).contiguous() for i in range(2)]
    ids, lq = zip(*[(a.to(DEV), b.to(DEV)) for a, b in (teacher(x.cpu(), 8, 3) for x in z)])

    def work(i, stream):
        a = torch_api.token_logprobs(z[i], ids[i], k=9, want_lse=True, stream=stream)
        return a["logp"], a["topk_ids"], torch_api.topk_distill(z[i], ids[i], lq[i], stream=stream)["dlogits"]

    ref = [work(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    got = [[], []]
    threads = [threading.Thread(target=lambda i=i: got[i].extend(work(i, streams[i]) for _ in range(10))) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 10
        for o in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(o, ref[i]))


def test_captured_wrappers():
    """Forward and backward of both wrappers in one graph, replayed on new
    logits, give the bits of the eager gradients."""
    R, V = 48, 5000
    zs = [logits(R, V, "bf16", 80 + i, sure=False).to(DEV).contiguous() for i in range(2)]
    ids = torch.randint(0, V, (R,), generator=torch.Generator().manual_seed(5)).to(DEV)
    tid, tlq = (t.to(DEV) for t in teacher(zs[0].cpu(), 8, 3))
    w = torch.randn(R, generator=torch.Generator().manual_seed(6)).to(DEV)
    mask = (torch.arange(R, device=DEV) % 5 != 1)
    ws = torch_api.new_distill_workspace(DEV)

    def grad(leaf):
        logp, ent = torch_api.TokenLogprobs.apply(leaf, ids, mask, 0.9)
        loss = torch_api.FusedTopkDistill.apply(leaf, tid, tlq, mask, dict(reverse=0.25, workspace=ws))
        return torch.autograd.grad((logp * w).sum() + 0.1 * ent.sum() + 3.0 * loss, leaf)[0]

    ref = [grad(z.clone().requires_grad_()) for z in zs]
    leaf = zs[0].clone().requires_grad_()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grad(leaf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = grad(leaf)
    for i in (1, 0, 1):
        with torch.no_grad():
            leaf.copy_(zs[i])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref[i])


def test_refusals_of_what_the_kernels_would_write_or_read_wrongly():
    z = logits(4, 64, "f32", 1).to(DEV).contiguous()
    ids = torch.zeros(4, dtype=torch.int64, device=DEV)
    one = torch.ones(4, device=DEV)
    lse = torch_api.token_logprobs(z, want_lse=True)["lse"]
    tid = torch.tensor([[0, 1]] * 4, device=DEV)
    tlq = torch.full((4, 2), -1.0, device=DEV)
    for st in (torch.zeros(1, dtype=torch.int32), torch.zeros(0, dtype=torch.int32, device=DEV),
               torch.zeros(1, dtype=torch.uint8, device=DEV), torch.zeros(1, device=DEV)):
        with pytest.raises(ValueError, match="status"):
            torch_api.token_logprobs(z, ids, status=st)
        with pytest.raises(ValueError, match="status"):
            torch_api.token_logprobs_backward(z, ids, one, lse, status=st)
    with pytest.raises(ValueError, match="ids"):
        torch_api.token_logprobs_backward(z, None, one, lse)
    for st in (torch.zeros((rl.DISTILL_STATS_BYTES, 2), dtype=torch.uint8, device=DEV)[:, 0],
               torch.zeros(1, dtype=torch.uint8, device=DEV).expand(rl.DISTILL_STATS_BYTES)):
        with pytest.raises(ValueError, match="stats"):
            torch_api.topk_distill(z, tid, tlq, stats=st)
    with pytest.raises(rl.RlLossError):  # off its 8-byte boundary
        torch_api.topk_distill(z, tid, tlq, stats=torch.zeros(1 + rl.DISTILL_STATS_BYTES, dtype=torch.uint8, device=DEV)[1:])
    leaf = z.clone().requires_grad_()
    for d in (None, z, "new"):
        with pytest.raises(ValueError, match="dlogits"):
            torch_api.FusedTopkDistill.apply(leaf, tid, tlq, None, dict(dlogits=d))
    assert torch_api.token_logprobs(z, torch.empty((4, 0), dtype=torch.int64, device=DEV))["logp"].shape == (4, 0)


@pytest.mark.parametrize("pattern", ["none", "random", "first", "last", "all"])
def test_rows_dealt_out_one_by_one(pattern):
    """Many rounds of long rows give the bits of the same rows in few rounds,
    wherever the masked rows lie; every masked row is written, none twice as
    something else."""
    R, V, k = 4000, 60000, 7
    gen = torch.Generator(device=DEV).manual_seed(9)
    z = torch.empty((R, V), dtype=torch.bfloat16, device=DEV).normal_(0.0, 3.0, generator=gen)
    ids = torch.randint(0, V, (R, 40), device=DEV, generator=gen)
    keep = {"none": torch.ones(R), "random": (torch.rand(R, generator=torch.Generator().manual_seed(1)) < 0.6),
            "first": torch.arange(R) < 1, "last": torch.arange(R) >= R - 900, "all": torch.zeros(R)}[pattern]
    mask = keep.to(torch.uint8).to(DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    for m in ([None, mask] if pattern == "none" else [mask]):
        out = torch_api.token_logprobs(z, ids, mask=m, k=k, want_lse=True, status=st)
        for a in range(0, R, 800):
            part = torch_api.token_logprobs(z[a:a + 800], ids[a:a + 800], mask=None if m is None else m[a:a + 800], k=k,
                                            want_lse=True)
            for n, t in part.items():
                assert torch.equal(out[n][a:a + 800], t), (n, a)
        off = mask == 0
        assert (out["topk_ids"][off] == -1).all()
        assert all((out[n][off] == 0).all() for n in ("logp", "entropy", "lse", "topk_logp"))
    assert int(st.item()) == 0


def test_dealt_rows_beside_another_call_and_replayed():
    """Two calls whose rows are dealt out run on two streams at once, and one is
    captured and replayed: the bits of a call alone."""
    R, V = 3000, 60000
    gen = torch.Generator(device=DEV).manual_seed(2)
    z = [torch.empty((R, V), dtype=torch.bfloat16, device=DEV).normal_(0.0, 3.0, generator=gen) for _ in range(2)]
    mask = (torch.rand(R, device=DEV, generator=gen) < 0.7)
    call = lambda i, s=None: torch_api.token_logprobs(z[i], mask=mask, k=5, want_lse=True, stream=s)  # noqa: E731
    ref = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    outs = [[call(i, streams[i]) for i in range(2)] for _ in range(5)]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = call(0)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for o in outs + [[got]]:
        for i, out in enumerate(o):
            assert all(torch.equal(out[n], ref[i][n]) for n in ("entropy", "lse", "topk_ids", "topk_logp"))
