"""Performance cases of the token log-probability and distillation operators.

Three operators over a [R, V] matrix of vocabulary logits (fp32, bf16 or fp16):

* ``logprobs``      log-probabilities of given tokens, entropy, log-sum-exp and
                    the k most likely alternatives of each row;
* ``logprobs_bwd``  the gradient of those log-probabilities and entropies with
                    respect to the logits;
* ``distill``       distillation from a teacher's top-k log-probabilities: the
                    loss and its gradient.

``run`` computes a case in plain torch operations (fp32, rounded once at the
end), or with this package's kernels where ``own`` is true; ``exact`` computes
it in fp64 from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TAIL_FLOOR = 2.0 ** -24     # the least mass of a teacher's tail
PROB_FLOOR = 2.0 ** -126    # the least probability whose logarithm is taken


def _case(op, R, V, dtype, **kw):
    c = dict(op=op, R=R, V=V, dtype=dtype, pad=0, k=0, n_ids=1, valid=1.0, banned=0.0, temperature=1.0,
             entropy=True, tail="bucket", reverse=0.0)
    c.update(kw)
    return c


def listed():
    cases = [
        # a decode step of one sequence: latency alone
        _case("logprobs", 1, 151936, "bf16", k=20, name="logprobs_one_token"),
        # a decode step of a batch of sequences
        _case("logprobs", 64, 151936, "bf16", k=20, name="logprobs_decode_batch"),
        # rollouts scored for an update: no alternatives, ragged sequences
        _case("logprobs", 4096, 151936, "bf16", valid=0.7, name="logprobs_rollouts"),
        # a teacher scoring a batch for distillation
        _case("logprobs", 8192, 151936, "bf16", k=64, n_ids=0, name="logprobs_teacher"),
        # short rows under a sampling temperature, part of the vocabulary ruled out
        _case("logprobs", 16384, 32000, "f16", k=16, valid=0.6, banned=0.2, temperature=0.7, name="logprobs_short_rows"),
        # fp32 logits of an odd vocabulary, several given tokens a row
        _case("logprobs", 777, 50257, "f32", pad=3, k=5, n_ids=4, name="logprobs_odd_f32"),
        # the tiny workload's gradient: latency alone
        _case("logprobs_bwd", 128, 1024, "f32", name="logprobs_bwd_tiny"),
        # a training step's gradient of log-probabilities and entropies
        _case("logprobs_bwd", 4096, 151936, "bf16", name="logprobs_bwd_entropy"),
        # several given tokens a row, an odd vocabulary, ragged sequences
        _case("logprobs_bwd", 3001, 32001, "f16", pad=7, n_ids=16, valid=0.6, entropy=False, name="logprobs_bwd_ids"),
        # the tiny workload's distillation: latency alone
        _case("distill", 128, 1024, "f32", k=8, name="distill_tiny"),
        # distillation of a batch from a teacher's top 64
        _case("distill", 8192, 151936, "bf16", k=64, name="distill_batch"),
        # both divergences mixed, short rows, ragged sequences, softened student
        _case("distill", 4095, 32000, "f16", k=32, valid=0.6, temperature=2.0, reverse=0.5, name="distill_mixed"),
    ]
    return cases


def draw(rng: random.Random):
    op = rng.choice(["logprobs", "logprobs", "logprobs_bwd", "distill", "distill"])
    V = int(math.exp(rng.uniform(math.log(300), math.log(262144))))
    most = 8192 * 151936 // (4 if op == "logprobs_bwd" else 1) // V
    R = int(math.exp(rng.uniform(0.0, math.log(max(2, min(most, 32768))))))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if dtype == "f32":
        R = max(1, R // 2)
    per = 4 if dtype == "f32" else 8           # row strides are multiples of 16 bytes
    pad = -V % per + per * rng.choice([0, 0, 1, 5])
    c = _case(op, R, V, dtype, pad=pad, valid=round(rng.uniform(0.4, 1.0), 2) if rng.random() < 0.5 else 1.0,
              temperature=rng.choice([1.0, 1.0, 0.7, 2.0]))
    if op == "distill":
        c["k"] = min(V, rng.randint(1, 128))
        c["tail"] = rng.choice(["bucket", "bucket", "renormalise"])
        c["reverse"] = rng.choice([0.0, 0.5, 1.0]) if c["tail"] == "bucket" else 0.0
    else:
        c["n_ids"] = rng.choice([1, 1, 1, 3, 16, 64])
        c["banned"] = rng.choice([0.0, 0.0, 0.3])
        if op == "logprobs":
            c["k"] = min(V, rng.choice([0, 1, 5, 20, 50, 128, rng.randint(2, 128)]))
        else:
            c["entropy"] = rng.random() < 0.5
    return c


def _inputs(case, seed):
    """The tensors of a case: logits of a peaked distribution, the tokens sampled from it, masks, gradients or the teacher's top."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + 17)
    R, V, ld, dt = case["R"], case["V"], case["V"] + case["pad"], DTYPES[case["dtype"]]
    z = torch.randn((R, ld), generator=gen, device=dev, dtype=torch.float32).mul_(3.0)
    # one token in eight stands out in its row, as where a model is sure of the next one
    sure = torch.rand(R, generator=gen, device=dev) < 0.125
    hot = torch.randint(0, V, (R,), generator=gen, device=dev)
    z[torch.arange(R, device=dev), hot] += torch.where(sure, 14.0, 0.0)
    if case["banned"] > 0:
        out = torch.rand(V, generator=gen, device=dev) < case["banned"]
        out[0] = False
        z[:, :V].masked_fill_(out, -math.inf)
    s = {"logits": z.to(dt)}
    T = min(R, 512)
    n_seq = -(-R // T)
    if case["valid"] < 1.0:
        lengths = torch.randint(0, max(1, int(2 * T * case["valid"])), (n_seq,), generator=gen, device=dev).clamp_(max=T)
        s["mask"] = (torch.arange(T, device=dev)[None, :] < lengths[:, None]).reshape(-1)[:R].to(torch.uint8).contiguous()
        s["mask"][0] = 1
    else:
        s["mask"] = None
    M = case["n_ids"]
    if case["op"] != "distill" and M:
        noise = torch.rand((R, V), generator=gen, device=dev).clamp_(min=1e-20).log_().neg_().log_().neg_()
        first = (s["logits"][:, :V].float() / case["temperature"] + noise).argmax(1, keepdim=True)
        rest = torch.randint(0, V, (R, M - 1), generator=gen, device=dev)
        s["ids"] = torch.cat([first, rest], 1) if M > 1 else first[:, 0].contiguous()
    else:
        s["ids"] = None
    if case["op"] == "logprobs_bwd":
        s["dlogp"] = torch.randn(s["ids"].shape, generator=gen, device=dev)
        s["dentropy"] = torch.randn(R, generator=gen, device=dev) if case["entropy"] else None
    if case["op"] == "distill":
        K = case["k"]
        t = (s["logits"][:, :V].float() + torch.randn((R, V), generator=gen, device=dev)).div_(case["temperature"])
        top, ids = t.topk(K, 1)
        s["teacher_ids"] = ids.contiguous()
        s["teacher_logp"] = (top - t.logsumexp(1, keepdim=True)).contiguous()
        s["grad_scale"] = float(R) if case["dtype"] == "f16" else 1.0
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "logprobs_bwd":  # what the forward pass left
        z = s["logits"][:, :case["V"]].float() / case["temperature"]
        s["lse"] = z.logsumexp(1)
        p = (z - s["lse"][:, None]).exp_()
        s["entropy"] = -torch.where(p > 0, p * (z - s["lse"][:, None]), 0.0).sum(1) if case["entropy"] else None
    if case["op"] == "distill":  # the scratch a training loop keeps
        s["workspace"] = torch.zeros(1 << 18, dtype=torch.uint8, device="cuda")
    s["case"] = dict(case)
    return s


# ------------------------------------------------------------------ the framework's kernels
def _run_own(s):
    from ppo_policy_loss_gb300 import torch_api
    c = s["case"]
    logits = s["logits"][:, :c["V"]]
    if c["op"] == "logprobs":
        return torch_api.token_logprobs(logits, s["ids"], mask=s["mask"], k=c["k"], temperature=c["temperature"], want_lse=True)
    if c["op"] == "logprobs_bwd":
        return {"dlogits": torch_api.token_logprobs_backward(
            logits, s["ids"], s["dlogp"], s["lse"], entropy=s["entropy"], dentropy=s["dentropy"], mask=s["mask"],
            temperature=c["temperature"])}
    out = torch_api.topk_distill(logits, s["teacher_ids"], s["teacher_logp"], mask=s["mask"], tail=c["tail"], reverse=c["reverse"],
                                 temperature=c["temperature"], grad_scale=s["grad_scale"], workspace=s["workspace"])
    return {n: out[n] for n in ("loss", "row_loss", "dlogits")}


# ------------------------------------------------------------------ plain forms
def _softmax_parts(z):
    """Row maximum, e^(z - max), its sum, and the sum's logarithm: where one token holds nearly all the mass the sum is next
    to 1, so it is summed in fp64 and only its logarithm is rounded."""
    m = z.amax(1, keepdim=True)
    e = (z - m).exp_()
    total = e.sum(1, keepdim=True, dtype=torch.float64)
    return m, e, total.float(), total.log().float()


def _plain_logprobs(s, c):
    V, T, k = c["V"], c["temperature"], c["k"]
    raw = s["logits"][:, :V].float()
    on = None if s["mask"] is None else s["mask"] != 0
    keep = (lambda x, empty=0: x) if on is None else (  # noqa: E731
        lambda x, empty=0: torch.where(on if x.dim() == 1 else on[:, None], x, torch.full((), empty, dtype=x.dtype, device=x.device)))
    z = raw / T
    m, e, total, log_total = _softmax_parts(z)
    lp = z.sub_(m).sub_(log_total)
    out = {"lse": keep((m + log_total)[:, 0])}
    if s["ids"] is not None:
        ids = s["ids"] if s["ids"].dim() == 2 else s["ids"][:, None]
        out["logp"] = keep(lp.gather(1, ids)).reshape(s["ids"].shape)
    out["entropy"] = keep(-torch.where(e > 0, e * lp, 0.0).sum(1, dtype=torch.float64).float() / total[:, 0])
    if k:
        # the largest first, ties to the lowest index: one integer orders both
        bits = (raw + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
        ids = (order * 2 ** 32 + torch.arange(V - 1, -1, -1, device=raw.device)).topk(k, 1).values
        ids = V - 1 - (ids & 0xFFFFFFFF)
        out["topk_ids"] = keep(ids, -1)
        out["topk_logp"] = keep(lp.gather(1, ids))
    return out


def _plain_logprobs_bwd(s, c):
    V, T = c["V"], c["temperature"]
    ids = s["ids"] if s["ids"].dim() == 2 else s["ids"][:, None]
    g = s["dlogp"] if s["dlogp"].dim() == 2 else s["dlogp"][:, None]
    lp = s["logits"][:, :V].float() / T - s["lse"][:, None]
    p = lp.exp()
    if s["dentropy"] is not None:
        slope = -s["dentropy"][:, None] * torch.where(p > 0, lp + s["entropy"][:, None], 0.0)
        d = p * (slope - g.sum(1, keepdim=True))
    else:
        d = p.mul_(-g.sum(1, keepdim=True))
    d.scatter_add_(1, ids, g)
    if s["mask"] is not None:
        d.mul_((s["mask"] != 0)[:, None])
    return {"dlogits": (d / T).to(s["logits"].dtype)}


def _plain_distill(s, c):
    V, T, rev = c["V"], c["temperature"], c["reverse"]
    ids, lq = s["teacher_ids"], s["teacher_logp"]
    R, K = ids.shape
    z = s["logits"][:, :V].float() / T
    m, e, total, log_total = _softmax_parts(z)
    at = z.gather(1, ids) - m
    e_at = at.exp()
    rest = e.scatter(1, ids, 0.0).sum(1, keepdim=True)  # the tail by itself: no difference of near numbers
    lp = at - log_total
    p = e_at / total
    q = lq.double().exp()
    if c["tail"] == "bucket":
        q_tail = (1.0 - q.sum(1, keepdim=True)).clamp_(min=TAIL_FLOOR).float()
        q = q.float()
        p_tail = (rest / total).clamp_(min=PROB_FLOOR)
        lp_tail, lq_tail = p_tail.log(), q_tail.log()
        if K == V:
            q_tail = torch.zeros_like(q_tail)
    else:
        q = (q / q.sum(1, keepdim=True)).float()
        q_tail = torch.zeros((R, 1), device=z.device)
        lq = q.log()
        p_tail, lp_tail, lq_tail = torch.ones_like(q_tail), torch.zeros_like(q_tail), torch.zeros_like(q_tail)
    mass = q.sum(1, keepdim=True) + q_tail
    fwd = torch.where(q > 0, q * (lq - lp), 0.0).sum(1, keepdim=True) + q_tail * (lq_tail - lp_tail)
    inside, outside = p * mass - q, mass - q_tail / p_tail
    loss = fwd
    if rev:
        lqr = lq.clamp(min=math.log(PROB_FLOOR))
        tail = torch.zeros_like(p_tail) if K == V else p_tail
        back = torch.where(p > 0, p * (lp - lqr), 0.0).sum(1, keepdim=True) + tail * (lp_tail - lq_tail)
        inside = (1 - rev) * inside + rev * torch.where(p > 0, p * (lp - lqr - back), 0.0)
        outside = (1 - rev) * outside + rev * (lp_tail - lq_tail - back)
        loss = (1 - rev) * fwd + rev * back
    on = torch.ones(R, device=z.device) if s["mask"] is None else (s["mask"] != 0).float()
    n = on.sum()
    d = (e / total).mul_(outside).scatter_(1, ids, inside)
    d.mul_((on * (s["grad_scale"] / (n * T)))[:, None])
    row = loss[:, 0] * on
    return {"loss": (row.double().sum() / n).float(), "row_loss": row, "dlogits": d.to(s["logits"].dtype)}


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    return {"logprobs": _plain_logprobs, "logprobs_bwd": _plain_logprobs_bwd, "distill": _plain_distill}[c["op"]](state, c)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    R, V, es = case["R"], case["V"], 4 if case["dtype"] == "f32" else 2
    n = max(1.0, R * (1.0 if case["valid"] >= 1.0 else _valid_share(case)))
    if case["op"] == "logprobs":
        return {"bytes": n * V * es + R * (12.0 * case["n_ids"] + 8 + 12 * case["k"]), "flops": 6.0 * n * V}
    if case["op"] == "logprobs_bwd":
        return {"bytes": (n + R) * V * es + R * (12.0 * case["n_ids"] + 12), "flops": 5.0 * n * V}
    return {"bytes": (n + R) * V * es + R * (12.0 * case["k"] + 5), "flops": 8.0 * n * V}


def _valid_share(case):
    """Mean share of valid rows: lengths are uniform on [0, 2 T valid), cut at T."""
    T = min(case["R"], 512)
    hi = max(1, int(2 * T * case["valid"]))
    return sum(min(x, T) for x in range(hi)) / hi / T


# ------------------------------------------------------------------ the definitions in fp64
def _exact_rows(case, s, lo, hi):
    """Rows [lo, hi) of a case from the definition, one distribution at a time over the last axis."""
    V, T, rows = case["V"], case["temperature"], slice(lo, hi)
    x = s["logits"][rows, :V].to(torch.float64) / T
    lse = torch.logsumexp(x, dim=-1)
    on = torch.ones(hi - lo, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"][rows].bool()
    if case["op"] == "logprobs":
        lp = x - lse.unsqueeze(-1)
        got = {"lse": lse * on, "entropy": torch.special.entr(lp.exp()).sum(-1) * on}
        if s["ids"] is not None:
            want = s["ids"][rows].reshape(hi - lo, -1)
            got["logp"] = torch.take_along_dim(lp, want, -1).masked_fill(~on[:, None], 0.0)
        if case["k"]:
            got["topk_logp"] = torch.topk(lp, case["k"], dim=-1, sorted=True).values.masked_fill(~on[:, None], 0.0)
        return got
    if case["op"] == "logprobs_bwd":
        p = torch.softmax(x, -1)
        g = s["dlogp"][rows].double().reshape(hi - lo, -1)
        d = torch.zeros_like(p).scatter_add_(-1, s["ids"][rows].reshape(hi - lo, -1), g) - p * g.sum(-1, keepdim=True)
        if s["dentropy"] is not None:
            # the entropy and log-sum-exp are inputs of this pass, as the forward pass rounded them
            given = s["entropy"][rows].double().unsqueeze(-1)
            d = d - s["dentropy"][rows].double().unsqueeze(-1) * (p * given - torch.special.entr(p))
        return {"dlogits": d / T * on.unsqueeze(-1)}
    ids, lq = s["teacher_ids"][rows], s["teacher_logp"][rows].double()
    K, w = ids.shape[1], case["reverse"]
    in_top = torch.zeros_like(x, dtype=torch.bool).scatter_(-1, ids, True)
    bucket = case["tail"] == "bucket"
    if not bucket:
        lq = torch.log_softmax(lq, -1)
    lp = torch.take_along_dim(x, ids, -1) - lse.unsqueeze(-1)
    if bucket and K < V:
        lq_t = torch.log((1.0 - lq.exp().sum(-1)).clamp(min=TAIL_FLOOR))
        lp_t = (torch.logsumexp(x.masked_fill(in_top, -math.inf), -1) - lse).clamp(min=math.log(PROB_FLOOR))
        lq, lp = torch.cat([lq, lq_t.unsqueeze(-1)], -1), torch.cat([lp, lp_t.unsqueeze(-1)], -1)
    q, pb = lq.exp(), lp.exp()
    gap = lp - lq.clamp(min=math.log(PROB_FLOOR))
    forward = torch.where(q > 0, q * (lq - lp), 0.0).sum(-1)
    back = torch.where(pb > 0, pb * gap, 0.0).sum(-1)
    # gradient with respect to a bucket's own logit mass, spread over its tokens by their share of it
    per = (1 - w) * (q.sum(-1, keepdim=True) - q / pb) + w * (gap - back.unsqueeze(-1))
    p = torch.softmax(x, -1)
    if bucket and K < V:
        slope = per[:, K:].expand_as(p)
    else:
        slope = ((1 - w) * q.sum(-1, keepdim=True) - w * back.unsqueeze(-1)).expand_as(p)
    inside = (1 - w) * (pb * q.sum(-1, keepdim=True) - q) + w * torch.where(pb > 0, pb * (gap - back.unsqueeze(-1)), 0.0)
    d = (p * slope).scatter(-1, ids, inside[:, :K])
    n = float(s["logits"].shape[0]) if s["mask"] is None else float(s["mask"].sum())
    return {"row_loss": ((1 - w) * forward + w * back) * on, "dlogits": d * (s["grad_scale"] / (n * T)) * on.unsqueeze(-1)}


def exact(case, seed):
    s = prepare(case, seed)
    R, V = case["R"], case["V"]
    step = max(1, (1 << 27) // V)
    parts = []
    for lo in range(0, R, step):
        got = _exact_rows(case, s, lo, min(R, lo + step))
        if "dlogits" in got:  # held in 32 bits: the kernels' results have fewer
            got["dlogits"] = got["dlogits"].float()
        parts.append(got)
    out = {n: torch.cat([p[n] for p in parts]) for n in parts[0]}
    if case["op"] == "logprobs":
        if "logp" in out:
            out["logp"] = out["logp"].reshape(s["ids"].shape)
        if case["k"]:
            out["topk_ids"] = None
    if case["op"] == "distill":
        n = float(R) if s["mask"] is None else float(s["mask"].sum())
        out["loss"] = out["row_loss"].sum() / n
    return out
