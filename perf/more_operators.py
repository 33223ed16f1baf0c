"""Performance cases of the rollout's operators.

Three operators of the half of a training step that draws tokens:

* ``quantize``  8-bit codes of a matrix's rows and a scale for each: hidden states token by token, or a
                head's weight channel by channel;
* ``logits``    the logits of an 8-bit head, from codes with a scale for each token and each channel;
* ``verify``    verification of drafted tokens against the target's probabilities from given random
                numbers: what a sequence keeps of its drafts, and the token drawn after them.  Without
                drafts it is a decode step's sampling.

``run`` computes a case in plain torch operations, or with this package's kernels where ``own`` is true;
``exact`` computes it in fp64 from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EXACT_SUM = 1024    # products of 8-bit codes whose sum fp32 holds without rounding: 1024 * 128^2 = 2^24


def _quantize(R, D, dtype, **kw):
    return dict(dict(op="quantize", R=R, D=D, dtype=dtype, pad=0), **kw)


def _logits(R, D, V, dtype, **kw):
    return dict(dict(op="logits", R=R, D=D, V=V, dtype=dtype, pad=0), **kw)


def _verify(B, G, V, dtype, **kw):
    return dict(dict(op="verify", B=B, G=G, V=V, dtype=dtype, pad=0, draft="model", noise=0.5, sure=0.125, ragged=False, temperature=1.0), **kw)


def listed():
    return [
        # the hidden states of a decode step of a few sequences: latency alone
        _quantize(8, 1024, "bf16", name="quantize_decode"),
        # a head's weight, channel by channel, after an update
        _quantize(151936, 1024, "bf16", name="quantize_weight"),
        # rows of an odd length, padded, in fp32
        _quantize(5003, 1001, "f32", pad=7, name="quantize_odd_f32"),
        # a decode step of one sequence
        _logits(1, 1024, 151936, "bf16", name="logits_one_token"),
        # a decode step of a batch of sequences
        _logits(64, 1024, 151936, "bf16", name="logits_decode_batch"),
        # a target's pass over four drafted tokens and the next of a batch of sequences
        _logits(320, 1024, 151936, "bf16", name="logits_verify_batch"),
        # rollouts scored by a quantised reference policy
        _logits(4096, 1024, 151936, "bf16", name="logits_rollouts"),
        # an odd vocabulary and batch, a wider model, fp32 logits
        _logits(777, 2500, 50257, "f32", pad=3, name="logits_odd_f32"),
        # sampling of one sequence's next token: latency alone
        _verify(1, 0, 151936, "bf16", name="verify_sample_one"),
        # verification of four drafted tokens for each sequence of a decode batch
        _verify(64, 4, 151936, "bf16", name="verify_decode_batch"),
        # a rollout's whole batch
        _verify(512, 4, 151936, "bf16", name="verify_rollouts"),
        # drafts looked up in the prompt (no distribution), as many as were found, fp32 logits of an odd vocabulary
        _verify(201, 7, 50257, "f32", pad=3, draft="lookup", sure=0.6, ragged=True, temperature=0.8, name="verify_lookup_f32"),
    ]


def _spread(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999))))


def draw(rng: random.Random):
    op = rng.choice(["quantize", "logits", "logits", "verify", "verify", "verify"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    per = 4 if dtype == "f32" else 8           # row strides are multiples of 16 bytes
    if op == "quantize":
        D = _spread(rng, 60, 16384)
        R = _spread(rng, 1, min(200000, 151936 * 1024 // D // (2 if dtype == "f32" else 1)))
        return _quantize(R, D, dtype, pad=-D % per + per * rng.choice([0, 0, 1, 5]))
    V = _spread(rng, 300, 262144)
    if op == "logits":
        D = _spread(rng, 60, 8192)
        R = _spread(rng, 1, max(1, min(8192, 4096 * 1024 * 151936 // (D * V) // (2 if dtype == "f32" else 1))))
        return _logits(R, D, V, dtype, pad=-V % per + per * rng.choice([0, 0, 1, 5]))
    G = rng.choice([0, 1, 2, 3, 4, 5, 8])
    B = _spread(rng, 1, min(1024, max(1, 512 * 5 * 151936 // ((G + 1) * V) // (2 if dtype == "f32" else 1))))
    return _verify(B, G, V, dtype, pad=-V % per + per * rng.choice([0, 0, 1, 5]), draft=rng.choice(["model", "model", "lookup"]),
                   noise=rng.choice([0.3, 0.5, 1.0]), sure=rng.choice([0.125, 0.6]), ragged=rng.random() < 0.3,
                   temperature=rng.choice([1.0, 1.0, 0.7, 1.5]))


# ------------------------------------------------------------------ inputs
def _codes(x):
    """8-bit codes of each row of x and the scale they stand for."""
    s = (x.abs().amax(1) / 127).float()
    q = (x / torch.where(s > 0, s, 1.0)[:, None]).round_().clamp_(-127, 127)
    return q.to(torch.int8), s


def _code_rows(R, D, std, gen, dev):
    """Codes in rows of a multiple of 16 bytes, as a 16-byte aligned load wants them."""
    q, s = _codes(torch.randn((R, D), generator=gen, device=dev) * std)
    room = torch.zeros((R, -(-D // 16) * 16), dtype=torch.int8, device=dev)
    room[:, :D] = q
    return room[:, :D], s


def _token_logits(shape, ld, sure, gen, dev):
    """Peaked distributions: some rows where the model is sure of the next token."""
    z = torch.randn((*shape, ld), generator=gen, device=dev).mul_(3.0)
    hot = torch.randint(0, max(1, ld - 64), (*shape, 1), generator=gen, device=dev)
    boost = torch.where(torch.rand((*shape, 1), generator=gen, device=dev) < sure, 18.0, 0.0)
    return z.scatter_add_(-1, hot, boost)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 6271 + 29)
    c, dt = case, DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if c["op"] == "quantize":
        x = torch.randn((c["R"], c["D"] + c["pad"]), generator=gen, device=dev)
        x.mul_(torch.rand((c["R"], 1), generator=gen, device=dev).mul_(3).exp_())     # rows of different sizes
        x[:, :: 97] *= 8.0                                                            # channels that stand out
        s["x"] = x.to(dt)[:, :c["D"]]
        return s
    if c["op"] == "logits":
        s["h"], s["h_scale"] = _code_rows(c["R"], c["D"], 1.0, gen, dev)
        s["w"], s["w_scale"] = _code_rows(c["V"], c["D"], 3.0 / math.sqrt(c["D"]), gen, dev)
        s["out"] = torch.empty((c["R"], c["V"] + c["pad"]), dtype=dt, device=dev)[:, :c["V"]]
        # the scratch that a decode loop keeps
        s["workspace"] = torch.zeros(c["R"] * (c["D"] + 256) * 2 + 4096, dtype=torch.uint8, device=dev)
        return s
    B, G, V, ld, T = c["B"], c["G"], c["V"], c["V"] + c["pad"], c["temperature"]
    z = _token_logits((B, G + 1), ld, c["sure"], gen, dev)
    s["target"] = z.to(dt)[..., :V]
    if G:
        zq = z[:, :G] + torch.randn((B, G, ld), generator=gen, device=dev) * c["noise"]
        s["draft"] = zq.to(dt)[..., :V]
        del z, zq
        noise = torch.rand((B, G, V), generator=gen, device=dev).clamp_(min=1e-20).log_().neg_().log_().neg_()
        s["ids"] = noise.add_(s["draft"].float() / T).argmax(-1)
        s["draft_lse"] = (s["draft"].float() / T).logsumexp(-1) if c["draft"] == "model" else None
        if c["draft"] != "model":
            s["draft"] = None
    else:
        s["draft"] = s["draft_lse"] = None
        s["ids"] = torch.zeros((B, 0), dtype=torch.int64, device=dev)
    s["n_draft"] = torch.randint(-1, G + 1, (B,), generator=gen, device=dev, dtype=torch.int32) if c["ragged"] else None
    s["u"] = torch.rand((B, G + 1), generator=gen, device=dev, dtype=torch.float64)
    return s


# ------------------------------------------------------------------ the framework's kernels
def _run_own(s):
    from ppo_policy_loss_gb300 import torch_api
    op = s["case"]["op"]
    if op == "quantize":
        codes, scale = torch_api.quantize_rows(s["x"])
        return {"codes": codes, "scale": scale}
    if op == "logits":
        return torch_api.lmhead_logits_int8(s["h"], s["h_scale"], s["w"], s["w_scale"], out=s["out"], workspace=s["workspace"])
    out = torch_api.verify_drafts(s["target"], s["ids"], s["u"], draft_logits=s["draft"], draft_lse=s["draft_lse"], n_draft=s["n_draft"],
                                  temperature=s["case"]["temperature"])
    return {n: out[n] for n in ("tokens", "n_accepted", "logp", "lse")}


# ------------------------------------------------------------------ plain forms
def _plain_quantize(s):
    x = s["x"].float()
    # both quotients in 64 bits: the scale is rounded once, and what lies next to a half goes to its own side
    scale = (x.abs().amax(1).double() / 127).float()
    q = x.double().div_(torch.where(scale > 0, scale, 1.0).double()[:, None]).round_().clamp_(-127, 127)
    return {"codes": q.to(torch.int8), "scale": scale}


def _plain_logits(s):
    h, w, D = s["h"], s["w"], s["h"].shape[1]
    if D <= EXACT_SUM:
        acc = h.float() @ w.float().t()
    else:
        acc = torch.zeros((h.shape[0], w.shape[0]), dtype=torch.float64, device=h.device)
        for k in range(0, D, EXACT_SUM):
            acc += h[:, k:k + EXACT_SUM].float() @ w[:, k:k + EXACT_SUM].float().t()
        acc = acc.float()
    s["out"].copy_(acc.mul_(s["h_scale"][:, None]).mul_(s["w_scale"]))
    return s["out"]


def _plain_verify(s):
    T = s["case"]["temperature"]
    B, n_rows, V = s["target"].shape
    G, dev = n_rows - 1, s["target"].device
    # in 64 bits: a drawn token is where a sum over the vocabulary passes a border
    z = s["target"].double() / T
    m = z.amax(-1, keepdim=True)
    z -= m
    e = z.exp()
    total = e.sum(-1, keepdim=True)
    lse = (m + total.log())[..., 0]
    n = torch.full((B,), G, device=dev) if s["n_draft"] is None else s["n_draft"].long()
    seq, at = torch.arange(B, device=dev), torch.arange(n_rows, device=dev)
    ids = s["ids"]
    p = e[:, :G].gather(-1, ids[..., None])[..., 0] / total[:, :G, 0]
    q = torch.ones_like(p)
    if s["draft"] is not None:
        q = (s["draft"].gather(-1, ids[..., None])[..., 0].double() / T - s["draft_lse"]).exp()
    ok = (s["u"][:, :G] * q < p) & (at[:G] < n[:, None])
    kept = ok.long().cumprod(1).sum(1)
    weight = e[seq, kept] / total[seq, kept]
    if G:
        lost = (kept < n)[:, None]
        row = kept.clamp(max=G - 1)
        if s["draft"] is not None:
            rest = (weight - (s["draft"][seq, row].double() / T - s["draft_lse"][seq, row][:, None]).exp()).clamp_(min=0.0)
        else:
            rest = weight.scatter(1, ids[seq, row][:, None], 0.0)
        lost = lost & (rest.sum(1, keepdim=True) > 0)
        weight = torch.where(lost, rest, weight)
    upto = weight.cumsum(1)
    last = (weight > 0).long().mul_(torch.arange(V, device=dev)).amax(1)
    new = torch.minimum((upto <= s["u"][:, G:] * upto[:, -1:]).sum(1), last)
    tokens = torch.cat([ids, new[:, None]], 1).scatter(1, kept[:, None], new[:, None])
    on = (at <= kept[:, None]) & (n >= 0)[:, None]
    tokens = torch.where(on, tokens, -1)
    logp = (z.gather(-1, tokens.clamp(min=0)[..., None]) - total.log())[..., 0]
    return {"tokens": tokens, "n_accepted": kept, "logp": torch.where(on, logp, 0.0).float(), "lse": torch.where(on, lse, 0.0).float()}


def run(state):
    if own:
        return _run_own(state)
    return {"quantize": _plain_quantize, "logits": _plain_logits, "verify": _plain_verify}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    es = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "quantize":
        n = case["R"] * case["D"]
        return {"bytes": n * (es + 1.0) + 4 * case["R"], "flops": 4.0 * n}
    if case["op"] == "logits":
        R, D, V = case["R"], case["D"], case["V"]
        return {"bytes": 1.0 * (R + V) * D + R * V * es + 4 * (R + V), "flops": 2.0 * R * V * D}
    # a sequence's rows up to its first rejection, and there the draft's
    rows, lost = _rows_read(case)
    return {"bytes": case["B"] * (rows + lost) * case["V"] * es, "flops": case["B"] * (6.0 * rows + 8 * lost) * case["V"]}


def _rows_read(case):
    """Mean number of a sequence's target and draft rows that decide its tokens.  Logits N(0, 9) with noise of deviation s keep a
    draft with probability 2 Phi(-s / 2), rows with one sure token nine times in ten; a looked-up token is kept where its row is sure."""
    G, sure = case["G"], case["sure"]
    if case["draft"] == "model":
        keep, drafts = sure * 0.9 + (1 - sure) * math.erfc(case["noise"] / case["temperature"] / math.sqrt(8)), 1.0
    else:
        keep, drafts = sure * 0.6, 0.0
    lengths = range(-1, G + 1) if case["ragged"] else [G]
    rows = lost = 0.0
    for n in lengths:
        rows += sum(keep ** i for i in range(n + 1))
        lost += (1 - keep ** n) * drafts if n > 0 else 0.0
    return rows / len(lengths), lost / len(lengths)


# ------------------------------------------------------------------ the definitions in fp64
def _exact_verify(case, s):
    T, G, V = case["temperature"], case["G"], case["V"]
    B = case["B"]
    names = ("tokens", "n_accepted", "logp", "lse")
    out = {"tokens": torch.full((B, G + 1), -1, dtype=torch.int64), "n_accepted": torch.zeros(B, dtype=torch.int64),
           "logp": torch.zeros((B, G + 1), dtype=torch.float64), "lse": torch.zeros((B, G + 1), dtype=torch.float64)}
    u, ids = s["u"].cpu(), s["ids"].cpu()
    counts = [G] * B if s["n_draft"] is None else s["n_draft"].cpu().tolist()
    for b in range(B):
        for i in range(counts[b] + 1):
            row = s["target"][b, i].to(torch.float64) / T
            lse = torch.logsumexp(row, -1)
            logp = row - lse
            p = logp.exp()
            out["lse"][b, i] = lse
            draft = q = None
            if i < counts[b]:
                draft = int(ids[b, i])
                if s["draft"] is None:
                    q = torch.zeros_like(p)
                    q[draft] = 1.0
                else:
                    q = torch.exp(s["draft"][b, i].to(torch.float64) / T - s["draft_lse"][b, i].double())
                if float(u[b, i]) * float(q[draft]) < float(p[draft]):
                    out["tokens"][b, i], out["logp"][b, i] = draft, logp[draft]
                    out["n_accepted"][b] += 1
                    continue
                p = torch.relu(p - q) if bool((p > q).any()) else p
            edges = torch.cumsum(p, 0)
            at = int(torch.searchsorted(edges, edges[-1:] * float(u[b, G]), right=True))
            if at >= V or not float(p[at]) > 0:
                at = int(torch.nonzero(p)[-1])
            out["tokens"][b, i], out["logp"][b, i] = at, logp[at]
            break
    dev = s["u"].device
    return {n: out[n].to(dev) for n in names}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"].to(torch.float64)
        scale = x.abs().max(dim=1).values / 127.0
        # the codes are of the scale as it is held, in 32 bits
        held = scale.float().double()
        return {"codes": torch.clip(torch.round(x / torch.where(held > 0, held, 1.0).unsqueeze(1)), -127, 127).to(torch.int8), "scale": scale}
    if case["op"] == "verify":
        return _exact_verify(case, s)
    step = max(1, (1 << 28) // case["V"])
    weight = s["w"].double().t()
    parts = [(s["h"][lo:lo + step].double() @ weight * s["h_scale"][lo:lo + step].double().unsqueeze(1) * s["w_scale"].double()).float()
             for lo in range(0, case["R"], step)]
    return torch.cat(parts)
