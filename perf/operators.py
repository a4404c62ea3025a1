"""Cases that measure the sequence operators: embedding, gated linear recurrence, distillation loss.

Each case is one pass through one operator.  With ``own`` false, ``run``
computes it in plain 32-bit torch operations; with ``own`` true it makes the
library's calls.  ``exact`` gives the same outputs from the definitions in
64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decoding step of 64 sequences: latency of a single small gather
        {"name": "embed_decode", "op": "embed", "n": 64, "vocab": 32000, "dim": 768, "dtype": "bf16"},
        # token ids of a long prompt batch (64 x 1024), fp32 table
        {"name": "embed_prompt", "op": "embed", "n": 65536, "vocab": 50257, "dim": 1024, "dtype": "f32"},
        # gradient of the table for the benchmark's token count (8 x 1024, width 768), bf16 weights and gradient
        {"name": "embed_grad_step", "op": "embed_grad", "n": 8192, "vocab": 50257, "dim": 768, "dtype": "bf16"},
        # gradient for a large batch of an odd width (no 16-byte rows) over a small vocabulary: long runs of one token
        {"name": "embed_grad_ragged", "op": "embed_grad", "n": 131071, "vocab": 8001, "dim": 771, "dtype": "f32"},
        # one token for each of 64 sequences, state updated from the last one: serving
        {"name": "glr_step", "op": "glr", "batch": 64, "time": 1, "width": 768, "dtype": "bf16", "fused": False, "reset": False},
        # prompt of odd length and odd width: forward only
        {"name": "glr_prompt_odd", "op": "glr", "batch": 3, "time": 4097, "width": 1537, "dtype": "bf16", "fused": False, "reset": False},
        # training step at the benchmark's 8 x 1024 tokens of width 768; inputs are slices of one projection, packed documents
        {"name": "glr_train", "op": "glr_grad", "batch": 8, "time": 1024, "width": 768, "dtype": "bf16", "fused": True, "reset": True},
        # one long sequence, fp32, training
        {"name": "glr_train_long", "op": "glr_grad", "batch": 1, "time": 65536, "width": 1000, "dtype": "f32", "fused": False, "reset": False},
        # evaluation of 512 tokens against a teacher's top 32
        {"name": "distill_eval", "op": "distill", "n": 512, "vocab": 50257, "k": 32, "temp": 1.0, "dtype": "bf16"},
        # training step on 8192 tokens, loss and its gradient, odd row length
        {"name": "distill_train", "op": "distill_grad", "n": 8192, "vocab": 50257, "k": 64, "temp": 2.0, "dtype": "bf16"},
        # fp32 logits, few teacher entries
        {"name": "distill_train_f32", "op": "distill_grad", "n": 1500, "vocab": 32003, "k": 7, "temp": 1.0, "dtype": "f32"},
        # a large vocabulary: one row does not fit an SM's shared memory
        {"name": "distill_train_wide", "op": "distill_grad", "n": 2048, "vocab": 200000, "k": 256, "temp": 1.5, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "glr", "glr_grad", "distill", "distill_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("embed"):
        n = _log_int(rng, 1, 131071)
        dim = rng.choice([1, 2, 8]) * _log_int(rng, 8, 128) + rng.choice([0, 0, 1, 3])
        return {"op": op, "n": n, "vocab": _log_int(rng, 500, 50000), "dim": min(dim, 771), "dtype": dtype}
    if op.startswith("glr"):
        batch, width = _log_int(rng, 1, 64), rng.choice([1, 2, 8]) * _log_int(rng, 16, 200) + rng.choice([0, 0, 0, 1])
        time = _log_int(rng, 1, max(1, min(65536, 48_000_000 // (batch * width))))
        return {"op": op, "batch": batch, "time": time, "width": width, "dtype": dtype,
                "fused": rng.random() < 0.4, "reset": rng.random() < 0.4}
    vocab = _log_int(rng, 1000, 200000)
    n = _log_int(rng, 1, max(2, min(8192, 300_000_000 // vocab)))
    return {"op": op, "n": n, "vocab": vocab, "k": _log_int(rng, 1, 256), "temp": rng.choice([0.5, 1.0, 2.0, 4.0]),
            "dtype": dtype}


def _tokens(n, vocab, gen):
    # frequencies fall as 1/rank, as words' do
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        t = torch.randn(*shape, generator=gen, device="cuda")
        return t.mul_(std).add_(mean).to(dtype)

    s = {"case": dict(case)}
    op = case["op"]
    if op.startswith("embed"):
        n, vocab, dim = case["n"], case["vocab"], case["dim"]
        s["ids"] = _tokens(n, vocab, gen)
        s["scale"] = math.sqrt(dim)
        if op == "embed":
            s["weight"] = normal(vocab, dim, std=dim ** -0.5)
        else:
            s["dy"] = normal(n, dim, std=0.1)
            s["vocab"] = vocab
    elif op.startswith("glr"):
        b, t, c = case["batch"], case["time"], case["width"]
        if case["fused"]:
            # x, r and g as one projection's slices
            s["x"], s["r"], s["g"] = normal(b, t, 3 * c).split(c, dim=-1)
        else:
            s["x"], s["r"], s["g"] = normal(b, t, c), normal(b, t, c), normal(b, t, c)
        # memory of two to some hundreds of steps
        tau = torch.exp(torch.rand(c, generator=gen, device="cuda") * math.log(150.0)) * 2.0
        s["decay"] = torch.log(torch.expm1(2.0 / tau))
        s["h0"] = normal(b, c, dtype=torch.float32)
        s["reset"] = (torch.rand(b, t, generator=gen, device="cuda") < 1.0 / 256) if case["reset"] else None
        if op == "glr_grad":
            s["dy"] = normal(b, t, c)
            s["dh_last"] = normal(b, c, dtype=torch.float32)
    else:
        n, vocab, k = case["n"], case["vocab"], case["k"]
        z = torch.randn(n, vocab, generator=gen, device="cuda").mul_(2.0)
        # the teacher's top logits, in falling order, at different tokens; some rows keep fewer of them (-1: no entry)
        gaps = torch.rand(n, k, generator=gen, device="cuda").log_().neg_().mul_(2.0 / torch.arange(1, k + 1, device="cuda"))
        teacher = 14.0 - gaps.cumsum(1)
        start = torch.randint(0, vocab, (n, 1), generator=gen, device="cuda")
        step = max(1, vocab // k)
        jitter = torch.randint(0, step, (n, k), generator=gen, device="cuda")
        ids = (start + torch.arange(k, device="cuda") * step + jitter * (jitter < step)) % vocab if step > 1 else \
            (start + torch.arange(k, device="cuda")) % vocab
        # the student has learned part of it
        z.scatter_add_(1, ids, teacher * 0.6 + torch.randn(n, k, generator=gen, device="cuda"))
        s["z"] = z.to(dt)
        kept = torch.randint(max(1, k // 2), k + 1, (n, 1), generator=gen, device="cuda")
        s["ids"] = torch.where(torch.arange(k, device="cuda") < kept, ids, -1).int()
        s["teacher"] = teacher
        # padded tokens weigh nothing
        s["weight"] = (torch.rand(n, generator=gen, device="cuda") < 15.0 / 16).float() / n
        s["temp"] = float(case["temp"])
    return s


# ---- plain forms ----
def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 (h before the first step is 0), by doubling."""
    t, d = a.shape[1], 1
    while d < t:
        b = torch.cat([b[:, :d], b[:, d:] + a[:, d:] * b[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return b


def _plain_embed(s):
    return (s["weight"][s["ids"]].float() * s["scale"]).to(s["weight"].dtype)


def _plain_embed_grad(s):
    dw = torch.zeros(s["vocab"], s["dy"].shape[1], device="cuda")
    dw.index_add_(0, s["ids"], s["dy"].float())
    return (dw * s["scale"]).to(s["dy"].dtype)


def _glr_parts(s):
    x, r, g = s["x"].float(), s["r"].float(), s["g"].float()
    sr, sg = torch.sigmoid(r), torch.sigmoid(g)
    log_a = -torch.nn.functional.softplus(s["decay"]) * sr
    a = torch.exp(log_a)
    m = torch.sqrt(-torch.expm1(2 * log_a))
    keep = a if s["reset"] is None else torch.where(s["reset"][..., None], 0.0, a)
    b = m * sg * x
    b[:, 0] += keep[:, 0] * s["h0"]
    return x, sr, sg, log_a, a, m, keep, _scan(keep, b)


def _plain_glr(s):
    h = _glr_parts(s)[-1]
    return {"y": h.to(s["x"].dtype), "h_last": h[:, -1]}


def _plain_glr_grad(s):
    x, sr, sg, log_a, a, m, keep, h = _glr_parts(s)
    dt = s["x"].dtype
    d = s["dy"].float().clone()
    d[:, -1] += s["dh_last"]
    # d_t = dy_t + keep_{t+1} d_{t+1}
    rev = torch.cat([torch.zeros_like(keep[:, :1]), keep[:, 1:].flip(1)], 1)
    d = _scan(rev, d.flip(1)).flip(1)
    before = torch.cat([s["h0"][:, None], h[:, :-1]], 1)
    if s["reset"] is not None:
        before = torch.where(s["reset"][..., None], 0.0, before)
    dlog = d * (a * before - a * a / m * sg * x)
    dx = d * m * sg
    dg = dx * x * (1 - sg)
    dr = dlog * log_a * (1 - sr)
    ddecay = (-(dlog * sr).sum((0, 1), dtype=torch.float64) * torch.sigmoid(s["decay"])).float()
    return {"y": h.to(dt), "h_last": h[:, -1], "dx": dx.to(dt), "dr": dr.to(dt), "dg": dg.to(dt),
            "ddecay": ddecay, "dh0": keep[:, 0] * d[:, 0]}


def _distill_parts(s):
    valid = s["ids"] >= 0
    ids = torch.where(valid, s["ids"], 0).long()
    t = torch.where(valid, s["teacher"] / s["temp"], -math.inf)
    e = torch.exp(t - t.amax(1, keepdim=True))
    esum = e.sum(1, keepdim=True)
    p = e / esum
    logp = torch.where(valid, t - t.amax(1, keepdim=True) - torch.log(esum), 0.0)
    z = s["z"].float() / s["temp"]
    z = z - z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z).sum(1, keepdim=True))
    loss = (p * (logp - z.gather(1, ids) + lse)).sum(1)
    return ids, p, z, lse, loss * s["weight"] * s["temp"] ** 2


def _plain_distill(s):
    return _distill_parts(s)[-1]


def _plain_distill_grad(s):
    ids, p, z, lse, loss = _distill_parts(s)
    dz = torch.exp(z)
    dz = dz / dz.sum(1, keepdim=True)
    dz.scatter_add_(1, ids, -p)
    dz *= (s["weight"] * s["temp"])[:, None]
    return {"loss": loss, "dlogits": dz.to(s["z"].dtype)}


# ---- the library's calls ----
def _own_embed(s):
    from kolmogorov_arnold_network_b200 import layer
    return layer.embed_forward(s["ids"], s["weight"], s["scale"])


def _own_embed_grad(s):
    from kolmogorov_arnold_network_b200 import layer
    return layer.embed_backward(s["ids"], s["dy"], s["vocab"], s["scale"], grad_dtype=s["dy"].dtype)


def _own_glr(s):
    from kolmogorov_arnold_network_b200 import layer
    y, h_last, _ = layer.glr_forward(s["x"], s["r"], s["g"], s["decay"], h0=s["h0"], reset=s["reset"])
    return {"y": y, "h_last": h_last}


def _own_glr_grad(s):
    from kolmogorov_arnold_network_b200 import layer
    y, h_last, kept = layer.glr_forward(s["x"], s["r"], s["g"], s["decay"], h0=s["h0"], reset=s["reset"], keep=True)
    dx, dr, dg, ddecay, dh0 = layer.glr_backward(s["x"], s["r"], s["g"], s["decay"], kept, s["dy"], reset=s["reset"],
                                                 dh_last=s["dh_last"])
    return {"y": y, "h_last": h_last, "dx": dx, "dr": dr, "dg": dg, "ddecay": ddecay, "dh0": dh0}


def _own_distill(s):
    from kolmogorov_arnold_network_b200 import layer
    loss, _ = layer.distill_forward(s["z"], s["ids"], s["teacher"], s["temp"], weight=s["weight"])
    return loss


def _own_distill_grad(s):
    from kolmogorov_arnold_network_b200 import layer
    loss, dz = layer.distill_loss_grad(s["z"], s["ids"], s["teacher"], s["temp"], weight=s["weight"])
    return {"loss": loss, "dlogits": dz}


_PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "glr": _plain_glr, "glr_grad": _plain_glr_grad,
          "distill": _plain_distill, "distill_grad": _plain_distill_grad}
_OWN = {"embed": _own_embed, "embed_grad": _own_embed_grad, "glr": _own_glr, "glr_grad": _own_glr_grad,
        "distill": _own_distill, "distill_grad": _own_distill_grad}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def work(case):
    op, esz = case["op"], (2 if case["dtype"] == "bf16" else 4)
    if op.startswith("embed"):
        n, vocab, dim = case["n"], case["vocab"], case["dim"]
        if op == "embed_grad":
            return {"bytes": 8 * n + esz * dim * (n + vocab), "flops": n * dim}
        edge = torch.log(torch.arange(1, vocab + 2, dtype=torch.float64)) / math.log(vocab + 1.0)
        rows = float((1 - (1 - edge.diff()) ** n).sum())   # distinct tokens to be expected
        return {"bytes": int(8 * n + esz * dim * (n + rows)), "flops": n * dim}
    if op.startswith("glr"):
        b, t, c = case["batch"], case["time"], case["width"]
        e = b * t * c
        extra = 4 * c + 8 * b * c + (b * t if case["reset"] else 0)
        if op == "glr":
            return {"bytes": 4 * esz * e + extra, "flops": 20 * e}
        # y, dx, dr and dg out; x, r, g and dy in
        return {"bytes": 8 * esz * e + extra + 4 * c + 8 * b * c, "flops": 60 * e}
    n, vocab, k = case["n"], case["vocab"], case["k"]
    small = n * (8 * k + 8)
    if op == "distill":
        return {"bytes": esz * n * vocab + small, "flops": 4 * n * vocab}
    return {"bytes": 2 * esz * n * vocab + small, "flops": 7 * n * vocab}


# ---- the definitions in 64 bits ----
def _exact_embed_grad(s):
    # rows of one token side by side, then differences of their running sums
    order = torch.argsort(s["ids"], stable=True)
    run_sum = s["dy"][order].double().cumsum(0)
    end = torch.bincount(s["ids"], minlength=s["vocab"]).cumsum(0)
    upto = torch.cat([run_sum.new_zeros(1, run_sum.shape[1]), run_sum])[end]
    return s["scale"] * torch.diff(upto, dim=0, prepend=upto.new_zeros(1, upto.shape[1]))


def _exact_glr(s, grad):
    x, r, g = (s[k].double() for k in ("x", "r", "g"))
    dec = s["decay"].double()
    lam = torch.log1p(torch.exp(-dec.abs())) + dec.clamp(min=0)
    sr, sg = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-g))
    a = torch.exp(-lam * sr)
    m = torch.sqrt(-torch.expm1(-2 * lam * sr))
    u = sg * x
    through = a if s["reset"] is None else a * (~s["reset"])[..., None]
    inp = m * u
    before = torch.empty_like(x)
    h = s["h0"].double()
    for t in range(x.shape[1]):
        before[:, t] = h
        h = torch.addcmul(inp[:, t], through[:, t], h)
    y = torch.cat([before[:, 1:], h[:, None]], 1)
    out = {"y": y, "h_last": h}
    if not grad:
        return out
    dy = s["dy"].double()
    d = torch.empty_like(x)
    flow = s["dh_last"].double()
    for t in range(x.shape[1] - 1, -1, -1):
        d[:, t] = dy[:, t] + flow
        flow = through[:, t] * d[:, t]
    # with q = lam * sr:  dh/dq = -through * before + u a^2 / m
    dq = d * (-through * before + u * a * a / m)
    out["dx"] = d * m * sg
    out["dr"] = dq * lam * sr * (1 - sr)
    out["dg"] = d * m * x * sg * (1 - sg)
    out["ddecay"] = (dq * sr).sum((0, 1)) / (1 + torch.exp(-dec))
    out["dh0"] = flow
    return out


def _exact_distill(s, grad):
    n, vocab = s["z"].shape
    tau = s["temp"]
    loss = torch.zeros(n, dtype=torch.float64, device="cuda")
    dz = torch.empty(n, vocab, dtype=torch.float64, device="cuda") if grad else None
    rows = max(1, 50_000_000 // vocab)
    for i in range(0, n, rows):
        sl = slice(i, min(n, i + rows))
        ids, t, w = s["ids"][sl].long(), s["teacher"][sl].double() / tau, s["weight"][sl].double()
        there = ids >= 0
        p = torch.where(there, torch.exp(t - torch.logsumexp(t.masked_fill(~there, -math.inf), 1, keepdim=True)), 0.0)
        logq = s["z"][sl].double() / tau
        logq = logq - torch.logsumexp(logq, 1, keepdim=True)
        at = logq.gather(1, ids.clamp(min=0))
        loss[sl] = w * tau * tau * torch.where(there, p * (torch.log(p) - at), 0.0).sum(1)
        if grad:
            target = torch.zeros_like(logq).scatter_add_(1, ids.clamp(min=0), p)
            dz[sl] = (w * tau)[:, None] * (torch.exp(logq) - target)
    return {"loss": loss, "dlogits": dz} if grad else loss


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        return s["weight"].double()[s["ids"]] * s["scale"]
    if op == "embed_grad":
        return _exact_embed_grad(s)
    if op.startswith("glr"):
        return _exact_glr(s, op == "glr_grad")
    return _exact_distill(s, op == "distill_grad")
