"""The operators around the fused norm projections, as they are measured: the
cases, their inputs, the plain form of each operator in elementary torch
operations, the call that a user makes of it, and its definition in 64 bits.

  proj       y = act(x @ W + bias) + residual: the projection that takes an
             attention or feed-forward result back into the residual stream
  moe        a whole mixture-of-experts feed-forward layer for a few tokens:
             RMSNorm, router, the chosen experts' SwiGLU, the weighted sum
  logprobs   log probabilities of given tokens with entropy and the top
             alternatives, from the logits of a head projection
  logprobs_backward   the gradient of the log probabilities and entropies with
             respect to the logits
"""
from __future__ import annotations

import math

import torch

own = False

EPS = 1e-6
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # attention output projection of one decoded token, added to the residual stream
        dict(name="proj_decode_m1", op="proj", M=1, K=4096, N=4096, ldx=4096, ldw=4096, bias=False, act="none",
             residual=True, out="bf16"),
        # a ragged small batch through a biased, activated projection; no size is a multiple of a tile
        dict(name="proj_ragged_m45", op="proj", M=45, K=2051, N=4099, ldx=2056, ldw=4104, bias=True,
             act="gelu_tanh", residual=False, out="fp32"),
        # a chunk of a prompt through the down projection of the FFN (K = 14336)
        dict(name="proj_chunk_m300", op="proj", M=300, K=14336, N=4096, ldx=14336, ldw=4096, bias=False, act="none",
             residual=True, out="bf16"),
        # a whole prefill batch through the same down projection, with a bias
        dict(name="proj_prefill_m4096", op="proj", M=4096, K=14336, N=4096, ldx=14336, ldw=4096, bias=True,
             act="none", residual=True, out="bf16"),
        # one decoded token, 8 of 64 experts
        dict(name="moe_decode_m1", op="moe", M=1, d=2048, I=1024, E=64, k=8, score="softmax", select_bias=False,
             renorm=True, route_scale=1.0, residual=True),
        # a small decode batch, 8 of 128 narrow experts, sigmoid scores with a selection bias
        dict(name="moe_batch_m13", op="moe", M=13, d=2048, I=768, E=128, k=8, score="sigmoid", select_bias=True,
             renorm=True, route_scale=2.5, residual=True),
        # the largest decode batch, 2 of 8 experts of the FFN's size: every expert is read
        dict(name="moe_wide_m64", op="moe", M=64, d=4096, I=14336, E=8, k=2, score="softmax", select_bias=False,
             renorm=True, route_scale=1.0, residual=True),
        # one sampled token with 20 alternatives
        dict(name="logprobs_m1", op="logprobs", M=1, V=131072, ld=131072, dtype="bf16", top_k=20, scale=1.0,
             masked=0.0),
        # a decode batch under a grammar mask; odd vocabulary, rows at odd addresses
        dict(name="logprobs_ragged_m33", op="logprobs", M=33, V=50021, ld=50021, dtype="fp32", top_k=5, scale=0.7,
             masked=0.4),
        # scoring of a prompt batch
        dict(name="logprobs_score_m4096", op="logprobs", M=4096, V=131072, ld=131072, dtype="bf16", top_k=8,
             scale=1.0, masked=0.0),
        # gradient of a small ragged batch
        dict(name="logprobs_backward_m61", op="logprobs_backward", M=61, V=32003, ld=32003, dtype="fp32", scale=1.0,
             masked=0.1, entropy_grad=True),
        # gradient of a training batch
        dict(name="logprobs_backward_m2048", op="logprobs_backward", M=2048, V=131072, ld=131072, dtype="bf16",
             scale=1.0, masked=0.0, entropy_grad=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["proj", "moe", "logprobs", "logprobs_backward"])
    if op == "proj":
        K, N = _log_int(rng, 16, 16384), _log_int(rng, 16, 16384)
        if rng.random() < 0.5:   # half of them at ordinary multiples
            K, N = (K + 63) // 64 * 64, (N + 63) // 64 * 64
        M = _log_int(rng, 1, 8192)
        M = max(1, min(M, 4096 * 14336 * 4096 // (K * N)))
        pad = 8 * rng.randint(0, 2)
        return dict(op=op, M=M, K=K, N=N, ldx=(K + 7) // 8 * 8 + pad, ldw=(N + 7) // 8 * 8 + pad,
                    bias=rng.random() < 0.5, act=rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"]),
                    residual=rng.random() < 0.6, out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "moe":
        E = _log_int(rng, 2, 256)
        d = 64 * _log_int(rng, 2, 80)
        most = max(1, min(112, 8 * 4096 * 14336 // (E * d * 128)))
        I = 128 * _log_int(rng, 1, most)
        return dict(op=op, M=_log_int(rng, 1, 64), d=d, I=I, E=E, k=rng.randint(1, min(8, E)),
                    score=rng.choice(["softmax", "sigmoid"]), select_bias=rng.random() < 0.5,
                    renorm=rng.random() < 0.7, route_scale=rng.choice([1.0, 2.5]), residual=rng.random() < 0.7)
    most = 1 << 28 if op == "logprobs_backward" else 1 << 29
    V = _log_int(rng, 2, 262144)
    M = max(1, min(_log_int(rng, 1, 8192), most // V))
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if dtype == "fp32":
        M = max(1, M // 2)
    c = dict(op=op, M=M, V=V, ld=V + rng.choice([0, 0, 1, 8]), dtype=dtype, scale=rng.choice([1.0, 0.7, 1.6]),
             masked=rng.choice([0.0, 0.0, 0.3, 0.9]))
    if op == "logprobs":
        c["top_k"] = rng.randint(0, min(32, V))
    else:
        c["entropy_grad"] = rng.random() < 0.5
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _rows(M, d, gen):
    """Activations with a scale of their own for each row."""
    s = torch.exp(torch.empty(M, 1, device="cuda").uniform_(math.log(0.1), math.log(10.0), generator=gen))
    return torch.randn(M, d, device="cuda", generator=gen) * s


def _weight(*shape, std, gen):
    return (torch.randn(*shape, device="cuda", generator=gen, dtype=torch.bfloat16)).mul_(std)


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "proj":
        M, K, N = case["M"], case["K"], case["N"]
        dt = _DTYPES[case["out"]]
        x = torch.empty(M, case["ldx"], device="cuda", dtype=torch.bfloat16)
        x.copy_(torch.randn(M, case["ldx"], device="cuda", generator=gen))
        s["x"] = x[:, :K]
        s["W"] = _weight(K, case["ldw"], std=K ** -0.5, gen=gen)[:, :N]
        s["bias"] = torch.randn(N, device="cuda", generator=gen) if case["bias"] else None
        s["residual"] = torch.randn(M, N, device="cuda", generator=gen).mul_(3).to(dt) if case["residual"] else None
        s["out"] = torch.empty(M, N, device="cuda", dtype=dt)
    elif op == "moe":
        M, d, I, E = case["M"], case["d"], case["I"], case["E"]
        s["x"] = _rows(M, d, gen).bfloat16()
        s["g"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=gen)).bfloat16().float()
        s["router"] = _weight(E, d, std=2 * d ** -0.5, gen=gen)
        # gate and up columns alternate in groups of 128, the norm gain folded in
        s["Wgu"] = _weight(E, d, 2 * I, std=d ** -0.5, gen=gen)
        s["Wd"] = _weight(E, I, d, std=2 * I ** -0.5, gen=gen)
        s["select_bias"] = torch.randn(E, device="cuda", generator=gen) * 0.2 if case["select_bias"] else None
        s["residual"] = s["x"] if case["residual"] else None
        s["out"] = torch.empty(M, d, device="cuda", dtype=torch.bfloat16)
    else:
        M, V, ld = case["M"], case["V"], case["ld"]
        dt = _DTYPES[case["dtype"]]
        buf = torch.empty(M, ld, device="cuda", dtype=dt)
        step = max(1, (1 << 26) // ld)
        for a in range(0, M, step):
            b = min(M, a + step)
            z = torch.randn(b - a, ld, device="cuda", generator=gen)
            # some rows flat, some with a clear favourite
            z *= torch.empty(b - a, 1, device="cuda").uniform_(0.5, 4.0, generator=gen)
            if case["masked"]:
                z[torch.rand(b - a, ld, device="cuda", generator=gen) < case["masked"]] = -math.inf
            buf[a:b] = z
        s["logits"] = buf[:, :V]
        t = torch.randint(0, V, (M,), device="cuda", generator=gen, dtype=torch.int32)
        if M > 4:
            t[torch.arange(3, M, 7, device="cuda")] = -1          # padding: no token
            if case["masked"]:
                s["logits"][2] = -math.inf                        # a mask that leaves nothing
        s["targets"] = t
        if op == "logprobs_backward":
            lse, H = [], []
            for a in range(0, M, step):
                z = s["logits"][a:a + step].double() * case["scale"]
                l = torch.logsumexp(z, -1)
                p = torch.exp(z - torch.where(torch.isinf(l), 0.0, l)[:, None])
                h = l - torch.where(p > 0, p * z, 0.0).sum(-1)
                lse.append(l)
                H.append(torch.where(torch.isinf(l), 0.0, h))
            s["lse"], s["entropy"] = torch.cat(lse).float(), torch.cat(H).float()
            s["grad_logprob"] = torch.randn(M, device="cuda", generator=gen)
            s["grad_entropy"] = torch.randn(M, device="cuda", generator=gen) * 0.1 if case["entropy_grad"] else None
            s["out"] = torch.empty(M, V, device="cuda", dtype=dt)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from rmsnorm_linear_projection_flashnorm_b200 import torch_api as T
        s["T"] = T
        if case["op"] in ("proj", "moe"):
            s["ws"] = T.Workspace("cuda")      # kept between calls, as a serving loop does
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _act(z, name):
    if name == "relu":
        return torch.maximum(z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _plain_proj(s):
    c = s["case"]
    z = s["x"].float() @ s["W"].float()
    if s["bias"] is not None:
        z = z + s["bias"]
    z = _act(z, c["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(_DTYPES[c["out"]])


def _split_gate_up(W, I):
    W = W.reshape(W.shape[0], I // 128, 2, 128)
    return W[:, :, 0].reshape(-1, I), W[:, :, 1].reshape(-1, I)


def _plain_moe(s):
    c = s["case"]
    M, I, E, k = c["M"], c["I"], c["E"], c["k"]
    x = s["x"].float()
    r64 = torch.rsqrt(s["x"].double().square().mean(-1, keepdim=True) + EPS)
    # which experts are chosen is a comparison of close values: 64 bits
    logits = r64 * ((s["x"].double() * s["g"].double()) @ s["router"].double().t())
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.max(-1, keepdim=True).values)
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    key = logits if s["select_bias"] is None else score + s["select_bias"].double()
    ids = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    w = w * c["route_scale"]
    h = x * r64.float()
    y = s["residual"].float() if s["residual"] is not None else torch.zeros_like(x)
    per_expert = torch.zeros(M, E, device=x.device).scatter_(1, ids, w.float())
    for e in range(E):
        Wg, Wu = _split_gate_up(s["Wgu"][e].float(), I)
        gate = h @ Wg
        a = gate / (1 + torch.exp(-gate)) * (h @ Wu)
        y = y + per_expert[:, e:e + 1] * (a @ s["Wd"][e].float())
    return y.bfloat16(), ids.int(), w.float()


def _plain_logprobs(s):
    c = s["case"]
    M, V = s["logits"].shape
    out = []
    step = max(1, (1 << 26) // V)
    for a in range(0, M, step):
        raw = s["logits"][a:a + step].float()
        t = s["targets"][a:a + step].long()
        z = raw * c["scale"]
        m = z.max(-1, keepdim=True).values
        m = torch.where(torch.isinf(m) & (m < 0), 0.0, m)
        e = torch.exp(z - m)
        tot = e.sum(-1, keepdim=True)
        none = tot[:, 0] == 0
        lse = (m + torch.log(tot))[:, 0]
        H = torch.log(tot[:, 0]) - torch.where(e > 0, (z - m) * e, 0.0).sum(-1) / tot[:, 0]
        H = torch.where(none, 0.0, H)
        lp = z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0] - lse
        lp = torch.where(none, -math.inf, lp)
        lp = torch.where(t < 0, 0.0, lp)
        k = c["top_k"]
        idx = torch.sort(raw, dim=-1, descending=True, stable=True).indices[:, :k]
        top = z.gather(1, idx) - lse[:, None]
        top = torch.where(none[:, None], -math.inf, top)
        out.append((lp, H, lse, idx.int(), top))
    return tuple(torch.cat(v) for v in zip(*out))


def _plain_logprobs_backward(s):
    c = s["case"]
    M, V = s["logits"].shape
    step = max(1, (1 << 26) // V)
    out = s["out"]
    for a in range(0, M, step):
        z = s["logits"][a:a + step].float() * c["scale"]
        t = s["targets"][a:a + step].long()
        lse = s["lse"][a:a + step][:, None]
        gl = torch.where(t < 0, 0.0, s["grad_logprob"][a:a + step])[:, None]
        logp = z - torch.where(torch.isinf(lse), 0.0, lse)
        p = torch.exp(logp)
        d = -gl * p
        if s["grad_entropy"] is not None:
            ent = p * (torch.where(p > 0, logp, 0.0) + s["entropy"][a:a + step][:, None])
            d = d - s["grad_entropy"][a:a + step][:, None] * ent
        d.scatter_add_(1, t.clamp(0, V - 1)[:, None], gl)
        d = torch.where(torch.isinf(lse) & (lse < 0), 0.0, d)
        out[a:a + step] = d * c["scale"]
    return out


def _own(s):
    c, T = s["case"], s["T"]
    op = c["op"]
    if op == "proj":
        return T.proj(s["x"], s["W"], bias=s["bias"], act=c["act"], residual=s["residual"], ws=s["ws"], out=s["out"])
    if op == "moe":
        return T.moe_swiglu(s["x"], s["g"], s["router"], s["Wgu"], s["Wd"], c["k"], EPS, score=c["score"],
                            select_bias=s["select_bias"], renorm=c["renorm"], route_scale=c["route_scale"],
                            residual=s["residual"], ws=s["ws"], out=s["out"])
    if op == "logprobs":
        r = T.token_logprobs(s["logits"], s["targets"], top_k=c["top_k"], scale=c["scale"])
        return r.logprob, r.entropy, r.lse, r.top_ids, r.top_logprobs
    return T.token_logprobs_backward(s["logits"], s["targets"], s["lse"], s["entropy"], s["grad_logprob"],
                                     s["grad_entropy"], scale=c["scale"], out=s["out"])


_PLAIN = {"proj": _plain_proj, "moe": _plain_moe, "logprobs": _plain_logprobs,
          "logprobs_backward": _plain_logprobs_backward}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, M = case["op"], case["M"]
    if op == "proj":
        K, N = case["K"], case["N"]
        ob = 2 if case["out"] == "bf16" else 4
        b = 2 * (M * K + K * N) + ob * M * N * (2 if case["residual"] else 1) + (4 * N if case["bias"] else 0)
        return {"bytes": b, "flops": 2 * M * K * N}
    if op == "moe":
        d, I, E, k = case["d"], case["I"], case["E"], case["k"]
        active = E * (1 - (1 - k / E) ** M)      # experts that some token chose, on average
        b = active * 6 * d * I + 2 * E * d + 4 * d + 2 * M * d * 2 + 8 * M * k
        return {"bytes": int(b), "flops": 6 * M * k * d * I + 2 * M * E * d}
    V, size = case["V"], 4 if case["dtype"] == "fp32" else 2
    if op == "logprobs":
        return {"bytes": M * V * size + M * (16 + 8 * case["top_k"]), "flops": 6 * M * V}
    return {"bytes": 2 * M * V * size + 20 * M, "flops": 8 * M * V}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_proj(s):
    c = s["case"]
    v = torch.mm(s["x"].to(torch.float64), s["W"].to(torch.float64))
    if s["bias"] is not None:
        v += s["bias"].to(torch.float64)
    a = c["act"]
    if a == "relu":
        v = v.clamp(min=0)
    elif a == "gelu":
        v = v * torch.special.ndtr(v)
    elif a == "gelu_tanh":
        # (1 + tanh u) / 2 is the logistic function of 2 u
        v = v * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    elif a == "silu":
        v = v * torch.sigmoid(v)
    if s["residual"] is not None:
        v += s["residual"].to(torch.float64)
    return v


def _exact_moe(s):
    c = s["case"]
    M, d, I, E, k = c["M"], c["d"], c["I"], c["E"], c["k"]
    x = s["x"].to(torch.float64)
    h = x / torch.sqrt((x * x).sum(1, keepdim=True) / d + EPS)
    l = torch.einsum("md,ed->me", h * s["g"].to(torch.float64), s["router"].to(torch.float64))
    score = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    order = l if s["select_bias"] is None else score + s["select_bias"].to(torch.float64)
    ids = torch.argsort(order, dim=1, descending=True, stable=True)[:, :k]
    w = torch.take_along_dim(score, ids, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["route_scale"]
    y = s["residual"].to(torch.float64).clone() if s["residual"] is not None else torch.zeros_like(x)
    for e in range(E):
        rows, slot = torch.nonzero(ids == e, as_tuple=True)
        if rows.numel() == 0:
            continue
        gu = (h[rows] @ s["Wgu"][e].to(torch.float64)).view(-1, I // 128, 2, 128)
        gate, up = gu[:, :, 0].reshape(-1, I), gu[:, :, 1].reshape(-1, I)
        down = (gate * torch.sigmoid(gate) * up) @ s["Wd"][e].to(torch.float64)
        y.index_add_(0, rows, down * w[rows, slot][:, None])
    return y, ids.int(), w


def _exact_logprobs(s):
    c = s["case"]
    M, V = s["logits"].shape
    res = []
    for a in range(0, M, max(1, (1 << 25) // V)):
        b = min(M, a + max(1, (1 << 25) // V))
        raw = s["logits"][a:b].to(torch.float64)
        t = s["targets"][a:b].to(torch.int64)
        z = raw * float(torch.tensor(c["scale"], dtype=torch.float32))
        lse = torch.logsumexp(z, 1)
        empty = torch.isneginf(lse)
        q = z - lse.masked_fill(empty, 0)[:, None]
        q = q.masked_fill(empty[:, None], -math.inf)
        H = torch.special.entr(torch.exp(q)).sum(1)
        lp = torch.take_along_dim(q, t.clamp(min=0)[:, None], 1)[:, 0].masked_fill(t < 0, 0)
        idx = torch.argsort(raw, dim=1, descending=True, stable=True)[:, :c["top_k"]]
        res.append((lp, H, lse, idx.int(), torch.take_along_dim(q, idx, 1)))
    return tuple(torch.cat(v) for v in zip(*res))


def _exact_logprobs_backward(s):
    c = s["case"]
    M, V = s["logits"].shape
    sc = float(torch.tensor(c["scale"], dtype=torch.float32))
    out = torch.empty(M, V, device="cuda", dtype=torch.float64)
    for a in range(0, M, max(1, (1 << 25) // V)):
        b = min(M, a + max(1, (1 << 25) // V))
        t = s["targets"][a:b].to(torch.int64)
        z = s["logits"][a:b].to(torch.float64) * sc
        p = torch.softmax(z, 1).nan_to_num(0.0)          # a row without tokens has no gradient
        gl = s["grad_logprob"][a:b].to(torch.float64).masked_fill(t < 0, 0)
        hot = torch.zeros_like(p)
        hot.scatter_(1, t.clamp(min=0)[:, None], 1.0)
        g = gl[:, None] * (hot - p)
        if s["grad_entropy"] is not None:
            ent = torch.special.entr(p)                   # -p log p
            g += s["grad_entropy"][a:b].to(torch.float64)[:, None] * (ent - p * ent.sum(1, keepdim=True))
        g[p.sum(1) == 0] = 0
        out[a:b] = g * sc
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    return {"proj": _exact_proj, "moe": _exact_moe, "logprobs": _exact_logprobs,
            "logprobs_backward": _exact_logprobs_backward}[case["op"]](s)
