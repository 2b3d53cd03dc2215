"""The gated-delta layers of a decode, the norms between its projections and the choice of its tokens, operator by operator.

Four operators of libkq serve what the decode workloads' model runs beside its attention layers:

  norm    kq_rms_norm     RMS norm of rows, with the residual's addition before it, a gate after it, an output in Q8_0
  conv    kq_causal_conv  the short causal convolution over a fused projection's channels, with its rolling state
  gdn     kq_gdn          the gated delta rule, token by token and over prompts, with its state
  sample  kq_sample       a token from each row of logits: temperature, top-k, top-p, min-p and a given random number

A case names an operator and its sizes.  The head layouts are that of the Bonsai-27B-shaped decode workload (a 5120 ->
10240 projection holds 16 query, 16 key and 48 value heads of 128, a 5120 -> 6144 one the gates of 48 heads) and generic
ones; the vocabularies are the two decode workloads' 248320 and 151936.  Request lengths follow from the case alone,
values from the seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
WIDTH = 4  # taps of the convolution

HEADS = {  # k_heads, v_heads, head_dim
    "h48": dict(k_heads=16, v_heads=48, head_dim=128),
    "h32": dict(k_heads=16, v_heads=32, head_dim=128),
    "same": dict(k_heads=4, v_heads=4, head_dim=128),
    "h64": dict(k_heads=4, v_heads=12, head_dim=64),
}


def _gdn(name, heads, **more):
    c = dict(op="gdn", **HEADS[heads], **more)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # the residual stream of a single user's token, fp32 as the GEMVs give it: pure latency
        dict(name="norm_one_f32", op="norm", tokens=1, heads=1, dim=5120, residual=True, gate=False, q8=False, dtype="f32"),
        # the residual stream of a prompt, its norm kept in 8 bits beside the 16-bit output
        dict(name="norm_prompt_bf16", op="norm", tokens=4099, heads=1, dim=5120, residual=True, gate=False, q8=True, dtype="bf16"),
        # the gated norm of a delta layer's heads over a prompt chunk, gates strided in their projection's rows
        dict(name="norm_heads_f16", op="norm", tokens=1024, heads=48, dim=128, residual=False, gate=True, q8=False, dtype="f16"),
        # a decode step of a batch: one token a request, the state of each shifted by one
        dict(name="conv_step_f16", op="conv", requests=64, new=1, ragged=False, channels=10240, fresh=False, dtype="f16"),
        # prompts of many lengths
        dict(name="conv_prompts_bf16", op="conv", requests=7, new=1900, ragged=True, channels=10240, fresh=True, dtype="bf16"),
        # a single user's next token: latency
        _gdn("gdn_one_f32", "h48", requests=1, new=1, ragged=False, fresh=False, dtype="f32"),
        # a decode step of a large batch: every request's state read and written
        _gdn("gdn_step_f16", "h48", requests=128, new=1, ragged=False, fresh=False, dtype="f16"),
        # tokens of short runs (a drafted run that was accepted) in fp32
        _gdn("gdn_run_f32", "h48", requests=8, new=5, ragged=True, fresh=False, dtype="f32"),
        # a long prompt
        _gdn("gdn_prompt_bf16", "h48", requests=1, new=8192, ragged=False, fresh=True, dtype="bf16"),
        # prompts of many lengths that go on from their states
        _gdn("gdn_prompts_f16", "h48", requests=6, new=1500, ragged=True, fresh=False, dtype="f16"),
        # a single user's token from the larger vocabulary with the usual settings
        dict(name="sample_one_f32", op="sample", rows=1, vocab=248320, temperature=0.7, top_k=20, top_p=0.8, min_p=0.0, dtype="f32"),
        # a batch's tokens without top-k: the mass is found over the whole row
        dict(name="sample_batch_f16", op="sample", rows=64, vocab=151936, temperature=1.0, top_k=0, top_p=0.95, min_p=0.02, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "conv", "gdn", "gdn", "gdn", "sample"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        if rng.random() < 0.5:
            dim = 32 * _log(rng, 4, 512)
            return dict(op=op, tokens=_log(rng, 1, min(8192, 20000000 // dim)), heads=1, dim=dim, residual=rng.random() < 0.7,
                        gate=False, q8=rng.random() < 0.3, dtype=dtype)
        return dict(op=op, tokens=_log(rng, 1, 1500), heads=rng.choice([4, 12, 32, 48]), dim=rng.choice([64, 128, 256]),
                    residual=False, gate=rng.random() < 0.8, q8=False, dtype=dtype)
    if op == "conv":
        requests = _log(rng, 1, 200)
        return dict(op=op, requests=requests, new=1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(4096, 8000 // requests))),
                    ragged=rng.random() < 0.6, channels=8 * _log(rng, 32, 1280), fresh=rng.random() < 0.5, dtype=dtype)
    if op == "sample":
        vocab = _log(rng, 1000, 260000)
        return dict(op=op, rows=_log(rng, 1, min(256, 9000000 // vocab)), vocab=vocab, temperature=rng.choice([0.0, 0.3, 0.7, 1.0, 1.3]),
                    top_k=rng.choice([0, 0, 1, 20, 50, _log(rng, 2, vocab)]), top_p=rng.choice([1.0, 0.8, 0.95, 0.3]),
                    min_p=rng.choice([0.0, 0.0, 0.05, 0.01]), dtype=dtype)
    heads = rng.choice(["h48", "h48", "h32", "same", "h64"])
    kind = rng.choice(["step", "run", "prompt", "prompt"])
    if kind == "prompt":
        new = _log(rng, 9, 2000 if dtype == "f32" else 6000)
        requests = _log(rng, 1, max(1, min(8, 8192 // new)))
    else:
        requests, new = _log(rng, 1, 128), 1 if kind == "step" else rng.randrange(2, 9)
    return _gdn(None, heads, requests=requests, new=new, ragged=rng.random() < 0.6 and requests > 1 and new > 1,
                fresh=rng.random() < 0.4, dtype=dtype)


# ---- lengths and work (from the case alone) ------------------------------------------------


def _new(case):
    """New tokens of each request."""
    b, new = case["requests"], case["new"]
    n = np.full(b, new)
    if case["ragged"]:
        r = np.random.RandomState(31 * b + new)
        n = r.randint(1, new + 1, b)
        n[r.randint(b)] = new
    return n


def work(case):
    s = SIZE[case["dtype"]]
    if case["op"] == "norm":
        v = case["tokens"] * case["heads"] * case["dim"]
        passes = 2 + 2 * case["residual"] + case["gate"]  # x and y; the residual both ways; the gate
        # codes and scales written, read back, and what they stand for out in 16 bits
        q8 = v * (1 + 2 / 32) * 2 + v * 2 if case["q8"] else 0
        return {"bytes": v * s * passes + 4 * case["dim"] + q8, "flops": 6 * v}
    if case["op"] == "sample":
        v = case["rows"] * case["vocab"]
        return {"bytes": v * s + 12 * case["rows"], "flops": 4 * v}
    t, b = int(_new(case).sum()), case["requests"]
    if case["op"] == "conv":
        c = case["channels"]
        state = b * (WIDTH - 1) * c * s * (1 if case["fresh"] else 2)
        return {"bytes": 2 * t * c * s + state + 4 * c * (WIDTH + 1) + 12 * b, "flops": 2 * t * c * WIDTH}
    hk, hv, d = case["k_heads"], case["v_heads"], case["head_dim"]
    state = b * hv * d * d * 4 * (1 if case["fresh"] else 2)
    # q, k, v and the output; two gates a value head; the states
    rows = t * (2 * hk * d + 2 * hv * d + 2 * hv) * s
    return {"bytes": rows + state + 8 * hv + 12 * b, "flops": 8 * t * hv * d * d}


# ---- inputs --------------------------------------------------------------------------------


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV, dtype=torch.float32)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _requests(st, case, g):
    """The step's arrays: where each request's tokens begin, its length with them, the slot of its state."""
    n, b = _new(case), case["requests"]
    cached = 0 if case["fresh"] else 100 + np.arange(b)
    st["tokens"], st["slots"] = int(n.sum()), b + 2
    st["q_start"] = _int(np.concatenate([[0], np.cumsum(n)]))
    st["kv_len"] = _int(n + cached)
    st["slot"] = torch.randperm(b + 2, generator=g, device=DEV)[:b].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st, dt = {"case": case}, TYPES[case["dtype"]]
    if case["op"] == "norm":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        st["x"] = (_normal(g, t, h, d) * torch.exp(0.5 * _normal(g, t, h, 1))).to(dt)
        st["weight"] = 0.5 + _uniform(g, d)
        st["residual"] = _normal(g, t, h, d).to(dt) if case["residual"] else None
        # the gates lie in the rows of a projection that holds something else too
        st["gate"] = _normal(g, t, h * d + 64).to(dt)[:, : h * d].unflatten(1, (h, d)) if case["gate"] else None
    elif case["op"] == "sample":
        r, v = case["rows"], case["vocab"]
        x = 2.2 * _normal(g, r, v)
        near = torch.randint(0, v, (r, 12), generator=g, device=DEV)  # the few that a model thinks likely
        x.scatter_add_(1, near, 6 + 6 * _uniform(g, r, 12))
        st["logits"] = x.to(dt)
        st["u"] = _uniform(g, r)
        full = lambda v, **k: torch.full((r,), v, device=DEV, **k)  # noqa: E731
        st["temperature"], st["top_p"], st["min_p"] = full(case["temperature"]), full(case["top_p"]), full(case["min_p"])
        st["top_k"] = full(case["top_k"], dtype=torch.int32)
    elif case["op"] == "conv":
        _requests(st, case, g)
        c = case["channels"]
        st["x"] = _normal(g, st["tokens"], c).to(dt)
        st["weight"] = 0.5 * _normal(g, c, WIDTH)
        st["bias"] = 0.1 * _normal(g, c)
        st["state"] = _normal(g, st["slots"], WIDTH - 1, c).to(dt)
    else:
        _requests(st, case, g)
        hk, hv, d = case["k_heads"], case["v_heads"], case["head_dim"]
        x = _normal(g, st["tokens"], (2 * hk + hv) * d)
        x += 0.3 * _normal(g, 1, (2 * hk + hv) * d)  # keys have a part in common
        st["x"] = x.to(dt)
        st["ab"] = _normal(g, st["tokens"], 2 * hv).to(dt)
        st["a_log"] = torch.log(1 + 15 * _uniform(g, hv))
        step = torch.exp(math.log(1e-3) + math.log(100) * _uniform(g, hv))
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))  # softplus gives `step` back
        st["state"] = 0.3 * _normal(g, st["slots"], hv, d, d)
    return _handles(st)


def _handles(st):
    """The descriptors and the workspace that a program keeps beside its buffers."""
    if not own:
        return st
    import quantized_weight_streaming_gb300 as kq

    c = st["case"]
    if c["op"] == "norm":
        st["p"] = kq.RMSNorm(c["heads"], c["dim"], st["weight"], eps=EPS)
    elif c["op"] == "conv":
        st["p"] = kq.CausalConv(st["weight"], st["bias"])
    elif c["op"] == "gdn":
        st["p"] = kq.GatedDelta(c["k_heads"], c["v_heads"], c["head_dim"], st["a_log"], st["dt_bias"], eps=EPS)
        n = kq.kq_gdn_workspace_bytes(st["p"], st["x"].dtype, c["requests"], st["tokens"], c["new"])
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return st


def _heads_of(st):
    """q, k, v of the convolution's rows and the two gates, as views."""
    c, x = st["case"], st["x"]
    hk, hv, d = c["k_heads"], c["v_heads"], c["head_dim"]
    q = x[:, : hk * d].unflatten(1, (hk, d))
    k = x[:, hk * d: 2 * hk * d].unflatten(1, (hk, d))
    v = x[:, 2 * hk * d:].unflatten(1, (hv, d))
    return q, k, v, st["ab"][:, :hv], st["ab"][:, hv:]


# ---- one pass ------------------------------------------------------------------------------


def run(st):
    return (_run_own if own else _run_plain)[st["case"]["op"]](st)


def _own_norm(st):
    import quantized_weight_streaming_gb300 as kq

    c, x = st["case"], st["x"]
    out = torch.empty_like(x)
    q8 = kq.QMatrix("q8_0", c["tokens"] * c["heads"], c["dim"]) if c["q8"] else None
    kq.kq_rms_norm(st["p"], x, out, residual=st["residual"], gate=st["gate"], out_q8=q8)
    r = {"out": out}
    if c["residual"]:
        r["residual"] = st["residual"]
    if c["q8"]:
        s = q8.scales.view(torch.float16).view(q8.n, -1)[:, : q8.k // 32]
        r["q8"] = q8.codes.view(torch.int8).view(q8.n, -1, 32) * s[:, :, None]
    return r


def _own_conv(st):
    import quantized_weight_streaming_gb300 as kq

    out = torch.empty_like(st["x"])
    kq.kq_causal_conv(st["p"], st["x"], st["q_start"], st["kv_len"], st["slot"], st["state"], out)
    return {"out": out, "state": st["state"]}


def _own_gdn(st):
    import quantized_weight_streaming_gb300 as kq

    q, k, v, a, b = _heads_of(st)
    out = torch.empty(v.shape, dtype=v.dtype, device=DEV)
    kq.kq_gdn(st["p"], q, k, v, a, b, st["q_start"], st["kv_len"], st["slot"], st["state"], out, st["case"]["new"], ws=st["ws"])
    return {"out": out, "state": st["state"]}


def _own_sample(st):
    import quantized_weight_streaming_gb300 as kq

    r = st["case"]["rows"]
    token, prob = torch.empty(r, dtype=torch.int32, device=DEV), torch.empty(r, device=DEV)
    kq.kq_sample(st["logits"], st["u"], token, prob, temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"],
                 min_p=st["min_p"])
    return {"token": token, "prob": prob}


def _plain_norm(st):
    c, dt = st["case"], st["x"].dtype
    x, r = st["x"].float(), {}
    if c["residual"]:
        st["residual"].copy_(x + st["residual"].float())  # the residual keeps the sum, and the norm is of what it keeps
        r["residual"] = st["residual"]
        x = st["residual"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * st["weight"]
    if c["gate"]:
        z = st["gate"].float()
        y = y * (z / (1 + torch.exp(-z)))
    r["out"] = y.to(dt)
    if c["q8"]:
        w = y.reshape(c["tokens"] * c["heads"], -1, 32)
        s = (w.abs().amax(-1, keepdim=True) / 127).half()
        f = torch.where(s == 0, torch.ones_like(s), s).double()
        q = w.double() / f
        q = torch.where(s == 0, torch.zeros_like(q), torch.sign(q) * torch.floor(q.abs() + 0.5)).clamp(-127, 127)
        r["q8"] = q.to(torch.int8) * s
    return r


def _request_of(st):
    """Each token's request and its place among the request's new tokens."""
    start = st["q_start"].long()
    n = start[1:] - start[:-1]
    req = torch.repeat_interleave(torch.arange(n.shape[0], device=DEV), n, output_size=st["tokens"])
    return req, torch.arange(st["tokens"], device=DEV) - start[req], start, n


def _plain_conv(st):
    x, w, slot = st["x"].float(), st["weight"], st["slot"].long()
    req, i, start, n = _request_of(st)
    old = st["state"][slot].float()
    old = torch.where((st["kv_len"].long() == n)[:, None, None], torch.zeros_like(old), old)  # nothing before the first token
    t = torch.arange(st["tokens"], device=DEV)
    y = st["bias"] + w[:, WIDTH - 1] * x
    for j in range(1, WIDTH):
        before = torch.where((i >= j)[:, None], x[(t - j).clamp(min=0)], old[req, (WIDTH - 1 + i - j).clamp(max=WIDTH - 2)])
        y += w[:, WIDTH - 1 - j] * before
    # the last inputs, those of the old state among them where a request brings fewer
    at = n[:, None] - (WIDTH - 1) + torch.arange(WIDTH - 1, device=DEV)[None, :]
    keep = torch.gather(old, 1, (WIDTH - 1 + at).clamp(0, WIDTH - 2)[:, :, None].expand(-1, -1, x.shape[1]))
    st["state"][slot] = torch.where((at >= 0)[:, :, None], x[(start[:-1, None] + at).clamp(min=0)], keep).to(st["x"].dtype)
    return {"out": (y / (1 + torch.exp(-y))).to(st["x"].dtype), "state": st["state"]}


def _plain_gdn(st):
    """In chunks: within one, the updates u of all tokens solve a triangular system; between them the state goes on."""
    c = st["case"]
    hk, hv, d, size = c["k_heads"], c["v_heads"], c["head_dim"], min(64, c["new"])
    req, i, start, n = _request_of(st)
    chunks = -(-c["new"] // size)
    row = start[:-1, None] + torch.arange(chunks * size, device=DEV)[None, :]
    real = torch.arange(chunks * size, device=DEV)[None, :] < n[:, None]
    row = row.clamp(max=st["tokens"] - 1)

    def lay(x, heads):  # [tokens, heads, ...] -> float32 [requests, value heads, chunks, size, ...], zeros past the end
        x = x.float()[row] * real.view(*real.shape, *[1] * (x.dim() - 1))
        x = x.unflatten(1, (chunks, size)).movedim(3, 1)
        return x.repeat_interleave(hv // heads, 1) if heads != hv else x

    q, k, v, a, b = _heads_of(st)
    unit = lambda x: x * torch.rsqrt((x * x).sum(-1, keepdim=True) + EPS)  # noqa: E731
    q, k, v = unit(lay(q, hk)) * d ** -0.5, unit(lay(k, hk)), lay(v, hv)
    soft = a.float() + st["dt_bias"]
    soft = torch.where(soft > 20, soft, torch.log1p(torch.exp(soft.clamp(max=20))))
    g = torch.cumsum(lay(-torch.exp(st["a_log"]) * soft, hv), -1)
    beta = lay(1 / (1 + torch.exp(-b.float())), hv)
    ratio = torch.exp((g[..., :, None] - g[..., None, :]).clamp(max=0))  # decay from token j to token i
    tri = torch.ones(size, size, device=DEV).tril()
    low = torch.matmul(k, k.transpose(-1, -2)) * ratio * beta[..., None] * tri.tril(-1)
    inner = torch.matmul(q, k.transpose(-1, -2)) * ratio * tri
    inv = torch.eye(size, device=DEV).expand(low.shape).contiguous()
    for r in range(1, size):  # rows of (1 + low)^-1, from the top
        inv[..., r, :r] = -torch.matmul(low[..., r: r + 1, :r], inv[..., :r, :r])[..., 0, :]
    slot = st["slot"].long()
    s = st["state"][slot]
    s = torch.where((st["kv_len"].long() == n)[:, None, None, None], torch.zeros_like(s), s)
    decay = torch.exp(g)
    last = torch.exp(g[..., -1:] - g)
    o = torch.empty_like(v)
    for m in range(chunks):
        e = decay[:, :, m, :, None]
        u = beta[:, :, m, :, None] * (v[:, :, m] - e * torch.matmul(k[:, :, m], s))
        u = torch.matmul(inv[:, :, m], u)
        o[:, :, m] = e * torch.matmul(q[:, :, m], s) + torch.matmul(inner[:, :, m], u)
        s = e[:, :, -1:] * s + torch.matmul((k[:, :, m] * last[:, :, m, :, None]).transpose(-1, -2), u)
    st["state"][slot] = s
    o = o.movedim(1, 3).flatten(1, 2)[req, i]
    return {"out": o.to(st["x"].dtype), "state": st["state"]}


def _plain_sample(st):
    """In 64 bits: a border of the kept set, or of the token that the number falls on, is no matter of rounding there."""
    x, c = st["logits"].double(), st["case"]
    r, v = x.shape
    val, at = torch.sort(x, dim=-1, descending=True, stable=True)
    t = st["temperature"].double()[:, None]
    e = torch.where(t > 0, torch.exp((val - val[:, :1]) / torch.where(t > 0, t, torch.ones_like(t))), torch.zeros_like(val))
    rank = torch.arange(v, device=DEV)[None, :]
    e = torch.where((t > 0) | (rank > 0), e, torch.ones_like(e))  # temperature 0: the largest alone
    k = torch.where(st["top_k"] > 0, st["top_k"], torch.full_like(st["top_k"], v)).long()[:, None]
    e = e * (rank < k)
    before = torch.cumsum(e, -1) - e
    keep = (before < st["top_p"].double()[:, None] * e.sum(-1, keepdim=True)) | (rank == 0)
    keep &= (e >= st["min_p"].double()[:, None]) | (rank == 0)
    e = torch.zeros_like(e).scatter(1, at, e * keep)  # in the order of the vocabulary
    total = e.sum(-1, keepdim=True)
    after = torch.cumsum(e, -1)
    past = (after > st["u"].double()[:, None] * total) & (e > 0)
    tail = torch.where(e > 0, rank, torch.zeros_like(rank)).amax(-1)
    token = torch.minimum(torch.where(past, rank, torch.full_like(rank, v)).amin(-1), tail)
    return {"token": token.int(), "prob": (torch.gather(e, 1, token[:, None]) / total)[:, 0].float()}


_run_own = {"norm": _own_norm, "conv": _own_conv, "gdn": _own_gdn, "sample": _own_sample}
_run_plain = {"norm": _plain_norm, "conv": _plain_conv, "gdn": _plain_gdn, "sample": _plain_sample}


# ---- the definitions, in 64 bits -------------------------------------------------------------


def _sigmoid(x):
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1 / (1 + e), e / (1 + e))


def _exact_norm(st, case):
    x, r = st["x"].double(), {}
    if case["residual"]:
        x = (x + st["residual"].double()).to(st["x"].dtype).double()
        r["residual"] = x
    y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * st["weight"].double()
    if case["gate"]:
        z = st["gate"].double()
        y = y * z * _sigmoid(z)
    r["out"] = y
    if case["q8"]:
        w = y.reshape(-1, case["dim"] // 32, 32)
        s = (w.abs().amax(-1, keepdim=True) / 127).half().double()
        n = torch.nan_to_num(w / s, nan=0.0, posinf=0.0, neginf=0.0)
        r["q8"] = torch.where(n >= 0, torch.floor(n + 0.5), torch.ceil(n - 0.5)).clamp(-127, 127) * s
    return r


def _exact_conv(st, case):
    """Request by request: its old state, then its tokens, as one signal."""
    out, state = torch.empty(st["x"].shape, dtype=torch.float64, device=DEV), st["state"].double()
    w = st["weight"].double()
    for r, (lo, hi) in enumerate(zip(st["q_start"].tolist()[:-1], st["q_start"].tolist()[1:])):
        slot = int(st["slot"][r])
        head = state[slot] * (0 if case["fresh"] else 1)
        x = torch.cat((head, st["x"][lo:hi].double()))
        y = sum(x[j: j + hi - lo] * w[:, j] for j in range(WIDTH)) + st["bias"].double()
        out[lo:hi] = y * _sigmoid(y)
        state[slot] = x[-(WIDTH - 1):]
    return {"out": out, "state": state}


def _exact_gdn(st, case):
    """Token by token, as the rule is written down."""
    hk, hv, d = case["k_heads"], case["v_heads"], case["head_dim"]
    q, k, v, a, b = (x.double() for x in _heads_of(st))
    q = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + EPS) / math.sqrt(d)
    k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + EPS)
    q, k = (x.repeat_interleave(hv // hk, 1) for x in (q, k))
    soft = a + st["dt_bias"].double()
    soft = soft.clamp(min=0) + torch.log1p(torch.exp(-soft.abs()))
    fade = torch.exp(-torch.exp(st["a_log"].double()) * soft)
    beta = _sigmoid(b)
    start, slot = st["q_start"].long(), st["slot"].long()
    n = _new(case)
    order = np.argsort(-n, kind="stable")  # the longest first: those that still run are a prefix
    first = start[:-1][torch.from_numpy(order).to(DEV)]
    s = st["state"].double()[slot[torch.from_numpy(order).to(DEV)]] * (0 if case["fresh"] else 1)
    out = torch.empty(v.shape, dtype=torch.float64, device=DEV)
    for i in range(int(n.max())):
        m = int((n > i).sum())
        t = first[:m] + i
        h = s[:m] * fade[t][:, :, None, None]
        u = beta[t][:, :, None] * (v[t] - torch.einsum("bhk,bhkv->bhv", k[t], h))
        h += k[t][..., None] * u[..., None, :]
        out[t] = torch.einsum("bhk,bhkv->bhv", q[t], h)
        s[:m] = h
    state = st["state"].double()
    state[slot[torch.from_numpy(order).to(DEV)]] = s
    return {"out": out, "state": state}


def _exact_sample(st, case):
    """The chance of the token that the definition gives, row by row on the host."""
    prob = np.empty(case["rows"])
    for r in range(case["rows"]):
        x = st["logits"][r].double().cpu().numpy()
        t, p, m, k = (float(st[n][r]) for n in ("temperature", "top_p", "min_p", "top_k"))
        order = np.lexsort((np.arange(x.size), -x))
        if t == 0:
            prob[r] = 1.0
            continue
        order = order[: int(k)] if k > 0 else order
        w = np.exp((x[order] - x[order[0]]) / t)
        n = int(np.searchsorted(np.cumsum(w), p * w.sum())) + 1  # the shortest prefix that holds the mass
        order, w = order[:n], w[:n]
        order = order[(w >= m) | (np.arange(w.size) == 0)]
        order.sort()
        w = np.exp((x[order] - x.max()) / t)
        at = min(int(np.searchsorted(np.cumsum(w), float(st["u"][r]) * w.sum(), side="right")), w.size - 1)
        prob[r] = w[at] / w.sum()
    return {"token": None, "prob": torch.from_numpy(prob).to(DEV)}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "gdn": _exact_gdn, "sample": _exact_sample}[case["op"]](st, case)
