"""The attention step between the quantized projections, measured operator by operator.

Four operators of libkq serve a decode or prompt step on a paged 4-bit cache:

  slots   kq_slot_map      block tables and slot maps from the requests' lengths
  norm    kq_qk_norm_rope  RMS norm of each query and key head, and the position rotation
  append  kq_kv_append     the same pass, with keys and values written to the cache in 4 bits
                           (and kq_kv_read, which gives back what the written codes stand for)
  attn    kq_attn_paged    attention of new tokens over the cache

A case names an operator and its sizes; head layouts are those of the decode
workloads of this repository (32 query and 8 key heads of 128; 24 and 4 heads
of 256 with 64 rotated dimensions and queries interleaved with gates) and two
generic ones.  Request lengths follow from the case alone, values from the
seed.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
GRANULE = 16  # tokens of one head that lie together in the cache

HEADS = {  # q_heads, kv_heads, head_dim, rope_dim, gated (q and a gate of the same size alternate, head by head)
    "h128": dict(q_heads=32, kv_heads=8, head_dim=128, rope_dim=128, gated=False),
    "h256": dict(q_heads=24, kv_heads=4, head_dim=256, rope_dim=64, gated=True),
    "h64": dict(q_heads=14, kv_heads=2, head_dim=64, rope_dim=64, gated=False),
    "mha": dict(q_heads=12, kv_heads=12, head_dim=128, rope_dim=128, gated=False),
}


def _case(name, op, heads="h128", **more):
    c = {"op": op}
    if op != "slots":
        c.update(HEADS[heads])
    c.update(more)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # one decode step's bookkeeping at a full batch: a token each, the odd request takes a page
        _case("slots_step_256", "slots", requests=256, new=1, ragged=False, context=6000, page=32),
        # a round of prompts of all lengths, some requests with nothing to do
        _case("slots_prompts_61", "slots", requests=61, new=2900, ragged=True, context=900, page=16),
        # one token of a single user: pure latency
        _case("norm_one_f32", "norm", tokens=1, run=1, dtype="f32"),
        # a prompt through wide heads of which a quarter is rotated, queries strided between gates
        _case("norm_prompt_bf16", "norm", "h256", tokens=4099, run=4099, dtype="bf16"),
        # a decode step of a batch: norms, rotation and the cache write in one launch
        _case("append_step_f16", "append", tokens=64, run=1, dtype="f16", page=32),
        # a long prompt written to the cache
        _case("append_prompt_bf16", "append", tokens=8192, run=8192, dtype="bf16", page=32),
        # a single user's next token in a short conversation: latency
        _case("attn_one_f32", "attn", requests=1, new=1, ragged=False, context=1300, page=32, window=0, dtype="f32"),
        # a decode step of a batch whose conversations differ in length
        _case("attn_step_bf16", "attn", requests=32, new=1, ragged=True, context=8000, page=32, window=0, dtype="bf16"),
        # the largest decode step: long contexts, wide heads
        _case("attn_long_f16", "attn", "h256", requests=64, new=1, ragged=False, context=16384, page=64, window=0, dtype="f16"),
        # drafted tokens verified together, fp32 as the GEMVs give it
        _case("attn_verify_f32", "attn", requests=8, new=4, ragged=False, context=4100, page=16, window=0, dtype="f32"),
        # a chunk of a long prompt on top of what is cached
        _case("attn_chunk_bf16", "attn", requests=1, new=2048, ragged=False, context=8192, page=32, window=0, dtype="bf16"),
        # prompts of many lengths with a sliding window over narrow heads, a group of seven
        _case("attn_prompts_f16", "attn", "h64", requests=9, new=1200, ragged=True, context=1800, page=48, window=1000, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "norm", "append", "attn", "attn", "attn"])
    heads = rng.choice(["h128", "h128", "h256", "h64", "mha"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "slots":
        requests = _log(rng, 1, 1000)
        if rng.random() < 0.5:
            return _case(None, op, requests=requests, new=1, ragged=False, context=_log(rng, 1, 16000), page=page)
        return _case(None, op, requests=requests, new=_log(rng, 2, max(2, 120000 // requests)), ragged=True,
                     context=_log(rng, 1, 8000), page=page)
    if op in ("norm", "append"):
        tokens = _log(rng, 1, 4096 if heads in ("h256", "mha") or dtype == "f32" else 8192)
        c = _case(None, op, heads, tokens=tokens, run=rng.choice([1, tokens, _log(rng, 1, tokens)]), dtype=dtype)
        return dict(c, page=page) if op == "append" else c
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    kind = rng.choice(["step", "step", "verify", "prompt"])
    per_token = HEADS[heads]["kv_heads"] * HEADS[heads]["head_dim"]  # cost limits follow the widest listed layout
    if kind == "prompt":
        new = _log(rng, 9, 2048)
        context = min(8192, new + _log(rng, 1, 6000))
        most = 2048 * 7168 * 4096 // (context * HEADS[heads]["q_heads"] * HEADS[heads]["head_dim"])  # new tokens in all
        new = min(new, most, 256 if dtype == "f32" else new)
        requests = _log(rng, 1, max(1, min(8, most // new)))
    else:
        requests = _log(rng, 1, 64)
        new = 1 if kind == "step" else rng.randrange(2, 9)
        most = 64 * 16384 * 1024 // (2 * requests * per_token)
        context = _log(rng, max(1, new), max(2, min(16384, most)))
    return _case(None, op, heads, requests=requests, new=new, ragged=rng.random() < 0.6 and requests > 1,
                 context=max(context, new), page=page, window=window, dtype=dtype)


# ---- lengths (from the case alone) -------------------------------------------------------


def _lengths(case):
    """(cached, new) of each request, as numpy arrays."""
    b, new, context = case["requests"], case["new"], case["context"]
    r = np.random.RandomState(97 * b + 13 * new + context)
    if case["op"] == "slots":
        cached = r.randint(0, context + 1, b)
        n = r.randint(0, new + 1, b) if case["ragged"] else np.full(b, new)
        if n.sum() == 0:
            n[-1] = new
        return cached, n
    n, total = np.full(b, new), np.full(b, context)
    if case["ragged"]:
        total = r.randint(max(1, context // 16), context + 1, b)
        total[r.randint(b)] = context
        if new > 1:
            n = r.randint(1, new + 1, b)
            n[r.randint(b)] = new
        n = np.minimum(n, total)
    return total - n, n


def _pairs(case):
    """Query-key pairs that attention has to look at, and keys that it has to read."""
    cached, new = _lengths(case)
    w, pairs, keys = case["window"], 0, 0
    for c, n in zip(cached.tolist(), new.tolist()):
        seen = np.arange(c + 1, c + n + 1)
        if w:
            seen = np.minimum(seen, w)
        pairs += int(seen.sum())
        keys += min(c + n, n - 1 + int(seen[0])) if n else 0
    return pairs, keys


def work(case):
    if case["op"] == "slots":
        cached, new = _lengths(case)
        p, t = case["page"], int(new.sum())
        fresh = int((-(-(cached + new) // p) - -(-cached // p)).sum())
        # lengths in; starts and totals out; a position and a slot for each token; a page id in and out for each
        # fresh page, and one in for each request that goes on within a page
        going_on = int(((cached % p > 0) & (new > 0)).sum())
        return {"bytes": 4 * (2 * len(new) + 2 * len(new) + 2 + 2 * t + 2 * fresh + going_on), "flops": 0}
    hq, hk, d, rd = case["q_heads"], case["kv_heads"], case["head_dim"], case["rope_dim"]
    s = SIZE[case["dtype"]]
    if case["op"] == "attn":
        pairs, keys = _pairs(case)
        tokens = int(_lengths(case)[1].sum())
        return {"bytes": keys * hk * 2 * (d // 2 + d // 16) + 2 * tokens * hq * d * s, "flops": 4 * pairs * hq * d}
    t = case["tokens"]
    both = t * (hq + hk) * d * s  # q and k in
    table = t * rd * 4 + t * 4 + 2 * d * 4
    if case["op"] == "norm":
        return {"bytes": 2 * both + table, "flops": 8 * t * (hq + hk) * d}
    cache = t * hk * 2 * (d // 2 + d // 16)
    # q, k, v in; q out; codes and scales written, read back, and their values out in 16 bits
    return {"bytes": both + t * hk * d * s + t * hq * d * s + table + 4 * t + 2 * cache + 4 * t + 2 * t * hk * d * 2,
            "flops": 12 * t * (hq + 2 * hk) * d}


# ---- the cache's layout, in elementary operations ------------------------------------------
#
# data: uint8 [pages][kv_heads][page / 16][granule bytes].  A granule holds 16
# tokens of one head: key codes, value codes, key scales, value scales.  The
# head dimension is cut into slabs of 128 (one slab of 64 where it is 64), a
# slab into groups of 32 that share a scale.
#   key codes    [slab][token 16][c 4][group][4 bytes]: the 8 nibbles of dimensions 32 group + 8 c + 0..7
#   value codes  [slab][token / 8][r 8][token % 8 / 2][group][token % 2][2 bytes]: dimensions 32 group + 4 r + 0..3
#   scales       fp16 [slab][token 16][group]
# A code q stands for scale * (q - 8).


def _dims(d):
    slabs = max(1, d // 128)
    return slabs, d // 32 // slabs


def _granule_bytes(d):
    return GRANULE * d * 9 // 8


def _nibbles(b):
    return torch.stack((b & 15, b >> 4), -1).flatten(-2)


def _unpack(g, d):
    """uint8 [..., granule bytes] -> (keys, values) float32 [..., 16, d]."""
    lead = g.shape[:-1]
    n = len(lead)
    slabs, groups = _dims(d)
    half = GRANULE * d // 2
    sc = GRANULE * d // 16
    k = _nibbles(g[..., :half].reshape(*lead, slabs, GRANULE, 4, groups, 4)).float() - 8
    k = k.permute(*range(n), n + 1, n, n + 3, n + 2, n + 4)  # token, slab, group, c, 8
    v = _nibbles(g[..., half: 2 * half].reshape(*lead, slabs, 2, 8, 4, groups, 2, 2)).float() - 8
    v = v.permute(*range(n), n + 1, n + 3, n + 5, n, n + 4, n + 2, n + 6)  # token, slab, group, r, 4
    scales = g[..., 2 * half:].contiguous().view(torch.float16).float()
    ks = scales[..., : sc // 2].reshape(*lead, slabs, GRANULE, groups).transpose(-3, -2)
    vs = scales[..., sc // 2:].reshape(*lead, slabs, GRANULE, groups).transpose(-3, -2)
    k = k.reshape(*lead, GRANULE, slabs, groups, 32) * ks[..., None]
    v = v.reshape(*lead, GRANULE, slabs, groups, 32) * vs[..., None]
    return k.reshape(*lead, GRANULE, d), v.reshape(*lead, GRANULE, d)


def _quantize(x):
    """float32 [..., d] -> (codes uint8 [..., d], scales float16 [..., d / 32])."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    top = g.abs() == g.abs().amax(-1, keepdim=True)
    top &= torch.cumsum(top, -1) == 1  # the first of the largest
    scale = ((g * top).sum(-1, keepdim=True) / -8).half()
    s = scale.float()
    r = torch.where(s == 0, torch.zeros_like(g), g / torch.where(s == 0, torch.ones_like(s), s))
    q = (torch.sign(r) * torch.floor(r.abs() + 0.5) + 8).clamp(0, 15)
    return q.to(torch.uint8).flatten(-2), scale.squeeze(-1)


def _bytes(nib):
    p = nib.reshape(*nib.shape[:-1], -1, 2)
    return p[..., 0] | (p[..., 1] << 4)


def _token_bytes(kq, ks, vq, vs, d):
    """Codes [..., d] and scales [..., d / 32] of tokens -> the bytes that each token has in its granule, in the order
    of _token_places."""
    slabs, groups = _dims(d)
    lead = kq.shape[:-1]
    n = len(lead)
    k = kq.reshape(*lead, slabs, groups, 4, 8).permute(*range(n), n, n + 2, n + 1, n + 3)  # slab, c, group, 8
    v = vq.reshape(*lead, slabs, groups, 8, 4).permute(*range(n), n, n + 2, n + 1, n + 3)  # slab, r, group, 4
    return torch.cat((_bytes(k.reshape(*lead, d)), _bytes(v.reshape(*lead, d)),
                      ks.contiguous().view(torch.uint8), vs.contiguous().view(torch.uint8)), -1)


def _token_places(d):
    """int64 [16][bytes of a token]: where they lie in the granule."""
    slabs, groups = _dims(d)
    half = GRANULE * d // 2
    t = np.arange(GRANULE)[:, None, None]
    s = np.arange(slabs)[None, :, None]
    wide = d // slabs // 2  # bytes of a token's slab
    i = np.arange(wide)[None, None, :]
    k = s * GRANULE * wide + t * wide + i
    r, g, b = i // (2 * groups), i // 2 % groups, i % 2
    v = half + (((((s * 2 + t // 8) * 8 + r) * 4 + t % 8 // 2) * groups + g) * 2 + t % 2) * 2 + b
    j = np.arange(2 * groups)[None, None, :]
    scale = (s * GRANULE + t) * 2 * groups + j
    at = np.concatenate([a.reshape(GRANULE, -1) for a in (k, v, 2 * half + scale, 2 * half + GRANULE * d // 16 + scale)], 1)
    return torch.from_numpy(at.astype(np.int64)).to(DEV)


# ---- inputs --------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _cache(g, case, pages):
    """A pool whose every slot holds quantized keys and values (keys as after the norm, some channels stronger)."""
    hk, d, per = case["kv_heads"], case["head_dim"], case["page"] // GRANULE
    data = torch.empty(pages, hk, per, _granule_bytes(d), dtype=torch.uint8, device=DEV)
    at = _token_places(d).flatten()
    channel = 0.5 + torch.rand(hk, 1, d, generator=g, device=DEV)
    step = max(1, (1 << 26) // (hk * case["page"] * d))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        k = _normal(g, n, per, hk, GRANULE, d) * channel
        v = _normal(g, n, per, hk, GRANULE, d)
        b = _token_bytes(*_quantize(k), *_quantize(v), d)
        block = torch.empty(n, per, hk, _granule_bytes(d), dtype=torch.uint8, device=DEV)
        block[..., at] = b.flatten(-2)
        data[p: p + n] = block.transpose(1, 2)
    return data.reshape(pages, hk, -1)


def _rope_table(positions, rope_dim, base=1e6):
    """float32 [positions][rope_dim]: cosines of the rope_dim / 2 angles, then sines; computed in 64 bits."""
    f = base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=DEV) / rope_dim)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * f[None, :]
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def _pages_of(case, g):
    """(cached, new, table, pages of the pool): every request's pages, drawn from a shuffled pool."""
    cached, new = _lengths(case)
    p = case["page"]
    need = -(-(cached + new) // p)
    pages = int(need.sum()) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    wide = max(1, int(need.max())) + 1
    start = np.cumsum(need) - need
    at = torch.from_numpy(start[:, None] + np.arange(wide)[None, :]).to(DEV)
    have = torch.from_numpy(np.arange(wide)[None, :] < need[:, None]).to(DEV)
    table = torch.where(have, perm[at.clamp(max=pages - 1)], torch.zeros((), dtype=torch.int32, device=DEV))
    return cached, new, table.contiguous(), pages


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "slots":
        p = case["page"]
        cached, new = _lengths(case)
        shift = np.random.RandomState(seed % (1 << 31)).randint(0, p, len(cached))  # the seed moves the fill of the last pages
        cached = cached + shift
        old, total = -(-cached // p), -(-(cached + new) // p)
        wide = int((-(-(case["context"] + case["new"] + p) // p))) + 1
        free = int((total - old).sum()) + 5
        pages = int(old.sum()) + free
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        at = torch.from_numpy((np.cumsum(old) - old)[:, None] + np.arange(wide)[None, :]).to(DEV)
        have = torch.from_numpy(np.arange(wide)[None, :] < old[:, None]).to(DEV)
        held = torch.cat((perm[free:], perm[:1] * 0))
        st["table"] = torch.where(have, held[at.clamp(max=pages - free)], perm[:1] * 0).contiguous()
        st["free"] = perm[:free].contiguous()
        st["cached"], st["new"] = _int(cached), _int(new)
        st["tokens"] = int(new.sum())
        return st
    dt = TYPES[case["dtype"]]
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if op == "attn":
        cached, new, table, pages = _pages_of(case, g)
        t = int(new.sum())
        st["q"] = (_normal(g, t, hq, d) * (0.5 + torch.rand(hq, d, generator=g, device=DEV))).to(dt)
        st["data"] = _cache(g, case, pages)
        st["table"], st["kv_len"] = table, _int(cached + new)
        st["q_start"] = _int(np.concatenate([[0], np.cumsum(new)]))
        st["max_new"], st["max_len"] = int(new.max()), int((cached + new).max())
        st["scale"] = d ** -0.5
        return _handles(st)
    t = case["tokens"]
    qw = hq * d * (2 if case["gated"] else 1)
    x = _normal(g, t, qw + 2 * hk * d)
    x *= torch.exp(0.5 * _normal(g, t, 1))
    st["x"] = x.to(dt)
    st["q_weight"] = 0.5 + torch.rand(d, generator=g, device=DEV)
    st["k_weight"] = 0.5 + torch.rand(d, generator=g, device=DEV)
    # runs of consecutive tokens, each a request's own that goes on at a position of its own
    run_ = min(case["run"], t)
    start = np.random.RandomState(seed % (1 << 31)).randint(0, 8000, -(-t // run_))
    at = np.arange(t)
    pos = start[at // run_] + at % run_
    st["rope"] = _rope_table(8000 + run_, case["rope_dim"])
    st["positions"] = _int(pos)
    if op == "append":
        p = case["page"]
        per = -(-run_ // p) + 1  # pages of a run at most
        pages = per * len(start)
        st["data"] = torch.zeros(pages, hk, p // GRANULE * _granule_bytes(d), dtype=torch.uint8, device=DEV)
        st["places"] = _token_places(d)
        perm = torch.randperm(pages, generator=g, device=DEV).cpu().numpy()
        st["slots"] = _int(perm[at // run_ * per + pos // p - (start // p)[at // run_]] * p + pos % p)
    return _handles(st)


def _views(st):
    """q, k, v of the fused projection's rows, as [tokens, heads, head_dim] views."""
    c, x = st["case"], st["x"]
    hq, hk, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    wide = 2 * d if c["gated"] else d
    q = x[:, : hq * wide].unflatten(1, (hq, wide))[:, :, :d]
    k = x[:, hq * wide: hq * wide + hk * d].unflatten(1, (hk, d))
    v = x[:, hq * wide + hk * d:].unflatten(1, (hk, d))
    return q, k, v


def _handles(st):
    """The descriptors and the workspace that a program keeps beside its buffers."""
    if not own:
        return st
    import quantized_weight_streaming_gb300 as kq

    c = st["case"]
    if "data" in st:
        st["cache"] = kq.KVCache(st["data"].shape[0], c["page"], c["kv_heads"], c["head_dim"], data=st["data"])
    if c["op"] == "attn":
        n = kq.kq_attn_workspace_bytes(st["cache"], c["q_heads"], c["requests"], st["q"].shape[0], st["max_new"])
        st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    else:
        st["qk"] = kq.QKNorm(c["q_heads"], c["kv_heads"], c["head_dim"], c["rope_dim"], st["q_weight"], st["k_weight"],
                             st["rope"], eps=EPS)
    return st


# ---- one pass ------------------------------------------------------------------------------


def run(st):
    return (_run_own if own else _run_plain)[st["case"]["op"]](st)


def _own_slots(st):
    import quantized_weight_streaming_gb300 as kq

    c, t, b = st["case"], st["tokens"], st["new"].shape[0]
    i = dict(dtype=torch.int32, device=DEV)
    q_start, kv_len, used = torch.empty(b + 1, **i), torch.empty(b, **i), torch.empty(1, **i)
    positions, slots = torch.empty(t, **i), torch.empty(t, **i)
    kq.kq_slot_map(st["cached"], st["new"], c["page"], st["free"], st["table"], q_start, kv_len, positions, slots, used)
    return {"table": st["table"], "q_start": q_start, "kv_len": kv_len, "positions": positions, "slots": slots, "used": used}


def _own_norm(st):
    import quantized_weight_streaming_gb300 as kq

    q, k, _ = _views(st)
    q_out, k_out = torch.empty(q.shape, dtype=q.dtype, device=DEV), torch.empty(k.shape, dtype=k.dtype, device=DEV)
    kq.kq_qk_norm_rope(st["qk"], q, k, st["positions"], q_out, k_out)
    return {"q": q_out, "k": k_out}


def _own_append(st):
    import quantized_weight_streaming_gb300 as kq

    q, k, v = _views(st)
    q_out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    k_val, v_val = (torch.empty(k.shape, dtype=torch.float16, device=DEV) for _ in range(2))
    kq.kq_kv_append(st["qk"], st["cache"], q, k, v, st["positions"], st["slots"], q_out)
    kq.kq_kv_read(st["cache"], st["slots"], k_val, v_val)
    return {"q": q_out, "k": k_val, "v": v_val}


def _own_attn(st):
    import quantized_weight_streaming_gb300 as kq

    out = torch.empty_like(st["q"])
    kq.kq_attn_paged(st["cache"], st["q"], st["q_start"], st["kv_len"], st["table"], out, st["scale"], st["max_new"],
                     window=st["case"]["window"], ws=st["ws"])
    return out


def _plain_slots(st):
    p, t = st["case"]["page"], st["tokens"]
    cached, new, table, free = (st[n].long() for n in ("cached", "new", "table", "free"))
    old = (cached + p - 1) // p
    need = (cached + new + p - 1) // p - old
    ends = torch.cumsum(new, 0)
    start = ends - new
    first = torch.cumsum(need, 0) - need
    req = torch.repeat_interleave(torch.arange(new.shape[0], device=DEV), new, output_size=t)
    pos = cached[req] + torch.arange(t, device=DEV) - start[req]
    at = pos // p
    page = torch.where(at >= old[req], free[(first[req] + at - old[req]).clamp(min=0)], table[req, at])
    st["table"][req, at] = page.int()
    q_start = torch.cat((torch.zeros_like(ends[:1]), ends))
    return {"table": st["table"], "q_start": q_start.int(), "kv_len": (cached + new).int(), "positions": pos.int(),
            "slots": (page * p + pos % p).int(), "used": need.sum().reshape(1).int()}


def _plain_rope(x, weight, table, rope_dim):
    """RMS norm and rotation of float32 heads [tokens, heads, head_dim]."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight
    h = rope_dim // 2
    cos, sin = table[:, None, :h], table[:, None, h:]
    a, b = x[..., :h], x[..., h:rope_dim]
    return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., rope_dim:]), -1)


def _plain_qk(st):
    q, k, v = _views(st)
    table, rd = st["rope"][st["positions"].long()], st["case"]["rope_dim"]
    return _plain_rope(q.float(), st["q_weight"], table, rd), _plain_rope(k.float(), st["k_weight"], table, rd), v.float()


def _plain_norm(st):
    q, k, _ = _plain_qk(st)
    dt = st["x"].dtype
    return {"q": q.to(dt), "k": k.to(dt)}


def _plain_append(st):
    c = st["case"]
    d, hk = c["head_dim"], c["kv_heads"]
    q, k, v = _plain_qk(st)
    b = _token_bytes(*_quantize(k), *_quantize(v), d)  # [tokens, kv_heads, bytes]
    slots = st["slots"].long()
    data = st["data"].view(st["data"].shape[0], hk, c["page"] // GRANULE, -1)
    page, granule, token = slots // c["page"], slots % c["page"] // GRANULE, slots % GRANULE
    head = torch.arange(hk, device=DEV)
    data[page[:, None, None], head[None, :, None], granule[:, None, None], st["places"][token][:, None, :]] = b
    got = data[page[:, None], head[None, :], granule[:, None]]  # the granules of each token, as written
    kv = _unpack(got, d)
    at = token[:, None, None, None].expand(-1, hk, 1, d)
    return {"q": q.to(st["x"].dtype), "k": torch.gather(kv[0], 2, at)[:, :, 0].half(),
            "v": torch.gather(kv[1], 2, at)[:, :, 0].half()}


def _plain_attn(st):
    c, q = st["case"], st["q"]
    hq, hk, d, per = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"] // GRANULE
    t, b, rows = q.shape[0], st["kv_len"].shape[0], st["max_new"]
    n = -(-st["max_len"] // c["page"])
    g = st["data"].view(-1, hk, per, _granule_bytes(d))[st["table"][:, :n].long()]  # [b, pages, heads, per, bytes]
    k, v = _unpack(g.permute(0, 2, 1, 3, 4).reshape(b, hk, n * per, -1), d)
    k, v = k.reshape(b, hk, -1, d), v.reshape(b, hk, -1, d)
    start, kv_len = st["q_start"].long(), st["kv_len"].long()
    new = start[1:] - start[:-1]
    i = torch.arange(rows, device=DEV)
    at = (start[:-1, None] + i[None, :]).clamp(max=t - 1)
    qp = q[at].float().reshape(b, rows, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    s = torch.matmul(qp, k.transpose(-1, -2)).view(b, hk, hq // hk, rows, -1) * st["scale"]
    pos = (kv_len - new)[:, None] + i[None, :]  # the position of each query
    key = torch.arange(k.shape[2], device=DEV)
    see = key[None, None, :] <= pos[:, :, None]
    if c["window"]:
        see &= key[None, None, :] > pos[:, :, None] - c["window"]
    s = s.masked_fill(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = s.sum(-1, keepdim=True)
    o = torch.matmul(s.reshape(b, hk, -1, s.shape[-1]), v).view(b, hk, hq // hk, rows, d)
    o = torch.where(z > 0, o / z, torch.zeros_like(o))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, rows, hq, d)
    req = torch.repeat_interleave(torch.arange(b, device=DEV), new, output_size=t)
    return o[req, torch.arange(t, device=DEV) - start[req]].to(q.dtype)


_run_own = {"slots": _own_slots, "norm": _own_norm, "append": _own_append, "attn": _own_attn}
_run_plain = {"slots": _plain_slots, "norm": _plain_norm, "append": _plain_append, "attn": _plain_attn}


# ---- the definitions, in 64 bits -------------------------------------------------------------


def _bit_of(d, what):
    """Byte and shift of each (token, dimension) of a granule's keys or values, one at a time."""
    slabs, groups = _dims(d)
    wide = d // slabs
    at = np.zeros((GRANULE, d), dtype=np.int64)
    shift = np.zeros((GRANULE, d), dtype=np.int64)
    for t in range(GRANULE):
        for e in range(d):
            s, g, i = e // wide, e % wide // 32, e % 32
            if what == "k":
                at[t, e] = s * GRANULE * wide // 2 + t * wide // 2 + (i // 8 * groups + g) * 4 + i % 8 // 2
            else:
                block = GRANULE * d // 2 + (s * 2 + t // 8) * 8 * wide // 2
                at[t, e] = block + ((i // 4 * 4 + t % 8 // 2) * groups + g) * 4 + t % 2 * 2 + i % 4 // 2
            shift[t, e] = 4 * (i % 2)
    return torch.from_numpy(at).to(DEV), torch.from_numpy(shift).to(DEV)


def _scale_of(d, what):
    slabs, groups = _dims(d)
    t, e = np.meshgrid(np.arange(GRANULE), np.arange(d), indexing="ij")
    s, g = e * slabs // d, e % (d // slabs) // 32
    at = (s * GRANULE + t) * groups + g + (0 if what == "k" else GRANULE * d // 32)
    return torch.from_numpy(at.astype(np.int64)).to(DEV)


def _exact_rope(x, w, table, rd):
    x = x.double()
    x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()
    z = torch.complex(x[..., : rd // 2], x[..., rd // 2: rd])
    z = z * torch.complex(table[..., : rd // 2].double(), table[..., rd // 2:].double())[:, None]
    return torch.cat((z.real, z.imag, x[..., rd:]), -1)


def _exact_codes(x):
    """What the codes of x stand for, group by group of 32."""
    g = x.unflatten(-1, (-1, 32))
    i = torch.arange(32, device=DEV)
    at = torch.where(g.abs() == g.abs().amax(-1, keepdim=True), i, 32).amin(-1, keepdim=True)  # the first of the largest
    s = (torch.gather(g, -1, at) / -8).half().double()
    r = torch.nan_to_num(g / s, nan=0.0, posinf=0.0, neginf=0.0)
    r = torch.where(r >= 0, torch.floor(r + 0.5), torch.ceil(r - 0.5))
    return (r.clamp(-8, 7) * s).flatten(-2)


def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers: they have to be equal
    st = prepare(case, seed)
    if case["op"] in ("norm", "append"):
        q, k, v = _views(st)
        table = st["rope"][st["positions"].long()]
        q = _exact_rope(q, st["q_weight"], table, case["rope_dim"])
        k = _exact_rope(k, st["k_weight"], table, case["rope_dim"])
        if case["op"] == "norm":
            return {"q": q, "k": k}
        return {"q": q, "k": _exact_codes(k), "v": _exact_codes(v.double())}
    hq, hk, d, p = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    cached, new = _lengths(case)
    where = {w: (*_bit_of(d, w), _scale_of(d, w)) for w in "kv"}
    out, first = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV), 0
    for r in range(case["requests"]):
        n, total = int(new[r]), int(cached[r] + new[r])
        pages = st["table"][r, : -(-total // p)].long()
        g = st["data"][pages].unflatten(-1, (p // GRANULE, -1)).transpose(0, 1).flatten(1, 2)  # [heads, granules, bytes]
        scales = g[..., GRANULE * d:].contiguous().view(torch.float16)
        q = st["q"][first: first + n].double()
        pos = torch.arange(total - n, total, device=DEV)[:, None]
        key = torch.arange(total, device=DEV)[None, :]
        hidden = key > pos
        if case["window"]:
            hidden = hidden | (pos - key >= case["window"])
        for h in range(hk):
            kv = []
            for w in "kv":
                at, shift, sc = where[w]
                code = (g[h][:, at.flatten()].view(-1, GRANULE, d) >> shift.to(torch.uint8)) & 15
                kv.append(((code.double() - 8) * scales[h][:, sc.flatten()].view(-1, GRANULE, d).double()).flatten(0, 1)[:total])
            for i in range(h * (hq // hk), (h + 1) * (hq // hk)):
                s = (q[:, i] @ kv[0].T) * st["scale"]
                s = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
                out[first: first + n, i] = s @ kv[1]
        first += n
    return out
