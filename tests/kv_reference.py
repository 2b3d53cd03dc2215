"""Plain FP64 statements of the attention-step operators (kq_slot_map,
kq_qk_norm_rope, kq_kv_append, kq_attn_paged) and the cache layout one element
at a time, for the tests.  Shares no code with the library."""
import numpy as np

GRANULE = 16


def block_bytes(page, d):
    return page * d * 9 // 8


def places(d):
    """Byte and shift of each (token, dimension) of a granule's keys and values, and the fp16 index of its scales."""
    wide = min(d, 128)
    groups = wide // 32
    t, e = np.meshgrid(np.arange(GRANULE), np.arange(d), indexing="ij")
    s, i = e // wide, e % wide
    g, j = i // 32, i % 32
    key = s * (GRANULE * wide // 2) + t * (wide // 2) + ((j // 8) * groups + g) * 4 + (j % 8) // 2
    unit = ((((s * 2 + t // 8) * 8 + j // 4) * 4 + (t % 8) // 2) * groups + g) * 2 + t % 2
    value = GRANULE * d // 2 + unit * 2 + (j % 4) // 2
    scale = GRANULE * d // 2 + (s * GRANULE + t) * groups + g  # fp16 index from the granule's start
    return key, value, 4 * (j % 2), scale, scale + d // 2


def pack(kc, ks, vc, vs):
    """Codes uint8 and scales fp16 [pages, heads, page, d] and [pages, heads, page, d / 32] -> bytes
    [pages, heads, block_bytes]."""
    pages, heads, page, d = kc.shape
    key, value, shift, si, vi = places(d)
    out = np.zeros((pages, heads, page // GRANULE, 18 * d), dtype=np.uint8)
    half = out.view(np.float16)
    for codes, at in ((kc, key), (vc, value)):
        c = codes.reshape(pages, heads, -1, GRANULE, d).astype(np.uint8)
        for t in range(GRANULE):
            for sh in (0, 4):
                m = shift[t] == sh
                out[..., at[t][m]] |= c[..., t, m] << sh
    for scales, at in ((ks, si), (vs, vi)):
        half[..., at[:, ::32]] = scales.reshape(pages, heads, -1, GRANULE, d // 32)
    return out.reshape(pages, heads, -1)


def unpack(data, page, d):
    """bytes -> (kc, ks, vc, vs), the inverse of pack."""
    pages, heads = data.shape[:2]
    key, value, shift, si, vi = places(d)
    g = data.reshape(pages, heads, page // GRANULE, 18 * d)
    half = g.view(np.float16)
    r = []
    for at, sc in ((key, si), (value, vi)):
        r.append(((g[..., at] >> shift.astype(np.uint8)) & 15).reshape(pages, heads, page, d))
        r.append(half[..., sc[:, ::32]].reshape(pages, heads, page, d // 32))
    return tuple(r)


def values(codes, scales):
    return (codes.astype(np.float64) - 8) * np.repeat(scales.astype(np.float64), 32, axis=-1)


def norm_rope(x, weight, table, positions, rope_dim, eps, norm=True, interleaved=False):
    """FP64 [tokens, heads, d]; positions outside the table give zeros."""
    x = x.astype(np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight.astype(np.float64)
    if rope_dim:
        ok = (positions >= 0) & (positions < len(table))
        tab = table.astype(np.float64)[np.where(ok, positions, 0)][:, None]
        c, s = tab[..., : rope_dim // 2], tab[..., rope_dim // 2:]
        y = x.copy()
        a_at = slice(0, rope_dim, 2) if interleaved else slice(0, rope_dim // 2)
        b_at = slice(1, rope_dim, 2) if interleaved else slice(rope_dim // 2, rope_dim)
        a, b = x[..., a_at], x[..., b_at]
        y[..., a_at] = a * c - b * s
        y[..., b_at] = b * c + a * s
        x = y * ok[:, None, None]
    return x


def slot_map(cached, new, page, free, table, tokens):
    """(table, q_start, kv_len, positions, slots, used, out of range) one token at a time."""
    table = table.copy()
    q_start, kv_len, positions, slots = [0], [], np.zeros(tokens, np.int64), np.full(tokens, -1, np.int64)
    used, bad, t = 0, False, 0
    for r, (c, n) in enumerate(zip(cached.tolist(), new.tolist())):
        bad |= c < 0 or n < 0
        c, n = max(c, 0), max(n, 0)
        old, need = -(-c // page), -(-(c + n) // page) - (-(-c // page))
        for i in range(n):
            pos, at = c + i, (c + i) // page
            if t < tokens:
                p = -1
                if at >= table.shape[1]:
                    bad = True
                elif at < old:
                    p = int(table[r, at])
                else:
                    f = used + at - old
                    if f < len(free):
                        p = int(free[f])
                    else:
                        bad = True
                    table[r, at] = p
                positions[t] = pos
                slots[t] = -1 if p < 0 else p * page + pos % page
            else:
                bad = True
            t += 1
        used += need
        q_start.append(t)
        kv_len.append(c + n)
    return table, np.array(q_start), np.array(kv_len), positions, slots, used, bad


def attention(q, k, v, q_start, kv_len, table, page, scale, window, q_dtype=np.float64):
    """FP64 [tokens, q_heads, d] from k, v [pages, kv_heads, page, d] (FP64 values)."""
    out = np.zeros(q.shape, dtype=np.float64)
    group = q.shape[1] // k.shape[1]
    for r in range(len(kv_len)):
        lo, hi, total = int(q_start[r]), int(q_start[r + 1]), int(kv_len[r])
        if hi == lo or total == 0:
            continue
        pages = table[r, : -(-total // page)]
        kk = k[pages].transpose(1, 0, 2, 3).reshape(k.shape[1], -1, k.shape[3])[:, :total]
        vv = v[pages].transpose(1, 0, 2, 3).reshape(k.shape[1], -1, k.shape[3])[:, :total]
        for t in range(lo, hi):
            pos = total - (hi - lo) + (t - lo)
            first = max(0, pos - window + 1) if window else 0
            if pos < 0:
                continue
            for h in range(q.shape[1]):
                s = scale * (kk[h // group, first: pos + 1] @ q[t, h].astype(np.float64))
                p = np.exp(s - s.max())
                out[t, h] = (p / p.sum()) @ vv[h // group, first: pos + 1]
    return out
