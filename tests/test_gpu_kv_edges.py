"""GPU checks of the attention-step operators at the far ends of what they take:
scores beyond fp32's whole numbers, pages and lengths near 31 bits, windows as
long as an int, grids that the caller's bounds make large, and the paths that
only long prompts reach.  Statements and tolerances are those of test_gpu_kv.py
unless a test says otherwise."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import kv_reference as ref  # noqa: E402
from test_gpu_kv import ATTN_TOL, Step, dev, f64, ints, kq, near, status  # noqa: E402,F401


def repack(s):
    s.cache.data.copy_(dev(ref.pack(s.kc, s.ks, s.vc, s.vs)))


# ---- scores of any size ---------------------------------------------------------------


def _one_key_rows(s, window=0, apart=2.0**-16):
    """(rows whose largest score stands out, the value row of that key): FP64 scores a fraction `apart` of the row's largest
    magnitude apart; 2^-16 is 16 times what fp32 products of exact operands can lose.  Where that is 100 or more, every
    other key's weight is below 2^-100 and the output is the key's value."""
    group = s.hq // s.kc.shape[1]
    k, v = (np.nan_to_num(ref.values(c, x)) for c, x in ((s.kc, s.ks), (s.vc, s.vs)))
    q = f64(s.q)
    stands, want = np.zeros(q.shape[:2], bool), np.zeros(q.shape)
    for r, total in enumerate(s.kv_len):
        at = np.arange(total)
        kk, vv = (x[s.table[r, at // s.page], :, at % s.page] for x in (k, v))
        lo, hi = s.q_start[r], s.q_start[r + 1]
        for t in range(lo, hi):
            pos = total - (hi - lo) + (t - lo)
            first = max(0, pos - window + 1) if window else 0
            for h in range(s.hq):
                e = s.scale * (kk[first: pos + 1, h // group] @ q[t, h])
                order = np.argsort(e)
                gap = e[order[-1]] - e[order[-2]] if len(e) > 1 else np.inf
                stands[t, h] = gap > max(100.0, apart * np.abs(e).max())
                want[t, h] = vv[first + order[-1], h // group]
    return stands, want


def _large(kq, rng, dt, hq, hk, d, size, side, new, lens):
    """A step whose scores are `size` and more: key scales powers of two (their products with codes are exact in fp16);
    `side` 1 or -1: every score of that sign."""
    s = Step(kq, rng, lens, new, hq, hk, d, 32, dt)
    s.ks = np.where(np.isnan(s.ks), s.ks, np.sign(s.ks) * np.float16(0.25))
    if side:
        s.ks = np.abs(s.ks)
        s.kc = np.maximum(s.kc, 9)
        s.q = (s.q.abs() * side).contiguous()
    if dt == "f16":
        s.scale *= size
    else:
        s.q = (s.q.float() * size).to(s.q.dtype)
    repack(s)
    return s


@pytest.mark.parametrize("side", [0, 1, -1])
@pytest.mark.parametrize("dt,size", [("bf16", 1e7), ("bf16", 1e8), ("bf16", 3e8), ("bf16", 1e12), ("bf16", 1e30), ("f16", 1e8), ("f16", 1e20)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 1, 256), (14, 2, 64)])
def test_prompt_of_very_large_scores(kq, hq, hk, d, dt, size, side):
    """The softmax of 16-bit prompts ends and stays finite whatever the scores' size; where one key stands out, its value
    is the output."""
    rng = np.random.default_rng(31 + d)
    s = _large(kq, rng, dt, hq, hk, d, size, side, [70, 45], [170, 45])
    for window in (0, 30):
        out = f64(s.run(window))
        assert status(kq) == kq.KQ_OK
        assert np.all(np.isfinite(out))
        stands, want = _one_key_rows(s, window)
        assert stands.mean() > 0.5
        near(out[stands], want[stands], dt)


@pytest.mark.parametrize("side", [0, 1, -1])
@pytest.mark.parametrize("dt,size", [("f32", 1e6), ("f32", 1e7), ("f32", 5e7), ("f32", 1e8), ("f32", 1e12), ("f32", 1e30),
                                     ("bf16", 1e7), ("bf16", 1e8), ("bf16", 1e30), ("f16", 1e8), ("f16", 1e20)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 1, 256), (14, 2, 64)])
@pytest.mark.parametrize("values", [0, -10])
def test_decode_of_very_large_scores(kq, hq, hk, d, dt, size, side, values):
    """The same of the kernel for few query rows, in rows that one warp ends and rows that several share.  (16-bit rows: the
    tensor instruction keeps 13 bits or more of a product with a code, so scores a fraction 2^-9 apart stand out.)"""
    rng = np.random.default_rng(33 + d)
    s = _large(kq, rng, dt, hq, hk, d, size, side, [1, 2, 3, 1], [170, 45, 30, 2000])
    s.vs = (s.vs.astype(np.float32) * 2.0**values).astype(np.float16)
    repack(s)
    for window in (0, 30):
        out = f64(s.run(window))
        assert status(kq) == kq.KQ_OK
        assert np.all(np.isfinite(out))
        stands, want = _one_key_rows(s, window, 2.0**-16 if dt == "f32" else 2.0**-9)
        assert stands.mean() > 0.5
        near(out[stands], want[stands], dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 1, 256), (14, 2, 64)])
def test_prompt_of_non_finite_queries_stays_in_its_rows(kq, dt, hq, hk, d):
    rng = np.random.default_rng(32 + d)
    s = Step(kq, rng, [300, 90], [100, 60], hq, hk, d, 32, dt)
    a = s.check()
    bad = torch.zeros(a.shape[:2], dtype=torch.bool, device="cuda")
    for t, h, e, x in ((0, 3, 5, "nan"), (37, 0, 0, "inf"), (99, hq - 1, d - 1, "-inf"), (150, 1, 7, "nan")):
        s.q[t, h, e] = float(x)
        bad[t, h] = True
    b = s.run()
    assert status(kq) == kq.KQ_OK
    assert torch.equal(a[~bad], b[~bad])
    assert not torch.any(torch.isfinite(b[bad]))


# ---- pages and lengths near 31 bits -------------------------------------------------------


@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_of_more_than_2_31_bytes(kq, d):
    """One page whose granules pass 32-bit byte offsets, as where a cache is used as one contiguous block: the write
    (row by row and by windows), reading back, and both attention kernels, at its last slots."""
    rng = np.random.default_rng(41 + d)
    page = 16 * ((1 << 31) // (18 * d) + 100)
    cache = kq.KVCache(1, page, 1, d)
    assert cache.data.numel() > 1 << 31
    p = kq.QKNorm(4, 1, d, norm=False)
    for n in (30, 20000):  # 20000: more than 4 windows an SM
        x = dev(rng.standard_normal((2, n, 1, d)).astype(np.float32))
        small = kq.KVCache(-(-n // 16), 16, 1, d)
        kq.kq_kv_append(p, small, None, x[0], x[1], None, ints(np.arange(n)), None)
        slots = ints(page - n + np.arange(n))
        kq.kq_kv_append(p, cache, None, x[0], x[1], None, slots, None)
        got, want = (torch.empty(2, n, 1, d, device="cuda") for _ in range(2))
        kq.kq_kv_read(cache, slots, got[0], got[1])
        kq.kq_kv_read(small, ints(np.arange(n)), want[0], want[1])
        assert status(kq) == kq.KQ_OK
        assert torch.equal(got, want)
    k, v = f64(got)  # [n, 1, d]
    for dt, new, window in (("f32", 1, 400), ("bf16", 2, 33), ("bf16", 60, 100)):
        q = dev(rng.standard_normal((new, 4, d)).astype(np.float32)).to({"f32": torch.float32, "bf16": torch.bfloat16}[dt])
        out = torch.empty_like(q)
        ws = torch.empty(kq.kq_attn_workspace_bytes(cache, 4, 1, new, new), dtype=torch.uint8, device="cuda")
        kq.kq_attn_paged(cache, q, ints([0, new]), ints([page]), ints([[0]]), out, d ** -0.5, new, window=window, ws=ws)
        assert status(kq) == kq.KQ_OK
        want = ref.attention(f64(q), k.transpose(1, 0, 2)[None], v.transpose(1, 0, 2)[None], [0, new], [n], np.array([[0]]),
                             n, d ** -0.5, window)
        near(f64(out), want, dt)


@pytest.mark.parametrize("d", [64, 128])
def test_lengths_up_to_2_31(kq, d):
    """Requests of 2^31 - 1 and a few less keys (a table that names one page again and again), seen through a window; the
    slots behind the length and before the window hold NaN."""
    rng = np.random.default_rng(42)
    page, window = 1 << 20, 90
    kc, vc = (rng.integers(0, 16, (1, 1, page, d)).astype(np.uint8) for _ in range(2))
    ks, vs = (rng.uniform(0.05, 0.4, (1, 1, page, d // 32)).astype(np.float16) for _ in range(2))
    ks[:, :, : page - 400] = vs[:, :, : page - 400] = np.nan
    for length in ((1 << 31) - 1, (1 << 31) - 17, (1 << 31) - 64):
        cut = page - ((1 << 31) - length)
        s = [x.copy() for x in (ks, vs)]
        for x in s:
            x[:, :, cut:] = np.nan
        cache = kq.KVCache(1, page, 1, d, data=dev(ref.pack(kc, s[0], vc, s[1])))
        table = torch.zeros(1, 2048, dtype=torch.int32, device="cuda")
        k, v = (ref.values(c, x)[:, :, cut - 300: cut] for c, x in zip((kc, vc), s))
        for dt, new in (("f32", 1), ("f16", 2), ("bf16", 130)):
            q = dev(rng.standard_normal((new, 4, d)).astype(np.float32)).to(
                {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt])
            out = torch.empty_like(q)
            ws = torch.empty(kq.kq_attn_workspace_bytes(cache, 4, 1, new, new), dtype=torch.uint8, device="cuda")
            kq.kq_attn_paged(cache, q, ints([0, new]), ints([length]), table, out, d ** -0.5, new, window=window, ws=ws)
            assert status(kq) == kq.KQ_OK
            want = ref.attention(f64(q), k, v, [0, new], [300], np.array([[0]]), 300, d ** -0.5, window)
            near(f64(out), want, dt)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (14, 2, 64), (6, 1, 256), (2, 2, 128)])
def test_longest_windows_over_requests_of_more_tokens_than_keys(kq, dt, hq, hk, d):
    """A window of 2^31 - 1 keys and more is no window, also where a request's first tokens stand before its first key."""
    rng = np.random.default_rng(43 + d)
    s = Step(kq, rng, [5, 100, 1, 40, 0], [6, 150, 90, 41, 3], hq, hk, d, 32, dt)
    for window in ((1 << 31) - 1, (1 << 31) - 2, 1 << 40):
        s.check(window=window)
    few = Step(kq, rng, [5, 3, 1], [11, 7, 2], hq, hk, d, 32, dt)
    few.check(window=(1 << 31) - 1)


# ---- the cache write ----------------------------------------------------------------------


@pytest.mark.parametrize("d", [64, 128, 256])
def test_append_without_eps_reports_nothing_for_rows_that_are_not_there(kq, d):
    """eps = 0 and no rotation: tokens that are skipped, and the lanes past the last token, are no zero rows to norm."""
    rng = np.random.default_rng(51)
    p = kq.QKNorm(2, 2, d, eps=0.0)
    for n in (1, 3, 16, 41):
        cache = kq.KVCache(8, 16, 2, d)
        x = dev(rng.standard_normal((n, 2, d)).astype(np.float32))
        slots = np.arange(n)
        slots[n // 2] = -1
        kq.kq_kv_append(p, cache, None, x, x, None, ints(slots), None)
        assert status(kq) == kq.KQ_OK
    x[:] = 0  # a zero row that is there: 0 / 0
    kq.kq_kv_append(p, cache, None, x, x, None, ints(slots), None)
    assert status(kq) == kq.KQ_ERR_NONFINITE


def test_append_of_skipped_tokens_asks_for_no_position(kq):
    """Keys and values alone: a skipped token's position is not looked at, however many tokens there are; a written one's is,
    and its key is zero."""
    rng = np.random.default_rng(52)
    hk, d = 64, 64
    p = kq.QKNorm(hk, hk, d, d, None, None, dev(kq.kq_rope_table_host(10, d, 1e4)))
    for n in (20, 330):  # 330: windows of tokens, more than four an SM
        cache = kq.KVCache(24, 16, hk, d)
        x = dev(rng.standard_normal((n, hk, d)).astype(np.float32))
        slots, pos = np.arange(n), rng.integers(0, 10, n)
        slots[[3, 11]] = -1
        pos[[3, 11]] = -1, 10
        kq.kq_kv_append(p, cache, None, x, x, ints(pos), ints(slots), None)
        assert status(kq) == kq.KQ_OK
        pos[7] = 10
        kq.kq_kv_append(p, cache, None, x, x, ints(pos), ints(slots), None)
        assert status(kq) == kq.KQ_ERR_RANGE
        k, v = (torch.empty(n, hk, d, device="cuda") for _ in range(2))
        kq.kq_kv_read(cache, ints(slots), k, v)
        assert torch.all(k[7] == 0) and torch.all(k[8].abs().amax(-1) > 0) and torch.all(v[7].abs().amax(-1) > 0)


# ---- slot maps -----------------------------------------------------------------------------


@pytest.mark.parametrize("cached,new", [([3, 0, 7], [1_200_000_000, 1_200_000_000, 2]),
                                        ([3] + [0] * 2499, [1_000_000] * 2500),
                                        ([3, 0, 0, 2147483640, 5], [30, 2147483647, 2147483647, 7, 2147483647]),
                                        ([3, 16], [2147483640, 2147483640])])
def test_slot_map_of_lengths_past_31_bits(kq, cached, new):
    """Totals past 2^31 - 1 are held there and reported; the tokens within the capacity get their places."""
    page, stride, capacity = 16, 4, 50
    free = np.arange(50, 57)
    table = np.full((len(cached), stride), 9)
    o = [ints(np.full(n, -7)) for n in (len(cached) + 1, len(cached), capacity, capacity, 1)]
    t = ints(table)
    kq.kq_slot_map(ints(cached), ints(new), page, ints(free), t, *o)
    assert status(kq) == kq.KQ_ERR_RANGE
    q_start, kv_len, positions, slots, used = (x.cpu().numpy().astype(np.int64) for x in o)
    most = (1 << 31) - 1
    cut = np.minimum(new, most - np.asarray(cached))  # a length of its own past 31 bits is cut, too
    assert np.array_equal(q_start, np.minimum(np.concatenate([[0], np.cumsum(cut)]), most))
    assert np.array_equal(kv_len, np.asarray(cached) + cut)
    need = -(-kv_len // page) - (-(-np.asarray(cached) // page))
    assert used[0] == min(need.sum(), most)
    t = t.cpu().numpy()
    for i in range(capacity):
        r = int(np.searchsorted(q_start, i, side="right")) - 1
        pos = cached[r] + i - q_start[r]
        assert positions[i] == pos
        at = pos // page
        old = -(-cached[r] // page)
        first = int(need[:r].sum())
        want = -1
        if at < stride:
            want = 9 if at < old else (free[first + at - old] if first + at - old < len(free) else -1)
            assert t[r, at] == want
        assert slots[i] == (-1 if want < 0 else want * page + pos % page)


# ---- bounds of lengths that are far from the lengths -----------------------------------------


@pytest.mark.parametrize("requests,longest", [(1025, 300), (600, 300), (7, 3000)])
def test_attention_of_few_tokens_under_large_bounds(kq, requests, longest):
    """tokens and max_new are a capacity and an upper bound: as large as they may be, with 128 query heads on one key head,
    cut rows are joined as with the smallest that fit, bit by bit (7 requests: by other CTAs)."""
    import ctypes

    rng = np.random.default_rng(61)
    s = Step(kq, rng, rng.integers(0, longest, requests), [1] * requests, 128, 1, 64, 16, "f32")
    want = s.run()
    assert status(kq) == kq.KQ_OK
    first = ref.attention(f64(s.q[:7]), np.nan_to_num(ref.values(s.kc, s.ks)), np.nan_to_num(ref.values(s.vc, s.vs)),
                          s.q_start[:8], s.kv_len[:7], s.table, 16, s.scale, 0)
    near(f64(want[:7]), first, "f32")
    tokens = (1 << 31) // 8192 - 1
    n = kq.kq_attn_workspace_bytes(s.cache, 128, requests, tokens, tokens)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.full(s.q.shape, 7.0, device="cuda")
    q_start, kv_len, table = ints(s.q_start), ints(s.kv_len), ints(s.table)
    view = lambda t: ctypes.byref(kq.kq_heads(t.data_ptr(), t.stride(0), t.stride(1)))  # noqa: E731
    assert kq.lib().kq_attn_paged(ctypes.byref(s.cache.desc), kq.KQ_F32, 128, view(s.q), q_start.data_ptr(), kv_len.data_ptr(),
                                  table.data_ptr(), table.shape[1], requests, tokens, tokens, s.scale, 0, view(out),
                                  ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream) == kq.KQ_OK
    assert status(kq) == kq.KQ_OK
    assert torch.equal(out, want)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 1, 256), (14, 2, 64)])
def test_attention_under_large_bounds(kq, dt, hq, hk, d):
    """Rows in few and in many parts, requests that see nothing, a malformed one and prompts, where the bounds allow a
    hundred thousand row tiles."""
    rng = np.random.default_rng(62 + d)
    lens = np.array([5000, 1, 0, 77, 3, 640, 0, 300] + [20] * 60)
    new = np.array([1, 1, 2, 3, 9, 70, 5, 1] + [1] * 60)
    s = Step(kq, rng, lens, new, hq, hk, d, 32, dt)
    q = s.q
    s.q = torch.cat([q, q.new_zeros(9000, hq, d)])
    out = s.run(max_new=9000)
    assert status(kq) == kq.KQ_OK
    assert torch.all(out[len(q):] == 7)
    s.q = q
    want = s.want()
    near(f64(out[: len(q)]), want, dt)
    one = Step(kq, rng, [20000], [1], hq, hk, d, 32, dt)  # one row tile in a thousand parts
    q = one.q
    one.q = torch.cat([q, q.new_zeros(60000, hq, d)])
    out = one.run(max_new=60000)
    assert status(kq) == kq.KQ_OK
    one.q = q
    near(f64(out[:1]), one.want(), dt)


# ---- paths that only long prompts reach, and what else a step promises --------------------------


def _prompt_slots(rng, tokens, page, pages):
    """Slots of a prompt step: requests that go on in the middle of a granule, tokens skipped within a run, and a stretch in
    no order at all (a window of 32 tokens then falls on more granules than it gathers)."""
    order = rng.permutation(pages)
    slots, at = np.full(tokens, -1), 0
    i = 0
    while i < tokens:
        n = int(min(tokens - i, rng.integers(1, 120)))
        first = int(rng.integers(0, page))
        need = -(-(first + n) // page)
        pos = first + np.arange(n)
        slots[i: i + n] = order[at + pos // page] * page + pos % page
        at += need
        i += n
    mixed = slice(tokens // 2, tokens // 2 + 100)
    slots[mixed] = rng.permutation(slots[mixed])
    slots[rng.random(tokens) < 0.05] = -1
    slots[-1] = -1
    return slots


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,rd,inter,tokens,page", [(128, 128, False, 700, 32), (128, 64, True, 613, 48), (64, 64, False, 650, 16),
                                                   (64, 32, True, 621, 32), (256, 64, False, 330, 16), (256, 256, True, 313, 64),
                                                   (128, 0, False, 641, 16)])
def test_append_of_prompts(kq, dt, d, rd, inter, tokens, page):
    """The windowed write (from 608 windows of 32 or 16 tokens of a head on): values are the host SCALE4 quantizer's bytes,
    keys within half a step of FP64, every byte that of the same tokens written in small calls, other slots untouched."""
    rng = np.random.default_rng(71 + d + tokens)
    hq, hk = 5, 32
    assert -(-tokens // (16 if d == 256 else 32)) * hk >= 608
    x = dev(rng.standard_normal((tokens, (2 * hq + 2 * hk) * d)).astype(np.float32) * 1.7,
            {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt])
    q = x[:, : 2 * hq * d].unflatten(1, (hq, 2 * d))[:, :, :d]
    k, v = x[:, 2 * hq * d: (2 * hq + hk) * d].unflatten(1, (hk, d)), x[:, (2 * hq + hk) * d:].unflatten(1, (hk, d))
    v[3, 1, :32] = 0
    v[3, 1, 7], v[3, 1, 20] = -2.0, 2.0
    pages = tokens // 4
    slots, pos = _prompt_slots(rng, tokens, page, pages), rng.integers(0, 300, tokens)
    table = kq.kq_rope_table_host(300, rd, 1e4) if rd else None
    w = rng.uniform(0.5, 1.5, d).astype(np.float32)
    p = kq.QKNorm(hq, hk, d, rd, None, dev(w), dev(table) if rd else None, interleaved=inter)
    cache, small = (kq.KVCache(pages, page, hk, d) for _ in range(2))
    for c in (cache, small):
        c.data.fill_(0x5A)
    qo, q2, k2 = (torch.empty(tokens, h, d, dtype=x.dtype, device="cuda") for h in (hq, hq, hk))
    kq.kq_kv_append(p, cache, q, k, v, ints(pos), ints(slots), qo)
    assert status(kq) == kq.KQ_OK
    for i in range(0, tokens, 64):
        j = min(tokens, i + 64)
        kq.kq_kv_append(p, small, None, k[i:j], v[i:j], ints(pos[i:j]), ints(slots[i:j]), None)
    kq.kq_qk_norm_rope(p, q, k, ints(pos), q2, k2)
    assert status(kq) == kq.KQ_OK
    assert torch.equal(qo, q2)
    assert torch.equal(cache.data, small.data)
    live = slots >= 0
    at = slots[live]
    kc, ks, vc, vs = (y[at // page, :, at % page] for y in ref.unpack(cache.data.cpu().numpy(), page, d))
    blocks = kq.kq_quantize_scale4(v.float().cpu().numpy()[live].reshape(-1, d)).reshape(live.sum(), hk, d // 32, 18)
    assert np.array_equal(vs.view(np.uint16), blocks[..., :2].copy().view(np.uint16)[..., 0])
    assert np.array_equal(vc, np.stack([blocks[..., 2:] & 15, blocks[..., 2:] >> 4], -1).reshape(live.sum(), hk, d))
    want = ref.norm_rope(f64(k), w, table, pos, rd, 1e-6, True, inter)[live]
    step = np.repeat(np.abs(ks.astype(np.float64)), 32, -1)
    # half a step, or up to one where 8 steps is the clamped end, and the fp16 rounding of the scale (8 steps of 2^-11)
    assert np.all(np.abs(ref.values(kc, ks) - want) <= step * np.where(kc == 15, 1.01, 0.505) + 1e-6)
    rest = np.ones(pages * page, bool)
    rest[at] = False
    blank = kq.KVCache(pages, page, hk, d)
    blank.data.fill_(0x5A)
    for y, z in zip(ref.unpack(cache.data.cpu().numpy(), page, d), ref.unpack(blank.data.cpu().numpy(), page, d)):
        y, z = (a.transpose(0, 2, 1, 3).reshape(pages * page, -1)[rest] for a in (y, z))
        assert np.array_equal(y.view(np.uint16) if y.dtype == np.float16 else y, z.view(np.uint16) if z.dtype == np.float16 else z)


def test_slot_map_repeated_writes_the_same(kq):
    rng = np.random.default_rng(72)
    cached, new = rng.integers(0, 300, 300), rng.integers(0, 40, 300)
    t, stride = int(new.sum()), 30
    need = int((-(-(cached + new) // 16) - (-(-cached // 16))).sum())
    args = [ints(cached), ints(new), 16, ints(rng.permutation(need))]
    table = ints(rng.integers(0, 1000, (300, stride)))
    o = [ints(np.zeros(n)) for n in (301, 300, t, t, 1)]
    kq.kq_slot_map(*args, table, *o)
    first = [x.clone() for x in (table, *o)]
    for x in o:
        x.fill_(-3)
    kq.kq_slot_map(*args, table, *o)
    assert status(kq) == kq.KQ_OK
    assert all(torch.equal(x, y) for x, y in zip(first, (table, *o)))


@pytest.mark.parametrize("dt,new", [("f32", [1, 1, 1, 1]), ("bf16", [1, 3, 1, 0]), ("f16", [90, 1, 200, 7])])
def test_whole_step_in_a_cuda_graph(kq, dt, new):
    """slot map -> append -> attention captured once and replayed over other lengths and values: the same bits as the calls."""
    rng = np.random.default_rng(73)
    hq, hk, d, page, pages, t, r = 8, 2, 128, 16, 200, sum(new), len(new)
    typ = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dt]
    rope = dev(kq.kq_rope_table_host(900, d, 1e4))
    p = kq.QKNorm(hq, hk, d, d, None, None, rope)

    class State:
        def __init__(self):
            self.cache = kq.KVCache(pages, page, hk, d)
            self.cached, self.new, self.free = ints(np.zeros(r)), ints(new), ints(np.arange(pages))
            self.table = ints(np.zeros((r, 60)))
            self.o = [ints(np.zeros(n)) for n in (r + 1, r, t, t, 1)]
            self.x = torch.zeros(t, hq + 2 * hk, d, dtype=typ, device="cuda")
            self.qo, self.out = (torch.zeros(t, hq, d, dtype=typ, device="cuda") for _ in range(2))
            n = kq.kq_attn_workspace_bytes(self.cache, hq, r, t, max(new))
            self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")

        def step(self):
            q_start, kv_len, positions, slots, used = self.o
            kq.kq_slot_map(self.cached, self.new, page, self.free, self.table, *self.o)
            kq.kq_kv_append(p, self.cache, self.x[:, :hq], self.x[:, hq: hq + hk], self.x[:, hq + hk:], positions, slots, self.qo)
            kq.kq_attn_paged(self.cache, self.qo, q_start, kv_len, self.table, self.out, d ** -0.5, max(new), ws=self.ws)

    plain, captured = State(), State()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        captured.step()  # first launches of the kernels, outside the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured.step()
    done, total = 0, np.zeros(r, int)
    for i in range(4):
        x = dev(rng.standard_normal((t, hq + 2 * hk, d)).astype(np.float32), typ)
        free = np.concatenate([np.arange(done, pages), np.arange(done)])
        for s in (plain, captured):
            s.x.copy_(x)
            s.cached.copy_(ints(total))
            s.free.copy_(ints(free))
        plain.step()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(plain.out, captured.out) and torch.equal(plain.table, captured.table)
        kc, ks, vc, vs = ref.unpack(plain.cache.data.cpu().numpy(), page, d)
        want = ref.attention(f64(plain.qo), ref.values(kc, ks), ref.values(vc, vs), plain.o[0].cpu().numpy(), total + new,
                             plain.table.cpu().numpy(), page, d ** -0.5, 0)
        near(f64(plain.out), want, dt)
        total += new
        done += int(plain.o[4].item())
    assert status(kq) == kq.KQ_OK
