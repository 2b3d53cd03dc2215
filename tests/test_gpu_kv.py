"""GPU checks of the attention-step operators against plain FP64 statements
(kv_reference.py): slot maps, norms and rotation, the 4-bit cache write, and
attention over the cache, at the sizes and masks where each can go wrong.

Tolerances.  fp32 results: every operation rounds relative to 2^-24, and the
longest chain (a score's sum over 256 dimensions, or a value sum) adds a few
dozen of them at random: 1e-5 of a row's norm for attention, 2e-6 for norms.
16-bit results of norms: one rounding of an fp32 value, half an ulp plus 2e-6.
16-bit attention: the output, the probabilities, and (on tensor-core tiles) the
dequantized keys and values are each rounded to at most 2^-11 relative (bf16
output: 2^-8), independent of one another, and a score's rounding is amplified
by its own size, below 4 here: 4 * 2^-11 (+ 2^-8) of a row's norm."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import kv_reference as ref  # noqa: E402

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ULP = {"f32": 0.0, "f16": 2.0**-11, "bf16": 2.0**-8}
ATTN_TOL = {"f32": 1e-5, "f16": 4 * 2.0**-11, "bf16": 4 * 2.0**-11 + 2.0**-8}


@pytest.fixture(scope="module")
def kq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import quantized_weight_streaming_gb300 as kq

    torch.cuda.set_device(0)
    kq.kq_device_status(True)
    return kq


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def ints(a):
    return dev(np.asarray(a, dtype=np.int32))


def status(kq):
    torch.cuda.synchronize()
    return kq.kq_device_status(True)


# ---- slot maps ------------------------------------------------------------------


def _slot_map(kq, cached, new, page, free, table, tokens, stream=None):
    r = len(cached)
    out = dict(q_start=ints(np.full(r + 1, -7)), kv_len=ints(np.full(r, -7)), positions=ints(np.full(tokens, -7)),
               slots=ints(np.full(tokens, -7)), used=ints([-7]))
    t = ints(table)
    kq.kq_slot_map(ints(cached), ints(new), page, ints(free), t, out["q_start"], out["kv_len"], out["positions"],
                   out["slots"], out["used"], stream=stream)
    got_status = status(kq)
    want = ref.slot_map(np.asarray(cached), np.asarray(new), page, free, np.asarray(table), tokens)
    for name, w in zip(("table", "q_start", "kv_len", "positions", "slots", "used"), want):
        g = (t if name == "table" else out[name]).cpu().numpy()
        assert np.array_equal(g, np.asarray(w).reshape(g.shape)), name
    assert got_status == (kq.KQ_ERR_RANGE if want[-1] else kq.KQ_OK)


@pytest.mark.parametrize("requests,page,most_new", [(1, 16, 1), (1, 32, 5000), (7, 48, 100), (256, 32, 1), (300, 16, 40),
                                                    (1024, 16, 3), (1025, 64, 9), (2500, 16, 2)])
def test_slot_map(kq, requests, page, most_new):
    rng = np.random.default_rng(requests + page)
    cached, new = rng.integers(0, 300, requests), rng.integers(0, most_new + 1, requests)
    cached[:: 3] = cached[:: 3] // page * page  # some end on a page
    new[0] = max(new[0], 1)
    stride = int((cached + new).max() - 1) // page + 1
    need = int((-(-(cached + new) // page) + (-cached // page)).sum())
    free = rng.permutation(100000)[: need + 3]
    table = rng.integers(0, 1000, (requests, stride))
    _slot_map(kq, cached, new, page, free, table, int(new.sum()))
    _slot_map(kq, cached, new, page, free, table, int(new.sum()) + 77)  # spare capacity


def test_slot_map_nothing_new_and_shortages(kq):
    table = np.arange(12).reshape(3, 4)
    _slot_map(kq, [5, 0, 16], [0, 0, 0], 16, [], table, 0)
    _slot_map(kq, [5, 0, 16], [0, 0, 0], 16, [], table, 6)
    _slot_map(kq, [5, 0, 16], [30, 2, 20], 16, [70, 71], table, 52)  # free list runs out
    _slot_map(kq, [60, 0, 16], [30, 2, 20], 16, list(range(50, 90)), table, 52)  # a row runs out
    _slot_map(kq, [5, 0, 16], [30, 2, 20], 16, list(range(50, 90)), table, 40)  # capacity runs out
    _slot_map(kq, [-5, 3, 16], [3, -2, 1], 16, list(range(50, 90)), table, 10)  # negative lengths


def test_slot_map_on_another_stream_and_again(kq):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _slot_map(kq, [5, 0, 16], [30, 2, 20], 16, list(range(50, 90)), np.arange(12).reshape(3, 4), 52, stream=s)


# ---- norms and rotation -----------------------------------------------------------


def _qk_inputs(rng, tokens, hq, hk, d, dt, gap=0, scale=1.0):
    """q, k, v as views of fused rows, `gap` elements between query heads."""
    wide = d + gap
    x = rng.standard_normal((tokens, hq * wide + 2 * hk * d)).astype(np.float32) * scale
    t = dev(x, TYPES[dt])
    q = t[:, : hq * wide].unflatten(1, (hq, wide))[:, :, :d]
    k = t[:, hq * wide: hq * wide + hk * d].unflatten(1, (hk, d))
    v = t[:, hq * wide + hk * d:].unflatten(1, (hk, d))
    return q, k, v


def f64(t):
    return t.double().cpu().numpy()


def _near_rows(got, want, dt, tol=2e-6):
    norm = np.linalg.norm(want, axis=-1, keepdims=True) / np.sqrt(want.shape[-1])
    assert np.all(np.abs(got - want) <= ULP[dt] * np.abs(want) + tol * (np.abs(want) + norm) + 1e-7)


CASES = [(1, 32, 8, 128, 128, 0), (3, 24, 4, 256, 64, 256), (17, 14, 2, 64, 64, 0), (5, 1, 1, 128, 32, 8), (2, 5, 5, 64, 16, 0),
         (700, 32, 8, 128, 128, 0), (511, 6, 3, 256, 256, 64), (2, 3, 1, 128, 0, 0), (33, 7, 7, 128, 112, 0)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,hq,hk,d,rd,gap", CASES)
def test_norm_rope(kq, dt, tokens, hq, hk, d, rd, gap):
    rng = np.random.default_rng(tokens + d)
    q, k, _ = _qk_inputs(rng, tokens, hq, hk, d, dt, gap, 2.5)
    table = kq.kq_rope_table_host(900, rd, 1e6) if rd else None
    pos = rng.integers(0, 900, tokens)
    wq, wk = (rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2))
    for norm, inter in ((True, False), (True, True), (False, False)):
        p = kq.QKNorm(hq, hk, d, rd, dev(wq) if norm else None, dev(wk) if norm and tokens != 3 else None,
                      dev(table) if rd else None, eps=1e-5, interleaved=inter, norm=norm)
        qo, ko = torch.empty(tokens, hq, d, dtype=q.dtype, device="cuda"), torch.empty(tokens, hk, d + 8, dtype=q.dtype,
                                                                                      device="cuda")[..., :d]
        kq.kq_qk_norm_rope(p, q, k, ints(pos), qo, ko)
        assert status(kq) == kq.KQ_OK
        for x, w, y in ((q, wq, qo), (k, wk if tokens != 3 else None, ko)):
            _near_rows(f64(y), ref.norm_rope(f64(x), w, table, pos, rd, 1e-5, norm, inter), dt)


def test_norm_rope_in_place_zero_rows_and_bad_positions(kq):
    rng = np.random.default_rng(0)
    q, k, _ = _qk_inputs(rng, 6, 4, 2, 128, "f32")
    q[1], k[2] = 0, 0  # a row of zeros stays zero: eps keeps the norm finite
    table = kq.kq_rope_table_host(50, 128, 1e4)
    p = kq.QKNorm(4, 2, 128, 128, None, None, dev(table))
    pos = np.array([0, 49, 7, 50, -1, 3])
    want = [ref.norm_rope(f64(x), None, table, pos, 128, 1e-6) for x in (q, k)]
    kq.kq_qk_norm_rope(p, q, k, ints(pos), q, k)  # in place, strided
    assert status(kq) == kq.KQ_ERR_RANGE
    for x, w in zip((q, k), want):
        _near_rows(f64(x), w, "f32")
        assert torch.all(x[3:5] == 0)
    kq.kq_qk_norm_rope(p, q[:0], k[:0], ints(pos), q[:0], k[:0])  # no tokens
    assert status(kq) == kq.KQ_OK


# ---- the cache write ----------------------------------------------------------------


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,hq,hk,d,rd,gap", CASES)
def test_append(kq, dt, tokens, hq, hk, d, rd, gap):
    """Values (taken as they are) get exactly the bytes of the host SCALE4 quantizer; keys are within half a step of the
    FP64 keys; queries are those of kq_qk_norm_rope; other slots keep their bytes; kq_kv_read gives the values back."""
    rng = np.random.default_rng(7 * tokens + d)
    page = 48 if tokens == 17 else 32
    q, k, v = _qk_inputs(rng, tokens, hq, hk, d, dt, gap, 1.7)
    v[0, 0, :32] = 0
    v[0, 0, 5], v[0, 0, 9] = 2.0, -2.0  # a tie of magnitude: the first counts
    v[-1, -1, 32:64] = 0  # a group of zeros
    pages = -(-tokens // page) + 4
    slots = rng.permutation(pages * page)[:tokens]
    skipped = tokens > 16
    if skipped:
        slots[3] = -1
    cache = kq.KVCache(pages, page, hk, d)
    cache.data.fill_(0xA5)
    before = cache.data.cpu().numpy().copy()
    table = kq.kq_rope_table_host(900, rd, 1e6) if rd else None
    pos = rng.integers(0, 900, tokens)
    w = [rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2)]
    p = kq.QKNorm(hq, hk, d, rd, dev(w[0]), dev(w[1]), dev(table) if rd else None)
    qo = torch.empty(tokens, hq, d, dtype=q.dtype, device="cuda")
    kq.kq_kv_append(p, cache, q, k, v, ints(pos), ints(slots), qo)
    assert status(kq) == kq.KQ_OK
    q2, k2 = torch.empty_like(qo), torch.empty(tokens, hk, d, dtype=q.dtype, device="cuda")
    kq.kq_qk_norm_rope(p, q, k, ints(pos), q2, k2)
    assert torch.equal(qo, q2)
    got = ref.unpack(cache.data.cpu().numpy(), page, d)
    rest = ref.unpack(before, page, d)
    live = slots >= 0
    at = slots[live]
    kc, ks, vc, vs = (x[at // page, :, at % page] for x in got)
    blocks = kq.kq_quantize_scale4(v.float().cpu().numpy()[live].reshape(-1, d)).reshape(live.sum(), hk, d // 32, 18)
    assert np.array_equal(vs.view(np.uint16), blocks[..., :2].copy().view(np.uint16)[..., 0])
    nib = np.stack([blocks[..., 2:] & 15, blocks[..., 2:] >> 4], -1).reshape(live.sum(), hk, d)
    assert np.array_equal(vc, nib)
    want = ref.norm_rope(f64(k), w[1], table, pos, rd, 1e-6)[live]
    step = np.repeat(np.abs(ks.astype(np.float64)), 32, -1)
    err = np.abs(ref.values(kc, ks) - want)
    # half a step, or up to one where 8 steps is the clamped end, and the fp16 rounding of the scale (8 steps of 2^-11)
    assert np.all(err <= step * np.where(kc == 15, 1.01, 0.505) + 1e-6)
    m = np.abs(want).reshape(*want.shape[:-1], -1, 32).max(-1)
    assert np.all(np.abs(np.abs(ks.astype(np.float64)) * 8 - m) <= m * 2.0**-10)
    keep = np.ones((pages, page), bool)
    keep[at // page, at % page] = False
    for x, y in zip(got, rest):
        x, y = x.transpose(0, 2, 1, 3)[keep], y.transpose(0, 2, 1, 3)[keep]
        assert np.array_equal(x.view(np.uint16) if x.dtype == np.float16 else x, y.view(np.uint16) if y.dtype == np.float16 else y)
    kr, vr = (torch.full((tokens, hk, d), 9.0, device="cuda") for _ in range(2))
    kq.kq_kv_read(cache, ints(slots), kr, vr)
    assert status(kq) == kq.KQ_OK
    assert np.array_equal(f64(kr)[live], ref.values(kc, ks)) and np.array_equal(f64(vr)[live], ref.values(vc, vs))
    assert torch.all(kr[~torch.from_numpy(live)] == 0)
    r16 = [torch.empty(tokens, hk, d, dtype=TYPES[dt], device="cuda") for _ in range(2)]
    kq.kq_kv_read(cache, ints(slots), *r16)
    assert torch.equal(r16[0], kr.to(TYPES[dt])) and torch.equal(r16[1], vr.to(TYPES[dt]))


def test_append_exact_keys_without_norm(kq):
    """Without norm and rotation keys too are the host quantizer's bytes, at halves of a step and tiny scales."""
    rng = np.random.default_rng(3)
    x = (rng.integers(-16, 17, (64, 2, 128)) * 0.5).astype(np.float32)  # d = 1 where the largest is 8: many exact halves
    x[:, :, ::32] = np.where(rng.random((64, 2, 4)) < 0.5, 8.0, -8.0)
    x[10:20] *= 1e-7
    x[20:30] = rng.standard_normal((10, 2, 128)) * 1e-6
    x[30:40] = rng.standard_normal((10, 2, 128)) * 4e4
    k = dev(x)
    cache = kq.KVCache(4, 16, 2, 128)
    p = kq.QKNorm(2, 2, 128, norm=False)
    kq.kq_kv_append(p, cache, None, k, k, None, ints(np.arange(64)), None)
    assert status(kq) == kq.KQ_OK
    kc, ks, vc, vs = (a.transpose(0, 2, 1, 3).reshape(64, 2, -1) for a in ref.unpack(cache.data.cpu().numpy(), 16, 128))
    blocks = kq.kq_quantize_scale4(x.reshape(-1, 128)).reshape(64, 2, 4, 18)
    nib = np.stack([blocks[..., 2:] & 15, blocks[..., 2:] >> 4], -1).reshape(64, 2, 128)
    for c, s in ((kc, ks), (vc, vs)):
        assert np.array_equal(s.view(np.uint16), blocks[..., :2].copy().view(np.uint16)[..., 0])
        assert np.array_equal(c, nib)


def test_append_reports_nonfinite_overflow_and_bad_slots(kq):
    k = torch.ones(4, 1, 64, device="cuda")
    p = kq.QKNorm(1, 1, 64, norm=False)

    def run(k, v, slots):
        cache = kq.KVCache(1, 16, 1, 64)
        kq.kq_kv_append(p, cache, None, k, v, None, ints(slots), None)
        s = status(kq)
        kr, vr = torch.empty(4, 1, 64, device="cuda"), torch.empty(4, 1, 64, device="cuda")
        kq.kq_kv_read(cache, ints([0, 1, 2, 3]), kr, vr)
        assert status(kq) == kq.KQ_OK
        return s, kr, vr

    v = k.clone()
    v[1, 0, 40] = float("nan")
    s, kr, vr = run(k, v, [0, 1, 2, 3])
    assert s == kq.KQ_ERR_NONFINITE
    assert torch.all(vr[1, 0, 32:].isnan()) and torch.all(vr[1, 0, :32] == 1) and torch.all(kr == 1)
    v = k.clone()
    v[2, 0, 3] = float("-inf")
    s, kr, vr = run(k, v, [0, 1, 2, 3])
    assert s == kq.KQ_ERR_NONFINITE and torch.all(vr[2, 0, :32].isnan())
    v = k.clone()
    v[2, 0, 3] = 6e5
    s, kr, vr = run(k, v, [0, 1, 2, 3])
    assert s == kq.KQ_ERR_RANGE and torch.all(vr[2, 0, :32].isnan()) and torch.all(vr[2, 0, 32:] == 1)
    v[2, 0, 3] = float("nan")
    s, kr, vr = run(k, v, [0, 1, -1, 16])  # a skipped token's NaN is not met; slot 16 is past the cache
    assert s == kq.KQ_ERR_RANGE and torch.all(vr[2:] == 0) and torch.all(vr[:2] == 1)
    kr = torch.empty(2, 1, 64, device="cuda")
    kq.kq_kv_read(kq.KVCache(1, 16, 1, 64), ints([16, -1]), kr, kr.clone())
    assert status(kq) == kq.KQ_ERR_RANGE and torch.all(kr == 0)


# ---- attention ------------------------------------------------------------------------


class Step:
    """A step's cache (codes and scales kept on the host), queries, lengths and table.  Slots past a request's length, and
    pages no request has, hold NaN scales: nothing may come of them."""

    def __init__(self, kq, rng, kv_len, new, hq, hk, d, page, dt, gap=0, sharp=1.0, spare=2, far=0):
        kv_len, new = np.asarray(kv_len), np.asarray(new)
        self.kq, self.dt, self.page, self.kv_len, self.new, self.hq = kq, dt, page, kv_len, new, hq
        need = -(-kv_len // page)
        pages = int(need.sum()) + spare
        self.kc, self.vc = (rng.integers(0, 16, (pages, hk, page, d)).astype(np.uint8) for _ in range(2))
        self.ks = (rng.uniform(0.05, 0.4, (pages, hk, page, d // 32)) * rng.choice([-1, 1], (pages, hk, page, d // 32))).astype(np.float16)
        self.vs = (rng.uniform(0.01, 0.4, (pages, hk, page, d // 32)) * rng.choice([-1, 1], (pages, hk, page, d // 32))).astype(np.float16)
        perm = rng.permutation(pages)
        self.table = np.full((len(kv_len), max(1, int(need.max())) + 1), -1)
        dirty = np.ones((pages, page), bool)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = perm[at: at + n]
            for j in range(int(kv_len[r])):
                dirty[self.table[r, j // page], j % page] = False
            at += n
        for s in (self.ks, self.vs):
            s.transpose(0, 2, 1, 3)[dirty] = np.nan
        data = dev(ref.pack(self.kc, self.ks, self.vc, self.vs))
        if far:  # the same pages at the end of a larger pool
            pool = torch.zeros(far + pages, hk, data.shape[2], dtype=torch.uint8, device="cuda")
            pool[far:] = data
            data = pool
        self.far = far
        self.cache = kq.KVCache(data.shape[0], page, hk, d, data=data)
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        t = int(self.q_start[-1])
        x = dev(rng.standard_normal((t, hq, d + gap)).astype(np.float32) * sharp, TYPES[dt])
        self.q = x[..., :d]
        self.scale = d ** -0.5

    def run(self, window=0, max_new=None, out=None, stream=None, table=None):
        kq, q = self.kq, self.q
        if out is None:
            out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        m = max_new or max(1, int(self.new.max()))
        n = kq.kq_attn_workspace_bytes(self.cache, self.hq, len(self.new), q.shape[0], m)
        ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        t = self.table if table is None else table
        kq.kq_attn_paged(self.cache, q, ints(self.q_start), ints(self.kv_len), ints(t + (t >= 0) * self.far), out, self.scale,
                         m, window=window, ws=ws, stream=stream)
        return out

    def want(self, window=0):
        return ref.attention(f64(self.q), np.nan_to_num(ref.values(self.kc, self.ks)),
                             np.nan_to_num(ref.values(self.vc, self.vs)), self.q_start, self.kv_len, self.table, self.page,
                             self.scale, window)

    def check(self, window=0, **kw):
        out = self.run(window, **kw)
        assert status(self.kq) == self.kq.KQ_OK
        near(f64(out), self.want(window), self.dt)
        return out


def near(got, want, dt):
    norm = np.linalg.norm(want, axis=-1)
    err = np.linalg.norm(got - want, axis=-1)
    assert np.all(np.isfinite(got))
    assert np.all(err <= ATTN_TOL[dt] * norm), (err / np.maximum(norm, 1e-30)).max()


HEADS = [(4, 1, 128), (32, 8, 128), (6, 1, 256), (14, 2, 64), (3, 3, 128), (16, 1, 64), (9, 1, 128), (5, 5, 256)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_attention_decode(kq, dt, hq, hk, d):
    rng = np.random.default_rng(hq + d)
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 0, 100, 257, 700]
    page = {1: 16, 2: 48, 3: 32}.get(hk, 64)
    s = Step(kq, rng, lens, [1] * len(lens), hq, hk, d, page, dt, gap=16 if hk == 1 else 0)
    s.check()
    s.check(window=1)
    s.check(window=40)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d", HEADS)
def test_attention_several_new_tokens(kq, dt, hq, hk, d):
    rng = np.random.default_rng(3 * hq + d)
    new = np.array([1, 4, 0, 3, 7, 2, 5])
    lens = np.array([40, 4, 9, 200, 130, 1, 0])  # the last two bring more tokens than their length: queries that see nothing
    s = Step(kq, rng, lens, new, hq, hk, d, 32, dt)
    out = s.check()
    assert torch.all(out[int(s.q_start[5])] == 0)
    s.check(window=3)
    s.check(max_new=50)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,page", [(8, 2, 128, 32), (6, 1, 256, 48), (14, 2, 64, 16), (2, 2, 128, 64)])
def test_attention_prompts(kq, dt, hq, hk, d, page):
    rng = np.random.default_rng(5 * hq + d)
    new = np.array([130, 1, 257, 64, 33])
    lens = np.array([130, 300, 400, 65, 20])
    s = Step(kq, rng, lens, new, hq, hk, d, page, dt)
    s.check()
    s.check(window=50)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attention_long_context_and_sharp_scores(kq, dt):
    rng = np.random.default_rng(11)
    Step(kq, rng, [9000, 5, 3001], [1, 1, 1], 4, 1, 128, 32, dt, sharp=6.0).check()
    Step(kq, rng, [6000], [2], 8, 2, 128, 16, dt, sharp=0.01).check()


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_attention_value_scales_of_all_sizes(kq, dt):
    """Value scales from the smallest fp16 normals to 2^11 in one context: each output row still meets its tolerance."""
    rng = np.random.default_rng(12)
    for low, high in ((-14, -12), (9, 11), (-10, 4)):
        s = Step(kq, rng, [500, 40], [1, 3], 4, 2, 128, 32, dt)
        f = np.exp2(rng.integers(low, high + 1, s.vs.shape)).astype(np.float16)
        s.vs = np.where(np.isnan(s.vs), s.vs, np.sign(s.vs) * f)
        s.cache.data.copy_(dev(ref.pack(s.kc, s.ks, s.vc, s.vs)))
        out = s.run()
        assert status(kq) == kq.KQ_OK
        near(f64(out), s.want(), dt)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d,page", [(8, 2, 128, 32), (7, 1, 64, 16), (6, 1, 256, 32)])
def test_attention_long_prompt_in_many_parts(kq, dt, hq, hk, d, page):
    """One prompt on a long context: its few row blocks are cut between all CTAs, some into more than two parts."""
    rng = np.random.default_rng(21 + d)
    s = Step(kq, rng, [2900], [150], hq, hk, d, page, dt)
    s.check()
    s.check(window=700)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (6, 1, 256), (7, 1, 64), (41, 1, 128), (65, 1, 64), (48, 1, 256)])
def test_attention_on_both_sides_of_the_change_of_kernels(kq, dt, hq, hk, d):
    """Requests of a few more and a few less than 40 or 64 query rows a key head, in one call and each alone; one key head
    for so many query heads that a single token has them."""
    rng = np.random.default_rng(23 + hq + d)
    new = np.array([6, 7, 9, 10, 11, 1])
    lens = np.array([6, 90, 300, 33, 1000, 513])
    s = Step(kq, rng, lens, new, hq, hk, d, 32, dt)
    s.check()
    s.check(window=8)
    for n, length in ((1, 1), (1, 700), (10, 200), (11, 200)):
        Step(kq, rng, [length], [n], hq, hk, d, 16, dt).check()


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_attention_mixed_batch(kq, dt):
    """Single tokens, drafts, prompts and idle requests in one call; more of them than a CTA has threads."""
    rng = np.random.default_rng(22)
    new = rng.choice([0, 1, 1, 1, 3, 40], 700)
    new[5], new[300] = 200, 90
    lens = new + rng.integers(0, 60, 700)
    lens[7] = new[7] + 900
    s = Step(kq, rng, lens, new, 4, 2, 64, 16, dt)
    s.check()
    s.check(window=20)


@pytest.mark.parametrize("sign", [-1.0, 0.0])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attention_of_negative_and_zero_scale(kq, dt, sign):
    rng = np.random.default_rng(23)
    s = Step(kq, rng, [300, 90, 70], [70, 1, 3], 8, 2, 128, 32, dt)
    s.scale *= sign
    s.check()


def test_attention_prompt_values_beyond_fp16(kq):
    """Key and value scales above 8188 (8 steps leave fp16) in some tiles of a bf16 prompt."""
    rng = np.random.default_rng(24)
    s = Step(kq, rng, [400, 130], [90, 64], 8, 2, 128, 32, "bf16")
    big = rng.random(s.vs.shape) < 0.02
    s.vs = np.where(big & ~np.isnan(s.vs), np.float16(20000), s.vs)
    s.ks = np.where(big & ~np.isnan(s.ks), np.float16(9000), s.ks)
    s.q.mul_(1e-4)
    s.cache.data.copy_(dev(ref.pack(s.kc, s.ks, s.vc, s.vs)))
    out = s.run()
    assert status(kq) == kq.KQ_OK
    near(f64(out), s.want(), "bf16")


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attention_of_poisoned_values_stays_behind_the_mask(kq, dt):
    """A visible key whose value scale is NaN: the rows that see it get NaN in its group of 32 dimensions, rows that the
    causal mask or the window keeps from it nothing."""
    rng = np.random.default_rng(25)
    s = Step(kq, rng, [200, 40], [100, 4], 8, 2, 128, 32, dt)
    want = s.want(window=60)
    for r, j, g in ((0, 150, 1), (1, 37, 3)):
        s.vs[s.table[r, j // 32], 0, j % 32, g] = np.nan
    s.cache.data.copy_(dev(ref.pack(s.kc, s.ks, s.vc, s.vs)))
    got = f64(s.run(window=60))
    assert status(kq) == kq.KQ_OK
    bad = np.zeros(got.shape, bool)
    pos0 = np.concatenate([np.arange(100, 200), np.arange(36, 40)])
    for r, j, g in ((0, 150, 1), (1, 37, 3)):
        rows = (np.arange(104) >= 100) == (r == 1)
        rows &= (pos0 >= j) & (pos0 < j + 60)
        bad[np.ix_(rows, np.arange(4), np.arange(32 * g, 32 * g + 32))] = True
    assert np.array_equal(np.isnan(got), bad)
    norm = np.linalg.norm(want, axis=-1, keepdims=True)
    assert np.all(np.abs(got - want)[~bad] <= (ATTN_TOL[dt] * norm * np.ones_like(want))[~bad])


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_attention_prompt_hides_bad_pages_and_freed_ones(kq, dt):
    """Pages below a sliding window may be gone (no status, no effect); a missing page inside it hides its keys."""
    rng = np.random.default_rng(26)
    s = Step(kq, rng, [400], [80], 4, 2, 128, 32, dt)
    table = s.table.copy()
    table[0, :6] = -1  # keys 0..191; the window's first is 400 - 80 - 99 = 221
    near(f64(s.run(window=100, table=table)), s.want(window=100), dt)
    assert status(kq) == kq.KQ_OK
    table[0, 9] = s.cache.pages + 3  # keys 288..319
    got = f64(s.run(table=np.where(s.table < 0, -1, np.where(np.arange(s.table.shape[1]) == 9, table, s.table))))
    assert status(kq) == kq.KQ_ERR_RANGE
    k, v = (np.nan_to_num(ref.values(c, x)) for c, x in ((s.kc, s.ks), (s.vc, s.vs)))
    for t in (0, 41, 79):
        keys = np.array([j for j in range(320 + t + 1) if not 288 <= j < 320])
        kk, vv = (x[s.table[0, keys // 32], :, keys % 32] for x in (k, v))
        for h in range(4):
            e = s.scale * kk[:, h // 2] @ f64(s.q)[t, h]
            p = np.exp(e - e.max())
            near(got[t, h], (p / p.sum()) @ vv[:, h // 2], dt)


def test_attention_leaves_out_malformed_requests(kq):
    """q_start that decreases or passes the tokens, and more new tokens than max_new: a status, the other requests'
    rows as they should be."""
    rng = np.random.default_rng(27)
    s = Step(kq, rng, [100, 60, 90], [60, 4, 1], 8, 2, 128, 32, "f16")
    want, good = s.want(), s.q_start
    for q_start in ([0, 60, 64, 900], [0, 60, 20, 65], [-4, 60, 64, 65]):
        s.q_start = np.array(q_start)
        out = f64(s.run(max_new=60))
        assert status(kq) == kq.KQ_ERR_RANGE
        claims = np.zeros(65, int)  # well-formed requests that a row belongs to
        for lo, hi in zip(q_start, q_start[1:]):
            if 0 <= lo <= hi <= 65:
                claims[lo:hi] += 1
        for r in range(3):
            lo, hi = q_start[r], q_start[r + 1]
            if (lo, hi) == (good[r], good[r + 1]):
                rows = lo + np.flatnonzero(claims[lo:hi] == 1)
                near(out[rows], want[rows], "f16")
    s.q_start = good
    out = f64(s.run(max_new=10))
    assert status(kq) == kq.KQ_ERR_RANGE
    assert np.all(out[:60] == 7)
    near(out[60:], want[60:], "f16")


def test_attention_offsets_past_32_bits(kq):
    rng = np.random.default_rng(13)
    far = (5 << 30) // (2 * ref.block_bytes(32, 128))
    s = Step(kq, rng, [70, 300], [1, 2], 4, 2, 128, 32, "f16", far=far)
    assert s.cache.data.numel() > (1 << 32)
    s.check()
    slot = int(s.table[1, 2] + far) * 32 + 5
    kr, vr = (torch.empty(1, 2, 128, device="cuda") for _ in range(2))
    kq.kq_kv_read(s.cache, ints([slot]), kr, vr)
    assert np.array_equal(f64(kr)[0], ref.values(s.kc, s.ks)[s.table[1, 2], :, 5])


def test_attention_same_bits_again_and_on_another_stream(kq):
    rng = np.random.default_rng(14)
    s = Step(kq, rng, [900, 77, 3], [1, 1, 1], 8, 2, 128, 32, "f32")
    a = s.check()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        b = s.check(stream=stream)
    assert torch.equal(a, b)


def test_attention_of_non_finite_queries_stays_in_its_row(kq):
    rng = np.random.default_rng(15)
    s = Step(kq, rng, [300, 40], [1, 3], 8, 2, 128, 32, "f32")
    a = s.check()
    s.q[0, 3, 5], s.q[2, 0, 0] = float("nan"), float("inf")
    b = s.run()
    assert status(kq) == kq.KQ_OK
    bad = torch.zeros(a.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 3] = bad[2, 0] = True
    assert torch.equal(a[~bad], b[~bad])
    assert not torch.any(torch.isfinite(b[bad]))


def test_attention_hides_bad_pages_and_lengths(kq):
    """A page id outside the pool hides its keys, a length past the table's row is cut: a status, no bad access."""
    rng = np.random.default_rng(16)
    s = Step(kq, rng, [100, 64], [1, 1], 4, 2, 128, 32, "f32")
    table = s.table.copy()
    table[0, 1] = s.cache.pages + 5
    table[1, 0] = -3
    out = s.run(table=table)
    assert status(kq) == kq.KQ_ERR_RANGE
    k, v = (np.nan_to_num(ref.values(c, x)) for c, x in ((s.kc, s.ks), (s.vc, s.vs)))
    for r, keys in ((0, [*range(32), *range(64, 100)]), (1, range(32, 64))):
        keys = np.array(list(keys))
        kk, vv = (x[s.table[r, keys // 32], :, keys % 32] for x in (k, v))  # [keys, heads, d]
        for h in range(4):
            e = s.scale * kk[:, h // 2] @ f64(s.q)[r, h]
            p = np.exp(e - e.max())
            near(f64(out)[r, h], (p / p.sum()) @ vv[:, h // 2], "f32")
    s.kv_len = np.array([100, 1000])
    s.run()
    assert status(kq) == kq.KQ_ERR_RANGE


def test_attention_leaves_other_rows_alone(kq):
    """Rows past q_start[requests], and the gaps of a strided output, keep their contents."""
    rng = np.random.default_rng(17)
    s = Step(kq, rng, [50, 20], [2, 1], 4, 2, 64, 16, "f16")
    big = torch.full((3, 4, 96), 5.0, dtype=torch.float16, device="cuda")
    s.check(out=big[..., :64])
    assert torch.all(big[..., 64:] == 5)
    q = s.q
    s.q = torch.cat([q, q])  # capacity of six tokens, three used
    out = s.run()
    assert status(kq) == kq.KQ_OK
    assert torch.all(out[3:] == 7)
    s.q = q
    near(f64(out[:3]), s.want(), "f16")


def test_whole_step(kq):
    """slot map -> append -> attention, prompt then single tokens, against FP64 attention over what was written."""
    rng = np.random.default_rng(18)
    hq, hk, d, page, pages = 8, 2, 128, 16, 40
    cache = kq.KVCache(pages, page, hk, d)
    table = ints(np.zeros((3, 8)))
    free = rng.permutation(pages)
    rope = dev(kq.kq_rope_table_host(200, d, 1e4))
    p = kq.QKNorm(hq, hk, d, d, None, None, rope)
    cached, used_all = np.zeros(3, int), 0
    for new in ([20, 1, 47], [1, 1, 1], [1, 0, 1], [3, 16, 2]):
        t = sum(new)
        q, k, v = _qk_inputs(rng, t, hq, hk, d, "f32")
        o = [ints(np.zeros(n)) for n in (4, 3, t, t, 1)]
        kq.kq_slot_map(ints(cached), ints(new), page, ints(free[used_all:]), table, *o)
        q_start, kv_len, positions, slots, used = o
        qo, out = torch.empty(t, hq, d, device="cuda"), torch.empty(t, hq, d, device="cuda")
        kq.kq_kv_append(p, cache, q, k, v, positions, slots, qo)
        n = kq.kq_attn_workspace_bytes(cache, hq, 3, t, max(new))
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        kq.kq_attn_paged(cache, qo, q_start, kv_len, table, out, d ** -0.5, max(new), ws=ws)
        assert status(kq) == kq.KQ_OK
        cached += new
        used_all += int(used.item())
        kc, ks, vc, vs = ref.unpack(cache.data.cpu().numpy(), page, d)
        want = ref.attention(f64(qo), ref.values(kc, ks), ref.values(vc, vs), q_start.cpu().numpy(), cached,
                             table.cpu().numpy(), page, d ** -0.5, 0)
        near(f64(out), want, "f32")


def test_example_decode_layer(kq):
    """The example's layer: prompt and steps through slot map, projections, append and attention, fp32 throughout."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layer.py")
    spec = importlib.util.spec_from_file_location("decode_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.main(requests=3, prompt=21, steps=3) < ATTN_TOL["f32"]
