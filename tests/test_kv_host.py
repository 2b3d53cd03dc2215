"""CPU checks of the attention-step operators: sizes, the rotation table, and
refusals, all decided on the host before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest

import kv_reference as ref


@pytest.fixture(scope="module")
def kq():
    import __graft_entry__

    __graft_entry__.build()
    import quantized_weight_streaming_gb300 as kq

    return kq


FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below is refused on the host


def _cache(kq, pages=4, page=32, heads=2, d=128, data=FAKE, reserved=0):
    return kq.kq_kv_cache(data, pages, page, heads, d, reserved)


def _norm(kq, **over):
    f = dict(q_heads=4, kv_heads=2, head_dim=128, rope_dim=64, interleaved=0, norm=1, eps=1e-6, reserved=0, q_weight=FAKE,
             k_weight=FAKE, d_rope=FAKE, rope_positions=10)
    f.update(over)
    return kq.kq_qk_norm(*[f[n] for n, _ in kq.kq_qk_norm._fields_])


def _view(kq, data=FAKE, token=512, head=128):
    return ctypes.byref(kq.kq_heads(data, token, head))


def test_block_bytes(kq):
    for page in (16, 32, 48, 128):
        for d in (64, 128, 256):
            assert kq.kq_kv_block_bytes(page, d) == ref.block_bytes(page, d)
    for page, d in ((0, 128), (8, 128), (24, 128), (-16, 64), (32, 96), (32, 0), (32, 512)):
        assert kq.kq_kv_block_bytes(page, d) == 0
    with pytest.raises(kq.KQError):
        kq.KVCache(1, 24, 1, 128, device="cpu")


@pytest.mark.parametrize("d", [64, 128, 256])
def test_layout_covers_each_byte_once(d):
    key, value, shift, ks, vs = ref.places(d)
    nibbles = np.concatenate([(key * 2 + shift // 4).ravel(), (value * 2 + shift // 4).ravel(),
                              (np.concatenate([ks[:, ::32].ravel(), vs[:, ::32].ravel()])[:, None] * 4 + np.arange(4)).ravel()])
    assert np.array_equal(np.sort(nibbles), np.arange(18 * d * 2))
    rng = np.random.default_rng(d)
    kc, vc = (rng.integers(0, 16, (2, 3, 32, d)).astype(np.uint8) for _ in range(2))
    s, u = (rng.random((2, 3, 32, d // 32)).astype(np.float16) for _ in range(2))
    for a, b in zip(ref.unpack(ref.pack(kc, s, vc, u), 32, d), (kc, s, vc, u)):
        assert np.array_equal(a, b)


def test_rope_table(kq):
    t = kq.kq_rope_table_host(1000, 64, 1e6)
    for p, i in ((0, 0), (1, 0), (999, 0), (999, 31), (517, 7)):
        a = p * 1e6 ** (-2 * i / 64)
        assert t[p, i] == np.float32(math.cos(a)) and t[p, 32 + i] == np.float32(math.sin(a))
    lib = kq.lib()
    out = np.empty(64, np.float32)
    assert lib.kq_rope_table_host(None, 1, 64, 1e4) == kq.KQ_ERR_INVALID_ARG
    assert lib.kq_rope_table_host(out.ctypes.data, 0, 64, 1e4) == kq.KQ_ERR_SHAPE
    assert lib.kq_rope_table_host(out.ctypes.data, 1, 63, 1e4) == kq.KQ_ERR_SHAPE
    assert lib.kq_rope_table_host(out.ctypes.data, 1, 64, 0.0) == kq.KQ_ERR_INVALID_ARG
    assert lib.kq_rope_table_host(out.ctypes.data, 1, 64, float("nan")) == kq.KQ_ERR_INVALID_ARG


def test_slot_map_refusals(kq):
    names = ("cached", "new", "requests", "page", "free", "free_count", "table", "stride", "q_start", "kv_len", "positions",
             "slots", "tokens", "used")

    def call(**over):
        a = dict(cached=FAKE, new=FAKE, requests=4, page=32, free=FAKE, free_count=3, table=FAKE, stride=8, q_start=FAKE,
                 kv_len=FAKE, positions=FAKE, slots=FAKE, tokens=5, used=FAKE)
        a.update(over)
        return kq.lib().kq_slot_map(*[a[n] for n in names], None)

    for n in ("cached", "new", "free", "table", "q_start", "kv_len", "positions", "slots", "used"):
        assert call(**{n: None}) == kq.KQ_ERR_INVALID_ARG, n
        assert call(**{n: FAKE + 4}) == kq.KQ_ERR_ALIGNMENT, n
    for over in (dict(requests=0), dict(stride=0), dict(free_count=-1), dict(tokens=-1), dict(page=0), dict(page=24)):
        assert call(**over) == kq.KQ_ERR_SHAPE, over
    assert kq.lib().kq_last_error()


def test_norm_rope_refusals(kq):
    def call(p=None, dtype=kq.KQ_F16, q=None, k=None, pos=FAKE, tokens=3, qo=None, ko=None):
        v = _view(kq)
        return kq.lib().kq_qk_norm_rope(ctypes.byref(p or _norm(kq)), dtype, q or v, k or v, pos, tokens, qo or v, ko or v,
                                        None)

    assert call(dtype=7) == kq.KQ_ERR_INVALID_ARG
    for over in (dict(reserved=1), dict(norm=2), dict(interleaved=-1), dict(eps=-1.0), dict(eps=float("nan")),
                 dict(norm=0), dict(d_rope=None)):
        assert call(_norm(kq, **over)) == kq.KQ_ERR_INVALID_ARG, over
    assert call(pos=None) == kq.KQ_ERR_INVALID_ARG
    for over in (dict(head_dim=96), dict(q_heads=0), dict(kv_heads=0), dict(rope_dim=24), dict(rope_dim=144),
                 dict(rope_dim=-16), dict(rope_positions=0)):
        assert call(_norm(kq, **over)) == kq.KQ_ERR_SHAPE, over
    assert call(tokens=-1) == kq.KQ_ERR_SHAPE
    for over in (dict(q_weight=FAKE + 4), dict(k_weight=FAKE + 8), dict(d_rope=FAKE + 4)):
        assert call(_norm(kq, **over)) == kq.KQ_ERR_ALIGNMENT, over
    assert call(pos=FAKE + 4) == kq.KQ_ERR_ALIGNMENT
    for n in ("q", "k", "qo", "ko"):
        assert call(**{n: _view(kq, None)}) == kq.KQ_ERR_INVALID_ARG
        assert call(**{n: _view(kq, FAKE + 2)}) == kq.KQ_ERR_ALIGNMENT
        assert call(**{n: _view(kq, token=513)}) == kq.KQ_ERR_ALIGNMENT
        assert call(**{n: _view(kq, head=132)}) == kq.KQ_ERR_ALIGNMENT  # 264 bytes
        assert call(**{n: _view(kq, token=-512)}) == kq.KQ_ERR_SHAPE
    assert call(tokens=0) == kq.KQ_OK  # nothing to do, nothing launched


def test_append_and_read_refusals(kq):
    lib = kq.lib()

    def append(p=None, cache=None, dtype=kq.KQ_F16, q="v", k="v", v="v", pos=FAKE, slots=FAKE, tokens=3, qo="v"):
        w = lambda x: _view(kq) if isinstance(x, str) else x  # noqa: E731
        return lib.kq_kv_append(ctypes.byref(p or _norm(kq)), ctypes.byref(cache or _cache(kq)), dtype, w(q), w(k), w(v),
                                pos, slots, tokens, w(qo), None)

    assert append(cache=_cache(kq, heads=3)) == kq.KQ_ERR_SHAPE
    assert append(cache=_cache(kq, d=64)) == kq.KQ_ERR_SHAPE
    assert append(cache=_cache(kq, page=20)) == kq.KQ_ERR_SHAPE
    assert append(cache=_cache(kq, pages=0)) == kq.KQ_ERR_SHAPE
    assert append(cache=_cache(kq, pages=1 << 27)) == kq.KQ_ERR_SHAPE  # 2^32 slots
    assert append(cache=_cache(kq, data=None)) == kq.KQ_ERR_INVALID_ARG
    assert append(cache=_cache(kq, data=FAKE + 8)) == kq.KQ_ERR_ALIGNMENT
    assert append(cache=_cache(kq, reserved=1)) == kq.KQ_ERR_INVALID_ARG
    assert append(q=None) == kq.KQ_ERR_INVALID_ARG  # q without q_out and the reverse
    assert append(qo=None) == kq.KQ_ERR_INVALID_ARG
    assert append(k=None) == kq.KQ_ERR_INVALID_ARG
    assert append(v=None) == kq.KQ_ERR_INVALID_ARG
    assert append(slots=None) == kq.KQ_ERR_INVALID_ARG
    assert append(slots=FAKE + 4) == kq.KQ_ERR_ALIGNMENT
    assert append(tokens=0) == kq.KQ_OK

    def read(cache=None, slots=FAKE, count=3, dtype=kq.KQ_F32, k=None, v=None):
        return lib.kq_kv_read(ctypes.byref(cache or _cache(kq)), slots, count, dtype, k or _view(kq), v or _view(kq), None)

    assert read(slots=None) == kq.KQ_ERR_INVALID_ARG
    assert read(count=-1) == kq.KQ_ERR_SHAPE
    assert read(dtype=3) == kq.KQ_ERR_INVALID_ARG
    assert read(k=_view(kq, FAKE + 4)) == kq.KQ_ERR_ALIGNMENT
    assert read(count=0) == kq.KQ_OK


def test_attention_refusals(kq):
    lib = kq.lib()

    def call(cache=None, dtype=kq.KQ_F16, q_heads=4, q=None, q_start=FAKE, kv_len=FAKE, table=FAKE, stride=8, requests=2,
             tokens=3, max_new=2, scale=0.1, window=0, out=None, ws=FAKE, ws_bytes=1 << 40):
        return lib.kq_attn_paged(ctypes.byref(cache or _cache(kq)), dtype, q_heads, q or _view(kq), q_start, kv_len, table,
                                 stride, requests, tokens, max_new, scale, window, out or _view(kq), ws, ws_bytes, None)

    assert call(dtype=-1) == kq.KQ_ERR_INVALID_ARG
    for n in ("q_start", "kv_len", "table"):
        assert call(**{n: None}) == kq.KQ_ERR_INVALID_ARG
        assert call(**{n: FAKE + 4}) == kq.KQ_ERR_ALIGNMENT
    for over in (dict(q_heads=3), dict(q_heads=0), dict(requests=0), dict(tokens=-1), dict(max_new=0), dict(stride=0),
                 dict(window=-1), dict(cache=_cache(kq, d=80))):
        assert call(**over) == kq.KQ_ERR_SHAPE, over
    assert call(scale=float("inf")) == kq.KQ_ERR_INVALID_ARG
    assert call(q=_view(kq, None)) == kq.KQ_ERR_INVALID_ARG
    assert call(out=_view(kq, FAKE + 2)) == kq.KQ_ERR_ALIGNMENT
    assert call(ws=FAKE + 4) == kq.KQ_ERR_ALIGNMENT
    c = _cache(kq)
    need = lib.kq_attn_workspace_bytes(ctypes.byref(c), 4, 2, 3, 2)
    if need:
        assert call(ws=None) == kq.KQ_ERR_WORKSPACE
        assert call(ws_bytes=need - 1) == kq.KQ_ERR_WORKSPACE
    assert lib.kq_attn_workspace_bytes(ctypes.byref(c), 3, 2, 3, 2) == 0
    assert call(tokens=0) == kq.KQ_OK


def test_binding_refuses_wrong_tensors(kq):
    import torch

    p = kq.QKNorm(4, 2, 128, eps=1e-6)
    q, k, pos = torch.zeros(3, 4, 128), torch.zeros(3, 2, 128), torch.zeros(3, dtype=torch.int32)
    for bad in (q.half(), q[:, :3], q[:2], q.transpose(1, 2), q.double()):
        with pytest.raises(kq.KQError):
            kq.kq_qk_norm_rope(p, q, k, pos, bad, k, stream=0)
    with pytest.raises(kq.KQError):
        kq.kq_qk_norm_rope(p, q, k, pos.long(), q, k, stream=0)
    with pytest.raises(kq.KQError):
        kq.kq_qk_norm_rope(p, q, k, pos[:2], q, k, stream=0)
    c = kq.KVCache(2, 16, 2, 128, device="cpu")
    with pytest.raises(kq.KQError):
        kq.KVCache(2, 16, 2, 128, data=c.data[:1])
    with pytest.raises(kq.KQError):
        kq.kq_attn_paged(c, q, pos, pos, torch.zeros(2, 4, dtype=torch.int32), q, 1.0, 1, stream=0)
