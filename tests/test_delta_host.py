"""CPU checks of the delta layers' operators, the norm and sampling: what the library and the binding refuse, decided
on the host before any CUDA call, and sizes of workspaces."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kq():
    import __graft_entry__

    __graft_entry__.build()
    import quantized_weight_streaming_gb300 as kq

    return kq


FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below is refused on the host
NAN, INF = float("nan"), float("inf")


def _view(kq, data=FAKE, token=8192, head=128):
    return ctypes.byref(kq.kq_heads(data, token, head))


def _struct(kind, base, over):
    base = dict(base, **over)
    return ctypes.byref(kind(*[base[n] for n, _ in kind._fields_]))


def test_norm_refusals(kq):
    q8 = kq.kq_qmat(kq.KQ_Q8_0, 0, 3 * 4, 128, FAKE, FAKE, None)

    def call(dtype=kq.KQ_F16, x="v", residual=None, gate=None, tokens=3, out="v", out_q8=None, **over):
        p = _struct(kq.kq_rms, dict(heads=4, dim=128, eps=1e-6, reserved=0, weight=FAKE), over)
        w = lambda t: _view(kq) if isinstance(t, str) else t  # noqa: E731
        return kq.lib().kq_rms_norm(p, dtype, w(x), w(residual), w(gate), tokens, w(out), out_q8, None)

    assert kq.lib().kq_rms_norm(None, 1, _view(kq), None, None, 3, _view(kq), None, None) == kq.KQ_ERR_INVALID_ARG
    assert call(dtype=5) == kq.KQ_ERR_INVALID_ARG
    for over in (dict(reserved=1), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(out=None), dict(x=None)):
        assert call(**over) == kq.KQ_ERR_INVALID_ARG, over
    for over in (dict(heads=0), dict(heads=5000), dict(dim=0), dict(dim=12), dict(dim=32776), dict(tokens=-1),
                 dict(tokens=1 << 30), dict(out=_view(kq, token=120)), dict(out=_view(kq, head=64)), dict(out=_view(kq, token=0)),
                 dict(residual=_view(kq, token=0)), dict(x=_view(kq, token=-8)),
                 dict(out=_view(kq, token=128, head=128)), dict(out=_view(kq, token=504, head=128)), dict(out=_view(kq, token=128, head=256)),
                 dict(residual=_view(kq, token=256, head=256))):
        assert call(**over) == kq.KQ_ERR_SHAPE, over
    for over in (dict(weight=FAKE + 4), dict(x=_view(kq, FAKE + 2)), dict(out=_view(kq, token=8196)), dict(gate=_view(kq, head=132)),
                 dict(residual=_view(kq, FAKE + 8))):
        assert call(**over) == kq.KQ_ERR_ALIGNMENT, over
    for n, k in ((11, 128), (12, 64)):
        q8.n, q8.k = n, k
        assert call(out_q8=ctypes.byref(q8)) == kq.KQ_ERR_SHAPE
    q8.n, q8.k, q8.fmt = 12, 128, kq.KQ_SCALE4
    assert call(out_q8=ctypes.byref(q8)) != kq.KQ_OK
    assert call(tokens=0) == kq.KQ_OK


def test_conv_refusals(kq):
    def call(dtype=kq.KQ_F16, x="v", out=None, q_start=FAKE, kv_len=FAKE, slot=FAKE, requests=2, tokens=3, state=FAKE, slots=4, **over):
        p = _struct(kq.kq_conv, dict(channels=64, width=4, silu=1, reserved=0, weight=FAKE, bias=FAKE), over)
        w = _view(kq) if isinstance(x, str) else x
        return kq.lib().kq_causal_conv(p, dtype, w, q_start, kv_len, slot, requests, tokens, state, slots,
                                       out or _view(kq, FAKE + (1 << 24)), None)

    for over in (dict(dtype=-1), dict(weight=None), dict(silu=2), dict(reserved=3), dict(q_start=None), dict(slot=None),
                 dict(state=None), dict(x=None), dict(out=_view(kq)), dict(out=_view(kq, FAKE + 64)),
                 dict(out=_view(kq, FAKE + 8192 * 2)), dict(out=_view(kq, FAKE + 16, token=4096))):
        assert call(**over) == kq.KQ_ERR_INVALID_ARG, over
    for over in (dict(channels=0), dict(channels=12), dict(channels=(1 << 20) + 8), dict(width=1), dict(width=5), dict(requests=0),
                 dict(tokens=-1), dict(tokens=(1 << 31) - 1), dict(slots=0), dict(out=_view(kq, FAKE + (1 << 24), token=56))):
        assert call(**over) == kq.KQ_ERR_SHAPE, over
    for over in (dict(weight=FAKE + 4), dict(bias=FAKE + 4), dict(q_start=FAKE + 4), dict(kv_len=FAKE + 4), dict(slot=FAKE + 8),
                 dict(state=FAKE + 2), dict(x=_view(kq, FAKE + 2))):
        assert call(**over) == kq.KQ_ERR_ALIGNMENT, over
    assert call(tokens=0) == kq.KQ_OK


def test_gdn_refusals_and_workspace(kq):
    base = dict(k_heads=2, v_heads=4, head_dim=128, unit=1, gates=1, eps=1e-6, scale=0.1, reserved=0, a_log=FAKE, dt_bias=FAKE)

    def call(dtype=kq.KQ_F32, q="v", k="v", v="v", a=FAKE, a_stride=4, b=FAKE, b_stride=4, q_start=FAKE, kv_len=FAKE, slot=FAKE,
             requests=2, tokens=300, max_new=200, state=FAKE, slots=4, out="v", ws=FAKE, ws_bytes=1 << 40, **over):
        w = lambda t: _view(kq) if isinstance(t, str) else t  # noqa: E731
        return kq.lib().kq_gdn(_struct(kq.kq_gdn_rule, base, over), dtype, w(q), w(k), w(v), a, a_stride, b, b_stride, q_start, kv_len,
                               slot, requests, tokens, max_new, state, slots, w(out), ws, ws_bytes, None)

    for over in (dict(dtype=3), dict(unit=2), dict(gates=-1), dict(gates=0), dict(reserved=1), dict(a_log=None), dict(dt_bias=None),
                 dict(eps=-1.0), dict(eps=INF), dict(scale=NAN), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(a=None),
                 dict(b=None), dict(q_start=None), dict(slot=None), dict(state=None)):
        assert call(**over) == kq.KQ_ERR_INVALID_ARG, over
    for over in (dict(head_dim=96), dict(head_dim=256), dict(k_heads=0), dict(k_heads=3), dict(v_heads=0), dict(v_heads=8192, k_heads=1),
                 dict(requests=0), dict(requests=1 << 30), dict(tokens=-1), dict(max_new=-1), dict(slots=0), dict(a_stride=-1),
                 dict(b_stride=-4), dict(out=_view(kq, token=64)), dict(out=_view(kq, head=0)), dict(out=_view(kq, token=256)),
                 dict(v_heads=2, tokens=(1 << 31) - 1)):
        assert call(**over) == kq.KQ_ERR_SHAPE, over
    for over in (dict(a=FAKE + 2), dict(b=FAKE + 1), dict(a_log=FAKE + 4), dict(dt_bias=FAKE + 4), dict(state=FAKE + 4),
                 dict(q_start=FAKE + 4), dict(kv_len=FAKE + 4), dict(slot=FAKE + 4), dict(q=_view(kq, FAKE + 4))):
        assert call(**over) == kq.KQ_ERR_ALIGNMENT, over
    assert call(tokens=0) == kq.KQ_OK

    def need(dtype=kq.KQ_F16, requests=2, tokens=300, max_new=200, **over):
        return kq.lib().kq_gdn_workspace_bytes(_struct(kq.kq_gdn_rule, base, over), dtype, requests, tokens, max_new)

    assert 0 < need() < need(tokens=3000) and need() < need(dtype=kq.KQ_F32)  # fp32 keys and queries have two parts
    # nothing is needed where every run goes token by token
    for over in (dict(head_dim=64), dict(max_new=1), dict(max_new=8), dict(unit=0), dict(gates=0, a_log=None, dt_bias=None)):
        assert need(**over) == 0, over
    for over in (dict(head_dim=96), dict(dtype=9), dict(requests=0), dict(tokens=-1), dict(reserved=1)):
        assert need(**over) == 0, over
    assert call(dtype=kq.KQ_F16, ws=None) == kq.KQ_ERR_WORKSPACE
    assert call(dtype=kq.KQ_F16, ws_bytes=need() - 1) == kq.KQ_ERR_WORKSPACE
    assert call(dtype=kq.KQ_F16, ws=FAKE + 8) == kq.KQ_ERR_ALIGNMENT


def test_sample_refusals(kq):
    names = ("dtype", "logits", "stride", "rows", "vocab", "temperature", "top_k", "top_p", "min_p", "u", "token", "prob")

    def call(**over):
        a = dict(dtype=kq.KQ_F16, logits=FAKE, stride=1000, rows=2, vocab=999, temperature=FAKE, top_k=FAKE, top_p=FAKE, min_p=FAKE,
                 u=FAKE, token=FAKE, prob=FAKE)
        a.update(over)
        return kq.lib().kq_sample(*[a[n] for n in names], None)

    for over in (dict(dtype=4), dict(logits=None), dict(u=None), dict(token=None)):
        assert call(**over) == kq.KQ_ERR_INVALID_ARG, over
    for over in (dict(vocab=0), dict(vocab=393217), dict(rows=-1), dict(rows=1 << 31), dict(stride=998), dict(stride=-1)):
        assert call(**over) == kq.KQ_ERR_SHAPE, over
    for over in (dict(logits=FAKE + 1), dict(dtype=kq.KQ_F32, logits=FAKE + 2), dict(u=FAKE + 2), dict(token=FAKE + 1), dict(prob=FAKE + 2),
                 dict(top_k=FAKE + 1), dict(top_p=FAKE + 2), dict(min_p=FAKE + 1), dict(temperature=FAKE + 2)):
        assert call(**over) == kq.KQ_ERR_ALIGNMENT, over
    assert call(rows=0) == kq.KQ_OK


def test_binding_refuses_wrong_tensors(kq):
    """Tensors of another type, shape or layout than the kernels read; the calls are refused before the library is reached."""
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    refused = lambda f, *a, **k: pytest.raises(kq.KQError, f, *a, **k)  # noqa: E731
    w = torch.ones(128)
    for bad in (w[:64], w.half(), torch.ones(256)[::2]):
        refused(kq.RMSNorm, 1, 128, bad)
    p, x = kq.RMSNorm(2, 128, w), torch.zeros(3, 2, 128)
    for bad in (x.half(), x[:2], x[:, :1], x.transpose(0, 1), torch.zeros(3, 2, 256)[:, :, ::2]):
        refused(kq.kq_rms_norm, p, x, bad, stream=0)
        refused(kq.kq_rms_norm, p, x, x, residual=bad, stream=0)
        refused(kq.kq_rms_norm, p, x, x, gate=bad, stream=0)

    for bad in (torch.ones(16), torch.ones(16, 4).half(), torch.ones(4, 16).T):
        refused(kq.CausalConv, bad)
    refused(kq.CausalConv, torch.ones(16, 4), torch.ones(8))
    c, y, state = kq.CausalConv(torch.ones(16, 4)), torch.zeros(5, 16), torch.zeros(2, 3, 16)
    good = dict(x=y, d_q_start=i(3), d_kv_len=i(2), d_slot=i(2), state=state, out=torch.zeros(5, 16))
    for over in (dict(x=y[:, :8]), dict(x=y.half()), dict(d_q_start=i(2)), dict(d_q_start=i(3).long()), dict(d_kv_len=i(1)),
                 dict(state=state.half()), dict(state=state[:, :2]), dict(state=torch.zeros(2, 16, 3).transpose(1, 2)),
                 dict(out=torch.zeros(4, 16)), dict(out=torch.zeros(5, 16).half()), dict(out=torch.zeros(5, 32)[:, ::2])):
        refused(kq.kq_causal_conv, c, **dict(good, **over), stream=0)

    refused(kq.GatedDelta, 1, 2, 64, torch.ones(3), torch.ones(2))
    refused(kq.GatedDelta, 1, 2, 64, torch.ones(2), torch.ones(2).half())
    r, q, v, g = kq.GatedDelta(1, 2, 64, torch.ones(2), torch.ones(2)), torch.zeros(5, 1, 64), torch.zeros(5, 2, 64), torch.zeros(5, 2)
    good = dict(q=q, k=q, v=v, a=g, b=g, d_q_start=i(3), d_kv_len=i(2), d_slot=i(2), state=torch.zeros(2, 2, 64, 64), out=v, max_new=5)
    for over in (dict(k=q.half()), dict(k=q[:4]), dict(v=q), dict(a=g[:, :1]), dict(a=g[:4]), dict(a=g.half()), dict(b=torch.zeros(2, 5).T),
                 dict(b=torch.zeros(10)), dict(d_q_start=i(2)), dict(d_kv_len=i(1)), dict(state=torch.zeros(2, 2, 64, 64).half()),
                 dict(state=torch.zeros(2, 1, 64, 64)), dict(state=torch.zeros(2, 2, 64, 128)[..., :64]), dict(out=v.half()), dict(out=q)):
        refused(kq.kq_gdn, r, **dict(good, **over), stream=0)

    logits, u, token = torch.zeros(3, 50), torch.zeros(3), i(3)
    for over in (dict(logits=torch.zeros(3, 2, 50)), dict(logits=torch.zeros(50, 3).T), dict(u=u[:2]), dict(u=u.double()), dict(d_token=i(2)),
                 dict(d_token=token.long()), dict(d_prob=u[:1]), dict(temperature=u.half()), dict(top_k=u), dict(top_p=i(3)),
                 dict(min_p=torch.zeros(6)[::2])):
        refused(kq.kq_sample, **dict(dict(logits=logits, u=u, d_token=token), **over), stream=0)
