"""CPU checks of views that may not overlap: what the library refuses for the norm and the delta rule, against bytes marked one
by one, and that it refuses nothing that lies apart."""
import ctypes
import random

import pytest

torch = pytest.importorskip("torch")

from test_delta_host import FAKE, _struct, kq  # noqa: E402,F401


def _bytes(view, tokens, heads, dim, size):
    at, ts, hs = view
    return {at + (t * ts + h * hs + i) * size for t in range(tokens) for h in range(heads) for i in range(0, dim, 16 // size)}


def _norm(kq, dtype, tokens, heads, dim, x, out, residual=None, gate=None):
    """Whether kq_rms_norm refuses the views for their overlaps.  A call that gets past these is refused for its planes."""
    v = lambda a: None if a is None else ctypes.byref(kq.kq_heads(*a))  # noqa: E731
    p = _struct(kq.kq_rms, dict(heads=heads, dim=dim, eps=1e-6, reserved=0, weight=None), {})
    q8 = ctypes.byref(kq.kq_qmat(kq.KQ_Q8_0, 0, tokens * heads + 1, dim, FAKE, FAKE, None))
    status = kq.lib().kq_rms_norm(p, dtype, v(x), v(residual), v(gate), tokens, v(out), q8, None)
    assert status in (kq.KQ_ERR_INVALID_ARG, kq.KQ_ERR_SHAPE)
    return status == kq.KQ_ERR_INVALID_ARG and "overlaps" in kq.lib().kq_last_error().decode()


def test_norm_refuses_views_that_cross(kq):  # noqa: F811
    d, n, whole, far = 128, 6, (FAKE, 512, 128), (FAKE + (1 << 24), 512, 128)
    for x, out in ((whole, (FAKE + 16, 512, 128)), (whole, (FAKE + 1024, 512, 128)), ((FAKE + 1024, 512, 128), whole),
                   ((FAKE, 0, 128), whole), ((FAKE, 0, 0), (FAKE + 5 * 1024, 512, 128)), (whole, (FAKE + 6 * 1024, 512, 128)),
                   ((FAKE, 1024, 256), (FAKE + 256, 1024, 256)), ((FAKE, 1024, 256), (FAKE + 240, 1024, 256)),
                   ((FAKE, 1024, 128), (FAKE + 1024, 1024, 128)), ((FAKE, 128, 6 * 128), (FAKE + 128, 128, 6 * 128)),
                   (far, whole)):
        share = bool(_bytes(x, n, 4, d, 2) & _bytes(out, n, 4, d, 2))
        assert _norm(kq, kq.KQ_F16, n, 4, d, x, out) == share, (x, out)
        assert _norm(kq, kq.KQ_F16, n, 4, d, x, (far[0] + (1 << 24), 512, 128), residual=out) == share, (x, out)
        assert _norm(kq, kq.KQ_F16, n, 4, d, far, out, gate=x) == share, (x, out)
    # one view for two
    for views in (dict(x=whole, out=whole), dict(x=far, out=whole, residual=whole), dict(x=far, out=whole, gate=whole),
                  dict(x=whole, out=far, residual=whole), dict(x=whole, out=whole, residual=whole)):
        assert not _norm(kq, kq.KQ_F16, n, 4, d, **views), views
    # the gate is read when the residual is written
    assert _norm(kq, kq.KQ_F16, n, 4, d, far, None, whole, whole)


def _gdn(kq, dtype, tokens, hk, hv, q, k, v, out, d=64, **over):
    w = lambda a: ctypes.byref(kq.kq_heads(*a))  # noqa: E731
    p = _struct(kq.kq_gdn_rule, dict(k_heads=hk, v_heads=hv, head_dim=d, unit=1, gates=1, eps=1e-6, scale=0.1, reserved=0, a_log=FAKE,
                                     dt_bias=FAKE), over)
    status = kq.lib().kq_gdn(p, dtype, w(q), w(k), w(v), FAKE, hv, FAKE, hv, FAKE, FAKE, FAKE, 2, tokens, 8, FAKE, 4, w(out), None, 0, None)
    text = kq.lib().kq_last_error().decode()
    return status == kq.KQ_ERR_INVALID_ARG and "overlaps" in text, status, text


def test_gdn_refuses_outputs_over_its_inputs(kq):  # noqa: F811
    apart = [(FAKE + (i << 24), 512, 64) for i in range(1, 5)]
    q, k, v, out = apart
    for i, dtype in enumerate((kq.KQ_F16, kq.KQ_F32, kq.KQ_BF16)):
        assert _gdn(kq, dtype, 9, 4, 4, q, k, v, q)[0]
        assert _gdn(kq, dtype, 9, 4, 4, q, k, v, k)[0]
        assert _gdn(kq, dtype, 9, 2, 4, q, k, v, (q[0] + 128 * (1 + (dtype == kq.KQ_F32)), 512, 64))[0]
        assert _gdn(kq, dtype, 9, 4, 4, q, k, v, (v[0] + 16, 512, 64))[0]  # the values' rows, but not their view
        assert _gdn(kq, dtype, 9, 4, 4, q, k, v, (v[0] + 512 * 2 * (1 + (dtype == kq.KQ_F32)), 512, 64))[0]


def test_overlaps_are_found_where_bytes_are_shared_and_nowhere_else(kq):  # noqa: F811
    """Random views of one buffer whose tokens are one stride apart, with heads that adjoin, lie apart or come first."""
    r = random.Random(5)
    found = 0
    for _ in range(4000):
        heads, dim, tokens = r.choice([1, 2, 3, 4]), 64, r.choice([1, 2, 5])
        head = r.choice([64, 72, 128])
        stride = (heads - 1) * head + 64 + 8 * r.choice([0, 1, 8, 40])
        x = (FAKE + 16 * r.randrange(200), stride, head)
        out = (FAKE + 16 * r.randrange(200), stride, r.choice([64, head]))
        if r.random() < 0.2:
            x, out = [(v[0], 64, 64 * tokens + 8) for v in (x, out)]
        elif r.random() < 0.3:
            x = (x[0], r.choice([0, stride]), r.choice([0, head]))
        same = x[0] == out[0] and (tokens == 1 or x[1] == out[1]) and (heads == 1 or x[2] == out[2])
        share = bool(_bytes(x, tokens, heads, dim, 2) & _bytes(out, tokens, heads, dim, 2))
        assert _norm(kq, kq.KQ_F16, tokens, heads, dim, x, out) == (share and not same), (tokens, heads, x, out)
        found += share and not same
    assert 1000 < found < 3000
