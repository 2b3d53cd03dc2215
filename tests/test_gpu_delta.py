"""The delta layers' operators, the norm and sampling against plain 64-bit implementations.

Tolerances.  A 16-bit output is rounded once: half a step, eps / 2 of its value.  Beneath that lies fp32 arithmetic, whose
errors are bounded below in the units h = 2^-24 of one fp32 rounding:
 - norm: the sum of n squares in partial sums of 32 and a tree (40 roundings at most, halved by the root), the root and its
   reciprocal (3), three products (3), SiLU by expf (2 ulp), a sum and a division (6): 40 h relative.
 - convolution: at most 5 terms, each with one rounding, on the sum of magnitudes, then SiLU (slope at most 1.1 and 6 h of
   its own): 12 h of the sum of magnitudes.
 - delta rule: a dot product of D terms of random signs errs by about sqrt(D) h / 2 of the norms' product, and a state takes
   such an error in at each token; without decay they add up at random: (16 + 2 sqrt(D n)) h of the norm of states and
   outputs after n tokens, and four times that where the factors are two fp16 parts (22 bits instead of 24).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
H = 2.0 ** -24


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


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _half(dt):
    return 0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2


def _int(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def _ok(kq):
    assert kq.kq_device_status(True) == kq.KQ_OK


# ---- norm --------------------------------------------------------------------------------------


def _norm_close(y, want, dt, tiny=0.0):
    err = (y.cpu().double() - want).abs()
    least = torch.finfo(dt).smallest_normal * _half(dt) * 2 if dt != torch.float32 else 1e-37
    bound = want.abs() * (_half(dt) + 40 * H) * 1.01 + least + tiny
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 8), (3, 1, 264), (5, 1, 1032), (1, 1, 5120), (700, 1, 2560), (2, 1, 8200),
                                              (3, 1, 32768), (17, 5, 64), (33, 3, 128), (9, 48, 128), (4, 2, 248), (1000, 1, 40),
                                              (6487, 3, 248), (15577, 5, 40), (9733, 4, 128), (311, 1, 5128), (305, 1, 16392)])
@pytest.mark.parametrize("residual,gate", [(False, False), (True, False), (False, True), (True, True)])
def test_norm(kq, dt, tokens, heads, dim, residual, gate):
    g, t = _gen(tokens + dim), TYPES[dt]
    make = lambda: torch.randn(tokens, heads, dim, generator=g).to(t)  # noqa: E731
    x, r, z = make(), make() if residual else None, make() if gate else None
    w = torch.rand(dim, generator=g) + 0.5
    want, kept = ref.rms_norm(x, r, z, w, 1e-6)
    out = torch.empty(tokens, heads, dim, dtype=t, device="cuda")
    rc = r.cuda() if residual else None
    kq.kq_rms_norm(kq.RMSNorm(heads, dim, w.cuda()), x.cuda(), out, residual=rc, gate=z.cuda() if gate else None)
    _norm_close(out, want, t)
    if residual:
        assert torch.equal(rc.cpu(), kept)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
def test_norm_strided_views_in_place_and_without_weight(kq, dt):
    t, g = TYPES[dt], _gen(5)
    rows = torch.randn(37, 6 * 128 + 64, generator=g).to(t).cuda()
    x = rows[:, 64:].unflatten(1, (3, 256))[:, :, :128]  # heads with something between them
    z = rows[:, 64:].unflatten(1, (3, 256))[:, :, 128:]
    want, _ = ref.rms_norm(x.cpu(), None, z.cpu(), None, 1e-5)
    before = rows.clone()
    kq.kq_rms_norm(kq.RMSNorm(3, 128, None, eps=1e-5), x, x, gate=z)
    _norm_close(x, want, t)
    assert torch.equal(rows[:, :64], before[:, :64]) and torch.equal(z, before[:, 64:].unflatten(1, (3, 256))[:, :, 128:])
    # the output over the residual: the sum is not kept then
    r = torch.randn(37, 3, 128, generator=g).to(t).cuda()
    want, _ = ref.rms_norm(z.cpu(), r.cpu(), None, None, 1e-5)
    kq.kq_rms_norm(kq.RMSNorm(3, 128, None, eps=1e-5), z, r, residual=r)
    _norm_close(r, want, t)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 32), (3, 4, 64), (70, 1, 2560), (2, 1, 5120), (5, 1, 96), (1, 1, 32768)])
def test_norm_q8(kq, dt, tokens, heads, dim):
    """The planes hold what the library's own quantizer makes of the fp32 norm."""
    g, t = _gen(dim), TYPES[dt]
    x = torch.randn(tokens, heads, dim, generator=g).to(t).cuda()
    x[0, 0, :32] = 0  # a block of zeros
    p = kq.RMSNorm(heads, dim, (torch.rand(dim, generator=g) + 0.5).cuda())
    q8, both, plain = (kq.QMatrix("q8_0", tokens * heads, dim) for _ in range(3))
    for m in (q8, both):
        m.codes.fill_(77)
        m.scales.fill_(77)
    out = torch.empty_like(x)
    kq.kq_rms_norm(p, x, None, out_q8=q8)
    kq.kq_rms_norm(p, x, out, out_q8=both)
    y = torch.empty(tokens, heads, dim, device="cuda")
    kq.kq_rms_norm(p, x.float(), y)
    kq.kq_quantize_q8_0_device(plain, y)
    for m in (q8, both):
        assert torch.equal(m.codes, plain.codes) and torch.equal(m.scales, plain.scales)
    want, _ = ref.rms_norm(x.cpu(), None, None, p.weight.cpu(), 1e-6)
    _norm_close(out, want, t)
    _ok(kq)


def test_norm_q8_ties_and_non_finite(kq):
    # eps = 0 and rows whose root mean square is a power of two: codes at exact halves
    x = torch.zeros(2, 1, 64)
    x[0, 0, :32] = torch.arange(32) * 0.5 + 0.25
    x[0, 0, 0] = 127 * 0.5
    p = kq.RMSNorm(1, 64, None, eps=0.0)
    y, a, b = torch.empty(2, 1, 64, device="cuda"), kq.QMatrix("q8_0", 2, 64), kq.QMatrix("q8_0", 2, 64)
    x[1] = torch.randn(64, generator=_gen(3))
    kq.kq_rms_norm(p, x.cuda(), y, out_q8=a)
    kq.kq_quantize_q8_0_device(b, y)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    _ok(kq)
    # a gate that is not finite spoils its block alone
    z = torch.ones(2, 1, 64)
    z[1, 0, 40] = math.nan
    kq.kq_rms_norm(p, x.cuda(), None, gate=z.cuda(), out_q8=a)
    assert kq.kq_device_status(True) == kq.KQ_ERR_NONFINITE
    s = a.scales.view(torch.float16).view(2, -1)
    assert bool(torch.isnan(s[1, 1])) and not bool(torch.isnan(s[0, :2]).any()) and not bool(torch.isnan(s[1, 0]))
    # a scale beyond fp16
    w = torch.full((64,), 1e8)
    kq.kq_rms_norm(kq.RMSNorm(1, 64, w.cuda()), x.cuda(), None, out_q8=a)
    assert kq.kq_device_status(True) == kq.KQ_ERR_RANGE
    assert bool(torch.isnan(a.scales.view(torch.float16).view(2, -1)[:, :1]).all())


# ---- convolution ---------------------------------------------------------------------------------


def _steps(kind, seed):
    """New tokens, cached tokens (0: the request begins) and slots of a step's requests."""
    r = np.random.default_rng(seed)
    new = {"one": [1], "step": [1] * 37, "short": [1, 2, 3, 4, 5, 0, 7, 2, 1, 3], "long": [1300], "ragged": [700, 1, 0, 0, 333, 64, 65, 2, 128],
           "mid": [63, 64, 65, 9, 130]}[kind]
    cached = r.integers(0, 3, len(new))  # some begin
    slot = r.permutation(len(new) + 3)[: len(new)]
    if len(new) > 4:
        slot[3] = -1  # padding
    return new, cached, slot


def _arrays(new, cached, slot):
    q_start = np.concatenate([[0], np.cumsum(new)])
    return q_start, np.asarray(new) + cached, slot


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("kind", ["one", "step", "short", "long", "ragged"])
@pytest.mark.parametrize("channels,width,silu", [(8, 4, True), (264, 2, True), (640, 3, False), (1032, 4, True)])
def test_conv(kq, dt, kind, channels, width, silu):
    t, g = TYPES[dt], _gen(channels)
    new, cached, slot = _steps(kind, channels)
    q_start, kv_len, slot = _arrays(new, cached, slot)
    tokens = int(q_start[-1])
    x = torch.randn(tokens + 5, channels + 24, generator=g).to(t).cuda()[:, 16: 16 + channels]  # strided, rows behind the last
    w = torch.randn(channels, width, generator=g)
    bias = torch.randn(channels, generator=g) if width != 3 else None
    state = torch.randn(len(slot) + 3, width - 1, channels, generator=g).to(t)
    want, after = ref.conv(x.cpu(), w, bias, silu, q_start, kv_len, slot, state)
    out = torch.full((tokens + 5, channels), 7.0, dtype=t, device="cuda")
    sc = state.cuda()
    kq.kq_causal_conv(kq.CausalConv(w.cuda(), None if bias is None else bias.cuda(), silu), x, _int(q_start), _int(kv_len),
                      _int(slot), sc, out)
    assert torch.equal(sc.cpu().double(), after)
    done = ~torch.isnan(want[:, 0])
    assert bool((out[(~done).cuda()] == 7).all())  # skipped requests, rows behind the last
    size, _ = ref.conv(x.cpu().abs(), w.abs(), None if bias is None else bias.abs(), False, q_start, kv_len, slot, state.abs())
    err = (out.cpu().double() - want).abs()[done]
    bound = (want.abs() * _half(t) * 1.01 + 12 * H * size)[done] + torch.finfo(t).smallest_normal * torch.finfo(t).eps
    assert bool((err <= bound).all()), float((err / bound).max())
    _ok(kq)


def test_conv_in_pieces_is_conv_at_once(kq):
    g = _gen(1)
    x, w = torch.randn(150, 64, generator=g).cuda(), torch.randn(64, 4, generator=g).cuda()
    p = kq.CausalConv(w)
    whole, parts = torch.empty_like(x), torch.empty_like(x)
    a, b = torch.ones(1, 3, 64, device="cuda"), torch.ones(1, 3, 64, device="cuda")
    kq.kq_causal_conv(p, x, _int([0, 150]), _int([150]), _int([0]), a, whole)
    at = 0
    for n in (1, 1, 2, 5, 90, 3, 48):
        kq.kq_causal_conv(p, x[at: at + n], _int([0, n]), _int([at + n]), _int([0]), b, parts[at: at + n])
        at += n
    assert torch.equal(whole, parts) and torch.equal(a, b)
    # without lengths every state goes on
    c = torch.ones(1, 3, 64, device="cuda")
    kq.kq_causal_conv(p, x, _int([0, 150]), None, _int([0]), c, parts)
    assert torch.equal(c, a) and not torch.equal(parts[:3], whole[:3]) and torch.equal(parts[3:], whole[3:])


@pytest.mark.parametrize("tokens", [700, 1500, 3100, 6100])
def test_conv_of_many_channels_is_that_of_few(kq, tokens):
    """Pieces are longer where there is more to do; nothing of a channel's arithmetic goes by them."""
    g, c = _gen(tokens), 10240
    x, w = torch.randn(tokens, c, generator=g).half().cuda(), torch.randn(c, 4, generator=g).cuda()
    new = [5, 0, 129, 1, 2, tokens - 400, 263]
    q_start, kv_len, slot = _arrays(new, np.array([0, 1, 1, 0, 3, 0, 2]), np.array([3, 0, 6, 1, 5, 2, 4]))
    state = torch.randn(8, 3, c, generator=g).half().cuda()
    args = _int(q_start), _int(kv_len), _int(slot)
    out, after = torch.zeros_like(x), state.clone()
    kq.kq_causal_conv(kq.CausalConv(w), x, *args, after, out)
    for lo in range(0, c, 1024):
        part, s = torch.zeros(tokens, 1024, dtype=x.dtype, device="cuda"), state[:, :, lo: lo + 1024].contiguous()
        kq.kq_causal_conv(kq.CausalConv(w[lo: lo + 1024].contiguous()), x[:, lo: lo + 1024], *args, s, part)
        assert torch.equal(part, out[:, lo: lo + 1024]) and torch.equal(s, after[:, :, lo: lo + 1024])
    _ok(kq)


def test_conv_malformed_requests(kq):
    x, w = torch.randn(20, 16).cuda(), torch.randn(16, 4).cuda()
    p = kq.CausalConv(w)
    for q_start, slot in (([0, 5, 30], [0, 1]), ([0, 5, 3], [0, 1]), ([-1, 5, 9], [0, 1]), ([0, 5, 9], [0, 4]),
                          ([25, 30, 31], [0, 1]), ([5, 2 ** 31 - 1, 5], [0, 1])):
        state, out = torch.zeros(3, 3, 16, device="cuda"), torch.empty(20, 16, device="cuda")
        kq.kq_causal_conv(p, x, _int(q_start), None, _int(slot), state, out)
        assert kq.kq_device_status(True) == kq.KQ_ERR_RANGE, (q_start, slot)


# ---- the gated delta rule ------------------------------------------------------------------------


class Delta:
    """Inputs of a step on the CPU, and what the rule makes of them in 64 bits."""

    def __init__(self, dt, kind, hk, hv, d, seed=0, unit=True, gates=True, strided=True, size=1.0, common=0.3, decay=None,
                 scale=None):
        t, g = TYPES[dt], _gen(seed)
        new, cached, slot = kind if isinstance(kind, tuple) else _steps(kind, seed + d)
        self.q_start, self.kv_len, self.slot = _arrays(new, cached, slot)
        self.tokens, self.new, self.dt = int(self.q_start[-1]), new, t
        wide = (2 * hk + hv) * d
        x = torch.randn(self.tokens + 3, wide + 32, generator=g) + common * torch.randn(1, wide + 32, generator=g)
        if not unit:
            x /= math.sqrt(d)
        x[:, 2 * hk * d: wide] *= size
        x = x.to(t)
        if not strided:
            x = x[:, :wide].contiguous()
        self.q = x[:, : hk * d].unflatten(1, (hk, d))
        self.k = x[:, hk * d: 2 * hk * d].unflatten(1, (hk, d))
        self.v = x[:, 2 * hk * d: wide].unflatten(1, (hv, d))
        ab = torch.randn(self.tokens + 3, 2 * hv + 3, generator=g)
        if not gates:
            ab = torch.cat((-ab.abs() * 0.1, ab.sigmoid()), 1)[:, : 2 * hv + 3]
            ab[:, :hv], ab[:, hv: 2 * hv] = -0.1 * torch.rand(ab[:, :hv].shape, generator=g), torch.rand(ab[:, :hv].shape, generator=g)
        ab = ab.to(t)
        self.a, self.b = ab[:, :hv], ab[:, hv: 2 * hv]
        self.a_log = torch.log(1 + 15 * torch.rand(hv, generator=g)) if gates else None
        self.dt_bias = torch.randn(hv, generator=g) - 3 if gates else None
        if decay is not None:
            self.dt_bias = torch.full((hv,), float(decay))
        self.state = size * torch.randn(len(slot) + 3, hv, d, d, generator=g) * 0.3
        self.shape = (hk, hv, d)
        self.unit = unit
        self.eps, self.scale = 1e-6, d ** -0.5 if scale is None else scale
        self.want, self.after = ref.gdn(self.q, self.k, self.v, self.a, self.b, self.a_log, self.dt_bias, unit, self.eps,
                                        self.scale, self.q_start, self.kv_len, self.slot, self.state)

    def rule(self, kq):
        cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
        return kq.GatedDelta(*self.shape, cuda(self.a_log), cuda(self.dt_bias), unit=self.unit, eps=self.eps,
                             scale=self.scale)

    def run(self, kq, max_new=None, ws=None, stream=None):
        p = self.rule(kq)
        most = max(self.new) if max_new is None else max_new
        out = torch.full(self.v.shape, 7.0, dtype=self.dt, device="cuda")
        state = self.state.cuda()
        n = kq.kq_gdn_workspace_bytes(p, self.dt, len(self.new), self.v.shape[0], most)
        ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        move = lambda t: torch.empty(t._base.shape, dtype=t.dtype, device="cuda").copy_(t._base).as_strided(  # noqa: E731
            t.shape, t.stride(), t.storage_offset()) if t._base is not None else t.cuda()
        kq.kq_gdn(p, move(self.q), move(self.k), move(self.v), move(self.a), move(self.b), _int(self.q_start), _int(self.kv_len),
                  _int(self.slot), state, out, most, ws=ws, stream=stream)
        torch.cuda.synchronize()
        return out.cpu(), state.cpu()

    def check(self, out, state, longest=None, factor=4):
        done = ~torch.isnan(self.want[:, 0, 0])
        assert bool((out[~done] == 7).all())
        used = [int(s) for s, n in zip(self.slot, self.new) if s >= 0 and n]
        idle = [s for s in range(self.state.shape[0]) if s not in used]
        assert torch.equal(state[idle], self.state[idle])
        tol = factor * (16 + 2 * math.sqrt(self.shape[2] * (longest or max(self.new)))) * H
        off = (state[used].double() - self.after[used]).norm() / self.after[used].norm()
        assert float(off) <= tol, ("state", float(off), tol)
        err, want = out.double()[done] - self.want[done], self.want[done]
        half = _half(self.dt)
        off = float(err.norm() / want.norm())
        assert off <= tol + half, ("out", off, tol)
        # element by element: a rounding of the output's own, and the arithmetic's share at five times the mean
        rms = float(want.pow(2).mean().sqrt())
        worst = float((err.abs() / (want.abs() * half * 1.01 + 5 * tol * (rms + want.abs()))).max())
        assert worst <= 1, ("out, one element", worst)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("kind", ["one", "step", "short", "mid"])
@pytest.mark.parametrize("hk,hv,d", [(1, 1, 128), (2, 6, 128), (3, 3, 64), (1, 4, 64)])
def test_gdn(kq, dt, kind, hk, hv, d):
    c = Delta(dt, kind, hk, hv, d)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("kind", ["long", "ragged"])
@pytest.mark.parametrize("hk,hv,d", [(1, 2, 128), (2, 2, 64)])
def test_gdn_prompts(kq, dt, kind, hk, hv, d):
    c = Delta(dt, kind, hk, hv, d, seed=3)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("unit,gates", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("kind", ["short", "mid"])
def test_gdn_gates_and_keys_as_they_are(kq, dt, unit, gates, kind):
    c = Delta(dt, kind, 2, 4, 128, seed=7, unit=unit, gates=gates, strided=False)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("decay", [-12.0, 4.0, 60.0])
def test_gdn_decays_from_none_to_all(kq, dt, decay):
    """Next to no decay (errors add up over all tokens), and decays that leave nothing of a state within a chunk."""
    c = Delta(dt, ([400, 65], [0, 9], np.array([1, 0])), 1, 2, 128, seed=11, decay=decay)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("common", [0.0, 10.0, 100.0])
def test_gdn_keys_alike(kq, dt, common):
    """Keys of one direction: the triangular system is as full as it gets."""
    c = Delta(dt, ([300], [1], np.array([0])), 1, 2, 128, seed=12, common=common, decay=-8.0)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("size", [1e-5, 30.0, 1e4, 1e12, 1e30])
def test_gdn_values_of_any_size(kq, size):
    if size > 1e4:
        c = Delta("bf16", "mid", 1, 2, 128, seed=13, size=size)
    else:
        c = Delta("f16", "mid", 1, 2, 128, seed=13, size=min(size, 1e4))
        c.after, c.want = c.after.clone(), c.want.clone()
    if size == 1e-5:  # fp16 outputs are subnormal: only the states are compared
        out, state = c.run(kq)
        used = [int(s) for s, n in zip(c.slot, c.new) if s >= 0 and n]
        assert float((state[used].double() - c.after[used]).norm() / c.after[used].norm()) <= 4 * (16 + 2 * math.sqrt(128 * 130)) * H
    else:
        c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_gdn_many_requests_of_all_lengths(kq, dt):
    """More than are ordered by length at a time, some of equal lengths, skipped or without tokens, short ones among them."""
    r = np.random.default_rng(31)
    new = [int(n) for n in r.choice([0, 1, 7, 32, 33, 64, 65, 130], 71)]
    slot = r.permutation(74)[:71]
    slot[r.choice(71, 9, replace=False)] = -1
    c = Delta(dt, (new, [int(n) for n in r.integers(0, 2, 71)], slot), 1, 2, 128, seed=32)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("new", [[1176], [89, 50, 70]])
def test_gdn_fp32_prompts_keep_fp32(kq, new):
    """Chunks lose no more than fp32 itself does: a factor in two fp16 parts is off by h at most (four of them in an output),
    and a product of 128 is eight additions that are cut off, by 2 h of what the sum is then, one of 64 four: 4 + 8 + 4 h."""
    c = Delta("f32", (new, [0] * len(new), np.arange(len(new))), 2, 4, 128, seed=3)
    out, state = c.run(kq)
    used, done = [int(i) for i in c.slot], ~torch.isnan(c.want[:, 0, 0])
    assert float((out.double()[done] - c.want[done]).norm() / c.want[done].norm()) <= 16 * H
    assert float((state[used].double() - c.after[used]).norm() / c.after[used].norm()) <= 16 * H
    _ok(kq)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["short", "mid"])
@pytest.mark.parametrize("scale", [1e-6, -1e6])
def test_gdn_scales_of_any_size(kq, dt, kind, scale):
    """Factors that no fp16 number comes near: a query's scale is the caller's."""
    c = Delta(dt, kind, 1, 2, 128, seed=14, scale=scale)
    c.check(*c.run(kq))
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
def test_gdn_in_pieces_is_gdn_at_once(kq, dt):
    """Prompt, short runs and single tokens go on from one another's states."""
    t, g, d = TYPES[dt], _gen(4), 128
    n = 333
    q, k, v = (torch.randn(n, h, d, generator=g).to(t).cuda() for h in (1, 1, 3))
    a, b = torch.randn(n, 3, generator=g).to(t).cuda(), torch.randn(n, 3, generator=g).to(t).cuda()
    p = kq.GatedDelta(1, 3, d, torch.zeros(3).cuda(), torch.zeros(3).cuda() - 4)
    want, after = ref.gdn(q.cpu(), k.cpu(), v.cpu(), a.cpu(), b.cpu(), torch.zeros(3), torch.zeros(3) - 4, True, 1e-6, d ** -0.5,
                          [0, n], [n], [0], torch.zeros(1, 3, d, d))
    state, out, at = torch.full((1, 3, d, d), math.nan).cuda(), torch.empty_like(v), 0
    for m in (64, 1, 1, 130, 3, 65, 5, 64):
        s = slice(at, at + m)
        ws = torch.empty(max(16, kq.kq_gdn_workspace_bytes(p, t, 1, m, m)), dtype=torch.uint8, device="cuda")
        kq.kq_gdn(p, q[s], k[s], v[s], a[s], b[s], _int([0, m]), _int([at + m]), _int([0]), state, out[s], m, ws=ws)
        at += m
    tol = 4 * (16 + 2 * math.sqrt(d * n)) * H
    assert float((state[0].cpu().double() - after[0]).norm() / after[0].norm()) <= tol
    assert float((out.cpu().double() - want).norm() / want.norm()) <= tol + _half(t)
    _ok(kq)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_gdn_output_over_the_values(kq, dt):
    c = Delta(dt, "mid", 2, 4, 128, seed=2, strided=False)
    out, state = c.run(kq)
    p = c.rule(kq)
    v, s = c.v.cuda().contiguous(), c.state.cuda()
    n = kq.kq_gdn_workspace_bytes(p, c.dt, len(c.new), v.shape[0], max(c.new))
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    kq.kq_gdn(p, c.q.cuda(), c.k.cuda(), v, c.a.cuda(), c.b.cuda(), _int(c.q_start), _int(c.kv_len), _int(c.slot), s, v,
              max(c.new), ws=ws)
    done = ~torch.isnan(c.want[:, 0, 0])
    assert torch.equal(v.cpu()[done], out[done]) and torch.equal(s.cpu(), state)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gdn_malformed_requests(kq, dt):
    t = TYPES[dt]
    p = kq.GatedDelta(1, 1, 128, torch.zeros(1).cuda(), torch.zeros(1).cuda())
    q, ab = torch.randn(200, 1, 128).to(t).cuda(), torch.randn(200, 1).to(t).cuda()
    for q_start, slot, most in (([0, 150, 230], [0, 1], 180), ([0, 150, 120], [0, 1], 180), ([-1, 5, 9], [0, 1], 180),
                                ([0, 5, 9], [0, 4], 180), ([0, 150, 152], [0, 1], 149), ([5, 2 ** 31 - 1, 5], [0, 1], 180)):
        state, out = torch.zeros(3, 1, 128, 128, device="cuda"), torch.empty(200, 1, 128, dtype=t, device="cuda")
        ws = torch.empty(max(16, kq.kq_gdn_workspace_bytes(p, t, 2, 200, most)), dtype=torch.uint8, device="cuda")
        kq.kq_gdn(p, q, q, q, ab, ab, _int(q_start), None, _int(slot), state, out, most, ws=ws)
        assert kq.kq_device_status(True) == kq.KQ_ERR_RANGE, (q_start, slot, most)


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_gdn_step_in_a_graph_and_on_another_stream(kq, dt):
    c = Delta(dt, "mid", 1, 2, 128, seed=21)
    out, state = c.run(kq)
    p, most = c.rule(kq), max(c.new)
    dev = [t.cuda() for t in (c.q, c.k, c.v, c.a, c.b)]
    arrays = _int(c.q_start), _int(c.kv_len), _int(c.slot)
    s, o = c.state.cuda(), torch.full(c.v.shape, 7.0, dtype=c.dt, device="cuda")
    n = kq.kq_gdn_workspace_bytes(p, c.dt, len(c.new), c.v.shape[0], most)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        kq.kq_gdn(p, *dev, *arrays, s, o, most, ws=ws)
    side.synchronize()
    assert torch.equal(o.cpu(), out) and torch.equal(s.cpu(), state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kq.kq_gdn(p, *dev, *arrays, s, o, most, ws=ws)
    for _ in range(2):
        s.copy_(c.state)
        o.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.cpu(), out) and torch.equal(s.cpu(), state)
    _ok(kq)


# ---- sampling --------------------------------------------------------------------------------------


def _logits(rows, vocab, dt, seed, spread=2.2):
    g = _gen(seed)
    x = spread * torch.randn(rows, vocab, generator=g)
    at = torch.randint(0, vocab, (rows, 9), generator=g)
    x.scatter_add_(1, at, 5 + 6 * torch.rand(rows, 9, generator=g))
    return x.to(TYPES[dt])


def _check_sample(kq, x, u, where=None, **settings):
    """Tokens equal to the definition's in 64 bits, but where u lies within rounding of a border: weights are good to 2^-21
    each (2 ulp of exp2f, 3 roundings around it), so running sums are to that share of the whole."""
    rows = x.shape[0]
    dev = where if where is not None else x.cuda()
    token, prob = torch.full((rows,), -7, dtype=torch.int32, device="cuda"), torch.full((rows,), -7.0, device="cuda")
    per = {}
    for name, val in settings.items():
        t = torch.int32 if name == "top_k" else torch.float32
        per[name] = torch.as_tensor(val, dtype=t).expand(rows).contiguous().cuda()
    kq.kq_sample(dev, u.cuda(), token, prob, **per)
    token, prob = token.cpu(), prob.cpu()
    for r in range(rows):
        mine = {n: (int if n == "top_k" else float)(per[n][r]) for n in per}
        want, p, slack = ref.sample(x[r], float(u[r]), **mine)
        if slack > 2.0 ** -21:
            assert int(token[r]) == want, (r, mine, float(u[r]), int(token[r]), want, slack)
            assert abs(float(prob[r]) - p) <= 2.0 ** -20 * p + 1e-30, (r, float(prob[r]), p)
        else:
            assert 0 <= int(token[r]) < x.shape[1]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 7), (5, 1000), (3, 4097), (4, 32003), (2, 151936), (1, 248320), (1, 393216)])
@pytest.mark.parametrize("settings", [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=20, top_p=0.8),
                                      dict(temperature=1.3, top_p=0.95, min_p=0.02), dict(top_k=1), dict(temperature=0.01),
                                      dict(temperature=100.0, top_p=0.5), dict(top_k=900, min_p=0.3), dict(top_p=0.0), dict(min_p=1.0)])
def test_sample(kq, dt, rows, vocab, settings):
    x = _logits(rows, vocab, dt, vocab)
    _check_sample(kq, x, torch.rand(rows, generator=_gen(vocab + 1)), **settings)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
def test_sample_ties(kq, dt):
    """Equal logits: the lowest ids are kept, however they are spread over the slices."""
    for vocab, values in ((5000, 1), (40000, 3), (40000, 40), (100000, 1)):
        g = _gen(vocab + values)
        x = torch.randint(0, values, (6, vocab), generator=g).to(TYPES[dt])
        u = torch.tensor([0.0, 0.2, 0.5, 0.77, 0.999, 1 - 2.0 ** -24])
        for s in (dict(top_k=7), dict(top_k=vocab // 2 + 1), dict(top_p=0.3), dict(top_k=100, top_p=0.5), dict(temperature=0.0),
                  dict(min_p=0.9), dict()):
            _check_sample(kq, x, u, **s)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("top_k", [2, 63, 64, 65, 128, 129, 256, 257])
def test_sample_both_sides_of_each_count(kq, dt, top_k):
    """Where few are ranked, sorted or found by a histogram; logits apart and in groups of equal ones; kept all and in part."""
    for vocab in (300, 5001, 40000):
        x = _logits(4, vocab, dt, vocab + top_k)
        x[2:] = (x[2:].float() * 4).round().to(x.dtype) / 4
        u = torch.rand(4, generator=_gen(top_k))
        for s in (dict(), dict(top_p=0.9), dict(temperature=0.6, top_p=0.97, min_p=0.05)):
            _check_sample(kq, x, u, top_k=top_k, **s)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("min_p", [1e-12, 1e-4, 0.02, 0.6])
def test_sample_min_p_on_either_side_of_top_p(kq, dt, min_p):
    """The border of one above, between and below that of the other, and of top_k's where there are three."""
    x, u = _logits(5, 30011, dt, 77), torch.rand(5, generator=_gen(78))
    x[3:] = (x[3:].float() * 8).round().to(x.dtype) / 8
    for s in (dict(top_p=0.2), dict(top_p=0.95), dict(top_p=0.9999), dict(top_p=0.95, top_k=700), dict(top_p=0.5, top_k=5000)):
        _check_sample(kq, x, u, min_p=min_p, **s)
    _ok(kq)


def test_sample_per_row_settings_and_strides(kq):
    x = _logits(9, 3001, "f32", 5)
    u = torch.rand(9, generator=_gen(6))
    settings = dict(temperature=[0.0, 0.5, 1.0, 2.0, 1.0, 0.3, 1.0, 1.0, 1.0], top_k=[0, 5, 3001, 4000, -3, 50, 2 ** 31 - 1, 2, 0],
                    top_p=[1.0, 0.9, 0.5, 2.0, -1.0, 0.99, 1.0, 1.0, 1e-6], min_p=[0.0, 0.1, 0.0, 0.01, 0.0, 0.5, 2.0, 0.0, -1.0])
    wide = torch.full((9, 3010), 50.0, device="cuda")
    wide[:, 5:3006] = x.cuda()
    _check_sample(kq, x, u, where=wide[:, 5:3006], **settings)
    half = _logits(4, 777, "f16", 8)
    wide = torch.full((4, 800), 50.0, dtype=torch.float16, device="cuda")
    wide[:, 3:780] = half.cuda()
    _check_sample(kq, half, u[:4], where=wide[:, 3:780], top_k=9)
    _check_sample(kq, x, torch.tensor([-1.0, 0.0, 1.0, 2.0, math.inf, -math.inf, 0.5, 0.5, 0.5]))
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
def test_sample_masked_and_infinite(kq, dt):
    least = torch.finfo(TYPES[dt]).min
    x = _logits(6, 20000, dt, 3)
    x[0, 100:] = -math.inf
    x[1, 1:] = least
    x[2, ::2] = least
    x[3, 5], x[3, 19000] = math.inf, math.inf
    x[4, :19999] = -math.inf
    x[5] = least  # all alike, if low
    u = torch.tensor([0.9, 0.9, 0.3, 0.7, 0.4, 0.25])
    for s in (dict(), dict(top_k=3), dict(top_p=0.9), dict(temperature=0.0), dict(top_k=30, top_p=0.99, min_p=1e-4)):
        _check_sample(kq, x, u, **s)
    _ok(kq)
    x[0, 7] = math.nan
    x[2] = -math.inf
    _check_sample(kq, x, u)
    assert kq.kq_device_status(True) == kq.KQ_ERR_NONFINITE
    token = torch.empty(4, dtype=torch.int32, device="cuda")
    kq.kq_sample(x[:4].cuda() * 0, u[:4].cuda(), token, temperature=torch.tensor([-1.0, math.nan, math.inf, 1.0]).cuda())
    assert token.cpu().tolist()[:3] == [-1] * 3
    assert kq.kq_device_status(True) == kq.KQ_ERR_NONFINITE


def test_sample_follows_the_distribution(kq):
    """4096 numbers evenly over [0, 1) meet each token as often as its probability says, to within one."""
    x = _logits(1, 500, "f32", 17)
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    token, prob = torch.empty(n, dtype=torch.int32, device="cuda"), torch.empty(n, device="cuda")
    kq.kq_sample(x.expand(n, -1).contiguous().cuda(), u.cuda(), token, prob, temperature=torch.full((n,), 1.5).cuda())
    p = torch.softmax(x[0].double() / 1.5, 0)
    count = torch.bincount(token.cpu().long(), minlength=500).double()
    assert float((count - n * p).abs().max()) <= 1 + 1e-3
    assert float((prob.cpu().double() - p[token.cpu().long()]).abs().max()) <= 2.0 ** -20
