"""The delta layers' operators, the norm and sampling where their accuracy shows: against 64-bit values, with bounds that
count the roundings of each step in units of H = 2^-24."""
import math

import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402
from test_gpu_delta import H, TYPES, _check_sample, _half, _int, _logits, _ok, kq  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def _silu_bound(dt, z):
    """fp32: the exponential instruction 4 (2^-22), its correction 1, its product with z 1, the sum 1, the reciprocal instruction 2
    (1 ulp), the last product 1: 10.  16-bit types: the argument's rounding and that of log2(e), 2^-24 + 2^-26.2 = 2^-23.7 of
    |z|; the two instructions and what is around them 2^-21; the result's own."""
    if dt == torch.float32:
        return 10 * H
    return z.abs() * 2.0 ** -23.7 + 2.0 ** -21 + _half(dt)


def _arguments(dt):
    g = torch.Generator().manual_seed(61)
    z = torch.cat((120 * torch.rand(30000, generator=g) - 60, 40 * torch.rand(2712, generator=g) - 100,
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 88.8, -88.8, -103.0, 5e4])))
    return z[: len(z) // 8 * 8].to(TYPES[dt])


def _check_silu(y, z, dt):
    z = z.double()
    want = z * ref.sigmoid(z)
    # nothing is left below -87.3, of less than 1.1e-36; subnormal results have steps of their own
    least = 1.1e-36 + (0 if dt == torch.float32 else torch.finfo(dt).smallest_normal * torch.finfo(dt).eps)
    bound = want.abs() * _silu_bound(dt, z) * 1.001 + least
    err = (y.cpu().double().flatten() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())


@pytest.mark.parametrize("dt", list(TYPES))
def test_silu_of_the_convolution_over_its_range(kq, dt):  # noqa: F811
    """A window that takes its last input alone leaves SiLU of the inputs."""
    z = _arguments(dt)
    for silu in (True, False):
        out, state = torch.empty(1, len(z), dtype=z.dtype, device="cuda"), torch.zeros(1, 1, len(z), dtype=z.dtype, device="cuda")
        p = kq.CausalConv(torch.tensor([0.0, 1.0]).expand(len(z), 2).contiguous().cuda(), None, silu)
        kq.kq_causal_conv(p, z.cuda()[None], _int([0, 1]), None, _int([0]), state, out)
        if silu:
            _check_silu(out, z, z.dtype)
        else:
            assert torch.equal(out.cpu()[0].float(), z.float())
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("heads,dim", [(1, 2048), (5, 128), (3, 40)])
def test_silu_of_the_norm_over_its_range(kq, dt, heads, dim):  # noqa: F811
    """Rows of +-1 have a root mean square of 1 exactly, so their gated norm is SiLU of the gates with the rows' signs."""
    z = _arguments(dt)
    z = z[: len(z) // (heads * dim) * heads * dim].view(-1, heads, dim)
    x = torch.where(torch.arange(dim) % 3 == 0, -1.0, 1.0).to(z.dtype).expand_as(z).contiguous()
    out = torch.empty_like(x, device="cuda")
    kq.kq_rms_norm(kq.RMSNorm(heads, dim, None, eps=0.0), x.cuda(), out, gate=z.cuda())
    _check_silu(out.cpu() * x, z.flatten(), z.dtype)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("vocab", [11, 1001, 40003])
@pytest.mark.parametrize("temperature", [1e36, 1e37, 1e38, 3.4e38])
def test_sample_masked_at_temperatures_that_leave_all_alike(kq, dt, vocab, temperature):  # noqa: F811
    """However high the temperature is, a logit of -infinity weighs nothing, and no more do those that fill a slice's last
    vector."""
    x = _logits(5, vocab, dt, vocab)
    x[0, 1:] = -math.inf
    x[1, ::3] = -math.inf
    x[2, vocab // 2:] = -math.inf
    x[3, : vocab - 1] = -math.inf
    u = torch.tensor([0.5, 0.999, 0.6, 0.1, 1 - 2.0 ** -24])
    for s in (dict(), dict(top_p=0.9), dict(top_k=7), dict(top_k=vocab - 1, top_p=0.99), dict(min_p=0.5)):
        _check_sample(kq, x, u, temperature=temperature, **s)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("vocab", [1500, 40003, 100000])
@pytest.mark.parametrize("temperature", [0.7, 5e36, 1.1e37, 1e38])
def test_sample_counts_down_into_masked_logits(kq, dt, vocab, temperature):  # noqa: F811
    """A top_k that reaches into logits of -infinity, of which all, a few or one remain, at temperatures whose 32 times fp32
    does not hold: the border is found, and whatever shared memory held before takes no part."""
    x = _logits(5, vocab, dt, vocab + 3)
    for r, finite in enumerate((3, 257, 700, vocab // 2, vocab - 1)):
        x[r].scatter_(0, torch.randperm(vocab, generator=torch.Generator().manual_seed(r))[finite:], -math.inf)
    u = torch.tensor([0.5, 0.999, 0.6, 0.1, 1 - 2.0 ** -24])
    for s in (dict(top_k=vocab - 1), dict(top_k=300), dict(top_k=vocab // 2 + 5, top_p=0.9), dict(top_k=1400, min_p=0.1)):
        _check_sample(kq, x, u, temperature=1.0, top_k=500)  # leaves a border of its own behind
        _check_sample(kq, x, u, temperature=temperature, **s)
    _ok(kq)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_sample_logits_as_large_as_fp32_holds(kq, dt):  # noqa: F811
    """Logits up to some 10^38 with temperatures of their size."""
    x, u = _logits(4, 30011, dt, 5), torch.tensor([0.2, 0.5, 0.9, 0.999])
    x = (x.float() * 5e36).to(TYPES[dt])
    for t in (5e36, 1e37, 4e37):
        for s in (dict(), dict(top_p=0.9), dict(top_k=20), dict(top_k=700), dict(top_p=0.99, min_p=0.01)):
            _check_sample(kq, x, u, temperature=t, **s)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("temperature", [1e-45, 1e-40, 1e-38, 1e-36, 1e-30, 1e-12])
def test_sample_temperatures_that_leave_the_largest(kq, dt, temperature):  # noqa: F811
    """However low the temperature is: the largest, or the equal ones at it by their share."""
    x, u = _logits(4, 30011, dt, 6), torch.tensor([0.2, 0.5, 0.9, 0.999])
    x[1, ::7] = x[1].max()
    x[2] = 1.5
    x[3, 5:] = -math.inf
    for s in (dict(), dict(top_p=0.9), dict(top_k=20), dict(top_k=700, top_p=0.4), dict(min_p=0.01), dict(top_p=0.7, min_p=0.01)):
        _check_sample(kq, x, u, temperature=temperature, **s)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
def test_sample_weights_where_the_difference_is_rounded(kq, dt):  # noqa: F811
    """The chance of the lesser of two logits, e / (1 + e).  Beside the largest of 16.5 small ones have bits that fp32's
    difference does not hold; e is off by 2^-21, and by 2^-24 of its exponent for 16-bit types, and by half of 2^-44; the sum and
    the quotient by a few 2^-53, the result by 2^-24."""
    small = [k * s * 2.0 ** -24 for k in (1, 3, 5, 9, 15, 17, 31) for s in (1, -1)] + [0.0, 2.0 ** -12, -0.37]
    cases = [(v, t) for v in small for t in (0.75, 0.8, 0.9, 1.0, 1.05, 1.1, 1.15, 1.3, 2.0, 5.0)]
    x = torch.tensor([[16.5, v] for v, _ in cases]).to(TYPES[dt])
    t = torch.tensor([t for _, t in cases])
    token, prob = torch.empty(len(cases), dtype=torch.int32, device="cuda"), torch.empty(len(cases), device="cuda")
    kq.kq_sample(x.cuda(), torch.ones(len(cases)).cuda(), token, prob, temperature=t.cuda())
    assert bool((token == 1).all())
    a = (x[:, 1].double() - 16.5) / t.double()
    e = torch.exp(a)
    bound = e * (2.0 ** -21 + (0 if dt == "f32" else 2.0 ** -24) * a.abs()) + 2.0 ** -45 + 2.0 ** -24 * e
    assert bool(((prob.cpu().double() - e / (1 + e)).abs() <= bound).all())
    _ok(kq)
