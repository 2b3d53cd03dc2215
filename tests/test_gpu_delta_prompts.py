"""The gated delta rule over prompts: every count of chunks around the walk's stages, and prompts that go in parts, with the
bound of fp32 that test_gdn_fp32_prompts_keep_fp32 derives (16 units of 2^-24 of the outputs' and states' norms; 16-bit
outputs their own rounding beside it)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402
from test_gpu_delta import H, TYPES, Delta, _half, _int, _ok, kq  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def _tight(c, out, state, units=16):
    used, done = [int(s) for s, n in zip(c.slot, c.new) if s >= 0 and n], ~torch.isnan(c.want[:, 0, 0])
    off = float((out.double()[done] - c.want[done]).norm() / c.want[done].norm())
    assert off <= units * H + _half(c.dt), off / H
    off = float((state[used].double() - c.after[used]).norm() / c.after[used].norm())
    assert off <= units * H, off / H


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("new", [[64], [65], [128], [190], [256], [64, 129, 320, 33, 200, 1, 70]])
def test_gdn_each_count_of_chunks(kq, dt, new):  # noqa: F811
    """Walks of fewer chunks than the stages and slots that they go through, of as many and of more; one right behind another on
    the same workspace, where each takes shared and tensor memory that the one before it has just left."""
    c = Delta(dt, (new, [i % 2 * 9 for i in range(len(new))], np.arange(len(new))[::-1].copy()), 2, 4, 128, seed=71)
    p = c.rule(kq)
    dev = [t.cuda() for t in (c.q, c.k, c.v, c.a, c.b)]
    arrays = _int(c.q_start), _int(c.kv_len), _int(c.slot)
    ws = torch.empty(kq.kq_gdn_workspace_bytes(p, c.dt, len(new), c.v.shape[0], max(new)), dtype=torch.uint8, device="cuda")
    states = [c.state.cuda() for _ in range(8)]
    outs = [torch.full(c.v.shape, 7.0, dtype=c.dt, device="cuda") for _ in range(8)]
    for s, o in zip(states, outs):
        kq.kq_gdn(p, *dev, *arrays, s, o, max(new), ws=ws)
    torch.cuda.synchronize()
    _tight(c, outs[0].cpu(), states[0].cpu())
    assert all(torch.equal(s, states[0]) for s in states) and all(torch.equal(o, outs[0]) for o in outs)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("new,cached,decay", [(1537, 0, None), (2100, 3, None), (2100, 3, -9.0)])
def test_gdn_prompts_in_parts_keep_fp32(kq, dt, new, cached, decay):  # noqa: F811
    """One request's prompt of 24 chunks and more, whose parts run beside one another.  With decays 16 H as above; where nothing
    fades the state's own rounding, half of H a chunk, adds up at random over the chunks: below sqrt(chunks) H."""
    c = Delta(dt, ([new], [cached], np.array([1])), 1, 2, 128, seed=81, decay=decay)
    out, state = c.run(kq)
    _tight(c, out, state, 16 + (0 if decay is None else (new / 64) ** 0.5))
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("eps", [1e-6, 1e-12])
@pytest.mark.parametrize("new", [[200], [70, 5, 130]])
def test_gdn_rows_of_zeros(kq, dt, eps, new):  # noqa: F811
    """Keys, queries, values and whole tokens of zeros among others, the first and the last of a request and of a chunk too: a key
    of zeros changes nothing, a query of zeros gives zeros."""
    c = Delta(dt, (new, [i % 2 * 9 for i in range(len(new))], np.arange(len(new))[::-1].copy()), 2, 4, 128, seed=91, strided=False)
    c.eps = eps
    for i, t in enumerate((0, 1, 17, 62, 63, 64, 66, sum(new) - 1)):
        if i % 2 == 0 or t >= 63:
            c.k[t, i % 2] = 0
        if i % 3 == 0:
            c.q[t] = 0
        if i % 4 == 1:
            c.v[t] = 0
    c.k[20: 30] = 0
    c.want, c.after = ref.gdn(c.q, c.k, c.v, c.a, c.b, c.a_log, c.dt_bias, True, eps, c.scale, c.q_start, c.kv_len, c.slot, c.state)
    out, state = c.run(kq)
    _tight(c, out, state)
    assert bool((out[0] == 0).all())
    _ok(kq)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("new,most", [(1, 64), (5, 100), (31, 40), (33, 33), (64, 3000), (100, 3000), (0, 100), (0, 3000)])
def test_gdn_one_request_shorter_than_its_bound(kq, dt, new, most):  # noqa: F811
    """A captured step is made for the most tokens that there may be; there are fewer, or none, and rows behind the last one stay
    as they are."""
    c = Delta(dt, ([new, 60], [7, 0], np.array([1, -1])), 2, 4, 128, seed=92)
    p, rows = c.rule(kq), 3100
    grow = lambda t: torch.cat((t, torch.ones(rows - len(t), *t.shape[1:], dtype=t.dtype))).cuda()  # noqa: E731
    state, out = c.state.cuda(), torch.full((rows, 4, 128), 7.0, dtype=c.dt, device="cuda")
    ws = torch.full((kq.kq_gdn_workspace_bytes(p, c.dt, 1, rows, most),), 255, dtype=torch.uint8, device="cuda")
    for slot in (-1, 1):  # a padded request first: nothing changes
        kq.kq_gdn(p, *[grow(t) for t in (c.q, c.k, c.v, c.a, c.b)], _int([0, new]), _int([new + 7]), _int([slot]), state, out, most, ws=ws)
        if slot < 0:
            assert torch.equal(state.cpu(), c.state) and bool((out == 7).all())
    assert bool((out[new:] == 7).all())
    if new:
        _tight(c, out.cpu()[: len(c.want)], state.cpu())
    else:
        assert torch.equal(state.cpu(), c.state)
    _ok(kq)


@pytest.mark.parametrize("size", [1e36, 2e37])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_gdn_values_near_the_end_of_fp32(kq, dt, size):  # noqa: F811
    c = Delta(dt, ([150, 64], [3, 0], np.array([1, 0])), 1, 2, 128, seed=93, size=size)
    _tight(c, *c.run(kq))
    _ok(kq)
