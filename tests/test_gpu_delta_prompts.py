"""The gated delta rule over prompts: every count of chunks around the walk's stages, and prompts that go in parts, with the
bound of fp32 that test_gdn_fp32_prompts_keep_fp32 derives (16 units of 2^-24 of the outputs' and states' norms; 16-bit
outputs their own rounding beside it)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402,F401
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
