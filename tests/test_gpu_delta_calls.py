"""The delta layers' operators, the norm and sampling as calls among others: inputs that the kernel launched just before has
written, on the GPU."""
import pytest

torch = pytest.importorskip("torch")

from test_gpu_delta import TYPES, _gen, _ok, kq  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,vocab", [(1, 8192), (3, 32768), (40, 4096)])
def test_sample_right_behind_what_writes_the_logits(kq, dt, rows, vocab):  # noqa: F811
    """The norm leaves the logits, and sampling starts while it runs: in one graph, replayed on new inputs,
    tokens are those of the logits as they are now."""
    t = TYPES[dt]
    p = kq.RMSNorm(1, vocab)
    x, logits = torch.zeros(rows, 1, vocab, dtype=t, device="cuda"), torch.zeros(rows, 1, vocab, dtype=t, device="cuda")
    u, tokens = torch.rand(rows, generator=_gen(3)).cuda(), [torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(3)]
    greedy, few = torch.zeros(rows, device="cuda"), torch.full((rows,), 5, dtype=torch.int32, device="cuda")

    def step():
        for token, s in zip(tokens, (dict(temperature=greedy), dict(top_k=few), dict())):
            kq.kq_rms_norm(p, x, logits)
            kq.kq_sample(logits[:, 0], u, token, **s)
            x.neg_()

    x.normal_()
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = _gen(4)
    for _ in range(20):
        x.copy_(3 * torch.randn(rows, 1, vocab, generator=g))
        y = x.clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logits[:, 0].gather(1, tokens[0].long()[:, None])[:, 0], logits[:, 0].amax(1))
        # of the same logits, one call by itself
        for token, sign, s in zip(tokens, (1, -1, 1), (dict(temperature=greedy), dict(top_k=few), dict())):
            alone, again = torch.empty_like(logits), torch.empty_like(token)
            kq.kq_rms_norm(p, sign * y, alone)
            torch.cuda.synchronize()
            kq.kq_sample(alone[:, 0], u, again, **s)
            assert torch.equal(again, token)
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
def test_views_side_by_side_in_one_buffer(kq, dt):  # noqa: F811
    """Rows that hold inputs and outputs next to one another, as a program's step buffer has them: nothing of it is refused, and
    the results are those of buffers apart."""
    t, g, hk, hv, d, n = TYPES[dt], _gen(7), 2, 4, 128, 70
    wide = (2 * hk + 3 * hv) * d
    rows = torch.randn(n, wide, generator=g).to(t).cuda()
    cut = lambda x, at, h: x[:, at * d: (at + h) * d].unflatten(1, (h, d))  # noqa: E731
    q, k, v, z, out = (cut(rows, at, h) for at, h in ((0, hk), (hk, hk), (2 * hk, hv), (2 * hk + hv, hv), (2 * hk + 2 * hv, hv)))
    ab = torch.randn(n, 2 * hv, generator=g).to(t).cuda()
    rule = kq.GatedDelta(hk, hv, d, torch.zeros(hv).cuda(), torch.full((hv,), -3.0).cuda())
    norm = kq.RMSNorm(hv, d)
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 50, 70], [50, 21], [1, 0])]
    state = torch.randn(2, hv, d, d, generator=g).cuda()
    ws = torch.empty(kq.kq_gdn_workspace_bytes(rule, t, 2, n, 50), dtype=torch.uint8, device="cuda")
    apart = [x.contiguous().clone() for x in (q, k, v, z)]
    s1, s2, o, y = state.clone(), state.clone(), torch.empty_like(apart[2]), torch.empty_like(apart[2])
    kq.kq_gdn(rule, *apart[:3], ab[:, :hv], ab[:, hv:], *ints, s1, o, 50, ws=ws)
    kq.kq_rms_norm(norm, o, y, gate=apart[3])
    kq.kq_gdn(rule, q, k, v, ab[:, :hv], ab[:, hv:], *ints, s2, out, 50, ws=ws)
    assert torch.equal(out, o) and torch.equal(s1, s2)
    kq.kq_rms_norm(norm, out, z, gate=z)
    assert torch.equal(z, y) and torch.equal(out, o)
    # twice the rows, the residual being the input's own view; outputs over the values
    x = apart[2].clone()
    kq.kq_rms_norm(norm, x, y, residual=x)
    assert torch.equal(x, (2 * apart[2].float()).to(t))
    s2.copy_(state)
    kq.kq_gdn(rule, q, k, v, ab[:, :hv], ab[:, hv:], *ints, s2, v, 50, ws=ws)
    assert torch.equal(v, o) and torch.equal(s1, s2)
    _ok(kq)
