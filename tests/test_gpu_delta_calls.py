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
