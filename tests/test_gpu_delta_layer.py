"""The delta layers' operators together, as a step uses them, and with tensors that pass 32 bits.  Tolerances as in
test_gpu_delta."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import delta_reference as ref  # noqa: E402
from test_gpu_delta import H, TYPES, Delta, _check_sample, _gen, _half, _int, _ok, kq  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_example_delta_layer(kq):  # noqa: F811
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_layer.py")
    spec = importlib.util.spec_from_file_location("delta_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    # the heads' norm divides by their size, so errors stay relative: those of convolution, rule and norm added up
    assert module.main(requests=3, prompt=33, steps=3) < 4 * (16 + 2 * math.sqrt(128 * 38)) * H


@pytest.mark.parametrize("dt", list(TYPES))
def test_layer_in_a_graph(kq, dt):  # noqa: F811
    """Norm, convolution, rule, gated norm and a choice of tokens in one captured graph: prompts, short runs, a request without
    tokens and a padded one.  Replays give what the same calls gave one by one, and the 64-bit pipeline's values."""
    t, g, hk, hv, d = TYPES[dt], _gen(9), 2, 4, 128
    new, cached, slot = [90, 0, 17, 1, 3, 1, 64], [0, 4, 5, 9, 0, 2, 64], [3, 0, 5, -1, 1, 6, 2]
    start = [sum(new[:r]) for r in range(len(new) + 1)]
    kv_len = [n + c for n, c in zip(new, cached)]
    tokens, channels, inner = start[-1], (2 * hk + hv) * d, hv * d
    x, res = (torch.randn(tokens, 1, channels, generator=g).to(t) for _ in range(2))
    z, ab = torch.randn(tokens, inner, generator=g).to(t), torch.randn(tokens, 2 * hv, generator=g).to(t)
    w, wc, wh = torch.rand(channels, generator=g) + 0.5, torch.randn(channels, 4, generator=g) * 0.5, torch.rand(d, generator=g) + 0.5
    past = torch.randn(8, 3, channels, generator=g).to(t)
    a_log, dt_bias = torch.rand(hv, generator=g), torch.rand(hv, generator=g) - 3
    state = torch.randn(8, hv, d, d, generator=g) * 0.2
    u = torch.rand(tokens, generator=g)
    dev = {n: v.cuda() for n, v in dict(x=x, z=z, ab=ab, u=u).items()}
    norm, head, conv = kq.RMSNorm(1, channels, w.cuda()), kq.RMSNorm(hv, d, wh.cuda()), kq.CausalConv(wc.cuda())
    rule = kq.GatedDelta(hk, hv, d, a_log.cuda(), dt_bias.cuda())
    arrays = _int(start), _int(kv_len), _int(slot)
    ws = torch.empty(max(16, kq.kq_gdn_workspace_bytes(rule, t, len(new), tokens, 90)), dtype=torch.uint8, device="cuda")
    buf = {n: torch.empty(s, dtype=t, device="cuda") for n, s in dict(y=(tokens, 1, channels), mixed=(tokens, channels),
                                                                       o=(tokens, hv, d), out=(tokens, hv, d)).items()}
    keep = dict(res=res.cuda(), past=past.cuda(), state=state.cuda(), token=torch.empty(tokens, dtype=torch.int32, device="cuda"))

    def layer():
        kq.kq_rms_norm(norm, dev["x"], buf["y"], residual=keep["res"])
        kq.kq_causal_conv(conv, buf["y"][:, 0], *arrays, keep["past"], buf["mixed"])
        h = buf["mixed"].unflatten(1, (-1, d))
        kq.kq_gdn(rule, h[:, :hk], h[:, hk: 2 * hk], h[:, 2 * hk:], dev["ab"][:, :hv], dev["ab"][:, hv:], *arrays, keep["state"],
                  buf["o"], 90, ws=ws)
        kq.kq_rms_norm(head, buf["o"], buf["out"], gate=dev["z"].unflatten(1, (hv, d)))
        kq.kq_sample(buf["out"].flatten(1), dev["u"], keep["token"])

    def reset():
        for v in buf.values():
            v.fill_(0.5)
        for n, v in dict(res=res, past=past, state=state).items():
            keep[n].copy_(v)

    reset()
    layer()
    first = {n: v.clone() for n, v in {**buf, **keep}.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for _ in range(3):
        reset()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for n, v in {**buf, **keep}.items():
            assert torch.equal(v, first[n]), n
    _ok(kq)
    # each operator's result from what the one before it gave
    c = lambda n: first[n].cpu()  # noqa: E731
    want, after = ref.conv(c("y")[:, 0], wc, None, True, start, kv_len, slot, past)
    done = ~torch.isnan(want[:, 0])
    assert torch.equal(c("past").double(), after) and bool((c("mixed")[~done] == 0.5).all())
    h = c("mixed").unflatten(1, (-1, d))
    want, after = ref.gdn(h[:, :hk], h[:, hk: 2 * hk], h[:, 2 * hk:], ab[:, :hv], ab[:, hv:], a_log, dt_bias, True, 1e-6, d ** -0.5, start,
                          kv_len, slot, state)
    tol = 4 * (16 + 2 * math.sqrt(d * 90)) * H
    assert float((c("o").double() - want)[done].norm() / want[done].norm()) <= tol + _half(t)
    used = [s for s, n in zip(slot, new) if s >= 0 and n]
    assert float((c("state").double() - after)[used].norm() / after[used].norm()) <= tol


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_gdn_states_past_32_bits(kq, dt):  # noqa: F811
    """Slots whose states lie more than 2^31 elements from the first."""
    c = Delta(dt, ([70, 1], [3, 2], [1, 0]), 1, 4, 128, seed=31)
    out, after = c.run(kq)
    p, far = c.rule(kq), [33000, 32999]
    big = torch.empty(33001, 4, 128, 128, device="cuda")
    for s, f in zip([1, 0], far):
        big[f].copy_(c.state[s])
    o = torch.full(c.v.shape, 7.0, dtype=c.dt, device="cuda")
    ws = torch.empty(max(16, kq.kq_gdn_workspace_bytes(p, c.dt, 2, c.v.shape[0], 70)), dtype=torch.uint8, device="cuda")
    kq.kq_gdn(p, *[x.cuda() for x in (c.q, c.k, c.v, c.a, c.b)], _int(c.q_start), _int(c.kv_len), _int(far), big, o, 70, ws=ws)
    assert torch.equal(o.cpu(), out)
    for s, f in zip([1, 0], far):
        assert torch.equal(big[f].cpu(), after[s])
    _ok(kq)


def test_rows_past_32_bits(kq):  # noqa: F811
    """Rows more than 2^31 elements apart: norm, convolution, sampling."""
    wide = 1 << 30
    base = torch.empty(2 * wide + 4096, dtype=torch.float16, device="cuda")
    rows = base.as_strided((3, 1024), (wide, 1))
    x = torch.randn(3, 1024, generator=_gen(2)).half()
    rows.copy_(x)
    y = torch.empty(3, 1, 1024, dtype=torch.float16, device="cuda")
    kq.kq_rms_norm(kq.RMSNorm(1, 1024), rows[:, None], y)
    near = torch.empty_like(y)
    kq.kq_rms_norm(kq.RMSNorm(1, 1024), x.cuda()[:, None], near)
    assert torch.equal(y, near)
    w = torch.randn(1024, 4, generator=_gen(3)).cuda()
    a, b = torch.zeros(1, 3, 1024, dtype=torch.float16, device="cuda"), torch.zeros(1, 3, 1024, dtype=torch.float16, device="cuda")
    far = base.as_strided((3, 1024), (wide, 1), 2048)
    kq.kq_causal_conv(kq.CausalConv(w), rows, _int([0, 3]), None, _int([0]), a, far)  # input and output side by side
    kq.kq_causal_conv(kq.CausalConv(w), x.cuda(), _int([0, 3]), None, _int([0]), b, near[:, 0])
    assert torch.equal(far, near[:, 0]) and torch.equal(a, b)
    _check_sample(kq, x, torch.tensor([0.1, 0.5, 0.9]), where=rows, top_k=50)
    _ok(kq)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_gdn_prompts_share_no_workspace_state(kq, dt):  # noqa: F811
    """Two calls one after the other on one workspace, and the larger one again: nothing of one is seen by the next."""
    big, small = Delta(dt, ([200, 131], [0, 7], [1, 0]), 1, 2, 128, seed=41), Delta(dt, ([77], [1], [0]), 1, 2, 128, seed=42)
    p = big.rule(kq)
    ws = torch.full((kq.kq_gdn_workspace_bytes(p, big.dt, 2, big.v.shape[0], 200),), 255, dtype=torch.uint8, device="cuda")
    one = big.run(kq, ws=ws)
    two = small.run(kq, ws=ws)
    again = big.run(kq, ws=ws)
    small.check(*two)
    big.check(*one)
    assert all(torch.equal(a, b) for a, b in zip(one, again))
    _ok(kq)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("new,cached,before", [(1537, 0, 0), (2100, 3, 71)])
def test_gdn_long_prompt_of_one_request(kq, dt, new, cached, before):  # noqa: F811
    """Prompts long enough that their chunks go in parts; one begins behind rows that are no request's."""
    c = Delta(dt, ([before, new], [0, cached], [-1, 2]), 1, 2, 128, seed=51, decay=-9.0)
    p = c.rule(kq)
    q, k, v, a, b = [x.cuda() for x in (c.q, c.k, c.v, c.a, c.b)]
    for _ in range(3):
        state, out = c.state.cuda(), torch.full(c.v.shape, 7.0, dtype=c.dt, device="cuda")
        n = kq.kq_gdn_workspace_bytes(p, c.dt, 1, v.shape[0], new)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        kq.kq_gdn(p, q, k, v, a, b, _int([before, before + new]), _int([new + cached]), _int([2]), state, out, new, ws=ws)
        c.check(out.cpu(), state.cpu(), longest=new)
    # a bound far above the tokens that there are
    ws = torch.full((kq.kq_gdn_workspace_bytes(p, c.dt, 1, v.shape[0], 100000),), 255, dtype=torch.uint8, device="cuda")
    state, again = c.state.cuda(), torch.full(c.v.shape, 7.0, dtype=c.dt, device="cuda")
    kq.kq_gdn(p, q, k, v, a, b, _int([before, before + new]), _int([new + cached]), _int([2]), state, again, 100000, ws=ws)
    assert torch.equal(again, out)
    # the outputs over the values
    state, over = c.state.cuda(), v.contiguous().clone()
    kq.kq_gdn(p, q, k, over, a, b, _int([before, before + new]), _int([new + cached]), _int([2]), state, over, new, ws=ws)
    assert torch.equal(over[before: before + new], out[before: before + new])
    _ok(kq)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_calls_of_two_streams(kq, dt):  # noqa: F811
    """Prompts in parts, ragged prompts, steps and sampling on two streams at once give what they give one after the other."""
    t, g = TYPES[dt], torch.Generator().manual_seed(9)
    hk, hv, d = 4, 12, 128
    p = kq.GatedDelta(hk, hv, d, torch.zeros(hv, device="cuda"), torch.full((hv,), -3.0, device="cuda"))
    steps = []
    for new in ([1700], [300, 20, 0, 65, 500], [1] * 9, [1900]):
        n, r = sum(new), len(new)
        q, k = (torch.randn(n, hk, d, generator=g).to(t).cuda() for _ in range(2))
        v = torch.randn(n, hv, d, generator=g).to(t).cuda()
        a, b = (torch.randn(n, hv, generator=g).to(t).cuda() for _ in range(2))
        ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (np.concatenate([[0], np.cumsum(new)]), [n + 1 for n in new], range(r))]
        logits, u = (2 * torch.randn(3, 50000, generator=g)).to(t).cuda(), torch.rand(3, generator=g).cuda()
        steps.append((new, q, k, v, a, b, ints, torch.randn(r, hv, d, d, generator=g).cuda(), logits, u))

    def run(order):
        got = []
        for i, s in order:
            new, q, k, v, a, b, ints, state, logits, u = steps[i]
            with torch.cuda.stream(s):
                out, state, token = torch.full_like(v, 7), state.clone(), torch.empty(3, dtype=torch.int32, device="cuda")
                ws = torch.empty(max(16, kq.kq_gdn_workspace_bytes(p, t, len(new), v.shape[0], max(new))), dtype=torch.uint8, device="cuda")
                kq.kq_gdn(p, q, k, v, a, b, *ints, state, out, max(new), ws=ws)
                kq.kq_sample(logits, u, token, top_p=torch.full((3,), 0.9, device="cuda"))
                got.append((i, out, state, token, ws))
        torch.cuda.synchronize()
        return sorted(got, key=lambda x: x[0])

    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    want = run([(i, torch.cuda.current_stream()) for i in range(4)])
    for _ in range(3):
        for x, y in zip(run([(0, s1), (3, s2), (1, s1), (2, s2)]), want):
            assert all(torch.equal(a, b) for a, b in zip(x[1:4], y[1:4])), x[0]
    _ok(kq)
