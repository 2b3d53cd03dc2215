"""One gated-delta layer of a decode, on the quantized weights, and the choice of a token.

    python examples/delta_layer.py [--requests 4] [--prompt 70] [--steps 4]

Runs a prompt and then single-token steps for a few requests through the calls that a
decode makes for such a layer (here one with the sizes of the Bonsai-27B-shaped decode
workload: hidden size 5120, 16 key and 48 value heads of 128):

    kq_rms_norm       the residual's addition and the norm before the projections
    kq_gemm_small_m   the fused q, k, v projection and the gates' (PQ2_0 weights, one stream for all rows)
    kq_causal_conv    the short convolution over the fused projection's channels
    kq_gdn            the gated delta rule
    kq_rms_norm       the norm of its heads, gated
    kq_gemm_small_m   the output projection; a small head
    kq_sample         a token of each request

and checks the last step's heads against the same in FP64, token by token.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_weight_streaming_gb300 as kq  # noqa: E402
import synth  # noqa: E402
import workloads  # noqa: E402

HIDDEN, K_HEADS, V_HEADS, D, WIDTH, VOCAB, EPS = 5120, 16, 48, 128, 4, 2000, 1e-6
CHANNELS, INNER = (2 * K_HEADS + V_HEADS) * D, V_HEADS * D


class Layer:
    """The layer's weights and the descriptors of its operators."""

    def __init__(self, seed=0):
        mat = lambda fmt, n, k, i: workloads.build_matrix(fmt, n, k, seed, synth.stream_id("test", synth.ROLE_W, 720 + i))  # noqa: E731
        self.qkv, self.z, self.out = mat("pq2_0", CHANNELS, HIDDEN, 0), mat("pq2_0", INNER, HIDDEN, 1), mat("pq2_0", HIDDEN, INNER, 2)
        self.ab, self.head = mat("q8_0", 2 * V_HEADS, HIDDEN, 3), mat("q8_0", VOCAB, HIDDEN, 4)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
        self.conv = kq.CausalConv(rand(CHANNELS, WIDTH) - 0.5)
        self.rule = kq.GatedDelta(K_HEADS, V_HEADS, D, torch.log(1 + 15 * rand(V_HEADS)), rand(V_HEADS) - 5, eps=EPS)
        self.norm, self.head_norm = kq.RMSNorm(1, HIDDEN, 0.5 + rand(HIDDEN), EPS), kq.RMSNorm(V_HEADS, D, 0.5 + rand(D), EPS)

    def project(self, W, x):
        """x [tokens, k] -> [tokens, n], at most 64 rows a call."""
        y = torch.empty(x.shape[0], W.n, device="cuda")
        ws = torch.empty(max(kq.kq_gemv_workspace_bytes(W, min(64, x.shape[0])), 16), dtype=torch.uint8, device="cuda")
        for i in range(0, x.shape[0], 64):
            m = min(64, x.shape[0] - i)
            kq.kq_gemm_small_m(W, x[i: i + m], m, y[i: i + m], ws)
        return y

    def step(self, x, residual, q_start, kv_len, slot, conv_state, state, most):
        """The layer's output for x [tokens, hidden]; returns (output, what the delta rule's part saw, its gated heads)."""
        t, r = x.shape[0], slot.numel()
        normed = torch.empty_like(x)
        kq.kq_rms_norm(self.norm, x[:, None], normed[:, None], residual=residual[:, None])
        qkv, z, ab = self.project(self.qkv, normed), self.project(self.z, normed), self.project(self.ab, normed)
        mixed = torch.empty_like(qkv)
        kq.kq_causal_conv(self.conv, qkv, q_start, kv_len, slot, conv_state, mixed)
        heads = mixed.unflatten(1, (-1, D))
        o = torch.empty(t, V_HEADS, D, device="cuda")
        n = kq.kq_gdn_workspace_bytes(self.rule, o.dtype, r, t, most)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        kq.kq_gdn(self.rule, heads[:, :K_HEADS], heads[:, K_HEADS: 2 * K_HEADS], heads[:, 2 * K_HEADS:], ab[:, :V_HEADS],
                  ab[:, V_HEADS:], q_start, kv_len, slot, state, o, most, ws=ws)
        kq.kq_rms_norm(self.head_norm, o, o, gate=z.unflatten(1, (V_HEADS, D)))
        return self.project(self.out, o.flatten(1)), (qkv, z, ab), o


class Fp64:
    """Convolution, delta rule and gated norm of one request at a time, in FP64."""

    def __init__(self, layer, requests):
        self.layer = layer
        self.past = torch.zeros(requests, WIDTH - 1, CHANNELS, dtype=torch.float64, device="cuda")
        self.state = torch.zeros(requests, V_HEADS, D, D, dtype=torch.float64, device="cuda")

    def step(self, r, qkv, z, ab):
        a = self.layer
        x = torch.cat((self.past[r], qkv.double()))
        self.past[r] = x[-(WIDTH - 1):]
        y = sum(x[j: j + len(qkv)] * a.conv.weight[:, j].double() for j in range(WIDTH))
        y = (y * torch.sigmoid(y)).unflatten(1, (-1, D))
        unit = lambda t: t / torch.sqrt(t.pow(2).sum(-1, keepdim=True) + EPS)  # noqa: E731
        group = V_HEADS // K_HEADS
        q = (unit(y[:, :K_HEADS]) * D ** -0.5).repeat_interleave(group, 1)
        k, v = unit(y[:, K_HEADS: 2 * K_HEADS]).repeat_interleave(group, 1), y[:, 2 * K_HEADS:]
        fade = torch.exp(-torch.exp(a.rule.a_log.double()) * torch.nn.functional.softplus(ab[:, :V_HEADS].double() + a.rule.dt_bias.double()))
        beta = torch.sigmoid(ab[:, V_HEADS:].double())
        s, out = self.state[r], []
        for t in range(len(qkv)):
            s = s * fade[t][:, None, None]
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", s, k[t]))
            s = s + k[t][:, :, None] * u[:, None]
            out.append(torch.einsum("hkv,hk->hv", s, q[t]))
        self.state[r] = s
        o, g = torch.stack(out), z.double().unflatten(1, (V_HEADS, D))
        o = o / torch.sqrt(o.pow(2).mean(-1, keepdim=True) + EPS) * a.head_norm.weight.double()
        return o * g * torch.sigmoid(g)


def main(requests=4, prompt=70, steps=4, seed=0):
    """Returns the last step's relative error against FP64."""
    layer, check = Layer(seed), None
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    slot, check = ints(list(range(requests))[::-1]), Fp64(layer, requests)
    conv_state = torch.empty(requests, WIDTH - 1, CHANNELS, device="cuda")  # a request that begins takes them as zeros
    state = torch.empty(requests, V_HEADS, D, D, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    length = [0] * requests
    for step in range(steps + 1):
        new = [prompt + i for i in range(requests)] if step == 0 else [1] * requests
        start = [sum(new[:r]) for r in range(requests + 1)]
        length = [n + m for n, m in zip(length, new)]
        x, residual = (torch.randn(sum(new), HIDDEN, generator=gen, device="cuda") for _ in range(2))
        y, seen, heads = layer.step(x, residual, ints(start), ints(length), slot, conv_state, state, max(new))
        want = torch.cat([check.step(r, *(t[start[r]: start[r + 1]] for t in seen)) for r in range(requests)])
    last = y[[s - 1 for s in start[1:]]]
    kq.kq_rms_norm(layer.norm, last[:, None], last[:, None])
    logits = layer.project(layer.head, last)
    token, prob = torch.empty(requests, dtype=torch.int32, device="cuda"), torch.empty(requests, device="cuda")
    kq.kq_sample(logits, torch.rand(requests, generator=gen, device="cuda"), token, prob,
                 temperature=torch.full((requests,), 0.8, device="cuda"), top_k=torch.full((requests,), 40, dtype=torch.int32, device="cuda"))
    if kq.kq_device_status() != kq.KQ_OK:
        raise RuntimeError("device status not ok: " + kq.lib().kq_last_error().decode())
    error = float((heads.double() - want).norm() / want.norm())
    print(f"{requests} requests of {length} tokens: heads within {error:.2e} of FP64; tokens {token.tolist()}")
    return error


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--requests", type=int, default=4)
    p.add_argument("--prompt", type=int, default=70)
    p.add_argument("--steps", type=int, default=4)
    a = p.parse_args()
    sys.exit(0 if main(a.requests, a.prompt, a.steps) < 1e-5 else 1)
