"""Plain 64-bit implementations of the delta layers' operators and of sampling (torch on the CPU)."""
import math

import torch


def sigmoid(x):
    e = torch.exp(-x.abs())
    return torch.where(x >= 0, 1 / (1 + e), e / (1 + e))


def rms_norm(x, residual, gate, weight, eps):
    """(y in 64 bits, the sum as the type holds it or None) of rows [..., dim]."""
    s = x.double()
    kept = None
    if residual is not None:
        kept = (x.double() + residual.double()).float().to(x.dtype) if x.dtype != torch.float32 else x + residual
        s = kept.double()
    y = s / torch.sqrt(s.pow(2).sum(-1, keepdim=True) / s.shape[-1] + eps)
    if weight is not None:
        y = y * weight.double()
    if gate is not None:
        y = y * gate.double() * sigmoid(gate.double())
    return y, kept


def conv(x, weight, bias, silu, q_start, kv_len, slot, state):
    """(y, state) of the requests that are computed; rows of others are NaN."""
    width = weight.shape[1]
    y = torch.full(x.shape, math.nan, dtype=torch.float64)
    state = state.double().clone()
    for r in range(len(slot)):
        lo, hi = q_start[r], q_start[r + 1]
        if hi == lo or slot[r] < 0:
            continue
        before = state[slot[r]] * (0 if kv_len is not None and kv_len[r] == hi - lo else 1)
        rows = torch.cat((before, x[lo:hi].double()))
        s = sum(rows[j: j + hi - lo] * weight[:, j].double() for j in range(width))
        if bias is not None:
            s = s + bias.double()
        y[lo:hi] = s * sigmoid(s) if silu else s
        state[slot[r]] = rows[-(width - 1):]
    return y, state


def gdn(q, k, v, a, b, a_log, dt_bias, unit, eps, scale, q_start, kv_len, slot, state):
    """The rule token by token; rows of requests that are not computed are NaN."""
    q, k, v, a, b = (t.double() for t in (q, k, v, a, b))
    hk, hv, d = k.shape[1], v.shape[1], v.shape[2]
    if unit:
        q = q / torch.sqrt(q.pow(2).sum(-1, keepdim=True) + eps)
        k = k / torch.sqrt(k.pow(2).sum(-1, keepdim=True) + eps)
    q = (q * scale).repeat_interleave(hv // hk, 1)
    k = k.repeat_interleave(hv // hk, 1)
    if a_log is not None:
        x = a + dt_bias.double()
        a = -torch.exp(a_log.double()) * (x.clamp(min=0) + torch.log1p(torch.exp(-x.abs())))
        b = sigmoid(b)
    out = torch.full(v.shape, math.nan, dtype=torch.float64)
    state = state.double().clone()
    for r in range(len(slot)):
        lo, hi = q_start[r], q_start[r + 1]
        if hi == lo or slot[r] < 0:
            continue
        s = state[slot[r]] * (0 if kv_len is not None and kv_len[r] == hi - lo else 1)
        for t in range(lo, hi):
            s = s * torch.exp(a[t])[:, None, None]
            u = b[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", s, k[t]))
            s = s + k[t][:, :, None] * u[:, None, :]
            out[t] = torch.einsum("hkv,hk->hv", s, q[t])
        state[slot[r]] = s
    return out, state


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob, slack) of one row: slack is how far u, or the mass at the kept set's border, is from where another token
    would come out, as a share of the whole."""
    x = logits.double()
    if torch.isnan(x).any() or x.max() == -math.inf:
        return -1, 0.0, 1.0
    order = torch.sort(x, descending=True, stable=True).indices
    if temperature == 0:
        return int(order[0]), 1.0, 1.0
    top = x[order[0]]
    w = (x == top).double() if math.isinf(float(top)) else torch.exp((x - top) / temperature)
    if top_k > 0:
        order = order[:top_k]
    slack = 1.0
    if top_p < 1:
        sums = torch.cumsum(w[order], 0)
        target = top_p * sums[-1]
        n = max(1, int((sums - w[order] < target).sum()))
        slack = min(slack, float((sums - target).abs().min() / sums[-1]))
        order = order[:n]
    order = torch.cat((order[:1], order[1:][w[order[1:]] >= min_p]))
    order = order.sort().values
    sums = torch.cumsum(w[order], 0)
    at = min(max(u, 0.0), 1.0) * sums[-1]
    slack = min(slack, float((sums - at).abs()[:-1].min() / sums[-1]) if len(order) > 1 else 1.0)
    i = min(int((sums <= at).sum()), len(order) - 1)
    while w[order[i]] == 0:
        i -= 1
    return int(order[i]), float(w[order[i]] / sums[-1]), slack
