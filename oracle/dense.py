"""CPU oracle of the dense gated delta rule and of layer norm: their definitions in 64 bits.

Test infrastructure only; it shares no code with the library. gated_delta walks the tokens as
the rule is defined, in torch float64 on the CPU, so that autograd gives the formula's
gradients.
"""

from __future__ import annotations

import torch


def gated_delta(state, k, v, beta, log_decay, q, scale, valid=None):
    """(readings [P, T, Hv, V], final state [P, Hv, K, V]) of float64 inputs; state None: zeros.
    Padding tokens (t >= valid[p]) leave the state alone and read 0, whatever they hold."""
    P, T, Hk, K = k.shape
    Hv, V = v.shape[2:]
    group = Hv // Hk
    S = torch.zeros(P, Hv, K, V, dtype=torch.float64) if state is None else state
    outs = []
    for t in range(T):
        rows, new = [], []
        for p in range(P):
            if valid is not None and t >= int(valid[p]):
                rows.append(torch.zeros(Hv, V, dtype=torch.float64))
                new.append(S[p])
                continue
            kt, qt = (x[p, t].repeat_interleave(group, 0) for x in (k, q))
            decayed = torch.exp(log_decay[p, t])[:, None, None] * S[p]
            u = beta[p, t][:, None] * (v[p, t] - torch.einsum("hk,hkv->hv", kt, decayed))
            s = decayed + kt[:, :, None] * u[:, None, :]
            rows.append(scale * torch.einsum("hk,hkv->hv", qt, s))
            new.append(s)
        S = torch.stack(new)
        outs.append(torch.stack(rows))
    out = torch.stack(outs, 1) if T else torch.zeros(P, 0, Hv, V, dtype=torch.float64)
    return out, S


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis of a float64 [rows, cols] x."""
    n = x.shape[-1]
    mean = x.sum(-1) / n
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).sum(-1) / n + eps)
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mean, rstd
