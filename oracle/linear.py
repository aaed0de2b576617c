"""CPU oracle of linear attention with a decay and of group norm with an activation: their definitions in 64 bits.

Test infrastructure only; it shares no code with the library. linear_attention walks the tokens as it is defined, in torch
float64 on the CPU, so that autograd gives the formula's gradients.
"""

from __future__ import annotations

import torch


def linear_attention(state, k, v, log_decay, q, scale, valid=None):
    """(readings [P, T, Hv, V], final state [P, Hv, K, V]) of float64 inputs; state None: zeros; log_decay [Hv] or
    [P, T, Hv]. Padding tokens (t >= valid[p]) leave the state alone and read 0, whatever they hold."""
    P, T, Hk, K = k.shape
    Hv, V = v.shape[2:]
    group = Hv // Hk
    outs, finals = [], []
    for p in range(P):
        S = torch.zeros(Hv, K, V, dtype=torch.float64) if state is None else state[p]
        n = T if valid is None else max(0, min(int(valid[p]), T))
        rows = []
        for t in range(n):
            g = log_decay if log_decay.dim() == 1 else log_decay[p, t]
            kt, qt = (x[p, t].repeat_interleave(group, 0) for x in (k, q))
            S = torch.exp(g)[:, None, None] * S + kt[:, :, None] * v[p, t][:, None, :]
            rows.append(scale * (qt[:, :, None] * S).sum(1))
        rows += [torch.zeros(Hv, V, dtype=torch.float64)] * (T - n)
        outs.append(torch.stack(rows) if T else torch.zeros(0, Hv, V, dtype=torch.float64))
        finals.append(S)
    return torch.stack(outs), torch.stack(finals)


def group_norm(x, groups, weight=None, bias=None, activation=None, eps=1e-5, valid=None):
    """(y, mean, rstd) of a float64 x [N, L, C]; rows at and past valid[n] do not count and give 0."""
    N, L, C = x.shape
    D = C // groups
    ys, means, rstds = [], [], []
    for n in range(N):
        rows = L if valid is None else max(0, min(int(valid[n]), L))
        live = x[n, :rows].reshape(rows, groups, D)
        m = live.sum((0, 2)) / max(1, rows * D)
        d = live - m[:, None]
        r = 1.0 / torch.sqrt((d * d).sum((0, 2)) / max(1, rows * D) + eps)
        z = (d * r[:, None]).reshape(rows, C)
        if weight is not None:
            z = z * weight
        if bias is not None:
            z = z + bias
        if activation == "silu":
            z = z / (1.0 + torch.exp(-z))
        elif activation == "gelu":
            z = 0.5 * z * torch.erfc(-z * 0.5 ** 0.5)
        ys.append(torch.cat([z, torch.zeros(L - rows, C, dtype=torch.float64)]))
        means.append(m)
        rstds.append(r)
    return torch.stack(ys), torch.stack(means), torch.stack(rstds)
