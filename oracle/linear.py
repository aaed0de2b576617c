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
