"""gated_delta_fwd on sequences that it walks in segments at once (few states, many chunks): what only such calls meet.

How many segments a call takes shows in its workspace: beyond what every call needs it holds, per segment, each head's
start state [KP, VP] and map [KP, KP] in float32. Every test asks for it, so that none runs unsegmented unseen.
"""

import pytest
import torch

from oracle import dense as oracle
from tests.test_gpu_delta import NAMES, close, f64_of, gpu_of, make

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def up(x, n):
    return (x + n - 1) // n * n


def segments(P, T, Hk, Hv, K, V, dtype):
    """(segments of a call, tokens of a segment), from its workspace."""
    import chunked_sparse_delta_amd as sdm
    b16 = dtype == torch.bfloat16
    KP, VP = 64 if K <= 64 else 128 if K <= 128 else 256, up(V, 16)
    C = 64 if b16 and K <= 128 else 32
    Nt = up(T, C) // C
    blocks = 3 if C == 64 else 1                    # of X and of P, 32 x 32 in float32, and 1 KB of gates
    base = up(P * Hv * Nt * (2 * blocks * 4096 + 1024), 256) + 2 * up(P * T * Hk * KP * (2 if b16 else 6), 256) \
        + up(P * T * Hv * up(V, 8) * (2 if b16 else 4), 256)
    left = sdm.gated_delta_workspace_bytes(P, T, Hk, Hv, K, V, dtype) - base
    each = P * Hv * KP * (VP + KP) * 4
    assert left % each == 0
    n = left // each or 1
    return n, up(Nt, n) // n * C


# P, T, Hk, Hv, K, V, dtype, valid: the last active segment of a ragged stream is one token long, one chunk, empty, or whole
CASES = [
    (1, 2050, 8, 16, 128, 128, "bf16", None), (1, 2111, 1, 2, 40, 20, "bf16", (1793,)),
    (3, 2112, 1, 1, 128, 64, "bf16", (449, 0, 2112)), (2, 700, 1, 1, 128, 128, "f32", (161, 699)),
    (1, 1500, 1, 3, 64, 64, "f32", None), (2, 1100, 1, 1, 200, 33, "bf16", (1100, 193)),
]


@pytest.mark.parametrize("busy", [False, True])
@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,valid", CASES)
def test_state_advanced_in_place(gpu, P, T, Hk, Hv, K, V, dtype, valid, busy):
    """The call's default, the state advanced in place, gives the bits that it gives with the final state elsewhere, on an idle
    device and beside another stream's work."""
    import chunked_sparse_delta_amd as sdm
    assert segments(P, T, Hk, Hv, K, V, DT[dtype])[0] > 2
    g = gpu_of(make(P, T, Hk, Hv, K, V, DT[dtype], seed=11), gpu)
    vt = None if valid is None else torch.tensor(valid, dtype=torch.int32, device=gpu)
    start, end = g["state"].clone(), torch.empty_like(g["state"])
    want = sdm.gated_delta_fwd(*(g[n] for n in NAMES), valid_tokens=vt, state_out=end)
    assert torch.equal(g["state"], start)
    side, a = torch.cuda.Stream(), torch.randn(2048, 2048, device=gpu)
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        state = start.clone()
        if busy:
            with torch.cuda.stream(side):
                for _ in range(8):
                    torch.mm(a, a)
        out = sdm.gated_delta_fwd(state, *(g[n] for n in NAMES[1:]), valid_tokens=vt)
        assert torch.equal(out, want) and torch.equal(state, end)
    torch.cuda.synchronize()


@pytest.mark.parametrize("decay", [0.3, 0.0])
@pytest.mark.parametrize("P,T,Hk,Hv,K,V,dtype,valid", [
    (3, 2112, 1, 1, 128, 64, "bf16", (449, 0, 2112)), (2, 700, 1, 1, 128, 128, "f32", (161, 0)),
    (4, 1400, 1, 2, 72, 24, "bf16", (0, 1, 0, 321)), (2, 1600, 2, 2, 33, 70, "f32", (1600, 0)),
])
def test_streams_of_few_or_no_tokens(gpu, P, T, Hk, Hv, K, V, dtype, valid, decay):
    """Streams that end in the first segment, at a segment's first token, or before their first token, beside whole ones, against the
    token loop in 64 bits."""
    import chunked_sparse_delta_amd as sdm
    assert segments(P, T, Hk, Hv, K, V, DT[dtype])[0] > 2
    x = make(P, T, Hk, Hv, K, V, DT[dtype], seed=12, decay=decay)
    y, g = f64_of(x), gpu_of(x, gpu)
    want, final = oracle.gated_delta(*(y[n] for n in NAMES), K ** -0.5, valid)
    end = torch.full((P, Hv, K, V), float("nan"), device=gpu)
    out = sdm.gated_delta_fwd(*(g[n] for n in NAMES), valid_tokens=torch.tensor(valid, dtype=torch.int32, device=gpu), state_out=end)
    close(out, want, "readings", DT[dtype])
    close(end, final, "state")
    for p in range(P):
        assert (out[p, valid[p]:] == 0).all()
        assert valid[p] > 0 or torch.equal(end[p], g["state"][p])


@pytest.mark.parametrize("P,T,Hv,K,V,dtype", [(1, 1500, 2, 64, 64, "f32"), (2, 1500, 2, 128, 40, "bf16")])
def test_graph(gpu, P, T, Hv, K, V, dtype):
    """A captured call in segments replays with the eager call's bits, other work in between; the state advances with every replay."""
    import chunked_sparse_delta_amd as sdm
    assert segments(P, T, 1, Hv, K, V, DT[dtype])[0] > 2
    g = gpu_of(make(P, T, 1, Hv, K, V, DT[dtype], seed=13), gpu)
    state, rest = g["state"].clone(), [g[n] for n in NAMES[1:]]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sdm.gated_delta_fwd(state, *rest)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        got = sdm.gated_delta_fwd(state, *rest)
    state.copy_(g["state"])
    mine = g["state"].clone()
    for seed in range(4):
        torch.cuda.synchronize()
        new = gpu_of(make(P, T, 1, Hv, K, V, DT[dtype], seed=seed), gpu)
        for n in NAMES[1:]:
            g[n].copy_(new[n])
        want = sdm.gated_delta_fwd(mine, *rest)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(state, mine)
