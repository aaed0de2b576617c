"""Linear attention as the first call of a process, and captured as its first one after another operator's: one-time setup."""

import subprocess
import sys

import pytest

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu

SCRIPT = """
import sys, torch
import chunked_sparse_delta_amd as sdm
gen = torch.Generator().manual_seed(0)
k, v, q = (torch.randn((1, 300, 2, 64), generator=gen).cuda() for _ in range(3))
g = -torch.rand(2, generator=gen).cuda()
go = torch.randn((1, 300, 2, 64), generator=gen).cuda()

def work():
    out = sdm.linear_attention_fwd(None, k, v, g, q)
    return [out, *sdm.linear_attention_bwd(None, k, v, g, q, go).values(), sdm.linear_attention_step(torch.zeros(1, 2, 64, 64, device="cuda"), k[:, :1], v[:, :1], g, q[:, :1])]

if sys.argv[1] == "captured":
    sdm.gated_delta_step(torch.zeros(1, 2, 64, 64, device="cuda"), k[:, :1], v[:, :1], torch.ones(1, 1, 2, device="cuda"), g.view(1, 1, 2), q[:, :1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, work()))
else:
    first, second = work(), work()
    assert all(torch.equal(a, b) for a, b in zip(first, second))
print("fine")
"""


@pytest.mark.parametrize("how", ["first", "captured"])
def test_first_call(gpu, how):
    done = subprocess.run([sys.executable, "-c", SCRIPT, how], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert done.returncode == 0 and done.stdout.endswith("fine\n"), done.stderr[-2000:]
