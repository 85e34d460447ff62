"""The first call of each kernel of the 8-bit products in a process, while a graph is captured."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

# (tile rows, features, shares of K), rows, features, columns, by index
CALLS = [((16, 128, 1), 3, 300, 144, 0), ((16, 128, 8), 3, 512, 4096, 0),
         ((16, 128, 8), 4, 512, 4096, 1), ((32, 128, 8), 20, 387, 2064, 0),
         ((32, 128, 8), 12, 387, 2064, 1), ((64, 128, 4), 140, 1000, 2064, 0),
         ((64, 128, 1), 2500, 387, 144, 1), ((128, 128, 1), 2500, 387, 144, 0),
         ((128, 256, 1), 1500, 1537, 144, 0), ((128, 256, 1), 2600, 2816, 144, 1),
         ((256, 256, 1), 1500, 1537, 656, 0), ((256, 256, 1), 700, 5003, 4112, 0)]

PROGRAM = """
import sys, torch
import block_diffusion_speculative_02_gb300 as dfl
space = dfl.alloc_fp8_workspace()
for call in sys.argv[1:]:
    r, c, s, m, n, k, index = map(int, call.split(","))
    assert dfl.dflash_fp8_plan(m, n, k, index, bool(index)) == (r, c, s), call
    x, xs = dfl.alloc_fp8_rows(m, k)
    w, ws = dfl.alloc_fp8_weight(1, n, k)
    x.copy_(torch.eye(m, k)), xs.fill_(1), ws.fill_(1)
    w.copy_((torch.arange(n * k) % 17).view(1, n, k).float())
    start = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    rows = torch.arange(m, dtype=torch.int32, device="cuda")
    out = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if index:
            dfl.dflash_fp8_grouped(x, xs, w, ws, start, rows, out, space)
        else:
            dfl.dflash_fp8_linear(x, xs, w[0], ws[0], out, space)
    graph.replay()
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(space) == 0, call
    assert torch.equal(out[:k].float(), w[0].float().T[:m]) and not bool(out[k:].any()), call
print("ran", len(sys.argv) - 1)
"""


@pytest.mark.parametrize("order", [1, -1])
def test_first_use_of_every_kernel_inside_a_capture(order):
    """(Each compiled kernel has work of its own to do once: limits, and for tiles a query.)"""
    calls = [",".join(map(str, (*plan, *size))) for plan, *size in CALLS[::order]]
    done = subprocess.run([sys.executable, "-c", PROGRAM, *calls], capture_output=True, text=True,
                          timeout=300, cwd=Path(__file__).resolve().parents[1])
    assert done.returncode == 0, done.stderr[-2000:]
    assert f"ran {len(CALLS)}" in done.stdout
