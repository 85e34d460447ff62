"""Waits of the 8-bit products that run out, without a fault: the self-test's kernel goes through
the waits on two barriers and the hand-over between a watching warp and those it watches for, with
the device functions that the products use."""
import re
import time
from pathlib import Path

import pytest
import torch

CSRC = Path(__file__).resolve().parents[1] / "block_diffusion_speculative_02_gb300" / "csrc"


def test_a_wait_that_gave_up_is_decided_by_the_whole_warp():
    """wait_on gives each lane its own answer and needs the whole warp: wherever one wait
    decides whether another is entered, the answer is made the warp's first."""
    for path in sorted(CSRC.glob("fp8*")):
        text = path.read_text()
        assert not re.search(r"wait_on\([^;]*?\)\s*&&\s*\(?wait_on\(", text), path.name
        for m in re.finditer(r"(?<![\w:])wait_on\(", text):
            assert text[:m.start()].endswith("all("), (path.name, text[m.start() - 40:m.start() + 40])


@pytest.mark.gpu
def test_waits_on_two_barriers_and_the_hand_over_end():
    import block_diffusion_speculative_02_gb300 as dfl
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        dfl.dflash.dflash_selftest_wait(True, ws)
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(ws) == 0
    t0 = time.perf_counter()
    dfl.dflash.dflash_selftest_wait(False, ws)
    torch.cuda.synchronize()
    assert 0.9 <= time.perf_counter() - t0 < 5.0
    assert dfl.dflash_read_status(ws) == dfl.dflash.STATUS_BITS["timeout"]
    # the products run as before
    x, xs = dfl.alloc_fp8_rows(600, 512)
    w, wscale = dfl.alloc_fp8_weight(1024, 512)
    x.copy_(torch.ones(600, 512)), w.copy_(torch.ones(1024, 512))
    xs.fill_(1), wscale.fill_(1)
    out, space = torch.empty(600, 1024, dtype=torch.bfloat16, device="cuda"), dfl.alloc_fp8_workspace()
    dfl.dflash_fp8_linear(x, xs, w, wscale, out, space)
    assert bool((out == 512).all()) and dfl.dflash_read_status(space) == 0
