"""Every wait on a barrier is one of the forms that the wait probe lets run out (moe_wait_timeout_probe), or is bounded by the
clock beside it."""
import os
import re
import time

import pytest
import torch

import bit_quantized_expert_gb300 as moe


def test_no_kernel_has_a_wait_of_its_own():
    csrc = os.path.join(moe.PKG_DIR, "csrc")
    for name in sorted(os.listdir(csrc)):
        if not name.endswith((".cu", ".cuh")) or name == "common.cuh":
            continue
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert "mbarrier.try_wait" not in text and "mbarrier.test_wait" not in text, name
        for m in re.finditer(r"mbar_try_wait\(", text):
            line = text[text.rindex("\n", 0, m.start()):text.index("\n", m.end())]
            assert "while (!mbar_try_wait(" in line and "clock64() - " in line, (name, line)


@pytest.mark.gpu
@pytest.mark.parametrize("limit", [1, 3000, 2_000_000, 200_000_000])
def test_the_waits_run_out_in_time(limit):
    """Three waits of about `limit` cycles each (at 1 to 2.1 GHz), the counted one by the time that a try takes."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    moe.wait_timeout_probe(ws, 1)
    torch.cuda.synchronize()
    t = time.perf_counter()
    moe.wait_timeout_probe(ws, limit)
    torch.cuda.synchronize()
    assert time.perf_counter() - t < 0.1 + 10 * limit * 1e-9
    assert moe.read_error_flags(ws) == moe.ERR_WAIT_TIMEOUT
