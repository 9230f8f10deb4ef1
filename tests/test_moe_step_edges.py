"""The serving step's operators at the borders of their checks, on the host; none of these calls reaches a device."""
import threading

import pytest
import torch

from fp8_block_scaled_sa_amd import DGError, ops

MISALIGNED = 3


@pytest.fixture
def host_tensors():
    ops._binding().any_device(True)
    yield
    ops._binding().any_device(False)


def calls():
    """A valid call of each operator on host tensors."""
    code = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x, r, y = torch.zeros((2, 256)), torch.zeros((2, 256)), torch.zeros((2, 256), dtype=torch.bfloat16)
    return (lambda: ops.dg_fp8_rmsnorm_quantize_1x128(x, torch.ones(256), residual=r, residual_out=r, y=y),
            lambda: ops.dg_moe_gate_topk(torch.zeros((2, 8)), 2),
            lambda: ops.dg_fp8_moe_layer(code(2, 256), torch.ones(2, 2), code(3, 256, 256), torch.ones(3, 2, 2),
                                         code(3, 256, 128), torch.ones(3, 2, 1),
                                         torch.zeros((2, 2), dtype=torch.int32), torch.ones(2, 2), code(65536)))


def test_host_addresses_never_reach_the_library(host_tensors):
    """With the switch that lets tests pass host tensors to an entry point of their own, the library's own entry
    points refuse them before the device is asked for anything."""
    for call in calls():
        with pytest.raises(DGError) as e:
            call()
        assert e.value.status == MISALIGNED


def test_host_tensors_are_one_threads_affair(host_tensors):
    seen = []

    def other():
        for call in calls():
            try:
                call()
            except Exception as e:
                seen.append(str(e))
    t = threading.Thread(target=other)
    t.start()
    t.join()
    assert len(seen) == 3 and all("must be a device tensor" in s for s in seen)
