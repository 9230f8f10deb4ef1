import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")


# Tests without the gpu marker that make valid calls with made-up addresses. They
# end at the library's device check on a host without a device; where there is
# one, the call would launch its kernel on unmapped memory.
NO_DEVICE_TESTS = {
    "test_abi.py::test_quantize_accepts_both_scale_layouts_up_to_the_device_check",
    "test_abi.py::test_gather_quantize_all_padding_needs_no_input",
    "test_moe_step_abi.py::test_norm_accepted_and_empty",
    "test_moe_step_abi.py::test_gate_accepted_and_empty",
    "test_moe_step_abi.py::test_layer_accepted_and_empty",
    "test_attention_step_abi.py::test_write_accepted_and_empty",
    "test_attention_step_abi.py::test_read_accepted_and_empty",
    "test_attention_step_abi.py::test_attention_accepted_and_empty",
    "test_attention_step_edges.py::test_write_in_place_accepted",
    "test_attention_step_edges.py::test_write_accepts_halves_of_one_tensor",
}


def pytest_collection_modifyitems(items):
    made_up = [i for i in items if i.nodeid.split("[")[0].split("/")[-1] in NO_DEVICE_TESTS]
    if not made_up:
        return
    import torch
    if torch.cuda.device_count():  # without initialising it
        for item in made_up:
            item.add_marker(pytest.mark.skip(reason="valid calls with made-up addresses: only without a device"))


@pytest.fixture(scope="session")
def gpu_device():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    return torch.device("cuda:0")
