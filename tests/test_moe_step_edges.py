"""The serving step's operators at the borders of their checks, on the host; none of these calls reaches a device."""
import contextlib
import inspect
import threading

import pytest
import torch

from fp8_block_scaled_sa_amd import DGError, ops
from tests.test_moe_step_abi import IDS, MISALIGNED, S, SHAPE, UNSUPPORTED, gate, norm


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


class StandIn:
    """In the place of a device tensor."""
    is_cuda = True

    def __init__(self):
        self.recorded = []

    def record_stream(self, stream):
        self.recorded.append(stream)


CALLS = sorted(n for n in vars(ops) if n.startswith("dg_") and "stream" in inspect.signature(getattr(ops, n)).parameters)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("positional", [False, True])
def test_every_call_with_a_stream_is_made_on_it(monkeypatch, name, positional):
    routed = []
    monkeypatch.setattr(ops, "_call_on", lambda stream, call, *args: routed.append((stream, call.__name__, args)))
    call = getattr(ops, name)
    parameters = list(inspect.signature(call).parameters.values())
    assert parameters[-1].name == "stream"
    args = [StandIn() if p.default is p.empty else p.default for p in parameters[:-1]]
    call(*args, 7) if positional else call(*args, stream=7)
    assert routed == [(7, name, tuple(args))]


def test_a_call_on_another_stream_allocates_there(monkeypatch):
    """The stream is torch's current one while the call runs; the one that was current is recorded on what the call
    returns, but not on what the caller gave it."""
    current = ["here"]

    @contextlib.contextmanager
    def enter(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: "side %d" % handle)
    made, given = StandIn(), StandIn()

    def call(*args):
        assert current[-1] == "side 7"
        return made, args[0], None

    assert ops._call_on(7, call, given, 3) == (made, given, None)
    assert current == ["here"] and made.recorded == ["here"] and given.recorded == []
    assert ops._call_on(7, lambda: made) is made and made.recorded == ["here", "here"]



@pytest.mark.parametrize("K,most", [(128, 2 ** 26 - 4), (1024, 2 ** 26 - 4), (1152, 2 ** 24 - 1), (8192, 2 ** 24 - 1),
                                    (8320, 2 ** 22 - 1), (65536, 2 ** 22 - 1)])
def test_norm_takes_the_rows_that_a_launch_can_hold(K, most):
    """The largest M passes the check of sizes (and is refused for its misaligned S), one more does not."""
    for M, status in ((most, MISALIGNED), (most + 1, UNSUPPORTED)):
        assert norm(M=M, K=K, ldx=K, ldr=K, ldro=K, ldy=K, ldq=K, s_m=K // 128, s_kb=1, S=S + 2) == status


def test_gate_takes_the_tokens_that_a_launch_can_hold():
    for T, status in ((2 ** 28 - 16, MISALIGNED), (2 ** 28 - 15, UNSUPPORTED)):
        assert gate(T=T, ids=IDS + 2) == status


@pytest.mark.parametrize("top_k", [9, 10 ** 12, 2 ** 62])
def test_gate_refuses_more_slots_than_experts_before_it_allocates_them(host_tensors, top_k):
    with pytest.raises(DGError) as e:
        ops.dg_moe_gate_topk(torch.zeros((2, 8)), top_k)
    assert e.value.status == SHAPE
