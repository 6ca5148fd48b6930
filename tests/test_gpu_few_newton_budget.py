"""The layer for few tokens and the experts' weights' update under an SM budget
(ep_set_num_sms): while a call runs on its SMs, all others are free."""
import time

import pytest
import torch

from combine_get_dispatch_gb300 import ep
from test_gpu_expert_budget import budget  # noqa: F401
from test_gpu_ll import _hold_lib, ctypes_stream

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
HOLD = 20   # ms


@pytest.fixture
def hold_lib(tmp_path):
    return _hold_lib(tmp_path)


def others_are_free(lib, n, call):
    """Kernels that take a whole SM each, one for every SM beside the n of the budget, all run at once while `call`
    (several times as long) runs: together they take as long as one."""
    ctas = torch.cuda.get_device_properties(0).multi_processor_count - n
    stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(stream):
        call()   # loads the kernels
    assert lib.hold_sms(ctas, 220 * 1024, 1000, ctypes_stream(side)) == 0
    torch.cuda.synchronize()
    ended, a, b = torch.cuda.Event(), torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(stream):
        call()
        ended.record()
    time.sleep(0.03)   # (norm and first X are over by then, and the products have begun)
    with torch.cuda.stream(side):
        a.record()
        assert lib.hold_sms(ctas, 220 * 1024, HOLD * 1_000_000, ctypes_stream(side)) == 0
        b.record()
    b.synchronize()
    assert not ended.query(), "the call was over before the SMs were free again"
    torch.cuda.synchronize()
    assert a.elapsed_time(b) < 1.8 * HOLD, f"{a.elapsed_time(b)} ms for {HOLD}"


@pytest.mark.parametrize("n", [2, 8])
def test_update_leaves_the_other_sms(budget, hold_lib, n):  # noqa: F811
    """Five steps of three products, of some 10 ms each."""
    count = 24 * n
    g = torch.randn((count, 1416, 2048), device="cuda").bfloat16()
    m, w, ws = torch.zeros_like(g, dtype=torch.float32), g.float(), ep.alloc_orthogonalize_workspace(g.shape)
    budget(n)
    others_are_free(hold_lib, n, lambda: ep.ep_muon_update(g, m, w, g, [QUINTIC] * 5, ws, lr=0.01))


@pytest.mark.parametrize("n", [2])
def test_small_updates_leave_the_other_sms(budget, hold_lib, n):  # noqa: F811
    """Calls of one launch, one behind the other."""
    g = torch.randn((1024, 128, 256), device="cuda").bfloat16()
    out, ws = torch.empty_like(g), ep.alloc_orthogonalize_workspace(g.shape)
    budget(n)
    others_are_free(hold_lib, n, lambda: [ep.ep_orthogonalize(g, [QUINTIC] * 5, out, ws) for _ in range(8)])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_few_leave_the_other_sms(budget, hold_lib, kind):  # noqa: F811
    from test_gpu_few import call, make
    s = make(1, 1, 16, 8, 32, 4096, 1408, kind)
    out, ws = torch.empty_like(s["x"]), ep.alloc_moe_few_workspace(1, 16, 8, 32, 1408)
    budget(2)
    others_are_free(hold_lib, 2, lambda: [call(s, "silu", out=out, workspace=ws) for _ in range(20)])
