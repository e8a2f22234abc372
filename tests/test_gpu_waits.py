"""The bounded wait's limit, as a user of a small one sees it."""
from __future__ import annotations

import pytest
import torch

import moe_expert_layer_07_gb300 as moe

from _gpu_common import build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return build_library()


@pytest.mark.parametrize("limit_ns", [1000, 100_000, 5_000_000])
def test_limit_is_passed_by_64_polls_at_most(lib, limit_ns):
    """64 polls of up to 20 us each, 1.3 ms, and as much again for the launch and the barrier that
    completes."""
    st, res = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):
        st.zero_()
        a.record()
        rc = lib.moe_selftest_bounded_wait(st.data_ptr(), limit_ns, res.data_ptr(),
                                           torch.cuda.current_stream().cuda_stream)
        b.record()
        torch.cuda.synchronize()
        assert rc == 0 and int(st) == moe.DEV_TIMEOUT and int(res) == 3
    assert limit_ns * 1e-6 <= a.elapsed_time(b) <= limit_ns * 1e-6 + 2.6
