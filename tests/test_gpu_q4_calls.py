"""Calls of the 4-bit operators at the edges of what they take, on the GPU, against tests/q4_ref.py."""

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
from test_gpu_q4 import BF16, F16, expect_written, handle, rows_step, same_pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    pa.build()


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rows_of_a_sequence_that_ends_behind_the_call(dtype):
    """The last sequence's end lies behind token_count: flagged, nothing of it written or read."""
    c = rows_step([3, 40, 9], [20, 9, 4], 2, 128, 16, dtype)
    cum = c["cum"].clone()
    cum[3] += 5
    op = handle(c)
    pools = [c["key_cache"].cuda(), c["value_cache"].cuda()]
    rest = [c["table"].cuda(), cum.cuda(), c["past_t"].cuda()]
    key, value = c["key"].cuda(), c["value"].cuda()
    op.write(key, value, *pools, *rest, 3, c["T"])
    assert op.device_error() == pa.PA_DEVERR_CUM
    for got, want in zip(pools, expect_written(dict(c, n=[20, 9, 0]))):
        same_pool(got, want, c)
    outs = [torch.full_like(key, -7.0) for _ in range(2)]
    op.read(*pools, *rest, 3, c["T"], *outs)
    assert op.device_error() == pa.PA_DEVERR_CUM
    for out in outs:
        assert bool((out[29:] == -7.0).all()) and not bool((out[:29] == -7.0).any())
