"""Calls of the 4-bit operators at the edges of what they take, on the GPU, against tests/q4_ref.py."""

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
import q4_ref
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


@pytest.mark.parametrize("n", [1, 60, 200])
@pytest.mark.parametrize("strong", [0, 70, 8191])
def test_a_long_tail_below_one_strong_key(n, strong):
    """One key outweighs each of 8,192 others by 2^25.4, which together still are all that some channels get.

    K's values are whole numbers, so a score is off by its 32-bit sums alone: (D + 8) 2^-24 of at most 9.4.  A unit of
    keys to each SM, so that they share a reference: a tail's weight is off by 2^-11 of itself, or by half of fp16's
    smallest number where the strong key's weight is at least 2^5: 2^-30 of that one."""
    D, bs, past = 64, 64, 8192
    Hk = torch.cuda.get_device_properties(0).multi_processor_count
    pages, scale = -(-(past + n) // bs), 1.17
    code_k, code_v = torch.zeros(pages, 1, bs, D, dtype=torch.int64), torch.zeros(pages, 1, bs, D, dtype=torch.int64)
    code_k[..., 0] = -8
    code_v[..., 32:] = 7
    code_k[strong // bs, 0, strong % bs, 0] = 7
    code_v[strong // bs, 0, strong % bs, :32] = 7
    code_v[strong // bs, 0, strong % bs, 32:] = 0
    ones = torch.ones(pages, 1, bs, D // 32, dtype=F16)
    kc, vc = (q4_ref.pack(x, ones).expand(-1, Hk, -1).contiguous().cuda() for x in (code_k, code_v))
    query = torch.zeros(n, Hk, D, dtype=F16, device="cuda")
    query[..., 0] = 1.0
    cfg = pa.make_config(Hk, Hk, D, bs, pages, pages, 1, n, scale=scale)
    op = pa.PagedQ4(cfg)
    out = torch.empty(n, Hk * D, dtype=F16, device="cuda")
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (list(range(pages)), [0, n], [past])]
    op.attention(query.view(n, -1), kc, vc, ints[0].view(1, pages), ints[1], ints[2], 1, n, out)
    assert op.device_error() == 0
    got = out.double().cpu().view(n, Hk, D)
    weak = torch.exp(torch.tensor(-15 * scale, dtype=torch.float64))
    keys = (past + torch.arange(n, dtype=torch.float64)).view(n, 1, 1)  # (weak ones of row j: past + j)
    tail, top = 7 * keys * weak / (1 + keys * weak), 7 / (1 + keys * weak)
    off = 2 * (D + 8) * 2.0 ** -24 * 8 * scale
    tol = tail * (2.0 ** -11 * 2 + off) + 7 * keys * 2.0 ** -30 + 136 * 2.0 ** -24
    assert ((got[..., 32:] - tail).abs() <= tol).all(), float((got[..., 32:] - tail).abs().max())
    assert ((got[..., :32] - top).abs() <= top * (2.0 ** -11 * 2 + off) + 136 * 2.0 ** -24).all()
