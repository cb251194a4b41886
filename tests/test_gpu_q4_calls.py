"""Calls of the 4-bit operators at the edges of what they take, on the GPU, against tests/q4_ref.py."""

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
import q4_ref
from test_gpu_q4 import BF16, F16, attend, check, expect_written, handle, rows_step, same_pool

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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [40, 150])
def test_small_keys_and_values_under_many_rows(D, n):
    """K and V around 1e-3, where the operands (eighths of the values) are off by half of fp16's smallest number: a value
    by 2^-22, so a score by that times the query's magnitudes (the bound of q4_ref has V's part)."""
    scale = 0.1
    c = q4_ref.make_case([300, 20], [n, 5], 4, 2, D, 16, q_std=150.0, scale=scale, v_std=1e-3, seed=D + n)
    held = c["key_cache"][:, :, 16 * D // 2:].view(F16)
    held *= 2.0 ** -10
    op, out = attend(c)
    assert op.device_error() == 0
    ref, tol = q4_ref.attention(c)
    got = out.double().cpu().view(c["T"], 4, D)
    off = scale * 2.0 ** -22 * c["query"].double().abs().view(c["T"], 4, D).sum(2, keepdim=True)
    assert ((got - ref).abs() <= tol + 2.2 * off * 6e-3).all()  # (in the weights: of V, below 6e-3)
    assert (got - ref).norm() <= 2.0 ** -8 * ref.norm()


def test_a_chunk_among_empty_slots():
    """No more tokens than batch rows, all but one of them of one sequence: computed as single tokens are, so that a NaN
    scale of V reaches its channels only."""
    c = q4_ref.make_case([500] + [7] * 80, [75] + [0] * 79 + [1], 16, 2, 128, 16, seed=9)
    clean, tol = q4_ref.attention(c)
    op, out = attend(c)
    check(c, out)
    p = 520
    c["value_cache"][int(c["table"][0, p // 16])][:, 16 * 64:].view(F16)[:, 16 + p % 16] = float("nan")
    got = attend(c, op)[1].double().cpu().view(c["T"], 16, 128)
    hit = torch.zeros(c["T"], 16, 128, dtype=torch.bool)
    hit[20:75, :, 32:64] = True
    assert got[hit].isnan().all() and not got[~hit].isnan().any()
    assert ((got - clean).abs() <= tol)[~hit].all()
    assert op.device_error() == 0


def test_a_handle_refuses_other_types_and_sizes():
    c = q4_ref.make_case([30, 20], [2, 1], 4, 2, 64, 16, sink=True)
    op, good = handle(c), [c[k].cuda() for k in ("query", "key_cache", "value_cache", "table", "cum", "past_t")]
    out, key = torch.zeros_like(good[0]), torch.zeros(c["T"], 128, dtype=F16, device="cuda")
    op.attention(*good, 2, c["T"], out, head_sink=c["sink"].cuda())
    op.write(key, key, *good[1:], 2, c["T"])
    bad = [good[0].float(), good[1][:-1], good[2].half(), good[3][:, 1:].contiguous(), good[4].long(), good[5].long()]
    for k, x in enumerate(bad):
        args = good[:k] + [x] + good[k + 1:]
        with pytest.raises(pa.PAError):
            op.attention(*args, 2, c["T"], out)
        if k:
            with pytest.raises(pa.PAError):
                op.write(key, key, *args[1:], 2, c["T"])
            with pytest.raises(pa.PAError):
                op.read(*args[1:], 2, c["T"], key, out)
    with pytest.raises(pa.PAError):
        op.write(key[:, :64], key, *good[1:], 2, c["T"])
    for sink in (c["sink"].cuda().float(), c["sink"][:3].cuda()):
        with pytest.raises(pa.PAError):
            op.attention(*good, 2, c["T"], out, head_sink=sink)
    assert op.device_error() == 0


@pytest.mark.parametrize("n", [1, 9, 40, 150])
@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("q_std", [1e8, 3e9, 1e12, 1e30, 4e37])
def test_very_large_queries(q_std, softcap, n):
    """Scores that are finite in 32 bits, up to their largest.  One key takes all, or with a cap those of positive
    scores; keys of score 0 are no NaN.  K's scales are a power of two, so that its values lose no bits anywhere and
    which key is the largest is as good as certain."""
    c = q4_ref.make_case([200, 60], [n, 1], 4, 2, 128, 16, q_std=q_std, scale=0.01, softcap=softcap, dtype=BF16, seed=n)
    held = c["key_cache"][:, :, 16 * 64:].view(F16)
    held[~held.isnan()] = 0.5
    held[c["table"][0, 0].item()] = 0.0  # 16 keys whose scores are 0
    check(c)
