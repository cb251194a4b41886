"""The 4-bit attention's kernel for sequences of many rows, with many key tiles to an SM: the rings of operands, masks and
units come round several times, and units of one and of two row tiles follow one another in a CTA.  Against
tests/q4_ref.py in 64 bits."""

import math

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
import q4_ref
from test_gpu_q4 import BF16, F16, attend, check, handle

pytestmark = pytest.mark.gpu

TILE, UNIT = 128, 256  # keys of a tile, rows of a unit


@pytest.fixture(scope="module", autouse=True)
def built():
    pa.build()


def tiles_of(c):
    """Key tiles of all units of the call."""
    G, total = c["H"] // c["Hk"], 0
    for past, n in zip(c["past"], c["n"]):
        if n * G <= 48:
            continue  # (the other kernel's, or too few to matter)
        for row0 in range(0, n * G, UNIT):
            first_pos, last_pos = past + row0 // G, past + (min(row0 + UNIT, n * G) - 1) // G
            lo = max(0, first_pos + 1 - c["window"]) // TILE * TILE if c["window"] > 0 else 0
            total += -(-min(c["first"], lo) // TILE) + -(-(last_pos + 1 - lo) // TILE)
    return total * c["Hk"]


def per_sm(c):
    return tiles_of(c) / torch.cuda.get_device_properties(0).multi_processor_count


# Short units in front of long ones, in calls of more than 128 rows to a
# sequence (one tile of rows at a time: short units leave half the softmax
# warps without work) and of fewer (both halves share a short unit's tile).
SHORT_AND_LONG = dict(past=[2900, 3100, 2500, 3300, 2700, 3000, 2950, 1700], n=[20, 75, 31, 65, 13, 90, 32, 100])
SHARED = dict(past=[2900, 3100, 2500, 3300, 2700, 3000, 2950, 1700, 900], n=[20, 31, 13, 16, 32, 27, 14, 70, 19])
REMAINDERS = dict(past=[3000, 2800, 3130, 2750], n=[65, 70, 96, 66])  # units of 256 rows with a short one behind each


def many_tiles(shape, D, dtype, unmap=(), seed=0, **extras):
    return q4_ref.make_case(**shape, H=32, Hk=8, D=D, bs=32, dtype=dtype, seed=seed, unmap=unmap, **extras)


def holes(shape, bs=32):
    """Pages without a place, other ones of each sequence: scattered, whole tiles, none."""
    out = []
    for b, (past, n) in enumerate(zip(shape["past"], shape["n"])):
        pages = -(-(past + n) // bs)
        if b % 3 == 0:
            out += [(b, p) for p in range(pages - 2) if (p * 7 + b) % 5 < 2]
        elif b % 3 == 1:
            out += [(b, p) for p in range(pages - 2) if p // 4 % 4 == 1]
    return out


@pytest.mark.parametrize("extras", [{}, dict(softcap=6.0, window=2300, first=40, sink=True)], ids=["plain", "extras"])
@pytest.mark.parametrize("D,dtype", [(64, F16), (64, BF16), (128, F16), (128, BF16)])
@pytest.mark.parametrize("shape,least", [(SHORT_AND_LONG, 12), (SHARED, 7), (REMAINDERS, 8)],
                         ids=["short_and_long", "shared", "remainders"])
def test_many_tiles_to_an_sm(shape, least, D, dtype, extras):
    c = many_tiles(shape, D, dtype, unmap=holes(shape), seed=D, **extras)
    assert per_sm(c) >= least
    assert (c["T"] * 4 > TILE * c["B"]) == (shape is not SHARED)
    op, out = attend(c)
    first = out.clone()
    check(c, out)
    for _ in range(6):
        assert torch.equal(attend(c, op)[1], first)
    assert op.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", [SHORT_AND_LONG, SHARED], ids=["short_and_long", "shared"])
def test_values_that_are_no_numbers_reach_their_rows_only(shape, D):
    """New rows of every other sequence whose V overflowed: its rows from there on are not finite, every other row is as
    if they were not there."""
    c = many_tiles(shape, D, F16, unmap=holes(shape), seed=3 + D)
    clean, tol = q4_ref.attention(c)
    hit = torch.zeros(c["T"], dtype=torch.bool)
    for b in range(0, c["B"], 2):
        j = 2 * c["n"][b] // 3
        p = c["past"][b] + j
        c["value_cache"][int(c["table"][b, p // 32])][:, 32 * D // 2:].view(torch.float16)[:, p % 32] = math.nan
        hit[int(c["cum"][b]) + j:int(c["cum"][b + 1])] = True
    op = handle(c)
    for _ in range(4):
        got = attend(c, op)[1].double().cpu().view(c["T"], 32, D)
        assert not got[~hit].isnan().any()
        assert ((got - clean).abs() <= tol)[~hit].all()
        assert got[hit].isnan().any(-1).all()
    assert op.device_error() == 0


def test_captured_calls_with_many_tiles():
    """A captured call, replayed where short and long units change places."""
    shapes = [SHORT_AND_LONG, dict(past=SHORT_AND_LONG["past"][::-1], n=SHORT_AND_LONG["n"][::-1])]
    cases = [many_tiles(s, 128, F16, seed=k) for k, s in enumerate(shapes)]
    names = ("query", "key_cache", "value_cache", "table", "cum", "past_t")
    dev = [cases[0][k].cuda() for k in names]
    out = torch.full((cases[0]["T"], 32 * 128), -7.0, dtype=F16, device="cuda")
    op, stream = handle(cases[0]), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        op.attention(*dev, cases[0]["B"], cases[0]["T"], out, stream=stream.cuda_stream)
    for c in cases + cases[::-1]:
        for d, k in zip(dev, names):
            d.copy_(c[k])
        out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        check(c, out)
    assert op.device_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("shape", [SHORT_AND_LONG, SHARED], ids=["short_and_long", "shared"])
def test_very_large_scores_over_many_tiles(shape, D):
    """Scores around 1e9, whose largest grows from tile to tile: the tiles' and ranges' references are in other units."""
    c = many_tiles(shape, D, BF16, seed=7, q_std=1e10, scale=0.01)
    held = c["key_cache"][:, :, 32 * D // 2:].view(F16)
    held[~held.isnan()] = 0.5  # (K's values lose no bits: the largest key is as good as certain)
    op, out = attend(c)
    check(c, out)
    assert op.device_error() == 0
