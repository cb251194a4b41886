"""The tree operators on the GPU against their 64-bit forms (tests/tree_ref.py)."""

import math

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
import tree_ref

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    pa.build()


def handle(c, **over):
    cfg = pa.make_config(c["H"], c["Hk"], c["D"], c["bs"], c["NB"], c["MB"], c["B"], max(c["T"], 1), scale=c["scale"],
                         softcap=c["softcap"], local_window_size=c["window"],
                         cache_dtype=pa.PA_CACHE_BF16 if c["dtype"] == BF16 else pa.PA_CACHE_FP16, **over)
    return pa.PagedTree(cfg, c["max_draft"])


def cuda(t):
    return None if t is None else t.cuda()


def attend(c, op=None, out=None, stream=None):
    op = op or handle(c)
    out = torch.full((c["T"], c["H"] * c["D"]), -7.0, dtype=c["dtype"], device="cuda") if out is None else out
    op.attention(c["query"].cuda(), c["key_cache"].cuda(), c["value_cache"].cuda(), c["table"].cuda(),
                 c["cum"].cuda(), c["past_t"].cuda(), c["B"], c["T"], out, positions=cuda(c["positions"]),
                 tree_mask=cuda(c["mask"]), distance_slopes=cuda(c["slopes"]), head_sink=cuda(c["sink"]),
                 stream=stream)
    torch.cuda.synchronize()
    return op, out


def check_attention(c):
    op, out = attend(c)
    assert op.device_error() == 0
    ref, tol = tree_ref.attention(c)
    got = out.double().cpu().view(c["T"], c["H"], c["D"])
    live = int(c["cum"][-1])
    assert not got[:live].isnan().any(), "NaN in the output"
    off = (got[:live] - ref[:live]).abs() - tol[:live]
    assert off.max() <= 0, f"{int((off > 0).sum())} of {off.numel()} values off, worst by {off.max():.3g}"
    assert bool((got[live:] == -7.0).all()), "padding rows were written"


CASES = {
    "one_token_no_context": dict(past=[0], n=[1], H=4, Hk=2, D=64, bs=16),
    "one_token": dict(past=[37], n=[1], H=4, Hk=1, D=128, bs=16),
    "empty_context_tree": dict(past=[0, 0], n=[7, 33], H=4, Hk=2, D=128, bs=16),
    "lengths_around_a_tile": dict(past=[127, 128, 129, 120, 0, 255], n=[1, 1, 3, 9, 128, 2], H=2, Hk=2, D=64, bs=32),
    "sequences_without_tokens": dict(past=[40, 300, 0, 5], n=[0, 4, 0, 6], H=8, Hk=2, D=128, bs=16),
    "shared_heads_5": dict(past=[200, 77], n=[9, 26], H=10, Hk=2, D=128, bs=64),
    "shared_heads_16": dict(past=[150, 600], n=[9, 40], H=16, Hk=1, D=64, bs=16, dtype=BF16),
    "many_rows": dict(past=[130], n=[70], H=16, Hk=2, D=128, bs=16, dtype=BF16),
    "longest_draft": dict(past=[65], n=[256], H=2, Hk=1, D=64, bs=128),
    "long_axis": dict(past=[9000], n=[5], H=2, Hk=1, D=128, bs=256, dtype=BF16),
    "causal_default": dict(past=[100, 31], n=[6, 17], H=4, Hk=2, D=128, bs=16, mask="none", positions=False),
    "random_mask_empty_rows": dict(past=[0, 0], n=[40, 3], H=4, Hk=4, D=64, bs=16, mask="random"),
    "random_mask": dict(past=[333, 1], n=[70, 200], H=4, Hk=2, D=128, bs=32, mask="random", dtype=BF16),
    "mask_wider_than_draft": dict(past=[50], n=[5], H=4, Hk=2, D=64, bs=16, max_draft=100),
    "softcap": dict(past=[300, 20], n=[12, 3], H=4, Hk=2, D=128, bs=16, softcap=5.0, q_std=6.0),
    "softcap_both_ways": dict(past=[900, 200], n=[12, 60], H=8, Hk=2, D=128, bs=16, softcap=5.5),
    "softcap_far_above": dict(past=[300, 20], n=[12, 3], H=4, Hk=2, D=64, bs=16, softcap=200.0, dtype=BF16),
    "window": dict(past=[500, 20, 64], n=[12, 30, 64], H=4, Hk=2, D=64, bs=16, window=33),
    "window_of_one": dict(past=[200, 0], n=[9, 4], H=4, Hk=2, D=128, bs=16, window=1),
    "window_wider_than_all": dict(past=[100], n=[9], H=4, Hk=2, D=128, bs=16, window=100000),
    "window_without_positions": dict(past=[300], n=[40], H=4, Hk=2, D=64, bs=16, window=20, positions=False),
    "bias": dict(past=[700, 3], n=[12, 20], H=4, Hk=2, D=64, bs=16, slopes=True, dtype=BF16),
    "sink": dict(past=[90, 0], n=[12, 20], H=4, Hk=2, D=128, bs=16, sink=True),
    "everything": dict(past=[700, 3, 129], n=[12, 20, 64], H=8, Hk=2, D=128, bs=32, softcap=8.0, window=250,
                       slopes=True, sink=True, dtype=BF16),
    "unmapped_pages": dict(past=[200, 64], n=[10, 5], H=4, Hk=2, D=128, bs=16, unmap=[(0, 0), (0, 5), (1, 1)]),
    "every_page_unmapped": dict(past=[30, 20], n=[2, 3], H=4, Hk=2, D=64, bs=16,
                                unmap=[(0, 0), (0, 1)]),
    "padding_rows": dict(past=[30, 20], n=[2, 3], H=4, Hk=2, D=64, bs=16, pad=9),
    "own_scale": dict(past=[60], n=[4], H=4, Hk=2, D=128, bs=16, scale=0.3),
    "d256_one_token": dict(past=[0, 63, 64], n=[1, 1, 1], H=2, Hk=1, D=256, bs=16),
    "d256_rows_over_tiles": dict(past=[130, 7], n=[70, 33], H=8, Hk=2, D=256, bs=32, dtype=BF16),
    "d256_everything": dict(past=[700, 3, 129], n=[12, 20, 64], H=8, Hk=2, D=256, bs=64, softcap=8.0, window=250,
                            slopes=True, sink=True),
    "d256_long_axis": dict(past=[5000], n=[9], H=2, Hk=1, D=256, bs=128, dtype=BF16),
    "d256_unmapped": dict(past=[200, 64], n=[10, 5], H=4, Hk=2, D=256, bs=16, unmap=[(0, 0), (0, 5), (1, 1)]),
    "d64_long_axis_32_rows": dict(past=[7001], n=[8], H=4, Hk=1, D=64, bs=16),
    "d64_long_axis_64_rows": dict(past=[6003, 100], n=[16, 9], H=8, Hk=2, D=64, bs=32, dtype=BF16, sink=True),
    "d64_everything_32_rows": dict(past=[700, 3, 129], n=[5, 7, 8], H=8, Hk=2, D=64, bs=32, softcap=8.0, window=250,
                                   slopes=True, sink=True, dtype=BF16),
    "d64_everything_64_rows": dict(past=[900, 0, 127], n=[12, 16, 1], H=8, Hk=2, D=64, bs=16, softcap=8.0,
                                   window=200, slopes=True, sink=True, mask="random"),
    "d64_pages_of_64": dict(past=[700, 63, 64], n=[12, 20, 1], H=4, Hk=2, D=64, bs=64, unmap=[(0, 3)]),
    "d64_pages_of_256": dict(past=[700, 255, 256], n=[40, 33, 1], H=8, Hk=1, D=64, bs=256, dtype=BF16, sink=True),
    "d256_pages_of_256": dict(past=[700, 255, 256], n=[12, 20, 1], H=4, Hk=2, D=256, bs=256, dtype=BF16),
    "long_axis_two_tiles": dict(past=[6000], n=[60], H=4, Hk=1, D=128, bs=64),
    "one_head_of_many_pieces": dict(past=[20000], n=[3], H=1, Hk=1, D=128, bs=128),
    "groups_of_128": dict(past=[100], n=[3], H=128, Hk=1, D=64, bs=16),
    "groups_of_100": dict(past=[300], n=[2], H=100, Hk=1, D=128, bs=16, dtype=BF16),
    "heads_beyond_the_sms": dict(past=[20, 0], n=[2, 1], H=200, Hk=200, D=64, bs=16),
    "many_sequences": dict(past=[(37 * i) % 90 for i in range(600)], n=[i % 3 for i in range(600)], H=2, Hk=1, D=64,
                           bs=16),
}


@pytest.mark.parametrize("name", CASES)
def test_attention(name):
    check_attention(tree_ref.make_case(**CASES[name], seed=sum(map(ord, name))))


@pytest.mark.parametrize("D,n", [(128, [40, 9]), (128, [70, 9]), (64, [14, 6]), (64, [30, 9]), (256, [40, 9])])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_keys_never_reach_a_row(dtype, bad, D, n):
    """Draft tokens whose K and V overflowed: the rows that do not admit them are as if they were not there; the
    rows that do are not finite."""
    c = tree_ref.make_case([130, 0], n, 4, 2, D, 16, dtype=dtype, seed=5)
    clean, _ = tree_ref.attention(c)
    victims = {0: [6, 11, n[0] - 1], 1: [4]}
    touched = torch.zeros(c["T"], dtype=torch.bool)
    for b, nodes in victims.items():
        for i in nodes:
            p = c["past"][b] + i
            slot = int(c["table"][b, p // c["bs"]]) * c["bs"] + p % c["bs"]
            c["key_cache"].view(-1, 2, D)[slot, :, 3] = bad
            c["value_cache"].view(-1, 2, D)[slot, :, 5] = bad
            rows = slice(int(c["cum"][b]), int(c["cum"][b + 1]))
            touched[rows] |= c["rows"][rows, i]
    _, out = attend(c)
    got = out.double().cpu().view(c["T"], 4, D)
    assert touched.any() and not touched.all()
    u = tree_ref.HALF_STEP[dtype]
    # (the bound of the clean step: weights and values of these rows are untouched)
    for b, nodes in victims.items():
        for i in nodes:
            p = c["past"][b] + i
            slot = int(c["table"][b, p // c["bs"]]) * c["bs"] + p % c["bs"]
            for name in ("key_cache", "value_cache"):
                c[name].view(-1, 2, D)[slot] = 0
    ref, tol = tree_ref.attention(c)
    keep = ~touched
    assert ((got[keep] - ref[keep]).abs() <= tol[keep]).all()
    assert not torch.isfinite(got[touched][..., 5]).any()
    assert u > 0 and torch.isfinite(clean).all()


@pytest.mark.parametrize("D,n,window", [(128, [40, 9], 50), (128, [70, 9], 129), (64, [14, 6], 20), (64, [30, 9], 2),
                                        (256, [40, 9], 75)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_keys_behind_the_window_never_reach_a_row(bad, D, n, window):
    """Context keys at the edge of the window, which some rows of a tree still admit, and behind it."""
    c = tree_ref.make_case([190, 140], n, 4, 2, D, 16, window=window, seed=9)
    # the edge's first two keys, the one before it, and in sequence 1 the last that some row leaves out
    low = [p - window + 1 for p in c["past"]]
    victims = [{low[0] - 1, low[0], low[0] + 1}, {low[1] - 1, low[1], int(c["pos"][n[0]:].max()) - window}]
    victims = [sorted(v & set(range(p))) for v, p in zip(victims, c["past"])]
    touched = torch.zeros(c["T"], dtype=torch.bool)
    for fill in (bad, 0.0):
        for b in range(2):
            rows = slice(int(c["cum"][b]), int(c["cum"][b + 1]))
            for p in victims[b]:
                slot = int(c["table"][b, p // 16]) * 16 + p % 16
                c["key_cache"].view(-1, 2, D)[slot, :, 3] = fill
                c["value_cache"].view(-1, 2, D)[slot, :, 5] = fill
                touched[rows] |= c["pos"][rows] - window < p
        if fill != 0.0:
            _, out = attend(c)
    assert touched.any() and not touched.all()
    got = out.double().cpu().view(c["T"], 4, D)
    ref, tol = tree_ref.attention(c)  # (the rows that admit no victim are those of the mended pools)
    assert ((got[~touched] - ref[~touched]).abs() <= tol[~touched]).all()
    assert not torch.isfinite(got[touched][..., 5]).any()


def ragged(B, lo, hi, n_max, seed, **over):
    """B sequences of lo..hi keys with trees of 1..n_max drafts, one of n_max among them."""
    g = torch.Generator().manual_seed(seed)
    past = torch.randint(lo, hi + 1, (B,), generator=g).tolist()
    n = torch.randint(1, n_max + 1, (B,), generator=g).tolist()
    n[B // 2] = n_max
    return tree_ref.make_case(past, n, over.pop("H"), over.pop("Hk"), over.pop("D"), over.pop("bs"), seed=seed, **over)


def attend_repeatedly(c, times=4):
    """The output of a step whose repetitions are the same bit for bit."""
    op = handle(c)
    outs = [attend(c, op)[1]]
    for _ in range(times - 1):
        assert torch.equal(attend(c, op)[1].view(torch.int16), outs[0].view(torch.int16))
    assert op.device_error() == 0
    return outs[0].double().cpu().view(c["T"], c["H"], c["D"])


def assert_close(got, ref, tol):
    off = (got - ref).abs() - tol
    assert not got.isnan().any() and off.max() <= 0, f"{int((off > 0).sum())} values off, worst by {off.max():.3g}"


# Rows of the widest tree: more than 128 per kv head (the K/V ring has 5 slots beside two tiles of Q), up to 128 (6).
@pytest.mark.parametrize("n_max,dtype", [(40, BF16), (40, F16), (32, BF16), (24, F16)])
def test_ragged_trees_over_long_segments(n_max, dtype):
    """Ranges of about 15 key tiles, so that a segment takes the K/V ring around several times; unused slots of the
    pages are NaN, and the last tiles' rows behind the sequence must be cleared in the tile itself."""
    c = ragged(64, 1000, 3000, n_max, 61, H=8, Hk=2, D=128, bs=16, dtype=dtype)
    ends = [(p + n) % 128 for p, n in zip(c["past"], c["n"])]
    assert any(0 < e < n for e, n in zip(ends, c["n"]))  # (some drafts lie over two key tiles)
    ref, tol = tree_ref.attention_by_sequence(c)
    assert_close(attend_repeatedly(c), ref, tol)


@pytest.mark.parametrize("n_max", [40, 32])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_masked_keys_never_reach_a_row_over_long_segments(bad, n_max):
    c = ragged(64, 1000, 3000, n_max, 62, H=8, Hk=2, D=128, bs=16, dtype=BF16)
    touched = torch.zeros(c["T"], dtype=torch.bool)
    for fill in (bad, 0.0):
        for b in range(c["B"]):
            rows = slice(int(c["cum"][b]), int(c["cum"][b + 1]))
            for i in {c["n"][b] // 2, c["n"][b] - 1} - {0}:
                p = c["past"][b] + i
                slot = int(c["table"][b, p // 16]) * 16 + p % 16
                c["key_cache"].view(-1, 2, 128)[slot, :, 3] = fill
                c["value_cache"].view(-1, 2, 128)[slot, :, 5] = fill
                touched[rows] |= c["rows"][rows, i]
        if fill != 0.0:
            got = attend_repeatedly(c)
    assert touched.any() and not touched.all()
    ref, tol = tree_ref.attention_by_sequence(c)  # (of the rows that admit none of them)
    assert_close(got[~touched], ref[~touched], tol[~touched])
    assert not torch.isfinite(got[touched][..., 5]).any()


# Steps whose CTAs work through segments of up to 16 to 68 key tiles, or many short ones, one after the other: the K/V ring and the ring
# of page masks go around many times, block ids are read 32 at a time, maxima move over a long row, and pieces that
# are themselves long are joined.
LONG = {
    "d128": dict(B=16, lo=5000, hi=6000, n_max=9, H=16, Hk=8, D=128, bs=16, dtype=BF16),
    "d128_six_slots_from_two_tiles": dict(B=20, lo=1500, hi=6000, n_max=64, H=16, Hk=8, D=128, bs=64),
    "d128_two_row_tiles": dict(B=12, lo=3000, hi=6000, n_max=100, H=16, Hk=8, D=128, bs=32, dtype=BF16),
    "d128_growing": dict(B=16, lo=3000, hi=6000, n_max=9, H=16, Hk=8, D=128, bs=16, q_std=6.0),
    "d128_window": dict(B=16, lo=3000, hi=6000, n_max=40, H=16, Hk=8, D=128, bs=16, window=2500, dtype=BF16),
    "d128_bias_cap_sink": dict(B=16, lo=3000, hi=6000, n_max=20, H=16, Hk=8, D=128, bs=256, slopes=True, sink=True,
                               softcap=20.0),
    "d64_four_replicas": dict(B=16, lo=4000, hi=6000, n_max=12, H=16, Hk=8, D=64, bs=16),
    "d64_two_replicas": dict(B=16, lo=4000, hi=6000, n_max=30, H=16, Hk=8, D=64, bs=32, dtype=BF16, slopes=True),
    "d64": dict(B=16, lo=4000, hi=6000, n_max=50, H=16, Hk=8, D=64, bs=128, dtype=BF16),
    "d64_two_row_tiles": dict(B=12, lo=2000, hi=6000, n_max=90, H=16, Hk=8, D=64, bs=16, softcap=30.0),
    "d64_window_without_positions": dict(B=16, lo=3000, hi=6000, n_max=30, H=16, Hk=8, D=64, bs=16, window=3001,
                                         positions=False),
    "d256": dict(B=8, lo=3000, hi=6000, n_max=20, H=16, Hk=8, D=256, bs=16, dtype=BF16),
    "d256_rows_over_tiles": dict(B=8, lo=3000, hi=5000, n_max=70, H=16, Hk=8, D=256, bs=64, sink=True),
    "d256_window": dict(B=8, lo=3000, hi=6000, n_max=20, H=16, Hk=8, D=256, bs=16, window=2000, slopes=True, dtype=BF16),
    "chunks_above_the_sms": dict(B=4, lo=700, hi=2500, n_max=9, H=100, Hk=100, D=64, bs=16),
    "segments_of_many_units": dict(B=300, lo=100, hi=900, n_max=20, H=16, Hk=8, D=128, bs=16, dtype=BF16),
}


@pytest.mark.parametrize("D,H,Hk", [(64, 2, 1), (128, 1, 1), (256, 2, 1)])
def test_more_sequences_than_32_groups(D, H, Hk):
    """2500 sequences, most of them empty: the schedule looks through groups of 32 sequences, 32 at a time."""
    g = torch.Generator().manual_seed(81)
    n = (torch.randint(0, 4, (2500,), generator=g) * (torch.rand(2500, generator=g) < 0.2)).tolist()
    n[1000:1200] = [0] * 200
    n[-40:] = [0] * 40
    c = tree_ref.make_case(torch.randint(0, 60, (2500,), generator=g).tolist(), n, H, Hk, D, 16, dtype=BF16, seed=81)
    ref, tol = tree_ref.attention_by_sequence(c)
    assert_close(attend_repeatedly(c, 2), ref, tol)


@pytest.mark.parametrize("unmapped", [False, True])
@pytest.mark.parametrize("name", LONG)
def test_long_segments(name, unmapped):
    over = dict(LONG[name])
    if unmapped:  # pages of the context, early and late, some of them next to each other
        over["unmap"] = [(b, p) for b in range(0, over["B"], 2) for p in (0, 1, 3 + b % 4)]
    c = ragged(seed=80 + len(name), **over)
    if unmapped:
        for b in range(1, c["B"], 2):  # the last pages of the context, one before the drafts'
            last = c["past"][b] // c["bs"] - 1
            c["table"][b, last], c["table"][b, last // 2] = -1, -1
    ref, tol = tree_ref.attention_by_sequence(c)
    assert_close(attend_repeatedly(c, 3), ref, tol)


def test_infinite_value_in_an_admitted_key_keeps_its_channel():
    """An infinite V element of an admitted draft key makes that channel infinite and leaves the others exact."""
    c = tree_ref.make_case([40], [12], 4, 2, 64, 16, seed=6)
    ref, tol = tree_ref.attention(c)
    p = 40 + 5
    slot = int(c["table"][0, p // 16]) * 16 + p % 16
    c["value_cache"].view(-1, 2, 64)[slot, :, 9] = math.inf
    _, out = attend(c)
    got = out.double().cpu().view(12, 4, 64)
    sees = c["rows"][:12, 5]
    assert torch.isposinf(got[sees][..., 9]).all()
    others = [ch for ch in range(64) if ch != 9]
    assert ((got - ref).abs() <= tol)[..., others].all()
    assert ((got - ref).abs() <= tol)[~sees].all()


UNFIT = {
    "one_tile": dict(past=[5], n=[3], H=4, Hk=2), "short": dict(past=[400], n=[5], H=4, Hk=2),
    "batch": dict(past=[700, 300, 129, 0, 1500], n=[12, 1, 30, 7, 5], H=8, Hk=2),
    "many_pieces": dict(past=[9000], n=[3], H=2, Hk=1), "two_row_tiles": dict(past=[3000], n=[70], H=8, Hk=2),
    "two_row_tiles_short": dict(past=[20], n=[70], H=8, Hk=2), "causal": dict(past=[0], n=[9], H=4, Hk=1, mask="none"),
}
FORMS = {"plain": {}, "capped": dict(softcap=5.0), "windowed": dict(window=120, sink=True), "biased": dict(slopes=True)}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("name", UNFIT)
def test_scores_that_are_no_numbers_stay_so(name, D, form):
    """A NaN in a query row makes the row NaN, one in a key every row that admits it, and an infinite score a row
    without a cap, however the sequence is cut into pieces; the other rows are as if it were not there."""
    c = tree_ref.make_case(**UNFIT[name], D=D, bs=16, seed=71, **FORMS[form])
    ref, tol = tree_ref.attention_by_sequence(c)
    H, G = c["H"], c["H"] // c["Hk"]
    q = c["query"].view(c["T"], H, D)
    lost = torch.zeros(c["T"], H, dtype=torch.bool)
    for t, h in ((0, 0), (c["T"] - 1, H - 1), (c["T"] // 2, H // 2)):
        q[t, h, 7] = math.nan
        lost[t, h] = True
    if not c["softcap"] and c["past"][0] > 100:  # (enough keys for a score of +inf; tanh takes it back)
        q[1, 1, 9] = math.inf
        lost[1, 1] = True
    b, p = len(c["past"]) - 1, c["past"][-1]  # the last sequence's first draft, seen by its own subtree
    slot = int(c["table"][b, p // 16]) * 16 + p % 16
    c["key_cache"].view(-1, c["Hk"], D)[slot, 0, 11] = math.nan
    rows = slice(int(c["cum"][b]), int(c["cum"][b + 1]))
    lost[rows, :G] |= c["rows"][rows, 0][:, None]
    _, out = attend(c)
    got = out.double().cpu().view(c["T"], H, D)
    assert lost.any() and (not lost.all() or c["Hk"] == 1)
    assert got[lost].isnan().all(), f"{int((~got[lost].isnan()).any(-1).sum())} of {int(lost.sum())} rows"
    if not lost.all():
        assert_close(got[~lost], ref[~lost], tol[~lost])


@pytest.mark.parametrize("kind", ["context", "draft"])
@pytest.mark.parametrize("D,H,Hk,n", [(128, 1, 1, [3, 1]), (128, 8, 2, [60, 40]), (64, 4, 1, [5, 2]), (256, 4, 2, [9, 1]),
                                      (64, 16, 2, [60, 7]), (128, 16, 16, [3, 1])])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_values_that_are_no_numbers_stay_so_at_any_weight(bad, D, H, Hk, n, kind):
    """A non-finite V element of a key whose weight is below the smallest float (scores 400 apart, in other pieces of
    the unit): 0 * inf is NaN in 32 bits, an infinity by the definition, and a number in neither."""
    c = tree_ref.make_case([5000, 300], n, H, Hk, D, 16, dtype=BF16, mask="none", seed=73)
    t = 400.0 / (2 * math.sqrt(D) * 3.0)
    c["query"][:] = 3.0
    K, V = (c[k].view(-1, Hk, D) for k in ("key_cache", "value_cache"))
    for b, past in enumerate(c["past"]):
        for p in range(past + n[b]):
            slot = int(c["table"][b, p // 16]) * 16 + p % 16
            K[slot] = -t if (p < past // 2) == (kind == "context") else t  # (half of the keys, whole pieces among them)
            if p == (17 if kind == "context" else past):
                V[slot, :, 5] = bad
    _, out = attend(c)
    got = out.double().cpu().view(c["T"], H, D)
    assert not torch.isfinite(got[..., 5]).any()
    V.nan_to_num_(0.0, 0.0, 0.0)
    ref, tol = tree_ref.attention_by_sequence(c)
    others = [ch for ch in range(D) if ch != 5]
    assert_close(got[..., others], ref[..., others], tol[..., others])


@pytest.mark.parametrize("form", ["plain", "windowed"])
@pytest.mark.parametrize("D,H,Hk,n", [(64, 4, 1, [5, 2, 8, 1]), (64, 8, 2, [12, 16, 3, 1]), (64, 4, 1, [40, 9, 2, 1]),
                                      (128, 4, 2, [9, 1, 40, 2]), (256, 4, 2, [9, 1, 20, 2])])
def test_infinite_values_of_context_keys_make_their_channels_infinite(D, H, Hk, n, form):
    """Infinities of one sign among the values that every row admits give that infinity, of both signs NaN: in one
    key, in two keys of a tile or of two tiles, and beside an infinite draft."""
    c = tree_ref.make_case([700, 40, 130, 5000], n, H, Hk, D, 16, dtype=BF16, seed=74, q_std=0.3, sink=True,
                           window=4000 if form == "windowed" else -1)
    ref, tol = tree_ref.attention_by_sequence(c)
    V = c["value_cache"].view(-1, Hk, D)

    def put(b, p, ch, v):
        V[int(c["table"][b, p // 16]) * 16 + p % 16, :, ch] = v

    want = {5: math.inf, 6: -math.inf, 7: math.inf, D - 1: math.nan, D - 2: math.nan}
    for b, past in enumerate(c["past"]):
        put(b, past - 2, 5, math.inf)
        put(b, past - 1, 6, -math.inf)
        put(b, past - 30, 6, -math.inf)
        put(b, past - 3, 7, math.inf)
        put(b, past - 35, 7, math.inf)
        put(b, past, 7, math.inf)  # the root of the tree
        put(b, past - 4, D - 1, math.inf)
        put(b, past - 39, D - 1, -math.inf)
        put(b, past - 5, D - 2, math.inf)
        put(b, past - 1, D - 2, math.nan)
    _, out = attend(c)
    got = out.double().cpu().view(c["T"], H, D)
    for ch, v in want.items():
        w = torch.full_like(got[..., ch], v)
        assert torch.equal(got[..., ch].nan_to_num(nan=0.5), w.nan_to_num(nan=0.5)), ch
    rest = [ch for ch in range(D) if ch not in want]
    assert_close(got[..., rest], ref[..., rest], tol[..., rest])


def test_bad_device_data_is_flagged_and_skipped():
    base = tree_ref.make_case([40, 50, 60], [3, 4, 5], 4, 2, 64, 16, seed=7)
    ref, tol = tree_ref.attention(base)

    def run(**over):
        c = {**base, **over}
        op, out = attend(c, handle(base))
        return op.device_error(), out.double().cpu().view(c["T"], 4, 64)

    err, out = run(past_t=torch.tensor([40, -1, 60], dtype=torch.int32))
    assert err == pa.PA_DEVERR_PAST and (out[3:7] == -7).all()
    assert ((out - ref).abs() <= tol)[:3].all() and ((out - ref).abs() <= tol)[7:].all()
    err, out = run(past_t=torch.tensor([40, 50, 100000], dtype=torch.int32))
    assert err == pa.PA_DEVERR_KV_BOUND and (out[7:] == -7).all() and ((out - ref).abs() <= tol)[:7].all()
    err, out = run(cum=torch.tensor([0, 3, 2, 12], dtype=torch.int32))
    assert err & pa.PA_DEVERR_CUM
    err, out = run(cum=torch.tensor([0, 3, 7, 99], dtype=torch.int32))
    assert err & pa.PA_DEVERR_CUM and ((out - ref).abs() <= tol)[:7].all()
    table = base["table"].clone()
    table[1, 1] = base["NB"] + 5
    err, out = run(table=table)
    assert err == pa.PA_DEVERR_BLOCK_ID and ((out - ref).abs() <= tol)[:3].all()
    err, out = run()
    assert err == 0 and ((out - ref).abs() <= tol).all()
    small = handle({**base, "max_draft": 4})
    _, out = attend({**base, "mask": None, "positions": None}, small)
    assert small.device_error() == pa.PA_DEVERR_Q_BOUND


def test_a_sequence_too_long_to_schedule_is_flagged():
    """2^24 key tiles for each of 256 units (one page that stands for all of a table) are refused on the device."""
    H, D, bs, n, MB = 128, 256, 256, 256, (1 << 30) // 256
    cfg = pa.make_config(H, 1, D, bs, 1, MB, 1, n, cache_dtype=pa.PA_CACHE_FP16)
    op = pa.PagedTree(cfg, n)
    kc, vc = torch.zeros(1, bs, 1, D, dtype=F16, device="cuda"), torch.zeros(1, bs, 1, D, dtype=F16, device="cuda")
    out = torch.full((n, H * D), -7.0, dtype=F16, device="cuda")
    op.attention(torch.zeros_like(out), kc, vc, torch.zeros(1, MB, dtype=torch.int32, device="cuda"),
                 torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                 torch.tensor([(1 << 30) - n], dtype=torch.int32, device="cuda"), 1, n, out)
    torch.cuda.synchronize()
    assert op.device_error() == pa.PA_DEVERR_KV_BOUND
    assert bool((out == -7.0).all())


def test_attention_is_the_same_every_time_and_in_a_graph():
    c = tree_ref.make_case([900, 3000, 17], [20, 8, 40], 8, 2, 128, 16, dtype=BF16, seed=8)
    op = handle(c)
    d = {k: cuda(c[k]) for k in ("query", "key_cache", "value_cache", "table", "cum", "past_t", "positions", "mask")}
    outs = [torch.empty(c["T"], 8 * 128, dtype=BF16, device="cuda") for _ in range(4)]

    def call(out, s):
        op.attention(d["query"], d["key_cache"], d["value_cache"], d["table"], d["cum"], d["past_t"], c["B"], c["T"],
                     out, positions=d["positions"], tree_mask=d["mask"], stream=s.cuda_stream)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for o in outs[:2]:
        call(o, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(outs[2], s)
        call(outs[3], s)
    outs[2].zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(outs[0], o)
    # new lengths under the captured addresses
    d["past_t"].copy_(torch.tensor([100, 3000, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    call(outs[0], s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and op.device_error() == 0


# ---------------------------------------------------------------- rotary


def phases(pos, f):
    """Angles in 64 bits: the product is exact to 2^-53 of it, so far positions are split first."""
    return torch.outer(pos.double(), f)


def rotate_ref(x, heads, D, R, off, inter, pos, f, m, sign=1.0):
    x = x.double().view(x.shape[0], heads, D)
    a = phases(pos, f)[:, None]
    c, s = m * torch.cos(a), sign * m * torch.sin(a)
    y = x.clone()
    i1, i2 = ((slice(off, off + R, 2), slice(off + 1, off + R, 2)) if inter else
              (slice(off, off + R // 2), slice(off + R // 2, off + R)))
    y[..., i1], y[..., i2] = x[..., i1] * c - x[..., i2] * s, x[..., i2] * c + x[..., i1] * s
    size = x.abs()
    both = size[..., i1] + size[..., i2]
    size[..., i1], size[..., i2] = abs(m) * both, abs(m) * both
    return y, size


def rotary_tol(y, size, dtype):
    """Half a step of the type for the rounding (fp16 below 2^-14: 2^-25), and for the fp32 arithmetic 2^-20 of the
    pair: cos and sin are off by the phase's conversion (2^-24 of up to pi) and sincospif's two units, each product
    and the sum by half a step."""
    return tree_ref.HALF_STEP[dtype] * y.abs() + (2.0 ** -25 if dtype == F16 else 0.0) + 2.0 ** -20 * size


ROTARY = [
    dict(T=1, H=4, Hk=1, D=64, R=64), dict(T=5, H=32, Hk=8, D=128, R=128), dict(T=3, H=3, Hk=1, D=72, R=48, off=16),
    dict(T=33, H=8, Hk=2, D=128, R=64, inter=True), dict(T=700, H=6, Hk=2, D=256, R=256, dtype=BF16),
    dict(T=7, H=2, Hk=2, D=512, R=512, dtype=torch.float32), dict(T=9, H=5, Hk=5, D=64, R=16, off=48, inter=True,
                                                                  dtype=torch.float32),
    dict(T=17, H=4, Hk=0, D=128, R=112, off=8, dtype=BF16), dict(T=17, H=0, Hk=3, D=128, R=112, off=16, inter=True),
    dict(T=20000, H=2, Hk=1, D=64, R=32),
]


@pytest.mark.parametrize("far", [10, 1000000, -5000, 2 ** 31 - 1])
@pytest.mark.parametrize("r", ROTARY, ids=lambda r: "-".join(str(v) for v in r.values()))
def test_rotary(r, far):
    T, H, Hk, D, R = (r[k] for k in ("T", "H", "Hk", "D", "R"))
    off, inter, dtype = r.get("off", 0), r.get("inter", False), r.get("dtype", F16)
    g = torch.Generator().manual_seed(T + D)
    steps, m = pa.pa_rotary_steps(R, pa.PA_ROTARY_SCALE_BY_PARTS, factor=4.0, original_positions=4096.0, low=1.0,
                                  high=32.0)
    f = torch.tensor([v * 2.0 ** -64 * 2 * math.pi for v in steps], dtype=torch.float64)
    pos = (far + torch.randint(-9, 1, (T,), generator=g)).int()
    q, k = (torch.randn(T, h * D, generator=g).to(dtype) for h in (H, Hk))
    rc = pa.make_rotary_config(D, R, off, int(inter), {F16: 0, BF16: 1, torch.float32: 2}[dtype], m)
    dq, dk = q.cuda(), k.cuda()
    qo, ko = torch.full_like(dq, 9.0), torch.full_like(dk, 9.0)
    pa.pa_rotary(rc, pa.rotary_steps_tensor(steps), pos.cuda(), T, H, dq, qo, Hk, dk, ko)
    torch.cuda.synchronize()
    # positions near 2^31 times a double frequency lose 2^-53 2^31 radians: nothing here
    for x, y, h in ((q, qo, H), (k, ko, Hk)):
        if not h:
            continue
        ref, size = rotate_ref(x, h, D, R, off, inter, pos, f, m)
        got = y.double().cpu().view(T, h, D)
        assert ((got - ref).abs() <= rotary_tol(ref, size, dtype)).all()
        outside = [c for c in range(D) if not off <= c < off + R]
        assert torch.equal(y.cpu().view(T, h, D)[..., outside], x.view(T, h, D)[..., outside])


def test_rotary_in_place_on_packed_rows():
    """Q and K slices of packed [Q|K|V] rows, rotated in place; V keeps its bits."""
    T, H, Hk, D = 37, 4, 2, 64
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(T, (H + 2 * Hk) * D, generator=g).to(BF16)
    dev = packed.cuda()
    steps, m = pa.pa_rotary_steps(D)
    f = torch.tensor([v * 2.0 ** -64 * 2 * math.pi for v in steps], dtype=torch.float64)
    pos = torch.arange(T, dtype=torch.int32) * 1001
    q, k = dev[:, :H * D], dev[:, H * D:(H + Hk) * D]
    rc = pa.make_rotary_config(D, dtype=pa.PA_ROTARY_BF16)
    pa.pa_rotary(rc, pa.rotary_steps_tensor(steps), pos.cuda(), T, H, q, q, Hk, k, k)
    torch.cuda.synchronize()
    for a, b, h in ((0, H * D, H), (H * D, (H + Hk) * D, Hk)):
        ref, size = rotate_ref(packed[:, a:b], h, D, D, 0, False, pos, f, m)
        assert ((dev[:, a:b].double().cpu().view(T, h, D) - ref).abs() <= rotary_tol(ref, size, BF16)).all()
    assert torch.equal(dev[:, (H + Hk) * D:].cpu(), packed[:, (H + Hk) * D:])


@pytest.mark.parametrize("inter", [0, 1])
def test_rotary_gradient(inter):
    """conjugate maps dy to dx: against autograd of the 64-bit form, and against central differences of the kernel
    itself (the map is linear, so they are exact up to the fp32 rounding of values of size one over a step of 1)."""
    T, H, D, R, off = 6, 3, 64, 32, 16
    g = torch.Generator().manual_seed(9)
    x = torch.randn(T, H * D, generator=g)
    dy = torch.randn(T, H * D, generator=g)
    pos = torch.tensor([0, 1, 77, 4096, 123456, -3], dtype=torch.int32)
    steps, _ = pa.pa_rotary_steps(R)
    f = torch.tensor([v * 2.0 ** -64 * 2 * math.pi for v in steps], dtype=torch.float64)
    m = 1.25
    dev_steps = pa.rotary_steps_tensor(steps)

    def kernel(v, conjugate):
        out = torch.empty(T, H * D, device="cuda")
        rc = pa.make_rotary_config(D, R, off, inter, pa.PA_ROTARY_FP32, m, conjugate)
        pa.pa_rotary(rc, dev_steps, pos.cuda(), T, H, v.cuda(), out)
        return out.double().cpu()

    x64 = x.double().requires_grad_(True)
    a = phases(pos, f)[:, None]
    i1, i2 = ((slice(off, off + R, 2), slice(off + 1, off + R, 2)) if inter else
              (slice(off, off + R // 2), slice(off + R // 2, off + R)))
    v = x64.view(T, H, D)
    y1 = m * (v[..., i1] * torch.cos(a) - v[..., i2] * torch.sin(a))
    y2 = m * (v[..., i2] * torch.cos(a) + v[..., i1] * torch.sin(a))
    d = dy.double().view(T, H, D)
    rest = [c for c in range(D) if not off <= c < off + R]
    loss = (y1 * d[..., i1]).sum() + (y2 * d[..., i2]).sum() + (v[..., rest] * d[..., rest]).sum()
    loss.backward()
    dx = kernel(dy, 1)
    _, size = rotate_ref(dy, H, D, R, off, bool(inter), pos, f, m)
    assert ((dx - x64.grad).abs().view(T, H, D) <= rotary_tol(x64.grad.view(T, H, D), size, torch.float32)).all()
    for ch in (0, off, off + 1, off + R // 2, off + R - 1, D - 1):
        e = torch.zeros(T, H, D)
        e[..., ch] = 0.5
        diff = kernel(x + e.view(T, -1), 0) - kernel(x - e.view(T, -1), 0)
        slope = (diff * dy.double()).view(T, H, D).sum(-1)
        # two outputs change, each off by 2^-20 of a pair of size below 2 * 1.25 * 6
        bound = 2.0 ** -20 * 16 * 2 * dy.double().view(T, H, D).abs().sum(-1) + 2.0 ** -19
        assert ((slope - dx.view(T, H, D)[..., ch]).abs() <= bound).all()


def write_case(c, R, off=0, inter=0, packed=False, seed=1):
    g = torch.Generator().manual_seed(seed)
    H, Hk, D, T = c["H"], c["Hk"], c["D"], c["T"]
    rows = torch.randn(T, (H + 2 * Hk) * D, generator=g).to(c["dtype"]).cuda()
    q, k, v = rows[:, :H * D], rows[:, H * D:(H + Hk) * D], rows[:, (H + Hk) * D:]
    if not packed:
        q, k, v = (t.contiguous() for t in (q, k, v))
    steps, m = pa.pa_rotary_steps(R, pa.PA_ROTARY_SCALE_LINEAR, factor=2.0)
    rc = pa.make_rotary_config(D, R, off, inter, pa.PA_ROTARY_BF16 if c["dtype"] == BF16 else pa.PA_ROTARY_FP16, m)
    return q, k, v, steps, rc


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("name", ["d256_unmapped", "empty_context_tree", "sequences_without_tokens", "unmapped_pages", "padding_rows",
                                  "many_rows", "many_sequences", "longest_draft"])
def test_tree_write(name, packed):
    c = tree_ref.make_case(**CASES[name], seed=2)
    H, Hk, D, T, bs = (c[k] for k in ("H", "Hk", "D", "T", "bs"))
    R, off, inter = D // 2, 16, int(packed)
    q, k, v, steps, rc = write_case(c, R, off, inter, packed)
    f = torch.tensor([s * 2.0 ** -64 * 2 * math.pi for s in steps], dtype=torch.float64)
    kc, vc = torch.full_like(c["key_cache"], 3.0).cuda(), torch.full_like(c["value_cache"], 4.0).cuda()
    out = torch.full((T, H * D), -7.0, dtype=c["dtype"], device="cuda")
    op = handle(c)
    op.write(rc, pa.rotary_steps_tensor(steps), c["pos"].cuda(), q, k, v, out, kc, vc, c["table"].cuda(),
             c["cum"].cuda(), c["past_t"].cuda(), c["B"], T)
    assert op.device_error() == 0
    live = int(c["cum"][-1])
    ref, size = rotate_ref(q.cpu(), H, D, R, off, bool(inter), c["pos"], f, 1.0)
    got = out.double().cpu().view(T, H, D)
    assert ((got - ref).abs() <= rotary_tol(ref, size, c["dtype"]))[:live].all() and (got[live:] == -7).all()
    ref, size = rotate_ref(k.cpu(), Hk, D, R, off, bool(inter), c["pos"], f, 1.0)
    tol = rotary_tol(ref, size, c["dtype"])
    want_v, got_k = torch.full_like(c["value_cache"], 4.0).view(-1, Hk * D), kc.cpu().view(-1, Hk, D)
    written = torch.zeros(c["NB"] * bs, dtype=torch.bool)
    for b in range(c["B"]):
        for j in range(c["n"][b]):
            p, t = c["past"][b] + j, int(c["cum"][b]) + j
            blk = int(c["table"][b, p // bs])
            if blk < 0:
                continue
            slot = blk * bs + p % bs
            written[slot] = True
            want_v[slot] = v[t].cpu()
            assert ((got_k[slot].double() - ref[t]).abs() <= tol[t]).all()
    assert torch.equal(vc.cpu().view(-1, Hk * D), want_v)
    assert (got_k[~written] == 3.0).all()


def test_tree_write_flags_bad_device_data():
    c = tree_ref.make_case([40, 50], [3, 4], 4, 2, 64, 16, seed=7)
    q, k, v, steps, rc = write_case(c, 64)
    op = handle(c)
    st = pa.rotary_steps_tensor(steps)

    def run(**over):
        d = {**c, **over}
        kc, vc = torch.zeros_like(c["key_cache"]).cuda(), torch.zeros_like(c["value_cache"]).cuda()
        out = torch.zeros(c["T"], 256, dtype=F16, device="cuda")
        op.write(rc, st, d["pos"].cuda(), q, k, v, out, kc, vc, d["table"].cuda(), d["cum"].cuda(),
                 d["past_t"].cuda(), 2, c["T"])
        return op.device_error(), (kc != 0).any(-1).any(-1).sum().item()

    assert run() == (0, 7)
    assert run(past_t=torch.tensor([-4, 50], dtype=torch.int32)) == (pa.PA_DEVERR_PAST, 4)
    assert run(past_t=torch.tensor([40, 2 ** 31 - 2], dtype=torch.int32)) == (pa.PA_DEVERR_KV_BOUND, 3)
    assert run(cum=torch.tensor([0, 3, 70], dtype=torch.int32))[0] & pa.PA_DEVERR_CUM
    table = c["table"].clone()
    table[0, 2] = c["NB"]
    assert run(table=table) == (pa.PA_DEVERR_BLOCK_ID, 4)


# ---------------------------------------------------------------- commit


def commit_ref(pools, c, paths):
    """pools [L, 2, NB * bs, row]."""
    out = pools.clone()
    for b, path in enumerate(paths):
        for i, a in enumerate(path):
            d, s = c["past"][b] + i, c["past"][b] + a
            db, sb = int(c["table"][b, d // c["bs"]]), int(c["table"][b, s // c["bs"]])
            if db >= 0 and sb >= 0:
                out[:, :, db * c["bs"] + d % c["bs"]] = pools[:, :, sb * c["bs"] + s % c["bs"]]
    return out


def commit(c, paths, layers=3, width=None, op=None, past=None, count=None, table=None):
    g = torch.Generator().manual_seed(4)
    pools = torch.randn(layers, 2, c["NB"], c["bs"], c["Hk"], c["D"], generator=g).to(c["dtype"])
    dev = pools.cuda()
    width = width or max(len(p) for p in paths)
    acc = torch.tensor([list(p) + [99] * (width - len(p)) for p in paths], dtype=torch.int32).cuda()
    cnt = torch.tensor([len(p) for p in paths], dtype=torch.int32) if count is None else count
    new = torch.full((c["B"],), -5, dtype=torch.int32, device="cuda")
    op = op or handle(c)
    op.commit(pa.layer_pools([p[0] for p in dev], [p[1] for p in dev]),
              (c["table"] if table is None else table).cuda(), (c["past_t"] if past is None else past).cuda(), acc,
              cnt.cuda(), c["B"], new_past=new)
    err = op.device_error()
    flat = (layers, 2, c["NB"] * c["bs"], c["Hk"] * c["D"])
    return err, pools.view(flat), dev.cpu().view(flat), new.cpu()


@pytest.mark.parametrize("D,Hk,bs,dtype,layers", [(64, 1, 16, F16, 1), (256, 2, 32, F16, 2), (128, 8, 16, BF16, 3), (128, 2, 64, F16, 130),
                                                  (64, 5, 32, BF16, 7)])
def test_commit(D, Hk, bs, dtype, layers):
    c = tree_ref.make_case([0, 37, 14, 5, 300, 2], [1, 40, 256, 9, 3, 20], Hk, Hk, D, bs, dtype=dtype, seed=1)
    paths = [[0], list(range(0, 40, 3)), list(range(56, 256)), [], [1, 2], list(range(20))]
    err, before, after, new = commit(c, paths, layers)
    assert err == 0
    assert torch.equal(after, commit_ref(before, c, paths))
    assert new.tolist() == [p + len(a) for p, a in zip(c["past"], paths)]


def test_commit_leaves_bad_paths_and_unmapped_pages():
    c = tree_ref.make_case([10, 20, 30, 40], [20, 20, 20, 20], 2, 2, 64, 16, seed=1)
    op = handle(c)
    for paths, word in (([[1, 3], [2, 2], [4], [5]], "equal"), ([[1, 3], [5, 2], [4], [5]], "descending"),
                        ([[1, 3], [-1, 2], [4], [5]], "negative"), ([[1, 3], [2, 2 ** 31 - 1], [4], [5]], "far")):
        err, before, after, new = commit(c, paths, op=op)
        good = [p if b != 1 else [] for b, p in enumerate(paths)]
        assert err == pa.PA_DEVERR_ACCEPTED, word
        assert torch.equal(after, commit_ref(before, c, good)) and new.tolist() == [12, 20, 31, 41]
    paths = [[1, 3], [2], [4], [5]]
    err, before, after, new = commit(c, paths, op=op, count=torch.tensor([2, 3, 1, -1], dtype=torch.int32))
    assert err == pa.PA_DEVERR_ACCEPTED and new.tolist() == [12, 20, 31, 40]
    assert torch.equal(after, commit_ref(before, c, [[1, 3], [], [4], []]))
    err, before, after, new = commit(c, paths, op=op, past=torch.tensor([10, -20, 30, 40], dtype=torch.int32))
    assert err == pa.PA_DEVERR_PAST and new.tolist() == [12, -20, 31, 41]
    table = c["table"].clone()
    table[0, 0], table[1, 1] = -1, c["NB"] + 1
    err, before, after, new = commit(c, paths, op=op, table=table)
    assert err == pa.PA_DEVERR_BLOCK_ID
    assert torch.equal(after, commit_ref(before, {**c, "table": table.clamp(max=c["NB"])}, [[], [], [4], [5]]))


@pytest.mark.parametrize("path", [[-9, -5], [-1000000, -999999, -999998], [-5, -9, -3], [15, 0, 1], [1000, 0, 1, 2],
                                  [0, 5, 1, 2], [-2 ** 31, -2 ** 31 + 1], [2 ** 31 - 1, -1, 0]])
def test_commit_of_paths_that_ascend_only_in_places(path):
    """Entries that are above the one before them, but below their own place: nothing is looked up for them, also in
    the first and the last sequence, whose rows are the table's ends."""
    c = tree_ref.make_case([0, 20, 251], [20, 20, 5], 2, 2, 64, 16, seed=1)
    op = handle(c)
    for victim in range(3):
        paths = [[1, 3], [0, 2, 4], [1]]
        paths[victim] = path
        err, before, after, new = commit(c, paths, op=op)
        good = [p if b != victim else [] for b, p in enumerate(paths)]
        assert err == pa.PA_DEVERR_ACCEPTED
        assert torch.equal(after, commit_ref(before, c, good))
        assert new.tolist() == [p + len(a) for p, a in zip(c["past"], good)]


def test_commit_of_indexes_that_are_no_drafts():
    """An index at or above max_draft_tokens names no draft, although its slot may be mapped."""
    c = tree_ref.make_case([10, 20, 40], [20, 11, 9], 2, 2, 64, 16, seed=1)
    assert c["max_draft"] == 20 and c["MB"] * c["bs"] > 20 + 21
    op = handle(c)
    for bad in (20, 21):  # (slots 40 and 41 of the second sequence)
        paths = [[1, 3], [2, bad], [2]]
        err, before, after, new = commit(c, paths, op=op)
        assert err == pa.PA_DEVERR_ACCEPTED
        assert torch.equal(after, commit_ref(before, c, [[1, 3], [], [2]])) and new.tolist() == [12, 20, 41]
    err, before, after, new = commit(c, [[1, 19], [2], [2]], op=op)
    assert err == 0 and torch.equal(after, commit_ref(before, c, [[1, 19], [2], [2]]))


def test_commit_refusals():
    c = tree_ref.make_case([10], [20], 2, 2, 64, 16)
    op = handle(c)
    pool = torch.zeros(4, *c["key_cache"].shape, dtype=F16, device="cuda")
    table, past = c["table"].cuda(), c["past_t"].cuda()
    acc, cnt = torch.zeros(1, 20, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def refused(layers, word, acc=acc, batch=1, new_past=None):
        with pytest.raises(pa.PAError) as e:
            op.commit(layers, table, past, acc, cnt, batch, new_past=new_past)
        assert e.value.status == pa.PA_INVALID_ARGUMENT and word in e.value.message, e.value

    good = pa.layer_pools([pool[0], pool[2]], [pool[1], pool[3]])
    op.commit(good, table, past, acc, cnt, 1)
    refused(pa.layer_pools([pool[0], pool[2]], [pool[1], pool[2]]), "overlap")
    refused(pa.layer_pools([pool[0]], [pool.view(-1)[64:]]), "overlap")
    refused(pa.layer_pools([], []), "num_layers")
    refused(good, "batch", batch=2)
    refused(good, "max_accepted", acc=torch.zeros(1, 21, dtype=torch.int32, device="cuda"))
    refused(good, "new_past", new_past=past)
    with pytest.raises(pa.PAError):
        pa.layer_pools([pool[0]], [])
    assert op.device_error() == 0


def test_outputs_over_small_inputs_are_refused():
    """What a call writes may not be what it reads its lengths, pages or positions from."""
    c = tree_ref.make_case([33], [3], 4, 2, 64, 16, seed=53)
    op = handle(c)
    q, k, v, steps, rc = write_case(c, 64)
    st = pa.rotary_steps_tensor(steps)
    kc, vc = c["key_cache"].cuda(), c["value_cache"].cuda()
    out = torch.zeros_like(q)
    d = dict(steps=st, positions=c["pos"].cuda(), block_table=c["table"].cuda(), cum=c["cum"].cuda(), past=c["past_t"].cuda())
    names = dict(cum="cumulative_sequence_lengths", past="past_sequence_lengths")
    acc, cnt = torch.zeros(1, 3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")

    def refused(word, f, *a, **kw):
        with pytest.raises(pa.PAError) as e:
            f(*a, **kw)
        assert e.value.status == pa.PA_INVALID_ARGUMENT and word in e.value.message, e.value

    for name in d:
        for where, big in (("query_out", out), ("key_cache", kc), ("value_cache", vc)):
            t = dict(d)
            t[name] = big.view(-1).view(d[name].dtype)[8:8 + d[name].numel()].view(d[name].shape)
            refused(f"{where} must not overlap {names.get(name, name)}", op.write, rc, t["steps"], t["positions"], q, k, v, out,
                    kc, vc, t["block_table"], t["cum"], t["past"], 1, 3)
    layers = pa.layer_pools([kc], [vc])
    refused("new_past must not overlap block_table", op.commit, layers, d["block_table"], d["past"], acc, cnt, 1,
            new_past=d["block_table"].view(-1)[1:2])
    for pool in (kc, vc):
        refused("new_past must not overlap the pools", op.commit, layers, d["block_table"], d["past"], acc, cnt, 1,
                new_past=pool.view(-1).view(torch.int32)[40:41])
    assert op.device_error() == 0


# ---------------------------------------------------------------- one step after the other


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_a_speculative_step_equals_plain_decoding(dtype):
    """write, attention, commit over two rounds; afterwards the pool and the next round's attention are those of the
    accepted tokens written one after the other."""
    H, Hk, D, bs, past = 8, 2, 128, 16, [45, 3]
    c = tree_ref.make_case(past, [12, 20], H, Hk, D, bs, dtype=dtype, seed=11)
    op = handle(c)
    q, k, v, steps, rc = write_case(c, D, seed=3)
    st = pa.rotary_steps_tensor(steps)
    kc, vc = c["key_cache"].cuda(), c["value_cache"].cuda()
    out, qr = torch.empty_like(q), torch.empty_like(q)
    d = {n: c[n].cuda() for n in ("table", "cum", "past_t", "pos", "mask")}
    op.write(rc, st, d["pos"], q, k, v, qr, kc, vc, d["table"], d["cum"], d["past_t"], 2, c["T"])
    op.attention(qr, kc, vc, d["table"], d["cum"], d["past_t"], 2, c["T"], out, positions=d["pos"],
                 tree_mask=d["mask"])
    host = {**c, "query": qr.cpu(), "key_cache": kc.cpu(), "value_cache": vc.cpu()}
    ref, tol = tree_ref.attention(host)
    assert ((out.double().cpu().view(c["T"], H, D) - ref).abs() <= tol).all()
    # the deepest node of each tree and its ancestors
    paths = []
    for b in range(2):
        rows = c["rows"][int(c["cum"][b]):int(c["cum"][b + 1])]
        leaf = int(rows.sum(1).argmax())
        paths.append([i for i in range(rows.shape[1]) if rows[leaf, i]])
    width = max(map(len, paths))
    acc = torch.tensor([p + [0] * (width - len(p)) for p in paths], dtype=torch.int32).cuda()
    cnt = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
    new_past = torch.zeros(2, dtype=torch.int32, device="cuda")
    op.commit(pa.layer_pools([kc], [vc]), d["table"], d["past_t"], acc, cnt, 2, new_past=new_past)
    # the same tokens as a plain run: positions past, past + 1, ... and no mask
    n2 = [len(p) for p in paths]
    rows = torch.tensor([int(c["cum"][b]) + i for b, p in enumerate(paths) for i in p]).cuda()
    kc2, vc2 = c["key_cache"].cuda(), c["value_cache"].cuda()
    cum2 = torch.tensor([0, n2[0], sum(n2)], dtype=torch.int32).cuda()
    pos2 = torch.tensor([past[b] + i for b in range(2) for i in range(n2[b])], dtype=torch.int32).cuda()
    q2 = torch.empty(sum(n2), H * D, dtype=dtype, device="cuda")
    op.write(rc, st, pos2, q[rows], k[rows], v[rows], q2, kc2, vc2, d["table"], cum2, d["past_t"], 2, sum(n2))
    assert torch.equal(q2, qr[rows])
    for b in range(2):
        for p in range(past[b] + n2[b]):
            slot = int(c["table"][b, p // bs]) * bs + p % bs
            for x, y in ((kc, kc2), (vc, vc2)):
                assert torch.equal(x.view(-1, Hk, D)[slot], y.view(-1, Hk, D)[slot])
    assert new_past.tolist() == [p + m for p, m in zip(past, n2)]
    # the accepted rows' outputs are those of plain causal decoding
    out2 = torch.empty_like(q2)
    op.attention(q2, kc2, vc2, d["table"], cum2, d["past_t"], 2, sum(n2), out2)
    both = tol.view(c["T"], -1)[rows.cpu()] * 2
    assert ((out2.double().cpu() - out[rows].double().cpu()).abs() <= both).all()
    assert op.device_error() == 0


# ---------------------------------------------------------------- how the calls are made


def test_pools_beyond_32_bits():
    """Pools of more than 2^32 elements whose used blocks lie at their end."""
    H, Hk, D, bs, past, n = 8, 8, 128, 128, [200, 30], [4, 6]
    c = tree_ref.make_case(past, n, H, Hk, D, bs, seed=21)
    NB = 2 ** 32 // (bs * Hk * D) + 9
    far = NB - c["NB"]
    kc, vc = (torch.empty(NB, bs, Hk, D, dtype=F16, device="cuda") for _ in range(2))
    kc[far:], vc[far:] = c["key_cache"].cuda(), c["value_cache"].cuda()
    cfg = pa.make_config(H, Hk, D, bs, NB, c["MB"], 2, c["T"])
    op = pa.PagedTree(cfg, c["max_draft"])
    table = torch.where(c["table"] >= 0, c["table"] + far, c["table"]).cuda()
    d = {k: c[k].cuda() for k in ("query", "cum", "past_t", "pos", "mask")}
    out = torch.empty(c["T"], H * D, dtype=F16, device="cuda")
    op.attention(d["query"], kc, vc, table, d["cum"], d["past_t"], 2, c["T"], out, positions=d["pos"],
                 tree_mask=d["mask"])
    ref, tol = tree_ref.attention(c)
    assert ((out.double().cpu().view(c["T"], H, D) - ref).abs() <= tol).all()
    q, k, v, steps, rc = write_case(c, D)
    qo, before_v = torch.empty_like(q), vc[far:].clone()
    op.write(rc, pa.rotary_steps_tensor(steps), d["pos"], q, k, v, qo, kc, vc, table, d["cum"], d["past_t"], 2, c["T"])
    for b in range(2):
        for j in range(n[b]):
            p = past[b] + j
            slot = int(c["table"][b, p // bs]) * bs + p % bs
            before_v.view(-1, Hk * D)[slot] = v[int(c["cum"][b]) + j]
    assert torch.equal(vc[far:].view(torch.int16), before_v.view(torch.int16))  # (bits: unused slots are NaN)
    acc = torch.tensor([[1, 3], [2, 5]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    op.commit(pa.layer_pools([kc], [vc]), table, d["past_t"], acc, cnt, 2)
    for b, path in enumerate(acc.tolist()):
        for i, a in enumerate(path):
            to, of = (int(c["table"][b, p // bs]) * bs + p % bs for p in (past[b] + i, past[b] + a))
            assert torch.equal(vc[far:].view(-1, Hk * D)[to], before_v.view(-1, Hk * D)[of])
    assert op.device_error() == 0


def test_two_handles_at_once_on_two_streams():
    """A handle per stream: steps that overlap on the GPU give what they give alone."""
    cs = [tree_ref.make_case([3000, 900], [20, 8], 8, 2, 128, 16, dtype=BF16, seed=31),
          tree_ref.make_case([500, 2500, 7], [5, 7, 8], 4, 1, 64, 32, seed=32)]
    ops = [handle(c) for c in cs]
    dev = [{k: cuda(c[k]) for k in ("query", "key_cache", "value_cache", "table", "cum", "past_t", "positions", "mask")}
           for c in cs]
    alone = [attend(c, op)[1] for c, op in zip(cs, ops)]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[torch.empty_like(a) for _ in range(20)] for a in alone]
    torch.cuda.synchronize()
    for i in range(20):
        for c, op, d, s, o in zip(cs, ops, dev, streams, outs):
            op.attention(d["query"], d["key_cache"], d["value_cache"], d["table"], d["cum"], d["past_t"], c["B"],
                         c["T"], o[i], positions=d["positions"], tree_mask=d["mask"], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(a, x) for x in o)
    assert all(op.device_error() == 0 for op in ops)


def test_a_captured_step_replays():
    """write, attention and commit in one graph, replayed on new tokens."""
    c = tree_ref.make_case([300, 45], [9, 12], 4, 2, 128, 16, seed=41)
    op = handle(c)
    q, k, v, steps, rc = write_case(c, 128)
    st = pa.rotary_steps_tensor(steps)
    d = {n: c[n].cuda() for n in ("table", "cum", "past_t", "pos", "mask")}
    kc, vc = c["key_cache"].cuda(), c["value_cache"].cuda()
    qr, out, new = torch.empty_like(q), torch.empty_like(q), torch.zeros(2, dtype=torch.int32, device="cuda")
    acc = torch.tensor([[0, 2, 5], [0, 1, 0]], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    layers = pa.layer_pools([kc], [vc])

    def step(s):
        op.write(rc, st, d["pos"], q, k, v, qr, kc, vc, d["table"], d["cum"], d["past_t"], 2, c["T"], stream=s)
        op.attention(qr, kc, vc, d["table"], d["cum"], d["past_t"], 2, c["T"], out, positions=d["pos"],
                     tree_mask=d["mask"], stream=s)
        op.commit(layers, d["table"], d["past_t"], acc, cnt, 2, new_past=new, stream=s)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(s.cuda_stream)
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda").to(F16))
        kc.copy_(c["key_cache"].cuda())
        vc.copy_(c["value_cache"].cuda())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qr, out, kc, vc, new)]
        kc.copy_(c["key_cache"].cuda())
        vc.copy_(c["value_cache"].cuda())
        step(None)
        torch.cuda.synchronize()
        for a, b in zip(got, (qr, out, kc, vc, new)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert op.device_error() == 0


def test_write_in_place_and_single_rows():
    c = tree_ref.make_case([33], [1], 4, 2, 64, 16, seed=51)
    op = handle(c)
    q, k, v, steps, rc = write_case(c, 64, packed=True)
    st = pa.rotary_steps_tensor(steps)
    kc, vc = c["key_cache"].cuda(), c["value_cache"].cuda()
    args = (kc, vc, c["table"].cuda(), c["cum"].cuda(), c["past_t"].cuda(), 1, 1)
    out = torch.empty(1, 256, dtype=F16, device="cuda")
    op.write(rc, st, c["pos"].cuda(), q, k, v, out, *args)
    q2 = q.clone()
    op.write(rc, st, c["pos"].cuda(), q2, k, v, q2, *args)
    assert torch.equal(out, q2) and op.device_error() == 0


def test_refusals_of_calls():
    c = tree_ref.make_case([33], [3], 4, 2, 64, 16, seed=52)
    op = handle(c)
    q, k, v, steps, rc = write_case(c, 64)
    st = pa.rotary_steps_tensor(steps)
    d = {n: c[n].cuda() for n in ("table", "cum", "past_t", "pos")}
    kc, vc = c["key_cache"].cuda(), c["value_cache"].cuda()
    out = torch.empty_like(q)

    def refused(word, f, *a, **kw):
        with pytest.raises(pa.PAError) as e:
            f(*a, **kw)
        assert e.value.status == pa.PA_INVALID_ARGUMENT and word in e.value.message, e.value

    w = lambda **o: [o.get("rc", rc), st, d["pos"], o.get("q", q), k, v, o.get("out", out), o.get("kc", kc),  # noqa: E731
                     o.get("vc", vc), d["table"], d["cum"], d["past_t"], o.get("batch", 1), o.get("T", 3)]
    refused("head_size and dtype", op.write, *w(rc=pa.make_rotary_config(128)))
    refused("head_size and dtype", op.write, *w(rc=pa.make_rotary_config(64, dtype=pa.PA_ROTARY_BF16)))
    refused("batch", op.write, *w(batch=2))
    refused("token_count", op.write, *w(T=4))
    refused("distinct", op.write, *w(vc=kc))
    refused("query_out", op.write, *w(out=k))
    refused("pools", op.write, *w(out=kc.view(-1, 256)[:3]))
    refused("2-D", op.write, *w(q=q.view(3, 4, 64)))
    a = lambda **o: [o.get("q", q), o.get("kc", kc), vc, d["table"], d["cum"], d["past_t"], o.get("batch", 1),  # noqa: E731
                     o.get("T", 3), o.get("out", out)]
    refused("contiguous", op.write, *w(out=torch.empty(3, 300, dtype=F16, device="cuda")[:, :256]))
    refused("contiguous", op.attention, *a(out=torch.empty(3, 300, dtype=F16, device="cuda")[:, :256]))
    refused("contiguous", op.attention, *a(q=torch.empty(3, 300, dtype=F16, device="cuda")[:, :256]))
    refused("output", op.attention, *a(out=q))
    refused("output", op.attention, *a(out=kc.view(-1, 256)[:3]))
    refused("positions", op.attention, *a(), positions=out.view(torch.int32).view(-1)[8:])
    refused("tree_mask", op.attention, *a(), tree_mask=out.view(torch.int32).view(-1)[100:])
    refused("distance_slopes", op.attention, *a(), distance_slopes=out.view(torch.float32).view(-1)[20:])
    refused("head_sink", op.attention, *a(), head_sink=out.view(-1)[:4])
    refused("batch", op.attention, *a(batch=0))
    refused("token_count", op.attention, *a(T=4))
    refused("aligned", op.attention, *a(out=torch.empty(3 * 256 + 1, dtype=F16, device="cuda")[1:]))
    refused("distinct", op.attention, *a(kc=vc))
    op.attention(*a(T=0))
    op.write(*w(T=0))
    assert op.device_error() == 0
