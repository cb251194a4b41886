"""Types and sizes that the 4-bit and page calls refuse before a kernel could read them as something else (no GPU)."""

import pytest
import torch

import paged_kv_cache_reshape_gb300 as pa
from paged_kv_cache_reshape_gb300 import builder as pabuild


@pytest.fixture(scope="module", autouse=True)
def built():
    pabuild.build()


def refused(word, f, *a, **kw):
    with pytest.raises(pa.PAError) as e:
        f(*a, **kw)
    assert e.value.status == pa.PA_INVALID_ARGUMENT and word in e.value.message, e.value


def i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def paged(**change):
    t = dict(key_cache=torch.zeros(5, 2, 576, dtype=torch.uint8), value_cache=torch.zeros(5, 2, 576, dtype=torch.uint8),
             block_table=i32(2, 3), cum=i32(3), past=i32(2))
    t.update(change)
    return [t[k] for k in ("key_cache", "value_cache", "block_table", "cum", "past")]


def rows(T=4, width=128, dtype=torch.float16):
    return torch.zeros(T, width, dtype=dtype)


SIZES = (3, 5 * 2 * 576, torch.float16, 128)  # columns, bytes of a pool, rows' type and width


def each_call(word, tensors, a=None, b=None, sizes=SIZES):
    a, b = rows() if a is None else a, rows() if b is None else b
    refused(word, pa.pa_q4_write, None, a, b, *tensors, 2, 4, sizes=sizes)
    refused(word, pa.pa_q4_read, None, *tensors, 2, 4, a, b, sizes=sizes)
    refused(word, pa.pa_q4_attention, None, a, *tensors, 2, 4, b, sizes=sizes)


def test_good_calls_reach_the_library():
    each_call("handle", paged())
    each_call("handle", paged(), sizes=None)
    each_call("handle", paged(block_table=i32(7, 3), cum=i32(9), past=i32(4)), rows(6), rows(5))


@pytest.mark.parametrize("which", ["block_table", "cum", "past"])
@pytest.mark.parametrize("sizes", [SIZES, None])
def test_whole_numbers_of_another_type(which, sizes):
    t = dict(block_table=i32(2, 3), cum=i32(3), past=i32(2))
    each_call("int32", paged(**{which: t[which].long()}), sizes=sizes)
    each_call("int32", paged(**{which: t[which].to(torch.int16)}), sizes=sizes)


@pytest.mark.parametrize("sizes", [SIZES, None])
def test_too_few_lengths(sizes):
    each_call("batch", paged(cum=i32(2)), sizes=sizes)
    each_call("batch", paged(past=i32(1)), sizes=sizes)


def test_tables_of_other_columns_or_too_few_rows():
    for table in (i32(2, 4), i32(2, 2), i32(1, 3), i32(6), i32(2, 3, 1)):
        each_call("columns", paged(block_table=table))


def test_pools_of_another_size_or_type():
    for pool in (torch.zeros(4, 2, 576, dtype=torch.uint8), torch.zeros(5, 2, 576, dtype=torch.float16),
                 torch.zeros(5, 2, 1152, dtype=torch.uint8)):
        each_call("bytes", paged(key_cache=pool))
        each_call("bytes", paged(value_cache=pool))


def test_rows_of_another_type_or_too_few():
    for k in range(2):
        for dtype in (torch.bfloat16, torch.float32):
            x = [rows(), rows()]
            x[k] = rows(dtype=dtype)
            each_call("float16", paged(), *x)
        x = [rows(), rows()]
        x[k] = rows(3)
        each_call("rows", paged(), *x)


def test_page_calls_with_whole_numbers_of_another_type():
    pools = pa.page_pools([i32(10, 16)])
    cases = [(pa.pa_pages_copy, [i32(4), i32(4)]),
             (pa.pa_pages_fork, [i32(3, 4), i32(3), i32(2), i32(10), i32(2, 4), i32(2), i32(10)]),
             (pa.pa_pages_resize, [i32(3, 4), i32(3), i32(3), i32(3), i32(10)]),
             (pa.pa_pages_compact, [i32(3, 4), i32(10), i32(3, 4), i32(10), i32(1)])]
    for f, good in cases:
        refused("handle", f, None, pools, *good)
        for k, t in enumerate(good):
            refused("int32", f, None, pools, *good[:k], t.long(), *good[k + 1:])
