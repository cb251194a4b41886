"""Host-side checks of the tree operators that need no GPU: frequencies, and every refusal by name."""

import ctypes
import math

import pytest

import paged_kv_cache_reshape_gb300 as pa
from paged_kv_cache_reshape_gb300 import builder as pabuild

A = 1 << 20  # a fake, suitably aligned "device address" (never dereferenced)


@pytest.fixture(scope="module", autouse=True)
def built():
    pabuild.build()


def turns(f):
    return round(f / (2 * math.pi) * 2.0 ** 64)


@pytest.mark.parametrize("R", [2, 16, 64, 128, 512])
def test_steps_unscaled_and_linear(R):
    for kind, s in ((pa.PA_ROTARY_SCALE_NONE, 1.0), (pa.PA_ROTARY_SCALE_LINEAR, 4.0)):
        steps, m = pa.pa_rotary_steps(R, kind, base=10000.0, factor=s)
        assert m == 1.0 and len(steps) == R // 2
        for i, v in enumerate(steps):
            want = turns(10000.0 ** (-2.0 * i / R) / s)
            # pow, divide, pi: a few half steps of a double; both sides round to whole numbers, half a unit each
            assert abs(v - want) <= 8 * 2.0 ** -52 * want + 1


def test_steps_of_the_scalings():
    """Ends and middles of the ramps, worked out by hand for R = 8, base 10000, L = 2 pi 1000."""
    R, base, s, L = 8, 10000.0, 4.0, 2 * math.pi * 1000.0
    f = [1.0, 0.1, 0.01, 0.001]
    steps, m = pa.pa_rotary_steps(R, pa.PA_ROTARY_SCALE_BASE, base=base, factor=s)
    for i, v in enumerate(steps):
        want = turns((base * s ** (8 / 6)) ** (-i / 4))
        assert abs(v - want) <= 1e-14 * want and m == 1.0
    # by wavelength: turns over L are 1000, 100, 10, 1; the ramp runs from 5 to 20
    steps, m = pa.pa_rotary_steps(R, pa.PA_ROTARY_SCALE_BY_WAVELENGTH, base=base, factor=s, original_positions=L,
                                  low=5.0, high=20.0)
    k = [1.0, 1.0, 1 / 3, 0.0]
    for i, v in enumerate(steps):
        want = turns(f[i] * (k[i] + (1 - k[i]) / s))
        assert abs(v - want) <= 1e-13 * want and m == 1.0
    # by parts: at(turns) = 8 ln(1000 / turns) / (2 ln 10000): at(100) = 1, at(1) = 3
    steps, m = pa.pa_rotary_steps(R, pa.PA_ROTARY_SCALE_BY_PARTS, base=base, factor=s, original_positions=L,
                                  low=1.01, high=99.0)
    r = [0.0, 0.0, 0.5, 1.0]  # lo = floor(1.004) = 1, hi = ceil(2.996) = 3
    for i, v in enumerate(steps):
        want = turns(f[i] * (1 - r[i]) + f[i] / s * r[i])
        assert abs(v - want) <= 1e-13 * want
    assert abs(m - (0.1 * math.log(s) + 1.0)) < 1e-6


@pytest.mark.parametrize("over,word", [
    (dict(rotary_dim=0), "rotary_dim"), (dict(rotary_dim=7), "rotary_dim"), (dict(rotary_dim=514), "rotary_dim"),
    (dict(type=5), "type"), (dict(type=-1), "type"), (dict(base=1.0), "base"), (dict(base=math.inf), "base"),
    (dict(type=1, factor=0.5), "factor"), (dict(type=1, factor=math.nan), "factor"),
    (dict(type=3, original_positions=0.0), "original_positions"),
    (dict(type=4, original_positions=8192.0, low=4.0, high=4.0), "low"),
    (dict(type=4, original_positions=8192.0, low=0.0, high=4.0), "low"),
])
def test_steps_refusals(over, word):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rotary_steps(**{**dict(rotary_dim=64, type=0), **over})
    assert e.value.status == pa.PA_INVALID_ARGUMENT and word in e.value.message


def rotary(rc=None, **over):
    rc = rc or pa.make_rotary_config(64)
    d = dict(steps=A, positions=A + 4096, token_count=3, num_heads=2, query=A + (1 << 16), query_stride=0,
             query_out=A + (1 << 17), query_out_stride=0, kv_num_heads=1, key=A + (1 << 18), key_stride=0,
             key_out=A + (1 << 19), key_out_stride=0)
    d.update(over)
    st = pa.lib().pa_rotary(rc, *d.values(), None)
    return st, pa.pa_last_error_message()


@pytest.mark.parametrize("over,word", [
    (dict(token_count=-1), "token_count"), (dict(num_heads=-1), "num_heads"),
    (dict(kv_num_heads=4097), "kv_num_heads"), (dict(steps=None), "steps"),
    (dict(steps=A + 4), "steps"), (dict(positions=None), "positions"), (dict(query=None), "query"),
    (dict(query=A + 8), "query"), (dict(query_out=None), "query_out"), (dict(key=None), "key"),
    (dict(key_out=None), "key_out"), (dict(query_stride=120), "query"), (dict(query_stride=132), "query"),
    (dict(key_out_stride=-64), "key_out"),
    (dict(query_out=A + (1 << 16) + 256), "query_out overlaps query"),
    (dict(key_out=A + (1 << 17)), "must not overlap"), (dict(key_out=A + (1 << 16)), "must not overlap"),
])
def test_rotary_refusals(over, word):
    st, msg = rotary(**over)
    assert st == pa.PA_INVALID_ARGUMENT and word in msg, (st, msg)


@pytest.mark.parametrize("over,word", [
    (dict(head_size=0), "head_size"), (dict(head_size=12), "head_size"), (dict(head_size=520), "head_size"),
    (dict(rotary_dim=24), "rotary_dim"), (dict(rotary_dim=80), "rotary_dim"), (dict(rotary_offset=4), "rotary_offset"),
    (dict(rotary_offset=8), "rotary_offset"), (dict(interleaved=2), "interleaved"), (dict(conjugate=-1), "conjugate"),
    (dict(dtype=3), "dtype"), (dict(attention_factor=math.inf), "attention_factor"),
    (dict(attention_factor=math.nan), "attention_factor"),
])
def test_rotary_config_refusals(over, word):
    st, msg = rotary(pa.make_rotary_config(**{**dict(head_size=64), **over}))
    assert st == pa.PA_INVALID_ARGUMENT and word in msg, (st, msg)


def test_rotary_of_nothing():
    assert rotary(token_count=0)[0] == pa.PA_OK
    assert rotary(num_heads=0, kv_num_heads=0)[0] == pa.PA_OK


def cfg(**over):
    c = pa.make_config(32, 8, 128, 16, 1000, 257, 64, 64)
    for k, v in over.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("over,draft,status,word", [
    (dict(num_heads=30), 8, pa.PA_INVALID_ARGUMENT, "num_heads"), (dict(), 0, pa.PA_INVALID_ARGUMENT, "max_draft"),
    (dict(), 257, pa.PA_INVALID_ARGUMENT, "max_draft"), (dict(head_size=96), 8, pa.PA_NOT_SUPPORTED, "head_size"),
    (dict(num_heads=8192), 8, pa.PA_NOT_SUPPORTED, "num_heads"),
    (dict(cache_dtype=pa.PA_CACHE_INT8, k_quant_type=1, v_quant_type=1), 8, pa.PA_NOT_SUPPORTED, "cache_dtype"),
    (dict(packed_qkv=1), 8, pa.PA_NOT_SUPPORTED, "packed_qkv"), (dict(qk_norm=1), 8, pa.PA_NOT_SUPPORTED, "qk_norm"),
    (dict(block_size=8), 8, pa.PA_INVALID_ARGUMENT, "block_size"),
    (dict(kv_cache_layout=1, kv_num_heads=1, head_size=576, v_head_size=512, scale=0.1, num_heads=16), 8,
     pa.PA_NOT_SUPPORTED, "separate"),
])
def test_tree_create_refusals(over, draft, status, word):
    with pytest.raises(pa.PAError) as e:
        pa.pa_tree_create(cfg(**over), draft)
    assert e.value.status == status and word in e.value.message, e.value


def test_tree_create_without_gpu_and_null_handles():
    import torch
    if not torch.cuda.is_available():
        with pytest.raises(pa.PAError) as e:
            pa.pa_tree_create(cfg(do_rotary=1, max_rotary_positions=0), 8)  # the layer's rotary is not read
        assert e.value.status == pa.PA_CUDA_ERROR
    L = pa.lib()
    assert L.pa_tree_destroy(None) == pa.PA_OK
    code = ctypes.c_int()
    assert L.pa_tree_check_device_error(None, ctypes.byref(code)) == pa.PA_INVALID_ARGUMENT
    assert L.pa_tree_attention(None, A, A, A, A, A, A, 1, 1, None, A, None) == pa.PA_INVALID_ARGUMENT
    assert L.pa_tree_write(None, pa.make_rotary_config(64), A, A, A, 0, A, 0, A, 0, A, A, A, A, A, A, 1, 1,
                           None) == pa.PA_INVALID_ARGUMENT
    assert L.pa_tree_commit(None, None, None, 1, A, A, A, A, 1, 1, None, None) == pa.PA_INVALID_ARGUMENT
    assert "handle" in L.pa_tree_last_error_message(None).decode()


def rows(T=3, width=128):
    import torch
    return torch.zeros(T, width, dtype=torch.float16)


def refused(word, f, *a, **kw):
    with pytest.raises(pa.PAError) as e:
        f(*a, **kw)
    assert e.value.status == pa.PA_INVALID_ARGUMENT and word in e.value.message, e.value


@pytest.mark.parametrize("which", ["query", "query_out", "key", "key_out"])
def test_rotary_refuses_rows_expanded_from_one(which):
    """A broadcast row has a stride of 0, which in the C call stands for dense rows."""
    import torch
    t = dict(query=rows(), query_out=rows(), key=rows(), key_out=rows())
    t[which] = rows(1).expand(3, 128)
    refused("stride", pa.pa_rotary, pa.make_rotary_config(64), torch.zeros(32, dtype=torch.int64),
            torch.zeros(3, dtype=torch.int32), 3, 2, t["query"], t["query_out"], 2, t["key"], t["key_out"])


@pytest.mark.parametrize("which", ["query", "key", "value"])
def test_write_refuses_rows_expanded_from_one(which):
    import torch
    t = dict(query=rows(), key=rows(), value=rows())
    t[which] = rows(1).expand(3, 128)
    i32 = torch.zeros(4, dtype=torch.int32)
    refused("stride", pa.pa_tree_write, None, pa.make_rotary_config(64), torch.zeros(32, dtype=torch.int64), i32,
            t["query"], t["key"], t["value"], rows(), rows(), rows(), i32.view(2, 2), i32, i32, 1, 3)


def test_single_rows_have_no_stride():
    """One row may be a slice of anything, an expanded one too: the calls go on to the next check."""
    import torch
    one = rows(1, 256)[:, :128]
    refused("token_count", pa.pa_rotary, pa.make_rotary_config(64), torch.zeros(32, dtype=torch.int64),
            torch.zeros(3, dtype=torch.int32), -1, 2, one, one, 2, rows(1).expand(1, 128), one)


def sliced(*size, dtype=None):
    """A view of that size with gaps between its rows."""
    import torch
    big = torch.zeros(size[0], *(2 * s for s in size[1:]), dtype=dtype or torch.int32)
    return big[tuple(slice(0, s) for s in size)] if len(size) > 1 else torch.zeros(2 * size[0], dtype=big.dtype)[::2]


@pytest.mark.parametrize("which", ["steps", "positions", "key_cache", "value_cache", "block_table", "cum", "past"])
def test_write_refuses_tensors_with_gaps(which):
    """A slice of a wider block table, or one side of interleaved pools, is not what the C call takes it for."""
    import torch
    i32 = torch.zeros(4, dtype=torch.int32)
    t = dict(steps=torch.zeros(32, dtype=torch.int64), positions=i32, key_cache=torch.zeros(2, 16, 2, 64),
             value_cache=torch.zeros(2, 16, 2, 64), block_table=i32.view(2, 2), cum=i32, past=i32)
    t[which] = sliced(*t[which].shape, dtype=t[which].dtype)
    refused("contiguous", pa.pa_tree_write, None, pa.make_rotary_config(64), t["steps"], t["positions"], rows(), rows(),
            rows(), rows(), t["key_cache"], t["value_cache"], t["block_table"], t["cum"], t["past"], 1, 3)


@pytest.mark.parametrize("which", ["key_cache", "value_cache", "block_table", "cum", "past", "positions", "tree_mask",
                                   "distance_slopes", "head_sink"])
def test_attention_refuses_tensors_with_gaps(which):
    import torch
    i32 = torch.zeros(4, dtype=torch.int32)
    t = dict(key_cache=torch.zeros(2, 16, 2, 64), value_cache=torch.zeros(2, 16, 2, 64), block_table=i32.view(2, 2),
             cum=i32, past=i32, positions=i32, tree_mask=i32.view(2, 2), distance_slopes=torch.zeros(4),
             head_sink=torch.zeros(4))
    t[which] = sliced(*t[which].shape, dtype=t[which].dtype)
    refused("contiguous", pa.pa_tree_attention, None, rows(), t["key_cache"], t["value_cache"], t["block_table"],
            t["cum"], t["past"], 1, 3, rows(), positions=t["positions"], tree_mask=t["tree_mask"],
            distance_slopes=t["distance_slopes"], head_sink=t["head_sink"])


@pytest.mark.parametrize("which", ["block_table", "past", "accepted", "count", "new_past"])
def test_commit_refuses_tensors_with_gaps(which):
    import torch
    i32 = torch.zeros(4, dtype=torch.int32)
    t = dict(block_table=i32.view(2, 2), past=i32, accepted=i32.view(2, 2), count=i32, new_past=i32)
    t[which] = sliced(*t[which].shape)
    layers = pa.layer_pools([torch.zeros(2, 16, 2, 64)], [torch.zeros(2, 16, 2, 64)])
    refused("contiguous", pa.pa_tree_commit, None, layers, t["block_table"], t["past"], t["accepted"], t["count"], 1,
            new_past=t["new_past"])


def test_rotary_and_layer_pools_refuse_tensors_with_gaps():
    import torch
    pool = torch.zeros(3, 2, 16, 2, 64)
    refused("contiguous", pa.layer_pools, [pool[:, 0]], [pool[0]])
    refused("contiguous", pa.layer_pools, [pool[0]], [pool[:, 1]])
    q, i32 = rows(), torch.zeros(3, dtype=torch.int32)
    steps = torch.zeros(32, dtype=torch.int64)
    refused("contiguous", pa.pa_rotary, pa.make_rotary_config(64), sliced(32, dtype=torch.int64), i32, 3, 2, q, q)
    refused("contiguous", pa.pa_rotary, pa.make_rotary_config(64), steps, sliced(3), 3, 2, q, q)


@pytest.mark.parametrize("over,word", [
    (dict(positions=A + (1 << 17)), "query_out must not overlap positions"),
    (dict(positions=A + (1 << 19) + 380), "key_out must not overlap positions"),
    (dict(steps=A + (1 << 17) + 760), "query_out must not overlap steps"),
    (dict(steps=A + (1 << 19) - 248), "key_out must not overlap steps"),
])
def test_rotary_refuses_outputs_over_its_tables(over, word):
    st, msg = rotary(**over)
    assert st == pa.PA_INVALID_ARGUMENT and word in msg, (st, msg)
