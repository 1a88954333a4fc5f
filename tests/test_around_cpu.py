"""C-ABI and binding checks of the operators around the decode that need no
GPU: struct layouts, the rotary table, and every refusal, made on the host
before any CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import around_ref as ar

from test_abi_cpu import api, declared_functions

INVALID, UNSUPPORTED = 1, 2
NEW = ("sparse_mla_rope_init", "sparse_mla_rope", "sparse_mla_cache_append", "sparse_mla_attn_weights",
       "sparse_mla_accumulate_weights", "sparse_mla_evict_select", "sparse_mla_evict_compact", "sparse_mla_evict")


def test_entry_points_are_declared_and_bound():
    assert set(NEW) <= set(declared_functions())
    for n in NEW:
        assert getattr(api.lib, n).argtypes is not None


def test_struct_layouts():
    assert ctypes.sizeof(api.RopeTableData) == 16 + 8 * 128 and api.RopeTableData.step.offset == 16
    assert ctypes.sizeof(api.RopeConfig) == 56 and api.RopeConfig.base.offset == 16
    assert ctypes.sizeof(api.RopeShape) == 64 and api.RopeShape.x_token_stride.offset == 32
    assert ctypes.sizeof(api.AppendShape) == 56 and api.AppendShape.x_dtype.offset == 24
    assert ctypes.sizeof(api.EvictShape) == 48 and api.EvictShape.num_kv_rows.offset == 32


# ------------------------------------------------------------ rotary table
@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(rope_dim=2), dict(rope_dim=256), dict(rope_dim=74, interleaved=False),
    dict(scaling="linear", factor=8.0), dict(scaling="linear", factor=0.05),
    dict(scaling="yarn", factor=40.0, original_ctx=4096),
    dict(scaling="yarn", factor=4.0, original_ctx=32768, beta_fast=16.0, beta_slow=2.0, base=1000000.0),
])
def test_rope_table_holds_the_frequencies(kw):
    t = api.RopeTable(**kw)
    dim = kw.get("rope_dim", 64)
    f = ar.rope_frequencies(dim, **{k: v for k, v in kw.items() if k not in ("rope_dim", "interleaved")})
    turns = np.array(t.turns())
    want = f / (2 * math.pi) % 1.0
    # double arithmetic of the reference side: pow within 2 ulp, three more roundings; the table within 2^-65
    assert np.abs(turns - want).max() <= 8 * 2.0 ** -53
    # far positions: the fraction of a turn at position 2^20 by exact integer arithmetic
    far = np.array([(t.data.step[i] << 20) % (1 << 64) / 2.0 ** 64 for i in range(dim // 2)])
    d = np.abs(far - (f / (2 * math.pi) * 2.0 ** 20) % 1.0)
    assert np.minimum(d, 1 - d).max() <= 2.0 ** 20 * 8 * 2.0 ** -53


@pytest.mark.parametrize("kw", [dict(rope_dim=0), dict(rope_dim=3), dict(rope_dim=258), dict(base=0.0),
                                dict(base=math.nan), dict(mscale=math.inf), dict(scaling="linear", factor=0.0),
                                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_ctx=10, base=1.0),
                                dict(scaling="yarn", factor=2.0, original_ctx=10, beta_slow=0.0)])
def test_bad_rope_tables_are_refused(kw):
    with pytest.raises(api.SmlaError) as e:
        api.RopeTable(**kw)
    assert e.value.code == INVALID
    with pytest.raises(ValueError):
        api.RopeTable(scaling="other")


def _table(**kw):
    t = api.RopeTable(**kw).data
    return ctypes.byref(t)


def _rope_shape(**kw):
    d = dict(tokens=4, heads=2, dim=64, offset=0, dtype=0, transpose=0, reserved=0, x_token_stride=128,
             x_head_stride=64, y_token_stride=128, y_head_stride=64)
    d.update(kw)
    return ctypes.byref(api.RopeShape(*d.values()))


def test_rope_refusals():
    f = api.lib.sparse_mla_rope
    t = _table()
    for kw in (dict(tokens=-1), dict(heads=0), dict(heads=65537), dict(dim=1), dict(dim=63), dict(offset=1),
               dict(offset=-1), dict(transpose=2), dict(reserved=1), dict(y_head_stride=0), dict(y_head_stride=63),
               dict(y_token_stride=0), dict(y_token_stride=127), dict(y_token_stride=64), dict(y_head_stride=128),
               dict(y_head_stride=-63), dict(tokens=1, y_head_stride=63), dict(heads=1, y_token_stride=63)):
        assert f(_rope_shape(**kw), t, 16, 16, 32, None) == INVALID, kw
    assert f(_rope_shape(dtype=3), t, 16, 16, 32, None) == UNSUPPORTED
    assert f(None, t, 16, 16, 32, None) == INVALID and f(_rope_shape(), None, 16, 16, 32, None) == INVALID
    for x, p, y in ((None, 16, 32), (16, None, 32), (16, 16, None), (17, 16, 32), (16, 18, 32), (16, 16, 33)):
        assert f(_rope_shape(), t, x, p, y, None) == INVALID
    assert f(_rope_shape(dtype=2), t, 18, 16, 32, None) == INVALID           # fp32 elements need 4 bytes
    assert f(_rope_shape(x_token_stride=256), t, 32, 16, 32, None) == INVALID   # in place with other strides
    assert f(_rope_shape(tokens=0), t, None, None, None, None) == 0           # nothing to do
    assert f(_rope_shape(tokens=0, y_head_stride=64, y_token_stride=128), t, None, None, None, None) == 0
    bad = api.RopeTableData()
    assert f(_rope_shape(), ctypes.byref(bad), 16, 16, 32, None) == INVALID


def _append_shape(**kw):
    d = dict(tokens=4, x_stride=576, num_kv_rows=640, x_dtype=0, kv_dtype=0, page_size=0, pages_per_seq=0, batch=0,
             eps=1e-6, reserved=0)
    d.update(kw)
    return ctypes.byref(api.AppendShape(*d.values()))


def _append(shape, x=16, w=16, table=None, pos=None, slots=16, seq=None, pt=None, kv=16, rs=None):
    return api.lib.sparse_mla_cache_append(shape, x, w, table, pos, slots, seq, pt, kv, rs, None)


def test_append_refusals():
    paged = dict(page_size=64, pages_per_seq=4, batch=2)
    for kw in (dict(tokens=-1), dict(x_stride=575), dict(num_kv_rows=0), dict(num_kv_rows=1 << 31), dict(reserved=1),
               dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(page_size=64, batch=2),
               dict(page_size=64, pages_per_seq=4)):
        assert _append(_append_shape(**kw), pt=16) == INVALID, kw
    for kw in (dict(kv_dtype=3), dict(x_dtype=3), dict(page_size=32), dict(kv_dtype=2), dict(kv_dtype=2, num_kv_rows=100, **paged)):
        assert _append(_append_shape(**kw), pt=16) == UNSUPPORTED, kw
    ok = _append_shape()
    assert _append(None) == INVALID
    for kw in (dict(x=None), dict(slots=None), dict(kv=None), dict(kv=8), dict(x=17), dict(slots=18), dict(w=8),
               dict(table=_table()), dict(table=_table(), pos=18), dict(rs=16)):
        assert _append(ok, **kw) == INVALID, kw
    assert _append(ok, table=_table(rope_dim=32), pos=16) == UNSUPPORTED
    assert _append(_append_shape(kv_dtype=1)) == INVALID                      # fp8 without row scales
    assert _append(_append_shape(kv_dtype=1), rs=18) == INVALID
    assert _append(_append_shape(**paged)) == INVALID                         # paged without a table
    assert _append(_append_shape(tokens=5, **paged), pt=16) == INVALID        # 5 tokens over 2 sequences, no seq
    assert _append(_append_shape(tokens=0), x=None, slots=None, kv=None) == 0


# ------------------------------------------------------- attention weights
def test_weights_refusals():
    f = api.lib.sparse_mla_attn_weights
    s = api.make_shape(2, 100, 1000)
    args = [16, 16, None, None, 16, 16, 0.04, 16, None]
    assert f(None, *args) == INVALID
    for i in (0, 1, 4, 5, 7):
        a = list(args)
        a[i] = None
        assert f(ctypes.byref(s), *a) == INVALID, i
    for i, v in ((0, 8), (1, 8), (4, 18), (5, 18), (7, 18), (6, math.nan), (6, math.inf), (2, 16)):
        a = list(args)
        a[i] = v
        assert f(ctypes.byref(s), *a) == INVALID, (i, v)
    assert f(ctypes.byref(api.make_shape(2, 100, 1000, fp8=True)), *args) == INVALID
    assert f(ctypes.byref(api.make_shape(2, 100, 1000, page_size=64, pages_per_seq=3)), *args) == INVALID
    bad = api.make_shape(2, 100, 1000)
    bad.num_heads = 32
    assert f(ctypes.byref(bad), *args) == UNSUPPORTED


def test_accumulate_refusals():
    f = api.lib.sparse_mla_accumulate_weights
    good = [2, 100, 50, 16, 16, 1.0, 16, None]
    for i, v in ((0, 0), (0, 65536), (1, 0), (1, (1 << 28) + 1), (2, 0), (2, (1 << 20) + 1), (3, None), (3, 18),
                 (4, None), (4, 18), (5, -0.1), (5, 1.1), (5, math.nan), (6, None), (6, 18)):
        a = list(good)
        a[i] = v
        assert f(*a) == INVALID, (i, v)


# ---------------------------------------------------------------- eviction
def _evict_shape(**kw):
    d = dict(batch=2, max_ctx=256, budget=100, sinks=4, recent=16, kv_dtype=0, pages_per_seq=4, new_pages_per_seq=0,
             num_kv_rows=640, num_key_rows=0)
    d.update(kw)
    return ctypes.byref(api.EvictShape(*d.values()))


def _evict(shape, acc=16, ctx=16, kept=16, new_len=16, out=16, pt=16, npt=None, kv=16, rs=None, keys=None):
    return api.lib.sparse_mla_evict(shape, acc, ctx, kept, new_len, out, pt, npt, kv, rs, keys, None)


def test_evict_refusals():
    for kw in (dict(batch=0), dict(batch=65536), dict(max_ctx=0), dict(max_ctx=(1 << 20) + 1, pages_per_seq=1 << 20),
               dict(budget=0), dict(budget=257), dict(sinks=-1), dict(recent=-1), dict(sinks=90), dict(sinks=2 ** 31 - 1),
               dict(pages_per_seq=3), dict(new_pages_per_seq=-1), dict(num_kv_rows=100), dict(num_kv_rows=0),
               dict(num_key_rows=100), dict(num_key_rows=-64)):
        assert _evict(_evict_shape(**kw)) == INVALID, kw
        assert api.lib.sparse_mla_evict_select(_evict_shape(**kw), 16, 16, 16, 16, 16, None) == INVALID, kw
        assert api.lib.sparse_mla_evict_compact(_evict_shape(**kw), 16, 16, 16, None, 16, None, None, None) == INVALID
    assert _evict(_evict_shape(kv_dtype=3)) == UNSUPPORTED and _evict(None) == INVALID
    ok = _evict_shape()
    for kw in (dict(acc=None), dict(ctx=None), dict(kept=None), dict(new_len=None), dict(out=None), dict(pt=None),
               dict(kv=None), dict(acc=18), dict(ctx=18), dict(kept=18), dict(new_len=18), dict(out=18), dict(pt=18),
               dict(npt=18), dict(kv=8), dict(rs=16), dict(keys=16), dict(npt=32)):
        assert _evict(ok, **kw) == INVALID, kw
    assert _evict(_evict_shape(new_pages_per_seq=1), npt=32) == INVALID       # too few new pages for the budget
    assert _evict(_evict_shape(kv_dtype=1)) == INVALID                        # fp8 without row scales
    assert _evict(_evict_shape(num_key_rows=640)) == INVALID                  # keys announced, none given
    assert _evict(_evict_shape(num_key_rows=640), keys=8) == INVALID


# ----------------------------------------------------------------- binding
def test_binding_rejects_bad_tensors():
    z = torch.zeros
    t = api.RopeTable()
    pos = z(2, dtype=torch.int32)
    for x, kw in ((z(2, 3, 64), {}), (z(2, 3, 64, dtype=torch.float64), {}), (z(2, 3, 63), {}),
                  (z(2, 3, 64), dict(offset=1)), (z(2, 3, 64), dict(out=z(2, 3, 65)))):
        with pytest.raises(ValueError):
            api.rope(x, pos, t, **kw)
    with pytest.raises(ValueError):
        api.rope(z(2, 3, 64), pos.long(), t)
    kv = z(128, 576, dtype=torch.bfloat16)
    slots = z(3, dtype=torch.int32)
    x = z(3, 576)
    for args, kw in (((x, kv, slots), {}), ((x[:, :512], kv, slots), {}), ((x, kv, slots[:2]), {}),
                     ((x, kv, slots), dict(norm_weight=z(576))), ((x, kv, slots), dict(rope=t)),
                     ((x, kv, slots), dict(page_size=64)), ((x, kv, slots), dict(seq=slots)),
                     ((x, kv, slots), dict(kv_row_scale=z(128))), ((x, kv.view(torch.uint8)[:, :576], slots), {})):
        with pytest.raises(ValueError):
            api.cache_append(*args, **kw)
    with pytest.raises(ValueError):
        api.attention_weights(z(1, 64, 576, dtype=torch.bfloat16), kv, z(1, 4, dtype=torch.int32), z(1, 64), 0.04)
    idx = z(1, 4, dtype=torch.int32)
    for args in ((z(1, 8), idx, z(1, 4)), (z(1, 8), idx.long(), z(1, 4)), (z(2, 8), idx, z(1, 4)), (z(1, 8), idx, z(1, 5))):
        with pytest.raises(ValueError):
            api.accumulate_weights(*args)
    pt = z(1, 2, dtype=torch.int32)
    for kw in ({}, dict(page_table=pt.long()), dict(k_cache=z(128, 64)), dict(kept=idx), dict(budget=5)):
        with pytest.raises(ValueError):
            api.evict(z(1, 8), z(1, dtype=torch.int32), **{"budget": 4, "page_table": pt, "kv": kv, **kw})
