"""GPU parity for the attention weights over DeepSeek-V4 slots where one dim of a
query stands far above the others.

Bound.  |w - w*| <= sum_h p_h (delta_h + 2^-17) as for other queries.  The query's
split: each head times the power of two that brings its largest |q| into [128,
256), as an e4m3 high part and an e5m2 low part.  A bf16 value has eight significant bits;
where the scaled value is at least 2^-6 the high part is within 2^-4 of half a
power of two, what is left is zero to eight units in the value's last place, and
that is three significant bits, which the low part holds.  Below 2^-6 the high part
leaves at most 2^-10 and the low part, with three significant bits, at most 2^-14 of
that.  In the query's own units, M the power of two at or below the head's largest
|q|: nothing for |q_i| >= 2^-13 M, at most 2^-21 M for the others.  Accumulators: 72 x 2^-23 A_h
covers the at most 32 updates by the tensor cores and the eight by the epilogue."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref
from sparse_mla_decode_05_b200 import inputs

from _helpers import Dev
from test_gpu_weights_slots import oracle_lse, run

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def check(w, got, lse):
    q = ref.bf16_bits_to_f64(w.np_q_bits())
    lse, got, scale = lse.double().cpu().numpy(), got.double().cpu().numpy(), float(np.float32(w.scale))
    for r in range(w.rows):
        want, k, valid = ar.list_weights(q[r], w.np_kv(), w.indices.numpy()[r], lse[r], scale, kv_format=w.kv_format,
                                         kv_row_scale=None, page_table_row=w.page_table.numpy()[r], page_size=64)
        s = scale * (q[r] @ k.T)
        e = s - lse[r][:, None]
        M = 2.0 ** np.floor(np.log2(np.abs(q[r]).max(1)))[:, None]
        lost = np.where(np.abs(q[r][:, :448]) >= 2.0 ** -13 * M, 0.0, 2.0 ** -21 * M) @ np.abs(k[:, :448]).T
        delta = scale * (72 * 2.0 ** -23 * (np.abs(q[r]) @ np.abs(k).T) + lost) + 2.0 ** -21 * (np.abs(s) + np.abs(e))
        tol = (np.exp(e) * (delta + 2.0 ** -17)).sum(0) + 1e-37
        assert np.all(got[r][~valid] == 0.0)
        err = np.abs(got[r][valid] - want[valid])
        assert np.all(err <= tol), (r, float((err / tol).max()))


@pytest.mark.parametrize("outlier", [100.0, 300.0, 500.0])
@pytest.mark.parametrize("dim", [17, 447, 500])
def test_one_dim_far_above_the_others(dim, outlier):
    """Keys of zero in that dim (of the coded ones): what is lost of the other dims shows undiluted."""
    w = inputs.paged_dsv4(2, 1024, 40, 300, seed=311)
    w.q[..., dim] = outlier
    w.q[:, 1::2, dim] = -outlier
    if dim < 448:
        w.kv[:, :64 * 576].view(-1, 64, 576)[..., dim] = 0
    else:
        w.kv[:, :64 * 576].view(-1, 64, 576)[..., 448 + 2 * (dim - 448):450 + 2 * (dim - 448)] = 0
    lse = oracle_lse(w)
    check(w, run(Dev(w), lse), lse)


@pytest.mark.parametrize("outlier", [30.0, 3000.0])
def test_outliers_that_the_keys_meet(outlier):
    """The outlier takes part in the scores too (its sign keeps them from one entry alone)."""
    w = inputs.paged_dsv4(2, 1024, 40, 300, seed=312)
    w.q[..., 100] *= outlier / 8
    lse = oracle_lse(w)
    check(w, run(Dev(w), lse), lse)
