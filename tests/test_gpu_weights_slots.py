"""GPU parity for the attention weights over DeepSeek-V4 slots, where codes are
multiplied as stored and each scale group has an accumulator of its own.

Bound.  As for the other layouts, |w - w*| <= sum_h p_h (delta_h + 2^-17), with the
query's split counted too: the head's values times a power of two that brings
the largest into [128, 256) are e4m3 high + low parts.  A bf16 value has eight
significant bits; the high part leaves a rest of at most four, which the low
part holds exactly unless it falls below e4m3's normal range, where it is off by
at most half of 2^-9: 2^-10 of at least 128, 2^-17 of the head's largest |q|, for
each of the 448 coded dims.  Accumulators: 72 x 2^-23 A_h covers the at most 32
updates by the tensor cores and the eight by the epilogue."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref
from sparse_mla_decode_05_b200 import inputs

from _helpers import Dev

pytestmark = pytest.mark.gpu
SCALES = 64 * 576                     # a page's scale blocks start here


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def oracle_lse(w):
    _, lse = ref.sparse_mla_decode(w.np_q_bits(), w.np_kv(), w.indices.numpy(), w.scale, kv_format=w.kv_format,
                                   page_table=w.page_table.numpy(), page_size=64)
    return torch.from_numpy(lse.astype(np.float32)).cuda()


def run(d, lse, **kw):
    return api().attention_weights(d.q, d.kv, d.indices, lse, d.w.scale, page_table=d.page_table, page_size=64, **kw)


def check(w, got, lse):
    q = ref.bf16_bits_to_f64(w.np_q_bits())
    lse, got, scale = lse.double().cpu().numpy(), got.double().cpu().numpy(), float(np.float32(w.scale))
    for r in range(w.rows):
        want, k, valid = ar.list_weights(q[r], w.np_kv(), w.indices.numpy()[r], lse[r], scale, kv_format=w.kv_format,
                                         kv_row_scale=None, page_table_row=w.page_table.numpy()[r], page_size=64)
        s = scale * (q[r] @ k.T)
        live = np.isfinite(lse[r])
        e = np.where(live[:, None], s - np.where(live, lse[r], 0.0)[:, None], -np.inf)
        split = 2.0 ** -17 * np.abs(q[r]).max(1)[:, None] * np.abs(k[:, :448]).sum(1)
        delta = (scale * (72 * 2.0 ** -23 * (np.abs(q[r]) @ np.abs(k).T) + split)
                 + 2.0 ** -21 * (np.abs(s) + np.where(np.isfinite(e), np.abs(e), 0.0)))
        tol = (np.exp(e) * (delta + 2.0 ** -17)).sum(0) + 1e-37
        assert np.all(got[r][~valid] == 0.0)
        err = np.abs(got[r][valid] - want[valid])
        assert np.all(err <= tol), (r, float((err / tol).max()))


def mixed_scales(w, seed):
    """Every group of every row a scale of its own, 2^-127 (byte 0) among them."""
    g = torch.Generator().manual_seed(seed)
    blocks = w.kv[:, SCALES:].view(-1, 64, 8)
    choice = torch.tensor([0, 1, 96, 110, 119, 120, 121], dtype=torch.uint8)
    blocks[..., :7] = choice[torch.randint(0, 7, (*blocks.shape[:2], 7), generator=g)]


@pytest.mark.parametrize("k", [1, 127, 128, 129, 640])
def test_groups_with_scales_far_apart(k):
    w = inputs.paged_dsv4(2, 1024, 40, k, seed=301)
    mixed_scales(w, 7)
    lse = oracle_lse(w)
    check(w, run(Dev(w), lse), lse)


@pytest.mark.parametrize("group", range(8))
def test_each_group_alone(group):
    """All dims but one group's zero in the query (group 7: the bf16 dims)."""
    w = inputs.paged_dsv4(1, 512, 8, 200, seed=302)
    mixed_scales(w, 8)
    keep = w.q[..., 64 * group:64 * group + 64].clone()
    w.q.zero_()
    w.q[..., 64 * group:64 * group + 64] = keep
    lse = oracle_lse(w)
    check(w, run(Dev(w), lse), lse)


@pytest.mark.parametrize("mult", [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 12])
def test_query_magnitudes(mult):
    """Heads of very different size; the power of two is each head's own."""
    w = inputs.paged_dsv4(1, 512, 8, 200, seed=303)
    w.q[:, ::2] *= mult
    w.q[:, 3] = 0
    lse = oracle_lse(w)
    check(w, run(Dev(w), lse), lse)


def test_slots_that_are_not_listed_do_not_matter():
    w = inputs.paged_dsv4(2, 1024, 40, 300, seed=304)
    w.indices[0, 50:80] = -1
    w.indices[1, 128:256] = -1
    listed = {int(w.page_table[b, int(i) >> 6]) * 64 + (int(i) & 63) for b in range(2) for i in w.indices[b] if i >= 0}
    assert 0 not in listed
    lse = oracle_lse(w)
    want = run(Dev(w), lse)
    check(w, want, lse)
    kv = w.kv.clone()
    rest = torch.tensor([r for r in range(40 * 64) if r not in listed])
    kv[:, :SCALES].view(-1, 64, 576)[rest // 64, rest % 64] = 0x7F        # NaN codes, NaN-like bf16
    kv[:, SCALES:].view(-1, 64, 8)[rest // 64, rest % 64] = 0xFF          # NaN scales
    assert torch.equal(run(Dev(inputs.dataclasses.replace(w, kv=kv)), lse), want)


@pytest.mark.parametrize("k", [64, 128, 129, 257])
def test_many_short_rows(k):
    """Several decode rows per SM, each with a query of its own and one to three
    tiles: the sums of the two halves of the heads meet in the right tile."""
    w = inputs.paged_dsv4(400, 320, 2000, k, seed=305)
    lse = oracle_lse(w)
    d = Dev(w)
    got = run(d, lse)
    check(w, got, lse)
    for _ in range(20):
        assert torch.equal(run(d, lse), got)
