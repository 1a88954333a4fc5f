"""GPU parity for the attention weights (sparse_mla_attn_weights) and their
accumulation (sparse_mla_accumulate_weights) against the fp64 oracle.

Weights.  A score is a dot product of at most 576 exact products accumulated in
fp32 by the tensor cores in K steps of 16 or 32: 36 accumulator updates, each
within 2 x 2^-23 of the running magnitude, which is at most A = sum_d |q_d k_d|;
an fp8 query's second half adds 2^-17 max|q| sum_d |k_d|; the row scale and the
fused scale - lse step add 2^-23 of |s| and of |s - lse|; the exponential is within
2^-21 relative plus 2^-23 |s - lse|; the sum of 64 terms within 6 x 2^-24 deep
pairs or 64 x 2^-24 in order.  So |w - w*| <= sum_h p_h (delta_h + 2^-17), delta_h =
scale (72 x 2^-23 A_h + 2^-17 max|q_h| sum|k|) + 2^-21 (|s_h| + |s_h - lse_h|).

Accumulation.  Fixed point: half a unit per entry, unit <= 2^-61 x entries (as a
power of two) x largest |weight|, then one fp32 rounding of the result and of
the decayed value's fp64 sum: 2^-24 of the result."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref
from sparse_mla_decode_05_b200 import inputs

from _helpers import Dev

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def run(d, lse, **kw):
    return api().attention_weights(d.q, d.kv, d.indices, lse, d.w.scale, kv_row_scale=d.kv_row_scale,
                                   page_table=d.page_table, page_size=d.w.page_size, **kw)


def check(w, got, lse, rows=None):
    """got against the oracle for the decode rows `rows` (default: all)."""
    q = ref.bf16_bits_to_f64(w.np_q_bits()).reshape(w.rows, 64, -1)
    idx = w.indices.numpy().reshape(w.rows, -1)
    lse = lse.double().cpu().numpy().reshape(w.rows, 64)
    got = got.double().cpu().numpy().reshape(w.rows, -1)
    scale = float(np.float32(w.scale))
    for r in range(w.rows) if rows is None else rows:
        want, k, valid = ar.list_weights(q[r], w.np_kv(), idx[r], lse[r], scale, kv_format=w.kv_format,
                                         kv_row_scale=None if w.kv_row_scale is None else w.kv_row_scale.numpy(),
                                         page_table_row=None if w.page_table is None else w.page_table.numpy()[r // w.tokens],
                                         page_size=w.page_size)
        s = scale * (q[r] @ k.T)
        live = np.isfinite(lse[r])
        A = np.abs(q[r]) @ np.abs(k).T
        split = 2.0 ** -17 * np.abs(q[r]).max(1)[:, None] * np.abs(k).sum(1) if w.kv_format.startswith("fp8") else 0.0
        e = np.where(live[:, None], s - np.where(live, lse[r], 0.0)[:, None], -np.inf)
        p = np.exp(e)
        delta = scale * (72 * 2.0 ** -23 * A + split) + 2.0 ** -21 * (np.abs(s) + np.where(np.isfinite(e), np.abs(e), 0.0))
        tol = (p * (delta + 2.0 ** -17)).sum(0) + 1e-37
        assert np.all(got[r][~valid] == 0.0)
        err = np.abs(got[r][valid] - want[valid])
        assert np.all(err <= tol), (r, float((err / tol).max()))


def oracle_lse(w):
    f = ref.sparse_mla_decode_multi_token if w.tokens > 1 else ref.sparse_mla_decode
    _, lse = f(w.np_q_bits(), w.np_kv(), w.indices.numpy(), w.scale, kv_format=w.kv_format,
               kv_row_scale=None if w.kv_row_scale is None else w.kv_row_scale.numpy(),
               page_table=None if w.page_table is None else w.page_table.numpy(), page_size=w.page_size)
    return torch.from_numpy(lse.astype(np.float32)).cuda()


SMALL = {
    "flat": lambda k: inputs.flat_per_seq(2, 2048, k, seed=201),
    "flat_peaky": lambda k: inputs.flat_per_seq(2, 2048, k, seed=202, q_mult=4.0),
    "paged_bf16": lambda k: inputs.paged_bf16(2, 2048, 80, k, seed=203),
    "fp8": lambda k: inputs.paged_fp8(2, 2048, 80, k, seed=204),
    "dsv4": lambda k: inputs.paged_dsv4(2, 2048, 80, k, seed=205),
}


@pytest.mark.parametrize("k", [1, 2, 31, 63, 64, 65, 127, 128, 129, 511, 1000])
@pytest.mark.parametrize("kind", sorted(SMALL))
def test_weights(kind, k):
    w = SMALL[kind](k)
    lse = oracle_lse(w)
    got = run(Dev(w), lse)
    assert got.shape == w.indices.shape
    check(w, got, lse)
    # the weights of a list sum to one per head
    assert np.allclose(got.double().sum(-1).cpu().numpy(), 64.0, rtol=2.0 ** -10)


@pytest.mark.parametrize("kind", ["flat", "fp8", "dsv4"])
def test_padding_and_empty_lists(kind):
    w = SMALL[kind](300)
    g = torch.Generator().manual_seed(9)
    w.indices[0][torch.randperm(300, generator=g)[:170]] = -1
    w.indices[1] = -1
    lse = oracle_lse(w)
    assert torch.all(lse[1] == -torch.inf)
    out = torch.full((2, 300), float("nan"), device="cuda")
    got = run(Dev(w), lse, out=out)
    assert got is out
    check(w, got, lse, rows=[0])
    assert torch.all(got[1] == 0)


def test_lse_of_minus_infinity_leaves_its_head_out():
    w = SMALL["flat"](100)
    lse = oracle_lse(w)
    lse[0, 5] = -torch.inf
    check(w, run(Dev(w), lse), lse)


def test_infinite_and_nan_rows_that_are_not_listed_do_not_matter():
    w = SMALL["flat"](200)
    lse = oracle_lse(w)
    want = run(Dev(w), lse)
    kv = torch.full_like(w.kv, float("nan"))
    listed = w.indices[w.indices >= 0].long()
    kv[listed] = w.kv[listed]
    w2 = inputs.dataclasses.replace(w, kv=kv)
    assert torch.equal(run(Dev(w2), lse), want)


@pytest.mark.parametrize("fp8,paged", [(True, True), (False, True), (False, False)])
def test_multi_token(fp8, paged):
    w = inputs.multi_token(3, 4, 1024, 60, 250, seed=206, fp8=fp8, paged=paged)
    w.indices[1, 2] = -1
    lse = oracle_lse(w)
    got = run(Dev(w), lse)
    check(w, got, lse, rows=[r for r in range(12) if r != 6])
    assert torch.all(got[1, 2] == 0)


@pytest.mark.parametrize("name,rows", [("c2", range(16)), ("c3", (0, 31, 63)), ("c4b", (0, 1)), ("c5", (0, 77, 127)),
                                       ("dsv4", (0, 31)), ("mt2", (0, 127))])
def test_full_workloads_with_the_decodes_own_lse(name, rows):
    w = inputs.make_config(name)
    d = Dev(w)
    out, lse = d.run()
    got = run(d, lse)
    check(w, got, lse, rows=list(rows))


def test_same_entry_twice_counts_each_time():
    w = SMALL["fp8"](64)
    w.indices[0, 10:20] = w.indices[0, 3]
    lse = oracle_lse(w)
    got = run(Dev(w), lse)
    check(w, got, lse)
    assert torch.all(got[0, 10:20] == got[0, 3])


def test_out_of_range_entries_read_as_padding():
    w = SMALL["paged_bf16"](100)
    lse = oracle_lse(w)
    d = Dev(w)
    want = run(d, lse).clone()
    bad = w.indices.clone()
    bad[0, 5], bad[1, 99] = 2048, 2 ** 31 - 1
    d.indices = bad.cuda()
    got = run(d, lse)
    assert api().device_error() == 4
    want[0, 5] = want[1, 99] = 0
    assert torch.equal(got, want)
    d.page_table[0, 0] = 80                                   # one page outside the pool
    got = run(d, lse)
    assert api().device_error() == 4
    gone = (bad[0] >= 0) & (bad[0] < 64)
    assert torch.all(got[0][gone.cuda()] == 0)


def test_repeat_stream_and_graph_are_bit_identical():
    for kind in ("flat", "fp8", "dsv4"):
        w = SMALL[kind](700)
        d, lse = Dev(w), oracle_lse(w)
        want = run(d, lse).clone()
        plan = api().AttentionWeightsPlan(d.q, d.kv, d.indices, lse, w.scale, kv_row_scale=d.kv_row_scale,
                                          page_table=d.page_table, page_size=w.page_size)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            plan.run()
        torch.cuda.synchronize()
        assert torch.equal(plan.out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan.run()
            plan.run()
        plan.out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out, want)


# ------------------------------------------------------------ accumulation
def check_acc(acc0, idx, w, decay, got):
    B = acc0.shape[0]
    idx, w = idx.cpu().numpy().reshape(B, -1), w.cpu().numpy().reshape(B, -1)
    d = float(np.float32(decay))
    want = ar.accumulate(acc0.double().cpu().numpy(), idx, w, d)
    top = np.abs(w).max(1, keepdims=True)
    n = 2.0 ** np.ceil(np.log2(max(idx.shape[1], 1)))
    # every entry may round by half a unit
    tol = idx.shape[1] * 0.5 * 2.0 ** -61 * n * top + 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -20) + 1e-45
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


@pytest.mark.parametrize("B,T,k,n,decay", [(1, 1, 1, 1, 1.0), (2, 1, 5, 3, 0.5), (3, 1, 512, 8192, 1.0), (2, 2, 700, 4097, 0.9),
                                           (4, 4, 64, 100, 1.0), (1, 1, 2048, 65536, 0.0), (2, 16, 33, 4096, 0.25), (1, 1, 40000, 7, 1.0)])
def test_accumulate(B, T, k, n, decay):
    rng = np.random.default_rng(k + n)
    idx = torch.from_numpy(rng.integers(-1, n, (B, T, k)).astype(np.int32)).cuda()      # repeats everywhere
    w = torch.from_numpy(rng.exponential(1.0, (B, T, k)).astype(np.float32) * 10.0 ** rng.integers(-6, 2, (B, T, k))).float().cuda()
    acc = torch.from_numpy(rng.random((B, n)).astype(np.float32)).cuda()
    if T == 1:
        idx, w = idx[:, 0].contiguous(), w[:, 0].contiguous()
    acc0 = acc.clone()
    assert api().accumulate_weights(acc, idx, w, decay=decay) is acc
    check_acc(acc0, idx, w, decay, acc)
    # any order of the entries gives the same bits
    again = acc0.clone()
    flat_i, flat_w = idx.view(B, -1), w.view(B, -1)
    perm = torch.randperm(flat_i.shape[1], device="cuda")
    api().accumulate_weights(again, flat_i[:, perm].contiguous(), flat_w[:, perm].contiguous(), decay=decay)
    assert torch.equal(again, acc)


def test_accumulate_leaves_untouched_positions_and_signs():
    acc = torch.tensor([[1.5, -0.0, float("nan"), float("inf"), 2.0]], device="cuda")
    idx = torch.tensor([[4, 4, -1, -7]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, -3.0, 5.0, float("nan")]], device="cuda")
    api().accumulate_weights(acc, idx, w)
    got = acc.cpu().numpy()[0]
    assert got[0] == 1.5 and np.signbit(got[1]) and np.isnan(got[2]) and np.isinf(got[3]) and got[4] == 0.0


def test_accumulate_nan_and_infinite_weights_stay_at_their_position():
    acc = torch.zeros(1, 6, device="cuda")
    idx = torch.tensor([[0, 1, 2, 2, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("nan"), float("inf"), 1.0, 2.0, 1e-30]], device="cuda")
    api().accumulate_weights(acc, idx, w, decay=0.5)
    got = acc.cpu().numpy()[0]
    assert np.isnan(got[0]) and np.isnan(got[1]) and got[2] == 3.0 and np.all(got[4:] == 0)


@pytest.mark.parametrize("decay", [1.0, 0.5])
def test_accumulate_nothing_but_nan_and_infinity(decay):
    acc = torch.ones(1, 5000, device="cuda")
    idx = torch.tensor([[7, 4999, 30, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[float("nan"), -float("inf"), 0.0, float("nan")]], device="cuda")
    api().accumulate_weights(acc, idx, w, decay=decay)
    got = acc.cpu().numpy()[0]
    assert np.isnan(got[7]) and np.isnan(got[4999]) and np.all(np.delete(got, [7, 4999]) == decay)


def test_accumulate_all_zero_or_no_weights_still_decays():
    acc = torch.ones(2, 5000, device="cuda")
    api().accumulate_weights(acc, torch.full((2, 3), -1, dtype=torch.int32, device="cuda"), torch.ones(2, 3, device="cuda"), decay=0.5)
    assert torch.all(acc == 0.5)
    api().accumulate_weights(acc, torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, 3, device="cuda"), decay=0.5)
    assert torch.all(acc == 0.25)


def test_accumulate_out_of_range_positions_are_reported():
    acc = torch.zeros(1, 10, device="cuda")
    api().accumulate_weights(acc, torch.tensor([[9, 10, 2 ** 31 - 1]], dtype=torch.int32, device="cuda"), torch.ones(1, 3, device="cuda"))
    assert api().device_error() == 4
    assert acc[0, 9] == 1 and acc.sum() == 1
