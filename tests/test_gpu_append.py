"""GPU parity for the cache append (sparse_mla_cache_append) against the fp64
oracle, and what it must leave alone.

Tolerances.  The normalised and rotated row in fp32: the mean square of 512
terms is within 2^-18 (at most 23 additions deep), rsqrtf and the products add
4 x 2^-23, so a value is within 2^-17 of itself; the rotation adds 2^-21 (|a| +
|b|).  Stored bf16 values round by 2^-8; e4m3 codes by 2^-4 of the value or half
a subnormal step, 2^-10 of the scale; a row scale by 2^-24.  A power-of-two
scale is the oracle's exactly, unless the group's amax lies within 2^-16 of the
border between two (none of the seeds does)."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PAGE_BYTES = 37376


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def make_cache(kind, rows, fill=0x5A):
    """A cache whose bytes are all `fill`."""
    if kind == "bf16":
        return torch.full((rows, 1152), fill, dtype=torch.uint8, device="cuda").view(torch.bfloat16), None
    if kind == "fp8":
        return torch.full((rows, 576), fill, dtype=torch.uint8, device="cuda"), torch.full((rows,), 9.0, device="cuda")
    return torch.full((rows // 64, PAGE_BYTES), fill, dtype=torch.uint8, device="cuda"), None


def raw(kv):
    return kv.view(torch.uint8).cpu().numpy().copy()


def check_rows(kind, kv, rs, phys, want):
    """Stored rows `phys` against the fp64 rows `want` [n, d]."""
    lead = 2.0 ** -17 * np.abs(want) + 2.0 ** -20 * np.abs(want[:, -64:]).max(1, keepdims=True) + 1e-30
    if kind == "bf16":
        got = ref.bf16_bits_to_f64(kv.view(torch.int16).cpu().numpy().view(np.uint16)[phys])
        assert np.all(np.abs(got - want) <= lead + 2.0 ** -8 * np.abs(want))
        return
    if kind == "fp8":
        codes = ref.e4m3fn_to_f64(kv.cpu().numpy()[phys])
        scale = rs.double().cpu().numpy()[phys]
        amax = np.abs(want).max(1)
        ws = np.where(amax > 0, amax / 448, 1.0)
        assert np.all(np.abs(scale - ws) <= 2.0 ** -16 * ws + 2.0 ** -126)
        err = np.abs(codes * scale[:, None] - want)
        assert np.all(err <= lead + np.maximum(2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -10), 2.0 ** -10 * scale[:, None]))
        return
    pages = kv.cpu().numpy()
    for i, r in enumerate(phys):
        slot = pages[r // 64, (r % 64) * 576:(r % 64) * 576 + 576]
        block = pages[r // 64, 36864 + (r % 64) * 8:36864 + (r % 64) * 8 + 8]
        assert block[7] == 0
        for g in range(7):
            v = want[i, 64 * g:64 * g + 64]
            e = ar.group_exponent(np.abs(v).max())
            assert block[g] == e + 127
            err = np.abs(ref.e4m3fn_to_f64(slot[64 * g:64 * g + 64]) * 2.0 ** e - v)
            assert np.all(err <= lead[i, 64 * g:64 * g + 64] + np.maximum(2.0 ** -4 * np.abs(v) * (1 + 2.0 ** -10), 2.0 ** (e - 10)))
        got = ref.bf16_bits_to_f64(slot[448:].copy().view(np.uint16))
        assert np.all(np.abs(got - want[i, 448:]) <= lead[i, 448:] + 2.0 ** -8 * np.abs(want[i, 448:]))


def only_touched(before, after, kind, phys):
    """No byte outside the rows `phys` differs."""
    if kind == "dsv4":
        mask = np.ones(before.shape, bool)
        for r in phys:
            mask[r // 64, (r % 64) * 576:(r % 64) * 576 + 576] = False
            mask[r // 64, 36864 + (r % 64) * 8:36864 + (r % 64) * 8 + 8] = False
        assert np.array_equal(before[mask], after[mask])
    else:
        keep = np.setdiff1d(np.arange(before.shape[0]), phys)
        assert np.array_equal(before[keep], after[keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
@pytest.mark.parametrize("n,B", [(1, 1), (5, 5), (64, 8), (137, 3)])
@pytest.mark.parametrize("norm,rot", [(True, "interleaved"), (True, "half"), (False, None), (False, "half"), (True, None)])
def test_append(n, B, kind, dtype, norm, rot):
    rng = np.random.default_rng(n * 7 + B)
    d = 512 if kind == "dsv4" else 576
    pps, rows = 5, (B * 5 + 2) * 64
    x = torch.from_numpy(rng.standard_normal((n, d)).astype(np.float32)).cuda().to(DT[dtype])
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(512)).astype(np.float32)).cuda() if norm else None
    pt = rng.permutation(B * 5 + 2)[:B * pps].reshape(B, pps).astype(np.int32)
    seq = np.sort(rng.integers(0, B, n)).astype(np.int32)
    slots = np.empty(n, np.int32)
    for b in range(B):                                  # distinct slots within a sequence
        m = int((seq == b).sum())
        slots[seq == b] = rng.choice(pps * 64, m, replace=False)
    slots[rng.random(n) < 0.1] = -1
    pos = rng.integers(0, 100000, n).astype(np.int32)
    kv, rs = make_cache(kind, rows)
    before, rs0 = raw(kv), None if rs is None else rs.cpu().numpy().copy()
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    table = api().RopeTable(64, interleaved=rot == "interleaved") if rot else None
    api().cache_append(x, kv, dev(slots), kv_row_scale=rs, page_table=dev(pt), page_size=64, seq=dev(seq), norm_weight=w,
                       eps=1e-5, rope=table, positions=dev(pos) if rot else None)
    torch.cuda.synchronize()
    phys = ar.slot_rows(slots, seq, pt)
    live = phys >= 0
    want = ar.append_rows(x.double().cpu().numpy(), norm_weight=None if w is None else w.double().cpu().numpy(), eps=1e-5,
                          freq=ar.rope_frequencies(64) if rot else None, positions=pos, interleaved=rot == "interleaved")
    check_rows(kind, kv, rs, phys[live], want[live])
    only_touched(before, raw(kv), kind, phys[live])
    if rs is not None:
        keep = np.setdiff1d(np.arange(rows), phys[live])
        assert np.array_equal(rs.cpu().numpy()[keep], rs0[keep])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_flat_pool_and_strided_rows(kind):
    rng = np.random.default_rng(11)
    wide = torch.from_numpy(rng.standard_normal((40, 700)).astype(np.float32)).cuda().to(torch.bfloat16)
    slots = torch.from_numpy(rng.permutation(300)[:40].astype(np.int32)).cuda()
    for off in (0, 8, 3):                               # 16-byte rows and element-aligned ones
        kv, rs = make_cache(kind, 300)
        x = wide[:, off:off + 576]
        api().cache_append(x, kv, slots, kv_row_scale=rs)
        torch.cuda.synchronize()
        check_rows(kind, kv, rs, slots.cpu().numpy(), x.double().cpu().numpy())


def test_equal_runs_without_seq_match_explicit_sequences():
    rng = np.random.default_rng(12)
    x = torch.from_numpy(rng.standard_normal((12, 576)).astype(np.float32)).cuda()
    pt = torch.from_numpy(rng.permutation(8).reshape(4, 2).astype(np.int32)).cuda()
    slots = torch.tensor([60, 61, 62] * 4, dtype=torch.int32, device="cuda")
    a, sa = make_cache("fp8", 512)
    b, sb = make_cache("fp8", 512)
    api().cache_append(x, a, slots, kv_row_scale=sa, page_table=pt, page_size=64)
    api().cache_append(x, b, slots, kv_row_scale=sb, page_table=pt, page_size=64,
                       seq=torch.arange(12, device="cuda", dtype=torch.int32) // 3)
    assert torch.equal(a, b) and torch.equal(sa, sb)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
def test_zero_tiny_and_huge_rows(kind):
    d = 512 if kind == "dsv4" else 576
    x = torch.zeros(4, d, device="cuda")
    x[1], x[2], x[3] = 3e-38, 1e30, torch.linspace(-1e-3, 1e3, d, device="cuda")
    kv, rs = make_cache(kind, 64)
    pt = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    paged = dict(page_table=pt, page_size=64) if kind == "dsv4" else {}
    api().cache_append(x, kv, torch.arange(4, device="cuda", dtype=torch.int32), kv_row_scale=rs, **paged)
    torch.cuda.synchronize()
    want = x.double().cpu().numpy()
    if kind == "dsv4":
        # row 1's scale stops at 2^-126, so it keeps what codes of that scale can say
        check_rows(kind, kv, rs, np.array([0, 2, 3]), want[[0, 2, 3]])
        got = ref.dsv4_rows_f64(kv.cpu().numpy(), np.array([1]))[0, :448]
        assert np.all(np.abs(got - 3e-38) <= 2.0 ** -4 * 3e-38)
    else:
        check_rows(kind, kv, rs, np.array([0, 2, 3]), want[[0, 2, 3]])


def test_out_of_range_places_write_nothing_and_are_reported():
    x = torch.randn(6, 576, device="cuda")
    kv, _ = make_cache("bf16", 256)
    before = raw(kv)
    api().cache_append(x, kv, torch.full((6,), 256, dtype=torch.int32, device="cuda"))
    assert api().device_error() == 4
    pt = torch.tensor([[0, 4], [-1, 1 << 26]], dtype=torch.int32, device="cuda")
    seq = torch.tensor([0, 0, 1, 1, 2, -1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([128, 64, 0, 64, 0, 0], dtype=torch.int32, device="cuda")
    api().cache_append(x, kv, slots, page_table=pt, page_size=64, seq=seq)
    assert api().device_error() == 4
    assert np.array_equal(before, raw(kv))
    api().cache_append(x[:0], kv, slots[:0])
    assert api().device_error() == 0


def test_many_tokens_loop_over_the_grid():
    """More tokens than resident warps: each row as if written alone."""
    x = torch.randn(30011, 576, device="cuda", generator=torch.Generator("cuda").manual_seed(13)).to(torch.bfloat16)
    w = torch.ones(512, device="cuda")
    slots = torch.randperm(30011, device="cuda", generator=torch.Generator("cuda").manual_seed(14)).to(torch.int32)
    pos = torch.arange(30011, device="cuda", dtype=torch.int32)
    t = api().RopeTable(64)
    kv, rs = make_cache("fp8", 30011)
    api().cache_append(x, kv, slots, kv_row_scale=rs, norm_weight=w, rope=t, positions=pos)
    at = torch.tensor([0, 1, 9471, 9472, 20000, 30010], device="cuda")
    one, rs1 = make_cache("fp8", 6)
    api().cache_append(x[at].contiguous(), one, torch.arange(6, device="cuda", dtype=torch.int32), kv_row_scale=rs1,
                       norm_weight=w, rope=t, positions=pos[at].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(kv[slots[at].long()], one) and torch.equal(rs[slots[at].long()], rs1)


def test_graph_replay_reads_new_tokens():
    x = torch.randn(3, 576, device="cuda")
    kv, rs = make_cache("fp8", 64)
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    plan = api().CacheAppendPlan(x, kv, slots, kv_row_scale=rs)
    plan.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.run()
    for k in range(2):
        x.normal_()
        slots.add_(3)
        g.replay()
        torch.cuda.synchronize()
        check_rows("fp8", kv, rs, slots.cpu().numpy(), x.double().cpu().numpy())
