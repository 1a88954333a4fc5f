"""GPU tests of the cache append's other forms: rows that are not 16-byte aligned
(loaded as they are needed instead of through the ring), long runs of tokens per
warp with skipped and refused places among them, and values whose codes are exact
or lie on the border between two.

Tolerances of normed and rotated rows are those of the aligned rows' tests.  Rows
that are only encoded have one right answer: bf16 the nearest value, ties to even; a
row scale the nearest fp32 to amax / 448; codes the nearest to the nearest fp32 of x /
scale, ties to even; scales of groups the least power of two."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref

from test_gpu_append import DT, check_rows, make_cache, only_touched, raw

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
@pytest.mark.parametrize("norm,rot", [(True, "interleaved"), (True, "half"), (False, None), (False, "interleaved")])
@pytest.mark.parametrize("off,width", [(1, 579), (3, 600), (0, 577)])
def test_rows_at_any_offset(off, width, kind, dtype, norm, rot):
    """Rows cut out of a wider buffer: an odd first element, an odd distance between rows, or both."""
    rng = np.random.default_rng(width + off)
    n, d = 37, 512 if kind == "dsv4" else 576
    x = torch.from_numpy(rng.standard_normal((n, width)).astype(np.float32)).cuda().to(DT[dtype])[:, off:off + d]
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(512)).astype(np.float32)).cuda() if norm else None
    pos = rng.integers(0, 100000, n).astype(np.int32)
    slots = rng.permutation(128)[:n].astype(np.int32)
    kv, rs = make_cache(kind, 128)
    before = raw(kv)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    table = api().RopeTable(64, interleaved=rot == "interleaved") if rot else None
    paged = dict(page_table=torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), page_size=64) if kind == "dsv4" else {}
    api().cache_append(x, kv, dev(slots), kv_row_scale=rs, norm_weight=w, eps=1e-5, rope=table,
                       positions=dev(pos) if rot else None, **paged)
    torch.cuda.synchronize()
    phys = (slots + 64) % 128 if kind == "dsv4" else slots
    want = ar.append_rows(x.double().cpu().numpy(), norm_weight=None if w is None else w.double().cpu().numpy(), eps=1e-5,
                          freq=ar.rope_frequencies(64) if rot else None, positions=pos, interleaved=rot == "interleaved")
    check_rows(kind, kv, rs, phys, want)
    only_touched(before, raw(kv), kind, phys)


# ------------------------------------------------------------------ one right answer
def nearest_codes(v):
    """e4m3 codes of fp32 values within its range, ties to even (torch's conversion on the CPU)."""
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8)


def border_rows(n, d, group, seed):
    """fp32 rows whose values lie on, just below and just above borders between two codes of their scale: the largest
    value of each `group` dims is 448 times a power of two."""
    g = torch.Generator().manual_seed(seed)
    mag = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = ((mag[1:] + mag[:-1]) / 2).float()                        # exact in fp32
    x = mid[torch.randint(0, 126, (n, d), generator=g)]
    side = torch.randint(-1, 2, (n, d), generator=g)
    x = torch.where(side > 0, torch.nextafter(x, torch.tensor(1e9)), torch.where(side < 0, torch.nextafter(x, torch.tensor(0.0)), x))
    x = torch.where(torch.rand(n, d, generator=g) < 0.5, -x, x)
    x[:, ::group] = 448.0
    return x * 2.0 ** torch.randint(-20, 20, (n, 1), generator=g)


@pytest.mark.parametrize("off", [0, 1])
def test_fp8_codes_and_scales_of_plain_rows(off):
    n = 400
    rows = torch.cat([border_rows(n, 576, 576, 1), border_rows(n, 576, 576, 2).bfloat16().float(),
                      torch.randn(n, 576, generator=torch.Generator().manual_seed(3)),
                      torch.randn(n, 576, generator=torch.Generator().manual_seed(4)).bfloat16().float(),
                      torch.randint(-448, 449, (n, 576), generator=torch.Generator().manual_seed(5)).float() * 2.0 ** -7])
    m = rows.shape[0]
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(m, 577, dtype=dtype, device="cuda") if off else torch.zeros(m, 576, dtype=dtype, device="cuda")
        x[:, off:] = rows.to(dtype).cuda()
        kv, rs = make_cache("fp8", m)
        api().cache_append(x[:, off:], kv, torch.arange(m, dtype=torch.int32, device="cuda"), kv_row_scale=rs)
        v = x[:, off:].float().cpu()
        scale = v.abs().amax(1) / 448                               # one fp32 division, rounded to nearest
        assert torch.equal(rs.cpu(), scale)
        want = nearest_codes((v.double() / scale.double()[:, None]).float())
        got = kv.cpu()
        same = (got == want) | ((got & 0x7F) == 0) & ((want & 0x7F) == 0)
        assert torch.all(same), int((~same).sum())


def test_dsv4_codes_and_scales_of_plain_rows():
    n = 200
    rows = torch.cat([border_rows(n, 512, 64, 6), torch.randn(n, 512, generator=torch.Generator().manual_seed(7)),
                      1e-3 * torch.randn(n, 512, generator=torch.Generator().manual_seed(8)) ** 5])
    rows[5, 64:128] = 0
    m = rows.shape[0]
    kv, _ = make_cache("dsv4", -(-m // 64) * 64)
    pt = torch.arange(-(-m // 64), dtype=torch.int32, device="cuda")[None]
    api().cache_append(rows.cuda(), kv, torch.arange(m, dtype=torch.int32, device="cuda"), page_table=pt, page_size=64)
    torch.cuda.synchronize()
    pages = kv.cpu()
    slots = pages[:, :36864].reshape(-1, 576)[:m]
    blocks = pages[:, 36864:].reshape(-1, 8)[:m]
    groups = rows[:, :448].reshape(m, 7, 64)
    e = torch.from_numpy(np.vectorize(ar.group_exponent)(groups.abs().amax(2).double().numpy()))
    assert torch.equal(blocks[:, :7].long(), e + 127) and torch.all(blocks[:, 7] == 0)
    want = nearest_codes((groups.double() * 2.0 ** -e[..., None].double()).reshape(m, 448))
    got = slots[:, :448]
    assert torch.all((got == want) | ((got & 0x7F) == 0) & ((want & 0x7F) == 0))
    assert torch.equal(slots[:, 448:].contiguous().view(torch.bfloat16), rows[:, 448:].bfloat16())


def test_bf16_rows_round_to_even():
    base = torch.randint(0x3000, 0x4800, (64, 576), generator=torch.Generator().manual_seed(9)).to(torch.int32) << 16
    low = torch.tensor([0x8000, 0x7FFF, 0x8001, 0])[torch.randint(0, 4, (64, 576), generator=torch.Generator().manual_seed(10))].to(torch.int32)
    x = (base | low).view(torch.float32)
    kv, _ = make_cache("bf16", 64)
    api().cache_append(x.cuda(), kv, torch.arange(64, dtype=torch.int32, device="cuda"))
    assert torch.equal(kv.cpu().view(torch.int16), x.bfloat16().view(torch.int16))


# ------------------------------------------------------------------ long runs
def stored(kind, kv, rs, phys):
    """(values, steps) of the rows `phys`: what they hold, and the scale of each dim's codes (0: bf16)."""
    if kind == "bf16":
        v = ref.bf16_bits_to_f64(kv.view(torch.int16).cpu().numpy().view(np.uint16)[phys])
        return v, np.zeros_like(v)
    if kind == "fp8":
        s = rs.double().cpu().numpy()[phys][:, None]
        v = ref.e4m3fn_to_f64(kv.cpu().numpy()[phys]) * s
        return v, np.broadcast_to(s, v.shape)
    b = kv[:, 36864:].cpu().numpy().reshape(-1, 8)[phys, :7].astype(np.float64)
    v = ref.dsv4_rows_f64(kv.cpu().numpy(), phys)
    return v, np.concatenate([np.repeat(2.0 ** (b - 127), 64, 1), np.zeros((len(phys), 64))], 1)


@pytest.mark.parametrize("kind,dtype,rot,n", [("bf16", "bf16", "interleaved", 9001), ("fp8", "fp32", "half", 9001),
                                              ("dsv4", "bf16", "interleaved", 9001), ("dsv4", "fp16", "half", 40013),
                                              ("bf16", "fp32", "half", 40013), ("fp8", "fp16", "interleaved", 40013)])
def test_long_runs_with_skipped_and_refused_places(kind, dtype, rot, n):
    """Three to twelve tokens per warp: uneven prompts over scattered pages, some tokens without a place, some with one
    outside; every row against the oracle, and every other byte as it was."""
    rng = np.random.default_rng(n + len(kind))
    d, B = 512 if kind == "dsv4" else 576, 7
    seq = np.sort(rng.integers(0, B, n)).astype(np.int32)
    first = np.searchsorted(seq, np.arange(B))
    slots = (np.arange(n) - first[seq]).astype(np.int32)
    pps = int(slots.max()) // 64 + 1
    pt = rng.permutation(B * pps + 3)[:B * pps].reshape(B, pps).astype(np.int32)
    skip, refuse = rng.random(n) < 0.05, rng.random(n) < 0.02
    given = slots.copy()
    given[skip] = -1
    given[refuse] = pps * 64 + rng.integers(0, 1000, int(refuse.sum()))
    live = ~skip & ~refuse
    x = torch.randn(n, d, device="cuda", generator=torch.Generator("cuda").manual_seed(n)).to(DT[dtype])
    w = torch.from_numpy((1 + 0.2 * rng.standard_normal(512)).astype(np.float32)).cuda()
    pos = rng.integers(0, 200000, n).astype(np.int32)
    kv, rs = make_cache(kind, (B * pps + 3) * 64)
    before = raw(kv)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    api().cache_append(x, kv, dev(given), kv_row_scale=rs, page_table=dev(pt), page_size=64, seq=dev(seq), norm_weight=w,
                       eps=1e-5, rope=api().RopeTable(64, interleaved=rot == "interleaved"), positions=dev(pos))
    torch.cuda.synchronize()
    assert api().device_error() == 4
    phys = (pt[seq, slots // 64].astype(np.int64) * 64 + slots % 64)[live]
    want = ar.append_rows(x.double().cpu().numpy()[live], norm_weight=w.double().cpu().numpy(), eps=1e-5,
                          freq=ar.rope_frequencies(64), positions=pos[live], interleaved=rot == "interleaved")
    got, step = stored(kind, kv, rs, phys)
    lead = 2.0 ** -17 * np.abs(want) + 2.0 ** -20 * np.abs(want[:, -64:]).max(1, keepdims=True)
    coded = np.maximum(2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -10), 2.0 ** -10 * step)
    assert np.all(np.abs(got - want) <= lead + np.where(step > 0, coded, 2.0 ** -8 * np.abs(want)))
    if kind == "fp8":
        assert np.all(np.abs(step[:, 0] * 448 / np.abs(want).max(1) - 1) <= 2.0 ** -16)
    keep = np.ones((B * pps + 3) * 64, bool)
    keep[phys] = False
    after = raw(kv)
    if kind == "dsv4":
        for lo, hi in ((0, 36864), (36864, 37376)):
            a, b = (t[:, lo:hi].reshape(len(keep), -1) for t in (before, after))
            assert np.array_equal(a[keep], b[keep])
    else:
        assert np.array_equal(before[keep], after[keep])


def test_runs_of_32_tokens_give_the_bits_of_single_ones():
    """120,000 tokens, more than the resident warps take in one run each, in the three layouts and without norm or
    rotation too, against calls of 3,000 tokens (one token per warp)."""
    n = 120_000
    slots = torch.randperm(n, device="cuda", generator=torch.Generator("cuda").manual_seed(15)).to(torch.int32)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    w = torch.linspace(0.5, 1.5, 512, device="cuda")
    pages = torch.randperm(n // 64, device="cuda", generator=torch.Generator("cuda").manual_seed(16)).to(torch.int32)[None]
    for kind, d, whole in (("bf16", 576, True), ("fp8", 576, False), ("dsv4", 512, True)):
        x = torch.randn(n, d, device="cuda", generator=torch.Generator("cuda").manual_seed(17)).to(torch.bfloat16)
        kw = dict(norm_weight=w, rope=api().RopeTable(64)) if whole else {}
        a, sa = make_cache(kind, n)
        b, sb = make_cache(kind, n)
        paged = dict(page_table=pages, page_size=64)
        one = torch.zeros(n, dtype=torch.int32, device="cuda")
        api().cache_append(x, a, slots, kv_row_scale=sa, positions=pos if whole else None, seq=one, **paged, **kw)
        for i in range(0, n, 3000):
            api().cache_append(x[i:i + 3000], b, slots[i:i + 3000], kv_row_scale=sb, positions=pos[i:i + 3000] if whole else None,
                               seq=one[i:i + 3000], **paged, **kw)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)) and (sa is None or torch.equal(sa, sb))
