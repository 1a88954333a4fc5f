"""GPU parity for the rotary positions (sparse_mla_rope) against the fp64
oracle.

Tolerance per element, from the arithmetic: the angle is a 64-bit fraction of
a turn rounded to 32 bits (2^-33 turns) and then to fp32 half turns (at most
pi 2^-25 rad), sincospif is within 2 ulp (2^-23), the product with m and the
two-product sum add four roundings of 2^-24: together below 2^-21 of m (|a| +
|b|).  Storing rounds by at most half a step, finfo.eps / 2 of the value (fp16:
or half its subnormal step, 2^-25)."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


def _check(got, x, pos, f, *, offset, interleaved, mscale=1.0, transpose=False):
    xd = x.double().cpu().numpy()
    want = ar.rope(xd, pos.cpu().numpy(), f, offset=offset, interleaved=interleaved, mscale=mscale, transpose=transpose)
    half = len(f)
    mag = np.zeros_like(want)
    a_at = offset + (2 * np.arange(half) if interleaved else np.arange(half))
    b_at = a_at + (1 if interleaved else half)
    both = abs(mscale) * (np.abs(xd[..., a_at]) + np.abs(xd[..., b_at]))
    mag[..., a_at] = mag[..., b_at] = both
    eps = torch.finfo(x.dtype).eps / 2 if x.dtype != torch.float32 else 0.0
    tol = 2.0 ** -21 * mag + eps * (np.abs(want) + 2.0 ** -21 * mag) + (2.0 ** -25 if x.dtype == torch.float16 else 0.0) * (mag > 0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert np.all(err <= tol), float((err - tol).max())


CASES = [
    # tokens, heads, dim, rope_dim, offset
    (1, 1, 64, 64, 0), (3, 64, 64, 64, 0), (16, 64, 576, 64, 512), (5, 7, 512, 64, 448), (9, 64, 128, 64, 0),
    (2, 3, 2, 2, 0), (7, 5, 11, 6, 3), (4, 2, 75, 74, 1), (2, 2, 256, 256, 0), (1000, 16, 64, 32, 16), (65, 1, 96, 8, 40),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_rope(shape, interleaved, dtype):
    n, heads, dim, rot, offset = shape
    g = torch.Generator("cuda").manual_seed(n * 1000 + dim)
    x = torch.randn(n, heads, dim, generator=g, device="cuda").to(DT[dtype])
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    t = api().RopeTable(rot, interleaved=interleaved)
    f = ar.rope_frequencies(rot)
    for transpose in (False, True):
        y = api().rope(x, pos, t, offset=offset, transpose=transpose)
        _check(y, x, pos, f, offset=offset, interleaved=interleaved, transpose=transpose)
        z = x.clone()
        assert api().rope(z, pos, t, offset=offset, transpose=transpose, out=z) is z
        assert torch.equal(z, y)                                      # in place: the same bits


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=8.0), dict(scaling="yarn", factor=40.0, original_ctx=4096)])
def test_scaled_tables_and_mscale(kw):
    x = torch.randn(33, 4, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    pos = torch.arange(33, device="cuda", dtype=torch.int32) * 31337
    y = api().rope(x, pos, api().RopeTable(64, mscale=1.369, **kw))
    _check(y, x, pos, ar.rope_frequencies(64, **kw), offset=0, interleaved=True, mscale=np.float32(1.369))


def test_extreme_positions():
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 12345678], dtype=torch.int32, device="cuda")
    x = torch.randn(6, 2, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    y = api().rope(x, pos, api().RopeTable(64))
    # the reference side's angles: 2^31 radians in doubles are good to 2^-22, so high-precision ones by splitting p f
    # into whole and fractional turns with integers
    t = api().RopeTable(64)
    turns = np.array([[(t.data.step[i] * int(p)) % (1 << 64) / 2.0 ** 64 for i in range(32)] for p in pos.tolist()])
    a, b = x.double().cpu().numpy()[..., 0::2], x.double().cpu().numpy()[..., 1::2]
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    got = y.double().cpu().numpy()
    tol = 2.0 ** -21 * (np.abs(a) + np.abs(b))
    assert np.all(np.abs(got[..., 0::2] - (a * c - b * s)) <= tol) and np.all(np.abs(got[..., 1::2] - (a * s + b * c)) <= tol)
    assert torch.equal(y[0], x[0])                                    # position 0 turns nothing


def test_strided_views_and_untouched_surroundings():
    """The rotary part of a projection into the rotary part of a query; every other byte stays."""
    g = torch.Generator("cuda").manual_seed(5)
    proj = torch.randn(6, 2, 64, 192, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.full((6, 2, 64, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.randint(0, 9000, (6, 2), generator=g, device="cuda", dtype=torch.int32)
    api().rope(proj[..., 128:], pos, api().RopeTable(64), out=q[..., 512:])
    _check(q[..., 512:], proj[..., 128:], pos, ar.rope_frequencies(64), offset=0, interleaved=True)
    assert torch.all(q[..., :512] == 7.0)
    # odd offsets: the element path
    buf = torch.randn(5, 3, 131, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.full((5, 3, 99), 3.0, dtype=torch.bfloat16, device="cuda")
    p = torch.arange(5, device="cuda", dtype=torch.int32)
    api().rope(buf[..., 1:68], p, api().RopeTable(64, interleaved=False), offset=3, out=out[..., 5:72])
    _check(out[..., 5:72], buf[..., 1:68], p, ar.rope_frequencies(64), offset=3, interleaved=False)
    assert torch.all(out[..., :5] == 3.0) and torch.all(out[..., 72:] == 3.0)
    # heads outermost, and one row broadcast to all heads
    xt = torch.randn(4, 9, 64, generator=g, device="cuda").transpose(0, 1)
    p = torch.arange(9, device="cuda", dtype=torch.int32)
    _check(api().rope(xt, p, api().RopeTable(64)), xt, p, ar.rope_frequencies(64), offset=0, interleaved=True)
    xe = torch.randn(9, 1, 64, generator=g, device="cuda").expand(9, 5, 64)
    _check(api().rope(xe, p, api().RopeTable(64)), xe, p, ar.rope_frequencies(64), offset=0, interleaved=True)


def test_refusals_on_the_device():
    x = torch.randn(4, 2, 64, device="cuda")
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    t = api().RopeTable(64)
    with pytest.raises(api().SmlaError):
        api().rope(x, p, t, out=torch.empty(4, 1, 64, device="cuda").expand(4, 2, 64))   # rows of out on one place
    with pytest.raises(ValueError):
        api().rope(x, p.cpu(), t)
    with pytest.raises(ValueError):
        api().rope(x.permute(0, 2, 1), p, api().RopeTable(2))
    assert api().rope(x[:0], p[:0], t).shape == (0, 2, 64)


def test_gradient_against_differences():
    """The transposed call is the gradient of sum(w * rope(x)): central differences of the fp64 oracle agree."""
    g = torch.Generator("cuda").manual_seed(6)
    x, w = (torch.randn(2, 1, 8, generator=g, device="cuda") for _ in range(2))
    pos = torch.tensor([3, 100], dtype=torch.int32, device="cuda")
    grad = api().rope(w, pos, api().RopeTable(8, interleaved=False, mscale=1.25), transpose=True).double().cpu().numpy()
    f, xd, wd = ar.rope_frequencies(8), x.double().cpu().numpy(), w.double().cpu().numpy()
    for i in np.ndindex(xd.shape):
        hi, lo = xd.copy(), xd.copy()
        hi[i] += 1e-3
        lo[i] -= 1e-3
        val = [(wd * ar.rope(v, [3, 100], f, offset=0, interleaved=False, mscale=1.25)).sum() for v in (hi, lo)]
        assert abs((val[0] - val[1]) / 2e-3 - grad[i]) <= 2.0 ** -21 * 1.25 * 2 * np.abs(wd).max() + 1e-9


def test_graph_stream_and_two_calls_at_once():
    g = torch.Generator("cuda").manual_seed(7)
    x = torch.randn(64, 64, 64, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(64, device="cuda", dtype=torch.int32)
    t = api().RopeTable(64)
    want, back = api().rope(x, pos, t), api().rope(x, pos, t, transpose=True)
    torch.cuda.synchronize()
    plan = api().RopePlan(x, pos, t)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        plan.run()
    with torch.cuda.stream(s2):
        other = api().rope(x, pos, t, transpose=True)
    torch.cuda.synchronize()
    assert torch.equal(plan.out, want) and torch.equal(other, back)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for k in (5, 77):
        pos.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(plan.out, api().rope(x, pos, t))


def test_many_items():
    """More head rows than one grid-wide index of 16 bits: spot rows of a 300,000-token call against the same rows alone."""
    x = torch.randn(300000, 8, 8, device="cuda", generator=torch.Generator("cuda").manual_seed(8)).to(torch.bfloat16)
    pos = torch.arange(300000, device="cuda", dtype=torch.int32)
    t = api().RopeTable(8)
    y = api().rope(x, pos, t)
    at = torch.tensor([0, 1, 65535, 65536, 299999], device="cuda")
    assert torch.equal(y[at], api().rope(x[at].contiguous(), pos[at].contiguous(), t))
