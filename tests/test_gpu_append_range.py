"""GPU tests of the cache append's norm at the ends of fp32's range, against the
fp64 oracle: rows whose values, products or squares leave the range that the
rest of the arithmetic expects, although the stored values are ordinary ones.

Tolerances.  As for other rows: a normed value within 2^-17 of itself, plus what
subnormal intermediates lose (half of 2^-149, times at most 2^15 on the way to
the stored value: below 2^-134).  Codes round by 2^-4 of the value or 2^-10 of the scale, bf16
by 2^-8 or half its subnormal step, 2^-134; the scale by 2^-16, at least 2^-126."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref

from test_gpu_append import make_cache

pytestmark = pytest.mark.gpu
LEAST = 2.0 ** -126


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def append(kind, x, w, eps, table=None, positions=None):
    """The rows x appended to a fresh cache: stored values and their steps [n, d] (bf16 steps are relative, 0)."""
    n = x.shape[0]
    rows = -(-n // 64) * 64
    kv, rs = make_cache(kind, rows)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    paged = dict(page_table=torch.arange(rows // 64, dtype=torch.int32, device="cuda")[None], page_size=64) if kind == "dsv4" else {}
    api().cache_append(x, kv, slots, kv_row_scale=rs, norm_weight=w, eps=eps, rope=table, positions=positions, **paged)
    torch.cuda.synchronize()
    if kind == "bf16":
        return ref.bf16_bits_to_f64(kv.view(torch.int16).cpu().numpy().view(np.uint16)[:n]), None
    if kind == "fp8":
        scale = rs.double().cpu().numpy()[:n]
        return ref.e4m3fn_to_f64(kv.cpu().numpy()[:n]) * scale[:, None], scale
    blocks = kv[:, 36864:].cpu().numpy().reshape(-1, 8)[:n, :7]
    return ref.dsv4_rows_f64(kv.cpu().numpy(), np.arange(n)), 2.0 ** (blocks.astype(np.float64) - 127)


def check(kind, got, scale, want):
    assert np.all(np.isfinite(got)), "a stored value is not finite"
    lead = 2.0 ** -17 * np.abs(want) + 2.0 ** -134
    coded = np.maximum(2.0 ** -4 * np.abs(want) * (1 + 2.0 ** -10), 0.0)
    as_bf16 = 2.0 ** -8 * np.abs(want) + 2.0 ** -134
    if kind == "bf16":
        tol = lead + as_bf16
    elif kind == "fp8":
        ws = np.maximum(np.abs(want).max(1) / 448, LEAST)
        ws = np.where(np.abs(want).max(1) > 0, ws, 1.0)
        assert np.all(np.abs(scale - ws) <= 2.0 ** -16 * ws)
        tol = lead + np.maximum(coded, 2.0 ** -10 * scale[:, None])
    else:
        groups = np.abs(want[:, :448]).reshape(-1, 7, 64).max(2)
        assert np.array_equal(scale, 2.0 ** np.vectorize(ar.group_exponent)(groups).astype(np.float64))
        step = np.repeat(scale, 64, 1) * 2.0 ** -10
        tol = np.concatenate([lead[:, :448] + np.maximum(coded[:, :448], step), lead[:, 448:] + as_bf16[:, 448:]], 1)
    err = np.abs(got - want)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
@pytest.mark.parametrize("weight", [1.0, 1e-5])
def test_normed_rows_of_tiny_values(kind, weight):
    """eps keeps 1 / rms near 1,000, so the row's largest value stands far below every other number on the way."""
    d = 512 if kind == "dsv4" else 576
    rng = np.random.default_rng(51)
    x = np.zeros((16, d), np.float32)
    for i, v in enumerate((3e-38, 1e-37, 1e-36, 6e-39, 1e-39, 1e-40, 3e-34, 1e-30)):
        x[i, 7 + 30 * i] = v                                        # one element, the rest zeros
        x[8 + i, :512] = v * rng.uniform(-1, 1, 512)                # a mix of magnitudes
        x[8 + i, ::3] = 0
    x = torch.from_numpy(x).cuda()
    w = torch.full((512,), weight, device="cuda")
    got, scale = append(kind, x, w, 1e-6)
    check(kind, got, scale, ar.append_rows(x.double().cpu().numpy(), norm_weight=w.double().cpu().numpy(), eps=float(np.float32(1e-6))))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
def test_tiny_weights_and_rotated_parts_of_every_size(kind):
    """Ordinary rows whose weights make the latent part tiny, beside a rotated part that is zero, tiny or ordinary."""
    d = 512 if kind == "dsv4" else 576
    rng = np.random.default_rng(52)
    x = rng.standard_normal((12, d)).astype(np.float32)
    if kind != "dsv4":
        for i, v in enumerate((0.0, 1e-37, 1e-20, 1.0)):
            x[3 * i:3 * i + 3, 512:] *= v
    x = torch.from_numpy(x).cuda()
    table, pos = api().RopeTable(64), torch.arange(12, dtype=torch.int32, device="cuda")
    for weight in (1e-36, 3e-30, 1e-12):
        w = torch.from_numpy((weight * (1 + 0.2 * rng.standard_normal(512))).astype(np.float32)).cuda()
        got, scale = append(kind, x, w, 1e-6, table, pos)
        want = ar.append_rows(x.double().cpu().numpy(), norm_weight=w.double().cpu().numpy(), eps=float(np.float32(1e-6)),
                              freq=ar.rope_frequencies(64), positions=np.arange(12))
        # the rotation adds 2^-20 of the pair to a rotated value, which the codes' own rounding of it need not cover
        both = np.zeros_like(want)
        both[:, -64:] = np.abs(want[:, -64:]).max(1, keepdims=True)
        near = np.abs(got - want) <= 2.0 ** -20 * both
        check(kind, np.where(near, want, got), scale, want)
