"""GPU tests of the accumulation over weights of very different size: a position's
sum keeps its digits whatever weight others of the sequence get.

Bound.  A position's weights are summed in fixed point whose unit is at most
2^-61 of (entries, as a power of two) x the position's own largest |weight|, half a
unit lost per entry; then one fp32 rounding of the result, 2^-24 of it, or half a
subnormal step, 2^-150."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def check(acc0, idx, w, decay, got):
    acc0, idx, w, got = (t.double().cpu().numpy() for t in (acc0, idx, w, got))
    n = 2.0 ** np.ceil(np.log2(idx.shape[1]))
    for b in range(idx.shape[0]):
        ok = idx[b] >= 0
        at = idx[b][ok].astype(np.int64)
        want, count, top = float(np.float32(decay)) * acc0[b], np.zeros(acc0.shape[1]), np.zeros(acc0.shape[1])
        np.add.at(want, at, w[b][ok])
        np.add.at(count, at, 1.0)
        np.maximum.at(top, at, np.abs(w[b][ok]))
        tol = 0.5 * count * 2.0 ** -61 * n * top + 2.0 ** -24 * np.abs(want) * (1 + 2.0 ** -20) + 2.0 ** -150
        assert np.all(np.abs(got[b] - want) <= tol), float((np.abs(got[b] - want) / tol).max())


def test_small_weights_beside_a_large_one():
    idx = torch.arange(4096, dtype=torch.int32, device="cuda")[None]
    w = torch.full((1, 4096), 64.0, device="cuda")
    w[0, 1:6] = torch.tensor([5e-14, 1e-12, 1e-20, 1e-30, 1e-40])
    acc = torch.zeros(1, 5000, device="cuda")
    api().accumulate_weights(acc, idx, w)
    assert torch.equal(acc[:, :4096], w)                       # one weight per position: nothing is rounded
    api().accumulate_weights(acc, idx, w, decay=0.5)
    check(w, idx, w, 0.5, acc[:, :4096])


@pytest.mark.parametrize("B,k,n,decay", [(1, 3, 2, 1.0), (2, 4096, 4096, 1.0), (3, 2048, 8192, 0.5), (70, 700, 9000, 1.0), (1, 30000, 5000, 0.25)])
def test_weights_over_the_whole_range(B, k, n, decay):
    g = torch.Generator("cuda").manual_seed(k + n)
    idx = torch.randint(-1, n, (B, k), generator=g, device="cuda", dtype=torch.int32)
    size = 10.0 ** torch.randint(-38, 30, (B, n + 1), generator=g, device="cuda").double()
    w = (torch.rand(B, k, generator=g, device="cuda").double() * size.gather(1, idx.long() % (n + 1))).float()
    w = torch.where(torch.rand(B, k, generator=g, device="cuda") < 0.2, -w, w)
    acc = torch.rand(B, n, generator=g, device="cuda") * size[:, :n].float() * 1e-3
    acc0 = acc.clone()
    api().accumulate_weights(acc, idx, w, decay=decay)
    check(acc0, idx, w, decay, acc)
    again = acc0.clone()
    perm = torch.randperm(k, device="cuda")
    api().accumulate_weights(again, idx[:, perm].contiguous(), w[:, perm].contiguous(), decay=decay)
    assert torch.equal(again, acc)
