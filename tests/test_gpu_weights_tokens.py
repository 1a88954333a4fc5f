"""GPU parity for the attention weights of several query tokens per sequence over
DeepSeek-V4 slots: every token has its own query and list, all of a sequence's read
its row of the page table."""
import numpy as np
import pytest
import torch

from sparse_mla_decode_05_b200 import inputs

from _helpers import Dev
from test_gpu_weights_outliers import check
from test_gpu_weights_slots import mixed_scales, oracle_lse, run

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


@pytest.mark.parametrize("B,T,k", [(1, 2, 1), (3, 4, 250), (2, 16, 129), (40, 5, 300), (1, 3, 700)])
def test_tokens_match_single_ones_and_the_oracle(B, T, k):
    # each token as a sequence of its own, its page-table row its sequence's
    w = inputs.paged_dsv4(B * T, 1024, B * T * 16, k, seed=321)
    mixed_scales(w, 9)
    w.page_table[:] = w.page_table[::T].repeat_interleave(T, 0)
    g = torch.Generator().manual_seed(11)
    for r in range(B * T):
        w.indices[r] = torch.randperm(1024, generator=g)[:k].int()
    if k > 100:
        w.indices[0, 40:77] = -1
        w.indices[B * T - 1, :60] = -1
    if B * T > 10:
        w.indices[7] = -1
    lse = oracle_lse(w)
    d = Dev(w)
    single = run(d, lse)
    rows = [r for r in range(B * T) if torch.any(w.indices[r] >= 0)]
    assert all(torch.all(single[r] == 0) for r in range(B * T) if r not in rows)
    sub = inputs.dataclasses.replace(w, q=w.q[rows], indices=w.indices[rows], page_table=w.page_table[rows])
    check(sub, single[rows], lse[rows])
    multi = api().attention_weights(d.q.view(B, T, 64, 512), d.kv, d.indices.view(B, T, k), lse.view(B, T, 64), w.scale,
                                    page_table=d.page_table[::T].contiguous(), page_size=64)
    assert multi.shape == (B, T, k) and torch.equal(multi.view(B * T, k), single)


def test_tokens_with_the_decodes_own_lse():
    B, T, k = 4, 2, 509
    w = inputs.paged_dsv4(B, 2048, 140, k, seed=322)
    g = torch.Generator().manual_seed(12)
    q = torch.randn(B, T, 64, 512, generator=g).to(torch.bfloat16).cuda()
    idx = torch.stack([torch.stack([torch.randperm(2048, generator=g)[:k] for _ in range(T)]) for _ in range(B)]).int().cuda()
    kv, pt = w.kv.cuda(), w.page_table.cuda()
    _, lse = api().decode(q, kv, idx, w.scale, page_table=pt, page_size=64)
    got = api().attention_weights(q, kv, idx, lse, w.scale, page_table=pt, page_size=64)
    assert np.allclose(got.double().sum(-1).cpu().numpy(), 64.0, rtol=2.0 ** -10)
