"""GPU tests of in-place compaction where several CTAs share a column: every
layout, one to eight CTAs, few and many steps, most rows moving a short way or a
long one.  Moved bytes are exact, so everything is compared for equality, several
times over."""
import numpy as np
import pytest
import torch

from test_gpu_evict import planes, random_cache

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
@pytest.mark.parametrize("B,n,budget", [(1, 1030, 1026), (1, 20000, 19990), (1, 20000, 700), (2, 9000, 5000), (5, 4000, 3900),
                                        (12, 3000, 1500), (40, 1500, 1400)])
def test_rows_of_every_layout(B, n, budget, kind):
    g = torch.Generator("cuda").manual_seed(B * n + budget)
    pps = -(-n // 64)
    pt = torch.randperm(B * pps, generator=g, device="cuda").to(torch.int32).view(B, pps)
    kv, rs = random_cache(kind, B * pps * 64, 5)
    keys = torch.randint(-9, 9, (B * pps * 64, 128), generator=g, device="cuda").to(torch.bfloat16)
    acc = torch.rand(B, n, generator=g, device="cuda")
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    ctx[0] = n - 1
    key = torch.where(torch.arange(n, device="cuda") < ctx[:, None], acc, -1.0)
    sel = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget].sort(1).values
    row = lambda p: (pt.gather(1, p // 64).long() * 64 + p % 64).cpu().numpy()  # noqa: E731
    src, dst = row(sel), row(torch.arange(budget, device="cuda").expand(B, -1))
    before = planes(kind, kv, rs, keys)
    want = {k: v.copy() for k, v in before.items()}
    for k in want:
        want[k][dst] = before[k][src]
    first = [t.clone() for t in (kv, keys)] + [None if rs is None else rs.clone()]
    for turn in range(4):
        kv.copy_(first[0])
        keys.copy_(first[1])
        if rs is not None:
            rs.copy_(first[2])
        kept, _, _ = api().evict(acc, ctx, budget, page_table=pt, kv=kv, kv_row_scale=rs, k_cache=keys,
                                 acc_out=torch.zeros_like(acc))
        assert torch.equal(kept.long(), sel)
        after = planes(kind, kv, rs, keys)
        for k in want:
            assert np.array_equal(after[k], want[k]), (k, turn)


@pytest.mark.parametrize("max_ctx", [8192, 8193, 40000, 70000])
def test_short_contexts_of_long_rows_with_lengths_in_place(max_ctx):
    """Nothing to evict, one to eight CTAs per sequence, the lengths written where the CTAs read them: out-of-range
    ones are clamped and reported."""
    B, budget = 40, max_ctx - 1
    pps = -(-max_ctx // 64)
    pt = torch.zeros(B, pps, dtype=torch.int32, device="cuda")
    kv, _ = random_cache("bf16", 64, 9)
    before = kv.view(torch.int16).clone()
    acc = torch.rand(B, max_ctx, device="cuda")
    lengths = [-5, 0, 1, budget, budget - 1] + [37 * b for b in range(B - 5)]
    for turn in range(3):
        ctx = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        out = torch.full_like(acc, 3.0)
        kept, new_len, _ = api().evict(acc, ctx, budget, page_table=pt, kv=kv, new_len=ctx, acc_out=out)
        torch.cuda.synchronize()
        assert new_len is ctx and ctx.tolist() == [max(n, 0) for n in lengths]
        for b, n in enumerate(lengths):
            n = max(n, 0)
            assert torch.equal(kept[b, :n], torch.arange(n, dtype=torch.int32, device="cuda")) and torch.all(kept[b, n:] == -1)
            assert torch.equal(out[b, :n], acc[b, :n]) and torch.all(out[b, n:] == 3.0)
        assert api().device_error() == 4
    assert torch.equal(kv.view(torch.int16), before)
