"""The operators around the decode in the settings that their own tests leave
out: side streams, captured graphs, rows beyond 2^32 bytes of a pool, pages at
the pool's end, and repeated runs that must give the same bits."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref

from test_gpu_append import check_rows, make_cache
from test_gpu_evict import random_cache

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


FAR = 4_000_000          # bf16 rows of 1,152 bytes: 4.6 GB


def test_append_weights_and_eviction_beyond_32_bit_offsets():
    a = api()
    rng = np.random.default_rng(31)
    kv = torch.empty(FAR, 576, dtype=torch.bfloat16, device="cuda")
    B, per = 2, 256
    pages = np.stack([np.arange(FAR // 64 - 4, FAR // 64), np.arange(FAR // 64 - 8, FAR // 64 - 4)]).astype(np.int32)
    pt = torch.from_numpy(pages).cuda()
    x = torch.from_numpy(rng.standard_normal((B * per, 576)).astype(np.float32)).cuda()
    slots = torch.arange(per, dtype=torch.int32, device="cuda").repeat(B)
    a.cache_append(x, kv, slots, page_table=pt, page_size=64)
    low = FAR - 8 * 64
    rows = kv[low:].clone()
    order = np.concatenate([np.arange(256) + 256, np.arange(256)])          # sequence 0 lies in the last four pages
    want = x.double().cpu().numpy()
    got = rows.double().cpu().numpy()
    assert np.all(np.abs(got[order] - want) <= 2.0 ** -8 * np.abs(want))
    # weights over the far rows, flat and paged, against a small copy of them
    q = torch.from_numpy(rng.standard_normal((B, 64, 576)).astype(np.float32)).cuda().to(torch.bfloat16)
    idx = torch.from_numpy(np.stack([rng.permutation(per)[:200] for _ in range(B)]).astype(np.int32)).cuda()
    lse = torch.full((B, 64), 3.0, device="cuda")
    near = a.attention_weights(q, rows, idx, lse, 1 / 24, page_table=pt - low // 64, page_size=64)
    far = a.attention_weights(q, kv, idx, lse, 1 / 24, page_table=pt, page_size=64)
    flat = (pt.gather(1, (idx // 64).long()) * 64 + idx % 64).to(torch.int32)
    assert torch.equal(near, far) and torch.equal(near, a.attention_weights(q, kv, flat, lse, 1 / 24))
    # eviction of the far pages, in place
    acc = torch.rand(B, per, device="cuda")
    ctx = torch.full((B,), per, dtype=torch.int32, device="cuda")
    kept, new_len, _ = a.evict(acc, ctx, 100, page_table=pt, kv=kv, acc_out=torch.zeros_like(acc))
    for b in range(B):
        assert kept[b].tolist() == ar.evict_select(acc[b].cpu().numpy(), per, 100, 0, 0)
        i = torch.arange(100, device="cuda")
        row = lambda p: pt[b, p // 64].long() * 64 + p % 64  # noqa: E731
        assert torch.equal(kv[row(i)], rows[row(kept[b].long()) - low])


def test_fp8_and_dsv4_rows_beyond_32_bit_offsets():
    a = api()
    n = 8_000_000                                                           # 4.6 GB of 576-byte rows
    x = torch.randn(3, 576, device="cuda")
    kv = torch.empty(n, 576, dtype=torch.uint8, device="cuda")
    rs = torch.empty(n, device="cuda")
    slots = torch.tensor([n - 1, n - 64, 7_900_001], dtype=torch.int32, device="cuda")
    a.cache_append(x, kv, slots, kv_row_scale=rs)
    at = slots.long()
    small, srs = kv[at].clone(), rs[at].clone()
    check_rows("fp8", small, srs, np.arange(3), x.double().cpu().numpy())
    q = torch.randn(1, 64, 576, device="cuda").to(torch.bfloat16)
    lse = torch.full((1, 64), 2.0, device="cuda")
    i3 = torch.arange(3, dtype=torch.int32, device="cuda")[None]
    assert torch.equal(a.attention_weights(q, kv, slots[None], lse, 0.04, kv_row_scale=rs),
                       a.attention_weights(q, small, i3, lse, 0.04, kv_row_scale=srs))
    del kv, rs
    pages = 130_000                                                         # 4.9 GB of 37,376-byte pages
    kv = torch.empty(pages, 37376, dtype=torch.uint8, device="cuda")
    pt = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 63, 17], dtype=torch.int32, device="cuda")
    a.cache_append(x[:, :512].contiguous(), kv, slots, page_table=pt, page_size=64)
    last = kv[pages - 1:].clone()
    check_rows("dsv4", last, None, slots.cpu().numpy(), x[:, :512].double().cpu().numpy())
    q = torch.randn(1, 64, 512, device="cuda").to(torch.bfloat16)
    assert torch.equal(a.attention_weights(q, kv, slots[None], lse, 0.04, page_table=pt, page_size=64),
                       a.attention_weights(q, last, slots[None], lse, 0.04, page_table=torch.zeros_like(pt), page_size=64))


def _step(a, seed=0):
    """One serving step's calls as plans over fixed buffers, and the buffers they write."""
    g = torch.Generator("cuda").manual_seed(seed)
    B, n, k = 6, 700, 300
    pps = 11
    perm = torch.randperm(B * pps, generator=g, device="cuda").to(torch.int32).view(B, pps)
    kv, rs = random_cache("fp8", B * pps * 64, seed)
    kv.view(torch.uint8).bitwise_and_(0x77)                                 # finite codes
    rs.fill_(0.01)
    x = torch.randn(B, 576, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(B, 64, 576, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.full((B,), n, dtype=torch.int32, device="cuda")
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    idx = torch.rand(B, n, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    acc = torch.rand(B, n, generator=g, device="cuda")
    lse = torch.full((B, 64), 1.0, device="cuda")
    t = a.RopeTable(64)
    paged = dict(kv_row_scale=rs, page_table=perm, page_size=64)
    w = a.AttentionWeightsPlan(q, kv, idx, lse, 1 / 24, **paged)
    plans = [a.CacheAppendPlan(x, kv, pos - 1, rope=t, positions=pos, norm_weight=torch.ones(512, device="cuda"), **paged),
             a.RopePlan(q, pos, t, out=q), w, a.AccumulateWeightsPlan(acc, idx, w.out, decay=0.9),
             a.EvictPlan(acc, ctx, 333, page_table=perm, kv=kv, kv_row_scale=rs, sinks=4, recent=50)]
    return plans, [kv, rs, q, w.out, acc, plans[-1].kept, plans[-1].new_len]


def test_a_step_on_a_side_stream_and_in_a_graph_gives_the_same_bits():
    a = api()
    plans, want = _step(a)
    for p in plans:
        p.run()
    torch.cuda.synchronize()
    for how in ("stream", "graph", "given stream"):
        plans, got = _step(a)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        if how == "stream":
            with torch.cuda.stream(s):
                for p in plans:
                    p.run()
        elif how == "given stream":
            for p in plans:
                p.run(s)
        else:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for p in plans:
                    p.run()
            g.replay()
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u, v), how


def test_two_steps_at_once_on_two_streams():
    """Calls that overlap share nothing: each stream's results are those it has alone."""
    a = api()
    want = []
    for seed in (1, 2):
        plans, out = _step(a, seed)
        for p in plans:
            p.run()
        torch.cuda.synchronize()
        want.append(out)
    for _ in range(5):
        both = [_step(a, seed) for seed in (1, 2)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for i in range(len(both[0][0])):
            for (plans, _), s in zip(both, streams):
                plans[i].run(s)
        torch.cuda.synchronize()
        for (_, got), w in zip(both, want):
            for u, v in zip(got, w):
                assert torch.equal(u, v)


def test_in_place_eviction_of_many_shapes_repeats_its_bits():
    """Batches and budgets that the compaction spreads over one to eight CTAs per column, against a gather."""
    a = api()
    for B, n, budget in ((1, 5000, 4990), (1, 4097, 600), (2, 9000, 5000), (7, 3000, 2900), (24, 2000, 1000), (70, 1500, 700)):
        g = torch.Generator("cuda").manual_seed(B * n)
        pps = -(-n // 64)
        pt = torch.randperm(B * pps, generator=g, device="cuda").to(torch.int32).view(B, pps)
        kv = torch.randn(B * pps * 64, 576, generator=g, device="cuda").to(torch.bfloat16)
        keys = torch.randn(B * pps * 64, 128, generator=g, device="cuda").to(torch.bfloat16)
        acc = torch.rand(B, n, generator=g, device="cuda")
        ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
        for _ in range(3):
            kv1, keys1 = kv.clone(), keys.clone()
            kept, _, _ = a.evict(acc, ctx, budget, page_table=pt, kv=kv1, k_cache=keys1, acc_out=torch.zeros_like(acc))
            src = (pt.gather(1, (kept // 64).long()) * 64 + kept % 64).long()
            i = torch.arange(budget, device="cuda").expand(B, -1)
            dst = (pt.gather(1, i // 64) * 64 + i % 64).long()
            want, wkeys = kv.clone(), keys.clone()
            want[dst], wkeys[dst] = kv[src], keys[src]
            assert torch.equal(kv1, want) and torch.equal(keys1, wkeys), (B, n, budget)


def test_accumulate_widest_row_and_graph():
    a = api()
    n = 1 << 20
    acc = torch.zeros(1, n, device="cuda")
    idx = torch.tensor([[0, n - 1, 4095, 4096, n - 1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, 2.0, 3.0, 4.0, 0.5]], device="cuda")
    plan = a.AccumulateWeightsPlan(acc, idx, w, decay=0.5)
    plan.run()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        plan.run()
    g.replay()
    torch.cuda.synchronize()
    assert acc[0, [0, 4095, 4096, n - 1]].tolist() == [1.5, 4.5, 6.0, 3.75] and acc.sum().item() == 15.75


def test_decode_reads_what_append_wrote():
    """Equal rows appended in the three layouts give the decode of those rows, padding-only sequences included."""
    a = api()
    rng = np.random.default_rng(41)
    for kind, d in (("bf16", 576), ("fp8", 576), ("dsv4", 512)):
        kv, rs = make_cache(kind, 256, fill=0)
        x = torch.from_numpy(rng.standard_normal((128, d)).astype(np.float32)).cuda()
        pt = torch.tensor([[3, 1], [0, 2]], dtype=torch.int32, device="cuda")
        paged = dict(kv_row_scale=rs, page_table=pt, page_size=64)
        a.cache_append(x, kv, torch.arange(64, dtype=torch.int32, device="cuda").repeat(2) + 60, **paged)
        q = torch.from_numpy(rng.standard_normal((2, 64, d)).astype(np.float32)).cuda().to(torch.bfloat16)
        idx = torch.full((2, 70), -1, dtype=torch.int32, device="cuda")
        idx[0, :64] = torch.randperm(64, device="cuda").int() + 60
        out, lse = a.decode(q, kv, idx, 0.04, **paged)
        w = a.attention_weights(q, kv, idx, lse, 0.04, **paged)
        rows = x[:64].double().cpu().numpy()
        o, l = ref.attend_rows(q[0].double().cpu().numpy(), rows, 0.04, 512)
        tol = {"bf16": 2.0 ** -7, "fp8": 2.0 ** -2, "dsv4": 2.0 ** -2}[kind]       # the rows' own rounding, amplified by the scores
        assert np.abs(out[0].double().cpu().numpy() - o).max() <= tol
        assert torch.all(out[1] == 0) and torch.all(w[1] == 0)
        assert abs(w[0].sum().item() - 64) <= 64 * 2.0 ** -10
