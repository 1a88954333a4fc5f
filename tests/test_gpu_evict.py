"""GPU tests of the eviction (sparse_mla_evict*): the selection and every moved
byte are exact, so everything is compared for equality; and the serving loop
that the operators make together, against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref

from test_gpu_append import make_cache

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


def planes(kind, kv, rs, keys):
    """name -> [rows, bytes] numpy copies of a cache."""
    if kind == "dsv4":
        a = kv.cpu().numpy()
        out = dict(slots=a[:, :36864].reshape(-1, 576).copy(), scales=a[:, 36864:].reshape(-1, 8).copy())
    else:
        out = dict(kv=kv.view(torch.uint8).cpu().numpy().reshape(kv.shape[0], -1).copy())
    if rs is not None:
        out["rs"] = rs.view(torch.uint8).cpu().numpy().reshape(-1, 4).copy()
    if keys is not None:
        out["keys"] = keys.view(torch.uint8).cpu().numpy().reshape(keys.shape[0], -1).copy()
    return out


def random_cache(kind, rows, seed):
    kv, rs = make_cache(kind, rows)
    g = torch.Generator("cuda").manual_seed(seed)
    kv.view(torch.uint8).copy_(torch.randint(0, 256, kv.view(torch.uint8).shape, generator=g, device="cuda", dtype=torch.uint8))
    if rs is not None:
        rs.normal_(generator=g)
    return kv, rs


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind,keys", [("bf16", False), ("fp8", True), ("dsv4", True)])
@pytest.mark.parametrize("max_ctx,budget,sinks,recent", [(1, 1, 0, 0), (64, 63, 1, 2), (130, 64, 0, 0), (1000, 333, 4, 100),
                                                         (5000, 1025, 0, 1025), (9001, 8191, 3, 77)])
def test_evict(max_ctx, budget, sinks, recent, kind, keys, in_place):
    rng = np.random.default_rng(max_ctx + budget)
    B, pps = 5, -(-max_ctx // 64) + 1
    npps = -(-budget // 64)
    pages = B * (pps + npps)
    perm = rng.permutation(pages).astype(np.int32)
    pt, npt = perm[:B * pps].reshape(B, pps), perm[B * pps:].reshape(B, npps)
    ctx = np.array([max_ctx, 0, min(budget, max_ctx), min(budget + 1, max_ctx), rng.integers(0, max_ctx + 1)], np.int32)
    acc = np.round(rng.exponential(1.0, (B, max_ctx)), 1).astype(np.float32)       # many ties
    acc[0, rng.random(max_ctx) < 0.3] = 0.0
    acc[3, rng.random(max_ctx) < 0.2] = np.nan
    acc[4, ::7] = -np.inf
    kv, rs = random_cache(kind, pages * 64, 1)
    k_cache = torch.randn(pages * 64, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(torch.bfloat16) if keys else None
    before = planes(kind, kv, rs, k_cache)
    dev = lambda a: torch.from_numpy(a.copy()).cuda()  # noqa: E731
    d_acc, d_ctx, d_pt, d_npt = dev(acc), dev(ctx), dev(pt), dev(npt)
    kw = dict(page_table=d_pt, kv=kv, kv_row_scale=rs, k_cache=k_cache, sinks=sinks, recent=recent,
              new_page_table=None if in_place else d_npt)
    if in_place:
        kept, new_len, out = api().evict(d_acc, d_ctx, budget, new_len=d_ctx, **kw)      # everything in place
        assert out is d_acc and new_len is d_ctx
        rest = acc
    else:
        rest = np.full((B, max_ctx), 5.0, np.float32)
        kept, new_len, out = api().evict(d_acc, d_ctx, budget, acc_out=dev(rest), **kw)
        assert torch.equal(d_acc.view(torch.int32), dev(acc).view(torch.int32)) and torch.equal(d_ctx, dev(ctx))
    torch.cuda.synchronize()
    after = planes(kind, kv, rs, k_cache)
    want = {k: v.copy() for k, v in before.items()}
    for b in range(B):
        sel = ar.evict_select(acc[b], int(ctx[b]), budget, sinks, recent)
        m = len(sel)
        assert new_len[b].item() == m and kept[b].tolist() == sel + [-1] * (budget - m)
        wa = rest[b].copy()
        wa[:ctx[b]] = 0
        wa[:m] = acc[b][sel]
        assert np.array_equal(out[b].cpu().numpy(), wa, equal_nan=True)
        src = np.array([pt[b, i // 64] * 64 + i % 64 for i in sel], np.int64)
        table = pt if in_place else npt
        dst = np.array([table[b, i // 64] * 64 + i % 64 for i in range(m)], np.int64)
        for k in want:
            want[k][dst] = before[k][src]
    for k in want:
        assert np.array_equal(after[k], want[k]), k


@pytest.mark.parametrize("n,budget", [(70000, 20000), (200001, 150000)])
def test_long_contexts(n, budget):
    g = torch.Generator("cuda").manual_seed(n)
    acc = torch.round(torch.rand(2, n, generator=g, device="cuda") * 1000) / 8            # ties
    pps = -(-n // 64)
    pt = torch.randperm(2 * pps, generator=g, device="cuda").to(torch.int32).view(2, pps)
    kv, rs = random_cache("fp8", 2 * pps * 64, 3)
    old, old_rs = kv.clone(), rs.clone()
    ctx = torch.tensor([n, n - 17], dtype=torch.int32, device="cuda")
    kept, new_len, out = api().evict(acc, ctx, budget, page_table=pt, kv=kv, kv_row_scale=rs, sinks=5, recent=999,
                                     acc_out=torch.zeros_like(acc))
    for b in range(2):
        m = int(ctx[b])
        key = acc[b, :m].clone()
        key[:5] = torch.inf
        key[m - 999:] = torch.inf
        sel = torch.sort(key, descending=True, stable=True).indices[:budget].sort().values
        assert torch.equal(kept[b].long(), sel) and int(new_len[b]) == budget
        assert torch.equal(out[b, :budget], acc[b][sel]) and torch.all(out[b, budget:] == 0)
        row = lambda p: pt[b, p // 64].long() * 64 + p % 64  # noqa: E731
        i = torch.arange(budget, device="cuda")
        assert torch.equal(kv[row(i)], old[row(sel)]) and torch.equal(rs[row(i)], old_rs[row(sel)])
        tail = torch.arange(budget, m, device="cuda")
        assert torch.equal(kv[row(tail)], old[row(tail)])


@pytest.mark.parametrize("n,budget", [(131072, 131000), (131073, 60000), (300000, 299990)])
def test_long_selection_in_place(n, budget):
    """The accumulated weights and the lengths overwritten in place, on both sides of the border between the two kernels."""
    g = torch.Generator("cuda").manual_seed(n)
    acc = torch.round(torch.rand(1, n, generator=g, device="cuda") * 50)
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    pps = -(-n // 64)
    pt = torch.arange(pps, dtype=torch.int32, device="cuda")[None]
    kv, rs = random_cache("fp8", pps * 64, 6)
    old, old_rs, before = kv.clone(), rs.clone(), acc.clone()
    kept, new_len, out = api().evict(acc, ctx, budget, page_table=pt, kv=kv, kv_row_scale=rs, recent=3, new_len=ctx)
    assert out is acc and new_len is ctx and ctx.item() == budget
    key = before[0].clone()
    key[n - 3:] = torch.inf
    sel = torch.sort(key, descending=True, stable=True).indices[:budget].sort().values
    assert torch.equal(kept[0].long(), sel)
    assert torch.equal(acc[0, :budget], before[0][sel]) and torch.all(acc[0, budget:] == 0)
    assert torch.equal(kv[:budget], old[sel]) and torch.equal(rs[:budget], old_rs[sel])
    assert torch.equal(kv[budget:], old[budget:])


def test_context_and_pages_out_of_range():
    acc = torch.rand(2, 128, device="cuda")
    kv, _ = random_cache("bf16", 256, 4)
    before = kv.view(torch.int16).clone()
    pt = torch.tensor([[0, 4], [-1, 2]], dtype=torch.int32, device="cuda")
    kept, new_len, _ = api().evict(acc, torch.tensor([500, -3], dtype=torch.int32, device="cuda"), 100, page_table=pt, kv=kv)
    torch.cuda.synchronize()
    assert api().device_error() == 4
    assert new_len.tolist() == [100, 0] and torch.all(kept[1] == -1)
    # rows of page 0 that came from the missing page were not moved, pages 1 - 3 were not touched
    assert torch.equal(kv.view(torch.int16)[64:], before[64:])
    moved = kept[0] < 64
    assert torch.equal(kv.view(torch.int16)[:100][:64][moved[:64]], before[kept[0][:64][moved[:64]].long()])


def test_selection_and_compaction_alone_and_in_a_graph():
    rng = np.random.default_rng(8)
    B, n, budget = 3, 640, 200
    pt = torch.from_numpy(rng.permutation(B * 10).reshape(B, 10).astype(np.int32)).cuda()
    kv, rs = random_cache("fp8", B * 640, 5)
    kv2, rs2 = kv.clone(), rs.clone()
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    acc = torch.rand(B, n, device="cuda")
    plan = api().EvictPlan(acc, ctx, budget, page_table=pt, kv=kv, kv_row_scale=rs, acc_out=torch.zeros_like(acc))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        plan.run()
    g.replay()
    torch.cuda.synchronize()
    import ctypes
    L, p = api().lib, lambda t: t.data_ptr()  # noqa: E731
    kept, new_len, out = torch.empty_like(plan.kept), torch.empty_like(plan.new_len), torch.zeros_like(acc)
    s = torch.cuda.current_stream().cuda_stream
    assert L.sparse_mla_evict_select(ctypes.byref(plan.shape), p(acc), p(ctx), p(kept), p(new_len), p(out), s) == 0
    assert L.sparse_mla_evict_compact(ctypes.byref(plan.shape), p(kept), p(new_len), p(pt), None, p(kv2), p(rs2), None, s) == 0
    torch.cuda.synchronize()
    assert torch.equal(kept, plan.kept) and torch.equal(out, plan.acc_out) and torch.equal(kv, kv2) and torch.equal(rs, rs2)


# ------------------------------------------------------- the loop they make
@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
def test_serving_loop(kind):
    """Prompt appended, decode steps with weights accumulated, one eviction, more steps: every decode against the oracle
    over the rows that the cache should then hold."""
    a = api()
    rng = np.random.default_rng(21)
    B, prompt, budget, steps, max_ctx = 3, 150, 96, 4, 192
    d = 512 if kind == "dsv4" else 576
    pps = max_ctx // 64
    pages = B * pps
    pt = torch.from_numpy(rng.permutation(pages).reshape(B, pps).astype(np.int32)).cuda()
    kv, rs = make_cache(kind, pages * 64, fill=0)
    paged = dict(kv_row_scale=rs, page_table=pt, page_size=64)
    table, scale = a.RopeTable(64), 1 / np.sqrt(d)
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(512)).astype(np.float32)).cuda()
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda().to(torch.bfloat16)  # noqa: E731
    i32 = lambda v: torch.as_tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ctx, position = np.full(B, prompt), prompt
    a.cache_append(normal(B * prompt, d), kv, i32(np.tile(np.arange(prompt), B)), norm_weight=w, rope=table,
                   positions=i32(np.tile(np.arange(prompt), B)), **paged)
    acc = torch.zeros(B, max_ctx, device="cuda")
    held = [list(range(prompt)) for _ in range(B)]           # original positions, in cache order
    total = np.zeros((B, max_ctx))
    fmt = {"bf16": "bf16", "fp8": "fp8_e4m3_rowscale", "dsv4": "dsv4_paged"}[kind]
    for step in range(2 * steps):
        if step == steps:
            kept, new_len, _ = a.evict(acc, i32(ctx), budget, page_table=pt, kv=kv, kv_row_scale=rs, sinks=2, recent=8)
            for b in range(B):
                k = kept[b, :int(new_len[b])].tolist()
                assert k == ar.evict_select(before_acc[b], int(ctx[b]), budget, 2, 8)
                held[b] = [held[b][i] for i in k]
                total[b] = np.concatenate([total[b][k], np.zeros(max_ctx - len(k))])
            ctx = new_len.cpu().numpy().astype(np.int64)
        a.cache_append(normal(B, d), kv, i32(ctx), norm_weight=w, rope=table, positions=i32(np.full(B, position)), **paged)
        for b in range(B):
            held[b].append(position)
        ctx, position = ctx + 1, position + 1
        q = normal(B, 64, d)
        a.rope(q, i32(np.full(B, position - 1)), table, out=q)
        idx = np.full((B, 160), -1, np.int32)
        for b in range(B):
            idx[b, :ctx[b]] = rng.permutation(ctx[b])
        out, lse = a.decode(q, kv, i32(idx), scale, **paged)
        if kind == "dsv4":                                  # the value's rotated dims are turned back
            a.rope(out, i32(np.full(B, position - 1)), table, transpose=True, out=out)
        weights = a.attention_weights(q, kv, i32(idx), lse, scale, **paged)
        a.accumulate_weights(acc, i32(idx), weights)
        before_acc = acc.cpu().numpy()
        bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        np_kv = kv.cpu().numpy() if kv.dtype == torch.uint8 else bits(kv)
        want, wl = ref.sparse_mla_decode(bits(q), np_kv, idx, scale, kv_format=fmt, page_table=pt.cpu().numpy(), page_size=64,
                                         kv_row_scale=None if rs is None else rs.cpu().numpy())
        if kind == "dsv4":
            want = ar.rope(want, np.full(B, position - 1), ar.rope_frequencies(64), offset=448, interleaved=True, transpose=True)
        assert np.abs(out.double().cpu().numpy() - want).max() <= 2e-2
        assert ref.lse_rel_err(lse.cpu().numpy(), wl).max() <= 1e-3
        qd = ref.bf16_bits_to_f64(bits(q))
        for b in range(B):
            one, _, _ = ar.list_weights(qd[b], np_kv, idx[b], wl[b], scale, kv_format=fmt, page_table_row=pt[b].cpu().numpy(),
                                        kv_row_scale=None if rs is None else rs.cpu().numpy(), page_size=64)
            total[b] = ar.accumulate(total[b:b + 1], idx[b:b + 1], one[None], 1.0)[0]
        # lse within 1e-3 of max(|lse|, 1) moves a weight by as much, relatively
        bound = 2e-3 * np.maximum(np.abs(wl).max(), 1) * (step + 1)
        assert np.all(np.abs(before_acc - total) <= bound * total + 1e-6)
        assert all(len(h) == c for h, c in zip(held, ctx))
