"""The serving loop that append, eviction and the rest make together, by the rows
it should then hold: the appended tokens are kept on the host, in fp64, by their
original position, and the cache is compared with them, not read back as truth.

A decode over the rows that should be held, in fp64, differs from the kernels' by
the cache's encoding: a score moves by at most scale x sum |q_d| e_d, e the bound of a
stored row's error (as for the append), a weight by that, relatively, twice (its own
score and the others' in the log-sum-exp), and likewise an output, times the largest
|value|, besides its own rounding."""
import numpy as np
import pytest
import torch

from oracle import around_ref as ar
from oracle import sparse_mla_ref as ref

from test_gpu_append import check_rows, make_cache

pytestmark = pytest.mark.gpu


def api():
    from sparse_mla_decode_05_b200 import api as a
    return a


@pytest.fixture(autouse=True)
def _no_device_errors():
    yield
    torch.cuda.synchronize()
    assert api().device_error() == 0


@pytest.mark.parametrize("new_pages", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "dsv4"])
def test_the_cache_holds_the_kept_tokens(kind, new_pages):
    a = api()
    rng = np.random.default_rng(71)
    B, prompt, budget, max_ctx = 3, 170, 100, 256
    d = 512 if kind == "dsv4" else 576
    pps = max_ctx // 64
    perm = rng.permutation(2 * B * pps)
    tables = [torch.from_numpy(t.reshape(B, pps).astype(np.int32)).cuda() for t in (perm[:B * pps], perm[B * pps:])]
    pt = tables[0]
    kv, rs = make_cache(kind, 2 * B * pps * 64, fill=0x11)
    table, scale = a.RopeTable(64), 1 / np.sqrt(d)
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(512)).astype(np.float32)).cuda()
    i32 = lambda v: torch.as_tensor(np.asarray(v), dtype=torch.int32, device="cuda")  # noqa: E731
    rows = [{} for _ in range(B)]                       # by original position: the row to be held, fp64
    held = [[] for _ in range(B)]                       # original positions in cache order
    acc = torch.zeros(B, max_ctx, device="cuda")
    expect = [np.zeros(0) for _ in range(B)]            # accumulated weights in cache order
    slack = [np.zeros(0) for _ in range(B)]

    def append(count):
        x = torch.from_numpy(rng.standard_normal((B * count, d)).astype(np.float32)).cuda().to(torch.bfloat16)
        slots = np.concatenate([len(held[b]) + np.arange(count) for b in range(B)])
        # (a position of its own per sequence, so that rows of two sequences never agree by chance)
        positions = np.concatenate([1000 * b + len(rows[b]) + np.arange(count) for b in range(B)])
        a.cache_append(x, kv, i32(slots), kv_row_scale=rs, page_table=pt, page_size=64, norm_weight=w, rope=table,
                       positions=i32(positions))
        want = ar.append_rows(x.double().cpu().numpy(), norm_weight=w.double().cpu().numpy(), freq=ar.rope_frequencies(64),
                              positions=positions)
        for i, p in enumerate(positions):
            b = i // count
            rows[b][int(p)] = want[i]
            held[b].append(int(p))
        for b in range(B):
            expect[b] = np.concatenate([expect[b], np.zeros(count)])
            slack[b] = np.concatenate([slack[b], np.zeros(count)])

    def check_cache():
        for b in range(B):
            at = np.arange(len(held[b]))
            phys = pt[b].cpu().numpy()[at // 64].astype(np.int64) * 64 + at % 64
            check_rows(kind, kv, rs, phys, np.stack([rows[b][p] for p in held[b]]))

    def step():
        q = torch.from_numpy(rng.standard_normal((B, 64, d)).astype(np.float32)).cuda().to(torch.bfloat16)
        idx = np.full((B, max_ctx), -1, np.int32)
        for b in range(B):
            idx[b, :len(held[b])] = rng.permutation(len(held[b]))
        paged = dict(kv_row_scale=rs, page_table=pt, page_size=64)
        out, lse = a.decode(q, kv, i32(idx), scale, **paged)
        weights = a.attention_weights(q, kv, i32(idx), lse, scale, **paged)
        a.accumulate_weights(acc, i32(idx), weights)
        got = acc.double().cpu().numpy()
        for b in range(B):
            k = np.stack([rows[b][p] for p in held[b]])
            qd = q[b].double().cpu().numpy()
            want, wl = ref.attend_rows(qd, k, scale, 512)
            half = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4, "dsv4": 2.0 ** -4}[kind]
            e = half * 1.01 * np.abs(k) + 2.0 ** -9 * np.abs(k).max(1, keepdims=True) / 448      # (or half a subnormal step)
            move = 2 * scale * (np.abs(qd) @ e.T).max(1)                                        # per head
            p = np.exp(scale * (qd @ k.T) - wl[:, None])
            grown = np.exp(move)[:, None] - 1 + 2e-3
            expect[b] += p.sum(0)
            slack[b] += (p * grown).sum(0)
            assert np.all(np.abs(got[b, :len(held[b])] - expect[b]) <= slack[b])
            assert np.all(got[b, len(held[b]):] == 0)
            v = np.abs(k[:, :512]).max()
            tol = (grown[:, 0] * v + half * v + 2e-2)[:, None]
            assert np.all(np.abs(out[b].double().cpu().numpy() - want) <= tol)
            # the accumulated weights as they are, from here on
            expect[b], slack[b] = got[b, :len(held[b])].copy(), np.zeros(len(held[b]))

    append(prompt)
    check_cache()
    for _ in range(3):
        step()
        append(1)
    check_cache()
    ctx = i32([len(h) for h in held])
    kept, new_len, acc = a.evict(acc, ctx, budget, page_table=pt, kv=kv, kv_row_scale=rs, sinks=3, recent=9,
                                 new_page_table=tables[1] if new_pages else None)
    for b in range(B):
        sel = ar.evict_select(np.asarray(expect[b], np.float32), len(held[b]), budget, 3, 9)
        assert kept[b].tolist() == sel and int(new_len[b]) == budget
        held[b] = [held[b][i] for i in sel]
        expect[b], slack[b] = expect[b][sel], np.zeros(budget)
    if new_pages:
        pt = tables[1]
    check_cache()
    for _ in range(3):
        append(1)
        step()
    check_cache()
