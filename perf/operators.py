"""Cases for the operators around the sparse-MLA decode step.

Five operators of the serving loop that surrounds the decode: rotary positions (rope), writing new tokens
into the cache (append: norm, rotation, encoding, paged store), the attention weight each listed cache row
received (weights), its accumulation per cache position (accumulate), and the eviction of the positions that
received least, with the compaction of the paged caches (evict).

``run`` computes them in elementary torch operations, or, with ``own``, through the library's entry points.
"""
import math

import torch

own = False

H, D_QK, D_V = 64, 576, 512
PAGE = 64
DSV4_PAGE_BYTES, DSV4_NOPE = 37376, 448
KV_BF16, KV_FP8, KV_DSV4 = "bf16", "fp8", "dsv4"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 16 sequences: the rotary part of the query projection goes into the decode's query
        dict(name="rope_decode", op="rope", n=16, heads=H, x_width=192, x_off=128, y_width=D_QK, y_off=512, dim=64,
             rot=64, rot_off=0, layout="interleaved", scaling="yarn", dtype="bf16", transpose=False, in_place=False,
             max_pos=131072),
        # a long prompt's gradient through the rotation (half layout), the rest of the head passed on
        dict(name="rope_prompt_grad", op="rope", n=16384, heads=H, x_width=128, x_off=0, y_width=128, y_off=0,
             dim=128, rot=64, rot_off=0, layout="half", scaling="none", dtype="bf16", transpose=True, in_place=False,
             max_pos=16384),
        # the new token of each of 64 sequences into a flat bf16 pool
        dict(name="append_decode_bf16", op="append", kind=KV_BF16, n=64, B=64, ctx=4096, paged=False, ragged=False,
             norm=True, rope=True, dtype="bf16"),
        # a chunk of prompt tokens of eight sequences into paged fp8 rows
        dict(name="append_prompt_fp8", op="append", kind=KV_FP8, n=65536, B=8, ctx=8192, paged=True, ragged=False,
             norm=True, rope=True, dtype="bf16"),
        # prompts of uneven length into DeepSeek-V4 pages
        dict(name="append_ragged_dsv4", op="append", kind=KV_DSV4, n=10007, B=13, ctx=2048, paged=True, ragged=True,
             norm=True, rope=True, dtype="bf16"),
        # one sequence, top-2048 of a 65,536-row cache, peaky softmax
        dict(name="weights_one_seq", op="weights", kind=KV_BF16, B=1, T=1, k=2048, ctx=65536, paged=False, pad=0,
             q_mult=4.0),
        # the full serving batch over paged fp8 rows
        dict(name="weights_batch_fp8", op="weights", kind=KV_FP8, B=128, T=1, k=2048, ctx=8192, paged=True, pad=0,
             q_mult=1.0),
        # two query tokens per sequence over DeepSeek-V4 pages, lists padded to an odd length
        dict(name="weights_tokens_dsv4", op="weights", kind=KV_DSV4, B=32, T=2, k=509, ctx=8192, paged=True, pad=61,
             q_mult=1.0),
        # the weights of one decode step of 16 sequences, summed onto their positions
        dict(name="accumulate_step", op="accumulate", B=16, T=1, k=512, max_ctx=8192, pad=37, decay=1.0),
        # two query tokens of 64 sequences with overlapping lists, older steps fading
        dict(name="accumulate_tokens", op="accumulate", B=64, T=2, k=2048, max_ctx=8192, pad=0, decay=0.98),
        # 32 sequences at their context limit halve their fp8 cache and indexer keys in place
        dict(name="evict_in_place_fp8", op="evict", kind=KV_FP8, B=32, max_ctx=8192, ragged=False, budget=4096,
             sinks=4, recent=512, keys=True, in_place=True),
        # one long bf16 sequence condensed into pages of its own, the source kept for another reader
        dict(name="evict_long_new_pages", op="evict", kind=KV_BF16, B=1, max_ctx=65536, ragged=False, budget=8192,
             sinks=64, recent=1024, keys=False, in_place=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "weights", "accumulate", "evict"])
    if op == "rope":
        n, heads = _log(rng, 1, 12000), rng.choice([1, 7, 16, 64, 64])
        layout, dtype = rng.choice(["interleaved", "half"]), rng.choice(["bf16", "bf16", "fp16", "fp32"])
        common = dict(op=op, n=n, heads=heads, layout=layout, scaling=rng.choice(["none", "linear", "yarn"]), dtype=dtype,
                      transpose=rng.random() < 0.4, max_pos=_log(rng, 64, 1 << 20))
        form = rng.choice(["query", "output", "indexer", "odd"])
        if form == "query":        # the rotary part of a projection into the decode's query
            return dict(common, x_width=192, x_off=128, y_width=D_QK, y_off=512, dim=64, rot=64, rot_off=0, in_place=False)
        if form == "output":       # the rotary part of a DeepSeek-V4 output, in place
            return dict(common, x_width=512, x_off=0, y_width=512, y_off=0, dim=512, rot=64, rot_off=448, in_place=True)
        if form == "indexer":      # the indexer's query
            return dict(common, x_width=128, x_off=0, y_width=128, y_off=0, dim=128, rot=64, rot_off=0, in_place=False)
        rot = 2 * rng.randint(1, 48)
        dim = rot + rng.randint(0, 30)
        off = rng.randint(0, dim - rot)
        return dict(common, x_width=dim + rng.randint(0, 9), x_off=0, y_width=dim + rng.randint(0, 9), y_off=0, dim=dim,
                    rot=rot, rot_off=off, in_place=False)
    if op == "append":
        kind = rng.choice([KV_BF16, KV_FP8, KV_FP8, KV_DSV4])
        B = _log(rng, 1, 128)
        n = B if rng.random() < 0.4 else max(B, _log(rng, 1, 60000))
        ragged = n > B and rng.random() < 0.7
        per = -(-n // B) if not ragged else -(-4 * n // B)
        if not ragged:
            n = B * per
        return dict(op=op, kind=kind, n=n, B=B, ctx=max(64, -(-per // 64) * 64 + 64 * rng.randint(0, 20)),
                    paged=kind == KV_DSV4 or rng.random() < 0.7, ragged=ragged, norm=rng.random() < 0.8,
                    rope=rng.random() < 0.8, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "weights":
        kind = rng.choice([KV_BF16, KV_FP8, KV_FP8, KV_DSV4])
        B, T = _log(rng, 1, 100), rng.choice([1, 1, 2, 3])
        k = _log(rng, 1, max(2, min(2300, 240000 // (B * T))))
        ctx = max(256, min(8192, 64 * _log(rng, 4, 128)))
        k = min(k, ctx)
        return dict(op=op, kind=kind, B=B, T=T, k=k, ctx=ctx, paged=kind == KV_DSV4 or rng.random() < 0.6,
                    pad=rng.choice([0, k // 5, k // 2]), q_mult=rng.choice([1.0, 1.0, 3.0]))
    if op == "accumulate":
        B, T = _log(rng, 1, 128), rng.choice([1, 1, 2, 4])
        max_ctx = _log(rng, 200, 60000 if B < 20 else 9000)
        k = min(max_ctx, _log(rng, 1, 2300))
        return dict(op=op, B=B, T=T, k=k, max_ctx=max_ctx, pad=rng.choice([0, k // 4]), decay=rng.choice([1.0, 1.0, 0.95]))
    kind = rng.choice([KV_BF16, KV_FP8, KV_DSV4])
    B = _log(rng, 1, 32)
    max_ctx = _log(rng, 100, 150000 // B)
    budget = max(1, int(max_ctx * rng.uniform(0.2, 0.8)))
    return dict(op="evict", kind=kind, B=B, max_ctx=max_ctx, ragged=rng.random() < 0.5, budget=budget,
                sinks=min(budget // 4, rng.choice([0, 4, 64])), recent=min(budget // 3, rng.choice([0, 1, 128, 1000])),
                keys=rng.random() < 0.5, in_place=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Radians per position of each rotated pair, and what multiplies cos and sin."""
    d = case["rot"]
    base = 10000.0
    freq = [base ** (-2.0 * i / d) for i in range(d // 2)]
    if case["scaling"] == "linear":
        return [f / 8.0 for f in freq], 1.0
    if case["scaling"] == "yarn":
        turns = lambda r: d * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), d - 1)
        ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(d // 2)]
        return [f * (1 - r) + f / 40.0 * r for f, r in zip(freq, ramp)], 0.1 * math.log(40.0) + 1.0
    return freq, 1.0


def _rope_arguments(case):
    scaling = {"none": {}, "linear": dict(scaling="linear", factor=8.0),
               "yarn": dict(scaling="yarn", factor=40.0, original_ctx=4096, mscale=0.1 * math.log(40.0) + 1.0)}
    return dict(rope_dim=case["rot"], interleaved=case["layout"] == "interleaved", **scaling[case["scaling"]])


def _pages(B, per_seq, g, spare=0):
    """A page table [B, per_seq] of distinct pages in random order, and `spare` more pages per sequence."""
    perm = torch.randperm(B * (per_seq + spare), generator=g, device=DEV).to(torch.int32)
    return perm[:B * per_seq].view(B, per_seq), perm[B * per_seq:].view(B, spare)


def _pool(kind, rows, g):
    """A cache of N(0, 1) rows in the given layout: (kv, kv_row_scale)."""
    if kind == KV_BF16:
        return torch.randn(rows, D_QK, generator=g, device=DEV, dtype=torch.bfloat16), None
    if kind == KV_FP8:
        x = torch.randn(rows, D_QK, generator=g, device=DEV)
        scale = x.abs().amax(1) / 448
        return x.div_(scale[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale
    pages = torch.zeros(rows // PAGE, DSV4_PAGE_BYTES, dtype=torch.uint8, device=DEV)
    x = torch.randn(rows, D_V, generator=g, device=DEV)
    nope = x[:, :DSV4_NOPE].reshape(rows, 7, 64)
    e = _ue8m0(nope.abs().amax(2))
    codes = (nope / torch.exp2(e.float())[..., None]).to(torch.float8_e4m3fn).view(rows, DSV4_NOPE)
    slots, scales = _dsv4_views(pages)
    slots[..., :DSV4_NOPE] = codes.view(torch.uint8).view(-1, PAGE, DSV4_NOPE)
    slots[..., DSV4_NOPE:] = x[:, DSV4_NOPE:].to(torch.bfloat16).view(torch.uint8).view(-1, PAGE, 128)
    scales[..., :7] = (e + 127).to(torch.uint8).view(-1, PAGE, 7)
    return pages, None


def _ue8m0(amax):
    """The smallest e with amax <= 448 * 2^e (whole number), at least -126; -126 for a group of zeros."""
    m, k = torch.frexp(amax)                       # amax = m 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    return torch.where(amax > 0, k - 9 + (m > 0.875).to(k.dtype), torch.full_like(k, -126)).clamp(-126, 127)


def _dsv4_views(pages):
    """(slots [P, 64, 576], scale blocks [P, 64, 8]) of DeepSeek-V4 pages."""
    P = pages.shape[0]
    return (pages[:, :PAGE * 576].unflatten(1, (PAGE, 576)), pages[:, PAGE * 576:].unflatten(1, (PAGE, 8))) if P else None


def _lists(rows, R, k, pad, g):
    """[rows, k] lists of distinct positions in [0, R), `pad` random entries of each -1."""
    idx = torch.rand(rows, R, generator=g, device=DEV).argsort(1)[:, :k]
    if pad:
        idx.scatter_(1, torch.rand(rows, k, generator=g, device=DEV).argsort(1)[:, :pad], -1)
    return idx.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = globals()["_prepare_" + case["op"]](case, g)
    s["case"] = case
    if own:
        from sparse_mla_decode_05_b200 import api
        s["plan"] = globals()["_plan_" + case["op"]](api, s)
    return s


def _prepare_rope(c, g):
    dt = DTYPES[c["dtype"]]
    x = torch.randn(c["n"], c["heads"], c["x_width"], generator=g, device=DEV).to(dt)
    y = x if c["in_place"] else torch.zeros(c["n"], c["heads"], c["y_width"], dtype=dt, device=DEV)
    positions = torch.randint(0, c["max_pos"], (c["n"],), generator=g, device=DEV, dtype=torch.int32)
    freq, mscale = _frequencies(c)
    return dict(x=x[..., c["x_off"]:c["x_off"] + c["dim"]], y=y[..., c["y_off"]:c["y_off"] + c["dim"]],
                positions=positions, freq=torch.tensor(freq, dtype=torch.float64, device=DEV), mscale=mscale)


def _prepare_append(c, g):
    B, n, per_seq = c["B"], c["n"], -(-c["ctx"] // PAGE)
    rows = B * per_seq * PAGE
    kind = c["kind"]
    d = D_V if kind == KV_DSV4 else D_QK
    s = dict(x=torch.randn(n, d, generator=g, device=DEV).to(DTYPES[c["dtype"]]), seq=None, page_table=None, rope=None,
             norm_weight=1 + 0.1 * torch.randn(D_V, generator=g, device=DEV) if c["norm"] else None)
    if c["ragged"]:
        # tokens of one sequence stand together; the lengths of the sequences are uneven
        cut = torch.rand(B, generator=g, device=DEV) + 0.5
        seq = torch.bucketize((torch.arange(n, device=DEV) + 0.5) / n, (cut / cut.sum()).cumsum(0)).clamp_(max=B - 1)
        first = torch.searchsorted(seq, torch.arange(B, device=DEV))
        s["seq"], slot = seq.to(torch.int32), torch.arange(n, device=DEV) - first[seq]
    else:
        seq = torch.arange(n, device=DEV) // (n // B)
        slot = torch.arange(n, device=DEV) % (n // B)
    start = torch.randint(0, max(1, c["ctx"] - int(slot.max())), (B,), generator=g, device=DEV)
    slot = slot + start[seq]
    s["positions"] = (slot + 1000).to(torch.int32)
    if c["paged"]:
        s["page_table"], _ = _pages(B, per_seq, g)
        s["slots"] = slot.to(torch.int32)
    else:
        s["slots"] = (seq * per_seq * PAGE + slot).to(torch.int32)
    if kind == KV_BF16:
        s["kv"], s["kv_row_scale"] = torch.zeros(rows, D_QK, dtype=torch.bfloat16, device=DEV), None
    elif kind == KV_FP8:
        s["kv"] = torch.zeros(rows, D_QK, dtype=torch.uint8, device=DEV)
        s["kv_row_scale"] = torch.ones(rows, device=DEV)
    else:
        s["kv"], s["kv_row_scale"] = torch.zeros(rows // PAGE, DSV4_PAGE_BYTES, dtype=torch.uint8, device=DEV), None
    if c["rope"]:
        s["rope"] = dict(rot=64, layout="interleaved", scaling="none")
        freq, s["mscale"] = _frequencies(s["rope"])
        s["freq"] = torch.tensor(freq, dtype=torch.float64, device=DEV)
    return s


def _prepare_weights(c, g):
    B, T, per_seq = c["B"], c["T"], -(-c["ctx"] // PAGE)
    d = D_V if c["kind"] == KV_DSV4 else D_QK
    q = (c["q_mult"] * torch.randn(B, T, H, d, generator=g, device=DEV)).to(torch.bfloat16)
    kv, kv_row_scale = _pool(c["kind"], B * per_seq * PAGE, g)
    idx = _lists(B * T, c["ctx"], c["k"], c["pad"], g).view(B, T, c["k"])
    page_table = None
    if c["paged"]:
        page_table, _ = _pages(B, per_seq, g)
    else:
        idx = torch.where(idx >= 0, idx + (torch.arange(B, device=DEV, dtype=torch.int32) * per_seq * PAGE)[:, None, None], idx)
    s = dict(q=q, kv=kv, kv_row_scale=kv_row_scale, page_table=page_table, indices=idx, scale=1 / math.sqrt(d))
    # the decode that ran before this left its log-sum-exp
    scores = _scores(c["kind"], s).masked_fill(idx[:, :, None] < 0, -math.inf)
    s["lse"] = torch.logsumexp(scores, -1)
    if T == 1:
        s.update(q=q[:, 0], indices=idx[:, 0].contiguous(), lse=s["lse"][:, 0].contiguous())
    s["q"] = s["q"].contiguous()
    return s


def _prepare_accumulate(c, g):
    B, T, k = c["B"], c["T"], c["k"]
    idx = _lists(B, c["max_ctx"], k, c["pad"], g)[:, None]
    if T > 1:                       # the later tokens keep about three quarters of the first one's list
        more = _lists(B * (T - 1), c["max_ctx"], k, c["pad"], g).view(B, T - 1, k)
        keep = torch.rand(B, T - 1, k, generator=g, device=DEV) < 0.75
        idx = torch.cat([idx, torch.where(keep, idx.expand(B, T - 1, k), more)], 1)
    w = torch.softmax(torch.randn(B, T, k, generator=g, device=DEV), -1) * H
    w = torch.where(idx >= 0, w, torch.zeros_like(w))
    acc = torch.rand(B, c["max_ctx"], generator=g, device=DEV)
    if T == 1:
        idx, w = idx[:, 0], w[:, 0]
    return dict(indices=idx.contiguous(), weights=w.contiguous(), acc=acc)


def _prepare_evict(c, g):
    B, per_seq, spare = c["B"], -(-c["max_ctx"] // PAGE), 0 if c["in_place"] else -(-c["budget"] // PAGE)
    rows = B * (per_seq + spare) * PAGE
    page_table, new_page_table = _pages(B, per_seq, g, spare)
    kv, kv_row_scale = _pool(c["kind"], rows, g)
    k_cache = torch.randn(rows, 128, generator=g, device=DEV, dtype=torch.bfloat16) if c["keys"] else None
    ctx = torch.full((B,), c["max_ctx"], dtype=torch.int32, device=DEV)
    if c["ragged"]:
        ctx = torch.randint(0, c["max_ctx"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    # accumulated weights fall off steeply; many positions never got any
    acc = torch.exp(3 * torch.randn(B, c["max_ctx"], generator=g, device=DEV) - 4)
    acc = torch.where(torch.rand(B, c["max_ctx"], generator=g, device=DEV) < 0.3, torch.zeros_like(acc), acc)
    acc = torch.where(torch.arange(c["max_ctx"], device=DEV) < ctx[:, None], acc, torch.zeros_like(acc))
    return dict(acc=acc, ctx_len=ctx, page_table=page_table, new_page_table=page_table if c["in_place"] else new_page_table,
                kv=kv, kv_row_scale=kv_row_scale, k_cache=k_cache, acc_out=torch.zeros_like(acc))


# ------------------------------------------------------------------ through the library
def _plan_rope(api, s):
    c = s["case"]
    return api.RopePlan(s["x"], s["positions"], api.RopeTable(**_rope_arguments(c)), offset=c["rot_off"],
                        transpose=c["transpose"], out=s["y"])


def _plan_append(api, s):
    rope = api.RopeTable(**_rope_arguments(s["rope"])) if s["rope"] else None
    return api.CacheAppendPlan(s["x"], s["kv"], s["slots"], kv_row_scale=s["kv_row_scale"], page_table=s["page_table"],
                               page_size=0 if s["page_table"] is None else PAGE,
                               seq=None if s["page_table"] is None else s["seq"],
                               norm_weight=s["norm_weight"], eps=1e-6, rope=rope,
                               positions=s["positions"] if rope else None)


def _plan_weights(api, s):
    return api.AttentionWeightsPlan(s["q"], s["kv"], s["indices"], s["lse"], s["scale"], kv_row_scale=s["kv_row_scale"],
                                    page_table=s["page_table"], page_size=0 if s["page_table"] is None else PAGE)


def _plan_accumulate(api, s):
    return api.AccumulateWeightsPlan(s["acc"], s["indices"], s["weights"], decay=s["case"]["decay"])


def _plan_evict(api, s):
    c = s["case"]
    return api.EvictPlan(s["acc"], s["ctx_len"], c["budget"], page_table=s["page_table"], kv=s["kv"],
                         kv_row_scale=s["kv_row_scale"], k_cache=s["k_cache"], sinks=c["sinks"], recent=c["recent"],
                         new_page_table=None if c["in_place"] else s["new_page_table"], acc_out=s["acc_out"])


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        s["plan"].run()
        if op == "rope":
            return s["plan"].out
        if op == "weights":
            return s["plan"].out
        if op == "accumulate":
            return s["acc"]
        if op == "evict":
            return dict(kept=s["plan"].kept, new_len=s["plan"].new_len, acc=s["acc_out"], **_cache_values(s))
        return _cache_values(s)
    return globals()["_plain_" + op](s)


def _cache_values(s):
    """The caches as the values that they hold (views of the state's buffers)."""
    kv = s["kv"]
    out = {}
    if kv.dtype == torch.bfloat16:
        out["kv"] = kv
    elif kv.shape[1] == DSV4_PAGE_BYTES:
        slots, scales = _dsv4_views(kv)
        out.update(codes=slots[..., :DSV4_NOPE].view(torch.float8_e4m3fn), rope=slots[..., DSV4_NOPE:].view(torch.bfloat16),
                   scales=scales.view(torch.float8_e8m0fnu))
    else:
        out.update(codes=kv.view(torch.float8_e4m3fn), row_scale=s["kv_row_scale"])
    if s.get("k_cache") is not None:
        out["keys"] = s["k_cache"]
    return out


def _rotate(x, positions, freq, mscale, layout, sign):
    """x [..., rot] fp32 turned by positions [...] (broadcast over x's other leading dims by the caller)."""
    angle = positions.double()[..., None] * freq       # radians, in 64 bits: far positions turn thousands of times
    c, s = (mscale * torch.cos(angle)).float(), (sign * mscale * torch.sin(angle)).float()
    if layout == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _plain_rope(s):
    c = s["case"]
    lo, hi = c["rot_off"], c["rot_off"] + c["rot"]
    r = _rotate(s["x"][..., lo:hi].float(), s["positions"][:, None], s["freq"], s["mscale"], c["layout"],
                -1.0 if c["transpose"] else 1.0)
    if not c["in_place"]:
        s["y"].copy_(s["x"])
    s["y"][..., lo:hi] = r.to(s["y"].dtype)
    return s["y"]


def _physical(slots, seq, page_table):
    slots = slots.long()
    if page_table is None:
        return slots
    return page_table[seq.long(), slots // PAGE].long() * PAGE + slots % PAGE


def _plain_append(s):
    c = s["case"]
    x = s["x"].float()
    if s["norm_weight"] is not None:
        latent = x[:, :D_V]
        latent = latent * torch.rsqrt(latent.square().mean(1, keepdim=True) + 1e-6) * s["norm_weight"]
        x = torch.cat([latent, x[:, D_V:]], 1)
    if s["rope"]:
        x = torch.cat([x[:, :-64], _rotate(x[:, -64:], s["positions"], s["freq"], s["mscale"], "interleaved", 1.0)], 1)
    n = x.shape[0]
    seq = s["seq"] if s["seq"] is not None else torch.arange(n, device=x.device) // (n // c["B"])
    row = _physical(s["slots"], seq, s["page_table"])
    if c["kind"] == KV_BF16:
        s["kv"][row] = x.to(torch.bfloat16)
    elif c["kind"] == KV_FP8:
        amax = x.abs().amax(1)
        scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        s["kv"][row] = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["kv_row_scale"][row] = scale
    else:
        nope = x[:, :DSV4_NOPE].reshape(n, 7, 64)
        e = _ue8m0(nope.abs().amax(2))
        codes = (nope / torch.exp2(e.float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(n, DSV4_NOPE)
        slots, scales = _dsv4_views(s["kv"])
        page, at = row // PAGE, row % PAGE
        slots[page, at] = torch.cat([codes.view(torch.uint8), x[:, DSV4_NOPE:].to(torch.bfloat16).view(torch.uint8)], 1)
        scales[page, at] = torch.cat([(e + 127).to(torch.uint8), torch.zeros(n, 1, dtype=torch.uint8, device=x.device)], 1)
    return _cache_values(s)


def _rows(kind, kv, kv_row_scale, row):
    """The cache rows named by `row` (any shape), in fp32."""
    if kind == KV_BF16:
        return kv[row].float()
    if kind == KV_FP8:
        return kv[row].view(torch.float8_e4m3fn).float() * kv_row_scale[row][..., None]
    slots, scales = _dsv4_views(kv)
    slot, e = slots[row // PAGE, row % PAGE], scales[row // PAGE, row % PAGE][..., :7]
    nope = slot[..., :DSV4_NOPE].view(torch.float8_e4m3fn).float().unflatten(-1, (7, 64))
    nope = nope * torch.exp2(e.float() - 127)[..., None]
    return torch.cat([nope.flatten(-2), slot[..., DSV4_NOPE:].contiguous().view(torch.bfloat16).float()], -1)


def _scores(kind, s):
    """scale * q . k over the listed rows: [B, T, 64, k] fp32 (q [B, T, 64, d], indices [B, T, k])."""
    idx = s["indices"]
    B = idx.shape[0]
    seq = torch.arange(B, device=idx.device)[:, None, None].expand_as(idx)
    row = _physical(idx.clamp(min=0), seq, s["page_table"])
    keys = _rows(kind, s["kv"], s["kv_row_scale"], row)
    return s["scale"] * torch.matmul(s["q"].float(), keys.transpose(-1, -2))


def _plain_weights(s):
    c = s["case"]
    one = s["q"].dim() == 3
    t = dict(s, q=s["q"][:, None], indices=s["indices"][:, None]) if one else s
    lse = s["lse"][:, None] if one else s["lse"]
    p = torch.exp(_scores(c["kind"], t) - lse[..., None])
    w = torch.where(t["indices"] >= 0, p.sum(2), torch.zeros((), device=p.device))
    return w[:, 0] if one else w


def _plain_accumulate(s):
    idx, w, acc = s["indices"].flatten(1).long(), s["weights"].flatten(1), s["acc"]
    acc.mul_(s["case"]["decay"])
    acc.scatter_add_(1, idx.clamp(min=0), torch.where(idx >= 0, w, torch.zeros_like(w)))
    return acc


def _plain_evict(s):
    c = s["case"]
    acc, ctx, n = s["acc"], s["ctx_len"][:, None], s["acc"].shape[1]
    pos = torch.arange(n, device=acc.device)
    protected = (pos < c["sinks"]) | (pos >= ctx - c["recent"])
    key = torch.where(protected, torch.full_like(acc, math.inf), acc)
    key = torch.where(pos < ctx, key, torch.full_like(acc, -math.inf))
    order = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :c["budget"]]
    order = torch.where(order < ctx, order, n).sort(1).values
    kept = torch.where(order < n, order, -1)
    new_len = torch.minimum(s["ctx_len"], torch.full_like(s["ctx_len"], c["budget"]))
    at = torch.arange(c["budget"], device=acc.device)
    s["acc_out"].masked_fill_(pos < ctx, 0.0)
    s["acc_out"][:, :c["budget"]] = torch.where(kept >= 0, acc.gather(1, kept.clamp(min=0)), s["acc_out"][:, :c["budget"]])
    seq = torch.arange(c["B"], device=acc.device)[:, None]
    to = _physical(at.expand_as(kept), seq, s["new_page_table"])
    src = torch.where(kept >= 0, _physical(kept.clamp(min=0), seq, s["page_table"]), to)   # rows past the end stay
    if c["kind"] == KV_DSV4:
        for part in _dsv4_views(s["kv"]):
            part[to // PAGE, to % PAGE] = part[src // PAGE, src % PAGE]
    else:
        s["kv"][to] = s["kv"][src]
    for pool in (s["kv_row_scale"], s["k_cache"]):
        if pool is not None:
            pool[to] = pool[src]
    return dict(kept=kept.to(torch.int32), new_len=new_len, acc=s["acc_out"], **_cache_values(s))


# ------------------------------------------------------------------ what a pass cannot do without
def _row_bytes(kind):
    return {KV_BF16: 1152, KV_FP8: 580, KV_DSV4: 583}[kind]


def work(c):
    if c["op"] == "rope":
        size = 4 if c["dtype"] == "fp32" else 2
        width = c["rot"] if c["in_place"] else c["dim"]
        return dict(bytes=2 * c["n"] * c["heads"] * width * size + 4 * c["n"], flops=3 * c["n"] * c["heads"] * c["rot"])
    if c["op"] == "append":
        d = D_V if c["kind"] == KV_DSV4 else D_QK
        size = 4 if c["dtype"] == "fp32" else 2
        return dict(bytes=c["n"] * (d * size + _row_bytes(c["kind"]) + 4 + (4 if c["rope"] else 0) + (4 if c["ragged"] else 0)),
                    flops=6 * c["n"] * d)
    if c["op"] == "weights":
        d = D_V if c["kind"] == KV_DSV4 else D_QK
        rows = c["B"] * c["T"]
        valid = rows * (c["k"] - c["pad"])
        distinct = min(valid, c["B"] * c["ctx"])
        return dict(bytes=distinct * _row_bytes(c["kind"]) + rows * (H * d * 2 + H * 4 + 8 * c["k"]), flops=valid * 2 * H * d)
    if c["op"] == "accumulate":
        touched = c["B"] * min(c["max_ctx"], c["T"] * (c["k"] - c["pad"]))
        if c["decay"] != 1.0:
            touched = c["B"] * c["max_ctx"]
        return dict(bytes=8 * c["B"] * c["T"] * c["k"] + 8 * touched, flops=c["B"] * c["T"] * c["k"] + touched)
    mean_ctx = c["max_ctx"] / 2 if c["ragged"] else c["max_ctx"]
    moved = c["B"] * min(c["budget"], mean_ctx)
    return dict(bytes=2 * moved * (_row_bytes(c["kind"]) + (256 if c["keys"] else 0)) + c["B"] * (4 * mean_ctx + 8 * c["budget"]),
                flops=c["B"] * mean_ctx)


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(c, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = globals()["_prepare_" + c["op"]](c, g)
    return globals()["_exact_" + c["op"]](c, s)


def _turn64(x, pos, freq, mscale, layout, sign):
    """Complex rotation in 64 bits: pair (a, b) -> mscale (a + i b) exp(i sign pos freq)."""
    z = x.double()
    half = z.shape[-1] // 2
    z = z.unflatten(-1, (half, 2)) if layout == "interleaved" else z.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_complex(z.contiguous()) * torch.polar(torch.full_like(freq * pos, mscale), sign * freq * pos)
    z = torch.view_as_real(z)
    return z.flatten(-2) if layout == "interleaved" else z.transpose(-1, -2).flatten(-2)


def _exact_rope(c, s):
    y = s["y"].double() if c["in_place"] else s["x"].double()
    part = slice(c["rot_off"], c["rot_off"] + c["rot"])
    y[..., part] = _turn64(s["x"][..., part], s["positions"].double()[:, None, None], s["freq"], s["mscale"], c["layout"],
                           -1 if c["transpose"] else 1)
    return y


def _nearest_e4m3(x):
    """The e4m3 value nearest to x (|x| <= 448), ties to even, in 64 bits: steps of 2^(e-3), e >= -6."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(c, s):
    x = s["x"].double()
    if s["norm_weight"] is not None:
        rms = (x[:, :D_V].pow(2).sum(1) / D_V + 1e-6).sqrt()
        x[:, :D_V] = x[:, :D_V] / rms[:, None] * s["norm_weight"].double()
    if s["rope"]:
        x[:, -64:] = _turn64(x[:, -64:], s["positions"].double()[:, None], s["freq"], s["mscale"], "interleaved", 1)
    slot = s["slots"].long()
    if s["page_table"] is not None:
        seq = s["seq"].long() if s["seq"] is not None else torch.arange(c["n"], device=DEV).div(c["n"] // c["B"], rounding_mode="floor")
        slot = s["page_table"].long()[seq].gather(1, (slot >> 6)[:, None])[:, 0] * 64 + (slot & 63)
    if c["kind"] == KV_BF16:
        kv = s["kv"].double()
        return dict(kv=kv.index_copy(0, slot, x))
    if c["kind"] == KV_FP8:
        scale = x.abs().max(1).values / 448
        scale[scale == 0] = 1
        codes = torch.zeros(s["kv"].shape, dtype=torch.float64, device=DEV)
        return dict(codes=codes.index_copy(0, slot, _nearest_e4m3(x / scale[:, None])),
                    row_scale=s["kv_row_scale"].double().index_copy(0, slot, scale))
    rows = s["kv"].shape[0] * 64
    group = x[:, :448].reshape(-1, 7, 64)
    scale = torch.exp2(torch.ceil(torch.log2(group.abs().amax(2).clamp(min=448 * 2.0 ** -126) / 448)))
    codes = torch.zeros(rows, 448, dtype=torch.float64, device=DEV).index_copy(0, slot, _nearest_e4m3(group / scale[..., None]).flatten(1))
    rope = torch.zeros(rows, 64, dtype=torch.float64, device=DEV).index_copy(0, slot, x[:, 448:])
    block = torch.full((rows, 8), 2.0 ** -127, dtype=torch.float64, device=DEV)
    block[slot, :7] = scale
    return dict(codes=codes.view(-1, 64, 448), rope=rope.view(-1, 64, 64), scales=block.view(-1, 64, 8))


def _exact_weights(c, s):
    B, T, k = c["B"], c["T"], c["k"]
    idx = s["indices"].view(B, T * k).long()
    q, lse = s["q"].double().view(B, T, H, -1), s["lse"].double().view(B, T, H)
    out = torch.zeros(B, T, k, dtype=torch.float64, device=DEV)
    for b in range(B):
        at = idx[b].clamp(min=0)
        if s["page_table"] is not None:
            at = s["page_table"][b].long()[at >> 6] * 64 + (at & 63)
        if c["kind"] == KV_DSV4:
            page, i = at >> 6, at & 63
            byte = s["kv"][page[:, None], (i * 576)[:, None] + torch.arange(576, device=DEV)]
            e = s["kv"][page[:, None], 36864 + (i * 8)[:, None] + torch.arange(7, device=DEV)]
            nope = byte[:, :448].contiguous().view(torch.float8_e4m3fn).double()
            rows = torch.cat([nope * torch.exp2(e.double() - 127).repeat_interleave(64, 1),
                              byte[:, 448:].contiguous().view(torch.bfloat16).double()], 1)
        elif c["kind"] == KV_FP8:
            rows = s["kv"][at].view(torch.float8_e4m3fn).double() * s["kv_row_scale"][at].double()[:, None]
        else:
            rows = s["kv"][at].double()
        rows = rows.view(T, k, -1)
        p = torch.exp(torch.einsum("thd,tkd->thk", q[b], rows) * s["scale"] - lse[b][:, :, None]).sum(1)
        out[b] = p * (idx[b].view(T, k) >= 0)
    return out[:, 0] if s["q"].dim() == 3 else out


def _exact_accumulate(c, s):
    acc = s["acc"].double() * c["decay"]
    idx, w = s["indices"].reshape(c["B"], -1).long(), s["weights"].reshape(c["B"], -1).double()
    for b in range(c["B"]):
        ok = idx[b] >= 0
        acc[b] += torch.bincount(idx[b][ok], w[b][ok], minlength=c["max_ctx"])
    return acc


def _exact_evict(c, s):
    kept = torch.full((c["B"], c["budget"]), -1, dtype=torch.int32, device=DEV)
    new_len = torch.zeros_like(s["ctx_len"])
    acc = s["acc_out"].double()
    wide = {k: v.double() for k, v in _cache_values(s).items()}
    for b in range(c["B"]):
        n = int(s["ctx_len"][b])
        take = list(range(n))
        if n > c["budget"]:
            w = s["acc"][b, :n].tolist()
            fixed = set(range(min(c["sinks"], n))) | set(range(max(0, n - c["recent"]), n))
            rest = sorted((i for i in range(n) if i not in fixed), key=lambda i: (-w[i], i))
            take = sorted(fixed | set(rest[:c["budget"] - len(fixed)]))
        m = new_len[b] = len(take)
        m = int(m)
        if not m:
            continue
        old = torch.tensor(take, device=DEV)
        kept[b, :m] = old
        acc[b, :n] = 0
        acc[b, :m] = s["acc"][b].double()[old]
        src = s["page_table"][b].long()[old >> 6] * 64 + (old & 63)
        i = torch.arange(m, device=DEV)
        dst = s["new_page_table"][b].long()[i >> 6] * 64 + (i & 63)
        for v in wide.values():
            flat = v.view(-1, v.shape[-1]) if v.dim() > 1 else v
            flat[dst] = flat[src]
    return dict(kept=kept, new_len=new_len, acc=acc, **wide)
