"""The token-by-token operators of the cache, measured: attention of new tokens over a paged key-value cache
(`attn_decode_paged`), inserts into it and evictions from it by accumulated attention weight (`kvcache_paged_insert`,
`kvcache_paged_evict`), and attention with a sliding window and first blocks that stay visible (`attn_fwd_window`).

`own` false: their plain forms in elementary torch operations, 32 bits, rounded once at the end.  `own` true: the
calls a user makes of the framework.
"""

import math

import torch

own = False

D = 128


def listed():
    return [
        # one stream's cache, a ring of 21 frames of 30 x 52 tokens read as pages of a frame, 12 heads: one new token
        dict(name="decode_ring_one", op="decode", n=1, hq=12, hkv=12, lq=1, page=1560, lo=32760, hi=32760, window=0,
             sinks=0, weight=False),
        # the smallest call: one token of one short stream, pages of 15 x 26 tokens, latency counts
        dict(name="decode_short", op="decode", n=1, hq=12, hkv=12, lq=1, page=390, lo=1951, hi=1951, window=0, sinks=0,
             weight=False),
        # a serving batch of ragged lengths, four query heads to a key head, small pages
        dict(name="decode_batch_ragged", op="decode", n=64, hq=32, hkv=8, lq=1, page=16, lo=1, hi=8192, window=0,
             sinks=0, weight=False),
        # four drafted tokens a stream, long streams of which a window and the first tokens are seen
        dict(name="decode_window_draft", op="decode", n=16, hq=32, hkv=4, lq=4, page=64, lo=16001, hi=32760,
             window=4096, sinks=64, weight=False),
        # the decode step of a bounded cache: attention that also adds up what weight each cached token got
        dict(name="decode_weight", op="decode", n=24, hq=24, hkv=8, lq=1, page=32, lo=2000, hi=4097, window=0, sinks=0,
             weight=True),
        # the eviction that follows it: every stream is one token over its budget
        dict(name="evict_step", op="evict", n=48, hkv=8, page=16, lo=4097, hi=4097, budget=4096, sinks=4, recent=256,
             mixed=True),
        # a long context cut down once: 21 frames to 5, the first frame and the last three kept
        dict(name="evict_compress", op="evict", n=2, hkv=12, page=1560, lo=32760, hi=32760, budget=7800, sinks=1560,
             recent=4680, mixed=False),
        # one new token for every stream of a batch
        dict(name="insert_step", op="insert", n=48, hkv=8, page=16, lo=1, hi=4097, new=1),
        # a window step's five frames of 1,560 tokens for two streams, into pages of a quarter frame
        dict(name="insert_frames", op="insert", n=2, hkv=12, page=390, lo=9360, hi=32760, new=7800),
        # prompt of a token stream: causal by token, window of 1,024 and 4 first tokens, four query heads to a key head
        dict(name="window_tokens", op="window", hq=16, hkv=4, lq=4097, lk=4097, gh=1, gw=1, block=1, window=1024, sinks=4,
             rope=False),
        # the rolling layer at 15 x 26: three frames seen and the first one, RoPE of Q and K in the kernel
        dict(name="window_mid", op="window", hq=12, hkv=12, lq=1950, lk=2730, gh=15, gw=26, block=1, window=3, sinks=1,
             rope=True),
        # the denoise pass at 30 x 52: blocks of 3 frames, four blocks seen and the first one
        dict(name="window_frames", op="window", hq=12, hkv=12, lq=23400, lk=32760, gh=30, gw=52, block=3, window=4,
             sinks=1, rope=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "evict", "insert", "window", "window"])
    if op == "window":
        if rng.random() < 0.5:      # token streams
            hkv, group = rng.choice([1, 2, 4, 12]), rng.choice([1, 2, 4, 7])
            lk = _log_int(rng, 60, 9000)
            lq = lk if rng.random() < 0.5 else _log_int(rng, 1, lk)
            return dict(op=op, hq=hkv * group, hkv=hkv, lq=lq, lk=lk, gh=1, gw=1, block=rng.choice([1, 1, 16]),
                        window=_log_int(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 130]), rope=False)
        gh, gw, frames = rng.randint(4, 30), rng.randint(6, 52), rng.randint(2, 21)
        hkv, group = rng.choice([1, 2, 6, 12]), rng.choice([1, 1, 2])
        lk = gh * gw * frames - rng.choice([0, 0, rng.randint(0, gh * gw - 1)])
        lk = min(lk, int(9.0e9 / (hkv * group * 23400)))
        return dict(op=op, hq=hkv * group, hkv=hkv, lq=rng.randint(1, min(lk, 23400)), lk=lk, gh=gh, gw=gw,
                    block=rng.randint(1, 3), window=rng.randint(1, 6), sinks=rng.randint(0, 2),
                    rope=rng.random() < 0.7)
    n = _log_int(rng, 1, 96)
    hkv = rng.choice([1, 2, 3, 4, 8, 12])
    page = rng.choice([1, 16, 24, 32, 64, 100, 390, 1560])
    top = max(40, min(32760, int(64 * 8 * 4096 / (n * hkv))))
    hi = _log_int(rng, 20, top)
    lo = hi if rng.random() < 0.3 else rng.randint(1, hi)
    if op == "decode":
        lq = rng.choice([1, 1, 1, 2, 5])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        window = 0 if rng.random() < 0.6 else _log_int(rng, 1, hi)
        return dict(op=op, n=n, hq=hkv * group, hkv=hkv, lq=lq, page=page, lo=lo, hi=hi, window=window,
                    sinks=rng.choice([0, 1, 4, 70]) if window else 0, weight=rng.random() < 0.4)
    if op == "evict":
        budget = max(4, int(hi * rng.choice([0.25, 0.5, 0.9, 1.0])) - rng.randint(0, 1))
        recent = rng.randint(0, budget // 2)
        return dict(op=op, n=n, hkv=hkv, page=page, lo=lo, hi=hi, budget=budget, sinks=rng.randint(0, min(8, budget - recent)),
                    recent=recent, mixed=rng.random() < 0.5)
    new = rng.choice([1, 1, 3, lo])
    return dict(op=op, n=n, hkv=hkv, page=page, lo=max(lo, new), hi=max(hi, lo, new), new=new)


# ---- sizes ---------------------------------------------------------------------------------------------------------


def _lens(case):
    """Lengths of the sequences: spread over [lo, hi], the longest one among them."""
    lo, hi, n = case["lo"], case["hi"], case["n"]
    got = [lo + int(math.modf((i + 1) * 0.6180339887498949)[0] * (hi - lo + 1)) for i in range(n)]
    got[n // 2] = hi
    return got


def _range(case, L, i):
    """Keys that query i of a sequence of L tokens sees: [0, a) and [b, c)."""
    c = L - case["lq"] + i + 1
    if c <= 0:
        return 0, 0, 0
    b = max(0, c - case["window"]) if case["window"] else 0
    return min(case["sinks"], b), b, c


def _offset(case):
    """Key frame of the first query frame of a window case: the queries are the last frames."""
    F = case["gh"] * case["gw"]
    return max(0, -(-case["lk"] // F) - -(-case["lq"] // F))


def _bounds(case):
    """Per query row of a window case: the first key of its window and the end of its keys."""
    F = case["gh"] * case["gw"]
    step, off = F * case["block"], _offset(case)
    qb = (off + torch.arange(case["lq"]) // F) // case["block"]
    return torch.clamp((qb - case["window"] + 1) * step, min=0), torch.clamp((qb + 1) * step, max=case["lk"]), step


def work(case):
    op, row = case["op"], 2 * D
    if op == "window":
        lo, end, step = _bounds(case)
        first = torch.minimum(torch.clamp(lo, max=case["sinks"] * step), end)
        seen = int((torch.clamp(end - lo, min=0) + first).sum())
        return {"bytes": row * (2 * case["lq"] * case["hq"] + 2 * case["lk"] * case["hkv"]),
                "flops": 4 * D * case["hq"] * seen}
    n, hkv = case["n"], case["hkv"]
    lens = _lens(case)
    if op == "decode":
        pairs = keys = 0
        for L in lens:
            r = [_range(case, L, i) for i in range(case["lq"])]
            pairs += sum(a + c - b for a, b, c in r)
            b0 = min((b for a, b, c in r if c > 0), default=0)
            keys += max((a for a, b, c in r), default=0) + max(0, r[-1][2] - b0)
        b = 2 * row * keys * hkv + 2 * row * n * case["lq"] * case["hq"] + 4 * n
        b += 8 * hkv * sum(lens) if case["weight"] else 0
        return {"bytes": b, "flops": 4 * D * case["hq"] * pairs}
    if op == "insert":
        return {"bytes": n * case["new"] * hkv * (4 * row + 8) + 8 * n, "flops": 0}
    b, B = 0, case["budget"]
    for L in lens:
        kept, moved = min(L, B), 0.0
        if L > B:
            guard = case["sinks"] + case["recent"]
            share = (B - guard) / max(1, L - guard)
            if case["mixed"]:
                moved = 1 + (L - B - 1) * B / L if case["recent"] else (L - B) * B / L
            else:
                tail = min(case["recent"], L - B)
                moved = tail + share * (L - B - tail)
        b += hkv * (8 * L + 8 * kept + 4 * row * int(moved))
    return {"bytes": b + 8 * n, "flops": 0}


# ---- inputs --------------------------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "window":
        s = dict(case=case, q=_normal(g, case["lq"], case["hq"], D), k=_normal(g, case["lk"], case["hkv"], D),
                 v=_normal(g, case["lk"], case["hkv"], D))
        s["o"] = torch.empty_like(s["q"])
        if own:
            from rolling_kv_cache_rope_b200 import rkv
            s["rope"] = rkv.make_rope(case["gh"], case["gw"])
            s["workspace"] = torch.empty(rkv.attn_fwd_varlen_workspace_size(1, case["hq"], D), dtype=torch.uint8,
                                         device="cuda")
        return s
    n, hkv, page = case["n"], case["hkv"], case["page"]
    lens = _lens(case)
    cols = -(-max(lens) // page)
    # a pool that holds every stream, its pages in no order
    table = torch.randperm(n * cols, generator=g, device="cuda").to(torch.int32).view(n, cols)
    s = dict(case=case, k=_normal(g, n * cols, page, hkv, D), v=_normal(g, n * cols, page, hkv, D), table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    cap = cols * page
    if case["op"] == "decode":
        s["q"] = _normal(g, n * case["lq"], case["hq"], D)
        s["o"] = torch.empty_like(s["q"])
        if case["weight"]:
            s["weight"] = torch.rand(n, hkv, cap, generator=g, device="cuda")
            s["weight_out"] = s["weight"].clone()
    elif case["op"] == "insert":
        s["k_new"] = _normal(g, n * case["new"], hkv, D)
        s["v_new"] = _normal(g, n * case["new"], hkv, D)
        s["next_pos"] = s["lens"] + 1000
        s["pos"] = torch.arange(cap, dtype=torch.int32, device="cuda").expand(n, hkv, cap).contiguous()
        s["weight"] = torch.rand(n, hkv, cap, generator=g, device="cuda")
    else:
        # accumulated weights: few tokens hold most of it, a tenth got none at all
        w = torch.exp(1.5 * torch.randn(n, hkv, cap, generator=g, device="cuda"))
        s["weight"] = w * (torch.rand(n, hkv, cap, generator=g, device="cuda") > 0.1)
        j = torch.arange(cap, device="cuda")
        L = s["lens"].long().view(n, 1, 1)
        pos = j.view(1, 1, cap).expand(n, hkv, cap)
        s["next_pos"] = s["lens"].clone()
        if case["mixed"]:
            # a cache that was evicted from before: the first tokens in place, the newest last, the others anywhere
            far = 2 * L
            old = torch.where(pos >= L - case["recent"], pos + far, 2 * pos)
            still = (pos < case["sinks"]) | (pos >= L - 1)
            place = torch.where(still, pos.double(), case["sinks"] + torch.rand(n, hkv, cap, generator=g, device="cuda").double() * 0.5)
            order = torch.argsort(place, dim=-1, stable=True)
            pos = torch.where(pos < case["sinks"], pos, old).gather(2, order)
            s["next_pos"] = (s["lens"] * 3).to(torch.int32)
        s["pos"] = pos.to(torch.int32).contiguous()
        s["weight_out"], s["pos_out"] = s["weight"].clone(), s["pos"].clone()
        s["lens_out"] = s["lens"].clone()
    if own:
        from rolling_kv_cache_rope_b200 import rkv
        s["cache"] = rkv.PagedKVCache(s["k"], s["v"], s["table"])
        size = 0
        if case["op"] == "decode":
            size = rkv.attn_decode_paged_workspace_size(s["cache"], case["hq"], case["lq"], case["weight"])
        elif case["op"] == "evict":
            size = rkv.kvcache_paged_evict_workspace_size(s["cache"], case["budget"])
        s["workspace"] = torch.empty(max(16, size), dtype=torch.uint8, device="cuda")
    return s


# ---- one pass ------------------------------------------------------------------------------------------------------


def run(state):
    return {"decode": _run_decode, "evict": _run_evict, "insert": _run_insert, "window": _run_window}[
        state["case"]["op"]](state)


def _run_decode(s):
    case = s["case"]
    if own:
        from rolling_kv_cache_rope_b200 import rkv
        o = rkv.attn_decode_paged(s["q"], s["cache"], s["lens"], o=s["o"], window=case["window"], sinks=case["sinks"],
                                  weight_in=s.get("weight"), weight_out=s.get("weight_out"), workspace=s["workspace"])
        return [o, s["weight_out"]] if case["weight"] else [o]
    n, hq, hkv, lq = case["n"], case["hq"], case["hkv"], case["lq"]
    K = s["k"][s["table"].long()].view(n, -1, hkv, D)
    V = s["v"][s["table"].long()].view(n, -1, hkv, D)
    cap = K.shape[1]
    j = torch.arange(cap, device="cuda")
    L = s["lens"].long().view(n, 1, 1)
    c = L - lq + torch.arange(lq, device="cuda").view(1, lq, 1)
    seen = j <= c
    if case["window"]:
        seen = seen & ((j > c - case["window"]) | (j < case["sinks"]))
    there = (j < L.view(n, 1))
    K = K.float().permute(0, 2, 3, 1)                                   # n hkv D cap
    V = (V.float() * there.view(n, cap, 1, 1)).permute(0, 2, 1, 3)      # n hkv cap D
    q = s["q"].float().view(n, lq, hkv, hq // hkv, D).permute(0, 2, 1, 3, 4).reshape(n, hkv, lq * (hq // hkv), D)
    p = torch.matmul(q, K).mul_(1.0 / math.sqrt(D)).view(n, hkv, lq, hq // hkv, cap)
    p.masked_fill_(~seen.view(n, 1, lq, 1, cap), -math.inf)
    top = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p.view(n, hkv, -1, cap), V).view(n, hkv, lq, hq // hkv, D)
    o = o.permute(0, 2, 1, 3, 4).reshape(n * lq, hq, D).to(torch.bfloat16)
    if not case["weight"]:
        return [o]
    got = s["weight"] + p.sum((2, 3))
    return [o, torch.where(there.view(n, 1, cap), got, s["weight"])]


def _rows(s, index):
    """Row of the flat page pool of each cache index [n, heads, m]."""
    n, page = s["case"]["n"], s["case"]["page"]
    at = s["table"].long().view(n, 1, -1).expand(n, index.shape[1], -1)
    return at.gather(2, index // page) * page + index % page


def _run_evict(s):
    case = s["case"]
    if own:
        from rolling_kv_cache_rope_b200 import rkv
        rkv.kvcache_paged_evict(s["cache"], s["lens"], s["weight"], s["pos"], s["next_pos"], case["budget"],
                                sinks=case["sinks"], recent=case["recent"], seq_lens_out=s["lens_out"],
                                weight_out=s["weight_out"], pos_out=s["pos_out"], workspace=s["workspace"])
        return [s["k"], s["v"], s["weight_out"], s["pos_out"], s["lens_out"]]
    n, hkv = case["n"], case["hkv"]
    cap = s["weight"].shape[2]
    B = min(case["budget"], cap)
    j = torch.arange(cap, device="cuda").expand(n, hkv, cap)
    L = s["lens"].long().view(n, 1, 1)
    there = j < L
    guard = (s["pos"] < case["sinks"]) | (s["pos"] >= s["next_pos"].view(n, 1, 1) - case["recent"])
    key = torch.where(there, torch.where(guard, torch.full_like(s["weight"], math.inf), s["weight"]),
                      torch.full_like(s["weight"], -math.inf))
    order = torch.sort(key, dim=2, descending=True, stable=True).indices
    kept = torch.zeros_like(there).scatter_(2, order[:, :, :B], True) & there
    hole, source = there & (j < B) & ~kept, kept & (j >= B)
    found = torch.zeros(n, hkv, cap + 1, dtype=torch.long, device="cuda")
    found.scatter_(2, torch.where(source, torch.cumsum(source, 2) - 1, torch.full_like(j, cap)), j)
    take = torch.where(hole, found.gather(2, torch.clamp(torch.cumsum(hole, 2) - 1, min=0)), j)[:, :, :B]
    to, frm = _rows(s, j[:, :, :B]), _rows(s, take)
    heads = torch.arange(hkv, device="cuda").view(1, hkv, 1)
    k, v = s["k"].view(-1, hkv, D), s["v"].view(-1, hkv, D)
    k[to, heads] = k[frm, heads]
    v[to, heads] = v[frm, heads]
    s["weight_out"][:, :, :B] = torch.where(there[:, :, :B], s["weight"].gather(2, take), s["weight_out"][:, :, :B])
    s["pos_out"][:, :, :B] = torch.where(there[:, :, :B], s["pos"].gather(2, take), s["pos_out"][:, :, :B])
    s["lens_out"].copy_(torch.clamp(s["lens"], max=case["budget"]))
    return [s["k"], s["v"], s["weight_out"], s["pos_out"], s["lens_out"]]


def _run_insert(s):
    case = s["case"]
    if own:
        from rolling_kv_cache_rope_b200 import rkv
        rkv.kvcache_paged_insert(s["cache"], s["k_new"], s["v_new"], s["lens"], next_pos=s["next_pos"], pos=s["pos"],
                                 weight=s["weight"])
        return [s["k"], s["v"], s["pos"], s["weight"]]
    n, hkv, new = case["n"], case["hkv"], case["new"]
    i = torch.arange(new, device="cuda").view(1, 1, new)
    at = (s["lens"].long().view(n, 1, 1) - new + i)
    to = _rows(s, at).view(-1)
    s["k"].view(-1, hkv, D)[to] = s["k_new"]
    s["v"].view(-1, hkv, D)[to] = s["v_new"]
    at = at.expand(n, hkv, new)
    s["pos"].scatter_(2, at, (s["next_pos"].view(n, 1, 1) - new + i).to(torch.int32).expand(n, hkv, new))
    s["weight"].scatter_(2, at, torch.zeros(n, hkv, new, device="cuda"))
    return [s["k"], s["v"], s["pos"], s["weight"]]


PAIRS = (22, 21, 21)    # rotary pairs of the t, h and w axes


def _rotate(x, case, t0):
    """Rotary embedding over (t, h, w) of rows [L, H, D] whose first frame is t0: angles in 64 bits."""
    F, gw = case["gh"] * case["gw"], case["gw"]
    i = torch.arange(x.shape[0], device="cuda")
    pos = torch.stack([t0 + i // F, (i % F) // gw, i % gw], 1).double()
    axis = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(PAIRS, device="cuda"), output_size=D // 2)
    k = torch.cat([torch.arange(m, device="cuda").double() / m for m in PAIRS])
    angle = pos[:, axis] * torch.pow(torch.full_like(k, 10000.0), -k)
    cos, sin = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _run_window(s):
    case = s["case"]
    off = _offset(case)
    if own:
        from rolling_kv_cache_rope_b200 import rkv
        seq = rkv.AttnSeq(s["q"], s["k"], s["v"], s["o"], q_t0=off, k_t0=0, rope_q=case["rope"], rope_k=case["rope"],
                          block_frames=case["block"], q_frame_offset=off)
        rkv.attn_fwd_window([seq], [(case["window"], case["sinks"])], s["rope"], workspace=s["workspace"])
        return [s["o"]]
    q, k = s["q"].float(), s["k"].float()
    if case["rope"]:
        q, k = _rotate(q, case, off), _rotate(k, case, 0)
    hq, hkv, lq, lk = case["hq"], case["hkv"], case["lq"], case["lk"]
    c = torch.arange(lk, device="cuda")
    lo, end, step = _bounds(case)
    lo, end = lo.cuda().unsqueeze(1), end.cuda().unsqueeze(1)
    hidden = (c >= end) | ((c < lo) & (c >= case["sinks"] * step))
    q = q.view(lq, hkv, hq // hkv, D).permute(1, 2, 0, 3)                              # hkv group lq D
    p = torch.matmul(q.reshape(hkv, -1, D), k.permute(1, 2, 0)).view(hkv, hq // hkv, lq, lk)
    p.mul_(1.0 / math.sqrt(D)).masked_fill_(hidden, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(hkv, -1, lk), s["v"].float().permute(1, 0, 2)).view(hkv, hq // hkv, lq, D)
    o.div_(torch.where(total == 0, torch.ones_like(total), total))
    return [o.permute(2, 0, 1, 3).reshape(lq, hq, D).to(torch.bfloat16)]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "evict": _exact_evict, "insert": _exact_insert, "window": _exact_window}[
        case["op"]](case, s)


def _softmax_rows(q, k, v, seen):
    """Rows of softmax(q k^T / sqrt(D)) over the seen keys, and their products with v; zeros where no key is seen."""
    z = (q @ k.T) / math.sqrt(D)
    z = torch.where(seen, z, torch.tensor(-math.inf, dtype=z.dtype, device=z.device))
    p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
    p = torch.where(seen, p, torch.zeros_like(p))
    return p, p @ v


def _exact_decode(case, s):
    group = case["hq"] // case["hkv"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    w = s["weight"].double() if case["weight"] else None
    for i, L in enumerate(_lens(case)):
        K = torch.cat([s["k"][t] for t in s["table"][i].tolist()])[:L].double()
        V = torch.cat([s["v"][t] for t in s["table"][i].tolist()])[:L].double()
        seen = torch.zeros(case["lq"], L, dtype=torch.bool, device="cuda")
        for r in range(case["lq"]):
            a, b, c = _range(case, L, r)
            seen[r, :a] = True
            seen[r, b:c] = True
        for h in range(case["hq"]):
            rows = slice(i * case["lq"], (i + 1) * case["lq"])
            p, got = _softmax_rows(s["q"][rows, h].double(), K[:, h // group], V[:, h // group], seen)
            o[rows, h] = got
            if w is not None:
                w[i, h // group, :L] += p.sum(0)
    return [o, w] if case["weight"] else [o]


def _exact_evict(case, s):
    page, B = case["page"], case["budget"]
    wo, po, lo = s["weight"].cpu(), s["pos"].cpu(), [min(L, B) for L in _lens(case)]
    weight, pos, nxt, table = wo.clone(), po.clone(), s["next_pos"].tolist(), s["table"].tolist()
    frm, to, heads = [], [], []
    for i, L in enumerate(_lens(case)):
        if L <= B:
            continue
        for g in range(case["hkv"]):
            ws, ps = weight[i, g, :L].tolist(), pos[i, g, :L].tolist()
            rank = sorted(range(L), key=lambda x: (not (ps[x] < case["sinks"] or ps[x] >= nxt[i] - case["recent"]),
                                                   0.0 if ps[x] < case["sinks"] or ps[x] >= nxt[i] - case["recent"] else -ws[x], x))
            kept = set(rank[:B])
            holes = [x for x in range(B) if x not in kept]
            moved = [x for x in range(B, L) if x in kept]
            for a, b in zip(moved, holes):
                wo[i, g, b], po[i, g, b] = weight[i, g, a], pos[i, g, a]
                frm.append(table[i][a // page] * page + a % page)
                to.append(table[i][b // page] * page + b % page)
                heads.append(g)
    out = []
    for t in (s["k"], s["v"]):
        flat = t.view(-1, case["hkv"], D).double()
        if frm:
            f, t_, h = (torch.tensor(x, device="cuda") for x in (frm, to, heads))
            flat[t_, h] = flat[f, h]
        out.append(flat.view(t.shape))
    return out + [wo.double(), po, torch.tensor(lo, dtype=torch.int32)]


def _exact_insert(case, s):
    k, v, pos, weight = s["k"].double(), s["v"].double(), s["pos"].clone(), s["weight"].double()
    table, page = s["table"].tolist(), case["page"]
    for i, L in enumerate(_lens(case)):
        first = L - case["new"]
        for j in range(first, L):
            k[table[i][j // page], j % page] = s["k_new"][i * case["new"] + j - first].double()
            v[table[i][j // page], j % page] = s["v_new"][i * case["new"] + j - first].double()
        pos[i, :, first:L] = torch.arange(L + 1000 - case["new"], L + 1000, dtype=torch.int32, device="cuda")
        weight[i, :, first:L] = 0.0
    return [k, v, pos, weight]


def _exact_rope(x, case, t0):
    F, out = case["gh"] * case["gw"], []
    at = torch.arange(x.shape[0], dtype=torch.float64, device="cuda")
    where = [t0 + torch.floor(at / F), torch.floor(torch.remainder(at, F) / case["gw"]), torch.remainder(at, case["gw"])]
    z, first = torch.view_as_complex(x.reshape(x.shape[0], D // 2, 2).contiguous()), 0
    for axis, pairs in enumerate(PAIRS):
        for m in range(pairs):
            out.append(z[:, first + m] * torch.exp(1j * where[axis] * 10000.0 ** (-m / pairs)))
        first += pairs
    return torch.view_as_real(torch.stack(out, 1)).reshape(x.shape[0], D)


def _exact_window(case, s):
    F = case["gh"] * case["gw"]
    off = max(0, math.ceil(case["lk"] / F) - math.ceil(case["lq"] / F))
    group, rows = case["hq"] // case["hkv"], 4096
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    kb = torch.arange(case["lk"], device="cuda") // (F * case["block"])
    qb = (off + torch.arange(case["lq"], device="cuda") // F) // case["block"]
    for g in range(case["hkv"]):
        k, v = s["k"][:, g].double(), s["v"][:, g].double()
        k = _exact_rope(k, case, 0) if case["rope"] else k
        for h in range(g * group, (g + 1) * group):
            q = s["q"][:, h].double()
            q = _exact_rope(q, case, off) if case["rope"] else q
            for a in range(0, case["lq"], rows):
                back = qb[a:a + rows, None] - kb[None, :]
                seen = (back >= 0) & ((back < case["window"]) | (kb < case["sinks"])[None, :])
                o[a:a + rows, h] = _softmax_rows(q[a:a + rows], k, v, seen)[1]
    return [o]
