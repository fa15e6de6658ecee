"""The workloads of the 8-bit ("narrow") paged cache and of sliding-window attention with
sinks: their cases, inputs, plain forms and 64-bit values.

Operators (``op`` of a case):

``write``    a chunk of tokens goes into a narrow cache: whole pages become e4m3 with one
             power-of-two scale per (page, kv head), the open page stays fp16, the boxes
             follow (``narrow_prefill``).
``step``     one decode step on a narrow cache: append, page bounds, top-K, attention over
             the kept pages (``narrow_decode_step``).
``dense``    attention of one query token over a whole narrow cache
             (``narrow_dense_decode``).
``window``   attention of the last ``n`` tokens of every sequence over the first ``sink``
             tokens and the last ``window`` ones: n = 1 on the decode path
             (``window_decode``, or ``narrow_window_decode``), n > 1 on the prompt path
             (``window_prefill``).
"""
import math

import torch

own = False

D = 128


def listed():
    return [
        # A whole 32K prompt of a model with 32 MHA heads, written into an empty cache.
        dict(name="write_prompt_32k", op="write", batch=1, hq=32, hkv=32, page=16, n=32768, ctx=0, ragged=False),
        # A chunk of a chunked prefill, sequences of different lengths that start mid-page.
        dict(name="write_chunk_ragged", op="write", batch=4, hq=32, hkv=8, page=32, n=519, ctx=2500, ragged=True),
        # The smallest decode step: 1K tokens, 4 heads; its latency counts.
        dict(name="step_tiny", op="step", batch=1, hq=4, hkv=4, page=16, ctx=1023, top_k=16, ragged=False),
        # The benchmark's shape: 32K tokens, 32 MHA heads, a budget of 2048 tokens.
        dict(name="step_32k", op="step", batch=1, hq=32, hkv=32, page=16, ctx=32780, top_k=128, ragged=False),
        # Full attention over four 64K sequences with grouped heads.
        dict(name="dense_gqa_64k", op="dense", batch=4, hq=32, hkv=8, page=16, ctx=65536, ragged=False),
        # One short chat turn by turn: a few hundred visible tokens; its latency counts.
        dict(name="window_decode_small", op="window", narrow=False, batch=1, hq=8, hkv=8, page=16, ctx=1000, n=1, sink=4, window=500, ragged=False),
        # A serving batch of long ragged sequences, 4K window.
        dict(name="window_decode_batch", op="window", narrow=False, batch=8, hq=32, hkv=32, page=16, ctx=32768, n=1, sink=4, window=4096, ragged=True),
        # The same with grouped heads on a narrow cache, pages of 32.
        dict(name="window_decode_narrow", op="window", narrow=True, batch=16, hq=32, hkv=8, page=32, ctx=65536, n=1, sink=64, window=8200, ragged=True),
        # A whole 8K prompt, 32 MHA heads, 4K window: the largest product.
        dict(name="window_prompt_8k", op="window", narrow=False, batch=1, hq=32, hkv=32, page=16, ctx=8192, n=8192, sink=4, window=4096, ragged=False),
        # One chunk of a long prompt, grouped heads.
        dict(name="window_chunk_2k", op="window", narrow=False, batch=1, hq=32, hkv=8, page=16, ctx=24576, n=2048, sink=4, window=4096, ragged=False),
        # Odd sizes: ragged sequences, one shorter than the chunk (its first rows are empty).
        dict(name="window_chunk_ragged", op="window", narrow=False, batch=4, hq=16, hkv=4, page=32, ctx=1900, n=333, sink=17, window=1001, ragged=True),
        # A few drafted tokens checked at once over a long window: few rows, a long axis.
        dict(name="window_draft_5", op="window", narrow=False, batch=1, hq=32, hkv=8, page=16, ctx=65536, n=5, sink=4, window=32768, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "step", "dense", "window", "window", "window"])
    hkv = rng.choice([1, 2, 4, 8, 16, 32])
    g = rng.choice([g for g in (1, 2, 4, 8) if g * hkv <= 32])
    c = dict(op=op, hq=g * hkv, hkv=hkv, page=rng.choice([16, 32]), ragged=rng.random() < 0.6)
    c["batch"] = _log_int(rng, 1, 8)
    room = 1 << 20  # tokens x kv heads of the largest listed cases
    most = max(64, min(65536, room // (hkv * c["batch"])))
    if op == "write":
        c["ctx"] = rng.choice([0, _log_int(rng, 1, most)])
        c["n"] = _log_int(rng, 1, most)
    elif op == "step":
        c["ctx"] = _log_int(rng, 40, most)
        c["top_k"] = max(4, min(256, _log_int(rng, 64, 4096) // c["page"]))
    elif op == "dense":
        c["ctx"] = _log_int(rng, 1, most)
    else:
        c["ctx"] = _log_int(rng, 1, most)
        c["sink"] = rng.choice([0, 1, 4, _log_int(rng, 1, 200)])
        c["window"] = _log_int(rng, 1, 2 * c["ctx"])
        c["narrow"] = rng.random() < 0.25
        cells = 1 << 31  # (query row, token) pairs of the largest listed case
        rows = max(2, min(2048, c["ctx"] + 9, cells // (c["batch"] * c["hq"] * (c["ctx"] + 256))))
        c["n"] = 1 if c["narrow"] or rng.random() < 0.4 else _log_int(rng, 2, rows)
    return c


def _lens(c):
    """The sequences' lengths before the call: ctx, or spread over [ctx / 4, ctx]; a ragged
    batch of prompts has one that is shorter than its chunk."""
    n = [c["ctx"]] * c["batch"]
    if c["ragged"]:
        n = [c["ctx"] - (c["ctx"] * 3 * b) // (4 * c["batch"]) - (3 * b if c["ctx"] > 64 else 0) for b in range(c["batch"])]
        if c["op"] == "window" and c["n"] > 2 and c["batch"] > 1:
            n[-1] = min(n[-1], c["n"] - c["n"] // 3)
    return n


def _pages(c):
    new = c["n"] if c["op"] == "write" else 1 if c["op"] == "step" else 0
    return (max(_lens(c)) + new + c["page"] - 1) // c["page"] + 1


# ------------------------------------------------------------------ the format
def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (448 = 0.875 * 2^9 is the largest
    e4m3 number); 1 where amax is 0."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), e - torch.where(m <= 0.875, 9, 8))
    return torch.where(amax > 0, s, torch.ones_like(s))


def _encode(pages):
    """fp32 [..., P, 128] -> (e4m3 codes as bytes, scale [...])."""
    s = _pow2_scale(pages.abs().amax(dim=(-1, -2)))
    return (pages / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _handles(st)
    return st


def _inputs(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    B, hkv, P, mp = c["batch"], c["hkv"], c["page"], _pages(c)
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    nph = B * mp + 3
    st = dict(case=c, start=lens, seq_lens=lens.clone())
    st["block_table"] = torch.randperm(nph, generator=gen, device=dev)[:B * mp].view(B, mp).to(torch.int32)
    narrow = c["op"] != "window" or c["narrow"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float16)

    k = normal(nph, hkv, P, D)
    v = normal(nph, hkv, P, D)
    if c["op"] == "step":
        # as many relevant pages per head as the budget holds beside the first and the last
        # page: their keys stand out from the rest
        r = torch.rand((B, hkv, mp), generator=gen, device=dev)
        last = (lens // P).long()  # the new token's page
        mid = torch.arange(mp, device=dev)[None, :]
        r = r.masked_fill(((mid == 0) | (mid >= last[:, None]))[:, None, :], 2.0)
        hot = r.argsort(-1).argsort(-1) < c["top_k"] - 2
        gain = torch.ones((nph, hkv), device=dev, dtype=torch.float16)
        gain[st["block_table"].long()] = torch.where(hot & (r < 1.5), 1.75, 1.0).to(torch.float16).transpose(1, 2)
        k *= gain[:, :, None, None]
    if narrow:
        # the open page's rows leave fp16 pages that the encoder never saw whole
        open_page = (lens // P).clamp(max=mp - 1).long()
        phys = st["block_table"].gather(1, open_page[:, None])[:, 0].long()
        st["k_open"], st["v_open"] = k[phys], v[phys]
        if c["op"] == "write":
            st["k_before"], st["v_before"] = k[phys], v[phys]
        kc, st["k_scale"] = _encode(k.float())
        vc, st["v_scale"] = _encode(v.float())
        st["k_pool"], st["v_pool"] = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    else:
        st["k_pool"], st["v_pool"] = k, v
    # boxes of the tokens present (step reads them; the others carry them along)
    st["meta"] = torch.zeros((B, hkv, mp, 2, D), dtype=torch.float16, device=dev)
    if c["op"] in ("write", "step"):
        rows = k[st["block_table"].long()].transpose(1, 2)  # [B, hkv, mp, P, D]
        pos = torch.arange(mp * P, device=dev).view(mp, P)
        live = (pos[None] < lens[:, None, None])[:, None, :, :, None]
        some = live.any(dim=-2)
        low = torch.where(live, rows, math.inf).amin(-2)
        high = torch.where(live, rows, -math.inf).amax(-2)
        st["meta"][:, :, :, 0] = torch.where(some, low, 0.0).to(torch.float16)
        st["meta"][:, :, :, 1] = torch.where(some, high, 0.0).to(torch.float16)
    n = c.get("n", 1)
    if c["op"] == "write":
        st["k"], st["v"] = normal(B, n, hkv, D), normal(B, n, hkv, D)
        st["v"] *= 3.0
    else:
        st["q"] = normal(B, n, c["hq"], D) if c["op"] == "window" and n > 1 else normal(B, c["hq"], D)
    if c["op"] == "step":
        st["k"], st["v"] = normal(B, 1, hkv, D), normal(B, 1, hkv, D)
    return st


def _handles(st):
    """What a program that uses the framework keeps between calls: the cache's descriptor,
    its workspace, a plan where it decodes in a loop."""
    import query_aware_kv_gb300 as q
    c = st["case"]
    if c["op"] == "window" and not c["narrow"]:
        cache = q.PagedCache(st["k_pool"], st["v_pool"], st["meta"], st["block_table"], st["seq_lens"], c["hq"])
        ws = q.window_workspace(cache, c["n"])
    else:
        cache = q.NarrowCache(st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], st["k_open"], st["v_open"],
                              st["meta"], st["block_table"], st["seq_lens"], c["hq"])
        ws = q.narrow_workspace(cache, c.get("top_k", 1))
    st["cache"], st["ws"] = cache, ws
    if c["op"] == "step":
        B, K = c["batch"], c["top_k"]
        st["idx"] = torch.empty((B, c["hkv"], K), dtype=torch.int32, device=ws.device)
        st["count"] = torch.empty((B, c["hkv"]), dtype=torch.int32, device=ws.device)
        st["plan"] = q.NarrowPlan(cache, K, ws, q.opts(sink_pages=1, local_pages=1), idx_out=st["idx"], count_out=st["count"])
    elif c["op"] == "dense":
        st["plan"] = q.NarrowPlan(cache, 1, ws)
    elif c["op"] == "window" and c["n"] == 1:
        st["plan"] = q.WindowPlan(cache, c["sink"], c["window"], ws)


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import query_aware_kv_gb300 as q
    op, cache, ws = st["case"]["op"], st["cache"], st["ws"]
    if op == "write":
        _rewind(st)
        q.narrow_prefill(cache, st["k"], st["v"], ws)
        return _written(st)
    if op == "step":
        st["seq_lens"].copy_(st["start"])
        out, lse = st["plan"].step(st["q"], st["k"][:, 0], st["v"][:, 0])
        return dict(out=out, lse=lse, idx=st["idx"], count=st["count"], **_written(st))
    if op == "dense":
        out, lse = st["plan"].dense(st["q"])
    elif st["case"]["n"] == 1:
        out, lse = st["plan"].decode(st["q"])
    else:
        out, lse = q.window_prefill(cache, st["q"], st["case"]["sink"], st["case"]["window"], ws)
    return dict(out=out, lse=lse)


def _rewind(st):
    """Every pass writes the same chunk at the same place, over the same open pages."""
    st["seq_lens"].copy_(st["start"])
    st["k_open"].copy_(st["k_before"])
    st["v_open"].copy_(st["v_before"])


def _written(st):
    return {n: st[n] for n in ("k_pool", "v_pool", "k_scale", "v_scale", "k_open", "v_open", "meta", "seq_lens")}


def _run_plain(st):
    op = st["case"]["op"]
    if op == "write":
        _rewind(st)
        _plain_write(st)
        return _written(st)
    if op == "step":
        return _plain_step(st)
    if op == "dense":
        c = st["case"]
        mp = st["block_table"].shape[1]
        idx = torch.arange(mp, device=st["q"].device).expand(c["batch"], c["hkv"], mp)
        out, lse = _plain_pages(st, idx, torch.ones_like(idx, dtype=torch.bool))
        return dict(out=out, lse=lse)
    return _plain_window(st)


def _plain_write(st):
    k, v, L = st["k"], st["v"], st["seq_lens"].long()
    B, n, hkv, _ = k.shape
    P = st["k_open"].shape[2]
    T = (n + P - 1) // P + 1  # pages a chunk can touch
    off, first = L % P, L // P
    seq = torch.arange(B, device=k.device)
    row = torch.arange(P, device=k.device)
    at = off[:, None] + torch.arange(n, device=k.device)
    have = torch.arange(T * P, device=k.device).view(1, T, P) < (off + n)[:, None, None]
    whole, some = have.all(-1), have.any(-1)
    page = first[:, None] + torch.arange(T, device=k.device)
    phys = st["block_table"].gather(1, page.clamp(max=st["block_table"].shape[1] - 1).long()).long()
    part = (off + n) // P  # the page left open
    left = (row < ((off + n) % P)[:, None])[:, None, :, None]

    def place(new, name):
        rows = torch.zeros((B, T * P, hkv, D), dtype=torch.float16, device=k.device)
        rows[:, :P] = st[name + "_open"].transpose(1, 2)
        rows[seq[:, None], at] = new
        pages = rows.view(B, T, P, hkv, D).transpose(2, 3)
        code, scale = _encode(pages[whole].float())
        st[name + "_pool"].view(torch.uint8)[phys[whole]] = code
        st[name + "_scale"][phys[whole]] = scale
        st[name + "_open"].copy_(torch.where(left, pages[seq, part], st[name + "_open"]))
        return pages

    pages = place(k, "k")
    place(v, "v")
    live = have[:, :, None, :, None]
    box = torch.stack([torch.where(live, pages, math.inf).amin(-2), torch.where(live, pages, -math.inf).amax(-2)], dim=-2)
    b_at, t_at = some.nonzero(as_tuple=True)
    st["meta"].transpose(1, 2)[b_at, page[b_at, t_at]] = box[b_at, t_at].to(torch.float16)
    st["seq_lens"] += n


def _plain_step(st):
    st["seq_lens"].copy_(st["start"])
    _plain_write(st)
    c = st["case"]
    L, P, K = st["seq_lens"].long(), c["page"], c["top_k"]
    N = (L + P - 1) // P
    q = st["q"].float().view(c["batch"], c["hkv"], -1, 1, D)
    box = st["meta"].float()[:, :, None]
    bound = torch.maximum(q * box[:, :, :, :, 0], q * box[:, :, :, :, 1]).sum(-1).amax(2)
    page = torch.arange(bound.shape[-1], device=bound.device)
    long = N[:, None] > K
    keep = long & ((page == 0) | (page == N[:, None] - 1))
    bound = torch.where(keep[:, None], math.inf, torch.where((page < N[:, None])[:, None], bound, -math.inf))
    rank = bound.sort(dim=-1, descending=True, stable=True).indices[..., :K]  # ties: the lower page
    count = N.clamp(max=K)[:, None].expand(-1, c["hkv"])
    none = torch.arange(rank.shape[-1], device=bound.device) >= count[..., None]
    idx = rank.masked_fill(none, 1 << 30).sort(-1).values
    out, lse = _plain_pages(st, idx.clamp(max=bound.shape[-1] - 1), idx < (1 << 30))
    sel = torch.full((c["batch"], c["hkv"], K), -1, dtype=torch.int32, device=bound.device)
    sel[..., :idx.shape[-1]] = idx.masked_fill(idx == (1 << 30), -1).to(torch.int32)
    return dict(out=out, lse=lse, idx=sel, count=count.to(torch.int32).contiguous(), **_written(st))


def _softmax(s, live, v):
    """(out, lse) of scores s [..., R, M] with a mask, values v [..., M, D]; a row without a
    visible token gives 0 and -inf."""
    s = torch.where(live, s, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    out = (e @ v) / torch.where(total > 0, total, 1.0)
    return out, (top + torch.log(total))[..., 0]


def _plain_pages(st, idx, kept):
    """Attention over the kept pages idx [B, hkv, K] of a narrow cache."""
    c = st["case"]
    B, hkv, P = c["batch"], c["hkv"], c["page"]
    L = st["seq_lens"].long()
    head = torch.arange(hkv, device=idx.device)[None, :, None]
    phys = st["block_table"].long()[torch.arange(B, device=idx.device)[:, None, None], idx]
    is_open = (idx == (L // P)[:, None, None])[..., None, None]

    def rows(name):
        x = st[name + "_pool"].view(torch.uint8)[phys, head].view(torch.float8_e4m3fn).float()
        x = x * st[name + "_scale"][phys, head][..., None, None]
        return torch.where(is_open, st[name + "_open"].float()[:, :, None], x).flatten(2, 3)

    pos = idx[..., None] * P + torch.arange(P, device=idx.device)
    live = ((pos < L[:, None, None, None]) & kept[..., None]).flatten(2, 3)[:, :, None]
    s = st["q"].float().view(B, hkv, -1, D) @ rows("k").transpose(-1, -2) / math.sqrt(D)
    v = torch.where(live[:, :, 0, :, None], rows("v"), 0.0)
    out, lse = _softmax(s, live, v)
    return out.reshape(B, c["hq"], D).to(torch.float16), lse.reshape(B, c["hq"])


def _plain_window(st):
    c = st["case"]
    B, n, hkv, P = c["batch"], c["n"], c["hkv"], c["page"]
    G = c["hq"] // hkv
    L = st["seq_lens"].long()
    room = st["block_table"].shape[1] * P
    sink = min(c["sink"], room)
    M = min(c["window"] + n - 1, room)  # the last M tokens, after the sinks
    v_at = torch.arange(sink + M, device=L.device)
    pos = torch.where(v_at < sink, v_at, L[:, None] - M + (v_at - sink))
    there = (pos >= 0) & (pos < L[:, None]) & ((v_at < sink) | (pos >= sink))
    pos = pos.clamp(0, room - 1)
    phys = st["block_table"].long().gather(1, pos // P)

    def rows(name):
        if not c["narrow"]:
            return st[name + "_pool"][phys, :, pos % P].float().transpose(1, 2)
        x = st[name + "_pool"].view(torch.uint8)[phys, :, pos % P].view(torch.float8_e4m3fn).float()
        x = x * st[name + "_scale"][phys][..., None]
        is_open = (pos // P == (L // P)[:, None])[..., None, None]
        now = st[name + "_open"][torch.arange(B, device=L.device)[:, None], :, pos % P].float()
        return torch.where(is_open, now, x).transpose(1, 2)

    at = L[:, None] - n + torch.arange(n, device=L.device)  # the queries' positions
    gap = at[:, :, None] - pos[:, None, :]
    live = there[:, None] & (gap >= 0) & ((pos[:, None] < sink) | (gap < c["window"]))  # [B, n, M]
    q = st["q"].float().view(B, n, hkv, G, D).permute(0, 2, 3, 1, 4)
    s = (q.reshape(B, hkv, G * n, D) @ rows("k").transpose(-1, -2) / math.sqrt(D)).view(B, hkv, G, n, -1)
    v = torch.where(there[:, None, :, None], rows("v"), 0.0)
    out, lse = _softmax(s, live[:, None, None], v[:, :, None])
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, c["hq"], D).to(torch.float16)
    lse = lse.permute(0, 3, 1, 2).reshape(B, n, c["hq"])
    return dict(out=out, lse=lse) if n > 1 else dict(out=out[:, 0], lse=lse[:, 0])


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "window" and c["n"] > 1 and sum(_seen(c)) * c["hq"] > 2e9:
        return None
    st = _inputs(case, seed)
    B, hkv, P = c["batch"], c["hkv"], c["page"]
    G = c["hq"] // hkv
    if c["op"] in ("write", "step"):
        state = _exact_write(st)
        if c["op"] == "write":
            return state
    lens = [int(x) + (c["op"] == "step") for x in _lens(c)]
    n = c.get("n", 1)
    dev = st["q"].device
    out = torch.zeros((B, n, c["hq"], D), dtype=torch.float64, device=dev)
    lse = torch.full((B, n, c["hq"]), -math.inf, dtype=torch.float64, device=dev)
    sel = torch.full((B, hkv, c.get("top_k", 1)), -1, dtype=torch.int32, device=dev)
    count = torch.zeros((B, hkv), dtype=torch.int32, device=dev)
    q = st["q"].double().view(B, n, hkv, G, D)
    for b in range(B):
        L = lens[b]
        N = -(-L // P)
        if N == 0:
            continue
        phys = st["block_table"][b, :N].long()
        for g in range(hkv):
            def logical(name):
                pool = st[name + "_pool"][phys, g].double()
                if name + "_scale" in st:
                    pool = pool * st[name + "_scale"][phys, g].double()[:, None, None]
                    if L % P:
                        pool[-1] = st[name + "_open"][b, g].double()
                return pool.reshape(-1, D)[:L]

            kk, vv = logical("k"), logical("v")
            j = torch.arange(L, device=dev)
            allowed = torch.ones((n, L), dtype=torch.bool, device=dev)
            if c["op"] == "window":
                at = torch.arange(L - n, L, device=dev)[:, None]
                allowed = (j <= at) & ((j < c["sink"]) | (j > at - c["window"]))
            elif c["op"] == "step":
                m = st["meta"][b, g, :N].double()
                ub = torch.stack([(torch.maximum(m[:, 0] * x, m[:, 1] * x)).sum(-1) for x in q[b, 0, g]]).amax(0)
                if N > c["top_k"]:
                    ub[0] = ub[-1] = math.inf
                keep = sorted(range(N), key=lambda p, u=ub.tolist(): (-u[p], p))[:c["top_k"]]
                sel[b, g, :len(keep)] = torch.tensor(sorted(keep), dtype=torch.int32)
                count[b, g] = len(keep)
                chosen = torch.zeros(N, dtype=torch.bool, device=dev)
                chosen[keep] = True
                allowed = chosen.repeat_interleave(P)[None, :L]
            for i0 in range(0, n, 1024):
                some = allowed[i0:i0 + 1024]
                for h in range(G):
                    s = (q[b, i0:i0 + 1024, g, h] @ kk.T) / math.sqrt(D)
                    s = s.masked_fill(~some, -math.inf)
                    z = torch.logsumexp(s, -1)
                    w = torch.exp(s - torch.where(torch.isinf(z), 0.0, z)[:, None])
                    out[b, i0:i0 + 1024, g * G + h] = w @ vv
                    lse[b, i0:i0 + 1024, g * G + h] = z
    if n == 1:
        out, lse = out[:, 0], lse[:, 0]
    if c["op"] == "step":
        return dict(out=out, lse=lse, idx=sel, count=count, **state)
    return dict(out=out, lse=lse)


def _exact_write(st):
    """The cache after the chunk, page by page from the definition (on st's own buffers for
    the step, whose attention reads them)."""
    P = st["k_open"].shape[2]
    new = {"k": st["k"].double(), "v": st["v"].double()}
    n = st["k"].shape[1]
    # the e4m3 numbers: 4-bit exponent, 3-bit fraction, subnormals below 2^-6, largest 448
    grid = torch.tensor([(m / 8) * 2.0 ** -6 for m in range(8)] +
                        [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=new["k"].device)
    mid = (grid[1:] + grid[:-1]) / 2
    for b, L in enumerate(st["start"].tolist()):
        first = L // P
        for name in ("k", "v"):
            keep = st[name + "_open"][b].double()[:, :L % P]
            rows = torch.cat([keep, new[name][b].transpose(0, 1)], 1)  # [hkv, tokens, D]
            full = rows.shape[1] // P
            if full:
                pages = rows[:, :full * P].reshape(rows.shape[0], full, P, D).transpose(0, 1)
                top = pages.abs().amax((-1, -2))
                scale = torch.exp2(torch.ceil(torch.log2(top / 448)))
                scale = torch.where(top > 0, scale, torch.ones_like(scale))
                y = pages / scale[..., None, None]
                # the nearest number, a tie to the even fraction
                lo = torch.searchsorted(mid, y.abs().contiguous())
                tie = (lo < mid.numel()) & (mid[lo.clamp(max=mid.numel() - 1)] == y.abs())
                near = grid[torch.where(tie & (lo % 2 == 1), lo + 1, lo)]
                at = st["block_table"][b, first:first + full].long()
                st[name + "_pool"][at] = torch.copysign(near, y).float().to(torch.float8_e4m3fn)
                st[name + "_scale"][at] = scale.float()
            rest = rows.shape[1] - full * P
            if rest:
                st[name + "_open"][b][:, :rest] = rows[:, full * P:].to(torch.float16)
            if name == "k":
                for t in range(-(-rows.shape[1] // P)):
                    one = rows[:, t * P:(t + 1) * P]
                    st["meta"][b, :, first + t, 0] = one.amin(1).to(torch.float16)
                    st["meta"][b, :, first + t, 1] = one.amax(1).to(torch.float16)
        st["seq_lens"][b] = L + n
    return {k: x.double() if x.is_floating_point() else x for k, x in _written(st).items()}


# ------------------------------------------------------------------ the work of a pass
def _seen(c):
    """Per sequence: the (query token, visible token) pairs of a window case."""
    S, W, n = c["sink"], c["window"], c["n"]
    total = []
    for L in _lens(c):
        seen = 0
        for t in range(max(0, L - n), L):
            lo = max(0, t - W + 1)
            seen += t + 1 - lo + min(S, lo)
        total.append(seen)
    return total


def work(case):
    c = case
    B, hq, hkv, P = c["batch"], c["hq"], c["hkv"], c["page"]
    io = 2 * B * hq * D * 2 + B * hq * 4  # q, out, lse
    if c["op"] == "write":
        byte = flop = 0
        for L in _lens(c):
            tail, full = (L + c["n"]) % P, (L + c["n"]) // P - L // P
            boxes = -(-(L + c["n"]) // P) - L // P
            byte += 2 * c["n"] * hkv * 2 * D  # the chunk
            if full:
                byte += 2 * hkv * (full * (P * D + 4) + (L % P + tail) * 2 * D)
            else:
                byte += 2 * hkv * c["n"] * 2 * D
            byte += hkv * (boxes * 4 * D + (4 * D if L % P else 0))
            flop += 6 * c["n"] * hkv * D
        return {"bytes": byte, "flops": flop}
    if c["op"] == "window":
        n, S, W = c["n"], c["sink"], c["window"]
        byte = 2 * B * n * hq * D * 2 + B * n * hq * 4
        row = 2 * D * (1 if c["narrow"] else 2)
        for L in _lens(c):
            lo = max(0, max(0, L - n) - W + 1)
            byte += (L - lo + min(S, lo)) * hkv * row
        return {"bytes": byte, "flops": sum(_seen(c)) * hq * 4 * D}
    byte, flop = io, 0
    for L in _lens(c):
        N = -(-L // P)
        if c["op"] == "step":
            N = -(-(L + 1) // P)
            byte += N * hkv * 4 * D + 4 * hkv * 2 * D + min(N, c["top_k"]) * hkv * 4
            flop += N * hq * 3 * D
            kept = min(L + 1, c["top_k"] * P)
        else:
            kept = L
        byte += kept * hkv * 2 * D + -(-kept // P) * hkv * 8
        flop += kept * hq * 4 * D
    return {"bytes": byte, "flops": flop}
