"""The workloads of rotary positions, of cache writes that rotate on the way, and of attention
over a prefix that sequences share: their cases, inputs, plain forms and 64-bit values.

Operators (``op`` of a case):

``rotate``   heads [tokens, heads, 128] turned by their tokens' positions, out of place; with
             ``transposed`` the other way round, which is the gradient (``rotate``).
``write``    a chunk's q, k and v, side by side as a projection leaves them: k is turned by its
             position and goes into the pages beside v, the boxes follow, q comes back turned
             (``prefill_rotary``; n = 1: a ``RotaryPlan``; narrow caches too).
``prefix``   one query token per sequence over its whole cache, where groups of sequences begin
             with the same pages (a ``PrefixPlan``).
"""
import math

import torch

own = False

D = 128
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # The queries of four decoded tokens: the smallest call, its latency counts.
        dict(name="rotate_tokens", op="rotate", n=4, heads=32, dtype="fp16", rd=128, inter=False, scaling="none", at=1000, packed=False, transposed=False),
        # The q and k heads of an 8K prompt inside the projection's output (q, k and v rows).
        dict(name="rotate_prompt_8k", op="rotate", n=8192, heads=40, dtype="fp16", rd=128, inter=False, scaling="none", at=0, packed=True, transposed=False),
        # A gradient of a bf16 model that turns half of each head, at far scaled positions.
        dict(name="rotate_far_gradient", op="rotate", n=1999, heads=24, dtype="bf16", rd=64, inter=True, scaling="yarn", at=1000000, packed=False, transposed=True),
        # fp32 heads, three quarters of each turned, an odd number of tokens.
        dict(name="rotate_fp32", op="rotate", n=4097, heads=8, dtype="fp32", rd=96, inter=False, scaling="linear", at=30000, packed=False, transposed=False),
        # A decode step of one short chat: one token's heads; its latency counts.
        dict(name="append_token", op="write", narrow=False, batch=1, hq=8, hkv=8, page=16, n=1, ctx=1000, ragged=False, dtype="fp16", rd=128, inter=False, scaling="none"),
        # A decode step of a serving batch of a bf16 model.
        dict(name="append_batch", op="write", narrow=False, batch=64, hq=32, hkv=8, page=16, n=1, ctx=3000, ragged=True, dtype="bf16", rd=64, inter=True, scaling="none"),
        # A whole 32K prompt of a model with 32 MHA heads: the largest write.
        dict(name="write_prompt_32k", op="write", narrow=False, batch=1, hq=32, hkv=32, page=16, n=32768, ctx=0, ragged=False, dtype="fp16", rd=128, inter=False, scaling="bands"),
        # A chunk of a chunked prefill into narrow caches, sequences that start mid-page.
        dict(name="write_chunk_narrow", op="write", narrow=True, batch=4, hq=32, hkv=8, page=32, n=519, ctx=2500, ragged=True, dtype="fp16", rd=128, inter=False, scaling="bands"),
        # A few chats behind one short instruction; its latency counts.
        dict(name="prefix_small", op="prefix", hq=8, hkv=8, page=16, groups="4x512", tail=100),
        # A batch of questions about one 32K document.
        dict(name="prefix_document_32k", op="prefix", hq=32, hkv=8, page=16, groups="32x32768", tail=512),
        # MHA heads, long answers behind a shared 8K prompt: most of the bytes are not shared.
        dict(name="prefix_mha_8k", op="prefix", hq=32, hkv=32, page=16, groups="16x8192", tail=2048),
        # Several prefixes in one batch, a sequence of its own, prefixes that end inside a page.
        dict(name="prefix_groups", op="prefix", hq=32, hkv=4, page=32, groups="20x6000 9x16400 1x0 18x333", tail=700),
    ]


def _groups(c):
    """(sequences, tokens of their common prefix) of the groups of a batch."""
    return [tuple(int(x) for x in g.split("x")) for g in c["groups"].split()]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "write", "write", "prefix", "prefix"])
    c = dict(op=op)
    if op != "prefix":
        c["rd"] = rng.choice([128, 128, 128, 96, 64, 32, 8 * rng.randint(1, 16)])
        c["inter"] = rng.random() < 0.4
        c["scaling"] = rng.choice(["none", "none", "linear", "ntk", "bands", "yarn"])
    if op == "rotate":
        c["dtype"] = rng.choice(["fp16", "fp16", "bf16", "fp32"])
        c["heads"] = rng.choice([1, 3, 4, 8, 24, 32, 40, 64])
        c["n"] = _log_int(rng, 1, (1 << 18) // c["heads"])
        c["at"] = rng.choice([0, _log_int(rng, 1, 1 << 20)])
        c["packed"] = rng.random() < 0.5
        c["transposed"] = rng.random() < 0.3
        return c
    c["hkv"] = rng.choice([1, 2, 4, 8, 16, 32])
    c["hq"] = c["hkv"] * rng.choice([g for g in (1, 2, 4, 8) if g * c["hkv"] <= 32])
    c["page"] = rng.choice([16, 32])
    if op == "write":
        c["dtype"] = rng.choice(["fp16", "fp16", "bf16"])
        c["narrow"] = rng.random() < 0.3
        c["batch"] = _log_int(rng, 1, 64)
        most = max(16, (1 << (13 if c["narrow"] else 18)) // (c["hkv"] * c["batch"]))
        c["n"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, most)
        c["ctx"] = rng.choice([0, _log_int(rng, 1, 4000)])
        c["ragged"] = rng.random() < 0.6
        return c
    room = (1 << 18) // c["hkv"]  # tokens, shared and not
    counts, prefixes = [], []
    for _ in range(rng.choice([1, 1, 2, 3])):
        counts.append(_log_int(rng, 1, 40))
        prefixes.append(min(32768, _log_int(rng, 16, max(17, room // 4))))
    c["groups"] = " ".join("%dx%d" % g for g in zip(counts, prefixes))
    c["tail"] = _log_int(rng, 1, max(2, min(4000, room // sum(counts))))
    return c


# ------------------------------------------------------------------ frequencies
#: What a scaled case asks for: factor, the length that the unscaled model knew.
FACTOR, LENGTH, BASE = 8.0, 4096, 10000.0


def _frequencies(c):
    """(radians per position of the rd / 2 pairs, what the cosines and sines are multiplied by)."""
    d, how = c["rd"], c["scaling"]
    i = torch.arange(d // 2, dtype=torch.float64)
    base = BASE * FACTOR ** (d / (d - 2)) if how == "ntk" else BASE
    f = base ** (-2 * i / d)
    if how == "linear":
        f = f / FACTOR
    elif how == "bands":  # long waves are stretched, short ones are not, those between in part
        turns = LENGTH * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = keep * f + (1 - keep) * f / FACTOR
    elif how == "yarn":
        low, high = (d * math.log(LENGTH / (2 * math.pi * r)) / (2 * math.log(BASE)) for r in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = ramp * f / FACTOR + (1 - ramp) * f
        return f, 0.1 * math.log(FACTOR) + 1
    return f, 1.0


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _handles(st)
    return st


def _lens(c):
    """The sequences' lengths before a write, or at a decode over prefixes."""
    if c["op"] == "write":
        n = [c["ctx"]] * c["batch"]
        if c["ragged"]:
            n = [c["ctx"] - (c["ctx"] * 3 * b) // (4 * c["batch"]) - (3 * b if c["ctx"] > 1000 else 0) for b in range(c["batch"])]
        return n
    B, lens = sum(count for count, _ in _groups(c)), []
    for count, prefix in _groups(c):
        for _ in range(count):
            lens.append(prefix + max(1, c["tail"] - (c["tail"] * 3 * len(lens)) // (4 * B)))
    return lens


def _inputs(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, dtype=torch.float16):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    if c["op"] == "rotate":
        st = dict(case=c)
        rows = normal(c["n"], c["heads"] + (8 if c["packed"] else 0), D, dtype=TYPES[c["dtype"]])
        st["x"] = rows[:, :c["heads"]]
        st["positions"] = (c["at"] + torch.arange(c["n"], device=dev)).to(torch.int32)
        st["positions"] = st["positions"][torch.randperm(c["n"], generator=gen, device=dev)].contiguous()
        st["out"] = torch.empty((c["n"], c["heads"], D), dtype=rows.dtype, device=dev)
        _angles_by(st)
        return st
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    B, hkv, P = len(lens), c["hkv"], c["page"]
    mp = (max(_lens(c)) + c.get("n", 0) + P - 1) // P + 1
    nph = B * mp + 3
    st = dict(case=c, start=lens, seq_lens=lens.clone())
    st["block_table"] = torch.randperm(nph, generator=gen, device=dev)[:B * mp].view(B, mp).to(torch.int32)
    if c["op"] == "prefix":
        # the sequences of a group begin with the pages of its first one
        counts, prefixes = torch.tensor(_groups(c)).T
        group = torch.repeat_interleave(torch.arange(len(counts)), counts).to(dev)
        st["heads"], st["prefix"] = (counts.cumsum(0) - counts).to(dev), prefixes.to(dev)
        first, shared = st["heads"][group], st["prefix"][group] // P
        same = torch.arange(mp, device=dev) < shared[:, None]
        bt = st["block_table"]
        bt = torch.where(same, bt[first], bt)
        # physical pages that are used, and no more (a whole pool would hold each prefix B times)
        used, bt = torch.unique(bt, return_inverse=True)
        nph = used.numel() + 3
        st["block_table"] = bt.to(torch.int32).contiguous()
        st["group"], st["first"] = group, first
        st["k_pool"], st["v_pool"] = normal(nph, hkv, P, D), normal(nph, hkv, P, D)
        # a prefix that ends inside a page: each sequence has that page to itself, with the same rows
        at = bt.gather(1, shared[:, None])[:, 0]
        same = (torch.arange(P, device=dev) < (st["prefix"][group] % P)[:, None])[:, None, :, None]
        for x in (st["k_pool"], st["v_pool"]):
            x[at] = torch.where(same, x[at[first]], x[at])
        st["meta"] = torch.zeros((B, hkv, mp, 2, D), dtype=torch.float16, device=dev)
        st["q"] = normal(B, c["hq"], D) * 1.5
        return st
    n, hq = c["n"], c["hq"]
    st["qkv"] = normal(B, n, hq + 2 * hkv, D, dtype=TYPES[c["dtype"]])
    st["q_out"] = torch.empty((B, n, hq, D), dtype=torch.float16, device=dev)
    st["meta"] = torch.zeros((B, hkv, mp, 2, D), dtype=torch.float16, device=dev)
    # what the open page holds already, and its box
    page = (lens // P).long()
    rows = [normal(B, hkv, P, D), normal(B, hkv, P, D)]
    live = (torch.arange(P, device=dev) < (lens % P)[:, None])[:, None, :, None]
    for e, x in enumerate((torch.where(live, rows[0], math.inf).amin(-2), torch.where(live, rows[0], -math.inf).amax(-2))):
        st["meta"][torch.arange(B, device=dev), :, page, e] = torch.where(live.any(-2), x, 0.0).to(torch.float16)
    if c["narrow"]:
        for name, row in zip("kv", rows):
            st[name + "_open"], st[name + "_before"] = row.clone(), row
            st[name + "_pool"] = torch.zeros((nph, hkv, P, D), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
            st[name + "_scale"] = torch.ones((nph, hkv), dtype=torch.float32, device=dev)
    else:
        at = st["block_table"].gather(1, page[:, None])[:, 0].long()
        for name, row in zip("kv", rows):
            st[name + "_pool"] = torch.zeros((nph, hkv, P, D), dtype=torch.float16, device=dev)
            st[name + "_pool"][at] = row
    _angles_by(st)
    return st


def _angles_by(st):
    f, magnitude = _frequencies(st["case"])
    st["inv_freq"], st["magnitude"] = f.cuda(), magnitude


def _handles(st):
    """What a program that uses the framework keeps between calls: the rotation, the cache's
    descriptor, its workspace, a plan where it decodes in a loop."""
    import query_aware_kv_gb300 as q
    c = st["case"]
    if c["op"] != "prefix":
        how = None if c["scaling"] == "none" else c["scaling"]
        st["rope"] = q.Rope(c["rd"], base=BASE, interleaved=c["inter"], scaling=how, factor=FACTOR, original_length=LENGTH)
    if c["op"] == "rotate":
        return
    if c["op"] == "write" and c["narrow"]:
        cache = q.NarrowCache(st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], st["k_open"], st["v_open"],
                              st["meta"], st["block_table"], st["seq_lens"], c["hq"])
        st["ws"] = q.narrow_workspace(cache)
    else:
        cache = q.PagedCache(st["k_pool"], st["v_pool"], st["meta"], st["block_table"], st["seq_lens"], c["hq"])
        if c["op"] == "prefix":
            groups = _groups(c)
            st["ws"] = q.prefix_workspace(cache, groups)
            st["plan"] = q.PrefixPlan(cache, groups, st["ws"])
        else:
            st["ws"] = q.window_workspace(cache)
    st["cache"] = cache
    if c["op"] == "write" and c["n"] == 1:
        st["plan"] = q.RotaryPlan(cache, st["rope"], st["ws"], q_out=st["q_out"][:, 0])


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _parts(st):
    """q, k and v of a write, views of the projection's rows."""
    c, x = st["case"], st["qkv"]
    return x[:, :, :c["hq"]], x[:, :, c["hq"]:c["hq"] + c["hkv"]], x[:, :, c["hq"] + c["hkv"]:]


def _run_own(st):
    import query_aware_kv_gb300 as q
    c = st["case"]
    if c["op"] == "rotate":
        return q.rotate(st["rope"], st["x"], st["positions"], out=st["out"], transposed=c["transposed"])
    if c["op"] == "prefix":
        out, lse = st["plan"].decode(st["q"])
        return dict(out=out, lse=lse)
    _rewind(st)
    qq, k, v = _parts(st)
    if c["n"] == 1:
        st["plan"].append(qq[:, 0], k[:, 0], v[:, 0])
    elif c["narrow"]:
        q.narrow_prefill_rotary(st["cache"], st["rope"], qq, k, v, st["ws"], q_out=st["q_out"])
    else:
        q.prefill_rotary(st["cache"], st["rope"], qq, k, v, st["ws"], q_out=st["q_out"])
    return _written(st)


def _rewind(st):
    """Every pass writes the same chunk at the same place, over the same open pages."""
    st["seq_lens"].copy_(st["start"])
    if st["case"]["narrow"]:
        st["k_open"].copy_(st["k_before"])
        st["v_open"].copy_(st["v_before"])


def _written(st):
    names = ["q_out", "k_pool", "v_pool", "meta", "seq_lens"]
    if st["case"]["narrow"]:
        names += ["k_scale", "v_scale", "k_open", "v_open"]
    return {n: st[n] for n in names}


def _run_plain(st):
    c = st["case"]
    if c["op"] == "rotate":
        st["out"].copy_(_turn(st, st["x"], st["positions"], c["transposed"]))
        return st["out"]
    if c["op"] == "prefix":
        return _plain_prefix(st)
    _rewind(st)
    return _plain_write(st)


def _turn(st, x, positions, transposed=False):
    """The heads x [..., heads, 128] turned by positions [...], in 32 bits (angles in 64)."""
    c = st["case"]
    rd = c["rd"]
    angle = positions.double()[..., None, None] * st["inv_freq"]
    cos = (torch.cos(angle) * st["magnitude"]).float()
    sin = (torch.sin(angle) * st["magnitude"]).float()
    if transposed:
        sin = -sin
    x = x.float()
    y = x.clone()
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if c["inter"] else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_write(st):
    c, L = st["case"], st["seq_lens"].long()
    B, n, hkv, P = st["qkv"].shape[0], c["n"], c["hkv"], c["page"]
    dev = L.device
    qq, k, v = _parts(st)
    at = L[:, None] + torch.arange(n, device=dev)
    st["q_out"].copy_(_turn(st, qq, at))
    T = (n + P - 1) // P + 1  # pages a chunk can touch
    off, first = L % P, L // P
    seq = torch.arange(B, device=dev)
    page = first[:, None] + torch.arange(T, device=dev)
    have = torch.arange(T * P, device=dev).view(1, T, P) < (off + n)[:, None, None]
    old = torch.arange(T * P, device=dev).view(1, T, P) < off[:, None, None]
    phys = st["block_table"].gather(1, page.clamp(max=st["block_table"].shape[1] - 1)).long()
    whole, some = have.all(-1), have.any(-1)
    part = (off + n) // P  # the page left open

    def place(name, new):
        rows = torch.zeros((B, T * P, hkv, D), dtype=torch.float16, device=dev)
        rows[:, :P] = (st[name + "_open"] if c["narrow"] else st[name + "_pool"][phys[:, 0]]).transpose(1, 2)
        rows[seq[:, None], off[:, None] + torch.arange(n, device=dev)] = new.to(torch.float16)
        pages = rows.view(B, T, P, hkv, D).transpose(2, 3)
        if not c["narrow"]:
            st[name + "_pool"][phys[some]] = torch.where((have & ~old)[some][:, None, :, None], pages[some], st[name + "_pool"][phys[some]])
            return pages
        full = pages[whole].float()
        m, e = torch.frexp(full.abs().amax(dim=(-1, -2)))  # 448 = 0.875 * 2^9 is the largest e4m3 number
        scale = torch.where(m > 0, torch.ldexp(torch.ones_like(m), e - torch.where(m <= 0.875, 9, 8)), 1.0)
        st[name + "_pool"].view(torch.uint8)[phys[whole]] = (full / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        st[name + "_scale"][phys[whole]] = scale
        left = (torch.arange(P, device=dev) < ((off + n) % P)[:, None])[:, None, :, None]
        st[name + "_open"].copy_(torch.where(left, pages[seq, part], st[name + "_open"]))
        return pages

    pages = place("k", _turn(st, k, at))
    place("v", v)
    live = have[:, :, None, :, None]
    box = torch.stack([torch.where(live, pages, math.inf).amin(-2), torch.where(live, pages, -math.inf).amax(-2)], dim=-2)
    b_at, t_at = some.nonzero(as_tuple=True)
    st["meta"].transpose(1, 2)[b_at, page[b_at, t_at]] = box[b_at, t_at].to(torch.float16)
    st["seq_lens"] += n
    return _written(st)


def _plain_prefix(st):
    """Every group's prefix once for all of its rows, every sequence's own tokens beside it."""
    c, bt, L = st["case"], st["block_table"].long(), st["seq_lens"].long()
    B, hkv, P, G = len(L), c["hkv"], c["page"], c["hq"] // c["hkv"]
    dev = L.device
    NG, C, S = (max(x) for x in zip((len(_groups(c)), 1, 1), *((0, n, t) for n, t in _groups(c))))
    group, rank, heads, prefix = st["group"], torch.arange(B, device=dev) - st["first"], st["heads"], st["prefix"]

    def rows(name, seq, pos):  # [len(seq), hkv, tokens, 128] at positions pos [len(seq), tokens]
        pos = pos.clamp(max=bt.shape[1] * P - 1)
        return st[name + "_pool"][bt[seq[:, None], pos // P], :, pos % P].float().transpose(1, 2)

    q = st["q"].float().view(B, hkv, G, D) / math.sqrt(D)
    s_at = torch.arange(S, device=dev).expand(NG, S)
    qg = torch.zeros((NG, C, hkv, G, D), device=dev)
    qg[group, rank] = q
    qg = qg.permute(0, 2, 1, 3, 4).reshape(NG, hkv, C * G, D)
    kp, vp = rows("k", heads, s_at), rows("v", heads, s_at)
    sp = (qg @ kp.transpose(-1, -2)).view(NG, hkv, C, G, S).permute(0, 2, 1, 3, 4)[group, rank]
    sp = torch.where((torch.arange(S, device=dev) < torch.minimum(prefix[group], L)[:, None])[:, None, None], sp, -math.inf)
    vp = torch.where((s_at < prefix[:, None])[:, None, :, None], vp, 0.0)
    t_at = prefix[group][:, None] + torch.arange(c["tail"], device=dev)
    seq = torch.arange(B, device=dev)
    kt, vt = rows("k", seq, t_at), rows("v", seq, t_at)
    live = t_at < L[:, None]
    stail = torch.where(live[:, None, None], q @ kt.transpose(-1, -2), -math.inf)
    vt = torch.where(live[:, None, :, None], vt, 0.0)
    top = torch.maximum(sp.amax(-1), stail.amax(-1))[..., None]
    ep, et = torch.exp(sp - top), torch.exp(stail - top)
    total = ep.sum(-1, keepdim=True) + et.sum(-1, keepdim=True)
    eg = torch.zeros((NG, C, hkv, G, S), device=dev)
    eg[group, rank] = ep
    og = eg.permute(0, 2, 1, 3, 4).reshape(NG, hkv, C * G, S) @ vp
    og = og.view(NG, hkv, C, G, D).permute(0, 2, 1, 3, 4)[group, rank]
    out = (og + et @ vt) / total
    return dict(out=out.reshape(B, c["hq"], D).to(torch.float16), lse=(top + torch.log(total)).reshape(B, c["hq"]))


# ------------------------------------------------------------------ the definition, in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "write" and c["n"] * c["hkv"] * c["batch"] > 300000:
        return None
    st = _inputs(case, seed)
    if c["op"] == "rotate":
        return _exact_turn(c, st["x"], st["positions"], c["transposed"])
    if c["op"] == "write":
        return _exact_write(st)
    B, hkv, P, G = len(st["start"]), c["hkv"], c["page"], c["hq"] // c["hkv"]
    out = torch.zeros((B, c["hq"], D), dtype=torch.float64, device=st["q"].device)
    lse = torch.zeros((B, c["hq"]), dtype=torch.float64, device=st["q"].device)
    for b, L in enumerate(st["start"].tolist()):
        phys = st["block_table"][b, :-(-L // P)].long()
        for g in range(hkv):
            kk = st["k_pool"][phys, g].double().reshape(-1, D)[:L]
            vv = st["v_pool"][phys, g].double().reshape(-1, D)[:L]
            s = st["q"][b, g * G:(g + 1) * G].double() @ kk.T / math.sqrt(D)
            z = torch.logsumexp(s, -1)
            out[b, g * G:(g + 1) * G] = torch.exp(s - z[:, None]) @ vv
            lse[b, g * G:(g + 1) * G] = z
    return dict(out=out, lse=lse)


def _exact_turn(c, x, positions, transposed=False):
    """Pairs as complex numbers, multiplied by magnitude * exp(+- i position * frequency)."""
    rd, x = c["rd"], x.double()
    f, magnitude = _frequencies(c)
    z = torch.polar(torch.full_like(f, magnitude).to(x.device).expand(*positions.shape, -1).contiguous(),
                    (positions.double()[..., None] * f.to(x.device)) * (-1 if transposed else 1))[..., None, :]
    y = x.clone()
    if c["inter"]:
        y[..., :rd] = torch.view_as_real(torch.view_as_complex(x[..., :rd].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(x[..., :rd // 2], x[..., rd // 2:rd]) * z
        y[..., :rd] = torch.cat([w.real, w.imag], -1)
    return y


def _exact_write(st):
    """The cache after the chunk, page by page from the definition: a turned key is what fp16
    holds of it, the boxes and codes are of those."""
    c = st["case"]
    P, n = c["page"], c["n"]
    lens = st["start"].long()
    qq, k, v = _parts(st)
    at = lens[:, None] + torch.arange(n, device=lens.device)
    new = {"k": _exact_turn(c, k, at), "v": v.double()}
    res = {name: x.double() if x.is_floating_point() else x.clone() for name, x in _written(st).items()}
    res["q_out"] = _exact_turn(c, qq, at)
    # the e4m3 numbers: 4-bit exponent, 3-bit fraction, subnormals below 2^-6, largest 448
    grid = torch.tensor([(m / 8) * 2.0 ** -6 for m in range(8)] +
                        [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=lens.device)
    mid = (grid[1:] + grid[:-1]) / 2
    for b, L in enumerate(lens.tolist()):
        first = L // P
        last = (L + n - 1) // P
        at = st["block_table"][b, first:last + 1].long()
        for name in ("k", "v"):
            held = st[name + "_open"][b] if c["narrow"] else st[name + "_pool"][at[0]]
            rows = new[name][b].transpose(0, 1)
            keep = held[:, :L % P].double()
            rows = torch.cat([keep, rows.to(torch.float16).double() if c["narrow"] else rows], 1)  # [hkv, tokens, D]
            if name == "k":
                for t in range(last + 1 - first):
                    res["meta"][b, :, first + t, 0] = rows[:, t * P:(t + 1) * P].amin(1)
                    res["meta"][b, :, first + t, 1] = rows[:, t * P:(t + 1) * P].amax(1)
            full = rows.shape[1] // P
            if not c["narrow"]:
                for t in range(last + 1 - first):
                    one = rows[:, t * P:(t + 1) * P]
                    res[name + "_pool"][at[t], :, :one.shape[1]] = one
                continue
            if full:
                pages = rows[:, :full * P].reshape(rows.shape[0], full, P, D).transpose(0, 1)
                top = pages.abs().amax((-1, -2))
                scale = torch.where(top > 0, torch.exp2(torch.ceil(torch.log2(top / 448))), 1.0)
                y = pages / scale[..., None, None]
                lo = torch.searchsorted(mid, y.abs().contiguous())  # the nearest number, a tie to the even fraction
                tie = (lo < mid.numel()) & (mid[lo.clamp(max=mid.numel() - 1)] == y.abs())
                near = grid[torch.where(tie & (lo % 2 == 1), lo + 1, lo)]
                res[name + "_pool"][at[:full]] = torch.copysign(near, y)
                res[name + "_scale"][at[:full]] = scale
            rest = rows[:, full * P:]
            res[name + "_open"][b, :, :rest.shape[1]] = rest
        res["seq_lens"][b] = L + n
    return res


# ------------------------------------------------------------------ the work of a pass
def work(case):
    c = case
    if c["op"] == "rotate":
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": 2 * c["n"] * c["heads"] * D * size + 4 * c["n"], "flops": 3 * c["n"] * c["heads"] * c["rd"]}
    P, hq, hkv = c["page"], c["hq"], c["hkv"]
    if c["op"] == "prefix":
        lens = _lens(c)
        byte = len(lens) * hq * (4 * D + 4)
        b = 0
        for count, prefix in _groups(c):
            shared = prefix // P * P
            own_tokens = sum(lens[b:b + count]) - count * shared
            byte += (shared + own_tokens) * hkv * 4 * D
            b += count
        return {"bytes": byte, "flops": sum(lens) * hq * 4 * D}
    B, n = c["batch"], c["n"]
    byte = B * n * (hq * 4 * D + 2 * hkv * 2 * D)  # q in and out, k and v in
    for L in _lens(c):
        tail, full = (L + n) % P, (L + n) // P - L // P
        boxes = -(-(L + n) // P) - L // P
        byte += hkv * (boxes * 4 * D + (4 * D if L % P else 0))
        if not c["narrow"]:
            byte += 2 * n * hkv * 2 * D
        elif full:
            byte += 2 * hkv * (full * (P * D + 4) + (L % P + tail) * 2 * D)
        else:
            byte += 2 * hkv * n * 2 * D
    return {"bytes": byte, "flops": 3 * B * n * (hq + hkv) * c["rd"]}
