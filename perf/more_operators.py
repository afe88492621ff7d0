"""Cases of the page-table and 4-bit-cache operators, for timing and comparison.

Three operators that a serving loop runs around the paged attention of this library:

  tables   sdpa_paged_tables: the page tables, row offsets, positions and cache slots of a step's
           batch, from past and new lengths and a list of free pages, all on the device
  append   sdpa_paged4_append: new keys (rotated on the way) and values into a cache of 4 bits a
           value, at the slots that the first operator found
  attn     sdpa_paged4_attn: attention of each sequence's new tokens (one, a few or a chunk) over
           its pages of that cache

`own` selects between the plain form of each operator in elementary torch operations and the
library's calls; both take the same prepared state.

A cached head row of D channels is a record of bytes: D / 2 bytes of codes (channel 2j in the low
half of byte j, channel 2j + 1 in the high half), then for each 32 channels a minimum and a scale
in the model's type.  A value is minimum + scale * code.
"""
import math
import random

import torch

own = False

GROUP = 32
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _row_bytes(D, es):
    return D // 2 + D // GROUP * 2 * es


# ----------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------

def _tables(name, B, lo_new, hi_new, lo_past, hi_past, page, ended, mix):
    """`ended`: of each hundred sequences, how many end with this step and give their pages back."""
    return {"name": name, "op": "tables", "B": B, "lo_new": lo_new, "hi_new": hi_new, "lo_past": lo_past,
            "hi_past": hi_past, "page": page, "ended": ended, "mix": mix}


def _append(name, dtype, B, lo_new, hi_new, lo_past, hi_past, Nkv, D, page, R, interleaved, mix):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "lo_new": lo_new, "hi_new": hi_new,
            "lo_past": lo_past, "hi_past": hi_past, "Nkv": Nkv, "D": D, "page": page, "R": R,
            "interleaved": interleaved, "mix": mix}


def _attn(name, dtype, B, lo_new, hi_new, chunks, lo_past, hi_past, Nq, Nkv, D, page, window, sink, softcap, mix):
    return {"name": name, "op": "attn", "dtype": dtype, "B": B, "lo_new": lo_new, "hi_new": hi_new, "chunks": chunks,
            "lo_past": lo_past, "hi_past": hi_past, "Nq": Nq, "Nkv": Nkv, "D": D, "page": page, "window": window,
            "sink": sink, "softcap": softcap, "mix": mix}


def listed():
    return [
        # one decoding step of 64 sequences, a few of which have ended: latency alone
        _tables("tables_token", 64, 1, 1, 0, 32000, 16, 6, 31),
        # ragged prompts admitted together: slots and positions of some hundred thousand tokens
        _tables("tables_prompts", 48, 100, 8000, 0, 500, 64, 0, 32),
        # a large batch of short answers with chunks among them
        _tables("tables_many", 2000, 1, 16, 0, 3000, 24, 10, 33),
        # one decoding step of 64 sequences: latency
        _append("append_token", "bf16", 64, 1, 1, 0, 4000, 8, 128, 16, 128, False, 41),
        # the prompt of the library's grouped-query prefill workload, two sequences
        _append("append_prompt", "bf16", 2, 2048, 2048, 0, 0, 8, 128, 64, 128, False, 42),
        # chunks of ragged prompts, small float16 heads, half of the channels turned in adjacent pairs
        _append("append_chunks", "f16", 12, 100, 2000, 0, 4000, 8, 64, 24, 32, True, 43),
        # a small batch early in its answers: launches and latency
        _attn("attn_token_short", "bf16", 4, 1, 1, 0, 50, 500, 32, 8, 128, 16, -1, False, 0.0, 51),
        # a serving batch with long ragged contexts: bound by the cache's bytes
        _attn("attn_token_long", "bf16", 128, 1, 1, 0, 1000, 32000, 64, 8, 128, 64, -1, False, 0.0, 52),
        # five drafted tokens a sequence checked at once, float16
        _attn("attn_draft", "f16", 16, 5, 5, 0, 2000, 30000, 32, 8, 128, 32, -1, False, 0.0, 53),
        # one chunk of a long prompt over what is cached of it: bound by the products
        _attn("attn_chunk", "bf16", 1, 2048, 2048, 0, 30000, 32000, 32, 8, 128, 64, -1, False, 0.0, 54),
        # chunks and single tokens in one batch, with the library's window and sink heads
        _attn("attn_mixed", "bf16", 28, 1, 1, 4, 300, 9000, 64, 8, 64, 16, 1024, True, 0.0, 55),
        # float32 and a page size that is no power of two
        _attn("attn_f32", "f32", 8, 1, 1, 0, 500, 4000, 16, 4, 64, 24, -1, False, 0.0, 56),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["tables", "append", "append", "attn", "attn", "attn"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    if op == "tables":
        hi = _log(rng, 1, 8000)
        B = _log(rng, 1, max(1, min(2000, 200000 // hi)))
        hi_past = _log(rng, 1, max(1, min(32000, 4000000 // B)))
        return _tables("drawn", B, rng.randrange(1, hi + 1), hi, 0, hi_past, page, rng.choice([0, 0, 5, 30]), mix)
    dtype = rng.choice(["bf16", "f16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Nkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        R = rng.choice([0, D, D, D // 2])
        lo = _log(rng, 1, 1000)
        B = _log(rng, 1, max(1, min(64, 6000 // lo)))
        return _append("drawn", dtype, B, lo, lo + rng.randrange(lo + 1), 0, _log(rng, 1, 4000), Nkv, D, page, R,
                       rng.random() < 0.4, mix)
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    window = rng.choice([-1, -1, -1, 100, 1024])
    sink = rng.random() < 0.3
    softcap = rng.choice([0.0, 0.0, 0.0, 30.0])
    kind = rng.choice(["token", "token", "few", "chunk", "mixed"])
    past = _log(rng, 60, 20000)
    B = _log(rng, 1, max(1, min(64, 300000 // past)))
    lo = hi = 1
    chunks = 0
    if kind == "few":
        lo, hi = 1, rng.randrange(2, 17)
    elif kind == "chunk":
        lo = _log(rng, 17, 1500 if dtype != "f32" else 200)
        B = min(B, 4, max(1, 3000 // lo))
        hi = lo + rng.randrange(1, 100)
    elif kind == "mixed":
        chunks = rng.randrange(1, 4)
        B = max(B, chunks + 1)
        if dtype == "f32":
            dtype = "bf16"
    return _attn("drawn", dtype, B, lo, hi, chunks, past // 8, past, Nkv * group, Nkv, D, page, window, sink, softcap, mix)


def _lengths(case):
    """New tokens and past keys of each sequence, from the case alone; -1 new tokens: the sequence has
    ended.  The first `chunks` sequences of a mixed batch bring 512 tokens or a little fewer."""
    rng = random.Random(case["mix"])
    new, past = [], []
    for b in range(case["B"]):
        n = rng.randint(case["lo_new"], case["hi_new"])
        if b < case.get("chunks", 0):
            n = rng.randint(400, 512)
        if rng.random() * 100 < case.get("ended", 0):
            n = -1
        new.append(n)
        past.append(rng.randint(case["lo_past"], case["hi_past"]))
    return new, past


# ----------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------

def _angles(rows, half, dtype):
    ang = torch.arange(rows, dtype=torch.float64, device="cuda").view(-1, 1) * \
        (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).view(1, -1)
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def _randn(gen, shape, dtype):
    if dtype == torch.float32:
        return torch.randn(shape, generator=gen, device="cuda")
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _paged(gen, lens, page, spare):
    """A table of shuffled pages for sequences of these lengths, two entries wider than needed, and
    the ids of `spare` more pages."""
    need = [(t + page - 1) // page for t in lens]
    width = max(need) + 2
    order = torch.randperm(sum(need) + spare, generator=gen, device="cuda").to(torch.int32)
    counts = torch.tensor(need, device="cuda").view(-1, 1)
    used = torch.arange(width, device="cuda").view(1, -1) < counts
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[used] = order[:sum(need)]
    return table, order[sum(need):].clone(), sum(need) + spare


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    new, past = _lengths(case)
    page = case["page"]
    if case["op"] == "tables":
        grown = sum((max(n, 0) + p + page - 1) // page - (p + page - 1) // page for n, p in zip(new, past))
        table, spare, pages = _paged(gen, past, page, grown + 5)
        wide = max((max(n, 0) + p + page - 1) // page for n, p in zip(new, past)) + 2
        st["table"] = torch.full((case["B"], wide), -1, dtype=torch.int32, device="cuda")
        st["table"][:, :table.shape[1]] = table[:, :wide]
        st["free"] = torch.zeros(pages, dtype=torch.int32, device="cuda")
        st["free"][:spare.numel()] = spare
        st["count"] = torch.tensor([spare.numel()], dtype=torch.int32, device="cuda")
        st["past"] = torch.tensor(past, dtype=torch.int32, device="cuda")
        st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        tokens = st["tokens"] = sum(max(n, 0) for n in new) + 3      # rows of the program's buffers, a few more than used
        st["out"] = dict(kv_lens=torch.empty_like(st["past"]), free_count_out=torch.empty_like(st["count"]),
                         cu_new=torch.empty(case["B"] + 1, dtype=torch.int32, device="cuda"),
                         positions=torch.empty(tokens, dtype=torch.int64, device="cuda"),
                         slots=torch.empty(tokens, dtype=torch.int64, device="cuda"))
        return st
    dt = _DT[case["dtype"]]
    B, Nkv, D = (case[x] for x in ("B", "Nkv", "D"))
    lens = [n + p for n, p in zip(new, past)]
    table, _, pages = _paged(gen, lens, page, 3)
    rb = _row_bytes(D, _SIZE[case["dtype"]])
    tokens = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["new"], st["lens_host"], st["cu_host"] = new, lens, cu
    if case["op"] == "append":
        st["k_pages"] = torch.zeros(pages, Nkv, page, rb, dtype=torch.uint8, device="cuda")
        st["v_pages"] = torch.zeros(pages, Nkv, page, rb, dtype=torch.uint8, device="cuda")
        # keys with channels of unlike size, as trained projections give them
        size = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda"))
        st["k"] = (torch.randn(tokens, Nkv, D, generator=gen, device="cuda") * size).to(dt)
        st["v"] = _randn(gen, (tokens, Nkv, D), dt)
        st["k_held"], st["v_held"] = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(new, device="cuda"))
        first = torch.tensor([p - c for p, c in zip(past, cu)], device="cuda")
        st["positions"] = first[seq] + torch.arange(tokens, device="cuda")
        st["slots"] = table[seq, st["positions"] // page].long() * page + st["positions"] % page
        if case["R"]:
            st["cos"], st["sin"] = _angles(max(lens), case["R"] // 2, dt)
        return st
    pools = []
    for _ in range(2):
        pool = torch.empty(pages, Nkv, page, rb, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // (Nkv * page * D))
        for at in range(0, pages, step):                         # bounded memory
            part = pool[at:at + step]
            x = _randn(gen, (*part.shape[:-1], D), dt)
            part.copy_(_pack(x, dt))
        pools.append(pool)
    st.update(k_pages=pools[0], v_pages=pools[1], table=table,
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_new=max(new))
    # one new token everywhere: the call is uniform and needs no offsets
    st["cu"] = None if max(new) == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda")
    st["q"] = _randn(gen, (tokens, case["Nq"], D), dt)
    st["sink"] = _randn(gen, (case["Nq"],), dt) if case["sink"] else None
    return st


# ----------------------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------------------

def _quantise(x, dtype):
    """x (..., D) -> codes (..., D / 32, 32), minimum and scale (..., D / 32, 1), in fp32; the two are
    values of `dtype`, and the codes refer to them as rounded."""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    fifteen = torch.full_like(lo, 15.0)
    scale = ((hi - lo) / fifteen).to(dtype).float()
    codes = torch.where(scale > 0, torch.round((x - lo) / scale), torch.zeros_like(x)).clamp(0, 15)
    return codes, lo, scale


def _pack(x, dtype):
    codes, lo, scale = _quantise(x, dtype)
    c = codes.to(torch.uint8).flatten(-2)
    side = torch.cat((lo, scale), -1).to(dtype).flatten(-2).contiguous().view(torch.uint8)
    return torch.cat((c[..., 0::2] | (c[..., 1::2] << 4), side), -1)


def _unpack(rows, D, dtype):
    """Records (..., row bytes) -> values (..., D) in fp32."""
    b = rows[..., :D // 2]
    codes = torch.stack((b & 15, b >> 4), -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    side = rows[..., D // 2:].contiguous().view(dtype).float().unflatten(-1, (-1, 2))
    return (codes * side[..., 1:] + side[..., :1]).flatten(-2)


def _rotate(x, c, s, R, interleaved):
    """x (..., D) with the first R channels rotated; c, s (..., R/2) broadcast over heads."""
    h = R // 2
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        r = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:R]
        r = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((r, x[..., R:]), -1) if R < x.shape[-1] else r


def _plain_tables(st):
    page, tokens = st["case"]["page"], st["tokens"]
    table, free, pages = st["table"], st["free"], st["free"].numel()
    past, new = st["past"].long(), st["new"].long()
    ended = new < 0
    n = torch.where(ended, 0, torch.minimum(new, table.shape[1] * page - past))
    before = n.cumsum(0) - n
    n = torch.minimum(n, (tokens - before).clamp(min=0))
    cu = torch.cat((torch.zeros_like(past[:1]), n.cumsum(0)))
    have = (past + page - 1) // page
    lens = torch.where(ended, 0, past + n)
    upto = torch.where(ended, have, (past + n + page - 1) // page)
    col = torch.arange(table.shape[1], device="cuda").view(1, -1)
    # the pages of ended sequences go on top of the list, those of grown ones come from there
    gone = (ended.view(-1, 1) & (col < have.view(-1, 1)) & (table >= 0) & (table < pages)).flatten()
    longer = torch.cat((free, free[:1]))
    longer[torch.where(gone, st["count"].long() + gone.cumsum(0) - 1, pages)] = table.flatten()
    free.copy_(longer[:pages])
    top = st["count"].long() + gone.sum()
    need = upto - have
    taken = need.cumsum(0) - need
    at = top - 1 - (taken.view(-1, 1) + col - have.view(-1, 1))
    ids = torch.where(at >= 0, free[at.clamp(0, pages - 1)], -1)
    table.copy_(torch.where((col >= have.view(-1, 1)) & (col < upto.view(-1, 1)), ids, table))
    t = torch.arange(tokens, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    live = b < past.numel()
    b = b.clamp(max=past.numel() - 1)
    pos = torch.where(live, past[b] + t - cu[b], 0)
    ids = table[b, pos // page].long()
    slots = torch.where(live & (ids >= 0), ids * page + pos % page, -1)
    return lens.int(), cu.int(), pos, slots, table, free, (top - need.sum()).int()


def _plain_append(st):
    case = st["case"]
    dt, D = _DT[case["dtype"]], case["D"]
    k, v = st["k"], st["v"]
    if case["R"]:
        c, s = st["cos"][st["positions"]].float().unsqueeze(1), st["sin"][st["positions"]].float().unsqueeze(1)
        k = _rotate(k.float(), c, s, case["R"], case["interleaved"]).to(dt)
    ids, slot = st["slots"] // case["page"], st["slots"] % case["page"]
    held = []
    for x, pool in ((k, st["k_pages"]), (v, st["v_pages"])):
        rows = _pack(x, dt)
        pool[ids, :, slot] = rows
        held.append(_unpack(rows, D, dt).to(dt))
    return held[0], held[1], st["k_pages"], st["v_pages"]


def _plain_attn(st):
    case = st["case"]
    page, D, Nkv = case["page"], case["D"], case["Nkv"]
    dt = _DT[case["dtype"]]
    group = case["Nq"] // Nkv
    scale = 1.0 / math.sqrt(D)
    y = torch.empty_like(st["q"])
    for b, n in enumerate(st["new"]):
        at, T = st["cu_host"][b], st["lens_host"][b]
        ids = st["table"][b, :(T + page - 1) // page].long()
        k = _unpack(st["k_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :T], D, dt)
        v = _unpack(st["v_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :T], D, dt)
        q = st["q"][at:at + n].float().view(n, Nkv, group, D).permute(1, 0, 2, 3).reshape(Nkv, n * group, D)
        pos = torch.arange(T - n, T, device="cuda").view(n, 1, 1)
        key = torch.arange(T, device="cuda")
        keep = key <= pos
        if case["window"] > 0:
            keep = keep & (key > pos - case["window"])
        s = (q @ k.transpose(1, 2)).view(Nkv, n, group, T) * scale
        if case["softcap"] > 0:
            s = case["softcap"] * torch.tanh(s / case["softcap"])
        s = s.masked_fill(~keep, -math.inf)
        m = s.amax(-1, keepdim=True)
        sink = None
        if st["sink"] is not None:
            sink = st["sink"].float().view(Nkv, 1, group, 1)
            m = torch.maximum(m, sink)
        p = torch.exp(s - m)
        den = p.sum(-1, keepdim=True)
        if sink is not None:
            den = den + torch.exp(sink - m)
        o = (p.view(Nkv, n * group, T) @ v).view(Nkv, n, group, D) / den
        y[at:at + n] = o.permute(1, 0, 2, 3).reshape(n, case["Nq"], D).to(y.dtype)
    return y


# ----------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return _plain_tables(state) if op == "tables" else _plain_append(state) if op == "append" else _plain_attn(state)
    from scaled_dot_product_gb300 import sdpa
    if op == "tables":
        lens, cu, pos, slots, count = sdpa.sdpa_paged_tables(state["table"], state["past"], state["new"], state["free"],
                                                             state["count"], page_size=case["page"],
                                                             tokens=state["tokens"], **state["out"])
        return lens, cu, pos, slots, state["table"], state["free"], count
    if op == "append":
        rot = {}
        if case["R"]:
            rot = dict(positions=state["positions"], cos_cache=state["cos"], sin_cache=state["sin"],
                       rotary_dim=case["R"], interleaved=case["interleaved"])
        kh, vh = state["k_held"], state["v_held"]
        kp, vp = sdpa.sdpa_paged4_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["slots"],
                                         k_held=kh, v_held=vh, **rot)
        return kh, vh, kp, vp
    return sdpa.sdpa_paged4_attn(state["q"], state["k_pages"], state["v_pages"], state["table"], state["lens"],
                                 cu_new=state["cu"], max_new=state["max_new"], window=case["window"],
                                 softcap=case["softcap"], head_sink=state["sink"])


# ----------------------------------------------------------------------------------------
# Work
# ----------------------------------------------------------------------------------------

def work(case):
    new, past = _lengths(case)
    page = case["page"]
    if case["op"] == "tables":
        tokens = sum(max(n, 0) for n in new) + 3
        pages = 0                # entries given back or taken: read from one list, written to the other
        read = 0                 # begun pages that take the first new tokens
        for n, p in zip(new, past):
            have = (p + page - 1) // page
            pages += have if n < 0 else (p + n + page - 1) // page - have
            read += 1 if n > 0 and p % page else 0
        return {"bytes": 16 * tokens + 8 * pages + 4 * read + 16 * case["B"] + 12, "flops": 4 * tokens}
    es = _SIZE[case["dtype"]]
    tokens, D, Nkv = sum(new), case["D"], case["Nkv"]
    rb = _row_bytes(D, es)
    if case["op"] == "append":
        rows = min(tokens, max(n + p for n, p in zip(new, past)))
        return {"bytes": tokens * Nkv * (4 * D * es + 2 * rb) + rows * case["R"] * es + tokens * (16 if case["R"] else 8),
                "flops": tokens * Nkv * (14 * D + 3 * case["R"])}
    keys = pairs = entries = 0
    for n, p in zip(new, past):
        first = max(0, p - case["window"] + 1) if case["window"] > 0 else 0
        keys += n + p - first
        entries += (n + p - 1) // page - first // page + 1
        if case["window"] > 0:
            pairs += sum(min(p + i + 1, case["window"]) for i in range(n))
        else:
            pairs += n * p + n * (n + 1) // 2
    return {"bytes": 2 * keys * Nkv * rb + 2 * tokens * case["Nq"] * D * es + 4 * entries + 8 * case["B"],
            "flops": 4 * D * pairs * case["Nq"]}


# ----------------------------------------------------------------------------------------
# The operators' definitions in 64 bits
# ----------------------------------------------------------------------------------------

def _stored(x, dtype):
    """What the cache holds of x (..., D), in 64 bits."""
    out = torch.empty_like(x)
    for g in range(0, x.shape[-1], GROUP):
        part = x[..., g:g + GROUP]
        low = part.min(-1).values[..., None]
        scale = ((part.max(-1).values[..., None] - low) / 15.0).to(dtype).double()
        steps = torch.round((part - low) / torch.where(scale == 0, torch.ones_like(scale), scale))
        out[..., g:g + GROUP] = low + scale * steps.clamp(0, 15)
    return out


def _values(rows, D, dtype):
    """Records as values in 64 bits, channel by channel out of their nibbles."""
    codes = torch.empty(*rows.shape[:-1], D, dtype=torch.float64, device=rows.device)
    codes[..., 0::2] = torch.remainder(rows[..., :D // 2], 16).double()
    codes[..., 1::2] = torch.div(rows[..., :D // 2], 16, rounding_mode="floor").double()
    pairs = rows[..., D // 2:].contiguous().view(dtype).double()
    low, scale = (pairs[..., i::2].repeat_interleave(GROUP, -1) for i in (0, 1))
    return low + scale * codes


def exact(case, seed):
    if case["op"] == "tables":
        return None                      # whole numbers alone: there is nothing to round
    st = prepare(case, seed)
    dt, D, page, Nkv = _DT[case["dtype"]], case["D"], case["page"], case["Nkv"]
    if case["op"] == "append":
        k = st["k"].double()
        if case["R"]:
            h = case["R"] // 2
            turn = torch.complex(st["cos"].double()[st["positions"]], st["sin"].double()[st["positions"]])[:, None]
            part = k[..., :case["R"]]
            part = part.unflatten(-1, (h, 2)) if case["interleaved"] else part.unflatten(-1, (2, h)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn)
            z = z.flatten(-2) if case["interleaved"] else z.transpose(-1, -2).flatten(-2)
            k = torch.cat((z, k[..., case["R"]:]), -1)
        # a turned key is held as rounded to the model's type; the pools are bytes, with no value in 64 bits
        return _stored(k.to(dt).double(), dt), _stored(st["v"].double(), dt), None, None
    if work(case)["flops"] > 4e12:
        return None
    new, past = _lengths(case)
    group = case["Nq"] // Nkv
    table = st["table"].long().cpu()
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["B"]):
        n, T = new[b], new[b] + past[b]
        rows = table[b, torch.arange(T) // page].cuda()
        slot = (torch.arange(T) % page).cuda()
        for h in range(Nkv):
            K = _values(st["k_pages"][rows, h, slot], D, dt)
            V = _values(st["v_pages"][rows, h, slot], D, dt)
            for i0 in range(0, n, 512):           # bounded memory: 512 tokens at a time
                i1 = min(n, i0 + 512)
                j = torch.arange(T, device="cuda")[None, :]
                p = (past[b] + torch.arange(i0, i1, device="cuda"))[:, None]
                out_of = j > p
                if case["window"] > 0:
                    out_of |= p - j >= case["window"]
                out_of = out_of.repeat_interleave(group, 0)
                q = st["q"][t0 + i0:t0 + i1, h * group:(h + 1) * group].double().flatten(0, 1)
                z = q @ K.T / D ** 0.5
                if case["softcap"] > 0:
                    z = torch.tanh(z / case["softcap"]) * case["softcap"]
                z[out_of] = -math.inf
                if st["sink"] is not None:
                    extra = st["sink"].double()[h * group:(h + 1) * group].repeat(i1 - i0)[:, None]
                    wts = torch.softmax(torch.cat((z, extra), 1), 1)[:, :T]
                else:
                    wts = torch.softmax(z, 1)
                y[t0 + i0:t0 + i1, h * group:(h + 1) * group] = (wts @ V).unflatten(0, (-1, group))
        t0 += n
    return y
