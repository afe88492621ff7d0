"""Cases of the paged-cache and query/key-norm operators, for timing and comparison.

Three operators that a decoder's attention layer runs around the dense ones of this library:

  norm_rotary   sdpa_qk_norm_rotary / sdpa_qk_norm_rotary_bwd: RMS norm of every query and key
                head, then the position rotation, in one pass; and its gradient
  append        sdpa_paged_append: new keys and values into a paged cache, the keys rotated on
                the way
  attn          sdpa_paged_attn: attention of each sequence's new tokens (one, a few or a chunk)
                over its pages

`own` selects between the plain form of each operator in elementary torch operations and the
library's calls; both take the same prepared state.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ----------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------

def _norm(name, grad, dtype, B, S, Nq, Nkv, D, R, interleaved):
    return {"name": name, "op": "norm_rotary", "grad": grad, "dtype": dtype, "B": B, "S": S, "Nq": Nq, "Nkv": Nkv,
            "D": D, "R": R, "interleaved": interleaved}


def _append(name, dtype, B, lo_new, hi_new, lo_past, hi_past, Nkv, D, page, R, interleaved, slots_first, mix):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "lo_new": lo_new, "hi_new": hi_new,
            "lo_past": lo_past, "hi_past": hi_past, "Nkv": Nkv, "D": D, "page": page, "R": R,
            "interleaved": interleaved, "slots_first": slots_first, "mix": mix}


def _attn(name, dtype, B, lo_new, hi_new, chunks, lo_past, hi_past, Nq, Nkv, D, page, window, sink, softcap, slots_first,
          mix):
    return {"name": name, "op": "attn", "dtype": dtype, "B": B, "lo_new": lo_new, "hi_new": hi_new, "chunks": chunks,
            "lo_past": lo_past, "hi_past": hi_past, "Nq": Nq, "Nkv": Nkv, "D": D, "page": page, "window": window,
            "sink": sink, "softcap": softcap, "slots_first": slots_first, "mix": mix}


def listed():
    return [
        # one decoding step of 32 sequences: a few hundred kilobytes, latency alone
        _norm("norm_rotary_token", False, "bf16", 32, 1, 32, 8, 128, 128, False),
        # the prompt of the library's grouped-query prefill workload
        _norm("norm_rotary_prompt", False, "bf16", 2, 2048, 32, 8, 128, 128, False),
        # an odd length, small heads, half of the channels rotated in adjacent pairs
        _norm("norm_rotary_partial", False, "f16", 3, 1501, 64, 8, 64, 32, True),
        # a training step's backward: gradients of queries, keys and both weight vectors
        _norm("norm_rotary_grad", True, "bf16", 2, 4096, 32, 8, 128, 128, False),
        # one decoding step of 64 sequences into pages of 16
        _append("append_token", "bf16", 64, 1, 1, 0, 500, 8, 128, 16, 128, False, True, 11),
        # chunks of ragged prompts in float16, pages of 64, heads before slots
        _append("append_chunks", "f16", 12, 100, 2000, 0, 3000, 8, 64, 64, 64, False, False, 12),
        # a small batch early in its answers: launches and latency
        _attn("attn_token_short", "bf16", 4, 1, 1, 0, 50, 500, 32, 8, 128, 16, -1, False, 0.0, True, 21),
        # a serving batch with long ragged contexts: bound by the cache's bytes
        _attn("attn_token_long", "bf16", 64, 1, 1, 0, 1000, 32000, 64, 8, 128, 64, -1, False, 0.0, True, 22),
        # five drafted tokens a sequence checked at once, float16
        _attn("attn_draft", "f16", 16, 5, 5, 0, 2000, 16000, 32, 8, 128, 32, -1, False, 0.0, True, 23),
        # one chunk of a long prompt over what is cached of it: bound by the products
        _attn("attn_chunk", "bf16", 1, 2048, 2048, 0, 30000, 32000, 32, 8, 128, 64, -1, False, 0.0, False, 24),
        # chunks and single tokens in one batch, with the library's window and sink heads
        _attn("attn_mixed", "bf16", 28, 1, 1, 4, 300, 9000, 64, 8, 64, 16, 1024, True, 0.0, True, 25),
        # float32 and a page size that is no power of two
        _attn("attn_f32", "f32", 8, 1, 1, 0, 500, 4000, 16, 4, 64, 24, -1, False, 0.0, True, 26),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ranges."""
    op = rng.choice(["norm", "norm", "append", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "f16", "bf16", "f32"])
    D = rng.choice([64, 128])
    Nkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    R = rng.choice([D, D, D // 2])
    if op == "norm":
        S = _log(rng, 1, 4000)
        B = _log(rng, 1, max(1, min(64, 8000 // S)))
        return _norm("drawn", rng.random() < 0.5, dtype, B, S, Nkv * group, Nkv, D, R, rng.random() < 0.4)
    page = rng.choice([8, 16, 24, 32, 64, 100, 128, 256])
    first = rng.random() < 0.6
    mix = rng.randrange(1 << 30)
    if op == "append":
        lo = _log(rng, 1, 1000)
        B = _log(rng, 1, max(1, min(64, 4000 // lo)))
        hi_past = _log(rng, 1, 4000)
        return _append("drawn", dtype, B, lo, lo + rng.randrange(lo + 1), 0, hi_past, Nkv, D, page,
                       rng.choice([0, R, R]), rng.random() < 0.4, first, mix)
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
    return _attn("drawn", dtype, B, lo, hi, chunks, past // 8, past, Nkv * group, Nkv, D, page, window, sink, softcap,
                 first, mix)


def _lengths(case):
    """New tokens and past keys of each sequence, from the case alone.  The first `chunks`
    sequences of a mixed batch bring 512 tokens or a little fewer."""
    rng = random.Random(case["mix"])
    new, past = [], []
    for b in range(case["B"]):
        n = rng.randint(case["lo_new"], case["hi_new"])
        if b < case.get("chunks", 0):
            n = rng.randint(400, 512)
        new.append(n)
        past.append(rng.randint(case["lo_past"], case["hi_past"]))
    return new, past


# ----------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------

def _tables(rows, half, dtype):
    ang = torch.arange(rows, dtype=torch.float64, device="cuda").view(-1, 1) * \
        (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).view(1, -1)
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def _randn(gen, shape, dtype):
    if dtype == torch.float32:
        return torch.randn(shape, generator=gen, device="cuda")
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    st = {"case": case}
    if case["op"] == "norm_rotary":
        B, S, Nq, Nkv, D, R = (case[x] for x in ("B", "S", "Nq", "Nkv", "D", "R"))
        st["q"] = _randn(gen, (B, S, Nq * D), dt)
        st["k"] = _randn(gen, (B, S, Nkv * D), dt)
        st["wq"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        st["wk"] = (1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        rows = S + 1500
        st["cos"], st["sin"] = _tables(rows, R // 2, dt)
        start = torch.randint(0, rows - S + 1, (B, 1), generator=gen, device="cuda")
        st["pos"] = (start + torch.arange(S, device="cuda").view(1, S)).contiguous()
        if case["grad"]:
            st["dyq"] = _randn(gen, (B, S, Nq * D), dt)
            st["dyk"] = _randn(gen, (B, S, Nkv * D), dt)
        return st
    new, past = _lengths(case)
    B, Nkv, D, page = (case[x] for x in ("B", "Nkv", "D", "page"))
    lens = [n + p for n, p in zip(new, past)]
    need = [(t + page - 1) // page for t in lens]
    width = max(need) + 2                         # tables are wider than what is used
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
    shape = (pool, page, Nkv, D) if case["slots_first"] else (pool, Nkv, page, D)
    kp, vp = _randn(gen, shape, dt), _randn(gen, shape, dt)
    if case["slots_first"]:
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    st.update(k_pages=kp, v_pages=vp, table=table, new=new, lens_host=lens,
              lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_new=max(new))
    tokens = sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st["cu_host"] = cu
    # one new token everywhere: the call is uniform and needs no offsets
    st["cu"] = None if max(new) == 1 else torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        st["k"], st["v"] = _randn(gen, (tokens, Nkv, D), dt), _randn(gen, (tokens, Nkv, D), dt)
        if case["R"]:
            st["cos"], st["sin"] = _tables(max(lens), case["R"] // 2, dt)
    else:
        st["q"] = _randn(gen, (tokens, case["Nq"], D), dt)
        st["sink"] = _randn(gen, (case["Nq"],), dt) if case["sink"] else None
    return st


# ----------------------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------------------

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


def _plain_norm(st):
    case = st["case"]
    B, S, D, R, inter = case["B"], case["S"], case["D"], case["R"], case["interleaved"]
    c = st["cos"][st["pos"]].float().unsqueeze(2)
    s = st["sin"][st["pos"]].float().unsqueeze(2)
    out = []
    for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])):
        xf = x.float().view(B, S, -1, D)
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
        y = _rotate(xf * r * w.float(), c, s, R, inter)
        out.append(y.view(B, S, -1).to(x.dtype))
    return tuple(out)


def _plain_norm_grad(st):
    case = st["case"]
    B, S, D, R, inter = case["B"], case["S"], case["D"], case["R"], case["interleaved"]
    c = st["cos"][st["pos"]].float().unsqueeze(2)
    s = st["sin"][st["pos"]].float().unsqueeze(2)
    dx, dw = [], []
    for x, w, dy in ((st["q"], st["wq"], st["dyq"]), (st["k"], st["wk"], st["dyk"])):
        xf = x.float().view(B, S, -1, D)
        r = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + 1e-6)
        g = _rotate(dy.float().view(B, S, -1, D), c, -s, R, inter)
        xh = xf * r
        dw.append((g * xh).double().sum((0, 1, 2)).to(w.dtype))
        gw = g * w.float()
        dx.append((r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).view(B, S, -1).to(x.dtype))
    return dx[0], dx[1], dw[0], dw[1]


def _plain_append(st):
    case = st["case"]
    page = case["page"]
    for b, n in enumerate(st["new"]):
        at, T = st["cu_host"][b], st["lens_host"][b]
        pos = torch.arange(T - n, T, device="cuda")
        k, v = st["k"][at:at + n], st["v"][at:at + n]
        if case["R"]:
            c, s = st["cos"][pos].float().unsqueeze(1), st["sin"][pos].float().unsqueeze(1)
            k = _rotate(k.float(), c, s, case["R"], case["interleaved"]).to(k.dtype)
        ids = st["table"][b].long()[pos // page]
        st["k_pages"][ids, :, pos % page] = k
        st["v_pages"][ids, :, pos % page] = v
    return st["k_pages"], st["v_pages"]


def _plain_attn(st):
    case = st["case"]
    page, D, Nkv = case["page"], case["D"], case["Nkv"]
    group = case["Nq"] // Nkv
    scale = 1.0 / math.sqrt(D)
    y = torch.empty_like(st["q"])
    for b, n in enumerate(st["new"]):
        at, T = st["cu_host"][b], st["lens_host"][b]
        ids = st["table"][b, :(T + page - 1) // page].long()
        k = st["k_pages"][ids].transpose(0, 1).reshape(Nkv, -1, D)[:, :T].float()
        v = st["v_pages"][ids].transpose(0, 1).reshape(Nkv, -1, D)[:, :T].float()
        q = st["q"][at:at + n].float().view(n, Nkv, group, D)
        pos = torch.arange(T - n, T, device="cuda").view(n, 1, 1)
        key = torch.arange(T, device="cuda")
        keep = key <= pos
        if case["window"] > 0:
            keep = keep & (key > pos - case["window"])
        for h in range(Nkv):
            s = (q[:, h].reshape(n * group, D) @ k[h].t()).view(n, group, T) * scale
            if case["softcap"] > 0:
                s = case["softcap"] * torch.tanh(s / case["softcap"])
            s = s.masked_fill(~keep, -math.inf)
            m = s.amax(-1, keepdim=True)
            sink = None
            if st["sink"] is not None:
                sink = st["sink"].float()[h * group:(h + 1) * group].view(1, group, 1)
                m = torch.maximum(m, sink)
            p = torch.exp(s - m)
            den = p.sum(-1, keepdim=True)
            if sink is not None:
                den = den + torch.exp(sink - m)
            o = (p.view(n * group, T) @ v[h]).view(n, group, D) / den
            y[at:at + n, h * group:(h + 1) * group] = o.to(y.dtype)
    return y


# ----------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "norm_rotary":
            return _plain_norm_grad(state) if case["grad"] else _plain_norm(state)
        return _plain_append(state) if op == "append" else _plain_attn(state)
    from scaled_dot_product_gb300 import sdpa
    if op == "norm_rotary":
        kw = dict(num_heads=case["Nq"], kv_num_heads=case["Nkv"], rotary_dim=case["R"], interleaved=case["interleaved"],
                  eps=1e-6)
        if case["grad"]:
            return sdpa.sdpa_qk_norm_rotary_bwd(state["q"], state["k"], state["dyq"], state["dyk"], state["wq"],
                                                state["wk"], state["cos"], state["sin"], state["pos"], **kw)
        return sdpa.sdpa_qk_norm_rotary(state["q"], state["k"], state["wq"], state["wk"], state["cos"], state["sin"],
                                        state["pos"], **kw)
    if op == "append":
        rot = {}
        if case["R"]:
            rot = dict(cos_cache=state["cos"], sin_cache=state["sin"], rotary_dim=case["R"],
                       interleaved=case["interleaved"])
        return sdpa.sdpa_paged_append(state["k"], state["v"], state["k_pages"], state["v_pages"], state["table"],
                                      state["lens"], cu_new=state["cu"], **rot)
    return sdpa.sdpa_paged_attn(state["q"], state["k_pages"], state["v_pages"], state["table"], state["lens"],
                                cu_new=state["cu"], max_new=state["max_new"], window=case["window"],
                                softcap=case["softcap"], head_sink=state["sink"])


# ----------------------------------------------------------------------------------------
# Work
# ----------------------------------------------------------------------------------------

def work(case):
    es = _SIZE[case["dtype"]]
    if case["op"] == "norm_rotary":
        B, S, D, R = case["B"], case["S"], case["D"], case["R"]
        N = case["Nq"] + case["Nkv"]
        data = B * S * N * D * es
        side = B * S * 8 + min(B * S, S + 1500) * R * es + 2 * D * es
        if case["grad"]:
            return {"bytes": 3 * data + side + 2 * D * es, "flops": B * S * N * (12 * D + 3 * R)}
        return {"bytes": 2 * data + side, "flops": B * S * N * (5 * D + 3 * R)}
    new, past = _lengths(case)
    tokens, page = sum(new), case["page"]
    if case["op"] == "append":
        data = 2 * tokens * case["Nkv"] * case["D"] * es
        entries = sum((n + p - 1) // page - p // page + 1 for n, p in zip(new, past))
        rows = min(tokens, max(n + p for n, p in zip(new, past)))
        return {"bytes": 2 * data + rows * case["R"] * es + 4 * entries + 8 * case["B"],
                "flops": 3 * tokens * case["Nkv"] * case["R"]}
    keys = pairs = entries = 0
    for n, p in zip(new, past):
        first = max(0, p - case["window"] + 1) if case["window"] > 0 else 0
        keys += n + p - first
        entries += (n + p - 1) // page - first // page + 1
        for i in range(n):
            pairs += min(p + i + 1, case["window"]) if case["window"] > 0 else p + i + 1
    D = case["D"]
    return {"bytes": 2 * keys * case["Nkv"] * D * es + 2 * tokens * case["Nq"] * D * es + 4 * entries + 8 * case["B"],
            "flops": 4 * D * pairs * case["Nq"]}


# ----------------------------------------------------------------------------------------
# The operators' definitions in 64 bits
# ----------------------------------------------------------------------------------------

def _turn(x, cos, sin, R, interleaved):
    """Each pair (a, b) of the first R channels as the complex number a + bi, times cos + i sin."""
    h = R // 2
    pairs = x[..., :R].reshape(*x.shape[:-1], h, 2) if interleaved else x[..., :R].reshape(*x.shape[:-1], 2, h).transpose(-1, -2)
    z = torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * torch.complex(cos, sin)
    out = torch.view_as_real(z)
    out = out.reshape(*x.shape[:-1], R) if interleaved else out.transpose(-1, -2).reshape(*x.shape[:-1], R)
    full = x.clone()
    full[..., :R] = out
    return full


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rotary":
        B, S, D = case["B"], case["S"], case["D"]
        cos, sin = (st[t].double()[st["pos"]][:, :, None, :] for t in ("cos", "sin"))
        res, weights = [], []
        for t in ("q", "k"):
            x = st[t].double().reshape(B, S, -1, D)
            w = st["w" + t].double()
            norm = torch.sqrt(x.square().sum(-1, keepdim=True) / D + 1e-6)
            if not case["grad"]:
                res.append(_turn(x / norm * w, cos, sin, case["R"], case["interleaved"]).reshape(B, S, -1))
                continue
            # dL/dy turned back; then d(x_i / norm)/dx_j = delta_ij / norm - x_i x_j / (D norm^3)
            g = _turn(st["dy" + t].double().reshape(B, S, -1, D), cos, -sin, case["R"], case["interleaved"])
            weights.append((g * x / norm).sum((0, 1, 2)))
            gw = g * w
            along = (gw * x).sum(-1, keepdim=True)
            res.append((gw / norm - x * along / (D * norm ** 3)).reshape(B, S, -1))
        return tuple(res + weights)
    new, past = _lengths(case)
    page, D, Nkv = case["page"], case["D"], case["Nkv"]
    table = st["table"].long().cpu()
    if case["op"] == "append":
        kp, vp = st["k_pages"].double(), st["v_pages"].double()
        k, v = st["k"].double(), st["v"].double()
        t = 0
        ids, slots, pos = [], [], []
        for b in range(case["B"]):
            for i in range(new[b]):
                p = past[b] + i
                ids.append(int(table[b, p // page]))
                slots.append(p % page)
                pos.append(p)
                t += 1
        ids, slots, pos = (torch.tensor(x, device="cuda") for x in (ids, slots, pos))
        if case["R"]:
            k = _turn(k, st["cos"].double()[pos][:, None], st["sin"].double()[pos][:, None], case["R"],
                      case["interleaved"])
        kp.permute(0, 2, 1, 3)[ids, slots] = k
        vp.permute(0, 2, 1, 3)[ids, slots] = v
        return kp, vp
    if work(case)["flops"] > 4e12:
        return None
    group = case["Nq"] // Nkv
    y = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    t0 = 0
    for b in range(case["B"]):
        n, T = new[b], new[b] + past[b]
        rows = table[b, torch.arange(T) // page].cuda()
        slot = (torch.arange(T) % page).cuda()
        for h in range(Nkv):
            K = st["k_pages"][rows, h, slot].double()
            V = st["v_pages"][rows, h, slot].double()
            for i0 in range(0, n, 512):           # bounded memory: 512 tokens at a time
                i1 = min(n, i0 + 512)
                j = torch.arange(T, device="cuda")[None, :]
                p = (past[b] + torch.arange(i0, i1, device="cuda"))[:, None]
                out_of = j > p
                if case["window"] > 0:
                    out_of |= p - j >= case["window"]
                for g in range(group):
                    hq = h * group + g
                    z = st["q"][t0 + i0:t0 + i1, hq].double() @ K.T / D ** 0.5
                    if case["softcap"] > 0:
                        z = torch.tanh(z / case["softcap"]) * case["softcap"]
                    z[out_of] = -math.inf
                    if st["sink"] is not None:
                        extra = st["sink"][hq].double().expand(i1 - i0, 1)
                        wts = torch.softmax(torch.cat((z, extra), 1), 1)[:, :T]
                    else:
                        wts = torch.softmax(z, 1)
                    y[t0 + i0:t0 + i1, hq] = wts @ V
        t0 += n
    return y
