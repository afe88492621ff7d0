"""Plain definitions of the page-table and 4-bit-cache operators, with the error each output may
carry, and seeded ragged problems.  Shares no code with the library."""
import dataclasses
import math

import torch

from paged_reference import HALF_STEP, U32, ragged

GROUP = 32


# ------------------------------------------------------------------ records

def row_bytes(D, dtype):
    return D // 2 + D // GROUP * 2 * torch.finfo(dtype).bits // 8


def codes_of(x, dtype):
    """x (..., D) of `dtype` -> integer codes (..., D/32, 32), minimum and scale (..., D/32) of `dtype`: every
    step one IEEE operation of fp32."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    spread = hi - lo
    scale = (spread / torch.tensor(15.0)).to(dtype)
    # a scale rounded up at the end of the type's range: one step down, so that code 15 has a value
    over = (lo.double() + 15 * scale.double()).float() > torch.finfo(dtype).max
    scale[over] = torch.nextafter(scale[over], torch.zeros_like(scale[over]))
    bad = ~torch.isfinite(spread)
    scale[bad], lo[bad] = float("nan"), float("nan")
    s = scale.float()[..., None]
    codes = torch.where(s > 0, torch.round((g - lo[..., None]) / s), torch.zeros_like(g)).clamp(0, 15)
    return codes.to(torch.uint8), lo.to(dtype), scale


def pack(x, dtype):
    codes, lo, scale = codes_of(x, dtype)
    c = codes.flatten(-2)
    side = torch.stack((lo, scale), -1).flatten(-2).contiguous().view(torch.uint8)
    return torch.cat((c[..., 0::2] + 16 * c[..., 1::2], side), -1)


def unpack64(rec, D, dtype):
    """Records -> (values, scale of each channel's group), float64 (..., D)."""
    b = rec[..., :D // 2].long()
    codes = torch.empty(*rec.shape[:-1], D, dtype=torch.float64)
    codes[..., 0::2], codes[..., 1::2] = (b % 16).double(), (b // 16).double()
    side = rec[..., D // 2:].contiguous().view(dtype).double()
    lo, scale = (side[..., i::2].repeat_interleave(GROUP, -1) for i in (0, 1))
    return lo + scale * codes, scale


# ------------------------------------------------------------------ ragged problems over records

def ragged4(new, past, *, tail=0.0, interleave=False, **kw):
    """-> (problem whose pools hold the records' values in float64, k records, v records, scales of v).
    Slots past a sequence's keys hold records of `tail`.  interleave: both pools are views of one tensor
    (pages, 2, heads, slots, record)."""
    r = ragged(new, past, tail=tail, slots_first=False, **kw)
    k4, v4 = pack(r.kp, r.dtype), pack(r.vp, r.dtype)
    if interleave:
        both = torch.stack((k4, v4), 1)
        k4, v4 = both[:, 0], both[:, 1]
    kd, _ = unpack64(k4, r.H, r.dtype)
    vd, vs = unpack64(v4, r.Hv, r.dtype)
    return dataclasses.replace(r, kp=kd, vp=vd), k4, v4, vs


def cuda4(t):
    """A copy on the GPU with the strides of a view into an interleaved pool."""
    if t.is_contiguous():
        return t.cuda()
    return torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)


def paged4_attn64(r, vs, *, scale=None, softcap=0.0, causal=True, window=-1, sink=None, operands="codes"):
    """-> (y, tolerance), both (tokens, Nq, Hv) float64.

    The terms of paged_attn64 (fp32 sums of H products, the exponential, T weights), and for the 16-bit
    types the operands of the value product, half a step hs of the type each:
    - operands "codes": codes are exact and a weight times its group's scale is rounded, which moves a
      term p (v - c) by hs of it, c being the value of code 8: at most 8 scales from the minimum, so by
      at most hs p 8 scale.  The scores' codes are exact.
    - operands "values": weights, values and keys are rounded: hs p |v| twice, and hs sum |q k| on a score.
    A score's sum of code products has terms as large as |q| (|k| + 16 scale); 4 times sum |q| |k|'s
    largest, taken over the row's keys, bounds it for the pools drawn here (|minimum| about 7 scales)."""
    scale = 1.0 / math.sqrt(r.H) if scale is None else scale
    group = r.Nq // r.Nkv
    hs = HALF_STEP[r.dtype]
    half = r.dtype != torch.float32
    y = torch.zeros(r.tokens, r.Nq, r.Hv, dtype=torch.float64)
    tol = torch.full_like(y, 1e-30)
    t0 = 0
    for b, n in enumerate(r.new):
        T = max(r.lens[b], 0)
        j = torch.arange(T)
        ids, at = r.table[b].long()[j // r.page], j % r.page
        K, V, S = (x.transpose(1, 2)[ids, at] for x in (r.kp, r.vp, vs))
        for i in range(n):
            pos = r.lens[b] - n + i
            lo = max(0, pos - window + 1) if window > 0 else 0
            hi = min(pos, T - 1) if causal else T - 1
            if hi < lo:
                continue
            for h in range(r.Nq):
                kk, vv, ss = (x[lo:hi + 1, h // group] for x in (K, V, S))
                qq = r.q[t0 + i, h].double()
                s = kk @ qq * scale
                mass = ((kk.abs() @ qq.abs()) * abs(scale)).max()
                ds = 4 * mass * (r.H + 4) * U32
                if half and operands == "values":
                    ds = ds + hs * mass
                if softcap > 0:
                    s = softcap * torch.tanh(s / softcap)
                    ds = ds + softcap * 2.0 ** -21
                m = s.max()
                if sink is not None:
                    m = torch.maximum(m, sink[h].double())
                p = torch.exp(s - m)
                den = p.sum() + (torch.exp(sink[h].double() - m) if sink is not None else 0.0)
                y[t0 + i, h] = p @ vv / den
                A, A8 = p @ vv.abs() / den, p @ (8 * ss) / den
                rel = 2 * ds + 2.0 ** -21 * (1 + s.abs().max()) + (hi - lo + 8) * U32
                t = hs * y[t0 + i, h].abs() + rel * (A + 2 * A8) + 1e-30
                if half:
                    t = t + (hs * A8 if operands == "codes" else 2 * hs * A)
                if r.dtype == torch.float16:
                    t = t + 2.0 ** -25           # half of the smallest subnormal step
                tol[t0 + i, h] = t
        t0 += n
    return y, tol


# ------------------------------------------------------------------ page tables

def tables_of(table, past, new, free, count, page, tokens):
    """The operator on Python lists, one sequence, page and token at a time: -> dict of its outputs and
    the words that its reports hold."""
    table, free, said = [list(r) for r in table], list(free), set()
    pages, width = len(free), len(table[0]) if table else 0
    if count > pages:
        said.add("cu_new")
    top = min(max(count, 0), pages)
    held, brought = [], []
    room = tokens
    for p, n in zip(past, new):
        q = min(max(p, 0), width * page)
        m = 0 if n < 0 else min(n, width * page - q, room)
        if q != p or (n >= 0 and m != n):
            said.add("cu_new")
        room -= m
        held.append(q)
        brought.append(m)
    for b, n in enumerate(new):
        if n < 0:
            for i in range(-(-held[b] // page)):
                if 0 <= table[b][i] < pages:
                    if top < pages:
                        free[top] = table[b][i]
                        top += 1
                    else:
                        said.add("cu_new")
                else:
                    said.add("page id")
    lens, cu, positions, slots = [], [0], [], []
    for b, n in enumerate(new):
        T = 0 if n < 0 else held[b] + brought[b]
        for i in range(-(-held[b] // page), -(-T // page)):
            top -= 1
            table[b][i] = free[top] if top >= 0 else -1
            if top < 0:
                said.add("ran out")
            elif not 0 <= table[b][i] < pages:
                table[b][i] = -1
                said.add("page id")
        for pos in range(held[b], held[b] + brought[b]):
            positions.append(pos)
            ok = 0 <= table[b][pos // page] < pages
            slots.append(table[b][pos // page] * page + pos % page if ok else -1)
            if not ok and pos // page < -(-held[b] // page):
                said.add("page id")
        lens.append(T)
        cu.append(cu[-1] + brought[b])
    positions += [0] * (tokens - len(positions))
    slots += [-1] * (tokens - len(slots))
    return dict(kv_lens=lens, cu_new=cu, positions=positions, slots=slots, free_count_out=[top], page_table=table,
                free_pages=free), said
