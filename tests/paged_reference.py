"""Plain 64-bit definitions of the paged-cache and query/key-norm operators, with the error each
output may carry, and seeded ragged problems.  Shares no code with the library."""
import dataclasses
import math
from typing import Optional

import torch

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.float16, torch.bfloat16)}
U32 = 2.0 ** -24                      # half a step of fp32


# ------------------------------------------------------------------ norm and rotation

def rotate64(x, cos, sin, R, interleaved):
    """x (..., D) float64, cos / sin (..., R/2): pairs (d, d + R/2) or (2d, 2d + 1) turned."""
    y = x.clone()
    i1 = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    i2 = i1 + 1 if interleaved else i1 + R // 2
    y[..., i1] = x[..., i1] * cos - x[..., i2] * sin
    y[..., i2] = x[..., i2] * cos + x[..., i1] * sin
    return y


def pair_abs(x, R, interleaved):
    """|x1| + |x2| of each channel's pair; |x| where nothing is rotated."""
    y = x.abs()
    i1 = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    i2 = i1 + 1 if interleaved else i1 + R // 2
    s = y[..., i1] + y[..., i2]
    y[..., i1], y[..., i2] = s, s
    return y


def norm_rotary64(x, w, cos, sin, R, interleaved, eps):
    """x (B, N, S, D), w (D), cos / sin (B, S, R/2) float64 -> (y, magnitude of its terms)."""
    u = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if R == 0:
        return u, u.abs()
    return rotate64(u, cos[:, None], sin[:, None], R, interleaved), pair_abs(u, R, interleaved)


def norm_rotary_grad64(x, w, dy, cos, sin, R, interleaved, eps):
    """-> (dx, dw, magnitude of dx's terms, sum of |terms| of dw)."""
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    g, ga = dy, dy.abs()
    if R:
        g = rotate64(dy, cos[:, None], -sin[:, None], R, interleaved)
        ga = pair_abs(dy, R, interleaved)
    gw, gwa = g * w, ga * w.abs()
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    mag = r * (gwa + xh.abs() * (gwa * xh.abs()).mean(-1, keepdim=True))
    return dx, (g * xh).sum((0, 1, 2)), mag, (ga * xh.abs()).sum((0, 1, 2))


# ------------------------------------------------------------------ ragged problems

@dataclasses.dataclass
class Ragged:
    dtype: torch.dtype
    new: list
    lens: list
    Nq: int
    Nkv: int
    H: int
    Hv: int
    page: int
    q: torch.Tensor                     # (tokens + extra, Nq, H)
    k: torch.Tensor
    v: torch.Tensor
    kp: torch.Tensor                    # (pages, Nkv, slots, dim) views
    vp: torch.Tensor
    table: torch.Tensor
    cu: Optional[torch.Tensor]
    kv_lens: torch.Tensor

    def to(self, dev):
        kw = {f.name: getattr(self, f.name) for f in dataclasses.fields(self)}
        for n, t in kw.items():
            if isinstance(t, torch.Tensor):
                m = t.to(dev)
                if n in ("kp", "vp") and t.stride() != m.stride():
                    m = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=dev).copy_(t)
                kw[n] = m
        return Ragged(**kw)

    @property
    def tokens(self):
        return sum(self.new)


def ragged(new, past, *, dtype=torch.bfloat16, Nq=4, Nkv=2, H=64, Hv=None, page=16, slots_first=True, interleave=False,
           uniform=False, extra_rows=0, extra_width=2, tail=float("nan"), seed=0):
    """past[b] may be negative (fewer keys than new tokens).  Slots past a sequence's keys and
    pages no sequence uses hold `tail`."""
    Hv = H if Hv is None else Hv
    g = torch.Generator().manual_seed(seed)
    lens = [n + p for n, p in zip(new, past)]
    need = [(max(t, 0) + page - 1) // page for t in lens]
    width = max(need + [0]) + extra_width
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((len(new), width), -7, dtype=torch.int32)
    at = 0
    kd, vd = (torch.full((pool, page, Nkv, d), tail).to(dtype) for d in (H, Hv))
    for b, c in enumerate(need):
        table[b, :c] = order[at:at + c]
        at += c
        for i in range(c):
            n = min(page, lens[b] - i * page)
            kd[table[b, i], :n] = torch.randn(n, Nkv, H, generator=g).to(dtype)
            vd[table[b, i], :n] = torch.randn(n, Nkv, Hv, generator=g).to(dtype)
    if interleave:                       # one pool (pages, 2, slots, heads, dim) holds both
        assert H == Hv
        both = torch.stack((kd, vd), 1)
        kp, vp = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    elif slots_first:
        kp, vp = kd.transpose(1, 2), vd.transpose(1, 2)
    else:
        kp, vp = kd.transpose(1, 2).contiguous(), vd.transpose(1, 2).contiguous()
    tokens = sum(new) + extra_rows
    q = torch.randn(tokens, Nq, H, generator=g).to(dtype)
    k = torch.randn(tokens, Nkv, H, generator=g).to(dtype)
    v = torch.randn(tokens, Nkv, Hv, generator=g).to(dtype)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return Ragged(dtype, list(new), lens, Nq, Nkv, H, Hv, page, q, k, v, kp, vp, table,
                  None if uniform else torch.tensor(cu, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32))


def gather64(r: Ragged, b: int):
    """Keys and values of sequence b, (T, Nkv, dim) float64."""
    T = max(r.lens[b], 0)
    j = torch.arange(T)
    ids, slots = r.table[b].long()[j // r.page], j % r.page
    return r.kp.transpose(1, 2)[ids, slots].double(), r.vp.transpose(1, 2)[ids, slots].double()


def paged_attn64(r: Ragged, *, scale=None, softcap=0.0, causal=True, window=-1, sink=None):
    """-> (y, tolerance), both (tokens, Nq, Hv) float64.

    Tolerance, term by term: the output is rounded once to its type (half a step of |y|); the
    weights enter the value products rounded to a 16-bit type (half a step each, so at most half
    a step of A = sum p |v|); the scores are fp32 sums of H products, off by
    (H + 4) U32 sum |q k| scale, which moves a weight and the sum by that much relatively, and a
    softcap shrinks it; log2 e and the exponential add about 2^-21 of the exponent's size; the
    fp32 sums of T weights and T products add T U32 of A."""
    scale = 1.0 / math.sqrt(r.H) if scale is None else scale
    group = r.Nq // r.Nkv
    hs = HALF_STEP[r.dtype]
    y = torch.zeros(r.tokens, r.Nq, r.Hv, dtype=torch.float64)
    tol = torch.full_like(y, 1e-30)
    t0 = 0
    for b, n in enumerate(r.new):
        K, V = gather64(r, b)
        T = K.shape[0]
        for i in range(n):
            pos = r.lens[b] - n + i
            lo = max(0, pos - window + 1) if window > 0 else 0
            hi = min(pos, T - 1) if causal else T - 1
            if hi < lo:
                continue
            for h in range(r.Nq):
                kk, vv = K[lo:hi + 1, h // group], V[lo:hi + 1, h // group]
                qq = r.q[t0 + i, h].double()
                s = kk @ qq * scale
                ds = ((kk.abs() @ qq.abs()) * abs(scale)).max() * (r.H + 4) * U32
                if softcap > 0:
                    s = softcap * torch.tanh(s / softcap)
                    ds = ds + softcap * 2.0 ** -21
                m = s.max()
                if sink is not None:
                    m = torch.maximum(m, sink[h].double())
                p = torch.exp(s - m)
                den = p.sum() + (torch.exp(sink[h].double() - m) if sink is not None else 0.0)
                y[t0 + i, h] = p @ vv / den
                A = p @ vv.abs() / den
                rel = 2 * ds + 2.0 ** -21 * (1 + s.abs().max()) + (hi - lo + 8) * U32
                if r.dtype != torch.float32:
                    rel = rel + hs
                tol[t0 + i, h] = hs * y[t0 + i, h].abs() + rel * A + 1e-30
                if r.dtype == torch.float16:
                    tol[t0 + i, h] += 2.0 ** -25      # half of the smallest subnormal step
        t0 += n
    return y, tol


# ------------------------------------------------------------------ gradients by differences

def slope64(f, h):
    """f'(0) of a smooth float64 function by central differences at h, h/2 and h/4, extrapolated twice
    over (their h^2 terms cancel), and a bound of its error: what the finer extrapolation still changed,
    which is about 16 times the error left, beside the rounding of the differences."""
    d = [(f(s) - f(-s)) / (2 * s) for s in (h, h / 2, h / 4)]
    coarse, fine = (4 * d[1] - d[0]) / 3, (4 * d[2] - d[1]) / 3
    return fine, abs(fine - coarse) + 2.0 ** -44 * max(abs(f(h)), abs(f(-h))) / h


def norm_slope_check(d, name, grads, cos, sin, R, interleaved, eps, seed):
    """The gradient of sum(q_out dq_out) + sum(k_out dk_out) along a direction of -1, 0 and 1 in
    d[name] against differences of the float64 forward: -> (error, tolerance).  d: rank-4 problem;
    grads[name]: the gradient in question.  The tolerance takes nothing from it: the slope's own
    bound, and fp32 arithmetic's error of each element (the sums of test_backward's bounds)."""
    gen = torch.Generator().manual_seed(seed)
    t = name[0]
    direction = torch.randint(-1, 2, d[name].shape, generator=gen).double()
    x, w, dy = d[t].double(), d[t + "_weight"].double(), d["d" + t + "_out"].double()

    def loss(step):
        at = {name: d[name].double() + step * direction}
        y, _ = norm_rotary64(at.get(t, x), at.get(t + "_weight", w), cos, sin, R, interleaved, eps)
        return (y * dy).sum().item()

    truth, tol = slope64(loss, 2.0 ** -6)
    dx, dw, mag, wsum = norm_rotary_grad64(x, w, dy, cos, sin, R, interleaved, eps)
    hs = HALF_STEP[d[name].dtype]
    each = hs * dx.abs() + 64 * U32 * mag if name == t else hs * dw.abs() + (x[..., 0].numel() + 64) * U32 * wsum
    inner = (grads[name].cpu().double() * direction).sum().item()
    return abs(inner - truth), tol + (each * direction.abs()).sum().item()
