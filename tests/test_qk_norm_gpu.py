"""The query/key norm with the rotation in the same pass, and its gradient, against float64.

Bounds.  The kernels work in fp32 and round once.  The sum of squares has at most 16 terms in a
row and five shuffle additions (all positive), so r is off by at most (21 / 2 + 4) U32 with the
reciprocal root; scaling, weight and rotation add at most six roundings of |u1| + |u2|: 24 U32 in
all.  The gradient's terms pass the rotation, the weight, a sum of D products and r: 64 U32 of the
magnitudes of its terms.  A weight's gradient sums one product per row: rows + 32 roundings of the
sum of the terms' magnitudes.
"""
import pytest
import torch

from paged_reference import HALF_STEP, U32, norm_rotary64, norm_rotary_grad64, norm_slope_check
from scaled_dot_product_gb300 import sdpa
from scaled_dot_product_gb300.workloads import rope_caches

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def draw(B, S, Nq, Nkv, D, dtype, rank, R, cache, seed=0, grad=False):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype)
    shape = (lambda N: (B, S, N * D)) if rank == 3 else (lambda N: (B, N, S, D))
    d = dict(q=rn(*shape(Nq)), k=rn(*shape(Nkv)), q_weight=(1 + 0.3 * torch.randn(D, generator=g)).to(dtype),
             k_weight=(1 + 0.3 * torch.randn(D, generator=g)).to(dtype))
    if grad:
        d.update(dq_out=rn(*shape(Nq)), dk_out=rn(*shape(Nkv)))
    if R:
        if cache == "ids":
            rows = 2 * S + 9
            d["cos_cache"], d["sin_cache"] = rope_caches(rows, R // 2, dtype)
            d["position_ids"] = torch.randint(0, rows, (B, S), generator=g)
        else:
            c, s = rope_caches(B * S, R // 2, dtype)
            d["cos_cache"], d["sin_cache"] = c.view(B, S, -1), s.view(B, S, -1)
    return d


def heads(t, N):
    return t if t.dim() == 4 else t.view(t.shape[0], t.shape[1], N, -1).permute(0, 2, 1, 3)


def tables(d):
    if "cos_cache" not in d:
        return None, None
    c, s = d["cos_cache"].double(), d["sin_cache"].double()
    return (c[d["position_ids"]], s[d["position_ids"]]) if "position_ids" in d else (c, s)


# B, S, Nq, Nkv, D, dtype, rank, R, interleaved, cache
SHAPES = [
    (2, 5, 4, 2, 64, BF, 3, 64, False, "ids"),
    (1, 1, 1, 1, 128, BF, 4, 128, False, "ids"),
    (3, 7, 5, 3, 128, HF, 3, 64, False, "token"),       # partial rotation, odd head counts
    (2, 9, 6, 1, 64, HF, 4, 32, True, "ids"),
    (1, 33, 9, 3, 128, BF, 3, 128, True, "token"),
    (2, 3, 2, 2, 256, BF, 4, 256, False, "ids"),
    (2, 3, 3, 1, 256, FP, 3, 128, True, "ids"),
    (1, 17, 4, 4, 64, FP, 3, 64, False, "ids"),
    (2, 5, 3, 2, 80, BF, 3, 80, False, "ids"),          # 16-byte vectors, no power of two
    (2, 5, 3, 2, 96, HF, 3, 20, False, "ids"),          # a half that is no vector: scalar
    (1, 6, 2, 1, 50, BF, 3, 50, False, "ids"),          # odd head size: scalar
    (1, 6, 2, 1, 7, FP, 4, 6, True, "ids"),
    (1, 6, 2, 2, 1, HF, 4, 0, False, "ids"),            # one channel, no rotation
    (2, 5, 4, 2, 128, BF, 3, 0, False, "ids"),          # norm alone
    (2, 700, 16, 4, 128, BF, 3, 128, False, "ids"),     # several heads per lane group
    (1, 2001, 24, 3, 64, HF, 3, 64, True, "ids"),
]


@pytest.mark.parametrize("B,S,Nq,Nkv,D,dtype,rank,R,inter,cache", SHAPES)
def test_forward(B, S, Nq, Nkv, D, dtype, rank, R, inter, cache):
    d = draw(B, S, Nq, Nkv, D, dtype, rank, R, cache)
    got = sdpa.sdpa_qk_norm_rotary(**{n: t.cuda() for n, t in d.items()}, rotary_dim=R, interleaved=inter,
                                   num_heads=Nq, kv_num_heads=Nkv, eps=1e-5)
    assert sdpa.sdpa_query_status() == 0
    cos, sin = tables(d)
    for t, w, N, out in (("q", "q_weight", Nq, got[0]), ("k", "k_weight", Nkv, got[1])):
        want, mag = norm_rotary64(heads(d[t], N).double(), d[w].double(), cos, sin, R, inter, 1e-5)
        err = (heads(out.cpu(), N).double() - want).abs()
        tol = HALF_STEP[dtype] * want.abs() + 24 * U32 * mag + (2.0 ** -25 if dtype == HF else 1e-38)
        assert (err <= tol).all(), (t, (err / tol).max())


@pytest.mark.parametrize("B,S,Nq,Nkv,D,dtype,rank,R,inter,cache", SHAPES)
def test_backward(B, S, Nq, Nkv, D, dtype, rank, R, inter, cache):
    d = draw(B, S, Nq, Nkv, D, dtype, rank, R, cache, grad=True)
    g = {n: t.cuda() for n, t in d.items()}
    kw = dict(rotary_dim=R, interleaved=inter, num_heads=Nq, kv_num_heads=Nkv, eps=1e-5)
    dq, dk, dwq, dwk = sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw)
    assert sdpa.sdpa_query_status() == 0
    cos, sin = tables(d)
    for t, w, N, dx, dw in (("q", "q_weight", Nq, dq, dwq), ("k", "k_weight", Nkv, dk, dwk)):
        wx, ww, mag, wsum = norm_rotary_grad64(heads(d[t], N).double(), d[w].double(), heads(d["d" + t + "_out"], N).double(),
                                               cos, sin, R, inter, 1e-5)
        err = (heads(dx.cpu(), N).double() - wx).abs()
        tol = HALF_STEP[dtype] * wx.abs() + 64 * U32 * mag + (2.0 ** -25 if dtype == HF else 1e-38)
        assert (err <= tol).all(), (t, (err / tol).max())
        err = (dw.cpu().double() - ww).abs()
        tol = HALF_STEP[dtype] * ww.abs() + (B * S * N + 64) * U32 * wsum
        assert (err <= tol).all(), (w, (err / tol).max())
    again = sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))      # a fixed order of sums


def test_gradient_against_differences():
    """Central differences of the kernel's own fp32 forward along random directions.  Their
    truncation error is that of the float64 formula at the same step; the forward's rounding
    enters as 24 U32 of the magnitudes over the step."""
    B, S, Nq, Nkv, D, R, h = 1, 4, 2, 1, 64, 64, 2.0 ** -6
    d = draw(B, S, Nq, Nkv, D, FP, 4, R, "ids", seed=3, grad=True)
    kw = dict(rotary_dim=R, eps=1e-5)
    g = {n: t.cuda() for n, t in d.items()}
    dq, dk, dwq, dwk = sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw)
    fw = {n: t for n, t in d.items() if not n.startswith("d")}
    cos, sin = tables(d)
    gen = torch.Generator().manual_seed(9)
    for name, grad in (("q", dq), ("k", dk), ("q_weight", dwq), ("k_weight", dwk)):
        # a direction of multiples of 2^-6: x + h dir is then rounded by at most U32 |x|
        direction = torch.randint(-1, 2, d[name].shape, generator=gen).float()

        def loss(sign, f64):
            p = dict(fw)
            p[name] = d[name] + sign * h * direction
            if f64:
                out = [norm_rotary64(p[t].double(), p[t + "_weight"].double(), cos, sin, R, False, 1e-5) for t in ("q", "k")]
                return sum((y * d["d" + t + "_out"].double()).sum() for t, (y, _) in zip("qk", out)), \
                    sum((m * d["d" + t + "_out"].double().abs()).sum() for t, (_, m) in zip("qk", out))
            y = sdpa.sdpa_qk_norm_rotary(**{n: t.cuda() for n, t in p.items()}, **kw)
            return sum((o.cpu().double() * d["d" + t + "_out"].double()).sum() for t, o in zip("qk", y)), None

        (lp, mag), (lm, _) = loss(1, True), loss(-1, True)
        kp, km = loss(1, False)[0], loss(-1, False)[0]
        inner = (grad.cpu().double() * direction.double()).sum()
        truth = (lp - lm) / (2 * h)
        tol = (truth - inner).abs() + 26 * U32 * mag / h        # truncation + rounding of both sides
        assert (truth - inner).abs() <= 0.02 * grad.abs().sum().item()           # the step is small enough to tell
        assert ((kp - km) / (2 * h) - inner).abs() <= tol, name


def test_in_place_and_strided_views():
    """Outputs over their inputs; heads sliced out of one packed projection (16-byte aligned and
    not)."""
    for off in (0, 2):
        B, S, Nq, Nkv, D = 2, 6, 4, 2, 64
        g = torch.Generator().manual_seed(1)
        packed = torch.randn(B, S, (Nq + 2 * Nkv) * D + 8, generator=g).to(BF).cuda()
        q = packed[..., off:off + Nq * D].unflatten(-1, (Nq, D)).transpose(1, 2)
        k = packed[..., off + Nq * D:off + (Nq + Nkv) * D].unflatten(-1, (Nkv, D)).transpose(1, 2)
        w = torch.rand(2, D, generator=g).to(BF).cuda()
        c, s = (t.cuda() for t in rope_caches(S + 3, D // 2, BF))
        pos = torch.arange(S, device="cuda").expand(B, S)
        before = packed.clone()
        want = sdpa.sdpa_qk_norm_rotary(q.contiguous(), k.contiguous(), w[0], w[1], c, s, pos)
        sdpa.sdpa_qk_norm_rotary(q, k, w[0], w[1], c, s, pos, q_out=q, k_out=k)
        # both kernels round once from fp32 sums that may differ in their last bits
        for a, b in zip((q, k), want):
            assert ((a.float() - b.float()).abs() <= torch.finfo(BF).eps * b.float().abs() + 1e-6).all()
        rest = torch.ones(packed.shape[-1], dtype=torch.bool)
        rest[off:off + (Nq + Nkv) * D] = False
        assert torch.equal(packed[..., rest], before[..., rest])
        dy = torch.randn(B, Nq, S, D, generator=g).to(BF).cuda(), torch.randn(B, Nkv, S, D, generator=g).to(BF).cuda()
        want = sdpa.sdpa_qk_norm_rotary_bwd(q, k, *dy, w[0], w[1], c, s, pos)
        got = sdpa.sdpa_qk_norm_rotary_bwd(q, k, *dy, w[0], w[1], c, s, pos, dq=dy[0], dk=dy[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and got[0] is dy[0]


def test_zero_rows_and_empty_batches():
    z = torch.zeros(1, 2, 3, 64, dtype=BF, device="cuda")
    w = torch.ones(64, dtype=BF, device="cuda")
    q, k = sdpa.sdpa_qk_norm_rotary(z, z.clone(), w, w)
    assert not q.any() and not k.any()
    e = torch.empty(2, 2, 0, 64, dtype=BF, device="cuda")
    q, k = sdpa.sdpa_qk_norm_rotary(e, e.clone(), w, w)
    assert q.shape == e.shape
    dw = torch.full((2, 64), 5.0, dtype=BF, device="cuda")
    sdpa.sdpa_qk_norm_rotary_bwd(e, e.clone(), e.clone(), e.clone(), w, w, dq_weight=dw[0], dk_weight=dw[1])
    assert not dw.any()                   # the sum over no rows


def test_positions_outside_the_cache_are_reported():
    q = torch.randn(1, 1, 2, 64, device="cuda").to(HF)
    w = torch.ones(64, dtype=HF, device="cuda")
    c, s = (t.cuda() for t in rope_caches(4, 32, HF))
    for bad in (4, -1):
        sdpa.sdpa_qk_norm_rotary(q, q.clone(), w, w, c, s, torch.tensor([[0, bad]], device="cuda"))
        assert sdpa.sdpa_query_status() == sdpa.SDPA_ERR_INVALID
        assert sdpa.sdpa_query_status() == 0


def test_other_stream_and_graph_replay():
    d = draw(2, 5, 4, 2, 64, BF, 3, 64, "ids", grad=True)
    g = {n: t.cuda() for n, t in d.items()}
    f = {n: t for n, t in g.items() if not n.startswith("d")}
    kw = dict(num_heads=4, kv_num_heads=2)
    want, wantb = sdpa.sdpa_qk_norm_rotary(**f, **kw), sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got, gotb = sdpa.sdpa_qk_norm_rotary(**f, **kw, stream=st), sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw, stream=st.cuda_stream)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gotb, want + wantb))
    # positions of another type, written late on the call's stream, are converted behind that write
    late = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for handle in (st, st.cuda_stream):
        late.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(20):
                busy = (busy @ busy).clamp_(-1, 1)
            late.copy_(g["position_ids"])
        got = sdpa.sdpa_qk_norm_rotary(**{**f, "position_ids": late}, **kw, stream=handle)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, gotb = sdpa.sdpa_qk_norm_rotary(**f, **kw), sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw)
    g["q"].neg_()                         # odd in x: outputs and weight gradients change sign
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], -want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(gotb[0], wantb[0]) and torch.equal(gotb[2], -wantb[2]) and torch.equal(gotb[3], wantb[3])


@pytest.mark.parametrize("Nq,Nkv,D,dtype,S", [(1, 700, 128, BF, 70), (700, 1, 64, HF, 40), (1, 2000, 50, BF, 3), (1, 900, 256, FP, 9)])
def test_gradient_of_very_unequal_head_counts(Nq, Nkv, D, dtype, S):
    """One side has nearly all the rows: the partial sums stay within a workspace of exactly the size
    asked for."""
    import ctypes
    d = draw(1, S, Nq, Nkv, D, dtype, 4, 0, "ids", seed=5, grad=True)
    g = {n: t.cuda() for n, t in d.items()}
    p = sdpa.sdpa_qk_norm_params(struct_size=ctypes.sizeof(sdpa.sdpa_qk_norm_params), B=1, Nq=Nq, Nkv=Nkv, S=S, D=D,
                                 dtype=sdpa._DTYPES[dtype], q=sdpa._view(g["q"], []), k=sdpa._view(g["k"], []),
                                 q_weight=g["q_weight"].data_ptr(), k_weight=g["k_weight"].data_ptr(), eps=1e-5)
    need = sdpa.lib().sdpa_qk_norm_workspace_size(ctypes.byref(p))
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    dq, dk, dwq, dwk = sdpa.sdpa_qk_norm_rotary_bwd(**g, eps=1e-5, workspace=room[:need])
    assert (room[need:] == 0xA5).all() and sdpa.sdpa_query_status() == 0
    for t, N, dx, dw in (("q", Nq, dq, dwq), ("k", Nkv, dk, dwk)):
        wx, ww, mag, wsum = norm_rotary_grad64(d[t].double(), d[t + "_weight"].double(), d["d" + t + "_out"].double(), None, None,
                                               0, False, 1e-5)
        assert ((dx.cpu().double() - wx).abs() <= HALF_STEP[dtype] * wx.abs() + 64 * U32 * mag + (2.0 ** -25 if dtype == HF else 0)).all()
        assert ((dw.cpu().double() - ww).abs() <= HALF_STEP[dtype] * ww.abs() + (S * N + 64) * U32 * wsum).all()


@pytest.mark.parametrize("rank", [3, 4])
def test_empty_batches_with_a_cache_row_per_token(rank):
    full = draw(2, 5, 4, 2, 64, BF, rank, 64, "token", grad=True)
    no_token = lambda t: t if t.dim() == 1 else t[:, :, :0] if t.dim() == 4 else t[:, :0]
    no_batch = lambda t: t if t.dim() == 1 else t[:0]
    for cut in (no_token, no_batch):
        g = {n: cut(t).cuda() for n, t in full.items()}
        f = {n: t for n, t in g.items() if not n.startswith("d")}
        kw = dict(num_heads=4, kv_num_heads=2, rotary_dim=64)
        q, k = sdpa.sdpa_qk_norm_rotary(**f, **kw)
        assert q.shape == g["q"].shape and k.shape == g["k"].shape
        dq, dk, dwq, dwk = sdpa.sdpa_qk_norm_rotary_bwd(**g, **kw)
        assert dq.shape == g["q"].shape and not dwq.any() and not dwk.any()      # sums over no rows
        assert sdpa.sdpa_query_status() == 0


@pytest.mark.parametrize("dtype,D,R,inter", [(FP, 64, 64, False), (FP, 128, 32, True), (FP, 50, 50, False), (FP, 256, 0, False),
                                             (BF, 128, 128, False), (HF, 64, 64, True)])
def test_gradient_against_differences_of_the_definition(dtype, D, R, inter):
    """Along random directions, within a bound that takes nothing from the gradient under test (the CPU
    tests show that a gradient without its mean term is well outside it)."""
    d = draw(1, 4, 2, 1, D, dtype, 4, R, "ids", seed=3, grad=True)
    out = sdpa.sdpa_qk_norm_rotary_bwd(**{n: t.cuda() for n, t in d.items()}, rotary_dim=R, interleaved=inter, eps=1e-5)
    grads = dict(zip(("q", "k", "q_weight", "k_weight"), out))
    cos, sin = tables(d)
    for name in grads:
        for seed in range(4):
            err, tol = norm_slope_check(d, name, grads, cos, sin, R, inter, 1e-5, seed)
            assert err <= tol, (name, err, tol)
