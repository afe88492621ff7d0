"""Argument checks of the query/key norm, the paged append and the paged attention: what the C
entry points refuse before any launch, and what the binding refuses."""
import ctypes

import pytest
import torch

from paged_reference import norm_rotary64, norm_rotary_grad64, norm_slope_check, rotate64
from scaled_dot_product_gb300 import sdpa

BF = torch.bfloat16
V = sdpa._view


def accepted(call):
    """The call passes every check.  Made only where there is no GPU to launch it on: its tensors
    are host memory."""
    return torch.cuda.is_available() or call() == sdpa.SDPA_ERR_CUDA


def norm(over=(), *, B=2, S=3, Nq=4, Nkv=2, D=64, dtype=BF, R=64, ids=True):
    z = lambda *s: torch.zeros(*s, dtype=dtype)
    q, k = z(B, Nq, S, D), z(B, Nkv, S, D)
    rot = (z(10, R // 2), z(10, R // 2), torch.zeros(B, S, dtype=torch.int64)) if R else (None, None, None)
    if R and not ids:
        rot = (z(B, S, R // 2), z(B, S, R // 2), None)
    # CPU tensors: the struct only carries their addresses
    p, q, k, keep = _norm_struct(q, k, z(D), z(D), *rot, R)
    for n, v in dict(over).items():
        setattr(p, n, v)
    return p, q, k, keep


def _norm_struct(q, k, qw, kw, cos, sin, pos, R):
    keep = [q, k, qw, kw, cos, sin, pos]
    p = sdpa.sdpa_qk_norm_params()
    p.struct_size = ctypes.sizeof(p)
    p.B, p.Nq, p.S, p.D = q.shape
    p.Nkv = k.shape[1]
    p.dtype = sdpa._DTYPES[q.dtype]
    p.q, p.k = V(q, keep), V(k, keep)
    p.q_weight, p.k_weight, p.eps = qw.data_ptr(), kw.data_ptr(), 1e-6
    if cos is not None:
        p.rotary_cos, p.rotary_sin, p.rotary_dim = cos.data_ptr(), sin.data_ptr(), R
        p.rotary_max_pos = cos.shape[0] if pos is not None else cos.shape[0] * cos.shape[1]
        p.position_ids = None if pos is None else pos.data_ptr()
    return p, q, k, keep


def norm_code(p, q, k, keep, q_out=None, k_out=None):
    q_out = torch.zeros_like(q) if q_out is None else q_out
    k_out = torch.zeros_like(k) if k_out is None else k_out
    return sdpa.lib().sdpa_qk_norm_rotary(ctypes.byref(p), V(q_out, keep), V(k_out, keep), None)


NORM_BAD = [
    (dict(struct_size=4), "INVALID"), (dict(dtype=7), "INVALID"), (dict(B=-1), "SHAPE"), (dict(Nkv=0), "SHAPE"),
    (dict(D=257), "UNSUPPORTED"), (dict(eps=-1.0), "INVALID"), (dict(eps=float("nan")), "INVALID"),
    (dict(q_weight=None), "NULL"), (dict(k_weight=None), "NULL"), (dict(rotary_sin=None), "INVALID"),
    (dict(rotary_dim=63), "INVALID"), (dict(rotary_dim=66), "INVALID"), (dict(rotary_interleaved=2), "INVALID"),
    (dict(rotary_max_pos=0), "SHAPE"), (dict(rotary_cos=None, rotary_sin=None), "NULL"), (dict(position_ids=12), "ALIGNMENT"),
    (dict(B=1 << 16, S=1 << 16), "OVERFLOW"), (dict(q=sdpa.sdpa_view(None, 1, 1, 1)), "NULL"),
    (dict(q=sdpa.sdpa_view(256, -8, 64, 64)), "INVALID"), (dict(q=sdpa.sdpa_view(257, 768, 192, 64)), "ALIGNMENT"),
]


@pytest.mark.parametrize("change,why", NORM_BAD)
def test_norm_refusals(change, why):
    assert norm_code(*norm(change)) == getattr(sdpa, "SDPA_ERR_" + why), sdpa.sdpa_last_error()


def test_norm_per_token_caches_need_a_row_per_token():
    assert norm_code(*norm(dict(rotary_max_pos=7), ids=False)) == sdpa.SDPA_ERR_SHAPE


def test_norm_aliases():
    p, q, k, keep = norm()
    assert accepted(lambda: norm_code(p, q, k, keep, q_out=q, k_out=k))       # in place
    assert norm_code(p, q, k, keep, k_out=q[:, :2]) == sdpa.SDPA_ERR_ALIAS
    both = torch.zeros(2, 4, 3, 64, dtype=BF)
    assert norm_code(p, q, k, keep, q_out=both, k_out=both[:, :2]) == sdpa.SDPA_ERR_ALIAS
    # heads of one packed projection interleave without sharing an element
    packed = torch.zeros(2, 3, 6 * 64, dtype=BF)
    qs, ks = packed[..., :256].unflatten(-1, (4, 64)).transpose(1, 2), packed[..., 256:].unflatten(-1, (2, 64)).transpose(1, 2)
    assert accepted(lambda: norm_code(p, q, k, keep, q_out=qs, k_out=ks)), sdpa.sdpa_last_error()
    ks = packed[..., 192:320].unflatten(-1, (2, 64)).transpose(1, 2)
    assert norm_code(p, q, k, keep, q_out=qs, k_out=ks) == sdpa.SDPA_ERR_ALIAS


def test_norm_backward_refusals():
    p, q, k, keep = norm()
    need = sdpa.lib().sdpa_qk_norm_workspace_size(ctypes.byref(p))
    assert need > 0
    ws = torch.zeros(need + 512, dtype=torch.uint8)
    at = (ws.data_ptr() + 255) & ~255
    z = torch.zeros_like
    w = torch.zeros(2, 64, dtype=BF)

    def code(dyq=None, dyk=None, dq=None, dk=None, dwq=w[0], dwk=w[1], where=at, size=need):
        ts = [z(q) if dyq is None else dyq, z(k) if dyk is None else dyk, z(q) if dq is None else dq, z(k) if dk is None else dk]
        ptr = lambda t: None if t is None else t.data_ptr()
        return sdpa.lib().sdpa_qk_norm_rotary_bwd(ctypes.byref(p), *[V(t, keep) for t in ts], ptr(dwq), ptr(dwk), where, size,
                                                  None)

    assert code(dwq=None) == sdpa.SDPA_ERR_NULL
    assert code(size=need - 1) == sdpa.SDPA_ERR_WORKSPACE and code(where=None) == sdpa.SDPA_ERR_WORKSPACE
    assert code(where=at + 16) == sdpa.SDPA_ERR_ALIGNMENT
    assert code(dq=q) == sdpa.SDPA_ERR_ALIAS
    assert code(dwq=w[0], dwk=w[0]) == sdpa.SDPA_ERR_ALIAS
    p.q_weight, kept = at + 128, p.q_weight              # the sums of the weights' gradients would overwrite it
    assert code() == sdpa.SDPA_ERR_ALIAS and "q_weight" in sdpa.sdpa_last_error()
    p.q_weight = kept
    both = torch.zeros_like(q)
    assert accepted(lambda: code(dyq=both, dq=both))
    bad, _, _, keep2 = norm(dict(eps=-1.0))
    assert sdpa.lib().sdpa_qk_norm_workspace_size(ctypes.byref(bad)) == 0 and "eps" in sdpa.sdpa_last_error()


def paged(over=(), *, B=2, tokens=4, Nq=4, Nkv=2, H=64, Hv=64, pages=6, page=16, width=3, dtype=BF):
    z = lambda *s: torch.zeros(*s, dtype=dtype)
    kp, vp = z(pages, Nkv, page, H), z(pages, Nkv, page, Hv)
    table, lens = torch.zeros(B, width, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    p, keep = sdpa.make_paged_params(kp, vp, table, lens, tokens, Nq, cu_new=cu), [lens, cu]
    for n, v in dict(over).items():
        setattr(p, n, v)
    rows = dict(q=z(tokens, Nq, H), k=z(tokens, Nkv, H), v=z(tokens, Nkv, Hv), y=z(tokens, Nq, Hv), kp=kp, vp=vp, table=table)
    return p, rows, keep


def packed(t):
    """The C view of packed rows (tokens, heads, dim)."""
    return sdpa.sdpa_view(t.data_ptr(), 0, t.stride(1), t.stride(0))


def append_code(p, rows, keep, **over):
    t = dict(rows, **over)
    return sdpa.lib().sdpa_paged_append(ctypes.byref(p), packed(t["k"]), packed(t["v"]), None)


def attn_code(p, rows, keep, where=256, size=1 << 40, **over):
    t = dict(rows, **over)
    return sdpa.lib().sdpa_paged_attn(ctypes.byref(p), packed(t["q"]), packed(t["y"]), where,
                                      size, None)


PAGED_BAD = [
    (dict(struct_size=8), "INVALID"), (dict(dtype=3), "INVALID"), (dict(B=-1), "SHAPE"), (dict(tokens=-1), "SHAPE"),
    (dict(num_pages=-1), "SHAPE"), (dict(max_pages=-1), "SHAPE"), (dict(page_size=0), "SHAPE"), (dict(Nq=5), "SHAPE"),
    (dict(H=12), "UNSUPPORTED"), (dict(Hv=264), "UNSUPPORTED"), (dict(max_pages=1 << 28), "OVERFLOW"),
    (dict(tokens=1 << 29), "OVERFLOW"), (dict(B=1 << 25), "OVERFLOW"), (dict(B=3, cu_new=None), "SHAPE"),
    (dict(B=0, cu_new=None), "SHAPE"), (dict(kv_lens=None), "NULL"), (dict(page_table=None), "NULL"), (dict(kv_lens=258), "ALIGNMENT"),
    (dict(page_table_stride=2), "INVALID"), (dict(page_table_stride=1 << 41), "OVERFLOW"),
    (dict(k_pages=sdpa.sdpa_view(None, 0, 0, 0)), "NULL"), (dict(k_pages=sdpa.sdpa_view(256, 2048, 1024, 0)), "INVALID"),
    (dict(v_pages=sdpa.sdpa_view(264, 2048, 1024, 64)), "ALIGNMENT"), (dict(v_pages=sdpa.sdpa_view(256, 2052, 1024, 64)), "ALIGNMENT"),
]


@pytest.mark.parametrize("change,why", PAGED_BAD)
def test_paged_refusals(change, why):
    want = getattr(sdpa, "SDPA_ERR_" + why)
    assert append_code(*paged(change)) == want, sdpa.sdpa_last_error()
    assert attn_code(*paged(change)) == want, sdpa.sdpa_last_error()


ATTN_BAD = [
    (dict(causal=sdpa.SDPA_CAUSAL_UPPER_LEFT), "INVALID"), (dict(window=0), "INVALID"), (dict(window=-2), "INVALID"),
    (dict(window=1 << 31), "INVALID"), (dict(window=4, causal=0), "INVALID"), (dict(softcap=float("inf")), "INVALID"),
    (dict(has_scale=1, scale=float("nan")), "INVALID"), (dict(max_new=-1), "SHAPE"), (dict(head_sink=257), "ALIGNMENT"),
]


@pytest.mark.parametrize("change,why", ATTN_BAD)
def test_attention_refusals(change, why):
    p, rows, keep = paged(change)
    assert attn_code(p, rows, keep) == getattr(sdpa, "SDPA_ERR_" + why), sdpa.sdpa_last_error()
    assert sdpa.lib().sdpa_paged_workspace_size(ctypes.byref(p)) == 0


def test_attention_workspace_and_aliases():
    p, rows, keep = paged()
    need = sdpa.lib().sdpa_paged_workspace_size(ctypes.byref(p))
    assert need > 0
    # independent of how many tokens, sequences and keys there are
    assert need == sdpa.lib().sdpa_paged_workspace_size(ctypes.byref(paged(B=2, tokens=4, pages=50, width=20)[0]))
    assert attn_code(p, rows, keep, size=need - 1) == sdpa.SDPA_ERR_WORKSPACE
    assert attn_code(p, rows, keep, where=None) == sdpa.SDPA_ERR_WORKSPACE
    assert attn_code(p, rows, keep, where=260) == sdpa.SDPA_ERR_ALIGNMENT
    assert attn_code(p, rows, keep, y=rows["q"]) == sdpa.SDPA_ERR_ALIAS
    assert attn_code(p, rows, keep, where=rows["kp"].data_ptr() & ~255) == sdpa.SDPA_ERR_ALIAS
    shifted = torch.zeros(4 * 4 * 64 + 4, dtype=BF)[4:].view(4, 4, 64)
    assert attn_code(p, rows, keep, q=shifted) == sdpa.SDPA_ERR_ALIGNMENT


def test_append_aliases_and_rotation():
    p, rows, keep = paged()
    assert append_code(p, rows, keep, k=rows["kp"][0].transpose(0, 1)[:4]) == sdpa.SDPA_ERR_ALIAS
    p.v_pages = p.k_pages
    assert append_code(p, rows, keep) == sdpa.SDPA_ERR_ALIAS
    # one pool that holds both, keys and values side by side: per page, per slot, per row
    for pool, kv in ((torch.zeros(6, 2, 2, 16, 64, dtype=BF), lambda t: (t[:, 0], t[:, 1])),
                     (torch.zeros(6, 16, 2, 2, 64, dtype=BF), lambda t: (t[:, :, 0].transpose(1, 2), t[:, :, 1].transpose(1, 2))),
                     (torch.zeros(6, 2, 16, 128, dtype=BF), lambda t: (t[..., :64], t[..., 64:]))):
        a, b = kv(pool)
        p.k_pages, p.v_pages = V(a, keep), V(b, keep)
        assert accepted(lambda: append_code(p, rows, keep)), sdpa.sdpa_last_error()
        p.v_pages = V(pool.view(-1)[8:8 + 6 * 2 * 16 * 64].view(6, 2, 16, 64), keep)
        assert append_code(p, rows, keep) == sdpa.SDPA_ERR_ALIAS
    p, rows, keep = paged(dict(rotary_dim=32))
    assert append_code(p, rows, keep) == sdpa.SDPA_ERR_NULL
    p, rows, keep = paged(dict(rotary_cos=256))
    assert append_code(p, rows, keep) == sdpa.SDPA_ERR_INVALID
    p, rows, keep = paged(dict(rotary_cos=1024, rotary_sin=4096, rotary_max_pos=4, rotary_dim=66))
    assert append_code(p, rows, keep) == sdpa.SDPA_ERR_INVALID


def test_null_params():
    v = sdpa.sdpa_view(None, 0, 0, 0)
    L = sdpa.lib()
    assert L.sdpa_qk_norm_rotary(None, v, v, None) == sdpa.SDPA_ERR_NULL
    assert L.sdpa_paged_append(None, v, v, None) == sdpa.SDPA_ERR_NULL
    assert L.sdpa_paged_attn(None, v, v, None, 0, None) == sdpa.SDPA_ERR_NULL
    assert L.sdpa_paged_workspace_size(None) == 0 and L.sdpa_qk_norm_workspace_size(None) == 0


def test_empty_batches_need_no_gpu():
    p, rows, keep = paged(B=2, tokens=0)
    assert append_code(p, rows, keep) == sdpa.SDPA_OK and attn_code(p, rows, keep) == sdpa.SDPA_OK
    assert norm_code(*norm(S=0)) == sdpa.SDPA_OK


def test_the_binding_refuses_host_tensors_and_wrong_types():
    q, w = torch.zeros(1, 2, 3, 64, dtype=BF), torch.zeros(64, dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.sdpa_qk_norm_rotary(q, q.clone(), w, w)
    p, rows, keep = paged()
    lens, cu = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.sdpa_paged_attn(rows["q"], rows["kp"], rows["vp"], rows["table"], lens, cu_new=cu)
    args = lambda **kw: sdpa.make_paged_params(**{**dict(k_pages=rows["kp"], v_pages=rows["vp"], page_table=rows["table"],
                                                         kv_lens=lens, tokens=4, Nq=4, cu_new=cu), **kw})
    args()
    for bad in (dict(page_table=rows["table"].long()), dict(kv_lens=lens.long()), dict(cu_new=cu[:2]),
                dict(v_pages=rows["vp"].float()), dict(v_pages=rows["vp"][:3]), dict(head_sink=torch.zeros(3, dtype=BF)),
                dict(k_pages=rows["kp"][0]), dict(page_table=rows["table"].t().contiguous().t()),
                dict(cos_cache=torch.zeros(4, 16, dtype=BF), sin_cache=torch.zeros(4, 16, dtype=BF))):
        with pytest.raises(ValueError):
            args(**bad)


# ------------------------------------------------------------------ the oracle itself

@pytest.mark.parametrize("R,inter", [(16, False), (8, True), (0, False)])
def test_gradient_formula_against_differences(R, inter):
    """The float64 gradient formulas against central differences (truncation h^2, rounding 2^-52 / h)."""
    g = torch.Generator().manual_seed(1)
    x, w, dy = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((2, 3, 2, 16), (16,), (2, 3, 2, 16)))
    ang = torch.rand(2, 2, R // 2, generator=g, dtype=torch.float64) * 6
    cos, sin = torch.cos(ang), torch.sin(ang)
    f = lambda x, w: (norm_rotary64(x, w, cos, sin, R, inter, 1e-3)[0] * dy).sum()
    dx, dw, _, _ = norm_rotary_grad64(x, w, dy, cos, sin, R, inter, 1e-3)
    h = 1e-5
    for t, grad in ((x, dx), (w, dw)):
        for i in range(0, t.numel(), 5):
            e = torch.zeros_like(t)
            e.view(-1)[i] = h
            d = (f(x + e, w) - f(x - e, w)) if t is x else (f(x, w + e) - f(x, w - e))
            assert abs(d / (2 * h) - grad.view(-1)[i]) < 1e-7


@pytest.mark.parametrize("dtype,H,Hv", [(BF, 64, 64), (torch.float16, 128, 128), (BF, 96, 96), (torch.float32, 64, 64), (BF, 128, 64)])
def test_one_workspace_serves_every_call(dtype, H, Hv):
    """Its size depends on the type and the head sizes: not on the tokens, the hint, the head counts,
    the pages or their strides, with offsets or without, whichever kernel and tile they pick."""
    size = lambda p: sdpa.lib().sdpa_paged_workspace_size(ctypes.byref(p))
    sizes = {}
    for tokens in (2, 4, 8, 12, 16, 32, 40, 200):
        for Nq, Nkv in ((1, 1), (4, 2), (16, 1)):
            for page in (7, 16, 64):
                for hint in (0, 1, 3, 17, 1000):
                    for cu in (True, False):
                        p, _, _ = paged(tokens=tokens, Nq=Nq, Nkv=Nkv, H=H, Hv=Hv, page=page, dtype=dtype)
                        p.max_new = hint
                        if not cu:
                            p.cu_new = None
                        sizes.setdefault(size(p), (tokens, Nq, Nkv, page, hint, cu))
    far = paged(tokens=200, H=H, Hv=Hv, dtype=dtype)[0]
    far.k_pages = sdpa.sdpa_view(far.k_pages.data, 1 << 39, 64 * H, H)         # strides that no TMA box takes
    sizes.setdefault(size(far), "strides")
    assert len(sizes) == 1 and 0 not in sizes, sizes
    p, rows, keep = paged(tokens=200, H=H, Hv=Hv, dtype=dtype)
    need = size(p)
    assert attn_code(p, rows, keep, size=need - 1) == sdpa.SDPA_ERR_WORKSPACE
    assert accepted(lambda: attn_code(p, rows, keep, where=1 << 60, size=need)), sdpa.sdpa_last_error()


@pytest.mark.parametrize("B,S", [(2, 0), (0, 3), (0, 0)])
def test_empty_batches_with_a_cache_row_per_token(B, S):
    """Caches (B, S, R/2) of no tokens have no elements and no address."""
    p, q, k, keep = norm(B=B, S=S, ids=False)
    assert p.rotary_max_pos == 0 and p.rotary_dim == 64
    assert norm_code(p, q, k, keep) == sdpa.SDPA_OK, sdpa.sdpa_last_error()
    for cos in (None, 4096):                        # a cache without rows may still have an address
        p.rotary_cos = p.rotary_sin = cos
        assert norm_code(p, q, k, keep) == sdpa.SDPA_OK, sdpa.sdpa_last_error()
        assert sdpa.lib().sdpa_qk_norm_workspace_size(ctypes.byref(p)) > 0
    p, q, k, keep = norm(dict(rotary_max_pos=0), ids=False)      # tokens without rows are refused as before
    assert norm_code(p, q, k, keep) == sdpa.SDPA_ERR_SHAPE


def grad_problem(R, inter, dtype=torch.float32, D=64):
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype)
    d = dict(q=rn(1, 2, 4, D), k=rn(1, 1, 4, D), q_weight=(1 + 0.3 * torch.randn(D, generator=g)).to(dtype),
             k_weight=(1 + 0.3 * torch.randn(D, generator=g)).to(dtype), dq_out=rn(1, 2, 4, D), dk_out=rn(1, 1, 4, D))
    ang = torch.rand(1, 4, max(R, 2) // 2, generator=g) * 6
    return d, torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def formula_grads(d, cos, sin, R, inter):
    out = {}
    for t in "qk":
        dx, dw, _, _ = norm_rotary_grad64(d[t].double(), d[t + "_weight"].double(), d["d" + t + "_out"].double(), cos.double(),
                                          sin.double(), R, inter, 1e-5)
        out[t], out[t + "_weight"] = dx, dw
    return out


@pytest.mark.parametrize("R,inter", [(64, False), (32, True), (0, False)])
def test_the_check_by_differences_tells_wrong_gradients(R, inter):
    """The formula's gradient passes with room; one without its mean term, one with 0.9 of the weights'
    sums and one turned the wrong way do not."""
    d, cos, sin = grad_problem(R, inter)
    good = formula_grads(d, cos, sin, R, inter)
    autograd = {}
    for t in "qk":
        x, w = d[t].double().requires_grad_(), d[t + "_weight"].double().requires_grad_()
        (norm_rotary64(x, w, cos.double(), sin.double(), R, inter, 1e-5)[0] * d["d" + t + "_out"].double()).sum().backward()
        autograd[t], autograd[t + "_weight"] = x.grad, w.grad
    no_mean, short, turned = {}, {}, formula_grads(d, cos, -sin, R, inter)
    for t in "qk":
        x, w = d[t].double(), d[t + "_weight"].double()
        dy = d["d" + t + "_out"].double()
        g = rotate64(dy, cos.double()[:, None], -sin.double()[:, None], R, inter) if R else dy
        no_mean[t] = g * w / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5)
        short[t + "_weight"] = 0.9 * good[t + "_weight"]
    for i, name in enumerate(("q", "k", "q_weight", "k_weight")):
        check = lambda grads: norm_slope_check(d, name, grads, cos.double(), sin.double(), R, inter, 1e-5, 9 + i)
        assert torch.allclose(good[name], autograd[name], rtol=1e-10, atol=1e-12)
        err, tol = check(good)
        assert err < 0.2 * tol
        for wrong in (no_mean, short) + ((turned,) if R else ()):
            if name in wrong:
                err, tol = check(wrong)
                assert err > 3 * tol, (name, err, tol)
