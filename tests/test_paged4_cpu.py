"""Argument checks of the page tables, the 4-bit append and the attention over it: what the C entry
points refuse before any launch, and what the binding refuses; and the plain definitions themselves."""
import ctypes

import pytest
import torch

from paged4_reference import pack, row_bytes, tables_of, unpack64
from scaled_dot_product_gb300 import sdpa

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def accepted(call):
    """The call passes every check.  Made only where there is no GPU to launch it on: its tensors
    are host memory."""
    return torch.cuda.is_available() or call() == sdpa.SDPA_ERR_CUDA


def view(t):
    return sdpa.sdpa_view(t.data_ptr(), *t.stride()[:3])


def packed(t):
    return sdpa.sdpa_view(None, 0, 0, 0) if t is None else sdpa.sdpa_view(t.data_ptr(), 0, t.stride(1), t.stride(0))


def aligned(*shape, dtype=torch.uint8):
    n = 1
    for s in shape:
        n *= s
    raw = torch.zeros(n * torch.empty(0, dtype=dtype).element_size() + 256, dtype=torch.uint8)
    off = -raw.data_ptr() % 256
    return raw[off:off + n * torch.empty(0, dtype=dtype).element_size()].view(dtype).view(shape)


@pytest.mark.parametrize("dtype,part", [(BF, 20), (HF, 20), (FP, 24)])
def test_row_bytes(dtype, part):
    for D in (32, 64, 96, 128, 256):
        assert sdpa.sdpa_paged4_row_bytes(D, dtype) == D // 32 * part == row_bytes(D, dtype)
    for D in (0, 16, 48, 288, -32):
        with pytest.raises(ValueError):
            sdpa.sdpa_paged4_row_bytes(D, dtype)
    assert sdpa.lib().sdpa_paged4_row_bytes(64, 9) == -1


# ------------------------------------------------------------------ append

def append(over=(), *, tokens=4, Nkv=2, H=64, Hv=64, pages=3, page=4, dtype=BF, R=0):
    kp, vp = aligned(pages, Nkv, page, row_bytes(H, dtype)), aligned(pages, Nkv, page, row_bytes(Hv, dtype))
    slots, pos = torch.arange(tokens), torch.arange(tokens)
    rows = dict(k=aligned(tokens, Nkv, H, dtype=dtype), v=aligned(tokens, Nkv, Hv, dtype=dtype), k_held=None, v_held=None)
    p = sdpa.sdpa_paged4_append_params()
    p.struct_size = ctypes.sizeof(p)
    p.tokens, p.Nkv, p.H, p.Hv, p.dtype, p.num_pages, p.page_size = tokens, Nkv, H, Hv, sdpa._DTYPES[dtype], pages, page
    p.k_pages, p.v_pages, p.slots, p.positions = view(kp), view(vp), slots.data_ptr(), pos.data_ptr()
    keep = [kp, vp, slots, pos]
    if R:
        cos, sin = aligned(9, R // 2, dtype=dtype), aligned(9, R // 2, dtype=dtype)
        p.rotary_cos, p.rotary_sin, p.rotary_max_pos, p.rotary_dim = cos.data_ptr(), sin.data_ptr(), 9, R
        keep += [cos, sin]
    for n, x in dict(over).items():
        setattr(p, n, x)
    return p, rows, keep


def append_code(p, rows, keep, **over):
    t = dict(rows, **over)
    return sdpa.lib().sdpa_paged4_append(ctypes.byref(p), packed(t["k"]), packed(t["v"]), packed(t["k_held"]), packed(t["v_held"]), None)


APPEND_BAD = [
    (dict(struct_size=8), "INVALID"), (dict(dtype=3), "INVALID"), (dict(tokens=-1), "SHAPE"), (dict(num_pages=-1), "SHAPE"),
    (dict(Nkv=0), "SHAPE"), (dict(page_size=0), "SHAPE"), (dict(H=48), "UNSUPPORTED"), (dict(Hv=288), "UNSUPPORTED"),
    (dict(H=8), "UNSUPPORTED"), (dict(slots=None), "NULL"), (dict(slots=4), "ALIGNMENT"), (dict(positions=12), "ALIGNMENT"),
    (dict(Nkv=1 << 17), "OVERFLOW"), (dict(tokens=1 << 30), "OVERFLOW"), (dict(rotary_dim=8), "NULL"), (dict(rotary_cos=64), "INVALID"),
    (dict(k_pages=sdpa.sdpa_view(None, 1, 1, 40)), "NULL"), (dict(k_pages=sdpa.sdpa_view(256, 320, 160, 48)), "INVALID"),
    (dict(v_pages=sdpa.sdpa_view(264, 320, 160, 40)), "ALIGNMENT"), (dict(v_pages=sdpa.sdpa_view(256, 328, 168, 40)), "ALIGNMENT"),
    (dict(v_pages=sdpa.sdpa_view(256, 0, 160, 40)), "INVALID"), (dict(v_pages=sdpa.sdpa_view(256, -320, 160, 40)), "INVALID"),
]


@pytest.mark.parametrize("change,why", APPEND_BAD)
def test_append_refusals(change, why):
    assert append_code(*append(change)) == getattr(sdpa, "SDPA_ERR_" + why), sdpa.sdpa_last_error()


def test_append_page_sizes():
    assert append_code(*append(page=3)) == sdpa.SDPA_ERR_ALIGNMENT          # 3 x 40 bytes
    assert accepted(lambda: append_code(*append(page=2)))
    assert accepted(lambda: append_code(*append(page=1, H=128, Hv=128)))
    assert append_code(*append(page=2, H=32, Hv=32)) == sdpa.SDPA_ERR_ALIGNMENT
    assert accepted(lambda: append_code(*append(page=1, H=64, Hv=64, dtype=FP)))


def test_append_rotation():
    assert accepted(lambda: append_code(*append(R=64)))
    for change, why in ((dict(rotary_dim=63), "INVALID"), (dict(rotary_dim=66), "INVALID"), (dict(rotary_sin=None), "INVALID"),
                        (dict(rotary_max_pos=0), "SHAPE"), (dict(rotary_interleaved=2), "INVALID"), (dict(positions=None), "NULL")):
        assert append_code(*append(change, R=64)) == getattr(sdpa, "SDPA_ERR_" + why)


def test_append_aliases_and_rows():
    p, rows, keep = append()
    assert accepted(lambda: append_code(p, rows, keep))
    for held in (dict(k_held=rows["k"]), dict(v_held=rows["v"]), dict(k_held=rows["v"])):
        assert append_code(p, rows, keep, **held) == sdpa.SDPA_ERR_ALIAS
    both = aligned(4, 4, 64, dtype=BF)
    assert append_code(p, rows, keep, k_held=both[:, :2], v_held=both[:, 1:3]) == sdpa.SDPA_ERR_ALIAS
    assert accepted(lambda: append_code(p, rows, keep, k_held=both[:, :2], v_held=both[:, 2:]))
    assert append_code(p, rows, keep, k=aligned(4, 2, 68, dtype=BF)[..., :64]) == sdpa.SDPA_ERR_ALIGNMENT
    p.v_pages = p.k_pages
    assert append_code(p, rows, keep) == sdpa.SDPA_ERR_ALIAS
    pool = aligned(3, 2, 2, 4, 40)                                          # (pages, k / v, heads, slots, record)
    p.k_pages, p.v_pages = view(pool[:, 0]), view(pool[:, 1])
    assert accepted(lambda: append_code(p, rows, keep + [pool]))
    p.slots = pool.data_ptr()
    assert append_code(p, rows, keep) == sdpa.SDPA_ERR_ALIAS


# ------------------------------------------------------------------ attention

def attn(over=(), *, B=2, tokens=4, Nq=4, Nkv=2, H=64, Hv=64, pages=3, page=4, width=3, dtype=BF):
    kp, vp = aligned(pages, Nkv, page, row_bytes(H, dtype)), aligned(pages, Nkv, page, row_bytes(Hv, dtype))
    table, lens, cu = torch.zeros(B, width, dtype=torch.int32), torch.zeros(B, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    p = sdpa.sdpa_paged_params()
    p.struct_size = ctypes.sizeof(p)
    p.B, p.tokens, p.Nq, p.Nkv, p.H, p.Hv, p.dtype = B, tokens, Nq, Nkv, H, Hv, sdpa._DTYPES[dtype]
    p.num_pages, p.page_size, p.max_pages = pages, page, width
    p.k_pages, p.v_pages = view(kp), view(vp)
    p.page_table, p.page_table_stride, p.kv_lens, p.cu_new = table.data_ptr(), width, lens.data_ptr(), cu.data_ptr()
    p.causal, p.window = sdpa.SDPA_CAUSAL_LOWER_RIGHT, -1
    for n, x in dict(over).items():
        setattr(p, n, x)
    rows = dict(q=aligned(tokens, Nq, H, dtype=dtype), y=aligned(tokens, Nq, Hv, dtype=dtype), kp=kp, vp=vp, table=table)
    return p, rows, [lens, cu]


def attn_code(p, rows, keep, where=None, size=None, **over):
    t = dict(rows, **over)
    need = sdpa.lib().sdpa_paged4_workspace_size(ctypes.byref(p))
    ws = aligned(max(need, 1))
    return sdpa.lib().sdpa_paged4_attn(ctypes.byref(p), packed(t["q"]), packed(t["y"]), ws.data_ptr() if where is None else where,
                                       need if size is None else size, None)


ATTN_BAD = [
    (dict(struct_size=4), "INVALID"), (dict(dtype=7), "INVALID"), (dict(B=-1), "SHAPE"), (dict(Nq=3), "SHAPE"), (dict(H=80), "UNSUPPORTED"),
    (dict(Hv=8), "UNSUPPORTED"), (dict(page_table=None), "NULL"), (dict(kv_lens=None), "NULL"), (dict(page_table_stride=1), "INVALID"),
    (dict(causal=1), "INVALID"), (dict(window=0), "INVALID"), (dict(window=5, causal=0), "INVALID"), (dict(softcap=float("nan")), "INVALID"),
    (dict(has_scale=1, scale=float("inf")), "INVALID"), (dict(max_new=-1), "SHAPE"), (dict(head_sink=257), "ALIGNMENT"),
    (dict(k_pages=sdpa.sdpa_view(256, 320, 160, 80)), "INVALID"), (dict(k_pages=sdpa.sdpa_view(256, 324, 164, 40)), "ALIGNMENT"),
    (dict(page_size=5), "ALIGNMENT"), (dict(max_pages=1 << 29, page_table_stride=1 << 30), "OVERFLOW"),
]


@pytest.mark.parametrize("change,why", ATTN_BAD)
def test_attn_refusals(change, why):
    assert attn_code(*attn(change)) == getattr(sdpa, "SDPA_ERR_" + why), sdpa.sdpa_last_error()
    assert sdpa.lib().sdpa_paged4_workspace_size(ctypes.byref(attn(change)[0])) == 0


def test_attn_workspace_and_aliases():
    p, rows, keep = attn()
    need = sdpa.lib().sdpa_paged4_workspace_size(ctypes.byref(p))
    assert need > 0 and accepted(lambda: attn_code(p, rows, keep))
    assert attn_code(p, rows, keep, size=need - 1) == sdpa.SDPA_ERR_WORKSPACE
    ws = aligned(need + 256)
    assert attn_code(p, rows, keep, where=ws.data_ptr() + 16) == sdpa.SDPA_ERR_ALIGNMENT
    assert attn_code(p, rows, keep, y=rows["q"]) == sdpa.SDPA_ERR_ALIAS
    # the size goes with the type and the head sizes alone
    for kw in (dict(tokens=900, Nq=16), dict(B=7, page=64, width=9), dict(over=dict(max_new=1)), dict(over=dict(window=5))):
        assert sdpa.lib().sdpa_paged4_workspace_size(ctypes.byref(attn(**kw)[0])) == need


# ------------------------------------------------------------------ tables

def tables(over=(), *, B=2, tokens=4, pages=6, width=3):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    t = dict(page_table=i(B, width), past_lens=i(B), new_lens=i(B), free_pages=i(pages), free_count=i(1), kv_lens=i(B), cu_new=i(B + 1),
             positions=torch.zeros(tokens, dtype=torch.int64), slots=torch.zeros(tokens, dtype=torch.int64), free_count_out=i(1))
    p = sdpa.sdpa_paged_tables_params()
    p.struct_size = ctypes.sizeof(p)
    p.B, p.tokens, p.page_size, p.max_pages, p.num_pages, p.page_table_stride = B, tokens, 16, width, pages, width
    for n, x in t.items():
        setattr(p, n, x.data_ptr())
    for n, x in dict(over).items():
        setattr(p, n, x)
    return p, t


def tables_code(p):
    return sdpa.lib().sdpa_paged_tables(ctypes.byref(p), None)


TABLES_BAD = [
    (dict(struct_size=4), "INVALID"), (dict(B=-1), "SHAPE"), (dict(tokens=-1), "SHAPE"), (dict(page_size=0), "SHAPE"),
    (dict(B=8193), "UNSUPPORTED"), (dict(max_pages=1 << 29), "OVERFLOW"), (dict(page_table_stride=2), "INVALID"),
    (dict(page_table_stride=1 << 41), "OVERFLOW"), (dict(slots=12), "ALIGNMENT"), (dict(kv_lens=6), "ALIGNMENT"),
] + [({n: None}, "NULL") for n in ("page_table", "past_lens", "new_lens", "free_pages", "free_count", "kv_lens", "cu_new", "positions",
                                   "slots", "free_count_out")]


@pytest.mark.parametrize("change,why", TABLES_BAD)
def test_tables_refusals(change, why):
    p, keep = tables(change)
    assert tables_code(p) == getattr(sdpa, "SDPA_ERR_" + why), sdpa.sdpa_last_error()


def test_tables_aliases():
    p, keep = tables()
    assert accepted(lambda: tables_code(p))
    p.kv_lens, p.free_count_out = p.past_lens, p.free_count                # in place
    assert accepted(lambda: tables_code(p))
    for out, other in (("kv_lens", "new_lens"), ("cu_new", "past_lens"), ("slots", "positions"), ("positions", "page_table"),
                       ("free_count_out", "cu_new"), ("free_pages", "past_lens"), ("kv_lens", "free_pages")):
        p, keep = tables(pages=64)
        setattr(p, out, getattr(p, other))
        if getattr(p, out) % 8 == 0 or out not in ("slots", "positions"):
            assert tables_code(p) == sdpa.SDPA_ERR_ALIAS, (out, other)


def test_binding_refusals():
    b, _ = sdpa._native()
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.sdpa_paged_tables(t, t[:, 0].contiguous(), t[:, 0].contiguous(), t[0], t[0, :1], page_size=4, tokens=3)
    k = torch.zeros(2, 2, 64, dtype=BF)
    kp = torch.zeros(1, 2, 4, 40, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.sdpa_paged4_append(k, k, kp, kp, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        sdpa.sdpa_paged4_attn(k, kp, kp, t[:, :1], t[:, 0].contiguous())


# ------------------------------------------------------------------ the definitions

@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_records_hold_their_values(dtype):
    g = torch.Generator().manual_seed(1)
    x = (torch.randn(50, 64, generator=g) * 3 + 1).to(dtype)
    value, scale = unpack64(pack(x, dtype), 64, dtype)
    step = torch.finfo(dtype).eps / 2
    assert ((value - x.double()).abs() <= scale * (0.5 + 16 * step)).all()
    assert torch.equal(value.unflatten(-1, (2, 32)).amin(-1), x.double().unflatten(-1, (2, 32)).amin(-1))      # the minimum is held as it is


def test_tables_by_hand():
    """Two pages given back and three taken, from the top of the stack."""
    out, said = tables_of([[4, 2, -1, -1], [0, -1, -1, -1], [1, 3, -1, -1]], [5, 4, 7], [2, 5, -1], [6, 5, 9, 9, 9, 9, 9], 2, 4, 9)
    assert out["free_pages"] == [6, 5, 1, 3, 9, 9, 9] and out["free_count_out"] == [2]
    assert out["page_table"] == [[4, 2, -1, -1], [0, 3, 1, -1], [1, 3, -1, -1]]
    assert out["kv_lens"] == [7, 9, 0] and out["cu_new"] == [0, 2, 7, 7]
    assert out["positions"] == [5, 6, 4, 5, 6, 7, 8, 0, 0] and out["slots"] == [9, 10, 12, 13, 14, 15, 4, -1, -1] and not said
