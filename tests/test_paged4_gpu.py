"""The append to a paged cache of 4 bits a value and the attention over it against float64
(paged4_reference states how far each output may be off, term by term)."""
import pytest
import torch

from paged4_reference import cuda4, pack, paged4_attn64, ragged4, row_bytes, unpack64
from paged_reference import HALF_STEP, rotate64
from scaled_dot_product_gb300 import sdpa
from scaled_dot_product_gb300.workloads import rope_caches

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == FP else torch.int16)


# ------------------------------------------------------------------ append

def turned(x, cos, sin, R, inter):
    """The rotated rows in fp32, an operation at a time, rounded once to their type."""
    if not R:
        return x
    y, c, s = x.float().clone(), cos.float()[:, None], sin.float()[:, None]
    i1 = torch.arange(0, R, 2) if inter else torch.arange(R // 2)
    i2 = i1 + 1 if inter else i1 + R // 2
    a, b = x.float()[..., i1], x.float()[..., i2]
    y[..., i1] = a * c - b * s
    y[..., i2] = b * c + a * s
    return y.to(x.dtype)


def rows(tokens, heads, D, dtype, seed, spread=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, D, generator=g)
    if spread:                         # groups of unlike size and offset
        x = x * torch.exp(2 * torch.randn(tokens, heads, D // 32, generator=g)).repeat_interleave(32, -1)
        x = x + torch.randn(tokens, heads, D // 32, generator=g).repeat_interleave(32, -1) * 3
    return x.to(dtype)


APPENDS = [
    # dtype, tokens, Nkv, H, Hv, page, R, interleaved, held
    (BF, 1, 1, 32, 32, 4, 0, False, True), (BF, 70, 8, 128, 128, 16, 128, False, True), (HF, 33, 3, 64, 64, 24, 32, True, True),
    (HF, 50, 2, 64, 128, 6, 64, False, False), (FP, 21, 2, 64, 96, 8, 64, False, True), (FP, 9, 2, 128, 32, 2, 10, True, True),
    (BF, 40, 2, 96, 96, 12, 20, False, True), (HF, 40, 1, 256, 224, 12, 256, False, True), (BF, 5, 40, 256, 256, 4, 64, True, True),
    (FP, 30, 2, 256, 64, 4, 250, False, True), (BF, 300, 1, 64, 64, 100, 48, False, False),
]


@pytest.mark.parametrize("dtype,tokens,Nkv,H,Hv,page,R,inter,held", APPENDS)
def test_append(dtype, tokens, Nkv, H, Hv, page, R, inter, held):
    """Records equal to the bit, and nothing else in the pool changed."""
    g = torch.Generator().manual_seed(tokens)
    k, v = rows(tokens, Nkv, H, dtype, 1), rows(tokens, Nkv, Hv, dtype, 2)
    pages = tokens // page + 3
    slots = torch.randperm(pages * page, generator=g)[:tokens]
    pos = torch.randint(0, 500, (tokens,), generator=g)
    if tokens > 4:
        slots[3] = -1                                           # not stored
    kp = torch.randint(0, 256, (pages, Nkv, page, row_bytes(H, dtype)), generator=g, dtype=torch.uint8)
    vp = torch.randint(0, 256, (pages, Nkv, page, row_bytes(Hv, dtype)), generator=g, dtype=torch.uint8)
    rot, kr = {}, k
    if R:
        cos, sin = rope_caches(500, R // 2, dtype)
        rot = dict(positions=pos.cuda(), cos_cache=cos.cuda(), sin_cache=sin.cuda(), rotary_dim=R, interleaved=inter)
        kr = turned(k, cos[pos], sin[pos], R, inter)
    kh, vh = (torch.full_like(t, 77.0).cuda() for t in (k, v)) if held else (None, None)
    dk, dv = kp.cuda(), vp.cuda()
    out = sdpa.sdpa_paged4_append(k.cuda(), v.cuda(), dk, dv, slots.cuda(), k_held=kh, v_held=vh, **rot)
    assert sdpa.sdpa_query_status() == 0 and out[0] is dk and out[1] is dv
    live = slots >= 0
    for pool, got, x, h, D in ((kp, dk, kr, kh, H), (vp, dv, v, vh, Hv)):
        rec = pack(x, dtype)
        pool[slots[live] // page, :, slots[live] % page] = rec[live]
        assert torch.equal(got.cpu(), pool)
        if held:
            value, _ = unpack64(rec, D, dtype)
            err = (h.cpu().double() - value).abs()[live]
            # rounded once to the type; in fp32 the product is rounded before the sum too
            tol = HALF_STEP[dtype] * value.abs() + (2.0 ** -25 if dtype == HF else 2.0 ** -23 * (x.double().abs().amax(-1, keepdim=True) * 3))
            assert (err <= tol[live]).all() and (h.cpu()[~live] == 77.0).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_append_error_of_a_value(dtype):
    """A value is held within half a step of its group, and what the scale's rounding adds to 15 steps."""
    k = rows(200, 2, 128, dtype, 3)
    kp = torch.zeros(20, 2, 16, row_bytes(128, dtype), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    sdpa.sdpa_paged4_append(k.cuda(), k.cuda(), kp, vp, torch.arange(200, device="cuda"))
    assert torch.equal(kp, vp)
    value, scale = unpack64(kp.cpu().transpose(1, 2).flatten(0, 1)[:200], 128, dtype)
    tol = scale * (0.5 + 16 * HALF_STEP[dtype]) + 2.0 ** -20
    assert ((value - k.double()).abs() <= tol).all()


def test_append_groups_at_the_edges():
    """Constant groups, ties, the type's lowest and largest values, subnormals, and values that are not
    numbers, each beside ordinary groups of its row."""
    for dtype in (BF, HF, FP):
        x = rows(16, 1, 64, dtype, 4, spread=False)
        big = torch.finfo(dtype).max
        x[0, 0, :32] = 3.0
        x[1, 0, :32] = 0.0
        x[2, 0, :32] = torch.arange(32) * 0.5                   # a step of 31/30: ties of the codes among them
        x[3, 0, :32] = -big if dtype == HF else -big / 4
        x[3, 0, 5] = big if dtype == HF else big / 4
        x[4, 0, :32] = torch.arange(32) * torch.finfo(dtype).smallest_normal / 16
        x[5, 0, 7] = float("nan")
        x[6, 0, 8] = float("inf")
        x[7, 0, 9] = float("-inf")
        x[8, 0, :32] = torch.tensor([0.0, 15.0] * 16)           # a step of one: codes 0 and 15
        x[9, 0, :32] = torch.arange(32) % 16 + 0.5 * (torch.arange(32) >= 16)
        x[10, 0, 0], x[10, 0, 1] = big, -big                     # wider than fp32 in bf16 and fp32
        kp = torch.zeros(1, 1, 16, row_bytes(64, dtype), dtype=torch.uint8, device="cuda")
        vp, held = torch.zeros_like(kp), torch.zeros_like(x).cuda()
        sdpa.sdpa_paged4_append(x.cuda(), x.cuda(), kp, vp, torch.arange(16, device="cuda"), v_held=held)
        want = pack(x, dtype)
        got = kp.cpu()[0, 0]
        # a NaN's bits are of no account
        side = lambda t: t[..., 32:].contiguous().view(dtype)
        nan = torch.isnan(side(want[:, 0]))
        assert torch.equal(nan, torch.isnan(side(got)))
        assert torch.equal(got[..., :32], want[:, 0, :32])
        assert torch.equal(bits(side(got))[~nan], bits(side(want[:, 0]))[~nan])
        h = held.cpu()[:, 0]
        for row in (5, 6, 7) + (() if dtype == HF else (10,)):
            assert torch.isnan(h[row, :32]).all() and torch.isfinite(h[row, 32:]).all()
        assert torch.isfinite(h[[0, 1, 2, 3, 4, 8, 9]]).all()


def test_append_held_rows_near_the_end_of_fp32():
    """bf16 groups whose 15 scales pass fp32's largest number while minimum + 15 scales does not: the value is held as
    defined, not as an infinity."""
    u = 2.0 ** 120
    x = torch.zeros(4, 1, 32, dtype=BF)
    for i, (hi, lo) in enumerate(((252.0, -3.953125), (251.0, -4.96875), (253.0, -2.984375), (3.953125, -252.0))):
        x[i, 0, 0], x[i, 0, 1] = hi * u, lo * u
    value, scale = unpack64(pack(x, BF), 32, BF)
    assert torch.isfinite(value).all() and (15 * scale >= 2.0 ** 128).all()
    kp = torch.zeros(1, 1, 4, row_bytes(32, BF), dtype=torch.uint8, device="cuda")
    vp, held = torch.zeros_like(kp), torch.zeros_like(x).cuda()
    sdpa.sdpa_paged4_append(x.cuda(), x.cuda(), kp, vp, torch.arange(4, device="cuda"), v_held=held)
    # rounded once to the type, from an fp32 number
    assert ((held.cpu().double() - value).abs() <= (HALF_STEP[BF] + 2.0 ** -24) * value.abs()).all()


def test_append_bad_slots_and_positions():
    k = rows(4, 2, 64, BF, 5)
    cos, sin = (t.cuda() for t in rope_caches(10, 32, BF))

    def run(slots, pos):
        kp = torch.zeros(3, 2, 4, row_bytes(64, BF), dtype=torch.uint8, device="cuda")
        vp = torch.zeros_like(kp)
        sdpa.sdpa_paged4_append(k.cuda(), k.cuda(), kp, vp, torch.tensor(slots).cuda(), torch.tensor(pos).cuda(), cos, sin)
        rc, text = sdpa.sdpa_query_status(), sdpa.sdpa_last_error()
        return vp.cpu(), rc, text

    want = pack(k, BF)
    for bad in (12, 1 << 31, 1 << 40):
        vp, rc, text = run([0, bad, 5, 11], [0, 1, 2, 3])
        assert rc == sdpa.SDPA_ERR_INVALID and "slot" in text
        assert torch.equal(vp[0, :, 0], want[0]) and torch.equal(vp[1, :, 1], want[2]) and torch.equal(vp[2, :, 3], want[3])
    for bad in (10, -1, 1 << 40):
        vp, rc, text = run([0, 1, 5, 11], [0, bad, 2, 3])
        assert rc == sdpa.SDPA_ERR_INVALID and "position" in text and torch.equal(vp[0, :, 1], want[1])
    assert run([0, -1, 5, 11], [0, 99, 2, 3])[1] == 0            # a token that goes nowhere


def test_append_strided_rows_and_an_interleaved_pool():
    """Rows cut out of a packed projection, both pools in one tensor."""
    qkv = rows(20, 6, 64, HF, 6).cuda()
    k, v = qkv[:, 2:4], qkv[:, 4:6]
    both = torch.zeros(3, 2, 2, 8, row_bytes(64, HF), dtype=torch.uint8, device="cuda")
    slots = torch.arange(20, device="cuda")
    sdpa.sdpa_paged4_append(k, v, both[:, 0], both[:, 1], slots)
    for i, x in ((0, k), (1, v)):
        assert torch.equal(both[:, i].transpose(1, 2).flatten(0, 1)[:20].cpu(), pack(x.cpu(), HF))


# ------------------------------------------------------------------ attention

def run_attn(r, k4, v4, *, sink=None, **kw):
    y = torch.full((r.q.shape[0], r.Nq, r.Hv), 77.0, dtype=r.dtype, device="cuda")
    out = sdpa.sdpa_paged4_attn(r.q.cuda(), cuda4(k4), cuda4(v4), r.table.cuda(), r.kv_lens.cuda(),
                                cu_new=None if r.cu is None else r.cu.cuda(), y=y, head_sink=None if sink is None else sink.cuda(), **kw)
    assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
    assert out is y or out.data_ptr() == y.data_ptr()
    return out.cpu()


def check_attn(problem, sink=None, causal="lower_right", **kw):
    r, k4, v4, vs = problem
    out = run_attn(r, k4, v4, sink=sink, causal=causal, **kw)
    kernel = sdpa.sdpa_last_kernel_name()
    ref = {n: x for n, x in kw.items() if n in ("scale", "softcap", "window")}
    want, tol = paged4_attn64(r, vs, sink=sink, causal=causal != "none", operands="values" if "_tc_" in kernel else "codes", **ref)
    err = (out[:r.tokens].double() - want).abs()
    assert (err <= tol).all(), ((err / tol).max(), kernel)            # a NaN fails too
    assert (out[r.tokens:] == 77.0).all()                             # rows behind the last sequence
    return kernel


ATTNS = [
    # new, past, keyword arguments of the problem, of the call
    ([1], [0], dict(H=128), {}),
    ([1, 1, 1], [0, 15, 40], dict(H=128, uniform=True), {}),
    ([1, 1], [3, 500], dict(H=64, Nq=1, Nkv=1, dtype=HF, uniform=True), {}),
    ([3, 0, 1, 20], [5, 9, 31, 0], dict(H=64, dtype=HF, page=24), {}),
    ([0, 17, 2], [0, 100, 7], dict(H=128, Nkv=3, Nq=6, page=100), {}),
    ([4], [200], dict(H=96, dtype=BF, page=4), {}),
    ([4, 1], [60, 129], dict(H=64, Hv=128, dtype=HF, page=2), {}),
    ([5, 1], [60, 129], dict(H=256, Hv=32, dtype=BF, page=8), {}),
    ([5, 1, 2], [300, 0, 1], dict(H=64, dtype=FP, page=5), {}),
    ([1, 1, 1], [900, 64, 65], dict(H=128, dtype=FP, Nq=2, Nkv=2, uniform=True), {}),
    ([9, 1], [700, 64], dict(H=256, dtype=FP, page=3), dict(window=50)),
    ([6, 40, 1], [90, 300, 17], dict(H=128, page=16, Nq=8), dict(window=33)),
    ([6, 40, 1], [90, 300, 17], dict(H=64, page=16, Nq=8, dtype=HF), dict(softcap=5.0)),
    ([6, 1], [90, 17], dict(H=128, page=16, Nq=8), dict(causal="none")),
    ([6, 1], [90, 17], dict(H=128, page=16, dtype=HF), dict(scale=-0.3)),
    ([130, 1, 70], [900, 640, 5], dict(H=128, page=16), {}),
    ([130, 1, 70], [900, 640, 5], dict(H=64, page=64, dtype=HF), dict(window=100, softcap=20.0)),
    ([33, 2], [-20, -1], dict(H=64, page=16), {}),                    # fewer keys than new tokens: rows that admit none
    ([2, 3], [4, 9], dict(H=128, page=16, extra_rows=4, dtype=HF), {}),
    ([1, 2, 4], [3000, 2000, 1], dict(H=128, page=256), {}),
]


@pytest.mark.parametrize("new,past,kw,call", ATTNS)
def test_attn(new, past, kw, call):
    check_attn(ragged4(new, past, seed=len(new) + sum(new), **kw), **call)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_attn_sink(dtype):
    sink = torch.tensor([0.5, -3.0, float("-inf"), 9.0]).to(dtype)
    for new in ([1, 3], [70, 2]):
        check_attn(ragged4(new, [30, 0], dtype=dtype, H=64, seed=3), sink=sink)
        check_attn(ragged4(new, [30, 0], dtype=dtype, H=128, seed=3), sink=sink, window=7)


@pytest.mark.parametrize("dtype,H,page", [(BF, 128, 16), (HF, 64, 10), (FP, 64, 7), (BF, 64, 256), (HF, 128, 3), (BF, 96, 8)])
def test_attn_slots_that_are_not_numbers(dtype, H, page):
    """What lies past a sequence's keys, and below every window, is not looked at; entries of pages below
    every window may be gone."""
    for new in ([1, 1, 1], [60, 1, 90], [3, 2, 1]):
        r, k4, v4, vs = ragged4(new, [500, 900, 70], dtype=dtype, H=H, page=page, tail=float("nan"), seed=8)
        check_attn((r, k4, v4, vs))
        k4, v4 = k4.clone(), v4.clone()
        for b, n in enumerate(new):
            first = max(0, (r.lens[b] - n - 99)) // page             # page of the first key that some row admits
            for i in range(first):
                k4[r.table[b, i].item()] = 255
                v4[r.table[b, i].item()] = 255
            r.table[b, :first] = -1
        check_attn((r, k4, v4, vs), window=100)


def test_attn_rows_that_are_not_numbers():
    """A NaN in a query makes its row NaN, one in an admitted key too, one in a value its channels' group;
    other heads and sequences stay."""
    for dtype, H in ((BF, 128), (HF, 64), (FP, 64)):
        for new in ([1, 2], [80, 2]):
            r, k4, v4, vs = ragged4(new, [100, 9], dtype=dtype, H=H, Nq=4, Nkv=2, seed=9)
            clean = run_attn(r, k4, v4)
            q = r.q.clone()
            q[0, 1, 3] = float("nan")
            y = sdpa.sdpa_paged4_attn(q.cuda(), k4.cuda(), v4.cuda(), r.table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda()).cpu()
            assert torch.isnan(y[0, 1]).all()
            y[0, 1] = clean[0, 1]
            assert torch.equal(y, clean)
            es = 2 if dtype != FP else 4
            page, slot = r.table[0, 2].item(), 5                     # key 37 of the first sequence
            nan = torch.full((1,), float("nan"), dtype=dtype).view(torch.uint8)
            for pool in (0, 1):
                kb, vb = k4.clone(), v4.clone()
                side = (kb, vb)[pool][page, 1, slot, H // 2:]        # kv head 1, group 0: minimum and scale
                side[:es], side[es:2 * es] = nan, nan
                y = run_attn(r, kb, vb)
                n = new[0]
                hurt = y[:n, 2:]
                assert torch.isnan(hurt if pool == 0 else hurt[..., :32]).all()
                if pool == 1:
                    assert torch.equal(hurt[..., 32:], clean[:n, 2:, 32:])
                assert torch.equal(y[:n, :2], clean[:n, :2]) and torch.equal(y[n:], clean[n:])


@pytest.mark.parametrize("dtype,H,Hv", [(BF, 128, 128), (HF, 64, 64), (FP, 64, 64), (HF, 96, 96)])
@pytest.mark.parametrize("Nq,Nkv,new", [(1, 1, [1]), (5, 1, [1]), (2, 2, [1, 3]), (8, 8, [2, 1, 1]), (8, 1, [1, 7])])
def test_attn_many_partial_results(dtype, H, Hv, Nq, Nkv, new):
    check_attn(ragged4(new, [9000, 700, 5000][:len(new)], dtype=dtype, H=H, Hv=Hv, page=32, Nq=Nq, Nkv=Nkv, seed=H + Hv))


@pytest.mark.parametrize("group", [1, 2, 3, 6, 16, 100, 130])
def test_attn_group_sizes(group):
    for new in ([1, 2], [30, 9]):
        check_attn(ragged4(new, [70, 200], dtype=BF, H=64, page=16, Nq=group, Nkv=1, seed=group))


@pytest.mark.parametrize("hint", [1, 2, 5, 1000])
@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64)])
def test_attn_the_hint_changes_no_result(dtype, H, hint):
    check_attn(ragged4([1, 33, 1, 2, 70, 1, 1], [0, 100, 127, 128, 300, 3000, 255], dtype=dtype, H=H, page=16, Nq=6, Nkv=2, seed=2),
               max_new=hint)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** 9])
def test_attn_values_of_other_sizes(dtype, size):
    """Values and keys far from one: the tolerance goes with them; and groups of a row of unlike size."""
    for H in (64, 128):
        for new in ([1, 1], [70, 3]):
            r, _, _, _ = ragged4(new, [300, 40], dtype=dtype, H=H, Nq=4, Nkv=2, seed=11)
            g = torch.Generator().manual_seed(1)
            x = torch.randn(r.vp.shape, generator=g) * size
            x = x * 2.0 ** torch.randint(-3, 4, (*x.shape[:-1], H // 32), generator=g).repeat_interleave(32, -1)
            v4 = pack(x.to(dtype), dtype)
            k4 = pack((torch.randn(r.kp.shape, generator=g) / size).to(dtype), dtype)
            r.q.mul_(size)
            r.kp, _ = unpack64(k4, H, dtype)
            r.vp, vs = unpack64(v4, H, dtype)
            check_attn((r, k4, v4, vs))


def test_attn_interleaved_pool_and_strided_rows():
    for new in ([1, 2], [70, 1]):
        r, k4, v4, vs = ragged4(new, [70, 200], dtype=HF, H=64, page=16, interleave=True, seed=3)
        wide = torch.zeros(r.q.shape[0], 10, 64, dtype=HF, device="cuda")
        wide[:, 3:7] = r.q.cuda()
        want = run_attn(r, k4, v4)
        out = sdpa.sdpa_paged4_attn(wide[:, 3:7], cuda4(k4), cuda4(v4), r.table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda(),
                                    y=torch.zeros_like(wide)[:, 1:5])
        assert torch.equal(out.cpu(), want)
        check_attn((r, k4, v4, vs))


def test_attn_bad_pages_and_lengths():
    for dtype, new in ((BF, [1, 1]), (BF, [70, 1]), (FP, [2, 1])):
        r, k4, v4, _ = ragged4(new, [100, 40], dtype=dtype, H=64, page=16, seed=4)
        clean = run_attn(r, k4, v4)

        def run(change):
            table, lens, cu = r.table.clone(), r.kv_lens.clone(), r.cu.clone()
            change(table, lens, cu)
            y = sdpa.sdpa_paged4_attn(r.q.cuda(), k4.cuda(), v4.cuda(), table.cuda(), lens.cuda(), cu_new=cu.cuda()).cpu()
            rc, text = sdpa.sdpa_query_status(), sdpa.sdpa_last_error()
            assert sdpa.sdpa_query_status() == 0
            return y, rc, text

        for bad in (-1, 1 << 30):
            y, rc, text = run(lambda t, l, c: t.__setitem__((0, 1), bad))
            assert rc == sdpa.SDPA_ERR_INVALID and "page" in text
            assert torch.equal(y[new[0]:], clean[new[0]:]) and torch.isfinite(y).all()
        for change in (lambda t, l, c: l.__setitem__(0, 10 ** 6), lambda t, l, c: l.__setitem__(0, -3), lambda t, l, c: c.__setitem__(2, 10 ** 6)):
            y, rc, text = run(change)
            # a length beyond the sequence's pages meets entries that are no pages too
            assert rc == sdpa.SDPA_ERR_INVALID and ("cu_new" in text or "page" in text)


def test_attn_streams_and_repeats():
    a = ragged4([1] * 4, [3000, 20, 800, 1], dtype=BF, H=128, page=16, Nq=8, Nkv=2, uniform=True, seed=5)
    b = ragged4([90, 1], [700, 4000], dtype=HF, H=64, page=16, Nq=8, Nkv=2, seed=6)
    args = [(r.q.cuda(), k4.cuda(), v4.cuda(), r.table.cuda(), r.kv_lens.cuda(), None if r.cu is None else r.cu.cuda())
            for r, k4, v4, _ in (a, b)]
    call = lambda x, **kw: sdpa.sdpa_paged4_attn(*x[:5], cu_new=x[5], **kw)
    want = call(args[0]), call(args[1])
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        ya, yb = call(args[0], stream=s), call(args[1], stream=t)
    torch.cuda.synchronize()
    assert torch.equal(ya, want[0]) and torch.equal(yb, want[1])
    for _ in range(5):
        assert torch.equal(call(args[0]), want[0]) and torch.equal(call(args[1]), want[1])


def test_attn_empty():
    q = torch.randn(3, 4, 64, device="cuda").to(BF)
    kp = torch.empty(0, 2, 16, row_bytes(64, BF), dtype=torch.uint8, device="cuda")
    table = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = sdpa.sdpa_paged4_attn(q, kp, kp.clone(), table, lens)
    assert sdpa.sdpa_query_status() == 0 and (y == 0).all()
    assert sdpa.sdpa_paged4_attn(q[:0], kp, kp.clone(), table, lens).shape == (0, 4, 64)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype,H,page", [(BF, 128, 16), (HF, 64, 6), (FP, 64, 16)])
def test_a_served_batch(dtype, H, page):
    """Prompts, then single tokens, one sequence ending and its pages going to another: the tables, the
    norm and rotation at the tables' positions, the append at its slots and the attention, each step captured
    operators' outputs fed to the next, against float64 over the rows that the cache holds."""
    Nq, Nkv, pages, width, B = 4, 2, 40, 20, 3
    g = torch.Generator().manual_seed(12)
    kp = torch.zeros(pages, Nkv, page, sdpa.sdpa_paged4_row_bytes(H, dtype), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(pages, generator=g).to(torch.int32).cuda(), torch.tensor([pages], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    w = (1 + 0.1 * torch.randn(H, generator=g)).to(dtype).cuda()
    cos, sin = (t.cuda() for t in rope_caches(400, H // 2, dtype))
    kept = [[[], []] for _ in range(B)]                    # rows of each sequence as held
    for step, new in enumerate([[37, 5, 0], [1, 1, 1], [1, 1, 1], [1, -1, 20], [1, 9, 1], [2, 1, 1]]):
        n = [max(x, 0) for x in new]
        tokens = sum(n) + 2
        q, k = (torch.randn(1, tokens, x * H, generator=g).to(dtype).cuda() for x in (Nq, Nkv))
        v = torch.randn(tokens, Nkv, H, generator=g).to(dtype).cuda()
        _, cu, pos, slots, _ = sdpa.sdpa_paged_tables(table, lens, torch.tensor(new, dtype=torch.int32, device="cuda"), free, count,
                                                      page_size=page, tokens=tokens, kv_lens=lens, free_count_out=count)
        qr, kr = sdpa.sdpa_qk_norm_rotary(q, k, w, w, cos, sin, pos.view(1, -1), num_heads=Nq, kv_num_heads=Nkv)
        qr, kr = qr.view(tokens, Nq, H), kr.view(tokens, Nkv, H)
        kh, vh = torch.zeros_like(kr), torch.zeros_like(v)
        sdpa.sdpa_paged4_append(kr, v, kp, vp, slots, k_held=kh, v_held=vh)
        y = sdpa.sdpa_paged4_attn(qr, kp, vp, table, lens, cu_new=cu, max_new=max(n))
        assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
        t = 0
        for b in range(B):
            if new[b] < 0:
                kept[b] = [[], []]
            for i in range(n[b]):
                kept[b][0].append(unpack64(pack(kr[t].cpu(), dtype), H, dtype)[0])
                kept[b][1].append(unpack64(pack(v[t].cpu(), dtype), H, dtype)[0])
                assert (kh[t].cpu().double() - kept[b][0][-1]).abs().max() <= HALF_STEP[dtype] * 16
                t += 1
            assert lens[b].item() == len(kept[b][0])
        t = 0
        for b in range(B):
            for i in range(n[b]):
                K, V = (torch.stack(x[:len(x) - n[b] + i + 1]) for x in kept[b])
                for h in range(Nq):
                    s = K[:, h // 2] @ qr[t, h].cpu().double() / H ** 0.5
                    want = torch.softmax(s, 0) @ V[:, h // 2]
                    # roundings of the output, the weights and, in chunks, keys and values: see paged4_attn64
                    mass = (K[:, h // 2].abs() @ qr[t, h].cpu().double().abs() / H ** 0.5).max()
                    tol = (HALF_STEP[dtype] * (4 + 2 * mass) + 2.0 ** -15) * V.abs().max()
                    assert (y[t, h].cpu().double() - want).abs().max() <= tol, (step, b, i, h)
                t += 1
    assert count.item() == pages - sum(-(-len(x[0]) // page) for x in kept)
