"""The paged append and the attention over a paged cache against float64 (paged_reference states
how far each output may be off, term by term)."""
import pytest
import torch

from paged_reference import HALF_STEP, U32, paged_attn64, pair_abs, ragged, rotate64
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

APPENDS = [
    # new, past, keyword arguments of the problem, rotary_dim (None: no rotation), interleaved
    ([1, 1, 1], [0, 15, 40], dict(H=128, uniform=True), 0, False),
    ([3, 0, 1, 20], [5, 9, 31, 0], dict(H=64, dtype=HF, page=16, slots_first=False), 32, False),
    ([0, 17, 2], [0, 100, 7], dict(H=128, Nkv=3, Nq=3, page=24, interleave=True), 0, True),
    ([40], [1], dict(H=64, dtype=FP, page=1), 0, False),
    ([5, 6], [0, 2], dict(H=80, Hv=48, Nkv=1, Nq=1, page=7), 0, False),
    ([5, 6], [0, 2], dict(H=96, Hv=256, Nkv=2, Nq=2, page=100), 20, False),      # scalar rotation
    ([5, 6], [3, 2], dict(H=24, Hv=8, dtype=FP), 6, True),                       # scalar, interleaved
    ([2, 9], [3, 2], dict(H=64, dtype=HF), None, False),
    ([1] * 300, [i % 40 for i in range(300)], dict(H=64, Nkv=1, Nq=1, page=8), 0, False),
    ([0] * 280 + [1, 3], [4] * 282, dict(H=64, Nkv=1, Nq=1, page=8, extra_rows=3), 0, False),
    ([3, 2], [4, 9], dict(H=256, Hv=256, Nkv=40, Nq=40, page=16), 0, False),     # a token wider than a block
]


@pytest.mark.parametrize("new,past,kw,R,inter", APPENDS)
def test_append(new, past, kw, R, inter):
    r = ragged(new, past, seed=len(new), tail=0.5, **kw)
    d = r.to("cuda")
    rot = {}
    if R is not None:
        R = R or r.H
        cos, sin = rope_caches(max(r.lens) + 2, R // 2, r.dtype)
        rot = dict(cos_cache=cos.cuda(), sin_cache=sin.cuda(), rotary_dim=R, interleaved=inter)
    out = sdpa.sdpa_paged_append(d.k, d.v, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, **rot)
    assert sdpa.sdpa_query_status() == 0 and out[0] is d.kp and out[1] is d.vp
    kp, vp = d.kp.cpu(), d.vp.cpu()
    want_v, touched = r.vp.clone(), torch.zeros(r.kp.shape[0], r.page, dtype=torch.bool)
    t = 0
    for b, n in enumerate(new):
        for i in range(n):
            pos = past[b] + i
            pg, sl = r.table[b, pos // r.page].item(), pos % r.page
            touched[pg, sl] = True
            want_v[pg, :, sl] = r.v[t]
            x = r.k[t].double()
            if R is None:
                assert torch.equal(bits(kp[pg, :, sl]), bits(r.k[t]))
            else:
                want = rotate64(x, cos[pos].double(), sin[pos].double(), R, inter)
                tol = HALF_STEP[r.dtype] * want.abs() + 3 * U32 * pair_abs(x, R, inter) + (2.0 ** -25 if r.dtype == HF else 0)
                assert ((kp[pg, :, sl].double() - want).abs() <= tol).all()
            t += 1
    assert torch.equal(bits(vp), bits(want_v))
    keep = ~touched
    assert torch.equal(bits(kp.transpose(1, 2)[keep]), bits(r.kp.transpose(1, 2)[keep]))


def test_append_equals_rotary_then_copy():
    """The rotation's bits are sdpa_rotary's."""
    r = ragged([9, 14], [3, 30], H=128, seed=5, tail=0.0)
    d = r.to("cuda")
    cos, sin = (t.cuda() for t in rope_caches(64, 64, BF))
    pos = torch.cat([torch.arange(p, p + n) for n, p in zip(r.new, (3, 30))]).cuda()
    want = sdpa.sdpa_rotary(d.k.reshape(1, r.tokens, -1), cos, sin, pos.view(1, -1), num_heads=r.Nkv).view_as(d.k)
    sdpa.sdpa_paged_append(d.k, d.v, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, cos_cache=cos, sin_cache=sin)
    seq = torch.tensor([0] * 9 + [1] * 14).cuda()
    ids = d.table[seq, pos // r.page].long()
    assert torch.equal(d.kp.transpose(1, 2)[ids, pos % r.page], want)


def test_append_skips_and_reports_bad_data():
    def run(change, **rot):
        r = ragged([2, 3, 1], [4, 20, 0], H=64, page=8, extra_rows=2, tail=0.0, seed=2)
        change(r)
        d = r.to("cuda")
        sdpa.sdpa_paged_append(d.k, d.v, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, **rot)
        rc, msg = sdpa.sdpa_query_status(), sdpa.sdpa_last_error()
        assert sdpa.sdpa_query_status() == 0
        return r, d, rc, msg

    for bad in (-1, 1 << 30):
        def page(r):
            r.table[1, 2] = bad
        r, d, rc, msg = run(page)
        assert rc == sdpa.SDPA_ERR_INVALID and "page" in msg
        assert torch.equal(d.vp.cpu()[r.table[0, 0], :, 4:6].transpose(0, 1), r.v[:2])      # the others arrived
    for change in (lambda r: r.kv_lens.__setitem__(1, 10 ** 6), lambda r: r.kv_lens.__setitem__(1, -3),
                   lambda r: r.kv_lens.__setitem__(1, 2), lambda r: r.cu.__setitem__(3, 10 ** 6),
                   lambda r: r.cu.__setitem__(1, -9), lambda r: r.cu.__setitem__(0, 1)):
        r, d, rc, msg = run(change)
        assert rc == sdpa.SDPA_ERR_INVALID and "cu_new" in msg
    # a sequence with fewer keys than new tokens is skipped as a whole, the others arrive
    r, d, _, _ = run(lambda r: r.kv_lens.__setitem__(1, 2))
    pages = r.table[1, :3].long()
    assert torch.equal(bits(d.vp.cpu()[pages]), bits(r.vp[pages])) and torch.equal(bits(d.kp.cpu()[pages]), bits(r.kp[pages]))
    assert torch.equal(d.vp.cpu()[r.table[0, 0], :, 4:6].transpose(0, 1), r.v[:2])
    cos, sin = (t.cuda() for t in rope_caches(22, 32, BF))
    _, _, rc, msg = run(lambda r: None, cos_cache=cos, sin_cache=sin)
    assert rc == sdpa.SDPA_ERR_INVALID and "position" in msg


# ------------------------------------------------------------------ attention

def run_attn(r, *, poison_y=True, sink=None, **kw):
    d = r.to("cuda")
    y = torch.full((d.q.shape[0], r.Nq, r.Hv), 77.0, dtype=r.dtype, device="cuda") if poison_y else None
    out = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, y=y,
                               head_sink=None if sink is None else sink.cuda(), **kw)
    assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
    return out.cpu()


def check_attn(r, sink=None, causal="lower_right", **kw):
    ref = {n: x for n, x in kw.items() if n in ("scale", "softcap", "window")}
    want, tol = paged_attn64(r, sink=sink, causal=causal != "none", **ref)
    out = run_attn(r, sink=sink, causal=causal, **kw)
    err = (out[:r.tokens].double() - want).abs()
    assert (err <= tol).all(), ((err / tol).max(), sdpa.sdpa_last_kernel_name())      # a NaN fails too
    assert (out[r.tokens:] == 77.0).all()                                               # rows behind the last sequence
    return sdpa.sdpa_last_kernel_name()


TYPES = [(BF, 128, 16), (HF, 64, 32), (HF, 128, 8), (BF, 64, 128), (FP, 64, 24), (FP, 128, 16)]


@pytest.mark.parametrize("dtype,H,page", TYPES)
@pytest.mark.parametrize("group", [1, 3, 8])
def test_single_tokens(dtype, H, page, group):
    r = ragged([1] * 6, [0, 1, 63, 64, 200, 777], dtype=dtype, H=H, page=page, Nq=2 * group, Nkv=2, uniform=True,
               seed=group)
    check_attn(r)


@pytest.mark.parametrize("dtype,H,page", TYPES)
@pytest.mark.parametrize("group", [1, 4, 5])
def test_a_few_tokens(dtype, H, page, group):
    r = ragged([5, 1, 0, 16, 2, 7], [130, 0, 50, 300, 62, 1], dtype=dtype, H=H, page=page, Nq=2 * group, Nkv=2,
               extra_rows=2, seed=group + 10)
    check_attn(r, max_new=16)
    check_attn(r)                          # the hint does not matter


@pytest.mark.parametrize("dtype,H,page", TYPES)
@pytest.mark.parametrize("group", [2, 7])
def test_chunks(dtype, H, page, group):
    r = ragged([70, 1, 0, 131], [200, 330, 5, 0], dtype=dtype, H=H, page=page, Nq=group, Nkv=1, extra_rows=1,
               seed=group + 20)
    check_attn(r, max_new=131)


@pytest.mark.parametrize("dtype,H,Hv", [(BF, 96, 96), (HF, 64, 128), (HF, 128, 64), (BF, 256, 256), (FP, 256, 32),
                                        (BF, 8, 8), (FP, 4, 4), (HF, 192, 128)])
def test_other_head_sizes(dtype, H, Hv):
    check_attn(ragged([1, 40, 3], [100, 17, 64], dtype=dtype, H=H, Hv=Hv, page=16, Nq=6, Nkv=2, seed=3))


@pytest.mark.parametrize("page", [1, 2, 7, 8, 40, 100, 256, 1000])
@pytest.mark.parametrize("new", [[1, 1], [90, 33]])
def test_page_sizes(page, new):
    check_attn(ragged(new, [150, 260], dtype=BF, H=128, page=page, Nq=4, Nkv=2, seed=page))
    check_attn(ragged(new, [150, 260], dtype=HF, H=64, page=page, Nq=4, Nkv=2, seed=page, slots_first=False))


RULES = [dict(window=1), dict(window=40), dict(window=128, sink=True), dict(softcap=5.0), dict(softcap=30.0, sink=True),
         dict(scale=0.3), dict(scale=-0.2), dict(scale=0.0), dict(causal="none"), dict(causal="none", softcap=2.0),
         dict(window=10 ** 9)]


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64), (FP, 64), (BF, 96)])
def test_rules(rule, dtype, H):
    rule = dict(rule)
    sink = torch.tensor([0.0, 3.0, -float("inf"), -2.0, 60.0, 1.0]).to(dtype) if rule.pop("sink", False) else None
    for new in ([1, 1, 1], [100, 3, 140]):
        check_attn(ragged(new, [300, 40, 0], dtype=dtype, H=H, page=16, Nq=6, Nkv=2, seed=4), sink=sink, **rule)


def test_large_scores_keep_their_maximum():
    for dtype, H in ((BF, 128), (HF, 64), (FP, 64)):
        for new in ([1, 2], [80, 90]):
            r = ragged(new, [500, 200], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=6)
            r.q *= 20
            check_attn(r)


@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64), (FP, 64)])
def test_rows_without_keys_are_zero(dtype, H):
    """Fewer keys than new tokens: the first rows sit before the first key."""
    for new, past in (([4, 1], [-3, -1]), ([100, 70], [-60, -70])):
        r = ragged(new, past, dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=8)
        check_attn(r)
        check_attn(r, sink=torch.zeros(4).to(dtype))
    r = ragged([2, 1], [-2, 5], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=8)
    check_attn(r, causal="none")


@pytest.mark.parametrize("dtype,H,page", TYPES)
def test_long_split_over_many_blocks(dtype, H, page):
    """One short sequence beside one whose keys are spread over all blocks."""
    r = ragged([1, 1], [3, 9000], dtype=dtype, H=H, page=page, Nq=4, Nkv=1, uniform=True, seed=12)
    check_attn(r)
    r = ragged([33], [5000], dtype=dtype, H=H, page=page, Nq=4, Nkv=1, seed=13)
    check_attn(r)


def test_many_sequences():
    new = [(i * 7) % 4 for i in range(700)]
    r = ragged(new, [(i * 13) % 50 for i in range(700)], dtype=BF, H=64, page=8, Nq=2, Nkv=1, seed=14)
    check_attn(r)
    r = ragged([1] * 650, [(i * 13) % 50 for i in range(650)], dtype=FP, H=64, page=8, Nq=1, Nkv=1, uniform=True, seed=14)
    check_attn(r)


def test_pages_shared_by_sequences_and_interleaved_pools():
    r = ragged([1, 40], [100, 61], dtype=BF, H=128, page=16, Nq=4, Nkv=2, interleave=True, seed=15)
    r.table[1, :3] = r.table[0, :3]        # a common prefix
    check_attn(r)


def test_strided_rows_and_empty_batches():
    r = ragged([1, 30], [100, 61], dtype=BF, H=64, page=16, Nq=4, Nkv=2, seed=16)
    want, tol = paged_attn64(r)
    d = r.to("cuda")
    packed = torch.zeros(31, 8, 64, dtype=BF, device="cuda")
    packed[:, ::2] = d.q
    wide = torch.full((31, 4, 128), 9.0, dtype=BF, device="cuda")
    y = sdpa.sdpa_paged_attn(packed[:, ::2], d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, y=wide[..., 64:])
    assert ((y.cpu().double() - want).abs() <= tol).all() and (wide[..., :64] == 9.0).all()
    e = sdpa.sdpa_paged_attn(d.q[:0], d.kp, d.vp, d.table, d.kv_lens, cu_new=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert e.shape == (0, 4, 64)
    # offsets that all are zero over rows that exist: nothing is written
    y = torch.full((31, 4, 64), 5.0, dtype=BF, device="cuda")
    sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=torch.zeros(3, dtype=torch.int32, device="cuda"), y=y)
    assert (y == 5.0).all() and sdpa.sdpa_query_status() == 0


@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64), (FP, 64)])
def test_bad_pages_and_lengths_are_reported(dtype, H):
    for new in ([1, 1, 1], [80, 1, 70]):
        base = ragged(new, [100, 20, 50], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=17)
        want, tol = paged_attn64(base)
        for bad in (-1, 1 << 30, base.kp.shape[0]):
            r = ragged(new, [100, 20, 50], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=17)
            r.table[0, 1] = bad
            d = r.to("cuda")
            y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu)
            assert sdpa.sdpa_query_status() == sdpa.SDPA_ERR_INVALID and sdpa.sdpa_query_status() == 0
            # its keys and values count as zeros; the other sequences are as before
            zero = ragged(new, [100, 20, 50], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=17)
            zero.kp[zero.table[0, 1].item()] = 0
            zero.vp[zero.table[0, 1].item()] = 0
            want, tol = paged_attn64(zero)
            assert ((y.cpu().double() - want).abs() <= tol).all()
        for change in (lambda r: r.kv_lens.__setitem__(2, 10 ** 6), lambda r: r.kv_lens.__setitem__(2, -5),
                       lambda r: r.cu.__setitem__(3, 10 ** 6), lambda r: r.cu.__setitem__(2, -1)):
            r = ragged(new, [100, 20, 50], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=17)
            change(r)
            d = r.to("cuda")
            sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu)
            assert sdpa.sdpa_query_status() == sdpa.SDPA_ERR_INVALID and sdpa.sdpa_query_status() == 0


def test_pools_beyond_32_bit_offsets():
    """Pages whose offset in elements and bytes passes 2^32."""
    pages, page, Nkv, H = 140000, 16, 8, 128                  # 2.3e9 elements a pool
    kp = torch.empty(pages, page, Nkv, H, dtype=BF, device="cuda").transpose(1, 2)
    vp = torch.empty(pages, page, Nkv, H, dtype=BF, device="cuda").transpose(1, 2)
    for new in ([1, 1], [50, 60]):
        r = ragged(new, [40, 90], dtype=BF, H=H, page=page, Nq=16, Nkv=Nkv, seed=18)
        want, tol = paged_attn64(r)
        d = r.to("cuda")
        far = torch.arange(pages - 1, pages - 1 - r.kp.shape[0], -1, device="cuda")
        kp[far], vp[far] = d.kp, d.vp
        table = torch.where(d.table >= 0, pages - 1 - d.table, -1).to(torch.int32)
        y = sdpa.sdpa_paged_attn(d.q, kp, vp, table, d.kv_lens, cu_new=d.cu)
        assert ((y.cpu().double() - want).abs() <= tol).all()
        sdpa.sdpa_paged_append(d.k, d.v, kp, vp, table, d.kv_lens, cu_new=d.cu)
        last = r.lens[1] - 1
        assert torch.equal(vp[table[1, last // page].item(), :, last % page], d.v[-1])
        assert sdpa.sdpa_query_status() == 0


@pytest.mark.parametrize("dtype,H,page", [(BF, 128, 16), (HF, 64, 64), (BF, 64, 7), (HF, 96, 16), (FP, 64, 24)])
@pytest.mark.parametrize("new,hint", [([1, 1, 1], 1), ([1, 3, 1], 300), ([90, 1, 200], 200)])
def test_keys_below_every_window_do_not_matter(dtype, H, page, new, hint):
    r = ragged(new, [700, 75, 1000], dtype=dtype, H=H, page=page, Nq=4, Nkv=2, seed=23)
    want, tol = paged_attn64(r, window=50)
    for b, (n, T) in enumerate(zip(r.new, r.lens)):
        j = torch.arange(max(0, T - n - 49))                   # the first new token admits T - n - 49 and on
        ids = r.table[b, j // page].long()
        for pool, x in ((r.kp, float("nan")), (r.vp, float("inf"))):
            pool[ids, :, j % page] = x
    d = r.to("cuda")
    y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, max_new=hint, window=50)
    assert sdpa.sdpa_query_status() == 0
    assert ((y.cpu().double() - want).abs() <= tol).all(), sdpa.sdpa_last_kernel_name()


def test_streams_graphs_and_a_shared_workspace():
    """Two captured calls that share one workspace, replayed in turn, and a call on another stream."""
    probs = [ragged([1, 1, 1], [700, 30, 5], dtype=BF, H=128, Nq=8, Nkv=2, uniform=True, seed=19).to("cuda"),
             ragged([60, 2], [300, 900], dtype=BF, H=128, Nq=8, Nkv=2, seed=20).to("cuda")]
    want = [sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu) for d in probs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for d, w in zip(probs, want):
        y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, stream=st)
        st.synchronize()
        assert torch.equal(y, w)
    ws = torch.full((1 << 27,), 255, dtype=torch.uint8, device="cuda")        # any contents
    graphs = []
    for d in probs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, workspace=ws)
        graphs.append((g, y))
    for _ in range(3):
        for (g, y), w in zip(graphs, want):
            y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, w)
    # lengths are read by the kernels: a replay follows them
    d = probs[0]
    d.kv_lens -= 3
    graphs[0][0].replay()
    fresh = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu)
    assert torch.equal(graphs[0][1], fresh) and not torch.equal(fresh, want[0])


# ------------------------------------------------------------------ a run of them together

@pytest.mark.parametrize("dtype,H,window", [(BF, 128, -1), (HF, 64, 50)])
def test_a_decoder_layer_step_by_step(dtype, H, window):
    """Two sequences take a chunk, then single tokens, then a few tokens at once: norm and
    rotation, append, attention.  Every step's rows equal those of dense attention over all rows
    so far (the library's own forward on the rows in order), within the two paths' roundings."""
    Nq, Nkv, page, steps = 8, 2, 16, [[90, 40], [1, 1], [1, 1], [4, 0], [0, 30]]
    total = [sum(s[b] for s in steps) for b in range(2)]
    g = torch.Generator().manual_seed(30)
    rn = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    q, k, v = ([rn(total[b], n, H) for b in range(2)] for n in (Nq, Nkv, Nkv))
    wq, wk = (1 + 0.2 * torch.randn(2, H, generator=g)).to(dtype).cuda()
    cos, sin = (t.cuda() for t in rope_caches(256, H // 2, dtype))
    width = 16
    kp = torch.full((2 * width, page, Nkv, H), float("nan"), dtype=dtype, device="cuda").transpose(1, 2)
    vp = torch.full_like(kp, float("nan"))
    table = torch.randperm(2 * width, generator=g).view(2, width).to(torch.int32).cuda()
    have = [0, 0]
    ys = [[], []]
    for step in steps:
        rows = lambda x: torch.cat([x[b][have[b]:have[b] + step[b]] for b in range(2)])
        pos = torch.cat([torch.arange(have[b], have[b] + step[b]) for b in range(2)]).cuda()
        t = len(pos)
        qn, kn = sdpa.sdpa_qk_norm_rotary(rows(q).view(1, t, -1), rows(k).view(1, t, -1), wq, wk, cos, sin,
                                          pos.view(1, -1), num_heads=Nq, kv_num_heads=Nkv)
        vn = rows(v)
        have = [h + n for h, n in zip(have, step)]
        lens = torch.tensor(have, dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, step[0], t], dtype=torch.int32, device="cuda")
        sdpa.sdpa_paged_append(kn.view(t, Nkv, H), vn, kp, vp, table, lens, cu_new=cu)
        y = sdpa.sdpa_paged_attn(qn.view(t, Nq, H), kp, vp, table, lens, cu_new=cu, window=window)
        ys[0].append(y[:step[0]])
        ys[1].append(y[step[0]:])
    assert sdpa.sdpa_query_status() == 0
    for b in range(2):
        T = total[b]
        pos = torch.arange(T, device="cuda").view(1, -1)
        qn, kn = sdpa.sdpa_qk_norm_rotary(q[b].view(1, T, -1), k[b].view(1, T, -1), wq, wk, cos, sin, pos, num_heads=Nq,
                                          kv_num_heads=Nkv)
        heads = lambda x, n: x.view(1, T, n, H).transpose(1, 2)
        dense = sdpa.sdpa_attn_fwd(heads(qn, Nq), heads(kn, Nkv), heads(v[b], Nkv), causal="lower_right", window=window)
        got, want = torch.cat(ys[b]).double(), dense[0].transpose(0, 1).double()
        # each path: half a step of the output, half a step of the weights on |v| <= its maximum
        tol = 2 * HALF_STEP[dtype] * (want.abs() + v[b].double().abs().max()) + 1e-4
        assert ((got - want).abs() <= tol).all()
