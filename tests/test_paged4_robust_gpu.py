"""The page tables, the 4-bit append and the attention over it under conditions other than the ordinary:
which kernel serves which problem, expired waits, the bounds-checking build, captured steps, pools
beyond 32 bits, the binding's refusals."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from paged4_reference import cuda4, pack, paged4_attn64, ragged4, row_bytes, unpack64
from scaled_dot_product_gb300 import sdpa

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.join(ROOT, "tests")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def attn(r, k4, v4, **kw):
    return sdpa.sdpa_paged4_attn(r.q.cuda(), cuda4(k4), cuda4(v4), r.table.cuda(), r.kv_lens.cuda(),
                                 cu_new=None if r.cu is None else r.cu.cuda(), **kw)


@pytest.mark.parametrize("dtype,H,Hv,page,new,max_new,kernel", [
    (BF, 128, 128, 16, [1, 1], None, "paged4_mma_bf16_h128"),
    (BF, 128, 128, 3, [8, 2], 8, "paged4_mma_bf16_h128"),         # 16 rows
    (BF, 128, 128, 16, [9, 2], 9, "paged4_tc_bf16_h128"),
    (HF, 64, 64, 16, [16, 2], 16, "paged4_mma_f16_h64"),          # 32 rows
    (HF, 64, 64, 10, [17, 2], None, "paged4_tc_f16_h64"),         # unknown: the tokens bound it
    (HF, 64, 128, 16, [40, 2], 40, "paged4_simt_f16"),
    (FP, 128, 128, 16, [40, 2], 40, "paged4_simt_f32"),
])
def test_which_kernel(dtype, H, Hv, page, new, max_new, kernel):
    r, k4, v4, vs = ragged4(new, [70, 9], dtype=dtype, H=H, Hv=Hv, page=page, Nq=4, Nkv=2, seed=1)
    want, tol = paged4_attn64(r, vs, operands="values" if "_tc_" in kernel else "codes")
    y = attn(r, k4, v4, max_new=max_new)
    assert sdpa.sdpa_last_kernel_name() == kernel
    assert ((y.cpu().double() - want).abs() <= tol).all()


def test_f16_weights_touch_the_distance_from_the_middle_alone():
    """Values far from zero beside their spread: an fp16 weight's rounding must not touch the minimum.  One
    half step of the output and one of the weights' spread, as the tolerance has it, is a hundredth of what a rounding
    of weight times minimum would move."""
    r, k4, _, _ = ragged4([1, 2], [400, 70], dtype=HF, H=128, Nq=8, Nkv=1, seed=5)
    v = (torch.randn(r.vp.shape, generator=torch.Generator().manual_seed(1)) * 0.02 + 3.0).to(HF)
    v4 = pack(v, HF)
    r.vp, vs = unpack64(v4, 128, HF)
    want, tol = paged4_attn64(r, vs)
    y = attn(r, k4, v4, max_new=2)
    assert sdpa.sdpa_last_kernel_name() == "paged4_mma_f16_h128"
    assert ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_scales_that_grow_and_vanish_along_a_sequence(dtype):
    """Values whose groups' scales go up and down by far more than the fp16 weights' range from key to key, and
    constant groups (a scale of zero), in single tokens and chunks."""
    g = torch.Generator().manual_seed(3)
    for new in ([1, 1], [40, 1]):
        for kind in range(4):
            r, k4, _, _ = ragged4(new, [700, 300], dtype=dtype, H=64, Nq=8, Nkv=1, page=16, seed=6)
            x = torch.randn(r.vp.shape, generator=g)
            if kind == 0:
                x = x * 2.0 ** (torch.arange(x.shape[0]) - 30.0).clamp(-12, 12).view(-1, 1, 1, 1)
            elif kind == 1:
                x = x * 2.0 ** torch.randint(-12, 13, (*x.shape[:-1], 1), generator=g)
            elif kind == 2:
                x = torch.full_like(x, 3.0)
            else:
                x = torch.where(torch.rand(*x.shape[:-1], 1, generator=g) < 0.5, torch.zeros_like(x), x)
            v4 = pack(x.to(dtype), dtype)
            r.vp, vs = unpack64(v4, 64, dtype)
            want, tol = paged4_attn64(r, vs, operands="values" if new[0] > 1 else "codes")
            y = attn(r, k4, v4, max_new=max(new)).cpu().double()
            assert ((y - want).abs() <= tol).all(), (kind, ((y - want).abs() / tol).max(), sdpa.sdpa_last_kernel_name())


EXPIRED = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from paged4_reference import ragged4
    from scaled_dot_product_gb300 import sdpa
    for dtype, H, page, new in ((torch.bfloat16, 128, 16, [1, 1]), (torch.float16, 64, 10, [2, 3]), (torch.bfloat16, 128, 5, [90, 1]),
                                (torch.float16, 64, 8, [90, 1]), (torch.bfloat16, 64, 64, [200, 300])):
        for Nq in (4, 6):
            r, k4, v4, _ = ragged4(new, [3000, 500], dtype=dtype, H=H, page=page, Nq=Nq, Nkv=2)
            sdpa.sdpa_paged4_attn(r.q.cuda(), k4.cuda(), v4.cuda(), r.table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda())
            print("STATUS", sdpa.sdpa_last_kernel_name(), sdpa.sdpa_query_status())
    print("AFTER", torch.arange(1024, device="cuda").sum().item(), sdpa.sdpa_query_status())
""")


def test_expired_waits_are_reported_and_leave_the_context_usable():
    """With the limit at 1 ns every wait that is not satisfied already expires (SDPA_WAIT_LIMIT_NS is
    read once per process); the kernels give up, let their copies land and report."""
    run = lambda **env: subprocess.run([sys.executable, "-c", EXPIRED.format(root=ROOT, tests=TESTS)],
                                       env=dict(os.environ, **env), capture_output=True, text=True, timeout=300)
    for env, status in ((dict(), 0), (dict(SDPA_WAIT_LIMIT_NS="1"), sdpa.SDPA_ERR_TIMEOUT)):
        out = run(**env)
        assert out.returncode == 0, out.stderr[-2000:]
        lines = [line.split() for line in out.stdout.splitlines()]
        got = [(line[1], int(line[2])) for line in lines if line[0] == "STATUS"]
        assert len(got) == 10 and {n.split("_")[1] for n, _ in got} == {"mma", "tc"}
        assert all(s == status for _, s in got), got
        assert lines[-1] == ["AFTER", str(sum(range(1024))), "0"]


LATE = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from paged4_reference import paged4_attn64, ragged4
    from scaled_dot_product_gb300 import sdpa
    dev = lambda p: [x.cuda() for x in (p[0].q, p[1], p[2], p[0].table, p[0].kv_lens, p[0].cu)]
    probs = [dev(ragged4(new, past, dtype=dtype, H=H, page=page, Nq=4, Nkv=2)) for dtype, H, page, new, past in
             ((torch.bfloat16, 128, 16, [1], [100]), (torch.bfloat16, 128, 16, [1, 1, 2], [150, 60, 0]),
              (torch.float16, 64, 6, [1, 3], [200, 90]), (torch.bfloat16, 128, 16, [40], [80]),
              (torch.float16, 64, 8, [90, 1], [60, 30]), (torch.bfloat16, 64, 64, [150], [0]))]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    x = torch.randn(512, 512, device="cuda")
    want = x @ x
    plain = ragged4([2, 3], [70, 9], dtype=torch.float32, H=64)
    y, tol = paged4_attn64(plain[0], plain[3])
    d = dev(plain)
    for i in range(10):
        for p in probs:
            flush.zero_()                          # pages and tables come from memory: the copies take their time
            sdpa.sdpa_paged4_attn(*p[:5], cu_new=p[5])
            same = torch.equal(x @ x, want)        # the next kernel on those SMs has its shared memory to itself
            got = sdpa.sdpa_paged4_attn(*d[:5], cu_new=d[5]).cpu().double()
            print("STATUS", int(same and bool(((got - y).abs() <= tol).all())), sdpa.sdpa_query_status())
    print("AFTER", sdpa.sdpa_query_status())
""")


@pytest.mark.parametrize("limit", ["1", "500", "2000"])
def test_waits_that_expire_behind_the_last_copy(limit):
    out = subprocess.run([sys.executable, "-c", LATE.format(root=ROOT, tests=TESTS)],
                         env=dict(os.environ, SDPA_WAIT_LIMIT_NS=limit), capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = [line.split() for line in out.stdout.splitlines()]
    got = [(int(line[1]), int(line[2])) for line in lines if line[0] == "STATUS"]
    assert len(got) == 60 and all(right and status in (0, sdpa.SDPA_ERR_TIMEOUT) for right, status in got), got
    assert limit != "1" or all(status == sdpa.SDPA_ERR_TIMEOUT for _, status in got)
    assert lines[-1] == ["AFTER", "0"]


BOUNDS = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from scaled_dot_product_gb300 import build, sdpa
    sdpa.LIB_PATH = build.build(bounds_check=True)
    from paged4_reference import paged4_attn64, ragged4
    names = set()
    for dtype, H, page in ((torch.bfloat16, 128, 16), (torch.float16, 64, 6), (torch.float16, 128, 7), (torch.float32, 64, 24)):
        for new in ([1, 2, 0], [90, 1, 30]):
            r, k4, v4, vs = ragged4(new, [600, 33, 0], dtype=dtype, H=H, page=page, Nq=6, Nkv=2, extra_rows=1, seed=3)
            want, tol = paged4_attn64(r, vs, window=300, operands="values")
            tol = tol + paged4_attn64(r, vs, window=300)[1]
            y = sdpa.sdpa_paged4_attn(r.q.cuda(), k4.cuda(), v4.cuda(), r.table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda(), window=300)
            names.add(sdpa.sdpa_last_kernel_name())
            assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
            assert ((y[:r.tokens].cpu().double() - want).abs() <= tol).all()
            pool, pos = k4.cuda(), torch.arange(r.k.shape[0]).cuda()
            cos = torch.ones(400, H // 2, dtype=dtype, device="cuda")
            sdpa.sdpa_paged4_append(r.k.cuda(), r.v.cuda(), pool, pool.clone(), pos, pos, cos, cos, k_held=torch.empty_like(r.k).cuda())
            assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for B, n in ((3, 5), (300, 3), (40, 2000)):
        new = [n] * B
        new[1] = -1
        table = torch.full((B, 300), -1, dtype=torch.int32, device="cuda")
        table[:, :2] = torch.arange(2 * B, device="cuda").view(B, 2)
        free = torch.arange(400 * B, device="cuda").to(torch.int32).flip(0).contiguous()
        sdpa.sdpa_paged_tables(table, i([20] * B), i(new), free, i([390 * B]), page_size=16, tokens=n * B)
        assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
    print("kernels", sorted(names))
""")


def test_the_bounds_checking_build_runs_clean():
    r = subprocess.run([sys.executable, "-c", BOUNDS.format(root=ROOT, tests=TESTS)], capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert all(k in r.stdout for k in ("paged4_mma", "paged4_tc", "paged4_simt")), r.stdout


@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64), (FP, 64)])
def test_captured_steps_follow_their_data(dtype, H):
    """Two captured serving steps (single tokens, drafted ones) that share a workspace and a cache, replayed in turn: lengths,
    tables, slots and rows change on the device between replays."""
    B, Nq, Nkv, page, pages, width = 3, 4, 2, 8, 60, 12
    g = torch.Generator().manual_seed(2)
    kp = torch.zeros(pages, Nkv, page, row_bytes(H, dtype), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.tensor([pages], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def step(n):
        T = n * B
        s = dict(q=torch.zeros(T, Nq, H, dtype=dtype, device="cuda"), k=torch.zeros(T, Nkv, H, dtype=dtype, device="cuda"),
                 v=torch.zeros(T, Nkv, H, dtype=dtype, device="cuda"), y=torch.zeros(T, Nq, H, dtype=dtype, device="cuda"),
                 new=torch.full((B,), n, dtype=torch.int32, device="cuda"), cu=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                 pos=torch.zeros(T, dtype=torch.int64, device="cuda"), slots=torch.zeros(T, dtype=torch.int64, device="cuda"))

        def run():
            sdpa.sdpa_paged_tables(table, lens, s["new"], free, count, page_size=page, tokens=T, kv_lens=lens, free_count_out=count,
                                   cu_new=s["cu"], positions=s["pos"], slots=s["slots"])
            sdpa.sdpa_paged4_append(s["k"], s["v"], kp, vp, s["slots"])
            sdpa.sdpa_paged4_attn(s["q"], kp, vp, table, lens, cu_new=s["cu"], max_new=n, y=s["y"], workspace=ws)
        state = [t.clone() for t in (table, free, count, lens, kp, vp)]
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for t, old in zip((table, free, count, lens, kp, vp), state):
            t.copy_(old)
        return s, graph

    steps = {n: step(n) for n in (1, 20)}
    kept = [[[], []] for _ in range(B)]
    for n in (20, 1, 1, 20, 1):
        s, graph = steps[n]
        for t in ("q", "k", "v"):
            s[t].copy_(torch.randn(s[t].shape, generator=g).to(dtype))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            for i in range(n):
                for x, t in zip(kept[b], ("k", "v")):
                    x.append(unpack64(pack(s[t][b * n + i].cpu(), dtype), H, dtype)[0])
        assert lens.tolist() == [len(x[0]) for x in kept]
        for b in range(B):
            for i in (0, n - 1):
                K, V = (torch.stack(x[:len(x) - n + i + 1]) for x in kept[b])
                for h in range(Nq):
                    q = s["q"][b * n + i, h].cpu().double()
                    want = torch.softmax(K[:, h // 2] @ q / H ** 0.5, 0) @ V[:, h // 2]
                    # roundings of the output, the weights and, in chunks, keys and values: see paged4_attn64
                    mass = (K[:, h // 2].abs() @ q.abs() / H ** 0.5).max()
                    tol = (torch.finfo(dtype).eps / 2 * (4 + 2 * mass) + 2.0 ** -15) * V.abs().max()
                    assert (s["y"][b * n + i, h].cpu().double() - want).abs().max() <= tol, (n, b, i, h)
    assert sdpa.sdpa_query_status() == 0


def test_pools_beyond_32_bits():
    """Pages behind 4 GiB of a pool, in every kernel."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    for dtype, H, new in ((BF, 128, [1, 2]), (HF, 64, [40, 1]), (FP, 64, [2, 1])):
        r, k4, v4, vs = ragged4(new, [100, 40], dtype=dtype, H=H, page=16, Nq=4, Nkv=2, seed=4)
        pages, per = k4.shape[0], 2 * 16 * row_bytes(H, dtype)
        total = (5 << 30) // per
        far = total - pages
        kp, vp = (torch.empty(total, 2, 16, row_bytes(H, dtype), dtype=torch.uint8, device="cuda") for _ in range(2))
        kp[far:], vp[far:] = k4.cuda(), v4.cuda()
        table = torch.where(r.table >= 0, r.table + far, r.table)
        want, tol = paged4_attn64(r, vs, operands="values")
        tol = tol + paged4_attn64(r, vs)[1]
        y = sdpa.sdpa_paged4_attn(r.q.cuda(), kp, vp, table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda())
        assert sdpa.sdpa_query_status() == 0 and ((y.cpu().double() - want).abs() <= tol).all()
        slots = (torch.arange(r.k.shape[0]) * 3 + far * 16).cuda()
        sdpa.sdpa_paged4_append(r.k.cuda(), r.v.cuda(), kp, vp, slots)
        got = kp[far:].cpu().transpose(1, 2).flatten(0, 1)[(slots - far * 16).cpu()]
        assert sdpa.sdpa_query_status() == 0 and torch.equal(got, pack(r.k, dtype))
        del kp, vp


def test_rows_far_apart():
    """Token strides of 2^31 elements and more."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    base = torch.empty((1 << 31) + 8192, dtype=HF, device="cuda")
    k = base.as_strided((2, 2, 64), (1 << 31, 64, 1))
    held = base.as_strided((2, 2, 64), (1 << 31, 64, 1), 1024)
    x = torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(1)).to(HF)
    k.copy_(x)
    kp = torch.zeros(1, 2, 4, row_bytes(64, HF), dtype=torch.uint8, device="cuda")
    vp = torch.zeros_like(kp)
    with pytest.raises(sdpa.SdpaError):            # ranges that interleave: refused, whatever their elements
        sdpa.sdpa_paged4_append(k, k, kp, vp, torch.tensor([1, 3], device="cuda"), v_held=held)
    sdpa.sdpa_paged4_append(k, k, kp, vp, torch.tensor([1, 3], device="cuda"))
    assert sdpa.sdpa_query_status() == 0 and torch.equal(kp, vp)
    assert torch.equal(kp[0, :, [1, 3]].cpu().transpose(0, 1), pack(x, HF))


def test_slots_beyond_31_bits():
    """More than 2^31 slots in a pool."""
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB")
    pages = (1 << 27) + 40
    both = torch.empty(2, pages, 1, 16, 20, dtype=torch.uint8, device="cuda")
    k = torch.randn(5, 1, 32, generator=torch.Generator().manual_seed(1)).to(BF)
    slots = torch.tensor([(1 << 31) - 1, 1 << 31, pages * 16 - 1, 7, (1 << 31) + 100])
    sdpa.sdpa_paged4_append(k.cuda(), k.cuda(), both[0], both[1], slots.cuda())
    assert sdpa.sdpa_query_status() == 0
    for i in (0, 1):
        got = torch.stack([both[i, s // 16, :, s % 16].cpu() for s in slots.tolist()])
        assert torch.equal(got, pack(k, BF))


def test_the_binding_refuses():
    r, k4, v4, _ = ragged4([2, 3], [40, 9], dtype=BF, H=64, page=16, Nq=4, Nkv=2, seed=7)
    d = r.to("cuda")
    kp, vp = k4.cuda(), v4.cuda()
    args = dict(q=d.q, k_pages=kp, v_pages=vp, page_table=d.table, kv_lens=d.kv_lens, cu_new=d.cu)
    for bad in (dict(q=d.q.float()), dict(q=d.q[0]), dict(q=d.q[..., :32]), dict(kv_lens=d.kv_lens.cpu()), dict(k_pages=kp.view(torch.int8)),
                dict(k_pages=kp[..., :39]), dict(v_pages=vp[..., :30]), dict(v_pages=vp.cpu()), dict(q=None), dict(head_sink=d.q[0, 0])):
        with pytest.raises((ValueError, AttributeError)):
            sdpa.sdpa_paged4_attn(**{**args, **bad})
    for bad in (dict(window=0), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), dict(k_pages=kp.transpose(1, 2)[:, :, :2])):
        with pytest.raises((sdpa.SdpaError, ValueError)):
            sdpa.sdpa_paged4_attn(**{**args, **bad})
    slots = torch.arange(5, device="cuda")
    args = dict(k=d.k, v=d.v, k_pages=kp, v_pages=vp, slots=slots)
    for bad in (dict(slots=slots.int()), dict(slots=slots[:3]), dict(k=d.k.float()), dict(k_held=d.k[:3]), dict(cos_cache=d.k), dict(v=d.v[:, :1]),
                dict(k_pages=kp[:, :1]), dict(positions=slots.float()), dict(k_pages=None)):
        with pytest.raises(ValueError):
            sdpa.sdpa_paged4_append(**{**args, **bad})
    with pytest.raises(sdpa.SdpaError):
        sdpa.sdpa_paged4_append(**args, k_held=d.k)               # an input
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    args = dict(page_table=i(2, 4), past_lens=i(2), new_lens=i(2), free_pages=i(9), free_count=i(1), page_size=4, tokens=6)
    for bad in (dict(past_lens=i(3)), dict(new_lens=i(2).long()), dict(free_count=i(2)), dict(tokens=-1), dict(cu_new=i(2)), dict(slots=i(6)),
                dict(page_table=i(8)), dict(free_pages=i(3, 3)), dict(kv_lens=i(2).cpu()), dict(page_table=i(2, 8)[:, ::2])):
        with pytest.raises(ValueError):
            sdpa.sdpa_paged_tables(**{**args, **bad})
    with pytest.raises(sdpa.SdpaError):
        sdpa.sdpa_paged_tables(**args, kv_lens=args["new_lens"])


def test_calls_on_a_stream_that_is_not_the_current_one():
    """Inputs made on another stream, outputs read on the current one after it has waited."""
    s = torch.cuda.Stream()
    r, k4, v4, vs = ragged4([1, 30], [300, 20], dtype=HF, H=64, page=16, Nq=4, Nkv=2, seed=9)
    want, tol = paged4_attn64(r, vs, operands="values")
    d, kp, vp = r.to("cuda"), k4.cuda(), v4.cuda()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        y = sdpa.sdpa_paged4_attn(d.q, kp, vp, d.table, d.kv_lens, cu_new=d.cu, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert ((y.cpu().double() - want).abs() <= tol).all()
