"""The paged and norm calls under conditions other than the ordinary: which kernel serves which
problem, expired waits, the bounds-checking build, several streams, the binding's refusals."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

from paged_reference import paged_attn64, ragged
from scaled_dot_product_gb300 import sdpa

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def attn(r, **kw):
    d = r.to("cuda")
    return sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, **kw)


@pytest.mark.parametrize("dtype,H,page,new,max_new,kernel", [
    (BF, 128, 16, [1, 1], None, "paged_mma_bf16_h128"),       # two tokens in all
    (BF, 128, 16, [40, 2], 40, "paged_tc_bf16_h128"),
    (BF, 128, 16, [40, 2], None, "paged_tc_bf16_h128"),       # unknown: the tokens bound it
    (HF, 64, 24, [40, 2], 40, "paged_tc_f16_h64"),
    (HF, 64, 100, [40, 2], 40, "paged_mma_f16_h64"),          # pages that eight-row boxes do not tile
    (HF, 64, 16, [3, 2], 3, "paged_mma_f16_h64"),
    (HF, 96, 16, [40, 2], 40, "paged_simt_f16"),
    (FP, 128, 16, [40, 2], 40, "paged_simt_f32"),
])
def test_which_kernel(dtype, H, page, new, max_new, kernel):
    r = ragged(new, [70, 9], dtype=dtype, H=H, page=page, Nq=4, Nkv=2, seed=1)
    want, tol = paged_attn64(r)
    y = attn(r, max_new=max_new)
    assert sdpa.sdpa_last_kernel_name() == kernel
    assert ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("hint", [1, 2, 5, 1000])
@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64)])
def test_the_hint_changes_no_result(dtype, H, hint):
    """Each kernel takes any counts, whatever the hint said: rows behind the first block of a unit,
    narrow units of the chunk kernel, one to many tiles of keys."""
    r = ragged([1, 33, 1, 2, 70, 1, 1], [0, 100, 127, 128, 300, 3000, 255], dtype=dtype, H=H, page=16, Nq=6, Nkv=2, seed=2)
    want, tol = paged_attn64(r)
    y = attn(r, max_new=hint)
    assert ((y.cpu().double() - want).abs() <= tol).all(), sdpa.sdpa_last_kernel_name()


@pytest.mark.parametrize("group", [1, 2, 3, 6, 16, 100, 130])
def test_group_sizes(group):
    """Groups that TMA boxes and groups that it does not, wider than a tile and not dividing one."""
    for new in ([1, 2], [30, 9]):
        r = ragged(new, [70, 200], dtype=BF, H=64, page=16, Nq=group, Nkv=1, seed=group)
        want, tol = paged_attn64(r)
        y = attn(r)
        assert ((y.cpu().double() - want).abs() <= tol).all(), sdpa.sdpa_last_kernel_name()


@pytest.mark.parametrize("dtype,H,Hv", [(HF, 96, 96), (FP, 64, 20), (FP, 128, 4), (BF, 128, 128), (HF, 64, 64), (BF, 256, 200)])
@pytest.mark.parametrize("Nq,Nkv,new", [(1, 1, [1]), (5, 1, [1]), (2, 2, [1, 3]), (8, 8, [2, 1, 1])])
def test_many_partial_results(dtype, H, Hv, Nq, Nkv, new):
    """Long sequences in few units: each is cut over many CTAs, whose partial results are joined in
    every way the joining kernel cuts its work (head sizes that are no power of two among them)."""
    r = ragged(new, [9000, 700, 5000][:len(new)], dtype=dtype, H=H, Hv=Hv, page=32, Nq=Nq, Nkv=Nkv, seed=H + Hv)
    want, tol = paged_attn64(r)
    y = attn(r, max_new=max(new))
    assert ((y.cpu().double() - want).abs() <= tol).all(), sdpa.sdpa_last_kernel_name()


def test_keys_that_are_not_numbers_outside_the_window():
    """Pages below every row's window may be gone (their ids are not looked at), and what lies past
    a sequence's keys is not a number."""
    for dtype, H, page in ((BF, 128, 16), (HF, 64, 64), (FP, 64, 16), (HF, 64, 12), (BF, 128, 256)):
        for new in ([1, 1, 1], [60, 1, 90]):
            r = ragged(new, [500, 1000, 700], dtype=dtype, H=H, page=page, Nq=4, Nkv=2, seed=4)
            want, tol = paged_attn64(r, window=100)
            for b, n in enumerate(new):
                first = (r.lens[b] - n - 99) // page          # page of the first key that some row admits
                for i in range(max(0, first)):
                    r.kp[r.table[b, i].item()] = float("nan")
                    r.vp[r.table[b, i].item()] = float("inf")
                r.table[b, :max(0, first)] = -1
            y = attn(r, window=100)
            assert sdpa.sdpa_query_status() == 0
            assert ((y.cpu().double() - want).abs() <= tol).all(), sdpa.sdpa_last_kernel_name()


def test_two_streams_at_once():
    a = ragged([1] * 4, [3000, 20, 800, 1], dtype=BF, H=128, page=16, Nq=8, Nkv=2, uniform=True, seed=5).to("cuda")
    b = ragged([90, 1], [700, 4000], dtype=HF, H=64, page=16, Nq=8, Nkv=2, seed=6).to("cuda")
    call = lambda r, **kw: sdpa.sdpa_paged_attn(r.q, r.kp, r.vp, r.table, r.kv_lens, cu_new=r.cu, **kw)
    want = call(a), call(b)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        ya, yb = call(a, stream=s), call(b, stream=t)
    torch.cuda.synchronize()
    assert torch.equal(ya, want[0]) and torch.equal(yb, want[1])
    # repeated calls agree bit for bit: partial results are joined in a fixed order
    for _ in range(5):
        assert torch.equal(call(a), want[0]) and torch.equal(call(b), want[1])


def test_tables_without_pages_and_empty_pools():
    q = torch.randn(3, 4, 64, device="cuda").to(BF)
    kp = torch.empty(0, 2, 16, 64, dtype=BF, device="cuda")
    table = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = sdpa.sdpa_paged_attn(q, kp, kp.clone(), table, lens)
    assert not y.any() and sdpa.sdpa_query_status() == 0
    lens += 1                                                  # more keys than the table can name
    y = sdpa.sdpa_paged_attn(q, kp, kp.clone(), table, lens)
    assert not y.any() and sdpa.sdpa_query_status() == sdpa.SDPA_ERR_INVALID


def test_the_binding_refuses():
    r = ragged([2, 3], [40, 9], dtype=BF, H=64, page=16, Nq=4, Nkv=2, seed=7).to("cuda")
    args = dict(q=r.q, k_pages=r.kp, v_pages=r.vp, page_table=r.table, kv_lens=r.kv_lens, cu_new=r.cu)
    for bad in (dict(q=r.q.float()), dict(q=r.q[0]), dict(q=r.q[:, :, ::2]), dict(kv_lens=r.kv_lens.cpu()), dict(cu_new=r.cu[:2]),
                dict(page_table=r.table.float()), dict(y=torch.empty(1, device="cuda")), dict(head_sink=r.q[0, 0]),
                dict(v_pages=r.vp.cpu()), dict(q=None), dict(kv_lens=7)):
        with pytest.raises((ValueError, AttributeError)):
            sdpa.sdpa_paged_attn(**{**args, **bad})
    with pytest.raises(sdpa.SdpaError) as e:
        sdpa.sdpa_paged_attn(**args, window=0)
    assert e.value.code == sdpa.SDPA_ERR_INVALID
    with pytest.raises(sdpa.SdpaError) as e:
        sdpa.sdpa_paged_attn(**args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == sdpa.SDPA_ERR_WORKSPACE
    x, w = torch.randn(1, 2, 3, 64, device="cuda").to(BF), torch.ones(64, dtype=BF, device="cuda")
    for bad in (dict(q_weight=w.float()), dict(k=x[:, :, :2]), dict(q_weight=w[:32]), dict(position_ids=torch.zeros(1, 3)),
                dict(cos_cache=x), dict(q_out=x.float()), dict(q=x[..., ::2], k=x[..., ::2]), dict(k_weight=w.cpu())):
        with pytest.raises(ValueError):
            sdpa.sdpa_qk_norm_rotary(**{**dict(q=x, k=x.clone(), q_weight=w, k_weight=w), **bad})
    # one byte that claims to be many
    many = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 27)
    with pytest.raises(ValueError, match="workspace"):
        sdpa.sdpa_paged_attn(**args, workspace=many)
    with pytest.raises(ValueError, match="workspace"):
        sdpa.sdpa_qk_norm_rotary_bwd(x, x.clone(), x.clone(), x.clone(), w, w, workspace=many)


EXPIRED = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from paged_reference import ragged
    from scaled_dot_product_gb300 import sdpa
    for dtype, H, page, new in ((torch.bfloat16, 128, 16, [1, 1]), (torch.float16, 64, 7, [2, 3]), (torch.bfloat16, 128, 16, [90, 1]),
                                (torch.float16, 64, 8, [90, 1]), (torch.bfloat16, 64, 64, [200, 300])):
        for Nq in (4, 6):
            r = ragged(new, [3000, 500], dtype=dtype, H=H, page=page, Nq=Nq, Nkv=2).to("cuda")
            sdpa.sdpa_paged_attn(r.q, r.kp, r.vp, r.table, r.kv_lens, cu_new=r.cu)
            print("STATUS", sdpa.sdpa_last_kernel_name(), sdpa.sdpa_query_status())
    print("AFTER", torch.arange(1024, device="cuda").sum().item(), sdpa.sdpa_query_status())
""")


def test_expired_waits_are_reported_and_leave_the_context_usable():
    """With the limit at 1 ns every wait that is not satisfied already expires (SDPA_WAIT_LIMIT_NS is
    read once per process); the kernels give up, let their copies land and report."""
    run = lambda **env: subprocess.run([sys.executable, "-c", EXPIRED.format(root=ROOT, tests=os.path.join(ROOT, "tests"))],
                                       env=dict(os.environ, **env), capture_output=True, text=True, timeout=300)
    for env, status in ((dict(), 0), (dict(SDPA_WAIT_LIMIT_NS="1"), sdpa.SDPA_ERR_TIMEOUT)):
        out = run(**env)
        assert out.returncode == 0, out.stderr[-2000:]
        lines = [line.split() for line in out.stdout.splitlines()]
        got = [(line[1], int(line[2])) for line in lines if line[0] == "STATUS"]
        assert len(got) == 10 and {n.split("_")[1] for n, _ in got} == {"mma", "tc"}
        assert all(s == status for _, s in got), got
        assert lines[-1] == ["AFTER", str(sum(range(1024))), "0"]


BOUNDS = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from scaled_dot_product_gb300 import build, sdpa
    sdpa.LIB_PATH = build.build(bounds_check=True)
    from paged_reference import paged_attn64, ragged
    names = set()
    for dtype, H, page in ((torch.bfloat16, 128, 16), (torch.float16, 64, 7), (torch.float16, 64, 8), (torch.float32, 64, 24)):
        for new in ([1, 2, 0], [90, 1, 30]):
            r = ragged(new, [600, 33, 0], dtype=dtype, H=H, page=page, Nq=6, Nkv=2, extra_rows=1, seed=3)
            want, tol = paged_attn64(r, window=300)
            d = r.to("cuda")
            y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, window=300)
            names.add(sdpa.sdpa_last_kernel_name())
            assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
            assert ((y[:r.tokens].cpu().double() - want).abs() <= tol).all()
            sdpa.sdpa_paged_append(d.k, d.v, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu)
            assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
    q, w = torch.randn(2, 5, 9, 128, device="cuda").bfloat16(), torch.ones(128, device="cuda").bfloat16()
    sdpa.sdpa_qk_norm_rotary(q, q.clone(), w, w)
    sdpa.sdpa_qk_norm_rotary_bwd(q, q.clone(), q.clone(), q.clone(), w, w)
    assert sdpa.sdpa_query_status() == 0, sdpa.sdpa_last_error()
    print("kernels", sorted(names))
""")


def test_the_bounds_checking_build_runs_clean():
    r = subprocess.run([sys.executable, "-c", BOUNDS.format(root=ROOT, tests=os.path.join(ROOT, "tests"))], capture_output=True,
                       text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert all(k in r.stdout for k in ("paged_mma", "paged_tc", "paged_simt")), r.stdout


LATE = textwrap.dedent("""
    import sys, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from paged_reference import paged_attn64, ragged
    from scaled_dot_product_gb300 import sdpa
    probs = [ragged(new, past, dtype=dtype, H=H, page=page, Nq=4, Nkv=2).to("cuda") for dtype, H, page, new, past in
             ((torch.bfloat16, 128, 16, [1], [100]), (torch.bfloat16, 128, 16, [1, 1, 2], [150, 60, 0]),
              (torch.float16, 64, 7, [1, 3], [200, 90]), (torch.bfloat16, 128, 16, [40], [80]),
              (torch.float16, 64, 8, [90, 1], [60, 30]), (torch.bfloat16, 64, 64, [150], [0]))]
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    x = torch.randn(512, 512, device="cuda")
    want = x @ x
    plain = ragged([2, 3], [70, 9], dtype=torch.float32, H=64)
    y, tol = paged_attn64(plain)
    d = plain.to("cuda")
    for i in range(20):
        for r in probs:
            flush.zero_()                          # pages and tables come from memory: the copies take their time
            sdpa.sdpa_paged_attn(r.q, r.kp, r.vp, r.table, r.kv_lens, cu_new=r.cu)
            same = torch.equal(x @ x, want)        # the next kernel on those SMs has its shared memory to itself
            got = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu).cpu().double()
            print("STATUS", int(same and bool(((got - y).abs() <= tol).all())), sdpa.sdpa_query_status())
    print("AFTER", sdpa.sdpa_query_status())
""")


@pytest.mark.parametrize("limit", ["1", "300", "900", "2000"])
def test_waits_that_expire_behind_the_last_copy(limit):
    """Shares of few tiles, whose copies are all issued before the first is there: a wait that expires
    then leaves no copy behind.  Whether it expires at all depends on the limit; the call ends, says
    so, and what runs next on the GPU is right."""
    out = subprocess.run([sys.executable, "-c", LATE.format(root=ROOT, tests=os.path.join(ROOT, "tests"))],
                         env=dict(os.environ, SDPA_WAIT_LIMIT_NS=limit), capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = [line.split() for line in out.stdout.splitlines()]
    got = [(int(line[1]), int(line[2])) for line in lines if line[0] == "STATUS"]
    assert len(got) == 120 and all(right and status in (0, sdpa.SDPA_ERR_TIMEOUT) for right, status in got), got
    assert limit != "1" or all(status == sdpa.SDPA_ERR_TIMEOUT for _, status in got)
    assert lines[-1] == ["AFTER", "0"]


@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64), (FP, 64)])
def test_a_serving_loop_keeps_one_workspace(dtype, H):
    """Allocated once, for the first step's single tokens, it takes larger batches, drafts, prompts and
    long sequences; nothing behind it is written."""
    import ctypes
    first = ragged([1, 1], [5, 9], dtype=dtype, H=H, page=16, Nq=8, Nkv=2, uniform=True).to("cuda")
    p = sdpa.make_paged_params(first.kp, first.vp, first.table, first.kv_lens, 2, 8)
    need = sdpa.lib().sdpa_paged_workspace_size(ctypes.byref(p))
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for new, past, page in (([1, 1], [5, 9], 16), ([1] * 30, [40] * 30, 16), ([1, 1], [9000, 20000], 16), ([4, 3], [100, 9], 16),
                            ([9, 5, 6], [300, 0, 1000], 7), ([200, 1, 33], [0, 700, 90], 64)):
        r = ragged(new, past, dtype=dtype, H=H, page=page, Nq=8, Nkv=2, seed=len(new))
        want, tol = paged_attn64(r)
        y = attn(r, workspace=room[:need])
        assert ((y.cpu().double() - want).abs() <= tol).all(), sdpa.sdpa_last_kernel_name()
    assert (room[need:] == 0xA5).all()


QUERY = textwrap.dedent("""
    import sys, time, torch
    sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
    from paged_reference import ragged
    from scaled_dot_product_gb300 import sdpa

    def median(n=300):
        ts = []
        for _ in range(n):
            t = time.perf_counter()
            sdpa.sdpa_query_status()
            ts.append(time.perf_counter() - t)
        return sorted(ts)[n // 2]

    torch.zeros(1, device="cuda")
    median(50)
    alone = median()
    # one call of each kind, each with one bad page or position: reported once by the query that follows
    seen = []
    for dtype, new in ((torch.bfloat16, [1, 1]), (torch.bfloat16, [90, 1]), (torch.float32, [1, 1])):
        r = ragged(new, [300, 50], dtype=dtype)
        r.table[1, 0] = -1
        d = r.to("cuda")
        sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu)
        seen += [sdpa.sdpa_query_status(), sdpa.sdpa_query_status()]
    r.table[1] = -1
    d = r.to("cuda")
    sdpa.sdpa_paged_append(d.k, d.v, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu)
    seen += [sdpa.sdpa_query_status(), sdpa.sdpa_query_status()]
    x, w = torch.randn(1, 2, 3, 64, device="cuda"), torch.ones(64, device="cuda")
    c = torch.ones(4, 32, device="cuda")
    pos = torch.tensor([[0, 1, 9]], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                    # captured, not run: nothing to report yet
        sdpa.sdpa_qk_norm_rotary(x, x, w, w, c, c, pos)
    seen.append(sdpa.sdpa_query_status())
    for _ in range(2):
        graph.replay()
        seen += [sdpa.sdpa_query_status(), sdpa.sdpa_query_status()]
    print("SEEN", *seen)
    print("TIMES", alone, median())
""")


def test_the_status_query_reads_what_the_process_has_used():
    """In a process that made no norm or paged call the query takes no longer than before there were
    any; what each of them reports still arrives, of replayed graphs too."""
    out = subprocess.run([sys.executable, "-c", QUERY.format(root=ROOT, tests=os.path.join(ROOT, "tests"))], capture_output=True,
                         text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = {line.split()[0]: line.split()[1:] for line in out.stdout.splitlines()}
    bad = str(sdpa.SDPA_ERR_INVALID)
    assert lines["SEEN"] == [bad, "0"] * 4 + ["0"] + [bad, "0"] * 2
    alone, after = (float(x) for x in lines["TIMES"])
    # four words are read by themselves, nine with all kernels used
    assert alone < 0.7 * after, (alone, after)
