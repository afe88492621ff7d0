"""The attention over a paged cache where a query, a key, a value or a sink is not a number: rows that
it enters are not numbers either, however the batch is cut, and the other rows are as ever."""
import pytest
import torch

from paged_reference import paged_attn64, ragged
from scaled_dot_product_gb300 import sdpa

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


# type, head size, page, new tokens of the sequence, the kernel
KERNELS = [(BF, 128, 16, 1, "paged_mma"), (HF, 64, 7, 3, "paged_mma"), (BF, 128, 16, 40, "paged_tc"), (HF, 64, 8, 150, "paged_tc"),
           (FP, 64, 16, 1, "paged_simt"), (FP, 128, 24, 5, "paged_simt"), (BF, 96, 16, 2, "paged_simt")]
# keys beside the new tokens: units that one block holds whole, units joined from a few partial
# results and from many
PAST = [0, 2, 30, 250, 600, 9000]


def problem(dtype, H, page, new, past, seed=0):
    """The sequence in question between two others."""
    return ragged([1, new, 2], [20, past, 300], dtype=dtype, H=H, page=page, Nq=4, Nkv=2, seed=past + seed)


def check(r, hint, sink=None, **kw):
    """NaN exactly where the definition has it, and the definition's values elsewhere."""
    want, tol = paged_attn64(r, sink=sink, **{n: x for n, x in kw.items() if n != "causal"})
    d = r.to("cuda")
    y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, max_new=hint,
                             head_sink=None if sink is None else sink.cuda(), **kw).cpu().double()
    assert sdpa.sdpa_query_status() == 0
    bad = want.isnan()
    assert bad.any() and not bad.all()
    assert y[bad].isnan().all(), (sdpa.sdpa_last_kernel_name(), (bad & ~y.isnan()).nonzero()[:4].tolist(), y[bad & ~y.isnan()][:4])
    assert ((y - want).abs()[~bad] <= tol[~bad]).all(), sdpa.sdpa_last_kernel_name()


def place(r, b, j):
    """Page and slot of key j of sequence b."""
    return r.table[b, j // r.page].item(), j % r.page


@pytest.mark.parametrize("dtype,H,page,new,kernel", KERNELS)
@pytest.mark.parametrize("past", PAST)
def test_a_query(dtype, H, page, new, kernel, past):
    r = problem(dtype, H, page, new, past)
    r.q[1 + new // 2, 2, 5] = NAN                      # one head of one token of the middle sequence
    check(r, new)
    assert sdpa.sdpa_last_kernel_name().startswith(kernel)


@pytest.mark.parametrize("dtype,H,page,new,kernel", KERNELS)
@pytest.mark.parametrize("past", PAST)
def test_a_key(dtype, H, page, new, kernel, past):
    """Key 0 is one that all rows of its sequence admit."""
    r = problem(dtype, H, page, new, past)
    pg, slot = place(r, 1, 0)
    r.kp[pg, 1, slot, 3] = NAN
    check(r, new)
    r = problem(dtype, H, page, new, past)             # every key of one head
    for j in range(r.lens[1]):
        pg, slot = place(r, 1, j)
        r.kp[pg, 0, slot] = NAN
    check(r, new)


@pytest.mark.parametrize("dtype,H,page,new,kernel", KERNELS)
@pytest.mark.parametrize("past", PAST)
def test_a_value(dtype, H, page, new, kernel, past):
    """One channel of key 0: that channel of the outputs, no other."""
    r = problem(dtype, H, page, new, past)
    pg, slot = place(r, 1, 0)
    r.vp[pg, 1, slot, 7] = NAN
    check(r, new)


@pytest.mark.parametrize("dtype,H,page,new,kernel", KERNELS)
@pytest.mark.parametrize("past", PAST)
def test_a_sink(dtype, H, page, new, kernel, past):
    r = problem(dtype, H, page, new, past)
    check(r, new, sink=torch.tensor([0.5, NAN, -1.0, 2.0]).to(dtype))


@pytest.mark.parametrize("dtype,H,page,new,kernel", KERNELS)
def test_rows_without_keys_stay_zero(dtype, H, page, new, kernel):
    """No admitted key: zeros, whatever the query and the sink hold."""
    r = ragged([1, new, 2], [20, -new, 300], dtype=dtype, H=H, page=page, Nq=4, Nkv=2, seed=3)
    r.q[1] = NAN
    sink = torch.tensor([0.5, NAN, -1.0, 2.0]).to(dtype)
    d = r.to("cuda")
    y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, max_new=new, head_sink=sink.cuda())
    assert not y[1:1 + new].any() and y[0, 1].isnan().all()


@pytest.mark.parametrize("dtype,H,page,new,kernel", KERNELS)
@pytest.mark.parametrize("past", PAST[1:])
def test_an_infinite_key(dtype, H, page, new, kernel, past):
    """A score of +inf has no softmax, one of -inf beside finite ones has weight 0: a row is NaN by the
    sign of its own query's channel, and by nothing else."""
    r = problem(dtype, H, page, new, past)
    pg, slot = place(r, 1, 0)
    r.kp[pg, 1, slot, 3] = float("inf")
    d = r.to("cuda")
    y = sdpa.sdpa_paged_attn(d.q, d.kp, d.vp, d.table, d.kv_lens, cu_new=d.cu, max_new=new).cpu()
    want = (r.q[1:1 + new, 2:, 3] > 0)[..., None].expand(new, 2, H)
    assert torch.equal(y[1:1 + new, 2:].isnan(), want), sdpa.sdpa_last_kernel_name()
    assert not y[:, :2].isnan().any() and not y[0].isnan().any() and not y[1 + new:].isnan().any()
