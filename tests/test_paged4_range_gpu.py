"""Attention over a 4-bit cache where weights and scales lie far apart: the few-row kernel's value products
have fp16 operands (a weight times its key's scale), whose range has to follow the largest product of each row and
group of channels, not the largest weight and the largest scale.

The tolerances are paged4_attn64's.  An operand in fp16's normal range is off by 2^-11 of itself at most, which its
"codes" term holds.  One far below the largest product of its row and group is off by 2^-24 of that at most: over T keys and
codes of up to 15 by T 2^-24 15 max(p scale) <= 2 T 2^-24 sum(p 8 scale), which the term of T fp32 sums holds."""
import pytest
import torch

from paged4_reference import pack, paged4_attn64, ragged4, unpack64
from scaled_dot_product_gb300 import sdpa

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def problem(dtype, H, q, k, v, new=1):
    """One sequence of one key head: q (new, Nq, H), k and v (T, H) in fp32, by key position."""
    T = k.shape[0]
    r, _, _, _ = ragged4([new], [T - new], dtype=dtype, H=H, Nq=q.shape[1], Nkv=1, page=16, seed=1)
    j = torch.arange(T)
    ids, at = r.table[0].long()[j // 16], j % 16
    pools = []
    for x in (k, v):
        pool = torch.zeros(r.kp.shape, dtype=torch.float32)
        pool[ids, 0, at] = x
        pools.append(pack(pool.to(dtype), dtype))
    r.q = q.to(dtype)
    r.kp, _ = unpack64(pools[0], H, dtype)
    r.vp, vs = unpack64(pools[1], H, dtype)
    return r, pools[0], pools[1], vs


def check(r, k4, v4, vs):
    want, tol = paged4_attn64(r, vs)
    y = sdpa.sdpa_paged4_attn(r.q.cuda(), k4.cuda(), v4.cuda(), r.table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda())
    assert sdpa.sdpa_last_kernel_name().startswith("paged4_mma") and sdpa.sdpa_query_status() == 0
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()


def rows(gen, n, Nq, H, at=1.0, spread=0.5):
    """Queries that lean towards all channels alike: a key of c in every channel scores about c sqrt(H) at with each."""
    return at + spread * torch.randn(n, Nq, H, generator=gen)


@pytest.mark.parametrize("H", [128, 64])
@pytest.mark.parametrize("dtype,octaves", [(t, o) for t in (BF, HF) for o in (12, 16, 20, 22, 24)] + [(BF, 30), (BF, 50)])
def test_a_large_value_of_no_weight(dtype, octaves, H):
    """One key whose values are 2^octaves the others' and whose score is some 60 octaves below the largest: early, late,
    in the middle, in the first group of channels or in all."""
    g = torch.Generator().manual_seed(octaves)
    for at in (0, 700, 1999):
        for groups in (1, H // 32):
            q = rows(g, 1, 8, H)
            k, v = torch.randn(2000, H, generator=g), torch.randn(2000, H, generator=g)
            k[at] = -45.0 / H ** 0.5
            if dtype == HF:
                v *= 2.0 ** -11
            v[at, :32 * groups] *= 2.0 ** octaves
            check(*problem(dtype, H, q, k, v))


@pytest.mark.parametrize("dtype,octaves,H", [(BF, 20, 128), (BF, 40, 64), (HF, 12, 128), (HF, 14, 64)])
def test_many_large_values_of_no_weight(dtype, octaves, H):
    """Small values with all the weight at both ends of a sequence, thousands of large ones without any between them."""
    g = torch.Generator().manual_seed(octaves)
    for n in (1, 2, 4 if H == 64 else 2):
        k, v = 0.5 * torch.randn(6000, H, generator=g), torch.randn(6000, H, generator=g)
        k[20:5700] = -45.0 / H ** 0.5
        v[:20] *= 2.0 ** -octaves
        v[5700:] *= 2.0 ** -octaves
        check(*problem(dtype, H, rows(g, n, 8, H), k, v, n))


@pytest.mark.parametrize("H", [128, 64])
@pytest.mark.parametrize("dtype,octaves", [(t, o) for t in (BF, HF) for o in (0, 6, 8, 12, 16)] + [(BF, 24), (BF, 40)])
def test_a_group_of_small_values_beside_a_large_one(dtype, octaves, H):
    """A key some 15 octaves of weight ahead of thousands, and channels 32 .. 63 of all keys 2^-octaves the others'."""
    g = torch.Generator().manual_seed(octaves)
    for first in (0, 3000):
        for dominant in (1.0, 2.0 ** -6):          # its value, beside the others'
            q = rows(g, 1, 8, H, spread=0.05)
            k, v = torch.zeros(6000, H), torch.randn(6000, H, generator=g)
            k[first] = 15 * 0.6931 / H ** 0.5
            v[first] *= dominant
            if dtype == HF:
                v *= 4.0
            v[:, 32:64] *= 2.0 ** -octaves
            check(*problem(dtype, H, q, k, v))


@pytest.mark.parametrize("H", [128, 64])
@pytest.mark.parametrize("octaves", [-80, -45, -30, 30, 100, 108])
def test_bf16_values_of_any_size(H, octaves):
    g = torch.Generator().manual_seed(3)
    for n in (1, 2):
        k, v = torch.randn(900, H, generator=g), torch.randn(900, H, generator=g) * 2.0 ** octaves
        check(*problem(BF, H, rows(g, n, 4, H), k, v, n))


@pytest.mark.parametrize("dtype,H", [(BF, 128), (BF, 64), (HF, 128), (HF, 64)])
def test_rows_that_lean_on_different_keys_and_groups(dtype, H):
    """Half of the heads give their weight to a key with one large group of channels, the others to one with another, each group
    far smaller in the other key; thousands of small keys beside them."""
    g = torch.Generator().manual_seed(5)
    low = 2.0 ** (-9 if dtype == HF else -22)
    q = 0.05 * torch.randn(1, 8, H, generator=g)
    q[:, :4, :H // 2] += 1.0
    q[:, 4:, H // 2:] += 1.0
    k, v = torch.zeros(3000, H), torch.randn(3000, H, generator=g) * low * 2.0 ** -4
    for at, half in ((10, 0), (40, 1)):
        k[at, half * H // 2:(half + 1) * H // 2] = 40.0 / H ** 0.5
        v[at] = torch.randn(H, generator=g)
        v[at, 32 * half:32 * half + 32] *= low
    for n in (1, 2, 4 if H == 64 else 2):
        check(*problem(dtype, H, q.expand(n, 8, H), k, v, n))


@pytest.mark.parametrize("dtype,H", [(BF, 128), (HF, 64)])
def test_weights_fall_as_scales_grow(dtype, H):
    """Products of weight and scale alike, each factor over many octaves, and in the other order; and products that grow
    along the sequence by far more than fp16's range."""
    g = torch.Generator().manual_seed(7)
    top = 12 if dtype == HF else 50
    for kind in range(4):
        e = torch.arange(1500) * top / 1500
        if kind == 1:
            e = e.flip(0)
        if kind == 2:
            e = e[torch.randperm(1500, generator=g)]
        q = rows(g, 1, 8, H, spread=0.0)
        k = (-e * 0.6931 / H ** 0.5).view(-1, 1).repeat(1, H) * (0.0 if kind == 3 else 1.0)
        v = torch.randn(1500, H, generator=g) * 2.0 ** (e - (8 if dtype == HF else 30)).view(-1, 1)
        check(*problem(dtype, H, q, k, v))


@pytest.mark.parametrize("octaves", [18, 24, 25, 26, 28])
@pytest.mark.parametrize("H", [64, 128])
def test_a_maximum_that_moves_far_within_a_tile(H, octaves):
    """Chunks in fp16: scores of the first half of a tile of 128 keys lie 7 octaves above the maximum so far and those of the second
    half `octaves` above it, whose values are zero: the output is what the first half's weights, made anew for the larger
    maximum, are worth.  Such a weight is rounded to fp16 twice, by 2^-25 of the maximum's power of two each where it is
    subnormal, which is at most 2^-23 of the largest weight, and not by more than itself."""
    q = torch.ones(40, 4, H)                   # 160 rows: each has every tile
    k, v = torch.zeros(300, H), torch.zeros(300, H)
    v[:192] = 1000 + 300 * torch.randn(192, H, generator=torch.Generator().manual_seed(1))
    score = torch.zeros(300)
    score[128:192], score[192:200] = 7.0, octaves
    k += (score * 0.6931 / H ** 0.5).view(-1, 1)
    r, k4, v4, vs = problem(HF, H, q, k, v, 40)
    want, tol = paged4_attn64(r, vs, operands="values")
    p = 2.0 ** (score.double() - octaves)
    far = torch.minimum(1.01 * p, torch.tensor(2.0 ** -23, dtype=torch.float64))
    tol = tol + (far @ v.abs().double() * 1.01 / p.sum()).view(1, 1, H)
    y = sdpa.sdpa_paged4_attn(r.q.cuda(), k4.cuda(), v4.cuda(), r.table.cuda(), r.kv_lens.cuda(), cu_new=r.cu.cuda(), max_new=40)
    assert sdpa.sdpa_last_kernel_name().startswith("paged4_tc_f16") and sdpa.sdpa_query_status() == 0
    err = (y.cpu().double() - want).abs()
    assert (err <= tol).all(), (err / tol).max()
