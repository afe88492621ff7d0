"""The page tables, the 4-bit append and the attention fed with one another's outputs, step by step: tables equal to
their definition, records equal to the bit in the slots that the tables name, and the attention equal to the bit to a call
over a cache that the host lays out anew, and within paged4_attn64's bound, term by term."""
import types

import pytest
import torch

from paged4_reference import pack, paged4_attn64, row_bytes, tables_of, unpack64
from scaled_dot_product_gb300 import sdpa

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dtype,H,page", [(BF, 128, 16), (HF, 128, 5), (BF, 64, 8), (HF, 64, 6), (FP, 64, 16), (BF, 96, 4)])
def test_a_served_batch_in_every_bit(dtype, H, page):
    Nq, Nkv, pages, width, B = 4, 2, 60, 24, 4
    g = torch.Generator().manual_seed(page)
    rb = row_bytes(H, dtype)
    kp, vp = (torch.full((pages, Nkv, page, rb), 255, dtype=torch.uint8, device="cuda") for _ in range(2))      # NaN where nothing is written
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free, count = torch.randperm(pages, generator=g).to(torch.int32).cuda(), torch.tensor([pages], dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kept = [[torch.empty(0, Nkv, rb, dtype=torch.uint8)] * 2 for _ in range(B)]          # records of each sequence
    for new in ([37, 5, 0, 1], [1, 1, 1, 1], [1, 1, 3, 2], [1, -1, 20, 1], [2, 9, 1, 1], [1, 1, 1, -1], [1, 1, 1, 1]):
        n = [max(x, 0) for x in new]
        tokens = sum(n) + 2
        want, _ = tables_of(table.tolist(), lens.tolist(), new, free.tolist(), count.item(), page, tokens)
        _, cu, _, slots, _ = out = sdpa.sdpa_paged_tables(table, lens, torch.tensor(new, dtype=torch.int32, device="cuda"), free, count,
                                                          page_size=page, tokens=tokens, kv_lens=lens, free_count_out=count)
        got = dict(zip(("kv_lens", "cu_new", "positions", "slots", "free_count_out"), out), page_table=table, free_pages=free)
        assert {name: t.tolist() for name, t in got.items()} == want
        q = torch.randn(tokens, Nq, H, generator=g).to(dtype)
        k, v = (torch.randn(tokens, Nkv, H, generator=g).to(dtype) for _ in range(2))
        before = [kp.cpu(), vp.cpu()]
        sdpa.sdpa_paged4_append(k.cuda(), v.cuda(), kp, vp, slots)
        live = slots.cpu()[:sum(n)]
        for was, pool, x in zip(before, (kp, vp), (k, v)):
            was[live // page, :, live % page] = pack(x, dtype)[:sum(n)]
            assert torch.equal(pool.cpu(), was)
        t = 0
        for b in range(B):
            for i, x in enumerate((k, v)):
                kept[b][i] = pack(x[:0], dtype) if new[b] < 0 else torch.cat((kept[b][i], pack(x[t:t + n[b]], dtype)))
            t += n[b]
        # the same keys in pages of the host's own
        T = [len(x[0]) for x in kept]
        need = [-(-x // page) for x in T]
        mine = torch.full((B, width), -1, dtype=torch.int32)
        pools = [torch.zeros(sum(need) + 1, Nkv, page, rb, dtype=torch.uint8) for _ in range(2)]
        at = 0
        for b in range(B):
            mine[b, :need[b]] = torch.arange(at, at + need[b]).flip(0).to(torch.int32)
            j = torch.arange(T[b])
            for i in range(2):
                pools[i][mine[b].long()[j // page], :, j % page] = kept[b][i]
            at += need[b]
        y = sdpa.sdpa_paged4_attn(q.cuda(), kp, vp, table, lens, cu_new=cu, max_new=max(n)).cpu()
        kernel = sdpa.sdpa_last_kernel_name()
        again = sdpa.sdpa_paged4_attn(q.cuda(), pools[0].cuda(), pools[1].cuda(), mine.cuda(), torch.tensor(T, dtype=torch.int32).cuda(),
                                      cu_new=cu, max_new=max(n)).cpu()
        assert sdpa.sdpa_query_status() == 0 and torch.equal(y[:sum(n)], again[:sum(n)])
        K, (V, S) = unpack64(pools[0], H, dtype)[0], unpack64(pools[1], H, dtype)
        r = types.SimpleNamespace(new=n, lens=T, Nq=Nq, Nkv=Nkv, H=H, Hv=H, page=page, dtype=dtype, q=q, kp=K, vp=V, table=mine,
                                  tokens=sum(n))
        ref, tol = paged4_attn64(r, S, operands="values" if "_tc_" in kernel else "codes")
        err = (y[:sum(n)].double() - ref).abs()
        assert (err <= tol).all(), ((err / tol).max(), kernel)
