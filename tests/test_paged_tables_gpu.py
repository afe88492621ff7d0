"""sdpa_paged_tables against its definition on Python lists: every output is a whole number and equal."""
import random

import pytest
import torch

from paged4_reference import tables_of
from scaled_dot_product_gb300 import sdpa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def problem(past, new, page, *, spare=None, width_extra=2, tokens_extra=3, seed=0):
    """A table of shuffled pages and a list with as many spare pages as the step takes, or `spare`."""
    rng = random.Random(seed)
    pages_of = lambda t: -(-max(t, 0) // page)
    need = [pages_of(p) for p in past]
    grow = sum(pages_of(p + max(n, 0)) - pages_of(p) for p, n in zip(past, new))
    spare = grow if spare is None else spare
    order = list(range(sum(need) + spare))
    rng.shuffle(order)
    width = max([pages_of(p + max(n, 0)) for p, n in zip(past, new)] + [0]) + width_extra
    table, at = [], 0
    for c in need:
        table.append(order[at:at + c] + [-7] * (width - c))
        at += c
    free = order[at:] + [rng.randrange(len(order)) for _ in range(at)]       # what lies above the top is of no account
    return dict(table=table, past=list(past), new=list(new), free=free, count=spare, page=page,
                tokens=sum(max(n, 0) for n in new) + tokens_extra)


def call(p, in_place=False, stride=None, **kw):
    B, width = len(p["table"]), len(p["table"][0]) if p["table"] else 0
    table = torch.full((B, stride or width), -9, dtype=torch.int32, device="cuda")[:, :width]
    if B and width:
        table.copy_(ints(p["table"]))
    past, new, free, count = ints(p["past"]), ints(p["new"]), ints(p["free"]), ints([p["count"]])
    out = dict(kv_lens=past, free_count_out=count) if in_place else {}
    r = sdpa.sdpa_paged_tables(table, past, new, free, count, page_size=p["page"], tokens=p["tokens"], **out, **kw)
    names = ("kv_lens", "cu_new", "positions", "slots", "free_count_out")
    got = dict(zip(names, r), page_table=table, free_pages=free)
    status = sdpa.sdpa_query_status()
    return {n: t.tolist() for n, t in got.items()}, status, sdpa.sdpa_last_error() if status else ""


def check(p, **kw):
    want, said = tables_of(p["table"], p["past"], p["new"], p["free"], p["count"], p["page"], p["tokens"])
    got, status, text = call(p, **kw)
    for name, value in want.items():
        assert got[name] == value, name
    assert (status == sdpa.SDPA_ERR_INVALID) == bool(said), (said, text)
    if said:
        assert any(word in text for word in said), (said, text)
    return want


CASES = [
    ([0], [1], 16), ([15, 16, 17, 0], [1, 1, 1, 1], 16), ([0, 0, 0], [5, 0, 40], 8), ([7, 0, 30], [0, 0, 0], 10),
    ([100, 33, 7], [-1, 1, -1], 16), ([100, 33, 7], [-1, 200, 3], 1), ([5] * 300, [1] * 300, 4),
    ([i * 7 % 90 for i in range(1500)], [(i * 13) % 9 - 1 for i in range(1500)], 24),
    ([i % 50 for i in range(8192)], [1 if i % 5 else -1 for i in range(8192)], 16),
    ([0, 9], [9000, 3], 64), ([1000] * 40, [700 + i for i in range(40)], 100), ([3, 5], [-4, -1], 2),
    ([0] * 257, [0] * 256 + [2], 16),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("past,new,page", CASES)
def test_against_the_definition(past, new, page, in_place):
    check(problem(past, new, page, seed=len(past)), in_place=in_place)


def test_a_wide_table_and_more_free_pages_than_needed():
    check(problem([20, 5, 64], [3, 100, -1], 16, spare=50), stride=40)
    check(problem([20, 5, 64], [3, 100, -1], 16, tokens_extra=0))


def test_pages_run_out():
    want = check(problem([10, 0, 16], [1, 60, 20], 16, spare=3))
    assert want["free_count_out"][0] < 0 and -1 in want["slots"]
    check(problem([10, 0, 16], [1, 60, 20], 16, spare=0))
    check(problem([10, 0, 50], [1, 60, -1], 16, spare=1))          # what an ended sequence gives back is taken at once


def test_data_out_of_range_is_cut_off_and_reported():
    base = problem([20, 5, 33], [3, 10, 4], 16, spare=20)
    for change in (dict(past=[20, -5, 33]), dict(past=[20, 5, 10 ** 9]), dict(new=[3, 2 ** 31 - 1, 4]), dict(tokens=5), dict(tokens=0),
                   dict(count=10 ** 9), dict(count=-3), dict(new=[2 ** 31 - 1] * 3)):
        check({**base, **change})
    for entry in (-1, 10 ** 6):
        p = problem([20, 5, 33], [3, 10, -4], 16, spare=20)
        p["table"][0][1] = entry                  # a begun page
        p["table"][2][0] = entry                  # of an ended sequence: not given back
        check(p)
    p = problem([20, 5], [3, 100], 16)
    p["free"][2] = -4
    check(p)


def test_what_is_reported_names_its_cause():
    """Lengths that do not fit, and a list that would be fuller than the pool: a count beyond it, or pages given back that
    were free already."""
    base = problem([20, 5, 33], [3, 10, -4], 16, spare=20)
    full = dict(count=len(base["free"]))
    for change, says in ((dict(past=[20, 5, 10 ** 9]), "past_lens"), (dict(tokens=5), "new_lens"), (dict(count=10 ** 9), "num_pages"),
                         (full, "given back twice"), (dict(full, new=[0, 0, -1]), "free pages")):
        check({**base, **change})
        _, status, text = call({**base, **change})
        assert status == sdpa.SDPA_ERR_INVALID and says in text, (change, text)


def test_random_steps():
    rng = random.Random(7)
    for seed in range(40):
        B = rng.choice([1, 3, 30, 250, 700])
        page = rng.choice([1, 2, 7, 16, 64])
        past = [rng.randrange(0, 200) for _ in range(B)]
        new = [rng.choice([-1, 0, 1, 1, 1, rng.randrange(0, 90)]) for _ in range(B)]
        check(problem(past, new, page, seed=seed, spare=rng.choice([None, 0, 5, 4000])))


def test_empty_batches():
    p = dict(table=[], past=[], new=[], free=[1, 0], count=2, page=16, tokens=3)
    check(p)
    check(dict(table=[[]], past=[0], new=[0], free=[], count=0, page=16, tokens=0))
    check(dict(table=[[]], past=[0], new=[4], free=[], count=0, page=16, tokens=4))      # no width at all


def test_calls_in_turn_in_a_graph():
    """A captured step, replayed: the state goes from replay to replay in place, and a list that is
    refilled between them is followed."""
    p = problem([3, 30, 0], [1, 1, 1], 4, spare=40, width_extra=12)
    table, past, new, free, count = ints(p["table"]), ints(p["past"]), ints(p["new"]), ints(p["free"]), ints([p["count"]])
    out = dict(cu_new=ints([0] * 4), positions=ints([0] * 3, torch.int64), slots=ints([0] * 3, torch.int64))
    step = lambda: sdpa.sdpa_paged_tables(table, past, new, free, count, page_size=4, tokens=3, kv_lens=past, free_count_out=count,
                                          **out)
    step()                                                    # loads the module outside the capture
    start = [t.clone() for t in (table, past, free, count)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((table, past, free, count), start):
        t.copy_(s)
    for k in range(9):
        if k == 5:
            new.copy_(ints([1, -1, 2]))
        want, _ = tables_of(table.tolist(), past.tolist(), new.tolist(), free.tolist(), count.item(), 4, 3)
        graph.replay()
        got = dict(kv_lens=past, free_count_out=count, page_table=table, free_pages=free, **out)
        assert {n: t.tolist() for n, t in got.items()} == want
        if k == 5:
            new.copy_(ints([1, 1, 1]))
    assert sdpa.sdpa_query_status() == 0


def test_many_tokens_captured():
    """A step of more tokens than one cluster takes (two kernels), captured and replayed in place."""
    p = problem([5, 0, 77] * 20, [900, 700, 800] * 20, 16, spare=9000, width_extra=60)
    table, past, new, free, count = ints(p["table"]), ints(p["past"]), ints(p["new"]), ints(p["free"]), ints([p["count"]])
    T = p["tokens"]
    assert T > 45000
    out = dict(cu_new=ints([0] * 61), positions=ints([0] * T, torch.int64), slots=ints([0] * T, torch.int64))
    step = lambda: sdpa.sdpa_paged_tables(table, past, new, free, count, page_size=16, tokens=T, kv_lens=past, free_count_out=count, **out)
    start = [t.clone() for t in (table, past, free, count)]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((table, past, free, count), start):
        t.copy_(s)
    for k in range(2):
        want, _ = tables_of(table.tolist(), past.tolist(), new.tolist(), free.tolist(), count.item(), 16, T)
        graph.replay()
        got = dict(kv_lens=past, free_count_out=count, page_table=table, free_pages=free, **out)
        assert {n: t.tolist() for n, t in got.items()} == want
        new.copy_(ints([-1, 300, 1] * 20))
    assert sdpa.sdpa_query_status() == 0
    check(problem([10, 40000, 16], [1, 60000, 20], 16, spare=30))          # pages run out in the second kernel's tokens
    p = problem([20, 5], [3, 50000], 16)
    p["table"][1][0] = -1
    check(p)                                                               # a begun page that is none


def test_another_stream():
    p = problem([20, 5, 33], [3, 100, -1], 16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    want = check(p)
    with torch.cuda.stream(s):
        check(p)
    got, _, _ = call(p, stream=s)
    torch.cuda.synchronize()
    assert got == want
