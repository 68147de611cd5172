"""q8_kv_plan against a plain loop over sequences and tokens (whole numbers, so equal)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAD, NO_PAGE = 0x8, 0x10


def reference(table, lens, new, ps, pages, T, free=None, count=0):
    """What the call leaves: (table, starts, slots, positions, lens_out, left, status)."""
    table = table.copy()
    B, width = table.shape
    room = width * ps
    slots, pos = np.full(T, -1, dtype=np.int64), np.zeros(T, dtype=np.int32)
    starts, out, status = [], [], 0
    row, taken = 0, 0
    if free is not None:
        c = min(max(count, 0), len(free))
        status |= BAD if c != count else 0
        count = c
    for b in range(B):
        starts.append(row)
        old = min(max(int(lens[b]), 0), room)
        n = min(max(int(new[b]), 0), room - old)
        if old != lens[b] or n != new[b]:
            status |= BAD
        if row + n > T:
            n, status = T - row, status | BAD
        had = -(-old // ps)
        for p in range(old, old + n):
            e = p // ps
            if free is not None and e >= had and p % ps == 0:
                if taken < count:
                    pg = int(free[count - 1 - taken])
                    if not 0 <= pg < pages:
                        pg, status = -1, status | BAD
                else:
                    pg, status = -1, status | NO_PAGE
                taken += 1
                table[b, e] = pg
            elif free is None or e < had:
                pg = int(table[b, e])
                if not 0 <= pg < pages:
                    pg, status = -1, status | BAD
            pos[row] = p
            if pg >= 0:
                slots[row] = pg * ps + p % ps
            row += 1
        out.append(old + n)
    left = max(count - taken, 0) if free is not None else None
    return table, np.array(starts + [row]), slots, pos, np.array(out, dtype=np.int32), left, status


def run(table, lens, new, ps, pages, T, free=None, count=0, in_place=False, stream=None):
    from block_quantized_int8_gb300 import q8
    ref = reference(table, lens, new, ps, pages, T, free, count)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    tab, ln, nw = dev(table), dev(lens), dev(new)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if free is not None:
        kw = dict(free_pages=dev(free), free_count=dev([count]))
        if in_place:
            kw["free_left"] = kw["free_count"]
    if in_place:
        kw["lens_out"] = ln
    torch.cuda.synchronize()
    starts, slots, pos, out, left = q8.q8_kv_plan(tab, ln, nw, ps, pages, T, dev_status=st, stream=stream, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == ref[6]
    for got, want in zip((tab, starts, slots, pos, out), ref[:5]):
        assert np.array_equal(got.cpu().numpy(), want)
    if free is not None:
        assert int(left.item()) == ref[5]
        assert np.array_equal(kw["free_pages"].cpu().numpy(), free)
    else:
        assert left is None
    return ref


def state(B, ps, max_len, max_new, seed, spare=5, some=1.0):
    r = np.random.default_rng(seed)
    lens = r.integers(0, max_len + 1, B)
    new = np.where(r.random(B) < some, r.integers(0, max_new + 1, B), 0)
    width = -(-(max_len + max_new) // ps)
    have = -(-lens // ps)
    pages = int((-(-(lens + new) // ps)).sum()) + spare
    order = r.permutation(pages)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    return table, lens, new, pages, order[at:]


@pytest.mark.parametrize("B,ps,max_len,max_new,pad", [(1, 16, 0, 1, 0), (1, 16, 100, 1, 0), (48, 16, 600, 1, 0), (7, 32, 90, 70, 5),
                                                      (1, 64, 10, 9000, 0), (300, 32, 400, 40, 1000), (511, 16, 40, 3, 0), (512, 16, 40, 3, 1),
                                                      (513, 16, 40, 30, 2), (1500, 16, 33, 17, 0), (3, 1024, 5000, 3000, 77)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_slots_and_positions(B, ps, max_len, max_new, pad, in_place):
    table, lens, new, pages, free = state(B, ps, max_len, max_new, B + ps)
    run(table, lens, new, ps, pages, int(new.sum()) + pad, free, len(free), in_place)


@pytest.mark.parametrize("B,T", [(1, 1), (40, 700), (600, 9000)])
def test_a_complete_table(B, T):
    r = np.random.default_rng(B)
    table = r.permutation(B * 8).reshape(B, 8)
    lens = r.integers(0, 100, B)
    new = r.integers(0, 29, B)
    while new.sum() > T:
        new //= 2
    run(table, lens, new, 16, B * 8, T)
    table[B // 2, :] = -1
    table[0, 7] = B * 8
    lens[0], new[0] = 112, min(5, int(new[0]))
    run(table, lens, new, 16, B * 8, T)


@pytest.mark.parametrize("in_place", [False, True])
def test_sequences_without_new_tokens(in_place):
    table, lens, new, pages, free = state(200, 16, 300, 200, 3, some=0.1)
    run(table, lens, new, 16, pages, int(new.sum()) + 3, free, len(free), in_place)
    run(table, lens, 0 * new, 16, pages, 0, free, len(free), in_place)
    run(table, lens, 0 * new, 16, pages, 6000, free, len(free), in_place)


def test_the_list_runs_out():
    table, lens, new, pages, free = state(30, 16, 100, 100, 4)
    need = len(free) - 5
    for count in (0, 1, need // 2, need - 1, need):
        status = run(table, lens, new, 16, pages, int(new.sum()), free, count)[6]
        assert bool(status & NO_PAGE) == (count < need)
    run(table, lens, new, 16, pages, int(new.sum()), free[:0], 0)


def test_bad_lengths_counts_and_pages():
    table, lens, new, pages, free = state(30, 16, 100, 50, 5)
    T = int(new.sum()) + 2000
    for i, v in ((3, -5), (4, 10 ** 6), (5, -2 ** 31), (6, 2 ** 31 - 1)):
        bad = lens.copy()
        bad[i] = v
        assert run(table, bad, new, 16, pages, T, free, len(free))[6] & BAD
        bad = new.copy()
        bad[i] = v
        assert run(table, lens, bad, 16, pages, T, free, len(free))[6] & BAD
    for count in (-1, len(free) + 1, 2 ** 31 - 1):
        assert run(table, lens, new, 16, pages, T, free, count)[6] & BAD
    f = free.copy()
    f[-1], f[-2] = pages, -7
    assert run(table, lens, new, 16, pages, T, f, len(f))[6] & BAD
    # fewer rows than tokens
    for T in (0, 1, int(new[:10].sum()) + 1, int(new.sum()) - 1):
        assert run(table, lens, new, 16, pages, T, free, len(free))[6] & BAD


def test_replayed_steps_take_page_after_page():
    """A captured step, its lengths and free count updated in place, run again and again."""
    from block_quantized_int8_gb300 import q8
    B, ps, width = 5, 16, 6
    r = np.random.default_rng(6)
    new = np.array([1, 3, 0, 7, 16])
    pages = B * width
    table, lens, count = np.full((B, width), -1), np.zeros(B, dtype=np.int64), pages
    free = r.permutation(pages)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    tab, ln, nw, fr, ct = dev(table), dev(lens), dev(new), dev(free), dev([count])
    out = [torch.empty(B + 1, dtype=torch.int32, device="cuda"), torch.empty(30, dtype=torch.int64, device="cuda"),
           torch.empty(30, dtype=torch.int32, device="cuda")]
    call = lambda: q8.q8_kv_plan(tab, ln, nw, ps, pages, 30, fr, ct, ct, *out, lens_out=ln)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(6):
        graph.replay()
        torch.cuda.synchronize()
        table, starts, slots, pos, lens, count, _ = reference(table, lens, new, ps, pages, 30, free, count)
        for got, want in zip((tab, *out, ln), (table, starts, slots, pos, lens)):
            assert np.array_equal(got.cpu().numpy(), want)
        assert int(ct.item()) == count


def test_no_sequences():
    from block_quantized_int8_gb300 import q8
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    starts, slots, pos, out, _ = q8.q8_kv_plan(torch.empty((0, 4), dtype=torch.int32, device="cuda"), e, e, 16, 4, 10)
    assert starts.tolist() == [0] and slots.tolist() == [-1] * 10 and pos.tolist() == [0] * 10 and out.shape == (0,)


def test_on_another_stream():
    s = torch.cuda.Stream()
    table, lens, new, pages, free = state(50, 16, 100, 200, 8)
    with torch.cuda.stream(s):
        run(table, lens, new, 16, pages, int(new.sum()), free, len(free))
    run(table, lens, new, 16, pages, int(new.sum()), free, len(free), stream=s)


@pytest.mark.parametrize("B,width,count", [(0, 4, 0), (3, 0, 0), (0, 4, 2), (3, 0, -1)])
def test_an_empty_free_list_beside_an_empty_table(B, width, count):
    """An empty list is a list all the same: what is left of it is given."""
    from block_quantized_int8_gb300 import q8
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    zeros = torch.zeros(B, dtype=torch.int32, device="cuda")
    st, left = i32(0), i32(77)
    starts, slots, pos, out, got = q8.q8_kv_plan(torch.empty((B, width), dtype=torch.int32, device="cuda"), zeros, zeros, 16, 4, 3,
                                                 free_pages=i32(), free_count=i32(count), free_left=left, dev_status=st)
    assert starts.tolist() == [0] * (B + 1) and slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and out.tolist() == [0] * B
    assert got is left and left.tolist() == [0] and int(st.item()) == (BAD if count else 0)
