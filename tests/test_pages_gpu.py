"""The page operators on the GPU against plain loops, and a beam search over an 8-bit cache with all of them together."""
from __future__ import annotations

import math
import random

import pytest
import torch

from split_bf16_gemm_swap_gb300 import fp8, layer, pages

pytestmark = pytest.mark.gpu

I32, F64, BF, FP8 = torch.int32, torch.float64, torch.bfloat16, torch.float8_e4m3fn


def gpu(x, dtype=I32):
    return torch.tensor(x, device="cuda", dtype=dtype)


def needed(n, page):
    return max(0, -(-n // page))


class Pool:
    """The operators' definitions, row by row."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.page = [list(r) for r in table], list(lens), list(refs), page
        self.width = len(table[0]) if table else 0

    def used(self, row):
        return min(needed(self.lens[row], self.page), self.width)

    def inside(self, p):
        return 0 <= p < len(self.refs)

    def fork(self, parents):
        old = [r[:self.used(i)] for i, r in enumerate(self.table)]
        rows = [old[p] if 0 <= p < len(old) else [] for p in parents]
        lens = [self.lens[p] if 0 <= p < len(old) else 0 for p in parents]
        for r in old:
            for p in r:
                if self.inside(p):
                    self.refs[p] -= 1
        for r in rows:
            for p in r:
                if self.inside(p):
                    self.refs[p] += 1
        self.table = [r + [-1] * (self.width - len(r)) for r in rows]
        self.lens = lens
        tails, again = [], []
        for i, n in enumerate(lens):
            whole = needed(n, self.page)
            p = self.table[i][whole - 1] if 0 < whole <= self.width and n % self.page else -1
            p = p if self.inside(p) else -1
            again.append(p >= 0 and p in tails)
            tails.append(p)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        src, dst, missing = [-1] * len(lens), [-1] * len(lens), 0
        for i, a in enumerate(again):
            if not a:
                continue
            if not free:
                missing += 1
                continue
            src[i], dst[i] = tails[i], free.pop(0)
            self.table[i][self.used(i) - 1] = dst[i]
            self.refs[dst[i]] = 1
            self.refs[src[i]] -= 1
        return src, dst, missing

    def extend(self, counts):
        free = [p for p, r in enumerate(self.refs) if r == 0]
        positions, slots, missing = [], [], 0
        for i, n in enumerate(counts):
            before, after = needed(self.lens[i], self.page), needed(self.lens[i] + n, self.page)
            for j in range(before, after):
                if j >= self.width:
                    missing += 1
                elif free:
                    self.table[i][j] = free.pop(0)
                    self.refs[self.table[i][j]] = 1
                else:
                    self.table[i][j] = -1
                    missing += 1
            for p in range(self.lens[i], self.lens[i] + n):
                at = self.table[i][p // self.page] if p // self.page < self.width else -1
                positions.append(p)
                slots.append(at * self.page + p % self.page if self.inside(at) else -1)
            self.lens[i] += n
        return positions, slots, missing

    def compact(self):
        total = sum(r != 0 for r in self.refs)
        movers = [p for p, r in enumerate(self.refs) if r != 0 and p >= total]
        holes = [p for p, r in enumerate(self.refs) if r == 0 and p < total]
        to = dict(zip(movers, holes))
        for i, r in enumerate(self.table):
            for j in range(self.used(i)):
                r[j] = to.get(r[j], r[j])
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        fill = [-1] * (len(self.refs) // 2 - len(movers))
        return movers + fill, holes + fill, total


def make(lens, page, pages_, seed=0, width=None, share=0):
    """Rows on shuffled pages; rows i with i % share > 0 begin with the whole pages of the row before them."""
    r = random.Random(seed)
    order = list(range(pages_))
    r.shuffle(order)
    refs, table = [0] * pages_, []
    width = max([needed(n, page) for n in lens] + [1]) + 1 if width is None else width
    for i, n in enumerate(lens):
        count = min(needed(n, page), width)
        row = []
        if share and i % share:
            row = table[-1][:min(lens[i - 1] // page, n // page, width)]
        row = row + [order.pop() for _ in range(count - len(row))]
        for p in row:
            refs[p] += 1
        table.append(row + [-1] * (width - len(row)))
    return table, refs


def on_gpu(pool):
    return gpu(pool.table).view(len(pool.table), pool.width), gpu(pool.lens), gpu(pool.refs)


def check_fork(pool, parents):
    table, lens, refs = on_gpu(pool)
    old = table.clone()
    got = pages.fork_pages(table, lens, gpu(parents), refs, pool.page)
    src, dst, missing = pool.fork(parents)
    assert torch.equal(table, old)
    assert got[0].tolist() == pool.table and got[1].tolist() == pool.lens
    assert got[2].tolist() == src and got[3].tolist() == dst and got[4].tolist() == [missing]
    assert refs.tolist() == pool.refs
    return pool


@pytest.mark.parametrize("page", [1, 16, 48])
@pytest.mark.parametrize("rows,new_rows", [(1, 1), (4, 7), (40, 24), (33, 60), (200, 300)])
def test_fork(page, rows, new_rows):
    r = random.Random(rows * page)
    lens = [r.randint(0, 5 * page) for _ in range(rows)]
    table, refs = make(lens, page, 6 * (rows + new_rows) + 5, seed=rows, share=4)
    check_fork(Pool(table, lens, refs, page), [r.randint(-1, rows) for _ in range(new_rows)])


def test_fork_without_free_pages():
    lens = [20, 33, 7]
    for spare in (0, 1, 3):
        table, refs = make(lens, 16, 6 + spare, seed=1)
        check_fork(Pool(table, lens, refs, 16), [0, 0, 1, 1, 1, 2, 2, 0])


def test_fork_takes_pages_that_it_gives_up():
    lens = [20, 33, 7]
    table, refs = make(lens, 16, 6, seed=1)
    pool = check_fork(Pool(table, lens, refs, 16), [0, 0, 0])          # the pages of rows 1 and 2
    assert all(d >= 0 for d in pool.table[1][:2])


def test_fork_of_nothing_and_to_nothing():
    table, refs = make([40, 10], 16, 9, seed=2)
    pool = check_fork(Pool(table, [40, 10], refs, 16), [])
    assert not any(pool.refs)
    empty = torch.zeros(0, 4, device="cuda", dtype=I32)
    got = pages.fork_pages(empty, gpu([]), gpu([0, -1]), gpu([0] * 9), 16)
    assert got[0].tolist() == [[-1] * 4] * 2 and got[1].tolist() == [0, 0] and got[4].tolist() == [0]


def test_fork_entries_outside_the_pool_and_rows_longer_than_the_table():
    table = [[3, 99, 1], [-4, 2, 0], [5, 6, 7]]
    refs = [1, 1, 1, 1, 0, 1, 1, 1, 0]
    check_fork(Pool(table, [40, 37, 1000], refs, 16), [1, 1, 0, 0, 2, 2])


def test_fork_into_memory_beside_the_old_table():
    lens = [20, 33, 7, 0]
    table, refs = make(lens, 16, 12, seed=1, width=4)
    pool = Pool(table, lens, refs, 16)
    old, n, r = on_gpu(pool)
    want = pool.fork([0, 0, 2, 1])
    both = torch.full((8, 11), 77, device="cuda", dtype=I32)
    for view in (lambda b: (b[:4, :4], b[:4, 4:8]), lambda b: (b[:4, 5:9], b[:4, 1:5]), lambda b: (b[4:, 2:6], b[:4, 2:6]),
                 lambda b: (b[:4, 7:11], b[1:5, :4])):
        both.fill_(77)
        a, b = view(both)
        a.copy_(old)
        counts = r.clone()
        got = pages.fork_pages(a, n, gpu([0, 0, 2, 1]), counts, 16, out=b)
        assert b.tolist() == pool.table and got[2].tolist() == want[0] and counts.tolist() == pool.refs
        assert torch.equal(a, old) and int((both == 77).sum()) == 88 - 32
    both.fill_(77)
    both[:4, 2:6].copy_(old)
    want = Pool(table, lens, refs, 16)
    want.fork([3])
    got = pages.fork_pages(both[:4, 2:6], n, gpu([3]), r.clone(), 16, out=both[2:3, 6:10])        # a row in the gap between rows
    assert got[0].tolist() == want.table and torch.equal(both[:4, 2:6], old)
    for a, b in ((both[:4, :4], both[:4, 3:7]), (both[:4, 3:7], both[:4, :4]), (both[:4, :4], both[3:7, :4])):
        with pytest.raises(layer.LowmError):
            pages.fork_pages(a, n, gpu([0, 0, 2, 1]), r.clone(), 16, out=b)


def test_fork_most_rows():
    rows = 8192
    lens = [17] * rows
    table, refs = make(lens, 16, 3 * rows, seed=3, width=2)
    check_fork(Pool(table, lens, refs, 16), [i // 3 for i in range(rows)])
    with pytest.raises(layer.LowmError):
        pages.fork_pages(*(gpu([[0]] * 8193), gpu([0] * 8193)), gpu([0]), gpu([0]), 16)


def check_extend(pool, counts, strided=False):
    table, lens, refs = on_gpu(pool)
    if strided:
        big = torch.full((len(pool.table), pool.width + 3), 77, device="cuda", dtype=I32)
        big[:, :pool.width] = table
        table = big[:, :pool.width]
    cu = [sum(counts[:i]) for i in range(len(counts) + 1)]
    got = pages.extend_pages(table, lens, gpu(cu), refs, pool.page, cu[-1])
    positions, slots, missing = pool.extend(counts)
    assert got[0].tolist() == positions and got[1].tolist() == slots and got[2].tolist() == [missing]
    assert table.tolist() == pool.table and lens.tolist() == pool.lens and refs.tolist() == pool.refs
    if strided:
        assert bool((big[:, pool.width:] == 77).all())


@pytest.mark.parametrize("page", [1, 16, 100])
@pytest.mark.parametrize("most", [1, 40, 3000])
@pytest.mark.parametrize("rows", [1, 5, 70])
def test_extend(page, most, rows):
    r = random.Random(page + most + rows)
    if rows * most > 20000 or (page == 1 and most > 100):
        most = 100
    lens = [r.randint(0, 3 * page) for _ in range(rows)]
    width = 4 + needed(most, page)
    table, refs = make(lens, page, rows * width + 5, seed=rows, width=width)
    check_extend(Pool(table, lens, refs, page), [r.randint(0, most) for _ in range(rows)], strided=rows == 5)


def test_extend_of_many_tokens():
    lens = [3, 0, 500]
    table, refs = make(lens, 16, 2000, seed=1, width=700)
    check_extend(Pool(table, lens, refs, 16), [9000, 0, 4001])


def test_extend_without_free_pages_and_past_the_table():
    for spare in (0, 1, 2, 5):
        lens = [16, 30, 0]
        table, refs = make(lens, 16, 3 + spare, seed=1, width=4)
        check_extend(Pool(table, lens, refs, 16), [1, 40, 20])
    lens = [60, 20]
    table, refs = make(lens, 16, 30, seed=1, width=4)
    check_extend(Pool(table, lens, refs, 16), [30, 70])


def test_extend_of_a_pool_that_is_full_at_the_front():
    lens = [9000 * 16]
    table, refs = make(lens, 16, 9003, seed=1, width=9002)
    order = sorted(table[0][:9000])
    pool = Pool([order + [-1, -1]], lens, refs, 16)
    check_extend(pool, [20])


def test_extend_tokens_behind_the_last_row():
    table, lens, refs = gpu([[0, -1]]), gpu([3]), gpu([1, 0])
    positions, slots, missing = pages.extend_pages(table, lens, gpu([0, 2]), refs, 16, 5)
    assert positions.tolist() == [3, 4, 0, 0, 0] and slots.tolist() == [3, 4, -1, -1, -1] and missing.tolist() == [0]


class SharedPool(Pool):
    """Extend where rows share unfinished pages: the longest of them, of equal ones the first, goes on in it."""

    def extend(self, counts):
        old, shared = list(self.lens), {}
        for i, n in enumerate(counts):
            e = old[i] // self.page
            p = self.table[i][e] if n and old[i] % self.page and e < self.width else -1
            if self.inside(p) and any(j != i and self.used(j) > e and self.table[j][e] == p and (old[j], -j) > (old[i], -i)
                                      for j in range(len(old))):
                shared[i] = e
        positions, slots, missing = super().extend(counts)
        rows = [i for i, n in enumerate(counts) for _ in range(n)]
        slots = [-1 if p // self.page == shared.get(i, -1) else s for i, p, s in zip(rows, positions, slots)]
        self.slots = slots
        return positions, slots, missing + len(shared)


@pytest.mark.parametrize("step", [1, 3, 20, 2000])
@pytest.mark.parametrize("spare", [0, 1, 40])
def test_extend_of_rows_that_a_fork_left_on_one_page(step, spare):
    lens = [20, 7, 33]
    table, refs = make(lens, 16, 6 + spare, seed=4, width=140)
    pool = SharedPool(table, lens, refs, 16)
    check_fork(pool, [0, 0, 0, 1, 1, 2])
    for i in range(4):
        lens, used = list(pool.lens), [pool.table[j][:pool.used(j)] for j in range(6)]
        counts = [step, step + i % 2, 0 if i == 1 else step, step, 2 * step, step]
        check_extend(pool, counts)
        written = [s for s in pool.slots if s >= 0]
        assert len(set(written)) == len(written)                    # no place twice, and none that a row holds already
        held = {row[p // 16] * 16 + p % 16 for row, n in zip(used, lens) for p in range(min(n, 16 * len(row))) if row[p // 16] >= 0}
        assert not held & set(written)


def test_extend_of_a_row_that_was_cut_back_into_a_shared_page():
    # row 0 holds places of page 2 that row 1, shorter, would write next; row 2 has pages that are counted outside of the table
    pool = SharedPool([[0, 2, -1, -1], [0, 2, -1, -1], [3, 4, -1, -1]], [27, 21, 30], [2, 1, 2, 2, 2, 0, 0, 0, 0], 16)
    pool.refs[1] = 0
    for counts in ([3, 3, 1], [1, 0, 5], [0, 9, 0], [3, 0, 0]):
        check_extend(pool, counts)


def test_extend_of_many_rows_on_one_page():
    rows = 3000
    pool = SharedPool([[5 + i // 3, -1] for i in range(rows)], [3 + i % 2 for i in range(rows)],
                      [0] * 5 + [3] * 1000 + [0] * 7, 16)
    check_extend(pool, [i % 4 for i in range(rows)])
    check_extend(pool, [14] * 100 + [0] * (rows - 100))


@pytest.mark.parametrize("pages_", [1, 2, 7, 4095, 4096, 4097, 20000])
@pytest.mark.parametrize("fill", [0.0, 0.3, 0.9, 1.0])
def test_compact(pages_, fill):
    r = random.Random(pages_)
    lens, left = [], int(pages_ * fill)
    while left > 0:
        n = min(left, r.randint(1, max(1, pages_ // 3)))
        lens.append(n * 16 - r.randint(0, 15))
        left -= n
    lens = lens or [0]
    table, refs = make(lens, 16, pages_, seed=pages_)
    pool = Pool(table, lens, refs, 16)
    pool.table.append(list(pool.table[0]))                                 # a row that shares all of the first one's pages
    pool.lens.append(pool.lens[0])
    for p in pool.table[0][:pool.used(0)]:
        pool.refs[p] += 1
    t, n, refs = on_gpu(pool)
    src, dst, used = pages.compact_pages(t, n, refs, 16)
    want = pool.compact()
    assert (src.tolist(), dst.tolist(), used.tolist()) == (want[0], want[1], [want[2]])
    assert t.tolist() == pool.table and refs.tolist() == pool.refs


@pytest.mark.parametrize("rows,width", [(64, 128), (64, 129), (1, 8192), (1, 8193), (8192, 1), (8193, 1), (41, 100)])
def test_compact_of_tables_around_the_size_for_one_launch(rows, width):
    r, pool_pages = random.Random(rows), 4096
    used = r.sample(range(pool_pages), 1500)
    table = [[r.choice(used) for _ in range(width)] for _ in range(rows)]
    lens = [r.randint(0, 16 * width + 5) for _ in range(rows)]
    refs = [0] * pool_pages
    pool = Pool(table, lens, refs, 16)
    for i, row in enumerate(table):
        for p in row[:pool.used(i)]:
            pool.refs[p] += 1
    t, n, counts = on_gpu(pool)
    src, dst, total = pages.compact_pages(t, n, counts, 16)
    want = pool.compact()
    assert (src.tolist(), dst.tolist(), total.tolist()) == (want[0], want[1], [want[2]])
    assert t.tolist() == pool.table and counts.tolist() == pool.refs


def test_compact_entries_that_no_count_knows():
    table, lens, refs = gpu([[8, 2, 50, -1]]), gpu([64]), gpu([0, 0, 1, 0, 0, 1, 0, 0, 0, 0])
    src, dst, used = pages.compact_pages(table, lens, refs, 16)
    assert used.tolist() == [2] and src.tolist()[:2] == [2, 5] and dst.tolist()[:2] == [0, 1]
    assert table.tolist() == [[8, 0, 50, -1]] and refs.tolist() == [1, 1] + [0] * 8


@pytest.mark.parametrize("shape,dtype", [((9, 16, 2, 64), torch.uint8), ((9, 3), torch.float32), ((9, 5), torch.uint8), ((9, 7), BF),
                                         ((9,), torch.int64), ((9, 40000), BF)])
def test_copy(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(0, 100, shape, device="cuda", generator=g).to(dtype)
    strided = torch.randint(0, 100, (9, 2, *shape[1:]), device="cuda", generator=g).to(dtype)
    src, dst = [3, -1, 8, 1, 2, 9, 0, 7], [0, 4, 5, -1, 2, 6, 12, 1]
    want, want_strided = x.clone(), strided.clone()
    for a, b in zip(src, dst):
        if 0 <= a < 9 and 0 <= b < 9:
            want[b], want_strided[b, 1] = x[a], strided[a, 1]
    pages.copy_pages([x, strided[:, 1]], gpu(src), gpu(dst))
    assert torch.equal(x, want) and torch.equal(strided, want_strided)


def test_copy_of_many_tensors_and_far_pages():
    tensors = [torch.full((4, 33), float(i), device="cuda") + torch.arange(4, device="cuda")[:, None] for i in range(300)]
    want = [x.clone() for x in tensors]
    for x in want:
        x[2] = x[1]
    pages.copy_pages(tensors, gpu([1]), gpu([2]))
    assert all(torch.equal(x, y) for x, y in zip(tensors, want))
    big = torch.zeros(90000, 65536, device="cuda", dtype=torch.uint8)      # 5.9 GB
    big[89999] = 7
    pages.copy_pages([big], gpu([89999]), gpu([70000]))
    assert bool((big[70000] == 7).all()) and not big[69999].any() and not big[70001].any()
    del big
    torch.cuda.empty_cache()


def test_refusals():
    t, n, refs = gpu([[0, 1]]), gpu([20]), gpu([1, 1, 0])
    for call in (lambda: pages.fork_pages(t.long(), n, n, refs, 16), lambda: pages.fork_pages(t, n, t, refs, 16),
                 lambda: pages.fork_pages(t, n, n, refs, 16, out=t), lambda: pages.fork_pages(t, n, n, refs[None], 16),
                 lambda: pages.extend_pages(t, n, gpu([0]), refs, 16, 1), lambda: pages.extend_pages(t, n, gpu([0, 1]), refs, 16, -1),
                 lambda: pages.compact_pages(t, n.float(), refs, 16), lambda: pages.copy_pages([t], n, gpu([0, 1])),
                 lambda: pages.copy_pages([t, n[None].expand(3, 1)], n, n), lambda: pages.copy_pages([t.cpu()], n, n),
                 lambda: pages.copy_pages([torch.zeros(4, 4, 4, device="cuda").transpose(1, 2)], n, n)):
        with pytest.raises((TypeError, ValueError)):
            call()
    with pytest.raises(layer.LowmError):
        pages.fork_pages(t, n, n, refs, 0)
    with pytest.raises(layer.LowmError):
        pages.compact_pages(t, n, refs, -1)


# ------------------------------------------------------------------------------------------- all together
def test_beams_over_an_8_bit_cache():
    """Steps of a beam search in one captured graph: rows follow their parents, unfinished pages are copied, each row appends a
    token and attends to its own history.  The histories are kept apart in plain torch."""
    heads, kv_heads, dim, page, block, layers, steps = 4, 2, 64, 16, 8, 2, 40
    prompts, beams = [21, 5], 3
    rows, pool, width = len(prompts) * beams, 64, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.empty(s, device="cuda", dtype=BF).normal_(generator=g)          # noqa: E731
    cache = [[torch.zeros(pool, page, kv_heads, dim, device="cuda", dtype=torch.uint8).view(FP8) for _ in range(2)]
             + [torch.ones(pool, page // block, kv_heads, device="cuda") for _ in range(2)] for _ in range(layers)]
    angle = torch.arange(128, device="cuda")[:, None] * 0.3 ** torch.arange(dim // 2, device="cuda")
    table_cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    table = torch.full((rows, width), -1, device="cuda", dtype=I32)
    lens, refs = gpu([0] * rows), gpu([0] * pool)
    kept = [[[] for _ in range(rows)] for _ in range(layers)]                                  # (k, v) dequantised by row

    def histories(table, lens):
        """What the cache holds for each row: [layers][rows] of (k, v) in 64 bits."""
        out = []
        for k, v, ks, vs in cache:
            line = []
            for r in range(rows):
                key = torch.arange(int(lens[r]), device="cuda")
                pg, place = table[r, key // page].long(), key % page
                line.append(tuple(c.view(torch.uint8)[pg, place].view(FP8).to(F64) * s[pg, place // block].to(F64)[..., None]
                                  for c, s in ((k, ks), (v, vs))))
            out.append(line)
        return out

    # Prompts into each request's first row, then everyone follows it.
    n = sum(prompts)
    firsts = [prompts[i // beams] if i % beams == 0 else 0 for i in range(rows)]
    cu = gpu([sum(firsts[:i]) for i in range(rows + 1)])
    positions, slots, missing = pages.extend_pages(table, lens, cu, refs, page, n)
    for l in range(layers):
        q, k, v = normal(n, heads, dim), normal(n, kv_heads, dim), normal(n, kv_heads, dim)
        fp8.rope_append_fp8(q, k, v, table_cs, positions, slots, *cache[l])

    qkv = [[normal(rows, h, dim) for h in (heads, kv_heads, kv_heads)] for _ in range(layers)]
    parents, new_cu = gpu([i - i % beams for i in range(rows)]), gpu(list(range(rows + 1)))
    views = [x for c in cache for x in c]
    lacking = torch.zeros(1, device="cuda", dtype=I32)
    outs = [torch.empty(rows, heads, dim, device="cuda", dtype=BF) for _ in range(layers)]
    state = [table, lens]

    def step():
        new_table, new_lens, src, dst, missing = pages.fork_pages(state[0], state[1], parents, refs, page)
        pages.copy_pages(views, src, dst)
        positions, slots, short = pages.extend_pages(new_table, new_lens, new_cu, refs, page, rows)
        lacking.add_(missing + short)
        for l in range(layers):
            q = fp8.rope_append_fp8(*qkv[l], table_cs, positions, slots, *cache[l])
            fp8.paged_attention_fp8(q, *cache[l], new_table, new_lens, new_cu, out=outs[l])
        state[0].copy_(new_table)
        state[1].copy_(new_lens)

    before = [x.clone() for x in [refs, *state, *views]]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):                                                               # warm up, then put all back
        step()
    torch.cuda.synchronize()
    for x, y in zip([refs, *state, *views], before):
        x.copy_(y) if x.dtype != FP8 else x.view(torch.uint8).copy_(y.view(torch.uint8))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    r = random.Random(5)
    for turn in range(steps):
        past = histories(state[0], state[1])
        choice = [i - i % beams for i in range(rows)] if turn == 0 else [i - i % beams + r.randrange(beams) for i in range(rows)]
        parents.copy_(gpu(choice))
        for l in range(layers):
            for x in qkv[l]:
                x.copy_(normal(*x.shape))
        graph.replay()
        assert lacking.item() == 0
        now = histories(state[0], state[1])
        for l in range(layers):
            for i in range(rows):
                k, v = now[l][i]
                pk, pv = past[l][choice[i]]
                assert k.shape[0] == pk.shape[0] + 1
                # the parent's history, but for codes that moved to a larger scale (half a step: 2^-4, of the block's largest
                # 2^-10 / 448 at least)
                for a, b in ((k[:-1], pk), (v[:-1], pv)):
                    assert bool(((a - b).abs() <= b.abs() * 2.0 ** -4 + 2.0 ** -10).all())
                new = qkv[l][2][i].to(F64)
                assert bool(((v[-1] - new).abs() <= new.abs() * 2.0 ** -4 + 2.0 ** -10).all())
            # attention over exactly what the cache holds
            c, s = table_cs[state[1].long() - 1, :dim // 2].to(F64)[:, None], table_cs[state[1].long() - 1, dim // 2:].to(F64)[:, None]
            a, b = qkv[l][0].to(F64).split(dim // 2, -1)
            q = torch.cat([a * c - b * s, a * s + b * c], -1).to(BF).to(F64)
            for i in range(rows):
                k, v = (x.repeat_interleave(heads // kv_heads, 1) for x in now[l][i])
                w = (torch.einsum("hd,jhd->hj", q[i], k) / math.sqrt(dim)).softmax(-1)
                want = torch.einsum("hj,jhd->hd", w, v)
                size = torch.einsum("hj,jhd->hd", w, v.abs())
                # q may round the other way where its fp32 rotation differs: 2^-8 of its terms in a score
                slack = 2.0 ** -8 * want.abs() + (2.0 ** -10 + 2.0 ** -7) * size
                assert bool(((outs[l][i].to(F64) - want).abs() <= slack + 1e-6).all())
    used = {p for r_ in range(rows) for p in state[0][r_].tolist() if p >= 0}
    assert sum(x > 0 for x in refs.tolist()) == len(used) < pool
    # Brought together, the cache says the same.
    said = histories(state[0], state[1])
    src, dst, count = pages.compact_pages(state[0], state[1], refs, page)
    pages.copy_pages(views, src, dst)
    assert count.item() == len(used) and int(state[0].max()) < len(used)
    for a, b in zip(said, histories(state[0], state[1])):
        for x, y in zip(a, b):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
