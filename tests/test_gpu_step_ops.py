"""GPU tests of the serving-step operators against oracle/step_ops.py, through
the public entry points: whole numbers exact, floating outputs within bounds
counted from the roundings of the computation."""
import math

import numpy as np
import pytest
import torch

import paged_mla_speculative_tree_gb300 as pkg
from oracle import step_ops as S
from oracle import tree_ops as T
from paged_mla_speculative_tree_gb300 import binding, workloads as W

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def err_word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# -------------------------------------------------------------- page tables

def page_state(seed, rows, per, page, fill=0.5, spare=3):
    rng = np.random.default_rng(seed)
    held = [int(x) for x in rng.integers(0, int(per * fill) + 1, rows)]
    ids = [int(x) for x in rng.permutation(rows * per + spare)]
    table = [[ids.pop() if j < held[r] else -7 for j in range(per)] for r in range(rows)]
    return rng, table, held, ids


class Pages:
    def __init__(self, table, held, free, capacity=None, stride=None):
        rows, per = len(table), len(table[0])
        buf = torch.full((rows, stride or per), -9, dtype=torch.int32, device=DEV)
        buf[:, :per] = i32(table)
        self.buf, self.table, self.held = buf, buf[:, :per], i32(held)
        self.free = torch.full((capacity if capacity is not None else len(free) + sum(held),), -5, dtype=torch.int32, device=DEV)
        self.free[:len(free)] = i32(free)
        self.num, self.err = i32([len(free)]), err_word()

    def update(self, lens, page):
        pkg.page_table_update(i32(lens), page, self.table, self.held, self.free, self.num, self.err)
        return self

    def expect(self, table, held, free, err=0):
        torch.cuda.synchronize()
        assert int(self.err) == err
        assert self.held.tolist() == list(held)
        assert int(self.num) == len(free)
        assert self.free[:len(free)].tolist() == list(free)
        assert self.table.tolist() == table
        return self


@pytest.mark.parametrize("rows,per,page", [(1, 1, 1), (1, 40, 16), (3, 7, 4), (64, 5, 16), (257, 33, 3), (1025, 9, 64),
                                           (8192, 3, 16), (40, 3000, 1)])
def test_pages_grow_shrink_and_mix(rows, per, page):
    rng, table, held, free = page_state(rows * 31 + per, rows, per, page)
    p = Pages(table, held, free, stride=per + 2)
    for step in range(3):
        lens = [int(x) for x in rng.integers(0, per * page + 1, rows)]
        if step == 1:
            lens = [-1 if rng.random() < 0.4 else n for n in lens]
        if step == 2:
            lens = [0 if rng.random() < 0.6 else n for n in lens]
        table, held, free, flagged = S.page_table_update(lens, page, table, held, free)
        assert not flagged
        p.update(lens, page).expect(table, held, free)
    assert bool((p.buf[:, per:] == -9).all())


def test_pages_roll_back_restores_the_stack():
    _, table, held, free = page_state(7, 300, 20, 16)
    lens = [h * 16 - (h > 0) * 5 for h in held]
    p = Pages(table, held, free)
    p.update([n + 64 for n in lens], 16).update(lens, 16)
    torch.cuda.synchronize()
    assert p.held.tolist() == held and p.free[:len(free)].tolist() == free and int(p.num) == len(free) and int(p.err) == 0


@pytest.mark.parametrize("rows", [5, 1500])
def test_pages_short_of_free_ones(rows):
    _, table, held, _ = page_state(rows, rows, 8, 4, fill=0.0)
    free = list(range(100, 100 + rows * 2))
    lens = [4 * (1 + r % 5) for r in range(rows)]  # 3 a row on average: the first rows get theirs
    lens[1] = 0
    t2, h2, f2, flagged = S.page_table_update(lens, 4, table, held, free)
    assert flagged and h2[0] == 1
    Pages(table, held, free).update(lens, 4).expect(t2, h2, f2, binding.DEVERR_PAGES)


def test_pages_released_in_the_same_call_are_enough():
    table, held = [[1, 2, 3, 4], [0, 0, 0, 0]], [4, 0]
    t2, h2, f2, flagged = S.page_table_update([0, 4], 1, table, held, [])
    assert not flagged and h2 == [0, 4]
    Pages(table, held, [], capacity=4).update([0, 4], 1).expect(t2, h2, f2)


def test_pages_bad_rows_are_left_and_flagged():
    table, held, free = [[1, 2, 3], [4, 5, 6], [7, 8, 9], [10, 11, 12]], [1, 9, 2, -1], [20, 21]
    lens = [100, 4, -3, 4]  # too long for a row, held past the row, bad length, negative held
    t2, h2, f2, flagged = S.page_table_update(lens, 4, table, held, free)
    assert flagged == [0, 1, 2, 3]
    Pages(table, held, free, capacity=9).update(lens, 4).expect(t2, h2, f2, binding.DEVERR_PAGES | binding.DEVERR_INDPTR)
    for bad in (-1, 10):  # a stack that is none: nothing is done
        p = Pages(table, [1, 2, 2, 0], free, capacity=9)
        p.num.fill_(bad)
        p.update([0, 0, 0, 12], 4)
        torch.cuda.synchronize()
        assert int(p.err) == binding.DEVERR_PAGES and int(p.num) == bad and p.held.tolist() == [1, 2, 2, 0]
        assert p.table.tolist() == table and p.free.tolist() == [20, 21] + [-5] * 7


def test_pages_pushed_past_the_capacity_are_lost():
    p = Pages([[1, 2, 3, 4]], [4], [9], capacity=3)
    p.update([0], 1)
    torch.cuda.synchronize()
    assert int(p.err) == binding.DEVERR_PAGES and int(p.num) == 3 and p.free.tolist() == [9, 4, 3]


def test_pages_capture_and_replay():
    _, table, held, free = page_state(11, 50, 12, 16, fill=0.3)
    lens = [h * 16 for h in held]
    p, up, down = Pages(table, held, free), i32([n + 40 for n in lens]), i32(lens)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pkg.page_table_update(up, 16, p.table, p.held, p.free, p.num, p.err)
            pkg.page_table_update(down, 16, p.table, p.held, p.free, p.num, p.err)
            pkg.page_table_update(up, 16, p.table, p.held, p.free, p.num, p.err)
    for add in (40, 0, 90):
        up.copy_(i32([n + add for n in lens]))
        graph.replay()
        for v in (up, down, up):
            table, held, free, flagged = S.page_table_update(v.tolist(), 16, table, held, free)
            assert not flagged
    p.expect(table, held, free)


@pytest.mark.parametrize("rows,per", [(900, 40), (1, 30000)])
def test_pages_of_a_large_table_capture_and_replay(rows, per):
    """Over 16384 entries: a grid of moves with the state written behind it."""
    _, table, held, free = page_state(rows, rows, per, 2, fill=0.4)
    lens = [h * 2 for h in held]
    p, up, down = Pages(table, held, free), i32([n + per // 2 for n in lens]), i32([max(0, n - per // 3) for n in lens])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for v in (up, down, up):
                pkg.page_table_update(v, 2, p.table, p.held, p.free, p.num, p.err)
    for _ in range(2):
        graph.replay()
        for v in (up, down, up):
            table, held, free, flagged = S.page_table_update(v.tolist(), 2, table, held, free)
            assert not flagged
    p.expect(table, held, free)


def test_pages_of_rows_without_entries():
    p = Pages([[1], [2]], [0, 0], [7, 8])
    empty = torch.empty((2, 0), dtype=torch.int32, device=DEV)
    pkg.page_table_update(i32([0, -1]), 4, empty, p.held, p.free, p.num, p.err)
    p.expect([[1], [2]], [0, 0], [7, 8])
    pkg.page_table_update(i32([0, 1]), 4, empty, p.held, p.free, p.num, p.err)
    p.expect([[1], [2]], [0, 0], [7, 8], binding.DEVERR_PAGES)


def test_two_updates_at_once_on_two_streams():
    states = [page_state(50 + k, 300, 90, 1, fill=0.5) for k in range(2)]
    pages = [Pages(*st[1:]) for st in states]
    lens = [[int(x) for x in st[0].integers(0, 91, 300)] for st in states]
    dev = [i32(v) for v in lens]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for k in range(2):
            pkg.page_table_update(dev[k], 1, pages[k].table, pages[k].held, pages[k].free, pages[k].num, pages[k].err,
                                  stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        pages[k].expect(*S.page_table_update(lens[k], 1, *states[k][1:])[:3])


# ---------------------------------------------------------------- slot maps

def build_slots(table, page, prefix, tree, rows=None, parents=None, kv_cap=None, q_cap=None, num_pages=None, pad=5,
                stride=None, positions=True):
    bs, per = len(prefix), len(table[0])
    buf = torch.full((len(table), stride or per), -3, dtype=torch.int32, device=DEV)
    buf[:, :per] = i32(table)
    kv_cap = sum(max(p, 0) for p in prefix) + pad if kv_cap is None else kv_cap
    q_cap = sum(max(n, 0) for n in tree) + pad if q_cap is None else q_cap
    o = dict(kv_indptr=torch.full((bs + 1,), -4, dtype=torch.int32, device=DEV),
             kv_indices=torch.full((kv_cap,), -4, dtype=torch.int64, device=DEV),
             qo_indptr=torch.full((bs + 1,), -4, dtype=torch.int64, device=DEV),
             out_cache_loc=torch.full((q_cap,), -4, dtype=torch.int64, device=DEV),
             positions=torch.full((q_cap,), -4, dtype=torch.int64, device=DEV) if positions else None)
    err = err_word()
    flat = None
    if parents is not None:
        flat = torch.full((q_cap,), -1, dtype=torch.int32)
        v = [x for per_req in parents for x in per_req][:q_cap]
        flat[:len(v)] = torch.tensor(v, dtype=torch.int32)
        flat = flat.to(DEV)
    pkg.slot_map_build(buf[:, :per], i32(prefix), i32(tree), page, o["kv_indptr"], o["kv_indices"], o["qo_indptr"],
                       o["out_cache_loc"], o["positions"], rows=None if rows is None else i32(rows), parents=flat,
                       num_pages=num_pages if num_pages is not None else max(max(t) for t in table) + 1, err=err)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in o.items() if v is not None}, int(err)


def check_slots(got, want):
    for name, w in zip(("kv_indptr", "kv_indices", "qo_indptr", "out_cache_loc", "positions"), want):
        np.testing.assert_array_equal(got[name][:len(w)], w, err_msg=name)
        assert (got[name][len(w):] == -4).all(), f"{name}: written behind the last request"


def slot_case(seed, bs, max_p, max_n, page, spare_rows=2):
    rng = np.random.default_rng(seed)
    prefix, tree = [int(x) for x in rng.integers(0, max_p + 1, bs)], [int(x) for x in rng.integers(0, max_n + 1, bs)]
    per = -(-(max_p + max_n) // page)
    table = rng.permutation((bs + spare_rows) * per).reshape(bs + spare_rows, per).tolist()
    rows = [int(x) for x in rng.permutation(bs + spare_rows)[:bs]]
    parents = [[int(rng.integers(-1, i)) if i else -1 for i in range(n)] for n in tree]
    return table, rows, prefix, tree, parents


@pytest.mark.parametrize("bs,max_p,max_n,page", [(1, 1, 1, 1), (1, 1000, 1, 64), (3, 17, 9, 4), (40, 300, 70, 16),
                                                 (600, 40, 3, 1), (2, 9000, 1500, 48), (5, 0, 8, 16), (8192, 2, 1, 2),
                                                 (7, 2049, 0, 100)])
def test_slot_maps(bs, max_p, max_n, page):
    table, rows, prefix, tree, parents = slot_case(bs * 7 + page, bs, max_p, max_n, page)
    if bs == 1:
        prefix, tree, parents = [max_p], [max_n], [[-1] * max_n]
    got, err = build_slots(table, page, prefix, tree, rows, parents, stride=len(table[0]) + 3)
    assert err == 0
    check_slots(got, S.slot_map(table, page, rows, prefix, tree, parents))
    got, err = build_slots(table, page, prefix, tree, rows, None)  # chains
    assert err == 0
    check_slots(got, S.slot_map(table, page, rows, prefix, tree, None))


def test_slot_maps_without_rows_trees_or_outputs():
    table, _, prefix, tree, _ = slot_case(4, 6, 100, 5, 8, spare_rows=0)
    got, err = build_slots(table, 8, prefix, tree, None, None, positions=False)
    assert err == 0
    check_slots(got, S.slot_map(table, 8, range(6), prefix, tree, None)[:4])
    kvp, qop, loc = i32([-4] * 7), i64([-4] * 7), i64([-4] * sum(tree))
    pkg.slot_map_build(i32(table), i32(prefix), None, 8, kvp, None, qop, None, num_pages=1 << 20)
    assert kvp.tolist() == [0] + np.cumsum(prefix).tolist() and qop.tolist() == [0] * 7
    pkg.slot_map_build(i32(table), i32(prefix), i32(tree), 8, kvp, None, qop, loc, num_pages=1 << 20)
    assert loc.tolist() == S.slot_map(table, 8, range(6), prefix, tree, None)[3].tolist()
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    pkg.slot_map_build(i32(table), empty, empty, 8, kvp[:1], i64([1]), qop[:1], i64([1]), num_pages=9)
    assert int(kvp[0]) == 0 and int(qop[0]) == 0


@pytest.mark.parametrize("bs,max_p,page", [(3, 5000, 16), (700, 9, 4), (20, 130, 1), (2, 70000, 64)])
def test_slot_maps_into_odd_addresses(bs, max_p, page):
    """kv_indices 8 bytes past a 16-byte boundary, its neighbours untouched."""
    table, rows, prefix, tree, _ = slot_case(bs + max_p, bs, max_p, 3, page)
    want = S.slot_map(table, page, rows, prefix, tree, None)
    buf = torch.full((sum(prefix) + 2,), -4, dtype=torch.int64, device=DEV)
    kvp, qop, loc = i32([0] * (bs + 1)), i64([0] * (bs + 1)), torch.empty(sum(tree) + 1, dtype=torch.int64, device=DEV)[1:]
    pkg.slot_map_build(i32(table), i32(prefix), i32(tree), page, kvp, buf[1:-1], qop, loc, rows=i32(rows), num_pages=1 << 20)
    np.testing.assert_array_equal(buf[1:-1].cpu().numpy(), want[1])
    np.testing.assert_array_equal(loc.cpu().numpy(), want[3])
    assert int(buf[0]) == -4 and int(buf[-1]) == -4


def test_slot_maps_capture_and_replay_with_new_lengths():
    table, rows, _, _, _ = slot_case(31, 6, 400, 20, 16)
    p, n, t, r = i32([0] * 6), i32([0] * 6), i32(table), i32(rows)
    o = dict(kv_indptr=i32([0] * 7), kv_indices=torch.full((2400,), -4, dtype=torch.int64, device=DEV), qo_indptr=i64([0] * 7),
             out_cache_loc=torch.full((120,), -4, dtype=torch.int64, device=DEV))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pkg.slot_map_build(t, p, n, 16, *o.values(), rows=r, num_pages=10000)
    rng = np.random.default_rng(8)
    for _ in range(3):
        prefix, tree = [int(x) for x in rng.integers(0, 401, 6)], [int(x) for x in rng.integers(0, 21, 6)]
        p.copy_(i32(prefix))
        n.copy_(i32(tree))
        for v in (o["kv_indices"], o["out_cache_loc"]):
            v.fill_(-4)
        graph.replay()
        torch.cuda.synchronize()
        check_slots({k: v.cpu().numpy() for k, v in o.items()}, S.slot_map(table, 16, rows, prefix, tree, None)[:4])


@pytest.mark.parametrize("shape", ["chain", "star", "deep"])
def test_positions_of_long_trees(shape):
    n = 1700
    par = {"chain": W.chain_parents(n), "star": W.star_parents(n),
           "deep": [max(i - 1 - (i % 7 == 0) * 3, -1) for i in range(n)]}[shape]
    table = [list(range(400))]
    got, err = build_slots(table, 16, [77], [n], [0], [par])
    assert err == 0
    check_slots(got, S.slot_map(table, 16, [0], [77], [n], [par]))


def test_slot_maps_flag_bad_input():
    table = [[3, 1, 99, 2], [0, 4, 5, 6]]
    want = S.slot_map([[3, 1, 99, 2], [0, 4, 5, 6]], 4, [0, 1], [10, 3], [2, 1], [[-1, 0], [-1]])
    got, err = build_slots(table, 4, [10, 3], [2, 1], [0, 1], [[-1, 0], [-1]], num_pages=7)  # page 99 is none
    assert err == binding.DEVERR_PAGES
    kv = want[1].copy()
    kv[8:10] = -1
    loc = want[3].copy()
    loc[:2] = -1
    check_slots(got, (want[0], kv, want[2], loc, want[4]))
    got, err = build_slots(table, 4, [3, 2], [1, 1], [0, 7], [[-1], [-1]], num_pages=100)  # no row 7
    assert err == binding.DEVERR_PAGES and got["kv_indices"][3:5].tolist() == [-1, -1] and got["kv_indices"][:3].tolist() == [12, 13, 14]
    got, err = build_slots(table, 4, [15, 2], [3, 1], [0, 1], [[-1, 0, 1], [-1]], num_pages=100)  # two tokens past the row
    assert err == binding.DEVERR_PAGES and got["out_cache_loc"][:3].tolist() == [11, -1, -1]
    got, err = build_slots(table, 4, [-5, 2], [2, -1], [0, 1], [[-1, 0], []], num_pages=100)
    assert err == binding.DEVERR_INDPTR and got["kv_indptr"].tolist() == [0, 0, 2] and got["qo_indptr"].tolist() == [0, 2, 2]
    got, err = build_slots(table, 4, [2], [4], [1], [[-1, 1, 0, -2]], num_pages=100)  # nodes 1 and 3: no tree
    assert err == binding.DEVERR_PARENT and got["positions"][:4].tolist() == [2, 2, 3, 2]


@pytest.mark.parametrize("page", [1, 2, 7, 64])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("odd", [0, 1])
def test_slots_of_a_bad_entry_in_a_long_run(page, where, odd):
    """Runs of up to 32 steps of 64 keys: one entry that is no page (negative, or
    past the pool) gives -1 for its own tokens, and its neighbours keep theirs."""
    prefix, num_pages = [5000, 3, 40000, 1111], 1 << 20
    per = -(-max(prefix) // page)
    table = np.random.default_rng(page).integers(0, num_pages, (4, per))
    flagged = table.copy()
    for r, p in enumerate(prefix):
        last = (p - 1) // page
        at = {"first": 0, "middle": last // 2, "last": last}[where]
        table[r, at], flagged[r, at] = (-1 - r if r % 2 else num_pages + r), -1
    j = [np.arange(p) for p in prefix]
    want = np.concatenate([np.where(flagged[r, x // page] < 0, -1, flagged[r, x // page] * page + x % page) for r, x in enumerate(j)])
    out = torch.full((sum(prefix) + 4,), -4, dtype=torch.int64, device=DEV)
    kvp, qop, err = i32([0] * 5), i64([0] * 5), err_word()
    for _ in range(3):
        out.fill_(-4)
        pkg.slot_map_build(i32(table.tolist()), i32(prefix), None, page, kvp, out[odd:odd + sum(prefix)], qop, None,
                           num_pages=num_pages, err=err)
        got = out.cpu().numpy()
        np.testing.assert_array_equal(got[odd:odd + sum(prefix)], want)
        assert (got[:odd] == -4).all() and (got[odd + sum(prefix):] == -4).all() and int(err) == binding.DEVERR_PAGES


@pytest.mark.parametrize("page", [1, 3, 16])
def test_slots_of_a_prefix_past_its_row(page):
    """A prefix of several thousand tokens, its table row three pages short."""
    prefix = [2500, 4000, 4001]
    per = -(-4000 // page) - 3
    table = np.random.default_rng(page).permutation(3 * per).reshape(3, per)
    slot = lambda r, j: int(table[r, j // page]) * page + j % page if j < per * page else -1  # noqa: E731
    out = torch.full((sum(prefix),), -4, dtype=torch.int64, device=DEV)
    kvp, qop, err = i32([0] * 4), i64([0] * 4), err_word()
    pkg.slot_map_build(i32(table.tolist()), i32(prefix), None, page, kvp, out, qop, None, num_pages=3 * per, err=err)
    assert out.tolist() == [slot(r, j) for r, p in enumerate(prefix) for j in range(p)]
    assert int(err) == binding.DEVERR_PAGES


def test_slot_maps_past_a_capacity():
    table, rows, prefix, tree, parents = slot_case(12, 5, 200, 30, 16)
    want = S.slot_map(table, 16, rows, prefix, tree, parents)
    kv_cap, q_cap = len(want[1]) - 7, len(want[3]) - 4
    got, err = build_slots(table, 16, prefix, tree, rows, parents, kv_cap=kv_cap, q_cap=q_cap)
    assert err == binding.DEVERR_INDPTR
    check_slots(got, (want[0], want[1][:kv_cap], want[2], want[3][:q_cap], want[4][:q_cap]))
    big = [2 ** 31 - 1, 5, 2 ** 30]
    got, err = build_slots([[0]], 16, big, [0, 0, 0], [0, 0, 0], None, kv_cap=8)
    assert err & binding.DEVERR_INDPTR and got["kv_indptr"].tolist() == [0] + [2 ** 31 - 1] * 3


@pytest.mark.parametrize("prefix", [[2 ** 31 - 1, 5, 2 ** 30, 20], [2 ** 30, 2 ** 30 + 100, 9, 33], [3, 2 ** 31 - 1, 0, 17]])
@pytest.mark.parametrize("with_keys", [True, False])
def test_slots_of_trees_behind_sums_past_32_bits(prefix, with_keys):
    """kv_indptr is held at 2^31 - 1; every tree keeps its own prefix length: its
    slots lie behind its prefix (or are none), never on a prefix's tokens."""
    page, tree, parents = 16, [2, 3, 1, 4], [[-1, 0], [-1, 0, 0], [-1], [-1, 0, 1, 0]]
    table = np.random.default_rng(3).permutation(4 * 3).reshape(4, 3)
    depth = [[0, 1], [0, 1, 1], [0], [0, 1, 2, 1]]
    kvp, qop, loc, pos, err = i32([0] * 5), i64([0] * 5), i64([-4] * 12), i64([-4] * 12), err_word()
    kvi = torch.full((8,), -4, dtype=torch.int64, device=DEV) if with_keys else None
    pkg.slot_map_build(i32(table.tolist()), i32(prefix), i32(tree), page, kvp, kvi, qop, loc, pos,
                       parents=i32([x for p in parents for x in p] + [-1, -1]), num_pages=12, err=err)
    slot = lambda r, j: int(table[r][j // page]) * page + j % page if j < 3 * page else -1  # noqa: E731
    assert loc.tolist() == [slot(r, p + t) for r, p in enumerate(prefix) for t in range(tree[r])] + [-4, -4]
    assert pos.tolist() == [p + d for r, p in enumerate(prefix) for d in depth[r]] + [-4, -4]
    assert kvp.tolist() == [0] + [min(int(n), 2 ** 31 - 1) for n in np.cumsum(prefix)]
    assert qop.tolist() == [0, 2, 5, 6, 10] and int(err) == binding.DEVERR_INDPTR | binding.DEVERR_PAGES


def test_slots_past_32_bits_in_bytes_and_far_pages():
    table = [[2 ** 31 - 1, 0, 2 ** 30]]
    got, err = build_slots(table, 1000, [2500], [3], [0], [[-1, 0, 1]], num_pages=2 ** 31)
    assert err == 0
    check_slots(got, S.slot_map(table, 1000, [0], [2500], [3], [[-1, 0, 1]]))


# ------------------------------------------------------------------- rotary

def rope_inputs(seed, tokens, heads, dim, dtype, q_width=None, q_off=0):
    g = torch.Generator().manual_seed(seed)
    full = torch.randn((tokens, heads, (q_width or dim)), generator=g).to(dtype).to(DEV)
    return full, full[:, :, q_off:q_off + dim]


def rope_tolerance(mag, y, dtype):
    """fp32 rotation: the phase rounded to fp32 half turns (2^-25 pi) and cut at 2^-32 turns,
    sincospi within 2^-23, the amplitude, both products and the sum 2^-24 each: under 2^-21 of
    |x1| + |x2|; then half a step of the output's type (2^-25 below fp16's normal range)."""
    return mag * 2.0 ** -21 + (np.abs(y) + mag * 2.0 ** -21) * torch.finfo(dtype).eps / 2 + (2.0 ** -25 if dtype == torch.float16 else 0)


def check_rope(got, x, positions, turns, amp, half, dtype, inverse=False):
    want, mag = S.rope(x.double().cpu().numpy(), positions, turns.tolist(), amp, half, inverse)
    diff = np.abs(got.double().cpu().numpy() - want)
    over = diff - rope_tolerance(mag, want, dtype)
    assert over.max() <= 0, f"off by {diff.max():.3e}, past the bound by {over.max():.3e}"


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 2), (1, 64, 64), (5, 3, 6), (9, 16, 64), (3, 5, 256), (4, 7, 48),
                                              (2, 128, 64)])
def test_rope_queries(dtype, half, tokens, heads, dim):
    dt = TYPES[dtype]
    turns, _ = pkg.rope_freqs(dim, 10000.0)
    rng = np.random.default_rng(dim)
    pos = [int(p) for p in rng.integers(0, 1 << 20, tokens)]
    for off, width in ((0, dim), (dim, 2 * dim), (1, dim + 3)):  # dense, an aligned part, an odd one
        full, x = rope_inputs(dim + off, tokens, heads, dim, dt, width, off)
        out = torch.full((tokens, heads, width), 7.0, dtype=dt, device=DEV)
        args = dict(layout=binding.ROPE_HALF if half else binding.ROPE_INTERLEAVED, amplitude=1.25)
        pkg.rope_write(turns.cuda(), i64(pos), q_in=x, q_out=out[:, :, off:off + dim], **args)
        check_rope(out[:, :, off:off + dim], x, pos, turns, 1.25, half, dt)
        assert bool((out[:, :, :off] == 7).all()) and bool((out[:, :, off + dim:] == 7).all())
        back = x.clone()
        pkg.rope_write(turns.cuda(), i64(pos), q_in=x, q_out=x, **args)  # in place
        assert torch.equal(x, out[:, :, off:off + dim])
        inv = torch.empty_like(back)
        pkg.rope_write(turns.cuda(), i64(pos), q_in=back, q_out=inv, inverse=True, **args)
        check_rope(inv, back, pos, turns, 1.25, half, dt, inverse=True)


def test_rope_far_and_negative_positions():
    turns, _ = pkg.rope_freqs(64, 10000.0)
    pos = [0, 1, 131071, 2 ** 31 - 1, 2 ** 31, 2 ** 40 + 12345, -1, -70000]
    _, x = rope_inputs(3, len(pos), 2, 64, torch.float32)
    out = torch.empty_like(x)
    pkg.rope_write(turns.cuda(), i64(pos), q_in=x, q_out=out)
    check_rope(out, x, pos, turns, 1.0, False, torch.float32)
    assert torch.equal(out[0], x[0])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_rope_latent_rows(dtype, half, pad):
    dt, tokens, slots = TYPES[dtype], 37, 90
    turns, _ = pkg.rope_freqs(64, 50000.0)
    g = torch.Generator().manual_seed(4 + pad)
    down = torch.randn((tokens, 576 + pad), generator=g).to(dt).to(DEV)
    c, k = down[:, :512], down[:, 512:576]
    loc = torch.randperm(slots, generator=g)[:tokens].to(DEV)
    pos = torch.randint(0, 200000, (tokens,), generator=g)
    pool = torch.full((slots, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    bad = loc.clone()
    bad[5], bad[6] = -1, slots
    err = err_word()
    valid = i64([tokens - 4])
    pkg.rope_write(turns.cuda(), pos.cuda(), layout=int(half), k_in=k, c_in=c, out_cache_loc=bad, kv_pool=pool,
                   num_valid=valid, err=err)
    torch.cuda.synchronize()
    assert int(err) == binding.DEVERR_SLOT_RANGE
    live = [t for t in range(tokens - 4) if t not in (5, 6)]
    rows = pool[loc[live]]
    assert torch.equal(rows[:, :512], c[live].to(torch.bfloat16))
    check_rope(rows[:, 512:], k[live], pos[live].tolist(), turns, 1.0, half, torch.bfloat16)
    rest = torch.ones(slots, dtype=torch.bool, device=DEV)
    rest[loc[live]] = False
    assert bool((pool[rest] == 3).all())


def test_rope_num_valid_bounds_the_queries_too():
    turns, _ = pkg.rope_freqs(64, 10000.0)
    _, x = rope_inputs(8, 6, 4, 64, torch.bfloat16)
    for n in (0, 2, 6, 9, -1):
        out = torch.full_like(x, 5.0)
        pkg.rope_write(turns.cuda(), i64([3] * 6), q_in=x, q_out=out, num_valid=i64([n]))
        k = max(0, min(n, 6))
        assert bool((out[k:] == 5).all())
        check_rope(out[:k], x[:k], [3] * k, turns, 1.0, False, torch.bfloat16) if k else None


def test_rope_special_values_and_empty_calls():
    turns, _ = pkg.rope_freqs(64, 10000.0)
    _, x = rope_inputs(8, 3, 2, 64, torch.float16)
    x[1, 0, 5], x[2, 1, 7] = math.inf, math.nan
    out = torch.zeros_like(x)
    pkg.rope_write(turns.cuda(), i64([3, 0, 9]), q_in=x, q_out=out)
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isnan(out[2, 1, 6:8]).all())
    assert bool(torch.isfinite(out[1, 1]).all()) and bool(torch.isfinite(out[2, 0]).all())
    empty = torch.empty((0, 2, 64), dtype=torch.float16, device=DEV)
    pkg.rope_write(turns.cuda(), i64([]), q_in=empty, q_out=empty)


def test_rope_strides_past_32_bits():
    """Head parts 2^31 elements apart (a 4.3 GB view), and a slot past 2^31 / 576 rows (4.3 GB)."""
    turns, _ = pkg.rope_freqs(64, 10000.0)
    buf = torch.zeros((1 << 31) + 256, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(buf, (2, 2, 64), (1 << 31, 64, 1))
    x.copy_(torch.randn((2, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16))
    keep = x.clone()
    pkg.rope_write(turns.cuda(), i64([5, 70000]), q_in=x, q_out=x)
    check_rope(x, keep, [5, 70000], turns, 1.0, False, torch.bfloat16)
    del buf, x
    slots = (1 << 31) // 576 + 50
    pool = torch.zeros((slots, 576), dtype=torch.bfloat16, device=DEV)
    row = torch.randn((1, 576), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    pkg.rope_write(turns.cuda(), i64([0]), k_in=row[:, 512:], c_in=row[:, :512], out_cache_loc=i64([slots - 1]), kv_pool=pool)
    assert torch.equal(pool[-1:], row) and not bool(pool[:-1].any())


# -------------------------------------------------------- log probabilities

def run_logprobs(logits, tokens, rows=None, inv=None, k=5):
    n, R = len(tokens), logits.shape[0]
    o = dict(logprobs=torch.full((n,), 9.0, device=DEV), stats=torch.full((3, R), 9.0, device=DEV),
             top_tokens=torch.full((k, R), -9, dtype=torch.int32, device=DEV), top_logprobs=torch.full((k, R), 9.0, device=DEV))
    err = err_word()
    pkg.token_logprobs(logits, o["stats"], i32(tokens), o["logprobs"], o["top_tokens"], o["top_logprobs"],
                       token_rows=None if rows is None else i32(rows), inv_temperature=inv, err=err)
    torch.cuda.synchronize()
    return {a: v.cpu().numpy() for a, v in o.items()}, int(err)


def check_logprobs(logits, tokens, rows=None, inv=None, k=5, err=0):
    got, word = run_logprobs(logits, tokens, rows, inv, k)
    assert word == err
    trow = list(range(len(tokens))) if rows is None else rows
    want = S.token_logprobs(logits.double().cpu().numpy(), None if inv is None else inv.cpu().numpy(), tokens, trow, k)
    np.testing.assert_array_equal(got["top_tokens"], want["top_tokens"])
    np.testing.assert_array_equal(got["stats"][0], want["stats"][0].astype(np.float32))
    # Relative error of S: one exponential and a change of reference within 2^-20, its argument's
    # roundings 2^-22 |d|, and a sum whose longest chain is under V / 128 + 64 additions of 2^-24.
    V = logits.shape[1]
    chain = (V / 128 + 64) * 2.0 ** -24
    rel_s = chain + 2.0 ** -20 + 2.0 ** -22 * want["mean"]
    with np.errstate(invalid="ignore", divide="ignore"):
        rel_u = chain + 2.0 ** -20 + 2.0 ** -22 * np.where(want["mean"] > 0, want["square"] / want["mean"], 0)
        tol_s = rel_s + 2.0 ** -22 * np.abs(want["stats"][1])
        tol_h = tol_s + want["mean"] * (rel_s + rel_u + 2.0 ** -22) + 2.0 ** -23 * np.abs(want["stats"][2])

        def near(g, w, tol, what):
            np.testing.assert_array_equal(np.isnan(g), np.isnan(w), err_msg=what)
            np.testing.assert_array_equal(np.isneginf(g), np.isneginf(w), err_msg=what)
            live = np.isfinite(w)
            over = np.abs(g - w)[live] - tol[live]
            assert not over.size or over.max() <= 0, f"{what}: past the bound by {over.max():.3e} at {np.abs(g - w)[live].max():.3e}"

        near(got["stats"][1], want["stats"][1], tol_s, "ln S")
        near(got["stats"][2], want["stats"][2], tol_h, "entropy")
        # z - m one rounding, the difference to ln S another
        lp = lambda w, r: tol_s[r] + 2.0 ** -23 * (2 * np.abs(w) + np.abs(want["stats"][1][r]))  # noqa: E731
        near(got["top_logprobs"], want["top_logprobs"], lp(want["top_logprobs"], np.arange(len(tol_s))), "top")
        ok = np.array([0 <= r < len(tol_s) for r in trow], dtype=bool)
        safe = np.where(ok, trow, 0) if len(trow) else np.zeros(0, dtype=int)
        near(got["logprobs"], want["logprobs"], lp(want["logprobs"], safe), "given tokens")
    return got


def make_logits(seed, rows, vocab, dtype, pad=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    buf = (torch.randn((rows, vocab + pad), generator=g) * spread).to(dtype).to(DEV)
    return buf[:, :vocab]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows,vocab,pad,k", [(1, 1, 0, 1), (3, 2, 0, 5), (2, 7, 1, 32), (5, 33, 2, 3), (4, 255, 0, 32),
                                              (9, 1000, 3, 20), (2, 4099, 0, 32), (1, 50257, 0, 20), (7, 50257, 1, 20),
                                              (300, 1537, 8, 1), (1, 131072, 0, 32), (40, 32000, 0, 8), (3, 1048576, 0, 20)])
def test_logprobs(dtype, rows, vocab, pad, k):
    x = make_logits(rows + vocab, rows, vocab, TYPES[dtype], pad)
    rng = np.random.default_rng(vocab)
    tokens = [int(t) for t in rng.integers(0, vocab, rows)]
    tokens[-1] = -1
    check_logprobs(x, tokens, k=k)
    inv = torch.from_numpy(rng.uniform(0.3, 3.0, rows).astype(np.float32)).to(DEV)
    many = [int(t) for t in rng.integers(0, vocab, 2 * rows + 3)]
    check_logprobs(x, many, [int(r) for r in rng.integers(0, rows, len(many))], inv, k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [9, 2050, 70001])
def test_logprobs_masks_ties_and_extremes(dtype, vocab):
    dt = TYPES[dtype]
    lowest, low = torch.finfo(dt).min, -math.inf
    rows = []

    def row(fill):
        rows.append(torch.full((vocab,), fill, dtype=dt))
        return rows[-1]

    row(0.0)                                  # uniform: ties everywhere
    row(low)                                  # nothing left
    row(low)[vocab - 1] = 2.5                 # one token left
    r = row(low)
    r[vocab // 2], r[vocab // 3] = 1.0, 1.0   # two equal ones
    row(lowest)                               # every token at the type's lowest value
    row(lowest)[vocab // 2] = 3.0
    r = row(-0.0)
    r[vocab // 2:] = 0.0                      # -0 and 0 are equal
    r = row(0.0)
    r[::8] = 5.0                              # a stripe: many of one thread's
    r = row(0.0)
    r[:] = torch.linspace(-8, 8, vocab).to(dt)   # sorted upwards
    r = row(0.0)
    r[:] = torch.linspace(8, -8, vocab).to(dt)   # sorted downwards
    r = row(-5.0)
    r[vocab - 3:] = 60.0                      # all mass at the end
    row(torch.finfo(dt).max)                  # every token at the type's largest value
    row(low)[0] = lowest
    x = torch.stack(rows).to(DEV)
    tokens = [vocab // 2] * len(rows)
    check_logprobs(x, tokens, k=20)
    check_logprobs(x, tokens, k=1)
    inv = torch.full((len(rows),), 0.25, device=DEV)
    check_logprobs(x, tokens, inv=inv, k=32)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [5, 3001, 40000])
def test_logprobs_flag_bad_rows_alone(dtype, vocab):
    x = make_logits(3, 6, vocab, TYPES[dtype])
    x[1, vocab - 1], x[2, 0], x[4, vocab // 2], x[5, 1] = math.nan, math.inf, -math.nan, -math.inf
    check_logprobs(x, [0] * 6, k=4, err=binding.DEVERR_LOGITS)
    y = make_logits(4, 6, vocab, TYPES[dtype])
    inv = torch.tensor([1.0, 0.0, -1.0, math.nan, math.inf, 1e-30], device=DEV)
    check_logprobs(y, [1] * 6, inv=inv, k=4, err=binding.DEVERR_LOGITS)
    if dtype != "fp16":
        z = torch.full((2, vocab), 3e38, dtype=TYPES[dtype], device=DEV)  # z past fp32's range
        z[1] = -3e38
        check_logprobs(z, [0, 0], inv=torch.tensor([2.0, 2.0], device=DEV), k=2, err=binding.DEVERR_LOGITS)


@pytest.mark.parametrize("vocab", [33, 40000])
def test_logprobs_masked_with_the_lowest_value_at_a_scale_of_one_bit(vocab):
    """c = log2(e) / temperature rounds to 1, so that a mask of fp32's lowest
    value scales to exactly the starting reference of the sums."""
    inv = np.float32(math.log(2.0))
    step = np.spacing(inv)
    inv = next(v for v in (inv, inv + step, inv - step, inv + 2 * step) if v * np.float32(1.4426950408889634) == np.float32(1))
    x = make_logits(8, 3, vocab, torch.float32).contiguous()
    x[0, :vocab // 2] = torch.finfo(torch.float32).min  # before the live ones
    x[1, vocab // 2:] = torch.finfo(torch.float32).min
    x[2, 3:] = torch.finfo(torch.float32).min
    check_logprobs(x, [vocab - 1, 0, 1], inv=torch.full((3,), float(inv), device=DEV), k=5)


def test_logprobs_far_from_zero_keep_their_differences():
    """Logits around 20000: log probabilities come from differences, not from a large ln sum."""
    x = (make_logits(5, 4, 5000, torch.float32) + 20000.0).contiguous()
    check_logprobs(x, [0, 1, 2, 3], k=8)
    check_logprobs(-x - 30000.0, [0, 1, 2, 3], inv=torch.tensor([0.7, 1.0, 1.9, 3.0], device=DEV), k=8)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [9, 3001, 150001])
@pytest.mark.parametrize("inv", [2.3e38, 2.4e38, 3.4028234663852886e38])
def test_logprobs_at_the_largest_temperatures(dtype, vocab, inv):
    """inv_temperature * log2(e) passes fp32's range from 2.3587e38 on, while z
    keeps inside it.  The largest logits are powers of two, so that z's maximum
    is exact; one row in one block, in several (150001), or in its edges (9)."""
    dt, low = TYPES[dtype], -math.inf
    rows = []

    def row(fill):
        rows.append(torch.full((vocab,), fill, dtype=dt))
        return rows[-1]

    row(-2.0 ** -7)[vocab // 2] = 0.0         # all mass on one token
    row(0.0)                                  # uniform, in every block
    r = row(-0.5)
    r[0], r[vocab - 1] = -2.0 ** -7, -2.0 ** -7  # two equal ones below 0, in two blocks
    row(low)[vocab - 1] = 0.0
    r = row(-1.0)
    r[1], r[vocab // 3], r[vocab - 2] = 0.0, -2.0 ** -126, -2.0 ** -127  # z of 0, -2.8 and -1.4 (fp16: three of 0)
    row(low)
    x = torch.stack(rows).to(DEV)
    scale = torch.full((len(rows),), inv, device=DEV)
    check_logprobs(x, [vocab // 2] * len(rows), inv=scale, k=3)
    check_logprobs(x, [0, 1, 0, vocab - 1, vocab - 2, 0, -1], [0, 1, 2, 3, 4, 5, 0], scale, 20)
    y = torch.full((1, vocab), -0.5, dtype=dt, device=DEV)
    y[0, vocab // 3] = -0.01                  # z's maximum rounds: its rest is in ln S, and goes out again
    got, word = run_logprobs(y, [vocab // 3], inv=scale[:1], k=1)
    assert word == 0 and got["top_tokens"].tolist() == [[vocab // 3]] and got["logprobs"].tolist() == [0.0]
    assert got["top_logprobs"].tolist() == [[0.0]] and got["stats"][2].tolist() == [0.0] and np.isfinite(got["stats"]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("skip", [0, 1])
@pytest.mark.parametrize("k", [32, 5, 1])
def test_logprobs_whose_large_logits_sit_in_few_threads(dtype, skip, k):
    """Fewer threads hold the large logits than ranks are asked for, in
    thousands of groups of 64 bytes: one search a rank.  Distinct values, equal
    ones, and the same behind a mask; rows at an odd address too."""
    dt, vocab = TYPES[dtype], 1 << 20
    buf = torch.zeros((4, vocab + skip), dtype=dt, device=DEV)
    x = buf[:, skip:]
    per = 64 // x.element_size()
    i = torch.arange(vocab, device=DEV)
    for r in range(4):
        head = (-(x[r].data_ptr() % 64) % 64) // x.element_size()
        res = torch.div(i - head, per, rounding_mode="floor") % 256
        # k - 1 buckets of four neighbouring threads (a block holds a multiple of 256 groups)
        few = (res // 32) * 8 + res % 8 < k - 1
        g = torch.Generator(device=DEV).manual_seed(40 + r)
        value = torch.rand((vocab,), generator=g, device=DEV) * (8 if r != 2 else 0) + 4
        low = torch.full_like(value, -math.inf) if r == 3 else torch.rand((vocab,), generator=g, device=DEV) * -8
        x[r] = torch.where(few, value, low).to(dt)
    x[3, vocab // 2] = -3.0  # (for k == 1 the only one left)
    check_logprobs(x, [0, vocab - 1, vocab // 3, vocab // 2], k=k)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("vocab", [61, 5000, 131072, 1 << 20])
@pytest.mark.parametrize("skip", [0, 1, 31])
def test_logprobs_count_every_logit_once(dtype, vocab, skip):
    """Logits of 0 and -inf alone: S is a whole number below 2^24, so that every
    sum of it is exact, and ln S is within fp32's rounding and logf's 1 ulp."""
    buf = torch.full((3, vocab + skip + 5), 9.0, dtype=TYPES[dtype], device=DEV)
    x = buf[:, skip:skip + vocab]
    x[0] = 0.0
    x[1] = -math.inf
    ends = min(vocab // 2, 40)  # the logits before and after the aligned ones, and a few more
    x[1, :ends] = 0.0
    x[1, vocab - ends + 1:] = 0.0
    x[2] = 0.0
    x[2, ::3] = -math.inf
    counts = [vocab, 2 * ends - 1, vocab - (vocab + 2) // 3]
    got, err = run_logprobs(x, [1, 1, 1], k=1)
    want = np.log(np.array(counts, dtype=np.float64))
    assert err == 0 and got["stats"][0].tolist() == [0.0] * 3
    assert np.abs(got["stats"][1] - want).max() <= 2.0 ** -22 * want.max()  # 2^-24 of ln S and an ulp of it, twice over
    missing = want - np.log(np.array(counts, dtype=np.float64) - 1)
    assert missing[1] > 2.0 ** -22 * want.max()  # one end left out would be seen
    np.testing.assert_allclose(got["stats"][2], want, atol=2.0 ** -21 * want.max())


def test_logprobs_bad_tokens_and_rows():
    x = make_logits(6, 3, 100, torch.bfloat16)
    check_logprobs(x, [100, -2, 5, -1, 7, 7], [0, 1, 3, 2, -1, 2], err=binding.DEVERR_TOKEN)
    check_logprobs(x, [100, -1, 7], err=binding.DEVERR_TOKEN)


def test_logprobs_optional_parts_and_empty_calls():
    x = make_logits(7, 3, 500, torch.float16)
    stats = torch.zeros((3, 3), device=DEV)
    pkg.token_logprobs(x, stats)
    want = S.token_logprobs(x.double().cpu().numpy(), None, [], [], 0)["stats"]
    np.testing.assert_allclose(stats.cpu().numpy(), want, rtol=1e-5)
    lp = torch.zeros(2, device=DEV)
    pkg.token_logprobs(x, stats, i32([4, 5]), lp)  # fewer tokens than rows
    want = S.token_logprobs(x.double().cpu().numpy(), None, [4, 5], [0, 1], 0)["logprobs"]
    np.testing.assert_allclose(lp.cpu().numpy(), want, rtol=1e-5)
    pkg.token_logprobs(x[:0], stats[:, :0].contiguous())
    one = x[0:1].expand(4, 500)  # rows that share memory
    check_logprobs(one, [1, 2, 3, 4], k=3)


def test_logprobs_row_offsets_past_32_bits():
    """A row 2^32 elements after the first (8.6 GB of bf16, most of it never read)."""
    V = 1000
    buf = torch.zeros((1 << 32) + V, dtype=torch.bfloat16, device=DEV)
    x = torch.as_strided(buf, (2, V), (1 << 32, 1))
    x.copy_(make_logits(9, 2, V, torch.bfloat16))
    check_logprobs(x, [3, 4], k=5)
    check_logprobs(x, [3, 4, 5], [1, 0, 1], k=5)


@pytest.mark.parametrize("rows", [1, 30, 700])
def test_logprobs_are_repeatable_and_capture(rows):
    x = make_logits(11, rows, 40001, torch.bfloat16)
    tokens, trow = i32([5] * rows), i32(list(range(rows)))
    outs = []
    for _ in range(2):
        o = [torch.zeros(rows, device=DEV), torch.zeros((3, rows), device=DEV), torch.zeros((6, rows), dtype=torch.int32, device=DEV),
             torch.zeros((6, rows), device=DEV)]
        outs.append(o)
    call = lambda o: pkg.token_logprobs(x, o[1], tokens, o[0], o[2], o[3], token_rows=trow)  # noqa: E731
    call(outs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call(outs[1])
    for shift in (0, 1):
        if shift:
            x.copy_(make_logits(12, rows, 40001, torch.bfloat16))
            call(outs[0])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b)


def test_two_calls_at_once_on_two_streams():
    """Rows and their tokens' kernel on two streams, each on its own buffers."""
    x = [make_logits(21 + k, 200, 20011, torch.bfloat16) for k in range(2)]
    trow = i32([(7 * i) % 200 for i in range(500)])
    tokens = i32([(131 * i) % 20011 for i in range(500)])
    new = lambda: [torch.zeros((3, 200), device=DEV), torch.zeros(500, device=DEV),  # noqa: E731
                   torch.zeros((4, 200), dtype=torch.int32, device=DEV), torch.zeros((4, 200), device=DEV)]
    want, got = [new(), new()], [new(), new()]
    for k in range(2):
        pkg.token_logprobs(x[k], want[k][0], tokens, *want[k][1:], token_rows=trow)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for k in range(2):
            pkg.token_logprobs(x[k], got[k][0], tokens, *got[k][1:], token_rows=trow, stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for a, b in zip(want[k], got[k]):
            assert torch.equal(a, b)


def test_a_call_runs_on_its_tensors_device(monkeypatch):
    """Another current device: the call enters the tensors' one (device 0 here)."""
    x = make_logits(30, 2, 300, torch.float32)
    a, b = torch.zeros((3, 2), device=DEV), torch.zeros((3, 2), device=DEV)
    pkg.token_logprobs(x, a)
    entered = []
    real = torch.cuda.device
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "device", lambda d: entered.append(d) or real(0))
    pkg.token_logprobs(x, b)
    monkeypatch.undo()
    assert entered == [0] and torch.equal(a, b)
    with pytest.raises(ValueError, match="one element"):
        pkg.rope_write(i64([1]), i64([0]), q_in=x.view(2, 1, 300)[:1, :, :2], q_out=x.view(2, 1, 300)[:1, :, :2], num_valid=i64([1, 1]))


def test_calls_of_several_host_threads():
    """Calls of 8192 and of 4000 requests from four threads that share nothing:
    what one call asks of the device (its shared memory) bounds no other's."""
    import threading
    lib, work = binding.load(), []
    for k, (rows, per) in enumerate([(8192, 3), (4000, 5)] * 2):
        rng, table, held, free = page_state(70 + k, rows, per, 4)
        p = Pages(table, held, free)
        prefix = [int(x) for x in rng.integers(0, 4 * per - 1, rows)]
        full = rng.permutation(rows * per).reshape(rows, per).tolist()
        keep = [i32([h * 4 + 4 for h in held]), i32([h * 4 for h in held]), i32(full), i32(prefix), i32([1] * rows)]
        out = [i32([0] * (rows + 1)), i64([0] * sum(prefix)), i64([0] * (rows + 1)), i64([0] * rows), i64([0] * rows)]
        stream, at = torch.cuda.Stream(), lambda t: t.data_ptr()
        update = lambda lens: (lib.mla_page_table_update, (  # noqa: E731
            at(lens), rows, 4, at(p.table), per, per, at(p.held), at(p.free), p.free.numel(), at(p.num), at(p.err),
            stream.cuda_stream))
        build = (lib.mla_slot_map_build, (
            at(keep[2]), per, rows, per, rows * per, 4, None, at(keep[3]), at(keep[4]), None, rows, at(out[0]), at(out[1]),
            out[1].numel(), at(out[2]), at(out[3]), at(out[4]), rows, at(p.err), stream.cuda_stream))
        work.append(dict(p=p, held=held, free=free, keep=keep, out=out, stream=stream, codes=set(),
                         calls=[update(keep[0]), update(keep[1]), build],
                         want=S.slot_map(full, 4, range(rows), prefix, [1] * rows, None)))
    torch.cuda.synchronize()
    start = threading.Barrier(len(work))

    def run(w):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(1000):
            for fn, args in w["calls"]:
                w["codes"].add(fn(*args))

    threads = [threading.Thread(target=run, args=(w,)) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w in work:
        assert w["codes"] == {0}
        for got, want in zip(w["out"], w["want"]):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        p, held, free = w["p"], w["held"], w["free"]
        assert p.held.tolist() == held and p.free[:len(free)].tolist() == free and int(p.err) == 0


def test_large_and_medium_calls_in_one_graph():
    """8192 rows, then 4000: the graph is instantiated after both."""
    sets = []
    for k, (rows, per) in enumerate([(8192, 3), (4000, 5)]):
        _, table, held, free = page_state(90 + k, rows, per, 4)
        sets.append((Pages(table, held, free), i32([4 * per] * rows), (table, held, free), [4 * per] * rows))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for p, lens, _, _ in sets:
                pkg.page_table_update(lens, 4, p.table, p.held, p.free, p.num, p.err)
    graph.replay()
    for p, _, state, lens in sets:
        t2, h2, f2, flagged = S.page_table_update(lens, 4, *state)
        assert not flagged
        p.expect(t2, h2, f2)


# ------------------------------------------------------------- the whole step

def test_a_serving_step_end_to_end():
    """Lengths to accepted tokens: pages for the trees, slot maps, rotated
    queries and latent rows, mask, verify attention, log probabilities of the
    drafts, acceptance, pages back -- against the oracles at each step."""
    import oracle
    from tests.gpu_util import compare
    rng = np.random.default_rng(17)
    bs, page, num_pages, vocab = 3, 16, 60, 997
    prefix, parents = [65, 31, 128], [W.chain_parents(4), W.star_parents(3), [-1, 0, 0, 1, 2]]
    tree = [len(p) for p in parents]
    ids = [int(x) for x in rng.permutation(num_pages)]
    held = [-(-p // page) for p in prefix]
    table = [[ids.pop() if j < held[r] else -1 for j in range(10)] for r in range(bs)]
    pg = Pages(table, held, ids, capacity=num_pages)
    t2, h2, f2, _ = S.page_table_update([p + n for p, n in zip(prefix, tree)], page, table, held, ids)
    pg.update([p + n for p, n in zip(prefix, tree)], page).expect(t2, h2, f2)

    total, kv_total = sum(tree), sum(prefix)
    par = i32([x for p in parents for x in p])
    kvp, kvi, qop = i32([0] * (bs + 1)), i64([0] * kv_total), i64([0] * (bs + 1))
    loc, pos, err = i64([0] * total), i64([0] * total), err_word()
    pkg.slot_map_build(pg.table, i32(prefix), i32(tree), page, kvp, kvi, qop, loc, pos, parents=par, num_pages=num_pages, err=err)
    want = S.slot_map(t2, page, range(bs), prefix, tree, parents)
    for got, w in zip((kvp, kvi, qop, loc, pos), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)

    g = torch.Generator().manual_seed(18)
    pool = torch.randn((num_pages * page, 576), generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn((total, 64, 576), generator=g).to(torch.bfloat16).to(DEV)
    down = torch.randn((total, 576), generator=g).to(torch.bfloat16).to(DEV)
    turns, amp = pkg.rope_freqs(64, 10000.0, pkg.RopeScaling(kind=binding.ROPE_SCALE_YARN, factor=4.0, original_len=100.0,
                                                             beta_fast=32.0, beta_slow=1.0))
    q0 = q.clone()
    pkg.rope_write(turns.cuda(), pos, amplitude=amp, q_in=q[:, :, 512:], q_out=q[:, :, 512:], k_in=down[:, 512:],
                   c_in=down[:, :512], out_cache_loc=loc, kv_pool=pool, num_valid=qop[bs:], err=err)
    check_rope(q[:, :, 512:], q0[:, :, 512:], want[4].tolist(), turns, amp, False, torch.bfloat16)
    check_rope(pool[loc][:, 512:], down[:, 512:], want[4].tolist(), turns, amp, False, torch.bfloat16)

    mask = torch.zeros(sum(n * (p + n) for p, n in zip(prefix, tree)), dtype=torch.uint8, device=DEV)
    mip = i64([0] * (bs + 1))
    binding.tree_mask_build(par, qop, kvp, bs, max(tree), binding.MASK_FULL_ROW, mask, mip, err)
    m = pkg.MlaTreeVerify(bs, max(tree), total, max(prefix))
    out, lse = m(q, pool, kvi, kvp, loc, qop, mask, mip, 192 ** -0.5)
    torch.cuda.synchronize()
    wl = W.Workload(**{**W.custom(prefix, parents, num_pages * page, seed=1).__dict__, "q": q.cpu(), "kv_pool": pool.cpu(),
                       "kv_indices": kvi.cpu(), "kv_indptr": kvp.cpu(), "out_cache_loc": loc.cpu(), "qo_indptr": qop.cpu(),
                       "custom_mask": mask.cpu(), "mask_indptr": mip.cpu(), "scale": 192 ** -0.5})
    compare(wl, out.float().cpu().reshape(-1, 512).numpy(), lse.cpu().reshape(-1).numpy(), tag="step")

    # rows 0 .. bs-1 of the logits follow the prefixes, row bs + i follows node i
    logits = make_logits(19, bs + total, vocab, torch.bfloat16)
    draft = torch.randint(0, vocab, (total,), generator=g, dtype=torch.int32).to(DEV)
    rows = [bs + int(want[2][r]) + p if p >= 0 else r for r in range(bs) for p in parents[r]]
    draft[0], draft[1] = int(logits[0].float().argmax()), int(logits[bs].float().argmax())  # request 0 follows two nodes
    got = check_logprobs(logits, draft.tolist(), rows, k=4)
    top = torch.from_numpy(got["top_tokens"][0]).to(DEV)
    alen, nodes = i32([0] * bs), torch.zeros((bs, max(tree)), dtype=torch.int32, device=DEV)
    slots, bonus = torch.zeros((bs, max(tree)), dtype=torch.int64, device=DEV), i32([0] * bs)
    binding.tree_accept(par, draft, top[bs:].contiguous(), top[:bs].contiguous(), loc, qop, bs, max(tree), alen, nodes, slots, bonus, err)
    for r in range(bs):
        a, b = int(want[2][r]), int(want[2][r + 1])
        path, bo, sl = T.tree_accept(parents[r], draft[a:b].tolist(), got["top_tokens"][0][bs + a:bs + b], got["top_tokens"][0][r], want[3][a:b])
        assert int(alen[r]) == len(path) and int(bonus[r]) == bo and slots[r, :len(path)].tolist() == sl
    assert int(alen[0]) >= 2 and int(err) == 0
    after = [p + int(a) for p, a in zip(prefix, alen.tolist())]
    pg.update(after, page).expect(*S.page_table_update(after, page, t2, h2, f2)[:3])
