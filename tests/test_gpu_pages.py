"""The page pool's calls on the GPU against their sequential host definitions:
tables, reference counts, copy lists and page contents, all exactly."""
import numpy as np
import pytest
import torch

from helpers_kv8 import dev_i32
from oracle import pages
from tree_verification_jsv_b200 import jsv

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from tree_verification_jsv_b200 import build
    build.build()
    jsv.load()


class Pool:
    """A pool on the device beside its host copy; every call is made on both
    and compared."""

    def __init__(self, num, B, width, ref=None, table=None):
        self.num, self.B, self.width = num, B, width
        self.ref = np.zeros(num, np.int32) if ref is None else np.asarray(ref, np.int32)
        self.table = np.full((B, width), -1, np.int32) if table is None else np.asarray(table, np.int32)
        self.dref, self.dtable = dev_i32(self.ref), dev_i32(self.table)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.pool = jsv.make_page_pool(num_pages=num, refcount=self.dref, dev_status=self.status)
        self.ws = torch.full((jsv.jsv_pages_workspace_size(num, max(B, 64)),), 255, dtype=torch.uint8, device="cuda")

    def check(self, errors):
        torch.cuda.synchronize()
        assert np.array_equal(self.dtable.cpu().numpy(), self.table)
        assert np.array_equal(self.dref.cpu().numpy(), self.ref)
        st = int(self.status.item())
        assert st in errors if errors else st == 0, (st, errors)
        self.status.zero_()
        return errors

    def alloc(self, begin, end, full_only=False):
        jsv.jsv_pages_alloc(self.pool, self.dtable, self.B, self.width, None if begin is None else dev_i32(begin),
                            dev_i32(end), full_only, self.ws)
        return self.check(pages.alloc(self.ref, self.table, begin, end, full_only))

    def fork(self, src, dst, length, full_only=False):
        n = len(src)
        lists = [torch.full((n + 1,), 55, dtype=torch.int32, device="cuda") for _ in range(2)]
        jsv.jsv_pages_fork(self.pool, self.dtable, self.B, self.width, n, dev_i32(src), dev_i32(dst), dev_i32(length),
                           full_only, *lists, self.ws)
        errors, copies = pages.fork(self.ref, self.table, np.asarray(src), np.asarray(dst), np.asarray(length), full_only)
        self.check(errors)
        got = [x.cpu().numpy() for x in lists]
        assert np.array_equal(np.stack([x[:n] for x in got], 1), copies) and got[0][n] == got[1][n] == 55
        return errors

    def trim(self, keep_begin, keep_end):
        jsv.jsv_pages_trim(self.pool, self.dtable, self.B, self.width,
                           None if keep_begin is None else dev_i32(keep_begin), dev_i32(keep_end))
        return self.check(pages.trim(self.ref, self.table, keep_begin, keep_end))

    def compact(self, in_place=False):
        most = max(self.num // 2, 1)
        lists = [torch.full((most + 1,), 55, dtype=torch.int32, device="cuda") for _ in range(2)]
        table = self.dtable.clone() if in_place else self.dtable
        new_table = table if in_place else torch.full_like(table, 99)
        new_ref, count = torch.full_like(self.dref, 99), torch.full((1,), 99, dtype=torch.int32, device="cuda")
        jsv.jsv_pages_compact(self.pool, table, self.B, self.width, new_table, new_ref, *lists, most, count, self.ws)
        errors, t, r, moves = pages.compact(self.ref, self.table)
        self.check(errors)
        assert np.array_equal(new_table.cpu().numpy(), t) and np.array_equal(new_ref.cpu().numpy(), r)
        want = np.full((most, 2), -1, np.int32)
        want[:len(moves)] = np.asarray(moves, np.int32).reshape(-1, 2)
        got = [x.cpu().numpy() for x in lists]
        assert np.array_equal(np.stack([x[:most] for x in got], 1), want) and got[0][most] == got[1][most] == 55
        assert int(count.item()) == len(moves)
        return new_table, new_ref, lists, count, errors


@pytest.mark.parametrize("num", [1, 7, 64, 5000, 70001])
def test_alloc_fork_trim_compact_turns(num):
    """Random turns on pools from one page to more than one run a thread."""
    rng = np.random.default_rng(num)
    B, width = 24, max(2, min(num // 8, 400))
    p = Pool(num, B, width)
    length = np.zeros(B, int)
    seen = set()
    for turn in range(8):
        length = np.where(rng.random(B) < 0.3, 0, length)
        keep = np.maximum(length - rng.integers(0, 20, B), 0)
        seen |= p.trim(None, keep)
        length = keep
        empty, held = np.flatnonzero(length == 0), np.flatnonzero(length > 0)
        if len(held) and len(empty):
            src, dst = rng.choice(held, len(empty)), rng.permutation(empty)
            ln = np.array([rng.integers(0, length[s] + 1) for s in src])
            if not p.fork(src, dst, ln):
                length[dst] = ln
            else:
                seen.add(pages.NO_PAGES)
                length = np.where((p.table >= 0).any(1), length, 0)
                for d, x in zip(dst, ln):
                    if (p.table[d] >= 0).any():
                        length[d] = x
        want = np.minimum(length + rng.integers(0, max(num * 16 // B, 2), B), width * 16)
        if not p.alloc(length, want):
            length = want
        p.compact(in_place=turn % 2 == 1)
    assert np.array_equal(np.bincount(p.table[p.table >= 0], minlength=num), p.ref)


def test_alloc_serves_rows_in_order_and_reports_exhaustion():
    p = Pool(5, 4, 8)
    assert p.alloc(None, [40, 0, 60, 10]) == {pages.NO_PAGES}
    assert p.alloc(None, [40, 0, 30, 0]) == set()
    assert p.alloc(None, [41, 0, 0, 1], full_only=True) == set()


def test_alloc_fills_holes_of_a_row_and_full_pages_only():
    table = np.full((3, 6), -1, np.int32)
    table[0, [0, 2]] = [9, 4]
    ref = np.zeros(12, np.int32)
    ref[[9, 4]] = 1
    p = Pool(12, 3, 6, ref, table)
    p.alloc([0, 17, 0], [96, 40, 31], full_only=True)
    p.alloc([0, 17, 0], [96, 40, 31])


@pytest.mark.parametrize("begin,end", [([5, 0], [4, 16]), ([-3, 0], [4, 16]), ([0, 0], [97, 16])])
def test_alloc_and_trim_refuse_bad_rows(begin, end):
    p = Pool(20, 2, 6)
    assert p.alloc(begin, end) == {pages.DEVICE_INPUT}
    assert p.trim(begin, end) == {pages.DEVICE_INPUT}


def test_fork_refusals_leave_everything_as_it_was():
    p = Pool(30, 6, 5)
    p.alloc(None, [37, 20, 0, 0, 0, 0])
    # same row twice (the first is made), a source that is a destination, a
    # mapped destination, itself, out of range, a length past the row, and a
    # partial page that is not there
    assert p.fork([0, 1, 0, 2, 0, 0, -1, 0, 0], [2, 2, 1, 3, 0, 6, 3, 4, 5], [37, 20, 5, 4, 3, 3, 3, 81, 60]) == {pages.DEVICE_INPUT}
    assert (p.table[2] >= 0).sum() == 3 and (p.table[3:] == -1).all()
    assert p.fork([], [], []) == set()


def test_fork_full_pages_only_and_without_free_pages():
    p = Pool(4, 4, 4)
    p.alloc(None, [50, 0, 0, 0])
    assert p.fork([0, 0], [1, 2], [50, 48]) == {pages.NO_PAGES}     # the first needs a fifth page
    assert p.fork([0, 0], [1, 3], [50, 33], full_only=True) == set()


def test_trim_reports_free_and_foreign_pages():
    table = np.array([[0, 7, 2, -1], [1, 1, -5, 3]], np.int32)
    p = Pool(4, 2, 4, [1, 1, 0, 3], table)
    assert p.trim(None, [0, 0]) == {pages.DEVICE_INPUT}
    assert (p.table == -1).all() and p.ref.tolist() == [0, 0, 0, 2]


def test_compact_reports_entries_of_free_pages():
    table = np.array([[5, 3, 1, -1, 9]], np.int32)
    p = Pool(6, 1, 5, [0, 1, 0, 0, 0, 2], table)
    assert p.compact()[-1] == {pages.DEVICE_INPUT}


@pytest.mark.parametrize("page_bytes,offset", [((4096, 64, 4), 0), ((20, 65536 + 16, 8), 0), ((48, 256, 12), 4)])
def test_copy_moves_whole_pages_of_every_buffer(page_bytes, offset):
    rng = np.random.default_rng(3)
    num, n = 40, 13
    order = rng.permutation(num)
    src, dst = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
    src[4], dst[4] = -1, -1
    dst[7] = src[7]
    raw = [torch.randint(0, 255, (num * b + 2 * offset,), dtype=torch.uint8, device="cuda") for b in page_bytes]
    bufs = [x[offset:offset + num * b].view(num, b) for x, b in zip(raw, page_bytes)]
    want = [x.cpu().numpy().copy() for x in raw]
    p = Pool(num, 1, 1)
    for use in (9, n):
        count = torch.tensor([use], dtype=torch.int32, device="cuda")
        jsv.jsv_pages_copy(p.pool, jsv.make_page_buffers(bufs, page_bytes), dev_i32(src), dev_i32(dst), n,
                           count if use == 9 else None)
        torch.cuda.synchronize()
        for x, w, b in zip(raw, want, page_bytes):
            v = w[offset:offset + num * b].reshape(num, b)
            for i in range(use):
                if src[i] >= 0:
                    v[dst[i]] = v[src[i]].copy()
            assert np.array_equal(x.cpu().numpy(), w)
    assert int(p.status.item()) == 0


def test_copy_many_buffers_and_bad_pairs():
    num = 6
    bufs = [torch.arange(num, dtype=torch.int32, device="cuda").view(num, 1) + 100 * i for i in range(150)]
    p = Pool(num, 1, 1)
    jsv.jsv_pages_copy(p.pool, jsv.make_page_buffers(bufs, [4] * 150), dev_i32([1, 6, 2, 3]), dev_i32([0, 4, -1, 6]), 4)
    torch.cuda.synchronize()
    for i, x in enumerate(bufs):
        assert x.view(-1).cpu().tolist() == [100 * i + v for v in (1, 1, 2, 3, 4, 5)]
    assert int(p.status.item()) == jsv.JSV_ERR_DEVICE_INPUT


def test_turn_in_a_graph_and_on_another_stream():
    """Trim, fork, alloc and copy captured once and replayed: a turn that
    starts from the same rows gives the same pages."""
    rng = np.random.default_rng(9)
    num, B, width = 200, 10, 20
    p = Pool(num, B, width)
    p.alloc(None, [100, 37] + [0] * 8)
    keep, src, dst = dev_i32([100, 37] + [0] * 8), dev_i32([0, 1, 0]), dev_i32([2, 5, 9])
    ln, end = dev_i32([100, 37, 64]), dev_i32([130, 60, 120, 0, 0, 70, 0, 0, 0, 80])
    lists = [torch.empty(3, dtype=torch.int32, device="cuda") for _ in range(2)]
    data = torch.randint(0, 255, (num, 256), dtype=torch.uint8, device="cuda")
    held = jsv.make_page_buffers([data], [256])

    def turn():
        jsv.jsv_pages_trim(p.pool, p.dtable, B, width, None, keep)
        jsv.jsv_pages_fork(p.pool, p.dtable, B, width, 3, src, dst, ln, False, *lists, p.ws)
        jsv.jsv_pages_alloc(p.pool, p.dtable, B, width, None, end, False, p.ws)
        jsv.jsv_pages_copy(p.pool, held, *lists, 3)

    turn()
    torch.cuda.synchronize()
    want = [x.clone() for x in (p.dtable, p.dref, *lists, data)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (p.dtable, p.dref, *lists, data)))
    assert int(p.status.item()) == 0
