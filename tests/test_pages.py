"""The page bookkeeping (resize, fork, compact) against the oracle: tables,
lengths, references and page contents equal, bit for bit.  Refusals and the
oracle's own invariants run on the CPU."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from relative_bias_gqa_b200 import build as build_mod


@pytest.fixture(scope="module")
def ra():
    build_mod.build()
    from relative_bias_gqa_b200 import rel_attn
    return rel_attn


@pytest.fixture(scope="module")
def gpu(ra):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return ra


def draw_book(rng, rows, longest, spare, width=None, window=0, sinks=0, free_rows=0.2, shared=0.3):
    """A consistent state: lengths, entries (some behind a window gone), some
    rows sharing the full pages of their neighbour's beginning."""
    lens = rng.integers(0, longest + 1, rows)
    lens[rng.random(rows) < free_rows] = 0
    width = width or -(-(longest + 200) // 64) + 2
    i = np.arange(width)[None]
    held = i * 64 < lens[:, None]
    if window:
        behind = lens[:, None] - max(window, 4) - 64 * rng.integers(0, 3, (rows, 1))
        held &= (i * 64 < sinks) | ((i + 1) * 64 > behind)
    n = int(held.sum()) + spare
    table = np.full((rows, width), -1, np.int32)
    table[held] = rng.permutation(n)[:held.sum()]
    for b in range(1, rows):
        if rng.random() < shared:
            both = held[b] & held[b - 1] & (np.arange(width) < rng.integers(0, min(lens[b], lens[b - 1]) // 64 + 1))
            table[b, both] = table[b - 1, both]
    refs = np.bincount(table[table >= 0], minlength=n).astype(np.int32)
    # what lies past a row's length may be anything
    junk = (i * 64 >= lens[:, None]) & (rng.random(table.shape) < 0.2)
    table[junk] = rng.integers(-5, 1 << 30, int(junk.sum()))
    return table, lens.astype(np.int32), refs


def to_gpu(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def same(t, ref, lens=None):
    got = t.cpu().numpy()
    if lens is None:
        assert np.array_equal(got, ref)
    else:                                         # entries within the rows' lengths
        for b, n in enumerate(np.asarray(lens).tolist()):
            k = -(-n // 64)
            assert np.array_equal(got[b, :k], ref[b, :k]), b


def references(table, lens, n):
    """Counts made anew from the table."""
    held = [p for b, L in enumerate(lens) for p in table[b, :-(-int(L) // 64)].tolist() if p >= 0]
    return np.bincount(np.array(held, dtype=np.int64), minlength=n)


# ------------------------------------------------------------------ oracle
def test_oracle_keeps_references_and_contexts():
    rng = np.random.default_rng(0)
    for window, sinks in ((0, 0), (100, 5), (1, 0)):
        table, lens, refs = draw_book(rng, 9, 700, 60, window=window, sinks=sinks)
        new = np.maximum(0, lens + rng.integers(-60, 60, 9))
        t, n, r = oracle.pages_resize_ref(table, lens, refs, new, window, sinks)
        assert np.array_equal(references(t, n, len(r)), r)
        free = np.flatnonzero(n == 0)
        if len(free) and n.max() > 0:
            pool = rng.integers(0, 1 << 30, (len(r), 3))
            t, n, r, (pool,) = oracle.pages_fork_ref(t, n, r, [int(n.argmax())], [int(free[0])], False, [pool])
            assert np.array_equal(references(t, n, len(r)), r)
            context = lambda tb, b, p: p[tb[b, :-(-int(n[b]) // 64)][tb[b, :-(-int(n[b]) // 64)] >= 0]]  # noqa: E731
            assert np.array_equal(context(t, free[0], pool), context(t, n.argmax(), pool))
            before = [context(t, b, pool) for b in range(9)]
            t, r, (pool,), live = oracle.pages_compact_ref(t, n, r, [pool])
            assert np.array_equal(references(t, n, len(r)), r) and (r[live:] == 0).all() and (r[:live] > 0).all()
            assert all(np.array_equal(x, context(t, b, pool)) for b, x in enumerate(before))


# ---------------------------------------------------------------- refusals
def book(ra, **kw):
    base = dict(num_seqs=4, max_pages_per_seq=10, num_pages=50, block_table=1 << 20, seq_lens=1 << 20, page_refs=1 << 20)
    base.update(kw)
    return ra.RelAttnPages(**base)


@pytest.mark.parametrize("kw", [dict(num_seqs=0), dict(max_pages_per_seq=0), dict(num_pages=0), dict(max_pages_per_seq=1 << 25),
                                dict(block_table=None), dict(seq_lens=2), dict(page_refs=6)])
def test_bad_books_are_refused(ra, kw):
    b, lib = book(ra, **kw), ra.lib
    ws, pool = 1 << 20, ra.RelAttnPool(1 << 20, 1024)
    assert lib.rel_attn_pages_resize(ctypes.byref(b), 1 << 20, 0, 0, ws, 1 << 30, None) == ra.REL_ATTN_ERR_INVALID_ARG
    assert lib.rel_attn_pages_fork(ctypes.byref(b), 1 << 20, 1 << 20, 1, 0, ctypes.byref(pool), 1, ws, 1 << 30, None) == ra.REL_ATTN_ERR_INVALID_ARG
    assert lib.rel_attn_pages_compact(ctypes.byref(b), ctypes.byref(pool), 1, 1 << 20, ws, 1 << 30, None) == ra.REL_ATTN_ERR_INVALID_ARG


def test_bad_arguments_are_refused(ra):
    b, lib, bad = book(ra), ra.lib, ra.REL_ATTN_ERR_INVALID_ARG
    need = int(lib.rel_attn_pages_workspace_bytes(ctypes.byref(b)))
    assert need > 256 and lib.rel_attn_pages_workspace_bytes(None) == 0
    ref, ok = ctypes.byref(b), 1 << 20
    assert lib.rel_attn_pages_resize(ref, ok, 0, 0, ok, need - 1, None) == ra.REL_ATTN_ERR_WORKSPACE_TOO_SMALL
    assert lib.rel_attn_pages_resize(ref, ok, 0, 0, ok + 16, need, None) == bad
    assert lib.rel_attn_pages_resize(ref, None, 0, 0, ok, need, None) == bad
    assert lib.rel_attn_pages_resize(ref, ok, 5, -1, ok, need, None) == bad
    pool = lambda data=ok, size=64: ctypes.byref(ra.RelAttnPool(data, size))  # noqa: E731
    for args in ((0, 0, pool(), 1), (5, 0, pool(), 1), (1, 2, pool(), 1), (1, 0, pool(ok + 8), 1), (1, 0, pool(ok, 24), 1),
                 (1, 0, pool(ok, 0), 1), (1, 0, pool(), 513), (1, 0, None, 1), (1, 0, pool(), -1)):
        assert lib.rel_attn_pages_fork(ref, ok, ok, *args, ok, need, None) == bad, args
    assert lib.rel_attn_pages_compact(ref, pool(), 1, None, ok, need, None) == bad
    assert "free pages" in ra.error_string(ra.REL_ATTN_ERR_NO_PAGES)


def test_cpu_tensors_are_refused(ra):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        ra.Pages(z(2, 3), z(2), z(9))


@pytest.mark.parametrize("kw", [dict(num_seqs=0), dict(max_pages_per_seq=1 << 25), dict(num_seqs=(1 << 30) + 1), dict(num_pages=(1 << 30) + 1),
                                dict(num_pages=(1 << 31) - 1), dict(num_seqs=(1 << 31) - 1)])
def test_sizes_out_of_range_are_refused(ra, kw):
    """... by the calls and by the query of their workspace alike."""
    b, ok, lib = ctypes.byref(book(ra, **kw)), 1 << 20, ra.lib
    assert lib.rel_attn_pages_workspace_bytes(b) == 0
    assert lib.rel_attn_pages_resize(b, ok, 0, 0, ok, 1 << 60, None) == ra.REL_ATTN_ERR_INVALID_ARG
    assert lib.rel_attn_pages_fork(b, ok, ok, 1, 0, None, 0, ok, 1 << 60, None) == ra.REL_ATTN_ERR_INVALID_ARG
    assert lib.rel_attn_pages_compact(b, None, 0, ok, ok, 1 << 60, None) == ra.REL_ATTN_ERR_INVALID_ARG


def test_an_empty_pool_is_refused(ra):
    z = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for pools in ((), (z(0, 16),)):
        with pytest.raises(ValueError, match="at least one page"):
            ra.Pages(z(2, 3), z(2), z(0), pools)


# --------------------------------------------------------------------- GPU
RESIZE = [dict(rows=1, longest=1, spare=3), dict(rows=1, longest=5000, spare=200), dict(rows=7, longest=300, spare=40),
          dict(rows=33, longest=2000, spare=500, window=100, sinks=70), dict(rows=300, longest=900, spare=3000, window=1, sinks=0),
          dict(rows=1100, longest=200, spare=9000), dict(rows=5, longest=40_000, spare=300, window=1024, sinks=4),
          dict(rows=20, longest=60, spare=70_000), dict(rows=2, longest=130_000, spare=5000, window=4096, sinks=200)]


@pytest.mark.gpu
@pytest.mark.parametrize("kw", RESIZE, ids=[str(k) for k in RESIZE])
def test_resize(gpu, kw):
    rng = np.random.default_rng(len(str(kw)))
    window, sinks = kw.get("window", 0), kw.get("sinks", 0)
    table, lens, refs = draw_book(rng, **kw)
    t, n, r = to_gpu(table, lens, refs)
    pages = gpu.Pages(t, n, r)
    for _ in range(4):
        new = np.where(rng.random(len(lens)) < 0.2, 0, np.maximum(0, lens + rng.integers(-70, 150, len(lens)))).astype(np.int32)
        new = np.minimum(new, kw["longest"] + 150)
        table, lens, refs = oracle.pages_resize_ref(table, lens, refs, new, window, sinks)
        pages.resize(*to_gpu(new), window, sinks)
        assert pages.read_status() == gpu.REL_ATTN_OK
        same(r, refs), same(n, lens), same(t, table, lens)


@pytest.mark.gpu
def test_resize_uses_pages_given_back_in_the_same_call_and_the_last_one(gpu):
    table = np.array([[3, 1, 0], [2, -1, -1], [-1, -1, -1]], np.int32)
    lens, refs = np.array([192, 64, 0], np.int32), np.array([1, 1, 1, 1], np.int32)
    t, n, r = to_gpu(table, lens, refs)
    pages = gpu.Pages(t, n, r)
    pages.resize(*to_gpu(np.array([0, 128, 128], np.int32)))
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(t, np.array([[-1, -1, -1], [2, 0, -1], [1, 3, -1]])), same(r, np.ones(4)), same(n, [0, 128, 128])


def unchanged(gpu, pages, before, status):
    assert pages.read_status() == status and pages.read_status() == gpu.REL_ATTN_OK
    for x, y in zip((pages.block_table, pages.seq_lens, pages.page_refs, *pages.pools), before):
        assert torch.equal(x, y)


@pytest.mark.gpu
def test_errors_change_nothing(gpu):
    rng = np.random.default_rng(5)
    table, lens, refs = draw_book(rng, 40, 3000, 10, window=500, sinks=64)
    pool = torch.randint(0, 1 << 30, (len(refs), 128), dtype=torch.int32, device="cuda")
    t, n, r = to_gpu(table, lens, refs)
    pages = gpu.Pages(t, n, r, [pool])
    before = [x.clone() for x in (t, n, r, pool)]
    grow = np.minimum(lens + 640, 3200).astype(np.int32)
    pages.resize(*to_gpu(grow), 500, 64)
    unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_NO_PAGES)
    for value in (-1, table.shape[1] * 64 + 1):
        bad = lens.copy()
        bad[11] = value
        pages.resize(*to_gpu(bad), 500, 64)
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
    full, free = np.flatnonzero(lens > 64), np.flatnonzero(lens == 0)
    for src, dst in (([full[0], full[1]], [free[0], free[0]]), ([full[0]], [full[1]]), ([40], [free[0]]), ([full[0]], [-1])):
        pages.fork(*to_gpu(np.array(src, np.int32), np.array(dst, np.int32)))
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
    many = np.resize(full, len(free)).astype(np.int32)
    pages.fork(*to_gpu(many, free.astype(np.int32)), copy_all=True)
    unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_NO_PAGES)
    # an entry outside the pool, and one whose page has no references
    for page in (len(refs), int(np.flatnonzero(refs == 0)[0])):
        b = int(full[0])
        old = int(t[b, 0])
        t[b, 0] = page
        before[0] = t.clone()
        pages.resize(*to_gpu(np.zeros(40, np.int32)), 500, 64)
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
        pages.fork(*to_gpu(np.array([b], np.int32), free[:1].astype(np.int32)))
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
        t[b, 0] = old


@pytest.mark.gpu
@pytest.mark.parametrize("rows,longest,spare", [(300, 600, 20), (30, 300, 40_000), (270, 40_000, 3000)])
def test_errors_of_large_plans_change_nothing(gpu, rows, longest, spare):
    """As above where a block per SM carries out the plan (many rows, many pages)."""
    rng = np.random.default_rng(rows)
    table, lens, refs = draw_book(rng, rows, longest, spare, window=500, sinks=64)
    pool = torch.randint(0, 1 << 30, (len(refs), 4), dtype=torch.int32, device="cuda")
    t, n, r = to_gpu(table, lens, refs)
    pages, live = gpu.Pages(t, n, r, [pool]), torch.full((1,), -7, dtype=torch.int32, device="cuda")
    before = [x.clone() for x in (t, n, r, pool)]
    full, free = np.flatnonzero(lens > 64), np.flatnonzero(lens == 0)
    bad = lens.copy()
    bad[rows // 2] = table.shape[1] * 64 + 1
    pages.resize(*to_gpu(bad), 500, 64)
    unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
    for src, dst in (([full[0], full[1]], [free[0], free[0]]), ([full[0]], [full[1]]), ([rows], [free[0]])):
        pages.fork(*to_gpu(np.array(src, np.int32), np.array(dst, np.int32)))
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
    if spare < 10_000:                            # more pages than are free
        pages.resize(*to_gpu(np.full(rows, table.shape[1] * 64, np.int32)))
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_NO_PAGES)
        many = np.resize(full[np.argsort(lens[full])[::-1][:8]], len(free)).astype(np.int32)
        if sum((table[m, :-(-lens[m] // 64)] >= 0).sum() for m in many) > (refs == 0).sum():
            pages.fork(*to_gpu(many, free.astype(np.int32)), copy_all=True)
            unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_NO_PAGES)
    b = int(full[-1])
    for page in (len(refs), int(np.flatnonzero(refs == 0)[0])):
        old = int(t[b, 0])
        t[b, 0] = page
        before[0] = t.clone()
        pages.resize(torch.zeros_like(n), 500, 64)
        unchanged(gpu, pages, before, gpu.REL_ATTN_ERR_BAD_SEQ)
        t[b, 0] = old
    # and then a plan that goes through
    new = np.maximum(0, lens - 30).astype(np.int32)
    want = oracle.pages_resize_ref(table, lens, refs, new, 500, 64)
    pages.resize(*to_gpu(new), 500, 64)
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(r, want[2]), same(n, want[1]), same(t, want[0], want[1])


@pytest.mark.gpu
def test_plans_of_more_tasks_than_one_round(gpu):
    """200,000 rows: more stretches of entries than the blocks hold at a time."""
    rng = np.random.default_rng(2)
    table, lens, refs = draw_book(rng, 200_000, 190, 150_000, free_rows=0.1, width=4)
    t, n, r = to_gpu(table, lens, refs)
    pages, live = gpu.Pages(t, n, r), torch.zeros(1, dtype=torch.int32, device="cuda")
    new = np.where(lens > 0, np.maximum(0, lens + rng.integers(-190, 60, len(lens))), 0).astype(np.int32)
    table, lens, refs = oracle.pages_resize_ref(table, lens, refs, new, 0, 0)
    pages.resize(*to_gpu(new))
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(r, refs), same(n, lens)
    assert np.array_equal(*(np.where(np.arange(4) * 64 < lens[:, None], x, -1) for x in (t.cpu().numpy(), table)))
    free, full = np.flatnonzero(lens == 0), np.flatnonzero(lens > 0)
    src, dst = np.resize(full, len(free)).astype(np.int32), free.astype(np.int32)
    table, lens, refs, _ = oracle.pages_fork_ref(table, lens, refs, src, dst, False)
    pages.fork(*to_gpu(src, dst))
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(r, refs), same(n, lens)
    assert np.array_equal(*(np.where(np.arange(4) * 64 < lens[:, None], x, -1) for x in (t.cpu().numpy(), table)))
    table, refs, _, count = oracle.pages_compact_ref(table, lens, refs)
    pages.compact(live)
    assert pages.read_status() == gpu.REL_ATTN_OK and int(live) == count
    same(r, refs)
    assert np.array_equal(*(np.where(np.arange(4) * 64 < lens[:, None], x, -1) for x in (t.cpu().numpy(), table)))


@pytest.mark.gpu
def test_one_page_shared_by_millions_of_entries(gpu):
    rows, width = 640, 20_000
    lens = np.zeros(rows, np.int32)
    lens[::2] = (width - np.arange(rows // 2) % 7) * 64
    i = np.arange(width)[None]
    held = i * 64 < lens[:, None]
    refs = np.zeros(100, np.int32)
    refs[0] = held.sum()
    t, n, r = to_gpu(np.where(held, 0, -1).astype(np.int32), lens, refs)
    pages = gpu.Pages(t, n, r)
    new = lens // 2
    new[::4] = 0
    pages.resize(*to_gpu(new))
    assert pages.read_status() == gpu.REL_ATTN_OK
    keep = held & (i * 64 < new[:, None])
    same(n, new)
    assert int(r[0]) == int(keep.sum()) and not r[1:].any()
    assert torch.equal(t, torch.from_numpy(np.where(keep, 0, -1).astype(np.int32)).cuda())


@pytest.mark.gpu
def test_wait_limit(gpu):
    """With an injected one-nanosecond limit the blocks of a large plan either
    meet at once or the call ends with TIMEOUT; with a fresh workspace and state
    the next one is right."""
    rng = np.random.default_rng(4)
    table, lens, refs = draw_book(rng, 400, 2000, 30_000)
    lens[-1] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    pool = rng.integers(0, 1 << 30, (len(refs), 4), dtype=np.int32)
    src, dst = np.array([int(lens.argmax())], np.int32), np.array([399], np.int32)
    new = np.where(lens > 0, lens + 100, 0).astype(np.int32)
    want = oracle.pages_resize_ref(table, lens, refs, new, 300, 10)
    want = oracle.pages_fork_ref(*want, src, dst, True, [pool])
    last = oracle.pages_compact_ref(want[0], want[1], want[2], want[3])
    for limit in (1, 1, 1, 0):
        t, n, r, p = to_gpu(table, lens, refs, pool)
        pages, live = gpu.Pages(t, n, r, [p]), torch.zeros(1, dtype=torch.int32, device="cuda")
        gpu.rel_attn_set_wait_limit(limit)
        try:
            for call in (lambda: pages.resize(*to_gpu(new), 300, 10), lambda: pages.fork(*to_gpu(src, dst), copy_all=True),
                         lambda: pages.compact(live)):
                call()
                status = pages.read_status()
                assert status == gpu.REL_ATTN_OK or (limit and status == gpu.REL_ATTN_ERR_TIMEOUT)
                if status != gpu.REL_ATTN_OK:
                    break
            else:
                same(r, last[1]), same(n, want[1]), same(t, last[0], want[1]), same(p, last[2][0])
        finally:
            gpu.rel_attn_set_wait_limit(0)


@pytest.mark.gpu
def test_rows_named_twice_and_lengths_that_are_the_books_own(gpu):
    """A source several times, free rows as sources, and resize with new_lens
    being seq_lens itself (pages behind a window given back)."""
    rng = np.random.default_rng(3)
    table, lens, refs = draw_book(rng, 12, 900, 200)
    lens[-5:] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    t, n, r = to_gpu(table, lens, refs)
    pages = gpu.Pages(t, n, r)
    a = int(lens.argmax())
    for src, dst in (([a, a, 11, 8], [7, 8, 9, 10]),):
        pages.fork(*to_gpu(np.array(src, np.int32), np.array(dst, np.int32)))
        table, lens, refs, _ = oracle.pages_fork_ref(table, lens, refs, src, dst, False)
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(r, refs), same(n, lens), same(t, table, lens)
    pages.resize(n, 100, 3)
    table, lens, refs = oracle.pages_resize_ref(table, lens, refs, lens, 100, 3)
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(r, refs), same(n, lens), same(t, table, lens)


FORK = [dict(rows=2, longest=64, spare=4), dict(rows=2, longest=65, spare=400), dict(rows=30, longest=700, spare=3000),
        dict(rows=50, longest=4000, spare=9000, window=300, sinks=70), dict(rows=2200, longest=130, spare=6000)]


@pytest.mark.gpu
@pytest.mark.parametrize("copy_all", [False, True])
@pytest.mark.parametrize("kw", FORK, ids=[str(k) for k in FORK])
def test_fork(gpu, kw, copy_all):
    rng = np.random.default_rng(len(str(kw)))
    table, lens, refs = draw_book(rng, free_rows=0.5, **kw)
    if (lens == 0).all():
        lens[:] = 0
    lens[-1] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    free, full = np.flatnonzero(lens == 0), np.flatnonzero(lens > 0)
    if len(full) == 0:
        table[0, 0], lens[0], refs[0] = 0, 33, 1
        free, full = np.flatnonzero(lens == 0), np.array([0])
    k = max(1, len(free) - 1)
    src, dst = rng.choice(full, k).astype(np.int32), rng.permutation(free)[:k].astype(np.int32)
    pools = [rng.integers(0, 255, (len(refs), 48), dtype=np.uint8), rng.integers(0, 1 << 30, (len(refs), 2, 8), dtype=np.int32)]
    t, n, r, *p = to_gpu(table, lens, refs, *pools)
    pages = gpu.Pages(t, n, r, p)
    pages.fork(*to_gpu(src, dst), copy_all=copy_all)
    try:
        table, lens, refs, pools = oracle.pages_fork_ref(table, lens, refs, src, dst, copy_all, pools)
        assert pages.read_status() == gpu.REL_ATTN_OK
    except oracle.NoPages:
        assert pages.read_status() == gpu.REL_ATTN_ERR_NO_PAGES
    same(r, refs), same(n, lens), same(t, table, lens)
    for x, y in zip(p, pools):
        same(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", FORK + [dict(rows=3, longest=900, spare=0), dict(rows=4, longest=100, spare=70_000)],
                         ids=lambda k: str(k))
def test_compact(gpu, kw):
    rng = np.random.default_rng(len(str(kw)) + 1)
    table, lens, refs = draw_book(rng, **kw)
    pools = [rng.integers(0, 255, (len(refs), 48), dtype=np.uint8), rng.integers(0, 1 << 30, (len(refs), 2, 8), dtype=np.int32)]
    t, n, r, *p = to_gpu(table, lens, refs, *pools)
    pages, live = gpu.Pages(t, n, r, p), torch.full((1,), -7, dtype=torch.int32, device="cuda")
    for _ in range(2):                            # the second time nothing moves
        pages.compact(live)
        table, refs, pools, count = oracle.pages_compact_ref(table, lens, refs, pools)
        assert pages.read_status() == gpu.REL_ATTN_OK and int(live) == count
        same(r, refs), same(n, lens), same(t, table, lens)
        for x, y in zip(p, pools):
            same(x, y)


@pytest.mark.gpu
def test_large_pages_of_many_pools(gpu):
    """Pages of other sizes than a whole number of chunks, 70 pools of them."""
    rng = np.random.default_rng(3)
    table, lens, refs = draw_book(rng, 6, 500, 30)
    lens[-1] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    sizes = [16, 8192, 16400, 16384, 50_000 // 16 * 16, 131_072] + [32] * 64
    pools = [torch.randint(0, 255, (len(refs), s), dtype=torch.uint8, device="cuda") for s in sizes]
    ref = [x.cpu().numpy() for x in pools]
    t, n, r = to_gpu(table, lens, refs)
    pages, live = gpu.Pages(t, n, r, pools), torch.zeros(1, dtype=torch.int32, device="cuda")
    src = np.array([int(lens.argmax())], np.int32)
    pages.fork(*to_gpu(src, np.array([5], np.int32)), copy_all=True)
    table, lens, refs, ref = oracle.pages_fork_ref(table, lens, refs, src, [5], True, ref)
    lens[0] = 0
    n[0] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    r.copy_(torch.from_numpy(refs))
    pages.compact(live)
    table, refs, ref, count = oracle.pages_compact_ref(table, lens, refs, ref)
    assert pages.read_status() == gpu.REL_ATTN_OK and int(live) == count
    same(r, refs), same(t, table, lens)
    for x, y in zip(pools, ref):
        same(x, y)


@pytest.mark.gpu
def test_captured_steps(gpu):
    """resize, fork and compact captured into one graph and replayed."""
    rng = np.random.default_rng(8)
    table, lens, refs = draw_book(rng, 12, 900, 200, width=40)
    lens[-2:] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    pool = rng.integers(0, 1 << 30, (len(refs), 32), dtype=np.int32)
    t, n, r, p = to_gpu(table, lens, refs, pool)
    new, src, dst = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (12, 1, 1))
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    keep = [x.clone() for x in (t, n, r, p)]
    pages = gpu.Pages(t, n, r, [p])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pages.resize(new, 300, 10)
            pages.fork(src, dst)
            pages.compact(live)
        for x, y in zip((t, n, r, p), keep):
            x.copy_(y)
        for step in range(5):
            to = np.minimum(np.where(lens > 0, lens + rng.integers(-5, 80, 12), 0).clip(0), 1500).astype(np.int32)
            to[10:] = 0
            new.copy_(torch.from_numpy(to))
            src.fill_(step % 9)
            dst.fill_(10 + step % 2)
            g.replay()
            s.synchronize()
            table, lens, refs = oracle.pages_resize_ref(table, lens, refs, to, 300, 10)
            table, lens, refs, (pool,) = oracle.pages_fork_ref(table, lens, refs, [step % 9], [10 + step % 2], False, [pool])
            table, refs, (pool,), count = oracle.pages_compact_ref(table, lens, refs, [pool])
            assert pages.read_status() == gpu.REL_ATTN_OK and int(live) == count
            same(r, refs), same(n, lens), same(t, table, lens), same(p, pool)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,forks", [(100, 40), (250, 120), (300, 140), (2100, 1000)])
@pytest.mark.parametrize("backwards", [False, True])
def test_free_rows_as_sources_that_the_same_call_fills(gpu, rows, forks, backwards):
    """A chain in one call: its first forks fill rows that its last forks (of other
    warps and blocks) have as sources, or the other way round; those sources count
    as they were, free.  Ten times over, each from the same state."""
    rng = np.random.default_rng(forks)
    table, lens, refs = draw_book(rng, rows, 200, 3 * rows + forks * 4, free_rows=0.0)
    lens[rows // 2:] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    half = forks // 2
    free = rows // 2 + rng.permutation(rows - rows // 2)
    filled, chained = free[:half], free[half:forks]
    src = np.concatenate([rng.choice(np.flatnonzero(lens > 0), half), filled]).astype(np.int32)
    dst = np.concatenate([filled, chained]).astype(np.int32)
    if backwards:
        src, dst = src[::-1], dst[::-1]
    want = oracle.pages_fork_ref(table, lens, refs, src, dst, False)
    assert (want[1][chained] == 0).all() and (want[1][filled] > 0).all()
    for _ in range(10):
        t, n, r = to_gpu(table, lens, refs)
        pages = gpu.Pages(t, n, r)
        pages.fork(*to_gpu(src, dst))
        assert pages.read_status() == gpu.REL_ATTN_OK
        same(n, want[1]), same(r, want[2]), same(t, want[0], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("rows,longest,spare", [(12, 900, 60), (300, 600, 300), (20, 300, 40_000)])
@pytest.mark.parametrize("moves", [False, True])
def test_compact_reports_a_bad_book(gpu, rows, longest, spare, moves):
    """A length out of range, an entry outside the pool and one whose page has no
    references, each by itself, where pages move and where none does: left as they
    were, reported, and the rest compacted as if they were not there."""
    rng = np.random.default_rng(rows)
    table, lens, refs = draw_book(rng, rows, longest, spare, free_rows=0.1)
    lens[:3] = longest // 2
    table[:3, :-(-longest // 128)] = -1
    refs = references(table, lens, len(refs)).astype(np.int32)
    if not moves:
        table, refs, _, _ = oracle.pages_compact_ref(table, lens, refs)
        refs = refs.astype(np.int32)
    hole = np.flatnonzero(refs == 0)
    faults = [dict(length=-1), dict(length=table.shape[1] * 64 + 1), dict(entry=len(refs)), dict(entry=2 ** 31 - 1),
              dict(entry=int(hole[0])), dict(entry=int(hole[-1]))]
    for fault in faults:
        bad, long = table.astype(np.int32), lens.copy()
        if "length" in fault:
            long[1] = fault["length"]
        else:
            bad[1, 2] = fault["entry"]
        t, n, r = to_gpu(bad, long, refs)
        pages, live = gpu.Pages(t, n, r), torch.zeros(1, dtype=torch.int32, device="cuda")
        pages.compact(live)
        assert pages.read_status() == gpu.REL_ATTN_ERR_BAD_SEQ and pages.read_status() == gpu.REL_ATTN_OK
        want, want_refs, _, count = oracle.pages_compact_ref(table, lens, refs)
        assert (want_refs != refs).any() == moves
        if "entry" in fault:
            want[1, 2] = fault["entry"]
        assert int(live) == count
        same(r, want_refs), same(n, long), same(t, want, lens)


@pytest.mark.gpu
def test_captured_steps_of_a_large_plan(gpu):
    """resize and fork in one graph, compact in another, replayed in turn: a plan of
    a block per SM, and both graphs on one workspace."""
    rng = np.random.default_rng(8)
    rows = 300
    table, lens, refs = draw_book(rng, rows, 900, 4000, width=40)
    lens[-60:] = 0
    refs = references(table, lens, len(refs)).astype(np.int32)
    pool = rng.integers(0, 1 << 30, (len(refs), 4), dtype=np.int32)
    t, n, r, p = to_gpu(table, lens, refs, pool)
    new, src, dst = (torch.zeros(k, dtype=torch.int32, device="cuda") for k in (rows, 20, 20))
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    pages = gpu.Pages(t, n, r, [p])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(one, stream=s):
            pages.resize(new, 300, 10)
            pages.fork(src, dst)
        with torch.cuda.graph(two, stream=s):
            pages.compact(live)
        for step in range(6):
            to = np.minimum(np.where(lens > 0, lens + rng.integers(-5, 80, rows), 0).clip(0), 1500).astype(np.int32)
            to[-60:] = 0
            a, b = rng.integers(0, rows - 60, 20).astype(np.int32), (rows - 60 + rng.permutation(60)[:20]).astype(np.int32)
            for x, y in ((new, to), (src, a), (dst, b)):
                x.copy_(torch.from_numpy(y))
            one.replay()
            two.replay()
            s.synchronize()
            table, lens, refs = oracle.pages_resize_ref(table, lens, refs, to, 300, 10)
            table, lens, refs, (pool,) = oracle.pages_fork_ref(table, lens, refs, a, b, False, [pool])
            table, refs, (pool,), count = oracle.pages_compact_ref(table, lens, refs, [pool])
            assert pages.read_status() == gpu.REL_ATTN_OK and int(live) == count
            same(r, refs), same(n, lens), same(t, table, lens), same(p, pool)


@pytest.mark.gpu
def test_two_large_plans_at_once(gpu):
    """Books of their own on two streams: each a block per SM, at the same time."""
    rng, runs = np.random.default_rng(6), []
    for rows in (300, 400):
        table, lens, refs = draw_book(rng, rows, 2000, 30_000)
        more = np.where(lens > 0, lens + 130, 0).astype(np.int32)
        want = oracle.pages_resize_ref(*oracle.pages_resize_ref(table, lens, refs, more, 0, 0), lens, 0, 0)
        t, n, r, up, down = to_gpu(table, lens, refs, more, lens)
        s = torch.cuda.Stream()
        runs.append((gpu.Pages(t, n, r, stream=s), up, down, want))
    torch.cuda.synchronize()
    for _ in range(20):
        for pages, up, down, _ in runs:
            pages.resize(up)
            pages.resize(down)
    torch.cuda.synchronize()
    for pages, _, _, want in runs:
        assert pages.read_status() == gpu.REL_ATTN_OK
        same(pages.page_refs, want[2]), same(pages.seq_lens, want[1]), same(pages.block_table, want[0], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, 5)])
def test_resize_with_the_largest_windows_and_sinks(gpu, window, sinks):
    rng = np.random.default_rng(3)
    table, lens, refs = draw_book(rng, 20, 900, 200)
    t, n, r = to_gpu(table, lens, refs)
    pages = gpu.Pages(t, n, r)
    new = np.maximum(0, lens + rng.integers(-70, 150, 20)).astype(np.int32)
    table, lens, refs = oracle.pages_resize_ref(table, lens, refs, new, window, sinks)
    pages.resize(*to_gpu(new), window, sinks)
    assert pages.read_status() == gpu.REL_ATTN_OK
    same(r, refs), same(n, lens), same(t, table, lens)
