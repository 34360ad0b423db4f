"""A page pool's calls (allocate, release, fork, compact, copy) against plain lists."""

import pytest
import torch

import pages_ref as P

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def gpu(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(pages, live, seed):
    """Counts of a pool, about `live` of whose pages are in use."""
    g = torch.Generator().manual_seed(seed)
    refs = torch.randint(1, 4, (pages,), generator=g)
    return torch.where(torch.rand(pages, generator=g) < live, refs, 0).tolist(), g


def make_caches(pages, g):
    """Pages of many sizes and layouts: 16-, 4- and 1-byte copies, heads outside of tokens, a stride
    between pages, a scale a page."""
    def ints(*shape):
        return torch.randint(0, 255, shape, generator=g, dtype=torch.uint8).cuda()
    wide = ints(pages, 300)
    return [ints(pages, 16, 2, 64), ints(pages, 2, 16, 128).view(BF16).transpose(1, 2), ints(pages, 7),
            ints(pages, 8, 4).view(torch.float32)[..., 0], wide[:, :290], wide[:, 292:296],
            ints(pages, 4128).view(torch.int32), ints(pages, 9000), ints(pages)]


def table_of(rows, width, refs, g, lens, page):
    """Rows that name pages in use (any, also twice), -1 behind their lengths."""
    held = [p for p, n in enumerate(refs) if n > 0] or [0]
    t = [[held[int(torch.randint(0, len(held), (1,), generator=g))] for _ in range(width)]
         for _ in range(rows)]
    for row, n in zip(t, lens):
        for c in range(-(-max(n, 0) // page), width):
            row[c] = -1
    return t


@pytest.mark.parametrize("pages,reqs,ql,page,width", [
    (40, 5, 1, 16, 8), (300, 64, 4, 128, 30), (5000, 7, 700, 16, 64), (70000, 300, 33, 32, 20),
    (8, 20, 1, 16, 4), (1, 1, 1, 128, 1), (3000, 3, 2048, 1, 3000)])
@pytest.mark.parametrize("live", [0.0, 0.5, 0.97])
def test_allocate(mm, pages, reqs, ql, page, width, live):
    refs, g = pool(pages, live, pages + ql)
    lens = torch.randint(0, width * page + 1, (reqs,), generator=g).tolist()
    lens[0] = width * page
    table = table_of(reqs, width, refs, g, [max(n - ql, 0) for n in lens], page)
    for row in table[::3]:                    # a draft taken back has left its page
        row[min(width - 1, lens[0] // page)] = 0
    r, t = gpu(refs), gpu(table)
    wide = torch.full((reqs, width + 3), 77, dtype=torch.int32, device="cuda")
    wide[:, :width] = t
    got = mm.allocate_pages(r, wide[:, :width], gpu(lens), query_len=ql, page_size=page)
    short = P.allocate_ref(refs, table, lens, ql, page)
    assert mm.get_device_error() == (mm.DEV_NO_PAGES if short else 0)
    assert got.tolist() == table and r.tolist() == refs and (wide[:, width:] == 77).all()
    # a second call finds every column taken
    mm.allocate_pages(r, wide[:, :width], gpu(lens), query_len=ql, page_size=page)
    assert r.tolist() == refs and wide[:, :width].tolist() == table
    mm.get_device_error()


def test_allocate_reports_lengths_beyond_the_table(mm):
    refs, table = [0] * 10, [[-1, -1], [-1, -1]]
    r, t = gpu(refs), gpu(table)
    mm.allocate_pages(r, t, gpu([40, -3]), query_len=2, page_size=16)
    P.allocate_ref(refs, table, [40, -3], 2, 16)
    assert mm.get_device_error() == mm.DEV_SEQ_TOO_LONG
    assert t.tolist() == table and r.tolist() == refs


@pytest.mark.parametrize("rows,width,pages", [(1, 1, 1), (3, 50, 20), (200, 300, 5000)])
def test_release(mm, rows, width, pages):
    refs, g = pool(pages, 0.7, rows)
    table = torch.randint(-2, pages, (rows, width), generator=g)
    want, missing = list(refs), False
    for p in table.flatten().tolist():
        if p >= 0:
            missing |= want[p] == 0
            want[p] = max(0, want[p] - 1)
    r, t = gpu(refs), table.to(torch.int32).cuda()
    assert mm.release_pages(r, t) is r
    assert r.tolist() == want and t.tolist() == table.tolist()
    assert mm.get_device_error() == (mm.DEV_NOT_HELD if missing else 0)


def test_release_by_lengths_and_bad_pages(mm):
    refs = [3] * 6
    table = gpu([[0, 1, 2, 9], [3, -1, 4, 4], [5, 5, 5, 5], [1, 1, 1, 1]])
    r = gpu(refs)
    mm.release_pages(r, table, seq_lens=gpu([33, 48, 0, -7]), page_size=16)
    assert r.tolist() == [2, 2, 2, 2, 2, 3] and mm.get_device_error() == 0
    mm.release_pages(r, table[:1], seq_lens=gpu([1000]), page_size=16)
    assert r.tolist() == [1, 1, 1, 2, 2, 3] and mm.get_device_error() == mm.DEV_BAD_PAGE


@pytest.mark.parametrize("pages,reqs,forks,page,width", [
    (60, 3, 4, 16, 12), (400, 8, 64, 128, 20), (9, 2, 12, 16, 3), (3000, 40, 500, 64, 33),
    (1, 1, 1, 16, 1)])
def test_fork(mm, pages, reqs, forks, page, width):
    refs, g = pool(pages, 0.6, pages)
    lens = torch.randint(0, width * page + 1, (reqs,), generator=g).tolist()
    lens[0] = width * page
    table = table_of(reqs, width, refs, g, lens, page)
    parents = torch.randint(-1, reqs, (forks,), generator=g).tolist()
    caches = make_caches(pages, g)
    before = [c.clone() for c in caches]
    r = gpu(refs)
    t, n = mm.fork_pages(r, gpu(table), gpu(lens), gpu(parents), caches, page_size=page)
    want_rows, want_lens, pairs = P.fork_ref(refs, table, lens, parents, page)
    asked = sum(1 for i in parents if i >= 0 and lens[i] % page)
    assert mm.get_device_error() == (mm.DEV_NO_PAGES if asked > len(pairs) else 0)
    assert t.tolist() == want_rows and n.tolist() == want_lens and r.tolist() == refs
    for c, was in zip(caches, before):
        for src, dst in pairs:
            was[dst] = was[src]
        assert torch.equal(P.raw(c), P.raw(was))


def test_fork_into_rows_of_the_same_table(mm):
    """A batch whose free slots are filled: `out` and `out_lens` are rows of the table and lengths."""
    page, refs = 16, [1] * 6 + [0] * 6
    table = gpu([[0, 1, 2, -1], [3, 4, -1, -1], [5, 5, 5, 5], [7, 7, 7, 7]])
    lens, r = gpu([40, 32, 0, 0]), gpu(refs)
    cache = torch.arange(12, device="cuda", dtype=torch.float32)[:, None].repeat(1, 40)
    ws = mm.new_pages_workspace(12, 2)
    ws.fill_(0xee)
    mm.fork_pages(r, table[:2], lens[:2], gpu([0, 1]), (cache,), page_size=page, out=table[2:],
                  out_lens=lens[2:], workspace=ws)
    assert table.tolist() == [[0, 1, 2, -1], [3, 4, -1, -1], [0, 1, 6, -1], [3, 4, -1, -1]]
    assert lens.tolist() == [40, 32, 40, 32]
    assert r.tolist() == [2, 2, 1, 2, 2, 1, 1, 0, 0, 0, 0, 0]
    assert cache[:, 0].tolist() == [0, 1, 2, 3, 4, 5, 2, 7, 8, 9, 10, 11]
    assert mm.get_device_error() == 0


def test_fork_reports(mm):
    r, lens = gpu([1, 1, 1, 0, 0, 0]), gpu([20, 20, 99])
    table = gpu([[0, 9], [-1, 1], [2, 2]])
    t, n = mm.fork_pages(r, table, lens, gpu([3]), [], page_size=16)
    assert mm.get_device_error() == mm.DEV_BAD_ROWS and t.tolist() == [[-1, -1]] and n.tolist() == [0]
    t, n = mm.fork_pages(r, table, lens, gpu([0, 1]), [], page_size=16)
    assert mm.get_device_error() == mm.DEV_BAD_PAGE
    assert t.tolist() == [[0, -1], [-1, 3]] and n.tolist() == [20, 20]
    assert r.tolist() == [2, 1, 1, 1, 0, 0]
    t, n = mm.fork_pages(r, table, lens, gpu([2]), [], page_size=16)
    assert mm.get_device_error() == mm.DEV_SEQ_TOO_LONG
    assert t.tolist() == [[2, 2]] and n.tolist() == [32] and r.tolist() == [2, 1, 3, 1, 0, 0]
    # nothing to fork; a table without columns
    mm.fork_pages(r, table, lens, gpu([]), [], page_size=16)
    t, n = mm.fork_pages(r, table[:, :0], gpu([0, 0, 0]), gpu([0]), [], page_size=16)
    assert tuple(t.shape) == (1, 0) and n.tolist() == [0] and mm.get_device_error() == 0


@pytest.mark.parametrize("pages", [1, 31, 300, 5000, 70001])
@pytest.mark.parametrize("live", [0.0, 0.1, 0.5, 0.98, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(mm, pages, live, in_place):
    refs, g = pool(pages, live, pages + int(10 * live))
    held = [p for p, n in enumerate(refs) if n]
    table = torch.randint(-1, pages, (5, 40), generator=g).tolist()   # free pages and none among them
    table.append(([held[k % len(held)] for k in range(40)] if held else [-1] * 40))
    caches = make_caches(pages, g) if pages <= 5000 else [torch.randn((pages, 8), generator=g).cuda()]
    before = [c.clone() for c in caches]
    r, t = gpu(refs), gpu(table)
    wide = torch.full((6, 50), 5, dtype=torch.int32, device="cuda")
    wide[:, :40] = t
    c = mm.compact_pages(r, wide[:, :40], caches, in_place=in_place)
    wr, wt, wl, pairs = P.compact_ref(refs, table)
    assert mm.get_device_error() == 0
    assert c.refs.tolist() == wr and c.page_table.tolist() == wt and c.live.tolist() == [wl]
    if in_place:
        assert c.refs is r and r.tolist() == wr and (wide[:, 40:] == 5).all()
    else:
        assert r.tolist() == refs and wide[:, :40].tolist() == table
    for got, was in zip(caches, before):
        src, dst = ([p[k] for p in pairs] for k in (0, 1))
        if pairs:
            was[dst] = was[src]
        assert torch.equal(P.raw(got), P.raw(was))
    # once more: nothing moves
    again = mm.compact_pages(c.refs, c.page_table, caches)
    assert again.refs.tolist() == wr and again.page_table.tolist() == wt
    assert all(torch.equal(P.raw(got), P.raw(was)) for got, was in zip(caches, before))
    mm.get_device_error()


def test_a_pool_of_two_million_pages(mm):
    """More pages than a warp of the scans has in one round."""
    pages = 2 ** 21 + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    refs = (torch.rand(pages, generator=g, device="cuda") < 0.5).to(torch.int32)
    cache = torch.arange(pages, device="cuda", dtype=torch.int32)[:, None].repeat(1, 4)
    live = refs > 0
    n = int(live.sum())
    page = torch.arange(pages, device="cuda")
    to, frm = (~live & (page < n)).nonzero()[:, 0], (live & (page >= n)).nonzero()[:, 0]
    table = page[live].to(torch.int32)[None]
    c = mm.compact_pages(refs, table, [cache])
    assert int(c.live) == n and bool((c.refs == (page < n)).all())
    assert torch.equal(cache[to, 2], frm.to(torch.int32))
    assert torch.equal(cache[c.page_table[0].long(), 0], table[0])
    # every free page is dealt out in order
    lens = torch.tensor([pages - n], dtype=torch.int32, device="cuda")
    t = torch.full((1, pages - n), -1, dtype=torch.int32, device="cuda")
    mm.allocate_pages(c.refs, t, lens, query_len=pages - n, page_size=1)
    assert torch.equal(t[0].long(), page[n:]) and bool((c.refs == 1).all())
    assert mm.get_device_error() == 0


def test_copy_pages(mm):
    g = torch.Generator().manual_seed(2)
    caches = make_caches(50, g)
    before = [c.clone() for c in caches]
    src, dst = [1, 4, -1, 7, 49, 3, 60, 5], [2, 0, 9, -1, 8, 3, 10, 50]
    mm.copy_pages(caches, gpu(src), gpu(dst))
    assert mm.get_device_error() == mm.DEV_BAD_PAGE
    for c, was in zip(caches, before):
        for a, b in ((1, 2), (4, 0), (49, 8)):
            was[b] = was[a]
        assert torch.equal(P.raw(c), P.raw(was))
    mm.copy_pages(tuple(caches), gpu([]), gpu([]))
    many = [torch.full((4, 5), k, device="cuda", dtype=torch.int16) for k in range(64)]
    for m in many:
        m[1] += 1000
    mm.copy_pages(many, gpu([1]), gpu([3]))
    assert all(m[:, 0].tolist() == [k, k + 1000, k, k + 1000] for k, m in enumerate(many))
    assert mm.get_device_error() == 0


def test_pages_on_streams_and_graphs(mm):
    """Allocation, forks, release and compaction captured once and replayed over fresh state, by two
    graphs that share a workspace."""
    page, pages, width = 16, 600, 12
    refs, g = pool(pages, 0.5, 3)
    lens = [100, 37, 0, 192]
    table = table_of(4, width, refs, g, lens, page)
    parents = [0, 0, 3, 1, -1, 0]
    caches = make_caches(pages, g)
    saved = [c.clone() for c in caches]
    r, t, n = gpu(refs), gpu(table), gpu(lens)
    out, out_lens = torch.empty((6, width), dtype=torch.int32, device="cuda"), gpu([0] * 6)
    r2, t2 = gpu(refs), gpu(table)
    ws = mm.new_pages_workspace(pages, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]

    def fork():
        mm.fork_pages(r, t, n, par, caches, page_size=page, out=out, out_lens=out_lens, workspace=ws)
        mm.release_pages(r, t, seq_lens=n, page_size=page)

    def compact():
        return mm.compact_pages(r2, t2, caches[:3], in_place=True, workspace=ws)

    par = gpu(parents)
    wr = list(refs)
    rows, wl, pairs = P.fork_ref(wr, table, lens, parents, page)
    for row, k in zip(table, lens):
        for p in row[:-(-k // page)]:
            wr[p] = max(0, wr[p] - 1)
    cr, ct, _, cpairs = P.compact_ref(refs, table)
    with torch.cuda.stream(side):
        for graph, f in zip(graphs, (fork, compact)):
            with torch.cuda.graph(graph, stream=side):
                f()
        for _ in range(3):
            for c, s in zip(caches, saved):
                c.copy_(s)
            for x, y in ((r, refs), (t, table), (r2, refs), (t2, table)):
                x.copy_(gpu(y))
            want = [s.clone() for s in saved]
            graphs[0].replay()
            graphs[1].replay()
            side.synchronize()
            for k, w in enumerate(want):
                for a, b in pairs:
                    w[b] = w[a]
                if k < 3 and cpairs:
                    w[[p[1] for p in cpairs]] = w[[p[0] for p in cpairs]]
            assert out.tolist() == rows and out_lens.tolist() == wl and r.tolist() == wr
            assert r2.tolist() == cr and t2.tolist() == ct
            assert all(torch.equal(P.raw(c), P.raw(w)) for c, w in zip(caches, want))
    torch.cuda.synchronize()
    mm.get_device_error()
    t3, _ = mm.fork_pages(gpu(refs), t, n, par, [], page_size=page, stream=side)
    side.synchronize()
    assert t3.tolist() == rows
    mm.get_device_error()


def test_binding_refuses_caches_and_outputs(mm):
    r, t, n, p = gpu([1, 0, 0]), gpu([[0, -1]]), gpu([5]), gpu([0])
    ok = torch.zeros((3, 4, 8), device="cuda")
    wide = torch.zeros((6, 4, 8), device="cuda")
    for bad in (ok.cpu(), ok[:2], ok[:, ::2], ok[:, :, ::2], ok[:, :1, :].expand(3, 4, 8),
                wide.view(3, 2, 4, 8)[:, 0].transpose(0, 1)[:3], torch.zeros((), device="cuda"),
                torch.zeros((3, 0), device="cuda"), ok[:1].expand(3, 4, 8)):
        with pytest.raises(ValueError):
            mm.fork_pages(r, t, n, p, [ok, bad], page_size=16)
        with pytest.raises(ValueError):
            mm.compact_pages(r, t, [ok, bad])
    with pytest.raises(TypeError):
        mm.copy_pages([ok, 3], p, p)
    with pytest.raises(ValueError):
        mm.copy_pages(ok, p, p)
    with pytest.raises(ValueError):
        mm.copy_pages([ok] * 65, p, p)
    with pytest.raises(ValueError):
        mm.copy_pages([], p, p)
    for kw in (dict(out=gpu([[0, 0, 0]])), dict(out=t.long()), dict(out_lens=gpu([0, 0])),
               dict(out=t.cpu()), dict(workspace=torch.zeros(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            mm.fork_pages(r, t, n, p, [ok], page_size=16, **kw)
    with pytest.raises(mm.Mm3idxError):
        mm.fork_pages(r, t, n, p, [ok], page_size=16, workspace=torch.zeros(64, dtype=torch.uint8,
                                                                            device="cuda"))
    with pytest.raises(mm.Mm3idxError):
        mm.fork_pages(r, t, n, p, [ok], page_size=0)
    assert r.tolist() == [1, 0, 0] and mm.get_device_error() == 0
    # what a page may be: strides between pages, dimensions in any order
    for good in (ok.transpose(1, 2), wide[::2], wide.view(3, 2, 4, 8)[:, 1]):
        mm.copy_pages([good], gpu([0]), gpu([2]))
    assert mm.get_device_error() == 0
