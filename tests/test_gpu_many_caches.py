"""Forks and compactions of pools with more caches than a call takes, the way that
their documentation names."""

import pytest
import torch

import pages_ref as P
from test_gpu_pages import gpu, pool, table_of

pytestmark = pytest.mark.gpu
CACHES = 150


@pytest.fixture(scope="module")
def mm(cuda_device):
    import sparse_attention_block_paged_gb300 as m
    m.get_device_error()
    return m


def make(pages, g):
    shapes = [(16, 64), (7,), (5, 4)]
    return [torch.randint(0, 255, (pages,) + shapes[k % 3], generator=g, dtype=torch.uint8).cuda()
            for k in range(CACHES)]


@pytest.mark.parametrize("pages,reqs,forks,page,width", [(80, 4, 9, 16, 8), (12, 3, 20, 32, 3),
                                                         (500, 9, 64, 128, 20)])
def test_a_fork(mm, pages, reqs, forks, page, width):
    refs, g = pool(pages, 0.6, pages)
    lens = torch.randint(0, width * page + 1, (reqs,), generator=g).tolist()
    lens[0], lens[-1] = width * page, 3 * page                      # no page to copy
    table = table_of(reqs, width, refs, g, lens, page)
    parents = torch.randint(-1, reqs, (forks,), generator=g).tolist()
    caches = make(pages, g)
    before = [c.clone() for c in caches]
    r, t, p = gpu(refs), gpu(table), gpu(parents)
    out, n = mm.fork_pages(r, t, gpu(lens), p, caches[:64], page_size=page)
    last = (n // page).clamp(max=width - 1).long()[:, None]
    part = n % page > 0
    src = torch.where(part, t[p.clamp(min=0).long()].gather(1, last)[:, 0], -1)
    dst = torch.where(part, out.gather(1, last)[:, 0], -1)
    for k in range(64, CACHES, 64):
        mm.copy_pages(caches[k:k + 64], src, dst)
    rows, want_lens, pairs = P.fork_ref(refs, table, lens, parents, page)
    assert out.tolist() == rows and n.tolist() == want_lens and r.tolist() == refs
    assert pairs
    for c, was in zip(caches, before):
        for a, b in pairs:
            was[b] = was[a]
        assert torch.equal(c, was)
    short = sum(1 for i in parents if i >= 0 and lens[i] % page) > len(pairs)
    assert mm.get_device_error() == (mm.DEV_NO_PAGES if short else 0)


@pytest.mark.parametrize("pages,live", [(90, 0.5), (700, 0.3), (9000, 0.6)])
def test_a_compaction(mm, pages, live):
    refs, g = pool(pages, live, pages)
    table = torch.randint(-1, pages, (5, 30), generator=g).tolist()
    caches = make(pages, g)
    before = [c.clone() for c in caches]
    r, t = gpu(refs), gpu(table)
    for k in range(0, CACHES, 64):
        c = mm.compact_pages(r, t, caches[k:k + 64], in_place=k + 64 >= CACHES)
    wr, wt, wl, pairs = P.compact_ref(refs, table)
    assert c.refs is r and r.tolist() == wr and t.tolist() == wt and c.live.tolist() == [wl]
    src, dst = ([p[k] for p in pairs] for k in (0, 1))
    for got, was in zip(caches, before):
        was[dst] = was[src]
        assert torch.equal(got, was)
    assert mm.get_device_error() == 0
