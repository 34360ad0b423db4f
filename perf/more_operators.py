"""The life of a paged key-value cache, as measured work.

Four operators that a serving loop runs around its decode steps:

* ``append``: new tokens' keys and values written into their requests' pages,
  in 16 bits or in e4m3 with one power-of-two scale a page and head, which
  grows (the page's older tokens then change with it) when new tokens need it.
* ``attend``: attention of a few new tokens a request over e4m3 pages with a
  scale for each page and head.
* ``fork``: the pages of finished requests given back, then requests continued
  by several others: full pages shared by counting references, the last one,
  partly filled, copied in every cache.
* ``compact``: a fragmented pool's live pages moved to its front.

With ``own`` false they are computed in elementary torch operations, with
``own`` true by the framework's calls.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0


def _cdiv(a, b):
    return (a + b - 1) // b


# --------------------------------------------------------------------- cases

def _attend(**kw):
    c = dict(op="attend", dtype="bf16", reqs=1, ql=1, qh=16, kvh=2, d=128, page=128, lo=1, hi=1024,
             order="nhd", weights=False, empty=False)
    c.update(kw)
    return c


def _append(**kw):
    c = dict(op="append", dtype="bf16", kv="e4m3", reqs=1, ql=1, kvh=2, d=128, page=128, lo=1,
             hi=1024, order="nhd", ragged=False, empty=False)
    c.update(kw)
    return c


def _fork(**kw):
    c = dict(op="fork", kv="bf16", reqs=1, children=4, kvh=2, d=128, page=128, lo=1, hi=1024,
             layers=1, free=0.25, scales=False)
    c.update(kw)
    return c


def _compact(**kw):
    c = dict(op="compact", kv="bf16", reqs=4, pages=256, live=0.5, kvh=2, d=128, page=128, layers=1,
             scales=False)
    c.update(kw)
    return c


def listed():
    return [
        # two short requests: the smallest decode step, where latency counts
        _attend(name="attend tiny", reqs=2, lo=300, hi=700),
        # the spec-decode batch: three drafted tokens and the last one, 4K-32K tokens
        _attend(name="attend spec-decode", reqs=64, ql=4, lo=4096, hi=32768),
        # a batch of long contexts
        _attend(name="attend long", reqs=16, lo=32768, hi=131072, qh=32, kvh=4, page=64),
        # one request alone with a long context, small heads and small pages
        _attend(name="attend one long", dtype="fp16", reqs=1, lo=131072, hi=131072, qh=32, kvh=8,
                d=64, page=16),
        # one decode step's tokens
        _append(name="append tokens", reqs=64, lo=4096, hi=32768),
        # a step of drafted tokens, small heads and pages; some slots of the batch are empty
        _append(name="append drafts", dtype="fp16", reqs=256, ql=4, kvh=8, d=64, page=16, lo=100,
                hi=2000, order="hnd", empty=True),
        # whole prompts
        _append(name="append prompts", reqs=4, ql=8192, kvh=8, page=64, lo=8192, hi=8192),
        # pieces of prompts of many lengths behind what is there, in 16 bits
        _append(name="append ragged", kv="bf16", reqs=32, ql=2048, kvh=4, page=32, lo=1, hi=16384,
                ragged=True),
        # one prompt continued four ways, small pages
        _fork(name="fork one", reqs=1, children=4, lo=500, hi=1000, page=16, scales=True),
        # several prompts continued eight ways each, pages of four layers
        _fork(name="fork samples", reqs=8, children=64, lo=1024, hi=8192, layers=4),
        # a small pool
        _compact(name="compact small", reqs=8, pages=512, page=16, scales=True),
        # half of a pool of two million tokens is free
        _compact(name="compact pool", reqs=128, pages=16384),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "append", "append", "fork", "compact"])
    d, page, kvh = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if op == "attend":
        ql = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 6, 7, 8, 12, 16) if g * ql <= 64])
        hi = _log_int(rng, 16, 131072)
        lo = max(ql, rng.randint(1, hi))
        hi = max(lo, hi)
        most = min(256, max(1, int(1.0e9 / (2 * kvh * d * hi))))
        return _attend(dtype=dtype, reqs=_log_int(rng, 1, most), ql=ql, qh=group * kvh, kvh=kvh,
                       d=d, page=page, lo=lo, hi=hi, order=rng.choice(["nhd", "hnd"]),
                       weights=rng.random() < 0.3, empty=rng.random() < 0.3)
    if op == "append":
        ragged = rng.random() < 0.4
        kv = rng.choice(["e4m3", "e4m3", dtype])
        ql = rng.choice([1, 1, 2, 3, 4, 8, _log_int(rng, 9, 8192), _log_int(rng, 9, 8192)])
        lo = max(1 if ragged else ql, _log_int(rng, 1, 8192))
        hi = max(lo, ql, rng.randint(lo, 2 * lo + 64))
        # rows of the batch, and tokens of its pool
        most = min(256, max(1, int(1.3e8 / (kvh * d * 4 * ql))), max(1, int(2.0e9 / (hi * kvh * d))))
        return _append(dtype=dtype, kv=kv, reqs=_log_int(rng, 1, most), ql=ql, kvh=kvh, d=d,
                       page=page, lo=lo, hi=hi, order=rng.choice(["nhd", "hnd"]), ragged=ragged,
                       empty=rng.random() < 0.3)
    kv, layers, scales = rng.choice(["bf16", "fp16", "e4m3"]), rng.choice([1, 2, 4]), rng.random() < 0.5
    size = 2 * page * kvh * d * SIZE[kv] * layers                       # a page in all caches
    if op == "fork":
        reqs = _log_int(rng, 1, 16)
        hi = _log_int(rng, 1, 16384)
        lo = rng.randint(1, hi)
        per = _cdiv(hi, page)
        most = max(1, min(128, int(2.0e9 / size) // (2 * per) - reqs))
        return _fork(kv=kv, reqs=reqs, children=_log_int(rng, 1, most), kvh=kvh, d=d, page=page,
                     lo=lo, hi=hi, layers=layers, free=rng.choice([0.0, 0.1, 0.5]), scales=scales)
    pages = _log_int(rng, 8, max(8, min(65536, int(2.0e9 / size))))
    return _compact(kv=kv, reqs=rng.randint(1, min(pages, 64)), pages=pages,
                    live=rng.choice([0.05, 0.3, 0.5, 0.7, 0.95, 1.0]), kvh=kvh, d=d, page=page,
                    layers=layers, scales=scales)


# -------------------------------------------------------------------- inputs

def _lengths(case, gen):
    n, lo, hi = case["reqs"], case["lo"], case["hi"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    s = (lo + torch.floor(u * (hi - lo + 1))).clamp(lo, hi).to(torch.int32)
    if case.get("empty"):
        s[2::5] = 0          # slots of the batch that hold no request
    return s


def _pages_of(lens, page, width, spare, gen):
    """(table [reqs, width], -1 behind the pages, number of pages): pages dealt at random from a pool
    that has all rows' width and `spare` more."""
    need = torch.div(lens + page - 1, page, rounding_mode="floor")
    pool = lens.shape[0] * width + spare
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    start = torch.cumsum(need, 0) - need
    col = torch.arange(width, device="cuda")
    at = (start[:, None] + col).clamp(max=pool - 1)
    return torch.where(col < need[:, None], perm[at], -1).to(torch.int32).contiguous(), pool


def _values(pages, case, kv, gen, step=4096):
    """Random [pages, page, kvh, d] of type `kv`, in the case's order in memory."""
    shape = (case["page"], case["kvh"], case["d"])
    hnd = case.get("order") == "hnd"
    x = torch.empty((pages, shape[1], shape[0], shape[2]) if hnd else (pages,) + shape,
                    dtype=TYPES[kv], device="cuda")
    for i in range(0, pages, step):                       # a bounded amount of 32-bit values
        v = torch.randn(x[i:i + step].shape, generator=gen, device="cuda")
        x[i:i + step] = (v * 100.0 if kv == "e4m3" else v).clamp(-E4M3_MAX, E4M3_MAX).to(TYPES[kv])
    return x.transpose(1, 2) if hnd else x


def _scales(pages, kvh, gen, power):
    """One scale a page and head, about 1/100 (codes are about 100), some heads and pages far off."""
    s = torch.exp(0.7 * torch.randn(pages, kvh, generator=gen, device="cuda")) / 100.0
    return torch.exp2(torch.floor(torch.log2(s))) if power else s


def _prepare_attend(case, gen):
    lens = _lengths(case, gen)
    reqs, ql, kvh, d, page = (case[k] for k in ("reqs", "ql", "kvh", "d", "page"))
    most = max(case["hi"], ql)
    table, pool = _pages_of(lens, page, _cdiv(most, page), 1, gen)
    q = torch.randn(reqs * ql, case["qh"], d, generator=gen, device="cuda").to(TYPES[case["dtype"]])
    s = dict(case=case, q=q, k=_values(pool, case, "e4m3", gen), v=_values(pool, case, "e4m3", gen),
             ks=_scales(pool, kvh, gen, False), vs=_scales(pool, kvh, gen, False), table=table,
             seq=lens, max_seq_len=most, sm_scale=d ** -0.5, out=torch.empty_like(q), weights=None,
             workspace=None)
    if case["weights"]:
        s["weights"] = torch.empty(reqs * ql, _cdiv(most, 128), device="cuda")
    return s


def _prepare_append(case, gen):
    lens = _lengths(case, gen)
    reqs, ql, kvh, d, page = (case[k] for k in ("reqs", "ql", "kvh", "d", "page"))
    most = max(case["hi"], ql)
    table, pool = _pages_of(lens, page, _cdiv(most, page), 1, gen)
    cu = None
    if case["ragged"]:
        u = torch.rand(reqs, generator=gen, device="cuda")
        n = torch.minimum((u * (ql + 1)).to(torch.int32).clamp(max=ql), lens)
        cu = torch.zeros(reqs + 1, dtype=torch.int32, device="cuda")
        cu[1:] = torch.cumsum(n, 0)
        rows = int(cu[-1])
    else:
        rows = reqs * ql
    k, v = (torch.randn(rows, kvh, d, generator=gen, device="cuda") for _ in range(2))
    k = k * torch.exp(0.5 * torch.randn(1, kvh, d, generator=gen, device="cuda"))  # uneven channels
    s = dict(case=case, nk=k.to(TYPES[case["dtype"]]), nv=v.to(TYPES[case["dtype"]]),
             k=_values(pool, case, case["kv"], gen), v=_values(pool, case, case["kv"], gen),
             table=table, seq=lens, cu=cu, max_seq_len=most, ks=None, vs=None)
    if case["kv"] == "e4m3":
        s["ks"], s["vs"] = _scales(pool, kvh, gen, True), _scales(pool, kvh, gen, True)
    return s


def _caches(case, pages, gen):
    c = [_values(pages, case, case["kv"], gen) for _ in range(2 * case["layers"])]
    if case["scales"]:
        c += [_scales(pages, case["kvh"], gen, True) for _ in range(2 * case["layers"])]
    return c


def _prepare_fork(case, gen):
    n, page = case["children"], case["page"]
    lens = _lengths(case, gen)
    old = _lengths(dict(case, reqs=n), gen)               # what the children's rows held before
    both = torch.cat([lens, old])
    width = _cdiv(case["hi"], page)
    spare = n + int(case["free"] * width * (case["reqs"] + n))
    table, pool = _pages_of(both, page, width, spare, gen)
    refs = torch.zeros(pool, dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    parents = torch.randint(0, case["reqs"], (n,), generator=gen, device="cuda").to(torch.int32)
    return dict(case=case, refs=refs, table=table[:case["reqs"]].contiguous(), seq=lens,
                child=table[case["reqs"]:].contiguous(), child_lens=old.clone(), parents=parents,
                caches=_caches(case, pool, gen), workspace=None)


def _prepare_compact(case, gen):
    pages, reqs = case["pages"], case["reqs"]
    live = max(1, min(pages, int(round(case["live"] * pages))))
    width = _cdiv(live, reqs)
    perm = torch.randperm(pages, generator=gen, device="cuda")[:live].to(torch.int32)
    table = torch.full((reqs * width,), -1, dtype=torch.int32, device="cuda")
    table[:live] = perm
    table = table.view(width, reqs).T.contiguous()        # rows of nearly equal lengths
    if width > 1:
        table[1::3, 0] = table[0, 0]                      # a common beginning, counted
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    at = table.flatten()
    refs.index_add_(0, at.clamp(min=0).long(), (at >= 0).to(torch.int32))
    return dict(case=case, refs=refs, table=table, caches=_caches(case, pages, gen), workspace=None)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"attend": _prepare_attend, "append": _prepare_append, "fork": _prepare_fork,
         "compact": _prepare_compact}[case["op"]](case, gen)
    if own and case["op"] != "append":
        # the scratch that a serving loop makes once and hands to every step
        import sparse_attention_block_paged_gb300 as mm
        if case["op"] == "attend":
            s["workspace"] = mm.new_attention_workspace(
                case["qh"], case["kvh"], case["d"], case["reqs"], case["ql"], s["max_seq_len"],
                block_weights=case["weights"])
        else:
            s["workspace"] = mm.new_pages_workspace(s["refs"].shape[0], case.get("children", 0))
    return s


# ---------------------------------------------------------------- plain forms

def _plain_attend(s):
    q, seq, ql, size = s["q"], s["seq"], s["case"]["ql"], s["k"].shape[1]
    reqs, (_, qh, d), kvh = seq.shape[0], q.shape, s["k"].shape[2]
    tokens = max(1, int(seq.max()))
    t = torch.arange(tokens, device=q.device)
    there = t < seq[:, None]
    page = torch.where(there, s["table"][:, t // size], 0).long()
    slot = (t % size).expand_as(page)
    k = s["k"][page, slot].float() * s["ks"][page][..., None]
    k = torch.where(there[..., None, None], k, 0.0)
    x = q.float().view(reqs, ql, kvh, qh // kvh, d) * s["sm_scale"]
    x = torch.einsum("bjhgd,bthd->bhgjt", x, k)
    del k
    last = seq[:, None] - ql + torch.arange(ql, device=q.device)
    x = torch.where((t <= last[..., None])[:, None, None], x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = torch.exp(x - top)
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-38)
    v = s["v"][page, slot].float() * s["vs"][page][..., None]
    v = torch.where(there[..., None, None], v, 0.0)
    out = torch.einsum("bhgjt,bthd->bjhgd", x, v).reshape(reqs * ql, qh, d).to(q.dtype)
    if s["weights"] is None:
        return {"out": out}
    x = torch.nn.functional.pad(x.sum((1, 2)), (0, -tokens % 128))
    x = x.view(reqs * ql, -1, 128).sum(-1)
    return {"out": out,
            "weights": torch.nn.functional.pad(x, (0, _cdiv(s["max_seq_len"], 128) - x.shape[1]))}


def _positions(s):
    """(request, position) of every new token."""
    c, seq = s["case"], s["seq"]
    row = torch.arange(s["nk"].shape[0], device=seq.device)
    if s["cu"] is None:
        req = torch.div(row, c["ql"], rounding_mode="floor")
        return req, seq[req] - c["ql"] + row % c["ql"]
    req = torch.searchsorted(s["cu"], row, right=True) - 1
    return req, seq[req] - s["cu"][req + 1] + row


def _power(x):
    """The smallest power of two that brings x to 448 or less, in the scales' range."""
    m, e = torch.frexp(x.clamp(min=1e-37))                # x = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
    e = (e - 9 + (m > 0.875)).clamp(-60, 60).to(torch.int32)
    return ((e + 127) << 23).view(torch.float32)          # 2^e exactly


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _plain_append(s):
    size = s["k"].shape[1]
    req, pos = _positions(s)
    at = (pos >= 0).nonzero()[:, 0]
    req, pos = req[at], pos[at]
    page, slot = s["table"][req, torch.div(pos, size, rounding_mode="floor")].long(), (pos % size).long()
    if s["ks"] is None:
        s["k"][page, slot] = s["nk"][at]
        s["v"][page, slot] = s["nv"][at]
        return {"k": s["k"], "v": s["v"]}
    pool, kvh = s["ks"].shape
    first = torch.full((pool,), size, device=page.device).scatter_reduce_(0, page, slot, "amin")
    some = (first < size).nonzero()[:, 0]                 # the pages that get tokens
    first = first[some]
    older = torch.arange(size, device=page.device) < first[:, None]
    for new, cache, scales in ((s["nk"], s["k"], s["ks"]), (s["nv"], s["v"], s["vs"])):
        x = new[at].float()
        top = torch.zeros(pool, kvh, device=x.device).scatter_reduce_(
            0, page[:, None].expand(-1, kvh), x.abs().amax(-1), "amax")
        was, now = scales[some], _power(top[some])
        now = torch.where((first > 0)[:, None], torch.maximum(now, was), now)
        y = cache[some]
        z = _codes(y.float() * (was / now)[:, None, :, None])
        cache[some] = torch.where(older[..., None, None], z, y)
        scales[some] = now
        cache[page, slot] = _codes(x / scales[page][..., None])
    return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}


def _plain_fork(s):
    refs, size, n = s["refs"], s["case"]["page"], s["parents"].shape[0]
    old = s["child"].flatten()                            # the children's pages go back
    refs.index_add_(0, old.clamp(min=0).long(), -(old >= 0).to(torch.int32))
    parent = s["parents"].long()
    lens, rows = s["seq"][parent], s["table"][parent]
    full = torch.div(lens, size, rounding_mode="floor")
    part = lens % size > 0
    page = torch.arange(refs.shape[0], device=refs.device)
    free = torch.where(refs == 0, page, refs.shape[0]).sort().values     # the lowest first
    new = free[(torch.cumsum(part, 0) - 1).clamp(min=0)].to(torch.int32)
    col = torch.arange(rows.shape[1], device=refs.device)
    shared = torch.where(col < full[:, None], rows, -1)
    last = (col == full[:, None]) & part[:, None]
    child = torch.where(last, new[:, None], shared)
    src = torch.where(last, rows, 0).sum(1)
    flat = shared.flatten()
    refs.index_add_(0, flat.clamp(min=0).long(), (flat >= 0).to(torch.int32))
    at = part.nonzero()[:, 0]
    src, new = src[at].long(), new[at].long()
    refs[new] = 1
    for c in s["caches"]:
        c[new] = c[src]
    s["child"].copy_(child)
    s["child_lens"].copy_(lens)
    return {"refs": refs, "table": s["child"], "lens": s["child_lens"], "caches": s["caches"]}


def _plain_compact(s):
    refs = s["refs"]
    page = torch.arange(refs.shape[0], device=refs.device)
    live = refs > 0
    count = live.sum()
    to, frm = (~live & (page < count)).nonzero()[:, 0], (live & (page >= count)).nonzero()[:, 0]
    new, moved = refs.clone(), page.to(torch.int32)
    new[to] = refs[frm]
    new[frm] = 0
    moved[frm] = to.to(torch.int32)
    table = torch.where(s["table"] >= 0, moved[s["table"].clamp(min=0).long()], s["table"])
    for c in s["caches"]:
        c[to] = c[frm]
    return {"refs": new, "table": table, "live": count.to(torch.int32).view(1), "caches": s["caches"]}


# ------------------------------------------------------------------------ run

def run(s):
    c = s["case"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork,
                "compact": _plain_compact}[c["op"]](s)
    import sparse_attention_block_paged_gb300 as mm
    if c["op"] == "attend":
        out = mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["seq"], query_len=c["ql"],
                                 max_seq_len=s["max_seq_len"], sm_scale=s["sm_scale"],
                                 k_scales=s["ks"], v_scales=s["vs"], out=s["out"],
                                 block_weights=s["weights"], workspace=s["workspace"])
        return {"out": out} if s["weights"] is None else {"out": out, "weights": s["weights"]}
    if c["op"] == "append":
        mm.append_kv(s["nk"], s["nv"], s["k"], s["v"], s["table"], s["seq"], query_len=c["ql"],
                     max_seq_len=s["max_seq_len"], k_scales=s["ks"], v_scales=s["vs"],
                     cu_seqlens_q=s["cu"])
        if s["ks"] is None:
            return {"k": s["k"], "v": s["v"]}
        return {"k": s["k"], "v": s["v"], "ks": s["ks"], "vs": s["vs"]}
    if c["op"] == "fork":
        mm.release_pages(s["refs"], s["child"])
        mm.fork_pages(s["refs"], s["table"], s["seq"], s["parents"], s["caches"],
                      page_size=c["page"], out=s["child"], out_lens=s["child_lens"],
                      workspace=s["workspace"])
        return {"refs": s["refs"], "table": s["child"], "lens": s["child_lens"],
                "caches": s["caches"]}
    r = mm.compact_pages(s["refs"], s["table"], s["caches"], workspace=s["workspace"])
    return {"refs": r.refs, "table": r.page_table, "live": r.live, "caches": s["caches"]}


# ----------------------------------------------------------------------- work

def work(case):
    kvh, d, page = case["kvh"], case["d"], case["page"]
    if case["op"] in ("attend", "append"):
        some = 0.8 if case["empty"] else 1.0              # about one slot in five is empty
        reqs, ql, mean = case["reqs"], case["ql"], (case["lo"] + case["hi"]) / 2 * some
    if case["op"] == "attend":
        rows, qh = reqs * ql, case["qh"]
        size = reqs * mean * kvh * (2 * d + 8 / page) + rows * qh * d * 2 * SIZE[case["dtype"]]
        if case["weights"]:
            size += 4 * rows * _cdiv(case["hi"], 128)
        return {"bytes": size, "flops": 4.0 * d * qh * rows * mean}
    if case["op"] == "append":
        rows = reqs * (min(ql, mean) / 2 if case["ragged"] else ql * some)
        size = rows * kvh * d * 2 * (SIZE[case["dtype"]] + SIZE[case["kv"]])
        if case["kv"] == "e4m3":
            size += 16 * kvh * reqs * some * (1 + (rows / reqs - 1) / page)
        return {"bytes": size, "flops": rows * kvh * d * 4}
    one = 2 * case["layers"] * kvh * (page * d * SIZE[case["kv"]] + (4 if case["scales"] else 0))
    if case["op"] == "fork":
        n, per = case["children"], (case["lo"] + case["hi"]) / 2 / page
        copied = n * (1 - 1 / page)
        pool = (case["reqs"] + n) * _cdiv(case["hi"], page) * (1 + case["free"]) + n
        return {"bytes": 2 * copied * one + n * per * (3 * 4 + 2 * 8) + 4 * pool, "flops": 0}
    pages, live = case["pages"], case["live"]
    moved = pages * live * (1 - live)
    return {"bytes": 2 * moved * one + 8 * pages + 8 * pages * live, "flops": 0}


# ---------------------------------------------------------------------- exact

def _exact_attend(s):
    q, seq, ql = s["q"], s["seq"].tolist(), s["case"]["ql"]
    rows, qh, d = q.shape
    size, kvh = s["k"].shape[1], s["k"].shape[2]
    group = qh // kvh
    out = torch.zeros(rows, qh, d, dtype=torch.float64, device=q.device)
    mass = torch.zeros(rows, _cdiv(s["max_seq_len"], 128), dtype=torch.float64, device=q.device)
    for i, n in enumerate(seq):
        if n <= 0:
            continue
        pages = s["table"][i, :_cdiv(n, size)].long()
        k = (s["k"][pages].double() * s["ks"][pages].double()[:, None, :, None]).flatten(0, 1)[:n]
        v = (s["v"][pages].double() * s["vs"][pages].double()[:, None, :, None]).flatten(0, 1)[:n]
        for j in range(ql):
            m = n - ql + j + 1
            if m <= 0:
                continue
            b = torch.arange(m, device=q.device) // 128
            for h in range(kvh):
                x = q[i * ql + j, h * group:(h + 1) * group].double()
                e = torch.softmax((x @ k[:m, h].T) * s["sm_scale"], -1)
                out[i * ql + j, h * group:(h + 1) * group] = e @ v[:m, h]
                mass[i * ql + j].index_add_(0, b, e.sum(0))
    return {"out": out} if s["weights"] is None else {"out": out, "weights": mass}


def _round_e4m3(x):
    """The nearest e4m3 value, ties to even, 448 at most: 4 significant bits, steps of 2^-9 below
    2^-6."""
    e = torch.frexp(x).exponent.double() - 4
    step = torch.exp2(torch.clamp(e, min=-9.0))
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _least_power(top):
    """The least 2^n, n in -60..60, with top / 2^n <= 448."""
    n = -60
    while n < 60 and math.ldexp(448.0, n) < top:
        n += 1
    return math.ldexp(1.0, n)


def _exact_append(s):
    # page by page on 64-bit copies; a scale is the least 2^n with max / 2^n <= 448
    case, size, seq = s["case"], s["case"]["page"], s["seq"].tolist()
    cu = s["cu"].tolist() if s["cu"] is not None else [i * case["ql"] for i in range(len(seq) + 1)]
    table, kvh = s["table"].cpu(), case["kvh"]
    if sum(_cdiv(b - a, size) + 1 for a, b in zip(cu, cu[1:])) > 6000:
        return None
    out = {}
    for name, scale, new in (("k", "ks", "nk"), ("v", "vs", "nv")):
        cache = s[name].double()
        scales = None if s[scale] is None else s[scale].double()
        for i, n in enumerate(seq):
            t = max(0, n - (cu[i + 1] - cu[i]))
            while t < n:
                end = min(n, (t // size + 1) * size)
                p, a, b = int(table[i, t // size]), t % size, (end - 1) % size + 1
                row = cu[i + 1] - n + t
                x = s[new][row:row + end - t].double()
                if scales is None:
                    cache[p, a:b] = x
                else:
                    now = torch.tensor([_least_power(float(m)) for m in x.abs().amax((0, 2)).cpu()],
                                       dtype=torch.float64, device=x.device)
                    if a > 0:
                        now = torch.maximum(now, scales[p])
                        cache[p, :a] = _round_e4m3(cache[p, :a] * (scales[p] / now)[:, None])
                    scales[p] = now
                    cache[p, a:b] = _round_e4m3(x / now[:, None])
                t = end
        out[name] = cache
        if scales is not None:
            out[scale] = scales
    return out


def _exact_fork(s):
    # whole numbers are compared as they are; every page is a copy of one
    size, refs, new = s["case"]["page"], s["refs"].tolist(), []
    for p in s["child"].flatten().tolist():
        if p >= 0:
            refs[p] -= 1
    free = [p for p in range(len(refs)) if refs[p] == 0]
    lens, table = s["seq"].tolist(), s["table"].cpu()
    for i in s["parents"].tolist():
        if lens[i] % size:
            new.append((free.pop(0), int(table[i, lens[i] // size])))
    for c in s["caches"]:
        for dst, src in new:
            c[dst].copy_(c[src])
    return {"refs": None, "table": None, "lens": None, "caches": s["caches"]}


def _exact_compact(s):
    live = s["refs"].cpu().numpy() > 0
    n = int(live.sum())
    to = [p for p in range(n) if not live[p]]
    frm = [p for p in range(n, len(live)) if live[p]]
    for c in s["caches"]:
        for dst, src in zip(to, frm):
            c[dst].copy_(c[src])
    return {"refs": None, "table": None, "live": None, "caches": s["caches"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "fork": _exact_fork,
            "compact": _exact_compact}[case["op"]](s)
