"""The serving operators next to the index selection, as measured work.

Three operators of one decode step over a paged cache:

* ``attend``: attention of a few new tokens a request over paged keys and
  values, either over all of a request's tokens or over the pages of its
  selected 128-token blocks; optionally with the attention weight that each
  block took.
* ``evict``: the blocks' accumulated weights brought up to date, then the
  lightest blocks of a request taken out of its block table.
* ``verify``: drafted tokens accepted or rejected against the target's
  probabilities from given random numbers.

With ``own`` false they are computed in elementary torch operations, with
``own`` true by the framework's calls.
"""

import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def _cdiv(a, b):
    return (a + b - 1) // b


# --------------------------------------------------------------------- cases

def _attend(**kw):
    c = dict(op="attend", dtype="bf16", kv="bf16", reqs=1, ql=1, qh=16, kvh=2, d=128, page=128,
             lo=1, hi=1024, log=False, topk=0, weights=False, order="nhd", empty=False)
    c.update(kw)
    return c


def listed():
    return [
        # two short requests: the smallest decode step, where latency counts
        _attend(name="attend tiny", reqs=2, lo=300, hi=700, qh=16, kvh=2),
        # the spec-decode batch: three drafted tokens and the last one, 4K-32K tokens
        _attend(name="attend spec-decode", reqs=64, ql=4, lo=4096, hi=32768, qh=16, kvh=2),
        # the spec-decode batch's rows over their 16 selected blocks, two pages a block, keys and
        # values of a block next to each other in one pool
        _attend(name="attend selected", reqs=64, ql=4, lo=4096, hi=32768, qh=64, kvh=4, page=64,
                topk=16, order="pair"),
        # a batch of long contexts with an 8-bit cache
        _attend(name="attend long e4m3", kv="e4m3", reqs=16, lo=32768, hi=131072, qh=32, kvh=4,
                page=64),
        # the high-batch lengths (log-uniform), half precision, with the blocks' weights
        _attend(name="attend weights", dtype="fp16", kv="fp16", reqs=128, lo=1024, hi=65536,
                log=True, qh=8, kvh=1, weights=True, page=32, order="hnd"),
        # one request alone with a long context, small heads and small pages
        _attend(name="attend one long", reqs=1, lo=131072, hi=131072, qh=32, kvh=8, d=64, page=16),
        # one step's weights of the selected blocks, and eviction to half of a 32K context
        dict(name="evict selected", op="evict", reqs=64, ql=4, lo=4096, hi=32768, topk=16,
             budget=128, init=1, local=2, decay=1.0, table=False),
        # dense weights of contexts of up to a million tokens, with a second table
        dict(name="evict long", op="evict", reqs=128, ql=1, lo=131072, hi=1048576, topk=0,
             budget=1024, init=4, local=8, decay=0.99, table=True),
        # a few requests and a small vocabulary
        dict(name="verify tiny", op="verify", reqs=4, k=3, vocab=32000, dtype="fp32", drafts=True),
        # the spec-decode batch
        dict(name="verify batch", op="verify", reqs=64, k=3, vocab=200000, dtype="fp32",
             drafts=True),
        # a large batch with long drafts
        dict(name="verify large", op="verify", reqs=256, k=7, vocab=131072, dtype="fp32",
             drafts=True),
        # drafts looked up in the prompt (no draft probabilities), odd vocabulary
        dict(name="verify lookup", op="verify", reqs=32, k=5, vocab=50257, dtype="bf16",
             drafts=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "evict", "verify", "verify"])
    if op == "attend":
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        kv = rng.choice([dtype, dtype, "e4m3"])
        ql = rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 6, 7, 8, 12, 16) if g * ql <= 64])
        kvh = rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 128, 128])
        page = rng.choice([16, 32, 64, 128])
        topk = rng.choice([0, 0, 0, 4, 16, 32])
        hi = _log_int(rng, 16, 131072)
        lo = max(ql, rng.randint(1, hi))
        hi = max(lo, hi)
        per = 2 * kvh * d * SIZE[kv] * (ql if topk else 1)
        # all requests at the longest length stay below the largest listed case
        most = min(256, max(1, int(1.0e9 / (per * hi))))
        reqs = _log_int(rng, 1, most)
        return _attend(dtype=dtype, kv=kv, reqs=reqs, ql=ql, qh=group * kvh, kvh=kvh, d=d,
                       page=page, lo=lo, hi=hi, log=False, topk=topk,
                       weights=rng.random() < 0.3, order=rng.choice(["nhd", "hnd", "pair"]),
                       empty=rng.random() < 0.3)
    if op == "evict":
        hi = _log_int(rng, 128, 1048576)
        lo = rng.randint(1, hi)
        n = _cdiv(hi, BLOCK)
        init, local = rng.randint(0, 4), rng.randint(1, 8)
        return dict(op="evict", reqs=_log_int(rng, 1, 128), ql=rng.choice([1, 1, 2, 4]), lo=lo,
                    hi=hi, topk=rng.choice([0, 4, 16, 32]),
                    budget=max(init + local, rng.randint(1, n)), init=init, local=local,
                    decay=rng.choice([1.0, 1.0, 0.9, 0.99]), table=rng.random() < 0.5)
    vocab = _log_int(rng, 100, 200000)
    return dict(op="verify", reqs=_log_int(rng, 1, 64), k=rng.randint(1, 7), vocab=vocab,
                dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), drafts=rng.random() < 0.7)


# -------------------------------------------------------------------- inputs

def _lengths(case, gen):
    n, lo, hi = case["reqs"], case["lo"], case["hi"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    if case.get("log"):
        s = torch.exp(math.log(lo) + u * (math.log(hi) - math.log(lo))).round()
    else:
        s = lo + torch.floor(u * (hi - lo + 1))
    s = s.clamp(lo, hi).to(torch.int32)
    if case.get("empty"):
        s[2::5] = 0          # slots of the batch that hold no request
    return s


def _selected(lens, topk, ql, gen):
    """ids [rows, topk] of each row's selected blocks (the first, the last two, others at random;
    ascending, -1 behind them) and the row's position."""
    rows = lens.repeat_interleave(ql)
    pos = rows - ql + torch.arange(ql, device="cuda").repeat(lens.shape[0])
    own_block = torch.where(pos >= 0, pos.div(BLOCK, rounding_mode="floor"), pos.clamp(max=-1))
    width = int(own_block.max().clamp(min=0)) + 1
    b = torch.arange(width, device="cuda")
    r = torch.rand(rows.shape[0], width, generator=gen, device="cuda")
    r = torch.where((b == 0) | (b > own_block[:, None] - 2), 2.0, r)
    r = torch.where(b <= own_block[:, None], r, -1.0)
    k = min(topk, width)
    best, ids = r.topk(k, dim=1)
    ids = torch.where(best >= 0, ids, width + 1).sort(dim=1).values
    ids = torch.where(ids < width, ids, -1).to(torch.int32)
    if k < topk:
        ids = torch.cat([ids, torch.full((ids.shape[0], topk - k), -1, device="cuda",
                                         dtype=torch.int32)], 1)
    return ids.contiguous(), pos.to(torch.int32)


def _prepare_attend(case, gen):
    lens = _lengths(case, gen)
    reqs, ql, kvh, d, page = (case[k] for k in ("reqs", "ql", "kvh", "d", "page"))
    q = torch.randn(reqs * ql, case["qh"], d, generator=gen, device="cuda").to(TYPES[case["dtype"]])
    per = BLOCK // page                                   # pages of a 128-token block
    blocks = torch.div(lens + BLOCK - 1, BLOCK, rounding_mode="floor")
    width = max(1, _cdiv(case["hi"], BLOCK))
    total = max(1, int(blocks.sum()))
    pool = total + total // 4 + 1
    perm = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    first = torch.cumsum(blocks, 0) - blocks
    col = torch.arange(width, device="cuda")
    used = col < blocks[:, None]
    block_table = torch.where(used, perm[(first[:, None] + col).clamp(max=pool - 1)], -1)
    pair = case["order"] == "pair"
    stride = 2 * per if pair else per
    kv = TYPES[case["kv"]]

    def values(n):
        shape = (n, kvh, page, d) if case["order"] == "hnd" else (n, page, kvh, d)
        x = torch.empty(shape, dtype=kv, device="cuda")
        for i in range(0, n, 4096):                       # a bounded amount of 32-bit values
            x[i:i + 4096] = torch.randn(x[i:i + 4096].shape, generator=gen, device="cuda").to(kv)
        return x.transpose(1, 2) if case["order"] == "hnd" else x

    if pair:                                              # K pages then V pages of each block
        both = values(pool * 2 * per)
        k, v = both[:-per], both[per:]
    else:
        k, v = values(pool * per), values(pool * per)
    off = torch.arange(per, device="cuda", dtype=torch.int32)
    if case["topk"]:
        ids, pos = _selected(lens, case["topk"], ql, gen)
        at = block_table.repeat_interleave(ql, 0).gather(1, ids.clamp(min=0).long())
        table = torch.where(ids[..., None] >= 0, at[..., None] * stride + off, -1).flatten(1)
        seen = torch.where(ids >= 0, (pos[:, None] + 1 - ids * BLOCK).clamp(max=BLOCK), 0).sum(1)
        seq, query_len, most = seen.to(torch.int32), 1, case["topk"] * BLOCK
    else:
        table = torch.where(used[..., None], block_table[..., None] * stride + off, -1).flatten(1)
        seq, query_len, most = lens, ql, max(case["hi"], ql)
    s = dict(case=case, q=q, k=k, v=v, table=table.to(torch.int32).contiguous(),
             seq=seq.contiguous(), query_len=query_len, max_seq_len=most, sm_scale=d ** -0.5,
             k_scale=0.75 if case["kv"] == "e4m3" else 1.0,
             v_scale=1.25 if case["kv"] == "e4m3" else 1.0,
             out=torch.empty_like(q), weights=None, workspace=None)
    if case["weights"]:
        s["weights"] = torch.empty(q.shape[0], _cdiv(most, BLOCK), device="cuda")
    return s


def _prepare_evict(case, gen):
    lens = _lengths(case, gen).clamp(min=case["ql"])
    reqs, ql = case["reqs"], case["ql"]
    most = max(case["hi"], ql)
    width = _cdiv(most, BLOCK)

    def mass(*shape):                                     # a few heavy blocks, many light ones
        return torch.exp(2.0 * torch.randn(*shape, generator=gen, device="cuda"))

    acc = mass(reqs, width)
    n = torch.div(lens + BLOCK - 1, BLOCK, rounding_mode="floor")
    ids = None
    if case["topk"]:
        ids, _ = _selected(lens, case["topk"], ql, gen)
        weights = torch.where(ids >= 0, mass(reqs * ql, case["topk"]), 0.0)
    else:
        weights = mass(reqs * ql, width)
        weights *= torch.arange(width, device="cuda") < n.repeat_interleave(ql)[:, None]
    table = torch.randperm(reqs * width, generator=gen, device="cuda").to(torch.int32)
    second = torch.randperm(reqs * width, generator=gen, device="cuda").to(torch.int32)
    return dict(case=case, acc=acc, weights=weights, ids=ids, lens=lens, max_seq_len=most,
                table=table.view(reqs, width),
                second=second.view(reqs, width) if case["table"] else None)


def _prepare_verify(case, gen):
    reqs, k, vocab, dtype = case["reqs"], case["k"], case["vocab"], TYPES[case["dtype"]]
    logits = 2.0 * torch.randn(reqs, k + 1, vocab, generator=gen, device="cuda")
    target = torch.softmax(logits, -1).to(dtype)
    logits = logits[:, :k] + 0.8 * torch.randn(reqs, k, vocab, generator=gen, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(reqs, k, vocab, generator=gen, device="cuda")
                                  .clamp(1e-20, 1 - 1e-7)))
    if case["drafts"]:
        tokens = (logits + noise).argmax(-1).to(torch.int32)
        draft = torch.softmax(logits, -1).to(dtype)
    else:                                                 # a guess that is often the likeliest token
        tokens = (1.5 * logits + noise).argmax(-1).to(torch.int32)
        draft = None
    lens = torch.full((reqs,), k, dtype=torch.int32, device="cuda")
    lens[1::3] = k // 2                                   # some requests had fewer drafts
    u = torch.rand(reqs, k + 1, generator=gen, device="cuda")
    return dict(case=case, target=target, draft=draft, tokens=tokens.contiguous(), lens=lens, u=u)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"attend": _prepare_attend, "evict": _prepare_evict,
         "verify": _prepare_verify}[case["op"]](case, gen)
    if own and case["op"] == "attend":
        # the scratch that a serving loop makes once and hands to every step
        import sparse_attention_block_paged_gb300 as mm
        s["workspace"] = mm.new_attention_workspace(
            case["qh"], case["kvh"], case["d"], s["seq"].shape[0], s["query_len"],
            s["max_seq_len"], block_weights=case["weights"])
    return s


# ---------------------------------------------------------------- plain forms

def _rows_of(cache, page, slot):
    if cache.dtype == torch.float8_e4m3fn:                # gathered as bytes
        return cache.view(torch.uint8)[page, slot].view(cache.dtype).float()
    return cache[page, slot].float()


def _plain_attend(s):
    q, seq, ql, size = s["q"], s["seq"], s["query_len"], s["k"].shape[1]
    reqs, (_, qh, d), kvh = seq.shape[0], q.shape, s["k"].shape[2]
    tokens = max(1, int(seq.max()))
    t = torch.arange(tokens, device=q.device)
    there = t < seq[:, None]
    page = torch.where(there, s["table"][:, t // size], 0).long()
    slot = (t % size).expand_as(page)
    k = torch.where(there[..., None, None], _rows_of(s["k"], page, slot), 0.0)
    x = q.float().view(reqs, ql, kvh, qh // kvh, d) * (s["sm_scale"] * s["k_scale"])
    x = torch.einsum("bjhgd,bthd->bhgjt", x, k)
    del k
    last = seq[:, None] - ql + torch.arange(ql, device=q.device)
    seen = (t <= last[..., None])[:, None, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    x = torch.exp(x - top)
    x = x / x.sum(-1, keepdim=True).clamp(min=1e-38)
    v = torch.where(there[..., None, None], _rows_of(s["v"], page, slot), 0.0)
    out = torch.einsum("bhgjt,bthd->bjhgd", x, v) * s["v_scale"]
    out = out.reshape(reqs * ql, qh, d).to(q.dtype)
    if s["weights"] is None:
        return out
    x = torch.nn.functional.pad(x.sum((1, 2)), (0, -tokens % BLOCK))
    x = x.view(reqs * ql, -1, BLOCK).sum(-1)
    return out, torch.nn.functional.pad(x, (0, _cdiv(s["max_seq_len"], BLOCK) - x.shape[1]))


def _plain_evict(s):
    c, reqs, width = s["case"], s["lens"].shape[0], s["acc"].shape[1]
    lens, w = s["lens"], s["weights"].double().view(reqs, -1)
    n = torch.div(lens + BLOCK - 1, BLOCK, rounding_mode="floor")[:, None]
    b = torch.arange(width, device=w.device)
    acc = s["acc"].double() * c["decay"]                  # in 64 bits, rounded once to 32
    if s["ids"] is None:
        acc = acc + w.view(reqs, c["ql"], width).sum(1)
    else:
        acc = acc.scatter_add(1, s["ids"].view(reqs, -1).clamp(min=0).long(), w)
    acc = torch.where(b < n, acc, s["acc"].double()).float()
    rank = torch.where((b < c["init"]) | (b >= n - c["local"]), math.inf, acc)
    rank = torch.where(b < n, rank, -math.inf)
    order = rank.sort(dim=1, descending=True, stable=True).indices
    place = torch.empty_like(order).scatter_(1, order, b.expand_as(order))
    stays = (place < c["budget"]) & (b < n)
    goes = (place >= c["budget"]) & (b < n)
    kept = torch.minimum(n, torch.full_like(n, c["budget"]))

    def packed(x, which, most, fill):                     # the marked columns, moved to the front
        at = torch.where(which, which.long().cumsum(1) - 1, most)
        new = torch.full((reqs, most + 1), fill, dtype=x.dtype, device=x.device)
        return new.scatter_(1, at, x.expand(reqs, width))[:, :most]

    most, gone = c["budget"], max(1, width - c["budget"])
    ids = packed(b.to(torch.int32), stays, most, -1)
    new = [ids, (lens - BLOCK * (n - kept)[:, 0]).to(torch.int32), packed(acc, stays, width, 0.0)]
    for table in (s["table"], s["second"]):
        if table is not None:
            new += [packed(table, stays, most, -1), packed(table, goes, gone, -1)]
    return new


def _plain_verify(s):
    p, q, tokens, u = s["target"], s["draft"], s["tokens"].long(), s["u"]
    reqs, k, vocab = p.shape[0], tokens.shape[1], p.shape[2]
    at = p[:, :k].gather(2, tokens[..., None])[..., 0].double()
    by = 1.0 if q is None else q.gather(2, tokens[..., None])[..., 0].double()
    took = (u[:, :k].double() * by < at) & (torch.arange(k, device=p.device) < s["lens"][:, None])
    count = took.long().cumprod(1).sum(1)
    row = torch.arange(reqs, device=p.device)
    rest = p[row, count].double()                         # 64 bits: sums next to a border
    again = count < s["lens"]
    j = count.clamp(max=k - 1)
    if q is None:
        less = torch.zeros_like(rest).scatter_(1, tokens[row, j][:, None], 2.0)
    else:
        less = q[row, j].double()
    left = (rest - less).clamp(min=0.0)
    use = again[:, None] & (left.sum(1, keepdim=True) > 0)
    cum = torch.where(use, left, rest).cumsum(1)
    picked = (cum <= u[:, k].double()[:, None] * cum[:, -1:]).sum(1).clamp(max=vocab - 1)
    col = torch.arange(k + 1, device=p.device)
    out = torch.where(col < count[:, None], torch.nn.functional.pad(tokens, (0, 1)), -1)
    out = torch.where(col == count[:, None], picked[:, None], out)
    return out.to(torch.int32), count.to(torch.int32)


# ------------------------------------------------------------------------ run

def run(s):
    c = s["case"]
    if not own:
        return {"attend": _plain_attend, "evict": _plain_evict,
                "verify": _plain_verify}[c["op"]](s)
    import sparse_attention_block_paged_gb300 as mm
    if c["op"] == "attend":
        out = mm.paged_attention(s["q"], s["k"], s["v"], s["table"], s["seq"],
                                 query_len=s["query_len"], max_seq_len=s["max_seq_len"],
                                 sm_scale=s["sm_scale"], k_scale=s["k_scale"],
                                 v_scale=s["v_scale"], out=s["out"], block_weights=s["weights"],
                                 workspace=s["workspace"])
        return out if s["weights"] is None else (out, s["weights"])
    if c["op"] == "evict":
        r = mm.evict_blocks(s["acc"], s["lens"], s["table"], budget=c["budget"],
                            init_blocks=c["init"], local_blocks=c["local"],
                            max_seq_len=s["max_seq_len"], block_weights=s["weights"],
                            ids=s["ids"], query_len=c["ql"], decay=c["decay"],
                            attention_block_table=s["second"])
        new = [r.ids, r.seq_lens, r.weights, r.block_table, r.freed]
        if s["second"] is not None:
            new += [r.attention_block_table, r.attention_freed]
        return new
    return mm.verify_drafts(s["target"], s["tokens"], s["u"], draft_probs=s["draft"],
                            draft_lens=s["lens"])


# ----------------------------------------------------------------------- work

def _mean_length(case):
    lo, hi = case["lo"], case["hi"]
    mean = (hi - lo) / math.log(hi / lo) if case.get("log") and hi > lo else (lo + hi) / 2
    return mean * 0.8 if case.get("empty") else mean      # about one slot in five is empty


def work(case):
    reqs = case["reqs"]
    if case["op"] == "attend":
        ql, qh, kvh, d = (case[k] for k in ("ql", "qh", "kvh", "d"))
        tokens, rows = _mean_length(case), reqs * ql
        if case["topk"]:
            # each row reads its own blocks; the rows of a request share the three forced ones, and
            # of the n - 3 others one is read if any of the rows has it
            seen = min(tokens, case["topk"] * BLOCK - BLOCK / 2)
            n = max(3.0, tokens / BLOCK)
            share = min(1.0, max(0, case["topk"] - 3) / max(1e-9, n - 3))
            distinct = 3 + (n - 3) * (1 - (1 - share) ** ql)
            read, pairs = reqs * min(tokens, distinct * BLOCK - BLOCK / 2), rows * seen
        else:
            read, pairs = reqs * tokens, rows * tokens
        size = read * kvh * d * 2 * SIZE[case["kv"]] + rows * qh * d * 2 * SIZE[case["dtype"]]
        if case["weights"]:
            size += 4 * rows * _cdiv(case["topk"] * BLOCK or case["hi"], BLOCK)
        return {"bytes": size, "flops": 4.0 * d * qh * pairs}
    if case["op"] == "evict":
        n = _mean_length(case) / BLOCK
        width = _cdiv(max(case["hi"], case["ql"]), BLOCK)
        entry = case["ql"] * (case["topk"] * 8 if case["topk"] else n * 4)
        tables = 2 if case["table"] else 1
        kept = min(n, case["budget"])
        return {"bytes": reqs * (n * 4 + width * 4 + entry + kept * 4 + 8
                                 + tables * (n + case["budget"] + max(1, width - case["budget"]))
                                 * 4),
                "flops": reqs * n * 2 * case["ql"]}
    # one row of the target's probabilities a request, and one of the drafter's where a draft
    # was rejected (about 45 of 100 are)
    k = case["k"]
    again = 1.0 - (2 * 0.55 ** k + 0.55 ** (k // 2)) / 3
    rows = 1.0 + (again if case["drafts"] else 0.0)
    return {"bytes": reqs * rows * case["vocab"] * SIZE[case["dtype"]] + reqs * (k + 1) * 16,
            "flops": reqs * rows * case["vocab"]}


# ---------------------------------------------------------------------- exact

def _exact_attend(s):
    q, seq, ql = s["q"], s["seq"].tolist(), s["query_len"]
    rows, qh, d = q.shape
    size, kvh = s["k"].shape[1], s["k"].shape[2]
    group = qh // kvh
    out = torch.zeros(rows, qh, d, dtype=torch.float64, device=q.device)
    mass = torch.zeros(rows, _cdiv(s["max_seq_len"], BLOCK), dtype=torch.float64, device=q.device)

    def tokens_of(cache, pages, n):
        x = cache.view(torch.uint8)[pages].view(cache.dtype) if cache.element_size() == 1 \
            else cache[pages]
        return x.flatten(0, 1)[:n].double()

    for i, n in enumerate(seq):
        if n <= 0:
            continue
        pages = s["table"][i, :_cdiv(n, size)].long()
        k, v = tokens_of(s["k"], pages, n), tokens_of(s["v"], pages, n)
        for h in range(kvh):
            x = q[i * ql:(i + 1) * ql, h * group:(h + 1) * group].double()
            sc = (x.reshape(-1, d) @ k[:, h].T) * (s["k_scale"] * s["sm_scale"])
            sc = sc.view(ql, group, n)
            for j in range(ql):
                m = n - ql + j + 1
                if m <= 0:
                    continue
                e = torch.softmax(sc[j, :, :m], -1)
                out[i * ql + j, h * group:(h + 1) * group] = e @ v[:m, h] * s["v_scale"]
                b = torch.arange(m, device=q.device) // BLOCK
                mass[i * ql + j].index_add_(0, b, e.sum(0))
    return out if s["weights"] is None else (out, mass)


def _exact_evict(s):
    # whole numbers are compared as they are; the kept weights in 64 bits
    c, lens = s["case"], s["lens"].tolist()
    acc, w = s["acc"].double().cpu(), s["weights"].double().cpu()
    ids = None if s["ids"] is None else s["ids"].cpu()
    new = torch.zeros(acc.shape, dtype=torch.float64)
    for i, length in enumerate(lens):
        n = _cdiv(length, BLOCK)
        a = acc[i, :n] * c["decay"]
        for j in range(i * c["ql"], (i + 1) * c["ql"]):
            if ids is None:
                a += w[j, :n]
            else:
                ok = ids[j] >= 0
                a.index_add_(0, ids[j][ok].long(), w[j][ok])
        a32 = a.float()
        free = [b for b in range(n) if c["init"] <= b < n - c["local"]]
        free.sort(key=lambda b: (-float(a32[b]), b))
        stays = sorted(set(range(n)) - set(free[max(0, c["budget"] - (n - len(free))):]))
        new[i, :len(stays)] = a[stays]
    tables = 2 if s["second"] is not None else 1
    return [None, None, new] + [None, None] * tables


def exact(case, seed):
    if case["op"] == "verify":
        return None                                       # whole numbers only
    s = prepare(case, seed)
    return _exact_attend(s) if case["op"] == "attend" else _exact_evict(s)
