"""Plain 64-bit forms of the operators that use the selection, and inputs for
their GPU tests.  They share no code with the library."""

import math

import torch

BLOCK = 128
F64 = torch.float64
# half a step of a type relative to the value
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# what a weight of the softmax loses before it multiplies a value: a pair of
# bf16 or fp16 numbers holds it to the square of half a step; over e4m3 values
# it is one fp16 number
WEIGHT = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22, torch.float8_e4m3fn: 2.0 ** -11}


def cdiv(a, b):
    return -(-a // b)


def make_attention(lens, *, ql=1, group=4, kvh=2, d=128, page=128, dtype=torch.bfloat16,
                   kv=None, order="nhd", seed=0, poison=float("nan"), spare=3, q_scale=1.0,
                   device="cuda"):
    """Inputs of one attention call: pages dealt in random order from a pool with ``spare`` unused
    ones; unused pages and the slots behind each request's last token hold ``poison``; table entries
    that no request uses hold 2^30."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    kv = kv or dtype
    lens_t = torch.tensor(lens, dtype=torch.int32)
    reqs = len(lens)
    need = [cdiv(max(0, n), page) for n in lens]
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    width = max(1, max(need, default=1))
    table = torch.full((max(reqs, 0), width), 2 ** 30, dtype=torch.int32)
    caches = []
    for c in range(2):
        x = torch.randn((pool, page, kvh, d), generator=g).to(kv).float()
        x = x.to(kv)
        f = x.float()
        used = torch.zeros(pool, dtype=torch.bool)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = perm[at:at + n]
            used[perm[at:at + n].long()] = True
            if lens[i] > 0 and lens[i] % page:
                f[int(perm[at + n - 1]), lens[i] % page:] = poison
            at += n
        f[~used] = poison
        caches.append(f.to(kv).to(device))
    k, v = caches
    if order == "hnd":
        k, v = (x.view(torch.uint8 if kv.itemsize == 1 else torch.int16).transpose(1, 2)
                .contiguous().transpose(1, 2).view(kv) for x in (k, v))
    elif order == "pair":
        # keys and values of a page next to each other in one pool
        raw = torch.uint8 if kv.itemsize == 1 else torch.int16
        both = torch.stack([k.view(raw), v.view(raw)], 1).flatten(0, 1).view(kv)
        k, v = both[:-1], both[1:]
        table = torch.where(table < pool, table * 2, table)
    q = (q_scale * torch.randn((reqs * ql, group * kvh, d), generator=g)).to(dtype).to(device)
    return dict(q=q, k=k, v=v, table=table.to(device), lens=lens_t.to(device), ql=ql,
                max_seq_len=max(ql, max(lens, default=1), 1), sm_scale=d ** -0.5)


def attention_ref(s, k_scale=1.0, v_scale=1.0, drop=()):
    """(out, lse, block weights, bound of out, bound of lse) in 64 bits; ``drop``: page ids whose
    tokens do not count.  The bounds count the roundings: half a step of the output; the weights'
    (WEIGHT); scores as fp32 sums of d exact products in any order, each off by at most 2^-23 of the
    sum of their magnitudes (e4m3 keys: the query scaled into fp16 first, off by 2^-24 of its
    largest); sums over n tokens of which no more than n / 16 are added one after another; fp16
    weights (fp16 and e4m3 caches) of which the largest is at least 2^11 (2^15 at most): each is off
    by half of the smallest step, 2^-25, so by 2^-36 of the sum."""
    q, k, v, table, lens, ql = (s[x] for x in ("q", "k", "v", "table", "lens", "ql"))
    rows, qh, d = q.shape
    page, kvh = k.shape[1], k.shape[2]
    group = qh // kvh
    width = cdiv(s["max_seq_len"], BLOCK)
    dev = q.device
    out = torch.zeros((rows, qh, d), dtype=F64, device=dev)
    tol = torch.zeros_like(out)
    lse = torch.full((rows, qh), -math.inf, dtype=F64, device=dev)
    ltol = torch.zeros_like(lse)
    mass = torch.zeros((rows, width), dtype=F64, device=dev)
    scale = s["sm_scale"] * k_scale
    tiny = 0.0 if v.dtype == torch.bfloat16 else 2.0 ** -36
    raw = torch.uint8 if k.dtype.itemsize == 1 else torch.int16
    for i, n in enumerate(lens.tolist()):
        n = min(max(n, 0), s["max_seq_len"])
        if n == 0:
            continue
        ids = table[i, :cdiv(n, page)].long()
        ok = torch.ones(n, dtype=torch.bool, device=dev)
        for p in range(ids.numel()):
            if int(ids[p]) in drop:
                ok[p * page:(p + 1) * page] = False
        ids = ids.clamp(0, k.shape[0] - 1)
        kk = k.view(raw)[ids].flatten(0, 1)[:n].view(k.dtype).to(F64)
        vv = v.view(raw)[ids].flatten(0, 1)[:n].view(v.dtype).to(F64)
        for j in range(ql):
            m = n - ql + j + 1
            if m <= 0:
                continue
            r = i * ql + j
            see = ok[:m].nonzero()[:, 0]
            if see.numel() == 0:
                continue
            for h in range(kvh):
                hs = slice(h * group, (h + 1) * group)
                x = q[r, hs].to(F64)
                kh, vh = kk[see, h], vv[see, h]
                sc = x @ kh.T * scale
                dev_s = d * 2.0 ** -23 * (x.abs() @ kh.abs().T).amax(1) * scale
                if k.dtype.itemsize == 1:
                    dev_s += d * 2.0 ** -24 * scale * x.abs().amax(1) * kh.abs().max()
                dev_s += 2.0 ** -22 * (sc.abs().amax(1) + 16)
                p = torch.softmax(sc, -1)
                out[r, hs] = p @ vh * v_scale
                lse[r, hs] = torch.logsumexp(sc, -1)
                sums = (64 + m / 16) * 2.0 ** -23
                size = p @ vh.abs() * abs(v_scale)
                tol[r, hs] = (HALF[q.dtype] * out[r, hs].abs()
                              + (2 * WEIGHT[v.dtype] + 2 * dev_s[:, None] + 2 * sums) * size
                              + tiny * m * vh.abs().max() * abs(v_scale) + 2.0 ** -24)
                ltol[r, hs] = dev_s + sums + 2.0 ** -22 * (lse[r, hs].abs() + 16)
                mass[r].index_add_(0, see // BLOCK, p.sum(0))
    return out, lse, mass, tol, ltol


def weights_bound(mass, ltol):
    """The weights' tolerance: twice the scores' and sums' relative error."""
    return mass * (4 * ltol.max() + 2.0 ** -20) + 1e-30


def evict_ref(acc, lens, tables, *, budget, init, local, max_seq_len, weights=None, ids=None,
              ql=1, decay=1.0):
    """Lists of numpy-free Python values: (acc64 after the sum, kept ids, new lengths)."""
    new, kept, out_lens = [], [], []
    for i, length in enumerate(lens):
        length = min(max(length, 0), max_seq_len)
        n = cdiv(length, BLOCK)
        a = acc[i].to(F64).clone()
        a[:n] *= decay
        for r in range(i * ql, (i + 1) * ql):
            if weights is None:
                continue
            if ids is None:
                a[:n] += weights[r, :n].to(F64)
            else:
                for k, b in enumerate(ids[r].tolist()):
                    if 0 <= b < n:
                        a[b] += weights[r, k].to(F64)
        a32 = a.float()
        stay = set(range(min(init, n))) | set(range(max(0, n - local), n))
        free = [b for b in range(n) if b not in stay]
        free.sort(key=lambda b: (0 if math.isnan(float(a32[b])) else 1,
                                 0.0 if math.isnan(float(a32[b])) else -float(a32[b]), b))
        room = budget - len(stay)
        stay |= set(free) if n <= budget else set(free[:room])
        kept.append(sorted(stay))
        new.append(a)
        out_lens.append(length - BLOCK * (n - len(stay)))
    return new, kept, out_lens


def verify_ref(target, tokens, u, draft=None, lens=None):
    """(tokens, accepted) as lists, in exact integers of 2^-46 where the library's are, for
    probabilities from 0 to 1."""
    reqs, rows, vocab = target.shape
    k = rows - 1

    def fixed(x):                       # 64-bit floats hold every value exactly
        x = x.to(F64)
        x = torch.where(torch.isnan(x), torch.zeros_like(x), x).clamp(0, 1)
        return torch.round(x * 2.0 ** 46).to(torch.int64)

    out, accepted = [], []
    for i in range(reqs):
        n = k if lens is None else min(max(int(lens[i]), 0), k)
        row, got = [], n
        for j in range(n):
            d = int(tokens[i, j])
            ok = 0 <= d < vocab
            if ok:
                q = 1.0 if draft is None else float(draft[i, j, d])
                ok = float(u[i, j]) * q < float(target[i, j, d])
            if not ok:
                got = j
                break
            row.append(d)
        w = fixed(target[i, got])
        if got < n:
            d = int(tokens[i, got])
            if draft is not None:
                left = (w - fixed(draft[i, got])).clamp(min=0)
            else:
                left = w.clone()
                if 0 <= d < vocab:
                    left[d] = 0
            if int(left.sum()) > 0:
                w = left
        cum = torch.cumsum(w, 0)
        total = int(cum[-1])
        un = min(max(float(u[i, k]), 0.0), 1.0 - 2.0 ** -24)
        x = int(un * 2.0 ** 64) * total >> 64
        hit = (cum > x).nonzero()
        row.append(int(hit[0]) if hit.numel() else vocab - 1)
        out.append(row + [-1] * (rows - len(row)))
        accepted.append(got)
    return out, accepted
