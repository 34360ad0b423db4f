"""Plain forms of the operators of a cache's pages, on the CPU, and inputs for
their GPU tests.  They share no code with the library."""

import math

import numpy as np
import torch

import serving_ref as R

F64 = torch.float64
E4M3 = torch.float8_e4m3fn


def raw(t):
    """The tensor's elements as integers."""
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    return t if t.dtype == kind else t.view(kind)


# ------------------------------------------------------------------ attention

def scaled_attention_ref(s, ks, vs, k_scale=1.0, v_scale=1.0, drop=()):
    """(out, lse, block weights, bound of out, bound of lse) of attention over pages with scales, in
    64 bits.  The bounds are those of serving_ref.attention_ref for e4m3 pages, in the scaled keys'
    and values' magnitudes, and for a page's scale of its values: its logarithm, rounded, is added
    to an exponent, each off by up to 2^-22 of its magnitude (three roundings); fp16 weights of which
    the largest, times its page's scale, is 2^11 at least, are off by 2^-25, so by 2^-36 of the
    largest scale for every token."""
    q, table, lens, ql = (s[x] for x in ("q", "table", "lens", "ql"))
    rows, qh, d = q.shape
    page, kvh = s["k"].shape[1], s["k"].shape[2]
    group, dev = qh // kvh, q.device
    out = torch.zeros((rows, qh, d), dtype=F64, device=dev)
    tol = torch.zeros_like(out)
    lse = torch.full((rows, qh), -math.inf, dtype=F64, device=dev)
    ltol = torch.zeros_like(lse)
    mass = torch.zeros((rows, R.cdiv(s["max_seq_len"], 128)), dtype=F64, device=dev)
    scale = s["sm_scale"] * k_scale
    for i, n in enumerate(lens.tolist()):
        n = min(max(n, 0), s["max_seq_len"])
        if n == 0:
            continue
        ids = table[i, :R.cdiv(n, page)].long()
        ok = torch.ones(n, dtype=torch.bool, device=dev)
        for p in range(ids.numel()):
            if int(ids[p]) in drop:
                ok[p * page:(p + 1) * page] = False
        ids = ids.clamp(0, s["k"].shape[0] - 1)

        def widened(c, sc):
            x = raw(c)[ids].flatten(0, 1)[:n].view(c.dtype).to(F64)
            return x, sc[ids].to(F64).clamp(2.0 ** -60, 2.0 ** 60).repeat_interleave(page, 0)[:n]

        (kc, kss), (vc, vss) = widened(s["k"], ks), widened(s["v"], vs)
        for j in range(ql):
            m = n - ql + j + 1
            see = ok[:max(m, 0)].nonzero()[:, 0]
            if see.numel() == 0:
                continue
            r = i * ql + j
            for h in range(kvh):
                hs = slice(h * group, (h + 1) * group)
                x = q[r, hs].to(F64)
                kh, vh = kc[see, h] * kss[see, h][:, None], vc[see, h] * vss[see, h][:, None]
                sc = x @ kh.T * scale
                dev_s = d * 2.0 ** -23 * (x.abs() @ kh.abs().T).amax(1) * scale
                dev_s += d * 2.0 ** -24 * scale * x.abs().amax(1) * kh.abs().max()
                power = vss[see, h].log2().abs().max()
                dev_s += 2.0 ** -22 * (sc.abs().amax(1) + 16 + 3 * power)
                p = torch.softmax(sc, -1)
                out[r, hs] = p @ vh * v_scale
                lse[r, hs] = torch.logsumexp(sc, -1)
                sums = (64 + m / 16) * 2.0 ** -23
                size = p @ vh.abs() * abs(v_scale)
                weight = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22
                tol[r, hs] = (R.HALF[q.dtype] * out[r, hs].abs()
                              + (2 * weight + 2 * dev_s[:, None] + 2 * sums) * size
                              + 2.0 ** -36 * m * vss[see, h].max() * vc[see, h].abs().max()
                              * abs(v_scale) + 2.0 ** -24)
                ltol[r, hs] = dev_s + sums + 2.0 ** -22 * (lse[r, hs].abs() + 16)
                mass[r].index_add_(0, see // 128, p.sum(0))
    return out, lse, mass, tol, ltol


# --------------------------------------------------------------------- append

def to_e4m3(x):
    """fp32 numpy to e4m3 (to the nearest, saturated; NaN stays), as a torch tensor."""
    return torch.from_numpy(np.ascontiguousarray(x)).clamp(-448.0, 448.0).to(E4M3)


def least_power(top):
    """The least 2^n with top / 2^n <= 448, n in -60..60."""
    n = -60
    while n < 60 and math.ldexp(448.0, n) < top:
        n += 1
    return np.float32(math.ldexp(1.0, n))


def clamp_scale(x):
    x = float(x)
    return np.float32(2.0 ** -60 if math.isnan(x) else min(max(x, 2.0 ** -60), 2.0 ** 60))


def append_ref(new, cache, scales, table, lens, counts, first_row, page_size, max_seq_len, scale=1.0):
    """One side (keys or values) after the call, in fp32 steps as they are documented: new and cache
    CPU tensors, scales a CPU tensor or None (both are changed in place); entries outside the pool are
    skipped.  Returns the set of (page, slot) that were written."""
    wrote = set()
    with np.errstate(all="ignore"):
        for i, n in enumerate(lens):
            n = min(max(n, 0), max_seq_len)
            t = max(0, n - counts[i])
            while t < n:
                end = min(n, (t // page_size + 1) * page_size)
                p = int(table[i, t // page_size])
                a, b = t % page_size, (end - 1) % page_size + 1
                row = first_row[i] + counts[i] - n + t
                t = end
                if not 0 <= p < cache.shape[0]:
                    continue
                wrote |= {(p, k) for k in range(a, b)}
                y = new[row:row + b - a].float().numpy() / np.float32(scale)
                if cache.dtype != E4M3:
                    cache[p, a:b] = torch.from_numpy(y).to(cache.dtype)
                    continue
                for h in range(cache.shape[2]):
                    z = y[:, h]
                    if scales is None:
                        cache[p, a:b, h] = to_e4m3(z)
                        continue
                    mag = np.abs(z)
                    mag = mag[np.isfinite(mag)]
                    now = least_power(mag.max() if mag.size else 0.0)
                    if a > 0:
                        old = clamp_scale(scales[p, h])
                        now = max(now, old)
                        if now != old:
                            f = np.float32(old / now)
                            cache[p, :a, h] = to_e4m3(cache[p, :a, h].float().numpy() * f)
                            wrote |= {(p, k) for k in range(a)}
                    scales[p, h] = float(now)
                    cache[p, a:b, h] = to_e4m3(z / now)
    return wrote


# ---------------------------------------------------------------------- pages

def allocate_ref(refs, table, lens, ql, page):
    """refs (list) and table (list of rows) in place; whether pages ran out."""
    free = [p for p, n in enumerate(refs) if n == 0]
    short = False
    for i, n in enumerate(lens):
        n = min(max(n, 0), len(table[i]) * page)
        for c in range(max(n - ql, 0) // page, R.cdiv(n, page)):
            if table[i][c] < 0:
                table[i][c] = free.pop(0) if free else -1
                short |= table[i][c] < 0
                if table[i][c] >= 0:
                    refs[table[i][c]] = 1
    return short


def fork_ref(refs, table, lens, parents, page):
    """(rows, lengths, pairs copied); refs (list) in place."""
    free = [p for p, n in enumerate(refs) if n == 0]
    width = len(table[0]) if table else 0
    rows, out_lens, pairs, ups = [], [], [], []
    for i in parents:
        row, n = [-1] * width, 0
        if 0 <= i < len(table):
            n = min(max(lens[i], 0), width * page)
            for c in range(R.cdiv(n, page)):
                p = table[i][c]
                if not 0 <= p < len(refs):
                    continue
                if (c + 1) * page <= n:
                    row[c] = p
                    ups.append(p)
                elif free:
                    row[c] = free.pop(0)
                    pairs.append((p, row[c]))
        rows.append(row)
        out_lens.append(n)
    for p in ups:
        refs[p] += 1
    for _, p in pairs:
        refs[p] = 1
    return rows, out_lens, pairs


def compact_ref(refs, table):
    """(refs, table, live, pairs)."""
    live = sum(n != 0 for n in refs)
    holes = [p for p in range(live) if refs[p] == 0]
    movers = [p for p in range(live, len(refs)) if refs[p] != 0]
    new = list(refs)
    moved = dict(zip(movers, holes))
    for src, dst in moved.items():
        new[dst], new[src] = refs[src], 0
    return new, [[moved.get(p, p) for p in row] for row in table], live, list(moved.items())
