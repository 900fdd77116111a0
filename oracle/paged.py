"""The paged 8-bit key/value cache in float64 / plain integers, one sequence and page at a time.

Written from the definitions at the calls of include/csa.h (the library's own: the pages compare the
compressed caches against a grouped-query cache and give none of its details).  Arrays: k / v
[n_pages][Hkv][page][D] e4m3 codes (uint8), k_scale / v_scale [n_pages][Hkv], table [B][cap], refs
[n_pages].  Functions that change state return changed copies.
"""

import numpy as np

from .formats import e4m3_decode, e4m3_encode

MIN_SCALE = 2.0 ** -126


def tokens(n_new, Tq, b):
    return Tq if n_new is None else int(min(max(int(n_new[b]), 0), Tq))


def page_scale(amax):
    """The smallest power of two s >= 2^-126 with amax / s <= 448."""
    s = MIN_SCALE
    if amax > 0:
        s = max(s, 2.0 ** np.ceil(np.log2(amax / 448.0)))
        while amax / s > 448:
            s *= 2
        while s / 2 >= MIN_SCALE and amax / (s / 2) <= 448:
            s /= 2
    return s


def append(k, v, k_scale, v_scale, table, refs, page, k_new, v_new, start, n_new):
    """Returns (k, v, k_scale, v_scale, error)."""
    k, v, k_scale, v_scale = k.copy(), v.copy(), k_scale.copy(), v_scale.copy()
    B, Tq, Hkv, _ = k_new.shape
    N, cap, error = len(refs), table.shape[1], False
    for b in range(B):
        n, s = tokens(n_new, Tq, b), int(start[b])
        if s < 0 or n == 0:
            continue
        for p in range(s // page, (s + n - 1) // page + 1):
            g = int(table[b, p]) if p < cap else -1
            if g < 0 or g >= N or refs[g] > 1:
                error = True
                continue
            lo, hi = max(s - p * page, 0), min(s + n - p * page, page)
            for store, scale, new in ((k, k_scale, k_new), (v, v_scale, v_new)):
                for h in range(Hkv):
                    x = new[b, p * page + lo - s:p * page + hi - s, h].astype(np.float64)
                    fin = np.abs(x[np.isfinite(x)])
                    now = page_scale(fin.max() if fin.size else 0.0)
                    if lo > 0:
                        old = float(scale[g, h])
                        now = max(now, old)
                        if now != old:
                            store[g, h, :lo] = e4m3_encode(e4m3_decode(store[g, h, :lo]) * (old / now))
                    code = e4m3_encode(np.nan_to_num(x / now, nan=0.0, posinf=448.0, neginf=-448.0))
                    store[g, h, lo:hi] = np.where(np.isnan(x), 0x7F, code)
                    scale[g, h] = now
    return k, v, k_scale, v_scale, error


def attend(k, v, k_scale, v_scale, table, page, q, start, n_new, n_max, window=0, first=0, sinks=None, scale=None):
    """Returns (out [B][Tq][H][D], asked [B][Tq], weight, logit): out is 0 where nothing is seen; weight =
    sum_i p_i |v_i| per channel and logit = the largest sum_d |q_d k_d| * scale over the keys seen, the
    quantities that rounding errors are proportional to."""
    B, Tq, H, D = q.shape
    N, Hkv = k.shape[:2]
    G = H // Hkv
    scale = scale or 1.0 / np.sqrt(D)
    out, weight = np.zeros((B, Tq, H, D)), np.zeros((B, Tq, H, D))
    logit, asked = np.zeros((B, Tq, H, 1)), np.zeros((B, Tq), bool)
    for b in range(B):
        n, s = tokens(n_new, Tq, b), int(start[b])
        if s < 0:
            continue
        end = min(s + n, n_max)
        pos = np.arange(max(end, 0))
        g = table[b, pos // page] if len(pos) else np.zeros(0, int)
        there = (g >= 0) & (g < N)
        gs, slot = np.where(there, g, 0), pos % page
        for h in range(Hkv):
            K = e4m3_decode(k[gs, h, slot]) * k_scale[gs, h, None].astype(np.float64)
            V = e4m3_decode(v[gs, h, slot]) * v_scale[gs, h, None].astype(np.float64)
            for j in range(n):
                t = s + j
                if t >= n_max:
                    continue
                asked[b, j] = True
                see = there & (pos <= t)
                if window:
                    see &= (pos > t - window) | (pos < first)
                if not see.any():
                    continue
                Q = q[b, j, h * G:(h + 1) * G].astype(np.float64)
                with np.errstate(invalid="ignore", over="ignore"):
                    z = Q @ K[see].T * scale
                    zz = z if sinks is None else np.concatenate([z, sinks[h * G:(h + 1) * G, None]], 1)
                    e = np.exp(zz - zz.max(1, keepdims=True))
                    p = (e / e.sum(1, keepdims=True))[:, :z.shape[1]]
                    out[b, j, h * G:(h + 1) * G] = p @ V[see]
                    weight[b, j, h * G:(h + 1) * G] = p @ np.abs(V[see])
                    logit[b, j, h * G:(h + 1) * G, 0] = (np.abs(Q) @ np.abs(K[see]).T * scale).max(1)
    return out, asked, weight, logit


def fork(table, refs, src, dst):
    """Returns (table, refs, error)."""
    was, table, refs, error = table, table.copy(), refs.copy(), False
    B, N = table.shape[0], len(refs)
    for i, (s, d) in enumerate(zip(src, dst)):
        if s == -1 and d == -1:
            continue
        if not (0 <= s < B and 0 <= d < B) or d in list(src) or d in list(dst[:i]):
            error = True
            continue
        new = np.where((was[s] >= 0) & (was[s] < N), was[s], -1)
        error |= bool((was[s] >= N).any() or (was[d] >= N).any())
        for g in new[new >= 0]:
            refs[g] += 1
        for g in was[d][(was[d] >= 0) & (was[d] < N)]:
            refs[g] -= 1
        table[d] = new
    return table, refs, error


def reserve(table, refs, page, start, n_new, Tq):
    """Returns (table, refs, copy_src, copy_dst, missing, error)."""
    B, cap = table.shape
    N, error = len(refs), False
    copy_src, copy_dst = np.full(B, -1, np.int32), np.full(B, -1, np.int32)
    wanted = []                                                   # (row, entry) in order
    for b in range(B):
        n, s = tokens(n_new, Tq, b), int(start[b])
        if s < 0 or n == 0:
            continue
        if s + n > cap * page:
            error = True
            continue
        for p in range(s // page, (s + n - 1) // page + 1):
            if table[b, p] >= N:
                error = True
            else:
                wanted.append((b, p))
    writers = {}
    for b, p in wanted:
        if table[b, p] >= 0:
            writers.setdefault(int(table[b, p]), []).append((b, p))
    need = []
    for b, p in wanted:
        g = int(table[b, p])
        if g < 0:
            need.append((b, p))
        elif len(writers[g]) < refs[g] or writers[g][-1] != (b, p):
            need.append((b, p))
    free = [g for g in range(N) if refs[g] == 0]
    if len(need) > len(free):
        return table.copy(), refs.copy(), copy_src, copy_dst, len(need) - len(free), error
    table, refs = table.copy(), refs.copy()
    for (b, p), g in zip(need, free):
        old = int(table[b, p])
        if old >= 0:
            refs[old] -= 1
            if p * page < start[b]:
                copy_src[b], copy_dst[b] = old, g
        table[b, p] = g
        refs[g] = 1
    return table, refs, copy_src, copy_dst, 0, error


def free(table, refs, page, keep, begin, first):
    table, refs = table.copy(), refs.copy()
    for b in range(table.shape[0]):
        for p in range(table.shape[1]):
            drop = keep is not None and keep[b] >= 0 and p * page >= keep[b]
            drop |= begin is not None and p * page >= first and (p + 1) * page <= begin[b]
            if drop:
                if 0 <= table[b, p] < len(refs):
                    refs[table[b, p]] -= 1
                table[b, p] = -1
    return table, refs


def compact(table, refs, max_moves):
    """Returns (table, refs, move_src, move_dst, count)."""
    table, refs = table.copy(), refs.copy()
    used, unused = np.flatnonzero(refs > 0)[::-1], np.flatnonzero(refs <= 0)
    pairs = [(s, d) for s, d in zip(used, unused) if d < s][:max_moves]
    move_src, move_dst = np.full(max_moves, -1, np.int32), np.full(max_moves, -1, np.int32)
    to = np.arange(len(refs))
    for i, (s, d) in enumerate(pairs):
        move_src[i], move_dst[i], to[s] = s, d, d
        refs[d], refs[s] = refs[s], 0
    ok = (table >= 0) & (table < len(refs))
    table = np.where(ok, to[np.where(ok, table, 0)], table).astype(np.int32)
    return table, refs, move_src, move_dst, len(pairs)
