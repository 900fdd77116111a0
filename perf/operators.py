"""Timed cases of the paged 8-bit key/value cache: attention over it, appending to it, forking and
compacting its pages.

The cache holds keys and values of grouped-query attention as e4m3 codes in pages of `page` tokens,
k / v [n_pages][Hkv][page][D], with one power-of-two scale per page and KV head, k_scale / v_scale
[n_pages][Hkv]; a page table [B][cap] names the page of each run of `page` tokens (-1: none) and refs
[n_pages] counts the table entries that name a page.  Token j of a call sits at position start[b] + j,
j < n_new[b].

  attend  o = sum_i p_i v_i, p = softmax over the keys i <= t that lie in the window (i > t - window,
          all of them when window is 0) or among the `first` tokens, with an optional sink logit per
          head in the denominator; a row that sees nothing is 0, a row past n_new[b] is left as it was
  append  the new tokens' keys and values are encoded into their pages; a page's scale is the smallest
          power of two (at least 2^-126) that fits its new values to 448, never below the scale its
          earlier tokens already have; where it grows, the earlier codes are rounded to the new scale
  fork    rows of the page table copied to other rows, pages for the next tokens reserved (lowest free
          page first, a shared page that would be written is replaced by a copy), those pages copied
  compact pages of ended sequences or of tokens behind the window released, the i-th highest used page
          moved to the i-th lowest free one while that is lower, tables rewritten, pages copied

`own` selects the framework's kernels in run(); otherwise run() is the plain form.
"""

import math

import torch

own = False

ACT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _attend(name, B, n, Tq, H, Hkv, D, page, window=0, first=0, act="bf16", spread=0.0, ragged=False, sink=False):
    return dict(name=name, op="attend", B=B, n=n, Tq=Tq, H=H, Hkv=Hkv, D=D, page=page, window=window, first=first,
                act=act, spread=spread, ragged=ragged, sink=sink)


def _append(name, B, n, Tq, Hkv, D, page, act="bf16", spread=0.0, ragged=False):
    return dict(name=name, op="append", B=B, n=n, Tq=Tq, Hkv=Hkv, D=D, page=page, act=act, spread=spread,
                ragged=ragged)


def _fork(name, rows, forks, n, Hkv, D, page, Tq):
    return dict(name=name, op="fork", rows=rows, forks=forks, n=n, Hkv=Hkv, D=D, page=page, Tq=Tq)


def _compact(name, live, ended, n, Hkv, D, page, moves, window=0, first=0):
    return dict(name=name, op="compact", live=live, ended=ended, n=n, Hkv=Hkv, D=D, page=page, moves=moves,
                window=window, first=first)


def listed():
    return [
        # one short chat turn in float32, as the small decode workload runs (8 heads, 2,048 tokens)
        _attend("decode f32 2k", 1, 2048, 1, 8, 2, 128, 16, act="f32"),
        # a serving batch at the 131,072-token workload's batch of 8, its sequences of unequal length, GQA-8
        _attend("decode 128k ragged", 8, 131072, 1, 64, 8, 128, 64, spread=0.6),
        # one sequence at 1,048,576 tokens, the length of the headline decode workload, GQA-8
        _attend("decode 1m", 1, 1048576, 1, 64, 8, 128, 64, sink=True),
        # a sliding-window layer in a large batch: window pages and the first page alone are left
        _attend("decode window 64 seqs", 64, 32768, 1, 64, 8, 128, 64, window=4096, first=4, spread=0.4),
        # a chunk of a prompt behind a prefix, 64 heads as the chunked prefill has
        _attend("chunk 2k after 14k", 1, 16384, 2048, 64, 8, 128, 64),
        # chunks of unequal length in one padded batch of a windowed layer with as many KV heads as heads
        _attend("chunk window ragged", 4, 5000, 513, 16, 16, 64, 32, window=1024, first=8, spread=0.5, ragged=True),
        # the tokens of one decode step, 64 sequences
        _append("append step", 64, 8191, 1, 8, 128, 64, spread=0.7),
        # the prefill chunk of 8,192 tokens, two prompts of unequal length that start inside a page
        _append("append chunk 8k", 2, 20001, 8192, 8, 128, 64, spread=0.3, ragged=True),
        # four samples of one request, each about to take its next token
        _fork("fork 4", 32, 4, 2003, 2, 64, 16, 1),
        # many requests sampled twice, each with a few tokens to check
        _fork("fork 128", 512, 128, 8190, 8, 128, 64, 5),
        # a small pool after a few requests ended
        _compact("compact small", 12, 5, 1500, 2, 64, 16, 90),
        # a large pool of windowed sequences, their pages behind the window released
        _compact("compact window", 64, 16, 8000, 8, 128, 64, 900, window=4096, first=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "fork", "compact"])
    D, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if op == "attend":
        Hkv, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16])
        act = rng.choice(["bf16", "bf16", "bf16", "f32"])
        window = rng.choice([0, 0, _log(rng, 16, 8192)])
        first = rng.choice([0, 1, 4, 64, 100]) if window else 0
        B = _log(rng, 1, 48)
        if rng.random() < 0.6:
            Tq, n = rng.choice([1, 1, 1, 2, 4, 7]), _log(rng, 8, max(9, 1048576 // B))
        else:
            Tq = _log(rng, 8, 1500)
            B = max(1, min(B, 2000 // Tq))
            n = Tq + _log(rng, 1, 12000)
            if act == "f32":
                Tq, n = min(Tq, 300), min(n, 4000)
        return _attend(None, B, max(n, Tq), Tq, Hkv * group, Hkv, D, page, window, first, act, rng.choice([0.0, 0.5, 0.9]),
                       rng.random() < 0.5, rng.random() < 0.5) | {"name": "a"}
    if op == "append":
        B, Tq = _log(rng, 1, 100), rng.choice([1, 1, _log(rng, 2, 8192)])
        B = max(1, min(B, 16384 // Tq))
        return _append(None, B, Tq + _log(rng, 1, min(16384, 400000 // B)), Tq, rng.choice([1, 2, 4, 8]), D, page,
                       rng.choice(["bf16", "bf16", "f32"]), rng.choice([0.0, 0.5]), rng.random() < 0.5) | {"name": "a"}
    Hkv, n = rng.choice([1, 2, 4, 8]), _log(rng, 100, 8000)
    if op == "fork":
        forks = _log(rng, 1, 100)
        return _fork(None, 2 * forks + rng.randrange(20), forks, n, Hkv, D, page, rng.choice([1, 3, 20])) | {"name": "a"}
    live, ended = _log(rng, 2, 40), _log(rng, 1, 20)
    pages = -(-n // page)
    window = rng.choice([0, max(1, n // 3)])
    after = live * (pages if not window else -(-window // page))
    return _compact(None, live, ended, n, Hkv, D, page, max(1, min(after, ended * pages) // rng.choice([2, 3, 5])),
                    window, 4 if window else 0) | {"name": "a"}


def _lens(case):
    """(start, n_new) of every sequence: they belong to the case, not to the seed."""
    B, n, Tq = case["B"], case["n"], case["Tq"]
    start, new = [], []
    for b in range(B):
        total = max(Tq, n - int(case["spread"] * n * b / max(1, B)))
        new.append(max(1, Tq - (b * 7) % (Tq // 2 + 1)) if case["ragged"] else Tq)
        start.append(total - new[-1])
    return start, new


def _visible(start, new, window, first):
    """Keys that the queries of one sequence see: the sum over the queries, and their union."""
    total = 0
    if not window:
        return new * start + new * (new + 1) // 2, start + new
    for t in range(start, start + new):
        lo = max(0, t + 1 - window)
        total += t + 1 - lo + min(first, lo)
    lo = max(0, start + 1 - window)
    return total, start + new - lo + min(first, lo)


def work(case):
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    if case["op"] in ("attend", "append"):
        start, new = _lens(case)
        a = 4 if case["act"] == "f32" else 2
        tokens = sum(new)
        if case["op"] == "append":
            pages = sum(-(-(s + m) // page) - s // page for s, m in zip(start, new))
            return {"bytes": 2 * tokens * Hkv * D * (a + 1) + 8 * pages * Hkv + 4 * pages, "flops": 0}
        seen = [_visible(s, m, case["window"], case["first"]) for s, m in zip(start, new)]
        keys, pairs = sum(u for _, u in seen), sum(t for t, _ in seen)
        return {"bytes": 2 * keys * Hkv * D + 8 * (keys // page + 1) * Hkv + 4 * (keys // page + 1)
                + 2 * tokens * case["H"] * D * a, "flops": 4 * case["H"] * D * pairs}
    pb = 2 * Hkv * page * D + 8 * Hkv                       # one page and its scales
    if case["op"] == "fork":
        copies = case["forks"] if case["n"] % page else 0
        return {"bytes": 2 * copies * pb + 4 * case["forks"] * 3 * (-(-case["n"] // page)), "flops": 0}
    p = _compact_plan(case)
    return {"bytes": 2 * case["moves"] * pb + 4 * (p["N"] + 2 * p["rows"] * p["cap"]), "flops": 0}


def _compact_plan(case):
    """Rows, row capacity, pages a row keeps and loses, pool size."""
    page, n = case["page"], case["n"]
    cap = -(-n // page)
    if case["window"]:
        gone = [p for p in range(cap) if p * page >= case["first"] and (p + 1) * page <= n - case["window"]]
    else:
        gone = []
    keep = [p for p in range(cap) if p not in set(gone)]
    used, freed = case["live"] * len(keep), case["live"] * len(gone) + case["ended"] * cap
    return dict(cap=cap, rows=case["live"] + case["ended"], keep=keep, gone=gone, used=used, freed=freed,
                N=used + max(freed, case["moves"]) + used // 8 + 1)


def _power(k):
    """2^k in float32, from its bits (a power function may be off in the last place)."""
    return ((k.to(torch.int32) + 127) << 23).view(torch.float32)


def _codes(gen, shape, dev):
    """e4m3 codes of normal values with a standard deviation of 100, and their pages' scales."""
    c = torch.empty(shape, dtype=torch.uint8, device=dev)
    flat = c.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        m = min(step, flat.numel() - i)
        z = torch.randn(m, generator=gen, device=dev).mul_(100.0).clamp_(-448, 448)
        flat[i:i + m] = z.to(torch.float8_e4m3fn).view(torch.uint8)
    e = torch.randint(-8, -5, shape[:2], generator=gen, device=dev)
    return c, _power(e)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    s = {"case": case}
    if case["op"] in ("attend", "append"):
        start, new = _lens(case)
        B, Tq = case["B"], case["Tq"]
        cap = max(-(-(a + m) // page) for a, m in zip(start, new))
        held = torch.zeros(B, cap, dtype=torch.bool, device=dev)
        p = torch.arange(cap, device=dev)
        s["start"] = torch.tensor(start, dtype=torch.int64, device=dev)
        s["n_new"] = torch.tensor(new, dtype=torch.int32, device=dev)
        end = (s["start"] + s["n_new"])[:, None]
        held |= p * page < end
        if case["op"] == "attend" and case["window"]:       # pages behind the window have been released
            held &= (p * page < case["first"]) | ((p + 1) * page > s["start"][:, None] + 1 - case["window"])
        count = int(held.sum())
        N = count + count // 8 + 2
        ids = torch.randperm(N, generator=gen, device=dev)[:count].to(torch.int32)
        s["table"] = torch.full((B, cap), -1, dtype=torch.int32, device=dev)
        s["table"][held] = ids
        s["refs"] = torch.zeros(N, dtype=torch.int32, device=dev)
        s["refs"][ids.long()] = 1
        s["n_max"] = max(a + m for a, m in zip(start, new))
        s["k"], s["k_scale"] = _codes(gen, (N, Hkv, page, D), dev)
        s["v"], s["v_scale"] = _codes(gen, (N, Hkv, page, D), dev)
        act = ACT[case["act"]]
        if case["op"] == "attend":
            H = case["H"]
            s["q"] = (2 * torch.randn(B, Tq, H, D, generator=gen, device=dev)).to(act)
            s["sinks"] = torch.randn(H, generator=gen, device=dev) if case["sink"] else None
            s["out"] = torch.zeros(B, Tq, H, D, dtype=act, device=dev)
        else:
            # projections of unequal size from head to head, some tokens far larger than their neighbours
            size = _power(torch.randint(-2, 3, (Hkv, 1), generator=gen, device=dev))
            big = 1 + 3 * (torch.rand(B, Tq, 1, 1, generator=gen, device=dev) > 0.98)
            s["k_new"] = (torch.randn(B, Tq, Hkv, D, generator=gen, device=dev) * size * big).to(act)
            s["v_new"] = (torch.randn(B, Tq, Hkv, D, generator=gen, device=dev) * size).to(act)
            pairs = [(b, i) for b in range(B) for i in range(-(-(start[b] + new[b]) // page) - start[b] // page)]
            s["touched"] = torch.tensor(pairs, dtype=torch.int64, device=dev)       # (sequence, page of the call)
    elif case["op"] == "fork":
        rows, forks, n, Tq = case["rows"], case["forks"], case["n"], case["Tq"]
        cap, held = -(-(n + Tq) // page), -(-n // page)
        # every second row of the first 2 * forks holds a sequence, the row after it is its fork; the rest hold others
        src = list(range(0, 2 * forks, 2))
        other = list(range(2 * forks, rows))
        share = max(1, held // 2)                           # the others have only their first half
        count = forks * held + len(other) * share
        fresh = 2 * forks * (cap - held + 1)
        N = count + fresh + 7
        ids = torch.randperm(N, generator=gen, device=dev)[:count].to(torch.int32)
        s["table"] = torch.full((rows, cap), -1, dtype=torch.int32, device=dev)
        s["table"][src, :held] = ids[:forks * held].view(forks, held)
        if other:
            s["table"][other, :share] = ids[forks * held:].view(len(other), share)
        s["refs"] = torch.zeros(N, dtype=torch.int32, device=dev)
        s["refs"][ids.long()] = 1
        s["src"] = torch.tensor(src, dtype=torch.int32, device=dev)
        s["dst"] = s["src"] + 1
        s["start"] = torch.full((rows,), -1, dtype=torch.int64, device=dev)
        s["start"][:2 * forks] = n
        s["n_new"] = torch.full((rows,), Tq, dtype=torch.int32, device=dev)
        s["k"], s["k_scale"] = _codes(gen, (N, Hkv, page, D), dev)
        s["v"], s["v_scale"] = _codes(gen, (N, Hkv, page, D), dev)
        s["copy_src"] = torch.empty(rows, dtype=torch.int32, device=dev)
        s["copy_dst"] = torch.empty(rows, dtype=torch.int32, device=dev)
        s["missing"] = torch.empty(1, dtype=torch.int32, device=dev)
    else:
        p = _compact_plan(case)
        N, U, M = p["N"], p["used"], case["moves"]
        below = torch.randperm(U, generator=gen, device=dev)
        above = U + torch.randperm(N - U, generator=gen, device=dev)
        stay = torch.cat([below[M:], above[:M]])            # pages in use after the release
        stay = stay[torch.randperm(U, generator=gen, device=dev)].to(torch.int32)
        freed = torch.cat([below[:M], above[M:]])
        freed = freed[torch.randperm(N - U, generator=gen, device=dev)][:p["freed"]].to(torch.int32)
        s["table"] = torch.full((p["rows"], p["cap"]), -1, dtype=torch.int32, device=dev)
        live = case["live"]
        g = live * len(p["gone"])
        s["table"][:live, torch.tensor(p["keep"], device=dev)] = stay.view(live, len(p["keep"]))
        if p["gone"]:
            s["table"][:live, torch.tensor(p["gone"], device=dev)] = freed[:g].view(live, len(p["gone"]))
        s["table"][live:] = freed[g:].view(case["ended"], p["cap"])
        s["refs"] = torch.zeros(N, dtype=torch.int32, device=dev)
        s["refs"][stay.long()] = 1
        s["refs"][freed.long()] = 1
        s["keep"] = torch.full((p["rows"],), -1, dtype=torch.int64, device=dev)
        s["keep"][live:] = 0
        s["begin"] = None
        if case["window"]:
            s["begin"] = torch.zeros(p["rows"], dtype=torch.int64, device=dev)
            s["begin"][:live] = case["n"] - case["window"]
        s["k"], s["k_scale"] = _codes(gen, (N, Hkv, page, D), dev)
        s["v"], s["v_scale"] = _codes(gen, (N, Hkv, page, D), dev)
        s["move_src"] = torch.empty(N, dtype=torch.int32, device=dev)
        s["move_dst"] = torch.empty(N, dtype=torch.int32, device=dev)
        s["count"] = torch.empty(1, dtype=torch.int32, device=dev)
    if own:
        from long_context_sparse_csa_b200 import binding as C
        s["G"] = C.make_gqa(case.get("H", Hkv), Hkv, D, case.get("window", 0), case.get("first", 0),
                            act_format=case.get("act", "bf16"))
        s["P"] = C.make_page_pool(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if case["op"] in ("attend", "append"):
            s["T"] = C.make_page_table(s["table"], s["refs"], page)
        if case["op"] == "attend":
            n = C.csa_paged_workspace_size(s["G"], s["T"], case["Tq"], s["n_max"])
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device=dev)
    return s


# ----------------------------------------------------------------------------- the framework's calls
def _run_own(s):
    from long_context_sparse_csa_b200 import binding as C
    case = s["case"]
    if case["op"] == "attend":
        C.csa_paged_attend(s["G"], s["P"], s["T"], s["q"], s["sinks"], s["start"], s["n_new"], case["Tq"], s["n_max"],
                           s["out"], s["ws"])
        return s["out"]
    if case["op"] == "append":
        C.csa_paged_append(s["G"], s["P"], s["T"], s["k_new"], s["v_new"], s["start"], s["n_new"], case["Tq"])
        return _held(s)
    # the bookkeeping is updated in place: each pass starts from the state's own
    table, refs = s["table"].clone(), s["refs"].clone()
    T = C.make_page_table(table, refs, case["page"])
    if case["op"] == "fork":
        rows = case["rows"]
        C.csa_pages_fork(T, s["src"], s["dst"], case["forks"])
        C.csa_pages_reserve(T, s["start"], s["n_new"], case["Tq"], s["copy_src"], s["copy_dst"], s["missing"])
        C.csa_pages_copy(s["G"], s["P"], T, s["copy_src"], s["copy_dst"], None, rows)
        return _pages(s, table, refs) | {"copy_src": s["copy_src"], "copy_dst": s["copy_dst"], "missing": s["missing"]}
    N = s["refs"].numel()
    C.csa_pages_free(T, s["keep"], s["begin"], case["first"])
    C.csa_pages_compact(T, N, s["move_src"], s["move_dst"], s["count"])
    C.csa_pages_copy(s["G"], s["P"], T, s["move_src"], s["move_dst"], s["count"], N)
    return _pages(s, table, refs) | {"move_src": s["move_src"], "move_dst": s["move_dst"], "count": s["count"]}


def _held(s):
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _pages(s, table, refs):
    return {"table": table, "refs": refs, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ----------------------------------------------------------------------------- the plain forms
def _rows(store, scale, page, g, slot, ok):
    """Rows [B][M][Hkv][D] in float32 of the tokens in slot `slot` of pages g; 0 where not ok."""
    g = torch.where(ok, g, 0).long()
    codes = store.permute(0, 2, 1, 3)[g, slot]
    x = codes.view(torch.float8_e4m3fn).float() * scale[g][..., None]
    return x.masked_fill_(~ok[..., None, None], 0.0)


def _plain_attend(s):
    case = s["case"]
    B, Tq, H, Hkv, D, page = (case[x] for x in ("B", "Tq", "H", "Hkv", "D", "page"))
    window, first = case["window"], case["first"]
    dev, table, start = s["q"].device, s["table"], s["start"]
    end = start + s["n_new"]
    if window:                                              # the first tokens, then those from the window's start on
        lo = (start + 1 - window).clamp(min=first)
        near = lo[:, None] + torch.arange(window + Tq - 1, device=dev)
        pos = torch.cat([torch.arange(first, device=dev).expand(B, first), near], 1)
    else:
        pos = torch.arange(s["n_max"], device=dev).expand(B, s["n_max"])
    p = pos // page
    inside = (pos < end[:, None]) & (p < table.shape[1])
    g = torch.gather(table, 1, torch.where(inside, p, 0))
    ok = inside & (g >= 0)
    k = _rows(s["k"], s["k_scale"], page, g, pos % page, ok)
    v = _rows(s["v"], s["v_scale"], page, g, pos % page, ok)
    t = start[:, None] + torch.arange(Tq, device=dev)       # [B][Tq]
    see = ok[:, None, :] & (pos[:, None, :] <= t[..., None])
    if window:
        see &= (pos[:, None, :] > t[..., None] - window) | (pos[:, None, :] < first)
    G = H // Hkv
    q = s["q"].float().view(B, Tq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Tq * G, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(D)).view(B, Hkv, Tq, G, -1)
    z.masked_fill_(~see[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, Hkv, 1, G, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    e = z.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + (sink - m).exp()
    o = torch.matmul(e.view(B, Hkv, Tq * G, -1), v.permute(0, 2, 1, 3)).view(B, Hkv, Tq, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, Tq, H, D)
    asked = (torch.arange(Tq, device=dev) < s["n_new"][:, None])[..., None, None]
    s["out"].copy_(torch.where(asked, o.to(s["out"].dtype), s["out"]))
    return s["out"]


def _pow2_scale(amax):
    f, e = torch.frexp(amax)
    k = torch.where(f <= 0.875, e - 9, e - 8).clamp(min=-126)
    return _power(torch.where(amax > 0, k, -126))


def _encode(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    case = s["case"]
    page, Tq = case["page"], case["Tq"]
    b, i = s["touched"].unbind(1)
    start, new = s["start"][b], s["n_new"][b].long()
    p = start // page + i
    g = s["table"][b, p].long()
    pos = p[:, None] * page + torch.arange(page, device=p.device)      # [pages][page]
    j = pos - start[:, None]
    fresh, old = (j >= 0) & (j < new[:, None]), j < 0
    j = j.clamp(0, Tq - 1)
    for x, store, scale in ((s["k_new"], s["k"], s["k_scale"]), (s["v_new"], s["v"], s["v_scale"])):
        rows = x[b[:, None], j].float().permute(0, 2, 1, 3)            # [pages][Hkv][page][D]
        rows = rows.masked_fill(~fresh[:, None, :, None], 0.0)
        before = torch.where(old.any(1)[:, None], scale[g], 0.0)
        after = torch.maximum(_pow2_scale(rows.abs().amax((2, 3))), before)
        codes = store[g]
        was = _encode(codes.view(torch.float8_e4m3fn).float() * (before / after)[..., None, None])
        now = _encode(rows / after[..., None, None])
        store[g] = torch.where(fresh[:, None, :, None], now, torch.where(old[:, None, :, None], was, codes))
        scale[g] = after
    return _held(s)


def _plain_copy(s, src, dst):
    """Page src[i] to page dst[i]; for -1 (nothing to do) the last page, which no copy goes to, is written onto itself."""
    ok = src >= 0
    at = torch.where(ok, dst, s["refs"].numel() - 1).long()
    by = torch.where(ok, src, s["refs"].numel() - 1).long()
    for x in ("k", "v", "k_scale", "v_scale"):
        s[x][at] = s[x][by]


def _plain_fork(s):
    case = s["case"]
    page, Tq = case["page"], case["Tq"]
    table, refs = s["table"].clone(), s["refs"].clone()
    N, (rows, cap) = refs.numel(), table.shape
    dev = table.device
    taken = table[s["src"].long()]
    table[s["dst"].long()] = taken
    one = (taken >= 0).to(torch.int32).view(-1)
    refs.index_add_(0, taken.clamp(min=0).view(-1).long(), one)
    # the pages that hold the positions [start, start + Tq) of each row
    K = Tq // page + 2
    start, new = s["start"][:, None], s["n_new"][:, None].long()
    p = start.clamp(min=0) // page + torch.arange(K, device=dev)
    wanted = (start >= 0) & (new > 0) & (p * page < start + new) & (p < cap)
    at = torch.where(wanted, p, 0)
    g = torch.gather(table, 1, at)
    held = wanted & (g >= 0)
    gl = g.clamp(min=0).long()
    shared = held & (refs[gl] > 1)
    inside = torch.zeros_like(refs).index_add_(0, gl.view(-1), shared.to(torch.int32).view(-1))
    row = torch.arange(rows, device=dev)[:, None].expand(rows, K)
    last = torch.full((N,), -1, dtype=torch.int64, device=dev)
    last.scatter_reduce_(0, gl.view(-1), torch.where(shared, row, -1).reshape(-1), "amax")
    keeps = shared & (inside[gl] == refs[gl]) & (last[gl] == row)
    need = (wanted & (g < 0)) | (shared & ~keeps)
    free = refs == 0
    order = torch.cumsum(need.view(-1).to(torch.int64), 0).view(rows, K) - 1
    total, have = need.sum(), free.sum()
    lowest = torch.argsort(free.to(torch.int8), descending=True, stable=True)
    enough = total <= have
    need &= enough
    fresh = lowest[order.clamp(min=0, max=N - 1)]
    refs.index_add_(0, gl.view(-1), -(need & shared).to(torch.int32).view(-1))
    refs.index_add_(0, fresh.view(-1), need.to(torch.int32).view(-1))
    partial = need & shared & (p * page < start)
    s["copy_src"].copy_(torch.where(partial, g.long(), -1).amax(1))
    s["copy_dst"].copy_(torch.where(partial, fresh, -1).amax(1))
    s["missing"].copy_((total - have).clamp(min=0))
    wide = torch.cat([table, table.new_zeros(rows, 1)], 1)
    wide.scatter_(1, torch.where(need, p, cap), fresh.to(torch.int32))
    table = wide[:, :cap].contiguous()
    _plain_copy(s, s["copy_src"], s["copy_dst"])
    return _pages(s, table, refs) | {"copy_src": s["copy_src"], "copy_dst": s["copy_dst"], "missing": s["missing"]}


def _plain_compact(s):
    case = s["case"]
    page, first = case["page"], case["first"]
    table, refs = s["table"].clone(), s["refs"].clone()
    N, cap = refs.numel(), table.shape[1]
    p = torch.arange(cap, device=table.device) * page
    keep = s["keep"][:, None]
    gone = (keep >= 0) & (p >= keep)
    if s["begin"] is not None:
        gone |= (p >= first) & (p + page <= s["begin"][:, None])
    gone &= table >= 0
    refs.index_add_(0, table.clamp(min=0).view(-1).long(), -gone.to(torch.int32).view(-1))
    table = torch.where(gone, -1, table)
    used = refs > 0
    high = torch.argsort(used.flip(0).to(torch.int8), descending=True, stable=True)
    high = N - 1 - high                                     # used pages, the highest first
    low = torch.argsort((~used).to(torch.int8), descending=True, stable=True)
    i = torch.arange(N, device=table.device)
    pairs = (i < used.sum()) & (i < N - used.sum()) & (low < high)
    s["move_src"].copy_(torch.where(pairs, high, -1))
    s["move_dst"].copy_(torch.where(pairs, low, -1))
    s["count"].copy_(pairs.sum())
    to = torch.arange(N + 1, device=table.device)
    to[torch.where(pairs, high, N)] = torch.where(pairs, low, N)
    table = torch.where(table >= 0, to[table.clamp(min=0).long()].to(torch.int32), table)
    moved = torch.where(pairs, refs[high], 0)
    refs = refs.index_add(0, high, -moved).index_add(0, low, moved)
    _plain_copy(s, s["move_src"], s["move_dst"])
    return _pages(s, table, refs) | {"move_src": s["move_src"], "move_dst": s["move_dst"], "count": s["count"]}


def run(state):
    if own:
        return _run_own(state)
    return {"attend": _plain_attend, "append": _plain_append, "fork": _plain_fork,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- 64 bits
def _values(codes):
    """The numbers that e4m3 codes stand for, from the format: 1 sign bit, 4 exponent bits (bias 7), 3 fraction bits."""
    c = torch.arange(256, dtype=torch.float64)
    e, f = torch.div(c % 128, 8, rounding_mode="floor"), c % 8
    mag = torch.where(e > 0, (1 + f / 8) * torch.pow(2.0, e - 7), f / 8 * 2.0 ** -6)
    mag[127] = mag[255] = math.nan
    return torch.where(c >= 128, -mag, mag).to(codes.device)[codes.long()]


def _nearest(y):
    """The nearest number that e4m3 has to each y, |y| <= 448, ties to the even one."""
    step = ((torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].long() + 1023 - 4) << 52).view(torch.float64)
    return torch.round(y / step) * step


def _next_power(x):
    """The smallest power of two that is not below x, and not below 2^-126."""
    f, e = torch.frexp(x.clamp(min=2.0 ** -126))
    return ((e.long() - (f == 0.5).long() + 1023) << 52).view(torch.float64)


def exact(case, seed):
    if case["op"] in ("fork", "compact"):
        return None                                         # page numbers and copied bytes
    s = prepare(case, seed)
    start, new = _lens(case)
    page, Hkv = case["page"], case["Hkv"]
    if case["op"] == "append":
        got = {}
        for name in ("k", "v"):
            store, scale = _values(s[name]), s[name + "_scale"].double()
            x = s[name + "_new"].double()
            for b in range(case["B"]):
                for p in range(start[b] // page, -(-(start[b] + new[b]) // page)):
                    g = int(s["table"][b, p])
                    lo, hi = max(start[b], p * page), min(start[b] + new[b], (p + 1) * page)
                    rows = x[b, lo - start[b]:hi - start[b]].transpose(0, 1)         # [Hkv][tokens][D]
                    need = _next_power(rows.abs().amax((1, 2)) / 448)
                    a = lo - p * page
                    now = torch.maximum(need, scale[g]) if a else need
                    if a:
                        store[g, :, :a] = _nearest(store[g, :, :a] * (scale[g] / now)[:, None, None])
                    store[g, :, a:a + hi - lo] = _nearest(rows / now[:, None, None])
                    scale[g] = now
            got[name], got[name + "_scale"] = store, scale
        return got
    H, D, Tq = case["H"], case["D"], case["Tq"]
    G = H // Hkv
    out = torch.zeros(case["B"], Tq, H, D, dtype=torch.float64, device=s["q"].device)
    for b in range(case["B"]):
        end = start[b] + new[b]
        row = s["table"][b, :-(-end // page)].long()
        # the keys that any query of the sequence sees
        i = torch.arange(end, device=out.device)
        if case["window"]:
            i = i[(i < case["first"]) | (i > start[b] - case["window"])]
        i = i[row[i // page] >= 0]
        t = start[b] + torch.arange(new[b], device=out.device)
        hidden = i[None] > t[:, None]
        if case["window"]:
            hidden |= (i[None] <= t[:, None] - case["window"]) & (i[None] >= case["first"])
        at, slot = row[i // page], i % page
        for h in range(Hkv):
            k = _values(s["k"][at, h, slot]) * s["k_scale"][at, h, None].double()
            v = _values(s["v"][at, h, slot]) * s["v_scale"][at, h, None].double()
            for r in range(G):
                c = h * G + r
                z = s["q"][b, :new[b], c].double() @ k.T / math.sqrt(D)
                z = z.masked_fill(hidden, -math.inf)
                if case["sink"]:
                    z = torch.cat([z, s["sinks"][c].double().expand(new[b], 1)], 1)
                w = torch.softmax(z, 1)[:, :i.numel()].nan_to_num(0.0)
                out[b, :new[b], c] = w @ v
    return out
