"""Paged 8-bit cache on the GPU: every call against the 64-bit oracle."""

import numpy as np
import pytest
import torch

from long_context_sparse_csa_b200 import binding as C
from oracle import paged as O
from oracle.formats import e4m3_decode, e4m3_encode

pytestmark = pytest.mark.gpu
BAD_PAGE = 4


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    C.lib()
    C.csa_device_error(None)
    yield
    torch.cuda.synchronize()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Cache:
    """A pool with random contents on the host, and its copy on the device."""

    def __init__(self, rng, N, Hkv, page, D, spread=3):
        self.page, self.Hkv, self.D, self.N = page, Hkv, D, N
        self.k = e4m3_encode(np.clip(rng.standard_normal((N, Hkv, page, D)) * 100, -448, 448))
        self.v = e4m3_encode(np.clip(rng.standard_normal((N, Hkv, page, D)) * 100, -448, 448))
        self.ks = (2.0 ** rng.integers(-9, -9 + spread, (N, Hkv))).astype(np.float32)
        self.vs = (2.0 ** rng.integers(-9, -9 + spread, (N, Hkv))).astype(np.float32)

    def up(self):
        self.d = [_dev(x) for x in (self.k, self.v, self.ks, self.vs)]
        return C.make_page_pool(*self.d)

    def host(self):
        return [x.cpu().numpy() for x in self.d]


def _table(rng, B, cap, N, held):
    """Row b holds held[b] entries, distinct pages in random order."""
    ids = rng.permutation(N)[:sum(held)]
    table, at = np.full((B, cap), -1, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    refs = np.bincount(ids, minlength=N).astype(np.int32)
    return table, refs


def _tolerance(act, ref, weight, logit):
    """Bound on |out - ref|: the output's rounding (half a step: 2^-8 of a bf16 value, 2^-24 of a float32
    value); P rounded to 11 (22) bits; logits summed in float32 from exact products over at most 128 dims
    in 8 instructions (each truncating at most at 2^-23 of the largest partial sum, and three float32
    roundings after: below 2^-19 of sum |q k| in all), which moves numerator and denominator, each by
    that much relative to sum p |v|; exponentials off by 2^-22, twice; and sums over the keys, 2^-20."""
    half, p = (2.0 ** -8, 2.0 ** -11) if act == "bf16" else (2.0 ** -24, 2.0 ** -22)
    return half * np.abs(ref) + weight * (p + 2 * (2.0 ** -19 * logit + 2.0 ** -21) + 2.0 ** -20) + 1e-37


def _attend(cache, table, start, n_new, Tq, H, act="bf16", window=0, first=0, sinks=None, scale=0.0, rng=None, q=None,
            n_max=None, error=0, stream=None):
    B, D = table.shape[0], cache.D
    rng = rng or np.random.default_rng(9)
    if q is None:
        q = rng.standard_normal((B, Tq, H, D)) * 2
    dt = torch.float32 if act == "f32" else torch.bfloat16
    qd = torch.from_numpy(q).to(dt).cuda()
    q = qd.float().cpu().numpy().astype(np.float64)
    pool = cache.up()
    refs = torch.zeros(cache.N, dtype=torch.int32, device="cuda")
    td = _dev(table)
    T = C.make_page_table(td, refs, cache.page)
    G = C.make_gqa(H, cache.Hkv, D, window, first, act, scale)
    n_max = table.shape[1] * cache.page if n_max is None else n_max
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, Tq, n_max), dtype=torch.uint8, device="cuda")
    mark = -123.0
    out = torch.full((B, Tq, H, D), mark, dtype=dt, device="cuda")
    sd = _dev(np.asarray(start, np.int64))
    nd = None if n_new is None else _dev(np.asarray(n_new, np.int32))
    kd = None if sinks is None else _dev(sinks.astype(np.float32))
    C.csa_paged_attend(G, pool, T, qd, kd, sd, nd, Tq, n_max, out, ws)
    assert C.csa_device_error(ws) == error
    once = out.clone()
    C.csa_paged_attend(G, pool, T, qd, kd, sd, nd, Tq, n_max, out, ws)       # the workspace is ready for the next call
    assert C.csa_device_error(ws) == error
    assert torch.equal(once.view(torch.uint8), out.view(torch.uint8))
    ref, asked, weight, logit = O.attend(cache.k, cache.v, cache.ks, cache.vs, table, cache.page, q, start, n_new,
                                         n_max, window, first, sinks, scale or None)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(got[~asked] == mark)
    got, ref, tol = got[asked], ref[asked], _tolerance(act, ref, weight, logit)[asked]
    return got, ref, tol


def _close(got, ref, tol):
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (np.isnan(got).sum(), np.isnan(ref).sum())
    ok = ~np.isnan(ref)
    worst = (np.abs(got - ref)[ok] / tol[ok]).max() if ok.any() else 0.0
    assert worst <= 1, worst


# ----------------------------------------------------------------------------- attention
@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,D,page", [(1, 1, 64, 16), (8, 1, 128, 16), (6, 2, 128, 32), (32, 2, 64, 64),
                                          (16, 2, 128, 128), (24, 8, 64, 32)])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17], [300, 1, 64, 129], [1000, 2051]])
def test_decode(act, H, Hkv, D, page, lens):
    rng = np.random.default_rng(sum(lens) + H + page)
    B, cap = len(lens), -(-max(lens) // page) + 1
    held = [-(-n // page) for n in lens]
    cache = Cache(rng, sum(held) + 3, Hkv, page, D)
    table, _ = _table(rng, B, cap, cache.N, held)
    sinks = rng.standard_normal(H) * 2 if len(lens) % 2 else None
    _close(*_attend(cache, table, np.array(lens) - 1, None, 1, H, act, sinks=sinks, rng=rng))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,H,Hkv", [(2, 4, 2), (3, 8, 1), (7, 16, 1), (5, 6, 2), (40, 8, 4), (130, 3, 1), (65, 16, 1)])
@pytest.mark.parametrize("window,first", [(0, 0), (16, 0), (33, 4), (100, 70)])
def test_several_tokens(act, Tq, H, Hkv, window, first):
    rng = np.random.default_rng(Tq + H + window)
    D, page = (128, 32) if H % 8 else (64, 16)
    start = np.array([0, 37, 200, -1, 500])
    n_new = np.array([Tq, 1, Tq + 9, Tq, max(1, Tq - 2)])
    held = [-(-(s + min(n, Tq)) // page) if s >= 0 else 0 for s, n in zip(start, n_new)]
    cache = Cache(rng, sum(held) + 1, Hkv, page, D)
    table, _ = _table(rng, 5, max(held), cache.N, held)
    _close(*_attend(cache, table, start, n_new, Tq, H, act, window, first, rng=rng))


@pytest.mark.parametrize("Tq,H,Hkv,D", [(300, 8, 1, 128), (257, 4, 1, 64), (129, 2, 2, 128)])
@pytest.mark.parametrize("window,first", [(0, 0), (150, 5)])
def test_a_prompt_chunk(Tq, H, Hkv, D, window, first):
    rng = np.random.default_rng(Tq)
    page, start = 64, np.array([0, 411])
    held = [-(-(s + Tq) // page) for s in start]
    cache = Cache(rng, sum(held), Hkv, page, D)
    table, _ = _table(rng, 2, max(held), cache.N, held)
    sinks = rng.standard_normal(H)
    _close(*_attend(cache, table, start, None, Tq, H, "bf16", window, first, sinks, rng=rng))


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_negative_and_zero_token_counts_leave_rows_alone(act):
    rng = np.random.default_rng(3)
    cache = Cache(rng, 12, 2, 16, 64)
    table, _ = _table(rng, 4, 3, 12, [3, 3, 3, 3])
    got, ref, tol = _attend(cache, table, [5, 20, 40, 30], [0, -7, 2, 100], 4, 4, act, rng=rng)
    assert len(ref) == 6
    _close(got, ref, tol)


@pytest.mark.parametrize("Tq", [1, 4, 70])
def test_tokens_behind_n_max_are_left_alone(Tq):
    rng = np.random.default_rng(4)
    cache = Cache(rng, 24, 2, 16, 128)
    table, _ = _table(rng, 4, 6, 24, [6] * 4)
    got, ref, tol = _attend(cache, table, [10, 18, 19, 2 ** 62], None, Tq, 8, n_max=20, rng=rng)
    _close(got, ref, tol)


def test_no_position_at_all():
    rng = np.random.default_rng(5)
    cache = Cache(rng, 4, 1, 16, 64)
    table, _ = _table(rng, 1, 2, 4, [2])
    got, *_ = _attend(cache, table, [3], None, 1, 2, n_max=0, rng=rng)
    assert got.size == 0


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq", [1, 3, 80])
def test_missing_pages_are_not_seen(act, Tq):
    rng = np.random.default_rng(6)
    page = 16
    cache = Cache(rng, 60, 1, page, 64)
    table, _ = _table(rng, 3, 20, 60, [20, 20, 20])
    table[0, 3:7] = -1
    table[1, :] = -1                                        # nothing to see: zeros
    table[2, -1] = -5
    got, ref, tol = _attend(cache, table, [320 - Tq, 100, 320 - Tq], None, Tq, 4, act, rng=rng)
    assert np.all(got[Tq:2 * Tq] == 0)
    _close(got, ref, tol)


@pytest.mark.parametrize("Tq", [1, 3, 80])
def test_page_numbers_out_of_range_are_reported_and_not_seen(Tq):
    rng = np.random.default_rng(7)
    cache = Cache(rng, 20, 1, 16, 64)
    table, _ = _table(rng, 1, 20, 20, [20])
    table[0, 2], table[0, 9] = 20, 2 ** 31 - 1
    _close(*_attend(cache, table, [320 - Tq], None, Tq, 4, error=BAD_PAGE, rng=rng))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,H", [(1, 4), (4, 4), (40, 8), (140, 2)])
@pytest.mark.parametrize("window,first", [(0, 0), (40, 3)])
def test_bytes_that_no_query_sees_change_nothing(act, Tq, H, window, first):
    rng = np.random.default_rng(8)
    page, D = 16, 64
    total = 210 + Tq
    held = -(-total // page) + 2                            # two pages more than there are tokens
    cache = Cache(rng, held, 1, page, D)
    table, _ = _table(rng, 1, held, held, [held])
    pos = np.arange(held * page)
    unseen = pos >= total
    if window:
        unseen |= (pos <= 210 - window) & (pos >= first)
    g, slot = table[0, pos[unseen] // page], pos[unseen] % page
    cache.k[g, 0, slot] = 0x7F
    cache.v[g, 0, slot] = 0xFF
    got, ref, tol = _attend(cache, table, [210], None, Tq, H, act, window, first, rng=rng)
    assert not np.isnan(ref).any()
    _close(got, ref, tol)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,H", [(1, 4), (4, 4), (20, 4), (140, 2)])
@pytest.mark.parametrize("scale", [np.nan, np.inf, 0.0, -1.0, 2.0 ** 120, 2.0 ** -126])
def test_scales_that_no_query_sees_change_nothing(act, Tq, H, scale):
    """Pages behind the window or behind the sequence that lie in tiles which are read."""
    rng = np.random.default_rng(20)
    page, D, total = 16, 64, 330 + Tq
    held = -(-total // page) + 3
    cache = Cache(rng, held, 1, page, D)
    table, _ = _table(rng, 1, held, held, [held])
    pos = np.arange(held) * page
    hidden = ((pos + page - 1 <= 330 - 70) & (pos >= 5)) | (pos >= total)
    g = table[0, hidden]
    cache.ks[g], cache.vs[g], cache.k[g], cache.v[g] = scale, scale, 0x7F, 0x7F
    got, ref, tol = _attend(cache, table, [330], None, Tq, H, act, 70, 5, rng=rng)
    assert not np.isnan(ref).any()
    _close(got, ref, tol)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_nan_reaches_the_queries_that_see_it_and_no_other(act, where):
    rng = np.random.default_rng(10)
    page, D, Tq = 16, 128, 12
    cache = Cache(rng, 8, 1, page, D)
    table, _ = _table(rng, 1, 8, 8, [8])
    for pos in (105, 20):                                   # seen from token 5 on; by tokens 0..2 only (window 83)
        getattr(cache, where)[table[0, pos // page], 0, pos % page, 7] = 0x7F
    got, ref, tol = _attend(cache, table, [100], None, Tq, 4, act, window=83, rng=rng)
    see = np.array([j < 3 or j >= 5 for j in range(Tq)])
    assert np.isnan(got[see][..., 7]).all() and not np.isnan(got[~see]).any()
    assert (np.abs(got - ref)[~see] <= tol[~see]).all()


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,H", [(1, 4), (40, 8)])
def test_value_scales_far_apart(act, Tq, H):
    """Pages whose values differ by 2^200, and logits that make the small ones count."""
    rng = np.random.default_rng(11)
    page, D, n = 16, 64, 256
    cache = Cache(rng, 16, 1, page, D)
    table, _ = _table(rng, 1, 16, 16, [16])
    cache.vs[:] = 2.0 ** rng.integers(-110, 100, cache.vs.shape)
    got, ref, tol = _attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng)
    _close(got, ref, tol)
    # only small pages: the result is as small, and as accurate
    cache.vs[:] = 2.0 ** rng.integers(-110, -50, cache.vs.shape)
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng))
    # a large page that no query gives weight to (its keys point away from every query)
    cache.vs[:] = 2.0 ** -6
    cache.vs[table[0, 5]] = 2.0 ** 60
    cache.k[table[0, 5], 0] = e4m3_encode(np.full((page, D), -400.0))
    cache.ks[table[0, 5]] = 1.0
    q = np.abs(rng.standard_normal((1, Tq, H, D))) + 1
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng, q=q))


def _logit_pages(rng, page, D, logits, vscale, Hkv=1):
    """A pool in table order whose page p holds keys of logit (log2 units) about logits[p] for the query (c, 0, ...)
    of `_along`, and values of scale vscale[p]."""
    N = len(logits)
    cache = Cache(rng, N, Hkv, page, D)
    cache.ks[:] = 2.0 ** -3
    cache.k[:] = e4m3_encode(rng.integers(-1, 2, cache.k.shape) * 1.0)
    for p, z in enumerate(logits):
        cache.k[p, ..., 0] = e4m3_encode(np.full(cache.k[p, ..., 0].shape, np.round(z / 16) * 16.0))
    cache.vs[:] = np.asarray(vscale, np.float64)[:, None].astype(np.float32)
    return cache, np.arange(N, dtype=np.int32)[None]


def _along(rng, Tq, H, D):
    """Queries whose first channel turns a key's first code into as many log2 units (scale 2^-3, 1/sqrt(D))."""
    q = rng.standard_normal((1, Tq, H, D)) * 0.25
    q[..., 0] = 8 * np.sqrt(D) / np.log2(np.e)
    return q


@pytest.mark.parametrize("act,Tq,H", [("bf16", 1, 4), ("f32", 3, 4), ("bf16", 5, 4), ("bf16", 40, 8), ("bf16", 300, 1)])
@pytest.mark.parametrize("order", [[0, 1], [1, 0], [0, 1, 2], [1, 2, 0], [2, 1, 0, 1], [2, 0, 2, 1, 2], [3, 1, 2], [2, 3, 2], [3, 2],
                                   [2, 4, 5], [0, 4, 1], [4, 3, 5, 0]])
@pytest.mark.parametrize("repeat", [24, 400])
def test_large_logits_on_pages_of_small_values(act, Tq, H, order, repeat):
    """The largest logits far above the others, on pages whose values are far below: the denominator's maximum has to
    follow the logits although the weighted values' maximum stays.  24 pages are a few tiles, 400 are more than a
    CTA's part."""
    rng = np.random.default_rng(len(order) + repeat)
    page, D = 16, 64
    kinds = {0: (0, 2.0 ** 100), 1: (160, 2.0 ** -110), 2: (0, 2.0 ** -8), 3: (144, 2.0 ** -126), 4: (320, 2.0 ** -100),
             5: (416, 2.0 ** -60)}
    pages = [kinds[i] for i in order for _ in range(repeat // len(order))]
    cache, table = _logit_pages(rng, page, D, [z for z, _ in pages], [s for _, s in pages])
    zero = np.array([z == 144 for z, _ in pages])
    cache.v[zero] = 0                                       # as an append of zeros leaves a page
    n = len(pages) * page
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng, q=_along(rng, Tq, H, D)))


@pytest.mark.parametrize("act,Tq,H", [("bf16", 1, 4), ("f32", 3, 4), ("bf16", 40, 8), ("bf16", 300, 1)])
@pytest.mark.parametrize("pages", [8, 300])
def test_sinks_far_above_logits_whose_values_are_large(act, Tq, H, pages):
    """Weights of 2^-140 and less beside the sink's, on pages whose scale makes their sum an ordinary number."""
    rng = np.random.default_rng(pages)
    cache, table = _logit_pages(rng, 16, 64, [0, 16] * (pages // 2), [2.0 ** 100, 2.0 ** 90] * (pages // 2))
    sinks = np.array([97.0, 104.0, 111.0, 132.0] * 2)[:H]
    n = 16 * pages
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, sinks=sinks, rng=rng, q=_along(rng, Tq, H, 64)))


@pytest.mark.parametrize("act,Tq,H", [("bf16", 1, 4), ("f32", 3, 4), ("bf16", 40, 8), ("bf16", 300, 1)])
@pytest.mark.parametrize("n", [300, 6400])
def test_value_scales_at_the_lower_end_keep_their_digits(act, Tq, H, n):
    """Outputs near 2^-118 are ordinary numbers of their type: the bound is the usual one, without its constant but
    for half of the type's smallest step (2^-134 for bf16, 2^-150 for float32) and one of float32."""
    rng = np.random.default_rng(n)
    N = -(-n // 16)
    cache = Cache(rng, N, 1, 16, 64)
    table, _ = _table(rng, 1, N, N, [N])
    cache.vs[:] = 2.0 ** rng.integers(-126, -124, cache.vs.shape)
    got, ref, tol = _attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng)
    _close(got, ref, tol - 1e-37 + 2.0 ** -149 + (2.0 ** -134 if act == "bf16" else 2.0 ** -150))


@pytest.mark.parametrize("act,Tq,H", [("bf16", 1, 4), ("bf16", 4, 4), ("f32", 3, 4), ("bf16", 40, 8), ("bf16", 300, 1)])
@pytest.mark.parametrize("down", [4, 12, 20, 30, 45])
def test_a_page_of_large_values_in_one_channel(act, Tq, H, down):
    """What is rounded is probability times value scale (w), so that a page whose values are large in one channel takes
    digits from the others' keys in all channels: 11 bits (22 for float32) down to 2^-18 (2^-17) of the largest w, half
    of 2^-29 (2^-40) of the largest w below that."""
    rng = np.random.default_rng(down)
    page, D, N = 16, 64, 24
    cache = Cache(rng, N, 1, page, D, spread=1)
    cache.k[:] = e4m3_encode(rng.integers(-1, 2, cache.k.shape) * 1.0)
    cache.vs[:] = 2.0 ** -down
    cache.vs[1::7] = 1.0
    cache.v[1::7, ..., 1:] = 0
    table, n = np.arange(N, dtype=np.int32)[None], N * page
    q = rng.standard_normal((1, Tq, H, D)) * 4
    got, ref, tol = _attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng, q=q)
    top, low = cache.vs.max(), 2.0 ** -30 if act == "bf16" else 2.0 ** -41
    Q = torch.from_numpy(q).to(torch.float32 if act == "f32" else torch.bfloat16).double().numpy()[0]
    K = e4m3_decode(cache.k[:, 0]).reshape(n, D) * np.repeat(cache.ks[:, 0], page)[:, None].astype(np.float64)
    codes = np.abs(e4m3_decode(cache.v[:, 0])).reshape(n, D)
    for j in range(Tq):
        seen = n - Tq + j + 1
        z = Q[j] @ K[:seen].T / np.sqrt(D)
        p = np.exp(z - z.max(1, keepdims=True))
        w = p / p.sum(1, keepdims=True) * np.repeat(cache.vs[:, 0], page)[:seen]
        assert (w.max(1) <= top).all()
        tol[j] += low * w.max(1)[:, None] * codes[:seen].sum(0)
    _close(got, ref, tol)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,H", [(1, 4), (40, 8)])
def test_key_scales_and_queries_far_from_one(act, Tq, H):
    rng = np.random.default_rng(12)
    page, D, n = 32, 128, 300
    cache = Cache(rng, 10, 1, page, D)
    table, _ = _table(rng, 1, 10, 10, [10])
    cache.ks[:] *= 2.0 ** 60
    q = rng.standard_normal((1, Tq, H, D)) * 2.0 ** -60
    q[..., 0] *= 2.0 ** -30                                 # small values of a row beside large ones
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng, q=q))
    cache.ks[:] *= 2.0 ** -120
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng, q=q * 2.0 ** 120))
    _close(*_attend(cache, table, [n - Tq], None, Tq, H, act, rng=rng, q=q * 0))


def test_sinks_far_above_and_below_the_logits():
    rng = np.random.default_rng(13)
    cache = Cache(rng, 8, 1, 16, 64)
    table, _ = _table(rng, 1, 8, 8, [8])
    sinks = np.array([-np.inf, -1e4, 30.0, 80.0])
    _close(*_attend(cache, table, [120], None, 1, 4, "f32", sinks=sinks, rng=rng))


def test_strided_queries_and_other_scale():
    rng = np.random.default_rng(14)
    B, Tq, H, Hkv, D, page = 3, 5, 8, 2, 64, 16
    cache = Cache(rng, 12, Hkv, page, D)
    table, _ = _table(rng, B, 4, 12, [4] * 3)
    fused = torch.randn(B, Tq, H + 2 * Hkv, D, device="cuda").bfloat16()
    q, k_new, v_new = fused[:, :, :H], fused[:, :, H:H + Hkv], fused[:, :, H + Hkv:]
    pool, start = cache.up(), torch.tensor([30, 0, 59], device="cuda")
    refs = torch.zeros(12, dtype=torch.int32, device="cuda")
    T, G = C.make_page_table(_dev(table), refs, page), C.make_gqa(H, Hkv, D, softmax_scale=0.3)
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, Tq, 64), dtype=torch.uint8, device="cuda")
    out = torch.zeros(B, Tq, H, D, dtype=torch.bfloat16, device="cuda")
    C.csa_paged_append(G, pool, T, k_new, v_new, start, None, Tq)
    C.csa_paged_attend(G, pool, T, q, None, start, None, Tq, 64, out, ws)
    assert C.csa_device_error(ws) == 0
    h = lambda x: x.float().cpu().numpy().astype(np.float64)  # noqa: E731
    st = O.append(cache.k, cache.v, cache.ks, cache.vs, table, refs.cpu().numpy(), page, h(k_new), h(v_new),
                  start.cpu().numpy(), None)
    for a, b in zip(cache.host(), st):
        assert np.array_equal(a, b)
    ref, _, w, z = O.attend(*st[:4], table, page, h(q), start.cpu().numpy(), None, 64, scale=float(np.float32(0.3)))
    _close(h(out), ref, _tolerance("bf16", ref, w, z))


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,H", [(1, 4), (40, 8), (150, 2)])
@pytest.mark.parametrize("window,first", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 2 ** 31 - 1), (1, 0), (1, 1)])
def test_windows_and_first_tokens_at_the_ends_of_their_range(act, Tq, H, window, first):
    rng = np.random.default_rng(16)
    cache = Cache(rng, 30, 1, 16, 64)
    table, _ = _table(rng, 2, 15, 30, [15, 15])
    _close(*_attend(cache, table, [240 - Tq, 3], [Tq, Tq // 2 + 1], Tq, H, act, window, first, rng=rng))


@pytest.mark.parametrize("Tq,H,Hkv", [(17, 1, 1), (40, 3, 1), (100, 4, 2), (33, 9, 1)])
def test_row_blocks_with_few_rows_in_them(Tq, H, Hkv):
    """Query rows that leave warps of a 128- or 256-row block without any."""
    rng = np.random.default_rng(17)
    lens = [70, 300, 129, 1025]
    held = [-(-n // 32) for n in lens]
    cache = Cache(rng, sum(held), Hkv, 32, 128)
    table, _ = _table(rng, 4, max(held), cache.N, held)
    n_new = [min(n, Tq) for n in lens]
    _close(*_attend(cache, table, np.array(lens) - n_new, n_new, Tq, H, rng=rng))


def test_long_sequences_split_over_the_gpu():
    """Hundreds of CTAs share a segment; the oracle is taken over a few heads of the same keys."""
    rng = np.random.default_rng(15)
    page, n = 128, 150000
    N = -(-n // page)
    cache = Cache(rng, N, 1, page, 64)
    table, _ = _table(rng, 1, N, N, [N])
    for act, H in (("bf16", 3), ("f32", 2)):
        _close(*_attend(cache, table, [n - 1], None, 1, H, act, rng=rng))


@pytest.mark.parametrize("Tq,H,Hkv,D", [(7, 32, 4, 128), (20, 8, 4, 64), (33, 16, 2, 64)])
def test_ctas_with_several_short_segments(Tq, H, Hkv, D):
    """More segments than SMs, of odd and even numbers of key tiles, cut at any place."""
    rng = np.random.default_rng(Tq)
    B, page = 44, 32
    start = rng.integers(0, 1500, B)
    held = [-(-(s + Tq) // page) for s in start]
    cache = Cache(rng, sum(held), Hkv, page, D)
    table, _ = _table(rng, B, max(held), cache.N, held)
    _close(*_attend(cache, table, start, rng.integers(0, Tq + 1, B), Tq, H, rng=rng))


@pytest.mark.parametrize("act,Tq,H", [("bf16", 1, 4), ("bf16", 4, 4), ("f32", 1, 4), ("bf16", 20, 4), ("bf16", 300, 1)])
def test_the_join_leaves_out_entries_that_name_no_cta(act, Tq, H):
    """A first launch whose wait gave up can leave an earlier call's bytes where the join looks for the first and last
    CTA of a sequence.  What names CTAs is joined; what does not is left alone, nothing is read out of range."""
    rng = np.random.default_rng(18)
    page, D, n = 128, 64, 60000
    N = -(-n // page)
    cache = Cache(rng, N, 1, page, D)
    pool, dt = cache.up(), torch.float32 if act == "f32" else torch.bfloat16
    T, G = C.make_page_table(_dev(np.arange(N, dtype=np.int32)[None]), _ints(N, 0), page), C.make_gqa(H, 1, D, act_format=act)
    q = torch.randn(1, Tq, H, D, device="cuda").to(dt)
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, Tq, n), dtype=torch.uint8, device="cuda")
    start, want = torch.tensor([n - Tq], device="cuda"), torch.full_like(q, 7.0)
    C.csa_paged_attend(G, pool, T, q, None, start, None, Tq, n, want, ws)
    blocks = -(-Tq * H // 256) if Tq * H > 128 else 1
    entries = ws[256:256 + 8 * blocks].view(torch.int32).view(blocks, 2)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (entries[:, 0] >= 0).all() and (entries[:, 1] > entries[:, 0]).all() and (entries[:, 1] < sms).all()
    out = torch.full_like(q, 7.0)
    C.csa_debug_paged_join(G, T, None, start, None, Tq, n, out, ws)
    assert torch.equal(out, want)
    out.fill_(7.0)
    for bad in ((-1, 3), (-2 ** 31, 2 ** 31 - 1), (0, sms), (sms, sms + 1), (0x3F800000, 0x40000000), (5, 5), (9, 2)):
        entries[:] = torch.tensor(bad, dtype=torch.int32, device="cuda")
        C.csa_debug_paged_join(G, T, None, start, None, Tq, n, out, ws)
        assert (out == 7.0).all(), bad


@pytest.mark.parametrize("Hkv,D,window", [(8, 64, 0), (6, 128, 300)])
def test_parts_that_begin_at_every_place_of_the_ring(Hkv, D, window):
    """Blocks of 128 rows, where two groups take the key tiles in turns: CTAs with many parts of one to nine tiles, so
    that parts begin at every entry of the ring of looked-up tiles; called again and again, the results are the same."""
    rng = np.random.default_rng(Hkv)
    B, Tq, page = 42, 20, 32
    start = rng.integers(0, 9 * 128 - Tq, B)
    held = [-(-(s + Tq) // page) for s in start]
    cache = Cache(rng, sum(held), Hkv, page, D)
    table, _ = _table(rng, B, max(held), cache.N, held)
    _close(*_attend(cache, table, start, None, Tq, Hkv, window=window, rng=rng))
    T, G = C.make_page_table(_dev(table), _ints(cache.N, 0), page), C.make_gqa(Hkv, Hkv, D, window)
    pool, q, n_max = cache.up(), torch.randn(B, Tq, Hkv, D, device="cuda").bfloat16(), table.shape[1] * page
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, Tq, n_max), dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(50)]
    for out in outs:
        C.csa_paged_attend(G, pool, T, q, None, _dev(start), None, Tq, n_max, out, ws)
    assert C.csa_device_error(ws) == 0
    assert all(torch.equal(out, outs[0]) for out in outs)


@pytest.mark.parametrize("act,Tq,G,n,B", [("bf16", 1, 8, 1 << 23, 0), ("bf16", 17, 1, 1 << 21, 0), ("bf16", 200, 1, 1 << 20, 0),
                                          ("f32", 1, 3, 1 << 20, 0), ("bf16", 30, 3, 257 * 128, 0), ("bf16", 30, 3, 513 * 128, 0),
                                          ("bf16", 200, 1, 257 * 128, 0), ("bf16", 20, 2, 22000 * 128, 3),
                                          ("bf16", 300, 1, 11000 * 128, 3), ("bf16", 5, 2, 4800 * 128, 201), ("f32", 2, 2, 4800 * 128, 201)])
def test_long_sums_are_not_cut_off(act, Tq, G, n, B):
    """One sequence's keys under as many table rows as there are SMs (or B), so that a CTA has all of them: chains of sums
    as long as they get; sums in several pieces, the last of one tile, and pieces of parts that begin or end elsewhere.  Values of one sign make a cut-off sum visible.  The bound is the usual one, and 2^-11 of the sum
    for bf16's chains of at most 2,048 products, each of which may cut off 2^-22.  The first and last rows are checked
    in float64."""
    page, D = 128, 64
    N, B = n // page, B or torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n + Tq)
    f8 = torch.float8_e4m3fn
    k = (torch.randn(N, 1, page, D, generator=gen, device="cuda") * 60).clamp_(-448, 448).to(f8)
    v = (torch.rand(N, 1, page, D, generator=gen, device="cuda") * 300 + 100).to(f8)
    ks, vs = (torch.full((N, 1), 2.0 ** e, device="cuda") for e in (-9, -8))
    table = torch.arange(N, dtype=torch.int32, device="cuda").expand(B, N).contiguous()
    T, L = C.make_page_table(table, _ints(N, 0), page), C.make_gqa(G, 1, D, act_format=act)
    q = torch.randn(B, Tq, G, D, generator=gen, device="cuda").to(torch.float32 if act == "f32" else torch.bfloat16)
    start = torch.full((B,), n - Tq, device="cuda")
    ws = torch.zeros(C.csa_paged_workspace_size(L, T, Tq, n), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    C.csa_paged_attend(L, C.make_page_pool(k, v, ks, vs), T, q, None, start, None, Tq, n, out, ws)
    assert C.csa_device_error(ws) == 0
    K, V = k.view(n, D), v.view(n, D)
    step = 1 << 18
    for b, j in ((0, 0), (B - 1, Tq - 1)):
        Q, seen = q[b, j].double(), n - Tq + j + 1
        z = torch.cat([Q @ (K[i:i + step].double() * 2.0 ** -9).T for i in range(0, n, step)], 1)[:, :seen] / D ** 0.5
        logit = max(float((Q.abs() @ (K[i:i + step].double().abs() * 2.0 ** -9).T).max()) for i in range(0, n, step)) / D ** 0.5
        p = torch.softmax(z, 1)
        ref = sum(p[:, i:i + step] @ (V[i:min(i + step, seen)].double() * 2.0 ** -8) for i in range(0, seen, step)).cpu().numpy()
        tol = _tolerance(act, ref, ref, logit) + (2.0 ** -11 * ref if act == "bf16" else 0)
        _close(out[b, j].double().cpu().numpy(), ref, tol)


def test_offsets_behind_2_31_bytes():
    """A pool of more than 2^32 bytes: the pages in use are its last."""
    Hkv, page, D, N = 8, 128, 128, 36000
    dev = "cuda"
    if torch.cuda.get_device_properties(0).total_memory < 20 << 30:
        pytest.skip("needs 10 GB")
    k = torch.zeros(N, Hkv, page, D, dtype=torch.uint8, device=dev)
    v, sc = torch.zeros_like(k), torch.ones(N, Hkv, device=dev)
    pool, start = C.make_page_pool(k, v, sc, sc.clone()), torch.tensor([0], device=dev)
    table = torch.tensor([[N - 1, N - 3]], dtype=torch.int32, device=dev)
    refs = torch.zeros(N, dtype=torch.int32, device=dev)
    T, G = C.make_page_table(table, refs, page), C.make_gqa(8, Hkv, D)
    x = torch.randn(1, 200, Hkv, D, device=dev).bfloat16()
    C.csa_paged_append(G, pool, T, x, x, start, None, 200)
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, 1, 256), dtype=torch.uint8, device=dev)
    out = torch.zeros(1, 1, 8, D, dtype=torch.bfloat16, device=dev)
    C.csa_paged_attend(G, pool, T, x[:, :1], None, torch.tensor([199], device=dev), None, 1, 256, out, ws)
    move = torch.tensor([N - 1, N - 3], dtype=torch.int32, device=dev), torch.tensor([5, N - 2], dtype=torch.int32, device=dev)
    C.csa_pages_copy(G, pool, T, *move, None, 2)
    assert C.csa_device_error(ws) == 0
    assert torch.equal(k[5], k[N - 1]) and torch.equal(v[N - 2], v[N - 3]) and k[N - 1].any()
    small = Cache(np.random.default_rng(0), 2, Hkv, page, D)
    small.k, small.v = k[[N - 1, N - 3]].cpu().numpy(), v[[N - 1, N - 3]].cpu().numpy()
    pv = [p.cpu().numpy()[[N - 1, N - 3]] for p in pool.keep[2:]]
    ref, _, w, z = O.attend(small.k, small.v, *pv, np.array([[0, 1]]), page, x[:, :1].float().cpu().numpy(), [199], None, 256)
    _close(out.float().cpu().numpy(), ref, _tolerance("bf16", ref, w, z))


@pytest.mark.parametrize("H,D", [(8, 128), (16, 64)])
def test_offsets_behind_2_31_bytes_of_many_rows(H, D):
    """The same for blocks of many query rows: 200 tokens written to and read from the last pages of such a pool."""
    Hkv, page, Tq = 8, 128, 200
    N, dev = 36000 * 128 // D, "cuda"
    if torch.cuda.get_device_properties(0).total_memory < 20 << 30:
        pytest.skip("needs 10 GB")
    k = torch.zeros(N, Hkv, page, D, dtype=torch.uint8, device=dev)
    v, sc = torch.zeros_like(k), torch.ones(N, Hkv, device=dev)
    pool, start = C.make_page_pool(k, v, sc, sc.clone()), torch.tensor([0], device=dev)
    table = torch.tensor([[N - 1, N - 3]], dtype=torch.int32, device=dev)
    T, G = C.make_page_table(table, torch.zeros(N, dtype=torch.int32, device=dev), page), C.make_gqa(H, Hkv, D)
    x, q = (torch.randn(1, Tq, h, D, device=dev).bfloat16() for h in (Hkv, H))
    C.csa_paged_append(G, pool, T, x, x, start, None, Tq)
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, Tq, 256), dtype=torch.uint8, device=dev)
    out = torch.zeros_like(q)
    C.csa_paged_attend(G, pool, T, q, None, start, None, Tq, 256, out, ws)
    assert C.csa_device_error(ws) == 0 and C.csa_device_error(None) == 0
    at = [N - 1, N - 3]
    ref, _, w, z = O.attend(k[at].cpu().numpy(), v[at].cpu().numpy(), *[p.cpu().numpy()[at] for p in pool.keep[2:]],
                            np.array([[0, 1]]), page, q.float().cpu().numpy(), [0], None, 256)
    _close(out.float().cpu().numpy(), ref, _tolerance("bf16", ref, w, z))


# ----------------------------------------------------------------------------- append
def _append(cache, table, refs, x, y, start, n_new, act):
    dt = torch.float32 if act == "f32" else torch.bfloat16
    xd, yd = torch.from_numpy(x).to(dt).cuda(), torch.from_numpy(y).to(dt).cuda()
    pool, rd = cache.up(), _dev(refs)
    T, G = C.make_page_table(_dev(table), rd, cache.page), C.make_gqa(cache.Hkv, cache.Hkv, cache.D, act_format=act)
    sd, nd = _dev(np.asarray(start, np.int64)), None if n_new is None else _dev(np.asarray(n_new, np.int32))
    C.csa_paged_append(G, pool, T, xd, yd, sd, nd, x.shape[1])
    ref = O.append(cache.k, cache.v, cache.ks, cache.vs, table, refs, cache.page, xd.float().cpu().numpy(),
                   yd.float().cpu().numpy(), start, n_new)
    assert C.csa_device_error(None) == (BAD_PAGE if ref[4] else 0)
    for a, b in zip(cache.host(), ref):
        assert np.array_equal(a, b), np.argwhere(a != b)[:4]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (2, 128, 16), (3, 64, 32), (2, 128, 64), (1, 128, 128)])
@pytest.mark.parametrize("Tq", [1, 2, 17, 200])
def test_append(act, Hkv, D, page, Tq):
    rng = np.random.default_rng(Tq + page)
    start = np.array([0, 5, page - 1, page, -3, 3 * page + 7])
    n_new = np.array([Tq, max(1, Tq // 2), Tq + 3, 0, Tq, Tq])
    held = [-(-(max(s, 0) + Tq) // page) for s in start]
    cache = Cache(rng, sum(held) + 2, Hkv, page, D)
    table, refs = _table(rng, 6, max(held), cache.N, held)
    shape = (6, Tq, Hkv, D)
    x = rng.standard_normal(shape) * np.exp(rng.uniform(-8, 8, (6, 1, Hkv, 1)))
    y = rng.standard_normal(shape) * np.exp(rng.uniform(-8, 8, (6, Tq, 1, 1)))
    _append(cache, table, refs, x, y, start, n_new, act)


@pytest.mark.parametrize("act", ["bf16", "f32"])
def test_append_of_zeros_infinities_nan_and_the_type_s_ends(act):
    rng = np.random.default_rng(1)
    page, D, Tq = 16, 64, 16
    cache = Cache(rng, 8, 1, page, D)
    table, refs = _table(rng, 8, 1, 8, [1] * 8)
    x = rng.standard_normal((8, Tq, 1, D))
    x[0] = 0
    x[1, 3, 0, 5], x[1, 4, 0, 6], x[1, 9, 0, 7] = np.inf, -np.inf, np.nan
    x[2] = np.nan
    x[3, :, 0] = 3.0e38
    x[4, :, 0] = 1e-38 * rng.standard_normal((Tq, D))
    x[5, 0, 0, 0], x[5, 0, 0, 1:] = 448.0, 447.0
    x[6, 0, 0, 0] = 448.0 * 2 + 4
    x[7] = -np.inf
    _append(cache, table, refs, x, -x, [0] * 8, None, act)


def test_append_leaves_out_tokens_without_a_page_of_their_own():
    rng = np.random.default_rng(2)
    page, D = 16, 64
    cache = Cache(rng, 12, 2, page, D)
    table, refs = _table(rng, 6, 3, 12, [2] * 6)
    table[1, 1], table[2, 0] = -1, 12
    refs[table[3, 1]] = 2
    x = rng.standard_normal((6, 20, 2, D))
    _append(cache, table, refs, x, x, [3, 3, 3, 3, 40, 2 ** 62], None, "bf16")
    # without counts a shared page is the caller's business
    pool, T = cache.up(), C.make_page_table(_dev(table), _dev(refs), page)
    T.refs = None
    xd = torch.from_numpy(x).bfloat16().cuda()
    C.csa_paged_append(C.make_gqa(2, 2, D), pool, T, xd, xd, _dev(np.array([-1, -1, -1, 3, -1, -1])), None, 20)
    assert C.csa_device_error(None) == 0
    ref = O.append(cache.k, cache.v, cache.ks, cache.vs, table[3:4], np.ones_like(refs), page,
                   xd[3:4].float().cpu().numpy(), xd[3:4].float().cpu().numpy(), [3], None)
    for a, b in zip(cache.host(), ref):
        assert np.array_equal(a, b)


def test_errors_of_the_paged_calls_reach_nobody_else():
    """A token without a page is reported where no workspace is asked about, and by its own status; the check of another
    call's workspace, and the decode step that checks its own, neither report nor clear it."""
    from csa_synth import decode_inputs, get_workload
    from long_context_sparse_csa_b200.state import LayerState

    td, rd, T = _book(np.full((1, 2), -1, np.int32), np.zeros(4, np.int32), 16)
    cache = Cache(np.random.default_rng(0), 4, 1, 16, 64)
    pool, x = cache.up(), torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    bad = lambda: C.csa_paged_append(C.make_gqa(1, 1, 64), pool, T, x, x, _dev(np.array([3])), None, 1)  # noqa: E731
    bad()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert C.csa_device_error(ws) == 0
    wl = get_workload("csa_decode_tiny_2k")
    d = decode_inputs(wl)
    st, L = LayerState.from_arrays(wl.layers[0], wl.B, d), wl.layers[0]
    args = [_dev(d[k]) for k in ("q", "idx_q", "idx_q_scale", "head_w", "x_new", "g_new", "t")]
    out = torch.zeros((1, L.H, L.D), dtype=torch.float32, device="cuda")
    topk = torch.zeros((1, L.top_k), dtype=torch.int32, device="cuda")
    assert C.csa_decode_step_scratch(st.L, st.cache(), st.params(), *args, out, topk, read_device_error=True) == 0
    assert C.csa_device_error(None) == BAD_PAGE and C.csa_device_error(None) == 0
    bad()
    assert C.lib().csa_device_error(None, 0, C._stream(), None) == 6
    ws.view(torch.int32)[0] = BAD_PAGE | 1
    assert C.lib().csa_device_error(C.ptr(ws), 256, C._stream(), None) == 5


# ----------------------------------------------------------------------------- bookkeeping
def _book(table, refs, page):
    td, rd = _dev(table), _dev(refs)
    return td, rd, C.make_page_table(td, rd, page)


def _ints(n, fill=77):
    return torch.full((n,), fill, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,cap,n", [(2, 1, 1), (40, 300, 17), (300, 20, 150)])
def test_fork(B, cap, n):
    rng = np.random.default_rng(B)
    N = B * cap + 5
    table, refs = _table(rng, B, cap, N, [int(rng.integers(0, cap + 1)) for _ in range(B)])
    rows = rng.permutation(B)
    src, dst = rows[rng.integers(0, B - n, n)] if B > n else rows[:n], rows[B - n:]
    td, rd, T = _book(table, refs, 16)
    C.csa_pages_fork(T, _dev(src.astype(np.int32)), _dev(dst.astype(np.int32)), n)
    assert C.csa_device_error(None) == 0
    t, r, err = O.fork(table, refs, src, dst)
    assert not err and np.array_equal(td.cpu().numpy(), t) and np.array_equal(rd.cpu().numpy(), r)
    C.csa_pages_fork(T, _dev(src.astype(np.int32)), _dev(dst.astype(np.int32)), n)       # once more: nothing changes
    assert np.array_equal(td.cpu().numpy(), t) and np.array_equal(rd.cpu().numpy(), r)


@pytest.mark.parametrize("src,dst,bad", [([-1], [-1], False), ([0], [0], True), ([9], [1], True), ([0], [-1], True),
                                         ([0, 2], [1, 1], True), ([0, 1], [1, 2], True), ([0, 0, -1], [1, 2, -1], False),
                                         ([-1, 0], [3, 3], True)])
def test_fork_pairs_that_are_left_out(src, dst, bad):
    rng = np.random.default_rng(1)
    table, refs = _table(rng, 4, 3, 12, [3, 1, 2, 0])
    td, rd, T = _book(table, refs, 16)
    C.csa_pages_fork(T, _dev(np.array(src, np.int32)), _dev(np.array(dst, np.int32)), len(src))
    t, r, err = O.fork(table, refs, src, dst)
    assert err == bad and C.csa_device_error(None) == (BAD_PAGE if bad else 0)
    assert np.array_equal(td.cpu().numpy(), t) and np.array_equal(rd.cpu().numpy(), r)


def test_fork_and_free_of_page_numbers_out_of_range():
    table = np.array([[0, 9, -1], [1, 2, 7]], np.int32)
    refs = np.array([1, 1, 1], np.int32)
    td, rd, T = _book(table, refs, 16)
    C.csa_pages_fork(T, _ints(1, 0), _ints(1, 1), 1)
    assert C.csa_device_error(None) == BAD_PAGE
    assert td.cpu().tolist() == [[0, 9, -1], [0, -1, -1]] and rd.cpu().tolist() == [2, 0, 0]
    C.csa_pages_free(T, _dev(np.array([0, 0])), None, 0)
    assert C.csa_device_error(None) == BAD_PAGE
    assert td.cpu().tolist() == [[-1] * 3] * 2 and rd.cpu().tolist() == [0, 0, 0]
    td.copy_(_dev(np.array([[1, -1, -1], [1, -1, -1]], np.int32)))        # a page that nobody counted
    rd[1] = 1
    C.csa_pages_free(T, _dev(np.array([0, 0])), None, 0)
    assert C.csa_device_error(None) == BAD_PAGE and rd.cpu().tolist() == [0, 0, 0]


def _reserve(table, refs, page, start, n_new, Tq):
    td, rd, T = _book(table, refs, page)
    B = table.shape[0]
    src, dst, missing = _ints(B), _ints(B), _ints(1)
    C.csa_pages_reserve(T, _dev(np.asarray(start, np.int64)),
                        None if n_new is None else _dev(np.asarray(n_new, np.int32)), Tq, src, dst, missing)
    t, r, cs, cd, miss, err = O.reserve(table, refs, page, start, n_new, Tq)
    assert C.csa_device_error(None) == (BAD_PAGE if err else 0)
    assert int(missing) == miss
    for a, b in ((td, t), (rd, r), (src, cs), (dst, cd)):
        assert np.array_equal(a.cpu().numpy(), b), np.argwhere(a.cpu().numpy() != b)[:5]
    return t, r


@pytest.mark.parametrize("B,Tq,page,N", [(1, 1, 16, 5), (7, 1, 16, 60), (300, 5, 16, 3000), (40, 200, 32, 2000),
                                         (3, 3000, 16, 700), (1200, 2, 128, 9001)])
@pytest.mark.parametrize("seed", [0, 1])
def test_reserve(B, Tq, page, N, seed):
    rng = np.random.default_rng(seed)
    cap = -(-(Tq + 100) // page) + 2
    held = [int(x) for x in rng.integers(0, min(cap, max(1, N // (2 * B))) + 1, B)]
    table, refs = _table(rng, B, cap, N, held)
    for i in range(B // 3):                                 # groups of rows that share their pages
        s, d = rng.integers(0, B, 2)
        if s != d:
            table, refs, _ = O.fork(table, refs, [s], [d])
            held[d] = held[s]
    start = [max(0, h * page - int(rng.integers(0, page + 1))) if h else 0 for h in held]
    start = [s if s + Tq <= cap * page and rng.random() < 0.9 else -1 for s in start]
    n_new = rng.integers(-1, Tq + 2, B)
    _reserve(table, refs, page, start, n_new, Tq)
    _reserve(table, refs, page, start, None, Tq)


def test_reserve_too_few_pages_changes_nothing():
    rng = np.random.default_rng(3)
    table, refs = _table(rng, 6, 4, 8, [1, 1, 1, 1, 1, 1])
    table, refs, _ = O.fork(table, refs, [0, 2], [1, 3])
    t, r = _reserve(table, refs, 16, [5, 5, 5, 5, 16, 15], None, 40)
    assert np.array_equal(t, table) and np.array_equal(r, refs)


@pytest.mark.parametrize("rows", [[0, 1], [0, 1, 2], [1, 2], [2, 1]])
def test_reserve_the_highest_row_keeps_a_page_that_all_its_holders_write(rows):
    table, refs = np.array([[3, -1], [3, -1], [3, -1], [4, -1]], np.int32), np.array([0, 0, 0, 3, 1, 0], np.int32)
    start = [7 if b in rows else -1 for b in range(4)]
    _reserve(table, refs, 16, start, None, 2)
    _reserve(table, refs, 16, start, None, 20)


def test_reserve_rows_that_end_and_pages_out_of_range():
    table = np.array([[0, 1], [2, 99], [3, -1], [-7, -1]], np.int32)
    refs = np.array([1, 1, 1, 1, 0, 0, 0, 0], np.int32)
    _reserve(table, refs, 16, [20, 15, 15, 2], None, 2)
    _reserve(table, refs, 16, [31, 2 ** 62, 15, -2 ** 62], None, 2)


def test_reserve_more_pages_than_one_round_of_the_list_holds():
    B, Tq, page = 40, 30000, 16
    cap = -(-Tq // page) + 1
    table = np.full((B, cap), -1, np.int32)
    refs = np.zeros(B * cap + 1000, np.int32)
    refs[::7] = 1
    refs = np.concatenate([refs, np.zeros(len(refs) // 5, np.int32)])
    _reserve(table, refs, page, np.arange(B) % 5, None, Tq)


@pytest.mark.parametrize("B,cap,page", [(1, 1, 16), (5, 40, 16), (700, 33, 64)])
def test_free(B, cap, page):
    rng = np.random.default_rng(B)
    N = B * cap
    table, refs = _table(rng, B, cap, N, [int(rng.integers(0, cap + 1)) for _ in range(B)])
    if B > 2:
        table, refs, _ = O.fork(table, refs, [0], [1])
    keep = np.where(rng.random(B) < 0.5, rng.integers(0, cap * page + 1, B), -1)
    begin = rng.integers(-1, cap * page, B)
    for k, w, first in ((keep, None, 0), (None, begin, 0), (keep, begin, 5), (None, begin, 2 * page)):
        td, rd, T = _book(table, refs, page)
        C.csa_pages_free(T, None if k is None else _dev(k), None if w is None else _dev(w), first)
        t, r = O.free(table, refs, page, k, w, first)
        assert C.csa_device_error(None) == 0
        assert np.array_equal(td.cpu().numpy(), t) and np.array_equal(rd.cpu().numpy(), r)


@pytest.mark.parametrize("N,B,cap", [(1, 1, 1), (7, 2, 3), (33, 3, 5), (5000, 40, 60), (70001, 300, 200)])
@pytest.mark.parametrize("fill", [0.0, 0.1, 0.6, 1.0])
def test_compact(N, B, cap, fill):
    rng = np.random.default_rng(N)
    held = [min(cap, int(fill * N / B)) for _ in range(B)]
    table, refs = _table(rng, B, cap, N, held)
    if B > 2:
        table, refs, _ = O.fork(table, refs, [0], [2])
    for most in sorted({0, 1, N // 3, N}):
        td, rd, T = _book(table, refs, 16)
        src, dst, count = _ints(max(most, 1)), _ints(max(most, 1)), _ints(1)
        C.csa_pages_compact(T, most, src if most else None, dst if most else None, count)
        t, r, ms, md, n = O.compact(table, refs, most)
        assert C.csa_device_error(None) == 0 and int(count) == n
        for a, b in ((td, t), (rd, r), (src[:most], ms), (dst[:most], md)):
            assert np.array_equal(a.cpu().numpy(), b)


def test_compact_reports_page_numbers_that_nobody_counted():
    table, refs = np.array([[5, 9], [3, -1]], np.int32), np.array([0, 0, 0, 0, 0, 1], np.int32)
    td, rd, T = _book(table, refs, 16)
    src, dst, count = _ints(6), _ints(6), _ints(1)
    C.csa_pages_compact(T, 6, src, dst, count)
    assert C.csa_device_error(None) == BAD_PAGE
    assert td.cpu().tolist() == [[0, 9], [3, -1]] and rd.cpu().tolist() == [1, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("Hkv,D,page", [(1, 64, 16), (3, 128, 16), (8, 128, 64), (2, 64, 128)])
def test_copy(Hkv, D, page):
    rng = np.random.default_rng(Hkv)
    N = 40
    cache = Cache(rng, N, Hkv, page, D)
    T, G = C.make_page_table(_dev(np.zeros((1, 1), np.int32)), _ints(N, 0), page), C.make_gqa(Hkv, Hkv, D)
    src = np.array([3, -1, 7, 39, 5, 6, 8], np.int32)
    dst = np.array([10, 11, -1, 12, 13, 14, 15], np.int32)
    for count in (None, 0, 5, 100):
        pool = cache.up()
        C.csa_pages_copy(G, pool, T, _dev(src), _dev(dst), None if count is None else _ints(1, count), 6)
        assert C.csa_device_error(None) == 0
        want = [x.copy() for x in (cache.k, cache.v, cache.ks, cache.vs)]
        for i in range(6 if count is None else min(count, 6)):
            if src[i] >= 0 and dst[i] >= 0:
                for w in want:
                    w[dst[i]] = w[src[i]]
        for a, b in zip(cache.host(), want):
            assert np.array_equal(a, b)
    pool = cache.up()
    C.csa_pages_copy(G, pool, T, _ints(1, N), _ints(1, 2), None, 1)
    C.csa_pages_copy(G, pool, T, _ints(1, 2), _ints(1, 2 ** 31 - 1), None, 1)
    assert C.csa_device_error(None) == BAD_PAGE
    assert np.array_equal(cache.host()[0], cache.k)


# ----------------------------------------------------------------------------- together
def _steps(B, Hkv, H, D, page, act, seed):
    """A prompt in two chunks, a fork, decode steps of both, an ended sequence, a compaction, more steps: yields
    the device's outputs beside the oracle's."""
    rng = np.random.default_rng(seed)
    N, cap, window, first = 60, 8, 50, 3
    cache = Cache(rng, N, Hkv, page, D)
    table, refs = np.full((B, cap), -1, np.int32), np.zeros(N, np.int32)
    pool = cache.up()
    td, rd, T = _book(table, refs, page)
    G = C.make_gqa(H, Hkv, D, window, first, act)
    dt = torch.float32 if act == "f32" else torch.bfloat16
    state = [cache.k, cache.v, cache.ks, cache.vs]
    src, dst, missing = _ints(B), _ints(B), _ints(1)
    ws = torch.zeros(max(C.csa_paged_workspace_size(G, T, q, cap * page) for q in (1, 40)), dtype=torch.uint8, device="cuda")

    def step(start, n_new, Tq):
        nonlocal table, refs, state
        x, y, q = (torch.from_numpy(rng.standard_normal((B, Tq, h, D))).to(dt).cuda() for h in (Hkv, Hkv, H))
        sd, nd = _dev(np.asarray(start, np.int64)), _dev(np.asarray(n_new, np.int32))
        out = torch.zeros(B, Tq, H, D, dtype=dt, device="cuda")
        C.csa_pages_reserve(T, sd, nd, Tq, src, dst, missing)
        C.csa_pages_copy(G, pool, T, src, dst, None, B)
        C.csa_paged_append(G, pool, T, x, y, sd, nd, Tq)
        C.csa_paged_attend(G, pool, T, q, None, sd, nd, Tq, cap * page, out, ws)
        assert C.csa_device_error(ws) == 0 and int(missing) == 0
        table, refs, cs, cd, _, _ = O.reserve(table, refs, page, start, n_new, Tq)
        for w in state:
            w[cd[cd >= 0]] = w[cs[cs >= 0]]
        h = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
        *state, err = O.append(*state, table, refs, page, h(x), h(y), start, n_new)
        assert not err
        ref, asked, w, z = O.attend(*state, table, page, h(q), start, n_new, cap * page, window, first)
        _close(h(out)[asked], ref[asked], _tolerance(act, ref, w, z)[asked])

    def same():
        assert np.array_equal(td.cpu().numpy(), table) and np.array_equal(rd.cpu().numpy(), refs)
        for a, b in zip(cache.host(), state):
            used = refs > 0
            assert np.array_equal(a[used], b[used])

    step([0, 0, -1, -1], [40, 23, 0, 0], 40)
    step([40, 23, -1, -1], [17, 40, 0, 0], 40)
    C.csa_pages_fork(T, _dev(np.array([0, 1], np.int32)), _dev(np.array([2, 3], np.int32)), 2)
    table, refs, _ = O.fork(table, refs, [0, 1], [2, 3])
    lens = np.array([57, 63, 57, 63])
    for i in range(4):
        step(lens, [1] * 4, 1)
        lens = lens + 1
        same()
    keep, begin = np.array([-1, 0, -1, -1]), lens + 1 - window
    C.csa_pages_free(T, _dev(keep), _dev(begin), first)
    table, refs = O.free(table, refs, page, keep, begin, first)
    move_src, move_dst, count = _ints(N), _ints(N), _ints(1)
    C.csa_pages_compact(T, N, move_src, move_dst, count)
    C.csa_pages_copy(G, pool, T, move_src, move_dst, count, N)
    table, refs, ms, md, n = O.compact(table, refs, N)
    for w in state:
        w[md[:n]] = w[ms[:n]]
    assert n > 0 and not refs[(refs > 0).sum():].any()
    same()
    lens[1] = -1
    for i in range(3):
        step(lens, [1, 0, 2, 3], 3)
        lens = lens + np.array([1, 0, 2, 3])
    same()


@pytest.mark.parametrize("act,Hkv,H,D,page", [("bf16", 2, 8, 128, 16), ("f32", 1, 3, 64, 16), ("bf16", 2, 4, 64, 32)])
def test_a_serving_run(act, Hkv, H, D, page):
    _steps(4, Hkv, H, D, page, act, seed=page)


def test_a_captured_step_follows_its_inputs():
    """Reserve, copy, append and attend in one CUDA graph: replayed as the sequence grows across pages."""
    rng = np.random.default_rng(5)
    B, Hkv, H, D, page, cap, N = 2, 1, 4, 64, 16, 4, 20
    cache = Cache(rng, N, Hkv, page, D)
    pool = cache.up()
    td, rd, T = _book(np.full((B, cap), -1, np.int32), np.zeros(N, np.int32), page)
    G = C.make_gqa(H, Hkv, D)
    start = torch.zeros(B, dtype=torch.int64, device="cuda")
    x, q = (torch.zeros(B, 1, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hkv, H))
    out = torch.zeros_like(q)
    src, dst, missing = _ints(B), _ints(B), _ints(1)
    ws = torch.zeros(C.csa_paged_workspace_size(G, T, 1, cap * page), dtype=torch.uint8, device="cuda")

    def call():
        C.csa_pages_reserve(T, start, None, 1, src, dst, missing)
        C.csa_pages_copy(G, pool, T, src, dst, None, B)
        C.csa_paged_append(G, pool, T, x, x, start, None, 1)
        C.csa_paged_attend(G, pool, T, q, None, start, None, 1, cap * page, out, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        start.fill_(-1)
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    table, refs, state = td.cpu().numpy().copy(), rd.cpu().numpy().copy(), [a.copy() for a in cache.host()]
    h = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    for i in range(40):
        start.copy_(torch.tensor([i, i // 2 if i % 2 == 0 else -1]))
        x.copy_(torch.randn_like(x))
        q.copy_(torch.randn_like(q))
        graph.replay()
        at = start.cpu().numpy()
        table, refs, *_ = O.reserve(table, refs, page, at, None, 1)
        *state, err = O.append(*state, table, refs, page, h(x), h(x), at, None)
        assert not err
        if i % 7 == 0 or i > 37:
            ref, asked, w, z = O.attend(*state, table, page, h(q), at, None, cap * page)
            _close(h(out)[asked], ref[asked], _tolerance("bf16", ref, w, z)[asked])
    assert C.csa_device_error(ws) == 0
    for a, b in zip(cache.host(), state):
        assert np.array_equal(a, b)
    del graph


def test_one_workspace_for_calls_of_different_shapes():
    """Nothing that a call leaves in the workspace reaches the next one, whatever its shape and kernel."""
    rng = np.random.default_rng(7)
    Hkv, D, page, cap, B = 2, 64, 32, 70, 6
    cache = Cache(rng, B * cap, Hkv, page, D)
    table, _ = _table(rng, B, cap, cache.N, [cap] * B)
    pool, td = cache.up(), _dev(table)
    calls = []
    for H, act, Tq, n in ((4, "bf16", 1, 6), (32, "bf16", 40, 6), (2, "f32", 3, 2), (2, "bf16", 300, 1), (16, "bf16", 5, 6),
                          (4, "bf16", 2, 3), (2, "bf16", 700, 6)):
        T = C.make_page_table(td[:n], _ints(cache.N, 0), page)
        G = C.make_gqa(H, Hkv, D, act_format=act)
        q = torch.randn(n, Tq, H, D, device="cuda").to(torch.float32 if act == "f32" else torch.bfloat16)
        start = _dev(rng.integers(-1, cap * page - Tq, n))
        n_new = _dev(rng.integers(0, Tq + 1, n).astype(np.int32))
        calls.append((G, T, q, start, n_new, Tq))
    size = max(C.csa_paged_workspace_size(c[0], c[1], c[5], cap * page) for c in calls)
    shared = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def run(c, ws):
        out = torch.zeros_like(c[2])
        C.csa_paged_attend(c[0], pool, c[1], c[2], None, c[3], c[4], c[5], cap * page, out, ws)
        return out

    alone = [run(c, torch.zeros(size, dtype=torch.uint8, device="cuda")) for c in calls]
    for i in rng.integers(0, len(calls), 60):
        assert torch.equal(run(calls[i], shared), alone[i]), i
    assert C.csa_device_error(shared) == 0


def test_a_paged_workspace_that_is_zeroed_serves_the_other_calls():
    """Both ways: the paged calls read nothing that others left but the error word, and after a zero-fill the others
    find what they need."""
    from csa_synth import decode_inputs, get_workload
    from long_context_sparse_csa_b200.state import LayerState, to_device

    wl = get_workload("csa_decode_128k", B=2, n=4 * 20000)
    layer, d = wl.layers[0], decode_inputs(get_workload("csa_decode_128k", B=2, n=4 * 20000))
    st = LayerState.from_arrays(layer, wl.B, d)
    cap = d["entries"].shape[1]
    rng = np.random.default_rng(19)
    cache = Cache(rng, 90, 1, 16, 64)
    table, _ = _table(rng, 1, 90, 90, [90])
    pool, T, G = cache.up(), C.make_page_table(_dev(table), _ints(90, 0), 16), C.make_gqa(8, 1, 64)
    q, start = torch.randn(1, 40, 8, 64, device="cuda").bfloat16(), torch.tensor([1400], device="cuda")
    size = max(st.workspace("index_topk", 1, cap).numel(), C.csa_paged_workspace_size(G, T, 40, 1440))
    args = [to_device(d[k]) for k in ("idx_q", "idx_q_scale", "head_w", "t")]
    shared, want_o, want_k = torch.zeros(size, dtype=torch.uint8, device="cuda"), None, None
    for _ in range(3):
        topk = torch.zeros((2, layer.top_k), dtype=torch.int32, device="cuda")
        C.csa_index_topk(st.L, st.cache(), *args, 1, cap, topk, None, shared)
        out = torch.zeros_like(q)
        C.csa_paged_attend(G, pool, T, q, None, start, None, 40, 1440, out, shared)
        assert C.csa_device_error(shared) == 0
        want_o, want_k = out if want_o is None else want_o, topk if want_k is None else want_k
        assert torch.equal(out, want_o) and torch.equal(topk, want_k)
        shared.zero_()


def test_a_captured_chunk_follows_its_inputs():
    """Prompt chunks of a padded batch in a graph, replayed beside an eager call on another stream."""
    rng = np.random.default_rng(8)
    B, Tq, H, Hkv, D, page, cap = 3, 70, 8, 2, 128, 16, 40
    cache = Cache(rng, B * cap, Hkv, page, D)
    table, _ = _table(rng, B, cap, cache.N, [cap] * B)
    pool = cache.up()
    T, G = C.make_page_table(_dev(table), _ints(cache.N, 0), page), C.make_gqa(H, Hkv, D, 200, 5)
    q = torch.randn(B, Tq, H, D, device="cuda").bfloat16()
    start, n_new = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    size = C.csa_paged_workspace_size(G, T, Tq, cap * page)
    ws, ws2 = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    out, other = torch.zeros_like(q), torch.zeros_like(q)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    C.csa_paged_attend(G, pool, T, q, None, start, n_new, Tq, cap * page, out, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        C.csa_paged_attend(G, pool, T, q, None, start, n_new, Tq, cap * page, out, ws)
    h = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    for i in range(6):
        start.copy_(_dev(rng.integers(-1, cap * page - Tq, B)))
        n_new.copy_(_dev(rng.integers(0, Tq + 1, B).astype(np.int32)))
        torch.cuda.synchronize()
        graph.replay()
        C.csa_paged_attend(G, pool, T, q, None, start, n_new, Tq, cap * page, other, ws2, stream=side)
        torch.cuda.synchronize()
        ref, asked, w, z = O.attend(cache.k, cache.v, cache.ks, cache.vs, table, page, h(q), start.cpu().numpy(),
                                    n_new.cpu().numpy(), cap * page, 200, 5)
        for o in (out, other):
            _close(h(o)[asked], ref[asked], _tolerance("bf16", ref, w, z)[asked])
    assert C.csa_device_error(ws) == 0 and C.csa_device_error(ws2) == 0
    del graph


def test_two_calls_at_once_on_two_streams():
    rng = np.random.default_rng(6)
    n, page = 4000, 32
    N = 2 * n // page
    cache = Cache(rng, N, 2, page, 128)
    table, _ = _table(rng, 2, n // page, N, [n // page] * 2)
    pool = cache.up()
    td = _dev(table)
    G = C.make_gqa(16, 2, 128)
    calls = []
    for b in range(2):
        T = C.make_page_table(td[b:b + 1], _ints(N, 0), page)
        q = torch.randn(1, 1, 16, 128, device="cuda").bfloat16()
        ws = torch.zeros(C.csa_paged_workspace_size(G, T, 1, n), dtype=torch.uint8, device="cuda")
        calls.append((T, q, torch.tensor([n - 1], device="cuda"), ws))
    alone = []
    for T, q, s, ws in calls:
        out = torch.empty_like(q)
        C.csa_paged_attend(G, pool, T, q, None, s, None, 1, n, out, ws)
        alone.append(out)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in calls], [[], []]
    for _ in range(20):
        for i, (T, q, s, ws) in enumerate(calls):
            out = torch.empty_like(q)
            C.csa_paged_attend(G, pool, T, q, None, s, None, 1, n, out, ws, stream=streams[i])
            outs[i].append(out)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, alone[i]) for o in outs[i])


def test_tensors_elsewhere_are_refused():
    table, refs = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(C.CsaError):
        C.csa_pages_fork(C.make_page_table(table, refs, 16), refs.cuda(), refs.cuda(), 1)
    T = C.make_page_table(table.cuda(), refs.cuda(), 16)
    with pytest.raises(C.CsaError):
        C.csa_pages_fork(T, refs, refs.cuda(), 1)
