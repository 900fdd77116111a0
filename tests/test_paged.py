"""Paged 8-bit cache, without a GPU: the oracle's own properties, and the calls' refusals."""

import ctypes

import numpy as np
import pytest
import torch

from long_context_sparse_csa_b200 import binding as C
from oracle import paged as O
from oracle.formats import e4m3_decode

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


# ----------------------------------------------------------------------------- oracle
@pytest.mark.parametrize("amax", [0.0, 2.0 ** -149, 1e-30, 447.9, 448.0, 448.1, 1.0, 3.4e38])
def test_page_scale_is_the_smallest_power_of_two(amax):
    s = O.page_scale(amax)
    assert np.log2(s) == np.round(np.log2(s)) and s >= 2.0 ** -126 and amax / s <= 448
    assert s == 2.0 ** -126 or amax / (s / 2) > 448


def _pool(rng, N, Hkv, page, D):
    k = rng.integers(0, 0x7F, (N, Hkv, page, D)).astype(np.uint8) | (rng.integers(0, 2, (N, Hkv, page, D)) << 7).astype(np.uint8)
    return k, 2.0 ** rng.integers(-8, -5, (N, Hkv)).astype(np.float32)


def test_append_in_pieces_never_loses_more_than_the_last_scale_allows():
    rng = np.random.default_rng(0)
    page, Hkv, D = 16, 2, 64
    x = rng.standard_normal((1, 40, Hkv, D)) * np.exp(rng.uniform(-4, 4, (1, 40, 1, 1)))
    k = np.zeros((4, Hkv, page, D), np.uint8)
    ks = np.zeros((4, Hkv), np.float32)
    table, refs = np.array([[2, 0, 3]], np.int32), np.array([1, 0, 1, 1], np.int32)
    state = (k, k.copy(), ks, ks.copy())
    at = 0
    for n in (1, 5, 20, 14):
        *state, err = O.append(*state, table, refs, page, x[:, at:at + n], x[:, at:at + n], [at], None)
        assert not err
        at += n
    for p, g in enumerate(table[0]):
        rows = x[0, p * page:(p + 1) * page].transpose(1, 0, 2)
        got = e4m3_decode(state[0][g]) * state[2][g][:, None, None]
        # each rounding is off by half a step: 2^-4 of the value, or half of the smallest step (2^-10 of the
        # scale).  A page of 16 tokens written in at most four pieces is rounded at most four times.
        n = rows.shape[1]
        assert np.all(np.abs(got[:, :n] - rows) <= 4 * (np.abs(rows) * 2.0 ** -4 * 1.3 + 2.0 ** -10 * state[2][g][:, None, None]))


def test_attend_of_one_key_is_its_value():
    rng = np.random.default_rng(1)
    k, ks = _pool(rng, 3, 1, 16, 64)
    v, vs = _pool(rng, 3, 1, 16, 64)
    q = rng.standard_normal((1, 1, 4, 64))
    out, asked, *_ = O.attend(k, v, ks, vs, np.array([[1]]), 16, q, [0], None, 1)
    assert asked.all() and np.allclose(out[0, 0], e4m3_decode(v[1, 0, 0]) * vs[1, 0], rtol=0, atol=0)


def test_fork_reserve_free_compact_keep_counts_and_contents():
    """A random life of a pool: counts always equal the table's entries, and every sequence keeps its page
    contents (tracked as a version number per page)."""
    rng = np.random.default_rng(2)
    B, cap, N, page = 6, 5, 20, 16
    table, refs = np.full((B, cap), -1, np.int32), np.zeros(N, np.int32)
    content = np.zeros(N, np.int64)
    lens, want = np.zeros(B, np.int64), {}
    version = 1
    for step in range(200):
        act = rng.integers(0, 4)
        if act == 0:
            s, d = rng.choice(B, 2, replace=False)
            table, refs, err = O.fork(table, refs, [s], [d])
            lens[d] = lens[s]
            want.update({(d, p): want.get((s, p)) for p in range(cap)})
            assert not err
        elif act == 1:
            n_new = rng.integers(0, 20, B)
            start = np.where(lens + n_new <= cap * page, lens, -1)
            table, refs, src, dst, missing, err = O.reserve(table, refs, page, start, n_new, 20)
            assert not err
            if missing == 0:
                for s, d in zip(src, dst):
                    if s >= 0:
                        content[d] = content[s]
                for b in range(B):
                    if start[b] >= 0 and n_new[b]:
                        for p in range(start[b] // page, (start[b] + n_new[b] - 1) // page + 1):
                            assert refs[table[b, p]] == 1
                            if p * page < start[b]:
                                assert content[table[b, p]] == want[b, p]
                            content[table[b, p]] = want[b, p] = version
                            version += 1
                        lens[b] += n_new[b]
        elif act == 2:
            keep = np.where(rng.random(B) < 0.3, 0, -1)
            table, refs = O.free(table, refs, page, keep, None, 0)
            lens[keep == 0] = 0
        else:
            table, refs, src, dst, n = O.compact(table, refs, int(rng.integers(0, N)))
            content[dst[:n]] = content[src[:n]]
        counts = np.bincount(table[table >= 0], minlength=N)
        assert np.array_equal(counts, refs)
        for b in range(B):
            for p in range(-(-lens[b] // page)):
                assert content[table[b, p]] == want[b, p]


# ----------------------------------------------------------------------------- refusals of the library
def _structs():
    buf = torch.zeros(1 << 16, dtype=torch.uint8)
    p = (buf.data_ptr() + 255) // 256 * 256
    G = C.make_gqa(8, 2, 64)
    pool = C.CsaPagePool(p, p, p, p)
    T = C.CsaPageTable(p, p, 4, 8, 2, 16)
    return buf, p, G, pool, T


def _attend(G, pool, T, p, **kw):
    a = dict(q=p, q_stride=0, sinks=None, start=p, n_new=None, Tq=1, n_max=64, out=p, ws=p, ws_bytes=1 << 40)
    a.update(kw)
    r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return C.lib().csa_paged_attend(r(G), r(pool), r(T), a["q"], a["q_stride"], a["sinks"], a["start"], a["n_new"],
                                    a["Tq"], a["n_max"], a["out"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(H=0), INVALID), (dict(H=9), INVALID), (dict(Hkv=0), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(act_format=2), INVALID), (dict(window=-1), INVALID), (dict(first=-1), INVALID),
    (dict(first=4), INVALID), (dict(softmax_scale=float("nan")), INVALID), (dict(softmax_scale=-1.0), INVALID),
    (dict(softmax_scale=float("inf")), INVALID), (dict(reserved=1), INVALID)])
def test_layers_that_no_kernel_serves_are_refused(kw, status):
    buf, p, G, pool, T = _structs()
    for name, value in kw.items():
        setattr(G, name, value)
    assert _attend(G, pool, T, p) == status
    assert C.csa_paged_workspace_size(G, T, 1, 64) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(table_cap=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(n_pages=2 ** 30 + 1), INVALID), (dict(table=None), INVALID),
    (dict(table_cap=3), INVALID)])
def test_tables_outside_the_limits_are_refused(kw, status):
    buf, p, G, pool, T = _structs()
    for name, value in kw.items():
        setattr(T, name, value)
    assert _attend(G, pool, T, p) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(start=None), INVALID), (dict(Tq=0), INVALID),
    (dict(Tq=2 ** 25), INVALID), (dict(n_max=-1), INVALID), (dict(n_max=65), INVALID), (dict(q_stride=8), INVALID),
    (dict(q_stride=8 * 64 + 4), INVALID), (dict(ws=None), WORKSPACE), (dict(ws_bytes=64), WORKSPACE)])
def test_attend_arguments_are_refused(kw, status):
    buf, p, G, pool, T = _structs()
    assert _attend(G, pool, T, p, **kw) == status
    assert C.lib().csa_last_error()


def test_misaligned_and_missing_pointers_are_refused():
    buf, p, G, pool, T = _structs()
    assert _attend(G, C.CsaPagePool(p + 4, p, p, p), T, p) == INVALID
    assert _attend(G, C.CsaPagePool(p, p, None, p), T, p) == INVALID
    assert _attend(G, pool, T, p, ws=p + 16) == WORKSPACE
    assert _attend(None, pool, T, p) == INVALID
    assert _attend(G, None, T, p) == INVALID
    assert _attend(G, pool, None, p) == INVALID
    T2 = C.CsaPageTable(p, p + 4, 4, 8, 2, 16)
    assert _attend(G, pool, T2, p) == INVALID


def test_bookkeeping_arguments_are_refused():
    h = C.lib()
    buf, p, G, pool, T = _structs()
    r = ctypes.byref
    no_refs = C.CsaPageTable(p, None, 4, 8, 2, 16)
    assert h.csa_pages_fork(r(no_refs), p, p, 1, None) == INVALID
    assert h.csa_pages_fork(r(T), p, p, -1, None) == INVALID
    assert h.csa_pages_fork(r(T), p, p, 4097, None) == INVALID
    assert h.csa_pages_fork(r(T), None, p, 1, None) == INVALID
    assert h.csa_pages_fork(r(T), None, None, 0, None) == 0
    assert h.csa_pages_reserve(r(T), p, None, 0, p, p, p, None) == INVALID
    assert h.csa_pages_reserve(r(T), p, None, 1, None, p, p, None) == INVALID
    assert h.csa_pages_reserve(r(T), p, None, 1, p, p, None, None) == INVALID
    assert h.csa_pages_reserve(r(C.CsaPageTable(p, p, 4, 8, 1 << 20, 16)), p, None, 1 << 20, p, p, p, None) == UNSUPPORTED
    assert h.csa_pages_free(r(T), None, None, 0, None) == INVALID
    assert h.csa_pages_free(r(T), p, None, -1, None) == INVALID
    assert h.csa_pages_compact(r(T), 9, p, p, p, None) == INVALID
    assert h.csa_pages_compact(r(T), -1, p, p, p, None) == INVALID
    assert h.csa_pages_compact(r(T), 1, None, p, p, None) == INVALID
    assert h.csa_pages_compact(r(T), 1, p, p, None, None) == INVALID
    assert h.csa_pages_copy(r(G), r(pool), r(T), p, p, None, -1, None) == INVALID
    assert h.csa_pages_copy(r(G), r(pool), r(T), None, p, None, 1, None) == INVALID
    assert h.csa_pages_copy(r(G), r(pool), r(T), None, None, None, 0, None) == 0
    assert h.csa_paged_append(r(G), r(pool), r(T), None, p, 0, p, None, 1, None) == INVALID
    assert h.csa_paged_append(r(G), r(pool), r(T), p, p, 64, p, None, 1, None) == INVALID
    assert h.csa_paged_append(r(G), r(pool), r(T), p, p, 0, None, None, 1, None) == INVALID


def test_struct_layouts():
    assert ctypes.sizeof(C.CsaGqa) == 32 and ctypes.sizeof(C.CsaPagePool) == 32
    assert ctypes.sizeof(C.CsaPageTable) == 40 and C.CsaPageTable.B.offset == 32


def test_binding_refuses_tensors_of_other_types_shapes_and_layouts():
    t32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(8, 2, 16, 64, dtype=torch.uint8)
    sc = torch.zeros(8, 2)
    C.make_page_pool(k, k, sc, sc)
    for bad in ((k.float(), k, sc, sc), (k, k[:4], sc, sc), (k, k, sc.double(), sc), (k, k, sc[:, :1], sc),
                (k.transpose(0, 1), k, sc, sc)):
        with pytest.raises(C.CsaError):
            C.make_page_pool(*bad)
    with pytest.raises(C.CsaError):
        C.make_page_table(t32(2, 4).long(), t32(8), 16)
    with pytest.raises(C.CsaError):
        C.make_page_table(t32(4, 2).t(), t32(8), 16)
    G, T = C.make_gqa(8, 2, 64), C.make_page_table(t32(2, 4), t32(8), 16)
    with pytest.raises(C.CsaError):                     # another page size than the table's
        C._paged_pool(G, C.make_page_pool(k.view(4, 2, 32, 64), k.view(4, 2, 32, 64), sc[:4], sc[:4]), T)
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    assert C._token_stride(x, "x", G, 2, 3, 2) == 128
    assert C._token_stride(torch.zeros(2, 3, 6, 64, dtype=torch.bfloat16)[:, :, :2], "x", G, 2, 3, 2) == 384
    for bad in (x.float(), x[:, :2], x.transpose(2, 3).contiguous().transpose(2, 3), x[:1].expand(2, 3, 2, 64),
                x[:, :1].expand(2, 3, 2, 64), torch.zeros(3, 2, 2, 64, dtype=torch.bfloat16).transpose(0, 1)):
        with pytest.raises(C.CsaError):
            C._token_stride(bad, "x", G, 2, 3, 2)
