"""ctypes binding of libcsa.so: the C ABI declared in include/csa.h, one Python
function per entry point with the same name.

Only argument marshalling happens here (torch tensors -> device pointers,
layer / cache / parameter structs, the current CUDA stream); every step of
the operator runs in the library's kernels.  A missing or unloadable library
raises immediately -- there is no fallback path.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

FMT = {"f32": 0, "bf16": 1, "mixed": 2, "e4m3": 3, "e2m1": 4}
SEGMENT = {"error_word": 0, "scores": 1, "topk_histogram": 2, "topk": 3, "partials": 4, "index_query": 5,
           "index_query_scale": 6}
KIND = {"csa": 0, "hca": 1}
OP = {"index_topk": 0, "sparse_attend": 1, "hca_attend": 2, "decode_step": 3, "prefill": 4, "decode_step_indexed": 5}
STATUS = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_WORKSPACE",
          4: "CSA_ERR_CUDA", 5: "CSA_ERR_DEVICE_TIMEOUT", 6: "CSA_ERR_DEVICE_PAGE"}


class CsaError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class CsaLayer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("B", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("d_rope", ctypes.c_int32), ("m", ctypes.c_int32), ("overlap", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("window", ctypes.c_int32), ("H_I", ctypes.c_int32),
                ("d_I", ctypes.c_int32), ("kv_format", ctypes.c_int32), ("idx_format", ctypes.c_int32),
                ("act_format", ctypes.c_int32), ("rope_base", ctypes.c_double), ("eps", ctypes.c_float),
                ("softmax_scale", ctypes.c_float), ("pos0", ctypes.c_int64)]


class CsaCache(ctypes.Structure):
    _fields_ = [("entries", ctypes.c_void_p), ("entry_cap", ctypes.c_int64), ("idx_keys", ctypes.c_void_p),
                ("idx_key_scale", ctypes.c_void_p), ("window", ctypes.c_void_p), ("window_cap", ctypes.c_int64),
                ("raw", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("raw_cap", ctypes.c_int64),
                ("raw_base", ctypes.c_int64)]


class CsaParams(ctypes.Structure):
    _fields_ = [("pos_bias", ctypes.c_void_p), ("gamma_kv", ctypes.c_void_p), ("gamma_q", ctypes.c_void_p),
                ("sinks", ctypes.c_void_p)]


class CsaIndexStream(ctypes.Structure):
    _fields_ = [("raw", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("pos_bias", ctypes.c_void_p)]


class CsaGqa(ctypes.Structure):
    _fields_ = [("H", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("act_format", ctypes.c_int32),
                ("window", ctypes.c_int32), ("first", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class CsaPagePool(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p)]


class CsaPageTable(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("refs", ctypes.c_void_p), ("table_cap", ctypes.c_int64),
                ("n_pages", ctypes.c_int64), ("B", ctypes.c_int32), ("page", ctypes.c_int32)]


_P = ctypes.c_void_p
_GQA = ctypes.POINTER(CsaGqa)
_POOL = ctypes.POINTER(CsaPagePool)
_TABLE = ctypes.POINTER(CsaPageTable)
_STREAM_S = ctypes.POINTER(CsaIndexStream)
_LAYER = ctypes.POINTER(CsaLayer)
_CACHE = ctypes.POINTER(CsaCache)
_PARAMS = ctypes.POINTER(CsaParams)
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t

_SIGS = {
    "csa_row_bytes": (_SZ, [_LAYER]),
    "csa_workspace_size": (_SZ, [_LAYER, _I32, _I32, _I64]),
    "csa_last_error": (ctypes.c_char_p, []),
    "csa_version": (ctypes.c_char_p, []),
    "csa_profile_events": (None, [_P, _P]),
    "csa_launch_count": (ctypes.c_uint64, []),
    "csa_profile_timeline": (None, [_P, _I32]),
    "csa_profile_timeline_count": (_I32, []),
    "csa_device_error": (ctypes.c_int, [_P, _SZ, _P, ctypes.POINTER(_I32)]),
    "csa_append": (ctypes.c_int, [_LAYER, _CACHE, _P, _P, _P, _I32, _P]),
    "csa_compress": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _I32, _P]),
    "csa_index_topk": (ctypes.c_int, [_LAYER, _CACHE, _P, _P, _P, _P, _I32, _I64, _P, _P, _P, _SZ, _P]),
    "csa_sparse_attend": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _I32, _P, _P, _P, _SZ, _P]),
    "hca_attend": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _I32, _I64, _P, _P, _SZ, _P]),
    "csa_decode_step": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "hca_decode_step": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "csa_decode_step_scratch": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                               ctypes.POINTER(_I32), _P]),
    "csa_prefill": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _P, _P, _P, _I32, _I64, _P, _P, _P, _SZ, _P]),
    "csa_debug_workspace_segment": (ctypes.c_int, [_LAYER, _I32, _I32, _I64, _I32, ctypes.POINTER(_SZ),
                                                   ctypes.POINTER(_SZ)]),
    "csa_debug_wait_probe": (ctypes.c_int, [_P, _SZ, ctypes.c_uint64, _P]),
    "csa_debug_scratch_copy": (ctypes.c_int, [_SZ, _P, _SZ, _I32, _P]),
    "csa_index_keys": (ctypes.c_int, [_LAYER, _CACHE, _STREAM_S, _P, _P, _P, _I32, _P]),
    "csa_index_query": (ctypes.c_int, [_LAYER, _P, _P, _I32, _I32, _P, _P, _P]),
    "csa_decode_step_indexed": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _STREAM_S, _P, _P, _P, _I32, _P, _P, _P, _P,
                                               _P, _P, _P, _P, _P, _SZ, _P]),
    "csa_shard_candidates": (ctypes.c_int, [_LAYER, _P, _I64, _P, _I64, _P, _P, _P]),
    "csa_shard_select": (ctypes.c_int, [_LAYER, _I32, _P, _P, _P, _P]),
    "csa_sparse_attend_partial": (ctypes.c_int, [_LAYER, _CACHE, _PARAMS, _P, _P, _P, _I64, _I32, _P, _P, _SZ, _P]),
    "csa_attend_merge": (ctypes.c_int, [_LAYER, _PARAMS, _P, _I32, _P, _P, _P]),
    "csa_paged_append": (ctypes.c_int, [_GQA, _POOL, _TABLE, _P, _P, _I64, _P, _P, _I32, _P]),
    "csa_paged_workspace_size": (_SZ, [_GQA, _TABLE, _I32, _I64]),
    "csa_paged_attend": (ctypes.c_int, [_GQA, _POOL, _TABLE, _P, _I64, _P, _P, _P, _I32, _I64, _P, _P, _SZ, _P]),
    "csa_debug_paged_join": (ctypes.c_int, [_GQA, _TABLE, _P, _P, _P, _I32, _I64, _P, _P, _SZ, _P]),
    "csa_pages_fork": (ctypes.c_int, [_TABLE, _P, _P, _I32, _P]),
    "csa_pages_reserve": (ctypes.c_int, [_TABLE, _P, _P, _I32, _P, _P, _P, _P]),
    "csa_pages_free": (ctypes.c_int, [_TABLE, _P, _P, _I64, _P]),
    "csa_pages_compact": (ctypes.c_int, [_TABLE, _I32, _P, _P, _P, _P]),
    "csa_pages_copy": (ctypes.c_int, [_GQA, _POOL, _TABLE, _P, _P, _P, _I32, _P]),
}

EXPORTED = tuple(_SIGS)

_lib = None


def lib():
    """The loaded library; raises if it was not built (no fallback exists)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m long_context_sparse_csa_b200.build`")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


def _check(status):
    if status != 0:
        raise CsaError(status, lib().csa_last_error().decode())


def ptr(t):
    """Device (or host) address of a tensor, or None."""
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_layer(kind, B, H, D, m, overlap, top_k=0, window=128, H_I=0, d_I=0, kv_format="bf16",
               idx_format="e4m3", act_format="bf16", rope_base=10000.0, eps=1e-6, softmax_scale=0.0,
               pos0=0, d_rope=64) -> CsaLayer:
    return CsaLayer(KIND[kind], B, H, D, d_rope, m, overlap, top_k, window, H_I, d_I, FMT[kv_format],
                    FMT[idx_format], FMT[act_format], float(rope_base), float(eps), float(softmax_scale), int(pos0))


def layer_from_spec(layer, B, pos0=0) -> CsaLayer:
    """CsaLayer from a csa_synth.configs.Layer."""
    return make_layer(layer.kind, B, layer.H, layer.D, layer.m, layer.ov, layer.top_k, layer.window, layer.H_I,
                      layer.d_I, layer.kv_format, layer.idx_format, layer.act_format, layer.rope_base, layer.eps,
                      0.0, pos0, layer.d_rope)


def make_cache(entries, window, raw=None, gate=None, idx_keys=None, idx_key_scale=None, raw_base=0) -> CsaCache:
    """Cache struct over tensors shaped [B, cap, ...] (entries, window, raw, gate, idx keys)."""
    return CsaCache(entries.data_ptr(), entries.shape[1], idx_keys.data_ptr() if idx_keys is not None else None,
                    idx_key_scale.data_ptr() if idx_key_scale is not None else None, window.data_ptr(),
                    window.shape[1], raw.data_ptr() if raw is not None else None,
                    gate.data_ptr() if gate is not None else None, raw.shape[1] if raw is not None else 0, raw_base)


def make_index_stream(raw, gate, pos_bias) -> CsaIndexStream:
    """Index-key stream struct over rings [B, raw_cap, d_I] and the slot biases [(1+ov)m, d_I]."""
    return CsaIndexStream(raw.data_ptr(), gate.data_ptr(), pos_bias.data_ptr())


def make_params(pos_bias=None, gamma_kv=None, gamma_q=None, sinks=None) -> CsaParams:
    g = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
    return CsaParams(g(pos_bias), g(gamma_kv), g(gamma_q), g(sinks))


def make_gqa(H, Hkv, D, window=0, first=0, act_format="bf16", softmax_scale=0.0) -> CsaGqa:
    return CsaGqa(H, Hkv, D, FMT[act_format], window, first, float(softmax_scale), 0)


def _tensor(t, name, dtypes, shape):
    """Refuses a tensor of another type, shape or layout than the call reads (None in shape: any size)."""
    if t.dtype not in dtypes:
        raise CsaError(1, f"{name} is {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != len(shape) or any(w is not None and w != g for w, g in zip(shape, t.shape)):
        raise CsaError(1, f"{name} has shape {tuple(t.shape)}, not {shape}")
    if not t.is_contiguous():
        raise CsaError(1, f"{name} is not contiguous")


def _one_device(*tensors):
    d = tensors[0].get_device()
    for t in tensors:
        if t.get_device() == d:
            continue
        raise CsaError(1, "tensors on different devices: " + ", ".join(str(t.device) for t in tensors))
    return d


def make_page_pool(k, v, k_scale, v_scale) -> CsaPagePool:
    """Page pool struct over codes [n_pages, Hkv, page, D] (uint8 or float8_e4m3fn) and scales [n_pages, Hkv]
    (float32).  It keeps the tensors alive."""
    codes = (torch.uint8, torch.float8_e4m3fn)
    _tensor(k, "k", codes, (None, None, None, None))
    _tensor(v, "v", codes, tuple(k.shape))
    _tensor(k_scale, "k_scale", (torch.float32,), tuple(k.shape[:2]))
    _tensor(v_scale, "v_scale", (torch.float32,), tuple(k.shape[:2]))
    p = CsaPagePool(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
    p.shape, p.keep, p.device = tuple(k.shape), (k, v, k_scale, v_scale), _one_device(k, v, k_scale, v_scale)
    return p


def make_page_table(table, refs, page) -> CsaPageTable:
    """Page table struct over table [B, table_cap] and refs [n_pages] (int32).  It keeps the tensors alive."""
    if not (table.dtype is refs.dtype is torch.int32 and table.dim() == 2 and refs.dim() == 1 and table.is_contiguous()
            and refs.is_contiguous()):
        raise CsaError(1, "table [B, table_cap] and refs [n_pages] must be contiguous torch.int32")
    B, cap = table.shape
    t = CsaPageTable(table.data_ptr(), refs.data_ptr(), cap, refs.numel(), B, page)
    t.keep, t.device = (table, refs), _one_device(table, refs)
    return t


# ----------------------------------------------------------------------------- entry points
def csa_row_bytes(L: CsaLayer) -> int:
    return lib().csa_row_bytes(ctypes.byref(L))


def csa_workspace_size(L: CsaLayer, op: str, Tq: int, entry_cap: int) -> int:
    return lib().csa_workspace_size(ctypes.byref(L), OP[op], Tq, entry_cap)


def csa_version() -> str:
    return lib().csa_version().decode()


def csa_profile_events(ev_start, ev_stop):
    """Record these torch.cuda.Events around each later indexer-score launch (None, None: off)."""
    h = lib()
    if ev_start is None or ev_stop is None:
        h.csa_profile_events(None, None)
    else:
        h.csa_profile_events(ctypes.c_void_p(ev_start.cuda_event), ctypes.c_void_p(ev_stop.cuda_event))


_timeline_keep = None


def csa_profile_timeline(events):
    """Arm a timeline of torch.cuda.Events (recorded before each later launch); None disarms."""
    global _timeline_keep
    h = lib()
    if not events:
        h.csa_profile_timeline(None, 0)
        _timeline_keep = None
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _timeline_keep = arr
    h.csa_profile_timeline(ctypes.cast(arr, ctypes.c_void_p), len(events))


def csa_profile_timeline_count() -> int:
    return lib().csa_profile_timeline_count()


def csa_launch_count() -> int:
    return lib().csa_launch_count()


def csa_device_error(workspace, stream=None) -> int:
    """OR of the workspace's error word and the library's own word; without a workspace (None), of the library's and
    the word of the paged-cache calls that take none.  The words read are cleared."""
    code = _I32(0)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().csa_device_error(ptr(workspace), nbytes, _stream(stream), ctypes.byref(code))
    if st not in (0, 5, 6):
        _check(st)
    return code.value


def csa_debug_workspace_segment(L, op, Tq, entry_cap, segment):
    """(byte offset, bytes) of a workspace segment (test aid)."""
    off, nb = _SZ(0), _SZ(0)
    _check(lib().csa_debug_workspace_segment(ctypes.byref(L), OP[op], Tq, entry_cap, SEGMENT[segment],
                                             ctypes.byref(off), ctypes.byref(nb)))
    return off.value, nb.value


def csa_debug_wait_probe(workspace, limit_ns, stream=None):
    """Launch the bounded-wait probe: its wait runs out after limit_ns and sets the error word (test aid)."""
    _check(lib().csa_debug_wait_probe(ptr(workspace), workspace.numel() * workspace.element_size(), int(limit_ns),
                                      _stream(stream)))


def csa_debug_scratch_copy(offset, buf, to_scratch, stream=None):
    """Copy between a tensor and the static scratch at byte `offset` (test aid; synchronises)."""
    _check(lib().csa_debug_scratch_copy(int(offset), ptr(buf), buf.numel() * buf.element_size(),
                                        1 if to_scratch else 0, _stream(stream)))


def csa_append(L, cache, x_new, g_new, q_pos, Tq, stream=None):
    _check(lib().csa_append(ctypes.byref(L), ctypes.byref(cache), ptr(x_new), ptr(g_new), ptr(q_pos), Tq,
                            _stream(stream)))


def csa_compress(L, cache, params, q_pos, Tq, stream=None):
    _check(lib().csa_compress(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q_pos), Tq,
                              _stream(stream)))


def csa_index_topk(L, cache, idx_q, idx_q_scale, head_w, q_pos, Tq, n_max, topk_idx, scores, workspace,
                   stream=None):
    _check(lib().csa_index_topk(ctypes.byref(L), ctypes.byref(cache), ptr(idx_q), ptr(idx_q_scale), ptr(head_w),
                                ptr(q_pos), Tq, n_max, ptr(topk_idx), ptr(scores), ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream)))


def csa_sparse_attend(L, cache, params, q, q_pos, Tq, topk_idx, out, workspace, stream=None):
    _check(lib().csa_sparse_attend(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q), ptr(q_pos),
                                   Tq, ptr(topk_idx), ptr(out), ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(stream)))


def hca_attend(L, cache, params, q, q_pos, Tq, n_max, out, workspace, stream=None):
    _check(lib().hca_attend(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q), ptr(q_pos), Tq,
                            n_max, ptr(out), ptr(workspace), workspace.numel() * workspace.element_size(),
                            _stream(stream)))


def csa_decode_step(L, cache, params, q, idx_q, idx_q_scale, head_w, x_new, g_new, q_pos, out, topk_idx,
                    workspace, stream=None):
    _check(lib().csa_decode_step(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q), ptr(idx_q),
                                 ptr(idx_q_scale), ptr(head_w), ptr(x_new), ptr(g_new), ptr(q_pos), ptr(out),
                                 ptr(topk_idx), ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)))


def csa_decode_step_scratch(L, cache, params, q, idx_q, idx_q_scale, head_w, x_new, g_new, q_pos, out, topk_idx,
                            read_device_error=False, stream=None):
    """csa_decode_step on the library's static device scratch (no workspace argument).  With
    read_device_error the call synchronises and returns the device error word (else None)."""
    code = _I32(0)
    st = lib().csa_decode_step_scratch(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q),
                                       ptr(idx_q), ptr(idx_q_scale), ptr(head_w), ptr(x_new), ptr(g_new),
                                       ptr(q_pos), ptr(out), ptr(topk_idx),
                                       ctypes.byref(code) if read_device_error else None, _stream(stream))
    if read_device_error and st == 5:      # CSA_ERR_DEVICE_TIMEOUT: the device error word is the result
        return code.value
    _check(st)
    return code.value if read_device_error else None


def hca_decode_step(L, cache, params, q, x_new, g_new, q_pos, out, workspace, stream=None):
    _check(lib().hca_decode_step(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q), ptr(x_new),
                                 ptr(g_new), ptr(q_pos), ptr(out), ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def csa_prefill(L, cache, params, q, idx_q, idx_q_scale, head_w, q_pos, Tq, n_max, out, topk_idx, workspace,
                stream=None):
    _check(lib().csa_prefill(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q), ptr(idx_q),
                             ptr(idx_q_scale), ptr(head_w), ptr(q_pos), Tq, n_max, ptr(out), ptr(topk_idx),
                             ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def csa_index_keys(L, cache, index_stream, x_new, g_new, q_pos, Tq, stream=None):
    _check(lib().csa_index_keys(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(index_stream), ptr(x_new),
                                ptr(g_new), ptr(q_pos), Tq, _stream(stream)))


def csa_index_query(L, c, W, rank, rows, idx_q, idx_q_scale, stream=None):
    _check(lib().csa_index_query(ctypes.byref(L), ptr(c), ptr(W), rank, rows, ptr(idx_q), ptr(idx_q_scale),
                                 _stream(stream)))


def csa_decode_step_indexed(L, cache, params, index_stream, q, c, W, rank, head_w, x_new, g_new, idx_x_new,
                            idx_g_new, q_pos, out, topk_idx, workspace, stream=None):
    _check(lib().csa_decode_step_indexed(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params),
                                         ctypes.byref(index_stream), ptr(q), ptr(c), ptr(W), rank, ptr(head_w),
                                         ptr(x_new), ptr(g_new), ptr(idx_x_new), ptr(idx_g_new), ptr(q_pos), ptr(out),
                                         ptr(topk_idx), ptr(workspace), workspace.numel() * workspace.element_size(),
                                         _stream(stream)))


def csa_shard_candidates(L, scores, n_local, topk_local, entry_offset, cand_score, cand_idx, stream=None):
    _check(lib().csa_shard_candidates(ctypes.byref(L), ptr(scores), n_local, ptr(topk_local), entry_offset,
                                      ptr(cand_score), ptr(cand_idx), _stream(stream)))


def csa_shard_select(L, shards, cand_score, cand_idx, topk_idx, stream=None):
    _check(lib().csa_shard_select(ctypes.byref(L), shards, ptr(cand_score), ptr(cand_idx), ptr(topk_idx),
                                  _stream(stream)))


def csa_sparse_attend_partial(L, cache, params, q, q_pos, topk_idx, entry_offset, with_window, partial, workspace,
                              stream=None):
    _check(lib().csa_sparse_attend_partial(ctypes.byref(L), ctypes.byref(cache), ctypes.byref(params), ptr(q),
                                           ptr(q_pos), ptr(topk_idx), entry_offset, 1 if with_window else 0,
                                           ptr(partial), ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream)))


def csa_attend_merge(L, params, q_pos, parts, partials, out, stream=None):
    _check(lib().csa_attend_merge(ctypes.byref(L), ctypes.byref(params), ptr(q_pos), parts, ptr(partials), ptr(out),
                                  _stream(stream)))


# ----------------------------------------------------------------------------- paged 8-bit cache
# These calls run once per layer and token, and their kernels take microseconds: the checks are kept to one
# look at each tensor, and pointers go to the library as plain numbers.
_ACT = {0: torch.float32, 1: torch.bfloat16}


def _here(T):
    """The device of the table's tensors, which has to be the current one (a kernel elsewhere could not read them)."""
    d = T.device
    if d < 0 or d != torch._C._cuda_getDevice():
        raise CsaError(1, f"the page table is on device {d} (-1: the CPU), not on the current device")
    return d


def _arg(t, name, dtype, n, d):
    """Address of a contiguous tensor of at least n values on device d; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous() or t.get_device() != d:
        raise CsaError(1, f"{name} must be {n} contiguous {dtype} on device {d}")
    return t.data_ptr()


def _raw_stream(stream, d):
    return torch._C._cuda_getCurrentRawStream(d) if stream is None else stream.cuda_stream


def _paged_pool(G, pool, T):
    """Refuses a pool that is not the layer's or not the table's."""
    if pool.shape != (T.n_pages, G.Hkv, T.page, G.D):
        raise CsaError(1, f"pool of {pool.shape}, not {(T.n_pages, G.Hkv, T.page, G.D)} as the layer and the table say")
    if pool.device != T.device:
        raise CsaError(1, f"the pool is on device {pool.device}, the table on device {T.device}")


def _token_stride(t, name, G, B, Tq, heads, d=None):
    """Elements between the tokens of t [B, Tq, heads, D] (or [B, Tq, heads * D]), each token contiguous."""
    if t.dtype is not _ACT.get(G.act_format):
        raise CsaError(1, f"{name} is {t.dtype}, not the layer's activation type")
    if d is not None and t.get_device() != d:
        raise CsaError(1, f"{name} is on {t.device}, not on device {d}")
    D = G.D
    shape, st = tuple(t.shape), t.stride()
    if shape == (B, Tq, heads, D):
        inner = st[3] == 1 and (st[2] == D or heads == 1)
    elif shape == (B, Tq, heads * D):
        inner = st[2] == 1
    else:
        raise CsaError(1, f"{name} has shape {shape}, not {(B, Tq, heads, D)}")
    step = st[1] if Tq > 1 else (st[0] if B > 1 else heads * D)
    if not inner or step < heads * D or (B > 1 and st[0] != Tq * step):
        raise CsaError(1, f"{name}: tokens must be contiguous rows at one distance from each other")
    return step


def csa_paged_append(G, pool, T, k_new, v_new, start, n_new, Tq, stream=None):
    """k_new, v_new: [B, Tq, Hkv, D]; a view whose tokens lie at one distance (a slice of a fused projection) is
    taken as it is."""
    d, B = _here(T), T.B
    _paged_pool(G, pool, T)
    stride = _token_stride(k_new, "k_new", G, B, Tq, G.Hkv, d)
    if _token_stride(v_new, "v_new", G, B, Tq, G.Hkv, d) != stride:
        raise CsaError(1, "k_new and v_new have tokens at different distances")
    _check(lib().csa_paged_append(G, pool, T, k_new.data_ptr(), v_new.data_ptr(), stride,
                                  _arg(start, "start", torch.int64, B, d), _arg(n_new, "n_new", torch.int32, B, d), Tq,
                                  _raw_stream(stream, d)))


def csa_paged_workspace_size(G, T, Tq, n_max) -> int:
    return lib().csa_paged_workspace_size(G, T, Tq, n_max)


def csa_paged_attend(G, pool, T, q, sinks, start, n_new, Tq, n_max, out, workspace, stream=None):
    """q: [B, Tq, H, D] (tokens at one distance from each other); out: [B, Tq, H, D], contiguous."""
    d, B, H = _here(T), T.B, G.H
    _paged_pool(G, pool, T)
    stride = _token_stride(q, "q", G, B, Tq, H, d)
    if _token_stride(out, "out", G, B, Tq, H, d) != H * G.D:
        raise CsaError(1, "out must be contiguous")
    if workspace.get_device() != d:
        raise CsaError(1, f"the workspace is on {workspace.device}, not on device {d}")
    _check(lib().csa_paged_attend(G, pool, T, q.data_ptr(), stride, _arg(sinks, "sinks", torch.float32, H, d),
                                  _arg(start, "start", torch.int64, B, d), _arg(n_new, "n_new", torch.int32, B, d), Tq,
                                  n_max, out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                  _raw_stream(stream, d)))


def csa_debug_paged_join(G, T, sinks, start, n_new, Tq, n_max, out, workspace, stream=None):
    """The join of cut sequences alone, over what an earlier csa_paged_attend left in the workspace (test aid)."""
    d, B = _here(T), T.B
    if _token_stride(out, "out", G, B, Tq, G.H, d) != G.H * G.D:
        raise CsaError(1, "out must be contiguous")
    if workspace.get_device() != d:
        raise CsaError(1, f"the workspace is on {workspace.device}, not on device {d}")
    _check(lib().csa_debug_paged_join(G, T, _arg(sinks, "sinks", torch.float32, G.H, d),
                                      _arg(start, "start", torch.int64, B, d), _arg(n_new, "n_new", torch.int32, B, d),
                                      Tq, n_max, out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
                                      _raw_stream(stream, d)))


def csa_pages_fork(T, src, dst, n, stream=None):
    d = _here(T)
    _check(lib().csa_pages_fork(T, _arg(src, "src", torch.int32, n, d), _arg(dst, "dst", torch.int32, n, d), n,
                                _raw_stream(stream, d)))


def csa_pages_reserve(T, start, n_new, Tq, copy_src, copy_dst, missing, stream=None):
    d, B, i32 = _here(T), T.B, torch.int32
    _check(lib().csa_pages_reserve(T, _arg(start, "start", torch.int64, B, d), _arg(n_new, "n_new", i32, B, d), Tq,
                                   _arg(copy_src, "copy_src", i32, B, d), _arg(copy_dst, "copy_dst", i32, B, d),
                                   _arg(missing, "missing", i32, 1, d), _raw_stream(stream, d)))


def csa_pages_free(T, keep, begin, first, stream=None):
    d, B = _here(T), T.B
    _check(lib().csa_pages_free(T, _arg(keep, "keep", torch.int64, B, d), _arg(begin, "begin", torch.int64, B, d), first,
                                _raw_stream(stream, d)))


def csa_pages_compact(T, max_moves, move_src, move_dst, count, stream=None):
    d, i32 = _here(T), torch.int32
    _check(lib().csa_pages_compact(T, max_moves, _arg(move_src, "move_src", i32, max_moves, d),
                                   _arg(move_dst, "move_dst", i32, max_moves, d), _arg(count, "count", i32, 1, d),
                                   _raw_stream(stream, d)))


def csa_pages_copy(G, pool, T, src, dst, count, n, stream=None):
    d, i32 = _here(T), torch.int32
    _paged_pool(G, pool, T)
    _check(lib().csa_pages_copy(G, pool, T, _arg(src, "src", i32, n, d), _arg(dst, "dst", i32, n, d),
                                _arg(count, "count", i32, 1, d), n, _raw_stream(stream, d)))
