"""W4A16 Mixture-of-Experts expert layer for GB300 (sm_103a).

Thin Python binding of the C ABI in include/moe_w4.h. Every function here
only marshals arguments (device pointers from torch tensors, the current
CUDA stream) and raises MoeError on a non-zero status; all arithmetic runs
in the CUDA kernels of libmoe_w4.so. There is no CPU fallback: if the
library has not been built, load() raises.

Names follow the C ABI: moe_route, moe_plan, moe_expert_ffn_w4,
moe_combine, moe_layer_w4, moe_workspace_bytes, moe_max_blocks,
moe_workspace_init, moe_query_device_status, moe_debug_dequant_w4,
moe_debug_dequant_w4_decode; for one sequence moe_attn_decode, moe_gdn_scan,
moe_gdn_chunked_scan; for a batch of requests over one page pool
moe_cache_fork, moe_cache_reserve, moe_cache_write, moe_cache_compact (with
moved: moe_cache_compact_map), moe_cache_copy_pages, moe_attn_batch,
moe_verify_drafts, moe_token_logprobs; over a cache held in 4 bits
moe_cache_write_q4, moe_cache_read_q4, moe_attn_batch_q4.
"""
import ctypes as C
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmoe_w4.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SHAPE = 2
MOE_ERR_WORKSPACE = 3
MOE_ERR_CUDA = 4
MOE_ERR_BAD_INPUT = 5
MOE_ERR_TIMEOUT = 6

# moe_dtype_t
DTYPES = {"bf16": 0, "fp16": 1, "fp32": 2}
_DTYPE_OF = (torch.bfloat16, torch.float16, torch.float32)

EXPORTS = ("moe_workspace_bytes", "moe_max_blocks", "moe_workspace_init", "moe_route",
           "moe_plan", "moe_expert_ffn_w4", "moe_combine", "moe_layer_w4",
           "moe_query_device_status", "moe_debug_dequant_w4", "moe_debug_dequant_w4_decode",
           "moe_status_string",
           "moe_last_error", "moe_plan_noalloc", "moe_layer_path", "moe_decode_layers",
           "moe_decoder_blocks", "moe_attn_workspace_bytes", "moe_attn_decode",
           "moe_gdn_scan", "moe_gdn_chunked_workspace_bytes", "moe_gdn_chunked_scan",
           "moe_cache_workspace_bytes", "moe_cache_fork", "moe_cache_reserve", "moe_cache_write",
           "moe_cache_compact", "moe_cache_compact_map", "moe_cache_copy_pages",
           "moe_verify_workspace_bytes", "moe_verify_drafts", "moe_attn_batch_workspace_bytes", "moe_attn_batch",
           "moe_cache_q4_units", "moe_cache_write_q4", "moe_cache_read_q4",
           "moe_attn_batch_q4_workspace_bytes", "moe_attn_batch_q4",
           "moe_logprobs_workspace_bytes", "moe_token_logprobs")


class MoeError(RuntimeError):
    def __init__(self, status, where=""):
        self.status = status
        lib = _lib
        text = lib.moe_status_string(status).decode() if lib else str(status)
        detail = lib.moe_last_error().decode() if lib else ""
        super().__init__("%s: %s (%d)%s" % (where, text, status, (" - " + detail) if detail else ""))


class Shape(C.Structure):
    _fields_ = [("T", C.c_int32), ("H", C.c_int32), ("E", C.c_int32), ("K", C.c_int32),
                ("I", C.c_int32), ("n_shared", C.c_int32), ("tile_rows", C.c_int32)]

    def __repr__(self):
        return "Shape(T=%d, H=%d, E=%d, K=%d, I=%d, n_shared=%d, tile_rows=%d)" % (
            self.T, self.H, self.E, self.K, self.I, self.n_shared, self.tile_rows)


class AttnShape(C.Structure):
    _fields_ = [("T", C.c_int32), ("n_q", C.c_int32), ("n_kv", C.c_int32), ("D", C.c_int32),
                ("L", C.c_int32), ("block", C.c_int32)]


class GdnShape(C.Structure):
    _fields_ = [("T", C.c_int32), ("n_k", C.c_int32), ("n_v", C.c_int32), ("dk", C.c_int32),
                ("dv", C.c_int32)]


class CacheShape(C.Structure):
    _fields_ = [("n_slots", C.c_int32), ("max_blocks", C.c_int32), ("n_phys", C.c_int32),
                ("n_kv", C.c_int32), ("D", C.c_int32), ("block", C.c_int32)]


class CacheMetaPtrs(C.Structure):
    _fields_ = [("table", C.c_void_p), ("lens", C.c_void_p), ("refs", C.c_void_p)]


class AttnBatchShape(C.Structure):
    _fields_ = [("n_slots", C.c_int32), ("T", C.c_int32), ("n_q", C.c_int32), ("n_kv", C.c_int32),
                ("D", C.c_int32), ("block", C.c_int32), ("max_blocks", C.c_int32),
                ("prefix_blocks", C.c_int32), ("dtype", C.c_int32)]


class VerifyShape(C.Structure):
    _fields_ = [("n_slots", C.c_int32), ("T", C.c_int32), ("V", C.c_int32), ("dtype", C.c_int32)]


class LogprobsShape(C.Structure):
    _fields_ = [("n_rows", C.c_int32), ("V", C.c_int32), ("k", C.c_int32), ("dtype", C.c_int32)]


class W4Weights(C.Structure):
    _fields_ = [("q_gate_up", C.c_void_p), ("s_gate_up", C.c_void_p), ("b_gate_up", C.c_void_p),
                ("q_down", C.c_void_p), ("s_down", C.c_void_p), ("b_down", C.c_void_p)]


class LayerWeights(C.Structure):
    _fields_ = [("w_router", C.c_void_p), ("router_bias", C.c_void_p),
                ("experts", W4Weights), ("shared", W4Weights)]


class PlanPtrs(C.Structure):
    _fields_ = [("counts", C.c_void_p), ("offsets", C.c_void_p), ("sorted_rows", C.c_void_p),
                ("row_pos", C.c_void_p), ("block_map", C.c_void_p), ("num_blocks", C.c_void_p)]


_lib = None
_lock = threading.Lock()


def load():
    """Load libmoe_w4.so (built by __graft_entry__.build()); raises if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise FileNotFoundError(
                    "libmoe_w4.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
            L = C.CDLL(LIB_PATH)
            P, I32, SZ = C.c_void_p, C.c_int32, C.c_size_t
            pS, pW, pP = C.POINTER(Shape), C.POINTER(W4Weights), C.POINTER(PlanPtrs)
            L.moe_workspace_bytes.restype = SZ
            L.moe_workspace_bytes.argtypes = [pS]
            L.moe_max_blocks.restype = I32
            L.moe_max_blocks.argtypes = [pS]
            L.moe_layer_path.restype = I32
            L.moe_layer_path.argtypes = [pS]
            L.moe_gdn_chunked_workspace_bytes.restype = SZ
            L.moe_gdn_chunked_workspace_bytes.argtypes = [C.POINTER(GdnShape)]
            L.moe_attn_workspace_bytes.restype = SZ
            L.moe_attn_workspace_bytes.argtypes = [C.POINTER(AttnShape)]
            pC, pM, pV = C.POINTER(CacheShape), C.POINTER(CacheMetaPtrs), C.POINTER(VerifyShape)
            L.moe_cache_workspace_bytes.restype = SZ
            L.moe_cache_workspace_bytes.argtypes = [pC]
            L.moe_verify_workspace_bytes.restype = SZ
            L.moe_verify_workspace_bytes.argtypes = [pV]
            pA = C.POINTER(AttnBatchShape)
            L.moe_attn_batch_workspace_bytes.restype = SZ
            L.moe_attn_batch_workspace_bytes.argtypes = [pA]
            L.moe_attn_batch_q4_workspace_bytes.restype = SZ
            L.moe_attn_batch_q4_workspace_bytes.argtypes = [pA]
            pL = C.POINTER(LogprobsShape)
            L.moe_logprobs_workspace_bytes.restype = SZ
            L.moe_logprobs_workspace_bytes.argtypes = [pL]
            L.moe_cache_q4_units.restype = I32
            L.moe_cache_q4_units.argtypes = [I32]
            I64 = C.c_int64
            for name, args in (
                    ("moe_workspace_init", [P, SZ, P]),
                    ("moe_route", [pS, P, P, P, P, P, P, SZ, P]),
                    ("moe_plan", [pS, P, pP, P, SZ, P]),
                    ("moe_expert_ffn_w4", [pS, P, pW, pW, pP, P, P, SZ, P]),
                    ("moe_combine", [pS, P, P, P, P, P, P]),
                    ("moe_layer_w4", [pS, P, P, P, pW, pW, P, P, P, P, P, SZ, P]),
                    ("moe_query_device_status", [P, SZ, P]),
                    ("moe_debug_dequant_w4", [P, P, P, P, I32, I32, P]),
                    ("moe_debug_dequant_w4_decode", [P, P, P, P, I32, I32, P]),
                    ("moe_plan_noalloc", [pS, P, pP, P]),
                    ("moe_decode_layers", [pS, I32, P, P, P, P, P, SZ, P]),
                    ("moe_decoder_blocks", [pS, I32, P, P, P, P, P, I32, P, P, SZ, P]),
                    ("moe_attn_decode", [C.POINTER(AttnShape), P, P, P, P, I32, P, P, SZ, P]),
                    ("moe_gdn_scan", [C.POINTER(GdnShape), P, P, P, P, P, P, P, P, P]),
                    ("moe_gdn_chunked_scan",
                     [C.POINTER(GdnShape), P, P, P, P, P, P, P, P, P, SZ, P]),
                    ("moe_cache_fork", [pC, pM, P, P, pM, P, SZ, P]),
                    ("moe_cache_reserve", [pC, pM, P, pM, P, P, I32, P, SZ, P]),
                    ("moe_cache_write", [pC, pM, P, I32, P, I64, P, I64, P, P, P, SZ, P]),
                    ("moe_cache_compact", [pC, pM, pM, P, P, I32, P, SZ, P]),
                    ("moe_cache_compact_map", [pC, pM, pM, P, P, P, I32, P, SZ, P]),
                    ("moe_cache_copy_pages", [pC, I32, P, P, P, P, I32, I32, P, SZ, P]),
                    ("moe_attn_batch", [pA, P, I64, P, P, I32, P, P, P, P, P, P, SZ, P]),
                    ("moe_cache_write_q4",
                     [pC, pM, P, I32, I32, P, I64, P, I64, P, P, P, SZ, P]),
                    ("moe_cache_read_q4",
                     [pC, pM, P, P, I32, P, P, I32, P, I64, P, I64, P, SZ, P]),
                    ("moe_attn_batch_q4", [pA, P, I64, P, P, I32, P, P, P, P, P, SZ, P]),
                    ("moe_token_logprobs", [pL, P, I64, P, P, P, P, P, P, SZ, P]),
                    ("moe_verify_drafts", [pV, P, P, P, P, P, P, P, P, SZ, P])):
                f = getattr(L, name)
                f.restype = C.c_int
                f.argtypes = args
            L.moe_status_string.restype = C.c_char_p
            L.moe_status_string.argtypes = [C.c_int]
            L.moe_last_error.restype = C.c_char_p
            L.moe_last_error.argtypes = []
            _lib = L
    return _lib


def _check(status, where):
    if status != MOE_OK:
        raise MoeError(status, where)


def _p(t):
    """Device pointer of a CUDA tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return C.c_void_p(t.data_ptr())


def _s(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def make_shape(T, H, E, K, I, n_shared=1, tile_rows=128):
    return Shape(T, H, E, K, I, n_shared, tile_rows)


def moe_workspace_bytes(shape):
    return load().moe_workspace_bytes(C.byref(shape))


def moe_max_blocks(shape):
    return load().moe_max_blocks(C.byref(shape))


def moe_layer_path(shape):
    """1: moe_layer_w4 runs the fused decode kernels; 0: the four calls; -1: bad shape."""
    return load().moe_layer_path(C.byref(shape))


def moe_workspace_init(ws, stream=None):
    _check(load().moe_workspace_init(_p(ws), ws.numel() * ws.element_size(), _s(stream)),
           "moe_workspace_init")


def moe_route(shape, x, w_router, router_bias, topk_ids, topk_w, ws, stream=None):
    _check(load().moe_route(C.byref(shape), _p(x), _p(w_router), _p(router_bias), _p(topk_ids),
                            _p(topk_w), _p(ws), ws.numel(), _s(stream)), "moe_route")


def moe_plan(shape, topk_ids, plan, ws, stream=None):
    _check(load().moe_plan(C.byref(shape), _p(topk_ids), C.byref(plan.ptrs), _p(ws), ws.numel(),
                           _s(stream)), "moe_plan")


def moe_expert_ffn_w4(shape, x, experts, shared, plan, y_slots, ws, stream=None):
    _check(load().moe_expert_ffn_w4(C.byref(shape), _p(x), C.byref(experts.ptrs),
                                    C.byref(shared.ptrs) if shared is not None else None,
                                    C.byref(plan.ptrs), _p(y_slots), _p(ws), ws.numel(),
                                    _s(stream)), "moe_expert_ffn_w4")


def moe_plan_noalloc(shape, topk_ids, plan, stream=None):
    """moe_plan without a workspace (static device scratch; see moe_w4.h)."""
    _check(load().moe_plan_noalloc(C.byref(shape), _p(topk_ids), C.byref(plan.ptrs), _s(stream)),
           "moe_plan_noalloc")


def moe_combine(shape, y_slots, row_pos, topk_w, y, x_next=None, stream=None):
    _check(load().moe_combine(C.byref(shape), _p(y_slots), _p(row_pos), _p(topk_w), _p(y),
                              _p(x_next), _s(stream)), "moe_combine")


def decode_layer_table(layers):
    """Host array of moe_layer_weights_t from (w_router, router_bias or None,
    experts, shared or None) tuples; keep it alive while it is used."""
    arr = (LayerWeights * len(layers))()
    for i, (wr, bias, ex, sh) in enumerate(layers):
        arr[i].w_router = _p(wr)
        arr[i].router_bias = _p(bias)
        arr[i].experts = ex.ptrs
        if sh is not None:
            arr[i].shared = sh.ptrs
    return arr


def moe_decode_layers(shape, layer_table, x, y, ws, x_next=None, stream=None):
    """n stacked decode layers (layer_table from decode_layer_table)."""
    _check(load().moe_decode_layers(C.byref(shape), len(layer_table),
                                    C.cast(layer_table, C.c_void_p), _p(x), _p(y), _p(x_next),
                                    _p(ws), ws.numel(), _s(stream)), "moe_decode_layers")


def make_attn_shape(T, n_q, n_kv, D, L, block=64):
    return AttnShape(T, n_q, n_kv, D, L, block)


def alloc_attn_workspace(shape, device="cuda", stream=None):
    n = load().moe_attn_workspace_bytes(C.byref(shape))
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "alloc_attn_workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def moe_attn_decode(shape, q, k_cache, v_cache, table, o, ws, stream=None):
    """Grouped-query decode attention over a block-paged key/value cache."""
    _check(load().moe_attn_decode(C.byref(shape), _p(q), _p(k_cache), _p(v_cache), _p(table),
                                  k_cache.shape[0], _p(o), _p(ws), ws.numel(), _s(stream)),
           "moe_attn_decode")


def make_gdn_shape(T, n_k, n_v, dk, dv):
    return GdnShape(T, n_k, n_v, dk, dv)


def moe_gdn_scan(shape, q, k, v, alpha, beta, state_in, state_out, o, stream=None):
    """Gated delta rule over shape.T tokens (state_out may be state_in)."""
    _check(load().moe_gdn_scan(C.byref(shape), _p(q), _p(k), _p(v), _p(alpha), _p(beta),
                               _p(state_in), _p(state_out), _p(o), _s(stream)), "moe_gdn_scan")


def alloc_gdn_workspace(shape, device):
    """Device workspace of the chunked scan (moe_gdn_chunked_workspace_bytes),
    zero-filled: its status header must start at zero."""
    nbytes = load().moe_gdn_chunked_workspace_bytes(C.byref(shape))
    if nbytes == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_gdn_chunked_workspace_bytes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def moe_gdn_chunked_scan(shape, q, k, v, alpha, beta, state_in, state_out, o, ws, stream=None):
    """Chunked (parallel) form of the gated delta rule; same results as
    moe_gdn_scan within fp32 rounding (state_out may be state_in)."""
    _check(load().moe_gdn_chunked_scan(C.byref(shape), _p(q), _p(k), _p(v), _p(alpha), _p(beta),
                                       _p(state_in), _p(state_out), _p(o), _p(ws),
                                       ws.numel() * ws.element_size(), _s(stream)),
           "moe_gdn_chunked_scan")


def gain_table(gains):
    """Host array of device pointers to per-layer bf16 [H] gains; keep it
    alive while it is used."""
    arr = (C.c_void_p * len(gains))()
    for i, g in enumerate(gains):
        arr[i] = _p(g)
    return arr


def moe_decoder_blocks(shape, layer_table, gains, h_out, ws, h_in=None, token_ids=None,
                     embed=None, stream=None):
    """n decoder blocks (pre-norm with gain, MoE layer, residual add); h_0 is
    h_in, or the rows of embed named by the device token ids."""
    if len(gains) != len(layer_table):
        raise ValueError("one gain table entry per layer")
    vocab = embed.shape[0] if embed is not None else 0
    _check(load().moe_decoder_blocks(C.byref(shape), len(layer_table),
                                   C.cast(layer_table, C.c_void_p), C.cast(gains, C.c_void_p),
                                   _p(h_in), _p(token_ids), _p(embed), vocab, _p(h_out),
                                   _p(ws), ws.numel(), _s(stream)), "moe_decoder_blocks")


# ------------------------------------------------- batch serving calls --
# A call of a few microseconds on the GPU must not wait for its checks: the
# helpers look at each tensor once, hand plain integers to ctypes and take
# the stream's handle without building a Stream object.
def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _bad(t, what, dtype, shape):
    raise ValueError("%s must be a contiguous CUDA tensor %s %s, got %s %s%s" % (
        what, dtype, shape, t.dtype, tuple(t.shape), "" if t.is_cuda else " on the host"))


def _ints(t, shape, what):
    """Address of a contiguous int32 CUDA tensor of this shape (None: 0)."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(t, what, "int32", shape)
    return t.data_ptr()


def _tensor(t, dtype, shape, what):
    """Address of a contiguous CUDA tensor of this type and shape; bf16 and
    fp16 tensors may come as int16 bits."""
    if (t.dtype is not dtype and not (dtype.itemsize == 2 and t.dtype is torch.int16)) or \
            t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(t, what, dtype, shape)
    return t.data_ptr()


def _tokens(t, shape, what):
    """Address and token stride (elements) of a 16-bit [n_slots][T][heads][D]
    tensor whose tokens lie evenly apart, each dense (a slice of a joint
    projection is)."""
    if t.shape != shape or not t.is_cuda or t.element_size() != 2:
        _bad(t, what, "of 16 bits", shape)
    n_slots, T, heads, D = shape
    s0, s1, s2, s3 = t.stride()
    if (D > 1 and s3 != 1) or (heads > 1 and s2 != D):
        raise ValueError("%s: a token's elements must be dense" % what)
    stride = s1 if T > 1 else s0 if n_slots > 1 else heads * D
    if T > 1 and n_slots > 1 and s0 != T * stride:
        raise ValueError("%s: tokens must lie evenly apart" % what)
    return t.data_ptr(), stride


def _ws(ws):
    if ws.dtype is not torch.uint8 or not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous uint8 CUDA tensor")
    return ws.data_ptr()


def _workspace(nbytes, device, stream, what):
    if nbytes == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, what)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws


def make_cache_shape(n_slots, max_blocks, n_phys, n_kv, D, block=64):
    return CacheShape(n_slots, max_blocks, n_phys, n_kv, D, block)


def alloc_cache_workspace(shape, device="cuda", stream=None):
    return _workspace(load().moe_cache_workspace_bytes(C.byref(shape)), device, stream,
                      "alloc_cache_workspace")


class CacheMeta:
    """State of a batch's cache (moe_cache_meta_t): table int32
    [n_slots][max_blocks], lens int32 [n_slots], refs int32 [n_phys]. The
    calls read one and write another; a program keeps two and swaps them.
    The addresses are taken once, so the tensors can be changed in place but
    not exchanged for others."""

    def __init__(self, table, lens, refs):
        if table.dim() != 2 or refs.dim() != 1:
            raise ValueError("table is [n_slots][max_blocks], refs [n_phys]")
        self._tensors = table, lens, refs
        self.ptrs = CacheMetaPtrs(_ints(table, table.shape, "table"),
                                  _ints(lens, table.shape[:1], "lens"),
                                  _ints(refs, refs.shape, "refs"))
        self._dims = tuple(table.shape) + tuple(refs.shape)
        self._ref = C.byref(self.ptrs)

    table = property(lambda self: self._tensors[0])
    lens = property(lambda self: self._tensors[1])
    refs = property(lambda self: self._tensors[2])

    @classmethod
    def empty(cls, shape, device="cuda"):
        """No slot holds anything, every page is free."""
        z = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        return cls(z(shape.n_slots, shape.max_blocks).fill_(-1), z(shape.n_slots), z(shape.n_phys))

    def of(self, shape):
        if self._dims != (shape.n_slots, shape.max_blocks, shape.n_phys):
            raise ValueError("the state is not of this cache shape")
        return self._ref


def pool_table(pools):
    """Host array of the pools' device pointers (16-bit [n_phys][n_kv][64][D]
    each) for moe_cache_reserve, moe_cache_compact and moe_cache_copy_pages;
    it keeps the tensors, whose addresses it has taken."""
    arr = (C.c_void_p * max(1, len(pools)))()
    for i, t in enumerate(pools):
        if t.dim() != 4:
            raise ValueError("pools are [n_phys][n_kv][64][D]")
        arr[i] = _pool(t, pools[0].shape, "every pool")
    arr.pools = tuple(pools)
    return arr


def _pools(shape, table, n_phys):
    n = len(table.pools)
    if n and table.pools[0].shape != (n_phys, shape.n_kv, shape.block, shape.D):
        raise ValueError("the pools are not of this cache shape")
    return C.addressof(table), n


def moe_cache_fork(shape, meta, parent, out, ws, keep=None, stream=None):
    """Slot s of `out` holds the first keep[s] positions of slot parent[s] of
    `meta` (-1: nothing): fork, reorder, cut and free."""
    n = (shape.n_slots,)
    _check((_lib or load()).moe_cache_fork(
        shape, meta.of(shape), _ints(parent, n, "parent"), _ints(keep, n, "keep"), out.of(shape),
        _ws(ws), ws.numel(), _raw_stream(stream)), "moe_cache_fork")


def moe_cache_reserve(shape, meta, n_new, out, granted, pools, ws, stream=None):
    """Room for n_new[s] positions more in every slot, shared last pages copied
    in all pools (pool_table); granted[s] = n_new[s], or 0 where refused."""
    n = (shape.n_slots,)
    ptr, k = _pools(shape, pools, shape.n_phys)
    _check((_lib or load()).moe_cache_reserve(
        shape, meta.of(shape), _ints(n_new, n, "n_new"), out.of(shape),
        _ints(granted, n, "granted"), ptr, k, _ws(ws), ws.numel(), _raw_stream(stream)),
        "moe_cache_reserve")


def moe_cache_write(shape, meta, n_new, k_new, v_new, k_cache, v_cache, ws, stream=None):
    """Keys and values [n_slots][T][n_kv][D] of the last n_new[s] positions
    (None: T) of every slot into one layer's pools of their type."""
    B, n_kv, D = shape.n_slots, shape.n_kv, shape.D
    new = (B, k_new.shape[1], n_kv, D)
    kp, ks = _tokens(k_new, new, "k_new")
    vp, vs = _tokens(v_new, new, "v_new")
    cache = (shape.n_phys, n_kv, shape.block, D)
    _alike(k_new, k_cache, "k_new and k_cache")
    _alike(v_new, v_cache, "v_new and v_cache")
    _check((_lib or load()).moe_cache_write(
        shape, meta.of(shape), _ints(n_new, (B,), "n_new"), new[1], kp, ks, vp, vs,
        _pool(k_cache, cache, "k_cache"), _pool(v_cache, cache, "v_cache"), _ws(ws), ws.numel(),
        _raw_stream(stream)), "moe_cache_write")


def _alike(a, b, what):
    """Rows are copied as they are: one type, or int16 bits on either side."""
    if a.dtype is not b.dtype and torch.int16 not in (a.dtype, b.dtype):
        raise ValueError("%s must be of one type, got %s and %s" % (what, a.dtype, b.dtype))


def _pool(t, shape, what):
    if t.shape != shape or t.element_size() != 2 or not t.is_cuda or not t.is_contiguous():
        _bad(t, what, "of 16 bits", shape)
    return t.data_ptr()


def moe_cache_compact(shape, meta, out, n_live, pools, ws, stream=None, moved=None):
    """Moves the held pages to the front of every pool; n_live[0] = how many.
    moved (int32 [n_phys], or None): each held page's new number, -1 for a free
    one. Page numbers kept outside the tables (a `prefix` of moe_attn_batch,
    pinned pages) are moved[old] from here on."""
    ptr, k = _pools(shape, pools, shape.n_phys)
    _check((_lib or load()).moe_cache_compact_map(
        shape, meta.of(shape), out.of(shape), _ints(n_live, (1,), "n_live"),
        _ints(moved, (shape.n_phys,), "moved"), ptr, k, _ws(ws), ws.numel(), _raw_stream(stream)),
        "moe_cache_compact")


def moe_cache_copy_pages(shape, src, dst, from_pools, to_pools, ws, stream=None):
    """Page src[i] of every pool of from_pools to page dst[i] of to_pools."""
    if not from_pools.pools or len(from_pools.pools) != len(to_pools.pools):
        raise ValueError("as many pools on both sides, one at least")
    for a, b in zip(from_pools.pools, to_pools.pools):
        _alike(a, b, "a pool and the one it is copied to")
    n_to = to_pools.pools[0].shape[0]
    a, k = _pools(shape, from_pools, shape.n_phys)
    b, _ = _pools(shape, to_pools, n_to)
    n = src.shape[:1]
    _check((_lib or load()).moe_cache_copy_pages(
        shape, n[0], _ints(src, n, "src"), _ints(dst, n, "dst"), a, b, k, n_to, _ws(ws),
        ws.numel(), _raw_stream(stream)), "moe_cache_copy_pages")


def make_attn_batch_shape(n_slots, T, n_q, n_kv, D, max_blocks, prefix_blocks=0, dtype="bf16",
                          block=64):
    return AttnBatchShape(n_slots, T, n_q, n_kv, D, block, max_blocks, prefix_blocks, DTYPES[dtype])


def alloc_attn_batch_workspace(shape, device="cuda", stream=None):
    return _workspace(load().moe_attn_batch_workspace_bytes(C.byref(shape)), device, stream,
                      "alloc_attn_batch_workspace")


def moe_attn_batch(shape, q, k_cache, v_cache, table, lens, o, ws, n_new=None, prefix=None,
                   stream=None):
    """Decode attention of every slot's last n_new[s] (None: T) tokens over its
    pages; the first shape.prefix_blocks blocks of all slots are the pages
    `prefix`, read once for the batch. q [n_slots][T][n_q][D] may be a slice
    of a joint projection; o is dense."""
    B, T, nq, D = shape.n_slots, shape.T, shape.n_q, shape.D
    dt = torch.float16 if shape.dtype == 1 else torch.bfloat16
    if q.dtype is not dt and q.dtype is not torch.int16:
        raise ValueError("q must be %s, got %s" % (dt, q.dtype))
    qp, qs = _tokens(q, (B, T, nq, D), "q")
    n_phys = k_cache.shape[0]
    cache = (n_phys, shape.n_kv, shape.block, D)
    _check((_lib or load()).moe_attn_batch(
        shape, qp, qs, _tensor(k_cache, dt, cache, "k_cache"),
        _tensor(v_cache, dt, cache, "v_cache"), n_phys, _ints(table, (B, shape.max_blocks), "table"),
        _ints(prefix, (shape.prefix_blocks,), "prefix"), _ints(lens, (B,), "lens"),
        _ints(n_new, (B,), "n_new"), _tensor(o, dt, (B, T, nq, D), "o"), _ws(ws), ws.numel(),
        _raw_stream(stream)), "moe_attn_batch")


def make_verify_shape(n_slots, T, V, dtype="fp32"):
    return VerifyShape(n_slots, T, V, DTYPES[dtype])


def alloc_verify_workspace(shape, device="cuda", stream=None):
    return _workspace(load().moe_verify_workspace_bytes(C.byref(shape)), device, stream,
                      "alloc_verify_workspace")


def moe_verify_drafts(shape, p, q, draft, n_draft, u, tokens, n_acc, ws, stream=None):
    """Accepts drafted tokens against the target's probabilities p
    [n_slots][T+1][V] and the draft's q [n_slots][T][V] (None: certain) with
    the random numbers u [n_slots][T+1], and draws the token after them."""
    B, T, V = shape.n_slots, shape.T, shape.V
    dt = _DTYPE_OF[shape.dtype]
    _check((_lib or load()).moe_verify_drafts(
        shape, _tensor(p, dt, (B, T + 1, V), "p"),
        None if q is None else _tensor(q, dt, (B, T, V), "q"), _ints(draft, (B, T), "draft"),
        _ints(n_draft, (B,), "n_draft"), _tensor(u, torch.float32, (B, T + 1), "u"),
        _ints(tokens, (B, T + 1), "tokens"), _ints(n_acc, (B,), "n_acc"), _ws(ws), ws.numel(),
        _raw_stream(stream)), "moe_verify_drafts")


# --------------------------------------------------- a cache held in 4 bits --
_Q4_UNITS = {}  # by D, as the library gives them


def moe_cache_q4_units(D):
    """16-bit units of a head's 4-bit row: 40 for D = 128, 24 for D = 64."""
    n = _Q4_UNITS.get(D)
    if n is None:
        n = load().moe_cache_q4_units(D)
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "moe_cache_q4_units")
        _Q4_UNITS[D] = n
    return n


def q4_page_shape(shape):
    """The cache shape under which the page calls (moe_cache_reserve,
    moe_cache_compact, moe_cache_copy_pages) move the 4-bit pools of `shape`."""
    return CacheShape(shape.n_slots, shape.max_blocks, shape.n_phys, shape.n_kv,
                      moe_cache_q4_units(shape.D), shape.block)


def alloc_q4_pool(shape, device="cuda"):
    """A pool of 4-bit rows, int16 [n_phys][n_kv][64][units] (uninitialised)."""
    return torch.empty((shape.n_phys, shape.n_kv, shape.block, moe_cache_q4_units(shape.D)),
                       dtype=torch.int16, device=device)


def _q4_pool(t, shape, what):
    if t.dtype is not torch.int16 or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(t, what, "int16", shape)
    return t.data_ptr()


def _rows_of(t, shape, dtype, what):
    """As _tokens, for outputs and rows of any element size."""
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda:
        _bad(t, what, dtype, shape)
    n_slots, T, heads, D = shape
    s0, s1, s2, s3 = t.stride()
    if s3 != 1 or (heads > 1 and s2 != D):
        raise ValueError("%s: a token's elements must be dense" % what)
    stride = s1 if T > 1 else s0 if n_slots > 1 else heads * D
    if T > 1 and n_slots > 1 and s0 != T * stride:
        raise ValueError("%s: tokens must lie evenly apart" % what)
    return t.data_ptr(), stride


def moe_cache_write_q4(shape, meta, n_new, k_new, v_new, k_cache, v_cache, ws, stream=None):
    """moe_cache_write into 4-bit pools (alloc_q4_pool): bf16 or fp16 rows
    [n_slots][T][n_kv][D] are quantised as they are written."""
    B, n_kv, D = shape.n_slots, shape.n_kv, shape.D
    dt = k_new.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError("k_new must be bfloat16 or float16, got %s" % dt)
    new = (B, k_new.shape[1], n_kv, D)
    kp, ks = _rows_of(k_new, new, dt, "k_new")
    vp, vs = _rows_of(v_new, new, dt, "v_new")
    cache = (shape.n_phys, n_kv, shape.block, moe_cache_q4_units(D))
    _check((_lib or load()).moe_cache_write_q4(
        shape, meta.of(shape), _ints(n_new, (B,), "n_new"), new[1], _DTYPE_OF.index(dt), kp, ks,
        vp, vs, _q4_pool(k_cache, cache, "k_cache"), _q4_pool(v_cache, cache, "v_cache"), _ws(ws),
        ws.numel(), _raw_stream(stream)), "moe_cache_write_q4")


def moe_cache_read_q4(shape, meta, first, n, k_cache, v_cache, k_out, v_out, ws, stream=None):
    """What positions first[s] .. first[s] + n[s] - 1 (None: from 0; T of them)
    of every slot stand for, to k_out and v_out [n_slots][T][n_kv][D] (bf16,
    fp16 or fp32); tokens from n[s] on stay as they were."""
    B, n_kv, D = shape.n_slots, shape.n_kv, shape.D
    dt = k_out.dtype
    if dt not in _DTYPE_OF:
        raise ValueError("k_out must be bfloat16, float16 or float32, got %s" % dt)
    out = (B, k_out.shape[1], n_kv, D)
    kp, ks = _rows_of(k_out, out, dt, "k_out")
    vp, vs = _rows_of(v_out, out, dt, "v_out")
    cache = (shape.n_phys, n_kv, shape.block, moe_cache_q4_units(D))
    _check((_lib or load()).moe_cache_read_q4(
        shape, meta.of(shape), _ints(first, (B,), "first"), _ints(n, (B,), "n"), out[1],
        _q4_pool(k_cache, cache, "k_cache"), _q4_pool(v_cache, cache, "v_cache"),
        _DTYPE_OF.index(dt), kp, ks, vp, vs, _ws(ws), ws.numel(), _raw_stream(stream)),
        "moe_cache_read_q4")


def alloc_attn_batch_q4_workspace(shape, device="cuda", stream=None):
    return _workspace(load().moe_attn_batch_q4_workspace_bytes(C.byref(shape)), device, stream,
                      "alloc_attn_batch_q4_workspace")


def moe_attn_batch_q4(shape, q, k_cache, v_cache, table, lens, o, ws, n_new=None, stream=None):
    """moe_attn_batch over 4-bit pools (shape.prefix_blocks is 0: pages that
    slots share stand in their tables, and each slot reads them)."""
    B, T, nq, D = shape.n_slots, shape.T, shape.n_q, shape.D
    dt = torch.float16 if shape.dtype == 1 else torch.bfloat16
    if q.dtype is not dt and q.dtype is not torch.int16:
        raise ValueError("q must be %s, got %s" % (dt, q.dtype))
    qp, qs = _tokens(q, (B, T, nq, D), "q")
    n_phys = k_cache.shape[0]
    cache = (n_phys, shape.n_kv, shape.block, moe_cache_q4_units(D))
    _check((_lib or load()).moe_attn_batch_q4(
        shape, qp, qs, _q4_pool(k_cache, cache, "k_cache"), _q4_pool(v_cache, cache, "v_cache"),
        n_phys, _ints(table, (B, shape.max_blocks), "table"), _ints(lens, (B,), "lens"),
        _ints(n_new, (B,), "n_new"), _tensor(o, dt, (B, T, nq, D), "o"), _ws(ws), ws.numel(),
        _raw_stream(stream)), "moe_attn_batch_q4")


# ----------------------------------------------------- log probabilities --
def make_logprobs_shape(n_rows, V, k=0, dtype="fp32"):
    return LogprobsShape(n_rows, V, k, DTYPES[dtype])


def alloc_logprobs_workspace(shape, device="cuda", stream=None):
    return _workspace(load().moe_logprobs_workspace_bytes(C.byref(shape)), device, stream,
                      "alloc_logprobs_workspace")


def moe_token_logprobs(shape, logits, tokens, logp, ws, entropy=None, top_ids=None, top_logp=None,
                       stream=None):
    """Log probabilities of tokens [n_rows] (-1: none) under logits
    [n_rows][V] (rows may lie apart), the rows' entropies and their shape.k
    likeliest ids with log probabilities [n_rows][k]."""
    n, V, k = shape.n_rows, shape.V, shape.k
    dt, f32 = _DTYPE_OF[shape.dtype], torch.float32
    if logits.dtype is not dt or logits.shape != (n, V) or not logits.is_cuda or \
            (V > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor %s %s with dense rows, got %s %s" % (
            dt, (n, V), logits.dtype, tuple(logits.shape)))
    stride = logits.stride(0) if n > 1 else V
    _check((_lib or load()).moe_token_logprobs(
        shape, logits.data_ptr(), stride, _ints(tokens, (n,), "tokens"),
        _tensor(logp, f32, (n,), "logp"),
        None if entropy is None else _tensor(entropy, f32, (n,), "entropy"),
        _ints(top_ids, (n, k), "top_ids"),
        None if top_logp is None else _tensor(top_logp, f32, (n, k), "top_logp"), _ws(ws),
        ws.numel(), _raw_stream(stream)), "moe_token_logprobs")


def moe_layer_w4(shape, x, w_router, router_bias, experts, shared, y, ws, x_next=None,
                 topk_ids=None, topk_w=None, stream=None):
    _check(load().moe_layer_w4(C.byref(shape), _p(x), _p(w_router), _p(router_bias),
                               C.byref(experts.ptrs),
                               C.byref(shared.ptrs) if shared is not None else None,
                               _p(y), _p(x_next), _p(topk_ids), _p(topk_w), _p(ws), ws.numel(),
                               _s(stream)), "moe_layer_w4")


def moe_query_device_status(ws, stream=None):
    """Synchronises the stream; returns the device status code (and clears it)."""
    return load().moe_query_device_status(_p(ws), ws.numel(), _s(stream))


def moe_debug_dequant_w4(q, s, b, out, stream=None):
    N, K8 = q.shape
    _check(load().moe_debug_dequant_w4(_p(q), _p(s), _p(b), _p(out), N, K8 * 8, _s(stream)),
           "moe_debug_dequant_w4")


def moe_debug_dequant_w4_decode(q, s, b, out, stream=None):
    N, K8 = q.shape
    _check(load().moe_debug_dequant_w4_decode(_p(q), _p(s), _p(b), _p(out), N, K8 * 8,
                                              _s(stream)),
           "moe_debug_dequant_w4_decode")


# ----------------------------------------------------- device-side holders --
class ExpertWeights:
    """Packed 4-bit weights of n experts resident on the device (layouts of
    moe_w4_weights_t); bf16 arrays are kept as int16 storage."""

    def __init__(self, q_gate_up, s_gate_up, b_gate_up, q_down, s_down, b_down):
        self.tensors = (q_gate_up, s_gate_up, b_gate_up, q_down, s_down, b_down)
        for t in self.tensors:
            if not (t.is_cuda and t.is_contiguous()):
                raise ValueError("expert weights must be contiguous CUDA tensors")
        self.ptrs = W4Weights(*[t.data_ptr() for t in self.tensors])

    @classmethod
    def from_numpy(cls, q_gate_up, s_gate_up, b_gate_up, q_down, s_down, b_down, device="cuda"):
        def dev(a):
            a = a.view("int32") if a.dtype.itemsize == 4 else a.view("int16")
            return torch.from_numpy(a.copy()).to(device)
        return cls(*[dev(a) for a in (q_gate_up, s_gate_up, b_gate_up, q_down, s_down, b_down)])

    @property
    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in self.tensors)


class PlanBuffers:
    """Caller-owned plan buffers (moe_plan_t) for one shape."""

    def __init__(self, shape, device="cuda"):
        R = shape.T * shape.K
        mb = moe_max_blocks(shape)
        z = lambda n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        self.counts = z(shape.E)
        self.offsets = z(shape.E + 1)
        self.sorted_rows = z(R)
        self.row_pos = z(R)
        self.block_map = z(mb * 3)
        self.num_blocks = z(1)
        self.ptrs = PlanPtrs(*[t.data_ptr() for t in (self.counts, self.offsets, self.sorted_rows,
                                                      self.row_pos, self.block_map,
                                                      self.num_blocks)])


def alloc_workspace(shape, device="cuda", stream=None):
    n = moe_workspace_bytes(shape)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED_SHAPE, "alloc_workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    moe_workspace_init(ws, stream)
    return ws
