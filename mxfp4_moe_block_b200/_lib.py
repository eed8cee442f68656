"""ctypes binding of libmxfp4_moe.so (declared in include/mxfp4_moe.h).

Argument marshalling only: every step of the path runs in the library's
CUDA kernels.  Torch supplies device memory and the current stream.  There
is no fallback: if the shared library is missing, or a tensor is not on a
CUDA device, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# MXFP4_MOE_CHECKS=1: the checked build (every caller-supplied index tested
# on the device before use; see build.py)
LIB_PATH = os.path.join(HERE, "libmxfp4_moe_checks.so" if os.environ.get("MXFP4_MOE_CHECKS") == "1"
                        else "libmxfp4_moe.so")

MOE_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error",
                4: "workspace", 5: "device status"}
# device status details (second value of moe_get_device_status)
DEV_OK, DEV_BAD_EXPERT, DEV_NO_MASS, DEV_BAD_TOKEN, DEV_TIMEOUT, DEV_BAD_INDEX = 0, 1, 2, 3, 4, 5
(FFN_AUTO, FFN_FMA, FFN_TENSOR, FFN_TENSOR_F8, FFN_TENSOR_F4, FFN_TENSOR_FUSED,
 FFN_TENSOR_F8_PAIR) = 0, 1, 2, 3, 4, 5, 6

_c_int, _c_float, _c_size, _vp = ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_void_p

# name -> (restype, argtypes)
SIGNATURES = {
    "moe_status_string": (ctypes.c_char_p, [_c_int]),
    "moe_version": (_c_int, []),
    "moe_route_topk": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "moe_permute": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp]),
    "moe_route_permute": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "mxfp4_moe_ffn_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "mxfp4_moe_ffn": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                               _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "mxfp4_moe_ffn_variant": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                       _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_size,
                                       _c_int, _vp]),
    "mxfp4_moe_ffn_workspace_h": (_vp, [_vp]),
    "mxfp4_moe_ffn_noalloc": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int,
                                       _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_combine": (_c_int, [_vp, _vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "moe_rms_norm": (_c_int, [_vp, _c_int, _c_int, _c_float, _vp, _vp]),
    "block_accept_greedy": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "block_accept_rejection": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                        _vp, _vp, _vp]),
    "block_accept_greedy_bonus": (_c_int, [_vp, _vp, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "block_accept_rejection_bonus": (_c_int, [_vp, _vp, _vp, _vp, _vp, _c_int, _c_int, _c_int,
                                              _vp, _vp, _vp]),
    "mxfp4_quantize": (_c_int, [_vp, ctypes.c_int64, _c_int, _vp, _vp, _vp]),
    "block_kv_append": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp,
                                 _c_float, _vp, _c_int, _c_int, _c_int, _vp, _vp, _c_int, _vp, _vp,
                                 _c_int, _c_int, _vp, _vp]),
    "block_attention_workspace_bytes": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    "block_attention": (_c_int, [_vp, _c_int, _c_int, _c_int, _c_int, _c_int, _vp, _vp, _c_int,
                                 _c_int, _vp, _c_int, _vp, _c_float, _c_int, _vp, _vp, _c_size, _vp]),
    "block_sample": (_c_int, [_vp, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_get_device_status": (_c_int, [_vp, ctypes.POINTER(_c_int)]),
    "moe_clear_device_status": (_c_int, [_vp]),
    "moe_set_wait_limit_ns": (_c_int, [ctypes.c_uint64, _vp]),
}

_LIB = None


class MoeError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({STATUS_NAMES.get(status, '?')})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the CUDA library once; raise if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m mxfp4_moe_block_b200.build`"
                + (" --checks" if LIB_PATH.endswith("_checks.so") else ""))
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(status: int, what: str):
    if status != MOE_OK:
        raise MoeError(status, what)


def _ptr(t: torch.Tensor | None, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def moe_route_topk(logits, k, topk_idx=None, topk_w=None, stream=None):
    T, E = logits.shape
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _check(lib().moe_route_topk(_ptr(logits, torch.float32, "logits"), T, E, k,
                                _ptr(topk_idx, torch.int32), _ptr(topk_w, torch.float32),
                                _stream(stream)), "moe_route_topk")
    return topk_idx, topk_w


def moe_permute(topk_idx, E, expert_offsets=None, sorted_pair=None, pair_row=None, stream=None):
    T, k = topk_idx.shape
    dev = topk_idx.device
    P = T * k
    if expert_offsets is None:
        expert_offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    if sorted_pair is None:
        sorted_pair = torch.empty(P, dtype=torch.int32, device=dev)
    if pair_row is None:
        pair_row = torch.empty(P, dtype=torch.int32, device=dev)
    _check(lib().moe_permute(_ptr(topk_idx, torch.int32, "topk_idx"), T, k, E,
                             _ptr(expert_offsets, torch.int32), _ptr(sorted_pair, torch.int32),
                             _ptr(pair_row, torch.int32), _stream(stream)), "moe_permute")
    return expert_offsets, sorted_pair, pair_row


def moe_route_permute(logits, k, E=None, topk_idx=None, topk_w=None, expert_offsets=None,
                      sorted_pair=None, pair_row=None, stream=None):
    """moe_route_topk + moe_permute in one call (one kernel for T <= 128)."""
    T, E_ = logits.shape
    E = E_ if E is None else E
    dev = logits.device
    P = T * k
    i32 = dict(dtype=torch.int32, device=dev)
    topk_idx = torch.empty((T, k), **i32) if topk_idx is None else topk_idx
    topk_w = torch.empty((T, k), dtype=torch.float32, device=dev) if topk_w is None else topk_w
    expert_offsets = torch.empty(E + 1, **i32) if expert_offsets is None else expert_offsets
    sorted_pair = torch.empty(P, **i32) if sorted_pair is None else sorted_pair
    pair_row = torch.empty(P, **i32) if pair_row is None else pair_row
    _check(lib().moe_route_permute(
        _ptr(logits, torch.float32, "logits"), T, E, k, _ptr(topk_idx, torch.int32),
        _ptr(topk_w, torch.float32), _ptr(expert_offsets, torch.int32),
        _ptr(sorted_pair, torch.int32), _ptr(pair_row, torch.int32), _stream(stream)),
        "moe_route_permute")
    return topk_idx, topk_w, expert_offsets, sorted_pair, pair_row


def mxfp4_moe_ffn_workspace_bytes(T, k, H, I):
    return int(lib().mxfp4_moe_ffn_workspace_bytes(T, k, H, I))


def alloc_workspace(T, k, H, I, device):
    n = mxfp4_moe_ffn_workspace_bytes(T, k, H, I)
    return torch.empty(n, dtype=torch.uint8, device=device)   # torch blocks are 256B-aligned


def mxfp4_moe_ffn(x, k, w13_codes, w13_scales, w2_codes, w2_scales, expert_offsets,
                  sorted_pair, y=None, workspace=None, variant=FFN_AUTO, stream=None):
    """x [T,H] bf16; weights uint8 as in the header; returns (y [T*k,H] f32, workspace)."""
    T, H = x.shape
    E, twoI, _ = w13_codes.shape
    I = twoI // 2
    dev = x.device
    if y is None:
        y = torch.empty((T * k, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(T, k, H, I, dev)
    _check(lib().mxfp4_moe_ffn_variant(
        _ptr(x, torch.bfloat16, "x"), T, H, I, E, k,
        _ptr(w13_codes, torch.uint8, "w13_codes"), _ptr(w13_scales, torch.uint8, "w13_scales"),
        _ptr(w2_codes, torch.uint8, "w2_codes"), _ptr(w2_scales, torch.uint8, "w2_scales"),
        _ptr(expert_offsets, torch.int32), _ptr(sorted_pair, torch.int32),
        _ptr(y, torch.float32, "y"), _ptr(workspace), workspace.numel(), variant,
        _stream(stream)), "mxfp4_moe_ffn")
    return y, workspace


NOALLOC_SCRATCH_BYTES = 8 << 20


def mxfp4_moe_ffn_noalloc(x, k, w13_codes, w13_scales, w2_codes, w2_scales, expert_offsets,
                          sorted_pair, y=None, stream=None):
    """mxfp4_moe_ffn without a caller-supplied workspace: the library uses its
    own fixed device scratch (NOALLOC_SCRATCH_BYTES), so the call allocates
    nothing when ``y`` is given.  For callers that may not allocate device
    memory; calls that overlap on the GPU share that scratch and race."""
    T, H = x.shape
    E, twoI, _ = w13_codes.shape
    I = twoI // 2
    if y is None:
        y = torch.empty((T * k, H), dtype=torch.float32, device=x.device)
    _check(lib().mxfp4_moe_ffn_noalloc(
        _ptr(x, torch.bfloat16, "x"), T, H, I, E, k,
        _ptr(w13_codes, torch.uint8, "w13_codes"), _ptr(w13_scales, torch.uint8, "w13_scales"),
        _ptr(w2_codes, torch.uint8, "w2_codes"), _ptr(w2_scales, torch.uint8, "w2_scales"),
        _ptr(expert_offsets, torch.int32), _ptr(sorted_pair, torch.int32),
        _ptr(y, torch.float32, "y"), _stream(stream)), "mxfp4_moe_ffn_noalloc")
    return y


def workspace_h(workspace, P, I):
    """View of the bf16 SwiGLU outputs h [P, I] kept in the FFN workspace."""
    return workspace[:P * I * 2].view(torch.bfloat16).view(P, I)


def moe_combine(y, pair_row, topk_w, residual=None, out=None, stream=None):
    T, k = topk_w.shape
    H = y.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y.device)
    _check(lib().moe_combine(_ptr(y, torch.float32, "y"), _ptr(pair_row, torch.int32),
                             _ptr(topk_w, torch.float32), T, k, H,
                             _ptr(residual, torch.bfloat16, "residual"),
                             _ptr(out, torch.bfloat16, "out"), _stream(stream)), "moe_combine")
    return out


def moe_rms_norm(x, eps=1e-6, out=None, stream=None):
    T, H = x.shape
    if out is None:
        out = torch.empty_like(x)
    _check(lib().moe_rms_norm(_ptr(x, torch.bfloat16, "x"), T, H, float(eps),
                              _ptr(out, torch.bfloat16, "out"), _stream(stream)), "moe_rms_norm")
    return out


def block_accept_greedy(logits, draft, accept_len=None, next_token=None, stream=None):
    S, K, V = logits.shape
    dev = logits.device
    if accept_len is None:
        accept_len = torch.empty(S, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(S, dtype=torch.int32, device=dev)
    _check(lib().block_accept_greedy(_ptr(logits, torch.float32, "logits"),
                                     _ptr(draft, torch.int32, "draft"), S, K, V,
                                     _ptr(accept_len, torch.int32), _ptr(next_token, torch.int32),
                                     _stream(stream)), "block_accept_greedy")
    return accept_len, next_token


def block_accept_rejection(p, q, draft, u_accept, u_resample, accept_len=None,
                           next_token=None, stream=None):
    S, K, V = p.shape
    dev = p.device
    if accept_len is None:
        accept_len = torch.empty(S, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(S, dtype=torch.int32, device=dev)
    _check(lib().block_accept_rejection(
        _ptr(p, torch.float32, "p"), _ptr(q, torch.float32, "q"), _ptr(draft, torch.int32, "draft"),
        _ptr(u_accept, torch.float32, "u_accept"), _ptr(u_resample, torch.float32, "u_resample"),
        S, K, V, _ptr(accept_len, torch.int32), _ptr(next_token, torch.int32), _stream(stream)),
        "block_accept_rejection")
    return accept_len, next_token


def block_accept_greedy_bonus(logits, draft, accept_len=None, next_token=None, stream=None):
    """logits [S, K+1, V] (row K: the target after the block), draft [S, K]."""
    S, K1, V = logits.shape
    K = K1 - 1
    if tuple(draft.shape) != (S, K):
        raise ValueError("draft must be [S, K] for logits [S, K+1, V]")
    dev = logits.device
    if accept_len is None:
        accept_len = torch.empty(S, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(S, dtype=torch.int32, device=dev)
    _check(lib().block_accept_greedy_bonus(_ptr(logits, torch.float32, "logits"),
                                           _ptr(draft, torch.int32, "draft"), S, K, V,
                                           _ptr(accept_len, torch.int32),
                                           _ptr(next_token, torch.int32), _stream(stream)),
           "block_accept_greedy_bonus")
    return accept_len, next_token


def block_accept_rejection_bonus(p, q, draft, u_accept, u_resample, accept_len=None,
                                 next_token=None, stream=None):
    """p [S, K+1, V] (row K: the target after the block), q [S, K, V]."""
    S, K1, V = p.shape
    K = K1 - 1
    if tuple(q.shape) != (S, K, V) or tuple(draft.shape) != (S, K):
        raise ValueError("q [S, K, V] and draft [S, K] for p [S, K+1, V]")
    dev = p.device
    if accept_len is None:
        accept_len = torch.empty(S, dtype=torch.int32, device=dev)
    if next_token is None:
        next_token = torch.empty(S, dtype=torch.int32, device=dev)
    _check(lib().block_accept_rejection_bonus(
        _ptr(p, torch.float32, "p"), _ptr(q, torch.float32, "q"), _ptr(draft, torch.int32, "draft"),
        _ptr(u_accept, torch.float32, "u_accept"), _ptr(u_resample, torch.float32, "u_resample"),
        S, K, V, _ptr(accept_len, torch.int32), _ptr(next_token, torch.int32), _stream(stream)),
        "block_accept_rejection_bonus")
    return accept_len, next_token


def mxfp4_quantize(w, codes=None, scales=None, stream=None):
    """w [R, K] bf16 -> (codes [R, K/2] uint8, scales [R, K/32] uint8), OCP MXFP4."""
    R, K = w.shape
    dev = w.device
    if codes is None:
        codes = torch.empty((R, K // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((R, K // 32), dtype=torch.uint8, device=dev)
    _check(lib().mxfp4_quantize(_ptr(w, torch.bfloat16, "w"), R, K, _ptr(codes, torch.uint8),
                                _ptr(scales, torch.uint8), _stream(stream)), "mxfp4_quantize")
    return codes, scales


class _On:
    """A context in which the device of `t` and the stream given (that device's
    current one if None) are current, so that outputs and scratch allocated in it
    belong to the stream the kernels run on."""
    __slots__ = ("_ctx",)

    def __init__(self, stream, t):
        if stream is None:
            self._ctx = torch.cuda.device(t.device)
        else:
            if stream.device != t.device:
                raise ValueError(f"stream of {stream.device} for tensors on {t.device}")
            self._ctx = torch.cuda.stream(stream)      # also makes its device current

    def __enter__(self):
        self._ctx.__enter__()

    def __exit__(self, *exc):
        self._ctx.__exit__(*exc)


def _elsewhere(stream, t, name):
    """Whether a call on `t` has to switch device or stream first (see _On)."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return stream is not None or index != torch._C._cuda_getDevice()


_device_of, _is_contiguous, _address = (torch.Tensor.get_device, torch.Tensor.is_contiguous,
                                        torch.Tensor.data_ptr)


def _pointers(kinds, *tensors):
    """Addresses of tensors (or None) of the given (name, dtype) kinds, all on the
    first one's device, and that device's current stream.  (One pass, each check once:
    these calls take a few microseconds on the GPU.)"""
    index = _device_of(tensors[0])
    out = []
    for t, (name, dtype) in zip(tensors, kinds):
        if t is None:
            out.append(None)
        elif t.dtype is dtype and _device_of(t) == index and _is_contiguous(t):
            out.append(_address(t))
        else:
            _ptr(t, dtype, name)
            raise ValueError("tensors on different devices: " + ", ".join(
                f"{n} {x.device}" for x, (n, _) in zip(tensors, kinds) if x is not None))
    out.append(torch._C._cuda_getCurrentRawStream(index))
    return out


_APPEND = (("qkv", torch.bfloat16), ("kv_len", torch.int32), ("block_table", torch.int32),
           ("k_cache", torch.bfloat16), ("v_cache", torch.bfloat16), ("cos_sin", torch.float32),
           ("q_weight", torch.bfloat16), ("k_weight", torch.bfloat16), ("q_out", torch.bfloat16))
_ATTENTION = (("q", torch.bfloat16), ("k_cache", torch.bfloat16), ("v_cache", torch.bfloat16),
              ("block_table", torch.int32), ("kv_len", torch.int32), ("out", torch.bfloat16),
              ("workspace", torch.uint8))
_SAMPLE = (("logits", torch.float32), ("temperature", torch.float32), ("top_k", torch.int32),
           ("top_p", torch.float32), ("min_p", torch.float32), ("u", torch.float32),
           ("token", torch.int32), ("probs", torch.float32))


def _shape(t, shape, name):
    if t is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _cache_shapes(k_cache, v_cache, kv_len, block_table, S, D):
    if k_cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_cache must be [pages, Hkv, page_size, D], block_table [S, max_pages]")
    pages, Hkv, page_size, Dk = k_cache.shape
    _shape(v_cache, (pages, Hkv, page_size, Dk), "v_cache")
    _shape(kv_len, (S,), "kv_len")
    rows, max_pages = block_table.shape
    if rows != S:
        raise ValueError(f"block_table must have {S} rows, got {rows}")
    if Dk != D:
        raise ValueError(f"k_cache must have heads of {D}, got {Dk}")
    return pages, Hkv, page_size, max_pages


def block_kv_append(qkv, kv_len, block_table, k_cache, v_cache, cos_sin=None, q_weight=None,
                    k_weight=None, norm=True, eps=1e-6, interleaved=False, q_out=None, stream=None):
    """Head norms of q and k, rotation, append of k and v to the paged cache.

    qkv [S, N, Hq + 2*Hkv, D] bf16; kv_len [S] int32 with the N new tokens counted;
    block_table [S, max_pages] int32; caches [pages, Hkv, page_size, D] bf16, updated in
    place; cos_sin [max_pos, rot] float or None (no rotation).  Returns q [S, N, Hq, D];
    rows of slots not in use are zero where the call allocates q, else left as they were."""
    if _elsewhere(stream, qkv, "qkv"):
        with _On(stream, qkv):
            return block_kv_append(qkv, kv_len, block_table, k_cache, v_cache, cos_sin, q_weight,
                                   k_weight, norm, eps, interleaved, q_out)
    S, N, heads, D = qkv.shape
    pages, Hkv, page_size, max_pages = _cache_shapes(k_cache, v_cache, kv_len, block_table, S, D)
    Hq = heads - 2 * Hkv
    if q_out is None and Hq > 0:
        q_out = torch.zeros((S, N, Hq, D), dtype=torch.bfloat16, device=qkv.device)
    _shape(q_out, (S, N, Hq, D), "q_out")
    _shape(q_weight, (D,), "q_weight")
    _shape(k_weight, (D,), "k_weight")
    max_pos, rot = cos_sin.shape if cos_sin is not None else (0, 0)
    p_qkv, p_len, p_table, p_k, p_v, p_cs, p_qw, p_kw, p_q, st = _pointers(
        _APPEND, qkv, kv_len, block_table, k_cache, v_cache, cos_sin, q_weight, k_weight, q_out)
    _check(lib().block_kv_append(p_qkv, S, N, Hq, Hkv, D, int(norm), p_qw, p_kw, float(eps), p_cs, max_pos,
                                 rot, int(interleaved), p_len, p_table, max_pages, p_k, p_v, pages,
                                 page_size, p_q, st), "block_kv_append")
    return q_out


@functools.lru_cache(maxsize=64)
def block_attention_workspace_bytes(S, N, Hq, Hkv, D):
    return int(lib().block_attention_workspace_bytes(S, N, Hq, Hkv, D))


def alloc_attention_workspace(S, N, Hq, Hkv, D, device):
    return torch.empty(max(block_attention_workspace_bytes(S, N, Hq, Hkv, D), 1),
                       dtype=torch.uint8, device=device)


def block_attention(q, k_cache, v_cache, block_table, kv_len, scale=None, window=0, out=None,
                    workspace=None, stream=None):
    """Attention of N tokens per sequence over the paged cache; q [S, N, Hq, D] bf16.

    scale defaults to D ** -0.5; window 0 sees the whole cache.  Returns out [S, N, Hq, D]."""
    if _elsewhere(stream, q, "q"):
        with _On(stream, q):
            return block_attention(q, k_cache, v_cache, block_table, kv_len, scale, window, out,
                                   workspace)
    S, N, Hq, D = q.shape
    pages, Hkv, page_size, max_pages = _cache_shapes(k_cache, v_cache, kv_len, block_table, S, D)
    if out is None:
        out = torch.empty_like(q)
    _shape(out, (S, N, Hq, D), "out")
    if workspace is None:
        workspace = alloc_attention_workspace(S, N, Hq, Hkv, D, q.device)
    p_q, p_k, p_v, p_table, p_len, p_out, p_ws, st = _pointers(
        _ATTENTION, q, k_cache, v_cache, block_table, kv_len, out, workspace)
    _check(lib().block_attention(
        p_q, S, N, Hq, Hkv, D, p_k, p_v, pages, page_size, p_table, max_pages, p_len,
        D ** -0.5 if scale is None else float(scale), int(window), p_out, p_ws, workspace.numel(), st),
        "block_attention")
    return out


def block_sample(logits, u=None, temperature=None, top_k=None, top_p=None, min_p=None,
                 with_probs=False, token=None, probs=None, stream=None):
    """logits [S, K, V] -> (token [S, K] int32 or None, probs [S, K, V] float or None).

    Tokens are drawn where u [S, K] is given; probabilities are written where
    with_probs is set or probs given.  The filters are [S] tensors or None (off)."""
    if _elsewhere(stream, logits, "logits"):
        with _On(stream, logits):
            return block_sample(logits, u, temperature, top_k, top_p, min_p, with_probs, token, probs)
    S, K, V = logits.shape
    _shape(u, (S, K), "u")
    _shape(temperature, (S,), "temperature")
    _shape(top_k, (S,), "top_k")
    _shape(top_p, (S,), "top_p")
    _shape(min_p, (S,), "min_p")
    if token is not None:
        _shape(token, (S, K), "token")
    elif u is not None:
        token = torch.empty_like(u, dtype=torch.int32)
    if probs is not None:
        _shape(probs, (S, K, V), "probs")
    elif with_probs:
        probs = torch.empty_like(logits)
    p_logits, p_t, p_k, p_p, p_m, p_u, p_token, p_probs, st = _pointers(
        _SAMPLE, logits, temperature, top_k, top_p, min_p, u, token, probs)
    _check(lib().block_sample(p_logits, S, K, V, p_t, p_k, p_p, p_m, p_u, p_token, p_probs, st),
           "block_sample")
    return token, probs


def moe_get_device_status(stream=None):
    """(status, detail): synchronises the stream and reads the status word."""
    d = ctypes.c_int(0)
    st = lib().moe_get_device_status(_stream(stream), ctypes.byref(d))
    return st, d.value


def moe_clear_device_status(stream=None):
    _check(lib().moe_clear_device_status(_stream(stream)), "moe_clear_device_status")


def moe_set_wait_limit_ns(ns=0, stream=None):
    """Limit of the FFN and attention kernels' bounded waits (0 = the 2 s default)."""
    _check(lib().moe_set_wait_limit_ns(int(ns), _stream(stream)), "moe_set_wait_limit_ns")
