"""Python binding of the gfx950 NVFP4 W4A4 linear-layer library.

Thin ctypes wrappers over the C ABI declared in include/nvfp4.h: the functions
named ``nvfp4_*`` take torch tensors, check nothing the library does not check
itself, pass ``data_ptr()`` values and torch's current HIP stream, and raise
``NVFP4Error`` on a non-OK status.  Every step of the computation runs in the
library's HIP kernels; torch only supplies device memory and the stream.
There is no fallback: if the library is not built, the first call into it
raises ImportError.

Convenience layer (allocation only): ``quantize_act``, ``pack_weight``,
``gemm`` and ``PackedWeight`` allocate outputs with torch and call the C ABI.
Their ``stream`` is a keyword-only ``torch.cuda.Stream`` (default: torch's
current stream); the ``nvfp4_*`` wrappers take a raw hipStream_t handle.
"""
import ctypes
import functools
import inspect
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4_w4a4.so")

NVFP4_MAX_SEGMENTS = 16
STATUS = {0: "NVFP4_OK", 1: "NVFP4_EINVAL", 2: "NVFP4_ESHAPE", 3: "NVFP4_EALIGN",
          4: "NVFP4_ESEGMENTS", 5: "NVFP4_EWORKSPACE", 6: "NVFP4_EHIP"}


class NVFP4Error(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        msg = _lib().nvfp4_status_str(status).decode()
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg})")


class Segment(ctypes.Structure):
    _fields_ = [("n_begin", ctypes.c_int32), ("n_end", ctypes.c_int32)]


DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.uint8: 2}     # nvfp4_dtype (uint8: E4M3 codes)


class KVCacheDesc(ctypes.Structure):
    """nvfp4_kv_cache: the host struct that describes a paged key-value cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_amax", ctypes.c_void_p),
                ("v_amax", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_LIB = None
_i64, _vp, _sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_i32, _f32 = ctypes.c_int32, ctypes.c_float


def _declare(lib):
    """Result and argument types of every function of the C ABI."""
    lib.nvfp4_abi_version.restype = ctypes.c_int
    lib.nvfp4_status_str.restype = ctypes.c_char_p
    lib.nvfp4_status_str.argtypes = [ctypes.c_int]
    lib.nvfp4_quantize_act_workspace_bytes.restype = _sz
    lib.nvfp4_quantize_act_workspace_bytes.argtypes = [_i64, _i64]
    lib.nvfp4_quantize_act.restype = ctypes.c_int
    lib.nvfp4_quantize_act.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.nvfp4_packed_weight_bytes.restype = ctypes.c_int
    lib.nvfp4_packed_weight_bytes.argtypes = [_i64, _i64, ctypes.POINTER(_sz), ctypes.POINTER(_sz)]
    lib.nvfp4_pack_weight_workspace_bytes.restype = _sz
    lib.nvfp4_pack_weight_workspace_bytes.argtypes = [_i64, _i64, ctypes.c_int32]
    lib.nvfp4_pack_weight.restype = ctypes.c_int
    lib.nvfp4_pack_weight.argtypes = [_vp, _i64, _i64, _i64, ctypes.POINTER(Segment), ctypes.c_int32,
                                      _vp, _vp, _vp, _vp, _sz, _vp]
    lib.nvfp4_weight_to_canonical.restype = ctypes.c_int
    lib.nvfp4_weight_to_canonical.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _vp]
    lib.nvfp4_gemm.restype = ctypes.c_int
    lib.nvfp4_gemm.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, ctypes.POINTER(Segment), _vp,
                               ctypes.c_int32, _vp, _i64, _vp]
    lib.nvfp4_gemm_form.restype = ctypes.c_int
    lib.nvfp4_gemm_form.argtypes = [_i64, _i64, _i64]
    lib.nvfp4_linear_workspace_bytes.restype = _sz
    lib.nvfp4_linear_workspace_bytes.argtypes = [_i64, _i64]
    lib.nvfp4_linear.restype = ctypes.c_int
    lib.nvfp4_linear.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                 ctypes.POINTER(Segment), _vp, ctypes.c_int32, _vp, _i64, _vp, _sz, _vp]
    lib.nvfp4_linear_noalloc.restype = ctypes.c_int
    lib.nvfp4_linear_noalloc.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                         ctypes.POINTER(Segment), _vp, ctypes.c_int32, _vp, _i64, _vp]
    lib.nvfp4_pack_weight_gate_up.restype = ctypes.c_int
    lib.nvfp4_pack_weight_gate_up.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.nvfp4_gemm_swiglu_quantize.restype = ctypes.c_int
    lib.nvfp4_gemm_swiglu_quantize.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                               _vp, _vp]
    lib.nvfp4_amax_observe_workspace_bytes.restype = _sz
    lib.nvfp4_amax_observe_workspace_bytes.argtypes = [_i64, _i64]
    lib.nvfp4_amax_observe.restype = ctypes.c_int
    lib.nvfp4_amax_observe.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _sz, _vp]
    lib.nvfp4_quantize_stats.restype = ctypes.c_int
    lib.nvfp4_quantize_stats.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
    lib.nvfp4_kv_fp8_encode.restype = ctypes.c_int
    lib.nvfp4_kv_fp8_encode.argtypes = [_vp, _i64, _vp, _vp, _vp]
    lib.nvfp4_kv_fp8_decode.restype = ctypes.c_int
    lib.nvfp4_kv_fp8_decode.argtypes = [_vp, _i64, _vp, _vp, _vp]
    lib.nvfp4_swiglu.restype = ctypes.c_int
    lib.nvfp4_swiglu.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _vp]
    lib.nvfp4_convert_sweep.restype = ctypes.c_int
    lib.nvfp4_convert_sweep.argtypes = [ctypes.c_int32, ctypes.c_uint32, _i64, _vp, _vp]
    lib.nvfp4_read_probe.restype = ctypes.c_int
    lib.nvfp4_read_probe.argtypes = [_vp, _i64, ctypes.c_int32, _vp, _vp]
    cache_p = ctypes.POINTER(KVCacheDesc)
    lib.nvfp4_kv_append.restype = ctypes.c_int
    lib.nvfp4_kv_append.argtypes = [_vp, _vp, _vp, _i32, _i64, _i32, _i64, _i64, _i64, _vp, _i32, _i64, _i32, _vp,
                                    _vp, cache_p, _vp, _i64, _vp]
    lib.nvfp4_kv_append_norm.restype = ctypes.c_int
    lib.nvfp4_kv_append_norm.argtypes = [_vp, _vp, _vp, _i32, _i64, _i32, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _i32,
                                         _i64, _i32, _vp, _vp, cache_p, _vp, _i64, _vp]
    lib.nvfp4_attn_decode_workspace_bytes.restype = _sz
    lib.nvfp4_attn_decode_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i64, _i64]
    lib.nvfp4_attn_decode.restype = ctypes.c_int
    lib.nvfp4_attn_decode.argtypes = [_vp, _i64, _i32, _i64, cache_p, _vp, _i64, _vp, _i64, _f32, _i64, _vp, _i64,
                                      _vp, _vp, _sz, _vp]
    lib.nvfp4_attn_tree_workspace_bytes.restype = _sz
    lib.nvfp4_attn_tree_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32, _i64, _i64]
    lib.nvfp4_attn_tree.restype = ctypes.c_int
    lib.nvfp4_attn_tree.argtypes = [_vp, _i64, _i32, _i32, _i64, cache_p, _vp, _i64, _vp, _vp, _i64, _f32, _i64, _vp, _i64,
                                    _vp, _vp, _sz, _vp]
    lib.nvfp4_verify_drafts_workspace_bytes.restype = _sz
    lib.nvfp4_verify_drafts_workspace_bytes.argtypes = [_i64, _i32, _i64, _i32]
    lib.nvfp4_verify_drafts.restype = ctypes.c_int
    lib.nvfp4_verify_drafts.argtypes = [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                        _vp]
    lib.nvfp4_kv_compact.restype = ctypes.c_int
    lib.nvfp4_kv_compact.argtypes = [cache_p, _i32, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp]
    lib.nvfp4_kv_copy_pages.restype = ctypes.c_int
    lib.nvfp4_kv_copy_pages.argtypes = [cache_p, _i32, _vp, _vp, _i64, _vp]
    gdn = [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64]
    lib.nvfp4_gdn_step.restype = ctypes.c_int
    lib.nvfp4_gdn_step.argtypes = gdn + [_i64, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _f32, _vp, _i64, _vp]
    lib.nvfp4_gdn_prefill_workspace_bytes.restype = _sz
    lib.nvfp4_gdn_prefill_workspace_bytes.argtypes = [_i64, _i64, _i32, _i32, _i32, _i32]
    lib.nvfp4_gdn_prefill.restype = ctypes.c_int
    lib.nvfp4_gdn_prefill.argtypes = gdn + [_i64, _i64, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _f32,
                                            _vp, _i64, _vp, _sz, _vp]


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run python -m nvfp4_w4a4_block_act_amd.build")
        lib = ctypes.CDLL(LIB_PATH)
        try:
            _declare(lib)
        except AttributeError as e:      # functions were added without a new NVFP4_ABI_VERSION
            raise ImportError(f"{LIB_PATH} is of an earlier build ({e}); run python -m "
                              "nvfp4_w4a4_block_act_amd.build") from None
        _LIB = lib
    return _LIB


def lib():
    """The loaded ctypes library (loads it on first use)."""
    return _lib()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is not None:
        return stream
    return torch.cuda.current_stream().cuda_stream


def _check(status, where):
    if status != 0:
        raise NVFP4Error(status, where)


def _segs(segments):
    arr = (Segment * max(1, len(segments)))()
    for i, (b, e) in enumerate(segments):
        arr[i].n_begin, arr[i].n_end = int(b), int(e)
    return arr, len(segments)


# ---- the C ABI, one wrapper per entry point ---------------------------------------
def nvfp4_abi_version():
    return _lib().nvfp4_abi_version()


def nvfp4_status_str(status):
    return _lib().nvfp4_status_str(int(status)).decode()


def nvfp4_quantize_act_workspace_bytes(M, K):
    return _lib().nvfp4_quantize_act_workspace_bytes(int(M), int(K))


def nvfp4_quantize_act(x, M, K, ldx, amax_in, codes, scales, g_dec_out, workspace, workspace_bytes, stream=None):
    _check(_lib().nvfp4_quantize_act(_ptr(x), M, K, ldx, _ptr(amax_in), _ptr(codes), _ptr(scales),
                                     _ptr(g_dec_out), _ptr(workspace), workspace_bytes, _stream(stream)),
           "nvfp4_quantize_act")


def nvfp4_packed_weight_bytes(N, K):
    cb, sb = _sz(0), _sz(0)
    _check(_lib().nvfp4_packed_weight_bytes(int(N), int(K), ctypes.byref(cb), ctypes.byref(sb)),
           "nvfp4_packed_weight_bytes")
    return cb.value, sb.value


def nvfp4_pack_weight_workspace_bytes(N, K, nseg):
    return _lib().nvfp4_pack_weight_workspace_bytes(int(N), int(K), int(nseg))


def nvfp4_pack_weight(w, N, K, ldw, segments, w_codes, w_scales, w_g_dec, workspace, workspace_bytes,
                      stream=None):
    arr, n = _segs(segments)
    _check(_lib().nvfp4_pack_weight(_ptr(w), N, K, ldw, arr, n, _ptr(w_codes), _ptr(w_scales), _ptr(w_g_dec),
                                    _ptr(workspace), workspace_bytes, _stream(stream)), "nvfp4_pack_weight")


def nvfp4_weight_to_canonical(w_codes, w_scales, N, K, codes, scales, stream=None):
    _check(_lib().nvfp4_weight_to_canonical(_ptr(w_codes), _ptr(w_scales), N, K, _ptr(codes), _ptr(scales),
                                            _stream(stream)), "nvfp4_weight_to_canonical")


def nvfp4_gemm(a_codes, a_scales, a_g_dec, M, K, w_codes, w_scales, N, segments, w_g_dec, out, ldo,
               stream=None):
    arr, n = _segs(segments)
    _check(_lib().nvfp4_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(a_g_dec), M, K, _ptr(w_codes), _ptr(w_scales),
                             N, arr, _ptr(w_g_dec), n, _ptr(out), ldo, _stream(stream)), "nvfp4_gemm")


def nvfp4_gemm_form(M, K, N):
    return _lib().nvfp4_gemm_form(int(M), int(K), int(N))


def nvfp4_linear_workspace_bytes(M, K):
    return _lib().nvfp4_linear_workspace_bytes(int(M), int(K))


def nvfp4_linear(x, M, K, ldx, amax_in, a_codes, a_scales, a_g_dec, w_codes, w_scales, N, segments, w_g_dec,
                 out, ldo, workspace, workspace_bytes, stream=None):
    arr, n = _segs(segments)
    _check(_lib().nvfp4_linear(_ptr(x), M, K, ldx, _ptr(amax_in), _ptr(a_codes), _ptr(a_scales), _ptr(a_g_dec),
                               _ptr(w_codes), _ptr(w_scales), N, arr, _ptr(w_g_dec), n, _ptr(out), ldo,
                               _ptr(workspace), workspace_bytes, _stream(stream)), "nvfp4_linear")


def nvfp4_linear_noalloc(x, M, K, ldx, amax_in, a_codes, a_scales, a_g_dec, w_codes, w_scales, N, segments,
                         w_g_dec, out, ldo, stream=None):
    arr, n = _segs(segments)
    _check(_lib().nvfp4_linear_noalloc(_ptr(x), M, K, ldx, _ptr(amax_in), _ptr(a_codes), _ptr(a_scales),
                                       _ptr(a_g_dec), _ptr(w_codes), _ptr(w_scales), N, arr, _ptr(w_g_dec), n,
                                       _ptr(out), ldo, _stream(stream)), "nvfp4_linear_noalloc")


def nvfp4_pack_weight_gate_up(w, I, K, ldw, w_codes, w_scales, w_g_dec, workspace, workspace_bytes, stream=None):
    _check(_lib().nvfp4_pack_weight_gate_up(_ptr(w), I, K, ldw, _ptr(w_codes), _ptr(w_scales), _ptr(w_g_dec),
                                            _ptr(workspace), workspace_bytes, _stream(stream)),
           "nvfp4_pack_weight_gate_up")


def nvfp4_gemm_swiglu_quantize(a_codes, a_scales, a_g_dec, M, K, w_codes, w_scales, I, w_g_dec, amax_h,
                               h_codes, h_scales, h_g_dec, stream=None):
    _check(_lib().nvfp4_gemm_swiglu_quantize(_ptr(a_codes), _ptr(a_scales), _ptr(a_g_dec), M, K, _ptr(w_codes),
                                             _ptr(w_scales), I, _ptr(w_g_dec), _ptr(amax_h), _ptr(h_codes),
                                             _ptr(h_scales), _ptr(h_g_dec), _stream(stream)),
           "nvfp4_gemm_swiglu_quantize")


def nvfp4_amax_observe_workspace_bytes(M, K):
    return _lib().nvfp4_amax_observe_workspace_bytes(int(M), int(K))


def nvfp4_amax_observe(x, M, K, ldx, running_amax, workspace, workspace_bytes, stream=None):
    _check(_lib().nvfp4_amax_observe(_ptr(x), M, K, ldx, _ptr(running_amax), _ptr(workspace), workspace_bytes,
                                     _stream(stream)), "nvfp4_amax_observe")


def nvfp4_quantize_stats(x, M, K, ldx, amax_in, counts, stream=None):
    _check(_lib().nvfp4_quantize_stats(_ptr(x), M, K, ldx, _ptr(amax_in), _ptr(counts), _stream(stream)),
           "nvfp4_quantize_stats")


def nvfp4_kv_fp8_encode(x, n, amax, codes, stream=None):
    _check(_lib().nvfp4_kv_fp8_encode(_ptr(x), n, _ptr(amax), _ptr(codes), _stream(stream)), "nvfp4_kv_fp8_encode")


def nvfp4_kv_fp8_decode(codes, n, amax, out, stream=None):
    _check(_lib().nvfp4_kv_fp8_decode(_ptr(codes), n, _ptr(amax), _ptr(out), _stream(stream)), "nvfp4_kv_fp8_decode")


def nvfp4_swiglu(gu, M, I, ldgu, h, ldh, stream=None):
    _check(_lib().nvfp4_swiglu(_ptr(gu), M, I, ldgu, _ptr(h), ldh, _stream(stream)), "nvfp4_swiglu")


def nvfp4_convert_sweep(op, first_bits, n, out, stream=None):
    _check(_lib().nvfp4_convert_sweep(int(op), int(first_bits), int(n), _ptr(out), _stream(stream)),
           "nvfp4_convert_sweep")


def nvfp4_read_probe(buf, nbytes, workgroups, sink, stream=None):
    _check(_lib().nvfp4_read_probe(_ptr(buf), int(nbytes), int(workgroups), _ptr(sink), _stream(stream)),
           "nvfp4_read_probe")


def nvfp4_kv_append(q, k, v, src_dtype, T, q_heads, ldq, ldk, ldv, rope, rot_dim, max_pos, interleaved, positions, slots,
                    cache, q_out, ldqo, stream=None):
    """``cache`` is a KVCacheDesc."""
    _check(_lib().nvfp4_kv_append(_ptr(q), k.data_ptr(), v.data_ptr(), src_dtype, T, q_heads, ldq, ldk, ldv, _ptr(rope), rot_dim,
                                  max_pos, interleaved, _ptr(positions), slots.data_ptr(), ctypes.byref(cache), _ptr(q_out),
                                  ldqo, _stream(stream)), "nvfp4_kv_append")


def nvfp4_kv_append_norm(q, k, v, src_dtype, T, q_heads, ldq, ldk, ldv, q_norm, k_norm, eps, rope, rot_dim, max_pos, interleaved,
                         positions, slots, cache, q_out, ldqo, stream=None):
    """``cache`` is a KVCacheDesc."""
    _check(_lib().nvfp4_kv_append_norm(_ptr(q), k.data_ptr(), v.data_ptr(), src_dtype, T, q_heads, ldq, ldk, ldv, _ptr(q_norm),
                                       _ptr(k_norm), eps, _ptr(rope), rot_dim, max_pos, interleaved, _ptr(positions),
                                       slots.data_ptr(), ctypes.byref(cache), _ptr(q_out), ldqo, _stream(stream)),
           "nvfp4_kv_append_norm")


def nvfp4_attn_decode_workspace_bytes(B, q_heads, kv_heads, head_dim, max_len, window):
    return _lib().nvfp4_attn_decode_workspace_bytes(B, q_heads, kv_heads, head_dim, max_len, window)


def nvfp4_attn_decode(q, B, q_heads, ldq, cache, block_table, ldt, seq_lens, max_len, scale, window, out, ldo, lse,
                      workspace, workspace_bytes, stream=None):
    """``cache`` is a KVCacheDesc."""
    _check(_lib().nvfp4_attn_decode(q.data_ptr(), B, q_heads, ldq, ctypes.byref(cache), block_table.data_ptr(), ldt,
                                    seq_lens.data_ptr(), max_len, scale, window, out.data_ptr(), ldo, _ptr(lse), _ptr(workspace),
                                    workspace_bytes, _stream(stream)), "nvfp4_attn_decode")


def nvfp4_gdn_step(q, ldq, k, ldk, v, ldv, g, ldg, beta, ldb, B, k_heads, v_heads, k_dim, v_dim, state, num_states,
                   state_index, scale, out, ldo, stream=None):
    _check(_lib().nvfp4_gdn_step(q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, g.data_ptr(), ldg, _ptr(beta), ldb, B, k_heads,
                                 v_heads, k_dim, v_dim, state.data_ptr(), num_states, _ptr(state_index), scale, out.data_ptr(),
                                 ldo, _stream(stream)), "nvfp4_gdn_step")


def nvfp4_gdn_prefill_workspace_bytes(T, B, k_heads, v_heads, k_dim, v_dim):
    return _lib().nvfp4_gdn_prefill_workspace_bytes(T, B, k_heads, v_heads, k_dim, v_dim)


def nvfp4_gdn_prefill(q, ldq, k, ldk, v, ldv, g, ldg, beta, ldb, T, B, cu_seqlens, k_heads, v_heads, k_dim, v_dim,
                      state, num_states, state_index, has_state, scale, out, ldo, workspace, workspace_bytes,
                      stream=None):
    _check(_lib().nvfp4_gdn_prefill(q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, g.data_ptr(), ldg, _ptr(beta), ldb, T, B,
                                    cu_seqlens.data_ptr(), k_heads, v_heads, k_dim, v_dim, state.data_ptr(), num_states,
                                    _ptr(state_index), _ptr(has_state), scale, out.data_ptr(), ldo, _ptr(workspace),
                                    workspace_bytes, _stream(stream)), "nvfp4_gdn_prefill")


def nvfp4_attn_tree_workspace_bytes(B, nodes, q_heads, kv_heads, head_dim, max_len, window):
    return _lib().nvfp4_attn_tree_workspace_bytes(B, nodes, q_heads, kv_heads, head_dim, max_len, window)


def nvfp4_attn_tree(q, B, nodes, q_heads, ldq, cache, block_table, ldt, ctx_lens, parents, max_len, scale, window, out, ldo, lse,
                    workspace, workspace_bytes, stream=None):
    """``cache`` is a KVCacheDesc."""
    _check(_lib().nvfp4_attn_tree(q.data_ptr(), B, nodes, q_heads, ldq, ctypes.byref(cache), block_table.data_ptr(), ldt,
                                  ctx_lens.data_ptr(), _ptr(parents), max_len, scale, window, out.data_ptr(), ldo, _ptr(lse),
                                  _ptr(workspace), workspace_bytes, _stream(stream)), "nvfp4_attn_tree")


def nvfp4_verify_drafts_workspace_bytes(B, nodes, vocab, with_draft_logits):
    return _lib().nvfp4_verify_drafts_workspace_bytes(B, nodes, vocab, with_draft_logits)


def nvfp4_verify_drafts(logits, B, nodes, vocab, ld, draft_logits, ldd, drafts, parents, temperature, uniforms, tokens, path,
                        counts, workspace, workspace_bytes, stream=None):
    _check(_lib().nvfp4_verify_drafts(logits.data_ptr(), B, nodes, vocab, ld, _ptr(draft_logits), ldd, drafts.data_ptr(),
                                      _ptr(parents), _ptr(temperature), _ptr(uniforms), tokens.data_ptr(), path.data_ptr(),
                                      counts.data_ptr(), _ptr(workspace), workspace_bytes, _stream(stream)),
           "nvfp4_verify_drafts")


def nvfp4_kv_compact(caches, layers, block_table, ldt, B, nodes, ctx_lens, path, counts, stream=None):
    """``caches`` is a ctypes array of KVCacheDesc."""
    _check(_lib().nvfp4_kv_compact(caches, layers, block_table.data_ptr(), ldt, B, nodes, ctx_lens.data_ptr(), path.data_ptr(),
                                   counts.data_ptr(), _stream(stream)), "nvfp4_kv_compact")


def nvfp4_kv_copy_pages(caches, layers, src, dst, n, stream=None):
    """``caches`` is a ctypes array of KVCacheDesc."""
    _check(_lib().nvfp4_kv_copy_pages(caches, layers, src.data_ptr(), dst.data_ptr(), n, _stream(stream)),
           "nvfp4_kv_copy_pages")


# ---- convenience layer: allocate with torch, call the C ABI --------------------------
def _on_stream(fn):
    """Runs a convenience function on ``stream`` (a torch.cuda.Stream, keyword-only):
    its tensors -- outputs and temporary scratch -- are allocated while that stream
    is current, so torch's caching allocator hands their memory to no other stream
    while the enqueued kernels may still use it; the C ABI gets the raw handle."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, stream=None, **kw)
        if not isinstance(stream, torch.cuda.Stream):
            raise TypeError(f"{fn.__name__}: stream must be a torch.cuda.Stream "
                            "(the nvfp4_* wrappers take raw handles)")
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream.cuda_stream, **kw)
    return wrapper


def _empty(n, dtype, device):
    return torch.empty(max(int(n), 1), dtype=dtype, device=device)


class Workspace:
    """A growable device scratch buffer owned by the caller.

    The kernels write into it, so calls that share one Workspace must be ordered
    (issued on one stream, or synchronized between streams).  Growing it frees the
    old buffer through torch's stream-ordered allocator, unless a captured call has it:
    a graph may be replayed at any time, so its buffer lives as long as the Workspace."""

    def __init__(self, device):
        self.device = device
        self.buf = None
        self._captured = False       # whether a captured call has the buffer
        self._kept = []              # earlier buffers that one has

    def get(self, nbytes):
        if nbytes == 0:
            return None, 0
        if self.buf is None or self.buf.numel() < nbytes:
            if self._captured:
                self._kept.append(self.buf)
                self._captured = False
            elif self.buf is not None and self.buf.is_cuda:
                # earlier calls may have used it on other streams than the one it was allocated on;
                # they are all ordered before this call, so this call's stream is the one to wait for
                self.buf.record_stream(torch.cuda.current_stream(self.buf.device))
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        if not self._captured and torch.cuda.is_current_stream_capturing():
            self._captured = True
        return self.buf, self.buf.numel()


@_on_stream
def quantize_act(x, amax=None, workspace=None, out=None, *, stream=None):
    """bf16 [M, K] cuda tensor -> (codes uint8 [M, K/2], scales uint8 [M, K/16], g_dec float32 [1])."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] <= 1)
    M, K = x.shape
    dev = x.device
    if out is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
        g = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        codes, scales, g = out
    need = nvfp4_quantize_act_workspace_bytes(M, K)
    ws = workspace if workspace is not None else Workspace(dev)
    buf, nbytes = ws.get(need)
    nvfp4_quantize_act(x, M, K, max(x.stride(0), K), amax, codes, scales, g, buf, nbytes, stream)
    return codes, scales, g


@dataclass
class PackedWeight:
    codes: torch.Tensor      # uint8, tiled layout
    scales: torch.Tensor     # uint8, tiled layout
    g_dec: torch.Tensor      # float32 [nseg]
    N: int
    K: int
    segments: list

    def nbytes(self):
        return self.codes.numel() + self.scales.numel()


@_on_stream
def pack_weight(w, segments=None, *, stream=None):
    """fp32 [N, K] cuda tensor + [(n_begin, n_end), ...] -> PackedWeight."""
    assert w.dtype == torch.float32 and w.dim() == 2 and (w.stride(1) == 1 or w.shape[1] <= 1)
    N, K = w.shape
    segments = [(0, N)] if segments is None else [tuple(s) for s in segments]
    cb, sb = nvfp4_packed_weight_bytes(N, K)
    codes = _empty(cb, torch.uint8, w.device)
    scales = _empty(sb, torch.uint8, w.device)
    g = torch.empty(len(segments), dtype=torch.float32, device=w.device)
    need = nvfp4_pack_weight_workspace_bytes(N, K, len(segments))
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=w.device)
    nvfp4_pack_weight(w, N, K, max(w.stride(0), K), segments, codes, scales, g, ws, need, stream)
    return PackedWeight(codes, scales, g, N, K, segments)


@_on_stream
def weight_to_canonical(pw, *, stream=None):
    codes = torch.empty((pw.N, pw.K // 2), dtype=torch.uint8, device=pw.codes.device)
    scales = torch.empty((pw.N, pw.K // 16), dtype=torch.uint8, device=pw.codes.device)
    nvfp4_weight_to_canonical(pw.codes, pw.scales, pw.N, pw.K, codes, scales, stream)
    return codes, scales


@_on_stream
def gemm(a_codes, a_scales, a_g_dec, pw, out=None, g_dec=None, *, stream=None):
    """NVFP4 activations x packed weight -> fp32 [M, N] (per-segment epilogue).

    ``g_dec`` overrides the weight's per-segment scales (same length)."""
    M = a_codes.shape[0]
    K = pw.K
    assert a_codes.shape[1] * 2 == K
    if out is None:
        out = torch.empty((M, pw.N), dtype=torch.float32, device=a_codes.device)
    wg = pw.g_dec if g_dec is None else g_dec
    nvfp4_gemm(a_codes, a_scales, a_g_dec, M, K, pw.codes, pw.scales, pw.N, pw.segments, wg, out,
               out.stride(0), stream)
    return out


@_on_stream
def linear(x, pw, amax=None, workspace=None, out=None, act_out=None, *, stream=None):
    """The whole W4A4 linear layer via nvfp4_linear: bf16 x [M, K] -> fp32 [M, N].

    Also returns the activation codes, scales and g_dec it produced."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] <= 1)
    M, K = x.shape
    assert K == pw.K
    dev = x.device
    if act_out is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=dev)
        g = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        codes, scales, g = act_out
    if out is None:
        out = torch.empty((M, pw.N), dtype=torch.float32, device=dev)
    ws = workspace if workspace is not None else Workspace(dev)
    buf, nbytes = ws.get(nvfp4_linear_workspace_bytes(M, K))
    nvfp4_linear(x, M, K, max(x.stride(0), K), amax, codes, scales, g, pw.codes, pw.scales, pw.N, pw.segments,
                 pw.g_dec, out, out.stride(0), buf, nbytes, stream)
    return out, (codes, scales, g)


@_on_stream
def pack_weight_gate_up(w, *, stream=None):
    """fp32 [2I, K] (gate rows, then up rows) -> PackedWeight in the interleaved
    gate/up layout, with the two modules' own scales (segments (0, I), (I, 2I))."""
    assert w.dtype == torch.float32 and w.dim() == 2 and w.is_cuda and w.stride(1) == 1
    N2, K = w.shape
    I = N2 // 2
    cb, sb = nvfp4_packed_weight_bytes(N2, K)
    codes = _empty(cb, torch.uint8, w.device)
    scales = _empty(sb, torch.uint8, w.device)
    g = torch.empty(2, dtype=torch.float32, device=w.device)
    need = nvfp4_pack_weight_workspace_bytes(N2, K, 2)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=w.device)
    nvfp4_pack_weight_gate_up(w, I, K, w.stride(0), codes, scales, g, ws, ws.numel(), stream)
    return PackedWeight(codes, scales, g, N2, K, [(0, I), (I, N2)])


@_on_stream
def gemm_swiglu_quantize(a_codes, a_scales, a_g_dec, pw, amax_h, out=None, *, stream=None):
    """NVFP4 activations x interleaved gate/up weight -> NVFP4 of bf16(silu(g) * u):
    (codes uint8 [M, I/2], scales uint8 [M, I/16], g_dec float32 [1])."""
    M = a_codes.shape[0]
    I = pw.N // 2
    dev = a_codes.device
    if out is None:
        out = (torch.empty((M, I // 2), dtype=torch.uint8, device=dev),
               torch.empty((M, I // 16), dtype=torch.uint8, device=dev),
               torch.empty(1, dtype=torch.float32, device=dev))
    c, s, g = out
    nvfp4_gemm_swiglu_quantize(a_codes, a_scales, a_g_dec, M, pw.K, pw.codes, pw.scales, I, pw.g_dec, amax_h,
                               c, s, g, stream)
    return out


@_on_stream
def swiglu(gu, *, stream=None):
    """fp32 [M, 2I] gate+up output -> bf16 [M, I] = bf16(silu(g) * u)."""
    assert gu.dtype == torch.float32 and gu.dim() == 2 and gu.stride(1) == 1
    M, N2 = gu.shape
    h = torch.empty((M, N2 // 2), dtype=torch.bfloat16, device=gu.device)
    nvfp4_swiglu(gu, M, N2 // 2, gu.stride(0), h, h.stride(0), stream)
    return h


@_on_stream
def kv_fp8_encode(x, amax, out=None, *, stream=None):
    """Contiguous bf16 cuda tensor + device amax [1] -> uint8 E4M3FN codes of the same shape."""
    assert x.dtype == torch.bfloat16 and x.is_contiguous()
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if out is None else out
    nvfp4_kv_fp8_encode(x, x.numel(), amax, codes, stream)
    return codes


@_on_stream
def kv_fp8_decode(codes, amax, out=None, *, stream=None):
    """uint8 E4M3FN codes + device amax [1] -> bf16 tensor of the same shape."""
    assert codes.dtype == torch.uint8 and codes.is_contiguous()
    y = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device) if out is None else out
    nvfp4_kv_fp8_decode(codes, codes.numel(), amax, y, stream)
    return y


class AmaxObserver:
    """Running maximum of |x| over calibration batches, kept on the device."""

    def __init__(self, device):
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)
        self.ws = torch.empty(max(nvfp4_amax_observe_workspace_bytes(0, 0), 16), dtype=torch.uint8, device=device)

    @_on_stream
    def observe(self, x, *, stream=None):
        assert x.dtype == torch.bfloat16 and x.dim() == 2 and (x.stride(1) == 1 or x.shape[1] <= 1)
        M, K = x.shape
        nvfp4_amax_observe(x, M, K, max(x.stride(0), K), self.amax, self.ws, self.ws.numel(), stream)
        return self.amax


@_on_stream
def quantize_stats(x, amax, *, stream=None):
    """(saturated-scale blocks, clipped elements) of bf16 x under the static maximum amax [1]."""
    M, K = x.shape
    counts = torch.empty(2, dtype=torch.int32, device=x.device)
    nvfp4_quantize_stats(x, M, K, max(x.stride(0), K), amax, counts, stream)
    return counts


# ---- token mixers: paged cache, decode attention, gated linear attention ----------------
# A GPU's current hipStream_t as an integer, without the Stream object that
# torch.cuda.current_stream builds (2.8 us of a call whose kernels take 4).
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _on_device(fn):
    """For the mixers: runs a function with its first tensor's GPU current, on that
    GPU's current stream or on ``stream`` (keyword-only, a torch.cuda.Stream of it), and
    allocates there (see _on_stream)."""
    name = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kw):
        first = args[0] if args else kw.get(name)
        if not isinstance(first, torch.Tensor):
            raise TypeError(f"{fn.__name__}: {name}: a tensor is needed")
        dev = first.get_device()
        if stream is None and dev >= 0 and dev == torch.cuda.current_device():
            return fn(*args, stream=_current_stream(dev), **kw)
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise TypeError(f"{fn.__name__}: stream must be a torch.cuda.Stream "
                            "(the nvfp4_* wrappers take raw handles)")
        assert first.is_cuda, f"{fn.__name__}: a cuda tensor is needed"
        assert stream is None or stream.device == first.device, f"{fn.__name__}: the stream is another GPU's"
        with torch.cuda.device(first.device):
            if stream is None:
                return fn(*args, stream=_current_stream(dev), **kw)
            with torch.cuda.stream(stream):
                return fn(*args, stream=stream.cuda_stream, **kw)
    return wrapper


def _rows3(x, dev, dtype, T, H, D, what):
    """Checks a [T, H, D] tensor whose heads lie next to each other; its token stride."""
    assert x.dtype is dtype and x.shape == (T, H, D) and x.get_device() == dev, what
    s0, s1, s2 = x.stride()
    if T > 1:
        assert s2 == 1 and (s1 == D or H == 1), f"{what}: a token's heads must be contiguous"
        return s0
    assert T == 0 or (s2 == 1 and (s1 == D or H == 1)), f"{what}: a token's heads must be contiguous"
    return H * D                                     # one row: any stride will do


def _rows2(x, dev, T, H, what):
    """Checks an fp32 [T, H] tensor; its token stride."""
    assert x.dtype is torch.float32 and x.shape == (T, H) and x.get_device() == dev, what
    s0, s1 = x.stride()
    assert s1 == 1 or H == 1 or T == 0, f"{what}: a token's values must be contiguous"
    return s0 if T > 1 else H


def _table(x, dev, dtype, n, what):
    if x is not None:
        assert x.dtype is dtype and x.shape == (n,) and x.get_device() == dev and (n <= 1 or x.stride(0) == 1), what
    return x


def _scratch(workspace, x, nbytes):
    """A caller's Workspace, or a new one, of x's GPU: its buffer and size."""
    buf, nbytes = (Workspace(x.device) if workspace is None else workspace).get(nbytes)
    assert buf is None or buf.get_device() == x.get_device(), "workspace: another device's"
    return buf, nbytes


class PagedKVCache:
    """A paged key-value cache over two tensors [pages, page_size, kv_heads, head_dim] of the
    same strides (any layout whose rows are contiguous, e.g. views of [pages, 2, page_size,
    ...] or permuted [pages, kv_heads, page_size, ...]): bf16, or uint8 E4M3 codes with the
    calibrated maxima k_amax and v_amax (fp32 [1] on the GPU).  It holds these tensors, whose
    addresses every call takes from ``desc``: write into them at will; for others (or after
    one's storage was moved) make a new cache."""

    def __init__(self, k, v, k_amax=None, v_amax=None):
        assert k.dim() == 4 and k.dtype in (torch.bfloat16, torch.uint8) and k.is_cuda, "k: a 4-d bf16 or uint8 cuda tensor"
        assert v.dtype == k.dtype and v.shape == k.shape and v.stride() == k.stride() and v.device == k.device, \
            "v: the type, shape, strides and device of k"
        assert k.stride(3) == 1 or k.numel() == 0, "rows must be contiguous"
        for a in (k_amax, v_amax):
            assert (a is None) == (k.dtype == torch.bfloat16), "k_amax and v_amax belong to E4M3 codes, and only to them"
            assert a is None or (a.dtype == torch.float32 and a.numel() == 1 and a.device == k.device), "amax: fp32 [1]"
        self._tensors = k, v, k_amax, v_amax
        self.device_index = k.get_device()
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = k.shape
        s = k.stride()
        self.desc = KVCacheDesc(k.data_ptr(), v.data_ptr(), _ptr(k_amax), _ptr(v_amax), self.num_pages, s[0], s[1],
                                s[2], self.page_size, self.kv_heads, self.head_dim, DTYPE[k.dtype])
        self._desc_bytes = bytes(self.desc)

    # read-only: another tensor in their place would leave desc with the address of freed memory
    k = property(lambda self: self._tensors[0])
    v = property(lambda self: self._tensors[1])
    k_amax = property(lambda self: self._tensors[2])
    v_amax = property(lambda self: self._tensors[3])

    @classmethod
    def empty(cls, num_pages, page_size, kv_heads, head_dim, device, k_amax=None, v_amax=None):
        """A new cache (contents unset): E4M3 if the calibrated maxima are given, else bf16."""
        dtype = torch.bfloat16 if k_amax is None else torch.uint8
        k, v = (torch.empty((num_pages, page_size, kv_heads, head_dim), dtype=dtype, device=device) for _ in range(2))
        return cls(k, v, k_amax, v_amax)


@_on_device
def kv_append(k, v, cache, slots, q=None, positions=None, rope=None, interleaved=False, q_out=None, q_norm=None, k_norm=None,
              eps=1e-6, *, stream=None):
    """Rotates k (and q) by position, and appends k and v to a PagedKVCache at rows ``slots``.

    k, v: fp32 or bf16 [T, kv_heads, head_dim]; q: the same type, [T, q_heads, head_dim].
    slots, positions: int64 [T] (slot < 0: a padded row); rope: fp32 [max_pos, rot_dim], the
    cosines of a position's angles, then their sines; None: no rotation.  q_norm, k_norm: fp32
    [head_dim], the weights of a norm of each head before the rotation, x / sqrt(mean(x^2) + eps) * w;
    None: no norm.  Returns q, rotated, as bf16 (None without q)."""
    dev, D = cache.device_index, cache.head_dim
    T = k.shape[0]
    assert k.dtype in (torch.float32, torch.bfloat16), "k: fp32 or bf16"
    ldk = _rows3(k, dev, k.dtype, T, cache.kv_heads, D, "k")
    ldv = _rows3(v, dev, k.dtype, T, cache.kv_heads, D, "v")
    _table(slots, dev, torch.int64, T, "slots: int64 [T]")
    _table(positions, dev, torch.int64, T, "positions: int64 [T]")
    rot, far = 0, 0
    if rope is not None:
        assert rope.dtype == torch.float32 and rope.dim() == 2 and rope.is_contiguous() and rope.get_device() == dev, \
            "rope: contiguous fp32 [max_pos, rot_dim]"
        assert positions is not None, "rope needs positions"
        far, rot = rope.shape
    heads, ldq, ldqo = 0, 0, 0
    if q is not None:
        heads = q.shape[1]
        ldq = _rows3(q, dev, k.dtype, T, heads, D, "q")
        if q_out is None:
            q_out = torch.empty((T, heads, D), dtype=torch.bfloat16, device=k.device)
        ldqo = _rows3(q_out, dev, torch.bfloat16, T, heads, D, "q_out")
    else:
        assert q_out is None, "q_out needs q"
    if q_norm is not None or k_norm is not None:
        _table(q_norm, dev, torch.float32, D, "q_norm: fp32 [head_dim]")
        _table(k_norm, dev, torch.float32, D, "k_norm: fp32 [head_dim]")
        assert q is not None or q_norm is None, "q_norm needs q"
        nvfp4_kv_append_norm(q, k, v, DTYPE[k.dtype], T, heads, ldq, ldk, ldv, q_norm, k_norm, eps, rope, rot, far,
                             bool(interleaved), positions, slots, cache.desc, q_out, ldqo, stream)
        return q_out
    nvfp4_kv_append(q, k, v, DTYPE[k.dtype], T, heads, ldq, ldk, ldv, rope, rot, far, bool(interleaved), positions, slots,
                    cache.desc, q_out, ldqo, stream)
    return q_out


@_on_device
def attn_decode(q, cache, block_table, seq_lens, max_len=None, scale=None, window=0, workspace=None, out=None,
                lse=None, *, stream=None):
    """Attention of one new token a sequence over a PagedKVCache -> (out bf16 [B, q_heads, head_dim],
    lse fp32 [B, q_heads]).

    q: bf16 [B, q_heads, head_dim]; block_table: int32 [B, pages]; seq_lens: int32 [B], the new
    token's own included.  max_len: a bound of the lengths (default: what the table holds);
    scale: default head_dim ** -0.5; window: the last tokens attended to (0: all)."""
    dev, D = cache.device_index, cache.head_dim
    B, H = q.shape[0], q.shape[1]
    ldq = _rows3(q, dev, torch.bfloat16, B, H, D, "q")
    assert block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == B and \
        block_table.get_device() == dev and (block_table.stride(1) == 1 or block_table.shape[1] <= 1), \
        "block_table: int32 [B, pages]"
    pages = block_table.shape[1]
    if max_len is None:
        max_len = pages * cache.page_size
    assert max_len <= pages * cache.page_size, "max_len: more than the block table holds"
    _table(seq_lens, dev, torch.int32, B, "seq_lens: int32 [B]")
    if out is None:
        out = torch.empty((B, H, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    assert lse.dtype == torch.float32 and lse.shape == (B, H) and lse.is_contiguous() and lse.get_device() == dev, "lse"
    ldo = _rows3(out, dev, torch.bfloat16, B, H, D, "out")
    buf, nbytes = _scratch(workspace, q, nvfp4_attn_decode_workspace_bytes(B, H, cache.kv_heads, D, max_len, window))
    nvfp4_attn_decode(q, B, H, ldq, cache.desc, block_table, block_table.stride(0) if B > 1 else pages, seq_lens, max_len,
                      D ** -0.5 if scale is None else scale, window, out, ldo, lse, buf, nbytes, stream)
    return out, lse


def _gdn_args(q, k, v, g, beta, state, state_index, B, scale, out):
    """Checks the tensors of a recurrent layer; the arguments the two calls share, and `out`."""
    dev, T = q.get_device(), q.shape[0]
    Hk, Dk, Hv, Dv = q.shape[1], q.shape[2], v.shape[1], v.shape[2]
    ldq = _rows3(q, dev, torch.bfloat16, T, Hk, Dk, "q")
    ldk = _rows3(k, dev, torch.bfloat16, T, Hk, Dk, "k")
    ldv = _rows3(v, dev, torch.bfloat16, T, Hv, Dv, "v")
    ldg = _rows2(g, dev, T, Hv, "g")
    ldb = _rows2(beta, dev, T, Hv, "beta") if beta is not None else 0
    assert state.dtype == torch.float32 and state.dim() == 4 and state.shape[1:] == (Hv, Dk, Dv) and \
        state.is_contiguous() and state.get_device() == dev, "state: contiguous fp32 [states, v_heads, k_dim, v_dim]"
    _table(state_index, dev, torch.int32, B, "state_index: int32 [B]")
    if out is None:
        out = torch.empty((T, Hv, Dv), dtype=torch.bfloat16, device=q.device)
    ldo = _rows3(out, dev, torch.bfloat16, T, Hv, Dv, "out")
    return (q, ldq, k, ldk, v, ldv, g, ldg, beta, ldb), (Hk, Hv, Dk, Dv), (Dk ** -0.5 if scale is None else scale), \
        out, ldo


@_on_device
def gdn_step(q, k, v, g, beta, state, state_index=None, scale=None, out=None, *, stream=None):
    """One token for each of B sequences through a gated-delta-rule layer -> out bf16 [B, v_heads, v_dim].

    q, k: bf16 [B, k_heads, k_dim]; v: bf16 [B, v_heads, v_dim]; g (log decay) and beta: fp32
    [B, v_heads], beta None for linear attention with a decay; state: fp32 [states, v_heads,
    k_dim, v_dim], updated in place; state_index: int32 [B] (negative: a padded row)."""
    B = q.shape[0]
    first, dims, scale, out, ldo = _gdn_args(q, k, v, g, beta, state, state_index, B, scale, out)
    nvfp4_gdn_step(*first, B, *dims, state, state.shape[0], state_index, scale, out, ldo, stream)
    return out


@_on_device
def gdn_prefill(q, k, v, g, beta, state, cu_seqlens, has_state=None, state_index=None, scale=None, workspace=None,
                out=None, *, stream=None):
    """The prompts of B sequences, rows cu_seqlens[b]..cu_seqlens[b + 1], through a gated-delta-rule
    layer -> out bf16 [T, v_heads, v_dim]; tensors as in gdn_step.  has_state: int32 [B], whether
    a sequence starts from its state (None: all start from zero)."""
    B, T = cu_seqlens.shape[0] - 1, q.shape[0]
    first, dims, scale, out, ldo = _gdn_args(q, k, v, g, beta, state, state_index, B, scale, out)
    _table(cu_seqlens, q.get_device(), torch.int32, B + 1, "cu_seqlens: int32 [B + 1]")
    _table(has_state, q.get_device(), torch.int32, B, "has_state: int32 [B]")
    buf, nbytes = _scratch(workspace, q, nvfp4_gdn_prefill_workspace_bytes(T, B, *dims))
    nvfp4_gdn_prefill(*first, T, B, cu_seqlens, *dims, state, state.shape[0], state_index, has_state, scale, out, ldo,
                      buf, nbytes, stream)
    return out


# ---- drafted tokens: tree attention, verification, cache rows and pages that move -------
def _block_table(x, dev, B):
    """Checks a block table [B, pages]; its row stride."""
    assert x.dtype is torch.int32 and x.dim() == 2 and x.shape[0] == B and x.get_device() == dev and \
        (x.stride(1) == 1 or x.shape[1] <= 1), "block_table: int32 [B, pages]"
    return x.stride(0) if B > 1 else x.shape[1]


def _dense(x, dev, dtype, shape, what):
    """Checks a contiguous tensor (None passes)."""
    if x is not None:
        assert x.dtype is dtype and x.shape == shape and x.get_device() == dev and x.is_contiguous(), what
    return x


@_on_device
def attn_tree(q, cache, block_table, ctx_lens, parents=None, max_len=None, scale=None, window=0, workspace=None, out=None,
              lse=None, *, stream=None):
    """Attention of a tree of drafted tokens a sequence over a PagedKVCache -> (out bf16 [B, nodes, q_heads,
    head_dim], lse fp32 [B, nodes, q_heads]).

    q: bf16 [B, nodes, q_heads, head_dim], up to 64 nodes; block_table: int32 [B, pages]; ctx_lens: int32 [B],
    the tokens before the tree, whose node i is in the cache at ctx_lens[b] + i.  parents: int32 [B, nodes], the
    node that each continues (-1: the context; anything else than an earlier node: a padded node); None: chains.
    A node attends to the context, its ancestors and itself, of these to the last ``window`` (0: all).  max_len:
    a bound of ctx_lens (default: what the table holds beside the nodes); scale: default head_dim ** -0.5."""
    dev, D = cache.device_index, cache.head_dim
    assert q.dim() == 4, "q: bf16 [B, nodes, q_heads, head_dim]"
    B, W, H = q.shape[0], q.shape[1], q.shape[2]
    assert B <= 1 or W <= 1 or q.stride(0) == W * q.stride(1), "q: a sequence's nodes must follow the last one's"
    ldq = _rows3(q.view(B * W, H, D) if q.is_contiguous() else q.flatten(0, 1), dev, torch.bfloat16, B * W, H, D, "q")
    ldt = _block_table(block_table, dev, B)
    room = block_table.shape[1] * cache.page_size - W
    if max_len is None:
        max_len = room
    assert 0 <= max_len <= room, "max_len: more than the block table holds beside the nodes"
    _table(ctx_lens, dev, torch.int32, B, "ctx_lens: int32 [B]")
    _dense(parents, dev, torch.int32, (B, W), "parents: contiguous int32 [B, nodes]")
    if out is None:
        out = torch.empty((B, W, H, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, W, H), dtype=torch.float32, device=q.device)
    _dense(out, dev, torch.bfloat16, (B, W, H, D), "out: contiguous bf16 [B, nodes, q_heads, head_dim]")
    _dense(lse, dev, torch.float32, (B, W, H), "lse: contiguous fp32 [B, nodes, q_heads]")
    buf, nbytes = _scratch(workspace, q, nvfp4_attn_tree_workspace_bytes(B, W, H, cache.kv_heads, D, max_len, window))
    nvfp4_attn_tree(q, B, W, H, ldq, cache.desc, block_table, ldt, ctx_lens, parents, max_len,
                    D ** -0.5 if scale is None else scale, window, out, H * D, lse, buf, nbytes, stream)
    return out, lse


@_on_device
def verify_drafts(logits, drafts, parents=None, temperature=None, uniforms=None, draft_logits=None, workspace=None, out=None, *,
                  stream=None):
    """Which drafted tokens the target model accepts, and the token after them -> (tokens int64 [B, nodes],
    path int32 [B, nodes], counts int32 [B]): the first counts[b] of tokens[b] are the accepted tokens and the
    last one, of path[b] node 0 and the accepted nodes; -1 behind them.

    logits: fp32 [B, nodes, vocab], the target's after each node; drafts: int64 [B, nodes], the nodes' tokens
    (node 0: the last token known, not read); parents: as for attn_tree (None: chains); temperature: fp32 [B],
    0 for the greedy rule (None: all of them); uniforms: fp32 [B, nodes + 1], random numbers of [0, 1): one for
    each node's children, then one for the last token; draft_logits: fp32 [B, nodes, vocab] where a chain's tokens
    were drawn from their softmax at the same temperature (None: the drafts were picked without chance)."""
    dev = logits.get_device()
    assert logits.dim() == 3, "logits: fp32 [B, nodes, vocab]"
    B, W, V = logits.shape

    def rows(x, what):
        assert x.dtype is torch.float32 and x.shape == (B, W, V) and x.get_device() == dev, what
        if x.is_contiguous():
            return V
        s0, s1, s2 = x.stride()
        assert (s2 == 1 or V == 1) and (B <= 1 or W <= 1 or s0 == W * s1), f"{what}: rows must be contiguous and evenly spaced"
        return s1 if W > 1 else (s0 if B > 1 else V)
    ld = rows(logits, "logits: fp32 [B, nodes, vocab]")
    ldd = rows(draft_logits, "draft_logits: fp32 [B, nodes, vocab]") if draft_logits is not None else 0
    _dense(drafts, dev, torch.int64, (B, W), "drafts: contiguous int64 [B, nodes]")
    _dense(parents, dev, torch.int32, (B, W), "parents: contiguous int32 [B, nodes]")
    _dense(temperature, dev, torch.float32, (B,), "temperature: contiguous fp32 [B]")
    _dense(uniforms, dev, torch.float32, (B, W + 1), "uniforms: contiguous fp32 [B, nodes + 1]")
    assert temperature is None or uniforms is not None, "temperature needs uniforms"
    if out is None:
        out = (torch.empty((B, W), dtype=torch.int64, device=logits.device),
               torch.empty((B, W), dtype=torch.int32, device=logits.device),
               torch.empty(B, dtype=torch.int32, device=logits.device))
    tokens, path, counts = out
    _dense(tokens, dev, torch.int64, (B, W), "tokens: contiguous int64 [B, nodes]")
    _dense(path, dev, torch.int32, (B, W), "path: contiguous int32 [B, nodes]")
    _dense(counts, dev, torch.int32, (B,), "counts: contiguous int32 [B]")
    sampled = draft_logits is not None and temperature is not None
    buf, nbytes = _scratch(workspace, logits, nvfp4_verify_drafts_workspace_bytes(B, W, V, sampled))
    nvfp4_verify_drafts(logits, B, W, V, ld, draft_logits, ldd, drafts, parents, temperature, uniforms, tokens, path, counts,
                        buf, nbytes, stream)
    return tokens, path, counts


def _layers(caches, dev):
    """The descriptors of one cache or of several layers' as an array."""
    caches = [caches] if isinstance(caches, PagedKVCache) else caches
    here = [c._desc_bytes for c in caches if c.device_index == dev]     # (arrays of structs are slow to fill one by one)
    assert len(here) == len(caches), "caches: another device's"
    return (KVCacheDesc * len(here)).from_buffer_copy(b"".join(here)), len(here)


@_on_device
def kv_compact(block_table, ctx_lens, path, counts, caches, *, stream=None):
    """Moves the rows of accepted nodes to where their sequences go on, in one PagedKVCache or those of all layers
    (a list of up to 64 of one shape): row ctx_lens[b] + path[b, i] to ctx_lens[b] + i for i < counts[b].

    block_table: contiguous int32 [B, pages]; ctx_lens, counts: int32 [B]; path: int32 [B, nodes] (see verify_drafts)."""
    dev = block_table.get_device()
    B = block_table.shape[0]
    ldt = _block_table(block_table, dev, B)
    # (lengths on the device may reach any of a row's ldt entries)
    assert ldt == block_table.shape[1], "block_table: contiguous int32 [B, pages]"
    assert path.dim() == 2, "path: int32 [B, nodes]"
    _dense(path, dev, torch.int32, (B, path.shape[1]), "path: contiguous int32 [B, nodes]")
    _table(ctx_lens, dev, torch.int32, B, "ctx_lens: int32 [B]")
    _table(counts, dev, torch.int32, B, "counts: int32 [B]")
    descs, n = _layers(caches, dev)
    nvfp4_kv_compact(descs, n, block_table, ldt, B, path.shape[1], ctx_lens, path, counts, stream)


@_on_device
def kv_copy_pages(src, dst, caches, *, stream=None):
    """Copies page src[i] to page dst[i] (int32 [n]) in one PagedKVCache or those of all layers (a list of up to 64
    of one shape)."""
    dev, n = src.get_device(), src.shape[0]
    _table(src, dev, torch.int32, n, "src: int32 [n]")
    _table(dst, dev, torch.int32, n, "dst: int32 [n]")
    descs, layers = _layers(caches, dev)
    nvfp4_kv_copy_pages(descs, layers, src, dst, n, stream)
