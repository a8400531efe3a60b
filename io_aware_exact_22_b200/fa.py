"""ctypes binding over libfa.so (C ABI in include/fa.h).

Every name in ``EXPORTS`` (``fa_fwd``, ``fa_bwd``, the split-KV, FP8, deterministic,
allocation-free and sharded-pieces entry points, the norm + rotation and paged-cache calls, the
status and self-test calls) has a function here with the C name that only marshals arguments:
torch tensors supply device pointers and the current CUDA stream, and every step of the
attention path runs in the library's kernels.  ``forward``, ``forward_splitkv``,
``forward_fp8``, ``backward``, ``qk_norm_rope``, ``qk_norm_rope_backward``, ``paged_plan``,
``paged_append`` and ``paged_decode`` additionally check their tensors and allocate the outputs
that are not given with torch (memory plumbing only); the last five do so in a small extension
(csrc/fa_torch.cpp), on the tensors' device and its current stream.

Loading fails loudly (``RuntimeError``) when the shared library is missing: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("FA_LIB_PATH", os.path.join(_HERE, "libfa.so"))

STATUS = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_CUDA",
          4: "FA_ERR_TIMEOUT", 5: "FA_ERR_DEVICE_CHECK"}
EXPORTS = ("fa_fwd", "fa_bwd", "fa_bwd_workspace_bytes", "fa_get_device_status",
           "fa_status_string", "fa_version", "fa_bwd_noalloc", "fa_selftest_wait_timeout",
           "fa_fwd_splitkv", "fa_fwd_splitkv_workspace_bytes", "fa_fwd_splitkv_default_splits",
           "fa_bwd_deterministic", "fa_fwd_fp8", "fa_fwd_partial", "fa_merge_partials", "fa_fwd_carry",
           "fa_bwd_prepare", "fa_bwd_accumulate", "fa_bwd_finish", "fa_bwd_contribute", "fa_bwd_acc_add",
           "fa_bwd_main", "fa_bwd_dq_post",
           "fa_qk_norm_rope", "fa_qk_norm_rope_bwd", "fa_qk_norm_rope_bwd_workspace_bytes",
           "fa_paged_plan", "fa_paged_append", "fa_paged_decode", "fa_paged_decode_workspace_bytes",
           "fa_debug_build", "fa_debug_visits")
# Size of the library's built-in scratch used by fa_bwd_noalloc (include/fa.h).
NOALLOC_MAX_SCRATCH_BYTES = 64 << 20
# fa_paged_plan: most requests of a step and the bits of its status (include/fa.h).
PLAN_MAX_REQUESTS = 12288
PAGED_MAX_LEN = 2**31 - 2**16  # most tokens of a row of the block table, and of a step
PLAN_NO_PAGES, PLAN_ROW_FULL, PLAN_TOO_MANY_TOKENS, PLAN_BAD_INPUT = 1, 2, 4, 8

_lib = None


class FAError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what} failed: {STATUS.get(code, code)}")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libfa.so once; raise RuntimeError if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfa.so not found at {LIB_PATH}; build it with "
                               "`python -m io_aware_exact_22_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd.restype = i
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_fp8.restype = i
        L.fa_fwd_partial.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_fwd_partial.restype = i
        L.fa_merge_partials.argtypes = [vp, vp, i, vp, vp, i, i, i, i, vp]
        L.fa_merge_partials.restype = i
        L.fa_fwd_carry.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
        L.fa_fwd_carry.restype = i
        L.fa_bwd_prepare.argtypes = [vp, vp, vp, vp, sz, i, i, i, i, vp]
        L.fa_bwd_prepare.restype = i
        L.fa_bwd_accumulate.argtypes = [vp, vp, vp, vp, vp, sz, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_accumulate.restype = i
        L.fa_bwd_finish.argtypes = [vp, sz, vp, vp, vp, vp, vp, i, i, i, i, f, vp]
        L.fa_bwd_finish.restype = i
        L.fa_bwd_contribute.argtypes = [vp, vp, vp, vp, vp, sz, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_contribute.restype = i
        L.fa_bwd_acc_add.argtypes = [vp, vp, i, i, i, i, vp]
        L.fa_bwd_acc_add.restype = i
        L.fa_bwd_main.argtypes = [vp, vp, vp, vp, vp, sz, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_main.restype = i
        L.fa_bwd_dq_post.argtypes = [vp, sz, vp, i, i, i, i, f, vp]
        L.fa_bwd_dq_post.restype = i
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, i, i, i, i, f, i, vp]
        L.fa_bwd.restype = i
        L.fa_bwd_workspace_bytes.argtypes = [i, i, i, i]
        L.fa_bwd_workspace_bytes.restype = sz
        L.fa_get_device_status.argtypes = [vp]
        L.fa_get_device_status.restype = i
        L.fa_status_string.argtypes = [i]
        L.fa_status_string.restype = ctypes.c_char_p
        L.fa_version.argtypes = []
        L.fa_version.restype = i
        L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        L.fa_bwd_noalloc.restype = i
        L.fa_selftest_wait_timeout.argtypes = [i, vp]
        L.fa_selftest_wait_timeout.restype = i
        L.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp, sz, vp]
        L.fa_fwd_splitkv.restype = i
        L.fa_fwd_splitkv_workspace_bytes.argtypes = [i, i, i, i, i]
        L.fa_fwd_splitkv_workspace_bytes.restype = sz
        L.fa_fwd_splitkv_default_splits.argtypes = [i, i, i, i, i]
        L.fa_fwd_splitkv_default_splits.restype = i
        L.fa_debug_build.argtypes = []
        L.fa_debug_build.restype = i
        L.fa_debug_visits.argtypes = [vp, sz, i, vp]
        L.fa_debug_visits.restype = i
        ll = ctypes.c_longlong
        rot = [vp, i, i, i, vp]  # rope, rope_rows, rot, interleaved, positions
        L.fa_qk_norm_rope.argtypes = [vp] * 4 + rot + [ll, vp, vp] + [i] * 5 + [ll] * 6 + [f, vp]
        L.fa_qk_norm_rope.restype = i
        L.fa_qk_norm_rope_bwd_workspace_bytes.argtypes = [i] * 5
        L.fa_qk_norm_rope_bwd_workspace_bytes.restype = sz
        L.fa_qk_norm_rope_bwd.argtypes = ([vp] * 6 + rot + [ll] + [vp] * 5 + [sz] + [i] * 5 + [ll] * 12 + [f, vp])
        L.fa_qk_norm_rope_bwd.restype = i
        L.fa_paged_plan.argtypes = [vp, vp, vp, ll, i, vp, i, vp, i, i, i] + [vp] * 8
        L.fa_paged_plan.restype = i
        L.fa_paged_append.argtypes = ([vp] * 5 + rot + [vp] * 4 + [i, vp, vp] + [i] * 6 + [ll] * 9 + [f, vp])
        L.fa_paged_append.restype = i
        L.fa_paged_decode.argtypes = ([vp] * 3 + [i, vp, vp, vp, ll, i, i] + [vp] * 5 + [sz] + [i] * 6 + [ll] * 5
                                      + [f, vp])
        L.fa_paged_decode.restype = i
        L.fa_paged_decode_workspace_bytes.argtypes = [i] * 4
        L.fa_paged_decode_workspace_bytes.restype = sz
        L.fa_bwd_deterministic.argtypes = L.fa_bwd.argtypes
        L.fa_bwd_deterministic.restype = i
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ C-named wrappers
def fa_fwd(q, k, v, o, lse, B, H, N, d, scale, causal, stream=None) -> int:
    return lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                        float(scale), int(causal), _stream(stream))


def fa_fwd_fp8(q, k, v, descale_q, descale_k, descale_v, o, lse, B, H, N, d, scale, causal,
               stream=None) -> int:
    return lib().fa_fwd_fp8(_ptr(q), _ptr(k), _ptr(v), _ptr(descale_q), _ptr(descale_k),
                            _ptr(descale_v), _ptr(o), _ptr(lse), B, H, N, d, float(scale),
                            int(causal), _stream(stream))


def fa_fwd_partial(q, k, v, o_part, lse_part, B, H, N, d, scale, causal, stream=None) -> int:
    return lib().fa_fwd_partial(_ptr(q), _ptr(k), _ptr(v), _ptr(o_part), _ptr(lse_part), B, H, N, d,
                                float(scale), int(causal), _stream(stream))


FA_CARRY_IN, FA_CARRY_FINAL = 1, 2


def fa_fwd_carry(q, k, v, o_part, lse_part, o, lse, B, H, N, d, scale, causal, flags, stream=None) -> int:
    return lib().fa_fwd_carry(_ptr(q), _ptr(k), _ptr(v), _ptr(o_part), _ptr(lse_part), _ptr(o), _ptr(lse), B, H,
                              N, d, float(scale), int(causal), int(flags), _stream(stream))


def fa_merge_partials(o_parts, lse_parts, nparts, o, lse, B, H, N, d, stream=None) -> int:
    return lib().fa_merge_partials(_ptr(o_parts), _ptr(lse_parts), int(nparts), _ptr(o), _ptr(lse), B, H,
                                   N, d, _stream(stream))


def fa_bwd_prepare(o, dO, lse, workspace, workspace_bytes, B, H, N, d, stream=None) -> int:
    return lib().fa_bwd_prepare(_ptr(o), _ptr(dO), _ptr(lse), _ptr(workspace), int(workspace_bytes), B, H,
                                N, d, _stream(stream))


def fa_bwd_accumulate(q, k, v, dO, workspace, workspace_bytes, dk_acc, dv_acc, B, H, N, d, scale,
                      causal, stream=None) -> int:
    return lib().fa_bwd_accumulate(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(workspace),
                                   int(workspace_bytes), _ptr(dk_acc), _ptr(dv_acc), B, H, N, d,
                                   float(scale), int(causal), _stream(stream))


def fa_bwd_finish(workspace, workspace_bytes, dk_acc, dv_acc, dq, dk, dv, B, H, N, d, scale,
                  stream=None) -> int:
    return lib().fa_bwd_finish(_ptr(workspace), int(workspace_bytes), _ptr(dk_acc), _ptr(dv_acc),
                               _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale), _stream(stream))


def fa_bwd_contribute(q, k, v, dO, workspace, workspace_bytes, dk_out, dv_out, B, H, N, d, scale, causal,
                      stream=None) -> int:
    return lib().fa_bwd_contribute(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(workspace), int(workspace_bytes),
                                   _ptr(dk_out), _ptr(dv_out), B, H, N, d, float(scale), int(causal),
                                   _stream(stream))


def fa_bwd_acc_add(acc, x, B, H, N, d, stream=None) -> int:
    return lib().fa_bwd_acc_add(_ptr(acc), _ptr(x), B, H, N, d, _stream(stream))


def fa_bwd_main(q, k, v, dO, workspace, workspace_bytes, dk, dv, B, H, N, d, scale, causal,
                stream=None) -> int:
    return lib().fa_bwd_main(_ptr(q), _ptr(k), _ptr(v), _ptr(dO), _ptr(workspace), int(workspace_bytes),
                             _ptr(dk), _ptr(dv), B, H, N, d, float(scale), int(causal), _stream(stream))


def fa_bwd_dq_post(workspace, workspace_bytes, dq, B, H, N, d, scale, stream=None) -> int:
    return lib().fa_bwd_dq_post(_ptr(workspace), int(workspace_bytes), _ptr(dq), B, H, N, d, float(scale),
                                _stream(stream))


def fa_fwd_splitkv(q, k, v, o, lse, B, H, N, d, scale, causal, num_splits, workspace,
                   workspace_bytes, stream=None) -> int:
    return lib().fa_fwd_splitkv(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                float(scale), int(causal), int(num_splits), _ptr(workspace),
                                int(workspace_bytes), _stream(stream))


def fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits) -> int:
    return lib().fa_fwd_splitkv_workspace_bytes(B, H, N, d, num_splits)


def fa_fwd_splitkv_default_splits(B, H, N, d, causal) -> int:
    return lib().fa_fwd_splitkv_default_splits(B, H, N, d, int(causal))


def fa_bwd(q, k, v, o, dO, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d, scale,
           causal, stream=None) -> int:
    return lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq),
                        _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes), B, H, N, d,
                        float(scale), int(causal), _stream(stream))


def fa_bwd_deterministic(q, k, v, o, dO, lse, dq, dk, dv, workspace, workspace_bytes, B, H, N, d,
                         scale, causal, stream=None) -> int:
    return lib().fa_bwd_deterministic(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                                      _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                      int(workspace_bytes), B, H, N, d, float(scale), int(causal),
                                      _stream(stream))


def fa_bwd_noalloc(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal,
                   stream=None) -> int:
    """fa_bwd without a workspace: the library's fixed scratch array is used instead, for
    callers that cannot allocate device memory.  Overlapping calls race on that array."""
    return lib().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse),
                                _ptr(dq), _ptr(dk), _ptr(dv), B, H, N, d, float(scale),
                                int(causal), _stream(stream))


def fa_bwd_workspace_bytes(B, H, N, d) -> int:
    return lib().fa_bwd_workspace_bytes(B, H, N, d)


def fa_qk_norm_rope(q, k, wq, wk, rope, rope_rows, rot, interleaved, positions, pos_sb, q_out, k_out, B, N, Hq, Hk,
                    d, q_strides, k_strides, eps, stream=None) -> int:
    """q_strides, k_strides: (batch, token, head) in elements."""
    return lib().fa_qk_norm_rope(_ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(rope), rope_rows, rot, int(interleaved),
                                 _ptr(positions), pos_sb, _ptr(q_out), _ptr(k_out), B, N, Hq, Hk, d, *q_strides,
                                 *k_strides, eps, _stream(stream))


def fa_qk_norm_rope_bwd_workspace_bytes(B, N, Hq, Hk, d) -> int:
    return lib().fa_qk_norm_rope_bwd_workspace_bytes(B, N, Hq, Hk, d)


def fa_qk_norm_rope_bwd(gq, gk, q, k, wq, wk, rope, rope_rows, rot, interleaved, positions, pos_sb, dq, dk, dwq, dwk,
                        workspace, workspace_bytes, B, N, Hq, Hk, d, q_strides, k_strides, dq_strides, dk_strides, eps,
                        stream=None) -> int:
    return lib().fa_qk_norm_rope_bwd(_ptr(gq), _ptr(gk), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), _ptr(rope), rope_rows,
                                     rot, int(interleaved), _ptr(positions), pos_sb, _ptr(dq), _ptr(dk), _ptr(dwq),
                                     _ptr(dwk), _ptr(workspace), int(workspace_bytes), B, N, Hq, Hk, d, *q_strides,
                                     *k_strides, *dq_strides, *dk_strides, eps, _stream(stream))


def fa_paged_plan(cached, new_tokens, block_table, table_stride, table_cols, free_pages, pool_pages, free_count,
                  page_size, R, max_tokens, lens, cu_tokens, slots, positions, token_req, free_count_out, plan_status,
                  stream=None) -> int:
    return lib().fa_paged_plan(_ptr(cached), _ptr(new_tokens), _ptr(block_table), table_stride, table_cols,
                               _ptr(free_pages), pool_pages, _ptr(free_count), page_size, R, max_tokens, _ptr(lens),
                               _ptr(cu_tokens), _ptr(slots), _ptr(positions), _ptr(token_req), _ptr(free_count_out),
                               _ptr(plan_status), _stream(stream))


def fa_paged_append(q, k, v, wq, wk, rope, rope_rows, rot, interleaved, positions, slots, q_out, k_cache, v_cache,
                    cache_fp8, k_descale, v_descale, num_pages, page_size, T, Hq, Hk, d, q_strides, k_strides,
                    v_strides, cache_strides, eps, stream=None) -> int:
    """q_strides, k_strides, v_strides: (token, head); cache_strides: (page, token, head)."""
    return lib().fa_paged_append(_ptr(q), _ptr(k), _ptr(v), _ptr(wq), _ptr(wk), _ptr(rope), rope_rows, rot,
                                 int(interleaved), _ptr(positions), _ptr(slots), _ptr(q_out), _ptr(k_cache),
                                 _ptr(v_cache), int(cache_fp8), _ptr(k_descale), _ptr(v_descale), num_pages, page_size,
                                 T, Hq, Hk, d, *q_strides, *k_strides, *v_strides, *cache_strides, eps,
                                 _stream(stream))


def fa_paged_decode_workspace_bytes(T, Hq, Hk, d) -> int:
    return lib().fa_paged_decode_workspace_bytes(T, Hq, Hk, d)


def fa_paged_decode(q, k_cache, v_cache, cache_fp8, k_descale, v_descale, block_table, table_stride, table_rows,
                    table_cols, lens, req, o, lse, workspace, workspace_bytes, num_pages, page_size, T, Hq, Hk, d,
                    q_strides, cache_strides, scale, stream=None) -> int:
    return lib().fa_paged_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), int(cache_fp8), _ptr(k_descale),
                                 _ptr(v_descale), _ptr(block_table), table_stride, table_rows, table_cols, _ptr(lens),
                                 _ptr(req), _ptr(o), _ptr(lse), _ptr(workspace), int(workspace_bytes), num_pages,
                                 page_size, T, Hq, Hk, d, *q_strides, *cache_strides, scale, _stream(stream))


def fa_get_device_status(stream=None) -> int:
    return lib().fa_get_device_status(_stream(stream))


def fa_selftest_wait_timeout(limit_ms: int, stream=None) -> int:
    return lib().fa_selftest_wait_timeout(int(limit_ms), _stream(stream))


def fa_status_string(code: int) -> str:
    return lib().fa_status_string(code).decode()


def fa_version() -> int:
    return lib().fa_version()


def fa_debug_build() -> int:
    return lib().fa_debug_build()


def fa_debug_visits(counts, n: int, clear: bool, stream=None) -> int:
    """Copies the first n visit counters of the debug build into `counts` (a contiguous CPU
    int32 tensor or numpy array), then zeroes them all when `clear`."""
    ptr = counts.ctypes.data if hasattr(counts, "ctypes") else _ptr(counts)
    return lib().fa_debug_visits(ptr, int(n), int(clear), _stream(stream))


# ------------------------------------------------------------------ tensor conveniences
def _check(t, name):
    if not (t.is_cuda and t.dtype == torch.bfloat16 and t.dim() == 4 and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous CUDA bf16 tensor [B,H,N,d]")


def forward(q, k, v, causal: bool, scale: float | None = None, out=None, lse=None):
    """O, LSE = attention(q, k, v) through fa_fwd.  Inputs: contiguous bf16 [B,H,N,d] on CUDA."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    B, H, N, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    rc = fa_fwd(q, k, v, out, lse, B, H, N, d, scale, causal)
    if rc:
        raise FAError(rc, "fa_fwd")
    return out, lse


def forward_fp8(q8, k8, v8, descale_q, descale_k, descale_v, causal: bool,
                scale: float | None = None, out=None, lse=None):
    """O (bf16), LSE = attention of FP8 inputs through fa_fwd_fp8.  q8, k8, v8: contiguous
    CUDA tensors [B,H,N,d] of E4M3 codes (torch.uint8 or torch.float8_e4m3fn); descale_*:
    fp32 CUDA tensors with B*H elements, or None for 1."""
    for t, n in ((q8, "q8"), (k8, "k8"), (v8, "v8")):
        if not (t.is_cuda and t.element_size() == 1 and t.dim() == 4 and t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous CUDA tensor of E4M3 codes [B,H,N,d]")
    B, H, N, d = q8.shape
    for t, n in ((descale_q, "descale_q"), (descale_k, "descale_k"), (descale_v, "descale_v")):
        if t is not None and not (t.is_cuda and t.dtype == torch.float32 and t.numel() == B * H
                                  and t.is_contiguous()):
            raise ValueError(f"{n} must be a contiguous CUDA fp32 tensor of B*H elements")
    scale = d ** -0.5 if scale is None else scale
    if out is None:
        out = torch.empty((B, H, N, d), device=q8.device, dtype=torch.bfloat16)
    if lse is None:
        lse = torch.empty((B, H, N), device=q8.device, dtype=torch.float32)
    rc = fa_fwd_fp8(q8, k8, v8, descale_q, descale_k, descale_v, out, lse, B, H, N, d, scale,
                    causal)
    if rc:
        raise FAError(rc, "fa_fwd_fp8")
    return out, lse


def forward_splitkv(q, k, v, causal: bool, scale: float | None = None, num_splits: int = 0,
                    out=None, lse=None, workspace=None):
    """Split-KV forward (fa_fwd_splitkv); the workspace is allocated with torch if not given."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    B, H, N, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    sp = num_splits if num_splits > 0 else fa_fwd_splitkv_default_splits(B, H, N, d, causal)
    sp = max(1, min(sp, (N + 127) // 128))
    nbytes = fa_fwd_splitkv_workspace_bytes(B, H, N, d, sp)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, device=q.device, dtype=torch.uint8)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), device=q.device, dtype=torch.float32)
    rc = fa_fwd_splitkv(q, k, v, out, lse, B, H, N, d, scale, causal, sp, workspace,
                        0 if workspace is None else workspace.numel())
    if rc:
        raise FAError(rc, "fa_fwd_splitkv")
    return out, lse


def backward(q, k, v, o, do, lse, causal: bool, scale: float | None = None, workspace=None,
             dq=None, dk=None, dv=None, deterministic: bool = False):
    """dQ, dK, dV through fa_bwd, or fa_bwd_deterministic (workspace allocated with torch when
    not given)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "dO")):
        _check(t, n)
    B, H, N, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    nbytes = fa_bwd_workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), device=q.device, dtype=torch.uint8)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    fn = fa_bwd_deterministic if deterministic else fa_bwd
    rc = fn(q, k, v, o, do, lse, dq, dk, dv, workspace, workspace.numel(), B, H, N, d, scale, causal)
    if rc:
        raise FAError(rc, fn.__name__)
    return dq, dk, dv


# ------------------------------------------------------------------ norm + rotation, paged cache
def rope_table(rows: int, rot: int, base: float = 10000.0, device="cuda"):
    """fp32 [rows, 2, rot/2]: cos and sin of p * base^(-2i/rot), p the row, from 64-bit angles (a
    plan made once, with torch)."""
    inv = base ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    ang = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * inv[None]
    return torch.stack([ang.cos(), ang.sin()], 1).float().contiguous()


# The calls below are as short on the device as marshalling them in Python would be on the host, so
# their tensors go to a small extension (csrc/fa_torch.cpp) that checks them, allocates the outputs
# that are not given, and calls the C function on the tensors' device and its current stream.
_ext = None


def _load_ext():
    """The extension, bound to the library that ``lib`` loads; raise RuntimeError if it is not built."""
    global _ext
    L = lib()
    try:
        from . import _fa_torch
    except ImportError as e:
        raise RuntimeError("_fa_torch.so not found beside fa.py, or not for this torch; build it with "
                           "`python -m io_aware_exact_22_b200.build`") from e
    _fa_torch.bind({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in EXPORTS})
    _ext = _fa_torch
    return _ext


def _result(r, name):
    """What the extension returned; a C status other than FA_OK is an error."""
    if type(r) is int and r:
        raise FAError(r, name)
    return r


def qk_norm_rope(q, k, wq, wk, rope, positions=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                 k_out=None):
    """Per-head RMS norm and position rotation of q [B,N,Hq,d] and k [B,N,Hk,d] (bf16, any strides
    with the last dimension contiguous, for instance views of one fused projection), written as
    contiguous [B,Hq,N,d] and [B,Hk,N,d], the layout that ``forward`` reads.  wq, wk: bf16 [d] or
    None; rope: ``rope_table``'s or None for the norm alone; positions: int32 [N] or [B,N], or
    None for 0..N-1."""
    return _result((_ext or _load_ext()).qk_norm_rope(q, k, wq, wk, rope, positions, eps, interleaved, q_out, k_out),
                   "fa_qk_norm_rope")


def qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope, positions=None, eps: float = 1e-6, interleaved: bool = False,
                          dq=None, dk=None, workspace=None):
    """dq, dk (bf16 [B,N,H,d]), dwq, dwk (fp32 [d]) from gq [B,Hq,N,d], gk [B,Hk,N,d], the
    gradients of qk_norm_rope's outputs (``backward``'s dq, dk); dq, dk may be given as views, for
    instance of a fused projection's gradient."""
    return _result((_ext or _load_ext()).qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope, positions, eps, interleaved,
                                                               dq, dk, workspace), "fa_qk_norm_rope_bwd")


def paged_plan(cached, new_tokens, block_table, free_pages, free_count, page_size: int, lens, cu_tokens, slots,
               positions, token_req, free_count_out, status):
    """One serving step's pages and slots (fa_paged_plan): int32 CUDA tensors cached [R], new_tokens
    [R] (-1 ends a request), block_table [R, cols] (updated), free_pages [pool] and free_count [1]
    (the stack of free pages, updated) in; lens [R], cu_tokens [R+1], slots (int64), positions,
    token_req [max_tokens], free_count_out [1], status [1] out.  lens may be ``cached`` and
    free_count_out ``free_count``.  Nothing is read back: a step that cannot be planned leaves a
    non-zero status (PLAN_*) on the device, slots of -1 and everything else as it was."""
    _result((_ext or _load_ext()).paged_plan(cached, new_tokens, block_table, free_pages, free_count, page_size, lens,
                                             cu_tokens, slots, positions, token_req, free_count_out, status),
            "fa_paged_plan")


def paged_append(q, k, v, wq, wk, rope, positions, slots, k_cache, v_cache, eps: float = 1e-6,
                 interleaved: bool = False, k_descale=None, v_descale=None, q_out=None):
    """qk_norm_rope for T new tokens, q [T,Hq,d], k, v [T,Hk,d] (bf16, strided views allowed), with k
    and v written to the paged cache at ``slots`` (int64 [T]; negative: the token is skipped and
    its row of q_out stays as it was).  Returns q_out [T,Hq,d]."""
    return _result((_ext or _load_ext()).paged_append(q, k, v, wq, wk, rope, positions, slots, k_cache, v_cache, eps,
                                                      interleaved, k_descale, v_descale, q_out), "fa_paged_append")


def paged_decode(q, k_cache, v_cache, block_table, lens, scale: float | None = None, req=None, k_descale=None,
                 v_descale=None, out=None, lse=None, workspace=None):
    """O [T,Hq,d] (bf16), LSE [T,Hq] of one query token per row, q [T,Hq,d], over the paged cache (scale: 1/sqrt(d)
    if None): row t sees lens[t] keys (int32, on the device) of row req[t] of the block table (int32; None: of
    row t; negative: the output row stays as it was).  A row with no key gets O = 0, LSE = -inf."""
    return _result((_ext or _load_ext()).paged_decode(q, k_cache, v_cache, block_table, lens, scale, req, k_descale,
                                                      v_descale, out, lse, workspace), "fa_paged_decode")
