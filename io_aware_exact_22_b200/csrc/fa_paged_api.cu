// fa_paged_api.cu - the C ABI of the norm + rotation calls and of the paged cache (declared in
// include/fa.h): argument validation and launches, as fa_api.cu does for the attention calls.
#include "fa.h"
#include "fa_internal.cuh"

#include <climits>
#include <cmath>
#include <cstdint>

using namespace fa;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// A tensor that must be there (16-byte aligned) when `used`.
bool rows_ok(const void* p, bool used) { return !used || (p && aligned(p, 16)); }

// A stride of `count` rows handed to 16-byte accesses: a multiple of `unit` elements, and small enough
// that no offset in use overflows (|stride| * count < 2^59).  Of one row, the stride is not looked at.
bool stride_ok(long long s, long long count, long long unit) {
  if (count <= 1) return true;
  return s % unit == 0 && std::fabs((double)s) * (double)count < 5.7e17;
}

// What the three norm + rotation calls share.
fa_status_t check_rope(const void* wq, const void* wk, const float* rope, int rope_rows, int rot, int interleaved,
                       int d, float eps) {
  if (interleaved != 0 && interleaved != 1) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(eps) && eps >= 0.f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (rot < 0 || rot > d) return FA_ERR_INVALID_ARG;
  if (rot % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (rot > 0 && (!rope || !aligned(rope, 16) || rope_rows < 1)) return FA_ERR_INVALID_ARG;
  if (!aligned(wq, 16) || !aligned(wk, 16)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Sizes of a [B, N, Hq + Hk (+ Hk), d] problem: non-negative, and a warp for every row at most.
bool sizes_ok(int B, int N, int Hq, int Hk, int d) {
  if (B < 0 || N < 0 || Hq < 0 || Hk < 0) return false;
  const double heads = (double)Hq + 2.0 * Hk;
  return heads < 2147483647.0 / 256 && (double)B * N * (heads + 1) < 8.0 * 2147483647.0 &&
         (double)B * N * heads * d < 4.6e18;
}

const __nv_bfloat16* bf(const void* p) { return static_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* bf(void* p) { return static_cast<__nv_bfloat16*>(p); }

// Partial weight gradients of the backward: a row for each block that it may have.  How many it has goes
// up and down with the problem (592 for 2368 tokens of 16 + 16 heads, 298 for 2372), the size does not:
// a buffer made for one problem serves every other of its d.
size_t bwd_bytes(int d) { return (size_t)kNormRopeBwdBlocks * d * 4; }

// The cache's shape: strides in elements of `size` bytes, all of them multiples of 16 bytes.
bool cache_ok(const void* k, const void* v, int num_pages, int page_size, int Hk, long long c_sp, long long c_st,
              long long c_sh, int size) {
  if (!rows_ok(k, true) || !rows_ok(v, true) || num_pages < 1 || page_size < 1) return false;
  const long long unit = 16 / size;
  if (c_sp < 0 || c_st < 0 || c_sh < 0) return false;
  return stride_ok(c_sp, num_pages, unit) && stride_ok(c_st, page_size, unit) && stride_ok(c_sh, Hk, unit);
}

}  // namespace

extern "C" {

fa_status_t fa_qk_norm_rope(const void* q, const void* k, const void* wq, const void* wk, const float* rope,
                            int rope_rows, int rot, int interleaved, const int* positions, long long pos_sb,
                            void* q_out, void* k_out, int B, int N, int Hq, int Hk, int d, long long q_sb,
                            long long q_sn, long long q_sh, long long k_sb, long long k_sn, long long k_sh, float eps,
                            void* stream) {
  if (!sizes_ok(B, N, Hq, Hk, d)) return FA_ERR_INVALID_ARG;
  fa_status_t st = check_rope(wq, wk, rope, rope_rows, rot, interleaved, d, eps);
  if (st != FA_OK) return st;
  if ((long long)B * N == 0 || Hq + Hk == 0) return FA_OK;
  if (!rows_ok(q, Hq > 0) || !rows_ok(k, Hk > 0) || !rows_ok(q_out, Hq > 0) || !rows_ok(k_out, Hk > 0))
    return FA_ERR_INVALID_ARG;
  if (Hq > 0 && !(stride_ok(q_sb, B, 8) && stride_ok(q_sn, N, 8) && stride_ok(q_sh, Hq, 8))) return FA_ERR_INVALID_ARG;
  if (Hk > 0 && !(stride_ok(k_sb, B, 8) && stride_ok(k_sn, N, 8) && stride_ok(k_sh, Hk, 8))) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || (rot > 0 && !positions && rope_rows < N)) return FA_ERR_INVALID_ARG;
  if ((st = (fa_status_t)device_check()) != FA_OK) return st;
  NormRopeArgs a = {};
  if (!(a.status = device_status_word())) return FA_ERR_CUDA;
  a.q = bf(q), a.k = bf(k), a.wq = bf(wq), a.wk = bf(wk);
  a.rope = rope, a.rope_rows = rope_rows, a.rot = rot;
  a.positions = positions, a.pos_sb = pos_sb;
  a.q_out = bf(q_out), a.k_out = bf(k_out);
  a.q_sb = q_sb, a.q_sn = q_sn, a.q_sh = q_sh, a.k_sb = k_sb, a.k_sn = k_sn, a.k_sh = k_sh;
  a.B = B, a.N = N, a.Hq = Hq, a.Hk = Hk, a.eps = eps;
  return launch_norm_rope(d, interleaved != 0, 0, a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_qk_norm_rope_bwd_workspace_bytes(int B, int N, int Hq, int Hk, int d) {
  if (!sizes_ok(B, N, Hq, Hk, d) || (d != 64 && d != 128) || (long long)B * N == 0 || Hq + Hk == 0) return 0;
  return bwd_bytes(d);
}

fa_status_t fa_qk_norm_rope_bwd(const void* gq, const void* gk, const void* q, const void* k, const void* wq,
                                const void* wk, const float* rope, int rope_rows, int rot, int interleaved,
                                const int* positions, long long pos_sb, void* dq, void* dk, float* dwq, float* dwk,
                                void* workspace, size_t workspace_bytes, int B, int N, int Hq, int Hk, int d,
                                long long q_sb, long long q_sn, long long q_sh, long long k_sb, long long k_sn,
                                long long k_sh, long long dq_sb, long long dq_sn, long long dq_sh, long long dk_sb,
                                long long dk_sn, long long dk_sh, float eps, void* stream) {
  if (!sizes_ok(B, N, Hq, Hk, d)) return FA_ERR_INVALID_ARG;
  fa_status_t st = check_rope(wq, wk, rope, rope_rows, rot, interleaved, d, eps);
  if (st != FA_OK) return st;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return FA_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if ((long long)B * N == 0 || Hq + Hk == 0) {  // the weights' gradients over no rows
    if ((dwq || dwk) && (st = (fa_status_t)device_check()) != FA_OK) return st;
    if (dwq && cudaMemsetAsync(dwq, 0, d * sizeof(float), s) != cudaSuccess) return FA_ERR_CUDA;
    if (dwk && cudaMemsetAsync(dwk, 0, d * sizeof(float), s) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }
  if (!rows_ok(gq, Hq > 0) || !rows_ok(q, Hq > 0) || !rows_ok(dq, Hq > 0) || !rows_ok(gk, Hk > 0) ||
      !rows_ok(k, Hk > 0) || !rows_ok(dk, Hk > 0))
    return FA_ERR_INVALID_ARG;
  if (Hq > 0 && !(stride_ok(q_sb, B, 8) && stride_ok(q_sn, N, 8) && stride_ok(q_sh, Hq, 8) && stride_ok(dq_sb, B, 8) &&
                  stride_ok(dq_sn, N, 8) && stride_ok(dq_sh, Hq, 8)))
    return FA_ERR_INVALID_ARG;
  if (Hk > 0 && !(stride_ok(k_sb, B, 8) && stride_ok(k_sn, N, 8) && stride_ok(k_sh, Hk, 8) && stride_ok(dk_sb, B, 8) &&
                  stride_ok(dk_sn, N, 8) && stride_ok(dk_sh, Hk, 8)))
    return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || (rot > 0 && !positions && rope_rows < N)) return FA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < bwd_bytes(d)) return FA_ERR_INVALID_ARG;
  if ((st = (fa_status_t)device_check()) != FA_OK) return st;
  NormRopeBwdArgs a = {};
  if (!(a.status = device_status_word())) return FA_ERR_CUDA;
  a.gq = bf(gq), a.gk = bf(gk), a.q = bf(q), a.k = bf(k), a.wq = bf(wq), a.wk = bf(wk);
  a.rope = rope, a.rope_rows = rope_rows, a.rot = rot;
  a.positions = positions, a.pos_sb = pos_sb;
  a.dq = bf(dq), a.dk = bf(dk), a.partial = static_cast<float*>(workspace);
  a.q_sb = q_sb, a.q_sn = q_sn, a.q_sh = q_sh, a.k_sb = k_sb, a.k_sn = k_sn, a.k_sh = k_sh;
  a.dq_sb = dq_sb, a.dq_sn = dq_sn, a.dq_sh = dq_sh, a.dk_sb = dk_sb, a.dk_sn = dk_sn, a.dk_sh = dk_sh;
  a.B = B, a.N = N, a.Hq = Hq, a.Hk = Hk, a.eps = eps;
  const NormRopeBwdPlan plan = norm_rope_bwd_plan((long long)B * N, Hq, Hk, d);
  return launch_norm_rope_bwd(d, interleaved != 0, a, plan, dwq, dwk, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_paged_plan(const int* cached, const int* new_tokens, int* block_table, long long table_stride,
                          int table_cols, int* free_pages, int pool_pages, const int* free_count, int page_size, int R,
                          int max_tokens, int* lens, int* cu_tokens, long long* slots, int* positions, int* token_req,
                          int* free_count_out, int* plan_status, void* stream) {
  if (R < 0 || max_tokens < 0 || table_cols < 0 || pool_pages < 0 || page_size < 1) return FA_ERR_INVALID_ARG;
  if (R > FA_PLAN_MAX_REQUESTS) return FA_ERR_UNSUPPORTED;
  if ((long long)table_cols * page_size > FA_PAGED_MAX_LEN || max_tokens > FA_PAGED_MAX_LEN ||
      pool_pages > FA_PAGED_MAX_LEN)
    return FA_ERR_INVALID_ARG;
  if (!free_count || !cu_tokens || !free_count_out || !plan_status) return FA_ERR_INVALID_ARG;
  if (R > 0 && (!cached || !new_tokens || !lens || (table_cols > 0 && !block_table))) return FA_ERR_INVALID_ARG;
  if (R > 0 && table_stride < table_cols) return FA_ERR_INVALID_ARG;
  if (pool_pages > 0 && !free_pages) return FA_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!slots || !positions || !token_req)) return FA_ERR_INVALID_ARG;
  const void* ints[] = {cached, new_tokens, block_table, free_pages, free_count, lens, cu_tokens, positions, token_req,
                        free_count_out, plan_status};
  for (const void* p : ints)
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return FA_ERR_INVALID_ARG;
  if (!stride_ok(table_stride, R, 1)) return FA_ERR_INVALID_ARG;
  fa_status_t st = (fa_status_t)device_check();
  if (st != FA_OK) return st;
  PlanArgs a = {};
  a.cached = cached, a.new_tokens = new_tokens, a.free_count = free_count;
  a.table = block_table, a.table_stride = table_stride, a.table_cols = table_cols;
  a.free_pages = free_pages, a.pool_pages = pool_pages, a.page_size = page_size;
  a.R = R, a.max_tokens = max_tokens;
  a.lens = lens, a.cu_tokens = cu_tokens, a.slots = slots, a.positions = positions, a.token_req = token_req;
  a.free_count_out = free_count_out, a.plan_status = plan_status;
  return launch_paged_plan(a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status_t fa_paged_append(const void* q, const void* k, const void* v, const void* wq, const void* wk,
                            const float* rope, int rope_rows, int rot, int interleaved, const int* positions,
                            const long long* slots, void* q_out, void* k_cache, void* v_cache, int cache_fp8,
                            const float* k_descale, const float* v_descale, int num_pages, int page_size, int T,
                            int Hq, int Hk, int d, long long q_st, long long q_sh, long long k_st, long long k_sh,
                            long long v_st, long long v_sh, long long c_sp, long long c_st, long long c_sh, float eps,
                            void* stream) {
  if (!sizes_ok(1, T, Hq, Hk, d) || (cache_fp8 != 0 && cache_fp8 != 1)) return FA_ERR_INVALID_ARG;
  fa_status_t st = check_rope(wq, wk, rope, rope_rows, rot, interleaved, d, eps);
  if (st != FA_OK) return st;
  if (T == 0 || Hq + Hk == 0) return FA_OK;
  if (!rows_ok(q, Hq > 0) || !rows_ok(q_out, Hq > 0) || !rows_ok(k, Hk > 0) || !rows_ok(v, Hk > 0))
    return FA_ERR_INVALID_ARG;
  if (num_pages < 1 || page_size < 1 || (double)num_pages * page_size >= 4.6e18) return FA_ERR_INVALID_ARG;
  if (Hk > 0 && !cache_ok(k_cache, v_cache, num_pages, page_size, Hk, c_sp, c_st, c_sh, cache_fp8 ? 1 : 2))
    return FA_ERR_INVALID_ARG;
  if (Hq > 0 && !(stride_ok(q_st, T, 8) && stride_ok(q_sh, Hq, 8))) return FA_ERR_INVALID_ARG;
  if (Hk > 0 && !(stride_ok(k_st, T, 8) && stride_ok(k_sh, Hk, 8) && stride_ok(v_st, T, 8) && stride_ok(v_sh, Hk, 8)))
    return FA_ERR_INVALID_ARG;
  if (!slots || !aligned(slots, 8) || !aligned(positions, 4) || (rot > 0 && !positions)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_descale, 4) || !aligned(v_descale, 4) || (!cache_fp8 && (k_descale || v_descale)))
    return FA_ERR_INVALID_ARG;
  if ((st = (fa_status_t)device_check()) != FA_OK) return st;
  NormRopeArgs a = {};
  if (!(a.status = device_status_word())) return FA_ERR_CUDA;
  a.q = bf(q), a.k = bf(k), a.v = bf(v), a.wq = bf(wq), a.wk = bf(wk);
  a.rope = rope, a.rope_rows = rope_rows, a.rot = rot;
  a.positions = positions, a.slots = slots;
  a.q_out = bf(q_out), a.k_cache = k_cache, a.v_cache = v_cache, a.k_descale = k_descale, a.v_descale = v_descale;
  a.q_sn = q_st, a.q_sh = q_sh, a.k_sn = k_st, a.k_sh = k_sh, a.v_sn = v_st, a.v_sh = v_sh;
  a.c_sp = c_sp, a.c_st = c_st, a.c_sh = c_sh, a.num_pages = num_pages, a.page_size = page_size;
  a.B = 1, a.N = T, a.Hq = Hq, a.Hk = Hk, a.eps = eps;
  return launch_norm_rope(d, interleaved != 0, cache_fp8 ? 2 : 1, a, (cudaStream_t)stream) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

size_t fa_paged_decode_workspace_bytes(int T, int Hq, int Hk, int d) {
  if (T <= 0 || Hq <= 0 || Hk <= 0 || (d != 64 && d != 128)) return 0;
  return paged_decode_workspace(T, Hq, Hk, d);
}

fa_status_t fa_paged_decode(const void* q, const void* k_cache, const void* v_cache, int cache_fp8,
                            const float* k_descale, const float* v_descale, const int* block_table,
                            long long table_stride, int table_rows, int table_cols, const int* lens, const int* req,
                            void* o, float* lse, void* workspace, size_t workspace_bytes, int num_pages, int page_size,
                            int T, int Hq, int Hk, int d, long long q_st, long long q_sh, long long c_sp,
                            long long c_st, long long c_sh, float scale, void* stream) {
  if (T < 0 || Hq < 0 || Hk < 0 || table_rows < 0 || table_cols < 0) return FA_ERR_INVALID_ARG;
  if (cache_fp8 != 0 && cache_fp8 != 1) return FA_ERR_INVALID_ARG;
  const float scale_log2 = (float)((double)scale * 1.4426950408889634074);
  if (!(std::isfinite(scale_log2) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (T == 0 || Hq == 0) return FA_OK;
  if (Hk == 0 || Hq % Hk != 0 || Hq > (1 << 20) || (double)T * Hq * d >= 4.6e18) return FA_ERR_INVALID_ARG;
  if (!rows_ok(q, true) || !rows_ok(o, true) || !lse || !aligned(lse, 4) || !lens || !aligned(lens, 4) ||
      !aligned(req, 4))
    return FA_ERR_INVALID_ARG;
  const int size = cache_fp8 ? 1 : 2;
  if (!cache_ok(k_cache, v_cache, num_pages, page_size, Hk, c_sp, c_st, c_sh, size)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_descale, 4) || !aligned(v_descale, 4) || (!cache_fp8 && (k_descale || v_descale)))
    return FA_ERR_INVALID_ARG;
  if (!stride_ok(q_st, T, 8) || !stride_ok(q_sh, Hq, 8)) return FA_ERR_INVALID_ARG;
  if ((table_cols > 0 && table_rows > 0 && !block_table) || !aligned(block_table, 4) || table_stride < table_cols ||
      !stride_ok(table_stride, table_rows, 1) || (long long)table_cols * page_size > FA_PAGED_MAX_LEN)
    return FA_ERR_INVALID_ARG;
  if (!req && table_rows < T) return FA_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < fa_paged_decode_workspace_bytes(T, Hq, Hk, d))
    return FA_ERR_INVALID_ARG;
  fa_status_t st = (fa_status_t)device_check();
  if (st != FA_OK) return st;
  DecodeArgs a = {};
  if (!(a.status = device_status_word())) return FA_ERR_CUDA;
  a.q = bf(q), a.k = static_cast<const uint8_t*>(k_cache), a.v = static_cast<const uint8_t*>(v_cache);
  a.kd = k_descale, a.vd = v_descale;
  a.table = block_table, a.table_stride = table_stride, a.table_rows = table_rows, a.table_cols = table_cols;
  a.lens = lens, a.req = req, a.o = bf(o), a.lse = lse, a.workspace = workspace;
  a.q_st = q_st, a.q_sh = q_sh;
  a.c_sp = c_sp * size, a.c_st = c_st * size, a.c_sh = c_sh * size;
  a.num_pages = num_pages, a.page_size = page_size, a.T = T, a.Hq = Hq, a.Hk = Hk;
  a.scale_log2 = scale_log2;
  return launch_paged_decode(d, cache_fp8 != 0, a, (cudaStream_t)stream) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
