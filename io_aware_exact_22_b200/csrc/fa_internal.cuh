// fa_internal.cuh - declarations shared by the host side of libfa.so (not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace fa {

struct FwdArgs {
  uint32_t* status;  // device status word
  float* lse;        // [BH, N] fp32; with key splits: [nsplit, BH, N] partial LSEs
  int N;             // sequence length
  int BH;            // batch * heads
  int nqb;           // query blocks of 256 rows per head
  int causal;        // 0 / 1
  float scale_log2;  // scale * log2(e)
  int nsplit;        // key-range splits per (head, query block); 1 = whole key range
  int group = 1;      // work order: heads per group, heaviest query block first within a group
  int persistent = 0;  // set by the launcher: CTAs walk the work list in pairs (see fa_fwd_kernel)
  // FP8 forward only: per-(b,h) dequantisation factors [BH], or null for 1
  const float* descale_q = nullptr;
  const float* descale_k = nullptr;
  const float* descale_v = nullptr;
  // Carried partial result (bf16 kernels, whole key range): when set, the rows continue from
  // a normalised output carry_o [BH, N, d] fp32 and its natural-log LSE carry_lse [BH, N] over
  // other keys (rows with LSE = -inf have seen none)
  const float* carry_o = nullptr;
  const float* carry_lse = nullptr;
  // debug build: visit counters [BH][ceil(N/128)][ceil(N/128)] (null in the release build)
  int* visits = nullptr;
  long long visits_cap = 0;
};

struct BwdArgs {
  uint32_t* status;  // device status word
  const float* lse;  // [BH, N] fp32, natural log
  const float* ld;   // [BH, ceil(N/64), 128] fp32: per 64-row query tile, 64 x LSE*log2(e)
                     // then 64 x D_i = rowsum(dO o O); rows past N hold +inf and 0
  float* dq_acc;     // [BH, N, d] fp32 accumulator (zeroed by the pre-kernel)
  int N;
  int BH;
  int causal;
  float scale;       // softmax scale
  float scale_log2;  // scale * log2(e)
  // When set (d = 128, with the dQ path): scale * dK and dV of this call are added into these
  // fp32 [BH, N, d] accumulators instead of being stored as bf16 (the sequence-sharded backward)
  float* dk_acc = nullptr;
  float* dv_acc = nullptr;
  int acc_overwrite = 0;  // with dk_acc: store into the accumulators instead of adding
  int group = 1;  // work order: heads per group, heaviest key tile first within a group
  // two ints in device memory, zero before each launch of the key-tile kernel (the pre-kernel
  // zeroes them; the kernel's last CTA zeroes them again on exit): the next unclaimed item
  // and the number of CTAs done
  int* work = nullptr;
  // debug build: visit counters of the kernel launched with these arguments (null in release)
  int* visits = nullptr;
  long long visits_cap = 0;
};

// Debug build: device address of the visit-counter block of one kernel kind (0 forward,
// 1 backward key-tile kernel, 2 deterministic dQ kernel), kDebugVisitInts counters each;
// nullptr in the release build.
constexpr long long kDebugVisitInts = 1LL << 20;
int* debug_visits(int kind);

// Backward dQ accumulation: of each 64-row query tile, the first kBwdDqRedRows rows are added
// into the fp32 accumulator with per-thread reductions, the rest with one TMA reduce-add
// (tensor-map box of 64 - kBwdDqRedRows rows).  Measured at B=2 H=16 N=4096, B=1 H=32
// N=16384 (causal) and B=4 H=16 N=4096 (non-causal): 0 (every row by TMA) is 0.5-1.8 %
// faster than 32, and 48 is 2.5-3 % slower.
constexpr int kBwdDqRedRows = 0;

// Device address of this library's status word on the current device (nullptr on error).
uint32_t* device_status_word();

// Launches the bounded-wait self-test kernel (see fa_selftest_wait_timeout).
cudaError_t launch_wait_probe(uint32_t* status, uint64_t limit_ns, cudaStream_t stream);

// Tensor maps for a bf16 [BH, N, d] tensor, 128-byte swizzle, box = 64 columns x `rows`
// (make_*: served from a cache of encoded maps; encode_*: always encodes).
// 3-D map over an E4M3 tensor [BH, N, d] (one byte per element), box {128, box_rows},
// 128-byte swizzle.
bool make_tmap_e4m3(CUtensorMap* m, const void* ptr, int BH, int N, int d, int box_rows);
bool make_tmap_bf16(CUtensorMap* m, const void* ptr, int BH, int N, int d, int box_rows);
bool encode_tmap_bf16(CUtensorMap* m, const void* ptr, int BH, int N, int d, int box_rows);
bool encode_tmap_f32(CUtensorMap* m, const void* ptr, int BH, int N, int d, int box_inner, int box_rows,
                     bool swizzle128);

// With a.nsplit == 1, `to` maps the bf16 output; with a.nsplit > 1 it maps the fp32 partial
// outputs [nsplit * BH, N, d] (box 32 x 32, 128-byte swizzle) and a.lse the partial LSEs.
cudaError_t launch_fwd(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& to, const FwdArgs& a, cudaStream_t stream);
// Partial outputs (fp32 O / l and LSE) for a.nsplit >= 1 key ranges, whatever a.nsplit is; `to`
// maps the fp32 partials [a.nsplit * BH, N, d].
cudaError_t launch_fwd_partial(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const CUtensorMap& to, const FwdArgs& a, cudaStream_t stream);
// FP8 (E4M3) inputs, d = 128, whole key range; Q/K/V maps from make_tmap_e4m3 (128-row boxes)
cudaError_t launch_fwd_fp8(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const CUtensorMap& to, const FwdArgs& a, cudaStream_t stream);
// Combines nsplit partial (O_s, LSE_s) into bf16 O and fp32 LSE.
cudaError_t launch_fwd_merge(const float* o_part, const float* lse_part, void* o, float* lse, int nsplit,
                             long long rows, int d, cudaStream_t stream);

cudaError_t launch_bwd_pre(const void* o, const void* dO, const float* lse, float* ld, float* dq_acc, int* work,
                           int BH, int N, int d, cudaStream_t stream);
// fp32 [BH, N, d] tensor map without swizzle, box = box_inner columns x box_rows rows.
bool make_tmap_f32(CUtensorMap* m, const void* ptr, int BH, int N, int d, int box_inner, int box_rows,
                   bool swizzle128 = false);

// with_dq = false: dK and dV only (no dQ accumulation; tdq and a.dq_acc unused).
cudaError_t launch_bwd_main(int d, const CUtensorMap& tq, const CUtensorMap& tk,
                            const CUtensorMap& tv, const CUtensorMap& tdo,
                            const CUtensorMap& tdk, const CUtensorMap& tdv,
                            const CUtensorMap& tdq, const BwdArgs& a, cudaStream_t stream,
                            bool with_dq = true);
// Deterministic dQ (query-tile-outer, accumulated in TMEM, written once): tq/tdo with 128-row
// boxes, tk/tv with 64-row boxes, tdq the bf16 dQ with 32-row boxes; needs a.ld filled.
cudaError_t launch_bwd_dq(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          const CUtensorMap& tdo, const CUtensorMap& tdq, const BwdArgs& a,
                          cudaStream_t stream);
// acc += x over elems fp32 values (a multiple of 4, 16-byte aligned).
cudaError_t launch_acc_add(float* acc, const float* x, long long elems, cudaStream_t stream);
cudaError_t launch_bwd_post(const float* dq_acc, void* dq, long long elems, float scale,
                            cudaStream_t stream);

// The current device is an sm_100 part (cached per device): FA_OK, FA_ERR_UNSUPPORTED or
// FA_ERR_CUDA as an int.
int device_check();

// ------------------------------------------------------------------ norm + rotation (fa_norm_rope.cu)
// Strides are in elements; rows are d contiguous elements, 16-byte aligned.
struct NormRopeArgs {
  uint32_t* status;
  const __nv_bfloat16 *q, *k, *v;    // v: serving form only
  const __nv_bfloat16 *wq, *wk;      // [d], or null for 1
  const float* rope;                 // [rope_rows, 2, rot/2]: cosines, then sines
  const int* positions;              // [B, N] (stride pos_sb), or null for n
  const long long* slots;            // serving form: [N]
  __nv_bfloat16 *q_out, *k_out;      // training form: [B,H,N,d]; serving form: q_out [N,Hq,d]
  void *k_cache, *v_cache;           // serving form
  const float *k_descale, *v_descale;  // E4M3 cache: [Hk], or null for 1
  long long q_sb, q_sn, q_sh, k_sb, k_sn, k_sh, v_sn, v_sh, pos_sb;
  long long c_sp, c_st, c_sh;        // cache strides: page, token, head
  int num_pages, page_size;
  int B, N, Hq, Hk, rot, rope_rows;
  float eps;
  int heads_per_unit, chunks;        // set by the launcher
};
struct NormRopeBwdArgs {
  uint32_t* status;
  const __nv_bfloat16 *gq, *gk;      // [B,H,N,d]
  const __nv_bfloat16 *q, *k, *wq, *wk;
  const float* rope;
  const int* positions;
  __nv_bfloat16 *dq, *dk;
  float* partial;                    // [blocks, d]
  long long q_sb, q_sn, q_sh, k_sb, k_sn, k_sh, dq_sb, dq_sn, dq_sh, dk_sb, dk_sn, dk_sh, pos_sb;
  int B, N, Hq, Hk, rot, rope_rows;
  float eps;
  int per_q, per_k, blocks_q;        // set by the launcher: heads per unit, blocks that take q
};
// mode: 0 training form, 1 bf16 cache, 2 E4M3 cache
cudaError_t launch_norm_rope(int d, bool interleaved, int mode, NormRopeArgs a, cudaStream_t stream);
// How the backward kernel goes over a problem: heads per unit, and blocks that take q and k, i.e. rows
// of the partial weight gradients (kNormRopeBwdBlocks at most).
constexpr int kNormRopeBwdBlocks = 148 * 4;
struct NormRopeBwdPlan {
  int per_q, per_k, q, k;
};
NormRopeBwdPlan norm_rope_bwd_plan(long long tokens, int Hq, int Hk, int d);
cudaError_t launch_norm_rope_bwd(int d, bool interleaved, NormRopeBwdArgs a, const NormRopeBwdPlan& plan, float* dwq,
                                 float* dwk, cudaStream_t stream);

// ------------------------------------------------------------------ paged cache (fa_paged.cu)
struct PlanArgs {
  const int *cached, *new_tokens, *free_count;
  int *table, *free_pages, *lens, *cu_tokens, *positions, *token_req, *free_count_out, *plan_status;
  long long* slots;
  long long table_stride;
  int table_cols, pool_pages, page_size, R, max_tokens;
  uint64_t page_mul;                 // set by the launcher: division by page_size
  int page_shift, wide;              // wide: the outputs per token are 16-byte aligned
};
cudaError_t launch_paged_plan(PlanArgs a, cudaStream_t stream);

struct DecodeArgs {
  uint32_t* status;
  const __nv_bfloat16* q;
  const uint8_t *k, *v;              // caches
  const float *kd, *vd;              // E4M3: [Hk], or null for 1
  const int *table, *lens, *req;     // req null: row t reads table row t
  __nv_bfloat16* o;                  // [T,Hq,d]
  float* lse;                        // [T,Hq]
  void* workspace;
  long long q_st, q_sh;              // elements
  long long c_sp, c_st, c_sh;        // bytes
  long long table_stride;
  int table_rows, table_cols, num_pages, page_size, T, Hq, Hk;
  float scale_log2;
  uint64_t page_mul;                 // set by the launcher: division by page_size
  int page_shift, hp;                // hp: kv heads that a CTA reads side by side (1, 2, 4)
};
size_t paged_decode_workspace(int T, int Hq, int Hk, int d);
cudaError_t launch_paged_decode(int d, bool fp8, DecodeArgs a, cudaStream_t stream);

}  // namespace fa
