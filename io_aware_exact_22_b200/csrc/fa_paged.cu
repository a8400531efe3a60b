// fa_paged.cu - the paged key/value cache: the plan of a serving step (pages, slots) and the
// attention of one query token per row over the cache.
#include "fa.h"
#include "fa_internal.cuh"
#include "sm100_ptx.cuh"

#include <algorithm>
#include <climits>

namespace fa {

namespace {

using namespace ptx;

// ====================================================================== plan
// Requests hold cached[b] tokens in ceil(cached[b] / page_size) pages; the step adds
// new_tokens[b] tokens, or releases the request (-1).  Released pages go on top of the free stack
// in the order (request, page), wanted pages come off its top in the same order, so the result
// depends on the inputs alone.  Bound by latency: 3.4 us for 16 decoding requests, 10.0 us for 1000
// mixed ones with 50 k tokens.  Everything is one kernel: every block of one cluster scans the
// requests for itself (a few bytes each, from L2), the cluster's barrier separates reading the
// inputs from writing, which is what lets the outputs alias them, and then the tokens are spread
// over all threads.  Nothing is written but `plan_status`, the unchanged lengths and the -1
// padding when the step cannot be planned.
constexpr int kPlanThreads = 1024;
// Blocks of the cluster: 16 where the device can place such a cluster (beyond the portable 8), which
// took a quarter off the mixed step's time (measured on an earlier form).
constexpr int kPlanMaxCtas = 16;
constexpr int kPlanRequests = 256;  // at most, per block: with released pages 1000 requests take 8.3 us on 4, 10.3 on 1
// Neighbouring tokens (or pages) per thread: one search, one store per output.  Chosen on clusters of 8
// blocks: 1000 requests with 50 k tokens took 12.0 us with 2, 14.2 with 1, 12.4 with 4 and 16.9 with 8
// (the longer chain of each thread shows); 100 requests of one token 3.3, 3.0, 3.8 and 5.0.
constexpr int kPlanPer = 2;
constexpr int kPlanEach = 8;       // released pages per lane and turn, when there are many
constexpr int kPlanPages = 16384;  // pages that may be released, per block

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Sum3 {
  long long want, grow, back;
};
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return {a.want + b.want, a.grow + b.grow, a.back + b.back};
}
__device__ __forceinline__ Sum3 shfl_up3(const Sum3& a, int o) {
  return {__shfl_up_sync(0xffffffffu, a.want, o), __shfl_up_sync(0xffffffffu, a.grow, o),
          __shfl_up_sync(0xffffffffu, a.back, o)};
}

// n / page_size for 0 <= n < 2^31 (see page_division).
__device__ __forceinline__ int div_page(int n, uint64_t mul, int shift) {
  return (int)(((uint64_t)(uint32_t)n * mul) >> shift);
}

// The last of R entries of the ascending array `first` that is not above i.
__device__ __forceinline__ int holder(const int* first, int R, int i) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) fa_paged_plan_kernel(const PlanArgs a) {
  // per request: cached length (complemented when released), and prefix sums over the requests of
  // wanted pages, released pages and new tokens
  extern __shared__ int sm[];
  int* s_cached = sm;
  int* s_want = sm + a.R;
  int* s_back = sm + 2 * a.R;    // R + 1
  int* s_cu = sm + 3 * a.R + 1;  // R + 1
  __shared__ Sum3 warp_sum[32];
  __shared__ Sum3 carry;
  __shared__ int s_bits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
  const int ps = a.page_size;
  const long long room = (long long)a.table_cols * ps;
  auto pages_of = [&](int n) { return n == 0 ? 0 : div_page(n - 1, a.page_mul, a.page_shift) + 1; };

  const int free0 = *a.free_count;
  int bits = 0;
  if (tid == 0) carry = {0, 0, 0}, s_bits = 0;
  __syncthreads();
  for (int base = 0; base < a.R; base += nt) {
    const int b = base + tid;
    Sum3 v = {0, 0, 0};
    int cached = 0, add = 0;
    if (b < a.R) {
      cached = a.cached[b];
      add = a.new_tokens[b];
      if (cached < 0 || cached > room || add < -1) {
        bits |= FA_PLAN_BAD_INPUT;
        cached = 0, add = 0;
      }
      const int used = pages_of(cached);
      if (add < 0) {
        v.back = used;
      } else if ((long long)cached + add > room) {
        bits |= FA_PLAN_ROW_FULL;
      } else {
        v.grow = add;
        v.want = pages_of(cached + add) - used;
      }
    }
    Sum3 x = v;  // inclusive scan over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sum3 y = shfl_up3(x, o);
      if (lane >= o) x = x + y;
    }
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    if (warp == 0) {
      Sum3 w = lane < nw ? warp_sum[lane] : Sum3{0, 0, 0};
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Sum3 y = shfl_up3(w, o);
        if (lane >= o) w = w + y;
      }
      if (lane < nw) warp_sum[lane] = w;
    }
    __syncthreads();
    Sum3 ex = carry;  // exclusive prefix of this request
    if (warp > 0) ex = ex + warp_sum[warp - 1];
    ex = ex + Sum3{x.want - v.want, x.grow - v.grow, x.back - v.back};
    if (b < a.R) {  // the low words are exact whenever the plan is accepted
      s_cached[b] = add < 0 ? ~cached : cached;
      s_want[b] = (int)ex.want;
      s_back[b] = (int)ex.back;
      s_cu[b] = (int)ex.grow;
    }
    __syncthreads();
    if (tid == 0) carry = carry + warp_sum[nw - 1];
    if (base + nt >= a.R && bits) atomicOr(&s_bits, bits);
    __syncthreads();
  }
  const Sum3 total = carry;
  bits = s_bits;
  const long long avail = free0 + total.back;
  if (free0 < 0 || avail > a.pool_pages) bits |= FA_PLAN_BAD_INPUT;
  else if (total.want > avail) bits |= FA_PLAN_NO_PAGES;
  if (total.grow > a.max_tokens) bits |= FA_PLAN_TOO_MANY_TOKENS;
  const bool ok = bits == 0;
  const int tokens = ok ? (int)total.grow : 0;
  const int back = ok ? (int)total.back : 0;
  if (tid == 0) s_cu[a.R] = tokens, s_back[a.R] = back;
  __syncthreads();
  const int gt = rank * nt + tid, gn = ctas * nt;
  // released pages onto the stack.  Few: neighbouring ones per thread, a search for each thread.
  // Many: a warp takes runs of 32 * kPlanEach, a lane every 32nd of a run, with one search for the
  // run and steps over the requests in between.  (1000 requests, 10 k pages on 4 blocks: 8.0 us in all
  // and 9.1; 622 requests, 590 k pages on 16: 17 us the second way.)
  if (back <= 4LL * kPlanPer * gn) {
    for (int p0 = gt * kPlanPer; p0 < back; p0 += gn * kPlanPer) {
      int b = holder(s_back, a.R, p0), page[kPlanPer];
#pragma unroll
      for (int i = 0; i < kPlanPer; ++i)
        if (p0 + i < back) {
          while (s_back[b + 1] <= p0 + i) ++b;
          page[i] = a.table[(long long)b * a.table_stride + (p0 + i - s_back[b])];
        }
#pragma unroll
      for (int i = 0; i < kPlanPer; ++i)
        if (p0 + i < back) a.free_pages[free0 + p0 + i] = page[i];
    }
  } else {
    const long long span = 32 * kPlanEach;
    for (long long p0 = (rank * nw + warp) * span; p0 < back; p0 += ctas * nw * span) {
      const int first = (int)p0 + lane, n = back - first;  // the lane's pages: 0, 32, ... below n
      int b = holder(s_back, a.R, (int)p0), page[kPlanEach];
#pragma unroll
      for (int i = 0; i < kPlanEach; ++i)
        if (32 * i < n) {
          while (s_back[b + 1] <= first + 32 * i) ++b;
          page[i] = a.table[(long long)b * a.table_stride + (first + 32 * i - s_back[b])];
        }
#pragma unroll
      for (int i = 0; i < kPlanEach; ++i)
        if (32 * i < n) a.free_pages[free0 + first + 32 * i] = page[i];
    }
  }
  // Every block has read the inputs (nothing that may be one of them is written before), and the
  // released pages are on the stack.
  if (ctas > 1) cluster_sync();
  else __syncthreads();
  if (gt == 0) {
    *a.free_count_out = ok ? (int)(avail - total.want) : free0;
    *a.plan_status = bits;
    a.cu_tokens[a.R] = tokens;
  }
  for (int b = gt; b < a.R; b += gn) {
    const int c = s_cached[b];
    a.lens[b] = !ok ? a.cached[b] : c < 0 ? 0 : c + s_cu[b + 1] - s_cu[b];
    a.cu_tokens[b] = ok ? s_cu[b] : 0;
  }
  const int top = (int)(avail - 1);
  for (int t0 = gt * kPlanPer; t0 < a.max_tokens; t0 += gn * kPlanPer) {
    int lo = t0 < tokens ? holder(s_cu, a.R, t0) : 0;
    int pos[kPlanPer], req[kPlanPer], page[kPlanPer], in[kPlanPer];
    int* enter[kPlanPer];
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int t = t0 + i;
      pos[i] = 0, req[i] = -1, page[i] = -1, in[i] = 0, enter[i] = nullptr;
      if (t < tokens) {
        while (s_cu[lo + 1] <= t) ++lo;
        req[i] = lo;
        const int c = s_cached[lo], used = pages_of(c);
        pos[i] = c + t - s_cu[lo];
        const int p = div_page(pos[i], a.page_mul, a.page_shift);
        in[i] = pos[i] - p * ps;
        int* entry = a.table + (long long)lo * a.table_stride + p;
        if (p >= used && in[i] == 0) enter[i] = entry;  // the first token of a page of this step
        page[i] = p < used ? *entry : a.free_pages[top - (s_want[lo] + p - used)];
      }
    }
    long long slot[kPlanPer];
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      slot[i] = t0 + i < tokens ? (long long)page[i] * ps + in[i] : -1;
      if (enter[i]) *enter[i] = page[i];
    }
    if (a.wide && t0 + kPlanPer <= a.max_tokens) {
      *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<int2*>(a.positions + t0) = make_int2(pos[0], pos[1]);
      *reinterpret_cast<int2*>(a.token_req + t0) = make_int2(req[0], req[1]);
    } else {
      for (int i = 0; i < kPlanPer && t0 + i < a.max_tokens; ++i)
        a.slots[t0 + i] = slot[i], a.positions[t0 + i] = pos[i], a.token_req[t0 + i] = req[i];
    }
  }
}

// ====================================================================== decode
// Row t, query head h over kv head h' = h / g, keys j < len:
//     s_j = scale q.K_j,  m = max s,  l = sum 2^(s-m),  O = (sum 2^(s-m) V_j) / l,  LSE = m + ln l
// (base 2 with log2 e folded into the scale), one pass over the keys.
//
// The work is a line of key tiles, row after row, kv head after kv head, cut into equal runs, one
// run per CTA, whatever the lengths are: the lengths live on the device, so the cut is computed
// there, by every CTA for itself.  A (row, kv head) that a cut divides leaves fp32 partial results
// (sum, max, unnormalised O) in the workspace, at most two per CTA, which a second kernel joins;
// the others are written by the CTA that computed them.
//
// Inside a CTA each warp owns one of `hp` neighbouring kv heads and every (kWarps / hp)-th run of
// KEYS keys, with its own ring of shared-memory stages, filled by 16-byte asynchronous copies
// straight from the pages, and keeps its own reference max, sum and O: no barrier until the heads
// end, when the warps of a head are joined in shared memory.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T (m16n8k16, fp32 accumulators):
// keys and value columns fill the 16-row side, the g query heads of a kv head the 8-wide side, so
// up to 8 heads cost no empty rows, K and V (and their conversion from E4M3) are read from shared
// memory once for 16 heads, and O takes D / 4 registers for 8 heads.  K and V come once from memory
// and feed 4 g flops per element, an order of magnitude below what the tensor pipe needs to be the
// bound at the copy bandwidth.  P goes in as the sum of 16-bit terms, each with a product of its own: three
// bf16 terms (to 2^-23), or, with an E4M3 cache, whose values are exact in fp16, two fp16 terms (22 bits).
// With one term fewer, and O as the matrix unit's own long sum (see there), the rounded outputs
// differed from fp32 arithmetic's by 1e-4 (bf16) and 9e-4 (E4M3) in relative norm; they now differ by less
// than 8e-5.  That costs nothing where memory is the bound and the clock holds, 2 % of the bf16 cases'
// times, and 6 % of the long E4M3 case's when it runs for seconds (121 for 113 us): the card is then at its
// power cap, and the clock gives way to the second product.
//
// Bound by HBM once contexts are long; about 8 us go to the launches, to the chain of lengths, pages
// and keys, and to the join.  On a B200, replayed from a graph: 2 x 131071 keys, 32 query and 4 kv heads,
// d=128, bf16 95 us (5.6 TB/s), 32 rows of 0 to 4096 keys, 32 and 8 heads 52 us (5.2 TB/s), 64 rows of
// 1024 to 8192 keys, 64 and 8 heads, E4M3 107.5 us (5.6 TB/s), one row of 300 keys 8.6 us.  More than 8
// query heads per kv head take a second column of products (32 rows of 4096 keys, 32 and 2 heads, d=128,
// bf16 40 us, 3.4 TB/s: the products and P's terms then count), more than 16 a second reading of K and V
// (4 x 32768 keys, 32 heads and 1 36.6 us, twice 1.8 TB/s, from L2 in part).
constexpr int kWarps = 4;
constexpr int kMaxCtasPerSm = 3;
constexpr int kMaxRows = 16;

template <int D, bool FP8, int NQ>
struct DecCfg {
  static constexpr int ROWB = D * (FP8 ? 1 : 2);          // bytes of a key's row
  static constexpr int CH = ROWB / 16;                    // 16-byte chunks of a row
  static constexpr int KEYS = ROWB == 256 ? 16 : 32;      // keys per warp and tile
  static constexpr int STAGE = 2 * KEYS * ROWB;           // K then V
  static constexpr int RPI = 32 / CH;                     // rows that one copy instruction covers
  // 2 CTAs of 3 stages per SM where a warp's registers want them (d = 128 with E4M3, whose conversions are the
  // longer chain, or with 16 query heads, which spill at 3 CTAs), else 3, of 2 stages for bf16.  2 of 3
  // against 3 of 2: bf16, d = 128, 16 heads per kv head, 32 x 4096 keys 41.8 and 45 us, 4 x 32768 36.7 and
  // 39.3; up to 8 heads, 128 x 1024 keys 98.0 and 95.7, 32 x 0-4096 52.7 and 52.1 (but 2 x 131071 92.2
  // and 94.5); E4M3, 64 x 1024-8192 keys 107.3 and 108.3, 16 heads 28 and 35.
  static constexpr bool WIDE = D == 128 && (FP8 || NQ == 2);
  static constexpr int STAGES = FP8 || WIDE ? 3 : 2;
  static constexpr int CTAS = WIDE ? 2 : kMaxCtasPerSm;
  static constexpr int RS = D + 4;                        // floats of a row of O at the join: off one bank
  static constexpr int SMEM = kWarps * STAGES * STAGE;
  static_assert(8 * RS * 4 <= STAGE, "a stage holds 8 rows of a warp's O at the join");
};

// Chunk c of row r sits at chunk c ^ swz(r): the 8 rows that one ldmatrix reads at equal c then
// cover all banks.
template <int CH>
__device__ __forceinline__ int swz(int r) {
  return CH >= 8 ? (r & 7) : ((r >> 1) & 3);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with sums that begin at zero.
template <bool F16>
__device__ __forceinline__ void mma16816_new(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// Two E4M3 codes (the low or the high 16 bits) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
// The 8x8 matrix of 16-bit values held as (row lane / 4, columns 2 (lane % 4), + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(u));
  return f;
}
// The largest value of 8 bits below x > 0 (0 for 0).  A split of P by it leaves no term zero or
// negative, so that an infinite V stays infinite through all their products.
__device__ __forceinline__ float below(float x) {
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float((u - min(u, 1u)) & 0xffff0000u);
}
// Two values of 8 bits as bf16.
__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}

// Number of keys of query row t; 0 writes an empty row's result, -1 leaves the row as it was.
// `r` is its row of the block table.
__device__ __forceinline__ int row_keys(const DecodeArgs& a, int t, int& r) {
  const int len = a.lens[t];
  r = a.req ? a.req[t] : t;
  if (r < 0) return -1;
  if (r >= a.table_rows) {
    atomicOr(a.status, FA_DEV_BOUNDS);
    return -1;
  }
  if (len < 0 || len > (long long)a.table_cols * a.page_size) {
    atomicOr(a.status, FA_DEV_BOUNDS);
    return 0;
  }
  return len;
}

// A place in the line of tiles: row t (of len keys, row r of the block table), group hm = (run of
// hp kv heads) * runs + (run of kMaxRows of their query heads), tile.
struct Cursor {
  int t, hm, tile, tiles, len, r;
};

__device__ __forceinline__ int tiles_of(int len, int shift) { return (max(len, 0) + (1 << shift) - 1) >> shift; }

__device__ __forceinline__ void cursor_next(const DecodeArgs& a, Cursor& c, int groups, int shift) {
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.hm < groups) return;
  c.hm = 0;
  do {
    ++c.t;
    if (c.t >= a.T) {  // past the end: nothing follows
      c.tiles = 0, c.len = 0;
      return;
    }
    c.len = row_keys(a, c.t, c.r);
    c.tiles = tiles_of(c.len, shift);
  } while (c.tiles == 0);
}

// Workspace: a header per divided group (row, group, first and last CTA; row -1: not divided),
// indexed by the CTA in which the group begins, or, when there are no more groups than CTAs, by
// the group; then per CTA two partial results, of a group that began before it and of one that
// runs past it: hp heads of kMaxRows (max, sum) pairs and rows of fp32 O.
constexpr int kMaxHeads = 4;
struct Part {
  int4* head;
  float2* ml;
  float* o;
};
__host__ __device__ __forceinline__ size_t part_head_bytes(int ctas) { return ((size_t)ctas * 16 + 255) & ~(size_t)255; }
__host__ __device__ __forceinline__ size_t part_ml_bytes(int ctas) { return (size_t)ctas * 2 * kMaxHeads * kMaxRows * 8; }
__device__ __forceinline__ Part part_of(void* ws, int ctas) {
  char* p = reinterpret_cast<char*>(ws);
  Part r;
  r.head = reinterpret_cast<int4*>(p);
  r.ml = reinterpret_cast<float2*>(p + part_head_bytes(ctas));
  r.o = reinterpret_cast<float*>(p + part_head_bytes(ctas) + part_ml_bytes(ctas));
  return r;
}

__device__ __forceinline__ void write_lse(const DecodeArgs& a, long long t, int h, float m, float l, float bias) {
  a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l) - bias) * 0.6931471805599453f;
}

// Finishes one output row's 4 elements: o = sum / l, and the row's LSE (once per row).
template <int D>
__device__ __forceinline__ void write_out(const DecodeArgs& a, long long t, int h, int c4, float4 x, float m, float l,
                                          float vscale, float bias) {
  const float inv = l > 0.f || l != l ? vscale / l : 0.f;
  uint2 u;
  u.x = pack_bf16(x.x * inv, x.y * inv);
  u.y = pack_bf16(x.z * inv, x.w * inv);
  *reinterpret_cast<uint2*>(a.o + (t * a.Hq + h) * D + c4 * 4) = u;
  if (c4 == 0) write_lse(a, t, h, m, l, bias);
}

// The reference max of a query row moves only when a score exceeds it by more than 2^kSlack, so P
// stays below 2^kSlack, and most tiles need no reduction over lanes and no rescaling of O.  P of
// the E4M3 form carries the power of two kPBias: at most 2^15 in fp16, and its low term held to 11 bits
// down to 2^-10 of the row's largest, below that to 2^-32 of it.
constexpr float kSlack = 8.f;
constexpr float kPBias = 7.f;

template <int D, bool FP8, int NQ>
__global__ void __launch_bounds__(kWarps * 32, DecCfg<D, FP8, NQ>::CTAS) fa_paged_decode_kernel(const DecodeArgs a) {
  using C = DecCfg<D, FP8, NQ>;
  constexpr int KEYS = C::KEYS, MT = KEYS / 16, CH = C::CH, ROWB = C::ROWB;
  constexpr int kStages = C::STAGES;
  constexpr int DC = D / 16;  // 16-wide steps of the score product, and 16-row tiles of O^T
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps];
  __shared__ Cursor s_start;
  __shared__ float s_m[kWarps][kMaxRows], s_l[kWarps][kMaxRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, cta = blockIdx.x;
  const int g = a.Hq / a.Hk, runs = NQ == 1 ? 1 : (g + kMaxRows - 1) / kMaxRows, groups = (a.Hk / a.hp) * runs;
  const int hw = warp % a.hp, kw = warp / a.hp, kws = kWarps / a.hp;  // the warp's head and run of keys
  const int shift = 31 - __clz(KEYS * kws);                          // keys per tile, a power of two
  const bool by_group = (long long)a.T * groups <= G;
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- the cut: tiles of a run of rows per thread, scanned over the block
  const int per_thread = (a.T + kWarps * 32 - 1) / (kWarps * 32);
  const int t0 = min(a.T, tid * per_thread), t1 = min(a.T, t0 + per_thread);
  long long mine = 0;
  int len = 0, r = 0;  // of the thread's last row: its only one, as a rule
  for (int t = t0; t < t1; ++t) {
    len = row_keys(a, t, r);
    mine += tiles_of(len, shift);
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_scan[warp] = x;
  __syncthreads();
  long long before = x - mine;
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  total *= groups;
  const long long ctas = min((long long)G, total);
  Part part = part_of(a.workspace, G);

  auto write_empty = [&]() {  // rows without a visible key
    for (int t = cta; t < a.T; t += G) {
      int r;
      const int n = row_keys(a, t, r);
      if (n > 0) continue;
      if (n == 0)
        for (int i = tid; i < a.Hq * (D / 4); i += kWarps * 32)
          write_out<D>(a, t, i / (D / 4), i % (D / 4), make_float4(0, 0, 0, 0), 0.f, 0.f, 0.f, 0.f);
      if (by_group)
        for (int i = tid; i < groups; i += kWarps * 32) part.head[t * groups + i] = make_int4(-1, 0, 0, 0);
    }
  };
  if (cta >= ctas) {
    write_empty();
    if (!by_group && tid == 0) part.head[cta] = make_int4(-1, 0, 0, 0);
    return;
  }
  // CTA c's run begins at tile c * per + min(c, extra) and has per tiles, one more below extra
  const long long per = quotient(total, ctas), extra = total - per * ctas, first = cta * per + min((long long)cta, extra);
  if (before * groups <= first && first < (before + mine) * groups) {
    long long at = before * groups;
    for (int t = t0; t < t1; ++t) {
      if (t1 - t0 > 1) len = row_keys(a, t, r);
      const long long n = tiles_of(len, shift);
      if (first < at + n * groups) {
        const long long hm = quotient(first - at, n);
        s_start = {t, (int)hm, (int)(first - at - hm * n), (int)n, len, r};
        break;
      }
      at += n * groups;
    }
  }
  __syncthreads();
  Cursor ahead = s_start;  // the next tile to fetch
  int fetch_left = (int)(per + (cta < extra));
  int left = fetch_left;

  // ---- fetching.  One copy instruction covers RPI keys.  A page size that is a multiple of RPI
  // keeps them on one page, which lane i looks up for copy i; else lane i looks up key i's.
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::STAGE;
  const bool joint = a.page_size % C::RPI == 0;
  const int crow = lane / CH, cc = lane % CH;  // the lane's key within a copy instruction, and chunk
  const int my_key = kw * KEYS + (joint ? lane * C::RPI % KEYS : lane % KEYS);
  const long long lane_off = (joint ? crow * a.c_st : 0) + cc * 16;
  const long long vk = a.v - a.k;
  long long off = -1;  // byte offset of the looked-up key, -1: none
  auto lookup = [&]() {
    const int key = (ahead.tile << shift) + my_key;
    off = -1;
    if (fetch_left > 0 && key < ahead.len) {
      const int p = div_page(key, a.page_mul, a.page_shift);
      const int page = __ldg(a.table + (long long)ahead.r * a.table_stride + p);
      if (page < 0 || page >= a.num_pages) atomicOr(a.status, FA_DEV_BOUNDS);
      else off = page * a.c_sp + (key - p * a.page_size) * a.c_st;
    }
  };
  auto fetch = [&](int stage) {  // copies the tile `ahead`, whose keys are at `off`
    if (fetch_left > 0) {
      const int live = ahead.len - ((ahead.tile << shift) + kw * KEYS);
      if (live > 0) {
        const long long head_off = (long long)((NQ == 1 ? ahead.hm : ahead.hm / runs) * a.hp + hw) * a.c_sh;
        const uint8_t* base = a.k + head_off + lane_off;
        const uint32_t dst0 = ring + stage * C::STAGE + crow * ROWB;
#pragma unroll
        for (int i = 0; i < KEYS / C::RPI; ++i) {
          const int row = i * C::RPI + crow;
          const long long o = __shfl_sync(0xffffffffu, off, joint ? i : row);
          const bool there = o >= 0 && row < live;  // else the key reads as zeros
          const uint8_t* src = base + (there ? o : -head_off - lane_off);
          const uint32_t dst = dst0 + i * C::RPI * ROWB + ((cc ^ swz<CH>(row)) * 16);
          cp_async16(dst, src, there ? 16 : 0);
          cp_async16(dst + KEYS * ROWB, src + vk, there ? 16 : 0);
        }
      }
      if (--fetch_left > 0) cursor_next(a, ahead, groups, shift);
    }
    cp_commit();
    lookup();
  };
  lookup();
  Cursor line[kStages];  // the tiles on their way, the one that is computed next in front
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    line[s] = ahead;
    fetch(s);
  }

  write_empty();

  // ---- computing.  The thread's share of S^T and O^T: query rows 8 n + 2 i4 + e of keys (or
  // columns) g8 and g8 + 8 of each 16.
  const int i4 = lane & 3, g8 = lane >> 2;
  float acc[DC][NQ][4];
  float m[NQ][2], l[NQ][2];
  uint32_t qb[DC][NQ][2];
  float sc[NQ][2];  // factor from the product to base-2 scores
  // The queries of c's (row, kv head), as stored.
  auto load_q = [&](const Cursor& c) {
    const int hg = NQ == 1 ? c.hm : c.hm / runs, row0 = (c.hm - hg * runs) * kMaxRows, rows = min(kMaxRows, g - row0);
    const __nv_bfloat16* q0 = a.q + c.t * a.q_st + ((long long)(hg * a.hp + hw) * g + row0) * a.q_sh;
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const bool live = 8 * n + g8 < rows;
      const __nv_bfloat16* qr = q0 + (live ? 8 * n + g8 : 0) * a.q_sh;
#pragma unroll
      for (int s = 0; s < DC; ++s) {
        if (FP8) {
          const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(qr + 16 * s + 4 * i4)) : make_uint2(0, 0);
          qb[s][n][0] = v.x, qb[s][n][1] = v.y;
        } else {
          qb[s][n][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 2 * i4)) : 0u;
          qb[s][n][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 8 + 2 * i4)) : 0u;
        }
      }
    }
  };
  load_q(line[0]);
  int stage = 0;
  bool fresh = true;
  int seg_tile0 = line[0].tile;
  while (left > 0) {
    const Cursor cur = line[0];
    const int hg = NQ == 1 ? cur.hm : cur.hm / runs, hk = hg * a.hp + hw;
    const int row0 = (cur.hm - hg * runs) * kMaxRows, rows = min(kMaxRows, g - row0);
    if (fresh) {  // a (row, kv head) begins: its queries are in qb
      fresh = false;
      seg_tile0 = cur.tile;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        if (!FP8) {
          sc[n][0] = sc[n][1] = a.scale_log2;
        } else {
          // q to fp16: the row is scaled by a power of two that brings its largest element into
          // [2^15, 2^16), where bf16's 8 bits still end at fp16's largest value.  Elements are then exact
          // down to 2^-32 of that one, and to 2^-40 of it below (fp16's smallest step is 2^-24).
          float big = 0.f;
#pragma unroll
          for (int s = 0; s < DC; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              big = fmaxf(big, fmaxf(fabsf(__uint_as_float(qb[s][n][e] << 16)), fabsf(__uint_as_float(qb[s][n][e] & 0xffff0000u))));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const int e = min(max((int)(__float_as_uint(big) >> 23), 16), 254);  // biased exponent
          const float down = __uint_as_float((uint32_t)(269 - e) << 23), up = __uint_as_float((uint32_t)(e - 15) << 23);
#pragma unroll
          for (int s = 0; s < DC; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              qb[s][n][e] = pack_f16(__uint_as_float(qb[s][n][e] << 16) * down,
                                     __uint_as_float(qb[s][n][e] & 0xffff0000u) * down);
          const float f = a.scale_log2 * (a.kd ? __ldg(a.kd + hk) : 1.f) * up;
          sc[n][0] = __shfl_sync(0xffffffffu, f, 8 * i4);
          sc[n][1] = __shfl_sync(0xffffffffu, f, 8 * i4 + 4);
        }
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int c = 0; c < DC; ++c) acc[c][n][0] = acc[c][n][1] = acc[c][n][2] = acc[c][n][3] = 0.f;
      }
    }

    cp_wait<kStages - 1>();
    __syncwarp();
    const int live = cur.len - ((cur.tile << shift) + kw * KEYS);
    if (live > 0) {
      const uint32_t kb = ring + stage * C::STAGE, vb = kb + KEYS * ROWB;
      float s[MT][NQ][4];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int row = t * 16 + (lane & 15);
#pragma unroll
        for (int n = 0; n < NQ; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          uint32_t r[4];
          ldsm4(r, kb + row * ROWB + (((c + (lane >> 4)) ^ swz<CH>(row)) * 16));
          if (!FP8) {
#pragma unroll
            for (int n = 0; n < NQ; ++n) mma16816<false>(s[t][n], r[0], r[1], r[2], r[3], qb[c / 2][n][0], qb[c / 2][n][1]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // a 16-byte chunk: the lane's 4 codes feed k slots 2 i4, + 1, + 8, + 9
              const uint32_t a0 = e4m3_lo(r[2 * e]), a1 = e4m3_lo(r[2 * e + 1]);
              const uint32_t a2 = e4m3_hi(r[2 * e]), a3 = e4m3_hi(r[2 * e + 1]);
#pragma unroll
              for (int n = 0; n < NQ; ++n) mma16816<true>(s[t][n], a0, a1, a2, a3, qb[c + e][n][0], qb[c + e][n][1]);
            }
          }
        }
      }
      // base-2 scores, the last keys masked; does any exceed its reference by too much?
      bool moved = false;
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& v = s[t][n][e];
            v *= sc[n][e & 1];
            if (live < KEYS && t * 16 + g8 + 8 * (e >> 1) >= live) v = -INFINITY;
            moved |= v > m[n][e & 1] + kSlack;
          }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mn = m[n][e];
#pragma unroll
            for (int t = 0; t < MT; ++t) mn = fmaxf(mn, fmaxf(s[t][n][e], s[t][n][e + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            const float al = mn == -INFINITY ? 1.f : ex2(m[n][e] - mn);
            m[n][e] = mn;
            l[n][e] *= al;
#pragma unroll
            for (int c = 0; c < DC; ++c) acc[c][n][e] *= al, acc[c][n][e + 2] *= al;
          }
      }
      // P: its terms for every 16 keys, transposed
      uint32_t hi[MT][NQ][2], lo[MT][NQ][2], last[MT][NQ][2];  // last: bf16 alone
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float ref = (m[n][e & 1] == -INFINITY ? 0.f : m[n][e & 1]) - (FP8 ? kPBias : 0.f);
            p[e] = ex2(s[t][n][e] - ref);
            l[n][e & 1] += p[e];
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (FP8) {
              const uint32_t u = pack_f16(p[2 * h], p[2 * h + 1]);
              const float2 f = unpack_f16(u);
              hi[t][n][h] = transpose8(u);
              lo[t][n][h] = transpose8(pack_f16(p[2 * h] - f.x, p[2 * h + 1] - f.y));
            } else {
              const float p0 = p[2 * h], p1 = p[2 * h + 1], a0 = below(p0), a1 = below(p1);
              const float r0 = p0 - a0, r1 = p1 - a1, b0 = below(r0), b1 = below(r1);
              hi[t][n][h] = transpose8(high_halves(a0, a1));
              lo[t][n][h] = transpose8(high_halves(b0, b1));
              last[t][n][h] = transpose8(pack_bf16(r0 - b0, r1 - b1));
            }
          }
        }
      // O^T += V^T P^T.  The matrix unit cuts its sums instead of rounding them, and what it cuts off a long
      // sum adds up (3e-5 of it over 128 tiles), so a tile's products are summed apart, the smallest
      // terms first, and added to O with rounding; 1 % of the long cases' times.
      if (!FP8) {
        const int half = (lane >> 3) & 1;
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          float x[NQ][4];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const int row = t * 16 + (lane & 7) + ((lane >> 4) << 3);
            uint32_t r[4];
            ldsm4t(r, vb + row * ROWB + (((2 * c + half) ^ swz<CH>(row)) * 16));
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
              if (t == 0) mma16816_new<false>(x[n], r[0], r[1], r[2], r[3], last[t][n][0], last[t][n][1]);
              else mma16816<false>(x[n], r[0], r[1], r[2], r[3], last[t][n][0], last[t][n][1]);
              mma16816<false>(x[n], r[0], r[1], r[2], r[3], lo[t][n][0], lo[t][n][1]);
              mma16816<false>(x[n], r[0], r[1], r[2], r[3], hi[t][n][0], hi[t][n][1]);
            }
          }
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][n][e] += x[n][e];
        }
      } else {
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          float x[2][NQ][4];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            const int row = t * 16 + (lane & 15);
            uint32_t r[4];
            ldsm4t(r, vb + row * ROWB + (((c + (lane >> 4)) ^ swz<CH>(row)) * 16));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // a register holds two keys of two neighbouring columns: the even columns become rows
              // g8 of the 16-row tile, the odd ones rows g8 + 8
              const uint32_t u0 = __byte_perm(r[2 * e], 0, 0x3120), u1 = __byte_perm(r[2 * e + 1], 0, 0x3120);
              const uint32_t a0 = e4m3_lo(u0), a1 = e4m3_hi(u0), a2 = e4m3_lo(u1), a3 = e4m3_hi(u1);
#pragma unroll
              for (int n = 0; n < NQ; ++n) {
                if (t == 0) mma16816_new<true>(x[e][n], a0, a1, a2, a3, lo[t][n][0], lo[t][n][1]);
                else mma16816<true>(x[e][n], a0, a1, a2, a3, lo[t][n][0], lo[t][n][1]);
                mma16816<true>(x[e][n], a0, a1, a2, a3, hi[t][n][0], hi[t][n][1]);
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[c + e][n][k] += x[e][n][k];
        }
      }
    }
    --left;

    const bool seg_end = cur.tile + 1 == cur.tiles;
    if (seg_end || left == 0) {  // join the warps, 8 rows at a time
      if (left > 0) load_q(line[1]);  // on their way meanwhile
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
          if (g8 == 0) s_m[warp][8 * n + 2 * i4 + e] = m[n][e], s_l[warp][8 * n + 2 * i4 + e] = l[n][e];
        }
      const bool whole = seg_end && seg_tile0 == 0;
      const int slot = 2 * cta + (seg_tile0 == 0 ? 1 : 0);
      if (tid == 0 && seg_tile0 == 0 && (by_group || left == 0)) {  // the group began here: is it divided?
        // the CTA that holds its last tile, if it is (its present tile is then the last of this CTA's run)
        const long long end = first + per + (cta < extra) - 1 + (cur.tiles - 1 - cur.tile), split = extra * (per + 1);
        const long long holder = end < split ? quotient(end, per + 1) : extra + quotient(end - split, per);
        part.head[by_group ? cur.t * groups + cur.hm : cta] =
            whole ? make_int4(-1, 0, 0, 0) : make_int4(cur.t, cur.hm, cta, (int)holder);
      }
      __syncthreads();
      // lane r of each warp: the max and sum of its head's query row r over the warps, and what its
      // own warp's O is to be multiplied by, so that the warps' O only have to be added
      float fac = 0.f;
      if (lane < 8 * NQ) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          if ((w & (a.hp - 1)) == hw) M = fmaxf(M, s_m[w][lane]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = s_m[w][lane], f = mw == -INFINITY ? (M == -INFINITY ? 1.f : 0.f) : ex2(mw - M);
          if ((w & (a.hp - 1)) == hw) L = fmaf(f, s_l[w][lane], L);
          if (w == warp) fac = f;
        }
        if (whole) fac *= L > 0.f || L != L ? (FP8 && a.vd ? __ldg(a.vd + hk) : 1.f) / L : 0.f;
        if (kw == 0 && lane < rows) {
          if (whole) write_lse(a, cur.t, hk * g + row0 + lane, M, L, FP8 ? kPBias : 0.f);
          else part.ml[((size_t)slot * a.hp + hw) * kMaxRows + lane] = make_float2(M, L);
        }
      }
      // through the stage just read, which is filled again only after the last barrier here
      float* join = reinterpret_cast<float*>(smem + stage * C::STAGE);
      constexpr int RS = C::RS, WS = kStages * C::STAGE / 4;
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const int nrows = min(8, rows - 8 * n);
        if (nrows <= 0) break;
        float* dst = join + warp * WS + 2 * i4 * RS;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = __shfl_sync(0xffffffffu, fac, 8 * n + 2 * i4 + e);
#pragma unroll
          for (int c = 0; c < DC; ++c) {
            if (FP8) {
              *reinterpret_cast<float2*>(dst + e * RS + c * 16 + 2 * g8) = make_float2(acc[c][n][e] * f, acc[c][n][e + 2] * f);
            } else {
              dst[e * RS + c * 16 + g8] = acc[c][n][e] * f;
              dst[e * RS + c * 16 + g8 + 8] = acc[c][n][e + 2] * f;
            }
          }
        }
        __syncthreads();
        const int c4 = tid % (D / 4);
        for (int h = 0; h < a.hp; ++h)
#pragma unroll 2
          for (int row = tid / (D / 4); row < nrows; row += kWarps * 32 / (D / 4)) {
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
              if ((w & (a.hp - 1)) == h) {
                const float4 v = *reinterpret_cast<const float4*>(join + w * WS + row * RS + c4 * 4);
                o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
              }
            if (whole) {
              const long long at = cur.t * (long long)a.Hq + (hg * a.hp + h) * g + row0 + 8 * n + row;
              *reinterpret_cast<uint2*>(a.o + at * D + c4 * 4) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            } else {
              const size_t pr = ((size_t)slot * a.hp + h) * kMaxRows + 8 * n + row;
              *reinterpret_cast<float4*>(part.o + pr * D + c4 * 4) = o;
            }
          }
        __syncthreads();
      }
      fresh = true;
    } else {
      __syncwarp();  // all lanes have read the stage that is filled next
    }
#pragma unroll
    for (int s = 0; s + 1 < kStages; ++s) line[s] = line[s + 1];
    line[kStages - 1] = ahead;
    fetch(stage);
    stage = stage == kStages - 1 ? 0 : stage + 1;
    if (left == 0) {
      if (tid == 0 && !by_group && seg_tile0 != 0) part.head[cta] = make_int4(-1, 0, 0, 0);  // no group began last
    }
  }
  cp_wait<0>();
}

// Joins the parts of one divided group (block x: see Workspace), rows y, y + gridDim.y, ... of its
// hp heads: a run of D / 4 threads per row, or several that share its parts when there are few
// rows, with a running max over kJoinBatch parts at a time (always in the same order).  Nothing
// but latency counts here: one round trip for the header, then one for each batch.
constexpr int kJoinBatch = 4;
template <int D, bool FP8>
__global__ void __launch_bounds__(256) fa_paged_join_kernel(const DecodeArgs a, int ctas) {
  constexpr int TPR = D / 4, RUNS = 256 / TPR;
  __shared__ float4 red[256];
  __shared__ float2 red_ml[RUNS];
  const int tid = threadIdx.x, c4 = tid % TPR;
  const Part part = part_of(a.workspace, ctas);
  const int g = a.Hq / a.Hk, runs = (g + kMaxRows - 1) / kMaxRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 head = part.head[blockIdx.x];  // row, group, first CTA, last CTA
  if (head.x < 0) return;
  const int hg = head.y / runs;
  const int row0 = (head.y - hg * runs) * kMaxRows, rows = min(kMaxRows, g - row0), n = head.w - head.z + 1;
  const int y = blockIdx.y, ny = gridDim.y;
  const int mine = (a.hp * rows - y + ny - 1) / ny;  // rows y + ny * (0 .. mine - 1) of hp * rows
  const int slices = max(1, RUNS / max(1, mine)), items = mine * slices;
  for (int base = 0; base < items; base += RUNS) {
    const int item = base + tid / TPR, q = item / slices, slice = item - q * slices;
    const int hr = y + ny * q, h = hr / rows, row = hr - h * rows;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0, 0, 0, 0);
    if (item < items) {
      for (int i0 = slice; i0 < n; i0 += kJoinBatch * slices) {
        float2 ml[kJoinBatch];
        float4 v[kJoinBatch];
        float mn = M;
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
          const int i = i0 + j * slices;
          ml[j] = make_float2(-INFINITY, 0.f);
          v[j] = make_float4(0, 0, 0, 0);
          if (i < n) {  // (the first part lies in its CTA's second slot)
            const size_t pr = (((size_t)2 * (head.z + i) + (i == 0 ? 1 : 0)) * a.hp + h) * kMaxRows + row;
            ml[j] = part.ml[pr];
            v[j] = *reinterpret_cast<const float4*>(part.o + pr * D + c4 * 4);
          }
        }
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) mn = fmaxf(mn, ml[j].x);
        const float f0 = M == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : ex2(M - mn);
        L *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
#pragma unroll
        for (int j = 0; j < kJoinBatch; ++j) {
          const float f = ml[j].x == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : ex2(ml[j].x - mn);
          L = fmaf(f, ml[j].y, L);
          o.x = fmaf(f, v[j].x, o.x), o.y = fmaf(f, v[j].y, o.y), o.z = fmaf(f, v[j].z, o.z), o.w = fmaf(f, v[j].w, o.w);
        }
        M = mn;
      }
    }
    if (slices > 1) {  // (then one round holds everything)
      red[tid] = o;
      if (c4 == 0) red_ml[tid / TPR] = make_float2(M, L);
      __syncthreads();
      if (item < items && slice == 0) {
        float mn = M;
        for (int i = 1; i < slices; ++i) mn = fmaxf(mn, red_ml[item + i].x);
        const float f0 = M == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : ex2(M - mn);
        L *= f0, o.x *= f0, o.y *= f0, o.z *= f0, o.w *= f0;
        for (int i = 1; i < slices; ++i) {
          const float2 ml = red_ml[item + i];
          const float4 v = red[tid + i * TPR];
          const float f = ml.x == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : ex2(ml.x - mn);
          L = fmaf(f, ml.y, L);
          o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
        }
        M = mn;
      }
    }
    if (item < items && slice == 0) {
      const int kvh = hg * a.hp + h;
      const float vscale = FP8 && a.vd ? __ldg(a.vd + kvh) : 1.f;
      write_out<D>(a, head.x, kvh * g + row0 + row, c4, o, M, L, vscale, FP8 ? kPBias : 0.f);
    }
  }
}

int sm_count() {
  static int cached[64];
  int dev = 0, v = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev >= 0 && dev < 64 && cached[dev]) return cached[dev];
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return 148;
  if (dev >= 0 && dev < 64) cached[dev] = v;
  return v;
}

int decode_ctas(int per_sm) { return per_sm * sm_count(); }

template <int D, bool FP8, int NQ>
cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t stream) {
  using C = DecCfg<D, FP8, NQ>;
  static_assert(C::CTAS * (C::SMEM + 2048) <= 228 * 1024, "CTAS CTAs fit an SM");
  static bool attr_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(fa_paged_decode_kernel<D, FP8, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int ctas = decode_ctas(C::CTAS);
  fa_paged_decode_kernel<D, FP8, NQ><<<ctas, kWarps * 32, C::SMEM, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // a block for every group that can be divided, and, when they are few, several for each
  const int g = a.Hq / a.Hk, groups = (a.Hk / a.hp) * ((g + kMaxRows - 1) / kMaxRows);
  const int nb = (int)std::min<long long>(ctas, (long long)a.T * groups);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nb, std::min(a.hp * std::min(g, kMaxRows), std::max(1, 4 * sm_count() / nb)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_join_kernel<D, FP8>, a, ctas);
}

}  // namespace

// n / page_size = n * mul >> shift for every n < 2^31 (Granlund and Montgomery, "Division by Invariant
// Integers using Multiplication").
static void page_division(int page_size, uint64_t* mul, int* shift) {
  int bits = 0;
  while ((1LL << bits) < page_size) ++bits;
  *shift = 31 + bits;
  *mul = (uint64_t)((((unsigned __int128)1 << *shift) + page_size - 1) / page_size);
}

// Prepares the plan kernel on the current device (once); the largest cluster of it that can run there.
static cudaError_t plan_ctas(int* most) {
  static int cached[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && cached[dev]) {
    *most = cached[dev];
    return cudaSuccess;
  }
  constexpr int smem = (4 * FA_PLAN_MAX_REQUESTS + 2) * 4;
  if ((e = cudaFuncSetAttribute(fa_paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(fa_paged_plan_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanMaxCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {kPlanMaxCtas, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, fa_paged_plan_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();  // (not an error of the call)
    clusters = 0;
  }
  *most = clusters > 0 ? kPlanMaxCtas : 8;
  if (dev >= 0 && dev < 64) cached[dev] = *most;
  return cudaSuccess;
}

cudaError_t launch_paged_plan(PlanArgs a, cudaStream_t stream) {
  page_division(a.page_size, &a.page_mul, &a.page_shift);
  a.wide = ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions) |
             reinterpret_cast<uintptr_t>(a.token_req)) & 15) == 0;
  const int smem = (4 * a.R + 2) * 4;
  int most = 0;
  cudaError_t e = plan_ctas(&most);
  if (e != cudaSuccess) return e;
  const long long share = (long long)kPlanThreads * kPlanPer;
  const int ctas = (int)std::min<long long>(
      most, std::max<long long>({1, (a.R + kPlanRequests - 1) / kPlanRequests, (a.max_tokens + share - 1) / share,
                                 std::min<long long>(a.pool_pages, (long long)a.R * a.table_cols) / kPlanPages}));
  const int need = std::max(a.R, ctas > 1 ? kPlanThreads : (a.max_tokens + kPlanPer - 1) / kPlanPer);
  const int threads = std::min(kPlanThreads, std::max(64, (need + 31) / 32 * 32));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fa_paged_plan_kernel, a);
}

size_t paged_decode_workspace(int T, int Hq, int Hk, int d) {
  (void)T, (void)Hq, (void)Hk, (void)d;
  const int ctas = decode_ctas(kMaxCtasPerSm);
  // hp * row bytes is at most 256, i.e. hp * d * 4 at most 1024 bytes (E4M3)
  return part_head_bytes(ctas) + part_ml_bytes(ctas) + (size_t)ctas * 2 * kMaxRows * 1024;
}

cudaError_t launch_paged_decode(int d, bool fp8, DecodeArgs a, cudaStream_t stream) {
  page_division(a.page_size, &a.page_mul, &a.page_shift);
  // Heads side by side: when a token's heads follow one another, as many as make up 256 bytes are read
  // at once; pieces of 128 bytes read alone, at different times, reach a tenth less bandwidth.
  const int row_bytes = d * (fp8 ? 1 : 2);
  a.hp = 1;
  while (a.c_sh == row_bytes && 2 * a.hp * row_bytes <= 256 && a.Hk % (2 * a.hp) == 0) a.hp *= 2;
  const bool few = a.Hq / a.Hk <= 8;
  if (d == 64) {
    if (fp8) return few ? launch_decode_t<64, true, 1>(a, stream) : launch_decode_t<64, true, 2>(a, stream);
    return few ? launch_decode_t<64, false, 1>(a, stream) : launch_decode_t<64, false, 2>(a, stream);
  }
  if (fp8) return few ? launch_decode_t<128, true, 1>(a, stream) : launch_decode_t<128, true, 2>(a, stream);
  return few ? launch_decode_t<128, false, 1>(a, stream) : launch_decode_t<128, false, 2>(a, stream);
}

}  // namespace fa
