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
// depends on the inputs alone.  Everything is one kernel: every block of one cluster scans the
// requests for itself (a few bytes each, from L2), the cluster's barrier separates reading the
// inputs from writing, which is what lets the outputs alias them, and then the tokens are spread
// over all threads.  Nothing is written but `plan_status`, the unchanged lengths and the -1
// padding when the step cannot be planned.
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxCtas = 8;
constexpr int kPlanTokensPerThread = 4;

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

__global__ void __launch_bounds__(kPlanThreads) fa_paged_plan_kernel(const PlanArgs a) {
  // per request: cached length (complemented when released), first wanted or released page in
  // the step's order, first token
  extern __shared__ int sm[];
  int* s_cached = sm;
  int* s_first = sm + a.R;
  int* s_cu = sm + 2 * a.R;  // R + 1
  __shared__ Sum3 warp_sum[32];
  __shared__ Sum3 carry;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x;  // the grid is one cluster
  const int ps = a.page_size;
  const long long room = (long long)a.table_cols * ps;

  const int free0 = *a.free_count;
  int bits = 0;
  if (tid == 0) carry = {0, 0, 0};
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
      const int used = (int)(((long long)cached + ps - 1) / ps);
      if (add < 0) {
        v.back = used;
      } else if ((long long)cached + add > room) {
        bits |= FA_PLAN_ROW_FULL;
      } else {
        v.grow = add;
        v.want = ((long long)cached + add + ps - 1) / ps - used;
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
      s_first[b] = (int)(add < 0 ? ex.back : ex.want);
      s_cu[b] = (int)ex.grow;
    }
    __syncthreads();
    if (tid == 0) carry = carry + warp_sum[nw - 1];
    __syncthreads();
  }
  const Sum3 total = carry;
  const long long avail = free0 + total.back;
  if (free0 < 0 || avail > a.pool_pages) bits |= FA_PLAN_BAD_INPUT;
  else if (total.want > avail) bits |= FA_PLAN_NO_PAGES;
  if (total.grow > a.max_tokens) bits |= FA_PLAN_TOO_MANY_TOKENS;
  bits = (__syncthreads_or(bits & 1) ? 1 : 0) | (__syncthreads_or(bits & 2) ? 2 : 0) |
         (__syncthreads_or(bits & 4) ? 4 : 0) | (__syncthreads_or(bits & 8) ? 8 : 0);
  const bool ok = bits == 0;
  const int tokens = ok ? (int)total.grow : 0;
  if (tid == 0) s_cu[a.R] = tokens;
  if (ctas > 1) cluster_sync();  // every block has read the inputs; nothing is written before
  else __syncthreads();

  const int gt = rank * nt + tid, gn = ctas * nt;
  if (gt == 0) {
    *a.free_count_out = ok ? (int)(avail - total.want) : free0;
    *a.plan_status = bits;
    a.cu_tokens[a.R] = tokens;
  }
  if (ok && total.back > 0) {  // released pages onto the stack, a warp per request
    for (int b = rank * nw + warp; b < a.R; b += ctas * nw) {
      const int c = s_cached[b];
      if (c >= 0) continue;
      const int used = (int)(((long long)~c + ps - 1) / ps);
      const int* row = a.table + (long long)b * a.table_stride;
      int* top = a.free_pages + free0 + s_first[b];
      for (int p = lane; p < used; p += 32) top[p] = row[p];
    }
    if (ctas > 1) cluster_sync();
    else __syncthreads();
  }
  for (int b = gt; b < a.R; b += gn) {
    const int c = s_cached[b];
    a.lens[b] = !ok ? a.cached[b] : c < 0 ? 0 : c + s_cu[b + 1] - s_cu[b];
    a.cu_tokens[b] = ok ? s_cu[b] : 0;
  }
  const int top = (int)(avail - 1);
  for (int t = gt; t < a.max_tokens; t += gn) {
    long long slot = -1;
    int pos = 0, req = -1;
    if (t < tokens) {
      int lo = 0, hi = a.R;  // the request with cu[lo] <= t < cu[lo + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      req = lo;
      const int c = s_cached[lo];
      pos = c + t - s_cu[lo];
      const int p = pos / ps, used = (int)(((long long)c + ps - 1) / ps), in = pos - p * ps;
      int page;
      if (p < used) {
        page = a.table[(long long)lo * a.table_stride + p];
      } else {  // a page of this step; its first token enters it in the table
        page = a.free_pages[top - (s_first[lo] + p - used)];
        if (in == 0) a.table[(long long)lo * a.table_stride + p] = page;
      }
      slot = (long long)page * ps + in;
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
    a.token_req[t] = req;
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
// Inside a CTA each warp owns every fourth run of KEYS keys and its own ring of shared-memory
// stages, filled by 16-byte asynchronous copies straight from the pages (a lane looks up the page
// of one key, so a page may end anywhere), and keeps its own running max, sum and O: no barrier
// until a (row, kv head) ends, when the four are joined in shared memory.
//
// The g query heads of a kv head are the rows of the matrix products (m16n8k16, fp32
// accumulators).  K and V come once from memory and feed 4 g flops per element, an order of
// magnitude below what the tensor pipe needs to be the bound at the copy bandwidth.  P is kept to
// 16 bits: in bf16 as the sum of two bf16 terms (a high and a low part, so the product's rounding
// stays below the output's), which with at most 8 rows ride in the unused half of the 16-row tile
// for free; with an E4M3 cache, whose values are exact in fp16, as one fp16 term.
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kMaxRows = 16;

template <int D, bool FP8>
struct DecCfg {
  static constexpr int ROWB = D * (FP8 ? 1 : 2);          // bytes of a key's row
  static constexpr int CH = ROWB / 16;                    // 16-byte chunks of a row
  static constexpr int KEYS = ROWB == 256 ? 16 : 32;      // keys per warp and tile
  static constexpr int TILE = KEYS * kWarps;              // keys per tile
  static constexpr int STAGE = 2 * KEYS * ROWB;           // K then V
  static constexpr int RPI = 32 / CH;                     // rows that one copy instruction covers
  static constexpr int PAD = FP8 ? 16 : 8;                // floats; keeps the joins off one bank
  static constexpr int SMEM = kWarps * kStages * STAGE;
  static_assert(8 * (D + PAD) * 4 <= STAGE, "a stage holds 8 rows of a warp's O at the join");
};

// Chunk c of row r sits at chunk c ^ swz(r): the 8 rows that one ldmatrix reads at equal c then
// cover all banks.
template <int CH>
__device__ __forceinline__ int swz(int r) {
  return CH >= 8 ? (r & 7) : ((r >> 1) & 3);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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
// Two E4M3 codes (low 16 bits) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Number of keys of query row t; 0 writes an empty row's result, -1 leaves the row as it was.
// `r` is its row of the block table.
__device__ __forceinline__ int row_keys(const DecodeArgs& a, int t, int& r) {
  r = a.req ? a.req[t] : t;
  if (r < 0) return -1;
  if (r >= a.table_rows) {
    atomicOr(a.status, FA_DEV_BOUNDS);
    return -1;
  }
  const int len = a.lens[t];
  if (len < 0 || len > (long long)a.table_cols * a.page_size) {
    atomicOr(a.status, FA_DEV_BOUNDS);
    return 0;
  }
  return len;
}

// A place in the line of tiles: row t, group hm = kv head * row tiles + row tile, tile.
struct Cursor {
  int t, hm, tile, tiles, len, r;
};

template <int TILE>
__device__ __forceinline__ void cursor_next_row(const DecodeArgs& a, Cursor& c) {
  do {
    ++c.t;
    if (c.t >= a.T) {  // past the end: nothing follows
      c.tiles = 0, c.len = 0;
      return;
    }
    c.len = row_keys(a, c.t, c.r);
    c.tiles = (max(c.len, 0) + TILE - 1) / TILE;
  } while (c.tiles == 0);
}
template <int TILE>
__device__ __forceinline__ void cursor_next(const DecodeArgs& a, Cursor& c, int hms) {
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.hm < hms) return;
  c.hm = 0;
  cursor_next_row<TILE>(a, c);
}

// Workspace: header[ctas] (segment that begins in the CTA and runs past it: row, group, last
// CTA), then per CTA two partial results of kMaxRows rows: (max, sum) pairs and fp32 O.
struct Part {
  int4* head;
  float2* ml;
  float* o;
};
__host__ __device__ __forceinline__ size_t part_head_bytes(int ctas) { return ((size_t)ctas * 16 + 255) & ~(size_t)255; }
__host__ __device__ __forceinline__ size_t part_ml_bytes(int ctas) { return (size_t)ctas * 2 * kMaxRows * 8; }
__device__ __forceinline__ Part part_of(void* ws, int ctas) {
  char* p = reinterpret_cast<char*>(ws);
  Part r;
  r.head = reinterpret_cast<int4*>(p);
  r.ml = reinterpret_cast<float2*>(p + part_head_bytes(ctas));
  r.o = reinterpret_cast<float*>(p + part_head_bytes(ctas) + part_ml_bytes(ctas));
  return r;
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
  if (c4 == 0) a.lse[t * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l) - bias) * 0.6931471805599453f;
}

// P of the E4M3 form carries this power of two, so that fp16 holds it to full precision down to
// 2^-28 of the row's largest.
constexpr float kPBias = 14.f;

template <int D, bool FP8, bool R8>
__global__ void __launch_bounds__(kWarps * 32, 2) fa_paged_decode_kernel(const DecodeArgs a) {
  using C = DecCfg<D, FP8>;
  constexpr int KEYS = C::KEYS, TILE = C::TILE, NT = KEYS / 8, CH = C::CH, ROWB = C::ROWB;
  constexpr int KS = D / 16;      // 16-wide steps of the score product
  constexpr int DN = D / 8;       // 8-wide tiles of O
  constexpr int H = R8 ? 1 : 2;   // row halves (rows lane/4 and lane/4 + 8) in use
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_scan[kWarps + 1];
  __shared__ int s_start[4];
  __shared__ float s_m[kWarps][kMaxRows], s_l[kWarps][kMaxRows];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = gridDim.x, cta = blockIdx.x;
  const int g = a.Hq / a.Hk, mt = (g + kMaxRows - 1) / kMaxRows, hms = a.Hk * mt;
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- the cut: tiles of a run of rows per thread, scanned over the block
  const int per_thread = (a.T + kWarps * 32 - 1) / (kWarps * 32);
  const int t0 = min(a.T, tid * per_thread), t1 = min(a.T, t0 + per_thread);
  long long mine = 0;
  for (int t = t0; t < t1; ++t) {
    int r;
    mine += (max(row_keys(a, t, r), 0) + TILE - 1) / TILE;
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
  total *= hms;
  const long long ctas = min((long long)G, total);
  Part part = part_of(a.workspace, G);

  // rows without a visible key
  for (int t = cta; t < a.T; t += G) {
    int r;
    if (row_keys(a, t, r) == 0)
      for (int i = tid; i < a.Hq * (D / 4); i += kWarps * 32)
        write_out<D>(a, t, i / (D / 4), i % (D / 4), make_float4(0, 0, 0, 0), 0.f, 0.f, 0.f, 0.f);
  }
  if (cta >= ctas) {
    if (tid == 0) part.head[cta] = make_int4(-1, 0, 0, 0);
    return;
  }
  const long long first = total * cta / ctas, last = total * (cta + 1) / ctas;  // [first, last)
  if (before * hms <= first && first < (before + mine) * hms) {
    long long at = before * hms;
    for (int t = t0; t < t1; ++t) {
      int r;
      const long long n = (max(row_keys(a, t, r), 0) + TILE - 1) / TILE;
      if (first < at + n * hms) {
        s_start[0] = t;
        s_start[1] = (int)((first - at) / n);
        s_start[2] = (int)((first - at) % n);
        break;
      }
      at += n * hms;
    }
  }
  __syncthreads();
  Cursor cur;
  cur.t = s_start[0];
  cur.hm = s_start[1];
  cur.tile = s_start[2];
  cur.len = row_keys(a, cur.t, cur.r);
  cur.tiles = (cur.len + TILE - 1) / TILE;
  Cursor ahead = cur;  // the next tile to fetch
  int fetch_left = (int)(last - first);
  int left = fetch_left;

  // ---- fetching: lane kk looks up key kk of the warp's share of a tile
  const uint32_t ring = smem_u32(smem) + warp * kStages * C::STAGE;
  const int kk = lane % KEYS;
  int page = 0;
  auto lookup = [&]() {
    const int key = ahead.tile * TILE + warp * KEYS + kk;
    page = -1;
    if (fetch_left > 0 && key < ahead.len) {
      page = __ldg(a.table + (long long)ahead.r * a.table_stride + key / a.page_size);
      if (page < 0 || page >= a.num_pages) {
        atomicOr(a.status, FA_DEV_BOUNDS);
        page = -1;
      }
    }
  };
  auto fetch = [&](int stage) {  // copies the tile `ahead`, whose pages are in `page`
    if (fetch_left > 0) {
      const int key0 = ahead.tile * TILE + warp * KEYS;
      if (key0 < ahead.len) {
        const int key = key0 + kk;
        long long off = -1;  // a key past the end (or on a page that does not exist) reads as zeros
        if (page >= 0)
          off = page * a.c_sp + (key % a.page_size) * a.c_st + (ahead.hm / mt) * a.c_sh;
        const uint32_t dst0 = ring + stage * C::STAGE;
#pragma unroll
        for (int i = 0; i < KEYS / C::RPI; ++i) {
          const int row = i * C::RPI + lane / CH, c = lane % CH;
          const long long o = __shfl_sync(0xffffffffu, off, row);
          const int n = o < 0 ? 0 : 16;
          const long long src = (o < 0 ? 0 : o) + c * 16;
          const uint32_t dst = dst0 + row * ROWB + ((c ^ swz<CH>(row)) * 16);
          cp_async16(dst, a.k + src, n);
          cp_async16(dst + KEYS * ROWB, a.v + src, n);
        }
      }
      --fetch_left;
      cursor_next<TILE>(a, ahead, hms);
    }
    cp_commit();
    lookup();
  };
  lookup();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s);

  // ---- computing
  float acc[DN][4];
  float m[H], l[H];
  uint32_t qa[KS][4];
  float sc[H];  // factor from the product to base-2 scores
  const int i4 = lane & 3, g8 = lane >> 2;
  int stage = 0;
  bool fresh = true;
  int seg_tile0 = cur.tile;
  while (left > 0) {
    const int hk = cur.hm / mt, rt = cur.hm - hk * mt, row0 = rt * kMaxRows, rows = min(kMaxRows, g - row0);
    if (fresh) {  // this (row, kv head)'s queries, and an empty result
      fresh = false;
      seg_tile0 = cur.tile;
      const __nv_bfloat16* q0 = a.q + cur.t * a.q_st + (long long)(hk * g + row0) * a.q_sh;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = g8 + 8 * h;
        const bool live = h < H && row < rows;
        const __nv_bfloat16* qr = q0 + (live ? row : 0) * a.q_sh;
        if (!FP8) {
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            qa[s][h] = live ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 2 * i4)) : 0u;
            qa[s][2 + h] = live ? __ldg(reinterpret_cast<const uint32_t*>(qr + 16 * s + 8 + 2 * i4)) : 0u;
          }
          if (h < H) sc[h] = a.scale_log2;
        } else {
          // q to fp16 exactly but for elements 2^-24 below the row's largest: the row is scaled
          // by a power of two that brings that one into [1, 2)
          uint2 v[KS];
          float big = 0.f;
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            v[s] = live ? __ldg(reinterpret_cast<const uint2*>(qr + 16 * s + 4 * i4)) : make_uint2(0, 0);
            big = fmaxf(big, fmaxf(fmaxf(fabsf(__uint_as_float(v[s].x << 16)), fabsf(__uint_as_float(v[s].x & 0xffff0000u))),
                                   fmaxf(fabsf(__uint_as_float(v[s].y << 16)), fabsf(__uint_as_float(v[s].y & 0xffff0000u)))));
          }
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const int e = min(max((int)(__float_as_uint(big) >> 23), 2), 252);  // biased exponent
          const float down = __uint_as_float((uint32_t)(254 - e) << 23), up = __uint_as_float((uint32_t)e << 23);
#pragma unroll
          for (int s = 0; s < KS; ++s) {
            qa[s][h] = pack_f16(__uint_as_float(v[s].x << 16) * down, __uint_as_float(v[s].x & 0xffff0000u) * down);
            qa[s][2 + h] = pack_f16(__uint_as_float(v[s].y << 16) * down, __uint_as_float(v[s].y & 0xffff0000u) * down);
          }
          if (h < H) sc[h] = a.scale_log2 * (a.kd ? __ldg(a.kd + hk) : 1.f) * up;
        }
      }
#pragma unroll
      for (int n = 0; n < DN; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
      for (int h = 0; h < H; ++h) m[h] = -INFINITY, l[h] = 0.f;
    }

    cp_wait<kStages - 2>();
    __syncwarp();
    const int key0 = cur.tile * TILE + warp * KEYS;
    if (key0 < cur.len) {
      const uint32_t kb = ring + stage * C::STAGE, vb = kb + KEYS * ROWB;
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = n * 8 + (lane & 7);
        if (!FP8) {
#pragma unroll
          for (int k = 0; k < KS / 2; ++k) {
            uint32_t b[4];
            ldsm4(b, kb + row * ROWB + (((4 * k + (lane >> 3)) ^ swz<CH>(row)) * 16));
            mma16816<false>(s[n], qa[2 * k][0], qa[2 * k][1], qa[2 * k][2], qa[2 * k][3], b[0], b[1]);
            mma16816<false>(s[n], qa[2 * k + 1][0], qa[2 * k + 1][1], qa[2 * k + 1][2], qa[2 * k + 1][3], b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < KS / 4; ++k) {
            uint32_t b[4];
            ldsm4(b, kb + row * ROWB + (((4 * k + (lane >> 3)) ^ swz<CH>(row)) * 16));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma16816<true>(s[n], qa[4 * k + e][0], qa[4 * k + e][1], qa[4 * k + e][2], qa[4 * k + e][3],
                             e4m3x2_f16x2(b[e]), e4m3x2_f16x2(b[e] >> 16));
          }
        }
      }
      // base-2 scores, the last keys masked, the new running max
      const int live = cur.len - key0;
      float mx[H];
#pragma unroll
      for (int h = 0; h < H; ++h) mx[h] = -INFINITY;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& v = s[n][2 * h + e];
            v *= sc[h];
            if (live < KEYS && n * 8 + 2 * i4 + e >= live) v = -INFINITY;
            mx[h] = fmaxf(mx[h], v);
          }
      bool moved = false;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        moved |= mx[h] > m[h];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float mn = fmaxf(m[h], mx[h]);
          const float al = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
          m[h] = mn;
          l[h] *= al;
#pragma unroll
          for (int n = 0; n < DN; ++n) {
            acc[n][2 * h] *= al;
            acc[n][2 * h + 1] *= al;
            if (R8) {  // the low part's rows
              acc[n][2] *= al;
              acc[n][3] *= al;
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float ref = (m[h] == -INFINITY ? 0.f : m[h]) - (FP8 ? kPBias : 0.f);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& v = s[n][2 * h + e];
            v = ex2(v - ref);
            l[h] += v;
          }
      }
      // O += P V, 16 keys at a time
#pragma unroll
      for (int kg = 0; kg < KEYS / 16; ++kg) {
        uint32_t hi[2][2], lo[2][2];  // [row half][keys 0-7 / 8-15 of the group]
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float p0 = s[2 * kg + e][2 * h], p1 = s[2 * kg + e][2 * h + 1];
            if (FP8) {
              hi[h][e] = pack_f16(p0, p1);
              lo[h][e] = 0u;
            } else {
              hi[h][e] = pack_bf16(p0, p1);
              lo[h][e] = pack_bf16(p0 - __uint_as_float(hi[h][e] << 16), p1 - __uint_as_float(hi[h][e] & 0xffff0000u));
            }
          }
        const int row = kg * 16 + (lane & 15);
#pragma unroll
        for (int c = 0; c < CH; c += 2) {
          uint32_t b[4];
          ldsm4t(b, vb + row * ROWB + (((c + (lane >> 4)) ^ swz<CH>(row)) * 16));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!FP8) {
              if (R8) {
                mma16816<false>(acc[c + e], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[2 * e], b[2 * e + 1]);
              } else {
                mma16816<false>(acc[c + e], hi[0][0], hi[H - 1][0], hi[0][1], hi[H - 1][1], b[2 * e], b[2 * e + 1]);
                mma16816<false>(acc[c + e], lo[0][0], lo[H - 1][0], lo[0][1], lo[H - 1][1], b[2 * e], b[2 * e + 1]);
              }
            } else {
              // a 16-byte chunk holds 16 values: its even and its odd ones are one 8-wide tile each
#pragma unroll
              for (int odd = 0; odd < 2; ++odd) {
                const uint32_t sel = odd ? 0x0031u : 0x0020u;
                mma16816<true>(acc[2 * (c + e) + odd], hi[0][0], R8 ? 0u : hi[H - 1][0], hi[0][1],
                               R8 ? 0u : hi[H - 1][1], e4m3x2_f16x2(__byte_perm(b[2 * e], 0, sel)),
                               e4m3x2_f16x2(__byte_perm(b[2 * e + 1], 0, sel)));
              }
            }
          }
        }
      }
    }
    __syncwarp();  // all lanes have read the stage that is filled next
    fetch(stage == 0 ? kStages - 1 : stage - 1);
    --left;

    const bool seg_end = cur.tile + 1 == cur.tiles;
    if (seg_end || left == 0) {  // join the warps, 8 rows at a time
#pragma unroll
      for (int h = 0; h < H; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (i4 == 0) s_m[warp][g8 + 8 * h] = m[h], s_l[warp][g8 + 8 * h] = l[h];
      }
      // through the stage just read, which the next fetch fills only after the last barrier here
      float* join = reinterpret_cast<float*>(smem + stage * C::STAGE);
      constexpr int RS = D + C::PAD, WS = kStages * C::STAGE / 4;
      const bool whole = seg_end && seg_tile0 == 0;
      const int slot = 2 * cta + (seg_tile0 == 0 ? 1 : 0);
      const float vscale = FP8 && a.vd ? __ldg(a.vd + hk) : 1.f;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const int nrows = min(8, rows - 8 * h);
        if (nrows <= 0) break;
        if (g8 < nrows) {
          float* dst = join + warp * WS + g8 * RS;
          if (!FP8) {
#pragma unroll
            for (int n = 0; n < DN; ++n) {
              float2 v = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
              if (R8) v.x += acc[n][2], v.y += acc[n][3];
              *reinterpret_cast<float2*>(dst + n * 8 + 2 * i4) = v;
            }
          } else {
#pragma unroll
            for (int c = 0; c < CH; ++c)
              *reinterpret_cast<float4*>(dst + c * 16 + 4 * i4) =
                  make_float4(acc[2 * c][2 * h], acc[2 * c + 1][2 * h], acc[2 * c][2 * h + 1], acc[2 * c + 1][2 * h + 1]);
          }
        }
        __syncthreads();
        for (int i = tid; i < nrows * (D / 4); i += kWarps * 32) {
          const int row = i / (D / 4), c4 = i % (D / 4);
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][8 * h + row]);
          float L = 0.f;
          float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float mw = s_m[w][8 * h + row];
            const float f = mw == -INFINITY ? (M == -INFINITY ? 1.f : 0.f) : ex2(mw - M);
            const float4 v = *reinterpret_cast<const float4*>(join + w * WS + row * RS + c4 * 4);
            L = fmaf(f, s_l[w][8 * h + row], L);
            o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
          }
          if (whole) {
            write_out<D>(a, cur.t, hk * g + row0 + 8 * h + row, c4, o, M, L, vscale, FP8 ? kPBias : 0.f);
          } else {
            const size_t pr = (size_t)slot * kMaxRows + 8 * h + row;
            *reinterpret_cast<float4*>(part.o + pr * D + c4 * 4) = o;
            if (c4 == 0) part.ml[pr] = make_float2(M, L);
          }
        }
        __syncthreads();
      }
      fresh = true;
    }
    stage = stage == kStages - 1 ? 0 : stage + 1;
    if (left == 0) {
      if (tid == 0) {
        int4 head = make_int4(-1, 0, 0, 0);
        if (!seg_end && seg_tile0 == 0) {  // this CTA holds the first part of a divided segment
          const long long end = last - 1 + (cur.tiles - 1 - cur.tile);  // its last tile
          head = make_int4(cur.t, cur.hm, (int)(((end + 1) * ctas - 1) / total), 0);
        }
        part.head[cta] = head;
      }
    } else {
      cursor_next<TILE>(a, cur, hms);
    }
  }
  cp_wait<0>();
}

// Joins the parts of the segment that begins in CTA `blockIdx.x` of the decode kernel (if one
// does): a thread per (row, 4 elements), the parts in order with a running max.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) fa_paged_join_kernel(const DecodeArgs a) {
  const int cta = blockIdx.x;
  const Part part = part_of(a.workspace, gridDim.x);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 head = part.head[cta];
  if (head.x < 0) return;
  const int g = a.Hq / a.Hk, mt = (g + kMaxRows - 1) / kMaxRows;
  const int hk = head.y / mt, row0 = (head.y - hk * mt) * kMaxRows, rows = min(kMaxRows, g - row0);
  const float vscale = FP8 && a.vd ? __ldg(a.vd + hk) : 1.f;
  for (int i = threadIdx.x; i < rows * (D / 4); i += blockDim.x) {
    const int row = i / (D / 4), c4 = i % (D / 4);
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 8
    for (int c = cta; c <= head.z; ++c) {
      const size_t pr = ((size_t)2 * c + (c == cta ? 1 : 0)) * kMaxRows + row;
      const float2 ml = part.ml[pr];
      const float4 v = *reinterpret_cast<const float4*>(part.o + pr * D + c4 * 4);
      const float mn = fmaxf(M, ml.x);
      const float f0 = M == -INFINITY ? 0.f : ex2(M - mn);
      const float f1 = ml.x == -INFINITY ? (mn == -INFINITY ? 1.f : 0.f) : ex2(ml.x - mn);
      L = L * f0 + ml.y * f1;
      o.x = o.x * f0 + v.x * f1, o.y = o.y * f0 + v.y * f1, o.z = o.z * f0 + v.z * f1, o.w = o.w * f0 + v.w * f1;
      M = mn;
    }
    write_out<D>(a, head.x, hk * g + row0 + row, c4, o, M, L, vscale, FP8 ? kPBias : 0.f);
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

int decode_ctas() { return 2 * sm_count(); }

template <int D, bool FP8, bool R8>
cudaError_t launch_decode_t(const DecodeArgs& a, cudaStream_t stream) {
  using C = DecCfg<D, FP8>;
  static_assert(2 * (C::SMEM + 2048) <= 228 * 1024, "two CTAs per SM");
  static bool attr_set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(fa_paged_decode_kernel<D, FP8, R8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  const int ctas = decode_ctas();
  fa_paged_decode_kernel<D, FP8, R8><<<ctas, kWarps * 32, C::SMEM, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_join_kernel<D, FP8>, a);
}

}  // namespace

cudaError_t launch_paged_plan(const PlanArgs& a, cudaStream_t stream) {
  const int smem = (3 * a.R + 1) * 4;
  if (smem > 48 * 1024) {
    static bool attr_set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
      e = cudaFuncSetAttribute(fa_paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (3 * FA_PLAN_MAX_REQUESTS + 1) * 4);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
  }
  const long long share = (long long)kPlanThreads * kPlanTokensPerThread;
  const int ctas = (int)std::min<long long>(kPlanMaxCtas, std::max<long long>(1, (a.max_tokens + share - 1) / share));
  const int need = std::max(a.R, ctas > 1 ? kPlanThreads : a.max_tokens);
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
  (void)T, (void)Hq, (void)Hk;
  const int ctas = decode_ctas();
  return part_head_bytes(ctas) + part_ml_bytes(ctas) + (size_t)ctas * 2 * kMaxRows * d * 4;
}

cudaError_t launch_paged_decode(int d, bool fp8, const DecodeArgs& a, cudaStream_t stream) {
  const bool r8 = a.Hq / a.Hk <= 8;
  if (d == 64) {
    if (fp8) return r8 ? launch_decode_t<64, true, true>(a, stream) : launch_decode_t<64, true, false>(a, stream);
    return r8 ? launch_decode_t<64, false, true>(a, stream) : launch_decode_t<64, false, false>(a, stream);
  }
  if (fp8) return r8 ? launch_decode_t<128, true, true>(a, stream) : launch_decode_t<128, true, false>(a, stream);
  return r8 ? launch_decode_t<128, false, true>(a, stream) : launch_decode_t<128, false, false>(a, stream);
}

}  // namespace fa
