// fa_norm_rope.cu - RMS norm of every query and key head with the position rotation in the same
// pass: the training form (token-major q, k in, [B,H,N,d] out), its gradient, and the serving
// form that writes K and V into the paged cache.
//
// Per row x of d values, weight w, position p:
//     r = 1 / sqrt(mean(x^2) + eps),  y = x r w,
//     out_a = y_a cos_i - y_b sin_i,  out_b = y_b cos_i + y_a sin_i   for each rotated pair (a, b),
// all in fp32 from the bf16 inputs, rounded once at the store.  Gradient, g = d out:
//     dy = R^T g,  dw = sum over rows of dy (x r),  u = dy w,  dx = r (u - xh mean(u xh)),  xh = x r,
// with r recomputed from x (the row is read for xh anyway, so a saved r would only add traffic).
//
// Layout: a lane holds 16 elements of a row, two 16-byte chunks that a rotation maps into each
// other (halves: chunk j of the first half of the rotated elements and of the second), so the
// rotation needs no exchange between lanes; a row is d/16 lanes, and a warp holds 4 (d = 128) or 8
// (d = 64) neighbouring tokens at a time.  A lane keeps its token's cos and sin in registers and
// walks over heads: the table row, as long as one row of data in fp32, is then read once per token
// instead of once per head, and the stores of neighbouring tokens adjoin.
// Rows come through a ring in shared memory that a lane fills (16-byte asynchronous copies) and
// reads for itself: bytes in flight then cost no registers, which hold too few of them at the
// occupancy that the arithmetic leaves, and no barrier is needed.
//
// Bound by HBM.  On a B200, replayed from a graph: B=1 N=16384, 64 heads, d=128 takes 87 us (6.2 TB/s,
// 0.95 of a copy; rows loaded to registers, two to four ahead, took 115 to 148), its gradient at B=2
// N=4096, 32 heads 37.3 us (5.5 TB/s, of which 2 us add up the weights' gradients), the cache form
// with 4099 tokens of 40 heads to E4M3 15.2 us (5.4 TB/s, from L2 in part: one wave of warps, whose slots,
// positions and table rows come one after the other), 8 tokens 3.0 us.
#include "fa_internal.cuh"
#include "sm100_ptx.cuh"

#include <algorithm>
#include <climits>

namespace fa {

namespace {

using namespace ptx;

constexpr int kThreads = 128;
constexpr int kDepth = 6;     // rows of the forward's ring
constexpr int kBwdDepth = 3;  // rows of x, and of g, of the backward's

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// Sum over the LPR lanes of a row (LPR a power of two, rows aligned to LPR lanes).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Arithmetic on a lane's chunks goes two elements an instruction (fp32 pairs).
__device__ __forceinline__ uint64_t pair(const float (&x)[8], int i) { return f2_pack(x[2 * i], x[2 * i + 1]); }
__device__ __forceinline__ void set_pair(float (&x)[8], int i, uint64_t v) { f2_unpack(v, x[2 * i], x[2 * i + 1]); }
// x *= y f
__device__ __forceinline__ void scale8(float (&x)[8], const float (&y)[8], float f) {
  const uint64_t ff = f2_pack(f, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) set_pair(x, i, f2_mul(pair(x, i), f2_mul(pair(y, i), ff)));
}
__device__ __forceinline__ void scale8(float (&x)[8], float f) {
  const uint64_t ff = f2_pack(f, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) set_pair(x, i, f2_mul(pair(x, i), ff));
}
__device__ __forceinline__ void mul8(float (&x)[8], const float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) set_pair(x, i, f2_mul(pair(x, i), pair(y, i)));
}
// acc + sum of x y, the even elements' and the odd ones' apart
__device__ __forceinline__ uint64_t dot8(const float (&x)[8], const float (&y)[8], uint64_t acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc = f2_fma(pair(x, i), pair(y, i), acc);
  return acc;
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a + b;
}

// One lane's share of a token's rotation: its chunks a and b (8 elements each), whether they are
// rotated, and the angles.  Halves: pair e is (a_e, b_e) with c[e], s[e]; both chunks are rotated or
// neither is.  Interleaved: pair i < 4 is (a_2i, a_2i+1) with c[i], s[i], and b's have c[4 + i], s[4 + i].
template <int D, bool INTER>
struct Rotation {
  static constexpr int LPR = D / 16;
  float c[8], s[8], ns[8];  // ns = -s
  int ca, cb;
  bool on_a, on_b;

  __device__ __forceinline__ Rotation(int rot, int j) {
    if (INTER) {
      ca = j, cb = j + LPR;
      on_a = 8 * ca < rot, on_b = 8 * cb < rot;
    } else {
      const int hl = rot >> 4;
      on_a = on_b = j < hl;
      ca = on_a ? j : hl + j;  // the rest of the chunks, from 2 hl on, halved among the other lanes
      cb = on_a ? j + hl : LPR + j;
    }
  }
  __device__ __forceinline__ void load(const float* __restrict__ rope, int rot, int pos) {
    const float* row = rope + (size_t)pos * rot;
    const int half = rot >> 1;
    if (INTER) {
      if (on_a) load4(0, row + 4 * ca, half);
      if (on_b) load4(4, row + 4 * cb, half);
    } else if (on_a) {
      load4(0, row + 8 * ca, half);
      load4(4, row + 8 * ca + 4, half);
    }
  }
  // a, b <- R (a, b), or R^T (a, b) with BACK (the rotation by the negative angle)
  template <bool BACK>
  __device__ __forceinline__ void apply(float (&a)[8], float (&b)[8]) const {
    if (INTER) {
      if (on_a) inside<BACK>(a, 0);
      if (on_b) inside<BACK>(b, 4);
    } else if (on_a) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t x = pair(a, i), y = pair(b, i);
        if (BACK) {  // (the backward has no registers for ns)
          set_pair(a, i, f2_fma(x, pair(c, i), f2_mul(y, pair(s, i))));
          set_pair(b, i, f2_fma(f2_mul(x, pair(s, i)), f2_pack(-1.f, -1.f), f2_mul(y, pair(c, i))));
        } else {
          set_pair(a, i, f2_fma(x, pair(c, i), f2_mul(y, pair(ns, i))));
          set_pair(b, i, f2_fma(y, pair(c, i), f2_mul(x, pair(s, i))));
        }
      }
    }
  }

 private:
  __device__ __forceinline__ void load4(int i, const float* p, int half) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p + half));
    c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
    s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
#pragma unroll
    for (int e = i; e < i + 4; ++e) ns[e] = -s[e];
  }
  template <bool BACK>
  __device__ __forceinline__ void inside(float (&x)[8], int i0) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1], sn = BACK ? -s[i0 + i] : s[i0 + i];
      x[2 * i] = a * c[i0 + i] - b * sn;
      x[2 * i + 1] = b * c[i0 + i] + a * sn;
    }
  }
};

// A lane's two chunks of a row, as stored.
struct Raw {
  uint4 a, b;
};
// A lane's ring: slot i holds chunk a at i * 1024 and chunk b 512 bytes behind it (a warp's lanes
// side by side).
__device__ __forceinline__ void copy_row(uint32_t slot, const __nv_bfloat16* p, int ca, int cb) {
  cp_async16(slot, p + 8 * ca);
  cp_async16(slot + 512, p + 8 * cb);
}
__device__ __forceinline__ Raw take_row(uint32_t slot) {
  Raw r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.a.x), "=r"(r.a.y), "=r"(r.a.z), "=r"(r.a.w) : "r"(slot) : "memory");
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.b.x), "=r"(r.b.y), "=r"(r.b.z), "=r"(r.b.w) : "r"(slot + 512) : "memory");
  return r;
}
__device__ __forceinline__ void st_row(__nv_bfloat16* p, int ca, int cb, const uint4& a, const uint4& b) {
  *reinterpret_cast<uint4*>(p + 8 * ca) = a;
  *reinterpret_cast<uint4*>(p + 8 * cb) = b;
}
__device__ __forceinline__ Raw ld_weight(const __nv_bfloat16* w, int ca, int cb) {
  const uint4 one = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  if (!w) return {one, one};
  return {__ldg(reinterpret_cast<const uint4*>(w) + ca), __ldg(reinterpret_cast<const uint4*>(w) + cb)};
}
// 1 / sqrt(mean of the row's squares + eps)
template <int D>
__device__ __forceinline__ float inv_rms(const float (&a)[8], const float (&b)[8], float eps) {
  return rsqrtf(row_sum<D / 16>(sum2(dot8(b, b, dot8(a, a, 0)))) * (1.f / D) + eps);
}
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8]) {
  return make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7]));
}

// a, b over f, such that the rounding to E4M3 that follows gives what it gives for the fp32 quotients.
// The product with 1 / f is within 2.5 units in the last place of the quotient, and E4M3's rounding
// borders (midpoints of its values, the subnormal ones too) have 19 zero bits at the end in fp32: a
// product that is more than 3 units from such a number rounds alike.  A lane with another one, or
// where 1 / f is not a normal number of usual size, divides.  (16 divisions for each K and V row took
// 2.6 of 18.7 us for 4099 tokens of 32 + 2 x 4 heads.)
__device__ __forceinline__ void divide(float (&a)[8], float (&b)[8], float f) {
  const float inv = 1.f / f;
  float qa[8], qb[8];
  uint32_t least = 0xffffffffu;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    qa[e] = a[e] * inv, qb[e] = b[e] * inv;
    least = min(least, min((__float_as_uint(qa[e]) + 3) & 0x7ffffu, (__float_as_uint(qb[e]) + 3) & 0x7ffffu));
  }
  const bool exact = (__float_as_uint(f) & 0x7fffffu) == 0;  // a power of two: so is the product
  const bool usual = fabsf(f) > 1e-30f && fabsf(f) < 1e30f;
  if (__builtin_expect(usual && (exact || least >= 7), 1)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = qa[e], b[e] = qb[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] /= f, b[e] /= f;
  }
}

enum Mode { kTrain, kCacheBf16, kCacheE4m3 };

// Forward.  A run of D/16 lanes per (token, run of heads_per_unit heads); heads count q's, then
// k's, then (serving) v's, which are copied unchanged.
template <int D, bool INTER, Mode MODE>
__global__ void __launch_bounds__(kThreads, 4) fa_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 16, G = 32 / LPR;
  __shared__ __align__(16) uint8_t ring[kThreads / 32 * kDepth * 1024];
  const int lane = threadIdx.x & 31, j = lane % LPR;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long run = quotient(unit, a.chunks);
  const long long tok = run * G + lane / LPR;
  const int h0 = (int)(unit - run * a.chunks) * a.heads_per_unit;
  const int heads = a.Hq + a.Hk * (MODE == kTrain ? 1 : 2);
  const int h1 = min(heads, h0 + a.heads_per_unit);
  const bool live = tok < (long long)a.B * a.N;
  const int b = MODE == kTrain && live ? (int)quotient(tok, a.N) : 0, n = live ? (int)(tok - (long long)b * a.N) : 0;
  Rotation<D, INTER> t(a.rot, j);

  // What the token needs; `go`: it is computed.
  bool go = live;
  long long slot = 0;
  int pos = n;
  if (MODE != kTrain) {
    slot = live ? a.slots[tok] : -1;
    go = slot >= 0;
  }
  if (a.rot > 0 && a.positions && live) pos = a.positions[(long long)b * a.pos_sb + n];

  // Rows on their way: the next head, where it is, and the last of its kind (0 q, 1 k, 2 v).
  const uint32_t slots = smem_u32(ring) + (threadIdx.x >> 5) * (kDepth * 1024) + lane * 16;
  auto kind_of = [&](int h) { return h < a.Hq ? 0 : MODE == kTrain || h < a.Hq + a.Hk ? 1 : 2; };
  auto first_of = [&](int kind) { return kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + a.Hk; };
  auto end_of = [&](int kind) { return min(h1, first_of(kind) + (kind == 0 ? a.Hq : a.Hk)); };
  int fh = h0, fend = h0;
  const __nv_bfloat16* fp = nullptr;
  long long fstep = 0;
  auto fetch = [&](int i) {
    if (fh < h1) {
      if (fh == fend) {
        const int kind = kind_of(fh);
        fend = end_of(kind);
        fstep = kind == 0 ? a.q_sh : kind == 1 ? a.k_sh : a.v_sh;
        fp = (kind == 0 ? a.q + b * a.q_sb + n * a.q_sn : kind == 1 ? a.k + b * a.k_sb + n * a.k_sn : a.v + n * a.v_sn) +
             (fh - first_of(kind)) * fstep;
      }
      if (live) copy_row(slots + i * 1024, fp, t.ca, t.cb);
      fp += fstep;
      ++fh;
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) fetch(i);

  const bool bad = (a.rot > 0 && (pos < 0 || pos >= a.rope_rows)) ||
                   (MODE != kTrain && slot >= (long long)a.num_pages * a.page_size);
  if (go && bad) {
    if (j == 0) atomicOr(a.status, FA_DEV_BOUNDS);
    go = false;
  }
  if (go) t.load(a.rope, a.rot, pos);
  long long cache_off = 0;
  if (MODE != kTrain && go) {
    const long long page = quotient(slot, a.page_size);
    cache_off = page * a.c_sp + (slot - page * a.page_size) * a.c_st;
  }
  int slot_i = 0;
  for (int hh = h0; hh < h1;) {
    const int kind = kind_of(hh), end = end_of(kind);
    int h = hh - first_of(kind);
    float wa[8], wb[8];
    if (MODE == kTrain || kind < 2) {
      const Raw w = ld_weight(kind == 0 ? a.wq : a.wk, t.ca, t.cb);
      unpack8(w.a, wa);
      unpack8(w.b, wb);
    }
    // the head's row in its output, and from a head to the next, in bytes
    char* dst;
    long long step;
    if (MODE == kTrain) {
      dst = reinterpret_cast<char*>((kind == 0 ? a.q_out + (((long long)b * a.Hq + h) * a.N + n) * D
                                               : a.k_out + (((long long)b * a.Hk + h) * a.N + n) * D));
      step = (long long)a.N * D * 2;
    } else if (kind == 0) {
      dst = reinterpret_cast<char*>(a.q_out + (tok * a.Hq + h) * D), step = D * 2;
    } else {
      constexpr int size = MODE == kCacheBf16 ? 2 : 1;
      dst = static_cast<char*>(kind == 2 ? a.v_cache : a.k_cache) + (cache_off + h * a.c_sh) * size, step = a.c_sh * size;
    }
    for (; hh < end; ++hh, ++h, dst += step) {
      cp_wait<kDepth - 1>();
      const Raw raw = take_row(slots + slot_i * 1024);
      float ya[8], yb[8];
      unpack8(raw.a, ya);
      unpack8(raw.b, yb);
      fetch(slot_i);
      slot_i = slot_i == kDepth - 1 ? 0 : slot_i + 1;
      if (MODE == kTrain || kind < 2) {
        const float r = inv_rms<D>(ya, yb, a.eps);
        scale8(ya, wa, r);
        scale8(yb, wb, r);
        t.template apply<false>(ya, yb);
      }
      if (!go) continue;
      if (MODE == kTrain || kind == 0) {
        st_row(reinterpret_cast<__nv_bfloat16*>(dst), t.ca, t.cb, pack8(ya), pack8(yb));
      } else if (MODE == kCacheBf16) {
        st_row(reinterpret_cast<__nv_bfloat16*>(dst), t.ca, t.cb, kind == 2 ? raw.a : pack8(ya),
               kind == 2 ? raw.b : pack8(yb));
      } else {
        // the value over its head's factor, rounded once to E4M3 (saturating)
        const float* ds = kind == 2 ? a.v_descale : a.k_descale;
        if (ds) divide(ya, yb, __ldg(ds + h));
        *reinterpret_cast<uint2*>(dst + 8 * t.ca) = pack8_e4m3(ya);
        *reinterpret_cast<uint2*>(dst + 8 * t.cb) = pack8_e4m3(yb);
      }
    }
  }
  cp_wait<0>();
}

// Backward.  The first blocks_q blocks walk q's units, the others k's, with a grid stride; a lane
// keeps the weight gradients of its 16 elements in registers over all its rows, the block adds
// them up in shared memory and writes one partial row; fa_norm_rope_dw_kernel adds the partials
// in block order.  No atomics: equal calls give equal bits.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 4) fa_norm_rope_bwd_kernel(const NormRopeBwdArgs a) {
  constexpr int LPR = D / 16, G = 32 / LPR, W = kThreads / 32;
  __shared__ __align__(16) uint8_t ring[W * kBwdDepth * 2048];
  static_assert(sizeof(ring) >= W * D * 4, "the ring holds the block's sums at the end");
  const int lane = threadIdx.x & 31, j = lane % LPR, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  const bool is_q = (int)blockIdx.x < a.blocks_q;
  const int block = is_q ? blockIdx.x : blockIdx.x - a.blocks_q;
  const int blocks = is_q ? a.blocks_q : gridDim.x - a.blocks_q;
  const int H = is_q ? a.Hq : a.Hk, per = is_q ? a.per_q : a.per_k, chunks = (H + per - 1) / per;
  const long long tokens = (long long)a.B * a.N, units = (tokens + G - 1) / G * chunks;
  const __nv_bfloat16* const xs = is_q ? a.q : a.k;
  const __nv_bfloat16* const gs = is_q ? a.gq : a.gk;
  __nv_bfloat16* const dxs = is_q ? a.dq : a.dk;
  const long long x_sh = is_q ? a.q_sh : a.k_sh, dx_sh = is_q ? a.dq_sh : a.dk_sh, g_sh = (long long)a.N * D;
  Rotation<D, INTER> t(a.rot, j);
  const Raw w = ld_weight(is_q ? a.wq : a.wk, t.ca, t.cb);
  float dwa[8], dwb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwa[e] = dwb[e] = 0.f;

  // A place in the warp's line of units: the lane's token, a head, and where its rows are.
  struct Place {
    long long unit, tok;
    const __nv_bfloat16 *x, *g;
    int h, h1, b, n;
  };
  auto enter = [&](Place& p) {  // the first head of p.unit
    const long long run = quotient(p.unit, chunks);
    p.tok = run * G + lane / LPR;
    p.h = (int)(p.unit - run * chunks) * per;
    p.h1 = min(H, p.h + per);
    if (p.tok < tokens) {
      p.b = (int)quotient(p.tok, a.N), p.n = (int)(p.tok - (long long)p.b * a.N);
      p.x = xs + p.b * (is_q ? a.q_sb : a.k_sb) + p.n * (is_q ? a.q_sn : a.k_sn) + p.h * x_sh;
      p.g = gs + (((long long)p.b * H + p.h) * a.N + p.n) * D;
    }
  };
  const uint32_t slots = smem_u32(ring) + warp * (kBwdDepth * 2048) + lane * 16;
  Place ahead;
  ahead.unit = (long long)block * W + warp;
  if (ahead.unit < units) enter(ahead);
  auto fetch = [&](int i) {  // copies the rows of `ahead` and moves it on
    if (ahead.unit < units) {
      if (ahead.tok < tokens) {
        copy_row(slots + i * 2048, ahead.x, t.ca, t.cb);
        copy_row(slots + i * 2048 + 1024, ahead.g, t.ca, t.cb);
      }
      ahead.x += x_sh, ahead.g += g_sh;
      if (++ahead.h == ahead.h1) {
        ahead.unit += (long long)blocks * W;
        if (ahead.unit < units) enter(ahead);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kBwdDepth; ++i) fetch(i);

  int slot_i = 0;
  for (long long unit = (long long)block * W + warp; unit < units; unit += (long long)blocks * W) {
    const long long run = quotient(unit, chunks);
    const long long tok = run * G + lane / LPR;
    const int h0 = (int)(unit - run * chunks) * per, h1 = min(H, h0 + per);
    bool go = tok < tokens;
    const int b = go ? (int)quotient(tok, a.N) : 0, n = go ? (int)(tok - (long long)b * a.N) : 0;
    int pos = n;
    if (a.rot > 0 && a.positions && go) pos = a.positions[(long long)b * a.pos_sb + n];
    if (go && a.rot > 0 && (pos < 0 || pos >= a.rope_rows)) {
      if (j == 0) atomicOr(a.status, FA_DEV_BOUNDS);
      go = false;
    }
    if (go) t.load(a.rope, a.rot, pos);
    __nv_bfloat16* dst = dxs + b * (is_q ? a.dq_sb : a.dk_sb) + n * (is_q ? a.dq_sn : a.dk_sn) + h0 * dx_sh;
    for (int h = h0; h < h1; ++h) {
      cp_wait<kBwdDepth - 1>();
      float xa[8], xb[8], ga[8], gb[8];
      {
        const Raw x = take_row(slots + slot_i * 2048), g = take_row(slots + slot_i * 2048 + 1024);
        unpack8(x.a, xa);
        unpack8(x.b, xb);
        unpack8(g.a, ga);
        unpack8(g.b, gb);
      }
      fetch(slot_i);
      slot_i = slot_i == kBwdDepth - 1 ? 0 : slot_i + 1;
      t.template apply<true>(ga, gb);
      const float r = inv_rms<D>(xa, xb, a.eps);
      float wa[8], wb[8];
      unpack8(w.a, wa);
      unpack8(w.b, wb);
      scale8(xa, r);
      scale8(xb, r);
      if (go) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          set_pair(dwa, i, f2_fma(pair(ga, i), pair(xa, i), pair(dwa, i)));
          set_pair(dwb, i, f2_fma(pair(gb, i), pair(xb, i), pair(dwb, i)));
        }
      }
      mul8(ga, wa);
      mul8(gb, wb);
      const float c = row_sum<LPR>(sum2(dot8(gb, xb, dot8(ga, xa, 0)))) * (1.f / D);
      const uint64_t rr = f2_pack(r, r), nc = f2_pack(-c, -c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        set_pair(ga, i, f2_mul(rr, f2_fma(pair(xa, i), nc, pair(ga, i))));
        set_pair(gb, i, f2_mul(rr, f2_fma(pair(xb, i), nc, pair(gb, i))));
      }
      if (go) st_row(dst, t.ca, t.cb, pack8(ga), pack8(gb));
      dst += dx_sh;
    }
  }
  cp_wait<0>();
  __syncthreads();
  float(*red)[D] = reinterpret_cast<float(*)[D]>(ring);
  // the warp's row groups, then the block's warps
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      dwa[e] += __shfl_xor_sync(0xffffffffu, dwa[e], o);
      dwb[e] += __shfl_xor_sync(0xffffffffu, dwb[e], o);
    }
    if (lane < LPR) red[warp][8 * t.ca + e] = dwa[e], red[warp][8 * t.cb + e] = dwb[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < W; ++v) s += red[v][i];
    a.partial[(size_t)blockIdx.x * D + i] = s;
  }
}

// dw[i] = sum over the blocks of its kind of partial[block][i], 32 columns per block, in a fixed
// order: blockIdx.x is the columns, blockIdx.y 0 for q, 1 for k.  A thread's share of 592 partials is
// two batches of loads: latency is all there is to this kernel (2 us behind the first one's end).
constexpr int kDwBatch = 10;
__global__ void __launch_bounds__(1024) fa_norm_rope_dw_kernel(const float* partial, int blocks_q, int blocks, int d,
                                                               float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float* const out = blockIdx.y == 0 ? dwq : dwk;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!out) return;
  const int end = blockIdx.y == 0 ? blocks_q : blocks;
  float s = 0.f;
  for (int r0 = (blockIdx.y == 0 ? 0 : blocks_q) + y; r0 < end; r0 += 32 * kDwBatch) {
    float v[kDwBatch];
#pragma unroll
    for (int i = 0; i < kDwBatch; ++i) v[i] = partial[(size_t)min(r0 + 32 * i, end - 1) * d + col];
#pragma unroll
    for (int i = 0; i < kDwBatch; ++i) s += r0 + 32 * i < end ? v[i] : 0.f;
  }
  red[y][c] = s;
  __syncthreads();
  float v = red[c][y];  // warp y now holds column y's 32 sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (c == 0) out[blockIdx.x * 32 + y] = v;
}

// Heads per run of lanes.  With few waves of warps, the number of waves counts (a wave of `per` heads
// costs about per + kStart heads: slots, positions and table rows arrive one after the other);
// with many, kMaxHeads at most lets the blocks even out over the SMs: at 16384 tokens of 64 heads
// 16 take 88 us, 32 take 94 and 8 take 97; at 4192 tokens of 40 heads, where 10 are 1.8 waves, 20
// are one.
constexpr int kMaxHeads = 16, kStart = 6, kWarpSlots = 148 * 16;
int heads_per_unit(long long token_runs, int heads, int slots) {
  const int least = (heads + kMaxHeads - 1) / kMaxHeads, most = (heads + least - 1) / least;  // runs of one length
  const long long units = token_runs * least;
  if (units >= 4LL * slots) return most;
  int best = most;
  long long cost = (units + slots - 1) / slots * (most + kStart);
  for (int waves = 1; waves <= 4; ++waves) {
    const long long chunks = std::min<long long>(heads, (long long)waves * slots / token_runs);
    if (chunks < 1) continue;
    const int per = (int)((heads + chunks - 1) / chunks);
    const long long n = token_runs * ((heads + per - 1) / per);
    const long long c = (n + slots - 1) / slots * (per + kStart);
    if (c < cost) cost = c, best = per;
  }
  return best;
}

long long token_runs(long long tokens, int d) { return (tokens + 32 / (d / 16) - 1) / (32 / (d / 16)); }

}  // namespace

// Blocks of the backward kernel: four per SM and no more than there are units.  Warps are shared out
// between q and k by what their units cost (heads, and about kUnitStart more: positions and the
// table's row come first), then k's are set to whole rounds over its units.  Measured against shares
// by heads alone: B=4 N=6900, 16 + 1 heads, d=64: 53 -> 38 us; one number of heads per unit for both,
// the larger share's: B=4 N=1017, 32 + 8 heads: 31 -> 25 us.
NormRopeBwdPlan norm_rope_bwd_plan(long long tokens, int Hq, int Hk, int d) {
  constexpr int all = kNormRopeBwdBlocks, W = kThreads / 32, kUnitStart = 3;
  const long long runs = token_runs(tokens, d);
  auto per = [&](int H) {
    return H == 0 ? 1 : heads_per_unit(runs, H, std::max<long long>(W, (long long)kWarpSlots * H / (Hq + Hk)));
  };
  NormRopeBwdPlan r = {per(Hq), per(Hk), 0, 0};
  const long long uq = runs * ((Hq + r.per_q - 1) / r.per_q), uk = runs * ((Hk + r.per_k - 1) / r.per_k);
  auto blocks = [&](long long warps) { return (int)std::min<long long>(all, (warps + W - 1) / W); };
  const double cq = (double)runs * Hq + (double)kUnitStart * uq, ck = (double)runs * Hk + (double)kUnitStart * uk;
  if (Hq == 0 || Hk == 0) {
    r.q = blocks(uq), r.k = blocks(uk);
    return r;
  }
  const double share = std::max(1.0, all * W * ck / (cq + ck));  // k's warps
  const long long rounds = std::max(1LL, (long long)(uk / share + 0.5));
  r.k = std::min(blocks((uk + rounds - 1) / rounds), all - 1);
  r.q = std::min(blocks(uq), all - r.k);
  return r;
}

cudaError_t launch_norm_rope(int d, bool interleaved, int mode, NormRopeArgs a, cudaStream_t stream) {
  const int heads = a.Hq + a.Hk * (mode == kTrain ? 1 : 2);
  const long long runs = token_runs((long long)a.B * a.N, d);
  a.heads_per_unit = heads_per_unit(runs, heads, kWarpSlots);
  a.chunks = (heads + a.heads_per_unit - 1) / a.heads_per_unit;
  const long long blocks = (runs * a.chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
#define FA_NR(DD, II, MM) fa_norm_rope_kernel<DD, II, MM><<<(unsigned)blocks, kThreads, 0, stream>>>(a)
#define FA_NR_M(DD, II)                                        \
  do {                                                         \
    if (mode == kTrain) FA_NR(DD, II, kTrain);                 \
    else if (mode == kCacheBf16) FA_NR(DD, II, kCacheBf16);    \
    else FA_NR(DD, II, kCacheE4m3);                            \
  } while (0)
  if (d == 64) {
    if (interleaved) FA_NR_M(64, true);
    else FA_NR_M(64, false);
  } else {
    if (interleaved) FA_NR_M(128, true);
    else FA_NR_M(128, false);
  }
#undef FA_NR_M
#undef FA_NR
  return cudaGetLastError();
}

cudaError_t launch_norm_rope_bwd(int d, bool interleaved, NormRopeBwdArgs a, const NormRopeBwdPlan& r, float* dwq,
                                 float* dwk, cudaStream_t stream) {
  a.per_q = r.per_q, a.per_k = r.per_k, a.blocks_q = r.q;
  const int blocks = r.q + r.k;
#define FA_NRB(DD, II) fa_norm_rope_bwd_kernel<DD, II><<<blocks, kThreads, 0, stream>>>(a)
  if (d == 64) {
    if (interleaved) FA_NRB(64, true);
    else FA_NRB(64, false);
  } else {
    if (interleaved) FA_NRB(128, true);
    else FA_NRB(128, false);
  }
#undef FA_NRB
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!dwq && !dwk)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d / 32, 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};  // its blocks may be in place before the partials are
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_norm_rope_dw_kernel, (const float*)a.partial, r.q, blocks, d, dwq, dwk);
}

}  // namespace fa
