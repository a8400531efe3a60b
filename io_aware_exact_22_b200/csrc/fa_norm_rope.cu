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
// Layout: a lane holds 8 consecutive elements of a row (one 16-byte access), so a row is d/8
// lanes and a warp holds 2 (d = 128) or 4 (d = 64) rows at a time.  A warp keeps one token's cos
// and sin in registers and walks over its heads: the table row, as long as one row of data in
// fp32, is then read once per token instead of once per head.
#include "fa_internal.cuh"
#include "sm100_ptx.cuh"

#include <algorithm>
#include <climits>

namespace fa {

namespace {

using namespace ptx;

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
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

// One lane's share of a token's rotation.  Halves: element i of the first `rot` pairs with
// i +- rot/2, which lies in another lane (`src`); the sign of the sine is folded into s.
// Interleaved: pairs (2i, 2i+1) lie in the lane itself and use c[0..3], s[0..3].
struct Rotation {
  float c[8], s[8];
  int src;
  bool on;  // the lane's elements are rotated
};

template <bool INTER>
__device__ __forceinline__ void load_rotation(Rotation& t, const float* __restrict__ rope, int rot, int pos, int j) {
  const int half = rot >> 1, hl = rot >> 4;
  t.src = j;
  t.on = 8 * j < rot;
#pragma unroll
  for (int e = 0; e < 8; ++e) t.c[e] = 1.f, t.s[e] = 0.f;
  if (!t.on) return;
  const float* row = rope + (size_t)pos * rot;
  if (INTER) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * j));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + 4 * j));
    t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
    t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
  } else {
    const bool first = j < hl;
    const float* cp = row + 8 * (first ? j : j - hl);
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(cp)), c1 = __ldg(reinterpret_cast<const float4*>(cp + 4));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(cp + half)),
                 s1 = __ldg(reinterpret_cast<const float4*>(cp + half + 4));
    const float sg = first ? -1.f : 1.f;
    t.c[0] = c0.x, t.c[1] = c0.y, t.c[2] = c0.z, t.c[3] = c0.w;
    t.c[4] = c1.x, t.c[5] = c1.y, t.c[6] = c1.z, t.c[7] = c1.w;
    t.s[0] = sg * s0.x, t.s[1] = sg * s0.y, t.s[2] = sg * s0.z, t.s[3] = sg * s0.w;
    t.s[4] = sg * s1.x, t.s[5] = sg * s1.y, t.s[6] = sg * s1.z, t.s[7] = sg * s1.w;
    t.src = first ? j + hl : j - hl;
  }
}

// y <- R y, or R^T y with BACK (the rotation by the negative angle).
template <int LPR, bool INTER, bool BACK>
__device__ __forceinline__ void rotate(float (&y)[8], const Rotation& t) {
  if (INTER) {
    if (!t.on) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1], s = BACK ? -t.s[i] : t.s[i];
      y[2 * i] = a * t.c[i] - b * s;
      y[2 * i + 1] = b * t.c[i] + a * s;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_sync(0xffffffffu, y[e], t.src, LPR);
      const float v = y[e] * t.c[e] + (BACK ? -o : o) * t.s[e];
      y[e] = t.on ? v : y[e];
    }
  }
}

enum Mode { kTrain, kCacheBf16, kCacheE4m3 };

// Forward.  One warp per (token, run of heads_per_warp heads); heads count q's, then k's, then
// (serving) v's, which are copied unchanged.
template <int D, bool INTER, Mode MODE, int U>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_kernel(const NormRopeArgs a) {
  constexpr int LPR = D / 8, G = 32 / LPR;
  const int lane = threadIdx.x & 31, j = lane % LPR, grp = lane / LPR;
  const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long tok = unit / a.chunks;
  if (tok >= (long long)a.B * a.N) return;
  const int h0 = (int)(unit - tok * a.chunks) * a.heads_per_warp;
  const int heads = a.Hq + a.Hk * (MODE == kTrain ? 1 : 2);
  const int h1 = min(heads, h0 + a.heads_per_warp);
  const int b = (int)(tok / a.N), n = (int)(tok - (long long)b * a.N);

  long long cache_off = 0;
  if (MODE != kTrain) {
    const long long slot = a.slots[tok];
    if (slot < 0) return;
    if (slot >= (long long)a.num_pages * a.page_size) {
      if (lane == 0) atomicOr(a.status, FA_DEV_BOUNDS);
      return;
    }
    const int page = (int)(slot / a.page_size);
    cache_off = page * a.c_sp + (slot - (long long)page * a.page_size) * a.c_st;
  }
  Rotation t;
  int pos = n;
  if (a.rot > 0) {
    if (a.positions) pos = a.positions[(long long)b * a.pos_sb + n];
    if (pos < 0 || pos >= a.rope_rows) {
      if (lane == 0) atomicOr(a.status, FA_DEV_BOUNDS);
      return;
    }
  }
  load_rotation<INTER>(t, a.rope, a.rot, pos, j);
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint4 wq = a.wq ? __ldg(reinterpret_cast<const uint4*>(a.wq) + j) : ones;
  const uint4 wk = a.wk ? __ldg(reinterpret_cast<const uint4*>(a.wk) + j) : ones;
  const __nv_bfloat16* qrow = a.q + b * a.q_sb + n * a.q_sn + 8 * j;
  const __nv_bfloat16* krow = a.k + b * a.k_sb + n * a.k_sn + 8 * j;
  const __nv_bfloat16* vrow = MODE == kTrain ? nullptr : a.v + n * a.v_sn + 8 * j;

  for (int hb = h0; hb < h1; hb += U * G) {
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * G + grp;
      x[u] = make_uint4(0, 0, 0, 0);
      if (h < h1) {
        const __nv_bfloat16* p = h < a.Hq ? qrow + h * a.q_sh
                                 : (MODE == kTrain || h < a.Hq + a.Hk) ? krow + (h - a.Hq) * a.k_sh
                                                                       : vrow + (h - a.Hq - a.Hk) * a.v_sh;
        x[u] = ld_stream(p);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * G + grp;
      float y[8], w[8];
      unpack8(x[u], y);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
      const bool is_q = h < a.Hq;
      unpack8(is_q ? wq : wk, w);
      uint4 out;
      float z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = y[e] * r * w[e];
      rotate<LPR, INTER, false>(z, t);
      if (h >= h1) continue;
      if (MODE == kTrain) {
        out = pack8(z);
        __nv_bfloat16* dst = is_q ? a.q_out + (((long long)b * a.Hq + h) * a.N + n) * D
                                  : a.k_out + (((long long)b * a.Hk + (h - a.Hq)) * a.N + n) * D;
        *reinterpret_cast<uint4*>(dst + 8 * j) = out;
      } else if (is_q) {
        *reinterpret_cast<uint4*>(a.q_out + (tok * a.Hq + h) * D + 8 * j) = pack8(z);
      } else {
        const bool is_v = h >= a.Hq + a.Hk;
        const int hk = h - a.Hq - (is_v ? a.Hk : 0);
        const long long off = cache_off + hk * a.c_sh + 8 * j;  // elements
        if (MODE == kCacheBf16) {
          __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(is_v ? a.v_cache : a.k_cache) + off;
          *reinterpret_cast<uint4*>(dst) = is_v ? x[u] : pack8(z);
        } else {
          // the value over its head's factor, rounded once to E4M3 (saturating)
          const float* ds = is_v ? a.v_descale : a.k_descale;
          const float f = ds ? __ldg(ds + hk) : 1.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = (is_v ? y[e] : z[e]) / f;
          uint8_t* dst = reinterpret_cast<uint8_t*>(is_v ? a.v_cache : a.k_cache) + off;
          *reinterpret_cast<uint2*>(dst) = make_uint2(pack_e4m3x4(z[0], z[1], z[2], z[3]),
                                                      pack_e4m3x4(z[4], z[5], z[6], z[7]));
        }
      }
    }
  }
}

// Backward.  Warps walk (token, run of heads) units with a grid stride; a lane keeps the weight
// gradients of its 8 elements in registers over all its rows, the block adds them up in shared
// memory and writes one partial row; fa_norm_rope_dw_kernel adds the partials in block order.  No
// atomics: equal calls give equal bits.
template <int D, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) fa_norm_rope_bwd_kernel(const NormRopeBwdArgs a) {
  constexpr int LPR = D / 8, G = 32 / LPR, W = kThreads / 32;
  __shared__ float red[W][2][D];
  const int lane = threadIdx.x & 31, j = lane % LPR, grp = lane / LPR, warp = threadIdx.x >> 5;
  const long long units = (long long)a.B * a.N * a.chunks;
  const int heads = a.Hq + a.Hk;
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint4 wq = a.wq ? __ldg(reinterpret_cast<const uint4*>(a.wq) + j) : ones;
  const uint4 wk = a.wk ? __ldg(reinterpret_cast<const uint4*>(a.wk) + j) : ones;
  float dwq[8], dwk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = 0.f, dwk[e] = 0.f;

  for (long long unit = (long long)blockIdx.x * W + warp; unit < units; unit += (long long)gridDim.x * W) {
    const long long tok = unit / a.chunks;
    const int h0 = (int)(unit - tok * a.chunks) * a.heads_per_warp;
    const int h1 = min(heads, h0 + a.heads_per_warp);
    const int b = (int)(tok / a.N), n = (int)(tok - (long long)b * a.N);
    int pos = n;
    if (a.rot > 0) {
      if (a.positions) pos = a.positions[(long long)b * a.pos_sb + n];
      if (pos < 0 || pos >= a.rope_rows) {
        if (lane == 0) atomicOr(a.status, FA_DEV_BOUNDS);
        continue;
      }
    }
    Rotation t;
    load_rotation<INTER>(t, a.rope, a.rot, pos, j);
    const __nv_bfloat16* qrow = a.q + b * a.q_sb + n * a.q_sn + 8 * j;
    const __nv_bfloat16* krow = a.k + b * a.k_sb + n * a.k_sn + 8 * j;
    for (int hb = h0; hb < h1; hb += U * G) {
      uint4 x[U], g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * G + grp;
        x[u] = g[u] = make_uint4(0, 0, 0, 0);
        if (h < h1) {
          const bool is_q = h < a.Hq;
          const int hh = is_q ? h : h - a.Hq;
          x[u] = ld_stream(is_q ? qrow + hh * a.q_sh : krow + hh * a.k_sh);
          const __nv_bfloat16* gp = is_q ? a.gq + (((long long)b * a.Hq + hh) * a.N + n) * D
                                         : a.gk + (((long long)b * a.Hk + hh) * a.N + n) * D;
          g[u] = ld_stream(gp + 8 * j);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = hb + u * G + grp;
        const bool is_q = h < a.Hq;
        float xh[8], dy[8], w[8];
        unpack8(x[u], xh);
        unpack8(g[u], dy);
        rotate<LPR, INTER, true>(dy, t);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(xh[e], xh[e], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + a.eps);
        unpack8(is_q ? wq : wk, w);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[e] *= r;
          const float p = dy[e] * xh[e];
          if (h < h1) {
            if (is_q) dwq[e] += p;
            else dwk[e] += p;
          }
          dot = fmaf(p, w[e], dot);
        }
        const float c = row_sum<LPR>(dot) * (1.f / D);
        if (h >= h1) continue;
        float dx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] = r * (dy[e] * w[e] - xh[e] * c);
        __nv_bfloat16* dst = is_q ? a.dq + b * a.dq_sb + n * a.dq_sn + h * a.dq_sh
                                  : a.dk + b * a.dk_sb + n * a.dk_sn + (h - a.Hq) * a.dk_sh;
        *reinterpret_cast<uint4*>(dst + 8 * j) = pack8(dx);
      }
    }
  }
  // the warp's row groups, then the block's warps
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      dwq[e] += __shfl_xor_sync(0xffffffffu, dwq[e], o);
      dwk[e] += __shfl_xor_sync(0xffffffffu, dwk[e], o);
    }
    if (grp == 0) red[warp][0][8 * j + e] = dwq[e], red[warp][1][8 * j + e] = dwk[e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) s += red[w][i / D][i % D];
    a.partial[(size_t)blockIdx.x * 2 * D + i] = s;
  }
}

// dw[i] = sum over blocks of partial[block][i], 32 columns per block, in a fixed order.
__global__ void __launch_bounds__(1024) fa_norm_rope_dw_kernel(const float* __restrict__ partial, int blocks, int d,
                                                               float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + c;
  float s = 0.f;
  for (int r = y; r < blocks; r += 32) s += partial[(size_t)r * 2 * d + col];
  red[y][c] = s;
  __syncthreads();
  float v = red[c][y];  // warp y now holds column y's 32 sums
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (c == 0) {
    const int i = blockIdx.x * 32 + y;
    float* out = i < d ? dwq : dwk;
    if (out) out[i < d ? i : i - d] = v;
  }
}

// Heads per warp: all of a token's heads when there are tokens enough to fill the GPU with a warp
// each, else runs short enough that the warps do, in whole steps of the inner loop.
int heads_per_warp(long long tokens, int heads, int step) {
  const long long want = 148LL * 32;
  long long chunks = std::max(1LL, want / std::max(1LL, tokens));
  long long per = (heads + chunks - 1) / chunks;
  per = (per + step - 1) / step * step;
  return (int)per;
}

}  // namespace

int norm_rope_bwd_blocks(long long tokens, int Hq, int Hk, int d) {
  const int G = 32 / (d / 8), U = 2;
  const int per = heads_per_warp(tokens, Hq + Hk, U * G);
  const long long units = tokens * ((Hq + Hk + per - 1) / per);
  return (int)std::max(1LL, std::min(148LL * 4, (units + 7) / 8));
}

cudaError_t launch_norm_rope(int d, bool interleaved, int mode, NormRopeArgs a, cudaStream_t stream) {
  constexpr int U = 4;
  const int G = 32 / (d / 8);
  const int heads = a.Hq + a.Hk * (mode == kTrain ? 1 : 2);
  const long long tokens = (long long)a.B * a.N;
  a.heads_per_warp = heads_per_warp(tokens, heads, G);
  a.chunks = (heads + a.heads_per_warp - 1) / a.heads_per_warp;
  const long long blocks = (tokens * a.chunks + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > INT_MAX) return cudaErrorInvalidValue;
#define FA_NR(DD, II, MM) fa_norm_rope_kernel<DD, II, MM, U><<<(unsigned)blocks, kThreads, 0, stream>>>(a)
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

cudaError_t launch_norm_rope_bwd(int d, bool interleaved, NormRopeBwdArgs a, float* dwq, float* dwk,
                                 cudaStream_t stream) {
  constexpr int U = 2;
  const int G = 32 / (d / 8);
  const long long tokens = (long long)a.B * a.N;
  a.heads_per_warp = heads_per_warp(tokens, a.Hq + a.Hk, U * G);
  a.chunks = (a.Hq + a.Hk + a.heads_per_warp - 1) / a.heads_per_warp;
  const int blocks = norm_rope_bwd_blocks(tokens, a.Hq, a.Hk, d);
#define FA_NRB(DD, II) fa_norm_rope_bwd_kernel<DD, II, U><<<blocks, kThreads, 0, stream>>>(a)
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
  fa_norm_rope_dw_kernel<<<2 * d / 32, 1024, 0, stream>>>(a.partial, blocks, d, dwq, dwk);
  return cudaGetLastError();
}

}  // namespace fa
