// s2attn_norm_rope.cu -- RMS norm of every q and k head and the rotary embedding, one pass.
//
// For a head's row x of D elements at position t:
//   xhat = x / sqrt(mean(x^2) + eps),  y = w * xhat  (or y = x without the norm)
//   the first R elements of y turn in pairs by the angles t * inv_freq[i], i < R/2:
//     (a, b) -> af * (a cos - b sin, b cos + a sin)
//   with pairs (i, i + R/2) or, interleaved, (2i, 2i + 1); the rest passes.
// Backward, with g the gradient turned back (angles negated) and gx = w * g:
//   dx = (gx - xhat * mean(gx * xhat)) / rms,   dw = sum over rows of g * xhat.
//
// HBM-bound: the forward moves each element twice, the backward three times, against about
// ten flops.  So a row is held in the registers of D/16 lanes from its load to its store:
// a lane takes two chunks of 8 elements that hold both halves of its pairs (chunk c and
// chunk c + R/16), hence the rotation needs no exchange, and the two sums of the norm are
// shuffles over the row's lanes.  cos and sin are the same for all heads of a token: a CTA
// takes a tile of tokens and computes them once into shared memory, so that no table of
// positions is kept in HBM and any position is served.  The turn t * inv_freq / 2pi is
// formed and reduced to [-1/2, 1/2] in 64 bits (in 32 a position of 100k would leave 2^-8
// of a turn's precision), then sincospif runs on the remainder in 32.
// All arithmetic is fp32; y, dx and dw are rounded once, at the end.
// dw: a thread keeps the sums of its 16 columns over all rows it takes, the CTA adds its
// rows' threads in a fixed order and writes one partial; a second kernel adds the partials
// in order, so dw does not depend on which CTA ran first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "s2_internal.h"
#include "s2attn.h"

namespace s2 {
namespace nr {

constexpr int THREADS = 256;
constexpr int MAX_TAB = 4096;   // (cos, sin) pairs a CTA holds: 32 KB

struct Side {                   // q or k
  const void* x;
  const void* dy;               // backward only
  void* y;                      // forward: the output; backward: dx
  const void* w;                // NULL: no weight
  int H;
  int ctas;                     // CTAs that take this side's tiles
  int tile;                     // tokens of a tile
  float* part;                  // backward with a weight: [ctas][D] partial sums
};

struct Params {
  Side s[2];
  const int* pos;
  const float* inv_freq;
  int tokens, N, D, R, pos0, interleaved, norm;
  float eps, af;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<__half>(const __half* p, float (&f)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store1(float* p, float f) { *p = f; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }
__device__ __forceinline__ void store1(__half* p, float f) { *p = __float2half_rn(f); }

// Sum over the LPR lanes of a row (every lane of the warp takes part).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Turns the pairs of chunks c0 (a) and c1 (b); cs is the token's (cos, sin) row.
// BACK turns by the negated angles.
template <bool BACK>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float2* cs, int c0, int c1, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 u = cs[4 * c0 + p], v = cs[4 * c1 + p];
      const float su = BACK ? -u.y : u.y, sv = BACK ? -v.y : v.y;
      const float a0 = a[2 * p], a1 = a[2 * p + 1], b0 = b[2 * p], b1 = b[2 * p + 1];
      a[2 * p] = a0 * u.x - a1 * su;
      a[2 * p + 1] = a1 * u.x + a0 * su;
      b[2 * p] = b0 * v.x - b1 * sv;
      b[2 * p + 1] = b1 * v.x + b0 * sv;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 u = cs[8 * c0 + e];
      const float s = BACK ? -u.y : u.y;
      const float x = a[e], y = b[e];
      a[e] = x * u.x - y * s;
      b[e] = y * u.x + x * s;
    }
  }
}

// LPR lanes hold a row (a power of two >= D/16; lanes beyond D/16 idle).
template <typename T, int LPR, bool BWD>
__global__ void __launch_bounds__(THREADS) norm_rope_kernel(const __grid_constant__ Params p) {
  extern __shared__ float2 tab[];                  // [tile][R/2]
  constexpr int ROWS = THREADS / LPR;              // rows of one step of the CTA
  const int side = (int)blockIdx.x < p.s[0].ctas ? 0 : 1;
  const Side& s = p.s[side];
  const int cta = (int)blockIdx.x - (side ? p.s[0].ctas : 0);
  const int lane = threadIdx.x % LPR, row0 = threadIdx.x / LPR;
  const int D = p.D, R = p.R, H = s.H, half = R / 2;
  const bool has = lane < D / 16;
  const bool rot = lane < R / 16;
  const int c0 = rot ? lane : R / 8 + 2 * (lane - R / 16);
  const int c1 = rot ? lane + R / 16 : c0 + 1;
  float w0[8], w1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w0[e] = w1[e] = 1.0f;
  if (s.w && has) {
    load8(static_cast<const T*>(s.w) + 8 * c0, w0);
    load8(static_cast<const T*>(s.w) + 8 * c1, w1);
  }
  float dw0[8], dw1[8];
  if (BWD) {
#pragma unroll
    for (int e = 0; e < 8; ++e) dw0[e] = dw1[e] = 0.0f;
  }
  const float inv_d = 1.0f / (float)D;
  const long long n_tiles = ((long long)p.tokens + s.tile - 1) / s.tile;
  for (long long tl = cta; tl < n_tiles; tl += s.ctas) {
    const int tok0 = (int)(tl * s.tile);
    const int n_tok = min(s.tile, p.tokens - tok0);
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * half; i += THREADS) {
      const int tk = i / half, f = i - tk * half;
      const int pos = p.pos ? p.pos[tok0 + tk] : p.pos0 + (tok0 + tk) % p.N;
      const double turns = (double)pos * (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
      float sn, cn;
      sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
      tab[i] = make_float2(cn * p.af, sn * p.af);
    }
    __syncthreads();
    const int n_rows = n_tok * H;
    const size_t base = (size_t)tok0 * H * D;
    for (int r0 = 0; r0 < n_rows; r0 += ROWS) {   // the same trip count for every lane
      const int r = r0 + row0;
      const bool live = has && r < n_rows;
      const size_t off = base + (size_t)r * D;
      float a[8], b[8], ga[8], gb[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = b[e] = ga[e] = gb[e] = 0.0f;
      if (live) {
        if (!BWD || p.norm) {
          load8(static_cast<const T*>(s.x) + off + 8 * c0, a);
          load8(static_cast<const T*>(s.x) + off + 8 * c1, b);
        }
        if (BWD) {
          load8(static_cast<const T*>(s.dy) + off + 8 * c0, ga);
          load8(static_cast<const T*>(s.dy) + off + 8 * c1, gb);
        }
      }
      const float2* cs = tab + (live ? r / H : 0) * half;
      float rstd = 1.0f;
      if (p.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
        rstd = rsqrtf(row_sum<LPR>(ss) * inv_d + p.eps);
      }
      if (!BWD) {
        if (p.norm) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            a[e] = a[e] * rstd * w0[e];
            b[e] = b[e] * rstd * w1[e];
          }
        }
        if (rot) turn<false>(a, b, cs, c0, c1, p.interleaved);
        if (live) {
          store8(static_cast<T*>(s.y) + off + 8 * c0, a);
          store8(static_cast<T*>(s.y) + off + 8 * c1, b);
        }
      } else {
        if (rot) turn<true>(ga, gb, cs, c0, c1, p.interleaved);
        if (p.norm) {
          float dot = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            a[e] *= rstd;   // xhat
            b[e] *= rstd;
            dw0[e] = fmaf(ga[e], a[e], dw0[e]);
            dw1[e] = fmaf(gb[e], b[e], dw1[e]);
            ga[e] *= w0[e];
            gb[e] *= w1[e];
            dot = fmaf(ga[e], a[e], fmaf(gb[e], b[e], dot));
          }
          dot = row_sum<LPR>(dot) * inv_d;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ga[e] = rstd * (ga[e] - a[e] * dot);
            gb[e] = rstd * (gb[e] - b[e] * dot);
          }
        }
        if (live) {
          store8(static_cast<T*>(s.y) + off + 8 * c0, ga);
          store8(static_cast<T*>(s.y) + off + 8 * c1, gb);
        }
      }
    }
  }
  if (BWD && s.part) {   // the CTA's sums, rows in order
    float* red = reinterpret_cast<float*>(tab);    // [ROWS][D]
    __syncthreads();
    if (has) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        red[row0 * D + 8 * c0 + e] = dw0[e];
        red[row0 * D + 8 * c1 + e] = dw1[e];
      }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += THREADS) {
      float sum = 0.0f;
      for (int r = 0; r < ROWS; ++r) sum += red[r * D + d];
      s.part[(size_t)cta * D + d] = sum;
    }
  }
}

// dw[d] = sum over the CTAs' partials, in order: 8 columns a block, 32 threads a column.
struct SumArgs {
  const float* part[2];
  void* dw[2];
  int n[2];
  int D;
};
template <typename T>
__global__ void __launch_bounds__(256) dw_sum_kernel(const __grid_constant__ SumArgs a) {
  __shared__ float red[32][8];
  const int side = blockIdx.y, col = (int)blockIdx.x * 8 + threadIdx.x % 8, slice = threadIdx.x / 8;
  float sum = 0.0f;
  if (a.part[side])
    for (int i = slice; i < a.n[side]; i += 32) sum += a.part[side][(size_t)i * a.D + col];
  red[slice][threadIdx.x % 8] = sum;
  __syncthreads();
  if (slice == 0 && a.part[side]) {
    float t = 0.0f;
    for (int i = 0; i < 32; ++i) t += red[i][threadIdx.x];
    store1(static_cast<T*>(a.dw[side]) + col, t);
  }
}

size_t smem_bytes(const Params& p, int lpr, bool bwd) {
  size_t tab = 0;
  for (int i = 0; i < 2; ++i)
    if (p.s[i].ctas) tab = std::max(tab, (size_t)p.s[i].tile * (p.R / 2) * sizeof(float2));
  const size_t red = bwd ? (size_t)(THREADS / lpr) * p.D * sizeof(float) : 0;
  return std::max(tab, red);
}

template <typename T, int LPR>
cudaError_t launch_lpr(const Params& p, bool bwd, cudaStream_t st) {
  const int grid = p.s[0].ctas + p.s[1].ctas;
  const size_t smem = smem_bytes(p, LPR, bwd);   // at most 32 KB
  if (bwd)
    norm_rope_kernel<T, LPR, true><<<grid, THREADS, smem, st>>>(p);
  else
    norm_rope_kernel<T, LPR, false><<<grid, THREADS, smem, st>>>(p);
  return cudaGetLastError();
}

int lanes(int D) { return D <= 64 ? 4 : D <= 128 ? 8 : 16; }

template <typename T>
cudaError_t launch_type(const Params& p, bool bwd, cudaStream_t st) {
  switch (lanes(p.D)) {
    case 4: return launch_lpr<T, 4>(p, bwd, st);
    case 8: return launch_lpr<T, 8>(p, bwd, st);
    default: return launch_lpr<T, 16>(p, bwd, st);
  }
}

// Tokens of a tile and CTAs of each side.  A tile has about four steps of rows so that the
// cos/sin work is shared by many rows; with few tokens it shrinks until every SM has one.
void plan(Params& p, int n_sm, int max_ctas) {
  const int rows = THREADS / lanes(p.D);
  const int heads = p.s[0].H + p.s[1].H;
  for (int i = 0; i < 2; ++i) {
    Side& s = p.s[i];
    if (!s.H) {
      s.ctas = 0;
      continue;
    }
    long long tile = (4LL * rows + s.H - 1) / s.H;
    const long long share = std::max(1LL, (long long)n_sm * s.H / heads);
    tile = std::min(tile, ((long long)p.tokens + share - 1) / share);
    if (p.R) tile = std::min(tile, (long long)MAX_TAB / (p.R / 2));
    s.tile = (int)std::max(1LL, tile);
    const long long tiles = ((long long)p.tokens + s.tile - 1) / s.tile;
    const long long cap = std::max(1LL, (long long)max_ctas * s.H / heads);
    s.ctas = (int)std::min(tiles, cap);
  }
}

Params make(const NormRopeArgs& a) {
  Params p{};
  p.s[0].x = a.q, p.s[1].x = a.k;
  p.s[0].dy = a.dq_out, p.s[1].dy = a.dk_out;
  p.s[0].y = a.q_dst, p.s[1].y = a.k_dst;
  p.s[0].w = a.wq, p.s[1].w = a.wk;
  p.s[0].H = a.q_dst ? a.Hq : 0, p.s[1].H = a.k_dst ? a.Hk : 0;
  p.pos = a.positions, p.inv_freq = a.inv_freq;
  p.tokens = a.B * a.N, p.N = a.N, p.D = a.D, p.R = a.R, p.pos0 = a.pos0;
  p.interleaved = a.interleaved, p.norm = a.norm, p.eps = a.eps, p.af = a.attn_factor;
  return p;
}

cudaError_t launch(const Params& p, int dtype, bool bwd, cudaStream_t st) {
  if (dtype == S2ATTN_BF16) return launch_type<__nv_bfloat16>(p, bwd, st);
  if (dtype == S2ATTN_FP16) return launch_type<__half>(p, bwd, st);
  return launch_type<float>(p, bwd, st);
}

}  // namespace nr

cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, int n_sm, cudaStream_t st) {
  nr::Params p = nr::make(a);
  nr::plan(p, n_sm, 16 * n_sm);
  return nr::launch(p, a.dtype, false, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, float* part, int n_sm, cudaStream_t st) {
  nr::Params p = nr::make(a);
  nr::plan(p, n_sm, std::min(kNormRopePartials, 4 * n_sm));
  if (a.dwq && p.s[0].H) p.s[0].part = part;
  if (a.dwk && p.s[1].H) p.s[1].part = part + (size_t)p.s[0].ctas * a.D;
  cudaError_t e = nr::launch(p, a.dtype, true, st);
  if (e != cudaSuccess || (!p.s[0].part && !p.s[1].part)) return e;
  nr::SumArgs s{};
  s.D = a.D;
  void* dw[2] = {a.dwq, a.dwk};
  for (int i = 0; i < 2; ++i) s.part[i] = p.s[i].part, s.dw[i] = dw[i], s.n[i] = p.s[i].ctas;
  const dim3 grid(a.D / 8, 2);
  if (a.dtype == S2ATTN_BF16)
    nr::dw_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(s);
  else if (a.dtype == S2ATTN_FP16)
    nr::dw_sum_kernel<__half><<<grid, 256, 0, st>>>(s);
  else
    nr::dw_sum_kernel<float><<<grid, 256, 0, st>>>(s);
  return cudaGetLastError();
}

}  // namespace s2
