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
constexpr int FWD_CTAS = 6, BWD_CTAS = 4;    // CTAs an SM, at most
constexpr int MAX_TAB = 4096;   // (cos, sin) pairs a CTA holds: 32 KB

struct Side {                   // q or k
  const void* x;
  const void* dy;               // backward only
  void* y;                      // forward: the output; backward: dx
  const void* w;                // NULL: no weight
  int H;
  int ctas;                     // CTAs that take this side's tiles
  int tile;                     // tokens of a tile
  // the CTA's lane groups take `toks` tokens at a time, `gp` groups to a token, each `per` of its
  // heads one after another (so that a lane keeps the token's angles in registers)
  int gp, per, toks;
  long long next_head, next_tok;   // elements from a row to the group's next one
  float* part;                  // backward with a weight: [ctas][D] partial sums
};

struct Params {
  Side s[2];
  const int* pos;
  const float* inv_freq;
  int tokens, N, D, R, pos0, interleaved, norm;
  float eps, af;
};

// Eight elements as loaded, and as fp32.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ void load_raw(Raw<T>& r, const T* p) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float2 (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = make_float2(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
    f[2 * i + 1] = make_float2(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
  }
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16>& r, float2 (&f)[4]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Raw<__half>& r, float2 (&f)[4]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float2 (&f)[4]);
template <>
__device__ __forceinline__ void store8<float>(float* p, const float2 (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[i].x, f[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void store8<__half>(__half* p, const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(f[i].x, f[i].y);
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

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The cosines and sines of a lane's pairs: of frequencies 8 c0 .. 8 c0 + 7 (half layout), or of
// 4 c0 .. 4 c0 + 3 and 4 c1 .. 4 c1 + 3 (interleaved).
struct Angles {
  float2 c[4], s[4];
};
__device__ __forceinline__ void get_angles(Angles& g, const float* cosr, const float* sinr, int c0, int c1,
                                           int interleaved) {
  const int f0 = interleaved ? 4 * c0 : 8 * c0, f1 = interleaved ? 4 * c1 : 8 * c0 + 4;
  const float4 a = *reinterpret_cast<const float4*>(cosr + f0), b = *reinterpret_cast<const float4*>(cosr + f1);
  const float4 u = *reinterpret_cast<const float4*>(sinr + f0), v = *reinterpret_cast<const float4*>(sinr + f1);
  g.c[0] = make_float2(a.x, a.y), g.c[1] = make_float2(a.z, a.w);
  g.c[2] = make_float2(b.x, b.y), g.c[3] = make_float2(b.z, b.w);
  g.s[0] = make_float2(u.x, u.y), g.s[1] = make_float2(u.z, u.w);
  g.s[2] = make_float2(v.x, v.y), g.s[3] = make_float2(v.z, v.w);
}

// Turns the pairs of chunks c0 (a) and c1 (b); BACK by the negated angles.
__device__ __forceinline__ float2 turn_one(float2 x, float c, float s) {
  return make_float2(x.x * c - x.y * s, x.y * c + x.x * s);
}
template <bool BACK>
__device__ __forceinline__ void turn(float2 (&a)[4], float2 (&b)[4], const Angles& g, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float2 s = BACK ? make_float2(-g.s[p].x, -g.s[p].y) : g.s[p];
      const float2 t = BACK ? make_float2(-g.s[p + 2].x, -g.s[p + 2].y) : g.s[p + 2];
      a[2 * p] = turn_one(a[2 * p], g.c[p].x, s.x);
      a[2 * p + 1] = turn_one(a[2 * p + 1], g.c[p].y, s.y);
      b[2 * p] = turn_one(b[2 * p], g.c[p + 2].x, t.x);
      b[2 * p + 1] = turn_one(b[2 * p + 1], g.c[p + 2].y, t.y);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 s = g.s[e], ns = make_float2(-s.x, -s.y);
      const float2 x = a[e], y = b[e];
      a[e] = __ffma2_rn(x, g.c[e], __fmul2_rn(y, BACK ? s : ns));
      b[e] = __ffma2_rn(y, g.c[e], __fmul2_rn(x, BACK ? ns : s));
    }
  }
}

// LPR lanes hold a row (a power of two >= D/16; lanes beyond D/16 idle).
template <typename T, int LPR, bool BWD>
__global__ void __launch_bounds__(THREADS, BWD ? 2 : 3) norm_rope_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) float tab[];     // cos [tile][R/2], then sin
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
  float2 w0[4], w1[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w0[e] = w1[e] = both(1.0f);
  if (s.w && has) {
    Raw<T> r;
    load_raw(r, static_cast<const T*>(s.w) + 8 * c0);
    unpack(r, w0);
    load_raw(r, static_cast<const T*>(s.w) + 8 * c1);
    unpack(r, w1);
  }
  float2 dw0[4], dw1[4];
  if (BWD) {
#pragma unroll
    for (int e = 0; e < 4; ++e) dw0[e] = dw1[e] = both(0.0f);
  }
  const float inv_d = 1.0f / (float)D;
  // this CTA's tokens, equal shares; a tile of them has its cos and sin in shared memory
  const int tok_begin = (int)((long long)p.tokens * cta / s.ctas);
  const int tok_end = (int)((long long)p.tokens * (cta + 1) / s.ctas);
  const bool need_x = !BWD || p.norm;
  for (int tok0 = tok_begin; tok0 < tok_end; tok0 += s.tile) {
    const int n_tok = min(s.tile, tok_end - tok0);
    const size_t base = (size_t)tok0 * H * D;
    const T* x = static_cast<const T*>(s.x) + base;
    const T* dy = static_cast<const T*>(s.dy) + base;
    T* y = static_cast<T*>(s.y) + base;
    // a row's loads go out one step before it is worked on, the first ones before the angles
    Raw<T> xa, xb, ya, yb;
    auto fetch = [&](int tok, size_t off) {
      if (!has || tok >= n_tok) return;
      if (need_x) {
        load_raw(xa, x + off + 8 * c0);
        load_raw(xb, x + off + 8 * c1);
      }
      if (BWD) {
        load_raw(ya, dy + off + 8 * c0);
        load_raw(yb, dy + off + 8 * c1);
      }
    };
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) xa.v[i] = xb.v[i] = ya.v[i] = yb.v[i] = make_uint4(0, 0, 0, 0);
    int tok = row0 / s.gp, k = 0;
    size_t off = ((size_t)tok * H + row0 % s.gp) * D;
    fetch(tok, off);
    __syncthreads();
    float* sin_tab = tab + n_tok * half;
    for (int i = threadIdx.x; i < n_tok * half; i += THREADS) {
      const int tk = i / half, f = i - tk * half;
      const int pos = p.pos ? p.pos[tok0 + tk] : p.pos0 + (tok0 + tk) % p.N;
      const double turns = (double)pos * (double)p.inv_freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
      float sn, cn;
      sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
      tab[i] = cn * p.af;
      sin_tab[i] = sn * p.af;
    }
    __syncthreads();
    Angles g;
#pragma unroll
    for (int e = 0; e < 4; ++e) g.c[e] = both(1.0f), g.s[e] = both(0.0f);
    const int steps = (n_tok + s.toks - 1) / s.toks * s.per;   // the same for every lane
    for (int i = 0; i < steps; ++i) {
      const bool live = has && tok < n_tok;
      const size_t at = off;
      float2 a[4], b[4], ga[4], gb[4];
      unpack(xa, a);
      unpack(xb, b);
      if (BWD) {
        unpack(ya, ga);
        unpack(yb, gb);
      }
      if (k == 0 && rot && live) get_angles(g, tab + tok * half, sin_tab + tok * half, c0, c1, p.interleaved);
      if (++k == s.per) {
        k = 0;
        tok += s.toks;
        off += s.next_tok;
      } else {
        off += s.next_head;
      }
      fetch(tok, off);
      float rstd = 1.0f;
      if (p.norm) {
        float2 ss = both(0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = __ffma2_rn(a[e], a[e], __ffma2_rn(b[e], b[e], ss));
        rstd = rsqrtf(row_sum<LPR>(ss.x + ss.y) * inv_d + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // xhat
          a[e] = __fmul2_rn(a[e], both(rstd));
          b[e] = __fmul2_rn(b[e], both(rstd));
        }
      }
      if (!BWD) {
        if (p.norm) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = __fmul2_rn(a[e], w0[e]);
            b[e] = __fmul2_rn(b[e], w1[e]);
          }
        }
        if (rot) turn<false>(a, b, g, p.interleaved);
        if (live) {
          store8(y + at + 8 * c0, a);
          store8(y + at + 8 * c1, b);
        }
      } else {
        if (rot) turn<true>(ga, gb, g, p.interleaved);
        if (p.norm) {
          float2 dot2 = both(0.0f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (live) {     // behind its last row a lane holds that row's values still
              dw0[e] = __ffma2_rn(ga[e], a[e], dw0[e]);
              dw1[e] = __ffma2_rn(gb[e], b[e], dw1[e]);
            }
            ga[e] = __fmul2_rn(ga[e], w0[e]);
            gb[e] = __fmul2_rn(gb[e], w1[e]);
            dot2 = __ffma2_rn(ga[e], a[e], __ffma2_rn(gb[e], b[e], dot2));
          }
          const float dot = row_sum<LPR>(dot2.x + dot2.y) * inv_d;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ga[e] = __fmul2_rn(both(rstd), __ffma2_rn(a[e], both(-dot), ga[e]));
            gb[e] = __fmul2_rn(both(rstd), __ffma2_rn(b[e], both(-dot), gb[e]));
          }
        }
        if (live) {
          store8(y + at + 8 * c0, ga);
          store8(y + at + 8 * c1, gb);
        }
      }
    }
  }
  if (BWD && s.part) {   // the CTA's sums, rows in order
    float* red = tab;                              // [ROWS][D]
    __syncthreads();
    if (has) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<float2*>(red + row0 * D + 8 * c0 + 2 * e) = dw0[e];
        *reinterpret_cast<float2*>(red + row0 * D + 8 * c1 + 2 * e) = dw1[e];
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
    if (p.s[i].ctas) tab = std::max(tab, (size_t)p.s[i].tile * (p.R / 2) * 2 * sizeof(float));
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

// CTAs of each side and the tokens of a tile.  A CTA should have at least a few steps of rows to
// share its cos and sin among, unless there are too few tokens to give every SM one.
void plan(Params& p, int n_sm, int max_ctas) {
  const int rows = THREADS / lanes(p.D);
  const int heads = p.s[0].H + p.s[1].H;
  for (int i = 0; i < 2; ++i) {
    Side& s = p.s[i];
    if (!s.H) {
      s.ctas = 0;
      continue;
    }
    const long long tile = std::max(1LL, 4LL * rows / s.H);          // tokens of four steps
    const long long share = std::max(1LL, (long long)max_ctas * s.H / heads);
    const long long one_each = std::max(1LL, 4LL * n_sm * s.H / heads);
    const long long least = std::max(1LL, (long long)rows / s.H);    // tokens of one step
    long long ctas = std::max(((long long)p.tokens + tile - 1) / tile,
                              std::min(((long long)p.tokens + least - 1) / least, one_each));
    s.ctas = (int)std::min(ctas, share);
    const long long toks = ((long long)p.tokens + s.ctas - 1) / s.ctas;
    s.tile = (int)(p.R ? std::min(toks, (long long)MAX_TAB / (p.R / 2)) : toks);
    // at least two heads a group where there are two: neighbouring groups then read neighbouring
    // rows, and a step of the CTA spans few tokens
    s.gp = 1;
    while (s.H % (2 * s.gp) == 0 && s.H / (2 * s.gp) >= 2 && 2 * s.gp <= rows) s.gp *= 2;
    s.per = s.H / s.gp;
    s.toks = rows / s.gp;
    s.next_head = (long long)s.gp * p.D;
    s.next_tok = (long long)s.toks * s.H * p.D - (s.per - 1) * s.next_head;
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
  nr::plan(p, n_sm, nr::FWD_CTAS * n_sm);
  return nr::launch(p, a.dtype, false, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, float* part, int n_sm, cudaStream_t st) {
  nr::Params p = nr::make(a);
  nr::plan(p, n_sm, std::min(kNormRopePartials, nr::BWD_CTAS * n_sm));
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
