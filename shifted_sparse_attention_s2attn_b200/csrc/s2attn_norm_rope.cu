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
// ten flops.  A row is held in the registers of D/16 lanes from its load to its store: a lane
// takes two chunks of 8 elements that hold both halves of its pairs (chunk c and chunk
// c + R/16), hence the rotation needs no exchange, and the two sums of the norm are shuffles
// over the row's lanes; the next row's loads go out before a row is worked on.  cos and sin
// are the same for all heads of a token, so a CTA computes them once for a tile of tokens, in
// shared memory: no table of positions is kept in HBM and any position is served.  The turn
// t * inv_freq / 2pi is formed and reduced to [-1/2, 1/2] in 64 bits (in 32 a position of 100k
// would leave 2^-8 of a turn's precision), then sincospif runs on the remainder in 32.
// All arithmetic is fp32; y, dx and dw are rounded once, at the end.
// dw: a thread keeps the sums of its 16 columns over all rows it takes, the CTA adds its
// rows' threads in a fixed order and writes one partial; a second kernel adds the partials
// in order, so dw does not depend on which CTA ran first.
// Measured (B200, bf16, D = 128): forward of a 32k prompt, 32 + 32 heads, 182-195 us = 5.5-5.9 TB/s, 0.84-0.90
// of the copy bandwidth; forward and backward at 8k, 32 + 8 heads, 84-90 us, 4.7-5.0 TB/s.  In fp32 395-400 us
// (0.82) and 153-158 us (0.83); its instances spill (8 bytes forward, 20 backward).  Tried and not
// kept: rows through a ring of bulk copies in shared memory (192 and 127 us), one chunk a lane with
// the other half shuffled (237 and 125), kernels of their own for each layout and for rows with and
// without the norm (181 and 90).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "s2_internal.h"
#include "s2attn.h"

namespace s2 {
namespace nr {

constexpr int THREADS = 256;
// CTAs an SM, all resident at once (a 32k prompt, 32 + 32 heads: 3 183 us, 2 215, 4 (64 registers,
// spills) 201; 8k forward and backward, 32 + 8 heads: backward at 2 90 us, at 3 (spills) 118)
constexpr int FWD_CTAS = 3, BWD_CTAS = 2;
constexpr double kAngleRows = 3.0;   // a token's angles cost as much as this many rows (R = D)
constexpr int MAX_TAB = 2048;   // (cos, sin) pairs of a tile, at most: 16 KB

struct Side {                   // q or k
  const void* x;
  const void* dy;               // backward only
  void* y;                      // forward: the output; backward: dx
  const void* w;                // NULL: no weight
  int H;                        // 0: no such side
  uint32_t inv_h;               // ceil(2^32 / H) for H > 1: row / H is the high half of row * inv_h, exactly for
                                // row * H < 2^32 (inv_h * H exceeds 2^32 by less than H)
  float* part;                  // backward with a weight: [ctas][D] partial sums
};

struct Params {
  Side s[2];
  const int* pos;
  const float* inv_freq;
  int tokens, N, D, R, pos0, interleaved, norm;
  int tile;                     // tokens whose cos and sin are held at a time
  int ctas_q;                   // backward: CTAs of q, the others take k
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
// Where a token's table holds frequency f: interleaved, in order; else the first four of each
// eight before the last four, so that neighbouring lanes read neighbouring 16 bytes.
__device__ __forceinline__ int tab_pos(int f, int R, int interleaved) {
  return interleaved ? f : ((f & 4) / 4 * (R / 16) + f / 8) * 4 + f % 4;
}
__device__ __forceinline__ void get_angles(Angles& g, const float* cosr, const float* sinr, int c0, int c1, int R,
                                           int interleaved) {
  const int f0 = 4 * c0, f1 = interleaved ? 4 * c1 : 4 * (R / 16 + c0);
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

// LPR lanes hold a row (a power of two >= D/16; lanes beyond D/16 idle).  Forward: a CTA takes the
// q and k rows of its tokens, which share the angles.  Backward: of one side, whose dw it sums.
template <typename T, int LPR, bool BWD>
__global__ void __launch_bounds__(THREADS, BWD ? BWD_CTAS : FWD_CTAS) norm_rope_kernel(const __grid_constant__ Params p) {
  constexpr int ROWS = THREADS / LPR;              // rows of one step of the CTA
  extern __shared__ __align__(16) float smem[];    // cos [tile][R/2], sin; backward, at the end: sums
  const int lane = threadIdx.x % LPR, row0 = threadIdx.x / LPR;
  const int D = p.D, R = p.R, half = R / 2;
  const bool has = lane < D / 16;
  const bool rot = lane < R / 16;
  const int c0 = rot ? lane : R / 8 + 2 * (lane - R / 16);
  const int c1 = rot ? lane + R / 16 : c0 + 1;
  const int apart = 8 * (c1 - c0);                 // elements from the lane's first chunk to its second
  const float inv_d = 1.0f / (float)D;
  // (the sum of dw may be scheduled now; it waits for this whole grid)
  if (BWD) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int side = BWD && (int)blockIdx.x >= p.ctas_q ? 1 : 0;
  const int cta = (int)blockIdx.x - (side ? p.ctas_q : 0);
  const int ctas = BWD ? (side ? (int)gridDim.x - p.ctas_q : p.ctas_q) : (int)gridDim.x;
  float* cos_tab = smem;
  float* sin_tab = cos_tab + p.tile * half;
  float2 dw0[4], dw1[4];
  if (BWD) {
#pragma unroll
    for (int e = 0; e < 4; ++e) dw0[e] = dw1[e] = both(0.0f);
  }
  Raw<T> xa, xb, ya, yb;                           // a row's x and dy, one step ahead
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) xa.v[i] = xb.v[i] = ya.v[i] = yb.v[i] = make_uint4(0, 0, 0, 0);
  auto fetch = [&](const T* x, const T* dy) {
    if (!BWD || p.norm) {
      load_raw(xa, x);
      load_raw(xb, x + apart);
    }
    if (BWD) {
      load_raw(ya, dy);
      load_raw(yb, dy + apart);
    }
  };
  // a thread's angles: one frequency (in turns: 1 / 2 pi), every ang_step-th token of a tile
  const int ang_step = half ? THREADS / half : 1, ang_f = half ? (int)threadIdx.x % half : 0;
  const int ang_tok = half && (int)threadIdx.x < ang_step * half ? (int)threadIdx.x / half : p.tile;
  const int ang_at = tab_pos(ang_f, R, p.interleaved);
  const double turn_freq = half ? (double)p.inv_freq[ang_f] * 0.15915494309189533577 : 0.0;
  // this CTA's tokens, an equal share
  const int tok_begin = (int)((long long)p.tokens * cta / ctas);
  const int tok_end = (int)((long long)p.tokens * (cta + 1) / ctas);
  for (int tok0 = tok_begin; tok0 < tok_end; tok0 += p.tile) {
    const int n_tok = min(p.tile, tok_end - tok0);
    __syncthreads();
    for (int tk = ang_tok; tk < n_tok; tk += ang_step) {
      const int pos = p.pos ? p.pos[tok0 + tk] : p.pos0 + (tok0 + tk) % p.N;
      const double turns = (double)pos * turn_freq;
      float sn, cn;
      sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cn);
      cos_tab[tk * half + ang_at] = cn * p.af;
      sin_tab[tk * half + ang_at] = sn * p.af;
    }
    __syncthreads();
#pragma unroll 1
    for (int sd = side; sd < (BWD ? side + 1 : 2); ++sd) {
      const Side& s = p.s[sd];
      const int n_rows = n_tok * s.H;
      if (n_rows == 0) continue;
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
      const size_t first = ((size_t)tok0 * s.H + row0) * D + 8 * c0;
      const T* x = static_cast<const T*>(s.x) + first;
      const T* dy = static_cast<const T*>(s.dy) + first;
      T* y = static_cast<T*>(s.y) + first;
      const int step = ROWS * D;
      if (has && row0 < n_rows) fetch(x, dy);
      for (int r = row0; r - row0 < n_rows; r += ROWS) {   // the same trip count for every lane
        const bool live = has && r < n_rows;
        float2 a[4], b[4], ga[4], gb[4];
        unpack(xa, a);
        unpack(xb, b);
        if (BWD) {
          unpack(ya, ga);
          unpack(yb, gb);
        }
        x += step;
        dy += step;
        if (has && r + ROWS < n_rows) fetch(x, dy);
        auto turn_row = [&](float2 (&u)[4], float2 (&v)[4]) {
          if (!rot || !live) return;
          const int tk = s.H == 1 ? r : (int)__umulhi((uint32_t)r, s.inv_h);
          Angles g;
          get_angles(g, cos_tab + tk * half, sin_tab + tk * half, c0, c1, R, p.interleaved);
          turn<BWD>(u, v, g, p.interleaved);
        };
        if (!BWD) {
          if (p.norm) {
            float2 ss = both(0.0f);
#pragma unroll
            for (int e = 0; e < 4; ++e) ss = __ffma2_rn(a[e], a[e], __ffma2_rn(b[e], b[e], ss));
            const float rstd = rsqrtf(row_sum<LPR>(ss.x + ss.y) * inv_d + p.eps);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a[e] = __fmul2_rn(__fmul2_rn(a[e], both(rstd)), w0[e]);
              b[e] = __fmul2_rn(__fmul2_rn(b[e], both(rstd)), w1[e]);
            }
          }
          turn_row(a, b);
        } else {
          turn_row(ga, gb);
          if (p.norm) {
            // both sums at once: of x^2, and of gx x (mean(gx xhat) is the latter times rstd / D)
            float2 ss = both(0.0f), gs = both(0.0f);
            float2 ha[4], hb[4];   // gx
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ha[e] = __fmul2_rn(ga[e], w0[e]);
              hb[e] = __fmul2_rn(gb[e], w1[e]);
              ss = __ffma2_rn(a[e], a[e], __ffma2_rn(b[e], b[e], ss));
              gs = __ffma2_rn(ha[e], a[e], __ffma2_rn(hb[e], b[e], gs));
            }
            float s2x = ss.x + ss.y, sgx = gs.x + gs.y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) {
              s2x += __shfl_xor_sync(0xffffffffu, s2x, o);
              sgx += __shfl_xor_sync(0xffffffffu, sgx, o);
            }
            const float rstd = rsqrtf(s2x * inv_d + p.eps);
            const float dot = rstd * sgx * inv_d;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 xa_hat = __fmul2_rn(a[e], both(rstd)), xb_hat = __fmul2_rn(b[e], both(rstd));
              if (live) {     // behind its last row a lane holds that row's values still
                dw0[e] = __ffma2_rn(ga[e], xa_hat, dw0[e]);
                dw1[e] = __ffma2_rn(gb[e], xb_hat, dw1[e]);
              }
              ga[e] = __fmul2_rn(both(rstd), __ffma2_rn(xa_hat, both(-dot), ha[e]));
              gb[e] = __fmul2_rn(both(rstd), __ffma2_rn(xb_hat, both(-dot), hb[e]));
            }
          }
        }
        if (live) {
          store8(y, BWD ? ga : a);
          store8(y + apart, BWD ? gb : b);
        }
        y += step;
      }
    }
  }
  if (BWD && p.s[side].part) {   // the CTA's sums, lane groups in order
    __syncthreads();
    float* red = smem;           // [ROWS][D]
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
      p.s[side].part[(size_t)cta * D + d] = sum;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

template <typename T, int LPR>
cudaError_t launch_lpr(const Params& p, int grid, bool bwd, cudaStream_t st) {
  const size_t tab = (size_t)p.tile * p.R * sizeof(float);      // at most 16 KB
  if (bwd)
    norm_rope_kernel<T, LPR, true>
        <<<grid, THREADS, std::max(tab, (size_t)(THREADS / LPR) * p.D * sizeof(float)), st>>>(p);
  else
    norm_rope_kernel<T, LPR, false><<<grid, THREADS, tab, st>>>(p);
  return cudaGetLastError();
}

int lanes(int D) { return D <= 64 ? 4 : D <= 128 ? 8 : 16; }

template <typename T>
cudaError_t launch_type(const Params& p, int grid, bool bwd, cudaStream_t st) {
  switch (lanes(p.D)) {
    case 4: return launch_lpr<T, 4>(p, grid, bwd, st);
    case 8: return launch_lpr<T, 8>(p, grid, bwd, st);
    default: return launch_lpr<T, 16>(p, grid, bwd, st);
  }
}

// CTAs for `heads` heads a token, at most `most`: with few tokens one step of rows each, so that
// every SM has work; else at least four steps, which share the angles.
int ctas_for(const Params& p, int heads, long long least, long long most) {
  const long long rows = THREADS / lanes(p.D), all = (long long)p.tokens * heads;
  const long long fine = std::min((all + rows - 1) / rows, least), coarse = (all + 4 * rows - 1) / (4 * rows);
  return (int)std::max(1LL, std::min({(long long)p.tokens, std::max(fine, coarse), most}));
}

// Tokens of a tile: a CTA's share, as far as the angles and the division by H (see Side) go.
int tile_for(const Params& p, int ctas) {
  long long t = ((long long)p.tokens + ctas - 1) / ctas;
  if (p.R) t = std::min(t, (long long)MAX_TAB / (p.R / 2));
  for (const Side& s : p.s)
    if (s.H > 1) t = std::min({t, ((1ll << 32) - 1) / ((long long)s.H * s.H), (1ll << 30) / s.H});
  return (int)t;
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
  for (Side& s : p.s)
    if (s.H > 1) s.inv_h = (uint32_t)(((1ull << 32) + s.H - 1) / s.H);
  return p;
}

cudaError_t launch(const Params& p, int grid, int dtype, bool bwd, cudaStream_t st) {
  if (dtype == S2ATTN_BF16) return launch_type<__nv_bfloat16>(p, grid, bwd, st);
  if (dtype == S2ATTN_FP16) return launch_type<__half>(p, grid, bwd, st);
  return launch_type<float>(p, grid, bwd, st);
}

}  // namespace nr

cudaError_t launch_norm_rope_fwd(const NormRopeArgs& a, int n_sm, cudaStream_t st) {
  nr::Params p = nr::make(a);
  const int grid = nr::ctas_for(p, p.s[0].H + p.s[1].H, 2 * n_sm, (long long)nr::FWD_CTAS * n_sm);
  p.tile = nr::tile_for(p, grid);
  return nr::launch(p, grid, a.dtype, false, st);
}

cudaError_t launch_norm_rope_bwd(const NormRopeArgs& a, float* part, int n_sm, cudaStream_t st) {
  nr::Params p = nr::make(a);
  // a side's share of the CTAs goes by its work, rows and angles (8k, 32 + 8 heads, forward and
  // backward: shares by rows alone 90 us, these 85)
  const long long most = std::min(kNormRopePartials, nr::BWD_CTAS * n_sm);
  double cost[2];
  for (int i = 0; i < 2; ++i) cost[i] = p.s[i].H ? p.s[i].H + nr::kAngleRows * p.R / p.D : 0.0;
  int ctas[2];
  for (int i = 0; i < 2; ++i)
    ctas[i] = p.s[i].H ? nr::ctas_for(p, p.s[i].H, (long long)(2 * n_sm * cost[i] / (cost[0] + cost[1])),
                                      std::max(1LL, (long long)(most * cost[i] / (cost[0] + cost[1])))) : 0;
  p.ctas_q = ctas[0];
  p.tile = nr::tile_for(p, ctas[0] && ctas[1] ? std::min(ctas[0], ctas[1]) : ctas[0] + ctas[1]);
  if (a.dwq && p.s[0].H) p.s[0].part = part;
  if (a.dwk && p.s[1].H) p.s[1].part = part + (size_t)ctas[0] * a.D;
  cudaError_t e = nr::launch(p, ctas[0] + ctas[1], a.dtype, true, st);
  if (e != cudaSuccess || (!p.s[0].part && !p.s[1].part)) return e;
  nr::SumArgs s{};
  s.D = a.D;
  void* dw[2] = {a.dwq, a.dwk};
  for (int i = 0; i < 2; ++i) s.part[i] = p.s[i].part, s.dw[i] = dw[i], s.n[i] = ctas[i];
  // a programmatic dependent launch: scheduled while the backward drains
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.D / 8, 2);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.dtype == S2ATTN_BF16) return cudaLaunchKernelEx(&cfg, nr::dw_sum_kernel<__nv_bfloat16>, s);
  if (a.dtype == S2ATTN_FP16) return cudaLaunchKernelEx(&cfg, nr::dw_sum_kernel<__half>, s);
  return cudaLaunchKernelEx(&cfg, nr::dw_sum_kernel<float>, s);
}

}  // namespace s2
