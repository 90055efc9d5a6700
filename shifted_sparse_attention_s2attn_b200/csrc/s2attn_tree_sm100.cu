// s2attn_tree_sm100.cu -- attention of drafted tokens over a paged cache (sm_100a).
//
// A decoding step checks M drafted tokens of each of B sequences at once.  Query m of
// sequence b sees every one of the cache's len[b] tokens and those drafted tokens j whose
// bit is set in row m of a mask (a tree's ancestors; without a mask j <= m):
//   o_m = sum_j softmax_j(q_m . k_j / sqrt(D)) v_j
// H query heads share Hkv key heads in groups of `group`, so one key head serves
// M * group query rows: rows (m, g) of up to 128 / group tokens make a 128-row tile of
// the tensor cores' M dimension.
//
// The step reads 2 * len * Hkv * D elements of K and V once and does 4 * D flops an
// element pair and row: bound by HBM up to about a hundred rows a key head, by the tensor
// and exponential units beyond.  The layout follows from the first case:
//   * unit = (key head, row tile); its work is the concatenation of all sequences' key
//     tiles (64 keys: first the cache's, then the drafted ones).  J CTAs share a unit and
//     each takes an equal run of that concatenation, found on the device from len: no
//     length is needed on the host (a captured graph follows growing sequences), and
//     sequences of any mix of lengths load every CTA alike.  A run covers the end of one
//     sequence, whole ones, and the start of another ("segments"); a sequence that lies in
//     one run is written out at once, one that spans runs leaves a partial (max, sum,
//     unnormalised output) per run, at most two per CTA, for the combine kernel.
//   * CTAs of the same run and different heads are neighbours in the grid, so that the
//     heads of a token are read at about the same time and DRAM pages are read in full.
//   * K and V stream by TMA, each through a ring and from a warp of its own; a page of at
//     least 64 tokens is one box per 64 columns, smaller pages one box each.
//   * S = Q K^T in TMEM (two buffers), the softmax's P written back over S in 16 bits, O += P V
//     from TMEM.  S and P V are issued by a warp each, so that S(i+1) runs as soon as P(i-1) V(i-1)
//     has left its buffer, while the softmax works on S(i).  Two CTAs share an SM (256 TMEM
//     columns and 106 KB of shared memory each).
// Measured (B200, bf16, D = 128; bytes: K and V once; both kernels; first back to back in a captured
// graph, then as calls among other work with cold caches):
//   one token, 32k cached, 32 + 32 heads      89-90 us, 0.91 of the copy bandwidth; 99-104 us, 0.79-0.83
//   16 sequences of 100 to 16384 tokens, up to 32 drafted, 32 heads over 8, pages of 16
//                                             65-66 us, 4.1-4.2 TB/s, 12 us of start and join; 72-75 us
//   100k cached, 64 drafted, 64 heads over 8  207-211 us, 1.02-1.04 PFLOP/s, 0.62-0.63 of the burst rate;
//                                             242-249 us, 0.86-0.89 PFLOP/s
//   the same with D = 64                      179-187 us, 0.58-0.60 PFLOP/s
//   two chats of at most 300 tokens, D = 64   12 us with their mask: start, one tile, join; 22-23 us
// 100k is bound by the chain of a tile (S, row max, exponentials, P V): 128-key tiles
// with one S buffer and four or eight softmax warps took 224 and 233 us where this took 226, and
// a share of the exponentials on the FMA pipe (a quarter, a third, a half) 210, 212 and 224 where
// this took 207.  Its N = 64 MMAs cost as much as N = 128 ones (A is read from shared memory at
// each): the tensor pipe is active 55 % of the cycles.
// P is rounded to the input's 16-bit type (the tensor cores take both operands in one type);
// its sum is kept from the unrounded fp32 values.  Scores, maxima, sums and O are fp32.  fp16
// holds nothing below 2^-25, so P is scaled there to a largest element of 2^11 at least (kShift).
//
// Keys that nobody may see are never multiplied: V rows behind the last token of a tile are
// zeroed in shared memory (0 * NaN is NaN), and a drafted V row that holds infinities or NaN
// reaches only the rows whose mask shows it (its elements are zeroed for the product and
// added back to those rows).
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

#include "s2_internal.h"
#include "s2_ptx.cuh"
#include "s2attn.h"

namespace s2 {
namespace tree {

constexpr int BM = 128, BN = 64;
constexpr int KST = 2, VST = 2;              // ring stages
constexpr int NTHREADS = 256;
constexpr int WARP_K = 4, WARP_V = 5, WARP_S = 6, WARP_PV = 7;
static_assert(NTHREADS == 32 * (WARP_PV + 1), "four softmax warps, then these");
constexpr uint32_t QBOX = BM * 128;          // 128 rows x 128 B (64 columns)
constexpr uint32_t KBOX = BN * 128;
constexpr int NBARS = 2 + 2 * KST + 2 * VST + 3 * 2 + 3 + 2;
// What a sequence's end costs, in key tiles.  With 1, 2, 3, 4, 5: two short chats 11.3, 12.0, 12.0, 12.3, 12.8 us;
// the batch of 16 64.4, 65.2, 65.3, 64.9, 65.4; 256 sequences of up to 2000 tokens 119.9, 115.3, 110.7, 108.5, 109.5.
constexpr int kSeqCost = 3;
constexpr uint32_t TM_COLS = 256;
constexpr uint32_t TM_O = 128;               // S buffers at columns 0 and 64

template <int HD>
struct Cfg {
  static constexpr int NB = HD / 64;         // 64-column boxes of a row
  static constexpr uint32_t QTILE = NB * QBOX, KTILE = NB * KBOX;
  static constexpr uint32_t OFF_K = QTILE;
  static constexpr uint32_t OFF_V = OFF_K + KST * KTILE;
  static constexpr uint32_t OFF_BAR = OFF_V + VST * KTILE;
  static constexpr uint32_t OFF_MISC = OFF_BAR + NBARS * 8;   // tmem address, abort flag, run
  static constexpr uint32_t OFF_LEN = OFF_MISC + 128;         // int len[kTreeMaxB], then new[kTreeMaxB]
  static constexpr uint32_t SMEM = OFF_LEN + 2 * kTreeMaxB * 4;
  static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two CTAs must fit on an SM");
};

struct Params {
  void* o;
  float* lse;
  float* part_o;     // [U * J][2][HD/4][slot_rows][4]: neighbouring rows' pieces side by side
  float* part_ml;    // [U * J][2][slot_rows][2]
  int* meta;         // [B * RT][2]: first and last run of a sequence
  const int* len;
  const int* new_len;
  const int* table;
  const unsigned long long* mask;
  const void* v_new;
  int B, M, H, Hkv, group, RT, tok, J, slot_rows;
  int page_shift, n_pages, width, words;
  float sl2;         // log2(e) / sqrt(D)
  int* err;
  int* index_err;
};

enum Site : int { SITE_LOAD = 1, SITE_MMA = 2, SITE_SOFTMAX = 3, SITE_DRAIN = 4, SITE_ALIGN = 5, SITE_STORE = 6 };

__device__ __forceinline__ int cap_tokens(const Params& p) {
  const long long c = (long long)p.width << p.page_shift;
  return c > 0x7fffff00LL ? 0x7fffff00 : (int)c;
}

// Key tiles of the cache, and of the drafted tokens, that sequence b contributes.
__device__ __forceinline__ int cache_tiles(int len) { return (int)(((long long)len + BN - 1) / BN); }
__device__ __forceinline__ int all_tiles(int len, int nw, int first_tok) {
  return nw > first_tok ? cache_tiles(len) + (nw + BN - 1) / BN : 0;
}

// Keys of tile t of a sequence.
__device__ __forceinline__ int tile_keys(int t, int len, int nw) {
  const int ct = cache_tiles(len);
  return t < ct ? min(BN, len - t * BN) : min(BN, nw - (t - ct) * BN);
}

// Walks the segments of a run: `b` and its tiles [t0, t0 + n) of `total`.
struct Segments {
  const int* len;
  const int* nw;
  int first_tok, b, t0, n, total, left;
  __device__ __forceinline__ Segments(const int* len_, const int* nw_, int first, int b_, int t_, int left_)
      : len(len_), nw(nw_), first_tok(first), b(b_), t0(t_), n(0), total(0), left(left_) {}
  __device__ __forceinline__ bool next() {
    if (n) {       // leave the current segment
      ++b;
      t0 = 0;
    }
    if (left <= 0) return false;
    while ((total = all_tiles(len[b], nw[b], first_tok)) == 0) ++b;
    n = min(left, total - t0);
    left -= n;
    return true;
  }
};

// A wait that ends the same way for every lane of the warp: by one lane's poll, or by all.
__device__ __forceinline__ bool wait_lane0(uint64_t* bar, uint32_t parity, int lane, volatile int* abort,
                                           const int* gerr) {
  int ok = 1;
  if (lane == 0) ok = wait_bounded(bar, parity, abort, gerr);
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, const int* gerr) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort, gerr));
}

// Columns [4 * piece, 4 * piece + 4) of row r of a partial (partials exist where a unit has several
// runs, of which the plan makes at most two waves: their pieces fit 32 bits).
template <int HD>
__device__ __forceinline__ float4* part_at(const Params& p, int slot, int piece, int r) {
  return reinterpret_cast<float4*>(p.part_o) + ((slot * (HD / 4) + piece) * p.slot_rows + r);
}
// True in one lane of the warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(x));
  return x != 0;
}

// S[128 x 64] = Q K^T, both K-major.
template <int HD>
__device__ __forceinline__ void issue_s(uint32_t d, uint32_t sq, uint32_t sk, uint32_t idesc) {
  const uint64_t dq = sdesc_sw128(sq, 16, 1024), dk = sdesc_sw128(sk, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < HD / 16; ++kk)
    mma_ss(d, sdesc_add(dq, (kk / 4) * QBOX + (kk % 4) * 32), sdesc_add(dk, (kk / 4) * KBOX + (kk % 4) * 32), idesc,
           kk > 0 ? 1u : 0u);
}

// O[128 x HD] (+)= P V over 16 * KSTEPS keys: P from TMEM, V seen MN-major.
template <int KSTEPS>
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t tp, uint32_t sv, uint32_t idesc, bool first) {
  const uint64_t dv = sdesc_sw128(sv, KBOX, 1024);
#pragma unroll
  for (int kk = 0; kk < KSTEPS; ++kk)
    mma_ts(d, tp + kk * 8, sdesc_add(dv, kk * 2048), idesc, (first && kk == 0) ? 0u : 1u);
}

// P = exp2(s log2(e) / sqrt(D) - m + kShift), with a running maximum m that moves only when it grows by
// more than kLag: P stays at or below 2^(kLag + kShift), inside the type's range.  fp16 ends at
// 2^16 and loses what is below 2^-25: shifted by 11 that is 2^-36 of the row's largest weight, and 100k keys
// of such weights 2^-19 (unshifted, one key 17.5 nats ahead of 100k others took them out of o).
// The sum and O carry the same factor; the maximum that leaves the run is m - kShift.
// Measured in fp16 (100k cached, 64 drafted, 64 heads over 8): 220 us as unshifted with a lag of 8, and
// as a lag of 8 with a shift of 7; with scores three times as wide, whose maximum moves more
// often, 230 against 225, which buys 2^-36 for 2^-32.
template <bool FP16>
constexpr float kLag = FP16 ? 4.0f : 8.0f;
template <bool FP16>
constexpr float kShift = FP16 ? 11.0f : 0.0f;

template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if (FP16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  return pack_bf16x2(lo, hi);
}
template <bool FP16>
__device__ __forceinline__ float unpack16(uint16_t x) {
  if (FP16) {
    const __half_raw r = {x};
    return __half2float(__half(r));
  }
  return __uint_as_float((uint32_t)x << 16);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// P row = exp2(s * sl2 + neg_m), zero in columns whose bit of (lo, hi) is clear (MASK), as 16-bit
// pairs over the first 32 columns of the row's S buffer; returns the fp32 row sum.
template <bool FP16, bool MASK>
__device__ __forceinline__ float p_row(const uint32_t (&sr)[64], uint32_t lo, uint32_t hi, float sl2, float neg_m,
                                       uint32_t t_s) {
  const float2 scale2 = make_float2(sl2, sl2), shift2 = make_float2(neg_m, neg_m);
  float2 sp[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sp[e] = make_float2(0.f, 0.f);
  uint32_t pk[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const float2 x =
        __ffma2_rn(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), scale2, shift2);
    float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    if (MASK) {
      const uint32_t w = c < 16 ? lo : hi;
      e.x = (w >> (2 * c % 32)) & 1u ? e.x : 0.f;
      e.y = (w >> (2 * c % 32 + 1)) & 1u ? e.y : 0.f;
    }
    sp[c % 4] = __fadd2_rn(sp[c % 4], e);
    pk[c] = pack16<FP16>(e.x, e.y);
  }
  tmem_st_x32(t_s, pk);
  const float2 a = __fadd2_rn(__fadd2_rn(sp[0], sp[1]), __fadd2_rn(sp[2], sp[3]));
  return a.x + a.y;
}

// Clears V rows behind the `keep` of a tile that the product reads (it goes in steps of 16) and,
// with `scan`, the elements of the others that are infinite or NaN, whose rows it notes in bad[2].  Row r of column box x lies at
// x * KBOX + r * 128 whatever the swizzle, which only permutes 16-byte pieces of the row.
template <int HD, bool FP16>
__device__ __forceinline__ void clean_v(uint8_t* v, int keep, bool scan, uint32_t* bad, int tid, int nthreads) {
  const uint32_t exp_mask = FP16 ? 0x7c00u : 0x7f80u;
  const int rows = (keep + 15) & ~15;
  for (int i = tid; i < rows * (HD / 8); i += nthreads) {
    const int c = i % (HD / 8), r = i / (HD / 8);   // c: 16-byte piece of the row
    uint4* at = reinterpret_cast<uint4*>(v + (c / 8) * KBOX + r * 128 + (c % 8) * 16);
    if (r >= keep) {
      *at = make_uint4(0, 0, 0, 0);
    } else if (scan) {
      uint4 u = *at;
      uint32_t* w = reinterpret_cast<uint32_t*>(&u);
      bool any = false;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((w[e] & exp_mask) == exp_mask) w[e] &= 0xffff0000u, any = true;
        if (((w[e] >> 16) & exp_mask) == exp_mask) w[e] &= 0x0000ffffu, any = true;
      }
      if (any) {
        *at = u;
        atomicOr(&bad[r / 32], 1u << (r % 32));
      }
    }
  }
}

template <int HD, bool FP16>
__global__ void __launch_bounds__(NTHREADS, 2)
    tree_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tkp,
                const __grid_constant__ CUtensorMap tvp, const __grid_constant__ CUtensorMap tkn,
                const __grid_constant__ CUtensorMap tvn, const Params p) {
  using C = Cfg<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = k_full + KST;
  uint64_t* v_full = k_empty + KST;
  uint64_t* v_empty = v_full + VST;
  uint64_t* s_full = v_empty + VST;     // [2]
  uint64_t* p_ready = s_full + 2;       // [2]
  uint64_t* pv_done = s_full + 4;       // [2]
  uint64_t* o_full = s_full + 6;
  uint64_t* o_free = s_full + 7;
  uint64_t* noted = s_full + 8;         // drafted rows with inf/NaN are noted
  uint64_t* drain = s_full + 9;         // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  int* run = reinterpret_cast<int*>(smem + C::OFF_MISC + 8);        // first sequence, its first tile, tiles
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 32);  // [3][4]: drafted rows with inf/NaN
  int* s_len = reinterpret_cast<int*>(smem + C::OFF_LEN);
  int* s_new = s_len + kTreeMaxB;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int U = p.Hkv * p.RT;
  const int u = (int)blockIdx.x % U, j = (int)blockIdx.x / U;
  const int kvh = u / p.RT, rt = u % p.RT;
  const int first_tok = rt * p.tok;                              // the row tile's first drafted token
  const int tile_toks = min(p.tok, p.M - first_tok);
  const int n_act = (tile_toks * p.group + 31) / 32;             // softmax warps with rows

  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) report_error(p.err, (K_TREE << 8) | SITE_ALIGN);
    return;
  }
  if (warp == WARP_K && lane == 0) {
    prefetch_tmap(&tq);
    prefetch_tmap(&tkp);
    prefetch_tmap(&tkn);
  }
  if (warp == WARP_V && lane == 0) {
    prefetch_tmap(&tvp);
    prefetch_tmap(&tvn);
  }
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_ready[s], n_act);
      mbar_init(&pv_done[s], 1);
      mbar_init(&drain[s], 1);
    }
    mbar_init(o_full, 1);
    mbar_init(o_free, n_act);
    mbar_init(noted, n_act);
    *abort_flag = (*(volatile int*)p.err != 0) ? 1 : 0;
    for (int i = 0; i < 12; ++i) bad[i] = 0;
    fence_mbar_init();
  }
  if (warp == WARP_S) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  if (warp == 0) {
    // The lengths, clamped to what the tables can hold.  They are read once, eight a lane in flight, and
    // a lane reads back only what it has stored: the run below and all segments come from the same
    // numbers whatever becomes of the lengths meanwhile, and one barrier does for all of the set-up.
    // A sequence weighs its tiles and kSeqCost more: what its end costs (masked tiles, the
    // output, the next Q).
    constexpr int AHEAD = 8;
    const int cap = cap_tokens(p);
    int sum = 0, weight = 0;       // the host has checked that these fit
    for (int base = lane; base < p.B; base += 32 * AHEAD) {
      int len[AHEAD], nw[AHEAD];
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int b = base + 32 * e;
        len[e] = b < p.B ? p.len[b] : 0;
        nw[e] = b < p.B && p.new_len ? p.new_len[b] : p.M;
      }
#pragma unroll
      for (int e = 0; e < AHEAD; ++e) {
        const int b = base + 32 * e;
        if (b >= p.B) break;
        const int cached = min(max(len[e], 0), cap), drafted = min(max(nw[e], 0), p.M);
        s_len[b] = cached;
        s_new[b] = drafted;
        if (cached != len[e] || drafted != nw[e]) report_error(p.index_err, (K_TREE << 8) | SITE_INDEX);
        const int n = all_tiles(cached, drafted, first_tok);
        sum += n;
        weight += n ? n + kSeqCost : 0;
      }
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    weight = __reduce_add_sync(0xffffffffu, weight);
    // this CTA's run: the tiles of an equal share of the weights
    const int runs = min(p.J, max(1, sum));
    const int each = weight / runs, more = weight - each * runs;   // the first `more` shares are one larger
    const int w0 = each * j + min(j, more), w1 = w0 + each + (j < more ? 1 : 0);
    // the sequence and tile that w0 falls on, and the tiles before w0 and w1
    int b0 = 0, t0 = 0, at0 = -1, at1 = -1, tiles_before = 0, weight_before = 0;
    for (int base = 0; base < p.B && j < runs; base += 32) {
      const int b = base + lane;
      const int n = b < p.B ? all_tiles(s_len[b], s_new[b], first_tok) : 0;
      int ti = n, wi = n ? n + kSeqCost : 0;      // inclusive sums over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ti, o), y = __shfl_up_sync(0xffffffffu, wi, o);
        if (lane >= o) ti += x, wi += y;
      }
      const int ws = weight_before + wi - (n ? n + kSeqCost : 0), ts = tiles_before + ti - n;
      const unsigned h0 = __ballot_sync(0xffffffffu, weight_before + wi > w0);
      if (at0 < 0 && h0) {
        const int f = __ffs(h0) - 1;
        const int tile = min(n, w0 - ws);         // in lane f; n: the sequence's end
        b0 = base + f;
        t0 = __shfl_sync(0xffffffffu, tile, f);
        at0 = __shfl_sync(0xffffffffu, ts + tile, f);
        if (t0 == __shfl_sync(0xffffffffu, n, f)) t0 = 0, ++b0;
      }
      const unsigned h1 = __ballot_sync(0xffffffffu, weight_before + wi > w1);
      if (h1) {
        const int f = __ffs(h1) - 1;
        at1 = __shfl_sync(0xffffffffu, ts + min(n, w1 - ws), f);
        break;
      }
      weight_before += __shfl_sync(0xffffffffu, wi, 31);
      tiles_before += __shfl_sync(0xffffffffu, ti, 31);
    }
    if (at0 < 0) at0 = sum;      // no tile is left for this run
    if (at1 < 0) at1 = sum;
    if (lane == 0) {
      run[0] = b0;
      run[1] = t0;
      run[2] = j < runs ? at1 - at0 : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_tiles = run[2];
  const bool skip = *abort_flag != 0 || n_tiles == 0;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Segments seg(s_len, s_new, first_tok, run[0], run[1], n_tiles);

  if (!skip && (warp == WARP_K || warp == WARP_V)) {
    // ---------------- producers: Q and K, or V ----------------
    const bool is_k = warp == WARP_K;
    const CUtensorMap* mp = is_k ? &tkp : &tvp;
    const CUtensorMap* mn = is_k ? &tkn : &tvn;
    uint64_t* full = is_k ? k_full : v_full;
    uint64_t* empty = is_k ? k_empty : v_empty;
    uint8_t* ring = smem + (is_k ? C::OFF_K : C::OFF_V);
    constexpr int NST = KST;
    static_assert(KST == VST, "one ring depth");
    const int box_keys = min(1 << p.page_shift, BN);
    const int new_box = min(p.M, BN);
    bool ok = true;
    int i = 0, n_seg = 0;
    while (ok && seg.next()) {
      const int b = seg.b, len = s_len[b], ct = cache_tiles(len);
      const int used = (int)(((long long)len + (1 << p.page_shift) - 1) >> p.page_shift);
      if (is_k) {
        // Q rows (token, head of the group) of the row tile
        if (n_seg > 0) ok = wait_lane0(q_empty, (n_seg - 1) & 1, lane, abort_flag, p.err);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(q_full, C::NB * 128 * p.group * min(p.tok, p.M));
          for (int x = 0; x < C::NB; ++x)
            tma_load_3d(smem + x * QBOX, &tq, x * 64, kvh * p.group, b * p.M + first_tok, q_full);
        }
        ++n_seg;
      }
      // page numbers, 32 at a time, the next 32 on the way
      int base = ((long long)seg.t0 * BN) >> p.page_shift;
      const int* row = p.table + (size_t)b * p.width;
      int ids = base + lane < used ? row[base + lane] : -1;
      int ids_next = base + 32 + lane < used ? row[base + 32 + lane] : -1;
      for (int t = seg.t0; t < seg.t0 + seg.n; ++t, ++i) {
        const int slot = i % NST;
        if (i >= NST) ok = wait_lane0(&empty[slot], ((i / NST) - 1) & 1, lane, abort_flag, p.err);
        if (!ok) break;
        uint8_t* dst = ring + slot * C::KTILE;
        if (t < ct) {
          const int key0 = t * BN;
          const int boxes = (min(BN, len - key0) + box_keys - 1) / box_keys;
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], boxes * C::NB * box_keys * 128);
          for (int x = 0; x < boxes; ++x) {
            const int key = key0 + x * box_keys;
            const int pg = key >> p.page_shift;
            if (pg - base >= 32) {
              base += 32;
              ids = ids_next;
              ids_next = base + 32 + lane < used ? row[base + 32 + lane] : -1;
            }
            int id = __shfl_sync(0xffffffffu, ids, pg - base);
            if (id < 0 || id >= p.n_pages) {   // recorded; the box reads as zeros
              if (lane == 0) report_error(p.index_err, (K_TREE << 8) | SITE_INDEX);
              id = p.n_pages;
            }
            if (lane == 0) {
              const int r = (id << p.page_shift) + (id < p.n_pages ? key & ((1 << p.page_shift) - 1) : 0);
              for (int y = 0; y < C::NB; ++y)
                tma_load_3d(dst + y * KBOX + x * box_keys * 128, mp, y * 64, kvh, r, &full[slot]);
            }
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(&full[slot], C::NB * new_box * 128);
          for (int y = 0; y < C::NB; ++y)
            tma_load_3d(dst + y * KBOX, mn, y * 64, kvh, b * p.M + (t - ct) * BN, &full[slot]);
        }
      }
    }
    if (!ok && lane == 0) {
      report_error(p.err, (K_TREE << 8) | SITE_LOAD);
      *abort_flag = 1;
    }
    if (lane == 0) {
      bool dok = true;
      if (is_k && n_seg > 0) dok &= wait_drain(q_full, (n_seg - 1) & 1);
      for (int s = (i > NST ? i - NST : 0); s < i; ++s) dok &= wait_drain(&full[s % NST], (s / NST) & 1);
      if (!dok) report_error(p.err, (K_TREE << 8) | SITE_DRAIN);
    }
    __syncwarp();
  } else if (!skip && warp >= WARP_S) {
    // ---------------- MMA issuers: S(i) = Q K(i), and P(i) V(i) ----------------
    // A warp each: issuing blocks while the tensor pipe works off what is queued, and with one
    // issuer S(i+1) waited behind P(i-1) V(i-1)'s issue as well as its execution.  Each warp
    // walks the tiles as a whole and one elected lane issues: where the compiler sees that one
    // lane runs, an MMA's operands go straight to uniform registers.
    const bool is_s = warp == WARP_S;
    const uint32_t fmt = FP16 ? ~((1u << 7) | (1u << 10)) : ~0u;   // A and B formats: 0 = f16, 1 = bf16
    const uint32_t id_s = idesc_bf16_f32(BM, BN, false, false) & fmt;
    const uint32_t id_pv = idesc_bf16_f32(BM, HD, false, true) & fmt;
    const uint32_t sq = smem_u32(smem), sk = smem_u32(smem + C::OFF_K), sv = smem_u32(smem + C::OFF_V);
    bool ok = true;
    int n_seg = 0, left = 0;        // segments begun; tiles left in the current one
    for (int i = 0; i < n_tiles && ok; ++i) {
      const bool first = left == 0;
      if (first) {
        seg.next();
        left = seg.n;
        // the segment's Q is there; O of the segment before has been read
        if (is_s)
          ok = wait_warp(q_full, n_seg & 1, abort_flag, p.err);
        else if (n_seg > 0)
          ok = wait_warp(o_free, (n_seg - 1) & 1, abort_flag, p.err);
        ++n_seg;
      }
      const uint32_t t_s = tmem + (uint32_t)BN * (i & 1);
      if (is_s) {
        if (ok) ok = wait_warp(&k_full[i % KST], (i / KST) & 1, abort_flag, p.err);
        // P of tile i - 2 lies in this S buffer until its product is done
        if (ok && i >= 2) ok = wait_warp(&pv_done[i & 1], ((i >> 1) - 1) & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after();
        --left;
        if (elect_one()) {
          issue_s<HD>(t_s, sq, sk + (i % KST) * C::KTILE, id_s);
          mma_commit(&s_full[i & 1]);
          mma_commit(&k_empty[i % KST]);
          if (left == 0) mma_commit(q_empty);
        }
        __syncwarp();
      } else {
        // a whole tile is one run of MMAs; the last tile's product stops behind its last key
        const int ksteps = (tile_keys(seg.t0 + seg.n - left, s_len[seg.b], s_new[seg.b]) + 15) / 16;
        const uint32_t v0 = sv + (i % VST) * C::KTILE;
        if (ok) ok = wait_warp(&v_full[i % VST], (i / VST) & 1, abort_flag, p.err);
        if (ok) ok = wait_warp(&p_ready[i & 1], (i >> 1) & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after();
        --left;
        if (elect_one()) {
          if (ksteps == BN / 16) {
            issue_pv<BN / 16>(tmem + TM_O, t_s, v0, id_pv, first);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < ksteps; ++kk)
              issue_pv<1>(tmem + TM_O, t_s + kk * 8, v0 + kk * 2048, id_pv, first && kk == 0);
          }
          mma_commit(&pv_done[i & 1]);
          mma_commit(&v_empty[i % VST]);
          if (left == 0) mma_commit(o_full);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      report_error(p.err, (K_TREE << 8) | SITE_MMA);
      *abort_flag = 1;
    }
    if (elect_one()) mma_commit(&drain[is_s ? 0 : 1]);
    __syncwarp();
    if (!wait_drain(&drain[is_s ? 0 : 1], 0) && lane == 0) report_error(p.err, (K_TREE << 8) | SITE_DRAIN);
    __syncwarp();
  } else if (!skip && warp < n_act) {
    // ---------------- softmax: thread = query row ----------------
    const int r = warp * 32 + lane;
    const int m = first_tok + r / p.group;                  // drafted token of the row
    const int h = kvh * p.group + r % p.group;
    const bool in_tile = r < tile_toks * p.group;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    const float sl2 = p.sl2;
    bool ok = true;
    int i = 0, n_seg = 0, n_draft = 0;
    while (ok && seg.next()) {
      const int b = seg.b, len = s_len[b], nw = s_new[b], ct = cache_tiles(len);
      const bool row_ok = in_tile && m < nw;
      uint32_t* bad_rows = bad + 4 * (n_draft % 3);        // of this sequence's drafted tiles
      const bool has_draft = seg.t0 + seg.n > ct;
      // which drafted keys the row sees
      unsigned long long see[2] = {0, 0};
      if (has_draft && row_ok) {
        if (p.mask) {
          const unsigned long long* w = p.mask + ((size_t)b * p.M + m) * p.words;
          see[0] = w[0];
          if (p.words > 1) see[1] = w[1];
        } else {     // j <= m
          see[0] = m >= 63 ? ~0ull : (2ull << m) - 1ull;
          see[1] = m < 64 ? 0ull : m >= 127 ? ~0ull : (2ull << (m - 64)) - 1ull;
        }
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int t = seg.t0; t < seg.t0 + seg.n && ok; ++t, ++i) {
        const int buf = i & 1;
        // keys of the tile, and which of them the row sees
        const bool draft = t >= ct;
        const int keep = tile_keys(t, len, nw);
        const bool edge = draft || keep < BN;
        uint32_t lo = 0xffffffffu, hi = 0xffffffffu;
        ok = wait_warp(&s_full[buf], (i >> 1) & 1, abort_flag, p.err);
        if (!ok) break;
        tc_fence_after();
        if (edge) {
          unsigned long long vis = keep >= 64 ? ~0ull : (1ull << keep) - 1ull;
          if (draft) vis &= t == ct ? see[0] : see[1];
          lo = (uint32_t)vis;
          hi = (uint32_t)(vis >> 32);
          // V(i): only now, behind the wait for S(i).  That was issued after the product that read
          // the slot's last tile, so the slot's barrier is in this tile's phase; before, it might
          // be in the last tile's, and a wait by parity would take the phase before that for this one.
          ok = wait_warp(&v_full[i % VST], (i / VST) & 1, abort_flag, p.err);
          if (!ok) break;
          clean_v<HD, FP16>(smem + C::OFF_V + (i % VST) * C::KTILE, keep, draft, bad_rows + 2 * (draft ? t - ct : 0),
                            threadIdx.x, n_act * 32);
          fence_proxy_async_smem();
        }
        const uint32_t t_s = lane_addr + (uint32_t)BN * buf;
        uint32_t s0[64];
        tmem_ld_x64(t_s, s0);
        float mxp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mxp[e] = -INFINITY;
        if (!edge) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            mxp[c % 8] = max3(mxp[c % 8], __uint_as_float(s0[2 * c]), __uint_as_float(s0[2 * c + 1]));
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint32_t w = c < 16 ? lo : hi;
            mxp[c % 8] = max3(mxp[c % 8], (w >> (2 * c % 32)) & 1u ? __uint_as_float(s0[2 * c]) : -INFINITY,
                              (w >> (2 * c % 32 + 1)) & 1u ? __uint_as_float(s0[2 * c + 1]) : -INFINITY);
          }
        }
        const float mx = fmaxf(fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])),
                               fmaxf(fmaxf(mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7])));
        // the running max moves only when it grows by more than kLag; a row that has seen no score
        // above -inf keeps -inf, and its P = exp2(-inf - 0) stays 0 (-inf - -inf is NaN)
        const float m_new = fmaxf(m_run, mx * sl2);
        const bool need = (m_new - m_run) > kLag<FP16>;
        const bool rescale = __any_sync(0xffffffffu, need);
        const float alpha = need ? ex2_approx(m_run - m_new) : 1.0f;
        if (need) m_run = m_new;
        l_run *= alpha;
        const float neg_m = m_run == -INFINITY ? 0.f : kShift<FP16> - m_run;
        l_run += edge ? p_row<FP16, true>(s0, lo, hi, sl2, neg_m, t_s) : p_row<FP16, false>(s0, lo, hi, sl2, neg_m, t_s);
        if (rescale && t > seg.t0) {
          // O was last written by the previous tile's product: wait for it, then scale the row
          ok = wait_warp(&pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, abort_flag, p.err);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < HD; c += 32) {
            uint32_t rr[32];
            tmem_ld_x32(lane_addr + TM_O + c, rr);
#pragma unroll
            for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st_x32(lane_addr + TM_O + c, rr);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[buf]);
      }
      if (ok) ok = wait_warp(o_full, n_seg & 1, abort_flag, p.err);
      if (!ok) break;
      tc_fence_after();
      uint32_t fix[4] = {0, 0, 0, 0};      // drafted rows with inf/NaN that this row sees
      if (has_draft) {
        // every warp has noted its rows; the notes of the sequence after the next start from
        // zero (all warps have read what is cleared here, none writes it before the next wait)
        if (lane == 0) mbar_arrive(noted);
        ok = wait_warp(noted, n_draft & 1, abort_flag, p.err);
        if (!ok) break;
        if (threadIdx.x < 4) bad[4 * ((n_draft + 2) % 3) + threadIdx.x] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) fix[e] = bad_rows[e] & (uint32_t)(see[e / 2] >> (32 * (e % 2)));
        ++n_draft;
      }
      const bool whole = seg.t0 == 0 && seg.n == seg.total;
      const int slot = (int)blockIdx.x * 2 + (seg.t0 == 0 ? 1 : 0);
      const size_t part = (size_t)slot * p.slot_rows + r;
      const size_t orow = ((size_t)b * p.M + m) * p.H + h;
      const bool st_ok =
          row_ok && (whole ? in_bounds(orow, 1, (size_t)p.B * p.M * p.H, p.err, (K_TREE << 8) | SITE_STORE)
                           : in_bounds(part, 1, (size_t)gridDim.x * 2 * p.slot_rows, p.err, (K_TREE << 8) | SITE_STORE));
      const float inv = l_run > 0.f || l_run != l_run ? 1.0f / l_run : 0.f;   // a row that sees nothing: 0
      // (rolled: code that runs once or twice a launch costs its fetch more than its time)
#pragma unroll 1
      for (int c = 0; c < HD; c += 32) {
        uint32_t rr[32];
        __syncwarp();
        tmem_ld_x32(lane_addr + TM_O + c, rr);
        if (st_ok && whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * HD + c);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t w[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              w[y] = pack16<FP16>(__uint_as_float(rr[8 * x + 2 * y]) * inv, __uint_as_float(rr[8 * x + 2 * y + 1]) * inv);
            dst[x] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else if (st_ok) {
          float4* dst = part_at<HD>(p, slot, c / 4, r);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            dst[(size_t)x * p.slot_rows] = make_float4(__uint_as_float(rr[4 * x]), __uint_as_float(rr[4 * x + 1]),
                                 __uint_as_float(rr[4 * x + 2]), __uint_as_float(rr[4 * x + 3]));
        }
      }
      if (st_ok && (fix[0] | fix[1] | fix[2] | fix[3])) {
        // add the infinities and NaN that clean_v took out, to what this thread has just written
#pragma unroll 1
        for (int key = 0; key < 2 * BN; ++key) {
          const uint32_t w = key < 64 ? (key < 32 ? fix[0] : fix[1]) : (key < 96 ? fix[2] : fix[3]);
          if (!((w >> (key % 32)) & 1u)) continue;
          const uint16_t* v = static_cast<const uint16_t*>(p.v_new) + (((size_t)b * p.M + key) * p.Hkv + kvh) * HD;
#pragma unroll 1
          for (int c = 0; c < HD; ++c) {
            const float f = unpack16<FP16>(v[c]);
            if (isfinite(f)) continue;
            if (whole) {
              uint16_t* at = static_cast<uint16_t*>(p.o) + orow * HD + c;
              *at = (uint16_t)pack16<FP16>(unpack16<FP16>(*at) + f, 0.f);
            } else {
              reinterpret_cast<float*>(part_at<HD>(p, slot, c / 4, r))[c % 4] += f;
            }
          }
        }
      }
      if (st_ok) {
        const float m_out = m_run - kShift<FP16>;
        if (whole) {
          p.lse[((size_t)b * p.H + h) * p.M + m] =
              l_run == 0.f ? -INFINITY : (m_out + log2f(l_run)) * 0.69314718055994531f;
        } else {
          // a row all of whose scores were NaN has no maximum: 0 takes its NaN sum through the join
          p.part_ml[part * 2] = l_run != l_run && m_run == -INFINITY ? 0.f : m_out;
          p.part_ml[part * 2 + 1] = l_run;
        }
      }
      if (kvh == 0 && threadIdx.x == 0) {
        if (seg.t0 == 0) p.meta[(b * p.RT + rt) * 2] = j;
        if (seg.t0 + seg.n == seg.total) p.meta[(b * p.RT + rt) * 2 + 1] = j;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      ++n_seg;
    }
    if (!ok) {
      report_error(p.err, (K_TREE << 8) | SITE_SOFTMAX);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == WARP_S) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

// o = sum_s 2^(m_s - mx) o_s / sum_s 2^(m_s - mx) l_s over the runs s of the row's sequence;
// lse = ln2 * (mx + log2 L).  Rows of a sequence that lay in one run were written by the run.
// A lane joins four columns of one row: block (sequence, unit, 32 rows, 8 / ws pieces of four
// columns).  The runs of a row are dealt to `ws` warps and, where fewer than 32 rows exist, to
// the lanes left over; each keeps a running (max, sum, output) and these are joined at the end.
constexpr int CW = 8;

struct Joined {
  float mx, L;
  float4 o;
};
__device__ __forceinline__ void join(Joined& a, float mx, float L, const float4& o) {
  const float top = fmaxf(a.mx, mx);
  if (top == -INFINITY) return;                 // neither has seen a key
  const float x = ex2_approx(a.mx - top), y = ex2_approx(mx - top);
  a.mx = top;
  a.L = fmaf(a.L, x, L * y);
  a.o = make_float4(fmaf(a.o.x, x, o.x * y), fmaf(a.o.y, x, o.y * y), fmaf(a.o.z, x, o.z * y), fmaf(a.o.w, x, o.w * y));
}

template <int HD, bool FP16>
__global__ void __launch_bounds__(CW * 32) tree_combine_kernel(const __grid_constant__ Params p, int ws, int rp) {
  __shared__ Joined part[CW][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int wc = CW / ws;                                 // pieces of a block
  const int piece = (int)blockIdx.y * wc + warp / ws, split = warp % ws;
  const int groups = (p.slot_rows + rp - 1) / rp, U = p.Hkv * p.RT;
  const int grp = (int)blockIdx.x % groups, u = (int)blockIdx.x / groups % U, b = (int)blockIdx.x / (groups * U);
  const int kvh = u / p.RT, rt = u % p.RT;
  const int r = grp * rp + lane % rp, sub = lane / rp, parts = ws * (32 / rp);
  const int m = rt * p.tok + r / p.group, h = kvh * p.group + r % p.group;
  // launched as a programmatic dependent of the attention kernel: wait for that whole grid
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int nw = p.new_len ? min(p.new_len[b], p.M) : p.M;
  // (the same for the whole block) no row of it exists, or an error ended the attention kernel
  if (nw <= rt * p.tok + grp * rp / p.group || *(volatile int*)p.err != 0) return;
  const int2 fl = *reinterpret_cast<const int2*>(p.meta + (b * p.RT + rt) * 2);
  const int first = max(fl.x, 0), last = min(fl.y, p.J - 1);
  if (first >= last) return;
  const bool live = r < p.slot_rows && m < nw;
  Joined a = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  // run s: slot 1 of CTA (u, first), slot 0 of the later ones
  constexpr int AHEAD = 4;
  for (int s0 = first + split * (32 / rp) + sub; s0 <= last && live; s0 += AHEAD * parts) {
    float2 ml[AHEAD];
    float4 v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int s = s0 + k * parts;
      if (s > last) break;
      const int slot = (s * U + u) * 2 + (s == first ? 1 : 0);
      ml[k] = reinterpret_cast<const float2*>(p.part_ml)[slot * p.slot_rows + r];
      v[k] = *part_at<HD>(p, slot, piece, r);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (s0 + k * parts > last) break;
      join(a, ml[k].x, ml[k].y, v[k]);
    }
  }
  __syncwarp();
  for (int o = rp; o < 32; o <<= 1) {     // the lanes that hold the same row
    Joined x;
    x.mx = __shfl_xor_sync(0xffffffffu, a.mx, o);
    x.L = __shfl_xor_sync(0xffffffffu, a.L, o);
    x.o = make_float4(__shfl_xor_sync(0xffffffffu, a.o.x, o), __shfl_xor_sync(0xffffffffu, a.o.y, o),
                      __shfl_xor_sync(0xffffffffu, a.o.z, o), __shfl_xor_sync(0xffffffffu, a.o.w, o));
    join(a, x.mx, x.L, x.o);
  }
  if (ws > 1) {
    part[warp][lane] = a;
    __syncthreads();
    if (split) return;
    for (int w = 1; w < ws; ++w) {
      const Joined& x = part[warp + w][lane];
      join(a, x.mx, x.L, x.o);
    }
  }
  if (!live || sub) return;
  const float inv = a.mx == -INFINITY ? 0.f : 1.0f / a.L;
  const size_t orow = ((size_t)b * p.M + m) * p.H + h;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + orow * HD + 4 * piece) =
      make_uint2(pack16<FP16>(a.o.x * inv, a.o.y * inv), pack16<FP16>(a.o.z * inv, a.o.w * inv));
  if (piece == 0)
    p.lse[((size_t)b * p.H + h) * p.M + m] =
        a.mx == -INFINITY ? -INFINITY : (a.mx + log2f(a.L)) * 0.69314718055994531f;
}

template <int HD, bool FP16>
cudaError_t launch(const TreeMaps& t, const Params& p, cudaStream_t st) {
  using C = Cfg<HD>;
  // the shared-memory limit is a per-device function attribute: set it once per device
  static std::atomic<uint64_t> done_mask{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (1ull << dev) : 0ull;
  if (!bit || !(done_mask.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(tree_kernel<HD, FP16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    done_mask.fetch_or(bit, std::memory_order_acq_rel);
  }
  const unsigned grid = (unsigned)(p.Hkv * p.RT * p.J);
  tree_kernel<HD, FP16><<<grid, NTHREADS, C::SMEM, st>>>(t.q, t.k_pages, t.v_pages, t.k_new, t.v_new, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.J == 1) return e;   // one run: every sequence was written whole
  cudaLaunchConfig_t cfg = {};
  // a sequence has about J / B runs: with many, four warps share a row's
  const int ws = p.J >= 16 * p.B ? 4 : 1;
  int rp = 1;
  while (rp < 32 && rp < p.slot_rows) rp *= 2;
  const long long blocks = (long long)p.B * p.Hkv * p.RT * ((p.slot_rows + rp - 1) / rp);
  cfg.gridDim = dim3((unsigned)blocks, HD / 4 / (CW / ws));
  cfg.blockDim = dim3(CW * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<HD, FP16>, p, ws, rp);
}

}  // namespace tree

// Row tiles and runs.  A unit's J CTAs should fill one wave of two CTAs an SM, or two where one
// cannot be filled well: the J with the least waves / J (the time of a unit's share times the
// waves), a second wave counted a fifth more for its start and its partials (16 to 32k tokens:
// 50 units, one wave of 250 CTAs 79 us, two of 550 83; 100 units, 200 CTAs 159 us, 500 149).
TreePlan tree_plan(int M, int H, int Hkv) {
  TreePlan t;
  t.group = H / Hkv;
  t.tok = tree::BM / t.group;
  t.RT = (M + t.tok - 1) / t.tok;
  const long long U = (long long)Hkv * t.RT;
  t.slot_rows = (t.tok < M ? t.tok : M) * t.group;
  t.J = 1;
  double best = 1e30;
  for (int J = 1; J == 1 || U * J <= 2 * kTreeSlots; ++J) {
    const double cost = (U * J <= kTreeSlots ? 1.0 : 1.2 * (double)((U * J + kTreeSlots - 1) / kTreeSlots)) / J;
    if (cost < best - 1e-9) {
      best = cost;
      t.J = J;
    }
  }
  return t;
}

cudaError_t launch_tree_decode(const TreeMaps& maps, const TreeArgs& a, const TreePlan& t, cudaStream_t st) {
  tree::Params p{};
  p.o = a.o, p.lse = a.lse, p.part_o = a.part_o, p.part_ml = a.part_ml, p.meta = a.meta;
  p.len = a.cache_len, p.new_len = a.new_len, p.table = a.page_table, p.mask = a.mask, p.v_new = a.v_new;
  p.B = a.B, p.M = a.M, p.H = a.H, p.Hkv = a.Hkv, p.group = t.group, p.RT = t.RT, p.tok = t.tok, p.J = t.J;
  p.slot_rows = t.slot_rows;
  p.page_shift = a.page_shift, p.n_pages = a.n_pages, p.width = a.width, p.words = (a.M + 63) / 64;
  p.sl2 = (float)(1.4426950408889634 / std::sqrt((double)a.D));
  p.err = a.err, p.index_err = a.index_err;
  const bool fp16 = a.dtype == S2ATTN_FP16;
  if (a.D == 128) return fp16 ? tree::launch<128, true>(maps, p, st) : tree::launch<128, false>(maps, p, st);
  return fp16 ? tree::launch<64, true>(maps, p, st) : tree::launch<64, false>(maps, p, st);
}

}  // namespace s2
