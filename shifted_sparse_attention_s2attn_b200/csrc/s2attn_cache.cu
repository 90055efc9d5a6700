// s2attn_cache.cu -- the paged key/value cache: new rows to their pages, page copies, and
// the ancestor masks of drafted-token trees.
//
// The copies are HBM-bound: each byte is read once and written once.  A thread moves four
// 16-byte pieces (of K and of V, when appending) and has all loads in flight before the first
// store.  Measured (B200): 32k tokens of 8 heads x 128 in bf16 appended in 43-46 us = 5.8-6.2 TB/s, 0.89-0.95
// of the copy bandwidth (59 us when every piece looked its row up); 500 pages of 131 KB copied in
// four pools in 84-90 us = 5.8-6.2 TB/s; 8 pages in 32 pools, and 32 sequences' accepted rows, in 3-4 us.
#include <algorithm>

#include "s2_internal.h"
#include "s2_ptx.cuh"

namespace s2 {
namespace cache {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;
constexpr int MAX_SLOTS = 256;   // of a block of the append kernel

struct AppendArgs {
  const uint4 *k_new, *v_new;  // [B, M, Hkv, D]
  uint4 *k_pages, *v_pages;  // [n_pages, page_size, Hkv, D]
  const int* table;          // [B, width]
  const int* len;            // [B]
  const int* rows;           // [B, A] or NULL: row j is new row j
  const int* n_rows;         // [B] or NULL: A rows each
  int B, M, A, width, n_pages, page_shift;
  int cpr;                   // 16-byte pieces of a row
  int tpb;                   // (sequence, row) slots a block takes
  int* index_err;
};

// Slot t = (b, j) of a block's `tpb`: its rows of k_new and v_new are found by one thread (a row
// outside the new rows, a negative length, a position outside the table or a page outside the
// pool is recorded and skipped), then all threads copy the slots' rows.
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ long long s_src[MAX_SLOTS], s_dst[MAX_SLOTS];   // first piece of the row; -1: no row
  const long long slot0 = (long long)blockIdx.x * a.tpb;
  const int slots = (int)min((long long)a.tpb, (long long)a.B * a.A - slot0);
  for (int i = threadIdx.x; i < slots; i += THREADS) {
    const long long slot = slot0 + i;
    const int b = (int)(slot / a.A), j = (int)(slot - (long long)b * a.A);
    long long src = -1, dst = -1;
    if (!a.n_rows || j < a.n_rows[b]) {
      const int row = a.rows ? a.rows[slot] : j;
      const int len = a.len[b];
      const long long pos = (long long)len + j, pg = pos >> a.page_shift;
      int page = -1;
      if (row >= 0 && row < a.M && len >= 0 && pg < a.width) page = a.table[(size_t)b * a.width + pg];
      if (page >= 0 && page < a.n_pages) {
        src = ((long long)b * a.M + row) * a.cpr;
        dst = (((long long)page << a.page_shift) + (pos & ((1 << a.page_shift) - 1))) * a.cpr;
      } else {
        report_error(a.index_err, (K_CACHE << 8) | SITE_INDEX);
      }
    }
    s_src[i] = src;
    s_dst[i] = dst;
  }
  __syncthreads();
  const int n = slots * a.cpr;
  for (int i0 = threadIdx.x; i0 < n; i0 += THREADS * UNROLL) {
    uint4 k[UNROLL], v[UNROLL];
    long long to[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int i = i0 + u * THREADS;
      to[u] = -1;
      if (i >= n) continue;
      const int s = i / a.cpr, c = i - s * a.cpr;
      if (s_dst[s] < 0) continue;
      to[u] = s_dst[s] + c;
      k[u] = a.k_new[s_src[s] + c];
      v[u] = a.v_new[s_src[s] + c];
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u)
      if (to[u] >= 0) {
        a.k_pages[to[u]] = k[u];
        a.v_pages[to[u]] = v[u];
      }
  }
}

struct CopyArgs {
  uint4* pool[kCacheMaxPools];
  int2 pair[kCacheCopyPairs];
  long long pieces;          // 16-byte pieces of a page
};

// blockIdx.x: a run of THREADS * UNROLL pieces, y: pair, z: pool.
__global__ void __launch_bounds__(THREADS) copy_kernel(const __grid_constant__ CopyArgs a) {
  uint4* pool = a.pool[blockIdx.z];
  const int2 pr = a.pair[blockIdx.y];
  const uint4* src = pool + (long long)pr.x * a.pieces;
  uint4* dst = pool + (long long)pr.y * a.pieces;
  const long long i0 = (long long)blockIdx.x * (THREADS * UNROLL) + threadIdx.x;
  uint4 v[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u)
    if (i0 + u * THREADS < a.pieces) v[u] = src[i0 + u * THREADS];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u)
    if (i0 + u * THREADS < a.pieces) dst[i0 + u * THREADS] = v[u];
}

// Ancestor sets of a tree by pointer doubling: after step k a node holds itself and its
// 2^k - 1 nearest ancestors, and points 2^k up.  One block a tree, one thread a node.
__global__ void __launch_bounds__(kTreeMaxM) tree_mask_kernel(const int* parents, unsigned long long* mask,
                                                              int* depth, int M, int words, int* index_err) {
  __shared__ unsigned long long set[2][2][kTreeMaxM];
  __shared__ int up[2][kTreeMaxM];
  const int m = threadIdx.x;
  const size_t row = (size_t)blockIdx.x * M + m;
  if (m < M) {
    int par = parents[row];
    if (par < -1 || par >= m) {
      report_error(index_err, (K_TREE << 8) | SITE_INDEX);
      par = -1;
    }
    up[0][m] = par;
    set[0][0][m] = m < 64 ? 1ull << m : 0ull;
    set[0][1][m] = m < 64 ? 0ull : 1ull << (m - 64);
  }
  __syncthreads();
  int cur = 0;
  for (int span = 1; span < M; span *= 2) {
    if (m < M) {
      const int par = up[cur][m];
      set[cur ^ 1][0][m] = set[cur][0][m] | (par >= 0 ? set[cur][0][par] : 0ull);
      set[cur ^ 1][1][m] = set[cur][1][m] | (par >= 0 ? set[cur][1][par] : 0ull);
      up[cur ^ 1][m] = par >= 0 ? up[cur][par] : -1;
    }
    cur ^= 1;
    __syncthreads();
  }
  if (m < M) {
    for (int w = 0; w < words; ++w) mask[row * words + w] = set[cur][w][m];
    if (depth) depth[row] = __popcll(set[cur][0][m]) + __popcll(set[cur][1][m]) - 1;
  }
}

}  // namespace cache

cudaError_t launch_cache_append(const void* k_new, const void* v_new, void* k_pages, void* v_pages, const int* table,
                                const int* len, const int* rows, const int* n_rows, int B, int M, int A, int width,
                                int n_pages, int page_shift, int row_bytes, int n_sm, int* index_err, cudaStream_t st) {
  cache::AppendArgs a{};
  a.k_new = static_cast<const uint4*>(k_new), a.v_new = static_cast<const uint4*>(v_new);
  a.k_pages = static_cast<uint4*>(k_pages), a.v_pages = static_cast<uint4*>(v_pages);
  a.table = table, a.len = len, a.rows = rows, a.n_rows = n_rows;
  a.B = B, a.M = M, a.A = A, a.width = width, a.n_pages = n_pages, a.page_shift = page_shift;
  a.cpr = row_bytes / 16;
  // one step of the block's threads, fewer slots where that leaves SMs without a block
  const int per_block = cache::THREADS * cache::UNROLL;
  const long long slots = (long long)B * A;
  a.tpb = (int)std::max(1LL, std::min({(long long)per_block / a.cpr, (long long)cache::MAX_SLOTS, slots / n_sm}));
  a.index_err = index_err;
  const long long blocks = (slots + a.tpb - 1) / a.tpb;
  cache::append_kernel<<<(unsigned)blocks, cache::THREADS, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_copy(void* const* pools, int n_pools, const int* pairs, int n_pairs, long long page_bytes,
                              cudaStream_t st) {
  cache::CopyArgs a{};
  for (int i = 0; i < n_pools; ++i) a.pool[i] = static_cast<uint4*>(pools[i]);
  a.pieces = page_bytes / 16;
  const long long per_block = cache::THREADS * cache::UNROLL;
  const unsigned gx = (unsigned)((a.pieces + per_block - 1) / per_block);
  for (int p0 = 0; p0 < n_pairs; p0 += kCacheCopyPairs) {
    const int n = n_pairs - p0 < kCacheCopyPairs ? n_pairs - p0 : kCacheCopyPairs;
    for (int i = 0; i < n; ++i) a.pair[i] = make_int2(pairs[2 * (p0 + i)], pairs[2 * (p0 + i) + 1]);
    cache::copy_kernel<<<dim3(gx, n, n_pools), cache::THREADS, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_tree_mask(const int* parents, unsigned long long* mask, int* depth, int B, int M, int* index_err,
                             cudaStream_t st) {
  cache::tree_mask_kernel<<<B, kTreeMaxM, 0, st>>>(parents, mask, depth, M, (M + 63) / 64, index_err);
  return cudaGetLastError();
}

}  // namespace s2
