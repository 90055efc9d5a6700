// s2attn_capi.cu -- the extern "C" boundary: argument validation, tensor-map
// construction, the RoPE table cache, the device error word, and kernel launches.
#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>
#include <vector>

#include "s2_internal.h"
#include "s2_ptx.cuh"
#include "s2attn.h"

namespace {

// [0]: the first failure inside a kernel (later kernels skip their work while it is set);
// [1]: the first index out of range (recorded only).
__device__ int g_error_word[2];

constexpr int kMaxDevices = 64;

// ---- error word -----------------------------------------------------------------
int* error_word_ptr() {
  static std::mutex mu;
  static int* cache[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_error_word) != cudaSuccess) return nullptr;
    cache[dev] = static_cast<int*>(p);
  }
  return cache[dev];
}

// ---- tensor maps ----------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A [B,N,H,D] tensor viewed as 3-D {D, H, B*N}; a box is box_rows tokens x box_cols
// elements of one head.
bool make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, size_t esize, int B, int N, int H, int D,
              uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle sw) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)B * (cuuint64_t)N};
  cuuint64_t strides[2] = {(cuuint64_t)D * esize, (cuuint64_t)H * D * esize};
  cuuint32_t box[3] = {box_cols, 1, box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool map_bf16_sw128(CUtensorMap* m, const void* base, const s2::Shape& s, uint32_t rows) {
  return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, s.B, s.N, s.H, s.D, 64, rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// A row-major bf16 matrix [outer, inner] (rank 2), or a stack [d2, outer, inner] (rank 3,
// boxes one matrix deep), with 128-byte swizzled boxes of box_inner x box_outer elements;
// out-of-range elements read as zero.  The rank must match the kernel's load instruction.
bool map_rows_bf16(CUtensorMap* m, const void* base, int rank, uint64_t inner, uint64_t outer, uint64_t d2,
                   uint32_t box_inner, uint32_t box_outer) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {inner, outer, d2};
  cuuint64_t strides[2] = {inner * 2, inner * outer * 2};
  cuuint32_t box[3] = {box_inner, box_outer, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  if (rank != 2 && rank != 3) return false;
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ---- validation -----------------------------------------------------------------
bool aligned16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_shape(int B, int N, int H, int D, int G, int shift_heads) {
  if (B < 1 || N < 1 || H < 1 || D < 1 || G < 1) return S2ATTN_ERR_INVALID_ARG;
  if (N % G != 0) return S2ATTN_ERR_INVALID_ARG;
  if (shift_heads < 0 || shift_heads > H) return S2ATTN_ERR_INVALID_ARG;
  if (shift_heads > 0 && (G % 2) != 0) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)B * N > INT_MAX / 2) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)B * N * H > (LLONG_MAX / 8) / D) return S2ATTN_ERR_INVALID_ARG;
  return S2ATTN_OK;
}

int check_tensor_core_shape(int B, int N, int H, int D, int G, int shift_heads) {
  int rc = check_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (D != 128) return S2ATTN_ERR_UNSUPPORTED;
  if (G % 128 != 0) return S2ATTN_ERR_UNSUPPORTED;
  if (shift_heads > 0 && (G / 2) % 128 != 0) return S2ATTN_ERR_UNSUPPORTED;
  if ((long long)B * H * (N / G) * (G / 128) > INT_MAX) return S2ATTN_ERR_UNSUPPORTED;
  return S2ATTN_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? S2ATTN_OK : S2ATTN_ERR_CUDA; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// ---- RoPE tables ------------------------------------------------------------------
struct RopeTable {
  float* cos_d = nullptr;
  float* sin_d = nullptr;
};

// theta_i = (float) base^(-2i/D) (pow in double); a = ((float)t * pos_scale) * theta_i in
// float; table entries (float) cos((double)a), (float) sin((double)a).
int rope_table(int dev, int N, int D, float pos_scale, float base, RopeTable* out) {
  static std::mutex mu;
  static std::map<std::tuple<int, int, int, uint32_t, uint32_t>, RopeTable> cache;
  uint32_t ps, bs;
  std::memcpy(&ps, &pos_scale, 4);
  std::memcpy(&bs, &base, 4);
  auto key = std::make_tuple(dev, N, D, ps, bs);
  std::lock_guard<std::mutex> lock(mu);
  auto it = cache.find(key);
  if (it != cache.end()) {
    *out = it->second;
    return S2ATTN_OK;
  }
  const int half = D / 2;
  std::vector<float> c((size_t)N * half), s((size_t)N * half);
  std::vector<float> theta(half);
  for (int i = 0; i < half; ++i) theta[i] = (float)std::pow((double)base, -2.0 * (double)i / (double)D);
  for (int t = 0; t < N; ++t) {
    volatile float pos = (float)t * pos_scale;
    for (int i = 0; i < half; ++i) {
      volatile float a = pos * theta[i];
      c[(size_t)t * half + i] = (float)std::cos((double)a);
      s[(size_t)t * half + i] = (float)std::sin((double)a);
    }
  }
  RopeTable tab;
  const size_t bytes = sizeof(float) * c.size();
  if (cudaMalloc(&tab.cos_d, bytes) != cudaSuccess) return S2ATTN_ERR_CUDA;
  if (cudaMalloc(&tab.sin_d, bytes) != cudaSuccess) {
    cudaFree(tab.cos_d);
    return S2ATTN_ERR_CUDA;
  }
  if (cudaMemcpy(tab.cos_d, c.data(), bytes, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaMemcpy(tab.sin_d, s.data(), bytes, cudaMemcpyHostToDevice) != cudaSuccess) {
    cudaFree(tab.cos_d);
    cudaFree(tab.sin_d);
    return S2ATTN_ERR_CUDA;
  }
  cache[key] = tab;
  *out = tab;
  return S2ATTN_OK;
}

// One thread waits on an mbarrier that nothing ever arrives at; the bounded wait must
// give up after timeout_ns and record (K_SELFTEST << 8) | 1 in the error word.
__global__ void selftest_wait_kernel(int* err, unsigned long long timeout_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    s2::mbar_init(&bar, 1);
    abort_flag = 0;
    s2::fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0 && !s2::wait_bounded_ns(&bar, 0, &abort_flag, err, timeout_ns))
    s2::report_error(err, (s2::K_SELFTEST << 8) | 1);
}

int sm_count();

int bwd_main_impl(const void* q, const void* k, const void* v, const void* dout, const float* lse,
                  const float* delta, float* dq_acc, void* dk, void* dv, const s2::Shape& s, cudaStream_t st) {
  CUtensorMap tq, tk, tv, tdo;
  if (!map_bf16_sw128(&tq, q, s, 128) || !map_bf16_sw128(&tk, k, s, 128) || !map_bf16_sw128(&tv, v, s, 128) ||
      !map_bf16_sw128(&tdo, dout, s, 128))
    return S2ATTN_ERR_CUDA;
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_bwd_sm100(tq, tk, tv, tdo, lse, delta, dq_acc, dk, dv, s, sm_count(), err, st));
}

// SM count of the current device, looked up once per device.
int sm_count() {
  static std::mutex mu;
  static int cache[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (!cache[dev] && cudaDeviceGetAttribute(&cache[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    cache[dev] = 0;
  return cache[dev];
}

int check_decode_shape(int B, int M, int N, int H, int D) {
  if (B < 1 || M < 1 || N < 1 || H < 1 || D < 1 || M > N) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)B * N > INT_MAX / 2) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)B * N * H > (LLONG_MAX / 8) / D) return S2ATTN_ERR_INVALID_ARG;
  if (D != 128 || M > s2::kDecodeMaxM) return S2ATTN_ERR_UNSUPPORTED;
  if ((long long)B * H * M > INT_MAX || (long long)B * H * s2::kDecodeMaxSplits > INT_MAX)
    return S2ATTN_ERR_UNSUPPORTED;
  return S2ATTN_OK;
}

// Splits the workspace is sized for: the most any device can get (1 per key tile,
// at most kDecodeMaxSplits), so that the size does not depend on the device.
int decode_max_splits(int N) {
  const int tiles = (N + s2::kDecodeTileKeys - 1) / s2::kDecodeTileKeys;
  return tiles < s2::kDecodeMaxSplits ? tiles : s2::kDecodeMaxSplits;
}

// LoRA workspace: u [parts, T, 64] bf16, then a_pad, then b_pad (each 256-byte aligned).
size_t lora_u_bytes(int T, int parts) { return align256((size_t)parts * T * s2::kLoraRankPad * 2); }

size_t decode_part_o_bytes(int B, int M, int N, int H, int D) {
  return align256((size_t)B * H * decode_max_splits(N) * M * D * sizeof(float));
}

// ---- rotary norm, tree attention, paged cache ---------------------------------------
bool aligned4(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int check_norm_rope(const s2::NormRopeArgs& a, bool bwd) {
  if (a.B < 1 || a.N < 1 || a.D < 16 || a.D % 16 != 0 || a.D > 256) return S2ATTN_ERR_INVALID_ARG;
  if (a.R < 0 || a.R > a.D || a.R % 16 != 0) return S2ATTN_ERR_INVALID_ARG;
  if (a.dtype != S2ATTN_BF16 && a.dtype != S2ATTN_FP16 && a.dtype != S2ATTN_F32) return S2ATTN_ERR_INVALID_ARG;
  if (!a.q_dst && !a.k_dst) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)a.B * a.N > INT_MAX / 2) return S2ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(a.eps) || a.eps < 0.f || !std::isfinite(a.attn_factor)) return S2ATTN_ERR_INVALID_ARG;
  if (a.R > 0 && !aligned4(a.inv_freq)) return S2ATTN_ERR_INVALID_ARG;
  if (a.positions && !aligned4(a.positions)) return S2ATTN_ERR_INVALID_ARG;
  if (!a.positions && (long long)a.pos0 + a.N > INT_MAX) return S2ATTN_ERR_INVALID_ARG;
  const void* src[2] = {a.q, a.k};
  const void* grad[2] = {a.dq_out, a.dk_out};
  const void* w[2] = {a.wq, a.wk};
  void* dst[2] = {a.q_dst, a.k_dst};
  void* dw[2] = {a.dwq, a.dwk};
  const int H[2] = {a.Hq, a.Hk};
  for (int i = 0; i < 2; ++i) {
    if ((w[i] && !a.norm) || (dw[i] && (!a.norm || !dst[i]))) return S2ATTN_ERR_INVALID_ARG;
    if (dw[i] && !aligned4(dw[i])) return S2ATTN_ERR_INVALID_ARG;
    if (!dst[i]) {
      if (src[i] && !bwd) return S2ATTN_ERR_INVALID_ARG;   // an input without its output
      continue;
    }
    if (H[i] < 1 || H[i] > s2::kNormRopeMaxHeads) return S2ATTN_ERR_INVALID_ARG;
    if (!aligned16(dst[i]) || (w[i] && !aligned16(w[i]))) return S2ATTN_ERR_INVALID_ARG;
    if ((!bwd || a.norm) && !aligned16(src[i])) return S2ATTN_ERR_INVALID_ARG;
    if (bwd && !aligned16(grad[i])) return S2ATTN_ERR_INVALID_ARG;
  }
  return S2ATTN_OK;
}

// log2 of a page size, or -1.
int page_shift_of(int page_size) {
  if (page_size < 16 || (page_size & (page_size - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

int check_pages(int n_pages, int page_size, int table_width) {
  if (n_pages < 1 || page_size < 1 || table_width < 1) return S2ATTN_ERR_INVALID_ARG;
  if (page_shift_of(page_size) < 0) return S2ATTN_ERR_UNSUPPORTED;
  if ((long long)n_pages * page_size > (long long)INT_MAX - 255) return S2ATTN_ERR_UNSUPPORTED;
  return S2ATTN_OK;
}

int check_tree_shape(int B, int M, int H, int Hkv, int D) {
  if (B < 1 || M < 1 || H < 1 || Hkv < 1 || D < 1 || H % Hkv != 0) return S2ATTN_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || M > s2::kTreeMaxM || B > s2::kTreeMaxB || H / Hkv > 128) return S2ATTN_ERR_UNSUPPORTED;
  if ((long long)B * M * H > INT_MAX) return S2ATTN_ERR_UNSUPPORTED;
  return S2ATTN_OK;
}

// A [rows, H, D] 16-bit tensor; a box is box_rows rows of box_heads heads, 64 columns.
bool map_heads(CUtensorMap* m, const void* base, int dtype, long long rows, int H, int D, int box_heads,
               int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt =
      dtype == S2ATTN_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return fn(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Partials of a tree attention call: outputs, then (max, sum) pairs; then the runs of each
// (sequence, row tile).
size_t tree_part_rows(const s2::TreePlan& t, int Hkv) { return (size_t)Hkv * t.RT * t.J * 2 * t.slot_rows; }

}  // namespace

namespace s2 {
int check_tensor_core_args(int B, int N, int H, int D, int G, int shift_heads) {
  return check_tensor_core_shape(B, N, H, D, G, shift_heads);
}
}  // namespace s2

extern "C" {

int s2attn_version(void) { return 100; }

const char* s2attn_status_string(int status) {
  switch (status) {
    case S2ATTN_OK: return "ok";
    case S2ATTN_ERR_INVALID_ARG: return "invalid argument";
    case S2ATTN_ERR_UNSUPPORTED: return "unsupported shape for this path";
    case S2ATTN_ERR_WORKSPACE: return "workspace missing or too small";
    case S2ATTN_ERR_CUDA: return "CUDA call failed";
    case S2ATTN_ERR_DEVICE_TIMEOUT: return "device-side wait timed out";
    case S2ATTN_ERR_DEVICE_INDEX: return "device-side index out of range";
    default: return "unknown status";
  }
}

int s2attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int N, int H, int D, int G,
               int shift_heads, void* stream) {
  int rc = check_tensor_core_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return S2ATTN_ERR_INVALID_ARG;
  const s2::Shape s{B, N, H, D, G, shift_heads};
  CUtensorMap tq, tk, tv;
  if (!map_bf16_sw128(&tq, q, s, 128) || !map_bf16_sw128(&tk, k, s, 128) || !map_bf16_sw128(&tv, v, s, 128))
    return S2ATTN_ERR_CUDA;
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_fwd_sm100(tq, tk, tv, o, lse, s, sm_count(), err, static_cast<cudaStream_t>(stream)));
}

size_t s2attn_bwd_workspace_bytes(int B, int N, int H, int D) {
  if (B < 1 || N < 1 || H < 1 || D < 1) return 0;
  return align256((size_t)B * N * H * D * sizeof(float)) + align256((size_t)B * H * N * sizeof(float));
}

int s2attn_bwd_preprocess(const void* o, const void* dout, float* delta, float* dq_acc, int B, int N, int H, int D,
                          void* stream) {
  int rc = check_shape(B, N, H, D, N, 0);
  if (rc) return rc;
  if (D != 128) return S2ATTN_ERR_UNSUPPORTED;
  if (!aligned16(o) || !aligned16(dout) || !aligned16(delta) || !aligned16(dq_acc)) return S2ATTN_ERR_INVALID_ARG;
  const s2::Shape s{B, N, H, D, N, 0};
  return cuda_status(s2::launch_bwd_preprocess(o, dout, delta, dq_acc, s, static_cast<cudaStream_t>(stream)));
}

int s2attn_bwd_main(const void* q, const void* k, const void* v, const void* dout, const float* lse,
                    const float* delta, float* dq_acc, void* dk, void* dv, int B, int N, int H, int D, int G,
                    int shift_heads, void* stream) {
  int rc = check_tensor_core_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(delta) || !aligned16(dq_acc) || !aligned16(dk) || !aligned16(dv))
    return S2ATTN_ERR_INVALID_ARG;
  const s2::Shape s{B, N, H, D, G, shift_heads};
  return bwd_main_impl(q, k, v, dout, lse, delta, dq_acc, dk, dv, s, static_cast<cudaStream_t>(stream));
}

int s2attn_bwd_dq_convert(const float* dq_acc, void* dq, int B, int N, int H, int D, void* stream) {
  int rc = check_shape(B, N, H, D, N, 0);
  if (rc) return rc;
  if (D % 8 != 0) return S2ATTN_ERR_UNSUPPORTED;
  if (!aligned16(dq_acc) || !aligned16(dq)) return S2ATTN_ERR_INVALID_ARG;
  const s2::Shape s{B, N, H, D, N, 0};
  return cuda_status(s2::launch_dq_convert(dq_acc, dq, s, static_cast<cudaStream_t>(stream)));
}

int s2attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
               void* dq, void* dk, void* dv, int B, int N, int H, int D, int G, int shift_heads, void* workspace,
               size_t workspace_bytes, void* stream) {
  int rc = check_tensor_core_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return S2ATTN_ERR_INVALID_ARG;
  const size_t need = s2attn_bwd_workspace_bytes(B, N, H, D);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return S2ATTN_ERR_WORKSPACE;
  float* dq_acc = static_cast<float*>(workspace);
  float* delta = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)B * N * H * D * 4));
  const s2::Shape s{B, N, H, D, G, shift_heads};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((rc = cuda_status(s2::launch_bwd_preprocess(o, dout, delta, dq_acc, s, st)))) return rc;
  if ((rc = bwd_main_impl(q, k, v, dout, lse, delta, dq_acc, dk, dv, s, st))) return rc;
  return cuda_status(s2::launch_dq_convert(dq_acc, dq, s, st));
}

int s2attn_halo_rows(void* const* x, void* const* buf, int n_tensors, int to_buf, int B, int N, int H, int D,
                     int G, int shift_heads, void* stream) {
  int rc = check_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (shift_heads < 1 || n_tensors < 1 || n_tensors > s2::kHaloMaxTensors || !x || !buf) return S2ATTN_ERR_INVALID_ARG;
  if ((D * 2) % 16 != 0) return S2ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < n_tensors; ++i)
    if (!aligned16(x[i]) || !aligned16(buf[i])) return S2ATTN_ERR_INVALID_ARG;
  const int n_sm = sm_count();
  if (n_sm <= 0) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_halo_rows(x, buf, n_tensors, to_buf ? 1 : 0, B, N, H, D, G, shift_heads, n_sm,
                                          static_cast<cudaStream_t>(stream)));
}

int s2attn_halo_lse(float* const* lse, float* const* buf, int n_tensors, int to_buf, int B, int N, int H, int G,
                    int shift_heads, void* stream) {
  int rc = check_shape(B, N, H, 1, G, shift_heads);
  if (rc) return rc;
  if (shift_heads < 1 || n_tensors < 1 || n_tensors > s2::kHaloMaxTensors || !lse || !buf)
    return S2ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < n_tensors; ++i)
    if (!lse[i] || !buf[i] || (reinterpret_cast<uintptr_t>(lse[i]) & 3u) || (reinterpret_cast<uintptr_t>(buf[i]) & 3u))
      return S2ATTN_ERR_INVALID_ARG;
  const int n_sm = sm_count();
  if (n_sm <= 0) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_halo_lse(lse, buf, n_tensors, to_buf ? 1 : 0, B, N, H, G, shift_heads, n_sm,
                                         static_cast<cudaStream_t>(stream)));
}

size_t s2attn_decode_workspace_bytes(int B, int M, int N, int H, int D) {
  if (check_decode_shape(B, M, N, H, D)) return 0;
  return decode_part_o_bytes(B, M, N, H, D) +
         align256((size_t)B * H * decode_max_splits(N) * M * 2 * sizeof(float));
}

int s2attn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int M, int N, int H,
                  int D, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_decode_shape(B, M, N, H, D);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return S2ATTN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < s2attn_decode_workspace_bytes(B, M, N, H, D) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return S2ATTN_ERR_WORKSPACE;
  const int n_sm = sm_count();
  if (n_sm <= 0) return S2ATTN_ERR_CUDA;
  float* part_o = static_cast<float*>(workspace);
  float* part_ml = reinterpret_cast<float*>(static_cast<char*>(workspace) + decode_part_o_bytes(B, M, N, H, D));
  const s2::Shape s{B, N, H, D, N, 0};
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int tps = 0;
  if (M <= s2::kDecodeSimtMaxM) {
    const int S = s2::decode_splits(B, N, H, n_sm, &tps);
    CUtensorMap tk, tv;
    if (!map_bf16_sw128(&tk, k, s, s2::kDecodeTileKeys) || !map_bf16_sw128(&tv, v, s, s2::kDecodeTileKeys))
      return S2ATTN_ERR_CUDA;
    return cuda_status(s2::launch_decode_sm100(tk, tv, q, o, lse, part_o, part_ml, B, M, N, H, S, tps, err, st));
  }
  const int S = s2::decode_splits_tc(B, N, H, n_sm, &tps);
  const s2::Shape sq{B, M, H, D, M, 0};
  CUtensorMap tq, tk, tv;
  if (!map_bf16_sw128(&tq, q, sq, 128) || !map_bf16_sw128(&tk, k, s, s2::kDecodeTileKeys) ||
      !map_bf16_sw128(&tv, v, s, s2::kDecodeTileKeys))
    return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_decode_tc_sm100(tq, tk, tv, o, lse, part_o, part_ml, B, M, N, H, S, tps, err, st));
}

int s2attn_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse, int B, int N, int H, int D,
                   int G, int shift_heads, void* stream) {
  int rc = check_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (D > 128) return S2ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return S2ATTN_ERR_INVALID_ARG;
  const s2::Shape s{B, N, H, D, G, shift_heads};
  return cuda_status(s2::launch_fwd_f32(q, k, v, o, lse, s, static_cast<cudaStream_t>(stream)));
}

int s2attn_bwd_f32(const float* q, const float* k, const float* v, const float* o, const float* dout,
                   const float* lse, float* dq, float* dk, float* dv, int B, int N, int H, int D, int G,
                   int shift_heads, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_shape(B, N, H, D, G, shift_heads);
  if (rc) return rc;
  if (D > 128) return S2ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) || !aligned16(lse) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return S2ATTN_ERR_INVALID_ARG;
  const size_t need = s2attn_bwd_workspace_bytes(B, N, H, D);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return S2ATTN_ERR_WORKSPACE;
  float* delta = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)B * N * H * D * 4));
  const s2::Shape s{B, N, H, D, G, shift_heads};
  return cuda_status(
      s2::launch_bwd_f32(q, k, v, o, dout, lse, dq, dk, dv, delta, s, static_cast<cudaStream_t>(stream)));
}

int rope_pi_apply(void* q, void* k, int B, int N, int H, int D, float pos_scale, float base, void* stream) {
  if (B < 1 || N < 1 || H < 1 || D < 16 || D % 16 != 0 || D > 256) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)B * N * H > (LLONG_MAX / 8) / D) return S2ATTN_ERR_INVALID_ARG;
  if (!q && !k) return S2ATTN_ERR_INVALID_ARG;
  if ((q && !aligned16(q)) || (k && !aligned16(k))) return S2ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(pos_scale) || !std::isfinite(base) || !(base > 0.f)) return S2ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return S2ATTN_ERR_CUDA;
  RopeTable tab;
  int rc = rope_table(dev, N, D, pos_scale, base, &tab);
  if (rc) return rc;
  return cuda_status(
      s2::launch_rope_pi(q, k, tab.cos_d, tab.sin_d, B, N, H, D, static_cast<cudaStream_t>(stream)));
}

int rope_pi_apply_offset(void* q, void* k, int B, int N, int H, int D, int pos0, float pos_scale, float base,
                         void* stream) {
  if (B < 1 || N < 1 || H < 1 || D < 16 || D % 16 != 0 || D > 256 || pos0 < 0) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)pos0 + N > (1LL << 24)) return S2ATTN_ERR_INVALID_ARG;
  if ((long long)B * N * H > (LLONG_MAX / 8) / D) return S2ATTN_ERR_INVALID_ARG;
  if (!q && !k) return S2ATTN_ERR_INVALID_ARG;
  if ((q && !aligned16(q)) || (k && !aligned16(k))) return S2ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(pos_scale) || !std::isfinite(base) || !(base > 0.f)) return S2ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return S2ATTN_ERR_CUDA;
  // Row p of a table holds position p whatever the table's length, so the table of the
  // next power of two >= pos0 + N (cached like any other) serves every offset below it,
  // and a decoding loop that grows its sequence builds only a few tables.
  int rows = 1024;
  while (rows < pos0 + N) rows *= 2;
  RopeTable tab;
  int rc = rope_table(dev, rows, D, pos_scale, base, &tab);
  if (rc) return rc;
  const size_t off = (size_t)pos0 * (D / 2);
  return cuda_status(s2::launch_rope_pi(q, k, tab.cos_d + off, tab.sin_d + off, B, N, H, D,
                                        static_cast<cudaStream_t>(stream)));
}

size_t lora_proj_workspace_bytes(int T, int K, int n_out, int parts, int r) {
  if (T < 1 || K < 1 || n_out < 1 || parts < 1 || r < 0 || r > s2::kLoraMaxRank) return 0;
  if (r == 0) return 0;
  return lora_u_bytes(T, parts) + align256((size_t)parts * s2::kLoraRankPad * K * 2) +
         align256((size_t)parts * n_out * s2::kLoraRankPad * 2);
}

int lora_proj_fwd(const void* x, const void* w, const void* lora_a, const void* lora_b, void* y, int T, int K,
                  int n_out, int parts, int r, float scaling, int rope_parts, int head_dim, int seq_len,
                  float pos_scale, float base, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 1 || K < 8 || K % 8 != 0 || n_out < 1 || parts < 1 || r < 0 || r > s2::kLoraMaxRank)
    return S2ATTN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(y)) return S2ATTN_ERR_INVALID_ARG;
  if (r > 0 && (!aligned16(lora_a) || !lora_b || !std::isfinite(scaling))) return S2ATTN_ERR_INVALID_ARG;
  if (rope_parts < 0 || rope_parts > parts) return S2ATTN_ERR_INVALID_ARG;
  if (rope_parts > 0) {
    if (head_dim != 32 && head_dim != 64 && head_dim != 128 && head_dim != 256) return S2ATTN_ERR_INVALID_ARG;
    if (seq_len < 1 || T % seq_len != 0) return S2ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(pos_scale) || !std::isfinite(base) || !(base > 0.f)) return S2ATTN_ERR_INVALID_ARG;
  }
  if (n_out % s2::kLoraProjTileN != 0) return S2ATTN_ERR_UNSUPPORTED;
  if (K < 64) return S2ATTN_ERR_UNSUPPORTED;   // the tensor maps' 64-column boxes must fit in a row of x and W
  if ((long long)parts * n_out > INT_MAX || (long long)T + 128 > INT_MAX) return S2ATTN_ERR_UNSUPPORTED;
  if (((long long)T + 127) / 128 * ((long long)parts * n_out / s2::kLoraProjTileN) > INT_MAX)
    return S2ATTN_ERR_UNSUPPORTED;
  if (r > 0) {
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return S2ATTN_ERR_WORKSPACE;
    if (workspace_bytes < lora_proj_workspace_bytes(T, K, n_out, parts, r)) return S2ATTN_ERR_WORKSPACE;
  }
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return S2ATTN_ERR_CUDA;
  RopeTable tab;
  if (rope_parts > 0) {
    int rc = rope_table(dev, seq_len, head_dim, pos_scale, base, &tab);
    if (rc) return rc;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tx, tw, tu, tb, ta;
  if (!map_rows_bf16(&tx, x, 2, K, T, 1, 64, 128) ||
      !map_rows_bf16(&tw, w, 2, K, (uint64_t)parts * n_out, 1, 64, s2::kLoraProjTileN))
    return S2ATTN_ERR_CUDA;
  tu = tx;
  tb = tw;
  if (r > 0) {
    char* ws = static_cast<char*>(workspace);
    void* u = ws;
    void* a_pad = ws + lora_u_bytes(T, parts);
    void* b_pad = ws + lora_u_bytes(T, parts) + align256((size_t)parts * s2::kLoraRankPad * K * 2);
    if (!map_rows_bf16(&ta, a_pad, 2, K, (uint64_t)parts * s2::kLoraRankPad, 1, 64, s2::kLoraRankPad) ||
        !map_rows_bf16(&tu, u, 3, s2::kLoraRankPad, T, parts, 64, 128) ||
        !map_rows_bf16(&tb, b_pad, 2, s2::kLoraRankPad, (uint64_t)parts * n_out, 1, 64, s2::kLoraProjTileN))
      return S2ATTN_ERR_CUDA;
    cudaError_t e = s2::launch_lora_pad(lora_a, lora_b, a_pad, b_pad, parts, r, K, n_out, st);
    if (e == cudaSuccess) e = s2::launch_lora_down(tx, ta, u, T, K, parts, scaling, sm_count(), err, st);
    if (e != cudaSuccess) return S2ATTN_ERR_CUDA;
  }
  return cuda_status(s2::launch_lora_proj(tx, tw, tu, tb, y, T, K, n_out, parts, r, rope_parts, head_dim, seq_len,
                                          tab.cos_d, tab.sin_d, sm_count(), err, st));
}

size_t lora_proj_bwd_workspace_bytes(int T, int K, int n_out, int parts, int r) {
  if (T < 1 || K < 1 || n_out < 1 || parts < 1 || r < 0 || r > s2::kLoraMaxRank) return 0;
  const size_t apad = align256((size_t)parts * s2::kLoraRankPad * K * 2);
  const size_t bpad = align256((size_t)parts * n_out * s2::kLoraRankPad * 2);
  const size_t da_acc = align256((size_t)((parts * s2::kLoraRankPad + 127) / 128) * 128 * K * 4);
  const size_t db_acc = align256((size_t)parts * n_out * s2::kLoraRankPad * 4);
  return 2 * lora_u_bytes(T, parts) + apad + bpad + da_acc + db_acc;   // u, g, a_pad, b_pad, accumulators
}

int lora_proj_bwd(const void* x, const void* w, const void* lora_a, const void* lora_b, const void* dy, void* dx,
                  void* d_lora_a, void* d_lora_b, int T, int K, int n_out, int parts, int r, float scaling,
                  void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 1 || K < 8 || K % 8 != 0 || n_out < 1 || parts < 1 || r < 0 || r > s2::kLoraMaxRank)
    return S2ATTN_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(dy) || !aligned16(dx)) return S2ATTN_ERR_INVALID_ARG;
  if (r > 0 && (!aligned16(lora_a) || !lora_b || !d_lora_a || !d_lora_b || !std::isfinite(scaling)))
    return S2ATTN_ERR_INVALID_ARG;
  if (n_out % s2::kLoraProjTileN != 0) return S2ATTN_ERR_UNSUPPORTED;
  if (K < 64) return S2ATTN_ERR_UNSUPPORTED;   // the tensor maps' 64-column boxes must fit in a row of x and W
  if ((long long)parts * n_out > INT_MAX || (long long)T + 128 > INT_MAX) return S2ATTN_ERR_UNSUPPORTED;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return S2ATTN_ERR_WORKSPACE;
  if (workspace_bytes < lora_proj_bwd_workspace_bytes(T, K, n_out, parts, r)) return S2ATTN_ERR_WORKSPACE;
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const size_t ub = lora_u_bytes(T, parts);
  void* u = ws;
  void* g = ws + ub;
  void* a_pad = ws + 2 * ub;
  void* b_pad = static_cast<char*>(a_pad) + align256((size_t)parts * s2::kLoraRankPad * K * 2);
  float* da_acc = reinterpret_cast<float*>(static_cast<char*>(b_pad) +
                                           align256((size_t)parts * n_out * s2::kLoraRankPad * 2));
  float* db_acc = reinterpret_cast<float*>(reinterpret_cast<char*>(da_acc) +
                                           align256((size_t)((parts * s2::kLoraRankPad + 127) / 128) * 128 * K * 4));
  const int RP = s2::kLoraRankPad;
  CUtensorMap dy_k, dy_mn, bpad, w_mn, g_k, apad, g_mn, x_mn, u_mn, tx, ta;
  bool ok = map_rows_bf16(&dy_k, dy, 3, n_out, T, parts, 64, 128) && map_rows_bf16(&dy_mn, dy, 3, n_out, T, parts, 64, 64) &&
            map_rows_bf16(&w_mn, w, 3, K, n_out, parts, 64, 64) && map_rows_bf16(&x_mn, x, 3, K, T, 1, 64, 64);
  if (r > 0)
    ok = ok && map_rows_bf16(&bpad, b_pad, 3, RP, n_out, parts, 64, 64) && map_rows_bf16(&g_k, g, 3, RP, T, parts, 64, 128) &&
         map_rows_bf16(&apad, a_pad, 3, K, RP, parts, 64, 64) && map_rows_bf16(&g_mn, g, 3, RP, T, parts, 64, 64) &&
         map_rows_bf16(&u_mn, u, 3, RP, T, parts, 64, 64) && map_rows_bf16(&tx, x, 2, K, T, 1, 64, 128) &&
         map_rows_bf16(&ta, a_pad, 2, K, (uint64_t)parts * RP, 1, 64, RP);
  else
    bpad = g_k = apad = g_mn = u_mn = dy_k;   // unused without an adapter
  if (!ok) return S2ATTN_ERR_CUDA;
  cudaError_t e = cudaSuccess;
  if (r > 0) {
    e = s2::launch_lora_pad(lora_a, lora_b, a_pad, b_pad, parts, r, K, n_out, st);
    if (e == cudaSuccess) e = s2::launch_lora_down(tx, ta, u, T, K, parts, scaling, sm_count(), err, st);
    if (e != cudaSuccess) return S2ATTN_ERR_CUDA;
  }
  return cuda_status(s2::launch_lora_bwd(dy_k, dy_mn, bpad, w_mn, g_k, apad, g_mn, x_mn, u_mn, g, dx, da_acc, db_acc,
                                         d_lora_a, d_lora_b, T, K, n_out, parts, r, scaling, sm_count(), err, st));
}

int qk_norm_rope_fwd(const void* q, const void* k, const void* wq, const void* wk, const int* positions,
                     const float* inv_freq, void* q_out, void* k_out, int B, int N, int Hq, int Hk, int D, int R,
                     int interleaved, int norm, float eps, float attn_factor, int pos0, int dtype, void* stream) {
  s2::NormRopeArgs a{};
  a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.positions = positions, a.inv_freq = inv_freq;
  a.q_dst = q_out, a.k_dst = k_out;
  a.B = B, a.N = N, a.Hq = Hq, a.Hk = Hk, a.D = D, a.R = R, a.pos0 = pos0;
  a.interleaved = interleaved ? 1 : 0, a.norm = norm ? 1 : 0, a.dtype = dtype, a.eps = eps, a.attn_factor = attn_factor;
  const int rc = check_norm_rope(a, false);
  if (rc) return rc;
  const int n_sm = sm_count();
  if (n_sm <= 0) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_norm_rope_fwd(a, n_sm, static_cast<cudaStream_t>(stream)));
}

size_t qk_norm_rope_bwd_workspace_bytes(int D) {
  if (D < 16 || D % 16 != 0 || D > 256) return 0;
  return align256((size_t)s2::kNormRopePartials * D * sizeof(float));
}

int qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out, const void* wq,
                     const void* wk, const int* positions, const float* inv_freq, void* dq, void* dk, void* dwq,
                     void* dwk, int B, int N, int Hq, int Hk, int D, int R, int interleaved, int norm, float eps,
                     float attn_factor, int pos0, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  s2::NormRopeArgs a{};
  a.q = q, a.k = k, a.dq_out = dq_out, a.dk_out = dk_out, a.wq = wq, a.wk = wk;
  a.positions = positions, a.inv_freq = inv_freq;
  a.q_dst = dq, a.k_dst = dk, a.dwq = dwq, a.dwk = dwk;
  a.B = B, a.N = N, a.Hq = Hq, a.Hk = Hk, a.D = D, a.R = R, a.pos0 = pos0;
  a.interleaved = interleaved ? 1 : 0, a.norm = norm ? 1 : 0, a.dtype = dtype, a.eps = eps, a.attn_factor = attn_factor;
  const int rc = check_norm_rope(a, true);
  if (rc) return rc;
  if ((dwq || dwk) && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                       workspace_bytes < qk_norm_rope_bwd_workspace_bytes(D)))
    return S2ATTN_ERR_WORKSPACE;
  const int n_sm = sm_count();
  if (n_sm <= 0) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_norm_rope_bwd(a, static_cast<float*>(workspace), n_sm, static_cast<cudaStream_t>(stream)));
}

int rope_inv_freq(float* inv_freq, float* attn_factor, int R, float base, int scaling, float factor,
                  int original_len, float beta_fast, float beta_slow) {
  if (!inv_freq || !attn_factor || R < 2 || R % 2 != 0 || R > 256) return S2ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(base) || !(base > 1.f) || !std::isfinite(factor) || !(factor >= 1.f)) return S2ATTN_ERR_INVALID_ARG;
  if (scaling < 0 || scaling > 3 || (scaling == 2 && R < 4)) return S2ATTN_ERR_INVALID_ARG;
  if (scaling == 3 && (original_len < 1 || !std::isfinite(beta_fast) || !(beta_slow > 0.f) || !(beta_fast > beta_slow)))
    return S2ATTN_ERR_INVALID_ARG;
  double b = base;
  if (scaling == 2) b *= std::pow((double)factor, (double)R / (R - 2));
  double low = 0, high = 0;
  if (scaling == 3) {
    const double turns = R / (2 * std::log((double)base));
    low = std::max(0.0, std::floor(turns * std::log(original_len / (2 * M_PI * beta_fast))));
    // (may lie behind the last frequency, R/2 - 1: the ramp then ends before it has reached 1)
    high = std::min(R - 1.0, std::ceil(turns * std::log(original_len / (2 * M_PI * beta_slow))));
  }
  for (int i = 0; i < R / 2; ++i) {
    double f = std::pow(b, -2.0 * i / R);
    if (scaling == 1) f /= factor;
    if (scaling == 3) {
      // a ramp of no width is a step behind `low`
      const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    inv_freq[i] = (float)f;
  }
  *attn_factor = scaling == 3 ? (float)(0.1 * std::log((double)factor) + 1.0) : 1.0f;
  return S2ATTN_OK;
}

int s2attn_tree_mask(const int* parents, unsigned long long* mask, int* depth, int B, int M, void* stream) {
  if (B < 1 || M < 1 || (long long)B * M > INT_MAX) return S2ATTN_ERR_INVALID_ARG;
  if (M > s2::kTreeMaxM) return S2ATTN_ERR_UNSUPPORTED;
  if (!aligned4(parents) || !mask || (reinterpret_cast<uintptr_t>(mask) & 7u) || (depth && !aligned4(depth)))
    return S2ATTN_ERR_INVALID_ARG;
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_tree_mask(parents, mask, depth, B, M, err + 1, static_cast<cudaStream_t>(stream)));
}

size_t s2attn_tree_decode_workspace_bytes(int B, int M, int H, int Hkv, int D) {
  if (check_tree_shape(B, M, H, Hkv, D)) return 0;
  const s2::TreePlan t = s2::tree_plan(M, H, Hkv);
  const size_t rows = tree_part_rows(t, Hkv);
  return align256(rows * D * sizeof(float)) + align256(rows * 2 * sizeof(float)) +
         align256((size_t)B * t.RT * 2 * sizeof(int));
}

int s2attn_tree_decode(const void* q, const void* k_new, const void* v_new, const void* k_pages,
                       const void* v_pages, const int* page_table, const int* cache_len, const int* new_len,
                       const unsigned long long* tree_mask, void* o, float* lse, int B, int M, int H, int Hkv, int D,
                       int n_pages, int page_size, int table_width, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int rc = check_tree_shape(B, M, H, Hkv, D);
  if (rc) return rc;
  if ((rc = check_pages(n_pages, page_size, table_width))) return rc;
  // the kernel counts key tiles of 64 (and a few more a sequence) in 32 bits
  if ((double)B * ((double)table_width * page_size / 64 + 16) >= 1073741824.0) return S2ATTN_ERR_UNSUPPORTED;
  if (dtype != S2ATTN_BF16 && dtype != S2ATTN_FP16) return S2ATTN_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) ||
      !aligned16(o) || !aligned4(lse) || !aligned4(page_table) || !aligned4(cache_len))
    return S2ATTN_ERR_INVALID_ARG;
  if ((new_len && !aligned4(new_len)) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u)) return S2ATTN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < s2attn_tree_decode_workspace_bytes(B, M, H, Hkv, D) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return S2ATTN_ERR_WORKSPACE;
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  const s2::TreePlan t = s2::tree_plan(M, H, Hkv);
  const size_t rows = tree_part_rows(t, Hkv);
  char* ws = static_cast<char*>(workspace);
  s2::TreeArgs a{};
  a.o = o, a.lse = lse;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float*>(ws + align256(rows * D * sizeof(float)));
  a.meta = reinterpret_cast<int*>(ws + align256(rows * D * sizeof(float)) + align256(rows * 2 * sizeof(float)));
  a.cache_len = cache_len, a.new_len = new_len, a.page_table = page_table, a.mask = tree_mask, a.v_new = v_new;
  a.B = B, a.M = M, a.H = H, a.Hkv = Hkv, a.D = D, a.page_shift = page_shift_of(page_size);
  a.n_pages = n_pages, a.width = table_width, a.dtype = dtype, a.err = err, a.index_err = err + 1;
  const int page_box = page_size < 64 ? page_size : 64, new_box = M < 64 ? M : 64;
  s2::TreeMaps maps;
  if (!map_heads(&maps.q, q, dtype, (long long)B * M, H, D, t.group, t.tok < M ? t.tok : M) ||
      !map_heads(&maps.k_pages, k_pages, dtype, (long long)n_pages * page_size, Hkv, D, 1, page_box) ||
      !map_heads(&maps.v_pages, v_pages, dtype, (long long)n_pages * page_size, Hkv, D, 1, page_box) ||
      !map_heads(&maps.k_new, k_new, dtype, (long long)B * M, Hkv, D, 1, new_box) ||
      !map_heads(&maps.v_new, v_new, dtype, (long long)B * M, Hkv, D, 1, new_box))
    return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_tree_decode(maps, a, t, static_cast<cudaStream_t>(stream)));
}

int s2attn_cache_append(const void* k_new, const void* v_new, void* k_pages, void* v_pages, const int* page_table,
                        const int* cache_len, const int* rows, const int* n_rows, int B, int M, int A, int Hkv, int D,
                        int n_pages, int page_size, int table_width, int elem_size, void* stream) {
  if (B < 1 || M < 1 || A < 1 || Hkv < 1 || D < 1) return S2ATTN_ERR_INVALID_ARG;
  if (!rows && A != M) return S2ATTN_ERR_INVALID_ARG;
  if (elem_size != 2 && elem_size != 4) return S2ATTN_ERR_INVALID_ARG;
  int rc = check_pages(n_pages, page_size, table_width);
  if (rc) return rc;
  const long long row_bytes = (long long)Hkv * D * elem_size;
  if (row_bytes % 16 != 0 || row_bytes > (1 << 20)) return S2ATTN_ERR_UNSUPPORTED;
  if ((long long)B * M > INT_MAX / 2 || (long long)B * A > INT_MAX / 2) return S2ATTN_ERR_UNSUPPORTED;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned4(page_table) ||
      !aligned4(cache_len) || (rows && !aligned4(rows)) || (n_rows && !aligned4(n_rows)))
    return S2ATTN_ERR_INVALID_ARG;
  int* err = error_word_ptr();
  const int n_sm = sm_count();
  if (!err || n_sm <= 0) return S2ATTN_ERR_CUDA;
  return cuda_status(s2::launch_cache_append(k_new, v_new, k_pages, v_pages, page_table, cache_len, rows, n_rows, B, M,
                                             A, table_width, n_pages, page_shift_of(page_size), (int)row_bytes, n_sm,
                                             err + 1, static_cast<cudaStream_t>(stream)));
}

int s2attn_cache_copy_pages(void* const* pools, int n_pools, const int* pairs, int n_pairs, int n_pages,
                            size_t page_bytes, void* stream) {
  if (!pools || n_pools < 1 || n_pools > s2::kCacheMaxPools || n_pairs < 0 || n_pages < 1 || page_bytes == 0)
    return S2ATTN_ERR_INVALID_ARG;
  if (page_bytes % 16 != 0 || page_bytes > ((size_t)1 << 40)) return S2ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < n_pools; ++i)
    if (!aligned16(pools[i])) return S2ATTN_ERR_INVALID_ARG;
  if (n_pairs == 0) return S2ATTN_OK;
  if (!pairs || n_pairs > n_pages) return S2ATTN_ERR_INVALID_ARG;   // each pair writes a page of its own
  // one bit a page: written by a pair so far
  uint32_t* written = static_cast<uint32_t*>(std::calloc((size_t)n_pages / 32 + 1, sizeof(uint32_t)));
  if (!written) return S2ATTN_ERR_INVALID_ARG;
  bool ok = true;
  for (int i = 0; i < n_pairs && ok; ++i) {
    const int src = pairs[2 * i], dst = pairs[2 * i + 1];
    ok = src >= 0 && src < n_pages && dst >= 0 && dst < n_pages && !(written[dst / 32] >> (dst % 32) & 1u);
    if (ok) written[dst / 32] |= 1u << (dst % 32);
  }
  for (int i = 0; i < n_pairs && ok; ++i) ok = !(written[pairs[2 * i] / 32] >> (pairs[2 * i] % 32) & 1u);
  std::free(written);
  if (!ok) return S2ATTN_ERR_INVALID_ARG;
  return cuda_status(s2::launch_cache_copy(pools, n_pools, pairs, n_pairs, (long long)page_bytes,
                                           static_cast<cudaStream_t>(stream)));
}

int s2attn_selftest_bounded_wait(unsigned timeout_us, void* stream) {
  if (timeout_us == 0 || timeout_us > 1000000u) return S2ATTN_ERR_INVALID_ARG;
  int* err = error_word_ptr();
  if (!err) return S2ATTN_ERR_CUDA;
  selftest_wait_kernel<<<1, 32, 0, static_cast<cudaStream_t>(stream)>>>(err, 1000ull * timeout_us);
  return cuda_status(cudaGetLastError());
}

int s2attn_get_device_error(int* detail) {
  int v[2] = {0, 0};
  if (cudaMemcpyFromSymbol(v, g_error_word, sizeof(v)) != cudaSuccess) return S2ATTN_ERR_CUDA;
  if (detail) *detail = v[0] ? v[0] : v[1];
  return v[0] ? S2ATTN_ERR_DEVICE_TIMEOUT : v[1] ? S2ATTN_ERR_DEVICE_INDEX : S2ATTN_OK;
}

int s2attn_clear_device_error(void) {
  const int zero[2] = {0, 0};
  return cudaMemcpyToSymbol(g_error_word, zero, sizeof(zero)) == cudaSuccess ? S2ATTN_OK : S2ATTN_ERR_CUDA;
}

}  // extern "C"
