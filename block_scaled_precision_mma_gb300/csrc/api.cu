// api.cu -- the C ABI: argument validation, per-device state, the scale workspace,
// the device-status word, tensor-map encoding and the wait-timeout probe.
//
// Validation follows the source pages' preconditions: 64-bit extents everywhere
// (launch arguments that overflowed 32 bits: "Experimental FlyDSL GEMM backend for
// TE PyTorch", BF16 skipped shapes; "Add FlyDSL grouped groupwise FP8 GEMM for
// ROCm", the commit passing operands with their natural shape), N and K multiples
// of 128 and m_sizes of length G for the grouped GEMM (same page, introduction and
// the format/rank check commit), OCP FP8 formats only.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <deque>
#include <mutex>
#include <vector>

#include "branch.h"
#include "epilogue.cuh"
#include "internal.h"
#include "moe_step.h"
#include "ptx.cuh"
#include "store_stage.cuh"

namespace bsmma {

// Latched device-side status, one per device that loads the library.
__device__ int g_device_status;

namespace {

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
bool g_dev_ready[kMaxDevices];
std::atomic<int64_t> g_launches{0};
std::atomic<uint64_t> g_wait_limit_ns{2000000000ull};
std::atomic<int> g_dense_variant{0};
std::atomic<int> g_grouped_width{0};
std::atomic<int> g_grouped_variant{0};
std::atomic<int> g_int8_tile{0};
std::atomic<bool> g_int8_fp16_tokens{false};

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

struct Workspace {
  int device;
  cudaStream_t stream;
  void* ptr;
  int64_t bytes;
  bool captured;   // handed to a kernel launch recorded into a CUDA graph
};
std::vector<Workspace> g_ws;
// The dense kernel's split workspace of one (device, stream): a fixed size per device, its
// arrival counters zero between launches.
struct SplitWorkspace {
  int device;
  cudaStream_t stream;
  void* ptr;
  int64_t counter_bytes;
};
std::vector<SplitWorkspace> g_sws;
// Buffers replaced by a larger one after a graph capture used them: a replay of that
// graph still reads and writes them, so they stay allocated until the process exits.
std::vector<void*> g_ws_kept;
// One mutex for each (device, stream) that has used a workspace (StreamLock).  A deque: they
// stay where they are.
struct StreamMutex {
  int device;
  cudaStream_t stream;
  std::mutex mu;
  StreamMutex(int d, cudaStream_t s) : device(d), stream(s) {}
};
std::deque<StreamMutex> g_stream_mu;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

const DeviceInfo* current_device(bsmma_status* err) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    *err = BSMMA_ERR_CUDA;
    return nullptr;
  }
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_dev_ready[dev]) {
    DeviceInfo d;
    d.device = dev;
    void* status = nullptr;
    if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaGetSymbolAddress(&status, g_device_status) != cudaSuccess) {
      *err = BSMMA_ERR_CUDA;
      return nullptr;
    }
    d.status = static_cast<int*>(status);
    g_dev[dev] = d;
    g_dev_ready[dev] = true;
  }
  return &g_dev[dev];
}

uint64_t wait_limit_ns() { return g_wait_limit_ns.load(); }
int dense_variant() { return g_dense_variant.load(); }
int grouped_tile_width() { return g_grouped_width.load(); }
int grouped_variant() { return g_grouped_variant.load(); }
int int8_tile() { return g_int8_tile.load(); }
bool int8_fp16_tokens() { return g_int8_fp16_tokens.load(); }
void count_launches(int n) { g_launches += n; }

bsmma_status encode_tmap_u8(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                            uint64_t row_stride, uint32_t box_inner, uint32_t box_outer) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                           cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn)
        return BSMMA_ERR_CUDA;
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
  }
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {row_stride};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSMMA_OK : BSMMA_ERR_INVALID_ARG;
}

bsmma_status encode_tmap_words(CUtensorMap* map, const void* base, uint64_t inner,
                               uint64_t outer, uint32_t box_inner, uint32_t box_outer) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                           cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn)
        return BSMMA_ERR_CUDA;
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
  }
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * 4};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSMMA_OK : BSMMA_ERR_INVALID_ARG;
}

bsmma_status encode_tmap_bf16_out(CUtensorMap* map, const void* base, uint64_t cols,
                                  uint64_t rows, uint32_t box_cols, uint32_t box_rows) {
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                           cudaEnableDefault, &q) != cudaSuccess ||
          q != cudaDriverEntryPointSuccess || !fn)
        return BSMMA_ERR_CUDA;
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
  }
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? BSMMA_OK : BSMMA_ERR_INVALID_ARG;
}

namespace {

__global__ void wait_probe_kernel(int* status, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // Nothing ever arrives on `bar`: the bounded wait must give up and latch a timeout.
  if (threadIdx.x == 0) mbar_wait(&bar, 0, limit_ns, &abort_flag, status);
}

constexpr int64_t kMaxTmaDim = (int64_t(1) << 32) - 1;
constexpr int64_t kMaxStride = (int64_t(1) << 40) - 16;

// Workspace of at least `bytes` for (current device, stream).
bsmma_status get_workspace(int64_t bytes, cudaStream_t stream, void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSMMA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  Workspace* w = nullptr;
  for (auto& e : g_ws)
    if (e.device == dev && e.stream == stream) w = &e;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return BSMMA_ERR_CUDA;
  const bool capturing = cap != cudaStreamCaptureStatusNone;
  if (w && w->bytes >= bytes) {
    if (capturing) w->captured = true;
    *out = w->ptr;
    return BSMMA_OK;
  }
  if (capturing) return BSMMA_ERR_WORKSPACE;
  int64_t grow = bytes + bytes / 4 + 4096;
  void* p = nullptr;
  if (cudaMalloc(&p, static_cast<size_t>(grow)) != cudaSuccess) return BSMMA_ERR_CUDA;
  if (w) {
    if (w->captured) {
      g_ws_kept.push_back(w->ptr);   // a captured graph may still be replayed on it
    } else {
      // earlier kernels on this stream may still read the old buffer
      if (cudaStreamSynchronize(stream) != cudaSuccess) {
        cudaFree(p);
        return BSMMA_ERR_CUDA;
      }
      cudaFree(w->ptr);
    }
    w->ptr = p;
    w->bytes = grow;
    w->captured = false;
  } else {
    g_ws.push_back(Workspace{dev, stream, p, grow, false});
  }
  *out = p;
  return BSMMA_OK;
}

int64_t align_up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

}  // namespace

StreamLock::StreamLock(cudaStream_t stream) {
  int dev = -1;
  cudaGetDevice(&dev);   // (a failure is the lookup's to report)
  std::mutex* mu = nullptr;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto& e : g_stream_mu)
      if (e.device == dev && e.stream == stream) mu = &e.mu;
    if (!mu) mu = &g_stream_mu.emplace_back(dev, stream).mu;
  }
  lk_ = std::unique_lock<std::mutex>(*mu);
}

bsmma_status stream_workspace(int64_t bytes, cudaStream_t stream, void** out) {
  return get_workspace(bytes, stream, out);
}

bsmma_status split_workspace(cudaStream_t stream, float** part, int** arrivals) {
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  std::lock_guard<std::mutex> lk(g_mu);
  for (auto& e : g_sws)
    if (e.device == dev->device && e.stream == stream) {
      *arrivals = static_cast<int*>(e.ptr);
      *part = reinterpret_cast<float*>(static_cast<uint8_t*>(e.ptr) + e.counter_bytes);
      return BSMMA_OK;
    }
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(stream, &cap) != cudaSuccess) return BSMMA_ERR_CUDA;
  if (cap != cudaStreamCaptureStatusNone) return BSMMA_ERR_WORKSPACE;
  const int64_t sms = dev->sm_count;
  const int64_t counter_bytes = align_up(sms * 8 * 4, 256);
  const int64_t bytes = counter_bytes + 2 * sms * 128 * 256 * 4;
  void* p = nullptr;
  if (cudaMalloc(&p, static_cast<size_t>(bytes)) != cudaSuccess) return BSMMA_ERR_CUDA;
  if (cudaMemsetAsync(p, 0, static_cast<size_t>(counter_bytes), stream) != cudaSuccess) {
    cudaFree(p);
    return BSMMA_ERR_CUDA;
  }
  g_sws.push_back(SplitWorkspace{dev->device, stream, p, counter_bytes});
  *arrivals = static_cast<int*>(p);
  *part = reinterpret_cast<float*>(static_cast<uint8_t*>(p) + counter_bytes);
  return BSMMA_OK;
}

bsmma_status validate_dense(const void* A, const void* sA, const void* B, const void* sB,
                            const void* D, int64_t M, int64_t N, int64_t K, bsmma_layout layout,
                            bsmma_fmt a_fmt, bsmma_fmt b_fmt) {
  if (M < 0 || N < 0 || K < 0 || K % 32 != 0) return BSMMA_ERR_INVALID_ARG;
  if (layout < BSMMA_NT || layout > BSMMA_TN) return BSMMA_ERR_INVALID_ARG;
  if (a_fmt < BSMMA_E4M3 || a_fmt > BSMMA_E2M1 || b_fmt < BSMMA_E4M3 || b_fmt > BSMMA_E2M1)
    return BSMMA_ERR_INVALID_ARG;
  const bool fp4a = a_fmt == BSMMA_E2M1, fp4b = b_fmt == BSMMA_E2M1;
  if (fp4a != fp4b) return BSMMA_ERR_UNSUPPORTED;
  if (fp4a && layout != BSMMA_NT) return BSMMA_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return BSMMA_OK;
  if (!D) return BSMMA_ERR_INVALID_ARG;
  if (N % 8 != 0 || !aligned16(D)) return BSMMA_ERR_MISALIGNED;
  if (K == 0) return BSMMA_OK;
  if (!A || !B || !sA || !sB) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(sA) || !aligned16(sB))
    return BSMMA_ERR_MISALIGNED;
  if (layout != BSMMA_NT && N % 16 != 0) return BSMMA_ERR_MISALIGNED;
  if (layout == BSMMA_TN && M % 16 != 0) return BSMMA_ERR_MISALIGNED;
  if (M > kMaxTmaDim || N > kMaxTmaDim || K > kMaxTmaDim) return BSMMA_ERR_INVALID_ARG;
  // tensor-copy coordinates are 32-bit signed
  if (M >= INT32_MAX || N >= INT32_MAX || K >= INT32_MAX) return BSMMA_ERR_INVALID_ARG;
  if (M > kMaxStride || N > kMaxStride || K > kMaxStride) return BSMMA_ERR_INVALID_ARG;
  // tile ids are 32-bit
  if ((M + 127) / 128 * ((N + 255) / 256) > INT32_MAX / 2) return BSMMA_ERR_INVALID_ARG;
  return BSMMA_OK;
}

// Validation of the fused output stage's extra arguments.
bsmma_status check_epilogue(const void* bias, bsmma_activation act) {
  if (act < BSMMA_ACT_NONE || act > BSMMA_ACT_SILU) return BSMMA_ERR_INVALID_ARG;
  if (bias && !aligned16(bias)) return BSMMA_ERR_MISALIGNED;
  return BSMMA_OK;
}

namespace {
// D[m][n] = act(bias[n]) (the output stage of an all-zero accumulator, K == 0).
__global__ void bias_act_fill_kernel(Epilogue e, __nv_bfloat16* D, int64_t M, int64_t N) {
  const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const int64_t vecs = M * (N / 8);
  for (int64_t v = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; v < vecs;
       v += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t m = v / (N / 8), c = (v - m * (N / 8)) * 8;
    store8(D + m * N + c, zero, c, e);
  }
}
}  // namespace

// K == 0: no products, so D = act(bias) per column (zero without a bias: every activation
// maps 0 to 0).
bsmma_status zero_k_epilogue(const void* bias, bsmma_activation act, void* D, int64_t M, int64_t N,
                             cudaStream_t s) {
  if (!bias) return cuda_ok(cudaMemsetAsync(D, 0, static_cast<size_t>(M * N * 2), s));
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  Epilogue e;
  e.bias = static_cast<const __nv_bfloat16*>(bias);
  e.act = static_cast<int>(act);
  bias_act_fill_kernel<<<dev->sm_count * 4, 256, 0, s>>>(e, static_cast<__nv_bfloat16*>(D), M, N);
  count_launches(1);
  return cuda_ok(cudaGetLastError());
}

}  // namespace bsmma

using namespace bsmma;

extern "C" {

int64_t mx_scale_tiled_bytes(int64_t rows, int64_t kblocks, bsmma_scale_role role) {
  if (role != BSMMA_SCALES_A && role != BSMMA_SCALES_B) return 0;
  return wide_scale_bytes(rows, kblocks, static_cast<int>(role));
}

bsmma_status mx_scale_relayout(const uint8_t* s_plain, int64_t rows, int64_t kblocks,
                               bsmma_scale_role role, uint8_t* s_tiled, bsmma_stream stream) {
  if (rows < 0 || kblocks < 0) return BSMMA_ERR_INVALID_ARG;
  if (role != BSMMA_SCALES_A && role != BSMMA_SCALES_B) return BSMMA_ERR_INVALID_ARG;
  if (rows == 0 || kblocks == 0) return BSMMA_OK;
  if (!s_plain || !s_tiled) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(s_tiled)) return BSMMA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (role == BSMMA_SCALES_A)
    return launch_wide_relayout(s_plain, rows, s_tiled, nullptr, 0, nullptr, kblocks, s);
  return launch_wide_relayout(nullptr, 0, nullptr, s_plain, rows, s_tiled, kblocks, s);
}

bsmma_status mx_gemm_tiled(const void* A, const uint8_t* sA_tiled, const void* B,
                           const uint8_t* sB_tiled, void* D, int64_t M, int64_t N, int64_t K,
                           bsmma_layout layout, bsmma_fmt a_fmt, bsmma_fmt b_fmt,
                           bsmma_stream stream) {
  bsmma_status st = validate_dense(A, sA_tiled, B, sB_tiled, D, M, N, K, layout, a_fmt, b_fmt);
  if (st != BSMMA_OK || M == 0 || N == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return cuda_ok(cudaMemsetAsync(D, 0, static_cast<size_t>(M * N * 2), s));
  return launch_mx_gemm(A, sA_tiled, B, sB_tiled, D, M, N, K, layout, a_fmt, b_fmt, s);
}

bsmma_status mx_gemm(const void* A, const uint8_t* sA, const void* B, const uint8_t* sB, void* D,
                     int64_t M, int64_t N, int64_t K, bsmma_layout layout, bsmma_fmt a_fmt,
                     bsmma_fmt b_fmt, bsmma_stream stream) {
  bsmma_status st = validate_dense(A, sA, B, sB, D, M, N, K, layout, a_fmt, b_fmt);
  if (st != BSMMA_OK || M == 0 || N == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return cuda_ok(cudaMemsetAsync(D, 0, static_cast<size_t>(M * N * 2), s));
  const int64_t bytes_a = align_up(wide_scale_bytes(M, K / 32, 0), 256);
  const int64_t bytes_b = wide_scale_bytes(N, K / 32, 1);
  const StreamLock lock(s);
  void* ws = nullptr;
  st = get_workspace(bytes_a + bytes_b, s, &ws);
  if (st != BSMMA_OK) return st;
  uint8_t* ta = static_cast<uint8_t*>(ws);
  uint8_t* tb = ta + bytes_a;
  st = launch_wide_relayout(sA, M, ta, sB, N, tb, K / 32, s);
  if (st != BSMMA_OK) return st;
  return launch_mx_gemm(A, ta, B, tb, D, M, N, K, layout, a_fmt, b_fmt, s);
}


bsmma_status mx_gemm_tiled_bias_act(const void* A, const uint8_t* sA_tiled, const void* B,
                                    const uint8_t* sB_tiled, const void* bias,
                                    bsmma_activation act, void* D, int64_t M, int64_t N,
                                    int64_t K, bsmma_layout layout, bsmma_fmt a_fmt,
                                    bsmma_fmt b_fmt, bsmma_stream stream) {
  bsmma_status st = validate_dense(A, sA_tiled, B, sB_tiled, D, M, N, K, layout, a_fmt, b_fmt);
  if (st == BSMMA_OK) st = check_epilogue(bias, act);
  if (st != BSMMA_OK || M == 0 || N == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_k_epilogue(bias, act, D, M, N, s);
  return launch_mx_gemm(A, sA_tiled, B, sB_tiled, D, M, N, K, layout, a_fmt, b_fmt, s, bias,
                        static_cast<int>(act));
}

bsmma_status mx_gemm_bias_act(const void* A, const uint8_t* sA, const void* B, const uint8_t* sB,
                              const void* bias, bsmma_activation act, void* D, int64_t M,
                              int64_t N, int64_t K, bsmma_layout layout, bsmma_fmt a_fmt,
                              bsmma_fmt b_fmt, bsmma_stream stream) {
  bsmma_status st = validate_dense(A, sA, B, sB, D, M, N, K, layout, a_fmt, b_fmt);
  if (st == BSMMA_OK) st = check_epilogue(bias, act);
  if (st != BSMMA_OK || M == 0 || N == 0) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (K == 0) return zero_k_epilogue(bias, act, D, M, N, s);
  const int64_t bytes_a = align_up(wide_scale_bytes(M, K / 32, 0), 256);
  const int64_t bytes_b = wide_scale_bytes(N, K / 32, 1);
  const StreamLock lock(s);
  void* ws = nullptr;
  st = get_workspace(bytes_a + bytes_b, s, &ws);
  if (st != BSMMA_OK) return st;
  uint8_t* ta = static_cast<uint8_t*>(ws);
  uint8_t* tb = ta + bytes_a;
  st = launch_wide_relayout(sA, M, ta, sB, N, tb, K / 32, s);
  if (st != BSMMA_OK) return st;
  return launch_mx_gemm(A, ta, B, tb, D, M, N, K, layout, a_fmt, b_fmt, s, bias,
                        static_cast<int>(act));
}

namespace {
bsmma_status check_grouped(const uint8_t* A, const float* sA, const uint8_t* B, const float* sB,
                           const void* D, const int64_t* m_sizes, int64_t total_M, int G,
                           int64_t N, int64_t K) {
  if (G < 1 || G > 64 || total_M < 0 || N <= 0 || K <= 0) return BSMMA_ERR_INVALID_ARG;
  if (N % 128 != 0 || K % 128 != 0) return BSMMA_ERR_INVALID_ARG;
  if (!B || !sB || !m_sizes) return BSMMA_ERR_INVALID_ARG;
  if (total_M > 0 && (!A || !sA || !D)) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(B) || (total_M > 0 && (!aligned16(A) || !aligned16(D))) ||
      (reinterpret_cast<uintptr_t>(m_sizes) & 7u) != 0)
    return BSMMA_ERR_MISALIGNED;
  if (total_M >= INT32_MAX || static_cast<int64_t>(G) * N >= INT32_MAX || K > kMaxStride)
    return BSMMA_ERR_INVALID_ARG;
  return BSMMA_OK;
}
}  // namespace

bsmma_status grouped_fp8_gemm(const uint8_t* A, const float* sA, const uint8_t* B,
                              const float* sB, void* D, const int64_t* m_sizes, int64_t total_M,
                              int G, int64_t N, int64_t K, bsmma_stream stream) {
  const bsmma_status st = check_grouped(A, sA, B, sB, D, m_sizes, total_M, G, N, K);
  if (st != BSMMA_OK) return st;
  return launch_grouped(A, sA, B, sB, D, m_sizes, total_M, G, N, K,
                        reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status grouped_fp8_gemm_packed(const uint8_t* A, const float* sA, const uint8_t* B_packed,
                                     const float* sB, void* D, const int64_t* m_sizes,
                                     int64_t total_M, int G, int64_t N, int64_t K,
                                     bsmma_stream stream) {
  const bsmma_status st = check_grouped(A, sA, B_packed, sB, D, m_sizes, total_M, G, N, K);
  if (st != BSMMA_OK) return st;
  return launch_grouped(A, sA, B_packed, sB, D, m_sizes, total_M, G, N, K,
                        reinterpret_cast<cudaStream_t>(stream), true);
}

bsmma_status grouped_fp8_pack_weights(const uint8_t* W, int64_t G, int64_t N, int64_t K,
                                      uint8_t* W_packed, bsmma_stream stream) {
  if (G < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return BSMMA_ERR_INVALID_ARG;
  if (G == 0 || N == 0 || K == 0) return BSMMA_OK;
  if (!W || !W_packed) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned16(W_packed)) return BSMMA_ERR_MISALIGNED;
  if (W == W_packed) return BSMMA_ERR_INVALID_ARG;   // not in place
  return launch_pack_weights(W, G, N, K, W_packed, reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status grouped_bf16_gemm(const void* X, const void* W, void* D, const int64_t* m_sizes,
                               int64_t total_M, int G, int64_t N, int64_t K,
                               bsmma_stream stream) {
  if (G < 1 || G > 64 || total_M < 0 || N <= 0 || K <= 0) return BSMMA_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0) return BSMMA_ERR_INVALID_ARG;
  if (!W || !m_sizes) return BSMMA_ERR_INVALID_ARG;
  if (total_M > 0 && (!X || !D)) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(W) || (total_M > 0 && (!aligned16(X) || !aligned16(D))) ||
      (reinterpret_cast<uintptr_t>(m_sizes) & 7u) != 0)
    return BSMMA_ERR_MISALIGNED;
  if (total_M >= INT32_MAX || static_cast<int64_t>(G) * N >= INT32_MAX || 2 * K > kMaxStride)
    return BSMMA_ERR_INVALID_ARG;
  return launch_grouped_bf16(X, W, D, m_sizes, total_M, G, N, K,
                             reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status mx_quantize(const void* x, bsmma_dtype x_dtype, int64_t rows, int64_t cols,
                         bsmma_fmt fmt, int colwise, uint8_t* codes, uint8_t* scales,
                         bsmma_stream stream) {
  if (x_dtype != BSMMA_BF16 && x_dtype != BSMMA_F32) return BSMMA_ERR_INVALID_ARG;
  if (fmt != BSMMA_E4M3 && fmt != BSMMA_E5M2 && fmt != BSMMA_E2M1) return BSMMA_ERR_INVALID_ARG;
  if (rows < 0 || cols < 0 || (colwise != 0 && colwise != 1)) return BSMMA_ERR_INVALID_ARG;
  if (colwise && fmt == BSMMA_E2M1) return BSMMA_ERR_UNSUPPORTED;
  if (colwise ? (rows % 32 != 0 || cols % 16 != 0) : (cols % 32 != 0)) return BSMMA_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return BSMMA_OK;
  if (!x || !codes || !scales) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes)) return BSMMA_ERR_MISALIGNED;
  return launch_mx_quantize(x, x_dtype == BSMMA_F32, rows, cols, fmt, colwise != 0, codes, scales,
                            reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status fp8_group_quantize(const void* x, bsmma_dtype x_dtype, int64_t total_M, int64_t K,
                                const int64_t* m_sizes, int G, uint8_t* codes, float* scales,
                                bsmma_stream stream) {
  if (x_dtype != BSMMA_BF16 && x_dtype != BSMMA_F32) return BSMMA_ERR_INVALID_ARG;
  if (G < 1 || G > 64 || total_M < 0 || K <= 0 || K % 128 != 0) return BSMMA_ERR_INVALID_ARG;
  if (!m_sizes) return BSMMA_ERR_INVALID_ARG;
  if (total_M > 0 && (!x || !codes || !scales)) return BSMMA_ERR_INVALID_ARG;
  if ((total_M + 63) / 64 * (K / 128) >= INT32_MAX) return BSMMA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(m_sizes) & 7u) != 0) return BSMMA_ERR_MISALIGNED;
  if (total_M > 0 && (!aligned16(x) || !aligned16(codes) ||
                      (reinterpret_cast<uintptr_t>(scales) & 3u) != 0))
    return BSMMA_ERR_MISALIGNED;
  return launch_group_quantize(x, x_dtype == BSMMA_F32, total_M, K, m_sizes, G, codes, scales,
                               reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status fp8_block_quantize(const void* w, bsmma_dtype w_dtype, int64_t G, int64_t N,
                                int64_t K, uint8_t* codes, float* scales, bsmma_stream stream) {
  if (w_dtype != BSMMA_BF16 && w_dtype != BSMMA_F32) return BSMMA_ERR_INVALID_ARG;
  if (G < 0 || N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return BSMMA_ERR_INVALID_ARG;
  if (G == 0 || N == 0 || K == 0) return BSMMA_OK;
  if (G * (N / 128) * (K / 128) >= INT32_MAX) return BSMMA_ERR_INVALID_ARG;
  if (!w || !codes || !scales) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(w) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3u) != 0)
    return BSMMA_ERR_MISALIGNED;
  return launch_block_quantize(w, w_dtype == BSMMA_F32, G, N, K, codes, scales,
                               reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool known_dtype(bsmma_dtype d) { return d == BSMMA_BF16 || d == BSMMA_F32; }

bsmma_status check_route(bsmma_dtype dtype, int64_t T, int E, int k, bsmma_moe_score score,
                         int renormalize) {
  if (!known_dtype(dtype) || (score != BSMMA_SOFTMAX && score != BSMMA_SIGMOID))
    return BSMMA_ERR_INVALID_ARG;
  if (T < 0 || T >= INT32_MAX || E < 1 || E > 1024 || k < 1 || k > 32 || k > E ||
      (renormalize != 0 && renormalize != 1))
    return BSMMA_ERR_INVALID_ARG;
  return BSMMA_OK;
}
}  // namespace

bsmma_status moe_route(const void* logits, bsmma_dtype logits_dtype, int64_t T, int E, int k,
                       bsmma_moe_score score, const float* bias, int groups, int topk_groups,
                       int group_top, int renormalize, float scale, int32_t* ids, float* weights,
                       bsmma_stream stream) {
  const bsmma_status st = check_route(logits_dtype, T, E, k, score, renormalize);
  if (st != BSMMA_OK) return st;
  if (groups < 1 || groups > 32 || E % groups != 0 || topk_groups < 1 || topk_groups > groups ||
      group_top < 1 || group_top > 2 || k > topk_groups * (E / groups))
    return BSMMA_ERR_INVALID_ARG;
  if (T == 0) return BSMMA_OK;
  if (!logits || !ids || !weights) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(bias, 4))
    return BSMMA_ERR_MISALIGNED;
  return launch_route(logits, logits_dtype == BSMMA_F32, T, E, k, score == BSMMA_SIGMOID, bias,
                      groups, topk_groups, group_top, renormalize != 0, scale, ids, weights,
                      reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status moe_route_backward(const void* logits, bsmma_dtype logits_dtype, int64_t T, int E,
                                int k, bsmma_moe_score score, int renormalize, float scale,
                                const int32_t* ids, const float* dweights, void* dlogits,
                                bsmma_stream stream) {
  const bsmma_status st = check_route(logits_dtype, T, E, k, score, renormalize);
  if (st != BSMMA_OK || T == 0) return st;
  if (!logits || !ids || !dweights || !dlogits) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(dlogits) || !aligned_to(ids, 4) || !aligned_to(dweights, 4))
    return BSMMA_ERR_MISALIGNED;
  return launch_route_backward(logits, logits_dtype == BSMMA_F32, T, E, k, score == BSMMA_SIGMOID,
                               renormalize != 0, scale, ids, dweights, dlogits,
                               reinterpret_cast<cudaStream_t>(stream));
}

int64_t moe_plan_workspace_bytes(int64_t T, int k, int E) {
  if (T <= 0 || k < 1 || E < 1 || T >= INT32_MAX) return 0;
  return plan_workspace_bytes(T * k, E);
}

bsmma_status moe_plan(const int32_t* ids, int64_t T, int k, int E, int64_t* m_sizes, int32_t* src,
                      int32_t* pos, bsmma_stream stream) {
  if (T < 0 || T >= INT32_MAX || k < 1 || E < 1 || E > 1024 || T * k >= INT32_MAX - 4096)
    return BSMMA_ERR_INVALID_ARG;
  if (!m_sizes) return BSMMA_ERR_INVALID_ARG;
  if (!aligned_to(m_sizes, 8)) return BSMMA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return cuda_ok(cudaMemsetAsync(m_sizes, 0, static_cast<size_t>(E) * 8, s));
  if (!ids || !src || !pos) return BSMMA_ERR_INVALID_ARG;
  if (!aligned_to(ids, 4) || !aligned_to(src, 4) || !aligned_to(pos, 4)) return BSMMA_ERR_MISALIGNED;
  const int64_t bytes = plan_workspace_bytes(T * k, E);
  if (bytes == 0) return launch_plan(ids, T * k, E, m_sizes, src, pos, nullptr, s);
  const StreamLock lock(s);
  void* ws = nullptr;
  const bsmma_status st = get_workspace(bytes, s, &ws);
  if (st != BSMMA_OK) return st;
  return launch_plan(ids, T * k, E, m_sizes, src, pos, ws, s);
}

bsmma_status int8_quantize(const void* x, bsmma_dtype x_dtype, int64_t x_rows, int64_t K,
                           const int32_t* src, int k, int64_t rows, int8_t* codes, float* scales,
                           bsmma_stream stream) {
  if (!known_dtype(x_dtype) || x_rows < 0 || rows < 0 || rows >= INT32_MAX || K <= 0 ||
      K % 16 != 0 || K >= INT32_MAX || k < 1)
    return BSMMA_ERR_INVALID_ARG;
  if (!src && rows != x_rows) return BSMMA_ERR_INVALID_ARG;
  if (rows == 0) return BSMMA_OK;
  if ((x_rows > 0 && !x) || !codes || !scales) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(codes) || !aligned_to(scales, 4) || !aligned_to(src, 4))
    return BSMMA_ERR_MISALIGNED;
  return launch_int8_quantize(x, x_dtype == BSMMA_F32, x_rows, rows, K, src, k, codes, scales,
                              reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status int8_gemm(const int8_t* A, const float* sA, const int8_t* B, const float* sB,
                       const void* bias, void* D, bsmma_dtype d_dtype, int64_t M, int64_t N,
                       int64_t K, bsmma_stream stream) {
  if (!known_dtype(d_dtype) || M < 0 || N < 0 || K < 0 || K % 16 != 0) return BSMMA_ERR_INVALID_ARG;
  // tile coordinates past the last row stay within 32 bits
  if (M >= INT32_MAX - 511 || N >= INT32_MAX - 511 || K >= INT32_MAX - 511) return BSMMA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return BSMMA_OK;
  if (!D || !sA || !sB || (K > 0 && (!A || !B))) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(D) || !aligned_to(sA, 4) || !aligned_to(sB, 4) ||
      !aligned_to(bias, 2))
    return BSMMA_ERR_MISALIGNED;
  return launch_int8_gemm(A, sA, B, sB, bias, D, d_dtype == BSMMA_F32, nullptr, M, 1, N, K,
                          reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status grouped_int8_gemm(const int8_t* X, const float* sX, const int8_t* W, const float* sW,
                               void* D, bsmma_dtype d_dtype, const int64_t* m_sizes,
                               int64_t total_M, int G, int64_t N, int64_t K, bsmma_stream stream) {
  if (!known_dtype(d_dtype) || G < 1 || G > 1024 || total_M < 0 || N <= 0 || K <= 0 || K % 16 != 0)
    return BSMMA_ERR_INVALID_ARG;
  if (total_M >= INT32_MAX - 511 || K >= INT32_MAX - 511 || N >= INT32_MAX - 511 ||
      static_cast<int64_t>(G) * N >= INT32_MAX - 511)
    return BSMMA_ERR_INVALID_ARG;
  if (!W || !sW || !m_sizes) return BSMMA_ERR_INVALID_ARG;
  if (total_M > 0 && (!X || !sX || !D)) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(W) || !aligned_to(sW, 4) || !aligned_to(m_sizes, 8) || !aligned16(X) ||
      !aligned_to(sX, 4) || !aligned16(D))
    return BSMMA_ERR_MISALIGNED;
  return launch_int8_gemm(X, sX, W, sW, nullptr, D, d_dtype == BSMMA_F32, m_sizes, total_M, G, N, K,
                          reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bsmma_status check_combine(bsmma_dtype dtype, int64_t R, int64_t H, int64_t T, int k) {
  if (!known_dtype(dtype) || H <= 0 || H > (1 << 24) || T < 0 || T >= INT32_MAX || R < 0 ||
      R >= INT32_MAX || k < 1 || k > 32 || T * k >= INT32_MAX)
    return BSMMA_ERR_INVALID_ARG;
  if (H % (dtype == BSMMA_F32 ? 4 : 8) != 0) return BSMMA_ERR_MISALIGNED;
  return BSMMA_OK;
}
}  // namespace

bsmma_status moe_combine(const void* Y, bsmma_dtype dtype, int64_t R, int64_t H, const int32_t* pos,
                         const float* weights, int64_t T, int k, void* out, bsmma_stream stream) {
  const bsmma_status st = check_combine(dtype, R, H, T, k);
  if (st != BSMMA_OK || T == 0) return st;
  if ((R > 0 && !Y) || !pos || !out) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(Y) || !aligned16(out) || !aligned_to(pos, 4) || !aligned_to(weights, 4))
    return BSMMA_ERR_MISALIGNED;
  return launch_combine(Y, dtype == BSMMA_F32, R, H, pos, weights, T, k, out,
                        reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status moe_combine_backward(const void* dout, bsmma_dtype dtype, int64_t H, const void* Y,
                                  const int32_t* src, const int32_t* pos, const float* weights,
                                  int64_t T, int k, void* dY, float* dweights, bsmma_stream stream) {
  const bsmma_status st = check_combine(dtype, 0, H, T, k);
  if (st != BSMMA_OK || T == 0) return st;
  if (!dout || (dweights && !Y) || !src || !pos || !dY) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(Y) || !aligned16(dY) || !aligned_to(src, 4) ||
      !aligned_to(pos, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4))
    return BSMMA_ERR_MISALIGNED;
  return launch_combine_backward(dout, dtype == BSMMA_F32, H, Y, src, pos, weights, T, k, dY,
                                 dweights, reinterpret_cast<cudaStream_t>(stream));
}

namespace {
bool known_norm(bsmma_norm n, bool none) {
  return n == BSMMA_NORM_RMS || n == BSMMA_NORM_LAYER || (none && n == BSMMA_NORM_NONE);
}
// The norm's own arguments; `more`: anything else that only a norm has.
bsmma_status check_norm(bsmma_norm norm, bool none, float eps, const float* weight, const float* bias,
                        bool more = false) {
  if (!known_norm(norm, none)) return BSMMA_ERR_INVALID_ARG;
  if (norm == BSMMA_NORM_NONE) return weight || bias || more ? BSMMA_ERR_INVALID_ARG : BSMMA_OK;
  if (!(eps > 0.f) || eps > 3.402823466e38f) return BSMMA_ERR_INVALID_ARG;
  return aligned16(weight) && aligned16(bias) ? BSMMA_OK : BSMMA_ERR_MISALIGNED;
}
bsmma_status check_rows(bsmma_dtype stream_dtype, bsmma_dtype branch_dtype, int64_t T, int64_t H) {
  if (!known_dtype(stream_dtype) || !known_dtype(branch_dtype) || T < 0 || T >= INT32_MAX || H < 8 ||
      H > 16384)
    return BSMMA_ERR_INVALID_ARG;
  if (stream_dtype == BSMMA_BF16 && branch_dtype == BSMMA_F32) return BSMMA_ERR_UNSUPPORTED;
  return H % 8 == 0 ? BSMMA_OK : BSMMA_ERR_MISALIGNED;
}
bool is_mx(bsmma_operand f) {
  return f == BSMMA_OPERAND_E4M3 || f == BSMMA_OPERAND_E5M2 || f == BSMMA_OPERAND_E2M1;
}
bsmma_status check_form(bsmma_operand form, bool f32_stream, int64_t T, int64_t H, const void* out,
                        const void* scales) {
  if (form < BSMMA_OPERAND_BF16 || form > BSMMA_OPERAND_E2M1) return BSMMA_ERR_INVALID_ARG;
  if (form == BSMMA_OPERAND_F32 && !f32_stream) return BSMMA_ERR_UNSUPPORTED;
  if (is_mx(form) && H % 32 != 0) return BSMMA_ERR_INVALID_ARG;
  if (T == 0) return BSMMA_OK;
  const bool coded = form == BSMMA_OPERAND_INT8 || is_mx(form);
  if (!out || coded != (scales != nullptr)) return BSMMA_ERR_INVALID_ARG;
  return aligned16(out) && (form != BSMMA_OPERAND_INT8 || aligned_to(scales, 4)) ? BSMMA_OK
                                                                                 : BSMMA_ERR_MISALIGNED;
}
bsmma_status check_gate(const void* gate, int64_t gate_rows) {
  if (gate && gate_rows < 1) return BSMMA_ERR_INVALID_ARG;
  return aligned16(gate) ? BSMMA_OK : BSMMA_ERR_MISALIGNED;
}
// p in 16 bits, and what keeps the mean.
bsmma_status make_drop(float p, const int64_t* rng, DropArgs* d) {
  if (!(p >= 0.f && p < 1.f)) return BSMMA_ERR_INVALID_ARG;
  const double steps = std::nearbyint(static_cast<double>(p) * 65536.0);
  d->threshold = steps > 65535.0 ? 65535u : static_cast<uint32_t>(steps);
  d->scale = static_cast<float>(65536.0 / (65536.0 - d->threshold));
  d->rng = rng;
  if (p > 0.f && !rng) return BSMMA_ERR_INVALID_ARG;
  return aligned_to(rng, 8) ? BSMMA_OK : BSMMA_ERR_MISALIGNED;
}
// A gate's rows as the kernels divide by them.
int64_t bounded_rows(int64_t gate_rows, int64_t T) { return gate_rows < T ? gate_rows : T; }

bsmma_status run_grad(const BranchGradArgs& a, bool leave, cudaStream_t s) {
  if (!a.dweight && !a.dbias && !(a.dgate && a.gate_rows > 1)) return launch_branch_grad(a, leave, nullptr, s);
  const StreamLock lock(s);
  void* ws = nullptr;
  const bsmma_status st = get_workspace(branch_grad_workspace_bytes(a.T, a.H), s, &ws);
  if (st != BSMMA_OK) return st;
  return launch_branch_grad(a, leave, ws, s);
}
bsmma_status clear_sums(float* dweight, float* dbias, int64_t H, cudaStream_t s) {
  for (float* p : {dweight, dbias})
    if (p && cudaMemsetAsync(p, 0, static_cast<size_t>(H) * 4, s) != cudaSuccess) return BSMMA_ERR_CUDA;
  return BSMMA_OK;
}
}  // namespace

#define BSMMA_TRY(expr)                        \
  do {                                         \
    const bsmma_status st_ = (expr);           \
    if (st_ != BSMMA_OK) return st_;           \
  } while (0)

bsmma_status branch_enter(const void* x, bsmma_dtype x_dtype, int64_t T, int64_t H, bsmma_norm norm,
                          float eps, const float* weight, const float* bias, bsmma_operand form,
                          void* out, void* scales, bsmma_stream stream) {
  BSMMA_TRY(check_rows(x_dtype, x_dtype, T, H));
  BSMMA_TRY(check_norm(norm, false, eps, weight, bias));
  BSMMA_TRY(check_form(form, x_dtype == BSMMA_F32, T, H, out, scales));
  if (T == 0) return BSMMA_OK;
  if (!x) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(x)) return BSMMA_ERR_MISALIGNED;
  EnterArgs a = {};
  a.x = x;
  a.x_f32 = x_dtype == BSMMA_F32;
  a.T = T;
  a.H = H;
  a.inv_h = 1.f / static_cast<float>(H);
  a.norm = {norm, eps, weight, bias};
  a.to = {form, out, scales};
  return launch_branch_enter(a, reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status branch_leave(const void* x, bsmma_dtype x_dtype, const void* y, bsmma_dtype y_dtype,
                          int64_t T, int64_t H, bsmma_norm norm, float eps, const float* weight,
                          const float* bias, const void* gate, int64_t gate_rows, float x_scale,
                          float y_scale, float p, const int64_t* rng, void* out, bsmma_norm next,
                          float next_eps, const float* next_weight, const float* next_bias,
                          bsmma_operand next_form, void* next_out, void* next_scales,
                          bsmma_stream stream) {
  BSMMA_TRY(check_rows(x_dtype, y_dtype, T, H));
  BSMMA_TRY(check_norm(norm, true, eps, weight, bias));
  BSMMA_TRY(check_gate(gate, gate_rows));
  BSMMA_TRY(check_norm(next, true, next_eps, next_weight, next_bias, next_out || next_scales));
  if (next != BSMMA_NORM_NONE)
    BSMMA_TRY(check_form(next_form, x_dtype == BSMMA_F32, T, H, next_out, next_scales));
  LeaveArgs a = {};
  BSMMA_TRY(make_drop(p, rng, &a.drop));
  if (T == 0) return BSMMA_OK;
  if (!x || !y || !out) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y) || !aligned16(out)) return BSMMA_ERR_MISALIGNED;
  a.x = x;
  a.x_f32 = x_dtype == BSMMA_F32;
  a.y = y;
  a.y_f32 = y_dtype == BSMMA_F32;
  a.T = T;
  a.H = H;
  a.inv_h = 1.f / static_cast<float>(H);
  a.norm = {norm, eps, weight, bias};
  a.gate = gate;
  a.gate_rows = bounded_rows(gate_rows, T);
  a.x_scale = x_scale;
  a.y_scale = y_scale;
  a.out = out;
  a.next = {next, next_eps, next_weight, next_bias};
  a.to = {next_form, next_out, next_scales};
  return launch_branch_leave(a, reinterpret_cast<cudaStream_t>(stream));
}

bsmma_status branch_enter_backward(const void* dh, bsmma_dtype h_dtype, const void* x,
                                   bsmma_dtype x_dtype, int64_t T, int64_t H, bsmma_norm norm,
                                   float eps, const float* weight, const void* dres, void* dx,
                                   float* dweight, float* dbias, bsmma_stream stream) {
  BSMMA_TRY(check_rows(x_dtype, h_dtype, T, H));
  BSMMA_TRY(check_norm(norm, false, eps, weight, nullptr));
  if (!aligned16(dweight) || !aligned16(dbias)) return BSMMA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return clear_sums(dweight, dbias, H, s);
  if (!dh || !x || !dx) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(dh) || !aligned16(x) || !aligned16(dres) || !aligned16(dx)) return BSMMA_ERR_MISALIGNED;
  BranchGradArgs a = {};
  a.d = dh;
  a.d_f32 = h_dtype == BSMMA_F32;
  a.v = x;
  a.v_f32 = x_dtype == BSMMA_F32;
  a.T = T;
  a.H = H;
  a.inv_h = 1.f / static_cast<float>(H);
  a.norm = {norm, eps, weight, nullptr};
  a.dres = dres;
  a.drop = {0u, 1.f, nullptr};
  a.dv = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  return run_grad(a, false, s);
}

bsmma_status branch_leave_backward(const void* dout, bsmma_dtype x_dtype, const void* y,
                                   bsmma_dtype y_dtype, int64_t T, int64_t H, bsmma_norm norm,
                                   float eps, const float* weight, const float* bias,
                                   const void* gate, int64_t gate_rows, float x_scale,
                                   float y_scale, float p, const int64_t* rng, void* dy, void* dx,
                                   float* dweight, float* dbias, float* dgate, bsmma_stream stream) {
  BSMMA_TRY(check_rows(x_dtype, y_dtype, T, H));
  BSMMA_TRY(check_norm(norm, true, eps, weight, bias, dweight || dbias));
  BSMMA_TRY(check_gate(gate, gate_rows));
  BranchGradArgs a = {};
  BSMMA_TRY(make_drop(p, rng, &a.drop));
  if (dgate && !gate) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(dweight) || !aligned16(dbias) || !aligned16(dgate)) return BSMMA_ERR_MISALIGNED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return clear_sums(dweight, dbias, H, s);
  if (!dout || !y || !dy) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(dout) || !aligned16(y) || !aligned16(dy) || !aligned16(dx)) return BSMMA_ERR_MISALIGNED;
  a.d = dout;
  a.d_f32 = x_dtype == BSMMA_F32;
  a.v = y;
  a.v_f32 = y_dtype == BSMMA_F32;
  a.T = T;
  a.H = H;
  a.inv_h = 1.f / static_cast<float>(H);
  a.norm = {norm, eps, weight, bias};
  a.gate = gate;
  a.gate_rows = bounded_rows(gate_rows, T);
  a.x_scale = x_scale;
  a.y_scale = y_scale;
  a.dv = dy;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dgate = dgate;
  return run_grad(a, true, s);
}

int64_t branch_backward_workspace_bytes(int64_t T, int64_t H) {
  if (T <= 0 || T >= INT32_MAX || H < 8 || H > 16384) return 0;
  return branch_grad_workspace_bytes(T, H);
}

bsmma_status dropout(const void* x, bsmma_dtype dtype, int64_t n, float p, const int64_t* rng, void* y,
                     bsmma_stream stream) {
  if (!known_dtype(dtype) || n < 0 || n >= (int64_t{1} << 40)) return BSMMA_ERR_INVALID_ARG;
  DropArgs d;
  BSMMA_TRY(make_drop(p, rng, &d));
  if (n == 0) return BSMMA_OK;
  if (!x || !y) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(y)) return BSMMA_ERR_MISALIGNED;
  return launch_dropout(x, dtype == BSMMA_F32, n, d, y, reinterpret_cast<cudaStream_t>(stream));
}

int64_t moe_step_workspace_bytes(int64_t T, int k, int64_t H, int64_t F) {
  if (T <= 0 || T > 32 || k < 1 || T * k > 1024 || H <= 0 || H > 65536 || F <= 0 || F > 65536) return 0;
  return step_workspace_bytes(T, k, H, F);
}

bsmma_status moe_step(const void* x, int64_t T, int64_t H, const int32_t* ids, const float* weights,
                      int k, int E, int64_t F, bsmma_operand form, const void* w_in,
                      const void* s_in, const void* w_out, const void* s_out,
                      bsmma_activation act, void* out, bsmma_stream stream) {
  if (form == BSMMA_OPERAND_F32) return BSMMA_ERR_UNSUPPORTED;
  if (form < BSMMA_OPERAND_BF16 || form > BSMMA_OPERAND_E2M1 || act < BSMMA_ACT_NONE || act > BSMMA_ACT_SILU)
    return BSMMA_ERR_INVALID_ARG;
  if (T < 0 || T > 32 || k < 1 || k > 1024 || T * k > 1024 || E < 1 || E > 1024 || H <= 0 || H > 65536 ||
      F <= 0 || F > 65536)
    return BSMMA_ERR_INVALID_ARG;
  const int piece = form == BSMMA_OPERAND_BF16 ? 8 : form == BSMMA_OPERAND_INT8 ? 16 : 32;
  if (H % piece != 0 || F % piece != 0) return BSMMA_ERR_INVALID_ARG;
  if ((form != BSMMA_OPERAND_BF16) != (s_in != nullptr) || (form != BSMMA_OPERAND_BF16) != (s_out != nullptr))
    return BSMMA_ERR_INVALID_ARG;
  if (T == 0) return BSMMA_OK;
  if (!x || !ids || !weights || !w_in || !w_out || !out) return BSMMA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_in) || !aligned16(w_out) || !aligned16(out) || !aligned_to(ids, 4) ||
      !aligned_to(weights, 4) || !aligned_to(s_in, 4) || !aligned_to(s_out, 4))
    return BSMMA_ERR_MISALIGNED;
  StepArgs a = {};
  a.x = x;
  a.T = T;
  a.H = H;
  a.ids = ids;
  a.weights = weights;
  a.k = k;
  a.E = E;
  a.F = F;
  a.w_in = w_in;
  a.s_in = s_in;
  a.w_out = w_out;
  a.s_out = s_out;
  a.act = act;
  a.out = static_cast<__nv_bfloat16*>(out);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const StreamLock lock(s);
  void* ws = nullptr;
  BSMMA_TRY(get_workspace(step_workspace_bytes(T, k, H, F), s, &ws));
  return launch_moe_step(a, form, ws, s);
}

bsmma_status bsmma_reserve_workspace(int64_t bytes, bsmma_stream stream) {
  if (bytes < 0) return BSMMA_ERR_INVALID_ARG;
  const StreamLock lock(reinterpret_cast<cudaStream_t>(stream));
  void* p = nullptr;
  bsmma_status st = get_workspace(bytes, reinterpret_cast<cudaStream_t>(stream), &p);
  if (st != BSMMA_OK) return st;
  float* part = nullptr;
  int* arrivals = nullptr;
  return split_workspace(reinterpret_cast<cudaStream_t>(stream), &part, &arrivals);
}

bsmma_status bsmma_device_status(bsmma_stream stream) {
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int v = 0, zero = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess) return BSMMA_ERR_CUDA;
  if (cudaMemcpy(&v, dev->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemcpy(dev->status, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess)
    return BSMMA_ERR_CUDA;
  if (v == BSMMA_DEV_TIMEOUT) {
    // a dense launch that gave up may have left split-unit arrival counts behind
    if (cudaDeviceSynchronize() != cudaSuccess) return BSMMA_ERR_CUDA;
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto& e : g_sws)
      if (e.device == dev->device &&
          cudaMemset(e.ptr, 0, static_cast<size_t>(e.counter_bytes)) != cudaSuccess)
        return BSMMA_ERR_CUDA;
  }
  return static_cast<bsmma_status>(v);
}

bsmma_status bsmma_set_wait_limit_ns(int64_t ns) {
  if (ns <= 0) return BSMMA_ERR_INVALID_ARG;
  g_wait_limit_ns = static_cast<uint64_t>(ns);
  return BSMMA_OK;
}

bsmma_status bsmma_set_dense_variant(int variant) {
  if (variant != 0 && variant != 1 && variant != 3) return BSMMA_ERR_INVALID_ARG;
  g_dense_variant = variant;
  return BSMMA_OK;
}

bsmma_status bsmma_set_grouped_tile_width(int width) {
  if (width != 0 && width != 128 && width != 256) return BSMMA_ERR_INVALID_ARG;
  g_grouped_width = width;
  return BSMMA_OK;
}

bsmma_status bsmma_set_grouped_variant(int variant) {
  if (variant != 0 && variant != 1 && variant != 3) return BSMMA_ERR_INVALID_ARG;
  g_grouped_variant = variant;
  return BSMMA_OK;
}

bsmma_status bsmma_set_int8_variant(int tile, int fp16_tokens) {
  const bool wide = fp16_tokens == 1 && (tile == 192 || tile == 256);
  const bool plain = fp16_tokens == 0 && (tile == 0 || tile == 1 || tile == 32 || tile == 64 ||
                                          tile == 128 || tile == 256);
  if (!wide && !plain) return BSMMA_ERR_INVALID_ARG;
  g_int8_tile = tile;
  g_int8_fp16_tokens = wide;
  return BSMMA_OK;
}

const char* bsmma_status_string(bsmma_status s) {
  switch (s) {
    case BSMMA_ERR_SCRATCH_LIMIT: return "BSMMA_ERR_SCRATCH_LIMIT";
    case BSMMA_OK: return "BSMMA_OK";
    case BSMMA_ERR_INVALID_ARG: return "BSMMA_ERR_INVALID_ARG";
    case BSMMA_ERR_UNSUPPORTED: return "BSMMA_ERR_UNSUPPORTED";
    case BSMMA_ERR_MISALIGNED: return "BSMMA_ERR_MISALIGNED";
    case BSMMA_ERR_WORKSPACE: return "BSMMA_ERR_WORKSPACE";
    case BSMMA_ERR_CUDA: return "BSMMA_ERR_CUDA";
    case BSMMA_DEV_TIMEOUT: return "BSMMA_DEV_TIMEOUT";
    case BSMMA_DEV_BAD_MSIZES: return "BSMMA_DEV_BAD_MSIZES";
    default: return "BSMMA_UNKNOWN_STATUS";
  }
}

int64_t bsmma_launch_count(void) { return g_launches.load(); }

bsmma_status bsmma_probe_wait_timeout(int64_t limit_ns, bsmma_stream stream) {
  if (limit_ns <= 0 || limit_ns > 10000000000ll) return BSMMA_ERR_INVALID_ARG;
  bsmma_status st;
  const DeviceInfo* dev = current_device(&st);
  if (!dev) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  st = bsmma_device_status(stream);   // clear anything latched before
  if (st == BSMMA_ERR_CUDA) return st;
  wait_probe_kernel<<<1, 32, 0, s>>>(dev->status, static_cast<uint64_t>(limit_ns));
  count_launches(1);
  if (cudaGetLastError() != cudaSuccess) return BSMMA_ERR_CUDA;
  return bsmma_device_status(stream);
}

}  // extern "C"
