// Entry points xgemmq_s / _h / _b: Y := alpha*diag(sw)*W^T*X*diag(sx) + beta*Y
// with W and X of 8-bit integers.
#include <algorithm>

#include "xsymv_q8_gemm.cuh"

namespace xsymv {
namespace {

// Y := beta * Y
template <class T>
__global__ void __launch_bounds__(256) scale_kernel(GemmqArgs<T> a) {
  await_predecessor();
  for (long long j = blockIdx.y; j < a.n; j += gridDim.y)
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < a.m; i += gridDim.x * 256LL)
      store_output(a, i, j, 0.f, 0.f, 0.f);
}

// ------------------------------------------------------------ a few tokens --

template <int NT, int R>
cudaError_t launch_dot(const GemmqAny& a, bool g, int sms, cudaStream_t st) {
  // threads a row: 4 pieces of 16 integers a thread where that fills the SMs, else
  // fewer pieces, down to one
  int threads = 4;
  while (threads < kDotBlock &&
         (threads * 64 < a.k ||
          (threads * 16 < a.k && (long long)a.m * threads / R < (long long)sms * 1024)))
    threads *= 2;
  while (threads > 32 && (long long)a.m * threads / R > (long long)sms * 8192) threads /= 2;
  const long long rows = (long long)(kDotBlock / threads) * R;
  return launch_after(g ? gemmq_dot<NT, R, true> : gemmq_dot<NT, R, false>,
                      (unsigned)((a.m + rows - 1) / rows), kDotBlock, 0, st, a, threads);
}

cudaError_t launch_few(const GemmqAny& a, int sms, cudaStream_t st) {
  auto on_grid = [](const int8_t* p, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0;
  };
  const bool g = a.k % 16 == 0 && on_grid(a.W, a.ldw) && on_grid(a.X, a.ldx);
  if (a.n == 1) return launch_dot<1, 1>(a, g, sms, st);
  if (a.n == 2) return launch_dot<2, 2>(a, g, sms, st);
  if (a.n <= 4) return launch_dot<4, 2>(a, g, sms, st);
  auto* kernel = a.n <= 8    ? (g ? gemmq_mma<1, true> : gemmq_mma<1, false>)
                 : a.n <= 16 ? (g ? gemmq_mma<2, true> : gemmq_mma<2, false>)
                 : a.n <= 24 ? (g ? gemmq_mma<3, true> : gemmq_mma<3, false>)
                 : a.n <= 32 ? (g ? gemmq_mma<4, true> : gemmq_mma<4, false>)
                             : (g ? gemmq_mma<5, true> : gemmq_mma<5, false>);
  return launch_after(kernel, (unsigned)((a.m + kMmaRows - 1LL) / kMmaRows), kMmaWarps * 32, 0, st,
                      a);
}

// ------------------------------------------------------------ tensor cores --

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's tensor map encoder (the library does not link the driver)
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// rows of `width` halves in boxes of kDepth halves by `box_rows` rows, zeros
// outside; base 256-byte aligned, width a multiple of kDepth
bool map_halves(CUtensorMap* map, __half* base, long long width, long long rows, int box_rows) {
  const EncodeTiled encode = encoder();
  if (encode == nullptr) return false;
  const cuuint64_t size[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t pitch[1] = {(cuuint64_t)width * sizeof(__half)};
  const cuuint32_t box[2] = {(cuuint32_t)kDepth, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, size, pitch, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_halves(int rows, int k, int kp, const int8_t* q, long long ldq, __half* out,
                          cudaStream_t st) {
  const bool g = k % kPack == 0 && reinterpret_cast<uintptr_t>(q) % 8 == 0 && ldq % 8 == 0;
  int along = 8;
  while (along < 256 && along * kPack < kp) along *= 2;
  const long long by = 256 / along, step = (long long)along * kPack;
  const dim3 grid((unsigned)((rows + by - 1) / by),
                  (unsigned)std::min<long long>((kp + step - 1) / step, 65535));
  return launch_after(g ? halves_kernel<true> : halves_kernel<false>, grid,
                      dim3(along, (unsigned)by), 0, st, rows, k, kp, q, ldq, out);
}

template <class T, int CTAS, int BN>
int gemmq_tiled(const GemmqArgs<T>& a, int sms, cudaStream_t st) {
  using S = Tile<CTAS, BN>;
  const int steps = (int)((a.k + (long long)kDepth - 1) / kDepth), kp = steps * kDepth;
  int status = XSYMV_OK, epoch = 0;
  int* word = static_cast<int*>(workspace(256, st, &status, 0, &epoch));
  if (word == nullptr) return status;
  const size_t bytes_w = ((size_t)a.m * kp * 2 + 255) / 256 * 256, bytes_x = (size_t)a.n * kp * 2;
  char* ws = static_cast<char*>(workspace(bytes_w + bytes_x, st, &status, kSlotOperands, nullptr));
  if (ws == nullptr) return status;
  __half* const w = reinterpret_cast<__half*>(ws);
  __half* const x = reinterpret_cast<__half*>(ws + bytes_w);
  CUtensorMap map_w, map_x;
  if (!map_halves(&map_w, w, kp, a.m, 128) || !map_halves(&map_x, x, kp, a.n, BN / CTAS))
    return XSYMV_ERR_CUDA;
  cudaError_t e = launch_halves(a.m, a.k, kp, a.W, a.ldw, w, st);
  if (e == cudaSuccess) e = launch_halves(a.n, a.k, kp, a.X, a.ldx, x, st);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(gemmq_tiles<T, CTAS, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::kSmem);
  if (e == cudaSuccess) {
    TileOrder order;
    order.tiles_m = (a.m + S::kChannels - 1) / S::kChannels;
    order.tiles_n = (a.n + BN - 1) / BN;
    order.tiles = order.tiles_m * order.tiles_n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(CTAS * std::min(order.tiles, sms / CTAS)));
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CTAS;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, gemmq_tiles<T, CTAS, BN>, map_w, map_x, a, order, steps, word,
                           epoch, wait_limit_ns(), test_extra_tx());
  }
  const int r = launched(e, 3, st);
  if (r == XSYMV_OK) note_call_status(st, word, epoch);
  return r;
}

template <class T>
int gemmq_entry(char type, int m, int n, int k, float alpha, const int8_t* W, int ldw, const float* sw,
                const int8_t* X, int ldx, const float* sx, float beta, T* Y, int ldy) {
  if (m < 0) return 1;
  if (n < 0) return 2;
  if (k < 0) return 3;
  if (short_ld(ldw, k)) return 6;
  if (short_ld(ldx, k)) return 9;
  if (short_ld(ldy, m)) return 13;
  if (m == 0 || n == 0) return XSYMV_OK;
  const bool no_product = alpha == 0.f || k == 0;
  if (no_product && beta == 1.f) return XSYMV_OK;
  if (Y == nullptr || (!no_product && (W == nullptr || X == nullptr))) return XSYMV_ERR_VALUE;
  int dev, sms;
  if (!current_device(&dev, &sms)) return XSYMV_ERR_DEVICE;
  cudaStream_t st = current_stream();
  const GemmqArgs<T> a{m, n, k, alpha, W, ldw, sw, X, ldx, sx, beta, Y, ldy};
  if (no_product)
    return launched(launch_after(scale_kernel<T>, dim3((m + 255) / 256, std::min(n, 65535)), 256, 0,
                                 st, a),
                    1, st);
  if (n <= 40 && k <= kDotMostDepth) {
    GemmqAny any;
    static_cast<GemmqArgs<void>&>(any) =
        GemmqArgs<void>{m, n, k, alpha, W, ldw, sw, X, ldx, sx, beta, Y, ldy};
    any.type = type;
    return launched(launch_few(any, sms, st), 1, st);
  }
  if (n <= 64) return gemmq_tiled<T, 1, 64>(a, sms, st);
  if (n <= 128) return gemmq_tiled<T, 1, 128>(a, sms, st);
  return gemmq_tiled<T, 2, 256>(a, sms, st);
}

}  // namespace
}  // namespace xsymv

#define XSYMV_Q8_GEMM(K, C, T)                                                                  \
  extern "C" XSYMV_API int xgemmq_##K(int m, int n, int k, float alpha, const signed char* W,   \
                                      int ldw, const float* sw, const signed char* X, int ldx,  \
                                      const float* sx, float beta, C* Y, int ldy) {             \
    return xsymv::gemmq_entry<T>(#K[0], m, n, k, alpha, W, ldw, sw, X, ldx, sx, beta,                  \
                                 reinterpret_cast<T*>(Y), ldy);                                 \
  }

XSYMV_Q8_GEMM(s, float, float)
XSYMV_Q8_GEMM(h, xsymv_f16, __half)
XSYMV_Q8_GEMM(b, xsymv_bf16, __nv_bfloat16)
