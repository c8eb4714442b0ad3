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


constexpr int kFewTokens = 8;
constexpr int kStreamTokens = 1024;
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

// `rows` rows of `width` elements, `pitch` bytes apart, in boxes of 128 bytes by
// box_rows rows under the 128-byte swizzle, zeros outside; base and pitch multiples of
// 16 bytes
bool map_rows(CUtensorMap* map, CUtensorMapDataType type, int bytes, const void* base,
              long long width, long long rows, long long pitch, int box_rows) {
  const EncodeTiled encode = encoder();
  if (encode == nullptr) return false;
  const cuuint64_t size[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t pitches[1] = {(cuuint64_t)pitch};
  const cuuint32_t box[2] = {128u / (cuuint32_t)bytes, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(base), size, pitches, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool map_halves(CUtensorMap* map, const __half* base, long long width, long long rows,
                int box_rows) {
  return map_rows(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, base, width, rows, width * 2, box_rows);
}

// blocks of 256 threads, a power of two of them along a row of `width` packs
dim3 pack_block(long long width) {
  unsigned along = 8;
  while (along < 256 && along < width) along *= 2;
  return dim3(along, 256 / along);
}
dim3 pack_grid(long long rows, long long width, dim3 block) {
  return dim3((unsigned)((rows + block.y - 1) / block.y),
              (unsigned)std::min<long long>((width + block.x - 1) / block.x, 65535));
}

cudaError_t launch_halves(int rows, int k, int kp, const int8_t* q, long long ldq, __half* out,
                          cudaStream_t st) {
  const bool g = k % kPack == 0 && reinterpret_cast<uintptr_t>(q) % 8 == 0 && ldq % 8 == 0;
  const dim3 block = pack_block(kp / kPack);
  return launch_after(g ? halves_kernel<true> : halves_kernel<false>,
                      pack_grid(rows, kp / kPack, block), block, 0, st, rows, k, kp, q, ldq, out);
}

// a workspace cut into pieces on 256-byte boundaries
struct Pieces {
  size_t bytes = 0;
  size_t add(size_t size) {
    const size_t at = bytes;
    bytes += (size + 255) / 256 * 256;
    return at;
  }
};

// The shared end of the two tensor-core forms: launch with clusters of `cluster`
// CTAs, record the status word that the kernel's bounded waits write
template <class... P, class... A>
cudaError_t launch_cluster(void (*kernel)(P...), unsigned grid, int cluster, int threads, int smem,
                           cudaStream_t st, A... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int* status_word(cudaStream_t st, int* status, int* epoch) {
  return static_cast<int*>(workspace(256, st, status, 0, epoch));
}

cudaError_t launch_align(int rows, int k, const int8_t* q, long long ldq, int8_t* out,
                         long long ldo, cudaStream_t st) {
  const dim3 block = pack_block(ldo / kPack);
  return launch_after(align_kernel, pack_grid(rows, ldo / kPack, block), block, 0, st, rows, k, q,
                      ldq, out, ldo);
}

template <int CTAS, int BN>
int gemmq_streamed(const GemmqAny& a, int sms, cudaStream_t st) {
  using S = Stream<CTAS, BN>;
  const int steps = (int)((a.k + (long long)kStepDepth - 1) / kStepDepth);
  const long long kp = (long long)steps * kStepDepth, ldo = (a.k + 15LL) / 16 * 16;
  // tensor copies need 16-byte boundaries: what is not on them is copied first
  auto on_grid = [](const int8_t* p, long long ld) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 16 == 0;
  };
  const bool move_w = !on_grid(a.W, a.ldw), move_x = S::kRaw && !on_grid(a.X, a.ldx);
  Pieces pieces;
  const size_t at_w = move_w ? pieces.add((size_t)a.m * ldo) : 0;
  const size_t at_x = S::kRaw ? (move_x ? pieces.add((size_t)a.n * ldo) : 0)
                              : pieces.add((size_t)a.n * kp * 2);
  int status = XSYMV_OK, epoch = 0, kernels = 1;
  int* const word = status_word(st, &status, &epoch);
  if (word == nullptr) return status;
  char* ws = nullptr;
  if (pieces.bytes > 0) {
    ws = static_cast<char*>(workspace(pieces.bytes, st, &status, kSlotOperands, nullptr));
    if (ws == nullptr) return status;
  }
  const int8_t* w = a.W;
  const int8_t* x = a.X;
  long long ldw = a.ldw, ldx = a.ldx;
  cudaError_t e = cudaSuccess;
  if (move_w) {
    int8_t* to = reinterpret_cast<int8_t*>(ws + at_w);
    e = launch_align(a.m, a.k, a.W, a.ldw, to, ldo, st);
    w = to, ldw = ldo, ++kernels;
  }
  if (e == cudaSuccess && move_x) {
    int8_t* to = reinterpret_cast<int8_t*>(ws + at_x);
    e = launch_align(a.n, a.k, a.X, a.ldx, to, ldo, st);
    x = to, ldx = ldo, ++kernels;
  }
  CUtensorMap map_w, map_x;
  bool mapped = map_rows(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, a.k, a.m, ldw, 128);
  if (S::kRaw) {
    mapped = mapped && map_rows(&map_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x, a.k, a.n, ldx, BN);
  } else {
    __half* to = reinterpret_cast<__half*>(ws + at_x);
    if (e == cudaSuccess) e = launch_halves(a.n, a.k, (int)kp, a.X, a.ldx, to, st);
    mapped = mapped && map_halves(&map_x, to, kp, a.n, BN / CTAS);
    ++kernels;
  }
  if (!mapped) return XSYMV_ERR_CUDA;
  if (e == cudaSuccess) {
    const long long tiles_m = (a.m + S::kChannels - 1LL) / S::kChannels;
    const long long tiles_n = (a.n + BN - 1LL) / BN;
    int split = 1;
    while (CTAS == 1 && split < 8 && split * 2 <= steps &&
           tiles_m * tiles_n * split * 2 <= (S::kRaw ? 2LL : 1LL) * sms)
      split *= 2;
    const int cluster = CTAS == 2 ? 2 : split;
    e = launch_cluster(gemmq_stream<CTAS, BN>, (unsigned)(tiles_m * tiles_n * cluster), cluster,
                       S::kThreads, S::kSmem, st, map_w, map_x, a, (int)tiles_n, steps, split, word,
                       epoch, wait_limit_ns(), test_extra_tx());
  }
  const int r = launched(e, kernels, st);
  if (r == XSYMV_OK) note_call_status(st, word, epoch);
  return r;
}

template <class T, int CTAS, int BN>
int gemmq_tiled(const GemmqArgs<T>& a, int sms, cudaStream_t st) {
  using S = Tile<CTAS, BN>;
  const int steps = (int)((a.k + (long long)kDepth - 1) / kDepth), kp = steps * kDepth;
  int status = XSYMV_OK, epoch = 0;
  int* const word = status_word(st, &status, &epoch);
  if (word == nullptr) return status;
  Pieces pieces;
  const size_t at_w = pieces.add((size_t)a.m * kp * 2), at_x = pieces.add((size_t)a.n * kp * 2);
  char* ws = static_cast<char*>(workspace(pieces.bytes, st, &status, kSlotOperands, nullptr));
  if (ws == nullptr) return status;
  __half* const w = reinterpret_cast<__half*>(ws + at_w);
  __half* const x = reinterpret_cast<__half*>(ws + at_x);
  CUtensorMap map_w, map_x;
  if (!map_halves(&map_w, w, kp, a.m, 128) || !map_halves(&map_x, x, kp, a.n, BN / CTAS))
    return XSYMV_ERR_CUDA;
  cudaError_t e = launch_halves(a.m, a.k, kp, a.W, a.ldw, w, st);
  if (e == cudaSuccess) e = launch_halves(a.n, a.k, kp, a.X, a.ldx, x, st);
  if (e == cudaSuccess) {
    TileOrder order;
    order.tiles_m = (a.m + S::kChannels - 1) / S::kChannels;
    order.tiles_n = (a.n + BN - 1) / BN;
    order.tiles = order.tiles_m * order.tiles_n;
    e = launch_cluster(gemmq_tiles<T, CTAS, BN>,
                       (unsigned)(CTAS * std::min(order.tiles, sms / CTAS)), CTAS, S::kThreads,
                       S::kSmem, st, map_w, map_x, a, order, steps, word, epoch, wait_limit_ns(),
                       test_extra_tx());
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
  GemmqAny any;
  static_cast<GemmqArgs<void>&>(any) =
      GemmqArgs<void>{m, n, k, alpha, W, ldw, sw, X, ldx, sx, beta, Y, ldy};
  any.type = type;
  if (n <= kFewTokens && k <= kDotMostDepth)
    return launched(launch_few(any, sms, st), 1, st);
  if (n <= 16) return gemmq_streamed<1, 16>(any, sms, st);
  if (n <= 32) return gemmq_streamed<1, 32>(any, sms, st);
  if (n <= 64) return gemmq_streamed<1, 64>(any, sms, st);
  if (n <= 128) return gemmq_streamed<1, 128>(any, sms, st);
  if (n <= kStreamTokens) return gemmq_streamed<2, 256>(any, sms, st);
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
