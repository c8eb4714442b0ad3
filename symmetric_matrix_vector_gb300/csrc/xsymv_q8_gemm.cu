// Entry points xgemmq_s / _h / _b: Y := alpha*diag(sw)*W^T*X*diag(sx) + beta*Y
// with W and X of 8-bit integers.
#include "xsymv_q8.cuh"

namespace xsymv {
namespace {

template <class T>
struct GemmqArgs {
  int m, n, k;
  float alpha;
  const int8_t* W;
  long long ldw;
  const float* sw;
  const int8_t* X;
  long long ldx;
  const float* sx;
  float beta;
  T* Y;
  long long ldy;
};

// acc * alpha * sw * sx + beta * y, rounded once
template <class T>
__device__ __forceinline__ void store_output(const GemmqArgs<T>& a, long long i, long long j,
                                             float acc) {
  float v = 0.f;
  if (a.alpha != 0.f && a.k > 0) {
    v = acc * (a.sw != nullptr ? a.sw[i] : 1.f);
    v = v * (a.sx != nullptr ? a.sx[j] : 1.f) * a.alpha;
  }
  T* y = a.Y + j * a.ldy + i;
  if (a.beta != 0.f) v = fmaf(a.beta, to_float(*y), v);
  *y = from_float<T>(v);
}

// One output per thread, a 32 x 8 tile of (channel, token) per block; sums in
// 64-bit integers.
template <class T>
__global__ void gemmq_kernel(GemmqArgs<T> a) {
  await_predecessor();
  const long long i = blockIdx.x * 32LL + threadIdx.x;
  for (long long j = blockIdx.y * 8LL + threadIdx.y; j < a.n; j += gridDim.y * 8LL) {
    if (i >= a.m) return;
    long long acc = 0;
    if (a.alpha != 0.f)
      for (int p = 0; p < a.k; ++p) acc += (int)a.W[i * a.ldw + p] * (int)a.X[j * a.ldx + p];
    store_output(a, i, j, (float)acc);
  }
}

template <class T>
int gemmq_entry(int m, int n, int k, float alpha, const int8_t* W, int ldw, const float* sw,
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
  const GemmqArgs<T> a{m, n, k, alpha, W, ldw, sw, X, ldx, sx, beta, Y, ldy};
  const dim3 grid((m + 31) / 32, (unsigned)min((n + 7LL) / 8, 65535LL));
  cudaStream_t st = current_stream();
  return launched(launch_after(gemmq_kernel<T>, grid, dim3(32, 8), 0, st, a), 1, st);
}

}  // namespace
}  // namespace xsymv

#define XSYMV_Q8_GEMM(K, C, T)                                                                  \
  extern "C" XSYMV_API int xgemmq_##K(int m, int n, int k, float alpha, const signed char* W,   \
                                      int ldw, const float* sw, const signed char* X, int ldx,  \
                                      const float* sx, float beta, C* Y, int ldy) {             \
    return xsymv::gemmq_entry<T>(m, n, k, alpha, W, ldw, sw, X, ldx, sx, beta,                  \
                                 reinterpret_cast<T*>(Y), ldy);                                 \
  }

XSYMV_Q8_GEMM(s, float, float)
XSYMV_Q8_GEMM(h, xsymv_f16, __half)
XSYMV_Q8_GEMM(b, xsymv_bf16, __nv_bfloat16)
