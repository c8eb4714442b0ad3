// Columns to 8 bits and back, the residual norm with 8-bit output and its
// gradient (x<quant>, x<dequant>, x<rmsquant>, x<rmsgrad> of xsymv.h).
// One thread block per column; all four are bound by the bytes of their
// operands.  Multiply-adds are written out as fmaf, so that a call with an
// optional operand left out rounds as the same call with that operand given.
#include "xsymv_q8.cuh"

namespace xsymv {
namespace {

constexpr int kThreads = 256;

template <class T>
__global__ void quant_kernel(int m, const T* X, long long ldx, int8_t* Q, long long ldq,
                             float* scale) {
  __shared__ float buf[32];
  const long long j = blockIdx.x;
  X += j * ldx;
  Q += j * ldq;
  uint32_t top = 0;
  for (int i = threadIdx.x; i < m; i += kThreads) top = max(top, magnitude_bits(to_float(X[i])));
  const Rounding r = rounding_of(block_max<kThreads>(top, buf));
  if (threadIdx.x == 0) scale[j] = r.scale;
  for (int i = threadIdx.x; i < m; i += kThreads) Q[i] = (int8_t)round_q8(to_float(X[i]), r);
}

template <class T>
__global__ void dequant_kernel(int m, const int8_t* Q, long long ldq, const float* scale, T* X,
                               long long ldx) {
  const long long j = blockIdx.x;
  const float s = scale[j];
  for (int i = threadIdx.x; i < m; i += kThreads)
    X[j * ldx + i] = from_float<T>((float)Q[j * ldq + i] * s);
}

template <class T>
struct RmsquantArgs {
  int m;
  const T* X;
  long long ldx;
  const T* R;
  long long ldr;
  const T* G;
  float eps;
  T* H;
  long long ldh;
  int8_t* Q;
  long long ldq;
  float* scale;
  float* rstd;
};

template <class T>
__global__ void rmsquant_kernel(RmsquantArgs<T> a) {
  __shared__ float buf[32];
  const long long j = blockIdx.x;
  // h in float, as stored: H may be X or R, so it is formed once per element
  // and pass from what that pass may read
  const T* src = a.H != nullptr ? a.H + j * a.ldh : a.X + j * a.ldx;
  const T* add = a.H == nullptr && a.R != nullptr ? a.R + j * a.ldr : nullptr;
  auto h_of = [&](int i) {
    float v = to_float(src[i]);
    if (add != nullptr) v = to_float(from_float<T>(v + to_float(add[i])));
    return v;
  };
  auto g_of = [&](int i) { return a.G != nullptr ? to_float(a.G[i]) : 1.f; };
  float sum = 0.f;
  uint32_t top = 0;
  for (int i = threadIdx.x; i < a.m; i += kThreads) {
    float v = to_float(a.X[j * a.ldx + i]);
    if (a.R != nullptr) v += to_float(a.R[j * a.ldr + i]);
    const T h = from_float<T>(v);
    if (a.H != nullptr) a.H[j * a.ldh + i] = h;
    v = to_float(h);
    sum += v * v;
    top = max(top, magnitude_bits(v));
  }
  sum = block_sum<kThreads>(sum, buf);
  top = block_max<kThreads>(top, buf);
  float rstd = 1.f / sqrtf(sum / (float)a.m + a.eps);
  if (top > 0 && top < kInfBits && !(sum > 0x1p-80f && sum < 0x1p127f)) {
    // squares out of float's range: scaled by the largest magnitude's power of two
    const int e = ilogbf(__uint_as_float(top));
    float t = 0.f;
    for (int i = threadIdx.x; i < a.m; i += kThreads) {
      const float v = scalbnf(h_of(i), -e);
      t += v * v;
    }
    t = block_sum<kThreads>(t, buf);
    rstd = (float)(1.0 / sqrt(scalbn((double)t / a.m, 2 * e) + (double)a.eps));
  }
  top = 0;
  for (int i = threadIdx.x; i < a.m; i += kThreads)
    top = max(top, magnitude_bits(h_of(i) * rstd * g_of(i)));
  const Rounding r = rounding_of(block_max<kThreads>(top, buf));
  if (threadIdx.x == 0) {
    a.scale[j] = r.scale;
    if (a.rstd != nullptr) a.rstd[j] = rstd;
  }
  for (int i = threadIdx.x; i < a.m; i += kThreads)
    a.Q[j * a.ldq + i] = (int8_t)round_q8(h_of(i) * rstd * g_of(i), r);
}

template <class T>
struct RmsgradArgs {
  int m, n;
  const T* dY;
  long long lddy;
  const T* H;
  long long ldh;
  const T* G;
  const float* rstd;
  const T* dR;
  long long lddr;
  T* dX;
  long long lddx;
  float* dG;
};

// dG before dX, which may overwrite dY or H: one thread per row i
template <class T>
__global__ void rmsgrad_weight_kernel(RmsgradArgs<T> a) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.m) return;
  float s = 0.f;
  for (long long j = 0; j < a.n; ++j)
    s = fmaf(to_float(a.dY[j * a.lddy + i]), to_float(a.H[j * a.ldh + i]) * a.rstd[j], s);
  a.dG[i] = s;
}

template <class T>
__global__ void rmsgrad_kernel(RmsgradArgs<T> a) {
  __shared__ float buf[32];
  const long long j = blockIdx.x;
  const float rstd = a.rstd[j];
  const T* dy = a.dY + j * a.lddy;
  const T* h = a.H + j * a.ldh;
  float s = 0.f;
  for (int i = threadIdx.x; i < a.m; i += kThreads) {
    const float g = a.G != nullptr ? to_float(a.G[i]) : 1.f;
    s = fmaf(to_float(dy[i]) * g, to_float(h[i]) * rstd, s);
  }
  const float c = block_sum<kThreads>(s, buf) / (float)a.m;
  for (int i = threadIdx.x; i < a.m; i += kThreads) {
    const float g = a.G != nullptr ? to_float(a.G[i]) : 1.f;
    const float d = a.dR != nullptr ? to_float(a.dR[j * a.lddr + i]) : 0.f;
    a.dX[j * a.lddx + i] = from_float<T>(
        fmaf(rstd, fmaf(-(to_float(h[i]) * rstd), c, to_float(dy[i]) * g), d));
  }
}

inline bool short_ld(int ld, int rows) { return ld < (rows > 1 ? rows : 1); }

bool device_ok() {
  int dev, sms;
  return current_device(&dev, &sms);
}

template <class T>
int quant_entry(int m, int n, const T* X, int ldx, int8_t* Q, int ldq, float* scale) {
  if (m < 0) return 1;
  if (n < 0) return 2;
  if (short_ld(ldx, m)) return 4;
  if (short_ld(ldq, m)) return 6;
  if (m == 0 || n == 0) return XSYMV_OK;
  if (X == nullptr || Q == nullptr || scale == nullptr) return XSYMV_ERR_VALUE;
  if (!device_ok()) return XSYMV_ERR_DEVICE;
  quant_kernel<T><<<n, kThreads, 0, current_stream()>>>(m, X, ldx, Q, ldq, scale);
  return launched(cudaGetLastError(), 1);
}

template <class T>
int dequant_entry(int m, int n, const int8_t* Q, int ldq, const float* scale, T* X, int ldx) {
  if (m < 0) return 1;
  if (n < 0) return 2;
  if (short_ld(ldq, m)) return 4;
  if (short_ld(ldx, m)) return 7;
  if (m == 0 || n == 0) return XSYMV_OK;
  if (X == nullptr || Q == nullptr || scale == nullptr) return XSYMV_ERR_VALUE;
  if (!device_ok()) return XSYMV_ERR_DEVICE;
  dequant_kernel<T><<<n, kThreads, 0, current_stream()>>>(m, Q, ldq, scale, X, ldx);
  return launched(cudaGetLastError(), 1);
}

template <class T>
int rmsquant_entry(int m, int n, const T* X, int ldx, const T* R, int ldr, const T* G, float eps,
                   T* H, int ldh, int8_t* Q, int ldq, float* scale, float* rstd) {
  if (m < 0) return 1;
  if (n < 0) return 2;
  if (short_ld(ldx, m)) return 4;
  if (R != nullptr && short_ld(ldr, m)) return 6;
  if (!(eps >= 0.f)) return 8;
  if (H != nullptr && short_ld(ldh, m)) return 10;
  if (short_ld(ldq, m)) return 12;
  if (m == 0 || n == 0) return XSYMV_OK;
  if (X == nullptr || Q == nullptr || scale == nullptr) return XSYMV_ERR_VALUE;
  if (!device_ok()) return XSYMV_ERR_DEVICE;
  const RmsquantArgs<T> a{m, X, ldx, R, ldr, G, eps, H, ldh, Q, ldq, scale, rstd};
  rmsquant_kernel<T><<<n, kThreads, 0, current_stream()>>>(a);
  return launched(cudaGetLastError(), 1);
}

template <class T>
int rmsgrad_entry(int m, int n, const T* dY, int lddy, const T* H, int ldh, const T* G,
                  const float* rstd, const T* dR, int lddr, T* dX, int lddx, float* dG) {
  if (m < 0) return 1;
  if (n < 0) return 2;
  if (short_ld(lddy, m)) return 4;
  if (short_ld(ldh, m)) return 6;
  if (dR != nullptr && short_ld(lddr, m)) return 10;
  if (short_ld(lddx, m)) return 12;
  if (m == 0 || (n == 0 && dG == nullptr)) return XSYMV_OK;
  if (n > 0 && (dY == nullptr || H == nullptr || rstd == nullptr || dX == nullptr))
    return XSYMV_ERR_VALUE;
  if (!device_ok()) return XSYMV_ERR_DEVICE;
  cudaStream_t st = current_stream();
  const RmsgradArgs<T> a{m, n, dY, lddy, H, ldh, G, rstd, dR, lddr, dX, lddx, dG};
  if (dG != nullptr) {
    rmsgrad_weight_kernel<T><<<(m + kThreads - 1) / kThreads, kThreads, 0, st>>>(a);
    const int s = launched(cudaGetLastError(), 1);
    if (s != XSYMV_OK) return s;
  }
  if (n == 0) return XSYMV_OK;
  rmsgrad_kernel<T><<<n, kThreads, 0, st>>>(a);
  return launched(cudaGetLastError(), 1);
}

template <class T, class C>
const T* in(const C* p) { return reinterpret_cast<const T*>(p); }
template <class T, class C>
T* out(C* p) { return reinterpret_cast<T*>(p); }

}  // namespace
}  // namespace xsymv

using xsymv::in;
using xsymv::out;

#define XSYMV_Q8_ROWS(K, C, T)                                                                   \
  extern "C" XSYMV_API int xquant_##K(int m, int n, const C* X, int ldx, signed char* Q,         \
                                      int ldq, float* scale) {                                   \
    return xsymv::quant_entry<T>(m, n, in<T>(X), ldx, Q, ldq, scale);                            \
  }                                                                                              \
  extern "C" XSYMV_API int xdequant_##K(int m, int n, const signed char* Q, int ldq,             \
                                        const float* scale, C* X, int ldx) {                     \
    return xsymv::dequant_entry<T>(m, n, Q, ldq, scale, out<T>(X), ldx);                         \
  }                                                                                              \
  extern "C" XSYMV_API int xrmsquant_##K(int m, int n, const C* X, int ldx, const C* R, int ldr, \
                                         const C* G, float eps, C* H, int ldh, signed char* Q,   \
                                         int ldq, float* scale, float* rstd) {                   \
    return xsymv::rmsquant_entry<T>(m, n, in<T>(X), ldx, in<T>(R), ldr, in<T>(G), eps,           \
                                    out<T>(H), ldh, Q, ldq, scale, rstd);                        \
  }                                                                                              \
  extern "C" XSYMV_API int xrmsgrad_##K(int m, int n, const C* dY, int lddy, const C* H,         \
                                        int ldh, const C* G, const float* rstd, const C* dR,     \
                                        int lddr, C* dX, int lddx, float* dG) {                  \
    return xsymv::rmsgrad_entry<T>(m, n, in<T>(dY), lddy, in<T>(H), ldh, in<T>(G), rstd,         \
                                   in<T>(dR), lddr, out<T>(dX), lddx, dG);                       \
  }

XSYMV_Q8_ROWS(s, float, float)
XSYMV_Q8_ROWS(h, xsymv_f16, __half)
XSYMV_Q8_ROWS(b, xsymv_bf16, __nv_bfloat16)
