// The product of 8-bit matrices on the tensor cores.
//
// GB300 has no fast integer path (mma.sync on 8-bit integers: 256 multiply-adds
// a clock and SM, as many as dp4a; on halves 1000; tcgen05 on halves 8192),
// so 8-bit integers are multiplied as halves: every value is exact in a half,
// every product exact in a float, and the float accumulators are exact while
// sums stay below 2^24.
#pragma once

#include <type_traits>

#include "xsymv_q8.cuh"
#include "xsymv_tensor.cuh"

namespace xsymv {

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

// sx[j] * alpha and sw[i]
template <class T>
__device__ __forceinline__ float token_factor(const GemmqArgs<T>& a, long long j) {
  return (a.sx != nullptr ? a.sx[j] : 1.f) * a.alpha;
}
template <class T>
__device__ __forceinline__ float channel_factor(const GemmqArgs<T>& a, long long i) {
  return a.sw != nullptr ? a.sw[i] : 1.f;
}
// Y(i, j) := (acc * sw) * (sx * alpha) + beta * Y(i, j), rounded once
template <class T>
__device__ __forceinline__ void store_output(const GemmqArgs<T>& a, long long i, long long j,
                                             float acc, float channel, float token) {
  float v = acc * channel * token;
  T* y = a.Y + j * a.ldy + i;
  if (a.beta != 0.f) v = fmaf(a.beta, to_float(*y), v);
  *y = from_float<T>(v);
}

// ... with the type of Y known at run time, for the kernels of a few tokens
struct GemmqAny : GemmqArgs<void> {
  char type;   // 's', 'h' or 'b'
};
__device__ __forceinline__ void store_any(const GemmqAny& a, long long i, long long j, float acc) {
  const float channel = a.sw != nullptr ? a.sw[i] : 1.f;
  const float token = (a.sx != nullptr ? a.sx[j] : 1.f) * a.alpha;
  auto put = [&](auto* y) {
    using T = std::remove_pointer_t<decltype(y)>;
    float v = acc * channel * token;
    if (a.beta != 0.f) v = fmaf(a.beta, to_float(*y), v);
    *y = from_float<T>(v);
  };
  const long long at = j * a.ldy + i;
  if (a.type == 's')
    put(static_cast<float*>(a.Y) + at);
  else if (a.type == 'h')
    put(static_cast<__half*>(a.Y) + at);
  else
    put(static_cast<__nv_bfloat16*>(a.Y) + at);
}

// four 8-bit integers as halves: xor 128 makes them 0 .. 255, which set into the
// low bits of 1024 (0x6400) read 1024 + v + 128
__device__ __forceinline__ void halves_of(uint32_t q, uint32_t& lo, uint32_t& hi) {
  q ^= 0x80808080u;
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
  uint32_t a = __byte_perm(q, 0x64646464u, 0x4140), b = __byte_perm(q, 0x64646464u, 0x4342);
  __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias);
  __half2 hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
  lo = *reinterpret_cast<uint32_t*>(&ha);
  hi = *reinterpret_cast<uint32_t*>(&hb);
}

// ---------------------------------------------------------- a few tokens --

// 16 integers first .. first+15 of the k of `row` (first a multiple of 16), at any
// alignment.  GRID: rows start on 16-byte boundaries and are multiples of 16
// long.  MASK: those beyond k are zero; else they are any integers (their
// partners are zero).  Only 16-byte pieces that hold an element of the row are
// read.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
template <bool GRID, bool MASK>
__device__ __forceinline__ uint4 load16(const int8_t* row, int first, int k) {
  uint4 z = make_uint4(0, 0, 0, 0);
  if (first >= k) return z;
  const int8_t* at = row + first;
  // X is read by many warps, W once
  auto piece = [](const void* p) {
    return MASK ? __ldg(reinterpret_cast<const uint4*>(p)) : load_once(p);
  };
  if (GRID) return piece(at);
  const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(at) % 16);
  const uint4 a = piece(at - off);
  if (off == 0) {
    z = a;
  } else {
    uint4 b = z;
    if (at - off + 16 < row + k) b = piece(at - off + 16);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    shift_words<4>(w, off);
    const unsigned bits = (off & 3) * 8;
    z = make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                   __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
  }
  if (MASK && first + 16 > k) {
    const int left = k - first;   // 1 .. 15
    auto keep = [&](uint32_t v, int at) {
      return left >= at + 4 ? v : left <= at ? 0u : v & ((1u << 8 * (left - at)) - 1u);
    };
    z = make_uint4(keep(z.x, 0), keep(z.y, 4), keep(z.z, 8), keep(z.w, 12));
  }
  return z;
}

// Up to 4 tokens: dot products of 8-bit integers (dp4a, 32-bit sums), bound
// by the bytes of W.  A row of W (a channel) is `threads` threads' work, a power of
// two from 4 to a whole block, R rows at a time; X comes from L1.
constexpr int kDotBlock = 256;
constexpr int kDotMostDepth = 1 << 22;   // a thread's sums stay below 2^31
template <int NT, int R, bool GRID>
__global__ void __launch_bounds__(kDotBlock) gemmq_dot(GemmqAny a, int threads) {
  __shared__ float buf[kDotBlock / 32][R * NT];
  await_predecessor();
  const int part = (int)threadIdx.x & (threads - 1);
  const long long i0 = ((long long)blockIdx.x * (kDotBlock / threads) + threadIdx.x / threads) * R;
  int acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t] = 0;
  const int8_t *w[R], *x[NT];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = a.W + min(i0 + r, a.m - 1LL) * a.ldw;
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = a.X + min(t, a.n - 1) * a.ldx;
  constexpr int U = 4 / R;   // 64 bytes of W on their way
  for (int p = part * 16; p < a.k; p += threads * 16 * U) {
    uint4 q[U][R];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r) q[u][r] = load16<GRID, false>(w[r], p + u * threads * 16, a.k);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint4 v = load16<GRID, true>(x[t], p + u * threads * 16, a.k);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          acc[r][t] = __dp4a((int)q[u][r].x, (int)v.x, acc[r][t]);
          acc[r][t] = __dp4a((int)q[u][r].y, (int)v.y, acc[r][t]);
          acc[r][t] = __dp4a((int)q[u][r].z, (int)v.z, acc[r][t]);
          acc[r][t] = __dp4a((int)q[u][r].w, (int)v.w, acc[r][t]);
        }
      }
  }
  // sums below 2^31 are added as integers, larger ones (k >= 2^17) as floats
  const bool whole = a.k < 1 << 17;
  float sum[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (whole) {
        int v = acc[r][t];
        for (int o = min(threads, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        sum[r][t] = __int_as_float(v);
      } else {
        float v = (float)acc[r][t];
        for (int o = min(threads, 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        sum[r][t] = v;
      }
    }
  if (threads > 32) {
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) buf[threadIdx.x / 32][r * NT + t] = sum[r][t];
    __syncthreads();
  }
  if (part != 0) return;
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (i0 + r >= a.m || t >= a.n) continue;
      float v;
      if (whole) {
        int s = __float_as_int(sum[r][t]);
        for (int w = 1; w < threads / 32; ++w)
          s += __float_as_int(buf[threadIdx.x / 32 + w][r * NT + t]);
        v = (float)s;
      } else {
        v = sum[r][t];
        for (int w = 1; w < threads / 32; ++w) v += buf[threadIdx.x / 32 + w][r * NT + t];
      }
      store_any(a, i0 + r, t, v);
    }
}

// 5 to 40 tokens: W and X become halves in registers, products on the
// warp-level tensor path (mma.sync, m16n8k16), whose 1000 multiply-adds a clock and SM
// keep up with the bytes of W up to about 40 tokens; above, tiles win.  A lane holds
// 16 consecutive integers of the rows g and g + 8 of a 16-row tile (g =
// lane / 4) and of token g: the depth is taken in whatever order makes them
// fragments, the same for W and X.  A warp has 2 row tiles and every 8th
// part of the depth; the block's 8 warps add their sums in shared memory, in
// warp order.
constexpr int kMmaWarps = 8, kMmaRows = 32;
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int NT8, bool GRID>
__global__ void __launch_bounds__(kMmaWarps * 32) gemmq_mma(GemmqAny a) {
  __shared__ float buf[kMmaWarps][kMmaRows][NT8 * 8 + 2];
  await_predecessor();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const long long i0 = (long long)blockIdx.x * kMmaRows;
  const int8_t *w[4], *x[NT8];
#pragma unroll
  for (int r = 0; r < 4; ++r) w[r] = a.W + min(i0 + g + 8 * r, a.m - 1LL) * a.ldw;
#pragma unroll
  for (int c = 0; c < NT8; ++c) x[c] = a.X + min(g + 8 * c, a.n - 1) * a.ldx;
  float acc[2][NT8][4];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < NT8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[h][c][e] = 0.f;
  uint4 next[4];
  const int step = kMmaWarps * 64;
  int p = warp * 64 + t * 16;
#pragma unroll
  for (int r = 0; r < 4; ++r) next[r] = load16<GRID, false>(w[r], p, a.k);
  for (; p - t * 16 < a.k; p += step) {
    uint4 q[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      q[r] = next[r];
      next[r] = load16<GRID, false>(w[r], p + step, a.k);
    }
    uint4 v[NT8];
#pragma unroll
    for (int c = 0; c < NT8; ++c) v[c] = load16<GRID, true>(x[c], p, a.k);
#pragma unroll
    for (int s = 0; s < 4; ++s) {   // 4 of the lane's 16 integers
      auto word = [s](const uint4& u) { return s == 0 ? u.x : s == 1 ? u.y : s == 2 ? u.z : u.w; };
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) halves_of(word(q[r]), lo[r], hi[r]);
#pragma unroll
      for (int c = 0; c < NT8; ++c) {
        uint32_t b0, b1;
        halves_of(word(v[c]), b0, b1);
        mma_16x8x16(acc[0][c], lo[0], lo[1], hi[0], hi[1], b0, b1);
        mma_16x8x16(acc[1][c], lo[2], lo[3], hi[2], hi[3], b0, b1);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int c = 0; c < NT8; ++c) {
      float* b = &buf[warp][h * 16 + g][c * 8 + 2 * t];
      b[0] = acc[h][c][0];
      b[1] = acc[h][c][1];
      b += 8 * (NT8 * 8 + 2);
      b[0] = acc[h][c][2];
      b[1] = acc[h][c][3];
    }
  __syncthreads();
  // lanes along the channels
  for (int c = warp; c < a.n; c += kMmaWarps) {
    float v = 0.f;
#pragma unroll
    for (int s = 0; s < kMmaWarps; ++s) v += buf[s][lane][c];
    if (i0 + lane < a.m) store_any(a, i0 + lane, c, v);
  }
}

// ------------------------------------------------------ operands as halves --

// Rows of kp halves (a multiple of kDepth, zeros beyond k) from rows of k
// integers at any alignment: what the tensor copies read.
constexpr int kDepth = 64;   // 128 bytes of halves
template <bool GRID>
__global__ void __launch_bounds__(256) halves_kernel(int rows, int k, int kp, const int8_t* q,
                                                     long long ldq, __half* out) {
  await_predecessor();
  const long long j = blockIdx.x * (long long)blockDim.y + threadIdx.y;
  if (j >= rows) return;
  q += j * ldq;
  out += j * kp;
  for (int first = (int)(blockIdx.y * blockDim.x + threadIdx.x) * kPack; first < kp;
       first += (int)(gridDim.y * blockDim.x) * kPack) {
    const Raw<int8_t> r = load8<GRID>(q, first, k);
    uint4 h;
    halves_of(r.w[0], h.x, h.y);
    halves_of(r.w[1], h.z, h.w);
    *reinterpret_cast<uint4*>(out + first) = h;
  }
}

// ... and rows of 8-bit integers on 16-byte boundaries, ldo a multiple of 16
__global__ void __launch_bounds__(256) align_kernel(int rows, int k, const int8_t* q, long long ldq,
                                                    int8_t* out, long long ldo) {
  await_predecessor();
  const long long j = blockIdx.x * (long long)blockDim.y + threadIdx.y;
  if (j >= rows) return;
  q += j * ldq;
  out += j * ldo;
  for (int first = (int)(blockIdx.y * blockDim.x + threadIdx.x) * kPack; first < ldo;
       first += (int)(gridDim.y * blockDim.x) * kPack) {
    const Raw<int8_t> r = load8<false>(q, first, k);
    *reinterpret_cast<uint2*>(out + first) = make_uint2(r.w[0], r.w[1]);
  }
}

// ------------------------------------------------------- the tiled product --

// A tile is 128 channels by BN tokens, or 256 by BN shared by a pair of CTAs
// (each holds its 128 channels' and half of the tokens' operands, and the
// accumulators of its channels).  Channels are the rows of the accumulator:
// a lane holds one channel and stores of 32 lanes side by side need no
// alignment.  Warp 0 copies, warp 1 multiplies (the pair's first CTA alone),
// warps 2 to 5 store a tile from one set of accumulators while the next is
// formed in the other.
template <int CTAS, int BN>
struct Tile {
  static constexpr int kChannels = 128 * CTAS, kTokens = BN;
  static constexpr int kBytesW = 128 * kDepth * 2, kBytesX = BN / CTAS * kDepth * 2;
  static constexpr int kStageBytes = kBytesW + kBytesX;
  static constexpr int kStages = 196608 / kStageBytes;
  static constexpr int kColumns = 2 * BN;   // of tensor memory
  static constexpr int kThreads = 192;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
};

struct TileOrder {
  int tiles_m, tiles_n, tiles;
  // Tiles that run at the same time are near one another in both directions:
  // bands of 8 tiles of tokens, channels advancing within a band
  __device__ __forceinline__ void at(int t, int& tm, int& tn) const {
    const int band = 8 * tiles_m, b = t / band, in = t - b * band;
    const int width = min(8, tiles_n - 8 * b);
    tm = in / width;
    tn = 8 * b + in - tm * width;
  }
};

template <class T, int CTAS, int BN>
__global__ void __launch_bounds__(192, 1)
    gemmq_tiles(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                GemmqArgs<T> a, TileOrder order, int steps, int* status, int epoch,
                unsigned long long limit_ns, uint32_t extra_tx) {
  using S = Tile<CTAS, BN>;
  extern __shared__ uint8_t raw_smem[];
  __shared__ alignas(8) uint64_t bar_words[2 * S::kStages + 4];
  __shared__ uint32_t tmem_word;
  __shared__ int dead_word;
  __shared__ float token_scale[2][BN];
  volatile int* const dead = &dead_word;
  const uint32_t tiles_smem = (smem_addr(raw_smem) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bar_words), empty = full + 8 * S::kStages;
  const uint32_t acc_full = empty + 8 * S::kStages, acc_empty = acc_full + 16;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = CTAS == 2 ? cluster_rank() : 0;
  const int first_tile = blockIdx.x / CTAS, stride = gridDim.x / CTAS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, 4 * CTAS);
    }
    dead_word = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<CTAS>(smem_addr(&tmem_word), S::kColumns);
  tensor_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();
  tensor_fence_after();
  const uint32_t tmem = tmem_word;
  await_predecessor();

  if (warp == 0 && lane == 0) {
    // ---- copies: this CTA's channels and its share of the tokens
    const uint32_t lead_full = CTAS == 2 ? cluster_address(full, 0) : full;
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < order.tiles; t += stride) {
      int tm, tn;
      order.at(t, tm, tn);
      const int row_w = tm * S::kChannels + (int)rank * 128;
      const int row_x = tn * BN + (int)rank * (BN / CTAS);
      for (int s = 0; s < steps; ++s) {
        if (!wait_or_dead(empty + 8 * stage, phase ^ 1, dead, limit_ns)) {
          ok = false;
          break;
        }
        if (rank == 0)
          mbar_arrive_expect_tx(full + 8 * stage, CTAS * S::kStageBytes + extra_tx);
        const uint32_t at = tiles_smem + stage * S::kStageBytes;
        tensor_g2s<CTAS>(at, &map_w, s * kDepth, row_w, lead_full + 8 * stage);
        tensor_g2s<CTAS>(at + S::kBytesW, &map_x, s * kDepth, row_x, lead_full + 8 * stage);
        issued = min(issued + 1, S::kStages);
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
    }
    // Every copy has landed, and every product that reads it is done, before
    // shared memory is given back: the last stages' empty barriers
    const unsigned long long t0 = global_ns();
    for (int s = 0; s < issued; ++s) {
      stage = stage == 0 ? S::kStages - 1 : stage - 1;
      if (stage == S::kStages - 1) phase ^= 1;
      while (!mbar_try_wait(empty + 8 * stage, phase))
        if (global_ns() - t0 > limit_ns) {
          *dead = 1;
          ok = false;
          break;
        }
    }
    if (!ok || *dead != 0) atomicMax(status, epoch);
  } else if (warp == 1 && rank == 0) {
    // ---- products
    constexpr uint32_t idesc = half_mma(S::kChannels, BN);
    const uint32_t one = elect_one();
    int stage = 0, set = 0;
    uint32_t phase = 0, set_phase = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < order.tiles; t += stride) {
      ok = __all_sync(0xffffffffu, wait_or_dead(acc_empty + 8 * set, set_phase ^ 1, dead, limit_ns));
      if (!ok) break;
      tensor_fence_after();
      for (int s = 0; s < steps; ++s) {
        ok = __all_sync(0xffffffffu, wait_or_dead(full + 8 * stage, phase, dead, limit_ns));
        if (!ok) break;
        tensor_fence_after();
        const uint32_t at = tiles_smem + stage * S::kStageBytes;
        const uint64_t dw = tile_descriptor(at), dx = tile_descriptor(at + S::kBytesW);
#pragma unroll
        for (int q = 0; q < kDepth / 16; ++q)   // 16 halves: 32 bytes, 2 units of the descriptor
          mma_half<CTAS>(tmem + set * BN, dw + 2 * q, dx + 2 * q, idesc, s > 0 || q > 0, one);
        mma_commit<CTAS>(empty + 8 * stage, one);
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
      if (ok) mma_commit<CTAS>(acc_full + 8 * set, one);
      set ^= 1;
      if (set == 0) set_phase ^= 1;
    }
    if (*dead != 0 && lane == 0) atomicMax(status, epoch);
  } else if (warp >= 2) {
    // ---- results: a warp may read the 32 lanes of tensor memory of its number mod 4
    const int quarter = warp % 4;
    const uint32_t lead_empty = CTAS == 2 ? cluster_address(acc_empty, 0) : acc_empty;
    int set = 0;
    uint32_t set_phase = 0;
    bool ok = true;
    for (int t = first_tile; t < order.tiles; t += stride) {
      int tm, tn;
      order.at(t, tm, tn);
      const long long i = (long long)tm * S::kChannels + (int)rank * 128 + quarter * 32 + lane;
      const long long j0 = (long long)tn * BN;
      for (int c = (int)threadIdx.x - 64; c < BN; c += 128)
        token_scale[set][c] = j0 + c < a.n ? token_factor(a, j0 + c) : 0.f;
      const float channel = i < a.m ? channel_factor(a, i) : 0.f;
      if (ok && !wait_or_dead(acc_full + 8 * set, set_phase, dead, limit_ns)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      asm volatile("bar.sync 1, 128;" ::: "memory");   // token_scale is complete
      tensor_fence_after();
      for (int c0 = 0; c0 < BN && j0 + c0 < a.n; c0 += 32) {
        uint32_t r[32];
        tmem_load32(r, tmem + ((uint32_t)(quarter * 32) << 16) + set * BN + c0);
        if (i < a.m) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (j0 + c0 + c < a.n)
              store_output(a, i, j0 + c0 + c,
                           ok ? __uint_as_float(r[c]) : __uint_as_float(0x7fc00000u), channel,
                           token_scale[set][c0 + c]);
        }
        __syncwarp();
      }
      tensor_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead_empty + 8 * set);
      set ^= 1;
      if (set == 0) set_phase ^= 1;
    }
    if (!ok && lane == 0) atomicMax(status, epoch);
  }
  __syncwarp();
  tensor_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();
  tensor_fence_after();
  if (warp == 1) tmem_free<CTAS>(tmem, S::kColumns);
}

// ------------------------------------------- tiles with W as it is stored --

// From 9 tokens to a few thousand, where converting W beforehand would cost more than
// the product: W reaches shared memory as 8-bit integers, eight warps make
// halves of it on the way to tensor memory, and the tensor cores take their
// first operand from there.  (In shared memory the halves would cost four
// times their 8-bit bytes of its bandwidth, more than an SM has at the rate W
// streams in.)  One tile a CTA, or 256 x 256 a pair; small shapes fit twice on an
// SM, so that one's ends overlap the other's middle.  `split` CTAs of a cluster
// share a tile's depth when there are few tiles and add their accumulators
// through each other's shared memory, in rank order.
//
// Up to 64 tokens X too arrives as 8-bit integers and four more warps make its
// halves in shared memory (RAW): the call is one kernel.  Wider tiles read halves
// that halves_kernel made: made here they would cost shared memory twice the traffic.
//
// Warp 0 copies W, warp 1 copies X, warp 2 multiplies, warp 3 holds the tensor memory,
// warps 4 to 11 convert W and store the results, warps 12 to 15 (RAW) convert X.
constexpr int kStepDepth = 128;   // of a step: 128 bytes of W, 256 of X's halves
template <int CTAS, int BN>
struct Stream {
  static constexpr bool kRaw = BN <= 64;   // and two CTAs an SM
  static constexpr int kChannels = 128 * CTAS;
  static constexpr int kBytesW = 128 * kStepDepth, kHalfX = BN / CTAS * 128;
  static constexpr int kBytesX = 2 * kHalfX, kBytesRaw = kRaw ? BN * kStepDepth : 0;
  // steps of W, of X's halves and of W's halves in tensor memory, of raw X
  static constexpr int kStagesA = kRaw ? 2 : 4, kStagesX = kStagesA, kStagesRaw = kRaw ? 2 : 0;
  static constexpr int kStagesW = kRaw ? (BN == 64 ? 3 : 5) : 4;
  static constexpr int kColumnsA = kStepDepth / 2;
  static constexpr int kColumns = kRaw ? 256 : 512;
  static constexpr int kThreads = kRaw ? 512 : 384;
  static constexpr int kAtX = kStagesW * kBytesW, kAtRaw = kAtX + kStagesX * kBytesX;
  static constexpr int kRing = kAtRaw + kStagesRaw * kBytesRaw;
  static constexpr int kSmem = kRing + 1024;
  static_assert(BN + kStagesA * kColumnsA <= kColumns, "tensor memory");
  static_assert(BN * 128 * 4 <= kRing, "the exchange of sums");
};

// v[c] * channel * token[c] + beta * y[c] to `count` of 16 tokens of a channel
template <class T>
__device__ __forceinline__ void store_tokens(T* y, long long ldy, int count, const float (&v)[16],
                                             float channel, const float* token, float beta) {
#pragma unroll
  for (int c = 0; c < 16; ++c)
    if (c < count) {
      float r = v[c] * channel * token[c];
      if (beta != 0.f) r = fmaf(beta, to_float(y[c * ldy]), r);
      y[c * ldy] = from_float<T>(r);
    }
}
__device__ __forceinline__ void store_tokens_any(const GemmqAny& a, long long i, long long j,
                                                 int count, const float (&v)[16], float channel,
                                                 const float* token) {
  const long long at = j * a.ldy + i;
  if (a.type == 's')
    store_tokens(static_cast<float*>(a.Y) + at, a.ldy, count, v, channel, token, a.beta);
  else if (a.type == 'h')
    store_tokens(static_cast<__half*>(a.Y) + at, a.ldy, count, v, channel, token, a.beta);
  else
    store_tokens(static_cast<__nv_bfloat16*>(a.Y) + at, a.ldy, count, v, channel, token, a.beta);
}

template <int CTAS, int BN>
__global__ void __launch_bounds__(Stream<CTAS, BN>::kThreads, Stream<CTAS, BN>::kRaw ? 2 : 1)
    gemmq_stream(const __grid_constant__ CUtensorMap map_w,
                 const __grid_constant__ CUtensorMap map_x, GemmqAny a, int tiles_n, int steps,
                 int split, int* status, int epoch, unsigned long long limit_ns,
                 uint32_t extra_tx) {
  using S = Stream<CTAS, BN>;
  constexpr bool RAW = S::kRaw;
  // the ring that X's copies fill: raw X, or its halves
  constexpr int COPIES = RAW ? S::kStagesRaw : S::kStagesX;
  extern __shared__ uint8_t raw_smem[];
  __shared__ alignas(8) uint64_t bar_words[2 * S::kStagesW + 2 * COPIES + 2 * S::kStagesA + 1];
  __shared__ uint32_t tmem_word;
  __shared__ int dead_word;
  __shared__ float token_scale[BN];
  volatile int* const dead = &dead_word;
  const uint32_t ring = (smem_addr(raw_smem) + 1023u) & ~1023u;
  const uint32_t w_full = smem_addr(bar_words), w_empty = w_full + 8 * S::kStagesW;
  const uint32_t x_full = w_empty + 8 * S::kStagesW, x_empty = x_full + 8 * COPIES;
  const uint32_t a_full = x_empty + 8 * COPIES, a_empty = a_full + 8 * S::kStagesA;
  const uint32_t acc_full = a_empty + 8 * S::kStagesA;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cluster = CTAS == 2 ? 2 : split;
  const int rank = cluster > 1 ? (int)cluster_rank() : 0;
  // tiles that share W side by side: it is read from HBM once
  const int tile = blockIdx.x / cluster, tm = tile / tiles_n, tn = tile - tm * tiles_n;
  // this CTA's channels and tokens, and its steps of the depth
  const int row_w = tm * S::kChannels + (CTAS == 2 ? rank * 128 : 0);
  const int row_x = tn * BN + (CTAS == 2 ? rank * (BN / CTAS) : 0);
  const int part = CTAS == 2 ? 0 : rank;
  const int s0 = (int)((long long)steps * part / split);
  const int mine = (int)((long long)steps * (part + 1) / split) - s0;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    // the first steps of W on their way to L2 while the predecessor still runs
    for (int u = 0; u < min(mine, 8); ++u)
      tensor_prefetch(&map_w, (s0 + u) * kStepDepth, row_w);
    for (int s = 0; s < S::kStagesW; ++s) {
      mbar_init(w_full + 8 * s, 1);
      mbar_init(w_empty + 8 * s, 8);
    }
    for (int s = 0; s < COPIES; ++s) {
      mbar_init(x_full + 8 * s, 1);
      mbar_init(x_empty + 8 * s, RAW ? 4 : 1);
    }
    for (int s = 0; s < S::kStagesA; ++s) {
      mbar_init(a_full + 8 * s, (RAW ? 12 : 8) * CTAS);
      mbar_init(a_empty + 8 * s, 1);
    }
    mbar_init(acc_full, 1);
    dead_word = 0;
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc<CTAS>(smem_addr(&tmem_word), S::kColumns);
  tensor_fence_before();
  __syncthreads();
  if (CTAS == 2) cluster_sync();
  tensor_fence_after();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t tmem = tmem_word, tmem_a = tmem + BN;
  const int group = (warp - 4) / 4, quarter = warp % 4;   // of warps 4 to 11
  const long long i = (long long)row_w + quarter * 32 + lane;   // this thread's channel
  const long long j0 = (long long)tn * BN;
  float channel = 0.f;
  bool ok = true;

  if (warp < 2 && lane == 0) {
    // ---- copies of W (warp 0) or X (warp 1)
    const bool w = warp == 0;
    const int stages = w ? S::kStagesW : COPIES;
    const uint32_t full = w ? w_full : x_full, empty = w ? w_empty : x_empty;
    const uint32_t lead_full = CTAS == 2 && !w ? cluster_address(x_full, 0) : full;
    int u = 0;
    for (; u < mine; ++u) {
      const int stage = u % stages, depth = (s0 + u) * kStepDepth;
      if (!wait_or_dead(empty + 8 * stage, (u / stages & 1) ^ 1, dead, limit_ns)) break;
      const uint32_t bar = full + 8 * stage;
      if (w) {
        mbar_arrive_expect_tx(bar, S::kBytesW + extra_tx);
        tensor_g2s<1>(ring + stage * S::kBytesW, &map_w, depth, row_w, bar);
      } else if (RAW) {
        mbar_arrive_expect_tx(bar, S::kBytesRaw + extra_tx);
        tensor_g2s<1>(ring + S::kAtRaw + stage * S::kBytesRaw, &map_x, depth, row_x, bar);
      } else {
        if (CTAS == 1 || rank == 0) mbar_arrive_expect_tx(bar, CTAS * S::kBytesX + extra_tx);
        const uint32_t lead = lead_full + 8 * stage, at = ring + S::kAtX + stage * S::kBytesX;
        tensor_g2s<CTAS>(at, &map_x, depth, row_x, lead);
        tensor_g2s<CTAS>(at + S::kHalfX, &map_x, depth + kDepth, row_x, lead);
      }
    }
    // the arrivals of the last products reach this CTA before it may exit
    if (u == mine && !w) {
      for (int s = max(0, mine - COPIES); ok && s < mine; ++s)
        ok = wait_or_dead(x_empty + 8 * (s % COPIES), s / COPIES & 1, dead, limit_ns);
      for (int s = max(0, mine - S::kStagesA); ok && s < mine; ++s)
        ok = wait_or_dead(a_empty + 8 * (s % S::kStagesA), s / S::kStagesA & 1, dead, limit_ns);
    }
    if (u < mine) {
      // given up: copies in flight land, or have had their time to
      const unsigned long long t0 = global_ns();
      for (int s = max(0, u - stages); s < u; ++s)
        while (!mbar_try_wait(full + 8 * (s % stages), s / stages & 1) &&
               global_ns() - t0 <= limit_ns) {
        }
      ok = false;
    }
  } else if (warp == 2 && (CTAS == 1 || rank == 0)) {
    // ---- products
    constexpr uint32_t idesc = half_mma(S::kChannels, BN);
    const uint32_t one = elect_one();
    for (int u = 0; u < mine; ++u) {
      const int sx = u % S::kStagesX, sa = u % S::kStagesA;
      if (!RAW) ok = wait_or_dead(x_full + 8 * sx, u / S::kStagesX & 1, dead, limit_ns);
      if (ok) ok = wait_or_dead(a_full + 8 * sa, u / S::kStagesA & 1, dead, limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tensor_fence_after();
      const uint32_t at = ring + S::kAtX + sx * S::kBytesX;
      const uint64_t lo = tile_descriptor(at), hi = tile_descriptor(at + S::kHalfX);
      const uint32_t ta = tmem_a + sa * S::kColumnsA;
#pragma unroll
      for (int q = 0; q < kStepDepth / 16; ++q)
        mma_half_tmem<CTAS>(tmem, ta + 8 * q, (q < 4 ? lo : hi) + 2 * (q % 4), idesc,
                            u > 0 || q > 0, one);
      if (!RAW) mma_commit<CTAS>(x_empty + 8 * sx, one);
      mma_commit<CTAS>(a_empty + 8 * sa, one);
    }
    if (ok) mma_commit<CTAS>(acc_full, one);
  } else if (warp >= 4 && warp < 12) {
    // ---- W to halves: a thread a channel, a group of four warps each half of the depth.
    // Every warp takes every step: a parity wait that skipped a phase would match the
    // one before it.
    const int row = quarter * 32 + lane;
    const uint32_t lead_full = CTAS == 2 ? cluster_address(a_full, 0) : a_full;
    if (i < a.m) channel = a.sw != nullptr ? a.sw[i] : 1.f;
    for (int u = 0; u < mine; ++u) {
      const int stage = u % S::kStagesW, sa = u % S::kStagesA;
      ok = wait_or_dead(w_full + 8 * stage, u / S::kStagesW & 1, dead, limit_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const uint32_t at = ring + stage * S::kBytesW + row * 128;
      uint4 q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) q[c] = lds128(at + (((4 * group + c) ^ (row & 7)) << 4));
      reads_done();
      if (lane == 0) mbar_arrive(w_empty + 8 * stage);
      ok = wait_or_dead(a_empty + 8 * sa, (u / S::kStagesA & 1) ^ 1, dead, limit_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tensor_fence_after();
      const uint32_t to =
          tmem_a + ((uint32_t)(quarter * 32) << 16) + sa * S::kColumnsA + group * 32;
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        uint32_t h[16];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          halves_of(q[c + e].x, h[8 * e], h[8 * e + 1]);
          halves_of(q[c + e].y, h[8 * e + 2], h[8 * e + 3]);
          halves_of(q[c + e].z, h[8 * e + 4], h[8 * e + 5]);
          halves_of(q[c + e].w, h[8 * e + 6], h[8 * e + 7]);
        }
        tmem_store16(to + 8 * c, h);
      }
      tmem_stored();
      tensor_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CTAS == 2)
          mbar_arrive_cluster(lead_full + 8 * sa);
        else
          mbar_arrive(a_full + 8 * sa);
      }
    }
    // the accumulators, complete
    if (ok) ok = wait_or_dead(acc_full, 0, dead, limit_ns);
    ok = __all_sync(0xffffffffu, ok);
  } else if (RAW && warp >= 12) {
    // ---- X to halves: 16 elements a thread in turn, 8 threads a token
    const int id = (int)threadIdx.x - 384;
    for (int u = 0; u < mine; ++u) {
      const int stage = u % COPIES, sa = u % S::kStagesA;
      ok = wait_or_dead(x_full + 8 * stage, u / COPIES & 1, dead, limit_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      uint4 q[BN / 16];
#pragma unroll
      for (int e = 0; e < BN / 16; ++e) {
        const int r = id / 8 + 16 * e, c = id % 8;
        q[e] = lds128(ring + S::kAtRaw + stage * S::kBytesRaw + r * 128 + ((c ^ (r & 7)) << 4));
      }
      reads_done();
      if (lane == 0) mbar_arrive(x_empty + 8 * stage);
      ok = wait_or_dead(a_empty + 8 * sa, (u / S::kStagesA & 1) ^ 1, dead, limit_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int e = 0; e < BN / 16; ++e) {
        const int r = id / 8 + 16 * e, c = id % 8;
        const uint32_t to = ring + S::kAtX + sa * S::kBytesX + c / 4 * S::kHalfX + r * 128;
        uint32_t h[8];
        halves_of(q[e].x, h[0], h[1]);
        halves_of(q[e].y, h[2], h[3]);
        halves_of(q[e].z, h[4], h[5]);
        halves_of(q[e].w, h[6], h[7]);
        sts128(to + (((c % 4 * 2) ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
        sts128(to + (((c % 4 * 2 + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
      }
      // what the tensor cores read, which see shared memory as copies do
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full + 8 * sa);
    }
  } else if (warp == 3) {
    for (int c = lane; c < BN; c += 32)
      token_scale[c] = j0 + c < a.n ? token_factor(a, j0 + c) : 0.f;
  }
  // a warp's failure is the CTA's: its results are NaN
  __syncwarp();
  if (!ok) *dead = 1;
  const float nan = __uint_as_float(0x7fc00000u);
  if (split == 1) {
    __syncthreads();
    tensor_fence_after();
    const bool good = *dead == 0;
    if (warp >= 4 && warp < 12)
      for (int c0 = group * 16; c0 < BN && j0 + c0 < a.n; c0 += 32) {
        uint32_t r[16];
        tmem_load16(r, tmem + ((uint32_t)(quarter * 32) << 16) + c0);
        float v[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = good ? __uint_as_float(r[c]) : nan;
        if (i < a.m)
          store_tokens_any(a, i, j0 + c0, (int)min(16LL, a.n - j0 - c0), v, channel,
                           token_scale + c0);
        __syncwarp();
      }
    if (CTAS == 2) {
      tensor_fence_before();
      cluster_sync();
    }
  } else {
    // CTA q of the cluster adds columns q*width .. of all: [rank][column / 4][channel][column % 4]
    // in its shared memory, which every CTA has finished with
    cluster_sync();
    tensor_fence_after();
    const int width = BN / split, chunk = min(width, 4);   // 2, 4 or more
    const bool good = *dead == 0;
    if (warp >= 4 && warp < 12)
      for (int c0 = group * 16; c0 < BN; c0 += 32) {
        uint32_t r[16];
        tmem_load16(r, tmem + ((uint32_t)(quarter * 32) << 16) + c0);
        if (!good)
#pragma unroll
          for (int c = 0; c < 16; ++c) r[c] = 0x7fc00000u;
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
          const int owner = (c0 + c) / width, col = (c0 + c) - owner * width;
          const uint32_t slot = (uint32_t)(rank * width + col) * 512u +
                                (uint32_t)(quarter * 32 + lane) * 4u * chunk;
          if (chunk == 4) {
            cluster_store4(cluster_address(ring, owner) + slot, r[c], r[c + 1], r[c + 2], r[c + 3]);
          } else {
            cluster_store2(cluster_address(ring, owner) + slot, r[c], r[c + 1]);
            cluster_store2(cluster_address(ring, owner + 1) + slot, r[c + 2], r[c + 3]);
          }
        }
      }
    cluster_sync();
    if (warp >= 4 && warp < 12)
      for (int c = group * chunk; c < width; c += 2 * chunk) {
        const int col = rank * width + c;
        float v[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = 0.f;
          if (e < chunk)
            for (int r = 0; r < split; ++r) {
              float p;
              asm volatile("ld.shared.f32 %0, [%1];"
                           : "=f"(p)
                           : "r"(ring + (r * width + c) * 512 +
                                 ((quarter * 32 + lane) * chunk + e) * 4)
                           : "memory");
              v[e] += p;
            }
        }
        if (j0 + col < a.n && i < a.m)
          store_tokens_any(a, i, j0 + col, (int)min((long long)chunk, a.n - j0 - col), v, channel,
                           token_scale + col);
      }
  }
  if (*dead != 0 && threadIdx.x == 0) atomicMax(status, epoch);
  __syncwarp();
  tensor_fence_before();
  __syncthreads();
  tensor_fence_after();
  if (warp == 3) tmem_free<CTAS>(tmem, S::kColumns);
}

}  // namespace xsymv
