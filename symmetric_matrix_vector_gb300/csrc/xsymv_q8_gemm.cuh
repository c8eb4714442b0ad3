// The product of 8-bit matrices on the tensor cores.
//
// GB300 has no fast integer path (mma.sync on 8-bit integers: 256 multiply-adds
// a clock and SM, as many as dp4a; on halves 1000; tcgen05 on halves 8192),
// so 8-bit integers are multiplied as halves: every value is exact in a half,
// every product exact in a float, and the float accumulators are exact while
// sums stay below 2^24.
#pragma once

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

// ------------------------------------------------------ operands as halves --

// Rows of kp halves (a multiple of kDepth, zeros beyond k) from rows of k
// integers at any alignment: what the tensor copies read.
constexpr int kDepth = 64;   // of a stage: 128 bytes of halves
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
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    constexpr uint32_t idesc = half_mma(S::kChannels, BN);
    int stage = 0, set = 0;
    uint32_t phase = 0, set_phase = 0;
    bool ok = true;
    for (int t = first_tile; ok && t < order.tiles; t += stride) {
      if (!wait_or_dead(acc_empty + 8 * set, set_phase ^ 1, dead, limit_ns)) break;
      tensor_fence_after();
      for (int s = 0; s < steps; ++s) {
        if (!wait_or_dead(full + 8 * stage, phase, dead, limit_ns)) {
          ok = false;
          break;
        }
        tensor_fence_after();
        const uint32_t at = tiles_smem + stage * S::kStageBytes;
        const uint64_t dw = tile_descriptor(at), dx = tile_descriptor(at + S::kBytesW);
#pragma unroll
        for (int q = 0; q < kDepth / 16; ++q)   // 16 halves: 32 bytes, 2 units of the descriptor
          mma_half<CTAS>(tmem + set * BN, dw + 2 * q, dx + 2 * q, idesc, s > 0 || q > 0);
        mma_commit<CTAS>(empty + 8 * stage);
        if (++stage == S::kStages) stage = 0, phase ^= 1;
      }
      if (ok) mma_commit<CTAS>(acc_full + 8 * set);
      set ^= 1;
      if (set == 0) set_phase ^= 1;
    }
    if (*dead != 0) atomicMax(status, epoch);
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

}  // namespace xsymv
