// RMS norm with the residual's addition, bf16 or e4m3 output, and its gradient (sm_100a).
//
//   h = x + residual,  r = 1 / sqrt(mean_j h_j^2 + eps),  y = h r gamma
//   e4m3 output: scale = max_j |y_j| / 448,  q = e4m3(y / scale)
//   gradient, with xhat = h r and a = dy gamma:
//     dx = r (a - xhat mean_j(a_j xhat_j)) + dh,   dgamma = sum_rows dy xhat
//
// Both are bound by HBM: every element is read once and written once, a row stays in registers
// between the statistics and the output, and all sums are held in fp32.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "kdkl_internal.h"
#include "layer_internal.h"
#include "sm100.cuh"

namespace kdkl {
namespace {

constexpr int kV = kNormVec;
constexpr float kE4m3Max = 448.0f;

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// kV consecutive elements of a bf16 or fp32 row, kept packed until they are used.
template <bool F32>
struct Pack;
template <>
struct Pack<false> {
  uint4 a;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  }
  __device__ __forceinline__ void load_pieces(const void* p, const void*) { a = *static_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[kV]) const {
    v[0] = bf_lo(a.x), v[1] = bf_hi(a.x), v[2] = bf_lo(a.y), v[3] = bf_hi(a.y);
    v[4] = bf_lo(a.z), v[5] = bf_hi(a.z), v[6] = bf_lo(a.w), v[7] = bf_hi(a.w);
  }
  __device__ static __forceinline__ void store(void* p, int64_t i, const float (&v)[kV]) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Pack<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void load_pieces(const void* p, const void* q) {
    a = *static_cast<const float4*>(p);
    b = *static_cast<const float4*>(q);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[kV]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ static __forceinline__ void store(void* p, int64_t i, const float (&v)[kV]) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ void load_gamma(const void* g, bool f32, int c, float (&v)[kV]) {
  if (f32) {
    Pack<true> p;
    p.load(g, c);
    p.get(v);
  } else {
    Pack<false> p;
    p.load(g, c);
    p.get(v);
  }
}

// The larger of two magnitudes, NaN if either is (so that a row with a NaN gets a NaN scale).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two e4m3 values (round to nearest even, finite values beyond 448 to 448, NaN kept).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// 1 / rms.  A row whose squares sum to 0, with eps = 0, has no direction: 0, so that y, the e4m3 scale and the row's
// share of the gradient are 0 instead of 0 x inf.  (Only a sum of 0 gives inf.  Testing the sum instead made the
// gradient kernel 2 to 13 % slower at 768 to 2048 columns.)
__device__ __forceinline__ float rstd_of(float mean_sq, float eps) {
  const float r = rsqrtf(mean_sq + eps);
  return r == INFINITY ? 0.f : r;
}

// Sum and, with Q, NaN-keeping maximum over the row's threads, with one exchange: a warp, or a block of `warps`
// warps through `slots`.
template <bool WARP, bool Q>
__device__ __forceinline__ void row_reduce(float& sum, float& top, float2* slots, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (Q) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if (WARP) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slots[threadIdx.x >> 5] = make_float2(sum, top);
  __syncthreads();
  // every thread reduces the same values in the same order: reading them is cheapest for a few warps, another
  // round of shuffles the shorter chain for many (2.1 against 2.4 us for one row of 4096)
  if (warps <= 8) {
    sum = slots[0].x;
    top = slots[0].y;
    for (int w = 1; w < warps; ++w) {
      sum += slots[w].x;
      if (Q) top = max_nan(top, slots[w].y);
    }
    return;
  }
  const float2 mine = lane < warps ? slots[lane] : make_float2(0.f, 0.f);
  sum = mine.x;
  top = mine.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (Q) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
}

// One row per warp (WARP: four rows a block, d <= 256 VPT) or per block.  A thread holds VPT steps of
// kV elements.  Nothing is kept between rows, so the grid is one block per row (or four rows): the
// next block's loads cover this one's barrier.  Measured (x and y bf16): 32768 x 4096 in 156 us, 6.9 TB/s;
// 65536 x 1024 in 80 us, 6.7 TB/s; e4m3 output 140 us, 6.7 TB/s; one row of 4096 in 1.9 us.  Rows above 16384
// elements (eight steps) spill up to 188 bytes a thread: 4096 x 32768 in 191 us, 5.6 TB/s.
template <bool XF32, bool HF32, bool Q, int VPT, bool WARP>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(const NormParams p) {
  __shared__ float2 s_red[32];
  const int lane_t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int row_threads = WARP ? 32 : blockDim.x;
  const int warps = blockDim.x >> 5;
  const int64_t n = WARP ? static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  pdl_launch();
  if (WARP && n >= p.N) return;
  const int64_t base = n * p.d;
  float v[VPT][kV];
  float ss = 0.f;
  {
    Pack<XF32> px[VPT];
    Pack<HF32> pr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
        px[i].load(p.x, base + c);
        if (p.residual) pr[i].load(p.residual, base + c);
        else pr[i].zero();
      } else {
        px[i].zero();
        pr[i].zero();
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float r[kV];
      px[i].get(v[i]);
      pr[i].get(r);
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        if (p.residual) v[i][j] += r[j];
        ss = fmaf(v[i][j], v[i][j], ss);
      }
    }
  }
  float gm[VPT][kV];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * row_threads + lane_t) * kV;
    if (c < p.d) {
      if (p.h) Pack<HF32>::store(p.h, base + c, v[i]);
      load_gamma(p.gamma, p.gamma_f32, c, gm[i]);
    }
  }
  // e4m3: q = y / scale does not depend on r, so the row's largest |h gamma| is found with the sum of squares
  float top = 0.f;
  if (Q) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          v[i][j] *= gm[i][j];
          top = max_nan(top, fabsf(v[i][j]));
        }
      }
    }
  }
  row_reduce<WARP, Q>(ss, top, s_red, warps);
  const float r = rstd_of(ss / static_cast<float>(p.d), p.eps);
  if (!Q) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
#pragma unroll
        for (int j = 0; j < kV; ++j) v[i][j] = v[i][j] * r * gm[i][j];
        Pack<false>::store(p.y, base + c, v[i]);
      }
    }
  } else {
    if (lane_t == 0) p.y_scale[n] = top * r / kE4m3Max;
    // q = h gamma (448 / top); a row of zeros (or whose squares overflow: y = 0) has scale 0 and q = 0, and a row
    // so small that 448 / top would overflow is first multiplied by a power of two, which is exact
    if (top < 1e-30f) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) v[i][j] *= 0x1p100f;
      top *= 0x1p100f;
    }
    const float inv = (top == 0.f || (r == 0.f && top < INFINITY)) ? 0.f : kE4m3Max / top;
    uint8_t* out = static_cast<uint8_t*>(p.y);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
        float q[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) q[j] = v[i][j] * inv;
        *reinterpret_cast<uint2*>(out + base + c) =
            make_uint2(pack_e4m3x2(q[0], q[1]) | (pack_e4m3x2(q[2], q[3]) << 16),
                       pack_e4m3x2(q[4], q[5]) | (pack_e4m3x2(q[6], q[7]) << 16));
      }
    }
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Gradient.  A block runs rows blockIdx.x, + gridDim.x, ... (WARP: a row per warp), so that each thread
// keeps its columns' share of dgamma in registers; the block's sums go to one row of `part`, which
// launch_colsum adds up in a fixed order (no atomics).
//
// A block's rows follow one another, so the next rows' loads have to be in flight while this one is
// reduced: each thread copies its own 16-byte pieces of the next kGradStages - 1 rows to shared memory
// asynchronously (it alone reads them, so no barrier is needed), which costs no registers.  Measured (bf16):
// 32768 x 4096 in 170 us with launch_colsum, 6.3 TB/s (where the ways to load were compared it took 161 us, against
// 183 with plain loads and 241 with the next row in registers, which halves the resident blocks); 1003 x 896 with an
// fp32 stream in 9.9 us.
constexpr int grad_pieces(int vpt, bool h_f32) { return vpt * (1 + 2 * (h_f32 ? 2 : 1)); }
constexpr int kGradStages = 3;
// Rows beyond 16 elements a thread do not fit the ring: they are read twice, the second time from L2, with nothing in
// flight across the barrier (fp32, 16384 x 8192: 409 us, 4.6 TB/s; bf16, 8192 x 16384: 353 us, 3.0 TB/s, and 16384 x
// 8200, one block an SM: 624 us, 1.7 TB/s).
constexpr bool grad_ring(int vpt) { return vpt <= 2; }

template <bool HF32, int VPT, bool WARP>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_grad_kernel(const NormGradParams p) {
  __shared__ __align__(16) float2 s_red[2][kNormMaxThreads / 32];
  extern __shared__ __align__(16) uint8_t s_dyn[];   // [stage][piece][thread] 16 bytes; then WARP: shares of dgamma
  constexpr bool kRing = grad_ring(VPT);
  constexpr int kP = grad_pieces(VPT, HF32);
  constexpr int kH = HF32 ? 2 : 1;                   // pieces of one step of h or dh
  const int lane_t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int row_threads = WARP ? 32 : blockDim.x;
  const int warps = blockDim.x >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * warps + warp : blockIdx.x;
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * warps : gridDim.x;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  const uint32_t ring = smem_u32(s_dyn) + threadIdx.x * 16;
  const uint32_t piece_bytes = blockDim.x * 16;
  constexpr int kSize = HF32 ? 4 : 2;
  auto fetch = [&](int64_t n, int stage) {
    if (!kRing) return;
    if (n < p.N) {
      const int64_t base = n * p.d;
      const uint32_t dst = ring + stage * kP * piece_bytes;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * row_threads + lane_t) * kV;
        if (c < p.d) {
          const uint32_t at = dst + i * (1 + 2 * kH) * piece_bytes;
          cp_async16(at, static_cast<const uint16_t*>(p.dy) + base + c);
#pragma unroll
          for (int k = 0; k < kH; ++k) {
            cp_async16(at + (1 + k) * piece_bytes, static_cast<const uint8_t*>(p.h) + (base + c) * kSize + k * 16);
            if (p.dh)
              cp_async16(at + (1 + kH + k) * piece_bytes,
                         static_cast<const uint8_t*>(p.dh) + (base + c) * kSize + k * 16);
          }
        }
      }
    }
    cp_async_commit();   // one group per row, empty past the end
  };
  auto piece = [&](int stage, int i, int k) {
    return s_dyn + static_cast<size_t>((stage * kP + i * (1 + 2 * kH) + k) * piece_bytes) + threadIdx.x * 16;
  };
  pdl_wait();
  pdl_launch();
  constexpr bool kKeep = kRing;   // gamma and the row stay in registers
  float acc[VPT][kV], gm[kKeep ? VPT : 1][kV];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * row_threads + lane_t) * kV;
#pragma unroll
    for (int j = 0; j < kV; ++j) acc[i][j] = 0.f;
    if (kKeep && c < p.d) load_gamma(p.gamma, p.gamma_f32, c, gm[i]);
  }
#pragma unroll
  for (int k = 0; k < kGradStages - 1; ++k) fetch(first + k * step, k);
  int flip = 0, stage = 0;
  for (int64_t n = first; n < p.N; n += step) {
    const int64_t base = n * p.d;
    fetch(n + (kGradStages - 1) * step, stage == 0 ? kGradStages - 1 : stage - 1);
    if (kRing) cp_async_wait<kGradStages - 1>();   // this row's pieces have landed
    Pack<false> pdy[kKeep ? VPT : 1];
    Pack<HF32> ph[kKeep ? VPT : 1];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      const int r = kKeep ? i : 0;
      if (c < p.d) {
        if (kRing) {
          pdy[r].load_pieces(piece(stage, i, 0), nullptr);
          ph[r].load_pieces(piece(stage, i, 1), piece(stage, i, kH));
        } else {
          pdy[r].load(p.dy, base + c);
          ph[r].load(p.h, base + c);
          load_gamma(p.gamma, p.gamma_f32, c, gm[r]);
        }
        float h[kV], dy[kV];
        ph[r].get(h);
        pdy[r].get(dy);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          ss = fmaf(h[j], h[j], ss);
          dot = fmaf(dy[j] * h[j], gm[r][j], dot);
        }
      }
    }
    // both sums at once: lanes 0-15 go on with ss, lanes 16-31 with dot
    {
      const bool up = lane & 16;
      const float mine = up ? dot : ss, other = up ? ss : dot;
      float v = mine + __shfl_xor_sync(0xffffffffu, other, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      const float w = __shfl_xor_sync(0xffffffffu, v, 16);
      ss = up ? w : v;
      dot = up ? v : w;
    }
    if (!WARP) {
      // alternate buffers: a slot is rewritten two rows later, after the next row's barrier
      if (lane == 0) s_red[flip][warp] = make_float2(ss, dot);
      __syncthreads();
      ss = dot = 0.f;
      for (int w = 0; w < warps; ++w) {
        const float2 q = s_red[flip][w];
        ss += q.x;
        dot += q.y;
      }
      flip ^= 1;
    }
    const float r = rstd_of(ss * inv_d, p.eps);
    const float rk = dot * inv_d * r * r * r;   // r mean(a xhat) per unit of xhat = (dot / d) r^3 per unit of h
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      const int q = kKeep ? i : 0;
      if (c < p.d) {
        if (!kKeep) {
          pdy[q].load(p.dy, base + c);
          ph[q].load(p.h, base + c);
          load_gamma(p.gamma, p.gamma_f32, c, gm[q]);
        }
        float h[kV], dy[kV], o[kV];
        ph[q].get(h);
        pdy[q].get(dy);
        if (p.dh) {
          Pack<HF32> pdh;
          if (kRing) pdh.load_pieces(piece(stage, i, 1 + kH), piece(stage, i, 2 * kH));
          else pdh.load(p.dh, base + c);
          pdh.get(o);
        } else {
#pragma unroll
          for (int j = 0; j < kV; ++j) o[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          o[j] = fmaf(r * gm[q][j], dy[j], fmaf(-rk, h[j], o[j]));
          acc[i][j] = fmaf(dy[j] * h[j], r, acc[i][j]);
        }
        Pack<HF32>::store(p.dx, base + c, o);
      }
    }
    stage = stage + 1 == kGradStages ? 0 : stage + 1;
  }
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.d;
  if (WARP) {
    float* shares = reinterpret_cast<float*>(s_dyn + static_cast<size_t>(kGradStages * kP) * piece_bytes);
    if (warp > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * 32 + lane) * kV;
        if (c < p.d) Pack<true>::store(shares, static_cast<int64_t>(warp - 1) * p.d + c, acc[i]);
      }
    }
    __syncthreads();
    if (warp > 0) return;
    for (int w = 0; w + 1 < warps; ++w) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * 32 + lane) * kV;
        if (c < p.d) {
          Pack<true> q;
          float o[kV];
          q.load(shares, static_cast<int64_t>(w) * p.d + c);
          q.get(o);
#pragma unroll
          for (int j = 0; j < kV; ++j) acc[i][j] += o[j];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * row_threads + lane_t) * kV;
    if (c < p.d) Pack<true>::store(part, c, acc[i]);
  }
}

// Column sums: 32 columns a block, 32 row groups, each summed in row order and then added up in order.
constexpr int kColsumRows = 32;
__global__ void __launch_bounds__(32 * kColsumRows)
    colsum_kernel(const float* __restrict__ part, int rows, int n, float* __restrict__ out) {
  __shared__ float s[kColsumRows][33];
  pdl_wait();
  pdl_launch();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < n) {
#pragma unroll 16
    for (int r = threadIdx.y; r < rows; r += kColsumRows) a += part[static_cast<int64_t>(r) * n + c];
  }
  s[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && c < n) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < kColsumRows; ++r) t += s[r][threadIdx.x];
    out[c] = t;
  }
}

// Shape of a row's threads: `warp` = one row per warp, else threads per row; VPT steps each.
struct NormShape {
  bool warp;
  int vpt;
  int threads;
};

NormShape block_shape(int vecs, int want) {
  int vpt = 1;
  while (vpt < 8 && (vecs + vpt - 1) / vpt > want) vpt *= 2;
  return {false, vpt, ((vecs + vpt - 1) / vpt + 31) / 32 * 32};
}

NormShape warp_shape(int vecs) {
  int vpt = 1;
  while (32 * vpt < vecs) vpt *= 2;
  return {true, vpt, 32};
}

// Forward.  Up to 1024 elements and with rows enough, a warp per row: no barrier.  Above, with few rows the
// fewest steps (the shortest chain of loads), else blocks of 256 threads, so that more rows are in flight per
// SM; with an e4m3 output four steps from 4096 elements on (32768 x 4096 with an fp32 stream: 213 against 232 us
// with two steps; with a bf16 stream both take 138 us).
NormShape norm_shape(int64_t N, int d, bool e4m3, int sms) {
  const int vecs = (d + kV - 1) / kV;
  if (vecs <= 32 * 4 && N >= sms) return warp_shape(vecs);
  if (N <= 2 * static_cast<int64_t>(sms) || vecs > 1024) return block_shape(vecs, kNormMaxThreads);
  return block_shape(vecs, e4m3 && vecs >= 512 ? (vecs + 3) / 4 : 256);
}

// Gradient.  Two steps a thread wherever they hold the row (a warp per row up to 512 elements, with rows
// enough): a row's fixed cost is shared by 16 elements, and the ring of the next rows fits beside it.
int grad_threads(int vecs) {   // of rows that are read twice
  const int vpt = vecs > 4 * kNormMaxThreads ? 8 : 4;
  return ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
}

NormShape norm_grad_shape(int64_t N, int d, bool h_f32, int sms) {
  const int vecs = (d + kV - 1) / kV;
  if (vecs <= 64 && N >= 8 * static_cast<int64_t>(sms)) return warp_shape(vecs);
  // two steps of 512 threads, of 480 with an fp32 stream: a larger ring does not fit shared memory
  if (vecs > (h_f32 ? 960 : 1024)) return {false, vecs > 4 * kNormMaxThreads ? 8 : 4, grad_threads(vecs)};
  return {false, 2, std::max(32, (vecs + 63) / 64 * 32)};
}

constexpr int kNormWarps = 4;       // rows of a block with a row per warp
constexpr int kNormGradWarps = 4;
constexpr int kGradSmemMax = 226 * 1024;
static_assert(kGradStages * grad_pieces(2, false) * 512 * 16 <= kGradSmemMax, "the ring of 512 threads, bf16");
static_assert(kGradStages * grad_pieces(2, true) * 480 * 16 <= kGradSmemMax, "the ring of 480 threads, fp32");

template <bool XF32, bool HF32, bool Q>
cudaError_t launch_norm(const NormParams& p, const NormShape& sh, cudaStream_t s) {
  if (sh.warp) {
    const LaunchConfig cfg(dim3(static_cast<unsigned>((p.N + kNormWarps - 1) / kNormWarps)), dim3(32 * kNormWarps), 0,
                           0, s);
    switch (sh.vpt) {
      case 1: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 1, true>, p);
      case 2: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 2, true>, p);
      default: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 4, true>, p);
    }
  }
  const LaunchConfig cfg(dim3(static_cast<unsigned>(p.N)), dim3(sh.threads), 0, 0, s);
  switch (sh.vpt) {
    case 1: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 1, false>, p);
    case 2: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 2, false>, p);
    case 4: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 4, false>, p);
    default: return cudaLaunchKernelEx(&cfg.c, rmsnorm_kernel<XF32, HF32, Q, 8, false>, p);
  }
}

struct GradLaunch {
  NormShape sh;
  int threads, smem, sms;
  int64_t rows;   // units of work: rows, or groups of rows with a row per warp
  int grid;       // out: blocks launched
};

template <bool HF32, int VPT, bool WARP>
cudaError_t grad_one(const NormGradParams& p, GradLaunch& g, cudaStream_t s) {
  // warps that an SM's registers hold of this kernel; set with its shared-memory limit on the first launch
  // on each device (past the 64th: on every launch)
  static std::atomic<int> reg_warps[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int warps = dev < 64 ? reg_warps[dev].load(std::memory_order_acquire) : 0;
  if (warps == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, rmsnorm_grad_kernel<HF32, VPT, WARP>);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(rmsnorm_grad_kernel<HF32, VPT, WARP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kGradSmemMax);
    if (e != cudaSuccess) return e;
    warps = 65536 / ((a.numRegs + 7) / 8 * 8 * 32);
    if (dev < 64) reg_warps[dev].store(warps, std::memory_order_release);
  }
  // The grid is at most the blocks that are resident at once (each runs its share of the rows to the end, and
  // one block more would run alone after all others), and no more than fill the rings' copies: beyond 512
  // threads an SM (1024 with a row per warp) more rows in flight were slower (2880 columns: 23.5 us with two
  // blocks an SM, 30.2 us with three).  A block gets two rows at least, which halves the partial sums.
  const int most = (WARP ? 1024 : 512) / g.threads;
  const int per_sm = std::min({kGradSmemMax / (g.smem + 2048), warps / (g.threads / 32), most});
  g.grid = static_cast<int>(std::min<int64_t>(
      {(g.rows + 1) / 2, kNormGradBlocks, static_cast<int64_t>(g.sms) * std::max(1, per_sm)}));
  const LaunchConfig cfg(dim3(g.grid), dim3(g.threads), g.smem, 0, s);
  return cudaLaunchKernelEx(&cfg.c, rmsnorm_grad_kernel<HF32, VPT, WARP>, p);
}

template <bool HF32>
cudaError_t launch_norm_grad(const NormGradParams& p, GradLaunch& g, cudaStream_t s) {
  if (g.sh.warp) {
    if (g.sh.vpt == 1) return grad_one<HF32, 1, true>(p, g, s);
    return grad_one<HF32, 2, true>(p, g, s);
  }
  switch (g.sh.vpt) {
    case 2: return grad_one<HF32, 2, false>(p, g, s);
    case 4: return grad_one<HF32, 4, false>(p, g, s);
    default: return grad_one<HF32, 8, false>(p, g, s);
  }
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams& p, int sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.N, p.d, p.y_e4m3, sms);
  if (p.y_e4m3) {
    if (p.x_f32) return p.h_f32 ? launch_norm<true, true, true>(p, sh, s) : launch_norm<true, false, true>(p, sh, s);
    return p.h_f32 ? launch_norm<false, true, true>(p, sh, s) : launch_norm<false, false, true>(p, sh, s);
  }
  if (p.x_f32) return p.h_f32 ? launch_norm<true, true, false>(p, sh, s) : launch_norm<true, false, false>(p, sh, s);
  return p.h_f32 ? launch_norm<false, true, false>(p, sh, s) : launch_norm<false, false, false>(p, sh, s);
}

int launch_rmsnorm_grad(const NormGradParams& p, int sms, cudaStream_t s, cudaError_t* err) {
  GradLaunch g;
  g.sh = norm_grad_shape(p.N, p.d, p.h_f32, sms);
  g.threads = g.sh.warp ? 32 * kNormGradWarps : g.sh.threads;
  g.smem = (grad_ring(g.sh.vpt) ? kGradStages * grad_pieces(g.sh.vpt, p.h_f32) * g.threads * 16 : 0) +
           (g.sh.warp ? (kNormGradWarps - 1) * p.d * 4 : 0);
  g.rows = g.sh.warp ? (p.N + kNormGradWarps - 1) / kNormGradWarps : p.N;
  g.sms = sms;
  g.grid = 0;
  *err = p.h_f32 ? launch_norm_grad<true>(p, g, s) : launch_norm_grad<false>(p, g, s);
  return g.grid;
}

cudaError_t launch_colsum(const float* part, int rows, int n, float* out, cudaStream_t s) {
  const LaunchConfig cfg(dim3((n + 31) / 32), dim3(32, kColsumRows), 0, 0, s);
  return cudaLaunchKernelEx(&cfg.c, colsum_kernel, part, rows, n, out);
}

}  // namespace kdkl
