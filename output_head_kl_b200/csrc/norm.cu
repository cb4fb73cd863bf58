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

// Sum (or NaN-keeping maximum) over the row's threads: a warp, or a block of `warps` warps that
// exchange through `slot` (one barrier; the caller alternates slots, so that a slot is rewritten
// only after a later barrier).
template <bool WARP, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* slot, int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  if (WARP) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) slot[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? slot[lane] : 0.f;   // every warp reduces the same values in the same order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, w) : v + w;
  }
  return v;
}

// One row per warp (WARP: four rows a block, d <= 256 VPT) or per block.  A thread holds VPT steps of
// kV elements.  Nothing is kept between rows, so the grid is one block per row (or four rows): the
// next block's loads cover this one's barrier.
template <bool XF32, bool HF32, bool Q, int VPT, bool WARP>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(const NormParams p) {
  __shared__ float s_red[2][32];
  const int lane_t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int row_threads = WARP ? 32 : blockDim.x;
  const int warps = blockDim.x >> 5;
  const int64_t n = WARP ? static_cast<int64_t>(blockIdx.x) * warps + (threadIdx.x >> 5) : blockIdx.x;
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
  ss = row_reduce<WARP, false>(ss, s_red[0], warps);
  const float r = 1.0f / sqrtf(ss / static_cast<float>(p.d) + p.eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * row_threads + lane_t) * kV;
    if (c < p.d) {
#pragma unroll
      for (int j = 0; j < kV; ++j) {
        v[i][j] = v[i][j] * r * gm[i][j];
        if (Q) top = max_nan(top, fabsf(v[i][j]));
      }
      if (!Q) Pack<false>::store(p.y, base + c, v[i]);
    }
  }
  if (Q) {
    top = row_reduce<WARP, true>(top, s_red[1], warps);
    if (lane_t == 0) p.y_scale[n] = top / kE4m3Max;
    // q = y * (448 / top); a row of zeros has scale 0 and q = 0, and a row so small that 448 / top
    // would overflow is divided by its scale instead
    const bool tiny = top < 1e-30f;
    const float inv = tiny ? 0.f : kE4m3Max / top;
    const float scale = top / kE4m3Max;
    uint8_t* out = static_cast<uint8_t*>(p.y);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
        float q[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j) q[j] = !tiny ? v[i][j] * inv : (scale > 0.f ? v[i][j] / scale : 0.f);
        *reinterpret_cast<uint2*>(out + base + c) =
            make_uint2(pack_e4m3x2(q[0], q[1]) | (pack_e4m3x2(q[2], q[3]) << 16),
                       pack_e4m3x2(q[4], q[5]) | (pack_e4m3x2(q[6], q[7]) << 16));
      }
    }
  }
}

// Gradient.  A block runs rows blockIdx.x, + gridDim.x, ... (WARP: a row per warp), so that each thread
// keeps its columns' share of dgamma in registers; the block's sums go to one row of `part`, which
// launch_colsum adds up in a fixed order (no atomics).
template <bool HF32, int VPT, bool WARP>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_grad_kernel(const NormGradParams p) {
  __shared__ float s_red[2][2][32];
  extern __shared__ float s_part[];   // WARP: [warps - 1][d] shares of dgamma
  const int lane_t = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int row_threads = WARP ? 32 : blockDim.x;
  const int warps = blockDim.x >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = WARP ? static_cast<int64_t>(blockIdx.x) * warps + warp : blockIdx.x;
  const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * warps : gridDim.x;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  float acc[VPT][kV];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < kV; ++j) acc[i][j] = 0.f;
  int flip = 0;
  for (int64_t n = first; n < p.N; n += step) {
    const int64_t base = n * p.d;
    Pack<false> pdy[VPT];
    Pack<HF32> ph[VPT], pdh[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
        pdy[i].load(p.dy, base + c);
        ph[i].load(p.h, base + c);
        if (p.dh) pdh[i].load(p.dh, base + c);
      } else {
        pdy[i].zero();
        ph[i].zero();
      }
      if (c >= p.d || !p.dh) pdh[i].zero();
    }
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
        float h[kV], dy[kV], g[kV];
        ph[i].get(h);
        pdy[i].get(dy);
        load_gamma(p.gamma, p.gamma_f32, c, g);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          ss = fmaf(h[j], h[j], ss);
          dot = fmaf(dy[j] * g[j], h[j], dot);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      ss += __shfl_xor_sync(0xffffffffu, ss, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    if (!WARP) {
      // alternate buffers: a slot is rewritten two rows later, after the next row's barrier
      if (lane == 0) {
        s_red[flip][0][warp] = ss;
        s_red[flip][1][warp] = dot;
      }
      __syncthreads();
      ss = lane < warps ? s_red[flip][0][lane] : 0.f;
      dot = lane < warps ? s_red[flip][1][lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      flip ^= 1;
    }
    const float r = 1.0f / sqrtf(ss * inv_d + p.eps);
    const float k = dot * inv_d * r * r;      // mean(a xhat) r = (dot / d) r^2 per unit of h
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * row_threads + lane_t) * kV;
      if (c < p.d) {
        float h[kV], dy[kV], g[kV], dh[kV], o[kV];
        ph[i].get(h);
        pdy[i].get(dy);
        pdh[i].get(dh);
        load_gamma(p.gamma, p.gamma_f32, c, g);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          o[j] = fmaf(r, fmaf(-k, h[j], dy[j] * g[j]), dh[j]);
          acc[i][j] = fmaf(dy[j], h[j] * r, acc[i][j]);
        }
        Pack<HF32>::store(p.dx, base + c, o);
      }
    }
  }
  float* part = p.part + static_cast<int64_t>(blockIdx.x) * p.d;
  if (WARP) {
    if (warp > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = (i * 32 + lane) * kV;
        if (c < p.d) Pack<true>::store(s_part, static_cast<int64_t>(warp - 1) * p.d + c, acc[i]);
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
          q.load(s_part, static_cast<int64_t>(w) * p.d + c);
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

// Column sums: 32 columns a block, 16 row groups, each summed in row order and then added up in order.
constexpr int kColsumRows = 16;
__global__ void __launch_bounds__(32 * kColsumRows)
    colsum_kernel(const float* __restrict__ part, int rows, int n, float* __restrict__ out) {
  __shared__ float s[kColsumRows][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float a = 0.f;
  if (c < n) {
#pragma unroll 8
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

// Steps per thread: a warp per row up to 1024 elements (no barrier); above, blocks of at most 256
// threads when there are rows enough to fill the device (more rows in flight per SM), and the
// fewest steps when there are few rows (the shortest chain of loads).
NormShape norm_shape(int64_t N, int d, int sms) {
  const int vecs = (d + kV - 1) / kV;
  if (vecs <= 32 * 4 && N >= sms) {
    int vpt = 1;
    while (32 * vpt < vecs) vpt *= 2;
    return {true, vpt, 32};
  }
  const int want = N > 2 * static_cast<int64_t>(sms) ? 256 : 512;
  int vpt = 1;
  while (vpt < 8 && (vecs + vpt - 1) / vpt > want) vpt *= 2;
  const int threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
  return {false, vpt, threads};
}

constexpr int kNormWarps = 4;   // rows of a block with a row per warp

template <bool XF32, bool HF32, bool Q>
cudaError_t launch_norm(const NormParams& p, const NormShape& sh, cudaStream_t s) {
  if (sh.warp) {
    const unsigned grid = static_cast<unsigned>((p.N + kNormWarps - 1) / kNormWarps);
    switch (sh.vpt) {
      case 1: rmsnorm_kernel<XF32, HF32, Q, 1, true><<<grid, 32 * kNormWarps, 0, s>>>(p); break;
      case 2: rmsnorm_kernel<XF32, HF32, Q, 2, true><<<grid, 32 * kNormWarps, 0, s>>>(p); break;
      default: rmsnorm_kernel<XF32, HF32, Q, 4, true><<<grid, 32 * kNormWarps, 0, s>>>(p); break;
    }
  } else {
    const unsigned grid = static_cast<unsigned>(p.N);
    switch (sh.vpt) {
      case 1: rmsnorm_kernel<XF32, HF32, Q, 1, false><<<grid, sh.threads, 0, s>>>(p); break;
      case 2: rmsnorm_kernel<XF32, HF32, Q, 2, false><<<grid, sh.threads, 0, s>>>(p); break;
      case 4: rmsnorm_kernel<XF32, HF32, Q, 4, false><<<grid, sh.threads, 0, s>>>(p); break;
      default: rmsnorm_kernel<XF32, HF32, Q, 8, false><<<grid, sh.threads, 0, s>>>(p); break;
    }
  }
  return cudaGetLastError();
}

template <bool HF32>
cudaError_t launch_norm_grad(const NormGradParams& p, const NormShape& sh, int grid, cudaStream_t s) {
  if (sh.warp) {
    const size_t smem = static_cast<size_t>(kNormWarps - 1) * p.d * 4;
    switch (sh.vpt) {
      case 1: rmsnorm_grad_kernel<HF32, 1, true><<<grid, 32 * kNormWarps, smem, s>>>(p); break;
      case 2: rmsnorm_grad_kernel<HF32, 2, true><<<grid, 32 * kNormWarps, smem, s>>>(p); break;
      default: rmsnorm_grad_kernel<HF32, 4, true><<<grid, 32 * kNormWarps, smem, s>>>(p); break;
    }
  } else {
    switch (sh.vpt) {
      case 1: rmsnorm_grad_kernel<HF32, 1, false><<<grid, sh.threads, 0, s>>>(p); break;
      case 2: rmsnorm_grad_kernel<HF32, 2, false><<<grid, sh.threads, 0, s>>>(p); break;
      case 4: rmsnorm_grad_kernel<HF32, 4, false><<<grid, sh.threads, 0, s>>>(p); break;
      default: rmsnorm_grad_kernel<HF32, 8, false><<<grid, sh.threads, 0, s>>>(p); break;
    }
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rmsnorm(const NormParams& p, int sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.N, p.d, sms);
  if (p.y_e4m3) {
    if (p.x_f32) return p.h_f32 ? launch_norm<true, true, true>(p, sh, s) : launch_norm<true, false, true>(p, sh, s);
    return p.h_f32 ? launch_norm<false, true, true>(p, sh, s) : launch_norm<false, false, true>(p, sh, s);
  }
  if (p.x_f32) return p.h_f32 ? launch_norm<true, true, false>(p, sh, s) : launch_norm<true, false, false>(p, sh, s);
  return p.h_f32 ? launch_norm<false, true, false>(p, sh, s) : launch_norm<false, false, false>(p, sh, s);
}

int rmsnorm_grad_blocks(int64_t N, int d, int sms) {
  const NormShape sh = norm_shape(N, d, sms);
  const int64_t rows = sh.warp ? (N + kNormWarps - 1) / kNormWarps : N;
  const int64_t cap = std::min<int64_t>(kNormGradBlocks, static_cast<int64_t>(sms) * 4);
  return static_cast<int>(std::min(rows, cap));
}

cudaError_t launch_rmsnorm_grad(const NormGradParams& p, int sms, cudaStream_t s) {
  const NormShape sh = norm_shape(p.N, p.d, sms);
  const int grid = rmsnorm_grad_blocks(p.N, p.d, sms);
  return p.h_f32 ? launch_norm_grad<true>(p, sh, grid, s) : launch_norm_grad<false>(p, sh, grid, s);
}

cudaError_t launch_colsum(const float* part, int rows, int n, float* out, cudaStream_t s) {
  colsum_kernel<<<(n + 31) / 32, dim3(32, kColsumRows), 0, s>>>(part, rows, n, out);
  return cudaGetLastError();
}

}  // namespace kdkl
