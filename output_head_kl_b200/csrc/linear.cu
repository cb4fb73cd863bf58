// Linear layer with bias, activation and residual in its epilogue, and its gradient (sm_100a).
//
//   forward   z = x W^T + b,  y = act(z) + r           x [M, d_in], W [d_out, d_in], y [M, d_out]
//   gradient  dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_rows dz
//
// Three tcgen05 kernels share the operand layouts (128-byte swizzled tiles fetched by TMA):
//
//   linear_pair_kernel   256 x BN output tiles by CTA pairs (cta_group::2), persistent, two accumulators
//                        in TMEM so that the epilogue of one tile runs under the next tile's MMAs.
//   linear_split_kernel  the same tiles, fewer than there are pairs: 2 or 4 pairs of a cluster share a tile's
//                        reduction and join over distributed shared memory.
//   linear_small_kernel  few rows: the operands swap roles, so that 128 rows of W fill the MMA's M and the
//                        rows of x its N (16 to 128), and a cluster of CTAs splits the reduction and joins
//                        the partial tiles over distributed shared memory in a fixed order.  The weights
//                        stream through all SMs at once however few the rows are.
//
// Sums are held in fp32 (TMEM accumulators, fp32 joins); z is rounded to bf16 only where it is
// stored, and dz once, as the MMA operand of both gradient products.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "../../include/kdkl.h"
#include "kdkl_internal.h"
#include "layer_internal.h"
#include "sm100.cuh"

namespace kdkl {
namespace {

constexpr float kLog2eL = 1.4426950408889634f;

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / (1 + e^-z).  The hardware exponential and reciprocal are within 2 ulp each, far below the
// bf16 rounding of the results; for z below -88 the exponential is inf and the result 0.
__device__ __forceinline__ float sigmoid_f(float z) { return rcp_approx(1.0f + ex2_approx(-kLog2eL * z)); }

// The normal distribution function Phi(z), and e = e^(-z^2 / 2), which the density needs too.  Its lower tail is
// Phi(-a) = e^(-a^2 / 2) P(t) with t = 1 / (1 + p a), P a polynomial: the form of Hastings (Approximations for Digital
// Computers, 1955), its coefficients a minimax fit to the scaled tail e^(a^2 / 2) Phi(-a) over 0 <= a <= 13.5, within
// 1.6 x 2^-24 of it.  Nothing cancels for z << 0, where 1 + erf(z / sqrt 2) is 4 % off at z = -5; and the
// exponential serves both.  Measured at 16384 x 1024 x 4096 with residual and z: 144 us, with erff 156, with erfcf
// 208-221; the slopes' column sums there 81, 115 and 155 us.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = rcp_approx(fmaf(0.305f, fabsf(z), 1.0f));
  float q = 0.0366991982f;
  q = fmaf(q, t, -0.15298833f);
  q = fmaf(q, t, 0.185716912f);
  q = fmaf(q, t, -0.0379768386f);
  q = fmaf(q, t, 0.121021681f);
  q = fmaf(q, t, 0.103420869f);
  q = fmaf(q, t, 0.122466817f);
  q = fmaf(q, t, 0.121639736f);
  e = ex2_approx(-0.5f * kLog2eL * z * z);
  q = q * t * e;
  return z < 0.f ? q : 1.0f - q;
}

// 2 u of the tanh form of GELU: 0.5 (1 + tanh u) = sigmoid(2 u).
__device__ __forceinline__ float gelu_2u(float z) { return 1.5957691216057308f * fmaf(0.044715f * z * z, z, z); }

template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if (ACT == KDKL_ACT_RELU) return z < 0.f ? 0.f : z;   // NaN passes
  if (ACT == KDKL_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  }
  if (ACT == KDKL_ACT_GELU_TANH) return z * sigmoid_f(gelu_2u(z));
  if (ACT == KDKL_ACT_SILU) return z * sigmoid_f(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad_f(float z) {
  if (ACT == KDKL_ACT_RELU) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);   // NaN passes
  if (ACT == KDKL_ACT_GELU) {
    float e;
    const float cdf = normal_cdf(z, e);
    return fmaf(z * 0.3989422804014327f, e, cdf);
  }
  if (ACT == KDKL_ACT_GELU_TANH) {
    // 2 u = z (k + k c z^2) and its slope k + 3 k c z^2, k = 2 sqrt(2 / pi), c = 0.044715; z^2 is held at 1e4, where
    // p (1 - p) is 0 long since, so that it does not become inf
    const float z2 = fminf(z * z, 1e4f);
    const float p = sigmoid_f(z * fmaf(0.0713548163f, z2, 1.5957691216f));
    return fmaf(z * p * (1.0f - p), fmaf(0.214064449f, z2, 1.5957691216f), p);
  }
  if (ACT == KDKL_ACT_SILU) {
    const float p = sigmoid_f(z);
    return fmaf(z * p, 1.0f - p, p);
  }
  return 1.0f;
}

template <int ACT, int N>
__device__ __forceinline__ void act_each(float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = act_f<ACT>(v[j]);
}

template <int N>
__device__ __forceinline__ void act_all(float (&v)[N], int act) {
  switch (act) {
    case KDKL_ACT_RELU: act_each<KDKL_ACT_RELU>(v); break;
    case KDKL_ACT_GELU: act_each<KDKL_ACT_GELU>(v); break;
    case KDKL_ACT_GELU_TANH: act_each<KDKL_ACT_GELU_TANH>(v); break;
    case KDKL_ACT_SILU: act_each<KDKL_ACT_SILU>(v); break;
    default: break;
  }
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// ---------------------------------------------------------------- PTX of these kernels
// Instruction descriptor for kind::f8f6f4 with e4m3 A/B (both K-major) and fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool F8, bool PAIR>
__device__ __forceinline__ void umma(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
  if (!F8) {
    if (PAIR) umma_bf16_pair(d_tmem, ad, bd, idesc, acc);
    else umma_bf16(d_tmem, ad, bd, idesc, acc);
  } else if (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
        : "memory");
  }
}

// 32 lanes x 16 consecutive 32-bit columns: thread i of the warp gets lane (base + i).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Cluster barrier that orders execution only: nothing this thread wrote is waited for.  It closes the
// kernels, where peers must not exit while their shared memory or TMEM is still in use.
__device__ __forceinline__ void cluster_sync_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// A 16-byte read that leaves L1 alone (read once).
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Brings a box of a tensor into L2.
__device__ __forceinline__ void tma_prefetch_l2(const CUtensorMap* m, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y)
               : "memory");
}

// Arrival on a barrier of either CTA of the pair that says "this TMEM buffer has been read": the
// tcgen05 fence before it orders the reads, so no cluster-wide release of other memory is waited for.
__device__ __forceinline__ void mbar_arrive_pair(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4u(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(saddr)
               : "memory");
  return v;
}

__device__ __forceinline__ float4 ld_cluster_v4f(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// Operand layout of a product: element type and which operands are MN-major.
template <int OP>
struct LinLayout {
  static constexpr bool kF8 = OP == kLinFwdE4M3;
  static constexpr bool kFull = OP == kLinFwd || OP == kLinFwdE4M3;   // scales, bias, activation, residual
  static constexpr int kStepElems = kF8 ? 128 : 64;                   // elements of one 128-byte reduction block
};

// Zeroes the flag word before any of this launch's waits can time out (they take kWaitLimitNs at
// least; the bounds-checking build, whose checks can fail at once, clears it ahead of the launch).
__device__ __forceinline__ void clear_flags(const LinParams& p) {
  if (p.clear_flags && blockIdx.x == 0 && threadIdx.x == 0) *p.flags = 0u;
}

// ---------------------------------------------------------------- the epilogue of large tiles
// One warp's epilogue of 32 rows x 32 columns of fp32 sums, thread = row: scales, bias, z out, activation, residual,
// y out.  Staging buffers of 32 x 32 bf16 (64-byte swizzle: 16-byte chunk c of row r at c ^ (r / 2 & 3)): two for
// stores, one into which the residual is loaded.  TMA clips what lies past M or N on both ways.
constexpr int kStageBuf = 2048;

template <int OP>
struct Finisher {
  using L = LinLayout<OP>;
  const LinParams& p;
  const CUtensorMap *out, *pre, *res;
  uint8_t *wbuf, *rbuf;
  uint64_t* res_full;    // this warp's barrier of the residual's loads
  uint32_t bias, scale;  // shared memory: fp32 bias and scales of the warp's columns
  int lane;
  const AbortState& ab;
  int sbuf = 0;
  uint32_t res_phase = 0;
  bool res_pending = false;

  __device__ __forceinline__ uint32_t swizzled(const uint8_t* buf, int c16) const {
    return smem_u32(buf) + static_cast<uint32_t>(lane) * 64u +
           ((static_cast<uint32_t>(c16) ^ (static_cast<uint32_t>(lane >> 1) & 3u)) << 4);
  }

  __device__ __forceinline__ void store32(const CUtensorMap* tm, const float (&v)[32], int col, int row) {
    uint8_t* buf = wbuf + sbuf * kStageBuf;
    if (lane == 0) bulk_wait_read<1>();   // the store before last has read this buffer
    __syncwarp();
#pragma unroll
    for (int c16 = 0; c16 < 4; ++c16)
      st_shared_v4(swizzled(buf, c16), pack_bf16x2(v[c16 * 8 + 0], v[c16 * 8 + 1]),
                   pack_bf16x2(v[c16 * 8 + 2], v[c16 * 8 + 3]), pack_bf16x2(v[c16 * 8 + 4], v[c16 * 8 + 5]),
                   pack_bf16x2(v[c16 * 8 + 6], v[c16 * 8 + 7]));
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && dbg_ok((col & 7) == 0 && col >= 0 && row >= 0, p.flags)) {
      tma_store_2d(tm, buf, col, row);
      bulk_commit();
    }
    sbuf ^= 1;
  }

  // Whole warp: starts the load of a residual chunk.
  __device__ __forceinline__ void load_res(int col, int row) {
    res_pending = true;
    if (lane == 0) {
      mbar_arrive_expect_tx(res_full, kStageBuf);
      tma_load_2d(rbuf, res, res_full, dbg_ok((col & 7) == 0, p.flags) ? col : (col & ~7), row);
    }
  }

  // bias and scales of columns [col, col + 4) at offset `at` of the warp's columns
  __device__ __forceinline__ void load_side(int col, int at) const {
    if (!dbg_ok(col >= 0 && col + 4 <= p.N, p.flags)) return;
    if (p.bias) {
      const uint2 b = *reinterpret_cast<const uint2*>(p.bias + col);
      st_shared_v4(bias + at * 4, __float_as_uint(bf_lo(b.x)), __float_as_uint(bf_hi(b.x)),
                   __float_as_uint(bf_lo(b.y)), __float_as_uint(bf_hi(b.y)));
    }
    if (L::kF8) {
      const uint4 w = *reinterpret_cast<const uint4*>(p.w_scale + col);
      st_shared_v4(scale + at * 4, w.x, w.y, w.z, w.w);
    }
  }

  // Finishes the chunk at (row, col) with side data at offset `at`; next_col >= 0 is the chunk whose residual
  // to load next.  False if a wait gave up.
  __device__ __forceinline__ bool finish(float (&v)[32], int row, int col, int at, float xs, int next_col) {
    if (L::kFull) {
      if (L::kF8) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 w = ld_shared_v4f(scale + (at + g * 4) * 4);
          v[g * 4 + 0] *= xs * w.x;
          v[g * 4 + 1] *= xs * w.y;
          v[g * 4 + 2] *= xs * w.z;
          v[g * 4 + 3] *= xs * w.w;
        }
      }
      if (p.bias) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 b = ld_shared_v4f(bias + (at + g * 4) * 4);
          v[g * 4 + 0] += b.x;
          v[g * 4 + 1] += b.y;
          v[g * 4 + 2] += b.z;
          v[g * 4 + 3] += b.w;
        }
      }
      if (p.pre) store32(pre, v, col, row);
      act_all(v, p.act);
      if (p.residual) {
        if (!mbar_wait(res_full, res_phase, ab)) return false;
        res_phase ^= 1u;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint4 r = ld_shared_v4u(swizzled(rbuf, g));
          v[g * 8 + 0] += bf_lo(r.x), v[g * 8 + 1] += bf_hi(r.x);
          v[g * 8 + 2] += bf_lo(r.y), v[g * 8 + 3] += bf_hi(r.y);
          v[g * 8 + 4] += bf_lo(r.z), v[g * 8 + 5] += bf_hi(r.z);
          v[g * 8 + 6] += bf_lo(r.w), v[g * 8 + 7] += bf_hi(r.w);
        }
        // The next chunk's load may overwrite the buffer only after every lane has its values: the sums
        // above have used them (a read that is merely issued is not ordered before a TMA write).
        __syncwarp();
        res_pending = false;
        if (next_col >= 0) load_res(next_col, row);
      }
    }
    store32(out, v, col, row);
    return true;
  }

  // Ends the warp's work: every store has finished, and so has (bounded wait) a residual load that nothing
  // consumed because a wait gave up.
  __device__ __forceinline__ void close() {
    if (lane == 0) {
      if (res_pending) {
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(res_full), res_phase) && globaltimer_ns() - t0 < kDrainLimitNs) {
        }
      }
      bulk_wait<0>();
    }
    __syncwarp();
  }
};

// ============================================================================
// large tiles: one 256 x BN tile per CTA pair and turn
//
// Warp 0 issues the TMA loads, warp 1 of the even CTA the MMAs, and eight epilogue warps read TMEM (two
// per 32-lane quarter, each half of the tile's columns).  Tiles are swept in groups of row_group row
// blocks, column by column, so that the pairs running at once share their A rows and B columns in L2.
//
// Bound by the tensor cores and, equally, by what an SM takes in from L2: a 64-wide reduction block of a 256 x 256
// tile is 512 cycles of MMA and 32 KB a CTA, 64 bytes a cycle.  Measured at 16384 x 4096 x 4096 under the power cap:
// plain product 404 us (cuBLAS 401), with bias, SiLU, residual and z stored 458-465; dx 408, dW 429 (the last
// wave split: 448 without).  An epilogue of one tile takes 4,000 (plain) to 10,700 cycles (everything).
// ============================================================================
constexpr int kPairThreads = 320;
constexpr int kEpiWarps = 8;

template <int OP, int BN>
struct PairCfg {
  using L = LinLayout<OP>;
  static constexpr bool kAmn = OP == kLinDw;
  static constexpr bool kBmn = OP == kLinDx || OP == kLinDw;
  static constexpr int kCtaN = BN / 2;                      // B rows held by each CTA of the pair
  static constexpr int kBAtoms = (kCtaN + 63) / 64;         // MN-major B: whole 64-column swizzle atoms
  static constexpr int kABytes = kBM * 128;
  static constexpr int kBBytes = kBmn ? kBAtoms * 8192 : kCtaN * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kTxBytes = 2 * kStageBytes;          // both CTAs' bytes, counted on the even CTA
  // per epilogue warp: two staging buffers for stores and, with the full epilogue, one for the residual and the
  // bias and scales of the warp's BN / 2 columns
  static constexpr int kBufs = L::kFull ? 3 : 2;
  static constexpr int kSideBytes = L::kFull ? (BN / 2) * 4 * (L::kF8 ? 2 : 1) : 0;
  static constexpr int kEpiWarpBytes = kBufs * kStageBuf + kSideBytes;
  static constexpr int kEpiBytes = (kEpiWarps * kEpiWarpBytes + 1023) / 1024 * 1024;
  static constexpr int kStagesFit = (232448 - 1024 - kEpiBytes - 512) / kStageBytes;
  static constexpr int kStages = kStagesFit > 8 ? 8 : kStagesFit;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + kEpiBytes + 512;
  static constexpr uint32_t kIdesc = L::kF8 ? idesc_e4m3_f32(256, BN) : idesc_bf16_f32(256, BN, kAmn, kBmn);
  static constexpr int kAccStride = BN <= 128 ? 128 : 256;
  static constexpr uint32_t kTmemCols = 2 * kAccStride;
  static_assert(BN % 64 == 0 && BN >= 128 && BN <= 256, "two halves of whole 32-column chunks");
  static_assert(kStages >= 4 && (2 * kStages + 5 + kEpiWarps) * 8 + 16 <= 512, "stages");
};

// Unit u: an output tile (row block mb, column tile t) and its reduction blocks [kb0, kb1).  The units from
// full_units on are the last, partly filled wave's tiles, each split into `splits` shares of the reduction;
// `share` counts them over all those tiles (-1 for a whole tile).
struct PairUnit {
  int mb, t, kb0, kb1, share;
};

__device__ __forceinline__ PairUnit pair_unit(const LinParams& p, int u) {
  PairUnit w;
  int tile = u;
  w.kb0 = 0;
  w.kb1 = p.k_blocks;
  w.share = -1;
  if (u >= p.full_units) {
    const int tail = p.tiles - p.full_units;
    const int s = (u - p.full_units) / tail, i = u - p.full_units - s * tail;
    tile = p.full_units + i;
    w.kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * s / p.splits);
    w.kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (s + 1) / p.splits);
    w.share = i * p.splits + s;
  }
  // groups of row_group row blocks, each swept column by column
  const int rows = p.tiles / p.n_tiles;
  const int r0 = tile / (p.row_group * p.n_tiles) * p.row_group;
  const int rg = min(p.row_group, rows - r0);
  const int off = tile - r0 * p.n_tiles;
  w.t = off / rg;
  w.mb = r0 + off - w.t * rg;
  return w;
}

template <int OP, int BN>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmPre,
                       const __grid_constant__ CUtensorMap tmRes, const LinParams p) {
  using C = PairCfg<OP, BN>;
  using L = LinLayout<OP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::kStages * C::kABytes;
  uint8_t* sEpi = sB + C::kStages * C::kBBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + C::kEpiBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* res_full = drain + 1;   // one per epilogue warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + kEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0 = the CTA that issues the MMAs
  const int group = static_cast<int>(blockIdx.x >> 1), ngroups = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 64) {   // the descriptors travel while the barriers are set up
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmOut);
    if (L::kFull && p.pre) tma_prefetch_desc(&tmPre);
    if (L::kFull && p.residual) tma_prefetch_desc(&tmRes);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&res_full[w], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // the even CTA's barriers are initialised before any peer signal
  tc_fence_after();
  pdl_wait();       // nothing above touches the tensors
  pdl_launch();
  clear_flags(p);
  const uint32_t tmem_base = *tmem_slot;
  const AbortState ab{abort_flag, p.flags};

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool wrapped = false, stop = false;
      for (int u = group; u < p.units && !stop; u += ngroups) {
        const PairUnit w = pair_unit(p, u);
        const int arow = w.mb * 256 + static_cast<int>(rank) * kBM;
        const int brow = w.t * BN + static_cast<int>(rank) * C::kCtaN;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, ab)) {
            stop = true;
            break;
          }
          uint8_t* a = sA + stage * C::kABytes;
          uint8_t* b = sB + stage * C::kBBytes;
          const uint32_t bar0 = mapa_shared(smem_u32(&full[stage]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::kTxBytes);
          if (C::kAmn) {
            tma_load_2d_pair(a, &tmA, bar0, arow, kb * 64);
            tma_load_2d_pair(a + 8192, &tmA, bar0, arow + 64, kb * 64);
          } else {
            tma_load_2d_pair(a, &tmA, bar0, kb * L::kStepElems, arow);
          }
          if (C::kBmn) {
#pragma unroll
            for (int q = 0; q < C::kBAtoms; ++q)
              tma_load_2d_pair(b + q * 8192, &tmB, bar0, brow + q * 64, kb * 64);
          } else {
            tma_load_2d_pair(b, &tmB, bar0, kb * L::kStepElems, brow);
          }
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
            wrapped = true;
          }
        }
      }
      if (rank == 0 && *abort_flag) {
        // giving up: wait (bounded) until the copies already issued have landed
        const uint64_t w0 = globaltimer_ns();
        for (int s2 = 0; s2 < C::kStages; ++s2) {
          if (!wrapped && s2 >= stage) break;
          const uint32_t par = s2 < stage ? phase : (phase ^ 1u);
          while (!mbar_try_wait(smem_u32(&full[s2]), par) && globaltimer_ns() - w0 < kDrainLimitNs) {
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA only)
    if (lane == 0 && rank == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (int u = group; u < p.units; u += ngroups) {
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u, ab)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * C::kAccStride);
        bool got = true;
        const PairUnit w = pair_unit(p, u);
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          got = mbar_wait(&full[stage], phase, ab);
          if (!got) break;
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + stage * C::kABytes);
          const uint32_t b_addr = smem_u32(sB + stage * C::kBBytes);
#pragma unroll
          for (int j = 0; j < 4; ++j) {   // 32 bytes of the reduction axis (16 bf16 or 32 e4m3) per MMA
            const uint64_t ad = C::kAmn ? sdesc_sw128(a_addr + j * 2048, 8192, 1024)
                                        : sdesc_sw128(a_addr + j * 32, 16, 1024);
            const uint64_t bd = C::kBmn ? sdesc_sw128(b_addr + j * 2048, 8192, 1024)
                                        : sdesc_sw128(b_addr + j * 32, 16, 1024);
            umma<L::kF8, true>(d_tmem, ad, bd, C::kIdesc, (kb != w.kb0 || j != 0) ? 1u : 0u);
          }
          umma_commit_pair(&empty[stage], 0x3);
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!got) break;
        umma_commit_pair(&acc_full[acc], 0x3);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // every MMA issued above has finished before TMEM or shared memory is released
      umma_commit_pair(drain, 0x1);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(drain), 0)) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
          atomicOr(p.flags, kFlagTimeout);
          break;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue warps
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    const uint32_t acc_empty0 = mapa_shared(smem_u32(&acc_empty[0]), 0);
    uint8_t* wbuf = sEpi + (warp - 2) * C::kBufs * kStageBuf;
    const uint32_t side = smem_u32(sEpi + kEpiWarps * C::kBufs * kStageBuf + (warp - 2) * C::kSideBytes);
    Finisher<OP> fin{p,    &tmOut, &tmPre, &tmRes, wbuf, wbuf + 2 * kStageBuf, &res_full[warp - 2], side,
                     side + (BN / 2) * 4, lane, ab};
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = group; u < p.units; u += ngroups) {
      const PairUnit w = pair_unit(p, u);
      const bool split = w.share >= 0;
      const int row0 = w.mb * 256 + static_cast<int>(rank) * kBM + q * 32;   // the warp's first row
      const int row = row0 + lane;
      const int c_first = w.t * BN + half * (BN / 2);
      // What the epilogue reads is fetched while the tile's MMAs run: the residual's first 32-column chunk
      // into shared memory and the others into L2, bias and scales as fp32 into shared memory.
      float xs = 1.f;
      if (L::kFull) {
        if (!split && p.residual && c_first < p.N) {
          fin.load_res(c_first, row0);
#pragma unroll
          for (int c = 1; c < BN / 64; ++c)
            if (lane == 0 && c_first + c * 32 < p.N) tma_prefetch_l2(&tmRes, c_first + c * 32, row0);
        }
        __syncwarp();   // every lane has read the last tile's bias and scales
        const int lc = lane * 4;
        if (lc < BN / 2 && c_first + lc < p.N) fin.load_side(c_first + lc, lc);
        if (L::kF8 && row < p.M) xs = p.x_scale[row];
        __syncwarp();
      }
      if (!mbar_wait(&acc_full[acc], acc_phase, ab)) break;
      tc_fence_after();
      const uint32_t tbase = tmem_base + lane_addr + static_cast<uint32_t>(acc * C::kAccStride + half * (BN / 2));
      auto release_acc = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(acc_empty0 + static_cast<uint32_t>(acc) * 8u);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      };
      // A share of a split tile: the warp leaves its partial sums in the workspace (as groups of four columns,
      // lane by lane) and takes a ticket; the warp with the last one adds the shares up in their order
      // and finishes the tile, so the result does not depend on which that is.
      const int64_t warp_floats = 32 * (BN / 2);
      const int wslot = static_cast<int>(rank) * kEpiWarps + (warp - 2);
      float4* mine = reinterpret_cast<float4*>(
          p.part + (static_cast<int64_t>(w.share) * (2 * kEpiWarps) + wslot) * warp_floats);
      if (split) {
        // the last share of this tile, and the tile's ticket, lie in their parts of the workspace
        const int tile0 = w.share / p.splits;
        const bool room = dbg_ok(static_cast<int64_t>(tile0 + 1) * p.splits * (2 * kEpiWarps) * warp_floats <=
                                         p.part_floats && tile0 < kMaxSplitTiles, p.flags);
#pragma unroll 1
        for (int c = 0; c < BN / 64 && room; ++c) {
          if (c_first + c * 32 >= p.N) break;
          float v[32];
          tmem_ld32(tbase + c * 32, v);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < 8; ++g)
            __stcg(mine + (c * 8 + g) * 32 + lane, make_float4(v[g * 4], v[g * 4 + 1], v[g * 4 + 2], v[g * 4 + 3]));
        }
        release_acc();
        if (!room) continue;
        __threadfence();
        __syncwarp();
        uint32_t* ticket = p.tickets + tile0 * (2 * kEpiWarps) + wslot;
        int last = 0;
        if (lane == 0) {
          last = atomicAdd(ticket, 1u) == static_cast<uint32_t>(p.splits - 1);
          if (last) *ticket = 0u;   // as the next launch finds it
        }
        if (!__shfl_sync(0xffffffffu, last, 0)) continue;
        __threadfence();
        if (L::kFull && p.residual && c_first < p.N) fin.load_res(c_first, row0);
      }
      const float4* shares = reinterpret_cast<const float4*>(
          p.part + (static_cast<int64_t>(split ? w.share / p.splits * p.splits : 0) * (2 * kEpiWarps) + wslot) *
                       warp_floats);
      bool got = true;
#pragma unroll 1
      for (int c = 0; c < BN / 64; ++c) {
        const int col = c_first + c * 32;
        if (col >= p.N) break;
        float v[32];
        if (!split) {
          tmem_ld32(tbase + c * 32, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
#pragma unroll 1
          for (int s2 = 0; s2 < p.splits; s2 += 2) {   // two shares' loads in flight, added in order
            const int64_t share_f4 = (2 * kEpiWarps) * (warp_floats / 4);
            const float4* from = shares + s2 * share_f4 + c * 256 + lane;
            const bool two = s2 + 1 < p.splits;
            float4 o[2][8];
#pragma unroll
            for (int g = 0; g < 8; ++g) o[0][g] = __ldcg(from + g * 32);
#pragma unroll
            for (int g = 0; g < 8; ++g)
              o[1][g] = two ? __ldcg(from + share_f4 + g * 32) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int g = 0; g < 8; ++g) {
              v[g * 4 + 0] = (v[g * 4 + 0] + o[0][g].x) + o[1][g].x;
              v[g * 4 + 1] = (v[g * 4 + 1] + o[0][g].y) + o[1][g].y;
              v[g * 4 + 2] = (v[g * 4 + 2] + o[0][g].z) + o[1][g].z;
              v[g * 4 + 3] = (v[g * 4 + 3] + o[0][g].w) + o[1][g].w;
            }
          }
        }
        got = fin.finish(v, row0, col, c * 32, xs, c + 1 < BN / 64 && col + 32 < p.N ? col + 32 : -1);
        if (!got) break;
      }
      if (!got) break;
      if (!split) release_acc();
    }
    fin.close();
  }

  if (*abort_flag) {
    // give copies that may still be landing in shared memory time to finish
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
  tc_fence_before();
  cluster_sync_relaxed();   // the peer's shared memory and TMEM stay alive until the pair is done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, C::kTmemCols);
  }
}

// ============================================================================
// large tiles, all of them split: 256 x BN per cluster of `splits` CTA pairs
//
// For products with so few tiles that most pairs would idle: each pair of a cluster (2 or 4 pairs) reduces its
// share of the reduction blocks of one tile, spills it to its shared memory over the drained operand stages
// ([32-column chunk][4 columns][row], so that both ways move consecutive 16-byte groups), and after a cluster
// barrier each CTA joins and finishes BN / splits columns of its 128 rows, adding the shares in pair order.
// The epilogue is shared out with the join, so splitting costs no more than it saves there: 512 x 4096 x 4096 in
// 17.7 us against 23.8 us unsplit, with bias, SiLU, residual and z in 19.6 against 29.0.
// ============================================================================
template <int OP, int BN>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmPre,
                        const __grid_constant__ CUtensorMap tmRes, const LinParams p) {
  using C = PairCfg<OP, BN>;
  using L = LinLayout<OP>;
  static_assert(BN * 128 * 4 <= C::kStages * C::kStageBytes, "the partial tile fits the stages");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::kStages * C::kABytes;
  uint8_t* sEpi = sB + C::kStages * C::kBBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + C::kEpiBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint64_t* res_full = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + kEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1u, share = crank >> 1;   // CTA of the pair, pair of the cluster
  const uint32_t even = crank & ~1u;                      // the CTA that issues this pair's MMAs
  const int tile = static_cast<int>(blockIdx.x) / (2 * p.splits);
  const int mb = tile / p.n_tiles, t = tile - mb * p.n_tiles;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * share / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (share + 1) / p.splits);

  if (threadIdx.x == 64) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmOut);
    if (L::kFull && p.pre) tma_prefetch_desc(&tmPre);
    if (L::kFull && p.residual) tma_prefetch_desc(&tmRes);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&res_full[w], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, BN <= 128 ? 128u : 256u);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  pdl_wait();       // nothing above touches the tensors
  pdl_launch();
  clear_flags(p);
  const uint32_t tmem_base = *tmem_slot;
  const AbortState ab{abort_flag, p.flags};

  if (warp == 0 && lane == 0) {
    const int arow = mb * 256 + static_cast<int>(rank) * kBM;
    const int brow = t * BN + static_cast<int>(rank) * C::kCtaN;
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(&empty[stage], phase ^ 1u, ab)) break;
      uint8_t* a = sA + stage * C::kABytes;
      uint8_t* b = sB + stage * C::kBBytes;
      const uint32_t bar0 = mapa_shared(smem_u32(&full[stage]), even);
      if (rank == 0) mbar_arrive_expect_tx(&full[stage], C::kTxBytes);
      tma_load_2d_pair(a, &tmA, bar0, kb * L::kStepElems, arow);   // A is K-major in every split product
      if (C::kBmn) {
#pragma unroll
        for (int q = 0; q < C::kBAtoms; ++q) tma_load_2d_pair(b + q * 8192, &tmB, bar0, brow + q * 64, kb * 64);
      } else {
        tma_load_2d_pair(b, &tmB, bar0, kb * L::kStepElems, brow);
      }
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    const uint16_t both = static_cast<uint16_t>(3u << even);
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait(&full[stage], phase, ab)) break;
      tc_fence_after();
      const uint32_t a_addr = smem_u32(sA + stage * C::kABytes);
      const uint32_t b_addr = smem_u32(sB + stage * C::kBBytes);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t bd = C::kBmn ? sdesc_sw128(b_addr + j * 2048, 8192, 1024)
                                    : sdesc_sw128(b_addr + j * 32, 16, 1024);
        umma<L::kF8, true>(tmem_base, sdesc_sw128(a_addr + j * 32, 16, 1024), bd, C::kIdesc,
                           (kb != kb0 || j != 0) ? 1u : 0u);
      }
      umma_commit_pair(&empty[stage], both);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    umma_commit_pair(done, both);   // every MMA has finished, in both CTAs
  }
  __syncwarp();

  // Epilogue warps: their chunks are number first + half, + 2, ... of the CTA's [first, last).
  constexpr int kChunks = BN / 32;
  const int first = kChunks * static_cast<int>(share) / p.splits, last = kChunks * (static_cast<int>(share) + 1) / p.splits;
  const int q = warp & 3, half = (warp - 2) >> 2;
  const int row0 = mb * 256 + static_cast<int>(rank) * kBM + q * 32;
  uint8_t* wbuf = sEpi + (warp - 2) * C::kBufs * kStageBuf;
  const uint32_t side = smem_u32(sEpi + kEpiWarps * C::kBufs * kStageBuf + (warp - 2) * C::kSideBytes);
  Finisher<OP> fin{p,    &tmOut, &tmPre, &tmRes, wbuf, wbuf + 2 * kStageBuf, &res_full[warp - 2], side,
                   side + (BN / 2) * 4, lane, ab};
  float xs = 1.f;
  if (L::kFull && warp >= 2) {
    // at most BN / 64 chunks a warp: eight lanes each fetch the bias and scales of one
    const int mine = first + half + 2 * (lane >> 3);
    const int col = t * BN + mine * 32 + (lane & 7) * 4;
    if (mine < last && (lane >> 3) < BN / 64 && col < p.N) fin.load_side(col, lane * 4);
    if (L::kF8 && row0 + lane < p.M) xs = p.x_scale[row0 + lane];
    const int col0 = t * BN + (first + half) * 32;
    if (p.residual && first + half < last && col0 < p.N) fin.load_res(col0, row0);
    __syncwarp();
  }
  const bool good = mbar_wait(done, 0, ab) && !*abort_flag;
  tc_fence_after();
  // Every MMA has read its operands and every load was waited for by an MMA: the stages can be overwritten.
  if (warp >= 2 && good) {
    const uint32_t lane_addr = static_cast<uint32_t>(q * 32) << 16;
    float4* spill = reinterpret_cast<float4*>(smem) + q * 32 + lane;
#pragma unroll 1
    for (int c = half; c < kChunks; c += 2) {
      if (t * BN + c * 32 >= p.N) break;
      float v[32];
      tmem_ld32(tmem_base + lane_addr + c * 32, v);
      tmem_wait_ld();
#pragma unroll
      for (int g = 0; g < 8; ++g)
        spill[(c * 8 + g) * 128] = make_float4(v[g * 4], v[g * 4 + 1], v[g * 4 + 2], v[g * 4 + 3]);
    }
  }
  if (!good) {
    // giving up: copies and MMAs already issued get time to finish before shared memory is released
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kDrainLimitNs) {
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // every share is in shared memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, BN <= 128 ? 128u : 256u);
  }
  if (warp >= 2) {
    const uint32_t spill = smem_u32(smem) + static_cast<uint32_t>(q * 32 + lane) * 16u;
    int at = 0;
#pragma unroll 1
    for (int c = first + half; c < last && good; c += 2, at += 32) {
      const int col = t * BN + c * 32;
      if (col >= p.N) break;
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.f;
#pragma unroll 1
      for (int s = 0; s < p.splits; s += 2) {   // two shares' reads in flight, added in order
        const uint32_t from = spill + static_cast<uint32_t>(c) * 8u * 2048u;
        const uint32_t s0 = mapa_shared(from, static_cast<uint32_t>(2 * s) + rank);
        const uint32_t s1 = mapa_shared(from, static_cast<uint32_t>(2 * s + 2) + rank);
        float4 o[2][8];
#pragma unroll
        for (int g = 0; g < 8; ++g) o[0][g] = ld_cluster_v4f(s0 + g * 2048u);
#pragma unroll
        for (int g = 0; g < 8; ++g) o[1][g] = ld_cluster_v4f(s1 + g * 2048u);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          v[g * 4 + 0] = (v[g * 4 + 0] + o[0][g].x) + o[1][g].x;
          v[g * 4 + 1] = (v[g * 4 + 1] + o[0][g].y) + o[1][g].y;
          v[g * 4 + 2] = (v[g * 4 + 2] + o[0][g].z) + o[1][g].z;
          v[g * 4 + 3] = (v[g * 4 + 3] + o[0][g].w) + o[1][g].w;
        }
      }
      const int next = col + 64;
      if (!fin.finish(v, row0, col, at, xs, c + 2 < last && next < p.N ? next : -1)) break;
    }
    fin.close();
  }
  __syncwarp();
  cluster_sync_relaxed();   // this CTA's share stays readable until every peer has joined its columns
}

// ============================================================================
// small tiles: 128 output columns x NT rows per cluster, the reduction split over its CTAs
//
// A = 128 rows of W (for dx: 128 columns of W, MN-major), B = NT rows of x (or dz).  Each CTA reduces its
// share of the reduction blocks into a [128 x NT] TMEM tile, spills it to shared memory as [row][column]
// fp32, and after a cluster barrier each CTA joins and finishes 1 / splits of the tile: for every output it
// adds the partial sums in CTA order.  No workspace, no atomics, one launch.  Bound by HBM while the weights stream
// (1 x 4096 x 4096: 9,300 of 16,600 cycles), else by set-up, the first bytes' latency and the join; back to back
// with the weights from HBM 8.9 us (from L2 7.2), 8 rows in e4m3 6.6 us (6.0).
// ============================================================================
constexpr int kSmallThreads = 192;
constexpr int kMaxSplits = 8;
constexpr int kBatch = 2;

template <int OP, int NT>
struct SmallCfg {
  using L = LinLayout<OP>;
  static constexpr bool kAmn = OP == kLinDx;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kBBytes = NT * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // about 100 KB of stages, so that two CTAs share an SM and one's set-up and join hide under the other's loads
  static constexpr int kStages = NT <= 32 ? 5 : (NT == 64 ? 4 : 3);
  static constexpr int kTileBytes = NT * 128 * 4;           // the partial tile, over the drained stages
  static constexpr int kDataBytes = kStages * kStageBytes;
  static constexpr int kSmem = 1024 + kDataBytes + 256;
  static constexpr uint32_t kIdesc = L::kF8 ? idesc_e4m3_f32(128, NT) : idesc_bf16_f32(128, NT, kAmn, false);
  static constexpr uint32_t kTmemCols = NT < 32 ? 32u : static_cast<uint32_t>(NT);
  static_assert(kTileBytes <= kDataBytes, "the partial tile fits the stages");
  static_assert(NT % 16 == 0 && NT >= 16 && NT <= 128, "NT");
};

template <int OP, int NT>
__global__ void __launch_bounds__(kSmallThreads)
    linear_small_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const LinParams p) {
  using C = SmallCfg<OP, NT>;
  using L = LinLayout<OP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + C::kStages * C::kABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kDataBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile = static_cast<int>(blockIdx.x) / p.splits;
  const int row_tiles = (p.M + NT - 1) / NT;
  const int ct = tile / row_tiles, rt = tile - ct * row_tiles;   // row tiles of one column tile run together
  const int col0 = ct * 128, row0 = rt * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / p.splits);

  auto load = [&](int kb, int stage) {
    uint8_t* a = sA + stage * C::kABytes;
    mbar_arrive_expect_tx(&full[stage], C::kStageBytes);
    if (C::kAmn) {
      tma_load_2d(a, &tmA, &full[stage], col0, kb * 64);
      tma_load_2d(a + 8192, &tmA, &full[stage], col0 + 64, kb * 64);
    } else {
      tma_load_2d(a, &tmA, &full[stage], kb * L::kStepElems, col0);
    }
    tma_load_2d(sB + stage * C::kBBytes, &tmB, &full[stage], kb * L::kStepElems, row0);
  };
  if (threadIdx.x == 0) {
    // the loading thread sets up the barriers and fills the stages before it meets the others
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();   // nothing above touches the tensors
  pdl_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages && kb0 + s < kb1; ++s) load(kb0 + s, s);
    clear_flags(p);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const AbortState ab{abort_flag, p.flags};

  // This CTA's share of the tile: items are groups of four columns of a row, kBatch of a thread at a time.
  // What the first batch reads beside the product is fetched while the product runs.
  const int rows = min(NT, p.M - row0);
  const int items = rows * 32;
  const int i0 = static_cast<int>(static_cast<int64_t>(items) * rank / p.splits);
  const int i1 = static_cast<int>(static_cast<int64_t>(items) * (rank + 1) / p.splits);
  struct Side {
    uint2 res, bias;
    float4 ws;
    float xs;
  };
  auto load_side = [&](int i, Side& d) {
    const int row = row0 + (i >> 5), col = col0 + (i & 31) * 4;
    d.res = d.bias = make_uint2(0u, 0u);
    d.xs = 1.f;
    if (!L::kFull || i >= i1 || col >= p.N || !dbg_ok(row < p.M && col + 4 <= p.N, p.flags)) return;
    if (p.residual) d.res = *reinterpret_cast<const uint2*>(p.residual + static_cast<int64_t>(row) * p.N + col);
    if (p.bias) d.bias = *reinterpret_cast<const uint2*>(p.bias + col);
    if (L::kF8) {
      d.xs = p.x_scale[row];
      d.ws = *reinterpret_cast<const float4*>(p.w_scale + col);
    }
  };
  Side side[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) load_side(i0 + static_cast<int>(threadIdx.x) + b * kSmallThreads, side[b]);

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 1;
      for (int kb = kb0 + C::kStages; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, ab)) break;
        load(kb, stage);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase, ab)) break;
        tc_fence_after();
        const uint32_t a_addr = smem_u32(sA + stage * C::kABytes);
        const uint32_t b_addr = smem_u32(sB + stage * C::kBBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t ad = C::kAmn ? sdesc_sw128(a_addr + j * 2048, 8192, 1024)
                                      : sdesc_sw128(a_addr + j * 32, 16, 1024);
          umma<L::kF8, false>(tmem_base, ad, sdesc_sw128(b_addr + j * 32, 16, 1024), C::kIdesc,
                              (kb != kb0 || j != 0) ? 1u : 0u);
        }
        umma_commit(&empty[stage]);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      umma_commit(done);
    }
    __syncwarp();
  }
  // Every MMA has read its operands once `done` completes, and every load was waited for by an MMA, so
  // the stages can be overwritten (on the abort path copies may still be landing: nothing is written).
  const bool good = mbar_wait(done, 0, ab) && !*abort_flag;
  tc_fence_after();
  float* part = reinterpret_cast<float*>(smem);   // [NT][128]
  if (warp >= 2 && good) {
    const int f = (warp & 3) * 32 + lane;         // output column of this thread's TMEM lane
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll 1
    for (int j0 = 0; j0 < NT; j0 += 16) {
      if (row0 + j0 >= p.M) break;
      float v[16];
      tmem_ld16(tbase + j0, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) part[(j0 + j) * 128 + f] = v[j];
    }
  }
  if (!good) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < kDrainLimitNs) {
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
  if (good) {
    const uint32_t base = smem_u32(part);
    for (int first = i0 + static_cast<int>(threadIdx.x); first < i1; first += kBatch * kSmallThreads) {
      float4 q[kBatch][kMaxSplits];   // all partial sums of the batch are in flight before the first is added
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        // only what is used below is read: its use orders the reads before the closing barrier
        const int i = first + b * kSmallThreads;
        const bool live = i < i1 && col0 + (i & 31) * 4 < p.N;
#pragma unroll
        for (int s = 0; s < kMaxSplits; ++s)
          if (s < p.splits && live)
            q[b][s] = ld_cluster_v4f(mapa_shared(base + static_cast<uint32_t>(i) * 16u, s));
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = first + b * kSmallThreads;
        const int row = row0 + (i >> 5), col = col0 + (i & 31) * 4;
        if (i >= i1 || col >= p.N || !dbg_ok(row < p.M && col + 4 <= p.N, p.flags)) continue;
        const int64_t at = static_cast<int64_t>(row) * p.N + col;
        float v[4] = {q[b][0].x, q[b][0].y, q[b][0].z, q[b][0].w};
#pragma unroll
        for (int s = 1; s < kMaxSplits; ++s)
          if (s < p.splits) {
            v[0] += q[b][s].x;
            v[1] += q[b][s].y;
            v[2] += q[b][s].z;
            v[3] += q[b][s].w;
          }
        if (L::kFull) {
          const Side& d = side[b];
          if (L::kF8) {
            v[0] *= d.xs * d.ws.x;
            v[1] *= d.xs * d.ws.y;
            v[2] *= d.xs * d.ws.z;
            v[3] *= d.xs * d.ws.w;
          }
          if (p.bias) v[0] += bf_lo(d.bias.x), v[1] += bf_hi(d.bias.x), v[2] += bf_lo(d.bias.y), v[3] += bf_hi(d.bias.y);
          if (p.pre)
            *reinterpret_cast<uint2*>(p.pre + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          act_all(v, p.act);
          if (p.residual) v[0] += bf_lo(d.res.x), v[1] += bf_hi(d.res.x), v[2] += bf_lo(d.res.y), v[3] += bf_hi(d.res.y);
        }
        *reinterpret_cast<uint2*>(p.out + at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) load_side(first + (kBatch + b) * kSmallThreads, side[b]);
    }
  }
  __syncwarp();
  cluster_sync_relaxed();   // this CTA's partial tile stays readable until every peer has joined its share
}

// ============================================================================
// dz = dy act'(pre), bf16, and the column sums of its fp32 values
//
// One block: 256 columns (8 per thread) x a range of rows, eight rows at a time.  Bound by HBM where dz is
// written: 16384 x 4096 with SiLU in 65 us, 6.2 TB/s, with the column sums 70 us; the column sums alone, which write
// nothing, by the slopes' arithmetic: 56 us, 4.8 TB/s (GELU 67 us).
// ============================================================================
constexpr int kActRows = 8;

template <int ACT>
__global__ void __launch_bounds__(32 * kActRows)
    act_grad_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ pre, int64_t M, int n,
                    uint16_t* __restrict__ dz, float* __restrict__ part, int64_t part_floats,
                    uint32_t* __restrict__ tickets, float* __restrict__ dbias, uint32_t* __restrict__ flags) {
  __shared__ float s[kActRows][32][9];
  __shared__ int s_last;
  pdl_wait();
  pdl_launch();
  const int col = (static_cast<int>(blockIdx.x) * 32 + static_cast<int>(threadIdx.x)) * 8;
  const int64_t r0 = M * blockIdx.y / gridDim.y, r1 = M * (blockIdx.y + 1) / gridDim.y;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  if (col < n) {
    constexpr int kU = 2;   // rows whose loads are in flight together
    int64_t r = r0 + threadIdx.y;
    for (; r < r1; r += kU * kActRows) {
      uint4 g[kU], z[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int64_t at = (r + u * kActRows) * n + col;
        if (r + u * kActRows < r1) {
          if (!dbg_ok(r1 <= M && at >= 0 && col + 8 <= n, flags)) return;
          g[u] = ld_stream16(dy + at);
          if (ACT != KDKL_ACT_NONE) z[u] = ld_stream16(pre + at);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (r + u * kActRows >= r1) break;
        float v[8] = {bf_lo(g[u].x), bf_hi(g[u].x), bf_lo(g[u].y), bf_hi(g[u].y),
                      bf_lo(g[u].z), bf_hi(g[u].z), bf_lo(g[u].w), bf_hi(g[u].w)};
        if (ACT != KDKL_ACT_NONE) {
          const float w[8] = {bf_lo(z[u].x), bf_hi(z[u].x), bf_lo(z[u].y), bf_hi(z[u].y),
                              bf_lo(z[u].z), bf_hi(z[u].z), bf_lo(z[u].w), bf_hi(z[u].w)};
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], act_grad_f<ACT>(w[j]));   // the same sums with and without dz
          if (dz)
            *reinterpret_cast<uint4*>(dz + (r + u * kActRows) * n + col) =
                make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                           pack_bf16x2(v[6], v[7]));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += v[j];
      }
    }
  }
  if (!dbias) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) s[threadIdx.y][threadIdx.x][j] = acc[j];
  __syncthreads();
  const int c = static_cast<int>(threadIdx.y) * 32 + static_cast<int>(threadIdx.x);   // one column each
  const int out = static_cast<int>(blockIdx.x) * 256 + c;
  auto column = [&] {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < kActRows; ++r) t += s[r][c >> 3][c & 7];
    return t;
  };
  if (!dbg_ok(static_cast<int64_t>(gridDim.y) * n <= part_floats, flags)) return;
  if (out < n) part[static_cast<int64_t>(blockIdx.y) * n + out] = column();
  // The block that finishes these columns last adds up the partial sums of all row ranges, in their order:
  // the result does not depend on which block that is.
  __threadfence();
  __syncthreads();
  if (c == 0) s_last = atomicAdd(&tickets[blockIdx.x], 1u) == gridDim.y - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  if (col < n) {
#pragma unroll 8
    for (int r = threadIdx.y; r < static_cast<int>(gridDim.y); r += kActRows) {
      const float4* q = reinterpret_cast<const float4*>(part + static_cast<int64_t>(r) * n + col);
      const float4 u = __ldcg(q), w = __ldcg(q + 1);
      acc[0] += u.x, acc[1] += u.y, acc[2] += u.z, acc[3] += u.w;
      acc[4] += w.x, acc[5] += w.y, acc[6] += w.z, acc[7] += w.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) s[threadIdx.y][threadIdx.x][j] = acc[j];
  __syncthreads();
  if (out < n) dbias[out] = column();
}

// Sets a kernel's dynamic shared-memory limit on its first launch on each device (devices past the 64th:
// on every launch).
template <class K>
cudaError_t configure(K* kernel, int smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int OP, int BN>
cudaError_t pair_one(const PairMaps& m, const LinParams& p, int grid, cudaStream_t s) {
  using C = PairCfg<OP, BN>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = configure(linear_pair_kernel<OP, BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const LaunchConfig cfg(dim3(grid), dim3(kPairThreads), C::kSmem, 2, s);
  return cudaLaunchKernelEx(&cfg.c, linear_pair_kernel<OP, BN>, m.a, m.b, m.out, m.pre, m.res, p);
}

template <int OP, int BN>
cudaError_t split_one(const PairMaps& m, const LinParams& p, cudaStream_t s) {
  using C = PairCfg<OP, BN>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = configure(linear_split_kernel<OP, BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const LaunchConfig cfg(dim3(p.tiles * 2 * p.splits), dim3(kPairThreads), C::kSmem, 2 * p.splits, s);
  return cudaLaunchKernelEx(&cfg.c, linear_split_kernel<OP, BN>, m.a, m.b, m.out, m.pre, m.res, p);
}

template <int OP>
cudaError_t split_op(int bn, const PairMaps& m, const LinParams& p, cudaStream_t s) {
  switch (bn) {
    case 256: return split_one<OP, 256>(m, p, s);
    case 192: return split_one<OP, 192>(m, p, s);
    case 128: return split_one<OP, 128>(m, p, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int OP>
cudaError_t pair_op(int bn, const PairMaps& m, const LinParams& p, int grid, cudaStream_t s) {
  switch (bn) {
    case 256: return pair_one<OP, 256>(m, p, grid, s);
    case 192: return pair_one<OP, 192>(m, p, grid, s);
    case 128: return pair_one<OP, 128>(m, p, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

template <int OP, int NT>
cudaError_t small_one(const CUtensorMap& tmA, const CUtensorMap& tmB, const LinParams& p, cudaStream_t s) {
  using C = SmallCfg<OP, NT>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = configure(linear_small_kernel<OP, NT>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>((p.N + 127) / 128) * ((p.M + NT - 1) / NT);
  const LaunchConfig cfg(dim3(static_cast<unsigned>(tiles * p.splits)), dim3(kSmallThreads), C::kSmem, p.splits, s);
  return cudaLaunchKernelEx(&cfg.c, linear_small_kernel<OP, NT>, tmA, tmB, p);
}

template <int OP>
cudaError_t small_op(int nt, const CUtensorMap& tmA, const CUtensorMap& tmB, const LinParams& p, cudaStream_t s) {
  switch (nt) {
    case 16: return small_one<OP, 16>(tmA, tmB, p, s);
    case 32: return small_one<OP, 32>(tmA, tmB, p, s);
    case 64: return small_one<OP, 64>(tmA, tmB, p, s);
    case 128: return small_one<OP, 128>(tmA, tmB, p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_linear_pair(int op, int bn, const PairMaps& m, const LinParams& p, int grid, cudaStream_t s) {
  switch (op) {
    case kLinFwd: return pair_op<kLinFwd>(bn, m, p, grid, s);
    case kLinFwdE4M3: return pair_op<kLinFwdE4M3>(bn, m, p, grid, s);
    case kLinDx: return pair_op<kLinDx>(bn, m, p, grid, s);
    case kLinDw: return pair_op<kLinDw>(bn, m, p, grid, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_linear_split(int op, int bn, const PairMaps& m, const LinParams& p, cudaStream_t s) {
  switch (op) {
    case kLinFwd: return split_op<kLinFwd>(bn, m, p, s);
    case kLinFwdE4M3: return split_op<kLinFwdE4M3>(bn, m, p, s);
    case kLinDx: return split_op<kLinDx>(bn, m, p, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_linear_small(int op, int nt, const CUtensorMap& tmA, const CUtensorMap& tmB, const LinParams& p,
                                cudaStream_t s) {
  switch (op) {
    case kLinFwd: return small_op<kLinFwd>(nt, tmA, tmB, p, s);
    case kLinFwdE4M3: return small_op<kLinFwdE4M3>(nt, tmA, tmB, p, s);
    case kLinDx: return small_op<kLinDx>(nt, tmA, tmB, p, s);
    default: return cudaErrorInvalidValue;
  }
}

int act_grad_chunks(int64_t M, int n, int sms) {
  const int64_t cols = (n + 255) / 256;
  const int64_t want = (8 * static_cast<int64_t>(sms) + cols - 1) / cols;   // about eight blocks per SM
  const int64_t most = (M + 4 * kActRows - 1) / (4 * kActRows);              // each with rows for all its threads
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({want, most, kMaxActChunks})));
}

cudaError_t launch_act_grad(const uint16_t* dy, const uint16_t* pre, int act, int64_t M, int n, uint16_t* dz,
                            float* part, int64_t part_floats, uint32_t* tickets, float* dbias, uint32_t* flags,
                            int chunks, cudaStream_t s) {
  const LaunchConfig cfg(dim3((n + 255) / 256, chunks), dim3(32, kActRows), 0, 0, s);
  const auto launch = [&](auto* kernel) {
    return cudaLaunchKernelEx(&cfg.c, kernel, dy, pre, M, n, dz, part, part_floats, tickets, dbias, flags);
  };
  switch (act) {
    case KDKL_ACT_NONE: return launch(act_grad_kernel<KDKL_ACT_NONE>);
    case KDKL_ACT_RELU: return launch(act_grad_kernel<KDKL_ACT_RELU>);
    case KDKL_ACT_GELU: return launch(act_grad_kernel<KDKL_ACT_GELU>);
    case KDKL_ACT_GELU_TANH: return launch(act_grad_kernel<KDKL_ACT_GELU_TANH>);
    case KDKL_ACT_SILU: return launch(act_grad_kernel<KDKL_ACT_SILU>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kdkl
