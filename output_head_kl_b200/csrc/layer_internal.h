// Internal declarations of the operators ahead of the output head (RMS norm and linear layer):
// launchers defined in norm.cu and linear.cu, called by layer_api.cu.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace kdkl {

// ---------------------------------------------------------------- RMS norm (norm.cu)
// A row is held in the registers of one warp or one block, kNormVec elements per thread and step.
constexpr int kNormVec = 8;
constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxD = kNormMaxThreads * kNormVec * 8;   // 8 steps of kNormVec elements per thread
// Blocks of the gradient kernel, each leaving one row of partial sums for dgamma.
constexpr int kNormGradBlocks = 1184;

struct NormParams {
  const void* x;
  const void* residual;   // may be null
  const void* gamma;
  void* h;                // may be null
  void* y;
  float* y_scale;         // e4m3 output only
  int64_t N;
  int d;
  float eps;
  bool x_f32, h_f32, gamma_f32, y_e4m3;
};
cudaError_t launch_rmsnorm(const NormParams& p, int sms, cudaStream_t s);

struct NormGradParams {
  const void* dy;         // bf16
  const void* h;
  const void* gamma;
  const void* dh;         // may be null
  void* dx;
  float* part;            // [blocks, d]
  int64_t N;
  int d;
  float eps;
  bool h_f32, gamma_f32;
};
// Returns the blocks (rows of `part`) it used; *err is its launch's status.
int launch_rmsnorm_grad(const NormGradParams& p, int sms, cudaStream_t s, cudaError_t* err);

// out[c] = sum over rows of part[rows, n], in a fixed order.
cudaError_t launch_colsum(const float* part, int rows, int n, float* out, cudaStream_t s);

// ---------------------------------------------------------------- linear layer (linear.cu)
// Operand layouts and epilogues of the products:
//   kLinFwd     y = act(x W^T + b) + r, bf16      A = x K-major,   B = W K-major
//   kLinFwdE4M3 the same from e4m3 operands       A = x K-major,   B = W K-major
//   kLinDx      dx = dz W                         A = dz K-major,  B = W MN-major
//   kLinDw      dW = dz^T x                       A = dz MN-major, B = x MN-major
enum LinOp { kLinFwd = 0, kLinFwdE4M3 = 1, kLinDx = 2, kLinDw = 3 };

struct LinParams {
  int M;                 // rows of the output
  int N;                 // columns of the output
  int k_blocks;          // 128-byte reduction blocks (dz and x as MN-major operands: 64 rows)
  int tiles;             // large tiles: output tiles, of which
  int full_units;        //   the first full_units are computed whole and the others in `splits` shares;
  int units;             //   units of work in all
  int n_tiles;           //   tiles along N
  int row_group;         //   row blocks swept together
  int splits;            // shares of the reduction (small tiles: the cluster size)
  float* part;           // large tiles: [shares][256 x bn] partial sums
  int64_t part_floats;   //   room for them
  uint32_t* tickets;     //   [split tiles][16] arrivals, zero before the launch and after it
  const uint16_t* bias;      // [N] bf16 or null
  const uint16_t* residual;  // [M, N] bf16 or null
  const float* x_scale;      // [M] or null
  const float* w_scale;      // [N] or null
  uint16_t* out;         // [M, N] bf16 (small tiles; large tiles store through a tensor map)
  uint16_t* pre;         // [M, N] bf16 or null
  int act;
  uint32_t* flags;       // device flag word
  int clear_flags;       // the first block zeroes the flag word
};

constexpr int kTileTickets = 16;   // epilogue warps of a CTA pair
// Shares of split tiles that a launch of large tiles may have (a wave of CTA pairs has 74 on B200; each leaves
// 256 x bn fp32 partial sums), and the tiles that have two at least.
constexpr int kMaxShares = 80;
constexpr int kMaxSplitTiles = kMaxShares / 2;
// Large tiles: 256 x bn (bn = 256, 192 or 128) by CTA pairs, persistent.
struct PairMaps {
  CUtensorMap a, b;           // operands
  CUtensorMap out, pre, res;  // 32 x 32 boxes of y, z and the residual (unused ones repeat `out`)
};
cudaError_t launch_linear_pair(int op, int bn, const PairMaps& m, const LinParams& p, int grid, cudaStream_t s);
// The same tiles, each shared by a cluster of p.splits (2 or 4) pairs that split its reduction; all but kLinDw.
cudaError_t launch_linear_split(int op, int bn, const PairMaps& m, const LinParams& p, cudaStream_t s);
// Small tiles: 128 output columns x nt rows (nt = 16, 32, 64 or 128) per cluster of p.splits CTAs; the
// roles of the operands are swapped (tmA reads W, tmB reads x or dz).  op: all but kLinDw.
cudaError_t launch_linear_small(int op, int nt, const CUtensorMap& tmA, const CUtensorMap& tmB, const LinParams& p,
                                cudaStream_t s);

// dz = dy * act'(pre) in bf16 (dz may be null: column sums only, of dy when act is none) and, with dbias, the
// column sums of its fp32 values, by way of part[chunks, n] and one ticket per 256 columns (zero before).  flags is
// written by the bounds-checking build only.
constexpr int kMaxSms = 512;         // workspaces are sized for any device up to this many SMs
constexpr int kMaxActChunks = 256;   // row ranges that the last block of a column range adds up
int act_grad_chunks(int64_t M, int n, int sms);
cudaError_t launch_act_grad(const uint16_t* dy, const uint16_t* pre, int act, int64_t M, int n, uint16_t* dz,
                            float* part, int64_t part_floats, uint32_t* tickets, float* dbias, uint32_t* flags,
                            int chunks, cudaStream_t s);

// Launch configuration of these kernels: all of them wait for the kernels before them by themselves
// (pdl_wait), so that their set-up overlaps the end of the one before.
struct LaunchConfig {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t c;
  LaunchConfig(dim3 grid, dim3 block, int smem, int cluster, cudaStream_t s) : attr{}, c{} {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = static_cast<size_t>(smem);
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = cluster > 0 ? 2 : 1;
  }
  LaunchConfig(const LaunchConfig&) = delete;
};

}  // namespace kdkl
