// C ABI of the operators ahead of the output head (RMS norm, linear layer): argument checks, tile
// planner, TMA descriptors and launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "../../include/kdkl.h"
#include "host_util.h"
#include "kdkl_internal.h"
#include "layer_internal.h"

namespace kdkl {
namespace {

constexpr int32_t kMaxWidth = 1 << 20;
constexpr size_t kFlagBytes = 256;
constexpr int kMaxTailSplits = 8;
constexpr size_t kTicketBytes = kMaxSplitTiles * kTileTickets * 4;

bool float_dtype(int32_t t) { return t == KDKL_BF16 || t == KDKL_F32; }

// ---------------------------------------------------------------- RMS norm
kdkl_status check_norm(int64_t N, int32_t d, float eps, int32_t h_dtype, int32_t gamma_dtype) {
  if (N < 0 || N > kMaxRows) return fail(KDKL_ERR_SHAPE, "N=%lld outside [0, %lld]", (long long)N, (long long)kMaxRows);
  if (d < 8 || d % 8 != 0) return fail(KDKL_ERR_SHAPE, "d=%d must be a positive multiple of 8", d);
  if (d > kNormMaxD) return fail(KDKL_ERR_UNSUPPORTED, "d=%d above %d", d, kNormMaxD);
  if (!std::isfinite(eps) || eps < 0.f) return fail(KDKL_ERR_SHAPE, "eps must be finite and >= 0");
  if (!float_dtype(h_dtype) || !float_dtype(gamma_dtype))
    return fail(KDKL_ERR_UNSUPPORTED, "h and gamma must be KDKL_BF16 or KDKL_F32");
  return KDKL_OK;
}

size_t norm_part_bytes(int64_t N, int32_t d) {
  const int64_t rows = std::max<int64_t>(1, std::min<int64_t>(N, kNormGradBlocks));
  return align_up(static_cast<size_t>(rows) * d * 4, 256);
}

// ---------------------------------------------------------------- linear layer
struct Plan {
  bool pair = true;
  int tile = 256;    // pair: columns of a tile; small: rows of a tile
  int splits = 1;    // pair: shares of each tile of the last wave; small: CTAs of a cluster
  int code() const { return pair ? tile + (splits > 1 ? 10000 * splits : 0) : splits * 1000 + tile; }
};

// Tiles of the last, partly filled wave of large tiles (0 when every wave is full).
int64_t tail_tiles(int64_t tiles, int sms) { return tiles % (sms / 2); }

// Clusters of 4 or 8 CTAs with an SM each that run at once: a cluster stays within one GPC, so some SMs are
// left over (B200, 148 SMs: 33 and 15 were found resident; one less is counted on).
int64_t cluster_slots(int sms, int ctas) { return static_cast<int64_t>(ctas == 4 ? 32 : 14) * sms / 148; }

// Whether a product's tiles, if they are split, are split by clusters, without the workspace: those of fewer
// tiles than a wave (of a B200's 74 pairs; on any device, so that the workspace's size does not depend on it).
constexpr int kWaveTiles = 74;
bool split_by_cluster(LinOp op, int64_t tiles) { return op != kLinDw && tiles < kWaveTiles; }

// Whether the tiles of the last wave can each be split into `sp` shares of the reduction: all shares run at
// once and keep at least four reduction blocks.  Where there is no full wave, a cluster of 2 or 4 pairs shares
// each tile (dW: any number of shares, by way of the workspace, as after full waves).
bool can_split(LinOp op, int64_t tiles, int k_blocks, int sms, int sp) {
  const int64_t tail = tail_tiles(tiles, sms);
  if (sp < 2 || sp > kMaxTailSplits || tail == 0 || k_blocks / sp < 4) return false;
  if (split_by_cluster(op, tiles)) return (sp == 2 || sp == 4) && tiles <= cluster_slots(sms, 2 * sp);
  return tail * sp <= std::min<int64_t>(sms / 2, kMaxShares);
}

// Product out[rows, cols] with `k_blocks` reduction blocks.
//
// Cost model in microseconds; its constants are a fit to the measured times of every plan of the forward at
// 196 sizes (rows 1 to 4096, widths 256 to 8192, bf16 and e4m3): there the plan it picks is 1.5 % slower than
// the fastest one on average and 22 % at worst.
//   pair tiles:  launch + last epilogue + per tile of a pair: kb[bn] per reduction block (a 256-wide
//                tile's two operands fill what an SM can take in from L2, so narrower ones cost nearly as
//                much) and the epilogue's share.  Splitting the last wave's tiles costs their join by way of the
//                workspace; a cluster's join shares out the epilogue and saves some of it.
//   small tiles: launch, join and, per wave of two CTAs an SM, kb + kb_row per row of the tile.
Plan plan_linear(LinOp op, int64_t rows, int64_t cols, int k_blocks, int sms) {
  Plan best;
  double lo = 1e300;
  const int pairs = sms / 2;
  const int64_t rb = (rows + 255) / 256;
  for (int bn : {256, 192, 128}) {
    const double kb = bn == 256 ? 0.321 : (bn == 192 ? 0.277 : 0.237);
    const double width = bn / 256.0;
    const int64_t tiles = rb * ((cols + bn - 1) / bn);
    const int64_t tail = tail_tiles(tiles, sms), full = tiles / pairs;
    for (int sp = 1; sp <= kMaxTailSplits; ++sp) {
      if (sp > 1 && !can_split(op, tiles, k_blocks, sms, sp)) continue;
      double t = 3.26 + 5.72 * width + static_cast<double>(full) * (k_blocks * kb + 0.441 * width);
      if (tail) t += (k_blocks + sp - 1) / sp * kb + (full ? 0.441 * width : 0.0);
      if (sp > 1) t += split_by_cluster(op, tiles) ? 1.85 - 3.13 * width : 9.74 + 0.488 * sp;
      if (t < lo) {
        lo = t;
        best = Plan{true, bn, sp};
      }
    }
  }
  if (op == kLinDw) return best;
  for (int nt : {16, 32, 64, 128}) {
    const int64_t tiles = ((cols + 127) / 128) * ((rows + nt - 1) / nt);
    for (int sp : {1, 2, 4, 8}) {
      const int64_t ctas = tiles * sp;
      if (sp > k_blocks || ctas > INT_MAX / 2) break;
      // CTAs that run at once, two an SM as far as clusters fit the GPCs (71 of 4 and 33 of 8 on B200)
      const int64_t slots = static_cast<int64_t>(sp == 8 ? 264 : (sp == 4 ? 284 : 296)) * sms / 148;
      const int64_t waves = (ctas + slots - 1) / slots;
      const double share = ctas <= sms ? 1.0 : (waves == 1 ? 1.27 : 2.0);   // two CTAs share an SM's intake
      const double block = (0.182 + 0.0818 * nt / 64) * share;
      const double t = 4.8 + 0.118 * sp + 2.19 * nt / (64.0 * sp) +
                       static_cast<double>(waves) * ((k_blocks + sp - 1) / sp * block + 0.527);
      if (t < lo) {
        lo = t;
        best = Plan{false, nt, sp};
      }
    }
  }
  return best;
}

// A plan code of the caller's; false when the product has no such plan.
bool decode_plan(int32_t code, LinOp op, int64_t rows, int64_t cols, int k_blocks, int sms, Plan& p) {
  const int bn = code % 10000;
  if (code > 0 && (bn == 128 || bn == 192 || bn == 256)) {
    const int sp = code / 10000;
    p = Plan{true, bn, sp == 0 ? 1 : sp};
    const int64_t tiles = ((rows + 255) / 256) * ((cols + bn - 1) / bn);
    return sp == 0 || can_split(op, tiles, k_blocks, sms, sp);
  }
  if (op == kLinDw || code < 1000) return false;
  const int sp = code / 1000, nt = code % 1000;
  if (sp != 1 && sp != 2 && sp != 4 && sp != 8) return false;
  if (nt != 16 && nt != 32 && nt != 64 && nt != 128) return false;
  if (sp > k_blocks) return false;
  p = Plan{false, nt, sp};
  return true;
}

kdkl_status check_linear_shape(int64_t M, int32_t d_in, int32_t d_out, int32_t operands) {
  if (operands != KDKL_BF16 && operands != KDKL_E4M3)
    return fail(KDKL_ERR_UNSUPPORTED, "operands must be KDKL_BF16 or KDKL_E4M3");
  if (M < 0 || M > kMaxRows) return fail(KDKL_ERR_SHAPE, "M=%lld outside [0, %lld]", (long long)M, (long long)kMaxRows);
  const int step = operands == KDKL_E4M3 ? 16 : 8;
  if (d_in < step || d_in % step != 0) return fail(KDKL_ERR_SHAPE, "d_in=%d must be a positive multiple of %d", d_in, step);
  if (d_out < 8 || d_out % 8 != 0) return fail(KDKL_ERR_SHAPE, "d_out=%d must be a positive multiple of 8", d_out);
  if (d_in > kMaxWidth || d_out > kMaxWidth) return fail(KDKL_ERR_UNSUPPORTED, "d_in=%d, d_out=%d above %d", d_in, d_out, kMaxWidth);
  // output tiles are counted in 32 bits (the smallest tiles: 16 rows x 128 columns, up to 8 CTAs each,
  // are only planned within it); the large tiles set the limit
  const int64_t rb = (M + 255) / 256;
  if (rb * ((std::max(d_in, d_out) + 127) / 128) > INT_MAX / 2)
    return fail(KDKL_ERR_UNSUPPORTED, "M=%lld with d_in=%d, d_out=%d has too many output tiles", (long long)M, d_in, d_out);
  return KDKL_OK;
}

kdkl_linear_options default_linear_options() {
  kdkl_linear_options o;
  std::memset(&o, 0, sizeof(o));
  o.operands = KDKL_BF16;
  o.activation = KDKL_ACT_NONE;
  return o;
}

struct LinearLayout {
  size_t tickets = 0, col_tickets = 0, shares = 0, share_bytes = 0, dz = 0, part = 0, total = 0;
};

// Bytes of the partial sums that a product out[rows, cols] may split its last wave into: the most of any tile
// width.  Neither the narrowest nor the widest tiles need the most everywhere: 385 to 512 columns are two tiles of
// 256 but three of 192, whose shares are larger in all.
size_t share_bytes(LinOp op, int64_t rows, int64_t cols) {
  size_t most = 0;
  for (int bn : {256, 192, 128}) {
    const int64_t tiles = ((rows + 255) / 256) * ((cols + bn - 1) / bn);
    if (split_by_cluster(op, tiles)) continue;
    const int64_t shares = std::min<int64_t>(kMaxShares, tiles * kMaxTailSplits);   // as can_split allows
    most = std::max(most, static_cast<size_t>(shares) * 256 * bn * 4);
  }
  return most;
}

// Workspace: the flag word and the tickets (everything before `shares` is cleared ahead of the launches that
// use it), the partial sums of split tiles; for the gradient also dz and the partial column sums of the most
// blocks act_grad runs.
LinearLayout linear_layout(int64_t M, int32_t d_in, int32_t d_out, bool backward) {
  LinearLayout L;
  L.tickets = kFlagBytes;
  L.col_tickets = L.tickets + kTicketBytes;
  L.shares = align_up(L.col_tickets + (backward ? static_cast<size_t>((d_out + 255) / 256) * 4 : 0), 256);
  L.share_bytes = backward ? std::max(share_bytes(kLinDx, M, d_in), share_bytes(kLinDw, d_out, d_in))
                           : share_bytes(kLinFwd, M, d_out);
  size_t off = L.shares + L.share_bytes;
  if (backward) {
    L.dz = off;
    off = align_up(off + static_cast<size_t>(M) * d_out * 2, 256);
    L.part = off;
    off = align_up(off + static_cast<size_t>(act_grad_chunks(M, d_out, kMaxSms)) * d_out * 4, 256);
  }
  L.total = off;
  return L;
}

int reduction_blocks(int32_t len, bool f8) { return (len + (f8 ? 127 : 63)) / (f8 ? 128 : 64); }

// One product: out[rows, cols] (bf16) of `op`'s operands a [rows or reduction] and b.
//   kLinFwd(E4M3): a = x [rows, len], b = W [cols, len]
//   kLinDx:        a = dz [rows, len], b = W [len, cols]
//   kLinDw:        a = dz [len, rows], b = x [len, cols]
cudaError_t run_product(LinOp op, const Plan& plan, const void* a, const void* b, int64_t rows, int64_t cols,
                        int64_t len, LinParams p, int sms, cudaStream_t s) {
  const bool f8 = op == kLinFwdE4M3;
  const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
  p.M = static_cast<int>(rows);
  p.N = static_cast<int>(cols);
  p.k_blocks = reduction_blocks(static_cast<int32_t>(len), f8);
  p.splits = plan.splits;
  bool made;
  if (plan.pair) {
    PairMaps m;
    const int bn = plan.tile;
    if (f8)
      made = make_map_u8(&m.a, a, len, rows, len, 128, kBM, sw) && make_map_u8(&m.b, b, len, cols, len, 128, bn / 2, sw);
    else if (op == kLinFwd)
      made = make_map(&m.a, a, len, rows, len, 64, kBM, sw) && make_map(&m.b, b, len, cols, len, 64, bn / 2, sw);
    else if (op == kLinDx)
      made = make_map(&m.a, a, len, rows, len, 64, kBM, sw) && make_map(&m.b, b, cols, len, cols, 64, 64, sw);
    else
      made = make_map(&m.a, a, rows, len, rows, 64, 64, sw) && make_map(&m.b, b, cols, len, cols, 64, 64, sw);
    const auto box = [&](CUtensorMap* map, const void* base) {
      return make_map(map, base, cols, rows, cols, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    };
    made = made && box(&m.out, p.out);
    if (!made) return cudaErrorInvalidValue;
    m.pre = m.res = m.out;
    if ((p.pre && !box(&m.pre, p.pre)) || (p.residual && !box(&m.res, p.residual))) return cudaErrorInvalidValue;
    p.n_tiles = static_cast<int>((cols + bn - 1) / bn);
    p.tiles = static_cast<int>((rows + 255) / 256) * p.n_tiles;
    if (plan.splits > 1 && split_by_cluster(op, p.tiles)) return launch_linear_split(op, bn, m, p, s);
    const int tail = plan.splits > 1 ? static_cast<int>(tail_tiles(p.tiles, sms)) : 0;
    p.full_units = p.tiles - tail;
    p.units = p.full_units + tail * plan.splits;
    if (static_cast<int64_t>(tail) * plan.splits * 256 * bn > p.part_floats) return cudaErrorInvalidValue;
    // When B (the weights, or x for dW) stays in L2, two row blocks at a time read A once while it is
    // hot: 412 against 424 us for 16384 x 4096 x 4096 at a steady clock; a B beyond L2 is swept for
    // eight row blocks at a time.
    p.row_group = static_cast<double>(cols) * len * (f8 ? 1 : 2) <= 48e6 ? 2 : 8;
    const int groups = std::min(p.units, sms / 2);
    return launch_linear_pair(op, bn, m, p, 2 * groups, s);
  }
  // small tiles: the weights take the MMA's M side
  CUtensorMap tmA, tmB;
  const int nt = plan.tile;
  if (f8)
    made = make_map_u8(&tmA, b, len, cols, len, 128, 128, sw) && make_map_u8(&tmB, a, len, rows, len, 128, nt, sw);
  else if (op == kLinFwd)
    made = make_map(&tmA, b, len, cols, len, 64, 128, sw) && make_map(&tmB, a, len, rows, len, 64, nt, sw);
  else
    made = make_map(&tmA, b, cols, len, cols, 64, 64, sw) && make_map(&tmB, a, len, rows, len, 64, nt, sw);
  if (!made) return cudaErrorInvalidValue;
  return launch_linear_small(op, nt, tmA, tmB, p, s);
}

// The plan of a product: the planner's (code 0) or the caller's.
kdkl_status pick_plan(int32_t code, LinOp op, int64_t rows, int64_t cols, int64_t len, int sms, const char* name,
                      Plan& plan) {
  const int kb = reduction_blocks(static_cast<int32_t>(std::min<int64_t>(len, INT_MAX / 2)), op == kLinFwdE4M3);
  if (code == 0) {
    plan = plan_linear(op, rows, cols, kb, sms);
    return KDKL_OK;
  }
  if (!decode_plan(code, op, rows, cols, kb, sms, plan)) return fail(KDKL_ERR_UNSUPPORTED, "%s=%d is no plan of this product", name, code);
  const int64_t tiles = plan.pair ? 0 : ((cols + 127) / 128) * ((rows + plan.tile - 1) / plan.tile) * plan.splits;
  if (tiles > INT_MAX / 2) return fail(KDKL_ERR_UNSUPPORTED, "%s=%d has too many tiles", name, code);
  return KDKL_OK;
}

kdkl_status check_activation(int32_t act) {
  if (act < KDKL_ACT_NONE || act > KDKL_ACT_SILU) return fail(KDKL_ERR_UNSUPPORTED, "unknown activation %d", act);
  return KDKL_OK;
}

kdkl_status device_with_pairs(Device& dv) {
  const kdkl_status st = current_device(dv);
  if (st != KDKL_OK) return st;
  if (dv.sms < 2) return fail(KDKL_ERR_UNSUPPORTED, "the linear layer needs CTA pairs");
  return KDKL_OK;
}

// Clears the flag word and the tickets of split tiles ahead of the launches.
kdkl_status clear_header(void* workspace, const LinearLayout& L, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(workspace, 0, L.shares, s);
  return e == cudaSuccess ? KDKL_OK : cuda_fail(e, "cudaMemsetAsync");
}

#ifdef KDKL_DEBUG
constexpr bool kClearAhead = true;    // the kernels' checks can fail at once
#else
constexpr bool kClearAhead = false;   // without split tiles the call's kernel clears the flag word itself
#endif

}  // namespace
}  // namespace kdkl

using namespace kdkl;

extern "C" {

kdkl_status kdkl_rmsnorm_forward(const void* x, const void* residual, const void* gamma, int64_t N, int32_t d,
                                 float eps, int32_t x_dtype, int32_t h_dtype, int32_t gamma_dtype, int32_t y_dtype,
                                 void* h, void* y, float* y_scale, void* stream) {
  kdkl_status st = check_norm(N, d, eps, h_dtype, gamma_dtype);
  if (st != KDKL_OK) return st;
  if (!float_dtype(x_dtype)) return fail(KDKL_ERR_UNSUPPORTED, "x must be KDKL_BF16 or KDKL_F32");
  if (y_dtype != KDKL_BF16 && y_dtype != KDKL_E4M3) return fail(KDKL_ERR_UNSUPPORTED, "y must be KDKL_BF16 or KDKL_E4M3");
  if (!gamma || (N > 0 && (!x || !y))) return fail(KDKL_ERR_NULL, "x, gamma and y must be non-NULL");
  if (N > 0 && (y_dtype == KDKL_E4M3) != (y_scale != nullptr))
    return fail(KDKL_ERR_NULL, "y_scale goes with a KDKL_E4M3 y, and only with one");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(h, 16) || !aligned(y, 16))
    return fail(KDKL_ERR_ALIGN, "x, residual, gamma, h and y must be 16-byte aligned");
  if (!aligned(y_scale, 4)) return fail(KDKL_ERR_ALIGN, "y_scale must be 4-byte aligned");
  Device dv;
  if ((st = current_device(dv)) != KDKL_OK) return st;
  if (N == 0) return ok();
  NormParams p;
  p.x = x;
  p.residual = residual;
  p.gamma = gamma;
  p.h = h;
  p.y = y;
  p.y_scale = y_scale;
  p.N = N;
  p.d = d;
  p.eps = eps;
  p.x_f32 = x_dtype == KDKL_F32;
  p.h_f32 = h_dtype == KDKL_F32;
  p.gamma_f32 = gamma_dtype == KDKL_F32;
  p.y_e4m3 = y_dtype == KDKL_E4M3;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = timed(kTNorm, s, [&] { return launch_rmsnorm(p, dv.sms, s); });
  if (e != cudaSuccess) return cuda_fail(e, "RMS norm launch");
  return ok();
}

size_t kdkl_rmsnorm_workspace_bytes(int64_t N, int32_t d) {
  if (check_norm(N, d, 0.f, KDKL_BF16, KDKL_BF16) != KDKL_OK) return 0;
  return norm_part_bytes(N, d);
}

kdkl_status kdkl_rmsnorm_backward(const void* dy, const void* h, const void* gamma, const void* dh, int64_t N,
                                  int32_t d, float eps, int32_t h_dtype, int32_t gamma_dtype, void* dx,
                                  float* dgamma, void* workspace, size_t workspace_bytes, void* stream) {
  kdkl_status st = check_norm(N, d, eps, h_dtype, gamma_dtype);
  if (st != KDKL_OK) return st;
  if (!gamma || !dgamma || !workspace || (N > 0 && (!dy || !h || !dx)))
    return fail(KDKL_ERR_NULL, "dy, h, gamma, dx, dgamma and workspace must be non-NULL");
  if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(gamma, 16) || !aligned(dh, 16) || !aligned(dx, 16))
    return fail(KDKL_ERR_ALIGN, "dy, h, gamma, dh and dx must be 16-byte aligned");
  if (!aligned(dgamma, 4)) return fail(KDKL_ERR_ALIGN, "dgamma must be 4-byte aligned");
  if (!aligned(workspace, 256)) return fail(KDKL_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t need = norm_part_bytes(N, d);
  if (workspace_bytes < need) return fail(KDKL_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, need);
  Device dv;
  if ((st = current_device(dv)) != KDKL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) {
    const cudaError_t e = cudaMemsetAsync(dgamma, 0, static_cast<size_t>(d) * 4, s);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    return ok();
  }
  NormGradParams p;
  p.dy = dy;
  p.h = h;
  p.gamma = gamma;
  p.dh = dh;
  p.dx = dx;
  p.part = static_cast<float*>(workspace);
  p.N = N;
  p.d = d;
  p.eps = eps;
  p.h_f32 = h_dtype == KDKL_F32;
  p.gamma_f32 = gamma_dtype == KDKL_F32;
  const cudaError_t e = timed(kTNormGrad, s, [&] {
    cudaError_t e1;
    const int blocks = launch_rmsnorm_grad(p, dv.sms, s, &e1);
    return e1 != cudaSuccess ? e1 : launch_colsum(p.part, blocks, d, dgamma, s);
  });
  if (e != cudaSuccess) return cuda_fail(e, "RMS norm gradient launch");
  return ok();
}

void kdkl_linear_options_init(kdkl_linear_options* options) {
  if (options) *options = default_linear_options();
}

size_t kdkl_linear_workspace_bytes(int64_t M, int32_t d_in, int32_t d_out, int32_t backward) {
  if (check_linear_shape(M, d_in, d_out, KDKL_BF16) != KDKL_OK) return 0;
  return linear_layout(M, d_in, d_out, backward != 0).total;
}

kdkl_status kdkl_linear_plan(int64_t M, int32_t d_in, int32_t d_out, int32_t operands, int32_t product,
                             int32_t sm_count, int32_t* plan_out) {
  if (!plan_out) return fail(KDKL_ERR_NULL, "plan_out must be non-NULL");
  kdkl_status st = check_linear_shape(M, d_in, d_out, operands);
  if (st != KDKL_OK) return st;
  if (product < KDKL_LINEAR_FORWARD || product > KDKL_LINEAR_DW)
    return fail(KDKL_ERR_UNSUPPORTED, "unknown product %d", product);
  if (product != KDKL_LINEAR_FORWARD && operands != KDKL_BF16)
    return fail(KDKL_ERR_UNSUPPORTED, "KDKL_E4M3 operands have no gradient");
  if (sm_count < 0 || sm_count == 1) return fail(KDKL_ERR_SHAPE, "sm_count must be 0 or >= 2");
  if (sm_count == 0) {
    Device dv;
    if ((st = device_with_pairs(dv)) != KDKL_OK) return st;
    sm_count = dv.sms;
  }
  Plan p;
  if (product == KDKL_LINEAR_FORWARD)
    st = pick_plan(0, operands == KDKL_E4M3 ? kLinFwdE4M3 : kLinFwd, M, d_out, d_in, sm_count, "plan", p);
  else if (product == KDKL_LINEAR_DX)
    st = pick_plan(0, kLinDx, M, d_in, d_out, sm_count, "dx_plan", p);
  else
    st = pick_plan(0, kLinDw, d_out, d_in, M, sm_count, "dw_plan", p);
  if (st != KDKL_OK) return st;
  *plan_out = p.code();
  return ok();
}

kdkl_status kdkl_linear_forward(const void* x, const void* W, const void* bias, const void* residual, int64_t M,
                                int32_t d_in, int32_t d_out, const kdkl_linear_options* options, void* y, void* pre,
                                void* workspace, size_t workspace_bytes, void* stream) {
  const kdkl_linear_options o = options ? *options : default_linear_options();
  kdkl_status st = check_linear_shape(M, d_in, d_out, o.operands);
  if (st != KDKL_OK) return st;
  if ((st = check_activation(o.activation)) != KDKL_OK) return st;
  if (!W || !workspace || (M > 0 && (!x || !y)))
    return fail(KDKL_ERR_NULL, "x, W, y and workspace must be non-NULL");
  const bool f8 = o.operands == KDKL_E4M3;
  if (f8 && (!o.w_scale || (M > 0 && !o.x_scale))) return fail(KDKL_ERR_NULL, "KDKL_E4M3 operands need x_scale and w_scale");
  if (!f8 && (o.x_scale || o.w_scale)) return fail(KDKL_ERR_UNSUPPORTED, "x_scale and w_scale go with KDKL_E4M3 operands only");
  if (!aligned(x, 16) || !aligned(W, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(y, 16) ||
      !aligned(pre, 16))
    return fail(KDKL_ERR_ALIGN, "x, W, bias, residual, y and pre must be 16-byte aligned");
  if (!aligned(o.x_scale, 4) || !aligned(o.w_scale, 16))
    return fail(KDKL_ERR_ALIGN, "x_scale must be 4-byte and w_scale 16-byte aligned");
  if (!aligned(workspace, 256)) return fail(KDKL_ERR_ALIGN, "workspace must be 256-byte aligned");
  const LinearLayout L = linear_layout(M, d_in, d_out, false);
  if (workspace_bytes < L.total) return fail(KDKL_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, L.total);
  Device dv;
  if ((st = device_with_pairs(dv)) != KDKL_OK) return st;
  const LinOp op = f8 ? kLinFwdE4M3 : kLinFwd;
  Plan plan;
  if ((st = pick_plan(o.plan, op, M, d_out, d_in, dv.sms, "plan", plan)) != KDKL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t tiles = plan.pair ? ((M + 255) / 256) * ((d_out + plan.tile - 1) / plan.tile) : 0;
  const bool clear_ahead =
      kClearAhead || M == 0 || (plan.pair && plan.splits > 1 && !split_by_cluster(op, tiles));
  if (clear_ahead && (st = clear_header(workspace, L, s)) != KDKL_OK) return st;
  if (M == 0) return ok();
  LinParams p = {};
  p.bias = static_cast<const uint16_t*>(bias);
  p.residual = static_cast<const uint16_t*>(residual);
  p.x_scale = o.x_scale;
  p.w_scale = o.w_scale;
  p.out = static_cast<uint16_t*>(y);
  p.pre = static_cast<uint16_t*>(pre);
  p.act = o.activation;
  p.flags = static_cast<uint32_t*>(workspace);
  p.clear_flags = clear_ahead ? 0 : 1;
  p.tickets = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + L.tickets);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.shares);
  p.part_floats = static_cast<int64_t>(L.share_bytes / 4);
  const cudaError_t e = timed(kTLinear, s, [&] { return run_product(op, plan, x, W, M, d_out, d_in, p, dv.sms, s); });
  if (e != cudaSuccess) return cuda_fail(e, "linear launch");
  return ok();
}

kdkl_status kdkl_linear_backward(const void* dy, const void* pre, const void* x, const void* W, int64_t M,
                                 int32_t d_in, int32_t d_out, const kdkl_linear_options* options, void* dx, void* dW,
                                 float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  const kdkl_linear_options o = options ? *options : default_linear_options();
  kdkl_status st = check_linear_shape(M, d_in, d_out, o.operands);
  if (st != KDKL_OK) return st;
  if (o.operands != KDKL_BF16) return fail(KDKL_ERR_UNSUPPORTED, "KDKL_E4M3 operands have no gradient");
  if ((st = check_activation(o.activation)) != KDKL_OK) return st;
  if (M > 0 && !dx && !dW && !dbias) return fail(KDKL_ERR_NULL, "one of dx, dW and dbias must be non-NULL");
  if (!workspace || (M > 0 && !dy)) return fail(KDKL_ERR_NULL, "dy and workspace must be non-NULL");
  if (dx && !W) return fail(KDKL_ERR_NULL, "dx needs W");
  if (M > 0 && dW && !x) return fail(KDKL_ERR_NULL, "dW needs x");
  const bool act = o.activation != KDKL_ACT_NONE;
  if (M > 0 && act && !pre) return fail(KDKL_ERR_NULL, "the activation's gradient needs pre");
  if (!aligned(dy, 16) || !aligned(pre, 16) || !aligned(x, 16) || !aligned(W, 16) || !aligned(dx, 16) ||
      !aligned(dW, 16))
    return fail(KDKL_ERR_ALIGN, "dy, pre, x, W, dx and dW must be 16-byte aligned");
  if (!aligned(dbias, 4)) return fail(KDKL_ERR_ALIGN, "dbias must be 4-byte aligned");
  if (!aligned(workspace, 256)) return fail(KDKL_ERR_ALIGN, "workspace must be 256-byte aligned");
  const LinearLayout L = linear_layout(M, d_in, d_out, true);
  if (workspace_bytes < L.total) return fail(KDKL_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, L.total);
  Device dv;
  if ((st = device_with_pairs(dv)) != KDKL_OK) return st;
  if (dv.sms > kMaxSms) return fail(KDKL_ERR_UNSUPPORTED, "a device with %d SMs", dv.sms);
  Plan dx_plan, dw_plan;
  if (dx && (st = pick_plan(o.dx_plan, kLinDx, M, d_in, d_out, dv.sms, "dx_plan", dx_plan)) != KDKL_OK) return st;
  if (dW && (st = pick_plan(o.dw_plan, kLinDw, d_out, d_in, M, dv.sms, "dw_plan", dw_plan)) != KDKL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if ((st = clear_header(workspace, L, s)) != KDKL_OK) return st;
  if (M == 0) {
    if (dW && (e = cudaMemsetAsync(dW, 0, static_cast<size_t>(d_out) * d_in * 2, s)) != cudaSuccess)
      return cuda_fail(e, "cudaMemsetAsync");
    if (dbias && (e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(d_out) * 4, s)) != cudaSuccess)
      return cuda_fail(e, "cudaMemsetAsync");
    return ok();
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* dz = dy;
  if (act || dbias) {
    uint16_t* dz_out = act && (dx || dW) ? reinterpret_cast<uint16_t*>(ws + L.dz) : nullptr;
    e = timed(kTActGrad, s, [&] {
      return launch_act_grad(static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(pre), o.activation, M,
                             d_out, dz_out, reinterpret_cast<float*>(ws + L.part),
                             static_cast<int64_t>((L.total - L.part) / 4),
                             reinterpret_cast<uint32_t*>(ws + L.col_tickets), dbias, reinterpret_cast<uint32_t*>(ws),
                             act_grad_chunks(M, d_out, dv.sms), s);
    });
    if (e != cudaSuccess) return cuda_fail(e, "activation gradient launch");
    if (act) dz = ws + L.dz;
  }
  LinParams p = {};
  p.flags = static_cast<uint32_t*>(workspace);
  p.tickets = reinterpret_cast<uint32_t*>(ws + L.tickets);
  p.part = reinterpret_cast<float*>(ws + L.shares);
  p.part_floats = static_cast<int64_t>(L.share_bytes / 4);
  if (dx) {
    p.out = static_cast<uint16_t*>(dx);
    e = timed(kTLinearDx, s, [&] { return run_product(kLinDx, dx_plan, dz, W, M, d_in, d_out, p, dv.sms, s); });
    if (e != cudaSuccess) return cuda_fail(e, "linear dx launch");
  }
  if (dW) {
    p.out = static_cast<uint16_t*>(dW);
    e = timed(kTLinearDw, s, [&] { return run_product(kLinDw, dw_plan, dz, x, d_out, d_in, M, p, dv.sms, s); });
    if (e != cudaSuccess) return cuda_fail(e, "linear dW launch");
  }
  return ok();
}

}  // extern "C"
