// Host-side declarations shared by the C ABI (abi.cu) and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gbnorm.h"

namespace gbn {

// Cached per-device facts.  Filled once per device by device_info().
struct DevInfo {
  int sms = 0;               // multiprocessor count (152 on GB300)
  int max_threads_sm = 0;    // resident threads per SM (2048)
  int smem_optin = 0;        // max dynamic shared memory per block (bytes)
  int smem_per_sm = 0;       // shared memory per SM (bytes)
  int smem_reserved = 0;     // shared memory the runtime reserves per block
  int l2_bytes = 0;          // L2 cache size
  int* status = nullptr;     // device address of the library status word
  bool fused_ok = false;     // the persistent BatchNorm kernel fits one CTA per SM
  bool ok = false;
};

// Returns nullptr (and leaves a CUDA error pending) if the device cannot be
// queried.  device < 0 means the current device.
const DevInfo* device_info(int device);

// ---- argument checks shared by the C entry points ----

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// a*b without int64 overflow; false on overflow or negative operands.
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a < 0 || b < 0) return false;
  if (a != 0 && b > INT64_MAX / a) return false;
  *out = a * b;
  return true;
}

inline int to_status(cudaError_t e) { return e == cudaSuccess ? GBN_OK : GBN_ECUDA; }

// dtype and sizes of a row-wise call.
inline int row_check(int dtype, int64_t R, int64_t H) {
  if (dtype != GBN_F32 && dtype != GBN_BF16) return GBN_EDTYPE;
  if (R < 0 || H < 0 || H > INT32_MAX / 16) return GBN_EINVAL;
  int64_t n;
  if (!mul_ok(R, H, &n) || n > (INT64_MAX >> 3)) return GBN_EINVAL;
  return GBN_OK;
}

// Launch `kern` with the given configuration; `pdl` adds the programmatic
// stream serialization attribute so the kernel may start while the
// preceding kernel on the stream drains (it then calls griddepcontrol.wait).
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem,
                   cudaStream_t stream, bool pdl, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  if (pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// ------------------------------------------------------------- BatchNorm --

constexpr int kBnThreads = 256;
constexpr int kBnBlocksPerSm = 4;   // resident 256-thread blocks per SM the grid fills
constexpr int64_t kBnMinElemsPerBlock = 4096;

// Shape facts derived once per call on the host.
struct BnPlan {
  int64_t B = 0, C = 0, P = 0;  // batch, channels, plane size (HW)
  int64_t M = 0;                // per-channel count B*P
  int grid_y = 0;               // blocks per channel
  int vec = 1;                  // elements per vector access
  size_t ws_partials = 0;       // two-launch partials bytes (2 * grid_y * C fp32 pairs, rounded)
  size_t ws_bytes = 0;          // workspace of the public calls: also fits the persistent path
};

// Fills grid_y / ws_bytes (device-dependent) for a shape; false on error.
int bn_set_wide_offsets(int force);  // 64-bit offsets in the two-launch kernels
bool bn_plan(int64_t B, int64_t C, int64_t HW, const DevInfo& dev, BnPlan* plan);

// Largest power-of-two vector width (<= 16 bytes) valid for all pointers.
int bn_vec_width(int dtype, int64_t P, const void* const* ptrs, int nptrs);

enum BnApplyMode { kApplyTrain = 0, kApplyStats = 1, kApplyInfer = 2 };

cudaError_t bn_launch_stats(const void* x, int dtype, const BnPlan& p, float2* part,
                            cudaStream_t st);
cudaError_t bn_launch_apply(const void* x, void* y, int dtype, const BnPlan& p, int mode,
                            const float2* part, const float* gamma, const float* beta,
                            float* stats, float* running_mean, float* running_var,
                            float momentum, float eps, const float* mean, const float* scale,
                            int act, float slope, cudaStream_t st, bool pdl);
// With act != GBN_ACT_NONE the backward kernels gate dy by d act / d pre,
// pre recomputed from x, the stats rows and beta (may be null: 0).
cudaError_t bn_launch_grad_sums(const void* x, const void* dy, int dtype, const BnPlan& p,
                                const float* stats, float2* part, const float* beta, int act,
                                float slope, cudaStream_t st);
cudaError_t bn_launch_dx(const void* x, const void* dy, void* dx, int dtype, const BnPlan& p,
                         const float* stats, const float2* part, float* grads, const float* beta,
                         int act, float slope, cudaStream_t st, bool pdl);

// Single-launch BatchNorm for small channels (bn_small.cu): one block per
// channel stages the channel's M <= lim elements in shared memory; up to
// kBnClusterMax * lim elements, a cluster of up to kBnClusterMax blocks per
// channel, each staging a share of at most lim (lim <= kBnSmallMaxM).
constexpr int64_t kBnSmallMaxM = 2048;
constexpr int kBnClusterMax = 8;
// Resident 256-thread blocks per SM the small-channel kernels are sized for
// (at most 64 registers a thread).
constexpr int kBnSmallBlocksPerSm = 4;
// Blocks per channel K (1, 2, 4 or 8) with which the small-channel kernels
// take a shape: the smallest K whose shares hold at most lim elements, and
// only while the grid is one latency chain per block (load, reduce,
// finalize, store) with no second wave: one block per channel while the C
// blocks fit kBnSmallBlocksPerSm per SM; a cluster while the C*K blocks fit
// one per SM (measured: 148 blocks beat the two-launch kernels by ~0.5 us,
// 256 tie, 608 lose by ~3 us).  0: not eligible.
int bn_small_blocks(int64_t M, int64_t C, int64_t lim, const DevInfo& dev);
cudaError_t bn_small_forward(int dtype, const void* x, void* y, int64_t B, int64_t C,
                             int64_t HW, const float* gamma, const float* beta, float* stats,
                             float* running_mean, float* running_var, float momentum, float eps,
                             int act, float slope, int K, cudaStream_t st);
cudaError_t bn_small_backward(int dtype, const void* x, const void* dy, void* dx, int64_t B,
                              int64_t C, int64_t HW, const float* stats, const float* beta,
                              int act, float slope, float* grads, int K, cudaStream_t st);

// Persistent single-launch BatchNorm (bn_fused.cu): one CTA per SM owns a
// contiguous range of the channel-major view; see that file.
constexpr int64_t kBnFusedMinVectors = 2048;  // 16-byte vectors per CTA, at least
constexpr int kBnFusedStages = 4;             // shared-memory ring depth

struct BnFusedPlan {
  bool ok = false;
  int64_t B = 0, C = 0, P = 0, M = 0;
  int64_t Pv = 0, Mv = 0;  // 16-byte vectors per plane / per channel
  int64_t Wv = 0;          // vectors per CTA
  int G = 0;               // CTAs
  int grid_y = 0;          // partial slots per channel
  int stage_v = 0;         // vectors per stage and input
  int nstage = 0;
  int l2_window = 0;       // phase-1 stages per CTA kept at normal L2 priority
  int tmem_stages = 0;     // stages per CTA kept in tensor memory between the phases
  int pool = 0;            // a CTA's first stages open to other CTAs in phase 2
  bool stream_out = true;  // outputs stored with the evict-first hint
  size_t smem = 0;         // dynamic shared memory (the ring)
  size_t part_offset = 0;  // partials offset in the workspace (sync words first)
  size_t ws_bytes = 0;
};

// False when the shape or device does not take the persistent path (plane
// not a whole number of 16-byte vectors, too many channels per CTA, ...).
bool bn_fused_plan(int dtype, bool backward, int64_t B, int64_t C, int64_t HW,
                   const DevInfo& dev, BnFusedPlan* plan);
// Whether later plans keep stages in TMEM (process-wide); returns the previous setting.
int bn_fused_set_tmem(int enable);
// Whether later plans let CTAs take other CTAs' last stages; returns the previous setting.
int bn_fused_set_steal(int enable);
cudaError_t bn_fused_forward(const BnFusedPlan& p, int dtype, const void* x, void* y,
                             const float* gamma, const float* beta, float* stats,
                             float* running_mean, float* running_var, float momentum, float eps,
                             int act, float slope, void* ws, int* status, cudaStream_t st);
cudaError_t bn_fused_backward(const BnFusedPlan& p, int dtype, const void* x, const void* dy,
                              void* dx, const float* stats, const float* beta, int act,
                              float slope, float* grads, void* ws, int* status,
                              cudaStream_t st);
// A fresh 64-bit value per call: the epoch of a launch whose workspace holds
// no valid epoch pair (kernels that hand results between resident CTAs).
unsigned long long next_nonce();
// Shared-memory limits and the one-CTA-per-SM check (called from device_info).
cudaError_t bn_fused_configure(int smem_optin, bool* ok);

// Training forward with a caller-fixed scratch buffer (the allocation-free
// entry point): `ws` must hold at least bn_partials_bytes(B, C, HW) bytes;
// the persistent kernel is used when `ws_bytes` also fits its workspace,
// else the two-launch kernels.  Same status codes as gbn_bn_forward_train.
size_t bn_partials_bytes(int64_t B, int64_t C, int64_t HW);
// The argument checks of the training forward that need no CUDA call (dtype,
// sizes, null pointers, stats alignment, eps / momentum): GBN_OK or the
// status the forward would return for them.
int bn_forward_check_args(const void* x, int dtype, int64_t B, int64_t C, int64_t HW,
                          const void* y, const float* stats, float momentum, float eps);
int bn_forward_train_scratch(const void* x, int dtype, int64_t B, int64_t C, int64_t HW,
                             const float* gamma, const float* beta, float* running_mean,
                             float* running_var, float momentum, float eps, void* y,
                             float* stats, void* ws, size_t ws_bytes, void* stream);

// ------------------------------------------------------------ row-wise --

// Column partials: [nout][nplanes][G][H] fp32; nplanes = 2 (hi, lo) when the
// outputs are fp32 (double-fp32 accumulation), 1 otherwise.
struct RowPlan {
  int64_t R = 0, H = 0;
  int kind = GBN_ROW_RMS;
  int dtype = GBN_F32;
  bool fast = false;   // bulk-copy persistent kernel (else the generic kernel)
  int threads = 0;     // block size
  int kv = 0;          // 16-byte vectors per thread per row (fast path)
  int rb = 1;          // rows per pipeline stage (fast path)
  int cps = 1;         // blocks per SM the launch is sized for (fast path)
  int nstage = 0;      // pipeline depth (fast path)
  int G = 0;           // blocks (= rows of column partials)
  int sms = 0;         // the device's, and its shared memory per block
  int smem_optin = 0;
  bool aligned = false;  // every tensor is 16-byte aligned
  int nout = 1;        // column outputs
  int nplanes = 1;     // 2 when fp32 outputs use hi/lo partials
  size_t smem = 0;     // dynamic shared memory per block
  uint32_t stage_bytes = 0;
  uint32_t off[5] = {0, 0, 0, 0, 0};  // per-stage offsets: dy, x, residual, mask, dz_extra
  int tprw = 0;        // LayerNorm ring: consumer warps per row slot
  int rs = 0;          // LayerNorm ring: row slots
  size_t part_offset = 0;  // column partials' offset in the workspace (flags first)
  size_t ws_bytes = 0;
};

// Consumer warps of the LayerNorm ring kernel: at most 14 when a thread owns
// one 16-byte vector of a row, 8 when it owns two (register budget).
constexpr int kLnRingWarpsKV1 = 14;
constexpr int kLnRingWarpsKVn = 8;

struct RngArgs;  // counter-based dropout mask (philox.cuh)

struct LnPtrs {
  const void* dy = nullptr;
  const void* x = nullptr;
  const void* residual = nullptr;
  const void* bias = nullptr;
  const uint8_t* mask = nullptr;
  const float* dz_extra = nullptr;
  const float* mean = nullptr;
  const float* rstd = nullptr;
  const void* gamma = nullptr;
  float scale = 1.f;
  void* dx = nullptr;
  void* dres = nullptr;
  void* dgamma = nullptr;
  void* dbeta = nullptr;
  void* dbias = nullptr;
  bool saved_z = false;   // x is the saved LayerNorm input z (fused outputs, no residual)
  bool dres_f32 = false;  // dres is fp32
  const RngArgs* rng = nullptr;  // fused: the mask is drawn (mask null, scale unused)
};

// Plans the launch.  `fast_ok` says whether pointers/shape allow the
// bulk-copy path; the workspace query plans with fast_ok=false and true and
// takes the larger size.
bool row_plan(int64_t R, int64_t H, int kind, int dtype, bool fast_ok, bool has_mask,
              bool has_dzx, const DevInfo& dev, RowPlan* plan);

cudaError_t rms_launch(const RowPlan& p, const void* dy, const void* x, const void* w,
                       const float* rstd, void* dx, void* dw, void* ws, int* status,
                       cudaStream_t st);
cudaError_t ln_launch(const RowPlan& p, const LnPtrs& a, void* ws, int* status,
                      cudaStream_t st);

// Row-wise training forwards (fwd_kernels.cu).
struct RowFwdPtrs {
  const void* x = nullptr;         // RMSNorm x / LayerNorm input
  const void* residual = nullptr;  // fused LayerNorm
  const void* bias = nullptr;
  const uint8_t* mask = nullptr;
  const void* w = nullptr;         // RMSNorm weight / LayerNorm gamma
  const void* beta = nullptr;
  void* y = nullptr;
  void* z = nullptr;
  float* mean = nullptr;
  float* rstd = nullptr;
  const RngArgs* rng = nullptr;  // fused LayerNorm: the mask is drawn (mask null)
  bool rows_aligned = false;     // drawn: x, residual, y and z are 16-byte aligned
};

// kind: GBN_ROW_RMS, GBN_ROW_LN or GBN_ROW_LN_FUSED.  vec_ok: every tensor
// is 16-byte aligned and a row is a whole number of 16-byte vectors (and of
// 8-byte mask words), so the register-resident vector kernels may run.
cudaError_t row_fwd_launch(int kind, int dtype, const RowFwdPtrs& p, int64_t R, int64_t H,
                           float eps, float scale, bool vec_ok, const DevInfo& dev,
                           cudaStream_t st);
cudaError_t row_fwd_configure();  // shared-memory limits (called from device_info)

// Column-partials reduction: out[o][h] = sum_g part[o][*][g][h] in a fixed
// order; outs[o] may be nullptr (skipped).  Launched with PDL after the row
// kernel when `pdl` is set.
cudaError_t colsum_launch(const float* part, int nout, int nplanes, int G, int64_t H, int dtype,
                          void* const* outs, cudaStream_t st, bool pdl);

// Set the kernels' dynamic shared memory limits (called from device_info).
cudaError_t row_kernels_configure(int smem_optin);

// Launches one block that waits on an mbarrier nothing completes, through
// the library's bounded wait, for at most limit_ns; the expired wait sets
// GBN_DEV_WAIT_TIMEOUT in *status.
cudaError_t selftest_bounded_wait(int* status, uint64_t limit_ns, cudaStream_t st);

// -------------------------------------------- GroupNorm, channels last --

struct GnPlan {
  int64_t N = 0, S = 0, C = 0, G = 0;  // samples, rows per sample, channels, groups
  bool backward = false;
  bool small = false;       // one launch, a cluster of `slices` blocks per sample
  int vec = 1;              // channels per vector (divides C)
  int TX = 1, TY = 1;       // block shape: vectors x rows
  int tiles = 1;            // channel tiles of TX vectors
  int slices = 1;           // row slices per sample
  int threads = 32;         // block size
  int tile_groups = 1;      // groups a tile can touch, at most
  int rps = 1;              // rows per slice
  size_t gpart_bytes = 0;   // group partials; the channel partials follow
  size_t ws_bytes = 0;
};
bool gn_plan(int64_t N, int64_t S, int64_t C, int64_t G, int vec, int64_t esize, bool backward,
             const DevInfo& dev, GnPlan* p);
// Workspace for any vector width and direction.
size_t gn_ws_bound(int64_t N, int64_t S, int64_t C, int64_t G, const DevInfo& dev);
cudaError_t gn_forward(const GnPlan& p, int dtype, const void* x, const float* gamma,
                       const float* beta, float eps, int act, float slope, void* y, float* stats,
                       void* ws, cudaStream_t st);
cudaError_t gn_backward(const GnPlan& p, int dtype, const void* x, const void* dy,
                        const float* stats, const float* gamma, const float* beta, int act,
                        float slope, void* dx, float* dgamma, float* dbeta, void* ws,
                        cudaStream_t st);

// ------------------------------- head RMSNorm and rotary positions --

constexpr int64_t kRopeMaxD = 512;  // head dimension

struct RopePlan {
  int vec = 1;        // elements per vector
  int ns = 1;         // slots (pairs of vectors) per lane
  int L = 1;          // lanes per team
  int cq = 0, ck = 0; // chunks of query / key heads
  int64_t bx = 1;     // backward: blocks per chunk
  size_t ws_bytes = 0;
};
struct RopePtrs {
  const void* x = nullptr;
  const void* dy = nullptr;
  void* out = nullptr;
  const void* pos = nullptr;
  bool pos64 = true;
  const uint64_t* freqs = nullptr;
  const void* wq = nullptr;  // null: no norm
  const void* wk = nullptr;
  float* rstd = nullptr;
  void* dwq = nullptr;
  void* dwk = nullptr;
  void* ws = nullptr;
  int64_t xt = 0, xh = 0, yt = 0, yh = 0, dt = 0, dh = 0;  // token / head strides
};
bool rope_plan(int64_t T, int64_t H, int64_t HQ, int64_t D, int64_t rot, bool inter, int dtype,
               int vec_max, int dir, const DevInfo& dev, RopePlan* p);
size_t rope_ws_bound(int64_t T, int64_t H, int64_t HQ, int64_t D, int64_t rot, int dtype,
                     const DevInfo& dev);
cudaError_t rope_configure();  // shared-memory limits (called from device_info)
// dir: 0 forward, 1 backward (without wq: the rotation back of dy).
cudaError_t rope_launch(const RopePlan& p, const RopePtrs& q, int dir, int dtype, int64_t T,
                        int64_t H, int64_t HQ, int64_t D, int64_t rot, bool inter, float scale,
                        float eps, cudaStream_t st);

// ------------------------------------------ dropout, mask never stored --

// 256-thread blocks per SM the grid fills: three leave each thread two rows of
// loads in flight (forward bf16 [8192, 8192] 71 us; other splits of the registers
// 75 to 85)
constexpr int kDBlocksPerSm = 3;

// Generator arguments for drop probability p in [0, 1].
RngArgs make_rng(double p, uint64_t seed, uint64_t offset, const uint64_t* state);

struct DropPlan {
  bool fast = false;    // 8-element chunks of a row per thread (else flat, or the tile kernel)
  int64_t gx = 1;       // column tiles
  int ltx = 0;          // fast: log2 of the chunks of a block's row
  int slices = 1;       // row slices (= rows of partial column sums)
  int flat = 0;         // blocks of the flat kernel (0: tensors not aligned)
  int team = 0;         // team kernel: threads of a row's team (0: the tile kernel)
  int threads = 0, team_blocks = 0;
  size_t ws_bytes = 0;  // backward with dbias: the partials
};
cudaError_t drop_configure();  // shared-memory limits (called from device_info)
// fast_ok: every tensor is 16-byte aligned.
DropPlan drop_plan(int64_t R, int64_t H, bool fast_ok, int dtype, const DevInfo& dev);
cudaError_t drop_forward(const DropPlan& p, int dtype, const void* x, const void* bias,
                         const void* res, void* y, int64_t R, int64_t H, const RngArgs& rng,
                         cudaStream_t st);
cudaError_t drop_backward(const DropPlan& p, int dtype, const void* dy, void* dx, void* dbias,
                          void* ws, int64_t R, int64_t H, const RngArgs& rng, cudaStream_t st);

// -------------------------------------------- BatchNorm, channels last --

struct NhwcPlan {
  int64_t M = 0, C = 0;  // rows (N*H*W) and channels
  int vec = 1;           // channels per vector (divides C)
  int TX = 1;            // vectors per block row
  int grid_y = 1;        // row slices
  size_t ws_bytes = 0;   // partials [2][grid_y][C] float2
};
bool nhwc_plan(int64_t M, int64_t C, int vec, const DevInfo& dev, NhwcPlan* p);
size_t nhwc_ws_bound(int64_t M, int64_t C, const DevInfo& dev);
cudaError_t nhwc_forward(const NhwcPlan& p, int dtype, const void* x, void* y,
                         const float* gamma, const float* beta, float* stats,
                         float* running_mean, float* running_var, float momentum, float eps,
                         int act, float slope, void* ws, cudaStream_t st);
// y = act(((x - shift) - (mean - shift))*scale + beta) from a training
// stats buffer, or (stats NULL) act((x - mean)*scale + beta) from
// per-channel mean and scale.
cudaError_t nhwc_apply(const NhwcPlan& p, int dtype, const void* x, void* y, const float* stats,
                       const float* mean, const float* scale, const float* beta, int act,
                       float slope, cudaStream_t st);
cudaError_t nhwc_backward(const NhwcPlan& p, int dtype, const void* x, const void* dy, void* dx,
                          const float* stats, const float* beta, int act, float slope,
                          float* grads, void* ws, cudaStream_t st);

}  // namespace gbn
