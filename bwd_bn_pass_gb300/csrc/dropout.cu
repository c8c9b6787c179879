// Dropout whose mask comes from a counter (philox.cuh) and is never stored,
// with an optional bias in front and an optional residual behind it:
//   forward   y  = residual + keep*s*(x + bias)
//   backward  dx = keep*s*dy,  dbias = sum over rows of dx
// over [R, H] rows.  The residual's gradient is dy itself.
//
// Bound: DRAM traffic (forward 2-3, backward 2 tensors).
//
// Two kernels:
//   * rows of whole 8-element chunks, 16-byte aligned tensors: a thread owns
//     one chunk of columns (one generator block per row; the bias, or the
//     bias gradient's sums, stay in registers) and strides down its block's
//     slice of rows, several rows in flight;
//   * everything else: a block owns 248 columns; eight rows at a time its 256
//     threads draw the 8 x 32 blocks that cover them into shared memory as
//     bits, then every thread walks its column.
// The bias gradient's per-block partial rows are added in a fixed order by
// colsum_kernel (no atomics).
#include "gbn_common.cuh"
#include "gbn_internal.h"
#include "philox.cuh"

namespace gbn {

namespace {

constexpr int kDThreads = 256;
constexpr int kDTileCols = 248;  // 248 + 7 elements span at most 32 blocks
constexpr int kDTileRows = 8;

struct DropArgs {
  const void* x;     // forward input / dy
  const void* res;   // forward: residual or null
  const void* bias;  // forward: bias or null
  void* y;           // y / dx
  float* part;       // backward: partial column sums [plane][slices][H], or null
  int64_t R;
  int32_t H;
  int32_t Hc;        // chunks per row (rows kernel)
  int32_t TX, TY;    // rows kernel: chunks x rows of a block
  int32_t slices;
  RngArgs rng;
};

// Eight elements of T as two or one 16-byte vectors.
template <typename T> struct Chunk8 {
  static constexpr int NV = sizeof(T) / 2;  // 16-byte vectors
  static constexpr int VE = 16 / sizeof(T);
  using V = Vec<T, VE>;
  uint4 raw[NV];
  __device__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < NV; ++k) raw[k] = V::ld(p + k * VE);
  }
  __device__ void get(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float t[VE];
      V::cvt(raw[k], t);
#pragma unroll
      for (int e = 0; e < VE; ++e) v[k * VE + e] = t[e];
    }
  }
  __device__ static void store(T* p, const float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float t[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) t[e] = v[k * VE + e];
      V::store(p + k * VE, t);
    }
  }
};

// fp32 sums carry their rounding errors (the fp32 bias gradient); bf16 ones
// are plain fp32, far below the output's rounding.
template <typename T> struct ColSum {
  DF s{0.f, 0.f};
  __device__ void add(float v) {
    if constexpr (sizeof(T) == 4) df_add(s, v);
    else s.hi += v;
  }
  __device__ void add(const DF& v) {
    if constexpr (sizeof(T) == 4) s = df_sum(s, v);
    else s.hi += v.hi;
  }
};

template <typename T, bool BWD, bool RES, bool STATE>
__global__ void __launch_bounds__(kDThreads, 4) dropout_rows_kernel(const DropArgs a) {
  constexpr int U = sizeof(T) == 2 ? (RES ? 2 : 4) : (RES ? 1 : 2);  // rows in flight
  using C8 = Chunk8<T>;
  extern __shared__ DF red[];  // [TY][TX][8] when sums are asked for
  const int ty = threadIdx.x / a.TX, tx = threadIdx.x - ty * a.TX;
  const int cv = blockIdx.x * a.TX + tx;
  const bool active = cv < a.Hc;
  const int64_t H = a.H;
  const int64_t r0 = a.R * blockIdx.y / a.slices, r1 = a.R * (blockIdx.y + 1) / a.slices;
  Philox<STATE> g;
  g.load(a.rng);
  const float scale = a.rng.scale;
  float b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] = 0.f;
  ColSum<T> sum[8];
  if (active) {
    if (!BWD && a.bias != nullptr) {
      C8 c;
      c.load(static_cast<const T*>(a.bias) + (int64_t)cv * 8);
      c.get(b);
    }
    const int64_t first = r0 + ty, step = (int64_t)a.TY * H;
    const T* x = static_cast<const T*>(a.x) + first * H + (int64_t)cv * 8;
    const T* res = static_cast<const T*>(a.res) + first * H + (int64_t)cv * 8;
    T* y = static_cast<T*>(a.y) + first * H + (int64_t)cv * 8;
    uint64_t blk = (uint64_t)(first * a.Hc + cv);
    const uint64_t bstep = (uint64_t)a.TY * a.Hc;
    int64_t left = r1 > first ? (r1 - first + a.TY - 1) / a.TY : 0;
    for (; left > 0; left -= U) {
      C8 cx[U], cr[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < left) {
          cx[u].load(x + u * step);
          if constexpr (RES) cr[u].load(res + u * step);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= left) continue;
        bool f[8];
        float v[8], o[8];
        g.template keep<8>(a.rng, blk << 3, f);
        cx[u].get(v);
        if constexpr (RES) cr[u].get(o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // a dropped element is exactly 0 (or the residual), whatever x holds
          const float t = f[e] ? (BWD ? v[e] : v[e] + b[e]) : 0.f;
          o[e] = RES ? fmaf(t, scale, o[e]) : t * scale;
          if constexpr (BWD) sum[e].add(o[e]);
        }
        C8::store(y + u * step, o);
        blk += bstep;
      }
      x += U * step;
      if constexpr (RES) res += U * step;
      y += U * step;
    }
  }
  if constexpr (BWD) {
    if (a.part == nullptr) return;
    // the block's rows of threads, added in order
    if (active)
#pragma unroll
      for (int e = 0; e < 8; ++e) red[((size_t)ty * a.TX + tx) * 8 + e] = sum[e].s;
    __syncthreads();
    if (ty == 0 && active) {
      for (int q = 1; q < a.TY; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e].add(red[((size_t)q * a.TX + tx) * 8 + e]);
      float* hi = a.part + (int64_t)blockIdx.y * H + (int64_t)cv * 8;
      float* lo = hi + (int64_t)a.slices * H;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = sum[e].s.hi;
        if constexpr (sizeof(T) == 4) lo[e] = sum[e].s.lo;
      }
    }
    pdl_launch_dependents();
  }
}

// Any H and alignment.
template <typename T, bool BWD>
__global__ void __launch_bounds__(kDThreads) dropout_tile_kernel(DropArgs a) {
  __shared__ uint8_t bits[kDTileRows][32];
  const int64_t H = a.H;
  const int64_t j0 = (int64_t)blockIdx.x * kDTileCols;
  const int64_t j = j0 + threadIdx.x;
  const bool active = threadIdx.x < kDTileCols && j < H;
  const int64_t r0 = a.R * blockIdx.y / a.slices, r1 = a.R * (blockIdx.y + 1) / a.slices;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  T* y = static_cast<T*>(a.y);
  PhiloxAny g;
  g.load(a.rng);
  const float b = !BWD && active && a.bias ? to_f32(static_cast<const T*>(a.bias)[j]) : 0.f;
  ColSum<T> sum;
  const int wr = threadIdx.x >> 5, wl = threadIdx.x & 31;
  for (int64_t r = r0; r < r1; r += kDTileRows) {
    // the loads first: the blocks are drawn while they are on their way
    float v[kDTileRows], q[kDTileRows];
#pragma unroll
    for (int u = 0; u < kDTileRows; ++u) {
      v[u] = q[u] = 0.f;
      if (active && r + u < r1) {
        v[u] = to_f32(x[(r + u) * H + j]);
        if (!BWD && res != nullptr) q[u] = to_f32(res[(r + u) * H + j]);
      }
    }
    if (r + wr < r1)
      bits[wr][wl] = (uint8_t)g.bits(a.rng, ((uint64_t)((r + wr) * H + j0) >> 3) + wl);
    __syncthreads();
    if (active) {
#pragma unroll
      for (int u = 0; u < kDTileRows; ++u) {
        if (r + u < r1) {
          const uint64_t i = (uint64_t)((r + u) * H + j);
          const uint64_t b0 = (uint64_t)((r + u) * H + j0) >> 3;
          const bool keep = (bits[u][(i >> 3) - b0] >> (i & 7)) & 1;
          const float t = keep ? v[u] + b : 0.f;
          const float o = fmaf(t, a.rng.scale, q[u]);
          y[i] = from_f32<T>(o);
          if constexpr (BWD) sum.add(o);
        }
      }
    }
    __syncthreads();  // the bits are read
  }
  if constexpr (BWD) {
    if (a.part != nullptr && active) {
      a.part[(int64_t)blockIdx.y * H + j] = sum.s.hi;
      if constexpr (sizeof(T) == 4) a.part[((int64_t)a.slices + blockIdx.y) * H + j] = sum.s.lo;
    }
    pdl_launch_dependents();
  }
}

template <typename T, bool STATE>
cudaError_t launch_rows(const DropPlan& p, const DropArgs& a, bool bwd, cudaStream_t st) {
  const dim3 grid((unsigned)p.gx, (unsigned)p.slices), block((unsigned)(p.TX * p.TY));
  if (bwd)
    return launch(dropout_rows_kernel<T, true, false, STATE>, grid, block,
                  a.part ? sizeof(DF) * 8 * (size_t)(p.TX * p.TY) : 0, st, false, a);
  if (a.res != nullptr)
    return launch(dropout_rows_kernel<T, false, true, STATE>, grid, block, 0, st, false, a);
  return launch(dropout_rows_kernel<T, false, false, STATE>, grid, block, 0, st, false, a);
}
template <typename T>
cudaError_t launch_drop(const DropPlan& p, const DropArgs& a, bool bwd, cudaStream_t st) {
  if (p.fast)
    return a.rng.state != nullptr ? launch_rows<T, true>(p, a, bwd, st)
                                  : launch_rows<T, false>(p, a, bwd, st);
  const dim3 grid((unsigned)p.gx, (unsigned)p.slices);
  return bwd ? launch(dropout_tile_kernel<T, true>, grid, dim3(kDThreads), 0, st, false, a)
             : launch(dropout_tile_kernel<T, false>, grid, dim3(kDThreads), 0, st, false, a);
}

}  // namespace

RngArgs make_rng(double p, uint64_t seed, uint64_t offset, const uint64_t* state) {
  RngArgs r;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
  for (int i = 0; i < 10; ++i) {
    r.key[2 * i] = k0;
    r.key[2 * i + 1] = k1;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  r.offset = offset;
  r.state = state;
  const uint32_t thr = (uint32_t)((1.0 - p) * 65536.0 + 0.5);  // 0 .. 65536
  r.all = thr == 65536 ? 1u : 0u;
  r.lim = thr << 16;
  r.scale = thr ? (float)(65536.0 / (double)thr) : 0.f;
  return r;
}

DropPlan drop_plan(int64_t R, int64_t H, bool fast_ok, int dtype, const DevInfo& dev) {
  DropPlan p;
  p.fast = fast_ok && H % 8 == 0;
  const int64_t rows_per_round = dtype == GBN_F32 ? 2 : 4;
  int64_t min_rows;
  if (p.fast) {
    const int64_t Hc = H / 8;
    p.gx = (Hc + kDThreads - 1) / kDThreads;
    p.TX = (int)((Hc + p.gx - 1) / p.gx);
    p.TY = kDThreads / p.TX;
    min_rows = rows_per_round * p.TY;  // one round of loads a block, at least
  } else {
    p.gx = (H + kDTileCols - 1) / kDTileCols;
    min_rows = kDTileRows;
  }
  // every resident block slot once
  int64_t s = ((int64_t)dev.sms * kDBlocksPerSm + p.gx - 1) / p.gx;
  const int64_t by_rows = (R + min_rows - 1) / min_rows;
  if (s > by_rows) s = by_rows;
  if (s < 1) s = 1;
  if (s > 65535) s = 65535;
  p.slices = (int)s;
  p.ws_bytes = ((size_t)(dtype == GBN_F32 ? 2 : 1) * (size_t)s * (size_t)H * 4 + 255) & ~(size_t)255;
  return p;
}

cudaError_t drop_forward(const DropPlan& p, int dtype, const void* x, const void* bias,
                         const void* res, void* y, int64_t R, int64_t H, const RngArgs& rng,
                         cudaStream_t st) {
  DropArgs a{x, res, bias, y, nullptr, R, (int32_t)H, (int32_t)(H / 8), p.TX, p.TY, p.slices, rng};
  return dtype == GBN_F32 ? launch_drop<float>(p, a, false, st) : launch_drop<bf16>(p, a, false, st);
}

cudaError_t drop_backward(const DropPlan& p, int dtype, const void* dy, void* dx, void* dbias,
                          void* ws, int64_t R, int64_t H, const RngArgs& rng, cudaStream_t st) {
  DropArgs a{dy, nullptr, nullptr, dx, dbias ? static_cast<float*>(ws) : nullptr, R, (int32_t)H,
             (int32_t)(H / 8), p.TX, p.TY, p.slices, rng};
  cudaError_t e =
      dtype == GBN_F32 ? launch_drop<float>(p, a, true, st) : launch_drop<bf16>(p, a, true, st);
  if (e != cudaSuccess || dbias == nullptr) return e;
  void* outs[3] = {dbias, nullptr, nullptr};
  return colsum_launch(a.part, 1, dtype == GBN_F32 ? 2 : 1, p.slices, H, dtype, outs, st, true);
}

}  // namespace gbn
