// Dropout whose mask comes from a counter (philox.cuh) and is never stored,
// with an optional bias in front and an optional residual behind it:
//   forward   y  = residual + keep*s*(x + bias)
//   backward  dx = keep*s*dy,  dbias = sum over rows of dx
// over [R, H] rows.  The residual's gradient is dy itself.
//
// Bound: DRAM traffic (forward 2-3, backward 2 tensors).  Measured, caches
// flushed: forward bf16 [8192, 8192] with bias and residual 71 us, 5.7 TB/s (0.84
// of the copy rate; repeated 65 us, 6.2 TB/s); backward bf16 [8192, 1600] with the
// bias gradient 21.6 us, in two launches.
//
// Four kernels:
//   * rows of whole 8-element chunks, 16-byte aligned tensors: a thread owns
//     one chunk of columns (one generator block per row; the bias, or the
//     bias gradient's sums, stay in registers) and strides down its block's
//     slice of rows, several rows in flight;
//   * other rows of aligned tensors, where no column is summed (forward, and the
//     backward without the bias gradient): a thread owns a chunk of the flat
//     tensor, whatever rows it spans, and walks the bias by the column;
//   * the backward with the bias gradient over such rows of at most kTeamMaxH
//     elements: a team of threads per row (row_team.cuh), the column sums in
//     shared memory;
//   * everything else: a block owns 248 columns; eight rows at a time its 256
//     threads draw the 8 x 32 blocks that cover them into shared memory as
//     bits, then every thread walks its column.
// The bias gradient's per-block partial rows are added in a fixed order by
// colsum_kernel (no atomics).
#include <type_traits>

#include "gbn_common.cuh"
#include "gbn_internal.h"
#include "packed.cuh"
#include "philox.cuh"
#include "row_team.cuh"

namespace gbn {

namespace {

constexpr int kDThreads = 256;
constexpr int kDTileCols = 248;  // 248 + 7 elements span at most 32 blocks
constexpr int kDTileRows = 8;
constexpr int kDTeamThreads = 1024;  // team kernel: at most

struct DropArgs {
  const void* x;     // forward input / dy
  const void* res;   // forward: residual or null
  const void* bias;  // forward: bias or null
  void* y;           // y / dx
  float* part;       // backward: partial column sums [plane][slices][H], or null
  int64_t R;
  int32_t H;
  int32_t Hc;        // chunks per row (rows kernel)
  int32_t ltx;       // rows kernel: log2 of the block's chunks per row
  int32_t slices;
  int32_t team;      // team kernel: threads of a row
  RngArgs rng;
};

// Eight elements of T as one or two 16-byte vectors, and as packed pairs.
template <typename T> struct Chunk8 {
  static constexpr int NV = sizeof(T) / 2;  // 16-byte vectors
  static constexpr int VE = 16 / sizeof(T);
  using V = Vec<T, VE>;
  uint4 raw[NV];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < NV; ++k) raw[k] = V::ld(p + k * VE);
  }
  __device__ __forceinline__ void get(f2 (&v)[4]) const {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      f2 t[VE / 2];
      to_pairs<T, VE>(raw[k], t);
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) v[k * (VE / 2) + e] = t[e];
    }
  }
  __device__ __forceinline__ static void store(T* p, const f2 (&v)[4]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      f2 t[VE / 2];
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) t[e] = v[k * (VE / 2) + e];
      store_pairs<T, VE>(p + k * VE, t);
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

// A block is 2^ltx chunks x 256 / 2^ltx rows.
template <typename T, bool BWD, bool RES>
__global__ void __launch_bounds__(kDThreads, kDBlocksPerSm)
    dropout_rows_kernel(const DropArgs a) {
  constexpr bool COMP = sizeof(T) == 4;
  constexpr int U = 2;  // rows in flight (four: 85 against 71 us for [8192, 8192] bf16)
  using C8 = Chunk8<T>;
  __shared__ DF red[BWD ? kDThreads / 32 : 1][BWD ? 32 * 8 : 1];  // [warp][column of the tile]
  const int TX = 1 << a.ltx, TY = kDThreads >> a.ltx;
  const int tx = threadIdx.x & (TX - 1), ty = threadIdx.x >> a.ltx;
  const int cv = (int)blockIdx.x * TX + tx;
  const bool active = cv < a.Hc;
  const int64_t H = a.H;
  const int64_t r0 = a.R * blockIdx.y / a.slices, r1 = a.R * (blockIdx.y + 1) / a.slices;
  __shared__ __align__(16) uint32_t keys[kPhiloxKeys];
  philox_fill(keys, a.rng);
  __syncthreads();
  Philox<true> g;
  g.load(a.rng, keys);
  const f2 scale2 = f2_splat(a.rng.scale);
  f2 b[4] = {0ull, 0ull, 0ull, 0ull};
  DF2 sum[4] = {{0ull, 0ull}, {0ull, 0ull}, {0ull, 0ull}, {0ull, 0ull}};
  if (active) {
    if (!BWD && a.bias != nullptr) {
      C8 c;
      c.load(static_cast<const T*>(a.bias) + (int64_t)cv * 8);
      c.get(b);
    }
    const int64_t first = r0 + ty, step = (int64_t)TY * H;
    const T* x = static_cast<const T*>(a.x) + first * H + (int64_t)cv * 8;
    const T* res = static_cast<const T*>(a.res) + first * H + (int64_t)cv * 8;
    T* y = static_cast<T*>(a.y) + first * H + (int64_t)cv * 8;
    uint64_t blk = (uint64_t)(first * a.Hc + cv);
    const uint64_t bstep = (uint64_t)TY * a.Hc;
    int64_t left = r1 > first ? (r1 - first + TY - 1) / TY : 0;
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
        f2 v[4], o[4];
        g.template keep<8>(blk << 3, f);
        cx[u].get(v);
        if constexpr (RES) cr[u].get(o);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          // a dropped element is exactly 0 (or the residual), whatever x holds
          const float2 t = f2_unpack(BWD ? v[p] : f2_add(v[p], b[p]));
          const f2 k = f2_pack(f[2 * p] ? t.x : 0.f, f[2 * p + 1] ? t.y : 0.f);
          o[p] = RES ? f2_fma(k, scale2, o[p]) : f2_mul_rounded(k, scale2);
          if constexpr (BWD) {
            if constexpr (COMP) df2_add(sum[p], o[p]);
            else sum[p].hi = f2_add(sum[p].hi, o[p]);
          }
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
    // the warp's rows by a fixed shuffle tree, then the warps in order
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 h = f2_unpack(sum[p].hi), lw = f2_unpack(sum[p].lo);
      DF u{h.x, lw.x}, w{h.y, lw.y};
      for (int o = 16; o >= TX; o >>= 1) {
        if constexpr (COMP) {
          u = df_sum(u, shfl_xor_df(u, o));
          w = df_sum(w, shfl_xor_df(w, o));
        } else {
          u.hi += __shfl_xor_sync(0xffffffffu, u.hi, o);
          w.hi += __shfl_xor_sync(0xffffffffu, w.hi, o);
        }
      }
      if (lane < TX) {
        red[warp][lane * 8 + 2 * p] = u;
        red[warp][lane * 8 + 2 * p + 1] = w;
      }
    }
    __syncthreads();
    const int64_t j = (int64_t)blockIdx.x * TX * 8 + threadIdx.x;
    if (threadIdx.x < TX * 8 && j < H) {
      ColSum<T> t;
#pragma unroll
      for (int q = 0; q < kDThreads / 32; ++q) t.add(red[q][threadIdx.x]);
      a.part[(int64_t)blockIdx.y * H + j] = t.s.hi;
      if constexpr (COMP) a.part[((int64_t)a.slices + blockIdx.y) * H + j] = t.s.lo;
    }
    pdl_launch_dependents();
  }
}

// Aligned tensors of any H, no column sums: the flat tensor in chunks of eight.
// (Forward with bias and residual, bf16 [4096, 4097] 27.8 us, [65536, 3] 9.3; the
// tile kernel below 68.7 and 44.1.)
template <typename T>
__global__ void __launch_bounds__(kDThreads, 4) dropout_flat_kernel(const DropArgs a) {
  constexpr int U = 2;  // chunks in flight
  using C8 = Chunk8<T>;
  __shared__ __align__(16) uint32_t keys[kPhiloxKeys];
  philox_fill(keys, a.rng);
  __syncthreads();
  Philox<true> g;
  g.load(a.rng, keys);
  const f2 scale2 = f2_splat(a.rng.scale);
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  const T* bias = static_cast<const T*>(a.bias);
  T* y = static_cast<T*>(a.y);
  const int64_t n = a.R * a.H, whole = n / 8, step = (int64_t)gridDim.x * kDThreads;
  const int64_t c0 = (int64_t)blockIdx.x * kDThreads + threadIdx.x;
  // the column of the chunk's first element, and its advance per chunk
  int j = bias != nullptr ? (int)(8 * c0 % a.H) : 0;
  const int jstep = bias != nullptr ? (int)(8 * step % a.H) : 0;
  for (int64_t c = c0; c < whole; c += U * step) {
    C8 cx[U], cr[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * step < whole) {
        cx[u].load(x + 8 * (c + u * step));
        if (res != nullptr) cr[u].load(res + 8 * (c + u * step));
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (c + u * step >= whole) continue;
      bool f[8];
      f2 v[4], o[4] = {0ull, 0ull, 0ull, 0ull};
      g.template keep<8>((uint64_t)(c + u * step) << 3, f);
      cx[u].get(v);
      if (res != nullptr) cr[u].get(o);
      if (bias != nullptr) {
        float b[8];
        int jj = j;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          b[e] = to_f32(bias[jj]);
          if (++jj == a.H) jj = 0;
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) v[p] = f2_add(v[p], f2_pack(b[2 * p], b[2 * p + 1]));
        j += jstep;
        if (j >= a.H) j -= a.H;
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 t = f2_unpack(v[p]);
        o[p] = f2_fma(f2_pack(f[2 * p] ? t.x : 0.f, f[2 * p + 1] ? t.y : 0.f), scale2, o[p]);
      }
      C8::store(y + 8 * (c + u * step), o);
    }
  }
  // the elements past the last whole chunk
  const int64_t i = whole * 8 + threadIdx.x;
  if (blockIdx.x == gridDim.x - 1 && i < n) {
    const bool keep = (g.bits((uint64_t)whole) >> threadIdx.x) & 1u;
    const float t = to_f32(x[i]) + (bias != nullptr ? to_f32(bias[i % a.H]) : 0.f);
    y[i] = from_f32<T>(fmaf(keep ? t : 0.f, a.rng.scale, res != nullptr ? to_f32(res[i]) : 0.f));
  }
}

// Backward with the bias gradient, aligned tensors, H <= kTeamMaxH.  A column's sum
// changes hands from row to row (a chunk starts at another column there), with the
// team's barrier in between.  bf16 [4096, 4097] 44 us (the tile kernel 65), [20000,
// 101] 15.5 (25.7), [65536, 3] 17.5 (42).
template <typename T>
__global__ void __launch_bounds__(kDTeamThreads, 1) dropout_team_kernel(const DropArgs a) {
  constexpr bool COMP = sizeof(T) == 4;
  using Sum = typename std::conditional<COMP, float2, float>::type;
  extern __shared__ __align__(16) unsigned char tsm[];
  __shared__ __align__(16) uint32_t keys[kPhiloxKeys];
  const int H = a.H, P = team_pitch(H), n = 8 * P, TY = blockDim.x / a.team;
  RowTeam team(nullptr, a.team);
  Sum* sums = reinterpret_cast<Sum*>(tsm);
  Sum* cols = sums + (size_t)team.team * n;
  int64_t r = (int64_t)blockIdx.x * TY + team.team;
  const int64_t step = (int64_t)gridDim.x * TY;
  RowChunk next(r, a.R, H, team.tx);
  Raw8<T> raw;
  auto load = [&] {
    if (r < a.R && next.any()) raw.load(static_cast<const T*>(a.x) + next.at, next);
  };
  load();
  philox_fill(keys, a.rng);
  for (int j = threadIdx.x; j < TY * n; j += blockDim.x) sums[j] = Sum{};
  __syncthreads();
  Philox<true> gen;
  gen.load(a.rng, keys);
  while (r < a.R) {
    const RowChunk c = next;
    float v[8];
    if (c.any()) raw.get(v);
    r += step;
    next = RowChunk(r, a.R, H, team.tx);
    load();
    if (c.any()) {
      const uint32_t kept = gen.bits((uint64_t)c.at >> 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = (kept >> e) & 1u ? v[e] * a.rng.scale : 0.f;
        if (!c.has(e)) continue;
        Sum& s = cols[c.word(e, team.tx, P)];
        if constexpr (COMP) {
          DF t{s.x, s.y};
          df_add(t, v[e]);
          s = make_float2(t.hi, t.lo);
        } else {
          s += v[e];
        }
      }
      chunk_store(static_cast<T*>(a.y) + c.at, v, c);
    }
    team.sync();
  }
  __syncthreads();
  pdl_launch_dependents();
  for (int j = threadIdx.x; j < H; j += blockDim.x) {
    ColSum<T> t;
    for (int y = 0; y < TY; ++y) {
      const Sum s = sums[(size_t)y * n + column_word(j, P)];
      if constexpr (COMP) t.add(DF{s.x, s.y});
      else t.add(s);
    }
    a.part[(int64_t)blockIdx.x * H + j] = t.s.hi;
    if constexpr (COMP) a.part[((int64_t)gridDim.x + blockIdx.x) * H + j] = t.s.lo;
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
  Philox<false> g;
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
      bits[wr][wl] = (uint8_t)g.bits(((uint64_t)((r + wr) * H + j0) >> 3) + wl);
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

template <typename T>
cudaError_t launch_rows(const DropPlan& p, const DropArgs& a, bool bwd, cudaStream_t st) {
  const dim3 grid((unsigned)p.gx, (unsigned)p.slices), block(kDThreads);
  if (bwd)
    return launch(dropout_rows_kernel<T, true, false>, grid, block, 0, st, false, a);
  if (a.res != nullptr)
    return launch(dropout_rows_kernel<T, false, true>, grid, block, 0, st, false, a);
  return launch(dropout_rows_kernel<T, false, false>, grid, block, 0, st, false, a);
}
template <typename T>
cudaError_t launch_drop(const DropPlan& p, const DropArgs& a, bool bwd, cudaStream_t st) {
  if (p.fast) return launch_rows<T>(p, a, bwd, st);
  if (p.flat > 0 && a.part == nullptr)
    return launch(dropout_flat_kernel<T>, dim3((unsigned)p.flat), dim3(kDThreads), 0, st, false, a);
  if (p.team > 0)
    return launch(dropout_team_kernel<T>, dim3((unsigned)p.team_blocks), dim3((unsigned)p.threads),
                  (size_t)(p.threads / p.team) * 8 * team_pitch(a.H) * (sizeof(T) == 4 ? 8 : 4), st,
                  false, a);
  const dim3 grid((unsigned)p.gx, (unsigned)p.slices);
  return bwd ? launch(dropout_tile_kernel<T, true>, grid, dim3(kDThreads), 0, st, false, a)
             : launch(dropout_tile_kernel<T, false>, grid, dim3(kDThreads), 0, st, false, a);
}

}  // namespace

RngArgs make_rng(double p, uint64_t seed, uint64_t offset, const uint64_t* state) {
  RngArgs r;
  r.seed = seed;
  r.offset = offset;
  r.state = state;
  const uint32_t thr = (uint32_t)((1.0 - p) * 65536.0 + 0.5);  // 0 .. 65536
  r.all = thr == 65536 ? 1u : 0u;
  r.lim = thr << 16;
  r.scale = thr ? (float)(65536.0 / (double)thr) : 0.f;
  return r;
}

cudaError_t drop_configure() {  // one long row's double-fp32 sums
  return cudaFuncSetAttribute(dropout_team_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              8 * kTeamMaxThreads * (int)sizeof(float2));
}

DropPlan drop_plan(int64_t R, int64_t H, bool fast_ok, int dtype, const DevInfo& dev) {
  DropPlan p;
  p.fast = fast_ok && H % 8 == 0;
  if (fast_ok && !p.fast) {
    // two chunks a thread at least, every resident block slot once
    const int64_t blocks = (R * H / 8 + 2 * kDThreads - 1) / (2 * kDThreads), cap = 4 * dev.sms;
    p.flat = (int)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
  }
  int64_t min_rows;
  if (p.fast) {
    // chunks of a block row: 32, 16 or 8 (at least 128 contiguous bytes),
    // whichever leaves the fewest idle threads, the widest on a tie; a narrower
    // row takes the power of two that holds it
    const int64_t Hc = H / 8;
    p.ltx = 5;
    auto padded = [Hc](int l) { return ((Hc + (1 << l) - 1) >> l) << l; };
    for (int l = 4; l >= 3; --l)
      if (padded(l) < padded(p.ltx)) p.ltx = l;
    while (p.ltx > 0 && Hc <= (1 << (p.ltx - 1))) --p.ltx;
    p.gx = (Hc + (1 << p.ltx) - 1) >> p.ltx;
    min_rows = 2 * (kDThreads >> p.ltx);  // two rows a thread, at least
  } else {
    p.gx = (H + kDTileCols - 1) / kDTileCols;
    min_rows = kDTileRows;
  }
  // every resident block slot once
  int64_t s = (int64_t)dev.sms * kDBlocksPerSm / p.gx;
  const int64_t by_rows = (R + min_rows - 1) / min_rows;
  if (s > by_rows) s = by_rows;
  if (s < 1) s = 1;
  if (s > 65535) s = 65535;
  p.slices = (int)s;
  if (fast_ok && !p.fast && H <= kTeamMaxH) {
    // two blocks of up to 512 threads an SM (one of a longer row's), a row a team
    // at least
    p.team = team_threads(H);
    const int most = p.team <= 512 ? 512 : kDTeamThreads;
    const int64_t cap = p.team <= 512 ? 2 * dev.sms : dev.sms;
    const int ty = teams_of_block(p.team, most, (R + cap - 1) / cap);
    p.threads = ty * p.team;
    const int64_t blocks = (R + ty - 1) / ty;
    p.team_blocks = (int)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
    if (s < p.team_blocks) s = p.team_blocks;
  }
  p.ws_bytes = ((size_t)(dtype == GBN_F32 ? 2 : 1) * (size_t)s * (size_t)H * 4 + 255) & ~(size_t)255;
  return p;
}

cudaError_t drop_forward(const DropPlan& p, int dtype, const void* x, const void* bias,
                         const void* res, void* y, int64_t R, int64_t H, const RngArgs& rng,
                         cudaStream_t st) {
  DropArgs a{x, res, bias, y, nullptr, R, (int32_t)H, (int32_t)(H / 8), p.ltx, p.slices, 0, rng};
  return dtype == GBN_F32 ? launch_drop<float>(p, a, false, st) : launch_drop<bf16>(p, a, false, st);
}

cudaError_t drop_backward(const DropPlan& p, int dtype, const void* dy, void* dx, void* dbias,
                          void* ws, int64_t R, int64_t H, const RngArgs& rng, cudaStream_t st) {
  DropArgs a{dy, nullptr, nullptr, dx, dbias ? static_cast<float*>(ws) : nullptr, R, (int32_t)H,
             (int32_t)(H / 8), p.ltx, p.slices, p.team, rng};
  cudaError_t e =
      dtype == GBN_F32 ? launch_drop<float>(p, a, true, st) : launch_drop<bf16>(p, a, true, st);
  if (e != cudaSuccess || dbias == nullptr) return e;
  void* outs[3] = {dbias, nullptr, nullptr};
  return colsum_launch(a.part, 1, dtype == GBN_F32 ? 2 : 1, p.team > 0 ? p.team_blocks : p.slices, H,
                       dtype, outs, st, true);
}

}  // namespace gbn
