// GroupNorm with an activation on channels-last tensors x[N, S, C] (S the
// flattened space, the channel innermost), training forward and backward.
// Group g of sample n holds S*Cg elements, Cg = C / G:
//   forward   mean, var over the group; pre = (x - mean)*rstd*gamma_c + beta_c,
//             y = act(pre)
//   backward  e = dy*act'(pre) (pre recomputed), xhat = (x - mean)*rstd,
//             dbeta_c = sum e, dgamma_c = sum e*xhat over samples and space,
//             dx = rstd*(gamma_c*e - k0 - xhat*k1) with k0, k1 the group means
//             of gamma_c*e and gamma_c*e*xhat.
//
// Bound: DRAM traffic, x (and dy) read once and the output written once; the
// second read of the inputs comes from L2 where they fit.
//
// Layout of a block: TX threads over 16-byte (or narrower) vectors of adjacent
// channels, TY thread rows down the block's slice of one sample's rows, so a
// warp reads contiguous bytes and a thread's channels never change.  A block
// covers a tile of at most 256 vectors; a group cut by a tile border simply has
// one partial in each tile (entry g + tile, unique because a border cuts at
// most one group).
//
// Statistics: a thread forms mean and centred sum of squares of each of its
// channels over a few rows held in registers (two passes over the registers),
// and merges such chunks pairwise (Chan, Golub, LeVeque, "Updating formulae and
// a pairwise algorithm for computing sample variances", 1979): no difference of
// large squares appears anywhere, whatever the first element is.  Means are
// kept relative to the sample's first row (x[n, 0, c]), so a large common
// offset costs nothing.  All combinations run in a fixed order: two runs give
// the same bits, and there are no atomics.
#include "gbn_common.cuh"
#include "gbn_internal.h"

namespace gbn {

namespace {

constexpr int kGThreads = 256;

struct GnGeom {
  int32_t S;          // rows per sample
  int32_t N, C, G, Cg;
  int32_t Cv;         // vectors per row
  int32_t TX, TY;     // block shape
  int32_t T;          // channel tiles
  int32_t slices;     // row slices per sample
  int32_t rps;        // rows per slice (the last may have fewer)
  int32_t E;          // group partials per (sample, slice): G + T - 1
  int32_t n0;         // first sample of this launch
};

struct GnArgs {
  const void* x;
  const void* dy;
  void* out;            // y or dx
  const float* gamma;   // null: ones
  const float* beta;    // null: zeros
  float* stats;         // [3][N][G]: mean, rstd, mean's low part
  float2* gpart;        // [N][slices][E]: forward (mean - shift, M2); backward sums
  float* cpart;         // backward: [2][2][N*slices][C] (dgamma, dbeta; hi, lo);
                        // forward: [N][G], the shifts (y may overwrite x's first row)
  GnGeom g;
  float eps, slope;
};

struct GnBlock {
  int n, slice, tile;
  int tx, ty;
  int cv;               // vector of this thread
  bool active;
  int r0, r1;           // rows of the slice
  int c0, c1;           // channels of the tile
  int g0, g1;           // groups with a channel in the tile
};

template <int VEC>
__device__ __forceinline__ GnBlock gn_block(const GnGeom& g) {
  GnBlock b;
  const uint32_t bi = blockIdx.x;
  const uint32_t q = bi / (uint32_t)g.T;
  b.tile = bi - q * g.T;
  const uint32_t n = q / (uint32_t)g.slices;
  b.slice = q - n * g.slices;
  b.n = g.n0 + (int)n;
  b.ty = (uint32_t)threadIdx.x / (uint32_t)g.TX;
  b.tx = threadIdx.x - b.ty * g.TX;
  b.cv = b.tile * g.TX + b.tx;
  b.active = b.ty < g.TY && b.cv < g.Cv;
  b.r0 = b.slice * g.rps;
  b.r1 = min(b.r0 + g.rps, g.S);
  b.c0 = b.tile * g.TX * VEC;
  b.c1 = min(b.c0 + g.TX * VEC, g.C);
  b.g0 = b.c0 / g.Cg;
  b.g1 = (b.c1 - 1) / g.Cg + 1;
  return b;
}

// ------------------------------------------------------------ activations --

template <int VEC> struct GnP {
  static constexpr int NP = (VEC + 1) / 2;  // packed pairs; VEC = 1 pads with 0
};
template <typename T, int VEC>
__device__ __forceinline__ void gn_pairs(typename Vec<T, VEC>::raw r, f2 (&p)[GnP<VEC>::NP]) {
  float v[VEC];
  Vec<T, VEC>::cvt(r, v);
#pragma unroll
  for (int k = 0; k < GnP<VEC>::NP; ++k) p[k] = f2_pack(v[2 * k], 2 * k + 1 < VEC ? v[2 * k + 1] : 0.f);
}
template <typename T, int VEC>
__device__ __forceinline__ void gn_store(T* p, const f2 (&o)[GnP<VEC>::NP]) {
  float v[VEC];
#pragma unroll
  for (int k = 0; k < GnP<VEC>::NP; ++k) {
    const float2 t = f2_unpack(o[k]);
    v[2 * k] = t.x;
    if (2 * k + 1 < VEC) v[2 * k + 1] = t.y;
  }
  Vec<T, VEC>::store(p, v);
}
template <int VEC>
__device__ __forceinline__ f2 gn_pair(const float (&v)[VEC], int k) {
  return f2_pack(v[2 * k], 2 * k + 1 < VEC ? v[2 * k + 1] : 0.f);
}

__device__ __forceinline__ float ex2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Sigmoid of a pair.  fp32 storage: expf and an IEEE division.  bf16 storage:
// the hardware exponential and reciprocal (a few 2^-22, far below bf16's 2^-9),
// and one reciprocal for both, 1/a = b/(a b): the special-function unit (16 a
// cycle and SM) would otherwise bound the backward, which evaluates the gate
// twice per element.  a b overflows only where both are below about -44 (a
// sigmoid of 1e-19), or one below -88: those pairs take two reciprocals.
template <typename T>
__device__ __forceinline__ f2 sigmoid2(f2 pre) {
  if constexpr (sizeof(T) == 4) {
    const float2 v = f2_unpack(pre);
    return f2_pack(1.f / (1.f + expf(-v.x)), 1.f / (1.f + expf(-v.y)));
  } else {
    const float2 m = f2_unpack(f2_mul(pre, f2_splat(-1.4426950408889634f)));
    const f2 ab = f2_add(f2_pack(ex2_fast(m.x), ex2_fast(m.y)), f2_splat(1.f));
    const float2 d = f2_unpack(ab);
    const float p = d.x * d.y;
    if (p < 1e37f) {
      const float r = rcp_fast(p);
      return f2_mul(f2_pack(d.y, d.x), f2_splat(r));
    }
    return f2_pack(rcp_fast(d.x), rcp_fast(d.y));
  }
}
template <typename T, int ACT>
__device__ __forceinline__ f2 gn_act(f2 pre, float slope) {
  if constexpr (ACT == GBN_ACT_SILU) {
    return f2_mul(pre, sigmoid2<T>(pre));
  } else if constexpr (ACT == GBN_ACT_NONE) {
    return pre;
  } else {
    const float2 v = f2_unpack(pre);
    return f2_pack(v.x > 0.f ? v.x : (ACT == GBN_ACT_RELU ? 0.f : v.x * slope),
                   v.y > 0.f ? v.y : (ACT == GBN_ACT_RELU ? 0.f : v.y * slope));
  }
}
// d * (d act / d pre)
template <typename T, int ACT>
__device__ __forceinline__ f2 gn_gated(f2 d, f2 pre, float slope) {
  if constexpr (ACT == GBN_ACT_SILU) {
    const f2 s = sigmoid2<T>(pre);
    const f2 w = f2_fma(s ^ 0x8000000080000000ull, s, s);  // s (1 - s)
    return f2_mul(d, f2_fma(pre, w, s));
  } else if constexpr (ACT == GBN_ACT_NONE) {
    return d;
  } else {
    const float2 v = f2_unpack(pre);
    const float neg = ACT == GBN_ACT_RELU ? 0.f : slope;
    return f2_mul(d, f2_pack(v.x > 0.f ? 1.f : neg, v.y > 0.f ? 1.f : neg));
  }
}

// ------------------------------------------------- merging of statistics --

// (n, mean, M2) of a set of values.
struct Mom {
  float n, mean, M2;
};
__device__ __forceinline__ void mom_add(Mom& a, const Mom& b) {
  const float n = a.n + b.n;
  if (b.n == 0.f) return;
  const float w = __fdividef(b.n, n), d = b.mean - a.mean;
  a.M2 = fmaf(d * d, a.n * w, a.M2 + b.M2);
  a.mean = fmaf(d, w, a.mean);
  a.n = n;
}

// Lanes that share a group's channels: the power of two that holds Cg, at most 32.
__device__ __forceinline__ int group_lanes(int Cg) {
  int l = 1;
  while (l < 32 && l < Cg) l *= 2;
  return l;
}

// ---------------------------------------------------------- statistics --

template <typename T, int VEC>
__global__ void __launch_bounds__(kGThreads, 3) gn_stats_kernel(GnArgs a) {
  constexpr int U = 8;  // rows of a chunk
  using V = Vec<T, VEC>;
  __shared__ float2 acc[kGThreads * VEC];  // [ty][channel of the tile]: mean - K, M2
  __shared__ float cnt[kGThreads];         // [ty]
  __shared__ float Ks[kGThreads * VEC];    // shifts: x[n, 0, c]
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  pdl_launch_dependents();
  const T* xs = static_cast<const T*>(a.x) + (int64_t)b.n * g.S * g.C;
  const int W = g.TX * VEC;  // channels of a full tile
  float cn = 0.f;
  if (b.active) {
    const T* p = xs + (int64_t)b.cv * VEC;
    float K[VEC], mean[VEC], M2[VEC];
    V::cvt(V::ld(p), K);
#pragma unroll
    for (int e = 0; e < VEC; ++e) mean[e] = M2[e] = 0.f;
    const int64_t step = (int64_t)g.TY * g.C;
    const T* q = p + (int64_t)(b.r0 + b.ty) * g.C;
    int left = b.r1 - b.r0 > b.ty ? (b.r1 - b.r0 - b.ty + g.TY - 1) / g.TY : 0;
    for (; left > 0; left -= U, q += U * step) {
      typename V::raw raw[U];
      const int m = min(left, U);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < m) raw[u] = V::ld(q + u * step);
      float cm[VEC], cs[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) cm[e] = cs[e] = 0.f;
      const float fm = (float)m, inv = __fdividef(1.f, fm);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < m) {
          float v[VEC];
          V::cvt(raw[u], v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) cm[e] += v[e] - K[e];
        }
#pragma unroll
      for (int e = 0; e < VEC; ++e) cm[e] *= inv;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < m) {
          float v[VEC];
          V::cvt(raw[u], v);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float d = (v[e] - K[e]) - cm[e];
            cs[e] = fmaf(d, d, cs[e]);
          }
        }
      const float tot = cn + fm, w = __fdividef(fm, tot), ww = cn * w;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = cm[e] - mean[e];
        mean[e] = fmaf(d, w, mean[e]);
        M2[e] = fmaf(d * d, ww, M2[e] + cs[e]);
      }
      cn = tot;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      acc[b.ty * W + b.tx * VEC + e] = make_float2(mean[e], M2[e]);
      if (b.ty == 0) Ks[b.tx * VEC + e] = K[e];
    }
    if (b.tx == 0) cnt[b.ty] = cn;
  }
  __syncthreads();
  // the thread rows of every channel
  int P = 1;
  while (P < g.TY) P *= 2;
  for (int step = P / 2; step >= 1; step /= 2) {
    float nn = 0.f;
    const bool on = b.active && b.ty < step && b.ty + step < g.TY;
    if (on) {
      const float n1 = cnt[b.ty + step];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = b.ty * W + b.tx * VEC + e;
        const float2 u = acc[i], v = acc[i + step * W];
        Mom m{cn, u.x, u.y};
        mom_add(m, Mom{n1, v.x, v.y});
        acc[i] = make_float2(m.mean, m.M2);
      }
      cn += n1;
      nn = cn;
    }
    __syncthreads();
    if (on && b.tx == 0) cnt[b.ty] = nn;
    __syncthreads();
  }
  // The channels of every group of the tile, relative to the group's first
  // channel in the tile: teams of lanes, two passes (equal counts).
  const int L = group_lanes(g.Cg), lane = threadIdx.x & (L - 1);
  const int teams = blockDim.x / L;
  const float rows = (float)(b.r1 - b.r0);
  for (int gb = b.g0; gb < b.g1; gb += teams) {
    const int gi = gb + threadIdx.x / L;
    const bool on = gi < b.g1;
    const int ca = on ? max(gi * g.Cg, b.c0) - b.c0 : 0;
    const int cb = on ? min((gi + 1) * g.Cg, b.c1) - b.c0 : 0;
    const float Kg = on ? Ks[ca] : 0.f;
    float s = 0.f;
    for (int c = ca + lane; c < cb; c += L) s += (Ks[c] - Kg) + acc[c].x;
    for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float nc = (float)(cb - ca), mean = s / nc;
    float q = 0.f;
    for (int c = ca + lane; c < cb; c += L) {
      const float d = ((Ks[c] - Kg) + acc[c].x) - mean;
      q += fmaf(rows * d, d, acc[c].y);
    }
    for (int o = L / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
    if (on && lane == 0) {
      // relative to the shift of the group's first channel overall
      const float K0 = gi * g.Cg >= b.c0 ? Kg : to_f32(xs[gi * g.Cg]);
      a.gpart[((int64_t)b.n * g.slices + b.slice) * g.E + gi + b.tile] =
          make_float2((Kg - K0) + mean, q);
      if (b.slice == 0 && gi * g.Cg >= b.c0) a.cpart[(int64_t)b.n * g.G + gi] = K0;
    }
  }
  pdl_wait();  // the previous launch of this call (another run of samples) is complete too
}

// Tiles that hold channels of group gi: first and one past the last.
template <int VEC>
__device__ __forceinline__ void gn_tiles_of(const GnGeom& g, int gi, int& t0, int& t1) {
  if (g.T == 1) {
    t0 = 0;
    t1 = 1;
    return;
  }
  const int W = g.TX * VEC;
  t0 = gi * g.Cg / W;
  t1 = ((gi + 1) * g.Cg - 1) / W + 1;
}

// Walks the partials of the tile's groups: thread row q of R takes slices q,
// q + R, ... of group gi = g0 + column, `take(partial, rows, channels)` per
// partial; `done(gi, q, R, on)` is called by every thread between barriers'
// needs (on: the thread has a group).  Groups beyond the block's width come in
// further rounds.
template <int VEC, typename Init, typename Take, typename Done>
__device__ __forceinline__ void gn_walk(const GnArgs& a, const GnBlock& b, Init init, Take take,
                                        Done done) {
  const GnGeom& g = a.g;
  const int ng = b.g1 - b.g0, cols = min(ng, (int)blockDim.x);
  const int R = blockDim.x / cols;
  const int q = (int)threadIdx.x / cols, col = threadIdx.x - q * cols;
  for (int gb = b.g0; gb < b.g1; gb += cols) {
    const int gi = gb + col;
    const bool on = q < R && gi < b.g1;
    init();
    if (on) {
      int t0, t1;
      gn_tiles_of<VEC>(g, gi, t0, t1);
      const int W = g.TX * VEC;
      const float2* part = a.gpart + (int64_t)b.n * g.slices * g.E + gi;
      for (int t = t0; t < t1; ++t) {
        const float ch = g.T == 1 ? (float)g.Cg
                                  : (float)(min((gi + 1) * g.Cg, (t + 1) * W) - max(gi * g.Cg, t * W));
        constexpr int U = 8;
        for (int j = q; j < g.slices; j += U * R) {
          float2 v[U];
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (j + u * R < g.slices) v[u] = __ldcg(part + (int64_t)(j + u * R) * g.E + t);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (j + u * R < g.slices) {
              const int rows = min(g.rps, g.S - (j + u * R) * g.rps);
              take(v[u], (float)rows, ch);
            }
        }
      }
    }
    done(gi, q, R, col, cols, on);
  }
}

// ---------------------------------------------------------------- apply --

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGThreads, 3) gn_apply_kernel(GnArgs a) {
  constexpr int U = 4;
  constexpr int NP = GnP<VEC>::NP;
  using V = Vec<T, VEC>;
  extern __shared__ float3 fin[];  // per group of the tile: mean hi, lo, rstd
  __shared__ Mom red[kGThreads];
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  const T* xs = static_cast<const T*>(a.x) + (int64_t)b.n * g.S * g.C;
  T* ys = static_cast<T*>(a.out) + (int64_t)b.n * g.S * g.C;
  pdl_wait();
  pdl_launch_dependents();
  Mom m{0.f, 0.f, 0.f};
  gn_walk<VEC>(
      a, b, [&] { m = Mom{0.f, 0.f, 0.f}; },
      [&](float2 v, float rows, float ch) { mom_add(m, Mom{rows * ch, v.x, v.y}); },
      [&](int gi, int q, int R, int col, int cols, bool on) {
        red[threadIdx.x] = m;
        __syncthreads();
        int P = 1;
        while (P < R) P *= 2;
        for (int step = P / 2; step >= 1; step /= 2) {
          if (on && q < step && q + step < R) {
            Mom t = red[q * cols + col];
            mom_add(t, red[(q + step) * cols + col]);
            red[q * cols + col] = t;
          }
          __syncthreads();
        }
        if (on && q == 0) {
          const Mom t = red[col];
          const DF mu = two_sum(__ldcg(a.cpart + (int64_t)b.n * g.G + gi), t.mean);
          const float rstd = 1.f / sqrtf(t.M2 / t.n + a.eps);
          fin[gi - b.g0] = make_float3(mu.hi, mu.lo, rstd);
          if (b.slice == 0 && gi * g.Cg >= b.c0) {
            const int64_t o = (int64_t)b.n * g.G + gi, ng = (int64_t)g.N * g.G;
            a.stats[o] = mu.hi;
            a.stats[ng + o] = rstd;
            a.stats[2 * ng + o] = mu.lo;
          }
        }
        __syncthreads();
      });
  if (!b.active) return;
  f2 nm[NP], sc[NP], be[NP];
  {
    float m0[VEC], m1[VEC], m2[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = b.cv * VEC + e;
      const float3 f = fin[c / g.Cg - b.g0];
      m0[e] = f.x;
      m1[e] = f.z * (a.gamma ? a.gamma[c] : 1.f);
      m2[e] = fmaf(-f.y, m1[e], a.beta ? a.beta[c] : 0.f);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      nm[k] = gn_pair(m0, k);
      sc[k] = gn_pair(m1, k);
      be[k] = gn_pair(m2, k);
    }
  }
  // from the slice's end: what the statistics pass read last is likeliest in L2
  const int64_t step = (int64_t)g.TY * g.C;
  int left = b.r1 - b.r0 > b.ty ? (b.r1 - b.r0 - b.ty + g.TY - 1) / g.TY : 0;
  int64_t o = (int64_t)(b.r0 + b.ty) * g.C + (int64_t)(left - 1) * step + (int64_t)b.cv * VEC;
  for (; left > 0; left -= U, o -= U * step) {
    typename V::raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < left) raw[u] = V::ld(xs + o - u * step);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < left) {
        f2 v[NP];
        gn_pairs<T, VEC>(raw[u], v);
#pragma unroll
        for (int k = 0; k < NP; ++k)
          v[k] = gn_act<T, ACT>(f2_fma(f2_sub(v[k], nm[k]), sc[k], be[k]), a.slope);
        gn_store<T, VEC>(ys + o - u * step, v);
      }
  }
}

// -------------------------------------------------------- backward sums --

// Running sum of pairs: fp32 storage carries the errors (its weight gradients
// are fp32 results of fp32 data), bf16 adds plain fp32 sums of a few rows.
template <typename T> struct GnSum {
  DF2 s{0ull, 0ull};
  __device__ __forceinline__ void add(f2 v) {
    if constexpr (sizeof(T) == 4) df2_add(s, v);
    else s.hi = f2_add(s.hi, v);
  }
};

// Per channel of the tile: sum e and sum e*xhat of the block's rows, to the
// column partials; and per group the sums of gamma*e and gamma*e*xhat.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGThreads, 2) gn_sums_kernel(GnArgs a) {
  constexpr int U = 4;  // rows in flight (two inputs)
  constexpr int NP = GnP<VEC>::NP;
  using V = Vec<T, VEC>;
  __shared__ DF sa[kGThreads * VEC], sb[kGThreads * VEC];  // [ty][channel]
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  pdl_launch_dependents();
  const int64_t off = (int64_t)b.n * g.S * g.C;
  const T* xs = static_cast<const T*>(a.x) + off;
  const T* ds = static_cast<const T*>(a.dy) + off;
  const int W = g.TX * VEC;
  const int64_t ng = (int64_t)g.N * g.G, so = (int64_t)b.n * g.G;
  if (b.active) {
    f2 nm[NP], sc[NP], be[NP];
    GnSum<T> A[NP], B[NP];
    {
      float m0[VEC], m1[VEC], m2[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = b.cv * VEC + e, gi = c / g.Cg;
        m0[e] = a.stats[so + gi];
        m1[e] = a.stats[ng + so + gi] * (a.gamma ? a.gamma[c] : 1.f);
        m2[e] = fmaf(-a.stats[2 * ng + so + gi], m1[e], a.beta ? a.beta[c] : 0.f);
      }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        nm[k] = gn_pair(m0, k);
        sc[k] = gn_pair(m1, k);
        be[k] = gn_pair(m2, k);
      }
    }
    const int64_t step = (int64_t)g.TY * g.C;
    int64_t o = (int64_t)(b.r0 + b.ty) * g.C + (int64_t)b.cv * VEC;
    int left = b.r1 - b.r0 > b.ty ? (b.r1 - b.r0 - b.ty + g.TY - 1) / g.TY : 0;
    for (; left > 0; left -= U, o += U * step) {
      typename V::raw rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < left) {
          rx[u] = V::ld(xs + o + u * step);
          rd[u] = V::ld(ds + o + u * step);
        }
      f2 ca[NP], cb[NP];
#pragma unroll
      for (int k = 0; k < NP; ++k) ca[k] = cb[k] = 0ull;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < left) {
          f2 v[NP], d[NP];
          gn_pairs<T, VEC>(rx[u], v);
          gn_pairs<T, VEC>(rd[u], d);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            const f2 xc = f2_sub(v[k], nm[k]);
            const f2 t = gn_gated<T, ACT>(d[k], f2_fma(xc, sc[k], be[k]), a.slope);
            ca[k] = f2_add(ca[k], t);
            cb[k] = f2_fma(t, xc, cb[k]);
          }
        }
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        A[k].add(ca[k]);
        B[k].add(cb[k]);
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = b.ty * W + b.tx * VEC + e;
      const float2 ah = f2_unpack(A[e / 2].s.hi), al = f2_unpack(A[e / 2].s.lo);
      const float2 bh = f2_unpack(B[e / 2].s.hi), bl = f2_unpack(B[e / 2].s.lo);
      sa[i] = (e & 1) ? DF{ah.y, al.y} : DF{ah.x, al.x};
      sb[i] = (e & 1) ? DF{bh.y, bl.y} : DF{bh.x, bl.x};
    }
  }
  __syncthreads();
  int P = 1;
  while (P < g.TY) P *= 2;
  for (int step = P / 2; step >= 1; step /= 2) {
    if (b.active && b.ty < step && b.ty + step < g.TY) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int i = b.ty * W + b.tx * VEC + e, j = i + step * W;
        sa[i] = df_sum(sa[i], sa[j]);
        sb[i] = df_sum(sb[i], sb[j]);
      }
    }
    __syncthreads();
  }
  // sum e*xhat = rstd*(sum e*(x - mean_hi) - mean_lo*sum e)
  const int64_t row = (int64_t)b.n * g.slices + b.slice, rows = (int64_t)g.N * g.slices;
  for (int k = threadIdx.x; k < b.c1 - b.c0; k += blockDim.x) {
    const int c = b.c0 + k, gi = c / g.Cg;
    const DF A = sa[k];
    const DF dg = df_norm(df_mul(df_sum(sb[k], df_neg(df_mul(A, a.stats[2 * ng + so + gi]))),
                                 a.stats[ng + so + gi]));
    float* p = a.cpart + row * g.C + c;
    p[0] = dg.hi;
    p[rows * g.C] = dg.lo;
    p[2 * rows * g.C] = A.hi;
    p[3 * rows * g.C] = A.lo;
    const float gm = a.gamma ? a.gamma[c] : 1.f;
    sa[k] = DF{gm * df_round(A), gm * df_round(dg)};
  }
  __syncthreads();
  const int L = group_lanes(g.Cg), lane = threadIdx.x & (L - 1);
  const int teams = blockDim.x / L;
  for (int gb = b.g0; gb < b.g1; gb += teams) {
    const int gi = gb + threadIdx.x / L;
    const bool on = gi < b.g1;
    const int ca = on ? max(gi * g.Cg, b.c0) - b.c0 : 0;
    const int cb = on ? min((gi + 1) * g.Cg, b.c1) - b.c0 : 0;
    float s = 0.f, q = 0.f;
    for (int c = ca + lane; c < cb; c += L) {
      s += sa[c].hi;
      q += sa[c].lo;
    }
    for (int o = L / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      q += __shfl_xor_sync(0xffffffffu, q, o);
    }
    if (on && lane == 0) a.gpart[row * g.E + gi + b.tile] = make_float2(s, q);
  }
  pdl_wait();  // the previous launch of this call (another run of samples) is complete too
}

// ------------------------------------------------------------------- dx --

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGThreads, 2) gn_dx_kernel(GnArgs a) {
  constexpr int U = 4;
  constexpr int NP = GnP<VEC>::NP;
  using V = Vec<T, VEC>;
  extern __shared__ float2 kk[];  // per group of the tile: k0, k1
  __shared__ float2 red[kGThreads];
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  const int64_t off = (int64_t)b.n * g.S * g.C;
  const T* xs = static_cast<const T*>(a.x) + off;
  const T* ds = static_cast<const T*>(a.dy) + off;
  T* os = static_cast<T*>(a.out) + off;
  const int64_t ng = (int64_t)g.N * g.G, so = (int64_t)b.n * g.G;
  pdl_wait();
  pdl_launch_dependents();
  float2 m = make_float2(0.f, 0.f);
  gn_walk<VEC>(
      a, b, [&] { m = make_float2(0.f, 0.f); },
      [&](float2 v, float, float) {
        m.x += v.x;
        m.y += v.y;
      },
      [&](int gi, int q, int R, int col, int cols, bool on) {
        red[threadIdx.x] = m;
        __syncthreads();
        int P = 1;
        while (P < R) P *= 2;
        for (int step = P / 2; step >= 1; step /= 2) {
          if (on && q < step && q + step < R) {
            const float2 u = red[q * cols + col], v = red[(q + step) * cols + col];
            red[q * cols + col] = make_float2(u.x + v.x, u.y + v.y);
          }
          __syncthreads();
        }
        if (on && q == 0) {
          const float inv = 1.f / ((float)g.S * (float)g.Cg);
          kk[gi - b.g0] = make_float2(red[col].x * inv, red[col].y * inv);
        }
        __syncthreads();
      });
  if (!b.active) return;
  // dx = sc*e + (x - mean_hi)*q1 + q0
  f2 nm[NP], sc[NP], be[NP], q1[NP], q0[NP];
  {
    float m0[VEC], m1[VEC], m2[VEC], m3[VEC], m4[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = b.cv * VEC + e, gi = c / g.Cg;
      const float rstd = a.stats[ng + so + gi], ml = a.stats[2 * ng + so + gi];
      const float2 k = kk[gi - b.g0];
      m0[e] = a.stats[so + gi];
      m1[e] = rstd * (a.gamma ? a.gamma[c] : 1.f);
      m2[e] = fmaf(-ml, m1[e], a.beta ? a.beta[c] : 0.f);
      m3[e] = -(rstd * rstd) * k.y;
      m4[e] = -fmaf(ml, m3[e], rstd * k.x);
    }
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      nm[k] = gn_pair(m0, k);
      sc[k] = gn_pair(m1, k);
      be[k] = gn_pair(m2, k);
      q1[k] = gn_pair(m3, k);
      q0[k] = gn_pair(m4, k);
    }
  }
  const int64_t step = (int64_t)g.TY * g.C;
  int left = b.r1 - b.r0 > b.ty ? (b.r1 - b.r0 - b.ty + g.TY - 1) / g.TY : 0;
  int64_t o = (int64_t)(b.r0 + b.ty) * g.C + (int64_t)(left - 1) * step + (int64_t)b.cv * VEC;
  for (; left > 0; left -= U, o -= U * step) {
    typename V::raw rx[U], rd[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < left) {
        rx[u] = V::ld(xs + o - u * step);
        rd[u] = V::ld(ds + o - u * step);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < left) {
        f2 v[NP], d[NP];
        gn_pairs<T, VEC>(rx[u], v);
        gn_pairs<T, VEC>(rd[u], d);
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const f2 xc = f2_sub(v[k], nm[k]);
          const f2 t = gn_gated<T, ACT>(d[k], f2_fma(xc, sc[k], be[k]), a.slope);
          v[k] = f2_fma(t, sc[k], f2_fma(xc, q1[k], q0[k]));
        }
        gn_store<T, VEC>(os + o - u * step, v);
      }
  }
}

// ----------------------------------------------------------------- host --

enum GnKernel { kGnStats, kGnApply, kGnSums, kGnDx };

template <typename T, int VEC, int ACT>
cudaError_t gn_run(GnKernel k, const GnPlan& p, const GnArgs& a, cudaStream_t st) {
  const bool chained = a.g.n0 > 0;  // not the call's first launch
  const int64_t n = p.N - a.g.n0 < p.run ? p.N - a.g.n0 : p.run;
  const dim3 grid((unsigned)(n * p.slices * p.tiles)), block((unsigned)p.threads);
  const size_t smem = (size_t)p.tile_groups;
  switch (k) {
    case kGnStats: return launch(gn_stats_kernel<T, VEC>, grid, block, 0, st, chained, a);
    case kGnApply:
      return launch(gn_apply_kernel<T, VEC, ACT>, grid, block, smem * sizeof(float3), st, true, a);
    case kGnSums: return launch(gn_sums_kernel<T, VEC, ACT>, grid, block, 0, st, chained, a);
    default:
      return launch(gn_dx_kernel<T, VEC, ACT>, grid, block, smem * sizeof(float2), st, true, a);
  }
}
template <typename T, int VEC>
cudaError_t gn_run_act(GnKernel k, int act, const GnPlan& p, const GnArgs& a, cudaStream_t st) {
  switch (act) {
    case GBN_ACT_RELU: return gn_run<T, VEC, GBN_ACT_RELU>(k, p, a, st);
    case GBN_ACT_LEAKY_RELU: return gn_run<T, VEC, GBN_ACT_LEAKY_RELU>(k, p, a, st);
    case GBN_ACT_SILU: return gn_run<T, VEC, GBN_ACT_SILU>(k, p, a, st);
    default: return gn_run<T, VEC, GBN_ACT_NONE>(k, p, a, st);
  }
}
cudaError_t gn_dispatch(GnKernel k, int dtype, int act, const GnPlan& p, const GnArgs& a,
                        cudaStream_t st) {
  if (dtype == GBN_F32) {
    switch (p.vec) {
      case 4: return gn_run_act<float, 4>(k, act, p, a, st);
      case 2: return gn_run_act<float, 2>(k, act, p, a, st);
      default: return gn_run_act<float, 1>(k, act, p, a, st);
    }
  }
  switch (p.vec) {
    case 8: return gn_run_act<bf16, 8>(k, act, p, a, st);
    case 4: return gn_run_act<bf16, 4>(k, act, p, a, st);
    case 2: return gn_run_act<bf16, 2>(k, act, p, a, st);
    default: return gn_run_act<bf16, 1>(k, act, p, a, st);
  }
}

GnArgs gn_args(const GnPlan& p, void* ws) {
  GnArgs a{};
  a.g.S = (int32_t)p.S;
  a.g.N = (int32_t)p.N;
  a.g.C = (int32_t)p.C;
  a.g.G = (int32_t)p.G;
  a.g.Cg = (int32_t)(p.C / p.G);
  a.g.Cv = (int32_t)(p.C / p.vec);
  a.g.TX = p.TX;
  a.g.TY = p.TY;
  a.g.T = p.tiles;
  a.g.slices = p.slices;
  a.g.rps = p.rps;
  a.g.E = (int32_t)(p.G + p.tiles - 1);
  a.gpart = static_cast<float2*>(ws);
  a.cpart = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + p.gpart_bytes);
  return a;
}

}  // namespace

bool gn_plan(int64_t N, int64_t S, int64_t C, int64_t G, int vec, int64_t esize, bool backward,
             const DevInfo& dev, GnPlan* p) {
  *p = GnPlan();
  p->N = N;
  p->S = S;
  p->C = C;
  p->G = G;
  p->vec = vec;
  const int64_t Cv = C / vec;
  p->tiles = (int)((Cv + kGThreads - 1) / kGThreads);
  p->TX = (int)((Cv + p->tiles - 1) / p->tiles);
  p->tiles = (int)((Cv + p->TX - 1) / p->TX);
  p->TY = kGThreads / p->TX;
  if (p->TY > S) p->TY = (int)S;
  p->threads = (p->TX * p->TY + 31) / 32 * 32;
  const int64_t W = (int64_t)p->TX * vec, Cg = C / G;
  p->tile_groups = (int)((W + Cg - 1) / Cg + 1);
  // Samples per pair of launches: runs whose inputs stay in half of L2 between
  // the two passes, so the second one reads no DRAM.
  const int64_t sample = S * C * esize * (backward ? 2 : 1);
  int64_t run = (int64_t)dev.l2_bytes / 2 / (sample > 0 ? sample : 1);
  if (run < 1) run = 1;
  if (run > N) run = N;
  run = (N + (N + run - 1) / run - 1) / ((N + run - 1) / run);  // even runs
  p->run = run;
  // the resident block slots once over a run's samples, at least one round of
  // loads a thread
  const int64_t slots = (int64_t)dev.sms * (backward ? 2 : 3);
  const int64_t per = (slots + run * p->tiles - 1) / (run * p->tiles);
  const int64_t round = (int64_t)p->TY * (backward ? 4 : 8);
  const int64_t rounds = (S + round - 1) / round;
  int64_t s = per < rounds ? per : rounds;
  if (s < 1) s = 1;
  p->rps = (int)((S + s - 1) / s);
  s = (S + p->rps - 1) / p->rps;
  p->slices = (int)s;
  if (run * s * p->tiles > INT32_MAX) return false;
  p->gpart_bytes = ((size_t)N * s * (G + p->tiles - 1) * sizeof(float2) + 255) & ~(size_t)255;
  const size_t rest = backward ? (size_t)4 * N * s * C : (size_t)N * G;
  p->ws_bytes = p->gpart_bytes + ((rest * sizeof(float) + 255) & ~(size_t)255);
  return true;
}

size_t gn_ws_bound(int64_t N, int64_t S, int64_t C, int64_t G, const DevInfo& dev) {
  size_t most = 256;
  for (int vec : {1, 2, 4, 8})
    for (int64_t es : {2, 4})
      for (bool bwd : {false, true}) {
        GnPlan p;
        if (C % vec == 0 && gn_plan(N, S, C, G, vec, es, bwd, dev, &p) && p.ws_bytes > most)
          most = p.ws_bytes;
      }
  return most;
}

cudaError_t gn_forward(const GnPlan& p, int dtype, const void* x, const float* gamma,
                       const float* beta, float eps, int act, float slope, void* y, float* stats,
                       void* ws, cudaStream_t st) {
  GnArgs a = gn_args(p, ws);
  a.x = x;
  a.out = y;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = stats;
  a.eps = eps;
  a.slope = slope;
  cudaError_t e = cudaSuccess;
  for (int64_t n = 0; n < p.N && e == cudaSuccess; n += p.run) {
    a.g.n0 = (int32_t)n;
    e = gn_dispatch(kGnStats, dtype, GBN_ACT_NONE, p, a, st);
    if (e == cudaSuccess) e = gn_dispatch(kGnApply, dtype, act, p, a, st);
  }
  return e;
}

cudaError_t gn_backward(const GnPlan& p, int dtype, const void* x, const void* dy,
                        const float* stats, const float* gamma, const float* beta, int act,
                        float slope, void* dx, float* dgamma, float* dbeta, void* ws,
                        cudaStream_t st) {
  GnArgs a = gn_args(p, ws);
  a.x = x;
  a.dy = dy;
  a.out = dx;
  a.gamma = gamma;
  a.beta = beta;
  a.stats = const_cast<float*>(stats);
  a.slope = slope;
  cudaError_t e = cudaSuccess;
  for (int64_t n = 0; n < p.N && e == cudaSuccess; n += p.run) {
    a.g.n0 = (int32_t)n;
    e = gn_dispatch(kGnSums, dtype, act, p, a, st);
    if (e == cudaSuccess) e = gn_dispatch(kGnDx, dtype, act, p, a, st);
  }
  if (e != cudaSuccess || (dgamma == nullptr && dbeta == nullptr)) return e;
  void* outs[3] = {dgamma, dbeta, nullptr};
  return colsum_launch(a.cpart, 2, 2, (int)(p.N * p.slices), p.C, GBN_F32, outs, st, true);
}

}  // namespace gbn
