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
  int64_t S;          // rows per sample
  int32_t N, C, G, Cg;
  int32_t Cv;         // vectors per row
  int32_t TX, TY;     // block shape
  int32_t T;          // channel tiles
  int32_t slices;     // row slices per sample
  int32_t E;          // group partials per (sample, slice): G + T - 1
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
  int64_t r0, r1;       // rows of the slice
  int c0, c1;           // channels of the tile
  int g0, g1;           // groups with a channel in the tile
};

template <int VEC>
__device__ __forceinline__ GnBlock gn_block(const GnGeom& g) {
  GnBlock b;
  const uint32_t bi = blockIdx.x;
  const uint32_t q = bi / g.T;
  b.tile = bi - q * g.T;
  b.n = q / g.slices;
  b.slice = q - b.n * g.slices;
  b.tx = threadIdx.x % g.TX;
  b.ty = threadIdx.x / g.TX;
  b.cv = b.tile * g.TX + b.tx;
  b.active = b.ty < g.TY && b.cv < g.Cv;
  b.r0 = g.S * b.slice / g.slices;
  b.r1 = g.S * (b.slice + 1) / g.slices;
  b.c0 = b.tile * g.TX * VEC;
  const int64_t c1 = (int64_t)(b.tile + 1) * g.TX * VEC;
  b.c1 = c1 < g.C ? (int)c1 : g.C;
  b.g0 = b.c0 / g.Cg;
  b.g1 = (b.c1 - 1) / g.Cg + 1;
  return b;
}

// Rows of thread row ty in rows [r0, r1).
__device__ __forceinline__ int64_t rows_of(int64_t r0, int64_t r1, int ty, int TY) {
  const int64_t n = r1 - r0 - ty;
  return n > 0 ? (n + TY - 1) / TY : 0;
}

// sigmoid.  bf16 storage: the fast exponential and division (a few 2^-23, far
// below bf16's 2^-9); fp32 storage: the accurate ones.
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-v));
  else return 1.f / (1.f + expf(-v));
}
template <typename T, int ACT>
__device__ __forceinline__ float gn_act(float pre, float slope) {
  if constexpr (ACT == GBN_ACT_SILU) return pre * sigmoid<T>(pre);
  else if constexpr (ACT == GBN_ACT_NONE) return pre;
  else return pre > 0.f ? pre : (ACT == GBN_ACT_RELU ? 0.f : pre * slope);
}
// d act / d pre
template <typename T, int ACT>
__device__ __forceinline__ float gn_gate(float pre, float slope) {
  if constexpr (ACT == GBN_ACT_SILU) {
    const float s = sigmoid<T>(pre);
    return s * fmaf(pre, 1.f - s, 1.f);
  } else if constexpr (ACT == GBN_ACT_NONE) {
    return 1.f;
  } else {
    return pre > 0.f ? 1.f : (ACT == GBN_ACT_RELU ? 0.f : slope);
  }
}

// ---------------------------------------------------------- statistics --

template <typename T, int VEC>
__global__ void __launch_bounds__(kGThreads) gn_stats_kernel(GnArgs a) {
  constexpr int U = 8;  // rows of a chunk
  using V = Vec<T, VEC>;
  __shared__ float2 acc[kGThreads * VEC];  // [ty][channel of the tile]: mean - K, M2
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  pdl_launch_dependents();
  const T* xs = static_cast<const T*>(a.x) + (int64_t)b.n * g.S * g.C;
  const int W = g.TX * VEC;  // channels of a full tile
  if (b.active) {
    const T* p = xs + (int64_t)b.cv * VEC;
    float K[VEC], mean[VEC], M2[VEC];
    V::cvt(V::ld(p), K);
#pragma unroll
    for (int e = 0; e < VEC; ++e) mean[e] = M2[e] = 0.f;
    float cnt = 0.f;
    for (int64_t r = b.r0 + b.ty; r < b.r1; r += (int64_t)U * g.TY) {
      typename V::raw raw[U];
      int m = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t ru = r + (int64_t)u * g.TY;
        if (ru < b.r1) {
          raw[u] = V::ld(p + ru * g.C);
          m = u + 1;
        }
      }
      float cm[VEC], cs[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) cm[e] = cs[e] = 0.f;
      const float fm = (float)m, inv = 1.f / fm;
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
      const float tot = cnt + fm, w = fm / tot, ww = cnt * w;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = cm[e] - mean[e];
        mean[e] = fmaf(d, w, mean[e]);
        M2[e] = fmaf(d * d, ww, M2[e] + cs[e]);
      }
      cnt = tot;
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      acc[b.ty * W + b.tx * VEC + e] = make_float2(mean[e], M2[e]);
  }
  __syncthreads();
  // One warp per group of the tile: the (thread row, channel) pairs, means
  // relative to the group's first channel in the sample's first row.
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const float rows = (float)(b.r1 - b.r0);
  for (int gi = b.g0 + (threadIdx.x >> 5); gi < b.g1; gi += nw) {
    const int ca = gi * g.Cg > b.c0 ? gi * g.Cg : b.c0;
    const int cb = (gi + 1) * g.Cg < b.c1 ? (gi + 1) * g.Cg : b.c1;
    const int nc = cb - ca, np = nc * g.TY;
    const float Kg = to_f32(xs[gi * g.Cg]);
    float s = 0.f;
    for (int k = lane; k < np; k += 32) {
      const int ty = k / nc, c = ca + (k - ty * nc);
      const float n = (float)rows_of(b.r0, b.r1, ty, g.TY);
      s = fmaf(n, (to_f32(xs[c]) - Kg) + acc[ty * W + (c - b.c0)].x, s);
    }
    const float mean = warp_sum(s) / (rows * (float)nc);
    float q = 0.f;
    for (int k = lane; k < np; k += 32) {
      const int ty = k / nc, c = ca + (k - ty * nc);
      const float n = (float)rows_of(b.r0, b.r1, ty, g.TY);
      const float2 v = acc[ty * W + (c - b.c0)];
      const float d = ((to_f32(xs[c]) - Kg) + v.x) - mean;
      q += fmaf(n * d, d, v.y);
    }
    q = warp_sum(q);
    if (lane == 0) {
      a.gpart[((int64_t)b.n * g.slices + b.slice) * g.E + gi + b.tile] = make_float2(mean, q);
      if (b.slice == 0 && gi * g.Cg >= b.c0) a.cpart[(int64_t)b.n * g.G + gi] = Kg;
    }
  }
}

// Tiles that hold channels of group gi: first and one past the last.
template <int VEC>
__device__ __forceinline__ void gn_tiles_of(const GnGeom& g, int gi, int& t0, int& t1) {
  const int W = g.TX * VEC;
  t0 = gi * g.Cg / W;
  t1 = ((gi + 1) * g.Cg - 1) / W + 1;
}

// Channels of group gi inside tile t.
template <int VEC>
__device__ __forceinline__ int gn_overlap(const GnGeom& g, int gi, int t) {
  const int W = g.TX * VEC;
  const int a = max(gi * g.Cg, t * W), b = min((gi + 1) * g.Cg, (t + 1) * W);
  return b - a;
}

// ---------------------------------------------------------------- apply --

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGThreads) gn_apply_kernel(GnArgs a) {
  constexpr int U = 8;
  using V = Vec<T, VEC>;
  extern __shared__ float3 fin[];  // per group of the tile: mean hi, lo, rstd
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  const T* xs = static_cast<const T*>(a.x) + (int64_t)b.n * g.S * g.C;
  T* ys = static_cast<T*>(a.out) + (int64_t)b.n * g.S * g.C;
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  pdl_wait();
  // finalize: one warp per group over its slices (and tiles)
  for (int gi = b.g0 + (threadIdx.x >> 5); gi < b.g1; gi += nw) {
    int t0, t1;
    gn_tiles_of<VEC>(g, gi, t0, t1);
    const int nt = t1 - t0, np = nt * g.slices;
    const float2* part = a.gpart + (int64_t)b.n * g.slices * g.E + gi;
    const float cnt = (float)g.S * (float)g.Cg;
    float s = 0.f;
    for (int k = lane; k < np; k += 32) {
      const int j = k / nt, t = t0 + (k - j * nt);
      const float n = (float)(g.S * (j + 1) / g.slices - g.S * j / g.slices) *
                      (float)gn_overlap<VEC>(g, gi, t);
      s = fmaf(n, part[(int64_t)j * g.E + t].x, s);
    }
    const float md = warp_sum(s) / cnt;
    float q = 0.f;
    for (int k = lane; k < np; k += 32) {
      const int j = k / nt, t = t0 + (k - j * nt);
      const float n = (float)(g.S * (j + 1) / g.slices - g.S * j / g.slices) *
                      (float)gn_overlap<VEC>(g, gi, t);
      const float2 v = part[(int64_t)j * g.E + t];
      const float d = v.x - md;
      q += fmaf(n * d, d, v.y);
    }
    const float var = warp_sum(q) / cnt;
    if (lane == 0) {
      const DF m = two_sum(a.cpart[(int64_t)b.n * g.G + gi], md);
      const float rstd = 1.f / sqrtf(var + a.eps);
      fin[gi - b.g0] = make_float3(m.hi, m.lo, rstd);
      if (b.slice == 0 && b.tile == t0) {
        const int64_t o = (int64_t)b.n * g.G + gi, ng = (int64_t)g.N * g.G;
        a.stats[o] = m.hi;
        a.stats[ng + o] = rstd;
        a.stats[2 * ng + o] = m.lo;
      }
    }
  }
  __syncthreads();
  if (!b.active) return;
  float mh[VEC], sc[VEC], be[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const int c = b.cv * VEC + e;
    const float3 f = fin[c / g.Cg - b.g0];
    mh[e] = f.x;
    sc[e] = f.z * (a.gamma ? a.gamma[c] : 1.f);
    be[e] = fmaf(-f.y, sc[e], a.beta ? a.beta[c] : 0.f);
  }
  // from the slice's end: what the statistics pass read last is likeliest in L2
  const int64_t nr = rows_of(b.r0, b.r1, b.ty, g.TY);
  for (int64_t jb = nr - 1; jb >= 0; jb -= U) {
    typename V::raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (jb - u >= 0)
        raw[u] = V::ld(xs + (b.r0 + b.ty + (jb - u) * g.TY) * g.C + (int64_t)b.cv * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (jb - u >= 0) {
        float v[VEC];
        V::cvt(raw[u], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          v[e] = gn_act<T, ACT>(fmaf(v[e] - mh[e], sc[e], be[e]), a.slope);
        V::store(ys + (b.r0 + b.ty + (jb - u) * g.TY) * g.C + (int64_t)b.cv * VEC, v);
      }
  }
}

// -------------------------------------------------------- backward sums --

// Per channel of the tile: sum e and sum e*xhat of the block's rows, to the
// column partials; and per group the sums of gamma*e and gamma*e*xhat.
template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGThreads, 2) gn_sums_kernel(GnArgs a) {
  constexpr int U = 4;  // rows in flight (two inputs)
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
    float mh[VEC], sc[VEC], be[VEC];
    DF A[VEC], B[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = b.cv * VEC + e, gi = c / g.Cg;
      mh[e] = a.stats[so + gi];
      sc[e] = a.stats[ng + so + gi] * (a.gamma ? a.gamma[c] : 1.f);
      be[e] = fmaf(-a.stats[2 * ng + so + gi], sc[e], a.beta ? a.beta[c] : 0.f);
      A[e] = B[e] = DF{0.f, 0.f};
    }
    for (int64_t r = b.r0 + b.ty; r < b.r1; r += (int64_t)U * g.TY) {
      typename V::raw rx[U], rd[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t ru = r + (int64_t)u * g.TY;
        if (ru < b.r1) {
          rx[u] = V::ld(xs + ru * g.C + (int64_t)b.cv * VEC);
          rd[u] = V::ld(ds + ru * g.C + (int64_t)b.cv * VEC);
        }
      }
      float ca[VEC], cb[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) ca[e] = cb[e] = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (r + (int64_t)u * g.TY < b.r1) {
          float v[VEC], d[VEC];
          V::cvt(rx[u], v);
          V::cvt(rd[u], d);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float xc = v[e] - mh[e];
            float t = d[e];
            if constexpr (ACT != GBN_ACT_NONE) t *= gn_gate<T, ACT>(fmaf(xc, sc[e], be[e]), a.slope);
            ca[e] += t;
            cb[e] = fmaf(t, xc, cb[e]);
          }
        }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        df_add(A[e], ca[e]);
        df_add(B[e], cb[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      sa[b.ty * W + b.tx * VEC + e] = A[e];
      sb[b.ty * W + b.tx * VEC + e] = B[e];
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
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  for (int gi = b.g0 + (threadIdx.x >> 5); gi < b.g1; gi += nw) {
    const int ca = max(gi * g.Cg, b.c0), cb = min((gi + 1) * g.Cg, b.c1);
    float s = 0.f, q = 0.f;
    for (int c = ca + lane; c < cb; c += 32) {
      s += sa[c - b.c0].hi;
      q += sa[c - b.c0].lo;
    }
    s = warp_sum(s);
    q = warp_sum(q);
    if (lane == 0) a.gpart[row * g.E + gi + b.tile] = make_float2(s, q);
  }
}

// ------------------------------------------------------------------- dx --

template <typename T, int VEC, int ACT>
__global__ void __launch_bounds__(kGThreads, 2) gn_dx_kernel(GnArgs a) {
  constexpr int U = 4;
  using V = Vec<T, VEC>;
  extern __shared__ float2 kk[];  // per group of the tile: k0, k1
  const GnGeom& g = a.g;
  const GnBlock b = gn_block<VEC>(g);
  const int64_t off = (int64_t)b.n * g.S * g.C;
  const T* xs = static_cast<const T*>(a.x) + off;
  const T* ds = static_cast<const T*>(a.dy) + off;
  T* os = static_cast<T*>(a.out) + off;
  const int64_t ng = (int64_t)g.N * g.G, so = (int64_t)b.n * g.G;
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  for (int gi = b.g0 + (threadIdx.x >> 5); gi < b.g1; gi += nw) {
    int t0, t1;
    gn_tiles_of<VEC>(g, gi, t0, t1);
    const int nt = t1 - t0, np = nt * g.slices;
    const float2* part = a.gpart + (int64_t)b.n * g.slices * g.E + gi;
    float s = 0.f, q = 0.f;
    for (int k = lane; k < np; k += 32) {
      const int j = k / nt;
      const float2 v = part[(int64_t)j * g.E + t0 + (k - j * nt)];
      s += v.x;
      q += v.y;
    }
    s = warp_sum(s);
    q = warp_sum(q);
    const float cnt = (float)g.S * (float)g.Cg;
    if (lane == 0) kk[gi - b.g0] = make_float2(s / cnt, q / cnt);
  }
  __syncthreads();
  if (!b.active) return;
  // dx = sc*e + (x - mean_hi)*q1 + q0
  float mh[VEC], sc[VEC], be[VEC], q1[VEC], q0[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    const int c = b.cv * VEC + e, gi = c / g.Cg;
    const float rstd = a.stats[ng + so + gi], ml = a.stats[2 * ng + so + gi];
    const float2 k = kk[gi - b.g0];
    mh[e] = a.stats[so + gi];
    sc[e] = rstd * (a.gamma ? a.gamma[c] : 1.f);
    be[e] = fmaf(-ml, sc[e], a.beta ? a.beta[c] : 0.f);
    q1[e] = -(rstd * rstd) * k.y;
    q0[e] = -fmaf(ml, q1[e], rstd * k.x);
  }
  const int64_t nr = rows_of(b.r0, b.r1, b.ty, g.TY);
  for (int64_t jb = nr - 1; jb >= 0; jb -= U) {
    typename V::raw rx[U], rd[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (jb - u >= 0) {
        const int64_t o = (b.r0 + b.ty + (jb - u) * g.TY) * g.C + (int64_t)b.cv * VEC;
        rx[u] = V::ld(xs + o);
        rd[u] = V::ld(ds + o);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (jb - u >= 0) {
        float v[VEC], d[VEC];
        V::cvt(rx[u], v);
        V::cvt(rd[u], d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xc = v[e] - mh[e];
          float t = d[e];
          if constexpr (ACT != GBN_ACT_NONE) t *= gn_gate<T, ACT>(fmaf(xc, sc[e], be[e]), a.slope);
          v[e] = fmaf(t, sc[e], fmaf(xc, q1[e], q0[e]));
        }
        V::store(os + (b.r0 + b.ty + (jb - u) * g.TY) * g.C + (int64_t)b.cv * VEC, v);
      }
  }
}

// ----------------------------------------------------------------- host --

enum GnKernel { kGnStats, kGnApply, kGnSums, kGnDx };

template <typename T, int VEC, int ACT>
cudaError_t gn_run(GnKernel k, const GnPlan& p, const GnArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)p.blocks), block((unsigned)p.threads);
  const size_t smem = (size_t)p.tile_groups;
  switch (k) {
    case kGnStats: return launch(gn_stats_kernel<T, VEC>, grid, block, 0, st, false, a);
    case kGnApply:
      return launch(gn_apply_kernel<T, VEC, ACT>, grid, block, smem * sizeof(float3), st, true, a);
    case kGnSums: return launch(gn_sums_kernel<T, VEC, ACT>, grid, block, 0, st, false, a);
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
  a.g.S = p.S;
  a.g.N = (int32_t)p.N;
  a.g.C = (int32_t)p.C;
  a.g.G = (int32_t)p.G;
  a.g.Cg = (int32_t)(p.C / p.G);
  a.g.Cv = (int32_t)(p.C / p.vec);
  a.g.TX = p.TX;
  a.g.TY = p.TY;
  a.g.T = p.tiles;
  a.g.slices = p.slices;
  a.g.E = (int32_t)(p.G + p.tiles - 1);
  a.gpart = static_cast<float2*>(ws);
  a.cpart = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + p.gpart_bytes);
  return a;
}

}  // namespace

bool gn_plan(int64_t N, int64_t S, int64_t C, int64_t G, int vec, bool backward,
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
  // the resident block slots once over all samples, at least one round of
  // loads a thread
  const int64_t slots = (int64_t)dev.sms * (backward ? 2 : 4);
  const int64_t per = (slots + N * p->tiles - 1) / (N * p->tiles);
  const int64_t rounds = (S + (int64_t)p->TY * (backward ? 4 : 8) - 1) /
                         ((int64_t)p->TY * (backward ? 4 : 8));
  int64_t s = per < rounds ? per : rounds;
  if (s < 1) s = 1;
  p->slices = (int)s;
  const int64_t blocks = N * s * p->tiles;
  if (blocks > INT32_MAX) return false;
  p->blocks = blocks;
  p->gpart_bytes = ((size_t)N * s * (G + p->tiles - 1) * sizeof(float2) + 255) & ~(size_t)255;
  const size_t rest = backward ? (size_t)4 * N * s * C : (size_t)N * G;
  p->ws_bytes = p->gpart_bytes + ((rest * sizeof(float) + 255) & ~(size_t)255);
  return true;
}

size_t gn_ws_bound(int64_t N, int64_t S, int64_t C, int64_t G, const DevInfo& dev) {
  size_t most = 256;
  for (int vec : {1, 2, 4, 8})
    for (bool bwd : {false, true}) {
      GnPlan p;
      if (C % vec == 0 && gn_plan(N, S, C, G, vec, bwd, dev, &p) && p.ws_bytes > most)
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
  cudaError_t e = gn_dispatch(kGnStats, dtype, GBN_ACT_NONE, p, a, st);
  if (e != cudaSuccess) return e;
  return gn_dispatch(kGnApply, dtype, act, p, a, st);
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
  cudaError_t e = gn_dispatch(kGnSums, dtype, act, p, a, st);
  if (e != cudaSuccess) return e;
  e = gn_dispatch(kGnDx, dtype, act, p, a, st);
  if (e != cudaSuccess || (dgamma == nullptr && dbeta == nullptr)) return e;
  void* outs[3] = {dgamma, dbeta, nullptr};
  return colsum_launch(a.cpart, 2, 2, (int)(p.N * p.slices), p.C, GBN_F32, outs, st, true);
}

}  // namespace gbn
