// RMSNorm of every query / key head followed by rotary positions, forward and
// backward, on rows of D elements: x[t, h, :] with token and head strides (the
// heads of a packed projection are read where they lie).
//   forward   u = x*rstd*w (rstd = 1/sqrt(mean x^2 + eps), w = wq for heads
//             below q_heads, wk after), y = R(t) u
//   backward  g = R(t)^T dy, dw = sum over tokens and heads of g*x*rstd,
//             dx = rstd*(g*w - x*rstd*mean(g*w*x*rstd))
// R turns pair i of the first `rot` elements -- (i, i + rot/2) in the half
// layout, (2i, 2i + 1) interleaved -- by pos[t]*f_i and multiplies it by
// `scale`; the other elements pass.  Without weights there is no norm and the
// backward is the rotation back.
//
// Angles: f_i comes as a fraction of a turn in 0.64 fixed point, so
// pos*f_i modulo 2^64 is the exact angle modulo one turn for every 64-bit
// position, with two integer multiplies and no double-precision arithmetic;
// its top bits then go through sincospif (2^-25 of a turn's half is the
// rounding of the angle, near or far).
//
// Bound: DRAM traffic (forward 2, backward 3 tensors); decoding: latency.
//
// Layout: a team of L lanes (L a power of two) owns a token and walks a chunk
// of its heads, so sines and cosines are formed once per token and chunk and
// stay in registers.  A lane owns NS slots; a slot is two vectors of VEC
// elements whose pairs are complete (half: the vectors at i and i + rot/2;
// interleaved: two neighbours), so no element crosses lanes and only the row
// sums are shuffled.
#include "gbn_common.cuh"
#include "gbn_internal.h"

namespace gbn {

namespace {

constexpr int kRThreads = 256;

struct RopeArgs {
  const void* x;
  const void* dy;        // backward
  void* out;             // y / dx
  const void* pos;       // int32 or int64 [T]
  const uint64_t* freqs; // [rot / 2]
  const void* wq;
  const void* wk;
  float* rstd;           // [T, H]: written (forward, may be null), read (backward)
  float* part;           // backward: [plane][rows][D], rows = blocks of q chunks, then of k
  int64_t T;
  int64_t xt, xh, yt, yh, dt, dh;  // token and head strides of x, out, dy
  int32_t H, HQ, D, rot;
  int32_t L;             // lanes per team
  int32_t hc;            // heads per chunk (forward)
  int32_t cq, ck;        // backward: chunks of query and of key heads
  int32_t pos64;
  float eps, scale;
};

// cos and sin (times scale) of pos * f turns.
__device__ __forceinline__ void rope_angle(uint64_t pos, uint64_t f, float scale, float& c,
                                           float& s) {
  const int32_t top = (int32_t)((pos * f) >> 32);  // in [-1/2, 1/2) turns
  float sn, cs;
  sincospif((float)top * (1.f / 2147483648.f), &sn, &cs);
  c = cs * scale;
  s = sn * scale;
}

template <int VEC, int NS, bool INTER> struct Slots {
  int ia[NS], ib[NS];       // first element of the two vectors
  bool va[NS], vb[NS];
  float cs[NS][VEC], sn[NS][VEC];
  uint32_t turn[NS];        // bit j: pair j of the slot turns

  __device__ __forceinline__ void place(const RopeArgs& a, int l) {
    const int half = a.rot / 2;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const int p = l + s * a.L;
      if (INTER) {
        ia[s] = 2 * p * VEC;
        ib[s] = ia[s] + VEC;
      } else if (p * VEC < half) {
        ia[s] = p * VEC;
        ib[s] = ia[s] + half;
      } else {
        ia[s] = 2 * p * VEC;  // rot + 2 (p VEC - half)
        ib[s] = ia[s] + VEC;
      }
      va[s] = ia[s] < a.D;
      vb[s] = ib[s] < a.D;
      turn[s] = 0;
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (p * VEC + j < half) turn[s] |= 1u << j;
    }
  }
  __device__ __forceinline__ void angles(const RopeArgs& a, int l, uint64_t pos) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        cs[s][j] = 1.f;
        sn[s][j] = 0.f;
        if ((turn[s] >> j) & 1u)
          rope_angle(pos, a.freqs[(l + s * a.L) * VEC + j], a.scale, cs[s][j], sn[s][j]);
      }
  }
  // (a, b) <- R (a, b), or its transpose (BACK)
  template <bool BACK>
  __device__ __forceinline__ void rotate(int s, float (&u)[VEC], float (&v)[VEC]) const {
    if constexpr (INTER && VEC > 1) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float& p = j < VEC / 2 ? u[2 * j] : v[2 * j - VEC];
        float& q = j < VEC / 2 ? u[2 * j + 1] : v[2 * j + 1 - VEC];
        turn_pair<BACK>(s, j, p, q);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) turn_pair<BACK>(s, j, u[j], v[j]);
    }
  }
  template <bool BACK>
  __device__ __forceinline__ void turn_pair(int s, int j, float& p, float& q) const {
    const float c = cs[s][j], w = BACK ? -sn[s][j] : sn[s][j];
    const float np = fmaf(p, c, -(q * w)), nq = fmaf(q, c, p * w);
    if ((turn[s] >> j) & 1u) {  // a passing element never meets its neighbour
      p = np;
      q = nq;
    }
  }
};

__device__ __forceinline__ uint64_t rope_pos(const RopeArgs& a, int64_t t) {
  return a.pos64 ? static_cast<const uint64_t*>(a.pos)[t]
                 : (uint64_t)(int64_t)static_cast<const int32_t*>(a.pos)[t];
}

__device__ __forceinline__ float team_total(float v, int L) {
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int VEC>
__device__ __forceinline__ void ld_vec(const T* p, bool ok, typename Vec<T, VEC>::raw& r) {
  if (ok) r = Vec<T, VEC>::ld(p);
  else r = typename Vec<T, VEC>::raw{};
}

// Forward (and, without a norm, the backward: BACK).  blockIdx.y: head chunk.
template <typename T, int VEC, int NS, bool INTER, bool NORM, bool BACK>
__global__ void __launch_bounds__(kRThreads) rope_fwd_kernel(RopeArgs a) {
  constexpr int UH = VEC * NS >= 8 ? 2 : 4;  // heads in flight
  using V = Vec<T, VEC>;
  const int l = threadIdx.x & (a.L - 1);
  const int64_t t = (int64_t)blockIdx.x * (kRThreads / a.L) + threadIdx.x / a.L;
  const bool live = t < a.T;
  const int h0 = blockIdx.y * a.hc, h1 = min(h0 + a.hc, a.H);
  const T* x = static_cast<const T*>(a.x) + (live ? t : 0) * a.xt;
  T* y = static_cast<T*>(a.out) + (live ? t : 0) * a.yt;
  Slots<VEC, NS, INTER> sl;
  sl.place(a, l);
  typename V::raw wa[2][NS], wb[2][NS];  // weights of query and key heads
  if constexpr (NORM) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const T* w = static_cast<const T*>(k ? a.wk : a.wq);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        ld_vec<T, VEC>(w + sl.ia[s], w != nullptr && sl.va[s], wa[k][s]);
        ld_vec<T, VEC>(w + sl.ib[s], w != nullptr && sl.vb[s], wb[k][s]);
      }
    }
  }
  sl.angles(a, l, live ? rope_pos(a, t) : 0);
  const float inv_D = 1.f / (float)a.D;
  for (int hb = h0; hb < h1; hb += UH) {
    typename V::raw ra[UH][NS], rb[UH][NS];
#pragma unroll
    for (int u = 0; u < UH; ++u)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const bool ok = live && hb + u < h1;
        const T* p = x + (int64_t)(hb + u) * a.xh;
        ld_vec<T, VEC>(p + sl.ia[s], ok && sl.va[s], ra[u][s]);
        ld_vec<T, VEC>(p + sl.ib[s], ok && sl.vb[s], rb[u][s]);
      }
#pragma unroll
    for (int u = 0; u < UH; ++u) {
      const int h = hb + u;
      float r = 1.f;
      if constexpr (NORM) {
        float q = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          float m[VEC], n[VEC];
          V::cvt(ra[u][s], m);
          V::cvt(rb[u][s], n);
#pragma unroll
          for (int e = 0; e < VEC; ++e) q = fmaf(m[e], m[e], fmaf(n[e], n[e], q));
        }
        r = 1.f / sqrtf(team_total(q, a.L) * inv_D + a.eps);
      }
      if (!live || h >= h1) continue;
      if (NORM && l == 0 && a.rstd != nullptr) a.rstd[t * a.H + h] = r;
      T* o = y + (int64_t)h * a.yh;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float m[VEC], n[VEC];
        V::cvt(ra[u][s], m);
        V::cvt(rb[u][s], n);
        if constexpr (NORM) {
          float w0[VEC], w1[VEC];
          V::cvt(h < a.HQ ? wa[0][s] : wa[1][s], w0);
          V::cvt(h < a.HQ ? wb[0][s] : wb[1][s], w1);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            m[e] = (m[e] * r) * w0[e];
            n[e] = (n[e] * r) * w1[e];
          }
        }
        sl.template rotate<BACK>(s, m, n);
        if (sl.va[s]) V::store(o + sl.ia[s], m);
        if (sl.vb[s]) V::store(o + sl.ib[s], n);
      }
    }
  }
}

// Backward with the norm.  blockIdx.y: a chunk of query heads (below cq) or of
// key heads; blocks stride over the tokens.  A block's weight gradient goes to
// its row of the partials.
template <typename T, int VEC, int NS, bool INTER>
__global__ void __launch_bounds__(kRThreads) rope_bwd_kernel(RopeArgs a) {
  constexpr bool COMP = sizeof(T) == 4;
  constexpr int UH = VEC * NS >= 8 ? 1 : 2;
  using V = Vec<T, VEC>;
  extern __shared__ DF red[];  // [teams][2 * NS * VEC * L]
  const int l = threadIdx.x & (a.L - 1), team = threadIdx.x / a.L, teams = kRThreads / a.L;
  const bool is_q = (int)blockIdx.y < a.cq;
  const int nh = is_q ? a.HQ : a.H - a.HQ, nc = is_q ? a.cq : a.ck;
  const int ch = is_q ? blockIdx.y : blockIdx.y - a.cq;
  const int hbase = is_q ? 0 : a.HQ;
  const int h0 = hbase + (int)((int64_t)nh * ch / nc), h1 = hbase + (int)((int64_t)nh * (ch + 1) / nc);
  const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
  Slots<VEC, NS, INTER> sl;
  sl.place(a, l);
  float w0[NS][VEC], w1[NS][VEC];
  DF acc[NS][2][VEC];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    typename V::raw r0, r1;
    ld_vec<T, VEC>(w + sl.ia[s], sl.va[s], r0);
    ld_vec<T, VEC>(w + sl.ib[s], sl.vb[s], r1);
    V::cvt(r0, w0[s]);
    V::cvt(r1, w1[s]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[s][0][e] = acc[s][1][e] = DF{0.f, 0.f};
  }
  const float inv_D = 1.f / (float)a.D;
  for (int64_t tb = (int64_t)blockIdx.x * teams; tb < a.T; tb += (int64_t)gridDim.x * teams) {
    const int64_t t = tb + team;
    const bool live = t < a.T;
    const T* x = static_cast<const T*>(a.x) + (live ? t : 0) * a.xt;
    const T* d = static_cast<const T*>(a.dy) + (live ? t : 0) * a.dt;
    T* o = static_cast<T*>(a.out) + (live ? t : 0) * a.yt;
    sl.angles(a, l, live ? rope_pos(a, t) : 0);
    for (int hb = h0; hb < h1; hb += UH) {
      typename V::raw xa[UH][NS], xb[UH][NS], da[UH][NS], db[UH][NS];
      float rs[UH];
#pragma unroll
      for (int u = 0; u < UH; ++u) {
        const bool ok = live && hb + u < h1;
        rs[u] = ok ? a.rstd[t * a.H + hb + u] : 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          const T* p = x + (int64_t)(hb + u) * a.xh;
          const T* q = d + (int64_t)(hb + u) * a.dh;
          ld_vec<T, VEC>(p + sl.ia[s], ok && sl.va[s], xa[u][s]);
          ld_vec<T, VEC>(p + sl.ib[s], ok && sl.vb[s], xb[u][s]);
          ld_vec<T, VEC>(q + sl.ia[s], ok && sl.va[s], da[u][s]);
          ld_vec<T, VEC>(q + sl.ib[s], ok && sl.vb[s], db[u][s]);
        }
      }
#pragma unroll
      for (int u = 0; u < UH; ++u) {
        float g0[NS][VEC], g1[NS][VEC], x0[NS][VEC], x1[NS][VEC];
        float q = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          V::cvt(xa[u][s], x0[s]);
          V::cvt(xb[u][s], x1[s]);
          V::cvt(da[u][s], g0[s]);
          V::cvt(db[u][s], g1[s]);
          sl.template rotate<true>(s, g0[s], g1[s]);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            x0[s][e] *= rs[u];
            x1[s][e] *= rs[u];
            const float p0 = g0[s][e] * x0[s][e], p1 = g1[s][e] * x1[s][e];
            if constexpr (COMP) {
              df_add(acc[s][0][e], p0);
              df_add(acc[s][1][e], p1);
            } else {
              acc[s][0][e].hi += p0;
              acc[s][1][e].hi += p1;
            }
            q = fmaf(p0, w0[s][e], fmaf(p1, w1[s][e], q));
          }
        }
        const float m = team_total(q, a.L) * inv_D;
        if (!live || hb + u >= h1) continue;
        T* ho = o + (int64_t)(hb + u) * a.yh;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            g0[s][e] = rs[u] * fmaf(-x0[s][e], m, g0[s][e] * w0[s][e]);
            g1[s][e] = rs[u] * fmaf(-x1[s][e], m, g1[s][e] * w1[s][e]);
          }
          if (sl.va[s]) V::store(ho + sl.ia[s], g0[s]);
          if (sl.vb[s]) V::store(ho + sl.ib[s], g1[s]);
        }
      }
    }
  }
  // the block's teams, added in order
  const int per = 2 * NS * VEC;
#pragma unroll
  for (int s = 0; s < NS; ++s)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      red[((size_t)team * per + (2 * s) * VEC + e) * a.L + l] = acc[s][0][e];
      red[((size_t)team * per + (2 * s + 1) * VEC + e) * a.L + l] = acc[s][1][e];
    }
  __syncthreads();
  const int64_t rows = (int64_t)gridDim.x * (a.cq + a.ck);
  float* row = a.part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.D;
  for (int k = threadIdx.x; k < per * a.L; k += kRThreads) {
    DF t{0.f, 0.f};
    for (int q = 0; q < teams; ++q) {
      const DF v = red[(size_t)q * per * a.L + k];
      if constexpr (COMP) t = df_sum(t, v);
      else t.hi += v.hi;
    }
    const int ll = k % a.L, e = k / a.L % VEC, sv = k / a.L / VEC;  // sv = 2 s + which
    const int p = ll + (sv / 2) * a.L, half = a.rot / 2;
    const int i0 = INTER || p * VEC >= half ? 2 * p * VEC : p * VEC;
    const int i1 = INTER || p * VEC >= half ? i0 + VEC : i0 + half;
    const int i = (sv & 1) ? i1 : i0;
    if (i < a.D) {
      row[i + e] = t.hi;
      if constexpr (COMP) row[rows * a.D + i + e] = t.lo;
    }
  }
  pdl_launch_dependents();
}

// dw[which] = sum of that side's partial rows, in a fixed order: 32 columns x
// 32 row groups a block, blockIdx.y = 0 query, 1 key.
template <typename T, bool COMP>
__global__ void __launch_bounds__(1024)
    rope_dw_kernel(const float* __restrict__ part, int64_t rq, int64_t rows, int D, T* dwq, T* dwk) {
  __shared__ DF sm[32][33];
  pdl_wait();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int j = blockIdx.x * 32 + tx;
  const int64_t r0 = blockIdx.y ? rq : 0, r1 = blockIdx.y ? rows : rq;
  DF t{0.f, 0.f};
  if (j < D)
#pragma unroll 4
    for (int64_t r = r0 + ty; r < r1; r += 32) {
      df_add(t, part[r * D + j]);
      if constexpr (COMP) t.lo += part[(rows + r) * D + j];
    }
  sm[ty][tx] = t;
  __syncthreads();
  T* out = blockIdx.y ? dwk : dwq;
  if (ty == 0 && j < D && out != nullptr) {
    DF s{0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 32; ++k) s = df_sum(s, sm[k][tx]);
    out[j] = from_f32<T>(df_round(s));
  }
}

// ----------------------------------------------------------------- host --

template <typename T, int VEC, int NS, bool INTER>
cudaError_t rope_run(const RopePlan& p, const RopeArgs& a, int dir, cudaStream_t st) {
  const bool norm = a.wq != nullptr;
  const int teams = kRThreads / p.L;
  if (dir == 0 || !norm) {
    const dim3 grid((unsigned)((a.T + teams - 1) / teams), (unsigned)((a.H + a.hc - 1) / a.hc));
    if (dir == 0)
      return norm ? launch(rope_fwd_kernel<T, VEC, NS, INTER, true, false>, grid, dim3(kRThreads), 0,
                           st, false, a)
                  : launch(rope_fwd_kernel<T, VEC, NS, INTER, false, false>, grid, dim3(kRThreads),
                           0, st, false, a);
    return launch(rope_fwd_kernel<T, VEC, NS, INTER, false, true>, grid, dim3(kRThreads), 0, st,
                  false, a);
  }
  const size_t smem = sizeof(DF) * 2 * NS * VEC * kRThreads;
  return launch(rope_bwd_kernel<T, VEC, NS, INTER>, dim3((unsigned)p.bx, (unsigned)(a.cq + a.ck)),
                dim3(kRThreads), smem, st, false, a);
}
template <typename T, int VEC, int NS>
cudaError_t rope_run_layout(const RopePlan& p, const RopeArgs& a, int dir, bool inter,
                            cudaStream_t st) {
  return inter ? rope_run<T, VEC, NS, true>(p, a, dir, st)
               : rope_run<T, VEC, NS, false>(p, a, dir, st);
}
template <typename T>
cudaError_t rope_dispatch(const RopePlan& p, const RopeArgs& a, int dir, bool inter,
                          cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (p.vec == 8) return rope_run_layout<T, 8, 1>(p, a, dir, inter, st);
  switch (p.vec) {
    case 4:
      return p.ns == 1 ? rope_run_layout<T, 4, 1>(p, a, dir, inter, st)
                       : rope_run_layout<T, 4, 2>(p, a, dir, inter, st);
    case 2:
      return p.ns == 1 ? rope_run_layout<T, 2, 1>(p, a, dir, inter, st)
                       : rope_run_layout<T, 2, 4>(p, a, dir, inter, st);
    default:
      return p.ns == 2 ? rope_run_layout<T, 1, 2>(p, a, dir, inter, st)
                       : rope_run_layout<T, 1, 8>(p, a, dir, inter, st);
  }
}

}  // namespace

// `vec_max`: the widest vector that alignment and strides allow.
bool rope_plan(int64_t T, int64_t H, int64_t HQ, int64_t D, int64_t rot, bool inter, int dtype,
               int vec_max, const DevInfo& dev, RopePlan* p) {
  *p = RopePlan();
  int v = dtype == GBN_F32 ? 4 : 8;
  while (v > 1 && (v > vec_max || D % v != 0 || (!inter && (rot / 2) % v != 0))) v /= 2;
  p->vec = v;
  const int64_t slots = (D + 2 * v - 1) / (2 * v);
  int L = 1;
  while (L < 32 && L < slots) L *= 2;
  const int64_t ns = (slots + L - 1) / L;
  switch (v) {  // the instances there are
    case 8: p->ns = 1; break;
    case 4: p->ns = ns <= 1 ? 1 : 2; break;
    case 2: p->ns = ns <= 1 ? 1 : 4; break;
    default: p->ns = ns <= 2 ? 2 : 8; break;
  }
  if (ns > p->ns) return false;
  // more than one slot a lane: the fewest lanes that hold the row
  while (L > 1 && (int64_t)(L / 2) * p->ns >= slots) L /= 2;
  p->L = L;
  // heads per chunk: as many as leave three quarters of the SMs' threads busy
  const int64_t want = (int64_t)dev.sms * 1536;
  int64_t hc = T * H * L / want;
  if (hc < 1) hc = 1;
  if (hc > H) hc = H;
  const int64_t chunks = (H + hc - 1) / hc;
  p->hc = (int)((H + chunks - 1) / chunks);
  // backward: chunks of query heads and of key heads apart
  const int64_t teams = kRThreads / L;
  const int64_t tb = (T + teams - 1) / teams;
  const int64_t blocks = (int64_t)dev.sms * 4;
  const int64_t HK = H - HQ;
  int64_t per = (tb * H + blocks - 1) / blocks;  // heads per chunk
  if (per < 1) per = 1;
  p->cq = (int)((HQ + per - 1) / per);
  p->ck = (int)((HK + per - 1) / per);
  const int64_t cap = (2 * blocks + p->cq + p->ck - 1) / (p->cq + p->ck);
  p->bx = tb < cap ? tb : cap;
  const size_t rows = (size_t)p->bx * (size_t)(p->cq + p->ck);
  p->ws_bytes = ((dtype == GBN_F32 ? 2 : 1) * rows * (size_t)D * 4 + 255) & ~(size_t)255;
  return true;
}

size_t rope_ws_bound(int64_t T, int64_t H, int64_t HQ, int64_t D, int64_t rot, int dtype,
                     const DevInfo& dev) {
  size_t most = 256;
  for (int v : {1, 2, 4, 8})
    for (bool inter : {false, true}) {
      RopePlan p;
      if (rope_plan(T, H, HQ, D, rot, inter, dtype, v, dev, &p) && p.ws_bytes > most)
        most = p.ws_bytes;
    }
  return most;
}

cudaError_t rope_launch(const RopePlan& p, const RopePtrs& q, int dir, int dtype, int64_t T,
                        int64_t H, int64_t HQ, int64_t D, int64_t rot, bool inter, float scale,
                        float eps, cudaStream_t st) {
  RopeArgs a;
  a.x = q.x;
  a.dy = q.dy;
  a.out = q.out;
  a.pos = q.pos;
  a.pos64 = q.pos64 ? 1 : 0;
  a.freqs = q.freqs;
  a.wq = q.wq;
  a.wk = q.wk;
  a.rstd = q.rstd;
  a.part = static_cast<float*>(q.ws);
  a.T = T;
  a.xt = q.xt;
  a.xh = q.xh;
  a.yt = q.yt;
  a.yh = q.yh;
  a.dt = q.dt;
  a.dh = q.dh;
  a.H = (int32_t)H;
  a.HQ = (int32_t)HQ;
  a.D = (int32_t)D;
  a.rot = (int32_t)rot;
  a.L = p.L;
  a.hc = p.hc;
  a.cq = p.cq;
  a.ck = p.ck;
  a.eps = eps;
  a.scale = scale;
  if (dir == 1 && a.wq == nullptr) {  // the rotation back of dy
    a.x = q.dy;
    a.xt = q.dt;
    a.xh = q.dh;
  }
  cudaError_t e = cudaSuccess;
  if (T > 0)
    e = dtype == GBN_F32 ? rope_dispatch<float>(p, a, dir, inter, st)
                         : rope_dispatch<bf16>(p, a, dir, inter, st);
  if (e != cudaSuccess || dir == 0 || a.wq == nullptr) return e;
  const int64_t rq = p.bx * p.cq, rows = p.bx * (p.cq + p.ck);
  const dim3 grid((unsigned)((D + 31) / 32), 2);
  const float* part = a.part;
  if (dtype == GBN_F32)
    return launch(rope_dw_kernel<float, true>, grid, dim3(1024), 0, st, true, part, rq, rows, (int)D,
                  static_cast<float*>(q.dwq), static_cast<float*>(q.dwk));
  return launch(rope_dw_kernel<bf16, false>, grid, dim3(1024), 0, st, true, part, rq, rows, (int)D,
                static_cast<bf16*>(q.dwq), static_cast<bf16*>(q.dwk));
}

}  // namespace gbn
