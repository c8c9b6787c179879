// Counter-based dropout mask: Philox4x32 with 10 rounds (Salmon, Moraes,
// Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011).
//
// Element i of a tensor (row-major, i = r*H + h) takes 16 bits: piece i mod 8
// (low half of word 0, high half of word 0, low half of word 1, ...) of the
// four output words of block i / 8, whose 128-bit counter is (block, offset),
// 64 bits each, and whose key is the 64-bit seed.  The element is kept iff its
// piece is below `thr` = floor((1 - p)*2^16 + 1/2), and a kept element is
// multiplied by 2^16 / thr, the reciprocal of the probability that the mask
// really has, so the expectation is exact for every thr > 0.
//
// Sixteen bits, not 32: one block then serves a whole 16-byte bf16 vector, and
// the generator costs 2 wide multiplies and 2 three-input xors a round, about
// 5 instructions an element.  Twice that would bound the elementwise kernels
// (a bf16 elementwise pass at the copy rate leaves ~23 issue slots an
// element).  The price is a probability rounded to a multiple of 2^-16.
//
// Nothing is stored: the backward draws the same bits again.
#pragma once

#include "gbn_common.cuh"

namespace gbn {

// What a launch gets.  state != nullptr: (seed, offset) are read from device
// memory when the kernel runs (a captured graph draws new masks on every
// replay once the two words are changed between replays).
struct RngArgs {
  uint32_t key[20] = {};  // round keys of the seed: constant-bank operands of the xors
  uint64_t offset = 0;
  const uint64_t* state = nullptr;
  uint32_t lim = 0;       // thr << 16: a piece in a word's high half is kept below it
  uint32_t all = 0;       // thr = 2^16: everything is kept
  float scale = 0.f;      // 2^16 / thr, or 0 where nothing is kept
};

// The generator of a launch.  STATE false: the round keys are the launch's
// arguments (no instruction adds them up); true: they come from device memory
// and grow round by round.
template <bool STATE> struct Philox {
  uint32_t k0, k1, c2, c3;
  uint32_t lim;
  bool all;

  __device__ __forceinline__ void load(const RngArgs& a) {
    uint64_t o = a.offset;
    k0 = k1 = 0;
    if constexpr (STATE) {
      const uint64_t s = a.state[0];
      o = a.state[1];
      k0 = (uint32_t)s;
      k1 = (uint32_t)(s >> 32);
    }
    c2 = (uint32_t)o;
    c3 = (uint32_t)(o >> 32);
    lim = a.lim;
    all = a.all != 0;
  }
  // The four words of block b.
  __device__ __forceinline__ uint4 block(const RngArgs& a, uint64_t b) const {
    uint32_t x0 = (uint32_t)b, x1 = (uint32_t)(b >> 32), x2 = c2, x3 = c3;
    uint32_t ka = k0, kb = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
      const uint32_t q0 = STATE ? ka : a.key[2 * r], q1 = STATE ? kb : a.key[2 * r + 1];
      const uint32_t n0 = (uint32_t)(p1 >> 32) ^ x1 ^ q0, n2 = (uint32_t)(p0 >> 32) ^ x3 ^ q1;
      x1 = (uint32_t)p1;
      x3 = (uint32_t)p0;
      x0 = n0;
      x2 = n2;
      if constexpr (STATE) {
        ka += 0x9E3779B9u;
        kb += 0xBB67AE85u;
      }
    }
    return make_uint4(x0, x1, x2, x3);
  }
  // Whether the low / high piece of a word is kept.
  __device__ __forceinline__ bool lo(uint32_t w) const { return (w << 16) < lim || all; }
  __device__ __forceinline__ bool hi(uint32_t w) const { return w < lim || all; }

  // The VE elements from element i on, i a multiple of VE; VE is 8 (a block)
  // or 4 (half a block).
  template <int VE>
  __device__ __forceinline__ void keep(const RngArgs& a, uint64_t i, bool (&f)[VE]) const {
    static_assert(VE == 4 || VE == 8, "a block is eight elements");
    const uint4 w = block(a, i >> 3);
    if constexpr (VE == 8) {
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        f[2 * p] = lo(v[p]);
        f[2 * p + 1] = hi(v[p]);
      }
    } else {
      const bool second = (i & 4) != 0;
      const uint32_t u = second ? w.z : w.x, v = second ? w.w : w.y;
      f[0] = lo(u);
      f[1] = hi(u);
      f[2] = lo(v);
      f[3] = hi(v);
    }
  }
  // The eight keep decisions of block b as bits (bit e: element 8 b + e).
  __device__ __forceinline__ uint32_t bits(const RngArgs& a, uint64_t b) const {
    bool f[8];
    keep<8>(a, b << 3, f);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m |= (f[e] ? 1u : 0u) << e;
    return m;
  }
};

// The generator of kernels whose threads own single elements, wherever the
// seed comes from.
struct PhiloxAny {
  Philox<true> g;
  __device__ __forceinline__ void load(const RngArgs& a) {
    if (a.state != nullptr) {
      g.load(a);
    } else {
      g.k0 = a.key[0];
      g.k1 = a.key[1];
      g.c2 = (uint32_t)a.offset;
      g.c3 = (uint32_t)(a.offset >> 32);
      g.lim = a.lim;
      g.all = a.all != 0;
    }
  }
  __device__ __forceinline__ uint32_t bits(const RngArgs& a, uint64_t b) const {
    return g.bits(a, b);
  }
};

// Keep bits of one row (elements o .. o + H - 1) in shared memory, one byte
// per block, for kernels whose threads own single elements: each block is
// drawn once per row instead of once per element.
struct RowBits {
  uint8_t* bits;  // null: rows too long for it, every element draws its block
  uint64_t b0;    // block of the row's first element
};
__device__ __forceinline__ void rowbits_fill(RowBits& rb, const PhiloxAny& g, const RngArgs& a,
                                             uint64_t o, int64_t H) {
  if (rb.bits == nullptr) return;
  rb.b0 = o >> 3;
  const int n = (int)(((o + (uint64_t)H + 7) >> 3) - rb.b0);
  __syncthreads();  // the previous row's reads
  for (int k = threadIdx.x; k < n; k += blockDim.x) rb.bits[k] = (uint8_t)g.bits(a, rb.b0 + k);
  __syncthreads();
}
__device__ __forceinline__ bool rowbits_keep(const RowBits& rb, const PhiloxAny& g,
                                             const RngArgs& a, uint64_t i) {
  const uint32_t m = rb.bits != nullptr ? rb.bits[(i >> 3) - rb.b0] : g.bits(a, i >> 3);
  return (m >> (i & 7)) & 1u;
}
// Rows up to this length keep their bits in shared memory (32 KB + 2 bytes).
constexpr int64_t kRowBitsMaxH = 1 << 18;
__host__ __device__ constexpr size_t rowbits_bytes(int64_t H) {
  return H <= kRowBitsMaxH ? (size_t)((H + 7) / 8 + 2) : 0;
}

}  // namespace gbn
