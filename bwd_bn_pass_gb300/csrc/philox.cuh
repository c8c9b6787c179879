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
  uint64_t seed = 0, offset = 0;
  const uint64_t* state = nullptr;
  uint32_t lim = 0;       // thr << 16: a piece in a word's high half is kept below it
  uint32_t all = 0;       // thr = 2^16: everything is kept
  float scale = 0.f;      // 2^16 / thr, or 0 where nothing is kept
};

// The ten rounds' key pairs (the seed's halves plus r times the Weyl constants).
constexpr int kPhiloxKeys = 20;
__device__ __forceinline__ void philox_round_key(const RngArgs& a, int r, uint32_t& k0,
                                                 uint32_t& k1) {
  const uint64_t s = a.state != nullptr ? a.state[0] : a.seed;
  k0 = (uint32_t)s + (uint32_t)r * 0x9E3779B9u;
  k1 = (uint32_t)(s >> 32) + (uint32_t)r * 0xBB67AE85u;
}

// The generator of a kernel.  SMEM: the round keys lie in shared memory (filled
// by philox_fill before a block barrier) and come in five 16-byte broadcasts a
// block; as launch arguments or sums the compiler kept them in 20 registers
// (spills, fewer warps) or added them up again (20 instructions a block).
// Without SMEM they are added up: for kernels that draw few blocks.
template <bool SMEM> struct Philox {
  uint32_t k0, k1;        // seed halves; SMEM: k0 is the keys' shared address
  uint32_t c2, c3;
  uint32_t lim;
  bool all;

  __device__ __forceinline__ void load(const RngArgs& a, const uint32_t* keys = nullptr) {
    k0 = k1 = 0;
    if constexpr (SMEM) k0 = smem_u32(keys);
    else philox_round_key(a, 0, k0, k1);
    const uint64_t o = a.state != nullptr ? a.state[1] : a.offset;
    c2 = (uint32_t)o;
    c3 = (uint32_t)(o >> 32);
    lim = a.lim;
    all = a.all != 0;
  }
  // The four words of block b.
  __device__ __forceinline__ uint4 block(uint64_t b) const {
    uint32_t x0 = (uint32_t)b, x1 = (uint32_t)(b >> 32), x2 = c2, x3 = c3;
    uint32_t ka = k0, kb = k1;
    uint32_t kk[4];
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      uint32_t q0, q1;
      if constexpr (SMEM) {
        if (r % 2 == 0)  // volatile: not kept in registers from one block to the next
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(kk[0]), "=r"(kk[1]), "=r"(kk[2]), "=r"(kk[3])
                       : "r"(k0 + 8u * r));
        q0 = kk[2 * (r % 2)];
        q1 = kk[2 * (r % 2) + 1];
      } else {
        q0 = ka;
        q1 = kb;
        ka += 0x9E3779B9u;
        kb += 0xBB67AE85u;
      }
      const uint64_t p0 = (uint64_t)x0 * 0xD2511F53u, p1 = (uint64_t)x2 * 0xCD9E8D57u;
      const uint32_t n0 = (uint32_t)(p1 >> 32) ^ x1 ^ q0, n2 = (uint32_t)(p0 >> 32) ^ x3 ^ q1;
      x1 = (uint32_t)p1;
      x3 = (uint32_t)p0;
      x0 = n0;
      x2 = n2;
    }
    return make_uint4(x0, x1, x2, x3);
  }
  // Whether the low / high piece of a word is kept.
  __device__ __forceinline__ bool lo(uint32_t w) const { return (w << 16) < lim || all; }
  __device__ __forceinline__ bool hi(uint32_t w) const { return w < lim || all; }

  // The VE elements from element i on, i a multiple of VE; VE is 8 (a block)
  // or 4 (half a block).
  template <int VE>
  __device__ __forceinline__ void keep(uint64_t i, bool (&f)[VE]) const {
    static_assert(VE == 4 || VE == 8, "a block is eight elements");
    const uint4 w = block(i >> 3);
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
  __device__ __forceinline__ uint32_t bits(uint64_t b) const {
    bool f[8];
    keep<8>(b << 3, f);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m |= (f[e] ? 1u : 0u) << e;
    return m;
  }
};
// Round keys to shared memory; a block barrier has to follow.
__device__ __forceinline__ void philox_fill(uint32_t* keys, const RngArgs& a) {
  if (threadIdx.x < kPhiloxKeys / 2) {
    uint32_t k0, k1;
    philox_round_key(a, (int)threadIdx.x, k0, k1);
    keys[2 * threadIdx.x] = k0;
    keys[2 * threadIdx.x + 1] = k1;
  }
}

// Keep bits of one row (elements o .. o + H - 1) in shared memory, one byte
// per block, for kernels whose threads own single elements: each block is
// drawn once per row instead of once per element.
struct RowBits {
  uint8_t* bits;  // null: rows too long for it, every element draws its block
  uint64_t b0;    // block of the row's first element
};
__device__ __forceinline__ void rowbits_fill(RowBits& rb, const Philox<false>& g, uint64_t o,
                                             int64_t H) {
  if (rb.bits == nullptr) return;
  rb.b0 = o >> 3;
  const int n = (int)(((o + (uint64_t)H + 7) >> 3) - rb.b0);
  __syncthreads();  // the previous row's reads
  for (int k = threadIdx.x; k < n; k += blockDim.x) rb.bits[k] = (uint8_t)g.bits(rb.b0 + k);
  __syncthreads();
}
__device__ __forceinline__ bool rowbits_keep(const RowBits& rb, const Philox<false>& g,
                                             uint64_t i) {
  const uint32_t m = rb.bits != nullptr ? rb.bits[(i >> 3) - rb.b0] : g.bits(i >> 3);
  return (m >> (i & 7)) & 1u;
}
// Rows up to this length keep their bits in shared memory (32 KB + 2 bytes).
constexpr int64_t kRowBitsMaxH = 1 << 18;
__host__ __device__ constexpr size_t rowbits_bytes(int64_t H) {
  return H <= kRowBitsMaxH ? (size_t)((H + 7) / 8 + 2) : 0;
}

}  // namespace gbn
