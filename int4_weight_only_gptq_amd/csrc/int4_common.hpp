// Device helpers of the int4 GPTQ kernels: code words, group metadata, epilogues.
#pragma once

#include "common.hpp"

namespace qg {

// ---------------------------------------------------------------------------
// helpers shared by the product kernels
// ---------------------------------------------------------------------------
template <int CPL>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[CPL]) {
  if constexpr (CPL == 8) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p), u = *reinterpret_cast<const u32x4*>(p + 4);
    w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    w[4] = u[0]; w[5] = u[1]; w[6] = u[2]; w[7] = u[3];
  } else if constexpr (CPL == 4) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
    w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
  } else if constexpr (CPL == 2) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    w[0] = v[0]; w[1] = v[1];
  } else {
    w[0] = *p;
  }
}

// Raw group metadata of CPL consecutive columns: their fp16 scales and the
// word holding their zero nibbles.  Loaded in the load phase and decoded only
// where it is used, so the loads do not force an early wait on everything in
// flight.
template <int CPL>
struct Meta {
  uint32_t s[CPL >= 4 ? CPL / 2 : 1];
  uint32_t z;
};

template <int CPL>
__device__ __forceinline__ Meta<CPL> load_meta(const uint16_t* __restrict__ sp, const uint32_t* __restrict__ zp) {
  Meta<CPL> r;
  if constexpr (CPL == 8) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(sp);
    r.s[0] = v[0];
    r.s[1] = v[1];
    r.s[2] = v[2];
    r.s[3] = v[3];
  } else if constexpr (CPL == 4) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(sp);
    r.s[0] = v[0];
    r.s[1] = v[1];
  } else if constexpr (CPL == 2) {
    r.s[0] = *reinterpret_cast<const uint32_t*>(sp);
  } else {
    r.s[0] = *sp;
  }
  r.z = *zp;
  return r;
}

// zshift = 4 * (col % 8): the nibble of the first of the CPL columns; zmask = 0
// without a zero point (z = 0).
template <int CPL>
__device__ __forceinline__ void decode_meta(const Meta<CPL>& mt, int zshift, uint32_t zmask, float (&s)[CPL],
                                            float (&bz)[CPL]) {
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    s[c] = half_bits_to_float((mt.s[c >> 1] >> (16 * (c & 1))) & 0xFFFFu);
    bz[c] = (float)(128u + (((mt.z & zmask) >> (zshift + 4 * c)) & 15u));
  }
}

__device__ __forceinline__ float dot2_bf16(uint32_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b),
                                         c, false);
}

__device__ __forceinline__ float bf16_bits_to_float(uint32_t h) { return __builtin_bit_cast(float, h << 16); }

// Row reduction of the epilogue: q is this lane's sum of squares of its
// rounded outputs of one row (0 without one); the G lanes of an aligned group
// (all on the same row) add theirs with cross-lane swaps, and the group's
// first lane adds the total to row_ss[row] with one atomic.  Every lane of a
// group must come here together.
template <int G>
__device__ __forceinline__ void add_row_sumsq(float* row_ss, float q, int64_t row, bool first, bool valid) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) q += __shfl_xor(q, o, G);
  if (first && valid) atomicAdd(row_ss + row, q);
}

}  // namespace qg
