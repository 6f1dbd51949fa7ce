// One output tile of the pipelined dense MFMA kernels (dense_kernels.hip, and by
// expert grouped_kernels.hip).
#pragma once

#include "common.hpp"
#include <type_traits>

namespace qg {

constexpr int DBK = 64;

// Pipeline kernel for all three layouts (K % 64 == 0, operands 16-byte
// vectorizable).  Tile BM x BN per workgroup of 4 waves (2 x 2, each
// (BM/2) x (BN/2)), k tiles of 64 in a STAGES-deep ring of LDS buffers filled
// by direct global-to-LDS loads (no staging registers): while tile kt is
// multiplied, tiles kt+1 .. kt+STAGES-1 are in flight.  One barrier per k tile,
// operand fragments read one 32-k step ahead of the MFMAs that use them.
//
// Operand tiles are stored in LDS in their memory orientation, in 16-byte
// chunks, with an XOR swizzle instead of padding (a direct load fills 64
// consecutive chunks per instruction):
//  * K-contiguous operand (A of NT/NN, B of NT): rows = m or n, 8 chunks of 8 k;
//    chunk c of row r sits at 8r + (c ^ (r & 7)).  A fragment is one 16-byte
//    read of row (lane % 16), chunk 4s + lane / 16.
//  * MN-contiguous operand (A of TN, B of NN and TN): rows = k, R/8 chunks of
//    8 m or n; chunk c of row k sits at k*R/8 + (c ^ f(k)), f(k) = 2((k & 3) |
//    ((k >> 1) & 4)).  A fragment is two transposing reads
//    (ds_read_b64_tr_b16): in each 16-lane group, lane 4r + q supplies columns
//    4q..4q+3 of k-row r and lane j receives column j of the 4 rows, i.e. 4
//    consecutive k of one column; the swizzle puts the 16 rows one read
//    touches two to a bank slot (the minimum for 512 bytes).
// Rows or columns past M or N load a clamped valid address; their results
// are discarded.  With TAIL, K may be any length (a multiple of 8 where an
// operand is K-contiguous; zero gives a tile of zeros): chunks past it are
// loaded from kZeroChunk on both sides, since what lies behind an operand's
// last row may be infinite or NaN.
__device__ __forceinline__ int fmn(int k) { return 2 * ((k & 3) | ((k >> 1) & 4)); }
// the same XOR limited to a row of R / 8 chunks (R = 64: 8 chunks)
template <int R>
__device__ __forceinline__ int fmn_r(int k) { return fmn(k) & (R / 8 - 1); }

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef s16x4 __attribute__((address_space(3))) lds_s16x4;

// 8 consecutive k of column `col` (0 .. R-1) from an MN-contiguous stage
// region with R columns (R/8 chunks per k-row); kb = first k (multiple of 8).
template <int R>
__device__ __forceinline__ u32x4 read_mn_frag(const u32x4* region, int kb, int col0, int lane) {
  const int j = lane & 15, r = j >> 2, q = j & 3;
  const int c = (col0 >> 3) + (q >> 1);
  const int k1 = kb + r, k2 = kb + 4 + r;
  const uint16_t* h1 = reinterpret_cast<const uint16_t*>(region + k1 * (R / 8) + (c ^ fmn_r<R>(k1))) + 4 * (q & 1);
  const uint16_t* h2 = reinterpret_cast<const uint16_t*>(region + k2 * (R / 8) + (c ^ fmn_r<R>(k2))) + 4 * (q & 1);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(h1));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(h2));
  u32x4 out;
  out[0] = (uint32_t)(uint16_t)lo[0] | ((uint32_t)(uint16_t)lo[1] << 16);
  out[1] = (uint32_t)(uint16_t)lo[2] | ((uint32_t)(uint16_t)lo[3] << 16);
  out[2] = (uint32_t)(uint16_t)hi[0] | ((uint32_t)(uint16_t)hi[1] << 16);
  out[3] = (uint32_t)(uint16_t)hi[2] | ((uint32_t)(uint16_t)hi[3] << 16);
  return out;
}

template <int LAYOUT, int DTYPE, int BM, int BN, int STAGES, int NWV, int WGM, bool KSPLIT, bool TAIL>
__device__ __forceinline__ void dense_pipe_tile(
    const uint16_t* __restrict__ A, int64_t lda, const uint16_t* __restrict__ B, int64_t ldb,
    uint16_t* __restrict__ C, int64_t ldc, int M, int N, int K, int t, int tm, int tn, int kslice,
    int vec_store, int ksplit, int kps, float* __restrict__ partials, uint32_t* __restrict__ tickets, int acq_rel) {
  constexpr bool A_MN = (LAYOUT == 2);           // A stored [K][M]
  constexpr bool B_MN = (LAYOUT != 0);           // B stored [K][N]
  // NWV waves as a WGM x (NWV / WGM) grid over the tile: 4 waves (one per
  // SIMD) or 8 (two per SIMD)
  constexpr int T = 64 * NWV;
  constexpr int WM = BM / WGM, WN = BN / (NWV / WGM), FM = WM / 16, FN = WN / 16;
  constexpr int A_SLOTS = BM * 8, B_SLOTS = BN * 8;           // 16-byte chunks per stage
  constexpr int STAGE = A_SLOTS + B_SLOTS;
  constexpr int A_LOADS = A_SLOTS / T, B_LOADS = B_SLOTS / T;   // per thread per stage
  static_assert(A_SLOTS % T == 0 && B_SLOTS % T == 0 && (NWV == 4 || NWV == 8), "loads per thread");
  constexpr int LOADS = A_LOADS + B_LOADS;
  static_assert(LOADS * (STAGES - 1) <= 63, "vmcnt range");
  extern __shared__ __attribute__((aligned(16))) u32x4 psm[];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cl = lane & 15, ks = lane >> 4;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wm0 = (wave % WGM) * WM, wn0 = (wave / WGM) * WN;
  const int kt0 = kslice * kps;
  A += A_MN ? (int64_t)kt0 * DBK * lda : (int64_t)kt0 * DBK;
  B += B_MN ? (int64_t)kt0 * DBK * ldb : (int64_t)kt0 * DBK;

  // source of each of this thread's chunks (chunk tid + 256 i of the operand's
  // stage region), at k tile 0; later tiles add k0 (K-contiguous) or k0 * ld
  // (koff: the first k of the chunk within its stage, for the end of k)
  const uint16_t* asrc[A_LOADS];
  const uint16_t* bsrc[B_LOADS];
  int a_koff[TAIL ? A_LOADS : 1], b_koff[TAIL ? B_LOADS : 1];
#pragma unroll
  for (int i = 0; i < A_LOADS; ++i) {
    const int slot = tid + T * i;
    if constexpr (A_MN) {
      const int k = slot / (BM / 8), c = (slot % (BM / 8)) ^ fmn_r<BM>(k);
      const int64_t gm = m0 + 8 * c < M ? m0 + 8 * c : (int64_t)M - 8;
      asrc[i] = A + (int64_t)k * lda + gm;
      if constexpr (TAIL) a_koff[i] = k;
    } else {
      const int r = slot >> 3, c = (slot & 7) ^ (r & 7);
      const int64_t gr = m0 + r < M ? m0 + r : (int64_t)M - 1;
      asrc[i] = A + gr * lda + 8 * c;
      if constexpr (TAIL) a_koff[i] = 8 * c;
    }
  }
#pragma unroll
  for (int i = 0; i < B_LOADS; ++i) {
    const int slot = tid + T * i;
    if constexpr (B_MN) {
      const int k = slot / (BN / 8), c = (slot % (BN / 8)) ^ fmn_r<BN>(k);
      const int64_t gn = n0 + 8 * c < N ? n0 + 8 * c : (int64_t)N - 8;
      bsrc[i] = B + (int64_t)k * ldb + gn;
      if constexpr (TAIL) b_koff[i] = k;
    } else {
      const int r = slot >> 3, c = (slot & 7) ^ (r & 7);
      const int64_t gr = n0 + r < N ? n0 + r : (int64_t)N - 1;
      bsrc[i] = B + gr * ldb + 8 * c;
      if constexpr (TAIL) b_koff[i] = 8 * c;
    }
  }
  const int64_t astep = A_MN ? (int64_t)DBK * lda : DBK;      // source advance per k tile
  const int64_t bstep = B_MN ? (int64_t)DBK * ldb : DBK;

  f32x4 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int c = 0; c < FN; ++c) acc[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int ktiles = TAIL ? (K + DBK - 1) / DBK
                          : (K / DBK - kt0 < kps ? K / DBK - kt0 : kps);   // this slice's k tiles
  // direct load j (0 .. LOADS-1) of stage st: each wave-instruction fills 64
  // consecutive chunks of the stage's buffer
  auto issue1 = [&](int st, int j) {
    u32x4* base = psm + (size_t)(st % STAGES) * STAGE;
    if (j < A_LOADS) {
      const uint16_t* src = asrc[j] + st * astep;
      if constexpr (TAIL) src = DBK * st + a_koff[j] < K ? src : reinterpret_cast<const uint16_t*>(&kZeroChunk);
      __builtin_amdgcn_global_load_lds((void*)src, (void*)(base + T * j + 64 * wave), 16, 0, 0);
    } else {
      const uint16_t* src = bsrc[j - A_LOADS] + st * bstep;
      if constexpr (TAIL)
        src = DBK * st + b_koff[j - A_LOADS] < K ? src : reinterpret_cast<const uint16_t*>(&kZeroChunk);
      __builtin_amdgcn_global_load_lds((void*)src, (void*)(base + A_SLOTS + T * (j - A_LOADS) + 64 * wave), 16, 0, 0);
    }
  };
  // operand fragment j (0 .. FM-1: rows of A, FM .. FM+FN-1: columns of B) of
  // k step s (32 k) of stage kt
  //
  // An M/N-contiguous fragment (column col0 + l % 16 of 8 k-rows) takes two
  // transposed 8-byte reads at k-rows kb + r and kb + 4 + r (r = (l % 16) / 4,
  // kb = 32 s + 8 (l / 16)).  Both rows get the same chunk XOR of the stage
  // layout, 2 (r | 4 (l / 16 % 2)), for either k step, and it only touches
  // the even part of the chunk index, so a fragment's address is a per-lane
  // base for its column group plus constant offsets for s and the row half.
  const int r4 = (lane & 15) >> 2, q4 = lane & 3;
  auto mn_base = [&](int R, int col0) {    // halfword offset in the operand region
    const int x = (2 * (r4 | 4 * (ks & 1))) & (R / 8 - 1);
    return ((8 * ks + r4) * (R / 8) + (((col0 >> 3) ^ x) | (q4 >> 1))) * 8 + 4 * (q4 & 1);
  };
  auto read_mn = [&](const u32x4* region, int R, int base, int s) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(region) + base + 32 * s * R;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(h));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(h + 4 * R));
    u32x4 out;
    out[0] = (uint32_t)(uint16_t)lo[0] | ((uint32_t)(uint16_t)lo[1] << 16);
    out[1] = (uint32_t)(uint16_t)lo[2] | ((uint32_t)(uint16_t)lo[3] << 16);
    out[2] = (uint32_t)(uint16_t)hi[0] | ((uint32_t)(uint16_t)hi[1] << 16);
    out[3] = (uint32_t)(uint16_t)hi[2] | ((uint32_t)(uint16_t)hi[3] << 16);
    return out;
  };
  auto read1 = [&](int kt, int s, int j, u32x4 (&a)[FM], u32x4 (&b)[FN]) {
    const u32x4* la = psm + (size_t)(kt % STAGES) * STAGE;
    const u32x4* lb = la + A_SLOTS;
    const int ch = 4 * s + ks;
    if (j < FM) {
      if constexpr (A_MN) a[j] = read_mn(la, BM, mn_base(BM, wm0 + 16 * j), s);
      else a[j] = la[swz(wm0 + 16 * j + cl, ch)];
    } else {
      const int c = j - FM;
      if constexpr (B_MN) b[c] = read_mn(lb, BN, mn_base(BN, wn0 + 16 * c), s);
      else b[c] = lb[swz(wn0 + 16 * c + cl, ch)];
    }
  };
  // the FN MFMAs of accumulator row f
  auto mma_row = [&](int f, const u32x4 (&a)[FM], const u32x4 (&b)[FN]) {
#pragma unroll
    for (int c = 0; c < FN; ++c)
      acc[f][c] = DTYPE == 0 ? mfma16_bf16(a[f], b[c], acc[f][c]) : mfma16_f16(a[f], b[c], acc[f][c]);
  };
  constexpr int NFRAG = FM + FN, RROWS = FM / 2;   // fragment reads spread over the first FM/2 rows

  // Every buffer starts filled.  Per k tile kt (its first k step already in
  // registers r0), with scheduling barriers fixing the order:
  //  1. MFMA rows of the first k step, the second k step read into r1
  //     between rows 0 .. FM/2-1;
  //  2. one barrier: stage kt + 1 has landed for every wave, and nobody reads
  //     stage kt any more (all reads of it are complete); stage kt's buffer
  //     is refilled with stage kt + STAGES;
  //  3. MFMA rows of the second k step, the first k step of kt + 1 read into
  //     r0 between rows 0 .. FM/2-1.
  // So the matrix unit waits for neither an operand read nor a load issue,
  // only at the one barrier per k tile.  Where the barrier and the refill go
  // is measured per operand form: with K-contiguous operands the barrier
  // follows the first k step and the refill loads are spread over the rows of
  // the second; with a transposed operand (whose loads take longer to land)
  // the barrier comes right after the reads of r1, half-way through the
  // first k step, and the refill is issued at once, a whole k tile before
  // it is needed.
  constexpr bool EARLY = A_MN || B_MN;
#pragma unroll
  for (int st = 0; st < STAGES; ++st)
    if (st < ktiles)
#pragma unroll
      for (int j = 0; j < LOADS; ++j) issue1(st, j);
  if (ktiles >= STAGES) __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 1)));
  else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  lds_barrier();
  u32x4 r0a[FM], r0b[FN], r1a[FM], r1b[FN];
#pragma unroll
  for (int j = 0; j < NFRAG; ++j) read1(0, 0, j, r0a, r0b);
  // one k tile; refill = kt + STAGES < ktiles, next = kt + 1 < ktiles, either
  // compile-time (std::true_type / false_type) or run-time uniform flags
  auto tile = [&](int kt, auto refill, auto next) {
    constexpr int BAR_ROW = EARLY ? RROWS : FM;        // first-step rows before the barrier
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~(0xF << 8));     // r0 complete
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < BAR_ROW; ++f) {
      mma_row(f, r0a, r0b);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NFRAG; ++j)
        if (j * RROWS / NFRAG == f) read1(kt, 1, j, r1a, r1b);
      __builtin_amdgcn_sched_barrier(0);
    }
    // stage kt + 1 landed (with a refill ahead, stages kt + 2 .. kt + STAGES - 1
    // may stay in flight; without, fewer were issued and all are waited for),
    // and this wave's reads of stage kt are complete
    if (refill) __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 2)) & ~(0xF << 8));
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & ~(0xF << 8));
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (EARLY) {
      if (refill) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j) issue1(kt + STAGES, j);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int f = BAR_ROW; f < FM; ++f) mma_row(f, r0a, r0b);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      mma_row(f, r1a, r1b);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (!EARLY) {
        if (refill) {
#pragma unroll
          for (int j = 0; j < LOADS; ++j)
            if (j * FM / LOADS == f) issue1(kt + STAGES, j);
        }
      }
      if (next) {
#pragma unroll
        for (int j = 0; j < NFRAG; ++j)
          if (j * RROWS / NFRAG == f) read1(kt + 1, 0, j, r0a, r0b);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if constexpr (!EARLY) {
    // K-contiguous operands: the last tiles in loops of their own, branch-free
    using T_ = std::true_type;
    using F_ = std::false_type;
    int kt = 0;
    for (; kt + STAGES < ktiles; ++kt) tile(kt, T_{}, T_{});
    for (; kt + 1 < ktiles; ++kt) tile(kt, F_{}, T_{});
    tile(kt, F_{}, F_{});
  } else {
    // with transposed reads, separate loops made the register allocator
    // shuffle accumulators between loops; one loop with uniform flags
    for (int kt = 0; kt < ktiles; ++kt) tile(kt, kt + STAGES < ktiles, kt + 1 < ktiles);
  }
  __syncthreads();

  if constexpr (KSPLIT) {
    // Split k: every slice stores its fp32 accumulators (fragment order:
    // element pair h of (f, c) of thread tid at ((f FN + c) 2 + h) T + tid,
    // 8-byte agent-coherent stores, 512 contiguous bytes per wave and store),
    // waits for them and takes a ticket; the last slice of the tile to arrive
    // adds the slices in slice order (its own from registers) and goes on to
    // the epilogue.  The exchange's ordering is that of the int4 split (acq_rel:
    // an acquire-release ticket).
    __shared__ int last_slice;
    uint64_t* part64 = reinterpret_cast<uint64_t*>(partials);
    uint64_t* mine = part64 + ((int64_t)t * ksplit + kslice) * (FM * FN * 2 * T);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < FN; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float lo = acc[f][c][2 * h], hi = acc[f][c][2 * h + 1];
          const uint64_t pair = (uint64_t)__builtin_bit_cast(uint32_t, lo) |
                                ((uint64_t)__builtin_bit_cast(uint32_t, hi) << 32);
          __hip_atomic_store(&mine[((f * FN + c) * 2 + h) * T + tid], pair, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
        }
    asm volatile("" ::: "memory");   // (no instruction: keeps the stores above the wait)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    if (tid == 0) last_slice = ticket_add(&tickets[t], acq_rel) == (uint32_t)(ksplit - 1);
    __syncthreads();
    if (!last_slice) return;
    // the O = ksplit - 1 other slices' pairs, FG row fragments per batch of
    // loads (at most 32 pairs in flight per thread), added in slice order
    constexpr int SLICE = FM * FN * 2 * T, PAIRS = FN * 2;
    const uint64_t* base = part64 + (int64_t)t * ksplit * SLICE;
    auto reduce = [&](auto o_) {
      constexpr int O = decltype(o_)::value;
      constexpr int FG0 = 32 / (O * PAIRS), FG = FG0 < 1 ? 1 : (FG0 > FM ? FM : FG0);
#pragma unroll
      for (int f0 = 0; f0 < FM; f0 += FG) {
        uint64_t w[FG][O][PAIRS];
#pragma unroll
        for (int g = 0; g < FG; ++g)
#pragma unroll
          for (int j = 0; j < O; ++j) {
            const int q = j < kslice ? j : j + 1;
            const uint64_t* src = base + (int64_t)q * SLICE + (f0 + g) * FN * 2 * T + tid;
#pragma unroll
            for (int e = 0; e < PAIRS; ++e)
              w[g][j][e] = f0 + g < FM ? __hip_atomic_load(src + e * T, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
          }
#pragma unroll
        for (int g = 0; g < FG; ++g) {
          const int f = f0 + g;
          if (f >= FM) break;
#pragma unroll
          for (int c = 0; c < FN; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int e = c * 2 + h;
              float lo = 0.f, hi = 0.f;
#pragma unroll
              for (int p = 0; p <= O; ++p) {
                const int jp = p < kslice ? p : p - 1;   // (selects: no indexed registers)
                uint64_t v = w[g][0][e];
#pragma unroll
                for (int j = 1; j < O; ++j) v = jp == j ? w[g][j][e] : v;
                lo += p == kslice ? acc[f][c][2 * h] : __builtin_bit_cast(float, (uint32_t)v);
                hi += p == kslice ? acc[f][c][2 * h + 1] : __builtin_bit_cast(float, (uint32_t)(v >> 32));
              }
              acc[f][c][2 * h] = lo;
              acc[f][c][2 * h + 1] = hi;
            }
        }
      }
    };
    if (ksplit == 2) reduce(std::integral_constant<int, 1>{});
    else if (ksplit == 3) reduce(std::integral_constant<int, 2>{});
    else reduce(std::integral_constant<int, 3>{});
    if (tid == 0) __hip_atomic_store(&tickets[t], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }

  // epilogue: accumulators -> output tile in LDS -> 16-byte stores
  uint16_t* osm = reinterpret_cast<uint16_t*>(psm);
  constexpr int OP = BN + 8;
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int c = 0; c < FN; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int row = wm0 + 16 * f + 4 * ks + v, col = wn0 + 16 * c + cl;
        uint16_t h;
        if constexpr (DTYPE == 0) h = (uint16_t)f32_to_bf16_bits(acc[f][c][v]);
        else h = __builtin_bit_cast(uint16_t, (_Float16)acc[f][c][v]);
        osm[row * OP + col] = h;
      }
  __syncthreads();
  constexpr int CPR = BN / 8;
  for (int c = tid; c < BM * CPR; c += T) {
    const int r = c / CPR, cc = c - r * CPR;
    const int64_t gr = m0 + r, gc = n0 + 8 * cc;
    if (gr >= M || gc >= N) continue;
    const uint16_t* src = &osm[r * OP + 8 * cc];
    if (vec_store && gc + 8 <= N) {
      *reinterpret_cast<u32x4*>(C + gr * ldc + gc) = *reinterpret_cast<const u32x4*>(src);
    } else {
      for (int e = 0; e < 8 && gc + e < N; ++e) C[gr * ldc + gc + e] = src[e];
    }
  }
}

}  // namespace qg
