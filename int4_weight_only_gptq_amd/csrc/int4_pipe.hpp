// One output tile of the pipelined int4 MFMA kernels (int4_kernels.hip, and by
// expert grouped_int4_kernels.hip).
#pragma once

#include "int4_common.hpp"
#include "launch.hpp"

namespace qg {

// ---------------------------------------------------------------------------
// Pipelined MFMA kernel for m > 16.
//
// Workgroup tile BM x BN = (NWM * 16 * FM) tokens x (NWN * 64) columns; wave
// (wm, wn) owns 16 * FM tokens x 64 columns as FM x 4 MFMA tiles of 16 x 16.
// Within a wave's 64 columns, N-fragment c holds columns 4 * l + c (l = lane
// % 16), so one 16-byte LDS read gives a lane the words of its four columns and
// the output of four adjacent columns lands in one lane.
//
// The k loop walks stages of 64 rows (half a quantization group).  Each stage
// is copied global -> LDS with direct buffer loads (no register
// round trip), STAGES deep:
//   activations  BM x 64 bf16, K-contiguous, XOR-swizzled 16-byte chunks
//   codes        8 word rows x BN columns (the qweight words of those 64 rows)
//   metadata     the group's BN fp16 scales and BN / 8 zero words
// The oldest stage is consumed once the wave's vmcnt shows its loads landed
// and a plain s_barrier shows every wave is past the previous stage.
//
// Per 32-row k step a wave turns each column's word into the bf16 pairs
// 128 + q (codes_as_bf16_pairs), reorders its activation fragments to the
// same pair order, and accumulates; a ones-MFMA on the raw activation
// fragments gives the per-token group sums in the accumulator layout.  After
// both stages of a group: total += s * (acc - (128 + z) * sum_x), fp32.
// ---------------------------------------------------------------------------
#ifndef QG_PIPE_INTERLEAVE
#define QG_PIPE_INTERLEAVE 1   // interleave the second k step's decode with the first step's MFMAs
#endif

template <int NWM, int NWN, int FM, bool PREP, bool LORA = false>
struct PipeShape {
  static constexpr int T = 64 * NWM * NWN;               // threads
  static constexpr int NW = NWM * NWN;                   // waves
  static constexpr int BM = NWM * 16 * FM, BN = NWN * 64;
  static constexpr int X_SLOTS = BM * 8;                 // 16-byte activation chunks per stage
  static constexpr int XL = X_SLOTS / T;                 // per thread
  static constexpr bool W16 = (2 * BN) % T == 0;         // words as 16-byte chunks, else dwords
  static constexpr int WL = W16 ? 2 * BN / T : 8 * BN / T;
  // metadata: 64-dword slots, one per wave and load: the BN scales (slot 0), the
  // BN / 8 zero words (slot 1) and, with the prepared activations, the group
  // sums of the BM tokens (slots 2 .. 2 + BM / 64 - 1); other slots are filler
  static constexpr int MSLOTS = 2 + (PREP ? BM / 64 : 0);
  static constexpr int ML = (MSLOTS + NW - 1) / NW;      // metadata loads per thread
  // LoRA: the stage's 16 x 64 block of lora_A (512 dwords, 4-byte loads)
  static constexpr int AL = LORA ? 512 / T : 0;
  static constexpr int LOADS = XL + WL + ML + AL;        // direct loads per thread per stage
  static constexpr int X_DW = 4 * X_SLOTS, W_DW = 8 * BN, M_DW = 64 * NW * ML, A_DW = LORA ? 512 : 0;
  static constexpr int STAGE_DW = X_DW + W_DW + M_DW + A_DW;   // dwords of LDS per stage
  static constexpr int OP = BN + 8;                      // output tile row pitch (bf16)
  static_assert(X_SLOTS % T == 0, "activation chunks per thread");
  static_assert((8 * BN) % T == 0, "word loads per thread");
  static_assert(BN == 128 && BM % 64 == 0, "metadata slots");
  static_assert(!LORA || (512 % T == 0 && NWN == 2), "lora_A block loads; two column waves share U");
};

template <int NWM, int NWN, int FM, int STAGES, bool PREP, bool LORA>
__device__ __forceinline__ void int4_pipe_tile(
    const uint16_t* __restrict__ x, int64_t ldx, const uint32_t* __restrict__ qweight,
    const uint16_t* __restrict__ scales, const uint32_t* __restrict__ qzeros,
    const float* __restrict__ xsum, int64_t xsum_ld, uint16_t* __restrict__ y, int64_t ldy, int m, int n, int k,
    int t, int tm, int tn, int kslice, int vec_store, int ksplit, int gps,
    float* __restrict__ partials, uint32_t* __restrict__ tickets, int acq_rel, const LoraEpi& lora) {
  using S = PipeShape<NWM, NWN, FM, PREP, LORA>;
  constexpr int T = S::T, BM = S::BM, BN = S::BN, XL = S::XL, WL = S::WL, LOADS = S::LOADS;
  static_assert(LOADS * (STAGES - 2) <= 63, "vmcnt range");
  extern __shared__ __attribute__((aligned(16))) uint32_t psm_i4[];

  const int gbeg = kslice * gps, gend = min(k >> 7, gbeg + gps);   // this slice's groups
  const int kt0 = 2 * gbeg;                                          // its first stage
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);   // wave-uniform: LDS bases stay scalar
  const int cl = lane & 15, ks = lane >> 4;
  const int m0 = tm * BM, n0 = tn * BN;
  const int wm0 = (wave % NWM) * 16 * FM, wn0 = (wave / NWM) * 64;

  // Direct loads go through buffer resources (base in SGPRs, rebased per
  // stage) with one fixed 32-bit byte offset per lane and load, so a stage's
  // issue costs no vector ALU work.  Rows past m and columns past n load a
  // clamped valid address; their results are discarded.
  uint32_t xoff[XL];
#pragma unroll
  for (int i = 0; i < XL; ++i) {
    const int slot = tid + T * i;
    const int r = slot >> 3, c = (slot & 7) ^ (r & 7);
    const int rl = m0 + r < m ? r : m - 1 - m0;
    xoff[i] = (uint32_t)(((int64_t)rl * ldx + 8 * c) * 2);
  }
  uint32_t woff[WL];
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    const int slot = tid + T * i;
    int wr, cw;
    if constexpr (S::W16) {
      wr = slot / (BN / 4);
      cw = n0 + 4 * (slot % (BN / 4)) < n ? 4 * (slot % (BN / 4)) : n - 4 - n0;
    } else {
      wr = slot / BN;
      cw = n0 + slot % BN < n ? slot % BN : n - 1 - n0;
    }
    woff[i] = (uint32_t)(((int64_t)wr * n + cw) * 4);
  }
  // metadata slot j = NW * i + wave of load i: 0 scales, 1 zero words,
  // 2.. the group sums of tokens m0 + 64 (j - 2) + lane; others: zero words
  const int zlane = (n0 >> 3) + lane < (n >> 3) ? lane : (n >> 3) - 1 - (n0 >> 3);
  uint32_t moff[S::ML];
#pragma unroll
  for (int i = 0; i < S::ML; ++i) {
    const int j = S::NW * i + wave;
    if (j == 0) {
      moff[i] = (uint32_t)((n0 + 2 * lane < n ? 2 * lane : n - 2 - n0) * 2);
    } else if (j >= 2 && j < S::MSLOTS) {
      const int r = 64 * (j - 2) + lane;
      moff[i] = (uint32_t)((m0 + r < m ? r : m - 1 - m0) * 4);
    } else {
      moff[i] = (uint32_t)(zlane * 4);
    }
  }
  // LoRA: dword d = T i + 64 wave + lane of the stage's lora_A block holds
  // rank r = d / 32, 16-byte slot c = (d % 32) / 4, dword d % 4, where slot c of
  // row r carries the row's chunk c ^ (r & 7) (8 k each): the 16 ranks of an
  // operand read then spread over the banks.  Ranks past the rank read row 0.
  uint32_t aoff[S::AL > 0 ? S::AL : 1];
#pragma unroll
  for (int i = 0; i < S::AL; ++i) {
    const int d = T * i + 64 * wave + lane, r = d >> 5, c = (d & 31) >> 2;
    aoff[i] = (uint32_t)(((r < lora.rank ? (int64_t)r * lora.lda : 0) + 8 * (c ^ (r & 7)) + 2 * (d & 3)) * 2);
  }
  const uint16_t* xbase = x + (int64_t)m0 * ldx;
  const uint32_t* wbase0 = qweight + n0;

  auto issue = [&](int st) {   // local stage st = global stage kt0 + st
    uint32_t* base = psm_i4 + (size_t)(st % STAGES) * S::STAGE_DW;
    const uint16_t* xs_base = xbase + 64 * (int64_t)(kt0 + st);
#pragma unroll
    for (int i = 0; i < XL; ++i) buffer_to_lds16(xs_base, xoff[i], base + 4 * (T * i + 64 * wave));
    uint32_t* wl = base + S::X_DW;
    const uint32_t* ws_base = wbase0 + 8 * (int64_t)(kt0 + st) * n;
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      if constexpr (S::W16) buffer_to_lds16(ws_base, woff[i], wl + 4 * (T * i + 64 * wave));
      else buffer_to_lds4(ws_base, woff[i], wl + T * i + 64 * wave);
    }
    const int64_t g = (kt0 + st) >> 1;
#pragma unroll
    for (int i = 0; i < S::ML; ++i) {
      const int j = S::NW * i + wave;
      // Every wave issues the same number of loads per stage (the waits count
      // them).  Without zero points the zero-word slots load a word of the
      // stage's scale row instead (in bounds: lane offsets stay below n / 2
      // bytes), which is never read.
      if (j == 0) buffer_to_lds4(scales + g * n + n0, moff[i], wl + S::W_DW + 64 * j);
      else if (j >= 2 && j < S::MSLOTS) buffer_to_lds4(xsum + g * xsum_ld + m0, moff[i], wl + S::W_DW + 64 * j);
      else if (qzeros) buffer_to_lds4(qzeros + g * (n >> 3) + (n0 >> 3), moff[i], wl + S::W_DW + 64 * j);
      else buffer_to_lds4(scales + g * n + n0, moff[i], wl + S::W_DW + 64 * j);
    }
    if constexpr (LORA) {
      uint32_t* al = wl + S::W_DW + S::M_DW;
      const uint16_t* abase = lora.a + 64 * (int64_t)(kt0 + st);
#pragma unroll
      for (int i = 0; i < S::AL; ++i) buffer_to_lds4(abase, aoff[i], al + T * i + 64 * wave);
    }
  };

  f32x4 total[FM][4], acc[FM][4], xs[PREP ? 1 : FM];
  f32x4 uacc[LORA ? FM : 1];   // LoRA: this wave's share of U for its rows (rank = lane % 16)
#pragma unroll
  for (int f = 0; f < (LORA ? FM : 1); ++f) uacc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wn = wave / NWM;     // column wave: takes U for k step wn of each stage
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int c = 0; c < 4; ++c) total[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  const u32x4 ones = {kOnesBf16x2, kOnesBf16x2, kOnesBf16x2, kOnesBf16x2};

  const int ktiles = 2 * (gend - gbeg);   // stages of this slice
  // raw fragments of one k step: FM activation chunks and one 16-byte word read
  u32x4 fa[FM], fw;
  auto read_step = [&](int kt, int s) {
    const uint32_t* st = psm_i4 + (size_t)(kt % STAGES) * S::STAGE_DW;
    const u32x4* la = reinterpret_cast<const u32x4*>(st);
#pragma unroll
    for (int f = 0; f < FM; ++f) fa[f] = la[swz(wm0 + 16 * f + cl, 4 * s + ks)];
    fw = *reinterpret_cast<const u32x4*>(st + S::X_DW + (4 * s + ks) * BN + wn0 + 4 * cl);
  };

  // LoRA add (once per output: slice 0 of a split tile): total starts at
  // scale * U[rows] . B[cols]^T, four 16x16x4 fp32 MFMAs per 16 x 16 block
  // with the block's rows of U as A and its fragment's columns 4 l + c of B
  // as B; MFMA j takes rank index r = 4 k4 + j (k4 = lane / 16) from both, so
  // a lane's operands are four consecutive entries of a U row (one 16-byte
  // load) and of a B row (one 8-byte load when B's rows hold 16 aligned
  // entries; else element loads).  The result lands in the layout of total.
  // The operands are loaded before the prologue's stage loads and multiplied
  // once the first stage has landed.  U's columns past the rank are zero; B
  // is used only below the rank (clamped addresses, selects after the loads).
  const bool lora_on = lora.u && kslice == 0;
  f32x4 ua[FM];
  float bb[4][4];
  if (lora_on) {
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      const int64_t row = m0 + wm0 + 16 * f + cl;
      const f32x4 v = *reinterpret_cast<const f32x4*>(lora.u + (row < m ? row : m - 1) * 16 + 4 * ks);
      ua[f] = row < m ? v : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    const bool bvec = lora.ldb >= 16 && (lora.ldb & 3) == 0 && ((uintptr_t)lora.b & 7u) == 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t col = n0 + wn0 + 4 * cl + c;
      const uint16_t* brow = lora.b + (col < n ? col : n - 1) * lora.ldb;
      uint32_t h[4];
      if (bvec) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(brow + 4 * ks);
        h[0] = w[0] & 0xFFFFu; h[1] = w[0] >> 16; h[2] = w[1] & 0xFFFFu; h[3] = w[1] >> 16;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = brow[4 * ks + j < lora.rank ? 4 * ks + j : 0];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) bb[j][c] = (col < n && 4 * ks + j < lora.rank) ? bf16_bits_to_float(h[j]) : 0.f;
    }
  }

  // all STAGES buffers start filling; stage 0 must land before the first read
#pragma unroll
  for (int st = 0; st < STAGES; ++st)
    if (st < ktiles) issue(st);
  if (ktiles >= STAGES) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 1)));
  } else {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
  }
  lds_barrier();
  read_step(0, 0);
  if (lora_on) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int c = 0; c < 4; ++c) total[f][c] = mfma16_f32(ua[f][j], bb[j][c], total[f][c]);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v) total[f][c][v] *= lora.scale;
  }

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < (ktiles >> 1); ++g) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kt = 2 * g + h;
      u32x4 bn[4];   // the second k step's decoded words, decoded under the first step's MFMAs
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        // reorder / decode this step's fragments (their LDS reads were issued
        // one step earlier, under the previous step's MFMAs); prepared
        // activations are already in pair order
        u32x4 ap[FM], b[4];
#pragma unroll
        for (int f = 0; f < FM; ++f) ap[f] = PREP ? fa[f] : x_pairs_permuted(fa[f]);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = s == 0 ? codes_as_bf16_pairs(fw[c]) : bn[c];
        if (s == 0) read_step(kt, 1);
        const bool first = h == 0 && s == 0;   // first k step of the group
        // the ones-MFMA sums the reordered activations; a sum's order does not matter
#pragma unroll
        for (int f = 0; f < FM; ++f) {
          if constexpr (!PREP) xs[f] = mfma16_bf16(ap[f], ones, first ? zero : xs[f]);
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[f][c] = mfma16_bf16(ap[f], b[c], first ? zero : acc[f][c]);
        }
        if constexpr (LORA) {
          // U[rows][rank] += x . lora_A^T for this k step, by one of the two column
          // waves (the other takes the stage's other step): lora_A row cl, chunk
          // 4 s + ks, in the activations' pair order
          if (wn == s) {
            const uint32_t* al = psm_i4 + (size_t)(kt % STAGES) * S::STAGE_DW + S::X_DW + S::W_DW + S::M_DW;
            const int q = 4 * s + ks;
            const u32x4 raw = *reinterpret_cast<const u32x4*>(al + 32 * cl + 4 * (q ^ (cl & 7)));
            const u32x4 av = cl < lora.rank ? x_pairs_permuted(raw) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int f = 0; f < FM; ++f) uacc[f] = mfma16_bf16(ap[f], av, uacc[f]);
          }
        }
        if (s == 0) {
          // the second step's words (fw now holds them once the reads above
          // land) are decoded while the first step's MFMAs run: the matrix
          // core and the vector ALU then work side by side.  Scheduling
          // order of this step: its own decode, the next step's LDS reads,
          // four MFMAs (covering the read latency), then one MFMA per three
          // decode instructions.
#pragma unroll
          for (int c = 0; c < 4; ++c) bn[c] = codes_as_bf16_pairs(fw[c]);
          if constexpr (PREP && QG_PIPE_INTERLEAVE) {
            __builtin_amdgcn_sched_group_barrier(0x002, 28, 0);   // VALU: this step's decode
            __builtin_amdgcn_sched_group_barrier(0x100, 5, 0);    // DS reads of the next step
            __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);    // MFMA
#pragma unroll
            for (int i = 0; i < 12; ++i) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // MFMA
              __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);  // VALU: next step's decode
            }
          }
        }
      }
      // the group's scales, zeros (and prepared group sums), read while stage
      // kt is still ours
      float sc[4], bz[4];
      f32x4 gs[FM];   // group sums of this lane's accumulator rows 4 ks + v
      if (h == 1) {
        const uint32_t* lm = psm_i4 + (size_t)(kt % STAGES) * S::STAGE_DW + S::X_DW + S::W_DW;
#pragma unroll
        for (int f = 0; f < FM; ++f)
          gs[f] = PREP ? *reinterpret_cast<const f32x4*>(lm + 128 + wm0 + 16 * f + 4 * ks) : xs[PREP ? 0 : f];
        const int col = wn0 + 4 * cl;
        const u32x2 sv = *reinterpret_cast<const u32x2*>(lm + (col >> 1));
        const uint32_t zw = qzeros ? lm[BN / 2 + (col >> 3)] >> (4 * (col & 7)) : 0u;
        sc[0] = half_bits_to_float(sv[0] & 0xFFFFu);
        sc[1] = half_bits_to_float(sv[0] >> 16);
        sc[2] = half_bits_to_float(sv[1] & 0xFFFFu);
        sc[3] = half_bits_to_float(sv[1] >> 16);
#pragma unroll
        for (int c = 0; c < 4; ++c) bz[c] = (float)(128u + ((zw >> (4 * c)) & 15u));
      }
      // Stage kt is fully read (fragments and metadata sit in registers).  With
      // the MFMAs above in flight: wait for this wave's loads of stage kt + 1,
      // meet the other waves (after which every wave is done with stage kt and
      // all of stage kt + 1 has landed), refill stage kt's buffer with stage
      // kt + STAGES and read the first fragments of stage kt + 1.
      if (kt + 1 < ktiles) {
        if (kt + STAGES - 1 < ktiles) {
          __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 2)));
        } else {
          __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        }
        lds_barrier();
        if (kt + STAGES < ktiles) issue(kt + STAGES);
        read_step(kt + 1, 0);
      }
      if (h == 1) {
        // end of group g: scale and remove the 128 + z offset
#pragma unroll
        for (int f = 0; f < FM; ++f)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              total[f][c][v] = __builtin_fmaf(sc[c], __builtin_fmaf(-bz[c], gs[f][v], acc[f][c][v]),
                                              total[f][c][v]);
      }
    }
  }
  if constexpr (LORA) {
    // total += scale * U . B^T for this slice's U (the sum over slices is linear,
    // so every slice adds its own).  The two column waves' shares of U meet in
    // LDS (the stages are done); then four 16x16x4 fp32 MFMAs per 16 x 16 block
    // with a block's U rows as A and its columns of B as B, as for a precomputed U.
    __syncthreads();
    float* ul = reinterpret_cast<float*>(psm_i4);   // [NWN][BM][16]
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v) ul[(wn * BM + wm0 + 16 * f + 4 * ks + v) * 16 + cl] = uacc[f][v];
    __syncthreads();
    f32x4 ua[FM];
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      const int row = wm0 + 16 * f + cl;
      const f32x4 u0 = *reinterpret_cast<const f32x4*>(ul + row * 16 + 4 * ks);
      const f32x4 u1 = *reinterpret_cast<const f32x4*>(ul + (BM + row) * 16 + 4 * ks);
      ua[f] = u0 + u1;
    }
    float bb[4][4];
    const bool bvec = lora.ldb >= 16 && (lora.ldb & 3) == 0 && ((uintptr_t)lora.b & 7u) == 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t col = n0 + wn0 + 4 * cl + c;
      const uint16_t* brow = lora.b + (col < n ? col : n - 1) * lora.ldb;
      uint32_t hh[4];
      if (bvec) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(brow + 4 * ks);
        hh[0] = w[0] & 0xFFFFu; hh[1] = w[0] >> 16; hh[2] = w[1] & 0xFFFFu; hh[3] = w[1] >> 16;
      } else {
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) hh[jj] = brow[4 * ks + jj < lora.rank ? 4 * ks + jj : 0];
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
        bb[jj][c] = (col < n && 4 * ks + jj < lora.rank) ? bf16_bits_to_float(hh[jj]) : 0.f;
    }
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        f32x4 lt = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) lt = mfma16_f32(ua[f][jj], bb[jj][c], lt);
#pragma unroll
        for (int v = 0; v < 4; ++v) total[f][c][v] = __builtin_fmaf(lora.scale, lt[v], total[f][c][v]);
      }
  }
  if (ksplit > 1) {
    // Split k: every slice stores its fp32 partial tile with agent-coherent
    // stores and takes a ticket; the last slice of the tile to arrive adds the
    // partials in slice order (deterministic) and writes Y.  No fences: the
    // partials are only written and read with agent-coherent accesses, and
    // every thread waits for its stores before the ticket is taken (or, with
    // acq_rel, the ticket orders them).
    // fragment order: element pair (f, v, c / 2) of thread tid at
    // ((f * 4 + v) * 2 + c / 2) * T + tid (8-byte words), so that each store
    // instruction of a wave covers 512 contiguous bytes; the last slice reads
    // with the same thread mapping
    uint64_t* mine = reinterpret_cast<uint64_t*>(partials) + ((int64_t)t * ksplit + kslice) * (BM * BN / 2);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          // (the element is copied to a scalar first: a bit cast applied to a
          // vector element directly read element 0 whatever the index)
          const float lo = total[f][2 * h2][v], hi = total[f][2 * h2 + 1][v];
          const uint64_t pair = (uint64_t)__builtin_bit_cast(uint32_t, lo) |
                                ((uint64_t)__builtin_bit_cast(uint32_t, hi) << 32);
          __hip_atomic_store(&mine[((f * 4 + v) * 2 + h2) * T + tid], pair, __ATOMIC_RELAXED,
                             __HIP_MEMORY_SCOPE_AGENT);
        }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    if (tid == 0)
      psm_i4[0] = ticket_add(&tickets[t], acq_rel) == (uint32_t)(ksplit - 1);
    __syncthreads();
    if (!psm_i4[0]) return;
    const uint64_t* base = reinterpret_cast<const uint64_t*>(partials) + (int64_t)t * ksplit * (BM * BN / 2);
    // slice by slice: the 8 FM pairs of a slice are loaded together (one round
    // trip per slice, not per element), then added; each element still sums
    // the slices in slice order
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < 4; ++c) total[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int p = 0; p < ksplit; ++p) {
      const uint64_t* sl = base + (int64_t)p * (BM * BN / 2);
      uint64_t pr[FM][4][2];
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2)
            pr[f][v][h2] = __hip_atomic_load(&sl[((f * 4 + v) * 2 + h2) * T + tid], __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int v = 0; v < 4; ++v)
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2) {
            total[f][2 * h2][v] += __builtin_bit_cast(float, (uint32_t)pr[f][v][h2]);
            total[f][2 * h2 + 1][v] += __builtin_bit_cast(float, (uint32_t)(pr[f][v][h2] >> 32));
          }
    }
    if (tid == 0) __hip_atomic_store(&tickets[t], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();

  // output tile through LDS, then 16-byte (or 8-byte) row stores
  uint16_t* osm = reinterpret_cast<uint16_t*>(psm_i4);
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = wm0 + 16 * f + 4 * ks + v;
      u32x2 o;
      o[0] = pack_bf16x2(total[f][0][v], total[f][1][v]);
      o[1] = pack_bf16x2(total[f][2][v], total[f][3][v]);
      *reinterpret_cast<u32x2*>(&osm[row * S::OP + wn0 + 4 * cl]) = o;
    }
  __syncthreads();
  constexpr int CPR = BN / 8;
  for (int c = tid; c < BM * CPR; c += T) {
    const int r = c / CPR, cc = c - r * CPR;
    const int gr = m0 + r, gc = n0 + 8 * cc;
    const bool in = gr < m && gc < n;
    const uint16_t* src = &osm[r * S::OP + 8 * cc];
    if (in) {
      uint16_t* dst = y + (int64_t)gr * ldy + gc;
      if (vec_store) {
        *reinterpret_cast<u32x4*>(dst) = *reinterpret_cast<const u32x4*>(src);
      } else {
        reinterpret_cast<u32x2*>(dst)[0] = reinterpret_cast<const u32x2*>(src)[0];
        reinterpret_cast<u32x2*>(dst)[1] = reinterpret_cast<const u32x2*>(src)[1];
      }
    }
    if (lora.row_ss) {   // the CPR lanes of a row: one aligned group
      float q = 0.f;
      if (in) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float lo = bf16_bits_to_float(w[i] & 0xFFFFu), hi = bf16_bits_to_float(w[i] >> 16);
          q = __builtin_fmaf(lo, lo, q);
          q = __builtin_fmaf(hi, hi, q);
        }
      }
      add_row_sumsq<CPR>(lora.row_ss, q, gr, cc == 0, gr < m);
    }
  }
}

}  // namespace qg
