// Dense products grouped by expert (rows sorted by group, see groups.hpp):
//
//   NT: C[r] = A[r] . B_e^T    NN: C[r] = A[r] . B_e    for the rows r of group e
//   TN: C_e = A[rows of e]^T . B[rows of e]
//
// bf16 / fp16 with fp32 accumulation, or fp32 throughout.  Three kernels:
//  * many rows a group: pipelined MFMA tiles, a workgroup on each CU going from tile
//    to tile;
//  * few rows a group (decoding): a workgroup takes a strip of columns over the whole of
//    k, split over its waves;
//  * any alignment and size, and fp32: a tile staged through registers.
#include "common.hpp"
#include "groups.hpp"
#include "launch.hpp"
#include <type_traits>

namespace qg {

// Row tiles per band of a group's tile order (GroupTiles): 4 x 8 tiles are
// in flight on an XCD's 32 CUs.
constexpr int kBand = 4;

template <int DTYPE>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return DTYPE == 0 ? mfma16_bf16(a, b, c) : mfma16_f16(a, b, c);
}
template <int DTYPE>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (DTYPE == 0) return (uint16_t)f32_to_bf16_bits(v);
  else return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// ---------------------------------------------------------------------------
// many rows a group: pipelined tiles, one workgroup a CU
//
// BM x BN output tiles, k tiles of 32 in a ring of STAGES LDS buffers filled by
// direct loads, operands in LDS in their memory orientation: K-contiguous ones are
// read as 16-byte chunks, chunk c of row r in slot 4 r + (c ^ (r / 2 % 4)) (the 8 lanes
// that LDS serves at a time then hold 8 different bank groups), M- or
// N-contiguous ones with transposing reads, chunk c of k-row k at k R / 8 + (c ^ fmn(k)).
// NWV waves as WGM row bands x NWV / WGM column bands.  (k tiles of 32 and twice the
// stages against tiles of 64 in the same LDS: the loads of a weight that is read from
// HBM once are in flight for three k tiles of four instead of one of two.)
//
// A workgroup stays on its CU and takes every 32nd (64th) tile of its XCD's run.  When a
// tile's last operands are in registers, the first stages of the next tile are
// issued before its results are written, so neither the first loads' latency nor
// the stores stand between two tiles: an expert's weight gradient has only a few
// k tiles to a 128 KB output tile.  The results go through a wave's own 16 rows of
// LDS, without a barrier.  Loads and stores are issued by every lane (through
// buffer resources that drop what lies outside), so the waits can count them.
//
// Groups end inside tiles.  Rows past the end are not loaded, and a wave whose rows
// or columns are all outside runs only the loads and barriers; bands are numbered so
// that the waves left over sit on different SIMDs.
// ---------------------------------------------------------------------------
constexpr int GBK = 32;    // k of a stage

template <int BM, int BN, int STAGES, int NWV, int WGM>
constexpr size_t grouped_pipe_lds() {
  return (size_t)STAGES * (BM + BN) * GBK * 2 + (size_t)NWV * 16 * (BN / (NWV / WGM)) * 2;
}

template <int LAYOUT, int DTYPE, int BM, int BN, int STAGES, int NWV, int WGM>
__global__ __launch_bounds__(64 * NWV) void grouped_pipe_kernel(GroupedArgs a, int tiles_m, int tiles_n, int vec) {
  constexpr bool A_MN = LAYOUT == 2, B_MN = LAYOUT != 0;      // A stored [K][M], B stored [K][N]
  constexpr int T = 64 * NWV, WGN = NWV / WGM;
  constexpr int WM = BM / WGM, WN = BN / WGN, FM = WM / 16, FN = WN / 16;
  constexpr int A_SLOTS = BM * 4, B_SLOTS = BN * 4, STAGE = A_SLOTS + B_SLOTS;   // 16-byte chunks
  constexpr int A_LOADS = A_SLOTS / T, B_LOADS = B_SLOTS / T, LOADS = A_LOADS + B_LOADS;
  constexpr int STORES = WM * WN / 512;                       // 16-byte stores of a lane per tile
  static_assert(A_SLOTS % T == 0 && B_SLOTS % T == 0 && T % 64 == 0 && WM * WN % 512 == 0, "chunks per thread");
  static_assert(LOADS * (STAGES - 1) + STORES <= 63, "vmcnt range");
  extern __shared__ __attribute__((aligned(16))) u32x4 gsm[];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cl = lane & 15, ks = lane >> 4;
  const int wm0 = (wave / WGN) * WM, wn0 = (wave % WGN) * WN;
  u32x4* stage_out = gsm + STAGES * STAGE + wave * (2 * WN);  // 16 rows x WN of 16-bit results
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3, slots = gridDim.x >> 3;

  // (in_vgpr below keeps a tile's address arithmetic inside the loop over tiles: hoisted
  // out of it, it would take the registers that the accumulators leave)
  // The tile being computed, and (from its last k tile on) the one being loaded.
  struct Tile {
    const uint16_t *A, *B;    // first row or column of the tile's operands, at k = 0
    uint16_t* C;              // its first element
    int m, n, k;              // rows and columns left from its first on, and k
  };
  const GroupTiles map(a.offsets, (int)a.groups, (int)a.rows, BM, tiles_n, kBand, lane);
  auto find = [&](int64_t i, Tile& t) {
    int64_t tm, tn, row0 = 0;
    if constexpr (LAYOUT == 2) {
      // every group has tiles_m x tiles_n tiles over its own number of rows; an XCD
      // takes one eighth of every group's tiles, since groups differ in length
      const int tiles = tiles_m * tiles_n, per = (tiles + 7) >> 3;
      const int64_t e = i / per;
      const int q = xcd * per + (int)(i - e * per);
      if (e >= a.groups) return false;
      const int b = q / (kBand * tiles_n), in = q - b * kBand * tiles_n;
      const int height = max(min(kBand, tiles_m - b * kBand), 1);
      const bool work = q < tiles;           // an XCD's share of a group may be short
      tn = work ? in / height : 0;
      tm = work ? b * kBand + in % height : 0;
      int lo;
      const int rows = map.rows_of((int)e, &lo);
      t.k = work ? rows : 0;
      t.A = a.A + lo * a.lda + tm * BM;
      t.B = a.B + lo * a.ldb + tn * BN;
      t.C = a.C + e * a.sc;
      t.m = work ? (int)a.M : 0;
    } else {
      const GroupTile g = map.find(xcd, i);
      if (g.group < 0) return false;
      tm = g.tm;
      tn = g.tn;
      row0 = g.row0;
      t.k = (int)a.K;
      t.A = a.A + (row0 + tm * BM) * a.lda;
      t.B = a.B + g.group * a.sb + (B_MN ? tn * BN : tn * BN * a.ldb);
      t.C = a.C;
      t.m = g.rows;
    }
    t.C += (row0 + tm * BM) * a.ldc + tn * BN;
    t.m -= (int)tm * BM;
    t.n = (int)(a.N - tn * BN);
    return true;
  };

  // Byte offset of chunk tid + T i of an operand's stage region from the tile's first
  // element (kOutside: past the operand's rows or columns), and its first k.
  uint32_t aoff[A_LOADS], boff[B_LOADS];
  auto chunk_k = [&](bool mn, int R, int i) {
    return mn ? (tid + T * i) / (R / 8) : 8 * ((tid & 3) ^ ((tid >> 3) & 3));
  };
  auto offset = [&](auto mn, auto r_, int s, int64_t ld, int left) {
    constexpr int R = decltype(r_)::value;
    if constexpr (decltype(mn)::value) {
      const int k = s / (R / 8), c = (s % (R / 8)) ^ fmn_r<R>(k);
      return 8 * c < left ? (uint32_t)(2 * (k * ld + 8 * c)) : kOutside;
    } else {
      const int r = s >> 2, c = (s & 3) ^ ((r >> 1) & 3);
      return r < left ? (uint32_t)(2 * (r * ld + 8 * c)) : kOutside;
    }
  };
  auto set_offsets = [&](const Tile& t) {
    const int id = (int)in_vgpr(tid);
#pragma unroll
    for (int i = 0; i < A_LOADS; ++i)
      aoff[i] = offset(std::bool_constant<A_MN>{}, std::integral_constant<int, BM>{}, id + T * i, a.lda, t.m);
#pragma unroll
    for (int i = 0; i < B_LOADS; ++i)
      boff[i] = offset(std::bool_constant<B_MN>{}, std::integral_constant<int, BN>{}, id + T * i, a.ldb, t.n);
  };
  const int64_t astep = A_MN ? GBK * a.lda : GBK, bstep = B_MN ? GBK * a.ldb : GBK;
  // direct load j of stage st: 64 consecutive chunks a wave; zeros past k
  auto issue1 = [&](const Tile& t, int st, int j) {
    u32x4* base = gsm + (st % STAGES) * STAGE + 64 * wave;
    const int left = t.k - GBK * st;
    if (j < A_LOADS)
      buffer_to_lds16_or_zero(t.A + st * astep, chunk_k(A_MN, BM, j) < left ? aoff[j] : kOutside, base + T * j);
    else
      buffer_to_lds16_or_zero(t.B + st * bstep, chunk_k(B_MN, BN, j - A_LOADS) < left ? boff[j - A_LOADS] : kOutside,
                              base + A_SLOTS + T * (j - A_LOADS));
  };
  auto issue_first = [&](const Tile& t) {
#pragma unroll
    for (int st = 0; st < STAGES; ++st)
#pragma unroll
      for (int j = 0; j < LOADS; ++j) issue1(t, st, j);
  };

  f32x4 acc[FM][FN];
  // Operand fragments of a k tile: row blocks of A, column blocks of B.
  // K-contiguous: a block is one 16-byte read, blocks 16 rows apart.  Transposed: two
  // 8-byte reads at k-rows 8 ks + r4 and 8 ks + 4 + r4, which have the same chunk XOR; the XOR
  // and a block's column bits do not carry into each other, so block c is at the first
  // one's address XOR 32 c bytes.
  const int r4 = (lane & 15) >> 2, q4 = lane & 3;
  auto first_at = [&](bool mn, int R, int first) -> uint32_t {    // bytes from the operand's region
    if (!mn) return (4 * (first + cl) + (ks ^ ((cl >> 1) & 3))) * 16;
    const int x = (2 * (r4 | 4 * (ks & 1))) & (R / 8 - 1);
    return ((8 * ks + r4) * (R / 8) + (((first >> 3) ^ x) | (q4 >> 1))) * 16 + 8 * (q4 & 1);
  };
  const uint32_t a_first = lds_address(gsm) + first_at(A_MN, BM, wm0);
  const uint32_t b_first = lds_address(gsm) + first_at(B_MN, BN, wn0) + 16 * A_SLOTS;
  auto read_rows = [&](uint32_t first, int kt, int block) {    // K-contiguous
    const char* l = reinterpret_cast<const char*>(gsm) + (first - lds_address(gsm));
    return *reinterpret_cast<const u32x4*>(l + kt % STAGES * (16 * STAGE) + 16 * 64 * block);
  };
  auto read_columns = [&](auto r_, uint32_t first, int kt, int block, auto& out) {    // transposed
    constexpr int R = decltype(r_)::value, N = sizeof(out) / sizeof(out[0]);
    uint32_t at[N];
#pragma unroll
    for (int i = 0; i < N; ++i) at[i] = (first + kt % STAGES * (16 * STAGE)) ^ (32 * (block + i));
    read_transposed<N, 8 * R>(at, out);
  };

  // A k tile is FM rows of FN matrix instructions.  Its one barrier (stage kt + 1 has landed
  // for every wave, nobody reads stage kt any more) sits AHEAD rows before its end, when
  // every operand of the stage is in registers; over the rows that are left the stage's
  // buffer is refilled with stage kt + STAGES and the next k tile's first operands are read.
  // K-contiguous row blocks of A are read AHEAD rows ahead into a ring, transposed ones four at
  // a time into two sets of four; B's column blocks one k tile ahead (set P holds this one's).
  // So only a few operands are held beside the accumulators.
  constexpr int AHEAD = 3, RING = AHEAD + 1;
  static_assert(FM % RING == 0 && (!A_MN || FM == 2 * RING), "the ring meets at the end of a k tile");
  u32x4 ra[A_MN ? 2 : 1][RING], rb[2][FN];
  // `behind`: stores of the previous tile were issued after this tile's first stages
  auto wait_stage = [&](bool behind, bool refill) {
    if (behind) __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 2) + STORES) & ~(0xF << 8));
    else if (refill) __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 2)) & ~(0xF << 8));
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & ~(0xF << 8));
    lds_barrier();
  };
  auto first_operands = [&](int kt, auto p_) {    // a k tile's, when nothing can be read ahead
    constexpr int P = decltype(p_)::value;
    if constexpr (B_MN) {
      read_columns(std::integral_constant<int, BN>{}, b_first, kt, 0, rb[P]);
    } else {
#pragma unroll
      for (int c = 0; c < FN; ++c) rb[P][c] = read_rows(b_first, kt, c);
    }
    if constexpr (A_MN) {
      read_columns(std::integral_constant<int, BM>{}, a_first, kt, 0, ra[0]);
    } else {
#pragma unroll
      for (int f = 0; f < AHEAD; ++f) ra[0][f] = read_rows(a_first, kt, f);
    }
  };
  // (refill = kt + STAGES < ktiles and next = kt + 1 < ktiles: constants where they are known)
  auto k_tile = [&](auto p_, const Tile& t, int kt, bool behind, auto refill, auto next) {
    constexpr int P = decltype(p_)::value;
#pragma unroll
    for (int q = 0; q < FM; ++q) {
      const int left = q - (FM - AHEAD);
      if (left == 0) {
        wait_stage(behind, refill);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!A_MN) {
        if (left < 0) ra[0][(q + AHEAD) % RING] = read_rows(a_first, kt, q + AHEAD);
        else if (next) ra[0][(q + AHEAD) % RING] = read_rows(a_first, kt + 1, left);
      } else {
        if (q == 1) read_columns(std::integral_constant<int, BM>{}, a_first, kt, RING, ra[1]);
        if (left == 2 && next) read_columns(std::integral_constant<int, BM>{}, a_first, kt + 1, 0, ra[0]);
      }
      if constexpr (!B_MN) {
#pragma unroll
        for (int c = 0; c < FN; ++c)
          if (left >= 0 && c * AHEAD / FN == left && next) rb[P ^ 1][c] = read_rows(b_first, kt + 1, c);
      } else {
        if (left == 1 && next) read_columns(std::integral_constant<int, BN>{}, b_first, kt + 1, 0, rb[P ^ 1]);
      }
      if (left >= 0 && refill) {
#pragma unroll
        for (int j = 0; j < LOADS; ++j)
          if (j * AHEAD / LOADS == left) issue1(t, kt + STAGES, j);
      }
      // B's fragment first: a lane then holds four adjacent columns (4 ks .. 4 ks + 3 of a
      // 16 x 16 block) of row cl
#pragma unroll
      for (int c = 0; c < FN; ++c) acc[q][c] = mfma16<DTYPE>(rb[P][c], ra[A_MN ? q / RING : 0][q % RING], acc[q][c]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Results of a tile: 16 rows at a time through the wave's LDS rows (16-byte chunk c of
  // row r in slot c ^ (r mod the chunks of a row)), then 16-byte stores.
  auto write = [&](const Tile& t) {
    constexpr int CPR = WN / 8;                        // 16-byte chunks a row
    const int rows = t.m - wm0, cols = t.n - wn0;
    const int id = (int)in_vgpr(lane), cl = id & 15, ks = id >> 4;
    uint16_t* C = t.C + (int64_t)wm0 * a.ldc + wn0;
#pragma unroll
    for (int f = 0; f < FM; ++f) {
#pragma unroll
      for (int c = 0; c < FN; ++c) {
        u32x2 o;
        if constexpr (DTYPE == 0) {
          o[0] = pack_bf16x2(acc[f][c][0], acc[f][c][1]);
          o[1] = pack_bf16x2(acc[f][c][2], acc[f][c][3]);
        } else {
          o[0] = pack_f16x2(acc[f][c][0], acc[f][c][1]);
          o[1] = pack_f16x2(acc[f][c][2], acc[f][c][3]);
        }
        u32x4* p = stage_out + cl * CPR + ((2 * c + (ks >> 1)) ^ (cl & (CPR - 1)));
        reinterpret_cast<u32x2*>(p)[ks & 1] = o;
      }
#pragma unroll
      for (int i = 0; i < 16 * CPR / 64; ++i) {
        const int r = (id + 64 * i) / CPR, c = (id + 64 * i) % CPR;
        const u32x4 v = stage_out[r * CPR + (c ^ (r & (CPR - 1)))];
        const int row = 16 * f + r;
        if (vec) {
          buffer_store16_or_none(C, row < rows && 8 * c < cols ? (uint32_t)(2 * (row * a.ldc + 8 * c)) : kOutside, v);
        } else if (row < rows) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (8 * c + e < cols) C[row * a.ldc + 8 * c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  };

  Tile cur;
  if (!find(slot, cur)) return;
  set_offsets(cur);
  issue_first(cur);
  bool behind = false;                                 // stores issued after cur's first stages
  for (int64_t i = slot;; i += slots) {
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < FN; ++c) acc[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int ktiles = (cur.k + GBK - 1) / GBK;
    // stage 0 has landed
    if (behind) __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 1) + STORES));
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 1)));
    lds_barrier();
    if (wm0 < cur.m && wn0 < cur.n) {
      first_operands(0, std::integral_constant<int, 0>{});
      int kt = 0;
      const std::integral_constant<int, 0> even;
      const std::integral_constant<int, 1> odd;
      for (; kt + 1 + STAGES < ktiles; kt += 2) {
        // (the first STAGES stages were issued before the previous tile's stores)
        k_tile(even, cur, kt, behind && kt <= STAGES - 2, std::true_type{}, std::true_type{});
        k_tile(odd, cur, kt + 1, behind && kt + 1 <= STAGES - 2, std::true_type{}, std::true_type{});
      }
      for (; kt < ktiles; kt += 2) {
        k_tile(even, cur, kt, behind && kt == 0, kt + STAGES < ktiles, kt + 1 < ktiles);
        if (kt + 1 < ktiles) k_tile(odd, cur, kt + 1, false, kt + 1 + STAGES < ktiles, kt + 2 < ktiles);
      }
    } else {
      for (int kt = 0; kt < ktiles; ++kt) {
        const bool refill = kt + STAGES < ktiles;
        wait_stage(behind && kt == 0, refill);
        if (refill) {
#pragma unroll
          for (int j = 0; j < LOADS; ++j) issue1(cur, kt + STAGES, j);
        }
      }
    }
    // nobody reads the stages any more, and nothing is on its way into them
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & ~(0xF << 8));
    lds_barrier();
    Tile nxt;
    const bool more = find(i + slots, nxt);
    if (more) {
      set_offsets(nxt);
      issue_first(nxt);
    }
    const bool mine = wm0 < cur.m && wn0 < cur.n;
    if (mine) write(cur);
    if (!more) return;
    // (element-wise stores are not counted: wait for them and the first stages)
    if (!vec) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    behind = mine && vec;
    cur = nxt;
  }
}

// ---------------------------------------------------------------------------
// few rows a group: strips of columns over the whole of k
//
// A workgroup owns 16 rows of a group and a strip of columns; its waves take blocks of
// k in turn, all loads of a block issued before its MFMAs, operands straight from memory
// into the MFMA lane layout (lane l: row or column l % 16, k chunk l / 16), and the waves'
// partial tiles are summed through LDS in wave order.  The activations are read from L2,
// only by the lanes whose rows there are.
// ---------------------------------------------------------------------------
// NT, B K-contiguous: strip of 16 columns, blocks of 256 k, so a column's 512
// contiguous bytes are read by one wave.
// NN, B N-contiguous: strip of 128 columns; lane (c, q) loads columns 8c .. 8c + 7
// of the 8 k-rows 8q .. 8q + 7 and transposes the 8 x 8 block in registers:
// fragment j then holds column 8c + j (256 contiguous bytes per k-row).
// Against the pipelined kernel (bf16, weights from HBM): 64 / 128 / 256 / 384 rows over 64 experts,
// 2048 -> 1024, NT 35.6 / 47.8 / 58.4 / 64.5 us here, 47.4 / 52.4 / 58.9 / 61.6 us there; 16 / 32 / 64 rows
// over 8, 4096 -> 8192, NT 72 / 93 / 115 against 85 / 98 / 106 us, NN 77 / 92 / 109 against 80 / 96 / 102 us: the
// small workgroups spread evenly over the CUs, the tiles load a weight once for all rows.
// So up to 4 rows a group on average, and up to 8 where the tiles would not reach every CU.
constexpr int kStripRows = 4, kStripRowsFew = 8;
constexpr int kStripK = 256;      // k per block, NT
constexpr int kStripKN = 32;      // k per block, NN

template <int LAYOUT, int DTYPE>
__global__ __launch_bounds__(512) void grouped_strip_kernel(GroupedArgs a, int strips) {
  constexpr int CT = LAYOUT == 0 ? 1 : 8;               // 16-column MFMA tiles of the strip
  constexpr int COLS = 16 * CT, ROWS = 16;
  extern __shared__ __attribute__((aligned(16))) float ssm[];   // [waves][ROWS][COLS + 4]
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const GroupTile g = find_group_tile(a.offsets, (int)a.groups, (int)a.rows, ROWS, strips, 1, blockIdx.x, lane);
  if (g.group < 0) return;
  const int cl = lane & 15, ks = lane >> 4;
  const int K = (int)a.K, N = (int)a.N;
  const int r0 = g.tm * ROWS, n0 = g.tn * COLS;
  const uint16_t* arow = a.A + (int64_t)(g.row0 + min(r0 + cl, g.rows - 1)) * a.lda;
  const uint16_t* B = a.B + (int64_t)g.group * a.sb;

  f32x4 acc[CT];
#pragma unroll
  for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0u, 0u, 0u, 0u};

  if constexpr (LAYOUT == 0) {
    const uint16_t* brow = B + (int64_t)min(n0 + cl, N - 1) * a.ldb;
    for (int k0 = kStripK * wave; k0 < K; k0 += kStripK * waves) {
      u32x4 b[8], x[8];
      // past the end of k both operands are zeros (loads from the row's start)
      if (k0 + kStripK <= K) {
#pragma unroll
        for (int s = 0; s < 8; ++s) b[s] = *reinterpret_cast<const u32x4*>(brow + k0 + 32 * s + 8 * ks);
#pragma unroll
        for (int s = 0; s < 8; ++s) x[s] = zero;
        if (r0 + cl < g.rows) {
#pragma unroll
          for (int s = 0; s < 8; ++s) x[s] = *reinterpret_cast<const u32x4*>(arow + k0 + 32 * s + 8 * ks);
        }
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int k = k0 + 32 * s + 8 * ks;
          b[s] = *reinterpret_cast<const u32x4*>(brow + (k < K ? k : 0));
          if (k >= K) b[s] = zero;
          x[s] = *reinterpret_cast<const u32x4*>(arow + (k < K ? k : 0));
          if (k >= K) x[s] = zero;
        }
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) acc[0] = mfma16<DTYPE>(x[s], b[s], acc[0]);
    }
  } else {
    const int col = min(n0 + 8 * cl, N - 8);
    for (int k0 = kStripKN * wave; k0 < K; k0 += kStripKN * waves) {
      u32x4 in[8], b[8], x;
      const int k = k0 + 8 * ks;
      if (k0 + kStripKN <= K) {
#pragma unroll
        for (int i = 0; i < 8; ++i) in[i] = *reinterpret_cast<const u32x4*>(B + (int64_t)(k + i) * a.ldb + col);
        x = zero;
        if (r0 + cl < g.rows) x = *reinterpret_cast<const u32x4*>(arow + k);
      } else {   // K % 8 == 0: a lane's 8 k-rows are all inside or all outside
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          in[i] = *reinterpret_cast<const u32x4*>(B + (int64_t)(k < K ? k + i : 0) * a.ldb + col);
          if (k >= K) in[i] = zero;
        }
        x = *reinterpret_cast<const u32x4*>(arow + (k < K ? k : 0));
        if (k >= K) x = zero;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int p = 0; p < 4; ++p) b[j][p] = __builtin_amdgcn_perm(in[2 * p + 1][j >> 1], in[2 * p][j >> 1], sel);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = mfma16<DTYPE>(x, b[j], acc[j]);
    }
  }

  // lane (cl, ks) holds rows 4 ks + v and column cl (NT) or 8 cl + c (NN)
  constexpr int P = COLS + 4;
  float* mine = ssm + wave * ROWS * P;
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int v = 0; v < 4; ++v) mine[(4 * ks + v) * P + (LAYOUT == 0 ? cl : 8 * cl + c)] = acc[c][v];
  __syncthreads();
  for (int i = tid; i < ROWS * COLS; i += blockDim.x) {
    const int r = i / COLS, c = i - r * COLS;
    if (r0 + r >= g.rows || n0 + c >= N) continue;
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += ssm[(w * ROWS + r) * P + c];
    a.C[(int64_t)(g.row0 + r0 + r) * a.ldc + n0 + c] = round16<DTYPE>(s);
  }
}

// ---------------------------------------------------------------------------
// any alignment, fp32: BM x 64 tiles staged through registers
//
// 4 waves (2 x 2, BM / 2 x 32 each), k tiles of 32 in two LDS buffers, loads guarded:
// zeros past M, N and k, so nothing outside the matrices is read.  Elements are
// loaded one by one along the operand's contiguous direction and stored K-contiguous
// in LDS; with VEC (fp32 whose rows start on 16 bytes and hold whole quadruples) four at
// a time, kept in their memory orientation.
//
// fp32 is bound by the matrix cores, and then by how evenly the tiles fall on the CUs:
// 1402 rows over 8 groups, 1000 -> 1416, take 79 us one by one with 64 rows, 70 us with VEC,
// 64 us with VEC and 32 rows (27 us at the rate of a large library product).
// ---------------------------------------------------------------------------
template <int LAYOUT, typename T, int BM, bool VEC>
__global__ __launch_bounds__(256) void grouped_tile_kernel(GroupedArgs a, int tiles_m, int tiles_n) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr bool BF = std::is_same<T, __bf16>::value;
  constexpr int BN = 64, BK = 32, P = BK + 8;     // LDS row pitch (16-byte rows)
  constexpr int FM = BM / 32;                                    // 16-row blocks of a wave
  __shared__ __attribute__((aligned(16))) T sm[2][(BM + BN) * P];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, cl = lane & 15, ks = lane >> 4;
  const T* A = reinterpret_cast<const T*>(a.A);
  const T* B = reinterpret_cast<const T*>(a.B);
  T* C = reinterpret_cast<T*>(a.C);
  int64_t M, K;
  int tm, tn;
  if constexpr (LAYOUT == 2) {
    const int tiles = tiles_m * tiles_n, e = blockIdx.x / tiles, t = blockIdx.x - e * tiles;
    int lo;
    K = group_rows(a.offsets, e, (int)a.rows, &lo);
    M = a.M;
    A += (int64_t)lo * a.lda;
    B += (int64_t)lo * a.ldb;
    C += e * a.sc;
    tm = t / tiles_n;
    tn = t - tm * tiles_n;
  } else {
    const GroupTile g = find_group_tile(a.offsets, (int)a.groups, (int)a.rows, BM, tiles_n, kBand, blockIdx.x, lane);
    if (g.group < 0) return;
    A += (int64_t)g.row0 * a.lda;
    B += (int64_t)g.group * a.sb;
    C += (int64_t)g.row0 * a.ldc;
    M = g.rows;
    K = a.K;
    tm = g.tm;
    tn = g.tn;
  }
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN, N = a.N;
  constexpr bool A_MN = LAYOUT == 2, B_MN = LAYOUT != 0;

  // element i of a thread: K-contiguous: row tid / 32 + 8 i, k tid % 32; else: row tid % R,
  // k tid / R + 256 / R i.  VEC, quadruple i: row tid / 8 + 32 i, k 4 (tid % 8); else: rows from
  // 4 (tid % (R / 4)) on, k tid / (R / 4) + 1024 / R i, in LDS k-rows of R + 4 elements.
  auto load = [&](auto r_, const T* p, int64_t ld, bool mn, int64_t first, int64_t end, int64_t k0, auto& reg) {
    constexpr int R = decltype(r_)::value, PER = R * BK / 256;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) {
        const int64_t r = first + (mn ? 4 * (tid % (R / 4)) : (tid >> 3) + 32 * i);
        const int64_t k = k0 + (mn ? tid / (R / 4) + 1024 / R * i : 4 * (tid & 7));
        const f32x4 v = r < end && k < K ? *reinterpret_cast<const f32x4*>(p + (mn ? k * ld + r : r * ld + k))
                                         : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) reg[4 * i + j] = v[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int64_t r = first + (mn ? tid % R : (tid >> 5) + 8 * i), k = k0 + (mn ? tid / R + 256 / R * i : tid & 31);
        reg[i] = r < end && k < K ? (mn ? p[k * ld + r] : p[r * ld + k]) : (T)0.f;
      }
    }
  };
  auto store = [&](auto r_, T* region, bool mn, const auto& reg) {
    constexpr int R = decltype(r_)::value, PER = R * BK / 256;
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < PER / 4; ++i)
        *reinterpret_cast<f32x4*>(region + (mn ? (tid / (R / 4) + 1024 / R * i) * (R + 4) + 4 * (tid % (R / 4))
                                               : ((tid >> 3) + 32 * i) * P + 4 * (tid & 7))) =
            f32x4{reg[4 * i], reg[4 * i + 1], reg[4 * i + 2], reg[4 * i + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        region[mn ? (tid % R) * P + tid / R + 256 / R * i : ((tid >> 5) + 8 * i) * P + (tid & 31)] = reg[i];
    }
  };
  // fp32: the k 16 q + 4 ks .. + 3 of a row (the same k of both operands)
  auto quad = [&](auto r_, const T* region, bool mn, int row, int q) {
    if constexpr (VEC) {
      constexpr int PM = decltype(r_)::value + 4;
      if (mn) {
        const T* c = region + (16 * q + 4 * ks) * PM + row;
        return f32x4{c[0], c[PM], c[2 * PM], c[3 * PM]};
      }
    }
    return *reinterpret_cast<const f32x4*>(region + row * P + 16 * q + 4 * ks);
  };
  const std::integral_constant<int, BM> RA;
  const std::integral_constant<int, BN> RB;
  f32x4 acc[FM][2];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int c = 0; c < 2; ++c) acc[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm = (wave & 1) * (BM / 2), wn = (wave >> 1) * 32;
  T ra[BM * BK / 256], rb[BN * BK / 256];
  const int64_t ktiles = (K + BK - 1) / BK;
  if (ktiles > 0) {
    load(RA, A, a.lda, A_MN, m0, M, 0, ra);
    load(RB, B, a.ldb, B_MN, n0, N, 0, rb);
    store(RA, sm[0], A_MN, ra);
    store(RB, sm[0] + BM * P, B_MN, rb);
  }
  __syncthreads();
  for (int64_t kt = 0; kt < ktiles; ++kt) {
    const int buf = (int)(kt & 1);
    const bool more = kt + 1 < ktiles;
    if (more) {
      load(RA, A, a.lda, A_MN, m0, M, (kt + 1) * BK, ra);
      load(RB, B, a.ldb, B_MN, n0, N, (kt + 1) * BK, rb);
    }
    const T *la = sm[buf], *lb = la + BM * P;
    if constexpr (F32) {
#pragma unroll
      for (int q = 0; q < BK / 16; ++q) {
        f32x4 x[FM], w[2];
#pragma unroll
        for (int f = 0; f < FM; ++f) x[f] = quad(RA, la, A_MN, wm + 16 * f + cl, q);
#pragma unroll
        for (int c = 0; c < 2; ++c) w[c] = quad(RB, lb, B_MN, wn + 16 * c + cl, q);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < FM; ++f)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[f][c] = mfma16_f32(x[f][j], w[c][j], acc[f][c]);
      }
    } else {
      u32x4 x[FM], w[2];
#pragma unroll
      for (int f = 0; f < FM; ++f) x[f] = *reinterpret_cast<const u32x4*>(la + (wm + 16 * f + cl) * P + 8 * ks);
#pragma unroll
      for (int c = 0; c < 2; ++c) w[c] = *reinterpret_cast<const u32x4*>(lb + (wn + 16 * c + cl) * P + 8 * ks);
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[f][c] = mfma16<BF ? 0 : 1>(x[f], w[c], acc[f][c]);
    }
    if (more) {
      store(RA, sm[buf ^ 1], A_MN, ra);
      store(RB, sm[buf ^ 1] + BM * P, B_MN, rb);
    }
    __syncthreads();
  }
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t r = m0 + wm + 16 * f + 4 * ks + v, n = n0 + wn + 16 * c + cl;
        if (r < M && n < N) C[r * a.ldc + n] = (T)acc[f][c][v];
      }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Whether 16-byte operand loads fit: the operands' contiguous extents, leading
// dimensions and group stride are multiples of 8 elements.
static bool vectorizable(const GroupedArgs& a) {
  if (!aligned16(a.A) || !aligned16(a.B) || a.lda % 8 || a.ldb % 8) return false;
  // the pipelined tile addresses 256 rows in 31 bits
  if (a.lda > (int64_t)1 << 21 || a.ldb > (int64_t)1 << 21 || a.ldc > (int64_t)1 << 21) return false;
  if (a.layout == 2) return a.M % 8 == 0 && a.N % 8 == 0;
  return a.sb % 8 == 0 && a.K % 8 == 0 && (a.layout == 0 || a.N % 8 == 0);
}

// The kernel a product takes: kind, rows and columns of a tile, threads.
struct GroupedPlan {
  enum Kind { kTile, kStrip, kPipe } kind;
  int bm, bn, threads;
  int64_t blocks;
};

constexpr int kCus = 256;

// Row tile of the pipelined kernel: a launch takes ceil(tiles / resident workgroups)
// rounds of one tile's time, relative to 256 x 256 taken as 0.78 for 128 x 256 and 0.65 for
// 64 x 128 with two workgroups a CU.  Measured with 256 / 128 / 64 rows (bf16): 8192 rows over
// 32 groups, 2048 -> 5632, NT 275 / 310 / 425 us; 4096 rows over 16, 5632 -> 2048, NN 147 / 199 /
// 205 us; 12000 rows over 16, 1024 -> 1024, NT 29.4 / 36.4 / 47.1 us; 3200 rows 24.6 / 18.1 /
// 17.4 us.  Groups' last row tiles are taken as half full.
static int pick_row_tile(int64_t rows, int64_t groups, int64_t N) {
  int best = 64;
  double best_cost = 1e300;
  for (int bm : {256, 128, 64}) {
    if (bm > 64 && bm / 4 > rows / groups) continue;
    const int64_t tiles = (rows / bm + (groups + 1) / 2) * (bm == 64 ? (N + 127) / 128 : (N + 255) / 256);
    const int64_t resident = bm == 64 ? 2 * kCus : kCus;
    const double cost = (double)((tiles + resident - 1) / resident) * (bm == 256 ? 1.0 : bm == 128 ? 0.78 : 0.65);
    if (cost < best_cost) {
      best_cost = cost;
      best = bm;
    }
  }
  return best;
}

static GroupedPlan plan_grouped(const GroupedArgs& a) {
  GroupedPlan p{GroupedPlan::kTile, 64, 64, 256, 0};
  const int64_t avg = a.rows / a.groups;
  if (a.dtype == 2) {
    // 32-row tiles while 64-row ones would be fewer than 4 a CU
    const int64_t row_tiles = a.layout == 2 ? a.groups * ((a.M + 63) / 64) : a.rows / 64 + (a.groups + 1) / 2;
    if (row_tiles * ((a.N + 63) / 64) < 4 * kCus) p.bm = 32;
  } else if (a.K > 0 && vectorizable(a)) {
    if (a.layout == 2) {
      // 128 x 256 tiles (4 waves, two workgroups a CU) where 256 x 256 ones would leave
      // half of the CUs idle
      const int64_t big = a.groups * ((a.M + 255) / 256) * ((a.N + 255) / 256);
      p = big > kCus / 2 ? GroupedPlan{GroupedPlan::kPipe, 256, 256, 512, 0}
                         : GroupedPlan{GroupedPlan::kPipe, 128, 256, 256, 0};
    } else if (avg <= kStripRows ||
               (avg <= kStripRowsFew && (a.rows < a.groups ? a.rows : a.groups) * ((a.N + 127) / 128) <= kCus)) {
      const int64_t k_block = a.layout == 0 ? kStripK : kStripKN, waves = (a.K + k_block - 1) / k_block;
      p = {GroupedPlan::kStrip, 16, a.layout == 0 ? 16 : 128, (int)(64 * (waves < 8 ? waves : 8)), 0};
    } else {
      const int bm = pick_row_tile(a.rows, a.groups, a.N);
      p = {GroupedPlan::kPipe, bm, bm == 64 ? 128 : 256, bm == 64 ? 256 : 512, 0};
    }
  }
  const int64_t tiles_n = (a.N + p.bn - 1) / p.bn;
  if (a.layout != 2) {
    p.blocks = group_tile_blocks(a.rows, a.groups, p.bm, tiles_n);
  } else {
    const int64_t tiles = (a.M + p.bm - 1) / p.bm * tiles_n;
    p.blocks = a.groups * (p.kind == GroupedPlan::kPipe ? (tiles + 7) / 8 * 8 : tiles);
  }
  // one workgroup of 8 waves a CU, or two of 4
  const int64_t resident = p.threads == 256 ? 2 * kCus : kCus;
  if (p.kind == GroupedPlan::kPipe && p.blocks > resident) p.blocks = resident;
  return p;
}

int64_t grouped_threads(const GroupedArgs& a) {
  const GroupedPlan p = plan_grouped(a);
  return p.blocks * p.threads;
}

template <int LAYOUT, int DTYPE, int BM, int BN, int STAGES, int NWV, int WGM>
static void pipe_launch(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  constexpr size_t lds = grouped_pipe_lds<BM, BN, STAGES, NWV, WGM>();
  static_assert(lds <= 160 * 1024, "LDS of a CU");
  const int vec = aligned16(a.C) && a.ldc % 8 == 0 && a.N % 8 == 0 && (LAYOUT != 2 || a.sc % 8 == 0);
  grouped_pipe_kernel<LAYOUT, DTYPE, BM, BN, STAGES, NWV, WGM><<<dim3((unsigned)p.blocks), dim3(64 * NWV), lds, stream>>>(
      a, LAYOUT == 2 ? (int)((a.M + BM - 1) / BM) : 0, (int)((a.N + BN - 1) / BN), vec);
}

template <int LAYOUT, int DTYPE>
static void strip_launch(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  const size_t lds = (size_t)(p.threads / 64) * 16 * (p.bn + 4) * 4;
  grouped_strip_kernel<LAYOUT, DTYPE><<<dim3((unsigned)p.blocks), dim3((unsigned)p.threads), lds, stream>>>(
      a, (int)((a.N + p.bn - 1) / p.bn));
}

template <int LAYOUT, typename T, int BM>
static void tile_launch(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  const int tiles_m = LAYOUT == 2 ? (int)((a.M + BM - 1) / BM) : 0, tiles_n = (int)((a.N + 63) / 64);
  if constexpr (sizeof(T) == 4) {
    const int64_t a_contig = LAYOUT == 2 ? a.M : a.K, b_contig = LAYOUT == 0 ? a.K : a.N;
    if (aligned16(a.A) && aligned16(a.B) && (a.lda | a.ldb | a.sb | a_contig | b_contig) % 4 == 0) {
      grouped_tile_kernel<LAYOUT, T, BM, true><<<grid, dim3(256), 0, stream>>>(a, tiles_m, tiles_n);
      return;
    }
  }
  grouped_tile_kernel<LAYOUT, T, BM, false><<<grid, dim3(256), 0, stream>>>(a, tiles_m, tiles_n);
}

template <int LAYOUT>
static void dispatch32(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  if (p.bm == 32) tile_launch<LAYOUT, float, 32>(a, p, stream);
  else tile_launch<LAYOUT, float, 64>(a, p, stream);
}

template <int LAYOUT, int DTYPE>
static void dispatch16(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  using T = std::conditional_t<DTYPE == 0, __bf16, _Float16>;
  if (p.kind == GroupedPlan::kTile) {
    tile_launch<LAYOUT, T, 64>(a, p, stream);
  } else if constexpr (LAYOUT == 2) {
    if (p.bm == 128) pipe_launch<LAYOUT, DTYPE, 128, 256, 3, 4, 1>(a, p, stream);
    else pipe_launch<LAYOUT, DTYPE, 256, 256, 4, 8, 2>(a, p, stream);
  } else if (p.kind == GroupedPlan::kStrip) {
    strip_launch<LAYOUT, DTYPE>(a, p, stream);
  } else {
    if (p.bm == 64) pipe_launch<LAYOUT, DTYPE, 64, 128, 6, 4, 1>(a, p, stream);
    else if (p.bm == 128) pipe_launch<LAYOUT, DTYPE, 128, 256, 5, 8, 2>(a, p, stream);
    else pipe_launch<LAYOUT, DTYPE, 256, 256, 4, 8, 2>(a, p, stream);
  }
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  const GroupedPlan p = plan_grouped(a);
  switch (a.layout * 3 + a.dtype) {
    case 0: dispatch16<0, 0>(a, p, stream); break;
    case 1: dispatch16<0, 1>(a, p, stream); break;
    case 2: dispatch32<0>(a, p, stream); break;
    case 3: dispatch16<1, 0>(a, p, stream); break;
    case 4: dispatch16<1, 1>(a, p, stream); break;
    case 5: dispatch32<1>(a, p, stream); break;
    case 6: dispatch16<2, 0>(a, p, stream); break;
    case 7: dispatch16<2, 1>(a, p, stream); break;
    case 8: dispatch32<2>(a, p, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace qg
