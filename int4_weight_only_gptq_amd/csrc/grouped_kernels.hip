// Dense products grouped by expert (rows sorted by group, see groups.hpp):
//
//   NT: C[r] = A[r] . B_e^T    NN: C[r] = A[r] . B_e    for the rows r of group e
//   TN: C_e = A[rows of e]^T . B[rows of e]
//
// bf16 / fp16 with fp32 accumulation, or fp32 throughout.  Three kernels:
//  * many rows a group: the pipelined MFMA tile of the dense products
//    (dense_pipe.hpp), each workgroup looking up its group first;
//  * few rows a group (decoding): the weights of the reached groups are read once
//    and that read is the time, so a workgroup takes a strip of columns over the
//    whole of k, split over its waves;
//  * any alignment and size, and fp32: a tile staged through registers.
#include "common.hpp"
#include "dense_pipe.hpp"
#include "groups.hpp"
#include "launch.hpp"

namespace qg {

// Row tiles per band of a group's tile order (find_group_tile): 8 x 4 tiles are
// in flight on an XCD's 32 CUs.
constexpr int kBand = 8;

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
// many rows a group: the pipelined tile
// ---------------------------------------------------------------------------
template <int LAYOUT, int DTYPE, int BM, int BN, int STAGES, int NWV, int WGM>
__global__ __launch_bounds__(64 * NWV) void grouped_pipe_kernel(GroupedArgs a, int tiles_m, int tiles_n, int vec) {
  if constexpr (LAYOUT == 2) {
    // every group has the same tiles_m x tiles_n tiles over its own number of
    // rows; an XCD takes one eighth of every group's tiles, since groups differ
    // in length
    const int tiles = tiles_m * tiles_n, per = (tiles + 7) >> 3;
    const int i = blockIdx.x >> 3, e = i / per, t = (blockIdx.x & 7) * per + (i - e * per);
    if (t >= tiles) return;
    int lo;
    const int rows = group_rows(a.offsets, e, (int)a.rows, &lo);
    const int b = t / (kBand * tiles_n), in = t - b * kBand * tiles_n, height = min(kBand, tiles_m - b * kBand);
    const int tn = in / height, tm = b * kBand + (in - tn * height);
    dense_pipe_tile<LAYOUT, DTYPE, BM, BN, STAGES, NWV, WGM, false, true>(
        a.A + (int64_t)lo * a.lda, a.lda, a.B + (int64_t)lo * a.ldb, a.ldb, a.C + e * a.sc, a.ldc, (int)a.M, (int)a.N,
        rows, t, tm, tn, 0, vec, 1, 0, nullptr, nullptr, 0);
  } else {
    const GroupTile g =
        find_group_tile(a.offsets, (int)a.groups, (int)a.rows, BM, tiles_n, kBand, blockIdx.x, threadIdx.x & 63);
    if (g.group < 0) return;
    dense_pipe_tile<LAYOUT, DTYPE, BM, BN, STAGES, NWV, WGM, false, true>(
        a.A + (int64_t)g.row0 * a.lda, a.lda, a.B + (int64_t)g.group * a.sb, a.ldb, a.C + (int64_t)g.row0 * a.ldc,
        a.ldc, g.rows, (int)a.N, (int)a.K, 0, g.tm, g.tn, 0, vec, 1, 0, nullptr, nullptr, 0);
  }
}

// ---------------------------------------------------------------------------
// few rows a group: strips of columns over the whole of k
//
// A workgroup owns 16 RT rows of a group and a strip of columns; its waves take
// blocks of k in turn, all loads of a block issued before its MFMAs, operands
// straight from memory into the MFMA lane layout (lane l: row or column l % 16, k
// chunk l / 16), and the waves' partial tiles are summed through LDS in wave
// order.  The activations are read from L2 (rows past the group's end repeat
// its last row: the same cache lines).
// ---------------------------------------------------------------------------
// NT, B K-contiguous: strip of 16 columns, blocks of 256 k, so a column's 512
// contiguous bytes are read by one wave.
// NN, B N-contiguous: strip of 128 columns; lane (c, q) loads columns 8c .. 8c + 7
// of the 8 k-rows 8q .. 8q + 7 and transposes the 8 x 8 block in registers:
// fragment j then holds column 8c + j (256 contiguous bytes per k-row).
constexpr int kStripK = 256;      // k per block, NT
constexpr int kStripKN = 32;      // k per block, NN

template <int LAYOUT, int DTYPE, int RT>
__global__ __launch_bounds__(512) void grouped_strip_kernel(GroupedArgs a, int strips) {
  constexpr int CT = LAYOUT == 0 ? 1 : 8;               // 16-column MFMA tiles of the strip
  constexpr int COLS = 16 * CT, ROWS = 16 * RT;
  extern __shared__ __attribute__((aligned(16))) float ssm[];   // [waves][ROWS][COLS + 4]
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const GroupTile g = find_group_tile(a.offsets, (int)a.groups, (int)a.rows, ROWS, strips, 1, blockIdx.x, lane);
  if (g.group < 0) return;
  const int cl = lane & 15, ks = lane >> 4;
  const int K = (int)a.K, N = (int)a.N;
  const int r0 = g.tm * ROWS, n0 = g.tn * COLS;
  const uint16_t* arow[RT];
#pragma unroll
  for (int f = 0; f < RT; ++f)
    arow[f] = a.A + (int64_t)(g.row0 + min(r0 + 16 * f + cl, g.rows - 1)) * a.lda;
  const uint16_t* B = a.B + (int64_t)g.group * a.sb;

  f32x4 acc[RT][CT];
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0u, 0u, 0u, 0u};

  if constexpr (LAYOUT == 0) {
    const uint16_t* brow = B + (int64_t)min(n0 + cl, N - 1) * a.ldb;
    for (int k0 = kStripK * wave; k0 < K; k0 += kStripK * waves) {
      u32x4 b[8], x[RT][8];
      // past the end of k both operands are zeros (loads from the row's start)
      if (k0 + kStripK <= K) {
#pragma unroll
        for (int s = 0; s < 8; ++s) b[s] = *reinterpret_cast<const u32x4*>(brow + k0 + 32 * s + 8 * ks);
#pragma unroll
        for (int f = 0; f < RT; ++f)
#pragma unroll
          for (int s = 0; s < 8; ++s) x[f][s] = *reinterpret_cast<const u32x4*>(arow[f] + k0 + 32 * s + 8 * ks);
      } else {
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          const int k = k0 + 32 * s + 8 * ks;
          b[s] = *reinterpret_cast<const u32x4*>(brow + (k < K ? k : 0));
          if (k >= K) b[s] = zero;
#pragma unroll
          for (int f = 0; f < RT; ++f) {
            x[f][s] = *reinterpret_cast<const u32x4*>(arow[f] + (k < K ? k : 0));
            if (k >= K) x[f][s] = zero;
          }
        }
      }
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int f = 0; f < RT; ++f) acc[f][0] = mfma16<DTYPE>(x[f][s], b[s], acc[f][0]);
    }
  } else {
    const int col = min(n0 + 8 * cl, N - 8);
    for (int k0 = kStripKN * wave; k0 < K; k0 += kStripKN * waves) {
      u32x4 in[8], b[8], x[RT];
      const int k = k0 + 8 * ks;
      if (k0 + kStripKN <= K) {
#pragma unroll
        for (int i = 0; i < 8; ++i) in[i] = *reinterpret_cast<const u32x4*>(B + (int64_t)(k + i) * a.ldb + col);
#pragma unroll
        for (int f = 0; f < RT; ++f) x[f] = *reinterpret_cast<const u32x4*>(arow[f] + k);
      } else {   // K % 8 == 0: a lane's 8 k-rows are all inside or all outside
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          in[i] = *reinterpret_cast<const u32x4*>(B + (int64_t)(k < K ? k + i : 0) * a.ldb + col);
          if (k >= K) in[i] = zero;
        }
#pragma unroll
        for (int f = 0; f < RT; ++f) {
          x[f] = *reinterpret_cast<const u32x4*>(arow[f] + (k < K ? k : 0));
          if (k >= K) x[f] = zero;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int p = 0; p < 4; ++p) b[j][p] = __builtin_amdgcn_perm(in[2 * p + 1][j >> 1], in[2 * p][j >> 1], sel);
      }
#pragma unroll
      for (int f = 0; f < RT; ++f)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[f][j] = mfma16<DTYPE>(x[f], b[j], acc[f][j]);
    }
  }

  // lane (cl, ks) holds rows 4 ks + v and column cl (NT) or 8 cl + c (NN)
  constexpr int P = COLS + 4;
  float* mine = ssm + wave * ROWS * P;
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) mine[(16 * f + 4 * ks + v) * P + (LAYOUT == 0 ? cl : 8 * cl + c)] = acc[f][c][v];
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
// any alignment, fp32: a 64 x 64 tile staged through registers
//
// 4 waves (2 x 2, 32 x 32 each), k tiles of 32 in two LDS buffers, elements
// loaded one by one along the operand's contiguous direction (guarded: zeros
// past M, N and k, so nothing outside the matrices is read).  Both operands are
// K-contiguous in LDS.
// ---------------------------------------------------------------------------
template <int LAYOUT, typename T>
__global__ __launch_bounds__(256) void grouped_tile_kernel(GroupedArgs a, int tiles_m, int tiles_n) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr bool BF = std::is_same<T, __bf16>::value;
  constexpr int BT = 64, BK = 32, P = F32 ? BK + 4 : BK + 8;     // LDS row pitch (16-byte rows)
  constexpr int PER = BT * BK / 256;                             // elements per thread and operand
  __shared__ __attribute__((aligned(16))) T sm[2][2][BT * P];
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
    const GroupTile g = find_group_tile(a.offsets, (int)a.groups, (int)a.rows, BT, tiles_n, kBand, blockIdx.x, lane);
    if (g.group < 0) return;
    A += (int64_t)g.row0 * a.lda;
    B += (int64_t)g.group * a.sb;
    C += (int64_t)g.row0 * a.ldc;
    M = g.rows;
    K = a.K;
    tm = g.tm;
    tn = g.tn;
  }
  const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT, N = a.N;
  constexpr bool A_MN = LAYOUT == 2, B_MN = LAYOUT != 0;

  // element i of a thread: K-contiguous: row tid / 32 + 8 i, k tid % 32;
  // else: row tid % 64, k tid / 64 + 4 i
  auto load = [&](const T* p, int64_t ld, bool mn, int64_t first, int64_t end, int64_t k0, T (&reg)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t r = first + (mn ? tid & 63 : (tid >> 5) + 8 * i), k = k0 + (mn ? (tid >> 6) + 4 * i : tid & 31);
      reg[i] = r < end && k < K ? (mn ? p[k * ld + r] : p[r * ld + k]) : (T)0.f;
    }
  };
  auto store = [&](T* region, bool mn, const T (&reg)[PER]) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      region[mn ? (tid & 63) * P + (tid >> 6) + 4 * i : ((tid >> 5) + 8 * i) * P + (tid & 31)] = reg[i];
  };
  f32x4 acc[2][2];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int c = 0; c < 2; ++c) acc[f][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm = (wave & 1) * 32, wn = (wave >> 1) * 32;
  T ra[PER], rb[PER];
  const int64_t ktiles = (K + BK - 1) / BK;
  if (ktiles > 0) {
    load(A, a.lda, A_MN, m0, M, 0, ra);
    load(B, a.ldb, B_MN, n0, N, 0, rb);
    store(sm[0][0], A_MN, ra);
    store(sm[0][1], B_MN, rb);
  }
  __syncthreads();
  for (int64_t kt = 0; kt < ktiles; ++kt) {
    const int buf = (int)(kt & 1);
    const bool more = kt + 1 < ktiles;
    if (more) {
      load(A, a.lda, A_MN, m0, M, (kt + 1) * BK, ra);
      load(B, a.ldb, B_MN, n0, N, (kt + 1) * BK, rb);
    }
    const T *la = sm[buf][0], *lb = sm[buf][1];
    if constexpr (F32) {
      // k order within 16: lane group ks takes 4 ks .. 4 ks + 3 of both operands
#pragma unroll
      for (int q = 0; q < BK / 16; ++q) {
        f32x4 x[2], w[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) x[f] = *reinterpret_cast<const f32x4*>(la + (wm + 16 * f + cl) * P + 16 * q + 4 * ks);
#pragma unroll
        for (int c = 0; c < 2; ++c) w[c] = *reinterpret_cast<const f32x4*>(lb + (wn + 16 * c + cl) * P + 16 * q + 4 * ks);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int c = 0; c < 2; ++c) acc[f][c] = mfma16_f32(x[f][j], w[c][j], acc[f][c]);
      }
    } else {
      u32x4 x[2], w[2];
#pragma unroll
      for (int f = 0; f < 2; ++f) x[f] = *reinterpret_cast<const u32x4*>(la + (wm + 16 * f + cl) * P + 8 * ks);
#pragma unroll
      for (int c = 0; c < 2; ++c) w[c] = *reinterpret_cast<const u32x4*>(lb + (wn + 16 * c + cl) * P + 8 * ks);
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[f][c] = mfma16<BF ? 0 : 1>(x[f], w[c], acc[f][c]);
    }
    if (more) {
      store(sm[buf ^ 1][0], A_MN, ra);
      store(sm[buf ^ 1][1], B_MN, rb);
    }
    __syncthreads();
  }
#pragma unroll
  for (int f = 0; f < 2; ++f)
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
  if (a.layout == 2) return a.M % 8 == 0 && a.N % 8 == 0;
  return a.sb % 8 == 0 && a.K % 8 == 0 && (a.layout == 0 || a.N % 8 == 0);
}

// The kernel a product takes: kind, rows and columns of a tile, threads.
struct GroupedPlan {
  enum Kind { kTile, kStrip, kPipe } kind;
  int bm, bn, threads;
  int64_t blocks;
};

static GroupedPlan plan_grouped(const GroupedArgs& a) {
  GroupedPlan p{GroupedPlan::kTile, 64, 64, 256, 0};
  const int64_t avg = a.rows / a.groups;
  if (a.dtype != 2 && a.K > 0 && vectorizable(a)) {
    if (a.layout == 2) {
      p = {GroupedPlan::kPipe, 256, 128, 512, 0};
    } else if (avg <= 24) {
      const int64_t k_block = a.layout == 0 ? kStripK : kStripKN, waves = (a.K + k_block - 1) / k_block;
      p = {GroupedPlan::kStrip, avg <= 8 ? 16 : 32, a.layout == 0 ? 16 : 128, (int)(64 * (waves < 8 ? waves : 8)), 0};
    } else if (avg <= 64) {
      p = {GroupedPlan::kPipe, 64, 128, 256, 0};
    } else {
      p = {GroupedPlan::kPipe, avg <= 128 ? 128 : 256, 128, 512, 0};
    }
  }
  const int64_t tiles_n = (a.N + p.bn - 1) / p.bn;
  if (a.layout != 2) {
    p.blocks = group_tile_blocks(a.rows, a.groups, p.bm, tiles_n);
  } else {
    const int64_t tiles = (a.M + p.bm - 1) / p.bm * tiles_n;
    p.blocks = a.groups * (p.kind == GroupedPlan::kPipe ? (tiles + 7) / 8 * 8 : tiles);
  }
  return p;
}

int64_t grouped_threads(const GroupedArgs& a) {
  const GroupedPlan p = plan_grouped(a);
  return p.blocks * p.threads;
}

template <int LAYOUT, int DTYPE, int BM, int BN, int STAGES, int NWV, int WGM>
static void pipe_launch(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  const int tiles_n = (int)((a.N + BN - 1) / BN), tiles_m = LAYOUT == 2 ? (int)((a.M + BM - 1) / BM) : 0;
  const int vec = aligned16(a.C) && a.ldc % 8 == 0 && (LAYOUT != 2 || a.sc % 8 == 0);
  const size_t main_bytes = (size_t)STAGES * (BM + BN) * 8 * 16, out_bytes = (size_t)BM * (BN + 8) * 2;
  grouped_pipe_kernel<LAYOUT, DTYPE, BM, BN, STAGES, NWV, WGM>
      <<<dim3((unsigned)p.blocks), dim3(64 * NWV), main_bytes > out_bytes ? main_bytes : out_bytes, stream>>>(
          a, tiles_m, tiles_n, vec);
}

template <int LAYOUT, int DTYPE, int RT>
static void strip_launch(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  const size_t lds = (size_t)(p.threads / 64) * 16 * RT * (p.bn + 4) * 4;
  grouped_strip_kernel<LAYOUT, DTYPE, RT><<<dim3((unsigned)p.blocks), dim3((unsigned)p.threads), lds, stream>>>(
      a, (int)((a.N + p.bn - 1) / p.bn));
}

template <int LAYOUT, typename T>
static void tile_launch(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  grouped_tile_kernel<LAYOUT, T><<<dim3((unsigned)p.blocks), dim3(256), 0, stream>>>(
      a, LAYOUT == 2 ? (int)((a.M + 63) / 64) : 0, (int)((a.N + 63) / 64));
}

template <int LAYOUT, int DTYPE>
static void dispatch16(const GroupedArgs& a, const GroupedPlan& p, hipStream_t stream) {
  using T = std::conditional_t<DTYPE == 0, __bf16, _Float16>;
  if (p.kind == GroupedPlan::kTile) {
    tile_launch<LAYOUT, T>(a, p, stream);
  } else if constexpr (LAYOUT == 2) {
    pipe_launch<LAYOUT, DTYPE, 256, 128, 3, 8, 4>(a, p, stream);
  } else if (p.kind == GroupedPlan::kStrip) {
    if (p.bm == 16) strip_launch<LAYOUT, DTYPE, 1>(a, p, stream);
    else strip_launch<LAYOUT, DTYPE, 2>(a, p, stream);
  } else {
    if (p.bm == 64) pipe_launch<LAYOUT, DTYPE, 64, 128, 4, 4, 2>(a, p, stream);
    else if (p.bm == 128) pipe_launch<LAYOUT, DTYPE, 128, 128, 4, 8, 2>(a, p, stream);
    else pipe_launch<LAYOUT, DTYPE, 256, 128, 3, 8, LAYOUT == 1 ? 2 : 4>(a, p, stream);
  }
}

hipError_t launch_grouped(const GroupedArgs& a, hipStream_t stream) {
  const GroupedPlan p = plan_grouped(a);
  switch (a.layout * 3 + a.dtype) {
    case 0: dispatch16<0, 0>(a, p, stream); break;
    case 1: dispatch16<0, 1>(a, p, stream); break;
    case 2: tile_launch<0, float>(a, p, stream); break;
    case 3: dispatch16<1, 0>(a, p, stream); break;
    case 4: dispatch16<1, 1>(a, p, stream); break;
    case 5: tile_launch<1, float>(a, p, stream); break;
    case 6: dispatch16<2, 0>(a, p, stream); break;
    case 7: dispatch16<2, 1>(a, p, stream); break;
    case 8: tile_launch<2, float>(a, p, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace qg
