// Microscaled 4-bit floating point (MXFP4, include/qgemm_mxfp4.h) for gfx950:
// quantisation, reading back, and the product of two MXFP4 matrices.
//
// The product runs on the scaled matrix instructions (f8f6f4 with both operands
// e2m1): a lane's operand is 32 consecutive elements of a row, 16 bytes, which is
// exactly one block, and the block's scale byte rides in a register beside it, so
// nothing is decoded.  The products are exact and the sums fp32.
#include "common.hpp"
#include "launch.hpp"
#include <type_traits>

namespace qg {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOneScales = 0x7F7F7F7Fu;   // four scale bytes of 1

template <int DTYPE>
using out_t = std::conditional_t<DTYPE == 0, __bf16, std::conditional_t<DTYPE == 1, _Float16, float>>;

// ---------------------------------------------------------------------------
// quantisation: eight elements a thread, the four threads of a block adjacent lanes
//
// Bound by memory: 16 bytes in and 4.25 out a thread (16-bit elements).  The block's
// exponent comes from the largest magnitude's bits, without a logarithm: as fp32
// its biased exponent field E is floor(log2 a) + 127 (a subnormal has E = 0, and its
// scale is held to 2^-127 anyway), so the scale byte is max(E - 2, 0).  The conversion
// instruction divides by the scale and rounds to nearest even, past 6 to 6.
// ---------------------------------------------------------------------------
template <int DTYPE>
__device__ __forceinline__ void load8(const void* x, int64_t i, bool vec, float (&v)[8]) {
  using T = out_t<DTYPE>;
  const T* p = static_cast<const T*>(x) + i;
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (float)p[j];
  } else if constexpr (DTYPE == 2) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint16_t h = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      v[j] = (float)__builtin_bit_cast(T, h);
    }
  }
}

__device__ __forceinline__ uint32_t max_of_quad(uint32_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));   // lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));   // lanes 2 3 0 1
#endif
  return v;
}

// 2^(byte - 127) as a float (byte 0: the subnormal 2^-127)
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __builtin_bit_cast(float, byte ? byte << 23 : 0x00400000u);
}

template <int DTYPE>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const void* __restrict__ x, int64_t ldx, int64_t rows,
                                                             int64_t k, uint8_t* __restrict__ codes, int64_t ldc,
                                                             uint8_t* __restrict__ scales, int64_t lds, int vec) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = k >> 3, row = t / per, c = t - row * per;
  if (row >= rows) return;                        // whole blocks leave together (k % 32 == 0)
  float v[8];
  load8<DTYPE>(x, row * ldx + 8 * c, vec, v);
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
  top = max_of_quad(top) >> 23;
  const bool finite = top < 255;
  const uint32_t byte = finite ? (top > 2 ? top - 2 : 0) : 255u;
  uint32_t out = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  if (finite) {
    const float s = scale_value(byte);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0], v[1], s, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2], v[3], s, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4], v[5], s, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6], v[7], s, 3);
  }
#endif
  *reinterpret_cast<uint32_t*>(codes + row * ldc + 4 * c) = out;
  if ((c & 3) == 0) scales[row * lds + (c >> 2)] = (uint8_t)byte;
}

// ---------------------------------------------------------------------------
// reading back: eight codes a thread
// ---------------------------------------------------------------------------
template <int DTYPE>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                               const uint8_t* __restrict__ scales, int64_t lds,
                                                               int64_t rows, int64_t k, void* __restrict__ y,
                                                               int64_t ldy, int vec) {
  using T = out_t<DTYPE>;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t per = k >> 3, row = t / per, c = t - row * per;
  if (row >= rows) return;
  [[maybe_unused]] const uint32_t w = *reinterpret_cast<const uint32_t*>(codes + row * ldc + 4 * c);
  const uint32_t byte = scales[row * lds + (c >> 2)];
  const float s = byte == 255 ? __builtin_nanf("") : scale_value(byte);
  float v[8];
#if defined(__HIP_DEVICE_COMPILE__)
  const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
  v[0] = p0[0]; v[1] = p0[1]; v[2] = p1[0]; v[3] = p1[1];
  v[4] = p2[0]; v[5] = p2[1]; v[6] = p3[0]; v[7] = p3[1];
#endif
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= s;
  T* p = static_cast<T*>(y) + row * ldy + 8 * c;
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = (T)v[j];
  } else if constexpr (DTYPE == 2) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = DTYPE == 0 ? pack_bf16x2(v[2 * j], v[2 * j + 1]) : pack_f16x2(v[2 * j], v[2 * j + 1]);
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(p));    // (4096 x 14336 and its quantisation 48.5 -> 45.8 us)
  }
}

// ---------------------------------------------------------------------------
// product, few rows: strips of 16 columns over the whole of k
//
// A workgroup owns 16 RT rows of A and 16 rows of B (columns of C); its waves take
// chunks of 512 k in turn.  Lane (r, q) holds blocks 4 q .. 4 q + 3 of row r's 16
// blocks of a chunk: 64 contiguous bytes of codes and one dword of scales, one block
// a 16x16x128 step (which blocks meet in a step does not matter, so long as both
// operands agree).  A strip's read of B is the time; A comes from L2, only by the lanes
// whose rows there are.
// ---------------------------------------------------------------------------
__device__ __forceinline__ i32x8 fp4_operand(u32x4 v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// The bytes of a scale matrix, first to one past the last row's last.
struct Bytes {
  const uint8_t *first, *end;
};

// Scales of one in place of those past the end of k (blocks kb ..).
template <int D>
__device__ __forceinline__ void ones_past_end(int kb, int blocks, uint32_t (&s)[D]) {
  if (kb + 4 * D <= blocks) return;
#pragma unroll
  for (int i = 0; i < D; ++i) {
    const int n = blocks - kb - 4 * i;             // valid bytes of dword i
    const uint32_t keep = n >= 4 ? 0xFFFFFFFFu : n <= 0 ? 0u : 0xFFFFFFFFu >> (32 - 8 * n);
    s[i] = (s[i] & keep) | (kOneScales & ~keep);
  }
}

// 4 D scale bytes from block kb on of a row of `blocks` blocks, ones past its end.  Rows
// may start on any byte: the D + 1 aligned dwords around them are loaded and shifted
// where those lie inside the matrix (K = 5152, rows of 161 bytes, 512 x 5120: 41.0 us byte by
// byte, 22.6 us so).
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* row, int kb, int blocks, Bytes all, uint32_t (&s)[D]) {
  const uint8_t* p = row + kb;
  const uint32_t shift = (uint32_t)(uintptr_t)p & 3u;
  const uint8_t* a = p - shift;
  if (a >= all.first && a + 4 * D + 4 <= all.end) {
    uint32_t w[D + 1];
#pragma unroll
    for (int i = 0; i <= D; ++i) w[i] = reinterpret_cast<const uint32_t*>(a)[i];
#pragma unroll
    for (int i = 0; i < D; ++i) s[i] = __builtin_amdgcn_alignbyte(w[i + 1], w[i], shift);
  } else {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      s[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (kb + 4 * i + j < blocks) s[i] |= (uint32_t)p[4 * i + j] << (8 * j);
    }
  }
  ones_past_end<D>(kb, blocks, s);
}

// One dword of them; dwords: the rows start on 4 bytes.
__device__ __forceinline__ uint32_t load_scales4(const uint8_t* row, int kb, int blocks, bool dwords, Bytes all) {
  if (dwords && kb + 4 <= blocks) return *reinterpret_cast<const uint32_t*>(row + kb);
  uint32_t s[1];
  load_scales<1>(row, kb, blocks, all, s);
  return s[0];
}

template <int RT, int DTYPE>
__global__ __launch_bounds__(512) void mxfp4_strip_kernel(MxGemmArgs g, int strips, int a_dwords, int b_dwords) {
  constexpr int ROWS = 16 * RT, P = 20;
  extern __shared__ __attribute__((aligned(16))) float xsm[];   // [waves][ROWS][P]
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tm = blockIdx.x / strips, tn = blockIdx.x - tm * strips;
  const int r = lane & 15, q = lane >> 4;
  const int64_t r0 = (int64_t)tm * ROWS, n0 = (int64_t)tn * 16;
  const int blocks = (int)(g.K >> 5);
  const Bytes a_all = {g.as, g.as + (g.M - 1) * g.ldas + blocks}, b_all = {g.bs, g.bs + (g.N - 1) * g.ldbs + blocks};
  const int64_t bn = min(n0 + r, g.N - 1);
  const uint8_t *bp = g.b + bn * g.ldb, *bs = g.bs + bn * g.ldbs;
  const uint8_t *ap[RT], *as[RT];
#pragma unroll
  for (int f = 0; f < RT; ++f) {
    const int64_t am = min(r0 + 16 * f + r, g.M - 1);
    ap[f] = g.a + am * g.lda;
    as[f] = g.as + am * g.ldas;
  }
  f32x4 acc[RT];
#pragma unroll
  for (int f = 0; f < RT; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int c = wave; 16 * c < blocks; c += waves) {
    const int kb = 16 * c + 4 * q;
    u32x4 b[4], a[RT][4];
    uint32_t sb, sa[RT];
    if (16 * c + 16 <= blocks) {
#pragma unroll
      for (int s = 0; s < 4; ++s) b[s] = *reinterpret_cast<const u32x4*>(bp + 16 * (kb + s));
      sb = load_scales4(bs, kb, blocks, b_dwords, b_all);
#pragma unroll
      for (int f = 0; f < RT; ++f) {
#pragma unroll
        for (int s = 0; s < 4; ++s) a[f][s] = u32x4{0u, 0u, 0u, 0u};
        sa[f] = kOneScales;
        if (r0 + 16 * f + r < g.M) {
#pragma unroll
          for (int s = 0; s < 4; ++s) a[f][s] = *reinterpret_cast<const u32x4*>(ap[f] + 16 * (kb + s));
          sa[f] = load_scales4(as[f], kb, blocks, a_dwords, a_all);
        }
      }
    } else {   // past the end of k: codes of zero, scales of one
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool in = kb + s < blocks;
        b[s] = *reinterpret_cast<const u32x4*>(bp + (in ? 16 * (kb + s) : 0));
        if (!in) b[s] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int f = 0; f < RT; ++f) {
          a[f][s] = *reinterpret_cast<const u32x4*>(ap[f] + (in ? 16 * (kb + s) : 0));
          if (!in) a[f][s] = u32x4{0u, 0u, 0u, 0u};
        }
      }
      sb = load_scales4(bs, kb, blocks, b_dwords, b_all);
#pragma unroll
      for (int f = 0; f < RT; ++f) sa[f] = load_scales4(as[f], kb, blocks, a_dwords, a_all);
    }
#pragma unroll
    for (int f = 0; f < RT; ++f) {
      acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[f][0]), fp4_operand(b[0]), acc[f], 4, 4, 0,
                                                                sa[f], 0, sb);
      acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[f][1]), fp4_operand(b[1]), acc[f], 4, 4, 1,
                                                                sa[f], 1, sb);
      acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[f][2]), fp4_operand(b[2]), acc[f], 4, 4, 2,
                                                                sa[f], 2, sb);
      acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[f][3]), fp4_operand(b[3]), acc[f], 4, 4, 3,
                                                                sa[f], 3, sb);
    }
  }
  float* mine = xsm + wave * ROWS * P;
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int v = 0; v < 4; ++v) mine[(16 * f + 4 * q + v) * P + r] = acc[f][v];
  __syncthreads();
  using T = out_t<DTYPE>;
  T* C = static_cast<T*>(g.c);
  for (int i = tid; i < ROWS * 16; i += blockDim.x) {
    const int64_t gr = r0 + (i >> 4), gc = n0 + (i & 15);
    if (gr >= g.M || gc >= g.N) continue;
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += xsm[(w * ROWS + (i >> 4)) * P + (i & 15)];
    C[gr * g.ldc + gc] = (T)s;
  }
}

// ---------------------------------------------------------------------------
// product, many rows: BM x BN tiles
//
// NWV waves as a WGM x (NWV / WGM) grid, FM x FN matrix tiles of 32 x 32 each.  k
// tiles of KB blocks (32 KB elements, 16 KB bytes a row) in a ring of STAGES LDS
// buffers filled by direct loads, 16-byte chunk c of row r in slot KB r + (c ^ x(r))
// with x(r) such that the 16 rows LDS serves together fall on different banks (with r mod 8
// for KB = 8 every two met: 2048 x 8192 at k = 8192 70.6 us, 67.2 with r / 2 mod 8).  Lane
// (r, h) of 32x32x64 step s takes block h KB / 2 + s of row r, so that its scales of a
// k tile are adjacent bytes.  Scales are staged 16 blocks (512 k) at a time, 16 bytes a
// row, through registers into two LDS buffers of four planes (dword j of every row side
// by side, so that their reads share no bank): the next ones are loaded in the first of
// those k tiles and written before the last one's barrier.
//
// One barrier a k tile, before its last step: by then every operand of the tile is
// in registers and the next tile has landed, so its buffer is refilled at once.
// Operands are read one step ahead of the matrix instructions that use them.
// ---------------------------------------------------------------------------
constexpr int kMxBand = 8;   // row tiles per band of the tile order

template <int BM, int BN, int KB, int STAGES>
struct MxTile {
  static constexpr int kStage = (BM + BN) * KB;                 // 16-byte chunks
  static constexpr int kScales = BM + BN;                       // 16-byte chunks per buffer
  static constexpr size_t bytes(int esize) {
    const size_t main_bytes = (size_t)(STAGES * kStage + 2 * kScales) * 16, out = (size_t)BM * (BN + 8) * 2;
    return esize == 2 && out > main_bytes ? out : main_bytes;
  }
};

template <int BM, int BN, int KB, int STAGES, int NWV, int WGM, int DTYPE, bool ALIGN16>
__global__ __launch_bounds__(64 * NWV) void mxfp4_tile_kernel(MxGemmArgs g, int tiles_m, int tiles_n, int per_xcd,
                                                              int vec) {
  constexpr int T = 64 * NWV, WM = BM / WGM, WN = BN / (NWV / WGM), FM = WM / 32, FN = WN / 32;
  constexpr int STEPS = KB / 2, PER = 16 / KB;                   // steps of a k tile; k tiles of a scale buffer
  using S = MxTile<BM, BN, KB, STAGES>;
  constexpr int LOADS = S::kStage / T, A_LOADS = BM * KB / T;
  static_assert((KB == 4 || KB == 8) && BM * KB % T == 0 && BN * KB % T == 0 && LOADS * (STAGES - 1) <= 63, "loads");
  extern __shared__ __attribute__((aligned(16))) u32x4 msm[];
  uint32_t* ssm = reinterpret_cast<uint32_t*>(msm + STAGES * S::kStage);   // scales [2][4][BM + BN]

  // tile order: each XCD a contiguous run; bands of kMxBand row tiles, column by column
  const int item = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per_xcd || item >= tiles_m * tiles_n) return;
  const int band = item / (kMxBand * tiles_n), in_band = item - band * kMxBand * tiles_n;
  const int height = min(kMxBand, tiles_m - band * kMxBand);
  const int tn = in_band / height, tm = band * kMxBand + (in_band - tn * height);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wm0 = (wave % WGM) * WM, wn0 = (wave / WGM) * WN;
  const int blocks = (int)(g.K >> 5), ktiles = (blocks + KB - 1) / KB;

  // chunk tid + T j of a stage: row (tid + T j) / KB of the tile's A rows then B rows
  // (rows past M or N repeat the last one), its k chunk the same for every j
  auto swizzle = [](int row, int c) { return KB == 8 ? c ^ ((row >> 1) & 7) : c ^ ((row >> 2) & 3); };
  static_assert(T / KB % 16 == 0, "one k chunk per thread");
  const int chunk = swizzle(tid / KB, tid % KB);
  const uint8_t *abase = g.a + m0 * g.lda, *bbase = g.b + n0 * g.ldb;
  uint32_t off[LOADS];      // (leading dimensions are at most 2^22 bytes)
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int row = (tid + T * j) / KB;
    off[j] = (j < A_LOADS ? (uint32_t)min((int64_t)row, g.M - 1 - m0) * (uint32_t)g.lda
                          : (uint32_t)min((int64_t)row - BM, g.N - 1 - n0) * (uint32_t)g.ldb) + 16 * chunk;
  }
  auto issue = [&](int kt) {
    u32x4* base = msm + (kt % STAGES) * S::kStage + 64 * wave;
    const bool in = KB * kt + chunk < blocks;    // else zeros: codes of 0
#pragma unroll
    for (int j = 0; j < LOADS; ++j)
      buffer_to_lds16_or_zero((j < A_LOADS ? abase : bbase) + (int64_t)kt * 16 * KB, in ? off[j] : kOutside,
                              base + T * j);
  };
  // Row tid of scales, A's then B's (a wave holds rows of one of them), 16 blocks at a time.
  // ALIGN16: every row starts on 16 bytes; a variant of its own, because the general form takes
  // registers that the largest tile has not (9 spilled, 2048 x 8192 at k = 8192 72 -> 80 us).
  // Its load ends with the dword that holds the matrix's last byte.
  static_assert(BM % 64 == 0 && BM + BN <= T, "rows of scales");
  const bool mine = tid < BM + BN, of_a = 64 * wave < BM;
  const uint8_t* sfirst = of_a ? g.as + m0 * g.ldas : g.bs + n0 * g.ldbs;
  const int64_t sld = of_a ? g.ldas : g.ldbs, srows = of_a ? g.M - m0 : g.N - n0;
  const uint32_t soff = (uint32_t)min((int64_t)(of_a ? tid : tid - BM), srows - 1) * (uint32_t)sld;
  const int64_t sbytes = (srows - 1) * sld + blocks;
  const uint32_t srange = (uint32_t)min((sbytes + 3) & ~(int64_t)3, (int64_t)kOutside - 4);
  u32x4 staged;
  auto stage_scales = [&](int kb) {
    if (!mine) return;
    uint32_t s[4];
    if constexpr (ALIGN16) {
      const u32x4 v = buffer_load16_within(sfirst, srange, soff + kb);
      s[0] = v[0]; s[1] = v[1]; s[2] = v[2]; s[3] = v[3];
      ones_past_end<4>(kb, blocks, s);
    } else {
      load_scales<4>(sfirst + soff, kb, blocks, Bytes{of_a ? g.as : g.bs, sfirst + sbytes}, s);
    }
    staged = u32x4{s[0], s[1], s[2], s[3]};
  };
  auto store_scales = [&](int buf) {
    if (!mine) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) ssm[(4 * buf + j) * S::kScales + tid] = staged[j];
  };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int c = 0; c < FN; ++c)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[f][c][v] = 0.f;

  struct Frags {
    u32x4 a[FM], b[FN];
  };
  auto read = [&](int kt, int s, Frags& x) {
    const u32x4* la = msm + (kt % STAGES) * S::kStage + KB * r + swizzle(r, STEPS * h + s);
#pragma unroll
    for (int f = 0; f < FM; ++f) x.a[f] = la[KB * (wm0 + 32 * f)];
#pragma unroll
    for (int c = 0; c < FN; ++c) x.b[c] = la[KB * (BM + wn0 + 32 * c)];
  };
  struct Scales {
    uint32_t a[FM], b[FN];
  };
  auto read_scales = [&](int kt, Scales& x) {
    // (dword kt % PER of the row, this lane half's two bytes; KB == 8: dword 2 (kt % PER) + h)
    const uint32_t* l = ssm + (kt / PER % 2 * 4 + (KB == 8 ? 2 * (kt % PER) + h : kt % PER)) * S::kScales + r;
    auto one = [&](int row) -> uint32_t {
      if constexpr (KB == 8) return l[row];
      else return reinterpret_cast<const uint16_t*>(l + row)[h];
    };
#pragma unroll
    for (int f = 0; f < FM; ++f) x.a[f] = one(wm0 + 32 * f);
#pragma unroll
    for (int c = 0; c < FN; ++c) x.b[c] = one(BM + wn0 + 32 * c);
  };
  auto multiply = [&](auto s_, const Frags& x, const Scales& sc) {
    constexpr int s = decltype(s_)::value;
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < FN; ++c)
        acc[f][c] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(x.a[f]), fp4_operand(x.b[c]), acc[f][c], 4,
                                                                    4, s, sc.a[f], s, sc.b[c]);
  };

#pragma unroll
  for (int st = 0; st < STAGES; ++st)
    if (st < ktiles) issue(st);
  stage_scales(0);
  store_scales(0);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  Frags x[2];
  Scales sc, next_sc;
  read(0, 0, x[0]);
  read_scales(0, sc);
  // one k tile; refill = kt + STAGES < ktiles, next = kt + 1 < ktiles (compile time)
  auto tile = [&](int kt, auto refill, auto next) {
    if (kt % PER == 0 && kt + PER < ktiles) stage_scales(KB * (kt + PER));
    auto step = [&](auto s_) {
      constexpr int s = decltype(s_)::value;
      read(kt, s + 1, x[(s + 1) & 1]);
      multiply(s_, x[s & 1], sc);
      __builtin_amdgcn_sched_barrier(0);
    };
    step(std::integral_constant<int, 0>{});
    if constexpr (STEPS == 4) {
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
    }
    if constexpr (decltype(next)::value) {
      if (kt % PER == PER - 1) store_scales((kt + 1) / PER % 2);
      // this wave's reads of stage kt, its scales' write and its loads of stage kt + 1
      // are complete (the empty asm keeps the write above the wait)
      asm volatile("" ::: "memory");
      if constexpr (decltype(refill)::value) __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (STAGES - 2)) & ~(0xF << 8));
      else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0) & ~(0xF << 8));
      lds_barrier();
      if constexpr (decltype(refill)::value) issue(kt + STAGES);
      read(kt + 1, 0, x[0]);
      read_scales(kt + 1, next_sc);
      __builtin_amdgcn_sched_barrier(0);
    }
    multiply(std::integral_constant<int, STEPS - 1>{}, x[1], sc);
    if constexpr (decltype(next)::value) sc = next_sc;
    __builtin_amdgcn_sched_barrier(0);
  };
  using T_ = std::true_type;
  using F_ = std::false_type;
  int kt = 0;
  for (; kt + STAGES < ktiles; ++kt) tile(kt, T_{}, T_{});
  for (; kt + 1 < ktiles; ++kt) tile(kt, F_{}, T_{});
  tile(kt, F_{}, F_{});

  // lane (r, h) holds column r and rows 8 (v / 4) + 4 h + v % 4 of each 32 x 32 block
  using O = out_t<DTYPE>;
  O* C = static_cast<O*>(g.c);
  if constexpr (DTYPE == 2) {
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < FN; ++c)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int64_t gr = m0 + wm0 + 32 * f + 8 * (v >> 2) + 4 * h + (v & 3), gc = n0 + wn0 + 32 * c + r;
          if (gr < g.M && gc < g.N) C[gr * g.ldc + gc] = acc[f][c][v];
        }
  } else {
    __syncthreads();
    constexpr int OP = BN + 8;
    uint16_t* osm = reinterpret_cast<uint16_t*>(msm);
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int c = 0; c < FN; ++c)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const O o = (O)acc[f][c][v];
          osm[(wm0 + 32 * f + 8 * (v >> 2) + 4 * h + (v & 3)) * OP + wn0 + 32 * c + r] = __builtin_bit_cast(uint16_t, o);
        }
    __syncthreads();
    uint16_t* out = static_cast<uint16_t*>(g.c);
    constexpr int CPR = BN / 8;
    for (int i = tid; i < BM * CPR; i += T) {
      const int row = i / CPR, cc = i - row * CPR;
      const int64_t gr = m0 + row, gc = n0 + 8 * cc;
      if (gr >= g.M || gc >= g.N) continue;
      const uint16_t* p = &osm[row * OP + 8 * cc];
      if (vec && gc + 8 <= g.N) {
        __builtin_nontemporal_store(*reinterpret_cast<const u32x4*>(p),
                                    reinterpret_cast<u32x4*>(out + gr * g.ldc + gc));
      } else {
        for (int e = 0; e < 8 && gc + e < g.N; ++e) out[gr * g.ldc + gc + e] = p[e];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
// Alignment in bytes (16, 4 or 1) that every row of a matrix starts on.
static int row_align(const void* p, int64_t ld_bytes) {
  const uint64_t v = (uint64_t)(uintptr_t)p | (uint64_t)ld_bytes;
  return v % 16 == 0 ? 16 : v % 4 == 0 ? 4 : 1;
}

template <int DTYPE>
static void quantize(const void* x, int64_t ldx, int64_t rows, int64_t k, uint8_t* codes, int64_t ldc, uint8_t* scales,
                     int64_t lds, hipStream_t stream) {
  const int vec = row_align(x, ldx * (int64_t)sizeof(out_t<DTYPE>)) == 16;
  mxfp4_quantize_kernel<DTYPE><<<dim3((unsigned)((rows * (k / 8) + 255) / 256)), dim3(256), 0, stream>>>(
      x, ldx, rows, k, codes, ldc, scales, lds, vec);
}

hipError_t launch_mxfp4_quantize(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t k, uint8_t* codes,
                                 int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t stream) {
  if (dtype == 0) quantize<0>(x, ldx, rows, k, codes, ldc, scales, lds, stream);
  else if (dtype == 1) quantize<1>(x, ldx, rows, k, codes, ldc, scales, lds, stream);
  else quantize<2>(x, ldx, rows, k, codes, ldc, scales, lds, stream);
  return hipGetLastError();
}

template <int DTYPE>
static void dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t rows, int64_t k,
                       void* y, int64_t ldy, hipStream_t stream) {
  const int vec = row_align(y, ldy * (int64_t)sizeof(out_t<DTYPE>)) == 16;
  mxfp4_dequantize_kernel<DTYPE><<<dim3((unsigned)((rows * (k / 8) + 255) / 256)), dim3(256), 0, stream>>>(
      codes, ldc, scales, lds, rows, k, y, ldy, vec);
}

hipError_t launch_mxfp4_dequantize(int dtype, const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds,
                                   int64_t rows, int64_t k, void* y, int64_t ldy, hipStream_t stream) {
  if (dtype == 0) dequantize<0>(codes, ldc, scales, lds, rows, k, y, ldy, stream);
  else if (dtype == 1) dequantize<1>(codes, ldc, scales, lds, rows, k, y, ldy, stream);
  else dequantize<2>(codes, ldc, scales, lds, rows, k, y, ldy, stream);
  return hipGetLastError();
}

struct MxPlan {
  bool strip;
  int bm, bn, threads;
  int64_t tiles_m, tiles_n;
};

constexpr int kCus = 256;

// Tiles of the many-row kernel, one workgroup a CU: a launch takes ceil(tiles / 256) rounds
// of one tile's time.  Measured per round against 256 x 256 (bf16, k = 5120, 43 us): 128 x 128
// half of it, 64 x 128 0.36.  512 x 5120 17.2 us with 128 x 128 against 23.6 (64) and 36.8 (256),
// 2000 x 1024 12.1 us with 64 x 128 against 18.0 (128), 2048 x 8192 at k = 8192 67 us with
// 256 x 256 against 108 (128).
struct MxTileSize {
  int bm, bn, threads;
  double cost;
};
static const MxTileSize kMxTiles[3] = {{256, 256, 512, 1.0}, {128, 128, 256, 0.5}, {64, 128, 256, 0.36}};

static double tile_cost(const MxTileSize& t, int64_t M, int64_t N) {
  const int64_t tiles = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
  return (double)((tiles + kCus - 1) / kCus) * t.cost;
}

static const MxTileSize& pick_tile(int64_t M, int64_t N) {
  const MxTileSize* best = &kMxTiles[0];
  for (const MxTileSize& t : kMxTiles)
    if (tile_cost(t, M, N) < tile_cost(*best, M, N)) best = &t;
  return *best;
}

// Columns of a first launch of whole rounds of 256 x 256 tiles when the columns that are
// left are cheaper in tiles of their own, a second launch being charged a tenth of a
// round; 0: one launch.  (2000 x 25600, 800 tiles: 24576 columns in three rounds and 1024 in one
// of 64 x 128 tiles, 165 -> 150 us; 1500 x 12000, K 4096, 66 -> 52 us.)
static int64_t first_columns(int64_t M, int64_t N) {
  const double one = tile_cost(pick_tile(M, N), M, N);
  const int64_t tiles_m = (M + 255) / 256, rounds = tiles_m * ((N + 255) / 256) / kCus;
  const int64_t n1 = rounds * kCus / tiles_m * 256;
  if (rounds == 0 || n1 <= 0 || n1 >= N) return 0;
  const double two = tile_cost(kMxTiles[0], M, n1) + tile_cost(pick_tile(M, N - n1), M, N - n1) + 0.1;
  return two < one ? n1 : 0;
}

static MxPlan plan_mxfp4(const MxGemmArgs& g) {
  MxPlan p{};
  if (g.M <= 32 || g.K == 0) {
    p.strip = true;
    p.bm = g.M <= 16 ? 16 : 32;
    p.bn = 16;
    const int64_t chunks = (g.K + 511) / 512;
    p.threads = (int)(64 * (chunks < 1 ? 1 : chunks < 8 ? chunks : 8));
  } else {
    const MxTileSize& t = pick_tile(g.M, g.N);
    p.bm = t.bm;
    p.bn = t.bn;
    p.threads = t.threads;
  }
  p.tiles_m = (g.M + p.bm - 1) / p.bm;
  p.tiles_n = (g.N + p.bn - 1) / p.bn;
  return p;
}

int64_t mxfp4_threads(const MxGemmArgs& g) {
  const MxPlan p = plan_mxfp4(g);
  if (p.tiles_m > ((int64_t)1 << 31) / p.tiles_n) return (int64_t)1 << 40;
  return (p.tiles_m * p.tiles_n + 7) / 8 * 8 * p.threads;
}

template <int BM, int BN, int KB, int STAGES, int NWV, int WGM, int DTYPE>
static void mx_tile_launch(const MxGemmArgs& g, const MxPlan& p, hipStream_t stream) {
  constexpr size_t lds = MxTile<BM, BN, KB, STAGES>::bytes(sizeof(out_t<DTYPE>));
  static_assert(lds <= 160 * 1024, "LDS budget");
  const int per_xcd = (int)((p.tiles_m * p.tiles_n + 7) / 8);
  const int vec = row_align(g.c, g.ldc * 2) == 16;
  const dim3 grid((unsigned)(8 * per_xcd)), block(64 * NWV);
  const int tm = (int)p.tiles_m, tn = (int)p.tiles_n;
  if (row_align(g.as, g.ldas) == 16 && row_align(g.bs, g.ldbs) == 16)
    mxfp4_tile_kernel<BM, BN, KB, STAGES, NWV, WGM, DTYPE, true><<<grid, block, lds, stream>>>(g, tm, tn, per_xcd, vec);
  else
    mxfp4_tile_kernel<BM, BN, KB, STAGES, NWV, WGM, DTYPE, false><<<grid, block, lds, stream>>>(g, tm, tn, per_xcd, vec);
}

template <int DTYPE>
static void mx_dispatch(const MxGemmArgs& g, hipStream_t stream) {
  const MxPlan p = plan_mxfp4(g);
  if (p.strip) {
    const dim3 grid((unsigned)(p.tiles_m * p.tiles_n)), block((unsigned)p.threads);
    const size_t lds = (size_t)(p.threads / 64) * p.bm * 20 * 4;
    const int ad = row_align(g.as, g.ldas) >= 4, bd = row_align(g.bs, g.ldbs) >= 4;
    if (p.bm == 16) mxfp4_strip_kernel<1, DTYPE><<<grid, block, lds, stream>>>(g, (int)p.tiles_n, ad, bd);
    else mxfp4_strip_kernel<2, DTYPE><<<grid, block, lds, stream>>>(g, (int)p.tiles_n, ad, bd);
  } else if (p.bm == 256) {
    mx_tile_launch<256, 256, 8, 2, 8, 2, DTYPE>(g, p, stream);
  } else if (p.bm == 128) {
    mx_tile_launch<128, 128, 8, 4, 4, 2, DTYPE>(g, p, stream);
  } else {
    mx_tile_launch<64, 128, 8, 4, 4, 1, DTYPE>(g, p, stream);
  }
}

hipError_t launch_mxfp4_gemm(int dtype, const MxGemmArgs& g, hipStream_t stream) {
  const int64_t n1 = g.M > 32 && g.K > 0 ? first_columns(g.M, g.N) : 0;
  if (n1 > 0) {
    MxGemmArgs lo = g, hi = g;
    lo.N = n1;
    hi.N = g.N - n1;
    hi.b = g.b + n1 * g.ldb;
    hi.bs = g.bs + n1 * g.ldbs;
    hi.c = static_cast<char*>(g.c) + n1 * (dtype == 2 ? 4 : 2);
    const hipError_t e = launch_mxfp4_gemm(dtype, lo, stream);
    return e != hipSuccess ? e : launch_mxfp4_gemm(dtype, hi, stream);
  }
  if (dtype == 0) mx_dispatch<0>(g, stream);
  else if (dtype == 1) mx_dispatch<1>(g, stream);
  else mx_dispatch<2>(g, stream);
  return hipGetLastError();
}

}  // namespace qg
