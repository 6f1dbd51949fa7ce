// int4 GPTQ products grouped by expert (rows sorted by expert, see groups.hpp):
// Y[r] = X[r] . dequant(W_e)^T for the rows r of expert e, the storage of
// int4_kernels.hip once per expert.
//
// As in the products of one weight, the activations are contracted with the exact
// bf16 values 128 + q and the offset is removed per 128-row group of k with the
// activations' sum; nothing is rounded below fp32 before the scale is applied.
// Two kernels:
//  * few rows an expert (decoding): the codes of the reached experts are read once
//    and that read is the time: a workgroup takes a strip of columns over the whole
//    of k, split over its waves;
//  * many rows: the pipelined MFMA tile (int4_pipe.hpp), with the activations
//    prepared by a first small kernel when there is a workspace.
#include "groups.hpp"
#include "int4_common.hpp"
#include "int4_pipe.hpp"
#include "launch.hpp"

namespace qg {

constexpr int kInt4Band = 8;   // row tiles per band of an expert's tile order

// ---------------------------------------------------------------------------
// few rows an expert: strips of 16 CPL columns over the whole of k
//
// A workgroup owns 16 RT rows of an expert and 16 CPL columns; wave w takes the
// k groups w, w + waves, ...  Lane (cl, ks) loads CPL adjacent words of word row
// 4 s + ks: fragment c of step s then holds column CPL cl + c, and a word row's
// 16 lanes read 64 CPL contiguous bytes.  Both operands go from memory into the
// MFMA lane layout; the activations come from L2, only by the lanes whose rows there
// are (an expert has a few of the 16: 64 rows over 16 experts, 4096 -> 14336, 126 -> 95 us,
// the time of the weights at a large copy's rate).  One group a wave at a time, so
// that four workgroups share a CU and hide each other's latency (two at a time, half
// as many: 119 us).  Strips of 64 columns where that gives two workgroups a CU, else
// 32 or 16 (32 at the size above: 192 us).  The waves' partial tiles are summed
// through LDS in wave order.
// ---------------------------------------------------------------------------

template <int RT, int CPL>
__global__ __launch_bounds__(512) void grouped_int4_strip_kernel(Int4GroupedArgs a, int strips) {
  constexpr int ROWS = 16 * RT, COLS = 16 * CPL, P = COLS + 4;
  extern __shared__ __attribute__((aligned(16))) float ism[];   // [waves][ROWS][P]
  const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const GroupTile t = find_group_tile(a.offsets, (int)a.experts, (int)a.m, ROWS, strips, 1, blockIdx.x, lane);
  if (t.group < 0) return;
  const int cl = lane & 15, ks = lane >> 4, n = (int)a.n, groups = (int)(a.k >> 7);
  const int r0 = t.tm * ROWS, n0 = t.tn * COLS;
  const int col = min(n0 + CPL * cl, n - CPL);
  const uint32_t* qp = a.qweight + (int64_t)t.group * (a.k >> 3) * n + col;
  const uint16_t* sp = a.scales + (int64_t)t.group * groups * n + col;
  // without zero points the word is taken from the scales (never used: zmask)
  const uint32_t* zp = a.qzeros ? a.qzeros + (int64_t)t.group * groups * (n >> 3) + (col >> 3)
                                : reinterpret_cast<const uint32_t*>(a.scales);
  const int64_t zstride = a.qzeros ? n >> 3 : 0;
  const uint32_t zmask = a.qzeros ? 0xFFFFFFFFu : 0u;
  const int zshift = 4 * (col & 7);
  const uint16_t* xr[RT];
#pragma unroll
  for (int f = 0; f < RT; ++f) xr[f] = a.x + (int64_t)(t.row0 + r0 + 16 * f + cl) * a.ldx;   // (read below t.rows)

  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  const u32x4 ones = {kOnesBf16x2, kOnesBf16x2, kOnesBf16x2, kOnesBf16x2};
  f32x4 total[RT][CPL];
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int c = 0; c < CPL; ++c) total[f][c] = zero;

  for (int g = wave; g < groups; g += waves) {
    uint32_t words[4][CPL];
    u32x4 x[RT][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      load_words<CPL>(qp + (int64_t)(16 * g + 4 * s + ks) * n, words[s]);
#pragma unroll
      for (int f = 0; f < RT; ++f) {
        x[f][s] = u32x4{0u, 0u, 0u, 0u};
        if (r0 + 16 * f + cl < t.rows) x[f][s] = *reinterpret_cast<const u32x4*>(xr[f] + 128 * g + 32 * s + 8 * ks);
      }
    }
    const Meta<CPL> meta = load_meta<CPL>(sp + (int64_t)g * n, zp + g * zstride);
    f32x4 acc[RT][CPL], xs[RT];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      u32x4 xp[RT];
#pragma unroll
      for (int f = 0; f < RT; ++f) {
        xp[f] = x_pairs_permuted(x[f][s]);
        xs[f] = mfma16_bf16(xp[f], ones, s == 0 ? zero : xs[f]);
      }
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const u32x4 w = codes_as_bf16_pairs(words[s][c]);
#pragma unroll
        for (int f = 0; f < RT; ++f) acc[f][c] = mfma16_bf16(xp[f], w, s == 0 ? zero : acc[f][c]);
      }
    }
    float sc[CPL], bz[CPL];
    decode_meta<CPL>(meta, zshift, zmask, sc, bz);
#pragma unroll
    for (int f = 0; f < RT; ++f)
#pragma unroll
      for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          total[f][c][v] = __builtin_fmaf(sc[c], __builtin_fmaf(-bz[c], xs[f][v], acc[f][c][v]), total[f][c][v]);
  }

  float* mine = ism + wave * ROWS * P;
#pragma unroll
  for (int f = 0; f < RT; ++f)
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int v = 0; v < 4; ++v) mine[(16 * f + 4 * ks + v) * P + CPL * cl + c] = total[f][c][v];
  __syncthreads();
  const int rows = min(ROWS, t.rows - r0);
  for (int i = tid; i < rows * COLS; i += blockDim.x) {
    const int r = i / COLS, c = i - r * COLS;
    if (n0 + c >= n) continue;
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += ism[(w * ROWS + r) * P + c];
    a.y[(int64_t)(t.row0 + r0 + r) * a.ldy + n0 + c] = (uint16_t)f32_to_bf16_bits(s);
  }
}

// ---------------------------------------------------------------------------
// many rows an expert
// ---------------------------------------------------------------------------
template <int NWM, int NWN, int FM, int STAGES, bool PREP>
__global__ __launch_bounds__(64 * NWM * NWN) __attribute__((amdgpu_waves_per_eu(2))) void grouped_int4_pipe_kernel(
    Int4GroupedArgs a, const float* __restrict__ xsum, int tiles_n, int vec) {
  const GroupTile t = find_group_tile(a.offsets, (int)a.experts, (int)a.m, 16 * FM * NWM, tiles_n, kInt4Band, blockIdx.x,
                                      threadIdx.x & 63);
  if (t.group < 0) return;
  const int64_t n = a.n, groups = a.k >> 7, e = t.group;
  const LoraEpi none{};
  int4_pipe_tile<NWM, NWN, FM, STAGES, PREP, false>(
      a.x + t.row0 * a.ldx, a.ldx, a.qweight + e * (a.k >> 3) * n, a.scales + e * groups * n,
      a.qzeros ? a.qzeros + e * groups * (n >> 3) : nullptr, PREP ? xsum + t.row0 : nullptr, a.m, a.y + t.row0 * a.ldy,
      a.ldy, t.rows, (int)n, (int)a.k, 0, t.tm, t.tn, 0, vec, 1, (int)groups, nullptr, nullptr, 0, none);
}

// The activations of the experts' rows in the decode's pair order, and their fp32
// sums over each 128-row group of k, xsum[g][row]; other rows are not read.
// Thread = (row, 8-element chunk); the 16 threads of a group are adjacent lanes.
__global__ __launch_bounds__(256) void grouped_int4_prep_kernel(Int4GroupedArgs a, uint16_t* __restrict__ xp,
                                                                float* __restrict__ xsum) {
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int cpr = (int)(a.k >> 3);
  const int64_t row = t / cpr;
  if (row >= a.m || row < a.offsets[0] || row >= a.offsets[a.experts]) return;   // (whole 16-lane groups)
  const int c = (int)(t - row * cpr);
  const u32x4 v = *reinterpret_cast<const u32x4*>(a.x + row * a.ldx + 8 * c);
  *reinterpret_cast<u32x4*>(xp + row * a.k + 8 * c) = x_pairs_permuted(v);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = dot2_bf16(v[i], kOnesBf16x2, sum);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 16);
  if ((c & 15) == 0) xsum[(int64_t)(c >> 4) * a.m + row] = sum;
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------
struct Int4GroupedPlan {
  bool strip;
  int bm, bn, threads;
  int64_t blocks;
};

static Int4GroupedPlan plan_int4_grouped(int64_t experts, int64_t m, int64_t n, int64_t k) {
  const int64_t avg = m / experts;
  Int4GroupedPlan p{};
  if (avg <= 24) {
    p.strip = true;
    p.bm = avg <= 8 ? 16 : 32;
    const int64_t reached = m < experts ? m : experts;
    p.bn = 64;
    while (p.bn > 16 && reached * ((n + p.bn - 1) / p.bn) < 512) p.bn /= 2;
    const int64_t waves = k / 128 < 8 ? k / 128 : 8;
    p.threads = (int)(64 * waves);
  } else {
    p.bm = avg <= 64 ? 64 : avg <= 128 ? 128 : 256;
    p.bn = 128;
    p.threads = 2 * p.bm;
  }
  p.blocks = group_tile_blocks(m, experts, p.bm, (n + p.bn - 1) / p.bn);
  return p;
}

int64_t int4_grouped_threads(int64_t experts, int64_t m, int64_t n, int64_t k) {
  const Int4GroupedPlan p = plan_int4_grouped(experts, m, n, k);
  return p.blocks * p.threads;
}

int64_t int4_grouped_workspace(int64_t experts, int64_t m, int64_t n, int64_t k) {
  return plan_int4_grouped(experts, m, n, k).strip ? 0 : m * k * 2 + (k / 128) * m * 4;
}

template <int RT, int CPL>
static void strip_launch(const Int4GroupedArgs& a, const Int4GroupedPlan& p, hipStream_t stream) {
  const size_t lds = (size_t)(p.threads / 64) * 16 * RT * (16 * CPL + 4) * 4;
  grouped_int4_strip_kernel<RT, CPL><<<dim3((unsigned)p.blocks), dim3((unsigned)p.threads), lds, stream>>>(
      a, (int)((a.n + p.bn - 1) / p.bn));
}

template <int NWM, int NWN, int FM, int STAGES, bool PREP>
static void pipe_launch(const Int4GroupedArgs& a, const Int4GroupedPlan& p, const float* xsum, hipStream_t stream) {
  using S = PipeShape<NWM, NWN, FM, PREP>;
  constexpr size_t main_bytes = (size_t)STAGES * S::STAGE_DW * 4, out = (size_t)S::BM * S::OP * 2;
  constexpr size_t lds = main_bytes > out ? main_bytes : out;
  static_assert(lds <= 160 * 1024, "LDS budget");
  const int vec = ((uintptr_t)a.y & 15u) == 0 && a.ldy % 8 == 0;
  grouped_int4_pipe_kernel<NWM, NWN, FM, STAGES, PREP><<<dim3((unsigned)p.blocks), dim3(S::T), lds, stream>>>(
      a, xsum, (int)((a.n + S::BN - 1) / S::BN), vec);
}

template <bool PREP>
static void pipe_dispatch(const Int4GroupedArgs& a, const Int4GroupedPlan& p, const float* xsum, hipStream_t stream) {
  if (p.bm == 256) pipe_launch<4, 2, 4, 4, PREP>(a, p, xsum, stream);
  else if (p.bm == 128) pipe_launch<2, 2, 4, 4, PREP>(a, p, xsum, stream);
  else pipe_launch<1, 2, 4, 4, PREP>(a, p, xsum, stream);
}

hipError_t launch_int4_grouped(const Int4GroupedArgs& a, void* ws, int64_t ws_bytes, hipStream_t stream) {
  const Int4GroupedPlan p = plan_int4_grouped(a.experts, a.m, a.n, a.k);
  if (p.strip) {
    switch (p.bm / 16 * 100 + p.bn) {
      case 116: strip_launch<1, 1>(a, p, stream); break;
      case 132: strip_launch<1, 2>(a, p, stream); break;
      case 164: strip_launch<1, 4>(a, p, stream); break;
      case 216: strip_launch<2, 1>(a, p, stream); break;
      case 232: strip_launch<2, 2>(a, p, stream); break;
      default: strip_launch<2, 4>(a, p, stream); break;
    }
  } else if (ws != nullptr && ws_bytes >= int4_grouped_workspace(a.experts, a.m, a.n, a.k)) {
    uint16_t* xp = (uint16_t*)ws;
    float* xsum = (float*)(xp + a.m * a.k);
    const int64_t threads = a.m * (a.k / 8);
    grouped_int4_prep_kernel<<<dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, stream>>>(a, xp, xsum);
    Int4GroupedArgs b = a;
    b.x = xp;
    b.ldx = a.k;
    pipe_dispatch<true>(b, p, xsum, stream);
  } else {
    pipe_dispatch<false>(a, p, nullptr, stream);
  }
  return hipGetLastError();
}

}  // namespace qg
