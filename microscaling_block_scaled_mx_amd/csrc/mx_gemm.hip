// Block-scaled MX GEMM for gfx950: C = A . B^T on K-major packed operands,
// on the CDNA4 scaled matrix cores (v_mfma_scale_f32_32x32x64_f8f6f4: E8M0
// block scales applied inside the instruction, binary32 accumulation).
//
// [P1] "feat(mxfp6): MXFP6 (E2M3) Flux linears, a fused MLP, and the MLPerf
//      recipe": MXFP6 GEMMs for forward, dgrad and wgrad, bias added in the
//      store epilogue into the fp32 accumulator (description, commit
//      messages).
// [P3] "MXFP4 training for Flux models": MXFP4 GEMM, NT layout
//      (Troubleshooting); 256x256 tiles at the Flux QKV shape (Tuned GEMMs).
// [P4] "MXFP8 cudnn-fe Swiglu fused Grouped MLP fwd/bwd and wgrad group
//      gemm": ragged grouped GEMM with the expert picked from the tile
//      coordinate (expert sizes are 128-row multiples, so a tile never
//      spans two experts), SwiGLU / dSwiGLU epilogues that quantize rowwise 1x32 and
//      columnwise 32x1 in the same launch, ragged-K weight gradient writing
//      zeros for empty experts (commit messages).
//
// The tile itself (staging, main loop, epilogues) is in mx_gemm_tile.h.
#include <atomic>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "mx_device.h"
#include "mx_gemm_tile.h"
#include "mx_kernels.h"

namespace mx {

namespace {

// One launch, one GEMM (or one grouped GEMM): workgroup (x, y, z) computes
// tile (x, y) of group z.
template <int FMT, int BM, int BN, int MODE, int EPI, int OCC = 1>
__global__ __launch_bounds__(tile_threads(BM, BN, EPI), OCC) void gemm_kernel(GemmParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[Cfg<FMT, BM, BN, MODE, EPI, OCC>::kSmem];
  gemm_tile<FMT, BM, BN, MODE, EPI, OCC>(p, blockIdx.x, blockIdx.y, blockIdx.z, smem);
}

// The dense tile shapes {BM, BN, workgroups per compute unit}, in the order
// of GemmMany::shape.
constexpr int kNumDense = 8;
constexpr int kDenseShapes[kNumDense][3] = {{256, 256, 1}, {256, 192, 1}, {192, 256, 1}, {192, 192, 1},
                                            {256, 128, 1}, {256, 128, 2}, {128, 256, 2}, {192, 192, 2}};

template <int FMT, int SH>
using DenseCfg = Cfg<FMT, kDenseShapes[SH][0], kDenseShapes[SH][1], kDense, kEpiStore, kDenseShapes[SH][2]>;

template <int FMT, int SH>
__device__ __forceinline__ void dense_tile_sh(const GemmParams& p, int local, uint8_t* smem) {
  gemm_tile<FMT, kDenseShapes[SH][0], kDenseShapes[SH][1], kDense, kEpiStore, kDenseShapes[SH][2]>(p, local, 0, 0,
                                                                                                    smem);
}

// Several dense GEMMs in one launch: workgroup w computes tile
// w - first[i] of GEMM i (first[i] <= w < first[i + 1]) with that GEMM's
// tile shape, SA or SB (indices into kDenseShapes); the branch is uniform
// across the workgroup.  Both shapes run the same number of wavefronts.
template <int FMT, int SA, int SB>
__global__ __launch_bounds__(tile_threads(kDenseShapes[SA][0], kDenseShapes[SA][1]), kDenseShapes[SA][2]) void gemm_many_kernel(GemmMany m) {
  static_assert(DenseCfg<FMT, SA>::kThreads == DenseCfg<FMT, SB>::kThreads, "one workgroup size per launch");
  static_assert(kDenseShapes[SA][2] == kDenseShapes[SB][2], "one residency per launch");
  constexpr int kA = DenseCfg<FMT, SA>::kSmem, kB = DenseCfg<FMT, SB>::kSmem;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kA > kB ? kA : kB];
  const int w = blockIdx.x;
  int i = 0;
  while (i + 1 < m.n && w >= m.first[i + 1]) ++i;
  const int local = w - m.first[i];
  if (SA == SB || m.shape[i] == SA) dense_tile_sh<FMT, SA>(m.p[i], local, smem);
  else dense_tile_sh<FMT, SB>(m.p[i], local, smem);
}

template <int FMT, int BM, int BN, int MODE, int EPI, int OCC = 1>
hipError_t launch_one(const GemmParams& p, hipStream_t stream) {
  dim3 grid;
  if (MODE == kDense) {
    const int64_t parts = EPI == kEpiSplit ? p.split_k : 1;
    if (parts < 1) return hipErrorInvalidValue;
    if ((p.M / BM) * (p.N / BN) * parts >= (1ll << 31)) return hipErrorInvalidValue;
    grid = dim3((unsigned)((p.M / BM) * (p.N / BN) * parts), 1, 1);
  } else if (MODE == kRaggedM) {
    // column tiles x an upper bound on the row tiles: sum over groups of
    // ceil(count / BM) <= R / BM + G; the surplus workgroups exit at once
    const int64_t nt = EPI == kEpiSwiglu ? 2 * p.F / BN : p.N / BN;
    const int64_t rows = p.R > 0 ? (p.R + BM - 1) / BM + p.G : 0;
    if (nt * rows >= (1ll << 31)) return hipErrorInvalidValue;
    grid = dim3((unsigned)(nt * rows), 1, 1);
  } else {
    grid = dim3((unsigned)(p.N / BN), (unsigned)(p.M / BM), (unsigned)p.G);
  }
  if (grid.x == 0 || grid.y == 0 || grid.z == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm_kernel<FMT, BM, BN, MODE, EPI, OCC>), grid, dim3(Cfg<FMT, BM, BN, MODE, EPI, OCC>::kThreads),
                     0, stream, p);
  return hipGetLastError();
}

// Dense tile shape (index into kDenseShapes): the one whose rounds of one
// tile per compute unit cost the least output area (rounds x BM x BN),
// larger tiles first on ties -- e.g. 4096 x 3072 takes 256 tiles of
// 256 x 192 in one round instead of 192 tiles of 256 x 256 on 192 of the 256
// compute units.  -1: no shape divides M x N.
int dense_shape(int64_t M, int64_t N) {
  const int64_t cus = cu_count();
  int best = -1;
  int64_t best_cost = 0;
  for (int i = 0; i < kNumDense; ++i) {
    const int bm = kDenseShapes[i][0], bn = kDenseShapes[i][1];
    if (kDenseShapes[i][2] != 1 || M % bm || N % bn) continue;
    const int64_t tiles = (M / bm) * (N / bn);
    const int64_t cost = ((tiles + cus - 1) / cus) * bm * bn;
    if (best < 0 || cost < best_cost) {
      best = i;
      best_cost = cost;
    }
  }
  return best;
}

// Measured launch plans (tile, workgroups per CU, K split) for the shapes
// of the Flux-12B block linears where the best of a sweep over every dense
// tiling and K split beat the rounds x tile-area rule: compute units,
// format, M, N, K, then the plan.  A plan with split_k > 1 needs a
// workspace, so mx_gemm (which has none) takes the rule for those shapes.
struct Tuned {
  int cus, fmt;
  int64_t M, N, K;
  GemmPlan plan;
};
constexpr Tuned kTuned[] = {
#include "mx_tuned.inc"
    {0, 0, 0, 0, 0, {0, 0, 0, 0}},  // end (no device has 0 compute units)
};

const Tuned* tuned(int fmt, int64_t M, int64_t N, int64_t K) {
  const int cus = cu_count();
  for (const Tuned& t : kTuned)
    if (t.cus == cus && t.fmt == fmt && t.M == M && t.N == N && t.K == K) return &t;
  return nullptr;
}

int shape_index(int bm, int bn, int wg) {
  for (int i = 0; i < kNumDense; ++i)
    if (kDenseShapes[i][0] == bm && kDenseShapes[i][1] == bn && kDenseShapes[i][2] == wg) return i;
  return -1;
}

// The shape a dense launch uses: the caller's (p.tile_shape = 1 + its
// index), else a tuned plan's without a K split, else the one dense_shape
// picks.
int dense_shape_of(int fmt, const GemmParams& p) {
  if (p.tile_shape > 0 && p.tile_shape <= kNumDense) return p.tile_shape - 1;
  const Tuned* t = tuned(fmt, p.M, p.N, p.K);
  if (t && t->plan.split_k <= 1) {
    const int i = shape_index(t->plan.tile_m, t->plan.tile_n, t->plan.wg_per_cu);
    if (i >= 0 && p.M % kDenseShapes[i][0] == 0 && p.N % kDenseShapes[i][1] == 0) return i;
  }
  return dense_shape(p.M, p.N);
}

// Split-K reduction: thread q sums 4 consecutive columns of one row over the
// parts in order, adds the bias and rounds once.
template <int S>
__global__ __launch_bounds__(256) void splitk_reduce_kernel(const float* __restrict__ ws, int64_t M, int64_t N,
                                                            const void* __restrict__ bias, int bias_f32,
                                                            void* __restrict__ c, int c_f32, int64_t ldc) {
  const int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t n4 = N / 4;
  if (q >= M * n4) return;
  const int64_t m = q / n4, n = (q - m * n4) * 4;
  const float* src = ws + m * N + n;
  float4 v[S];
#pragma unroll
  for (int s = 0; s < S; ++s) v[s] = *reinterpret_cast<const float4*>(src + s * (M * N));
  float4 a = v[0];
#pragma unroll
  for (int s = 1; s < S; ++s) {
    a.x = a.x + v[s].x;
    a.y = a.y + v[s].y;
    a.z = a.z + v[s].z;
    a.w = a.w + v[s].w;
  }
  if (bias != nullptr) {
    float4 b;
    if (bias_f32) {
      b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(bias) + n);
    } else {
      const uint2 h = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(bias) + n);
      b = make_float4(bf16_lo(h.x), bf16_hi(h.x), bf16_lo(h.y), bf16_hi(h.y));
    }
    a.x = a.x + b.x;
    a.y = a.y + b.y;
    a.z = a.z + b.z;
    a.w = a.w + b.w;
  }
  if (c_f32) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(c) + m * ldc + n) = a;
  } else {
    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(c) + m * ldc + n) =
        make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

template <int FMT, int EPI>
hipError_t launch_dense(const GemmParams& p, hipStream_t stream) {
  switch (dense_shape_of(FMT, p)) {
    case 0: return launch_one<FMT, 256, 256, kDense, EPI>(p, stream);
    case 1: return launch_one<FMT, 256, 192, kDense, EPI>(p, stream);
    case 2: return launch_one<FMT, 192, 256, kDense, EPI>(p, stream);
    case 3: return launch_one<FMT, 192, 192, kDense, EPI>(p, stream);
    case 4: return launch_one<FMT, 256, 128, kDense, EPI>(p, stream);
    case 5: return launch_one<FMT, 256, 128, kDense, EPI, 2>(p, stream);
    case 6: return launch_one<FMT, 128, 256, kDense, EPI, 2>(p, stream);
    case 7: return launch_one<FMT, 192, 192, kDense, EPI, 2>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

template <int FMT>
hipError_t launch_fmt(const GemmParams& p, int mode, int epi, hipStream_t stream) {
  if (mode == kDense) {
    if (epi == kEpiAccum) return launch_dense<FMT, kEpiAccum>(p, stream);
    if (epi == kEpiSplit) return launch_dense<FMT, kEpiSplit>(p, stream);
    return launch_dense<FMT, kEpiStore>(p, stream);
  }
  if (mode == kRaggedM) {
    // 256-row tiles for the plain store.  The epilogues that quantize take
    // 128 rows with 8 wavefronts: dSwiGLU's two bf16 LDS tiles would not fit
    // at 256, and SwiGLU measured 8-9% faster (at expert sizes that are
    // multiples of 128, every 128-row tile is full, so no round ends part
    // empty; the plain store gained nothing from it)
    if (epi == kEpiSwiglu) return launch_one<FMT, 128, 256, kRaggedM, kEpiSwiglu>(p, stream);
    if (epi == kEpiDSwiglu) return launch_one<FMT, 128, 256, kRaggedM, kEpiDSwiglu>(p, stream);
    return launch_one<FMT, 256, 256, kRaggedM, kEpiStore>(p, stream);
  }
  return launch_one<FMT, 256, 256, kRaggedK, kEpiStore>(p, stream);
}

// Workgroup ranges of a many-launch whose shapes are set.
bool plan_many(GemmMany& m) {
  int64_t tiles = 0;
  for (int i = 0; i < m.n; ++i) {
    const int sh = m.shape[i];
    m.first[i] = (int)tiles;
    tiles += (m.p[i].M / kDenseShapes[sh][0]) * (m.p[i].N / kDenseShapes[sh][1]);
  }
  m.first[m.n] = (int)tiles;
  return tiles < (1ll << 31);
}

template <int FMT, int SA, int SB>
hipError_t launch_many_k(GemmMany m, hipStream_t stream) {
  if (!plan_many(m)) return hipErrorInvalidValue;
  const unsigned tiles = (unsigned)m.first[m.n];
  if (tiles == 0) return hipSuccess;
  hipLaunchKernelGGL((gemm_many_kernel<FMT, SA, SB>), dim3(tiles), dim3(DenseCfg<FMT, SA>::kThreads), 0, stream, m);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_many_single(const GemmMany& m, int sh, hipStream_t stream) {
  switch (sh) {
    case 0: return launch_many_k<FMT, 0, 0>(m, stream);
    case 1: return launch_many_k<FMT, 1, 1>(m, stream);
    case 2: return launch_many_k<FMT, 2, 2>(m, stream);
    case 3: return launch_many_k<FMT, 3, 3>(m, stream);
    case 4: return launch_many_k<FMT, 4, 4>(m, stream);
    case 5: return launch_many_k<FMT, 5, 5>(m, stream);
    case 6: return launch_many_k<FMT, 6, 6>(m, stream);
    case 7: return launch_many_k<FMT, 7, 7>(m, stream);
    default: return hipErrorInvalidValue;
  }
}

// Two tile shapes can share a launch when they run the same number of
// wavefronts at the same residency: the 4-wavefront shapes at one workgroup
// per CU (256x192, 192x256, 192x192, 256x128) pairwise, and those at two
// (256x128, 128x256, 192x192) pairwise except 128x256 with 192x192 (their
// union spills at half the register file).  256x256 runs 8 wavefronts
// alone.
constexpr bool pairable(int a, int b) {
  return a != b && a != 0 && b != 0 && kDenseShapes[a][2] == kDenseShapes[b][2] && !(a == 6 && b == 7) &&
         !(a == 7 && b == 6);
}
template <int FMT>
hipError_t launch_many_pair(const GemmMany& m, int a, int b, hipStream_t stream) {
  switch (a * kNumDense + b) {  // a < b
    case 1 * kNumDense + 2: return launch_many_k<FMT, 1, 2>(m, stream);
    case 1 * kNumDense + 3: return launch_many_k<FMT, 1, 3>(m, stream);
    case 1 * kNumDense + 4: return launch_many_k<FMT, 1, 4>(m, stream);
    case 2 * kNumDense + 3: return launch_many_k<FMT, 2, 3>(m, stream);
    case 2 * kNumDense + 4: return launch_many_k<FMT, 2, 4>(m, stream);
    case 3 * kNumDense + 4: return launch_many_k<FMT, 3, 4>(m, stream);
    case 5 * kNumDense + 6: return launch_many_k<FMT, 5, 6>(m, stream);
    case 5 * kNumDense + 7: return launch_many_k<FMT, 5, 7>(m, stream);
    default: return hipErrorInvalidValue;
  }
}

// The GEMMs grouped into launches: the shapes in use taken in table order,
// each with the first later shape it can share a launch with (a linear
// layer's forward / data-gradient 256x192 and weight-gradient 192x192 at
// the Flux shapes are one such pair); items keep their order in a launch.
template <int FMT>
hipError_t launch_many_fmt(const GemmMany& all, hipStream_t stream) {
  bool used[kNumDense] = {};
  for (int i = 0; i < all.n; ++i) used[all.shape[i]] = true;
  for (int a = 0; a < kNumDense; ++a) {
    if (!used[a]) continue;
    used[a] = false;
    int b = -1;
    for (int k = a + 1; k < kNumDense && b < 0; ++k)
      if (used[k] && pairable(a, k)) b = k;
    if (b >= 0) used[b] = false;
    GemmMany m;
    memset(&m, 0, sizeof m);
    for (int i = 0; i < all.n; ++i)
      if (all.shape[i] == a || all.shape[i] == b) {
        m.p[m.n] = all.p[i];
        m.shape[m.n] = all.shape[i];
        ++m.n;
      }
    const hipError_t e = b >= 0 ? launch_many_pair<FMT>(m, a, b, stream) : launch_many_single<FMT>(m, a, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int cu_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

int dense_tile_index(int bm, int bn, int wg_per_cu, int64_t M, int64_t N) {
  for (int i = 0; i < kNumDense; ++i)
    if (kDenseShapes[i][0] == bm && kDenseShapes[i][1] == bn && kDenseShapes[i][2] == wg_per_cu)
      return (M % bm || N % bn) ? -1 : i;
  return -1;
}

hipError_t launch_gemm_many(GemmMany m, int fmt, hipStream_t stream) {
  if (m.n < 1 || m.n > kGemmManyMax) return hipErrorInvalidValue;
  for (int i = 0; i < m.n; ++i)
    if ((m.shape[i] = dense_shape_of(fmt, m.p[i])) < 0) return hipErrorInvalidValue;
  switch (fmt) {
    case kE2M1: return launch_many_fmt<kE2M1>(m, stream);
    case kE2M3: return launch_many_fmt<kE2M3>(m, stream);
    case kE4M3: return launch_many_fmt<kE4M3>(m, stream);
    default: return hipErrorInvalidValue;
  }
}

bool plan_gemm(int fmt, int64_t M, int64_t N, int64_t K, GemmPlan* out) {
  if (const Tuned* t = tuned(fmt, M, N, K)) {
    *out = t->plan;
    return true;
  }
  const int sh = dense_shape(M, N);
  if (sh < 0) return false;
  *out = GemmPlan{kDenseShapes[sh][0], kDenseShapes[sh][1], kDenseShapes[sh][2], 1};
  return true;
}

hipError_t launch_splitk_reduce(const float* ws, int split_k, int64_t M, int64_t N, const void* bias, int bias_f32,
                                void* c, int c_f32, int64_t ldc, hipStream_t stream) {
  const int64_t threads = M * (N / 4);
  if (threads == 0) return hipSuccess;
  const int64_t blocks = (threads + 255) / 256;
  if (blocks >= (1ll << 31)) return hipErrorInvalidValue;
#define MX_REDUCE(S)                                                                                         \
  case S:                                                                                                    \
    hipLaunchKernelGGL(splitk_reduce_kernel<S>, dim3((unsigned)blocks), dim3(256), 0, stream, ws, M, N, bias, \
                       bias_f32, c, c_f32, ldc);                                                             \
    break;
  switch (split_k) {
    MX_REDUCE(2)
    MX_REDUCE(3)
    MX_REDUCE(4)
    MX_REDUCE(5)
    MX_REDUCE(6)
    MX_REDUCE(7)
    MX_REDUCE(8)
    MX_REDUCE(9)
    MX_REDUCE(10)
    MX_REDUCE(11)
    MX_REDUCE(12)
    MX_REDUCE(13)
    MX_REDUCE(14)
    MX_REDUCE(15)
    MX_REDUCE(16)
    default: return hipErrorInvalidValue;
  }
#undef MX_REDUCE
  return hipGetLastError();
}

hipError_t launch_gemm(const GemmParams& p, int fmt, int mode, int epi, hipStream_t stream) {
  switch (fmt) {
    case kE2M1: return launch_fmt<kE2M1>(p, mode, epi, stream);
    case kE2M3: return launch_fmt<kE2M3>(p, mode, epi, stream);
    case kE4M3: return launch_fmt<kE4M3>(p, mode, epi, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mx
