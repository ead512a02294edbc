// mx_gemm_act: C = act(A . B^T + bias) + residual on packed operands, with
// the 8-bit checkpoint of the pre-activation from the same epilogue, for any
// number of rows.
//
// Two kernels.  Many rows: the output tile of mx_gemm_tile.h (operands
// through LDS, 32x32x64 matrix instructions) with the epilogue kEpiAct, bound
// by the matrix cores.  Few rows, down to one: gemm_rows_kernel below, whose
// wavefronts each stage their operands through a ring in LDS, bound by the one
// pass over the weights; they split K inside the workgroup, so that a short
// product still keeps enough loads in flight and needs no second launch.
#include <type_traits>

#include "mx_act.h"
#include "mx_device.h"
#include "mx_gemm_tile.h"
#include "mx_kernels.h"
#include "mx_linear.h"

namespace mx {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

// ------------------------------------------------------------------ many rows
// The products of a launch, one or two of them: workgroups from `first` on
// compute tiles of the second.  (A type of its own for one: indexed by the
// workgroup, the arguments would be loaded again wherever they are used, which
// cost a few-rows launch 0.5 us.)
template <int COUNT>
struct Products {
  GemmActParams p[COUNT];
  int first;  // tiles of p[0]
  int summing;      // COUNT = 2: workgroups before them that finish column sums
  ColumnSums sums;
};
template <int COUNT>
__device__ __forceinline__ const GemmActParams& product_of(const Products<COUNT>& all, int& tile) {
  if constexpr (COUNT == 1) return all.p[0];
  if (tile < all.first) return all.p[0];
  tile -= all.first;
  return all.p[1];
}
// Whether this workgroup's work was column sums; if not, its tile.
template <int COUNT>
__device__ __forceinline__ bool summed(const Products<COUNT>& all, int& tile) {
  tile = blockIdx.x;
  if constexpr (COUNT == 2) {
    if (tile < all.summing) {
      finish_column_sum(all.sums, (int64_t)tile * blockDim.x + threadIdx.x);
      return true;
    }
    tile -= all.summing;
  }
  return false;
}

// Kernel times (E4M3 8191 x 2048 x 8192, bias and residual): 114 us, 2.41
// PFLOP/s, where mx_gemm reaches 2.44 on large products; E2M1 16384 x 8192 x
// 4096, bias: 278 us, 3.96 PFLOP/s.  With GELU and a checkpoint (E2M3
// 8192 x 8192 x 2048) 136 us, 2.02 PFLOP/s: products and epilogue alternate in
// a workgroup.
template <int FMT, int BM, int BN, int OCC, int COUNT>
__global__ __launch_bounds__(tile_threads(BM, BN, kEpiAct), OCC) void gemm_act_kernel(Products<COUNT> all) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[Cfg<FMT, BM, BN, kDense, kEpiAct, OCC>::kSmem];
  int tile;
  if (summed(all, tile)) return;
  const GemmActParams& p = product_of(all, tile);
  gemm_tile<FMT, BM, BN, kDense, kEpiAct, OCC>(p, tile, 0, 0, smem);
}

// ------------------------------------------------------------------ few rows
// v_mfma_scale_f32_16x16x128_f8f6f4 takes one whole K group: lane l holds row
// l % 16, and of the group's 128 elements (g = l / 16) E2M1 / E2M3 the 32
// of block g, E4M3 [16g, 16g+16) and [64+16g, 64+16g+16); its scale operand is
// the byte of block g (layouts measured).  With B as the first operand, a lane
// ends with C row l % 16 and the four columns 4g .. 4g+3.
//
// W wavefronts compute a 16 MI x 16 NJ tile of C, wavefront w from the K groups
// w, w + W, ...; each stages its groups in a ring of D buffers of its own in
// LDS, filled by direct global -> LDS loads that need no registers and no
// barrier.  The loads take a panel's rows back to back, lane after lane, so a
// wavefront's load is whole cache lines (the layout above takes 16 bytes of
// each of 16 rows at a time); the 16-byte chunks of a row are permuted on the way so that
// the reads of 16 rows spread over the LDS banks.  The partial tiles meet in
// LDS and are summed in wavefront order: the result does not depend on
// timing.  Rows past the operands' ends are loaded as the last row and never
// stored.  Device time of a replayed graph: 1 x 12288 x 4096 E2M1 6.8 us, 3.9
// TB/s of weights; 24 x 4096 x 12288 E4M3 11.5 us, 4.6 TB/s (a large copy
// reaches 5.27).
template <int FMT, int MI, int NJ, int W, int D>
struct RowsCfg {
  static constexpr int kTR = 16 * MI, kTC = 16 * NJ;
  static constexpr int kGB = 16 * FmtTraits<FMT>::kBits;  // code bytes of a row in one K group
  static constexpr int kChunks = kGB / 16;
  // 16-byte loads per lane and stage; the last one may cover 32 lanes only
  static constexpr int kALoads = (kTR * kChunks + 63) / 64, kBLoads = (kTC * kChunks + 63) / 64;
  static constexpr int kLoads = kALoads + kBLoads + 2;  // + the scale dwords of A and of B
  static constexpr int kAOff = 0, kBOff = kTR * kGB, kSOff = kBOff + kTC * kGB;
  static constexpr int kStage = kSOff + 2 * 256;  // (64 scale dwords each)
  static constexpr int kRing = W * D * kStage;
  // epilogue: units of four columns, and how many a thread takes
  static constexpr int kUnits = kTR * kTC / 4, kPerRow = kTC / 4, kSteps = (kUnits + 64 * W - 1) / (64 * W);
  static_assert(kUnits % 64 == 0, "whole wavefronts");
  static constexpr int kPitch = kTC + 4;  // floats: the 16 rows of a write start in different banks
  static constexpr int kRed = W * kTR * kPitch * 4;
  static constexpr int kSmem = kRing > kRed ? kRing : kRed;
  static_assert(D >= 2 && kLoads * (D - 1) < 64, "outstanding loads are counted in six bits");
  static_assert(kSmem <= 163840 && MI <= 4 && NJ >= 2 && NJ <= 4, "LDS budget; scale slots; whole checkpoint blocks");
};

// Place of 16-byte chunk c of row x (of 16) in its staged row.
template <int FMT>
__device__ __forceinline__ int rows_place(int x, int c) {
  if constexpr (FMT == kE4M3) return c ^ ((x >> 1) & 7);
  else if constexpr (FMT == kE2M1) return c ^ ((x >> 2) & 3);
  else return c + (x >> 3) == 6 ? 0 : c + (x >> 3);
}
template <int FMT>
__device__ __forceinline__ int rows_chunk(int x, int place) {
  if constexpr (FMT == kE2M3) return place < (x >> 3) ? 5 : place - (x >> 3);
  else return rows_place<FMT>(x, place);
}

// This lane's operand from a staged panel of 16 rows; `row` is the operand's
// row (its bit 4 orders the tails of an E2M3 group).
template <int FMT>
__device__ __forceinline__ v8i rows_fragment(const uint8_t* panel, int x, int g, uint32_t row) {
  constexpr int kGB = 16 * FmtTraits<FMT>::kBits;
  const uint8_t* at = panel + x * kGB;
  const v4i a = *reinterpret_cast<const v4i*>(at + 16 * rows_place<FMT>(x, g));
  if constexpr (FMT == kE2M1) {
    return v8i{a.x, a.y, a.z, a.w, 0, 0, 0, 0};
  } else if constexpr (FMT == kE2M3) {
    const int tail = g ^ (int)((row >> 4) & 1u);  // which 8 of the last 32 bytes
    const v2i h = *reinterpret_cast<const v2i*>(at + 16 * rows_place<FMT>(x, 4 + (tail >> 1)) + 8 * (tail & 1));
    return v8i{a.x, a.y, a.z, a.w, h.x, h.y, 0, 0};
  } else {
    const v4i b = *reinterpret_cast<const v4i*>(at + 16 * rows_place<FMT>(x, 4 + g));
    return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
}

// Four consecutive elements (8 bytes of bf16, 16 of binary32) and their values.
__device__ __forceinline__ uint4 load_four(const uint8_t* at, int f32) {
  const uint2 lo = *reinterpret_cast<const uint2*>(at);
  uint2 hi = make_uint2(0u, 0u);
  if (f32) hi = *reinterpret_cast<const uint2*>(at + 8);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void add_four(float (&v)[4], const uint4& q, int f32) {
  v[0] = v[0] + (f32 ? __uint_as_float(q.x) : bf16_lo(q.x));
  v[1] = v[1] + (f32 ? __uint_as_float(q.y) : bf16_hi(q.x));
  v[2] = v[2] + (f32 ? __uint_as_float(q.z) : bf16_lo(q.y));
  v[3] = v[3] + (f32 ? __uint_as_float(q.w) : bf16_hi(q.y));
}

// A point that no memory access is moved across.
__device__ __forceinline__ void memory_fence() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" ::: "memory");
#endif
}

template <int FMT, int MI, int NJ, int W, int D, int COUNT>
__global__ __launch_bounds__(64 * W) void gemm_rows_kernel(Products<COUNT> all) {
  using CF = RowsCfg<FMT, MI, NJ, W, D>;
  int tile;
  if (summed(all, tile)) return;
  const GemmActParams& p = product_of(all, tile);
  __shared__ __attribute__((aligned(16))) uint8_t smem[CF::kSmem];
  const int t = threadIdx.x, lane = t & 63, wave = wave_uniform(t >> 6);
  const int x = lane & 15, g = lane >> 4;
  // (M and N are below 2^31, a tile's rows and columns below 64)
  const uint32_t M = (uint32_t)p.M, N = (uint32_t)p.N;
  const int tiles_m = (int)((M + CF::kTR - 1) / CF::kTR);
  const int tn = tile / tiles_m, tm = tile - tn * tiles_m;
  const uint32_t m0 = (uint32_t)tm * CF::kTR, n0 = (uint32_t)tn * CF::kTC;
  const int nq = (int)((p.K + 127) / 128);
  const int n_own = wave < nq ? (nq - wave + W - 1) / W : 0;  // this wavefront's K groups

  // byte offsets of this lane's loads within a K group (32-bit: operands are
  // under 2 GiB)
  const auto row_of = [](uint32_t first, int r, uint32_t rows) {
    const uint32_t row = first + (uint32_t)r;
    return row < rows ? row : rows - 1;
  };
  uint32_t a_off[CF::kALoads], b_off[CF::kBLoads];
#pragma unroll
  for (int i = 0; i < CF::kBLoads; ++i) {
    const uint32_t s = 64 * i + lane, r = s / CF::kChunks;
    b_off[i] = row_of(n0, r, N) * CF::kGB + 16 * rows_chunk<FMT>(r & 15, s - r * CF::kChunks);
  }
#pragma unroll
  for (int i = 0; i < CF::kALoads; ++i) {
    const uint32_t s = 64 * i + lane, r = s / CF::kChunks;
    a_off[i] = row_of(m0, r, M) * CF::kGB + 16 * rows_chunk<FMT>(r & 15, s - r * CF::kChunks);
  }
  const uint32_t sa_off = row_of(m0, lane < CF::kTR ? lane : 0, M) * 4;
  const uint32_t sb_off = row_of(n0, lane < CF::kTC ? lane : 0, N) * 4;

  uint8_t* const ring = smem + wave * (D * CF::kStage);
  const uint32_t ring_lds = (uint32_t)wave_uniform((int)lds_addr(ring));
  const auto issue = [&](int it, int buf) __attribute__((always_inline)) {
    const uint64_t q = (uint64_t)(wave + it * W);
    const uint32_t at = ring_lds + (uint32_t)(buf * CF::kStage);
    const uint8_t* ac = p.a_codes + q * (M * CF::kGB);  // (a K group's bytes fit 32 bits)
    const uint8_t* bc = p.b_codes + q * (N * CF::kGB);
#pragma unroll
    for (int i = 0; i < CF::kBLoads; ++i)
      if (64 * (i + 1) <= CF::kTC * CF::kChunks || lane < 32) lds_dma16_s(bc, b_off[i], at + CF::kBOff + 1024 * i);
#pragma unroll
    for (int i = 0; i < CF::kALoads; ++i)
      if (64 * (i + 1) <= CF::kTR * CF::kChunks || lane < 32) lds_dma16_s(ac, a_off[i], at + CF::kAOff + 1024 * i);
    lds_dma4_s(p.a_scales + q * (M * 4), sa_off, at + CF::kSOff);
    lds_dma4_s(p.b_scales + q * (N * 4), sb_off, at + CF::kSOff + 256);
  };

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  // (every branch here is uniform; the wait that ends a group lets the loads
  // of the D - 1 groups after it stay in flight)
#pragma unroll
  for (int it = 0; it < D - 1; ++it)
    if (it < n_own) issue(it, it);
  // the epilogue's inputs, read beside the sums (older in the count of
  // outstanding loads than any that a group's wait lets fly)
  const int c_bytes = p.c_f32 ? 4 : 2, bias_bytes = p.bias_f32 ? 4 : 2;
  const uint8_t* const res0 = reinterpret_cast<const uint8_t*>(p.residual) + ((int64_t)m0 * p.ldr + n0) * c_bytes;
  const uint8_t* const bias0 = reinterpret_cast<const uint8_t*>(p.bias) + (int64_t)n0 * bias_bytes;
  uint4 bias[CF::kSteps], residual[CF::kSteps];
#pragma unroll
  for (int u = 0; u < CF::kSteps; ++u) {
    const int q = t + 64 * W * u, r = q / CF::kPerRow, c = 4 * (q % CF::kPerRow);
    const bool in = q < CF::kUnits && m0 + r < M && n0 + c < N;
    bias[u] = residual[u] = make_uint4(0u, 0u, 0u, 0u);
    if (in && p.bias != nullptr) bias[u] = load_four(bias0 + c * bias_bytes, p.bias_f32);
    if (in && p.residual != nullptr) residual[u] = load_four(res0 + (r * p.ldr + c) * c_bytes, p.c_f32);
  }
  int buf = 0;
  for (int it = 0; it < n_own; ++it) {
    if (it + D - 1 < n_own) {
      issue(it + D - 1, buf == 0 ? D - 1 : buf - 1);
      wait_vmcnt<CF::kLoads * (D - 1)>();
    } else {
      wait_vmcnt<0>();
    }
    memory_fence();
    const uint8_t* stage = ring + buf * CF::kStage;
    v8i b[NJ];
    int sb[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      b[j] = rows_fragment<FMT>(stage + CF::kBOff + 16 * j * CF::kGB, x, g, row_of(n0, 16 * j + x, N));
      sb[j] = (int)(*reinterpret_cast<const uint32_t*>(stage + CF::kSOff + 256 + 4 * (16 * j + x)) >> (8 * g));
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const v8i a = rows_fragment<FMT>(stage + CF::kAOff + 16 * i * CF::kGB, x, g, row_of(m0, 16 * i + x, M));
      const int sa = (int)(*reinterpret_cast<const uint32_t*>(stage + CF::kSOff + 4 * (16 * i + x)) >> (8 * g));
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b[j], a, acc[i][j], MfmaFmt<FMT>::kCode,
                                                                    MfmaFmt<FMT>::kCode, 0, sb[j], 0, sa);
    }
    wait_lgkmcnt0();  // every read of this buffer done before the next group is loaded into it
    memory_fence();
    buf = buf + 1 == D ? 0 : buf + 1;
  }
  __syncthreads();  // all wavefronts are done with their rings before the partial tiles take the LDS
  float* const red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      *reinterpret_cast<v4f*>(red + (wave * CF::kTR + 16 * i + x) * CF::kPitch + 16 * j + 4 * g) = acc[i][j];
  __syncthreads();

  // Epilogue: four columns of a row per thread and step, rows in order; the
  // eight lanes of a 32-column block are neighbours.
  // A tile's columns lie in one K group of the checkpoint.
  uint8_t* const codes0 = p.saved_codes + code_group(m0, n0, M, 8) + (n0 & 127);
  uint8_t* const scales0 = p.saved_scales + scale_offset(m0, n0 >> 5, M);
  uint8_t* const c0 = reinterpret_cast<uint8_t*>(p.c) + ((int64_t)m0 * p.ldc + n0) * c_bytes;
#pragma unroll
  for (int u = 0; u < CF::kSteps; ++u) {
    const int q = t + 64 * W * u;
    if (q >= CF::kUnits) break;  // (whole wavefronts)
    const int r = q / CF::kPerRow, c = 4 * (q % CF::kPerRow);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const v4f part = *reinterpret_cast<const v4f*>(red + (w * CF::kTR + r) * CF::kPitch + c);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + part[e];
    }
    const bool in = m0 + r < M && n0 + c < N;
    if (p.bias != nullptr) add_four(v, bias[u], p.bias_f32);
    if (p.saved_codes != nullptr) {
      const uint32_t s = scale_byte<kE4M3, kRceil>(max_over8(abs_max(v)));
      float x4[4] = {v[0], v[1], v[2], v[3]};
      uint32_t w[1];
      e4m3_encode(x4, s, w);
      if (in) {
        *reinterpret_cast<uint32_t*>(codes0 + (r * 128 + c)) = w[0];
        if ((lane & 7) == 0) scales0[r * 4 + (c >> 5)] = (uint8_t)s;
      }
    }
    if (p.act == kActGelu) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_value<kActGelu>(v[e]);
    } else if (p.act == kActSilu) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_value<kActSilu>(v[e]);
    }
    if (p.residual != nullptr) add_four(v, residual[u], p.c_f32);
    if (in && p.c != nullptr) {
      uint8_t* const at = c0 + (r * p.ldc + c) * c_bytes;
      if (p.c_f32) *reinterpret_cast<float4*>(at) = make_float4(v[0], v[1], v[2], v[3]);
      else *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  }
  // the pad blocks of the checkpoint's last K group: 0, 32, 64 or 96 columns
  if (p.saved_codes != nullptr && n0 + CF::kTC >= N) {
    const int pad = (int)(((N + 127) & ~127u) - N);
    for (int q = t; q < CF::kTR * pad / 4; q += 64 * W) {
      const int r = q / (pad / 4);
      const uint32_t m = m0 + r, n = N + 4 * (q - r * (pad / 4));
      if (m < M) {
        *reinterpret_cast<uint32_t*>(p.saved_codes + code_group(m, n, M, 8) + (n & 127)) = 0u;
        if ((n & 31) == 0) p.saved_scales[scale_offset(m, n >> 5, M)] = 0;
      }
    }
  }
}

// ------------------------------------------------------------------ launch
int64_t tile_count(const GemmActParams& p, int bm, int bn) { return ((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn); }

// A second product and column sums for the same launch.
struct Second {
  const GemmActParams& q;
  const ColumnSums& sums;
};

template <class F>
hipError_t launch_one_product(F kernel, int threads, int bm, int bn, const GemmActParams& p, hipStream_t stream) {
  const int64_t tiles = tile_count(p, bm, bn);
  if (tiles >= (1ll << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(threads), 0, stream, (Products<1>{{p}, (int)tiles, 0, {}}));
  return hipGetLastError();
}

template <class F>
hipError_t launch_two_products(F kernel, int threads, int bm, int bn, const GemmActParams& p, const Second& more,
                               hipStream_t stream) {
  const int64_t summing = more.sums.out ? (more.sums.cols + threads - 1) / threads : 0;
  const int64_t first = tile_count(p, bm, bn), all = summing + first + tile_count(more.q, bm, bn);
  if (all >= (1ll << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kernel, dim3((unsigned)all), dim3(threads), 0, stream,
                     (Products<2>{{p, more.q}, (int)first, (int)summing, more.sums}));
  return hipGetLastError();
}

// PAIRS: whether the variant is built for two products, or for one and column
// sums (takes_two).
template <int FMT, int BM, int BN, int OCC, bool PAIRS>
hipError_t launch_tiles(const GemmActParams& p, const Second* more, hipStream_t stream) {
  constexpr int kThreads = Cfg<FMT, BM, BN, kDense, kEpiAct, OCC>::kThreads;
  if (!more) return launch_one_product(gemm_act_kernel<FMT, BM, BN, OCC, 1>, kThreads, BM, BN, p, stream);
  if constexpr (PAIRS) return launch_two_products(gemm_act_kernel<FMT, BM, BN, OCC, 2>, kThreads, BM, BN, p, *more, stream);
  return hipErrorInvalidValue;
}

template <int FMT, int MI, int NJ, int W, int D>
hipError_t launch_rows(const GemmActParams& p, const Second* more, hipStream_t stream) {
  if (!more) return launch_one_product(gemm_rows_kernel<FMT, MI, NJ, W, D, 1>, 64 * W, 16 * MI, 16 * NJ, p, stream);
  return launch_two_products(gemm_rows_kernel<FMT, MI, NJ, W, D, 2>, 64 * W, 16 * MI, 16 * NJ, p, *more, stream);
}

// The kernel variants: rows_<tile>, the few-rows kernel, and tile_<size>.
enum Shape {
  kRows16x32, kRows16x32Deep, kRows32x32, kRows32x32Deep, kRows64x32, kRows64x64, kTile128, kTile256x128, kTile256
};

// Whether a launch of the variant can take a second product or column sums.
// 256x128 cannot: of a layer's two products only the weight gradient ever
// takes it (the other has no epilogue inputs), so no pair shares it, and the
// column sums go beside the other product.
constexpr bool takes_two(int shape) { return shape != kTile256x128; }

// Which one (device times in us, measured with one variant after the other on
// the same operands; E2M1 / E2M3 / E4M3):
//  - M <= 32: one row of tiles, so the weights are read once.  Four
//    wavefronts where the column panels fill the chip (1 x 12288 x 4096:
//    6.6 / 8.4 / 9.7, eight 6.9 / 8.5 / 11.0), else eight over K
//    (8 x 4096 x 12288: 7.0 / 8.5 / 10.2, four 7.9 / 8.9 / 10.1).
//  - up to 320 tiles of 64 x 64 (or M <= 64, whose 128-row tiles would be half
//    empty) the few-rows kernel with the largest tile that still gives most
//    compute units one: 512 x 2048 x 2048 64x64 7.7 / 9.3 / 10.8, 64x32
//    6.5 / 8.3 / 11.1, 128x128 7.9 / 9.3 / 14.9; 128 x 4096 x 4096 64x32
//    6.6 / 7.6 / 9.4, 64x64 9.1 / 10.0 / 11.2; 64 x 2048 x 12288 32x32
//    7.9 / 10.1 / 12.7, 64x32 10.8 / 12.5 / 14.6.  With at most three K groups
//    the four wavefronts have too little to share and the 128x128 tiles are
//    taken (768 x 2048 x 224, GELU: 6.5 / 6.8 / 7.1, 64x64 6.2 / 9.5 / 9.7).
//  - beyond, 256x256 tiles or, where those would leave compute units idle,
//    128x128 at two per unit: 8191 x 2048 x 8192 256x256 64 / 78 / 111, 128x128
//    72 / 103 / 138; 1500 x 4096 x 4096 26 / 29 / 45 against 21 / 25 / 30.
//    Their cost per round of the chip goes by area, 128x128 15% more.
//  - over several rounds, with a checkpoint (E2M1: or a residual, or an
//    activation) in the epilogue and short sums, 256x128 at two per unit: one
//    tile's epilogue then runs beside another's products, at the price of a
//    slower main loop.  8192 x 8192 x 2048, GELU and checkpoint 118 / 141 /
//    190, 256x256 136 / 154 / 183; residual 140 / 177 / 201 against 153 / 172 /
//    202; 8192 x 8192 x 4096, GELU and checkpoint 174 / 218 / 317 against
//    181 / 211 / 276; GELU alone 163 / 206 / 298 against 161 / 190 / 256.
//    overlap_k is the longest K that takes them, -1 where none does (an empty
//    sum is no shorter than that).
constexpr int64_t overlap_k(int fmt, bool saved, bool residual, bool act) {
  return fmt == kE2M1 ? (saved || residual ? 4096 : act ? 2048 : -1) : fmt == kE2M3 && saved ? 2048 : -1;
}
int pick_shape(int fmt, const GemmActParams& p) {
  const int64_t cus = cu_count();
  if (p.M <= 16) return tile_count(p, 16, 32) >= cus ? kRows16x32 : kRows16x32Deep;
  if (p.M <= 32) return tile_count(p, 32, 32) >= cus ? kRows32x32 : kRows32x32Deep;
  const int64_t t64 = tile_count(p, 64, 64);
  if (p.M <= 64 || t64 <= cus + cus / 4) {
    if (t64 < cus * 5 / 8) return tile_count(p, 64, 32) >= cus / 2 ? kRows64x32 : kRows32x32Deep;
    if (p.M <= 64 || p.K > 3 * 128) return kRows64x64;
    return kTile128;
  }
  const int64_t t256 = tile_count(p, 256, 256), t128 = tile_count(p, 128, 128);
  const int64_t rest = t128 % (2 * cus);  // a last round of at most one tile per unit takes 2/3 of a full one
  const int64_t cost256 = (t256 + cus - 1) / cus * 65536;
  const int64_t cost128 = (t128 / (2 * cus) * 32768 + (rest == 0 ? 0 : rest <= cus ? 22000 : 32768)) * 115 / 100;
  if (cost256 > cost128) return kTile128;
  const int64_t longest = overlap_k(fmt, p.saved_codes != nullptr, p.residual != nullptr, p.act != kActNone);
  return p.K <= longest && t256 > cus ? kTile256x128 : kTile256;
}

template <int FMT>
hipError_t launch_shape(const GemmActParams& p, const Second* more, int shape, hipStream_t stream) {
  switch (shape) {
    case kRows16x32: return launch_rows<FMT, 1, 2, 4, 3>(p, more, stream);
    case kRows16x32Deep: return launch_rows<FMT, 1, 2, 8, 2>(p, more, stream);
    case kRows32x32: return launch_rows<FMT, 2, 2, 4, 2>(p, more, stream);
    case kRows32x32Deep: return launch_rows<FMT, 2, 2, 8, 2>(p, more, stream);
    case kRows64x32: return launch_rows<FMT, 4, 2, 4, 2>(p, more, stream);
    case kRows64x64: return launch_rows<FMT, 4, 4, 4, 2>(p, more, stream);
    case kTile128: return launch_tiles<FMT, 128, 128, 2, takes_two(kTile128)>(p, more, stream);
    case kTile256x128:
      if constexpr (overlap_k(FMT, true, true, true) >= 0)
        return launch_tiles<FMT, 256, 128, 2, takes_two(kTile256x128)>(p, more, stream);
      return hipErrorInvalidValue;
    case kTile256: return launch_tiles<FMT, 256, 256, 1, takes_two(kTile256)>(p, more, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_fmt(int fmt, const GemmActParams& p, const Second* more, int shape, hipStream_t stream) {
  switch (fmt) {
    case kE2M1: return launch_shape<kE2M1>(p, more, shape, stream);
    case kE2M3: return launch_shape<kE2M3>(p, more, shape, stream);
    case kE4M3: return launch_shape<kE4M3>(p, more, shape, stream);
    default: return hipErrorInvalidValue;
  }
}

// The variant that serves both products, or -1.  Each keeps its own where
// those agree.  Else the smaller tile's product takes the larger's variant,
// which saves a launch and the end of one: its sums are then split over fewer
// wavefronts, or over none, so they have to be short.  200 tokens 2048 -> 768
// in E4M3 take 8.1 us so, 10.7 in two launches; 24 tokens 4096 -> 2048, at the
// limit of 16 groups, 12.9 / 13.4 / 16.5 against 12.2 / 13.1 / 13.6 (E2M1 /
// E2M3 / E4M3); 8 tokens 160 -> 128 2.9 against 5.0.
int pair_shape(int fmt, const GemmActParams& p, const GemmActParams& q) {
  const int a = pick_shape(fmt, p), b = pick_shape(fmt, q);
  if (a == b) return takes_two(a) ? a : -1;
  const int large = a > b ? a : b;
  const int64_t groups = ((a > b ? q : p).K + 127) / 128;
  if (large < kTile128) return groups <= 48 ? large : -1;
  return large == kTile128 && groups <= 16 ? large : -1;
}

}  // namespace

hipError_t launch_gemm_act(const GemmActParams& p, int fmt, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  return launch_fmt(fmt, p, nullptr, pick_shape(fmt, p), stream);
}

// The product with the longer sums goes first, so that the shorter tiles even
// out the end (4095 tokens 2016 -> 2080 in E2M1: 30.4 us, the other way round
// 32.3, in two launches 34.7).
hipError_t launch_gemm_act_pair(const GemmActParams& p, const GemmActParams& q, const ColumnSums& sums, int fmt,
                                hipStream_t stream) {
  if (q.K > p.K) return launch_gemm_act_pair(q, p, sums, fmt, stream);
  const bool both = p.M > 0 && p.N > 0 && q.M > 0 && q.N > 0;
  const int shared = both ? pair_shape(fmt, p, q) : -1;
  const Second more = {q, sums};
  if (shared >= 0) return launch_fmt(fmt, p, &more, shared, stream);
  // a launch each, the column sums beside the first one that can take them
  bool summing = sums.out != nullptr && sums.cols > 0;
  for (const GemmActParams* x : {&p, &q}) {
    if (x->M == 0 || x->N == 0) continue;
    const int shape = pick_shape(fmt, *x);
    const bool carries = summing && takes_two(shape);
    GemmActParams none = *x;
    none.M = 0;
    const Second only_sums = {none, sums};
    const hipError_t e = launch_fmt(fmt, *x, carries ? &only_sums : nullptr, shape, stream);
    if (e != hipSuccess) return e;
    if (carries) summing = false;
  }
  return summing ? launch_colsum_finish(sums.partials, sums.rows, sums.cols, sums.out, 1, stream) : hipSuccess;
}

}  // namespace mx
