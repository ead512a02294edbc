// mx_gemm_act: C = act(A . B^T + bias) + residual on packed operands, with
// the 8-bit checkpoint of the pre-activation from the same epilogue, for any
// number of rows.
//
// Two kernels.  Many rows: the output tile of mx_gemm_tile.h (operands
// through LDS, 32x32x64 matrix instructions) with the epilogue kEpiAct, bound
// by the matrix cores.  Few rows, down to one: gemm_rows_kernel below, which
// reads its operands straight into registers, bound by the one pass over the
// weights; its wavefronts split K inside the workgroup, so that a short
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
template <int FMT, int BM, int BN, int OCC>
__global__ __launch_bounds__(tile_threads(BM, BN, kEpiAct), OCC) void gemm_act_kernel(GemmActParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[Cfg<FMT, BM, BN, kDense, kEpiAct, OCC>::kSmem];
  gemm_tile<FMT, BM, BN, kDense, kEpiAct, OCC>(p, blockIdx.x, 0, 0, smem);
}

// ------------------------------------------------------------------ few rows
// v_mfma_scale_f32_16x16x128_f8f6f4 takes one whole K group: lane l holds row
// l % 16, and of the group's 128 elements (g = l / 16) E2M1 / E2M3 the 32
// of block g, E4M3 [16g, 16g+16) and [64+16g, 64+16g+16); its scale operand is
// the byte of block g (layouts measured).  With B as the first operand, a lane
// ends with C row l % 16 and the four columns 4g .. 4g+3.
template <int FMT>
__device__ __forceinline__ v8i rows_operand(const uint8_t* at, int row, int g) {
  if constexpr (FMT == kE2M1) {
    const v4i a = *reinterpret_cast<const v4i*>(at + 16 * g);
    return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  } else if constexpr (FMT == kE2M3) {
    const v4i a = *reinterpret_cast<const v4i*>(at + 16 * g);
    const v2i h = *reinterpret_cast<const v2i*>(at + 64 + 8 * (g ^ ((row >> 4) & 1)));
    const v4i h4 = __builtin_shufflevector(h, h, 0, 1, -1, -1);
    return __builtin_shufflevector(a, h4, 0, 1, 2, 3, 4, 5, -1, -1);
  } else {
    const v4i a = *reinterpret_cast<const v4i*>(at + 16 * g);
    const v4i b = *reinterpret_cast<const v4i*>(at + 64 + 16 * g);
    return v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
}

// W wavefronts compute a 16 MI x 16 NJ tile of C: wavefront w the K groups
// w, w + W, ..., U of them in flight.  The partial tiles meet in LDS and are
// summed in wavefront order, so the result does not depend on timing.  Rows
// past the operands' ends are loaded as the last row and never stored.
template <int FMT, int MI, int NJ, int W>
struct RowsCfg {
  static constexpr int kTR = 16 * MI, kTC = 16 * NJ;
  static constexpr int kPitch = kTC + 4;  // floats: the 16 rows of a write start in different banks
  static constexpr int kRegs = (FMT == kE4M3 ? 8 : FMT == kE2M3 ? 6 : 4) + 1;
  // K groups in flight per wavefront: as many as about 96 registers hold
  static constexpr int kFit = 96 / (kRegs * (MI + NJ));
  static constexpr int kU = kFit >= 8 ? 8 : kFit >= 4 ? 4 : kFit >= 2 ? 2 : 1;
};

template <int FMT, int MI, int NJ, int W>
__global__ __launch_bounds__(64 * W) void gemm_rows_kernel(GemmActParams p) {
  using CF = RowsCfg<FMT, MI, NJ, W>;
  constexpr int kGB = 16 * FmtTraits<FMT>::kBits;  // code bytes of a row in one K group
  constexpr int U = CF::kU;
  __shared__ __attribute__((aligned(16))) float red[W][CF::kTR][CF::kPitch];
  const int t = threadIdx.x, lane = t & 63, wave = wave_uniform(t >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int tiles_m = (int)((p.M + CF::kTR - 1) / CF::kTR);
  const int tn = blockIdx.x / tiles_m, tm = blockIdx.x - tn * tiles_m;
  const int64_t m0 = (int64_t)tm * CF::kTR, n0 = (int64_t)tn * CF::kTC;
  const int nq = (int)((p.K + 127) / 128);

  // operand rows of this lane (32-bit byte offsets: operands are under 2 GiB)
  uint32_t a_row[MI], b_row[NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int64_t m = m0 + 16 * i + r16;
    a_row[i] = (uint32_t)(m < p.M ? m : p.M - 1);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t n = n0 + 16 * j + r16;
    b_row[j] = (uint32_t)(n < p.N ? n : p.N - 1);
  }

  v4f acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t a_rows = (uint32_t)p.M, b_rows = (uint32_t)p.N;
  for (int q0 = wave; q0 < nq; q0 += W * U) {
    v8i a[U][MI], b[U][NJ];
    uint32_t sa[U][MI], sb[U][NJ];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a group past the end loads the last one again and is not multiplied
      const uint32_t q = (uint32_t)(q0 + W * u < nq ? q0 + W * u : nq - 1);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        b[u][j] = rows_operand<FMT>(p.b_codes + (uint64_t)q * b_rows * kGB + b_row[j] * (uint32_t)kGB, b_row[j], g);
        sb[u][j] = *reinterpret_cast<const uint32_t*>(p.b_scales + (uint64_t)q * b_rows * 4 + b_row[j] * 4u);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        a[u][i] = rows_operand<FMT>(p.a_codes + (uint64_t)q * a_rows * kGB + a_row[i] * (uint32_t)kGB, a_row[i], g);
        sa[u][i] = *reinterpret_cast<const uint32_t*>(p.a_scales + (uint64_t)q * a_rows * 4 + a_row[i] * 4u);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (q0 + W * u < nq) {  // uniform
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                b[u][j], a[u][i], acc[i][j], MfmaFmt<FMT>::kCode, MfmaFmt<FMT>::kCode, 0, (int)(sb[u][j] >> (8 * g)),
                0, (int)(sa[u][i] >> (8 * g)));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) *reinterpret_cast<v4f*>(&red[wave][16 * i + r16][16 * j + 4 * g]) = acc[i][j];
  __syncthreads();

  // Epilogue: four columns of a row per thread and step, rows in order; the
  // eight lanes of a 32-column block are neighbours.
  constexpr int kUnits = CF::kTR * CF::kTC / 4, kPerRow = CF::kTC / 4;
  static_assert(kUnits % 64 == 0, "whole wavefronts");
  for (int q = t; q < kUnits; q += 64 * W) {
    const int r = q / kPerRow, c = 4 * (q % kPerRow);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const v4f x = *reinterpret_cast<const v4f*>(&red[w][r][c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] + x[e];
    }
    const int64_t m = m0 + r, n = n0 + c;
    const bool in = m < p.M && n < p.N;
    if (in && p.bias != nullptr) {
      if (p.bias_f32) {
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.bias) + n);
        v[0] = v[0] + x.x;
        v[1] = v[1] + x.y;
        v[2] = v[2] + x.z;
        v[3] = v[3] + x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.bias) + n);
        v[0] = v[0] + bf16_lo(x.x);
        v[1] = v[1] + bf16_hi(x.x);
        v[2] = v[2] + bf16_lo(x.y);
        v[3] = v[3] + bf16_hi(x.y);
      }
    }
    if constexpr (NJ >= 2) {
      if (p.saved_codes != nullptr) {
        const uint32_t s = scale_byte<kE4M3, kRceil>(max_over8(abs_max4(v)));
        const uint32_t w = e4m3_encode4(v, s);
        if (in) {
          *reinterpret_cast<uint32_t*>(p.saved_codes + code_group(m, n, p.M, 8) + (n & 127)) = w;
          if ((lane & 7) == 0) p.saved_scales[scale_offset(m, n >> 5, p.M)] = (uint8_t)s;
        }
      }
    }
    if (!in || p.c == nullptr) continue;
    if (p.act == kActGelu) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_value<kActGelu>(v[e]);
    } else if (p.act == kActSilu) {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = act_value<kActSilu>(v[e]);
    }
    if (p.c_f32) {
      if (p.residual != nullptr) {
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.residual) + m * p.ldr + n);
        v[0] = v[0] + x.x;
        v[1] = v[1] + x.y;
        v[2] = v[2] + x.z;
        v[3] = v[3] + x.w;
      }
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.c) + m * p.ldc + n) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      if (p.residual != nullptr) {
        const uint2 x =
            *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.residual) + m * p.ldr + n);
        v[0] = v[0] + bf16_lo(x.x);
        v[1] = v[1] + bf16_hi(x.x);
        v[2] = v[2] + bf16_lo(x.y);
        v[3] = v[3] + bf16_hi(x.y);
      }
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.c) + m * p.ldc + n) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  }
  if constexpr (NJ >= 2) {
    // the pad blocks of the checkpoint's last K group
    if (p.saved_codes != nullptr && n0 + CF::kTC >= p.N) {
      const int pad = (int)(((p.N + 127) & ~(int64_t)127) - p.N);  // 0, 32, 64 or 96 columns
      for (int q = t; q < CF::kTR * pad / 4; q += 64 * W) {
        const int r = q / (pad / 4);
        const int64_t m = m0 + r, n = p.N + 4 * (q - r * (pad / 4));
        if (m < p.M) {
          *reinterpret_cast<uint32_t*>(p.saved_codes + code_group(m, n, p.M, 8) + (n & 127)) = 0u;
          if ((n & 31) == 0) p.saved_scales[scale_offset(m, n >> 5, p.M)] = 0;
        }
      }
    }
  }
}

// ------------------------------------------------------------------ launch
template <int FMT, int BM, int BN, int OCC>
hipError_t launch_tiles(const GemmActParams& p, hipStream_t stream) {
  const int64_t tiles = ((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
  if (tiles >= (1ll << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_act_kernel<FMT, BM, BN, OCC>), dim3((unsigned)tiles),
                     dim3(Cfg<FMT, BM, BN, kDense, kEpiAct, OCC>::kThreads), 0, stream, p);
  return hipGetLastError();
}

template <int FMT, int MI, int NJ, int W>
hipError_t launch_rows(const GemmActParams& p, hipStream_t stream) {
  using CF = RowsCfg<FMT, MI, NJ, W>;
  const int64_t tiles = ((p.M + CF::kTR - 1) / CF::kTR) * ((p.N + CF::kTC - 1) / CF::kTC);
  if (tiles >= (1ll << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((gemm_rows_kernel<FMT, MI, NJ, W>), dim3((unsigned)tiles), dim3(64 * W), 0, stream, p);
  return hipGetLastError();
}

// Kernel variants.
enum Shape { kRows1x1, kRows1x2, kRows2x2, kRows4x2, kRows4x4, kTile128x256, kTile256x128, kTile256x256, kNumShapes };

int pick_shape(const GemmActParams& p) {
  if (p.M <= 16) return p.saved_codes == nullptr ? kRows1x1 : kRows1x2;
  if (p.M <= 32) return kRows2x2;
  if (p.M <= 64) return kRows4x2;
  const int64_t cus = cu_count();
  const int64_t t256 = ((p.M + 255) / 256) * ((p.N + 255) / 256);
  if (t256 >= cus) return kTile256x256;
  const int64_t t128 = ((p.M + 127) / 128) * ((p.N + 255) / 256);
  if (t128 >= cus) return kTile128x256;
  return kRows4x4;
}

template <int FMT>
hipError_t launch_shape(const GemmActParams& p, int shape, hipStream_t stream) {
  switch (shape) {
    case kRows1x1: return launch_rows<FMT, 1, 1, 8>(p, stream);
    case kRows1x2: return launch_rows<FMT, 1, 2, 8>(p, stream);
    case kRows2x2: return launch_rows<FMT, 2, 2, 8>(p, stream);
    case kRows4x2: return launch_rows<FMT, 4, 2, 8>(p, stream);
    case kRows4x4: return launch_rows<FMT, 4, 4, 4>(p, stream);
    case kTile128x256: return launch_tiles<FMT, 128, 256, 2>(p, stream);
    case kTile256x128: return launch_tiles<FMT, 256, 128, 2>(p, stream);
    case kTile256x256: return launch_tiles<FMT, 256, 256, 1>(p, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_gemm_act_shape(const GemmActParams& p, int fmt, int shape, hipStream_t stream) {
  if (p.M == 0 || p.N == 0) return hipSuccess;
  if (shape < 0) shape = pick_shape(p);
  switch (fmt) {
    case kE2M1: return launch_shape<kE2M1>(p, shape, stream);
    case kE2M3: return launch_shape<kE2M3>(p, shape, stream);
    case kE4M3: return launch_shape<kE4M3>(p, shape, stream);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_gemm_act(const GemmActParams& p, int fmt, hipStream_t stream) {
  return launch_gemm_act_shape(p, fmt, -1, stream);
}

}  // namespace mx
