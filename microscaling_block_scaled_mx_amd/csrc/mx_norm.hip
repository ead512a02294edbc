// Layer norm: y = (x - mean) rstd gamma + beta with y packed as it is formed,
// and its backward pass with the reduction of the weights' gradients.
//
// A row is held in registers, eight values a lane and step, by a wavefront
// (C up to 2048) or a workgroup, so x is read once and the variance is taken
// from the differences to the mean (two sums; one pass over the data).  Both
// kernels are bound by HBM.  Workgroups walk over rows with a fixed stride:
// the weights stay in registers, the next row's loads are in flight while the
// current one is reduced, and the backward pass keeps its share of dgamma and
// dbeta in registers until its rows are done.  Sums are binary32.
#include "mx_lanes.h"
#include "mx_train.h"

namespace mx {

namespace {

// Rows of the thread groups: T threads a row, NV steps of 8 values each, WG
// threads a workgroup (WG / T rows side by side).
template <int T, int NV, int WG>
struct RowCfg {
  static constexpr int kRows = WG / T, kWaves = WG / 64, kPer = T / 64;  // wavefronts a row
  static_assert(T % 64 == 0 && WG % T == 0, "whole wavefronts");
  static constexpr int kMaxC = T * NV * 8;
};

// Sums of N values over the T threads of a row, in all of them; `red` is one
// of two LDS arrays used in turn, so that one barrier is enough.
template <class CF, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*red)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = wave_sum(v[n]);
  if constexpr (CF::kPer > 1) {
    const int wave = threadIdx.x >> 6, first = wave / CF::kPer * CF::kPer;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) red[wave][n] = v[n];
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = red[first][n];
#pragma unroll
    for (int w = 1; w < CF::kPer; ++w) {
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = v[n] + red[first + w][n];
    }
  }
}

// ------------------------------------------------------------------ forward
template <int X32, int T, int NV, int WG>
__global__ __launch_bounds__(WG) void norm_fwd_kernel(NormFwdParams p) {
  using CF = RowCfg<T, NV, WG>;
  __shared__ float red[2][CF::kWaves][1];
  const int t = threadIdx.x, tr = t % T;
  const int64_t step = (int64_t)gridDim.x * CF::kRows;
  const int64_t packed_c = (p.C + 127) & ~(int64_t)127;
  Lane8<X32> next[NV];
  const auto load = [&](int64_t r) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = 8 * (int64_t)(tr + T * i);
      next[i] = r < p.M && c < p.C ? lane8_load<X32>(p.x, r * p.ldx + c) : lane8_zero<X32>();
    }
  };
  int64_t r = (int64_t)blockIdx.x * CF::kRows + t / T;
  load(r);
  // (the weights as they lie in memory would take half the registers in bf16,
  // but a branch on their type for every row)
  float gamma[NV][8], beta[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = 8 * (int64_t)(tr + T * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      gamma[i][e] = 1.0f;
      beta[i][e] = 0.0f;
    }
    if (c < p.C) {
      if (p.gamma != nullptr) lane8_read(p.gamma, c, p.w_f32, gamma[i]);
      if (p.beta != nullptr) lane8_read(p.beta, c, p.w_f32, beta[i]);
    }
  }
  // every thread group of the workgroup makes the same number of turns
  for (int64_t r0 = (int64_t)blockIdx.x * CF::kRows; r0 < p.M; r0 += step, r += step) {
    float v[NV][8], sum[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      lane8_values<X32>(next[i], v[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] = sum[0] + v[i][e];
    }
    load(r + step);
    row_sums<CF>(sum, red[0]);
    const float mean = sum[0] * p.inv_c;
    float sq[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (8 * (int64_t)(tr + T * i) < p.C) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[i][e] = v[i][e] - mean;
          sq[0] = __builtin_fmaf(v[i][e], v[i][e], sq[0]);
        }
      }
    }
    row_sums<CF>(sq, red[1]);
    const float rstd = 1.0f / __builtin_sqrtf(__builtin_fmaf(sq[0], p.inv_c, p.eps));
    const bool in_m = r < p.M;
    if (in_m && tr == 0) {
      if (p.mean != nullptr) p.mean[r] = mean;
      if (p.rstd != nullptr) p.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = 8 * (int64_t)(tr + T * i);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = __builtin_fmaf(v[i][e] * rstd, gamma[i][e], beta[i][e]);
      if (in_m && c < p.C && p.y != nullptr) lane8_store(p.y, r * p.ldy + c, p.y_f32, v[i]);
      if (p.row_codes != nullptr || p.saved_codes != nullptr) {
        // the packs take y rounded to bf16; columns past C are pad blocks: zeros
        const bool in = in_m && c < packed_c;
        const int64_t group = (c >> 7) * p.M + r;
        float u[8], w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = w[e] = c < p.C ? round_bf16(v[i][e]) : 0.0f;
        uint8_t* const scales = p.row_scales + 4 * group;
        if (p.row_codes == nullptr) {
        } else if (p.fmt == kE2M1) {
          lane8_quantize<kE2M1, kFloor, 0>(u, p.row_codes + 64 * group, scales, r, in);
        } else if (p.fmt == kE2M3 && p.had) {
          lane8_quantize<kE2M3, kFloor, 1>(u, p.row_codes + 96 * group, scales, r, in);
        } else if (p.fmt == kE2M3) {
          lane8_quantize<kE2M3, kFloor, 0>(u, p.row_codes + 96 * group, scales, r, in);
        } else if (p.mode == kRceil) {
          lane8_quantize<kE4M3, kRceil, 0>(u, p.row_codes + 128 * group, scales, r, in);
        } else {
          lane8_quantize<kE4M3, kFloor, 0>(u, p.row_codes + 128 * group, scales, r, in);
        }
        if (p.saved_codes != nullptr)
          lane8_quantize<kE4M3, kRceil, 0>(w, p.saved_codes + 128 * group, p.saved_scales + 4 * group, r, in);
      }
    }
  }
}

// ------------------------------------------------------------------ backward
// With h = (x - mean) rstd and g = dy gamma: dx = rstd (g - mean(g) - h mean(g h)).
template <int X32, int D32, int T, int NV, int WG>
__global__ __launch_bounds__(WG) void norm_bwd_kernel(NormBwdParams p) {
  using CF = RowCfg<T, NV, WG>;
  // 1024 threads have 128 registers each: no room for the next row and gamma
  constexpr bool kAhead = WG < 1024;
  __shared__ float red[2][CF::kWaves][2];
  __shared__ float part[CF::kRows > 1 ? 2 * CF::kMaxC : 1];
  const int t = threadIdx.x, tr = t % T;
  const int64_t step = (int64_t)gridDim.x * CF::kRows;
  Lane8<X32> next_x[NV];
  Lane8<D32> next_d[NV];
  float next_mean = 0.0f, next_rstd = 0.0f;
  const auto load = [&](int64_t r) {
    const bool in_m = r < p.M;
    next_mean = in_m ? p.mean[r] : 0.0f;
    next_rstd = in_m ? p.rstd[r] : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = 8 * (int64_t)(tr + T * i);
      const bool in = in_m && c < p.C;
      next_x[i] = in ? lane8_load<X32>(p.x, r * p.ldx + c) : lane8_zero<X32>();
      next_d[i] = in ? lane8_load<D32>(p.dy, r * p.lddy + c) : lane8_zero<D32>();
    }
  };
  int64_t r = (int64_t)blockIdx.x * CF::kRows + t / T;
  if constexpr (kAhead) load(r);
  float gamma[kAhead ? NV : 1][8], dgamma[NV][8], dbeta[NV][8];
  const auto load_gamma = [&](int i, float (&w)[8]) {
    const int64_t c = 8 * (int64_t)(tr + T * i);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    if (c < p.C && p.gamma != nullptr) lane8_read(p.gamma, c, p.w_f32, w);
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (kAhead) load_gamma(i, gamma[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dgamma[i][e] = dbeta[i][e] = 0.0f;
  }
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * CF::kRows; r0 < p.M; r0 += step, r += step, turn ^= 1) {
    if constexpr (!kAhead) load(r);
    float h[NV][8], g[NV][8], sum[2] = {0.0f, 0.0f};
    const float mean = next_mean, rstd = next_rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&w)[8] = gamma[kAhead ? i : 0];
      if constexpr (!kAhead) load_gamma(i, w);
      lane8_values<X32>(next_x[i], h[i]);
      lane8_values<D32>(next_d[i], g[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // (rows and columns past the end: dy = 0, so only h might not be 0)
        h[i][e] = (h[i][e] - mean) * rstd;
        dgamma[i][e] = __builtin_fmaf(g[i][e], h[i][e], dgamma[i][e]);
        dbeta[i][e] = dbeta[i][e] + g[i][e];
        g[i][e] = g[i][e] * w[e];
        sum[0] = sum[0] + g[i][e];
        sum[1] = __builtin_fmaf(g[i][e], h[i][e], sum[1]);
      }
    }
    if constexpr (kAhead) load(r + step);
    if (p.dx == nullptr) continue;  // (uniform)
    row_sums<CF>(sum, red[turn]);
    const float m1 = sum[0] * p.inv_c, m2 = sum[1] * p.inv_c;
    if (r < p.M) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int64_t c = 8 * (int64_t)(tr + T * i);
        if (c < p.C) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = 0.0f;
          if (p.residual != nullptr) lane8_read(p.residual, r * p.ldr + c, p.dx_f32, o);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __builtin_fmaf(rstd, __builtin_fmaf(-h[i][e], m2, g[i][e] - m1), o[e]);
          lane8_store(p.dx, r * p.lddx + c, p.dx_f32, o);
        }
      }
    }
  }
  if (p.partials == nullptr) return;  // (uniform)
  // the workgroup's partial sums: its thread groups' in order
  float* const out = p.partials + (int64_t)blockIdx.x * 2 * p.C;
  if constexpr (CF::kRows > 1) {
    for (int k = 0; k < CF::kRows; ++k) {
      if (t / T == k) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = 8 * (tr + T * i);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            part[c + e] = k == 0 ? dgamma[i][e] : part[c + e] + dgamma[i][e];
            part[CF::kMaxC + c + e] = k == 0 ? dbeta[i][e] : part[CF::kMaxC + c + e] + dbeta[i][e];
          }
        }
      }
      __syncthreads();
    }
    for (int c = 4 * t; c < p.C; c += 4 * WG) {
      *reinterpret_cast<float4*>(out + c) = *reinterpret_cast<const float4*>(part + c);
      *reinterpret_cast<float4*>(out + p.C + c) = *reinterpret_cast<const float4*>(part + CF::kMaxC + c);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = 8 * (int64_t)(tr + T * i);
      if (c < p.C) {
        lane8_store(out, c, 1, dgamma[i]);
        lane8_store(out, p.C + c, 1, dbeta[i]);
      }
    }
  }
}

// dgamma and dbeta from the partials [rows][2][C]: 64 columns a workgroup, its
// four wavefronts taking every fourth row, their sums in wavefront order.
__global__ __launch_bounds__(256) void norm_weights_kernel(const float* __restrict__ partials, int64_t rows, int64_t C,
                                                           float* __restrict__ dgamma, float* __restrict__ dbeta,
                                                           int accumulate) {
  __shared__ float red[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;  // of 2 C
  float sum = 0.0f;
  if (c < 2 * C) {
#pragma unroll 8
    for (int64_t r = wave; r < rows; r += 4) sum = sum + partials[r * 2 * C + c];
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || c >= 2 * C) return;
  const float total = ((red[0][lane] + red[1][lane]) + red[2][lane]) + red[3][lane];
  float* const out = c < C ? dgamma : dbeta;
  const int64_t at = c < C ? c : c - C;
  if (out != nullptr) out[at] = accumulate ? out[at] + total : total;
}

// ------------------------------------------------------------------ launch
template <int X32, int T, int NV, int WG>
hipError_t fwd(const NormFwdParams& p, hipStream_t stream) {
  const int64_t rows = WG / T, wanted = (p.M + rows - 1) / rows, most = (int64_t)cu_count() * (2048 / WG);
  hipLaunchKernelGGL((norm_fwd_kernel<X32, T, NV, WG>), dim3((unsigned)(wanted < most ? wanted : most)), dim3(WG), 0,
                     stream, p);
  return hipGetLastError();
}

template <int X32>
hipError_t fwd_of(const NormFwdParams& p, hipStream_t stream) {
  if (p.C <= 512) return fwd<X32, 64, 1, 256>(p, stream);
  if (p.C <= 1024) return fwd<X32, 64, 2, 256>(p, stream);
  if (p.C <= 2048) return fwd<X32, 128, 2, 256>(p, stream);
  if (p.C <= 4096) return fwd<X32, 256, 2, 256>(p, stream);
  if (p.C <= 8192) return fwd<X32, 512, 2, 512>(p, stream);
  return fwd<X32, 1024, 2, 1024>(p, stream);
}

constexpr int64_t kMostPartials = 256;

int64_t bwd_rows_side_by_side(int64_t C) { return C <= 1024 ? 8 : C <= 2048 ? 4 : C <= 4096 ? 2 : 1; }

template <int X32, int D32, int T, int NV, int WG>
hipError_t bwd(const NormBwdParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((norm_bwd_kernel<X32, D32, T, NV, WG>), dim3((unsigned)norm_partial_rows(p.M, p.C)), dim3(WG), 0,
                     stream, p);
  return hipGetLastError();
}

template <int X32, int D32>
hipError_t bwd_of(const NormBwdParams& p, hipStream_t stream) {
  if (p.C <= 512) return bwd<X32, D32, 64, 1, 512>(p, stream);
  if (p.C <= 1024) return bwd<X32, D32, 64, 2, 512>(p, stream);
  if (p.C <= 2048) return bwd<X32, D32, 128, 2, 512>(p, stream);
  if (p.C <= 4096) return bwd<X32, D32, 256, 2, 512>(p, stream);
  if (p.C <= 8192) return bwd<X32, D32, 512, 2, 512>(p, stream);
  return bwd<X32, D32, 1024, 2, 1024>(p, stream);
}

}  // namespace

hipError_t launch_norm_fwd(const NormFwdParams& p, int x_f32, hipStream_t stream) {
  return x_f32 ? fwd_of<1>(p, stream) : fwd_of<0>(p, stream);
}

int64_t norm_partial_rows(int64_t M, int64_t C) {
  const int64_t side = bwd_rows_side_by_side(C), wanted = (M + side - 1) / side;
  return wanted < kMostPartials ? wanted : kMostPartials;
}

hipError_t launch_norm_bwd(const NormBwdParams& p, int x_f32, int dy_f32, hipStream_t stream) {
  if (x_f32) return dy_f32 ? bwd_of<1, 1>(p, stream) : bwd_of<1, 0>(p, stream);
  return dy_f32 ? bwd_of<0, 1>(p, stream) : bwd_of<0, 0>(p, stream);
}

hipError_t launch_norm_weights(const float* partials, int64_t rows, int64_t C, float* dgamma, float* dbeta,
                               int accumulate, hipStream_t stream) {
  hipLaunchKernelGGL(norm_weights_kernel, dim3((unsigned)((2 * C + 63) / 64)), dim3(256), 0, stream, partials, rows, C,
                     dgamma, dbeta, accumulate);
  return hipGetLastError();
}

}  // namespace mx
