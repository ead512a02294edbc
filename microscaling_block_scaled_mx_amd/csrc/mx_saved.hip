// Activation checkpoints in 8 bits and the packs that read them.
//
// A checkpoint of x [R][C] is its rowwise MXFP8 operand: E4M3 codes with one
// E8M0 exponent per 32 columns (RCEIL, so nothing saturates), in the packed
// layout of [R] x K=C -- 8.25 bits a value, and itself an operand of an MXFP8
// GEMM.  Three kernels, each one pass over its data:
//   checkpoint_save_kernel   bf16 / binary32 -> checkpoint,
//   checkpoint_load_kernel   checkpoint -> bf16 / binary32,
//   quantize_saved_kernel    checkpoint (and a gradient) -> the operands of
//                            the backward GEMMs, rowwise and columnwise, with
//                            the activation or its slope in between.
#include "mx_act.h"
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_linear.h"

namespace mx {

namespace {

// Eight values of a row at column c: one 16-byte load of bf16, two of binary32.
template <int F32>
struct Eight {
  uint4 w[F32 ? 2 : 1];
};
template <int F32>
__device__ __forceinline__ Eight<F32> load8(const void* base, int64_t at) {
  Eight<F32> q;
  if constexpr (F32) {
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(base) + at);
    q.w[0] = src[0];
    q.w[1] = src[1];
  } else {
    q.w[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + at);
  }
  return q;
}
template <int F32>
__device__ __forceinline__ void values8(const Eight<F32>& q, float (&v)[8]) {
  if constexpr (F32) {
    const uint32_t a[4] = {q.w[0].x, q.w[0].y, q.w[0].z, q.w[0].w}, b[4] = {q.w[1].x, q.w[1].y, q.w[1].z, q.w[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    const uint32_t a[4] = {q.w[0].x, q.w[0].y, q.w[0].z, q.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(a[i]);
      v[2 * i + 1] = bf16_hi(a[i]);
    }
  }
}

// ------------------------------------------------------------------ save and load
// A workgroup takes 64 rows of one 128-column K group: 16 lanes a row, eight
// values a lane, four rows a thread.  Reads are 256-byte (bf16) row segments,
// writes one contiguous run (the layout puts a K group's rows back to back).
// Bound by HBM: 8191 x 12288 in bf16, 305 MB each way, saves in 57 us (5.3 TB/s;
// median 64) and loads in 55 (5.5), repeated over the same buffers.
// One row of 4096 takes 2.8 and 2.1 us.
constexpr int kCkptRows = 64, kCkptSteps = 4;

template <int F32>
__global__ __launch_bounds__(256) void checkpoint_save_kernel(const void* __restrict__ x, int64_t R, int64_t C,
                                                              int64_t ldx, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales, int groups) {
  const int t = threadIdx.x, ch = t & 15, row = t >> 4;
  const int64_t q = blockIdx.x % groups, r0 = (int64_t)(blockIdx.x / groups) * kCkptRows + row;
  const int64_t c = q * 128 + ch * 8;
  Eight<F32> in[kCkptSteps];
#pragma unroll
  for (int i = 0; i < kCkptSteps; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < R && c < C) in[i] = load8<F32>(x, r * ldx + c);
    else in[i] = Eight<F32>{};  // pad blocks: zero codes
  }
#pragma unroll
  for (int i = 0; i < kCkptSteps; ++i) {
    const int64_t r = r0 + 16 * i;
    float v[8];
    values8<F32>(in[i], v);
    // an all-zero block gets scale byte 0, and so does a pad block
    const uint32_t s = scale_byte<kE4M3, kRceil>(max_over4(abs_max(v)));
    uint32_t w[2];
    e4m3_encode(v, s, w);
    // the row's scale dword: byte b from the lanes of block b = ch / 4
    uint32_t d = s << (8 * (ch >> 2));
    d |= dpp_move<kDppRor8>(d);
    d |= dpp_move<kDppRor4>(d);
    if (r < R) {
      *reinterpret_cast<uint2*>(codes + (q * R + r) * 128 + ch * 8) = make_uint2(w[0], w[1]);
      if (ch == 0) *reinterpret_cast<uint32_t*>(scales + (q * R + r) * 4) = d;
    }
  }
}

template <int F32>
__global__ __launch_bounds__(256) void checkpoint_load_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t R,
                                                              int64_t C, void* __restrict__ y, int64_t ldy,
                                                              int groups) {
  const int t = threadIdx.x, ch = t & 15, row = t >> 4;
  const int64_t q = blockIdx.x % groups, r0 = (int64_t)(blockIdx.x / groups) * kCkptRows + row;
  const int64_t c = q * 128 + ch * 8;
  uint2 w[kCkptSteps];
  uint32_t s[kCkptSteps];
#pragma unroll
  for (int i = 0; i < kCkptSteps; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < R && c < C) {
      w[i] = *reinterpret_cast<const uint2*>(codes + (q * R + r) * 128 + ch * 8);
      s[i] = *reinterpret_cast<const uint32_t*>(scales + (q * R + r) * 4);
    }
  }
#pragma unroll
  for (int i = 0; i < kCkptSteps; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < R && c < C) {
      const float sc = e8m0_value((s[i] >> (8 * (ch >> 2))) & 255u);
      float lo[4], hi[4];
      e4m3_decode4(w[i].x, sc, lo);
      e4m3_decode4(w[i].y, sc, hi);
      if constexpr (F32) {
        float4* dst = reinterpret_cast<float4*>(reinterpret_cast<float*>(y) + r * ldy + c);
        dst[0] = make_float4(lo[0], lo[1], lo[2], lo[3]);
        dst[1] = make_float4(hi[0], hi[1], hi[2], hi[3]);
      } else {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(y) + r * ldy + c) =
            make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(hi[0], hi[1]),
                       pack_bf16x2(hi[2], hi[3]));
      }
    }
  }
}

// ------------------------------------------------------------------ packs from a checkpoint
// One 512-thread workgroup turns a 128 x 128 tile of v into rows' and columns'
// blocks: inputs -> v in registers (its column sums are taken there, in
// binary32) -> bf16 in LDS -> one quantization pass per axis.  Tile geometry
// as in the bf16 packer: row pitch 272 bytes, every 32-row block shifted by a
// further 32 so that a column pass's four blocks fall in different banks.
// Bound by vector issue where there is an activation and a rotation: both
// packs of 8192 x 8192 (GELU slope) and 8192 x 2048 in E2M3 take 84 us for
// 307 MB, 3.7 TB/s.  512 threads make one block a thread and pass: the pack of
// 8192 x 8192 alone, timed by itself, went from 84 to 80 us with them.
constexpr int kTile = 128, kPitch = kTile * 2 + 16, kBlockSkew = 32;
constexpr int kTileBytes = kTile * kPitch + 3 * kBlockSkew;
constexpr int kSteps = 4;  // 32-row steps of a tile
__device__ __forceinline__ int lds_row_at(int row) { return row * kPitch + (row >> 5) * kBlockSkew; }

// Sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 (a fixed order).
__device__ __forceinline__ float sum_over_rows4(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t b = __float_as_uint(v);
  const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t h = __float_as_uint(__uint_as_float(x[0]) + __uint_as_float(x[1]));
  const auto y = __builtin_amdgcn_permlane32_swap(h, h, false, false);
  return __uint_as_float(y[0]) + __uint_as_float(y[1]);
#else
  return v;
#endif
}

// STEPS 32-row steps of a tile from step i0 on: every load in flight, then v,
// its column sums, and bf16 in LDS.  HASX: v = x act'(saved) (ACT none: v = x,
// no checkpoint), else v = act(saved).
template <int ACT, int HASX, int STEPS>
__device__ __forceinline__ void form_steps(const SavedPackParams& p, int64_t bx, int64_t by, int i0, uint8_t* tile,
                                           float (&sum)[8]) {
  constexpr bool kSaved = !HASX || ACT != kActNone;
  const int t = threadIdx.x, ch = t & 15, row_t = t >> 4;
  const int64_t r0 = by * kTile + 32 * i0, c = bx * kTile + ch * 8;
  uint8_t* const lds = tile + i0 * (32 * kPitch + kBlockSkew) + row_t * kPitch + ch * 16;
  uint4 x[STEPS];
  uint2 w[STEPS];
  uint32_t s[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t r = r0 + row_t + 32 * i;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    w[i] = make_uint2(0u, 0u);
    s[i] = 0u;
    if (r < p.R && c < p.C) {
      if constexpr (HASX) x[i] = *reinterpret_cast<const uint4*>(p.x + r * p.ldx + c);
      if constexpr (kSaved) {
        w[i] = *reinterpret_cast<const uint2*>(p.saved_codes + (bx * p.R + r) * 128 + ch * 8);
        s[i] = *reinterpret_cast<const uint32_t*>(p.saved_scales + (bx * p.R + r) * 4);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    float v[8];
    if constexpr (kSaved) {
      const float sc = e8m0_value((s[i] >> (8 * (ch >> 2))) & 255u);
      float lo[4], hi[4];
      e4m3_decode4(w[i].x, sc, lo);
      e4m3_decode4(w[i].y, sc, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = HASX ? act_slope<ACT>(lo[e]) : act_value<ACT>(lo[e]);
        v[4 + e] = HASX ? act_slope<ACT>(hi[e]) : act_value<ACT>(hi[e]);
      }
    }
    if constexpr (HASX) {
      const uint32_t d[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = kSaved ? bf16_lo(d[e]) * v[2 * e] : bf16_lo(d[e]);
        v[2 * e + 1] = kSaved ? bf16_hi(d[e]) * v[2 * e + 1] : bf16_hi(d[e]);
      }
    }
    // (rows and columns past the end hold zeros: act(0) = 0, 0 act'(0) = 0)
    if (p.partials != nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = sum[e] + v[e];
    }
    *reinterpret_cast<uint4*>(lds + i * (32 * kPitch + kBlockSkew)) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  }
}

// Step 1 of a tile.  A tile with steps that hold no row (past R; nothing reads
// them) takes the others one by one: a tile of a few rows then costs a
// quarter.
template <int ACT, int HASX>
__device__ __forceinline__ void form_tile(const SavedPackParams& p, int64_t bx, int64_t by, uint8_t* tile,
                                          float (&part)[8][kTile]) {
  const int t = threadIdx.x, ch = t & 15;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
  const int64_t rows = p.R - by * kTile;
  if (rows > kTile - 32) {  // all steps
    form_steps<ACT, HASX, kSteps>(p, bx, by, 0, tile, sum);
  } else {
#pragma unroll 1
    for (int i = 0; 32 * i < rows; ++i) form_steps<ACT, HASX, 1>(p, bx, by, i, tile, sum);
  }
  if (p.partials != nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = sum_over_rows4(sum[e]);
    if ((t & 63) < 16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) part[t >> 6][ch * 8 + e] = sum[e];
    }
  }
}

// The packs of a launch, one or two: workgroups from `first` on take tiles of
// the second.
template <int COUNT>
struct SavedPacks {
  SavedPackParams p[COUNT];
  int first;  // tiles of p[0]
};

template <int FMT, int MODE, int HAD, int COUNT>
__global__ __launch_bounds__(512) void quantize_saved_kernel(SavedPacks<COUNT> all) {
  constexpr int B = FmtTraits<FMT>::kBits;
  __shared__ __attribute__((aligned(16))) uint8_t tile[kTileBytes];
  __shared__ float part[8][kTile];
  const int second = COUNT == 2 && (int)blockIdx.x >= all.first ? 1 : 0;
  const SavedPackParams& p = all.p[COUNT == 2 ? second : 0];
  const int local = blockIdx.x - (second ? all.first : 0);
  const int t = threadIdx.x;
  const int tx = (int)((p.C + kTile - 1) / kTile);
  const int64_t by = local / tx, bx = local - by * tx;
  const int64_t r0 = by * kTile, c0 = bx * kTile;
  if (p.x != nullptr) {  // (uniform)
    if (p.act == kActGelu) form_tile<kActGelu, 1>(p, bx, by, tile, part);
    else if (p.act == kActSilu) form_tile<kActSilu, 1>(p, bx, by, tile, part);
    else form_tile<kActNone, 1>(p, bx, by, tile, part);
  } else {
    if (p.act == kActGelu) form_tile<kActGelu, 0>(p, bx, by, tile, part);
    else if (p.act == kActSilu) form_tile<kActSilu, 0>(p, bx, by, tile, part);
    else form_tile<kActNone, 0>(p, bx, by, tile, part);
  }
  __syncthreads();
  if (p.partials != nullptr && t < kTile && c0 + t < p.C) {
    float total = part[0][t];
#pragma unroll
    for (int w = 1; w < 8; ++w) total = total + part[w][t];
    p.partials[by * p.C + c0 + t] = total;
  }

  // 2. rowwise blocks: the four of a row come from four adjacent lanes
  if (p.row_codes != nullptr) {
    uint8_t* const codes = p.row_codes + (bx * p.R + r0) * (16 * B);
    uint8_t* const scales = p.row_scales + (bx * p.R + r0) * 4;
    const int row = t >> 2, blk = t & 3;
    const int64_t r = r0 + row;
    if (r < p.R) {
      if (c0 + blk * 32 < p.C) {
        float v[32];
        lds_row_block(tile + lds_row_at(row), 0, 0, blk * 32, v);
        quant_store<FMT, MODE, HAD>(v, codes + row * (16 * B), blk, r, scales + (row * 4 + blk));
      } else {
        scales[row * 4 + blk] = 0;
        zero_block<FMT>(codes + row * (16 * B), blk, r);
      }
    }
  }

  // 3. columnwise blocks, written as a K-major operand; a block that ends
  //    past R is filled with zero rows, one past R is a pad block
  if (p.col_codes != nullptr) {
    uint8_t* const codes = p.col_codes + (by * p.C + c0) * (16 * B);
    uint8_t* const scales = p.col_scales + (by * p.C + c0) * 4;
    const int col = t >> 2, blk = t & 3;
    if (c0 + col < p.C) {
      if (r0 + blk * 32 < p.R) {
        float v[32];
        const uint16_t* src = reinterpret_cast<const uint16_t*>(tile + lds_row_at(32 * blk)) + col;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = bf16_to_f32(src[i * (kPitch / 2)]);
        quant_store<FMT, MODE, HAD>(v, codes + col * (16 * B), blk, c0 + col, scales + (col * 4 + blk));
      } else {
        scales[col * 4 + blk] = 0;
        zero_block<FMT>(codes + col * (16 * B), blk, c0 + col);
      }
    }
  }
}

template <int FMT, int MODE, int HAD>
hipError_t launch_packs(const SavedPackParams& p, const SavedPackParams* q, int64_t first, int64_t all,
                        hipStream_t stream) {
  if (q)
    hipLaunchKernelGGL((quantize_saved_kernel<FMT, MODE, HAD, 2>), dim3((unsigned)all), dim3(512), 0, stream,
                       (SavedPacks<2>{{p, *q}, (int)first}));
  else
    hipLaunchKernelGGL((quantize_saved_kernel<FMT, MODE, HAD, 1>), dim3((unsigned)all), dim3(512), 0, stream,
                       (SavedPacks<1>{{p}, (int)first}));
  return hipGetLastError();
}

int64_t pack_tiles(const SavedPackParams& p) {
  return ((p.C + kTile - 1) / kTile) * ((p.R + kTile - 1) / kTile);
}

// Workgroups of a save / load launch, or -1 for 2^32 threads or more (the
// runtime's limit; also keeps `groups` and the block index in 31 bits).
int64_t checkpoint_grid(int64_t R, int64_t C, int* groups) {
  const int64_t g = (C + 127) / 128, n = g * ((R + kCkptRows - 1) / kCkptRows);
  *groups = (int)g;
  return n < (1ll << 32) / 256 ? n : -1;
}

}  // namespace

hipError_t launch_checkpoint_save(const void* x, int x_f32, int64_t R, int64_t C, int64_t ldx, uint8_t* codes,
                                  uint8_t* scales, hipStream_t stream) {
  int groups = 0;
  const int64_t n = checkpoint_grid(R, C, &groups);
  if (n < 0) return hipErrorInvalidValue;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL((x_f32 ? checkpoint_save_kernel<1> : checkpoint_save_kernel<0>), dim3((unsigned)n), dim3(256), 0,
                     stream, x, R, C, ldx, codes, scales, groups);
  return hipGetLastError();
}

hipError_t launch_checkpoint_load(const uint8_t* codes, const uint8_t* scales, int64_t R, int64_t C, void* y,
                                  int y_f32, int64_t ldy, hipStream_t stream) {
  int groups = 0;
  const int64_t n = checkpoint_grid(R, C, &groups);
  if (n < 0) return hipErrorInvalidValue;
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL((y_f32 ? checkpoint_load_kernel<1> : checkpoint_load_kernel<0>), dim3((unsigned)n), dim3(256), 0,
                     stream, codes, scales, R, C, y, ldy, groups);
  return hipGetLastError();
}

hipError_t launch_quantize_saved(const SavedPackParams& p, const SavedPackParams* q, int fmt, int mode, int had,
                                 hipStream_t stream) {
  const int64_t first = pack_tiles(p), all = first + (q ? pack_tiles(*q) : 0);
  if (all >= (1ll << 32) / 512) return hipErrorInvalidValue;
  if (all == 0) return hipSuccess;
  if (fmt == kE2M1 && mode == kFloor && !had) return launch_packs<kE2M1, kFloor, 0>(p, q, first, all, stream);
  if (fmt == kE2M3 && mode == kFloor && !had) return launch_packs<kE2M3, kFloor, 0>(p, q, first, all, stream);
  if (fmt == kE2M3 && mode == kFloor && had) return launch_packs<kE2M3, kFloor, 1>(p, q, first, all, stream);
  if (fmt == kE4M3 && mode == kRceil && !had) return launch_packs<kE4M3, kRceil, 0>(p, q, first, all, stream);
  if (fmt == kE4M3 && mode == kFloor && !had) return launch_packs<kE4M3, kFloor, 0>(p, q, first, all, stream);
  return hipErrorInvalidValue;
}

}  // namespace mx
