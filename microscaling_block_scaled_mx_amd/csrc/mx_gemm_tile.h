// One output tile of the block-scaled MX GEMM for gfx950: C = A . B^T on
// K-major packed operands, on the CDNA4 scaled matrix cores
// (v_mfma_scale_f32_32x32x64_f8f6f4: E8M0 block scales applied inside the
// instruction, binary32 accumulation).  Shared by the dense and grouped
// kernels (mx_gemm.hip) and the kernels with an activation epilogue
// (mx_gemm_act.hip).
//
// Tiling.  256 threads = 4 wavefronts in a 2 x 2 grid over a BM x BN output
// tile; a wavefront owns (BM/2) x (BN/2) = (BM/64) x (BN/64) MFMA tiles of
// 32 x 32, whose accumulators live in AGPRs (one wavefront per SIMD).
// 256 x 256 tiles instead run 512 threads = 8 wavefronts in a 2 x 4 grid
// (128 x 64 each, two per SIMD).  K
// advances BK elements per stage (128 for E2M1/E2M3, 64 for E4M3), in steps
// of 64 (one MFMA per output tile).  Stages form a ring of S = 3 or 4
// buffers in LDS filled by direct global -> LDS loads (global_load_lds:
// each lane's 16 bytes land at M0 + 16 * lane), so no registers are spent
// on staging.  A stage's rows are stored densely; the 16-byte chunks of each
// row are permuted (XOR for E2M1 / E4M3, a rotation for E2M3's six chunks)
// so that the 32 rows one operand read touches spread over all LDS banks.
// The main loop is software-pipelined by step: the LDS reads of the next
// step's operands, and the global loads of a stage S - 1 ahead, are threaded
// between the current step's MFMAs, and the one barrier per stage sits at
// the start of its last step, so that the next stage's first operands are
// read while the current stage's last MFMAs run.

// The epilogue kEpiAct (GemmActParams) adds a bias, applies an activation,
// writes the 8-bit checkpoint of the pre-activation and adds a residual, for
// any number of rows.

// Dense tiles are ordered for cache reuse: workgroups are dealt round-robin
// to the 8 XCDs (each with its own L2), so consecutive workgroup ids are
// remapped to give every XCD a contiguous range of tiles, and each range is
// walked in groups of 8 tile rows so that concurrent tiles share A and B
// panels.
//
// MFMA operand layout (measured): lane l holds row l%32 of A (of B) and the
// 32-element K block g = l/32 of the 64-element step.  E2M1 / E2M3 take the
// block's 32 codes contiguously (16 / 24 bytes); E4M3 takes K [16g, 16g+16)
// in bytes 0-15 and [32+16g, 32+16g+16) in bytes 16-31.  The lane's scale
// operand is the E8M0 byte of (its row, block g).  The instruction computes
// X . Y^T with lane l's 16 accumulators holding rows 8*(i/4) + 4*(l/32) + i%4,
// column l%32; the kernel passes the B fragment as X and the A fragment as
// Y, so a lane holds C row l%32 and the four consecutive columns
// 8*(i/4) + 4*(l/32) + {0..3} for each i/4 -- 8 contiguous bytes of bf16.
#pragma once

#include <type_traits>

#include "mx_act.h"
#include "mx_device.h"
#include "mx_kernels.h"
#include "mx_linear.h"

namespace mx {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));


template <int FMT> struct MfmaFmt;
template <> struct MfmaFmt<kE4M3> { static constexpr int kCode = 0; };
template <> struct MfmaFmt<kE2M3> { static constexpr int kCode = 2; };
template <> struct MfmaFmt<kE2M1> { static constexpr int kCode = 4; };

// Threads per workgroup of a BM x BN tile: 8 wavefronts for 256 x 256 and
// for the SwiGLU / dSwiGLU epilogues' 128 x 256 (two per SIMD, so that the
// epilogue's long VALU dependency chains of one wavefront interleave with
// another's), else 4.
constexpr int tile_threads(int bm, int bn, int epi = 0) {
  return ((bm == 256 && bn == 256) || (bm == 128 && bn == 256 && (epi == 1 || epi == 2))) ? 512 : 256;
}

// OCC: workgroups resident per compute unit (1 or 2).  With 2, each takes at
// most half the LDS and, per wavefront, half the register file, so that one
// workgroup's MFMAs run while the other waits on its loads, its barrier or
// its prologue and epilogue.
template <int FMT, int BM, int BN, int MODE, int EPI, int OCC = 1>
struct Cfg {
  static_assert(OCC == 1 || OCC == 2, "workgroups per compute unit");
  static constexpr int kLds = 163840 / OCC;              // LDS bytes one workgroup may take
  static constexpr int kBits = FmtTraits<FMT>::kBits;
  // 256 x 256 tiles run 8 wavefronts (2 per SIMD, 2 x 4 over the tile, 128
  // accumulator registers each), so that one wavefront's MFMAs can cover
  // the other's LDS and barrier waits (measured 2-4% faster than 4
  // wavefronts of 256 accumulators each); the other shapes run 4 (2 x 2)
  static constexpr int kThreads = tile_threads(BM, BN, EPI);
  static constexpr int kWaves = kThreads / 64;
  static constexpr int kWavesN = kWaves / 2;  // wavefronts across N (2 across M)
  // K elements per stage: one 128-element K group (64 / 96 / 128 bytes per
  // row); E4M3 tiles whose 128-element stages would not fit a ring of two in
  // the LDS, or whose accumulators take more than 144 registers (leaving too
  // few for double-buffered 8-register fragments), take half a group (64
  // bytes) per stage.  Every stage ends in a
  // workgroup barrier: at 256 x 256, two 128-element E4M3 stages measured
  // 4-8% faster than four of 64 (MXFP8 16384 x 9216 x 3072: 504 -> 466 us;
  // the grouped step 954 -> 899 us, same box).
  static constexpr int kAccRegs = (BM / 64) * (BN / kWavesN / 32) * 16;  // accumulator registers per lane
  static constexpr int kBK = FMT == kE4M3 && (2 * ((BM + BN) * 128 + 2048) > kLds || kAccRegs > 144) ? 64 : 128;
  static constexpr int kRowBytes = kBK * kBits / 8;      // 64 / 96 / 128 (or 64) bytes per row per stage
  static constexpr int kChunks = kRowBytes / 16;         // 16-byte chunks per row per stage
  static constexpr int kScaleDw = 1;                     // scale dword (4 blocks of 32 along K) per row per stage
  static constexpr int kSJ = 512 / kThreads;            // scale-dword loads per thread per stage (512 slots)
  // 16-byte loads per thread per stage; a tile side whose chunks do not fill
  // whole loads (192 rows of 96 bytes) leaves the last load of some
  // wavefronts idle: they load a valid chunk into a junk area, so that every
  // wavefront issues the same number of loads (the vmcnt waits count them)
  static constexpr int kAIters = (BM * kChunks + kThreads - 1) / kThreads;
  static constexpr int kBIters = (BN * kChunks + kThreads - 1) / kThreads;
  static constexpr int kARem = (BM * kChunks) % kThreads;  // slots of a partial last load (0: none)
  static constexpr int kBRem = (BN * kChunks) % kThreads;
  static_assert(kARem % 64 == 0 && kBRem % 64 == 0, "partial loads cover whole wavefronts");
  // The ring of kStages stage buffers is laid out region by region: the A
  // rows of buffers 0 .. S-1, then their B rows, then their scale dwords
  // ([A rows, then B rows], 512 slots), then a junk area for idle load
  // slots.  Every read of one operand from any buffer is then within the
  // 16-bit offset of a ds_read from one per-lane base.
  static constexpr int kARegion = BM * kRowBytes;
  static constexpr int kBRegion = BN * kRowBytes;
  static constexpr int kSRegion = kScaleDw * 512 * 4;
  static constexpr int kJunk = (kARem || kBRem) ? 1024 : 0;
  static constexpr int kStage = kARegion + kBRegion + kSRegion;  // bytes per stage
  static constexpr int kStages = (4 * kStage + kJunk <= kLds) ? 4 : (3 * kStage + kJunk <= kLds) ? 3 : 2;
  static_assert(kStages * kStage + kJunk <= kLds, "two stages fit the LDS");
  static constexpr int aoff(int b) { return b * kARegion; }
  static constexpr int boff(int b) { return kStages * kARegion + b * kBRegion; }
  static constexpr int soff(int b) { return kStages * (kARegion + kBRegion) + b * kSRegion; }
  static constexpr int kJOff = kStages * kStage;
  static constexpr int kWM = BM / 2, kWN = BN / kWavesN;
  static_assert(kWN % 32 == 0, "wavefront tile width");
  static constexpr int kMI = kWM / 32, kNJ = kWN / 32;
  static constexpr int kLoads = kAIters + kBIters + kSJ * kScaleDw;  // vector-memory instructions per stage per wave
  static_assert(BM + BN <= 512, "scale slots");
  // epilogue staging
  static constexpr int kCPitch = kWN * 2 + 8;         // bf16 store: per-wave kWM x kWN tile
  static constexpr int kZPitch = BN * 2 + 16;         // SwiGLU: gate | up tile BM x BN, then z in its gate half
  static constexpr int kDPitch = BN * 2 + 16;         // dSwiGLU: two BM x BN tiles, 16-byte rows
  static constexpr int kEpiBytes = EPI == kEpiSwiglu    ? BM * kZPitch
                                   : EPI == kEpiDSwiglu ? 2 * BM * kDPitch
                                                        : kWaves * kWM * kCPitch;
  static constexpr int kBiasAt = (kJOff + kJunk > kEpiBytes) ? kJOff + kJunk : kEpiBytes;
  static constexpr int kSmem = kBiasAt + (EPI == kEpiAct ? BN * 4 : 0);  // kEpiAct: the tile's bias beside the ring
  // kEpiAct: the residual's tile waits in registers while the sums run, where
  // the accumulators leave them
  static constexpr bool kResidualAhead = EPI == kEpiAct && kAccRegs <= 64;
  static_assert(kSmem <= kLds, "LDS budget");
};

// Position of logical 16-byte chunk c of row r among the row's NCH stored
// chunks, chosen so that the 16-byte operand reads of one chunk by the 32
// rows of a wavefront (its two halves reading adjacent chunks) take the
// minimum four LDS cycles (measured with the bank-conflict counter on
// gfx950): NCH = 8 (128-byte rows): c ^ ((r ^ (r >> 3)) & 7);  NCH = 4
// (64-byte rows): c ^ ((r >> 2) & 3) -- a permutation that also depends on
// row bit 4, or on rows r >> 1, costs twice that;  NCH = 6 (96-byte rows,
// whose bases repeat every 8 rows modulo 64 banks): (c + ((r >> 3) & 1)) %
// 6, which moves rows 8..15 of every 16 by one 4-bank step.
template <int NCH>
__device__ __forceinline__ int chunk_pos(int r, int c) {
  static_assert(NCH == 4 || NCH == 6 || NCH == 8, "chunks per row");
  if constexpr (NCH == 6) { const int q = c + ((r >> 3) & 1); return q >= 6 ? q - 6 : q; }
  else if constexpr (NCH == 8) return c ^ ((r ^ (r >> 3)) & 7);
  else return c ^ ((r >> 2) & 3);
}
// Inverse: the logical chunk stored at position pos of row r.
template <int NCH>
__device__ __forceinline__ int chunk_at(int r, int pos) {
  if constexpr (NCH == 6) { const int q = pos - ((r >> 3) & 1); return q < 0 ? q + 6 : q; }
  else return chunk_pos<NCH>(r, pos);  // the XOR permutations are involutions
}

// The intrinsics below exist only for the GPU; their bodies are compiled in
// the device pass alone, so the host pass sees plain declarations.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
#if defined(__HIP_DEVICE_COMPILE__)
  // s_waitcnt: vmcnt[3:0] + vmcnt[5:4] at bits 15:14; expcnt (7) and lgkmcnt (15) left unconstrained
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
#endif
}

// Wait for every outstanding LDS read of this wavefront.
__device__ __forceinline__ void wait_lgkmcnt0() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // vmcnt and expcnt unconstrained, lgkmcnt 0
#endif
}

// Workgroup barrier without a memory fence (the stage loads are awaited
// explicitly with vmcnt); the empty asm keeps the compiler from moving LDS
// accesses across it.
__device__ __forceinline__ void stage_barrier() {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#endif
}

// Direct global -> LDS copy of 16 (4) bytes per lane: lane l's bytes land at
// LDS byte address lds + 16 * l (lds + 4 * l); lds must be the same for the
// whole wavefront (it goes to M0, which an LDS DMA needs one wait state
// after writing).  Written as inline assembly: the compiler models the
// intrinsic as a flat access to both global memory and the LDS, and while
// one is in flight it turns every LDS wait it inserts into a wait for all
// outstanding reads.  Kernels order these loads with explicit vmcnt waits
// and barriers.
__device__ __forceinline__ uint32_t lds_addr(const void* lds) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)lds;
}
__device__ __forceinline__ void lds_dma16(const void* g, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "{m0}"(lds) : "memory");
#endif
}
// The same from a wavefront-uniform base (scalar registers) plus a per-lane
// 32-bit byte offset, so that the per-lane part stays fixed across stages.
__device__ __forceinline__ void lds_dma16_s(const void* base, uint32_t off, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
#endif
}
__device__ __forceinline__ void lds_dma4_s(const void* base, uint32_t off, uint32_t lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
#endif
}

// A pointer the compiler must take as produced here: it stays in scalar
// registers (or is spilled) instead of being loaded again where it is used.
template <typename T>
__device__ __forceinline__ void held_in_sgprs(T*& v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+s"(v));
#endif
}

// Materialize a kernel argument in scalar registers at this point.  The
// epilogue's arguments are pinned before the main loop: a scalar load still
// in flight there shares the LDS wait counter, and the compiler then turns
// every LDS wait in the loop into a wait for all outstanding reads.
template <typename T>
__device__ __forceinline__ void pin_arg(T v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" ::"s"(v));
#endif
}

// Keep the machine scheduler from moving instructions across this point.
__device__ __forceinline__ void sched_fence() {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_sched_barrier(0);
#endif
}

__device__ __forceinline__ int wave_uniform(int v) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_readfirstlane(v);
#else
  return v;
#endif
}

// Read one lane's A/B operand for K step ks of the stage from row r of the
// LDS tile (row base rowp); g = lane / 32 picks the 32-element K block.
template <int FMT, int NCH>
__device__ __forceinline__ v8i lds_operand(const uint8_t* rowp, int r, int ks, int g) {
  v8i v;
  if constexpr (FMT == kE4M3) {  // chunks 4 ks + g and 4 ks + 2 + g
    const v4i a = *reinterpret_cast<const v4i*>(rowp + 16 * chunk_pos<NCH>(r, 4 * ks + g));
    const v4i b = *reinterpret_cast<const v4i*>(rowp + 16 * chunk_pos<NCH>(r, 4 * ks + 2 + g));
    v = v8i{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  } else if constexpr (FMT == kE2M1) {  // chunk 2 ks + g
    // the instruction reads 4 dwords of an E2M1 operand: the upper half is
    // left undefined so that those registers stay free
    const v4i a = *reinterpret_cast<const v4i*>(rowp + 16 * chunk_pos<NCH>(r, 2 * ks + g));
    v = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  } else {
    // block b = 2 ks + g of the group: its first 16 bytes are chunk b, its
    // last 8 bytes half g (g ^ 1 in rows with bit 4 set) of chunk 4 + ks (the
    // E2M3 order inside a K group); the instruction reads 6 dwords of an
    // E2M3 operand.  Both reads are conflict-free across the 64 banks.
    const v4i w = *reinterpret_cast<const v4i*>(rowp + 16 * chunk_pos<NCH>(r, 2 * ks + g));
    const v2i h = *reinterpret_cast<const v2i*>(rowp + 16 * chunk_pos<NCH>(r, 4 + ks) + 8 * (g ^ ((r >> 4) & 1)));
    const v4i h4 = __builtin_shufflevector(h, h, 0, 1, -1, -1);
    v = __builtin_shufflevector(w, h4, 0, 1, 2, 3, 4, 5, -1, -1);
  }
  return v;
}

// Dense tile order: XCD-contiguous ranges, then groups of 8 tile rows.
__device__ __forceinline__ void dense_tile(int bid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int T = tiles_m * tiles_n;
  if ((T & 7) == 0) bid = (bid & 7) * (T >> 3) + (bid >> 3);
  const int GM = 8;
  const int per_group = GM * tiles_n;
  const int group = bid / per_group;
  const int first_m = group * GM;
  const int gsize = (tiles_m - first_m) < GM ? (tiles_m - first_m) : GM;
  const int r = bid - group * per_group;
  tm = first_m + r % gsize;
  tn = r / gsize;
}

// One row's 32-byte E4M3 block from a 32-column MFMA tile: lane l holds
// columns 8 (e / 4) + 4 (l / 32) + e % 4 (e = 0..15) of row l % 32, so the
// row's maximum and its bytes come from lanes l and l ^ 32: one exchange of
// half wavefronts for the maximum, two for the codes, after which each lane
// owns the 16 bytes at 16 (l / 32).  Returns the scale byte.
__device__ __forceinline__ uint32_t checkpoint_block(float (&v)[16], uint4& codes) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t m = abs_max(v);
  const auto mm = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  const uint32_t s = scale_byte<kE4M3, kRceil>(max_u32(mm[0], mm[1]));
  uint32_t w[4];
  e4m3_encode(v, s, w);
  const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  codes = make_uint4(x[0], x[1], y[0], y[1]);
  return s;
#else
  return 0u;
#endif
}

// P: GemmParams, or GemmActParams for kEpiAct, whose M and N need not be
// whole tiles: operand rows past the end are loaded as the last row and
// never stored.
template <int FMT, int BM, int BN, int MODE, int EPI, int OCC = 1, class P = GemmParams>
__device__ __forceinline__ void gemm_tile(const P& p, int bx, int by, int bz, uint8_t* smem) {
  using CF = Cfg<FMT, BM, BN, MODE, EPI, OCC>;
  constexpr int kBits = CF::kBits;

  const int t = threadIdx.x;
  const int lane = t & 63, wave = t >> 6;
  const int wm = wave / CF::kWavesN, wn = wave % CF::kWavesN;
  constexpr int kThreads = CF::kThreads;
  const int lrow = lane & 31, g = lane >> 5;

  // ---------------------------------------------------------------- tile
  int tm, tn;
  int split = 0;  // split K: this workgroup's part of the K range
  if constexpr (MODE == kDense) {
    constexpr int kUp = EPI == kEpiAct ? 1 : 0;  // whole tiles, or a partial one at each end
    const int tiles_m = (int)((p.M + kUp * (BM - 1)) / BM), tiles_n = (int)((p.N + kUp * (BN - 1)) / BN);
    int local = bx;
    if constexpr (EPI == kEpiSplit) {  // workgroups [s * T, (s + 1) * T) compute part s
      split = bx / (tiles_m * tiles_n);
      local = bx - split * (tiles_m * tiles_n);
    }
    dense_tile(local, tiles_m, tiles_n, tm, tn);
  } else if constexpr (MODE == kRaggedM) {
    // 1-D grid of (row tile, column tile) pairs, column tiles fastest.  Each
    // XCD takes a contiguous range, so the tiles of one row panel (and of
    // one group's weights) share that XCD's L2 -- except under dSwiGLU,
    // whose epilogue reads H rows scattered over its tile and measured 17%
    // faster with consecutive tiles spread over the XCDs (the other
    // epilogues 3-7% slower that way).
    const int nt = (int)(EPI == kEpiSwiglu ? 2 * p.F / BN : p.N / BN);
    const int T = (int)gridDim.x;
    int bid = bx;
    if (EPI != kEpiDSwiglu && (T & 7) == 0) bid = (bid & 7) * (T >> 3) + (bid >> 3);
    tn = bid % nt;
    tm = bid / nt;
  } else {
    tn = bx;
    tm = by;
  }
  int64_t m0 = (int64_t)tm * BM;
  int64_t m_end = 0;  // ragged-M: end of this tile's group (rows of C it may write)
  const int64_t n0 = (int64_t)tn * BN;  // SwiGLU: tile tn covers z columns [tn*BN/2, (tn+1)*BN/2)
  int64_t kbeg = 0, kend = p.K;
  int64_t b_row0 = 0;  // first B row of this tile's group
  int64_t b_soff = 0;  // byte offset of this tile's group in the B scales (one blocked array per group)
  int64_t b_coff = 0;  // byte offset of this tile's group in the B codes (one K-group-major array per group)
  int64_t c_off = 0;   // element offset of this tile's group in C
  if constexpr (MODE == kRaggedM) {
    // Group gi's rows [start, end) are cut into ceil((end - start) / BM)
    // tiles (counts are multiples of 128, so a 256-row tile at a group's
    // end may hold 128 rows); row tile tm walks the groups in order.  Rows
    // of a tile past its group's end are loaded as the group's last row and
    // never stored, so nothing at or past the last end is read or written.
    // Offsets are a caller invariant; clamping them into [start, R] and down
    // to a multiple of 128 keeps every access inside the buffers (and every
    // 32-row column block inside one tile) even if they are broken.
    int64_t start = 0;
    int rem = tm, gi = -1;
    for (int q = 0; q < p.G; ++q) {
      int64_t e = p.offsets[q];
      e = (e < start ? start : (e > p.R ? p.R : e)) & ~(int64_t)127;
      const int64_t nt = (e - start + BM - 1) / BM;
      if (rem < nt) {
        gi = q;
        m0 = start + (int64_t)rem * BM;
        m_end = e;
        break;
      }
      rem -= (int)nt;
      start = e;
    }
    if (gi < 0) return;  // past the last group's tiles
    b_row0 = (int64_t)gi * p.b_group_rows;
    b_soff = (int64_t)gi * scale_bytes(p.b_group_rows, p.ktot);
    b_coff = (int64_t)gi * code_bytes(p.b_group_rows, p.ktot, kBits);
  }
  if constexpr (MODE == kDense && EPI == kEpiSplit) {
    {
      const int64_t part = p.K / p.split_k;
      kbeg = split * part;
      kend = kbeg + part;
      c_off = split * p.M * p.ldc;
    }
  }
  if constexpr (MODE == kRaggedK) {
    const int gi = bz;
    kbeg = gi ? p.offsets[gi - 1] : 0;
    kend = p.offsets[gi];
    kbeg = (kbeg < 0 ? 0 : (kbeg > p.R ? p.R : kbeg)) & ~(int64_t)127;
    kend = (kend < 0 ? 0 : (kend > p.R ? p.R : kend)) & ~(int64_t)127;
    if (kend < kbeg) kend = kbeg;
    c_off = (int64_t)gi * p.M * p.N;
  }
  if constexpr (EPI == kEpiAct) kend = (p.K + 127) & ~(int64_t)127;  // pad codes and scales are zero
  // rows of the A / B operands (of one group's B): the stride between K
  // groups of their codes and scales
  const int64_t a_rows = p.M;
  const int64_t b_rows = MODE == kRaggedM ? p.b_group_rows : p.N;
  constexpr int kGB = 16 * kBits;  // code bytes of one row in one 128-element K group
  const int nk = (int)((kend - kbeg) / CF::kBK);

  // LDS row r of the B tile -> global B row
  auto b_row = [&](int r) -> int64_t {
    if constexpr (EPI == kEpiSwiglu) {
      const int64_t zb = (int64_t)tn * (BN / 2);
      return b_row0 + (r < BN / 2 ? zb + r : p.F + zb + (r - BN / 2));
    } else if constexpr (EPI == kEpiAct) {
      return n0 + r < p.N ? n0 + r : p.N - 1;
    } else {
      return b_row0 + n0 + r;
    }
  };

  // ---------------------------------------------------------------- loads
  // Stage slot s (16-byte units, s = i * 256 + t for load i of thread t)
  // holds row s / kChunks, position s % kChunks, i.e. logical chunk
  // chunk_at(row, position) of the row's stage segment.  A stage lies inside
  // one 128-element K group: its segment of a row starts (k0 % 128) * bits/8
  // bytes into the row's kGB-byte run of that group.  Offsets from the
  // group's start are 32-bit (operands < 2 GiB).
  constexpr int BK = CF::kBK;
  uint32_t a_off[CF::kAIters], b_off[CF::kBIters];
#pragma unroll
  for (int i = 0; i < CF::kAIters; ++i) {
    const int q = t + kThreads * i, r = q / CF::kChunks, pos = q % CF::kChunks;
    const int rr = r < BM ? r : 0;  // junk slots read a valid chunk
    const int c = chunk_at<CF::kChunks>(rr, pos);
    int64_t ar = MODE == kRaggedM && m0 + rr >= m_end ? m_end - 1 : m0 + rr;
    if constexpr (EPI == kEpiAct) ar = ar < p.M ? ar : p.M - 1;
    a_off[i] = (uint32_t)(ar * kGB + 16 * c);
  }
#pragma unroll
  for (int i = 0; i < CF::kBIters; ++i) {
    const int q = t + kThreads * i, r = q / CF::kChunks, pos = q % CF::kChunks;
    const int rr = r < BN ? r : 0;
    const int c = chunk_at<CF::kChunks>(rr, pos);
    b_off[i] = (uint32_t)(b_coff + (b_row(rr) - b_row0) * kGB + 16 * c);
  }
  // scale dwords (4 blocks of 32 along K, blocked layout): slot t + kThreads j
  // of [A rows | B rows]; slots past BM + BN load row 0's dword into unused
  // slots, so every wave issues the same number of loads.  BM and BN are
  // multiples of 64, so a wavefront's 64 slots are all A rows, all B rows or
  // all unused: each load takes a wavefront-uniform base and K-group stride
  // (scalar registers) and a fixed per-lane 32-bit offset, and no vector
  // address arithmetic is left in the main loop.
  static_assert(BM % 64 == 0 && BN % 64 == 0, "scale slots of a wavefront are one operand's");
  const uint8_t* s_base[CF::kSJ];
  uint32_t s_step[CF::kSJ];  // bytes between consecutive K groups
  uint32_t s_off[CF::kSJ];
#pragma unroll
  for (int j = 0; j < CF::kSJ; ++j) {
    const int r = t + kThreads * j;
    const int rw = wave_uniform(r);  // the wavefront's first slot
    const bool is_b = rw >= BM && rw < BM + BN;
    int64_t ar = MODE == kRaggedM && m0 + (r < BM ? r : 0) >= m_end ? m_end - 1 : m0 + (r < BM ? r : 0);
    if constexpr (EPI == kEpiAct) ar = ar < p.M ? ar : p.M - 1;
    s_base[j] = is_b ? p.b_scales + b_soff : p.a_scales;
    s_off[j] = (uint32_t)(is_b ? (b_row(r - BM) - b_row0) * 4 : ar * 4);
    s_step[j] = (uint32_t)((is_b ? b_rows : a_rows) * 4);
  }
  // bytes between consecutive K groups of the A / B codes; every offset
  // into an operand fits 32 bits (operands < 2 GiB), so a stage's base is
  // one 32-bit product and one 64-bit add
  const uint32_t a_gb = (uint32_t)(a_rows * kGB), b_gb = (uint32_t)(b_rows * kGB);
  // the operand bases, held in scalar registers for the whole loop: taken
  // through an empty asm, the compiler cannot re-derive them by loading the
  // kernel argument again (a scalar load in the loop shares the LDS wait
  // counter, and its wait would also wait for every LDS read in flight)
  const uint8_t* a_codes = p.a_codes;
  const uint8_t* b_codes = p.b_codes;
  held_in_sgprs(a_codes);
  held_in_sgprs(b_codes);
  const int wave_u = wave_uniform(wave);
  const uint32_t smem_lds = wave_uniform((int)lds_addr(smem));  // LDS byte address of smem

  // Load q (0 <= q < kLoads) of stage k into ring buffer buf: A chunks, then
  // B chunks, then scale dwords (K group d, slot half j).  Every use sits in
  // fully unrolled code, so q is a constant and each use compiles to one
  // load instruction.
#define MX_PIECE(k, buf, q)                                                                               \
  do {                                                                                                   \
    const uint32_t k0_ = (uint32_t)kbeg + (uint32_t)(k) * BK;                                            \
    const uint32_t g_ = k0_ >> 7, w_ = (k0_ & 127) * kBits / 8;                                          \
    const uint32_t st_ = smem_lds;                                                                       \
    if ((q) < CF::kAIters) {                                                                             \
      const int i_ = (q) < CF::kAIters ? (q) : 0;                                                        \
      const bool junk_ = CF::kARem && i_ == CF::kAIters - 1 && wave_u * 64 >= CF::kARem;                 \
      lds_dma16_s(a_codes + (g_ * a_gb + w_), a_off[i_],                                                \
                  st_ + (junk_ ? CF::kJOff : CF::aoff(buf) + (i_ * kThreads + wave_u * 64) * 16));            \
    } else if ((q) < CF::kAIters + CF::kBIters) {                                                        \
      const int i_ = (q) >= CF::kAIters && (q) < CF::kAIters + CF::kBIters ? (q) - CF::kAIters : 0;      \
      const bool junk_ = CF::kBRem && i_ == CF::kBIters - 1 && wave_u * 64 >= CF::kBRem;                 \
      lds_dma16_s(b_codes + (g_ * b_gb + w_), b_off[i_],                                                \
                  st_ + (junk_ ? CF::kJOff : CF::boff(buf) + (i_ * kThreads + wave_u * 64) * 16));            \
    } else {                                                                                             \
      const int e_ = (q) >= CF::kAIters + CF::kBIters ? (q) - CF::kAIters - CF::kBIters : 0;             \
      const int d_ = e_ / CF::kSJ, j_ = e_ % CF::kSJ;                                                    \
      lds_dma4_s(s_base[j_] + (g_ + d_) * s_step[j_], s_off[j_],                                        \
               st_ + CF::soff(buf) + (d_ * 512 + j_ * kThreads + wave_u * 64) * 4);                     \
    }                                                                                                    \
  } while (0)
#define MX_ISSUE(k, buf)                                                                                  \
  do {                                                                                                   \
    _Pragma("unroll") for (int q_ = 0; q_ < CF::kLoads; ++q_) MX_PIECE(k, buf, q_);                     \
  } while (0)

  // ---------------------------------------------------------------- main loop
  v16f acc[CF::kMI][CF::kNJ];
#pragma unroll
  for (int i = 0; i < CF::kMI; ++i)
#pragma unroll
    for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // LDS rows this lane reads
  int arow[CF::kMI], brow[CF::kNJ];
#pragma unroll
  for (int i = 0; i < CF::kMI; ++i) arow[i] = wm * CF::kWM + 32 * i + lrow;
#pragma unroll
  for (int j = 0; j < CF::kNJ; ++j) {
    if constexpr (EPI == kEpiSwiglu) {  // j < NJ/2: gate columns, j >= NJ/2: the matching up columns
      constexpr int H = CF::kNJ / 2;
      brow[j] = (j < H ? 0 : BN / 2) + wn * (CF::kWN / 2) + 32 * (j % H) + lrow;
    } else {
      brow[j] = wn * CF::kWN + 32 * j + lrow;
    }
  }

  // Software pipeline over K steps of 64 (KS per stage).  The MFMAs of a step
  // use operand fragments already in registers; the LDS reads of the next
  // step's fragments are threaded between them, and so are the global -> LDS
  // loads of a stage S - 1 ahead.  Each A fragment is re-read right after
  // the last MFMA of the step that uses it; B fragments are double-buffered
  // by step parity for E2M1 / E2M3, and re-read after their last use like A
  // for E4M3, whose MFMAs take twice as long (the registers an E4M3 operand
  // needs do not fit twice).  The last step of stage it first waits for
  // stage it + 1 to land and passes the one barrier of the stage, so that
  // its MFMAs overlap the reads of stage it + 1's first fragments and
  // scales; after that barrier no wave reads buffer it % S any more, and the
  // loads of stage it + S may refill it.  The loads of a stage are issued
  // over a window of KS steps: the last step of stage st - S (after its
  // barrier), then the first KS - 1 steps of stage st - S + 1, so at every
  // barrier exactly the S - 2 stages after the awaited one may still be in
  // flight.  Stages past the last one re-load the last stage's K range into
  // their (free) ring buffers, and the last stage still passes its barrier
  // and reads "its successor", so the loop has no branches and every wait
  // count is a constant; the epilogue waits for those extra loads before it
  // reuses the LDS.
  constexpr int S = CF::kStages;
  constexpr int KS = BK / 64;
  constexpr bool kBDouble = KS == 2;
  constexpr int kMf = CF::kMI * CF::kNJ;  // MFMAs per step
  constexpr int kWin = KS * kMf;          // MFMA slots in a stage's load window
  constexpr int kPart0 = (CF::kLoads + KS - 1) / KS;  // loads in the window's first step
  static_assert(CF::kLoads <= 2 * kWin, "two loads per MFMA slot at most");
  static_assert(KS == 1 || KS == 2, "steps per stage");
  // fragment reads (and, across a stage boundary, the scale reads) go in
  // the first three quarters of a step's MFMA slots where the registers
  // allow, so that they have landed when the next step starts
  constexpr int kReadSlots = kMf > 4 ? (3 * kMf) / 4 : kMf;
  // slot of read unit u (issued after that slot's MFMA): spread over the
  // read slots, but a single-buffered fragment no earlier than the last MFMA
  // that uses it.  Units: [the scales,] A0, B0 .. B(NJ-1), A1 .. A(MI-1).
  auto read_slot = [](int u, bool with_scales) constexpr {
    const int nu = CF::kMI + CF::kNJ + (with_scales ? 1 : 0);
    const int v = with_scales ? u - 1 : u;
    const int nominal = u * kReadSlots / nu;
    int first = 0;
    if (v == 0 || v > CF::kNJ) first = (v == 0 ? 0 : v - CF::kNJ) * CF::kNJ + CF::kNJ - 1;  // A
    else if (v > 0 && !kBDouble) first = (CF::kMI - 1) * CF::kNJ + (v - 1);                 // B
    return nominal > first ? nominal : first;
  };

  v8i af[CF::kMI], bf[kBDouble ? 2 : 1][CF::kNJ];
  uint32_t sca[CF::kMI], scb[CF::kNJ];  // this stage's scale dwords, shifted so byte 0 is its block g
  uint32_t nsa[CF::kMI], nsb[CF::kNJ];  // the next stage's scale dwords as stored

  // scale dwords and operand fragments of ring buffer b (a constant)
  auto read_scales = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < CF::kMI; ++i) nsa[i] = *reinterpret_cast<const uint32_t*>(smem + CF::soff(b) + arow[i] * 4);
#pragma unroll
    for (int j = 0; j < CF::kNJ; ++j)
      nsb[j] = *reinterpret_cast<const uint32_t*>(smem + CF::soff(b) + (BM + brow[j]) * 4);
  };
  // fragment v of a step (v = 0: A0, 1 .. NJ: B0 .. B(NJ-1), then A1 ..)
  auto read_frag = [&](int reg, int v, int b, int ks) __attribute__((always_inline)) {
    if (v == 0 || v > CF::kNJ) {
      const int i = v == 0 ? 0 : v - CF::kNJ;
      af[i] = lds_operand<FMT, CF::kChunks>(smem + CF::aoff(b) + arow[i] * CF::kRowBytes, arow[i], ks, g);
    } else {
      const int j = v - 1;
      bf[kBDouble ? reg : 0][j] =
          lds_operand<FMT, CF::kChunks>(smem + CF::boff(b) + brow[j] * CF::kRowBytes, brow[j], ks, g);
    }
  };

  // one step: stage it (in ring buffer B = it % S, a constant), K step ks
  auto step = [&](int it, auto ksc, auto bc) __attribute__((always_inline)) {
    constexpr int ks = decltype(ksc)::value, B = decltype(bc)::value;
    constexpr int cur = kBDouble ? ks : 0;  // B fragment buffer of this step
    constexpr int sel = 2 * ks;             // byte of the shifted scale dwords: block 2 ks + g of the stage
    constexpr bool last = ks == KS - 1;
    if (last) {
      wait_vmcnt<CF::kLoads * (S - 2)>();  // this wave's loads of stage it + 1 landed
      wait_lgkmcnt0();  // every read of buffer it % S done before the barrier frees it
      stage_barrier();
    }
    constexpr int rbuf = last ? (B + 1) % S : B;  // the next step's stage buffer
    constexpr int rks = last ? 0 : ks + 1;
    const int lst = last ? it + S : it + S - 1;  // stage whose loads this step issues
    constexpr int w = last ? 0 : ks + 1;         // ... and its window step
    const int lk = lst < nk ? lst : nk - 1;      // its K range (the last stage's past the end)
    constexpr int lbuf = last ? B : (B + S - 1) % S;
    constexpr int U = CF::kMI + CF::kNJ + (last ? 1 : 0);  // read units: [scales,] fragments
#pragma unroll
    for (int f = 0; f < kMf; ++f) {
      const int i = f / CF::kNJ, j = f % CF::kNJ;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          bf[cur][j], af[i], acc[i][j], MfmaFmt<FMT>::kCode, MfmaFmt<FMT>::kCode, sel, (int)scb[j], sel, (int)sca[i]);
      sched_fence();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (read_slot(u, last) == f) {
          if (last && u == 0) read_scales(rbuf);
          else read_frag(cur ^ 1, last ? u - 1 : u, rbuf, rks);
        }
#pragma unroll
      for (int q = 0; q < CF::kLoads; ++q)
        if (q * kWin / CF::kLoads == w * kMf + f) MX_PIECE(lk, lbuf, q);
      sched_fence();
    }
  };
  auto stage = [&](int it, auto bc) __attribute__((always_inline)) {
    // K block of byte 0: g, or 2 (it & 1) + g for 64-element stages (a
    // dword holds the four blocks of one 128-element group)
    const int sh = 8 * g + (KS == 1 ? 16 * (it & 1) : 0);
#pragma unroll
    for (int i = 0; i < CF::kMI; ++i) sca[i] = nsa[i] >> sh;
#pragma unroll
    for (int j = 0; j < CF::kNJ; ++j) scb[j] = nsb[j] >> sh;
    step(it, std::integral_constant<int, 0>{}, bc);
    if constexpr (KS == 2) step(it, std::integral_constant<int, 1>{}, bc);
  };

  pin_arg(p.c);
  pin_arg(p.ldc);
  pin_arg(p.c_f32);
  if constexpr (EPI == kEpiStore || EPI == kEpiAccum || EPI == kEpiSplit) {
    pin_arg(p.bias);
    pin_arg(p.bias_f32);
  } else if constexpr (EPI == kEpiAct) {
    pin_arg(p.bias);
    pin_arg(p.bias_f32);
    pin_arg(p.residual);
    pin_arg(p.ldr);
    pin_arg(p.act);
    pin_arg(p.saved_codes);
    pin_arg(p.saved_scales);
    pin_arg(p.M);
    pin_arg(p.N);
  } else {
    pin_arg(p.F);
    pin_arg(p.R);
    pin_arg(p.q_mode);
    pin_arg(p.q_row_codes);
    pin_arg(p.q_row_scales);
    pin_arg(p.q_col_codes);
    pin_arg(p.q_col_scales);
    if constexpr (EPI == kEpiDSwiglu) pin_arg(p.aux);
  }
  // kEpiAct: the epilogue's inputs, asked for before the operands so that their
  // latency is hidden.  Unconditional loads (an `if` around them would be
  // waited for at its end): what is not wanted is read from the output.
  constexpr int kRowChunks = CF::kWN / 8;
  constexpr int kAhead = CF::kResidualAhead ? CF::kWM * kRowChunks / 64 : 1;
  [[maybe_unused]] uint4 ahead[kAhead];
  [[maybe_unused]] uint32_t bias_word = 0;
  if constexpr (EPI == kEpiAct) {
    const uint8_t* const any = p.c != nullptr ? reinterpret_cast<const uint8_t*>(p.c) : p.saved_codes;
    const int64_t n = n0 + t % BN < p.N ? n0 + t % BN : p.N - 1;
    const uint8_t* const at = p.bias == nullptr ? any
                              : p.bias_f32      ? reinterpret_cast<const uint8_t*>(p.bias) + 4 * n
                                                : reinterpret_cast<const uint8_t*>(p.bias) + 2 * (n & ~(int64_t)1);
    bias_word = *reinterpret_cast<const uint32_t*>(at);
    if constexpr (CF::kResidualAhead) {
      const bool wanted = p.residual != nullptr && !p.c_f32;
      const uint8_t* const base = wanted ? reinterpret_cast<const uint8_t*>(p.residual) : any;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int q = lane + 64 * i;
        const int64_t m = m0 + wm * CF::kWM + q / kRowChunks, c = n0 + wn * CF::kWN + 8 * (q % kRowChunks);
        const int64_t off = (m < p.M ? m : p.M - 1) * p.ldr + (c < p.N ? c : p.N - 8);
        ahead[i] = *reinterpret_cast<const uint4*>(base + (wanted ? 2 * off : 0));
      }
    }
  }
  if (nk > 0) {  // (a ragged-K group may be empty)
    // prologue: stages 0 .. S - 2 and the first window step of stage S - 1
    // in flight; stage 0's scales and first fragments read
#pragma unroll
    for (int st = 0; st < S - 1; ++st) MX_ISSUE(st < nk ? st : nk - 1, st);
#pragma unroll
    for (int q = 0; q < kPart0; ++q) MX_PIECE(S - 1 < nk ? S - 1 : nk - 1, S - 1, q);
    wait_vmcnt<CF::kLoads * (S - 2) + kPart0>();
    stage_barrier();
    read_scales(0);
#pragma unroll
    for (int v = 0; v < CF::kMI + CF::kNJ; ++v) read_frag(0, v, 0, 0);
    // unrolled by S so that every stage's ring buffer is a constant
    for (int it0 = 0; it0 < nk; it0 += S) {
      stage(it0, std::integral_constant<int, 0>{});
      if (it0 + 1 < nk) stage(it0 + 1, std::integral_constant<int, 1>{});
      if constexpr (S > 2) {
        if (it0 + 2 < nk) stage(it0 + 2, std::integral_constant<int, 2 % S>{});
      }
      if constexpr (S > 3) {
        if (it0 + 3 < nk) stage(it0 + 3, std::integral_constant<int, 3 % S>{});
      }
    }
    wait_vmcnt<0>();  // the loads past the last stage, before the LDS is reused
  }
#undef MX_PIECE
#undef MX_ISSUE
  __syncthreads();  // all wavefronts are done with the stage ring before the epilogue reuses LDS

  // ---------------------------------------------------------------- epilogues
  // Lane (row lrow, column group q = 8 * (e / 4) + 4 * g) of MFMA tile (i, j)
  // holds acc[i][j][4 * (e / 4) + 0..3] = C[row][col + 0..3].
  if constexpr (EPI == kEpiStore || EPI == kEpiAccum || EPI == kEpiSplit) {
    // bias of this lane's columns, read once (one uniform branch); a split
    // part is binary32 without the bias, which the reduction adds
    constexpr bool kPart = EPI == kEpiSplit;
    float bv[CF::kNJ][16];
    if (kPart || p.bias == nullptr) {
#pragma unroll
      for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) bv[j][e] = 0.0f;
    } else if (p.bias_f32) {
      const float* bias32 = reinterpret_cast<const float*>(p.bias);
#pragma unroll
      for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const float4 q = *reinterpret_cast<const float4*>(bias32 + n0 + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g);
          bv[j][4 * e4 + 0] = q.x;
          bv[j][4 * e4 + 1] = q.y;
          bv[j][4 * e4 + 2] = q.z;
          bv[j][4 * e4 + 3] = q.w;
        }
    } else {
      const uint16_t* bias16 = reinterpret_cast<const uint16_t*>(p.bias);
#pragma unroll
      for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const uint2 q = *reinterpret_cast<const uint2*>(bias16 + n0 + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g);
          bv[j][4 * e4 + 0] = bf16_lo(q.x);
          bv[j][4 * e4 + 1] = bf16_hi(q.x);
          bv[j][4 * e4 + 2] = bf16_lo(q.y);
          bv[j][4 * e4 + 3] = bf16_hi(q.y);
        }
    }
    // C += A . B^T (mx_gemm_accumulate: a weight gradient added into a
    // caller-owned main_grad): the previous C joins the binary32 result
    // after the bias, before the store's one rounding.  The old values of
    // one 32-row block of MFMA tiles are loaded together (no load sits under
    // a per-element branch); the accumulators themselves are never
    // rewritten.  A kernel of its own, so that the plain store's register
    // allocation is not touched.
    constexpr bool accumulate = EPI == kEpiAccum;
    auto load_old = [&](int i, float (&o)[CF::kNJ][16]) {
      const int64_t m = m0 + wm * CF::kWM + 32 * i + lrow;
      if (p.c_f32) {
        const float* Co = reinterpret_cast<const float*>(p.c) + m * p.ldc;
        float4 w[CF::kNJ][4];
#pragma unroll
        for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4)
            w[j][e4] = *reinterpret_cast<const float4*>(Co + n0 + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g);
#pragma unroll
        for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            o[j][4 * e4 + 0] = w[j][e4].x;
            o[j][4 * e4 + 1] = w[j][e4].y;
            o[j][4 * e4 + 2] = w[j][e4].z;
            o[j][4 * e4 + 3] = w[j][e4].w;
          }
      } else {
        const uint16_t* Co = reinterpret_cast<const uint16_t*>(p.c) + m * p.ldc;
        uint2 w[CF::kNJ][4];
#pragma unroll
        for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4)
            w[j][e4] = *reinterpret_cast<const uint2*>(Co + n0 + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g);
#pragma unroll
        for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            o[j][4 * e4 + 0] = bf16_lo(w[j][e4].x);
            o[j][4 * e4 + 1] = bf16_hi(w[j][e4].x);
            o[j][4 * e4 + 2] = bf16_lo(w[j][e4].y);
            o[j][4 * e4 + 3] = bf16_hi(w[j][e4].y);
          }
      }
    };
    // value of element e of MFMA tile (i, j): fl32(acc + bias) (+ old)
    if (kPart || p.c_f32) {
      float* C = reinterpret_cast<float*>(p.c) + c_off;
      auto store_f32 = [&](auto with_old) {
        constexpr bool kOld = decltype(with_old)::value;
#pragma unroll
        for (int i = 0; i < CF::kMI; ++i) {
          float o[CF::kNJ][16];
          if constexpr (kOld) load_old(i, o);
          const int64_t m = m0 + wm * CF::kWM + 32 * i + lrow;
          if (MODE == kRaggedM && m >= m_end) continue;
#pragma unroll
          for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const int64_t n = n0 + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g;
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] = acc[i][j][4 * e4 + q] + bv[j][4 * e4 + q];
                if constexpr (kOld) v[q] = v[q] + o[j][4 * e4 + q];
              }
              *reinterpret_cast<float4*>(C + m * p.ldc + n) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
      };
      if constexpr (accumulate) {
        store_f32(std::true_type{});
      } else {
#pragma unroll
        for (int i = 0; i < CF::kMI; ++i)
#pragma unroll
          for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const int64_t m = m0 + wm * CF::kWM + 32 * i + lrow;
              const int64_t n = n0 + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g;
              const v16f& a = acc[i][j];
              if (MODE == kRaggedM && m >= m_end) continue;
              *reinterpret_cast<float4*>(C + m * p.ldc + n) =
                  make_float4(a[4 * e4 + 0] + bv[j][4 * e4 + 0], a[4 * e4 + 1] + bv[j][4 * e4 + 1],
                              a[4 * e4 + 2] + bv[j][4 * e4 + 2], a[4 * e4 + 3] + bv[j][4 * e4 + 3]);
            }
      }
    } else {
      // bf16: stage the wavefront's tile in LDS with 8-byte writes, then
      // write 16-byte row chunks
      uint8_t* wt = smem + wave * CF::kWM * CF::kCPitch;
      auto stage_bf16 = [&](auto with_old) {
        constexpr bool kOld = decltype(with_old)::value;
#pragma unroll
        for (int i = 0; i < CF::kMI; ++i) {
          float o[CF::kNJ][16];
          if constexpr (kOld) load_old(i, o);
#pragma unroll
          for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const int r = 32 * i + lrow, cl = 32 * j + 8 * e4 + 4 * g;
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[q] = acc[i][j][4 * e4 + q] + bv[j][4 * e4 + q];
                if constexpr (kOld) v[q] = v[q] + o[j][4 * e4 + q];
              }
              *reinterpret_cast<uint2*>(wt + r * CF::kCPitch + cl * 2) =
                  make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            }
        }
      };
      // without a bias the sums are rounded as they are (one uniform branch)
      auto stage_sums = [&](auto with_bias) __attribute__((always_inline)) {
        constexpr bool kBias = decltype(with_bias)::value;
#pragma unroll
        for (int i = 0; i < CF::kMI; ++i)
#pragma unroll
          for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const int r = 32 * i + lrow, cl = 32 * j + 8 * e4 + 4 * g;
              const v16f& a = acc[i][j];
              float v[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = kBias ? a[4 * e4 + q] + bv[j][4 * e4 + q] : a[4 * e4 + q];
              *reinterpret_cast<uint2*>(wt + r * CF::kCPitch + cl * 2) =
                  make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            }
      };
      if constexpr (accumulate) {
        stage_bf16(std::true_type{});
      } else if (p.bias != nullptr) {
        stage_sums(std::true_type{});
      } else {
        stage_sums(std::false_type{});
      }
      __syncthreads();
      uint16_t* C = reinterpret_cast<uint16_t*>(p.c) + c_off;
      constexpr int kRowChunks = CF::kWN / 8;
#pragma unroll 4
      for (int q = lane; q < CF::kWM * kRowChunks; q += 64) {
        const int r = q / kRowChunks, ch = q % kRowChunks;
        const uint2 lo = *reinterpret_cast<const uint2*>(wt + r * CF::kCPitch + ch * 16);
        const uint2 hi = *reinterpret_cast<const uint2*>(wt + r * CF::kCPitch + ch * 16 + 8);
        const int64_t m = m0 + wm * CF::kWM + r;
        if (MODE == kRaggedM && m >= m_end) continue;
        *reinterpret_cast<uint4*>(C + m * p.ldc + n0 + wn * CF::kWN + ch * 8) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  } else if constexpr (EPI == kEpiAct) {
    // P = acc + bias in binary32; its checkpoint straight from the
    // registers; then act(P) + residual, rounded once.  Columns are
    // whole 32-column MFMA tiles or none (N is a multiple of 32), rows are
    // masked one by one.  bf16: the residual's tile comes into the wavefront's
    // LDS tile as coalesced 16-byte row chunks, each value is replaced by the
    // result there, and the tile leaves the same way.
    const int64_t mw = m0 + wm * CF::kWM, nw = n0 + wn * CF::kWN;
    uint8_t* wt = smem + wave * CF::kWM * CF::kCPitch;
    const bool staged = p.c != nullptr && !p.c_f32;
    if (staged && p.residual != nullptr) {
      const uint16_t* R = reinterpret_cast<const uint16_t*>(p.residual);
#pragma unroll
      for (int i = 0; i < CF::kWM * kRowChunks / 64; ++i) {
        const int q = lane + 64 * i, r = q / kRowChunks, ch = q % kRowChunks;
        uint4 x;
        if constexpr (CF::kResidualAhead) x = ahead[i];
        else if (mw + r < p.M && nw + 8 * ch < p.N) x = *reinterpret_cast<const uint4*>(R + (mw + r) * p.ldr + nw + 8 * ch);
        *reinterpret_cast<uint2*>(wt + r * CF::kCPitch + ch * 16) = make_uint2(x.x, x.y);
        *reinterpret_cast<uint2*>(wt + r * CF::kCPitch + ch * 16 + 8) = make_uint2(x.z, x.w);
      }
    }
    float* const tile_bias = reinterpret_cast<float*>(smem + CF::kBiasAt);
    if (t < BN) {
      const float b = p.bias_f32 ? __uint_as_float(bias_word) : ((n0 + t) & 1) ? bf16_hi(bias_word) : bf16_lo(bias_word);
      tile_bias[t] = p.bias != nullptr ? b : 0.0f;
    }
    __syncthreads();
    float bv[CF::kNJ][16];
#pragma unroll
    for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
      for (int e4 = 0; e4 < 4; ++e4) {
        const float4 q = *reinterpret_cast<const float4*>(tile_bias + wn * CF::kWN + 32 * j + 8 * e4 + 4 * g);
        bv[j][4 * e4 + 0] = q.x;
        bv[j][4 * e4 + 1] = q.y;
        bv[j][4 * e4 + 2] = q.z;
        bv[j][4 * e4 + 3] = q.w;
      }
    auto finish = [&](auto actc) __attribute__((always_inline)) {
      constexpr int ACT = decltype(actc)::value;
#pragma unroll
      for (int i = 0; i < CF::kMI; ++i) {
        const int r = 32 * i + lrow;
        const int64_t m = mw + r;
        const bool in_m = m < p.M;
        // this row's part of the checkpoint: 64 columns of one K group
        uint8_t* row_codes = p.saved_codes + code_group(m, nw, p.M, 8) + (nw & 127) + 16 * g;
        uint32_t scales = 0;
#pragma unroll
        for (int j = 0; j < CF::kNJ; ++j) {
          const int64_t n = nw + 32 * j;
          if (n >= p.N) continue;
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = acc[i][j][e] + bv[j][e];
          if (p.saved_codes != nullptr) {
            float u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) u[e] = v[e];
            uint4 codes;
            scales |= checkpoint_block(u, codes) << (8 * j);
            if (in_m) *reinterpret_cast<uint4*>(row_codes + 32 * j) = codes;
          }
          if (p.c == nullptr) continue;
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = act_value<ACT>(v[e]);
          if (p.c_f32) {
            float* C = reinterpret_cast<float*>(p.c) + m * p.ldc + n + 4 * g;
            const float* R = reinterpret_cast<const float*>(p.residual) + m * p.ldr + n + 4 * g;
            if (in_m) {
              if (p.residual != nullptr) {
                float4 o[4];
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) o[e4] = *reinterpret_cast<const float4*>(R + 8 * e4);
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) {
                  v[4 * e4 + 0] = v[4 * e4 + 0] + o[e4].x;
                  v[4 * e4 + 1] = v[4 * e4 + 1] + o[e4].y;
                  v[4 * e4 + 2] = v[4 * e4 + 2] + o[e4].z;
                  v[4 * e4 + 3] = v[4 * e4 + 3] + o[e4].w;
                }
              }
#pragma unroll
              for (int e4 = 0; e4 < 4; ++e4)
                *reinterpret_cast<float4*>(C + 8 * e4) =
                    make_float4(v[4 * e4 + 0], v[4 * e4 + 1], v[4 * e4 + 2], v[4 * e4 + 3]);
            }
          } else {
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              uint2* at = reinterpret_cast<uint2*>(wt + r * CF::kCPitch + (32 * j + 8 * e4 + 4 * g) * 2);
              if (p.residual != nullptr) {
                const uint2 o = *at;
                v[4 * e4 + 0] = v[4 * e4 + 0] + bf16_lo(o.x);
                v[4 * e4 + 1] = v[4 * e4 + 1] + bf16_hi(o.x);
                v[4 * e4 + 2] = v[4 * e4 + 2] + bf16_lo(o.y);
                v[4 * e4 + 3] = v[4 * e4 + 3] + bf16_hi(o.y);
              }
              *at = make_uint2(pack_bf16x2(v[4 * e4 + 0], v[4 * e4 + 1]), pack_bf16x2(v[4 * e4 + 2], v[4 * e4 + 3]));
            }
          }
        }
        if (p.saved_codes != nullptr && in_m && nw < ((p.N + 127) & ~(int64_t)127)) {
          // pad blocks (past N, to the end of the last K group): zeros
#pragma unroll
          for (int j = 0; j < CF::kNJ; ++j)
            if (nw + 32 * j >= p.N) *reinterpret_cast<uint4*>(row_codes + 32 * j) = make_uint4(0u, 0u, 0u, 0u);
          if (g == 0) *reinterpret_cast<uint16_t*>(p.saved_scales + scale_offset(m, nw >> 5, p.M)) = (uint16_t)scales;
        }
      }
    };
    static_assert(CF::kWN == 64, "a wavefront's columns are two blocks of one K group");
    if (p.act == kActGelu) finish(std::integral_constant<int, kActGelu>{});
    else if (p.act == kActSilu) finish(std::integral_constant<int, kActSilu>{});
    else finish(std::integral_constant<int, kActNone>{});
    if (staged) {
      __syncthreads();
      uint16_t* C = reinterpret_cast<uint16_t*>(p.c);
#pragma unroll 4
      for (int q = lane; q < CF::kWM * kRowChunks; q += 64) {
        const int r = q / kRowChunks, ch = q % kRowChunks;
        if (mw + r < p.M && nw + 8 * ch < p.N) {
          const uint2 lo = *reinterpret_cast<const uint2*>(wt + r * CF::kCPitch + ch * 16);
          const uint2 hi = *reinterpret_cast<const uint2*>(wt + r * CF::kCPitch + ch * 16 + 8);
          *reinterpret_cast<uint4*>(C + (mw + r) * p.ldc + nw + 8 * ch) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
  } else if constexpr (EPI == kEpiSwiglu) {
    // A lane holds gate (j < NJ/2) and up (j + NJ/2) of the same (row, z
    // columns).  Both are staged in LDS as bf16, the gate half in columns
    // [0, BN/2) of the tile and the up half in [BN/2, BN).  Then each thread
    // takes 8-column chunks of z in row order: H's gate and up chunks go out
    // as coalesced 16-byte stores (a wavefront writes whole 256-byte row
    // segments of each half), and z = SwiGLU(gate, up) replaces the gate
    // chunk; z is then quantized rowwise and columnwise out of LDS.
    constexpr int H2 = CF::kNJ / 2;
    uint8_t* zt = smem;  // pitch kZPitch: the staged gate | up tile, then z in the gate half
    const int64_t zb = (int64_t)tn * (BN / 2);
    uint16_t* Hc = reinterpret_cast<uint16_t*>(p.c);
#pragma unroll
    for (int i = 0; i < CF::kMI; ++i)
#pragma unroll
      for (int j = 0; j < H2; ++j)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const int ml = wm * CF::kWM + 32 * i + lrow;
          const int zc = wn * (CF::kWN / 2) + 32 * j + 8 * e4 + 4 * g;
          const v16f& ag = acc[i][j];
          const v16f& au = acc[i][j + H2];
          *reinterpret_cast<uint2*>(zt + ml * CF::kZPitch + zc * 2) =
              make_uint2(pack_bf16x2(ag[4 * e4 + 0], ag[4 * e4 + 1]), pack_bf16x2(ag[4 * e4 + 2], ag[4 * e4 + 3]));
          *reinterpret_cast<uint2*>(zt + ml * CF::kZPitch + BN + zc * 2) =
              make_uint2(pack_bf16x2(au[4 * e4 + 0], au[4 * e4 + 1]), pack_bf16x2(au[4 * e4 + 2], au[4 * e4 + 3]));
        }
    __syncthreads();
    {
      constexpr int kChunksRow = BN / 16;                // 8-column chunks of z per tile row
      constexpr int kPer = BM * kChunksRow / kThreads;   // chunks per thread
      static_assert(BM * kChunksRow % kThreads == 0, "whole chunks per thread");
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        const int q = t + kThreads * k, row = q / kChunksRow, ch = q % kChunksRow;
        uint4* gp = reinterpret_cast<uint4*>(zt + row * CF::kZPitch + 16 * ch);
        const uint4 gw = *gp;
        const uint4 uw = *reinterpret_cast<const uint4*>(zt + row * CF::kZPitch + BN + 16 * ch);
        const int64_t m = m0 + row;
        if (m < m_end) {
          *reinterpret_cast<uint4*>(Hc + m * 2 * p.F + zb + 8 * ch) = gw;
          *reinterpret_cast<uint4*>(Hc + m * 2 * p.F + p.F + zb + 8 * ch) = uw;
        }
        const uint32_t gs[4] = {gw.x, gw.y, gw.z, gw.w}, us[4] = {uw.x, uw.y, uw.z, uw.w};
        uint32_t z[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
          z[w] = (__float_as_uint(swiglu_bf16(bf16_lo(gs[w]), bf16_lo(us[w]))) >> 16) |
                 (__float_as_uint(swiglu_bf16(bf16_hi(gs[w]), bf16_hi(us[w]))) & 0xffff0000u);
        *gp = make_uint4(z[0], z[1], z[2], z[3]);
      }
    }
    __syncthreads();
    constexpr int QB = FmtTraits<FMT>::kBits;
    constexpr int ZC = BN / 2;  // z columns in the tile
    for (int q = t; q < BM * (ZC / 32); q += kThreads) {
      const int row = q / (ZC / 32), blk = q % (ZC / 32);
      if (m0 + row >= m_end) continue;
      float v[32];
      lds_row_block(zt, CF::kZPitch, row, blk * 32, v);
      const int64_t m = m0 + row, col = zb + 32 * blk;
      if (p.q_mode == kRceil)
        quant_store<FMT, kRceil, 0>(v, p.q_row_codes + code_group(m, col, p.R, QB), (int)((col >> 5) & 3), m,
                                    p.q_row_scales + scale_offset(m, col / 32, p.R));
      else
        quant_store<FMT, kFloor, 0>(v, p.q_row_codes + code_group(m, col, p.R, QB), (int)((col >> 5) & 3), m,
                                    p.q_row_scales + scale_offset(m, col / 32, p.R));
    }
    for (int q = t; q < ZC * (BM / 32); q += kThreads) {
      const int col = q % ZC, rb2 = q / ZC;
      if (m0 + 32 * rb2 >= m_end) continue;
      float v[32];
      lds_col_block(zt, CF::kZPitch, rb2 * 32, col, v);
      const int64_t cz = zb + col, m = m0 + 32 * rb2;
      if (p.q_mode == kRceil)
        quant_store<FMT, kRceil, 0>(v, p.q_col_codes + code_group(cz, m, p.F, QB), (int)((m >> 5) & 3), cz,
                                    p.q_col_scales + scale_offset(cz, m / 32, p.F));
      else
        quant_store<FMT, kFloor, 0>(v, p.q_col_codes + code_group(cz, m, p.F, QB), (int)((m >> 5) & 3), cz,
                                    p.q_col_scales + scale_offset(cz, m / 32, p.F));
    }
  } else {  // kEpiDSwiglu
    // dz = bf16(acc) is staged in LDS tile tg first.  Then each thread takes
    // 8-column chunks of the tile in row order: H's gate and up chunks of
    // that row arrive as coalesced 16-byte loads (a wavefront reads whole
    // 512-byte row segments), dz comes from LDS, d_gate replaces dz in tg
    // and d_up goes to tile tu.  Both tiles are then quantized rowwise and
    // columnwise out of LDS.
    uint8_t* tg = smem;
    uint8_t* tu = smem + BM * CF::kDPitch;
    const uint16_t* H = p.aux;
#pragma unroll
    for (int i = 0; i < CF::kMI; ++i)
#pragma unroll
      for (int j = 0; j < CF::kNJ; ++j)
#pragma unroll
        for (int e4 = 0; e4 < 4; ++e4) {
          const int ml = wm * CF::kWM + 32 * i + lrow;
          const int nl = wn * CF::kWN + 32 * j + 8 * e4 + 4 * g;
          const v16f& a = acc[i][j];
          *reinterpret_cast<uint2*>(tg + ml * CF::kDPitch + nl * 2) =
              make_uint2(pack_bf16x2(a[4 * e4 + 0], a[4 * e4 + 1]), pack_bf16x2(a[4 * e4 + 2], a[4 * e4 + 3]));
        }
    constexpr int kChunksRow = BN / 8;                    // 8-column chunks per tile row
    constexpr int kPer = BM * kChunksRow / kThreads;      // chunks per thread
    static_assert(BM * kChunksRow % kThreads == 0, "whole chunks per thread");
    // every H load of this thread in flight at once; rows past the group's
    // end (none while groups are 128-row multiples and BM = 128) read its
    // last row and are never stored
    uint4 hg[kPer], hu[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = t + kThreads * k, row = q / kChunksRow, ch = q % kChunksRow;
      const int64_t m = m0 + row;
      const uint16_t* hrow = H + (m < m_end ? m : m_end - 1) * 2 * p.F + n0 + 8 * ch;
      hg[k] = *reinterpret_cast<const uint4*>(hrow);
      hu[k] = *reinterpret_cast<const uint4*>(hrow + p.F);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int q = t + kThreads * k, row = q / kChunksRow, ch = q % kChunksRow;
      uint4* zp = reinterpret_cast<uint4*>(tg + row * CF::kDPitch + 16 * ch);
      const uint4 zw = *zp;
      const uint32_t zs[4] = {zw.x, zw.y, zw.z, zw.w};
      const uint32_t gs[4] = {hg[k].x, hg[k].y, hg[k].z, hg[k].w};
      const uint32_t us[4] = {hu[k].x, hu[k].y, hu[k].z, hu[k].w};
      uint32_t dg[4], du[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float g0, g1, u0, u1;
        dswiglu_pair_bf16(bf16_lo(zs[w]), bf16_lo(gs[w]), bf16_lo(us[w]), g0, u0);
        dswiglu_pair_bf16(bf16_hi(zs[w]), bf16_hi(gs[w]), bf16_hi(us[w]), g1, u1);
        dg[w] = (__float_as_uint(g0) >> 16) | (__float_as_uint(g1) & 0xffff0000u);
        du[w] = (__float_as_uint(u0) >> 16) | (__float_as_uint(u1) & 0xffff0000u);
      }
      const int64_t m = m0 + row;
      if (p.c && m < m_end)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.c) + m * p.F + n0 + 8 * ch) = zw;
      *zp = make_uint4(dg[0], dg[1], dg[2], dg[3]);
      *reinterpret_cast<uint4*>(tu + row * CF::kDPitch + 16 * ch) = make_uint4(du[0], du[1], du[2], du[3]);
    }
    __syncthreads();
    constexpr int QB = FmtTraits<FMT>::kBits;
    const int64_t W = 2 * p.F;  // dH width
    for (int q = t; q < 2 * BM * (BN / 32); q += kThreads) {
      const int half = q / (BM * (BN / 32)), rq = q % (BM * (BN / 32));
      const int row = rq / (BN / 32), blk = rq % (BN / 32);
      if (m0 + row >= m_end) continue;
      float v[32];
      lds_row_block(half ? tu : tg, CF::kDPitch, row, blk * 32, v);
      const int64_t m = m0 + row, col = (half ? p.F : 0) + n0 + 32 * blk;
      if (p.q_mode == kRceil)
        quant_store<FMT, kRceil, 0>(v, p.q_row_codes + code_group(m, col, p.R, QB), (int)((col >> 5) & 3), m,
                                    p.q_row_scales + scale_offset(m, col / 32, p.R));
      else
        quant_store<FMT, kFloor, 0>(v, p.q_row_codes + code_group(m, col, p.R, QB), (int)((col >> 5) & 3), m,
                                    p.q_row_scales + scale_offset(m, col / 32, p.R));
    }
    for (int q = t; q < 2 * BN * (BM / 32); q += kThreads) {
      const int half = q / (BN * (BM / 32)), cq = q % (BN * (BM / 32));
      const int col = cq % BN, rb2 = cq / BN;
      if (m0 + 32 * rb2 >= m_end) continue;
      float v[32];
      lds_col_block(half ? tu : tg, CF::kDPitch, rb2 * 32, col, v);
      const int64_t cw = (half ? p.F : 0) + n0 + col, m = m0 + 32 * rb2;
      if (p.q_mode == kRceil)
        quant_store<FMT, kRceil, 0>(v, p.q_col_codes + code_group(cw, m, W, QB), (int)((m >> 5) & 3), cw,
                                    p.q_col_scales + scale_offset(cw, m / 32, W));
      else
        quant_store<FMT, kFloor, 0>(v, p.q_col_codes + code_group(cw, m, W, QB), (int)((m >> 5) & 3), cw,
                                    p.q_col_scales + scale_offset(cw, m / 32, W));
    }
  }
}

}  // namespace

}  // namespace mx
