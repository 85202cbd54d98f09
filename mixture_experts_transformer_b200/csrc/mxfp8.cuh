// MXFP8 variant of the block: expert and shared Linears with e4m3 weights and
// e4m3 activations, both in groups of 32 along the reduction with one
// power-of-two scale per group (mxformat.cuh); the router stays bf16.
//
// Storage (also the tcgen05 block-scaled operand layout):
//   codes  [rows][K] bytes, K-major;
//   scales [ceil(rows/128)][ceil(K/128)][512] bytes (mx_sf_offset), rows and
//          groups past the end hold code 0.
//
// The GEMM (mx_gemm_kernel) has the NVFP4 GEMM's structure with
// `tcgen05.mma.kind::mxf8f6f4.block_scale.block32`: one 128-K stage is 128
// bytes of every operand row and exactly one scale atom per 128-row block, so
// a stage's scales are one 512-byte copy each; the MMA thread copies them to the
// stage's TMEM slot (tcgen05.cp) ahead of its MMAs - scale warps as in the NVFP4
// GEMM, whose stages hold four times the atoms, cost more than they saved (T = 64
// 200 -> 193 us without). The four 32-K MMAs of the stage pick their byte of the
// slot's words by the scale id of the instruction descriptor. A reduction that ends inside a stage (K a multiple
// of 64) issues only the MMAs it has.
//
// The MMA thread's own instructions set the pace where HBM does not: with descriptors built per MMA and one lane in the
// loops a stage took 770 cycles to issue (its MMAs run 512); a uniform warp with one elected lane takes 310 (T = 4096
// gate|up 256 -> 188 us, down 157 -> 132 us). What is left at T = 4096 is shared memory: a stage writes 48 KB and its
// MMAs read 48 KB, 768 cycles at 128 bytes a cycle against 512 of MMA, and gate|up takes 812 a stage (tensor pipe 66%
// busy); down adds the epilogue's staging and, with 6 stages a tile and TMEM for one 256-column accumulator beside the
// scales, waits for its epilogue (40%). At T = 64 the two stream the weights at 80% of the measured copy rate.
#pragma once

#include "grouped_gemm.cuh"
#include "mxformat.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"
#include "router.cuh"

namespace moe {

__host__ __device__ constexpr int mx_kblocks(int K) { return (K + 127) / 128; }

// ------------------------------------------------------------- quantisers

__device__ __forceinline__ void load32_bf16(const __nv_bfloat16* p, float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + q);
    const __nv_bfloat16* pa = reinterpret_cast<const __nv_bfloat16*>(&a);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[8 * q + i] = __bfloat162float(pa[i]);
  }
}

// One thread per (n, 32-group of K) of w [G][K][N] (N contiguous): codes into
// q [G][N][K], scale into the atoms of sf (cleared beforehand).
__global__ void mx_weight_quant_kernel(const __nv_bfloat16* __restrict__ w, int K, int N, uint8_t* __restrict__ q,
                                       uint8_t* __restrict__ sf) {
  pdl_wait_then_release();
  const size_t g = blockIdx.y;
  const int groups = K / kMxGroup;
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= static_cast<long long>(N) * groups) return;
  const int n = static_cast<int>(idx % N);
  const int kg = static_cast<int>(idx / N);
  const __nv_bfloat16* src = w + (g * K + kg * kMxGroup) * N + n;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __bfloat162float(src[static_cast<size_t>(i) * N]);
  uint4 codes[2];
  const uint32_t sc = mx_group(v, codes);
  uint4* dst = reinterpret_cast<uint4*>(q + (g * N + n) * K + kg * kMxGroup);
  dst[0] = codes[0];
  dst[1] = codes[1];
  const size_t nb = (N + 127) / 128;
  sf[g * nb * mx_kblocks(K) * 512 + mx_sf_offset(n, kg, mx_kblocks(K))] = static_cast<uint8_t>(sc);
}

// x [rows][K] bf16 -> q [rows][K], scale [rows][K/32]; one thread per group.
__global__ void mx_act_quant_kernel(const __nv_bfloat16* __restrict__ x, size_t groups, uint8_t* __restrict__ q,
                                    uint8_t* __restrict__ scale) {
  pdl_wait_then_release();
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < groups;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    float v[32];
    load32_bf16(x + i * kMxGroup, v);
    uint4 codes[2];
    scale[i] = static_cast<uint8_t>(mx_group(v, codes));
    reinterpret_cast<uint4*>(q)[2 * i] = codes[0];
    reinterpret_cast<uint4*>(q)[2 * i + 1] = codes[1];
  }
}

// The MXFP8 block's scatter: one warp per token, as route_scatter_fp4_kernel.
// The row's codes come from x (quantised here, once) or, already in MXFP8,
// from xq / xs (codes [T][D], scales [T][D/32]); each lane handles whole
// groups. Written: the codes and scale atoms of the token's k routed rows, the
// token-order scale atoms (the shared MLP's), and - without xq, which the shared
// MLP reads in place - the token-order codes. The blocks of a grid column (y) take
// every gridDim.y-th 32 groups: with one warp for a whole row too few loads were in
// flight. A store instruction of the warp covers 512 contiguous bytes of a row (each lane storing its own two pieces
// left half of every sector to the next instruction: T = 4096 35 us; now 26 us for 130 MB, 76% of the copy rate).
__global__ void __launch_bounds__(256) route_scatter_mx_kernel(
    const int32_t* __restrict__ idx, const uint32_t* __restrict__ masks, const int32_t* __restrict__ base, int T,
    int k, int E, int D, const __nv_bfloat16* __restrict__ x, const uint8_t* __restrict__ xq,
    const uint8_t* __restrict__ xs, int32_t* __restrict__ row_of, uint8_t* __restrict__ xq_perm,
    uint8_t* __restrict__ xsf_perm, uint8_t* __restrict__ xq_tok, uint8_t* __restrict__ xsf_tok, int rows,
    uint32_t* __restrict__ err) {
  __shared__ int s_rows[8][128];  // k <= num_experts <= 128
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int ng = D / kMxGroup, kb = mx_kblocks(D);
  for (int t = blockIdx.x * 8 + wid; t < T; t += gridDim.x * 8) {
    for (int j = lane; j < k; j += 32) {
      const size_t a = static_cast<size_t>(t) * k + j;
      const int e = __ldg(idx + a);
      int row = -1;
      if (e >= 0 && e < E) {
        const size_t cw = static_cast<size_t>(t / kMaskTokens) * E + e;
        const uint32_t below = __ldg(masks + cw) & ((1u << (t & (kMaskTokens - 1))) - 1u);
        row = __ldg(base + cw) + __popc(below);
        if (row < 0 || row >= rows) {  // never write outside the routed-row buffers
          atomicOr(err, kErrBadIndex);
          row = -1;
        } else {
          if (blockIdx.y == 0) row_of[a] = row;
        }
      }
      s_rows[wid][j] = row;
    }
    __syncwarp();
    for (int g0 = blockIdx.y * 32; g0 < ng; g0 += 32 * gridDim.y) {
      const int g = g0 + lane;
      const bool in = g < ng;
      // the 32 groups as 64 pieces of 16 bytes: pieces `lane` and 32 + lane are this lane's to store
      const int p0 = 2 * g0 + lane, p1 = p0 + 32;
      const bool in0 = p0 < 2 * ng, in1 = p1 < 2 * ng;
      uint4 c0 = make_uint4(0, 0, 0, 0), c1 = c0;
      uint32_t sc = 0;
      if (xq) {
        const uint4* src = reinterpret_cast<const uint4*>(xq + static_cast<size_t>(t) * D);
        if (in0) c0 = __ldg(src + p0);
        if (in1) c1 = __ldg(src + p1);
        if (in) sc = __ldg(xs + static_cast<size_t>(t) * ng + g);
      } else {
        uint4 codes[2] = {c0, c0};
        if (in) {
          float v[32];
          load32_bf16(x + static_cast<size_t>(t) * D + g * kMxGroup, v);
          sc = mx_group(v, codes);
        }
        // lane l has pieces 2 l and 2 l + 1
        const int from = lane >> 1;
        auto piece = [&](int lane_of) -> uint4 {
          const uint4 a = codes[0], b = codes[1];
          uint4 lo, hi;
          lo.x = __shfl_sync(0xffffffffu, a.x, lane_of), hi.x = __shfl_sync(0xffffffffu, b.x, lane_of);
          lo.y = __shfl_sync(0xffffffffu, a.y, lane_of), hi.y = __shfl_sync(0xffffffffu, b.y, lane_of);
          lo.z = __shfl_sync(0xffffffffu, a.z, lane_of), hi.z = __shfl_sync(0xffffffffu, b.z, lane_of);
          lo.w = __shfl_sync(0xffffffffu, a.w, lane_of), hi.w = __shfl_sync(0xffffffffu, b.w, lane_of);
          return lane & 1 ? hi : lo;
        };
        c0 = piece(from);
        c1 = piece(16 + from);
        uint4* qt = reinterpret_cast<uint4*>(xq_tok + static_cast<size_t>(t) * D);
        if (in0) qt[p0] = c0;
        if (in1) qt[p1] = c1;
      }
      // the four scales of a 128-K block are one aligned word of the atom
      uint32_t scw = sc << (8 * (lane & 3));
      scw |= __shfl_xor_sync(0xffffffffu, scw, 1);
      scw |= __shfl_xor_sync(0xffffffffu, scw, 2);
      const bool word = in && (lane & 3) == 0;
      if (word) *reinterpret_cast<uint32_t*>(xsf_tok + mx_sf_offset(t, g, kb)) = scw;
      for (int j = 0; j < k; ++j) {
        const int row = s_rows[wid][j];
        if (row < 0) continue;
        uint4* qp = reinterpret_cast<uint4*>(xq_perm + static_cast<size_t>(row) * D);
        if (in0) qp[p0] = c0;
        if (in1) qp[p1] = c1;
        if (word) *reinterpret_cast<uint32_t*>(xsf_perm + mx_sf_offset(row, g, kb)) = scw;
      }
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------- MXFP8 GEMM

constexpr int kMxKStage = 128;                    // K elements (= bytes of a row) per stage
constexpr int kMxABytes = 128 * kMxKStage;        // 128 rows
constexpr int kMxSfBytes = 512;                   // one atom per 128-row block
constexpr int kMxProd1 = 10;                      // warps of copying threads 1 and 2 (thread 0: warp 0)
constexpr int kMxThreads = 32 * (kMxProd1 + 2);   // copy, MMA, 8 epilogue, 2 copy warps
constexpr int kMxASmallRows = 32;                 // rows of the small A boxes
constexpr int kMxAMidRows = 64;
constexpr int kMxBBytes = 2 * 128 * kMxKStage;    // two 128-row blocks
constexpr int kMxStages = 4;
constexpr int kMxStgWarpBytes = 2048;             // epilogue staging per warp (32 rows x 64 B)
constexpr int kMxSmemBytes =
    kMxStages * (kMxABytes + kMxBBytes + 3 * kMxSfBytes) + 8 * kMxStgWarpBytes + 1024 + 512;

struct MxProblem {
  int K;          // multiple of 64
  int N;          // multiple of 64
  int groups;
  int a_rows;     // rows the tiles may start in (a multiple of 128)
  const uint8_t* sfa;   // [a_rows/128][ceil(K/128)][512]
  const uint8_t* sfb0;  // [groups][ceil(N/128)][ceil(K/128)][512]
  const uint8_t* sfb1;  // (up; GATEUP only)
  void* out;            // GATEUP: codes [rows][N]; DOWN: bf16 / fp32 [rows][ldo]
  uint8_t* out_sf;      // GATEUP: scales [rows/128][ceil(N/128)][512]
  int ldo;
  int out_f32;
};

struct MxParams {
  CUtensorMap tmA[2];   // codes [rows][K] u8, box 128 x 128, 128-byte swizzle
  CUtensorMap tmAs[2];  // the same, boxes 128 x 32 and 128 x 64: tiles of at most as many rows copy only those
  CUtensorMap tmAm[2];
  CUtensorMap tmB0[2];  // codes [groups][N][K] u8, box 128 x 128 x 1
  CUtensorMap tmB1[2];
  CUtensorMap tmBw[2];  // down: box 128 x 256 x 1
  MxProblem prob[2];
  int nprob;
  const Tile* tiles;
  const int32_t* num_tiles;
  int32_t* next_tile;
  uint32_t* err;
};

// Instruction descriptor of kind::mxf8f6f4 (e4m3 A and B, ue8m0 scales),
// K-major A and B, M = 128; sf_id picks the scale byte of A's and B's words.
__host__ __device__ constexpr uint32_t idesc_mxf8_m128(int n, int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4)        // B scale id
         | (static_cast<uint32_t>(n >> 3) << 17)    // N / 8
         | (1u << 23)                               // scales are ue8m0
         | (static_cast<uint32_t>(128 >> 4) << 24)    // M / 16
         | (static_cast<uint32_t>(sf_id) << 29);    // A scale id
}
// the two scale ids alone
__host__ __device__ constexpr uint32_t idesc_mxf8_sf(int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4) | (static_cast<uint32_t>(sf_id) << 29);
}

// The two words of an sdesc_sw128 descriptor: only the low one moves with the address (+ bytes / 16), so an MMA thread
// adds to it instead of building 64-bit descriptors - its instruction stream is what a chunk or stage waits for
// otherwise (few-token kernel: 16 MMAs with built descriptors took 0.6 us to issue; here the 4 of a stage 770 cycles).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) { return (saddr >> 4) | ((lbo >> 4) << 16); }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }

__device__ __forceinline__ void umma_mxf8(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                          uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], a, b, %5, [%7], [%8], p;\n\t}" ::"r"(d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// A 512-byte scale tile from shared memory into 4 TMEM columns of every lane quarter (row i of 16 bytes to lane i).
// In order with this thread's MMAs. The column has to be a multiple of 4. Descriptor: no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr) {
  asm volatile(
      "{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\ttcgen05.cp.cta_group::1.32x128b.warpx4 [%0], a;\n\t}" ::"r"(taddr),
      "r"(saddr >> 4), "r"((128u >> 4) | (1u << 14))
      : "memory");
}

// What an epilogue warp does with its 32 rows (rows_valid of them, from row on) of a tile's accumulator, a row a thread:
// GeGLU and MXFP8 codes, or output rows through the warp's staging buffer (whole-sector stores in row order). Routed rows
// are rounded to bf16 for the combine, as in the bf16 block: in fp32 they would add 185 MB written and as much read at T =
// 4096, 56 us of 490 at the copy rate, for an error of 0.0017 of the output that is nearly all its own rounding to bf16
// (0.00173 -> 0.00177). The shared rows stay fp32.
template <bool GATEUP>
__device__ __forceinline__ void mx_epilogue(const MxProblem& pr, uint32_t (&acc)[4][32], int rows_valid, int row, int n0,
                                            int wn, int half, int lane, uint8_t* stg) {
  if (rows_valid <= 0) return;
  if constexpr (GATEUP) {
    const int kbo = mx_kblocks(pr.N);
    uint8_t* q = reinterpret_cast<uint8_t*>(pr.out) + static_cast<size_t>(row + lane) * pr.N + n0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int j = half * 32 + 64 * c;
      if (j >= wn) continue;
      float v[32];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        v[i] = gelu_tanh_exact(__uint_as_float(acc[2 * c][i])) * __uint_as_float(acc[2 * c + 1][i]);
      uint4 codes[2];
      const uint32_t sc = mx_group(v, codes);
      if (lane < rows_valid) {
        reinterpret_cast<uint4*>(q + j)[0] = codes[0];
        reinterpret_cast<uint4*>(q + j)[1] = codes[1];
        pr.out_sf[mx_sf_offset(row + lane, (n0 + j) / 32, kbo)] = static_cast<uint8_t>(sc);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int j = half * 32 + 64 * c;
      if (j >= wn) continue;
      uint32_t* a = acc[c];
      const size_t at = static_cast<size_t>(row) * pr.ldo + n0 + j;
      if (pr.out_f32) {
        uint8_t* base = reinterpret_cast<uint8_t*>(reinterpret_cast<float*>(pr.out) + at);
#pragma unroll
        for (int q = 0; q < 4; ++q) store_rows_32B(stg, a + 8 * q, lane, base + 32 * q, pr.ldo * 4, rows_valid);
      } else {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
        store_rows_bf16x32(stg, pk, lane, reinterpret_cast<__nv_bfloat16*>(pr.out) + at, pr.ldo, rows_valid);
      }
    }
  }
}

// A value that is the same in all lanes, marked so for the compiler: what it computes from such values it keeps in
// uniform registers, which is where the tensor instructions take their operands from.
__device__ __forceinline__ int warp_uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// TMEM columns [0, 256): the accumulator (GATEUP: gate 0..127, up 128..255;
// DOWN: output columns n0 .. n0+255); from 256: one scale slot per stage, A
// scales at +0, B block 0 at +4, B block 1 at +8.
template <bool GATEUP>
__global__ void __launch_bounds__(kMxThreads, 1) mx_gemm_kernel(const __grid_constant__ MxParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + kMxStages * kMxABytes;
  uint8_t* sSf = sB + kMxStages * kMxBBytes;  // per stage: A atom, B block 0 atom, B block 1 atom
  uint8_t* sStg = sSf + kMxStages * 3 * kMxSfBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sStg + 8 * kMxStgWarpBytes);
  uint64_t* empty = full + kMxStages;
  uint64_t* acc_full = empty + kMxStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* drain = acc_empty + 1;
  uint64_t* tile_full = drain + 1;
  uint64_t* tile_empty = tile_full + kTileRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tile_empty + kTileRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int4* tile_ring = reinterpret_cast<int4*>((reinterpret_cast<uintptr_t>(tmem_slot + 2) + 15) & ~uintptr_t(15));

  const int warp = warp_uniform(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 8);  // one arrival per epilogue warp
    mbar_init(drain, 1);
    for (int r = 0; r < kTileRing; ++r) {
      mbar_init(&tile_full[r], 1);
      mbar_init(&tile_empty[r], 1 + 8 + 2);  // MMA thread, epilogue and copy warps read each index
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    for (int p = 0; p < P.nprob; ++p) {
      tma_prefetch_desc(&P.tmA[p]);
      tma_prefetch_desc(&P.tmAs[p]);
      tma_prefetch_desc(&P.tmB0[p]);
      tma_prefetch_desc(GATEUP ? &P.tmB1[p] : &P.tmBw[p]);
    }
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  // The kernel may start while the one that makes A runs (the scatter; for down the gate|up GEMM): that one has passed
  // its own wait, so the tile list of the scan before it is there. Weights and tiles are read ahead, only thread 0, which
  // copies A, waits; nothing is computed or written without A. (4 us of 162 at T = 64. The list is read past L1, which may
  // hold an earlier call's.)
  // Tiles: the producer takes their indices from the work counter and publishes the tiles in the ring (pg, row0, rows,
  // n0; pg -1 ends the work), the other roles read them in order.
  int rs = 0;
  uint32_t rph = 0;
  auto next_tile = [&](bool whole_warp) -> Tile {
    int4 v = make_int4(-1, 0, 0, 0);
    if (lane == 0) {
      if (mbar_wait_cycles(&tile_full[rs], rph, abort_flag, P.err)) {
        v = tile_ring[rs];
        mbar_arrive(&tile_empty[rs]);
      }
    }
    if (whole_warp) v = make_int4(warp_uniform(v.x), warp_uniform(v.y), warp_uniform(v.z), warp_uniform(v.w));
    if (++rs == kTileRing) {
      rs = 0;
      rph ^= 1;
    }
    return Tile{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
  };

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------ TMA producer
      int s = 0, issued = 0;
      uint32_t ph = 0;
      bool waited = false;
      const int num_tiles = __ldcg(P.num_tiles);
      int ti = atomicAdd(P.next_tile, 1);
      while (true) {
        if (!mbar_wait_cycles(&tile_empty[rs], rph ^ 1, abort_flag, P.err)) break;
        const int4 tv = ti < num_tiles ? __ldcg(reinterpret_cast<const int4*>(P.tiles + ti)) : make_int4(-1, 0, 0, 0);
        const Tile tile{tv.x, tv.y, tv.z, tv.w, 0, 0, 0, 0};
        const int p = tile.pg >> 16, g = tile.pg & 0xFFFF;
        bool ok = true;
        if (ti < num_tiles) {  // checked before the other roles see the tile
          ok = tile.pg >= 0 && p < P.nprob;
          if (ok) {
            const MxProblem& pr = P.prob[p];
            ok = g < pr.groups && tile.row0 >= 0 && tile.row0 < pr.a_rows && !(tile.row0 & 127) && tile.n0 >= 0 &&
                 tile.n0 < pr.N && !(tile.n0 & 127);
          }
          if (!ok) atomicOr(P.err, kErrBadTile);
        }
        tile_ring[rs] = ok ? tv : make_int4(-1, 0, 0, 0);
        mbar_arrive(&tile_full[rs]);
        if (++rs == kTileRing) {
          rs = 0;
          rph ^= 1;
        }
        if (!ok || ti >= num_tiles) break;
        if (!waited) pdl_wait_then_release();
        waited = true;
        const int next = atomicAdd(P.next_tile, 1);  // its latency hides behind this tile's loads
        const MxProblem& pr = P.prob[p];
        const int kb = mx_kblocks(pr.K);
        const uint8_t* sfa = pr.sfa + static_cast<size_t>(tile.row0 >> 7) * kb * 512;
        const bool two_b = GATEUP || (tile.n0 + 128 < pr.N);
        const bool small = tile.rows <= kMxASmallRows, mid = !small && tile.rows <= kMxAMidRows;
        const CUtensorMap* ma = small ? &P.tmAs[p] : mid ? &P.tmAm[p] : &P.tmA[p];
        const uint32_t bytes = (small ? kMxASmallRows * kMxKStage : mid ? kMxAMidRows * kMxKStage : kMxABytes) +
                               (two_b ? 2 : 1) * (kMxBBytes / 2) + kMxSfBytes * (two_b ? 3 : 2);
        for (int ks = 0; ks < kb; ++ks) {
          if (!mbar_wait_cycles(&empty[s], ph ^ 1, abort_flag, P.err)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], bytes);
          tma_load_2d(sA + s * kMxABytes, ma, &full[s], ks * kMxKStage, tile.row0);
          bulk_load(sSf + s * 3 * kMxSfBytes, sfa + static_cast<size_t>(ks) * 512, kMxSfBytes, &full[s]);
          ++issued;
          if (++s == kMxStages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        ti = next;
      }
      if (*abort_flag) {  // wait for the copies in flight before the CTA's shared memory goes away
        int st = s;
        uint32_t sp = ph;
        const int pending = issued < kMxStages ? issued : kMxStages;
        for (int i = 0; i < pending; ++i) {
          if (--st < 0) {
            st = kMxStages - 1;
            sp ^= 1;
          }
          uint32_t dummy = 0;
          mbar_wait_cycles(&full[st], sp, reinterpret_cast<volatile int*>(&dummy), P.err, kWaitTimeoutCycles / 20);
        }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    // The whole warp walks the loops and one lane issues. (With one lane in the loops the operands were moved to
    // uniform registers one by one for every instruction.)
    int s = 0;
    uint32_t ph = 0, acc_ph = 0;
    bool any = false;
    while (true) {
      const Tile tile = next_tile(true);
      if (tile.pg < 0) break;
      const MxProblem& pr = P.prob[tile.pg >> 16];
      const int K = warp_uniform(pr.K);
      const bool two_b = warp_uniform(GATEUP || (tile.n0 + 128 < pr.N));
      const uint32_t idesc = idesc_mxf8_m128(two_b ? 256 : 128, 0);
      if (!__all_sync(0xffffffffu, mbar_wait_cycles(acc_empty, acc_ph ^ 1, abort_flag, P.err))) break;
      tc_fence_after_sync();
      bool ok = true;
      for (int k0 = 0; k0 < K; k0 += kMxKStage) {
        if (!__all_sync(0xffffffffu, mbar_wait_cycles(&full[s], ph, abort_flag, P.err))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t al = desc_lo(smem_u32(sA + s * kMxABytes), 16), bl = desc_lo(smem_u32(sB + s * kMxBBytes), 16);
        const uint32_t slot = tmem_base + kAccCols + s * 16, sf = smem_u32(sSf + s * 3 * kMxSfBytes);
        if (elect_one()) {
          // the stage's scale atoms, in order before its MMAs; the slot's last readers were done when the stage was refilled
          tmem_cp_scales(slot, sf);
          tmem_cp_scales(slot + 4, sf + kMxSfBytes);
          if (two_b) tmem_cp_scales(slot + 8, sf + 2 * kMxSfBytes);
          // 32 K of e4m3 = 32 B per row inside the 128-byte swizzled rows; both B blocks are consecutive halves of the
          // stage and their scale words sit at +4 and +8: one MMA of N = 256 covers both
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j == 2 && K - k0 <= 64) break;
            umma_mxf8(tmem_base, al + j * 2, desc_hi(1024), bl + j * 2, desc_hi(1024), idesc + idesc_mxf8_sf(j), slot,
                      slot + 4, j != 0 || k0 != 0);
          }
          umma_commit(&empty[s]);
        }
        __syncwarp();
        any = true;
        if (++s == kMxStages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (elect_one()) umma_commit(acc_full);
      acc_ph ^= 1;
    }
    if (any && elect_one()) {
      umma_commit(drain);
      uint32_t dummy = 0;
      mbar_wait_cycles(drain, 0, reinterpret_cast<volatile int*>(&dummy), P.err);
    }
    __syncwarp();
  } else if (warp >= kMxProd1) {
    // --------------------------------------------------- copy threads 1, 2
    // B and its scale atoms: thread 1 the gate weights (down: all 256 rows, or
    // the only 128), thread 2 the up weights (down: the atoms). A copy may land before
    // thread 0 announces the stage's bytes; the stage completes with both.
    if (lane == 0) {
      const bool up = warp != kMxProd1;
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok) {
        const Tile tile = next_tile(false);
        if (tile.pg < 0) break;
        const int p = tile.pg >> 16, g = tile.pg & 0xFFFF;
        const MxProblem& pr = P.prob[p];
        const int kb = mx_kblocks(pr.K);
        const size_t atom = (static_cast<size_t>(g) * ((pr.N + 127) / 128) + (tile.n0 >> 7)) * kb;
        const bool two_b = GATEUP || (tile.n0 + 128 < pr.N);
        const CUtensorMap* m = GATEUP ? (up ? &P.tmB1[p] : &P.tmB0[p]) : two_b ? &P.tmBw[p] : &P.tmB0[p];
        const uint8_t* src = (GATEUP && up ? pr.sfb1 : pr.sfb0) + atom * 512;
        for (int ks = 0; ks < kb; ++ks) {
          if (!mbar_wait_cycles(&empty[s], ph ^ 1, abort_flag, P.err)) {
            ok = false;
            break;
          }
          uint8_t* sf = sSf + s * 3 * kMxSfBytes + kMxSfBytes;
          if (GATEUP || !up)
            tma_load_3d(sB + s * kMxBBytes + (up ? kMxBBytes / 2 : 0), m, &full[s], ks * kMxKStage, tile.n0, g);
          if (GATEUP) {
            bulk_load(sf + (up ? kMxSfBytes : 0), src + static_cast<size_t>(ks) * 512, kMxSfBytes, &full[s]);
          } else if (up) {
            bulk_load(sf, src + static_cast<size_t>(ks) * 512, kMxSfBytes, &full[s]);
            if (two_b) bulk_load(sf + kMxSfBytes, src + static_cast<size_t>(kb + ks) * 512, kMxSfBytes, &full[s]);
          }
          if (++s == kMxStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue
    // warps 2..9: TMEM lane quarter warp % 4, column half (warp - 2) / 4;
    // 32-column chunks j = half * 32 + 64 c, which are whole MXFP8 groups
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    uint32_t acc_ph = 0;
    while (true) {
      const Tile tile = next_tile(true);
      if (tile.pg < 0) break;
      const MxProblem& pr = P.prob[tile.pg >> 16];
      const int wn = min(GATEUP ? 128 : 256, pr.N - tile.n0);
      int got = 1;
      if (lane == 0) got = mbar_wait_cycles(acc_full, acc_ph, abort_flag, P.err);
      if (!__shfl_sync(0xffffffffu, got, 0)) break;
      tc_fence_after_sync();
      acc_ph ^= 1;
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
      // all of a thread's accumulator values first, so that the next tile's MMAs start before this one's arithmetic
      uint32_t acc[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)  // GATEUP: gate, up of columns half * 32 .., then of those 64 further
        tmem_ld_32x32b_x32(tbase + half * 32 + (GATEUP ? 64 * (c >> 1) + 128 * (c & 1) : 64 * c), acc[c]);
      tmem_ld_wait();
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);
      mx_epilogue<GATEUP>(pr, acc, tile.rows - quarter * 32, tile.row0 + quarter * 32, tile.n0, wn, half, lane,
                          sStg + (warp - 2) * kMxStgWarpBytes);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

}  // namespace moe
