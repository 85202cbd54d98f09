// The whole MoE layer for a few tokens (T <= 16) in two kernels: a small one for
// the router's logits and x as MMA operands (norm_pre, or MXFP8 quantisation),
// and one cooperative kernel for top-k, experts, shared MLP, combine and (bf16
// form) norm_post and residual.
//
// A few tokens read every touched expert's weights once and compute almost
// nothing per byte, so the layer is bound by HBM: the kernel is built as one
// uninterrupted stream of weight chunks per SM. Split over several kernels,
// that stream stops at every kernel boundary and at every wave's ragged end;
// here
//   * the work of each phase is one list of 32 KB weight chunks (gate|up: 128
//     output columns of both, down: 256 columns; 64 K deep in bf16, 128 K in 8
//     bits), cut into equal contiguous ranges, one per CTA, wherever that
//     falls inside an output column's reduction; CTAs that share a column
//     leave fp32 partial sums, and the last of them adds them up in CTA order;
//   * producer threads keep a ring of TMA copies full across the phases: the
//     shared MLP's chunks need no routing, so they stream while the experts are
//     chosen, and the first down chunks are already in flight while the last
//     GeGLU rows are being finished elsewhere. (They start when the small kernel
//     has ended: the barrier behind this kernel's wait for it holds every warp.)
//
// Phases (chunk lists): S the shared MLP's gate|up, E the touched experts'
// gate|up, D all down projections: for each 256 output columns the shared MLP's
// reduction, then each touched expert's. Grid-wide waits: D needs all GeGLU rows,
// the output all parts of D. The grid is launched cooperatively (all CTAs
// resident), and every wait is bounded. The router as a phase of this kernel put
// two more such hand-overs before the first expert chunk (routing known 11.9 us
// after the start at T = 1).
//
// Products: tcgen05.mma with the weight columns as M = 128 and the tokens as
// N = 16, one lane issuing 8 MMAs per chunk, so the SM's issue slots play no
// part. (With mma.sync on eight warps - M = 16 tiles of columns, N = 8 or 16 -
// the MXFP8 form executed 136 instructions per 32 K of a warp's tile and took
// 155 us at T = 8; its chunks cost 1.9 us each against 0.75 us of HBM time.)
// Every token's column is computed for every touched expert; a token takes an
// expert's result only if it is routed there (a select, so that nothing of an
// expert reaches other tokens).
//
// Measured (embed 2816, 128 experts of 704, top-8, shared 2112; of the measured copy rate): bf16 T = 1 45 us (45%),
// 5 with norms 106 us (66%), 16 173-187 us (83-90%: 972 MB from HBM); MXFP8 T = 1 37 us, 8 70 us (73%). Outside the
// stream: the small kernel and the gap to this one 6 us, the hand-over to D 7 us (every CTA waits for all GeGLU rows, also
// those of sources that it does not read next), the output 4 us.
//
// Numerics: fp32 accumulation. bf16 form: the GeGLU rows enter the down product as
// the sum of two bf16 values (hi + lo, 16 bits of mantissa), the routed sums are
// weighted and added in fp32: nothing is rounded to bf16 before the output
// (and after norm_pre). MXFP8 form: GeGLU rows in MXFP8, as the large-batch path.
#pragma once

#include "mxformat.cuh"
#include "mxfp8.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kFewMaxTokens = 16;
constexpr int kFewMaxTopK = 32;
constexpr int kFewMaxDim = 4096;  // at most 16 CTAs share the router's reduction
constexpr int kFewPrepThreads = 512;
constexpr int kFewConsWarps = 8;
constexpr int kFewProdWarps = 4;  // copying threads 0..3, one a warp (the TMEM lane quarter of warp w is w % 4)
constexpr int kFewMmaWarp = kFewProdWarps + 2 * kFewConsWarps;  // after 8 consumer and 8 routing warps
constexpr int kFewProdWarp4 = kFewMmaWarp + 1;                  // copying thread 4
constexpr int kFewThreads = 32 * (kFewMmaWarp + 2);
constexpr int kFewWBytes = 32768;    // weights of a chunk
constexpr int kFewSfBytes = 1024;    // MXFP8: two scale tiles of a chunk
constexpr int kFewRouterRows = 256;  // K rows of the router per CTA of the small kernel
constexpr int kFewGuCols = 128;      // output columns of a gate|up chunk, per projection
constexpr int kFewDnCols = 256;      // output columns of a down chunk
constexpr int kFewMaxStages = 8;
constexpr int kFewMaxCtas = 148;
constexpr int kFewMaxHidden = 16384;  // at most 128 units of the shared MLP, fewer than CTAs
constexpr int kFewTmemCols = 256;    // two accumulators, then (MXFP8) 16 columns of scales per stage
constexpr int kFewTmemAcc = 64;      // columns of an accumulator: two M tiles of 16, bf16 down of up to 32 (high, low parts)
constexpr int kFewTmemSf = 128;

// ------------------------------------------------------ shared host / device sizes

template <bool MX>
__host__ __device__ constexpr int few_kc() {  // K elements of a chunk: 128 bytes of a K-major operand row
  return MX ? 128 : 64;
}
// Token rows of the MMA's B operand in memory: bf16 with at most 8 tokens keeps 8 (the other 8 columns read them
// again through a stride of 0).
template <bool MX>
__host__ __device__ constexpr int few_rows(int T) {
  return !MX && T <= 8 ? 8 : 16;
}
// B operand of one K chunk - x for gate|up, the GeGLU rows for down: rows x 128 bytes (128-byte swizzle); the bf16
// GeGLU rows as high parts, then low parts; MXFP8 codes, then a scale tile
template <bool MX>
__host__ __device__ constexpr int few_xchunk(int rows) {
  return MX ? rows * 128 + 512 : rows * 128;
}
template <bool MX>
__host__ __device__ constexpr int few_hchunk(int rows) {
  return MX ? rows * 128 + 512 : 2 * rows * 128;
}
template <bool MX>
__host__ __device__ constexpr int few_stage_bytes(int rows) {
  return kFewWBytes + (MX ? kFewSfBytes : 0) + ((few_hchunk<MX>(rows) + 1023) & ~1023);
}
constexpr int kFewFixedBytes = 128 * 16 * 4 + 128 * 4 + 128            // weights, token masks, list of the touched experts
                               + kFewMaxTokens * kFewMaxTopK * 5         // selected logits and experts
                               + 3 * (kFewMaxCtas + 1) * 4 + 2 * 16 * 4  // ranges of the phases, CTAs of the output tiles
                               + 512 /* barriers, flags */ + 1024 /* alignment */;

struct FewParams {
  // experts (tmS*: shared). bf16 [el][K][N] in 64-column blocks of 64 K: G, U two adjacent blocks per copy, D four.
  // MXFP8 [el][N][K]: G, U 128 B x 128 rows, D 128 B x 256 rows. 128-byte swizzle.
  CUtensorMap tmG, tmU, tmD;
  CUtensorMap tmSg, tmSu, tmSd;
  const uint8_t* sfg;  // MXFP8 scale tiles
  const uint8_t* sfu;
  const uint8_t* sfd;
  const uint8_t* sfsg;
  const uint8_t* sfsu;
  const uint8_t* sfsd;
  int T, k, D, E, F, S, e0, el;
  int stages;
  const __nv_bfloat16* x;
  const uint8_t* xq;  // MXFP8: the rows in 8 bits (optional)
  const uint8_t* xs;
  const __nv_bfloat16* norm_pre;
  uint8_t* xb;  // x as B operands, one few_xchunk per K chunk
  const __nv_bfloat16* w_router;
  const __nv_bfloat16* norm_post;
  int residual;
  const float* bias;
  uint32_t* counters;  // cleared by few_prep_kernel: hidden, down, shared, rows, then (8) one per E unit
  int ncounters;
  float* logit_part;   // [ceil(D / 256)][16][128]
  uint8_t* h;          // GeGLU rows, one few_hchunk per K chunk of down
  float* part_gu;      // [CTA][2 phases][2][2 projections][16][128]
  float* f;            // [T][D] the sums before norm_post / residual
  float* part_dn;      // [CTA][2][16][256]
  __nv_bfloat16* out;
  float* out_f32;
  int32_t* idx_out;
  float* w_out;
  int32_t* cnt_out;
  float* logits_out;
  uint32_t* err;
};

// How a phase's list of `total` chunks is cut: a range of base or base + 1 chunks per CTA (at most one CTA per chunk, so
// that no range is empty). A chunk that lies half outside its matrix counts as a whole one: it holds a ring stage as
// long (weighting it half gave its CTAs ranges with half the bytes in flight: T = 1 48 -> 58 us).
struct FewSplit {
  int total, ctas, base, rem;
  __device__ FewSplit(int total_, int grid) : total(total_) {
    ctas = max(1, min(total, grid));
    base = total / ctas;
    rem = total - base * ctas;
  }
  __device__ int begin(int c) const { return c >= ctas ? total : c * base + min(c, rem); }
  // the CTA whose range holds chunk i
  __device__ int cta_of(int i) const {
    const int big = rem * (base + 1);
    return i < big ? i / (base + 1) : rem + (i - big) / base;
  }
};

// ------------------------------------------------------------ small PTX pieces

__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// generic-proxy accesses of this thread <-> async-proxy (bulk copy, MMA) accesses
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Wait until *p >= want; bounded as mbar_wait_cycles.
__device__ __forceinline__ bool counter_wait(const uint32_t* p, uint32_t want, volatile int* abort, uint32_t* err) {
  if (ld_acquire(p) >= want) return true;
  const long long t0 = clock64();
  while (true) {
    if (ld_acquire(p) >= want) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitTimeoutCycles) {
      *abort = 1;
      atomicOr(err, kErrWaitTimeout);
      return false;
    }
  }
}

// 8 / 16 consecutive fp32 TMEM columns of this warp's 32 lanes (one row per thread).
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// kind::f16, bf16, M = 128, A with its M index contiguous (bit 15), B K-major.
__host__ __device__ constexpr uint32_t few_idesc_bf16(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void few_umma_bf16(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// fp32 (no NaN) as an unsigned integer of the same order; zeros of either sign are equal, -infinity is above 0
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = v == 0.f ? 0u : __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Byte of (token row t, 16-byte piece p) in a block of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swz128(int t, int p) { return t * 128 + ((p ^ (t & 7)) << 4); }

// The small kernel. CTA c: partial logits of all tokens over K rows 256 c .. (fp32 multiply-adds of bf16 values, a
// thread four experts over 16 rows, the 16 row groups added in order), token c as B operands, a share of the counters
// cleared. Rows past T of the operands are left as they are: a token is a column of every product, and columns past T
// are never read.
template <bool MX>
__global__ void __launch_bounds__(kFewPrepThreads) few_prep_kernel(const __grid_constant__ FewParams P) {
  constexpr int kWarps = kFewPrepThreads / 32;
  constexpr int kRowsPer = kFewRouterRows / kWarps;  // K rows of a warp
  constexpr int kTB = 4;                             // tokens per pass
  __shared__ __align__(16) __nv_bfloat16 s_x[kFewMaxTokens][kFewRouterRows];
  __shared__ float4 s_part[kWarps][kTB][32];
  __shared__ float s_rms[kFewMaxTokens];
  const int c = blockIdx.x, tx = threadIdx.x, lane = tx & 31, warp = tx >> 5;
  // the slice's weights into L2 while the previous kernel ends (a prefetch reads no value: it may come early)
  if (tx < kFewRouterRows && c * kFewRouterRows + tx < P.D)
    for (int o = 0; o < P.E; o += 64)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(P.w_router + static_cast<size_t>(c * kFewRouterRows + tx) * P.E + o));
  pdl_wait_then_release();
  for (int i = c * kFewPrepThreads + tx; i < P.ncounters; i += gridDim.x * kFewPrepThreads) P.counters[i] = 0;
  const int D = P.D, nvec = D >> 3;  // 16-byte vectors of a bf16 row
  const uint4* xrow = reinterpret_cast<const uint4*>(P.x);
  const int k0 = c * kFewRouterRows;
  const bool route = k0 < D, lay = c < P.T;
  // the router's weights of this thread: experts 4 lane .., its warp's 16 rows
  uint2 w[kRowsPer];
  const bool in = route && lane * 4 < P.E;
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    const int k = k0 + warp * kRowsPer + i;
    w[i] = in && k < D ? __ldg(reinterpret_cast<const uint2*>(P.w_router + static_cast<size_t>(k) * P.E) + lane)
                       : make_uint2(0, 0);
  }
  if constexpr (!MX) {
    if (P.norm_pre) {  // 1 / rms of every row, a warp each
      if (warp < P.T) {
        float ss = 0.f;
#pragma unroll 4
        for (int v = lane; v < nvec; v += 32) {
          const uint4 q = __ldg(xrow + static_cast<size_t>(warp) * nvec + v);
          const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(&q);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(__bfloat162float(b[i]), __bfloat162float(b[i]), ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) s_rms[warp] = 1.0f / sqrtf(ss / static_cast<float>(D) + 1e-6f);
      }
      __syncthreads();
    }
  }
  // eight values of row t, after norm_pre (rounded to bf16: the layer's input)
  auto load_x = [&](int t, int v) -> uint4 {
    uint4 q = __ldg(xrow + static_cast<size_t>(t) * nvec + v);
    if (!MX && P.norm_pre) {
      const uint4 gv = __ldg(reinterpret_cast<const uint4*>(P.norm_pre) + v);
      const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(&q);
      const __nv_bfloat16* g = reinterpret_cast<const __nv_bfloat16*>(&gv);
      const float r = s_rms[t];
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __bfloat162float(b[j]) * r * __bfloat162float(g[j]);
      q = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    }
    return q;
  };
  if (lay) {  // token c: at most one vector per thread
    static_assert(kFewMaxDim / 8 <= kFewPrepThreads, "a row fits the block");
    const int v = tx;
    if constexpr (!MX) {
      const int rows = few_rows<MX>(P.T);
      if (v < nvec) *reinterpret_cast<uint4*>(P.xb + (v >> 3) * rows * 128 + swz128(c, v & 7)) = load_x(c, v);
    } else {
      const int xchunk = few_xchunk<true>(16);
      if (P.xq) {
        const int ng = D / kMxGroup;
        if (v < (D >> 4))
          *reinterpret_cast<uint4*>(P.xb + (v >> 3) * xchunk + swz128(c, v & 7)) =
              __ldg(reinterpret_cast<const uint4*>(P.xq) + static_cast<size_t>(c) * (D >> 4) + v);
        if (v < ng) P.xb[(v >> 2) * xchunk + 16 * 128 + 16 * c + (v & 3)] = __ldg(P.xs + static_cast<size_t>(c) * ng + v);
      } else {
        const uint4 q = v < nvec ? load_x(c, v) : make_uint4(0, 0, 0, 0);
        const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(&q);
        float f[8];
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[j] = __bfloat162float(b[j]);
          m = max(m, abs_bits(f[j]));
        }
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));  // four lanes hold a group
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const uint32_t sc = mx_scale_code(m);
        const float inv = mx_inv_scale(sc);
        if (v < nvec) {
          uint8_t* at = P.xb + (v >> 4) * xchunk;
          *reinterpret_cast<uint2*>(at + swz128(c, (v >> 1) & 7) + (v & 1) * 8) =
              make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                         e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
          if ((v & 3) == 0) at[16 * 128 + 16 * c + ((v >> 2) & 3)] = static_cast<uint8_t>(sc);
        }
      }
    }
  }
  if (!route) return;
  for (int i = tx; i < P.T * (kFewRouterRows / 8); i += kFewPrepThreads) {
    const int t = i / (kFewRouterRows / 8), v = i % (kFewRouterRows / 8);
    const uint4 q = k0 + v * 8 < D ? load_x(t, (k0 >> 3) + v) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(&s_x[t][v * 8]) = q;
  }
  __syncthreads();
  for (int t0 = 0; t0 < P.T; t0 += kTB) {
    float4 acc[kTB];
#pragma unroll
    for (int j = 0; j < kTB; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kRowsPer; ++i) {
      const float w0 = __uint_as_float(w[i].x << 16), w1 = __uint_as_float(w[i].x & 0xFFFF0000u);
      const float w2 = __uint_as_float(w[i].y << 16), w3 = __uint_as_float(w[i].y & 0xFFFF0000u);
#pragma unroll
      for (int j = 0; j < kTB; ++j) {  // (rows of s_x past T hold anything; their sums are not stored)
        const float x = __bfloat162float(s_x[t0 + j][warp * kRowsPer + i]);
        acc[j].x = fmaf(x, w0, acc[j].x);
        acc[j].y = fmaf(x, w1, acc[j].y);
        acc[j].z = fmaf(x, w2, acc[j].z);
        acc[j].w = fmaf(x, w3, acc[j].w);
      }
    }
#pragma unroll
    for (int j = 0; j < kTB; ++j) s_part[warp][j][lane] = acc[j];
    __syncthreads();
    if (tx < kTB * 32 && t0 + (tx >> 5) < P.T) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int g = 0; g < kWarps; ++g) {
        const float4 b = s_part[g][tx >> 5][lane];
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
      }
      reinterpret_cast<float4*>(P.logit_part)[(c * 16 + t0 + (tx >> 5)) * 32 + lane] = a;
    }
    __syncthreads();
  }
}

template <bool MX>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewParams P) {
  constexpr int kKC = few_kc<MX>();
  constexpr int kHOff = kFewWBytes + (MX ? kFewSfBytes : 0);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int D = P.D;
  const int rows = few_rows<MX>(P.T);
  const int stage_bytes = few_stage_bytes<MX>(rows);
  const int hchunk = few_hchunk<MX>(rows), xchunk = few_xchunk<MX>(rows);
  const int ck = (D + kKC - 1) / kKC;  // chunks of a gate|up reduction
  uint8_t* ring = smem;
  float* sW = reinterpret_cast<float*>(ring + P.stages * stage_bytes);  // [list entry][16]
  uint32_t* sBits = reinterpret_cast<uint32_t*>(sW + 128 * 16);   // [list entry] tokens routed there
  uint8_t* sList = reinterpret_cast<uint8_t*>(sBits + 128);       // [list entry] local expert
  float* sSel = reinterpret_cast<float*>(sList + 128);            // [token][slot] selected logits, then weights
  uint8_t* sCh = reinterpret_cast<uint8_t*>(sSel + kFewMaxTokens * kFewMaxTopK);  // [token][slot] selected experts
  int* sBegS = reinterpret_cast<int*>(sCh + kFewMaxTokens * kFewMaxTopK);  // [CTA] first chunk of each range, S
  int* sBegE = sBegS + kFewMaxCtas + 1;                                    // E
  int* sBegD = sBegE + kFewMaxCtas + 1;                                    // D
  int* sTileA = sBegD + kFewMaxCtas + 1;                                   // [tile] first CTA of an output tile
  int* sTileB = sTileA + 16;                                               // [tile] last CTA
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uintptr_t>(sTileB + 16 + 1) & ~uintptr_t(7));
  uint64_t* hfull = full + kFewMaxStages;
  uint64_t* empty = hfull + kFewMaxStages;
  uint64_t* acc_full = empty + kFewMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* routed = acc_empty + 2;
  uint64_t* weighted = routed + 1;  // the routing's second half: weights and masks
  uint64_t* drain = weighted + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* sTouched = tmem_slot + 1;  // [4] bitmask of experts
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sTouched + 4);
  int* sCount = const_cast<int*>(abort_flag) + 1;  // touched experts
  int* sLast = sCount + 1;

  const int warp = warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int nr = (D + kFewRouterRows - 1) / kFewRouterRows;  // parts of the logits
  const int ks_dn = (P.S + kKC - 1) / kKC, ke_dn = (P.F + kKC - 1) / kKC;
  const int su = (P.S + kFewGuCols - 1) / kFewGuCols, fu = (P.F + kFewGuCols - 1) / kFewGuCols;
  const int nd = (D + kFewDnCols - 1) / kFewDnCols;
  uint32_t* c_hidden = P.counters;
  uint32_t* c_down = P.counters + 1;
  uint32_t* c_shared = P.counters + 2;
  uint32_t* c_rows = P.counters + 3;
  uint32_t* c_eu = P.counters + 8;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&hfull[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kFewConsWarps);
    }
    mbar_init(routed, 1);
    mbar_init(weighted, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *sCount = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 4) sTouched[threadIdx.x] = 0;
  if (warp == kFewMmaWarp) {
    tmem_alloc(tmem_slot, kFewTmemCols);
    tmem_relinquish();
  }
  // The kernel may be set up while few_prep_kernel runs (barriers, TMEM); the __syncthreads() below holds the copying
  // warps too until that one has ended.
  if (warp >= kFewProdWarps) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x <= grid) sBegS[threadIdx.x] = FewSplit(su * ck, grid).begin(threadIdx.x);
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  // The next kernel may be set up from now on (the library's wait for this one's end before they touch memory).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp < kFewProdWarps || warp == kFewProdWarp4) {
    const int role = warp == kFewProdWarp4 ? 4 : warp;
    if (lane != 0 || (!MX && (role == 2 || role == 3))) return;
    // --------------------------------------------------------- producers
    // Thread 0: gate and down weights (it announces a stage's bytes on full[]);
    // 1: up weights; 2, 3 (MXFP8): the scale tiles of gate | up, or of the two
    // 128-column halves of down; 4: the B operand, x or in D the GeGLU rows (on
    // hfull[]). Each walks the whole chunk list and waits for a stage to be free by itself; a
    // copy may land before thread 0's announcement, the stage completes with both.
    int s = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto acquire = [&]() -> bool {
      if (!mbar_wait_cycles(&empty[s], ph ^ 1, abort_flag, P.err)) return ok = false;
      ++issued;
      return true;
    };
    auto advance = [&]() {
      if (++s == P.stages) {
        s = 0;
        ph ^= 1;
      }
    };
    // gate and up of 128 output columns n0 of N, K chunk kc, weight g
    auto issue_gu = [&](const CUtensorMap* mg, const CUtensorMap* mu, const uint8_t* sg, const uint8_t* sup, int N, int g,
                        int n0, int kc) {
      uint8_t* st = ring + s * stage_bytes;
      if (role == 0) mbar_arrive_expect_tx(&full[s], kFewWBytes + (MX ? kFewSfBytes : 0) + xchunk);
      if (role == 4) {
        bulk_load(st + kHOff, P.xb + kc * xchunk, xchunk, &full[s]);
      } else if (role < 2) {
        const CUtensorMap* m = role == 0 ? mg : mu;
        if constexpr (MX) {
          tma_load_3d(st + role * (kFewWBytes / 2), m, &full[s], kc * 128, n0, g);
        } else {
          tma_load_4d(st + role * (kFewWBytes / 2), m, &full[s], 0, kc * 64, n0 >> 6, g);
        }
      } else {
        const size_t tile = (static_cast<size_t>(g) * ((N + 127) / 128) + (n0 >> 7)) * ck + kc;
        bulk_load(st + kFewWBytes + (role - 2) * 512, (role == 2 ? sg : sup) + tile * 512, 512, &full[s]);
      }
    };
    if (role == 0) {
      tma_prefetch_desc(&P.tmSg);
      tma_prefetch_desc(&P.tmG);
      tma_prefetch_desc(&P.tmSd);
      tma_prefetch_desc(&P.tmD);
    } else if (role == 1) {
      tma_prefetch_desc(&P.tmSu);
      tma_prefetch_desc(&P.tmU);
    }
    for (int i = sBegS[cta], e = sBegS[cta + 1]; i < e; ++i) {
      if (!ok || !acquire()) break;
      issue_gu(&P.tmSg, &P.tmSu, P.sfsg, P.sfsu, P.S, 0, (i / ck) * kFewGuCols, i % ck);
      advance();
    }
    if (ok && !mbar_wait_cycles(routed, 0, abort_flag, P.err)) ok = false;
    uint32_t h_par = 0;  // per stage: the parity of its next hfull phase (thread 4)
    int h_issued = 0;
    if (ok) {
      const int nact = *sCount;
      for (int i = sBegE[cta], e = sBegE[cta + 1]; i < e; ++i) {
        if (!acquire()) break;
        const int u = i / ck;
        issue_gu(&P.tmG, &P.tmU, P.sfg, P.sfu, P.F, sList[u / fu], (u % fu) * kFewGuCols, i % ck);
        advance();
      }
      const int len = ks_dn + nact * ke_dn;
      const int i0 = sBegD[cta], i1 = sBegD[cta + 1];
      if (ok && role == 4 && i0 < i1) {
        // The weights of the first stages are on their way; the GeGLU rows have to be complete everywhere.
        if (!counter_wait(c_hidden, grid, abort_flag, P.err)) ok = false;
        fence_proxy_async();  // they were written by ordinary stores of other SMs
      }
      for (int i = i0; ok && i < i1; ++i) {
        if (!acquire()) break;
        const int n0 = (i / len) * kFewDnCols, kc = i % len;
        uint8_t* st = ring + s * stage_bytes;
        const bool sh = kc < ks_dn;
        const int g = sh ? 0 : sList[(kc - ks_dn) / ke_dn];
        const int kl = sh ? kc : (kc - ks_dn) % ke_dn;
        const bool two = n0 + 128 < D;  // the tile has a second 128-column half
        if (role == 0) {
          const CUtensorMap* m = sh ? &P.tmSd : &P.tmD;
          mbar_arrive_expect_tx(&full[s], kFewWBytes + (MX ? (two ? 1024 : 512) : 0));
          if constexpr (MX) {
            tma_load_3d(st, m, &full[s], kl * 128, n0, g);
          } else {
            tma_load_4d(st, m, &full[s], 0, kl * 64, n0 >> 6, g);
          }
        } else if (role == 4) {
          mbar_arrive_expect_tx(&hfull[s], hchunk);
          bulk_load(st + kHOff, P.h + static_cast<size_t>(kc) * hchunk, hchunk, &hfull[s]);
          h_par ^= 1u << s;
          ++h_issued;
        } else if (role == 2 || (role == 3 && two)) {
          const size_t tile =
              (static_cast<size_t>(g) * ((D + 127) / 128) + (n0 >> 7) + (role - 2)) * (sh ? ks_dn : ke_dn) + kl;
          bulk_load(st + kFewWBytes + (role - 2) * 512, (sh ? P.sfsd : P.sfd) + tile * 512, 512, &full[s]);
        }
        advance();
      }
    }
    if (*abort_flag) {
      // gave up: wait (bounded) for the copies in flight before shared memory goes away
      const int pending = issued < P.stages ? issued : P.stages;
      for (int i = 0; i < pending; ++i) {
        if (--s < 0) {
          s = P.stages - 1;
          ph ^= 1;
        }
        uint32_t dummy = 0;
        mbar_wait_cycles(&full[s], ph, reinterpret_cast<volatile int*>(&dummy), P.err, kWaitTimeoutCycles / 20);
        if (i < h_issued) {
          dummy = 0;
          mbar_wait_cycles(&hfull[s], ((h_par >> s) & 1u) ^ 1u, reinterpret_cast<volatile int*>(&dummy), P.err, kWaitTimeoutCycles / 20);
        }
      }
    }
    return;
  }

  const uint32_t tmem = *tmem_slot;

  if (warp == kFewMmaWarp) {
    // ------------------------------------------------------- MMA issuer: the whole warp walks, one lane issues
    int s = 0;
    uint32_t ph = 0, hph = 0, q = 0;  // q: accumulators used so far
    bool ok = true, any = false;
    const uint32_t xhi = desc_hi(rows == 8 ? 0 : 1024);
    auto begin_acc = [&]() -> uint32_t {  // the accumulator's first TMEM column
      ok = ok && __all_sync(0xffffffffu, mbar_wait_cycles(&acc_empty[q & 1], ((q >> 1) & 1) ^ 1, abort_flag, P.err));
      tc_fence_after_sync();
      return tmem + (q & 1) * kFewTmemAcc;
    };
    auto end_acc = [&]() {
      if (ok && elect_one()) umma_commit(&acc_full[q & 1]);
      ++q;
    };
    auto end_chunk = [&]() {
      __syncwarp();
      any = true;
      if (++s == P.stages) {
        s = 0;
        ph ^= 1;
      }
    };
    // MXFP8: both M = 128 tiles of a chunk (accumulators d and d + n) over the K it has left (64: half a chunk)
    auto mma_mx = [&](uint32_t d, int n, uint32_t a, uint32_t b, bool first, int k_left) {
      const uint32_t sf = tmem + kFewTmemSf + s * 16;
      tmem_cp_scales(sf, a + kFewWBytes);
      tmem_cp_scales(sf + 4, a + kFewWBytes + 512);
      tmem_cp_scales(sf + 8, b + 16 * 128);
      const uint32_t al = desc_lo(a, 16), bl = desc_lo(b, 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j == 2 && k_left <= 64) break;
        umma_mxf8(d, al + j * 2, desc_hi(1024), bl + j * 2, desc_hi(1024), idesc_mxf8_m128(16, j), sf, sf + 8,
                  !first || j != 0);
        umma_mxf8(d + n, al + kFewWBytes / 32 + j * 2, desc_hi(1024), bl + j * 2, desc_hi(1024),
                  idesc_mxf8_m128(16, j), sf + 4, sf + 8, !first || j != 0);
      }
    };
    // a phase of gate|up chunks
    auto run_gu = [&](const int* begin) {
      const int i1 = warp_uniform(begin[cta + 1]);
      for (int i = warp_uniform(begin[cta]); ok && i < i1;) {
        const int iend = min(i1, (i / ck + 1) * ck);
        const uint32_t d = begin_acc();
        int kc = i % ck;
        for (bool first = true; ok && i < iend; ++i, ++kc, first = false) {
          if (!__all_sync(0xffffffffu, mbar_wait_cycles(&full[s], ph, abort_flag, P.err))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a = smem_u32(ring + s * stage_bytes), b = a + kHOff;
          if (elect_one()) {
            if constexpr (MX) {
              mma_mx(d, 16, a, b, first, D - kc * 128);
            } else {
              const uint32_t al = desc_lo(a, 8192), bl = desc_lo(b, 16);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                few_umma_bf16(d, al + j * 128, desc_hi(1024), bl + j * 2, xhi, few_idesc_bf16(16), !first || j != 0);
                few_umma_bf16(d + 16, al + kFewWBytes / 32 + j * 128, desc_hi(1024), bl + j * 2, xhi, few_idesc_bf16(16),
                              !first || j != 0);
              }
            }
            umma_commit(&empty[s]);
          }
          end_chunk();
        }
        end_acc();
      }
    };
    run_gu(sBegS);
    ok = ok && __all_sync(0xffffffffu, mbar_wait_cycles(routed, 0, abort_flag, P.err));
    if (ok) {
      const int nact = warp_uniform(*sCount);
      run_gu(sBegE);
      const int len = ks_dn + nact * ke_dn;
      const int i1 = warp_uniform(sBegD[cta + 1]);
      for (int i = warp_uniform(sBegD[cta]); ok && i < i1;) {  // one accumulator per run of chunks of one source
        const int u = i / len;
        int kc = i - u * len;
        const int run_end = kc < ks_dn ? ks_dn : ks_dn + ((kc - ks_dn) / ke_dn + 1) * ke_dn;
        const int iend = min(i1, u * len + run_end);
        const int run0 = kc < ks_dn ? 0 : run_end - ke_dn;
        const int K = kc < ks_dn ? P.S : P.F;
        const uint32_t d = begin_acc();
        for (bool first = true; ok && i < iend; ++i, ++kc, first = false) {
          if (!__all_sync(0xffffffffu, mbar_wait_cycles(&full[s], ph, abort_flag, P.err) &&
                                           mbar_wait_cycles(&hfull[s], (hph >> s) & 1u, abort_flag, P.err))) {
            ok = false;
            break;
          }
          hph ^= 1u << s;
          tc_fence_after_sync();
          const uint32_t a = smem_u32(ring + s * stage_bytes), b = a + kHOff;
          if (elect_one()) {
            if constexpr (MX) {
              mma_mx(d, 16, a, b, first, K - (kc - run0) * 128);
            } else {
              // B: the high, then the low parts of the GeGLU rows, as N = 2 rows
              const uint32_t al = desc_lo(a, 8192), bl = desc_lo(b, 16), id = few_idesc_bf16(2 * rows);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                few_umma_bf16(d, al + j * 128, desc_hi(1024), bl + j * 2, desc_hi(1024), id, !first || j != 0);
                few_umma_bf16(d + 32, al + kFewWBytes / 32 + j * 128, desc_hi(1024), bl + j * 2, desc_hi(1024), id,
                              !first || j != 0);
              }
            }
            umma_commit(&empty[s]);
          }
          end_chunk();
        }
        end_acc();
      }
    }
    if (any && elect_one()) {
      umma_commit(drain);
      uint32_t dummy = 0;
      mbar_wait_cycles(drain, 0, reinterpret_cast<volatile int*>(&dummy), P.err);
    }
    __syncwarp();
    bar_named(4, 32 * (kFewConsWarps + 1));  // the consumers have read their last accumulator
    tc_fence_after_sync();
    tmem_dealloc(tmem, kFewTmemCols);
    return;
  }

  const int wx = warp - kFewProdWarps;  // 0..15
  if (wx >= kFewConsWarps) {
    // ------------------------------------------------------------- routing
    const int wr = wx - kFewConsWarps;  // 0..7: tokens wr, wr + 8
    const int rt = wr * 32 + lane;
    if (wr < P.T) {
      // tokens wr and wr + 8 (if there) side by side; this lane's experts 4 lane .. 4 lane + 3
      const int ntok = wr + 8 < P.T ? 2 : 1;
      const int e4 = lane * 4;
      const bool in = e4 < P.E;
      float l[2][4] = {};
      const float4* parts = reinterpret_cast<const float4*>(P.logit_part) + wr * 32 + lane;
      auto add_part = [&](float (&a)[4], const float4& v) {
        a[0] += v.x;
        a[1] += v.y;
        a[2] += v.z;
        a[3] += v.w;
      };
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ntok == 1) {
        for (int r0 = 0; r0 < nr; r0 += 12) {  // the partial logits in order
          float4 v[12];
#pragma unroll
          for (int r = 0; r < 12; ++r) v[r] = r0 + r < nr ? __ldcg(parts + (r0 + r) * 16 * 32) : zero;
#pragma unroll
          for (int r = 0; r < 12; ++r) add_part(l[0], v[r]);
        }
      } else {
        for (int r0 = 0; r0 < nr; r0 += 6) {
          float4 v[2][6];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 6; ++r) v[h][r] = r0 + r < nr ? __ldcg(parts + ((r0 + r) * 16 + 8 * h) * 32) : zero;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 6; ++r) add_part(l[h], v[h][r]);
        }
      }
      uint32_t key[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (in && P.bias) l[h][i] += __ldg(P.bias + e4 + i);
          // a NaN counts as -infinity, as in the block's own routing; key 0: not to be taken
          key[h][i] = in ? order_key(isnan(l[h][i]) ? -INFINITY : l[h][i]) : 0u;
          if (in && h < ntok && cta == 0 && P.logits_out)
            P.logits_out[static_cast<size_t>(wr + 8 * h) * P.E + e4 + i] = l[h][i];
        }
      // k rounds of: the largest key, the lowest expert among equals; slot j stays in lane j
      uint32_t my_key[2] = {0, 0};
      int my_e[2] = {0, 0};
      for (int j = 0; j < P.k; ++j) {
        uint32_t bk[2], top[2];
        int be[2], e[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bk[h] = key[h][0];
          be[h] = e4;
#pragma unroll
          for (int i = 1; i < 4; ++i)
            if (key[h][i] > bk[h]) {
              bk[h] = key[h][i];
              be[h] = e4 + i;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) top[h] = __reduce_max_sync(0xffffffffu, bk[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          e[h] = static_cast<int>(
              __reduce_min_sync(0xffffffffu, bk[h] == top[h] ? static_cast<uint32_t>(be[h]) : 0xFFFFu));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (e4 + i == e[h]) key[h][i] = 0u;
          if (lane == j) {
            my_key[h] = top[h];
            my_e[h] = e[h];
          }
        }
      }
      for (int h = 0; h < ntok; ++h) {
        const int t = wr + 8 * h;
        // the key's logit; softmax over the kept ones (slot 0 holds the largest)
        const float logit = __uint_as_float((my_key[h] & 0x80000000u) ? my_key[h] ^ 0x80000000u : ~my_key[h]);
        const float mx = __shfl_sync(0xffffffffu, logit, 0);
        const float ex = lane < P.k ? expf(logit - mx) : 0.f;
        float sum = ex;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane < P.k) {
          const int e = my_e[h];
          sSel[t * kFewMaxTopK + lane] = ex / sum;
          sCh[t * kFewMaxTopK + lane] = static_cast<uint8_t>(e);
          if (e >= P.e0 && e < P.e0 + P.el) atomicOr(&sTouched[e >> 5], 1u << (e & 31));
          if (cta == 0 && P.w_out) P.w_out[static_cast<size_t>(t) * P.k + lane] = ex / sum;
          if (cta == 0 && P.idx_out) P.idx_out[static_cast<size_t>(t) * P.k + lane] = e;
        }
      }
    }
    for (int i = rt; i < 128 * 16; i += 256) sW[i] = 0.f;
    if (rt < 128) sBits[rt] = 0;
    bar_named(2, 32 * kFewConsWarps);
    // the list of touched experts, ascending, and the ranges: what the copying threads need
    const uint32_t touched[4] = {sTouched[0], sTouched[1], sTouched[2], sTouched[3]};
    auto position = [&](int e) -> int {
      int pos = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pos += i < (e >> 5) ? __popc(touched[i]) : i == (e >> 5) ? __popc(touched[i] & ((1u << (e & 31)) - 1u)) : 0;
      return pos;
    };
    const int n = __popc(touched[0]) + __popc(touched[1]) + __popc(touched[2]) + __popc(touched[3]);
    if (rt < 128 && ((sTouched[rt >> 5] >> (rt & 31)) & 1u)) sList[position(rt)] = static_cast<uint8_t>(rt - P.e0);
    if (rt == 0) *sCount = n;
    const int len = ks_dn + n * ke_dn;
    const FewSplit sd(nd * len, grid);
    if (rt <= grid) {
      sBegE[rt] = FewSplit(n * fu * ck, grid).begin(rt);
      sBegD[rt] = sd.begin(rt);
    }
    bar_named(2, 32 * kFewConsWarps);
    if (rt == 0) mbar_arrive(routed);
    // what the consumers need: weights, masks, the CTAs of each output tile
    if (rt < nd) {
      sTileA[rt] = sd.cta_of(rt * len);
      sTileB[rt] = sd.cta_of((rt + 1) * len - 1);
    }
    for (int a = rt; a < kFewMaxTokens * kFewMaxTopK; a += 256) {
      const int t = a / kFewMaxTopK, j = a % kFewMaxTopK;
      if (t >= P.T || j >= P.k) continue;
      const int e = sCh[a];
      if (e < P.e0 || e >= P.e0 + P.el) continue;
      const int pos = position(e);
      sW[pos * 16 + t] = sSel[a];
      atomicOr(&sBits[pos], 1u << t);
    }
    bar_named(2, 32 * kFewConsWarps);
    if (rt == 0) mbar_arrive(weighted);
    if (cta == 0 && P.cnt_out && rt < P.E)
      P.cnt_out[rt] = ((sTouched[rt >> 5] >> (rt & 31)) & 1u) ? __popc(sBits[position(rt)]) : 0;
    return;
  }

  // ------------------------------------------------------------- consumers
  // The eight warps read finished accumulators: warp quarter wc % 4 the TMEM
  // lanes (output columns) 32 (wc % 4) .., half wc / 4 a half of the tokens (R, S, E)
  // or of the 256 columns (D). After a wait gave up (ok = false) a warp does no more
  // work but keeps to the loops: their counts, and so the named barriers in
  // them, are the same for all eight warps.
  const int wc = wx;              // 0..7
  const int ct = wc * 32 + lane;  // 0..255
  const int half = wc >> 2, col = (wc & 3) * 32 + lane;
  const uint32_t tlane = tmem + (static_cast<uint32_t>((wc & 3) * 32) << 16);
  uint32_t q = 0;
  bool ok = true;
  auto wait_acc = [&]() {  // the next accumulator is complete
    int got = 0;
    if (ok && lane == 0) got = mbar_wait_cycles(&acc_full[q & 1], (q >> 1) & 1, abort_flag, P.err);
    ok = __shfl_sync(0xffffffffu, got, 0) != 0;
    tc_fence_after_sync();
  };
  auto free_acc = [&]() {
    tmem_ld_wait();
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0 && ok) mbar_arrive(&acc_empty[q & 1]);
    ++q;
  };
  // All the warps' writes so far, seen by whoever sees the count: a barrier, then one thread's fence and atomic.
  auto publish = [&](uint32_t* counter) -> uint32_t {
    bar_named(1, 32 * kFewConsWarps);
    uint32_t before = 0;
    if (ct == 0 && ok) {
      __threadfence();
      before = atomicAdd(counter, 1u);
      __threadfence();
    }
    return before;
  };
  // ---- S, E: a unit's sums (this thread: column `col`, tokens 8 half ..) come from one CTA, or as parts from several,
  // each part in its CTA's slot of part_gu. The shared MLP's GeGLU rows are made by all CTAs while the first experts'
  // weights arrive; an expert unit's by the last of its CTAs.
  constexpr size_t kUnit = 2 * 16 * kFewGuCols;  // floats of a unit's partial sums
  auto load_acc = [&](float (&g)[8], float (&v)[8]) {
    wait_acc();
    uint32_t a[8], b[8];
    tmem_ld_32x32b_x8(tlane + (q & 1) * kFewTmemAcc + half * 8, a);
    tmem_ld_32x32b_x8(tlane + (q & 1) * kFewTmemAcc + 16 + half * 8, b);
    free_acc();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = __uint_as_float(a[j]);
      v[j] = __uint_as_float(b[j]);
    }
  };
  auto part_of = [&](int c, int phase, int seg) -> float* {  // gate sums [16][128], then up
    return P.part_gu + ((static_cast<size_t>(c) * 2 + phase) * 2 + seg) * kUnit;
  };
  auto store_partial = [&](int phase, int seg, uint32_t tokens, const float (&g)[8], const float (&v)[8]) {
    float* part = part_of(cta, phase, seg);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = half * 8 + j;
      if ((tokens >> t) & 1u) {
        part[t * kFewGuCols + col] = g[j];
        part[(16 + t) * kFewGuCols + col] = v[j];
      }
    }
  };
  // One GeGLU value (token t, hidden unit f of N) into the down chunks from chunk0 on. A warp's lanes hold 32
  // consecutive f, an MXFP8 group.
  auto emit_hidden = [&](int t, int f, int N, int chunk0, float gate, float up) {
    const float h = gelu_tanh_exact(gate) * up;
    if constexpr (MX) {
      const uint32_t sc = mx_scale_code(__reduce_max_sync(0xffffffffu, abs_bits(h)));
      if (f < N) {
        uint8_t* hc = P.h + static_cast<size_t>(chunk0 + (f >> 7)) * hchunk;
        const float x = h * mx_inv_scale(sc);
        hc[swz128(t, (f & 127) >> 4) + (f & 15)] = static_cast<uint8_t>(e4m3x4(x, x, x, x) & 0xFFu);
        if (lane == 0) hc[16 * 128 + 16 * t + ((f & 127) >> 5)] = static_cast<uint8_t>(sc);
      }
    } else if (f < N) {
      const __nv_bfloat16 hi = __float2bfloat16_rn(h);
      // an infinity or NaN stays in the high part
      const float lo = abs_bits(__bfloat162float(hi)) >= 0x7F800000u ? 0.f : h - __bfloat162float(hi);
      uint8_t* at = P.h + static_cast<size_t>(chunk0 + (f >> 6)) * hchunk + swz128(t, (f & 63) >> 3) + (f & 7) * 2;
      *reinterpret_cast<__nv_bfloat16*>(at) = hi;
      *reinterpret_cast<__nv_bfloat16*>(at + rows * 128) = __float2bfloat16_rn(lo);
    }
  };
  for (int i = sBegS[cta]; i < sBegS[cta + 1];) {  // at most two units: there are no more units than CTAs
    const int u = i / ck;
    i = min(sBegS[cta + 1], (u + 1) * ck);
    float g[8], v[8];
    load_acc(g, v);
    store_partial(0, u == sBegS[cta] / ck ? 0 : 1, (1u << P.T) - 1u, g, v);
  }
  publish(c_shared);
  if (ct == 0)
    *sLast = mbar_wait_cycles(weighted, 0, abort_flag, P.err) && counter_wait(c_shared, grid, abort_flag, P.err) ? 1 : 0;
  bar_named(1, 32 * kFewConsWarps);
  const bool go = *sLast != 0;  // without a routing all eight warps stop here (the wait has raised abort)
  bar_named(1, 32 * kFewConsWarps);
  if (go) {
    const int nact = *sCount;
    const FewSplit split_s(su * ck, grid);
    for (int it = cta * 256 + ct; it < P.T * P.S; it += grid * 256) {
      const int t = it / P.S, f = it - t * P.S, u = f / kFewGuCols;
      const int ca = split_s.cta_of(u * ck), cb = split_s.cta_of((u + 1) * ck - 1);
      float gs = 0.f, us = 0.f;
      for (int c0 = ca; c0 <= cb; c0 += 8) {
        float a[8], b[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          a[c] = b[c] = 0.f;
          if (c0 + c <= cb) {  // slot 0: the unit is the first of the CTA's range
            const float* at = part_of(c0 + c, 0, sBegS[c0 + c] >= u * ck ? 0 : 1) + t * kFewGuCols + f % kFewGuCols;
            a[c] = __ldcg(at);
            b[c] = __ldcg(at + 16 * kFewGuCols);
          }
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          gs += a[c];
          us += b[c];
        }
      }
      emit_hidden(t, f, P.S, 0, gs, us);
    }
    fence_proxy_async();
    const int e0 = sBegE[cta], e1 = sBegE[cta + 1];
    for (int i = e0; i < e1;) {
      const int u = i / ck;
      const int seg = u == e0 / ck ? 0 : 1;  // (middle units of a range are whole and leave no part)
      i = min(e1, (u + 1) * ck);
      float g[8], v[8];
      load_acc(g, v);
      // the CTAs that share the unit: this one's neighbours
      int ca = cta, cb = cta;
      while (sBegE[ca] > u * ck) --ca;
      while (sBegE[cb + 1] < (u + 1) * ck) ++cb;
      const uint32_t tokens = sBits[u / fu];  // only the tokens routed to the expert are kept
      bool own = true;                        // this CTA's part is still in registers
      if (ca != cb) {
        // When all others have left their parts, this one's need not go through memory.
        const uint32_t others = static_cast<uint32_t>(cb - ca);
        if (ct == 0) *sLast = ok && ld_acquire(c_eu + u) == others ? 1 : 0;
        bar_named(1, 32 * kFewConsWarps);
        if (*sLast == 0) {
          bar_named(1, 32 * kFewConsWarps);
          own = false;
          store_partial(1, seg, tokens, g, v);
          const uint32_t before = publish(c_eu + u);
          if (ct == 0) *sLast = ok && before == others ? 1 : 0;
          bar_named(1, 32 * kFewConsWarps);
        }
      } else {
        if (ct == 0) *sLast = ok ? 1 : 0;
        bar_named(1, 32 * kFewConsWarps);
      }
      if (*sLast) {
        const int e = u / fu, f = (u - e * fu) * kFewGuCols + col;
#pragma unroll
        for (int j0 = 0; j0 < 8; j0 += 4) {
          if (((tokens >> (half * 8 + j0)) & 15u) == 0) continue;
          float gs[4] = {}, us[4] = {};
          for (int c0 = ca; c0 <= cb; c0 += 2) {
            float a[2][4], b[2][4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const bool mine = own && c0 + c == cta, in = c0 + c <= cb && !mine;
              const float* at = part_of(c0 + c, 1, in && sBegE[c0 + c] < u * ck ? 1 : 0) + (half * 8 + j0) * kFewGuCols + col;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const bool get = in && ((tokens >> (half * 8 + j0 + j)) & 1u);
                a[c][j] = get ? __ldcg(at + j * kFewGuCols) : mine ? g[j0 + j] : 0.f;
                b[c][j] = get ? __ldcg(at + (16 + j) * kFewGuCols) : mine ? v[j0 + j] : 0.f;
              }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                gs[j] += a[c][j];
                us[j] += b[c][j];
              }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((tokens >> (half * 8 + j0 + j)) & 1u) emit_hidden(half * 8 + j0 + j, f, P.F, ks_dn + e * ke_dn, gs[j], us[j]);
        }
        fence_proxy_async();
      }
      bar_named(1, 32 * kFewConsWarps);  // sLast is free again
    }
    publish(c_hidden);

    // ---- D: this thread's output column of the tile, all 16 tokens
    const int len = ks_dn + nact * ke_dn;
    const int i0 = sBegD[cta], i1 = sBegD[cta + 1];
    for (int i = i0; i < i1;) {
      const int u = i / len;
      const int uend = min(i1, (u + 1) * len);
      const int seg = u == i0 / len ? 0 : 1;
      float tot[16] = {};
      while (i < uend) {  // runs of one source: -1 the shared MLP, else a touched expert
        const int kc = i - u * len;
        const int src = kc < ks_dn ? -1 : (kc - ks_dn) / ke_dn;
        i = min(uend, u * len + ks_dn + (src + 1) * ke_dn);
        wait_acc();
        float a[16];
        {
          const uint32_t at = tlane + (q & 1) * kFewTmemAcc + half * (MX ? 16 : 32);
          uint32_t hi[16];
          tmem_ld_32x32b_x16(at, hi);
          if constexpr (MX) {
            free_acc();
#pragma unroll
            for (int t = 0; t < 16; ++t) a[t] = __uint_as_float(hi[t]);
          } else {  // the high and the low parts' sums: columns t and rows + t
            uint32_t lo[16];
            if (rows == 16) tmem_ld_32x32b_x16(at + 16, lo);
            free_acc();
#pragma unroll
            for (int t = 0; t < 16; ++t)
              a[t] = rows == 16 ? __uint_as_float(hi[t]) + __uint_as_float(lo[t])
                                : __uint_as_float(hi[t & 7]) + __uint_as_float(hi[8 + (t & 7)]);
          }
        }
        if (!ok) continue;
        const uint32_t bits = src < 0 ? 0xFFFFu : sBits[src];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const float w = src < 0 ? 1.f : sW[src * 16 + t];
          if ((bits >> t) & 1u) tot[t] = fmaf(w, a[t], tot[t]);
        }
      }
      float* mine = P.part_dn + (static_cast<size_t>(cta) * 2 + seg) * 16 * kFewDnCols;
#pragma unroll
      for (int t = 0; t < 16; ++t)
        if (t < P.T) mine[t * kFewDnCols + half * 128 + col] = tot[t];
    }
    publish(c_down);

    // ---- the output: every CTA adds up a share of the columns, the parts in CTA order
    if (ct == 0) *sLast = counter_wait(c_down, grid, abort_flag, P.err) ? 1 : 0;
    bar_named(1, 32 * kFewConsWarps);
    auto column_sum = [&](int t, int c) -> float {
      const int u = c / kFewDnCols;
      const int ca = sTileA[u], cb = sTileB[u];
      const float* src = P.part_dn + t * kFewDnCols + (c - u * kFewDnCols);
      float a = 0.f;
      for (int c0 = ca; c0 <= cb; c0 += 8) {
        float b[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          b[j] = 0.f;
          if (c0 + j <= cb)
            b[j] = __ldcg(src + (static_cast<size_t>(c0 + j) * 2 + (sBegD[c0 + j] >= u * len ? 0 : 1)) * 16 * kFewDnCols);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) a += b[j];
      }
      return a;
    };
    if (*sLast == 0) {
      // (gave up)
    } else {
      const bool post = P.norm_post || P.residual;
      const int n = P.T * D;
      for (int it = cta * 256 + ct; it < n; it += grid * 256) {
        const int t = it / D;
        const float a = column_sum(t, it - t * D);
        if (post) {
          P.f[it] = a;
        } else {
          if (P.out) P.out[it] = __float2bfloat16_rn(a);
          if (P.out_f32) P.out_f32[it] = a;
        }
      }
      if (post) publish(c_rows);
    }
    if (*sLast != 0 && (P.norm_post || P.residual) && cta < P.T) {  // (*sLast and cta: the same for all eight warps)
      const bool rows_ok = ct != 0 || counter_wait(c_rows, grid, abort_flag, P.err);
      bar_named(1, 32 * kFewConsWarps);
      if (ct == 0 && !rows_ok) *sLast = 0;
      bar_named(1, 32 * kFewConsWarps);
    }
    if (*sLast != 0 && (P.norm_post || P.residual) && cta < P.T) {  // norm_post needs whole rows: a CTA each
      constexpr int kV = kFewMaxDim / 256;
      __shared__ float s_red[kFewConsWarps];
      float v[kV];
      float ss = 0.f;
#pragma unroll
      for (int u = 0; u < kV; ++u) {
        const int c = ct + u * 256;
        v[u] = c < D ? __ldcg(P.f + static_cast<size_t>(cta) * D + c) : 0.f;
        ss = fmaf(v[u], v[u], ss);
      }
      float r = 1.f;
      if (P.norm_post) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) s_red[wc] = ss;
        bar_named(1, 32 * kFewConsWarps);
        float tot = 0.f;
#pragma unroll
        for (int i = 0; i < kFewConsWarps; ++i) tot += s_red[i];
        r = 1.0f / sqrtf(tot / static_cast<float>(D) + 1e-6f);
      }
#pragma unroll
      for (int u = 0; u < kV; ++u) {
        const int c = ct + u * 256;
        if (c >= D) continue;
        const size_t at = static_cast<size_t>(cta) * D + c;
        float o = v[u] * r;
        if (P.norm_post) o *= __bfloat162float(P.norm_post[c]);
        if (P.residual) o += __bfloat162float(P.x[at]);
        if (P.out) P.out[at] = __float2bfloat16_rn(o);
        if (P.out_f32) P.out_f32[at] = o;
      }
    }
  }
  tc_fence_before_sync();
  bar_named(4, 32 * (kFewConsWarps + 1));
}

}  // namespace moe
