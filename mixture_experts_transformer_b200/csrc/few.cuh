// The whole MoE layer for a few tokens (T <= 16) in one cooperative kernel:
// router, top-k, experts, shared MLP, combine and (bf16 form) the norms and
// residual around them.
//
// A few tokens read every touched expert's weights once and compute almost
// nothing per byte, so the layer is bound by HBM: the kernel is built as one
// uninterrupted stream of weight chunks per SM. Split over several kernels,
// that stream stops at every kernel boundary and at every wave's ragged end;
// here
//   * the work of each phase is one list of 16 KB weight chunks (64 output
//     columns of gate and up, or 128 of down, times 64 K in bf16 / 128 K in
//     8 bits), cut into equal contiguous ranges, one per CTA, wherever that
//     falls inside an output column's reduction; CTAs that share a column
//     leave fp32 partial sums, and the last of them adds them up in CTA order;
//   * a producer thread keeps a ring of TMA copies full across the phases: the
//     shared MLP's chunks need no routing, so they stream while the router's
//     result is reduced, and the first down chunks are already in flight while
//     the last GeGLU rows are being finished elsewhere.
//
// Phases (chunk lists): R the router (the first CTAs, 256 K rows each),
// S the shared MLP's gate|up, E the touched experts' gate|up, D all down
// projections: for each 128 output columns the shared MLP's reduction, then each touched
// expert's. Two grid-wide waits: the top-k needs all partial logits, D needs
// all GeGLU rows. The grid is launched cooperatively (all CTAs resident), and
// every wait is bounded.
//
// Products: tensor cores (mma.sync m16n8k16 bf16, or m16n8k32 e4m3), the weight
// columns as M and the tokens as N = 8 or 16, so that a chunk costs each of the eight
// consumer warps a few instructions whatever T is. tcgen05's M = 128 tile
// would need the whole 128 columns in TMEM per expert switch and reads back
// through the epilogue path; at N <= 16 the tensor rate is irrelevant. Every token's
// column is computed for every touched expert; a token takes an expert's result
// only if it is routed there (a select, so that nothing of an expert reaches
// other tokens).
//
// Numerics: fp32 accumulation. bf16 form: the GeGLU rows enter the down product as
// the sum of two bf16 values (hi + lo, 16 bits of mantissa), the routed sums are
// weighted and added in fp32: nothing is rounded to bf16 before the output
// (and after norm_pre). MXFP8 form: GeGLU rows in MXFP8, as the large-batch path.
#pragma once

#include "mxformat.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kFewMaxTokens = 16;
constexpr int kFewMaxDim = 4096;      // x rows stay in shared memory
constexpr int kFewConsWarps = 8;
constexpr int kFewThreads = 32 * (1 + 2 * kFewConsWarps);  // producer, 8 consumer and 8 routing warps
constexpr int kFewWBytes = 16384;     // weights of a chunk
constexpr int kFewSfBytes = 1024;     // MXFP8: two scale tiles of a chunk
constexpr int kFewRouterRows = 256;   // K rows of the router per CTA (4 chunks)
constexpr int kFewMaxStages = 12;
constexpr int kFewGPitch = 68;        // floats per token row of the gate / up exchange buffer

// ------------------------------------------------------ shared host / device sizes

template <bool MX>
__host__ __device__ constexpr int few_kc() {  // K elements of a chunk
  return MX ? 128 : 64;
}
// GeGLU rows of one K chunk of down, in the order the MMA's B fragments take them
template <bool MX, int NT>
__host__ __device__ constexpr int few_hchunk() {
  return MX ? NT * (1024 + 32) : NT * 2048;
}
template <bool MX, int NT>
__host__ __device__ constexpr int few_stage_bytes() {
  return kFewWBytes + (MX ? kFewSfBytes : 0) + ((few_hchunk<MX, NT>() + 1023) & ~1023);
}
template <bool MX, int NT>
__host__ __device__ constexpr int few_xpitch(int D) {  // bytes; rows land 16 B apart modulo the banks
  return (MX ? D : 2 * D) + 16;
}
template <bool MX, int NT>
__host__ __device__ constexpr int few_fixed_bytes(int D) {
  return 8 * NT * few_xpitch<MX, NT>(D)                 // x
         + (MX ? 8 * NT * (D / kMxGroup) * 4 : 0)       // its scales as floats
         + (MX ? 8 * NT * (2 * kFewRouterRows + 16) : 0)  // the router's bf16 slice of x
         + 2 * 8 * NT * kFewGPitch * 4                  // gate / up exchange
         + 128 * 16 * 4 + 128 * 4 + 128 * 4             // weights, token masks, list of the touched experts
         + kFewMaxTokens * 128 * 4                      // selected logits
         + 1024 /* barriers, flags */ + 1024 /* alignment */;
}

struct FewParams {
  CUtensorMap tmR;            // w_router [D][E] bf16, box 64 x 64
  CUtensorMap tmG, tmU, tmD;  // experts: bf16 [el][K][N], boxes 64 x 64 (D: two adjacent chunks); MXFP8 [el][N][K], 128 B x 64 (D: 128) rows
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
  const __nv_bfloat16* norm_post;
  int residual;
  const float* bias;
  uint32_t* counters;  // zero at launch: router, hidden, tiles done, -, then one per S unit, E unit, D tile
  float* logit_part;   // [ceil(D / 256)][16][128]
  uint8_t* h;          // GeGLU rows, one few_hchunk per K chunk of down
  float* part_gu;      // [CTA][2 phases][2][2 projections][8 NT][64]
  float* part_dn;      // [CTA][2][8 NT][128]
  float* f;            // [T][D] the sums before norm_post / residual
  __nv_bfloat16* out;
  float* out_f32;
  int32_t* idx_out;
  float* w_out;
  int32_t* cnt_out;
  float* logits_out;
  uint32_t* err;
};

// A phase's chunk list: `units` output column blocks of `len` chunks each, cut into
// `ctas` equal ranges (at most one CTA per chunk, so no range is empty).
struct FewSplit {
  long long total;
  int len, ctas;
  __device__ FewSplit(int units, int len_, int grid) : total(static_cast<long long>(units) * len_), len(len_) {
    ctas = total < grid ? static_cast<int>(total) : grid;
  }
  __device__ int begin(int c) const {
    return c >= ctas ? static_cast<int>(total) : static_cast<int>(total * c / ctas);
  }
  // the CTA whose range holds chunk i
  __device__ int cta_of(int i) const { return static_cast<int>((static_cast<long long>(i + 1) * ctas - 1) / total); }
};

// ------------------------------------------------------------ small PTX pieces

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x2(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// generic-proxy accesses of this thread <-> async-proxy (bulk copy) accesses
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Wait until *p >= want; bounded as mbar_wait.
__device__ __forceinline__ bool counter_wait(const uint32_t* p, uint32_t want, volatile int* abort, uint32_t* err) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (ld_acquire(p) >= want) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      *abort = 1;
      atomicOr(err, kErrWaitTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ void bulk_load_g2s(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// fp32 as an unsigned integer of the same order (a positive NaN above infinity)
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

template <bool MX, int NT>
__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewParams P) {
  constexpr int kTok = 8 * NT;
  constexpr int kKC = few_kc<MX>();
  constexpr int kStage = few_stage_bytes<MX, NT>();
  constexpr int kHChunk = few_hchunk<MX, NT>();
  constexpr int kHOff = kFewWBytes + (MX ? kFewSfBytes : 0);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int D = P.D;
  const int xpitch = few_xpitch<MX, NT>(D);
  constexpr int kRPitch = 2 * kFewRouterRows + 16;
  uint8_t* ring = smem;
  uint8_t* sX = ring + P.stages * kStage;
  float* sXs = reinterpret_cast<float*>(sX + kTok * xpitch);  // MXFP8: [D / 32][kTok]
  uint8_t* sXr = reinterpret_cast<uint8_t*>(sXs) + (MX ? kTok * (D / kMxGroup) * 4 : 0);
  float* sG = reinterpret_cast<float*>(sXr + (MX ? kTok * kRPitch : 0));  // [2][kTok][kFewGPitch]
  float* sW = sG + 2 * kTok * kFewGPitch;                                 // [list entry][16]
  uint32_t* sBits = reinterpret_cast<uint32_t*>(sW + 128 * 16);           // [list entry] tokens routed there
  int* sList = reinterpret_cast<int*>(sBits + 128);                       // [list entry] local expert
  float* sSel = reinterpret_cast<float*>(sList + 128);                    // [token][slot] selected logits, then weights
  uint64_t* full = reinterpret_cast<uint64_t*>(sSel + kFewMaxTokens * 128);
  uint64_t* hfull = full + kFewMaxStages;
  uint64_t* empty = hfull + kFewMaxStages;
  uint64_t* routed = empty + kFewMaxStages;
  uint32_t* sTouched = reinterpret_cast<uint32_t*>(routed + 1);  // [4] bitmask of experts
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sTouched + 4);
  int* sCount = const_cast<int*>(abort_flag) + 1;  // touched experts
  int* sLast = sCount + 1;
  int* sRouteOk = sCount + 2;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, grid = gridDim.x;
  const int nr = (D + kFewRouterRows - 1) / kFewRouterRows;  // router CTAs (at most 16: the grid is larger)
  const int ck = (D + kKC - 1) / kKC;                        // chunks of a gate|up reduction
  const int ks_dn = (P.S + kKC - 1) / kKC, ke_dn = (P.F + kKC - 1) / kKC;
  const int su = P.S / 64, fu = P.F / 64;
  const int nd = (D + 127) / 128;
  uint32_t* c_router = P.counters;
  uint32_t* c_hidden = P.counters + 1;
  uint32_t* c_tiles = P.counters + 2;
  uint32_t* c_su = P.counters + 4;
  uint32_t* c_eu = c_su + su;
  uint32_t* c_dn = c_eu + static_cast<size_t>(P.el) * fu;

  if (threadIdx.x == 0) {
    for (int s = 0; s < P.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&hfull[s], 1);
      mbar_init(&empty[s], kFewConsWarps);
    }
    mbar_init(routed, 1);
    *abort_flag = 0;
    *sCount = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 4) sTouched[threadIdx.x] = 0;
  __syncthreads();

  const FewSplit split_s(su, ck, grid);

  if (warp == 0) {
    if (lane != 0) return;
    // ---------------------------------------------------------- producer
    tma_prefetch_desc(&P.tmSg);
    tma_prefetch_desc(&P.tmSu);
    int s = 0, issued = 0;
    uint32_t ph = 0, h_asked = 0, h_par = 0;  // per stage: GeGLU rows asked for in its latest use; parity of the next hfull phase
    bool ok = true;
    auto acquire = [&]() -> bool {
      if (!mbar_wait(&empty[s], ph ^ 1, abort_flag, P.err)) return ok = false;
      ++issued;
      h_asked &= ~(1u << s);
      return true;
    };
    auto advance = [&]() {
      if (++s == P.stages) {
        s = 0;
        ph ^= 1;
      }
    };
    // gate and up of 64 output columns n0, K chunk kc
    auto issue_gu = [&](const CUtensorMap* mg, const CUtensorMap* mu, const uint8_t* sg, const uint8_t* sup, int N, int g,
                        int n0, int kc) {
      uint8_t* st = ring + s * kStage;
      mbar_arrive_expect_tx(&full[s], kFewWBytes + (MX ? kFewSfBytes : 0));
      if (MX) {
        tma_load_3d(st, mg, &full[s], kc * 128, n0, g);
        tma_load_3d(st + 8192, mu, &full[s], kc * 128, n0, g);
        const size_t tile = (static_cast<size_t>(g) * ((N + 127) / 128) + (n0 >> 7)) * ck + kc;
        bulk_load_g2s(st + kFewWBytes, sg + tile * 512, 512, &full[s]);
        bulk_load_g2s(st + kFewWBytes + 512, sup + tile * 512, 512, &full[s]);
      } else {
        tma_load_3d(st, mg, &full[s], n0, kc * 64, g);
        tma_load_3d(st + 8192, mu, &full[s], n0, kc * 64, g);
      }
    };
    if (cta < nr) {  // the router's rows: 128 experts x 64 K per chunk
      for (int k0 = cta * kFewRouterRows; k0 < min(D, (cta + 1) * kFewRouterRows) && ok; k0 += 64) {
        if (!acquire()) break;
        mbar_arrive_expect_tx(&full[s], kFewWBytes);
        tma_load_3d(ring + s * kStage, &P.tmR, &full[s], 0, k0, 0);
        tma_load_3d(ring + s * kStage + 8192, &P.tmR, &full[s], 64, k0, 0);
        advance();
      }
    }
    for (int i = split_s.begin(cta); ok && i < split_s.begin(cta + 1); ++i) {
      if (!acquire()) break;
      issue_gu(&P.tmSg, &P.tmSu, P.sfsg, P.sfsu, P.S, 0, (i / ck) * 64, i % ck);
      advance();
    }
    tma_prefetch_desc(&P.tmG);
    tma_prefetch_desc(&P.tmU);
    tma_prefetch_desc(&P.tmD);
    tma_prefetch_desc(&P.tmSd);
    if (ok && !mbar_wait(routed, 0, abort_flag, P.err)) ok = false;
    int h_pending = 0;  // chunks of D whose weights, but not yet whose GeGLU rows, were asked for
    if (ok) {
      const int nact = *sCount;
      const FewSplit split_e(nact * fu, ck, grid);
      if (nact > 0) {
        for (int i = split_e.begin(cta); ok && i < split_e.begin(cta + 1); ++i) {
          if (!acquire()) break;
          const int u = i / ck;
          issue_gu(&P.tmG, &P.tmU, P.sfg, P.sfu, P.F, sList[u / fu], (u % fu) * 64, i % ck);
          advance();
        }
      }
      const int len = ks_dn + nact * ke_dn;
      const FewSplit split_d(nd, len, grid);
      const int i0 = split_d.begin(cta), i1 = split_d.begin(cta + 1);
      auto issue_h = [&](int stage, int kc) {
        mbar_arrive_expect_tx(&hfull[stage], kHChunk);
        bulk_load_g2s(ring + stage * kStage + kHOff, P.h + static_cast<size_t>(kc) * kHChunk, kHChunk, &hfull[stage]);
        h_asked |= 1u << stage;
        h_par ^= 1u << stage;
      };
      bool ready = false;
      const int first_stage = s;
      for (int i = i0; ok && i < i1; ++i) {
        if (!acquire()) break;
        const int n0 = (i / len) * 128, kc = i % len;
        uint8_t* st = ring + s * kStage;
        const bool sh = kc < ks_dn;
        const int g = sh ? 0 : sList[(kc - ks_dn) / ke_dn];
        const int kl = sh ? kc : (kc - ks_dn) % ke_dn;
        const CUtensorMap* m = sh ? &P.tmSd : &P.tmD;
        mbar_arrive_expect_tx(&full[s], kFewWBytes + (MX ? 512 : 0));
        if (MX) {
          tma_load_3d(st, m, &full[s], kl * 128, n0, g);
          const size_t tile = (static_cast<size_t>(g) * nd + (n0 >> 7)) * (sh ? ks_dn : ke_dn) + kl;
          bulk_load_g2s(st + kFewWBytes, (sh ? P.sfsd : P.sfd) + tile * 512, 512, &full[s]);
        } else {
          tma_load_4d(st, m, &full[s], 0, kl * 64, n0 >> 6, g);
        }
        if (ready) {
          issue_h(s, kc);
        } else {
          ++h_pending;
        }
        advance();
        // The first ring of weights is asked for before the GeGLU rows are complete everywhere.
        if (!ready && (h_pending == P.stages || i + 1 == i1)) {
          if (!counter_wait(c_hidden, grid, abort_flag, P.err)) {
            ok = false;
            break;
          }
          fence_proxy_async();  // the rows were written by ordinary stores of other SMs
          int hs = first_stage;
          for (int j = 0; j < h_pending; ++j) {
            issue_h(hs, (i0 + j) % len);
            if (++hs == P.stages) hs = 0;
          }
          h_pending = 0;
          ready = true;
        }
      }
    }
    if (!ok || *abort_flag) {
      // gave up: wait for the copies in flight before shared memory goes away
      const int pending = issued < P.stages ? issued : P.stages;
      for (int i = 0; i < pending; ++i) {
        if (--s < 0) {
          s = P.stages - 1;
          ph ^= 1;
        }
        uint32_t dummy = 0;
        mbar_wait(&full[s], ph, reinterpret_cast<volatile int*>(&dummy), P.err, 100000000ull);
        if ((h_asked >> s) & 1u) {
          dummy = 0;
          mbar_wait(&hfull[s], ((h_par >> s) & 1u) ^ 1u, reinterpret_cast<volatile int*>(&dummy), P.err, 100000000ull);
        }
      }
    }
    return;
  }

  // ------------------------------------------- x into shared memory (16 warps)
  const int wx = warp - 1;  // 0..15: a token row each
  if (wx < kTok) {
    uint8_t* row = sX + wx * xpitch;
    const bool live = wx < P.T;
    const uint4* src = reinterpret_cast<const uint4*>(P.x + static_cast<size_t>(wx) * D);
    const int nvec = D >> 3;
    if constexpr (!MX) {
      float r = 1.f;
      if (P.norm_pre && live) {
        float ss = 0.f;
        for (int v = lane; v < nvec; v += 32) {
          const uint4 xv = __ldg(src + v);
          const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(&xv);
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(__bfloat162float(xb[i]), __bfloat162float(xb[i]), ss);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = 1.0f / sqrtf(ss / static_cast<float>(D) + 1e-6f);
      }
      for (int v = lane; v < nvec; v += 32) {
        uint4 xv = live ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
        if (P.norm_pre && live) {
          const uint4 gv = __ldg(reinterpret_cast<const uint4*>(P.norm_pre) + v);
          const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(&xv);
          const __nv_bfloat16* gb = reinterpret_cast<const __nv_bfloat16*>(&gv);
          float o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __bfloat162float(xb[i]) * r * __bfloat162float(gb[i]);
          xv = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                          pack_bf16x2(o[6], o[7]));
        }
        reinterpret_cast<uint4*>(row)[v] = xv;
      }
    } else {
      const int ng = D / kMxGroup;
      if (P.xq) {
        const uint4* q = reinterpret_cast<const uint4*>(P.xq + static_cast<size_t>(wx) * D);
        for (int v = lane; v < (D >> 4); v += 32)
          reinterpret_cast<uint4*>(row)[v] = live ? __ldg(q + v) : make_uint4(0, 0, 0, 0);
        for (int g = lane; g < ng; g += 32)
          sXs[g * kTok + wx] = live ? mx_scale_value(__ldg(P.xs + static_cast<size_t>(wx) * ng + g)) : 0.f;
      } else {
        for (int v0 = 0; v0 < nvec; v0 += 32) {  // four lanes hold a group
          const int v = v0 + lane;
          const bool in = v < nvec;
          const uint4 xv = in && live ? __ldg(src + v) : make_uint4(0, 0, 0, 0);
          const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(&xv);
          float f[8];
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[i] = __bfloat162float(xb[i]);
            m = max(m, abs_bits(f[i]));
          }
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
          const uint32_t sc = mx_scale_code(m);
          const float inv = mx_inv_scale(sc);
          if (in) {
            reinterpret_cast<uint2*>(row)[v] =
                make_uint2(e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                           e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
            if ((v & 3) == 0) sXs[(v >> 2) * kTok + wx] = live ? mx_scale_value(sc) : 0.f;
          }
        }
      }
      if (cta < nr) {  // the router's bf16 columns
        const int k0 = cta * kFewRouterRows;
        const int nv = min(kFewRouterRows, D - k0) >> 3;
        for (int v = lane; v < nv; v += 32)
          reinterpret_cast<uint4*>(sXr + wx * kRPitch)[v] = live ? __ldg(src + (k0 >> 3) + v) : make_uint4(0, 0, 0, 0);
      }
    }
  }
  bar_named(3, 2 * 32 * kFewConsWarps);

  if (warp > kFewConsWarps) {
    // ------------------------------------------------------------- routing
    const int wr = warp - 1 - kFewConsWarps;  // 0..7: tokens wr, wr + 8
    const int rt = wr * 32 + lane;
    if (rt == 0) *sRouteOk = counter_wait(c_router, nr, abort_flag, P.err) ? 1 : 0;  // one poller per CTA
    bar_named(2, 32 * kFewConsWarps);
    const bool ok = *sRouteOk != 0;
    if (ok) {
      for (int t = wr; t < P.T; t += 8) {
        // this lane's experts 4 lane .. 4 lane + 3: the partial logits in CTA order
        float l[4] = {0.f, 0.f, 0.f, 0.f};
        const int e4 = lane * 4;
        const bool in = e4 < P.E;
        for (int r = 0; r < nr; ++r) {
          const float4 v =
              __ldcg(reinterpret_cast<const float4*>(P.logit_part + (static_cast<size_t>(r) * 16 + t) * 128) + lane);
          l[0] += v.x;
          l[1] += v.y;
          l[2] += v.z;
          l[3] += v.w;
        }
        uint32_t key[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (in && P.bias) l[i] += __ldg(P.bias + e4 + i);
          key[i] = in ? max(order_key(l[i] + 0.f), 1u) : 0u;  // (-0 + 0 = +0); key 0: not to be taken
          if (in && cta == 0 && P.logits_out) P.logits_out[static_cast<size_t>(t) * P.E + e4 + i] = l[i];
        }
        for (int j = 0; j < P.k; ++j) {
          // the largest key, the lowest expert among equals
          uint32_t bk = key[0];
          int be = e4;
#pragma unroll
          for (int i = 1; i < 4; ++i)
            if (key[i] > bk) {
              bk = key[i];
              be = e4 + i;
            }
          const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
          const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, bk == top ? static_cast<uint32_t>(be) : 0xFFFFu));
          if (e4 == (e & ~3)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((e & 3) == i) {
                sSel[t * 128 + j] = l[i];
                key[i] = 0u;
              }
          }
          if (lane == 0) {
            if (cta == 0 && P.idx_out) P.idx_out[static_cast<size_t>(t) * P.k + j] = e;
            if (e >= P.e0 && e < P.e0 + P.el) atomicOr(&sTouched[e >> 5], 1u << (e & 31));
          }
          if (lane == 0) reinterpret_cast<int*>(sW)[t * 128 + j] = e;  // sW holds the choices until the list is built
        }
        __syncwarp();
        // softmax over the kept logits (slot 0 holds the largest)
        const float top = sSel[t * 128];
        float sum = 0.f;
        for (int j = lane; j < P.k; j += 32) sum += expf(sSel[t * 128 + j] - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncwarp();
        for (int j = lane; j < P.k; j += 32) {
          const float w = expf(sSel[t * 128 + j] - top) / sum;
          sSel[t * 128 + j] = w;
          if (cta == 0 && P.w_out) P.w_out[static_cast<size_t>(t) * P.k + j] = w;
        }
      }
    }
    bar_named(2, 32 * kFewConsWarps);
    // The list of touched experts, ascending. The chosen experts sit in sW
    // ([token][slot] as ints) and move to registers before sW becomes the weight table.
    int mine[kFewMaxTokens * 128 / 256];
#pragma unroll
    for (int i = 0; i < kFewMaxTokens * 128 / 256; ++i) mine[i] = reinterpret_cast<int*>(sW)[rt + 256 * i];
    bar_named(2, 32 * kFewConsWarps);
    for (int i = rt; i < 128 * 16; i += 256) sW[i] = 0.f;
    for (int i = rt; i < 128; i += 256) sBits[i] = 0;
    if (rt < 128) {
      const uint32_t word = sTouched[rt >> 5];
      if ((word >> (rt & 31)) & 1u) {
        int pos = __popc(word & ((1u << (rt & 31)) - 1u));
        for (int i = 0; i < (rt >> 5); ++i) pos += __popc(sTouched[i]);
        sList[pos] = rt - P.e0;
      }
    }
    if (rt == 0) *sCount = ok ? __popc(sTouched[0]) + __popc(sTouched[1]) + __popc(sTouched[2]) + __popc(sTouched[3]) : 0;
    bar_named(2, 32 * kFewConsWarps);
    if (ok) {
#pragma unroll
      for (int i = 0; i < kFewMaxTokens * 128 / 256; ++i) {
        const int a = rt + 256 * i, t = a >> 7, j = a & 127;
        if (t < P.T && j < P.k) {
          const int e = mine[i];
          if (e >= P.e0 && e < P.e0 + P.el) {
            int pos = __popc(sTouched[e >> 5] & ((1u << (e & 31)) - 1u));
            for (int q = 0; q < (e >> 5); ++q) pos += __popc(sTouched[q]);
            sW[pos * 16 + t] = sSel[t * 128 + j];
            atomicOr(&sBits[pos], 1u << t);
          }
        }
      }
    }
    bar_named(2, 32 * kFewConsWarps);
    if (rt == 0 && ok) mbar_arrive(routed);
    if (ok && cta == 0 && P.cnt_out && rt < P.E) {
      const uint32_t word = sTouched[rt >> 5];
      int c = 0;
      if ((word >> (rt & 31)) & 1u) {
        int pos = __popc(word & ((1u << (rt & 31)) - 1u));
        for (int i = 0; i < (rt >> 5); ++i) pos += __popc(sTouched[i]);
        c = __popc(sBits[pos]);
      }
      P.cnt_out[rt] = c;
    }
    return;
  }

  // ------------------------------------------------------------- consumers
  const int wc = warp - 1;           // 0..7
  const int ct = wc * 32 + lane;     // 0..255
  const int mrow = (wc & 3) * 16;    // this warp's 16 output columns inside its 64-column half
  int s = 0;
  uint32_t ph = 0, hph = 0;          // hph: bit per stage, parity of its next hfull phase
  auto wait_full = [&]() -> bool {
    int got = 1;
    if (lane == 0) got = mbar_wait(&full[s], ph, abort_flag, P.err);
    return __shfl_sync(0xffffffffu, got, 0) != 0;
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    if (++s == P.stages) {
      s = 0;
      ph ^= 1;
    }
  };
  // One bf16 chunk (64 K): A from the stage ([K][64 columns], 128-byte swizzle,
  // read transposed), B from rows xrow(token) + byte offset kb of bf16 x.
  auto mma_chunk_bf16 = [&](float (&acc)[NT][4], const uint8_t* xb, int pitch, int kb) {
    const uint32_t a0 = smem_u32(ring + s * kStage) + (wc >> 2) * 8192;
    const int r8 = lane & 7, q = lane >> 3;
    const int krow = r8 + ((q & 2) ? 8 : 0);
    const uint32_t colb = static_cast<uint32_t>((mrow + ((q & 1) ? 8 : 0)) * 2);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      uint32_t a[4];
      const int kk = ks * 16 + krow;
      ldsm_x4_trans(a0 + kk * 128 + (colb ^ ((kk & 7) << 4)), a);
      if constexpr (NT == 2) {
        uint32_t b[4];
        ldsm_x4(smem_u32(xb) + (r8 + ((q & 2) ? 8 : 0)) * pitch + kb + ks * 32 + ((q & 1) ? 16 : 0), b);
        mma_bf16(acc[0], a, b[0], b[1]);
        mma_bf16(acc[1], a, b[2], b[3]);
      } else {
        uint32_t b0, b1;
        ldsm_x2(smem_u32(xb) + r8 * pitch + kb + ks * 32 + ((q & 1) ? 16 : 0), b0, b1);
        mma_bf16(acc[0], a, b0, b1);
      }
    }
  };
  // The scale (as a float) of output column r (0..127 of its 128-block), group c, in a stage's scale tile.
  auto wscale = [&](const uint8_t* tile, int r, int c) -> float {
    return mx_scale_value(tile[16 * (r & 31) + 4 * (r >> 5) + c]);
  };
  // A of one MXFP8 32-K step: rows are output columns, 128-byte swizzled
  auto lda_mx = [&](int ks, uint32_t (&a)[4]) {
    const int r8 = lane & 7, q = lane >> 3;
    const int row = mrow + r8 + ((q & 1) ? 8 : 0);
    ldsm_x4(smem_u32(ring + s * kStage) + (wc >> 2) * 8192 + row * 128 +
                ((ks * 32 + ((q & 2) ? 16 : 0)) ^ ((row & 7) << 4)),
            a);
  };

  // After a wait gave up (ok = false) a warp does no more work and frees no more
  // stages, but keeps to the loops: their counts, and so the named barriers in them,
  // are the same for all eight warps.
  bool ok = true;
  // ---- R: partial logits of 256 K rows
  if (cta < nr) {
    float acc[NT][4] = {};
    const int k0 = cta * kFewRouterRows, k1 = min(D, k0 + kFewRouterRows);
    for (int kk = k0; kk < k1 && ok; kk += 64) {
      if (!wait_full()) {
        ok = false;
        break;
      }
      if constexpr (MX) {
        mma_chunk_bf16(acc, sXr, kRPitch, (kk - k0) * 2);
      } else {
        mma_chunk_bf16(acc, sX, xpitch, kk * 2);
      }
      release();
    }
    if (ok) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = n * 8 + 2 * (lane & 3) + (i & 1);
          const int e = (wc >> 2) * 64 + mrow + (lane >> 2) + ((i & 2) ? 8 : 0);
          if (t < P.T) P.logit_part[(static_cast<size_t>(cta) * 16 + t) * 128 + e] = acc[n][i];
        }
      __threadfence();
    }
    bar_named(1, 32 * kFewConsWarps);
    if (ct == 0 && ok) atomicAdd(c_router, 1u);
  }

  // ---- S, E: gate and up; warps 0..3 gate, 4..7 up
  // GeGLU rows of a unit (64 columns from hidden chunk position hk0 on) from this thread's four columns of one
  // token. Layout: the B fragments of down, so a K chunk is one contiguous copy.
  auto store_hidden = [&](int t, int c4, const float4& g, const float4& u, int chunk, int col0) {
    float v[4] = {gelu_tanh_exact(g.x) * u.x, gelu_tanh_exact(g.y) * u.y, gelu_tanh_exact(g.z) * u.z,
                  gelu_tanh_exact(g.w) * u.w};
    uint8_t* hc = P.h + static_cast<size_t>(chunk) * kHChunk;
    if constexpr (MX) {
      uint32_t m = max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 4));
      const uint32_t sc = mx_scale_code(m);
      const float inv = mx_inv_scale(sc);
      const int f = col0 + c4 * 4, ks = f >> 5, kk = f & 31;  // col0: 0 or 64 inside the 128-chunk
      // lane of the fragment: token, four K; register: K half
      *reinterpret_cast<uint32_t*>(hc + ((t >> 3) * 4 + ks) * 256 + ((t & 7) * 4 + ((kk & 15) >> 2)) * 8 +
                                   (kk >> 4) * 4) = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
      if ((c4 & 7) == 0) hc[NT * 1024 + t * 4 + ks] = static_cast<uint8_t>(sc);
    } else {
      const int f = c4 * 4, ks = f >> 4;
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        const int kk = (f + 2 * pr) & 15;
        float hi[2], lo[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = v[2 * pr + i];
          hi[i] = __bfloat162float(__float2bfloat16_rn(x));
          lo[i] = abs_bits(hi[i]) >= 0x7F800000u ? 0.f : x - hi[i];  // infinities and NaN stay in the high part
        }
        uint8_t* at = hc + (((t >> 3) * 4 + ks) * 2) * 256 + ((t & 7) * 4 + ((kk & 7) >> 1)) * 8 + (kk >> 3) * 4;
        *reinterpret_cast<uint32_t*>(at) = pack_bf16x2(hi[0], hi[1]);
        *reinterpret_cast<uint32_t*>(at + 256) = pack_bf16x2(lo[0], lo[1]);
      }
    }
  };
  auto run_gu = [&](const FewSplit& sp, int phase, int units_per, int chunk_base, int chunks_per, uint32_t* counters) {
    const int i0 = sp.begin(cta), i1 = sp.begin(cta + 1);
    for (int i = i0; i < i1;) {
      const int u = i / ck;
      const int iend = min(i1, (u + 1) * ck);
      const bool whole = i == u * ck && iend == (u + 1) * ck;
      const int seg = u == i0 / ck ? 0 : 1;
      const int half64 = ((u % units_per) & 1) * 64;  // MXFP8: this unit's half of the 128-row scale tiles
      float acc[NT][4] = {};
      for (; i < iend; ++i) {
        if (!ok || !wait_full()) {
          ok = false;
          continue;
        }
        const int kc = i - u * ck;
        if constexpr (MX) {
          const uint8_t* tile = ring + s * kStage + kFewWBytes + (wc >> 2) * 512;
          const int n32 = min(4, (D - kc * 128) / 32);
          for (int ks = 0; ks < n32; ++ks) {
            uint32_t a[4];
            lda_mx(ks, a);
            const float s0 = wscale(tile, half64 + mrow + (lane >> 2), ks);
            const float s1 = wscale(tile, half64 + mrow + (lane >> 2) + 8, ks);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              uint32_t b0, b1;
              const int r8 = lane & 7, q = lane >> 3;
              ldsm_x2(smem_u32(sX) + (n * 8 + r8) * xpitch + kc * 128 + ks * 32 + ((q & 1) ? 16 : 0), b0, b1);
              const float2 sx =
                  *reinterpret_cast<const float2*>(sXs + (kc * 4 + ks) * kTok + n * 8 + 2 * (lane & 3));
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_e4m3(d, a, b0, b1);
              acc[n][0] = fmaf(d[0], s0 * sx.x, acc[n][0]);
              acc[n][1] = fmaf(d[1], s0 * sx.y, acc[n][1]);
              acc[n][2] = fmaf(d[2], s1 * sx.x, acc[n][2]);
              acc[n][3] = fmaf(d[3], s1 * sx.y, acc[n][3]);
            }
          }
        } else {
          mma_chunk_bf16(acc, sX, xpitch, kc * 128);
        }
        release();
      }
      // exchange: [projection][token][column]
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sG[((wc >> 2) * kTok + n * 8 + 2 * (lane & 3) + (e & 1)) * kFewGPitch + mrow + (lane >> 2) +
             ((e & 2) ? 8 : 0)] = acc[n][e];
      bar_named(1, 32 * kFewConsWarps);
      const int t = ct >> 4, c4 = ct & 15;
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), up = g;
      if (t < kTok) {
        g = *reinterpret_cast<const float4*>(sG + t * kFewGPitch + c4 * 4);
        up = *reinterpret_cast<const float4*>(sG + (kTok + t) * kFewGPitch + c4 * 4);
      }
      bool finish = whole;
      if (!whole) {
        const size_t unit_f4 = 2 * kTok * 16;  // float4 of one partial unit
        float4* mine = reinterpret_cast<float4*>(P.part_gu) + ((static_cast<size_t>(cta) * 2 + phase) * 2 + seg) * unit_f4;
        if (t < kTok) {
          mine[t * 16 + c4] = g;
          mine[(kTok + t) * 16 + c4] = up;
        }
        __threadfence();
        bar_named(1, 32 * kFewConsWarps);
        const int ca = sp.cta_of(u * ck), cb = sp.cta_of((u + 1) * ck - 1);
        if (ct == 0) *sLast = ok && atomicAdd(counters + u, 1u) == static_cast<uint32_t>(cb - ca) ? 1 : 0;
        bar_named(1, 32 * kFewConsWarps);
        finish = *sLast != 0;
        if (finish) {
          __threadfence();
          g = make_float4(0.f, 0.f, 0.f, 0.f);
          up = g;
          if (t < kTok) {
            for (int c = ca; c <= cb; ++c) {
              const int sg = sp.begin(c) / ck == u ? 0 : 1;
              const float4* src =
                  reinterpret_cast<const float4*>(P.part_gu) + ((static_cast<size_t>(c) * 2 + phase) * 2 + sg) * unit_f4;
              const float4 a = __ldcg(src + t * 16 + c4), b = __ldcg(src + (kTok + t) * 16 + c4);
              g.x += a.x; g.y += a.y; g.z += a.z; g.w += a.w;
              up.x += b.x; up.y += b.y; up.z += b.z; up.w += b.w;
            }
          }
        }
      }
      if (finish) {
        const int ul = u % units_per;  // unit inside its expert
        const int chunk = chunk_base + (u / units_per) * chunks_per + (MX ? ul >> 1 : ul);
        if (t < kTok) store_hidden(t, c4, g, up, chunk, MX ? (ul & 1) * 64 : 0);
        fence_proxy_async();
        __threadfence();
      }
      bar_named(1, 32 * kFewConsWarps);  // sG and sLast are free again, the rows are written
    }
  };
  run_gu(split_s, 0, su, 0, ks_dn, c_su);
  if (ct == 0) *sLast = mbar_wait(routed, 0, abort_flag, P.err) ? 1 : 0;
  bar_named(1, 32 * kFewConsWarps);
  if (*sLast == 0) return;  // no routing: all eight warps leave (the wait has raised abort)
  const int nact = *sCount;
  bar_named(1, 32 * kFewConsWarps);  // sLast is free again
  if (nact > 0) {
    const FewSplit split_e(nact * fu, ck, grid);
    run_gu(split_e, 1, fu, ks_dn, ke_dn, c_eu);
  }
  // run_gu ends with a barrier after every thread's rows are written and fenced
  if (ct == 0 && ok) {
    __threadfence();
    atomicAdd(c_hidden, 1u);
  }

  // ---- D: down; each warp 16 of the tile's 128 columns
  const int len = ks_dn + nact * ke_dn;
  const FewSplit sp(nd, len, grid);
  const int i0 = sp.begin(cta), i1 = sp.begin(cta + 1);
  for (int i = i0; i < i1;) {
    const int u = i / len;
    const int iend = min(i1, (u + 1) * len);
    const int seg = u == i0 / len ? 0 : 1;
    float tot[NT][4] = {}, acc[NT][4] = {};
    int src = -2;  // the entry acc belongs to: -1 the shared MLP, else a touched expert
    auto fold = [&]() {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = n * 8 + 2 * (lane & 3) + (e & 1);
          if (src == -1) {
            tot[n][e] += acc[n][e];
          } else if (src >= 0 && ((sBits[src] >> t) & 1u)) {
            tot[n][e] = fmaf(sW[src * 16 + t], acc[n][e], tot[n][e]);
          }
          acc[n][e] = 0.f;
        }
    };
    for (; i < iend; ++i) {
      const int kc = i - u * len;
      const int from = kc < ks_dn ? -1 : (kc - ks_dn) / ke_dn;
      if (from != src) {
        fold();
        src = from;
      }
      if (!ok || !wait_full()) {
        ok = false;
        continue;
      }
      int got = 1;
      if (lane == 0) got = mbar_wait(&hfull[s], (hph >> s) & 1u, abort_flag, P.err);
      if (!__shfl_sync(0xffffffffu, got, 0)) {
        ok = false;
        continue;
      }
      hph ^= 1u << s;
      const uint8_t* hs = ring + s * kStage + kHOff;
      if constexpr (MX) {
        const int kl = from < 0 ? kc : (kc - ks_dn) % ke_dn;
        const int n32 = min(4, ((from < 0 ? P.S : P.F) - kl * 128) / 32);
        const uint8_t* tile = ring + s * kStage + kFewWBytes;
        const int r = (wc >> 2) * 64 + mrow + (lane >> 2);
        for (int ks = 0; ks < n32; ++ks) {
          uint32_t a[4];
          lda_mx(ks, a);
          const float s0 = wscale(tile, r, ks), s1 = wscale(tile, r + 8, ks);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 b = *reinterpret_cast<const uint2*>(hs + (n * 4 + ks) * 256 + lane * 8);
            const float x0 = mx_scale_value(hs[NT * 1024 + (n * 8 + 2 * (lane & 3)) * 4 + ks]);
            const float x1 = mx_scale_value(hs[NT * 1024 + (n * 8 + 2 * (lane & 3) + 1) * 4 + ks]);
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma_e4m3(d, a, b.x, b.y);
            acc[n][0] = fmaf(d[0], s0 * x0, acc[n][0]);
            acc[n][1] = fmaf(d[1], s0 * x1, acc[n][1]);
            acc[n][2] = fmaf(d[2], s1 * x0, acc[n][2]);
            acc[n][3] = fmaf(d[3], s1 * x1, acc[n][3]);
          }
        }
      } else {
        const uint32_t a0 = smem_u32(ring + s * kStage) + (wc >> 2) * 8192;
        const int krow = (lane & 7) + ((lane & 16) ? 8 : 0);
        const uint32_t colb = static_cast<uint32_t>((mrow + ((lane & 8) ? 8 : 0)) * 2);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          uint32_t a[4];
          const int kk = ks * 16 + krow;
          ldsm_x4_trans(a0 + kk * 128 + (colb ^ ((kk & 7) << 4)), a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 bh = *reinterpret_cast<const uint2*>(hs + ((n * 4 + ks) * 2) * 256 + lane * 8);
            const uint2 bl = *reinterpret_cast<const uint2*>(hs + ((n * 4 + ks) * 2 + 1) * 256 + lane * 8);
            mma_bf16(acc[n], a, bh.x, bh.y);
            mma_bf16(acc[n], a, bl.x, bl.y);
          }
        }
      }
      release();
    }
    fold();
    float* mine = P.part_dn + (static_cast<size_t>(cta) * 2 + seg) * kTok * 128;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        mine[(n * 8 + 2 * (lane & 3) + (e & 1)) * 128 + (wc >> 2) * 64 + mrow + (lane >> 2) + ((e & 2) ? 8 : 0)] =
            tot[n][e];
    __threadfence();
    bar_named(1, 32 * kFewConsWarps);
    const int ca = sp.cta_of(u * len), cb = sp.cta_of((u + 1) * len - 1);
    if (ct == 0) *sLast = ok && atomicAdd(c_dn + u, 1u) == static_cast<uint32_t>(cb - ca) ? 1 : 0;
    bar_named(1, 32 * kFewConsWarps);
    if (*sLast) {  // the tile's last CTA adds the parts in CTA order
      __threadfence();
      const int col = u * 128 + (ct & 31) * 4;
      const bool post = P.norm_post || P.residual;
      for (int t = ct >> 5; t < P.T; t += 8) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = ca; c <= cb; ++c) {
          const int sg = sp.begin(c) / len == u ? 0 : 1;
          const float4 b = __ldcg(
              reinterpret_cast<const float4*>(P.part_dn + ((static_cast<size_t>(c) * 2 + sg) * kTok + t) * 128) + (ct & 31));
          a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
        }
        if (col < D) {
          const size_t at = static_cast<size_t>(t) * D + col;
          if (post) {
            *reinterpret_cast<float4*>(P.f + at) = a;
          } else {
            if (P.out) *reinterpret_cast<uint2*>(P.out + at) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
            if (P.out_f32) *reinterpret_cast<float4*>(P.out_f32 + at) = a;
          }
        }
      }
      if (post) {  // norm_post needs whole rows: the CTA that finishes the last tile applies it
        __threadfence();
        bar_named(1, 32 * kFewConsWarps);
        if (ct == 0) *sLast = atomicAdd(c_tiles, 1u) == static_cast<uint32_t>(nd - 1) ? 2 : 1;
        bar_named(1, 32 * kFewConsWarps);
        if (*sLast == 2) {
          __threadfence();
          for (int t = wc; t < P.T; t += 8) {
            const float4* f = reinterpret_cast<const float4*>(P.f + static_cast<size_t>(t) * D);
            float r = 1.f;
            if (P.norm_post) {
              float ss = 0.f;
              for (int v = lane; v < (D >> 2); v += 32) {
                const float4 a = __ldcg(f + v);
                ss = fmaf(a.x, a.x, fmaf(a.y, a.y, fmaf(a.z, a.z, fmaf(a.w, a.w, ss))));
              }
#pragma unroll
              for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
              r = 1.0f / sqrtf(ss / static_cast<float>(D) + 1e-6f);
            }
            for (int v = lane; v < (D >> 2); v += 32) {
              const float4 a = __ldcg(f + v);
              float o[4] = {a.x * r, a.y * r, a.z * r, a.w * r};
              if (P.norm_post) {
                const uint2 gv = __ldg(reinterpret_cast<const uint2*>(P.norm_post) + v);
                const __nv_bfloat16* gb = reinterpret_cast<const __nv_bfloat16*>(&gv);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] *= __bfloat162float(gb[j]);
              }
              if (P.residual) {
                const uint2 xv = __ldg(reinterpret_cast<const uint2*>(P.x + static_cast<size_t>(t) * D) + v);
                const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(&xv);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] += __bfloat162float(xb[j]);
              }
              if (P.out)
                reinterpret_cast<uint2*>(P.out + static_cast<size_t>(t) * D)[v] =
                    make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
              if (P.out_f32)
                reinterpret_cast<float4*>(P.out_f32 + static_cast<size_t>(t) * D)[v] = make_float4(o[0], o[1], o[2], o[3]);
            }
          }
        }
      }
    }
    bar_named(1, 32 * kFewConsWarps);  // sLast is free again
  }
}

}  // namespace moe
