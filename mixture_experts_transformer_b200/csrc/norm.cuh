// RMSNorm of rows with a learned scale: the pre-FFN norm of the block's
// normalisation sandwich (Gemma-4-26B-A4B model card: "Normalization layer
// type in the blocks": RMSNorm, "Pre-norm, post-norm, or sandwich":
// sandwich, epsilon 1e-06).
//
//   out[t, :] = RNE_bf16(gamma * x[t, :] / sqrt(mean(x[t, :]^2) + 1e-6))
//
// in fp32: one 128-thread CTA per row, each thread holding up to 4 of the
// row's 8-column vectors in registers (D <= 4096), so the row is read once;
// each thread sums its squares in order, then a fixed warp-xor tree and the
// warps in order: deterministic.
#pragma once

#include "mxformat.cuh"
#include "ptx.cuh"

namespace moe {

constexpr int kNormThreads = 128;
constexpr int kNormVec = 4;  // D <= 128 * 4 * 8 = 4096

__global__ void __launch_bounds__(kNormThreads) rms_norm_rows_kernel(const __nv_bfloat16* __restrict__ x,
                                                                    const __nv_bfloat16* __restrict__ gamma, int T,
                                                                    int D, __nv_bfloat16* __restrict__ out) {
  __shared__ float s_red[kNormThreads / 32];
  pdl_wait_then_release();
  const int t = blockIdx.x;
  const int nvec = D >> 3;
  const uint4* row = reinterpret_cast<const uint4*>(x + static_cast<size_t>(t) * D);
  uint4 xv[kNormVec];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < kNormVec; ++u) {
    const int v = threadIdx.x + u * kNormThreads;
    xv[u] = v < nvec ? __ldg(row + v) : make_uint4(0, 0, 0, 0);
    const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(&xv[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float f = __bfloat162float(xb[i]);
      ss = fmaf(f, f, ss);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = ss;
  __syncthreads();
  float tot = 0.f;
#pragma unroll
  for (int i = 0; i < kNormThreads / 32; ++i) tot += s_red[i];
  const float r = 1.0f / sqrtf(tot / static_cast<float>(D) + 1e-6f);
  uint4* dst = reinterpret_cast<uint4*>(out + static_cast<size_t>(t) * D);
#pragma unroll
  for (int u = 0; u < kNormVec; ++u) {
    const int v = threadIdx.x + u * kNormThreads;
    if (v >= nvec) continue;
    const uint4 gv = __ldg(reinterpret_cast<const uint4*>(gamma) + v);
    const __nv_bfloat16* xb = reinterpret_cast<const __nv_bfloat16*>(&xv[u]);
    const __nv_bfloat16* gb = reinterpret_cast<const __nv_bfloat16*>(&gv);
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = __bfloat162float(xb[i]) * r * __bfloat162float(gb[i]);
    dst[v] = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                        pack_bf16x2(o[6], o[7]));
  }
}

// Residual addition, RMSNorm and 8-bit output in one pass over the rows - the
// seam between two sub-layers of the sandwich (post-norm of one, residual,
// pre-norm of the next):
//
//   s[t] = residual[t] + (gamma_post x[t] / rms(x[t])  or  x[t])
//   y[t] = gamma s[t] / rms(s[t]),   rms(v) = sqrt(mean(v^2) + eps)
//
// in fp32; sum = RNE_bf16(s), y = RNE_bf16(y), q / scale = MXFP8(y) (one
// rounding each). e4m3 has 3 mantissa bits, so an fp32 y a few units from the
// middle of two codes can land on the wrong side of it, which is a whole code
// step: the codes of such values are decided in 64 bits, from x on
// (exact_codes). What fp32 keeps a part in is the sum of squares of s, eight
// at a time: at most 4.5 units of y, and nearly always under a tenth of one
// (the whole row in 64 bits, where a value is open: T = 64 3 -> 5 us, 16384
// rows 77 -> 83). Memory bound: 4 bytes in and up to 5 + 1/32 out
// per element, the row held in registers between the passes. A row belongs to
// TPR threads, each with NV 8-column vectors: a warp per row up to 1024
// columns (no block barrier, and small rows fill the warp), 128 threads up to
// 4096 (three vectors each up to 3/4 of that, four above), 512 up to 16384.
// Four neighbouring lanes hold one 32-group, so its maximum takes two
// shuffles. Sums: a thread's squares in order, a fixed xor tree, the warps in
// order - the same bits on every run.
// The loads are plain (not the read-only path): sum and y may overwrite
// residual or x in place.
template <int TPR>
__device__ __forceinline__ double row_sum(double v, double* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += s_red[i];
  }
  return v;
}

struct AddNormParams {
  int T, D;
  float eps;
  double inv_d;  // 1 / D
  const __nv_bfloat16* x;
  const __nv_bfloat16* residual;
  const __nv_bfloat16* gamma_post;
  const __nv_bfloat16* gamma;
  __nv_bfloat16* sum;
  __nv_bfloat16* y;
  uint8_t* q;
  uint8_t* scale;
};

// Two fp32 values in a 64-bit register pair, handled by the packed fp32
// instructions: with one instruction per value the kernel spent 62% of its
// issue slots and 78 us on 16384 rows of 2816 (every output), at 4.7 TB/s,
// against 70 us with them; 78 us with the codes' 64-bit decision (82% of the
// measured copy rate), and 21 us on 4096 rows without a post-norm.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 bf16x2_to_f32x2(uint32_t u) {
  return pack2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(f32x2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
// the larger magnitude; a NaN stays one
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}
// The magnitude of a bf16 value in 64 bits, by its bits: the exponent's bias is 896 larger. 0 becomes 2^-127 and
// infinities and NaN 2^128 and more, which a sum of squares shows.
__device__ __forceinline__ double bf16_abs_to_double(float v) {
  return __hiloint2double(static_cast<int>(((__float_as_uint(v) & 0x7FFFFFFFu) >> 3) + (896u << 20)), 0);
}

// The codes of a lane's eight values (8-column vector v of row t) and its group's scale code, decided in 64 bits from x,
// the residual and the gammas. All lanes of a warp together: the kernel comes here for the warps that hold a value, or a
// group maximum, that fp32 leaves open (1% of them). r, r1: 1 / rms of s and of x, in 64 bits. (Only rows whose sums are
// finite get here; a group of the warp may be NaN through gamma.)
__device__ __noinline__ void exact_codes(const AddNormParams& P, size_t row, int v, bool in, double r, double r1, uint4 xv,
                                         uint4 rv) {
  uint4 gv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), pv = gv;
  if (P.gamma && in) gv = __ldg(reinterpret_cast<const uint4*>(P.gamma) + v);
  if (P.gamma_post && in) pv = __ldg(reinterpret_cast<const uint4*>(P.gamma_post) + v);
  const __nv_bfloat16* x = reinterpret_cast<const __nv_bfloat16*>(&xv);
  const __nv_bfloat16* z = reinterpret_cast<const __nv_bfloat16*>(&rv);
  const __nv_bfloat16* g = reinterpret_cast<const __nv_bfloat16*>(&gv);
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(&pv);
  double y[8], top = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // (the product of two bf16 is exact in fp32)
    const double a = static_cast<double>(__bfloat162float(x[i]) * __bfloat162float(p[i])) * r1;
    y[i] = (a + __bfloat162float(z[i])) * (r * __bfloat162float(g[i]));
    // past fp32's largest value, or NaN (a gamma that is not finite): the group is NaN, as in fp32
    top = fabs(y[i]) <= 3.4028234663852886e38 ? fmax(top, fabs(y[i])) : INFINITY;
  }
  top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const long long b = __double_as_longlong(top);
  const int c = static_cast<int>(b >> 52) - 1023 + 127 - 8 + ((b & 0xFFFFFFFFFFFFFll) > 0xC000000000000ll ? 1 : 0);
  const uint32_t sc = isinf(top) ? 0xFFu : c < 0 ? 0u : static_cast<uint32_t>(c);
  const double inv = mx_inv_scale(sc);
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // to fp32 rounded to odd, so that the rounding to e4m3 is the only one
    const double w = y[i] * inv;
    const float o = __double2float_rz(w);
    f[i] = static_cast<double>(o) == w ? o : __uint_as_float(__float_as_uint(o) | 1u);
  }
  if (!in) return;
  reinterpret_cast<uint2*>(P.q + row)[v] = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
  if ((v & 3) == 0) P.scale[(row >> 5) + (v >> 2)] = static_cast<uint8_t>(sc);
}

// KEEP: 8-bit output with sum or y over x or residual: exact_codes finds both in shared memory.
__host__ __device__ constexpr int norm_threads(int tpr) { return tpr < 128 ? 128 : tpr; }
__host__ __device__ constexpr int norm_smem(int tpr, int nv, bool keep) { return keep ? norm_threads(tpr) * nv * 2 * 16 : 0; }
// Blocks an SM holds by their registers: 56 a thread for up to three vectors, 64 for four (72 in a warp's row).
__host__ __device__ constexpr int norm_blocks(int tpr, int nv) {
  return 65536 / (norm_threads(tpr) * (nv < 4 ? 56 : tpr == 32 ? 72 : 64));
}
template <int TPR, int NV, bool KEEP>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks(TPR, NV)) add_rms_norm_kernel(const __grid_constant__ AddNormParams P) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  __shared__ double s_red[3][TPR / 32];
  extern __shared__ uint4 s_keep[];  // [NV][x, residual][thread]
  pdl_wait_then_release();
  const int lane = threadIdx.x % TPR;
  const int t = blockIdx.x * kRows + threadIdx.x / TPR;
  if (t >= P.T) return;  // TPR < 128 only: whole warps, no block barrier follows
  const int nvec = P.D >> 3;
  const size_t row = static_cast<size_t>(t) * P.D;
  uint4 xv[NV], rv[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int v = lane + u * TPR;
    xv[u] = rv[u] = make_uint4(0, 0, 0, 0);
    if (v < nvec) xv[u] = reinterpret_cast<const uint4*>(P.x + row)[v];
  }
  if (P.residual) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = lane + u * TPR;
      if (v < nvec) rv[u] = reinterpret_cast<const uint4*>(P.residual + row)[v];
    }
  }
  if constexpr (KEEP) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      s_keep[(2 * u) * norm_threads(TPR) + threadIdx.x] = xv[u];
      s_keep[(2 * u + 1) * norm_threads(TPR) + threadIdx.x] = rv[u];
    }
  }
  f32x2 s[NV][4];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&xv[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[u][i] = bf16x2_to_f32x2(w[i]);
  }
  // the sum of squares of the row in s (elements past D are zero): a vector's in fp32, at most 5 roundings, then 64 bits
  auto sum_squares = [&](double* red) -> double {
    double ss = 0.0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      f32x2 p = mul2(s[u][0], s[u][0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) p = fma2(s[u][i], s[u][i], p);
      float lo, hi;
      unpack2(p, lo, hi);
      ss += static_cast<double>(lo + hi);
    }
    return row_sum<TPR>(ss, red);
  };
  auto mean_eps = [&](double ss) -> double { return ss * P.inv_d + static_cast<double>(P.eps); };
  double r1 = 1.0;
  if (P.gamma_post) {
    // 1 / rms of x in 64 bits, and as two fp32 values: where the residual cancels the post-norm, its error would be all
    // that is left
    double part[4] = {};
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[2];
        unpack2(s[u][i], f[0], f[1]);
        const double lo = bf16_abs_to_double(f[0]), hi = bf16_abs_to_double(f[1]);
        part[i] = fma(lo, lo, fma(hi, hi, part[i]));
      }
    double ss = row_sum<TPR>((part[0] + part[1]) + (part[2] + part[3]), s_red[0]);
    if (ss >= 0x1p256) ss = sum_squares(s_red[2]);  // an infinity or NaN in the row, or nearly one: as fp32 has it
    r1 = rsqrt(mean_eps(ss));
    const float rh = static_cast<float>(r1), rl = static_cast<float>(r1 - rh);
    const f32x2 r_hi = pack2(rh, rh), r_lo = pack2(rl, rl);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = lane + u * TPR;
      if (v >= nvec) continue;  // (stays zero)
      const uint4 gv = __ldg(reinterpret_cast<const uint4*>(P.gamma_post) + v);
      const uint32_t* g = reinterpret_cast<const uint32_t*>(&gv);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&rv[u]);  // (zero without a residual)
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // the product of two bf16 is exact in fp32: a rounding for each half of r1
        const f32x2 xg = mul2(s[u][i], bf16x2_to_f32x2(g[i]));
        s[u][i] = fma2(xg, r_lo, fma2(xg, r_hi, bf16x2_to_f32x2(w[i])));
      }
    }
  } else if (P.residual) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&rv[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u][i] = add2(s[u][i], bf16x2_to_f32x2(w[i]));
    }
  }
  if (P.sum) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = lane + u * TPR;
      if (v < nvec)
        reinterpret_cast<uint4*>(P.sum + row)[v] = make_uint4(f32x2_to_bf16x2(s[u][0]), f32x2_to_bf16x2(s[u][1]),
                                                              f32x2_to_bf16x2(s[u][2]), f32x2_to_bf16x2(s[u][3]));
    }
  }
  if (!P.y && !P.q) return;
  const double ss = sum_squares(s_red[1]);
  // (this root by rsqrt in 64 bits: 3 us more of 65 for 16384 rows, all of it latency)
  const float r32 = 1.0f / sqrtf(static_cast<float>(mean_eps(ss)));
  const f32x2 r = pack2(r32, r32);
  // How far y may be off, in 2^-24 of itself: s 1 (after a post-norm its two roundings and, unless the residual leaves
  // less than 2^-20 of it, a trace of r1's), r half of the sum's 5 and of what s brings twice, and 2.5 of its own (its
  // mean, the root, the quotient), the products 2. So y (1 - d) and y (1 + d) lie on either side of it, and where both
  // round to one code it is y's. (Their scaling rounds once more. The bits' distance from the middles' patterns, subnormal
  // codes apart: 85 us against 78 for 16384 rows.)
  const uint32_t off = P.gamma_post ? 12 : 9;
  const float d = P.gamma_post ? 7.f / 8388608 : 5.f / 8388608;
  uint32_t near = 0;  // bit u: vector u holds a value that fp32 leaves open
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int v = lane + u * TPR;
    const bool in = v < nvec;
    f32x2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = mul2(s[u][i], r);
    if (P.gamma && in) {
      const uint4 gv = __ldg(reinterpret_cast<const uint4*>(P.gamma) + v);
      const uint32_t* g = reinterpret_cast<const uint32_t*>(&gv);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = mul2(o[i], bf16x2_to_f32x2(g[i]));
    }
    if (P.y && in)
      reinterpret_cast<uint4*>(P.y + row)[v] = make_uint4(f32x2_to_bf16x2(o[0]), f32x2_to_bf16x2(o[1]),
                                                          f32x2_to_bf16x2(o[2]), f32x2_to_bf16x2(o[3]));
    if (P.q) {
      float f[8], mf = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unpack2(o[i], f[2 * i], f[2 * i + 1]);
        mf = max_abs(max_abs(mf, f[2 * i]), f[2 * i + 1]);
      }
      // the four lanes of a 32-group (D is a multiple of 32: all in range, or none)
      uint32_t m = __float_as_uint(mf) & 0x7FFFFFFFu;
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const uint32_t sc = mx_scale_code(m);
      auto codes_of = [&](float inv) -> uint2 {
        const f32x2 i2 = pack2(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack2(mul2(o[i], i2), f[2 * i], f[2 * i + 1]);
        return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
      };
      const float inv = mx_inv_scale(sc);
      const uint2 codes = codes_of(inv * (1.f + d)), other = codes_of(inv * (1.f - d));
      // or a maximum as near to where the scale changes, or one of the smallest scales, where an fp32 y may hold fewer bits
      // of a value that is not rounded to zero (24 bits of 2^-10 2^(sc - 127) end at 2^-149 for sc = 11)
      if (codes.x != other.x || codes.y != other.y || ((m & 0x7FFFFFu) - 0x600000u + off) <= 2 * off ||
          (sc < 11 && m != 0))
        near |= 1u << u;
      if (in) {
        reinterpret_cast<uint2*>(P.q + row)[v] = codes;
        if ((v & 3) == 0) P.scale[static_cast<size_t>(t) * (P.D >> 5) + (v >> 2)] = static_cast<uint8_t>(sc);
      }
    }
  }
  if (!P.q) return;
#pragma unroll 1
  for (int u = 0; u < NV; ++u) {
    if (!__any_sync(0xffffffffu, (near >> u) & 1u)) continue;
    const int v = lane + u * TPR;
    uint4 x = make_uint4(0, 0, 0, 0), z = x;
    if constexpr (KEEP) {
      x = s_keep[(2 * u) * norm_threads(TPR) + threadIdx.x];
      z = s_keep[(2 * u + 1) * norm_threads(TPR) + threadIdx.x];
    } else if (v < nvec) {
      x = reinterpret_cast<const uint4*>(P.x + row)[v];
      if (P.residual) z = reinterpret_cast<const uint4*>(P.residual + row)[v];
    }
    exact_codes(P, row, v, v < nvec, rsqrt(mean_eps(ss)), r1, x, z);
  }
}

}  // namespace moe
