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
// in fp32; sum = RNE_bf16(s), y = RNE_bf16(y), q / scale = MXFP8(y) from the
// fp32 y (one rounding each), and where fp32 leaves a code open from y in 64
// bits (exact_codes). Memory bound: 4 bytes in and up to 5 + 1/32 out
// per element, the row held in registers between the passes. A row belongs to
// TPR threads, each with NV 8-column vectors: a warp per row up to 1024
// columns (no block barrier, and small rows fill the warp), 128 threads up to
// 4096, 512 up to 16384. Four neighbouring lanes hold one 32-group, so its
// maximum takes two shuffles. Sums: a thread's squares in order, a fixed
// xor tree, the warps in order - the same bits on every run.
// The loads are plain (not the read-only path): sum may overwrite residual or x in place.
// (The sum over a thread's columns is fp32, everything after it 64 bits.)
template <int TPR>
__device__ __forceinline__ double row_sum(float part, double* s_red) {
  double v = part;
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
// issue slots and 78 us on 16384 rows of 2816 (every output), at 4.7 TB/s; it
// now takes 73 us there (5.7 TB/s, 87% of the measured copy rate; 70 us
// without exact_codes, whose few warps end last) and 21 us on 4096 rows.
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

// The codes of a lane's eight values (s of 8-column vector v) and its group's scale code, decided in 64 bits. All lanes of
// a warp together. e4m3 has 3 mantissa bits, so an fp32 value a few units from the middle of two codes can land on the
// wrong side of it, which is a whole code step; the kernel comes here for the warps that hold such a value (0.2% of
// them), or a group maximum as near to 1.75 2^e. (Only rows of finite s and sums get here; a group of the warp may be NaN through
// gamma.)
__device__ __noinline__ void exact_codes(const AddNormParams& P, size_t row, int v, bool in, double ss, f32x2 s0,
                                         f32x2 s1, f32x2 s2, f32x2 s3) {
  const double a = ss * P.inv_d + static_cast<double>(P.eps), r0 = 1.0f / sqrtf(static_cast<float>(a));
  const double r = r0 * (1.5 - 0.5 * a * r0 * r0);  // a Newton step on fp32's: good to 2^-44
  uint4 gv = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  if (P.gamma && in) gv = __ldg(reinterpret_cast<const uint4*>(P.gamma) + v);
  const __nv_bfloat16* g = reinterpret_cast<const __nv_bfloat16*>(&gv);
  float f[8];
  unpack2(s0, f[0], f[1]);
  unpack2(s1, f[2], f[3]);
  unpack2(s2, f[4], f[5]);
  unpack2(s3, f[6], f[7]);
  double y[8], top = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = f[i] * (r * __bfloat162float(g[i]));
    // past fp32's largest value, or NaN (a gamma that is not finite): the group is NaN, as in fp32
    top = fabs(y[i]) <= 3.4028234663852886e38 ? fmax(top, fabs(y[i])) : INFINITY;
  }
  top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmax(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const long long b = __double_as_longlong(top);
  const int c = static_cast<int>(b >> 52) - 1023 + 127 - 8 + ((b & 0xFFFFFFFFFFFFFll) > 0xC000000000000ll ? 1 : 0);
  const uint32_t sc = isinf(top) ? 0xFFu : c < 0 ? 0u : static_cast<uint32_t>(c);
  const double inv = mx_inv_scale(sc);
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // to fp32 rounded to odd, so that the rounding to e4m3 is the only one
    const double w = y[i] * inv;
    const float z = __double2float_rz(w);
    f[i] = static_cast<double>(z) == w ? z : __uint_as_float(__float_as_uint(z) | 1u);
  }
  if (!in) return;
  reinterpret_cast<uint2*>(P.q + row)[v] = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
  if ((v & 3) == 0) P.scale[(row >> 5) + (v >> 2)] = static_cast<uint8_t>(sc);
}

template <int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) add_rms_norm_kernel(const __grid_constant__ AddNormParams P) {
  constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
  __shared__ double s_red[2][TPR / 32];
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
  f32x2 s[NV][4];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&xv[u]);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[u][i] = bf16x2_to_f32x2(w[i]);
  }
  // the sum of squares of the row in s (elements past D are zero), and 1 / rms
  auto sum_squares = [&](double* red) -> double {
    f32x2 ss = pack2(0.f, 0.f);
#pragma unroll
    for (int u = 0; u < NV; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = fma2(s[u][i], s[u][i], ss);
    float lo, hi;
    unpack2(ss, lo, hi);
    return row_sum<TPR>(lo + hi, red);
  };
  auto inv_rms = [&](double ss) -> float { return 1.0f / sqrtf(static_cast<float>(ss * P.inv_d) + P.eps); };
  if (P.gamma_post) {
    const float r1 = inv_rms(sum_squares(s_red[0]));
    const f32x2 r = pack2(r1, r1);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int v = lane + u * TPR;
      if (v >= nvec) continue;  // (stays zero)
      const uint4 gv = __ldg(reinterpret_cast<const uint4*>(P.gamma_post) + v);
      const uint32_t* g = reinterpret_cast<const uint32_t*>(&gv);
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&rv[u]);  // (zero without a residual)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // the product of two bf16 is exact in fp32: one rounding
        s[u][i] = fma2(mul2(s[u][i], bf16x2_to_f32x2(g[i])), r, bf16x2_to_f32x2(w[i]));
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
  const float r1 = inv_rms(ss);
  const f32x2 r = pack2(r1, r1);
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
      const float i1 = mx_inv_scale(sc);
      const f32x2 inv = pack2(i1, i1);
#pragma unroll
      for (int i = 0; i < 4; ++i) unpack2(mul2(o[i], inv), f[2 * i], f[2 * i + 1]);
      // a value within 4 units of the middle of two codes (r, s r and the product with gamma err by less), or a maximum
      // as near to where the scale changes
      constexpr uint32_t kNear = 4;
      uint32_t off = ((m & 0x7FFFFFu) - 0x600000u + kNear) & 0x7FFFFFu;
      float least = INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        off = min(off, (__float_as_uint(f[i]) - 0x80000u + kNear) & 0xFFFFFu);
        least = fminf(least, fabsf(f[i]));
      }
      // Below 2^-6 codes are 2^-9 apart, as in the binade from 2^-6 on: 2^-6 more has the middles' bits. At the smallest
      // scale an fp32 y may hold fewer than 24 bits.
      if (least < 0.015625f) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (fabsf(f[i]) < 0.015625f)
            off = min(off, (__float_as_uint(fabsf(f[i]) + 0.015625f) - 0x80000u + kNear) & 0xFFFFFu);
      }
      if (sc == 0 && m != 0) off = 0;
      if (off <= 2 * kNear) near |= 1u << u;
      if (in) {
        reinterpret_cast<uint2*>(P.q + row)[v] = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
        if ((v & 3) == 0) P.scale[static_cast<size_t>(t) * (P.D >> 5) + (v >> 2)] = static_cast<uint8_t>(sc);
      }
    }
  }
  if (!P.q) return;
#pragma unroll
  for (int u = 0; u < NV; ++u)
    if (__any_sync(0xffffffffu, (near >> u) & 1u))
      exact_codes(P, row, lane + u * TPR, lane + u * TPR < nvec, ss, s[u][0], s[u][1], s[u][2], s[u][3]);
}

}  // namespace moe
