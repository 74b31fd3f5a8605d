// RMS norm with the residual's addition, fused with the activation quantizer: the step
// before every quantized linear layer of a pre-norm decoder (the activations that the
// BATQuant note, en.papernotes.org, Method > Key Designs 4, transforms before qkv and
// gate/up).
//
//   h = x + r            (fp32; the bf16 rounding of h is the new residual stream)
//   y = h * (mean_k(h^2) + eps)^(-1/2) * w       (fp32, never rounded before the transform)
//   codes, scales = Q(clip(y P))                 (transform, clip and MX formats of the
//                                                 row quantizer)
//
// Bound: HBM. It reads x and r (4 bytes an element) and writes r' and the codes (2 + 1, or
// 2 + 1/2): 7 bytes an element for MXFP8, against 13 for a norm kernel that writes bf16
// followed by the quantizer. About 25 instructions an element, so that the issue slots stay
// below the memory time.
//
// Layout: eight consecutive channels (one 16-byte load) a lane, so the four lanes of a quad
// hold the four rows of a block's 4 x 8 view X_r. (X_r A) is a product within the lane
// (A's rows read from shared memory, the same address for the whole warp), B_b^T (X_r A)
// mixes the quad's rows by shuffles: 12 multiply-adds an element instead of the 32 of the
// 32 x 32 block matrix. A row stays in registers between the norm's sum and the
// quantization (kV vectors a thread), and the next row of the CTA is requested before the
// sum's barrier. Rows too wide for that (K > kMaxCachedK) are read twice.
#pragma once

#include "bat_common.cuh"

namespace bat {

namespace norm {
constexpr int kMaxThreads = 512;
constexpr int kMaxCachedK = kMaxThreads * 8 * 4;  // widest row that stays in registers
}  // namespace norm

struct NormParams {
  const uint16_t* x;    // bf16 [M][K]
  const uint16_t* res;  // bf16 [M][K] or null
  const uint16_t* w;    // bf16 [K]
  const float* a;       // [s][s] or null (no transform)
  const float* b;       // [K/32][t][t]
  const float* g_lo;    // [K/32] clip logits or null
  const float* g_hi;
  uint16_t* res_out;    // bf16 [M][K] or null; may be `res`
  uint8_t* codes;
  uint8_t* scales;
  float* y_out;         // optional fp32 [M][K]: y P before the clip
  int64_t M, mpad;      // mpad: M rounded up to 128 (scale padding rows)
  int K, nb, nbp4, ls;
  float eps, inv_k;
};

__device__ __forceinline__ void norm_unpack(const uint4& w, float (&v)[8]) {
  v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}

__device__ __forceinline__ uint32_t norm_pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Transform, clip, scale and codes of the eight channels 8 vec .. 8 vec + 7 (y: the
// normalised values). Every lane of the warp calls it; lanes without a vector (has false)
// take part in the shuffles with zeros.
//   kX: 0 no transform, 1 the 8 x 8 / 4 x 4 split, 2 any other split.
template <int kX, bool kFp8>
__device__ __forceinline__ void norm_quant_vec(const NormParams& p, float (&y)[8], int vec, bool has,
                                               int64_t row, const float* sa, const float (&bq)[4],
                                               float r_lo, float r_hi) {
  const int lane = threadIdx.x & 31;
  const int blk = vec >> 2;
  if (kX == 1) {
    uint64_t z[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(sa + 8 * k);
      const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(sa + 8 * k + 4);
      const uint64_t yy = pack2(y[k], y[k]);
      z[0] = ffma2(yy, a0.x, z[0]);
      z[1] = ffma2(yy, a0.y, z[1]);
      z[2] = ffma2(yy, a1.x, z[2]);
      z[3] = ffma2(yy, a1.y, z[3]);
    }
    // output row j (this lane's) = sum_i B[i][j] (X_r A)[i]; the lane at distance d holds
    // row j ^ d, and bq[d] = B[j ^ d][j]
    const uint64_t b0 = pack2(bq[0], bq[0]);
    uint64_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = fmul2(b0, z[q]);
#pragma unroll
    for (int d = 1; d < 4; ++d) {
      const uint64_t bd = pack2(bq[d], bq[d]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float lo, hi;
        unpack2(z[q], lo, hi);
        lo = __shfl_xor_sync(0xffffffffu, lo, d);
        hi = __shfl_xor_sync(0xffffffffu, hi, d);
        o[q] = ffma2(bd, pack2(lo, hi), o[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) unpack2(o[q], y[2 * q], y[2 * q + 1]);
  } else if (kX == 2) {
    const int sm = (1 << p.ls) - 1, t = 32 >> p.ls, n0 = 8 * (lane & 3);
    const float* bb = p.b + static_cast<int64_t>(has ? blk : 0) * t * t;
    float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float xk = __shfl_sync(0xffffffffu, y[k & 7], (lane & ~3) + (k >> 3));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int n = n0 + j;
        const float pk = __fmul_rn(__ldg(bb + (k >> p.ls) * t + (n >> p.ls)),
                                   __ldg(p.a + ((k & sm) << p.ls) + (n & sm)));
        o[j] = __fmaf_rn(xk, pk, o[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = o[j];
  }
  float mn = y[0], mx = y[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mn = fminf(mn, y[j]);
    mx = fmaxf(mx, y[j]);
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  }
  const float lo = __fmul_rn(r_lo, mn), hi = __fmul_rn(r_hi, mx);
  const float amax = fmaxf(fabsf(fminf(fmaxf(mn, lo), hi)), fabsf(fminf(fmaxf(mx, lo), hi)));
  constexpr int kEmax = kFp8 ? 8 : 2;
  const int ef = static_cast<int>(__float_as_uint(amax) >> 23);
  const int sbyte = has && ef > kEmax ? ef - kEmax : 0;
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - sbyte) << 23);
  float v[8];
  // the addend 0 makes an exact zero +0
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __fmaf_rn(fminf(fmaxf(y[j], lo), hi), inv, 0.0f);
  const int64_t e0 = row * p.K + 8 * static_cast<int64_t>(vec);
  if (has) {
    if (kFp8) {
      uint2 c;
      c.x = e4m3x4(v[0], v[1], v[2], v[3]);
      c.y = e4m3x4(v[4], v[5], v[6], v[7]);
      *reinterpret_cast<uint2*>(p.codes + e0) = c;
    } else {
      *reinterpret_cast<uint32_t*>(p.codes + e0 / 2) = e2m1x8(v);
    }
    if (p.y_out) {
      *reinterpret_cast<float4*>(p.y_out + e0) = make_float4(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<float4*>(p.y_out + e0 + 4) = make_float4(y[4], y[5], y[6], y[7]);
    }
  }
  // the scale bytes of blocks 4g .. 4g+3 are one word of the tiled layout; blocks past nb
  // come from lanes without a vector and are the layout's zero padding
  uint32_t word = static_cast<uint32_t>(sbyte) << (8 * (blk & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  word |= __shfl_xor_sync(0xffffffffu, word, 8);
  if (has && (lane & 15) == 0)
    *reinterpret_cast<uint32_t*>(p.scales + scale_offset(row, blk, p.nbp4)) = word;
}

// Sum of v over the CTA (every thread gets it; fixed order). `red` holds one float a warp
// and is free again after the next barrier.
__device__ __forceinline__ float norm_cta_sum(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// kV > 0: the row's kV vectors a thread stay in registers (kV * 8 * blockDim.x >= K).
// kV == 0: any K, the row is read once for the sum and once for the codes.
template <int kV, int kX, bool kFp8>
__global__ void __launch_bounds__(norm::kMaxThreads)
    bat_rmsnorm_quantize_kernel(const NormParams p) {
  __shared__ __align__(16) float sa[64];
  __shared__ float red[2][norm::kMaxThreads / 32];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = p.K >> 3;
  if (kX == 1 && tid < 64) sa[tid] = p.a[tid];
  __syncthreads();
  constexpr int kN = kV > 0 ? kV : 1;
  float bq[kN][4], r_lo[kN], r_hi[kN];
  uint4 wv[kN];
  auto load_block = [&](int i, int vec) {
    const bool has = vec < nvec;
    const int blk = has ? vec >> 2 : 0, j = tid & 3;
    if (kX == 1) {
#pragma unroll
      for (int d = 0; d < 4; ++d) bq[i][d] = __ldg(p.b + 16 * static_cast<int64_t>(blk) + 4 * (j ^ d) + j);
    }
    r_lo[i] = p.g_lo ? clip_ratio(__ldg(p.g_lo + blk)) : 1.0f;
    r_hi[i] = p.g_hi ? clip_ratio(__ldg(p.g_hi + blk)) : 1.0f;
    wv[i] = has ? __ldg(reinterpret_cast<const uint4*>(p.w) + vec) : make_uint4(0u, 0u, 0u, 0u);
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (kV > 0) {
    uint4 xv[kN], rv[kN];
    auto fetch = [&](int64_t row) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int vec = tid + i * nt;
        const bool has = vec < nvec && row < p.M;
        xv[i] = has ? *(reinterpret_cast<const uint4*>(p.x + row * p.K) + vec) : zero;
        rv[i] = has && p.res ? *(reinterpret_cast<const uint4*>(p.res + row * p.K) + vec) : zero;
      }
    };
    int64_t row = blockIdx.x;
    fetch(row);
#pragma unroll
    for (int i = 0; i < kN; ++i) load_block(i, tid + i * nt);
    int turn = 0;
    for (; row < p.M; row += gridDim.x, turn ^= 1) {
      float h[kN][8], ss = 0.0f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float r8[8];
        norm_unpack(xv[i], h[i]);
        norm_unpack(rv[i], r8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[i][j] += r8[j];
          ss = __fmaf_rn(h[i][j], h[i][j], ss);
        }
        const int vec = tid + i * nt;
        if (p.res_out && vec < nvec) {
          uint4 o;
          o.x = norm_pack_bf16(h[i][0], h[i][1]);
          o.y = norm_pack_bf16(h[i][2], h[i][3]);
          o.z = norm_pack_bf16(h[i][4], h[i][5]);
          o.w = norm_pack_bf16(h[i][6], h[i][7]);
          *(reinterpret_cast<uint4*>(p.res_out + row * p.K) + vec) = o;
        }
      }
      fetch(row + gridDim.x);
      const float inv = __frsqrt_rn(__fmaf_rn(norm_cta_sum(ss, red[turn]), p.inv_k, p.eps));
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        float w8[8];
        norm_unpack(wv[i], w8);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * inv * w8[j];
        const int vec = tid + i * nt;
        norm_quant_vec<kX, kFp8>(p, h[i], vec, vec < nvec, row, sa, bq[i], r_lo[i], r_hi[i]);
      }
    }
  } else {
    const int iters = (nvec + nt - 1) / nt;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
      const uint4* xr = reinterpret_cast<const uint4*>(p.x + row * p.K);
      const uint4* rr = reinterpret_cast<const uint4*>(p.res + row * p.K);
      float ss = 0.0f;
      for (int vec = tid; vec < nvec; vec += nt) {
        float h[8], r8[8];
        norm_unpack(xr[vec], h);
        norm_unpack(p.res ? rr[vec] : zero, r8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[j] += r8[j];
          ss = __fmaf_rn(h[j], h[j], ss);
        }
      }
      const float inv = __frsqrt_rn(__fmaf_rn(norm_cta_sum(ss, red[turn]), p.inv_k, p.eps));
      for (int it = 0; it < iters; ++it) {
        const int vec = tid + it * nt;
        const bool has = vec < nvec;
        load_block(0, vec);
        float h[8], r8[8], w8[8];
        norm_unpack(has ? xr[vec] : zero, h);
        norm_unpack(has && p.res ? rr[vec] : zero, r8);
        norm_unpack(wv[0], w8);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r8[j];
        if (p.res_out && has) {
          uint4 o;
          o.x = norm_pack_bf16(h[0], h[1]);
          o.y = norm_pack_bf16(h[2], h[3]);
          o.z = norm_pack_bf16(h[4], h[5]);
          o.w = norm_pack_bf16(h[6], h[7]);
          *(reinterpret_cast<uint4*>(p.res_out + row * p.K) + vec) = o;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = h[j] * inv * w8[j];
        norm_quant_vec<kX, kFp8>(p, h, vec, has, row, sa, bq[0], r_lo[0], r_hi[0]);
      }
    }
  }
  // padding rows of the tiled scale layout
  const int64_t pad = (p.mpad - p.M) * p.nbp4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * nt + tid; i < pad; i += static_cast<int64_t>(gridDim.x) * nt)
    *reinterpret_cast<uint32_t*>(p.scales + scale_offset(p.M + i / p.nbp4, 4 * (i % p.nbp4), p.nbp4)) = 0u;
}

}  // namespace bat
