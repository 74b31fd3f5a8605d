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
// followed by the quantizer. The issue slots come next (27 instructions an element), and the
// layout below is chosen for few of them.
//
// Layout: 16 consecutive channels (two 16-byte loads) a lane, so a pair of lanes holds the four
// rows of a block's 4 x 8 view X_r, two each. (X_r A) is a product within the lane (A's rows from
// shared memory, one address for the whole warp, each used for both rows); B_b^T (X_r A) takes the
// other lane's two rows by 16 shuffles. 12 multiply-adds an element instead of the 32 of the
// 32 x 32 block matrix. (8 channels a lane, a quad a block: 332 instead of 219 instructions for
// 8 channels; 16384 x 4096 took 132 us.) 16384 x 4096 in MXFP8: 102 us, 4.6 TB/s.
// Other splits (kX 2) form each coefficient from A and B as it comes and spill (up to 6 KB a thread for rows of 8192 to
// 16384 channels): right, but 16384 x 4096 takes 4.1 ms (1.0 with s = 16).
// The transform is linear and the norm's root a factor of the whole row, so the transform runs
// on h w while the row's sum is still on its way through the barrier, and the root is multiplied
// in afterwards. A row stays in registers, and the next row of the CTA is requested before that
// barrier. Rows too wide for that (K > kMaxCachedK) are read twice.
#pragma once

#include "bat_common.cuh"

namespace bat {

namespace norm {
constexpr int kMaxThreads = 512;
constexpr int kMaxCachedK = kMaxThreads * 16 * 2;  // widest row that stays in registers
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

// y = (h w) P of the lane's 16 channels 16 vec .. 16 vec + 15 (y: h w), without the row's root.
// Every lane of the warp calls it; lanes without channels (has false) take part with zeros.
//   kX: 0 no transform, 1 the 8 x 8 / 4 x 4 split, 2 any other split.
//   bq: for output row j and input row i of the lane's half: own B[2 h + i][2 h + j] at 2 j + i, and
//   from the other lane's half B[2 (1 - h) + i][2 h + j] at 4 + 2 j + i.
template <int kX>
__device__ __forceinline__ void norm_transform(const NormParams& p, float (&y)[16], int vec, bool has,
                                               const float* sa, const float (&bq)[8]) {
  const int lane = threadIdx.x & 31;
  if (kX == 1) {
    uint64_t z[2][4] = {{0ull, 0ull, 0ull, 0ull}, {0ull, 0ull, 0ull, 0ull}};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(sa + 8 * k);
      const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(sa + 8 * k + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint64_t yy = pack2(y[8 * i + k], y[8 * i + k]);
        z[i][0] = ffma2(yy, a0.x, z[i][0]);
        z[i][1] = ffma2(yy, a0.y, z[i][1]);
        z[i][2] = ffma2(yy, a1.x, z[i][2]);
        z[i][3] = ffma2(yy, a1.y, z[i][3]);
      }
    }
    uint64_t o[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[j][q] = ffma2(pack2(bq[2 * j + 1], bq[2 * j + 1]), z[1][q], fmul2(pack2(bq[2 * j], bq[2 * j]), z[0][q]));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float lo, hi;
        unpack2(z[i][q], lo, hi);
        const uint64_t other = pack2(__shfl_xor_sync(0xffffffffu, lo, 1), __shfl_xor_sync(0xffffffffu, hi, 1));
#pragma unroll
        for (int j = 0; j < 2; ++j) o[j][q] = ffma2(pack2(bq[4 + 2 * j + i], bq[4 + 2 * j + i]), other, o[j][q]);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) unpack2(o[j][q], y[8 * j + 2 * q], y[8 * j + 2 * q + 1]);
  } else if (kX == 2) {
    const int sm = (1 << p.ls) - 1, t = 32 >> p.ls, n0 = 16 * (lane & 1);
    const float* bb = p.b + static_cast<int64_t>(has ? vec >> 1 : 0) * t * t;
    float o[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float xk = __shfl_sync(0xffffffffu, y[k & 15], (lane & ~1) + (k >> 4));
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int n = n0 + j;
        const float pk = __fmul_rn(__ldg(bb + (k >> p.ls) * t + (n >> p.ls)),
                                   __ldg(p.a + ((k & sm) << p.ls) + (n & sm)));
        o[j] = __fmaf_rn(xk, pk, o[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = o[j];
  }
}

// (a NaN among the operands stays)
__device__ __forceinline__ float norm_min(float a, float b, float c) {
  float r;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float norm_max(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 1 / sqrt(sum / K + eps). A sum that fp32 does not hold would give 0, and so codes 0: it makes the row NaN.
__device__ __forceinline__ float norm_root(const NormParams& p, float sum) {
  const float r = __frsqrt_rn(__fmaf_rn(sum, p.inv_k, p.eps));
  return r > 0.0f ? r : NAN;
}

// Clip, scale and codes of the lane's channels, y = (h w) P without the root `inv`.
template <bool kFp8>
__device__ __forceinline__ void norm_quant(const NormParams& p, float (&y)[16], int vec, bool has, int64_t row,
                                           float inv, float r_lo, float r_hi) {
  const int lane = threadIdx.x & 31, blk = vec >> 1;
  float mn = y[0], mx = y[0];
#pragma unroll
  for (int j = 1; j < 15; j += 2) {
    mn = norm_min(mn, y[j], y[j + 1]);
    mx = norm_max(mx, y[j], y[j + 1]);
  }
  mn = norm_min(mn, y[15], __shfl_xor_sync(0xffffffffu, norm_min(mn, y[15], y[15]), 1));
  mx = norm_max(mx, y[15], __shfl_xor_sync(0xffffffffu, norm_max(mx, y[15], y[15]), 1));
  // (rounding is monotonic: the extremes of the rounded products are the rounded extremes)
  mn = __fmul_rn(mn, inv);
  mx = __fmul_rn(mx, inv);
  // a block with a value that is not finite: scale byte NaN, codes 0 (the clip to [0, 0])
  const bool bad = !(fabsf(mn) < INFINITY && fabsf(mx) < INFINITY);
  const float lo = bad ? 0.0f : __fmul_rn(r_lo, mn), hi = bad ? 0.0f : __fmul_rn(r_hi, mx);
  const float amax = fmaxf(fabsf(fminf(fmaxf(mn, lo), hi)), fabsf(fminf(fmaxf(mx, lo), hi)));
  constexpr int kEmax = kFp8 ? 8 : 2;
  const int ef = static_cast<int>(__float_as_uint(amax) >> 23);
  const int sbyte = has && ef > kEmax ? ef - kEmax : 0;
  const float down = __uint_as_float(static_cast<uint32_t>(254 - sbyte) << 23);
  const uint64_t inv2 = pack2(inv, inv), down2 = pack2(down, down);
#pragma unroll
  for (int j = 0; j < 16; j += 2) unpack2(fmul2(pack2(y[j], y[j + 1]), inv2), y[j], y[j + 1]);
  float v[16];
  // the addend 0 makes an exact zero +0
#pragma unroll
  for (int j = 0; j < 16; j += 2)
    unpack2(ffma2(pack2(fminf(fmaxf(y[j], lo), hi), fminf(fmaxf(y[j + 1], lo), hi)), down2, 0ull), v[j], v[j + 1]);
  if (has) {
    const int64_t e0 = row * p.K + 16 * vec;
    if (kFp8) {
      uint4 c;
      c.x = e4m3x4(v[0], v[1], v[2], v[3]);
      c.y = e4m3x4(v[4], v[5], v[6], v[7]);
      c.z = e4m3x4(v[8], v[9], v[10], v[11]);
      c.w = e4m3x4(v[12], v[13], v[14], v[15]);
      *reinterpret_cast<uint4*>(p.codes + e0) = c;
    } else {
      uint2 c;
      c.x = e2m1x8(reinterpret_cast<const float(&)[8]>(v[0]));
      c.y = e2m1x8(reinterpret_cast<const float(&)[8]>(v[8]));
      *reinterpret_cast<uint2*>(p.codes + e0 / 2) = c;
    }
    if (p.y_out) {
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(p.y_out + e0 + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
    }
  }
  // the scale bytes of blocks 4g .. 4g+3 are one word of the tiled layout; blocks past nb
  // come from lanes without channels and are the layout's zero padding
  uint32_t word = static_cast<uint32_t>(has && bad ? 255 : sbyte) << (8 * (blk & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  if (has && (lane & 7) == 0)
    *reinterpret_cast<uint32_t*>(p.scales + scale_offset(row, blk, p.nbp4)) = word;
}

// The CTA's sum: a warp's part into `red` (before a barrier) and the whole of it (after; the
// same order for every thread).
__device__ __forceinline__ void norm_sum_put(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
}
__device__ __forceinline__ float norm_sum_get(const float* red) {
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  float s = lane < nw ? red[lane] : 0.0f;
#pragma unroll
  for (int d = norm::kMaxThreads / 64; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return __shfl_sync(0xffffffffu, s, 0);
}

// h = x + r of 16 channels.
__device__ __forceinline__ void norm_add(const uint4 (&xv)[2], const uint4 (&rv)[2], float (&h)[16]) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float a[8], b[8];
    norm_unpack(xv[g], a);
    norm_unpack(rv[g], b);
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      unpack2(fadd2(pack2(a[j], a[j + 1]), pack2(b[j], b[j + 1])), h[8 * g + j], h[8 * g + j + 1]);
  }
}
__device__ __forceinline__ float norm_squares(const float (&h)[16]) {
  uint64_t s = 0ull;
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const uint64_t v = pack2(h[j], h[j + 1]);
    s = ffma2(v, v, s);
  }
  float a, b;
  unpack2(s, a, b);
  return a + b;
}
__device__ __forceinline__ void norm_store_res(uint16_t* dst, const float (&h)[16]) {
  uint4 o[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    o[g].x = norm_pack_bf16(h[8 * g], h[8 * g + 1]);
    o[g].y = norm_pack_bf16(h[8 * g + 2], h[8 * g + 3]);
    o[g].z = norm_pack_bf16(h[8 * g + 4], h[8 * g + 5]);
    o[g].w = norm_pack_bf16(h[8 * g + 6], h[8 * g + 7]);
    reinterpret_cast<uint4*>(dst)[g] = o[g];
  }
}
__device__ __forceinline__ void norm_weight(const uint4 (&wv)[2], float (&h)[16]) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float w[8];
    norm_unpack(wv[g], w);
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      unpack2(fmul2(pack2(h[8 * g + j], h[8 * g + j + 1]), pack2(w[j], w[j + 1])), h[8 * g + j], h[8 * g + j + 1]);
  }
}

// kV > 0: the row's kV vectors of 16 a thread stay in registers (kV * 16 * blockDim.x >= K).
// kV == 0: any K, the row is read once for the sum and once for the codes.
// kThreads: the most threads a CTA is launched with; up to 256, two CTAs share an SM (three, at
// 80 registers a thread, spill: 16384 x 4096 in 109 us when two took 100).
template <int kV, int kX, bool kFp8, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == 256 ? 2 : 1)
    bat_rmsnorm_quantize_kernel(const NormParams p) {
  __shared__ __align__(16) float sa[64];
  __shared__ float red[2][norm::kMaxThreads / 32];
  const int tid = threadIdx.x, nt = blockDim.x, nvec = p.K >> 4;
  grid_dependency_wait();  // launched with programmatic serialization
  allow_dependents();      // the GEMM after it waits for this kernel's end
  if (kX == 1 && tid < 64) sa[tid] = p.a[tid];
  constexpr int kN = kV > 0 ? kV : 1;
  float bq[kN][8], r_lo[kN], r_hi[kN];
  uint4 wv[kN][2];
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto load_block = [&](int i, int vec) {
    const bool has = vec < nvec;
    const int blk = has ? vec >> 1 : 0, h = vec & 1;
    if (kX == 1) {
      const float* b = p.b + 16 * static_cast<int64_t>(blk);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          bq[i][2 * j + k] = __ldg(b + 4 * (2 * h + k) + 2 * h + j);
          bq[i][4 + 2 * j + k] = __ldg(b + 4 * (2 * (1 - h) + k) + 2 * h + j);
        }
    }
    r_lo[i] = p.g_lo ? clip_ratio(__ldg(p.g_lo + blk)) : 1.0f;
    r_hi[i] = p.g_hi ? clip_ratio(__ldg(p.g_hi + blk)) : 1.0f;
#pragma unroll
    for (int g = 0; g < 2; ++g) wv[i][g] = has ? __ldg(reinterpret_cast<const uint4*>(p.w) + 2 * vec + g) : zero;
  };
  int turn = 0;
  if (kV > 0) {
    uint4 xv[kN][2], rv[kN][2];
    auto fetch = [&](int64_t row) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int vec = tid + i * nt;
        const bool has = vec < nvec && row < p.M;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          xv[i][g] = has ? *(reinterpret_cast<const uint4*>(p.x + row * p.K) + 2 * vec + g) : zero;
          rv[i][g] = has && p.res ? *(reinterpret_cast<const uint4*>(p.res + row * p.K) + 2 * vec + g) : zero;
        }
      }
    };
    int64_t row = blockIdx.x;
    fetch(row);
#pragma unroll
    for (int i = 0; i < kN; ++i) load_block(i, tid + i * nt);
    __syncthreads();
    for (; row < p.M; row += gridDim.x, turn ^= 1) {
      float y[kN][16], ss = 0.0f;
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        norm_add(xv[i], rv[i], y[i]);
        ss += norm_squares(y[i]);
        const int vec = tid + i * nt;
        if (p.res_out && vec < nvec) norm_store_res(p.res_out + row * p.K + 16 * vec, y[i]);
      }
      norm_sum_put(ss, red[turn]);
      fetch(row + gridDim.x);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        norm_weight(wv[i], y[i]);
        const int vec = tid + i * nt;
        norm_transform<kX>(p, y[i], vec, vec < nvec, sa, bq[i]);
      }
      __syncthreads();
      const float inv = norm_root(p, norm_sum_get(red[turn]));
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const int vec = tid + i * nt;
        norm_quant<kFp8>(p, y[i], vec, vec < nvec, row, inv, r_lo[i], r_hi[i]);
      }
    }
  } else {
    __syncthreads();
    const int iters = (nvec + nt - 1) / nt;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, turn ^= 1) {
      const uint4* xr = reinterpret_cast<const uint4*>(p.x + row * p.K);
      const uint4* rr = reinterpret_cast<const uint4*>(p.res + row * p.K);
      float ss = 0.0f;
      for (int vec = tid; vec < nvec; vec += nt) {
        float h[16];
        const uint4 xv[2] = {xr[2 * vec], xr[2 * vec + 1]};
        const uint4 rv[2] = {p.res ? rr[2 * vec] : zero, p.res ? rr[2 * vec + 1] : zero};
        norm_add(xv, rv, h);
        ss += norm_squares(h);
      }
      norm_sum_put(ss, red[turn]);
      __syncthreads();
      const float inv = norm_root(p, norm_sum_get(red[turn]));
      for (int it = 0; it < iters; ++it) {
        const int vec = tid + it * nt;
        const bool has = vec < nvec;
        load_block(0, vec);
        float y[16];
        const uint4 xv[2] = {has ? xr[2 * vec] : zero, has ? xr[2 * vec + 1] : zero};
        const uint4 rv[2] = {has && p.res ? rr[2 * vec] : zero, has && p.res ? rr[2 * vec + 1] : zero};
        norm_add(xv, rv, y);
        if (p.res_out && has) norm_store_res(p.res_out + row * p.K + 16 * vec, y);
        norm_weight(wv[0], y);
        norm_transform<kX>(p, y, vec, has, sa, bq[0]);
        norm_quant<kFp8>(p, y, vec, has, row, inv, r_lo[0], r_hi[0]);
      }
    }
  }
  // padding rows of the tiled scale layout
  const int64_t pad = (p.mpad - p.M) * p.nbp4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * nt + tid; i < pad; i += static_cast<int64_t>(gridDim.x) * nt)
    *reinterpret_cast<uint32_t*>(p.scales + scale_offset(p.M + i / p.nbp4, 4 * (i % p.nbp4), p.nbp4)) = 0u;
}

}  // namespace bat
