// Attention of chunks of new tokens over the paged MXFP8 / MXFP4 cache on the 5th-generation
// tensor cores (see bat_attn.cuh for the operator, the work split and the partial results).
//
// A unit is 256 query rows (two tiles of 128; one for heads wider than 128 channels) of one
// KV head: rows run over tokens and the group's heads, so grouped heads share every K and V
// tile. Its visible tokens come in chunks of 128. Warp roles:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one row a thread: S from TMEM, weights back into
//                   S's columns as the A operand of the second product; the output
//   warps 8-15      K and V: loads of codes a chunk ahead, expansion to f16 (K) and bf16 (V) in
//                   swizzled shared memory, 16 tokens of a chunk each
//   warp 16         issues the MMAs and owns TMEM
//   warps 17, 18    page lookups, cache rows and the scales' factors of 64 tokens each, up to
//                   three chunks ahead (done by the loader warps themselves these took a third of
//                   their time)
//   warp 19         q tiles by TMA, while the unit before is still in its last products
// q comes from bat_attn_q_rows_kernel: f16 rows (times P_q) in the order [KV head][token][head of the
// group], so that a tile's 128 rows lie together whatever the group's size.
// Per chunk and tile: S = q K^T (M 128, N 128, K = D, kind::f16 on f16) and
// o += P V (N = D, K = 128, kind::f16 on bf16, P from TMEM). The MMAs of one tile run while the
// other tile's warps are in their softmax. The maximum is lazy: the scores go against a
// reference that is within 2^40 below the row's maximum, which bf16 weights and fp32 sums hold without
// loss, so S is read once and o hardly ever rescaled.
// (Tried and not kept: S in halves of 64 tokens, the next chunk's first half computed before P V of
// this one: the softmax waits less, but a kind::f16 MMA takes about 120 cycles with N = 64 as with 128,
// and a 2048-token chunk over 16384 ran 801 us instead of 717. The weights' sum as the test of the
// reference instead of the maximum: 758 us. An issuing warp for each tile: 848 us, the tiles' MMAs then
// cut into each other. Without any softmax, stores or loads the MMAs and their hand-offs alone take 535.)
// (Those figures are from before the paths for keys far apart and for large scores, which cost 3 %.)
// What bounds it: latency along a chunk's chain (scores, softmax, P V, next scores), with the tensor pipe
// and the exponentials' unit each about 30 % busy. 2048 new tokens over 16384 (32 / 8 heads of 128, KV8):
// 729 us, 707 TFLOP/s, 0.43 of a cuBLAS bf16 product's rate; about 6000 cycles a chunk of 256 rows where
// MMAs and exponentials at their nominal rates would take 2048 each.
// Weights are bf16 (8 bits) because V is: the two operands of an MMA have one type, and f16 does not hold
// V's scales. Each is rounded to nearest, so that their errors average out; the sum keeps fp32.
//
// A NaN in V must not reach rows that do not see its token, but 0 times NaN in the MMA would
// carry it there: the loader stores 0 in its place and notes (token, block);
// the rows that see the token look up its channels and put the NaN back at the end.
#pragma once

#include "bat_attn.cuh"

namespace bat {

namespace attn_tile {
constexpr int kPanelBytes = 128 * 128;  // 128 rows of 64 16-bit channels, 128-byte swizzle
constexpr int kLoadWarps = 8;
constexpr int kThreads = 640;  // the register split goes by four warps
constexpr int kRegsSoftmax = 112, kRegsLoad = 104, kRegsOther = 48;
static_assert(2 * kRegsSoftmax + 2 * kRegsLoad + kRegsOther <= 5 * 96, "the split stays within the launch's registers");
constexpr int kInfo = 8;                // chunks whose notes are kept
// A note is overwritten eight chunks on, by a warp that is at most kSlots chunks ahead of the loaders,
// and they at most kStages / 2 chunks ahead of the products whose softmax read it. (A unit's last note is read
// after its last product: by a tile that the next unit has too before its first weights there, by tile 1 where the
// next unit lacks it before its warps' arrival there, without which that unit gets no q.)

template <int kDP>
struct Cfg {
  static constexpr int kTiles = kDP <= 128 ? 2 : 1;   // tiles of 128 rows a unit
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kPanels = kDP / 64;
  static constexpr int kStageBytes = kPanels * kPanelBytes;
  static constexpr int kStages = kDP == 64 ? 8 : (kDP == 128 ? 4 : 2);
  static constexpr int kSlots = kDP == 256 ? 2 : 3;  // chunks whose rows and factors are kept
  static_assert(kSlots + kStages / 2 <= kInfo - 1, "notes outlive their readers");
  static constexpr int kQBytes = kTiles * kPanels * kPanelBytes;
  static constexpr int kSmem = 1024 + kQBytes + kStages * kStageBytes;  // dynamic, 1024 for alignment
};
}  // namespace attn_tile

// What the loader warps note about a chunk for the softmax warps.
struct AttnNote {
  float kfac[8];      // 2^(largest K scale of the warp's 16 tokens), 1 where they are apart
  int any[8];         // of its tokens: kNoteSome some are hidden (bad page) or hold a NaN in V, kNoteApart
                      // their K scales are too far apart for one factor, kNoteWide a token's own are
  uint32_t tok[128];  // bit 31: hidden; bit 30: wide; bits 16-23: scale byte of the token's K column (127:
                      // none); bit b: NaN in V's block b
};
constexpr int kNoteSome = 1, kNoteApart = 2, kNoteWide = 4;
// A chunk's cache rows (0 for none) and factors (16-bit pairs) for the loader warps.
template <int kNB>
struct AttnIndex {
  uint32_t row[128];
  uint32_t fac[2][128][kNB];  // K, V
};
__device__ __forceinline__ int attn_note_any(const AttnNote& n) {
  const volatile int4* a = reinterpret_cast<const volatile int4*>(n.any);
  return a[0].x | a[0].y | a[0].z | a[0].w | a[1].x | a[1].y | a[1].z | a[1].w;
}
// idesc of kind::f16, fp32 accumulation, A K-major; kBf16: both operands bf16, else f16;
// kMnB: B is MN-major.
template <bool kBf16, bool kMnB>
__device__ __forceinline__ constexpr uint32_t attn_idesc(int n) {
  return 1u << 4 | (kBf16 ? 1u << 7 | 1u << 10 : 0u) | (kMnB ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | 8u << 24;
}
__device__ __forceinline__ void attn_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void attn_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// One lane of a converged warp. (An MMA issued under a plain lane test takes about 400 cycles of
// its thread; the compiler has to assume that several lanes get there.)
__device__ __forceinline__ bool attn_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// TMEM loads in flight: the wait names the registers, so that nothing uses them before it.
__device__ __forceinline__ void attn_tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// 16 columns, complete on return (the rare paths).
__device__ __forceinline__ void attn_tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// One column.
__device__ __forceinline__ void attn_tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}

// The scores of a chunk's tokens whose K scales are too far apart for one factor (rare; the whole warp calls it): the
// columns that were taken by the token's own scale, times that scale, a power of two: exact; and those of tokens
// whose own blocks are too far apart, a block at a time in fp32 on the CUDA cores. qrow: the lane's row among the
// prepared q rows, or -1. (Out of line, for the softmax loop's sake.)
template <bool kFp8>
__device__ __noinline__ void attn_far_keys(const AttnParams& p, const AttnNote& note, uint32_t taddr, int64_t qrow, int b,
                                           int h, AttnSpan span, int i0) {
#pragma unroll 1
  for (int k = 0; k < 128; k += 16) {
    if (!(note.any[k >> 4] & kNoteApart)) continue;
    uint32_t s[16];
    attn_tmem_ld16(taddr + k, s);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float x = __uint_as_float(s[j]), y = x * attn_scale_value(note.tok[k + j] >> 16 & 255u);
      s[j] = __float_as_uint(fabsf(y) == INFINITY && fabsf(x) != INFINITY ? copysignf(3e38f, x) : y);
    }
    tmem_st_32x32b_x16(taddr + k, s);
  }
  tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < 128; ++c) {
    if ((note.tok[c] >> 30) != 1u) continue;  // wide and not hidden
    float s = 0.0f;
    if (qrow >= 0) {
      const int64_t row = attn_cache_row(p, p.table + static_cast<int64_t>(b) * p.max_pages, span.token(i0 + c), h);
      const uint8_t* codes = p.k_codes + row * (kFp8 ? p.D : p.D / 2);
      const uint4* q = reinterpret_cast<const uint4*>(p.qt + qrow * p.D);
#pragma unroll 1
      for (int blk = 0; blk < p.nb; ++blk) {
        float d = 0.0f;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // 8 channels
          uint32_t kk[4];
          if (kFp8) {
            const uint2 w = *reinterpret_cast<const uint2*>(codes + 32 * blk + 8 * i);
            attn_e4m3_f16(w.x, kk[0], kk[1]);
            attn_e4m3_f16(w.y, kk[2], kk[3]);
          } else {
            attn_e2m1_f16(*reinterpret_cast<const uint32_t*>(codes + 16 * blk + 4 * i), kk);
          }
          const uint4 w = q[4 * blk + i];
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x0, x1, k0, k1;
            attn_f16_floats(x[j], x0, x1);
            attn_f16_floats(kk[j], k0, k1);
            d = __fmaf_rn(x0, k0, d);
            d = __fmaf_rn(x1, k1, d);
          }
        }
        s = __fmaf_rn(d, attn_scale_value(p.k_scales[row * p.nb + blk]), s);
      }
    }
    __syncwarp();
    attn_tmem_st1(taddr + c, s);
  }
  tmem_wait_st();
}

// Channel order that the expansion of V leaves (see attn_e4m3_bits, attn_e2m1_bits): position
// i of an 8-channel group holds channel attn_v_order(i).
template <bool kFp8>
__host__ __device__ constexpr int attn_v_order(int i) {
  return kFp8 ? (i & ~3) | ((i & 1) << 1) | ((i >> 1) & 1) : (i & ~7) | ((i >> 1) & 3) | ((i & 1) << 2);
}

// Rows of q (P_q) in f16, times the power of two that brings the row's largest channel to
// [2^14, 2^15), and the factor that takes it back. kL lanes a row, 8 channels each; a warp has
// four steps' rows on their way at once (bound: HBM, 4 bytes an element).
struct AttnQRowsParams {
  const uint16_t* q;
  int64_t q_stride;
  const float* a;  // factors of P_q, or null
  const float* b;
  uint16_t* out;   // f16 [Hkv][T][G][D]
  float* fac;      // [Hkv][T][G]
  int64_t T;
  int Hq, G, D, nb, ls;
  float sign, scale_log2;
};
template <int kL>
__global__ void __launch_bounds__(256) bat_attn_q_rows_kernel(const AttnQRowsParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kRows = 32 / kL, kAhead = 4;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int v = lane % kL, sub = lane / kL;
  float* sx = smem + (warp * kRows + sub) * (8 * kL + 4);  // the row in fp32
  // (in this order: the tile kernel reads the cache and the lengths without a wait of its own, so it
  // may not start before the kernels ahead of this one are complete)
  grid_dependency_wait();
  allow_dependents();
  AttnFactors f{nullptr, nullptr, 3};
  if (p.a) {
    f = attn_stage_factors(smem + 8 * kRows * (8 * kL + 4), p.a, p.b, p.nb, p.ls, threadIdx.x, blockDim.x);
    __syncthreads();
  }
  const bool in = 8 * v < p.D;
  const uint32_t hq_n = p.Hq;
  const uint32_t rows = static_cast<uint32_t>(p.T) * hq_n;  // at most 2^30
  const uint32_t step = gridDim.x * 8 * kRows;
  for (uint32_t r0 = (blockIdx.x * 8 + warp) * kRows; r0 < rows; r0 += kAhead * step) {
    uint4 w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t row = r0 + k * step + sub;
      const uint32_t t = row / hq_n;
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows && in)
        w[k] = __ldg(reinterpret_cast<const uint4*>(p.q + t * p.q_stride + static_cast<int64_t>(row - t * hq_n) * p.D) + v);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint32_t row = r0 + k * step + sub;
      if (r0 + k * step >= rows) break;
      float x[8] = {bf16lo(w[k].x), bf16hi(w[k].x), bf16lo(w[k].y), bf16hi(w[k].y),
                    bf16lo(w[k].z), bf16hi(w[k].z), bf16lo(w[k].w), bf16hi(w[k].w)};
      if (p.a) {
        *reinterpret_cast<float4*>(sx + 8 * v) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(sx + 8 * v + 4) = make_float4(x[4], x[5], x[6], x[7]);
        __syncwarp();
        // lane v takes outputs v % 8 and that + 8, + 16, + 24 of blocks v / 8 and kL / 8 more
        constexpr int kPer = kL >= 8 ? 2 : 4;  // 2 kL such items a row
        float y[kPer][4];
#pragma unroll
        for (int g = 0; g < kPer; ++g) {
          const int item = v + g * kL;
          if (item < 8 * p.nb) attn_block_apply(f, item >> 3, sx + 32 * (item >> 3), item & 7, y[g]);
        }
        __syncwarp();
#pragma unroll
        for (int g = 0; g < kPer; ++g) {
          const int item = v + g * kL;
          if (item < 8 * p.nb)
#pragma unroll
            for (int j = 0; j < 4; ++j) sx[32 * (item >> 3) + 8 * j + (item & 7)] = y[g][j];
        }
        __syncwarp();
        const float4 a = *reinterpret_cast<const float4*>(sx + 8 * v), b = *reinterpret_cast<const float4*>(sx + 8 * v + 4);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        __syncwarp();
      }
      float mx = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) mx = in ? fmaxf(mx, fabsf(x[j])) : 0.0f;
#pragma unroll
      for (int d = kL / 2; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      float down;
      const float up = attn_row_up(mx, down) * p.sign;
      if (row >= rows) continue;
      const uint32_t t = row / hq_n, hq = row - t * hq_n, h = hq / p.G;
      const int64_t dst = (h * p.T + t) * p.G + (hq - h * p.G);
      if (in)
        *(reinterpret_cast<uint4*>(p.out + dst * p.D) + v) =
            make_uint4(attn_pack_f16(x[0] * up, x[1] * up), attn_pack_f16(x[2] * up, x[3] * up),
                       attn_pack_f16(x[4] * up, x[5] * up), attn_pack_f16(x[6] * up, x[7] * up));
      if (v == 0) p.fac[dst] = down * p.scale_log2;
    }
  }
}

// A run of chunks, unit after unit.
template <int kTile>
struct AttnRun {
  AttnPlace pl;
  AttnSeq seq;
  AttnSpan span;
  int nv;
  int left;  // chunks, this one among them (a CTA's run is below 2^31)
  __device__ __forceinline__ void enter(const AttnParams& p) {
    span = attn_tile_span<kTile>(p, seq, pl.tile);
    nv = span.count();
  }
  __device__ __forceinline__ void start(const AttnParams& p, const AttnPlace& place, int64_t n) {
    pl = place;
    left = static_cast<int>(n);
    if (left > 0) {
      seq = attn_seq(p, pl.b);
      enter(p);
    }
  }
  __device__ __forceinline__ void next_chunk(const AttnParams& p) {
    if (--left <= 0) return;
    if (++pl.chunk < pl.chunks) return;
    attn_next_unit<kTile>(p, pl, seq);
    enter(p);
  }
  // skips to the next unit after n chunks of this one
  __device__ __forceinline__ void next_unit(const AttnParams& p, int n) {
    left -= n;
    if (left <= 0) return;
    attn_next_unit<kTile>(p, pl, seq);
    enter(p);
  }
  __device__ __forceinline__ int chunks_here() const {
    return min(pl.chunks - pl.chunk, left);
  }
  // tiles of 128 rows that hold rows
  __device__ __forceinline__ int tiles(const AttnParams& p) const {
    return static_cast<int64_t>(seq.n) * p.G - static_cast<int64_t>(pl.tile) * kTile > 128 ? kTile / 128 : 1;
  }
};

template <bool kFp8, int kDP>
__global__ void __launch_bounds__(attn_tile::kThreads, 1) bat_attn_tile_kernel(
    const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap qmap) {
  using C = attn_tile::Cfg<kDP>;
  constexpr int kTile = C::kRows, kStages = C::kStages;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ __align__(16) AttnNote notes[attn_tile::kInfo];
  __shared__ AttnIndex<kDP / 32> s_index[C::kSlots];
  __shared__ uint32_t s_nan[C::kRows][kDP / 32];  // written only where a NaN was seen
  __shared__ __align__(16) float s_oa[64];
  __shared__ __align__(16) float s_ob[kDP / 32 * 16];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 2 * 5 + 2 * C::kSlots + 2];
  __shared__ uint32_t s_tmem;
  __shared__ AttnPlace s_place;
  __shared__ int64_t s_run;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t q_base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t st_base = q_base + C::kQBytes;
  const uint32_t bars = smem_u32(s_bar);
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto q_full = [&](int t) { return bars + 8 * (2 * kStages + t); };
  auto s_full = [&](int t) { return bars + 8 * (2 * kStages + 2 + t); };
  auto p_full = [&](int t) { return bars + 8 * (2 * kStages + 4 + t); };
  auto o_full = [&](int t) { return bars + 8 * (2 * kStages + 6 + t); };
  auto q_free = [&](int t) { return bars + 8 * (2 * kStages + 8 + t); };
  auto i_full = [&](int s) { return bars + 8 * (2 * kStages + 10 + s); };
  auto i_empty = [&](int s) { return bars + 8 * (2 * kStages + 10 + C::kSlots + s); };
  const uint32_t drain = bars + 8 * (2 * kStages + 10 + 2 * C::kSlots);
  // (the barrier behind it: tile 1's warps have left a unit for one that has no tile 1)

  allow_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), attn_tile::kLoadWarps);
      mbar_init(empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_free(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);
      mbar_init(o_full(t), 1);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(i_full(i), 2);
      mbar_init(i_empty(i), attn_tile::kLoadWarps);
    }
    mbar_init(drain, 1);
    mbar_init(drain + 8, 4);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  if (warp == 15) {
    int64_t n;
    AttnSeq seq0;
    const AttnMark mk = attn_mark<kTile>(p, blockIdx.x, lane, n, seq0);
    if (lane == 0) {
      s_place = mk.place;
      s_run = n;
      p.marks[blockIdx.x] = mk;
    }
  }
  if (p.oa != nullptr && p.ols == 3 && warp == 14) {
    s_oa[lane] = p.oa[lane];
    s_oa[lane + 32] = p.oa[lane + 32];
    for (int i = lane; i < 16 * p.nb; i += 32) s_ob[i] = p.ob[i];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // columns: S of tile 0, 1 (the weights in the first half of them), o of tile 0, 1
  auto s_col = [&](int t) { return tmem + 128u * t; };
  auto o_col = [&](int t) { return tmem + 128u * C::kTiles + static_cast<uint32_t>(kDP) * t; };
  AttnRun<kTile> run;
  run.start(p, s_place, s_run);

  if (warp < 8) {
    // ================================================================ softmax
    setmaxnreg_inc<attn_tile::kRegsSoftmax>();
    const int t = warp >> 2;
    const int rr = threadIdx.x & 127;        // row within the tile = TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, bits 16 up
    uint32_t n_s = 0;  // chunks of this tile so far (phases of s_full, o_full)
    uint32_t n_c = 0;  // chunks of the run so far (the notes' ring)
    uint32_t n_left = 0;  // n_s at the last unit without this tile
    bool ok = t < C::kTiles;
    grid_dependency_wait();  // the q rows' factors
    for (int seg = 0; ok && run.left > 0; ++seg) {
      const int n = run.chunks_here();
      if (t >= run.tiles(p)) {
        if (n_s != n_left) {
          if (lane == 0) mbar_arrive(drain + 8);
          n_left = n_s;
        }
        run.next_unit(p, n);
        n_c += n;
        continue;
      }
      const int base = run.seq.len - run.seq.n;
      int pos;
      float cs;
      {
        const int64_t row = static_cast<int64_t>(run.pl.tile) * kTile + 128 * t + rr;
        const int64_t rt = row / p.G;
        const bool valid = rt < run.seq.n;
        pos = valid ? base + static_cast<int>(rt) : -1;
        cs = valid ? p.qt_fac[(run.pl.hu * p.T + run.seq.t0) * p.G + row] : 0.0f;
      }
      // the row's visible columns, as indices among the unit's visible tokens: [v_lo, v_hi) and
      // [0, v_sink)
      const AttnSpan sp = run.span;
      int v_hi = pos >= sp.lo ? sp.ns + (pos - sp.lo + 1) : min(sp.ns, pos + 1);
      v_hi = min(v_hi, run.nv);
      int v_lo = 0, v_sink = 0;
      if (p.window > 0) {
        const int a = pos - p.window + 1;
        v_lo = a > sp.lo ? sp.ns + (a - sp.lo) : sp.ns;
        v_sink = p.sinks <= sp.lo ? sp.ns : min(p.sinks, run.nv);
        if (sp.lo == 0 && a <= 0) v_lo = 0;
      }
      // columns below all_lo or in [all_lo, all_hi) are seen by every row of the unit
      const int64_t unit_rows0 = static_cast<int64_t>(run.pl.tile) * kTile;
      const int pos_f = base + static_cast<int>(unit_rows0 / p.G);
      const int64_t last_t = (unit_rows0 + kTile - 1) / p.G;
      const int pos_l = base + static_cast<int>(last_t < run.seq.n - 1 ? last_t : run.seq.n - 1);
      const int all_hi = min(run.nv, pos_f >= sp.lo ? sp.ns + (pos_f - sp.lo + 1) : min(sp.ns, pos_f + 1));
      const int all_lo = p.window > 0 && pos_l - p.window + 1 > sp.lo ? sp.ns + (pos_l - p.window + 1 - sp.lo) : sp.ns;

      float m = -INFINITY, l0 = 0.0f, l1 = 0.0f;
      float thr = -INFINITY;  // a score above it takes the way round: a new reference, or one of a large size
      bool nan_seen = false;  // the row saw a NaN in V; its channels are in s_nan
      auto see_nan = [&](uint32_t c0, int chunk) {
        const AttnNote& nt = notes[c0 % attn_tile::kInfo];
        for (int c = 0; c < 128; ++c) {
          const uint32_t f = nt.tok[c];
          const int idx = chunk * 128 + c;
          if ((f & 0xFFFFu) == 0u || (f >> 31) || idx >= v_hi || (idx < v_lo && idx >= v_sink)) continue;
          if (!nan_seen) {
            for (int b = 0; b < kDP / 32; ++b) s_nan[128 * t + rr][b] = 0u;
            nan_seen = true;
          }
          // which channels: from the cache again
          const int64_t vrow = attn_cache_row(p, p.table + static_cast<int64_t>(run.pl.b) * p.max_pages,
                                              sp.token(idx), run.pl.hu);
          for (int b = 0; b < p.nb; ++b) {
            if (!(f >> b & 1u)) continue;
            uint32_t ch = 0u;
            if ((attn_scale_pair<kFp8>(p.v_scales[vrow * p.nb + b]) & 0x7FFFu) == 0x7FFFu) {
              ch = ~0u;
            } else if (kFp8) {
              for (int d = 0; d < 32; ++d)
                ch |= static_cast<uint32_t>((p.v_codes[vrow * p.D + 32 * b + d] & 0x7F) == 0x7F) << d;
            }
            s_nan[128 * t + rr][b] |= ch;
          }
        }
      };
      for (int i = 0; i < n; ++i, ++n_s, ++n_c) {
        const int chunk = run.pl.chunk + i;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(t), n_s & 1u, kErrWaitFull));
        if (!ok) break;
        tc_fence_after();
        // V of the chunk before is complete: its notes
        if (i > 0 && (attn_note_any(notes[(n_c - 1) % attn_tile::kInfo]) & kNoteSome)) {
          see_nan(n_c - 1, chunk - 1);
          __syncwarp();
        }
        const AttnNote& note = notes[n_c % attn_tile::kInfo];
        // factor of 16 columns (their tokens share a loader warp)
        auto cc = [&](int g) { return fmaxf(cs * note.kfac[g], 1e-37f); };
        const int i0 = chunk * 128;
        // masked columns go to TMEM as -inf, so that the pass below needs no test
        const bool whole = (i0 >= all_lo || i0 + 128 <= sp.ns) && i0 + 128 <= all_hi;
        // (one lane's view for the warp: the loaders may be adding to the note)
        const int some = __shfl_sync(0xffffffffu, attn_note_any(note), 0);
        if (!whole || some) {
          if (some & (kNoteApart | kNoteWide)) {
            const int64_t row = static_cast<int64_t>(run.pl.tile) * kTile + 128 * t + rr;
            const int64_t qrow = (run.pl.hu * p.T + run.seq.t0) * p.G + row;
            attn_far_keys<kFp8>(p, note, s_col(t) + lane_base, row < static_cast<int64_t>(run.seq.n) * p.G ? qrow : -1,
                                run.pl.b, run.pl.hu, sp, i0);
          }
          const int c_hi = v_hi - i0, c_lo = v_lo - i0, c_sink = v_sink - i0;
#pragma unroll 1
          for (int k = 0; k < 128; k += 32) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(s_col(t) + lane_base + k, s);
            attn_tmem_wait(s);
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int c = k + j;
              if (!(c < c_hi && (c >= c_lo || c < c_sink))) s[j] = 0xFF800000u;
              if (some && (note.tok[c] >> 31)) s[j] = 0xFF800000u;
            }
            tmem_st_32x32b_x16(s_col(t) + lane_base + k, reinterpret_cast<const uint32_t(&)[16]>(s[0]));
            tmem_st_32x32b_x16(s_col(t) + lane_base + k + 16, reinterpret_cast<const uint32_t(&)[16]>(s[16]));
          }
          tmem_wait_st();
        }
        // 32 columns at a time, once: scores against the reference m, weights (up to 2^40) into
        // S's columns 16 k .. that are already read. (Not unrolled: the instruction caches hold the
        // roles' loops then.)
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t x[32];
          tmem_ld_32x32b_x32(s_col(t) + lane_base + 32 * k, x);
          float c0 = cc(2 * k), c1 = cc(2 * k + 1);
          attn_tmem_wait(x);
          float mx[2] = {__uint_as_float(x[0]), __uint_as_float(x[16])};
#pragma unroll
          for (int g = 0; g < 2; ++g) {
#pragma unroll
            for (int j = 16 * g + 1; j < 16 * g + 15; j += 2)
              asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[g]) : "f"(__uint_as_float(x[j])), "f"(__uint_as_float(x[j + 1])));
            mx[g] = fmaxf(mx[g], __uint_as_float(x[16 * g + 15]));
          }
          const float top = fmaxf(mx[0] * c0, mx[1] * c1);
          if (__builtin_expect(__any_sync(0xffffffffu, top > thr), 0)) {
            const bool grow = m == -INFINITY ? top > -INFINITY : top > m + 40.0f;
            if (__any_sync(0xffffffffu, grow)) {
              // a new reference, a whole number, so that what is already there is scaled exactly
              const float mn = grow ? ceilf(top) : m;
              const float2 al = m == -INFINITY ? make_float2(1.0f, 1.0f) : attn_exp2_two(m - mn);
              m = mn;
              l0 *= al.x * al.y;
              l1 *= al.x * al.y;
              if (i > 0) {
                // o of the chunks before: all their MMAs are done
                ok = __all_sync(0xffffffffu, mbar_wait(o_full(t), (n_s - 1) & 1u, kErrWaitTmemFull)) && ok;
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < p.D; d += 16) {
                  uint32_t o[16];
                  attn_tmem_ld16(o_col(t) + lane_base + d, o);
#pragma unroll
                  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al.x * al.y);
                  tmem_st_32x32b_x16(o_col(t) + lane_base + d, o);
                }
              }
              tmem_wait_st();
#pragma unroll 1
              for (int d = 0; d < 16 * k; d += 16) {
                uint32_t w[16];
                attn_tmem_ld16(s_col(t) + lane_base + d, w);
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j] = attn_mul_bf16x2(attn_mul_bf16x2(w[j], attn_pack(al.x, al.x)), attn_pack(al.y, al.y));
                tmem_st_32x32b_x16(s_col(t) + lane_base + d, w);
              }
            }
            // From 2^24 on: below, score times factor less m is not rounded between, and what the rounding of m
            // left of the largest would no longer be small.
            const bool large = fabsf(m) >= 0x1p24f && m != -INFINITY;
            thr = m == -INFINITY || large ? -INFINITY : m + 40.0f;
            if (large) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * (j < 16 ? c0 : c1));
              c0 = c1 = 1.0f;
            }
            __syncwarp();
          }
          const float ms = m == -INFINITY ? 0.0f : m;
          const uint64_t m2 = pack2(-ms, -ms);
          uint64_t sum2 = pack2(l0, l1);
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a, b;
            const float cg = j < 8 ? c0 : c1;
            unpack2(ffma2(pack2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), pack2(cg, cg), m2), a, b);
            a = attn_exp2(a);
            b = attn_exp2(b);
            sum2 = fadd2(sum2, pack2(a, b));
            w[j] = attn_pack(a, b);  // bf16: off by half a step 2^-8 of each weight, unbiased
          }
          unpack2(sum2, l0, l1);
          tmem_st_32x32b_x16(s_col(t) + lane_base + 16 * k, w);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t));
      }
      if (!ok) break;
      // ---- the unit's end
      ok = __all_sync(0xffffffffu, mbar_wait(o_full(t), (n_s - 1) & 1u, kErrWaitTmemFull));
      if (!ok) break;
      tc_fence_after();
      if (attn_note_any(notes[(n_c - 1) % attn_tile::kInfo]) & kNoteSome) see_nan(n_c - 1, run.pl.chunk + n - 1);
      const int64_t row = static_cast<int64_t>(run.pl.tile) * kTile + 128 * t + rr;
      const int64_t rt = row / p.G;
      const bool valid = rt < run.seq.n;
      const int64_t tok = run.seq.t0 + rt;
      const int head = run.pl.hu * p.G + static_cast<int>(row - rt * p.G);
      const float l = l0 + l1;
      const bool part = !(run.pl.chunk == 0 && n == run.pl.chunks);
      const int64_t prow = (2 * static_cast<int64_t>(blockIdx.x) + (seg == 0 ? 0 : 1)) * kTile + 128 * t + rr;
      const float inv = l > 0.0f ? attn::kUp / l : (l == 0.0f ? 0.0f : l);
      for (int b = 0; b < p.nb; ++b) {
        uint32_t o[32];
        __syncwarp();  // (rows that are not there or saw a NaN took another way)
        tmem_ld_32x32b_x32(o_col(t) + lane_base + 32 * b, o);
        tmem_wait_ld();
        float v[32];
        const float f = part ? attn::kUp * 0x1p-40f : inv;
        // (a row that saw nothing: its sums are 0, whatever a NaN in q may have left in them)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[attn_v_order<kFp8>(j)] = l == 0.0f ? 0.0f : __uint_as_float(o[j]) * f;
        if (nan_seen) {
          const uint32_t ch = s_nan[128 * t + rr][b];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (ch >> j & 1u) v[j] = NAN;
        }
        if (!valid) continue;
        if (part) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + prow * p.D + 32 * b);
#pragma unroll
          for (int j = 0; j < 8; ++j) dst[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          continue;
        }
        if (p.oa != nullptr) {
          if (p.ols == 3) {
            // y = B^T (X_r A), X_r the block's 4 x 8 view
            uint64_t y[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q) y[i][q] = 0ull;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint64_t z[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const ulonglong2 a0 = *reinterpret_cast<const ulonglong2*>(s_oa + 8 * k);
                const ulonglong2 a1 = *reinterpret_cast<const ulonglong2*>(s_oa + 8 * k + 4);
                const uint64_t x = pack2(v[8 * i + k], v[8 * i + k]);
                z[0] = ffma2(x, a0.x, z[0]);
                z[1] = ffma2(x, a0.y, z[1]);
                z[2] = ffma2(x, a1.x, z[2]);
                z[3] = ffma2(x, a1.y, z[3]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float bj = s_ob[16 * b + 4 * i + j];
                const uint64_t b2 = pack2(bj, bj);
#pragma unroll
                for (int q = 0; q < 4; ++q) y[j][q] = ffma2(b2, z[q], y[j][q]);
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) unpack2(y[j][q], v[8 * j + 2 * q], v[8 * j + 2 * q + 1]);
          } else {
            // other splits: coefficients as they come (slow; the same sums)
            const int sm = (1 << p.ols) - 1, tt = 32 >> p.ols;
            const float* bb = p.ob + static_cast<int64_t>(b) * tt * tt;
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (tok * p.Hq + head) * p.D + 32 * b);
#pragma unroll 1
            for (int j = 0; j < 32; j += 2) {
              float y[2] = {0.0f, 0.0f};
#pragma unroll
              for (int k = 0; k < 32; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  y[e] = __fmaf_rn(v[k], __fmul_rn(__ldg(bb + (k >> p.ols) * tt + ((j + e) >> p.ols)),
                                                   __ldg(p.oa + ((k & sm) << p.ols) + ((j + e) & sm))), y[e]);
              dst[j >> 1] = attn_pack(y[0], y[1]);
            }
            continue;
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(p.out + (tok * p.Hq + head) * p.D + 32 * b);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dst[j] = make_uint4(attn_pack(v[8 * j], v[8 * j + 1]), attn_pack(v[8 * j + 2], v[8 * j + 3]),
                              attn_pack(v[8 * j + 4], v[8 * j + 5]), attn_pack(v[8 * j + 6], v[8 * j + 7]));
      }
      if (valid) {
        if (part) {
          // (against the reference's upper bound: parts then stay as small as the output)
          p.part_ml[2 * prow] = m + 40.0f;
          p.part_ml[2 * prow + 1] = l * 0x1p-40f;
        } else if (p.lse) {
          p.lse[tok * p.Hq + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      __syncwarp();
      run.next_unit(p, n);
    }
  } else if (warp < 16) {
    // ================================================================ K and V
    setmaxnreg_inc<attn_tile::kRegsLoad>();
    constexpr int kLpt = kFp8 ? kDP / 16 : kDP / 32;     // lanes a token: 16 bytes of codes each
    constexpr int kTpi = 32 / kLpt;                      // tokens a load instruction
    constexpr int kTasks = 16 / kTpi;                    // 16-byte pieces a thread (a warp has 16 tokens)
    static_assert(kTasks >= 1 && 16 % kTpi == 0, "a warp's tokens are whole load instructions");
    constexpr int kBatch = kTasks < 4 ? kTasks : 4;
    constexpr int kNB = kTasks / kBatch;                 // batches a tile: 1 or 2
    const int lw = warp - 8;
    const int row_bytes = kFp8 ? p.D : p.D / 2;
    // the lanes of a quarter-warp take the pieces of one panel of neighbouring tokens, so that
    // their 16-byte stores fall on different banks of the swizzled rows
    constexpr int kPp = kFp8 ? 4 : 2;  // pieces a panel
    const int piece = ((lane >> 3) % C::kPanels) * kPp + lane % kPp;
    const int sub = (lane >> 3) / C::kPanels * (8 / kPp) + lane % 8 / kPp;
    const bool has = piece * 16 < row_bytes;
    const int pblk = has ? (kFp8 ? piece >> 1 : piece) : 0;  // its 32-channel block
    bool ok = true;
    uint4 buf[2][kBatch];
    // (tokens that are not there read row 0, lanes past the head's channels its first piece: K's
    // scores of such tokens are masked, V's weights are 0, the pieces are not stored)
    const uint32_t piece_off = has ? 16u * piece : 0u;
    auto load_batch = [&](const AttnIndex<kDP / 32>& ix, const uint8_t* codes, int b, uint4 (&dst)[kBatch]) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const uint32_t row = ix.row[16 * lw + (b * kBatch + k) * kTpi + sub];
        dst[k] = __ldg(reinterpret_cast<const uint4*>(codes + piece_off + static_cast<uint64_t>(row) * static_cast<uint32_t>(row_bytes)));
      }
    };
    constexpr int kX = kFp8 ? 8 : 16;  // words a piece expands to
    // shared-memory place of this lane's piece of its token k of a batch: token 16 lw + k kTpi + sub,
    // 8-channel groups kX / 4 piece + u; k kTpi and sub share no bits, so the swizzle's exclusive or
    // splits
    const uint32_t put_row = (16 * lw + sub) * 128 + (kX / 4 * piece >> 3) * attn_tile::kPanelBytes;
    const uint32_t put_unit = ((kX / 4 * piece & 7) ^ (sub & 7)) << 4;
    auto put = [&](uint32_t stage, int k, const uint32_t (&x)[kX]) {
      if (!has) return;
#pragma unroll
      for (int u = 0; u < kX / 4; ++u) {
        const uint32_t at = stage + put_row + k * kTpi * 128 + (put_unit ^ (((k * kTpi & 7) ^ u) << 4));
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[4 * u]), "r"(x[4 * u + 1]),
                     "r"(x[4 * u + 2]), "r"(x[4 * u + 3])
                     : "memory");
      }
    };
    const int total = run.left;
    auto index_wait = [&](uint32_t c) {
      ok = __all_sync(0xffffffffu, mbar_wait(i_full(c % C::kSlots), (c / C::kSlots) & 1u, kErrWaitFull)) && ok;
    };
    if (total > 0) {
      index_wait(0);
      if (ok) {
        load_batch(s_index[0], p.k_codes, 0, buf[0]);
        if (kNB == 2)
          load_batch(s_index[0], p.k_codes, kNB - 1, buf[1]);
        else
          load_batch(s_index[0], p.v_codes, 0, buf[1]);
      }
    }
    uint32_t el = 0;  // tiles put so far (K and V in turn)
    for (uint32_t c = 0; ok && static_cast<int>(c) < total; ++c) {
      const AttnIndex<kDP / 32>& ix = s_index[c % C::kSlots];
      const AttnIndex<kDP / 32>& ix_next = s_index[(c + 1) % C::kSlots];
      const bool more = static_cast<int>(c) + 1 < total;
      AttnNote& note = notes[c % attn_tile::kInfo];
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++el) {
        const uint32_t sidx = el % kStages;
        const uint32_t stage = st_base + sidx * C::kStageBytes;
        ok = __all_sync(0xffffffffu, mbar_wait(empty(sidx), ((el / kStages) & 1u) ^ 1u, kErrWaitEmpty)) && ok;
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
          constexpr int kSeq = 2 * kNB;
          const int e = kv * kNB + b;
            uint4(&src)[kBatch] = buf[e & 1];
          uint32_t nan = 0u;  // some byte's bit 7: the batch's V goes the rare way (a NaN code, or its scale)
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int tk = 16 * lw + (b * kBatch + k) * kTpi + sub;
            const uint32_t w[4] = {src[k].x, src[k].y, src[k].z, src[k].w};
            const uint32_t f = ix.fac[kv][tk][pblk];
            uint32_t x[kX];
            if (kv == 0) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (kFp8)
                  attn_e4m3_f16(w[q], x[2 * q], x[2 * q + 1]);
                else
                  attn_e2m1_f16(w[q], reinterpret_cast<uint32_t(&)[4]>(x[4 * q]));
              }
#pragma unroll
              for (int q = 0; q < kX; ++q) x[q] = attn_mul_f16x2(x[q], f);
            } else {
              if (f >= 0x7F800000u) nan = 0x80u;  // a NaN or a large scale
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if (kFp8) {
                  nan |= attn_e4m3_nan(w[q]);
                  x[2 * q] = attn_mul_bf16x2(attn_e4m3_bits(w[q] << 8), f);
                  x[2 * q + 1] = attn_mul_bf16x2(attn_e4m3_bits(w[q]), f);
                } else {
#pragma unroll
                  for (int h = 0; h < 4; ++h)
                    x[4 * q + h] = attn_mul_bf16x2(attn_e2m1_bits(w[q] << (12 - 4 * h)), f);
                }
              }
            }
            put(stage, b * kBatch + k, x);
          }
          if (kv == 1 && (nan & 0x80808080u) != 0u) {
            // the rare way round: pieces with a NaN again (from the cache), with 0 in its place and a note,
            // and pieces with a scale that takes two steps
#pragma unroll 1
            for (int k = b * kBatch; k < (b + 1) * kBatch; ++k) {
              const int tk = 16 * lw + k * kTpi + sub;
              const uint32_t f = ix.fac[1][tk][pblk];
              const bool all = f == 0x7FFF7FFFu, large = !all && f >= 0x7F800000u;
              const uint32_t f1 = large ? 0x7F007F00u : f;
              const uint32_t f2 = (large ? 127u + (f & 0x7Fu) : 127u) << 7, f22 = f2 << 16 | f2;
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(
                  p.v_codes + piece_off + static_cast<uint64_t>(ix.row[tk]) * static_cast<uint32_t>(row_bytes)));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              uint32_t x[kX], any = 0u;
#pragma unroll
              for (int q = 0; q < kX; ++q) x[q] = 0u;
              if (!all) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (kFp8) {
                    const uint32_t z = attn_e4m3_nan(w[q]) & 0x80808080u;
                    any |= z;
                    x[2 * q] = attn_mul_bf16x2(attn_mul_bf16x2(attn_e4m3_bits(w[q] << 8), f1), f22) &
                               ((z & 0x80u ? 0u : 0xFFFFu) | (z & 0x800000u ? 0u : 0xFFFF0000u));
                    x[2 * q + 1] = attn_mul_bf16x2(attn_mul_bf16x2(attn_e4m3_bits(w[q]), f1), f22) &
                                   ((z & 0x8000u ? 0u : 0xFFFFu) | (z & 0x80000000u ? 0u : 0xFFFF0000u));
                  } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                      x[4 * q + h] = attn_mul_bf16x2(attn_mul_bf16x2(attn_e2m1_bits(w[q] << (12 - 4 * h)), f1), f22);
                  }
                }
              }
              if (large) put(stage, k, x);
              if (any != 0u || all) {
                put(stage, k, x);
                if (has) {
                  atomicOr(&note.tok[tk], 1u << pblk);
                  atomicOr(&note.any[tk >> 4], kNoteSome);
                }
              }
            }
          }
          // the batch two steps on
          const int e2 = e + 2;
          const int e3 = e2 >= kSeq ? e2 - kSeq : e2;
          if (e2 == kSeq && more) index_wait(c + 1);
          if (ok && (e2 < kSeq || more)) load_batch(e2 >= kSeq ? ix_next : ix, e3 < kNB ? p.k_codes : p.v_codes, e3 % kNB, src);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full(sidx));
          if (kv == 1) mbar_arrive(i_empty(c % C::kSlots));
        }
      }
    }
  } else {
    // ================================================================ MMA
    setmaxnreg_dec<attn_tile::kRegsOther>();
    // the whole warp walks the runs and waits; one elected lane issues
    if (warp == 16) {
    const uint32_t id_s = attn_idesc<false, false>(128), id_o = attn_idesc<true, true>(p.D);
    const int ksteps = p.D / 16;
    uint32_t el = 0;             // tiles taken from the ring
    uint32_t n_q[2] = {0u, 0u}, n_p[2] = {0u, 0u};
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned int code) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, code));
    };
    auto issue_s = [&](int t, uint32_t stage) {
      tc_fence_after();
      if (attn_elect()) {
        const uint64_t a = smem_desc(q_base + t * C::kPanels * attn_tile::kPanelBytes, 16, 1024, 2);
        const uint64_t b = smem_desc(st_base + stage * C::kStageBytes, 16, 1024, 2);
#pragma unroll
        for (int k = 0; k < kDP / 16; ++k) {
          const uint64_t off = ((k >> 2) * attn_tile::kPanelBytes + (k & 3) * 32) >> 4;
          if (k < ksteps) attn_mma_ss(s_col(t), a + off, b + off, id_s, k > 0);
        }
        tc_commit(s_full(t));
      }
      __syncwarp();
    };
    auto commit = [&](uint32_t bar) {
      if (attn_elect()) tc_commit(bar);
      __syncwarp();
    };
    while (ok && run.left > 0) {
      const int n = run.chunks_here();
      const int tiles = C::kTiles == 1 ? 1 : run.tiles(p);
      // first chunk's scores
      const uint32_t k0 = el % kStages;
      for (int t = 0; ok && t < tiles; ++t) {
        wait(q_full(t), n_q[t]++ & 1u, kErrWaitFull);
        if (t == 0) wait(full(k0), (el / kStages) & 1u, kErrWaitFull);
        if (ok) issue_s(t, k0);
        if (ok && n == 1) commit(q_free(t));
      }
      if (!ok) break;
      commit(empty(k0));
      ++el;
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t vst = el % kStages, vph = (el / kStages) & 1u;
        const uint32_t kst = (el + 1) % kStages, kph = ((el + 1) / kStages) & 1u;
        const bool more = i + 1 < n;
        for (int t = 0; ok && t < tiles; ++t) {
          if (t == 0) wait(full(vst), vph, kErrWaitFull);
          wait(p_full(t), n_p[t]++ & 1u, kErrWaitTmemEmpty);
          if (!ok) break;
          tc_fence_after();
          if (attn_elect()) {
            const uint64_t b = smem_desc(st_base + vst * C::kStageBytes, attn_tile::kPanelBytes, 1024, 2);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              attn_mma_ts(o_col(t), s_col(t) + 8 * k, b + ((k * 2048) >> 4), id_o, i > 0 || k > 0);
            tc_commit(o_full(t));
          }
          __syncwarp();
          if (more) {
            if (t == 0) wait(full(kst), kph, kErrWaitFull);
            if (ok) issue_s(t, kst);
            if (ok && i + 2 == n) commit(q_free(t));  // the unit's last use of q
          }
        }
        if (!ok) break;
        commit(empty(vst));
        if (more) commit(empty(kst));
        el += more ? 2 : 1;
      }
      run.next_unit(p, n);
    }
    // all MMAs done before TMEM is freed and the CTA's shared memory goes
    commit(drain);
    mbar_wait(drain, 0, kErrWaitTmemFull);
    __syncwarp();
    } else if (warp < 19) {
      // ============================================================== rows and factors
      // Three steps a chunk, each on the loads of the step before in the chunk before: the table's
      // entries, the rows and their scales, the factors.
      constexpr int kW = (kDP / 32 + 3) / 4;
      const int tk0 = 64 * (warp - 17) + lane;  // this lane's tokens: tk0 and tk0 + 32
      int off[2] = {-1, -1}, page[2] = {0, 0}, h_ahead = 0;
      uint32_t sck[2][kW], scv[2][kW];
      bool bad[2] = {false, false}, ok = true;
      const int total = run.left;
      auto look = [&]() {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          off[x] = -1;
          const int idx = run.pl.chunk * 128 + tk0 + 32 * x;
          if (run.left <= 0 || idx >= run.nv) continue;
          const int j = run.span.token(idx), pg = attn_page_of(p, j);
          page[x] = __ldg(p.table + static_cast<int64_t>(run.pl.b) * p.max_pages + pg);
          off[x] = j - pg * p.page_size;
        }
        h_ahead = run.pl.hu;
        run.next_chunk(p);
      };
      auto load_scales = [&](const uint8_t* scales, int row, uint32_t (&sc)[kW]) {
        const uint8_t* src = scales + static_cast<int64_t>(max(row, 0)) * p.nb;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          sc[w] = 0u;
          if (row < 0) continue;
          if (p.scale_words) {
            if (4 * w < p.nb) sc[w] = __ldg(reinterpret_cast<const uint32_t*>(src) + w);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (4 * w + k < p.nb) sc[w] |= static_cast<uint32_t>(__ldg(src + 4 * w + k)) << (8 * k);
          }
        }
      };
      look();
      for (int c = 0; ok && c <= total; ++c) {
        int row[2] = {-1, -1};
        bool hide[2] = {false, false};
        if (c < total) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            row[x] = off[x] >= 0 ? attn_row_at(p, page[x], off[x], h_ahead) : -1;
            hide[x] = off[x] >= 0 && row[x] < 0;
          }
          look();
        }
        if (c > 0) {
          // factors and notes of chunk c - 1
          const int at = c - 1;
          AttnIndex<kDP / 32>& ix = s_index[at % C::kSlots];
          AttnNote& nt = notes[at % attn_tile::kInfo];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int tk = tk0 + 32 * x;
            // f16 holds every code times 2^(e - top) for e from top - kReach on
            constexpr int kReach = kFp8 ? 15 : 23;
            int own = 0, low = 255;
#pragma unroll
            for (int b = 0; b < kDP / 32; ++b) {
              const int e = (sck[x][b / 4] >> (8 * (b & 3))) & 255;
              own = e != 255 ? max(own, e) : own;            // NaN scales do not set the common scale
              low = e != 255 && e != 0 ? min(low, e) : low;  // (byte 0: in practice zeros)
            }
            int top = own, low16 = low;
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
              top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
              low16 = min(low16, __shfl_xor_sync(0xffffffffu, low16, d));
            }
            // 16 tokens too far apart for one factor: each by its own largest scale, put right in its column of
            // scores, so that no token's bits hang on its neighbours; a token that is too far apart in
            // itself goes without the tensor cores. (Nor has a row's factor times 2^(top - 127) to stay finite
            // for very large ones.)
            const bool apart = top - low16 > kReach || top > 200, wide = own - low > kReach;
            const int ref = apart ? own : top;
#pragma unroll
            for (int b = 0; b < kDP / 32; ++b) {
              const int ek = (sck[x][b / 4] >> (8 * (b & 3))) & 255, ev = (scv[x][b / 4] >> (8 * (b & 3))) & 255;
              ix.fac[0][tk][b] = ek == 255 ? 0x7E007E00u : attn_f16_pow2(ref - ek);
              ix.fac[1][tk][b] = attn_scale_pair<kFp8>(ev);
            }
            nt.tok[tk] = (bad[x] ? 0x80000000u : 0u) | (wide ? 0x40000000u : 0u) | (apart ? own : 127) << 16;
            const unsigned any = __ballot_sync(0xffffffffu, bad[x]), any_wide = __ballot_sync(0xffffffffu, wide);
            if ((lane & 15) == 0) {
              const unsigned half = 0xFFFFu << (lane & 16);
              nt.kfac[tk >> 4] = apart ? 1.0f : attn_scale_value(top);
              nt.any[tk >> 4] = (any & half ? kNoteSome : 0) | (apart ? kNoteApart : 0) | (any_wide & half ? kNoteWide : 0);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(i_full(at % C::kSlots));
        }
        if (c < total) {
          const int slot = c % C::kSlots;
          ok = __all_sync(0xffffffffu, mbar_wait(i_empty(slot), ((c / C::kSlots) & 1u) ^ 1u, kErrWaitEmpty));
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            s_index[slot].row[tk0 + 32 * x] = max(row[x], 0);
            load_scales(p.k_scales, row[x], sck[x]);
            load_scales(p.v_scales, row[x], scv[x]);
            bad[x] = hide[x];
          }
        }
      }
    } else {
      // ============================================================== q tiles
      uint32_t n_q[2] = {0u, 0u}, n_left = 0u;
      bool ok = true, two = false;
      grid_dependency_wait();  // the q rows
      while (ok && run.left > 0) {
        const int tiles = C::kTiles == 1 ? 1 : run.tiles(p);
        // (a unit of one tile goes at tile 0's pace, and tile 1's warps may still be reading the unit before's
        // last note: it gets its q, and so begins, when they have left that unit)
        if (two && tiles == 1)
          ok = __all_sync(0xffffffffu, mbar_wait(drain + 8, n_left++ & 1u, kErrWaitEmpty));
        two = tiles == 2;
        for (int t = 0; ok && t < tiles; ++t) {
          ok = __all_sync(0xffffffffu, mbar_wait(q_free(t), (n_q[t] & 1u) ^ 1u, kErrWaitEmpty));
          if (!ok) break;
          ++n_q[t];
          // (rows past the sequence's end are other sequences' or past the tensor, read as 0: their
          // scores are not used)
          if (attn_elect()) {
            const int64_t row0 = (run.pl.hu * p.T + run.seq.t0) * p.G + static_cast<int64_t>(run.pl.tile) * kTile + 128 * t;
            mbar_expect_tx(q_full(t), C::kPanels * attn_tile::kPanelBytes);
#pragma unroll
            for (int k = 0; k < C::kPanels; ++k)
              tma_load_2d(q_base + (t * C::kPanels + k) * attn_tile::kPanelBytes, &qmap, q_full(t), 64 * k,
                          static_cast<int32_t>(row0));
          }
          __syncwarp();
        }
        run.next_unit(p, run.chunks_here());
      }
      // copies in flight land before the CTA's shared memory goes
      for (int t = 0; t < C::kTiles; ++t)
        if (n_q[t]) mbar_wait(q_full(t), (n_q[t] - 1) & 1u, kErrWaitFull);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
}

}  // namespace bat
