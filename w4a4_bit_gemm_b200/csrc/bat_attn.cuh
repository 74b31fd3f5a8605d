// Attention of new tokens over the paged MXFP8 / MXFP4 cache (the KV8 / KV4 settings of the
// BATQuant note, en.papernotes.org, Method > Key Designs 4 and Loss & Training): what every
// attention kernel of the library shares, the kernel for few rows (decode), and the kernel
// that joins partial results.
//
//   row (t, h) of a sequence with n new tokens and L cached ones (the new ones among them)
//   sits at position p = L - n + i and sees j <= p with (no window, or j > p - window, or
//   j < sinks):   o = sum_j softmax_j(scale q'.k_j) v_j,   q' = q P_q,   out = o P_o
//   (P_q, P_o: the block transforms given, or none). A row that sees nothing gives 0.
//
// Work split: a unit is a tile of query rows that share one KV head; its visible tokens are
// cut into chunks. The chunks of all units, in a fixed order, are dealt out in equal runs
// over the CTAs, which work out their run from the lengths on the device: the load is even
// for any mix of lengths and nothing about the lengths has to be known on the host. A
// unit that one CTA does alone is finished there; a unit that runs over several CTAs leaves
// one partial (unnormalised o, maximum, sum) a CTA, at most two for each CTA, which
// bat_attn_join_kernel adds in the order of the CTAs. No atomics: results do not
// depend on timing.
//
// The tokens a unit sees are numbered without gaps, i -> j = i < ns ? i : lo + (i - ns)
// (ns sinks below the window's first token lo), so windows and sinks cost nothing in chunks
// that hold no border.
#pragma once

#include "bat_common.cuh"
#include "bat_kv.cuh"

namespace bat {

namespace attn {
constexpr int kChunk = 128;   // visible tokens a chunk
constexpr int kWarps = 8;     // row kernel: warps a CTA, 16 tokens of a chunk each
constexpr int kThreads = 32 * kWarps;
// V's stored elements go to bf16 through their bits, which leaves them 2^120 (E4M3) or 2^126
// (E2M1) too small; the MX scale's multiplication puts that right up to 2^-32, so that
// scales from 2^-127 to 2^39 (E4M3; 2^33 E2M1) stay within bf16. Outputs are multiplied by 2^32
// at the end; a product below 2^-94 may be lost to fp32's smallest number.
constexpr float kUp = 0x1p32f;
}  // namespace attn

// A place in the order of all chunks: sequence, tile, head unit, chunk.
struct AttnPlace {
  int b, tile, hu, chunk;
  int chunks;      // chunks of this unit
};
// Where a CTA's run begins, for the joining kernel.
struct AttnMark {
  int64_t x, total;  // its first chunk, all chunks
  AttnPlace place;   // (nothing if x == total)
};

struct AttnParams {
  const uint16_t* q;       // bf16, token stride q_stride elements, [Hq][D] within a token
  int64_t q_stride;
  const uint8_t* k_codes;
  const uint8_t* k_scales;
  const uint8_t* v_codes;
  const uint8_t* v_scales;
  const int32_t* table;    // [B][max_pages]
  const int32_t* kv_lens;  // [B]
  const int32_t* q_starts; // [B + 1]
  const float* qa;         // factors of P_q (null: none)
  const float* qb;
  const float* oa;         // factors of P_o (null: none)
  const float* ob;
  uint16_t* out;           // bf16 [T][Hq][D]
  float* lse;              // fp32 [T][Hq] or null
  float* part_o;           // [2 * ctas][rows][D]
  float* part_ml;          // [2 * ctas][rows][2]
  AttnMark* marks;         // [ctas]
  int64_t T, num_slots;
  int64_t capacity;        // max_pages * page_size
  int B, max_pages, page_size;
  uint32_t page_mul;       // j / page_size = (j * page_mul) >> page_shift for 0 <= j < 2^31
  int page_shift;
  int Hq, Hkv, G, D, nb;
  int qls, ols;
  int window, sinks;       // window 0: none
  int ctas;                // CTAs the chunks are dealt over
  int unit_rows;           // query rows of a unit
  int head_units;          // row kernel: units a token (Hkv * groups of rows); tile kernel: Hkv
  float scale_log2;        // |scale| * log2(e)
  float q_sign;            // sign of the scale, taken into q
  const uint16_t* qt;      // tile kernel with P_q: f16 rows of q P_q (attn_q_rows), or null
  const float* qt_fac;     // and their factors, [T][Hq]
};

// One sequence's facts, from the device arrays, made safe: n >= 0, tokens inside [0, T),
// the length inside the table's capacity.
struct AttnSeq {
  int t0, n;   // first new token, new tokens
  int len;     // cached tokens
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b) {
  AttnSeq s;
  const int64_t a = p.q_starts[b], e = p.q_starts[b + 1];
  const int64_t a0 = a < 0 ? 0 : (a > p.T ? p.T : a);
  const int64_t e0 = e < a0 ? a0 : (e > p.T ? p.T : e);
  s.t0 = static_cast<int>(a0);
  s.n = static_cast<int>(e0 - a0);
  const int64_t l = p.kv_lens[b];
  s.len = static_cast<int>(l < 0 ? 0 : (l > p.capacity ? p.capacity : l));
  if (l > p.capacity || l < 0 || a < 0 || a > p.T || e < a || e > p.T) atomicOr(&g_dev_error, kErrBadIndex);
  return s;
}

// Visible tokens of the rows at positions first .. last (first <= last): the sinks [0, ns)
// and [lo, hi).
struct AttnSpan {
  int ns, lo, hi;
  __device__ int count() const { return ns + hi - lo; }
  __device__ int token(int i) const { return i < ns ? i : lo + (i - ns); }
};
__device__ __forceinline__ AttnSpan attn_span(const AttnParams& p, int first, int last) {
  AttnSpan s;
  s.hi = last + 1 > 0 ? last + 1 : 0;
  s.lo = p.window > 0 && first + 1 > p.window ? first + 1 - p.window : 0;
  if (s.lo > s.hi) s.lo = s.hi;
  s.ns = p.sinks < s.lo ? p.sinks : s.lo;
  return s;
}

// Units of a sequence: tiles of unit rows for the tile kernel (rows run over tokens and the
// group's heads), single tokens for the row kernel. kTile: rows a tile, 0 for the row kernel.
template <int kTile>
__device__ __forceinline__ int attn_tiles(const AttnParams& p, const AttnSeq& s) {
  return kTile ? static_cast<int>((static_cast<int64_t>(s.n) * p.G + kTile - 1) / (kTile ? kTile : 1)) : s.n;
}
template <int kTile>
__device__ __forceinline__ AttnSpan attn_tile_span(const AttnParams& p, const AttnSeq& s, int tile) {
  int first = tile, last = tile;
  if (kTile) {
    first = static_cast<int>(static_cast<int64_t>(tile) * kTile / p.G);
    const int64_t l = (static_cast<int64_t>(tile + 1) * kTile - 1) / p.G;
    last = static_cast<int>(l < s.n - 1 ? l : s.n - 1);
  }
  const int base = s.len - s.n;
  return attn_span(p, base + first, base + last);
}
template <int kTile>
__device__ __forceinline__ int attn_chunks(const AttnParams& p, const AttnSeq& s, int tile) {
  const int n = attn_tile_span<kTile>(p, s, tile).count();
  return n > 0 ? (n - 1) / attn::kChunk + 1 : 1;  // a tile that sees nothing still writes its rows
}
template <int kTile>
__device__ __forceinline__ int64_t attn_seq_chunks(const AttnParams& p, const AttnSeq& s) {
  int64_t c = 0;
  const int nt = attn_tiles<kTile>(p, s);
  for (int t = 0; t < nt; ++t) c += attn_chunks<kTile>(p, s, t);
  return c * p.head_units;
}

__device__ __forceinline__ int64_t attn_warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// Chunks of all sequences (one warp, together).
template <int kTile>
__device__ __forceinline__ int64_t attn_total(const AttnParams& p, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < p.B; b += 32) sum += attn_seq_chunks<kTile>(p, attn_seq(p, b));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  return sum;
}

// The place of chunk x, 0 <= x < total (one warp, together; every lane gets it).
template <int kTile>
__device__ __forceinline__ AttnPlace attn_locate(const AttnParams& p, int64_t x, int lane) {
  AttnPlace pl;
  pl.b = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int64_t w = b < p.B ? attn_seq_chunks<kTile>(p, attn_seq(p, b)) : 0;
    const int64_t inc = attn_warp_scan(w, lane);
    const int64_t all = __shfl_sync(0xffffffffu, inc, 31);
    if (x < all) {
      const unsigned m = __ballot_sync(0xffffffffu, inc > x);
      const int src = __ffs(static_cast<int>(m)) - 1;
      pl.b = b0 + src;
      x -= __shfl_sync(0xffffffffu, inc - w, src);
      break;
    }
    x -= all;
  }
  const AttnSeq s = attn_seq(p, pl.b);
  const int nt = attn_tiles<kTile>(p, s);
  pl.tile = 0;
  pl.chunks = 1;
  for (int t0 = 0; t0 < nt; t0 += 32) {
    const int t = t0 + lane;
    const int c = t < nt ? attn_chunks<kTile>(p, s, t) : 0;
    const int64_t w = static_cast<int64_t>(c) * p.head_units;
    const int64_t inc = attn_warp_scan(w, lane);
    const int64_t all = __shfl_sync(0xffffffffu, inc, 31);
    if (x < all) {
      const unsigned m = __ballot_sync(0xffffffffu, inc > x);
      const int src = __ffs(static_cast<int>(m)) - 1;
      pl.tile = t0 + src;
      pl.chunks = __shfl_sync(0xffffffffu, c, src);
      x -= __shfl_sync(0xffffffffu, inc - w, src);
      break;
    }
    x -= all;
  }
  pl.hu = static_cast<int>(x / pl.chunks);
  pl.chunk = static_cast<int>(x % pl.chunks);
  return pl;
}

// The first chunk of CTA i's run.
__device__ __forceinline__ int64_t attn_start(int64_t total, int i, int ctas) {
  return total / ctas * i + (total % ctas) * i / ctas;
}

// The unit after (b, tile, hu) that exists.
template <int kTile>
__device__ __forceinline__ void attn_next_unit(const AttnParams& p, AttnPlace& pl, AttnSeq& s) {
  pl.chunk = 0;
  if (++pl.hu < p.head_units) return;
  pl.hu = 0;
  ++pl.tile;
  while (pl.tile >= attn_tiles<kTile>(p, s) && pl.b + 1 < p.B) {
    ++pl.b;
    pl.tile = 0;
    s = attn_seq(p, pl.b);
  }
  pl.chunks = attn_chunks<kTile>(p, s, pl.tile);
}

// Cache row (slot * Hkv + head) of token j of a sequence, or -1 for a page outside the cache, in
// two steps, so that the table's entry can be on its way while other work is done.
__device__ __forceinline__ int attn_page_of(const AttnParams& p, int j) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(j)) * p.page_mul) >> p.page_shift);
}
__device__ __forceinline__ int attn_row_at(const AttnParams& p, int page, int j, int h) {
  const int64_t slot = static_cast<int64_t>(page) * p.page_size + (j - attn_page_of(p, j) * p.page_size);
  if (slot < 0 || slot >= p.num_slots) {
    atomicOr(&g_dev_error, kErrBadIndex);
    return -1;
  }
  return static_cast<int>(slot * p.Hkv + h);
}
__device__ __forceinline__ int attn_cache_row(const AttnParams& p, const int32_t* pages, int j, int h) {
  return attn_row_at(p, __ldg(pages + attn_page_of(p, j)), j, h);
}

__device__ __forceinline__ float attn_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---------------------------------------------------------------- stored elements -> f16, bf16
// K's products run in f16: a conversion instruction gives two codes exactly, q (P_q) keeps 11
// significant bits instead of bf16's 8, and f16's narrow range is no limit since both sides
// are scaled by powers of two: a row of q by its largest channel, the K values by the largest MX
// scale of their token (row kernel) or chunk (tile kernel). What falls below f16's range is
// below 2^-25 of the largest products in the sum it belongs to. V cannot be scaled that way (its
// channels and tokens are not summed with one maximum), so it goes to bf16, whose range is fp32's.
__device__ __forceinline__ uint32_t attn_mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The E4M3 pairs (bytes 0, 1) and (bytes 2, 3) of a word as f16 pairs.
__device__ __forceinline__ void attn_e4m3_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// The E2M1 pairs of a word's four bytes (low nibble first) as f16 pairs.
__device__ __forceinline__ void attn_e2m1_f16(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}
// 2^-d as a pair of f16 (0 below 2^-24).
__device__ __forceinline__ uint32_t attn_f16_pow2(int d) {
  const uint32_t h = d <= 14 ? static_cast<uint32_t>(15 - d) << 10 : (d <= 24 ? 1u << (24 - d) : 0u);
  return h * 0x00010001u;
}
// Value of a scale byte.
__device__ __forceinline__ float attn_scale_value(int byte) {
  return byte == 255 ? NAN : (byte == 0 ? 0x1p-127f : __uint_as_float(static_cast<uint32_t>(byte) << 23));
}
// The power of two that brings a row of largest magnitude m to [2^14, 2^15), and its inverse.
__device__ __forceinline__ float attn_row_up(float m, float& down) {
  int e = static_cast<int>(__float_as_uint(m) >> 23) - 127 - 14;  // m < 2^(e + 15)
  e = e < -100 ? -100 : e;  // (rows below 2^-86 keep fewer bits)
  down = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}
__device__ __forceinline__ uint32_t attn_pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void attn_mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t attn_mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Multiplier of a scale byte as a pair of bf16: 2^(byte - 127 + 88) for E4M3, + 94 for E2M1
// (see kUp). Bytes past the range (see kUp; 255 is NaN by the format) give NaN.
template <bool kFp8>
__device__ __forceinline__ uint32_t attn_scale_pair(uint32_t byte) {
  constexpr uint32_t kAdd = kFp8 ? 88u : 94u;
  const uint32_t f = byte + kAdd > 254u ? 0x7FFFu : (byte + kAdd) << 7;
  return f * 0x00010001u;
}
// Bits 15..8 of both halves of x hold E4M3 bytes -> their bits as bf16 (2^120 too small).
// 0x07F0 in a half's magnitude is a NaN.
__device__ __forceinline__ uint32_t attn_e4m3_bits(uint32_t x) {
  return (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
}
// Bits 15..12 of both halves hold E2M1 codes -> their bits as bf16 (2^126 too small).
__device__ __forceinline__ uint32_t attn_e2m1_bits(uint32_t x) {
  return (x & 0x80008000u) | ((x >> 6) & 0x01C001C0u);
}
// Bit 7 of a byte set where the E4M3 byte of w is a NaN (each magnitude is below 128).
__device__ __forceinline__ uint32_t attn_e4m3_nan(uint32_t w) { return (w & 0x7F7F7F7Fu) + 0x01010101u; }
// The pairs of attn_e4m3_bits with NaN put in for the NaN codes.
__device__ __forceinline__ uint32_t attn_nan_pair(uint32_t r) {
  if ((r & 0x7FFFu) == 0x07F0u) r |= 0x7FFFu;
  if ((r & 0x7FFF0000u) == 0x07F00000u) r |= 0x7FFF0000u;
  return r;
}

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16) on the warp.
__device__ __forceinline__ void attn_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t attn_transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t attn_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Rows' results from unnormalised sums in shared memory: o[r * ldo + d] (in units of 2^-32),
// ml[2 r] the maximum, ml[2 r + 1] the sum. P_o (po, null: none) is applied to the normalised
// fp32 values, and the output is rounded to bf16 once. (token, head) of row r from `where`.
template <class Where>
__device__ __forceinline__ void attn_finish(const AttnParams& p, const float* o, int ldo, const float* ml,
                                            int rows, const float* po, Where where) {
  const int pairs = p.D >> 1;
  for (int i = threadIdx.x; i < rows * pairs; i += blockDim.x) {
    const int r = i / pairs, d = 2 * (i - r * pairs);
    int64_t tok;
    int head;
    if (!where(r, tok, head)) continue;
    const float l = ml[2 * r + 1];
    const float inv = l > 0.0f ? attn::kUp / l : (l == 0.0f ? 0.0f : l);  // l NaN stays NaN
    float v0, v1;
    if (po == nullptr) {
      v0 = o[r * ldo + d] * inv;
      v1 = o[r * ldo + d + 1] * inv;
    } else {
      const float* src = o + r * ldo + (d & ~31);
      const float* pb = po + (d >> 5) * 1024 + (d & 31);
      v0 = v1 = 0.0f;
#pragma unroll 8
      for (int k = 0; k < 32; ++k) {
        const float x = src[k] * inv;
        const float2 c = *reinterpret_cast<const float2*>(pb + 32 * k);
        v0 = __fmaf_rn(x, c.x, v0);
        v1 = __fmaf_rn(x, c.y, v1);
      }
    }
    *reinterpret_cast<uint32_t*>(p.out + (tok * p.Hq + head) * p.D + d) = attn_pack(v0, v1);
    if (p.lse && d == 0)
      p.lse[tok * p.Hq + head] = l == 0.0f ? -INFINITY : (ml[2 * r] + log2f(l)) * 0.69314718055994531f;
  }
}

// ---------------------------------------------------------------- few rows (decode)
// A unit is one token and up to 8 kNT of its heads that share a KV head; a warp takes 16 of
// the chunk's 128 tokens, keeps its own running maximum, sum and o, and the eight warps join
// at the unit's end. Products on mma.sync with the tokens on the 16-row side,
//   S^T = K q^T (16 tokens x 8 heads),   o^T += V^T P^T (D x 16 tokens),
// so that 8 heads fill the other side; both contractions may run over permuted indices, and
// the order is chosen so that each lane's operands are its own 16-byte loads of stored
// codes: lane 4 r + c holds channels of block c (and c + 4) of tokens r and r + 8 for K, and 1/8
// of the channels of tokens 2c, 2c+1, 2c+8, 2c+9 for V. Codes go from global memory to
// registers to the MMA; nothing is staged in shared memory. All rows of a unit see the
// same tokens, so a masked token is simply not loaded (its weight and value are 0).
// Bound: HBM; a CTA has 32 KB of MXFP8 codes in flight, two CTAs an SM.
template <bool kFp8, int kNB4>
struct AttnRowRegs {
  static constexpr int kKw = kFp8 ? 8 : 4;           // K words a token and block
  static constexpr int kVw = (kFp8 ? 4 : 2) * kNB4;  // V words a token
  uint32_t k[2][kNB4][kKw];
  uint32_t v[4][kVw];
  uint32_t ks[2][kNB4];  // scale bytes
  uint32_t vs[4];
};

template <bool kFp8, int kNB4, int kNT>
__global__ void __launch_bounds__(attn::kThreads, kNB4 == 1 && kNT == 1 ? 2 : 1)
    bat_attn_rows_kernel(const AttnParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kDP = 128 * kNB4, kR = 8 * kNT;
  constexpr int kKw = kFp8 ? 8 : 4, kVw = (kFp8 ? 4 : 2) * kNB4;
  constexpr int kMT = kDP / 16;  // m16 tiles of o^T
  // shared memory: [warps][kR][kDP + 4] o, [warps][kR][2] maximum and sum, q rows, P_q, P_o
  constexpr int kLdo = kDP + 4;
  float* so = smem;
  float* sml = so + attn::kWarps * kR * kLdo;
  float* fml = sml + attn::kWarps * kR * 2;  // [kR][2]
  uint16_t* sq = reinterpret_cast<uint16_t*>(fml + kR * 2);  // [kR][kDP] f16
  float* sqf = reinterpret_cast<float*>(sq + kR * kDP);      // [kR] factors of the q rows
  float* fac = sqf + kR;                                     // kFacFloats when factors are given
  const bool any_fac = p.qa != nullptr || p.oa != nullptr;
  float* pq = fac + (any_fac ? kv::kFacFloats : 0);
  float* po = pq + (p.qa ? p.nb * 1024 : 0);
  __shared__ AttnPlace s_place;
  __shared__ int64_t s_run[2];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane & 3, r = lane >> 2;
  allow_dependents();
  if (warp == 0) {
    const int64_t total = attn_total<0>(p, lane);
    const int64_t x0 = attn_start(total, blockIdx.x, p.ctas), x1 = attn_start(total, blockIdx.x + 1, p.ctas);
    AttnPlace pl{};
    if (x0 < total) pl = attn_locate<0>(p, x0, lane);
    if (lane == 0) {
      s_place = pl;
      s_run[0] = x0;
      s_run[1] = x1;
      p.marks[blockIdx.x] = AttnMark{x0, total, pl};
    }
  }
  if (p.qa) kv_build_p(pq, fac, p.qa, p.qb, p.nb, p.qls);
  if (p.oa) {
    __syncthreads();
    kv_build_p(po, fac, p.oa, p.ob, p.nb, p.ols);
  }
  __syncthreads();
  AttnPlace pl = s_place;
  int64_t left = s_run[1] - s_run[0];
  if (left <= 0) return;
  AttnSeq seq = attn_seq(p, pl.b);
  const int hgs = p.head_units / p.Hkv;  // groups of kR heads of a KV head
  const int row_bytes = kFp8 ? p.D : p.D / 2;

  for (int seg = 0; left > 0; ++seg) {
    const int h = pl.hu / hgs, hg = pl.hu - h * hgs;
    const int64_t tok = seq.t0 + pl.tile;
    const int head0 = h * p.G + hg * kR;
    const int nrows = min(kR, p.G - hg * kR);
    const AttnSpan span = attn_tile_span<0>(p, seq, pl.tile);
    const int nv = span.count();
    const int first = pl.chunk;
    const int last = static_cast<int>(min(static_cast<int64_t>(pl.chunks), first + left));  // chunks [first, last)
    const int32_t* pages = p.table + static_cast<int64_t>(pl.b) * p.max_pages;

    // q rows (times P_q) in fp32, then in f16 with the row's power of two
    for (int i = threadIdx.x; i < kR * (kDP / 2); i += attn::kThreads) {
      const int n = i / (kDP / 2), d = 2 * (i - n * (kDP / 2));
      float y0 = 0.0f, y1 = 0.0f;
      if (n < nrows && d < p.D) {
        const uint16_t* src = p.q + tok * p.q_stride + static_cast<int64_t>(head0 + n) * p.D;
        if (p.qa == nullptr) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(src + d);
          y0 = bf16lo(w);
          y1 = bf16hi(w);
        } else {
          const uint32_t* s2 = reinterpret_cast<const uint32_t*>(src + (d & ~31));
          const float* pb = pq + (d >> 5) * 1024 + (d & 31);
#pragma unroll 4
          for (int k = 0; k < 16; ++k) {
            const uint32_t x = s2[k];
            const float2 c0 = *reinterpret_cast<const float2*>(pb + 64 * k);
            const float2 c1 = *reinterpret_cast<const float2*>(pb + 64 * k + 32);
            y0 = __fmaf_rn(bf16lo(x), c0.x, y0);
            y1 = __fmaf_rn(bf16lo(x), c0.y, y1);
            y0 = __fmaf_rn(bf16hi(x), c1.x, y0);
            y1 = __fmaf_rn(bf16hi(x), c1.y, y1);
          }
        }
      }
      *reinterpret_cast<float2*>(so + n * kLdo + d) = make_float2(y0, y1);
    }
    __syncthreads();
    for (int n = warp; n < kR; n += attn::kWarps) {
      float y[kDP / 32], mx = 0.0f;
#pragma unroll
      for (int k = 0; k < kDP / 64; ++k) {
        const float2 v = *reinterpret_cast<const float2*>(so + n * kLdo + 64 * k + 2 * lane);
        y[2 * k] = v.x;
        y[2 * k + 1] = v.y;
        mx = fmaxf(mx, fmaxf(fabsf(v.x), fabsf(v.y)));
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      float down;
      const float up = attn_row_up(mx, down) * p.q_sign;
#pragma unroll
      for (int k = 0; k < kDP / 64; ++k)
        *reinterpret_cast<uint32_t*>(sq + n * kDP + 64 * k + 2 * lane) = attn_pack_f16(y[2 * k] * up, y[2 * k + 1] * up);
      if (lane == 0) sqf[n] = down * p.scale_log2;
    }
    __syncthreads();
    // this lane's q operands: heads r (and r + 8), the channels of its K words; the factors
    // of its score columns
    uint32_t qf[kNT][kNB4][16];
    float cs[kNT][2];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      cs[t][0] = sqf[8 * t + 2 * c];
      cs[t][1] = sqf[8 * t + 2 * c + 1];
#pragma unroll
      for (int b4 = 0; b4 < kNB4; ++b4) {
        const uint4* src = reinterpret_cast<const uint4*>(sq + (8 * t + r) * kDP + 32 * (c + 4 * b4));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint4 w = src[s];
          qf[t][b4][4 * s] = w.x;
          qf[t][b4][4 * s + 1] = w.y;
          qf[t][b4][4 * s + 2] = w.z;
          qf[t][b4][4 * s + 3] = w.w;
        }
      }
    }

    float m[kNT][2], l[kNT][2], o[kNT][kMT][4];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < kMT; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
    }

    // cache row of token `lane` of this warp's 16 (lanes 16..31 repeat), -1: none
    auto lookup = [&](int chunk) -> int {
      const int i = chunk * attn::kChunk + 16 * warp + (lane & 15);
      if (chunk >= last || i >= nv) return -1;
      return attn_cache_row(p, pages, span.token(i), h);
    };
    AttnRowRegs<kFp8, kNB4> g;
    auto load_k = [&](int rows16) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = __shfl_sync(0xffffffffu, rows16, r + 8 * x);
#pragma unroll
        for (int b4 = 0; b4 < kNB4; ++b4) {
          const int blk = c + 4 * b4;
          const bool ok = row >= 0 && blk < p.nb;
          const uint4* src = reinterpret_cast<const uint4*>(p.k_codes + static_cast<int64_t>(row) * row_bytes +
                                                            blk * (kFp8 ? 32 : 16));
#pragma unroll
          for (int k = 0; k < kKw / 4; ++k) {
            const uint4 w = ok ? __ldg(src + k) : make_uint4(0u, 0u, 0u, 0u);
            g.k[x][b4][4 * k] = w.x;
            g.k[x][b4][4 * k + 1] = w.y;
            g.k[x][b4][4 * k + 2] = w.z;
            g.k[x][b4][4 * k + 3] = w.w;
          }
          g.ks[x][b4] = ok ? __ldg(p.k_scales + static_cast<int64_t>(row) * p.nb + blk) : 0u;
        }
      }
    };
    const bool v_has = 16 * kNB4 * r < p.D;
    auto load_v = [&](int rows16) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int row = __shfl_sync(0xffffffffu, rows16, 2 * c + (x & 1) + 8 * (x >> 1));
        const bool ok = row >= 0 && v_has;
        const uint8_t* src = p.v_codes + static_cast<int64_t>(row) * row_bytes + r * (kVw * 4);
        if (kVw == 2) {
          const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0u, 0u);
          g.v[x][0] = w.x;
          g.v[x][1] = w.y;
        } else {
#pragma unroll
          for (int k = 0; k < kVw / 4; ++k) {
            const uint4 w = ok ? __ldg(reinterpret_cast<const uint4*>(src) + k) : make_uint4(0u, 0u, 0u, 0u);
            g.v[x][4 * k] = w.x;
            g.v[x][4 * k + 1] = w.y;
            g.v[x][4 * k + 2] = w.z;
            g.v[x][4 * k + 3] = w.w;
          }
        }
        g.vs[x] = ok ? __ldg(p.v_scales + static_cast<int64_t>(row) * p.nb + (16 * kNB4 * r >> 5)) : 0u;
      }
    };

    int rows_now = lookup(first);
    load_k(rows_now);
    load_v(rows_now);
    int rows_next = lookup(first + 1);
    for (int ch = first; ch < last; ++ch) {
      // ---- S^T = K q^T
      float s[kNT][4];
#pragma unroll
      for (int t = 0; t < kNT; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
      int top[2];  // the tokens' largest scale bytes (the quad holds a token's blocks)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[x] = static_cast<int>(g.ks[x][0]);
        if (kNB4 == 2) top[x] = max(top[x], static_cast<int>(g.ks[x][kNB4 - 1]));
        top[x] = max(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
        top[x] = max(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
      }
#pragma unroll
      for (int b4 = 0; b4 < kNB4; ++b4) {
        const uint32_t f0 = attn_f16_pow2(top[0] - static_cast<int>(g.ks[0][b4]));
        const uint32_t f1 = attn_f16_pow2(top[1] - static_cast<int>(g.ks[1][b4]));
#pragma unroll
        for (int w = 0; w < kKw; ++w) {
          // a word holds one k-step's (E4M3) or two k-steps' (E2M1) operands of this lane
          uint32_t a[2][4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (kFp8)
              attn_e4m3_f16(g.k[x][b4][w], a[x][0], a[x][1]);
            else
              attn_e2m1_f16(g.k[x][b4][w], a[x]);
#pragma unroll
            for (int e = 0; e < (kFp8 ? 2 : 4); ++e) a[x][e] = attn_mul_f16x2(a[x][e], x ? f1 : f0);
          }
#pragma unroll
          for (int e = 0; e < (kFp8 ? 2 : 4); e += 2) {
            const int st = kFp8 ? w : 2 * w + e / 2;
#pragma unroll
            for (int t = 0; t < kNT; ++t)
              attn_mma_f16(s[t], a[0][e], a[1][e], a[0][e + 1], a[1][e + 1], qf[t][b4][2 * st], qf[t][b4][2 * st + 1]);
          }
        }
      }
      const float kv0 = attn_scale_value(top[0]), kv1 = attn_scale_value(top[1]);
      const bool see0 = __shfl_sync(0xffffffffu, rows_now, r) >= 0;
      const bool see1 = __shfl_sync(0xffffffffu, rows_now, r + 8) >= 0;
      load_k(rows_next);
      const int rows_after = lookup(ch + 2);
      // ---- softmax over the tokens, for the columns 2c and 2c + 1
      uint32_t pb[kNT][2];
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        float x[4], mx[2];
        x[0] = see0 ? s[t][0] * kv0 * cs[t][0] : -INFINITY;
        x[1] = see0 ? s[t][1] * kv0 * cs[t][1] : -INFINITY;
        x[2] = see1 ? s[t][2] * kv1 * cs[t][0] : -INFINITY;
        x[3] = see1 ? s[t][3] * kv1 * cs[t][1] : -INFINITY;
        mx[0] = fmaxf(x[0], x[2]);
        mx[1] = fmaxf(x[1], x[3]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], d));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], d));
        }
        const bool up = mx[0] > m[t][0] || mx[1] > m[t][1];
        if (__any_sync(0xffffffffu, up)) {
          float al[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float mn = fmaxf(m[t][k], mx[k]);
            al[k] = mn == -INFINITY ? 1.0f : attn_exp2(m[t][k] - mn);
            m[t][k] = mn;
            l[t][k] *= al[k];
          }
#pragma unroll
          for (int i = 0; i < kMT; ++i) {
            o[t][i][0] *= al[0];
            o[t][i][1] *= al[1];
            o[t][i][2] *= al[0];
            o[t][i][3] *= al[1];
          }
        }
        const float m0 = m[t][0] == -INFINITY ? 0.0f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.0f : m[t][1];
        x[0] = attn_exp2(x[0] - m0);
        x[1] = attn_exp2(x[1] - m1);
        x[2] = attn_exp2(x[2] - m0);
        x[3] = attn_exp2(x[3] - m1);
        l[t][0] += x[0] + x[2];
        l[t][1] += x[1] + x[3];
        // weights in bf16 (half a step 2^-9 of each, unbiased); the sum keeps fp32
        pb[t][0] = attn_transpose8(attn_pack(x[0], x[1]));
        pb[t][1] = attn_transpose8(attn_pack(x[2], x[3]));
      }
      // ---- o^T += V^T P^T
      const uint32_t fl = (attn_scale_pair<kFp8>(g.vs[0]) & 0xFFFFu) | (attn_scale_pair<kFp8>(g.vs[1]) << 16);
      const uint32_t fh = (attn_scale_pair<kFp8>(g.vs[2]) & 0xFFFFu) | (attn_scale_pair<kFp8>(g.vs[3]) << 16);
      bool slow = false;
      if (kFp8) {
        // a stored NaN: the rare way round, with NaN put in
        uint32_t nv4 = 0u;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int k = 0; k < kVw; ++k) nv4 |= attn_e4m3_nan(g.v[x][k]);
        slow = __any_sync(0xffffffffu, (nv4 & 0x80808080u) != 0u);
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        uint32_t a[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = 2 * i + e;  // the lane's channel
          uint32_t lo, hi;
          if (kFp8) {
            const int by = d & 3;
            const uint32_t sel = static_cast<uint32_t>(by) << 4 | static_cast<uint32_t>(4 + by) << 12;
            lo = attn_e4m3_bits(__byte_perm(g.v[0][d >> 2], g.v[1][d >> 2], sel));
            hi = attn_e4m3_bits(__byte_perm(g.v[2][d >> 2], g.v[3][d >> 2], sel));
            if (slow) {
              lo = attn_nan_pair(lo);
              hi = attn_nan_pair(hi);
            }
          } else {
            const int by = (d & 7) >> 1;
            const uint32_t sel = static_cast<uint32_t>(by) << 4 | static_cast<uint32_t>(4 + by) << 12;
            uint32_t x0 = __byte_perm(g.v[0][d >> 3], g.v[1][d >> 3], sel);
            uint32_t x1 = __byte_perm(g.v[2][d >> 3], g.v[3][d >> 3], sel);
            if (!(d & 1)) {
              x0 <<= 4;
              x1 <<= 4;
            }
            lo = attn_e2m1_bits(x0);
            hi = attn_e2m1_bits(x1);
          }
          a[e] = attn_mul_bf16x2(lo, fl);
          a[2 + e] = attn_mul_bf16x2(hi, fh);
        }
#pragma unroll
        for (int t = 0; t < kNT; ++t) attn_mma(o[t][i], a[0], a[1], a[2], a[3], pb[t][0], pb[t][1]);
      }
      load_v(rows_next);
      rows_now = rows_next;
      rows_next = rows_after;
    }

    // ---- join the warps
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][k] += __shfl_xor_sync(0xffffffffu, l[t][k], d);
      if (r == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float* ml = sml + (warp * kR + 8 * t + 2 * c + k) * 2;
          ml[0] = m[t][k];
          ml[1] = l[t][k];
        }
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        // rows r and r + 8 of the tile are the lane's channels 16 kNB4 r + 2 i and + 1
        const int d = 16 * kNB4 * r + 2 * i;
        float* o0 = so + (warp * kR + 8 * t + 2 * c) * kLdo + d;
        *reinterpret_cast<float2*>(o0) = make_float2(o[t][i][0], o[t][i][2]);
        *reinterpret_cast<float2*>(o0 + kLdo) = make_float2(o[t][i][1], o[t][i][3]);
      }
    }
    __syncthreads();
    const bool whole = first == 0 && last == pl.chunks;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (seg == 0 ? 0 : 1);
    float* dst = whole ? so : p.part_o + static_cast<int64_t>(slot) * kR * p.D;
    const int ldd = whole ? kLdo : p.D;
    float* dml = whole ? fml : p.part_ml + static_cast<int64_t>(slot) * kR * 2;
    for (int i = threadIdx.x; i < nrows * p.D; i += attn::kThreads) {
      const int n = i / p.D, d = i - n * p.D;
      float mm = -INFINITY;
      bool bad = false;
#pragma unroll
      for (int w = 0; w < attn::kWarps; ++w) {
        const float mw = sml[(w * kR + n) * 2];
        mm = fmaxf(mm, mw);
        bad |= sml[(w * kR + n) * 2 + 1] != sml[(w * kR + n) * 2 + 1];
      }
      float acc = 0.0f, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < attn::kWarps; ++w) {
        const float mw = sml[(w * kR + n) * 2];
        const float f = mw == -INFINITY ? 0.0f : attn_exp2(mw - mm);
        acc = __fmaf_rn(so[(w * kR + n) * kLdo + d], f, acc);
        sum = __fmaf_rn(sml[(w * kR + n) * 2 + 1], f, sum);
      }
      if (bad) acc = sum = NAN;
      // warp 0's slice is read by this thread alone at (n, d): the sum may replace it
      dst[n * ldd + d] = acc;
      if (d == 0) {
        dml[2 * n] = mm;
        dml[2 * n + 1] = sum;
      }
    }
    __syncthreads();
    if (whole) {
      attn_finish(p, so, kLdo, fml, nrows, p.oa ? po : nullptr, [&](int n, int64_t& t, int& hd) {
        t = tok;
        hd = head0 + n;
        return true;
      });
      __syncthreads();
    }
    left -= last - first;
    if (left > 0) attn_next_unit<0>(p, pl, seq);
  }
}

// ---------------------------------------------------------------- joining partial results
// CTA (x, y): if CTA x + 1's run begins inside a unit, and no earlier run does, the parts
// of that unit (the last of CTA x, then the first of x + 1, x + 2, ...) are joined here, a warp a
// row. kTile as in the kernel that wrote them. Bound: the parts' bytes, or launch latency.
template <int kTile>
__global__ void __launch_bounds__(256) bat_attn_join_kernel(const AttnParams p) {
  extern __shared__ __align__(16) float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i1 = blockIdx.x + 1;
  float* so = smem + warp * 260;  // [D] of this warp's row, its maximum and sum
  float* po = nullptr;
  grid_dependency_wait();
  const AttnMark mk = p.marks[i1];
  const int64_t total = mk.total, x = mk.x;
  if (x >= total) return;
  const AttnPlace pl = mk.place;
  const int64_t u0 = x - pl.chunk, u1 = u0 + pl.chunks;
  if (pl.chunk == 0 || attn_start(total, i1 - 1, p.ctas) > u0) return;  // no split here, or an earlier CTA's
  int end = i1 + 1;  // parts of CTAs [i1 - 1, end)
  while (end < p.ctas && attn_start(total, end, p.ctas) < u1) ++end;
  if (p.oa) {
    po = smem + 8 * 260 + kv::kFacFloats;
    kv_build_p(po, smem + 8 * 260, p.oa, p.ob, p.nb, p.ols);
  }
  const int rows = p.unit_rows;
  const AttnSeq seq = attn_seq(p, pl.b);
  const int hgs = p.head_units / p.Hkv;
  const int h = pl.hu / hgs, hg = pl.hu - h * hgs;
  for (int rr = blockIdx.y * 8 + warp; rr < rows; rr += gridDim.y * 8) {
    int64_t tok;
    int head;
    if (kTile) {
      const int64_t row = static_cast<int64_t>(pl.tile) * kTile + rr;
      const int64_t t = row / p.G;
      if (t >= seq.n) break;
      tok = seq.t0 + t;
      head = h * p.G + static_cast<int>(row - t * p.G);
    } else {
      if (hg * rows + rr >= p.G) break;
      tok = seq.t0 + pl.tile;
      head = h * p.G + hg * rows + rr;
    }
    // running over the parts in order: maximum, sum and o, as in the kernels
    float mm = -INFINITY, sum = 0.0f;
    float2 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float2(0.0f, 0.0f);
    bool bad = false;
    for (int i = i1 - 1; i < end; ++i) {
      const int64_t xi = attn_start(total, i, p.ctas);
      if (xi >= attn_start(total, i + 1, p.ctas)) continue;  // an empty run
      // the unit is the first of CTA i's run if the run begins inside the unit (or at it)
      const int64_t at = (2 * static_cast<int64_t>(i) + (xi >= u0 ? 0 : 1)) * rows + rr;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * at);
      float2 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (64 * k + 2 * lane < p.D) v[k] = *reinterpret_cast<const float2*>(p.part_o + at * p.D + 64 * k + 2 * lane);
      bad |= ml.y != ml.y;
      if (ml.x == -INFINITY) continue;  // saw nothing
      const float mn = fmaxf(mm, ml.x);
      const float fo = attn_exp2(mm - mn), fi = attn_exp2(ml.x - mn);
      mm = mn;
      sum = sum * fo + ml.y * fi;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (64 * k + 2 * lane < p.D) {
          acc[k].x = acc[k].x * fo + v[k].x * fi;
          acc[k].y = acc[k].y * fo + v[k].y * fi;
        }
    }
    if (bad) sum = NAN;
    const float inv = sum > 0.0f ? attn::kUp / sum : (sum == 0.0f ? 0.0f : sum);
    uint16_t* dst = p.out + (tok * p.Hq + head) * p.D;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      acc[k].x *= inv;
      acc[k].y *= inv;
      if (po != nullptr && 64 * k + 2 * lane < p.D) *reinterpret_cast<float2*>(so + 64 * k + 2 * lane) = acc[k];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = 64 * k + 2 * lane;
      if (d >= p.D) break;
      if (po != nullptr) {
        const float* src = so + (d & ~31);
        const float* pb = po + (d >> 5) * 1024 + (d & 31);
        acc[k] = make_float2(0.0f, 0.0f);
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
          const float2 cf = *reinterpret_cast<const float2*>(pb + 32 * j);
          acc[k].x = __fmaf_rn(src[j], cf.x, acc[k].x);
          acc[k].y = __fmaf_rn(src[j], cf.y, acc[k].y);
        }
      }
      *reinterpret_cast<uint32_t*>(dst + d) = attn_pack(acc[k].x, acc[k].y);
    }
    __syncwarp();
    if (p.lse && lane == 0)
      p.lse[tok * p.Hq + head] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * 0.69314718055994531f;
  }
}

}  // namespace bat
