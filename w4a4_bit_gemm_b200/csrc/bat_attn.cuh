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
constexpr int kWarps = 4;     // row kernel: warps a CTA, 32 tokens of a chunk each
constexpr int kThreads = 32 * kWarps;
// V's stored elements go to bf16 through their bits, which leaves them 2^120 (E4M3) or 2^126
// (E2M1) too small; the MX scale's multiplication puts that right up to 2^-32, in one step for
// scales from 2^-127 to 2^39 (E4M3; 2^33 E2M1), in two for larger ones. Outputs are multiplied by 2^32
// at the end; a product below 2^-94 may be lost to fp32's smallest number, and with weights of up to 2^40
// (the tile kernel's reference) sums of values above 2^100 may leave its range.
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
  float* part_o;           // [2 * ctas][rows][D], unnormalised
  float* part_ml;          // [2 * ctas][rows][2]
  AttnMark* marks;         // [ctas]
  int64_t T;
  int64_t capacity;        // max_pages * page_size
  int B, max_pages, page_size;
  uint32_t page_mul;       // j / page_size = (j * page_mul) >> (32 + page_shift) for 0 <= j < 2^31
  int page_shift;
  uint32_t pages, slots;   // of the cache: ceil(slots / page_size), slots (< 2^30)
  int Hq, Hkv, G, D, nb;
  int qls, ols;
  int window, sinks;       // window 0: none
  int ctas;                // CTAs the chunks are dealt over
  int unit_rows;           // query rows of a unit
  int head_units;          // row kernel: units a token (Hkv * groups of rows); tile kernel: Hkv
  int scale_words;         // the scale arrays may be read by 32-bit words (nb % 4 == 0, aligned)
  float scale_log2;        // |scale| * log2(e)
  float q_sign;            // sign of the scale, taken into q
  const uint16_t* qt;      // tile kernel: prepared q rows, f16 [Hkv][T][G][D]
  const float* qt_fac;     // and their factors, [Hkv][T][G]
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

// The first chunk of CTA i's run: total / ctas chunks each, the remainder spread (ctas < 2^15).
struct AttnDeal {
  int64_t per;
  uint32_t rem, ctas;
  __device__ __forceinline__ AttnDeal(int64_t total, int n) {
    ctas = static_cast<uint32_t>(n);
    per = total < (int64_t{1} << 31) ? static_cast<int64_t>(static_cast<uint32_t>(total) / ctas) : total / n;
    rem = static_cast<uint32_t>(total - per * n);
  }
  __device__ __forceinline__ int64_t start(int i) const { return per * i + rem * static_cast<uint32_t>(i) / ctas; }
};

// The chunks of all sequences, and the place of the first chunk of CTA i's run, with its sequence
// (one warp, together; every lane gets them).
template <int kTile>
__device__ __forceinline__ AttnMark attn_mark(const AttnParams& p, int cta, int lane, int64_t& run, AttnSeq& seq) {
  AttnMark mk;
  seq = AttnSeq{0, 0, 0};
  if (lane < p.B) seq = attn_seq(p, lane);
  const int64_t w0 = lane < p.B ? attn_seq_chunks<kTile>(p, seq) : 0;
  int64_t total = w0;
  for (int b = lane + 32; b < p.B; b += 32) total += attn_seq_chunks<kTile>(p, attn_seq(p, b));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  const AttnDeal deal(total, p.ctas);
  int64_t x = deal.start(cta);
  run = deal.start(cta + 1) - x;
  mk.x = x;
  mk.total = total;
  mk.place = AttnPlace{};
  if (x >= total) return mk;
  AttnPlace& pl = mk.place;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    const int64_t w = b0 == 0 ? w0 : (b < p.B ? attn_seq_chunks<kTile>(p, attn_seq(p, b)) : 0);
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
  if (pl.b < 32) {
    seq.t0 = __shfl_sync(0xffffffffu, seq.t0, pl.b);
    seq.n = __shfl_sync(0xffffffffu, seq.n, pl.b);
    seq.len = __shfl_sync(0xffffffffu, seq.len, pl.b);
  } else {
    seq = attn_seq(p, pl.b);
  }
  const int nt = attn_tiles<kTile>(p, seq);
  for (int t0 = 0; t0 < nt; t0 += 32) {
    const int t = t0 + lane;
    const int c = t < nt ? attn_chunks<kTile>(p, seq, t) : 0;
    if (nt == 1) {  // (the usual decode step)
      pl.chunks = __shfl_sync(0xffffffffu, c, 0);
      break;
    }
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
  // x < head_units * chunks < 2^31 (at most 2^30 rows of the cache are seen once by each head)
  pl.hu = static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(pl.chunks));
  pl.chunk = static_cast<int>(x) - pl.hu * pl.chunks;
  return mk;
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
  // (page_mul 0: pages of one token)
  return p.page_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(j), p.page_mul) >> p.page_shift) : j;
}
__device__ __forceinline__ int attn_row_at(const AttnParams& p, int page, int offset, int h) {
  // pages within the cache: their slots fit 30 bits
  const uint32_t slot = static_cast<uint32_t>(page) * static_cast<uint32_t>(p.page_size) + static_cast<uint32_t>(offset);
  if (static_cast<uint32_t>(page) >= p.pages || slot >= p.slots) {
    atomicOr(&g_dev_error, kErrBadIndex);
    return -1;
  }
  return static_cast<int>(slot * static_cast<uint32_t>(p.Hkv) + static_cast<uint32_t>(h));
}
__device__ __forceinline__ int attn_cache_row(const AttnParams& p, const int32_t* pages, int j, int h) {
  const int pg = attn_page_of(p, j);
  return attn_row_at(p, __ldg(pages + pg), j - pg * p.page_size, h);
}

__device__ __forceinline__ float attn_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (a NaN among the operands is passed over)
__device__ __forceinline__ float attn_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float attn_min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 2^d as the product of two numbers, for what is larger than its reference and so may outlast fp32's least 2^d.
__device__ __forceinline__ float2 attn_exp2_two(float d) {
  const float h = floorf(0.5f * d);
  return make_float2(attn_exp2(h), attn_exp2(d - h));
}

// ---------------------------------------------------------------- stored elements -> f16, bf16
// f16 takes two codes from one conversion instruction, exactly, and gives q P_q and the weights 11
// significant bits instead of bf16's 8. Its narrow range is no limit where both sides of a sum
// are scaled by powers of two: a row of q by its largest channel; in the row kernel the scores of
// each 32-channel block by its MX scale in fp32, and V through the weights (below); in the
// tile kernel K by the largest scale of 16 neighbouring tokens where f16 then holds all their codes, by
// each token's own largest where it does not. The tile kernel's V goes to bf16, whose range is
// fp32's: there the weights cannot take its scales up.
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
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8) on the warp, f16 operands.
__device__ __forceinline__ void attn_mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same on bf16 operands.
__device__ __forceinline__ void attn_mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
// (see kUp). 255, NaN by the format, is 0x7FFF; a byte whose multiplier bf16 does not hold is 0x7F80 plus the
// powers of two above 2^127 that are missing (at most 94).
template <bool kFp8>
__device__ __forceinline__ uint32_t attn_scale_pair(uint32_t byte) {
  constexpr uint32_t kAdd = kFp8 ? 88u : 94u;
  const uint32_t f = byte + kAdd <= 254u ? (byte + kAdd) << 7 : (byte == 255u ? 0x7FFFu : 0x7F80u + (byte + kAdd - 254u));
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
__device__ __forceinline__ uint32_t attn_transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t attn_pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void attn_f16_floats(uint32_t x, float& lo, float& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(x));
}
// A pair of f16 code values (at most 4 significant bits) as bf16.
__device__ __forceinline__ uint32_t attn_f16_to_bf16(uint32_t x) {
  float lo, hi;
  attn_f16_floats(x, lo, hi);
  return attn_pack(lo, hi);
}

// ---------------------------------------------------------------- block transforms
// Factors of P staged in shared memory: A, then B (when they fit; else read where they are).
struct AttnFactors {
  const float* a;
  const float* b;
  int ls;
};
__host__ __device__ constexpr int attn_factor_floats(int nb, int ls) {
  const int na = 1 << (2 * ls), nbf = nb << (10 - 2 * ls);
  return (na + 3) / 4 * 4 + nbf <= kv::kFacFloats ? (na + 3) / 4 * 4 + (nbf + 3) / 4 * 4 : 0;
}
// (no barrier: the caller's next one orders it)
// Threads from `tid` 0 up, `nt` of them, take part (a negative tid does not).
__device__ __forceinline__ AttnFactors attn_stage_factors(float* dst, const float* a, const float* b, int nb, int ls,
                                                          int tid, int nt) {
  if (attn_factor_floats(nb, ls) == 0) return AttnFactors{a, b, ls};
  const int na = 1 << (2 * ls), nbf = nb << (10 - 2 * ls);
  float* db = dst + (na + 3) / 4 * 4;
  if (tid < 0) return AttnFactors{dst, db, ls};
  for (int i = tid; i < na; i += nt) dst[i] = __ldg(a + i);
  for (int i = tid; i < nbf; i += nt) db[i] = __ldg(b + i);
  return AttnFactors{dst, db, ls};
}
// The four outputs n = q, 8 + q, 16 + q, 24 + q (q < 8) of block `blk`: y = x (B_blk (x) A), x the
// block's 32 values. The 8 x 8 / 4 x 4 split goes by its two small products.
__device__ __forceinline__ void attn_block_apply(const AttnFactors& f, int blk, const float* x, int q, float (&y)[4]) {
  if (f.ls == 3) {
    y[0] = y[1] = y[2] = y[3] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float z = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) z = __fmaf_rn(x[8 * i + k], f.a[8 * k + q], z);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = __fmaf_rn(z, f.b[16 * blk + 4 * i + j], y[j]);
    }
    return;
  }
  const int sm = (1 << f.ls) - 1, t = 32 >> f.ls;
  const float* bb = f.b + static_cast<int64_t>(blk) * t * t;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = 8 * j + q;
    float acc = 0.0f;
#pragma unroll 4
    for (int k = 0; k < 32; ++k)
      acc = __fmaf_rn(x[k], __fmul_rn(bb[(k >> f.ls) * t + (n >> f.ls)], f.a[((k & sm) << f.ls) + (n & sm)]), acc);
    y[j] = acc;
  }
}

// ---------------------------------------------------------------- few rows (decode)
// A unit is one token and up to 8 kNT of its heads that share a KV head; a warp takes 32 of
// the chunk's 128 tokens, keeps its own running maximum, sum and o, and the four warps join
// at the unit's end. Products on mma.sync with the tokens on the 16-row side,
//   S^T = K q^T (16 tokens x 8 heads),   o^T += V^T P^T (channels x 16 tokens),
// so that 8 heads fill the other side. All rows of a unit see the same tokens, so a masked token is
// simply not loaded (zeros in its place).
// Each warp streams its tokens through its own ring in shared memory (16-byte asynchronous
// copies, kStages tiles of 32 tokens, refilled as soon as a tile is used), so no
// barrier is met between a unit's start and its end, and the loads' latency is covered whatever
// the lengths. A lane looks up one token of the tile, its page, row and scales.
// Scales: S^T of each 32-channel block is multiplied by the tokens' K scales in fp32. For V, with E
// the largest scale exponent of a token, the weights are taken as
//   w = 2^(x + E - M + 13),  M the running maximum of x + E  (x: the score in log2 units),
// and multiplied by 2^(e_b - E) <= 1 for block b, so V's codes enter the product as they are.
// Both are f16 where every factor w 2^(e_b - E) of the tile is a normal f16 number (2^-14 and more: x + E
// within 2^27 of M for blocks of one size), which keeps the weights' 11 bits. A tile where one is not, be it a
// weight far below the maximum or a block far below its token's largest, takes the wide way: the
// weights as the sum of two bf16 numbers (16 bits, fp32's range), twice the products.
// Bound: latency for KV8 (two warps a scheduler; 3.3 to 3.8 TB/s of the measured 6.5), the instructions for
// KV4 (908 a warp and tile): 8 x 65536 tokens of 8 heads of 128 in 227 us (2.5 TB/s). A step of 16
// sequences of up to 4096 tokens: 42 us, 8 of them a unit's start (look-ups, q, first copies). Where every tile
// takes the wide way: 8 x 16384 tokens 135 instead of 104 us in KV8, 116 instead of 80 in KV4.
template <bool kFp8, int kNB>
struct AttnRowCfg {
  static constexpr int kTok = 32;                            // tokens of a warp's tile
  static constexpr int kBytes = kFp8 ? 32 * kNB : 16 * kNB;  // codes of a token, padded to kNB blocks
  // row strides in shared memory that keep the fragment loads free of bank conflicts: K is read
  // by 8 bytes (E4M3) at 8 c of tokens r, by 4 (E2M1); V by 4 or 2 bytes of tokens 2c
  static constexpr int kKs = kFp8 ? kBytes + 32 : kBytes + 16;
  static constexpr int kVs = kBytes + 16;
  static constexpr int kStages = !kFp8 && kNB == 2 ? 3 : 2;
  static constexpr int kStageBytes = kTok * (kKs + kVs);
  // factors of a tile: K scales fp32 [32][kNB], V factors f16 [kNB][32], E and the least e_b bf16 [32][2]
  static constexpr int kFacBytes = kTok * kNB * 4 + kTok * kNB * 2 + kTok * 4;
  static constexpr int kWarpBytes = kStages * kStageBytes + 2 * kFacBytes;
};
constexpr size_t attn_rows_ring_bytes(int warp_bytes, int nt, int nb) {
  const size_t ring = static_cast<size_t>(attn::kWarps) * warp_bytes;
  const size_t join = static_cast<size_t>(attn::kWarps) * 8 * nt * (32 * nb + 4) * 4;  // takes the ring's place
  return ring > join ? ring : join;
}
// CTAs an SM that registers and shared memory allow.
constexpr int attn_rows_per_sm(bool fp8, int nb, int nt) {
  return nb * nt <= 4 ? (fp8 && nb == 4 ? 2 : 4) : (fp8 && nb == 8 ? 1 : 2);
}

__device__ __forceinline__ void attn_copy16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void attn_copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void attn_copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

template <bool kFp8, int kNB, int kNT>
__global__ void __launch_bounds__(attn::kThreads, attn_rows_per_sm(kFp8, kNB, kNT)) bat_attn_rows_kernel(const AttnParams p) {
  using C = AttnRowCfg<kFp8, kNB>;
  extern __shared__ __align__(16) float smem[];
  constexpr int kDP = 32 * kNB, kR = 8 * kNT, kS = C::kStages;
  constexpr int kLdo = kDP + 4;
  float* so = smem;  // the rings; at a unit's end [warps][kR][kLdo] o
  float* sml = smem + attn_rows_ring_bytes(C::kWarpBytes, kNT, kNB) / 4;  // [warps][kR][2] maximum and sum
  float* fml = sml + attn::kWarps * kR * 2;                    // [kR][2]
  float* sy = fml + kR * 2;                                    // [kR][kLdo] q rows in fp32
  float* sqf = sy + kR * kLdo;                                 // [kR] factors of the q rows
  uint16_t* sq = reinterpret_cast<uint16_t*>(sqf + kR);        // [kR][kDP] f16
  float* fac_q = reinterpret_cast<float*>(sq + kR * kDP);
  float* fac_o = fac_q + (p.qa ? attn_factor_floats(p.nb, p.qls) : 0);
  __shared__ AttnPlace s_place;
  __shared__ AttnSeq s_seq;
  __shared__ int64_t s_run;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane & 3, r = lane >> 2;
  // everything below reads what kernels before this one write; the joining kernel may start its
  // set-up once that is complete
  grid_dependency_wait();
  allow_dependents();
  if (warp == 0) {
    int64_t run;
    AttnSeq seq0;
    const AttnMark mk = attn_mark<0>(p, blockIdx.x, lane, run, seq0);
    if (lane == 0) {
      s_place = mk.place;
      s_seq = seq0;
      s_run = run;
      p.marks[blockIdx.x] = mk;
    }
  }
  // the other warps bring the factors in meanwhile
  AttnFactors fq{nullptr, nullptr, 3}, fo{nullptr, nullptr, 3};
  if (p.qa) fq = attn_stage_factors(fac_q, p.qa, p.qb, p.nb, p.qls, static_cast<int>(threadIdx.x) - 32, attn::kThreads - 32);
  if (p.oa) fo = attn_stage_factors(fac_o, p.oa, p.ob, p.nb, p.ols, static_cast<int>(threadIdx.x) - 32, attn::kThreads - 32);
  __syncthreads();
  AttnPlace pl = s_place;
  int64_t left = s_run;
  if (left <= 0) return;
  AttnSeq seq = s_seq;
  const int hgs = p.head_units / p.Hkv;  // groups of kR heads of a KV head
  const int row_bytes = kFp8 ? p.D : p.D / 2;
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem) + warp * C::kWarpBytes;
  uint8_t* facs = ring + kS * C::kStageBytes;
  const uint32_t ring32 = smem_u32(ring);

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

    // ---- the warp's stream: a lane a token of its tiles
    int page_ahead = 0, off_ahead = -1;
    auto look = [&](int chunk, int& page, int& off) {
      const int i = chunk * attn::kChunk + 32 * warp + lane;
      off = -1;
      if (chunk >= last || i >= nv) return;
      const int j = span.token(i), pg = attn_page_of(p, j);
      page = __ldg(pages + pg);
      off = j - pg * p.page_size;
    };
    auto found = [&](int page, int off) -> int { return off >= 0 ? attn_row_at(p, page, off, h) : -1; };
    // two lanes copy 32 bytes of a token each time
    auto copy = [&](int row, int st) {
      const uint32_t kd = ring32 + st * C::kStageBytes + (lane >> 1) * C::kKs + (lane & 1) * 16;
      const uint32_t vd = ring32 + st * C::kStageBytes + C::kTok * C::kKs + (lane >> 1) * C::kVs + (lane & 1) * 16;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int rx = __shfl_sync(0xffffffffu, row, (lane >> 1) + 16 * x);
        const int64_t off = static_cast<int64_t>(max(rx, 0)) * row_bytes + (lane & 1) * 16;
        const uint8_t* ks = p.k_codes + off;
        const uint8_t* vs = p.v_codes + off;
#pragma unroll
        for (int k = 0; k < C::kBytes; k += 32) {
          // (a row of 16 bytes, one block of E2M1, has no second half)
          const bool in = kFp8 ? k < row_bytes : k + (lane & 1) * 16 < row_bytes;
          if (k > 0 && !(k < row_bytes)) break;
          attn_copy16(kd + 16 * x * C::kKs + k, in ? ks + k : p.k_codes, in && rx >= 0);
          attn_copy16(vd + 16 * x * C::kVs + k, in ? vs + k : p.v_codes, in && rx >= 0);
        }
      }
      attn_copy_commit();
    };
    // the lane's token's scale bytes, four a word
    constexpr int kW = (kNB + 3) / 4;
    uint32_t sck[kW], scv[kW];
    auto load_scales = [&](int row) {
      const int64_t at = static_cast<int64_t>(max(row, 0)) * p.nb;
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        sck[w] = scv[w] = 0u;
        if (row < 0) continue;
        if (p.scale_words) {
          if (4 * w < p.nb) {
            sck[w] = __ldg(reinterpret_cast<const uint32_t*>(p.k_scales + at) + w);
            scv[w] = __ldg(reinterpret_cast<const uint32_t*>(p.v_scales + at) + w);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (4 * w + k < p.nb) {
              sck[w] |= static_cast<uint32_t>(__ldg(p.k_scales + at + 4 * w + k)) << (8 * k);
              scv[w] |= static_cast<uint32_t>(__ldg(p.v_scales + at + 4 * w + k)) << (8 * k);
            }
        }
      }
    };
    auto put_scales = [&](int par) {
      float* fk = reinterpret_cast<float*>(facs + par * C::kFacBytes);
      uint16_t* fv = reinterpret_cast<uint16_t*>(fk + C::kTok * kNB);
      uint32_t* fe = reinterpret_cast<uint32_t*>(fv + C::kTok * kNB);
      uint32_t nan = 0u;  // a byte 255
#pragma unroll
      for (int w = 0; w < kW; ++w)
        nan |= (((sck[w] & 0x7F7F7F7Fu) + 0x01010101u) & sck[w]) | (((scv[w] & 0x7F7F7F7Fu) + 0x01010101u) & scv[w]);
      nan &= 0x80808080u;
      float kf[kNB];
      int top = 0, low = 255;
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        const int ek = (sck[b / 4] >> (8 * (b & 3))) & 255u, ev = (scv[b / 4] >> (8 * (b & 3))) & 255u;
        kf[b] = __uint_as_float(max(static_cast<uint32_t>(ek) << 23, 0x00400000u));  // (byte 0: 2^-127)
        top = max(top, ev);
        low = min(low, (ev - 1) & 255);  // (byte 0 last)
      }
      if (nan) {
        top = 0;
        for (int b = 0; b < kNB; ++b) {
          const int ev = (scv[b / 4] >> (8 * (b & 3))) & 255u;
          top = ev != 255 ? max(top, ev) : top;
        }
      }
      // tokens 2c, 2c + 1, 2c + 8, 2c + 9 of a half side by side
      const int at = (lane & 16) + (lane & 6) * 2 + (lane & 1) + ((lane >> 3) & 1) * 2;
#pragma unroll
      for (int b = 0; b < kNB; b += 2) {
        // 2^(e - top), by fp32 to f16 (which takes care of what is below its normal range)
        const int e0 = (scv[b / 4] >> (8 * (b & 3))) & 255u, e1 = (scv[b / 4] >> (8 * (b & 3) + 8)) & 255u;
        const float f0 = __uint_as_float(static_cast<uint32_t>(max(127 + e0 - top, 0)) << 23);
        const float f1 = __uint_as_float(static_cast<uint32_t>(max(127 + e1 - top, 0)) << 23);
        uint32_t f = attn_pack_f16(f0, f1);
        if (nan) {
          if (e0 == 255) f |= 0x7FFFu;
          if (e1 == 255) f |= 0x7FFF0000u;
          if (((sck[b / 4] >> (8 * (b & 3))) & 255u) == 255u) kf[b] = NAN;
          if (((sck[b / 4] >> (8 * (b & 3) + 8)) & 255u) == 255u) kf[b + 1] = NAN;
        }
        fv[b * 32 + at] = static_cast<uint16_t>(f);
        fv[(b + 1) * 32 + at] = static_cast<uint16_t>(f >> 16);
      }
#pragma unroll
      for (int b = 0; b < kNB; b += 2)
        *reinterpret_cast<float2*>(fk + lane * kNB + b) = make_float2(kf[b], kf[b + 1]);
      // E and the least e_b (blocks of scale byte 0, in practice all zeros, do not count; -inf where f16 does not
      // hold 2^(e_b - E))
      const float least = low == 255 ? INFINITY : (top - 1 - low > 24 ? -INFINITY : static_cast<float>(low - 126));
      fe[lane] = attn_pack(static_cast<float>(top - 127), least);
    };

    int rw[kS + 1];  // cache rows of tiles i .. i + kS - 1 of the warp, a token a lane
    {
      // the table's entries of all first tiles and the q rows are on their way together
      int page[kS], off[kS];
#pragma unroll
      for (int k = 0; k < kS; ++k) look(first + k, page[k], off[k]);
      look(first + kS, page_ahead, off_ahead);
      const int q_lines = (nrows * p.D * 2 + 127) / 128;
      if (static_cast<int>(threadIdx.x) < q_lines)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + tok * p.q_stride + static_cast<int64_t>(head0) * p.D + 64 * threadIdx.x));
#pragma unroll
      for (int k = 0; k < kS; ++k) rw[k] = found(page[k], off[k]);
    }
    load_scales(rw[0]);
#pragma unroll
    for (int k = 0; k < kS; ++k) copy(rw[k], k);

    // ---- q rows (times P_q) in fp32, then in f16 with the row's power of two
    for (int i = threadIdx.x; i < kR * kNB * 8; i += attn::kThreads) {
      const int q = i & 7, blk = (i >> 3) % kNB, n = (i >> 3) / kNB;
      const bool has = n < nrows && blk < p.nb;
      const uint16_t* src = p.q + tok * p.q_stride + static_cast<int64_t>(head0 + n) * p.D + 32 * blk;
      float* dst = sy + n * kLdo + 32 * blk;
      if (p.qa == nullptr) {
        const uint2 w = has ? *reinterpret_cast<const uint2*>(src + 4 * q) : make_uint2(0u, 0u);
        *reinterpret_cast<float4*>(dst + 4 * q) = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
      } else {
        float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (has) {
          float x[32];
          rows_load_block(src, x);
          attn_block_apply(fq, blk, x, q, y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[8 * j + q] = y[j];
      }
    }
    __syncthreads();
    for (int n = warp; n < kR; n += attn::kWarps) {
      float y[kDP / 32], mx = 0.0f;
#pragma unroll
      for (int k = 0; k < kDP / 64; ++k) {
        const float2 v = *reinterpret_cast<const float2*>(sy + n * kLdo + 64 * k + 2 * lane);
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
    // this lane's q operands: heads r (and r + 8), channels 8 c .. 8 c + 7 of every block; the
    // factors of its score columns
    uint32_t qf[kNT][kNB][4];
    float cs[kNT][2];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      cs[t][0] = sqf[8 * t + 2 * c];
      cs[t][1] = sqf[8 * t + 2 * c + 1];
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        const uint4 w = *reinterpret_cast<const uint4*>(sq + (8 * t + r) * kDP + 32 * b + 8 * c);
        qf[t][b][0] = w.x;
        qf[t][b][1] = w.y;
        qf[t][b][2] = w.z;
        qf[t][b][3] = w.w;
      }
    }
    put_scales(0);
    load_scales(rw[1]);

    // m: running reference of the scores, within 2^8 of the maximum (0 before anything is seen); mv = M - m
    // with M that of score + E, within 2^2 (-inf before). The scores x below are all relative to m, so that large
    // ones do not take E's bits.
    float m[kNT][2], mv[kNT][2], l[kNT][2], o[kNT][2 * kNB][4];
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      m[t][0] = m[t][1] = 0.0f;
      mv[t][0] = mv[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * kNB; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
    }

    int st = 0;
    for (int ch = first; ch < last; ++ch) {
      const int par = (ch - first) & 1;
      rw[kS] = found(page_ahead, off_ahead);
      look(ch + kS + 1, page_ahead, off_ahead);
      put_scales(par ^ 1);
      load_scales(rw[2]);
      attn_copy_wait<kS - 1>();
      __syncwarp();
      const uint8_t* kt = ring + st * C::kStageBytes;
      const uint8_t* vt = kt + C::kTok * C::kKs;
      const float* fk = reinterpret_cast<const float*>(facs + par * C::kFacBytes);
      const uint16_t* fv = reinterpret_cast<const uint16_t*>(fk + C::kTok * kNB);
      const uint32_t* fe = reinterpret_cast<const uint32_t*>(fv + C::kTok * kNB);
      // ---- S^T = K q^T for the tile's halves of 16 tokens, a block at a time
      float s[2][kNT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int t = 0; t < kNT; ++t) s[u][t][0] = s[u][t][1] = s[u][t][2] = s[u][t][3] = 0.0f;
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        if (b >= p.nb) break;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t a[2][4];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint8_t* src = kt + (16 * u + r + 8 * x) * C::kKs;
            if (kFp8) {
              const uint2 w = *reinterpret_cast<const uint2*>(src + 32 * b + 8 * c);
              attn_e4m3_f16(w.x, a[x][0], a[x][1]);
              attn_e4m3_f16(w.y, a[x][2], a[x][3]);
            } else {
              attn_e2m1_f16(*reinterpret_cast<const uint32_t*>(src + 16 * b + 4 * c), a[x]);
            }
          }
          const float k0 = fk[(16 * u + r) * kNB + b], k1 = fk[(16 * u + r + 8) * kNB + b];
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            attn_mma_f16(d, a[0][0], a[1][0], a[0][1], a[1][1], qf[t][b][0], qf[t][b][1]);
            attn_mma_f16(d, a[0][2], a[1][2], a[0][3], a[1][3], qf[t][b][2], qf[t][b][3]);
            s[u][t][0] = __fmaf_rn(d[0], k0, s[u][t][0]);
            s[u][t][1] = __fmaf_rn(d[1], k0, s[u][t][1]);
            s[u][t][2] = __fmaf_rn(d[2], k1, s[u][t][2]);
            s[u][t][3] = __fmaf_rn(d[3], k1, s[u][t][3]);
          }
        }
      }
      // ---- softmax over the tokens, for the columns 2c and 2c + 1
      const unsigned there = __ballot_sync(0xffffffffu, rw[0] >= 0);
      if (there == 0u) {  // (a NaN in q does not count then)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int t = 0; t < kNT; ++t) s[u][t][0] = s[u][t][1] = s[u][t][2] = s[u][t][3] = 0.0f;
      }
      // E, the least e_b (infinite for tokens that are not there), and 0 or -inf
      float e[2][2], el[2][2], bias[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w = fe[16 * u + 8 * k + r];
          e[u][k] = bf16lo(w);
          el[u][k] = bf16hi(w);
          bias[u][k] = there >> (16 * u + 8 * k + r) & 1u ? 0.0f : -INFINITY;
        }
      // A normal f16 factor needs x + E - mv + 13 - (E - e_b) >= -14.
      bool far[kNT][2], wide = false;  // columns that go the wide way; any of the warp's
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        float top[2], topv[2], low[2];
        const uint64_t cs2 = pack2(cs[t][0], cs[t][1]), m2 = pack2(-m[t][0], -m[t][1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // tokens r and r + 8 of the half, columns 2c and 2c + 1 side by side
          float xe[2][2], xl[2][2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float &x0 = s[u][t][2 * k], &x1 = s[u][t][2 * k + 1];
            // (the score is rounded first: the largest one less m is then 0 or exact, however large)
            const uint64_t x = fadd2(ffma2(pack2(x0, x1), cs2, pack2(bias[u][k], bias[u][k])), m2);
            unpack2(x, x0, x1);
            unpack2(fadd2(x, pack2(e[u][k], e[u][k])), xe[k][0], xe[k][1]);
            unpack2(fadd2(x, pack2(el[u][k], el[u][k])), xl[k][0], xl[k][1]);
          }
          // (-inf + inf, of a token that is not there, is NaN and passed over)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            top[k] = u ? attn_max3(top[k], s[u][t][k], s[u][t][2 + k]) : fmaxf(s[u][t][k], s[u][t][2 + k]);
            topv[k] = u ? attn_max3(topv[k], xe[0][k], xe[1][k]) : fmaxf(xe[0][k], xe[1][k]);
            low[k] = u ? attn_min3(low[k], xl[0][k], xl[1][k]) : fminf(xl[0][k], xl[1][k]);
          }
        }
        const bool up = top[0] > 8.0f || top[1] > 8.0f || topv[0] > mv[t][0] + 2.0f || topv[1] > mv[t][1] + 2.0f;
        far[t][0] = low[0] < mv[t][0] - 27.0f;
        far[t][1] = low[1] < mv[t][1] - 27.0f;
        if (__any_sync(0xffffffffu, up || far[t][0] || far[t][1])) {
          if (__any_sync(0xffffffffu, up)) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const bool first = mv[t][k] == -INFINITY;  // nothing seen yet
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], d));
              top[k] = fmaxf(top[k], first ? -INFINITY : 0.0f);
              const float mn = top[k] == -INFINITY ? m[t][k] : m[t][k] + top[k], by = mn - m[t][k];
              m[t][k] = mn;
              low[k] -= by;
              topv[k] = -INFINITY;
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  s[u][t][2 * x + k] -= by;
                  topv[k] = fmaxf(topv[k], s[u][t][2 * x + k] + e[u][x]);
                }
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) topv[k] = fmaxf(topv[k], __shfl_xor_sync(0xffffffffu, topv[k], d));
              topv[k] = fmaxf(mv[t][k] - by, topv[k]);
              l[t][k] *= first ? 1.0f : attn_exp2(-by);
              f[k] = first ? 1.0f : attn_exp2(mv[t][k] - by - topv[k]);
              mv[t][k] = topv[k];
            }
#pragma unroll
            for (int i = 0; i < 2 * kNB; ++i) {
              o[t][i][0] *= f[0];
              o[t][i][1] *= f[1];
              o[t][i][2] *= f[0];
              o[t][i][3] *= f[1];
            }
          }
          // (a column's way goes by its own scores and the tokens' scales, not by the other heads)
          const unsigned mine = 0x11111111u << c;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const unsigned any = __ballot_sync(0xffffffffu, low[k] < mv[t][k] - 27.0f);
            far[t][k] = (any & mine) != 0u;
            wide |= any != 0u;
          }
        }
      }
      // V of block b, half u of the tile, as f16: channel 4 r + k: tokens (2c, 2c + 1), (2c + 8, 2c + 9)
      auto load_v = [&](int b, int u, uint32_t (&v)[4][2]) {
        const uint8_t* src = vt + (16 * u + 2 * c) * C::kVs;
        if (kFp8) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w0 = *reinterpret_cast<const uint32_t*>(src + 8 * x * C::kVs + 32 * b + 4 * r);
            const uint32_t w1 = *reinterpret_cast<const uint32_t*>(src + (8 * x + 1) * C::kVs + 32 * b + 4 * r);
            attn_e4m3_f16(__byte_perm(w0, w1, 0x5140), v[0][x], v[1][x]);
            attn_e4m3_f16(__byte_perm(w0, w1, 0x7362), v[2][x], v[3][x]);
          }
        } else {
          // nibbles of the same channel side by side: even channels, odd channels
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = *reinterpret_cast<const uint16_t*>(src + ((x & 1) + 8 * (x >> 1)) * C::kVs + 16 * b + 2 * r);
          const uint32_t a = w[0] | w[2] << 16, d = w[1] | w[3] << 16;
          uint32_t ev[4], od[4];
          attn_e2m1_f16((a & 0x0F0F0F0Fu) | ((d << 4) & 0xF0F0F0F0u), ev);
          attn_e2m1_f16(((a >> 4) & 0x0F0F0F0Fu) | (d & 0xF0F0F0F0u), od);
          v[0][0] = ev[0];
          v[2][0] = ev[1];
          v[0][1] = ev[2];
          v[2][1] = ev[3];
          v[1][0] = od[0];
          v[3][0] = od[1];
          v[1][1] = od[2];
          v[3][1] = od[3];
        }
      };
      uint32_t pb[2][kNT][2];
#pragma unroll
      for (int t = 0; t < kNT; ++t) {
        float vs[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) vs[k] = far[t][k] ? INFINITY : (mv[t][k] == -INFINITY ? 0.0f : mv[t][k] - 13.0f);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          l[t][0] += attn_exp2(s[u][t][0]) + attn_exp2(s[u][t][2]);
          l[t][1] += attn_exp2(s[u][t][1]) + attn_exp2(s[u][t][3]);
          // weights up to 2^15 in f16 (off by half a step, 2^-11 of each); their sum l keeps fp32
          pb[u][t][0] = attn_transpose8(attn_pack_f16(attn_exp2(s[u][t][0] + (e[u][0] - vs[0])),
                                                      attn_exp2(s[u][t][1] + (e[u][0] - vs[1]))));
          pb[u][t][1] = attn_transpose8(attn_pack_f16(attn_exp2(s[u][t][2] + (e[u][1] - vs[0])),
                                                      attn_exp2(s[u][t][3] + (e[u][1] - vs[1]))));
        }
      }
      // ---- o^T += V^T P^T, a block at a time: lane r has channels 4 r .. 4 r + 3 of the block
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        if (b >= p.nb) break;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint2 f = *reinterpret_cast<const uint2*>(fv + b * 32 + 16 * u + 4 * c);
          uint32_t v[4][2];
          load_v(b, u, v);
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            const uint32_t q0 = attn_mul_f16x2(pb[u][t][0], f.x), q1 = attn_mul_f16x2(pb[u][t][1], f.y);
            attn_mma_f16(o[t][2 * b], v[0][0], v[1][0], v[0][1], v[1][1], q0, q1);
            attn_mma_f16(o[t][2 * b + 1], v[2][0], v[3][0], v[2][1], v[3][1], q0, q1);
          }
        }
      }
      if (__builtin_expect(wide, 0)) {
        // ---- the wide way, for the columns that take it (the others' weights are 0)
        uint32_t mine[kW];  // the token's V scales again
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          mine[w] = 0u;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (rw[0] >= 0 && 4 * w + k < p.nb)
              mine[w] |= static_cast<uint32_t>(__ldg(p.v_scales + static_cast<int64_t>(rw[0]) * p.nb + 4 * w + k)) << (8 * k);
        }
        int top = 0;
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
          const int ev = (mine[b / 4] >> (8 * (b & 3))) & 255u;
          top = ev != 255 ? max(top, ev) : top;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // top and scale bytes of this lane's four tokens
          int tt[4];
          uint32_t sv[4][kW];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int src = 16 * u + 2 * c + (x & 1) + 8 * (x >> 1);
            tt[x] = __shfl_sync(0xffffffffu, top, src);
#pragma unroll
            for (int w = 0; w < kW; ++w) sv[x][w] = __shfl_sync(0xffffffffu, mine[w], src);
          }
          uint32_t hi[kNT][2], lo[kNT][2];
#pragma unroll
          for (int t = 0; t < kNT; ++t) {
            float w[4], vs[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) vs[k] = far[t][k] ? mv[t][k] - 13.0f : INFINITY;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = attn_exp2(s[u][t][k] + (e[u][k >> 1] - vs[k & 1]));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t h = attn_pack(w[2 * x], w[2 * x + 1]);
              hi[t][x] = attn_transpose8(h);
              lo[t][x] = attn_transpose8(attn_pack(w[2 * x] - bf16lo(h), w[2 * x + 1] - bf16hi(h)));
            }
          }
#pragma unroll
          for (int b = 0; b < kNB; ++b) {
            if (b >= p.nb) break;
            uint32_t v[4][2], f[2];
            load_v(b, u, v);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t h[2];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int ev = (sv[2 * x + k][b / 4] >> (8 * (b & 3))) & 255u, d = tt[2 * x + k] - ev;
                h[k] = ev == 255 ? 0x7FFFu : static_cast<uint32_t>(max(127 - d, 0)) << 7;  // 2^-d
              }
              f[x] = h[0] | h[1] << 16;
#pragma unroll
              for (int k = 0; k < 4; ++k) v[k][x] = attn_f16_to_bf16(v[k][x]);
            }
#pragma unroll
            for (int t = 0; t < kNT; ++t)
#pragma unroll
              for (int g = 0; g < 2; ++g) {
                const uint32_t q0 = attn_mul_bf16x2(g ? lo[t][0] : hi[t][0], f[0]);
                const uint32_t q1 = attn_mul_bf16x2(g ? lo[t][1] : hi[t][1], f[1]);
                attn_mma_bf16(o[t][2 * b], v[0][0], v[1][0], v[0][1], v[1][1], q0, q1);
                attn_mma_bf16(o[t][2 * b + 1], v[2][0], v[3][0], v[2][1], v[3][1], q0, q1);
              }
          }
        }
      }
      __syncwarp();
      copy(rw[kS], st);
      if (++st == kS) st = 0;
#pragma unroll
      for (int k = 0; k < kS; ++k) rw[k] = rw[k + 1];
    }
    attn_copy_wait<0>();
    __syncthreads();  // the rings are free

    // ---- join the warps
#pragma unroll
    for (int t = 0; t < kNT; ++t) {
      float2 f[2];  // 2^(mv - 13)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][k] += __shfl_xor_sync(0xffffffffu, l[t][k], d);
        f[k] = mv[t][k] == -INFINITY ? make_float2(0.0f, 0.0f) : attn_exp2_two(mv[t][k] - 13.0f);
        if (r == 0) {
          float* ml = sml + (warp * kR + 8 * t + 2 * c + k) * 2;
          ml[0] = mv[t][k] == -INFINITY ? -INFINITY : m[t][k];
          ml[1] = l[t][k];
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * kNB; ++i) {
        // rows r and r + 8 of m-tile i are channels 32 (i / 2) + 4 r + 2 (i % 2) and the next
        const int d = 32 * (i >> 1) + 4 * r + 2 * (i & 1);
        float* o0 = so + (warp * kR + 8 * t + 2 * c) * kLdo + d;
        *reinterpret_cast<float2*>(o0) = make_float2(o[t][i][0] * f[0].x * f[0].y, o[t][i][2] * f[0].x * f[0].y);
        *reinterpret_cast<float2*>(o0 + kLdo) = make_float2(o[t][i][1] * f[1].x * f[1].y, o[t][i][3] * f[1].x * f[1].y);
      }
    }
    __syncthreads();
    const bool whole = first == 0 && last == pl.chunks;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (seg == 0 ? 0 : 1);
    float* dst = whole ? sy : p.part_o + static_cast<int64_t>(slot) * kR * p.D;
    const int ldd = whole ? kLdo : p.D;
    float* dml = whole ? fml : p.part_ml + static_cast<int64_t>(slot) * kR * 2;
    const int quads = p.D >> 2;
    for (int i = threadIdx.x; i < nrows * quads; i += attn::kThreads) {
      const int n = i / quads, d = 4 * (i - n * quads);
      float mm = -INFINITY, sum = 0.0f;
      float2 f[attn::kWarps];
#pragma unroll
      for (int w = 0; w < attn::kWarps; ++w) mm = fmaxf(mm, sml[(w * kR + n) * 2]);
#pragma unroll
      for (int w = 0; w < attn::kWarps; ++w) {
        const float2 ml = *reinterpret_cast<const float2*>(sml + (w * kR + n) * 2);
        f[w] = ml.x == -INFINITY ? make_float2(0.0f, 0.0f) : attn_exp2_two(ml.x - mm);
        sum = ml.y != ml.y ? NAN : __fmaf_rn(ml.y * f[w].x, f[w].y, sum);  // (a NaN stays: NaN * f + anything)
      }
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < attn::kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(so + (w * kR + n) * kLdo + d);
        acc.x = __fmaf_rn(v.x * f[w].x, f[w].y, acc.x);
        acc.y = __fmaf_rn(v.y * f[w].x, f[w].y, acc.y);
        acc.z = __fmaf_rn(v.z * f[w].x, f[w].y, acc.z);
        acc.w = __fmaf_rn(v.w * f[w].x, f[w].y, acc.w);
      }
      if (whole) {
        const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
        acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (p.oa == nullptr)
          *reinterpret_cast<uint2*>(p.out + (tok * p.Hq + head0 + n) * p.D + d) =
              make_uint2(attn_pack(acc.x, acc.y), attn_pack(acc.z, acc.w));
        if (p.lse && d == 0)
          p.lse[tok * p.Hq + head0 + n] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * 0.69314718055994531f;
      } else if (d == 0) {
        dml[2 * n] = mm;
        dml[2 * n + 1] = sum;
      }
      if (!whole || p.oa != nullptr) *reinterpret_cast<float4*>(dst + n * ldd + d) = acc;
    }
    if (whole && p.oa != nullptr) {
      __syncthreads();
      for (int i = threadIdx.x; i < nrows * p.nb * 8; i += attn::kThreads) {
        const int q = i & 7, blk = (i >> 3) % p.nb, n = (i >> 3) / p.nb;
        float y[4];
        attn_block_apply(fo, blk, sy + n * kLdo + 32 * blk, q, y);
        uint16_t* out = p.out + (tok * p.Hq + head0 + n) * p.D + 32 * blk + q;
#pragma unroll
        for (int j = 0; j < 4; ++j) out[8 * j] = __bfloat16_as_ushort(__float2bfloat16_rn(y[j]));
      }
    }
    __syncthreads();
    left -= last - first;
    if (left > 0) attn_next_unit<0>(p, pl, seq);
  }
}

// ---------------------------------------------------------------- joining partial results
// CTA (x, y): if CTA x + 1's run begins inside a unit, and no earlier run does, the parts
// of that unit (the last of CTA x, then the first of x + 1, x + 2, ...) are joined here, a warp a row
// for the row kernel's units, four rows a warp at a time for the tile kernel's (their parts on
// their way together). kTile as in the kernel that wrote them. Bound:
// the parts' bytes from L2, or latency.
template <int kTile>
struct AttnJoin {
  static constexpr int kRows = kTile ? 4 : 1;
};
template <int kTile>
__global__ void __launch_bounds__(256) bat_attn_join_kernel(const AttnParams p) {
  extern __shared__ __align__(16) float smem[];
  constexpr int kR = AttnJoin<kTile>::kRows;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i1 = blockIdx.x + 1;
  float* so = smem + warp * (kR * 260);  // [kR][260]: this warp's rows, when P_o is applied
  AttnFactors fo{nullptr, nullptr, 3};
  if (p.oa) fo = attn_stage_factors(smem + 8 * kR * 260, p.oa, p.ob, p.nb, p.ols, threadIdx.x, blockDim.x);
  __syncthreads();
  grid_dependency_wait();
  allow_dependents();
  const AttnMark mk = p.marks[i1];
  const int64_t total = mk.total, x = mk.x;
  if (x >= total) return;
  const AttnPlace pl = mk.place;
  const AttnDeal deal(total, p.ctas);
  const int64_t u0 = x - pl.chunk, u1 = u0 + pl.chunks;
  if (pl.chunk == 0 || deal.start(i1 - 1) > u0) return;  // no split here, or an earlier CTA's
  int end = i1 + 1;  // parts of CTAs [i1 - 1, end)
  while (end < p.ctas && deal.start(end) < u1) ++end;
  const int rows = p.unit_rows;
  const AttnSeq seq = attn_seq(p, pl.b);
  const int hgs = p.head_units / p.Hkv;
  const int h = pl.hu / hgs, hg = pl.hu - h * hgs;
  // rows of the unit that are there
  const int64_t there = kTile ? static_cast<int64_t>(seq.n) * p.G - static_cast<int64_t>(pl.tile) * kTile
                              : p.G - hg * rows;
  const int nrows = static_cast<int>(there < rows ? there : rows);
  const int quads = p.D >> 2;  // float4 a row: this lane's are lane and lane + 32
  for (int r0 = (blockIdx.y * 8 + warp) * kR; r0 < nrows; r0 += gridDim.y * 8 * kR) {
    // running over the parts in order: maximum, sum and o, as in the kernels
    float mm[kR], sum[kR];
    float4 acc[kR][2];
    bool bad[kR];
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      mm[k] = -INFINITY;
      sum[k] = 0.0f;
      bad[k] = false;
      acc[k][0] = acc[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
#pragma unroll kR == 1 ? 4 : 1
    for (int i = i1 - 1; i < end; ++i) {
      const int64_t xi = deal.start(i);
      if (xi >= deal.start(i + 1)) continue;  // an empty run
      // the unit is the first of CTA i's run if the run begins inside the unit (or at it)
      const int64_t at = (2 * static_cast<int64_t>(i) + (xi >= u0 ? 0 : 1)) * rows;
      float2 ml[kR];
      float4 v[kR][2];
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const int64_t row = at + min(r0 + k, nrows - 1);
        ml[k] = *reinterpret_cast<const float2*>(p.part_ml + 2 * row);
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (lane + 32 * g < quads) v[k][g] = *(reinterpret_cast<const float4*>(p.part_o + row * p.D) + lane + 32 * g);
      }
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        bad[k] |= ml[k].y != ml[k].y;
        if (ml[k].x == -INFINITY) continue;  // saw nothing
        const float mn = fmaxf(mm[k], ml[k].x);
        const float2 f0 = mm[k] == -INFINITY ? make_float2(0.0f, 0.0f) : attn_exp2_two(mm[k] - mn);
        const float2 f1 = attn_exp2_two(ml[k].x - mn);
        mm[k] = mn;
        sum[k] = sum[k] * f0.x * f0.y + ml[k].y * f1.x * f1.y;
#pragma unroll
        for (int g = 0; g < 2; ++g)
          if (lane + 32 * g < quads) {
            acc[k][g].x = acc[k][g].x * f0.x * f0.y + v[k][g].x * f1.x * f1.y;
            acc[k][g].y = acc[k][g].y * f0.x * f0.y + v[k][g].y * f1.x * f1.y;
            acc[k][g].z = acc[k][g].z * f0.x * f0.y + v[k][g].z * f1.x * f1.y;
            acc[k][g].w = acc[k][g].w * f0.x * f0.y + v[k][g].w * f1.x * f1.y;
          }
      }
    }
#pragma unroll
    for (int k = 0; k < kR; ++k) {
      if (r0 + k >= nrows) break;
      int64_t tok;
      int head;
      if (kTile) {
        const int64_t row = static_cast<int64_t>(pl.tile) * kTile + r0 + k;
        const int64_t t = row / p.G;
        tok = seq.t0 + t;
        head = h * p.G + static_cast<int>(row - t * p.G);
      } else {
        tok = seq.t0 + pl.tile;
        head = h * p.G + hg * rows + r0 + k;
      }
      const float l = bad[k] ? NAN : sum[k];
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
      uint16_t* dst = p.out + (tok * p.Hq + head) * p.D;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int q = lane + 32 * g;
        if (q >= quads) break;
        const float4 y = make_float4(acc[k][g].x * inv, acc[k][g].y * inv, acc[k][g].z * inv, acc[k][g].w * inv);
        if (p.oa != nullptr)
          *reinterpret_cast<float4*>(so + k * 260 + 4 * q) = y;
        else
          *reinterpret_cast<uint2*>(dst + 4 * q) = make_uint2(attn_pack(y.x, y.y), attn_pack(y.z, y.w));
      }
      if (p.oa != nullptr) {
        __syncwarp();
        for (int i = lane; i < p.nb * 8; i += 32) {
          float y[4];
          attn_block_apply(fo, i >> 3, so + k * 260 + 32 * (i >> 3), i & 7, y);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dst[32 * (i >> 3) + 8 * j + (i & 7)] = __bfloat16_as_ushort(__float2bfloat16_rn(y[j]));
        }
        __syncwarp();
      }
      if (p.lse && lane == 0)
        p.lse[tok * p.Hq + head] = l == 0.0f ? -INFINITY : (mm[k] + log2f(l)) * 0.69314718055994531f;
    }
  }
}

}  // namespace bat
