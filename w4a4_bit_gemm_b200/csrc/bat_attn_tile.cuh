// Attention of chunks of new tokens over the paged MXFP8 / MXFP4 cache on the 5th-generation
// tensor cores (see bat_attn.cuh for the operator, the work split and the partial results).
//
// A unit is 256 query rows (two tiles of 128; one for heads wider than 128 channels) of one
// KV head: rows run over tokens and the group's heads, so grouped heads share every K and V
// tile. Its visible tokens come in chunks of 128. Warp roles:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one row a thread: S from TMEM, weights back into
//                   S's columns as the A operand of the second product; q staging and the output
//   warps 8-15      K and V: page lookup, loads of codes and scales a chunk ahead, expansion
//                   to f16 (K) and bf16 (V) in swizzled shared memory
//   warp 16         issues the MMAs and owns TMEM
// Per chunk and tile: S = q K^T (M 128, N 128, K = D, kind::f16 on f16) and
// o += P V (N = D, K = 128, kind::f16 on bf16, P from TMEM). The MMAs of one tile run while the
// other tile's warps are in their softmax. The maximum is lazy: o is rescaled only when the
// row's maximum grew by more than 2^8, which bf16 weights and fp32 sums hold without loss.
// What bounds it: the tensor pipe and the exponentials' unit about equally (a chunk of 256
// rows: 2048 cycles of MMA at the nominal rate, 2048 cycles of 16 exponentials a cycle).
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
constexpr int kThreads = 640;  // 17 warps work; the register split goes by four warps
constexpr int kRegsSoftmax = 120, kRegsLoad = 104, kRegsMma = 32;
static_assert(2 * kRegsSoftmax + 2 * kRegsLoad + kRegsMma <= 5 * 96, "the split stays within the launch's registers");
constexpr int kInfo = 8;                // chunks whose notes are kept (see the ring's order)

template <int kDP>
struct Cfg {
  static constexpr int kTiles = kDP <= 128 ? 2 : 1;   // tiles of 128 rows a unit
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kPanels = kDP / 64;
  static constexpr int kStageBytes = kPanels * kPanelBytes;
  static constexpr int kStages = kDP == 64 ? 8 : (kDP == 128 ? 4 : 2);
  static constexpr int kQBytes = kTiles * kPanels * kPanelBytes;
  static constexpr int kSmem = 1024 + kQBytes + kStages * kStageBytes;  // dynamic, 1024 for alignment
};
}  // namespace attn_tile

// What the loader notes about a chunk for the softmax warps.
struct AttnNote {
  float kfac;         // 2^(largest K scale of the chunk)
  int any;            // some token is hidden (bad page) or holds a NaN in V
  uint32_t tok[128];  // bit 31: hidden; bit b: NaN in V's block b
};

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
// Loader warps only: a barrier of their 256 threads that also agrees on `ok`, so that all of them
// leave together after a wait that ran out.
__device__ __forceinline__ bool attn_load_sync(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}

// Channel order that the expansion of V leaves (see attn_e4m3_bits, attn_e2m1_bits): position
// i of an 8-channel group holds channel attn_v_order(i).
template <bool kFp8>
__host__ __device__ constexpr int attn_v_order(int i) {
  return kFp8 ? (i & ~3) | ((i & 1) << 1) | ((i >> 1) & 1) : (i & ~7) | ((i >> 1) & 3) | ((i & 1) << 2);
}

// Rows of q P_q in f16 with their factors, for units that many tiles share: warp a row.
struct AttnQRowsParams {
  const uint16_t* q;
  int64_t q_stride;
  const float* a;
  const float* b;
  uint16_t* out;   // f16 [T][Hq][D]
  float* fac;      // [T][Hq]
  int64_t rows;    // T * Hq
  int Hq, D, nb, ls;
  float sign, scale_log2;
};
__global__ void __launch_bounds__(256) bat_attn_q_rows_kernel(const AttnQRowsParams p) {
  __shared__ __align__(16) float sp[8 * 1024];
  __shared__ __align__(16) float fac[kv::kFacFloats];
  allow_dependents();
  kv_build_p(sp, fac, p.a, p.b, p.nb, p.ls);
  const int lane = threadIdx.x & 31, u = lane & 7;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); row < p.rows; row += step) {
    const int64_t t = row / p.Hq;
    const uint16_t* src = p.q + t * p.q_stride + (row - t * p.Hq) * p.D;
    float y[2][4], mx = 0.0f;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int blk = 4 * g + (lane >> 3);
      const bool has = blk < p.nb;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (has) {
        const uint2 w = *reinterpret_cast<const uint2*>(src + 32 * blk + 4 * u);
        x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
      }
      y[g][0] = y[g][1] = y[g][2] = y[g][3] = 0.0f;
      if (4 * g < p.nb) kv_block_product(sp + (has ? blk : 0) * 1024, x, lane, y[g]);
      if (!has) y[g][0] = y[g][1] = y[g][2] = y[g][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) mx = fmaxf(mx, fabsf(y[g][j]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    float down;
    const float up = attn_row_up(mx, down) * p.sign;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int blk = 4 * g + (lane >> 3);
      if (blk < p.nb)
        *reinterpret_cast<uint2*>(p.out + row * p.D + 32 * blk + 4 * u) =
            make_uint2(attn_pack_f16(y[g][0] * up, y[g][1] * up), attn_pack_f16(y[g][2] * up, y[g][3] * up));
    }
    if (lane == 0) p.fac[row] = down * p.scale_log2;
  }
}

// A run of chunks, unit after unit.
template <int kTile>
struct AttnRun {
  AttnPlace pl;
  AttnSeq seq;
  AttnSpan span;
  int nv;
  int64_t left;  // chunks, this one among them
  __device__ __forceinline__ void enter(const AttnParams& p) {
    span = attn_tile_span<kTile>(p, seq, pl.tile);
    nv = span.count();
  }
  __device__ __forceinline__ void start(const AttnParams& p, const AttnPlace& place, int64_t n) {
    pl = place;
    left = n;
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
    const int64_t n = pl.chunks - pl.chunk;
    return static_cast<int>(n < left ? n : left);
  }
  // tiles of 128 rows that hold rows
  __device__ __forceinline__ int tiles(const AttnParams& p) const {
    return static_cast<int64_t>(seq.n) * p.G - static_cast<int64_t>(pl.tile) * kTile > 128 ? kTile / 128 : 1;
  }
};

template <bool kFp8, int kDP>
__global__ void __launch_bounds__(attn_tile::kThreads, 1) bat_attn_tile_kernel(const AttnParams p) {
  using C = attn_tile::Cfg<kDP>;
  constexpr int kTile = C::kRows, kStages = C::kStages;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ AttnNote notes[attn_tile::kInfo];
  __shared__ int s_rows[2][128];
  __shared__ uint8_t s_scale[2][2][128][kDP / 32];
  __shared__ int s_top[2][4];
  __shared__ uint32_t s_nan[C::kRows][kDP / 32];  // written only where a NaN was seen
  __shared__ __align__(16) float s_oa[64];
  __shared__ __align__(16) float s_ob[kDP / 32 * 16];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 2 * 4 + 1];
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
  const uint32_t drain = bars + 8 * (2 * kStages + 8);

  allow_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), attn_tile::kLoadWarps);
      mbar_init(empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 4);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t), 4);
      mbar_init(o_full(t), 1);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  if (warp == 15) {
    int64_t n;
    const AttnMark mk = attn_mark<kTile>(p, blockIdx.x, lane, n);
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
    bool ok = t < C::kTiles;
    grid_dependency_wait();  // the transformed q rows, where a kernel before this one writes them
    for (int seg = 0; ok && run.left > 0; ++seg) {
      const int n = run.chunks_here();
      if (t >= run.tiles(p)) {
        run.next_unit(p, n);
        n_c += n;
        continue;
      }
      const int64_t row = static_cast<int64_t>(run.pl.tile) * kTile + 128 * t + rr;
      const int64_t rt = row / p.G;
      const bool valid = rt < run.seq.n;
      const int64_t tok = run.seq.t0 + rt;
      const int head = run.pl.hu * p.G + static_cast<int>(row - rt * p.G);
      const int base = run.seq.len - run.seq.n;
      const int pos = valid ? base + static_cast<int>(rt) : -1;
      // ---- q row to shared memory (read twice: for its largest channel, and converted)
      float cs = 0.0f;
      {
        const uint32_t qrow = q_base + (t * C::kPanels) * attn_tile::kPanelBytes + rr * 128;
        const bool ready = p.qt != nullptr;
        const uint4* src = reinterpret_cast<const uint4*>(
            ready ? p.qt + (tok * p.Hq + head) * p.D : p.q + tok * p.q_stride + static_cast<int64_t>(head) * p.D);
        float up = 1.0f;
        if (!ready) {
          float mx = 0.0f;
#pragma unroll 8
          for (int v = 0; v < kDP / 8; ++v) {
            const uint4 w = valid && 8 * v < p.D ? __ldg(src + v) : make_uint4(0u, 0u, 0u, 0u);
            const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(e[k])), fabsf(bf16hi(e[k]))));
          }
          float down;
          up = attn_row_up(mx, down) * p.q_sign;
          cs = down * p.scale_log2;
        } else if (valid) {
          cs = __ldg(p.qt_fac + tok * p.Hq + head);
        }
#pragma unroll 8
        for (int v = 0; v < kDP / 8; ++v) {
          uint4 w = valid && 8 * v < p.D ? __ldg(src + v) : make_uint4(0u, 0u, 0u, 0u);
          if (!ready) {
            w.x = attn_pack_f16(bf16lo(w.x) * up, bf16hi(w.x) * up);
            w.y = attn_pack_f16(bf16lo(w.y) * up, bf16hi(w.y) * up);
            w.z = attn_pack_f16(bf16lo(w.z) * up, bf16hi(w.z) * up);
            w.w = attn_pack_f16(bf16lo(w.w) * up, bf16hi(w.w) * up);
          }
          const uint32_t a = qrow + (v >> 3) * attn_tile::kPanelBytes + (((v & 7) ^ (rr & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(t));

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
        if (i > 0 && *reinterpret_cast<volatile int*>(&notes[(n_c - 1) % attn_tile::kInfo].any)) see_nan(n_c - 1, chunk - 1);
        const AttnNote& note = notes[n_c % attn_tile::kInfo];
        const float cc = fmaxf(cs * note.kfac, 1e-37f);
        const int i0 = chunk * 128;
        // masked columns go to TMEM as -inf, so that the two passes below need no test (S is read
        // twice, 32 columns at a time, instead of being held: 120 registers a thread do)
        const bool whole = (i0 >= all_lo || i0 + 128 <= sp.ns) && i0 + 128 <= all_hi;
        const bool hidden = *reinterpret_cast<const volatile int*>(&note.any) != 0;
        if (!whole || hidden) {
          const int c_hi = v_hi - i0, c_lo = v_lo - i0, c_sink = v_sink - i0;
#pragma unroll 1
          for (int k = 0; k < 128; k += 32) {
            uint32_t s[32];
            tmem_ld_32x32b_x32(s_col(t) + lane_base + k, s);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int c = k + j;
              if (!(c < c_hi && (c >= c_lo || c < c_sink))) s[j] = 0xFF800000u;
              if (hidden && (note.tok[c] >> 31)) s[j] = 0xFF800000u;
            }
            tmem_st_32x32b_x16(s_col(t) + lane_base + k, reinterpret_cast<const uint32_t(&)[16]>(s[0]));
            tmem_st_32x32b_x16(s_col(t) + lane_base + k + 16, reinterpret_cast<const uint32_t(&)[16]>(s[16]));
          }
          tmem_wait_st();
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 32) {
          uint32_t s[32];
          tmem_ld_32x32b_x32(s_col(t) + lane_base + k, s);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[0]) : "f"(__uint_as_float(s[j])), "f"(__uint_as_float(s[j + 1])));
            asm("max.f32 %0, %0, %1, %2;" : "+f"(mx[1]) : "f"(__uint_as_float(s[j + 2])), "f"(__uint_as_float(s[j + 3])));
          }
        }
        const float mn = fmaxf(mx[0], mx[1]) * cc;
        if (i == 0) {
          m = mn;
        } else {
          const bool grow = mn > m + 8.0f;
          if (__any_sync(0xffffffffu, grow)) {
            // o of the chunks before: all their MMAs are done
            ok = __all_sync(0xffffffffu, mbar_wait(o_full(t), (n_s - 1) & 1u, kErrWaitTmemFull));
            if (!ok) break;
            tc_fence_after();
            const float al = grow ? attn_exp2(m - mn) : 1.0f;
            if (grow) m = mn;
            l0 *= al;
            l1 *= al;
            for (int d = 0; d < p.D; d += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_col(t) + lane_base + d, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
              tmem_st_32x32b_x16(o_col(t) + lane_base + d, reinterpret_cast<const uint32_t(&)[16]>(o[0]));
              tmem_st_32x32b_x16(o_col(t) + lane_base + d + 16, reinterpret_cast<const uint32_t(&)[16]>(o[16]));
            }
          }
        }
        const float ms = m == -INFINITY ? 0.0f : m;
        const uint64_t c2 = pack2(cc, cc), m2 = pack2(-ms, -ms);
        uint64_t sum2 = pack2(l0, l1);
        // weights over the columns already read: S's columns 32 k .. give way to 16 k ..
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t s[32], w[16];
          tmem_ld_32x32b_x32(s_col(t) + lane_base + 32 * k, s);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a, b;
            unpack2(ffma2(pack2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), c2, m2), a, b);
            a = attn_exp2(a);
            b = attn_exp2(b);
            sum2 = fadd2(sum2, pack2(a, b));
            w[j] = attn_pack(a, b);  // bf16: off by half a step 2^-8 of each weight, unbiased
          }
          tmem_st_32x32b_x16(s_col(t) + lane_base + 16 * k, w);
        }
        unpack2(sum2, l0, l1);
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
      if (*reinterpret_cast<volatile int*>(&notes[(n_c - 1) % attn_tile::kInfo].any)) see_nan(n_c - 1, run.pl.chunk + n - 1);
      const float l = l0 + l1;
      const bool part = !(run.pl.chunk == 0 && n == run.pl.chunks);
      const int64_t prow = (2 * static_cast<int64_t>(blockIdx.x) + (seg == 0 ? 0 : 1)) * kTile + 128 * t + rr;
      const float inv = l > 0.0f ? attn::kUp / l : (l == 0.0f ? 0.0f : l);
      for (int b = 0; b < p.nb; ++b) {
        uint32_t o[32];
        tmem_ld_32x32b_x32(o_col(t) + lane_base + 32 * b, o);
        tmem_wait_ld();
        float v[32];
        const float f = part ? attn::kUp : inv;
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
          p.part_ml[2 * prow] = m;
          p.part_ml[2 * prow + 1] = l;
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
    const int lw = warp - 8, tid = threadIdx.x - 256;
    const int my_tok = tid & 127, my_kv = tid >> 7;      // token and side (K or V) of this thread's lookups
    const int row_bytes = kFp8 ? p.D : p.D / 2;
    // the lanes of a quarter-warp take the pieces of one panel of neighbouring tokens, so that
    // their 16-byte stores fall on different banks of the swizzled rows
    constexpr int kPp = kFp8 ? 4 : 2;  // pieces a panel
    const int piece = ((lane >> 3) % C::kPanels) * kPp + lane % kPp;
    const int sub = (lane >> 3) / C::kPanels * (8 / kPp) + lane % 8 / kPp;
    const bool has = piece * 16 < row_bytes;
    const int pblk = kFp8 ? piece >> 1 : piece;          // its 32-channel block
    const uint8_t* my_scales = my_kv ? p.v_scales : p.k_scales;
    bool ok = true;
    uint4 buf[2][kBatch];

    // this thread's token of the chunk the run stands at: its offset in the page (-1: none), the table's entry
    int off_ahead = -1, h_ahead = 0, page_ahead = 0;
    auto look = [&]() {
      off_ahead = -1;
      if (run.left <= 0) return;
      const int idx = run.pl.chunk * 128 + my_tok;
      if (idx >= run.nv) return;
      const int j = run.span.token(idx), pg = attn_page_of(p, j);
      h_ahead = run.pl.hu;
      page_ahead = __ldg(p.table + static_cast<int64_t>(run.pl.b) * p.max_pages + pg);
      off_ahead = j - pg * p.page_size;
    };
    auto found = [&](bool& bad) -> int {
      const int r = off_ahead >= 0 ? attn_row_at(p, page_ahead, off_ahead, h_ahead) : -1;
      bad = off_ahead >= 0 && r < 0;
      return r;
    };
    uint32_t sc[kDP / 32];
    auto load_scales = [&](int row) {
#pragma unroll
      for (int b = 0; b < kDP / 32; ++b)
        sc[b] = row >= 0 && b < p.nb ? __ldg(my_scales + static_cast<int64_t>(row) * p.nb + b) : 0u;
    };
    // scales, the largest of K's, and the notes of chunk c (parity c & 1), before a barrier
    auto publish = [&](uint32_t c, bool bad) {
      int top = 0;
#pragma unroll
      for (int b = 0; b < kDP / 32; ++b) {
        s_scale[c & 1][my_kv][my_tok][b] = static_cast<uint8_t>(sc[b]);
        // NaN scales stand for themselves and do not set the common scale
        if (sc[b] != 255u) top = max(top, static_cast<int>(sc[b]));
      }
      if (my_kv == 0) {
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) s_top[c & 1][lw] = top;
        AttnNote& nt = notes[c % attn_tile::kInfo];
        nt.tok[my_tok] = bad ? 0x80000000u : 0u;
        if (tid == 0) nt.any = 0;
      }
    };
    auto load_batch = [&](int par, const uint8_t* codes, int b, uint4 (&dst)[kBatch]) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int row = s_rows[par][16 * lw + (b * kBatch + k) * kTpi + sub];
        dst[k] = row >= 0 && has
                     ? __ldg(reinterpret_cast<const uint4*>(codes + static_cast<int64_t>(row) * row_bytes) + piece)
                     : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    constexpr int kX = kFp8 ? 8 : 16;  // words a piece expands to
    auto put = [&](uint32_t stage, int tk, const uint32_t (&x)[kX]) {
      if (!has) return;
#pragma unroll
      for (int u = 0; u < kX / 4; ++u) {
        const int unit = kX / 4 * piece + u;  // 8-channel group of the token's row
        const uint32_t at = stage + (unit >> 3) * attn_tile::kPanelBytes + tk * 128 + (((unit & 7) ^ (tk & 7)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[4 * u]), "r"(x[4 * u + 1]),
                     "r"(x[4 * u + 2]), "r"(x[4 * u + 3])
                     : "memory");
      }
    };

    bool bad_now = false, bad_next = false;
    {
      look();
      const int row = found(bad_now);
      run.next_chunk(p);
      look();
      if (my_kv == 0) s_rows[0][my_tok] = row;
      load_scales(row);
      publish(0, bad_now);
      ok = attn_load_sync(true);
      load_batch(0, p.k_codes, 0, buf[0]);
      if (kNB == 2)
        load_batch(0, p.k_codes, kNB - 1, buf[1]);
      else
        load_batch(0, p.v_codes, 0, buf[1]);
    }
    const int64_t total = s_run;
    uint32_t el = 0;  // tiles put so far (K and V in turn)
    for (int64_t c64 = 0; ok && c64 < total; ++c64) {
      const uint32_t c = static_cast<uint32_t>(c64);
      const int par = c & 1;
      // rows and scales of the next chunk, the table's entries of the one after
      const int row_next = found(bad_next);
      if (my_kv == 0) s_rows[par ^ 1][my_tok] = row_next;
      load_scales(row_next);
      run.next_chunk(p);
      look();
      if (!(ok = attn_load_sync(ok))) break;

      const int top = max(max(s_top[par][0], s_top[par][1]), max(s_top[par][2], s_top[par][3]));
      AttnNote& note = notes[c % attn_tile::kInfo];
      if (tid == 0) note.kfac = attn_scale_value(top);
      if (bad_now && my_kv == 0) note.any = 1;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++el) {
        const uint32_t sidx = el % kStages;
        const uint32_t stage = st_base + sidx * C::kStageBytes;
        ok = mbar_wait(empty(sidx), ((el / kStages) & 1u) ^ 1u, kErrWaitEmpty) && ok;
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
          constexpr int kSeq = 2 * kNB;
          const int e = kv * kNB + b;
          uint4(&src)[kBatch] = buf[e & 1];
          uint32_t nan = 0u;  // some byte's bit 7: a NaN among the batch's V codes
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int tk = 16 * lw + (b * kBatch + k) * kTpi + sub;
            const uint32_t w[4] = {src[k].x, src[k].y, src[k].z, src[k].w};
            const uint32_t sb = has ? s_scale[par][kv][tk][pblk] : 0u;
            uint32_t x[kX];
            if (kv == 0) {
              const uint32_t f = sb == 255u ? 0x7E007E00u : attn_f16_pow2(top - static_cast<int>(sb));
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
              const uint32_t f = attn_scale_pair<kFp8>(sb);
              if ((f & 0x7FFFu) == 0x7FFFu) nan = 0x80u;
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
            put(stage, tk, x);
          }
          if (kv == 1 && (nan & 0x80808080u) != 0u) {
            // the rare way round: the pieces with a NaN again, with 0 in its place, and a note
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int tk = 16 * lw + (b * kBatch + k) * kTpi + sub;
              const uint32_t w[4] = {src[k].x, src[k].y, src[k].z, src[k].w};
              const uint32_t f = attn_scale_pair<kFp8>(has ? s_scale[par][1][tk][pblk] : 0u);
              const bool all = (f & 0x7FFFu) == 0x7FFFu;
              uint32_t x[kX], any = 0u;
#pragma unroll
              for (int q = 0; q < kX; ++q) x[q] = 0u;
              if (kFp8 && !all) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  const uint32_t z = attn_e4m3_nan(w[q]) & 0x80808080u;
                  any |= z;
                  x[2 * q] = attn_mul_bf16x2(attn_e4m3_bits(w[q] << 8), f) &
                             ((z & 0x80u ? 0u : 0xFFFFu) | (z & 0x800000u ? 0u : 0xFFFF0000u));
                  x[2 * q + 1] = attn_mul_bf16x2(attn_e4m3_bits(w[q]), f) &
                                 ((z & 0x8000u ? 0u : 0xFFFFu) | (z & 0x80000000u ? 0u : 0xFFFF0000u));
                }
              }
              if (any != 0u || all) {
                put(stage, tk, x);
                atomicOr(&note.tok[tk], 1u << pblk);
                note.any = 1;
              }
            }
          }
          // the batch two steps on
          const int e2 = e + 2;
          const int nxt = e2 >= kSeq ? 1 : 0, e3 = nxt ? e2 - kSeq : e2;
          load_batch(par ^ nxt, e3 < kNB ? p.k_codes : p.v_codes, e3 % kNB, src);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full(sidx));
      }
      publish(c + 1, bad_next);
      bad_now = bad_next;
      if (!(ok = attn_load_sync(ok))) break;
    }
  } else {
    // ================================================================ MMA
    setmaxnreg_dec<attn_tile::kRegsMma>();
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
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
}

}  // namespace bat
