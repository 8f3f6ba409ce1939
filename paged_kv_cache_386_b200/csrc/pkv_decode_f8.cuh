// pkv_decode_f8.cuh -- decode attention over the FP8 cache (e4m3 codes, one
// scale for each block, kv head and K or V).
//
// Work.  A tile is one (block, kv head): K and V codes, 32 D contiguous
// bytes.  A segment is the context of one sequence for up to 16 rows (query,
// head) of one kv head.  The tiles of all segments in order are cut into equal
// ranges, one per warp ("unit"); W consecutive units are a CTA's.  Each warp
// copies its own tiles, one TMA box each, a ring ahead of their use.
// Nothing waits for another CTA: a segment that several warps of one CTA
// share is merged in shared memory when the CTA is done, one that several CTAs
// share by the CTA that finishes it last (a counter per CTA where such a
// segment starts), always in the order of the context, so that the bits do
// not depend on which CTA that is.
//
// Arithmetic of a warp's step, two tiles (32 tokens) of one segment.  With s_K,
// s_V a block's scales and e = floor(log2 s_V), f = s_V 2^-e:
//   S^T = K Q^T            mma m16n8k16 f16: 16 tokens x 8 rows, codes as f16
//                          (exact), Q as f16 (exact; bf16 rows are first scaled
//                          by a power of two), fp32 sums
//   y   = S s_K c + e - m  c = scale log2(e), m the row's reference
//   O^T += V^T (2^y f)^T   16 dims x 8 rows, codes as f16, weights as f16
//   l   += 2^y 2^-e
// so that a block's V scale costs one addition in the exponent, weights are
// largest where p V is, and out = O / l.  The reference m is 2^7 below the
// largest p s_V seen and moves only when a weight would pass 2^14: a vote per
// step, a reduction over tokens when it moves (at a segment's first tiles),
// and weights keep f16's full precision down to 2^-21 of the largest.  With
// f16 data the rounding of the weights (2^-11 at most) is as large as that of
// the output, so their remainders take a second product.  With bf16 data it is an
// eighth of the output's (2^-8): outputs next to a tie may round the other way, but
// the error against 64 bits is the same with remainders and without (0.0017 of the
// norm), and remainders cost 3, 7 and 4 % (64 mixed lengths 56.2 -> 58.0 us, 32 x 4
// queries 41.4 -> 44.1, 4 x 131072 184.2 -> 192.1).
//
// Rows on the n side of the product halve the products for 8 rows or fewer
// (16 MMAs for a tile of 16 x 128 K and V, not 32) and the accumulators.
#pragma once

#include "pkv_append_f8.cuh"
#include "pkv_prefix_tc.cuh"

namespace pkv {

// Tiles under way on an SM.  More only lengthens the memory's queues: 256 mixed
// lengths, 32/32 heads of 128: 223 us with 192 KiB, 214 with 128; 4 x 131072: 175,
// 168.5; heads of 64: 36.5, 36.1 (37.9 with 64); 16 rows: 42.0, 41.5 (44.9 with 64).
constexpr int kF8RingBytes = 128 * 1024;
// Slots that make a unit worth its merge (one sequence of 4096 tokens, 32/8 heads:
// 14.7 us with 1, 13.6 with 2, 16.7 with 4).
constexpr int kF8MinSlots = 2;
// A segment's fixed work, in tiles.  Measured with none: the slowest warp of 256
// mixed lengths of 1 to 1300 tokens, 32/32 heads, ended 25% after the mean (263 us,
// 216 with two); with 16 rows, seven against two: 46.4 -> 42.8 us (32 x 4 queries).
__host__ __device__ constexpr int f8_seg_slots(int NR) { return NR == 1 ? 2 : 7; }
// Warps of a CTA with up to 8 rows a segment, and with up to 16: as many as their
// registers allow (128 and 255 a thread).  8 rows, 64 mixed lengths: 58.0 us with
// 12 warps, 57.6 with 16; 4 x 131072: 186, 178.  16 rows, 32 x 4 queries: 42.1 with
// 8, 44.9 with 12.
constexpr int kF8W1 = 16, kF8W2 = 8;
constexpr int kF8HeaderBytes = 4096;                  // workspace: the arrivals at each CTA's segment, 8 bytes
constexpr float kF8RefBelow = 7.f, kF8RefSlack = 14.f;

struct DecodeF8Params {
  const uint16_t* q;  // [batch][q_len][n_q][D], f16 or bf16
  uint16_t* out;
  const float2* scales;  // [num_blocks][n_kv]
  const int32_t* block_tables;
  const int32_t* context_lens;
  // [CTAs]: the CTAs done with the segment that starts in that one and goes on behind
  // it.  Each adds `arrival`: 1 in the bits from 48 on, below them a number that differs
  // from call to call, so that a word the workspace held before is told from arrivals
  // (f8_settle).  0 again after a launch.
  unsigned long long* arrivals;
  unsigned long long arrival;
  float* unit_recs;        // [units][rec_floats]: a segment that ends inside a unit and began before it
  float* cta_recs;         // [CTAs][2][rec_floats]: the CTA's share of a segment from before it, of one that goes on
  int32_t max_blocks_per_seq, batch, num_blocks, n_q_heads, n_kv_heads, q_len;
  int32_t group;       // query heads per kv head
  int32_t total_rows;  // group * q_len rows of a kv head: row i is query i / group, head i % group
  int32_t rows;        // rows of a segment (the last one of a kv head may have fewer)
  int32_t nseg;        // segments of a kv head
  int32_t ng;          // segments of a sequence, n_kv * nseg
  int32_t rec_floats;  // rows * (D + 4)
  float scale_log2;
  // Test hook: the first tile is never copied of the unit that runs the start of this
  // one's share (itself, or the next one where its range is empty); -1: none.
  int32_t withhold_unit;
  uint64_t wait_limit_ns;
};

// 3-D box of one tile: D bytes x 32 rows (16 of K, 16 of V) of one (block, kv head).
__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, uint64_t* bar, int c2,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(0), "r"(c2), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ void cp_async_8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// One arrival on `bar` (counted in its initial count) when this thread's cp.asyncs so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Two 16 x 16 byte matrices, transposed: lane (g, t) = (lane / 4, lane % 4)
// holds bytes 4 t .. 4 t + 3 (rows) of columns g (r0) and g + 8 (r1), then of
// the second matrix (r2, r3).  Lane l gives row l % 16 of matrix l / 16.
__device__ __forceinline__ void ldsm_b8_x2_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                                 uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// Adds `x`, ordered on both sides at gpu scope (for the CTA, between two of its barriers).
__device__ __forceinline__ unsigned long long add_acq_rel(unsigned long long* at, unsigned long long x) {
  unsigned long long r;
  asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], %2;" : "=l"(r) : "l"(at), "l"(x) : "memory");
  return r;
}

__device__ __forceinline__ unsigned long long load_relaxed(const unsigned long long* at) {
  unsigned long long r;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(r) : "l"(at) : "memory");
  return r;
}

// Sets a word of the arrivals to 0 unless it holds some of this call's n already
// (j `arrival`, j < n).  `word` is what it held when last read.  Every CTA does this
// in front of its own arrival, so that none is counted on top of, or lost with, what
// was there before the call: a workspace needs no clearing.
__device__ __forceinline__ void f8_settle(unsigned long long* at, unsigned long long word, unsigned long long arrival,
                                          int n) {
  while (true) {
    const unsigned long long j = word >> 48;
    if (j < static_cast<unsigned long long>(n) && word == j * arrival) return;
    const unsigned long long now = atomicCAS(at, word, 0ull);
    if (now == word) return;
    word = now;  // another CTA of the call has settled it, or arrived
  }
}

// 8 x 8 transpose of packed 16-bit pairs: lane (g, t) holds row g, columns 2 t, 2 t + 1 before and after.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Element offset in q and out of row `i` (of the kv head's total_rows).
__device__ __forceinline__ size_t f8_row_at(const DecodeF8Params& p, int b, int kvh, int i, int D) {
  const int qi = i / p.group;
  return ((static_cast<size_t>(b) * p.q_len + qi) * p.n_q_heads + kvh * p.group + (i - qi * p.group)) * D;
}

// 16-byte chunk c of token row `tok` in a swizzled tile (128-byte rows: c ^
// row % 8; 64-byte rows: c ^ (row / 2) % 4, the 64-byte swizzle).
template <int D>
__device__ __forceinline__ uint32_t f8_chunk_at(int tok, int c) {
  return static_cast<uint32_t>(tok * D + (D == 128 ? c ^ (tok & 7) : c ^ ((tok >> 1) & 3)) * 16);
}

// Token of row g of a tile's S^T product (k-index g of P V), and of row g + 8
// (4 further); with matrix row i of V at token f8_v_token(i), lane (g, t)'s
// four V bytes are the tokens of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9.  Eight
// successive rows of either are eight rows of the swizzle, so that no read
// conflicts.
__device__ __forceinline__ int f8_k_token(int g) { return (g & 3) + 8 * (g >> 2); }
__device__ __forceinline__ int f8_v_token(int i) { return f8_k_token(2 * (i >> 2) + (i & 1)) + 2 * (i & 2); }

// Four codes to two packed half pairs (exact).
__device__ __forceinline__ void f8_unpack4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}

// A step's tiles: shared-memory address and scales; a dead one (behind the
// segment or the unit, or of a bad block id) adds nothing.
struct F8Step {
  uint32_t base[2];
  float ks[2], vs[2];
  bool dead[2];
  int rem;  // context tokens from the first tile's first on
};

template <int D, int NR, bool kBf16>
struct F8Consumer {
  static constexpr bool kRest = !kBf16;  // P's rounding to f16 is followed by its remainder
  static constexpr int KS = D / 16;      // k-steps of S
  static constexpr int MT = D / 16;      // 16-dim tiles of O
  static constexpr int RS = D + 4;       // floats of a record's row: O, m, l, and padding against bank conflicts
  uint32_t qb[NR][KS][2];
  float o[NR][MT][4];                  // dims 16 mt + g (+ 8), rows 8 nr + 2 t (+ 1)
  float m[NR][2], l[NR][2], c[NR][2];  // reference, sum over this lane's tokens, factor of s_K, of those rows
  int hide[NR][2];                     // tokens at the context's end that the row does not see

  __device__ __forceinline__ void begin(const DecodeF8Params& p, const uint8_t* qbuf, int first_row, int rows,
                                        int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int DL = D / 4;  // consecutive dims of a lane: k-step kk takes 4 of them, K alike
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      const int row = 8 * nr + g;
      uint32_t w[DL / 2];
      const uint4* src = reinterpret_cast<const uint4*>(qbuf + row * D * 2 + t * DL * 2);
#pragma unroll
      for (int i = 0; i < DL / 8; ++i) {
        const uint4 v = row < rows ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
      float cs = p.scale_log2;
      if constexpr (kBf16) {
        // The row's largest magnitude to [2^13, 2^14): what is more than 2^28
        // times smaller keeps fewer bits.
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < DL / 2; ++i) {
          float lo, hi;
          unpack2<true>(w[i], lo, hi);
          mx = fmaxf(mx, fmaxf(fabsf(lo), fabsf(hi)));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 127);
        // 2^(13 - e) as two factors that are both in range.
        const int up = 13 - e, u1 = up / 2, u2 = up - u1;
        const float f1 = __uint_as_float((u1 + 127) << 23), f2 = __uint_as_float((u2 + 127) << 23);
#pragma unroll
        for (int i = 0; i < DL / 2; ++i) {
          float lo, hi;
          unpack2<true>(w[i], lo, hi);
          w[i] = pack2<false>(lo * f1 * f2, hi * f1 * f2);
        }
        cs = p.scale_log2 * __uint_as_float((127 - u1) << 23) * __uint_as_float((127 - u2) << 23);
      }
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) qb[nr][kk][0] = w[2 * kk], qb[nr][kk][1] = w[2 * kk + 1];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        c[nr][r] = __shfl_sync(0xffffffffu, cs, (2 * t + r) * 4);
        hide[nr][r] = p.q_len - 1 - (first_row + 8 * nr + 2 * t + r) / p.group;
        m[nr][r] = -INFINITY;
        l[nr][r] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) o[nr][i][0] = o[nr][i][1] = o[nr][i][2] = o[nr][i][3] = 0.f;
    }
  }

  __device__ __forceinline__ void step(const F8Step& st, int q_len, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int tok = f8_k_token(g);

    float s[2][NR][4], y[2][NR][4], a[2][NR][2], fe[2], f[2], inv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < NR * 4; ++i) s[h][i >> 2][i & 3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        uint32_t ka[4], kb[4];
        lds128(st.base[h] + f8_chunk_at<D>(tok, D / 64 * t + i), ka);
        lds128(st.base[h] + f8_chunk_at<D>(tok + 4, D / 64 * t + i), kb);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a0, a1, a2, a3;
          f8_unpack4(ka[w], a0, a2);
          f8_unpack4(kb[w], a1, a3);
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
            mma_16816<false>(s[h][nr], a0, a1, a2, a3, qb[nr][4 * i + w][0], qb[nr][4 * i + w][1]);
        }
      }
      // s_V = f 2^e.
      const uint32_t vbits = __float_as_uint(st.vs[h]);
      const int e = static_cast<int>(vbits >> 23) - 127;
      fe[h] = static_cast<float>(e);
      f[h] = __uint_as_float((vbits & 0x7fffffu) | 0x3f800000u);
      inv[h] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        a[h][nr][0] = st.ks[h] * c[nr][0];
        a[h][nr][1] = st.ks[h] * c[nr][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[h][nr][i] = fmaf(s[h][nr][i], a[h][nr][i & 1], fe[h] - m[nr][i & 1]);
      }
    }
    // Tokens that some row does not see: the context's last q_len - 1, and dead tiles.
    const bool edge = st.dead[0] || st.dead[1] || st.rem - (q_len - 1) < 2 * kBlockTokens;
    auto hidden = [&](int h, int nr, int i) {
      return st.dead[h] || 16 * h + tok + 2 * (i & 2) >= st.rem - hide[nr][i & 1];
    };
    if (edge) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (hidden(h, nr, i)) y[h][nr][i] = s[h][nr][i] = -INFINITY;
    }
    bool far = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int i = 0; i < 4; ++i) far = far || y[h][nr][i] > kF8RefSlack;
    if (__any_sync(0xffffffffu, far)) {
      // Where a row's largest grew by more than the slack: a new reference.
      // (A hidden score is -inf; times a negative factor it would not be.)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = r; i < 4; i += 2)
              if (s[h][nr][i] != -INFINITY) mx = fmaxf(mx, fmaf(s[h][nr][i], a[h][nr][r], fe[h]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          if (mx > m[nr][r] + kF8RefSlack) {
            const float ref = mx - kF8RefBelow;
            const float alpha = m[nr][r] == -INFINITY ? 0.f : exp2f(m[nr][r] - ref);
            m[nr][r] = ref;
            l[nr][r] *= alpha;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nr][i][r] *= alpha;
              o[nr][i][2 + r] *= alpha;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = r; i < 4; i += 2)
                y[h][nr][i] = s[h][nr][i] == -INFINITY ? -INFINITY : fmaf(s[h][nr][i], a[h][nr][r], fe[h] - ref);
          }
        }
    }

    uint32_t ph[2][NR][2], pl[2][NR][2];  // the weights as b operands, and their remainders
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[h][nr][i] = ex2_ftz(y[h][nr][i]);
        l[nr][0] = fmaf(y[h][nr][0] + y[h][nr][2], inv[h], l[nr][0]);
        l[nr][1] = fmaf(y[h][nr][1] + y[h][nr][3], inv[h], l[nr][1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float p0 = y[h][nr][2 * k] * f[h], p1 = y[h][nr][2 * k + 1] * f[h];
          const uint32_t hi = pack2<false>(p0, p1);
          ph[h][nr][k] = transpose_8x8(hi);
          if constexpr (kRest) {
            float h0, h1;
            unpack2<false>(hi, h0, h1);
            pl[h][nr][k] = transpose_8x8(pack2<false>(p0 - h0, p1 - h1));
          }
        }
      }

    const uint32_t v0 = st.base[0] + kBlockTokens * D, v1 = st.base[1] + kBlockTokens * D;
    if (edge) {
      clear_behind(v0, st.dead[0] ? 0 : st.rem, lane);
      if (v1 != v0) clear_behind(v1, st.dead[1] ? 0 : st.rem - kBlockTokens, lane);
      __syncwarp();
      if (q_len > 1)
        for (int i = max(0, st.rem - q_len + 1); i < min(2 * kBlockTokens, st.rem); ++i)
          if (!st.dead[i >> 4]) nan_of_token(i < kBlockTokens ? v0 : v1, i, st.rem, lane);
      // The next copy into the slot comes after these writes.
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    pv(v0, ph[0], pl[0], lane);
    pv(v1, ph[1], pl[1], lane);
  }

  // V rows behind the context (from token n on) may hold anything: zeros.
  __device__ __forceinline__ static void clear_behind(uint32_t v, int n, int lane) {
    for (int i = max(n, 0) * (D / 16) + lane; i < kBlockTokens * (D / 16); i += 32)
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + i * 16), "r"(0u) : "memory");
  }

  // Several queries: a NaN value of token `i` (of the step), which some rows
  // do not see, would reach them as 0 x NaN.  It is taken out and put into
  // the rows that see it.
  __device__ __forceinline__ void nan_of_token(uint32_t v, int i, int rem, int lane) {
    const int g = lane >> 2, tok = i & 15;
    uint32_t w;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(v + tok * D + (lane % (D / 4)) * 4) : "memory");
    if (!__any_sync(0xffffffffu, (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0)) return;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint32_t at = v + f8_chunk_at<D>(tok, mt) + g;
      uint32_t c0, c1;
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(c0) : "r"(at) : "memory");
      asm volatile("ld.shared.u8 %0, [%1];" : "=r"(c1) : "r"(at + 8) : "memory");
      __syncwarp();
      if ((c0 & 0x7f) == 0x7f) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(0u) : "memory");
      if ((c1 & 0x7f) == 0x7f) asm volatile("st.shared.u8 [%0], %1;" ::"r"(at + 8), "r"(0u) : "memory");
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (i < rem - hide[nr][r]) {
            if ((c0 & 0x7f) == 0x7f) o[nr][mt][r] = __int_as_float(0x7fc00000);
            if ((c1 & 0x7f) == 0x7f) o[nr][mt][2 + r] = __int_as_float(0x7fc00000);
          }
    }
    __syncwarp();
  }

  // O^T += V^T P^T of one tile.
  __device__ __forceinline__ void pv(uint32_t v, const uint32_t (&ph)[NR][2], const uint32_t (&pl)[NR][2], int lane) {
    const int vt = f8_v_token(lane & 15), vc = lane >> 4;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t r[4];
      ldsm_b8_x2_trans(v + f8_chunk_at<D>(vt, 2 * i + vc), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a0, a1, a2, a3;
        f8_unpack4(r[2 * h], a0, a2);
        f8_unpack4(r[2 * h + 1], a1, a3);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          mma_16816<false>(o[nr][2 * i + h], a0, a1, a2, a3, ph[nr][0], ph[nr][1]);
          if constexpr (kRest) mma_16816<false>(o[nr][2 * i + h], a0, a1, a2, a3, pl[nr][0], pl[nr][1]);
        }
      }
    }
  }

  // The rows' state as a record, or (rec null) their output.
  __device__ __forceinline__ void finish(const DecodeF8Params& p, float* rec, int b, int kvh, int first_row, int rows,
                                         int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[nr][r];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = 8 * nr + 2 * t + r;
        if (row >= rows) continue;
        if (rec != nullptr) {
          float* at = rec + row * RS;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            at[16 * i + g] = o[nr][i][r];
            at[16 * i + 8 + g] = o[nr][i][2 + r];
          }
          if (g == 0) {
            at[D] = m[nr][r];
            at[D + 1] = sum;
          }
        } else {
          // A sum of 0 is a row with no token (bad block ids): zeros.  NaN stays NaN.
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          uint16_t* at = p.out + f8_row_at(p, b, kvh, first_row + row, D);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const float x = o[nr][i][r] * inv, z = o[nr][i][2 + r] * inv;
            const uint32_t w = pack2<kBf16>(x, z);
            at[16 * i + g] = static_cast<uint16_t>(w);
            at[16 * i + 8 + g] = static_cast<uint16_t>(w >> 16);
          }
        }
      }
  }
};

// The n pieces of a segment, in the order of the context: `first`, then base + j
// stride, and `last` for piece n - 1 where it lies elsewhere (else null).
struct F8Pieces {
  const float* first;
  const float* base;
  const float* last;
  int stride;  // floats
  int n;
};

// Pieces merged by a warp, online over a few of them at a time whose loads go
// out together:
//   M = max m_i,  w_i = 2^(m_i - M),  O = sum w_i O_i,  l = sum w_i l_i.
// Eight lanes hold a row (D / 8 dims each).  kSplit false: rows row .. row + 3
// at once, where pieces are few; true: row `row` alone, each group of lanes over
// every fourth piece, then the groups' states combined, where they are many.
// Written to the record `to`, or normalised to the output.  The pieces are in
// shared memory or were written by any SM: generic loads at gpu scope.
template <int D, bool kBf16, bool kSplit>
__device__ __noinline__ void f8_merge(const DecodeF8Params& p, const F8Pieces pc, int row, int rows, float* to, int b,
                                      int kvh, int first_row) {
  constexpr int DL = D / 8, RS = D + 4, kStep = kSplit ? 4 : 1, kBatch = 2;
  const int lane = threadIdx.x & 31, group = lane >> 3, dim = (lane & 7) * DL;
  if (!kSplit) row += group;
  const bool live = row < rows;
  const int at = (live ? row : 0) * RS;
  float M = -INFINITY, L = 0.f, acc[DL];
#pragma unroll
  for (int i = 0; i < DL; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int j0 = kSplit ? group : 0; j0 < pc.n; j0 += kBatch * kStep) {
    float mj[kBatch], lj[kBatch], o[kBatch][DL];
#pragma unroll
    for (int jj = 0; jj < kBatch; ++jj) {
      const int j = j0 + jj * kStep;  // predicated loads: no branch between them
      const int is = j < pc.n;
      const float* r = at + (j == 0 ? pc.first : j == pc.n - 1 && pc.last != nullptr ? pc.last : pc.base + j * static_cast<int64_t>(pc.stride));
      mj[jj] = -INFINITY;
      lj[jj] = 0.f;
      asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %3, 0;\n @p ld.relaxed.gpu.v2.f32 {%0, %1}, [%2];\n}"
                   : "+f"(mj[jj]), "+f"(lj[jj])
                   : "l"(r + D), "r"(is));
#pragma unroll
      for (int i = 0; i < DL; i += 4) {
        o[jj][i] = o[jj][i + 1] = o[jj][i + 2] = o[jj][i + 3] = 0.f;
        asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %5, 0;\n @p ld.relaxed.gpu.v4.f32 {%0, %1, %2, %3}, [%4];\n}"
                     : "+f"(o[jj][i]), "+f"(o[jj][i + 1]), "+f"(o[jj][i + 2]), "+f"(o[jj][i + 3])
                     : "l"(r + dim + i), "r"(is));
      }
    }
    // -inf: no token seen so far; those pieces' sums are 0 (or NaN, which stays).
    float Mb = M;
#pragma unroll
    for (int jj = 0; jj < kBatch; ++jj) Mb = fmaxf(Mb, mj[jj]);
    const float alpha = M == -INFINITY ? 1.f : exp2f(M - Mb);
    L *= alpha;
#pragma unroll
    for (int i = 0; i < DL; ++i) acc[i] *= alpha;
#pragma unroll
    for (int jj = 0; jj < kBatch; ++jj) {
      const float w = mj[jj] == -INFINITY ? 1.f : exp2f(mj[jj] - Mb);
      L = fmaf(w, lj[jj], L);
#pragma unroll
      for (int i = 0; i < DL; ++i) acc[i] = fmaf(w, o[jj][i], acc[i]);
    }
    M = Mb;
  }
  if constexpr (kSplit) {
#pragma unroll
    for (int x = 8; x < 32; x *= 2) {
      const float Mb = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float w = M == -INFINITY ? 1.f : exp2f(M - Mb);
      L *= w;
      L += __shfl_xor_sync(0xffffffffu, L, x);
#pragma unroll
      for (int i = 0; i < DL; ++i) {
        acc[i] *= w;
        acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], x);
      }
      M = Mb;
    }
  }
  if (!live || (kSplit && group > 0)) return;
  if (to != nullptr) {
    to += at;
#pragma unroll
    for (int i = 0; i < DL; i += 4)
      *reinterpret_cast<float4*>(to + dim + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
    if (dim == 0) *reinterpret_cast<float2*>(to + D) = make_float2(M, L);
    return;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint16_t* out = p.out + f8_row_at(p, b, kvh, first_row + row, D) + dim;
#pragma unroll
  for (int i = 0; i < DL; i += 4)
    *reinterpret_cast<uint2*>(out + i) = make_uint2(pack2<kBf16>(acc[i] * inv, acc[i + 1] * inv),
                                                    pack2<kBf16>(acc[i + 2] * inv, acc[i + 3] * inv));
}

// Work is counted in slots: a segment has f8_seg_slots for its start and end (Q,
// the first maxima, the output), then one for each tile.  A unit's range of
// slots begins at its share of them, or at the segment's first slot where that
// share begins before the segment's second tile.
struct F8Walk {
  int b, hg;   // segment
  int st, nb;  // its first slot, its tiles
  int j;       // tile
};

// The segment of slot k.
template <int kSeg>
__device__ __forceinline__ F8Walk f8_find(const int* prefix, const int* ctxs, int B, int k) {
  int lo = 0, hi = B;  // prefix[lo] <= k < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= k) lo = mid; else hi = mid;
  }
  F8Walk w;
  w.b = lo;
  w.nb = (ctxs[lo] + kBlockTokens - 1) / kBlockTokens;
  const int local = k - prefix[lo];
  w.hg = local / (w.nb + kSeg);
  w.st = k - local + w.hg * (w.nb + kSeg);
  w.j = max(0, k - w.st - kSeg);
  return w;
}

template <int kSeg>
__device__ __forceinline__ void f8_next_segment(F8Walk& w, const int* prefix, const int* ctxs, int B, int ng) {
  w.st += w.nb + kSeg;
  w.j = 0;
  if (++w.hg == ng) {
    w.hg = 0;
    do {
      ++w.b;
    } while (w.b < B && prefix[w.b + 1] == prefix[w.b]);
    w.nb = w.b < B ? (ctxs[w.b] + kBlockTokens - 1) / kBlockTokens : 0;
  }
}

// Where unit u's slots begin, and (but for the end of all) the tile there.
template <int kSeg>
__device__ __forceinline__ int f8_unit_begin(const Sched& sc, int u, const int* prefix, const int* ctxs, int B,
                                             F8Walk* at) {
  const int k = unit_begin(sc, u);
  if (u >= sc.U) return k;
  const F8Walk w = f8_find<kSeg>(prefix, ctxs, B, k);
  *at = w;
  return w.j == 0 ? w.st : k;
}

// Rows of a segment that this CTA holds in several units, or shares with other CTAs.
struct F8Group {
  int b, hg, st, en;  // the segment's slots [st, en)
  int ua, ub;         // first and last unit of this CTA with a piece of it
  int c0, n_ctas;     // its CTAs: the one of its first tile, how many
  int kvh, first, rows;
};

// The CTA's segments with a share in several units or CTAs, in order: of the
// candidates that one comes from before the CTA, and one starts in each unit and
// goes on behind it.  By one warp, while the first copies are under way.
template <int W, int kSeg>
__device__ __noinline__ void f8_find_groups(const DecodeF8Params& p, const Sched sc, int per_cta, int u0, int n_units,
                                            const int* bnd, const int* prefix, const int* ctxs, F8Group* groups,
                                            int* n_groups) {
  static_assert(W < 32, "a lane for each candidate");
  const int lane = threadIdx.x & 31, A = bnd[0], E = bnd[n_units];
  bool valid = false;
  F8Group gr;
  if (lane <= n_units && A < E) {
    const int w = max(0, lane - 1), k = lane == 0 ? A : bnd[w + 1] - 1;
    const F8Walk f = f8_find<kSeg>(prefix, ctxs, p.batch, k);
    gr.b = f.b;
    gr.hg = f.hg;
    gr.st = f.st;
    gr.en = f.st + f.nb + kSeg;
    valid = lane == 0 ? gr.st < A : bnd[w] < bnd[w + 1] && gr.st >= bnd[w] && gr.en > bnd[w + 1];
    const int last = unit_of_tile(sc, gr.en - 1);
    gr.ua = w;
    gr.ub = min(last - u0, n_units - 1);
    if (lane == 0)  // units in front of the first tile have no piece
      while (bnd[gr.ua + 1] == A) ++gr.ua;
    gr.c0 = unit_of_tile(sc, gr.st + kSeg) / per_cta;
    gr.n_ctas = last / per_cta - gr.c0 + 1;
    gr.kvh = gr.hg / p.nseg;
    gr.first = (gr.hg - gr.kvh * p.nseg) * p.rows;
    gr.rows = min(p.rows, p.total_rows - gr.first);
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, valid);
  if (valid) groups[__popc(mask & ((1u << lane) - 1u))] = gr;
  if (lane == 0) *n_groups = __popc(mask);
}

// Warps of a CTA, each a unit.
__host__ __device__ constexpr int f8_warps(int NR) { return NR == 1 ? kF8W1 : kF8W2; }

// Ring slots of a warp (2 to 8).
__host__ __device__ constexpr int f8_stages(int D, int NR) { return kF8RingBytes / (f8_warps(NR) * f8_tile_bytes(D)); }

// Shared memory: each warp's ring, its Q rows, a barrier, a scale pair and a flag of each ring slot; lengths.
__host__ __device__ constexpr size_t f8_smem_bytes(int D, int NR, int rows, int batch) {
  return 1024 + kF8RingBytes + static_cast<size_t>(f8_warps(NR)) * (f8_stages(D, NR) * 20 + rows * D * 2) + 16 +
         (2 * static_cast<size_t>(batch) + 1) * 4;
}

template <int D, int NR, bool kBf16>
__global__ void __launch_bounds__(f8_warps(NR) * 32, 1)
    pkv_decode_f8_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ DecodeF8Params p) {
  constexpr int kTile = f8_tile_bytes(D);
  constexpr int W = f8_warps(NR), kThreads = W * 32, kSeg = f8_seg_slots(NR);
  using Consumer = F8Consumer<D, NR, kBf16>;
  constexpr int RS = Consumer::RS;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* rings = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  constexpr int S = f8_stages(D, NR), n_slots = W * S;
  static_assert(S >= 2 && S * kTile >= 8 * NR * RS * 4, "a step's tiles, and a record, in a warp's ring");
  static_assert(n_slots <= kThreads, "a thread for each barrier's set-up");
  const int q_bytes = p.rows * D * 2;
  uint8_t* qbufs = rings + static_cast<size_t>(n_slots) * kTile;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(qbufs + W * q_bytes);  // [W][S]: the slot's copies have landed
  float2* slot_scale = reinterpret_cast<float2*>(full_bar + n_slots);
  int* slot_bad = reinterpret_cast<int*>(slot_scale + n_slots);
  volatile int* abort_flag = slot_bad + n_slots;
  int* prefix = const_cast<int*>(abort_flag) + 4;  // [batch + 1]: slots before each sequence
  int* ctxs = prefix + p.batch + 1;                // [batch]
  __shared__ int warp_sums[W];
  __shared__ int bnd[W + 1];  // where this CTA's units begin, and the tiles there
  __shared__ F8Walk starts[W + 1];
  __shared__ F8Group groups[W + 1];
  __shared__ int n_groups;
  __shared__ int last_of[2];  // this CTA finishes: the segment from before it, the one that goes on behind it

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = p.batch;

  if (threadIdx.x < n_slots) {
    mbar_init(&full_bar[threadIdx.x], 2);  // the codes' bytes, and the scales
    mbar_fence_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    tma_prefetch_desc(&tm);
  }
  wait_for_kernel_before();

  {
    const int per = (B + kThreads - 1) / kThreads;
    const int lo = min(B, static_cast<int>(threadIdx.x) * per), hi = min(B, lo + per);
    const int max_ctx = p.max_blocks_per_seq * kBlockTokens;
    auto slots_of = [&](int c) { return c > 0 ? ((c + kBlockTokens - 1) / kBlockTokens + kSeg) * p.ng : 0; };
    int local = 0;
    for (int b = lo; b < hi; ++b) {
      const int c0 = p.context_lens[b];
      int c = clamp_ctx(c0, max_ctx);
      if (c > 0 && c < p.q_len) c = 0;
      if (c != c0) flag_error(PKV_DEVERR_CONTEXT);
      ctxs[b] = c;
      local += slots_of(c);
    }
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += v;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sums[w];
    int run = base + incl - local;
    for (int b = lo; b < hi; ++b) {
      prefix[b] = run;
      run += slots_of(ctxs[b]);
    }
    if (threadIdx.x == kThreads - 1) prefix[B] = base + incl;
  }
  __syncthreads();

  // Sequences without a token: zeros.
  for (int b = blockIdx.x; b < B; b += gridDim.x)
    if (ctxs[b] == 0) {
      uint4* at = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(b) * p.q_len * p.n_q_heads * D);
      const int n = p.q_len * p.n_q_heads * (D / 8);
      for (int i = threadIdx.x; i < n; i += kThreads) at[i] = make_uint4(0u, 0u, 0u, 0u);
    }

  const int T = prefix[B];
  const Sched sc = make_sched(T, min(static_cast<int>(gridDim.x) * W, max(1, T / kF8MinSlots)), 0, 1000);
  // A small problem's units go over all CTAs, fewer to each.
  const int per_cta = (sc.U + gridDim.x - 1) / static_cast<int>(gridDim.x);
  const int u0 = blockIdx.x * per_cta, n_units = min(sc.U - u0, per_cta);  // this CTA's units
  if (T == 0 || n_units <= 0) return;
  if (threadIdx.x <= n_units)
    bnd[threadIdx.x] = f8_unit_begin<kSeg>(sc, u0 + threadIdx.x, prefix, ctxs, B, &starts[threadIdx.x]);
  __syncthreads();

  // Rows of segment hg of a sequence: kv head, first of its rows, how many.
  auto seg_rows = [&](int hg, int& kvh, int& first) {
    kvh = hg / p.nseg;
    first = (hg - kvh * p.nseg) * p.rows;
    return min(p.rows, p.total_rows - first);
  };

  if (warp < n_units && bnd[warp] < bnd[warp + 1]) {
    const int k0 = bnd[warp], k1 = bnd[warp + 1], slot_begin = warp * S, slot_end = slot_begin + S;
    const uint64_t policy = p.nseg == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();

    uint8_t* ring = rings + static_cast<size_t>(warp) * S * kTile;
    uint8_t* qbuf = qbufs + warp * q_bytes;
    auto fetch_q = [&](int b, int hg) {
      int kvh, first;
      const int rows = seg_rows(hg, kvh, first);
      constexpr int kChunks = D / 8;
      for (int i = lane; i < rows * kChunks; i += 32)
        cp_async_16(qbuf + i * 16, p.q + f8_row_at(p, b, kvh, first + i / kChunks, D) + (i % kChunks) * 8);
      cp_async_commit();
    };
    F8Walk wk = starts[warp];
    fetch_q(wk.b, wk.hg);  // in front of the copies that fill the memory's queues

    // Issue side: the warp copies its own tiles, a ring ahead of their use.
    // Block ids come in windows of 32 (lane i holds entry wj + i of sequence
    // wb's table); the window that is needed next is loaded when one is taken.
    F8Walk wi = wk;
    int left = k1 - max(k0, wi.st + kSeg);  // slots from tile wi.j on; a tile while positive
    auto table = [&](int b, int j) {
      const int at = j + lane;
      return at < p.max_blocks_per_seq ? p.block_tables[static_cast<size_t>(b) * p.max_blocks_per_seq + at] : -1;
    };
    int wb = -1, wj = 0, ids = 0, nxb = -1, nxj = 0, nx_ids = 0;
    auto window = [&]() {
      if (wi.b == wb && static_cast<unsigned>(wi.j - wj) < 32u) return;
      if (wi.b == nxb && static_cast<unsigned>(wi.j - nxj) < 32u) {
        wb = nxb, wj = nxj, ids = nx_ids;
      } else {
        wb = wi.b, wj = wi.nb <= 32 ? 0 : wi.j;
        ids = table(wb, wj);
      }
      nxb = wb, nxj = 0;
      if (wj + 32 < wi.nb) {
        nxj = wj + 32;
      } else if (wi.hg + 1 == p.ng || wi.nb <= 32) {  // else the next head of the same sequence, from its start
        do {
          ++nxb;
        } while (nxb < B && ctxs[nxb] == 0);
      }
      if (nxb < B) nx_ids = table(nxb, nxj);
    };
    // Tile wi.j + i into a slot, by one lane.
    auto copy = [&](int phys, int slot) {
      const bool bad = phys < 0 || phys >= p.num_blocks;
      slot_bad[slot] = bad;  // published by the arrivals
      if (bad) {             // nothing is copied; the tile is left out
        flag_error(PKV_DEVERR_BLOCK_ID);
        mbar_arrive(&full_bar[slot]);
        mbar_arrive(&full_bar[slot]);
      } else {
        const int at = phys * p.n_kv_heads + wi.hg / p.nseg;
        mbar_arrive_expect_tx(&full_bar[slot], kTile);
        tma_load_3d_hint(rings + static_cast<size_t>(slot) * kTile, &tm, &full_bar[slot], at, policy);
        cp_async_8(&slot_scale[slot], p.scales + at);
        cp_async_arrive(&full_bar[slot]);
      }
    };
    // The next tiles into n slots from `slot` on, a lane for each.
    const int withhold_at = p.withhold_unit < sc.U ? unit_begin(sc, p.withhold_unit) : -1;
    const int withheld = withhold_at >= k0 && withhold_at < k1 ? 0 : -1;  // which of the unit's tiles
    int issued = 0;
    auto issue = [&](int slot, int n) {
      while (n > 0 && left > 0) {
        window();
        const int off = wi.j - wj, k = min(min(n, left), min(wi.nb - wi.j, 32 - off));
        const int phys = __shfl_sync(0xffffffffu, ids, off + lane);
        if (lane < k && issued + lane != withheld) copy(phys, slot + lane < slot_end ? slot + lane : slot + lane - S);
        slot += k;
        if (slot >= slot_end) slot -= S;
        n -= k;
        issued += k;
        left -= k;
        wi.j += k;
        if (wi.j == wi.nb) {
          f8_next_segment<kSeg>(wi, prefix, ctxs, B, p.ng);
          left -= kSeg;
        }
      }
    };
    issue(slot_begin, S);
    if (warp == W - 1) f8_find_groups<W, kSeg>(p, sc, per_cta, u0, n_units, bnd, prefix, ctxs, groups, &n_groups);

    Consumer cs;
    int slot = slot_begin;
    uint32_t phase = 0;
    bool ok = true;
    // Segment by segment; `end` is the first tile that is not this unit's.
    while (true) {
      int kvh, first;
      const int rows = seg_rows(wk.hg, kvh, first);
      const int end = min(wk.nb, k1 - wk.st - kSeg), ctx = ctxs[wk.b];
      F8Walk nx = wk;
      f8_next_segment<kSeg>(nx, prefix, ctxs, B, p.ng);
      const bool more = nx.st < k1;
      cp_async_wait_all();
      __syncwarp();
      cs.begin(p, qbuf, first, rows, lane);
      __syncwarp();
      if (more) fetch_q(nx.b, nx.hg);  // the next segment's Q, behind this one's tiles
#pragma unroll 1
      for (int j = wk.j; j < end; j += 2) {
        const bool two = j + 1 < end;
        const int slot0 = slot;
        ok = mbar_wait_bounded(&full_bar[slot0], phase, abort_flag, p.wait_limit_ns);
        if (++slot == slot_end) {
          slot -= S;
          phase ^= 1u;
        }
        const int slot1 = slot;
        if (two) {
          ok = ok && mbar_wait_bounded(&full_bar[slot1], phase, abort_flag, p.wait_limit_ns);
          if (++slot == slot_end) {
            slot -= S;
            phase ^= 1u;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        F8Step st;
        // Without a second tile the first one stands in for it (the next
        // slot's copy may be under way), dead.
        st.base[0] = smem_u32(rings) + slot0 * kTile;
        st.base[1] = two ? smem_u32(rings) + slot1 * kTile : st.base[0];
        st.dead[0] = slot_bad[slot0] != 0;
        st.dead[1] = !two || slot_bad[slot1] != 0;
        const float2 one = make_float2(1.f, 1.f);
        const float2 s0 = st.dead[0] ? one : slot_scale[slot0], s1 = st.dead[1] ? one : slot_scale[slot1];
        st.ks[0] = s0.x, st.vs[0] = s0.y, st.ks[1] = s1.x, st.vs[1] = s1.y;
        st.rem = ctx - j * kBlockTokens;
        cs.step(st, p.q_len, lane);
        __syncwarp();  // every lane has read the slots
        issue(slot0, two ? 2 : 1);
      }
      if (!ok) break;
      // A whole segment's output; a share of one that reaches the unit's end
      // in this warp's drained ring, else in its record.
      float* rec = nullptr;
      if (wk.st < k0 || nx.st > k1)
        rec = nx.st >= k1 ? reinterpret_cast<float*>(ring) : p.unit_recs + static_cast<size_t>(u0 + warp) * p.rec_floats;
      cs.finish(p, rec, wk.b, kvh, first, rows, lane);
      if (!more) break;
      wk = nx;
    }
    cp_async_wait_all();
    if (!ok && lane == 0)  // do not leave while copies may still be landing
      for (int i = max(0, issued - S); i < issued; ++i) {
        const uint64_t since = global_timer_ns();
        while (!mbar_try_wait(&full_bar[slot_begin + i % S], static_cast<uint32_t>((i / S) & 1)) &&
               global_timer_ns() - since < p.wait_limit_ns) {
        }
      }
  } else if (warp == W - 1) {
    f8_find_groups<W, kSeg>(p, sc, per_cta, u0, n_units, bnd, prefix, ctxs, groups, &n_groups);
  }
  __syncthreads();

  // ---------------- the CTA's shared segments ----------------
  const int A = bnd[0], E = bnd[n_units], ng = n_groups;
  // Four rows a warp.  (A row a warp, its pieces shared by the groups of lanes:
  // 59 us against 43 for 32 x 4 queries, no gain where there are few rows.)
  const int items = (p.rows + 3) / 4;
  // The first group may come from before the CTA, the last may go on behind it (one may do both).
  const bool from_before = ng > 0 && groups[0].st < A;
  const bool goes_on = ng > 0 && groups[ng - 1].en > E && groups[ng - 1].st >= A;
  // Their words are settled beside the merges, by the warp that has the fewest of them.
  const bool settles = warp == W - 1 && (lane == 0 ? from_before : lane == 1 && goes_on);
  unsigned long long word = 0;
  if (settles) word = load_relaxed(p.arrivals + groups[lane == 0 ? 0 : ng - 1].c0);
  for (int i = warp; i < ng * items; i += W) {
    const F8Group& gr = groups[i / items];
    F8Pieces pc;  // in the rings; the last one in its unit's record if more follows it there
    pc.n = gr.ub - gr.ua + 1;
    pc.stride = S * kTile / 4;
    pc.base = pc.first = reinterpret_cast<const float*>(rings) + static_cast<size_t>(gr.ua) * pc.stride;
    pc.last = nullptr;
    if (gr.en < bnd[gr.ub + 1]) {
      pc.last = p.unit_recs + static_cast<size_t>(u0 + gr.ub) * p.rec_floats;
      if (pc.n == 1) pc.first = pc.last;
    }
    float* to = nullptr;
    if (gr.st < A || gr.en > E) to = p.cta_recs + (static_cast<size_t>(blockIdx.x) * 2 + (gr.st < A ? 0 : 1)) * p.rec_floats;
    f8_merge<D, kBf16, false>(p, pc, i % items * 4, gr.rows, to, gr.b, gr.kvh, gr.first);
  }

  // ---------------- segments shared with other CTAs ----------------
  if (!from_before && !goes_on) return;
  if (settles) {
    const F8Group& gr = groups[lane == 0 ? 0 : ng - 1];
    f8_settle(p.arrivals + gr.c0, word, p.arrival, gr.n_ctas);
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    int fin = 0;
    if (threadIdx.x == 0 ? from_before : goes_on) {
      const F8Group& gr = groups[threadIdx.x == 0 ? 0 : ng - 1];
      unsigned long long* at = p.arrivals + gr.c0;
      // After every record of this CTA, before any it reads.
      if (add_acq_rel(at, p.arrival) == static_cast<unsigned long long>(gr.n_ctas - 1) * p.arrival) {
        fin = 1;
        *at = 0;
      }
    }
    last_of[threadIdx.x] = fin;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (last_of[k] == 0) continue;
    const F8Group& gr = groups[k == 0 ? 0 : ng - 1];
    F8Pieces pc;  // the first CTA's share goes on behind it, the others' come from before
    pc.n = gr.n_ctas;
    pc.stride = 2 * p.rec_floats;
    pc.base = p.cta_recs + static_cast<size_t>(gr.c0) * pc.stride;
    pc.first = pc.base + p.rec_floats;
    pc.last = nullptr;
    // Many shares: a warp a row (one sequence of 4096: 13.6 us, 18.7 with four
    // rows a warp); few: four rows a warp (32 x 4 queries: 42.7 us, 45.0).
    if (pc.n > 4) {
      for (int i = warp; i < gr.rows; i += W) f8_merge<D, kBf16, true>(p, pc, i, gr.rows, nullptr, gr.b, gr.kvh, gr.first);
    } else {
      for (int i = warp * 4; i < gr.rows; i += W * 4)
        f8_merge<D, kBf16, false>(p, pc, i, gr.rows, nullptr, gr.b, gr.kvh, gr.first);
    }
  }
}

}  // namespace pkv
