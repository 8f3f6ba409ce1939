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
// f16 data the rounding of the weights (2^-12) is as large as that of the
// output, so their remainders take a second product.
//
// Rows on the n side of the product halve the products for 8 rows or fewer
// (16 MMAs for a tile of 16 x 128 K and V, not 32) and the accumulators.
#pragma once

#include "pkv_append_f8.cuh"
#include "pkv_prefix_tc.cuh"

namespace pkv {

constexpr int kF8MaxStages = 6;                       // ring slots of a warp
constexpr int kF8MinTiles = 2;                        // tiles that make a unit worth its merge
constexpr int kF8HeaderBytes = 4096;                  // workspace: a counter per CTA
constexpr int kF8BadTile = 0x7fc0bad0;                 // K scale of a tile whose block id is out of range (a NaN)
constexpr float kF8RefBelow = 7.f, kF8RefSlack = 14.f;

struct DecodeF8Params {
  const uint16_t* q;  // [batch][q_len][n_q][D], f16 or bf16
  uint16_t* out;
  const float2* scales;  // [num_blocks][n_kv]
  const int32_t* block_tables;
  const int32_t* context_lens;
  unsigned int* counters;  // [CTAs], 0 between launches
  float* unit_recs;        // [units][rec_floats]: a segment that ends inside a unit and began before it
  float* cta_recs;         // [CTAs][2][rec_floats]: the CTA's share of a segment from before it, of one that goes on
  int32_t max_blocks_per_seq, batch, num_blocks, n_q_heads, n_kv_heads, q_len;
  int32_t group;       // query heads per kv head
  int32_t total_rows;  // group * q_len rows of a kv head: row i is query i / group, head i % group
  int32_t rows;        // rows of a segment (the last one of a kv head may have fewer)
  int32_t nseg;        // segments of a kv head
  int32_t ng;          // segments of a sequence, n_kv * nseg
  int32_t stages;
  int32_t rec_floats;  // rows * (D + 4)
  float scale_log2;
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
    if (!edge) {
      pv<false>(v0, 0u, ph[0], pl[0], lane);
      pv<false>(v1, 0u, ph[1], pl[1], lane);
    } else {
      // V bytes behind the context may hold anything: cleared.
      const int n0 = st.dead[0] ? 0 : st.rem, n1 = st.dead[1] ? 0 : st.rem - kBlockTokens;
      if (q_len > 1 && (nan_in(v0, keep_bytes(n0, t), lane) || nan_in(v1, keep_bytes(n1, t), lane))) {
        // A row that does not see a NaN's token would take 0 x NaN: the
        // product once for each query, over the tokens that it sees.
#pragma unroll 1
        for (int hq = 0; hq < q_len; ++hq) {
          pv<true>(v0, keep_bytes(n0 - hq, t), ph[0], pl[0], lane, hq);
          pv<true>(v1, keep_bytes(n1 - hq, t), ph[1], pl[1], lane, hq);
        }
      } else {
        pv<true>(v0, keep_bytes(n0, t), ph[0], pl[0], lane);
        pv<true>(v1, keep_bytes(n1, t), ph[1], pl[1], lane);
      }
    }
  }

  // Mask of this lane's four V bytes, of a tile with n tokens.
  __device__ __forceinline__ static uint32_t keep_bytes(int n, int t) {
    uint32_t keep = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (f8_v_token(4 * t + i) < n) keep |= 0xffu << (8 * i);
    return keep;
  }

  // O^T += V^T P^T of one tile; only_hide >= 0: only rows with that many hidden tokens take it.
  template <bool kKeep>
  __device__ __forceinline__ void pv(uint32_t v, uint32_t keep, const uint32_t (&ph)[NR][2], const uint32_t (&pl)[NR][2],
                                     int lane, int only_hide = -1) {
    const int vt = f8_v_token(lane & 15), vc = lane >> 4;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t r[4];
      ldsm_b8_x2_trans(v + f8_chunk_at<D>(vt, 2 * i + vc), r[0], r[1], r[2], r[3]);
      if constexpr (kKeep) {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] &= keep;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a0, a1, a2, a3;
        f8_unpack4(r[2 * h], a0, a2);
        f8_unpack4(r[2 * h + 1], a1, a3);
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          if constexpr (kKeep) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = o[nr][2 * i + h][k];
            mma_16816<false>(x, a0, a1, a2, a3, ph[nr][0], ph[nr][1]);
            if constexpr (kRest) mma_16816<false>(x, a0, a1, a2, a3, pl[nr][0], pl[nr][1]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (only_hide < 0 || hide[nr][k & 1] == only_hide) o[nr][2 * i + h][k] = x[k];
          } else {
            mma_16816<false>(o[nr][2 * i + h], a0, a1, a2, a3, ph[nr][0], ph[nr][1]);
            if constexpr (kRest) mma_16816<false>(o[nr][2 * i + h], a0, a1, a2, a3, pl[nr][0], pl[nr][1]);
          }
        }
      }
    }
  }

  __device__ __forceinline__ static bool nan_in(uint32_t v, uint32_t keep, int lane) {
    const int vt = f8_v_token(lane & 15), vc = lane >> 4;
    uint32_t found = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint32_t r[4];
      ldsm_b8_x2_trans(v + f8_chunk_at<D>(vt, 2 * i + vc), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int k = 0; k < 4; ++k) found |= ((r[k] & keep & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    }
    return __any_sync(0xffffffffu, found != 0);
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

// Dims [d0 + DPL lane, + DPL) of one row merged over n pieces, in order:
//   M = max m_i,  w_i = 2^(m_i - M),  O = sum w_i O_i,  l = sum w_i l_i,
// online over batches whose loads go out together.  `at(j)`: the row in piece
// j.  Written to the record row `to`, or normalised to `out`.  kGlobal: the
// pieces were written by other SMs (read through L2).
template <int D, int DPL, bool kGlobal, bool kBf16, class At>
__device__ __forceinline__ void f8_merge_row(const At& at, int n, int d0, int lane, float* to, uint16_t* out) {
  constexpr int kBatch = DPL == 1 ? 16 : 8;
  const int dim = d0 + lane * DPL;
  float M = -INFINITY, L = 0.f, acc[DPL];
#pragma unroll
  for (int i = 0; i < DPL; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < n; j0 += kBatch) {
    float mj[kBatch], lj[kBatch], o[kBatch][DPL];
#pragma unroll
    for (int jj = 0; jj < kBatch; ++jj) {
      const float* r = at(min(j0 + jj, n - 1));
      if constexpr (kGlobal) {
        mj[jj] = ld_cg(r + D);
        lj[jj] = ld_cg(r + D + 1);
        if constexpr (DPL == 4) {
          const float4 v = ld_cg4(r + dim);
          o[jj][0] = v.x, o[jj][1] = v.y, o[jj][2] = v.z, o[jj][3] = v.w;
        } else if constexpr (DPL == 2) {
          const float2 v = ld_cg2(r + dim);
          o[jj][0] = v.x, o[jj][1] = v.y;
        } else {
          o[jj][0] = ld_cg(r + dim);
        }
      } else {
        mj[jj] = r[D];
        lj[jj] = r[D + 1];
#pragma unroll
        for (int i = 0; i < DPL; ++i) o[jj][i] = r[dim + i];
      }
    }
    float Mb = M;
#pragma unroll
    for (int jj = 0; jj < kBatch; ++jj)
      if (j0 + jj < n) Mb = fmaxf(Mb, mj[jj]);
    // -inf: no token seen so far; those pieces' sums are 0 (or NaN, which stays).
    const float alpha = M == -INFINITY ? 1.f : exp2f(M - Mb);
    L *= alpha;
#pragma unroll
    for (int i = 0; i < DPL; ++i) acc[i] *= alpha;
#pragma unroll
    for (int jj = 0; jj < kBatch; ++jj) {
      if (j0 + jj >= n) continue;
      const float w = mj[jj] == -INFINITY ? 1.f : exp2f(mj[jj] - Mb);
      L = fmaf(w, lj[jj], L);
#pragma unroll
      for (int i = 0; i < DPL; ++i) acc[i] = fmaf(w, o[jj][i], acc[i]);
    }
    M = Mb;
  }
  if (to != nullptr) {
#pragma unroll
    for (int i = 0; i < DPL; ++i) to[dim + i] = acc[i];
    if (lane == 0 && d0 == 0) {
      to[D] = M;
      to[D + 1] = L;
    }
    return;
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < (DPL + 1) / 2; ++i) {
    const float x = acc[2 * i] * inv, z = DPL > 1 ? acc[(2 * i + 1) % DPL] * inv : 0.f;
    w[i] = pack2<kBf16>(x, z);
  }
  if constexpr (DPL == 4)
    *reinterpret_cast<uint2*>(out + dim) = make_uint2(w[0], w[1]);
  else if constexpr (DPL == 2)
    *reinterpret_cast<uint32_t*>(out + dim) = w[0];
  else
    out[dim] = static_cast<uint16_t>(w[0]);
}

// Rows of a segment that this CTA holds in several units, or shares with other CTAs.
struct F8Group {
  int b, hg, st, en;  // the segment's tiles [st, en)
  int ua, ub;         // first and last unit of this CTA with a piece of it
};

// Warps of a CTA, each a unit.
__host__ __device__ constexpr int f8_warps(int NR) { return NR == 1 ? 12 : 8; }

// Shared memory: each warp's ring, its Q rows, a scale pair and a barrier of each slot; lengths.
__host__ __device__ constexpr size_t f8_smem_bytes(int D, int W, int stages, int rows, int batch) {
  return 1024 + static_cast<size_t>(W) * (stages * (f8_tile_bytes(D) + 16) + rows * D * 2) + 16 +
         (2 * static_cast<size_t>(batch) + 1) * 4;
}

template <int D, int NR, bool kBf16>
__global__ void __launch_bounds__(f8_warps(NR) * 32, 1)
    pkv_decode_f8_kernel(const __grid_constant__ CUtensorMap tm, const DecodeF8Params p) {
  constexpr int kTile = f8_tile_bytes(D);
  constexpr int W = f8_warps(NR), kThreads = W * 32;
  using Consumer = F8Consumer<D, NR, kBf16>;
  constexpr int RS = Consumer::RS;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* rings = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int S = p.stages, q_bytes = p.rows * D * 2;
  uint8_t* qbufs = rings + static_cast<size_t>(W) * S * kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(qbufs + W * q_bytes);  // [W][S]: the slot's copies have landed
  float2* slot_scales = reinterpret_cast<float2*>(bars + W * S);      // [W][S]
  volatile int* abort_flag = reinterpret_cast<int*>(slot_scales + W * S);
  int* prefix = const_cast<int*>(abort_flag) + 4;  // [batch + 1]
  int* ctxs = prefix + p.batch + 1;                // [batch]
  __shared__ int warp_sums[W];
  __shared__ F8Group groups[W + 1];
  __shared__ int n_groups;
  __shared__ int last_of[2];  // this CTA finishes: the segment from before it, the one that goes on behind it

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int B = p.batch;
  uint8_t* ring = rings + static_cast<size_t>(warp) * S * kTile;  // this warp's
  uint64_t* bar = bars + warp * S;
  float2* slot_scale = slot_scales + warp * S;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tm);
    *abort_flag = 0;
  }
  if (lane == 0) {
    for (int i = 0; i < S; ++i) mbar_init(&bar[i], 2);  // the codes' bytes, and the scales
    mbar_fence_init();
  }

  // Tiles before each sequence.
  {
    const int per = (B + kThreads - 1) / kThreads;
    const int lo = min(B, static_cast<int>(threadIdx.x) * per), hi = min(B, lo + per);
    const int max_ctx = p.max_blocks_per_seq * kBlockTokens;
    int local = 0;
    for (int b = lo; b < hi; ++b) {
      const int c0 = __ldg(p.context_lens + b);
      int c = clamp_ctx(c0, max_ctx);
      if (c > 0 && c < p.q_len) c = 0;
      if (c != c0) flag_error(PKV_DEVERR_CONTEXT);
      ctxs[b] = c;
      local += ((c + kBlockTokens - 1) / kBlockTokens) * p.ng;
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
      run += ((ctxs[b] + kBlockTokens - 1) / kBlockTokens) * p.ng;
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
  const Sched sc = make_sched(T, min(static_cast<int>(gridDim.x) * W, max(1, T / kF8MinTiles)), 0, 1000);
  const int u0 = blockIdx.x * W, u_end = min(sc.U, u0 + W);  // this CTA's units
  if (T == 0 || u0 >= sc.U) return;

  // Rows of segment hg of a sequence: kv head, first of its rows, how many.
  auto seg_rows = [&](int hg, int& kvh, int& first) {
    kvh = hg / p.nseg;
    first = (hg - kvh * p.nseg) * p.rows;
    return min(p.rows, p.total_rows - first);
  };

  if (u0 + warp < u_end) {
    const int u = u0 + warp, k0 = unit_begin(sc, u), k1 = unit_begin(sc, u + 1);
    const uint64_t policy = p.nseg == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();

    // Issue side: the warp copies its own tiles, S ahead of their use.  Block
    // ids come in windows of 32 (lane i holds entry wj + i of sequence wb's
    // table); the window that is needed next is loaded when one is taken.
    Walk wi;
    walk_begin(wi, prefix, ctxs, B, k0, k1);
    auto table = [&](int b, int j) {
      const int at = j + lane;
      return at < p.max_blocks_per_seq ? __ldg(p.block_tables + static_cast<size_t>(b) * p.max_blocks_per_seq + at) : -1;
    };
    int wb = -1, wj = 0, ids = 0, nxb = -1, nxj = 0, nx_ids = 0;
    auto window = [&]() {
      if (wi.b == wb && wi.j >= wj && wi.j < wj + 32) return;
      if (wi.b == nxb && wi.j >= nxj && wi.j < nxj + 32) {
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
    auto issue = [&](int slot) {
      window();
      const int phys = __shfl_sync(0xffffffffu, ids, wi.j - wj);
      if (lane == 0) {
        if (phys < 0 || phys >= p.num_blocks) {  // nothing is copied; a NaN K scale marks the tile
          flag_error(PKV_DEVERR_BLOCK_ID);
          slot_scale[slot] = make_float2(__int_as_float(kF8BadTile), 0.f);
          mbar_arrive(&bar[slot]);
          mbar_arrive(&bar[slot]);
        } else {
          const int at = phys * p.n_kv_heads + wi.hg / p.nseg;
          mbar_arrive_expect_tx(&bar[slot], kTile);
          tma_load_3d_hint(ring + slot * kTile, &tm, &bar[slot], at, policy);
          cp_async_8(&slot_scale[slot], p.scales + at);
          cp_async_arrive(&bar[slot]);
        }
      }
      walk_next(wi, prefix, ctxs, B, p.ng);
    };
    int issued = 0;
    for (; issued < S && wi.k < k1; ++issued) issue(issued);

    uint8_t* qbuf = qbufs + warp * q_bytes;
    auto fetch_q = [&](int b, int hg) {
      int kvh, first;
      const int rows = seg_rows(hg, kvh, first);
      constexpr int kChunks = D / 8;
      for (int i = lane; i < rows * kChunks; i += 32)
        cp_async_16(qbuf + i * 16, p.q + f8_row_at(p, b, kvh, first + i / kChunks, D) + (i % kChunks) * 8);
      cp_async_commit();
    };
    Walk wk;
    walk_begin(wk, prefix, ctxs, B, k0, k1);
    fetch_q(wk.b, wk.hg);
    Consumer cs;
    int slot = 0, kvh = 0, first = 0, rows = 0;
    uint32_t phase = 0;
    bool fresh = true, ok = true;
    while (true) {
      if (fresh) {
        fresh = false;
        rows = seg_rows(wk.hg, kvh, first);
        cp_async_wait_all();
        __syncwarp();
        cs.begin(p, qbuf, first, rows, lane);
        __syncwarp();
      }
      const int n = min(min(2, wk.nb - wk.j), k1 - wk.k);  // tiles of this step
      const bool last = wk.k + n >= k1, seg_last = wk.j + n >= wk.nb;
      if (seg_last && !last) {  // the next segment's Q
        Walk nx = wk;
        nx.j = nx.nb - 1;
        walk_next(nx, prefix, ctxs, B, p.ng);
        fetch_q(nx.b, nx.hg);
      }
      const int slot1 = slot + 1 == S ? 0 : slot + 1;
      const uint32_t phase1 = phase ^ (slot1 == 0 ? 1u : 0u);
      ok = mbar_wait_bounded(&bar[slot], phase, abort_flag, p.wait_limit_ns);
      if (n == 2) ok = ok && mbar_wait_bounded(&bar[slot1], phase1, abort_flag, p.wait_limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      F8Step st;
      const float2 s0 = slot_scale[slot], s1 = n == 2 ? slot_scale[slot1] : make_float2(1.f, 1.f);
      st.base[0] = smem_u32(ring + slot * kTile);
      st.base[1] = smem_u32(ring + slot1 * kTile);
      st.ks[0] = s0.x, st.vs[0] = s0.y, st.ks[1] = s1.x, st.vs[1] = s1.y;
      st.dead[0] = __float_as_int(s0.x) == kF8BadTile;
      st.dead[1] = n == 1 || __float_as_int(s1.x) == kF8BadTile;
      st.rem = wk.ctx - wk.j * kBlockTokens;
      cs.step(st, p.q_len, lane);
      __syncwarp();  // every lane has read the slots
      if (wi.k < k1) {
        issue(slot);
        ++issued;
      }
      if (n == 2 && wi.k < k1) {
        issue(slot1);
        ++issued;
      }
      phase = n == 2 ? phase1 ^ (slot1 + 1 == S ? 1u : 0u) : phase1;
      slot = n == 2 ? (slot1 + 1 == S ? 0 : slot1 + 1) : slot1;
      if (seg_last || last) {
        // A whole segment's output; a share of one that reaches the unit's
        // end in this warp's drained ring, else in its record.
        const int nb = wk.nb, start = wk.k - wk.j;
        float* rec = nullptr;
        if (start < k0 || start + nb > k1)
          rec = last ? reinterpret_cast<float*>(ring) : p.unit_recs + static_cast<size_t>(u) * p.rec_floats;
        cs.finish(p, rec, wk.b, kvh, first, rows, lane);
        fresh = true;
      }
      if (last) break;
      wk.k += n - 1;
      wk.j += n - 1;
      walk_next(wk, prefix, ctxs, B, p.ng);
    }
    cp_async_wait_all();
    if (!ok && lane == 0) {  // do not leave while copies may still be landing
      for (int i = max(0, issued - S); i < issued; ++i) {
        const uint64_t since = global_timer_ns();
        while (!mbar_try_wait(&bar[i % S], static_cast<uint32_t>((i / S) & 1)) &&
               global_timer_ns() - since < p.wait_limit_ns) {
        }
      }
    }
  }
  __syncthreads();

  // ---------------- the CTA's shared segments ----------------
  // Candidates: the segment that comes from before the CTA, and for each unit
  // the segment that starts in it and goes on behind it.
  const int A = unit_begin(sc, u0), E = unit_begin(sc, u_end);
  if (warp == 0) {
    bool valid = false;
    F8Group gr;
    if (lane <= u_end - u0) {
      const int u = u0 + max(0, lane - 1);
      const int k = lane == 0 ? A : unit_begin(sc, u + 1) - 1;
      Walk w;
      walk_begin(w, prefix, ctxs, B, k, k + 1);
      gr.b = w.b;
      gr.hg = w.hg;
      gr.st = k - w.j;
      gr.en = gr.st + w.nb;
      gr.ua = u;
      gr.ub = min(unit_of_tile(sc, gr.en - 1), u_end - 1);
      valid = lane == 0 ? gr.st < A : gr.st >= unit_begin(sc, u) && gr.en > k + 1;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, valid);
    if (valid) groups[__popc(mask & ((1u << lane) - 1u))] = gr;
    if (lane == 0) n_groups = __popc(mask);
  }
  __syncthreads();
  const int ng = n_groups;
  for (int i = warp; i < ng * p.rows; i += W) {
    const F8Group gr = groups[i / p.rows];
    const int row = i % p.rows;
    int kvh, first;
    if (row >= seg_rows(gr.hg, kvh, first)) continue;
    auto at = [&](int j) -> const float* {
      const int u = gr.ua + j;
      const float* rec = gr.en >= unit_begin(sc, u + 1)
                             ? reinterpret_cast<const float*>(rings + static_cast<size_t>(u - u0) * S * kTile)
                             : p.unit_recs + static_cast<size_t>(u) * p.rec_floats;
      return rec + row * RS;
    };
    float* to = nullptr;
    if (gr.st < A || gr.en > E)
      to = p.cta_recs + (static_cast<size_t>(blockIdx.x) * 2 + (gr.st < A ? 0 : 1)) * p.rec_floats + row * RS;
    f8_merge_row<D, D / 32, false, kBf16>(at, gr.ub - gr.ua + 1, 0, lane, to,
                                   p.out + f8_row_at(p, gr.b, kvh, first + row, D));
  }

  // ---------------- segments shared with other CTAs ----------------
  // The first group may come from before the CTA, the last may go on behind it (one may do both).
  const bool from_before = ng > 0 && groups[0].st < A;
  const bool goes_on = ng > 0 && groups[ng - 1].en > E && groups[ng - 1].st >= A;
  if (!from_before && !goes_on) return;
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2) {
    int fin = 0;
    if (threadIdx.x == 0 ? from_before : goes_on) {
      const F8Group& gr = groups[threadIdx.x == 0 ? 0 : ng - 1];
      const int c0 = unit_of_tile(sc, gr.st) / W, n = unit_of_tile(sc, gr.en - 1) / W - c0 + 1;
      const unsigned int before = atomicAdd(p.counters + c0, 1u);
      if (before >= static_cast<unsigned int>(n)) flag_error(PKV_DEVERR_SCHEDULE);
      if (before + 1 >= static_cast<unsigned int>(n)) {
        fin = 1;
        p.counters[c0] = 0;
      }
    }
    last_of[threadIdx.x] = fin;
    __threadfence();
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (last_of[k] == 0) continue;
    const F8Group gr = groups[k == 0 ? 0 : ng - 1];
    const int c0 = unit_of_tile(sc, gr.st) / W, n = unit_of_tile(sc, gr.en - 1) / W - c0 + 1;
    int kvh, first;
    const int rows = seg_rows(gr.hg, kvh, first);
    auto row_at = [&](int row, int j) -> const float* {  // the first CTA's share goes on behind it, the others' come from before
      return p.cta_recs + (static_cast<size_t>(c0 + j) * 2 + (j == 0 ? 1 : 0)) * p.rec_floats + row * RS;
    };
    if (n > 8) {  // many pieces: D / 32 warps share a row
      for (int i = warp; i < rows * (D / 32); i += W) {
        const int row = i / (D / 32);
        f8_merge_row<D, 1, true, kBf16>([&](int j) { return row_at(row, j); }, n, i % (D / 32) * 32, lane, nullptr,
                                 p.out + f8_row_at(p, gr.b, kvh, first + row, D));
      }
    } else {
      for (int row = warp; row < rows; row += W)
        f8_merge_row<D, D / 32, true, kBf16>([&](int j) { return row_at(row, j); }, n, 0, lane, nullptr,
                                      p.out + f8_row_at(p, gr.b, kvh, first + row, D));
    }
  }
}

}  // namespace pkv
