// pkv_append_f8.cuh -- sm_100a kernels that rotate and store new tokens:
//   pkv_append_rope_kernel   rotary position embedding of the new queries and
//                            keys, and the scatter of keys and values into a
//                            cache of the same type
//   pkv_append_f8_kernel     the same scatter (rotation optional) into the FP8
//                            cache: e4m3 codes, one power-of-two scale for
//                            each (block, kv head, K or V)
//   pkv_copy_blocks_f8_kernel  copy-on-write of whole FP8 blocks
//
// All three only move bytes (a few flops per element), so they are laid out
// for wide accesses: a thread owns 16 dims of a head row, the two 8-dim pieces
// that the rotation pairs with each other, so that no value crosses threads and
// queries may be rotated in place.
#pragma once

#include "pkv_kernels.cuh"

namespace pkv {

// These kernels are launched while the kernel in front of them on the stream ends
// (launch_early), and wait here until its writes can be seen, before they read or
// write any memory but their own shared memory.  Inputs are read by ordinary loads:
// the read-only path (ld.global.nc) is for memory that nothing writes from a kernel's
// start on.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Sixteen elements of a head row as fp32: two pieces of eight consecutive dims.
template <int DT>
struct Piece8 {
  // The raw 8 elements as loaded (16 or 32 bytes).
  uint4 a, b;
  __device__ __forceinline__ void load(const uint8_t* p) {
    a = *reinterpret_cast<const uint4*>(p);
    if constexpr (DT == kF32) b = *reinterpret_cast<const uint4*>(p + 16);
  }
  __device__ __forceinline__ void store(uint8_t* p) const {
    *reinterpret_cast<uint4*>(p) = a;
    if constexpr (DT == kF32) *reinterpret_cast<uint4*>(p + 16) = b;
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    if constexpr (DT == kF32) {
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
      unpack2<DT == kBF16>(a.x, x[0], x[1]);
      unpack2<DT == kBF16>(a.y, x[2], x[3]);
      unpack2<DT == kBF16>(a.z, x[4], x[5]);
      unpack2<DT == kBF16>(a.w, x[6], x[7]);
    }
  }
  // Rounds to nearest even for 16-bit types: the result's one rounding.
  __device__ __forceinline__ void narrow(const float (&x)[8]) {
    if constexpr (DT == kF32) {
      a = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      b = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    } else {
      a = make_uint4(pack2<DT == kBF16>(x[0], x[1]), pack2<DT == kBF16>(x[2], x[3]), pack2<DT == kBF16>(x[4], x[5]),
                     pack2<DT == kBF16>(x[6], x[7]));
    }
  }
};

// The rotation of one token: row `pos` of the table holds rot / 2 cosines,
// then rot / 2 sines.  Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) when
// interleaved; dims from `rot` on are left as they are.
struct RopeTable {
  const float* table;  // [max_pos][rot]
  const int64_t* positions;
  int64_t max_pos;
  int32_t rot;
  int32_t interleaved;
};

// First dims of chunk c's two 8-dim pieces: of a row that is rotated, the
// two halves of eight pairs; else sixteen consecutive dims.
__device__ __forceinline__ void chunk_dims(int c, bool rotate, const RopeTable& t, int& i0, int& i1) {
  const bool split = rotate && !t.interleaved && c * 16 < t.rot;
  i0 = split ? c * 8 : c * 16;
  i1 = split ? t.rot / 2 + c * 8 : c * 16 + 8;
}

// Two fp32 values in a register pair: both products at once, each rounded as the
// scalar product is.
__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// cos and sin of the chunk's eight pairs.
__device__ __forceinline__ void load_cos_sin(const RopeTable& t, int64_t pos, int c, float (&cs)[8], float (&sn)[8]) {
  const float* row = t.table + pos * t.rot + c * 8;
  const float4 c0 = reinterpret_cast<const float4*>(row)[0], c1 = reinterpret_cast<const float4*>(row)[1];
  row += t.rot / 2;
  const float4 s0 = reinterpret_cast<const float4*>(row)[0], s1 = reinterpret_cast<const float4*>(row)[1];
  cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
  sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
}

// (a, b) -> (a c - b s, b c + a s).  Every product and sum is rounded to fp32
// by itself (no fused multiply-add): the codes of the FP8 cache are decided by
// these values, and so are those of a restatement in plain fp32 operations.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float y0 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = y0;
}

__device__ __forceinline__ void rotate_chunk(float (&x0)[8], float (&x1)[8], const float (&cs)[8],
                                             const float (&sn)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate_pair(x0[2 * i], x0[2 * i + 1], cs[i], sn[i]);
      rotate_pair(x1[2 * i], x1[2 * i + 1], cs[4 + i], sn[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // The sums stay scalar: packed products and packed sums were joined
      // into fused multiply-adds.
      const uint64_t a = pack_f2(x0[i], x0[i + 1]), b = pack_f2(x1[i], x1[i + 1]);
      const uint64_t c = pack_f2(cs[i], cs[i + 1]), s = pack_f2(sn[i], sn[i + 1]);
      float ac[2], bs[2], bc[2], as[2];
      unpack_f2(mul_f2(a, c), ac[0], ac[1]);
      unpack_f2(mul_f2(b, s), bs[0], bs[1]);
      unpack_f2(mul_f2(b, c), bc[0], bc[1]);
      unpack_f2(mul_f2(a, s), as[0], as[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x0[i + k] = __fsub_rn(ac[k], bs[k]);
        x1[i + k] = __fadd_rn(bc[k], as[k]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Rotation and append, same type
// ---------------------------------------------------------------------------
// The heads of a token are listed as n_q query heads, n_kv key heads, n_kv
// value heads (the FP8 append uses the query heads alone).
struct RopeAppendParams {
  const uint8_t* q;  // null: no queries (n_q = 0)
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // bytes between tokens
  const int64_t* slot_mapping;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t num_slots;
  RopeTable rope;
  int32_t num_tokens, n_q, n_kv, head_dim;
  int32_t heads_per_thread;  // consecutive listed heads that a thread walks
};

// One thread's item: 16 dims (chunk c) of heads_per_thread listed heads of one
// token.  The cosines and sines are read once for all of them.  Loads of
// up to kU heads go out before their stores.
template <int DT>
__device__ __forceinline__ void rope_append_item(const RopeAppendParams& p, uint32_t item, int head_group,
                                                 int n_heads) {
  constexpr int kBytes = DTypeInfo<DT>::kBytes;
  constexpr int kU = 2;
  const uint32_t chunks = static_cast<uint32_t>(p.head_dim) / 16u;  // item = token * chunks + c
  if (item >= static_cast<uint32_t>(p.num_tokens) * chunks) return;
  const int64_t tok = item / chunks;
  const int c = static_cast<int>(item % chunks);
  const int h_begin = head_group * p.heads_per_thread;
  const int h_end = min(n_heads, h_begin + p.heads_per_thread);
  const int64_t pos = p.rope.positions[tok];
  if (pos < 0 || pos >= p.rope.max_pos) {
    if (c == 0 && h_begin == 0) flag_error(PKV_DEVERR_POSITION);
    return;
  }
  int64_t slot = -1;
  if (h_end > p.n_q) {
    slot = p.slot_mapping[tok];
    if (slot >= p.num_slots) {
      if (c == 0 && h_end == n_heads) flag_error(PKV_DEVERR_SLOT);
      slot = -1;
    }
  }
  const bool turns = c * 16 < p.rope.rot && h_begin < p.n_q + p.n_kv;
  float cs[8], sn[8];
  if (turns) load_cos_sin(p.rope, pos, c, cs, sn);
  const int64_t blk = slot >> 4, off = slot & 15;  // 16-token blocks; not used when slot < 0
  for (int h0 = h_begin; h0 < h_end; h0 += kU) {
    Piece8<DT> x[kU], y[kU];
    uint8_t* dst[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u;
      dst[u] = nullptr;
      if (h >= h_end) continue;
      const uint8_t* src;
      if (h < p.n_q) {
        src = p.q + tok * p.q_stride + static_cast<int64_t>(h) * p.head_dim * kBytes;
        dst[u] = p.q_out + tok * p.q_out_stride + static_cast<int64_t>(h) * p.head_dim * kBytes;
      } else {
        if (slot < 0) continue;
        const bool is_v = h >= p.n_q + p.n_kv;
        const int kh = h - p.n_q - (is_v ? p.n_kv : 0);
        src = (is_v ? p.v + tok * p.v_stride : p.k + tok * p.k_stride) + static_cast<int64_t>(kh) * p.head_dim * kBytes;
        dst[u] = (is_v ? p.v_cache : p.k_cache) +
                 ((blk * p.n_kv + kh) * kBlockTokens + off) * p.head_dim * kBytes;
      }
      int i0, i1;
      chunk_dims(c, h < p.n_q + p.n_kv, p.rope, i0, i1);
      x[u].load(src + i0 * kBytes);
      y[u].load(src + i1 * kBytes);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (dst[u] == nullptr) continue;
      const bool rotate = h0 + u < p.n_q + p.n_kv;
      int i0, i1;
      chunk_dims(c, rotate, p.rope, i0, i1);
      if (rotate && turns) {
        float a[8], b[8];
        x[u].widen(a);
        y[u].widen(b);
        rotate_chunk(a, b, cs, sn, p.rope.interleaved != 0);
        x[u].narrow(a);
        y[u].narrow(b);
      }
      x[u].store(dst[u] + i0 * kBytes);
      y[u].store(dst[u] + i1 * kBytes);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(256, DT == kF32 ? 3 : 4) pkv_append_rope_kernel(const RopeAppendParams p) {
  wait_for_kernel_before();
  rope_append_item<DT>(p, blockIdx.x * 256u + threadIdx.x, blockIdx.y, p.n_q + 2 * p.n_kv);
}

// ---------------------------------------------------------------------------
// FP8 cache
// ---------------------------------------------------------------------------
// kv [num_blocks][n_kv][2][16][D] e4m3 codes (K, then V), scales
// [num_blocks][n_kv][2] fp32; a value is code x scale.
constexpr int kF8MinExp = -48, kF8MaxExp = 48;  // exponents of the scales that an append writes

__host__ __device__ constexpr int f8_tile_bytes(int D) { return 2 * kBlockTokens * D; }

// The smallest power of two s = 2^e, e in [kF8MinExp, kF8MaxExp], with amax
// <= 448 s (448 = 1.75 x 2^8 is the largest e4m3 value).  With amax = m 2^k,
// m in [1, 2): e = k - 8 if m <= 1.75, else k - 7; adding 0x1fffff carries into
// the exponent just when the mantissa is above .75.
__device__ __forceinline__ float f8_scale_for(float amax) {
  const int e = static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
  return __uint_as_float(static_cast<uint32_t>(min(max(e, kF8MinExp), kF8MaxExp) + 127) << 23);
}

// Two fp32 to two e4m3 codes (lo in bits 0..7): nearest even, magnitudes past
// 448 (infinities too) to 448, NaN to NaN.
__device__ __forceinline__ uint32_t f8_pack2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes to a packed half pair (exact).
__device__ __forceinline__ uint32_t f8_unpack2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Sixteen codes times `ratio`, rounded to e4m3 again.
__device__ __forceinline__ uint4 f8_rescale(uint4 v, float ratio) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b, c, d;
    unpack2<false>(f8_unpack2(w[i] & 0xffffu), a, b);
    unpack2<false>(f8_unpack2(w[i] >> 16), c, d);
    w[i] = f8_pack2(a * ratio, b * ratio) | (f8_pack2(c * ratio, d * ratio) << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct AppendF8Params {
  RopeAppendParams rp;  // inputs, strides, rotation (rope.rot = 0: none) and the query part
  uint8_t* kv;
  float* scales;
  int32_t tokens_per_pair;  // 1 or 16 tokens whose runs a pair of warps starts
  int32_t token_chunks;     // ceil(num_tokens / tokens_per_pair)
  int32_t kv_ctas;          // CTAs of the K/V part; later CTAs rotate queries,
  int32_t q_ctas;           // this many for each group of heads_per_thread heads
};

// Magnitudes of two packed 16-bit values and the larger of each (NaN is passed over).
template <bool kBf16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t w) {
  uint32_t r;
  w &= 0x7fff7fffu;
  if constexpr (kBf16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w));
  return r;
}

// The larger of two warps' maxima, the same in all their lanes.  `buf` takes turns
// (0, 1), so that a value stays until both have read it.
__device__ __forceinline__ float pair_max(float a, float (*exchange)[8], int buf, int warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) exchange[buf][warp] = a;
  named_bar_sync(1 + (warp >> 1), 64);
  return fmaxf(a, exchange[buf][warp ^ 1]);
}

template <int D>
struct F8Rows {
  static constexpr int kLanes = D / 16;      // lanes of one head row, 16 dims each
  static constexpr int kRows = 32 / kLanes;  // rows at a time
  static constexpr int kIter = kBlockTokens / 2 / kRows;
};

// One kv head's K or V of a run: this lane's part of the rows tok[it] (token of
// the call, -1: none) at block offsets row0 + it kRows.
template <int DT, int D, bool kRotate>
__device__ __forceinline__ void append_f8_rows(const AppendF8Params& p, int64_t blk, int head, bool is_v,
                                               const int (&tok)[F8Rows<D>::kIter], int c, int row0, bool fresh, int warp,
                                               float (*exchange)[8], int& buf) {
  constexpr int kBytes = DTypeInfo<DT>::kBytes;
  constexpr int kRows = F8Rows<D>::kRows, kIter = F8Rows<D>::kIter;
  constexpr float kLargest = 3.402823466e38f;
  const RopeAppendParams& rp = p.rp;
  const int64_t block_head = blk * rp.n_kv + head;
  float* scale_at = p.scales + block_head * 2 + (is_v ? 1 : 0);
  const float s_old = *scale_at;
  const uint8_t* base = (is_v ? rp.v : rp.k) + static_cast<int64_t>(head) * D * kBytes;
  const int64_t stride = is_v ? rp.v_stride : rp.k_stride;
  int i0, i1;
  chunk_dims(c, kRotate, rp.rope, i0, i1);
  // Not rotated, the rows stay as loaded and are widened where they are used;
  // rotated ones are kept as fp32.
  Piece8<DT> x[kIter], y[kIter];
  float v0[kRotate ? kIter : 1][8], v1[kRotate ? kIter : 1][8];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    x[it].a = x[it].b = y[it].a = y[it].b = make_uint4(0u, 0u, 0u, 0u);
    if (tok[it] < 0) continue;
    x[it].load(base + tok[it] * stride + i0 * kBytes);
    y[it].load(base + tok[it] * stride + i1 * kBytes);
  }
  if constexpr (kRotate) {
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      x[it].widen(v0[it]);
      y[it].widen(v1[it]);
      if (c * 16 < rp.rope.rot && tok[it] >= 0) {
        float cs[8], sn[8];
        load_cos_sin(rp.rope, rp.rope.positions[tok[it]], c, cs, sn);
        rotate_chunk(v0[it], v1[it], cs, sn, rp.rope.interleaved != 0);
      }
    }
  }
  auto values = [&](int it, float (&a)[8], float (&b)[8]) {
    if constexpr (kRotate) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = v0[it][i], b[i] = v1[it][i];
    } else {
      x[it].widen(a);
      y[it].widen(b);
    }
  };

  float amax = 0.f;
  if constexpr (DT != kF32 && !kRotate) {
    uint32_t m2 = 0u;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      const uint32_t w[8] = {x[it].a.x, x[it].a.y, x[it].a.z, x[it].a.w, y[it].a.x, y[it].a.y, y[it].a.z, y[it].a.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) m2 = max_abs2<DT == kBF16>(m2, w[i]);
    }
    float lo, hi;
    unpack2<DT == kBF16>(m2, lo, hi);
    amax = fmaxf(lo, hi);
  } else {
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      float a[8], b[8];
      values(it, a, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(a[i]), fabsf(b[i])));
    }
  }
  amax = pair_max(amax, exchange, buf, warp);
  buf ^= 1;
  if (amax > kLargest) {  // an infinity does not set the scale
    amax = 0.f;
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      float a[8], b[8];
      values(it, a, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (fabsf(a[i]) <= kLargest) amax = fmaxf(amax, fabsf(a[i]));
        if (fabsf(b[i]) <= kLargest) amax = fmaxf(amax, fabsf(b[i]));
      }
    }
    amax = pair_max(amax, exchange, buf, warp);
    buf ^= 1;
  }
  const float need = f8_scale_for(amax);
  const float s_new = fresh ? need : fmaxf(s_old, need);
  const float inv = 1.0f / s_new;  // exact: a power of two, if the block's old scale is one
  uint8_t* tile = p.kv + block_head * f8_tile_bytes(D) + (is_v ? kBlockTokens * D : 0);
  const bool regrid = !fresh && s_new != s_old;
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    uint8_t* row = tile + (row0 + it * kRows) * D;
    if (tok[it] >= 0) {
      float a[8], b[8];
      values(it, a, b);
      uint32_t w[4];
      const uint64_t inv2 = pack_f2(inv, inv);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = i < 2 ? a[4 * i + k] : b[4 * (i - 2) + k];
        unpack_f2(mul_f2(pack_f2(v[0], v[1]), inv2), v[0], v[1]);
        unpack_f2(mul_f2(pack_f2(v[2], v[3]), inv2), v[2], v[3]);
        w[i] = f8_pack2(v[0], v[1]) | (f8_pack2(v[2], v[3]) << 16);
      }
      if constexpr (kRotate) {
        *reinterpret_cast<uint2*>(row + i0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(row + i1) = make_uint2(w[2], w[3]);
      } else {
        *reinterpret_cast<uint4*>(row + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else if (fresh) {
      *reinterpret_cast<uint4*>(row + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    } else if (regrid) {
      uint4* at = reinterpret_cast<uint4*>(row + c * 16);
      *at = f8_rescale(*at, s_old * inv);
    }
  }
  // (The other warp has read the old scale: in front of the exchange.)
  if ((threadIdx.x & 31) == 0 && (warp & 1) == 0 && (fresh || regrid)) *scale_at = s_new;
}

// Consecutive tokens of the call in the same block are a run; two warps take a
// whole run of one kv head, K and then V (a step's single tokens: either), a
// half of the block's rows each, so that the block's scale is decided in one
// place: no atomics, and the result does not depend on scheduling.  Of two
// tokens with the same slot in a run the last counts.
//
// D / 16 lanes hold a row, all rows of the half at once, 16 registers of 16-bit
// data: what bounds a prompt is how many rows are under way, and 64 registers
// a thread let four CTAs fit an SM.  (One warp a run, all of it as fp32: 128
// registers, 32.2 us for 16384 bf16 tokens of 8 heads of 128; now 20.4, the
// floor is 15.4.  The next head's rows requested ahead, or the call's rows
// before its slots are known: more registers, slower.)
template <int DT, int D, bool kRope>
__device__ __forceinline__ void append_f8_run(const AppendF8Params& p, int64_t blk, int first, int head, int lane, int warp,
                                              float (*exchange)[8], int& buf, int kind_begin, int kind_end) {
  constexpr int kLanes = F8Rows<D>::kLanes, kRows = F8Rows<D>::kRows, kIter = F8Rows<D>::kIter;
  const int row0 = (warp & 1) * (kBlockTokens / 2) + lane / kLanes;
  const RopeAppendParams& rp = p.rp;
  // Token of the call for each offset of the block (lane = offset), -1 none.
  int src = -1;
  for (int base = first;; base += 32) {
    int64_t s = -1;
    if (base + lane < rp.num_tokens) s = rp.slot_mapping[base + lane];
    // A slot beyond the pool is skipped where it stands, in the middle of a run too.
    const bool here = (s >> 4) == blk;
    const uint32_t other = __ballot_sync(0xffffffffu, !here && s < rp.num_slots);
    const int n = other ? __ffs(other) - 1 : 32;
    int off = -1;
    if (lane < n && here) {
      off = static_cast<int>(s & 15);
      if constexpr (kRope) {
        const int64_t pos = rp.rope.positions[base + lane];
        if (pos < 0 || pos >= rp.rope.max_pos) {  // left out, as if it were padding
          flag_error(PKV_DEVERR_POSITION);
          off = -1;
        }
      }
    }
    const int off0 = __shfl_sync(0xffffffffu, off, 0);
    if (__all_sync(0xffffffffu, lane >= n || (off0 >= 0 && off == off0 + lane))) {  // in order, as prompts and steps are
      if (lane >= off0 && lane < off0 + n) src = base + lane - off0;
    } else {
#pragma unroll 1
      for (int j = 0; j < kBlockTokens; ++j) {
        const uint32_t at = __ballot_sync(0xffffffffu, off == j);
        if (lane == j && at) src = base + 31 - __clz(at);
      }
    }
    if (n < 32) break;
  }
  if (!__any_sync(0xffffffffu, src >= 0)) return;
  const bool fresh = __shfl_sync(0xffffffffu, src, 0) >= 0;

  const int c = lane % kLanes;
  int tok[kIter];
#pragma unroll
  for (int it = 0; it < kIter; ++it) tok[it] = __shfl_sync(0xffffffffu, src, row0 + it * kRows);
  for (int kind = kind_begin; kind < kind_end; ++kind) {
    const bool is_v = kind == 1;
    if (kRope && !is_v)
      append_f8_rows<DT, D, true>(p, blk, head, false, tok, c, row0, fresh, warp, exchange, buf);
    else
      append_f8_rows<DT, D, false>(p, blk, head, is_v, tok, c, row0, fresh, warp, exchange, buf);
  }
}

template <int DT, int D, bool kRope>
__global__ void __launch_bounds__(256, DT == kF32 ? 3 : 4) pkv_append_f8_kernel(const AppendF8Params p) {
  wait_for_kernel_before();
  const RopeAppendParams& rp = p.rp;
  if (kRope && static_cast<int>(blockIdx.x) >= p.kv_ctas) {  // queries
    const uint32_t i = blockIdx.x - p.kv_ctas;
    rope_append_item<DT>(rp, (i % p.q_ctas) * 256u + threadIdx.x, i / p.q_ctas, rp.n_q);
    return;
  }
  __shared__ float exchange[2][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int buf = 0;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 6) + (warp >> 1);
  const bool one_kind = p.tokens_per_pair == 1;  // K and V to a pair each
  const int items = one_kind ? 2 * rp.n_kv : rp.n_kv;
  const int64_t chunk = w / items;
  if (chunk >= p.token_chunks) return;
  const int item = static_cast<int>(w % items), head = one_kind ? item >> 1 : item;
  const int kind_begin = one_kind ? item & 1 : 0, kind_end = one_kind ? kind_begin + 1 : 2;
  // Lane l looks at token l - 1 of the chunk, so that lane 0 holds the token before it.
  const int64_t t = chunk * p.tokens_per_pair + lane - 1;
  constexpr int64_t kBeyond = -2;  // a slot beyond the pool, as if its token were not there
  int64_t blk = -1;
  if (t >= 0 && t < rp.num_tokens && lane <= p.tokens_per_pair) {
    const int64_t s = rp.slot_mapping[t];
    if (s >= rp.num_slots) {
      if (item == 0 && lane > 0) flag_error(PKV_DEVERR_SLOT);
      blk = kBeyond;
    } else if (s >= 0) {
      blk = s >> 4;
    }
  }
  int64_t before = __shfl_up_sync(0xffffffffu, blk, 1);
  if (__any_sync(0xffffffffu, before == kBeyond)) {
    for (int64_t u = t - 1; before == kBeyond; --u) {  // u: the last token looked at
      const int64_t s = u > 0 ? rp.slot_mapping[u - 1] : -1;
      before = s >= rp.num_slots ? kBeyond : s >= 0 ? s >> 4 : -1;
    }
  }
  uint32_t starts = __ballot_sync(0xffffffffu, lane > 0 && blk >= 0 && blk != before);
  while (starts) {
    const int l = __ffs(starts) - 1;
    starts &= starts - 1;
    append_f8_run<DT, D, kRope>(p, __shfl_sync(0xffffffffu, blk, l), static_cast<int>(chunk * p.tokens_per_pair) + l - 1,
                                head, lane, warp, exchange, buf, kind_begin, kind_end);
  }
}

struct CopyF8Params {
  uint8_t* kv;
  float* scales;
  const int32_t* src;
  const int32_t* dst;
  int32_t n_pairs;
  int32_t num_blocks;
  int32_t chunks;  // 16-byte chunks of one block's codes
  int32_t n_scales;  // scales of one block
};

// CTAs stride over the pairs, four 16-byte loads in flight per thread.
__global__ void __launch_bounds__(256) pkv_copy_blocks_f8_kernel(const CopyF8Params p) {
  for (int pair = blockIdx.x; pair < p.n_pairs; pair += gridDim.x) {
    const int32_t s = p.src[pair], d = p.dst[pair];
    if (s < 0 || s >= p.num_blocks || d < 0 || d >= p.num_blocks) {
      if (threadIdx.x == 0) flag_error(PKV_DEVERR_BLOCK_ID);
      continue;
    }
    const uint4* from = reinterpret_cast<const uint4*>(p.kv) + static_cast<int64_t>(s) * p.chunks;
    uint4* to = reinterpret_cast<uint4*>(p.kv) + static_cast<int64_t>(d) * p.chunks;
    for (int c0 = threadIdx.x; c0 < p.chunks; c0 += 4 * blockDim.x) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + u * 256 < p.chunks) v[u] = from[c0 + u * 256];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (c0 + u * 256 < p.chunks) to[c0 + u * 256] = v[u];
    }
    for (int i = threadIdx.x; i < p.n_scales; i += blockDim.x)
      p.scales[static_cast<int64_t>(d) * p.n_scales + i] = p.scales[static_cast<int64_t>(s) * p.n_scales + i];
  }
}

}  // namespace pkv
