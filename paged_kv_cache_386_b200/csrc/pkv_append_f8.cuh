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

// cos and sin of the chunk's eight pairs.
__device__ __forceinline__ void load_cos_sin(const RopeTable& t, int64_t pos, int c, float (&cs)[8], float (&sn)[8]) {
  const float* row = t.table + pos * t.rot + c * 8;
  const float4 c0 = __ldg(reinterpret_cast<const float4*>(row)), c1 = __ldg(reinterpret_cast<const float4*>(row) + 1);
  row += t.rot / 2;
  const float4 s0 = __ldg(reinterpret_cast<const float4*>(row)), s1 = __ldg(reinterpret_cast<const float4*>(row) + 1);
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
    for (int i = 0; i < 8; ++i) rotate_pair(x0[i], x1[i], cs[i], sn[i]);
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
  constexpr int kU = DT == kF32 ? 2 : 4;
  const uint32_t chunks = static_cast<uint32_t>(p.head_dim) / 16u;  // item = token * chunks + c
  if (item >= static_cast<uint32_t>(p.num_tokens) * chunks) return;
  const int64_t tok = item / chunks;
  const int c = static_cast<int>(item % chunks);
  const int h_begin = head_group * p.heads_per_thread;
  const int h_end = min(n_heads, h_begin + p.heads_per_thread);
  const int64_t pos = __ldg(p.rope.positions + tok);
  if (pos < 0 || pos >= p.rope.max_pos) {
    if (c == 0 && h_begin == 0) flag_error(PKV_DEVERR_POSITION);
    return;
  }
  int64_t slot = -1;
  if (h_end > p.n_q) {
    slot = __ldg(p.slot_mapping + tok);
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
__global__ void __launch_bounds__(256) pkv_append_rope_kernel(const RopeAppendParams p) {
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
  int32_t tokens_per_warp;  // 1 or 16 tokens whose runs a warp starts
  int32_t token_chunks;     // ceil(num_tokens / tokens_per_warp)
  int32_t kv_ctas;          // CTAs of the K/V part; later CTAs rotate queries,
  int32_t q_ctas;           // this many for each group of heads_per_thread heads
};

// Consecutive tokens of the call in the same block are a run; a warp takes a
// whole run of one kv head, for K or for V, so that the block's scale is
// decided in one place: no atomics, and the result does not depend on
// scheduling.  Of two tokens with the same slot in a run the last counts.
template <int DT, int D>
__device__ __forceinline__ void append_f8_run(const AppendF8Params& p, int64_t blk, int64_t first, int head, bool is_v,
                                              int lane) {
  constexpr int kBytes = DTypeInfo<DT>::kBytes;
  constexpr int kLanes = D / 16;           // lanes of one head row, 16 dims each
  constexpr int kRows = 32 / kLanes;       // rows at a time
  constexpr int kIter = kBlockTokens / kRows;
  const RopeAppendParams& rp = p.rp;
  const bool has_rope = rp.rope.rot > 0;
  // Token of the call for each offset of the block (lane = offset), -1 none.
  int64_t src = -1;
  for (int64_t base = first;; base += 32) {
    int64_t s = -1;
    if (base + lane < rp.num_tokens) s = __ldg(rp.slot_mapping + base + lane);
    const uint32_t other = __ballot_sync(0xffffffffu, s < 0 || (s >> 4) != blk);
    const int n = other ? __ffs(other) - 1 : 32;
    int off = -1;
    if (lane < n) {
      off = static_cast<int>(s & 15);
      if (has_rope) {
        const int64_t pos = __ldg(rp.rope.positions + base + lane);
        if (pos < 0 || pos >= rp.rope.max_pos) {  // left out, as if it were padding
          flag_error(PKV_DEVERR_POSITION);
          off = -1;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBlockTokens; ++j) {
      const uint32_t at = __ballot_sync(0xffffffffu, off == j);
      if (lane == j && at) src = base + 31 - __clz(at);
    }
    if (n < 32) break;
  }
  if (!__any_sync(0xffffffffu, src >= 0)) return;
  const bool fresh = __shfl_sync(0xffffffffu, src, 0) >= 0;

  float* scale_at = p.scales + (blk * rp.n_kv + head) * 2 + (is_v ? 1 : 0);
  const float s_old = *scale_at;
  const int c = lane % kLanes;
  const bool rotate = has_rope && !is_v;
  int i0, i1;
  chunk_dims(c, rotate, rp.rope, i0, i1);
  const uint8_t* base = (is_v ? rp.v : rp.k) + static_cast<int64_t>(head) * D * kBytes;
  const int64_t stride = is_v ? rp.v_stride : rp.k_stride;
  Piece8<DT> x[kIter], y[kIter];
  int64_t tok[kIter];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    tok[it] = __shfl_sync(0xffffffffu, src, it * kRows + lane / kLanes);
    x[it].a = x[it].b = y[it].a = y[it].b = make_uint4(0u, 0u, 0u, 0u);
    if (tok[it] < 0) continue;
    x[it].load(base + tok[it] * stride + i0 * kBytes);
    y[it].load(base + tok[it] * stride + i1 * kBytes);
  }
  float v0[kIter][8], v1[kIter][8];
  float amax = 0.f;
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    x[it].widen(v0[it]);
    y[it].widen(v1[it]);
    if (rotate && c * 16 < rp.rope.rot && tok[it] >= 0) {
      float cs[8], sn[8];
      load_cos_sin(rp.rope, __ldg(rp.rope.positions + tok[it]), c, cs, sn);
      rotate_chunk(v0[it], v1[it], cs, sn, rp.rope.interleaved != 0);
    }
    // Infinities and NaN do not set the scale.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(v0[it][i]), b = fabsf(v1[it][i]);
      if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
      if (b <= 3.402823466e38f) amax = fmaxf(amax, b);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float need = f8_scale_for(amax);
  const float s_new = fresh ? need : fmaxf(s_old, need);
  const float inv = 1.0f / s_new;  // exact: a power of two
  uint8_t* tile = p.kv + (static_cast<int64_t>(blk) * rp.n_kv + head) * f8_tile_bytes(D) + (is_v ? kBlockTokens * D : 0);
  const bool regrid = !fresh && s_new != s_old;
  const float ratio = s_old * inv;
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    uint8_t* row = tile + (it * kRows + lane / kLanes) * D;
    if (tok[it] >= 0) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[i] = f8_pack2(v0[it][4 * i] * inv, v0[it][4 * i + 1] * inv) |
               (f8_pack2(v0[it][4 * i + 2] * inv, v0[it][4 * i + 3] * inv) << 16);
        w[2 + i] = f8_pack2(v1[it][4 * i] * inv, v1[it][4 * i + 1] * inv) |
                   (f8_pack2(v1[it][4 * i + 2] * inv, v1[it][4 * i + 3] * inv) << 16);
      }
      *reinterpret_cast<uint2*>(row + i0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + i1) = make_uint2(w[2], w[3]);
    } else if (fresh) {
      *reinterpret_cast<uint4*>(row + c * 16) = make_uint4(0u, 0u, 0u, 0u);
    } else if (regrid) {
      uint4* at = reinterpret_cast<uint4*>(row + c * 16);
      *at = f8_rescale(*at, ratio);
    }
  }
  if (lane == 0 && (fresh || regrid)) *scale_at = s_new;
}

template <int DT, int D>
__global__ void __launch_bounds__(256) pkv_append_f8_kernel(const AppendF8Params p) {
  const RopeAppendParams& rp = p.rp;
  if (static_cast<int>(blockIdx.x) >= p.kv_ctas) {  // queries
    const uint32_t i = blockIdx.x - p.kv_ctas;
    rope_append_item<DT>(rp, (i % p.q_ctas) * 256u + threadIdx.x, i / p.q_ctas, rp.n_q);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int heads2 = 2 * rp.n_kv;
  const int64_t chunk = w / heads2;
  if (chunk >= p.token_chunks) return;
  const int h2 = static_cast<int>(w % heads2);
  // Lane l looks at token l - 1 of the chunk, so that lane 0 holds the token before it.
  const int64_t t = chunk * p.tokens_per_warp + lane - 1;
  int64_t blk = -1;
  if (t >= 0 && t < rp.num_tokens && lane <= p.tokens_per_warp) {
    const int64_t s = __ldg(rp.slot_mapping + t);
    if (s >= rp.num_slots) {
      if (h2 == 0 && lane > 0) flag_error(PKV_DEVERR_SLOT);
    } else if (s >= 0) {
      blk = s >> 4;
    }
  }
  const int64_t before = __shfl_up_sync(0xffffffffu, blk, 1);
  uint32_t starts = __ballot_sync(0xffffffffu, lane > 0 && blk >= 0 && blk != before);
  while (starts) {
    const int l = __ffs(starts) - 1;
    starts &= starts - 1;
    append_f8_run<DT, D>(p, __shfl_sync(0xffffffffu, blk, l), chunk * p.tokens_per_warp + l - 1, h2 >> 1, h2 & 1, lane);
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
    const int32_t s = __ldg(p.src + pair), d = __ldg(p.dst + pair);
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
