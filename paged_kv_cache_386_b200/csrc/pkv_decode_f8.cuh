// pkv_decode_f8.cuh -- decode attention over the FP8 cache (e4m3 codes, one
// scale for each block, kv head and K or V).
#pragma once

#include "pkv_append_f8.cuh"

namespace pkv {

constexpr int kF8MaxRows = 16;  // (query, head) rows that share a pass over K and V

struct DecodeF8Params {
  const uint16_t* q;  // [batch][q_len][n_q][D], f16 or bf16
  uint16_t* out;
  const uint8_t* kv;
  const float* scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t max_blocks_per_seq, batch, num_blocks, n_q_heads, n_kv_heads, q_len;
  int32_t gp;     // query heads per segment
  int32_t rows;   // gp * q_len
  int32_t ng;     // segments per sequence
  int32_t bf16;
  float scale_log2;
};

// One CTA of 128 threads per segment (the rows of one kv head of one
// sequence): 128 tokens at a time, a thread first owns a token (scores), then
// a dim (output).
template <int D>
__global__ void __launch_bounds__(128) pkv_decode_f8_kernel(const DecodeF8Params p) {
  __shared__ float q_s[kF8MaxRows][D];
  __shared__ float w_s[kF8MaxRows][128];
  __shared__ float v_scale[8];
  __shared__ int block_id[8];
  __shared__ float red[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.ng, hg = blockIdx.x % p.ng;
  const int kvh = hg * p.gp / (p.n_q_heads / p.n_kv_heads);
  int ctx = __ldg(p.context_lens + b);
  const int max_ctx = p.max_blocks_per_seq * kBlockTokens;
  if (ctx < 0 || ctx > max_ctx || (ctx > 0 && ctx < p.q_len)) {
    if (tid == 0) flag_error(PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 || ctx < p.q_len ? 0 : max_ctx;
  }
  auto row_at = [&](int r) {
    return ((static_cast<size_t>(b) * p.q_len + r / p.gp) * p.n_q_heads + hg * p.gp + r % p.gp) * D;
  };
  auto to_f = [&](uint16_t h) {
    float lo, hi;
    if (p.bf16) unpack2<true>(h, lo, hi); else unpack2<false>(h, lo, hi);
    return lo;
  };
  for (int i = tid; i < p.rows * D; i += 128) q_s[i / D][i % D] = to_f(p.q[row_at(i / D) + i % D]);
  float o[kF8MaxRows], m[kF8MaxRows], l[kF8MaxRows];
  for (int r = 0; r < kF8MaxRows; ++r) o[r] = 0.f, m[r] = -INFINITY, l[r] = 0.f;
  for (int t0 = 0; t0 < ctx; t0 += 128) {
    __syncthreads();
    if (tid < 8) {
      const int j = t0 / kBlockTokens + tid;
      int id = j * kBlockTokens < ctx ? __ldg(p.block_tables + static_cast<size_t>(b) * p.max_blocks_per_seq + j) : -2;
      if (id != -2 && (id < 0 || id >= p.num_blocks)) {
        flag_error(PKV_DEVERR_BLOCK_ID);
        id = -1;
      }
      block_id[tid] = id;
      v_scale[tid] = id >= 0 ? p.scales[(static_cast<size_t>(id) * p.n_kv_heads + kvh) * 2 + 1] : 0.f;
    }
    __syncthreads();
    const int t = t0 + tid, id = block_id[tid / 16];
    const bool live = id >= 0 && t < ctx;
    float s[kF8MaxRows];
    for (int r = 0; r < kF8MaxRows; ++r) s[r] = 0.f;
    if (live) {
      const size_t tile = static_cast<size_t>(id) * p.n_kv_heads + kvh;
      const uint8_t* k = p.kv + tile * f8_tile_bytes(D) + (tid % 16) * D;
      const float ks = p.scales[tile * 2] * p.scale_log2;
      for (int e = 0; e < D; e += 2) {
        float k0, k1;
        unpack2<false>(f8_unpack2(*reinterpret_cast<const uint16_t*>(k + e)), k0, k1);
        for (int r = 0; r < p.rows; ++r) s[r] += q_s[r][e] * k0 + q_s[r][e + 1] * k1;
      }
      for (int r = 0; r < kF8MaxRows; ++r) s[r] *= ks;
    }
    for (int r = 0; r < p.rows; ++r) {
      const bool seen = live && t < ctx - p.q_len + r / p.gp + 1;
      const float x = seen ? s[r] : -INFINITY;
      float mx = x;
      for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      if (lane == 0) red[warp] = mx;
      __syncthreads();
      mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
      __syncthreads();
      const float mn = fmaxf(m[r], mx);
      const float alpha = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mn);
      const float w = seen ? exp2f(x - mn) : 0.f;
      o[r] *= alpha;
      l[r] = l[r] * alpha + w;
      m[r] = mn;
      w_s[r][tid] = w;
    }
    __syncthreads();
    if (tid < D) {
      for (int j = 0; j < 128 && t0 + j < ctx; ++j) {
        const int vid = block_id[j / 16];
        if (vid < 0) continue;
        const uint8_t c = p.kv[(static_cast<size_t>(vid) * p.n_kv_heads + kvh) * f8_tile_bytes(D) +
                               (kBlockTokens + j % 16) * D + tid];
        float v, unused;
        unpack2<false>(f8_unpack2(c), v, unused);
        v *= v_scale[j / 16];
        for (int r = 0; r < p.rows; ++r)  // a row's own causal limit: what it does not see may be NaN
          if (t0 + j < ctx - p.q_len + r / p.gp + 1) o[r] += w_s[r][j] * v;
      }
    }
  }
  for (int r = 0; r < p.rows; ++r) {
    float sum = l[r];
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = red[0] + red[1] + red[2] + red[3];
    if (tid < D) {
      const float y = sum == 0.f ? 0.f : o[r] / sum;
      p.out[row_at(r) + tid] = static_cast<uint16_t>(p.bf16 ? pack2<true>(y, 0.f) : pack2<false>(y, 0.f));
    }
  }
}

}  // namespace pkv
