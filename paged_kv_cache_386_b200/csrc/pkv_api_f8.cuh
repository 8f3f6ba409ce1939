// pkv_api_f8.cuh -- C ABI of the rotating append and of the FP8 cache (part of
// pkv_api.cu's translation unit).
#pragma once

namespace pkv {
namespace {

// Checks of the new tokens' inputs that the rotating and the FP8 append share;
// fills the inputs of `p`.  Strides are in elements.
pkv_status rope_append_params(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, pkv_dtype dtype, const int64_t* positions, const float* cos_sin,
                              int64_t max_positions, int32_t rot_dim, int32_t interleaved,
                              const int64_t* slot_mapping, int32_t num_tokens, int32_t num_blocks,
                              int32_t block_size, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                              void* q_out, int64_t q_out_stride, RopeAppendParams* p) {
  if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_q_heads < 0 ||
      rot_dim < 0 || rot_dim > head_dim || (interleaved != 0 && interleaved != 1))
    return PKV_ERR_INVALID_ARG;
  const int es = elem_bytes(dtype);
  if (es == 0 || block_size != kBlockTokens || head_dim % 16 != 0 || rot_dim % 16 != 0) return PKV_ERR_UNSUPPORTED;
  const int64_t kv_row = static_cast<int64_t>(n_kv_heads) * head_dim, q_row = static_cast<int64_t>(n_q_heads) * head_dim;
  if (kv_row > INT32_MAX || q_row > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_tokens) * (head_dim / 16) > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  *p = {};
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || (n_q_heads > 0) != (q != nullptr) || (n_q_heads > 0 && !q_out))
    return PKV_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!positions || !cos_sin || max_positions <= 0)) return PKV_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(q) || !aligned16(q_out) || !aligned16(cos_sin) ||
      (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 7u))
    return PKV_ERR_INVALID_ARG;
  const int64_t strides[4] = {q_stride, k_stride, v_stride, q_out_stride};
  for (int i = 0; i < 4; ++i)
    if (strides[i] < 0 || strides[i] > INT64_MAX / 8 || (strides[i] * es) % 16 != 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens > 1 && q && q_out_stride < q_row) return PKV_ERR_INVALID_ARG;  // rows would overlap
  if (num_tokens > 1 && q && q_out == q && q_out_stride != q_stride) return PKV_ERR_INVALID_ARG;
  p->q = static_cast<const uint8_t*>(q);
  p->k = static_cast<const uint8_t*>(k);
  p->v = static_cast<const uint8_t*>(v);
  p->q_out = static_cast<uint8_t*>(q_out);
  p->q_stride = q_stride * es;
  p->k_stride = k_stride * es;
  p->v_stride = v_stride * es;
  p->q_out_stride = q_out_stride * es;
  p->slot_mapping = slot_mapping;
  p->num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p->rope = {cos_sin, positions, max_positions, rot_dim, interleaved};
  p->num_tokens = num_tokens;
  p->n_q = n_q_heads;
  p->n_kv = n_kv_heads;
  p->head_dim = head_dim;
  return PKV_OK;
}

// Heads that one thread of the rotation walks, sharing a token's cosines
// and sines: as many as leave a thread for every one the device holds, at
// most 8.  (8192 tokens, 32/8 heads: 36.4 us, 48.4 with one head a thread; one
// token: 2.3 us, 4.6 with eight.)
int rope_heads_per_thread(int64_t columns, int heads, int sm_count) {
  const int64_t want = static_cast<int64_t>(sm_count) * 2048;
  for (int hp = 8; hp > 1; hp /= 2)
    if (columns * ((heads + hp - 1) / hp) >= want) return hp;
  return 1;
}

// The launch overlaps the end of the kernel in front on the stream, whose writes
// the kernel waits for itself.  Calls back to back on a stream, one token's
// rotating append: 2.0 us, 4.1 without; a step's FP8 append 3.7, 6.2; one sequence's
// decode 12.6, 14.4; in a graph 0.2 to 0.6 us less.  (The next launch allowed from
// a kernel's start on, not from its end: 2.2, 4.3 and 12.9, its blocks are in the way.)
template <typename... P>
pkv_status launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, const P&... p) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, p...) == cudaSuccess ? PKV_OK : cuda_failed();
}

template <int DT>
pkv_status launch_append_f8(const AppendF8Params& p, unsigned grid, cudaStream_t s) {
  const bool rope = p.rp.rope.rot > 0;
  if (p.rp.head_dim == 64)
    return launch_early(rope ? pkv_append_f8_kernel<DT, 64, true> : pkv_append_f8_kernel<DT, 64, false>, grid, 256, 0,
                        s, p);
  return launch_early(rope ? pkv_append_f8_kernel<DT, 128, true> : pkv_append_f8_kernel<DT, 128, false>, grid, 256, 0,
                      s, p);
}

// paged_kv_append_fp8 and paged_kv_append_rope_fp8 (rot_dim 0: no rotation, no queries).
pkv_status append_f8(const RopeAppendParams& rp, pkv_dtype dtype, uint8_t* kv_cache, float* kv_scales,
                     cudaStream_t s) {
  if (rp.num_tokens == 0) return PKV_OK;
  if (!kv_cache || !kv_scales || !aligned16(kv_cache) || (reinterpret_cast<uintptr_t>(kv_scales) & 7u))
    return PKV_ERR_INVALID_ARG;
  DeviceInfo di;
  if (device_info(&di) != PKV_OK) return PKV_ERR_CUDA;
  AppendF8Params p;
  p.rp = rp;
  p.kv = kv_cache;
  p.scales = kv_scales;
  // A token a pair of warps while all of them fit the device at once (a decode
  // step: every token its own run); else 16, so that a prompt's warps are not
  // mostly ones without a run start.  (64 single tokens, 32/8 heads: 4.3 us,
  // 36.7 with 16; 16384 prompt tokens, 8 heads: 20.8 us, 117 with one.)  Steps of
  // many sequences come out on the wrong side of it, 16 runs behind one another
  // in a pair: 310 single tokens, 8 heads, 37.8 us, 9.9 with one; 512, 37.3, 14.3;
  // 256, 32 heads, 40.9, 23.3; at 4096, 8 heads, 66.5, 105.5.
  p.tokens_per_pair = static_cast<int64_t>(rp.num_tokens) * rp.n_kv <= static_cast<int64_t>(di.sm_count) * 16 ? 1 : 16;
  p.token_chunks = (rp.num_tokens + p.tokens_per_pair - 1) / p.tokens_per_pair;
  const int64_t items = static_cast<int64_t>(p.token_chunks) * rp.n_kv * (p.tokens_per_pair == 1 ? 2 : 1);
  const int64_t kv_ctas = (items + 3) / 4;
  const int64_t columns = static_cast<int64_t>(rp.num_tokens) * (rp.head_dim / 16);
  int64_t groups = 0;
  p.q_ctas = static_cast<int32_t>((columns + 255) / 256);
  if (rp.n_q > 0) {
    p.rp.heads_per_thread = rope_heads_per_thread(columns, rp.n_q, di.sm_count);
    groups = (rp.n_q + p.rp.heads_per_thread - 1) / p.rp.heads_per_thread;
  }
  const int64_t grid = kv_ctas + groups * p.q_ctas;
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  p.kv_ctas = static_cast<int32_t>(kv_ctas);
  switch (dtype) {
    case PKV_F32: return launch_append_f8<kF32>(p, static_cast<unsigned>(grid), s);
    case PKV_F16: return launch_append_f8<kF16>(p, static_cast<unsigned>(grid), s);
    default: return launch_append_f8<kBF16>(p, static_cast<unsigned>(grid), s);
  }
}

// Rows of a segment: all rows of a kv head up to 16, else equal parts.  (16 rows,
// 32 x 4 queries: 42.7 us, 52.1 as twice 8; 12 rows, 64 mixed lengths: 67.1,
// 90.6 as twice 6.  4 rows in the kernel of 16: 65.3, 54.5 in that of 8.)
void decode_f8_segments(int total_rows, int* nseg, int* rows) {
  *nseg = (total_rows + 15) / 16;
  *rows = (total_rows + *nseg - 1) / *nseg;
}

// A call's step of the arrivals in its workspace: 1 in the bits from 48 on, below them
// a pseudo-random odd number of 39 bits (its multiples for up to 512 arrivals stay
// below bit 48).  What a workspace held before is taken for arrivals of the call,
// whose word would have to be 0 or a multiple, with a chance of 2^-38 a word.
unsigned long long f8_arrival() {
  static std::atomic<uint64_t> calls{static_cast<uint64_t>(std::chrono::steady_clock::now().time_since_epoch().count())};
  uint64_t x = (calls.fetch_add(1, std::memory_order_relaxed) * 2 + 1) * 0x9e3779b97f4a7c15ull;
  x ^= x >> 32;
  return (1ull << 48) | (x & ((1ull << 39) - 1)) | 1ull;
}

size_t decode_f8_workspace(int sm_count, int rows, int head_dim) {
  const size_t records = static_cast<size_t>(sm_count) * (f8_warps(rows <= 8 ? 1 : 2) + 2);  // a unit's each, two of each CTA
  return kF8HeaderBytes + records * rows * (head_dim + 4) * sizeof(float);
}

template <int D, int NR, bool kBf16>
pkv_status launch_decode_f8(const CUtensorMap& map, DecodeF8Params p, const DeviceInfo& di, cudaStream_t s) {
  auto kern = pkv_decode_f8_kernel<D, NR, kBf16>;
  static bool opted_in[kMaxDevices] = {};
  int dev = 0;
  cudaFuncAttributes fa;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return PKV_ERR_CUDA;
  constexpr int kStatic = 2048;  // more than the kernel's static shared memory
  if (!opted_in[dev]) {
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.sharedSizeBytes > kStatic ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.smem_optin - kStatic) != cudaSuccess)
      return cuda_failed();
    opted_in[dev] = true;
  }
  const size_t smem = f8_smem_bytes(D, NR, p.rows, p.batch);
  if (smem > static_cast<size_t>(di.smem_optin - kStatic)) return PKV_ERR_UNSUPPORTED;
  return launch_early(kern, di.sm_count, f8_warps(NR) * 32, smem, s, map, p);
}

template <bool kBf16>
pkv_status dispatch_decode_f8(int head_dim, const CUtensorMap& map, const DecodeF8Params& p, const DeviceInfo& di,
                              cudaStream_t s) {
  if (head_dim == 64)
    return p.rows <= 8 ? launch_decode_f8<64, 1, kBf16>(map, p, di, s) : launch_decode_f8<64, 2, kBf16>(map, p, di, s);
  return p.rows <= 8 ? launch_decode_f8<128, 1, kBf16>(map, p, di, s) : launch_decode_f8<128, 2, kBf16>(map, p, di, s);
}

}  // namespace
}  // namespace pkv

extern "C" {

pkv_status paged_kv_append_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                int64_t v_stride, const int64_t* positions, const float* cos_sin,
                                int64_t max_positions, int32_t rot_dim, int32_t interleaved,
                                const int64_t* slot_mapping, int32_t num_tokens, void* k_cache, void* v_cache,
                                int32_t num_blocks, int32_t block_size, int32_t n_q_heads, int32_t n_kv_heads,
                                int32_t head_dim, void* q_out, int64_t q_out_stride, pkv_dtype dtype, void* stream) {
  if (rot_dim == 0) return PKV_ERR_INVALID_ARG;
  RopeAppendParams p;
  const pkv_status st =
      rope_append_params(q, q_stride, k, k_stride, v, v_stride, dtype, positions, cos_sin, max_positions, rot_dim,
                         interleaved, slot_mapping, num_tokens, num_blocks, block_size, n_q_heads, n_kv_heads,
                         head_dim, q_out, q_out_stride, &p);
  if (st != PKV_OK || num_tokens == 0) return st;
  if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_INVALID_ARG;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  DeviceInfo di;
  if (device_info(&di) != PKV_OK) return PKV_ERR_CUDA;
  const int heads = n_q_heads + 2 * n_kv_heads;
  const int64_t columns = static_cast<int64_t>(num_tokens) * (head_dim / 16);
  p.heads_per_thread = rope_heads_per_thread(columns, heads, di.sm_count);
  const int64_t groups = (heads + p.heads_per_thread - 1) / p.heads_per_thread;
  if (groups > 65535) return PKV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>((columns + 255) / 256), static_cast<unsigned>(groups));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case PKV_F32: return launch_early(pkv_append_rope_kernel<kF32>, grid, 256, 0, s, p);
    case PKV_F16: return launch_early(pkv_append_rope_kernel<kF16>, grid, 256, 0, s, p);
    default: return launch_early(pkv_append_rope_kernel<kBF16>, grid, 256, 0, s, p);
  }
}

pkv_status paged_kv_append_fp8(const void* k, int64_t k_stride, const void* v, int64_t v_stride, pkv_dtype dtype,
                               const int64_t* slot_mapping, int32_t num_tokens, uint8_t* kv_cache, float* kv_scales,
                               int32_t num_blocks, int32_t block_size, int32_t n_kv_heads, int32_t head_dim,
                               void* stream) {
  RopeAppendParams p;
  const pkv_status st =
      rope_append_params(nullptr, 0, k, k_stride, v, v_stride, dtype, nullptr, nullptr, 0, 0, 0, slot_mapping,
                         num_tokens, num_blocks, block_size, 0, n_kv_heads, head_dim, nullptr, 0, &p);
  if (st != PKV_OK) return st;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  return append_f8(p, dtype, kv_cache, kv_scales, static_cast<cudaStream_t>(stream));
}

pkv_status paged_kv_append_rope_fp8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                    int64_t v_stride, const int64_t* positions, const float* cos_sin,
                                    int64_t max_positions, int32_t rot_dim, int32_t interleaved,
                                    const int64_t* slot_mapping, int32_t num_tokens, uint8_t* kv_cache,
                                    float* kv_scales, int32_t num_blocks, int32_t block_size, int32_t n_q_heads,
                                    int32_t n_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_stride,
                                    pkv_dtype dtype, void* stream) {
  if (rot_dim == 0) return PKV_ERR_INVALID_ARG;
  RopeAppendParams p;
  const pkv_status st =
      rope_append_params(q, q_stride, k, k_stride, v, v_stride, dtype, positions, cos_sin, max_positions, rot_dim,
                         interleaved, slot_mapping, num_tokens, num_blocks, block_size, n_q_heads, n_kv_heads,
                         head_dim, q_out, q_out_stride, &p);
  if (st != PKV_OK) return st;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  return append_f8(p, dtype, kv_cache, kv_scales, static_cast<cudaStream_t>(stream));
}

pkv_status paged_kv_copy_blocks_fp8(uint8_t* kv_cache, float* kv_scales, const int32_t* src_blocks,
                                    const int32_t* dst_blocks, int32_t n_pairs, int32_t num_blocks,
                                    int32_t block_size, int32_t n_kv_heads, int32_t head_dim, void* stream) {
  if (n_pairs < 0 || num_blocks <= 0 || block_size <= 0 || n_kv_heads <= 0 || head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (block_size != kBlockTokens || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  if (n_pairs == 0) return PKV_OK;
  if (!kv_cache || !kv_scales || !src_blocks || !dst_blocks || !aligned16(kv_cache) ||
      (reinterpret_cast<uintptr_t>(kv_scales) & 7u) || (reinterpret_cast<uintptr_t>(src_blocks) & 3u) ||
      (reinterpret_cast<uintptr_t>(dst_blocks) & 3u))
    return PKV_ERR_INVALID_ARG;
  const int64_t chunks = static_cast<int64_t>(n_kv_heads) * f8_tile_bytes(head_dim) / 16;
  if (chunks > INT32_MAX - 1024) return PKV_ERR_UNSUPPORTED;
  DeviceInfo di;
  if (device_info(&di) != PKV_OK) return PKV_ERR_CUDA;
  const CopyF8Params p = {kv_cache,   kv_scales, src_blocks, dst_blocks, n_pairs,
                          num_blocks, static_cast<int32_t>(chunks), 2 * n_kv_heads};
  const int grid = n_pairs < di.sm_count * 8 ? n_pairs : di.sm_count * 8;
  pkv_copy_blocks_f8_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status paged_attention_fp8_workspace_size(int32_t batch, int32_t q_len, int32_t n_q_heads, int32_t n_kv_heads,
                                              int32_t head_dim, size_t* bytes) {
  if (!bytes || batch < 0 || q_len < 1 || n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads != 0)
    return PKV_ERR_INVALID_ARG;
  if (q_len > 16 || batch > PKV_MAX_BATCH || (head_dim != 64 && head_dim != 128)) return PKV_ERR_UNSUPPORTED;
  DeviceInfo di;
  if (device_info(&di) != PKV_OK) return PKV_ERR_CUDA;
  // Calls with fewer rows can need more (8 rows: 16 warps a CTA, 9 rows: 8): the
  // most that any of them does, so that a size serves smaller q_len and groups too.
  const int64_t total_rows = static_cast<int64_t>(n_q_heads / n_kv_heads) * q_len;
  *bytes = 0;
  for (int total = 1; total <= (total_rows < 16 ? static_cast<int>(total_rows) : 16); ++total) {
    int nseg, rows;
    decode_f8_segments(total, &nseg, &rows);
    const size_t need = decode_f8_workspace(di.sm_count, rows, head_dim);
    if (need > *bytes) *bytes = need;
  }
  return PKV_OK;
}

pkv_status paged_attention_decode_fp8(const void* q, const uint8_t* kv_cache, const float* kv_scales,
                                      const int32_t* block_tables, int32_t max_blocks_per_seq,
                                      const int32_t* context_lens, int32_t batch, int32_t q_len, int32_t num_blocks,
                                      float scale, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                      int32_t block_size, void* out, pkv_dtype dtype, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  return paged_attention_decode_fp8_ex(q, kv_cache, kv_scales, block_tables, max_blocks_per_seq, context_lens, batch,
                                       q_len, num_blocks, scale, n_q_heads, n_kv_heads, head_dim, block_size, out,
                                       dtype, workspace, workspace_bytes, stream, nullptr);
}

pkv_status paged_attention_decode_fp8_ex(const void* q, const uint8_t* kv_cache, const float* kv_scales,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t batch, int32_t q_len, int32_t num_blocks,
                                         float scale, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                         int32_t block_size, void* out, pkv_dtype dtype, void* workspace,
                                         size_t workspace_bytes, void* stream, const pkv_decode_options* options) {
  pkv_status st = check_decode_args(q, kv_cache, kv_cache, block_tables, max_blocks_per_seq, context_lens, batch,
                                    num_blocks, scale, n_q_heads, n_kv_heads, head_dim, block_size, out, dtype);
  if (st != PKV_OK) return st;
  if (q_len < 1) return PKV_ERR_INVALID_ARG;
  if (q_len > 16 || dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
  pkv_decode_options opt = {};
  if (options) opt = *options;
  if (opt.num_units || opt.force_simt || opt.balance_chunks || opt.static_permille || opt.wait_limit_us < 0 ||
      opt.test_withhold_unit < 0 || opt.reserved[0] || opt.reserved[1])
    return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!kv_scales || (reinterpret_cast<uintptr_t>(kv_scales) & 7u)) return PKV_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_blocks) * n_kv_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;  // a TMA coordinate
  DeviceInfo di;
  if (device_info(&di) != PKV_OK) return PKV_ERR_CUDA;
  if (static_cast<size_t>(di.sm_count) * sizeof(unsigned long long) > kF8HeaderBytes) return PKV_ERR_UNSUPPORTED;
  DecodeF8Params p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.scales = reinterpret_cast<const float2*>(kv_scales);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.batch = batch;
  p.num_blocks = num_blocks;
  p.n_q_heads = n_q_heads;
  p.n_kv_heads = n_kv_heads;
  p.q_len = q_len;
  p.group = n_q_heads / n_kv_heads;
  p.total_rows = p.group * q_len;
  decode_f8_segments(p.total_rows, &p.nseg, &p.rows);
  p.ng = n_kv_heads * p.nseg;
  if (static_cast<int64_t>(batch) * (max_blocks_per_seq + f8_seg_slots(2)) * p.ng > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  p.rec_floats = p.rows * (head_dim + 4);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = opt.wait_limit_us > 0 ? static_cast<uint64_t>(opt.wait_limit_us) * 1000u : kWaitLimitNs;
  p.withhold_unit = opt.test_withhold_unit - 1;

  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t need = decode_f8_workspace(di.sm_count, p.rows, head_dim);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (ws && (workspace_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u))) return PKV_ERR_WORKSPACE;
  CUtensorMap map;
  st = cached_map(kMapF8, &map, kv_cache, dtype, num_blocks, n_kv_heads, head_dim);
  if (st != PKV_OK) return st;
  const bool own = ws == nullptr;
  if (own) {
    void* at = nullptr;
    if (cudaMallocAsync(&at, need, s) != cudaSuccess) return cuda_failed();
    ws = static_cast<uint8_t*>(at);
  }
  p.arrivals = reinterpret_cast<unsigned long long*>(ws);
  p.arrival = f8_arrival();
  p.unit_recs = reinterpret_cast<float*>(ws + kF8HeaderBytes);
  p.cta_recs = p.unit_recs + static_cast<size_t>(di.sm_count) * f8_warps(p.rows <= 8 ? 1 : 2) * p.rec_floats;
  st = dtype == PKV_BF16 ? dispatch_decode_f8<true>(head_dim, map, p, di, s)
                         : dispatch_decode_f8<false>(head_dim, map, p, di, s);
  if (own && cudaFreeAsync(ws, s) != cudaSuccess) {
    const pkv_status failed = cuda_failed();
    if (st == PKV_OK) st = failed;
  }
  return st;
}

}  // extern "C"
