// Attention of new tokens over a paged key/value cache held in 4 bits, whose
// first prefix_len keys all requests share.
//
// Mathematics: that of bsa_paged.cu, with k_j and v_j = codes times scales of
// their groups of 32 channels (bsa_quant.h).
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <string>

#include "bsa_ptx.cuh"
#include "bsa_quant.h"

namespace bsa {
namespace {

struct QAttnParams {
  const uint8_t* k; const uint8_t* v;
  int64_t k_page, k_head, v_page, v_head;      // byte strides
  const __nv_bfloat16* q;
  int64_t q_sb, q_ss, q_sh;
  int B, T, Hq, Hkv, G, blocks_shift, num_pages, max_pages, prefix_len, causal;
  const int32_t* page_table; int64_t table_stride;
  const int32_t* kv_lens; const int32_t* new_lens;
  const int32_t* prefix_table;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
};

// Channel c of slot i of a block: K by slot, V by channel.
template <int D, bool kV>
__device__ __forceinline__ float held(const uint8_t* block, int i, int c) {
  const int number = kV ? i : c % kGroup;
  const int base = kV ? c * 8 : (c / kGroup * kBlockSlots + i) * (kGroup / 2);
  const uint32_t word = *reinterpret_cast<const uint32_t*>(block + base + number / 8 * 4);
  const int code = (int)((word >> (4 * (number % 8 / 2) + 16 * (number % 2))) & 15u) - 8;
  const uint32_t s2 = twice_scale(block[code_bytes(D) + c / kGroup * kBlockSlots + i]);
  return (float)code * 0.5f * __uint_as_float(s2 << 16);
}

// Block: token i of request b under one KV head; four warps take every fourth key.
template <int D>
__global__ void __launch_bounds__(128) quant_attention_kernel(const __grid_constant__ QAttnParams p) {
  constexpr int kPer = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int i = blockIdx.x, hk = blockIdx.y, b = blockIdx.z;
  const int n = p.new_lens ? min(max(p.new_lens[b], 0), p.T) : p.T;
  int kv = 0;
  if (p.max_pages > 0) {
    kv = p.kv_lens[b];
    if (threadIdx.x == 0 && (kv < 0 || kv > p.max_pages << (4 + p.blocks_shift))) atomicOr(&g_bsa_error, kErrPage);
    kv = min(max(kv, 0), p.max_pages << (4 + p.blocks_shift));
  }
  const int own = p.causal ? min(max(kv - n + i + 1, 0), kv) : kv;
  const int keys = i < n ? p.prefix_len + own : 0;
  for (int g = 0; g < p.G; ++g) {
    const int h = hk * p.G + g;
    float q[kPer], o[kPer] = {}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < kPer; ++e)
      q[e] = __bfloat162float(p.q[b * p.q_sb + i * p.q_ss + h * p.q_sh + lane * kPer + e]);
    for (int j = warp; j < keys; j += 4) {
      const bool pre = j < p.prefix_len;
      const int key = pre ? j : j - p.prefix_len;
      const int32_t* table = pre ? p.prefix_table : p.page_table + b * p.table_stride;
      int page = table[key >> (4 + p.blocks_shift)];
      if (page < 0 || page >= p.num_pages) {
        if (lane == 0) atomicOr(&g_bsa_error, kErrPage);
        continue;
      }
      const int64_t in_page = ((key >> 4) & ((1 << p.blocks_shift) - 1)) * block_bytes(D);
      const uint8_t* kb = p.k + page * p.k_page + hk * p.k_head + in_page;
      const uint8_t* vb = p.v + page * p.v_page + hk * p.v_head + in_page;
      float z = 0.f;
      for (int e = 0; e < kPer; ++e) z = fmaf(q[e], held<D, false>(kb, key & 15, lane * kPer + e), z);
      for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
      z *= p.scale_log2;
      const float m2 = fmaxf(m, z), use = m2 == -INFINITY ? 0.f : m2;
      const float a = m == -INFINITY ? 0.f : exp2f(m - use), w = exp2f(z - use);
      m = m2;
      l = l * a + w;
      for (int e = 0; e < kPer; ++e) o[e] = o[e] * a + w * held<D, true>(vb, key & 15, lane * kPer + e);
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
    for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = o[e];
    __syncthreads();
    if (warp == 0) {
      const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3])), use = top == -INFINITY ? 0.f : top;
      float w[4], sum = 0.f;
      for (int x = 0; x < 4; ++x) { w[x] = exp2f(sm[x] - use); sum += sl[x] * w[x]; }
      const int64_t row = ((int64_t)b * p.T + i) * p.Hq + h;
      for (int e = 0; e < kPer; ++e) {
        float y = 0.f;
        for (int x = 0; x < 4; ++x) y += so[x][lane * kPer + e] * w[x];
        p.out[row * D + lane * kPer + e] = __float2bfloat16(keys > 0 ? y / sum : 0.f);
      }
      if (lane == 0 && p.lse)
        p.lse[((int64_t)b * p.Hq + h) * p.T + i] = keys > 0 ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
    }
    __syncthreads();
  }
}

std::string s(int64_t v) { return std::to_string(v); }

struct QAttnPlan {
  size_t bytes;
};

QAttnPlan plan_quant(int64_t, int64_t, int64_t, int64_t, int64_t, bool, int) { return QAttnPlan{256}; }

}  // namespace

unsigned int read_and_clear_quant_attn_error() { return take_error_word(); }

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsaq_forward_workspace_size(int B, int T, int Hq, int Hkv, int d, int has_prefix, int sms) {
  if (B <= 0 || B > kMaxPagedBatch || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq > kMaxHeads || Hq % Hkv ||
      (d != 64 && d != 128) || sms < 0 || (int64_t)B * T * (Hq / Hkv) > INT32_MAX / 16)
    return 0;
  return plan_quant(B, T, Hq, Hkv, d, has_prefix != 0, sms > 0 ? sms : num_sms()).bytes;
}

bsa_status bsaq_forward(const bsa_tensor* q, const bsaq_cache* k_cache, const bsaq_cache* v_cache,
                        const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                        const int32_t* new_lens, const int32_t* prefix_table, int32_t prefix_len, int32_t causal,
                        float softmax_scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                        bsa_stream_t stream) {
  clear_error();
  const char* fn = "bsaq_forward";
  bsa_tensor qv{};
  QuantArgs a{};
  bsa_status st = check_view(q, fn, "q", false, &qv);
  if (st != BSA_OK) return st;
  if ((st = check_quant(fn, k_cache, v_cache, page_table, table_stride, max_pages, kv_lens, qv.B, &a)) != BSA_OK) return st;
  if ((st = check_aligned(fn, "new_lens", new_lens, 4)) != BSA_OK) return st;
  if (qv.D != a.k.D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": head dim of q (" + s(qv.D) +
                                              ") != head dim of the cache (" + s(a.k.D) + ")");
  if (qv.H % a.k.heads)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": Hq (" + s(qv.H) + ") is not a multiple of Hkv (" +
                                              s(a.k.heads) + ")");
  if (prefix_len < 0 || prefix_len > INT32_MAX / 2)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": prefix_len " + s(prefix_len) + " out of range");
  if (prefix_len > 0 && !prefix_table)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": prefix_table is NULL");
  if (prefix_len > 0 && (st = check_aligned(fn, "prefix_table", prefix_table, 4)) != BSA_OK) return st;
  if (!out) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": out is NULL");
  if ((st = check_aligned(fn, "out", out, 16)) != BSA_OK) return st;
  if ((st = check_aligned(fn, "lse", lse, 4)) != BSA_OK) return st;
  if (!std::isfinite(softmax_scale))
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": softmax_scale is not finite");
  // times -inf and log2(e) on the device, where subnormal numbers may count as 0
  if (softmax_scale > 0.f && (softmax_scale < FLT_MIN || softmax_scale > FLT_MAX / 2))
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": softmax_scale is subnormal or above half the largest float");
  const int64_t G = qv.H / a.k.heads;
  const int sms = num_sms();
  if (qv.B * qv.S * G > INT32_MAX / 16)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(qv.B * qv.S * G) + " rows are too many for one call");
  const QAttnPlan plan = plan_quant(qv.B, qv.S, qv.H, a.k.heads, qv.D, prefix_len > 0, sms);
  const size_t need = plan.bytes;
  if (!workspace) return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace is NULL (needs " + s(need) + " bytes)");
  if (ws_bytes < need)
    return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace of " + s(ws_bytes) +
                                            " bytes is smaller than the " + s(need) + " bytes needed");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace is not 256-byte aligned");
  const bsa_tensor ov = contiguous_like(qv, out);
  // What is written against what other blocks still read.
  const Bytes writes[] = {bytes_of("out", ov), bytes_at("lse", lse, 4 * qv.B * qv.H * qv.S),
                          bytes_at("workspace", workspace, (int64_t)need)};
  const Bytes reads[] = {bytes_of("q", qv), bytes_of("k_cache", a.k), bytes_of("v_cache", a.v),
                         bytes_at("page_table", max_pages ? page_table : nullptr,
                                  4 * ((qv.B - 1) * table_stride + max_pages)),
                         bytes_at("kv_lens", max_pages ? kv_lens : nullptr, 4 * qv.B), bytes_at("new_lens", new_lens, 4 * qv.B),
                         bytes_at("prefix_table", prefix_len ? prefix_table : nullptr,
                                  4 * cdiv64(prefix_len, a.k.blocks * kBlockSlots))};
  for (const Bytes& w : writes)
    for (const Bytes& r : reads)
      if ((st = check_apart(fn, r, w)) != BSA_OK) return st;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(fn, writes[j], writes[i])) != BSA_OK) return st;
  QAttnParams p{};
  p.k = static_cast<const uint8_t*>(a.k.ptr); p.v = static_cast<const uint8_t*>(a.v.ptr);
  p.k_page = a.k.stride_page; p.k_head = a.k.stride_head; p.v_page = a.v.stride_page; p.v_head = a.v.stride_head;
  p.q = static_cast<const __nv_bfloat16*>(qv.ptr); p.q_sb = qv.stride_b; p.q_ss = qv.stride_s; p.q_sh = qv.stride_h;
  p.B = (int)qv.B; p.T = (int)qv.S; p.Hq = (int)qv.H; p.Hkv = (int)a.k.heads; p.G = (int)G;
  while ((1 << p.blocks_shift) < a.k.blocks) ++p.blocks_shift;
  p.num_pages = (int)a.k.pages; p.max_pages = max_pages; p.prefix_len = prefix_len; p.causal = causal ? 1 : 0;
  p.page_table = page_table; p.table_stride = table_stride; p.kv_lens = kv_lens; p.new_lens = new_lens;
  p.prefix_table = prefix_table;
  p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)qv.D)) * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)p.T, (unsigned)p.Hkv, (unsigned)p.B);
  if (qv.D == 128) quant_attention_kernel<128><<<grid, 128, 0, cs>>>(p);
  else quant_attention_kernel<64><<<grid, 128, 0, cs>>>(p);
  return cuda_check(cudaGetLastError(), "quant_attention_kernel launch");
}

}  // extern "C"
