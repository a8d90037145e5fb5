// Attention of new tokens over a paged key/value cache whose first prefix_len
// keys all requests share.
//
// Mathematics: row i of request b and query head h sees the prefix keys and
// its request's own keys up to a limit; out = sum_j e^{z_j} v_j / sum_j
// e^{z_j}, computed over any split of the keys as partial (max, sum, sum of
// v) triples that are joined by rescaling to the common maximum.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "bsa_paged.h"
#include "bsa_ptx.cuh"

namespace bsa {
namespace {

struct PagedParams {
  const __nv_bfloat16* q;
  int64_t q_sb, q_ss, q_sh;
  const __nv_bfloat16* k; int64_t k_sp, k_ss, k_sh;
  const __nv_bfloat16* v; int64_t v_sp, v_ss, v_sh;
  int B, T, Hq, Hkv, G, page_shift, num_pages, max_pages, prefix_len, causal;
  const int32_t* page_table; int64_t table_stride;
  const int32_t* kv_lens; const int32_t* new_lens;
  const int32_t* prefix_table;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
};

// Request b's own keys and new tokens, clamped to what the tables hold.
__device__ __forceinline__ int own_keys(const PagedParams& p, int b) {
  if (p.max_pages == 0) return 0;
  const int kv = __ldg(p.kv_lens + b), most = p.max_pages << p.page_shift;
  return min(max(kv, 0), most);
}
__device__ __forceinline__ int new_tokens(const PagedParams& p, int b) {
  return p.new_lens ? min(max(__ldg(p.new_lens + b), 0), p.T) : p.T;
}

// One block of four warps per output row; each warp takes every fourth key.
template <int D>
__global__ void __launch_bounds__(128) paged_rows_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kPer = D / 32;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t row = blockIdx.x;                 // (b * T + i) * Hq + h
  const int h = (int)(row % p.Hq);
  const int64_t bt = row / p.Hq;
  const int b = (int)(bt / p.T), i = (int)(bt % p.T), hk = h / p.G;
  const int n = new_tokens(p, b), kv = own_keys(p, b);
  if (threadIdx.x == 0 && i == 0 && p.max_pages > 0 && (p.kv_lens[b] < 0 || p.kv_lens[b] > p.max_pages << p.page_shift))
    atomicOr(&g_bsa_error, kErrPage);
  const int own = i >= n ? 0 : (p.causal ? max(min(kv - n + i + 1, kv), 0) : kv);
  const int total = i >= n ? 0 : p.prefix_len + own;
  float q[kPer], acc[kPer], m = -INFINITY, l = 0.f;
  const __nv_bfloat16* qr = p.q + b * p.q_sb + i * p.q_ss + h * p.q_sh + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q[e] = __bfloat162float(qr[e]);
    acc[e] = 0.f;
  }
  for (int j = warp; j < total; j += 4) {
    const int32_t* table = j < p.prefix_len ? p.prefix_table : p.page_table + b * p.table_stride;
    const int jj = j < p.prefix_len ? j : j - p.prefix_len;
    const int page = __ldg(table + (jj >> p.page_shift)), slot = jj & ((1 << p.page_shift) - 1);
    const bool there = page >= 0 && page < p.num_pages;
    if (!there && lane == 0) atomicOr(&g_bsa_error, kErrPage);
    const __nv_bfloat16* kr = p.k + page * p.k_sp + slot * p.k_ss + hk * p.k_sh + lane * kPer;
    const __nv_bfloat16* vr = p.v + page * p.v_sp + slot * p.v_ss + hk * p.v_sh + lane * kPer;
    float z = 0.f, vv[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      z = fmaf(q[e], there ? __bfloat162float(kr[e]) : 0.f, z);
      vv[e] = there ? __bfloat162float(vr[e]) : 0.f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z *= p.scale_log2;
    const float m2 = fmaxf(m, z), a = exp2f(m - m2), w = exp2f(z - m2);
    m = m2;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * a + w * vv[e];
  }
  __shared__ float sm[4], sl[4], so[4][D];
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
  for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < D) {
    const float mm = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float o = 0.f, ll = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float a = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - mm);
      o += a * so[w][threadIdx.x];
      ll += a * sl[w];
    }
    p.out[row * D + threadIdx.x] = __float2bfloat16_rn(ll > 0.f ? o / ll : 0.f);
    if (threadIdx.x == 0 && p.lse)
      p.lse[((int64_t)b * p.Hq + h) * p.T + i] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
  }
}

std::string s(int64_t v) { return std::to_string(v); }

}  // namespace

unsigned int read_and_clear_paged_error() { return take_error_word(); }

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsap_forward_workspace_size(int B, int T, int Hq, int Hkv, int d, int has_prefix, int num_sms) {
  (void)has_prefix; (void)num_sms;
  if (B <= 0 || B > kMaxPagedBatch || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || (d != 64 && d != 128)) return 0;
  return 256;
}

bsa_status bsap_forward(const bsa_tensor* q, const bsa_tensor* k_cache, const bsa_tensor* v_cache,
                        const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                        const int32_t* new_lens, const int32_t* prefix_table, int32_t prefix_len, int32_t causal,
                        float softmax_scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                        bsa_stream_t stream) {
  clear_error();
  const char* fn = "bsap_forward";
  bsa_tensor qv{};
  PagedArgs a{};
  bsa_status st = check_view(q, fn, "q", false, &qv);
  if (st != BSA_OK) return st;
  if ((st = check_paged(fn, k_cache, v_cache, page_table, table_stride, max_pages, kv_lens, new_lens, qv.B, &a)) !=
      BSA_OK)
    return st;
  if (qv.D != a.k.D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": head dim of q (" + s(qv.D) +
                                              ") != head dim of the cache (" + s(a.k.D) + ")");
  if (qv.H % a.k.H)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": Hq (" + s(qv.H) + ") is not a multiple of Hkv (" +
                                              s(a.k.H) + ")");
  if (prefix_len < 0 || prefix_len > INT32_MAX / 2)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": prefix_len " + s(prefix_len) + " out of range");
  if (prefix_len > 0 && !prefix_table)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": prefix_table is NULL");
  if (!out) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": out is NULL");
  if (reinterpret_cast<uintptr_t>(out) & 15u)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": out is not 16-byte aligned");
  if (!std::isfinite(softmax_scale))
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": softmax_scale is not finite");
  const size_t need = bsap_forward_workspace_size((int)qv.B, (int)qv.S, (int)qv.H, (int)a.k.H, (int)qv.D,
                                                  prefix_len > 0, 0);
  if (!workspace) return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace is NULL (needs " + s(need) + " bytes)");
  if (ws_bytes < need)
    return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace of " + s(ws_bytes) +
                                            " bytes is smaller than the " + s(need) + " bytes needed");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace is not 256-byte aligned");
  PagedParams p{};
  p.q = static_cast<const __nv_bfloat16*>(qv.ptr); p.q_sb = qv.stride_b; p.q_ss = qv.stride_s; p.q_sh = qv.stride_h;
  p.k = static_cast<const __nv_bfloat16*>(a.k.ptr); p.k_sp = a.k.stride_b; p.k_ss = a.k.stride_s; p.k_sh = a.k.stride_h;
  p.v = static_cast<const __nv_bfloat16*>(a.v.ptr); p.v_sp = a.v.stride_b; p.v_ss = a.v.stride_s; p.v_sh = a.v.stride_h;
  p.B = (int)qv.B; p.T = (int)qv.S; p.Hq = (int)qv.H; p.Hkv = (int)a.k.H; p.G = p.Hq / p.Hkv;
  p.page_shift = 4;
  while ((1 << p.page_shift) < a.k.S) ++p.page_shift;
  p.num_pages = (int)a.k.B; p.max_pages = max_pages; p.prefix_len = prefix_len; p.causal = causal ? 1 : 0;
  p.page_table = page_table; p.table_stride = table_stride; p.kv_lens = kv_lens; p.new_lens = new_lens;
  p.prefix_table = prefix_table;
  p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)qv.D)) * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse;
  const unsigned rows = (unsigned)(qv.B * qv.S * qv.H);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (qv.D == 128) paged_rows_kernel<128><<<rows, 128, 0, cs>>>(p);
  else paged_rows_kernel<64><<<rows, 128, 0, cs>>>(p);
  return cuda_check(cudaGetLastError(), "paged_rows_kernel launch");
}

}  // extern "C"
