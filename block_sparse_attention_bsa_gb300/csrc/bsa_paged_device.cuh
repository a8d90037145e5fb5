// Device code that the attention over bf16 pages and the one over 4-bit pages share:
// waits of whole warps, divisions by fixed numbers, and the join of partial results.
#pragma once

#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "bsa_join.h"
#include "bsa_ptx.cuh"

namespace bsa {
namespace {

// Division by a fixed divisor: n / d = (umulhi(n, mul) + n) >> shift for
// 0 <= n < 2^31 (Granlund and Montgomery, Division by invariant integers
// using multiplication).
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int quot(int n) const { return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift); }
};
FastDiv fast_div(uint32_t d) {
  uint32_t shift = 0;
  while ((1ull << shift) < d) ++shift;
  return FastDiv{d, (uint32_t)((((1ull << shift) - d) << 32) / d + 1), shift};
}

__device__ __forceinline__ int warp_inclusive_sum(int v) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Orders this thread's shared-memory writes before later reads by the async
// proxy (the MMAs read Q and V through it).
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// For a kernel that reads what earlier ones have written with no griddepcontrol.wait of
// its own before it, but behind a kernel that has waited for them.  PTX gives a launch
// that is let in early no more than leave to run, so the order is made on both sides:
// in front the thread that lets the next kernel in passes this between its wait and
// that instruction (no path may come to it without the wait), and behind it whoever
// reads passes it before, or stands behind a barrier with a thread that has.
__device__ __forceinline__ void fence_waited() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

// 32 bytes, a whole sector, to a 32-byte aligned address.
__device__ __forceinline__ void store_32(void* dst, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// 1 / (sum of a row's weights), 0 for a row without a key.  Whether it has one
// follows from the lengths: the sum of a row with a NaN or an infinite score is
// NaN, which no comparison with 0 tells from an empty row's, and so is the result.
__device__ __forceinline__ float inverse_sum(bool keyed, float l) { return keyed ? 1.f / l : 0.f; }
// Such a row's log-sum-exp from its largest score (in units of log 2) and its sum.
__device__ __forceinline__ float row_lse(bool keyed, float m, float l) {
  return keyed ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}
// Two values of its output.
__device__ __forceinline__ uint32_t output_pair(float inv_l, float a, float b) {
  return inv_l != 0.f ? pack_bf16x2(a * inv_l, b * inv_l) : 0u;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(e));
  return e != 0;
}

// mbar_wait with one copy of its loop in the code; `bar` and `abort` are
// shared-memory addresses.
__device__ __noinline__ bool wait_loop(uint32_t bar, uint32_t parity, uint32_t abort) {
  return mbar_wait(bar, parity, reinterpret_cast<volatile int*>(__cvta_shared_to_generic(abort)));
}
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, uint32_t abort) {
  return mbar_try_wait(bar, parity) || wait_loop(bar, parity, abort);
}
// The same by all lanes of a warp, with one answer for all of them (what
// follows uses warp-wide instructions).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint32_t abort) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, abort));
}

template <int N>
__device__ __forceinline__ void advance(uint32_t& stage, uint32_t& phase) {
  if (++stage == N) { stage = 0; phase ^= 1u; }
}

// One output row from its partial results, those of a prefix segment and those of
// a segment of own keys.  kLanes lanes of kWarps warps share a row; all lanes of a
// warp come here, also those that have nothing to write.
template <int D, int kLanes, int kWarps>
__device__ __forceinline__ void join_row(const float* part_ml, const float* part_o, const Parts& pre, const Parts& own,
                                         bool write, bool keyed, __nv_bfloat16* out, float* lse) {
  constexpr int kPer = D / kLanes;                 // values per lane, kVec at a time
  constexpr int kVec = kPer < 4 ? kPer : 4;
  constexpr int kLoads = kWarps == 8 ? 4 : kLanes == 32 ? 8 : 2;      // partial rows in flight per lane
  static_assert(kWarps == 1 || kLanes == 32, "several warps take whole rows");
  const int lane = threadIdx.x % kLanes, part = threadIdx.x / 32 % kWarps;
  // Lane x holds the maximum and the sum of partial result base + x; then the
  // rows themselves are read, each warp every kWarps-th of them.
  const int parts = write ? pre.n + own.n : 0;
  const int most = __reduce_max_sync(0xffffffffu, parts);
  float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int base = 0; base < most; base += kLanes) {
    const int x = base + lane;
    const int at = x < pre.n ? pre.at + x * pre.step : own.at + (x - pre.n) * own.step;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (x < parts) ml = reinterpret_cast<const float2*>(part_ml)[at];
    const int here = min(kLanes, most - base);
    // Rows are asked for before their weights are known, one wait less (4-bit pages, one
    // token of one request 9.4 -> 9.2 us, 64 requests on one prompt 35.4 -> 34.6; bf16
    // pages 12.1 -> 11.9, 45.7 -> 44.7).  Not where four rows share a warp, whose many
    // loads are in each other's way (256 samples of one prompt 156 -> 158, 177 -> 179).
    constexpr bool kFirst = kLanes == 32;
    float o[kLoads][kPer], wy[kLoads];
    auto fetch = [&](int y0) {
#pragma unroll
      for (int z = 0; z < kLoads; ++z) {
        const int y = y0 + z * kWarps;
        const float* src = part_o + (int64_t)__shfl_sync(0xffffffffu, at, y % kLanes, kLanes) * D + lane * kVec;
        const bool real = kFirst ? y < kLanes && base + y < parts : wy[z] > 0.f;
#pragma unroll
        for (int v = 0; v < kPer / kVec; ++v) {
          if constexpr (kVec == 4) {
            const float4 f = real ? *reinterpret_cast<const float4*>(src + v * kLanes * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
            o[z][4 * v] = f.x; o[z][4 * v + 1] = f.y; o[z][4 * v + 2] = f.z; o[z][4 * v + 3] = f.w;
          } else {
            const float2 f = real ? *reinterpret_cast<const float2*>(src + v * kLanes * 2) : make_float2(0.f, 0.f);
            o[z][2 * v] = f.x; o[z][2 * v + 1] = f.y;
          }
        }
      }
    };
    if (kFirst) fetch(part);
    float m2 = fmaxf(m, ml.x);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    const float a = m == -INFINITY ? 0.f : ex2_approx(m - m2), w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - m2);
    float sum = ml.y * w;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    m = m2;
    l = l * a + sum;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= a;
#pragma unroll 1
    for (int y0 = part; y0 < here; y0 += kWarps * kLoads) {
      // a group without a tile, or a row without a key there, has left no row
#pragma unroll
      for (int z = 0; z < kLoads; ++z) {
        const int y = y0 + z * kWarps;
        wy[z] = __shfl_sync(0xffffffffu, w, y % kLanes, kLanes);
        if (y >= here) wy[z] = 0.f;
      }
      if (!kFirst || y0 > part) fetch(y0);
#pragma unroll
      for (int z = 0; z < kLoads; ++z)
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(!kFirst || wy[z] > 0.f ? o[z][e] : 0.f, wy[z], acc[e]);
    }
  }
  if constexpr (kWarps > 1) {
    __shared__ float so[kWarps][D];    // m and l are the same in all warps
#pragma unroll
    for (int e = 0; e < kPer; ++e) so[part][lane * kPer + e] = acc[e];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      float o = so[0][lane * kPer + e];
#pragma unroll
      for (int x = 1; x < kWarps; ++x) o += so[x][lane * kPer + e];
      acc[e] = o;
    }
  }
  if (!write) return;
  const float inv_l = inverse_sum(keyed, l);
  __nv_bfloat16* dst = out + lane * kVec;
#pragma unroll
  for (int v = 0; v < kPer / kVec; ++v) {
    uint32_t pk[kVec / 2];
#pragma unroll
    for (int e = 0; e < kVec / 2; ++e)
      pk[e] = output_pair(inv_l, acc[v * kVec + 2 * e], acc[v * kVec + 2 * e + 1]);
    if constexpr (kVec == 4)
      *reinterpret_cast<uint2*>(dst + v * kLanes * 4) = make_uint2(pk[0], pk[1]);
    else
      *reinterpret_cast<uint32_t*>(dst + v * kLanes * 2) = pk[0];
  }
  if (lane == 0 && lse) *lse = row_lse(keyed, m, l);
}

}  // namespace
}  // namespace bsa
