// Host- and device-side declarations of the 4-bit cache calls.
#pragma once

#include <cuda_bf16.h>

#include "../../include/bsa_quant.h"
#include "bsa_paged.h"

namespace bsa {

unsigned int read_and_clear_quant_error();        // append and read
unsigned int read_and_clear_quant_attn_error();
bsa_status launch_quant_wait_probe(unsigned long long limit_ns, cudaStream_t stream);

constexpr int kGroup = 32;                        // channels that share a scale
constexpr int kBlockSlots = 16;
// Bytes of a block of 16 slots of one head: codes and scales.
__host__ __device__ constexpr int code_bytes(int D) { return kBlockSlots * D / 2; }
__host__ __device__ constexpr int block_bytes(int D) { return code_bytes(D) + kBlockSlots * D / kGroup; }

// The two caches and their tables, checked.
struct QuantArgs {
  bsaq_cache k, v;
  const int32_t* page_table; int64_t table_stride; int max_pages;
  const int32_t* kv_lens;
};
// Attention of many rows over 4-bit pages (bsa_paged.cu): its workspace, and the
// launch for arguments that bsaq_forward has checked.
size_t wide_quant_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t d, bool prefix, int sms);
bsa_status launch_wide_quant(const bsa_tensor& q, const QuantArgs& a, const int32_t* new_lens, const int32_t* prefix_table,
                             int32_t prefix_len, int32_t causal, float softmax_scale, void* out, float* lse,
                             void* workspace, cudaStream_t stream);
// The same kernel for the prefix alone, whose partial results the narrow kernel's
// join reads: row tiles of the batch under a KV head (256 rows each; 0 where the
// prefix goes with the requests' own keys), rows of a partial result, and of all.
struct PrefixPart {
  int rt, slot_rows;
  size_t rows;
};
constexpr int kWideRows = 256, kWideHalf = 128;
PrefixPart prefix_part(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t d, int sms);
// The kernel launched behind it may start beside it, and waits for it at its end.
bsa_status launch_prefix_quant(const bsa_tensor& q, const QuantArgs& a, const int32_t* new_lens,
                               const int32_t* prefix_table, int32_t prefix_len, float softmax_scale, void* seg_ctas,
                               float* part_ml, float* part_o, cudaStream_t stream);
bsa_status check_quant(const char* fn, const bsaq_cache* k_cache, const bsaq_cache* v_cache,
                       const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                       int64_t B, QuantArgs* a);
Bytes bytes_of(const char* name, const bsaq_cache& c);

#ifdef __CUDACC__
// ---- the format on the device ----

// Twice a scale, as bf16 bits (NaN for 255).  The byte's eight bits stand in a
// bf16's exponent and mantissa as they are, shifted; 15 becomes 127.
__device__ __forceinline__ uint32_t twice_scale(uint32_t b) { return b == 255u ? 0x7FFFu : (b << 4) + 0x3880u; }

// The codes of two neighbours from bits 4 i of a word: the four bits below the
// exponent of 8.0 are 8 + (c + 8) / 2 in bf16.  `eights`: 8.0 twice, kEights; where
// it is a kernel parameter, not a constant, the two masks are one instruction (as
// constants of one instruction they became two: 16 x 8,192 keys 53 -> 45 us).
constexpr uint32_t kEights = 0x41004100u;
__device__ __forceinline__ uint32_t raised_codes(uint32_t word, int i, uint32_t eights) {
  const uint32_t at = i == 0 ? word << 3 : word >> (4 * i - 3);
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(at), "n"(0x00780078), "r"(eights));      // (at & mask) | eights
  return r;
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Two values c s from raised codes and twice their scales: (8 + (c + 8) / 2 - 12)
// 2 s.  12 times twice a scale has six significant bits and the result seven, so
// that one multiply-add gives it without a rounding.
__device__ __forceinline__ uint32_t code_values(uint32_t raised, uint32_t scales2, uint32_t offset) {
  return as_u32(__hfma2(as_bf16x2(raised), as_bf16x2(scales2), as_bf16x2(offset)));
}
__device__ __forceinline__ uint32_t scale_offset(uint32_t scales2) {
  return as_u32(__hmul2(as_bf16x2(scales2), as_bf16x2(0xC140C140u)));        // times -12
}
// A scale times 2^n (255 is not told apart).
__device__ __forceinline__ float scale_float(uint32_t b, int n) { return __uint_as_float((b << 20) + ((112u + n) << 23)); }

// The codes of eight neighbours in a word, without their scale: r[i] are those of
// numbers 2 i and 2 i + 1, divided by 64 where i is even and by 8 where it is odd.
// Four bits at the foot of a bf16, or four bits higher with the lowest one of its
// exponent among them, are (c + 8) 2^-133 and (c + 8) 2^-129: numbers below and just
// above the border of the subnormal ones are equally spaced.  One mask each, where
// numbers that carry their exponent take a shift, too.
__device__ __forceinline__ void bare_codes(uint32_t word, uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? word : word >> 8;
    r[i] = i % 2 == 0 ? as_u32(__hfma2(as_bf16x2(w & 0x000F000Fu), as_bf16x2(0x7F007F00u), as_bf16x2(0xBE00BE00u)))    // 2^127, -1/8
                      : as_u32(__hfma2(as_bf16x2(w & 0x00F000F0u), as_bf16x2(0x7E807E80u), as_bf16x2(0xBF80BF80u)));   // 2^126, -1
  }
}

// A segment's way in and out in the kernel of few rows, in tiles.
constexpr int kSegmentWay = 1;

// SMs of `sms` that the prefix gets where its tiles (of rows above 128 or not) and own
// tiles (and ways) of few rows are two kernels side by side, in pairs of SMs.  1.75 and
// 1.0 are the times of a prefix's tile in us.  0.42 is not that of an own tile, which is
// 0.56 for 4 rows of heads of 128 (and others for other rows and heads, not told apart
// here): it was chosen by the times of whole calls, 0.62 taking 3 us more for 64 requests
// on one prompt of 8,209 keys and for 256 samples of one of 32,768.  It has to stand in
// for what is not counted, the way in and out of the prefix's segments; shapes in between
// are up to a sixth slower than at their best split (64 requests on 1,200 keys 25.8 to 30
// us by where the cut falls).  Results do not depend on it.
__device__ __forceinline__ int prefix_sms(int sms, int prefix_tiles, bool two_jobs, int own_tiles) {
  if (own_tiles == 0) return sms;
  const float w = (float)prefix_tiles * (two_jobs ? 1.75f : 1.0f), o = (float)own_tiles * 0.42f;
  const int pair = sms % 2 == 0 ? 2 : 1;
  return max(min((int)((float)(sms / pair) * w / (w + o) + 0.5f) * pair, sms - pair), pair);
}

// Shared memory by its address.
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint2 v) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t* r) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t v) {
  asm volatile("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tst.shared.b16 [%0], lo;\n\t}" ::"r"(addr), "r"(v) : "memory");
}
#endif

}  // namespace bsa
