// The paged cache in 4 bits: quantising keys and values as they are written, and
// reading them back to bf16 rows.  The format is described in bsa_quant.h.
//
// Mathematics: s = a / 7 rounded to four bits and c = floor(|x| / s + 1/2) are
// decided exactly without a division per value: x and (n + 1/2) s have 8 significant
// bits each, so that where they differ they differ by 2^-8 of either or more, and
// |x| (1 / s)(1 + 2^-14), with a factor that is right to 2^-21, rounds to the right
// code, ties away from zero.  The sum with 1.5 2^23 + 8 does that rounding and leaves
// the code in the lowest bits, so that a value takes three instructions.  No value of
// a finite group is above 7.44 s, but where s is the largest scale.
//
// Layout of the work: a warp takes a block of 16 slots of a head (two heads of
// 64).  A lane holds 4 channels of all 16 slots, so that the codes of V, which
// stand by channel, are whole words of one lane, and those of K, which stand by
// slot, are exchanged in shared memory.  Both kernels move whole rows and whole
// blocks, in whole sectors of 32 bytes.
//
// Bound by DRAM: 16 requests' 4,096 tokens of 8 heads of 128 are written in 55.8 us
// (340 MB, 90 % of the measured copy rate) and read back in 52.5 us (95 %); 5 of
// 4,099 tokens in 20.1 and 18.3 us, where the way in and out counts 3 us; one token
// each of 64 requests takes 2.7 us.  What it took: the rows are asked for before the
// page is known (a warp waits once instead of twice) and stores of half sectors were
// joined, 66.8 -> 60.4 us; 820 -> 690 instructions a warp (rows stepped through,
// largest magnitudes of half the words at each step of the exchange), 60.4 -> 55.8, and
// 680 -> 420 in reading, 53.4 -> 52.5.
#include <cuda_bf16.h>

#include <cstdint>
#include <string>

#include "bsa_quant.h"

namespace bsa {
namespace {

__device__ unsigned int g_quant_error = 0;

constexpr int kQuantThreads = 128;
constexpr int kStageWords = 4 * 72;   // of a warp: [4 groups][2 halves of 8 slots][8 slots][4 words], padded

struct QuantParams {
  const __nv_bfloat16* x[2];          // append: K and V; read: unused
  __nv_bfloat16* y[2];                // read: K and V
  int64_t sb[2], ss[2], sh[2];        // their strides (elements)
  uint8_t* cache[2];
  int64_t c_page[2], c_head[2];       // byte strides
  int S, H, blocks_shift, num_pages, max_pages, head_groups;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* kv_lens;
  const int32_t* other;               // append: new_lens; read: first
  uint32_t eights;                    // kEights
};

// What one warp works on.
struct Place {
  int b, which, h, l;                 // request, 0 = K, 1 = V, head, lane of its row
  bool active;                        // the head exists
  int64_t t0;                         // token (row) of the block's first slot
  int first, end;                     // slots of the block that count
  int page, in_page;                  // page, block of the page
};

// The block of 16 slots of a warp: rows t = key - from, 0 <= t < n, and the entry of
// the page table that names its page (-1: none).  False where none of its slots counts.
template <int D>
__device__ __forceinline__ bool find_place(const QuantParams& p, int64_t from, int64_t n, Place* w) {
  constexpr int kLanes = D / 4;                        // of a row
  const int lane = threadIdx.x % 32;
  const int wid = blockIdx.x * (kQuantThreads / 32) + threadIdx.x / 32;
  const int blk = wid / p.head_groups;
  w->h = (wid - blk * p.head_groups) * (32 / kLanes) + lane / kLanes;
  w->l = lane % kLanes;
  w->active = w->h < p.H;
  const int64_t pos0 = ((from >> 4) + blk) * 16;       // rounds down where negative, too
  w->t0 = pos0 - from;
  w->first = (int)(w->t0 < 0 ? -w->t0 : 0);
  const int64_t left = n - w->t0;                      // may be below what 32 bits hold
  if (left <= w->first) return false;
  w->end = (int)(left < 16 ? left : 16);
  const int64_t at = pos0 >> (4 + p.blocks_shift);
  w->page = -1;
  if (pos0 >= 0 && at < p.max_pages) w->page = p.page_table[w->b * p.table_stride + at];
  w->in_page = (int)(pos0 >> 4) & ((1 << p.blocks_shift) - 1);
  return true;
}

// Its bytes in the cache; null, and the error noted, where the page is none of it.
template <int D>
__device__ __forceinline__ uint8_t* find_block(const QuantParams& p, const Place& w) {
  if (w.page < 0 || w.page >= p.num_pages) {
    if (threadIdx.x % 32 == 0) atomicOr(&g_quant_error, kErrPage);
    return nullptr;
  }
  return p.cache[w.which] + w.page * p.c_page[w.which] + (w.active ? w.h : 0) * p.c_head[w.which] +
         w.in_page * block_bytes(D);
}

// Where slot i of a group's staged codes begins, in words: the 32 lanes' words of
// one slot (of either half), and a lane's 16-byte pieces, fall on different banks.
__device__ __forceinline__ int stage_at(int group, int slot) { return group * 72 + (slot >> 3) * 36 + (slot & 7) * 4; }

// The larger magnitudes of two pairs of bf16.
__device__ __forceinline__ uint32_t largest2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(__habs2(*reinterpret_cast<__nv_bfloat162*>(&a)), __habs2(*reinterpret_cast<__nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Grid: x = (block, heads), y = request, z = K or V.
template <int D>
__global__ void __launch_bounds__(kQuantThreads) quantise_kernel(const __grid_constant__ QuantParams p) {
  __shared__ __align__(16) uint32_t stage_all[kQuantThreads / 32][kStageWords];
  uint32_t* stage = stage_all[threadIdx.x / 32];
  const int lane = threadIdx.x % 32, l8 = lane % 8, group = lane / 8;
  Place w;
  w.b = blockIdx.y;
  w.which = blockIdx.z;
  // Launched when the blocks of the kernel before leave: nothing it may have
  // written is read before this point.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n = p.other ? min(max(p.other[w.b], 0), p.S) : p.S;
  if (!find_place<D>(p, (int64_t)p.kv_lens[w.b] - n, n, &w)) return;

  // 4 channels of 16 slots (zeros where a slot is not written)
  const uint32_t fresh = w.active ? (1u << w.end) - (1u << w.first) : 0u;
  uint2 x[16];
  const __nv_bfloat16* src = p.x[w.which] + w.b * p.sb[w.which] + w.h * p.sh[w.which] + w.t0 * p.ss[w.which] + w.l * 4;
#pragma unroll
  for (int i = 0; i < 16; ++i, src += p.ss[w.which]) {
    x[i] = make_uint2(0u, 0u);
    if (fresh >> i & 1u) x[i] = *reinterpret_cast<const uint2*>(src);
  }
  // the page has come while those are on their way
  uint8_t* block = find_block<D>(p, w);
  if (!block) return;
  // Largest magnitudes, two slots in a word; NaN stays NaN.
  uint32_t most[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = largest2(x[2 * i].x, x[2 * i].y), b = largest2(x[2 * i + 1].x, x[2 * i + 1].y);
    most[i] = largest2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  }
  // Of eight words a lane gives half away at each step, so that lane l8 of a group's
  // eight ends with word l8: it works out the scales of slots 2 l8 and 2 l8 + 1.
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    const bool upper = l8 & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? most[i] : most[i + o], o);
      most[i] = largest2(upper ? most[i + o] : most[i], got);
    }
  }
  const uint32_t mine = most[0];
  uint32_t byte[2];
  float inv[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t bits = e ? mine >> 16 : mine & 0xFFFFu;
    // a / 7, a quotient and its remainder's (exact where it has few bits)
    const float a = __uint_as_float(bits << 16), near = a * (1.f / 7.f);
    const float seventh = fmaf(fmaf(near, -7.f, a), 1.f / 7.f, near);
    // to four significant bits, ties to even; the bias from 127 to 15
    const uint32_t q = __float_as_uint(seventh);
    const int r = (int)((q + 0x0007FFFFu + ((q >> 20) & 1u)) >> 20) - (112 << 3);
    byte[e] = (uint32_t)min(max(r, 0), 254);
    inv[e] = __fdividef(1.00006103515625f, __uint_as_float((byte[e] << 20) + (112u << 23)));     // 1 + 2^-14
    if (bits >= 0x7F80u) {
      byte[e] = 255u;
      inv[e] = 0.f;
    }
  }
  // Values above 7.5 of their scale are there only where it is the largest one, or
  // where the group is not finite: those are cut to 7 of the largest scale.
  if (__any_sync(0xffffffffu, max(mine >> 16, mine & 0xFFFFu) >= 0x4940u)) {
    const __nv_bfloat162 most7 = __float2bfloat162_rn(802816.f), least7 = __float2bfloat162_rn(-802816.f);   // 7 (1.75) 2^16
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      __nv_bfloat162* v = reinterpret_cast<__nv_bfloat162*>(&x[i]);
      v[0] = __hmax2(__hmin2(v[0], most7), least7);
      v[1] = __hmax2(__hmin2(v[1], most7), least7);
    }
  }
  uint8_t* scales = block + code_bytes(D) + (group % (D / kGroup)) * kBlockSlots;
  // (whole blocks' stores fill whole sectors of 32 bytes each)
  if (fresh == 0xFFFFu) {
    *reinterpret_cast<uint16_t*>(scales + 2 * l8) = (uint16_t)(byte[0] | byte[1] << 8);
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (fresh >> (2 * l8 + e) & 1u) scales[2 * l8 + e] = (uint8_t)byte[e];
  }

  // the group's 16 factors, by way of the stage
  float rs[16];
  reinterpret_cast<float2*>(stage)[lane] = make_float2(inv[0], inv[1]);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(rs + 4 * i) = reinterpret_cast<const float4*>(stage)[group * 4 + i];
  __syncwarp();

  // 1.5 2^23 + 8 + c, whose bits are kRaised + c + 8: words of codes are sums of these.
  // The product is not rounded on its own.
  constexpr uint32_t kRaised = 0x4B400000u;
  auto low = [](uint32_t word, float r) { return __float_as_uint(fmaf(__uint_as_float(word << 16), r, 12582920.f)); };
  auto high = [](uint32_t word, float r) {
    return __float_as_uint(fmaf(__uint_as_float(word & 0xFFFF0000u), r, 12582920.f));
  };
  if (w.which == 0) {
    // K: of eight channels in a word a lane has four, another the other four
    const bool odd = lane & 1;
    uint32_t part[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float r = rs[i];
      const uint32_t u = low(x[i].x, r) + (low(x[i].y, r) << 4) + (high(x[i].x, r) << 16) + (high(x[i].y, r) << 20) -
                         kRaised * (1u + (1u << 4) + (1u << 16) + (1u << 20));
      part[i] = odd ? u << 8 : u;
    }
    const int word = l8 / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? part[i] : part[8 + i], 1);
      stage[stage_at(group, (odd ? 8 : 0) + i) + word] = (odd ? part[8 + i] : part[i]) | got;
    }
    __syncwarp();
    uint4* dst = reinterpret_cast<uint4*>(block + (group % (D / kGroup)) * (kBlockSlots * kGroup / 2));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int slot = 8 * e + l8;
      if (fresh >> slot & 1u) dst[slot] = *reinterpret_cast<const uint4*>(stage + stage_at(group, slot));
    }
  } else {
    // V: 16 slots of a channel are two words; those of slots that are not new stay
    constexpr uint32_t kSum = kRaised * 0x11111111u;
    uint32_t v[4][2] = {{0u - kSum, 0u - kSum}, {0u - kSum, 0u - kSum}, {0u - kSum, 0u - kSum}, {0u - kSum, 0u - kSum}};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float r = rs[i];
      const int at = 4 * (i % 8 / 2) + 16 * (i % 2);
      v[0][i / 8] += low(x[i].x, r) << at;
      v[1][i / 8] += high(x[i].x, r) << at;
      v[2][i / 8] += low(x[i].y, r) << at;
      v[3][i / 8] += high(x[i].y, r) << at;
    }
    uint4* dst = reinterpret_cast<uint4*>(block + w.l * 32);
    if (__all_sync(0xffffffffu, fresh == 0xFFFFu)) {
      // two lanes' 64 bytes, 32 with each store
      const bool odd = lane & 1;
      uint32_t got[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) got[c] = __shfl_xor_sync(0xffffffffu, odd ? v[c / 2][c % 2] : v[2 + c / 2][c % 2], 1);
      const uint4 far = make_uint4(got[0], got[1], got[2], got[3]);
      dst -= odd;
      dst[0] = odd ? far : make_uint4(v[0][0], v[0][1], v[1][0], v[1][1]);
      dst[2] = odd ? make_uint4(v[2][0], v[2][1], v[3][0], v[3][1]) : far;
      return;
    }
    if (!w.active) return;
    uint32_t mask[2] = {0u, 0u};                       // the new ones' bits
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (fresh >> i & 1u) mask[i / 8] |= 15u << (4 * (i % 8 / 2) + 16 * (i % 2));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint4 old = dst[e];
      dst[e] = make_uint4((v[2 * e][0] & mask[0]) | (old.x & ~mask[0]), (v[2 * e][1] & mask[1]) | (old.y & ~mask[1]),
                          (v[2 * e + 1][0] & mask[0]) | (old.z & ~mask[0]),
                          (v[2 * e + 1][1] & mask[1]) | (old.w & ~mask[1]));
    }
  }
}

// The same grid; rows of the block are written.
template <int D>
__global__ void __launch_bounds__(kQuantThreads) read_kernel(const __grid_constant__ QuantParams p) {
  __shared__ __align__(16) uint32_t stage_all[kQuantThreads / 32][kStageWords];
  uint32_t* stage = stage_all[threadIdx.x / 32];
  const int lane = threadIdx.x % 32, l8 = lane % 8, group = lane / 8;
  Place w;
  w.b = blockIdx.y;
  w.which = blockIdx.z;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t from = p.other ? max(p.other[w.b], 0) : 0;
  const int kv = p.kv_lens[w.b];
  if (kv < 0) {                                        // no block of such a request is looked up: said here
    if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(&g_quant_error, kErrPage);
    return;
  }
  const int64_t keys = kv - from;
  if (!find_place<D>(p, from, keys < p.S ? keys : p.S, &w)) return;
  const uint8_t* block = find_block<D>(p, w);
  if (!block) return;

  const uint4* codes = reinterpret_cast<const uint4*>(block + w.l * 32);
  const uint4 c0 = codes[0], c1 = codes[1];
  const uint4 sc = *reinterpret_cast<const uint4*>(block + code_bytes(D) + (group % (D / kGroup)) * kBlockSlots);
  // twice the scales of slots 2 i and 2 i + 1; 255 stands for NaN
  uint32_t scale[8];
  const uint32_t four[4] = {sc.x, sc.y, sc.z, sc.w};
  uint32_t full = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t word = four[i / 2];
    scale[i] = (__byte_perm(word, 0u, i % 2 ? 0x4342 : 0x4140) << 4) + 0x38803880u;
    full |= ((word & 0x7F7F7F7Fu) + 0x01010101u) & word;      // bit 7 of a byte of 255
  }
  if (full & 0x80808080u) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      scale[i] = twice_scale((four[i / 2] >> (16 * (i % 2))) & 255u) | twice_scale((four[i / 2] >> (16 * (i % 2) + 8)) & 255u) << 16;
  }
  const uint32_t wanted = w.active ? (1u << w.end) - (1u << w.first) : 0u;
  __nv_bfloat16* dst = p.y[w.which] + w.b * p.sb[w.which] + w.h * p.sh[w.which] + w.t0 * p.ss[w.which] + w.l * 4;
  auto put = [&](int i, uint32_t lo, uint32_t hi) {    // i = 0 .. 15 in turn
    if (wanted >> i & 1u) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    dst += p.ss[w.which];
  };
  if (w.which == 0) {
    *reinterpret_cast<uint4*>(stage + stage_at(group, 2 * l8)) = c0;
    *reinterpret_cast<uint4*>(stage + stage_at(group, 2 * l8 + 1)) = c1;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t word = stage[stage_at(group, i) + l8 / 2] >> (lane & 1 ? 8 : 0);
      const uint32_t s2 = __byte_perm(scale[i / 2], 0u, i % 2 ? 0x3232 : 0x1010), off = scale_offset(s2);
      put(i, code_values(raised_codes(word, 0, p.eights), s2, off), code_values(raised_codes(word, 1, p.eights), s2, off));
    }
  } else {
    const uint32_t word[4][2] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
    for (int i = 0; i < 16; i += 2) {                  // two slots at a time, then two channels
      const uint32_t s2 = scale[i / 2], off = scale_offset(s2);
      uint32_t v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = code_values(raised_codes(word[c][i / 8], i % 8 / 2, p.eights), s2, off);
      put(i, __byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410));
      put(i + 1, __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
    }
  }
}

std::string s(int64_t v) { return std::to_string(v); }

bsa_status check_cache(const char* fn, const char* name, const bsaq_cache* c, bsaq_cache* view) {
  if (!c) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " descriptor is NULL");
  if (!c->ptr) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + "->ptr is NULL");
  if (c->pages <= 0 || c->heads <= 0 || c->blocks <= 0 || c->D <= 0)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " has a non-positive size [" + s(c->pages) +
                                              "," + s(c->heads) + "," + s(c->blocks) + "], D " + s(c->D));
  if (c->D != 64 && c->D != 128)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": head dim " + s(c->D) + " of " + name +
                                              " is not supported (64 or 128)");
  if (c->heads > kMaxHeads)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(c->heads) + " heads of " + name +
                                              " above the limit " + s(kMaxHeads));
  if (c->blocks > 16 || (c->blocks & (c->blocks - 1)))
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": page size " + s(c->blocks * 16) +
                                              " is not supported (16, 32, 64, 128 or 256)");
  if (c->pages > INT32_MAX / 2 / (c->blocks * 16))
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + name + " has more than 2^30 slots");
  if (reinterpret_cast<uintptr_t>(c->ptr) & 15u)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + "->ptr is not 16-byte aligned");
  *view = *c;
  if (c->pages == 1) view->stride_page = 0;
  if (c->heads == 1) view->stride_head = 0;
  const int64_t unit = c->blocks * block_bytes((int)c->D);
  const int64_t sp = view->stride_page, sh = view->stride_head;
  if (sp % 16 || sh % 16 || sp < 0 || sh < 0)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name +
                                              " strides must be positive multiples of 16 bytes; got " + s(sp) + ", " + s(sh));
  const bool page_inside = c->pages > 1 && c->heads > 1 && sp < sh;
  const bool apart = page_inside ? sp >= unit && sh >= unit + (c->pages - 1) * sp
                                 : (c->heads == 1 || sh >= unit) &&
                                       (c->pages == 1 || sp >= unit + (c->heads - 1) * sh);
  if (!apart) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " blocks overlap");
  return BSA_OK;
}

// Launches a kernel over blocks of up to S rows of every request.
bsa_status launch_blocks(QuantParams& p, int64_t B, int64_t D, const QuantArgs& a, void (*k64)(QuantParams),
                         void (*k128)(QuantParams), const char* what, const char* fn, cudaStream_t stream) {
  p.H = (int)a.k.heads;
  p.eights = kEights;
  p.blocks_shift = 0;
  while ((1 << p.blocks_shift) < a.k.blocks) ++p.blocks_shift;
  p.num_pages = (int)a.k.pages; p.max_pages = a.max_pages;
  p.page_table = a.page_table; p.table_stride = a.table_stride; p.kv_lens = a.kv_lens;
  const bsaq_cache* caches[2] = {&a.k, &a.v};
  for (int i = 0; i < 2; ++i) {
    p.cache[i] = static_cast<uint8_t*>(caches[i]->ptr);
    p.c_page[i] = caches[i]->stride_page; p.c_head[i] = caches[i]->stride_head;
  }
  const int heads = 128 / (int)D;                      // of a warp
  p.head_groups = (int)cdiv64(p.H, heads);
  // S rows that begin anywhere in a block touch (S + 14) / 16 + 1 blocks at most
  const int64_t warps = ((p.S + 14) / 16 + 1) * (int64_t)p.head_groups;
  if (warps > INT32_MAX - kQuantThreads)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(p.S) + " rows of " + s(p.H) + " heads are too many for one call");
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)cdiv64(warps, kQuantThreads / 32), (unsigned)B, 2);
  cfg.blockDim = dim3(kQuantThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, D == 128 ? k128 : k64, p), what);
}

}  // namespace

unsigned int read_and_clear_quant_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_quant_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0 && cudaMemcpyToSymbol(g_quant_error, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

Bytes bytes_of(const char* name, const bsaq_cache& c) {
  return bytes_at(name, c.ptr,
                  (c.pages - 1) * c.stride_page + (c.heads - 1) * c.stride_head + c.blocks * block_bytes((int)c.D));
}

bsa_status check_quant(const char* fn, const bsaq_cache* k_cache, const bsaq_cache* v_cache,
                       const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                       int64_t B, QuantArgs* a) {
  bsa_status st;
  if ((st = check_cache(fn, "k_cache", k_cache, &a->k)) != BSA_OK) return st;
  if ((st = check_cache(fn, "v_cache", v_cache, &a->v)) != BSA_OK) return st;
  if (a->k.pages != a->v.pages || a->k.heads != a->v.heads || a->k.blocks != a->v.blocks || a->k.D != a->v.D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": v_cache shape differs from k_cache shape");
  if (B > kMaxPagedBatch)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": batch " + s(B) + " above the limit " + s(kMaxPagedBatch));
  if (max_pages < 0 || max_pages > INT32_MAX / 2 / (a->k.blocks * 16))
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": max_pages " + s(max_pages) + " out of range");
  if (max_pages > 0) {
    if (!page_table || !kv_lens)
      return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": page_table and kv_lens must be non-NULL");
    if (table_stride < max_pages && B > 1)
      return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": table_stride " + s(table_stride) +
                                                " is below max_pages " + s(max_pages));
    if ((st = check_aligned(fn, "page_table", page_table, 4)) != BSA_OK) return st;
    if ((st = check_aligned(fn, "kv_lens", kv_lens, 4)) != BSA_OK) return st;
  }
  a->page_table = page_table; a->table_stride = table_stride; a->max_pages = max_pages; a->kv_lens = kv_lens;
  return BSA_OK;
}

// Checks of both calls' rows against the caches; `rows` names them.
static bsa_status check_rows(const char* fn, const bsa_tensor* k, const bsa_tensor* v, const char* const names[2],
                             bool written, bsa_tensor view[2]) {
  bsa_status st = check_view(k, fn, names[0], written, &view[0]);
  if (st != BSA_OK) return st;
  if ((st = check_view(v, fn, names[1], written, &view[1])) != BSA_OK) return st;
  if (view[0].B != view[1].B || view[0].S != view[1].S || view[0].H != view[1].H || view[0].D != view[1].D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + names[1] + " shape differs from " + names[0] + " shape");
  return BSA_OK;
}

static bsa_status check_rows_caches(const char* fn, const bsa_tensor view[2], const char* const names[2],
                                    const QuantArgs& a) {
  if (a.max_pages == 0) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": max_pages is 0");
  if (a.k.heads != view[0].H || a.k.D != view[0].D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": the cache has " + s(a.k.heads) + " heads of " + s(a.k.D) +
                                              ", " + names[0] + " has " + s(view[0].H) + " of " + s(view[0].D));
  bsa_status st;
  for (int i = 0; i < 2; ++i) {
    if ((st = check_apart(fn, bytes_of(names[i], view[i]), bytes_of("k_cache", a.k))) != BSA_OK) return st;
    if ((st = check_apart(fn, bytes_of(names[i], view[i]), bytes_of("v_cache", a.v))) != BSA_OK) return st;
  }
  return BSA_OK;
}

// What a call writes against the tables and lengths that its other blocks still read.
static bsa_status check_tables_apart(const char* fn, const Bytes written[2], const QuantArgs& a, int64_t B,
                                     const char* other_name, const int32_t* other) {
  const Bytes reads[] = {bytes_at("page_table", a.page_table, 4 * ((B - 1) * a.table_stride + a.max_pages)),
                         bytes_at("kv_lens", a.kv_lens, 4 * B), bytes_at(other_name, other, 4 * B)};
  bsa_status st;
  for (int i = 0; i < 2; ++i)
    for (const Bytes& r : reads)
      if ((st = check_apart(fn, r, written[i])) != BSA_OK) return st;
  return BSA_OK;
}

}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsaq_cache_append(const bsa_tensor* k, const bsa_tensor* v, const bsaq_cache* k_cache,
                             const bsaq_cache* v_cache, const int32_t* page_table, int64_t table_stride,
                             int32_t max_pages, const int32_t* kv_lens, const int32_t* new_lens,
                             bsa_stream_t stream) {
  clear_error();
  const char* fn = "bsaq_cache_append";
  const char* const names[2] = {"k", "v"};
  bsa_tensor x[2] = {};
  QuantArgs a{};
  bsa_status st = check_rows(fn, k, v, names, false, x);
  if (st != BSA_OK) return st;
  if ((st = check_quant(fn, k_cache, v_cache, page_table, table_stride, max_pages, kv_lens, x[0].B, &a)) != BSA_OK)
    return st;
  if ((st = check_aligned(fn, "new_lens", new_lens, 4)) != BSA_OK) return st;
  if ((st = check_rows_caches(fn, x, names, a)) != BSA_OK) return st;
  if (a.k.ptr == a.v.ptr) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": v_cache shares memory with k_cache");
  const Bytes written[2] = {bytes_of("k_cache", a.k), bytes_of("v_cache", a.v)};
  if ((st = check_tables_apart(fn, written, a, x[0].B, "new_lens", new_lens)) != BSA_OK) return st;
  QuantParams p{};
  for (int i = 0; i < 2; ++i) {
    p.x[i] = static_cast<const __nv_bfloat16*>(x[i].ptr);
    p.sb[i] = x[i].stride_b; p.ss[i] = x[i].stride_s; p.sh[i] = x[i].stride_h;
  }
  p.S = (int)x[0].S;
  p.other = new_lens;
  return launch_blocks(p, x[0].B, x[0].D, a, quantise_kernel<64>, quantise_kernel<128>, "quantise_kernel launch", fn,
                       reinterpret_cast<cudaStream_t>(stream));
}

bsa_status bsaq_cache_read(const bsaq_cache* k_cache, const bsaq_cache* v_cache, const int32_t* page_table,
                           int64_t table_stride, int32_t max_pages, const int32_t* kv_lens, const int32_t* first,
                           const bsa_tensor* k_out, const bsa_tensor* v_out, bsa_stream_t stream) {
  clear_error();
  const char* fn = "bsaq_cache_read";
  const char* const names[2] = {"k_out", "v_out"};
  bsa_tensor y[2] = {};
  QuantArgs a{};
  bsa_status st = check_rows(fn, k_out, v_out, names, true, y);
  if (st != BSA_OK) return st;
  if ((st = check_quant(fn, k_cache, v_cache, page_table, table_stride, max_pages, kv_lens, y[0].B, &a)) != BSA_OK)
    return st;
  if ((st = check_aligned(fn, "first", first, 4)) != BSA_OK) return st;
  if ((st = check_rows_caches(fn, y, names, a)) != BSA_OK) return st;
  if ((st = check_apart(fn, "k_out", y[0], "v_out", y[1])) != BSA_OK) return st;
  const Bytes written[2] = {bytes_of("k_out", y[0]), bytes_of("v_out", y[1])};
  if ((st = check_tables_apart(fn, written, a, y[0].B, "first", first)) != BSA_OK) return st;
  QuantParams p{};
  for (int i = 0; i < 2; ++i) {
    p.y[i] = static_cast<__nv_bfloat16*>(const_cast<void*>(y[i].ptr));
    p.sb[i] = y[i].stride_b; p.ss[i] = y[i].stride_s; p.sh[i] = y[i].stride_h;
  }
  p.S = (int)y[0].S;
  p.other = first;
  return launch_blocks(p, y[0].B, y[0].D, a, read_kernel<64>, read_kernel<128>, "read_kernel launch", fn,
                       reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
