// Rotary positions with several axes (forward and backward) and the append of
// new keys and values to a paged cache with the rotation applied on the way.
//
// Mathematics: pair p of a head's channels is a plane; token position
// pos[axes[p]] turns it by angle = pos * inv_freq[p]; the backward pass turns
// it back (the rotation's transpose).  One kernel does all of it: up to three
// jobs (Q, K, V), each "read rows, turn or copy, write rows", to contiguous
// memory or into pages.
//
// Angles: inv_freq / 2 pi is held as a 64-bit fraction of a turn, and its
// product with the integer position is taken modulo 2^64, i.e. modulo whole
// turns: three integer multiply-adds, exact at any position, where an fp32
// product loses 0.06 rad at position 10^6 and an fp64 one runs on a pipe of 2
// operations per clock and SM.  The top 32 bits give the half-turns in
// [-1, 1) for sincospif.
//
// What bounds it: memory (720p latent, 32 + 8 heads of 128: 512 us, 6.9 TB/s;
// 480p, 24 + 8 heads: 120.7 us, 6.6 TB/s, neighbours paired 120.1, half of the
// channels 120.9; append with Q of 5 x 4,099 ragged tokens: 56.4 us, 6.0 TB/s,
// of K and V alone without rotation 16.0 us, 5.3 TB/s).  A thread owns 16 channels
// of a token (8 pairs) in two accesses of 16 bytes, and goes through a group of
// heads, so that the sines and cosines of a token are computed once per thread
// and not once per head.  Where halves are paired, neighbouring threads make
// whole 128-byte lines with each access; where neighbours are, and in channels
// that are copied, a thread's two accesses lie beside each other and only the two
// together make whole lines (which takes the same time, see above).
#include <cuda_bf16.h>
#include <math_constants.h>

#include <cstdint>
#include <string>

#include "bsa_paged.h"

namespace bsa {
namespace {

__device__ unsigned int g_rope_error = 0;

constexpr int kRopeThreads = 128;
constexpr int kMaxAxes = 4;
constexpr int kBatch = 4;         // heads whose loads are in flight together (720p: 2 550 us, 4 527, 8 533 with a loop over tokens)

struct RotJob {
  const __nv_bfloat16* x;
  int64_t sb, ss, sh;             // input strides (elements)
  __nv_bfloat16* y;
  int64_t yb, ys, yh;             // output strides; paged: page, slot, head
  const int32_t* pos;
  int64_t pb, ps, pa;
  int n_tokens, S, H;             // B * S, S, heads
  int rotate, paged;
};

struct RotParams {
  RotJob job[3];
  int group_end[3];               // head groups of jobs 0 .. j
  int heads_per_group;
  const double* inv_freq;
  const int32_t* axes;
  int pairs, n_axes, back;
  const int32_t* page_table;
  int64_t table_stride;
  int max_pages, page_shift, num_pages;
  const int32_t* kv_lens;
  const int32_t* new_lens;
};

// f / 2 pi as a fraction of a turn in units of 2^-64, modulo one turn.  The
// double is taken apart: f = m 2^e with a 53-bit m, and m times 2^64 / 2 pi is
// shifted by e.
__device__ __forceinline__ uint64_t turns_per_position(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int ex = (int)((bits >> 52) & 2047u);
  if (ex == 0 || ex == 2047) return 0;                            // zero and subnormal: no turn; not finite: not defined
  const uint64_t m = (bits & ((1ull << 52) - 1)) | (1ull << 52);
  const int e = ex - 1075;
  constexpr uint64_t k = 0x28BE60DB9391054Aull;                   // floor(2^64 / 2 pi)
  const uint64_t lo = m * k, hi = __umul64hi(m, k);
  uint64_t t;
  if (e >= 0) t = e < 64 ? lo << e : 0;
  else if (e > -64) t = (lo >> -e) | (hi << (64 + e));
  else t = e > -128 ? hi >> (-e - 64) : 0;
  return (bits >> 63) ? 0 - t : t;
}

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Turns the 8 pairs of a unit.  A pair without an axis (its sine is NaN) keeps its
// bits: a turn by 0 would make NaN of an infinity's or a NaN's neighbour.  (Chosen
// for every pair: 480p 120.0 -> 120.9 us, append of 5 x 4,099 tokens 55.8 -> 56.2;
// a branch around the choice, or a loop of its own, costs more registers and 1 to
// 3 % of the time.)
template <bool kInterleaved>
__device__ __forceinline__ void turn_unit(uint4& u0, uint4& u1, const float* cs, const float* sn) {
  float a[8], c[8], ya[8], yc[8];
  unpack8(u0, a);
  unpack8(u1, c);
  const uint4 x0 = u0, x1 = u1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kInterleaved) {                 // pairs (2i, 2i + 1): 4 in each chunk
      if (i % 2 == 0) {
        ya[i] = fmaf(a[i], cs[i / 2], -a[i + 1] * sn[i / 2]);
        ya[i + 1] = fmaf(a[i + 1], cs[i / 2], a[i] * sn[i / 2]);
        yc[i] = fmaf(c[i], cs[4 + i / 2], -c[i + 1] * sn[4 + i / 2]);
        yc[i + 1] = fmaf(c[i + 1], cs[4 + i / 2], c[i] * sn[4 + i / 2]);
      }
    } else {
      ya[i] = fmaf(a[i], cs[i], -c[i] * sn[i]);
      yc[i] = fmaf(c[i], cs[i], a[i] * sn[i]);
    }
  }
  u0 = pack8(ya);
  u1 = pack8(yc);
  uint32_t lo[4], hi[4];           // bits to keep of each word, channels 2 i and 2 i + 1 of a chunk
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      lo[i] = isnan(sn[i]) ? 0xFFFFFFFFu : 0u;
      hi[i] = isnan(sn[4 + i]) ? 0xFFFFFFFFu : 0u;
    } else {
      lo[i] = hi[i] = (isnan(sn[2 * i]) ? 0xFFFFu : 0u) | (isnan(sn[2 * i + 1]) ? 0xFFFF0000u : 0u);
    }
  }
  u0 = make_uint4((u0.x & ~lo[0]) | (x0.x & lo[0]), (u0.y & ~lo[1]) | (x0.y & lo[1]), (u0.z & ~lo[2]) | (x0.z & lo[2]),
                  (u0.w & ~lo[3]) | (x0.w & lo[3]));
  u1 = make_uint4((u1.x & ~hi[0]) | (x1.x & hi[0]), (u1.y & ~hi[1]) | (x1.y & hi[1]), (u1.z & ~hi[2]) | (x1.z & hi[2]),
                  (u1.w & ~hi[3]) | (x1.w & hi[3]));
}

// Grid: x = token blocks, y = head groups of all jobs.
template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rotate_kernel(const __grid_constant__ RotParams p) {
  constexpr int kUnits = D / 16;                  // threads per token
  constexpr int kTokens = kRopeThreads / kUnits;  // tokens per block
  const int gy = blockIdx.y;
  const int ji = gy < p.group_end[0] ? 0 : (gy < p.group_end[1] ? 1 : 2);
  const RotJob& jb = p.job[ji];
  const int h0 = (gy - (ji ? p.group_end[ji - 1] : 0)) * p.heads_per_group;
  const int h1 = min(h0 + p.heads_per_group, jb.H);
  const int unit = threadIdx.x % kUnits;
  const bool turn = jb.rotate && unit < p.pairs / 8;
  // the unit's two 16-byte chunks: the low and the high halves of its pairs,
  // or 16 channels in a row
  const bool apart = turn && !kInterleaved;
  const int c0 = apart ? unit * 8 : unit * 16;
  const int c1 = apart ? unit * 8 + p.pairs : c0 + 8;

  const int tok = blockIdx.x * kTokens + threadIdx.x / kUnits;
  // Launched when the blocks of the kernel before leave: nothing it may have
  // written is read before this point, nor by the read-only path, whose loads may
  // be moved (append of 5 x 4,099 tokens in a row of calls 58.6 -> 56.1 us).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tok >= jb.n_tokens) return;
  const int b = tok / jb.S, s = tok - b * jb.S;
  const __nv_bfloat16* xr = jb.x + b * jb.sb + s * jb.ss;
  __nv_bfloat16* yr;
  if (jb.paged) {
    const int n = p.new_lens ? min(max(p.new_lens[b], 0), jb.S) : jb.S;
    if (s >= n) return;
    const int64_t slot = (int64_t)p.kv_lens[b] - n + s;
    const int64_t at = slot >> p.page_shift;
    int page = -1;
    if (slot >= 0 && at < p.max_pages) page = p.page_table[b * p.table_stride + at];
    if (page < 0 || page >= p.num_pages) {
      if (unit == 0) atomicOr(&g_rope_error, kErrPage);
      return;
    }
    yr = jb.y + page * jb.yb + (slot & ((1 << p.page_shift) - 1)) * jb.ys;
  } else {
    yr = jb.y + b * jb.yb + s * jb.ys;
  }
  // four heads at a time: all their loads are in flight before the first
  // store (which may be to the same memory, so the compiler keeps the order);
  // the first ones are on their way while the angles are worked out
  uint4 u0[kBatch], u1[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h + j < h1) {
        u0[j] = *reinterpret_cast<const uint4*>(xr + (h + j) * jb.sh + c0);
        u1[j] = *reinterpret_cast<const uint4*>(xr + (h + j) * jb.sh + c1);
      }
    }
  };
  load(h0);
  float cs[8], sn[8];
  if (turn) {
    const int32_t* pr = jb.pos + b * jb.pb + s * jb.ps;
    int where[kMaxAxes];
#pragma unroll
    for (int a = 0; a < kMaxAxes; ++a) where[a] = a < p.n_axes ? pr[a * jb.pa] : 0;
    const int sign = p.back ? -1 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t f = turns_per_position(p.inv_freq[unit * 8 + i]);
      const int a = p.axes[unit * 8 + i];
      const int w = a == 0 ? where[0] : a == 1 ? where[1] : a == 2 ? where[2] : a == 3 ? where[3] : 0;
      const uint64_t t = f * (uint64_t)((int64_t)w * sign);
      sincospif((float)(int32_t)(t >> 32) * 0x1p-31f, &sn[i], &cs[i]);
      if (a < 0 || a >= p.n_axes) sn[i] = CUDART_NAN_F;           // passes through
    }
  }
  for (int h = h0; h < h1; h += kBatch) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h + j < h1) {
        if (turn) turn_unit<kInterleaved>(u0[j], u1[j], cs, sn);
        *reinterpret_cast<uint4*>(yr + (h + j) * jb.yh + c0) = u0[j];
        *reinterpret_cast<uint4*>(yr + (h + j) * jb.yh + c1) = u1[j];
      }
    }
    load(h + kBatch);
  }
}

std::string s(int64_t v) { return std::to_string(v); }

bsa_status check_rope(const char* fn, const bsap_rope* r, int64_t D) {
  if (!r) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": rope is NULL");
  if (!r->inv_freq || !r->axes)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": inv_freq and axes must be non-NULL");
  bsa_status st;
  if ((st = check_aligned(fn, "inv_freq", r->inv_freq, 8)) != BSA_OK) return st;
  if ((st = check_aligned(fn, "axes", r->axes, 4)) != BSA_OK) return st;
  if (r->pairs <= 0 || 2 * (int64_t)r->pairs > D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + s(r->pairs) + " pairs for head dim " + s(D));
  if (r->pairs % 8)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(r->pairs) + " pairs is not a multiple of 8");
  if (r->n_axes < 1 || r->n_axes > kMaxAxes)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": n_axes " + s(r->n_axes) + " is not 1 to 4");
  return BSA_OK;
}

bsa_status check_positions(const char* fn, const char* name, const bsap_positions* p) {
  if (!p || !p->ptr) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " is NULL");
  if (p->stride_b < 0 || p->stride_s < 0 || p->stride_a < 0)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " strides must not be negative");
  return check_aligned(fn, name, p->ptr, 4);
}

bsa_status check_out(const char* fn, const char* name, const void* out) {
  if (!out) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " is NULL");
  return check_aligned(fn, name, out, 16);
}

RotJob make_job(const bsa_tensor& x, const bsap_positions* pos, bool rotate) {
  RotJob j{};
  j.x = static_cast<const __nv_bfloat16*>(x.ptr);
  j.sb = x.stride_b; j.ss = x.stride_s; j.sh = x.stride_h;
  j.S = (int)x.S; j.H = (int)x.H; j.n_tokens = (int)(x.B * x.S);
  j.rotate = rotate;
  if (pos) { j.pos = pos->ptr; j.pb = pos->stride_b; j.ps = pos->stride_s; j.pa = pos->stride_a; }
  return j;
}

void to_contiguous(RotJob* j, void* y, int64_t D) {
  j->y = static_cast<__nv_bfloat16*>(y);
  j->yh = D; j->ys = j->H * D; j->yb = (int64_t)j->S * j->ys;
}

bsa_status launch_rotate(RotParams& p, int n_jobs, int64_t D, bool interleaved, cudaStream_t stream) {
  const int tokens_per_block = kRopeThreads / (int)(D / 16);
  int64_t most = 0;
  int heads = 0;
  for (int i = 0; i < n_jobs; ++i) {
    if (p.job[i].n_tokens > most) most = p.job[i].n_tokens;
    if (p.job[i].H > heads) heads = p.job[i].H;
  }
  const int64_t blocks = cdiv64(most, tokens_per_block);
  // Heads per thread: as many as leave 8 blocks of 128 threads per SM, since a
  // thread's sines and cosines, and its way through the page table, serve all
  // its heads (at 32 blocks per SM the 480p rotation took 3 % longer, the
  // append of 5 x 4,099 tokens 30 %).
  const int64_t full = (int64_t)num_sms() * 8;
  int hpg = heads;
  while (hpg > 1 && blocks * cdiv64(heads, hpg) < full) hpg = (hpg + 1) / 2;
  p.heads_per_group = hpg;
  int groups = 0;
  for (int i = 0; i < 3; ++i) {
    if (i < n_jobs) groups += (int)cdiv64(p.job[i].H, hpg);
    p.group_end[i] = groups;
  }
  const dim3 grid((unsigned)blocks, (unsigned)groups);
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_check(D == 128 ? (interleaved ? cudaLaunchKernelEx(&cfg, rotate_kernel<128, true>, p)
                                            : cudaLaunchKernelEx(&cfg, rotate_kernel<128, false>, p))
                             : (interleaved ? cudaLaunchKernelEx(&cfg, rotate_kernel<64, true>, p)
                                            : cudaLaunchKernelEx(&cfg, rotate_kernel<64, false>, p)),
                    "rotate_kernel launch");
}

}  // namespace

unsigned int read_and_clear_rope_error() {
  unsigned int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v != 0 && cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  return v;
}

bsa_status check_aligned(const char* fn, const char* name, const void* ptr, int size) {
  if (reinterpret_cast<uintptr_t>(ptr) % (uintptr_t)size == 0) return BSA_OK;
  return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " is not " + s(size) + "-byte aligned");
}

bsa_status check_view(const bsa_tensor* t, const char* fn, const char* name, bool cache, bsa_tensor* view) {
  if (!t) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " descriptor is NULL");
  if (!t->ptr) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + "->ptr is NULL");
  if (t->B <= 0 || t->S <= 0 || t->H <= 0 || t->D <= 0)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " has a non-positive dim [" + s(t->B) + "," +
                                              s(t->S) + "," + s(t->H) + "," + s(t->D) + "]");
  if (t->D != 64 && t->D != 128)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": head dim " + s(t->D) + " of " + name +
                                              " is not supported (64 or 128)");
  if (t->H > kMaxHeads)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(t->H) + " heads of " + name +
                                              " above the limit " + s(kMaxHeads));
  if (t->B > INT32_MAX / 2 / t->S)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + name + " has more than 2^30 rows");
  if (reinterpret_cast<uintptr_t>(t->ptr) & 15u)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + "->ptr is not 16-byte aligned");
  *view = *t;
  const int64_t len[3] = {t->B, t->S, t->H};
  int64_t* st[3] = {&view->stride_b, &view->stride_s, &view->stride_h};
  for (int i = 0; i < 3; ++i) {
    if (len[i] == 1) { *st[i] = 0; continue; }
    if (*st[i] % 8)
      return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name +
                                                " strides must be multiples of 8 elements (16 bytes); got " + s(*st[i]));
    if (*st[i] < 0 || (cache && *st[i] == 0))
      return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " strides must " +
                                                (cache ? "be positive" : "not be negative"));
  }
  if (cache) {
    // slots apart: each axis, smallest stride first, steps over all that lies below it
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (*st[order[j]] > *st[order[j + 1]]) { const int x = order[j]; order[j] = order[j + 1]; order[j + 1] = x; }
    int64_t extent = t->D;
    for (int i : order) {
      if (len[i] == 1) continue;
      if (*st[i] < extent) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + name + " slots overlap");
      extent += (len[i] - 1) * *st[i];
    }
  }
  return BSA_OK;
}

bsa_tensor contiguous_like(const bsa_tensor& x, void* ptr) {
  bsa_tensor y = x;
  y.ptr = ptr;
  y.stride_h = x.D; y.stride_s = x.H * x.D; y.stride_b = x.S * y.stride_s;
  return y;
}

Bytes bytes_at(const char* name, const void* ptr, int64_t n) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(ptr);
  return Bytes{name, lo, ptr ? lo + (uintptr_t)n : lo};
}

Bytes bytes_of(const char* name, const bsa_tensor& t) {
  return bytes_at(name, t.ptr,
                  2 * ((t.B - 1) * t.stride_b + (t.S - 1) * t.stride_s + (t.H - 1) * t.stride_h + t.D));
}

bsa_status check_apart(const char* fn, const Bytes& x, const Bytes& y) {
  if (x.lo >= y.hi || y.lo >= x.hi) return BSA_OK;
  return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": " + y.name + " shares memory with " + x.name);
}

bsa_status check_apart(const char* fn, const char* x_name, const bsa_tensor& x, const char* y_name,
                       const bsa_tensor& y, bool in_place) {
  if (in_place && x.ptr == y.ptr && (x.H == 1 || x.stride_h == x.D) && (x.S == 1 || x.stride_s == x.H * x.D) &&
      (x.B == 1 || x.stride_b == x.S * x.H * x.D))
    return BSA_OK;
  return check_apart(fn, bytes_of(x_name, x), bytes_of(y_name, y));
}

bsa_status check_paged(const char* fn, const bsa_tensor* k_cache, const bsa_tensor* v_cache,
                       const int32_t* page_table, int64_t table_stride, int32_t max_pages, const int32_t* kv_lens,
                       const int32_t* new_lens, int64_t B, PagedArgs* a) {
  bsa_status st;
  if ((st = check_view(k_cache, fn, "k_cache", true, &a->k)) != BSA_OK) return st;
  if ((st = check_view(v_cache, fn, "v_cache", true, &a->v)) != BSA_OK) return st;
  if (a->k.B != a->v.B || a->k.S != a->v.S || a->k.H != a->v.H || a->k.D != a->v.D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": v_cache shape differs from k_cache shape");
  const int64_t ps = a->k.S;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": page size " + s(ps) +
                                              " is not supported (16, 32, 64, 128 or 256)");
  if (B > kMaxPagedBatch)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": batch " + s(B) + " above the limit " + s(kMaxPagedBatch));
  if (max_pages < 0 || max_pages > INT32_MAX / 2 / ps)
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
  if ((st = check_aligned(fn, "new_lens", new_lens, 4)) != BSA_OK) return st;
  a->page_table = page_table; a->table_stride = table_stride; a->max_pages = max_pages;
  a->kv_lens = kv_lens; a->new_lens = new_lens;
  return BSA_OK;
}

}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsap_rope_axes(const bsa_tensor* q, const bsa_tensor* k, const bsap_positions* pos_q,
                          const bsap_positions* pos_k, const bsap_rope* rope, int32_t backward, void* q_out,
                          void* k_out, bsa_stream_t stream) {
  clear_error();
  const char* fn = "bsap_rope_axes";
  bsa_tensor qv{}, kv{};
  bsa_status st = check_view(q, fn, "q", false, &qv);
  if (st != BSA_OK) return st;
  if ((st = check_rope(fn, rope, qv.D)) != BSA_OK) return st;
  if ((st = check_positions(fn, "pos_q", pos_q)) != BSA_OK) return st;
  if ((st = check_out(fn, "q_out", q_out)) != BSA_OK) return st;
  if (k) {
    if ((st = check_view(k, fn, "k", false, &kv)) != BSA_OK) return st;
    if (kv.D != qv.D)
      return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": head dim of q (" + s(qv.D) + ") != head dim of k (" +
                                                s(kv.D) + ")");
    if ((st = check_positions(fn, "pos_k", pos_k)) != BSA_OK) return st;
    if ((st = check_out(fn, "k_out", k_out)) != BSA_OK) return st;
  }
  const bsa_tensor qo = contiguous_like(qv, q_out);
  if ((st = check_apart(fn, "q", qv, "q_out", qo, true)) != BSA_OK) return st;
  if (k) {
    const bsa_tensor ko = contiguous_like(kv, k_out);
    if ((st = check_apart(fn, "k", kv, "k_out", ko, true)) != BSA_OK) return st;
    if ((st = check_apart(fn, "k", kv, "q_out", qo)) != BSA_OK) return st;
    if ((st = check_apart(fn, "q", qv, "k_out", ko)) != BSA_OK) return st;
    if ((st = check_apart(fn, "q_out", qo, "k_out", ko)) != BSA_OK) return st;
  }
  RotParams p{};
  p.inv_freq = rope->inv_freq; p.axes = rope->axes; p.pairs = rope->pairs; p.n_axes = rope->n_axes;
  p.back = backward ? 1 : 0;
  p.job[0] = make_job(qv, pos_q, true);
  to_contiguous(&p.job[0], q_out, qv.D);
  if (k) {
    p.job[1] = make_job(kv, pos_k, true);
    to_contiguous(&p.job[1], k_out, kv.D);
  }
  return launch_rotate(p, k ? 2 : 1, qv.D, rope->interleaved != 0, reinterpret_cast<cudaStream_t>(stream));
}

bsa_status bsap_cache_append(const bsa_tensor* k, const bsa_tensor* v, const bsa_tensor* k_cache,
                             const bsa_tensor* v_cache, const int32_t* page_table, int64_t table_stride,
                             int32_t max_pages, const int32_t* kv_lens, const int32_t* new_lens,
                             const bsap_rope* rope, const bsap_positions* pos, const bsa_tensor* q, void* q_out,
                             bsa_stream_t stream) {
  clear_error();
  const char* fn = "bsap_cache_append";
  bsa_tensor kv{}, vv{}, qv{};
  PagedArgs a{};
  bsa_status st = check_view(k, fn, "k", false, &kv);
  if (st != BSA_OK) return st;
  if ((st = check_view(v, fn, "v", false, &vv)) != BSA_OK) return st;
  if (vv.B != kv.B || vv.S != kv.S || vv.H != kv.H || vv.D != kv.D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": v shape differs from k shape");
  if ((st = check_paged(fn, k_cache, v_cache, page_table, table_stride, max_pages, kv_lens, new_lens, kv.B, &a)) !=
      BSA_OK)
    return st;
  if (max_pages == 0) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": max_pages is 0");
  if (a.k.H != kv.H || a.k.D != kv.D)
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": the cache has " + s(a.k.H) + " heads of " + s(a.k.D) +
                                              ", k has " + s(kv.H) + " of " + s(kv.D));
  if (rope) {
    if ((st = check_rope(fn, rope, kv.D)) != BSA_OK) return st;
    if ((st = check_positions(fn, "pos", pos)) != BSA_OK) return st;
  }
  if (q) {
    if (!rope) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": q is given without rope");
    if ((st = check_view(q, fn, "q", false, &qv)) != BSA_OK) return st;
    if (qv.B != kv.B || qv.S != kv.S || qv.D != kv.D)
      return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": q's batch, length or head dim differs from k's");
    if ((st = check_out(fn, "q_out", q_out)) != BSA_OK) return st;
  }
  const bsa_tensor* caches[2] = {&a.k, &a.v};
  if (a.k.ptr == a.v.ptr) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": v_cache shares memory with k_cache");
  const bsa_tensor qo = q ? contiguous_like(qv, q_out) : bsa_tensor{};
  if (q) {
    if ((st = check_apart(fn, "q", qv, "q_out", qo, true)) != BSA_OK) return st;
    if ((st = check_apart(fn, "k", kv, "q_out", qo)) != BSA_OK) return st;
    if ((st = check_apart(fn, "v", vv, "q_out", qo)) != BSA_OK) return st;
  }
  for (const bsa_tensor* c : caches) {
    const char* name = c == &a.k ? "k_cache" : "v_cache";
    if ((st = check_apart(fn, "k", kv, name, *c)) != BSA_OK) return st;
    if ((st = check_apart(fn, "v", vv, name, *c)) != BSA_OK) return st;
    if (q && (st = check_apart(fn, "q", qv, name, *c)) != BSA_OK) return st;
    if (q && (st = check_apart(fn, "q_out", qo, name, *c)) != BSA_OK) return st;
  }
  RotParams p{};
  if (rope) {
    p.inv_freq = rope->inv_freq; p.axes = rope->axes; p.pairs = rope->pairs; p.n_axes = rope->n_axes;
  }
  int shift = 4;
  while ((1 << shift) < a.k.S) ++shift;
  p.page_shift = shift; p.num_pages = (int)a.k.B; p.max_pages = max_pages;
  p.page_table = page_table; p.table_stride = table_stride;
  p.kv_lens = kv_lens; p.new_lens = new_lens;
  p.job[0] = make_job(kv, pos, rope != nullptr);
  p.job[1] = make_job(vv, nullptr, false);
  for (int i = 0; i < 2; ++i) {
    p.job[i].paged = 1;
    p.job[i].y = static_cast<__nv_bfloat16*>(const_cast<void*>(caches[i]->ptr));
    p.job[i].yb = caches[i]->stride_b; p.job[i].ys = caches[i]->stride_s; p.job[i].yh = caches[i]->stride_h;
  }
  if (q) {
    p.job[2] = make_job(qv, pos, true);
    to_contiguous(&p.job[2], q_out, qv.D);
  }
  return launch_rotate(p, q ? 3 : 2, kv.D, rope && rope->interleaved, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
