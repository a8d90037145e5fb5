// Attention of new tokens over a paged key/value cache whose first prefix_len
// keys all requests share (tcgen05 + TMEM + TMA).
//
// Mathematics: row i of request b and query head h sees the prefix keys and
// its request's own keys up to a limit; out = sum_j e^{z_j} v_j / sum_j
// e^{z_j}, computed over any split of the keys as partial (max, sum, sum of
// v) triples that are joined by rescaling to the common maximum.
//
// What bounds it: for one token per request, reading K and V once (each 64 KB
// of a 128-key tile of K and V at head dim 128 takes an SM 1.5 us at its share
// of the memory rate, while its two products and its softmax take 0.7 us);
// with hundreds of rows on one prefix, the chain S -> softmax -> P V (0.87 us a
// job of 128 rows and 128 keys with two groups in turn, of which the tensor
// cores are busy 0.53 us and the exponential unit 0.27 us); with a few short
// requests, the way from the launch to the join (10 us, one tile included).
//
// Layout of the work:
//  * A segment is up to 256 query rows that read the same keys: for the prefix
//    any 256 rows (b, i, g) of the whole batch under one KV head, so that the
//    prefix is read once for all; for a request's own keys the rows (i, g) of
//    that request under one KV head.  A GQA group's heads are rows of one tile.
//    Where the requests' own rows fill their tiles, sharing saves nothing: the
//    prefix is folded into the own segments then, as their first key tiles.
//  * All segments' 128-key tiles are put in one row and cut into equal pieces,
//    one for each CTA, whatever the lengths are (they are read from the device,
//    so a captured graph follows them).  A cut segment leaves one partial
//    result per CTA; the pair (segment, CTA) only ever steps forward along the
//    row, so segment + CTA numbers the partial results without gaps of meaning
//    and without a table.
//  * One CTA per SM: warp 2 goes through the CTA's segments, hands them to the
//    others through a ring and loads their Q rows; warps 0 and 3 gather K and V
//    tiles page by page with TMA into a second ring, in the order the products
//    use them (K_0, K_1, V_0, K_2, V_1 ..); warp 1 issues the MMAs, S = Q K^T
//    and O += P V; warps 4-7 and 8-11 are two softmax groups, one row per
//    thread, that take the jobs in turn, each with an S and an O of its own in
//    TMEM and P staying there.  A job is 128 rows on one key tile: a segment of
//    more rows makes two jobs of each tile, which read the same K and V; in a
//    smaller one the groups take every other tile, and each leaves a partial
//    result (one group took 1.1 us a tile of 128 rows, and 3 us for a segment
//    of one tile, in which nothing hid the way from S to the result's store).
//    Code is kept short (one copy of the schedule, rolled loops where
//    nothing is gained by unrolling): short segments run each role's code once
//    per microsecond, and with 143 KB of it they took 7 us each.
//  * paged_join_kernel adds up the partial results (launched when the blocks of
//    the first kernel leave).
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <string>

#include "bsa_paged.h"
#include "bsa_paged_device.cuh"
#include "bsa_quant.h"

namespace bsa {
namespace {

constexpr int kTileKeys = 128;
constexpr int kRowTile = 256;        // rows of a segment
constexpr int kHalf = 128;           // rows of a job
constexpr int kMaxBlocks = kMaxPagedBatch / 32;     // blocks of 32 requests in the schedule

// kQ4: the pages hold 4 bits (bsa_quant.h).  Warps 12-15 make the K and V tiles of the
// ring then, from blocks that warp 0 copies into a ring of their own.
template <int D, bool kQ4>
struct PagedCfg {
  static constexpr unsigned int kErr = kQ4 ? kErrQuantPage : kErrPage;      // a bad page or length, told by the call's name
  static constexpr int kThreads = kQ4 ? 512 : 384;
  static constexpr int kChunks = D / 64;                      // 128-byte chunks per row
  static constexpr int kQBytes = kHalf * 128 * kChunks;      // 128 rows
  static constexpr int kTileBytes = kTileKeys * 128 * kChunks;
  static constexpr int kBarBytes = 2048;
  static constexpr int kSmemMax = 232448;                     // 227 KB per CTA
  static constexpr int kRaw = kQ4 && D == 64 ? 8 : 3;         // places for blocks of 128 keys (of 4 bits)
  static constexpr int kRawBytes = kQ4 ? kTileKeys / kBlockSlots * block_bytes(D) : 0;
  static constexpr int kScaleBytes = kQ4 ? 2 * (D / kGroup) * kTileKeys * 2 : 0;
  static constexpr int kRest = kSmemMax - 1024 - kBarBytes - 2 * kQBytes - kRaw * kRawBytes - kScaleBytes;
  static constexpr int kFit = kRest / kTileBytes;
  static constexpr int kStages = kFit > 10 ? 10 : kFit;       // 5 of 32 KB, 10 of 16 KB; 4 and 9 beside blocks
  static constexpr int kSmemBytes = kSmemMax - kRest + kStages * kTileBytes;
};

struct PagedParams {
  CUtensorMap tk, tv;             // [pages, Hkv, slots, D] of the whole cache
  const uint8_t* k4; const uint8_t* v4;                       // or, of 4 bits, its bytes
  int64_t k4_page, k4_head, v4_page, v4_head;
  uint32_t eights;                // kEights
  int early;                      // the kernel behind starts beside this one, on the SMs that it leaves (and waits for it at its end)
  int beside_keys;                // own keys at most of a request, which are that kernel's
  const __nv_bfloat16* q;
  int64_t q_sb, q_ss, q_sh;
  int B, T, Hq, Hkv, G, page_shift, num_pages, max_pages, prefix_len, causal;
  FastDiv div_G, div_TG;
  int TG;                         // rows of a request under one KV head
  int own_rt;                     // row tiles of a request
  int pre_rt;                     // row tiles of the whole batch (prefix)
  int pre_tiles;                  // key tiles of the prefix as segments of its own
  int fold;                       // key tiles of the prefix at the head of each own segment (one of the two is 0)
  int pre_slot_rows, own_slot_rows;   // rows of one of a slot's two partial results
  int ctas, pre_w, pre_over, own_w;    // weights: see where they are set
  const int32_t* page_table; int64_t table_stride;
  const int32_t* kv_lens; const int32_t* new_lens;
  const int32_t* prefix_table;
  float scale_log2;
  __nv_bfloat16* out;
  float* lse;
  int2* seg_ctas;                 // workspace: first and last CTA of each segment that has tiles
  float* part_ml;                 // workspace: partial results' (max, sum) and rows,
  float* part_o;                  // those of the prefix first,
  int own_first;                  // from here on those of own keys
};

// Request b's own keys and new tokens, clamped to what the tables hold.
__device__ __forceinline__ int own_keys(const PagedParams& p, int b) {
  if (p.max_pages == 0) return 0;
  return min(max(p.kv_lens[b], 0), p.max_pages << p.page_shift);
}
__device__ __forceinline__ int new_tokens(const PagedParams& p, int b) {
  return p.new_lens ? min(max(p.new_lens[b], 0), p.T) : p.T;
}
// Own keys that row i of a request with kv keys and n new tokens sees.
__device__ __forceinline__ int seen_keys(const PagedParams& p, int kv, int n, int i) {
  return p.causal ? max(kv - n + i + 1, 0) : kv;
}
// Key tiles of row tile rt of such a request (behind those of a folded prefix).
__device__ __forceinline__ int own_tiles(const PagedParams& p, int kv, int n, int rt) {
  const int first = p.div_G.quot(rt * kRowTile);
  if (first >= n) return 0;
  const int last = min(n - 1, p.div_G.quot(rt * kRowTile + kRowTile - 1));
  return p.fold + (seen_keys(p, kv, n, last) + kTileKeys - 1) / kTileKeys;
}
// Key tiles of a request under one KV head.
__device__ __forceinline__ int request_tiles(const PagedParams& p, int kv, int n) {
  int sum = 0;
#pragma unroll 1
  for (int rt = 0; rt < p.own_rt; ++rt) sum += own_tiles(p, kv, n, rt);
  return sum;
}

// The row of tiles is cut by weight: a prefix tile counts pre_w units, a tile
// of own keys own_w.  The CTAs that get some (every one of them at least one
// tile: its units are no fewer than a tile's), and the first tile of CTA c of n.
struct Cut {
  int pre, pre_w, own_w;          // prefix tiles, weights
  int n, q, r;                    // CTAs, units of all tiles = q n + r
  float inv_n;                    // 1 / n
  __device__ __forceinline__ Cut(const PagedParams& p, int own, int ctas) {
    pre = p.pre_tiles * p.pre_rt * p.Hkv;
    pre_w = p.pre_w;
    own_w = p.own_w;
    // the way in and out of the prefix's segments, as far as a block's share is
    // more than a tile (a tile that weighs more would leave blocks without one)
    pre_w += min(p.pre_over, max((pre * pre_w + own * own_w) / ctas - pre_w, 0));
    const int units = pre * pre_w + own * own_w;
    n = min(ctas, units / max(pre > 0 ? pre_w : 0, own > 0 ? own_w : 1));
    // Two tiles each where some CTA has two anyway, or where a tile leaves 128 KB
    // of partial results (33 tiles of 8 heads 13.0 -> 12.3 us, 16 prefix tiles of
    // 8 heads for 256 rows 21.4 -> 19.1 us).
    if (pre + own > ctas || (pre > 0 && p.B * p.TG > kHalf)) n = min(n, max((pre + own) / 2, min(n, 1)));
    q = n > 0 ? units / n : 0;
    r = units - q * n;
    inv_n = 1.f / (float)max(n, 1);
  }
  // floor(c units / n); the small quotient is exact in fp32 (c r < 2^20)
  __device__ __forceinline__ int begin_unit(int c) const { return c * q + (int)(((float)(c * r) + 0.5f) * inv_n); }
  // the first tile that begins at or behind a CTA's first unit
  __device__ __forceinline__ int begin(int c) const {
    const int u = begin_unit(c), pre_units = pre * pre_w;
    return u < pre_units ? (u + pre_w - 1) / pre_w : pre + (u - pre_units + own_w - 1) / own_w;
  }
};

// Keys of a segment's key tile, whose keys end at `end` (the last tile of a
// folded prefix ends with the prefix).
__device__ __forceinline__ int tile_keys(const PagedParams& p, int end, int tile) {
  return min((tile == p.fold - 1 ? p.prefix_len : end) - tile * kTileKeys, kTileKeys);
}

// A segment's part that one CTA works on, as it stands in the segment ring.
struct __align__(16) Segment {
  int b;               // request, -1: prefix
  int hk;
  int row0, rows;      // first flat row (b * T + i) * G + g, and how many
  int tile0, tiles;    // first key tile and how many
  int slot;            // number of the partial result (segment + CTA)
  int whole;           // this CTA has all tiles of the segment
  int keys;            // where its keys end, counted in tiles of 128 from its first one
  int kv, n;           // of the request
  int pad;
};
constexpr int kSegRing = 4;
constexpr int kSegReaders = 11;      // warps that read every segment (one producer less of 4-bit pages)

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// 8 columns from `col` on of a row at `row`: fp32, or divided by the row's sum
// to bf16 (which may be aligned to 16 bytes only).
__device__ __forceinline__ void store_row(unsigned long long row, int col, const float* v, float inv_l, bool bf16,
                                          bool real) {
  if (!real) return;
  if (bf16) {
    uint32_t pk[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) pk[e] = output_pair(inv_l, v[2 * e], v[2 * e + 1]);
    *reinterpret_cast<uint4*>(row + col * 2) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
  } else {
    store_32(reinterpret_cast<void*>(row + col * 4), v);
  }
}

// 16 lanes x 32 columns: lane t gets of row t / 4 (a) and of row t / 4 + 8 (b)
// columns 8 j + 2 (t % 4) and the next one, j = 0 .. 3.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float* a, float* b) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(a[0]), "=f"(a[1]), "=f"(b[0]), "=f"(b[1]), "=f"(a[2]), "=f"(a[3]), "=f"(b[2]), "=f"(b[3]), "=f"(a[4]),
        "=f"(a[5]), "=f"(b[4]), "=f"(b[5]), "=f"(a[6]), "=f"(a[7]), "=f"(b[6]), "=f"(b[7])
      : "r"(taddr)
      : "memory");
}

// Lane k of four holds pairs (columns 8 j + 2 k, + 1) in v[2 j], v[2 j + 1];
// afterwards columns 8 k .. 8 k + 7.
__device__ __forceinline__ void quad_transpose(float* v) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
  for (int j = 0; j < 4; j += 2)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float got = __shfl_xor_sync(0xffffffffu, odd ? v[2 * j + e] : v[2 * j + 2 + e], 1);
      if (odd) v[2 * j + e] = got;
      else v[2 * j + 2 + e] = got;
    }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float got = __shfl_xor_sync(0xffffffffu, high ? v[2 * j + e] : v[2 * j + 4 + e], 2);
      if (high) v[2 * j + e] = got;
      else v[2 * j + 4 + e] = got;
    }
}

// A warp's place in the segment ring.
struct SegmentReader {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ bool take(const Segment* ring, uint32_t seg_full, uint32_t seg_empty, uint32_t abort,
                                       Segment& s) {
    if (!warp_wait(seg_full + 8 * slot, phase, abort)) return false;
    const int4* src = reinterpret_cast<const int4*>(ring + slot);
    const int4 a = src[0], b = src[1], c = src[2];
    s.b = a.x; s.hk = a.y; s.row0 = a.z; s.rows = a.w;
    s.tile0 = b.x; s.tiles = b.y; s.slot = b.z; s.whole = b.w;
    s.keys = c.x; s.kv = c.y; s.n = c.z;
    release(seg_empty);
    return true;
  }
  __device__ __forceinline__ void release(uint32_t seg_empty) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(seg_empty + 8 * slot);
    if (++slot == kSegRing) { slot = 0; phase ^= 1u; }
  }
};

template <int D, bool kQ4>
__global__ void __launch_bounds__(PagedCfg<D, kQ4>::kThreads, 1) paged_attention_kernel(const __grid_constant__ PagedParams p) {
  using C = PagedCfg<D, kQ4>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* q_smem = smem;                                  // [2] Q buffers of 128 rows
  uint8_t* ring = smem + 2 * C::kQBytes;
  uint8_t* raw = ring + kStages * C::kTileBytes;           // [kRaw] blocks of 128 keys
  uint8_t* scales = raw + C::kRaw * C::kRawBytes;          // [2][D / 32][128] twice the scales of a V tile, bf16
  Segment* segs = reinterpret_cast<Segment*>(scales + C::kScaleBytes);           // [kSegRing]
  // barriers, as shared-memory addresses 8 bytes apart
  const uint32_t q_full = smem_u32(segs + kSegRing);   // [2] 32 loader threads
  const uint32_t q_empty = q_full + 16;                // [2] commit
  const uint32_t s_full = q_full + 32;                 // [2] commit
  const uint32_t p_full = q_full + 48;                 // [2] 4 softmax warps
  const uint32_t o_empty = q_full + 64;                // [2] 4 softmax warps
  // P V of even and of odd jobs [2], commit.  A parity tells only neighbouring
  // phases apart: who waits for P V of job q knows that P V of job q - 2 is
  // done, since S of job q was issued behind it.
  const uint32_t pv_done = q_full + 80;
  const uint32_t mma_end = q_full + 96;                // commit
  const uint32_t seg_full = q_full + 112;              // [kSegRing] the scheduler
  const uint32_t seg_empty = seg_full + 8 * kSegRing;  // [kSegRing] the 11 warps that read it
  const uint32_t full = seg_empty + 8 * kSegRing;      // [kStages] transaction bytes, or the 4 warps that make tiles
  const uint32_t empty = full + 8 * kStages;           // [kStages] commit
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(segs + kSegRing) + 2 * (14 + 2 * kSegRing + 2 * kStages);
  const uint32_t abort_flag = empty + 8 * kStages + 4; // behind tmem_slot
  int* total_slot = reinterpret_cast<int*>(tmem_slot + 2);
  int* block_sum = total_slot + 1;      // [kMaxBlocks]: tiles of own keys before request 32 i
  // of 4-bit pages
  int* raw_info = block_sum + kMaxBlocks;                // [kRaw] keys, + 256 where they are of V
  int* beside = raw_info + C::kRaw;                      // [warps] tiles of the kernel beside
  const uint32_t raw_full = (smem_u32(beside + C::kThreads / 32) + 7) & ~7u;    // [kRaw] transaction bytes
  const uint32_t raw_empty = raw_full + 8 * C::kRaw;     // [kRaw] 4 warps
  const uint32_t scale_bar = raw_empty + 8 * C::kRaw;    // 4 warps
  static_assert(kSegRing * sizeof(Segment) + (14 + 2 * kSegRing + 2 * kStages) * 8 + 12 + kMaxBlocks * 4 + C::kRaw * 20 + 16 + 64 <=
                    C::kBarBytes,
                "barrier block");

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 32);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(o_empty + 8 * i, 4);
      mbar_init(pv_done + 8 * i, 1);
    }
    mbar_init(mma_end, 1);
    for (int i = 0; i < kSegRing; ++i) {
      mbar_init(seg_full + 8 * i, 1);
      mbar_init(seg_empty + 8 * i, kSegReaders - (kQ4 ? 1 : 0));
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full + 8 * i, kQ4 ? 4 : 1);
      mbar_init(empty + 8 * i, 1);
    }
    if constexpr (kQ4) {
      for (int i = 0; i < C::kRaw; ++i) {
        mbar_init(raw_full + 8 * i, 1);
        mbar_init(raw_empty + 8 * i, 4);
      }
      mbar_init(scale_bar, 4);
    }
    tmem_slot[1] = 0;                   // abort flag
    fence_mbar_init();
    if constexpr (!kQ4) {
      tma_prefetch_desc(&p.tk);
      tma_prefetch_desc(&p.tv);
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // Launched when the blocks of the kernel before leave: up to here nothing is
  // read or written that it uses (and nothing by the read-only path, whose loads
  // may be taken from before this point).  2 us less a call in a row of them.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kQ4 && p.early && threadIdx.x == C::kThreads - 32) {            // the last warp has the least to do here
    fence_waited();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  // the schedule: tiles of own keys per block of 32 requests, then their sums
  const int nblk = (p.B + 31) / 32;
#pragma unroll 1
  for (int blk = warp; blk < nblk; blk += C::kThreads / 32) {
    const int b = blk * 32 + lane;
    const int mine = b < p.B ? request_tiles(p, own_keys(p, b), new_tokens(p, b)) * p.Hkv : 0;
    const int incl = warp_inclusive_sum(mine);
    if (lane == 31) block_sum[blk] = incl;
    if (cta == 0 && b < p.B) {
      if (p.max_pages > 0) {
        const int kv = p.kv_lens[b];
        if (kv < 0 || kv > p.max_pages << p.page_shift) atomicOr(&g_bsa_error, C::kErr);
      }
    }
  }
  if (kQ4 && p.early) {
    int tiles = 0;
#pragma unroll 1
    for (int b = threadIdx.x; b < p.B && p.beside_keys > 0; b += C::kThreads)      // without own keys: no lengths either
      if (const int own = new_tokens(p, b) > 0 ? min(max(p.kv_lens[b], 0), p.beside_keys) : 0)
        tiles += (own + kTileKeys - 1) / kTileKeys + kSegmentWay;
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    if (lane == 0) beside[warp] = tiles;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int before = 0;
#pragma unroll 1
    for (int i = 0; i < nblk; i += 32) {
      const int v = i + lane < nblk ? block_sum[i + lane] : 0;
      const int incl = warp_inclusive_sum(v) + before;
      if (i + lane < nblk) block_sum[i + lane] = incl - v;
      before = __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *total_slot = before;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  int begin = 0, end = 0;
  {
    int ctas = p.ctas;
    if (kQ4 && p.early) {
      int tiles = 0;
#pragma unroll 1
      for (int i = 0; i < C::kThreads / 32; ++i) tiles += beside[i];
      ctas = prefix_sms(p.ctas, p.pre_tiles * p.pre_rt * p.Hkv, p.B * p.TG > kHalf, tiles * p.Hkv);
    }
    const Cut cut(p, *total_slot, ctas);
    if (cta < cut.n) {
      begin = cut.begin(cta);
      end = cut.begin(cta + 1);
    }
  }
  bool ok = true;

  if (kQ4 && warp == 0) {
    // ------------------------------------------------- copies of 4-bit blocks ---
    // In the order of the ring's tiles: of rows above 128 K_0, V_0, K_1, V_1 .., else
    // K_0, K_1, V_0, K_2, V_1 ..  Lane x copies page x of a tile.
    const int per_tile = p.page_shift >= 7 ? 1 : kTileKeys >> p.page_shift;
    const int per_page = kTileKeys / kBlockSlots / per_tile;                    // blocks of a page in a tile
    uint32_t it = 0;
    const uint8_t* v_from = nullptr;               // this lane's part of the V that is still to come
    int v_count = 0, v_keys = 0;
    bool v_left = false;
    SegmentReader reader;
    auto put = [&](const uint8_t* from, int count, int keys, bool is_v) {
      const uint32_t at = it % C::kRaw;
      if (!warp_wait(raw_empty + 8 * at, (it / C::kRaw & 1u) ^ 1u, abort_flag)) return false;
      if (lane == 0) {
        raw_info[at] = keys + (is_v ? 256 : 0);
        mbar_arrive_expect_tx(raw_full + 8 * at, (keys + kBlockSlots - 1) / kBlockSlots * block_bytes(D));
      }
      __syncwarp();
      if (lane < per_tile && count > 0)
        bulk_load(smem_u32(raw) + at * C::kRawBytes + lane * per_page * block_bytes(D), from, count * block_bytes(D),
                  raw_full + 8 * at);
      ++it;
      return true;
    };
#pragma unroll 1
    for (int t = begin; t < end && ok;) {
      Segment s;
      if (!(ok = reader.take(segs, seg_full, seg_empty, abort_flag, s))) break;
      const bool wide = s.rows > kHalf;
      const int32_t* own_table = p.page_table + s.b * p.table_stride;
      auto page_of = [&](int j) {
        const bool pre = s.b < 0 || j < p.fold;
        const int key = (pre ? j : j - p.fold) * kTileKeys + lane * per_page * kBlockSlots;
        int page = 0;
        if (lane < per_tile && key < (pre ? p.prefix_len : s.kv)) {
          page = (pre ? p.prefix_table : own_table)[key >> p.page_shift];
          if (page < 0 || page >= p.num_pages) {
            atomicOr(&g_bsa_error, C::kErr);
            page = 0;
          }
        }
        return page;
      };
      int page = page_of(s.tile0);
#pragma unroll 1
      for (int j = 0; j < s.tiles && ok; ++j) {
        const int next = j + 1 < s.tiles ? page_of(s.tile0 + j + 1) : 0;
        const int tile = s.tile0 + j, source = tile - (tile < p.fold ? 0 : p.fold);       // tile of its table
        const int keys = tile_keys(p, s.keys, tile);
        const int count = min((keys + kBlockSlots - 1) / kBlockSlots - lane * per_page, per_page);
        const int64_t in_page =
            (source * (kTileKeys / kBlockSlots) & ((1 << (p.page_shift - 4)) - 1) & ~(per_page - 1)) * block_bytes(D);
        const uint8_t* vf = p.v4 + page * p.v4_page + s.hk * p.v4_head + in_page;
        ok = put(p.k4 + page * p.k4_page + s.hk * p.k4_head + in_page, count, keys, false);
        if (ok && v_left) ok = put(v_from, v_count, v_keys, true);
        if (ok && wide) ok = put(vf, count, keys, true);
        v_left = !wide;
        v_from = vf; v_count = count; v_keys = keys;
        page = next;
      }
      t += s.tiles;
    }
    if (ok && v_left) put(v_from, v_count, v_keys, true);
    // the copies in flight land before the CTA may leave
    if (lane == 0)
#pragma unroll 1
      for (uint32_t i = it > C::kRaw ? it - C::kRaw : 0; i < it; ++i) mbar_drain(raw_full + 8 * (i % C::kRaw), i / C::kRaw & 1u);
    __syncwarp();
  } else if (kQ4 && warp >= 12) {
    // ------------------------------------------------------ codes to bf16 ---
    // K: a thread a key, rows of 64 channels; V: a thread a channel, rows of 64 keys
    // (the transposed tile, which takes whole pieces of 16 bytes from a thread); 16-byte
    // pieces exchanged within 8 rows, as the MMAs read them.
    const int th = threadIdx.x % 128;
    const uint32_t slot_at = (th / kBlockSlots) * block_bytes(D), slot = th % kBlockSlots, swap = (th % 8) * 16;
    uint32_t stage = 0, phase = 0, v_no = 0;
#pragma unroll 1
    for (uint32_t it = 0; it < 2u * (uint32_t)(end - begin); ++it) {
      const uint32_t at = it % C::kRaw;
      if (!(ok = warp_wait(raw_full + 8 * at, it / C::kRaw & 1u, abort_flag))) break;
      const int info = raw_info[at], keys = info & 255;
      const uint32_t from = smem_u32(raw) + at * C::kRawBytes, to = smem_u32(ring) + stage * C::kTileBytes;
      if (info < 256) {
        if (!(ok = warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag))) break;
#pragma unroll
        for (int g = 0; g < D / kGroup; ++g) {
          const uint4 c = lds128(from + slot_at + g * 256 + slot * 16);
          const uint32_t s2 = twice_scale(lds8(from + slot_at + code_bytes(D) + g * kBlockSlots + slot)) * 0x10001u;
          const uint32_t off = scale_offset(s2), word[4] = {c.x, c.y, c.z, c.w};
          const uint32_t row = to + (g / 2) * (kTileKeys * 128) + th * 128;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = code_values(raised_codes(word[x], i, p.eights), s2, off);
            sts128(row + (((g % 2) * 4 + x) * 16 ^ swap), r);
          }
        }
      } else {
        // twice the scales, 0 behind the last key: what stands there must not count (who
        // still reads the ones before has not come to this barrier)
        const uint32_t scale_to = smem_u32(scales) + (v_no & 1u) * (C::kScaleBytes / 2);
#pragma unroll
        for (int g = 0; g < D / kGroup; ++g)
          sts16(scale_to + (g * kTileKeys + th) * 2,
                th < keys ? twice_scale(lds8(from + slot_at + code_bytes(D) + g * kBlockSlots + slot)) : 0u);
        __syncwarp();
        if (lane == 0) mbar_arrive(scale_bar);
        if (!(ok = warp_wait(scale_bar, v_no & 1u, abort_flag))) break;
        ++v_no;
        if (!(ok = warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag))) break;
        if (th < D) {
#pragma unroll
          for (int x = 0; x < kTileKeys / kBlockSlots; ++x) {
            const uint2 c = lds64(from + x * block_bytes(D) + th * 8);
            const uint32_t scale_at = scale_to + (th / kGroup) * (kTileKeys * 2) + x * 32;
            const uint4 sa = lds128(scale_at), sb = lds128(scale_at + 16);
            const uint32_t s2[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              r[i] = code_values(raised_codes(i < 4 ? c.x : c.y, i % 4, p.eights), s2[i], scale_offset(s2[i]));
            const uint32_t row = to + (x / 4) * (D * 128) + th * 128;
            sts128(row + ((x % 4) * 32 ^ swap), r);
            sts128(row + (((x % 4) * 32 + 16) ^ swap), r + 4);
          }
        }
      }
      fence_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(raw_empty + 8 * at);
        mbar_arrive(full + 8 * stage);
      }
      advance<kStages>(stage, phase);
    }
  } else if (!kQ4 && (warp == 0 || warp == 3)) {
    // ----------------------------------------------------- TMA producers ---
    // K of tile q, then V of tile q - 1, for every tile of the CTA's row: warp 0
    // fetches K and warp 3 V, each at its places in the ring.  (One warp for both
    // was busy all the time where pages are small: looking up a tile's pages
    // takes it 0.4 us, asking for 8 of them 0.5.  137 requests of 1,700 keys in
    // pages of 32 124 -> 100 us, 103 x 30 in pages of 16 25.3 -> 22.6.)
    const int per_tile = p.page_shift >= 7 ? 1 : kTileKeys >> p.page_shift;   // pages per tile
    const int box_rows = kTileKeys / per_tile;
    const uint32_t ring_base = smem_u32(ring);
    uint32_t stage = 0, phase = 0, issued = 0;     // whose last copy is this warp's
    int v_page = 0, v_slot = 0, v_hk = 0;          // the tile whose V is still to come,
    bool v_left = false;                           // if there is one
    SegmentReader reader;
#pragma unroll 1
    for (int t = begin; begin < end;) {
      const bool more = t < end;        // after the last segment there is one V left, or none
      Segment s;
      s.rows = s.tiles = 1;
      s.tile0 = s.hk = s.kv = 0;
      s.b = -1;
      if (more && !(ok = reader.take(segs, seg_full, seg_empty, abort_flag, s))) break;
      const int32_t* own_table = p.page_table + s.b * p.table_stride;
      // lane's page of key tile j (a page past the end reads zeros)
      auto page_of = [&](int j) {
        const bool pre = s.b < 0 || j < p.fold;
        const int key = (pre ? j : j - p.fold) * kTileKeys + lane * box_rows;
        int page = p.num_pages;
        if (lane < per_tile && key < (pre ? p.prefix_len : s.kv)) {
          page = (pre ? p.prefix_table : own_table)[key >> p.page_shift];
          if (page < 0 || page >= p.num_pages) {
            atomicOr(&g_bsa_error, C::kErr);
            page = p.num_pages;
          }
        }
        return page;
      };
      // K of a job's tile, then V of the job before it, each at its first use
      const bool wide = s.rows > kHalf;
      int page = p.num_pages;
#pragma unroll 1
      for (int j = -1; j < s.tiles && ok; ++j) {
        const int next = more && j + 1 < s.tiles ? page_of(s.tile0 + j + 1) : 0;
        const int source = s.tile0 + j - (s.tile0 + j < p.fold ? 0 : p.fold);       // tile of its table
        const int slot = (source * kTileKeys) & ((1 << p.page_shift) - 1) & ~(box_rows - 1);
#pragma unroll 1
        for (int which = j < 0 ? 3 : 0; which < 3; ++which) {
          if (which == 0 ? !more : which == 1 ? !v_left : !more || !wide) continue;
          if ((which == 0) != (warp == 0)) {       // not awaited: it may be used up and gone by now
            issued &= ~(1u << stage);
            advance<kStages>(stage, phase);
            continue;
          }
          if (!(ok = warp_wait(empty + 8 * stage, phase ^ 1u, abort_flag))) break;
          issued |= 1u << stage;
          const bool old = which == 1;
          const int from = old ? v_page : page, at = old ? v_slot : slot, head = old ? v_hk : s.hk;
          if (elect_one()) mbar_arrive_expect_tx(full + 8 * stage, C::kTileBytes);
          uint32_t dst = ring_base + stage * C::kTileBytes;
#pragma unroll 1
          for (int x = 0; x < per_tile; ++x, dst += box_rows * 128) {
            const int pg = __shfl_sync(0xffffffffu, from, x);
            if (elect_one()) {
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_4d(dst + c * (kTileKeys * 128), which == 0 ? &p.tk : &p.tv, full + 8 * stage, c * 64, at, head, pg);
            }
            __syncwarp();
          }
          advance<kStages>(stage, phase);
        }
        if (j >= 0) {
          v_left = !wide;
          v_page = page; v_slot = slot; v_hk = s.hk;
        }
        page = next;
      }
      if (!more || !ok) break;
      t += s.tiles;
    }
    // the copies in flight land before the CTA may leave
    if (lane == 0) {
#pragma unroll 1
      for (int i = 0; i < kStages; ++i) {
        if (issued >> stage & 1u) mbar_drain(full + 8 * stage, phase ^ 1u);
        advance<kStages>(stage, phase);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer ---
    // S of job q, then P V of job q - 1 (MMAs of one thread run in order, so S
    // of job q may overwrite P of job q - 2 without a wait).  The whole warp
    // goes through the loop and one lane issues: the descriptors then stay in
    // uniform registers (in a branch of one lane each MMA took 26 instructions).
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTileKeys, false);
    constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, !kQ4);     // of 4-bit pages V is transposed
    const uint64_t qdesc0 = sdesc_sw128(smem_u32(q_smem), 16, 1024);
    const uint64_t kdesc0 = sdesc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t vdesc0 = sdesc_sw128(smem_u32(ring), kQ4 ? 16 : kTileKeys * 128, 1024);
    uint32_t stage = 0, phase = 0;      // next item of the ring
    uint32_t q = 0, qi = 0;             // next job, next Q buffer
    uint32_t k_stage = 0, v_stage = 0;
    uint32_t uses0 = 0, uses1 = 0;      // segments that each O has been used for
    bool v_first = false, v_new = false, v_last = false;   // job q - 1: starts its O; takes, releases its V tile
    int v_keys = 0;                     // its tile's keys
    SegmentReader reader;
#pragma unroll 1
    for (int t = begin; begin < end;) {
      const bool more = t < end;        // after the last segment there is one P V left
      Segment s;
      s.rows = s.tiles = 1;
      s.keys = s.tile0 = 0;
      if (more && !reader.take(segs, seg_full, seg_empty, abort_flag, s)) break;
      const bool wide = s.rows > kHalf;
      const int jobs = wide ? 2 * s.tiles : s.tiles;
#pragma unroll 1
      for (int j = 0; j < jobs; ++j) {
        if (more) {
          const uint32_t half = wide ? j & 1 : 0, qb = (qi + half) & 1u, w = q & 1u;
          if (half == 0) {
            if (!(ok = warp_wait(full + 8 * stage, phase, abort_flag))) break;
            k_stage = stage;
            advance<kStages>(stage, phase);
          }
          if (j <= (int)half) {
            if (!(ok = warp_wait(q_full + 8 * qb, ((qi + half) >> 1) & 1u, abort_flag))) break;
            fence_async_shared();                  // Q rows come by ordinary copies
          }
          tc_fence_after();
          const uint64_t as = qdesc0 + (uint64_t)((qb * C::kQBytes) >> 4);
          const uint64_t bs = kdesc0 + (uint64_t)((k_stage * C::kTileBytes) >> 4);
          const uint32_t d_t = tmem + w * 128;
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              constexpr int kChunk = (kTileKeys * 128) >> 4;
              const uint64_t off = (uint64_t)((kk / 4) * kChunk + (kk % 4) * 2);
              if (kk == 0) mma_ss_acc<0>(d_t, as + off, bs + off, idesc_s);
              else mma_ss_acc<1>(d_t, as + off, bs + off, idesc_s);
            }
            mma_commit(s_full + 8 * w);
            if (!wide || half == 1) mma_commit(empty + 8 * k_stage);
            if (j >= jobs - (wide ? 2 : 1)) mma_commit(q_empty + 8 * qb);
          }
          __syncwarp();
        }
        if (q > 0) {                    // O (+)= P V of job q - 1
          const uint32_t job = q - 1, w = job & 1u;
          if (v_first && !(ok = warp_wait(o_empty + 8 * w, ((w ? uses1++ : uses0++) & 1u) ^ 1u, abort_flag))) break;
          if (v_new) {
            v_stage = stage;
            if (!(ok = warp_wait(full + 8 * stage, phase, abort_flag))) break;
            advance<kStages>(stage, phase);
            // Behind the last key the page holds whatever stood there: V rows
            // up to the end of the MMA step that it lies in are zeroed (0 times
            // infinity or NaN is NaN), the steps behind are left out.
            const int rest = -v_keys & 15;
            if (!kQ4 && v_keys < kTileKeys && rest != 0) {
              const uint32_t at = smem_u32(ring) + v_stage * C::kTileBytes + v_keys * 128;
#pragma unroll 1
              for (int x = lane; x < rest * (D / 8); x += 32) {
                const int row = x / (D / 8), c = x % (D / 8);
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + (c / 8) * (kTileKeys * 128) + row * 128 +
                                                                             (c % 8) * 16),
                             "r"(0)
                             : "memory");
              }
              fence_async_shared();
              __syncwarp();
            }
          }
          if (!(ok = warp_wait(p_full + 8 * w, (job >> 1) & 1u, abort_flag))) break;
          tc_fence_after();
          const uint64_t bs = vdesc0 + (uint64_t)((v_stage * C::kTileBytes) >> 4);
          const uint32_t d_t = tmem + 256 + w * 128, a_t = tmem + w * 128;
          if (elect_one()) {
            mma_ts(d_t, a_t, bs, idesc_o, !v_first);
#pragma unroll
            for (int kk = 1; kk < kTileKeys / 16; ++kk)
              if (kk * 16 < v_keys)
                mma_ts_acc<1>(d_t, a_t + kk * 8,
                              bs + (uint64_t)(kQ4 ? (kk / 4) * ((D * 128) >> 4) + (kk % 4) * 2 : kk * ((16 * 128) >> 4)), idesc_o);
            mma_commit(pv_done + 8 * w);
            if (v_last) mma_commit(empty + 8 * v_stage);
          }
          __syncwarp();
        }
        ++q;
        v_first = j < 2;
        v_new = !wide || (j & 1) == 0;
        v_last = !wide || (j & 1) == 1;
        v_keys = tile_keys(p, s.keys, s.tile0 + (wide ? j >> 1 : j));
      }
      if (!ok || !more) break;
      qi += wide ? 2 : 1;
      t += s.tiles;
    }
    if (elect_one()) {
      mma_commit(mma_end);    // nothing of the MMAs is in flight when TMEM is freed, after an abort either
      mbar_drain(mma_end, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // Q rows of a segment into the next one or two Q buffers: each lane works
    // out the address of one of 32 rows, then 32 / kVec rows are copied at a time.
    constexpr int kVec = D / 8;                    // 16-byte pieces of a row
    constexpr int kRowsPer = 32 / kVec;            // rows per warp-wide copy
    const int c = lane % kVec;
    uint32_t qi = 0;
    // Warp 2 is the scheduler, too: it finds the segments of tiles [begin, end)
    // in their order.  Its lane l holds request 32 blk + l: its lengths, tiles,
    // and the tiles up to its end.
    const int pre = p.pre_tiles * p.pre_rt * p.Hkv;
    int blk = -1, blk_end = 0, kv = 0, n = 0, mine = 0, upto = 0;
    uint32_t slot = 0, phase = 0;
    for (int t = begin; t < end && ok;) {
      Segment s;
      {
        int t0, t1;
        if (t < pre) {
          const int seg = t / p.pre_tiles;
          t0 = seg * p.pre_tiles;
          t1 = t0 + p.pre_tiles;
          s.b = -1;
          s.hk = seg / p.pre_rt;
          s.row0 = (seg - s.hk * p.pre_rt) * kRowTile;
          s.rows = min(kRowTile, p.B * p.TG - s.row0);
          s.slot = seg + cta;
          s.keys = p.prefix_len;
          s.kv = s.n = 0;
        } else {
          const int u = t - pre;
          if (u >= blk_end) {                          // the last block that begins at or before u
            ++blk;
            while (blk + 1 < nblk && block_sum[blk + 1] <= u) ++blk;
            const int b = blk * 32 + lane;
            kv = b < p.B ? own_keys(p, b) : 0;
            n = b < p.B ? new_tokens(p, b) : 0;
            mine = b < p.B ? request_tiles(p, kv, n) : 0;
            upto = warp_inclusive_sum(mine * p.Hkv) + block_sum[blk];
            blk_end = __shfl_sync(0xffffffffu, upto, 31);
          }
          const int src = __ffs(__ballot_sync(0xffffffffu, upto > u)) - 1;   // there is one: u < blk_end
          const int per_head = __shfl_sync(0xffffffffu, mine, src);
          const int first = __shfl_sync(0xffffffffu, upto, src) - per_head * p.Hkv;
          s.b = blk * 32 + src;
          s.kv = __shfl_sync(0xffffffffu, kv, src);
          s.n = __shfl_sync(0xffffffffu, n, src);
          s.hk = (u - first) / per_head;
          t0 = pre + first + s.hk * per_head;
          int rt = 0, m = p.own_rt == 1 ? per_head : own_tiles(p, s.kv, s.n, 0);
#pragma unroll 1
          while (t >= t0 + m) {
            t0 += m;
            m = own_tiles(p, s.kv, s.n, ++rt);
          }
          t1 = t0 + m;
          s.row0 = s.b * p.TG + rt * kRowTile;
          s.rows = min(kRowTile, s.n * p.G - rt * kRowTile);
          s.slot = (s.b * p.Hkv + s.hk) * p.own_rt + rt + cta;
          s.keys = p.fold * kTileKeys + s.kv;
        }
        s.tile0 = t - t0;
        s.tiles = min(t1, end) - t;
        s.whole = begin <= t0 && t1 <= end;
        s.pad = 0;
        if (!(ok = warp_wait(seg_empty + 8 * slot, phase ^ 1u, abort_flag))) break;
        if (lane == 0) {
          int2* who = p.seg_ctas + (s.b < 0 ? 0 : p.pre_rt * p.Hkv) + s.slot - cta;     // the join looks here
          if (t == t0) who->x = cta;
          if (t1 <= end) who->y = cta;
          segs[slot] = s;
          mbar_arrive(seg_full + 8 * slot);
        }
        __syncwarp();
        if (++slot == kSegRing) { slot = 0; phase ^= 1u; }
      }
      const __nv_bfloat16* head = p.q + (int64_t)s.hk * p.G * p.q_sh + c * 8;
#pragma unroll 1
      for (int r0 = 0; r0 < s.rows; r0 += kHalf, ++qi) {
        const uint32_t qb = qi & 1u;
        if (!warp_wait(q_empty + 8 * qb, ((qi >> 1) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t base = smem_u32(q_smem) + qb * C::kQBytes + (c / 8) * (kHalf * 128) + (lane / kVec) * 128;
        const int rows = min(kHalf, s.rows - r0);
#pragma unroll 1
        for (int r32 = 0; r32 < rows; r32 += 32) {
          const int row = s.row0 + r0 + min(r32 + lane, rows - 1);
          const int b = p.div_TG.quot(row), rem = row - b * p.TG, i = p.div_G.quot(rem), g = rem - i * p.G;
          const uint32_t off = (uint32_t)((b * p.q_sb + i * p.q_ss + g * p.q_sh) / 8);    // below 2^32: host check
#pragma unroll 8
          for (int x = 0; x < kVec && r32 + x * kRowsPer < rows; ++x) {
            const int in = x * kRowsPer + lane / kVec, r = r32 + in;
            const __nv_bfloat16* src = head + (uint64_t)__shfl_sync(0xffffffffu, off, in) * 8;
            if (r < rows)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(base + (r32 + x * kRowsPer) * 128 +
                                                                             ((c % 8) ^ (in % 8)) * 16),
                           "l"(src)
                           : "memory");
          }
        }
        // arrives when this lane's copies have landed; the warp goes on
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(q_full + 8 * qb) : "memory");
      }
      t += s.tiles;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");         // after an abort, too
    __syncwarp();
  } else if (warp >= 4 && warp < 12) {
    // --------------------------------------------------- softmax + results ---
    const uint32_t w = (warp - 4) / 4;             // the group: it takes the jobs q with q % 2 == w
    const int wq = warp % 4;
    const int r = wq * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_t = tmem + lane_base + w * 128;
    const uint32_t o_t = tmem + lane_base + 256 + w * 128;
    uint32_t q = 0;                                // first job of the segment
    // The segment's fields stay in the ring until the group is through with it.
    SegmentReader reader;
    for (int t = begin; t < end && ok;) {
      if (!(ok = warp_wait(seg_full + 8 * reader.slot, reader.phase, abort_flag))) break;
      const Segment& s = segs[reader.slot];
      const bool wide = s.rows > kHalf;
      const int jobs = wide ? 2 * s.tiles : s.tiles;
      const int j0 = (int)((w ^ q) & 1u);          // this group's first job of the segment
      if (j0 >= jobs) {                            // the other group has the segment's only tile
        const bool direct = p.pre_tiles == 0 && s.whole;
        if (!direct && r < s.rows)
          reinterpret_cast<float2*>(p.part_ml)[(s.b < 0 ? 0 : p.own_first) +
                                               (s.slot * 2 + (int)w) * (s.b < 0 ? p.pre_slot_rows : p.own_slot_rows) + r] =
              make_float2(-INFINITY, 0.f);
        q += jobs;
        t += s.tiles;
        reader.release(seg_empty);
        continue;
      }
      const int half = wide ? j0 : 0;              // and the rows that its jobs have
      const int rows = min(kHalf, s.rows - half * kHalf);
      const bool active = wq * 32 < rows;          // some row of this warp is real
      int limit = s.keys;                          // keys that the row sees (a row that is none: all)
      if (s.b >= 0 && r < rows) {
        const int rem = s.row0 + half * kHalf + r - s.b * p.TG;
        limit = p.fold * kTileKeys + min(seen_keys(p, s.kv, s.n, p.div_G.quot(rem)), s.kv);
      }
      float m_ref = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = j0; j < jobs; j += 2) {
        const int tile = wide ? j >> 1 : j;
        ok = warp_wait(s_full + 8 * w, ((q + j) >> 1) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          // S is read twice, 64 columns at a time: held whole in registers the
          // code is three times as long, and the roles' loops no longer fit the
          // instruction cache together (32 at a time measured 3 % slower).
          const int valid = tile_keys(p, limit, s.tile0 + tile);
          // columns below `least` are seen by all rows of the warp, those from
          // `most` on by none
          const int least = __reduce_min_sync(0xffffffffu, valid), most = __reduce_max_sync(0xffffffffu, valid);
#pragma unroll 1
          for (int c = max(least, 0) & ~31; c < min((most + 63) & ~63, kTileKeys); c += 32) {
            float v[32];
            tmem_ld32f(s_t + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c + e >= valid) v[e] = -INFINITY;
            tmem_st32f(s_t + c, v);
            tmem_wait_st();
          }
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < min(most, kTileKeys); c += 64) {
            float v[64];
            tmem_ld32f(s_t + c, v);
            tmem_ld32f(s_t + c + 32, v + 32);
            tmem_wait_ld();
            float m0 = mx, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 64; e += 8) {
              m0 = max3f(m0, v[e], v[e + 1]);
              m1 = max3f(m1, v[e + 2], v[e + 3]);
              m2 = max3f(m2, v[e + 4], v[e + 5]);
              m3 = max3f(m3, v[e + 6], v[e + 7]);
            }
            mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
          }
          const float m_new = fmaxf(m_ref, mx * p.scale_log2);
          const bool grow = m_new > m_ref + 8.0f;
          const bool rescale = grow && m_ref != -INFINITY;
          const float alpha = rescale ? ex2_approx(m_ref - m_new) : 1.f;
          if (grow) m_ref = m_new;
          const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-m_use, -m_use);
          float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < kTileKeys; c += 64) {
            float v[64];
            uint32_t pk[32];
            if (c >= most) {                       // P of keys that no row sees
#pragma unroll
              for (int e = 0; e < 32; ++e) pk[e] = 0u;
              tmem_st32(s_t + c / 2, pk);
              continue;
            }
            tmem_ld32f(s_t + c, v);
            tmem_ld32f(s_t + c + 32, v + 32);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const float2 a = __ffma2_rn(make_float2(v[e], v[e + 1]), sc2, nm2);
              const float2 b = __ffma2_rn(make_float2(v[e + 2], v[e + 3]), sc2, nm2);
              const float2 e0 = make_float2(ex2_approx(a.x), ex2_approx(a.y));
              const float2 e1 = make_float2(ex2_approx(b.x), ex2_approx(b.y));
              ls0 = __fadd2_rn(ls0, e0);
              ls1 = __fadd2_rn(ls1, e1);
              // The weights meet V in bf16, as the tensor cores take it beside
              // bf16 V (a second product with what the rounding leaves would
              // double P V); their sum is of the unrounded ones.  Relative error
              // of the output against 64 bits 0.0023, with fp32 weights 0.0017.
              pk[e / 2] = pack_bf16x2(e0.x, e0.y);
              pk[e / 2 + 1] = pack_bf16x2(e1.x, e1.y);
            }
            tmem_st32(s_t + c / 2, pk);            // P of these 64 keys over S of keys read already
          }
          l = l * alpha + ((ls0.x + ls0.y) + (ls1.x + ls1.y));
          // O is rescaled only when the maximum grew by more than 2^8 (P V of the
          // group's job before is done: S of this one was issued behind it)
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              float o[32];
              tmem_ld32f(o_t + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= alpha;
              tmem_st32f(o_t + c * 32, o);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * w);
      }
      if (!ok) break;
      const int last_j = jobs - 1 - ((jobs - 1 - j0) & 1);     // this group's last job
      ok = warp_wait(pv_done + 8 * w, ((q + last_j) >> 1) & 1u, abort_flag);
      if (!ok) break;
      tc_fence_after();
      // a segment of more rows, or of one tile, that no other CTA works on and
      // no prefix stands beside: the result; else a partial one
      const bool direct = p.pre_tiles == 0 && s.whole && (wide || s.tiles == 1);
      const bool mine = r < rows;
      const int row = s.row0 + half * kHalf + r;
      const int fb = p.div_TG.quot(row), rem = row - fb * p.TG, i = p.div_G.quot(rem), g = rem - i * p.G;
      const int at = (s.b < 0 ? 0 : p.own_first) +
                     (s.slot * 2 + (wide ? half : (int)w)) * (s.b < 0 ? p.pre_slot_rows : p.own_slot_rows) + r;
      float2* ml = reinterpret_cast<float2*>(p.part_ml) + at;
      if (active) {
        const float inv_l = inverse_sum(limit > 0, l);
        const int64_t orow = ((int64_t)fb * p.T + i) * p.Hq + s.hk * p.G + g;
        const unsigned long long dst = direct ? reinterpret_cast<unsigned long long>(p.out + orow * D)
                                              : reinterpret_cast<unsigned long long>(p.part_o + (int64_t)at * D);
        if (rows > 32) {
          // 16 rows and 32 columns at a time: four lanes share a row, and after
          // the exchange each holds 8 columns in a row of it, so that a store
          // covers whole lines (with a row per lane, one store of 32 bytes each,
          // 16 MB of partial results took 6 us to drain behind the kernel).
#pragma unroll 1
          for (int hf = 0; hf < 32 && wq * 32 + hf < rows; hf += 16) {
            const int ra = hf + lane / 4, rb = ra + 8;
            const unsigned long long da = __shfl_sync(0xffffffffu, dst, ra), db = __shfl_sync(0xffffffffu, dst, rb);
            const float ia = __shfl_sync(0xffffffffu, inv_l, ra), ib = __shfl_sync(0xffffffffu, inv_l, rb);
            const int at_col = 8 * (lane % 4);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float a[8], b[8];
              tmem_ld_16x32(o_t + (static_cast<uint32_t>(hf) << 16) + c, a, b);
              tmem_wait_ld();
              quad_transpose(a);
              quad_transpose(b);
              store_row(da, c + at_col, a, ia, direct, wq * 32 + ra < rows);
              store_row(db, c + at_col, b, ib, direct, wq * 32 + rb < rows);
            }
          }
        } else {
          // few rows: the shorter code (256 requests with 256 own keys 164 us,
          // through the exchange 189)
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld32f(o_t + c, o);
            tmem_wait_ld();
            if (mine && direct) {
              uint32_t pk[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = output_pair(inv_l, o[2 * e], o[2 * e + 1]);
#pragma unroll
              for (int e = 0; e < 4; ++e)            // out may be aligned to 16 bytes only
                reinterpret_cast<uint4*>(dst + c * 2)[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
            } else if (mine) {
#pragma unroll
              for (int e = 0; e < 4; ++e) store_32(reinterpret_cast<void*>(dst + c * 4 + e * 32), o + 8 * e);
            }
          }
        }
        if (mine) {
          if (!direct)
            *ml = make_float2(m_ref, l);
          else if (p.lse)
            p.lse[((int64_t)fb * p.Hq + s.hk * p.G + g) * p.T + i] = row_lse(limit > 0, m_ref, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty + 8 * w);
      q += jobs;
      t += s.tiles;
      reader.release(seg_empty);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Output row (b, i, h): joins the partial results of its prefix segment and of
// its own segment.  kLanes lanes of kWarps warps share a row: eight lanes where
// there are many rows (a warp's way through its dependent loads takes 4 us, so
// four rows go it together), a warp or eight warps where there are fewer.
template <int D, int kLanes, int kWarps>
__global__ void __launch_bounds__(kWarps > 1 ? 32 * kWarps : 128) paged_join_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kRows = kWarps > 1 ? 1 : 128 / kLanes;   // rows per block
  const int64_t R = (int64_t)blockIdx.x * kRows + (kWarps > 1 ? 0 : threadIdx.x / kLanes);
  const bool real = R < (int64_t)p.B * p.T * p.Hq;
  const int r0 = real ? (int)R : 0;
  const int bt = r0 / p.Hq, h = r0 - bt * p.Hq;
  const int b = bt / p.T, i = bt - b * p.T, hk = p.div_G.quot(h), g = h - hk * p.G;
  const int row = i * p.G + g, flat = b * p.TG + row, rt = row / kRowTile;
  const int pre_seg = hk * p.pre_rt + flat / kRowTile, own_seg = (b * p.Hkv + hk) * p.own_rt + rt;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // One wait on memory for all of it: a segment's CTAs are read before the lengths tell
  // whether it has any (if not, they are any bytes and not looked at).
  const int2 pc = p.pre_tiles > 0 ? p.seg_ctas[pre_seg] : make_int2(0, 0), oc = p.seg_ctas[p.pre_rt * p.Hkv + own_seg];
  const int kv = own_keys(p, b), n = new_tokens(p, b);
  // Partial results: from each CTA of a segment one, or two of a segment of up
  // to 128 rows (one of each group).
  Parts pre{0, 0, 0}, own{0, 0, 0};
  bool direct = false;
  const bool keyed = real && i < n && (p.prefix_len > 0 || min(seen_keys(p, kv, n, i), kv) > 0);
  if (real && i < n) {
    const int mine = own_tiles(p, kv, n, rt);
    if (p.pre_tiles > 0) {
      const bool two = p.B * p.TG - (flat - flat % kRowTile) <= kHalf;
      pre = segment_parts(pc.x, pc.y, p.ctas, pre_seg, two, flat % kRowTile / kHalf, p.pre_slot_rows, flat % kHalf);
    }
    if (mine > 0) {
      const bool two = n * p.G - rt * kRowTile <= kHalf;
      own = segment_parts(oc.x, oc.y, p.ctas, own_seg, two, row % kRowTile / kHalf, p.own_slot_rows, row % kHalf);
      own.at += p.own_first;
      direct = p.pre_tiles == 0 && own.n > 0 && oc.x == oc.y && (!two || mine == 1);   // written by the first kernel
    }
  }
  join_row<D, kLanes, kWarps>(p.part_ml, p.part_o, pre, own, real && !direct, keyed, p.out + R * D,
                              p.lse ? p.lse + ((int64_t)b * p.Hq + h) * p.T + i : nullptr);
}

std::string s(int64_t v) { return std::to_string(v); }

// Where the partial results lie in the workspace.
struct PagedPlan {
  int TG, own_rt, pre_rt, pre_slot_rows, own_slot_rows;
  bool fold;
  size_t own_first, part_ml, part_o, bytes;
};

PagedPlan plan_paged(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t d, bool prefix, int sms) {
  PagedPlan w{};
  const int64_t G = Hq / Hkv;
  w.TG = (int)(T * G);
  w.own_rt = (int)cdiv64(w.TG, kRowTile);
  // The prefix is folded into the own segments where that adds at most an
  // eighth of jobs: rows of 128 per request against rows of 128 of the batch (500
  // tokens of two prompts 92 -> 90 us).  The host knows T, not the lengths: a
  // batch of single tokens padded to one request's chunk counts as full (a chunk
  // of 500 and 63 single tokens on 8,192 shared keys 551 us, in two calls 76 + 47).
  w.fold = prefix && 8 * B * cdiv64(w.TG, kHalf) <= 9 * cdiv64(B * w.TG, kHalf);
  prefix = prefix && !w.fold;
  w.pre_rt = prefix ? (int)cdiv64(B * w.TG, kRowTile) : 0;
  w.own_slot_rows = w.TG < kHalf ? w.TG : kHalf;
  w.pre_slot_rows = (int)(B * w.TG < kHalf ? B * w.TG : kHalf);
  auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // a slot of two partial results for every number segment + CTA
  const size_t own = (size_t)(B * Hkv * w.own_rt + sms) * 2 * w.own_slot_rows;
  const size_t pre = prefix ? (size_t)(Hkv * w.pre_rt + sms) * 2 * w.pre_slot_rows : 0;
  w.own_first = pre;
  w.part_ml = al((size_t)Hkv * (w.pre_rt + B * w.own_rt) * 8);      // behind the segments' CTAs
  w.part_o = w.part_ml + al((pre + own) * 8);
  w.bytes = w.part_o + al((pre + own) * d * 4);
  return w;
}

// The driver's cuTensorMapEncodeTiled, looked up once per process.
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static std::once_flag once;
  static EncodeFn fn = nullptr;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

// Map of a cache view: dims (D, slots, Hkv, pages), box (64, min(slots, 128),
// 1, 1), 128-byte swizzle; a page number past the end reads zeros.
bsa_status encode_cache(CUtensorMap* m, const bsa_tensor& t, const char* fn, const char* name) {
  const EncodeFn enc = encode_fn();
  if (!enc) return set_error(BSA_ERR_CUDA, std::string(fn) + ": cuTensorMapEncodeTiled is not available from the driver");
  // strides of axes of length 1 are free: the smallest legal one
  auto bytes = [](int64_t stride) { return (cuuint64_t)(stride > 0 ? stride * 2 : 16); };
  cuuint64_t dims[4] = {(cuuint64_t)t.D, (cuuint64_t)t.S, (cuuint64_t)t.H, (cuuint64_t)t.B};
  cuuint64_t strides[3] = {bytes(t.stride_s), bytes(t.stride_h), bytes(t.stride_b)};
  cuuint32_t box[4] = {64u, (cuuint32_t)(t.S < kTileKeys ? t.S : kTileKeys), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  // What a tile reads in a row: a slot's D values, or all of them where slots
  // follow one another.  Fetching 256 bytes for a lone 128 would bring another
  // head's keys, which are gone from L2 when their turn comes (16 requests of
  // 32,768 keys, 8 heads of 64: 216 us, with 256 bytes 265).
  const CUtensorMapL2promotion promotion =
      t.D == 64 && t.stride_s != t.D ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.ptr), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promotion,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return set_error(BSA_ERR_CUDA, std::string(fn) + ": cuTensorMapEncodeTiled failed for " + name + " (CUresult " +
                                       s((int)r) + ")");
  return BSA_OK;
}

template <int D, bool kQ4>
bsa_status set_smem() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  bsa_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != BSA_OK) return st;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 64 || !done[dev]) {
    st = cuda_check(cudaFuncSetAttribute(paged_attention_kernel<D, kQ4>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PagedCfg<D, kQ4>::kSmemBytes),
                    "cudaFuncSetAttribute(paged_attention_kernel)");
    if (st != BSA_OK) return st;
    if (dev < 64) done[dev] = true;
  }
  return BSA_OK;
}

template <int D, bool kQ4>
bsa_status launch_paged(const PagedParams& p, cudaStream_t stream, bool join = true) {
  bsa_status st = set_smem<D, kQ4>();
  if (st != BSA_OK) return st;
  cudaLaunchAttribute attrs[2] = {};
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  // Beside another kernel: pairs of CTAs, so that those without tiles leave pairs of SMs
  // to it.  (An SM of this kernel whose neighbour had four CTAs of the other took up to
  // 203 us where it takes 135; which SMs are neighbours was up to chance.)
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = 2;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = p.early && p.ctas % 2 == 0 ? 2 : 1;
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(PagedCfg<D, kQ4>::kThreads);
  cfg.dynamicSmemBytes = PagedCfg<D, kQ4>::kSmemBytes;
  if ((st = cuda_check(cudaLaunchKernelEx(&cfg, paged_attention_kernel<D, kQ4>, p), "paged_attention_kernel launch")) != BSA_OK)
    return st;
  if (!join) return BSA_OK;
  cfg.numAttrs = 1;
  const int64_t rows = (int64_t)p.B * p.T * p.Hq;
  // Eight warps, one warp or eight lanes a row, by the number of rows (us of the
  // join: 32 rows of 40 partial results 6.4, with one warp 9; 2,048 rows of 2 to
  // 10 with one warp 7.7, four 11, eight lanes 13; 24,000 rows of 2 to 4 with
  // eight lanes 12, one warp 19; 8,192 rows 12 either way).
  const int lanes = rows < (int64_t)num_sms() * 4 ? 256 : rows < (int64_t)num_sms() * 40 ? 32 : 8;
  cfg.blockDim = dim3(lanes == 256 ? 256 : 128);
  cfg.gridDim = dim3((unsigned)cdiv64(rows, cfg.blockDim.x / lanes));
  cfg.dynamicSmemBytes = 0;
  return cuda_check(lanes == 256  ? cudaLaunchKernelEx(&cfg, paged_join_kernel<D, 32, 8>, p)
                    : lanes == 32 ? cudaLaunchKernelEx(&cfg, paged_join_kernel<D, 32, 1>, p)
                                  : cudaLaunchKernelEx(&cfg, paged_join_kernel<D, 8, 1>, p),
                    "paged_join_kernel launch");
}

// What a launch takes but for the cache itself; `a`: its tables and lengths.
PagedParams make_params(const bsa_tensor& qv, int64_t Hkv, int64_t page, int64_t pages, const PagedArgs& a,
                        const int32_t* prefix_table, int32_t prefix_len, int32_t causal, float softmax_scale, void* out,
                        float* lse, void* workspace, const PagedPlan& plan, int64_t most_tiles, int sms) {
  PagedParams p{};
  const int64_t G = qv.H / Hkv, flat_rows = qv.B * qv.S * G;
  p.q = static_cast<const __nv_bfloat16*>(qv.ptr); p.q_sb = qv.stride_b; p.q_ss = qv.stride_s; p.q_sh = qv.stride_h;
  p.B = (int)qv.B; p.T = (int)qv.S; p.Hq = (int)qv.H; p.Hkv = (int)Hkv; p.G = (int)G;
  p.page_shift = 4;
  while ((1 << p.page_shift) < page) ++p.page_shift;
  p.num_pages = (int)pages; p.max_pages = a.max_pages; p.prefix_len = prefix_len; p.causal = causal ? 1 : 0;
  p.div_G = fast_div((uint32_t)G); p.div_TG = fast_div((uint32_t)plan.TG);
  p.TG = plan.TG; p.own_rt = plan.own_rt; p.pre_rt = plan.pre_rt;
  p.pre_tiles = plan.fold ? 0 : (int)cdiv64(prefix_len, kTileKeys);
  p.fold = plan.fold ? (int)cdiv64(prefix_len, kTileKeys) : 0;
  p.pre_slot_rows = plan.pre_slot_rows; p.own_slot_rows = plan.own_slot_rows;
  p.ctas = sms;
  // Weights of about an eighth of a microsecond: a wide prefix tile (two jobs of
  // 0.9 us on the tensor cores, more while others fetch) against a tile of own
  // keys for a few rows (1.5 us at its share of the memory rate).  us at prefix :
  // own = 1:1 / 4:3 / 5:3 / 2:1 -- 64 requests, 8k prefix, 512 own keys 57 / 52 /
  // 49 / 46; 64, 4k, 1,024 80 / 68 / 60 / 59; 256, 32k, 256 175 / 164 / 163 / 188;
  // 256, 32k, ragged up to 512 187 / 177 / 180 / 205.  The way in and out of the
  // prefix's segment (Q rows, results: 7 us where it is wide) is spread over its
  // tiles: 61 requests with 28 shared and 775 own keys 70 -> 47 us, their prefix
  // being 8 segments of one tile that one block got; nothing from 8k on.
  p.pre_w = p.own_w = 1;
  p.pre_over = 0;
  if (p.pre_tiles > 0 && most_tiles < INT32_MAX / 80) {
    const bool wide_pre = flat_rows > kHalf, wide_own = qv.S * G > kHalf;
    p.pre_w = wide_pre ? 20 : 12;
    p.pre_over = (wide_pre ? 56 : 24) / p.pre_tiles;
    p.own_w = wide_own ? 20 : 12;
  }
  p.page_table = a.page_table; p.table_stride = a.table_stride; p.kv_lens = a.kv_lens; p.new_lens = a.new_lens;
  p.prefix_table = prefix_table;
  p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)qv.D)) * 1.4426950408889634f;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.seg_ctas = reinterpret_cast<int2*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + plan.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o);
  p.own_first = (int)plan.own_first;
  return p;
}

}  // namespace

int64_t most_tiles_of(const bsa_tensor& qv, int64_t Hkv, int64_t page, int64_t max_pages, int64_t prefix_len) {
  const int64_t G = qv.H / Hkv;
  return qv.B * Hkv * cdiv64(qv.S * G, kRowTile) * (cdiv64(max_pages * page, kTileKeys) + cdiv64(prefix_len, kTileKeys)) +
         Hkv * cdiv64(qv.B * qv.S * G, kRowTile) * cdiv64(prefix_len, kTileKeys);
}

unsigned int read_and_clear_paged_error() { return take_error_word(); }

bsa_status launch_paged_wait_probe(unsigned long long limit_ns, cudaStream_t stream) {
  wait_probe_kernel<<<1, 32, 0, stream>>>(limit_ns);
  return cuda_check(cudaGetLastError(), "wait_probe_kernel launch (paged attention)");
}

size_t wide_quant_bytes(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t d, bool prefix, int sms) {
  return plan_paged(B, T, Hq, Hkv, d, prefix, sms).bytes;
}

// The arguments of a launch over 4-bit pages.
static PagedParams quant_params(const bsa_tensor& qv, const QuantArgs& a, const int32_t* new_lens, const int32_t* prefix_table,
                                int32_t prefix_len, int32_t causal, float softmax_scale, void* out, float* lse,
                                void* workspace) {
  const int64_t page = a.k.blocks * kBlockSlots;
  const int sms = num_sms();
  PagedArgs t{};
  t.page_table = a.page_table; t.table_stride = a.table_stride; t.max_pages = a.max_pages; t.kv_lens = a.kv_lens;
  t.new_lens = new_lens;
  PagedParams p = make_params(qv, a.k.heads, page, a.k.pages, t, prefix_table, prefix_len, causal, softmax_scale, out, lse,
                              workspace, plan_paged(qv.B, qv.S, qv.H, a.k.heads, qv.D, prefix_len > 0, sms),
                              most_tiles_of(qv, a.k.heads, page, a.max_pages, prefix_len), sms);
  p.k4 = static_cast<const uint8_t*>(a.k.ptr); p.v4 = static_cast<const uint8_t*>(a.v.ptr);
  p.k4_page = a.k.stride_page; p.k4_head = a.k.stride_head; p.v4_page = a.v.stride_page; p.v4_head = a.v.stride_head;
  p.eights = kEights;
  return p;
}

bsa_status launch_wide_quant(const bsa_tensor& qv, const QuantArgs& a, const int32_t* new_lens, const int32_t* prefix_table,
                             int32_t prefix_len, int32_t causal, float softmax_scale, void* out, float* lse,
                             void* workspace, cudaStream_t stream) {
  const PagedParams p = quant_params(qv, a, new_lens, prefix_table, prefix_len, causal, softmax_scale, out, lse, workspace);
  return qv.D == 128 ? launch_paged<128, true>(p, stream) : launch_paged<64, true>(p, stream);
}

PrefixPart prefix_part(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t d, int sms) {
  const PagedPlan w = plan_paged(B, T, Hq, Hkv, d, true, sms);
  return PrefixPart{w.pre_rt, w.pre_slot_rows, w.own_first};
}

bsa_status launch_prefix_quant(const bsa_tensor& qv, const QuantArgs& a, const int32_t* new_lens,
                               const int32_t* prefix_table, int32_t prefix_len, float softmax_scale, void* seg_ctas,
                               float* part_ml, float* part_o, cudaStream_t stream) {
  QuantArgs alone = a;
  alone.max_pages = 0;
  PagedParams p = quant_params(qv, alone, new_lens, prefix_table, prefix_len, 1, softmax_scale, nullptr, nullptr, nullptr);
  p.seg_ctas = static_cast<int2*>(seg_ctas);
  p.part_ml = part_ml;
  p.part_o = part_o;
  p.early = 1;
  p.beside_keys = (int)(a.max_pages * a.k.blocks * kBlockSlots);
  return qv.D == 128 ? launch_paged<128, true>(p, stream, false) : launch_paged<64, true>(p, stream, false);
}

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsap_forward_workspace_size(int B, int T, int Hq, int Hkv, int d, int has_prefix, int sms) {
  if (B <= 0 || B > kMaxPagedBatch || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq > kMaxHeads || Hq % Hkv ||
      (d != 64 && d != 128) || sms < 0 || (int64_t)B * T * (Hq / Hkv) > INT32_MAX / 16)
    return 0;
  return plan_paged(B, T, Hq, Hkv, d, has_prefix != 0, sms > 0 ? sms : num_sms()).bytes;
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
  if (prefix_len > 0 && (st = check_aligned(fn, "prefix_table", prefix_table, 4)) != BSA_OK) return st;
  if (!out) return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": out is NULL");
  if ((st = check_aligned(fn, "out", out, 16)) != BSA_OK) return st;
  if ((st = check_aligned(fn, "lse", lse, 4)) != BSA_OK) return st;
  if (!std::isfinite(softmax_scale))
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": softmax_scale is not finite");
  // times -inf and log2(e) on the device, where subnormal numbers may count as 0
  if (softmax_scale > 0.f && (softmax_scale < FLT_MIN || softmax_scale > FLT_MAX / 2))
    return set_error(BSA_ERR_INVALID_ARG, std::string(fn) + ": softmax_scale is subnormal or above half the largest float");
  const int64_t G = qv.H / a.k.H;
  const int sms = num_sms();
  // rows, tiles and slot numbers are 32-bit on the device
  const int64_t flat_rows = qv.B * qv.S * G;
  const int64_t q_extent = (qv.B - 1) * qv.stride_b + (qv.S - 1) * qv.stride_s + qv.H * qv.stride_h + qv.D;
  if (q_extent >= (int64_t)1 << 35)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": q reaches over " + s(q_extent) + " elements (2^35 at most)");
  const int64_t most_tiles = most_tiles_of(qv, a.k.H, a.k.S, max_pages, prefix_len);
  if (flat_rows > INT32_MAX / 16 || most_tiles > INT32_MAX / 8 || flat_rows * a.k.H > INT32_MAX)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(flat_rows) + " rows of up to " +
                                              s(max_pages * a.k.S + prefix_len) + " keys are too many for one call");
  const PagedPlan plan = plan_paged(qv.B, qv.S, qv.H, a.k.H, qv.D, prefix_len > 0, sms);
  const size_t need = plan.bytes;
  if (need / (4 * (size_t)qv.D) > INT32_MAX)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": too many rows for one call");
  if (!workspace) return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace is NULL (needs " + s(need) + " bytes)");
  if (ws_bytes < need)
    return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace of " + s(ws_bytes) +
                                            " bytes is smaller than the " + s(need) + " bytes needed");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return set_error(BSA_ERR_WORKSPACE, std::string(fn) + ": workspace is not 256-byte aligned");
  const bsa_tensor ov = contiguous_like(qv, out);
  // What is written against what other blocks, or the join, still read.
  const Bytes writes[] = {bytes_of("out", ov), bytes_at("lse", lse, 4 * qv.B * qv.H * qv.S),
                          bytes_at("workspace", workspace, (int64_t)need)};
  const Bytes reads[] = {bytes_of("q", qv), bytes_of("k_cache", a.k), bytes_of("v_cache", a.v),
                         bytes_at("page_table", max_pages ? page_table : nullptr,
                                  4 * ((qv.B - 1) * table_stride + max_pages)),
                         bytes_at("kv_lens", max_pages ? kv_lens : nullptr, 4 * qv.B), bytes_at("new_lens", new_lens, 4 * qv.B),
                         bytes_at("prefix_table", prefix_len ? prefix_table : nullptr, 4 * cdiv64(prefix_len, a.k.S))};
  for (const Bytes& w : writes)
    for (const Bytes& r : reads)
      if ((st = check_apart(fn, r, w)) != BSA_OK) return st;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(fn, writes[j], writes[i])) != BSA_OK) return st;
  PagedParams p = make_params(qv, a.k.H, a.k.S, a.k.B, a, prefix_table, prefix_len, causal, softmax_scale, out, lse, workspace,
                              plan, most_tiles, sms);
  if ((st = encode_cache(&p.tk, a.k, fn, "k_cache")) != BSA_OK) return st;
  if ((st = encode_cache(&p.tv, a.v, fn, "v_cache")) != BSA_OK) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  return qv.D == 128 ? launch_paged<128, false>(p, cs) : launch_paged<64, false>(p, cs);
}

}  // extern "C"
