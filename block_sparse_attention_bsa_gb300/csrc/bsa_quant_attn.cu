// Attention of new tokens over a paged key/value cache held in 4 bits, whose
// first prefix_len keys all requests share (tcgen05 + TMEM + bulk copies).
//
// Mathematics: that of bsa_paged.cu, with k_j and v_j = codes times scales of
// their groups of 32 channels (bsa_quant.h).  A code times a scale is exact in
// bf16, so that the products are those of bf16 pages that hold the same values.
//
// Layout of the work:
//  * The keys are the rows of the products, S^T = K Q^T and O^T += V^T P^T: K and
//    V become bf16 on their way from the pages' bytes, a thread a key of K or a
//    channel of V, straight into TMEM, where the tensor cores take their first
//    operand from; Q and P, which are few rows, are the second, in shared memory.
//    (As second operands K and V would go through shared memory, which a tile
//    would then pass 195 KB of, where it now passes 45.)
//  * A segment is up to N query rows that read the same keys: for the prefix any N
//    rows (b, i, g) of the whole batch under one KV head, for a request's own keys
//    the rows (i, g) of that request.  All segments' tiles of 128 keys are put in
//    one row and cut into equal pieces, one for each CTA, whatever the lengths are
//    (they are read from the device); a segment's way in and out counts as a tile (24
//    heads of one row 75 -> 70 us, five drafts 15.6 -> 14.2).  A cut segment, or one beside a prefix, leaves
//    partial results that quant_join_kernel puts together; segment + CTA numbers them.
//  * Four CTAs per SM, each through its piece by itself: while one waits for its
//    products or its data the others work, with no hand-over between them.  (One CTA
//    of 20 warps, each role's warps handing tiles to the next role's, took 1,790
//    cycles a tile, most of it in one warp's way through its part of a tile.)  A CTA's
//    warp 4 goes through its segments, loads their Q rows, copies each tile's blocks
//    page by page into three places (K_0, V_0, K_1, V_1 ..) and issues the products;
//    warps 0-3 turn K into bf16, a key per thread, scores into weights, and V into
//    bf16, a channel per thread, over K's place in TMEM.
//  * A code without its scale takes half an instruction (bare_codes).  So the scales
//    stand beside the products where TMEM has columns for a set per group of 32
//    channels, up to 8 rows of heads of 128 and 16 of 64: with the scales in K and V,
//    24 heads of one row took 89 us instead of 74.
//  * The maximum of a row moves only when a score passes it by more than 2^8, so that
//    most tiles need one barrier of the four warps.
//  * A prefix of more rows than a segment's, unless it is short, is the work of bsa_paged.cu's
//    kernel (its rows are the products' rows), which runs beside this one on SMs shared
//    out by their tiles; the join reads the partial results of both.  64 requests on one
//    prompt of 8,209 keys, up to 1,024 own ones each: 35 us; this kernel alone 83, that
//    one alone 50.
//
// Bound by instructions: a tile of 128 keys takes an SM about 1,150 cycles, in which its
// schedulers issue 65 to 70 % of the time (2.9 instructions a value of K and V, of
// which 1.3 make bf16 of the codes); DRAM could bring a tile of heads of 128 in 748.
// Device times, of the measured copy rate: 16 requests of 1,024 to 65,536 keys, 32
// heads over 8 of 128: 135 us (69 %); 20 of 500 to 9,000 keys, 24 heads of one row each:
// 70 us (59 %); one request of 4,097 keys 9.1 us, of which 4 are the way in, the join
// and the launches; 24 requests with five drafts on 1,000 shared keys, heads of 64: 14 us.
#include <cuda_bf16.h>
#include <math_constants.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <string>

#include "bsa_paged_device.cuh"
#include "bsa_quant.h"

namespace bsa {
namespace {

constexpr int kTileKeys = 128;
constexpr int kTileBlocks = kTileKeys / kBlockSlots;
constexpr int kThreads = 160;
constexpr int kCtasPerSm = 4;        // 16 x 8,192 keys in 44 us; three 47, five (72 registers a thread) 45
constexpr int kMaxBlocks = kMaxPagedBatch / 32;      // blocks of 32 requests in the schedule
constexpr float kLowest = -3e38f;                    // stands for a maximum of no score yet

// R: rows of a segment.  kBare: K and V are made of the codes alone, and the scales
// stand beside the products: S has a set of columns for each group of 32 channels,
// whose rows of Q are 0 in the others, and so has P, each set times its group's
// scales of V.  Else (16 rows of heads of 128, whose sets TMEM has no room for) the
// scales are multiplied into K and V.
template <int D, int R>
struct Cfg {
  static constexpr bool kBare = D / kGroup * R <= 32;
  static constexpr int kGroups = D / kGroup;
  static constexpr int kSets = kBare ? kGroups : 1;
  static constexpr int kCols = kSets * R < 16 ? 16 : kSets * R;        // columns of S and of O, rows of Q and of P
  static constexpr int kSegSlots = R == 4 ? 3 : 2;                     // segments, with their Q rows
  static constexpr int kQBytes = kCols * D * 2;                        // as the MMAs read them
  static constexpr int kQSlotBytes = kBare ? R * D * 2 : kQBytes;      // of a segment; bare: as they come
  static constexpr int kQTotal = kSegSlots * kQSlotBytes + (kBare ? kQBytes : 0);
  static constexpr int kPBytes = kCols * kTileKeys * 2;
  static constexpr int kTileBytes = kTileBlocks * block_bytes(D);      // of K or of V
  static constexpr int kSlots = 3;                                     // places for the blocks of a tile of K or of V
  static constexpr int kScaleBytes = kBare ? 0 : kGroups * kTileKeys * 2;
  static constexpr int kAhead = kBare ? 1 : 0;         // quarters of a tile made before their place is free
  static constexpr int kBarBytes = 2048;
  static constexpr int kSmemBytes = 1024 + kQTotal + kPBytes + kSlots * kTileBytes + kScaleBytes + kBarBytes;
  static constexpr int kA = 0, kS = 64, kO = kS + kCols, kColumns = 128;       // TMEM columns: K, then V; S; O
  static_assert(kPBytes % 1024 == 0 && kQBytes % 1024 == 0, "the MMAs' rows are exchanged within 1024 bytes");
  static_assert(kO + kCols <= kColumns && kCtasPerSm * kColumns <= 512 && kCtasPerSm * (kSmemBytes + 1024) <= 233472, "an SM's columns and shared memory");
};

struct QAttnParams {
  const uint8_t* k; const uint8_t* v;
  int64_t k_page, k_head, v_page, v_head;      // byte strides
  const __nv_bfloat16* q;
  int64_t q_sb, q_ss, q_sh;
  int B, T, Hq, Hkv, G, page_shift, num_pages, max_pages, prefix_len, causal;
  FastDiv div_G, div_TG;
  int R;                          // rows of a segment
  int TG;                         // rows of a request under one KV head
  int pre_rt;                     // row tiles of the whole batch (prefix)
  int pre_tiles;                  // key tiles of the prefix
  int pre_slot_rows, own_slot_rows;   // rows of a partial result
  int ctas;
  int wide_ctas;                  // CTAs of the launch before, which has the prefix (pre_tiles is 0 here), or 0
  const int32_t* page_table; int64_t table_stride;
  const int32_t* kv_lens; const int32_t* new_lens;
  const int32_t* prefix_table;
  float scale_log2;
  uint32_t eights;                // kEights
  __nv_bfloat16* out;
  float* lse;
  int2* seg_ctas;                 // workspace: first and last CTA of each segment that has tiles
  float* part_ml;                 // workspace: partial results' (max, sum) and rows,
  float* part_o;                  // those of the prefix first,
  int own_first;                  // from here on those of own keys
};

// A length, from behind L1: the schedule reads it beside the fence that the rest of the
// kernel stands behind (a fence in front of it took 1 us more).
__device__ __forceinline__ int load_length(const int32_t* x) {
  int v;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(x) : "memory");
  return v;
}
// Request b's own keys and new tokens, clamped to what the tables hold.
__device__ __forceinline__ int own_keys(const QAttnParams& p, int b) {
  if (p.max_pages == 0) return 0;
  return min(max(load_length(p.kv_lens + b), 0), p.max_pages << p.page_shift);
}
__device__ __forceinline__ int new_tokens(const QAttnParams& p, int b) {
  return p.new_lens ? min(max(load_length(p.new_lens + b), 0), p.T) : p.T;
}
// Own keys that row i of a request with kv keys and n new tokens sees.
__device__ __forceinline__ int seen_keys(const QAttnParams& p, int kv, int n, int i) {
  return p.causal ? min(max(kv - n + i + 1, 0), kv) : kv;
}
// Key tiles of such a request under one KV head (whose rows are one segment's).
__device__ __forceinline__ int own_tiles(const QAttnParams& p, int kv, int n) {
  return n > 0 ? (seen_keys(p, kv, n, n - 1) + kTileKeys - 1) / kTileKeys : 0;
}
// Places in the row that a segment of so many tiles takes: its way in and out, then its tiles.
__device__ __forceinline__ int segment_units(int tiles) { return tiles > 0 ? kSegmentWay + tiles : 0; }

// The row of all segments, cut into equal pieces.
struct Cut {
  int n, q, r;                    // CTAs that get some; units = q n + r
  __device__ __forceinline__ Cut(const QAttnParams& p, int own, int ctas) {
    const int units = segment_units(p.pre_tiles) * p.pre_rt * p.Hkv + own;
    n = min(ctas, units);
    q = n > 0 ? units / n : 0;
    r = units - q * n;
  }
  __device__ __forceinline__ int begin(int c) const { return c * q + min(c, r); }
};

// A segment's part that one CTA works on, as it stands in the segment ring.
struct __align__(16) Segment {
  int b;               // request, -1: prefix
  int hk;
  int row0, rows;      // first flat row (b * T + i) * G + g, and how many
  int tile0, tiles;    // first key tile and how many; 0: no further segment
  int slot;            // number of the partial result (segment + CTA)
  int keys;            // where its keys end
  int kv, n;           // of the request
  int whole;           // this CTA has all tiles of the segment
  int pad;
};

// A barrier of warps 0-3 that tells all of them whether some thread says yes.  No
// warp leaves them between two of these but all together, so that none waits for one
// that gave up.
__device__ __forceinline__ bool sync_any(bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)mine)
      : "memory");
  return r != 0;
}

// 4, 8, 16 or 32 consecutive 32-bit columns of this thread's lane.
__device__ __forceinline__ void tmem_ld_4(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3])
               : "r"(taddr)
               : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, float* r) {
  if constexpr (N == 32) {
    tmem_ld32f(taddr, r);
  } else if constexpr (N == 4) {
    tmem_ld_4(taddr, r);
  } else if constexpr (N == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    static_assert(N == 16, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
  }
}
__device__ __forceinline__ void tmem_st_4(uint32_t taddr, const float* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "f"(r[0]), "f"(r[1]), "f"(r[2]),
               "f"(r[3])
               : "memory");
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) quant_attention_kernel(const __grid_constant__ QAttnParams p) {
  using C = Cfg<D, R>;
  constexpr bool kBare = C::kBare;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t p_smem = smem_u32(smem);                              // P rows
  const uint32_t q_smem = p_smem + C::kPBytes;                         // bare: Q as the MMAs read it; [kSegSlots] Q rows
  const uint32_t q_rows = q_smem + (kBare ? C::kQBytes : 0);
  const uint32_t ring = q_smem + C::kQTotal;                           // [kSlots] blocks of K_0, V_0, K_1, V_1 ..
  const uint32_t vscale = ring + C::kSlots * C::kTileBytes;          // [D / 32][128] twice the scales of V, bf16
  uint8_t* rest = smem + (vscale - p_smem) + C::kScaleBytes;
  float* mr = reinterpret_cast<float*>(rest);                          // [R] running maxima
  float* of_row = mr + R;                                              // [R] factors, then sums
  Segment* segs = reinterpret_cast<Segment*>(of_row + R);           // [kSegSlots]
  int* block_units = reinterpret_cast<int*>(segs + C::kSegSlots);      // [kMaxBlocks] units of own keys of requests 32 i ..
  int* block_sum = block_units + kMaxBlocks;                           // [kMaxBlocks] and of those before
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(block_sum + kMaxBlocks);
  int* abort_slot = block_sum + kMaxBlocks + 1;
  // barriers, as shared-memory addresses 8 bytes apart
  const uint32_t seg_full = smem_u32(block_sum + kMaxBlocks + 2);           // [kSegSlots] the segment, and 32 lanes' copies of Q rows
  const uint32_t seg_empty = seg_full + 8 * C::kSegSlots;        // [kSegSlots] 4 warps
  const uint32_t full = seg_empty + 8 * C::kSegSlots;            // [kSlots] transaction bytes
  const uint32_t k_ready = full + 8 * C::kSlots;                 // 4 warps: K stands in TMEM
  const uint32_t s_done = k_ready + 8;                           // commit
  const uint32_t pv_ready = s_done + 8;                          // 4 warps: V stands in TMEM, P in shared memory
  const uint32_t pv_done = pv_ready + 8;                         // commit
  const uint32_t mma_end = pv_done + 8;                          // commit
  static_assert((2 * R + 2 * kMaxBlocks + 2) * 4 + C::kSegSlots * sizeof(Segment) + (2 * C::kSegSlots + C::kSlots + 5) * 8 <=
                    C::kBarBytes, "barrier block");
  const uint32_t abort_flag = smem_u32(abort_slot);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSegSlots; ++i) {
      mbar_init(seg_full + 8 * i, 33);
      mbar_init(seg_empty + 8 * i, 4);
    }
    for (int i = 0; i < C::kSlots; ++i) mbar_init(full + 8 * i, 1);
    mbar_init(k_ready, 4);
    mbar_init(s_done, 1);
    mbar_init(pv_ready, 4);
    mbar_init(pv_done, 1);
    mbar_init(mma_end, 1);
    *abort_slot = 0;
    fence_mbar_init();
  }
  if constexpr (kBare) {                           // what is not of a row's group stays 0
    for (int i = threadIdx.x; i < C::kQBytes / 16; i += kThreads) reinterpret_cast<uint4*>(smem + C::kPBytes)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), C::kColumns);
    tmem_relinquish();
  }
  // Launched when the blocks of the kernel before leave: up to here nothing is
  // read or written that it uses.  The join may then come in as room is left (its
  // launch shows less: one token 9.9 -> 9.2 us).  Beside the prefix's kernel, which has
  // waited for what came before it and shares nothing with this one, one CTA waits at
  // the end, as the join behind waits for this kernel only; the join is not let in
  // before, when the SMs with room are few.  What came before both is read without a
  // wait then: the lengths from behind L1, all else behind the fence and the barrier (64
  // requests on 1,200 keys 0.8 us more than without the fence).
  if (p.wide_ctas == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 32) {
    fence_waited();
    if (p.wide_ctas == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  // the schedule: units of own keys per block of 32 requests; warp 4, which looks for
  // segments, keeps the first block's
  const int nblk = (p.B + 31) / 32;
  int kv = 0, n = 0, mine = 0, upto = 0;           // of this lane's request: keys, new tokens, units under a head, units up to its end
#pragma unroll 1
  for (int blk = 4 - warp; blk < nblk; blk += kThreads / 32) {
    const int b = blk * 32 + lane;
    const int kv_b = b < p.B ? own_keys(p, b) : 0, n_b = b < p.B ? new_tokens(p, b) : 0;
    const int mine_b = segment_units(own_tiles(p, kv_b, n_b));
    const int incl = warp_inclusive_sum(mine_b * p.Hkv);
    if (lane == 31) block_units[blk] = incl;
    if (blk == 0) { kv = kv_b; n = n_b; mine = mine_b; upto = incl; }
    if (cta == 0 && b < p.B && p.max_pages > 0) {
      const int given = load_length(p.kv_lens + b);
      if (given < 0 || given > p.max_pages << p.page_shift) atomicOr(&g_bsa_error, kErrPage);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int total = 0;
#pragma unroll 1
  for (int i = 0; i < nblk; i += 32) {
    const int v = i + lane < nblk ? block_units[i + lane] : 0;
    const int incl = warp_inclusive_sum(v) + total;
    if (warp == 4 && i + lane < nblk) block_sum[i + lane] = incl - v;
    total = __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
  const uint32_t tmem_a = *tmem_slot + C::kA, tmem_s = *tmem_slot + C::kS, tmem_o = *tmem_slot + C::kO;
  int begin = 0, end = 0;
  {
    // beside the prefix's kernel: the SMs that it leaves (the first CTAs are placed there,
    // those behind have no tiles)
    int ctas = p.ctas;
    if (p.wide_ctas > 0)
      ctas = kCtasPerSm * max(p.wide_ctas - prefix_sms(p.wide_ctas, (p.prefix_len + kTileKeys - 1) / kTileKeys * p.pre_rt * p.Hkv,
                                                       p.B * p.TG > kWideHalf, total), 1);
    const Cut cut(p, total, ctas);
    if (cta < cut.n) {
      begin = cut.begin(cta);
      end = cut.begin(cta + 1);
    }
  }
  bool ok = true;

  if (warp == 4) {
    // ------------------------------- segments, Q rows, copies of tiles, MMAs ---
    // In turn: S of tile i, V of tile i + 1, P V of tile i, K of tile i + 2, whose segment
    // is found where a new one begins.
    // Lane l holds request 32 blk + l: its lengths, units, and the units up to its end.
    constexpr int kVec = D / 8;                    // 16-byte pieces of a row
    constexpr int kRowsPer = 32 / kVec;            // rows per warp-wide copy
    constexpr uint32_t idesc = idesc_bf16_f32(128, C::kCols, false);
    constexpr int kChunk = (C::kCols * 128) >> 4;
    const uint64_t pdesc = sdesc_sw128(p_smem, 16, 1024);
    const int c = lane % kVec;
    const int pre_units = segment_units(p.pre_tiles), pre = pre_units * p.pre_rt * p.Hkv;
    int blk = 0, blk_end = __shfl_sync(0xffffffffu, upto, 31);
    // Lane x copies page x of a tile.
    const int per_tile = p.page_shift >= 7 ? 1 : kTileKeys >> p.page_shift;      // pages of a tile
    const int per_page = kTileBlocks / per_tile;                                 // blocks of a page in it
    const bool copies = lane < per_tile;
    int at_unit = begin;                           // up to where segments have been found
    int tiles = INT32_MAX;                         // of this CTA, once the last segment is known
    uint32_t seg_no = 0;                           // segments found
    int left = 0, tile = 0, keys = 0, page = 0;    // of the last one: tiles to copy, the next, where its keys end, this lane's page
    const int32_t* table = nullptr;
    const uint8_t* k_head = nullptr;
    const uint8_t* v_head = nullptr;
    uint32_t starts = 0;                           // bit i % 4: tile i is the first of a segment
    auto page_of = [&](int t) {
      const int key = t * kTileKeys + lane * per_page * kBlockSlots;
      return copies && key < keys ? table[key >> p.page_shift] : 0;          // looked at when it is used
    };
    // The segment at the row's unit at_unit, as far as it is this CTA's; one of no tiles
    // when there is none.
    auto find_segment = [&]() {
      Segment s{};
      int seg = 0, start = 0, m = 0;               // its number, first unit, tiles
      left = 0;
      if (at_unit < end) {
        if (at_unit < pre) {
          seg = at_unit / pre_units;
          start = seg * pre_units;
          m = p.pre_tiles;
          s.b = -1;
          s.hk = seg / p.pre_rt;
          s.row0 = (seg - s.hk * p.pre_rt) * R;
          s.rows = min(R, p.B * p.TG - s.row0);
          s.keys = p.prefix_len;
        } else {
          const int u = at_unit - pre;
          if (u >= blk_end) {                          // the last block that begins at or before u
            ++blk;
            while (blk + 1 < nblk && block_sum[blk + 1] <= u) ++blk;
            const int b = blk * 32 + lane;
            kv = b < p.B ? own_keys(p, b) : 0;
            n = b < p.B ? new_tokens(p, b) : 0;
            mine = b < p.B ? segment_units(own_tiles(p, kv, n)) : 0;
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
          s.row0 = s.b * p.TG;
          s.rows = s.n * p.G;
          s.keys = s.kv;
          seg = s.b * p.Hkv + s.hk;
          start = pre + first + s.hk * per_head;
          m = per_head - kSegmentWay;
        }
        s.tile0 = max(at_unit - start - kSegmentWay, 0);
        left = max(min(m, end - start - kSegmentWay) - s.tile0, 0);
        s.tiles = left;
        s.whole = left == m;
        s.slot = seg + cta;
        at_unit = start + kSegmentWay + m;
        // its first tile's pages are on their way while its place is waited for
        tile = s.tile0; keys = s.keys;
        table = s.b < 0 ? p.prefix_table : p.page_table + s.b * p.table_stride;
        k_head = p.k + s.hk * p.k_head;
        v_head = p.v + s.hk * p.v_head;
        page = left > 0 ? page_of(tile) : 0;
      }
      const uint32_t qb = seg_no % C::kSegSlots;
      if (!warp_wait(seg_empty + 8 * qb, (seg_no / C::kSegSlots & 1u) ^ 1u, abort_flag)) return false;
      if (lane == 0) {
        int2* who = p.seg_ctas + (s.b < 0 ? 0 : p.pre_rt * p.Hkv) + seg;     // the join looks here
        if (left > 0 && s.tile0 == 0) who->x = cta;
        if (left > 0 && s.tile0 + left == m) who->y = cta;
        segs[qb] = s;
        mbar_arrive(seg_full + 8 * qb);
      }
      __syncwarp();
      ++seg_no;
      if (left == 0) {
        mbar_arrive(seg_full + 8 * qb);
        return true;
      }
      // Q rows, and rows of zeros up to a multiple of four
      const __nv_bfloat16* qh = p.q + (int64_t)s.hk * p.G * p.q_sh + c * 8;
      const uint32_t to = q_rows + qb * C::kQSlotBytes;
      const int row = s.row0 + min(lane, s.rows - 1);
      const int b = p.div_TG.quot(row), rem = row - b * p.TG, i = p.div_G.quot(rem), g = rem - i * p.G;
      const uint32_t off = (uint32_t)((b * p.q_sb + i * p.q_ss + g * p.q_sh) / 8);    // below 2^32: host check
#pragma unroll 4
      for (int y = 0; y * kRowsPer < ((s.rows + 3) & ~3); ++y) {
        const int r = y * kRowsPer + lane / kVec;
        const __nv_bfloat16* src = qh + (uint64_t)__shfl_sync(0xffffffffu, off, r) * 8;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         to + (kBare ? r * (D * 2) + c * 16 : (c / 8) * (C::kCols * 128) + r * 128 + ((c % 8) ^ (r % 8)) * 16)),
                     "l"(src), "r"(r < s.rows ? 16 : 0)
                     : "memory");
      }
      // arrives when this lane's copies have landed; the warp goes on
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(seg_full + 8 * qb) : "memory");
      return true;
    };
    // The copies that have a place: K of tile i where V of tile i - 2 stood, once P V of
    // that has been asked for; V of tile i where K of tile i - 1 stood, once that is in
    // TMEM.  (A segment's place is that of the kSegSlots-th before it, all P V of which
    // have been asked for by then: its results are on their way out.)
    int copied = 0, s_issued = 0, pv_issued = 0;   // tiles of K and of V, S, P V
    auto copy_tiles = [&]() {
#pragma unroll 1
      for (;; ++copied) {
        const int i = copied >> 1;
        const bool v = copied & 1;
        if (i >= tiles || (v ? i > s_issued : i > pv_issued + 1)) return true;
        if (!v) {
          starts &= ~(1u << (i & 3));
          if (left == 0) {
            if (!find_segment()) return false;
            if (left == 0) {
              tiles = i;
              return true;
            }
            starts |= 1u << (i & 3);
          }
        }
        if (page < 0 || page >= p.num_pages) {
          atomicOr(&g_bsa_error, kErrPage);
          page = 0;
        }
        const int blocks = (min(keys - tile * kTileKeys, kTileKeys) + kBlockSlots - 1) / kBlockSlots;
        const int count = min(blocks - lane * per_page, per_page);
        const int in_page = tile * kTileBlocks & ((1 << (p.page_shift - 4)) - 1) & ~(per_page - 1);
        const uint32_t at = copied % C::kSlots;
        if (lane == 0) mbar_arrive_expect_tx(full + 8 * at, blocks * block_bytes(D));
        __syncwarp();
        if (copies && count > 0)
          bulk_load(ring + at * C::kTileBytes + lane * per_page * block_bytes(D),
                    (v ? v_head + page * p.v_page : k_head + page * p.k_page) + in_page * block_bytes(D), count * block_bytes(D),
                    full + 8 * at);
        if (v) {
          ++tile;
          if (--left > 0) page = page_of(tile);
        }
      }
    };
    ok = copy_tiles();
    uint32_t qb = C::kSegSlots - 1;                // of the tile's segment
    bool first = false;
#pragma unroll 1
    for (int i = 0; i < tiles && ok; ++i) {
      first = starts >> (i & 3) & 1u;
      if (first && ++qb == C::kSegSlots) qb = 0;
      if (!(ok = warp_wait(k_ready, i & 1, abort_flag))) break;
      fence_async_shared();                        // Q rows, which who made K has waited for, come by ordinary copies
      tc_fence_after();
      const uint64_t qdesc = sdesc_sw128(q_smem + (kBare ? 0 : qb * C::kQBytes), 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)((kk / 4) * kChunk + (kk % 4) * 2);
          if (kk == 0) mma_ts_acc<0>(tmem_s, tmem_a, qdesc, idesc);
          else mma_ts_acc<1>(tmem_s, tmem_a + kk * 8, qdesc + off, idesc);
        }
        mma_commit(s_done);
      }
      __syncwarp();
      ++s_issued;
      if (!(ok = copy_tiles())) break;
      if (!(ok = warp_wait(pv_ready, i & 1, abort_flag))) break;
      tc_fence_after();
      if (elect_one()) {
        mma_ts(tmem_o, tmem_a, pdesc, idesc, !first);
#pragma unroll
        for (int kk = 1; kk < kTileKeys / 16; ++kk)
          mma_ts_acc<1>(tmem_o, tmem_a + kk * 8, pdesc + (uint64_t)((kk / 4) * kChunk + (kk % 4) * 2), idesc);
        mma_commit(pv_done);
      }
      __syncwarp();
      ++pv_issued;
      ok = copy_tiles();
    }
    // Nothing is in flight when the CTA leaves or frees its TMEM, after an abort either.
    if (elect_one()) {
#pragma unroll 1
      for (int i = max(copied - C::kSlots, 0); i < copied; ++i) mbar_drain(full + 8 * (i % C::kSlots), i / C::kSlots & 1);
      mma_commit(mma_end);
      mbar_drain(mma_end, 0);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  } else {
    // ------------------------------------------- codes, products, weights, results ---
    const int th = threadIdx.x;                    // key of a tile, and channel of V and O
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t a_t = tmem_a + lanes, s_t = tmem_s + lanes;
    // of a set of weights for each group, the columns of this channel's
    const uint32_t o_t = tmem_o + lanes + (kBare ? warp % C::kGroups * R : 0);
    const uint32_t slot_at = (th / kBlockSlots) * block_bytes(D), slot = th % kBlockSlots;
    // where this key's weights stand in P: rows of 64 keys, 16-byte pieces exchanged within 8 rows
    uint32_t p_at[8];                              // of rows r, r % 8 = 0 .. 7, but for 128 r
#pragma unroll
    for (int r = 0; r < 8; ++r) p_at[r] = (p_smem + (th / 64) * (C::kCols * 128) + th % 64 * 2) ^ (r << 4);
    // Joins a value of each thread for every row over the 128 threads, by way of P's
    // memory (128 / kPass threads a row), and gives it to one of them.
    constexpr int kPass = C::kPBytes / 512 < R ? C::kPBytes / 512 : R, kShare = 128 / kPass;
    float* const scratch = reinterpret_cast<float*>(smem);
    auto rows_of_threads = [&](const float* x, auto first, auto join, auto put) {
#pragma unroll
      for (int r0 = 0; r0 < R; r0 += kPass) {
        if (r0 > 0) sync_any(false);
#pragma unroll
        for (int r = 0; r < kPass; ++r) scratch[r * 128 + th] = first(x[r0 + r]);
        sync_any(false);
        float y;
#pragma unroll
        for (int i = 0; i < kPass / 4; ++i) {
          const float4 f = reinterpret_cast<const float4*>(scratch + th / kShare * 128)[th % kShare + i * kShare];
          const float z = join(join(f.x, f.y), join(f.z, f.w));
          y = i == 0 ? z : join(y, z);
        }
#pragma unroll
        for (int o = kShare / 2; o > 0; o >>= 1) y = join(y, __shfl_xor_sync(0xffffffffu, y, o));
        if (th % kShare == 0) put(r0 + th / kShare, y);
      }
    };
    uint32_t it = 0, seg_no = 0;
#pragma unroll 1
    for (;; ++seg_no) {
      const uint32_t qb = seg_no % C::kSegSlots;
      ok = warp_wait(seg_full + 8 * qb, seg_no / C::kSegSlots & 1u, abort_flag);
      const Segment& s = segs[qb];                 // stays there until all are through with it
      if (th < R) mr[th] = kLowest;
      const bool none = s.tiles == 0;
      if (kBare && !none) {
        // Q rows of each group, 0 elsewhere; every second pair of channels by 8, as K's
        // codes there come out 8 times as large (all S so far are done)
#pragma unroll
        for (int x = th; x < R * D / 4; x += 128) {
          const int r = x / (D / 4), ch = x % (D / 4) * 4, n = ch / kGroup * R + r;
          uint2 q4 = lds64(q_rows + qb * C::kQSlotBytes + x * 8);
          q4.y = as_u32(__hmul2(as_bf16x2(q4.y), as_bf16x2(0x3E003E00u)));
          sts64(q_smem + (ch / 64) * (C::kCols * 128) + n * 128 + ((ch % 64 / 8) ^ (n % 8)) * 16 + ch % 8 * 2, q4);
        }
        fence_async_shared();
      }
      if (sync_any(!ok || none)) break;
      const int rows = s.rows, tiles = s.tiles, keys = s.keys, tile0 = s.tile0;
      const int sb = s.b, skv = s.kv, sn = s.n;
      // the keys of the first row; further rows' rise with the token
      const int rem0 = s.row0 - sb * p.TG;
      const bool even = sb < 0 || !p.causal;
      const int least = even ? keys : seen_keys(p, skv, sn, p.div_G.quot(rem0));
      float l[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = 0.f;
      int j = 0;
#pragma unroll 1
      for (; j < tiles; ++j, ++it) {
        const uint32_t nk = 2 * it, nv = nk + 1, k_at = nk % C::kSlots, v_at = nv % C::kSlots;
        const int tile_keys = min(keys - (tile0 + j) * kTileKeys, kTileKeys);
        const uint32_t k_tile = ring + k_at * C::kTileBytes, v_tile = ring + v_at * C::kTileBytes;
        // K, made while P V of the tile before, whose V it takes the place of, is on its way
        ok = warp_wait(full + 8 * k_at, nk / C::kSlots & 1u, abort_flag) && ok;
        uint32_t ab[16];                           // of K, then of V: 32 of this thread's values
        {
          const uint32_t from = k_tile + slot_at + slot * 16;
          const uint32_t scale_at = k_tile + slot_at + code_bytes(D) + slot;
          auto group = [&](int g, uint32_t* r) {
            const uint4 c = lds128(from + g * 256);
            const uint32_t word[4] = {c.x, c.y, c.z, c.w};
            if constexpr (kBare) {
#pragma unroll
              for (int i = 0; i < 4; ++i) bare_codes(word[i], r + 4 * i);
            } else {
              const uint32_t s2 = twice_scale(lds8(scale_at + g * kBlockSlots)) * 0x10001u, off = scale_offset(s2);
#pragma unroll
              for (int i = 0; i < 16; ++i) r[i] = code_values(raised_codes(word[i / 4], i % 4, p.eights), s2, off);
            }
          };
#pragma unroll
          for (int g = 0; g < C::kAhead; ++g) group(g, ab);
          ok = warp_wait(pv_done, (it & 1u) ^ 1u, abort_flag) && ok;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < C::kAhead; ++g) tmem_st16(a_t + g * 16, ab);
#pragma unroll kBare ? 4 : 1
          for (int g = C::kAhead; g < C::kGroups; ++g) {
            group(g, ab);
            tmem_st16(a_t + g * 16, ab);
          }
        }
        // This key's scales, times what the codes lack; not finite: NaN, but 0 behind the
        // last key, whatever stands there.
        auto read_scales = [&](uint32_t tile, int n, float* s) {
          uint32_t most = 0;
#pragma unroll
          for (int g = 0; g < C::kSets; ++g) {
            const uint32_t b = lds8(tile + slot_at + code_bytes(D) + g * kBlockSlots + slot);
            s[g] = scale_float(b, n);
            most = max(most, b);
          }
          if (most == 255u) {
#pragma unroll
            for (int g = 0; g < C::kSets; ++g)
              if (lds8(tile + slot_at + code_bytes(D) + g * kBlockSlots + slot) == 255u) s[g] = th < tile_keys ? CUDART_NAN_F : 0.f;
          }
        };
        float ks[C::kSets];
        if constexpr (kBare) read_scales(k_tile, 6, ks);
        // twice the scales of V, 0 behind the last key: what stands there must not count
        if constexpr (!kBare) {
          ok = warp_wait(full + 8 * v_at, nv / C::kSlots & 1u, abort_flag) && ok;
#pragma unroll
          for (int g = 0; g < C::kGroups; ++g)
            sts16(vscale + (g * kTileKeys + th) * 2,
                  th < tile_keys ? twice_scale(lds8(v_tile + slot_at + code_bytes(D) + g * kBlockSlots + slot)) : 0u);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_ready);
        // V of slots 32 x .. 32 x + 31 under this thread's channel
        auto v_codes = [&](int x, uint32_t* r) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint2 c = lds64(v_tile + (2 * x + y) * block_bytes(D) + th * 8);
            if constexpr (kBare) {
              bare_codes(c.x, r + y * 8);
              bare_codes(c.y, r + y * 8 + 4);
            } else {
              const uint32_t scale_at = vscale + (th / kGroup) * (kTileKeys * 2) + (2 * x + y) * 32;
              const uint4 sa = lds128(scale_at), sb = lds128(scale_at + 16);
              const uint32_t s2[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
              for (int i = 0; i < 8; ++i)
                r[y * 8 + i] = code_values(raised_codes(i < 4 ? c.x : c.y, i % 4, p.eights), s2[i], scale_offset(s2[i]));
            }
          }
        };
        float vs[C::kSets];
        if constexpr (kBare) {
          ok = warp_wait(full + 8 * v_at, nv / C::kSlots & 1u, abort_flag) && ok;
          read_scales(v_tile, th & 2 ? 3 : 6, vs);
          if (th < D) {
#pragma unroll
            for (int x = 0; x < C::kAhead; ++x) v_codes(x, ab);
          }
        }
        ok = warp_wait(s_done, it & 1u, abort_flag) && ok;
        tc_fence_after();
        if constexpr (!kBare) sync_any(false);   // the scales of V are there
        const int key = (tile0 + j) * kTileKeys + th;
        const bool cut = (tile0 + j + 1) * kTileKeys > least;       // some row does not see all of the tile
        float v[R];
        bool grow = j == 0, again = false;
#pragma unroll 1
        for (;;) {
          // Scores in units of log 2, those of keys that a row does not see -inf.
          {
            float d[C::kSets * R];
            tmem_ld_n<C::kSets * R>(s_t, d);
            tmem_wait_ld();
#pragma unroll
            for (int r = 0; r < R; r += 2) {
              float2 z = make_float2(d[r], d[r + 1]);
              if constexpr (kBare) {
                z = __fmul2_rn(z, make_float2(ks[0], ks[0]));
#pragma unroll
                for (int g = 1; g < C::kGroups; ++g)
                  z = __ffma2_rn(make_float2(d[g * R + r], d[g * R + r + 1]), make_float2(ks[g], ks[g]), z);
              }
              z = __fmul2_rn(z, make_float2(p.scale_log2, p.scale_log2));
              v[r] = z.x;
              v[r + 1] = z.y;
            }
          }
          if (cut) {
            if (even) {
#pragma unroll
              for (int r = 0; r < R; ++r)
                if (key >= least) v[r] = -INFINITY;
            } else {
#pragma unroll
              for (int r = 0; r < R; ++r)
                if (key >= min(seen_keys(p, skv, sn, p.div_G.quot(rem0 + r)), keys)) v[r] = -INFINITY;
            }
          }
          if (grow) {
            // The maximum moves to the largest score so far: of rows that some threads
            // share, written where P will stand (NaN, and what is below kLowest, as that).
            rows_of_threads(
                v, [](float z) { return z > kLowest ? z : kLowest; }, [](float a, float b) { return fmaxf(a, b); },
                [&](int r, float top) {
                  const float m = mr[r];
                  mr[r] = fmaxf(m, top);
                  of_row[r] = ex2_approx(m - fmaxf(m, top));
                });
            sync_any(false);
#pragma unroll
            for (int r4 = 0; r4 < R; r4 += 4)
              if (r4 < rows) {
                const float4 a = *reinterpret_cast<const float4*>(of_row + r4);
                l[r4] *= a.x; l[r4 + 1] *= a.y; l[r4 + 2] *= a.z; l[r4 + 3] *= a.w;
                if (j > 0) {
                  float o[4];
                  tmem_ld_4(o_t + r4, o);
                  tmem_wait_ld();
                  o[0] *= a.x; o[1] *= a.y; o[2] *= a.z; o[3] *= a.w;
                  tmem_st_4(o_t + r4, o);
                }
              }
            if (j > 0) tmem_wait_st();
          }
          float top = -INFINITY;
#pragma unroll
          for (int r4 = 0; r4 < R; r4 += 4)
            if (r4 < rows) {
              const float4 m = *reinterpret_cast<const float4*>(mr + r4);
              const float2 e01 = __fadd2_rn(make_float2(v[r4], v[r4 + 1]), make_float2(-m.x, -m.y));
              const float2 e23 = __fadd2_rn(make_float2(v[r4 + 2], v[r4 + 3]), make_float2(-m.z, -m.w));
              const float e[4] = {e01.x, e01.y, e23.x, e23.y};
              top = max3f(max3f(top, e[0], e[1]), e[2], e[3]);
#pragma unroll
              for (int x = 0; x < 4; ++x) v[r4 + x] = ex2_approx(e[x]);
              // The weights meet V in bf16; their sum is of the unrounded ones.
#pragma unroll
              for (int g = 0; g < C::kSets; ++g)
#pragma unroll
                for (int x = 0; x < 4; x += 2) {
                  const int r = g * R + r4 + x;
                  float2 w = make_float2(v[r4 + x], v[r4 + x + 1]);
                  if constexpr (kBare) w = __fmul2_rn(w, make_float2(vs[g], vs[g]));
                  const uint32_t both = pack_bf16x2(w.x, w.y);
                  sts16(p_at[r & 7] + r * 128, both);
                  sts16(p_at[(r + 1) & 7] + (r + 1) * 128, both >> 16);
                }
            }
          if (!again && th < D) {
            // V over K, whose product is done
#pragma unroll
            for (int x = 0; x < C::kAhead; ++x) tmem_st16(a_t + x * 16, ab);
#pragma unroll kBare ? 4 : 1
            for (int x = C::kAhead; x < 4; ++x) {
              v_codes(x, ab);
              tmem_st16(a_t + x * 16, ab);
            }
            tmem_wait_st();
          }
          fence_async_shared();
          tc_fence_before();
          // Weights of up to 2^8 are as exact as others; above, the maximum moves and
          // they are taken again.
          grow = sync_any(top > 8.f || !ok);
          if (!grow || again) break;
          again = true;
          if (sync_any(!ok)) break;
        }
        if (grow) break;                           // some wait gave up
        if (lane == 0) mbar_arrive(pv_ready);
#pragma unroll
        for (int r4 = 0; r4 < R; r4 += 4)
          if (r4 < rows) {
#pragma unroll
            for (int r = r4; r < r4 + 4; r += 2) {
              const float2 sum = __fadd2_rn(make_float2(l[r], l[r + 1]), make_float2(v[r], v[r + 1]));
              l[r] = sum.x;
              l[r + 1] = sum.y;
            }
          }
      }
      if (j < tiles) break;
      ok = warp_wait(pv_done, (it & 1u) ^ 1u, abort_flag);
      rows_of_threads(
          l, [](float z) { return z; }, [](float a, float b) { return a + b; }, [&](int r, float sum) { of_row[r] = sum; });
      if (sync_any(!ok)) break;
      tc_fence_after();
      const bool direct = p.pre_rt == 0 && s.whole;
      if (th < rows) {
        const float sum = of_row[th];
        // no score above kLowest: nothing is left, or NaN
        const float m = mr[th] > kLowest ? mr[th] : sum == 0.f ? -INFINITY : 0.f;
        if (!direct) {
          reinterpret_cast<float2*>(p.part_ml)[(s.b < 0 ? 0 : p.own_first) +
                                               s.slot * (s.b < 0 ? p.pre_slot_rows : p.own_slot_rows) + th] = make_float2(m, sum);
        } else if (p.lse) {
          const int rem = rem0 + th, i = p.div_G.quot(rem), g = rem - i * p.G;
          p.lse[((int64_t)s.b * p.Hq + s.hk * p.G + g) * p.T + i] = row_lse(seen_keys(p, s.kv, s.n, i) > 0, m, sum);
        }
      }
      {
        float o[R];
        tmem_ld_n<R>(o_t, o);
        tmem_wait_ld();
        if (th < D) {
          if (!direct) {
            float* dst = p.part_o + (int64_t)((s.b < 0 ? 0 : p.own_first) +
                                              s.slot * (s.b < 0 ? p.pre_slot_rows : p.own_slot_rows)) * D + th;
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (r < rows) dst[r * D] = o[r];
          } else {
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (r < rows) {
                const int rem = rem0 + r, i = p.div_G.quot(rem), g = rem - i * p.G;
                const float inv = inverse_sum(seen_keys(p, s.kv, s.n, i) > 0, of_row[r]);
                p.out[(((int64_t)s.b * p.T + i) * p.Hq + s.hk * p.G + g) * D + th] = __float2bfloat16(inv != 0.f ? o[r] * inv : 0.f);
              }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(seg_empty + 8 * qb);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, C::kColumns);
  }
  if (p.wide_ctas != 0 && cta == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Output row (b, i, h): joins the partial results of its prefix segment and of its
// own segment, one from each CTA.
template <int D, int kLanes, int kWarps>
__global__ void __launch_bounds__(kWarps > 1 ? 32 * kWarps : 128) quant_join_kernel(const __grid_constant__ QAttnParams p) {
  constexpr int kRows = kWarps > 1 ? 1 : 128 / kLanes;   // rows per block
  const int64_t R = (int64_t)blockIdx.x * kRows + (kWarps > 1 ? 0 : threadIdx.x / kLanes);
  const bool real = R < (int64_t)p.B * p.T * p.Hq;
  const int r0 = real ? (int)R : 0;
  const int bt = r0 / p.Hq, h = r0 - bt * p.Hq;
  const int b = bt / p.T, i = bt - b * p.T, hk = p.div_G.quot(h), g = h - hk * p.G;
  const int row = i * p.G + g, flat = b * p.TG + row;
  const int pre_seg = hk * p.pre_rt + flat / (p.wide_ctas > 0 ? kWideRows : p.R), own_seg = b * p.Hkv + hk;
  // Read before the wait, which is for the partial results.
  fence_waited();
  const int kv = own_keys(p, b), n = new_tokens(p, b);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");      // what follows waits in its turn
  // (of a segment without tiles these are any bytes, not looked at)
  const int2 pc = p.pre_rt > 0 ? p.seg_ctas[pre_seg] : make_int2(0, 0), oc = p.seg_ctas[p.pre_rt * p.Hkv + own_seg];
  Parts pre{0, 0, 0}, own{0, 0, 0};
  bool direct = false;
  // CTAs first .. last have a part each; a pair that no schedule makes (a wait gave up) none
  auto partial = [&](const int2& c, int seg, int slot_rows, int r) {
    if (c.x < 0 || c.y < c.x || c.y >= p.ctas) return Parts{0, 0, 0};
    return Parts{c.y - c.x + 1, (seg + c.x) * slot_rows + r, slot_rows};
  };
  const bool keyed = real && i < n && (p.prefix_len > 0 || seen_keys(p, kv, n, i) > 0);
  if (real && i < n) {
    if (p.wide_ctas > 0) {
      const bool two = p.B * p.TG - (flat - flat % kWideRows) <= kWideHalf;
      pre = segment_parts(pc.x, pc.y, p.wide_ctas, pre_seg, two, flat % kWideRows / kWideHalf, p.pre_slot_rows, flat % kWideHalf);
    } else if (p.pre_rt > 0) {
      pre = partial(pc, pre_seg, p.pre_slot_rows, flat % p.R);
    }
    if (own_tiles(p, kv, n) > 0) {
      own = partial(oc, own_seg, p.own_slot_rows, row);
      own.at += p.own_first;
      direct = p.pre_rt == 0 && own.n == 1;       // written by the first kernel
    }
  }
  join_row<D, kLanes, kWarps>(p.part_ml, p.part_o, pre, own, real && !direct, keyed, p.out + R * D,
                              p.lse ? p.lse + ((int64_t)b * p.Hq + h) * p.T + i : nullptr);
}

std::string s(int64_t v) { return std::to_string(v); }

// How a call is split, the rows of a segment, and where the partial results lie.
struct QAttnPlan {
  // kNarrow: this file's kernel alone; kWide: that of the bf16 pages alone; kBoth: that
  // one for the prefix, this one for the requests' own keys
  enum { kNarrow, kWide, kBoth } way;
  int R, TG, pre_rt, pre_slot_rows, own_slot_rows;
  size_t own_first, part_ml, part_o, bytes;
};

// Up to so many rows of a segment the keys are the first operand.  16 requests of
// 8,192 keys, heads of 128 (us here / with the rows as the first operand): 8 rows 51 /
// 104, 16 rows 65 / 104; with a form for 32 rows 96 / 104 for 24 and 102 / 102 for 32,
// and 41 / 34 where the keys were 300.
constexpr int kNarrowRows = 16;

// A prefix of few tiles stays with this kernel though its rows are many, up to one tile
// a CTA.  us alone / with the prefix in the other kernel: 64 requests of 8 heads of 4
// rows, 128 shared keys (0.8 tiles a CTA) 25.8 / 31.2, 300 (2.5) 32.5 / 29.8; 16
// requests, 500 keys (0.8) 16.5 / 23.6; 24 of 2 heads of 10 rows, 1,000 keys (0.4) 15.7 /
// 17.7, 4,000 (1.6) 20.0 / 20.8; 64 of 8 heads of 12 rows, 300 keys (1.9) 41.5 / 35.1.

QAttnPlan plan_quant(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t d, int64_t prefix_len, int sms) {
  QAttnPlan w{};
  const bool prefix = prefix_len > 0;
  w.TG = (int)(T * (Hq / Hkv));
  const int64_t most = prefix ? B * w.TG : w.TG;
  const PrefixPart wide = prefix ? prefix_part(B, T, Hq, Hkv, d, sms) : PrefixPart{};
  const int64_t rows = most <= kNarrowRows ? most : w.TG;
  w.R = rows <= 4 ? 4 : rows <= 8 ? 8 : 16;
  const bool few = w.TG <= kNarrowRows && wide.rt > 0 &&
                   Hkv * cdiv64(B * w.TG, w.R) * cdiv64(prefix_len, kTileKeys) <= kCtasPerSm * sms;
  w.way = most <= kNarrowRows || few ? QAttnPlan::kNarrow
          : w.TG <= kNarrowRows && wide.rt > 0 ? QAttnPlan::kBoth
                                               : QAttnPlan::kWide;
  if (w.way == QAttnPlan::kWide) {
    w.bytes = wide_quant_bytes(B, T, Hq, Hkv, d, prefix, sms);
    return w;
  }
  w.own_slot_rows = w.TG;              // at most R
  // a partial result for every number segment + CTA
  const size_t own = (size_t)(B * Hkv + kCtasPerSm * sms) * w.own_slot_rows;
  size_t pre = 0;
  if (w.way == QAttnPlan::kBoth) {
    w.pre_rt = wide.rt;
    w.pre_slot_rows = wide.slot_rows;
    pre = wide.rows;
  } else if (prefix) {
    w.pre_rt = (int)cdiv64(B * w.TG, w.R);
    w.pre_slot_rows = (int)(B * w.TG < w.R ? B * w.TG : w.R);
    pre = (size_t)(Hkv * w.pre_rt + kCtasPerSm * sms) * w.pre_slot_rows;
  }
  auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
  w.own_first = pre;
  w.part_ml = al((size_t)Hkv * (w.pre_rt + B) * 8);      // behind the segments' CTAs
  w.part_o = w.part_ml + al((pre + own) * 8);
  w.bytes = w.part_o + al((pre + own) * d * 4);
  return w;
}

template <int D, int R>
bsa_status launch_quant(const QAttnParams& p, cudaStream_t stream) {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  bsa_status st = cuda_check(cudaGetDevice(&dev), "cudaGetDevice");
  if (st != BSA_OK) return st;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      st = cuda_check(cudaFuncSetAttribute(quant_attention_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           Cfg<D, R>::kSmemBytes),
                      "cudaFuncSetAttribute(quant_attention_kernel)");
      if (st != BSA_OK) return st;
      if (dev < 64) done[dev] = true;
    }
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D, R>::kSmemBytes;
  if ((st = cuda_check(cudaLaunchKernelEx(&cfg, quant_attention_kernel<D, R>, p), "quant_attention_kernel launch")) != BSA_OK)
    return st;
  // Eight warps, one warp or eight lanes a row, as in the join of bsa_paged.cu.
  const int64_t rows = (int64_t)p.B * p.T * p.Hq;
  const int lanes = rows < (int64_t)num_sms() * 4 ? 256 : rows < (int64_t)num_sms() * 40 ? 32 : 8;
  cfg.blockDim = dim3(lanes == 256 ? 256 : 128);
  cfg.gridDim = dim3((unsigned)cdiv64(rows, cfg.blockDim.x / lanes));
  cfg.dynamicSmemBytes = 0;
  return cuda_check(lanes == 256  ? cudaLaunchKernelEx(&cfg, quant_join_kernel<D, 32, 8>, p)
                    : lanes == 32 ? cudaLaunchKernelEx(&cfg, quant_join_kernel<D, 32, 1>, p)
                                  : cudaLaunchKernelEx(&cfg, quant_join_kernel<D, 8, 1>, p),
                    "quant_join_kernel launch");
}

}  // namespace

unsigned int read_and_clear_quant_attn_error() { return take_error_word(); }

bsa_status launch_quant_wait_probe(unsigned long long limit_ns, cudaStream_t stream) {
  wait_probe_kernel<<<1, 32, 0, stream>>>(limit_ns);
  return cuda_check(cudaGetLastError(), "wait_probe_kernel launch (4-bit paged attention)");
}

}  // namespace bsa

using namespace bsa;

extern "C" {

size_t bsaq_forward_workspace_size(int B, int T, int Hq, int Hkv, int d, int has_prefix, int sms) {
  if (B <= 0 || B > kMaxPagedBatch || T <= 0 || Hq <= 0 || Hkv <= 0 || Hq > kMaxHeads || Hq % Hkv ||
      (d != 64 && d != 128) || sms < 0 || (int64_t)B * T * (Hq / Hkv) > INT32_MAX / 16)
    return 0;
  if (sms == 0) sms = num_sms();
  if (!has_prefix) return plan_quant(B, T, Hq, Hkv, d, 0, sms).bytes;
  // of a short prefix and of a long one
  return std::max(plan_quant(B, T, Hq, Hkv, d, 1, sms).bytes, plan_quant(B, T, Hq, Hkv, d, INT32_MAX / 2, sms).bytes);
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
  // rows, tiles and slot numbers are 32-bit on the device
  const int64_t flat_rows = qv.B * qv.S * G, page = a.k.blocks * kBlockSlots;
  const int64_t q_extent = (qv.B - 1) * qv.stride_b + (qv.S - 1) * qv.stride_s + qv.H * qv.stride_h + qv.D;
  const QAttnPlan plan = plan_quant(qv.B, qv.S, qv.H, a.k.heads, qv.D, prefix_len, sms);
  const int64_t most_tiles = most_tiles_of(qv, a.k.heads, page, max_pages, prefix_len);
  const size_t need = plan.bytes;
  if (flat_rows > INT32_MAX / 16 || most_tiles > INT32_MAX / 8 || flat_rows * a.k.heads > INT32_MAX ||
      need / (4 * (size_t)qv.D) > INT32_MAX)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": " + s(flat_rows) + " rows of up to " +
                                              s(max_pages * page + prefix_len) + " keys are too many for one call");
  if (q_extent >= (int64_t)1 << 35)
    return set_error(BSA_ERR_UNSUPPORTED, std::string(fn) + ": q reaches over " + s(q_extent) + " elements (2^35 at most)");
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
                                  4 * cdiv64(prefix_len, page))};
  for (const Bytes& w : writes)
    for (const Bytes& r : reads)
      if ((st = check_apart(fn, r, w)) != BSA_OK) return st;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(fn, writes[j], writes[i])) != BSA_OK) return st;
  if (plan.way == QAttnPlan::kWide)
    return launch_wide_quant(qv, a, new_lens, prefix_table, prefix_len, causal, softmax_scale, out, lse, workspace,
                             reinterpret_cast<cudaStream_t>(stream));
  QAttnParams p{};
  p.k = static_cast<const uint8_t*>(a.k.ptr); p.v = static_cast<const uint8_t*>(a.v.ptr);
  p.k_page = a.k.stride_page; p.k_head = a.k.stride_head; p.v_page = a.v.stride_page; p.v_head = a.v.stride_head;
  p.q = static_cast<const __nv_bfloat16*>(qv.ptr); p.q_sb = qv.stride_b; p.q_ss = qv.stride_s; p.q_sh = qv.stride_h;
  p.B = (int)qv.B; p.T = (int)qv.S; p.Hq = (int)qv.H; p.Hkv = (int)a.k.heads; p.G = (int)G;
  p.page_shift = 4;
  while ((1 << p.page_shift) < page) ++p.page_shift;
  p.num_pages = (int)a.k.pages; p.max_pages = max_pages; p.prefix_len = prefix_len; p.causal = causal ? 1 : 0;
  p.div_G = fast_div((uint32_t)G); p.div_TG = fast_div((uint32_t)plan.TG);
  p.R = plan.R; p.TG = plan.TG; p.pre_rt = plan.pre_rt;
  p.pre_tiles = plan.way == QAttnPlan::kBoth ? 0 : (int)cdiv64(prefix_len, kTileKeys);
  p.wide_ctas = plan.way == QAttnPlan::kBoth ? sms : 0;
  p.pre_slot_rows = plan.pre_slot_rows; p.own_slot_rows = plan.own_slot_rows;
  p.ctas = kCtasPerSm * sms;
  p.page_table = page_table; p.table_stride = table_stride; p.kv_lens = kv_lens; p.new_lens = new_lens;
  p.prefix_table = prefix_table;
  p.scale_log2 = (softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt((float)qv.D)) * 1.4426950408889634f;
  p.eights = kEights;
  p.out = static_cast<__nv_bfloat16*>(out); p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.seg_ctas = reinterpret_cast<int2*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + plan.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + plan.part_o);
  p.own_first = (int)plan.own_first;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (plan.way == QAttnPlan::kBoth &&
      (st = launch_prefix_quant(qv, a, new_lens, prefix_table, prefix_len, softmax_scale, p.seg_ctas, p.part_ml, p.part_o,
                                cs)) != BSA_OK)
    return st;
  if (plan.R == 4) return qv.D == 128 ? launch_quant<128, 4>(p, cs) : launch_quant<64, 4>(p, cs);
  if (plan.R == 8) return qv.D == 128 ? launch_quant<128, 8>(p, cs) : launch_quant<64, 8>(p, cs);
  return qv.D == 128 ? launch_quant<128, 16>(p, cs) : launch_quant<64, 16>(p, cs);
}

}  // extern "C"
