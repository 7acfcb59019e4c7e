// tree.cu - attention of drafted tokens over a paged raw K/V cache.
//
// Node i of sequence b (row r of the call) sees the committed rows s < L_b of its
// sequence (with a window: s > pos_r - W) and those drafted rows L_b + j whose
// bit j its mask holds; one softmax over both:
//   O = sum_s p_s v_s,  p_s = exp(scale q.k_s - lse),  lse = log sum_s exp(scale q.k_s).
// One token per sequence with mask 1 is ordinary decode over the cache.
//
// Work.  The rows of one (sequence, key head) are its nodes times the G = H/Hk
// query heads that share the key head, 128 to a tensor tile (TMEM lane = row).
// Up to 256 rows make one item, which walks the keys of its sequence in tiles of
// 128 from the first one that any row sees.  All items' key tiles, each as long as it
// takes, form one line, cut into equal shares, one per CTA (one CTA per SM,
// persistent): lengths may be as ragged as they like.  A share that covers an item
// only in part writes an fp32 partial (O, lse); tree_combine_kernel merges those.
// Lengths are read on the device, so the cut follows them in a captured graph.
//
// One CTA:
//   warps 0..3, 4..7  two softmax streams, one thread per row;
//   warp 8            walks the share and publishes its segments;
//   warps 8, 10       fetch K and V pages by TMA (one box per page and 64 channels);
//   warp 9            TMEM and MMA issue.
// An item of more than 128 rows gives each stream one row tile, and both use
// every K/V tile; a smaller item gives both streams the same rows and alternate
// key tiles.  Either way one stream's softmax runs while the tensor pipe works on
// the other's tile.  Per stream and key tile: S = Q K^T (tcgen05, fp32 in TMEM),
// online softmax with one thread a row, P as bf16 back
// over S's columns, O += P V with A = P from TMEM.  The tensor pipe runs one
// thread's products in the order of issue, so S of a stream's next tile may be
// issued right behind the PV that reads the P in the same columns, and a
// completed S means that the PV before it is complete too: the accumulator can be
// rescaled without a further wait.
//
// Masks: whole tiles below every row's window are never fetched; in the others a
// row's visible columns are four 32-bit words (committed range, shifted draft
// mask), built only for tiles that some row sees in part.  K outside is masked
// after the product (selected, never added, so NaN there does nothing); V rows
// that no row of the sequence sees are zeroed in shared memory before the
// product, since 0 * NaN would not be 0.
//
// Bound and measured (without the host): one token of 16 sequences of 64 k .. 131 k rows, 64
// heads of 128 on one key head (807 MB): HBM, 139 us, 5.8 TB/s (6.3 while streaming).  Trees of
// 8 .. 16 nodes over 21 k .. 33 k rows, the same heads: the softmax of 128 x 128 logits, 1024
// clocks of the SFU at least, beside 1024 clocks of products; 1.9 us for a pair of row tiles,
// 165 us and 0.96 PFLOP/s, 180 .. 197 us and 0.80 .. 0.88 under the power cap.  32 heads of 64 on 8 key heads, window 4096:
// the chain from S over the softmax to PV, 1.0 us a tile, and 3 .. 4 us to change segments; 64 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <type_traits>

#include "checks.cuh"
#include "sm100.cuh"

namespace csa {

using namespace sm100;

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn get_encode_fn();

namespace {

constexpr int kTile = 128;          // rows of a tensor tile, keys of a key tile
constexpr int kItemRows = 2 * kTile;
constexpr int kSoftmaxWarps = 8;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLoadWarp2 = 10;
constexpr int kThreads = 352;       // 11 warps, up to 168 registers a thread (d = 64 spills 8 bytes)
constexpr int kMaxNodes = 64;       // bits of a mask
constexpr int kMaxSeqs = 65536;     // every CTA adds up all sequences' tiles, within the bound of the other roles' waits
// Lengths on the line of all items' key tiles, in key tiles of a single row tile (1.0 us;
// a pair of row tiles takes 1.9 us): a tile of a single row tile, of a pair, and what
// starting an item costs beside them (the outputs before it written, query rows read,
// the pipeline filled).
constexpr int kSingleCost = 1, kPairCost = 2, kItemCost = 6;
// A CTA's share at least: an item's cost and three key tiles.  Fewer, longer shares save the
// merge of partial results where all fit one CTA; beyond that more CTAs win (verification step
// of 8 sequences of 1 k .. 8 k rows, 8 drafts each: 39.4 us with twelve key tiles, 36.4 with six,
// 35.2 with four, 34.5 with three, 35.3 with two; 15 sequences of 500 rows: 23.0, 20.7, 19.3,
// 18.3, 16.7).
constexpr int kMinShare = kItemCost + 3 * kSingleCost;
constexpr float kRescaleSlack = 8.0f;  // raise the running max only when it grows by > 2^8
constexpr float kLn2 = 0.69314718055994531f;

struct alignas(64) TreeMaps {
  CUtensorMap k, v;
};

struct TreeArgs {
  const __nv_bfloat16* q;
  const int32_t *table, *lens, *q_start;
  const uint64_t* mask;
  const int64_t* pos;
  int64_t R, n_pages;
  int B, H, Hk, G, max_pages, page_shift, W;
  float scale_log2;
  void* O;
  int o_f32;
  float* lse;
  int* status;
  // partial results of shares that cover an item in part: slot 2c the first
  // segment of CTA c, 2c+1 its last; [slots][part_rows][D] and [slots][part_rows]
  float *part_o, *part_lse;
  int part_rows;
  int4* split;  // [grid]: the item that CTA c starts and does not finish (see tree_combine_kernel)
};

// What one sequence asks for.
struct Seq {
  int r0, n;        // first row of the call, nodes
  int L, S;         // committed rows, all rows (max_pages * page < 2^31 - 128)
  int lo;           // first row that any node may see
  int tile0;        // first key tile
  int tiles;        // key tiles (one at least: an item without keys still writes its rows)
  int units;        // row tiles per key head: ceil(n * G / 128)
  __device__ int64_t pair() const { return kItemCost + (int64_t)kPairCost * tiles; }  // an item of two row tiles
  // length of one key head: its pairs, then perhaps an item of a single row tile
  __device__ int64_t head() const {
    return (units >> 1) * pair() + (units & 1) * (kItemCost + (int64_t)kSingleCost * tiles);
  }
  __device__ int64_t total(int Hk) const { return tiles > 0 ? head() * Hk : 0; }
};

// 2^x with the SFU (ex2.approx, ~2 ulp; -inf -> +0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Packed fp32 pairs (per component the scalar IEEE operation).
__device__ __forceinline__ unsigned long long pair_bits(float2 a) {
  unsigned long long x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  return x;
}
__device__ __forceinline__ float2 bits_pair(unsigned long long x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long z;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return bits_pair(z);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long z;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return bits_pair(z);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// The first committed row that a node at position pos sees (pos may be anything).
__device__ __forceinline__ int window_start(int64_t pos, int W, int L) {
  if (pos < W) return 0;  // pos - W + 1 is at most 0
  return pos - W >= L ? L : (int)(pos - W) + 1;
}

__device__ __forceinline__ Seq load_seq(const TreeArgs& a, int b, bool tell) {
  Seq q;
  q.r0 = a.q_start[b];
  const int r1 = a.q_start[b + 1];
  q.L = a.lens[b];
  q.n = 0;
  q.S = 0;
  q.lo = 0;
  // compared before they are subtracted: the numbers may be anything, their difference may wrap
  const bool rows = q.r0 >= 0 && r1 >= q.r0 && r1 <= a.R && r1 - q.r0 <= kMaxNodes;
  if (rows && q.L >= 0 && (int64_t)q.L + (r1 - q.r0) <= ((int64_t)a.max_pages << a.page_shift)) {
    q.n = r1 - q.r0;
  } else if (tell) {
    report(a.status, CSA_ERR_INDEX);
  }
  if (q.n == 0) {
    q.tiles = q.units = 0;
    q.tile0 = 0;
    return q;
  }
  q.S = q.L + q.n;
  if (a.W >= 0) {
    int64_t p = a.pos[q.r0];
#pragma unroll 8
    for (int i = 1; i < q.n; ++i) {
      const int64_t x = a.pos[q.r0 + i];
      p = x < p ? x : p;
    }
    q.lo = window_start(p, a.W, q.L);
  }
  q.tile0 = q.lo / kTile;
  q.tiles = (q.S - q.tile0 * kTile + kTile - 1) / kTile;
  if (q.tiles < 1) q.tiles = 1;
  q.units = (int)ceil_div((int64_t)q.n * a.G, kTile);
  return q;
}

// a / b for a >= 0, b > 0; a 64-bit division takes several times a 32-bit one.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// One segment of a share: part of one item.
struct Segment {
  int valid;
  int b, r0, n;       // the sequence, its first row and nodes
  int row0, rows;     // the item's first (node, head) row and its rows
  int hk;
  int t0, t1;         // its key tiles, counted from tile 0 of the sequence
  int L, lo;
  int slot;           // partial result slot, or -1: the whole item, final
};

template <int D>
struct TreeSmem {
  static constexpr int kHalf = kTile * 128;               // one 64-channel half of a tile
  static constexpr int kTileBytes = (D / 64) * kHalf;     // 128 rows x D bf16
  static constexpr int kStages = D == 128 ? 5 : 10;       // K and V tiles in flight, 160 KB
  static constexpr size_t off_q = 0;                      // 2 row tiles (the second: statistics of merging streams)
  static constexpr size_t off_kv = 2 * kTileBytes;
  static constexpr size_t off_bar = off_kv + (size_t)kStages * kTileBytes;
  static constexpr size_t off_seg = off_bar + 48 * 8;
  static constexpr size_t off_misc = off_seg + 2 * 128;
  static constexpr size_t bytes = off_misc + 64 + 1024;
};
static_assert(sizeof(Segment) <= 128, "segment slot");

__device__ __forceinline__ void st_shared4(uint32_t addr, const float* v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}
__device__ __forceinline__ float4 ld_shared4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// A value that is the same in every lane, said so that the compiler may keep it (and
// what follows from it, operand descriptors above all) in uniform registers.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Shared-memory descriptor from the halves that make_sdesc builds: the high one is a
// constant of the layout, places are added to the low one.
__device__ __forceinline__ uint64_t sdesc(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}

// Bits [lo, hi) of a 32-bit word (lo and hi anything).
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  if (lo < 0) lo = 0;
  if (hi > 32) hi = 32;
  if (lo >= hi) return 0u;
  return (0xFFFFFFFFu >> (32 - (hi - lo))) << lo;
}

// Visible columns off .. off+31 of a row: committed rows [lo, L), drafted rows by mask.
__device__ __forceinline__ uint32_t visible(int off, int lo, int L, uint64_t mask) {
  uint32_t w = bit_range(lo - off, L - off);
  const int sh = off - L;
  if (sh >= 0) {
    if (sh < 64) w |= (uint32_t)(mask >> sh);
  } else if (sh > -32) {
    w |= (uint32_t)(mask << -sh);
  }
  return w;
}

// The drafted rows of a sequence that some node sees: each lane loads two nodes' masks, their OR
// over the warp is formed where it is needed.
__device__ __forceinline__ uint64_t lane_masks(const TreeArgs& a, const Segment& s, int lane) {
  return (lane < s.n ? a.mask[s.r0 + lane] : 0) | (lane + 32 < s.n ? a.mask[s.r0 + 32 + lane] : 0);
}
__device__ __forceinline__ uint64_t seen_drafts(uint64_t lane_masks, int n) {
  return ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(lane_masks >> 32)) << 32 |
          __reduce_or_sync(0xffffffffu, (uint32_t)lane_masks)) &
         (n < 64 ? (1ull << n) - 1 : ~0ull);
}
// Whether some node sees one of the rows key .. key + rows - 1 (rows at most 128).
__device__ __forceinline__ bool box_seen(int key, int rows, int lo, int L, uint64_t drafts) {
  if ((key > lo ? key : lo) < (key + rows < L ? key + rows : L)) return true;
  const int from = key > L ? key - L : 0, end = key + rows - L;
  return end > from && from < kMaxNodes &&
         (drafts >> from & (end - from < 64 ? (1ull << (end - from)) - 1 : ~0ull)) != 0;
}

// The rest of a bounded wait, out of line: the waits' code stays small.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* aborted, int* status) {
  const long long start = clock64();
  while (!*aborted) {
    if (mbar_try_wait(bar, parity)) return true;
    if (clock64() - start > CSA_WAIT_CYCLES) {
      report(status, CSA_ERR_DEVICE_TIMEOUT);
      *aborted = 1;
    }
  }
  return false;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ TreeMaps maps) {
  using L = TreeSmem<D>;
  constexpr int kStages = L::kStages;
  constexpr int HALVES = D / 64;
  constexpr uint32_t kHalfBytes = L::kHalf;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem + L::off_q;
  uint8_t* s_kv = smem + L::off_kv;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::off_bar);
  uint64_t* kv_full = bar;                  // [kStages] tile landed
  uint64_t* kv_empty = bar + kStages;       // [kStages] its products complete
  uint64_t* q_full = bar + 2 * kStages;        // [2] row tile in shared memory
  uint64_t* s_full = bar + 2 * kStages + 2;    // [2] S of a stream's tile complete
  uint64_t* p_full = bar + 2 * kStages + 4;    // [2][2] P of a stream's tile written: keys 0..63, 64..127
  uint64_t* o_full = bar + 2 * kStages + 8;    // [2] a stream's last PV of a segment complete
  uint64_t* o_free = bar + 2 * kStages + 10;   // the segment's outputs read out of TMEM
  uint64_t* seg_full = bar + 2 * kStages + 11;  // [2] a segment's description is in its slot
  uint64_t* seg_free = bar + 2 * kStages + 13;  // [2] every role is done with the slot
  uint64_t* mma_fin = bar + 2 * kStages + 15;  // every product complete
  uint64_t* ex_full = bar + 2 * kStages + 16;  // statistics of merging streams: written, then read
  uint8_t* s_seg = smem + L::off_seg;
  int* misc = reinterpret_cast<int*>(smem + L::off_misc);  // [0] tmem
  volatile int* s_abort = misc + 1;  // set by the first wait that timed out; every role then stops

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- setup: barriers, TMEM
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&seg_full[i], 1);
      mbar_init(&seg_free[i], kSoftmaxWarps + 2);
    }
    mbar_init(mma_fin, 1);
    mbar_init(o_free, kSoftmaxWarps);
    mbar_init(ex_full, kSoftmaxWarps);
    *s_abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(reinterpret_cast<uint32_t*>(&misc[0]), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = (uint32_t)misc[0];
  // TMEM columns: the streams' S (and P over it), then their outputs
  constexpr uint32_t kTmemS = 0, kTmemO = 256;

  // Bounded wait that also stops once any role of this CTA has given up.
  auto wait = [&](uint64_t* b_, uint32_t ph) -> bool {
    if (mbar_try_wait(b_, ph)) return true;
    return wait_on(b_, ph, s_abort, a.status);
  };
  // the next segment's description (in place until the role releases it), or null
  auto next_segment = [&](int n) -> const Segment* {
    if (!wait(&seg_full[n & 1], (uint32_t)((n >> 1) & 1))) return nullptr;
    const Segment* s = reinterpret_cast<const Segment*>(s_seg + (n & 1) * 128);
    return s->valid ? s : nullptr;
  };
  auto release_segment = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&seg_free[n & 1]);
  };

  // K and V tiles of a segment, by two warps (a tile's fetch takes a warp about 0.5 us: page
  // numbers, and some 80 cycles a box): each takes every other place of the ring.  Order of
  // the places, the order in which the MMA warp uses the tiles: K0 V0 K1 V1 .. when both
  // streams work on every tile, K0 K1 V0 K2 V1 .. when they alternate.
  const int loader = warp == kLoadWarp ? 0 : 1;
  int loads = 0;    // ring position of the segment's first tile
  int issued = -1;  // this warp's last
  auto load_tiles = [&](const Segment& s, int n) -> bool {
    const bool dual = s.rows > kTile;
    const int nt = s.t1 - s.t0, S = s.L + s.n;
    const int box_rows = a.page_shift < 7 ? 1 << a.page_shift : kTile;
    const int boxes = kTile / box_rows * HALVES;  // per tile, at most 16
    const int my_row = lane / HALVES * box_rows, my_half = lane % HALVES;
    uint8_t* const dst = s_kv + my_half * kHalfBytes + my_row * 128;
    const int lo = s.lo, hk_row = s.hk << a.page_shift, page_mask = (1 << a.page_shift) - 1;
    // page numbers are read ahead: lane l holds entries from + l and from + 32 + l of the
    // sequence's table (a tile's pages lie within one run of 32: both start at multiples
    // of 128 keys)
    const int32_t* table = a.table + (int64_t)s.b * a.max_pages;
    const int last_page = (S - 1) >> a.page_shift;  // (a sequence with a node has S >= 1)
    auto entry = [&](int p) { return p <= last_page ? table[p] : -1; };
    int from = (s.t0 * kTile) >> a.page_shift;
    int now = entry(from + lane), next = entry(from + 32 + lane);
    const uint64_t masks = lane_masks(a, s, lane);
    bool hold = n == 0;
#pragma unroll 1
    for (int i = loader; i < 2 * nt; i += 2) {
      int t, kind;
      if (dual) {
        t = i >> 1, kind = loader;
      } else if (i == 0 || i == 2 * nt - 1) {
        t = i == 0 ? 0 : nt - 1, kind = i == 0 ? 0 : 1;
      } else {
        kind = loader ? 0 : 1;
        t = kind ? i / 2 - 1 : (i + 1) / 2;
      }
      // at the start the query rows go first: behind a ring full of K and V they would wait
      // for all of it
      if (hold && i >= (dual || nt == 1 ? 1 : 2)) {
        if (!wait(&q_full[0], 0) || (dual && !wait(&q_full[1], 0))) return false;
        hold = false;
      }
      const int key0 = (s.t0 + t) * kTile, key = key0 + my_row;
      if (key0 >> a.page_shift >= from + 32) {
        from += 32;
        now = next;
        next = entry(from + 32 + lane);
      }
      int page = __shfl_sync(0xffffffffu, now, ((key >> a.page_shift) - from) & 31);
      // boxes without a row that some node sees are left out, their page numbers unused
      bool need = lane < boxes && key + box_rows > lo;
      if (key0 + kTile > s.L) need = box_seen(key, box_rows, lo, s.L, seen_drafts(masks, s.n)) && lane < boxes;
      if (need && (page < 0 || page >= a.n_pages)) {
        report(a.status, CSA_ERR_INDEX);
        page = a.n_pages > 0 ? (int)a.n_pages : 1;  // outside the map: zeros
      }
      const int count = __popc(__ballot_sync(0xffffffffu, need));
      const int at = loads + i, sg = at % kStages;
      if (at >= kStages && !wait(&kv_empty[sg], (uint32_t)((at / kStages - 1) & 1))) return false;
      issued = at;
      if (lane == 0) mbar_arrive_expect_tx(&kv_full[sg], (uint32_t)(count * box_rows * 128));
      __syncwarp();
      if (need)
        tma_load_3d(dst + (size_t)sg * L::kTileBytes, kind ? &maps.v : &maps.k, &kv_full[sg], my_half * 64,
                    hk_row + (key & page_mask), page);
    }
    loads += 2 * nt;
    return true;
  };
  // after an abort, wait (bounded) for this warp's loads still landing in shared memory
  auto drain = [&]() {
    if (*s_abort && lane == 0)
      for (int at = issued; at >= 0 && at > issued - kStages; at -= 2)
        mbar_wait(&kv_full[at % kStages], (uint32_t)((at / kStages) & 1));
  };

  if (warp == kLoadWarp) {
    // =========================== the share: its segments and their K / V tiles
    griddep_launch_dependents();
    // what every sequence asks for, 32 of them at a time (lane: sequence block + lane); the
    // sum over all first, then the sequence that holds the share's first position
    const bool skip = *reinterpret_cast<volatile int*>(a.status) == CSA_ERR_DEVICE_TIMEOUT;
    int block = 0;
    Seq mine = lane < a.B ? load_seq(a, lane, blockIdx.x == 0) : Seq{};
    int64_t total = mine.total(a.Hk);
#pragma unroll 1
    for (int b = 32 + lane; b < a.B; b += 32) total += load_seq(a, b, blockIdx.x == 0).total(a.Hk);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    int64_t ctas = total < (int64_t)gridDim.x * kMinShare ? (int)total / kMinShare : gridDim.x;
    if (ctas < 1) ctas = 1;
    // shares of `len` positions, the first `longer` of them one more
    const int64_t c = blockIdx.x, len = quotient(total, ctas), longer = total - len * ctas;
    auto share_start = [&](int64_t i) { return i * len + (i < longer ? i : longer); };
    int64_t first = c < ctas ? share_start(c) : 0, last = c < ctas ? share_start(c + 1) : 0;
    if (skip) first = last = 0;
    int4 split = make_int4(0, 0, 0, 0);
    int b = 0;
    int64_t at = 0;  // positions before sequence b
    if (first < last) {
      for (;;) {
        int64_t up = mine.total(a.Hk);  // inclusive prefix
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, up, o);
          if (lane >= o) up += y;
        }
        const uint32_t over = __ballot_sync(0xffffffffu, at + up > first);
        if (over) {
          const int w = __ffs(over) - 1;
          b = block + w;
          at += __shfl_sync(0xffffffffu, up - mine.total(a.Hk), w);
          break;
        }
        at += __shfl_sync(0xffffffffu, up, 31);
        block += 32;
        if (block >= a.B) break;
        mine = block + lane < a.B ? load_seq(a, block + lane, false) : Seq{};
      }
    }
    // sequence b (of the current block, or the first of the next)
    auto sequence = [&](int b_) -> Seq {
      if (b_ >= block + 32) {
        block += 32;
        mine = block + lane < a.B ? load_seq(a, block + lane, false) : Seq{};
      }
      const int w = b_ - block;
      Seq q;
      q.r0 = __shfl_sync(0xffffffffu, mine.r0, w);
      q.n = __shfl_sync(0xffffffffu, mine.n, w);
      q.L = __shfl_sync(0xffffffffu, mine.L, w);
      q.S = __shfl_sync(0xffffffffu, mine.S, w);
      q.lo = __shfl_sync(0xffffffffu, mine.lo, w);
      q.tile0 = __shfl_sync(0xffffffffu, mine.tile0, w);
      q.tiles = __shfl_sync(0xffffffffu, mine.tiles, w);
      q.units = __shfl_sync(0xffffffffu, mine.units, w);
      return q;
    };
    int n = 0;  // segments published
#pragma unroll 1
    for (int64_t g = first; g < last;) {
      Seq q = sequence(b);
      while (g >= at + q.total(a.Hk) && b + 1 < a.B) {
        at += q.total(a.Hk);
        q = sequence(++b);
      }
      if (q.tiles == 0) break;
      // the item that holds position g
      const int64_t head = q.head(), pair = q.pair();
      Segment s;
      s.valid = 1;
      s.b = b;
      s.r0 = q.r0;
      s.n = q.n;
      s.hk = (int)quotient(g - at, head);
      const int set = (int)quotient(g - at - s.hk * head, pair);
      s.row0 = set * kItemRows;
      const int left = q.n * a.G - s.row0;
      s.rows = left < kItemRows ? left : kItemRows;
      const int wide = s.rows > kTile ? kPairCost : kSingleCost;
      const int64_t i0 = at + s.hk * head + set * pair, i1 = i0 + kItemCost + (int64_t)wide * q.tiles;
      const int64_t end = i1 < last ? i1 : last;
      // a key tile goes to the share that holds its first position; the item's own cost comes first
      auto tile_from = [&](int64_t pos) {
        const int64_t d = pos - i0 - kItemCost;
        return d <= 0 ? 0 : ((int)d + wide - 1) / wide;
      };
      const int t0 = tile_from(g), t1 = tile_from(end);
      g = end;
      if (t0 == t1) continue;
      s.t0 = q.tile0 + t0;
      s.t1 = q.tile0 + t1;
      s.L = q.L;
      s.lo = q.lo;
      s.slot = t0 == 0 && t1 == q.tiles ? -1 : (int)(2 * c) + (n == 0 ? 0 : 1);
      if (t0 == 0 && t1 < q.tiles) {  // the item goes on in the next CTAs: tell the combine
        const int64_t tail = i0 + kItemCost + (int64_t)wide * (q.tiles - 1);  // its last tile
        const int64_t cl = tail < (len + 1) * longer ? quotient(tail, len + 1) : longer + quotient(tail - (len + 1) * longer, len);
        split = make_int4(s.rows, s.slot, (int)(cl - c + 1), 0);
        // first output row: (r0 * H + hk * G) and the item's rows from row0
        if (lane == 0) {
          a.split[2 * c + 1] = make_int4(s.r0, s.hk, s.row0, 0);
        }
      }
      // publish
      if (n >= 2 && !wait(&seg_free[n & 1], (uint32_t)((n / 2 - 1) & 1))) break;
      if (lane == 0) {
        *reinterpret_cast<Segment*>(s_seg + (n & 1) * 128) = s;
        mbar_arrive(&seg_full[n & 1]);
      }
      // the rows that the softmax warps will read when they get to this segment (n > 0: while
      // the one before runs), into L2 now: behind the ring's loads they take up to 13 us
      if (n > 0) {
        for (int i = lane; i < s.rows; i += 32) {
          const int row = s.row0 + i;
          const int64_t orow = (int64_t)(s.r0 + row / a.G) * a.H + s.hk * a.G + row % a.G;
#pragma unroll
          for (int h = 0; h < HALVES; ++h) prefetch_l2(a.q + orow * D + 64 * h);
        }
      }
      if (!load_tiles(s, n)) break;
      ++n;
    }
    if (lane == 0) a.split[2 * c] = split;
    // no more segments
    if ((n < 2 || wait(&seg_free[n & 1], (uint32_t)((n / 2 - 1) & 1))) && lane == 0) {
      reinterpret_cast<Segment*>(s_seg + (n & 1) * 128)->valid = 0;
      mbar_arrive(&seg_full[n & 1]);
    }
    drain();
  } else if (warp == kMmaWarp) {
    // =========================== MMA issue
    // The tensor pipe runs dry whenever this warp's scalar work between two products is
    // longer than the products that are queued, so the loop is kept short: streams and
    // barriers are compile-time, ring stages counted, operand descriptors in uniform
    // registers, and the issue predicated instead of branched.
    const uint32_t skv = smem_u32(s_kv);
    constexpr uint32_t kTile16 = L::kTileBytes / 16;
    // descriptors of the first row tile, of a K and of a V tile in stage 0; other places are
    // added to the address field (16-byte units)
    const uint64_t q_desc = make_sdesc(smem_u32(s_q), 16, 1024, kSwizzle128);
    const uint64_t k_desc = make_sdesc(skv, 16, 1024, kSwizzle128);
    const uint64_t v_desc = make_sdesc(skv, kHalfBytes, 1024, kSwizzle128);
    const uint32_t q_lo = (uint32_t)q_desc, qk_hi = (uint32_t)(k_desc >> 32);
    const uint32_t k_lo = (uint32_t)k_desc, v_lo = (uint32_t)v_desc, v_hi = (uint32_t)(v_desc >> 32);
    const uint32_t tmem = (uint32_t)uniform((int)tbase);
    const uint32_t leader = elect_one();
    bool live = true;
    int ring = 0;              // stage of the next K / V tile
    uint32_t ring_phase = 0;   // and the parity of its barrier
    uint32_t q1_phase = 0;     // parity of the second row tile's barrier
    uint32_t p_phase[2] = {0, 0};
    // the next tile of the ring, once it has landed: its stage, or -1
    auto next_tile = [&]() -> int {
      if (!wait(&kv_full[ring], ring_phase)) return -1;
      const int st = ring;
      if (++ring == kStages) ring = 0, ring_phase ^= 1;
      return st;
    };
#pragma unroll 1
    for (int n = 0; live; ++n) {
      const Segment* sp = next_segment(n);
      if (sp == nullptr) break;
      const Segment& s = *sp;
      const bool dual = uniform(s.rows) > kTile;
      const int t0 = uniform(s.t0), nt = uniform(s.t1) - t0;
      const int jobs = dual ? 2 * nt : nt;  // job x: stream x & 1, key tile dual ? x / 2 : x
      // tiles [whole0, whole1) of the segment have no hidden row
      const int whole0 = uniform((s.lo + kTile - 1) / kTile) - t0, whole1 = uniform(s.L / kTile) - t0;
      // drafted rows that some node sees (used, and waited for, at the first tile with hidden rows)
      const uint64_t masks = lane_masks(a, s, lane);
      if (!wait(&q_full[0], (uint32_t)(n & 1)) || (dual && !wait(&q_full[1], q1_phase))) break;
      if (dual) q1_phase ^= 1;
      int ks = 0, vs = 0;      // stages of the K tile of the S to issue and of the V tile of the PV
      uint32_t steps = 0xFFu;  // steps of 16 keys of that V tile that some row sees
      // S = Q K^T; in a dual item the second stream's frees the K tile
      auto issue_s = [&](auto stream) -> bool {
        constexpr int st = decltype(stream)::value;
        if (!(dual && st) && (ks = next_tile()) < 0) return false;
        __syncwarp();
        tc_fence_after();
        const uint32_t qd = q_lo + (dual && st ? kTile16 : 0u), kd = k_lo + (uint32_t)ks * kTile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) / 16;
          mma_bf16_ss_if(leader, tmem + kTmemS + st * 128, sdesc(qd + off, qk_hi), sdesc(kd + off, qk_hi),
                         idesc_bf16(128, kTile, 0, 0), kk > 0);
        }
        mma_commit_if(leader, &s_full[st]);
        if (!dual || st) mma_commit_if(leader, &kv_empty[ks]);
        return true;
      };
      // job x: O += P V, the first 64 keys as soon as their P is written; then S of the stream's
      // next tile over the same columns
      auto job = [&](auto stream, int x) -> bool {
        constexpr int st = decltype(stream)::value;
        if (!(dual && st)) {
          if ((vs = next_tile()) < 0) return false;
          const int t = dual ? x >> 1 : x;
          steps = 0xFFu;
          if (t < whole0 || t >= whole1) {
            // Rows that no node sees hold anything (or were not fetched).  Sixteen keys are one
            // step of the product: steps without a visible row are left out, the hidden rows of
            // the others zeroed.
            const uint32_t seen =
                visible((t0 + t) * kTile + 16 * (lane & 7), s.lo, s.L, seen_drafts(masks, s.n)) & 0xFFFFu;
            steps = __ballot_sync(0xffffffffu, seen != 0) & 0xFFu;
            if (steps == 0) steps = 1;  // (a segment without any visible row still writes its output)
            uint32_t mend = __ballot_sync(0xffffffffu, seen != 0xFFFFu) & steps;
            while (mend != 0) {
              const int k = __ffs(mend) - 1;
              mend &= mend - 1;
              if (!(__shfl_sync(0xffffffffu, seen, k) >> (lane >> 1) & 1)) {
                const uint32_t row = skv + (uint32_t)vs * L::kTileBytes + (uint32_t)(16 * k + (lane >> 1)) * 128 +
                                     (uint32_t)(lane & 1) * 64;
#pragma unroll
                for (int i = 0; i < 4 * HALVES; ++i)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(row + (i >> 2) * kHalfBytes +
                                                                                (i & 3) * 16),
                               "r"(0)
                               : "memory");
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        const uint32_t vd = v_lo + (uint32_t)vs * kTile16;
        constexpr uint32_t kS = kTmemS + st * 128, kO = kTmemO + st * D;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!wait(&p_full[2 * st + h], p_phase[st])) return false;
          __syncwarp();
          tc_fence_after();
          if (steps == 0xFFu) {
#pragma unroll
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              mma_bf16_ts_if(leader, tmem + kO, tmem + kS + 8 * k, sdesc(vd + k * 128, v_hi),
                             idesc_bf16(128, D, 0, 1), k > 0 ? 1u : x >= 2);
          } else {
#pragma unroll 1
            for (int k = 4 * h; k < 4 * h + 4; ++k)
              if (steps >> k & 1)
                mma_bf16_ts_if(leader, tmem + kO, tmem + kS + 8 * k, sdesc(vd + k * 128, v_hi),
                               idesc_bf16(128, D, 0, 1), (x >= 2 || (steps & ((1u << k) - 1))) ? 1u : 0u);
          }
        }
        p_phase[st] ^= 1;
        if (!dual || st) mma_commit_if(leader, &kv_empty[vs]);
        if (x + 2 < jobs) return issue_s(stream);
        mma_commit_if(leader, &o_full[st]);
        return true;
      };
      using S0 = std::integral_constant<int, 0>;
      using S1 = std::integral_constant<int, 1>;
      live = issue_s(S0{}) && (jobs < 2 || issue_s(S1{}));
      // the outputs of the segment before must be out of TMEM before the first PV
      if (live && n > 0) live = wait(o_free, (uint32_t)((n - 1) & 1));
#pragma unroll 1
      for (int x = 0; x < jobs && live; x += 2) live = job(S0{}, x) && (x + 1 >= jobs || job(S1{}, x + 1));
      // a single tile: the second stream had nothing, its barrier keeps step
      if (live && jobs == 1) mma_commit_if(leader, &o_full[1]);
      release_segment(n);
    }
    // every MMA this warp issued has completed before TMEM is freed
    __syncwarp();
    mma_commit_if(leader, mma_fin);
    mbar_wait(mma_fin, 0);
  } else if (warp == kLoadWarp2) {
    // =========================== the other half of the K / V tiles
#pragma unroll 1
    for (int n = 0;; ++n) {
      const Segment* sp = next_segment(n);
      if (sp == nullptr || !load_tiles(*sp, n)) break;
      release_segment(n);
    }
    drain();
  } else {
    // =========================== softmax streams (warps 0..3, 4..7): one row per thread
    const int st = warp >> 2;
    const int trow = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t lane_base = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t scol = lane_base + kTmemS + st * 128;
    const float c = a.scale_log2;  // > 0: max of raw logits * c = max of scaled logits
    int jobs_seen = 0;             // tiles of this stream so far: the phase of its S barrier
#pragma unroll 1
    for (int n = 0;; ++n) {
      const Segment* sp = next_segment(n);
      if (sp == nullptr) break;
      const Segment& s = *sp;
      const bool dual = s.rows > kTile;
      const int jobs = dual ? 2 * (s.t1 - s.t0) : s.t1 - s.t0;
      const int row = trow + (dual && st ? kTile : 0);  // row of the item
      const bool mine = row < s.rows;
      // its (node, head); the tensors' rows are counted from the sequence's first node and the
      // key head's first query head, where they fit 32 bits.  A row beyond the item's stands
      // in for the first: it is computed and never written
      const int nh = s.row0 + (mine ? row : 0), node = nh / a.G;
      const int rel = node * a.H + nh - node * a.G;
      const int64_t row00 = (int64_t)s.r0 * a.H + s.hk * a.G;
      uint64_t mask = 0;
      int lo = 0;
      if (mine) {
        mask = a.mask[s.r0 + node] & (s.n < 64 ? (1ull << s.n) - 1 : ~0ull);
        if (a.W >= 0) lo = window_start(a.pos[s.r0 + node], a.W, s.L);
      }
      // this warp's query rows into the stream's row tile (128-byte swizzle).  The products
      // that read the rows before are complete: this warp has seen the last PV (o_full) of
      // every stream that used the tile
      if (st == 0 || dual) {
        // D/8 lanes copy a row, 16 bytes each
        constexpr int LPR = D / 8, RPW = 32 / LPR;
        const int ch = lane % LPR;
        const uint32_t dst = smem_u32(s_q) + (uint32_t)(st * L::kTileBytes + (ch >> 3) * kHalfBytes);
        const __nv_bfloat16* from = a.q + row00 * D + 8 * ch;
        uint4 v[LPR];
#pragma unroll
        for (int i = 0; i < LPR; ++i)
          v[i] = *reinterpret_cast<const uint4*>(
              from + (int64_t)__shfl_sync(0xffffffffu, rel, i * RPW + lane / LPR) * D);
#pragma unroll
        for (int i = 0; i < LPR; ++i) {
          const int r = (warp & 3) * 32 + i * RPW + lane / LPR;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + r * 128 +
                                                                        (uint32_t)(((ch & 7) ^ (r & 7)) << 4)),
                       "r"(v[i].x), "r"(v[i].y), "r"(v[i].z), "r"(v[i].w)
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[st]);
      }
      const bool warp_mine = __any_sync(0xffffffffu, mine);
      float m_run = -INFINITY;
      float2 l2 = make_float2(0.f, 0.f);
      bool live = true;
#pragma unroll 1
      for (int x = st; x < jobs; x += 2) {
        const int base = (s.t0 + (dual ? x >> 1 : x)) * kTile;
        if (!wait(&s_full[st], (uint32_t)(jobs_seen++ & 1))) {
          live = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        if (warp_mine) {
          // Columns out of sight become -inf where they stand, 32 at a time, before the row is
          // read (few tiles have any: their code stays small and out of the unrolled part)
          if (!__all_sync(0xffffffffu, lo <= base && base + kTile <= s.L)) {
#pragma unroll 1
            for (int w = 0; w < 4; ++w) {
              const uint32_t bits = visible(base + 32 * w, lo, s.L, mask);
              uint32_t t[32];
              tmem_ld32p(scol + 32 * w, t);
              tmem_wait_ld_regs32(t);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(bits >> e & 1)) t[e] = 0xFF800000u;
              tmem_st32p(scol + 32 * w, t);
            }
            tmem_wait_st();
          }
          // raw logits of the row, read in two halves and, but for the first, again for the weights:
          // the loop's code stays small (the warps of a quarter of the SM are in different places
          // of it and wait for instructions otherwise), and half a row fits the 168 registers of
          // a thread.  The whole row in registers took 201 us for drafted trees (187 now)
          uint32_t v[64];
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int h = 64; h >= 0; h -= 64) {
            tmem_ld32p(scol + h, v);
            tmem_ld32p(scol + h + 32, v + 32);
            tmem_wait_ld_regs32(v);
            tmem_tie32(v + 32);
#pragma unroll
            for (int e = 0; e < 64; e += 2)
              mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
          }
          const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const bool raise = mt > m_run + kRescaleSlack || (m_run == -INFINITY && mt > -INFINITY);
          const float m_new = raise ? mt : m_run;
          const float m_use = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet: every weight is 0
          if (__any_sync(0xffffffffu, raise && x >= 2)) {
            // S of this tile is complete, so the PV of the tile before is, too
            const float alpha = raise ? fast_exp2(m_run - m_new) : 1.f;
            l2.x *= alpha, l2.y *= alpha;
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
              uint32_t o[32];
              tmem_ld32p(lane_base + kTmemO + st * D + j, o);
              tmem_wait_ld_regs32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32p(lane_base + kTmemO + st * D + j, o);
            }
          }
          m_run = m_new;
          // p = 2^(s c - m); the sums take the unrounded weights, the product with V
          // their bf16 rounding (the tensor pipe's operand type).  P of the first half covers
          // columns 0 .. 31, so the second half's logits still stand
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float2 z = fma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), both(c),
                              both(-m_use));
              z.x = fast_exp2(z.x), z.y = fast_exp2(z.y);
              l2 = add2(l2, z);
              pk[e / 2] = pack_bf16x2(z.x, z.y);
            }
            tmem_st32p(scol + 32 * h, pk);
            if (h == 0) {
              tmem_ld32p(scol + 64, v);
              tmem_ld32p(scol + 96, v + 32);
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&p_full[2 * st]);
              tmem_wait_ld_regs32(v);
              tmem_tie32(v + 32);
            }
          }
          tmem_wait_st();
        } else if (lane == 0) {
          mbar_arrive(&p_full[2 * st]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * st + 1]);
      }
      // ---- outputs
      if (!live || !wait(&o_full[st], (uint32_t)(n & 1))) break;
      float l = l2.x + l2.y;
      float f[2] = {st == 0 ? 1.f : 0.f, st == 0 ? 0.f : 1.f};  // weights of the two accumulators
      if (!dual) {
        // the streams hold the same rows: exchange (max, sum), then each writes half the channels
        if (!wait(&o_full[st ^ 1], (uint32_t)(n & 1))) break;
        float2* ex = reinterpret_cast<float2*>(s_q + L::kTileBytes);
        ex[st * kTile + trow] = make_float2(m_run, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(ex_full);
        if (!wait(ex_full, 0)) break;
        const float2 e0 = ex[trow], e1 = ex[kTile + trow];
        __syncwarp();
        if (lane == 0) mbar_arrive(ex_full);
        if (!wait(ex_full, 1)) break;
        m_run = fmaxf(e0.x, e1.x);
        f[0] = e0.y != 0.f ? fast_exp2(e0.x - m_run) : 0.f;
        f[1] = e1.y != 0.f ? fast_exp2(e1.x - m_run) : 0.f;
        l = e0.y * f[0] + e1.y * f[1];
      }
      __syncwarp();
      tc_fence_after();
      // l = 0: the row sees nothing; a query that is not finite makes it NaN, which goes on
      const float inv = l != 0.f ? 1.f / l : 0.f;
      f[0] *= inv, f[1] *= inv;
      const float lse2 = l != 0.f ? m_run + log2f(l) : -INFINITY;
      // rows of this warp, 32 channels at a time: scaled, staged in the shared memory of the
      // warp's own query rows (free now, and no other warp writes there; 16-byte pieces
      // swizzled by row), written out by whole rows
      const bool part = s.slot >= 0, f32 = part || a.o_f32;
      const int64_t out0 = part ? (int64_t)s.slot * a.part_rows : row00;
      const int to = mine ? (part ? row : rel) : -1;
      float* of = (part ? a.part_o : static_cast<float*>(a.O)) + out0 * D;
      __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(a.O) + out0 * D;
      const int c0 = !dual && st ? D / 2 : 0, c1 = !dual && !st ? D / 2 : D;
      const bool merge = !dual;
      const float w0 = merge || st == 0 ? f[0] : f[1], w1 = merge ? f[1] : 0.f;
      if (warp_mine) {
        const uint32_t stage = smem_u32(s_q) + (uint32_t)(st * L::kTileBytes + (warp & 3) * 32 * 128);
#pragma unroll 1
        for (int j = c0; j < c1; j += 32) {
          uint32_t x0[32];
          float o[32];
          __syncwarp();  // (the pieces staged before have been read)
          tmem_ld32p(lane_base + kTmemO + (merge ? 0 : st * D) + j, x0);
          tmem_wait_ld_regs32(x0);
          // an accumulator without a key holds no data: weight 0 exactly
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = w0 != 0.f ? __uint_as_float(x0[e]) * w0 : 0.f;
          if (merge) {
            tmem_ld32p(lane_base + kTmemO + D + j, x0);
            tmem_wait_ld_regs32(x0);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (w1 != 0.f) o[e] = fmaf(__uint_as_float(x0[e]), w1, o[e]);
          }
          if (f32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) st_shared4(stage + lane * 128 + ((e ^ (lane & 7)) << 4), o + 4 * e);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // 8 lanes a row
              const int r = 4 * i + (lane >> 3), e = lane & 7;
              const int at = __shfl_sync(0xffffffffu, to, r);
              const float4 v = ld_shared4(stage + r * 128 + ((e ^ (r & 7)) << 4));
              if (at >= 0) *reinterpret_cast<float4*>(of + (int64_t)at * D + j + 4 * e) = v;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 pk = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                          pack_bf16x2(o[8 * e + 4], o[8 * e + 5]),
                                          pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
              st_shared4(stage + lane * 64 + ((e ^ (lane >> 1 & 3)) << 4), reinterpret_cast<const float*>(&pk));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // 4 lanes a row
              const int r = 8 * i + (lane >> 2), e = lane & 3;
              const int at = __shfl_sync(0xffffffffu, to, r);
              const float4 v = ld_shared4(stage + r * 64 + ((e ^ (r >> 1 & 3)) << 4));
              if (at >= 0) *reinterpret_cast<float4*>(ob + (int64_t)at * D + j + 8 * e) = v;
            }
          }
        }
      }
      if (mine && (dual || st == 0)) {
        if (part) a.part_lse[out0 + row] = lse2;
        else if (a.lse) a.lse[out0 + rel] = lse2 * kLn2;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      release_segment(n);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// Items that several CTAs share: CTA c of the attention started one and recorded
//   split[2c] = (rows, slot of its own part, parts, -), split[2c+1] = (first row of
//   the sequence, key head, first row of the item); parts 2, 3, .. are the first
//   slots of CTAs c+1, c+2, ..
// O = sum_i 2^(lse_i - lse) O_i with lse = log2 sum_i 2^lse_i, in the parts' order.
// Latency bound: a block finds the rows of all items from one read of the records;
// a warp takes a row and loads eight parts' log-sum-exps and outputs at once (d = 128 spills 84
// bytes of the 64 registers a thread that four blocks an SM leave).  With fewer rows than blocks
// the eight warps of a block share the parts of one row.
constexpr int kMaxCtas = 256;

template <int D>
__global__ void __launch_bounds__(kMaxCtas, 4) tree_combine_kernel(const __grid_constant__ TreeArgs a, int ctas) {
  constexpr int kWarps = kMaxCtas / 32;
  constexpr int C = D / 32;  // channels of a lane
  __shared__ int s_rows[kMaxCtas + 1];  // rows before CTA c's item
  __shared__ int4 s_item[kMaxCtas][2];
  __shared__ int s_warp[kWarps];
  __shared__ float s_o[kWarps][D];
  __shared__ float2 s_ml[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();  // the partial results come from the attention kernel before
  {
    const int c = threadIdx.x;
    int4 e = make_int4(0, 0, 0, 0), w = e;
    if (c < ctas) e = a.split[2 * c], w = a.split[2 * c + 1];
    const int rows = e.z > 0 ? e.x : 0;
    int up = rows;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += y;
    }
    if (lane == 31) s_warp[warp] = up;
    __syncthreads();
    for (int i = 0; i < warp; ++i) up += s_warp[i];
    s_rows[c] = up - rows;
    s_item[c][0] = e, s_item[c][1] = w;
    if (c == kMaxCtas - 1) s_rows[kMaxCtas] = up;
    __syncthreads();
  }
  const int rows = s_rows[kMaxCtas];
  const bool shared = rows <= (int)gridDim.x;  // a block per row
  const int step = shared ? gridDim.x : gridDim.x * kWarps;
  for (int i = shared ? blockIdx.x : blockIdx.x * kWarps + warp; i < rows; i += step) {
    int c0 = 0, c1 = kMaxCtas;  // the last c with s_rows[c] <= i has rows
    while (c1 - c0 > 1) {
      const int mid = (c0 + c1) / 2;
      if (s_rows[mid] <= i) c0 = mid;
      else c1 = mid;
    }
    const int4 e = s_item[c0][0], w = s_item[c0][1];
    const int row = i - s_rows[c0];
    const int parts = e.z;
    // running maximum m of the log-sum-exps, sum l of the weights 2^(lse - m), weighted outputs
    float m = -INFINITY, l = 0.f, acc[C] = {};
    const int stride = shared ? kWarps : 1;
    for (int p0 = shared ? warp : 0; p0 < parts; p0 += 8 * stride) {
      float ls[8], o[8][C];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = p0 + j * stride;
        const int64_t at = (int64_t)(p == 0 ? e.y : 2 * (c0 + p)) * a.part_rows + row;
        ls[j] = p < parts ? a.part_lse[at] : -INFINITY;
#pragma unroll
        for (int k = 0; k < C; ++k) o[j][k] = p < parts ? a.part_o[at * D + 32 * k + lane] : 0.f;
      }
      float mn = m;
#pragma unroll
      for (int j = 0; j < 8; ++j) mn = max_nan(mn, ls[j]);
      if (mn == -INFINITY) continue;  // no part has a key yet
      const float f = fast_exp2(m - mn);
      m = mn, l *= f;
#pragma unroll
      for (int k = 0; k < C; ++k) acc[k] *= f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wt = fast_exp2(ls[j] - m);
        l += wt;
#pragma unroll
        for (int k = 0; k < C; ++k) acc[k] = fmaf(wt, o[j][k], acc[k]);
      }
    }
    if (shared) {
#pragma unroll
      for (int k = 0; k < C; ++k) s_o[warp][32 * k + lane] = acc[k];
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        float mn = m;
        for (int p = 1; p < kWarps; ++p) mn = max_nan(mn, s_ml[p].x);
        const float m_use = mn == -INFINITY ? 0.f : mn;
        const float f = fast_exp2(m - m_use);
        m = mn, l *= f;
#pragma unroll
        for (int k = 0; k < C; ++k) acc[k] *= f;
        for (int p = 1; p < kWarps; ++p) {
          const float wt = fast_exp2(s_ml[p].x - m_use);
          l += wt * s_ml[p].y;
#pragma unroll
          for (int k = 0; k < C; ++k) acc[k] = fmaf(wt, s_o[p][32 * k + lane], acc[k]);
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const int nh = w.z + row;  // (node, head) of the sequence's rows for this key head
    const int64_t orow = (int64_t)(w.x + nh / a.G) * a.H + w.y * a.G + nh % a.G;
    const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int64_t to = orow * D + 32 * k + lane;
      if (a.o_f32) static_cast<float*>(a.O)[to] = acc[k] * inv;
      else static_cast<__nv_bfloat16*>(a.O)[to] = __float2bfloat16(acc[k] * inv);
    }
    if (a.lse && lane == 0) a.lse[orow] = l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

// K / V pages as [n_pages][Hk * page][d] bf16, fetched in boxes of up to 128 rows of
// one page x 64 channels (128-byte swizzle).
bool page_map(CUtensorMap* m, const void* base, int64_t n_pages, int Hk, int page, int d) {
  EncodeFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hk * page, (cuuint64_t)n_pages};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)Hk * page * d * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)(page < kTile ? page : kTile), 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a call: one per SM, fewer when even the longest sequences that the
// tables can hold give less than kMinShare key tiles each.  Without a page a sequence has
// no node, or is reported: one CTA looks.
int tree_ctas(int B, int64_t R, int H, int Hk, int page, int max_pages) {
  if (max_pages == 0) return 1;
  const int64_t sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  const int64_t nodes = R < kMaxNodes ? R : kMaxNodes;
  const int64_t seqs = B < R ? B : R;  // with a node
  const int64_t items = Hk * (seqs + R * (H / Hk) / kTile);  // row tiles
  const int64_t tiles = ceil_div((int64_t)max_pages * page, kTile) + (nodes > 0 ? 1 : 0);
  const int64_t most = items * (kItemCost + tiles * kSingleCost) / kMinShare;
  return (int)(most < 1 ? 1 : most < sms ? most : sms);
}

int part_rows(int64_t R, int H, int Hk) {
  const int64_t rows = (R < kMaxNodes ? R : kMaxNodes) * (H / Hk);
  return (int)(rows < kItemRows ? rows : kItemRows);
}

template <int D>
cudaError_t launch_tree(const TreeArgs& a, const TreeMaps& maps, int ctas, cudaStream_t stream) {
  constexpr size_t smem = TreeSmem<D>::bytes;
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess)
    e = launch_kernel(tree_attn_kernel<D>, dim3(ctas), dim3(kThreads), smem, stream, false, a, maps);
  // at most a warp per row of the call, and what the GPU holds at once
  const int64_t rows = ceil_div(a.R * a.H, kMaxCtas / 32), most = 4 * (int64_t)sm_count();
  const unsigned grid = (unsigned)(rows < most ? rows : most);
  if (e == cudaSuccess && ctas > 1)
    e = launch_kernel(tree_combine_kernel<D>, dim3(grid), dim3(kMaxCtas), 0, stream, true, a, ctas);
  return e;
}

}  // namespace
}  // namespace csa

using namespace csa;

extern "C" {

// [header][split 2 x int4 per CTA][partial lse][partial O], two slots per CTA: for every
// call that launches one (the header alone where csa_tree_attn refuses or has no rows)
size_t csa_tree_attn_workspace_bytes(int B, int64_t R, int H, int Hk, int d, int page, int max_pages) {
  if (B <= 0 || R <= 0 || H <= 0 || Hk <= 0 || H < Hk || (d != 64 && d != 128) || page <= 0 || max_pages < 0)
    return kWorkspaceHeader;
  const int ctas = tree_ctas(B, R, H, Hk, page, max_pages);
  const size_t rows = ctas > 1 ? (size_t)2 * ctas * part_rows(R, H, Hk) : 0;
  return kWorkspaceHeader + align256((size_t)ctas * 32) + align256(rows * 4) + align256(rows * d * 4);
}

int csa_tree_attn(const void* q, const void* Kpages, const void* Vpages, const int32_t* block_table,
                  const int32_t* seq_lens, const int32_t* q_start, const uint64_t* mask, const int64_t* pos, int64_t R,
                  int B, int H, int Hk, int d, int page, int64_t n_pages, int max_pages, int W, float scale, void* O,
                  int o_dtype, float* lse, void* workspace, size_t workspace_bytes, csa_stream_t stream) {
  const float scale_log2 = scale * 1.4426950408889634f;
  if (R < 0 || R > 0x7FFFFFFF || B < 0 || H < 1 || Hk < 1 || n_pages < 0 || max_pages < 0 || W < -1 ||
      !(std::isfinite(scale_log2) && scale_log2 > 0.f) || !valid_odtype(o_dtype))
    return CSA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || !valid_page(page) || H > 1024 || H % Hk != 0 || B > kMaxSeqs)
    return CSA_ERR_UNSUPPORTED_SHAPE;
  if ((int64_t)max_pages * page > 0x7FFFFFFF - kTile || n_pages > 0x7FFFFFFE) return CSA_ERR_UNSUPPORTED_SHAPE;
  int rc = check_ws(workspace, workspace_bytes, csa_tree_attn_workspace_bytes(B, R, H, Hk, d, page, max_pages));
  if (rc) return rc;
  if (R == 0 || B == 0) return CSA_OK;
  if ((rc = check_ptrs(q, seq_lens, q_start, mask, O))) return rc;
  if (W >= 0 && (rc = check_ptrs(pos))) return rc;
  if (max_pages > 0 && (rc = check_ptrs(block_table))) return rc;
  if (n_pages > 0 && (rc = check_ptrs(Kpages, Vpages))) return rc;
  if ((rc = check_opt(lse))) return rc;
  // a share writes its outputs while others still read what all of them share
  const size_t cache = (size_t)n_pages * Hk * page * d * 2;
  const Bytes out{O, span(R, (int64_t)H * d, H, d, o_dtype)}, sums{lse, (size_t)R * H * 4};
  for (const Bytes& o : {out, sums})
    if (overlap_any(o, {{q, span(R, (int64_t)H * d, H, d, CSA_BF16)},
                        {Kpages, cache},
                        {Vpages, cache},
                        {block_table, (size_t)B * max_pages * 4},
                        {seq_lens, (size_t)B * 4},
                        {q_start, (size_t)(B + 1) * 4},
                        {mask, (size_t)R * 8},
                        {W >= 0 ? pos : nullptr, (size_t)R * 8}}))
      return CSA_ERR_INVALID_ARG;
  if (overlap_any(out, {sums})) return CSA_ERR_INVALID_ARG;
  TreeArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.table = block_table;
  a.lens = seq_lens;
  a.q_start = q_start;
  a.mask = mask;
  a.pos = pos;
  a.R = R;
  a.n_pages = n_pages;
  a.B = B;
  a.H = H;
  a.Hk = Hk;
  a.G = H / Hk;
  a.max_pages = max_pages;
  while ((1 << a.page_shift) < page) ++a.page_shift;
  a.W = W;
  a.scale_log2 = scale_log2;
  a.O = O;
  a.o_f32 = o_dtype == CSA_F32;
  a.lse = lse;
  a.status = status_word(workspace);
  const int ctas = tree_ctas(B, R, H, Hk, page, max_pages);
  a.part_rows = part_rows(R, H, Hk);
  uint8_t* w = static_cast<uint8_t*>(workspace) + kWorkspaceHeader;
  a.split = reinterpret_cast<int4*>(w);
  w += align256((size_t)ctas * 32);
  a.part_lse = reinterpret_cast<float*>(w);
  a.part_o = reinterpret_cast<float*>(w + align256((size_t)2 * ctas * a.part_rows * 4));
  TreeMaps maps;
  const void* kb = n_pages > 0 ? Kpages : q;  // no pages: every page number is out of bounds, nothing is fetched
  const void* vb = n_pages > 0 ? Vpages : q;
  if (!page_map(&maps.k, kb, n_pages > 0 ? n_pages : 1, n_pages > 0 ? Hk : 1, page, d) ||
      !page_map(&maps.v, vb, n_pages > 0 ? n_pages : 1, n_pages > 0 ? Hk : 1, page, d))
    return cuda_fail(cudaErrorInvalidValue);
  cudaError_t e = d == 128 ? launch_tree<128>(a, maps, ctas, (cudaStream_t)stream)
                           : launch_tree<64>(a, maps, ctas, (cudaStream_t)stream);
  return e == cudaSuccess ? CSA_OK : cuda_fail(e);
}

}  // extern "C"
