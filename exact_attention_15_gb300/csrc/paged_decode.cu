// Attention of a few new query rows per sequence over a paged key-value cache:
// one token per sequence (decoding), or chunks of a few tokens.
//
// Every key and value is read once and meets only the query rows of its KV
// head, so the bytes bound the work. The query rows of a sequence that share a
// KV head (tokens x heads of the group, row = token * group + head) are cut into
// chunks of R = 8 or 16 rows; a work unit is one 64-key tile of one (sequence,
// KV head, chunk). The units are numbered with the tile innermost and dealt out
// evenly and in order, so every CTA streams the same number of tiles whatever
// the sequences' lengths are. A CTA whose run ends inside an item leaves its
// (m, l, O) in the workspace; paged_join_kernel merges the pieces of an item in
// their order, so results do not depend on timing.
//
// Of short contexts, dealing out and the second kernel would be most of the time: a
// cluster of 1 to 8 CTAs takes an item whole, each an even run of its tiles, and its CTAs
// join their pieces through each other's shared memory (one sequence of 777 keys, 32
// heads on 8: 7.3 -> 5.6 us; 16 of 256: 9.0 -> 6.1; 64 new tokens: 8.5 -> 4.9).
//
// Warp roles (160 threads): warps 0-3 each take 16 keys of a tile, S = Q K^T
// and O += P V on mma.sync m16n8k16 with the online softmax in registers
// (tcgen05 wants 128 rows; here there are 16 at most, and the tensor work is
// small against the tile's bytes); warp 4 walks the work, hands its pieces to the
// others through a ring and loads the tiles with TMA.
#include "paged.cuh"

namespace attn {

namespace {

constexpr int kTile = kStreamTile;
constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kRing = 4;  // pieces that the loading warp can be ahead

template <int D, int R, bool FP8>
struct StreamCfg {
  static constexpr int kEs = FP8 ? 1 : 2;
  static constexpr int kCtas = stream_ctas(R, D * kEs);
  // a tile is kept as blocks of 64 rows x (at most) 128 bytes, swizzled
  static constexpr int kRowBytes = D * kEs < 128 ? D * kEs : 128;
  static constexpr int kBlocks = D * kEs / kRowBytes;
  static constexpr int kBlockBytes = kTile * kRowBytes;
  static constexpr int kTileBytes = kBlocks * kBlockBytes;  // K or V
  static constexpr int kStages = kCtas == 3 ? 49152 / (2 * kTileBytes) : kTileBytes == 16384 ? 3 : 6;
  static constexpr int kMergeOff = kStages * 2 * kTileBytes;
  static constexpr int kMergeBytes = 16384;
  static constexpr int kMlOff = kMergeOff + kMergeBytes;
  static constexpr int kRingOff = kMlOff + kWarps * 16 * 2 * 4;
  static constexpr int kBarOff = kRingOff + kRing * 48;
  static constexpr int kPieceOff = kBarOff + (2 * kStages + 2 * kRing + 2) * 8;  // clusters: [16][2]
  static constexpr int kSmemBytes = kPieceOff + 16 * 2 * 4;
  // the CTAs share an SM's 228 KB, of which each takes 1 KB besides its own
  static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory of an SM");
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <bool FP16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};" : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};" : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 block of 16-bit values held as accumulator columns.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Beginning and ending an item (its queries' latency, the merge of the warps)
// costs a CTA about as much as two tiles of it: it counts as units of its own, so
// that runs of short items are not dealt out as if they were free. Measured on
// 128 ragged e4m3 sequences of 64 to 4096 keys, 4 KV heads: 48.3 us with 0 units,
// 46.7 with 1, 2 or 3; on 32 ragged ones with 16 heads of 64: 29.5, 28.7, 29.0, 29.1.
constexpr int kItemCost = 2;
// Work units of sequence b: (key tiles + kItemCost) x KV heads x chunks of R rows.
__device__ __forceinline__ long long units_of(const StreamParams& p, int b, int R) {
  const int n = new_span(p.s, b).len;
  const long long chunks = (static_cast<long long>(n) * p.group + R - 1) / R;
  const long long tiles = (static_cast<long long>(kv_len(p.s, b)) + kTile - 1) / kTile;
  return tiles > 0 ? (tiles + kItemCost) * p.H_kv * chunks : 0;
}
// CTAs that `total` units are dealt to (each of them has one unit at least).
__device__ __forceinline__ int busy_ctas(long long total, int grid) {
  return static_cast<int>(min(total, static_cast<long long>(grid)));
}
// First unit of CTA c of `grid` busy ones, and the CTA that holds unit u.
__device__ __forceinline__ long long first_unit(long long total, int grid, int c) {
  return total * c / grid;
}
__device__ __forceinline__ int owner_of(long long total, int grid, long long u) {
  return static_cast<int>(((u + 1) * grid - 1) / total);
}

// The piece of an item that a CTA works on.
struct __align__(16) Piece {
  int b, h, rc;      // sequence (< 0: no piece more), KV head, row chunk
  int t0, t1;        // key tiles [t0, t1)
  int tiles;         // of the whole item
  int len, n, row0;  // keys; query rows of the sequence and the first of them
  int slot;          // of the partial results, or -1: the piece is a whole item
  int pad[2];
};
static_assert(sizeof(Piece) == 48, "a place of the ring");

// Walks the units [u, end) of a CTA piece by piece.
struct Walk {
  long long u, end, base;  // next unit; first unit of sequence b
  int b;
};
template <int R>
__device__ __forceinline__ bool next_piece(const StreamParams& p, Walk& w, Piece& x) {
  while (w.u < w.end) {
    for (;;) {
      if (w.b >= p.s.B) return false;
      const long long n = units_of(p, w.b, R);
      if (w.u < w.base + n) break;
      w.base += n;
      ++w.b;
    }
    x.b = w.b;
    x.len = kv_len(p.s, w.b);
    const SeqSpan sp = new_span(p.s, w.b);
    x.n = sp.len;
    x.row0 = sp.start;
    x.tiles = (x.len + kTile - 1) / kTile;
    const int cost = x.tiles + kItemCost;
    const int chunks = static_cast<int>((static_cast<long long>(x.n) * p.group + R - 1) / R);
    const long long off = w.u - w.base;
    // (a 32-bit division where it will do)
    const int item = off <= 0xffffffffll ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(cost))
                                         : static_cast<int>(off / cost);
    const int o0 = static_cast<int>(off - static_cast<long long>(item) * cost);
    const int o1 = static_cast<int>(min(static_cast<long long>(cost), o0 + (w.end - w.u)));
    w.u += o1 - o0;
    x.t0 = max(0, o0 - kItemCost);
    x.t1 = max(0, o1 - kItemCost);
    if (x.t0 == x.t1) continue;  // only the item's beginning
    x.h = item / chunks;
    x.rc = item - x.h * chunks;
    return true;
  }
  return false;
}

// Clusters of 2^cluster_shift CTAs for an item each: this CTA's piece (one warp, the
// same in every lane). There can be more clusters than items (b < 0).
constexpr int kMaxCluster = kStreamCluster;
__device__ __forceinline__ int cluster_tile(const StreamParams& p, int tiles, int rank) {
  return (tiles * rank) >> p.cluster_shift;  // (2^25 tiles at most)
}
// A CTA of the cluster has the whole item.
__device__ __forceinline__ bool cluster_whole(const StreamParams& p, int tiles) {
  return tiles == 1 || (p.cluster_shift == 0 && tiles > 0);
}
template <int R>
__device__ __forceinline__ void cluster_piece(const StreamParams& p, int lane, Piece& x) {
  const int item = blockIdx.x >> p.cluster_shift, rank = blockIdx.x - (item << p.cluster_shift);
  const int row = item / p.H_kv;  // chunk of query rows, counted over the sequences
  x.h = item - row * p.H_kv;
  x.t0 = x.t1 = x.tiles = x.len = x.n = 0;
  if (!p.s.cu_seqlens) {
    const int chunks = (p.group + R - 1) / R;
    x.b = row / chunks;
    x.rc = row - x.b * chunks;
  } else {
    auto chunks_of = [&](int b) {
      return (static_cast<long long>(new_span(p.s, b).len) * p.group + R - 1) / R;
    };
    // every lane sums a run of sequences, and the run that holds the chunk is walked
    const int run = (p.s.B + 31) >> 5, b1 = min(p.s.B, (lane + 1) * run);
    long long mine = 0;
    for (int b = lane * run; b < b1; ++b) mine += chunks_of(b);
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    x.b = -1;
    if (row >= __shfl_sync(0xffffffffu, before, 31)) return;
    before -= mine;
    const int at = 31 - __clz(__ballot_sync(0xffffffffu, before <= row));
    x.b = at * run;
    long long base = __shfl_sync(0xffffffffu, before, at);
    for (long long n = chunks_of(x.b); row >= base + n; n = chunks_of(x.b)) {
      base += n;
      ++x.b;
    }
    x.rc = static_cast<int>(row - base);
  }
  x.len = kv_len(p.s, x.b);
  const SeqSpan sp = new_span(p.s, x.b);
  x.n = sp.len;
  x.row0 = sp.start;
  x.tiles = (x.len + kTile - 1) / kTile;
  x.t0 = cluster_tile(p, x.tiles, rank);
  x.t1 = cluster_tile(p, x.tiles, rank + 1);
}

// O = 0 and LSE = -inf for the query rows of a sequence without keys (one warp).
template <int D>
__device__ __forceinline__ void write_empty(const StreamParams& p, SeqSpan rows, int lane) {
  uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) +
                                      static_cast<size_t>(rows.start) * p.H_q * D);
  const long long chunks = static_cast<long long>(rows.len) * p.H_q * (D / 8);
  for (long long i = lane; i < chunks; i += 32) o[i] = make_uint4(0, 0, 0, 0);
  for (long long i = lane; i < static_cast<long long>(rows.len) * p.H_q; i += 32) {
    const int r = static_cast<int>(i / p.H_q), head = static_cast<int>(i - static_cast<long long>(r) * p.H_q);
    p.lse[(rows.start + r) * p.lse_row + head * p.lse_head] = -INFINITY;
  }
}

// CLUSTER: the CTAs of a cluster share one item and join their pieces through each
// other's shared memory.
template <int D, int R, bool FP8, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, StreamCfg<D, R, FP8>::kCtas)
paged_stream_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                    const StreamParams p) {
  using Cfg = StreamCfg<D, R, FP8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* merge = reinterpret_cast<float*>(smem + Cfg::kMergeOff);
  float* ml = reinterpret_cast<float*>(smem + Cfg::kMlOff);  // [warp][16][2]
  Piece* ring = reinterpret_cast<Piece*>(smem + Cfg::kRingOff);
  const uint32_t full = smem_addr(smem + Cfg::kBarOff), empty = full + 8 * Cfg::kStages;
  const uint32_t given = empty + 8 * Cfg::kStages, taken = given + 8 * kRing;  // of the ring
  const uint32_t merge_free = taken + 8 * kRing;  // the merge buffer has been read
  const uint32_t merge_full = merge_free + 8;     // the four warps have written it
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long lim = p.wait_limit;

  if (tid == 0) {
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, kWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(given + 8 * i, 1);
      mbar_init(taken + 8 * i, kWarps);
    }
    mbar_init(merge_free, kWarps);
    mbar_init(merge_full, kWarps);
    fence_barrier_init();
  }
  float* piece_o = reinterpret_cast<float*>(smem);  // clusters: [R][D], once the tiles are read
  float* piece_ml = reinterpret_cast<float*>(smem + Cfg::kPieceOff);
  const int cta = blockIdx.x;
  __syncthreads();
  grid_wait();
  int stage = 0;
  uint32_t phase = 0;

  if (warp == kWarps) {
    // ------------------------------------------------------------ TMA producer
    // The units before each sequence: every lane sums a run of sequences, the sums
    // are scanned, and the run that holds this CTA's first unit is walked.
    long long total = 0;
    int grid = 0;
    Walk w;
    if constexpr (!CLUSTER) {
      const int run = (p.s.B + 31) >> 5;
      long long before;
      const int b1 = min(p.s.B, (lane + 1) * run);
      long long mine = 0;
#pragma unroll 4
      for (int b = lane * run; b < b1; ++b) mine += units_of(p, b, R);
      before = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
      }
      total = __shfl_sync(0xffffffffu, before, 31);
      before -= mine;
      grid = busy_ctas(total, gridDim.x);
      w.u = w.end = w.base = 0;
      w.b = 0;
      if (cta < grid) {
        w.u = first_unit(total, grid, cta);
        w.end = first_unit(total, grid, cta + 1);
        // the last run that starts at or before the first unit (lane 0's does)
        const int at = 31 - __clz(__ballot_sync(0xffffffffu, before <= w.u));
        w.b = at * run;
        w.base = __shfl_sync(0xffffffffu, before, at);
      }
    }
    // Lane (page j of the tile, K or V, block) issues one box per tile.
    const int box_shift = min(p.s.page_shift, 6);
    const int n_box = kTile >> box_shift;  // pages (or the part of one) in a tile
    constexpr int kPer = 2 * Cfg::kBlocks;
    const int j = lane / kPer, which = (lane / Cfg::kBlocks) & 1, blk = lane % Cfg::kBlocks;
    const int box_row = j << box_shift;
    const bool has_box = j < n_box;
    const uint32_t dst0 = smem_addr(smem) + which * Cfg::kTileBytes + blk * Cfg::kBlockBytes +
                          box_row * Cfg::kRowBytes;
    const CUtensorMap* map = which ? &tm_v : &tm_k;
    if (lane == 0) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    bool ok = true, split_head = false;
    Piece x;
    // Gives piece number k to the other warps.
    auto give = [&](int k) {
      const int at = k % kRing;
      if (k >= kRing && !mbar_wait_warp(taken + 8 * at, ((k / kRing) - 1) & 1, lim)) return false;
      if (lane == 0) {
        ring[at] = x;
        mbar_arrive(given + 8 * at);
      }
      __syncwarp();
      return true;
    };
    int nth = 0;
    auto next = [&]() {
      if constexpr (!CLUSTER) return next_piece<R>(p, w, x);
      if (nth == 0) cluster_piece<R>(p, lane, x);
      return nth == 0;
    };
    for (; ok && next(); ++nth) {
      // a CTA's first and last piece can be parts of an item
      const bool whole = x.t1 - x.t0 == x.tiles;
      x.slot = whole ? -1 : 2 * cta + (nth == 0 ? 0 : 1);
      if (!(ok = give(nth))) break;
      if (!CLUSTER && x.t0 == 0 && !whole) {
        // for the join: the item begins in this CTA and ends in a later one
        split_head = true;
        if (lane == 0) {
          const int end = owner_of(total, grid, w.u + (x.tiles - x.t1) - 1);
          p.heads[2 * cta] = make_int4(end - cta + 1, x.slot, x.row0, min(R, x.n * p.group - x.rc * R));
          p.heads[2 * cta + 1] = make_int4(x.h, x.rc * R, 0, 0);
        }
      }
      auto page_at = [&](int t) {
        const int key = t * kTile + box_row;
        return has_box && key < x.len ? page_of(p.s, x.b, key >> p.s.page_shift) : 0;
      };
      int id = page_at(x.t0);
      for (int t = x.t0; t < x.t1; ++t) {
        const int key0 = t * kTile;
        const int here = id;
        if (t + 1 < x.t1) id = page_at(t + 1);
        if (!mbar_wait_warp(empty + 8 * stage, phase ^ 1, lim)) { ok = false; break; }
        // boxes that hold a key; the rows of the others keep what they held
        const int boxes = min(n_box, (x.len - key0 + (1 << box_shift) - 1) >> box_shift);
        if (lane == 0)
          mbar_arrive_expect_tx(full + 8 * stage, boxes * kPer * (Cfg::kRowBytes << box_shift));
        __syncwarp();
        if (j < boxes)
          tma_load_4d(dst0 + stage * 2 * Cfg::kTileBytes, map, full + 8 * stage,
                      blk * (Cfg::kRowBytes / Cfg::kEs),
                      (key0 + box_row) & ((1 << p.s.page_shift) - 1), x.h, here);
        if (++stage == Cfg::kStages) { stage = 0; phase ^= 1; }
      }
    }
    if (!CLUSTER && ok) {
      x.b = -1;
      ok = give(nth);
    }
    if (!ok) {
      if (lane == 0) record_error(p.s.err, kErrTimeout);
      // no copy may still be on its way when the CTA's shared memory goes
      for (int s = 0; s < Cfg::kStages; ++s) mbar_wait_warp(full + 8 * s, s < stage ? phase : phase ^ 1, lim);
    }
    // off the way of the loads: what no work unit covers
    if (!CLUSTER && !split_head && lane == 0) p.heads[2 * cta] = make_int4(0, 0, 0, 0);
    if (cta == 0) check_paged_seqs(p.s, lane, 32);
    for (int b = cta; !CLUSTER && b < p.s.B; b += gridDim.x)
      if (kv_len(p.s, b) == 0) write_empty<D>(p, new_span(p.s, b), lane);
    if constexpr (CLUSTER) {
      __syncwarp();
      if (x.b >= 0 && !cluster_whole(p, x.tiles)) {
        cluster_sync_all();
        cluster_sync_all();
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  // Both products keep the query rows in N = 8 columns: S^T = K Q^T (M = 16 keys)
  // and O^T += V^T P^T (M = 16 columns of V), so 8 rows fill the instruction that
  // 16 would need in M. Lane: accumulator rows ar and ar + 8 (keys, or columns
  // of V), accumulator columns 2 qd and 2 qd + 1 (query rows).
  const int qd = lane & 3, ar = lane >> 2;
  const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: matrix and row of this lane's address
  const int krow = warp * 16 + (mi & 1) * 8 + mr, vrow = warp * 16 + (mi >> 1) * 8 + mr;
  // byte offset of this lane's row and first chunk; chunk c (even) lies at
  // (offset + block) ^ (c << 4), since the swizzle is an XOR on those bits
  auto row_off = [&](int row, int ch) {
    const int sw = Cfg::kRowBytes == 128 ? row & 7 : (row >> 1) & 3;
    return row * Cfg::kRowBytes + ((ch ^ sw) << 4);
  };
  const uint32_t koff = row_off(krow, mi >> 1), voff = row_off(vrow, mi & 1);
  constexpr int kChunks = Cfg::kRowBytes / 16;  // 16-byte chunks of a block's row
  auto chunk_at = [&](uint32_t base, int c) {
    return (base + (c / kChunks) * Cfg::kBlockBytes) ^ ((c % kChunks) << 4);
  };
  constexpr int NB = R / 8;  // blocks of 8 query rows
  // Query rows as B fragments: row nb * 8 + ar. The next piece's rows are loaded
  // before the merge of the last one, which hides their latency.
  uint32_t qb[NB][D / 16][2];
  auto load_q = [&](const Piece& x) {
    const int rows = min(R, x.n * p.group - x.rc * R);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) qb[nb][kk][0] = qb[nb][kk][1] = 0u;
      if (nb * 8 + ar >= rows) continue;
      const int rr = x.rc * R + nb * 8 + ar;
      const int tok = rr / p.group, head = rr - tok * p.group;
      const uint8_t* src = static_cast<const uint8_t*>(p.q) +
          ((static_cast<size_t>(x.row0 + tok) * p.H_q + x.h * p.group + head) * D) * 2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if constexpr (FP8) {  // the lane's four consecutive columns
          const uint2 q4 = *reinterpret_cast<const uint2*>(src + kk * 32 + qd * 8);
          qb[nb][kk][0] = q4.x;
          qb[nb][kk][1] = q4.y;
        } else {
          qb[nb][kk][0] = *reinterpret_cast<const uint32_t*>(src + kk * 32 + qd * 4);
          qb[nb][kk][1] = *reinterpret_cast<const uint32_t*>(src + kk * 32 + qd * 4 + 16);
        }
      }
    }
  };
  bool ok = true;
  Piece x;
  x.b = -2;     // not known
  int nth = 0;  // pieces taken
  auto take = [&]() {  // the next piece, in every lane
    const int at = nth % kRing;
    if (!mbar_wait_warp(given + 8 * at, (nth / kRing) & 1, lim) || (p.fault == kFaultLeaveWarp && warp == 1)) {
      if (lane == 0) record_error(p.s.err, kErrTimeout);
      return false;
    }
    const int4* src = reinterpret_cast<const int4*>(&ring[at]);
    int4* dst = reinterpret_cast<int4*>(&x);
#pragma unroll
    for (int i = 0; i < 3; ++i) dst[i] = src[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(taken + 8 * at);
    ++nth;
    return x.b >= 0;
  };
  constexpr float lift = FP8 ? kLift : 0.0f;
  uint32_t merges = 0;  // uses of the merge buffer
  bool have = take();
  if (CLUSTER) have = have && x.t0 < x.t1;
  if (have) load_q(x);
  while (have) {
    const int rows = min(R, x.n * p.group - x.rc * R);  // of this chunk
    // Over an e4m3 cache the products run in fp16, which holds every e4m3 value
    // exactly; each query row is brought to [1, 2) by a power of two first.
    float c[NB][2];   // exponent scale of the lane's accumulator columns
    int last[NB][2];  // keys that those rows see
    const float k_scale = FP8 && p.k_scale ? __ldg(p.k_scale + x.h) : 1.0f;
    const float v_scale = FP8 && p.v_scale ? __ldg(p.v_scale + x.h) : 1.0f;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float up = 1.0f;  // the power of two that the row was divided by
      if constexpr (FP8) {
        float top = 0.0f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            top = fmaxf(top, fmaxf(fabsf(bf16lo_to_f32(qb[nb][kk][e])), fabsf(bf16hi_to_f32(qb[nb][kk][e]))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float down;
        up = row_power(top, down);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            qb[nb][kk][e] = pack_f16x2(bf16lo_to_f32(qb[nb][kk][e]) * down, bf16hi_to_f32(qb[nb][kk][e]) * down);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = nb * 8 + 2 * qd + e, tok = (x.rc * R + r) / p.group;
        c[nb][e] = p.scale_log2 * k_scale * __shfl_sync(0xffffffffu, up, (2 * qd + e) * 4);
        last[nb][e] = r >= rows ? 0 : p.causal ? min(x.len, x.len - x.n + tok + 1) : x.len;
      }
    }
    float acc[NB][D / 16][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nb][j][e] = 0.0f;
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) { m[nb][e] = -INFINITY; l[nb][e] = 0.0f; }

    for (int t = x.t0; t < x.t1; ++t) {
      if (ok && !mbar_wait_warp(full + 8 * stage, phase, lim)) {
        // the copies may still be on their way: one more bounded wait, then the
        // rest of the work is walked without waiting
        if (lane == 0) record_error(p.s.err, kErrTimeout);
        mbar_wait_warp(full + 8 * stage, phase, lim);
        ok = false;
      }
      const int key0 = t * kTile + warp * 16;
      if (key0 < x.len) {
        const uint32_t tile = smem_addr(smem) + stage * 2 * Cfg::kTileBytes;
        const uint32_t kb = tile + koff, vb = tile + Cfg::kTileBytes + voff;
        // S in two independent chains of products: half the columns each with 8
        // rows, one per block with 16
        constexpr int kChains = NB == 1 ? 2 : 1;
        float sc[NB][kChains][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < kChains; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[nb][h][e] = 0.0f;
        if constexpr (FP8) {
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t f[4];
            ldsm4(chunk_at(kb, 2 * cc), f);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t a[4] = {e4m3x2_to_f16x2(f[2 * u]), e4m3x2_to_f16x2(f[2 * u + 1]),
                                     e4m3x2_to_f16x2(f[2 * u] >> 16), e4m3x2_to_f16x2(f[2 * u + 1] >> 16)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<true>(sc[nb][u % kChains], a, qb[nb][2 * cc + u][0], qb[nb][2 * cc + u][1]);
            }
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t f[4];
            ldsm4(chunk_at(kb, 2 * kk), f);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<false>(sc[nb][kk % kChains], f, qb[nb][kk][0], qb[nb][kk][1]);
          }
        }
        // scaled scores s[nb][e]: key ar + 8 (e >> 1), query row 2 qd + (e & 1)
        float sv[NB][4];
        bool grew = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + ar + 8 * (e >> 1);
            const float v = (kChains == 2 ? sc[nb][0][e] + sc[nb][kChains - 1][e] : sc[nb][0][e]) * c[nb][e & 1];
            sv[nb][e] = key < last[nb][e & 1] ? v : -INFINITY;
            grew |= sv[nb][e] - m[nb][e & 1] > kTau;
          }
        // The bias moves only when some score exceeds it by more than 2^tau;
        // until then no maximum has to be taken at all.
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(fmaxf(sv[nb][e], sv[nb][e + 2]), m[nb][e]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const float f = mx > m[nb][e] ? ex2_approx(m[nb][e] - mx) : 1.0f;
              m[nb][e] = mx;
              l[nb][e] *= f;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                acc[nb][j][e] *= f;
                acc[nb][j][e + 2] *= f;
              }
            }
        }
        // P sums up in 32 bits before it is rounded to the product's 16-bit type
        // (bf16 as in the prompt kernels, fp16 over an e4m3 cache); its 8 x 8
        // blocks are transposed into B fragments.
        uint32_t pb[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float pv[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              pv[e] = ex2_approx(sv[nb][2 * h + e] - (m[nb][e] == -INFINITY ? 0.0f : m[nb][e] - lift));
              l[nb][e] += pv[e];
            }
            pb[nb][h] = transpose8x8(FP8 ? pack_f16x2(pv[0], pv[1]) : pack_bf16x2(pv[0], pv[1]));
          }
        // Rows of V past the sequence's end can hold anything (a page's unused
        // rows, an earlier tile): they are replaced by zeros, since 0 x NaN is NaN.
        uint32_t vm[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int key = key0 + n * 8 + 2 * qd;
          vm[n] = (key < x.len ? 0x0000ffffu : 0u) | (key + 1 < x.len ? 0xffff0000u : 0u);
        }
        if constexpr (FP8) {
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t f[4];
            ldsm4_t(chunk_at(vb, 2 * cc), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] &= vm[e >> 1];
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // rows ar and ar + 8: columns 2 ar and 2 ar + 1
              const uint32_t a[4] = {e4m3x2_to_f16x2(__byte_perm(f[u], 0, 0x4420)),
                                     e4m3x2_to_f16x2(__byte_perm(f[u], 0, 0x4431)),
                                     e4m3x2_to_f16x2(__byte_perm(f[2 + u], 0, 0x4420)),
                                     e4m3x2_to_f16x2(__byte_perm(f[2 + u], 0, 0x4431))};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<true>(acc[nb][2 * cc + u], a, pb[nb][0], pb[nb][1]);
            }
          }
        } else {
#pragma unroll
          for (int jj = 0; jj < D / 16; ++jj) {
            uint32_t f[4];
            ldsm4_t(chunk_at(vb, 2 * jj), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] &= vm[e >> 1];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<false>(acc[nb][jj], f, pb[nb][0], pb[nb][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * stage);
      if (++stage == Cfg::kStages) { stage = 0; phase ^= 1; }
    }

    // ---- merge of the four warps' keys
    const Piece y = x;
    have = !CLUSTER && take();
    if (have) load_q(x);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], o);
    const bool whole = y.slot < 0;
    // O passes through shared memory in runs of kCols columns, each 8-column
    // group moved within its row so that the warps' stores spread over the banks.
    // The warps leave their sums as they are; who adds them up knows the factors.
    constexpr int kCols = D * R * kWarps * 4 <= Cfg::kMergeBytes ? D : Cfg::kMergeBytes / (R * kWarps * 4);
    constexpr int kPerRow = kCols / 8;  // threads per row of the result
    static_assert(R * kPerRow <= 32 * kWarps, "one 8-column group per thread");
    const int r = tid / kPerRow, g8 = tid % kPerRow;
#pragma unroll
    for (int c0 = 0; c0 < D; c0 += kCols) {
      // the buffer's last readers are done
      if (merges > 0 && ok && !mbar_wait_warp(merge_free, (merges - 1) & 1, lim)) {
        if (lane == 0) record_error(p.s.err, kErrTimeout);
        ok = false;
      }
      ++merges;
      if (c0 == 0 && ar == 0) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float2*>(ml + (warp * 16 + nb * 8 + 2 * qd + e) * 2) = make_float2(m[nb][e] - lift, l[nb][e]);
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* dst = merge + (warp * R + nb * 8 + 2 * qd + e) * kCols;
#pragma unroll
          for (int j = c0 / 16; j < (c0 + kCols) / 16; ++j) {
            const float a = acc[nb][j][e], b = acc[nb][j][e + 2];
            const int col = j * 16 - c0;
            if constexpr (FP8) {
              *reinterpret_cast<float2*>(dst + ((col + 2 * ar) ^ (qd << 3))) = make_float2(a, b);
            } else {
              dst[(col + ar) ^ (qd << 3)] = a;
              dst[(col + ar + 8) ^ (qd << 3)] = b;
            }
          }
        }
      // A warp whose wait for a piece ran out has left, so the others may wait for it here
      // in vain: not a counted barrier, which would hold them for ever.
      __syncwarp();
      if (lane == 0) mbar_arrive(merge_full);
      if (!mbar_wait_warp(merge_full, (merges - 1) & 1, ok ? lim : 0)) {
        if (lane == 0) record_error(p.s.err, kErrTimeout);
        ok = false;
      }
      if (r < rows) {
        float2 w[kWarps];
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int g = 0; g < kWarps; ++g) {
          w[g] = *reinterpret_cast<const float2*>(ml + (g * 16 + r) * 2);
          top = fmaxf(top, w[g].x);
        }
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.0f;
#pragma unroll
        for (int g = 0; g < kWarps; ++g) {
          const float* src = merge + (g * R + r) * kCols + ((g8 * 8) ^ (((r >> 1) & 3) << 3));
          const float4 a = *reinterpret_cast<const float4*>(src);
          const float4 d4 = *reinterpret_cast<const float4*>(src + 4);
          const float f = ex2_approx(w[g].x - (top == -INFINITY ? 0.0f : top));
          sum += w[g].y * f;
          o[0] += a.x * f; o[1] += a.y * f; o[2] += a.z * f; o[3] += a.w * f;
          o[4] += d4.x * f; o[5] += d4.y * f; o[6] += d4.z * f; o[7] += d4.w * f;
        }
        const float f = whole ? (sum == 0.0f ? 0.0f : v_scale / sum) : v_scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f;
        if (whole) {
          const int rr = y.rc * R + r;
          const int tok = rr / p.group, head = y.h * p.group + rr - tok * p.group;
          const size_t row = static_cast<size_t>(y.row0 + tok);
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (row * p.H_q + head) * D + c0 +
                                    g8 * 8) =
              make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]),
                         pack_bf16x2(o[6], o[7]));
          if (c0 == 0 && g8 == 0)
            p.lse[row * p.lse_row + head * p.lse_head] =
                sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
        } else {
          float* dst = (CLUSTER ? piece_o + r * D : p.part_o + (static_cast<size_t>(y.slot) * 16 + r) * D) + c0 + g8 * 8;
          *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
          if (c0 == 0 && g8 == 0)
            *reinterpret_cast<float2*>(CLUSTER ? piece_ml + r * 2 : p.part_ml + (y.slot * 16 + r) * 2) =
                make_float2(top, sum);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(merge_free);
    }
  }
  if constexpr (CLUSTER) {
    // ---- join: row r of the item in CTA r mod the cluster's size, a warp each
    __syncwarp();
    if (x.b == -1 || (x.b >= 0 && cluster_whole(p, x.tiles))) return;
    cluster_sync_all();
    const int cluster = 1 << p.cluster_shift;
    const int rows = x.b < 0 ? 0 : min(R, x.n * p.group - x.rc * R);
    for (int r = (cta & (cluster - 1)) + cluster * warp; r < rows; r += cluster * kWarps) {
      constexpr int kV = D / 32;
      float2 w[kMaxCluster];
      float o[kMaxCluster][kV];
#pragma unroll
      for (int g = 0; g < kMaxCluster; ++g) {
        // (a CTA without a tile left nothing)
        const bool live = g < cluster && cluster_tile(p, x.tiles, g) < cluster_tile(p, x.tiles, g + 1);
        w[g] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int e = 0; e < kV; ++e) o[g][e] = 0.0f;
        if (live) {
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(w[g].x), "=f"(w[g].y)
                       : "r"(cluster_map(smem_addr(piece_ml + r * 2), g)) : "memory");
#pragma unroll
          for (int e = 0; e < kV; e += 2)
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(o[g][e]), "=f"(o[g][e + 1])
                         : "r"(cluster_map(smem_addr(piece_o + r * D + lane * kV + e), g)) : "memory");
        }
      }
      float top = -INFINITY, sum = 0.0f, acc[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] = 0.0f;
#pragma unroll
      for (int g = 0; g < kMaxCluster; ++g) top = fmaxf(top, w[g].x);
#pragma unroll
      for (int g = 0; g < kMaxCluster; ++g) {
        const float f = ex2_approx(w[g].x - (top == -INFINITY ? 0.0f : top));
        sum += w[g].y * f;
#pragma unroll
        for (int e = 0; e < kV; ++e) acc[e] += o[g][e] * f;
      }
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int rr = x.rc * R + r, tok = rr / p.group, head = x.h * p.group + rr - tok * p.group;
      const size_t row = static_cast<size_t>(x.row0) + tok;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) +
                                                  (row * p.H_q + head) * D + lane * kV);
#pragma unroll
      for (int e = 0; e < kV / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
      if (lane == 0)
        p.lse[row * p.lse_row + head * p.lse_head] = sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another one reads its pieces
  }
}

// Sums pieces part, part + step, ... of an item's row r: maximum, sum and the lane's
// D / 32 columns of O. Four pieces at a time, all their loads before the first is
// used (a place behind the last piece loads the last again, with no weight).
template <int D>
__device__ __forceinline__ void sum_pieces(const StreamParams& p, int c, int pieces, int slot0, int r, int part,
                                           int step, int lane, float& m, float& l, float (&acc)[D / 32]) {
  constexpr int kV = D / 32;
  const auto* ml_at = reinterpret_cast<const float2*>(p.part_ml) + r;
  const float* o_at = p.part_o + static_cast<size_t>(r) * D + lane * kV;
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] = 0.0f;
  for (int i0 = part; i0 < pieces; i0 += 4 * step) {
    float2 ml[4];
    float o[4][kV];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = min(i0 + step * k, pieces - 1);
      const int slot = i == 0 ? slot0 : 2 * (c + i);
      ml[k] = ml_at[slot * 16];
      const float* src = o_at + static_cast<size_t>(slot) * 16 * D;
      if constexpr (kV == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        o[k][0] = v.x; o[k][1] = v.y; o[k][2] = v.z; o[k][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        o[k][0] = v.x; o[k][1] = v.y;
      }
    }
    const float before = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, ml[k].x);
    const float bias = m == -INFINITY ? 0.0f : m, f = ex2_approx(before - bias);
    l *= f;
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] *= f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool live = i0 + step * k < pieces;
      const float g = ex2_approx(ml[k].x - bias);
      l += live ? ml[k].y * g : 0.0f;
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] += live ? o[k][e] * g : 0.0f;
    }
  }
}

// Merges the pieces of split items in their order. CTA (c, y) does some query rows of
// the item that begins in the streaming kernel's CTA c and ends in a later one; there
// are fewer such items than CTAs. kShare warps share a row: four where there are fewer
// items than SMs and so many pieces of each (with one, the pieces of a long sequence
// are joined 3 us later), one else, which takes fewer CTAs (32 ragged sequences of 16
// heads of 64: 30.6 us with four, 29.2 with one).
//
// Neither this kernel nor the streaming one lets the next grid launch early: the
// next streaming kernel's CTAs would find some SMs still full, and two of three would
// run there to the end (37 us for the same sequences).
template <int D, int kRows, int kShare>
__global__ void __launch_bounds__(32 * kRows * kShare)
paged_join_kernel(const StreamParams p) {
  __shared__ float sh_o[kShare > 1 ? kRows : 1][kShare][D];
  __shared__ float2 sh_ml[kShare > 1 ? kRows : 1][kShare];
  grid_wait();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, part = warp % kShare, lane = threadIdx.x & 31;
  const int at_row = warp / kShare, r = blockIdx.y * kRows + at_row;
  const int4 a = p.heads[2 * c], d = p.heads[2 * c + 1];
  const int pieces = a.x, rows = a.w;
  if (pieces == 0) return;
  constexpr int kV = D / 32;
  float acc[kV], m, l;
  if (r < rows) {
    sum_pieces<D>(p, c, pieces, a.y, r, part, kShare, lane, m, l, acc);
    if constexpr (kShare > 1) {
#pragma unroll
      for (int e = 0; e < kV; ++e) sh_o[at_row][part][lane * kV + e] = acc[e];
      if (lane == 0) sh_ml[at_row][part] = make_float2(m, l);
    }
  }
  if constexpr (kShare > 1) __syncthreads();
  if (r >= rows || part > 0) return;
  if constexpr (kShare > 1) {
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < kShare; ++g) top = fmaxf(top, sh_ml[at_row][g].x);
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] = 0.0f;
#pragma unroll
    for (int g = 0; g < kShare; ++g) {
      const float f = ex2_approx(sh_ml[at_row][g].x - (top == -INFINITY ? 0.0f : top));
      l += sh_ml[at_row][g].y * f;
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] += sh_o[at_row][g][lane * kV + e] * f;
    }
    m = top;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  const int rr = d.y + r, tok = rr / p.group, head = d.x * p.group + rr - tok * p.group;
  const size_t row = static_cast<size_t>(a.z) + tok;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (row * p.H_q + head) * D + lane * kV);
#pragma unroll
  for (int e = 0; e < kV / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0) p.lse[row * p.lse_row + head * p.lse_head] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
}

template <int D, int R, bool FP8>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, StreamParams p, int n_sm,
                   cudaStream_t stream) {
  using Cfg = StreamCfg<D, R, FP8>;
  p.grid = min(Cfg::kCtas * n_sm, kStreamCtas);
  int slot = prof_begin(kKPagedDecode, stream);
  cudaError_t e;
  if (p.cluster > 0) {
    for (p.cluster_shift = 0; 1 << p.cluster_shift < p.cluster;) ++p.cluster_shift;
    e = launch_clusters<paged_stream_kernel<D, R, FP8, true>>(
        p.cluster, dim3(static_cast<unsigned>(p.items * p.cluster)), kThreads, Cfg::kSmemBytes, stream, tk, tv, p);
    prof_end(slot, stream);
    return e;
  }
  e = launch_chained<paged_stream_kernel<D, R, FP8, false>>(dim3(p.grid), kThreads, Cfg::kSmemBytes, stream, tk, tv, p);
  prof_end(slot, stream);
  if (e != cudaSuccess) return e;
  slot = prof_begin(kKPagedJoin, stream);
  if (static_cast<long long>(p.s.B) * p.H_kv < n_sm)
    e = launch_chained<paged_join_kernel<D, R / 8, 4>>(dim3(p.grid, 8), 128 * (R / 8), 0, stream, p);
  else
    e = launch_chained<paged_join_kernel<D, 4, 1>>(dim3(p.grid, R / 4), 128, 0, stream, p);
  prof_end(slot, stream);
  return e;
}

}  // namespace

cudaError_t launch_paged_stream(const CUtensorMap& tk, const CUtensorMap& tv, const StreamParams& p,
                                int d, int rows, bool e4m3, int n_sm, cudaStream_t stream) {
  if (d == 128) {
    if (rows == 8) return e4m3 ? launch<128, 8, true>(tk, tv, p, n_sm, stream) : launch<128, 8, false>(tk, tv, p, n_sm, stream);
    return e4m3 ? launch<128, 16, true>(tk, tv, p, n_sm, stream) : launch<128, 16, false>(tk, tv, p, n_sm, stream);
  }
  if (rows == 8) return e4m3 ? launch<64, 8, true>(tk, tv, p, n_sm, stream) : launch<64, 8, false>(tk, tv, p, n_sm, stream);
  return e4m3 ? launch<64, 16, true>(tk, tv, p, n_sm, stream) : launch<64, 16, false>(tk, tv, p, n_sm, stream);
}

}  // namespace attn
