// Attention of chunks of new tokens over a paged key-value cache on the tensor
// cores (whole prompts, the next chunk of a prompt).
//
// The query rows of a sequence that share a KV head form the tiles: row r of a
// 128-row tile is token r / group, head r % group of the KV head, so a tile
// covers floor(128 / group) tokens and every key that it loads meets all the
// heads that use it. A work tile is two such tiles in a row; the CTA that owns it
// streams the keys and values that they see, 128 at a time, from the pages.
// Roles, TMEM plan and pipeline are those of the packed forward kernel at d = 128: P
// takes the place of S, so that softmax(j), P V(j) and S(j + 1) of a query tile follow one
// another, and two query tiles take turns. (At 64 that kernel keeps P in columns of its
// own; this one does not.)
//   warp 0      TMA producer: both Q tiles, then K_j / V_j into a ring; the lanes
//               look up the pages of a tile and issue one box each.
//   warp 1      TMEM owner and MMA issuer: S_i = Q_i K_j^T, O_i += P_i V_j.
//   warp 2      claims work tiles from a counter (longest sequences first) and
//               hands them to the other roles.
//   warps 4-11  softmax and epilogue, one warpgroup per query tile.
// Rows of V past the sequence's end can hold anything, and 0 x NaN is NaN: the
// MMA warp zeroes them in shared memory before the last P V product.
//
// Over an e4m3 cache the products run in fp16, which holds every e4m3 value exactly
// (the instructions take no operands of two types): half tiles of 64 keys land in a
// small ring of their own, and warps 2 and 3 widen one half each of every tile into
// the K / V ring (and put the zeros past the end); lane 0 of warp 2 looks for work
// between the tiles. The queries come as fp16 rows scaled by powers of two. One
// widening warp, which loads, converts and stores 16 values at a time, took 1181 us
// for the next 1024 tokens of two prompts of 25,000 (32 heads on 8, d 128); with a
// row's loads ahead of its conversions 773; two warps 661 (bf16: 506).
//
// With many work tiles the CTAs claim them one by one. With few, what the last
// wave leaves idle costs more: every CTA takes the same number of whole tiles, and
// the rest (fewer tiles than CTAs) is cut by keys into one share per CTA, such that
// all have the same work. A piece of a tile leaves its (m, l, O) in the workspace,
// and paged_fwd_join_kernel merges the pieces in order.
//
// TMEM (512 columns): O_0 [0, d), O_1 [d, 2d), S_0/P_0 [2d, 2d + 128), S_1/P_1
// [2d + 128, 2d + 256).
#include "fwd_softmax.cuh"
#include "paged.cuh"

namespace attn {

namespace {

template <int D, bool E4M3>
struct PagedFwdCfg {
  static constexpr int kBlocks = D / 64;                // 64-column blocks of a tile
  static constexpr int kBlockBytes = kTileM * 64 * 2;   // 16 KB
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  // e4m3: half tiles as they are in the cache, rows of D bytes swizzled over their
  // width, take the place of a quarter of the K / V ring
  static constexpr int kHalf = kTileN / 2;
  static constexpr int kRawBytes = kHalf * D;
  static constexpr int kRawStages = E4M3 ? 32768 / kRawBytes : 1;
  static constexpr int kStages = (D == 128 ? 4 : 8) * (E4M3 ? 3 : 4) / 4;
  static constexpr int kKVOff = 2 * kTileBytes;
  static constexpr int kRawOff = kKVOff + kStages * kTileBytes;
  static constexpr int kBarOff = kRawOff + (E4M3 ? kRawStages * kRawBytes : 0);
  static constexpr int kEpiOff = kBarOff + 1024;        // one staging block per warpgroup
  static constexpr int kSmemBytes = kEpiOff + 2 * kBlockBytes + 1024;
  static constexpr uint32_t kColS = 2 * D;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

struct __align__(16) PagedTile {
  int b, h;        // sequence (< 0 ends the list), KV head
  int row0;        // first packed row of the sequence
  int q0;          // first token of tile 0 within the chunk
  int n_new, len;  // tokens of the chunk, keys of the sequence
  int kt0;         // first key tile of this piece
  int n[2];        // key tiles that each query tile visits here
  int slot;        // of the partial results, or -1: the piece is whole
  int pad[2];
};

constexpr int kSlots = 2;     // of the ring that hands out work tiles
constexpr int kReaders = 10;  // producer warp, MMA warp, eight softmax warps (e4m3: and two that widen)

struct PagedBars {
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t raw_full[8], raw_empty[8];  // e4m3
  uint64_t sched_full[kSlots], sched_empty[kSlots];
  uint64_t drained;  // after a failure: the products in flight
  int sched_taken;  // work tiles that the producer has taken so far
  PagedTile sched_t[kSlots];
  uint32_t tmem_base;
};

// Work tiles of a sequence of n new tokens: blocks of 2 tok_tile tokens x KV heads.
__device__ __forceinline__ int m_blocks(const PagedFwdParams& p, int n) {
  const int rows = 2 * p.tok_tile;
  return (n + rows - 1) / rows;
}
// Keys that the tokens [q0, q0 + tok_tile) see: an upper bound for each of them.
__device__ __forceinline__ int keys_seen(const PagedFwdParams& p, int q0, int n, int len) {
  if (q0 >= n) return 0;
  return p.causal ? max(0, len - n + min(q0 + p.tok_tile, n)) : len;
}
// Work tile `local` of sequence b (rows row0 .. row0 + n of q, len keys): the tiles
// run from its last block of tokens (which sees most keys) to its first, the KV heads
// innermost. All its keys.
__device__ __forceinline__ void expand_tile(const PagedFwdParams& p, int local, int b, int row0, int n, int len,
                                            PagedTile& t) {
  t.b = b;
  t.row0 = row0;
  t.n_new = n;
  t.len = len;
  const int mi = local / p.H_kv;
  t.h = local - mi * p.H_kv;
  t.q0 = (m_blocks(p, n) - 1 - mi) * 2 * p.tok_tile;
  t.kt0 = 0;
  for (int i = 0; i < 2; ++i)
    t.n[i] = (keys_seen(p, t.q0 + i * p.tok_tile, t.n_new, t.len) + kTileN - 1) / kTileN;
  t.slot = -1;
}
// The last of `count` entries of a non-decreasing array that is <= x (the first
// one is). Entries without anything of their own share the next one's value and
// are never found.
__device__ __forceinline__ int find_last(const int* a, int count, int x) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}
// Units of a work tile: its key tiles, and what beginning and ending it costs
// (about two of them).
constexpr int kItemCost = 2;
__device__ __forceinline__ int tile_units(const PagedTile& t) { return max(t.n[0], t.n[1]) + kItemCost; }

// The k-th work tile of this CTA, as the scheduler warp published it; false at
// the end of the list, or when the wait ran out (`ok`).
__device__ __forceinline__ bool take_tile(PagedBars* bars, int k, PagedTile& t, long long lim, bool& ok) {
  const int slot = k % kSlots;
  if (!mbar_wait_warp(smem_addr(&bars->sched_full[slot]), (k / kSlots) & 1, lim)) {
    ok = false;
    return false;
  }
  const int4* src = reinterpret_cast<const int4*>(&bars->sched_t[slot]);
  int4* dst = reinterpret_cast<int4*>(&t);
#pragma unroll
  for (int w = 0; w < static_cast<int>(sizeof(PagedTile) / 16); ++w) dst[w] = src[w];
  // lane 0's copy, so that every field is known to be the same in all lanes
  int* f = reinterpret_cast<int*>(&t);
#pragma unroll
  for (int w = 0; w < static_cast<int>(sizeof(PagedTile) / 4); ++w)
    f[w] = __shfl_sync(0xffffffffu, f[w], 0);
  if ((threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&bars->sched_empty[slot]));
  return t.b >= 0;
}

// Publishes work tile k in the ring once every reader has taken tile k - kSlots.
__device__ __forceinline__ bool publish_tile(PagedBars* bars, int k, const PagedTile& t,
                                             const PagedFwdParams& p) {
  const int slot = k % kSlots;
  if (k >= kSlots &&
      !mbar_wait_sleep(smem_addr(&bars->sched_empty[slot]), ((k / kSlots) - 1) & 1, p.wait_limit, 200)) {
    record_error(p.s.err, kErrTimeout);
    return false;
  }
  bars->sched_t[slot] = t;
  mbar_arrive(smem_addr(&bars->sched_full[slot]));
  return true;
}

// The work tiles of a CTA, one after the other (one thread). Split: whole waves, then
// the CTA's share of the rest. Else the CTA starts with work tile blockIdx.x and claims
// every further one from the counter that the planning kernel zeroed.
struct TileSource {
  const PagedFwdParams& p;
  int total, grid, cta;
  int lo_tile = 0, hi_tile = -1, seq = 0;  // work tiles of the last sequence looked up
  int item = -1;                           // the last tile (claimed), or wave (split)
  int u = 0, end = 0, x = -1;              // split: units left of the share, and their tile

  __device__ explicit TileSource(const PagedFwdParams& params) : p(params) {
    total = p.tile_start[p.s.B];
    grid = gridDim.x;
    cta = blockIdx.x;
  }
  __device__ void expand(int tile, PagedTile& t) {
    if (tile < kFwdListed) {
      int4* w = reinterpret_cast<int4*>(&t);
#pragma unroll
      for (int i = 0; i < 3; ++i) w[i] = p.tiles[3 * tile + i];
      return;
    }
    if (tile < lo_tile || tile >= hi_tile) {
      const int v = find_last(p.tile_start, p.s.B, tile);
      seq = p.seq_order[v];
      lo_tile = p.tile_start[v];
      hi_tile = p.tile_start[v + 1];
    }
    const SeqSpan sp = new_span(p.s, seq);
    expand_tile(p, tile - lo_tile, seq, sp.start, sp.len, kv_len(p.s, seq), t);
  }
  __device__ bool near_end() const {
    constexpr int kNearRounds = 4;
    return !p.split && item + kNearRounds * static_cast<long long>(grid) >= total;
  }
  // t.b < 0 behind the last one
  __device__ void next(PagedTile& t) {
    if (!p.split) {
      if (item < 0) {
        item = cta;
      } else {
        const unsigned c = atomicAdd(reinterpret_cast<unsigned*>(p.tile_ctr), 1u);
        item = c >= static_cast<unsigned>(total)
                   ? total
                   : static_cast<int>(min(static_cast<unsigned>(total), static_cast<unsigned>(grid) + c));
      }
      if (item < total) expand(item, t); else t.b = -1;
      return;
    }
    const int waves = total / grid;
    if (item + 1 < waves) {
      ++item;
      expand(item * grid + cta, t);
      return;
    }
    if (x < 0) {
      const int4 share = p.shares[cta];  // first unit, end, tile of the first unit
      u = share.x;
      end = share.y;
      x = share.z;
    }
    while (u < end) {
      const int first = p.rest_units[x], after = p.rest_units[x + 1], stop = min(end, after);
      const int k0 = max(0, u - first - kItemCost), k1 = max(0, stop - first - kItemCost);
      const bool empty = after - first == kItemCost;  // a tile that sees no key
      const bool mine = k0 < k1 || (empty && u == first), part = !empty && (k0 > 0 || stop < after);
      u = stop;
      ++x;
      if (!mine) continue;
      expand(waves * grid + x - 1, t);
      if (part) {
        t.slot = 2 * cta + (k0 == 0 ? 1 : 0);
        t.kt0 = k0;
        for (int i = 0; i < 2; ++i) t.n[i] = max(0, min(t.n[i], k1) - k0);
      }
      return;
    }
    t.b = -1;
  }
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(384, 1)
paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const PagedFwdParams p) {
  using Cfg = PagedFwdCfg<D, E4M3>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  PagedBars* bars = reinterpret_cast<PagedBars*>(smem + Cfg::kBarOff);
  static_assert(sizeof(PagedBars) <= 1024, "barrier block");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(smem_addr(&bars->q_full), 1);
    mbar_init(smem_addr(&bars->q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars->s_full[i]), 1);
      mbar_init(smem_addr(&bars->p_full[i]), 128);
      mbar_init(smem_addr(&bars->pv_done[i]), 1);
    }
    for (int i = 0; i < Cfg::kStages; ++i) {
      mbar_init(smem_addr(&bars->kv_full[i]), 1 + E4M3);  // the copies, or two warps
      mbar_init(smem_addr(&bars->kv_empty[i]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_addr(&bars->sched_full[i]), 1);
      mbar_init(smem_addr(&bars->sched_empty[i]), kReaders + 2 * E4M3);
    }
    for (int i = 0; E4M3 && i < Cfg::kRawStages; ++i) {
      mbar_init(smem_addr(&bars->raw_full[i]), 1);
      mbar_init(smem_addr(&bars->raw_empty[i]), 1);
    }
    mbar_init(smem_addr(&bars->drained), 1);
    bars->sched_taken = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&bars->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const long long lim = p.wait_limit;
  grid_wait();

  // Register split: 128 x 88 (warps 0-3) + 256 x 208 (softmax) = 384 x 168.
  if (warp < 4) {
    regs_dec<88>();
    if (warp == 0) {
      // -------------------------------------------------------- TMA producer
      // Lane (page j of a key tile, column block) issues one box per tile.
      const int box_shift = min(p.s.page_shift, E4M3 ? 6 : 7);
      const int n_box = kTileN >> box_shift;
      constexpr int kCols = E4M3 ? 1 : Cfg::kBlocks;  // boxes side by side in a row
      const int j_box = lane / kCols, blk = lane % kCols;
      const int box_row = j_box << box_shift;
      const uint32_t dst0 = smem_addr(smem + Cfg::kKVOff) + blk * Cfg::kBlockBytes + box_row * 128;
      const uint32_t raw0 = smem_addr(smem + Cfg::kRawOff) + (box_row & (Cfg::kHalf - 1)) * D;
      const int q_bytes = p.tok_tile * p.group * 128;  // one column block of a Q tile
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      uint32_t ld = 0;  // K/V tiles (e4m3: half tiles) loaded so far
      int qk = 0;       // work tiles whose Q was loaded
      bool ok = true;
      PagedTile t;
      for (int k = 0; ok && take_tile(bars, k, t, lim, ok); ++k) {
        if (lane == 0) *reinterpret_cast<volatile int*>(&bars->sched_taken) = k + 1;
        const int n_kv = max(t.n[0], t.n[1]);
        if (n_kv == 0) continue;
        auto page_at = [&](int j) {
          const int key = (t.kt0 + j) * kTileN + box_row;
          return j < n_kv && j_box < n_box && key < t.len ? page_of(p.s, t.b, key >> p.s.page_shift) : 0;
        };
        int id = page_at(0);
        // Q goes in once the previous tile's last S MMA has read its buffer
        if (qk > 0 && !mbar_wait_warp(smem_addr(&bars->q_empty), (qk - 1) & 1, lim)) {
          ok = false;
          break;
        }
        ++qk;
        if (lane == 0) {
          const uint32_t qbar = smem_addr(&bars->q_full);
          mbar_arrive_expect_tx(qbar, ((t.n[0] > 0) + (t.n[1] > 0)) * Cfg::kBlocks * q_bytes);
          for (int i = 0; i < 2; ++i) {
            if (t.n[i] == 0) continue;
            for (int hf = 0; hf < Cfg::kBlocks; ++hf)
              tma_load_3d(smem_addr(smem) + i * Cfg::kTileBytes + hf * Cfg::kBlockBytes, &tm_q, qbar,
                          hf * 64, t.h * p.group, t.row0 + t.q0 + i * p.tok_tile);
          }
        }
        for (int j = 0; ok && j < n_kv; ++j) {
          const int here = id;
          id = page_at(j + 1);
          const int key0 = (t.kt0 + j) * kTileN;
          // boxes that hold a key; the rows of the others keep what they held
          const int boxes = min(n_box, (t.len - key0 + (1 << box_shift) - 1) >> box_shift);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const CUtensorMap* map = kv ? &tm_v : &tm_k;
            const int in_page = (key0 + box_row) & ((1 << p.s.page_shift) - 1);
            if constexpr (E4M3) {
              const int per = n_box >> 1;  // boxes of a half
#pragma unroll
              for (int half = 0; half < 2; ++half, ++ld) {
                const uint32_t stage = ld % Cfg::kRawStages, round = ld / Cfg::kRawStages;
                if (!mbar_wait_warp(smem_addr(&bars->raw_empty[stage]), (round & 1) ^ 1, lim)) { ok = false; break; }
                const uint32_t fbar = smem_addr(&bars->raw_full[stage]);
                if (lane == 0)
                  mbar_arrive_expect_tx(fbar, max(0, min(per, boxes - half * per)) * (D << box_shift));
                __syncwarp();
                if (j_box < boxes && j_box >= half * per && j_box < (half + 1) * per)
                  tma_load_4d(raw0 + stage * Cfg::kRawBytes, map, fbar, 0, in_page, t.h, here);
              }
              if (!ok) break;
            } else {
              const uint32_t stage = ld % Cfg::kStages, round = ld / Cfg::kStages;
              if (!mbar_wait_warp(smem_addr(&bars->kv_empty[stage]), (round & 1) ^ 1, lim)) { ok = false; break; }
              const uint32_t fbar = smem_addr(&bars->kv_full[stage]);
              if (lane == 0) mbar_arrive_expect_tx(fbar, boxes * Cfg::kBlocks * (128 << box_shift));
              __syncwarp();
              if (j_box < boxes)
                tma_load_4d(dst0 + stage * Cfg::kTileBytes, map, fbar, blk * 64, in_page, t.h, here);
              ++ld;
            }
          }
        }
      }
      if (!ok) {
        if (lane == 0) record_error(p.s.err, kErrTimeout);
        // no copy may still be on its way when the CTA's shared memory goes
        constexpr uint32_t kRing = E4M3 ? Cfg::kRawStages : Cfg::kStages;
        uint64_t* landed = E4M3 ? bars->raw_full : bars->kv_full;
        for (uint32_t n = ld > kRing ? ld - kRing : 0; n < ld; ++n)
          mbar_wait_warp(smem_addr(&landed[n % kRing]), (n / kRing) & 1, lim);
        if (qk > 0) mbar_wait_warp(smem_addr(&bars->q_full), (qk - 1) & 1, lim);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      const bool leader = elect_one_sync();
      constexpr uint32_t kIdS = E4M3 ? make_idesc_f16(128, 128, 0, 0) : make_idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t kIdPV = E4M3 ? make_idesc_f16(128, D, 0, 1) : make_idesc_bf16(128, D, 0, 1);
      const uint32_t kv_base = smem_addr(smem + Cfg::kKVOff);
      const uint64_t q_desc = make_sdesc_sw128(smem_addr(smem), 16, 1024);  // K-major
      const uint64_t k_desc = make_sdesc_sw128(kv_base, 16, 1024);          // K-major
      const uint64_t v_desc = make_sdesc_sw128(kv_base, Cfg::kBlockBytes, 1024);  // MN-major
      uint32_t ld = 0;  // K/V tiles consumed by earlier work tiles (K_j = 2 j, V_j = 2 j + 1)
      auto stage_of = [&](int it) { return (ld + it) % Cfg::kStages; };
      auto wait_full = [&](int it) {
        return mbar_wait_warp(smem_addr(&bars->kv_full[stage_of(it)]), ((ld + it) / Cfg::kStages) & 1, lim);
      };
      auto issue_s = [&](int i, int it) {
        const uint64_t qa = q_desc + ((i * Cfg::kTileBytes) >> 4);
        const uint64_t kb = k_desc + ((stage_of(it) * Cfg::kTileBytes) >> 4);
        const uint32_t d_tmem = tmem + Cfg::kColS + i * 128;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * Cfg::kBlockBytes + (kk & 3) * 32) >> 4;
          mma_ss_by(leader, d_tmem, qa + off, kb + off, kIdS, kk > 0);
        }
        mma_commit_by(leader, smem_addr(&bars->s_full[i]));
      };
      auto issue_pv = [&](int i, int it, bool acc) {
        const uint64_t vb = v_desc + ((stage_of(it) * Cfg::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < kTileN / 16; ++kk)
          mma_ts_by(leader, tmem + i * D, tmem + Cfg::kColS + i * 128 + kk * 8, vb + kk * (2048 >> 4), kIdPV,
                    (acc || kk > 0));
      };
      int pw[2] = {0, 0};  // p_full waits so far, per query tile
      int qk = 0;
      bool ok = true;
      PagedTile t;
      for (int k = 0; ok && take_tile(bars, k, t, lim, ok); ++k) {
        const int n_kv = max(t.n[0], t.n[1]);
        if (n_kv == 0) continue;  // no keys: the epilogue writes O = 0, LSE = -inf
        ok = mbar_wait_warp(smem_addr(&bars->q_full), qk & 1, lim);
        ++qk;
        if (ok) ok = wait_full(0);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (t.n[i] > 0) issue_s(i, 0);
        mma_commit_by(leader, smem_addr(&bars->kv_empty[stage_of(0)]));
        if (n_kv == 1) mma_commit_by(leader, smem_addr(&bars->q_empty));
        for (int j = 0; j < n_kv; ++j) {
          const int itv = 2 * j + 1, itk = 2 * j + 2;
          const bool next_k = j + 1 < n_kv;
          if (!(ok = wait_full(itv))) break;
          const int live = t.len - (t.kt0 + j) * kTileN;  // rows of V_j that are keys
          if (!E4M3 && live < kTileN) {
            const uint32_t vs = kv_base + stage_of(itv) * Cfg::kTileBytes;
            for (int x = lane; x < (kTileN - live) * 8 * Cfg::kBlocks; x += 32) {
              const int blk = x / ((kTileN - live) * 8), y = x - blk * (kTileN - live) * 8;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                               vs + blk * Cfg::kBlockBytes + live * 128 + y * 16),
                           "r"(0) : "memory");
            }
            fence_async_shared();
            __syncwarp();
          }
          if (next_k && !(ok = wait_full(itk))) break;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (j >= t.n[i]) continue;
            if (!mbar_wait_warp(smem_addr(&bars->p_full[i]), pw[i] & 1, lim)) { ok = false; break; }
            tc_fence_after();
            issue_pv(i, itv, j > 0);
            ++pw[i];
            // only the last PV of a tile is signalled (to the epilogue); earlier
            // ones are covered by the commit of the S MMA issued after them
            if (j + 1 == t.n[i]) mma_commit_by(leader, smem_addr(&bars->pv_done[i]));
            else issue_s(i, itk);
          }
          if (!ok) break;
          mma_commit_by(leader, smem_addr(&bars->kv_empty[stage_of(itv)]));
          if (next_k) mma_commit_by(leader, smem_addr(&bars->kv_empty[stage_of(itk)]));
          if (j + 2 == n_kv) mma_commit_by(leader, smem_addr(&bars->q_empty));
        }
        ld += 2 * n_kv;
      }
      if (!ok) {
        if (leader) record_error(p.s.err, kErrTimeout);
        // nor may a product be when its memory goes
        mma_commit_by(leader, smem_addr(&bars->drained));
        mbar_wait_warp(smem_addr(&bars->drained), 0, lim);
      }
    } else if (!E4M3 && warp == 2 && lane == 0) {
      // -------------------------------------------------------- scheduler
      // Near the end of a claimed list a tile is claimed only once the producer has
      // taken the one before, so no CTA holds tiles that an idle one could run.
      TileSource source(p);
      for (int k = 0;; ++k) {
        PagedTile t;
        source.next(t);
        if (!publish_tile(bars, k, t, p)) break;
        if (t.b < 0) break;
        if (source.near_end()) {
          bool taken = *reinterpret_cast<volatile int*>(&bars->sched_taken) > k;
          const long long t0 = clock64();
          while (!taken && clock64() - t0 <= lim) {
            __nanosleep(100);
            taken = *reinterpret_cast<volatile int*>(&bars->sched_taken) > k;
          }
          if (!taken) {  // the other roles' bounded waits end the CTA
            record_error(p.s.err, kErrTimeout);
            break;
          }
        }
      }
    } else if (E4M3 && warp >= 2) {
      // -------------------------------------------------------- widening (e4m3)
      // Warp 2 the first, warp 3 the second half of every tile, a row per lane; both
      // rings are swizzled, so neither side's accesses meet in a bank. Lane 0 of
      // warp 2 publishes the next work tile when it takes one.
      const int half = warp - 2;
      const uint32_t raw0 = smem_addr(smem + Cfg::kRawOff), kv0 = smem_addr(smem + Cfg::kKVOff);
      uint32_t ld = 0;  // tiles widened so far
      bool ok = true;
      TileSource source(p);
      PagedTile t;
      if (half == 0 && lane == 0) {
        source.next(t);
        publish_tile(bars, 0, t, p);
      }
      __syncwarp();
      for (int k = 0; ok && take_tile(bars, k, t, lim, ok); ++k) {
        if (half == 0 && lane == 0) {
          PagedTile next;
          source.next(next);
          publish_tile(bars, k + 1, next, p);
        }
        __syncwarp();
        const int n_kv = max(t.n[0], t.n[1]);
        for (int it = 0; it < 2 * n_kv; ++it, ++ld) {
          const uint32_t rs = (2 * ld + half) % Cfg::kRawStages, rr = (2 * ld + half) / Cfg::kRawStages;
          const uint32_t ks = ld % Cfg::kStages, kr = ld / Cfg::kStages;
          if (!mbar_wait_warp(smem_addr(&bars->raw_full[rs]), rr & 1, lim) ||
              !mbar_wait_warp(smem_addr(&bars->kv_empty[ks]), (kr & 1) ^ 1, lim)) {
            ok = false;
            break;
          }
          // rows of V past the end become zeros
          const int live = (it & 1) ? t.len - (t.kt0 + (it >> 1)) * kTileN : kTileN;
          const uint32_t src = raw0 + rs * Cfg::kRawBytes, dst = kv0 + ks * Cfg::kTileBytes;
#pragma unroll 1
          for (int in = lane; in < Cfg::kHalf; in += 32) {
            const int row = half * Cfg::kHalf + in;
            const uint32_t from = src + in * D;
            const int sw = D == 128 ? row & 7 : (row >> 1) & 3;
            const bool keep = row < live;
            // all loads of the row first: one latency for them
            uint32_t w[D / 16][4];
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[c][0]), "=r"(w[c][1]), "=r"(w[c][2]), "=r"(w[c][3])
                           : "r"(from + ((c ^ sw) << 4)));
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t to = dst + (c >> 2) * Cfg::kBlockBytes;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t a = keep ? w[c][2 * h] : 0u, b = keep ? w[c][2 * h + 1] : 0u;
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 to + sw128_offset(row, 2 * (c & 3) + h)),
                             "r"(e4m3x2_to_f16x2(a)), "r"(e4m3x2_to_f16x2(a >> 16)), "r"(e4m3x2_to_f16x2(b)),
                             "r"(e4m3x2_to_f16x2(b >> 16)));
              }
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&bars->kv_full[ks]));
            mbar_arrive(smem_addr(&bars->raw_empty[rs]));
          }
        }
      }
      if (!ok && lane == 0) record_error(p.s.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    regs_inc<208>();
    // ---------------------------------------------------------- softmax + epilogue
    const int i = (warp - 4) >> 2;      // query tile of this warpgroup
    const int r = tid - 128 * (1 + i);  // row of the tile == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(r & ~31) << 16;
    const uint32_t col_s = Cfg::kColS + i * 128, col_o = i * D;
    const int tok_r = r / p.group, head_r = r - tok_r * p.group;
    int sw = 0, pvw = 0;  // s_full and pv_done waits so far
    constexpr float lift = E4M3 ? kLift : 0.0f;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      PagedTile t;
      if (!take_tile(bars, k, t, lim, ok)) break;
      const int my_n = i ? t.n[1] : t.n[0];
      const int q0 = t.q0 + i * p.tok_tile;           // first token of this query tile
      const int see0 = t.len - t.n_new + q0;          // the last key that it sees (causal)
      const int tok = q0 + tok_r;
      // keys that this row sees: one comparison per score covers both masks
      const int see = p.causal ? min(t.len, see0 + tok_r + 1) : t.len;
      float c = p.scale_log2;
      if constexpr (E4M3) c *= p.k_scale ? __ldg(p.k_scale + t.h) : 1.0f;
      // the same in every lane: softmax_row_max votes within either branch
      const bool pos = c > 0.0f;
      if constexpr (E4M3) {
        if (tok_r < p.tok_tile && tok < t.n_new)
          c *= p.q_up[(static_cast<size_t>(t.row0) + tok) * p.H_q + t.h * p.group + head_r];
        // A row of tiny queries can bring c to 0, and -inf of a masked score times 0 is NaN:
        // the smallest normal number in its place moves no score by more than 2^-108.
        if (pos) c = fmaxf(c, 1.17549435e-38f);
      }
      // Rows of the tile that are no query row of this sequence (what an earlier call left
      // behind the last whole token, the next sequence's rows) have no part in the warp's
      // votes: a bias of +inf never moves, and their P is 0 or NaN in their own rows of O,
      // which are not written.
      float m_used = tok_r < p.tok_tile && tok < t.n_new ? -INFINITY : INFINITY, l = 0.0f;
      for (int j = 0; j < my_n; ++j) {
        if (!mbar_wait_warp(smem_addr(&bars->s_full[i]), sw & 1, lim)) { ok = false; break; }
        ++sw;
        tc_fence_after();
        float s[128];
        uint32_t* sr = reinterpret_cast<uint32_t*>(s);
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          tmem_ld32(tmem + lane_base + col_s + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(sr + cc * 32));
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(sr + cc * 32));
        const int kv0 = (t.kt0 + j) * kTileN;
        const bool need_mask = kv0 + kTileN > t.len || (p.causal && kv0 + kTileN - 1 > see0);
        uint32_t pk[64];
        bool rescale_warp;
        float factor;
        const float mb = pos ? softmax_row_max<true>(s, c, m_used, l, kv0, 0, see, need_mask, 0,
                                                     rescale_warp, factor)
                             : softmax_row_max<false>(s, c, m_used, l, kv0, 0, see, need_mask, 0,
                                                      rescale_warp, factor);
        uint64_t sum2[2] = {0ull, 0ull};
        if (pos) softmax_row_exp<0, true, 0, 64, E4M3>(s, c, mb - lift, need_mask, pk, sum2);
        else softmax_row_exp<0, false, 0, 64, E4M3>(s, c, mb - lift, need_mask, pk, sum2);
        if (rescale_warp && j > 0 && __any_sync(0xffffffffu, factor != 1.0f)) {
          // O is complete: the commit that signalled S_j came after PV_{j-1}
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_base + col_o + cc * 32, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * factor);
            tmem_st32(tmem + lane_base + col_o + cc * 32, ov);
          }
        }
        tmem_st32(tmem + lane_base + col_s, *reinterpret_cast<uint32_t(*)[32]>(pk));
        tmem_st32(tmem + lane_base + col_s + 32, *reinterpret_cast<uint32_t(*)[32]>(pk + 32));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_addr(&bars->p_full[i]));
        l += softmax_row_sum(sum2);
      }
      if (!ok) break;
      // -------------------------------------------------------- epilogue
      // The O columns are reused by the next tile's first PV MMA, which waits
      // for this warpgroup's next p_full arrival, i.e. after these loads.
      if (q0 >= t.n_new) continue;
      if (my_n > 0) {
        if (!mbar_wait_warp(smem_addr(&bars->pv_done[i]), pvw & 1, lim) ||
            (p.fault == kFaultLeaveWarp && (warp & 3) == 1)) {
          ok = false;
          break;
        }
        ++pvw;
        tc_fence_after();
      }
      const bool row_ok = tok_r < p.tok_tile && tok < t.n_new;
      const int hq = t.h * p.group + head_r;
      uint32_t ov[D];
      if (my_n > 0) {
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc)
          tmem_ld32(tmem + lane_base + col_o + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(ov + cc * 32));
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(ov + cc * 32));
      } else {
#pragma unroll
        for (int e = 0; e < D; ++e) ov[e] = 0u;
      }
      const float v_scale = E4M3 && p.v_scale ? __ldg(p.v_scale + t.h) : 1.0f;
      uint32_t buf_off = Cfg::kEpiOff + i * Cfg::kBlockBytes;
      asm volatile("" : "+r"(buf_off));  // computed here, not kept across the key loop
      uint8_t* buf = smem + buf_off;
      const int rows = min(p.tok_tile, t.n_new - q0) * p.group;
      if (t.slot >= 0) {
        // A piece: maxima, sums and O as they are. O passes through the warp's part of the
        // staging block, 32 columns at a time, so that the stores are whole lines: straight
        // from the registers, 16 bytes of a row each, they cost 4 us more where 128 tiles are
        // cut (d 128).
        const size_t slot = (static_cast<size_t>(t.slot) * 2 + i) * kTileM;
        if (row_ok) *reinterpret_cast<float2*>(p.part_ml + (slot + r) * 2) = make_float2(m_used - lift, l);
        if (my_n > 0) {
          const int row0 = r & ~31;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
#pragma unroll
            for (int ch = 0; ch < 8; ++ch) {
              float f[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(ov[c0 + 4 * ch + e]) * v_scale;
              *reinterpret_cast<float4*>(buf + sw128_offset(r, ch)) = make_float4(f[0], f[1], f[2], f[3]);
            }
            __syncwarp();
#pragma unroll
            for (int x = lane; x < 256; x += 32) {
              const int rr = row0 + (x >> 3);
              if (rr < rows)
                *reinterpret_cast<float4*>(p.part_o + (slot + rr) * D + c0 + (x & 7) * 4) =
                    *reinterpret_cast<const float4*>(buf + sw128_offset(rr, x & 7));
            }
            __syncwarp();
          }
        }
        continue;
      }
      // a row with a NaN score has l = NaN and keeps it
      const float inv_l = l == 0.0f ? 0.0f : v_scale / l;
      const size_t row = static_cast<size_t>(t.row0) + tok;
      // O leaves through the warp's part of the staging block, 64 columns at a time, in
      // 128-byte runs: a row's place in o comes from the lane that holds it. The warps of a
      // tile do not wait for one another anywhere, so that one whose wait runs out leaves
      // alone. (A TMA store of whole tiles, with two barriers of the four warps for each 64
      // columns and waits made thread by thread, took as long over 8 prompts, 236 us, and
      // 49.4 us instead of 50.4 over 16 prompts with heads of 64.)
      const uint32_t to = row_ok ? static_cast<uint32_t>(row * p.H_q + hq) : 0xffffffffu;
#pragma unroll
      for (int hf = 0; hf < Cfg::kBlocks; ++hf) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16x2(__uint_as_float(ov[hf * 64 + 8 * ch + 2 * e]) * inv_l,
                               __uint_as_float(ov[hf * 64 + 8 * ch + 2 * e + 1]) * inv_l);
          *reinterpret_cast<uint4*>(buf + sw128_offset(r, ch)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int in = x * 4 + (lane >> 3);
          const uint32_t at = __shfl_sync(0xffffffffu, to, in);
          if (at != 0xffffffffu)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + static_cast<size_t>(at) * D + hf * 64 +
                                      (lane & 7) * 8) =
                *reinterpret_cast<const uint4*>(buf + sw128_offset((r & ~31) + in, lane & 7));
        }
        __syncwarp();
      }
      if (row_ok)
        p.lse[static_cast<size_t>(hq) * p.s.T + row] = l == 0.0f ? -INFINITY : (m_used - lift) * kLn2 + logf(l);
    }
    if (!ok) record_error(p.s.err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Orders the sequences by their keys, longest first (ties in input order), and
// numbers their work tiles; zeroes the claim counter. One CTA. Offsets that make
// more work items than the host made room for (they overlap) leave no work.
constexpr int kPlanThreads = 640;
static_assert(kFwdListed <= kPlanThreads && kPlanThreads <= 1024, "one thread per listed tile");
__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const PagedFwdParams p, int sort) {
  extern __shared__ int plan_smem[];
  // when sorting: keys, first rows, rows and order of the sequences [B] and the first
  // tiles [B]; otherwise they are looked up where they are needed
  int* key = plan_smem;
  int* row0 = key + p.s.B;
  int* rows = row0 + p.s.B;
  int* ord = rows + p.s.B;
  int* start = sort ? ord + p.s.B : p.tile_start;
  __shared__ long long warp_sum[33];
  __shared__ int unit[kFwdListed];
  __shared__ int rest_units[kFwdSms + 1], rest_start[kFwdSms + 1];
  __shared__ int longest;  // CTA's units when the rest's tiles stay whole
  if (threadIdx.x == 0) longest = 0;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, B = p.s.B;
  grid_wait();
  grid_release();
  if (tid == 0) *p.tile_ctr = 0;
  check_paged_seqs(p.s, tid, blockDim.x);  // (its loads are those that follow)
  // the sum of x over the threads before this one, and over all
  auto scan = [&](auto x, auto& all) {
    auto in = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[w] = in;
    __syncthreads();
    auto sum = static_cast<decltype(x)>(lane < kPlanThreads / 32 ? warp_sum[lane] : 0);
    const auto own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const auto y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    all = __shfl_sync(0xffffffffu, sum, 31);
    return __shfl_sync(0xffffffffu, sum - own, w) + in - x;
  };
  if (sort) {
    for (int b = tid; b < B; b += blockDim.x) {
      key[b] = kv_len(p.s, b);
      const SeqSpan sp = new_span(p.s, b);
      row0[b] = sp.start;
      rows[b] = sp.len;
    }
    __syncthreads();
    for (int b = tid; b < B; b += blockDim.x) {
      const int mine = key[b];
      int rank = 0;
      for (int u = 0; u < B; ++u) rank += key[u] > mine || (key[u] == mine && u < b);
      ord[rank] = b;
    }
    __syncthreads();
  }
  const int run = (B + blockDim.x - 1) / blockDim.x;
  const int v0 = min(B, tid * run), v1 = min(B, v0 + run);
  auto tiles_of = [&](int v) {
    return static_cast<long long>(m_blocks(p, sort ? rows[ord[v]] : new_span(p.s, v).len)) * p.H_kv;
  };
  long long mine = 0, all;
  for (int v = v0; v < v1; ++v) mine += tiles_of(v);
  long long at = scan(mine, all);
  const bool fits = all <= p.max_work;
  const int total = fits ? static_cast<int>(all) : 0;
  for (int v = v0; v < v1; ++v) {
    const int first = fits ? static_cast<int>(at) : 0;
    p.seq_order[v] = sort ? ord[v] : v;
    p.tile_start[v] = first;
    start[v] = first;
    at += tiles_of(v);
  }
  if (tid == 0) {
    p.tile_start[B] = total;
    if (!fits) record_error(p.s.err, kErrSeqlens);
  }
  __syncthreads();
  // the first tiles of the list, so that the CTAs need not look them up
  if (tid < min(total, kFwdListed)) {
    const int v = find_last(start, B, tid);
    PagedTile t;
    t.pad[0] = t.pad[1] = 0;
    if (sort) {
      const int b = ord[v];
      expand_tile(p, tid - start[v], b, row0[b], rows[b], key[b], t);
    } else {
      const SeqSpan sp = new_span(p.s, v);
      expand_tile(p, tid - start[v], v, sp.start, sp.len, kv_len(p.s, v), t);
    }
    const int4* words = reinterpret_cast<const int4*>(&t);
    const int first_rest = p.split ? total / p.grid * p.grid : total;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      p.tiles[3 * tid + i] = words[i];
      if (tid >= first_rest) p.rest_tiles[3 * (tid - first_rest) + i] = words[i];
    }
    unit[tid] = tile_units(t);
  }
  if (!p.split) return;
  // Few work tiles: the units of every CTA's whole tiles, of each tile of the rest,
  // and the shares of the rest that even the CTAs out.
  __syncthreads();
  const int grid = p.grid, waves = total / grid, rest = total - waves * grid;
  int rest_all;  // (less than 152 tiles of 2^23 units)
  const int first = scan(tid < rest ? unit[waves * grid + tid] : 0, rest_all);
  if (tid <= rest) {
    rest_units[tid] = tid < rest ? first : rest_all;
    p.rest_units[tid] = rest_units[tid];
  }
  long long whole = 0, whole_all = 0, share_all;
  if (waves > 0) {
    if (tid < grid)
      for (int i = 0; i < waves; ++i) whole += unit[i * grid + tid];
    scan(whole, whole_all);
  }
  // Kept whole, tile x of the rest goes to CTA grid - rest + x (the last ones' whole
  // tiles are the shortest).
  const int spare = grid - rest;
  if (tid >= spare && tid < grid) atomicMax(&longest, static_cast<int>(whole) + unit[waves * grid + tid - spare]);
  // Cut, pieces of less than six units cost more than they spread: the last `wide`
  // CTAs share the rest, each at least a tile's worth.
  const int wide = max(rest, min(grid, rest_all / 6));
  const long long level = waves > 0 ? (whole_all + rest_all) / grid : 0;
  // Leaving and joining the pieces takes as long as about three units, and one more for
  // every 16 tiles of the rest (d 128; 32 for 64): below that the tiles stay whole. 1000
  // new tokens of one prompt, 32 heads on 8, 128 tiles: whole 24.9 us, cut 34.4; 1500 of 8
  // heads of 64, 48 tiles: 25.6 and 23.0.
  const long long even = waves > 0 ? level : wide > 0 ? rest_all / wide : 0;
  __syncthreads();
  if (longest <= even + 3 + (rest * p.d >> 11)) {
    if (tid < grid) {
      const int x = tid - spare;
      p.shares[tid] = x >= 0 ? make_int4(rest_units[x], rest_units[x + 1], x, 0) : make_int4(0, 0, 0, 0);
      p.rest_owners[tid] = make_int2(0, 0);
    }
    return;
  }
  const long long share = tid >= grid || tid < grid - wide ? 0
                          : waves == 0 || wide < grid      ? 1
                                                           : max(0ll, level - whole);
  const long long before = scan(share, share_all);
  // (without room below the mean the last CTA takes the rest)
  if (tid <= grid)
    rest_start[tid] = tid == grid ? rest_all : share_all > 0 ? static_cast<int>(rest_all * before / share_all) : 0;
  __syncthreads();
  // three searches, by different threads
  const int part = tid / kFwdSms, c = tid - part * kFwdSms;
  if (c >= grid) return;
  if (part == 0) {
    const int u = rest_start[c], end = rest_start[c + 1];
    p.shares[c] = make_int4(u, end, u < end ? find_last(rest_units, rest, u) : 0, 0);
  } else if (part < 3) {
    // the CTAs that hold the first and the last unit of tile c's keys
    const int begin = c < rest ? rest_units[c] + kItemCost : 0, end = c < rest ? rest_units[c + 1] : 0;
    reinterpret_cast<int*>(p.rest_owners)[2 * c + part - 1] =
        begin < end ? find_last(rest_start, grid, part == 1 ? begin : end - 1) : 0;
  }
}

// Merges the pieces of the rest's split work tiles in order. CTA (x, y): rows 16 y ..
// 16 y + 15 of tile x of the rest, two at once for each warp. Latency is what it costs,
// so all loads of four pieces are on their way together: of 3 sequences of 198 new tokens behind
// 15000 keys (5 heads on 1, d 64), a call takes 31 us, with one load after the other 43.
// Where 128 tiles are cut (d 128), one row at a time costs 2 us more, and four, which
// leave one CTA on an SM, 12.
constexpr int kJoinRows = 16;
template <int D>
__global__ void __launch_bounds__(256)
paged_fwd_join_kernel(const PagedFwdParams p) {
  grid_wait();
  const int2 own = p.rest_owners[blockIdx.x];  // the CTAs that hold its first and its last key tile
  PagedTile t;
  {
    int4* words = reinterpret_cast<int4*>(&t);
#pragma unroll
    for (int i = 0; i < 3; ++i) words[i] = p.rest_tiles[3 * blockIdx.x + i];
  }
  if (own.x == own.y) return;  // written whole, or no tile
  const int c0 = own.x, c1 = own.y;
  const int lane = threadIdx.x & 31;
  constexpr int kV = D / 32, kRows = kJoinRows / 8, kAtOnce = 4;
  const int row0 = blockIdx.y * kJoinRows + (threadIdx.x >> 5) * kRows;
  const int i = row0 >> 7, r0 = row0 & 127;
  // rows of this query tile
  const int rows = max(0, min(p.tok_tile, t.n_new - t.q0 - i * p.tok_tile)) * p.group;
  if (r0 >= rows) return;
  auto slot_row = [&](int c, int n) {
    return (static_cast<size_t>(2 * c + (c == c0 ? 1 : 0)) * 2 + i) * kTileM + min(r0 + n, rows - 1);
  };
  float acc[kRows][kV], m[kRows], l[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    m[n] = -INFINITY;
    l[n] = 0.0f;
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[n][e] = 0.0f;
  }
  // Four pieces at a time, all loads before the first is used (the last piece again
  // behind it, with no weight). A share can be empty, and a piece whose keys a row does
  // not see left no O.
  for (int base = c0; base <= c1; base += kAtOnce) {
    float o[kAtOnce][kRows][kV];
    float2 ml[kAtOnce][kRows];
    bool some[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int c = min(base + k, c1);
      const int4 share = p.shares[c];
      some[k] = base + k <= c1 && share.x != share.y;
#pragma unroll
      for (int n = 0; n < kRows; ++n) {
        const size_t at = slot_row(c, n);
        ml[k][n] = *reinterpret_cast<const float2*>(p.part_ml + at * 2);
        const float* src = p.part_o + at * D + lane * kV;
#pragma unroll
        for (int e = 0; e < kV; ++e) o[k][n][e] = src[e];
      }
    }
#pragma unroll
    for (int n = 0; n < kRows; ++n) {
      float top = m[n];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (some[k]) top = fmaxf(top, ml[k][n].x);
      const float bias = top == -INFINITY ? 0.0f : top, f = ex2_approx(m[n] - bias);
      m[n] = top;
      l[n] *= f;
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[n][e] *= f;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        if (!some[k] || ml[k][n].y == 0.0f) continue;
        const float g = ex2_approx(ml[k][n].x - bias);
        l[n] += ml[k][n].y * g;
#pragma unroll
        for (int e = 0; e < kV; ++e) acc[n][e] += o[k][n][e] * g;
      }
    }
  }
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    const int r = r0 + n;
    if (r >= rows) break;
    const float inv = l[n] == 0.0f ? 0.0f : 1.0f / l[n];
    const int tok_r = r / p.group;
    const size_t to = static_cast<size_t>(t.row0) + t.q0 + i * p.tok_tile + tok_r;
    const int head = t.h * p.group + r - tok_r * p.group;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + (to * p.H_q + head) * D + lane * kV);
#pragma unroll
    for (int e = 0; e < kV / 2; ++e) out[e] = pack_bf16x2(acc[n][2 * e] * inv, acc[n][2 * e + 1] * inv);
    if (lane == 0)
      p.lse[static_cast<size_t>(head) * p.s.T + to] = l[n] == 0.0f ? -INFINITY : m[n] * kLn2 + logf(l[n]);
  }
}

// One warp per row of queries.
template <int D>
__global__ void __launch_bounds__(256)
queries_f16_kernel(const uint2* q, uint2* q16, float* q_up, long long rows) {
  grid_wait();
  grid_release();
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const bool mine = lane < D / 4;
  uint2 x = mine ? q[row * (D / 4) + lane] : make_uint2(0u, 0u);
  const float v[4] = {bf16lo_to_f32(x.x), bf16hi_to_f32(x.x), bf16lo_to_f32(x.y), bf16hi_to_f32(x.y)};
  float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float down;
  const float up = row_power(top, down);
  if (mine)
    q16[row * (D / 4) + lane] = make_uint2(pack_f16x2(v[0] * down, v[1] * down), pack_f16x2(v[2] * down, v[3] * down));
  if (lane == 0) q_up[row] = up;
}

template <int D, bool E4M3>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const PagedFwdParams& p, cudaStream_t stream) {
  // sorting compares every pair of sequences and keeps them in shared memory
  const int sort = p.s.B <= 1024;
  int slot = prof_begin(kKPagedPlan, stream);
  cudaError_t e = launch_chained<paged_plan_kernel>(dim3(1), kPlanThreads,
                                 sort ? 5 * p.s.B * static_cast<int>(sizeof(int)) : 0, stream, p, sort);
  prof_end(slot, stream);
  if (e != cudaSuccess) return e;
  slot = prof_begin(kKPagedFwd, stream);
  e = launch_chained<paged_fwd_kernel<D, E4M3>>(dim3(p.grid), 384, PagedFwdCfg<D, E4M3>::kSmemBytes, stream, tq, tk,
                     tv, p);
  prof_end(slot, stream);
  if (e != cudaSuccess || !p.split) return e;
  slot = prof_begin(kKPagedJoin, stream);
  e = launch_chained<paged_fwd_join_kernel<D>>(dim3(min(p.grid, p.max_work), 2 * kTileM / kJoinRows), 256, 0, stream, p);
  prof_end(slot, stream);
  return e;
}

}  // namespace

cudaError_t launch_paged_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedFwdParams& p, int d, bool e4m3, cudaStream_t stream) {
  if (e4m3) return d == 128 ? launch<128, true>(tq, tk, tv, p, stream) : launch<64, true>(tq, tk, tv, p, stream);
  return d == 128 ? launch<128, false>(tq, tk, tv, p, stream) : launch<64, false>(tq, tk, tv, p, stream);
}

cudaError_t launch_queries_f16(const void* q, void* q16, float* q_up, long long rows, int d,
                               cudaStream_t stream) {
  const int slot = prof_begin(kKPagedQueries, stream);
  const dim3 grid(static_cast<unsigned>((rows + 7) / 8));
  const uint2* from = static_cast<const uint2*>(q);
  uint2* to = static_cast<uint2*>(q16);
  const cudaError_t e = d == 128 ? launch_chained<queries_f16_kernel<128>>(grid, 256, 0, stream, from, to, q_up, rows)
                                 : launch_chained<queries_f16_kernel<64>>(grid, 256, 0, stream, from, to, q_up, rows);
  prof_end(slot, stream);
  return e;
}

}  // namespace attn
