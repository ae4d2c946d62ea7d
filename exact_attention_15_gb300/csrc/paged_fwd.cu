// Attention of chunks of new tokens over a paged key-value cache on the tensor
// cores (whole prompts, the next chunk of a prompt).
//
// The query rows of a sequence that share a KV head form the tiles: row r of a
// 128-row tile is token r / group, head r % group of the KV head, so a tile
// covers floor(128 / group) tokens and every key that it loads meets all the
// heads that use it. A work tile is two such tiles in a row; the CTA that owns it
// streams the keys and values that they see, 128 at a time, from the pages.
// Roles, TMEM plan and pipeline are those of the packed forward kernel:
//   warp 0      TMA producer: both Q tiles, then K_j / V_j into a ring; the lanes
//               look up the pages of a tile and issue one box each.
//   warp 1      TMEM owner and MMA issuer: S_i = Q_i K_j^T, O_i += P_i V_j.
//   warp 2      claims work tiles from a counter (longest sequences first) and
//               hands them to the other roles.
//   warps 4-11  softmax and epilogue, one warpgroup per query tile.
// Rows of V past the sequence's end can hold anything, and 0 x NaN is NaN: the
// MMA warp zeroes them in shared memory before the last P V product.
//
// With fewer work tiles than SMs the keys of a tile are cut into `splits` pieces
// of equal length that different CTAs take; each leaves its (m, l, O) in the
// workspace and paged_fwd_join_kernel merges them in order.
//
// TMEM (512 columns): O_0 [0, d), O_1 [d, 2d), S_0/P_0 [2d, 2d + 128), S_1/P_1
// [2d + 128, 2d + 256).
#include "fwd_softmax.cuh"
#include "paged.cuh"

namespace attn {

namespace {

template <int D>
struct PagedFwdCfg {
  static constexpr int kBlocks = D / 64;                // 64-column blocks of a tile
  static constexpr int kBlockBytes = kTileM * 64 * 2;   // 16 KB
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kKVOff = 2 * kTileBytes;
  static constexpr int kBarOff = kKVOff + kStages * kTileBytes;
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
  int item;        // work item, for the partial results
  int pad[2];
};

constexpr int kSlots = 2;     // of the ring that hands out work tiles
constexpr int kReaders = 10;  // producer warp, MMA warp, eight softmax warps

struct PagedBars {
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t sched_full[kSlots], sched_empty[kSlots];
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
// The key tiles of piece `s` of a work tile: [first, first + count) of its `all`.
__device__ __forceinline__ int piece_start(int all, int s, int splits) {
  return static_cast<int>(static_cast<long long>(all) * s / splits);
}

// Work item w = (tile, piece); the tiles of a sequence run from its last block
// of tokens (which sees most keys) to its first, the KV heads innermost.
__device__ __forceinline__ void expand_item(const PagedFwdParams& p, int item, int b, int tile0,
                                            PagedTile& t) {
  const int tile = item / p.splits, piece = item - tile * p.splits;
  const SeqSpan sp = new_span(p.s, b);
  t.b = b;
  t.row0 = sp.start;
  t.n_new = sp.len;
  t.len = kv_len(p.s, b);
  const int local = tile - tile0;
  const int mi = local / p.H_kv;
  t.h = local - mi * p.H_kv;
  t.q0 = (m_blocks(p, sp.len) - 1 - mi) * 2 * p.tok_tile;
  int n[2];
  for (int i = 0; i < 2; ++i)
    n[i] = (keys_seen(p, t.q0 + i * p.tok_tile, t.n_new, t.len) + kTileN - 1) / kTileN;
  const int all = max(n[0], n[1]);
  t.kt0 = piece_start(all, piece, p.splits);
  const int end = piece_start(all, piece + 1, p.splits);
  for (int i = 0; i < 2; ++i) t.n[i] = max(0, min(n[i], end) - t.kt0);
  t.item = item;
}

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

template <int D>
__global__ void __launch_bounds__(384, 1)
paged_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                 const PagedFwdParams p) {
  using Cfg = PagedFwdCfg<D>;
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
      mbar_init(smem_addr(&bars->kv_full[i]), 1);
      mbar_init(smem_addr(&bars->kv_empty[i]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_addr(&bars->sched_full[i]), 1);
      mbar_init(smem_addr(&bars->sched_empty[i]), kReaders);
    }
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
  grid_release();

  // Register split: 128 x 88 (warps 0-3) + 256 x 208 (softmax) = 384 x 168.
  if (warp < 4) {
    regs_dec<88>();
    if (warp == 0) {
      // -------------------------------------------------------- TMA producer
      // Lane (page j of a key tile, column block) issues one box per tile.
      const int box_shift = min(p.s.page_shift, 7);
      const int n_box = kTileN >> box_shift;
      const int j_box = lane / Cfg::kBlocks, blk = lane % Cfg::kBlocks;
      const int box_row = j_box << box_shift;
      const uint32_t dst0 = smem_addr(smem + Cfg::kKVOff) + blk * Cfg::kBlockBytes + box_row * 128;
      const int q_bytes = p.tok_tile * p.group * 128;  // one column block of a Q tile
      if (lane == 0) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
      }
      uint32_t ld = 0;  // K/V tiles loaded so far
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
          for (int kv = 0; kv < 2; ++kv, ++ld) {
            const uint32_t stage = ld % Cfg::kStages, round = ld / Cfg::kStages;
            if (!mbar_wait_warp(smem_addr(&bars->kv_empty[stage]), (round & 1) ^ 1, lim)) {
              ok = false;
              break;
            }
            const uint32_t fbar = smem_addr(&bars->kv_full[stage]);
            if (lane == 0) mbar_arrive_expect_tx(fbar, boxes * Cfg::kBlocks * (128 << box_shift));
            __syncwarp();
            if (j_box < boxes)
              tma_load_4d(dst0 + stage * Cfg::kTileBytes, kv ? &tm_v : &tm_k, fbar, blk * 64,
                          (key0 + box_row) & ((1 << p.s.page_shift) - 1), t.h, here);
          }
        }
      }
      if (!ok && lane == 0) record_error(p.s.err, kErrTimeout);
    } else if (warp == 1) {
      // -------------------------------------------------------- MMA issuer
      const bool leader = elect_one_sync();
      constexpr uint32_t kIdS = make_idesc_bf16(128, 128, 0, 0);
      constexpr uint32_t kIdPV = make_idesc_bf16(128, D, 0, 1);
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
          if (live < kTileN) {
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
      if (!ok && leader) record_error(p.s.err, kErrTimeout);
    } else if (warp == 2 && lane == 0) {
      // -------------------------------------------------------- scheduler
      // The CTA starts with work item blockIdx.x and claims every further one
      // from the counter that the planning kernel zeroed. Near the end of the
      // list an item is claimed only once the producer has taken the one before,
      // so no CTA holds items that an idle one could run.
      const int total = p.tile_start[p.s.B] * p.splits;
      constexpr int kNearRounds = 4;
      int lo_item = 0, hi_item = -1, seq = 0, tile0 = 0;  // items of the last sequence found
      int item = blockIdx.x;
      for (int k = 0;; ++k) {
        PagedTile t;
        if (item < total) {
          if (item < lo_item || item >= hi_item) {
            const int tile = item / p.splits;
            int lo = 0, hi = p.s.B;  // the last sequence whose first tile is <= tile
            while (hi - lo > 1) {
              const int mid = (lo + hi) >> 1;
              if (p.tile_start[mid] <= tile) lo = mid; else hi = mid;
            }
            seq = p.seq_order[lo];
            tile0 = p.tile_start[lo];
            lo_item = tile0 * p.splits;
            hi_item = p.tile_start[lo + 1] * p.splits;
          }
          expand_item(p, item, seq, tile0, t);
        } else {
          t = PagedTile{};
          t.b = -1;
        }
        const int slot = k % kSlots;
        if (k >= kSlots &&
            !mbar_wait_sleep(smem_addr(&bars->sched_empty[slot]), ((k / kSlots) - 1) & 1, lim, 200)) {
          record_error(p.s.err, kErrTimeout);
          break;
        }
        bars->sched_t[slot] = t;
        mbar_arrive(smem_addr(&bars->sched_full[slot]));
        if (t.b < 0) break;
        if (item + kNearRounds * static_cast<long long>(gridDim.x) >= total) {
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
        const unsigned c = atomicAdd(reinterpret_cast<unsigned*>(p.tile_ctr), 1u);
        item = c >= static_cast<unsigned>(total) ? total : static_cast<int>(min(
                   static_cast<unsigned>(total), gridDim.x + c));
      }
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
    const float c = p.scale_log2;
    int sw = 0, pvw = 0;  // s_full and pv_done waits so far
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
      float m_used = -INFINITY, l = 0.0f;
      for (int j = 0; j < my_n; ++j) {
        if (!mbar_wait(smem_addr(&bars->s_full[i]), sw & 1, lim)) { ok = false; break; }
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
        const bool pos = c > 0.0f;
        const float mb = pos ? softmax_row_max<true>(s, c, m_used, l, kv0, 0, see, need_mask, 0,
                                                     rescale_warp, factor)
                             : softmax_row_max<false>(s, c, m_used, l, kv0, 0, see, need_mask, 0,
                                                      rescale_warp, factor);
        uint64_t sum2[2] = {0ull, 0ull};
        if (pos) softmax_row_exp<0, true, 0, 64>(s, c, mb, need_mask, pk, sum2);
        else softmax_row_exp<0, false, 0, 64>(s, c, mb, need_mask, pk, sum2);
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
        if (!mbar_wait(smem_addr(&bars->pv_done[i]), pvw & 1, lim)) { ok = false; break; }
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
      if (p.splits > 1) {
        const size_t slot = (static_cast<size_t>(t.item) * 2 + i) * kTileM + r;
        if (row_ok) {
          *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(m_used, l);
          if (my_n > 0) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + slot * D);
#pragma unroll
            for (int e = 0; e < D / 4; ++e)
              dst[e] = make_uint4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
          }
        }
        continue;
      }
      // a row with a NaN score has l = NaN and keeps it
      const float inv_l = l == 0.0f ? 0.0f : 1.0f / l;
      const size_t row = static_cast<size_t>(t.row0) + tok;
      // O leaves through shared memory, 64 columns at a time: by one TMA store of
      // whole rows where the tile ends inside the sequence, else (the store's box
      // would reach into the next sequence) by 128-byte runs of the rows it has
      const bool box = q0 + p.tok_tile <= t.n_new;
      const int rows = min(p.tok_tile, t.n_new - q0) * p.group;
      uint32_t buf_off = Cfg::kEpiOff + i * Cfg::kBlockBytes;
      asm volatile("" : "+r"(buf_off));  // computed here, not kept across the key loop
      uint8_t* buf = smem + buf_off;
#pragma unroll
      for (int hf = 0; hf < Cfg::kBlocks; ++hf) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          w[e] = pack_bf16x2(__uint_as_float(ov[hf * 64 + 2 * e]) * inv_l,
                             __uint_as_float(ov[hf * 64 + 2 * e + 1]) * inv_l);
        if (r == 0) bulk_wait_group_read<0>();
        named_bar_sync(2 + i, 128);
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
          *reinterpret_cast<uint4*>(buf + sw128_offset(r, ch)) =
              make_uint4(w[4 * ch], w[4 * ch + 1], w[4 * ch + 2], w[4 * ch + 3]);
        if (box) fence_async_shared();
        named_bar_sync(2 + i, 128);
        if (box) {
          if (r == 0) {
            tma_store_3d(&tm_o, smem_addr(buf), hf * 64, t.h * p.group, t.row0 + q0);
            bulk_commit_group();
          }
        } else {
          for (int x = r; x < rows * 8; x += 128) {
            const int rr = x >> 3, tk = rr / p.group;
            const size_t at = (static_cast<size_t>(t.row0 + q0 + tk) * p.H_q + t.h * p.group + rr - tk * p.group) * D;
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + at + hf * 64 + (x & 7) * 8) =
                *reinterpret_cast<const uint4*>(buf + sw128_offset(rr, x & 7));
          }
        }
      }
      if (row_ok)
        p.lse[static_cast<size_t>(hq) * p.s.T + row] = l == 0.0f ? -INFINITY : m_used * kLn2 + logf(l);
    }
    // the O stores have read the staging buffer before the CTA's shared memory goes
    if (r == 0) bulk_wait_group<0>();
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
__global__ void __launch_bounds__(1024)
paged_plan_kernel(const PagedFwdParams p, int sort) {
  extern __shared__ int plan_smem[];
  int* key = plan_smem;          // [B] when sorting
  int* ord = plan_smem + p.s.B;  // [B] when sorting
  __shared__ long long warp_sum[33];
  const int tid = threadIdx.x, B = p.s.B;
  grid_wait();
  grid_release();
  if (tid == 0) *p.tile_ctr = 0;
  check_paged_seqs(p.s, tid, blockDim.x);
  if (sort) {
    for (int b = tid; b < B; b += blockDim.x) key[b] = kv_len(p.s, b);
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
    return static_cast<long long>(m_blocks(p, new_span(p.s, sort ? ord[v] : v).len)) * p.H_kv;
  };
  long long mine = 0;
  for (int v = v0; v < v1; ++v) mine += tiles_of(v);
  const int lane = tid & 31, w = tid >> 5;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[w] = incl;
  __syncthreads();
  if (w == 0) {
    long long x = warp_sum[lane];
    const long long own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    warp_sum[lane] = x - own;
    if (lane == 31) warp_sum[32] = x;
  }
  __syncthreads();
  const bool fits = warp_sum[32] * p.splits <= p.max_work;
  long long at = warp_sum[w] + incl - mine;
  for (int v = v0; v < v1; ++v) {
    const int b = sort ? ord[v] : v;
    p.seq_order[v] = b;
    p.tile_start[v] = fits ? static_cast<int>(at) : 0;
    p.seq_tile[b] = fits ? static_cast<int>(at) : 0;
    at += tiles_of(v);
  }
  if (tid == 0) {
    p.tile_start[B] = fits ? static_cast<int>(warp_sum[32]) : 0;
    if (!fits) record_error(p.s.err, kErrSeqlens);
  }
}

// One warp per query row and head: merges the pieces of its work tile in order.
template <int D>
__global__ void __launch_bounds__(128)
paged_fwd_join_kernel(const PagedFwdParams p) {
  grid_wait();
  grid_release();
  const long long at = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (at >= static_cast<long long>(p.s.T) * p.H_q || p.tile_start[p.s.B] == 0) return;
  const int t = static_cast<int>(at / p.H_q), head = static_cast<int>(at - static_cast<long long>(t) * p.H_q);
  int lo = 0, hi = p.s.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.s.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
  }
  const SeqSpan sp = new_span(p.s, lo);
  if (t < sp.start || t >= sp.start + sp.len) return;
  const int tok = t - sp.start, h = head / p.group;
  const int mb = tok / (2 * p.tok_tile), in = tok - mb * 2 * p.tok_tile;
  const int i = in >= p.tok_tile;
  const int r = (in - i * p.tok_tile) * p.group + head - h * p.group;
  const long long tile = p.seq_tile[lo] + static_cast<long long>(m_blocks(p, sp.len) - 1 - mb) * p.H_kv + h;
  auto slot = [&](int s) { return ((tile * p.splits + s) * 2 + i) * kTileM + r; };
  float top = -INFINITY;
  for (int s = 0; s < p.splits; ++s) top = fmaxf(top, p.part_ml[slot(s) * 2]);
  const float mbias = top == -INFINITY ? 0.0f : top;
  constexpr int kV = D / 32;
  float acc[kV], l = 0.0f;
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] = 0.0f;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + slot(s) * 2);
    if (ml.y == 0.0f) continue;  // a piece without keys left no O
    const float f = ex2_approx(ml.x - mbias);
    l += ml.y * f;
    const float* src = p.part_o + slot(s) * D + lane * kV;
#pragma unroll
    for (int e = 0; e < kV; ++e) acc[e] += src[e] * f;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) +
                                              (static_cast<size_t>(t) * p.H_q + head) * D + lane * kV);
#pragma unroll
  for (int e = 0; e < kV / 2; ++e) out[e] = pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  if (lane == 0)
    p.lse[static_cast<size_t>(head) * p.s.T + t] = l == 0.0f ? -INFINITY : top * kLn2 + logf(l);
}

template <int D>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CUtensorMap& to, const PagedFwdParams& p, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  // sorting compares every pair of sequences and keeps them in shared memory
  const int sort = p.s.B <= 1024;
  int slot = prof_begin(kKPagedPlan, stream);
  cudaError_t e = launch_chained(paged_plan_kernel, dim3(1), 1024,
                                 sort ? 2 * p.s.B * static_cast<int>(sizeof(int)) : 0, stream, smem_set, p, sort);
  prof_end(slot, stream);
  if (e != cudaSuccess) return e;
  slot = prof_begin(kKPagedFwd, stream);
  e = launch_chained(paged_fwd_kernel<D>, dim3(p.grid), 384, PagedFwdCfg<D>::kSmemBytes, stream, smem_set, tq, tk,
                     tv, to, p);
  prof_end(slot, stream);
  if (e != cudaSuccess || p.splits == 1) return e;
  slot = prof_begin(kKPagedJoin, stream);
  const long long rows = static_cast<long long>(p.s.T) * p.H_q;
  e = launch_chained(paged_fwd_join_kernel<D>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, stream,
                     smem_set, p);
  prof_end(slot, stream);
  return e;
}

}  // namespace

cudaError_t launch_paged_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const CUtensorMap& to, const PagedFwdParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch<128>(tq, tk, tv, to, p, stream) : launch<64>(tq, tk, tv, to, p, stream);
}

}  // namespace attn
