// Choosing the pages that a query token attends to by bounds of their keys.
//
// The bounds of a page and KV head are the elementwise minimum lo and maximum hi of its keys, so
// that no key k of the page has a product with q above
//   bound(q) = sum_i max(q_i, 0) hi_i + min(q_i, 0) lo_i.
// paged_bounds_kernel keeps them up, paged_select_kernel takes for each token and KV head the
// pages with the largest bounds (over the query heads of the KV head).
#include <type_traits>

#include "paged.cuh"

namespace attn {

namespace {

// ---------------------------------------------------------------- bounds
// A CTA for each touched page and KV head, four rows or more at a time: thread (row, 16-byte
// column) keeps the minimum and maximum of its column's elements, packed as the cache's values
// are (bf16, or e4m3 widened to fp16, both exact), NaN before anything else. Every byte of
// the pages is read once; they bound it.
constexpr int kBoundsThreads = 128;

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b, bool f16) {
  uint32_t r;
  if (f16) asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b, bool f16) {
  uint32_t r;
  if (f16) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D, int KIND>
__global__ void __launch_bounds__(kBoundsThreads)
paged_bounds_kernel(const BoundsParams p) {
  constexpr bool F16 = KIND != kBf16;
  constexpr int kRowChunks = D * (F16 ? 1 : 2) / 16;   // 16-byte pieces of a row
  constexpr int kRows = kBoundsThreads / kRowChunks;   // rows at a time
  constexpr int kWords = F16 ? 8 : 4;                  // packed pairs of a piece
  constexpr int kWarpLanes = kRowChunks < 32 ? 32 / kRowChunks : 1;  // lanes of a warp with the same column
  __shared__ uint32_t part[kBoundsThreads / 32][2][kRowChunks][kWords];
  const PagedSeqs& s = p.s;
  grid_wait();
  grid_release();
  if (blockIdx.x == 0) check_paged_seqs(s, threadIdx.x, kBoundsThreads);
  const int h = static_cast<int>(blockIdx.x % p.H_kv);
  TouchedPage x;
  if (!touched_page(s, blockIdx.x / p.H_kv, x)) return;
  const int id = __ldg(s.page_table + static_cast<size_t>(x.b) * s.table_stride + x.at);
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(s.num_pages)) {
    if (threadIdx.x == 0) record_error(s.err, kErrPages);
    return;
  }
  const int rows = min(1 << s.page_shift, x.len - (x.at << s.page_shift));
  const int col = threadIdx.x % kRowChunks, row0 = threadIdx.x / kRowChunks;
  const uint4* keys = reinterpret_cast<const uint4*>(
      static_cast<const uint8_t*>(p.k) +
      (static_cast<long long>(id) * p.k_page + (static_cast<long long>(h) << s.page_shift) * D) * (F16 ? 1 : 2));
  constexpr uint32_t kPlusInf = F16 ? 0x7c007c00u : 0x7f807f80u, kMinusInf = kPlusInf | 0x80008000u;
  uint32_t lo[kWords], hi[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) { lo[i] = kPlusInf; hi[i] = kMinusInf; }
#pragma unroll 8
  for (int r = row0; r < rows; r += kRows) {
    const uint4 v = keys[r * kRowChunks + col];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t y = F16 ? e4m3x2_to_f16x2(w[(i / 2) & 3] >> (16 * (i & 1))) : w[i & 3];
      lo[i] = min2(lo[i], y, F16);
      hi[i] = max2(hi[i], y, F16);
    }
  }
  // lanes with the same column lie kRowChunks apart
#pragma unroll
  for (int i = 0; i < kWords; ++i)
#pragma unroll
    for (int o = kRowChunks; o < kRowChunks * kWarpLanes; o <<= 1) {
      lo[i] = min2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o), F16);
      hi[i] = max2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o), F16);
    }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane < kRowChunks) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      part[warp][0][col][i] = lo[i];
      part[warp][1][col][i] = hi[i];
    }
  }
  __syncthreads();
  // thread: a pair of columns of the minimum or of the maximum
  if (threadIdx.x >= D) return;
  const int side = threadIdx.x / (D / 2), at = threadIdx.x % (D / 2);
  uint32_t y = part[0][side][at / kWords][at % kWords];
#pragma unroll
  for (int w = 1; w < kBoundsThreads / 32; ++w) {
    const uint32_t z = part[w][side][at / kWords][at % kWords];
    y = side ? max2(y, z, F16) : min2(y, z, F16);
  }
  int to = side;
  if constexpr (F16) {
    float scale = 1.0f;
    if constexpr (KIND == kE4m3Pages) scale = power_of_two(page_exponent(p.k_exp, id, p.H_kv, h));
    else if (p.k_scale) scale = __ldg(p.k_scale + h);
    const float2 f = f16x2_to_f32(y);
    y = pack_bf16x2(f.x * scale, f.y * scale);
    if (scale < 0.0f) to = 1 - side;  // turns the order round
  }
  reinterpret_cast<uint32_t*>(p.bounds)[((static_cast<size_t>(id) * p.H_kv + h) * 2 + to) * (D / 2) + at] = y;
}

// ---------------------------------------------------------------- selection
// One cluster of 1 to 8 CTAs for each token and KV head; each takes a run of the pages.
//
// 1. Bounds as products on mma.sync m16n8k16: 16 pages in M, the heads of the group in N,
//    (lo, hi) and (min(q, 0), max(q, 0)) side by side in K. A lane's fragment of A is 16 bytes of
//    a page's bounds at a time (the order of K does not matter as long as B has the same), so
//    they go from memory to the registers, each byte once: the bytes bound this part.
// 2. A histogram of the scores over their range finds the interval that the last chosen
//    score lies in.
// 3. The products are exact, their sums are not: with eps a bound on the sums' error, pages
//    more than 2 eps above the interval are chosen for certain, pages more than 2 eps below it are
//    not, and the few between are scored again in 64 bits, where ties go to the lower page. So
//    the choice is that of 64-bit scores, whatever the order of the sums.
// 4. The chosen pages are written in their order.
constexpr int kSelThreads = 256, kSelWarps = kSelThreads / 32, kBins = 2048;
// Up to this many pages to be ranked in 64 bits are compared pair by pair, more by digits:
// 256 threads of a CTA compare 512 with 512 in the time of about two of the ten digits.
constexpr int kPairs = 512;
// Error of a sum relative to the sum of the magnitudes: 2 d / 16 = 16 instructions, each of which
// adds 17 terms, each to 2^-23 of the largest at least, is below 2^-14.9.
constexpr float kSumError = 6.103515625e-05f;  // 2^-14
// Sums below this stay finite, so that no score is an infinity or a NaN; above its inverse, what
// products below the normal numbers lose (256 times 2^-126 at most) is less than the bound.
constexpr float kLargest = 1.2676506e30f;  // 2^100

// An order of floats as unsigned numbers; NaN above all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ unsigned long long ordered(double x) {
  if (x != x) return ~0ull;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));  // (-0 as 0)
  return b ^ (static_cast<unsigned long long>(static_cast<long long>(b) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) { return static_cast<uint32_t>(ld_cluster_s32(addr)); }
__device__ __forceinline__ unsigned long long ld_cluster_u64(uint32_t addr) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What a CTA shows the others of its cluster.
struct SelectShared {
  uint32_t hist[kBins];
  uint32_t l1, k_most;       // largest sum of a query row's magnitudes; largest magnitude of the bounds
  uint32_t least, most;      // scores, ordered
  uint32_t sure, unsure, chosen;
  uint32_t bin, above;       // the bin that was looked for, and what lies above it
  uint32_t warp_sum[kSelWarps];
};

// Finds the bin from the top that holds the k-th of the clusters' numbers (k >= 1 and at most as
// many as there are): sh.bin, and how many lie above it, sh.above. kPer bins a thread.
template <int kPer>
__device__ __forceinline__ void find_bin(SelectShared& sh, int cluster, uint32_t k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t v[kPer];
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = 0;
  const uint32_t at = smem_addr(sh.hist + tid * kPer);
  for (int r = 0; r < cluster; ++r) {
    const uint32_t from = cluster_map(at, r);
    if constexpr (kPer == 8) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        uint32_t w[4];
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from + 4 * i) : "memory");
#pragma unroll
        for (int u = 0; u < 4; ++u) v[i + u] += w[u];
      }
    } else {
      v[0] += ld_cluster_u32(from);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine += v[i];
  // the sum over the threads from this one on
  uint32_t from_here = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_down_sync(0xffffffffu, from_here, o);
    if (lane + o < 32) from_here += y;
  }
  if (lane == 0) sh.warp_sum[warp] = from_here;
  __syncthreads();
  for (int w = warp + 1; w < kSelWarps; ++w) from_here += sh.warp_sum[w];
  uint32_t above = from_here - mine;
  if (above < k && k <= from_here) {
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) {
      if (above < k && k <= above + v[i]) {
        sh.bin = tid * kPer + i;
        sh.above = above;
        above = 0xffffffffu;  // found
      } else if (above != 0xffffffffu) {
        above += v[i];
      }
    }
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kSelThreads, 2)
paged_select_kernel(const SelectParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SelectShared sh;
  constexpr int kQStride = 4 * D + 64;  // bytes of a query row (the gap spreads rows over the banks)
  const PagedSeqs& s = p.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = 1 << p.cluster_shift, rank = blockIdx.x & (cluster - 1);
  const long long item = blockIdx.x >> p.cluster_shift;
  const int t = static_cast<int>(item / p.H_kv), h = static_cast<int>(item % p.H_kv);
  const int q_tiles = (p.group + 7) / 8;
  uint8_t* qs = smem;
  unsigned long long* list_key = reinterpret_cast<unsigned long long*>(smem + q_tiles * 8 * kQStride);
  float* score = reinterpret_cast<float*>(list_key + p.slice);
  uint32_t* list = reinterpret_cast<uint32_t*>(score + p.slice);
  auto sync = [&]() {
    if (cluster > 1) cluster_sync_all(); else __syncthreads();
  };
  auto total = [&](const uint32_t& x) {
    uint32_t sum = 0;
    for (int r = 0; r < cluster; ++r) sum += ld_cluster_u32(cluster_map(smem_addr(&x), r));
    return sum;
  };
  grid_wait();
  grid_release();
  if (blockIdx.x == 0) check_paged_seqs(s, tid, kSelThreads);

  // ---- the token's sequence and what it sees
  int b = t;
  SeqSpan span{t, 1};
  if (s.cu_seqlens) {
    int lo = 0, hi = s.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(s.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
    }
    b = lo;
    span = seq_span(s.cu_seqlens, b, s.T, 0);
    if (t < span.start || t >= span.start + span.len) return;  // behind the last sequence
  }
  const int len = max(0, kv_len(s, b) - span.len + (t - span.start) + 1);
  const int pages = (len + (1 << s.page_shift) - 1) >> s.page_shift;
  int* out = p.pages + item * p.count;
  if (h == 0 && rank == 0 && tid == 0)
    p.lens[t] = len - (max(0, pages - p.count) << s.page_shift);
  if (pages <= p.count) {  // all of them
    for (int i = rank * kSelThreads + tid; i < p.count; i += cluster * kSelThreads)
      out[i] = i < pages ? page_of(s, b, i) : -1;
    return;
  }
  const int room = p.count - p.first - p.last;  // pages to choose
  const int n_all = pages - p.first - p.last;   // pages to choose from
  if (rank == 0) {
    for (int i = tid; i < p.first; i += kSelThreads) out[i] = page_of(s, b, i);
    for (int i = tid; i < p.last; i += kSelThreads) out[p.count - p.last + i] = page_of(s, b, pages - p.last + i);
  }
  if (room == 0) return;
  const int per = ((n_all + cluster - 1) / cluster + 15) & ~15;
  const int begin = min(n_all, rank * per), n = min(n_all, begin + per) - begin;

  // ---- queries: a warp for each row
  if (tid == 0) {
    sh.l1 = sh.k_most = 0;
    sh.least = 0xffffffffu;
    sh.most = 0;
    sh.sure = sh.unsure = sh.chosen = 0;
  }
  for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
  __syncthreads();
  for (int r = warp; r < q_tiles * 8; r += kSelWarps) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.q) +
                                                            ((static_cast<size_t>(t) * p.H_q + h * p.group + r) * D) * 2);
    uint32_t* dst = reinterpret_cast<uint32_t*>(qs + r * kQStride);
    float sum = 0.0f;
#pragma unroll
    for (int i = lane; i < D / 2; i += 32) {
      const uint32_t w = r < p.group ? src[i] : 0u;
      sum += fabsf(bf16lo_to_f32(w)) + fabsf(bf16hi_to_f32(w));
      dst[i] = min2(w, 0u, false);
      dst[D / 2 + i] = max2(w, 0u, false);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) atomicMax(&sh.l1, __float_as_uint(sum) & 0x7fffffffu);
  }
  __syncthreads();

  // ---- scores of 16 pages a warp
  const int qd = lane & 3, ar = lane >> 2;
  constexpr int kSteps = 2 * D / 32;  // 16-byte pieces of a lane in a row
  const uint4* bounds = static_cast<const uint4*>(p.bounds);
  uint32_t k_most = 0;
  float least = INFINITY, most = -INFINITY;
  for (int tile = warp; tile * 16 < n; tile += kSelWarps) {
    const int i0 = tile * 16 + ar;
    uint4 a[2][kSteps];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int id = page_of(s, b, p.first + begin + min(i0 + 8 * u, n - 1));
      const uint4* src = bounds + (static_cast<size_t>(id) * p.H_kv + h) * (2 * D / 8) + qd;
#pragma unroll
      for (int c = 0; c < kSteps; ++c) a[u][c] = __ldg(src + 4 * c);
    }
    float best[2] = {-INFINITY, -INFINITY};
    for (int nt = 0; nt < q_tiles; ++nt) {
      const uint8_t* rows = qs + (nt * 8 + ar) * kQStride + qd * 16;
      float acc[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][e] = 0.0f;
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const uint4 w = *reinterpret_cast<const uint4*>(rows + c * 64);
        mma_bf16(acc[0], a[0][c].x, a[1][c].x, a[0][c].y, a[1][c].y, w.x, w.y);
        mma_bf16(acc[1], a[0][c].z, a[1][c].z, a[0][c].w, a[1][c].w, w.z, w.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (nt * 8 + 2 * qd + (e & 1) < p.group) best[e >> 1] = fmaxf(best[e >> 1], acc[0][e] + acc[1][e]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        const uint32_t x = __vmaxu2(a[u][c].x & 0x7fff7fffu, a[u][c].y & 0x7fff7fffu);
        const uint32_t y = __vmaxu2(a[u][c].z & 0x7fff7fffu, a[u][c].w & 0x7fff7fffu);
        k_most = __vmaxu2(k_most, __vmaxu2(x, y));
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      best[u] = fmaxf(best[u], __shfl_xor_sync(0xffffffffu, best[u], 1));
      best[u] = fmaxf(best[u], __shfl_xor_sync(0xffffffffu, best[u], 2));
      const int i = i0 + 8 * u;
      if (i < n) {
        if (qd == 0) score[i] = best[u];
        least = fminf(least, best[u]);
        most = fmaxf(most, best[u]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    k_most = __vmaxu2(k_most, __shfl_xor_sync(0xffffffffu, k_most, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if (lane == 0) {
    atomicMax(&sh.k_most, max(k_most & 0xffffu, k_most >> 16) << 16);
    atomicMin(&sh.least, ordered(least));
    atomicMax(&sh.most, ordered(most));
  }
  sync();

  // ---- the interval [lo, hi] of the last score to be chosen
  uint32_t k_bits = 0, lo_bits = 0xffffffffu, hi_bits = 0;
  for (int r = 0; r < cluster; ++r) {
    k_bits = max(k_bits, ld_cluster_u32(cluster_map(smem_addr(&sh.k_most), r)));
    lo_bits = min(lo_bits, ld_cluster_u32(cluster_map(smem_addr(&sh.least), r)));
    hi_bits = max(hi_bits, ld_cluster_u32(cluster_map(smem_addr(&sh.most), r)));
  }
  const float size = __uint_as_float(sh.l1) * __uint_as_float(k_bits);  // of the products' sums at most
  // every product is zero; else sums outside these bounds are taken in 64 bits alone
  const bool zero = sh.l1 == 0 || k_bits == 0;
  const bool finite = zero || (size < kLargest && size > 1.0f / kLargest);
  const float eps = size * kSumError;
  float lo = unordered(lo_bits), hi = unordered(hi_bits);
  const float range = hi - lo;
  if (finite && range > eps) {
    // (bins by the same rounded expression for every page, so their order is that of the scores)
    const float low = lo, inv = kBins / range;
    auto bin_of = [&](float x) { return min(kBins - 1, static_cast<int>((x - low) * inv)); };
    for (int i = tid; i < n; i += kSelThreads) atomicAdd(&sh.hist[bin_of(score[i])], 1u);
    sync();
    find_bin<kBins / kSelThreads>(sh, cluster, room);
    const int bin = sh.bin;
    uint32_t above = sh.above;
    lo = low + bin * (range / kBins);
    hi = low + (bin + 1) * (range / kBins);
    // a bin far wider than eps (a few scores far from the rest): its own pages again
    if (range > 64.0f * kBins * eps) {
      const float low2 = lo, inv2 = kBins / (range / kBins);
      auto bin2_of = [&](float x) { return max(0, min(kBins - 1, static_cast<int>((x - low2) * inv2))); };
      sync();
      for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads)
        if (bin_of(score[i]) == bin) atomicAdd(&sh.hist[bin2_of(score[i])], 1u);
      sync();
      find_bin<kBins / kSelThreads>(sh, cluster, room - above);
      const float w2 = range / kBins / kBins;
      lo = low2 + sh.bin * w2;
      hi = low2 + (sh.bin + 1) * w2;
    }
  }
  // (twice the bound; the bins' and the ends' own rounding is below eps / 2 and 2^-19 of the range)
  const float margin = 2.5f * eps + range * 1.9073486e-06f;
  const float low_cut = lo - margin, high_cut = hi + margin;

  // ---- pages chosen for certain, and those to be scored again
  for (int i0 = warp * 32; i0 < n; i0 += kSelThreads) {
    const int i = i0 + lane;
    const float x = i < n ? score[i] : -INFINITY;
    const bool sure = finite && i < n && x > high_cut, unsure = i < n && !sure && !(finite && x < low_cut);
    const uint32_t a = __ballot_sync(0xffffffffu, sure), u = __ballot_sync(0xffffffffu, unsure);
    uint32_t at = 0;
    if (lane == 0) {
      if (a) atomicAdd(&sh.sure, __popc(a));
      if (u) at = atomicAdd(&sh.unsure, __popc(u));
    }
    at = __shfl_sync(0xffffffffu, at, 0);
    if (unsure) list[at + __popc(u & ((1u << lane) - 1))] = i;
  }
  sync();
  const uint32_t n_unsure = total(sh.unsure), need = room - total(sh.sure);
  const int mine = sh.unsure;
  if (n_unsure == need) {
    for (int e = tid; e < mine; e += kSelThreads) score[list[e]] = INFINITY;
    if (tid == 0) sh.chosen = mine;
  } else {
    for (int e = warp; e < mine; e += kSelWarps) {
      unsigned long long key = 0;
      if (zero) {
        key = ordered(0.0);
      } else {
        const int id = page_of(s, b, p.first + begin + list[e]);
        const uint32_t* src = static_cast<const uint32_t*>(p.bounds) + (static_cast<size_t>(id) * p.H_kv + h) * D;
        for (int r = 0; r < p.group; ++r) {
          const uint32_t* q = reinterpret_cast<const uint32_t*>(qs + r * kQStride);
          double sum = 0.0;
#pragma unroll
          for (int i = lane; i < D; i += 32) {  // pairs of (lo, hi)
            const uint32_t x = q[i], y = __ldg(src + i);
            sum = fma(static_cast<double>(bf16lo_to_f32(x)), static_cast<double>(bf16lo_to_f32(y)), sum);
            sum = fma(static_cast<double>(bf16hi_to_f32(x)), static_cast<double>(bf16hi_to_f32(y)), sum);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          key = max(key, ordered(sum));
        }
      }
      if (lane == 0) list_key[e] = key;
    }
    sync();
    if (n_unsure <= kPairs) {
      for (int e = tid; e < mine; e += kSelThreads) {
        const unsigned long long key = list_key[e];
        const int place = begin + list[e];
        uint32_t better = 0;
        for (int r = 0; r < cluster; ++r) {
          const uint32_t theirs = ld_cluster_u32(cluster_map(smem_addr(&sh.unsure), r));
          const uint32_t keys = cluster_map(smem_addr(list_key), r), places = cluster_map(smem_addr(list), r);
#pragma unroll 4
          for (uint32_t i = 0; i < theirs; ++i) {
            const unsigned long long other = ld_cluster_u64(keys + 8 * i);
            better += other > key || (other == key && static_cast<int>(ld_cluster_u32(places + 4 * i)) + r * per < place);
          }
        }
        if (better < need) atomicAdd(&sh.chosen, 1u);
        // (the list's scores are not read by others)
        score[list[e]] = better < need ? INFINITY : -INFINITY;
      }
    } else {
      // By digits of 8 bits from the top: eight of the score, two of the place (lower ones first).
      unsigned long long key = 0;
      uint32_t place = 0, left = need;
      auto place_of = [&](int e) { return 0xffffu - (begin + list[e]); };
      for (int digit = 0; digit < 10; ++digit) {
        for (int i = tid; i < 256; i += kSelThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int e = tid; e < mine; e += kSelThreads) {
          const unsigned long long x = list_key[e];
          const uint32_t y = place_of(e);
          if (digit < 8) {
            if (digit == 0 || (x ^ key) >> (64 - 8 * digit) == 0) atomicAdd(&sh.hist[(x >> (56 - 8 * digit)) & 255], 1u);
          } else if (x == key && (digit == 8 || (y ^ place) >> 8 == 0)) {
            atomicAdd(&sh.hist[(y >> (8 * (9 - digit))) & 255], 1u);
          }
        }
        sync();
        find_bin<1>(sh, cluster, left);
        left -= sh.above;
        if (digit < 8) key |= static_cast<unsigned long long>(sh.bin) << (56 - 8 * digit);
        else place |= sh.bin << (8 * (9 - digit));
        sync();
      }
      for (int e = tid; e < mine; e += kSelThreads) {
        const unsigned long long x = list_key[e];
        const bool in = x > key || (x == key && place_of(e) >= place);
        if (in) atomicAdd(&sh.chosen, 1u);
        score[list[e]] = in ? INFINITY : -INFINITY;
      }
    }
  }
  sync();

  // ---- the chosen pages in their order: a run of them for each warp
  uint32_t at = p.first;
  for (int r = 0; r < rank; ++r)
    at += ld_cluster_u32(cluster_map(smem_addr(&sh.sure), r)) + ld_cluster_u32(cluster_map(smem_addr(&sh.chosen), r));
  const float cut = finite ? high_cut : 0.0f;
  const int run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
  uint32_t before = 0;
  for (int i = i0; i < i1; i += 32) before += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && score[i + lane] > cut));
  if (lane == 0) sh.warp_sum[warp] = before;
  __syncthreads();
  for (int w = 0; w < warp; ++w) at += sh.warp_sum[w];
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1 && score[i + lane] > cut;
    const uint32_t all = __ballot_sync(0xffffffffu, in);
    if (in) out[at + __popc(all & ((1u << lane) - 1))] = page_of(s, b, p.first + begin + i + lane);
    at += __popc(all);
  }
  if (cluster > 1) cluster_sync_all();  // no CTA leaves while another one reads its counts
}

template <int D>
cudaError_t launch_select(SelectParams p, int n_sm, cudaStream_t stream) {
  // More CTAs of a cluster while they find places at once (two on an SM) and each has a full
  // round of its warps.
  const long long items = static_cast<long long>(p.s.T) * p.H_kv;
  int cluster = 1;
  p.cluster_shift = 0;
  while (cluster < kSelectCluster &&
         (p.s.max_pages > kSelectSlice * cluster ||
          (items * 2 * cluster <= 2ll * n_sm && p.s.max_pages >= 2 * cluster * 16 * kSelWarps))) {
    cluster *= 2;
    ++p.cluster_shift;
  }
  p.slice = ((p.s.max_pages + cluster - 1) / cluster + 15) & ~15;
  if (items * cluster > 0x7fffffffll) return cudaErrorInvalidValue;
  const int smem = (p.group + 7) / 8 * 8 * (4 * D + 64) + p.slice * 16;
  const cudaError_t e = allow_smem<paged_select_kernel<D>>(kTileM * (4 * D + 64) + kSelectSlice * 16);
  if (e != cudaSuccess) return e;
  return launch_clusters<paged_select_kernel<D>>(cluster, dim3(static_cast<unsigned>(items * cluster)), kSelThreads, smem,
                                                 stream, p);
}

}  // namespace

cudaError_t launch_paged_bounds(const BoundsParams& p, int d, int kind, cudaStream_t stream) {
  const long long blocks = touched_numbers(p.s.T, p.s.B, p.s.page_shift, p.s.cu_seqlens != nullptr) * p.H_kv;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(blocks));
  const int slot = prof_begin(kKPagedBounds, stream);
  auto of_kind = [&](auto k) {
    constexpr int K = decltype(k)::value;
    return d == 128 ? launch_chained<paged_bounds_kernel<128, K>>(grid, kBoundsThreads, 0, stream, p)
                    : launch_chained<paged_bounds_kernel<64, K>>(grid, kBoundsThreads, 0, stream, p);
  };
  const cudaError_t e = kind == kBf16   ? of_kind(std::integral_constant<int, kBf16>{})
                        : kind == kE4m3 ? of_kind(std::integral_constant<int, kE4m3>{})
                                        : of_kind(std::integral_constant<int, kE4m3Pages>{});
  prof_end(slot, stream);
  return e;
}

cudaError_t launch_paged_select(const SelectParams& p, int d, int n_sm, cudaStream_t stream) {
  const int slot = prof_begin(kKPagedSelect, stream);
  const cudaError_t e = d == 128 ? launch_select<128>(p, n_sm, stream) : launch_select<64>(p, n_sm, stream);
  prof_end(slot, stream);
  return e;
}

}  // namespace attn
