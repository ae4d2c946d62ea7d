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
// A warp for each touched page and KV head, two rows or more at a time: lane (row, 16-byte
// column) keeps the minimum and maximum of its column's elements, packed as the cache's values
// are (bf16, or e4m3 widened to fp16, both exact), NaN before anything else. Every byte of
// the pages is read once; they bound it where there are many pages (40,000 tokens of 8 KV heads of 128 in
// pages of 32, bf16: 12.8 us, 73% of a copy's rate), and the latency of the lookups and a page's
// rows where there are few (64 pages of 64: 2.8 us). Four warps for a page were 0.3 us faster or
// slower for few pages (by their size) and 3 us slower for many.
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
  constexpr int kCols = D * (F16 ? 1 : 2) / 16;  // 16-byte pieces of a row
  constexpr int kWarpRows = 32 / kCols;          // rows of a warp at a time
  constexpr int kWords = F16 ? 8 : 4;            // packed pairs of a piece
  const PagedSeqs& s = p.s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  grid_wait();
  grid_release();
  if (blockIdx.x == 0) check_paged_seqs(s, threadIdx.x, kBoundsThreads);
  const uint32_t unit = blockIdx.x * (kBoundsThreads / 32) + warp, number = unit / static_cast<uint32_t>(p.H_kv);
  const int h = static_cast<int>(unit - number * p.H_kv);
  TouchedPage x;
  if (number >= touched_numbers(s.T, s.B, s.page_shift, s.cu_seqlens != nullptr) || !touched_page(s, number, x)) return;
  const int id = page_entry(s, x.b, x.at);
  if (static_cast<unsigned>(id) >= static_cast<unsigned>(s.num_pages)) {
    if (lane == 0) record_error(s.err, kErrPages);
    return;
  }
  const int rows = min(1 << s.page_shift, x.len - (x.at << s.page_shift));
  const int col = lane % kCols;
  const uint4* keys = reinterpret_cast<const uint4*>(
      static_cast<const uint8_t*>(p.k) +
      (static_cast<long long>(id) * p.k_page + (static_cast<long long>(h) << s.page_shift) * D) * (F16 ? 1 : 2)) + col;
  constexpr uint32_t kPlusInf = F16 ? 0x7c007c00u : 0x7f807f80u, kMinusInf = kPlusInf | 0x80008000u;
  uint32_t lo[kWords], hi[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) { lo[i] = kPlusInf; hi[i] = kMinusInf; }
  constexpr int kAtOnce = 8;  // (all loads before the first is used)
  for (int first = 0; first < rows; first += kAtOnce * kWarpRows) {
    uint4 v[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int r = min(first + k * kWarpRows + lane / kCols, rows - 1);  // (behind the last row that again)
      if (first + k * kWarpRows < rows)
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w) : "l"(keys + r * kCols));
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      if (first + k * kWarpRows >= rows) break;
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t y = F16 ? e4m3x2_to_f16x2(w[(i / 2) & 3] >> (16 * (i & 1))) : w[i & 3];
        lo[i] = min2(lo[i], y, F16);
        hi[i] = max2(hi[i], y, F16);
      }
    }
  }
  // lanes with the same column lie kCols apart
#pragma unroll
  for (int i = 0; i < kWords; ++i)
#pragma unroll
    for (int o = kCols; o < 32; o <<= 1) {
      lo[i] = min2(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o), F16);
      hi[i] = max2(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o), F16);
    }
  if (lane >= kCols) return;
  bool turned = false;
  if constexpr (F16) {
    float scale = 1.0f;
    if constexpr (KIND == kE4m3Pages) scale = power_of_two(page_exponent(p.k_exp, id, p.H_kv, h));
    else if (p.k_scale) scale = __ldg(p.k_scale + h);
    turned = scale < 0.0f;  // turns the order round
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const float2 a = f16x2_to_f32(lo[i]), b = f16x2_to_f32(hi[i]);
      lo[i] = pack_bf16x2(a.x * scale, a.y * scale);
      hi[i] = pack_bf16x2(b.x * scale, b.y * scale);
    }
  }
  uint4* out = reinterpret_cast<uint4*>(p.bounds) + (static_cast<size_t>(id) * p.H_kv + h) * (D / 4);
#pragma unroll
  for (int i = 0; i < kWords; i += 4) {
    out[(turned ? D / 8 : 0) + col * (kWords / 4) + i / 4] = make_uint4(lo[i], lo[i + 1], lo[i + 2], lo[i + 3]);
    out[(turned ? 0 : D / 8) + col * (kWords / 4) + i / 4] = make_uint4(hi[i], hi[i + 1], hi[i + 2], hi[i + 3]);
  }
}

template <int D, int KIND>
cudaError_t launch_bounds(const BoundsParams& p, cudaStream_t stream) {
  const long long units = touched_numbers(p.s.T, p.s.B, p.s.page_shift, p.s.cu_seqlens != nullptr) * p.H_kv;
  const long long blocks = (units + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
  if (units > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_chained<paged_bounds_kernel<D, KIND>>(dim3(static_cast<unsigned>(blocks)), kBoundsThreads, 0, stream, p);
}

// ---------------------------------------------------------------- selection
// One cluster of 1 to 16 CTAs for each token and KV head; each scores a run of the pages. Where
// the first CTA's shared memory holds all scores it does the rest alone; behind wider tables
// (10,000 pages or so) every CTA keeps its own, and they count together. (Each step that
// a cluster takes together costs a barrier and reads of the others' shared memory: of 4096 pages
// on 8 CTAs the steps behind the scores took 19 of 26 us. With 16 CTAs and all scores in one of them
// they take 7 of 13.)
//
// 1. Bounds as products on mma.sync m16n8k16: 16 pages in M, the heads of the group in N,
//    (lo, hi) and (min(q, 0), max(q, 0)) side by side in K, whose order does not matter as long as
//    both operands have the same: a lane reads 16 bytes of a row at a time. The bytes bound
//    this part: every warp has a place of its own for 16 pages' bounds, filled by bulk copies while
//    other warps compute. (With loads to registers, 64 of a thread, too few CTAs find place on an
//    SM: 64 sequences of 64 to 512 pages took 34 us in all, with copies 24; two places for a warp, and
//    so half the CTAs, 35.)
// 2. A histogram of the scores over their range finds the interval that the last chosen
//    score lies in.
// 3. The products are exact, their sums are not: with eps a bound on the sums' error, pages
//    more than 2 eps above the interval are chosen for certain, pages more than 2 eps below it are
//    not, and the few between are scored again: as 64-bit integers, in units of 2^-61 of what
//    the sums can be, so that they do not depend on an order (in 64-bit floating point where the sums
//    are outside [2^-40, 2^100] or a query has an infinity). Ties go to the lower page. A page with an
//    infinity or a NaN among its bounds has a key of its own and leaves the others what they are (one of
//    4096 pages: 19 us, none 14; 8700 while it sent all to the second scores).
// 4. The chosen pages are written in their order.
template <int THREADS>  // (one warp has 160 pages at most)
constexpr int select_bins = THREADS == 32 ? 256 : 1024;
// Up to this many pages to be ranked in 64 bits are compared pair by pair, more by digits (8
// tokens and heads with 100 equal pages take 43 us either way, with 512 163 and 109).
constexpr int kPairs = 64;
// Error of a sum relative to the sum of the magnitudes: two chains of d / 16 = 8 instructions,
// each of which adds 17 terms, each to 2^-23 of the largest at least, and the chains' sum to 2^-24,
// is below 136 * 2^-23 + 2^-24 = 1.63e-5. (On random products, some a thousand times the others, the
// largest seen was 2.3e-6 after eight instructions.)
constexpr float kSumError = 1.75e-5f;
// Sums of numbers below this stay finite; above the other, what products below the normal numbers lose (256
// times 2^-126 at most) is less than 2^-77 of it.
constexpr float kLargest = 1.2676506e30f, kSmallest = 9.0949470e-13f;  // 2^100, 2^-40

// An order of floats as unsigned numbers; NaN above all.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k ^ (k & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ long long ordered(double x) {  // (signed)
  if (x != x) return 0x7fffffffffffffffll;
  const long long b = __double_as_longlong(x + 0.0);  // (-0 as 0)
  return b ^ static_cast<long long>(static_cast<unsigned long long>(b >> 63) >> 1);
}
constexpr long long kNoKey = -0x7fffffffffffffffll - 1;  // below them all
// The key of a score that is no number, next to those in units of 2^-61 (below 2^62 in magnitude).
__device__ __forceinline__ long long key_of_none(float x) {
  return x != x ? 0x7fffffffffffffffll : x > 0.0f ? 0x7ffffffffffffffell : kNoKey;
}
// x (below 2^61 in magnitude) rounded to an integer, by two conversions to 32 bits: one to 64
// runs at a fraction of their rate.
__device__ __forceinline__ long long in_units(float x) {
  const int high = __float2int_rn(x * 4.656612873e-10f);  // 2^-31
  const int low = __float2int_rn(fmaf(static_cast<float>(high), -2147483648.0f, x));
  return (static_cast<long long>(high) << 31) + low;
}
// The larger, a NaN above all.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) < INFINITY; }
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float x) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) { return static_cast<uint32_t>(ld_cluster_s32(addr)); }
__device__ __forceinline__ long long ld_cluster_s64(uint32_t addr) {
  long long v;
  asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where score i is kept: runs of 16 or 32 scores begin in different banks.
__host__ __device__ __forceinline__ int spread(int i) { return i + (i >> 5); }
__host__ __device__ __forceinline__ int spread_size(int n) { return (spread(n) + 3) & ~3; }

// What a CTA shows the others of its cluster.
template <int THREADS>
struct SelectShared {
  uint32_t hist[select_bins<THREADS>];
  uint32_t l1, k_most;       // largest sum of a query row's magnitudes; largest magnitude of the bounds
  uint32_t least, most;      // scores, ordered (the least as its complement)
  uint32_t sure, unsure, chosen;
  uint32_t none;             // some bounds are infinities or NaN
  uint32_t bin, above;       // the bin that was looked for, and what lies above it
  uint32_t warp_sum[THREADS / 32];
  uint64_t full[THREADS / 32];
};

// Finds the bin from the top that holds the k-th of the clusters' numbers (k >= 1 and at most as
// many as there are): sh.bin, and how many lie above it, sh.above. kPer bins a thread.
template <int kPer, int THREADS>
__device__ __forceinline__ void find_bin(SelectShared<THREADS>& sh, int cluster, uint32_t k) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t v[kPer], mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = sh.hist[tid * kPer + i];
  if (cluster > 1) {
    const int rank = cluster_ctarank();
    const uint32_t at = smem_addr(sh.hist + tid * kPer);
    for (int r = 1; r < cluster; ++r) {
      const uint32_t from = cluster_map(at, (rank + r) & (cluster - 1));
      uint32_t w[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) w[i] = ld_cluster_u32(from + 4 * i);
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] += w[i];
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
  for (int w = warp + 1; w < THREADS / 32; ++w) from_here += sh.warp_sum[w];
  uint32_t above = from_here - mine;
  if (above < k && k <= from_here) {
    bool found = false;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i) {
      if (!found && k <= above + v[i]) {
        sh.bin = tid * kPer + i;
        sh.above = above;
        found = true;
      }
      above += v[i];
    }
  }
  __syncthreads();
}

template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 32 ? 12 : THREADS == 128 ? 5 : 2)
paged_select_kernel(const SelectParams p) {
  constexpr int kSelThreads = THREADS, kSelWarps = THREADS / 32, kBins = select_bins<THREADS>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SelectShared<THREADS> sh;
  constexpr int kStride = 4 * D + 64;  // bytes of a row of queries or bounds (the gap spreads rows over the banks)
  const PagedSeqs& s = p.s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ctas = 1 << p.cluster_shift, rank = blockIdx.x & (ctas - 1);
  const int item = static_cast<int>(blockIdx.x >> p.cluster_shift), t = item / p.H_kv, h = item - t * p.H_kv;
  const int q_tiles = (p.group + 7) / 8;
  uint8_t* qs = smem;
  float* score = reinterpret_cast<float*>(qs + q_tiles * 8 * kStride);
  // 16 pages' bounds for each warp, and when every page has its score those to be scored again
  uint8_t* bounds_at = reinterpret_cast<uint8_t*>(score + spread_size(p.slice));
  uint8_t* tile = bounds_at + warp * 16 * kStride;
  long long* list_key = reinterpret_cast<long long*>(bounds_at);
  uint32_t* list = reinterpret_cast<uint32_t*>(list_key + p.slice);
  for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
  if (tid == 0) {
    sh.l1 = sh.k_most = sh.most = sh.least = 0;
    sh.sure = sh.unsure = sh.chosen = sh.none = 0;
  }
  const uint32_t full = smem_addr(&sh.full[warp]);
  if (lane == 0) {
    mbar_init(full, 1);
    fence_barrier_init();
  }
  // The zeros stand before any warp adds to them: the queries' magnitudes (keep_row) come before the
  // CTA's next barrier. (Here it overlaps the end of the grid before.)
  __syncthreads();
  grid_wait();
  grid_release();
  if (blockIdx.x == 0) check_paged_seqs(s, tid, kSelThreads);

  // ---- queries: a warp for each row, loaded before the token's sequence is looked up
  constexpr int kPairs32 = D / 64;  // words of a lane
  auto query_word = [&](int r, int i) {
    return r < p.group ? __ldg(reinterpret_cast<const uint32_t*>(p.q) +
                               (static_cast<size_t>(t) * p.H_q + h * p.group + r) * (D / 2) + i * 32 + lane)
                       : 0u;
  };
  constexpr int kFirst = kSelWarps < 8 ? 8 / kSelWarps : 1;  // rows of a warp among the first eight
  uint32_t first_rows[kFirst][kPairs32];
#pragma unroll
  for (int k = 0; k < kFirst; ++k)
#pragma unroll
    for (int i = 0; i < kPairs32; ++i) first_rows[k][i] = query_word(warp + k * kSelWarps, i);

  // ---- the token's sequence and what it sees
  int b = t;
  SeqSpan span{t, 1};
  if (s.cu_seqlens) {
    // the last one that begins at or before it, found by each warp 32 places at a time: two
    // dependent loads for up to 1024 sequences and not ten
    int n = s.B;
    for (b = 0; n > 1;) {
      const int step = (n + 31) >> 5;
      const bool below = lane * step < n && __ldg(s.cu_seqlens + b + lane * step) <= t;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
      n = min(step, n - last * step);
      b += last * step;
    }
    span = seq_span(s.cu_seqlens, b, s.T, 0);
    if (t < span.start || t >= span.start + span.len) return;  // behind the last sequence
  }
  const int len = max(0, kv_len(s, b) - span.len + (t - span.start) + 1);
  const int pages = (len + (1 << s.page_shift) - 1) >> s.page_shift;
  int* out = p.pages + static_cast<size_t>(item) * p.count;
  if (h == 0 && rank == 0 && tid == 0)
    p.lens[t] = len - (max(0, pages - p.count) << s.page_shift);
  if (pages <= p.count) {  // all of them
    for (int i = rank * kSelThreads + tid; i < p.count; i += ctas * kSelThreads)
      out[i] = i < pages ? page_of(s, b, i) : -1;
    return;
  }
  const int room = p.count - p.first - p.last;  // pages to choose
  const int n_all = pages - p.first - p.last;   // pages to choose from
  if (rank == ctas - 1) {
    for (int i = tid; i < p.first; i += kSelThreads) out[i] = page_of(s, b, i);
    for (int i = tid; i < p.last; i += kSelThreads) out[p.count - p.last + i] = page_of(s, b, pages - p.last + i);
  }
  if (room == 0) return;
  const int per = ((n_all + ctas - 1) / ctas + 15) & ~15;
  int begin = min(n_all, rank * per), n = min(n_all, begin + per) - begin;

  // ---- scores of 16 pages a warp
  const int qd = lane & 3, ar = lane >> 2;
  constexpr int kSteps = 2 * D / 32;  // 16-byte pieces of a lane in a row
  const int tiles = (n + 15) / 16, my_tiles = tiles > warp ? (tiles - warp + kSelWarps - 1) / kSelWarps : 0;
  // lane i < 16 copies page i of a tile (behind the last page that again); the table's entries are
  // checked where they are used, so that their loads do not wait for one another
  const int* table = s.page_table + static_cast<size_t>(b) * s.table_stride + p.first;
  auto entry_at = [&](int k) {
    return lane < 16 ? __ldg(table + begin + min((warp + k * kSelWarps) * 16 + lane, n - 1)) : 0;
  };
  auto copy = [&](int entry) {
    const int id = checked_page(s, entry);
    if (lane == 0) mbar_arrive_expect_tx(full, 16 * 4 * D);
    __syncwarp();
    if (lane < 16)
      bulk_load(smem_addr(tile + lane * kStride),
                static_cast<const uint8_t*>(p.bounds) + (static_cast<size_t>(id) * p.H_kv + h) * (4 * D), 4 * D, full);
  };
  int next = my_tiles > 0 ? entry_at(0) : 0;
  if (ctas > 1) cluster_arrive();  // (this CTA's shared memory is ready for the others)
  if (my_tiles > 0) {
    copy(next);
    if (my_tiles > 1) next = entry_at(1);
  }
  auto keep_row = [&](int r, const uint32_t (&row)[kPairs32]) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(qs + r * kStride);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPairs32; ++i) {
      const uint32_t w = row[i];
      sum += fabsf(bf16lo_to_f32(w)) + fabsf(bf16hi_to_f32(w));
      dst[i * 32 + lane] = min2(w, 0u, false);
      dst[D / 2 + i * 32 + lane] = max2(w, 0u, false);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) atomicMax(&sh.l1, __float_as_uint(sum) & 0x7fffffffu);
  };
#pragma unroll
  for (int k = 0; k < kFirst; ++k) keep_row(warp + k * kSelWarps, first_rows[k]);
  for (int r = warp + kFirst * kSelWarps; r < q_tiles * 8; r += kSelWarps) {
    uint32_t row[kPairs32];
#pragma unroll
    for (int i = 0; i < kPairs32; ++i) row[i] = query_word(r, i);
    keep_row(r, row);
  }
  __syncthreads();
  if (ctas > 1) cluster_wait();
  const uint32_t scores_to = p.gather ? cluster_map(smem_addr(score), 0) : smem_addr(score);
  const int score0 = p.gather ? begin : 0;
  uint32_t k_most = 0;
  float least = INFINITY, most = -INFINITY;
  bool ok = true;
  for (int k = 0; k < my_tiles; ++k) {
    const int i0 = (warp + k * kSelWarps) * 16 + ar;
    // After a wait that ran out nothing more is copied, what is on its way is waited for once
    // more, and the pages that are left count as 0.
    if (ok && !mbar_wait_warp(full, k & 1, p.wait_limit)) {
      if (lane == 0) record_error(s.err, kErrTimeout);
      mbar_wait_warp(full, k & 1, p.wait_limit);
      ok = false;
    }
    const uint8_t* pages_at = tile + ar * kStride + qd * 16;
    float best[2] = {-INFINITY, -INFINITY};
    for (int nt = 0; nt < q_tiles; ++nt) {
      const uint8_t* rows = qs + (nt * 8 + ar) * kStride + qd * 16;
      float acc[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[u][e] = 0.0f;
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        uint4 a[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) a[u] = *reinterpret_cast<const uint4*>(pages_at + 8 * u * kStride + c * 64);
        const uint4 w = *reinterpret_cast<const uint4*>(rows + c * 64);
        mma_bf16(acc[0], a[0].x, a[1].x, a[0].y, a[1].y, w.x, w.y);
        mma_bf16(acc[1], a[0].z, a[1].z, a[0].w, a[1].w, w.z, w.w);
        if (nt == 0) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = __vmaxu2(a[u].x & 0x7fff7fffu, a[u].y & 0x7fff7fffu);
            const uint32_t y = __vmaxu2(a[u].z & 0x7fff7fffu, a[u].w & 0x7fff7fffu);
            k_most = __vmaxu2(k_most, __vmaxu2(x, y));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (nt * 8 + 2 * qd + (e & 1) < p.group) best[e >> 1] = max_nan(best[e >> 1], acc[0][e] + acc[1][e]);
    }
    __syncwarp();
    if (ok && k + 1 < my_tiles) {
      copy(next);
      if (k + 2 < my_tiles) next = entry_at(k + 2);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      best[u] = max_nan(best[u], __shfl_xor_sync(0xffffffffu, best[u], 1));
      best[u] = max_nan(best[u], __shfl_xor_sync(0xffffffffu, best[u], 2));
      if (!ok) best[u] = 0.0f;
      const int i = i0 + 8 * u;
      if (i < n) {
        if (qd == 0) st_cluster_f32(scores_to + 4 * spread(score0 + i), best[u]);
        least = fminf(least, best[u]);
        most = fmaxf(most, best[u]);
      }
    }
  }
  // A page with an infinity or a NaN among its bounds has a score that is none either, whatever the queries: it
  // is no part of the scores' range, and of its bounds those that are numbers count. Where this warp has
  // met one its pages are gone through again, a lane for each.
  if (__any_sync(0xffffffffu, __vcmpgeu2(k_most, 0x7f807f80u))) {
    __syncwarp();  // (its lanes read each other's scores)
    k_most = 0;
    least = INFINITY;
    most = -INFINITY;
    for (int k = 0; k < my_tiles; ++k) {
      const int i = (warp + k * kSelWarps) * 16 + (lane & 15);
      if (i >= n) continue;
      const int id = checked_page(s, __ldg(table + begin + i));
      const uint4* at = static_cast<const uint4*>(p.bounds) + (static_cast<size_t>(id) * p.H_kv + h) * (D / 4);
#pragma unroll 4
      for (int x = 0; x < D / 4; ++x) {
        const uint4 y = __ldg(at + x);
        const uint32_t w[4] = {y.x & 0x7fff7fffu, y.y & 0x7fff7fffu, y.z & 0x7fff7fffu, y.w & 0x7fff7fffu};
#pragma unroll
        for (int e = 0; e < 4; ++e) k_most = __vmaxu2(k_most, w[e] & ~__vcmpgeu2(w[e], 0x7f807f80u));
      }
      const float x = __uint_as_float(ld_cluster_u32(scores_to + 4 * spread(score0 + i)));
      if (is_finite(x)) {
        least = fminf(least, x);
        most = fmaxf(most, x);
      }
    }
    if (lane == 0)
      for (int r = 0; r < (p.gather ? 1 : ctas); ++r) max_cluster_u32(cluster_map(smem_addr(&sh.none), r), 1u);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    k_most = __vmaxu2(k_most, __shfl_xor_sync(0xffffffffu, k_most, o));
    least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  if (lane == 0) {
    // (the least as the most of what is opposite to it; every CTA gets every other's, or the first all)
    const uint32_t x = max(k_most & 0xffffu, k_most >> 16) << 16, y = ~ordered(least), z = ordered(most);
    for (int r = 0; r < (p.gather ? 1 : ctas); ++r) {
      max_cluster_u32(cluster_map(smem_addr(&sh.k_most), r), x);
      max_cluster_u32(cluster_map(smem_addr(&sh.least), r), y);
      max_cluster_u32(cluster_map(smem_addr(&sh.most), r), z);
    }
  }
  if (ctas > 1) cluster_sync_all(); else __syncthreads();
  if (p.gather) {
    if (rank > 0) return;
    begin = 0;
    n = n_all;
  }
  // the CTAs that share the rest
  const int cluster = p.gather ? 1 : ctas;
  auto sync = [&]() {
    if (cluster > 1) cluster_sync_all(); else __syncthreads();
  };
  auto total = [&](uint32_t& x) {
    if (cluster == 1) return x;
    uint32_t sum = 0;
    for (int r = 0; r < cluster; ++r) sum += ld_cluster_u32(cluster_map(smem_addr(&x), r));
    return sum;
  };

  // ---- the interval [lo, hi] of the last score to be chosen
  // Every page whose bounds are numbers has a score of zero, or, where a query row has a NaN, every page one
  // that is none; else sums outside these bounds are taken in floating point alone. With queries that are
  // numbers and sums within the bounds a score is no number only for a page whose bounds are none, and then
  // that of the exact sum: such pages are never chosen for certain, but by a key of their own.
  const float l1 = __uint_as_float(sh.l1);
  const float product = l1 * __uint_as_float(sh.k_most);  // of the products' sums at most
  const bool same = l1 != l1 || (product == 0.0f && (sh.l1 == 0 || sh.k_most == 0));
  const float size = same ? 0.0f : product;
  const bool finite = same || (size < kLargest && size > kSmallest);
  const bool none = finite && (sh.none || l1 != l1);  // some scores are no numbers
  const float eps = size * kSumError;
  float lo = unordered(~sh.least), hi = unordered(sh.most);
  const float range = hi - lo;
  if (finite && range > eps) {
    // (bins by the same rounded expression for every page, so their order is that of the scores)
    const float low = lo, inv = kBins / range;
    // (plus infinity and NaN to the top, minus infinity to the bottom)
    auto bin_at = [](float at) { return static_cast<int>(fmaxf(0.0f, fminf(at, kBins - 1.0f))); };
    auto bin_of = [&](float x) { return bin_at((x - low) * inv); };
    if (none) {
      for (int i = tid; i < n; i += kSelThreads) atomicAdd(&sh.hist[bin_of(score[spread(i)])], 1u);
    } else {  // (the same of numbers)
      for (int i = tid; i < n; i += kSelThreads)
        atomicAdd(&sh.hist[min(kBins - 1, static_cast<int>((score[spread(i)] - low) * inv))], 1u);
    }
    sync();
    find_bin<kBins / kSelThreads>(sh, cluster, room);
    const int bin = sh.bin;
    const uint32_t above = sh.above;
    lo = low + bin * (range / kBins);
    hi = low + (bin + 1) * (range / kBins);
    // a bin far wider than eps (a few scores far from the rest): its own pages again
    if (range > 65536.0f * eps) {
      const float low2 = lo, inv2 = kBins / (range / kBins);
      auto bin2_of = [&](float x) { return bin_at((x - low2) * inv2); };
      sync();
      for (int i = tid; i < kBins; i += kSelThreads) sh.hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads)
        if (bin_of(score[spread(i)]) == bin) atomicAdd(&sh.hist[bin2_of(score[spread(i)])], 1u);
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

  // ---- pages chosen for certain, and those to be scored again: a run of up to 32 a thread
  const int run = (n + kSelThreads - 1) / kSelThreads, run0 = tid * run, run_n = max(0, min(run, n - run0));
  uint32_t chosen = 0, unsure = 0;  // of the run, a bit each
  auto cut = [&](auto numbers) {
#pragma unroll 4
    for (int i = 0; i < run_n; ++i) {
      const float x = score[spread(run0 + i)];
      const bool number = finite && (decltype(numbers)::value || is_finite(x)), sure = number && x > high_cut;
      chosen |= static_cast<uint32_t>(sure) << i;
      unsure |= static_cast<uint32_t>(!sure && !(number && x < low_cut)) << i;
    }
  };
  if (none) cut(std::false_type{});
  else cut(std::true_type{});
  for (uint32_t left = unsure; left; left &= left - 1) {
    const uint32_t at = atomicAdd(&sh.unsure, 1u);
    const int i = run0 + __ffs(left) - 1;
    const float x = score[spread(i)];
    list[at] = i;
    list_key[at] = none && !is_finite(x) ? key_of_none(x) : same ? 0 : kNoKey;
  }
  const uint32_t sures = __reduce_add_sync(0xffffffffu, __popc(chosen));
  if (lane == 0 && sures) atomicAdd(&sh.sure, sures);
  sync();
  const uint32_t n_unsure = total(sh.unsure), need = room - total(sh.sure);
  const int mine = sh.unsure;
  if (n_unsure == need) {
    for (int e = tid; e < mine; e += kSelThreads) score[spread(list[e])] = INFINITY;
    if (tid == 0) sh.chosen = mine;
  } else {
    if (!same) {
      // 2^62 over a power of two that the sums' magnitudes stay below
      const int top = static_cast<int>(__float_as_uint(size) >> 23) - 126;
      const float unit = power_of_two(max(-126, min(126, 61 - top)));
      // a warp for each page and four query rows; the next page's bounds are loaded before
      const int quads = (p.group + 3) / 4;
      uint32_t next[D / 32];
      auto load = [&](int x) {
        const int page = page_of(s, b, p.first + begin + list[x / quads]);
        const uint32_t* src = static_cast<const uint32_t*>(p.bounds) + (static_cast<size_t>(page) * p.H_kv + h) * D;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) next[i] = __ldg(src + i * 32 + lane);
      };
      if (warp < mine * quads) load(warp);
      for (int x = warp; x < mine * quads; x += kSelWarps) {
        const int e = x / quads, r0 = (x - e * quads) * 4;
        uint32_t y[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) y[i] = next[i];
        if (x + kSelWarps < mine * quads) load(x + kSelWarps);
        if (none && !is_finite(score[spread(list[e])])) continue;  // (has its key)
        long long key = kNoKey;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (r0 + u >= p.group) break;
          const uint32_t* q = reinterpret_cast<const uint32_t*>(qs + (r0 + u) * kStride);
          long long of_row = 0;
          if (finite) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const uint32_t w = q[i * 32 + lane];
              of_row += in_units(bf16lo_to_f32(w) * bf16lo_to_f32(y[i]) * unit);
              of_row += in_units(bf16hi_to_f32(w) * bf16hi_to_f32(y[i]) * unit);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) of_row += __shfl_xor_sync(0xffffffffu, of_row, o);
          } else {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              const uint32_t w = q[i * 32 + lane];
              sum = fma(static_cast<double>(bf16lo_to_f32(w)), static_cast<double>(bf16lo_to_f32(y[i])), sum);
              sum = fma(static_cast<double>(bf16hi_to_f32(w)), static_cast<double>(bf16hi_to_f32(y[i])), sum);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            of_row = ordered(sum);
          }
          key = max(key, of_row);
        }
        if (lane == 0) atomicMax(list_key + e, key);
      }
    }
    sync();
    if (n_unsure <= kPairs) {
      for (int e = tid; e < mine; e += kSelThreads) {
        const long long key = list_key[e];
        const int place = begin + list[e];
        uint32_t better = 0;
        if (cluster == 1) {
          for (int i = 0; i < mine; ++i)
            better += list_key[i] > key || (list_key[i] == key && static_cast<int>(list[i]) < place);
        } else {
          for (int r = 0; r < cluster; ++r) {
            const uint32_t theirs = ld_cluster_u32(cluster_map(smem_addr(&sh.unsure), r));
            const uint32_t keys = cluster_map(smem_addr(list_key), r), places = cluster_map(smem_addr(list), r);
            for (uint32_t i = 0; i < theirs; ++i) {
              const long long other = ld_cluster_s64(keys + 8 * i);
              better += other > key || (other == key && static_cast<int>(ld_cluster_u32(places + 4 * i)) + r * per < place);
            }
          }
        }
        if (better < need) atomicAdd(&sh.chosen, 1u);
        // (the list's scores are not read by others)
        score[spread(list[e])] = better < need ? INFINITY : -INFINITY;
      }
    } else {
      // By digits of 8 bits from the top: eight of the score, two of the place (lower ones first).
      unsigned long long key = 0;
      uint32_t place = 0, left = need;
      auto key_of = [&](int e) { return static_cast<unsigned long long>(list_key[e]) ^ 0x8000000000000000ull; };
      auto place_of = [&](int e) { return 0xffffu - (begin + list[e]); };
      for (int digit = 0; digit < 10; ++digit) {
        for (int i = tid; i < 256; i += kSelThreads) sh.hist[i] = 0;
        __syncthreads();
        for (int e = tid; e < mine; e += kSelThreads) {
          const unsigned long long x = key_of(e);
          const uint32_t y = place_of(e);
          if (digit < 8) {
            if (digit == 0 || (x ^ key) >> (64 - 8 * digit) == 0) atomicAdd(&sh.hist[(x >> (56 - 8 * digit)) & 255], 1u);
          } else if (x == key && (digit == 8 || (y ^ place) >> 8 == 0)) {
            atomicAdd(&sh.hist[(y >> (8 * (9 - digit))) & 255], 1u);
          }
        }
        sync();
        find_bin<256 / kSelThreads>(sh, cluster, left);
        left -= sh.above;
        if (digit < 8) key |= static_cast<unsigned long long>(sh.bin) << (56 - 8 * digit);
        else place |= sh.bin << (8 * (9 - digit));
        sync();
      }
      for (int e = tid; e < mine; e += kSelThreads) {
        const unsigned long long x = key_of(e);
        const bool in = x > key || (x == key && place_of(e) >= place);
        if (in) atomicAdd(&sh.chosen, 1u);
        score[spread(list[e])] = in ? INFINITY : -INFINITY;
      }
    }
  }
  sync();

  // ---- the chosen pages in their order
  int at = p.first;
  for (int r = 0; r < (cluster == 1 ? 0 : rank); ++r)
    at += ld_cluster_u32(cluster_map(smem_addr(&sh.sure), r)) + ld_cluster_u32(cluster_map(smem_addr(&sh.chosen), r));
  for (uint32_t left = unsure; left; left &= left - 1) {
    const int i = __ffs(left) - 1;
    chosen |= static_cast<uint32_t>(score[spread(run0 + i)] == INFINITY) << i;
  }
  int before = __popc(chosen);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += y;
  }
  if (lane == 31) sh.warp_sum[warp] = before;
  __syncthreads();
  at += before - __popc(chosen);
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) at += w < warp ? sh.warp_sum[w] : 0;
  for (uint32_t left = chosen; left; left &= left - 1)
    out[at++] = page_of(s, b, p.first + begin + run0 + __ffs(left) - 1);
  if (cluster > 1) cluster_sync_all();  // no CTA leaves while another one reads its counts
}

template <int D, int THREADS>
cudaError_t launch_select(const SelectParams& p, int cluster, long long ctas, int smem, int most, cudaStream_t stream) {
  cudaError_t e = allow_smem<paged_select_kernel<D, THREADS>>(most);
  if (e == cudaSuccess) e = allow_wide_clusters<paged_select_kernel<D, THREADS>>();
  if (e != cudaSuccess) return e;
  return launch_clusters<paged_select_kernel<D, THREADS>>(cluster, dim3(static_cast<unsigned>(ctas)), THREADS, smem, stream, p);
}

template <int D>
cudaError_t plan_select(SelectParams p, int n_sm, cudaStream_t stream) {
  constexpr int kStride = 4 * D + 64, kMost = 218 * 1024;  // (beside the static shared memory)
  // More CTAs of a cluster while they find places at once (two on an SM) and each has a
  // round of its warps.
  const long long items = static_cast<long long>(p.s.T) * p.H_kv;
  int cluster = 1;
  p.cluster_shift = 0;
  while (cluster < kSelectCluster &&
         (p.s.max_pages > kSelectSlice * cluster ||
          (items * 2 * cluster <= 2ll * n_sm && p.s.max_pages >= 2 * cluster * 128))) {
    cluster *= 2;
    ++p.cluster_shift;
  }
  const long long ctas = items * cluster;
  // Few pages for each of many tokens and heads: a warp for each, of which twelve find place on an
  // SM. Against four warps each, five on an SM (32 heads on 16 of 128, us): 200 tokens over 21 pages 22.2
  // and 39.9, over 95 36.9 and 45.2, over 144 47.9 and 61.7, over 238 69.9 and 73.4, with heads of 64 60.5
  // and 57.7; 800 tokens and heads, all at once on the SMs either way, 17.2 and 16.2, 1600 24.4 and 26.0.
  const bool small = cluster == 1 && p.s.max_pages <= 160 && items > 10ll * n_sm;
  const int warps = cluster > 1 ? 8 : small ? 1 : 4;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  auto bytes = [&](int share) {
    p.slice = ((p.s.max_pages + share - 1) / share + 15) & ~15;
    return (p.group + 7) / 8 * 8 * kStride + spread_size(p.slice) * 4 + max(warps * 16 * kStride, p.slice * 12);
  };
  p.gather = cluster > 1 && p.s.max_pages <= 32 * 256 && bytes(1) <= kMost;
  const int smem = bytes(p.gather ? 1 : cluster);
  return cluster > 1 ? launch_select<D, 256>(p, cluster, ctas, smem, kMost, stream)
         : small     ? launch_select<D, 32>(p, cluster, ctas, smem, kMost, stream)
                     : launch_select<D, 128>(p, cluster, ctas, smem, kMost, stream);
}

}  // namespace

cudaError_t launch_paged_bounds(const BoundsParams& p, int d, int kind, cudaStream_t stream) {
  const int slot = prof_begin(kKPagedBounds, stream);
  auto of_kind = [&](auto k) {
    constexpr int K = decltype(k)::value;
    return d == 128 ? launch_bounds<128, K>(p, stream) : launch_bounds<64, K>(p, stream);
  };
  const cudaError_t e = kind == kBf16   ? of_kind(std::integral_constant<int, kBf16>{})
                        : kind == kE4m3 ? of_kind(std::integral_constant<int, kE4m3>{})
                                        : of_kind(std::integral_constant<int, kE4m3Pages>{});
  prof_end(slot, stream);
  return e;
}

cudaError_t launch_paged_select(const SelectParams& p, int d, int n_sm, cudaStream_t stream) {
  const int slot = prof_begin(kKPagedSelect, stream);
  const cudaError_t e = d == 128 ? plan_select<128>(p, n_sm, stream) : plan_select<64>(p, n_sm, stream);
  prof_end(slot, stream);
  return e;
}

}  // namespace attn
