// What the kernels over a paged key-value cache share: the cache's description,
// the sequences' lengths and the page look-up, all of them clamped so that no
// access leaves the cache or the page table whatever the device arrays hold.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "attn_common.cuh"

namespace attn {

// What the cache holds (the values of ATTN_CACHE_*): bf16; e4m3 with an fp32 scale for each
// KV head; e4m3 with a power of two for each page and KV head.
constexpr int kBf16 = 0, kE4m3 = 1, kE4m3Pages = 3;

// Exponents of the powers of two. Attention works with the weights times the values' 2^ev, in
// 32 bits, and takes 2^ev out of their sum again: a weight w of a page beside one whose ev is higher
// by s is lost below 2^-126 2^s, with 88 powers between the ends below 2^-38 of the largest. (448
// 2^24 is 7.5e9; a page of zeros has the lowest.)
constexpr int kMinExp = -64, kMaxExp = 24;
__device__ __forceinline__ uint32_t page_byte(const uint8_t* exps, int page, int H_kv, int h) {
  return __ldg(exps + static_cast<size_t>(page) * H_kv + h);
}
__device__ __forceinline__ int exponent_of(uint32_t byte) {
  return max(kMinExp, min(kMaxExp, static_cast<int>(byte) - 127));
}
__device__ __forceinline__ int page_exponent(const uint8_t* exps, int page, int H_kv, int h) {
  return exponent_of(page_byte(exps, page, H_kv, h));
}
// 2^e, e from -126 to 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Two fp16 values, widened.
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

// Sequences, their lengths in the cache and their pages.
struct PagedSeqs {
  const int* cu_seqlens;  // new tokens: packed offsets [B + 1]; nullptr: one per sequence
  const int* kv_lens;     // [B] keys of each sequence, its new tokens among them
  const int* page_table;  // [B, max_pages], rows table_stride apart
  int B, T;               // sequences; rows of q
  int max_pages, num_pages;
  long long table_stride;  // entries between rows of page_table
  long long head_stride;   // entries between the KV heads of a row, 0: they share their pages
  int page_shift;         // log2(page_size)
  int* err;               // device error word
};

// Keys of sequence b, clamped into what its page table row can hold.
__device__ __forceinline__ int kv_len(const PagedSeqs& s, int b) {
  const long long most = static_cast<long long>(s.max_pages) << s.page_shift;
  return static_cast<int>(min(static_cast<long long>(max(__ldg(s.kv_lens + b), 0)), most));
}
// Rows of q that belong to sequence b.
__device__ __forceinline__ SeqSpan new_span(const PagedSeqs& s, int b) {
  return s.cu_seqlens ? seq_span(s.cu_seqlens, b, s.T, 0) : SeqSpan{b, b < s.T ? 1 : 0};
}
// The page that holds place `i` of sequence b's page table row (i < max_pages), for KV head h
// where the heads have pages of their own. An index outside the cache is recorded and page 0
// taken for it.
// A warp that looks pages up ahead keeps the table's entry and checks it when it uses it: the check
// waits for the load.
__device__ __forceinline__ int page_entry(const PagedSeqs& s, int b, int i, int h = 0) {
  return __ldg(s.page_table + static_cast<size_t>(b) * s.table_stride + h * s.head_stride + i);
}
__device__ __forceinline__ int checked_page(const PagedSeqs& s, int id) {
  if (static_cast<unsigned>(id) < static_cast<unsigned>(s.num_pages)) return id;
  record_error(s.err, kErrPages);
  return 0;
}
__device__ __forceinline__ int page_of(const PagedSeqs& s, int b, int i, int h = 0) {
  return checked_page(s, page_entry(s, b, i, h));
}
// A page that new tokens of a sequence go to.
struct TouchedPage {
  int b, at;   // sequence, place in its page table row
  int lo, hi;  // positions of the new tokens in it
  int row;     // row of q, k and v of the first
  int len;     // keys of the sequence
};
// The pages that new tokens touch are numbered sequence by sequence: sequence b's numbers
// begin at cu[b] / page_size + 2 b, which leaves it floor(n / page_size) + 2, and n tokens touch
// floor((n - 2) / page_size) + 2 at most. So no sum over the sequences is needed; some numbers
// stay without a page. One token for each sequence: number b is its page.
__host__ __device__ __forceinline__ long long touched_numbers(int T, int B, int page_shift, bool packed) {
  return packed ? (T >> page_shift) + 2ll * B : B;
}
// (The same number in every lane of a warp, which look for the sequence together: 32 places of the
// offsets at a time, so that up to 1024 sequences take two dependent loads and not ten.)
__device__ __forceinline__ bool touched_page(const PagedSeqs& s, long long number, TouchedPage& x) {
  x.b = static_cast<int>(number);
  long long first = number;
  if (s.cu_seqlens) {
    auto base = [&](int b) { return (min(max(__ldg(s.cu_seqlens + b), 0), s.T) >> s.page_shift) + 2ll * b; };
    const int lane = threadIdx.x & 31;
    // the last sequence whose numbers begin at or before it lies in [lo, lo + n)
    int lo = 0, n = s.B;
    while (n > 1) {
      const int step = (n + 31) >> 5, at = lo + lane * step;
      const bool below = lane * step < n && base(at) <= number;
      const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
      n = min(step, n - last * step);
      lo += last * step;
    }
    x.b = lo;
    first = base(lo);
  }
  const SeqSpan span = new_span(s, x.b);
  x.len = kv_len(s, x.b);
  const int before = x.len - span.len, begin = max(before, 0);  // before < 0: padding
  const long long at = (begin >> s.page_shift) + (number - first);
  if (span.len == 0 || x.len == 0 || number < first || at > (x.len - 1) >> s.page_shift) return false;
  x.at = static_cast<int>(at);
  x.lo = max(begin, x.at << s.page_shift);
  x.hi = min(x.len, (x.at + 1) << s.page_shift);
  x.row = span.start + (x.lo - before);
  return true;
}
// Records lengths that the clamps above would change: thread `tid` of
// `nthreads` checks its share. Rows of q behind the last sequence are allowed.
__device__ __forceinline__ void check_paged_seqs(const PagedSeqs& s, int tid, int nthreads) {
  const long long most = static_cast<long long>(s.max_pages) << s.page_shift;
  for (int b = tid; b < s.B; b += nthreads) {
    const int len = __ldg(s.kv_lens + b);
    if (len < 0 || len > most) record_error(s.err, kErrPages);
    if (s.cu_seqlens) {
      const int a = __ldg(s.cu_seqlens + b), e = __ldg(s.cu_seqlens + b + 1);
      if ((b == 0 && a != 0) || a > e || e > s.T) record_error(s.err, kErrSeqlens);
    }
  }
}

// Allows a kernel that much shared memory, once per device: the most that it is launched with.
template <auto Kernel>
cudaError_t allow_smem(int most) {
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Allows a kernel clusters of 16 CTAs, once per device.
template <auto Kernel>
cudaError_t allow_wide_clusters() {
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Launches a kernel that calls grid_wait() in every thread before it touches
// memory: its launch and set-up overlap the end of the grid before it. Clusters of
// `cluster` CTAs. (A kernel whose shared memory differs from call to call calls allow_smem with
// the most before.)
template <auto Kernel, typename... Args>
cudaError_t launch_clusters(int cluster, dim3 grid, int threads, int smem, cudaStream_t stream, const Args&... args) {
  if (smem > 48 * 1024) {
    const cudaError_t e = allow_smem<Kernel>(smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, Kernel, args...);
}
template <auto Kernel, typename... Args>
cudaError_t launch_chained(dim3 grid, int threads, int smem, cudaStream_t stream, const Args&... args) {
  return launch_clusters<Kernel>(1, grid, threads, smem, stream, args...);
}

// A power of two that brings a row whose largest magnitude is `top` to [1, 2) when
// it divides the row; its inverse is in `down`. fp16 then holds bf16 values exactly from
// 2^-17 on, those below to half a step of 2^-24, whatever the row's range was: an element
// moves by 2^-25 of the largest at most.
// Infinities stay infinities; a row of zeros is left alone (its power would be 2^-126).
__device__ __forceinline__ float row_power(float top, float& down) {
  int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  ex = ex > 127 || top == 0.0f ? 0 : max(-126, min(126, ex));
  down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
}

// Over an e4m3 cache P goes into its product as fp16, at 2^kLift times its value (which
// the sums share): at most 2^15, and what lies above 2^-21 of a row's largest keeps its
// 11 bits.
constexpr float kLift = kTau < 15.0f ? 15.0f - kTau : 0.0f;

// ---- appending
struct AppendParams {
  PagedSeqs s;
  const void* q; const void* k; const void* v;  // bf16, [T, heads, d], any token stride
  void* q_out;
  long long q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  void* k_cache; void* v_cache;
  long long k_page, v_page;  // elements between pages
  const float* k_scale; const float* v_scale;  // e4m3: [H_kv] or nullptr
  const double* inv_freq;    // [rotary_dim / 2] radians per position, or nullptr
  uint8_t* k_exp; uint8_t* v_exp;  // a scale for each page: [num_pages, H_kv]
  int H_q, H_kv, d, rotary_dim, interleaved, e4m3;
};
cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream);
// Over a cache with a scale for each page; where many tokens are appended by rows, with maps of k
// and v in boxes of kAppendRows tokens and append_box_heads heads.
constexpr int kAppendRows = 16;
bool append_by_rows(const PagedSeqs& s);
int append_box_heads(int H_kv, int d);
cudaError_t launch_paged_append_pages(const AppendParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      long long wait_limit, cudaStream_t stream);

// ---- choosing pages by bounds of their keys
struct BoundsParams {
  PagedSeqs s;
  const void* k;  // the cache's keys
  long long k_page;  // elements between pages
  const float* k_scale;  // e4m3: [H_kv] or nullptr
  const uint8_t* k_exp;  // a scale for each page
  void* bounds;  // bf16 [num_pages, H_kv, 2, d]: minimum, maximum
  int H_kv;
};
cudaError_t launch_paged_bounds(const BoundsParams& p, int d, int kind, cudaStream_t stream);

struct SelectParams {
  PagedSeqs s;
  const void* q;       // bf16 [T, H_q, d]
  const void* bounds;
  int* pages;          // [T, H_kv, count]
  int* lens;           // [T]
  int H_q, H_kv, group, count, first, last;
  // set by the launch: CTAs of a token and KV head, whether the first of them has all the scores, and
  // how many a CTA can have
  int cluster_shift, gather, slice;
  long long wait_limit;
};
// Pages that a row of a page table may have: 16 CTAs keep 4096 scores each.
constexpr int kSelectSlice = 4096, kSelectCluster = 16, kSelectPages = kSelectSlice * kSelectCluster;
cudaError_t launch_paged_select(const SelectParams& p, int d, int n_sm, cudaStream_t stream);

// ---- streaming attention: few query rows per sequence
constexpr int kStreamCtas = 456;  // CTAs the workspace holds partial results for
constexpr int kStreamTile = 64;   // keys per tile
constexpr int kStreamCluster = 8;  // CTAs of a cluster at most
// CTAs on an SM: three where the registers (8 query rows) and shorter tiles (rows of
// `row_bytes` of K or V) allow it, and over pages with scales with 16 query rows of 64 (4 drafted tokens
// behind 4000 to 32,000 keys, 8 sequences, 32 heads on 8: 41.5 us with two, 38.1 with three; rows of
// 128 spill: 35.3 and 49.6).
constexpr int stream_ctas(int rows, int row_bytes, bool pages) {
  return (rows == 8 && row_bytes <= 128) || (pages && row_bytes <= 64) ? 3 : 2;
}

struct StreamParams {
  PagedSeqs s;
  const void* q;  // bf16 [T, H_q, d]
  void* o;        // bf16 [T, H_q, d]
  float* lse;
  long long lse_row, lse_head;  // elements between rows and between heads of lse
  const float* k_scale; const float* v_scale;
  const uint8_t* k_exp; const uint8_t* v_exp;  // kE4m3Pages: [num_pages, H_kv]
  int H_q, H_kv, group, causal;
  float scale_log2;
  int4* heads;            // workspace: [kStreamCtas, 2] where the pieces of a split item begin
  float* part_ml;         // workspace: [2 kStreamCtas, 16, 2]
  float* part_o;          // workspace: [2 kStreamCtas, 16, d]
  int cluster;        // CTAs of a cluster, 0: the units are dealt out
  long long items;    // clusters
  int grid, cluster_shift;  // set by the launch
  int fault;
  long long wait_limit;
};
cudaError_t launch_paged_stream(const CUtensorMap& tk, const CUtensorMap& tv, const StreamParams& p,
                                int d, int rows, int kind, int n_sm, cudaStream_t stream);

// ---- tensor-core attention: many query rows per sequence
constexpr int kFwdSms = 152;               // SMs that calls and workspaces are planned for
constexpr int kFwdListed = 4 * kFwdSms;    // work tiles that the planning kernel describes

struct PagedFwdParams {
  PagedSeqs s;
  void* o;     // bf16 [T, H_q, d]
  float* lse;  // [H_q, T]
  int H_q, H_kv, group, d, causal;
  int tok_tile;      // query tokens per 128-row tile: floor(128 / group)
  int split;         // few work tiles: whole waves of them, the rest cut evenly
  int max_work;      // work tiles that the host expects at most
  float scale_log2;
  const float* k_scale; const float* v_scale;  // e4m3: [H_kv] or nullptr
  const uint8_t* k_exp; const uint8_t* v_exp;  // kE4m3Pages: [num_pages, H_kv]
  const float* q_up;  // e4m3, workspace: what each row of the fp16 queries was divided by [T, H_q]
  int* seq_order;    // workspace: sequences, longest first [B]
  int* tile_start;   // workspace: first work tile of each of them [B + 1]
  int* tile_ctr;     // workspace: claim counter (split == 0)
  int4* tiles;       // workspace: the first kFwdListed work tiles, three words each
  int4* rest_tiles;  // workspace, split: the work tiles of the rest [grid], three words each
  int4* shares;      // workspace, split: each CTA's share of the rest [grid]
  int* rest_units;   // workspace, split: first unit of each work tile of the rest [grid + 1]
  int2* rest_owners; // workspace, split: first and last CTA of each of them [grid]
  float* part_ml;    // workspace, split: [2 grid, 2, 128, 2]
  float* part_o;     // workspace, split: [2 grid, 2, 128, d]
  int grid;
  int fault;
  long long wait_limit;
};
cudaError_t launch_paged_fwd(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedFwdParams& p, int d, int kind, cudaStream_t stream);
// Queries as fp16 for products with an e4m3 cache: each row divided by a power of
// two (kept in q_up) that brings its largest value to [1, 2).
cudaError_t launch_queries_f16(const void* q, void* q16, float* q_up, long long rows, int d,
                               cudaStream_t stream);

}  // namespace attn
