// What the kernels over a paged key-value cache share: the cache's description,
// the sequences' lengths and the page look-up, all of them clamped so that no
// access leaves the cache or the page table whatever the device arrays hold.
#pragma once

#include <atomic>

#include "attn_common.cuh"

namespace attn {

// Sequences, their lengths in the cache and their pages.
struct PagedSeqs {
  const int* cu_seqlens;  // new tokens: packed offsets [B + 1]; nullptr: one per sequence
  const int* kv_lens;     // [B] keys of each sequence, its new tokens among them
  const int* page_table;  // [B, max_pages], rows table_stride apart
  int B, T;               // sequences; rows of q
  int max_pages, num_pages;
  long long table_stride;  // entries between rows of page_table
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
// The page that holds place `i` of sequence b's page table row (i < max_pages).
// An index outside the cache is recorded and page 0 taken for it.
__device__ __forceinline__ int page_of(const PagedSeqs& s, int b, int i) {
  const int id = __ldg(s.page_table + static_cast<size_t>(b) * s.table_stride + i);
  if (static_cast<unsigned>(id) < static_cast<unsigned>(s.num_pages)) return id;
  record_error(s.err, kErrPages);
  return 0;
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

// Launches a kernel that calls grid_wait() in every thread before it touches
// memory: its launch and set-up overlap the end of the grid before it. The
// shared-memory size is set once per device. Clusters of `cluster` CTAs.
template <auto Kernel, typename... Args>
cudaError_t launch_clusters(int cluster, dim3 grid, int threads, int smem, cudaStream_t stream, const Args&... args) {
  if (smem > 48 * 1024) {
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      ready.fetch_or(bit, std::memory_order_relaxed);
    }
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
  int H_q, H_kv, d, rotary_dim, interleaved, e4m3;
};
cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream);

// ---- streaming attention: few query rows per sequence
constexpr int kStreamCtas = 456;  // CTAs the workspace holds partial results for
constexpr int kStreamTile = 64;   // keys per tile
constexpr int kStreamCluster = 8;  // CTAs of a cluster at most
// CTAs on an SM: three where the registers (8 query rows) and shorter tiles (rows of
// `row_bytes` of K or V) allow it.
constexpr int stream_ctas(int rows, int row_bytes) { return rows == 8 && row_bytes <= 128 ? 3 : 2; }

struct StreamParams {
  PagedSeqs s;
  const void* q;  // bf16 [T, H_q, d]
  void* o;        // bf16 [T, H_q, d]
  float* lse;
  long long lse_row, lse_head;  // elements between rows and between heads of lse
  const float* k_scale; const float* v_scale;
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
                                int d, int rows, bool e4m3, int n_sm, cudaStream_t stream);

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
                             const PagedFwdParams& p, int d, bool e4m3, cudaStream_t stream);
// Queries as fp16 for products with an e4m3 cache: each row divided by a power of
// two (kept in q_up) that brings its largest value to [1, 2).
cudaError_t launch_queries_f16(const void* q, void* q16, float* q_up, long long rows, int d,
                               cudaStream_t stream);

}  // namespace attn
