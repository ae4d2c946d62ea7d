// Host side of the paged key-value cache calls declared in include/attn.h:
// argument checks, tensor maps over the cache, workspace plan and launches.
#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/attn.h"
#include "host.h"
#include "paged.cuh"

using namespace attn;

namespace {

static_assert(kBf16 == ATTN_CACHE_BF16 && kE4m3 == ATTN_CACHE_E4M3 && kE4m3Pages == ATTN_CACHE_E4M3_PAGES, "types");
bool in_bytes(const attn_paged_cache* c) { return c->type != kBf16; }

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_cache(const attn_paged_cache* c) {
  if (!c) return ATTN_ERR_NULL_PTR;
  if (c->d != 64 && c->d != 128) return ATTN_ERR_UNSUPPORTED_HEADDIM;
  if (c->type != kBf16 && c->type != kE4m3 && c->type != kE4m3Pages) return ATTN_ERR_BAD_SHAPE;
  if (c->num_pages < 1 || c->H_kv < 1 || c->H_kv > 65535) return ATTN_ERR_BAD_SHAPE;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return ATTN_ERR_BAD_SHAPE;
  if (!c->k || !c->v) return ATTN_ERR_NULL_PTR;
  if (c->type == kE4m3Pages && (!c->k_exp || !c->v_exp)) return ATTN_ERR_NULL_PTR;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return ATTN_ERR_ALIGNMENT;
  const long long page = static_cast<long long>(c->H_kv) * c->page_size * c->d;
  const long long es = in_bytes(c) ? 1 : 2;
  // tensor maps hold strides below 2^40 bytes
  for (long long stride : {c->k_page_stride, c->v_page_stride}) {
    if (stride < page || stride >= (1ll << 39)) return ATTN_ERR_BAD_SHAPE;
    if ((stride * es) & 15) return ATTN_ERR_ALIGNMENT;
  }
  return ATTN_OK;
}

int check_seqs(const attn_paged_cache* c, int T, int B, int H_q, const int* seqlens,
               const int* kv_lens, const int* page_table, int max_pages, long long table_stride) {
  if (T < 0 || B < 0 || H_q < 0 || H_q > 65535 || max_pages < 0) return ATTN_ERR_BAD_SHAPE;
  if (H_q % c->H_kv != 0) return ATTN_ERR_GQA_RATIO;
  if (!seqlens && T != B) return ATTN_ERR_BAD_SHAPE;
  if (T > 0 && B == 0) return ATTN_ERR_BAD_SHAPE;
  if (max_pages > 0 && table_stride < max_pages) return ATTN_ERR_BAD_SHAPE;
  if (static_cast<long long>(max_pages) * c->page_size > (1ll << 30)) return ATTN_ERR_BAD_SHAPE;
  if (static_cast<long long>(T) * H_q > 0x7fffffffll) return ATTN_ERR_BAD_SHAPE;
  if (T > 0 && (!kv_lens || (max_pages > 0 && !page_table))) return ATTN_ERR_NULL_PTR;
  if (!aligned(seqlens, 4) || !aligned(kv_lens, 4) || !aligned(page_table, 4)) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

PagedSeqs seqs_of(const attn_paged_cache* c, int T, int B, const int* seqlens, const int* kv_lens,
                  const int* page_table, int max_pages, long long table_stride, int* err) {
  PagedSeqs s;
  s.cu_seqlens = seqlens;
  s.kv_lens = kv_lens;
  s.page_table = page_table;
  s.B = B;
  s.T = T;
  s.max_pages = max_pages;
  s.table_stride = table_stride;
  s.head_stride = 0;
  s.num_pages = c->num_pages;
  s.page_shift = 0;
  while ((1 << s.page_shift) < c->page_size) ++s.page_shift;
  s.err = err;
  return s;
}

// 4-D map over the pages of k or v: boxes of `rows` rows of one head of one
// page, at most 128 bytes of each, swizzled over the box's row width.
int encode_pages_map(const HostDevice& dev, CUtensorMap* m, const attn_paged_cache* c, const void* base,
                     long long page_stride, unsigned rows) {
  const bool e4m3 = in_bytes(c);
  const cuuint64_t es = e4m3 ? 1 : 2, d = static_cast<cuuint64_t>(c->d);
  const cuuint64_t page = static_cast<cuuint64_t>(c->page_size);
  cuuint64_t dims[4] = {d, page, static_cast<cuuint64_t>(c->H_kv), static_cast<cuuint64_t>(c->num_pages)};
  cuuint64_t strides[3] = {d * es, d * es * page, static_cast<cuuint64_t>(page_stride) * es};
  const unsigned width = static_cast<unsigned>(d * es < 128 ? d : 128 / es);
  cuuint32_t box[4] = {width, rows, 1, 1};
  cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = dev.encode(
      m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
      const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      width * es == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// 3-D map over q, k or v, [T, H, d] bf16 (or fp16), tokens `stride` elements apart: boxes of `width`
// columns, `heads` heads and `tokens` tokens, with a 128-byte swizzle or none.
int encode_rows_map(const HostDevice& dev, CUtensorMap* m, const void* base, int d, int H, int T, long long stride,
                    int width, int heads, int tokens, bool f16, bool swizzle) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(width), static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  cuuint32_t step[3] = {1, 1, 1};
  const CUresult r = dev.encode(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                                const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// Workspace of the streaming kernel: what each CTA says about the split item that
// begins in it, then the partial results.
struct StreamPlan {
  size_t ml_off, o_off, total;
};
StreamPlan stream_plan(int d) {
  StreamPlan w;
  w.ml_off = align256(static_cast<size_t>(2 * kStreamCtas) * sizeof(int4));
  w.o_off = w.ml_off + align256(static_cast<size_t>(2 * kStreamCtas) * 16 * 2 * sizeof(float));
  w.total = w.o_off + static_cast<size_t>(2 * kStreamCtas) * 16 * d * sizeof(float);
  return w;
}

// Work tiles of the tensor-core kernel at most, and its workspace: order and
// first tile of the sequences, the claim counter, and where there are few tiles for
// each SM the shares of the rest and the partial results of its pieces.
struct FwdPlan {
  int tok_tile;
  long long tiles;
  bool split;
  size_t tiles_off, ml_off, o_off, q16_off, up_off, total;
};
FwdPlan fwd_plan(int T, int B, int group, int H_kv, int d, bool e4m3) {
  FwdPlan f;
  f.tok_tile = kTileM / group;
  const long long rows = 2ll * f.tok_tile;
  // every sequence with new tokens has ceil(n / rows) blocks
  f.tiles = (T + (rows - 1) * B) / rows;
  if (f.tiles > T) f.tiles = T;
  f.tiles *= H_kv;
  // From four waves on, claiming leaves an SM idle for less than the join costs.
  f.split = f.tiles < kFwdListed;
  const size_t slots = f.split ? static_cast<size_t>(2 * kFwdSms) * 2 * kTileM : 0;
  // ints, then the listed and the rest's tiles, the shares and the owners of the rest
  f.tiles_off = align256((2 * static_cast<size_t>(B) + 2 + kFwdSms + 1) * sizeof(int));
  f.ml_off = f.tiles_off + align256((3 * (kFwdListed + kFwdSms) + kFwdSms) * sizeof(int4) + kFwdSms * sizeof(int2));
  f.o_off = f.ml_off + align256(slots * 2 * sizeof(float));
  // e4m3: the queries as fp16 and their rows' powers of two
  const size_t rows_q = e4m3 ? static_cast<size_t>(T) * group * H_kv : 0;
  f.q16_off = f.o_off + align256(slots * d * sizeof(float));
  f.up_off = f.q16_off + align256(rows_q * d * 2);
  f.total = f.up_off + rows_q * sizeof(float);
  return f;
}

// Chunks of 16 query rows at most go to the streaming kernel, which reads each key
// once per 16 rows and deals the keys out evenly; more rows to the tensor-core
// kernel, whose tiles hold 128. The host knows the mean of the sequences' rows.
bool few_rows(int T, int B, int group) {
  return group > kTileM || static_cast<long long>(T) * group <= 16ll * B;
}
// So does little work, by its items (16 rows of a KV head) and what the page table can
// hold: tiles of 64 keys, by their bytes, and about ten more for each item. 20 new tokens
// of each of 2 prompts behind 2500 keys, 32 heads on 8 (4800 units), take 19.4 us there and 26.0
// with the planning kernel and its tiles, 20 of one behind 9000 (7200) 27.4 and 30.3, 64 behind
// 4000 (10,000) 31.9 and 28.0; 350 of a prompt over an e4m3 cache (9200) 27.7 and 20.1.
bool little_work(const attn_paged_cache* c, int T, int B, int group, int max_pages) {
  const long long items = ((static_cast<long long>(T) * group + 15) / 16 + B) * c->H_kv;
  const long long keys = static_cast<long long>(max_pages) * c->page_size;
  const long long bytes = keys * c->d * (in_bytes(c) ? 1 : 2);
  return items * (bytes / (kStreamTile * 256) + 10) <= 8000;
}

// How the streaming kernel runs a call: chunks of 8 query rows where a sequence's rows of
// one KV head fill no more, else 16; `items` clusters of `cluster` CTAs, one for each
// (sequence, KV head, chunk), or 0 where the units are dealt out instead.
//
// More CTAs of a cluster shorten an item's run of tiles but join longer and share the
// SMs: a cluster of c is worth twice the CTAs from 1, 3 or 6 tiles for each of c on, where
// that makes one, two or three CTAs on an SM. Clusters all run at once (with 304 CTAs in places
// for 304, clusters of 8 do not fit: 38 sequences of 100 keys, one head: 11.7 us, dealt out 6.9;
// with 264 5.3). Above 8 tiles for each CTA, dealing out evens ragged lengths better
// than it costs (20 sequences of 1 to 4096 keys, 32 heads on 4, 16 tiles each: 13.4 us,
// dealt out 11.4). Single CTAs may take two turns of 4 tiles (64 sequences of 256 keys, 32 heads on
// 8: 16.4 us, dealt out 18.1; of 1024 in 4 turns 31.9 and 29.4). Where the tensor-core kernel
// is the other choice, twice that (4 chunks of 64 behind 200 keys: 16.7 us, there 21.5).
struct StreamShape {
  int rows, cluster;
  long long items;
};
StreamShape stream_shape(const attn_paged_cache* c, int T, int B, int group, bool packed, int max_pages) {
  constexpr int n_sm = kFwdSms;
  const bool or_tensor_cores = packed && !few_rows(T, B, group);
  StreamShape s;
  s.rows = static_cast<long long>(T) * group <= 8ll * B ? 8 : 16;
  // no sequence has more than rows - 1 rows too few for its last chunk
  const long long chunks = packed ? (static_cast<long long>(T) * group + (s.rows - 1ll) * B) / s.rows
                                  : static_cast<long long>(B) * ((group + s.rows - 1) / s.rows);
  s.items = chunks * c->H_kv;
  const long long tiles = (static_cast<long long>(max_pages) * c->page_size + kStreamTile - 1) / kStreamTile;
  const long long grid = static_cast<long long>(stream_ctas(s.rows, c->d * (in_bytes(c) ? 1 : 2), c->type == kE4m3Pages)) * n_sm;
  s.cluster = 1;
  while (2 * s.cluster <= kStreamCluster && 8 * s.items * 2 * s.cluster <= 7 * grid) {
    const long long per_sm = (s.items * 2 * s.cluster + n_sm - 1) / n_sm;
    if (tiles <= s.cluster * per_sm * (per_sm + 1) / 2) break;
    s.cluster *= 2;
  }
  const long long turns = s.cluster > 1 ? 1 : (s.items + grid - 1) / grid, more = or_tensor_cores ? 2 : 1;
  if (turns > 1 + more || turns * tiles > 8 * more * s.cluster) s.cluster = 0;
  return s;
}

// Workspace of a call whatever its page table, and of one call.
size_t workspace_bytes_of(int T, int B, int group, int H_kv, int d, bool e4m3) {
  const size_t stream = stream_plan(d).total;
  if (few_rows(T, B, group)) return stream;
  const size_t fwd = fwd_plan(T, B, group, H_kv, d, e4m3).total;
  return fwd > stream ? fwd : stream;
}
size_t workspace_of_call(const attn_paged_cache* c, int T, int B, int group, bool packed, const StreamShape& shape) {
  if (shape.cluster > 0) return 0;
  return packed ? workspace_bytes_of(T, B, group, c->H_kv, c->d, c->type == kE4m3) : stream_plan(c->d).total;
}

int launch_stream(const HostDevice& dev, const attn_paged_cache* c, const PagedSeqs& seqs, const void* q,
                  void* o, float* lse, int H_q, int causal, float scale, uint8_t* ws, long long lse_row,
                  long long lse_head, const StreamShape& shape, cudaStream_t cs) {
  const unsigned rows = c->page_size < kStreamTile ? c->page_size : kStreamTile;
  CUtensorMap tk, tv;
  int st;
  if ((st = encode_pages_map(dev, &tk, c, c->k, c->k_page_stride, rows)) != ATTN_OK ||
      (st = encode_pages_map(dev, &tv, c, c->v, c->v_page_stride, rows)) != ATTN_OK)
    return st;
  const StreamPlan plan = stream_plan(c->d);
  StreamParams p;
  p.s = seqs;
  p.q = q;
  p.o = o;
  p.lse = lse;
  p.lse_row = lse_row;
  p.lse_head = lse_head;
  p.k_scale = c->type == kE4m3 ? c->k_scale : nullptr;
  p.v_scale = c->type == kE4m3 ? c->v_scale : nullptr;
  p.k_exp = c->type == kE4m3Pages ? c->k_exp : nullptr;
  p.v_exp = c->type == kE4m3Pages ? c->v_exp : nullptr;
  p.H_q = H_q;
  p.H_kv = c->H_kv;
  p.group = H_q / c->H_kv;
  p.causal = causal ? 1 : 0;
  p.scale_log2 = scale * kLog2e;
  p.heads = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + plan.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + plan.o_off);
  p.wait_limit = dev.wait_limit;
  p.fault = dev.fault;
  p.cluster = shape.cluster;
  p.items = shape.items;
  return launch_paged_stream(tk, tv, p, c->d, shape.rows, c->type, dev.n_sm, cs) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

int launch_fwd(const HostDevice& dev, const attn_paged_cache* c, const PagedSeqs& seqs, const void* q, void* o,
               float* lse, int H_q, int causal, float scale, uint8_t* ws, cudaStream_t cs) {
  const int group = H_q / c->H_kv;
  const bool e4m3 = c->type == kE4m3;  // fp16 queries
  const FwdPlan plan = fwd_plan(seqs.T, seqs.B, group, c->H_kv, c->d, e4m3);
  const int box = in_bytes(c) ? kTileN / 2 : kTileN;  // rows that land together
  const unsigned rows = c->page_size < box ? c->page_size : box;
  CUtensorMap tq, tk, tv;
  int st;
  const void* queries = e4m3 ? ws + plan.q16_off : q;
  if ((st = encode_rows_map(dev, &tq, queries, c->d, H_q, seqs.T, static_cast<long long>(H_q) * c->d, 64, group,
                            plan.tok_tile, e4m3, true)) != ATTN_OK ||
      (st = encode_pages_map(dev, &tk, c, c->k, c->k_page_stride, rows)) != ATTN_OK ||
      (st = encode_pages_map(dev, &tv, c, c->v, c->v_page_stride, rows)) != ATTN_OK)
    return st;
  PagedFwdParams p;
  p.s = seqs;
  p.o = o;
  p.lse = lse;
  p.H_q = H_q;
  p.H_kv = c->H_kv;
  p.group = group;
  p.d = c->d;
  p.causal = causal ? 1 : 0;
  p.tok_tile = plan.tok_tile;
  if (plan.tiles > 0x3fffffffll) return ATTN_ERR_BAD_SHAPE;
  p.split = plan.split ? 1 : 0;
  p.max_work = static_cast<int>(plan.tiles);
  p.scale_log2 = scale * kLog2e;
  p.k_scale = c->type == kE4m3 ? c->k_scale : nullptr;
  p.v_scale = c->type == kE4m3 ? c->v_scale : nullptr;
  p.k_exp = c->type == kE4m3Pages ? c->k_exp : nullptr;
  p.v_exp = c->type == kE4m3Pages ? c->v_exp : nullptr;
  p.q_up = reinterpret_cast<const float*>(ws + plan.up_off);
  p.seq_order = reinterpret_cast<int*>(ws);
  p.tile_start = p.seq_order + seqs.B;
  p.tile_ctr = p.tile_start + seqs.B + 1;
  p.rest_units = p.tile_ctr + 1;
  p.tiles = reinterpret_cast<int4*>(ws + plan.tiles_off);
  p.rest_tiles = p.tiles + 3 * kFwdListed;
  p.shares = p.rest_tiles + 3 * kFwdSms;
  p.rest_owners = reinterpret_cast<int2*>(p.shares + kFwdSms);
  p.part_ml = reinterpret_cast<float*>(ws + plan.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + plan.o_off);
  const int sms = dev.n_sm < kFwdSms ? dev.n_sm : kFwdSms;
  p.grid = plan.split ? sms : dev.n_sm < p.max_work ? dev.n_sm : p.max_work;
  p.wait_limit = dev.wait_limit;
  p.fault = dev.fault;
  if (e4m3 && launch_queries_f16(q, ws + plan.q16_off, reinterpret_cast<float*>(ws + plan.up_off),
                                 static_cast<long long>(seqs.T) * H_q, c->d, cs) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return launch_paged_fwd(tq, tk, tv, p, c->d, c->type, cs) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Both attention calls, after the checks they share.
int paged_attention(const attn_paged_cache* c, const void* q, void* o, float* lse, int T, int B, int H_q,
                    const int* seqlens, const int* kv_lens, const int* page_table, int max_pages,
                    long long table_stride, int causal, float scale, void* workspace,
                    size_t workspace_bytes, long long lse_row, long long lse_head, cudaStream_t cs,
                    long long head_stride = 0) {
  int st = check_cache(c);
  if (st != ATTN_OK) return st;
  if ((st = check_seqs(c, T, B, H_q, seqlens, kv_lens, page_table, max_pages, table_stride)) != ATTN_OK)
    return st;
  if (H_q < 1 || !std::isfinite(scale)) return ATTN_ERR_BAD_SHAPE;
  if (T == 0) return ATTN_OK;
  if (!q || !o || !lse) return ATTN_ERR_NULL_PTR;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 16)) return ATTN_ERR_ALIGNMENT;
  const int group = H_q / c->H_kv;
  const StreamShape shape = stream_shape(c, T, B, group, seqlens != nullptr, max_pages);
  const size_t need = workspace_of_call(c, T, B, group, seqlens != nullptr, shape);
  if (need > 0 && (!workspace || workspace_bytes < need)) return ATTN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return ATTN_ERR_ALIGNMENT;
  HostDevice dev;
  if ((st = host_setup(&dev)) != ATTN_OK) return st;
  PagedSeqs seqs = seqs_of(c, T, B, seqlens, kv_lens, page_table, max_pages, table_stride, dev.err);
  seqs.head_stride = head_stride;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!seqlens || few_rows(T, B, group) || shape.cluster > 0 ||
      little_work(c, T, B, group, max_pages))
    return launch_stream(dev, c, seqs, q, o, lse, H_q, causal, scale, ws, lse_row, lse_head, shape, cs);
  return launch_fwd(dev, c, seqs, q, o, lse, H_q, causal, scale, ws, cs);
}

}  // namespace

extern "C" {

int attn_paged_append(const attn_paged_cache* cache, const void* q, const void* k, const void* v,
                      void* q_out, long long q_stride, long long k_stride, long long v_stride,
                      long long q_out_stride, int T, int B, int H_q, const int* seqlens,
                      const int* kv_lens, const int* page_table, int max_pages,
                      long long table_stride, const double* inv_freq, int rotary_dim,
                      int interleaved, attn_stream_t stream) {
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if ((st = check_seqs(cache, T, B, H_q, seqlens, kv_lens, page_table, max_pages, table_stride)) != ATTN_OK)
    return st;
  const int d = cache->d;
  if (rotary_dim < 0 || rotary_dim > d || rotary_dim % 16 != 0) return ATTN_ERR_BAD_SHAPE;
  const long long kv_row = static_cast<long long>(cache->H_kv) * d, q_row = static_cast<long long>(H_q) * d;
  if (k_stride < kv_row || v_stride < kv_row || (H_q > 0 && (q_stride < q_row || q_out_stride < q_row)))
    return ATTN_ERR_BAD_SHAPE;
  if (T == 0) return ATTN_OK;
  if (!k || !v || (H_q > 0 && (!q || !q_out)) || (rotary_dim > 0 && !inv_freq)) return ATTN_ERR_NULL_PTR;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(inv_freq, 8) || ((k_stride | v_stride) & 7) || (H_q > 0 && ((q_stride | q_out_stride) & 7)))
    return ATTN_ERR_ALIGNMENT;
  HostDevice dev;
  if ((st = host_setup(&dev)) != ATTN_OK) return st;
  AppendParams p;
  p.s = seqs_of(cache, T, B, seqlens, kv_lens, page_table, max_pages, table_stride, dev.err);
  p.q = q; p.k = k; p.v = v; p.q_out = q_out;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride; p.q_out_stride = q_out_stride;
  p.k_cache = cache->k; p.v_cache = cache->v;
  p.k_page = cache->k_page_stride; p.v_page = cache->v_page_stride;
  p.e4m3 = cache->type == kE4m3 ? 1 : 0;
  p.k_scale = p.e4m3 ? cache->k_scale : nullptr;
  p.v_scale = p.e4m3 ? cache->v_scale : nullptr;
  p.k_exp = cache->type == kE4m3Pages ? cache->k_exp : nullptr;
  p.v_exp = cache->type == kE4m3Pages ? cache->v_exp : nullptr;
  p.inv_freq = inv_freq;
  p.H_q = H_q; p.H_kv = cache->H_kv; p.d = d;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved ? 1 : 0;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->type == kE4m3Pages) {
    CUtensorMap tk, tv;
    if (append_by_rows(p.s)) {
      // tensor maps hold strides below 2^40 bytes
      if (k_stride >= (1ll << 39) || v_stride >= (1ll << 39)) return ATTN_ERR_BAD_SHAPE;
      const int heads = append_box_heads(p.H_kv, d);
      if ((st = encode_rows_map(dev, &tk, k, d, p.H_kv, T, k_stride, d, heads, kAppendRows, false, false)) != ATTN_OK ||
          (st = encode_rows_map(dev, &tv, v, d, p.H_kv, T, v_stride, d, heads, kAppendRows, false, false)) != ATTN_OK)
        return st;
    }
    e = launch_paged_append_pages(p, tk, tv, dev.wait_limit, cs);
  } else {
    e = launch_paged_append(p, cs);
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

size_t attn_paged_decode_workspace_bytes(int d) { return d == 64 || d == 128 ? stream_plan(d).total : 0; }

size_t attn_paged_fwd_workspace_bytes(int T, int B, int H_q, int H_kv, int d, int type) {
  if (T < 0 || B < 0 || H_q < 1 || H_kv < 1 || H_q > 65535 || H_q % H_kv != 0 || (d != 64 && d != 128) ||
      (type != kBf16 && type != kE4m3 && type != kE4m3Pages))
    return 0;
  return workspace_bytes_of(T, B, H_q / H_kv, H_kv, d, type == kE4m3);
}

size_t attn_paged_call_workspace_bytes(const attn_paged_cache* cache, int T, int B, int H_q, int packed, int max_pages) {
  if (check_cache(cache) != ATTN_OK || T < 1 || B < 1 || H_q < 1 || H_q > 65535 || H_q % cache->H_kv != 0 ||
      max_pages < 0 || (!packed && T != B))
    return 0;
  const int group = H_q / cache->H_kv;
  return workspace_of_call(cache, T, B, group, packed != 0, stream_shape(cache, T, B, group, packed != 0, max_pages));
}

int attn_paged_decode(const attn_paged_cache* cache, const void* q, void* o, float* lse, int B, int H_q,
                      const int* kv_lens, const int* page_table, int max_pages,
                      long long table_stride, float scale, void* workspace, size_t workspace_bytes,
                      attn_stream_t stream) {
  return paged_attention(cache, q, o, lse, B, B, H_q, nullptr, kv_lens, page_table, max_pages,
                         table_stride, 0, scale, workspace, workspace_bytes, H_q, 1,
                         reinterpret_cast<cudaStream_t>(stream));
}

int attn_paged_fwd(const attn_paged_cache* cache, const void* q, void* o, float* lse, int T, int B,
                   int H_q, const int* seqlens, const int* kv_lens, const int* page_table,
                   int max_pages, long long table_stride, int causal, float scale, void* workspace,
                   size_t workspace_bytes, attn_stream_t stream) {
  if (T > 0 && !seqlens) return ATTN_ERR_NULL_PTR;
  return paged_attention(cache, q, o, lse, T, B, H_q, seqlens, kv_lens, page_table, max_pages,
                         table_stride, causal, scale, workspace, workspace_bytes, 1, T,
                         reinterpret_cast<cudaStream_t>(stream));
}

int attn_paged_decode_lists(const attn_paged_cache* cache, const void* q, void* o, float* lse, int B, int H_q,
                            const int* kv_lens, const int* lists, int max_pages, long long list_stride,
                            long long head_stride, float scale, void* workspace, size_t workspace_bytes,
                            attn_stream_t stream) {
  if (max_pages > 0 && head_stride < max_pages) return ATTN_ERR_BAD_SHAPE;
  return paged_attention(cache, q, o, lse, B, B, H_q, nullptr, kv_lens, lists, max_pages, list_stride, 0, scale,
                         workspace, workspace_bytes, H_q, 1, reinterpret_cast<cudaStream_t>(stream), head_stride);
}

int attn_paged_bounds(const attn_paged_cache* cache, void* bounds, int T, int B, const int* seqlens,
                      const int* kv_lens, const int* page_table, int max_pages, long long table_stride,
                      attn_stream_t stream) {
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if ((st = check_seqs(cache, T, B, 0, seqlens, kv_lens, page_table, max_pages, table_stride)) != ATTN_OK) return st;
  if (T == 0) return ATTN_OK;
  if (!bounds) return ATTN_ERR_NULL_PTR;
  if (!aligned(bounds, 16)) return ATTN_ERR_ALIGNMENT;
  HostDevice dev;
  if ((st = host_setup(&dev)) != ATTN_OK) return st;
  BoundsParams p;
  p.s = seqs_of(cache, T, B, seqlens, kv_lens, page_table, max_pages, table_stride, dev.err);
  p.k = cache->k;
  p.k_page = cache->k_page_stride;
  p.k_scale = cache->type == kE4m3 ? cache->k_scale : nullptr;
  p.k_exp = cache->type == kE4m3Pages ? cache->k_exp : nullptr;
  p.bounds = bounds;
  p.H_kv = cache->H_kv;
  return launch_paged_bounds(p, cache->d, cache->type, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

int attn_paged_select(const attn_paged_cache* cache, const void* q, const void* bounds, int* pages, int* lens,
                      int T, int B, int H_q, const int* seqlens, const int* kv_lens, const int* page_table,
                      int max_pages, long long table_stride, int count, int keep_first, int keep_last,
                      attn_stream_t stream) {
  int st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if ((st = check_seqs(cache, T, B, H_q, seqlens, kv_lens, page_table, max_pages, table_stride)) != ATTN_OK)
    return st;
  if (H_q < 1 || count < 1 || keep_first < 0 || keep_last < 1 ||
      static_cast<long long>(keep_first) + keep_last > count || max_pages > kSelectPages ||
      static_cast<long long>(count) * cache->page_size > (1ll << 30))
    return ATTN_ERR_BAD_SHAPE;
  if (H_q / cache->H_kv > kTileM) return ATTN_ERR_GQA_RATIO;
  if (T == 0) return ATTN_OK;
  if (!q || !bounds || !pages || !lens) return ATTN_ERR_NULL_PTR;
  if (!aligned(q, 16) || !aligned(bounds, 16) || !aligned(pages, 4) || !aligned(lens, 4)) return ATTN_ERR_ALIGNMENT;
  HostDevice dev;
  if ((st = host_setup(&dev)) != ATTN_OK) return st;
  SelectParams p;
  p.s = seqs_of(cache, T, B, seqlens, kv_lens, page_table, max_pages, table_stride, dev.err);
  p.q = q;
  p.bounds = bounds;
  p.pages = pages;
  p.lens = lens;
  p.H_q = H_q;
  p.H_kv = cache->H_kv;
  p.group = H_q / cache->H_kv;
  p.count = count;
  p.first = keep_first;
  p.last = keep_last;
  p.wait_limit = dev.wait_limit;
  return launch_paged_select(p, cache->d, dev.n_sm, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // extern "C"
