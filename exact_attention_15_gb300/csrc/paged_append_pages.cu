// Appends new tokens to a paged e4m3 cache that has a power of two for each page and KV head:
// a stored value x stands for x 2^e. e is the smallest from kMinExp to kMaxExp with which 448 2^e reaches
// the largest finite magnitude that was written to the page and head, so finite values saturate above
// 448 2^24 = 7.5e9 alone, and none loses bits for the size of another page's or head's. Where new tokens need a larger e than the
// page has, its rows are encoded again; a power of two costs them bits only below 2^-6 of the
// stored range.
//
// A turned key is at most sqrt 2 of what it was before, so keys that are turned count with 1.5 times
// their magnitude before the turn: e is then an exact function of the inputs, whatever the
// rounding of the angles, and known before a single angle is.
//
// Few new tokens per sequence (paged_append_few_kernel): a warp for each (page, KV head, K or V)
// holds the new rows (the first 16 of 128) in registers, finds their largest magnitude, looks up what the page has, and turns,
// scales and stores; the last CTAs of the grid turn the queries, a token on 8 to 128 threads.
//
// More (paged_append_rows_kernel): a cluster for each page and 8 KV heads of 128 (16 of 64), a CTA for
// 16 rows of the page. They come to shared memory in two copies while the CTA turns its tokens'
// queries; then each tells the others its rows' largest magnitudes, and encodes them. Every byte is
// moved once; 40,000 tokens of 16 prompts (32 query and 8 KV heads of 128) take 171 us, where a copy of
// all bytes takes 133. What is left are the steps of a CTA one after the other, of which three find
// place on an SM (31 us: 15 the queries, 4 to 7 until the page is known and the copies are
// issued, 8 the rest). Measured beside it: exponents in a kernel of their own, which reads K and V
// twice, 185 (33 of them, 40 with eight loads of a thread at once, which leaves fewer CTAs on an SM);
// a copy for each row instead of a tensor map's box, and the magnitudes read from the other
// CTAs, 178; pages in registers, a warp or 128 threads for a KV head's, 218, as the angles are then
// computed for every head.
#include <type_traits>

#include "append.cuh"

namespace attn {

namespace {

constexpr int kThreads = 128;

// The largest magnitude among bf16 pairs, as a pair of bf16 bits: of all of them (infinities and
// NaN are above the numbers), or of the finite ones, which takes three times the instructions and
// is asked for where the first is not finite.
constexpr uint32_t kInfinities = 0x7f807f80u;
template <bool FINITE>
__device__ __forceinline__ uint32_t larger(uint32_t most, const uint4& x) {
  const uint32_t w[4] = {x.x & 0x7fff7fffu, x.y & 0x7fff7fffu, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu};
#pragma unroll
  for (int i = 0; i < 4; ++i) most = __vmaxu2(most, FINITE ? w[i] & ~__vcmpgeu2(w[i], kInfinities) : w[i]);
  return most;
}
template <bool FINITE>
__device__ __forceinline__ uint32_t larger(uint32_t most, const Part& x) {
  return larger<FINITE>(larger<FINITE>(most, x.a), x.b);
}
// The smallest e from kMinExp to kMaxExp with most <= 448 2^e = 1.75 2^(e + 8).
__device__ __forceinline__ int exponent_for(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return max(kMinExp, min(kMaxExp, e));
}
// Eight values times `scale` (a power of two) as e4m3.
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
  return make_uint2(pack_e4m3x2(x[0] * scale, x[1] * scale) | pack_e4m3x2(x[2] * scale, x[3] * scale) << 16,
                    pack_e4m3x2(x[4] * scale, x[5] * scale) | pack_e4m3x2(x[6] * scale, x[7] * scale) << 16);
}
// 16 elements of a row: two runs of 8, or one of 16.
__device__ __forceinline__ void store16_e4m3(uint8_t* row, int e0, int e1, const float (&x0)[8], const float (&x1)[8],
                                             float scale) {
  const uint2 a = encode8(x0, scale), b = encode8(x1, scale);
  if (e1 != e0 + 8) {
    *reinterpret_cast<uint2*>(row + e0) = a;
    *reinterpret_cast<uint2*>(row + e1) = b;
  } else {
    *reinterpret_cast<uint4*>(row + e0) = make_uint4(a.x, a.y, b.x, b.y);
  }
}
// Four stored values times `scale`, encoded again.
__device__ __forceinline__ uint32_t encode_again(uint32_t w, float scale) {
  const float2 a = f16x2_to_f32(e4m3x2_to_f16x2(w));
  const float2 b = f16x2_to_f32(e4m3x2_to_f16x2(w >> 16));
  return pack_e4m3x2(a.x * scale, a.y * scale) | pack_e4m3x2(b.x * scale, b.y * scale) << 16;
}

// page_exponent() of an exponent that this kernel may write.
__device__ __forceinline__ int plain_exponent(const uint8_t* exps, int page, int H_kv, int h) {
  return exponent_of(exps[static_cast<size_t>(page) * H_kv + h]);
}
// Re-encodes the `kept` rows of a head of a page, which are contiguous, for an exponent that is
// larger by `more`; thread `tid` of `nthreads`.
__device__ __forceinline__ void encode_kept(uint8_t* head, int kept, int d, int more, int tid, int nthreads) {
  uint4* old = reinterpret_cast<uint4*>(head);
  const int n = kept * d >> 4;
  const float scale = power_of_two(max(-126, -more));
#pragma unroll 8
  for (int i = tid; i < n; i += nthreads) {
    const uint4 w = old[i];
    old[i] = make_uint4(encode_again(w.x, scale), encode_again(w.y, scale), encode_again(w.z, scale),
                        encode_again(w.w, scale));
  }
}
// The magnitude (as 32 bits) that counts for the exponent.
__device__ __forceinline__ float counted(uint32_t most, bool turned) {
  const float top = __uint_as_float(most);
  return turned ? top * 1.5f : top;
}

// The queries' part of the grid: CTA `block` of it, 2^shift threads per token, their angles at
// cs[THREADS >> shift][64]. The first parts are loaded before the token is looked up.
template <int THREADS>
__device__ __forceinline__ void turn_queries(const AppendParams& p, int block, int shift, float2* shared_cs) {
  constexpr int kAhead = 2;
  const int W = 1 << shift, local = threadIdx.x >> shift, tid = threadIdx.x & (W - 1);
  const int t = block * (THREADS >> shift) + local;
  const PagedSeqs& s = p.s;
  float2* cs = shared_cs + local * 64;
  const int head_shift = p.d == 128 ? 3 : 2, j = tid & ((1 << head_shift) - 1);  // the same in every head
  const bool turn = 16 * j < p.rotary_dim, split = turn && !p.interleaved;
  const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + (p.rotary_dim >> 1) : 16 * j + 8;
  const int h0 = tid >> head_shift, heads = W >> head_shift;  // the first head, heads at a time
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride;
  auto load = [&](int h) {
    return Part{*reinterpret_cast<const uint4*>(src + h * p.d + e0), *reinterpret_cast<const uint4*>(src + h * p.d + e1)};
  };
  Part ahead[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (t < s.T && h0 + k * heads < p.H_q) ahead[k] = load(h0 + k * heads);
  int b = t, pos = -1;
  if (t < s.T) {
    SeqSpan span{t, 1};
    bool mine = true;
    if (s.cu_seqlens) {
      int lo = 0, hi = s.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(s.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
      }
      b = lo;
      span = seq_span(s.cu_seqlens, b, s.T, 0);
      mine = t >= span.start && t < span.start + span.len;  // else behind the last sequence
    }
    if (mine) pos = kv_len(s, b) - span.len + (t - span.start);  // < 0: padding
  }
  if (pos >= 0)
    for (int i = tid; i < p.rotary_dim >> 1; i += W)
      cs[(i & 7) * (p.rotary_dim >> 4) + (i >> 3)] = turn_at(turn_fraction(__ldg(p.inv_freq + i)), pos);
  if (W <= 32) __syncwarp(); else __syncthreads();
  if (pos < 0) return;
  float2 of[8];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) of[e] = cs[e * (p.rotary_dim >> 4) + j];
  }
  auto put = [&](const Part& w, int h) {
    float x0[8], x1[8];
    widen8(w.a, x0);
    widen8(w.b, x1);
    if (split) turn_halves(x0, x1, of);
    else if (turn) turn_neighbours(x0, x1, of);
    store8(dst + h * p.d + e0, x0);
    store8(dst + h * p.d + e1, x1);
  };
  for (int h = h0; h < p.H_q; h += kAhead * heads) {
    Part now[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) now[k] = ahead[k];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h + (k + kAhead) * heads < p.H_q) ahead[k] = load(h + (k + kAhead) * heads);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (h + k * heads < p.H_q) put(now[k], h + k * heads);
  }
}

// KP parts of 16 elements a lane are held in registers, what there is besides is read again.
template <int KP>
__global__ void __launch_bounds__(kThreads)
paged_append_few_kernel(const AppendParams p, int kv_blocks, int q_shift) {
  constexpr int kGroups = kThreads / 32;
  __shared__ float2 cs[16 * 64];
  __shared__ unsigned long long fraction[64];
  const PagedSeqs& s = p.s;
  grid_wait();
  grid_release();
  if (blockIdx.x >= static_cast<unsigned>(kv_blocks)) {
    turn_queries<kThreads>(p, blockIdx.x - kv_blocks, q_shift, cs);
    return;
  }
  if (blockIdx.x == 0) check_paged_seqs(s, threadIdx.x, kThreads);
  const int tid = threadIdx.x % 32;
  // (64-bit divisions took 0.3 us of 6.2)
  const uint32_t at = blockIdx.x * kGroups + threadIdx.x / 32, per = 2u * p.H_kv, number = at / per;
  const int which = static_cast<int>(at - number * per), h = which >> 1;
  const bool is_v = which & 1;
  TouchedPage x;
  bool live = number < touched_numbers(s.T, s.B, s.page_shift, s.cu_seqlens != nullptr) && touched_page(s, number, x);
  const int head_shift = p.d == 128 ? 3 : 2, j = tid & ((1 << head_shift) - 1);  // the same in every row
  const bool turn = !is_v && 16 * j < p.rotary_dim, split = turn && !p.interleaved;
  const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + (p.rotary_dim >> 1) : 16 * j + 8;
  int page = 0, e = kMinExp, kept = 0;
  Part held[KP];
  uint32_t most = 0;
  const __nv_bfloat16* src = nullptr;
  long long stride = 0;
  int parts = 0;
  uint8_t* exps = is_v ? p.v_exp : p.k_exp;
  auto load = [&](int i) {
    const __nv_bfloat16* row = src + (i >> head_shift) * stride;
    return Part{*reinterpret_cast<const uint4*>(row + e0), *reinterpret_cast<const uint4*>(row + e1)};
  };
  if (live) {
    stride = is_v ? p.v_stride : p.k_stride;
    src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + x.row * stride + h * p.d;
    parts = (x.hi - x.lo) << head_shift;
    page = __ldg(s.page_table + static_cast<size_t>(x.b) * s.table_stride + x.at);
    kept = x.lo & ((1 << s.page_shift) - 1);  // rows that the page holds already
#pragma unroll
    for (int k = 0; k < KP; ++k)
      if (tid + k * 32 < parts) held[k] = load(tid + k * 32);
    live = static_cast<unsigned>(page) < static_cast<unsigned>(s.num_pages);
    if (!live) {
      if (tid == 0) record_error(s.err, kErrPages);
    } else if (kept) {
      e = plain_exponent(exps, page, p.H_kv, h);
    }
#pragma unroll
    for (int k = 0; k < KP; ++k)
      if (tid + k * 32 < parts) most = larger<true>(most, held[k]);
    for (int i = tid + KP * 32; i < parts; i += 32) most = larger<true>(most, load(i));
  }
  // (every thread of the CTA comes here)
  for (int i = threadIdx.x; i < p.rotary_dim >> 1; i += kThreads) fraction[i] = turn_fraction(__ldg(p.inv_freq + i));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
  __syncthreads();
  if (!live) return;
  const int before = e;
  e = max(e, exponent_for(counted(max(most & 0xffffu, most >> 16) << 16, !is_v && p.rotary_dim > 0)));
  const long long head0 = static_cast<long long>(page) * (is_v ? p.v_page : p.k_page) +
                          (static_cast<long long>(h) << s.page_shift) * p.d;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + head0;
  if (kept && e > before) encode_kept(dst, kept, p.d, e - before, tid, 32);
  if (tid == 0 && (!kept || e != before)) exps[static_cast<size_t>(page) * p.H_kv + h] = static_cast<uint8_t>(e + 127);
  const float scale = power_of_two(-e);
  unsigned long long f[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fraction[8 * j + i];
  }
  auto put = [&](const Part& w, int i) {
    float x0[8], x1[8];
    widen8(w.a, x0);
    widen8(w.b, x1);
    const int r = i >> head_shift;
    if (turn) {
      float2 of[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) of[u] = turn_at(f[u], x.lo + r);
      if (split) turn_halves(x0, x1, of);
      else turn_neighbours(x0, x1, of);
    }
    store16_e4m3(dst + (kept + r) * p.d, e0, e1, x0, x1, scale);
  };
#pragma unroll
  for (int k = 0; k < KP; ++k)
    if (tid + k * 32 < parts) put(held[k], tid + k * 32);
  for (int i = tid + KP * 32; i < parts; i += 32) put(load(i), i);
}

// Many tokens: a cluster for each page and up to 64 KB / 16 rows of KV heads, a CTA for 16 rows. The
// rows of K and V are copied to shared memory while the CTA turns its tokens' queries; then the
// CTAs find the page's largest magnitudes together and each encodes its rows.
constexpr int kRows = kAppendRows, kRowBytes = 64 * 1024;
struct RowsShared {
  uint32_t most[64];  // of the page's new rows: the KV heads' keys, then their values
  int before[64], e[64];
  uint64_t full;
  int4 found;  // position of the page's first new token, new tokens, sequence, place in its table row
  int row;     // of the first
};

template <int kRowThreads>
__global__ void __launch_bounds__(kRowThreads, 768 / kRowThreads)
paged_append_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const AppendParams p, int cluster_shift, int heads, int groups, int q_shift, long long wait_limit) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RowsShared sh;
  const PagedSeqs& s = p.s;
  const int tid = threadIdx.x, cluster = 1 << cluster_shift, rank = blockIdx.x & (cluster - 1);
  const int block = blockIdx.x >> cluster_shift, number = block / groups, group = block - number * groups;
  const int h0 = group * heads, n_heads = min(heads, p.H_kv - h0);
  const int head_shift = p.d == 128 ? 3 : 2;  // log2(16-element parts of a head)
  const uint32_t bar = smem_addr(&sh.full);
  if (tid == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (tid < 64) sh.most[tid] = 0;
  __syncthreads();
  if (cluster > 1) cluster_arrive();  // (ready for the others' magnitudes)
  grid_wait();
  grid_release();
  if (blockIdx.x == 0) check_paged_seqs(s, tid, kRowThreads);
  // ---- the page, and copies of this CTA's rows of `heads` heads, K and then V (what lies behind
  // the page's rows or the heads comes along and is not used)
  const uint32_t row_bytes = static_cast<uint32_t>(heads) * p.d * 2, v_off = kRows * row_bytes;
  if (tid < 32) {
    TouchedPage x;
    const bool some = touched_page(s, number, x);
    const int n = some ? max(0, min(kRows, x.hi - x.lo - rank * kRows)) : 0;
    if (tid == 0) {
      sh.found = make_int4(x.lo, some ? x.hi - x.lo : 0, x.b, x.at);
      sh.row = x.row;
      if (n > 0) {
        mbar_arrive_expect_tx(bar, 2 * v_off);
        tma_load_3d(smem_addr(smem), &tm_k, bar, 0, h0, x.row + rank * kRows);
        tma_load_3d(smem_addr(smem) + v_off, &tm_v, bar, 0, h0, x.row + rank * kRows);
      }
    }
  }
  __syncthreads();
  if (sh.found.y == 0) {  // no page of that number: the whole cluster leaves
    if (cluster > 1) cluster_wait();
    return;
  }
  const int lo = sh.found.x + rank * kRows, n = max(0, min(kRows, sh.found.y - rank * kRows));
  const int kept = sh.found.x & ((1 << s.page_shift) - 1);  // rows that the page holds already
  const int page = page_entry(s, sh.found.z, sh.found.w);
  const bool page_ok = static_cast<unsigned>(page) < static_cast<unsigned>(s.num_pages);
  if (!page_ok && tid == 0) record_error(s.err, kErrPages);
  if (tid < 2 * n_heads)
    sh.before[tid] = kept && page_ok ? plain_exponent(tid < n_heads ? p.k_exp : p.v_exp, page, p.H_kv,
                                                      h0 + (tid < n_heads ? tid : tid - n_heads))
                                     : kMinExp;
  // ---- angles
  const int pairs = p.rotary_dim >> 1, j_count = p.rotary_dim >> 4;
  float2* angles = reinterpret_cast<float2*>(smem + 2 * v_off);  // [row][e][part]
  if (pairs) {  // (a thread has one frequency and every so many rows)
    const int step = kRowThreads / pairs, r0 = tid / pairs, place = tid - r0 * pairs, e = place / j_count;
    if (r0 < step) {
      const unsigned long long f = turn_fraction(__ldg(p.inv_freq + 8 * (place - e * j_count) + e));
      for (int r = r0; r < n; r += step) angles[r * pairs + place] = turn_at(f, lo + r);
    }
  }
  __syncthreads();
  // ---- queries: 2^q_shift threads a token, this group's share of the heads
  if (p.H_q > 0) {
    const int W = 1 << q_shift, i0 = tid & (W - 1), j = i0 & ((1 << head_shift) - 1);
    const bool turn = 16 * j < p.rotary_dim, split = turn && !p.interleaved;
    const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + (p.rotary_dim >> 1) : 16 * j + 8;
    const int share = (p.H_q + groups - 1) / groups, h_end = min(p.H_q, (group + 1) * share);
    const long long t0 = sh.row + rank * kRows;
    // four tokens' parts are loaded before the first is stored (q_out may be q)
    constexpr int kAhead = 4;
    const int step = kRowThreads >> q_shift;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + t0 * p.q_stride;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t0 * p.q_out_stride;
    for (int h = group * share + (i0 >> head_shift); h < h_end; h += W >> head_shift)
      for (int r0 = tid >> q_shift; r0 < n; r0 += kAhead * step) {
        Part w[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const __nv_bfloat16* at = src + min(r0 + k * step, n - 1) * p.q_stride + h * p.d;
          w[k] = Part{*reinterpret_cast<const uint4*>(at + e0), *reinterpret_cast<const uint4*>(at + e1)};
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int r = r0 + k * step;
          if (r >= n) break;
          float x0[8], x1[8];
          widen8(w[k].a, x0);
          widen8(w[k].b, x1);
          if (turn) {
            float2 of[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) of[e] = angles[r * pairs + e * j_count + j];
            if (split) turn_halves(x0, x1, of);
            else turn_neighbours(x0, x1, of);
          }
          __nv_bfloat16* to = dst + r * p.q_out_stride + h * p.d;
          store8(to + e0, x0);
          store8(to + e1, x1);
        }
      }
  }
  // ---- the largest magnitudes: a thread has a 16-byte column of the rows
  bool ok = n == 0 || mbar_wait(bar, 0, wait_limit);
  if (!ok) {
    // the copies may still be on their way: once more, then the rows are not written
    record_error(s.err, kErrTimeout);
    mbar_wait(bar, 0, wait_limit);
  }
  ok = !__syncthreads_or(!ok);
  if (cluster > 1) cluster_wait();
  const int cols = n_heads << (head_shift + 2);  // of K and of V
  for (int col0 = 0; col0 < cols; col0 += kRowThreads) {
    const int col = col0 + tid, in_half = col >= cols >> 1 ? col - (cols >> 1) : col;
    const uint8_t* at = smem + (col >= cols >> 1 ? v_off : 0) + in_half * 16;
    uint32_t most = 0;
    auto look = [&](auto finite) {
      most = 0;
      if (col < cols) {
#pragma unroll 4
        for (int r = 0; r < n; ++r)
          most = larger<decltype(finite)::value>(most, *reinterpret_cast<const uint4*>(at + r * row_bytes));
      }
    };
    look(std::false_type{});
    if (__vcmpgeu2(most, kInfinities)) look(std::true_type{});
    // (a head's columns are 8 or 16 lanes of a warp)
    for (int o = 1; o < 2 << head_shift; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
    // each of its lanes tells one CTA of the cluster, so that nobody has to ask
    const int to = col & ((2 << head_shift) - 1);
    if (col < cols && n > 0)
      for (int r = to; r < cluster; r += 2 << head_shift)
        max_cluster_u32(cluster_map(smem_addr(&sh.most[col >> (head_shift + 1)]), r), max(most & 0xffffu, most >> 16) << 16);
  }
  if (cluster > 1) cluster_sync_all(); else __syncthreads();
  // ---- exponents
  if (tid < 2 * n_heads) {
    const bool is_v = tid >= n_heads;
    sh.e[tid] = max(sh.before[tid], exponent_for(counted(sh.most[tid], !is_v && p.rotary_dim > 0)));
    if (rank == 0 && page_ok && (!kept || sh.e[tid] != sh.before[tid]))
      (is_v ? p.v_exp : p.k_exp)[static_cast<size_t>(page) * p.H_kv + h0 + (is_v ? tid - n_heads : tid)] =
          static_cast<uint8_t>(sh.e[tid] + 127);
  }
  __syncthreads();
  if (page_ok && ok) {
    const long long k_at = static_cast<long long>(page) * p.k_page + (static_cast<long long>(h0) << s.page_shift) * p.d;
    const long long v_at = static_cast<long long>(page) * p.v_page + (static_cast<long long>(h0) << s.page_shift) * p.d;
    const int head_bytes = p.d << s.page_shift;
    if (kept && rank == 0) {
      for (int i = 0; i < 2 * n_heads; ++i)
        if (sh.e[i] > sh.before[i])
          encode_kept(i < n_heads ? static_cast<uint8_t*>(p.k_cache) + k_at + i * head_bytes
                                  : static_cast<uint8_t*>(p.v_cache) + v_at + (i - n_heads) * head_bytes,
                      kept, p.d, sh.e[i] - sh.before[i], tid, kRowThreads);
    }
    // ---- the new rows: a thread has a part of 16 elements of every so many
    const int parts = 2 * n_heads << head_shift, at_once = kRowThreads / parts;  // (128 parts at most)
    const int r0 = tid / parts, part = tid - r0 * parts, head = part >> head_shift, j = part & ((1 << head_shift) - 1);
    const bool is_v = head >= n_heads;
    const bool turn = !is_v && 16 * j < p.rotary_dim, split = turn && !p.interleaved;
    const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + (p.rotary_dim >> 1) : 16 * j + 8;
    const uint8_t* from = smem + (is_v ? v_off + (head - n_heads) * p.d * 2 : head * p.d * 2);
    uint8_t* to = (is_v ? static_cast<uint8_t*>(p.v_cache) + v_at + (head - n_heads) * head_bytes
                        : static_cast<uint8_t*>(p.k_cache) + k_at + head * head_bytes) +
                  (kept + rank * kRows) * p.d;
    const float scale = r0 < at_once ? power_of_two(-sh.e[head]) : 0.0f;
#pragma unroll 2
    for (int r = r0; r0 < at_once && r < n; r += at_once) {
      float x0[8], x1[8];
      widen8(*reinterpret_cast<const uint4*>(from + r * row_bytes + e0 * 2), x0);
      widen8(*reinterpret_cast<const uint4*>(from + r * row_bytes + e1 * 2), x1);
      if (turn) {
        float2 of[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) of[e] = angles[r * pairs + e * j_count + j];
        if (split) turn_halves(x0, x1, of);
        else turn_neighbours(x0, x1, of);
      }
      store16_e4m3(to + r * p.d, e0, e1, x0, x1, scale);
    }
  }
}

// Threads of a token's queries, as a power of two: all for few tokens, else about four parts a thread.
int query_shift(const AppendParams& p) {
  const int parts = p.H_q * (p.d >> 4);
  int shift = 7;
  if (p.s.T >= 304)
    for (shift = 3; shift < 7 && (1 << shift) < (parts + 3) / 4;) ++shift;
  return shift;
}

template <int KP>
cudaError_t launch_few(const AppendParams& p, cudaStream_t stream) {
  const long long units = touched_numbers(p.s.T, p.s.B, p.s.page_shift, p.s.cu_seqlens != nullptr) * 2 * p.H_kv;
  const long long kv_blocks = (units * 32 + kThreads - 1) / kThreads;
  const int q_shift = query_shift(p), tokens = kThreads >> q_shift;
  const long long q_blocks = p.H_q > 0 ? (p.s.T + tokens - 1) / tokens : 0;
  if (units > 0x7fffffffll || kv_blocks + q_blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const int slot = prof_begin(kKPagedAppend, stream);
  const cudaError_t e = launch_chained<paged_append_few_kernel<KP>>(
      dim3(static_cast<unsigned>(kv_blocks + q_blocks)), kThreads, 0, stream, p, static_cast<int>(kv_blocks), q_shift);
  prof_end(slot, stream);
  return e;
}

cudaError_t launch_rows(const AppendParams& p, const CUtensorMap& tk, const CUtensorMap& tv, long long wait_limit,
                        cudaStream_t stream) {
  const int heads = append_box_heads(p.H_kv, p.d), groups = (p.H_kv + heads - 1) / heads;
  const int cluster_shift = p.s.page_shift - 4;  // a CTA for 16 rows
  const long long ctas = touched_numbers(p.s.T, p.s.B, p.s.page_shift, true) * groups << cluster_shift;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  const int smem = kRows * heads * p.d * 4 + kRows * (p.rotary_dim / 2) * 8;
  const int slot = prof_begin(kKPagedAppend, stream);
  auto with = [&](auto threads) {
    constexpr int kThreadsOf = decltype(threads)::value;
    // a token's query parts of a group, one or a few a thread
    const int parts = (p.H_q + groups - 1) / groups * (p.d >> 4);
    int q_shift = 3;
    while ((2 << q_shift) <= kThreadsOf && (2 << q_shift) <= parts) ++q_shift;
    cudaError_t e = allow_smem<paged_append_rows_kernel<kThreadsOf>>(kRowBytes + kRows * 64 * 8);
    if (e == cudaSuccess) e = allow_wide_clusters<paged_append_rows_kernel<kThreadsOf>>();
    if (e != cudaSuccess) return e;
    return launch_clusters<paged_append_rows_kernel<kThreadsOf>>(1 << cluster_shift, dim3(static_cast<unsigned>(ctas)),
                                                                 kThreadsOf, smem, stream, tk, tv, p, cluster_shift, heads,
                                                                 groups, q_shift, wait_limit);
  };
  // 12 parts of 16 elements a thread at least (25,000 tokens with 2 query and 2 KV heads of 128, 768
  // parts: 27.1 us with 256 threads, 23.8 with 64; 750 with 8 and 4, 2048 parts: 5.2 us with 256,
  // 6.3 with 128), and a thread at least for each part of a row of K and V.
  const int row = 2 * heads * (p.d >> 4), all = kRows * ((p.H_q + groups - 1) / groups * (p.d >> 4) + row);
  const cudaError_t e = all <= 12 * 64 && row <= 64     ? with(std::integral_constant<int, 64>{})
                        : all <= 12 * 128 && row <= 128 ? with(std::integral_constant<int, 128>{})
                                                        : with(std::integral_constant<int, 256>{});
  prof_end(slot, stream);
  return e;
}

}  // namespace

// By rows where the sequences have more than 24 new tokens on the mean. By rows a sequence's pages cost
// clusters that are mostly empty, with a warp for each page and head the angles are computed for every head and
// rows beyond the 16 that it holds are read twice. us with few / by rows, 48 sequences, 32 query and 8 KV heads
// of 128: 17 tokens in pages of 64 8.1 / 18.9, 24 in pages of 16 8.6 / 14.5, 32 in pages of 64 12.5 / 22.6 and
// without queries 11.0 / 11.4, 64 21.7 / 26.1 and 19.9 / 12.4, 128 in pages of 256 51 / 70 and 40 / 34. One KV
// head of 128 without queries, pages of 32: 17 tokens 6.3 / 6.0, 32 7.6 / 6.0; 4 sequences of 256 tokens in
// pages of 128 30 / 14. So 24 is where neither costs more than 4%. A prompt of 4000 tokens beside 200 single
// ones, which the mean sends the first way, 25 / 36; beside 100, which it sends the second, 26 / 27.
bool append_by_rows(const PagedSeqs& s) { return s.cu_seqlens && s.T > 24ll * s.B; }
int append_box_heads(int H_kv, int d) {
  const int most = kRowBytes / (kRows * 4 * d), groups = (H_kv + most - 1) / most;  // 8 of 128, 16 of 64
  return (H_kv + groups - 1) / groups;
}

cudaError_t launch_paged_append_pages(const AppendParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                                      long long wait_limit, cudaStream_t stream) {
  if (append_by_rows(p.s)) return launch_rows(p, tk, tv, wait_limit, stream);
  return p.s.cu_seqlens ? launch_few<4>(p, stream) : launch_few<1>(p, stream);
}

}  // namespace attn
