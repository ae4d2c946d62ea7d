// Appends new tokens to a paged e4m3 cache that has a power of two for each page and KV head:
// a stored value x stands for x 2^e. e is the smallest with which 448 2^e reaches the largest
// finite magnitude that was written to the page and head, so nothing saturates and no value
// loses bits for the size of another page's or head's. Where new tokens need a larger e than the
// page has, its rows are encoded again; a power of two costs them bits only below 2^-6 of the
// stored range.
//
// A turned key is at most sqrt 2 of what it was before, so keys that are turned count with 1.5 times
// their magnitude before the turn: e is then an exact function of the inputs, whatever the
// rounding of the angles, and known before a single angle is.
//
// Few new tokens per sequence (paged_append_few_kernel): a warp for each (page, KV head, K or V)
// holds the new rows in registers, finds their largest magnitude, looks up what the page has, and turns,
// scales and stores; the last CTAs of the grid turn the queries, a token on 8 to 128 threads.
//
// More: the exponents first (paged_append_exps_kernel), which reads the new keys and values once more
// than there is need, then the tokens as over the other caches (paged_append.cu). 40,000 tokens of 16
// prompts (32 query and 8 KV heads of 128): 31 us and 153, where a plain copy of all bytes takes 133; with
// the rows of a page in shared memory between both, which reads them once, 189 to 216 (the angles are
// then computed for every few heads, and what waits for a page's largest value keeps few CTAs busy).
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
// The smallest e from -kMaxExp to kMaxExp with most <= 448 2^e = 1.75 2^(e + 8).
__device__ __forceinline__ int exponent_for(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return max(-kMaxExp, min(kMaxExp, e));
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
  const int e = static_cast<int>(exps[static_cast<size_t>(page) * H_kv + h]) - 127;
  return max(-kMaxExp, min(kMaxExp, e));
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
  const long long at = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / 32;
  const int which = static_cast<int>(at % (2 * p.H_kv));
  const int h = which >> 1;
  const bool is_v = which & 1;
  TouchedPage x;
  bool live = at / (2 * p.H_kv) < touched_numbers(s.T, s.B, s.page_shift, s.cu_seqlens != nullptr) &&
              touched_page(s, at / (2 * p.H_kv), x);
  const int head_shift = p.d == 128 ? 3 : 2, j = tid & ((1 << head_shift) - 1);  // the same in every row
  const bool turn = !is_v && 16 * j < p.rotary_dim, split = turn && !p.interleaved;
  const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + (p.rotary_dim >> 1) : 16 * j + 8;
  int page = 0, e = -kMaxExp, kept = 0;
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

// The exponents alone, for calls of many tokens: a CTA for each page, 2^heads_shift KV heads and K or
// V reads the new rows, a 16-byte column a thread, and encodes the page's other rows again.
constexpr int kExpThreads = 256, kExpHeads = 32;
__global__ void __launch_bounds__(kExpThreads)
paged_append_exps_kernel(const AppendParams p, int heads_shift) {
  __shared__ uint32_t most_of[kExpHeads];
  const PagedSeqs& s = p.s;
  const int tid = threadIdx.x, heads = 1 << heads_shift, groups = (p.H_kv + heads - 1) >> heads_shift;
  const int col_shift = p.d == 128 ? 4 : 3;  // log2(16-byte columns of a head)
  if (tid < kExpHeads) most_of[tid] = 0;
  grid_wait();
  grid_release();
  if (blockIdx.x == 0) check_paged_seqs(s, tid, kExpThreads);
  // K and V, then the groups of heads innermost: neighbours read neighbouring columns
  const int number = blockIdx.x / (2 * groups), which = blockIdx.x - number * 2 * groups;
  const bool is_v = which >= groups;
  const int h0 = (is_v ? which - groups : which) << heads_shift, n_heads = min(heads, p.H_kv - h0);
  TouchedPage x;
  if (!touched_page(s, number, x)) return;
  const int page = __ldg(s.page_table + static_cast<size_t>(x.b) * s.table_stride + x.at);
  const int cols = heads << col_shift, col = tid & (cols - 1), step = kExpThreads / cols;
  const int col_head = col >> col_shift, rows = x.hi - x.lo, row0 = tid / cols;
  const long long stride = is_v ? p.v_stride : p.k_stride;
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(is_v ? p.v : p.k) + x.row * stride + h0 * p.d + col * 8;
  uint32_t most = 0;
  auto look = [&](auto finite) {
    most = 0;
    if (col_head < n_heads) {
      constexpr int kAtOnce = 8;  // (all loads before the first is used)
      for (int r0 = row0; r0 < rows; r0 += kAtOnce * step) {
        uint4 w[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
          w[k] = make_uint4(0u, 0u, 0u, 0u);
          if (r0 + k * step < rows)
            asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[k].x), "=r"(w[k].y), "=r"(w[k].z), "=r"(w[k].w) : "l"(src + (r0 + k * step) * stride));
        }
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) most = larger<decltype(finite)::value>(most, w[k]);
      }
    }
  };
  look(std::false_type{});
  if (__vcmpgeu2(most, kInfinities)) look(std::true_type{});
  for (int o = 1; o < 1 << col_shift; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
  __syncthreads();
  if ((col & ((1 << col_shift) - 1)) == 0 && col_head < n_heads)
    atomicMax(&most_of[col_head], max(most & 0xffffu, most >> 16) << 16);
  __syncthreads();
  // (a bad index is recorded where the tokens are written)
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(s.num_pages)) return;
  const bool turned = !is_v && p.rotary_dim > 0;
  const int kept = x.lo & ((1 << s.page_shift) - 1);
  uint8_t* exps = is_v ? p.v_exp : p.k_exp;
  int before = -kMaxExp;
  if (kept) {
    uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                   static_cast<long long>(page) * (is_v ? p.v_page : p.k_page) +
                   (static_cast<long long>(h0) << s.page_shift) * p.d;
    for (int h = 0; h < n_heads; ++h) {
      const int was = plain_exponent(exps, page, p.H_kv, h0 + h), is = max(was, exponent_for(counted(most_of[h], turned)));
      if (is > was) encode_kept(dst + (h * p.d << s.page_shift), kept, p.d, is - was, tid, kExpThreads);
    }
    if (tid < n_heads) before = plain_exponent(exps, page, p.H_kv, h0 + tid);
    __syncthreads();  // (everyone has read the exponents)
  }
  if (tid < n_heads) {
    const int e = max(before, exponent_for(counted(most_of[tid], turned)));
    if (!kept || e != before) exps[static_cast<size_t>(page) * p.H_kv + h0 + tid] = static_cast<uint8_t>(e + 127);
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
  if (kv_blocks + q_blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const int slot = prof_begin(kKPagedAppend, stream);
  const cudaError_t e = launch_chained<paged_append_few_kernel<KP>>(
      dim3(static_cast<unsigned>(kv_blocks + q_blocks)), kThreads, 0, stream, p, static_cast<int>(kv_blocks), q_shift);
  prof_end(slot, stream);
  return e;
}

cudaError_t launch_many(const AppendParams& p, cudaStream_t stream) {
  // heads for a quarter of the threads: 4 of 128, 8 of 64
  int shift = 0;
  while ((1 << shift) < p.H_kv && (2 << shift) * p.d <= kExpThreads * 2) ++shift;
  const int groups = (p.H_kv + (1 << shift) - 1) >> shift;
  const long long blocks = touched_numbers(p.s.T, p.s.B, p.s.page_shift, true) * 2 * groups;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const int slot = prof_begin(kKPagedAppend, stream);
  const cudaError_t e =
      launch_chained<paged_append_exps_kernel>(dim3(static_cast<unsigned>(blocks)), kExpThreads, 0, stream, p, shift);
  prof_end(slot, stream);
  return e == cudaSuccess ? launch_paged_append(p, stream) : e;
}

}  // namespace

cudaError_t launch_paged_append_pages(const AppendParams& p, cudaStream_t stream) {
  // Up to 16 new tokens of each sequence on the mean a warp has them in registers.
  if (!p.s.cu_seqlens) return launch_few<1>(p, stream);
  return p.s.T <= 16ll * p.s.B ? launch_few<4>(p, stream) : launch_many(p, stream);
}

}  // namespace attn
