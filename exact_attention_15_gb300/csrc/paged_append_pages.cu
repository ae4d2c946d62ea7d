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
// Work is dealt out by (page, KV head, K or V): W threads hold the new rows of one in registers,
// find their largest magnitude, look up what the page has, and turn, scale and store. The last
// CTAs of the grid turn the queries, a token on 8 to 128 threads as in paged_append.cu.
#include "append.cuh"

namespace attn {

namespace {

constexpr int kThreads = 128;

// The largest finite magnitude among bf16 pairs, as a pair of bf16 bits.
__device__ __forceinline__ uint32_t larger(uint32_t most, uint32_t pair) {
  const uint32_t size = pair & 0x7fff7fffu;
  return __vmaxu2(most, size & ~__vcmpgeu2(size, 0x7f807f80u));
}
__device__ __forceinline__ uint32_t larger(uint32_t most, const Part& x) {
  const uint32_t w[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) most = larger(most, w[i]);
  return most;
}
// The smallest e from -kMaxExp to kMaxExp with most <= 448 2^e = 1.75 2^(e + 8).
__device__ __forceinline__ int exponent_for(float most) {
  const uint32_t bits = __float_as_uint(most);
  const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
  return max(-kMaxExp, min(kMaxExp, e));
}
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float scale) {
  return make_uint2(pack_e4m3x2(x[0] * scale, x[1] * scale) | pack_e4m3x2(x[2] * scale, x[3] * scale) << 16,
                    pack_e4m3x2(x[4] * scale, x[5] * scale) | pack_e4m3x2(x[6] * scale, x[7] * scale) << 16);
}
// Four stored values times `scale`, encoded again.
__device__ __forceinline__ uint32_t encode_again(uint32_t w, float scale) {
  const float2 a = f16x2_to_f32(e4m3x2_to_f16x2(w));
  const float2 b = f16x2_to_f32(e4m3x2_to_f16x2(w >> 16));
  return pack_e4m3x2(a.x * scale, a.y * scale) | pack_e4m3x2(b.x * scale, b.y * scale) << 16;
}

// The queries' part of the grid: CTA `block` of it, 2^shift threads per token.
__device__ __forceinline__ void turn_queries(const AppendParams& p, int block, int shift,
                                             float2 (*shared_cs)[64]) {
  const int W = 1 << shift, local = threadIdx.x >> shift, tid = threadIdx.x & (W - 1);
  const int t = block * (kThreads >> shift) + local;
  const PagedSeqs& s = p.s;
  float2* cs = shared_cs[local];
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
  const int head_shift = p.d == 128 ? 3 : 2, j = tid & ((1 << head_shift) - 1);  // the same in every head
  const bool turn = 16 * j < p.rotary_dim, split = turn && !p.interleaved;
  const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + (p.rotary_dim >> 1) : 16 * j + 8;
  float2 of[8];
  if (turn) {
#pragma unroll
    for (int e = 0; e < 8; ++e) of[e] = cs[e * (p.rotary_dim >> 4) + j];
  }
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride;
  const int heads = W >> head_shift;  // at a time
#pragma unroll 4
  for (int h = tid >> head_shift; h < p.H_q; h += heads) {
    float x0[8], x1[8];
    widen8(*reinterpret_cast<const uint4*>(src + h * p.d + e0), x0);
    widen8(*reinterpret_cast<const uint4*>(src + h * p.d + e1), x1);
    if (split) turn_halves(x0, x1, of);
    else if (turn) turn_neighbours(x0, x1, of);
    store8(dst + h * p.d + e0, x0);
    store8(dst + h * p.d + e1, x1);
  }
}

// KP parts of 16 elements a thread are held in registers, what there is besides is read again.
template <int W, int KP>
__global__ void __launch_bounds__(kThreads)
paged_append_pages_kernel(const AppendParams p, int kv_blocks, int q_shift) {
  constexpr int kGroups = kThreads / W;
  __shared__ float2 cs[16][64];
  __shared__ unsigned long long fraction[64];
  __shared__ uint32_t warp_most[kThreads / 32];
  const PagedSeqs& s = p.s;
  grid_wait();
  grid_release();
  if (blockIdx.x >= static_cast<unsigned>(kv_blocks)) {
    turn_queries(p, blockIdx.x - kv_blocks, q_shift, cs);
    return;
  }
  if (blockIdx.x == 0) check_paged_seqs(s, threadIdx.x, kThreads);
  const int tid = threadIdx.x % W;
  const long long at = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / W;
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
      if (tid + k * W < parts) held[k] = load(tid + k * W);
    live = static_cast<unsigned>(page) < static_cast<unsigned>(s.num_pages);
    if (!live) {
      if (tid == 0) record_error(s.err, kErrPages);
    } else if (kept) {
      e = page_exponent(exps, page, p.H_kv, h);
    }
#pragma unroll
    for (int k = 0; k < KP; ++k)
      if (tid + k * W < parts) most = larger(most, held[k]);
    for (int i = tid + KP * W; i < parts; i += W) most = larger(most, load(i));
  }
  // (every thread of the CTA comes here)
  for (int i = threadIdx.x; i < p.rotary_dim >> 1; i += kThreads) fraction[i] = turn_fraction(__ldg(p.inv_freq + i));
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (W > 32 && threadIdx.x % 32 == 0) warp_most[threadIdx.x / 32] = most;
  __syncthreads();
  if (!live) return;
  if (W > 32) {
#pragma unroll
    for (int w = 0; w < W / 32; ++w) most = __vmaxu2(most, warp_most[w]);
  }
  const float top = __uint_as_float(max(most & 0xffffu, most >> 16) << 16);
  const int before = e;
  e = max(e, exponent_for(!is_v && p.rotary_dim > 0 ? top * 1.5f : top));
  const long long head0 = static_cast<long long>(page) * (is_v ? p.v_page : p.k_page) +
                          (static_cast<long long>(h) << s.page_shift) * p.d;
  uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + head0;
  if (kept && e > before) {
    // the rows that are there: the head's are contiguous
    uint4* old = reinterpret_cast<uint4*>(dst);
    const int n = kept * p.d >> 4;
    const float scale = power_of_two(max(-126, before - e));
#pragma unroll 4
    for (int i = tid; i < n; i += W) {
      const uint4 w = old[i];
      old[i] = make_uint4(encode_again(w.x, scale), encode_again(w.y, scale), encode_again(w.z, scale),
                          encode_again(w.w, scale));
    }
  }
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
    uint8_t* to = dst + (kept + r) * p.d;
    const uint2 a = encode8(x0, scale), b = encode8(x1, scale);
    if (split) {
      *reinterpret_cast<uint2*>(to + e0) = a;
      *reinterpret_cast<uint2*>(to + e1) = b;
    } else {
      *reinterpret_cast<uint4*>(to + e0) = make_uint4(a.x, a.y, b.x, b.y);
    }
  };
#pragma unroll
  for (int k = 0; k < KP; ++k)
    if (tid + k * W < parts) put(held[k], tid + k * W);
  for (int i = tid + KP * W; i < parts; i += W) put(load(i), i);
}

template <int W, int KP>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  const long long units = touched_numbers(p.s.T, p.s.B, p.s.page_shift, p.s.cu_seqlens != nullptr) * 2 * p.H_kv;
  const long long kv_blocks = (units * W + kThreads - 1) / kThreads;
  // queries: all threads for few tokens, else about four parts a thread
  const int parts = p.H_q * (p.d >> 4);
  int q_shift = 7;
  if (p.s.T >= 304)
    for (q_shift = 3; q_shift < 7 && (1 << q_shift) < (parts + 3) / 4;) ++q_shift;
  const int tokens = kThreads >> q_shift;
  const long long q_blocks = p.H_q > 0 ? (p.s.T + tokens - 1) / tokens : 0;
  if (kv_blocks + q_blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_chained<paged_append_pages_kernel<W, KP>>(dim3(static_cast<unsigned>(kv_blocks + q_blocks)), kThreads, 0,
                                                           stream, p, static_cast<int>(kv_blocks), q_shift);
}

}  // namespace

cudaError_t launch_paged_append_pages(const AppendParams& p, cudaStream_t stream) {
  const int slot = prof_begin(kKPagedAppend, stream);
  // the new rows of a page at most
  const int page = 1 << p.s.page_shift;
  const int rows = !p.s.cu_seqlens ? 1 : page < p.s.T ? page : p.s.T, parts = rows * (p.d >> 4);
  const cudaError_t e = parts <= 32    ? launch<32, 1>(p, stream)
                        : parts <= 128 ? launch<32, 4>(p, stream)
                        : parts <= 512 ? launch<128, 4>(p, stream)
                                       : launch<128, 8>(p, stream);
  prof_end(slot, stream);
  return e;
}

}  // namespace attn
