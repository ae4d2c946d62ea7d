// Appends new tokens to a paged key-value cache, with the rotary position
// embedding of queries and keys applied on the way.
//
// A pair (a, b) of a query or key at position p turns into
// (a cos t - b sin t, a sin t + b cos t) with t = p * inv_freq[i]. Far positions
// make t large (10^6 radians at a million tokens), where 32-bit products lose
// the angle: the turn count p * inv_freq / 2 pi is kept as a 64-bit binary
// fraction, whose integer product with p drops whole turns exactly; its top 24
// bits after that are the angle.
#include "paged.cuh"

namespace attn {

namespace {

constexpr int kAppendThreads = 128;

__device__ __forceinline__ void widen8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(u[i]);
    x[2 * i + 1] = bf16hi_to_f32(u[i]);
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// Two values to e4m3, nearest-even, what lies beyond 448 to 448 (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// x / s, rounded to nearest, from the rounded inverse of s: the product's residual
// corrects it (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990). The product stands where the residual is no number to
// correct with: NaN for an infinite or NaN x, an infinity where x is finite and the product
// passes 32 bits (3e38 by 0.5), whose correction would be the NaN inf - inf. The inverse
// alone would now and then land on the other side of a rounding border of e4m3; a division
// per value cost a sixth of the kernel's time over an e4m3 cache.
__device__ __forceinline__ float quotient(float x, float s, float inverse) {
  const float q = x * inverse, r = __fmaf_rn(-q, s, x);
  return fabsf(r) < INFINITY ? __fmaf_rn(r, inverse, q) : q;
}
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&x)[8], float scale, float inverse) {
  float y[8];
  // (an inverse outside the normal numbers cannot be corrected)
  const float size = fabsf(scale);
  if (size > 1e-30f && size < 1e30f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = quotient(x[i], scale, inverse);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], scale);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_e4m3x2(y[0], y[1]) | pack_e4m3x2(y[2], y[3]) << 16,
                                            pack_e4m3x2(y[4], y[5]) | pack_e4m3x2(y[6], y[7]) << 16);
}

// 16 elements of a head: two runs of 8.
struct Part {
  uint4 a, b;
};
// Which 16 elements part i of a token is: the threads of a head take a pair of
// 8-element runs half the rotated width apart (so that each holds whole pairs), or
// 16 elements in a row.
struct Place {
  int kind;  // 0: q, 1: k, 2: v
  int h, j;  // head, thread of the head
  int e0, e1;
  bool turn, split;
};
__device__ __forceinline__ Place place_of(const AppendParams& p, int i) {
  Place x;
  const int shift = p.d == 128 ? 3 : 2;  // log2(threads of a head)
  const int head = i >> shift;
  x.j = i & ((1 << shift) - 1);
  x.kind = head < p.H_q ? 0 : head < p.H_q + p.H_kv ? 1 : 2;
  x.h = x.kind == 0 ? head : x.kind == 1 ? head - p.H_q : head - p.H_q - p.H_kv;
  x.turn = x.kind < 2 && 16 * x.j < p.rotary_dim;
  x.split = x.turn && !p.interleaved;
  x.e0 = x.split ? 8 * x.j : 16 * x.j;
  x.e1 = x.split ? 8 * x.j + (p.rotary_dim >> 1) : 16 * x.j + 8;
  return x;
}
__device__ __forceinline__ Part load_part(const AppendParams& p, const Place& x, int t) {
  const __nv_bfloat16* src =
      x.kind == 0 ? static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride
                  : x.kind == 1 ? static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride
                                : static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride;
  src += x.h * p.d;
  return Part{*reinterpret_cast<const uint4*>(src + x.e0), *reinterpret_cast<const uint4*>(src + x.e1)};
}

// W threads per token. The first kAhead parts of every thread are loaded before the
// token's sequence, position and page are looked up (three dependent loads) and
// its angles computed, once for all heads; then they are turned and stored. What
// bounds it is the bytes: 36,696 tokens of 16 ragged prompts (32 query and 8 KV heads
// of 128, 902 MB) take 135 to 145 us, 6.2 to 6.7 TB/s, 91 to 98% of a plain copy's rate. Measured
// beside it: without the loads ahead 155 us, with a read of the angles from shared
// memory for every part 158, with a warp or 64 threads per token 158 or more, with
// registers held down for more CTAs 156 or more.
//
// W is a multiple of a head's 8 or 4 threads, so that each keeps its place in every
// head; a CTA takes kAppendThreads / W tokens: with few heads a CTA per token would
// leave most threads idle.
constexpr int kAhead = 3;
template <int W>
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const AppendParams p) {
  __shared__ float2 shared_cs[kAppendThreads / W][64];
  const int t = blockIdx.x * (kAppendThreads / W) + threadIdx.x / W, tid = threadIdx.x % W;
  float2* cs = shared_cs[threadIdx.x / W];
  const PagedSeqs& s = p.s;
  grid_wait();
  grid_release();
  const int parts = (p.H_q + 2 * p.H_kv) * (p.d >> 4);
  bool live = t < s.T;
  Part ahead[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = tid + k * W;
    if (live && i < parts) ahead[k] = load_part(p, place_of(p, i), t);
  }
  if (blockIdx.x == 0) check_paged_seqs(s, threadIdx.x, kAppendThreads);
  int b = t, pos = 0, page = 0;
  if (live) {
    SeqSpan span{t, 1};
    if (s.cu_seqlens) {
      // the last sequence that starts at or before row t
      int lo = 0, hi = s.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(s.cu_seqlens + mid) <= t) lo = mid; else hi = mid;
      }
      b = lo;
      span = seq_span(s.cu_seqlens, b, s.T, 0);
      live = t >= span.start && t < span.start + span.len;  // else behind the last sequence
    }
    pos = kv_len(s, b) - span.len + (t - span.start);
    live = live && pos >= 0;  // else padding: the sequence is shorter than its rows
  }
  if (live) {
    page = __ldg(s.page_table + static_cast<size_t>(b) * s.table_stride + (pos >> s.page_shift));
    for (int i = tid; i < p.rotary_dim >> 1; i += W) {
      double turns = __ldg(p.inv_freq + i) * 0.15915494309189533577;  // 1 / 2 pi
      turns -= floor(turns);
      const unsigned long long f = static_cast<unsigned long long>(turns * 18446744073709551616.0);
      const long long whole = static_cast<long long>(f * static_cast<unsigned long long>(pos));
      // half turns in [-1, 1)
      const float half = static_cast<float>(static_cast<int>(whole >> 32)) * (1.0f / 2147483648.0f);
      float sn, c;
      sincospif(half, &sn, &c);
      cs[(i & 7) * (p.rotary_dim >> 4) + (i >> 3)] = make_float2(c, sn);
    }
  }
  if (W <= 32) __syncwarp(); else __syncthreads();
  if (!live) return;
  const bool page_ok = static_cast<unsigned>(page) < static_cast<unsigned>(s.num_pages);
  if (!page_ok && tid == 0) record_error(s.err, kErrPages);
  const int row = pos & ((1 << s.page_shift) - 1);
  // A thread has the same place in every head, so its eight angles stay with it
  // (pair 8 j + e lies at e times the threads + j: neighbours read neighbours).
  float2 turn[8];
  {
    const Place x = place_of(p, tid);
    const int j = 16 * x.j < p.rotary_dim ? x.j : 0;
    if (p.rotary_dim > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) turn[e] = cs[e * (p.rotary_dim >> 4) + j];
    }
  }
  for (int k = 0, i = tid; i < parts; ++k, i += W) {
    const Place x = place_of(p, i);
    const Part w = k == 0 ? ahead[0] : k == 1 ? ahead[1] : k == 2 ? ahead[2] : load_part(p, x, t);
    float x0[8], x1[8];
    widen8(w.a, x0);
    widen8(w.b, x1);
    if (x.split) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 r = turn[e];
        const float a = x0[e], c = x1[e];
        x0[e] = a * r.x - c * r.y;
        x1[e] = a * r.y + c * r.x;
      }
    } else if (x.turn) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 r = turn[e], u = turn[4 + e];
        const float a = x0[2 * e], c = x0[2 * e + 1], a1 = x1[2 * e], c1 = x1[2 * e + 1];
        x0[2 * e] = a * r.x - c * r.y;
        x0[2 * e + 1] = a * r.y + c * r.x;
        x1[2 * e] = a1 * u.x - c1 * u.y;
        x1[2 * e + 1] = a1 * u.y + c1 * u.x;
      }
    }
    if (x.kind == 0) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride + x.h * p.d;
      store8(dst + x.e0, x0);
      store8(dst + x.e1, x1);
    } else if (page_ok) {
      const bool is_v = x.kind == 2;
      const size_t at = static_cast<size_t>(page) * (is_v ? p.v_page : p.k_page) +
                        ((static_cast<size_t>(x.h) << s.page_shift) + row) * p.d;
      if (p.e4m3) {
        const float* sc = is_v ? p.v_scale : p.k_scale;
        const float scale = sc ? __ldg(sc + x.h) : 1.0f, inverse = __frcp_rn(scale);
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + at;
        store8_e4m3(dst + x.e0, x0, scale, inverse);
        store8_e4m3(dst + x.e1, x1, scale, inverse);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + at;
        store8(dst + x.e0, x0);
        store8(dst + x.e1, x1);
      }
    }
  }
}

template <int W>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
  constexpr int kTokens = kAppendThreads / W;
  return launch_chained<paged_append_kernel<W>>(dim3((p.s.T + kTokens - 1) / kTokens), kAppendThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream) {
  const int slot = prof_begin(kKPagedAppend, stream);
  const int parts = (p.H_q + 2 * p.H_kv) * (p.d >> 4);
  // About four parts a thread (14,000 tokens of 28 heads of 64: 47 us with a CTA per
  // token, 28.9 with two parts a thread, 26.9 with four; 17,000 of 6 heads: 46, 12.3,
  // 11.8); few tokens take all the threads they can get.
  const int want = (parts + 3) / 4;
  const cudaError_t e = p.s.T < 304   ? launch<128>(p, stream)
                        : want <= 8  ? launch<8>(p, stream)
                        : want <= 16 ? launch<16>(p, stream)
                        : want <= 32 ? launch<32>(p, stream)
                        : want <= 64 ? launch<64>(p, stream)
                                     : launch<128>(p, stream);
  prof_end(slot, stream);
  return e;
}

}  // namespace attn
