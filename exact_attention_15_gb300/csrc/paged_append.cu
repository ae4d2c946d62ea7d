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

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
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
// The scale divides (not its rounded inverse), so the stored value is the
// nearest to x / scale.
__device__ __forceinline__ void store8_e4m3(uint8_t* p, const float (&x)[8], float scale) {
  uint2 w;
  w.x = pack_e4m3x2(__fdiv_rn(x[0], scale), __fdiv_rn(x[1], scale)) |
        pack_e4m3x2(__fdiv_rn(x[2], scale), __fdiv_rn(x[3], scale)) << 16;
  w.y = pack_e4m3x2(__fdiv_rn(x[4], scale), __fdiv_rn(x[5], scale)) |
        pack_e4m3x2(__fdiv_rn(x[6], scale), __fdiv_rn(x[7], scale)) << 16;
  *reinterpret_cast<uint2*>(p) = w;
}

// One CTA per token: the token's 64 angles at most are computed once for all
// heads, then each thread turns or copies 16 elements of a head at a time.
__global__ void __launch_bounds__(kAppendThreads)
paged_append_kernel(const AppendParams p) {
  __shared__ float2 cs[64];
  const int t = blockIdx.x, tid = threadIdx.x;
  const PagedSeqs& s = p.s;
  grid_wait();
  grid_release();
  if (t == 0) check_paged_seqs(s, tid, kAppendThreads);
  int b = t;
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
    if (t < span.start || t >= span.start + span.len) return;  // behind the last sequence
  }
  const int pos = kv_len(s, b) - span.len + (t - span.start);
  if (pos < 0) return;  // padding: the sequence is shorter than its rows
  const int page = __ldg(s.page_table + static_cast<size_t>(b) * s.table_stride + (pos >> s.page_shift));
  const bool page_ok = static_cast<unsigned>(page) < static_cast<unsigned>(s.num_pages);
  if (!page_ok && tid == 0) record_error(s.err, kErrPages);
  const int row = pos & ((1 << s.page_shift) - 1);
  const int pairs = p.rotary_dim >> 1;
  if (tid < pairs) {
    double turns = __ldg(p.inv_freq + tid) * 0.15915494309189533577;  // 1 / 2 pi
    turns -= floor(turns);
    const unsigned long long f = static_cast<unsigned long long>(turns * 18446744073709551616.0);
    const long long whole = static_cast<long long>(f * static_cast<unsigned long long>(pos));
    // half turns in [-1, 1)
    const float half = static_cast<float>(static_cast<int>(whole >> 32)) * (1.0f / 2147483648.0f);
    float sn, c;
    sincospif(half, &sn, &c);
    cs[tid] = make_float2(c, sn);
  }
  __syncthreads();
  const int per_head = p.d >> 4;  // threads per head
  const int heads = p.H_q + 2 * p.H_kv;
  for (int i = tid; i < heads * per_head; i += kAppendThreads) {
    const int head = i / per_head, j = i - head * per_head;
    const bool is_q = head < p.H_q, is_v = head >= p.H_q + p.H_kv;
    const int h = is_q ? head : is_v ? head - p.H_q - p.H_kv : head - p.H_q;
    const __nv_bfloat16* src =
        is_q ? static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride + h * p.d
             : is_v ? static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride + h * p.d
                    : static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride + h * p.d;
    // the thread's 16 elements: a pair of 8-element runs half the rotated width
    // apart, or 16 in a row
    const bool turn = !is_v && 16 * j < p.rotary_dim;
    const bool split = turn && !p.interleaved;
    const int e0 = split ? 8 * j : 16 * j, e1 = split ? 8 * j + pairs : 16 * j + 8;
    float x0[8], x1[8];
    load8(src + e0, x0);
    load8(src + e1, x1);
    if (split) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 w = cs[8 * j + e];
        const float a = x0[e], c = x1[e];
        x0[e] = a * w.x - c * w.y;
        x1[e] = a * w.y + c * w.x;
      }
    } else if (turn) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 w = cs[8 * j + e], u = cs[8 * j + 4 + e];
        const float a = x0[2 * e], c = x0[2 * e + 1], a1 = x1[2 * e], c1 = x1[2 * e + 1];
        x0[2 * e] = a * w.x - c * w.y;
        x0[2 * e + 1] = a * w.y + c * w.x;
        x1[2 * e] = a1 * u.x - c1 * u.y;
        x1[2 * e + 1] = a1 * u.y + c1 * u.x;
      }
    }
    if (is_q) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.q_out) + t * p.q_out_stride + h * p.d;
      store8(dst + e0, x0);
      store8(dst + e1, x1);
    } else if (page_ok) {
      const size_t at = static_cast<size_t>(page) * (is_v ? p.v_page : p.k_page) +
                        ((static_cast<size_t>(h) << s.page_shift) + row) * p.d;
      if (p.e4m3) {
        const float* sc = is_v ? p.v_scale : p.k_scale;
        const float scale = sc ? __ldg(sc + h) : 1.0f;
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + at;
        store8_e4m3(dst + e0, x0, scale);
        store8_e4m3(dst + e1, x1, scale);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.v_cache : p.k_cache) + at;
        store8(dst + e0, x0);
        store8(dst + e1, x1);
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_append(const AppendParams& p, cudaStream_t stream) {
  const int slot = prof_begin(kKPagedAppend, stream);
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t e = launch_chained(paged_append_kernel, dim3(p.s.T), kAppendThreads, 0, stream, smem_set, p);
  prof_end(slot, stream);
  return e;
}

}  // namespace attn
