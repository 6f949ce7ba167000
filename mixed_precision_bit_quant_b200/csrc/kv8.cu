// The paged 8-bit cache: append (quantise new tokens into pages) and eviction by
// accumulated attention weight.  HyQuant: Hybrid-Precision Quantization for LLM
// Attention (abstract, decode stage) compresses the cache it decodes from and
// keeps the tokens that many queries attend to; this is the library's serving
// form of it.
#include "kv8.cuh"

namespace thrift {
namespace kv8 {

constexpr int kAppendThreads = 256;

struct AppendParams {
  const uint4 *x[2];        // new tokens of K and V
  long long stride[2];      // token stride in 16-byte units
  uint8_t* codes[2];
  uint8_t* scales[2];
  const int32_t *table, *lens, *cu;
  int Hkv, page, table_cols, n, max_q, max_len, num_pages, fp16;
};

// One CTA per (page that a sequence's new tokens touch, kv head, K or V); it owns the page,
// so the exponent's rise and the codes need no atomics.  A thread holds its NV 16-byte vectors
// in registers between the maximum and the codes, so the inputs are read once: the append is
// bound by HBM (2 + 1 bytes an element).  The loads have no branch (past the end they take the
// last vector again, which changes no maximum): under a branch each was waited for by itself
// (4 x 8192 tokens of 8 heads of 128: 49 us, now 39, 5.2 TB/s).  The maximum of |x| is taken on the 15 low
// bits, which order like the values in both types.
// Its CTAs are short chains of latencies, so as many as fit are kept on an SM.
template <int D, int NV>
__global__ void __launch_bounds__(kAppendThreads, NV <= 4 ? 8 : 5) append_kernel(const AppendParams p) {
  constexpr int VR = D / 8;  // 16-byte vectors per row
  const int b = blockIdx.z, h = blockIdx.y >> 1, op = blockIdx.y & 1;
  const Seq s = load_seq(p.lens, p.cu, b, p.n, p.max_q, p.max_len);
  const bool reporter = threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0;
  if (s.bad && reporter) raise_bad();
  const int start = max(s.pos0, 0);
  const int col = start / p.page + blockIdx.x;
  if (s.nq == 0 || col * p.page >= s.len) return;
  const int page = __ldg(p.table + (long long)b * p.table_cols + col);
  if (page < 0 || page >= p.num_pages) {
    if (threadIdx.x == 0) raise_bad();
    return;
  }
  const int lo = max(start, col * p.page), hi = min(s.len, (col + 1) * p.page);
  const int items = (hi - lo) * VR;
  const long long stride = op ? p.stride[1] : p.stride[0];
  const uint4* src = (op ? p.x[1] : p.x[0]) + (long long)(s.q0 + lo - s.pos0) * stride + h * VR;
  uint4 v[NV];
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int it = min((int)threadIdx.x + i * kAppendThreads, items - 1);
    v[i] = ldg16_now(src + (long long)(it / VR) * stride + it % VR);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    am = __vmaxu2(am, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
    am = __vmaxu2(am, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
  }
  am = max(am & 0xFFFFu, am >> 16);
  am = __reduce_max_sync(0xffffffffu, am);
  __shared__ uint32_t wmax[kAppendThreads / 32];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = am;
  uint8_t* sc = (op ? p.scales[1] : p.scales[0]) + (long long)page * p.Hkv + h;
  const int e_old = (int)*sc - 127;  // read by every thread before the barrier, written after it
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) am = max(am, wmax[i]);
  // the smallest e >= -127 with amax <= 448 * 2^e = 1.75 * 2^(e + 8)
  const uint32_t bits = __float_as_uint(pair_to_float2(am, p.fp16).x);
  int e = max(-127, (int)(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
  uint8_t* dst = (op ? p.codes[1] : p.codes[0]) + ((long long)page * p.Hkv + h) * p.page * D;
  const int held = lo - col * p.page;  // tokens of the sequence already in the page
  if (held > 0) {
    if (e > e_old) {
      const __half2 down = recode_factor(e - e_old);
      uint4* old = reinterpret_cast<uint4*>(dst);
      for (int i = threadIdx.x; i < held * (D / 16); i += kAppendThreads) {
        const uint4 w = old[i];
        old[i] = make_uint4(recode4(w.x, down), recode4(w.y, down), recode4(w.z, down), recode4(w.w, down));
      }
    }
    e = max(e, e_old);
  }
  if (threadIdx.x == 0) *sc = (uint8_t)(e + 127);
  const float m = pow2f(-e);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int it = threadIdx.x + i * kAppendThreads;
    if (it >= items) break;
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = pair_to_float2(w[k], p.fp16);
      c[k] = cvt_e4m3x2(f.x * m, f.y * m);
    }
    reinterpret_cast<uint2*>(dst + held * D)[it] = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
}

template <int D>
static void launch_append(const AppendParams& p, int vectors, dim3 grid, cudaStream_t s) {
  if (vectors <= 1) append_kernel<D, 1><<<grid, kAppendThreads, 0, s>>>(p);
  else if (vectors == 2) append_kernel<D, 2><<<grid, kAppendThreads, 0, s>>>(p);
  else if (vectors == 4) append_kernel<D, 4><<<grid, kAppendThreads, 0, s>>>(p);
  else append_kernel<D, 8><<<grid, kAppendThreads, 0, s>>>(p);
}

// ---------------------------------------------------------------------------
// Eviction.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;

struct SelectParams {
  const float* w;
  const int32_t* lens;
  float* dst_w;
  int32_t *dst_lens, *kept;
  long long w_cols, dst_w_cols;
  int Hkv, keep, sinks, recent, max_len;
};

// FP32 -> unsigned that orders like the value (-0 counts as 0), within [1, 2^32 - 2]: a token past
// the end has kNone, one that stays in any case kForced.
constexpr uint32_t kNone = 0u, kForced = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return min(max(b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u), kNone + 1), kForced - 1);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// One CTA per (sequence, kv head).  Sinks and recent tokens carry the highest key, so that the
// `keep` largest keys stay.  Three passes of 11, 11 and 10 bits of the key narrow the keep-th largest
// down to one value; tokens above it stay, and of those equal to it the first ones.  A warp
// takes a contiguous share of the tokens, so that it can count and write its kept ones in order; up
// to 32 KEYS tokens a warp (max_len <= 1024 KEYS) their keys are loaded once and stay in registers
// (at 64 heads of up to 32768 tokens 43 us when every pass loaded them again, 27 with them).
//   A lane holds four neighbours of each 128 tokens: 16-byte loads where the rows of w allow them,
// and one running count for four tokens (with single tokens 27 us, of whose 54,000 clocks a CTA the
// final pass took 17,000: ballots and bit counts; now 21).  A CTA is bound by its own instructions
// and latencies.  With single tokens, clusters of 4 CTAs a head that joined their histograms through
// shared memory took 22 us, four copies of the histogram 28.
template <int KEYS>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const SelectParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t wsum[32], wties[32];
  __shared__ uint32_t s_prefix, s_left;
  const int b = blockIdx.x / p.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int n = __ldg(p.lens + b);
  if (n < 0 || n > p.max_len) {
    if (tid == 0) raise_bad();
    n = 0;
  }
  const int m = min(n, p.keep);
  const float* w = p.w + (long long)blockIdx.x * p.w_cols;
  float* dw = p.dst_w + (long long)blockIdx.x * p.dst_w_cols;
  int32_t* kept = p.kept + (long long)blockIdx.x * p.keep;
  if (tid == 0 && blockIdx.x % p.Hkv == 0) p.dst_lens[b] = m;
  for (long long i = m + tid; i < p.dst_w_cols; i += kSelThreads) dw[i] = 0.0f;
  for (int i = m + tid; i < p.keep; i += kSelThreads) kept[i] = -1;
  if (n <= p.keep) {
    for (int i = tid; i < n; i += kSelThreads) {
      kept[i] = i;
      dw[i] = w[i];
    }
    return;
  }
  const int lo = p.sinks, hi = n - p.recent;  // keep >= sinks + recent and n > keep: lo < hi
  // this lane's tokens: w0 + 128 i + 0 .. 3
  const int steps = (n + 4 * kSelThreads - 1) / (4 * kSelThreads), w0 = warp * steps * 128 + 4 * lane;
  const bool vec = p.w_cols % 4 == 0;
  // Tokens past the end take values of the same row, which have no effect.
  auto load = [&](int t, uint32_t (&k)[4]) {
    if (vec) {
      const uint4 u = ldg16_now(w + min((long long)t, p.w_cols - 4));
      k[0] = u.x; k[1] = u.y; k[2] = u.z; k[3] = u.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = __float_as_uint(ldg4_now(w + min(t + e, n - 1)));
    }
  };
  auto to_keys = [&](int t, uint32_t (&k)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool free = t + e >= lo && t + e < hi;
      k[e] = free ? order_key(__uint_as_float(k[e])) : t + e < n ? kForced : kNone;
    }
  };
  constexpr int Q = KEYS > 0 ? KEYS / 4 : 1;
  uint32_t key[Q][4];
  if constexpr (KEYS > 0) {
#pragma unroll
    for (int i = 0; i < Q; ++i) load(w0 + 128 * min(i, steps - 1), key[i]);
#pragma unroll
    for (int i = 0; i < Q; ++i) to_keys(w0 + 128 * i, key[i]);
  }
  auto each = [&](auto&& f) {  // f(first token, keys) for this lane's tokens, in step with the warp
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
        if (i >= steps) break;
        f(w0 + 128 * i, key[i]);
      }
    } else {
#pragma unroll 4
      for (int i = 0; i < steps; ++i) {
        uint32_t k[4];
        load(w0 + 128 * i, k);
        to_keys(w0 + 128 * i, k);
        f(w0 + 128 * i, k);
      }
    }
  };
  uint32_t left = (uint32_t)m, prefix = 0;
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
    const uint32_t high = pass == 0 ? 0u : ~0u << (shift + bits);
    hist[tid] = hist[tid + 1024] = 0;
    __syncthreads();
    each([&](int, const uint32_t (&k)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (((k[e] ^ prefix) & high) == 0 && k[e] != kNone) atomicAdd(&hist[(k[e] >> shift) & ((1u << bits) - 1u)], 1u);
    });
    __syncthreads();
    // the bin that holds the left-th largest: suffix sums, two bins a thread
    const uint2 c = reinterpret_cast<const uint2*>(hist)[tid];
    uint32_t above = c.x + c.y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_down_sync(0xffffffffu, above, o);
      if (lane + o < 32) above += y;
    }
    if (lane == 0) wsum[warp] = above;
    __syncthreads();
    above += __reduce_add_sync(0xffffffffu, lane > warp ? wsum[lane] : 0u);
    above -= c.x + c.y;  // tokens in higher bins
    if (above < left && above + c.x + c.y >= left) {
      const bool upper = above + c.y >= left;
      s_prefix = prefix | ((2u * tid + (upper ? 1u : 0u)) << shift);
      s_left = left - above - (upper ? 0u : c.y);
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // the threshold key is `prefix`, of which the first `left` tokens stay
  uint32_t cnt = 0, ties = 0;
  each([&](int, const uint32_t (&k)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      cnt += k[e] > prefix;
      ties += k[e] == prefix;
    }
  });
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) {
    wsum[warp] = cnt;
    wties[warp] = ties;
  }
  __syncthreads();
  // kept tokens and ties before this warp's share
  uint32_t at = __reduce_add_sync(0xffffffffu, lane < warp ? wsum[lane] : 0u);
  uint32_t tie_at = __reduce_add_sync(0xffffffffu, lane < warp ? wties[lane] : 0u);
  at += min(tie_at, left);
  // how many of 0 .. 4 a lane the lanes before this one have
  auto before = [&](uint32_t c) -> uint32_t {
    const uint32_t below = (1u << lane) - 1u;
    return __popc(__ballot_sync(0xffffffffu, c & 1u) & below) + 2 * __popc(__ballot_sync(0xffffffffu, c & 2u) & below) +
           4 * __popc(__ballot_sync(0xffffffffu, c & 4u) & below);
  };
  each([&](int t, const uint32_t (&k)[4]) {
    bool stay[4], tie[4];
    uint32_t c = 0, ct = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      stay[e] = k[e] > prefix;
      tie[e] = k[e] == prefix;
      ct += tie[e];
    }
    if (__any_sync(0xffffffffu, ct != 0)) {
      const uint32_t first = before(ct);
      uint32_t r = tie_at + first;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        stay[e] = stay[e] || (tie[e] && r < left);
        r += tie[e];
      }
      tie_at += __shfl_sync(0xffffffffu, first + ct, 31);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c += stay[e];
    const uint32_t first = before(c);
    uint32_t r = at + first;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (stay[e] && r < (uint32_t)p.keep) {  // always below, unless the inputs change under the call
        kept[r] = t + e;
        dw[r] = k[e] == kForced ? __ldg(w + t + e) : key_value(k[e]);
      }
      r += stay[e];
    }
    at += __shfl_sync(0xffffffffu, first + c, 31);
  });
}

struct MoveParams {
  const uint8_t* src[2];
  const uint8_t* ssc[2];
  uint8_t* dst[2];
  uint8_t* dsc[2];
  const int32_t *table, *lens, *dst_table, *kept;
  int Hkv, page, table_cols, dst_cols, keep, max_len, num_pages, dst_pages;
};

constexpr int kMoveThreads = 256;

// One CTA per (destination page, kv head, sequence), K and V: a destination page's exponent
// is the largest of its tokens' source pages', and each token's codes are rounded again by
// the difference (copied where there is none).  Bound by HBM: every kept row is read and
// written once, in whole rows of D bytes.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 6) evict_move_kernel(const MoveParams p) {
  constexpr int VR = D / 16;
  const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  __shared__ long long row[128];  // source row, -1: none
  __shared__ uint8_t sc[2][128];
  __shared__ int top[2];
  int n = __ldg(p.lens + b);
  if (n < 0 || n > p.max_len) n = 0;  // reported by the selection
  const int m = min(n, p.keep), r0 = j * p.page, cnt = min(p.page, m - r0);
  if (cnt <= 0) return;
  const int dp = __ldg(p.dst_table + (long long)b * p.dst_cols + j);
  if (dp < 0 || dp >= p.dst_pages) {
    if (threadIdx.x == 0) raise_bad();
    return;
  }
  if (threadIdx.x < 2) top[threadIdx.x] = 0;
  __syncthreads();
  int most[2] = {0, 0};
  if ((int)threadIdx.x < cnt) {
    const int t = __ldg(p.kept + ((long long)b * p.Hkv + h) * p.keep + r0 + threadIdx.x);
    const bool in = t >= 0 && t < n;  // always, unless the inputs change under the call
    const int pg = __ldg(p.table + (long long)b * p.table_cols + (in ? t / p.page : 0));
    const bool ok = in && pg >= 0 && pg < p.num_pages;
    if (!ok) raise_bad();
    const long long ph = (long long)pg * p.Hkv + h;
    row[threadIdx.x] = ok ? ph * p.page + t % p.page : -1;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const uint8_t c = ok ? __ldg(p.ssc[o] + ph) : 0;
      sc[o][threadIdx.x] = c;
      most[o] = c;
    }
  }
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int c = __reduce_max_sync(0xffffffffu, most[o]);
    if ((threadIdx.x & 31) == 0 && c > 0) atomicMax(&top[o], c);
  }
  __syncthreads();
  const long long dh = (long long)dp * p.Hkv + h;
  if (threadIdx.x < 2) p.dsc[threadIdx.x][dh] = (uint8_t)top[threadIdx.x];
  // UN vectors each of K and V a thread and turn, loaded without a branch (a token of no
  // page takes row 0 and becomes zero)
  constexpr int UN = 2;
  for (int i0 = threadIdx.x; i0 < cnt * VR; i0 += UN * kMoveThreads) {
    uint4 w[2][UN];
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = min(i0 + u * kMoveThreads, cnt * VR - 1);
        w[o][u] = ldg16_now((o ? p.src[1] : p.src[0]) + max(row[i / VR], 0ll) * D + 16 * (i % VR));
      }
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + u * kMoveThreads;
        if (i >= cnt * VR) break;
        const int s = i / VR, k = top[o] - (int)sc[o][s];
        uint4 x = row[s] >= 0 ? w[o][u] : make_uint4(0, 0, 0, 0);
        if (k > 0) {
          const __half2 down = recode_factor(k);
          x = make_uint4(recode4(x.x, down), recode4(x.y, down), recode4(x.z, down), recode4(x.w, down));
        }
        reinterpret_cast<uint4*>(p.dst[o] + dh * p.page * D)[i] = x;
      }
  }
}

}  // namespace kv8

cudaError_t read_and_clear_kv8_error(uint32_t* word) { return kv8::read_and_clear_word(word); }

cudaError_t launch_kv8_append(const Kv8Args& a, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              cudaStream_t s) {
  kv8::AppendParams p;
  p.x[0] = static_cast<const uint4*>(k);
  p.x[1] = static_cast<const uint4*>(v);
  p.stride[0] = k_stride / 8;
  p.stride[1] = v_stride / 8;
  p.codes[0] = a.cache.k;
  p.codes[1] = a.cache.v;
  p.scales[0] = a.cache.ks;
  p.scales[1] = a.cache.vs;
  p.table = a.table; p.lens = a.lens; p.cu = a.cu;
  p.Hkv = a.s.Hkv; p.page = a.s.page; p.table_cols = a.s.table_cols;
  p.n = a.s.n; p.max_q = a.s.max_q; p.max_len = a.s.max_len;
  p.num_pages = a.cache.num_pages;
  p.fp16 = a.s.dtype == THRIFT_FP16;
  // a run of max_q tokens touches at most this many pages, and a sequence has this many
  const int pages = (a.s.max_len + a.s.page - 1) / a.s.page;
  const int touched = (a.s.max_q + a.s.page - 2) / a.s.page + 1;
  const dim3 grid(touched < pages ? touched : pages, 2 * a.s.Hkv, a.s.B);
  // vectors a thread: a page's over the CTA's threads
  const int vectors = a.s.page * (a.s.d / 8) / kv8::kAppendThreads;
  if (a.s.d == 128) kv8::launch_append<128>(p, vectors, grid, s);
  else kv8::launch_append<64>(p, vectors, grid, s);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_kv8_evict(const Kv8Args& a, const Kv8Evict& e, cudaStream_t s) {
  kv8::SelectParams p;
  p.w = e.w; p.lens = a.lens; p.dst_w = e.dst_w; p.dst_lens = e.dst_lens; p.kept = e.kept;
  p.w_cols = e.w_cols; p.dst_w_cols = e.dst_w_cols;
  p.Hkv = a.s.Hkv; p.keep = e.keep; p.sinks = e.sinks; p.recent = e.recent; p.max_len = a.s.max_len;
  if (a.s.max_len <= 8 * 1024) kv8::evict_select_kernel<8><<<a.s.B * a.s.Hkv, kv8::kSelThreads, 0, s>>>(p);
  else if (a.s.max_len <= 32 * 1024) kv8::evict_select_kernel<32><<<a.s.B * a.s.Hkv, kv8::kSelThreads, 0, s>>>(p);
  else kv8::evict_select_kernel<0><<<a.s.B * a.s.Hkv, kv8::kSelThreads, 0, s>>>(p);
  kv8::MoveParams m;
  m.src[0] = a.cache.k; m.src[1] = a.cache.v; m.ssc[0] = a.cache.ks; m.ssc[1] = a.cache.vs;
  m.dst[0] = e.dst.k; m.dst[1] = e.dst.v; m.dsc[0] = e.dst.ks; m.dsc[1] = e.dst.vs;
  m.table = a.table; m.lens = a.lens; m.dst_table = e.dst_table; m.kept = e.kept;
  m.Hkv = a.s.Hkv; m.page = a.s.page; m.table_cols = a.s.table_cols; m.dst_cols = e.dst_cols;
  m.keep = e.keep; m.max_len = a.s.max_len; m.num_pages = a.cache.num_pages; m.dst_pages = e.dst.num_pages;
  const int most = e.keep < a.s.max_len ? e.keep : a.s.max_len;
  const dim3 grid((most + a.s.page - 1) / a.s.page, a.s.Hkv, a.s.B);
  if (a.s.d == 128)
    kv8::evict_move_kernel<128><<<grid, kv8::kMoveThreads, 0, s>>>(m);
  else
    kv8::evict_move_kernel<64><<<grid, kv8::kMoveThreads, 0, s>>>(m);
  count_launches(2);
  return cudaGetLastError();
}

}  // namespace thrift
