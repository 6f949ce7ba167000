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
// so the exponent's rise and the codes need no atomics.  A thread holds its rows' 16-bit
// inputs in registers (at most 8 x 16 bytes) between the maximum and the codes, so the
// inputs are read once: the append is bound by HBM (2 + 1 bytes an element).  The maximum of
// |x| is taken on the 15 low bits, which order like the values in both types.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendParams p) {
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
  const uint4* src = p.x[op] + (long long)(s.q0 + lo - s.pos0) * p.stride[op] + h * VR;
  uint4 v[8];
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int it = threadIdx.x + i * kAppendThreads;
    v[i] = make_uint4(0, 0, 0, 0);
    if (it < items) v[i] = __ldg(src + (long long)(it / VR) * p.stride[op] + it % VR);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    am = __vmaxu2(am, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
    am = __vmaxu2(am, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
  }
  am = max(am & 0xFFFFu, am >> 16);
  am = __reduce_max_sync(0xffffffffu, am);
  __shared__ uint32_t wmax[kAppendThreads / 32];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = am;
  uint8_t* sc = p.scales[op] + (long long)page * p.Hkv + h;
  const int e_old = (int)*sc - 127;  // read by every thread before the barrier, written after it
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kAppendThreads / 32; ++i) am = max(am, wmax[i]);
  // the smallest e >= -127 with amax <= 448 * 2^e = 1.75 * 2^(e + 8)
  const uint32_t bits = __float_as_uint(pair_to_float2(am, p.fp16).x);
  int e = max(-127, (int)(bits >> 23) - 135 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0));
  uint8_t* dst = p.codes[op] + ((long long)page * p.Hkv + h) * p.page * D;
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
  for (int i = 0; i < 8; ++i) {
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

// FP32 -> unsigned that orders like the value (-0 counts as 0).
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// One CTA per (sequence, kv head).  The free tokens are [lo, hi) (between the sinks and the
// recent ones); `want` of them stay.  Three passes of 11, 11 and 10 bits of the key narrow
// the want-th largest key down to one value; tokens above it stay, and of those equal to it
// the first ones.  Then each warp counts and writes its own contiguous share in order.
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
  uint32_t left = (uint32_t)(m - p.sinks - p.recent), prefix = 0;
  if (left > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t k = order_key(w[t]);
        if (pass == 0 || (k >> (shift + bits)) == (prefix >> (shift + bits)))
          atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // the bin that holds the left-th largest: suffix sums over the bins, 64 a lane
      if (warp == 0) {
        const int per = (1 << bits) / 32;
        uint32_t own = 0;
        for (int i = 0; i < per; ++i) own += hist[lane * per + ((i + lane) & (per - 1))];
        uint32_t above = own;  // inclusive suffix sum over lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_down_sync(0xffffffffu, above, o);
          if (lane + o < 32) above += y;
        }
        above -= own;  // tokens in higher lanes' bins
        if (above < left && above + own >= left) {
          for (int i = per - 1; i >= 0; --i) {
            const uint32_t c = hist[lane * per + i];
            if (above + c >= left) {
              s_prefix = prefix | ((uint32_t)(lane * per + i) << shift);
              s_left = left - above;
              break;
            }
            above += c;
          }
        }
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_left;
    }
  }
  // the threshold key is `prefix`, of which the first `left` tokens stay
  const bool any = m > p.sinks + p.recent;
  auto above = [&](int t, uint32_t k) -> bool { return t < lo || t >= hi || (any && k > prefix); };
  const int share = ((n + 1023) / 1024) * 32, w0 = warp * share, w1 = min(n, w0 + share);
  uint32_t cnt = 0, ties = 0;
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t k = t < w1 ? order_key(w[t]) : 0u;
    const bool a = t < w1 && above(t, k);
    cnt += a;
    ties += t < w1 && !a && any && k == prefix;
  }
  cnt = __reduce_add_sync(0xffffffffu, cnt);
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) {
    wsum[warp] = cnt;
    wties[warp] = ties;
  }
  __syncthreads();
  uint32_t at = 0, tie_at = 0;  // kept tokens and ties before this warp's share
  for (int i = 0; i < warp; ++i) {
    at += wsum[i];
    tie_at += wties[i];
  }
  at += min(tie_at, left);
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const float x = t < w1 ? w[t] : 0.0f;
    const uint32_t k = order_key(x);
    const bool a = t < w1 && above(t, k), tie = t < w1 && !a && any && k == prefix;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t bt = __ballot_sync(0xffffffffu, tie);
    const bool stay = a || (tie && tie_at + __popc(bt & below) < left);
    const uint32_t bs = __ballot_sync(0xffffffffu, stay);
    if (stay) {
      const uint32_t r = at + __popc(bs & below);
      kept[r] = t;
      dw[r] = x;
    }
    at += __popc(bs);
    tie_at += __popc(bt);
  }
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
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const MoveParams p) {
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
  if ((int)threadIdx.x < cnt) {
    const int t = __ldg(p.kept + ((long long)b * p.Hkv + h) * p.keep + r0 + threadIdx.x);
    const int pg = __ldg(p.table + (long long)b * p.table_cols + t / p.page);
    const bool ok = pg >= 0 && pg < p.num_pages;
    if (!ok) raise_bad();
    const long long ph = (long long)pg * p.Hkv + h;
    row[threadIdx.x] = ok ? ph * p.page + t % p.page : -1;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const uint8_t c = ok ? __ldg(p.ssc[o] + ph) : 0;
      sc[o][threadIdx.x] = c;
      atomicMax(&top[o], (int)c);
    }
  }
  __syncthreads();
  const long long dh = (long long)dp * p.Hkv + h;
  if (threadIdx.x < 2) p.dsc[threadIdx.x][dh] = (uint8_t)top[threadIdx.x];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    uint4* dst = reinterpret_cast<uint4*>(p.dst[o] + dh * p.page * D);
    const uint4* src = reinterpret_cast<const uint4*>(p.src[o]);
#pragma unroll 4
    for (int i = threadIdx.x; i < cnt * VR; i += kMoveThreads) {
      const int s = i / VR;
      const long long r = row[s];
      uint4 w = make_uint4(0, 0, 0, 0);
      if (r >= 0) w = __ldg(src + r * VR + i % VR);
      const int k = top[o] - (int)sc[o][s];
      if (k > 0) {
        const __half2 down = recode_factor(k);
        w = make_uint4(recode4(w.x, down), recode4(w.y, down), recode4(w.z, down), recode4(w.w, down));
      }
      dst[i] = w;
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
  if (a.s.d == 128)
    kv8::append_kernel<128><<<grid, kv8::kAppendThreads, 0, s>>>(p);
  else
    kv8::append_kernel<64><<<grid, kv8::kAppendThreads, 0, s>>>(p);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_kv8_evict(const Kv8Args& a, const Kv8Evict& e, cudaStream_t s) {
  kv8::SelectParams p;
  p.w = e.w; p.lens = a.lens; p.dst_w = e.dst_w; p.dst_lens = e.dst_lens; p.kept = e.kept;
  p.w_cols = e.w_cols; p.dst_w_cols = e.dst_w_cols;
  p.Hkv = a.s.Hkv; p.keep = e.keep; p.sinks = e.sinks; p.recent = e.recent; p.max_len = a.s.max_len;
  kv8::evict_select_kernel<<<a.s.B * a.s.Hkv, kv8::kSelThreads, 0, s>>>(p);
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
