// Attention over the paged 8-bit cache for few rows: how four warps take 8 or 16 query rows over a run
// of tokens.  The kernels of kv8_attn.cu are made of it; kv8_prefill.cu takes it for runs of pages whose
// scales lie too far apart for its own products.
#pragma once
#include "kv8_attn.cuh"

namespace thrift {
namespace kv8 {

constexpr int kTile = 16;         // tokens of a warp's step (the m16 of its products)
constexpr int kSplitThreads = 128;
constexpr int kSplitWarps = kSplitThreads / 32;

// D[16x8] += A[16x16] B[16x8], FP16 operands, FP32 accumulation.  Fragments (two FP16 per
// register, the lower k in the low half; g = lane / 4, t = lane % 4): a0 (row g, k 2t, 2t+1),
// a1 (row g+8, same k), a2 (row g, k 2t+8, +9), a3 (row g+8, same); b0 (k 2t, 2t+1, col g),
// b1 (k 2t+8, +9, col g); d0, d1 (row g, cols 2t, 2t+1), d2, d3 (row g+8).
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8x8 matrix of 16-bit values held as fragments (row g, cols 2t, 2t+1).
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Query row `r` as the FP16 B fragments of the logits' products, times 2^-e with
// e = floor(log2 amax) - 14: its largest component lands in [2^14, 2^15), so a component
// is exact unless it is 2^31 (BF16) or 2^28 (FP16) times smaller, and then at most 2^-39 of
// the largest is lost.  Step s pairs k = 2t, 2t+1 and 2t+8, 2t+9 with four
// consecutive channels, 64 (s / 4) + 16 t + 4 (s % 4) and up, so that a lane's codes of a token
// are whole 16-byte vectors.  The row's four lanes (t = 0..3) share e; scale_query returns it.
template <int D>
__device__ __forceinline__ void load_query(const uint32_t* q, int t, uint32_t (&f)[D / 16][2]) {
#pragma unroll
  for (int v = 0; v < D / 64; ++v)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint4 u = ldg16_now(q + 32 * v + 8 * t + 4 * x);
      f[4 * v + 2 * x][0] = u.x;
      f[4 * v + 2 * x][1] = u.y;
      f[4 * v + 2 * x + 1][0] = u.z;
      f[4 * v + 2 * x + 1][1] = u.w;
    }
}
template <int D>
__device__ __forceinline__ int scale_query(bool held, bool fp16, uint32_t (&f)[D / 16][2]) {
  uint32_t am = 0;
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) f[i][x] = held ? f[i][x] : 0u;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) am = __vmaxu2(am, __vmaxu2(f[i][0] & 0x7FFF7FFFu, f[i][1] & 0x7FFF7FFFu));
  am = max(am & 0xFFFFu, am >> 16);
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
  const int ex = (int)(__float_as_uint(pair_to_float2(am, fp16).x) >> 23) - 127;
  const int e = max(-100, ex - 14);
  const float down = pow2f(-e);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float2 a = pair_to_float2(f[i][x], fp16);
      const __half2 h = __floats2half2_rn(a.x * down, a.y * down);
      f[i][x] = *reinterpret_cast<const uint32_t*>(&h);
    }
  return e;
}

// The codes of a tile of 16 tokens as a lane loads them.  K: of tokens g and g+8 the 16
// channels from 16 t (and from 64 + 16 t); V: of tokens 2t, 2t+1, 2t+8, 2t+9 the D/8 channels from g D/8.
// A warp's load covers whole 32-byte sectors of a token's row in both.
template <int D>
struct Codes {
  uint4 k[2][D / 64];
  uint32_t v[4][D / 32];
};

template <int D>
__device__ __forceinline__ void load_k(const uint8_t* kp, int g, int t, uint4 (&k)[2][D / 64]) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int x = 0; x < D / 64; ++x) k[r][x] = ldg16_now(kp + (g + 8 * r) * D + 64 * x + 16 * t);
}
template <int D>
__device__ __forceinline__ void load_v(const uint8_t* vp, int g, int t, uint32_t (&v)[4][D / 32]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint8_t* a = vp + (2 * t + (r & 1) + 8 * (r >> 1)) * D + g * (D / 8);
    if constexpr (D == 128) {
      const uint4 u = ldg16_now(a);
      v[r][0] = u.x; v[r][1] = u.y; v[r][2] = u.z; v[r][3] = u.w;
    } else {
      const uint2 u = ldg8_now(a);
      v[r][0] = u.x; v[r][1] = u.y;
    }
  }
}

__device__ __forceinline__ uint32_t word_of(const uint4& u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// Raw logits (code units) of 16 tokens x 8 NT rows.
template <int D, int NT>
__device__ __forceinline__ void tile_logits(const uint4 (&k)[2][D / 64], const uint32_t (&qf)[NT][D / 16][2], float (&s)[NT][4]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint32_t lo = word_of(k[0][i / 4], i % 4), hi = word_of(k[1][i / 4], i % 4);
    const uint32_t a0 = e4m3x2_to_h2(lo & 0xFFFFu), a2 = e4m3x2_to_h2(lo >> 16);
    const uint32_t a1 = e4m3x2_to_h2(hi & 0xFFFFu), a3 = e4m3x2_to_h2(hi >> 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16816(s[n], a0, a1, a2, a3, qf[n][i][0], qf[n][i][1]);
  }
}

constexpr float kLazy = 4.0f;  // a row's maximum is raised only when exceeded by 2^4
constexpr float kPShift = 11.0f;  // P enters FP16 times 2^11: at most 2^(4 + 11) = 2^15

// Where a segment's state goes, besides a slot of the workspace: kToRun - i is run i of prefill_kernel's.
constexpr long long kWhole = -1, kToCluster = -2, kToRun = -3;
// Shared memory in floats: the warps' outputs, their maxima and sums, then (for a cluster) the
// CTA's own.
__host__ __device__ constexpr int cluster_ml_at(int d, int nt) { return kSplitWarps * 8 * nt * (d + 4 + 2); }
__host__ __device__ constexpr int split_smem(int d, int nt) { return 4 * (cluster_ml_at(d, nt) + 8 * nt * 2); }

// A barrier of the threads that share a segment.
template <bool GROUP>
__device__ __forceinline__ void split_sync() {
  if constexpr (GROUP) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / kSplitThreads), "n"(kSplitThreads) : "memory");
  else __syncthreads();
}

// Each warp walks its own tiles of 16 tokens straight from global memory into matrix
// fragments -- the codes' layout in a page is the fragments' layout, so nothing is staged --
// with the next tile's loads in flight, and keeps its own softmax state; the warps' states are
// joined at the end of a segment.
//   S^T = K Q^T (m = tokens, n = rows): the e4m3 codes are exact in FP16; the page's scale,
// the row's and the softmax's multiply the FP32 logits.
//   O^T += V^T P^T: P goes to FP16 as p 2^(e_v - e_r + 11), where e_v is the page's V exponent, so
// the products see bare codes; S's fragment becomes P's by one 8x8 transpose.  Both the maximum of
// p and e_r are the row's own: max p 2^e_r is its largest p 2^e_v so far, so that what it sees of
// small scale is not lost beside pages that it does not see or hardly weighs (one e_r for the tile,
// the largest e_v, did).  They are raised (and O rescaled) only when a logit, or a logit with its
// page's scale, exceeds them by 4 binades: the common step needs one vote and no cross-lane maximum.
//   Bound by HBM at 8 rows (8 sequences of 32768 tokens, 4 heads a group: 93 us, 5.8 TB/s); at 16
// rows a step's own latencies bind (two passes of 16 rows over 8 x 16384 tokens: 79 us against 26
// for the bytes; one pass of 32 rows with the codes in a shared-memory ring took 67, but the ring cost
// the 8-row case 20 us).
//   GROUP: one of several groups of kSplitThreads threads of a CTA (prefill_kernel's), with few
// registers: the next tile's loads are not kept in flight, and tiles of the span may be ones that none of
// the rows sees.
template <int D, int NT, bool GROUP = false>
__device__ __forceinline__ void split_segment(const AttnParams& p, const Seq& s, int b, int hk, int rt, const Span<kTile>& span,
                                              int v0, int v1, long long slot, float* sm) {
  constexpr int R = 8 * NT;
  const int tid = GROUP ? threadIdx.x % kSplitThreads : threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int r_base = rt * R, r_cnt = min(s.nq * p.G - r_base, R);
  const int p_lo = s.pos0 + r_base / p.G, p_hi = s.pos0 + (r_base + r_cnt - 1) / p.G;
  float* logit_row = p.logits + (((long long)b * p.Hkv + hk) * p.row_tiles + rt) * p.logit_tokens * p.logit_w;
  float* so = sm;                              // [warps][R][D + 4]
  float* sml = sm + kSplitWarps * R * (D + 4);  // [warps][R][2]

  // the query rows and the first tile's codes are on their way together
  uint32_t qf[NT][D / 16][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) load_query<D>(query_row(p, s, hk, r_base + min(8 * n + g, r_cnt - 1), D), t, qf[n]);
  float acc[NT][D / 16][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][j][e] = 0.0f;
  const int32_t* trow = p.table + (long long)b * p.table_cols;
  const int page_mask = (1 << p.page_log2) - 1;
  int l_page = -1, l_ks = 0, l_vs = 0;  // lane's tile of the current batch of 32 of this warp's tiles
  const int count = v1 > v0 + warp ? (v1 - v0 - warp + kSplitWarps - 1) / kSplitWarps : 0;

  auto batch = [&](int it0) {
    const int v = v0 + warp + (it0 + lane) * kSplitWarps;
    l_page = -1;
    if (v < v1 && (!GROUP || any_visible(p, span.token(v), kTile, p_lo, p_hi))) {
      const int pg = __ldg(trow + (span.token(v) >> p.page_log2));
      if (pg >= 0 && pg < p.num_pages) {
        l_page = pg;
        l_ks = __ldg(p.ks + (long long)pg * p.Hkv + hk);
        l_vs = __ldg(p.vs + (long long)pg * p.Hkv + hk);
      } else {
        raise_bad();
      }
    }
  };
  auto fetch = [&](int it, Codes<D>& c, int& pg) {
    // loaded without a branch (page 0 for one that is not to be read): a load under a branch
    // would be waited for where the branches join
    pg = __shfl_sync(0xffffffffu, l_page, it & 31);
    const int tok = span.token(v0 + warp + it * kSplitWarps);
    const long long off = (((long long)max(pg, 0) * p.Hkv + hk) << p.page_log2) * D + (tok & page_mask) * D;
    load_k<D>(p.k + off, g, t, c.k);
    load_v<D>(p.v + off, g, t, c.v);
  };
  Codes<D> ca, cb;
  int pa = -1, pbg = -1;
  if (count > 0) {
    batch(0);
    fetch(0, ca, pa);
  }
  float fs[NT][2];   // per column 2t, 2t+1: logits' scale without the page's
  int pos[NT][2];    // per column: the query's position
  float m[NT][2], l[NT][2], er[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int e = scale_query<D>(8 * n + g < r_cnt, p.fp16, qf[n]);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int ec = __shfl_sync(0xffffffffu, e, 4 * (2 * t + x));
      fs[n][x] = pow2f(ec) * p.scale_log2;
      const int c = 8 * n + 2 * t + x;
      pos[n][x] = c < r_cnt ? s.pos0 + (r_base + c) / p.G : -1;
      m[n][x] = -INFINITY;
      l[n][x] = 0.0f;
      er[n][x] = 0.0f;
    }
  }
  auto step = [&](int it, Codes<D>& c, int pg, int ksc, int vsc) {
    const int v = v0 + warp + it * kSplitWarps, tok = span.token(v);
    if (pg < 0) {  // not visible: no weight
      if (p.logits != nullptr)
        for (int i = lane; i < kTile * p.logit_w; i += 32) logit_row[(long long)v * kTile * p.logit_w + i] = -INFINITY;
      return;
    }
    float x[NT][4];
    tile_logits<D, NT>(c.k, qf, x);
    const float kscale = scale_value((uint32_t)ksc);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[n][e] *= fs[n][e & 1] * kscale;
    if (!all_visible(p, tok, kTile, p_lo, p_hi)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tt = tok + g + 8 * (e >> 1), pp = pos[n][e & 1];
          const bool see = tt <= pp && (p.window == 0 || tt > pp - p.window || tt < p.sinks);
          if (!see) x[n][e] = -INFINITY;
        }
      // codes of tokens that no row sees may be NaN: a zero probability does not silence them
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tt = tok + 2 * t + (r & 1) + 8 * (r >> 1);
        const bool see = tt <= p_hi && (p.window == 0 || tt > p_lo - p.window || tt < p.sinks);
        if (!see) {
#pragma unroll
          for (int y = 0; y < D / 32; ++y) c.v[r][y] = 0u;
        }
      }
    }
    if (p.logits != nullptr) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (8 * n + 2 * t < p.logit_w) {
          float* at = logit_row + (long long)(v * kTile + g) * p.logit_w + 8 * n + 2 * t;
          *reinterpret_cast<float2*>(at) = make_float2(x[n][0], x[n][1]);
          *reinterpret_cast<float2*>(at + 8 * p.logit_w) = make_float2(x[n][2], x[n][3]);
        }
    }
    const float ev = (float)(vsc - 127);
    bool raise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        raise |= fmaxf(x[n][y], x[n][y + 2]) + fmaxf(ev - er[n][y], 0.0f) > m[n][y] + kLazy;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float mm = fmaxf(x[n][y], x[n][y + 2]);
          mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 4));
          mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 8));
          mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, 16));
          const float mn = fmaxf(m[n][y], mm);
          const float down = m[n][y] == -INFINITY ? -INFINITY : m[n][y] - mn;
          const float en = mm == -INFINITY ? er[n][y] : fmaxf(er[n][y] + down, ev + (mm - mn));
          const float f = ex2_approx(down + (er[n][y] - en));
          l[n][y] *= ex2_approx(down);
          m[n][y] = mn;
          er[n][y] = en;
#pragma unroll
          for (int j = 0; j < D / 16; ++j) {
            acc[n][j][y] *= f;
            acc[n][j][y + 2] *= f;
          }
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float pv[2];  // (bounded, so that times the 0 of an unseen token it stays 0)
#pragma unroll
      for (int y = 0; y < 2; ++y) pv[y] = ex2_approx(fminf(ev - er[n][y] + kPShift, 126.0f));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float mu = m[n][e & 1];
        x[n][e] = mu == -INFINITY ? 0.0f : ex2_approx(x[n][e] - mu);
        l[n][e & 1] += x[n][e];
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const __half2 h = __floats2half2_rn(x[n][2 * y] * pv[0], x[n][2 * y + 1] * pv[1]);
        pb[n][y] = movmatrix(*reinterpret_cast<const uint32_t*>(&h));
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // words w of four tokens -> channels 4w .. 4w+3 as pairs of tokens
      const uint32_t a01 = __byte_perm(c.v[0][w], c.v[1][w], 0x5140), a23 = __byte_perm(c.v[0][w], c.v[1][w], 0x7362);
      const uint32_t b01 = __byte_perm(c.v[2][w], c.v[3][w], 0x5140), b23 = __byte_perm(c.v[2][w], c.v[3][w], 0x7362);
      const uint32_t a0 = e4m3x2_to_h2(a01 & 0xFFFFu), a1 = e4m3x2_to_h2(a01 >> 16);
      const uint32_t a2 = e4m3x2_to_h2(b01 & 0xFFFFu), a3 = e4m3x2_to_h2(b01 >> 16);
      const uint32_t c0 = e4m3x2_to_h2(a23 & 0xFFFFu), c1 = e4m3x2_to_h2(a23 >> 16);
      const uint32_t c2 = e4m3x2_to_h2(b23 & 0xFFFFu), c3 = e4m3x2_to_h2(b23 >> 16);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(acc[n][2 * w], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        mma16816(acc[n][2 * w + 1], c0, c1, c2, c3, pb[n][0], pb[n][1]);
      }
    }
  };

  if constexpr (GROUP) {
    for (int it = 0; it < count; ++it) {
      if (it > 0) {
        if ((it & 31) == 0) batch(it);
        fetch(it, ca, pa);
      }
      step(it, ca, pa, __shfl_sync(0xffffffffu, l_ks, it & 31), __shfl_sync(0xffffffffu, l_vs, it & 31));
    }
  }
  for (int it = 0; !GROUP && it < count; it += 2) {
    // the lane that holds a tile's page also holds its scales; a batch is 32 tiles (even)
    int ksc = __shfl_sync(0xffffffffu, l_ks, it & 31), vsc = __shfl_sync(0xffffffffu, l_vs, it & 31);
    const int ksc1 = __shfl_sync(0xffffffffu, l_ks, (it + 1) & 31), vsc1 = __shfl_sync(0xffffffffu, l_vs, (it + 1) & 31);
    if (it + 1 < count) fetch(it + 1, cb, pbg);
    step(it, ca, pa, ksc, vsc);
    if (it + 2 < count) {
      if (((it + 2) & 31) == 0) batch(it + 2);
      fetch(it + 2, ca, pa);
    }
    if (it + 1 < count) step(it + 1, cb, pbg, ksc1, vsc1);
  }

  // ---- join the warps' states
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      float ll = l[n][y];
      ll += __shfl_xor_sync(0xffffffffu, ll, 4);
      ll += __shfl_xor_sync(0xffffffffu, ll, 8);
      ll += __shfl_xor_sync(0xffffffffu, ll, 16);
      const int c = 8 * n + 2 * t + y;
      if (g == 0) {
        sml[(warp * R + c) * 2] = m[n][y];
        sml[(warp * R + c) * 2 + 1] = ll;
      }
      // back to values: 2^(e_r - 11) in steps (e_r may be below -126)
      const float f1 = ex2_approx(0.5f * er[n][y]), f2 = 1.0f / (1 << (int)kPShift);
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        *reinterpret_cast<float2*>(so + (warp * R + c) * (D + 4) + g * (D / 8) + 2 * j) =
            make_float2(acc[n][j][y] * f2 * f1 * f1, acc[n][j][y + 2] * f2 * f1 * f1);
    }
  split_sync<GROUP>();
  for (int i = tid; i < r_cnt * (D / 4); i += kSplitThreads) {
    const int r = i / (D / 4), c4 = i % (D / 4);
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) mm = fmaxf(mm, sml[(w * R + r) * 2]);
    float ll = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) {
      const float mw = sml[(w * R + r) * 2];
      const float f = mw == -INFINITY ? 0.0f : ex2_approx(mw - mm);
      const float4 x = *reinterpret_cast<const float4*>(so + (w * R + r) * (D + 4) + 4 * c4);
      ll += sml[(w * R + r) * 2 + 1] * f;
      o.x += x.x * f;
      o.y += x.y * f;
      o.z += x.z * f;
      o.w += x.w * f;
    }
    if (slot == kToCluster) {  // left in shared memory for the cluster's other CTAs
      *reinterpret_cast<float4*>(so + r * (D + 4) + 4 * c4) = o;  // where only this thread has read
      if (c4 == 0) *reinterpret_cast<float2*>(sm + cluster_ml_at(D, NT) + 2 * r) = make_float2(mm, ll);
    } else if (slot == kWhole) {  // the whole unit: final
      const long long row = packed_row(p, s, hk, r_base + r);
      const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
      reinterpret_cast<uint2*>(p.o)[row * (D / 4) + c4] =
          make_uint2(float2_to_pair(o.x * inv, o.y * inv, p.fp16), float2_to_pair(o.z * inv, o.w * inv, p.fp16));
      if (c4 == 0) write_lse(p, row, mm, ll);
    } else {
      const long long at = GROUP ? packed_row(p, s, hk, r_base + r) * p.nsplit + (kToRun - slot) : slot * R + r;
      *reinterpret_cast<float4*>(p.part_o + at * D + 4 * c4) = o;
      if (c4 == 0) p.part_ml[at] = make_float2(mm, ll);
    }
  }
}

}  // namespace kv8
}  // namespace thrift
