// Attention over the paged 8-bit cache: causal, with an optional sliding window and
// first tokens that stay visible, for any number of new tokens per sequence.
// HyQuant: Hybrid-Precision Quantization for LLM Attention (abstract, decode
// stage): the dequantisation is fused into the attention over the compressed
// cache; sink tokens and the local window are what a windowed call keeps.
//
// The query rows of one kv head's group are taken together: row r = i * G + g is
// query head hk * G + g of new token i.  Kernels:
//   split_kernel   few rows: every CTA takes the same share of all visible tokens of all tiles
//                  of 8 or 16 rows; online softmax; writes the output, or a run's
//                  state (maximum, sum, unnormalised output) where several CTAs share a tile
//   cluster_kernel few rows of short units: a cluster takes one and joins its states itself
//   prefill_kernel (kv8_prefill.cu) many rows
//   merge_kernel   joins the runs' states of a row
//   logit_weights_kernel, tile_weights_kernel (kv8_prefill.cu)  add the rows' final weights to
//                  the running sums of the tokens
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

// The visible tokens of sequence b, in 16-token tiles, of one kv head: over the tiles of R rows.
template <int R>
__device__ __forceinline__ Span<kTile> row_tile_span(const AttnParams& p, const Seq& s, int rt) {
  const int rows = min(s.nq * p.G - rt * R, R);
  if (rows <= 0) return Span<kTile>{0, 0, 0};
  return visible_span<kTile>(s.pos0 + rt * R / p.G, s.pos0 + (rt * R + rows - 1) / p.G, p.window, p.sinks);
}

// All tiles of the call in one line -- sequence, kv head, row tile, token -- of which every CTA
// takes the same share (a multiple of kSplitWarps), so that sequences of any lengths load all
// SMs evenly; the lengths are read here, not on the host.  A CTA's piece of one (sequence, kv
// head, row tile), its unit, is a segment; segment cta + unit is its slot in the workspace
// (both only grow along the line, so slots are distinct and below CTAs + units).
struct Share {
  int at, end;      // this CTA's tiles (the host bounds their number below 2^31)
  int share;        // tiles of a CTA
  int b, b_at, b_c; // the sequence of `at`, its first tile and its tiles
  Seq s;
};
template <int R>
__device__ __forceinline__ Share find_share(const AttnParams& p, int B) {
  __shared__ int scan[kSplitWarps];
  __shared__ Share found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) found.at = found.end = 0;
  // first pass: the number of tiles, hence the share; second pass: the sequence it starts in
  // (one pass finds both where the CTA's threads hold all sequences)
  int total = 0;
  for (int pass = B <= kSplitThreads ? 1 : 0; pass < 2; ++pass) {
    int base = 0;
    for (int b0 = 0; b0 < B; b0 += kSplitThreads) {
      const int b = b0 + threadIdx.x;
      int c = 0;
      Seq s{0, 0, 0, 0, false};
      if (b < B) {
        s = load_seq(p.lens, p.cu, b, p.n, p.max_q, p.max_len);
        if (s.bad && pass == 1 && blockIdx.x == 0) raise_bad();
        for (int rt = 0; rt < p.row_tiles; ++rt) c += row_tile_span<R>(p, s, rt).count;
        c *= p.Hkv;
      }
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();  // the last chunk's sums are read
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      x += base;
#pragma unroll
      for (int w = 0; w < kSplitWarps; ++w) {
        if (w < warp) x += scan[w];
        base += scan[w];
      }
      // x: tiles up to and with sequence b
      if (pass == 1) {
        if (B <= kSplitThreads) total = base;
        const int each = (int)(((unsigned)total + gridDim.x - 1) / gridDim.x);
        const int share = (each + kSplitWarps - 1) / kSplitWarps * kSplitWarps;
        const long long at = (long long)blockIdx.x * share;
        if (at >= x - c && at < x) found = Share{(int)at, (int)min((long long)total, at + share), share, b, x - c, c, s};
      }
    }
    total = base;
  }
  __syncthreads();
  return found;
}

// Where a segment's state goes, besides a slot of the workspace.
constexpr long long kWhole = -1, kToCluster = -2;
// Shared memory in floats: the warps' outputs, their maxima and sums, then (for a cluster) the
// CTA's own.
__host__ __device__ constexpr int cluster_ml_at(int d, int nt) { return kSplitWarps * 8 * nt * (d + 4 + 2); }
__host__ __device__ constexpr int split_smem(int d, int nt) { return 4 * (cluster_ml_at(d, nt) + 8 * nt * 2); }

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
//   Bound by HBM at 8 rows (8 sequences of 32768 tokens, 4 heads a group: 95 us, 5.6 TB/s); at 16
// rows a step's own latencies bind (two passes of 16 rows over 8 x 16384 tokens: 74 us against 26
// for the bytes; one pass of 32 rows with the codes in a shared-memory ring took 67, but the ring cost
// the 8-row case 20 us).
template <int D, int NT>
__device__ __forceinline__ void split_segment(const AttnParams& p, const Seq& s, int b, int hk, int rt, const Span<kTile>& span,
                                              int v0, int v1, long long slot, float* sm) {
  constexpr int R = 8 * NT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
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
    if (v < v1) {
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
    const int tok = span.token(v0 + warp + it * kSplitWarps);
    if (pg < 0) {  // not visible: no weight
      if (p.logits != nullptr)
        for (int i = lane; i < kTile * p.logit_w; i += 32) logit_row[(long long)tok * p.logit_w + i] = -INFINITY;
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
          float* at = logit_row + (long long)(tok + g) * p.logit_w + 8 * n + 2 * t;
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

  for (int it = 0; it < count; it += 2) {
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
  __syncthreads();
  for (int i = threadIdx.x; i < r_cnt * (D / 4); i += kSplitThreads) {
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
      *reinterpret_cast<float4*>(p.part_o + (slot * R + r) * D + 4 * c4) = o;
      if (c4 == 0) p.part_ml[slot * R + r] = make_float2(mm, ll);
    }
  }
}

// CTAs that an SM holds (their registers), of which the plan launches one wave.
__host__ __device__ constexpr int resident_ctas(int d, int nt) { return d == 128 ? (nt == 1 ? 3 : 2) : (nt == 1 ? 4 : 3); }

template <int D, int NT>
__global__ void __launch_bounds__(kSplitThreads, resident_ctas(D, NT)) split_kernel(const AttnParams p, int B) {
  constexpr int R = 8 * NT;
  extern __shared__ __align__(16) float sm[];
  const Share sh = find_share<R>(p, B);
  int at = sh.at, b_at = sh.b_at, b_c = sh.b_c;
  Seq s = sh.s;
  for (int b = sh.b; at < sh.end;) {
    const int per_head = b_c / p.Hkv;
    while (at < sh.end && at < b_at + b_c) {
      const int hk = (at - b_at) / per_head;
      int v = (at - b_at) - hk * per_head, rt = 0;
      Span<kTile> span = row_tile_span<R>(p, s, 0);
      while (v >= span.count) {
        v -= span.count;
        span = row_tile_span<R>(p, s, ++rt);
      }
      const int v1 = min(span.count, v + (sh.end - at));
      const int unit = (b * p.Hkv + hk) * p.row_tiles + rt;
      const bool whole = v == 0 && v1 == span.count;
      if (v == 0 && threadIdx.x == 0)  // the unit's first slot and how many it has
        p.unit_slots[unit] = make_int2((int)blockIdx.x + unit, (at + span.count - 1) / sh.share - (int)blockIdx.x + 1);
      split_segment<D, NT>(p, s, b, hk, rt, span, v, v1, whole ? kWhole : (long long)blockIdx.x + unit, sm);
      at += v1 - v;
      __syncthreads();  // shared memory is free again
    }
    b_at += b_c;
    if (at < sh.end) {
      s = load_seq(p.lens, p.cu, ++b, p.n, p.max_q, p.max_len);
      b_c = 0;
      for (int rt = 0; rt < p.row_tiles; ++rt) b_c += row_tile_span<R>(p, s, rt).count;
      b_c *= p.Hkv;
    }
  }
}

// A short unit (few tiles, and few units): one cluster of eight CTAs takes it, an eighth of its
// tiles each, and joins the states through the cluster's shared memory -- no search for the
// shares, no workspace, no second launch.  At one sequence of 517 tokens and 12 heads of 64
// 5.3 us where split_kernel and merge_kernel take 6.5 + 3.1; at four windows of 4096 tokens 14.3
// where they take 15.7 + 3.6.
constexpr int kCluster = 8;
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int D, int NT>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSplitThreads, resident_ctas(D, NT))
    cluster_kernel(const AttnParams p) {
  constexpr int R = 8 * NT;
  extern __shared__ __align__(16) float sm[];
  const int rank = blockIdx.x % kCluster, unit = blockIdx.x / kCluster;
  const int rt = unit % p.row_tiles, bk = unit / p.row_tiles, b = bk / p.Hkv, hk = bk % p.Hkv;
  const Seq s = load_seq(p.lens, p.cu, b, p.n, p.max_q, p.max_len);
  if (s.bad && threadIdx.x == 0 && rank == 0 && hk == 0 && rt == 0) raise_bad();
  const int r_base = rt * R, r_cnt = min(s.nq * p.G - r_base, R);
  if (r_cnt <= 0) return;  // the whole cluster
  const Span<kTile> span = row_tile_span<R>(p, s, rt);
  const int v0 = span.count * rank / kCluster, v1 = span.count * (rank + 1) / kCluster;
  split_segment<D, NT>(p, s, b, hk, rt, span, v0, v1, kToCluster, sm);
  cluster_sync();
  const uint32_t so = smem_u32(sm), sml = smem_u32(sm + cluster_ml_at(D, NT));
  for (int i = rank * kSplitThreads + threadIdx.x; i < r_cnt * (D / 4); i += kCluster * kSplitThreads) {
    const int r = i / (D / 4), c4 = i % (D / 4);
    float4 x[kCluster];
    float2 ml[kCluster];
    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                   : "=f"(ml[k].x), "=f"(ml[k].y) : "r"(peer_address(sml + 8 * r, k)));
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(x[k].x), "=f"(x[k].y), "=f"(x[k].z), "=f"(x[k].w)
                   : "r"(peer_address(so + 4 * (r * (D + 4) + 4 * c4), k)));
    }
#pragma unroll
    for (int k = 0; k < kCluster; ++k) mm = fmaxf(mm, ml[k].x);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      const float f = ml[k].x == -INFINITY ? 0.0f : ex2_approx(ml[k].x - mm);
      ll += ml[k].y * f;
      o.x += x[k].x * f;
      o.y += x[k].y * f;
      o.z += x[k].z * f;
      o.w += x[k].w * f;
    }
    const long long row = packed_row(p, s, hk, r_base + r);
    const float inv = ll > 0.0f ? 1.0f / ll : 0.0f;
    reinterpret_cast<uint2*>(p.o)[row * (D / 4) + c4] =
        make_uint2(float2_to_pair(o.x * inv, o.y * inv, p.fp16), float2_to_pair(o.z * inv, o.w * inv, p.fp16));
    if (c4 == 0) write_lse(p, row, mm, ll);
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

// Joins the runs' states of a row: one CTA per (new token and query head, sequence).  The
// warps share the runs, four loads in flight each (a warp alone took 40 us for 64 runs: one
// dependent load after the other), and are joined in shared memory.  Run order and warp
// order are fixed, so the sum is.  R: rows of split_kernel's tiles, or 0 where prefill_kernel
// cut the call into p.nsplit runs per row.
constexpr int kMergeWarps = 4;
template <int D, int R>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_kernel(const AttnParams p) {
  constexpr int C = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Seq s = load_seq(p.lens, p.cu, blockIdx.y, p.n, p.max_q, p.max_len);
  const int i = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
  if (i >= s.nq) return;
  const long long row = (long long)(s.q0 + i) * p.Hq + h;
  // state k of the row is element first + k * step
  long long first, step;
  int count;
  if constexpr (R == 0) {
    first = row * p.nsplit;
    step = 1;
    count = p.nsplit;
  } else {
    const int r = i * p.G + h % p.G, rt = r / R;
    if (row_tile_span<R>(p, s, rt).count == 0) {  // no row of the tile sees anything: no segment
      if (threadIdx.x < D / 2) static_cast<uint32_t*>(p.o)[row * (D / 2) + threadIdx.x] = 0u;
      if (threadIdx.x == 0) write_lse(p, row, -INFINITY, 0.0f);
      return;
    }
    const int2 slots = p.unit_slots[(blockIdx.y * p.Hkv + h / p.G) * p.row_tiles + rt];
    if (slots.y == 1) return;  // written by its only segment
    first = (long long)slots.x * R + r % R;
    step = R;
    count = slots.y;
  }
  const float2* ml = p.part_ml + first;
  const float* po = p.part_o + first * D + lane * C;
  __shared__ float so[kMergeWarps][D];
  __shared__ float sl[kMergeWarps];
  float mm = -INFINITY;
  for (int k = lane; k < count; k += 32) mm = fmaxf(mm, ml[k * step].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  float ll = 0.0f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.0f;
  for (int k0 = warp; k0 < count; k0 += 4 * kMergeWarps) {
    float x[4][C], f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = k0 + u * kMergeWarps;
      f[u] = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c) x[u][c] = 0.0f;
      if (k < count) {
        const float2 y = ml[k * step];
        if (y.x != -INFINITY) {  // an empty run wrote no output
          f[u] = ex2_approx(y.x - mm);
          ll += y.y * f[u];
          if constexpr (C == 4) {
            const float4 z = *reinterpret_cast<const float4*>(po + k * step * D);
            x[u][0] = z.x; x[u][1] = z.y; x[u][2] = z.z; x[u][3] = z.w;
          } else {
            const float2 z = *reinterpret_cast<const float2*>(po + k * step * D);
            x[u][0] = z.x; x[u][1] = z.y;
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += x[u][c] * f[u];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) so[warp][lane * C + c] = acc[c];
  if (lane == 0) sl[warp] = ll;
  __syncthreads();
  if (threadIdx.x < D / 2) {
    float l = 0.0f, a = 0.0f, b = 0.0f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      l += sl[w];
      a += so[w][2 * threadIdx.x];
      b += so[w][2 * threadIdx.x + 1];
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    static_cast<uint32_t*>(p.o)[row * (D / 2) + threadIdx.x] = float2_to_pair(a * inv, b * inv, p.fp16);
    if (threadIdx.x == 0) write_lse(p, row, mm, l);
  }
}

// The weight sums of few rows: split_kernel left every visible logit (log2 domain, FP32), and
// a thread adds up one token's rows with their final log-sum-exp.  Storing the logits costs
// 8 bytes a row and token, a fraction of the token's 2 D bytes of codes (4 rows and D = 128:
// 1/8); computing them again took as long as the attention itself (75 us of 142 at 32
// sequences of up to 8191 tokens, against 8).  One thread adds a token's rows in order: the sum does
// not depend on how the work was spread.
constexpr int kWeightRows = 64;  // the most rows of split_kernel
constexpr int kWeightThreads = 256;
__host__ __device__ constexpr int weight_tokens(int rw) { return rw <= 4 ? 4 : rw == 8 ? 2 : 1; }  // of a thread

template <int RW>
__global__ void __launch_bounds__(kWeightThreads) logit_weights_kernel(const AttnParams p, int R) {
  constexpr int T = weight_tokens(RW);
  __shared__ float lse2[kWeightRows];
  __shared__ int pos[kWeightRows];
  const int bk = blockIdx.y, b = bk / p.Hkv, hk = bk % p.Hkv;
  const Seq s = load_seq(p.lens, p.cu, b, p.n, p.max_q, p.max_len);
  const int rows = s.nq * p.G, t0 = blockIdx.x * kWeightThreads * T + threadIdx.x;
  if (blockIdx.x * kWeightThreads * T >= s.len || rows == 0) return;
  float* w = p.w + (long long)bk * p.w_cols;
  float sum[T], was[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    sum[i] = 0.0f;
    was[i] = w[min(t0 + i * kWeightThreads, s.len - 1)];
  }
  // a row whose tokens all lie on pages outside the pool has the log-sum-exp -inf, as its
  // logits: it gives no weight (-inf less -inf would be NaN)
  if ((int)threadIdx.x < rows) {
    const float x = p.lse2[packed_row(p, s, hk, threadIdx.x)];
    lse2[threadIdx.x] = x == -INFINITY ? INFINITY : x;
    pos[threadIdx.x] = s.pos0 + threadIdx.x / p.G;
  }
  __syncthreads();
  for (int r0 = 0; r0 < rows; r0 += R) {
    const float* at = p.logits + ((long long)bk * p.row_tiles + r0 / R) * p.logit_tokens * RW;
    // a logit that its row does not see may be unwritten: it is loaded (without a branch, so
    // that the loads go out together) and dropped
    float2 x[T][RW / 2];
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int c = 0; c < RW / 2; ++c)
        x[i][c] = *reinterpret_cast<const float2*>(at + (long long)min(t0 + i * kWeightThreads, s.len - 1) * RW + 2 * c);
#pragma unroll
    for (int c = 0; c < RW; ++c) {
      if (r0 + c >= rows) break;
      const float nl = lse2[r0 + c];
      const int pp = pos[r0 + c];
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int tok = t0 + i * kWeightThreads;
        const bool see = tok <= pp && (p.window == 0 || tok > pp - p.window || tok < p.sinks);
        sum[i] += see ? ex2_approx((c & 1 ? x[i][c / 2].y : x[i][c / 2].x) - nl) : 0.0f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int tok = t0 + i * kWeightThreads;
    if (tok < s.len && any_visible(p, tok, 1, max(s.pos0, 0), s.len - 1)) w[tok] = was[i] + sum[i];
  }
}

template <int RW>
static void launch_logit_weights(const AttnParams& p, const Plan& plan, const thrift_kv8_shape& s, cudaStream_t st) {
  const int per = kWeightThreads * weight_tokens(RW);
  logit_weights_kernel<RW><<<dim3((s.max_len + per - 1) / per, s.B * s.Hkv), kWeightThreads, 0, st>>>(p, 8 * plan.nt);
}

constexpr int kClusterTiles = 12;
static Plan make_plan(const thrift_kv8_shape& s, const thrift_kv8_mask& m, bool with_w) {
  Plan p{};
  const long long G = s.Hq / s.Hkv, rows = (long long)s.max_q * G;
  p.tiles128 = rows > 64;
  p.nt = rows <= 8 ? 1 : 2;
  const int R = p.tiles128 ? kPrefillRows : 8 * p.nt, T = p.tiles128 ? kPrefillTile : kTile;
  p.row_tiles = (int)((rows + R - 1) / R);
  // tokens that one row tile can see, rounded up to tiles at the sinks' and the window's ends
  long long span = s.max_len;
  if (m.window > 0 && m.window < s.max_len) {
    const long long w = (long long)m.window + (R + G - 1) / G + 2 * T + m.sinks + T;
    if (w < span) span = w;
  }
  const long long tiles = (span + T - 1) / T + 1;
  const long long units = (long long)s.B * s.Hkv * p.row_tiles;
  if (p.tiles128) {
    const long long ns = 148 / units < 1 ? 1 : 148 / units;
    p.chunk = (int)((tiles + ns - 1) / ns);
    if (p.chunk < 2) p.chunk = 2;
  } else {
    const int resident = resident_ctas(s.d, p.nt);
    // one wave of clusters, and at most kClusterTiles tiles a warp: beyond that a unit needs more CTAs
    p.cluster = units * kCluster <= 148 * resident && tiles <= kClusterTiles * kCluster * kSplitWarps;
    const long long most = (tiles * units + kSplitWarps - 1) / kSplitWarps;
    p.ctas = (int)(most < 148 * resident ? most : 148 * resident);
  }
  const size_t nrow = (size_t)s.n * s.Hq;
  size_t states, at = 0;
  if (p.tiles128) {
    p.nsplit = (int)((tiles + p.chunk - 1) / p.chunk);
    states = p.nsplit > 1 ? nrow * p.nsplit : 0;
  } else {
    p.nsplit = 0;
    states = p.cluster ? 0 : (size_t)(p.ctas + units) * R;
  }
  auto take = [&](size_t n) { const size_t o = at; at += (n + 255) / 256 * 256; return o; };
  p.ml_off = take(states * sizeof(float2));
  p.o_off = take(states * s.d * sizeof(float));
  p.slots_off = take(p.tiles128 || p.cluster ? 0 : (size_t)units * sizeof(int2));
  p.lse_off = take(with_w ? nrow * sizeof(float) : 0);
  p.logit_w = rows <= 2 ? 2 : rows <= 4 ? 4 : 8 * p.nt;
  p.logit_tokens = (s.max_len + kTile - 1) / kTile * kTile;
  // prefill_kernel's query tiles for tile_weights_kernel
  const size_t tiles128 = with_w && p.tiles128 ? (size_t)units * 2 : 0;
  p.image_off = take(tiles128 * 128 * s.d * 2);
  p.scale_off = take(tiles128 * sizeof(float));
  p.logits_off = take(with_w && !p.tiles128 ? sizeof(float) * units * p.logit_tokens * p.logit_w : 0);
  p.bytes = at;
  return p;
}

template <int D, int NT>
static void launch_split(const AttnParams& p, const Plan& plan, const thrift_kv8_shape& s, cudaStream_t st) {
  constexpr int sm = split_smem(D, NT);
  if (plan.cluster) {
    const unsigned units = (unsigned)(s.B * s.Hkv * plan.row_tiles);
    cluster_kernel<D, NT><<<units * kCluster, kSplitThreads, sm, st>>>(p);
    return;
  }
  split_kernel<D, NT><<<plan.ctas, kSplitThreads, sm, st>>>(p, s.B);
  merge_kernel<D, 8 * NT><<<dim3(s.max_q * s.Hq, s.B), 32 * kMergeWarps, 0, st>>>(p);
}

template <int D>
static cudaError_t launch_attn_d(const AttnParams& p, const Plan& plan, const thrift_kv8_shape& s, cudaStream_t st) {
  int launches = 1;
  if (plan.tiles128) {
    const cudaError_t e = launch_prefill(p, s, st);
    if (e != cudaSuccess) return e;
    if (plan.nsplit > 1) {
      merge_kernel<D, 0><<<dim3(s.max_q * s.Hq, s.B), 32 * kMergeWarps, 0, st>>>(p);
      ++launches;
    }
  } else {
    if (plan.nt == 1) launch_split<D, 1>(p, plan, s, st);
    else launch_split<D, 2>(p, plan, s, st);
    if (!plan.cluster) ++launches;
  }
  if (p.w != nullptr && plan.tiles128) {
    const cudaError_t e = launch_tile_weights(p, s, st);
    if (e != cudaSuccess) return e;
    ++launches;
  } else if (p.w != nullptr) {
    switch (plan.logit_w) {
      case 2: launch_logit_weights<2>(p, plan, s, st); break;
      case 4: launch_logit_weights<4>(p, plan, s, st); break;
      case 8: launch_logit_weights<8>(p, plan, s, st); break;
      default: launch_logit_weights<16>(p, plan, s, st);
    }
    ++launches;
  }
  count_launches(launches);
  return cudaGetLastError();
}

}  // namespace kv8

cudaError_t read_and_clear_kv8_attn_error(uint32_t* word) { return kv8::read_and_clear_word(word); }

size_t kv8_attn_workspace(const thrift_kv8_shape& s, const thrift_kv8_mask& m, bool with_w) {
  return kv8::make_plan(s, m, with_w).bytes;
}

cudaError_t launch_kv8_attn(const Kv8Args& a, const Kv8Attn& t, cudaStream_t st) {
  const kv8::Plan plan = kv8::make_plan(a.s, t.mask, t.w != nullptr);
  kv8::AttnParams p;
  p.k = a.cache.k; p.v = a.cache.v; p.ks = a.cache.ks; p.vs = a.cache.vs;
  p.q = t.q; p.q_stride = t.q_stride;
  p.table = a.table; p.lens = a.lens; p.cu = a.cu;
  p.o = t.o; p.lse = t.lse;
  uint8_t* ws = static_cast<uint8_t*>(t.ws);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.ml_off);
  p.part_o = reinterpret_cast<float*>(ws + plan.o_off);
  p.unit_slots = reinterpret_cast<int2*>(ws + plan.slots_off);
  p.w = t.w; p.w_cols = t.w_cols;
  p.lse2 = t.w != nullptr ? reinterpret_cast<float*>(ws + plan.lse_off) : nullptr;
  p.logits = t.w != nullptr && !plan.tiles128 ? reinterpret_cast<float*>(ws + plan.logits_off) : nullptr;
  p.q_image = t.w != nullptr && plan.tiles128 ? ws + plan.image_off : nullptr;
  p.q_scale = reinterpret_cast<float*>(ws + plan.scale_off);
  p.logit_w = plan.logit_w; p.logit_tokens = plan.logit_tokens;
  p.Hq = a.s.Hq; p.Hkv = a.s.Hkv; p.G = a.s.Hq / a.s.Hkv;
  p.page_log2 = 31 - __builtin_clz((unsigned)a.s.page);
  p.table_cols = a.s.table_cols; p.n = a.s.n; p.max_q = a.s.max_q; p.max_len = a.s.max_len;
  p.num_pages = a.cache.num_pages;
  // a window no sequence can outgrow hides nothing; the kernels' positions stay within 2^25
  p.window = t.mask.window < a.s.max_len ? t.mask.window : 0;
  p.sinks = t.mask.sinks < a.s.max_len ? t.mask.sinks : a.s.max_len;
  p.fp16 = a.s.dtype == THRIFT_FP16;
  p.nsplit = plan.nsplit; p.chunk = plan.chunk; p.row_tiles = plan.row_tiles;
  const float scale = t.mask.softmax_scale > 0.0f ? t.mask.softmax_scale : 1.0f / sqrtf((float)a.s.d);
  p.scale_log2 = scale * kv8::kLog2e;
  return a.s.d == 128 ? kv8::launch_attn_d<128>(p, plan, a.s, st) : kv8::launch_attn_d<64>(p, plan, a.s, st);
}

}  // namespace thrift
