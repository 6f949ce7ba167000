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
#include "kv8_split.cuh"

namespace thrift {
namespace kv8 {

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
// 5.3 us (kernels run over and over) where split_kernel and merge_kernel take 6.5 + 3.1; at four windows of 4096 tokens 14.3
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
// a thread adds up one token's rows with their final log-sum-exp.  The logits lie in the order of
// a row tile's span, so a window's take the window's room.  Storing them costs 8 bytes a row and
// token: 1/8 of the token's 2 D bytes of codes for 4 rows and D = 128, and as much as the codes
// for 32 rows; computing them again took as long as the attention itself (75 us of 142 at 32
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
  const int rows = s.nq * p.G, t0 = blockIdx.x * kWeightThreads * T + (int)threadIdx.x;
  const int tb = blockIdx.x * kWeightThreads * T;
  if (tb >= s.len || rows == 0 || !any_visible(p, tb, kWeightThreads * T, max(s.pos0, 0), s.len - 1)) return;
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
    const Span<kTile> span = visible_span<kTile>(s.pos0 + r0 / p.G, s.pos0 + (min(rows, r0 + R) - 1) / p.G, p.window, p.sinks);
    // a logit that its row does not see may be unwritten or have no place: one is loaded all the
    // same (without a branch, so that the loads go out together) and dropped
    float2 x[T][RW / 2];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const int tok = t0 + i * kWeightThreads, v = span.index(tok / kTile);
      const long long row = v < span.count ? (long long)v * kTile + tok % kTile : 0;
#pragma unroll
      for (int c = 0; c < RW / 2; ++c) x[i][c] = *reinterpret_cast<const float2*>(at + row * RW + 2 * c);
    }
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
  // (a row tile's span has at most `tiles` tiles, and those of the longest sequence)
  const long long whole = (s.max_len + kTile - 1) / kTile;
  p.logit_tokens = (int)(tiles < whole ? tiles : whole) * kTile;
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
