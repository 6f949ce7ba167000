// Attention over the paged 8-bit cache: what its kernels share.
#pragma once
#include "kv8.cuh"

namespace thrift {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;

struct AttnParams {
  const uint8_t *k, *v, *ks, *vs;
  const void* q;
  long long q_stride;  // elements
  const int32_t *table, *lens, *cu;
  void* o;
  float* lse;
  // states of runs: maximum (log2 domain) and sum, and the unnormalised output; element
  // row * nsplit + run (prefill_kernel) or slot * R + row of the tile (split_kernel)
  float2* part_ml;
  float* part_o;
  int2* unit_slots;  // split_kernel: first slot and slots of a (sequence, kv head, row tile)
  float* lse2;      // [row] log2-domain log-sum-exp for the weights (or null)
  float* logits;    // split_kernel's logits for the weight sums, [sequence, kv head, row tile][token of the span][logit_w] (or null)
  uint8_t* q_image;  // prefill_kernel's query tiles and rows' scales for the weight sums (or null)
  float* q_scale;
  int logit_w, logit_tokens;
  float* w;
  long long w_cols;
  int Hq, Hkv, G, page_log2, table_cols, n, max_q, max_len, num_pages, window, sinks, fp16;
  int nsplit, chunk, row_tiles;  // prefill_kernel: runs per row, 128-token tiles of a run
  float scale_log2;
};

// The tokens that query rows at positions p_lo .. p_hi can see, as an index space of tiles
// of T tokens: [0, s_tiles) are the sinks' tiles, the rest start at tile a_tile.
template <int T>
struct Span {
  int s_tiles, a_tile, count;
  __device__ __forceinline__ int token(int v) const { return (v < s_tiles ? v : a_tile + (v - s_tiles)) * T; }
  // the place of a sequence's tile: `count` or more for one past the end or between the two parts
  __device__ __forceinline__ int index(int tile) const {
    return tile < s_tiles ? tile : tile >= a_tile ? tile - a_tile + s_tiles : 0x7FFFFFFF;
  }
};
template <int T>
__device__ __forceinline__ Span<T> visible_span(int p_lo, int p_hi, int window, int sinks) {
  Span<T> s{0, 0, 0};
  if (p_hi < 0) return s;
  if (window > 0) {
    const int a = max(0, p_lo - window + 1) / T;
    const int z = (min(sinks, p_hi + 1) + T - 1) / T;
    if (a > z) {
      s.s_tiles = z;
      s.a_tile = a;
    }
  }
  s.count = s.s_tiles + (p_hi + T) / T - s.a_tile;
  return s;
}

// A row's log-sum-exp from its maximum (log2 domain) and sum.
__device__ __forceinline__ void write_lse(const AttnParams& p, long long row, float m, float l) {
  const float x = l > 0.0f ? m + log2f(l) : -INFINITY;
  if (p.lse != nullptr) p.lse[row] = x * kLn2;
  if (p.lse2 != nullptr) p.lse2[row] = x;
}

// Row r's packed index (token * Hq + head).
__device__ __forceinline__ long long packed_row(const AttnParams& p, const Seq& s, int hk, int r) {
  return (long long)(s.q0 + r / p.G) * p.Hq + hk * p.G + r % p.G;
}
__device__ __forceinline__ const uint32_t* query_row(const AttnParams& p, const Seq& s, int hk, int r, int d) {
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + (long long)(s.q0 + r / p.G) * p.q_stride + (hk * p.G + r % p.G) * d;
  return reinterpret_cast<const uint32_t*>(q);
}

// Whether some row at positions p_lo .. p_hi sees some token of [a, a + n); whether all rows see all of them.
__device__ __forceinline__ bool any_visible(const AttnParams& p, int a, int n, int p_lo, int p_hi) {
  return a <= p_hi && (p.window == 0 || a + n - 1 > p_lo - p.window || a < p.sinks);
}
__device__ __forceinline__ bool all_visible(const AttnParams& p, int a, int n, int p_lo, int p_hi) {
  return a + n - 1 <= p_lo && (p.window == 0 || a > p_hi - p.window || a + n <= p.sinks);
}

// How a call is cut up.  The same for the workspace's size and the launch.
struct Plan {
  bool tiles128;  // prefill_kernel (128-row tiles) instead of split_kernel
  bool cluster;   // cluster_kernel instead of split_kernel and merge_kernel
  int nt, row_tiles, nsplit, chunk, ctas;
  size_t ml_off, o_off, slots_off, lse_off, logits_off, image_off, scale_off, bytes;
  int logit_w, logit_tokens;
};

cudaError_t launch_prefill(const AttnParams& p, const thrift_kv8_shape& s, cudaStream_t st);
cudaError_t launch_tile_weights(const AttnParams& p, const thrift_kv8_shape& s, cudaStream_t st);
constexpr int kPrefillRows = 256, kPrefillTile = 128;  // query rows of a CTA, tokens of its step

}  // namespace kv8
}  // namespace thrift
