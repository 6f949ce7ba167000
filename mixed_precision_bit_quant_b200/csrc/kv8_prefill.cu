// Attention over the paged 8-bit cache for many query rows (prompt chunks, verification of
// several tokens): tcgen05 products on tiles of 128 query rows and 128 tokens.
//
// One CTA takes 256 rows of one kv head's group as two tiles of 128 and walks the visible
// tokens in tiles of 128 (or a run of them, whose state merge_kernel joins).  16 warps:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: one thread owns one query row (= TMEM
//              lane): S from TMEM, mask on edge tiles, running maximum, exponentials, P as
//              FP16 back into S's columns; O is rescaled only when a row's maximum grew by 2^6
//   warps 8-11 converters: a tile's K and V codes from global memory to FP16 in shared memory,
//              each loaded while the tile before it is converted or waited for
//   warp 12    tensor-memory allocator and issuer of S = Q K^T and O += P V; the row tiles
//              alternate, so that one tile's products run under the other's exponentials
// The products need one type for both operands: e4m3 codes are exact in FP16, with a
// page's scale relative to the largest of the run (2^(e - e_ref), exact down to 2^-24, that is
// for pages up to 2^21 smaller); the query enters as FP16 scaled by a power of two per row tile.
// A run whose pages' scales lie further apart (K: 2^21; V: 2^12, beyond which small weights on
// large pages would be lost in P's FP16) is walked as kv8_split.cuh does, where K and P carry each
// page's scale for itself (8.7 ms instead of 1.0 for the case below, every fifth page's V 2^21 smaller);
// only pages of exponent -127 (zeros, and values below 2^-118) may lie further below the
// others, and count as zero then.
// 4096 queries over 16389 tokens (32 heads of 128, 4 a kv head): 987 us, 975 TFLOP/s, in repeated
// calls (1015 us, 948 TFLOP/s, in turn with other work).  No pipe
// bounds it: at 2048 queries over 4096 tokens the tensor cores work 40 % of the clocks in the mean
// over the SMs (55 % on the busiest), the special-function unit 41 %, the ALUs 34 %.  A step's chain
// of waits does -- S to registers, maximum, exponentials, P to tensor memory, two products -- of
// which two row tiles keep two in flight; tensor memory holds no third.  Copies that skip work, at
// 990 us with all of it: no exponentials 968, no conversion 1004, an eighth of Q K^T and a quarter of
// P V 899, all three left out so 805.  Tried and slower: exp2 on the FMA pipe (1085, 1177 and 1256 us for 1, 3
// and 4 of 8 pairs, against 1051 for that build without), two threads a row (1225 against 990),
// persistent CTAs with equal shares of the steps (1140 to 1230 against 990).
#include "kv8_split.cuh"

namespace thrift {
namespace kv8 {

constexpr int kPfThreads = 512;
constexpr int kPfSoftmaxRegs = 192, kPfConvRegs = 72, kPfOtherRegs = 56;
static_assert(2 * kPfSoftmaxRegs + kPfConvRegs + kPfOtherRegs <= 512, "register split exceeds the launch budget");
constexpr uint64_t kPfWaitNs = 2000000000ull;  // 2 s per wait: far above any legitimate wait
constexpr int kUp = 6;          // codes enter FP16 times 2^6: at most 448 * 64 < 65504
constexpr float kPfLazy = 6.0f;  // a row's maximum is raised when exceeded by 2^6
constexpr float kTiny = 1.17549435e-38f;  // a logit's scale is never 0: -inf times it stays -inf
constexpr float kPfShift = 9.0f; // P enters FP16 times 2^9: at most 2^15
constexpr int kNearK = 21, kNearV = 12;  // exponents of a run's pages that lie at most this far apart

enum PfBar : int {
  KFULL = 0, KEMPTY = 2, VFULL = 4, VEMPTY = 6, SFULL = 8,
  PFULL = 10,  // [half of the tokens][row tile]
  PVDONE = 14, DRAIN = 16, NPFBAR = 17 };

template <int D>
struct PfLayout {
  static constexpr int TILE = 128 * D * 2;  // FP16 tile: D/64 blocks of 128 rows x 128 bytes, 128-byte swizzle
  static constexpr int OFF_Q = 0;             // two row tiles
  static constexpr int OFF_K = 2 * TILE;      // two stages
  static constexpr int OFF_V = 4 * TILE;      // two stages
  static constexpr int OFF_BAR = 6 * TILE;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NPFBAR + 8;  // tmem holder, abort, 12 + 8 + 8 words of the start
  static constexpr int BYTES = OFF_MISC + 128;
  // at least 116 KB, so that one CTA (and its 512 TMEM columns) owns an SM
  static constexpr int DYN = (BYTES + 1024 > 116 * 1024) ? BYTES + 1024 : 116 * 1024;
  static constexpr uint32_t S_COL = 0, O_COL = 256;  // S of tile t at 128 t (P over its first half), O at 256 + D t
};

// kind::f16 with FP16 inputs, FP32 accumulation, M = 128; `mn_b`: B is N-major (its rows are k).
__host__ __device__ constexpr uint32_t idesc_f16(int n, int mn_b) {
  return (1u << 4) | ((uint32_t)mn_b << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t hmul2_u32(uint32_t a, __half2 m) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), m);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The lowest n bits (n may be negative or above 32).
__device__ __forceinline__ uint32_t bits_below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

__device__ __forceinline__ void pf_raise(volatile int* abort) {
  *abort = 1;
  atomicOr(&g_error_word, 2u);
}

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) prefill_kernel(const AttnParams p) {
  using L = PfLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bk = blockIdx.y, b = bk / p.Hkv, hk = bk % p.Hkv;
  // the last rows of a prompt see the most tokens: they start first
  const int split = blockIdx.x % p.nsplit, rt = p.row_tiles - 1 - blockIdx.x / p.nsplit;
  const Seq s = load_seq(p.lens, p.cu, b, p.n, p.max_q, p.max_len);
  if (s.bad && tid == 0 && blockIdx.x == 0 && hk == 0) raise_bad();
  const int r_base = rt * kPrefillRows, r_cnt = min(s.nq * p.G - r_base, kPrefillRows);
  if (r_cnt <= 0) return;
  const int p_lo = s.pos0 + r_base / p.G, p_hi = s.pos0 + (r_base + r_cnt - 1) / p.G;
  const Span<kPrefillTile> span = visible_span<kPrefillTile>(p_lo, p_hi, p.window, p.sinks);
  const int v0 = split * p.chunk, nj = min(span.count, v0 + p.chunk) - v0;
  if (nj <= 0) {  // nothing in this run: an empty state, or rows that see nothing
    for (int r = tid; r < r_cnt; r += kPfThreads) {
      const long long row = packed_row(p, s, hk, r_base + r);
      if (p.nsplit > 1) {
        p.part_ml[row * p.nsplit + split] = make_float2(-INFINITY, 0.0f);
      } else {
        write_lse(p, row, -INFINITY, 0.0f);
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(p.o)[row * (D / 8) + c] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  const int ntile = r_cnt > 128 ? 2 : 1;

  auto BAR = [&](int k) -> uint32_t { return sb + L::OFF_BAR + 8 * k; };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  volatile uint32_t* ekey = misc + 2;  // of each of warps 12-15: largest exponents of K and of V, a bad page
  volatile uint32_t* qkey = misc + 14;  // of each softmax warp: its largest |q|, as bits
  volatile uint32_t* elow = misc + 22;  // of each of warps 12-15: smallest exponents above -127 of K and of V
  if (tid == 0) {
    for (int k = 0; k < NPFBAR; ++k)
      mbar_init(BAR(k), (k >= KFULL && k < KFULL + 2) || (k >= VFULL && k < VFULL + 2) || (k >= PFULL && k < PFULL + 4) ? 4 : 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(smem + L::OFF_MISC), 512);
    tmem_relinquish();
  }
  const int32_t* trow = p.table + (long long)b * p.table_cols;
  const int page_tok = 1 << p.page_log2;
  constexpr int LPR = D / 16, RPI = 32 / LPR;  // lanes per token, tokens per load of a warp
  const int cw = warp - 8, c = lane % LPR, rr = lane / LPR;
  // lane l of a batch: tile l / 2, group of 16 tokens 2 cw + (l & 1) of it
  int l_page = -1, l_ks = 0, l_vs = 0;
  auto batch = [&](int j0) {
    const int j = j0 + (lane >> 1);
    l_page = -1;
    if (j < nj) {
      const int tok = span.token(v0 + j) + 32 * cw + 16 * (lane & 1);
      if (any_visible(p, tok, 16, p_lo, p_hi)) {
        const int pg = __ldg(trow + (tok >> p.page_log2));
        if (pg >= 0 && pg < p.num_pages) {
          l_page = pg;
          l_ks = __ldg(p.ks + (long long)pg * p.Hkv + hk);
          l_vs = __ldg(p.vs + (long long)pg * p.Hkv + hk);
        }
      }
    }
  };
  // Where this lane's rows of group g (16 of the warp's 32 tokens) of tile j are.  A group that is not
  // to be read takes page 0 and is zeroed below: a load under a branch would be waited for
  // where the branches join.
  auto place = [&](const uint8_t* base, int j, int g) -> const uint8_t* {
    const int tok = span.token(v0 + j) + 32 * cw + 16 * g;
    const int pg = max(0, __shfl_sync(0xffffffffu, l_page, 2 * (j & 15) + g));
    return base + ((((long long)pg * p.Hkv + hk) << p.page_log2) + (tok & (page_tok - 1)) + rr) * D + 16 * c;
  };
  // The latencies of the start run side by side: the softmax warps load the query rows (whole
  // rows at a time: one row a thread took 4096 wavefronts), the converters the first tile's
  // codes, and the last four warps look through the run's pages.
  const int tile = warp >> 2;  // of a softmax warp
  const int row = (warp & 3) * 32 + lane;
  constexpr int QV = D / 8;  // 16-byte vectors of a query row
  uint4 uk[LPR], uv[LPR];    // converters: the next tile's codes; softmax warps: vectors 0 .. LPR - 1 and the rest of QV
  if (warp < 8) {
    if (tile < ntile) {
#pragma unroll
      for (int i = 0; i < QV; ++i) {
        const int at = row + 128 * i, r = min(tile * 128 + at / QV, r_cnt - 1);
        const uint4 u = ldg16_now(query_row(p, s, hk, r_base + r, D) + 4 * (at % QV));
        if (i < LPR) uk[i % LPR] = u;
        else uv[i % LPR] = u;
      }
      uint32_t am = 0;
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        am = __vmaxu2(am, __vmaxu2(__vmaxu2(uk[i].x & 0x7FFF7FFFu, uk[i].y & 0x7FFF7FFFu), __vmaxu2(uk[i].z & 0x7FFF7FFFu, uk[i].w & 0x7FFF7FFFu)));
        am = __vmaxu2(am, __vmaxu2(__vmaxu2(uv[i].x & 0x7FFF7FFFu, uv[i].y & 0x7FFF7FFFu), __vmaxu2(uv[i].z & 0x7FFF7FFFu, uv[i].w & 0x7FFF7FFFu)));
      }
      am = __reduce_max_sync(0xffffffffu, max(am & 0xFFFFu, am >> 16));
      if (lane == 0) qkey[warp] = am;
    }
  } else if (warp < 12) {
    batch(0);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint8_t* at = place(p.k, 0, g);
#pragma unroll
      for (int i = 0; i < LPR / 2; ++i) uk[g * (LPR / 2) + i] = ldg16_now(at + i * RPI * D);
    }
  } else {
    int ek = 0, ev = 0;
    uint32_t lk = 255, lv = 255;
    bool bad = false;
    const int per = page_tok < kPrefillTile ? kPrefillTile >> p.page_log2 : 1;  // pages of a tile
    for (int i = tid - 384; i < nj * per; i += 128) {
      const int tok = span.token(v0 + i / per) + (i % per) * page_tok;
      if (!any_visible(p, tok, page_tok, p_lo, p_hi)) continue;
      const int pg = __ldg(trow + (tok >> p.page_log2));
      if (pg < 0 || pg >= p.num_pages) {
        bad = true;
        continue;
      }
      const int ksc = __ldg(p.ks + (long long)pg * p.Hkv + hk), vsc = __ldg(p.vs + (long long)pg * p.Hkv + hk);
      ek = max(ek, ksc);
      ev = max(ev, vsc);
      if (ksc > 0) lk = min(lk, (uint32_t)ksc);
      if (vsc > 0) lv = min(lv, (uint32_t)vsc);
    }
    ek = __reduce_max_sync(0xffffffffu, ek);
    ev = __reduce_max_sync(0xffffffffu, ev);
    lk = __reduce_min_sync(0xffffffffu, lk);
    lv = __reduce_min_sync(0xffffffffu, lv);
    if (bad) raise_bad();
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
      ekey[warp - 12] = ek;
      ekey[warp - 8] = ev;
      ekey[warp - 4] = bad;
      elow[warp - 12] = lk;
      elow[warp - 8] = lv;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int kref = max(max(ekey[0], ekey[1]), max(ekey[2], ekey[3]));
  const int vref = max(max(ekey[4], ekey[5]), max(ekey[6], ekey[7]));
  const int klow = min(min(elow[0], elow[1]), min(elow[2], elow[3]));
  const int vlow = min(min(elow[4], elow[5]), min(elow[6], elow[7]));
  const bool bad_pages = (ekey[8] | ekey[9] | ekey[10] | ekey[11]) != 0;
  // The rows as FP16, scaled by a power of two.  The 128 rows of a tile share it (their largest
  // component lands in [2^14, 2^15)), so that a logit's scale is the tile's: a component 2^31
  // (BF16) times below the tile's largest loses bits, and then at most 2^-39 of it -- logits
  // are off by that much of the tile's largest possible one.
  float sc = 0.0f;  // of a logit
  if (warp < 8 && tile < ntile) {
    const uint32_t am = max(max(qkey[4 * tile], qkey[4 * tile + 1]), max(qkey[4 * tile + 2], qkey[4 * tile + 3]));
    const int e = max(-100, (int)(__float_as_uint(pair_to_float2(am, p.fp16).x) >> 23) - 127 - 14);
    const float down = pow2f(-e), qscale = pow2f(e) * p.scale_log2;
    sc = fmaxf(qscale * pow2f(max(-126, kref - 127 - kUp)), kTiny);
    // the weight sums' kernel reads the tile as it lies here
    uint8_t* image = nullptr;
    if (p.q_image != nullptr && split == 0) {
      const long long at = ((long long)bk * p.row_tiles + rt) * 2 + tile;
      image = p.q_image + at * L::TILE;
      if (row == 0) p.q_scale[at] = qscale;
    }
#pragma unroll
    for (int i = 0; i < QV; ++i) {
      const int at = row + 128 * i, r = at / QV, c = at % QV;
      const uint4 u = i < LPR ? uk[i % LPR] : uv[i % LPR];
      const uint32_t in[4] = {u.x, u.y, u.z, u.w};
      uint32_t h[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = pair_to_float2(in[x], p.fp16);
        const __half2 hh = __floats2half2_rn(f.x * down, f.y * down);
        h[x] = tile * 128 + r < r_cnt ? *reinterpret_cast<const uint32_t*>(&hh) : 0u;
      }
      const uint32_t off = (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      sts128(sb + L::OFF_Q + tile * L::TILE + off, make_uint4(h[0], h[1], h[2], h[3]));
      if (image != nullptr) *reinterpret_cast<uint4*>(image + off) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (kref - klow > kNearK || vref - vlow > kNearV) {
    // scales too far apart: four groups of four warps take 8 rows each as split_kernel does
    if (warp == 12) tmem_dealloc(tmem, 512);
    constexpr int F = kPrefillTile / kTile, GROUPS = kPfThreads / kSplitThreads;
    static_assert(GROUPS * split_smem(D, 1) <= L::OFF_BAR, "the groups' shared memory lies over the barriers");
    const Span<kTile> all{F * span.s_tiles, F * span.a_tile, F * span.count};
    float* sm = reinterpret_cast<float*>(smem + (tid / kSplitThreads) * split_smem(D, 1));
    for (int t = tid / kSplitThreads; 8 * t < r_cnt; t += GROUPS) {
      split_segment<D, 1, true>(p, s, b, hk, rt * (kPrefillRows / 8) + t, all, F * v0, F * (v0 + nj),
                                p.nsplit > 1 ? kToRun - split : kWhole, sm);
      split_sync<true>();  // shared memory is free again
    }
    return;
  }
  volatile int never = 0;

  if (warp >= 12) {
    regs_dec<kPfOtherRegs>();
    if (warp == 12) {
      // ------------------------------------------------------------ issuer (one converged warp)
      const uint32_t el = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t q_lo = desc_lo(sb + L::OFF_Q, 16), k_lo = desc_lo(sb + L::OFF_K, 16), v_lo = desc_lo(sb + L::OFF_V, 16384);
      constexpr uint32_t HI = desc_hi(1024, SWZ_128B), TSTEP = L::TILE >> 4;
      auto qk = [&](int t, int st) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
          mma_f16_ss_el(el, tm + L::S_COL + 128 * t, q_lo + t * TSTEP + off, HI, k_lo + st * TSTEP + off, HI,
                        idesc_f16(128, 0), k > 0);
        }
        tc_commit_el(el, BAR(SFULL + t));
      };
      auto wait = [&](int bar, int parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(BAR(bar), parity, abort, kPfWaitNs));
      };
      bool ok = wait(KFULL, 0);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < ntile; ++t) qk(t, 0);
        tc_commit_el(el, BAR(KEMPTY));
      }
      for (int j = 0; ok && j < nj; ++j) {
        const int st = j & 1, sn = st ^ 1;
        // operands first: once a tile's P is there, its products go out without another wait
        if (!wait(VFULL + st, (j >> 1) & 1) || (j + 1 < nj && !wait(KFULL + sn, ((j + 1) >> 1) & 1))) ok = false;
        for (int t = 0; ok && t < ntile; ++t) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && wait(PFULL + 2 * half + t, j & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)  // 16 tokens a step: 16 rows of 128 bytes
              mma_f16_ts_el(el, tm + L::O_COL + D * t, tm + L::S_COL + 128 * t + 8 * k, v_lo + st * TSTEP + 128 * k, HI,
                            idesc_f16(D, 1), (j > 0 || k > 0) ? 1u : 0u);
          }
          if (!ok) break;
          tc_commit_el(el, BAR(PVDONE + t));
          if (j + 1 < nj) qk(t, sn);
        }
        if (!ok) break;
        tc_commit_el(el, BAR(VEMPTY + st));
        if (j + 1 < nj) tc_commit_el(el, BAR(KEMPTY + sn));
      }
      if (!ok && lane == 0) pf_raise(abort);
      tc_commit_el(el, BAR(DRAIN));  // every product issued above completes before TMEM is released
      mbar_wait(BAR(DRAIN), 0, &never, kPfWaitNs);
    }
  } else if (warp >= 8) {
    regs_dec<kPfConvRegs>();
    // -------------------------------------------------------------- converters
    // K and V of a tile by one piece of code (the two roles' loops together are near what the
    // instruction cache holds: windowed prompts of 4096 took 120 us with a copy each, 117 with one): its
    // rows become FP16 in shared memory, and each register is loaded for the next half step as soon as it
    // is used.
    bool ok = true;
    for (int h = 0; h < 2 * nj; ++h) {
      const int op = h & 1, j = h >> 1, st = j & 1, use = j >> 1, tok = span.token(v0 + j) + 32 * cw;
      const int ref = op ? vref : kref, code = op ? l_vs : l_ks;
      __half2 m[2];
      bool held[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const int e = __shfl_sync(0xffffffffu, code, 2 * (j & 15) + g);
        held[g] = __shfl_sync(0xffffffffu, l_page, 2 * (j & 15) + g) >= 0;
        m[g] = __float2half2_rn(pow2f(max(-126, e - ref + kUp)));  // (0 below 2^-24)
      }
      if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(BAR(KEMPTY + 4 * op + st), (use - 1) & 1, abort, kPfWaitNs))) {
        ok = false;
        break;
      }
      // rows that no query row sees or whose page is not of the pool become zero (their codes
      // may be NaN)
      if (bad_pages || !all_visible(p, tok - 32 * cw, kPrefillTile, p_lo, p_hi)) {
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < LPR / 2; ++i)
            if (!held[g] || !any_visible(p, tok + 16 * g + i * RPI + rr, 1, p_lo, p_hi))
              uk[g * (LPR / 2) + i] = make_uint4(0, 0, 0, 0);
      }
      const int jn = min(j + op, nj - 1);  // the next half step's tile (past the end: the last again)
      if (op && ((j + 1) & 15) == 0) batch(j + 1);
      const uint32_t dst = sb + (op ? L::OFF_V : L::OFF_K) + st * L::TILE;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint8_t* at = place(op ? p.k : p.v, jn, g);
        const __half2 f = m[g];
#pragma unroll
        for (int i2 = 0; i2 < LPR / 2; ++i2) {
          const int i = g * (LPR / 2) + i2, r = 32 * cw + i * RPI + rr;
          const uint4 u = uk[i];
          const uint4 lo = make_uint4(hmul2_u32(e4m3x2_to_h2(u.x & 0xFFFFu), f), hmul2_u32(e4m3x2_to_h2(u.x >> 16), f),
                                      hmul2_u32(e4m3x2_to_h2(u.y & 0xFFFFu), f), hmul2_u32(e4m3x2_to_h2(u.y >> 16), f));
          const uint4 hi = make_uint4(hmul2_u32(e4m3x2_to_h2(u.z & 0xFFFFu), f), hmul2_u32(e4m3x2_to_h2(u.z >> 16), f),
                                      hmul2_u32(e4m3x2_to_h2(u.w & 0xFFFFu), f), hmul2_u32(e4m3x2_to_h2(u.w >> 16), f));
          uk[i] = ldg16_now(at + i2 * RPI * D);
          // chunks 2c and 2c + 1 of the row; the row's second half writes them in the other
          // order, so that eight lanes' stores meet all banks
          const int ch = 2 * c, blk = ch >> 3, x0 = (ch & 7), sw = (c >> 2) & 1;
          const uint32_t rowa = dst + blk * 16384 + r * 128;
          sts128(rowa + (((x0 + sw) ^ (r & 7)) << 4), sw ? hi : lo);
          sts128(rowa + (((x0 + 1 - sw) ^ (r & 7)) << 4), sw ? lo : hi);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(KFULL + 4 * op + st));
    }
    if (!ok && lane == 0) pf_raise(abort);
  } else {
    regs_inc<kPfSoftmaxRegs>();
    // -------------------------------------------------------------- softmax
    if (tile < ntile) {
      const int r = tile * 128 + row;  // row of the CTA
      const int pos = r < r_cnt ? s.pos0 + (r_base + r) / p.G : -1;
      const int t_lo = s.pos0 + (r_base + tile * 128) / p.G;
      const int t_hi = s.pos0 + (r_base + min(r_cnt, tile * 128 + 128) - 1) / p.G;
      const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t s_addr = lane_base + L::S_COL + 128 * tile, o_addr = lane_base + L::O_COL + D * tile;
      const bool idle = tile * 128 + (warp & 3) * 32 >= r_cnt;
      float m_ref = -INFINITY, l = 0.0f;
      bool ok = true;
      for (int j = 0; j < nj; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(BAR(SFULL + tile), j & 1, abort, kPfWaitNs))) { ok = false; break; }
        tc_fence_after();
        if (idle) {  // no row of this warp is one of the call's
          if (lane == 0) {
            mbar_arrive(BAR(PFULL + tile));
            mbar_arrive(BAR(PFULL + 2 + tile));
          }
          continue;
        }
        uint32_t v[4][32];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) tmem_ld32(s_addr + 32 * c4, v[c4]);
        const int tok = span.token(v0 + j);
        const bool edge = bad_pages || !all_visible(p, tok, kPrefillTile, t_lo, t_hi);
        uint32_t see[4] = {0, 0, 0, 0};
        if (edge) {
          // columns [lo, hi] are in sight, and those below `sk`
          const int hi = pos - tok, lo = p.window > 0 ? pos - p.window + 1 - tok : 0;
          const int sk = p.window > 0 ? min(p.sinks - tok, hi + 1) : 0;
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4)
            see[c4] = (bits_below(hi + 1 - 32 * c4) & ~bits_below(lo - 32 * c4)) | bits_below(sk - 32 * c4);
          if (bad_pages) {  // tokens of pages that are not of the pool
            for (int g = 0; g < 8; ++g) {
              const int tg = tok + 16 * g;
              if (!any_visible(p, tg, 16, p_lo, p_hi)) continue;
              const int pg = __ldg(trow + (tg >> p.page_log2));
              if (pg < 0 || pg >= p.num_pages) see[g >> 1] &= ~(0xFFFFu << (16 * (g & 1)));
            }
          }
        }
        // the row's maximum (all loads are waited for at once: a wait a chunk cost their latency each)
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) tmem_ld_wait32(v[c4]);
        float mc[4];
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {
          if (edge) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(see[c4] & (1u << c))) v[c4][c] = __float_as_uint(-INFINITY);
          }
          float t1[11];
#pragma unroll
          for (int c = 0; c < 10; ++c)
            t1[c] = fmax3(__uint_as_float(v[c4][3 * c]), __uint_as_float(v[c4][3 * c + 1]), __uint_as_float(v[c4][3 * c + 2]));
          t1[10] = fmaxf(__uint_as_float(v[c4][30]), __uint_as_float(v[c4][31]));
          mc[c4] = fmax3(fmax3(t1[0], t1[1], t1[2]), fmax3(t1[3], t1[4], t1[5]),
                         fmax3(fmax3(t1[6], t1[7], t1[8]), t1[9], t1[10]));
        }
        const float mloc = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])) * sc;
        float alpha = 1.0f;
        const bool grow = mloc > m_ref + kPfLazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = fmaxf(m_ref, mloc);
          alpha = m_ref == -INFINITY ? 0.0f : ex2_approx(m_ref - m_new);
          m_ref = m_new;
          l *= alpha;
          if (j > 0) {
            if (!__all_sync(0xffffffffu, mbar_wait(BAR(PVDONE + tile), (j - 1) & 1, abort, kPfWaitNs))) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int c4 = 0; c4 < D / 16; ++c4) {  // 16 columns at a time: S's 128 registers are live
              uint32_t o[16];
              tmem_ld16(o_addr + 16 * c4, o);
              tmem_ld_wait();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st16(o_addr + 16 * c4, o);
            }
          }
        }
        const float nb = m_ref == -INFINITY ? 0.0f : kPfShift - m_ref;
        const uint64_t sc2 = f2pack(sc, sc), nb2 = f2pack(nb, nb);
        uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            const uint64_t y = ffma2(f2pack(__uint_as_float(v[ch][2 * t]), __uint_as_float(v[ch][2 * t + 1])), sc2, nb2);
            float a0, a1;
            f2unpack(y, a0, a1);
            a0 = ex2_approx(a0);
            a1 = ex2_approx(a1);
            acc[t & 3] = fadd2(acc[t & 3], f2pack(a0, a1));
            const __half2 h = __floats2half2_rn(a0, a1);
            pk[t] = *reinterpret_cast<const uint32_t*>(&h);
          }
          tmem_st16(s_addr + 16 * ch, pk);
          if (ch & 1) {  // half of the tokens: their part of O += P V may start
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(PFULL + ch - 1 + tile));
          }
        }
        float x0, x1, x2, x3;
        f2unpack(fadd2(acc[0], acc[1]), x0, x1);
        f2unpack(fadd2(acc[2], acc[3]), x2, x3);
        l += (x0 + x1) + (x2 + x3);
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(BAR(PVDONE + tile), (nj - 1) & 1, abort, kPfWaitNs));
      if (!ok) {
        if (lane == 0) pf_raise(abort);
      } else {
        tc_fence_after();
        const long long prow = r < r_cnt ? packed_row(p, s, hk, r_base + r) : -1;
        // codes' units back to values: 2^(e_ref - 6), in two steps (e_ref may be -127)
        const float back = scale_value((uint32_t)vref), down = 1.0f / (1 << kUp);
        const float f = p.nsplit > 1 ? down : (l > 0.0f ? down / l : 0.0f);
        // The tile's query rows are done with: each thread leaves its row there (16-byte chunks,
        // swizzled as the operands are) and the warp writes its 32 rows out in whole lines;
        // a partial output's FP32 rows go in two halves.
        const uint32_t stage = sb + L::OFF_Q + tile * L::TILE;
        const bool part = p.nsplit > 1;
        for (int half = 0; half < (part ? 2 : 1); ++half) {
#pragma unroll
          for (int c4 = 0; c4 < D / 32; ++c4) {
            if (part && c4 / (D / 64) != half) continue;
            uint32_t o[32];
            tmem_ld32(o_addr + 32 * c4, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f * back);
            if (!part) {
#pragma unroll
              for (int c = 0; c < 16; ++c)
                o[c] = float2_to_pair(__uint_as_float(o[2 * c]), __uint_as_float(o[2 * c + 1]), p.fp16);
            }
            const int ch0 = part ? 8 * (c4 % (D / 64)) : 4 * c4;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (!part && c >= 4) continue;
              const int ch = ch0 + c;
              sts128(stage + (ch >> 3) * 16384 + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                     make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
            }
          }
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < QV; ++i) {
            const int at = lane + 32 * i, rl = at / QV, ch = at % QV, rw = (warp & 3) * 32 + rl;
            const uint4 x = *reinterpret_cast<const uint4*>(smem + L::OFF_Q + tile * L::TILE + (ch >> 3) * 16384 + rw * 128 +
                                                            (((ch & 7) ^ (rw & 7)) << 4));
            const long long to = __shfl_sync(0xffffffffu, prow, rl);
            if (to >= 0) {
              if (part) reinterpret_cast<uint4*>(p.part_o)[(to * p.nsplit + split) * (D / 4) + half * QV + ch] = x;
              else reinterpret_cast<uint4*>(p.o)[to * QV + ch] = x;
            }
          }
          __syncwarp();
        }
        if (r < r_cnt) {
          if (part) p.part_ml[prow * p.nsplit + split] = make_float2(l > 0.0f ? m_ref - kPfShift : -INFINITY, l);
          else write_lse(p, prow, m_ref - kPfShift, l);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// The weight sums of many rows: w[t] += sum over rows exp(s - lse).
//
// One CTA takes 128 tokens of a sequence and kv head and walks the tiles of 128 query rows
// that see them: S^T = K Q^T puts a token on a TMEM lane, so a token's sum over rows
// is a thread's sum over columns -- no exchange, and in a fixed order.  K's codes enter bare, and a
// page's scale multiplies its tokens' logits: a thread's own factor.
//   warps 0-3, 4-7  the even and the odd row tiles' exponentials and sums
//   warp 8     brings the row tiles' FP16 images, which prefill_kernel left in the workspace,
//              by bulk copies, and the rows' scales and log-sum-exps
//   warp 9     tensor-memory allocator and issuer
// Two CTAs an SM: the exponentials of one run under the other's waits.  Making the images here,
// once per token tile, took 368 us where this takes 115 (1996 new tokens of two sequences of 4096
// and 1933, 32 heads).  Bound by the exponentials (16 a clock and SM) and, next, by the waits of
// 1.3 waves of CTAs.
// ---------------------------------------------------------------------------
// The rows' numbers lie in six slots: when warp 8 fills tile j's, product j - 2 has completed,
// so S of tile j - 4 was read and tile j - 6, the slot's last, is done with.
constexpr int kTwStages = 2, kTwRowSlots = 6, kTwThreads = 320;
enum TwBar : int { QFULL = 0, QEMPTY = 2, WFULL = 4, WEMPTY = 6, WDRAIN = 8, ROWS = 9, NTWBAR = ROWS + kTwRowSlots };

template <int D>
struct TwLayout {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = TILE;                        // kTwStages row tiles
  static constexpr int OFF_ROW = OFF_Q + kTwStages * TILE;  // [slot] 128 rows' -lse, the tile's scale
  static constexpr int ROW = 528;
  static constexpr int OFF_SUM = OFF_ROW + kTwRowSlots * ROW;  // [128] the odd tiles' sums
  static constexpr int OFF_BAR = OFF_SUM + 512;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NTWBAR + 8;
  static constexpr int DYN = OFF_MISC + 32 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kTwThreads, 2) tile_weights_kernel(const AttnParams p) {
  using L = TwLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bk = blockIdx.y, b = bk / p.Hkv, hk = bk % p.Hkv;
  const Seq s = load_seq(p.lens, p.cu, b, p.n, p.max_q, p.max_len);
  const int t0 = blockIdx.x * 128;
  // the rows that see some of the tokens, in whole tiles
  const int i0 = max(0, t0 - s.pos0);
  int i1 = s.nq;
  if (p.window > 0 && t0 >= p.sinks) i1 = min(i1, t0 + 127 + p.window - s.pos0);
  if (t0 >= s.len || i0 >= i1) return;
  const int rows = s.nq * p.G, rt0 = i0 * p.G / 128, nt = (i1 * p.G + 127) / 128 - rt0;

  auto BAR = [&](int k) -> uint32_t { return sb + L::OFF_BAR + 8 * k; };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 4);
  if (tid == 0) {
    for (int k = 0; k < NTWBAR; ++k) mbar_init(BAR(k), k >= WEMPTY && k < WDRAIN ? 4 : 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(smem + L::OFF_MISC), 256);
    tmem_relinquish();
  }
  const int32_t* trow = p.table + (long long)b * p.table_cols;
  // Whether some row sees a token whose page is of the pool, and the place of the page's head.
  // The table's entries of pages that none sees may be stale numbers of the pool: neither their
  // codes nor their scales are read.
  auto place = [&](int tok, long long& ph) -> bool {
    if (tok >= s.len || !any_visible(p, tok, 1, s.pos0, s.len - 1)) return false;
    const int pg = __ldg(trow + (tok >> p.page_log2));
    ph = (long long)pg * p.Hkv + hk;
    return pg >= 0 && pg < p.num_pages;
  };
  bool held = false;  // this thread's token has a place
  float kf = 0.0f;    // and its page this scale
  if (warp < 8) {
    // K's codes as FP16
    constexpr int VR = D / 16, ITEMS = 128 * VR / 256;
    uint4 u[ITEMS];
    long long ph;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int it = tid + 256 * i, tok = t0 + it / VR;
      u[i] = make_uint4(0, 0, 0, 0);
      if (place(tok, ph))
        u[i] = __ldg(reinterpret_cast<const uint4*>(p.k + ((ph << p.page_log2) + (tok & ((1 << p.page_log2) - 1))) * D) + it % VR);
    }
    held = place(t0 + (tid & 127), ph);
    if (held) kf = scale_value(__ldg(p.ks + ph));
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int it = tid + 256 * i, r = it / VR, ch = 2 * (it % VR);
      const uint32_t rowa = sb + L::OFF_K + (ch >> 3) * 16384 + r * 128;
      sts128(rowa + (((ch & 7) ^ (r & 7)) << 4),
             make_uint4(e4m3x2_to_h2(u[i].x & 0xFFFFu), e4m3x2_to_h2(u[i].x >> 16),
                        e4m3x2_to_h2(u[i].y & 0xFFFFu), e4m3x2_to_h2(u[i].y >> 16)));
      sts128(rowa + ((((ch & 7) + 1) ^ (r & 7)) << 4),
             make_uint4(e4m3x2_to_h2(u[i].z & 0xFFFFu), e4m3x2_to_h2(u[i].z >> 16),
                        e4m3x2_to_h2(u[i].w & 0xFFFFu), e4m3x2_to_h2(u[i].w >> 16)));
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  volatile int never = 0;
  float sum = 0.0f;
  bool ok = true;

  if (warp == 9) {
    const uint32_t el = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t k_lo = desc_lo(sb + L::OFF_K, 16), q_lo = desc_lo(sb + L::OFF_Q, 16);
    constexpr uint32_t HI = desc_hi(1024, SWZ_128B), TSTEP = L::TILE >> 4;
    for (int j = 0; j < nt; ++j) {
      const int st = j % kTwStages, buf = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(BAR(QFULL + st), (j / kTwStages) & 1, abort, kPfWaitNs) &&
                                       (j < 2 || mbar_wait(BAR(WEMPTY + buf), ((j >> 1) - 1) & 1, abort, kPfWaitNs)))) {
        if (lane == 0) pf_raise(abort);
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
        mma_f16_ss_el(el, tm + 128 * buf, k_lo + off, HI, q_lo + st * TSTEP + off, HI, idesc_f16(128, 0), k > 0);
      }
      tc_commit_el(el, BAR(QEMPTY + st));
      tc_commit_el(el, BAR(WFULL + buf));
    }
    tc_commit_el(el, BAR(WDRAIN));
    mbar_wait(BAR(WDRAIN), 0, &never, kPfWaitNs);
  } else if (warp == 8) {
    const long long tile0 = (long long)bk * p.row_tiles * 2 + rt0;
    int issued = 0;
    float lse2[4], qs;
    // loads without a branch (clamped to the last row): they are not waited for before use
    auto fetch = [&](int j) {
      const int jj = min(j, nt - 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) lse2[i] = ldg4_now(p.lse2 + packed_row(p, s, hk, min((rt0 + jj) * 128 + 4 * lane + i, rows - 1)));
      qs = ldg4_now(p.q_scale + tile0 + jj);
    };
    fetch(0);
    for (int j = 0; j < nt; ++j) {
      const int st = j % kTwStages;
      if (j >= kTwStages && !__all_sync(0xffffffffu, mbar_wait(BAR(QEMPTY + st), (j / kTwStages - 1) & 1, abort, kPfWaitNs))) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_expect_tx(BAR(QFULL + st), L::TILE);
        bulk_load(sb + L::OFF_Q + st * L::TILE, p.q_image + (tile0 + j) * L::TILE, L::TILE, BAR(QFULL + st));
      }
      issued = j + 1;
      // a row that sees nothing (lse = -inf) or is none gets -inf: its exponentials are 0
#pragma unroll
      for (int i = 0; i < 4; ++i)
        lse2[i] = (rt0 + j) * 128 + 4 * lane + i >= rows || lse2[i] == -INFINITY ? -INFINITY : -lse2[i];
      float* rp = reinterpret_cast<float*>(smem + L::OFF_ROW + (j % kTwRowSlots) * L::ROW);
      reinterpret_cast<float4*>(rp)[lane] = make_float4(lse2[0], lse2[1], lse2[2], lse2[3]);
      if (lane == 0) rp[128] = qs;
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(ROWS + j % kTwRowSlots));
      fetch(j + 1);
    }
    if (!ok) {  // the copies in flight land before the CTA's shared memory goes away
      if (lane == 0) pf_raise(abort);
      for (int k = 0; k < kTwStages && k < issued; ++k) {
        const int n = issued - 1 - k;
        mbar_wait(BAR(QFULL + n % kTwStages), (n / kTwStages) & 1, &never, kPfWaitNs / 4);
      }
    }
  } else {
    const int grp = warp >> 2, tok = t0 + (warp & 3) * 32 + lane;
    const uint32_t base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 128 * grp;
    uint64_t acc[2] = {0, 0};
    for (int j = grp; j < nt; j += 2) {
      if (!__all_sync(0xffffffffu, mbar_wait(BAR(WFULL + grp), (j >> 1) & 1, abort, kPfWaitNs) &&
                                       mbar_wait(BAR(ROWS + j % kTwRowSlots), (j / kTwRowSlots) & 1, abort, kPfWaitNs))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float4* rp = reinterpret_cast<const float4*>(smem + L::OFF_ROW + (j % kTwRowSlots) * L::ROW);
      const float sc = fmaxf(reinterpret_cast<const float*>(rp)[128] * kf, kTiny);
      const uint64_t sc2 = f2pack(sc, sc);
      const int r0 = (rt0 + j) * 128;
      const bool edge = !all_visible(p, t0, 128, s.pos0 + r0 / p.G, s.pos0 + (min(rows, r0 + 128) - 1) / p.G);
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        uint32_t v[32];
        tmem_ld32(base + 32 * c4, v);
        tmem_ld_wait();
        if (c4 == 3) {  // S is read: its buffer may take the next product
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(BAR(WEMPTY + grp));
        }
        if (edge) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int pos = s.pos0 + (r0 + 32 * c4 + c) / p.G;
            const bool see = tok <= pos && (p.window == 0 || tok > pos - p.window || tok < p.sinks);
            if (!see) v[c] = __float_as_uint(-INFINITY);
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 nl = rp[8 * c4 + i];
          float a0, a1;
          f2unpack(ffma2(f2pack(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), sc2, f2pack(nl.x, nl.y)), a0, a1);
          acc[0] = fadd2(acc[0], f2pack(ex2_approx(a0), ex2_approx(a1)));
          f2unpack(ffma2(f2pack(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), sc2, f2pack(nl.z, nl.w)), a0, a1);
          acc[1] = fadd2(acc[1], f2pack(ex2_approx(a0), ex2_approx(a1)));
        }
      }
    }
    if (!ok && lane == 0) pf_raise(abort);
    float a0, a1;
    f2unpack(fadd2(acc[0], acc[1]), a0, a1);
    sum = a0 + a1;
    if (grp == 1) reinterpret_cast<float*>(smem + L::OFF_SUM)[tok - t0] = sum;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  if (tid < 128 && held) {
    float* w = p.w + (long long)bk * p.w_cols + t0 + tid;
    *w += sum + reinterpret_cast<const float*>(smem + L::OFF_SUM)[tid];
  }
}

template <int D>
static cudaError_t launch_prefill_d(const AttnParams& p, const thrift_kv8_shape& s, cudaStream_t st) {
  auto kern = prefill_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, PfLayout<D>::DYN);
  if (e != cudaSuccess) return e;
  kern<<<dim3(p.nsplit * p.row_tiles, s.B * s.Hkv), kPfThreads, PfLayout<D>::DYN, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_prefill(const AttnParams& p, const thrift_kv8_shape& s, cudaStream_t st) {
  return s.d == 128 ? launch_prefill_d<128>(p, s, st) : launch_prefill_d<64>(p, s, st);
}

template <int D>
static cudaError_t launch_tile_weights_d(const AttnParams& p, const thrift_kv8_shape& s, cudaStream_t st) {
  auto kern = tile_weights_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, TwLayout<D>::DYN);
  if (e != cudaSuccess) return e;
  kern<<<dim3((s.max_len + 127) / 128, s.B * s.Hkv), kTwThreads, TwLayout<D>::DYN, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tile_weights(const AttnParams& p, const thrift_kv8_shape& s, cudaStream_t st) {
  return s.d == 128 ? launch_tile_weights_d<128>(p, s, st) : launch_tile_weights_d<64>(p, s, st);
}

}  // namespace kv8

cudaError_t read_and_clear_kv8_prefill_error(uint32_t* word) { return kv8::read_and_clear_word(word); }

}  // namespace thrift
