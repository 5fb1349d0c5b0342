// Attention of tiles of query rows over a range of cached positions, on tcgen05.
//
// Serves two operations with one body:
//   * role prefill: group b is a sequence, its query rows are the sequence's last n_b positions;
//     the row at p sees  DENSE: t <= p,  STREAM: t <= p and (t < sink or t > p - window);
//   * shared-prefix decode: group i is a prefix, its query rows are the sequences that continue it,
//     and every row sees all P_i tokens.
//
// Rows.  The G q heads of a KV head read the same K / V rows, so a tile of 128 matrix rows packs
// PT = 128 / G tokens x G heads (row r: token r / G, head r % G; G = 7 fills 126 of 128).  A CTA
// owns two such tiles of one group and KV head, and `splits` CTAs share their key range when there
// are few tiles.
//
// Pipeline.  One warp brings Q once and then K and V tiles of BN tokens by TMA (128-byte swizzle)
// into a ring of ST tiles; one thread issues, for tile t = 0, 1 in turn,
//     O_t += P_t V_j  (P from TMEM),   S_t = Q_t K_{j+1}^T,
// so that while the tensor core works for one tile the four warps of the other turn its scores into
// weights; one thread holds one row, no shuffles.  S_t and P_t share TMEM columns: MMAs of one
// thread run in issue order, so P_t has been read when S_t is overwritten.
//     TMEM columns: S_0 / P_0 [0, 128), S_1 / P_1 [128, 256), O_0 [256, 256 + D), O_1 behind it.
//
// Softmax.  m is a reference value of the row, not always its running maximum: weights are
// 2^(scale (s - m)), and O and l are rescaled only when the maximum has outgrown m by more than 2^8, which
// is seldom after a row's first tile (the relative rounding of weights, O and l does not depend on m).
// A limit of 2^60 measured the same (383 us a prompt of 8192, 439 us 1000 tokens on 32768, either way) and
// took 2^52 from the values that O can hold: it is not yet divided by l, so 2^8 L max |v| has to stay in fp32.
//
// Weights in the product with V: PARTS = 1 rounds them to bf16 (2^-9 relative, of the order of the
// rounding of a bf16 output); PARTS = 3, for fp32 outputs, keeps 24 bits as three bf16 terms, each
// multiplied with V (two terms and key tiles of 128 were a tenth faster and twice as far off).  Two terms for
// bf16 outputs, too, took 490 us instead of 383 on a prompt of 8192 and 566 instead of 439 on 1000 tokens behind
// 31768; with one the output is 1.3 to 1.4 times as far from the exact value as its own rounding takes it.
//
// Segments.  The accumulation in TMEM drops the bits below the accumulator's last, always towards zero, which
// adds up along a row (9e-6 after 3600 tokens of random values, 6e-3 after a million of one sign).  A
// row's O is therefore added to a partial in memory (which stays in L2) after every segment of key tiles,
// and begins again from zero: after 256 tokens with PARTS = 3, after 131072 with PARTS = 1, where shorter rows
// need no partial.
//
// Bound and measured (B200).  Long rows run at the pace of one tile's chain: scores from TMEM, maximum,
// exponentials (a quarter of them on the FMA pipe), weights back, then the products of both tiles: 3050
// cycles per 128 keys and two tiles where the products alone take 2048.  1000 new tokens on 32768
// (32 heads on 8, d 128): 433 us, 1220 TFLOP/s on 128 of 148 SMs, and 505 us, 1050 TFLOP/s in a long run at the
// power limit; a prompt of 8192 with 2 of 8 groups retrieval heads: 382 us, 1186 TFLOP/s, and 445; ragged
// prompts of 301 to 2500: 91 us, 585 TFLOP/s (short CTAs: setting up and taking out cost as much as five
// key tiles).  96 sequences behind two documents of 20011 to 32768: 142 us with their own tokens.
#pragma once

#include <type_traits>

#include "dense_pass.cuh"

namespace aoh {

constexpr int kTaThreads = 384;       // softmax of tile 0, of tile 1, and a warpgroup of load / MMA warps
constexpr int kTaRegsSoftmax = 208;   // 2 x 128 x 208 + 128 x 88 = 384 x 168 registers
constexpr int kTaRegsOther = 88;
constexpr int kTaRegsLaunch = 168;
constexpr int kTaPoly = 1, kTaPolyOf = 4;  // of kTaPolyOf pairs of weights, kTaPoly come from the FMA pipe
constexpr int kTaSegment = 4;         // key tiles of a segment, PARTS = 3: 9.5e-7 off (fp32 torch operations: 2e-7 to
                                      // 3e-6).  8: 1.7e-6, 131 us instead of 142 on 96 sequences behind two documents
                                      // and the same on 64 behind 8192 tokens; 2: 5.6e-7, 174 us
constexpr int kTaSegmentLong = 1024;  // the same, PARTS = 1
constexpr int kTaSplitTiles = 16;     // key tiles of a split at least, where every split leaves partials
constexpr float kTaGrowth = 8.f;      // log2 of the largest weight before a rescale

template <int D, int PARTS>
struct TaTile {
  static constexpr int BN = PARTS == 1 ? 128 : 64;  // tokens per K / V tile: 128 columns hold S and the P parts
  static constexpr int C0 = BN / 2;                 // tokens whose weights go to the product first, while the
                                                    // others' are computed
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kKvBytes = BN * D * 2;
  static constexpr int kRing = (229 * 1024 - 5 * 1024 - 2 * kQBytes) / kKvBytes;
  static constexpr int ST = kRing > 12 ? 12 : kRing;
  static constexpr int kSmem = 1024 + 2 * kQBytes + ST * kKvBytes;
};

struct alignas(64) TileParams {
  CUtensorMap qmap, kmap, vmap;
  const int32_t* offsets;    // [B + 1] of the cache
  const int32_t* lengths;    // [B] or null
  const int32_t* q_offsets;  // [B + 1] rows of every group, or null: one group of all rows
  uint16_t* out;             // splits == 1: bf16 [total_q][Hq][D]
  // else partials per (split, tile of rows): rows are the fastest index, a row per lane
  float2* part_ml;           // (m, l) [splits][tiles][128], m times scale_log2
  float4* part_acc;          // [splits][tiles][D / 4][128]
  int32_t B, Hq, G, PT, total_q, sink, window, splits, n_listed, slots;
  int32_t segment;           // key tiles of a segment (PARTS = 1; more than any row has: no room for partials)
  float scale_log2;          // > 0; a negative scale negates Q in the product
  uint32_t neg;
  uint8_t heads[kMaxHeads];
  uint8_t roles[kMaxHeads];
  uint8_t slot[kMaxHeads];
};

// The group and first row of CTA `slot`: group b's tiles of P2 rows take the slots from
// floor((q_offsets[b] + b (P2 - 1)) / P2) on, room for ceil(n_b / P2) of them.
struct TaPlace {
  int b, i0, n, q0, off, L;
};
__device__ __forceinline__ bool ta_locate(const TileParams& p, int slot, TaPlace* w) {
  const int P2 = 2 * p.PT;
  int lo = 0, hi = p.B - 1, s0 = 0, q1 = p.total_q;
  w->q0 = 0;
  if (p.q_offsets) {
    auto first = [&](int i) { return (int)(((int64_t)p.q_offsets[i] + (int64_t)i * (P2 - 1)) / P2); };
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first(mid) <= slot) lo = mid; else hi = mid - 1;
    }
    w->q0 = p.q_offsets[lo];
    q1 = p.q_offsets[lo + 1];
    s0 = first(lo);
  } else {
    lo = 0;
  }
  w->b = lo;
  w->L = seq_length(p.offsets, p.lengths, lo, false, &w->off);
  w->n = q1 - w->q0;
  const int64_t i = (int64_t)(slot - s0) * P2;
  w->i0 = (int)i;
  return w->q0 >= 0 && i >= 0 && i < w->n && w->q0 + i < p.total_q;  // (rows past those of q are recorded)
}

// 2^x of two numbers without the special-function unit, x <= kTaGrowth: x = i + f with |f| <= 1/2 (i by adding
// 1.5 * 2^23), 2^f as a cubic, i added to the exponent.  The cubic is 1 at 0 and fitted here to the
// smallest relative error, 2^-13.3: a twentieth of the rounding of the weight to bf16 that follows.  x is
// raised to -127, where the sum of the exponents is zero and so is the result (a subnormal just above).
static_assert(kTaGrowth <= 126.f, "the exponent that ex2_poly adds to stays below 255");
constexpr float kEx2C1 = 0.693282902f, kEx2C2 = 0.242210954f, kEx2C3 = 0.0550089292f;

__device__ __forceinline__ void ex2_poly(uint64_t v, float& x, float& y) {
  f2_split(v, x, y);
  const uint64_t c = f2(fmaxf(x, -127.f), fmaxf(y, -127.f));
  const uint64_t i = f2_add(c, f2(12582912.f, 12582912.f));
  const uint64_t f = f2_add(c, f2_fma(f2_add(i, f2(-12582912.f, -12582912.f)), f2(-1.f, -1.f), 0));
  uint64_t r = f2_fma(f2(kEx2C3, kEx2C3), f, f2(kEx2C2, kEx2C2));
  r = f2_fma(r, f, f2(kEx2C1, kEx2C1));
  r = f2_fma(r, f, f2(1.f, 1.f));
  float ix, iy;
  f2_split(i, ix, iy);
  f2_split(r, x, y);
  x = __uint_as_float(__float_as_uint(x) + (__float_as_uint(ix) << 23));
  y = __uint_as_float(__float_as_uint(y) + (__float_as_uint(iy) << 23));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D, int PARTS>
__global__ void __launch_bounds__(kTaThreads, 1) tile_attend_kernel(const __grid_constant__ TileParams p) {
  using T = TaTile<D, PARTS>;
  constexpr int BN = T::BN, ST = T::ST, C0 = T::C0;
  constexpr uint32_t kO = 256;
  extern __shared__ uint8_t ta_smem[];
  __shared__ __align__(8) uint64_t s_bar[2 * ST + 11];
  __shared__ uint32_t s_tmem;
  __shared__ int s_stop;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), wg = warp >> 2;  // the same register for the whole warp
  const uint32_t smem = (smem_u32(ta_smem) + 1023u) & ~1023u;
  const uint32_t q_s = smem, kv_s = smem + 2 * T::kQBytes;
  const uint32_t bars = smem_u32(s_bar);
  auto bar_full = [&](int s) { return bars + 8 * s; };
  auto bar_empty = [&](int s) { return bars + 8 * (ST + s); };
  auto bar_s = [&](int t) { return bars + 8 * (2 * ST + t); };                    // S_t holds new scores
  auto bar_o = [&](int t) { return bars + 8 * (2 * ST + 2 + t); };                // O_t is complete
  auto bar_p = [&](int t, int h) { return bars + 8 * (2 * ST + 4 + 2 * t + h); };  // piece h of P_t written (O_t rescaled)
  const uint32_t bar_q = bars + 8 * (2 * ST + 8), bar_fix = bars + 8 * (2 * ST + 9);
  const uint32_t bar_end = bars + 8 * (2 * ST + 10);

  if (tid == 0) {
    tma_prefetch_map(&p.qmap);
    tma_prefetch_map(&p.kmap);
    tma_prefetch_map(&p.vmap);
    for (int s = 0; s < ST; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_s(t), 1);
      mbar_init(bar_p(t, 0), 4);
      mbar_init(bar_p(t, 1), 4);
      mbar_init(bar_o(t), 1);
    }
    mbar_init(bar_q, 1);
    mbar_init(bar_fix, 1);
    mbar_init(bar_end, 1);
    mbar_init_fence();
    s_stop = 0;
  }
  if (warp == 10) tmem_alloc<512>(smem_u32(&s_tmem));
  grid_dep_wait();
  grid_dep_launch();
  if (p.q_offsets && tid == 0 && (blockIdx.x | blockIdx.y) == 0 && p.q_offsets[p.B] > p.total_q)
    record_error(kCheckPosition, p.B, p.q_offsets[p.B], p.total_q);  // rows past those of q are skipped
  // later rows first, all heads of a tile together: the longest rows start first
  const int slot_id = (int)((gridDim.x - 1 - blockIdx.x) / p.n_listed), y = (int)(blockIdx.x % p.n_listed);
  TaPlace at;
  const bool some = ta_locate(p, slot_id, &at);
  const int b = at.b, i0 = at.i0, n = at.n, q0 = at.q0, off = at.off, L = at.L;
  const int g = p.heads[y];
  constexpr bool causal = PARTS == 1;  // rows of a shared prefix see all of it
  const bool dense = !causal || p.roles[g] == 1;
  const int PT = p.PT;
  // tokens of this CTA (one minimum of a difference: min(min(2 PT, n - i0), total_q - q0 - i0) came out of
  // nvcc 12.9 without its second term)
  const int row_end = min(q0 + n, p.total_q), np = min(row_end - (q0 + i0), 2 * PT);
  const int tiles = !some ? 0 : np > PT ? 2 : 1;
  // key tiles that some row sees: [0, a1) and [b0, b1)
  const int p_lo = causal ? max(L - n + i0, -1) : L - 1;
  const int p_hi = causal ? max(L - n + i0 + np - 1, -1) : L - 1;
  int a1 = 0, b0 = 0;
  const int b1 = (p_hi + BN) / BN;  // ceil((p_hi + 1) / BN)
  if (!dense) {
    a1 = (min(p.sink, p_hi + 1) + BN - 1) / BN;
    b0 = p.window == 0 ? b1 : max(a1, max(0, p_lo + 1 - p.window) / BN);
  }
  const int n_all = some ? a1 + max(0, b1 - b0) : 0;
  const int j_lo = (int)((int64_t)n_all * blockIdx.y / p.splits);
  const int n_it = (int)((int64_t)n_all * (blockIdx.y + 1) / p.splits) - j_lo;
  const int segment = PARTS > 1 ? kTaSegment : p.segment;
  auto key_tile = [&](int j) { return (j_lo + j < a1 ? j_lo + j : b0 + j_lo + j - a1) * BN; };

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  volatile int* stop = &s_stop;

  if (wg == 2) {
    regs_dec<kTaRegsOther>();
    if (warp == 8 && n_it > 0) {  // ---------------------------------------------- loads
      if (lane == 0) {
        mbar_expect_tx(bar_q, tiles * (D / 64) * 128 * PT * p.G);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(q_s + t * T::kQBytes + h * 16384, &p.qmap, h * 64, g * p.G, q0 + i0 + t * PT, bar_q);
      }
      const int slot = p.slot[g];
      int fixes = 0;
      for (int i = 0; i < 2 * n_it; ++i) {  // K_0, V_0, K_1, V_1, ...
        const int s = i % ST, t0 = key_tile(i >> 1);
        const bool is_v = i & 1;
        if (!warp_wait(bar_empty(s), ((i / ST) & 1) ^ 1, stop)) break;
        // V rows past the length may hold anything, and a zero weight times a NaN is a NaN: the last
        // tile's are cleared before the MMA may see it
        const bool fix = is_v && t0 + BN > L;
        const uint32_t dst = kv_s + s * T::kKvBytes;
        const uint32_t bar = fix ? bar_fix : bar_full(s);
        if (lane == 0) {
          mbar_expect_tx(bar, T::kKvBytes);
          for (int h = 0; h < D / 64; ++h)
            tma_load_3d(dst + h * (BN * 128), is_v ? &p.vmap : &p.kmap, h * 64, slot, off + t0, bar);
        }
        __syncwarp();
        if (fix) {
          const bool ok = warp_wait(bar_fix, fixes & 1, stop);
          ++fixes;
          if (!ok) break;
          const int r0 = L - t0, chunks = (BN - r0) * 8;  // 16-byte pieces of one half
          for (int e = lane; e < chunks * (D / 64); e += 32) {
            const uint32_t at = dst + (e / chunks) * (BN * 128) + r0 * 128 + (e % chunks) * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(at), "r"(0) : "memory");
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_full(s));
        }
      }
    } else if (warp == 9 && n_it > 0) {  // ----------------------------------------- matrix products
      // The whole warp walks through the loop and one elected lane issues, so that descriptors stay in
      // uniform registers (issued from a branch on the lane, 16 products took 1500 to 2400 cycles and
      // bounded the kernel).  All 512 columns are this block's, so TMEM addresses start at column 0.
      const uint32_t idesc_s = mma_idesc(BN, false) | (p.neg ? kMmaNegA : 0u);
      constexpr uint32_t idesc_o = mma_idesc(D, true);
      const uint64_t q_d = smem_desc(q_s, 16), k_d = smem_desc(kv_s, 16), v_d = smem_desc(kv_s, BN * 128);
      auto scores = [&](int t, int s) {  // S_t = Q_t K^T
        const uint64_t a = q_d + (t * T::kQBytes >> 4), c = k_d + (s * T::kKvBytes >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ss(t * 128, a + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4), c + (((ks >> 2) * (BN * 128) + (ks & 3) * 32) >> 4),
                 idesc_s, ks > 0);
        mma_commit(bar_s(t));
      };
      auto run = [&]() {
        if (!warp_wait(bar_q, 0, stop) || !warp_wait(bar_full(0), 0, stop)) return;
        tc_fence_after();
        if (elect_one()) {
          for (int t = 0; t < tiles; ++t) scores(t, 0);
          mma_commit(bar_empty(0));
        }
        __syncwarp();
        int sv = 1, ph = 0;  // stage and phase of V_j; K_{j+1} is in the next one
        int left = segment;  // key tiles of this segment
        for (int j = 0; j < n_it; ++j) {
          const bool more = j + 1 < n_it, first = left == segment, last = !more || left == 1;
          left = left == 1 ? segment : left - 1;
          const int sk = sv + 1 == ST ? 0 : sv + 1, pk = sv + 1 == ST ? ph ^ 1 : ph;
          if (!warp_wait(bar_full(sv), ph, stop)) return;
          if (more && !warp_wait(bar_full(sk), pk, stop)) return;
          const uint64_t c = v_d + (sv * T::kKvBytes >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (t == tiles) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (!warp_wait(bar_p(t, h), j & 1, stop)) return;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int ks = h ? C0 / 16 : 0; ks < (h ? BN : C0) / 16; ++ks)
#pragma unroll
                  for (int part = 0; part < PARTS; ++part)
                    mma_ts(kO + t * D, t * 128 + part * (BN / 2) + ks * 8, c + (ks * 2048 >> 4), idesc_o,
                           !first || ks > 0 || part > 0);
                if (h == 1) {
                  if (last) mma_commit(bar_o(t));
                  if (more) scores(t, sk);
                  if (t + 1 == tiles) {
                    mma_commit(bar_empty(sv));
                    if (more) mma_commit(bar_empty(sk));
                  }
                }
              }
              __syncwarp();
            }
          }
          ph = sk + 1 == ST ? pk ^ 1 : pk;
          sv = sk + 1 == ST ? 0 : sk + 1;
        }
      };
      run();
    }
  } else {  // ---------------------------------------------------------------------- softmax of tile wg
    regs_inc<kTaRegsSoftmax>();
    const int t = wg, r = tid & 127, wr = r & ~31;
    const int tok = t * PT + r / p.G;
    const bool valid = r < PT * p.G && tok < np;
    const bool live = t < tiles && wr < PT * p.G && t * PT + wr / p.G < np;  // some row of the warp exists
    const int pos = causal ? max(L - n + i0 + tok, -1) : L - 1;
    const int w_tok_hi = min(t * PT + min(wr + 31, PT * p.G - 1) / p.G, np - 1);
    const int w_lo = causal ? max(L - n + i0 + t * PT + wr / p.G, -1) : L - 1;
    const int w_hi = causal ? max(L - n + i0 + w_tok_hi, -1) : L - 1;
    const float sc = p.scale_log2;
    const uint64_t sc2 = f2(sc, sc);
    const uint32_t lanes = tmem + ((uint32_t)(wr & 96) << 16);
    const uint32_t s_t = lanes + t * 128, o_t = lanes + kO + t * D;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const bool part = PARTS > 1 || p.splits > 1;
    float fac = 1.f;  // what the row's partial in memory is still to be scaled by
    // O and l of the row; add: to the partial written before; last: of the row's segments
    auto take_out = [&](bool have, bool add, bool last) {
      const bool to_memory = PARTS > 1 || part || !last;
      const float inv = part ? 1.f : (l > 0.f ? 1.f / l : 0.f);
      const int64_t pt = ((int64_t)blockIdx.y * p.slots * p.n_listed + (int64_t)slot_id * p.n_listed + y) * 2 + t;
      float4* acc_out = p.part_acc + pt * (D / 4) * 128 + r;
      if (part) p.part_ml[pt * 128 + r] = make_float2(valid && l > 0.f ? m * sc : -INFINITY, l);
      // A finished row goes through the warp's rows of Q in shared memory (no product reads Q any more),
      // 16-byte pieces XOR-swizzled, so that whole rows leave in full lines.
      const uint32_t stage = q_s + t * T::kQBytes + wr * (D * 2);
      auto piece = [&](int rr, int ch) { return stage + rr * (D * 2) + ((ch ^ (rr & 7)) << 4); };
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (have) {
          tmem_ld32(o, o_t + c);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        // A partial is written and read by the same thread.  (Two forms of the same sums: each instance spills
        // half a kilobyte a thread with the other's.)
        if (PARTS > 1) {
          float4 old[8];
          if (add)
#pragma unroll
            for (int e = 0; e < 8; ++e) old[e] = __ldcg(acc_out + (c / 4 + e) * 128);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 v = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                   __uint_as_float(o[4 * e + 3]));
            if (add) {
              v.x = fmaf(old[e].x, fac, v.x);
              v.y = fmaf(old[e].y, fac, v.y);
              v.z = fmaf(old[e].z, fac, v.z);
              v.w = fmaf(old[e].w, fac, v.w);
            }
            __stcg(acc_out + (c / 4 + e) * 128, v);
          }
          continue;
        }
        if (add) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 v = __ldcg(acc_out + (c / 4 + e) * 128);
            o[4 * e] = __float_as_uint(fmaf(v.x, fac, __uint_as_float(o[4 * e])));
            o[4 * e + 1] = __float_as_uint(fmaf(v.y, fac, __uint_as_float(o[4 * e + 1])));
            o[4 * e + 2] = __float_as_uint(fmaf(v.z, fac, __uint_as_float(o[4 * e + 2])));
            o[4 * e + 3] = __float_as_uint(fmaf(v.w, fac, __uint_as_float(o[4 * e + 3])));
          }
        }
        if (to_memory) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            __stcg(acc_out + (c / 4 + e) * 128, make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                           __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3])));
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              v[u] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * u]) * inv, __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(piece(lane, c / 8 + e)), "r"(v[0]), "r"(v[1]),
                         "r"(v[2]), "r"(v[3])
                         : "memory");
          }
        }
      }
      __syncwarp();
      if (!to_memory) {
        constexpr int LPR = D / 8;  // lanes per row
#pragma unroll 4
        for (int k = 0; k < LPR; ++k) {
          const int rr = k * (32 / LPR) + lane / LPR, ch = lane % LPR, rw = wr + rr;
          const int tk = t * PT + rw / p.G;
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(piece(rr, ch)));
          if (rw < PT * p.G && tk < np)
            *reinterpret_cast<uint4*>(p.out + ((int64_t)(q0 + i0 + tk) * p.Hq + g * p.G + rw % p.G) * D + ch * 8) = v;
        }
      }
      fac = 1.f;
    };
    auto weigh = [&](int j, bool first) {  // the scores of key tile j become weights; first: of a segment
      tc_fence_after();
      const int t0 = key_tile(j);
      // (a warp without rows leaves P as it is: rows of a product do not mix)
      const bool none = t0 > w_hi || (!dense && t0 >= p.sink && t0 + BN - 1 <= w_lo - p.window);
      if (live && none) {
        uint32_t z[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) z[e] = 0;
#pragma unroll
        for (int c = 0; c < PARTS * BN / 2; c += 32) tmem_st32(s_t + c, z);
        tmem_wait_st();
      } else if (live) {
        uint32_t s[BN];
#pragma unroll
        for (int c = 0; c < BN; c += 32) tmem_ld32(s + c, s_t + c);
        tmem_wait_ld();
        const bool all = t0 + BN - 1 <= w_lo && (dense || t0 <= p.sink - BN || t0 > w_hi - p.window);
        if (!all) {
          // hidden: behind hi, and the `gap` tokens from sk on.  (Selects: as conditions joined by && and || these
          // became a branch per token in some builds, 25 us more per CTA.)
          const int hi = pos - t0, lo = dense ? -1 : pos - p.window - t0, sk = dense ? 0 : p.sink - t0;
          const uint32_t gap = lo >= sk ? (uint32_t)lo - (uint32_t)sk + 1u : 0u;
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = ((c > hi) | ((uint32_t)c - (uint32_t)sk < gap)) ? 0xff800000u : s[c];
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < BN; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx[e] = max3(mx[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool grow = (top - m) * sc > kTaGrowth;  // false while nothing has been seen
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? top : m;
          const float al = grow ? ex2((m - mn) * sc) : 1.f;
          l *= al;
          fac *= al;
          m = mn;
          if (!first) {
            const uint64_t al2 = f2(al, al);
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o, o_t + c);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float x, y;
                f2_split(f2_mul(f2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), al2), x, y);
                o[e] = __float_as_uint(x);
                o[e + 1] = __float_as_uint(y);
              }
              tmem_st32(o_t + c, o);
            }
          }
        }
        const float ms = m == -INFINITY ? 0.f : -m * sc;
        const uint64_t ms2 = f2(ms, ms);
        uint64_t sum = 0;
        auto weights = [&](auto& w, int c0, int n) {  // of tokens c0 .. c0 + 2 n - 1
#pragma unroll
          for (int e = 0; e < n; ++e) {
            const int c = c0 + 2 * e;
            const uint64_t v2 = f2_fma(f2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sc2, ms2);
            float x, y;
            if (PARTS == 1 && e % kTaPolyOf < kTaPoly) {
              ex2_poly(v2, x, y);
            } else {
              f2_split(v2, x, y);
              x = ex2(x);
              y = ex2(y);
            }
            sum = f2_add(sum, f2(x, y));
#pragma unroll
            for (int part = 0; part < PARTS; ++part) {
              const uint32_t v = pack_bf16x2(x, y);
              w[part][e] = v;
              x -= bf16lo(v);
              y -= bf16hi(v);
            }
          }
        };
        auto publish = [&](int h) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_p(t, h));
        };
        uint32_t w0[PARTS][C0 / 2];
        weights(w0, 0, C0 / 2);
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int c = 0; c < C0 / 2; c += 16) tmem_st16(s_t + part * (BN / 2) + c, w0[part] + c);
        publish(0);
        uint32_t w1[PARTS][(BN - C0) / 2];
        weights(w1, C0, (BN - C0) / 2);
#pragma unroll
        for (int part = 0; part < PARTS; ++part)
#pragma unroll
          for (int c = 0; c < (BN - C0) / 2; c += 16) tmem_st16(s_t + part * (BN / 2) + C0 / 2 + c, w1[part] + c);
        publish(1);
        float x, y;
        f2_split(sum, x, y);
        l += x + y;
      }
      if (!live || none) {
        tc_fence_before();
        __syncwarp();
        if (lane < 2) mbar_arrive(bar_p(t, lane));
      }
    };
    if (t < tiles) {
      if (PARTS > 1) {
        for (int j = 0; j < n_it; ++j) {
          if (!(ok = warp_wait(bar_s(t), j & 1, stop))) break;
          weigh(j, j % kTaSegment == 0);
          if (j + 1 == n_it || (j + 1) % kTaSegment == 0) {
            if (!(ok = warp_wait(bar_o(t), (j / kTaSegment) & 1, stop))) break;
            tc_fence_after();
            if (live) take_out(true, j >= kTaSegment, false);
          }
        }
      } else {
        int j = 0;
        for (int sg = 0; j < n_it && ok; ++sg) {
          const int j_seg = j, j_end = n_it - j > segment ? j + segment : n_it;
          for (; j < j_end && (ok = warp_wait(bar_s(t), j & 1, stop)); ++j) weigh(j, j == j_seg);
          ok = ok && warp_wait(bar_o(t), sg & 1, stop);
          tc_fence_after();
          if (ok && live) take_out(true, sg > 0, j == n_it);
        }
      }
      if (n_it == 0 && live) take_out(false, false, true);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_stop && warp == 9 && elect_one()) {
    // a wait ran out: what is in flight must land before shared memory and TMEM are given back
    record_error(kCheckStall, b, g, (int)blockIdx.y);
    mma_commit(bar_end);
    for (int i = 0; i < kWaitLimit && !mbar_try(bar_end, 0); ++i) {
    }
    for (int i = 0; i < (1 << 16); ++i) __nanosleep(20);  // TMA copies issued (about a millisecond)
  }
  __syncthreads();
  if (warp == 10) tmem_dealloc<512>(tmem);
}

// ---------------------------------------------------------------------- joining partial rows
struct MergeParams {
  const float2* part_ml;     // tile partials, `splits` of every tile of rows
  const float4* part_acc;
  const int32_t* q_offsets;  // rows of every group ([B + 1]) or null: one group of all rows
  void* out;                 // bf16 or fp32 [total_q][Hq][D]
  int32_t B, Hq, G, PT, total_q, splits, n_listed, slots;
  // the rows' own tokens (row b is sequence b) and, with own.NP, its prefix, or no own.pre; without
  // own.packed what one CTA finished is in out, not divided by its sum
  DenseRows own;
  uint8_t heads[kMaxHeads];
};

constexpr int kTmThreads = 256, kTmFlight = 8;

// grid (32 (row, q head of the group) pairs, listed heads): a pair per lane, so that the partials of a
// tile are read as they were written; warps share the D / 4 pieces of the rows.  Partials are added in
// a fixed order.
template <int D, bool BF16>
__global__ void __launch_bounds__(kTmThreads) tile_merge_kernel(const MergeParams p) {
  grid_dep_wait();
  constexpr int NC = D / 4 / (kTmThreads / 32);  // pieces of a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = (int64_t)blockIdx.x * 32 + lane;
  const int row = (int)(item / p.G), hq = (int)(item % p.G), y = blockIdx.y, h = p.heads[y] * p.G + hq;
  if (row >= p.total_q) return;
  bool tiles = true;
  int i = 0, first = 0;  // the row's group and its first row
  if (p.q_offsets) {
    tiles = row >= p.q_offsets[0] && row < p.q_offsets[p.B];  // rows that no group holds have no tile partials
    if (!tiles && !p.own.pre) return;
    if (!tiles && y == 0 && hq == 0 && warp == 0) record_error(kCheckPosition, row, -1, p.B);
    int hi = p.B - 1;
    while (i < hi) {
      const int mid = (i + hi) >> 1;
      if (p.q_offsets[mid + 1] > row) hi = mid; else i = mid + 1;
    }
    first = max(0, p.q_offsets[i]);
    tiles = tiles && row >= first;
  }
  const int P2 = 2 * p.PT, rel = row - first;
  const int64_t slot = p.q_offsets ? ((int64_t)first + (int64_t)i * (P2 - 1)) / P2 + rel / P2 : rel / P2;
  const int64_t n_tiles = (int64_t)p.slots * p.n_listed * 2, u = (slot * p.n_listed + y) * 2 + (rel % P2) / p.PT;
  const int rr = (rel % p.PT) * p.G + hq;
  const int ns = tiles && slot < p.slots ? p.splits : 0;
  const int nv = p.own.NP + p.total_q;
  int no = 0, c0 = 0, c1 = 0;
  if (p.own.pre && dense_row(p.own, p.n_listed, nv, y, p.own.NP + row, &c0, &c1)) no = c1 - c0 + 1;
  int np = 0, d0 = 0, d1 = 0;  // partials of the row's prefix in the dense pass
  if (p.own.NP && tiles && (rel + 1) * p.G <= p.own.nqp && dense_row(p.own, p.n_listed, nv, y, i, &d0, &d1)) np = d1 - d0 + 1;
  const int64_t tr = (int64_t)row * p.Hq + h;
  // part s: of the tiles, of the row's own tokens, of its prefix
  auto dense_at = [&](int s, bool* whole) {
    const bool own = s < ns + no;
    const int a = own ? c0 : d0, e = own ? c1 : d1, v = own ? p.own.NP + row : i;
    *whole = a == e;
    return (a == e ? (int64_t)y * nv + v : dense_part(a, s - ns - (own ? 0 : no))) * p.own.nqp +
           (own ? hq : rel * p.G + hq);
  };
  auto ml_of = [&](int s) {
    if (s < ns) return p.part_ml[(s * n_tiles + u) * 128 + rr];
    bool whole;
    const int64_t r = dense_at(s, &whole);
    return *reinterpret_cast<const float2*>((whole ? p.own.row_ml : p.own.part_ml) + r * 2);
  };
  auto acc_of = [&](int s, int64_t* step) {  // first piece and the distance of the next, in float4
    if (s < ns) {
      *step = 128;
      return p.part_acc + (s * n_tiles + u) * (D / 4) * 128 + rr;
    }
    bool whole;
    const int64_t r = dense_at(s, &whole);
    *step = 1;
    const float* a = !whole ? p.own.part_acc + r * D : p.own.packed ? p.own.row_acc + r * D : p.own.row_acc + tr * D;
    return reinterpret_cast<const float4*>(a);
  };
  const int nt = ns + no + np;
  float4 acc[NC];
  float M = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < nt; s0 += kTmFlight) {
    float4 v[kTmFlight][NC];
    float2 ml[kTmFlight];
    float top = M;
#pragma unroll
    for (int k = 0; k < kTmFlight; ++k) {
      ml[k] = make_float2(-INFINITY, 0.f);
      if (s0 + k < nt) {
        ml[k] = ml_of(s0 + k);
        int64_t step;
        const float4* a = acc_of(s0 + k, &step);
#pragma unroll
        for (int c = 0; c < NC; ++c) v[k][c] = a[(warp * NC + c) * step];
      }
    }
#pragma unroll
    for (int k = 0; k < kTmFlight; ++k) top = fmaxf(top, ml[k].x);
    const float al = M == -INFINITY ? 0.f : ex2(M - top);
    M = top;
    l *= al;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      acc[c].x *= al;
      acc[c].y *= al;
      acc[c].z *= al;
      acc[c].w *= al;
    }
#pragma unroll
    for (int k = 0; k < kTmFlight; ++k) {
      if (ml[k].x == -INFINITY) continue;  // nothing was seen, and its acc may never have been written
      const float w = ex2(ml[k].x - M);
      l = fmaf(w, ml[k].y, l);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        acc[c].x = fmaf(w, v[k][c].x, acc[c].x);
        acc[c].y = fmaf(w, v[k][c].y, acc[c].y);
        acc[c].z = fmaf(w, v[k][c].z, acc[c].z);
        acc[c].w = fmaf(w, v[k][c].w, acc[c].w);
      }
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int d = (warp * NC + c) * 4;
    if (BF16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + tr * D + d) =
          make_uint2(pack_bf16x2(acc[c].x * inv, acc[c].y * inv), pack_bf16x2(acc[c].z * inv, acc[c].w * inv));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + tr * D + d) =
          make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv);
  }
}

}  // namespace aoh
