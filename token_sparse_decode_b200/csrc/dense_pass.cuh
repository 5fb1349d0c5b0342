// One pass over a whole ragged cache for few query rows per KV head: decode attention over
// [0, L_b) of every (sequence, KV head), persistent and TMA-fed.
//
// For the NQ query rows h of KV head g:  x_ht = scale q_h . k_t,  m = max_t x, l = sum 2^(x - m),
// acc = sum 2^(x - m) v_t, and, when asked, every x (the accumulated-weight decode turns them into
// weights once m and l are known).
//
// Work split.  The cache is cut into tiles of 64 tokens; the tiles of all rows (head-major, then
// sequence) form one line, and CTA c of C takes the c-th of C equal pieces of it.  A ragged batch
// thereby keeps every SM busy to the end with one CTA per SM (a grid of fixed chunks per row left
// 15 % of the time to its last wave and as much to refilling each CTA's ring).  A row inside one
// piece is finished by its CTA; a row that pieces cut leaves one partial per CTA, joined by the
// kernel that follows.  At most two rows of a CTA are cut: part 2 c (a row that began before the
// piece) and 2 c + 1 (a row that begins in it).
//
// One warp copies K and V tiles by TMA (128-byte swizzle) into a ring; eight warps take 16-token
// sub-tiles, tokens on the M side of mma.m16n8k16 (the query rows are the N side: 7 rows fill 7 of
// 8 columns).  Weights enter the product with V as three bf16 terms, so that fp32 outputs keep
// fp32 weights, and every sub-tile's product starts from zero and is added by the FMA units: the
// tensor cores' own accumulation rounds towards zero, 3e-6 along 900 tokens.
//
// Bound by the K / V bytes with up to 16 query rows.  Measured (B200): 131072 tokens x 8 heads, d 128 in 90 us,
// 5.96 TB/s (91 % of the measured copy rate); 48 sequences of 1 to 8000 x 4 heads in 71 us, 5.5 TB/s (a grid of
// fixed chunks fed by cp.async took 120 and 91 us).  More query rows on one KV head, 8 x 131072 tokens, d 128: 8
// rows 99 us, 16 rows 109 us (4.9 TB/s); 17 to 32 rows, four times the products per byte, 191 us (2.8 TB/s).
#pragma once

#include <cuda.h>

#include "tcgen05.cuh"

namespace aoh {

constexpr int kDpTile = 64;
constexpr int kDpWarps = 8;
constexpr int kDpThreads = 32 * (kDpWarps + 1);
constexpr int kDpSeqs = 1024;  // sequences whose tile counts a CTA sums up itself (more: dense_plan_kernel)

template <int D>
struct DpTile {
  static constexpr int kHalf = kDpTile * 128;              // 64 columns of a tile
  static constexpr int kTile = kDpTile * D * 2;
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRed = kDpWarps * 8 * (2 + D) * 4;  // the warps' (m, l) and acc
  static constexpr int ST = (218 * 1024 - kRed) / kStage > 10 ? 10 : (218 * 1024 - kRed) / kStage;
  static constexpr int kSmem = 1024 + ST * kStage + kRed;
};

struct alignas(64) DenseParams {
  CUtensorMap kmap[2], vmap[2];  // the sequences' cache, the prefixes'
  const uint16_t* q;         // [B][Hq][D]
  const int32_t* offsets;
  const int32_t* lengths;    // or null
  int32_t* pre;              // [NP + B + 1] tiles of one head before entry v
  float* out;                // fp32 [B][Hq][D]: rows of one CTA, unless row_acc
  float* row_acc;            // [n_listed][NP + B][NQP][D] or null
  float* row_ml;             // [n_listed][NP + B][NQP][2]: (m, l) of the same
  float* part_ml;            // [2 C][NQP][2]
  float* part_acc;           // [2 C][NQP][D]
  float* logits;             // [Hkv][T][logit_pitch] or null
  int64_t T;
  int32_t logit_pitch;       // even, >= NQ
  int32_t B, Hq, G, n_listed;
  // Entries 0 .. NP - 1 of the line are shared prefixes, whose query rows are those of the sequences
  // [seq_start[v], seq_start[v + 1]) (null: all), G each; the sequences follow.
  int32_t NP;
  const int32_t* pre_offsets;
  const int32_t* pre_lengths;
  const int32_t* seq_start;
  int32_t planned;           // 1: pre is there already (only with NP = 0)
  int32_t normalise;         // 1: out = acc / l, 0: acc
  int32_t late_wait;         // 1: the launch before is of the same call (it waited for what came before the
                             //    call) and writes nothing that is read here: run beside it, and end after it
  float scale_log2;
  uint8_t heads[kMaxHeads];
  uint8_t slot[kMaxHeads];
  uint8_t pre_slot[kMaxHeads];
};

// Entry v of the line: its length, first token, first sequence and query rows
struct DenseEntry {
  int L, off, seq, nq;
};
__device__ __forceinline__ DenseEntry dense_entry(const DenseParams& p, int v) {
  DenseEntry e;
  if (v >= p.NP) {
    e.seq = v - p.NP;
    e.nq = p.G;
    e.L = seq_length(p.offsets, p.lengths, e.seq, false, &e.off);
  } else {
    e.seq = p.seq_start ? max(0, min(p.seq_start[v], p.B)) : 0;
    const int end = p.seq_start ? max(e.seq, min(p.seq_start[v + 1], p.B)) : p.B;
    e.nq = (end - e.seq) * p.G;
    e.L = seq_length(p.pre_offsets, p.pre_lengths, v, false, &e.off);
    if (e.nq == 0) e.L = 0;  // nobody continues it
  }
  return e;
}

// Tiles before every entry: an exclusive sum by one block
template <typename Len>
__device__ __forceinline__ void dense_plan(Len len, int n, int32_t* pre, int tid, int threads, int* scratch) {
  int base = 0;
  for (int v0 = 0; v0 < n; v0 += threads) {
    const int c = v0 + tid < n ? (len(v0 + tid) + kDpTile - 1) / kDpTile : 0;
    int total;
    const int at = block_exclusive_scan(c, scratch, &total);
    if (v0 + tid < n) pre[v0 + tid] = base + at;
    base += total;
  }
  if (tid == 0) pre[n] = base;
}

struct PlanParams {
  const int32_t* offsets;
  const int32_t* lengths;
  int32_t* pre;
  int32_t B;
};
__global__ void __launch_bounds__(1024) dense_plan_kernel(const PlanParams p) {
  grid_dep_wait();
  __shared__ int scratch[33];
  dense_plan([&](int v) {
    int off;
    return seq_length(p.offsets, p.lengths, v, false, &off);
  }, p.B, p.pre, threadIdx.x, 1024, scratch);
}

// The piece of CTA c: [dense_piece(n, c, C), dense_piece(n, c + 1, C)) of n tiles
__device__ __forceinline__ int64_t dense_piece(int64_t n, int c, int C) { return n * c / C; }
// The CTA whose piece holds tile x
__device__ __forceinline__ int dense_owner(int64_t n, int64_t x, int C) { return (int)(((x + 1) * C - 1) / n); }

// First sequence b with pre[b + 1] > x
__device__ __forceinline__ int dense_seq(const int32_t* pre, int B, int x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] > x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

template <int D, int NT>
__global__ void __launch_bounds__(kDpThreads, 1) dense_pass_kernel(const __grid_constant__ DenseParams p) {
  using T = DpTile<D>;
  constexpr int ST = T::ST, KS = D / 16, NQP = NT * 8, WT = kDpWarps / NT;
  extern __shared__ uint8_t dp_smem[];
  __shared__ __align__(8) uint64_t s_bar[2 * ST];
  __shared__ int32_t s_pre[kDpSeqs + 1];
  __shared__ int s_scan[33];
  __shared__ int s_stop;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t ring = (smem_u32(dp_smem) + 1023u) & ~1023u;
  float* red_ml = reinterpret_cast<float*>(dp_smem + (ring - smem_u32(dp_smem)) + ST * T::kStage);  // [warps][8][2]
  float* red_acc = red_ml + kDpWarps * 8 * 2;                                                       // [warps][8][D]
  const uint32_t bars = smem_u32(s_bar);
  auto bar_full = [&](int s) { return bars + 8 * s; };
  auto bar_empty = [&](int s) { return bars + 8 * (ST + s); };
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), kDpWarps);
    }
    mbar_init_fence();
    s_stop = 0;
  }
  if (!p.late_wait) grid_dep_wait();
  grid_dep_launch();
  const int nv = p.NP + p.B;
  const int32_t* pre = p.pre;
  if (!p.planned) {
    dense_plan([&](int v) { return dense_entry(p, v).L; }, nv, s_pre, tid, kDpThreads, s_scan);
    __syncthreads();
    pre = s_pre;
    if (blockIdx.x == 0)
      for (int v = tid; v <= nv; v += kDpThreads) p.pre[v] = s_pre[v];
  }
  __syncthreads();
  const int per_head = pre[nv], c = blockIdx.x;
  const int64_t n_all = (int64_t)per_head * p.n_listed;
  const int C = (int)min((int64_t)gridDim.x, n_all);  // no piece is empty
  if (c >= C) {
    if (p.late_wait && c == 0) grid_dep_wait();
    return;
  }
  const int64_t w0 = dense_piece(n_all, c, C), w1 = dense_piece(n_all, c + 1, C);
  volatile int* stop = &s_stop;

  if (warp == kDpWarps) {  // ------------------------------------------------------------ copies
    int i = 0;
    bool ok = true;
    for (int64_t w = w0; w < w1 && ok;) {
      const int y = (int)(w / per_head), x = (int)(w % per_head), v = dense_seq(pre, nv, x);
      const int n = (int)min((int64_t)(pre[v + 1] - x), w1 - w);
      const bool own = v >= p.NP;
      const int tok = (own ? p.offsets[v - p.NP] : p.pre_offsets[v]) + (x - pre[v]) * kDpTile;
      const int slot = own ? p.slot[p.heads[y]] : p.pre_slot[p.heads[y]];
      const CUtensorMap *km = &p.kmap[own ? 0 : 1], *vm = &p.vmap[own ? 0 : 1];
      for (int t = 0; t < n; ++t, ++i) {
        const int s = i % ST;
        if (!(ok = warp_wait(bar_empty(s), ((i / ST) & 1) ^ 1, stop))) break;
        if (elect_one()) {
          const uint32_t dst = ring + s * T::kStage;
          mbar_expect_tx(bar_full(s), T::kStage);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            tma_load_3d(dst + h * T::kHalf, km, h * 64, slot, tok + t * kDpTile, bar_full(s));
            tma_load_3d(dst + T::kTile + h * T::kHalf, vm, h * 64, slot, tok + t * kDpTile, bar_full(s));
          }
        }
        __syncwarp();
      }
      w += n;
    }
  } else {  // --------------------------------------------------------------------------- attention
    const int nt = warp % NT, tg = warp / NT;
    auto tile_off = [](int r, int dd) -> uint32_t {
      return (uint32_t)((dd >> 6) * T::kHalf + r * 128 + ((((dd & 63) >> 3) ^ (r & 7)) << 4));
    };
    int i = 0;
    bool ok = true;
    for (int64_t w = w0; w < w1;) {
      const int y = (int)(w / per_head), x = (int)(w % per_head), v = dense_seq(pre, nv, x), g = p.heads[y];
      const int t0 = x - pre[v], n = (int)min((int64_t)(pre[v + 1] - x), w1 - w);
      const DenseEntry en = dense_entry(p, v);
      const int L = en.L, off = en.off, nq = min(en.nq, NQP);
      uint32_t bq[KS][2];  // Q as B fragments: column lane / 4 of the n-tile
      {
        const int qr = nt * 8 + (lane >> 2);
        const uint16_t* qp = p.q + ((int64_t)(en.seq + qr / p.G) * p.Hq + g * p.G + qr % p.G) * D + 2 * (lane & 3);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          bq[ks][0] = qr < nq ? *reinterpret_cast<const uint32_t*>(qp + ks * 16) : 0u;
          bq[ks][1] = qr < nq ? *reinterpret_cast<const uint32_t*>(qp + ks * 16 + 8) : 0u;
        }
      }
      float acc[KS][4];
#pragma unroll
      for (int e = 0; e < KS; ++e) acc[e][0] = acc[e][1] = acc[e][2] = acc[e][3] = 0.f;
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // query rows 2 (lane % 4) and + 1
      for (int t = 0; t < n; ++t, ++i) {
        // Every warp follows every stage, also the ones it does not read (with 8 token groups every other
        // one): a wait by parity must not skip a round of a stage.
        const bool mine = NT > 1 || (i & 1) == (tg >> 2);
        const int s = i % ST;
        ok = ok && warp_wait(bar_full(s), (i / ST) & 1, stop);
        const uint32_t kt = ring + s * T::kStage, vt = kt + T::kTile;
#pragma unroll
        for (int uu = 0; uu < (WT >= 4 ? 1 : 4 / WT); ++uu) {
          const int r0 = 16 * (WT >= 4 ? (tg & 3) : tg + WT * uu);
          const int pos = (t0 + t) * kDpTile + r0, nv = L - pos;  // first position, valid ones
          if (nv <= 0 || !ok || !mine) continue;
          if (nv < 16) {  // V rows past the length may hold anything, and a zero weight times a NaN is a NaN
            for (int e = lane; e < (16 - nv) * (D / 8); e += 32) {
              const uint32_t at = vt + tile_off(r0 + nv + e / (D / 8), (e % (D / 8)) * 8);
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(at), "r"(0) : "memory");
            }
            fence_async_smem();  // the ring's next copy follows these stores
            __syncwarp();
          }
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
          {
            const int r = r0 + (lane & 7) + ((lane >> 3) & 1) * 8, dsel = (lane >> 4) * 8;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
              uint32_t a[4];
              ldsm_x4(a, kt + tile_off(r, ks * 16 + dsel));
              mma_16816(s4, a, bq[ks][0], bq[ks][1]);
            }
          }
          const int ta = lane >> 2, tb = ta + 8;
          const float x0 = ta < nv ? s4[0] * p.scale_log2 : -INFINITY;
          const float x1 = ta < nv ? s4[1] * p.scale_log2 : -INFINITY;
          const float x2 = tb < nv ? s4[2] * p.scale_log2 : -INFINITY;
          const float x3 = tb < nv ? s4[3] * p.scale_log2 : -INFINITY;
          const int qc = nt * 8 + 2 * (lane & 3);
          if (p.logits && qc < p.logit_pitch) {
            float* lg = p.logits + ((int64_t)g * p.T + off + pos) * p.logit_pitch + qc;
            if (ta < nv) *reinterpret_cast<float2*>(lg + (int64_t)ta * p.logit_pitch) = make_float2(x0, x1);
            if (tb < nv) *reinterpret_cast<float2*>(lg + (int64_t)tb * p.logit_pitch) = make_float2(x2, x3);
          }
          float mx0 = fmaxf(x0, x2), mx1 = fmaxf(x1, x3);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
          }
          const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);  // finite: nv >= 1
          if (__any_sync(0xffffffffu, mn0 != m0 || mn1 != m1)) {
            const float al0 = ex2(m0 - mn0), al1 = ex2(m1 - mn1);
            l0 *= al0;
            l1 *= al1;
#pragma unroll
            for (int e = 0; e < KS; ++e) {
              acc[e][0] *= al0;
              acc[e][1] *= al1;
              acc[e][2] *= al0;
              acc[e][3] *= al1;
            }
            m0 = mn0;
            m1 = mn1;
          }
          float p0 = ex2(x0 - m0), p1 = ex2(x1 - m1), p2 = ex2(x2 - m0), p3 = ex2(x3 - m1);
          l0 += p0 + p2;
          l1 += p1 + p3;
          uint32_t pa[3], pb[3];
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t h01 = pack_bf16x2(p0, p1), h23 = pack_bf16x2(p2, p3);
            p0 -= bf16lo(h01);
            p1 -= bf16hi(h01);
            p2 -= bf16lo(h23);
            p3 -= bf16hi(h23);
            pa[part] = movmatrix_trans(h01);
            pb[part] = movmatrix_trans(h23);
          }
          {
            const int r = r0 + (lane & 7) + (lane >> 4) * 8, dsel = ((lane >> 3) & 1) * 8;
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              uint32_t a[4];
              ldsm_x4_trans(a, vt + tile_off(r, mt * 16 + dsel));
              float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int part = 2; part >= 0; --part) mma_16816(o, a, pa[part], pb[part]);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[mt][e] += o[e];
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty(s));
      }
      // ---- the row's piece is done: the warps of an n-tile are added in a fixed order
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      {
        const int c0 = 2 * (lane & 3);
        if (lane < 4) {
          red_ml[(warp * 8 + c0) * 2 + 0] = m0;
          red_ml[(warp * 8 + c0) * 2 + 1] = l0;
          red_ml[(warp * 8 + c0 + 1) * 2 + 0] = m1;
          red_ml[(warp * 8 + c0 + 1) * 2 + 1] = l1;
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int d0 = mt * 16 + (lane >> 2);
          red_acc[(warp * 8 + c0) * D + d0] = acc[mt][0];
          red_acc[(warp * 8 + c0 + 1) * D + d0] = acc[mt][1];
          red_acc[(warp * 8 + c0) * D + d0 + 8] = acc[mt][2];
          red_acc[(warp * 8 + c0 + 1) * D + d0 + 8] = acc[mt][3];
        }
      }
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
      const bool before = t0 > 0, after = x + n < pre[v + 1], cut = before || after;
      const int64_t part = 2 * c + (before ? 0 : 1);
      float* ml = cut ? p.part_ml + part * NQP * 2 : p.row_ml + ((int64_t)y * nv + v) * NQP * 2;
      for (int e = tid; e < nq * (D / 4); e += 32 * kDpWarps) {
        const int qr = e / (D / 4), dd = (e % (D / 4)) * 4, ntq = qr >> 3, cq = qr & 7;
        float M = -INFINITY, Ls = 0.f;
#pragma unroll
        for (int t = 0; t < WT; ++t) M = fmaxf(M, red_ml[((ntq + NT * t) * 8 + cq) * 2]);
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int t = 0; t < WT; ++t) {
          const int ws = (ntq + NT * t) * 8 + cq;
          const float f = red_ml[ws * 2] == -INFINITY ? 0.f : ex2(red_ml[ws * 2] - M);
          const float4 a4 = *reinterpret_cast<const float4*>(red_acc + ws * D + dd);
          Ls += f * red_ml[ws * 2 + 1];
          A.x += f * a4.x;
          A.y += f * a4.y;
          A.z += f * a4.z;
          A.w += f * a4.w;
        }
        if (dd == 0) *reinterpret_cast<float2*>(ml + qr * 2) = make_float2(M, Ls);
        if (cut) {
          *reinterpret_cast<float4*>(p.part_acc + (part * NQP + qr) * D + dd) = A;
        } else {
          const float inv = p.normalise ? 1.f / Ls : 1.f;
          float* o = p.row_acc ? p.row_acc + (((int64_t)y * nv + v) * NQP + qr) * D
                               : p.out + ((int64_t)en.seq * p.Hq + g * p.G + qr) * D;
          *reinterpret_cast<float4*>(o + dd) = make_float4(A.x * inv, A.y * inv, A.z * inv, A.w * inv);
        }
      }
      asm volatile("bar.sync 1, 256;\n" ::: "memory");
      w += n;
    }
  }
  __syncthreads();
  if (s_stop && tid == 0) {
    // a wait ran out: copies in flight must land before shared memory is given back (about a millisecond)
    record_error(kCheckStall, c, -1, -1);
    for (int e = 0; e < (1 << 16); ++e) __nanosleep(20);
  }
  __syncthreads();
  // what follows this kernel relies on the one before it, too; one block that waits for it will do
  if (p.late_wait && blockIdx.x == 0) grid_dep_wait();
}

// ---------------------------------------------------------------------- where a row's results are
struct DenseRows {
  const int32_t* pre;
  const float* row_ml;
  const float* row_acc;      // packed: [n_listed][NP + B][NQP][D], else out: [B][Hq][D]
  const float* part_ml;
  const float* part_acc;
  int32_t C, nqp;            // CTAs launched
  int32_t packed, NP;
};
// The CTAs [c0, c1] that hold pieces of head y's entry v (of nv); false: it is empty
__device__ __forceinline__ bool dense_row(const DenseRows& d, int n_listed, int nv, int y, int v, int* c0, int* c1) {
  const int per_head = d.pre[nv], a = d.pre[v], e = d.pre[v + 1];
  if (a == e) return false;
  const int64_t n = (int64_t)per_head * n_listed, f = (int64_t)y * per_head;
  const int C = (int)min((int64_t)d.C, n);
  *c0 = dense_owner(n, f + a, C);
  *c1 = dense_owner(n, f + e - 1, C);
  return true;
}
// Part of CTA c0 + s of a row cut over CTAs c0 ..
__device__ __forceinline__ int dense_part(int c0, int s) { return 2 * (c0 + s) + (s == 0 ? 1 : 0); }

}  // namespace aoh
