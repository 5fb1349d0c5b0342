// Eviction from a cache by accumulated attention weight.
//
// A row (sequence b, KV head g) of L positions keeps n = min(budget, L) of them: the first
// `sink`, the last `recent`, and of the others those with the largest accumulated weight
// mass[g][offsets[b] + p] (equal weights: the lower position).  The kept rows move, in the
// order of their positions, to the front of the row's region in another cache:
//     K'[j] = K[idx[j]],  V'[j] = V[idx[j]],  mass'[j] = mass[idx[j]],   j < n,
// and lengths'[b] = n.  Each KV head keeps positions of its own, all heads equally many.
//
//   select_cluster_kernel<true>  (rows up to 131072 positions) the exact top-n select on the weights,
//                      keys in registers: protected positions before every weight, a NaN as the lightest;
//   evict_key_kernel and the library's select (longer rows): the same with the keys in memory;
//   evict_copy_kernel  moves the rows.
// Measured: 32 sequences of 700 to 4500 x 8 heads to 2048 rows in 94 us, the copy 75 us of it (6.5 TB/s
// read and written, the measured copy rate); two of 65536 to 8192 in 44 us in a long run, 38 in a short one: copy
// 24, the rest the select, which takes four cluster barriers.  Rows above 131072 positions take six launches: one of
// 200000 x 8 heads to 8192 in 48 us, of 300000 in 157, of a million in 464.
// The copy is bound by memory: 8 d + 8 bytes per kept row read and written once; the selects by
// latency, beside 4 bytes per (head, position) for the weights.
#pragma once

#include "select_cluster.cuh"

namespace aoh {

struct EvictParams {
  const float* mass;          // [Hkv][T]
  float* scores;              // [Hkv][T]
  uint32_t* counters;         // [n_counters] the select's counters in the workspace
  int64_t n_counters;
  const int32_t* offsets;     // [B + 1]
  const int32_t* lengths;     // [B] or null
  const int32_t* idx;         // [B][Hkv][budget]
  const int32_t* count;       // [B][Hkv]
  // source rows
  const uint16_t* k;
  const uint16_t* v;
  int64_t stride_tok, stride_head;
  int64_t T;
  // destination
  uint16_t* dk;
  uint16_t* dv;
  const int32_t* doffsets;    // [B + 1]
  int32_t* dlengths;          // [B]
  float* dmass;               // [Hkv][dT] or null
  int64_t dstride_tok, dstride_head;
  int64_t dT;
  int32_t B, Hkv, budget, sink, recent;
  int32_t n_listed;
  uint8_t heads[kMaxHeads];
  uint8_t slot[kMaxHeads];    // head slots in the source
  uint8_t dslot[kMaxHeads];
};

constexpr int kEvictThreads = 256;

// grid (position chunks of kEvictThreads * 4, listed heads, sequences).  Also clears the counters that the
// select behind it expects at zero: their place depends on the cache, and the workspace may have
// served another one.
__global__ void __launch_bounds__(kEvictThreads) evict_key_kernel(const EvictParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t block = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  const int64_t threads = (int64_t)gridDim.x * gridDim.y * gridDim.z * kEvictThreads;
  for (int64_t i = block * kEvictThreads + threadIdx.x; i < p.n_counters; i += threads) p.counters[i] = 0u;
  const int b = blockIdx.z, g = p.heads[blockIdx.y];
  int off;
  const int L = seq_length(p.offsets, p.lengths, b, false, &off);
  const float* src = p.mass + (int64_t)g * p.T + off;
  float* dst = p.scores + (int64_t)g * p.T + off;
  const int p0 = blockIdx.x * (kEvictThreads * 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pos = p0 + i * kEvictThreads + threadIdx.x;
    if (pos < L) {
      dst[pos] = evict_score(src[pos], pos, L, p.sink, p.recent);
    }
  }
}

// grid (chunks of kEvictRows kept rows, listed heads, sequences): D / 8 lanes copy one row's 16-byte
// pieces of K and V; a thread has the loads of all its rows in flight before the first store.  The rows
// kept are taken from the select's counts, not from the source's lengths: dlengths may be that array.
constexpr int kEvictRows = 64;

template <int D>
__global__ void __launch_bounds__(kEvictThreads) evict_copy_kernel(const EvictParams p) {
  grid_dep_wait();
  grid_dep_launch();
  constexpr int LPR = D / 8;                   // lanes per row
  constexpr int RPP = kEvictThreads / LPR;     // rows per pass
  constexpr int NP = kEvictRows / RPP;         // passes
  const int b = blockIdx.z, g = p.heads[blockIdx.y], tid = threadIdx.x;
  const int off = p.offsets[b], cap = p.offsets[b + 1] - off;
  const int kept = p.count[(int64_t)b * p.Hkv + g];
  const int doff = p.doffsets[b], dcap = p.doffsets[b + 1] - doff;
  // the list is padded to the budget, so that its loads need not wait for the count's
  const int32_t* lst = p.idx + ((int64_t)b * p.Hkv + g) * p.budget;
  const int j0 = blockIdx.x * kEvictRows, ch = (tid % LPR) * 8, r0 = tid / LPR;
  int pos[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int j = j0 + i * RPP + r0;
    pos[i] = j < p.budget ? lst[j] : -1;
  }
  const bool region = dcap >= 0 && doff >= 0 && (int64_t)doff + dcap <= p.dT;
  const int n = region && kept <= dcap ? kept : 0;  // rows moved: all or none
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    if (n < kept || !region) record_error(kCheckCapacity, b, kept, dcap);
    p.dlengths[b] = n;
  }
  if (!region) return;
  if (p.dmass) {  // slots past the kept rows start without weight
    float* dm = p.dmass + (int64_t)g * p.dT + doff;
    for (int j = n + blockIdx.x * kEvictThreads + tid; j < dcap; j += gridDim.x * kEvictThreads) dm[j] = 0.f;
  }
  if (j0 >= n) return;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int j = j0 + i * RPP + r0;
    if (j < n && (pos[i] < 0 || pos[i] >= cap)) record_error(kCheckPosition, b, g, pos[i]);
    if (j >= n || pos[i] >= cap) pos[i] = -1;
  }
  const uint16_t* kb = p.k + (int64_t)off * p.stride_tok + (int64_t)p.slot[g] * p.stride_head + ch;
  const uint16_t* vb = p.v + (int64_t)off * p.stride_tok + (int64_t)p.slot[g] * p.stride_head + ch;
  uint4 kr[NP], vr[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (pos[i] >= 0) {
      kr[i] = ld_stream_v4(kb + (int64_t)pos[i] * p.stride_tok);
      vr[i] = ld_stream_v4(vb + (int64_t)pos[i] * p.stride_tok);
    }
  uint16_t* dkb = p.dk + (int64_t)(doff + j0 + r0) * p.dstride_tok + (int64_t)p.dslot[g] * p.dstride_head + ch;
  uint16_t* dvb = p.dv + (int64_t)(doff + j0 + r0) * p.dstride_tok + (int64_t)p.dslot[g] * p.dstride_head + ch;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    if (pos[i] >= 0) {
      *reinterpret_cast<uint4*>(dkb + (int64_t)(i * RPP) * p.dstride_tok) = kr[i];
      *reinterpret_cast<uint4*>(dvb + (int64_t)(i * RPP) * p.dstride_tok) = vr[i];
    }
  if (p.dmass && tid < kEvictRows && j0 + tid < n) {
    const int s = lst[j0 + tid];
    if (s >= 0 && s < cap) p.dmass[(int64_t)g * p.dT + doff + j0 + tid] = p.mass[(int64_t)g * p.T + off + s];
  }
}

}  // namespace aoh
