// Decode attention of a batch whose sequences share long prefixes.
//
// Sequences [seq_start[i], seq_start[i + 1]) continue prefix i (P_i cached tokens, stored once);
// sequence b has L_b tokens of its own.  For every q head h of KV head g:
//     out[b][h] = softmax-weighted sum of v over the P_i prefix tokens and the L_b own tokens.
#pragma once

#include "device_common.cuh"

namespace aoh {

struct PrefixParams {
  const uint16_t* q;           // [B][Hq][d]
  const uint16_t* pk;          // prefix cache
  const uint16_t* pv;
  const int32_t* poffsets;     // [NP + 1]
  const int32_t* plengths;     // [NP] or null
  const int32_t* seq_start;    // [NP + 1] or null (one prefix, every sequence)
  int64_t pstride_tok, pstride_head;
  const uint16_t* k;           // the sequences' own caches
  const uint16_t* v;
  const int32_t* offsets;
  const int32_t* lengths;
  int64_t stride_tok, stride_head;
  float* out;                  // fp32 [B][Hq][d]
  int32_t B, NP, Hq, Hkv, G;
  float scale_log2;
  int32_t n_listed;
  uint8_t heads[kMaxHeads];
  uint8_t slot[kMaxHeads];
  uint8_t pslot[kMaxHeads];
};

// The prefix that sequence b continues (-1: none; recorded)
__device__ __forceinline__ int prefix_of(const int32_t* seq_start, int NP, int b) {
  if (!seq_start) return 0;
  for (int i = 0; i < NP; ++i)
    if (b >= seq_start[i] && b < seq_start[i + 1]) return i;
  return -1;
}

// One warp per (sequence, q head)
template <int D>
__global__ void __launch_bounds__(128) prefix_decode_kernel(const PrefixParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int per_row = p.n_listed * p.G;
  const int b = (int)(item / per_row), hl = (int)(item % per_row);
  if (b >= p.B) return;
  const int g = p.heads[hl / p.G], h = g * p.G + hl % p.G;
  float q[E], acc[E];
  const uint16_t* qp = p.q + ((int64_t)b * p.Hq + h) * D + lane * E;
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)qp[e] << 16) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto attend = [&](const uint16_t* kb, const uint16_t* vb, int64_t stride, int L) {
    for (int t = 0; t < L; ++t) {
      const uint16_t* kp = kb + (int64_t)t * stride;
      const uint16_t* vp = vb + (int64_t)t * stride;
      float x = 0.f;
      for (int e = 0; e < E; ++e) x = fmaf(q[e], __uint_as_float((uint32_t)kp[e] << 16), x);
      for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      const float mn = fmaxf(m, x), al = exp2f(m - mn), w = exp2f(x - mn);
      l = l * al + w;
      m = mn;
      for (int e = 0; e < E; ++e) acc[e] = fmaf(w, __uint_as_float((uint32_t)vp[e] << 16), acc[e] * al);
    }
  };
  int off;
  const int i = prefix_of(p.seq_start, p.NP, b);
  if (i < 0) {
    if (lane == 0) record_error(kCheckPosition, b, -1, p.NP);
  } else {
    const int P = seq_length(p.poffsets, p.plengths, i, false, &off);
    const int64_t base = (int64_t)off * p.pstride_tok + (int64_t)p.pslot[g] * p.pstride_head + lane * E;
    attend(p.pk + base, p.pv + base, p.pstride_tok, P);
  }
  const int L = seq_length(p.offsets, p.lengths, b, false, &off);
  const int64_t base = (int64_t)off * p.stride_tok + (int64_t)p.slot[g] * p.stride_head + lane * E;
  attend(p.k + base, p.v + base, p.stride_tok, L);
  float* op = p.out + ((int64_t)b * p.Hq + h) * D + lane * E;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int e = 0; e < E; ++e) op[e] = acc[e] * inv;
}

}  // namespace aoh
