// Attention of new tokens by head role (prompt, chunk of a prompt, or single tokens).
//
// Sequence b has n_b = q_offsets[b + 1] - q_offsets[b] query rows, the last n_b of its L_b
// cached positions: row i stands at p = L_b - n_b + i and sees
//     DENSE:   t <= p
//     STREAM:  t <= p and (t < sink or t > p - window)
// out[i][h] = sum_t softmax_t(scale q_ih . k_t) v_t over the seen t; nothing seen: zeros.
#pragma once

#include "device_common.cuh"

namespace aoh {

struct PrefillParams {
  const uint16_t* q;          // [total_q][Hq][d]
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* offsets;     // [B + 1]
  const int32_t* lengths;     // [B] or null
  const int32_t* q_offsets;   // [B + 1]
  uint16_t* out;              // bf16 [total_q][Hq][d]
  int64_t stride_tok, stride_head;
  int32_t B, Hq, Hkv, G, total_q, sink, window;
  float scale_log2;
  int32_t n_listed;
  uint8_t heads[kMaxHeads];
  uint8_t roles[kMaxHeads];
  uint8_t slot[kMaxHeads];
};

// One warp per (query row, q head); lane j holds dims j * D / 32 ..
template <int D>
__global__ void __launch_bounds__(128) role_prefill_kernel(const PrefillParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int per_row = p.n_listed * p.G;
  const int row = (int)(item / per_row), hl = (int)(item % per_row);
  if (row >= p.total_q || row >= p.q_offsets[p.B]) return;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {  // the sequence of the row
    const int mid = (lo + hi + 1) >> 1;
    if (p.q_offsets[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int b = lo, g = p.heads[hl / p.G], h = g * p.G + hl % p.G;
  const int n = p.q_offsets[b + 1] - p.q_offsets[b];
  int off;
  const int L = seq_length(p.offsets, p.lengths, b, false, &off);
  const int pos = L - n + row - p.q_offsets[b];
  float q[E], acc[E];
  const uint16_t* qp = p.q + ((int64_t)row * p.Hq + h) * D + lane * E;
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)qp[e] << 16) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t base = (int64_t)off * p.stride_tok + (int64_t)p.slot[g] * p.stride_head + lane * E;
  const int first = p.roles[g] == 1 ? pos + 1 : min(p.sink, pos + 1);
  const int second = max(first, p.window > pos ? 0 : pos + 1 - p.window);
  for (int t = 0; t <= pos; ++t) {
    if (t == first) t = second;
    if (t > pos) break;
    const uint16_t* kp = p.k + base + (int64_t)t * p.stride_tok;
    const uint16_t* vp = p.v + base + (int64_t)t * p.stride_tok;
    float x = 0.f;
    for (int e = 0; e < E; ++e) x = fmaf(q[e], __uint_as_float((uint32_t)kp[e] << 16), x);
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const float mn = fmaxf(m, x), al = exp2f(m - mn), w = exp2f(x - mn);
    l = l * al + w;
    m = mn;
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, __uint_as_float((uint32_t)vp[e] << 16), acc[e] * al);
  }
  uint16_t* op = p.out + ((int64_t)row * p.Hq + h) * D + lane * E;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int e = 0; e < E; ++e) op[e] = __bfloat16_as_ushort(__float2bfloat16_rn(acc[e] * inv));
}

}  // namespace aoh
