// Decode attention that accumulates the attention weight of every cached token.
//
// For query rows h of KV head g and the positions t < L_b of sequence b:
//     x_ht = scale q_h . k_t,  w_ht = exp(x_ht - m_h) / l_h,  out_h = sum_t w_ht v_t,
//     mass_out[g][t] = decay mass_in[g][t] + sum_{h in g} w_ht.
// The final m_h and l_h are known only when the whole row has been read, so the work is two
// launches: dense_pass_kernel reads K and V once and stores the logits (4 bytes per query row and
// token, against 4 d for the token's K and V: they stay in L2); accum_merge_kernel joins the rows
// that several CTAs shared and, with each row's m and l, turns the logits into weights and adds
// them to the mass.  Bound by the K / V bytes of the first launch: 131072 tokens x 8 heads in 103 us (90 + 12
// for the weights and the gap), 48 sequences of 1 to 8000 x 4 heads in 89 us (71 + 17).  Loading a token's
// logits before its row's statistics are joined, and chunks of 512 or 2048 tokens, were 1 to 6 us slower.
#pragma once

#include "dense_pass.cuh"

namespace aoh {

constexpr int kAmThreads = 256;
constexpr int kAmTokens = 1024;               // tokens per CTA of the merge
constexpr int kAmOut = 64;                    // float4 outputs per CTA
constexpr int kAmGroups = kAmThreads / kAmOut;

struct AccumParams {
  DenseRows rows;
  const int32_t* offsets;
  const int32_t* lengths;
  const float* logits;    // [Hkv][T][logit_pitch]
  const float* mass_in;   // [Hkv][T] or null
  float* mass_out;        // [Hkv][T], may be mass_in
  float* out;             // fp32 [B][Hq][D]
  int64_t T;
  int32_t logit_pitch, B, Hq, G, n_listed;
  float decay;
  uint8_t heads[kMaxHeads];
};

// grid (max(token chunks, output slices), listed heads, sequences)
template <int D, int NT>
__global__ void __launch_bounds__(kAmThreads) accum_merge_kernel(const AccumParams p) {
  grid_dep_wait();
  constexpr int NQP = NT * 8;
  extern __shared__ __align__(16) uint8_t am_smem[];
  float* sml = reinterpret_cast<float*>(am_smem);  // [nsplit][NQP][2]: (m, l), then (w, l)
  __shared__ float sM[NQP], sInv[NQP], s_part[kAmThreads];
  __shared__ float4 sred[kAmGroups][kAmOut];
  const int tid = threadIdx.x, b = blockIdx.z, y = blockIdx.y, g = p.heads[y];
  int off, c0, c1;
  const int L = seq_length(p.offsets, p.lengths, b, false, &off);
  const int n_out = p.G * (D / 4), o0 = blockIdx.x * kAmOut, t0 = blockIdx.x * kAmTokens;
  if (!dense_row(p.rows, p.n_listed, p.B, y, b, &c0, &c1)) {  // no position: zero rows
    if (o0 < n_out && tid < kAmOut && o0 + tid < n_out) {
      const int o = o0 + tid;
      *reinterpret_cast<float4*>(p.out + ((int64_t)b * p.Hq + g * p.G + o / (D / 4)) * D + (o % (D / 4)) * 4) =
          make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const bool joined = c0 == c1;  // one CTA had the whole row and wrote its output
  if ((joined || o0 >= n_out) && t0 >= L) return;
  const int nsplit = c1 - c0 + 1;
  const float* row_ml = p.rows.row_ml + ((int64_t)y * p.B + b) * NQP * 2;
  for (int e = tid; e < nsplit * NQP * 2; e += kAmThreads)
    sml[e] = __ldcg(joined ? row_ml + e : p.rows.part_ml + (int64_t)dense_part(c0, e / (NQP * 2)) * NQP * 2 + e % (NQP * 2));
  __syncthreads();
  // row statistics: M_q = max m, L_q = sum 2^(m - M_q) l, in a fixed order
  constexpr int SP = kAmThreads / NQP;
  const int rq = tid % NQP, sj = tid / NQP;
  float M = -INFINITY;
  for (int s = sj; s < nsplit; s += SP) M = fmaxf(M, sml[(s * NQP + rq) * 2]);
  s_part[tid] = M;
  __syncthreads();
  if (tid < NQP) {
    M = s_part[tid];
    for (int j = 1; j < SP; ++j) M = fmaxf(M, s_part[j * NQP + tid]);
    sM[tid] = M;
  }
  __syncthreads();
  float Ls = 0.f;
  for (int s = sj; s < nsplit; s += SP) {
    const float w = exp2f(sml[(s * NQP + rq) * 2] - sM[rq]);
    sml[(s * NQP + rq) * 2] = w;
    Ls += w * sml[(s * NQP + rq) * 2 + 1];
  }
  s_part[tid] = Ls;
  __syncthreads();
  if (tid < NQP) {
    Ls = 0.f;
    for (int j = 0; j < SP; ++j) Ls += s_part[j * NQP + tid];
    sInv[tid] = 1.f / Ls;
  }
  __syncthreads();

  // the mass of this CTA's tokens
  if (t0 < L) {
    const int t1 = min(L, t0 + kAmTokens);
    const float* mi = p.mass_in ? p.mass_in + (int64_t)g * p.T + off : nullptr;
    float* mo = p.mass_out + (int64_t)g * p.T + off;
    const float* lg = p.logits + ((int64_t)g * p.T + off) * p.logit_pitch;
    constexpr int PT = kAmTokens / kAmThreads;  // tokens of a thread, their loads in flight together
    float w[PT], old[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int t = t0 + tid + i * kAmThreads;
      w[i] = 0.f;
      old[i] = mi && t < t1 ? mi[t] : 0.f;
    }
    for (int q = 0; q < p.G; q += 2) {
      float2 x[PT];
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        const int t = t0 + tid + i * kAmThreads;
        x[i] = t < t1 ? __ldcg(reinterpret_cast<const float2*>(lg + (int64_t)t * p.logit_pitch + q)) : make_float2(-INFINITY, -INFINITY);
      }
      const bool two = q + 1 < p.G;
      const float M0 = sM[q], I0 = sInv[q], M1 = two ? sM[q + 1] : 0.f, I1 = two ? sInv[q + 1] : 0.f;
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        w[i] += ex2(x[i].x - M0) * I0;
        if (two) w[i] += ex2(x[i].y - M1) * I1;
      }
    }
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int t = t0 + tid + i * kAmThreads;
      if (t < t1) mo[t] = mi ? fmaf(p.decay, old[i], w[i]) : w[i];
    }
  }

  // the outputs: slices of kAmOut float4, kAmGroups threads over the splits of each
  if (o0 < n_out && !joined) {
    const int ol = tid % kAmOut, s0 = tid / kAmOut, o = o0 + ol;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    const int qr = o / (D / 4), dd = (o % (D / 4)) * 4;
    if (o < n_out) {
      for (int s = s0; s < nsplit; s += kAmGroups) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(
            p.rows.part_acc + ((int64_t)dense_part(c0, s) * NQP + qr) * D + dd));
        const float w = sml[(s * NQP + qr) * 2];
        A.x += w * v.x;
        A.y += w * v.y;
        A.z += w * v.z;
        A.w += w * v.w;
      }
    }
    sred[s0][ol] = A;
    __syncthreads();
    if (s0 == 0 && o < n_out) {
      float4 T = sred[0][ol];
#pragma unroll
      for (int j = 1; j < kAmGroups; ++j) {
        T.x += sred[j][ol].x;
        T.y += sred[j][ol].y;
        T.z += sred[j][ol].z;
        T.w += sred[j][ol].w;
      }
      const float inv = sInv[qr];
      float4* out = reinterpret_cast<float4*>(p.out + ((int64_t)b * p.Hq + g * p.G + qr) * D + dd);
      *out = make_float4(T.x * inv, T.y * inv, T.z * inv, T.w * inv);
    }
  }
}

}  // namespace aoh
