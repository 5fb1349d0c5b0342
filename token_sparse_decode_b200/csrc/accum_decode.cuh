// Decode attention that accumulates the attention weight of every cached token.
//
// For query rows h of KV head g and the positions t < L_b of sequence b:
//     x_ht = scale q_h . k_t,  w_ht = exp(x_ht - m_h) / l_h,  out_h = sum_t w_ht v_t,
//     mass_out[g][t] = decay mass_in[g][t] + sum_{h in g} w_ht.
// The final m_h and l_h are known only when the whole row has been read, so the work is two
// launches: the split-K gather reads K and V once, leaves (m, l, acc) per split and stores the
// logits (4 bytes per query row and token, against 4 d for the token's K and V: they stay in L2);
// accum_merge_kernel combines the splits' outputs and, with the row's m and l, turns the logits
// into weights and adds them to the mass.  Bound by the K / V bytes of the first launch.
#pragma once

#include "flash_gather.cuh"

namespace aoh {

constexpr int kAmThreads = 256;
constexpr int kAmTokens = 1024;               // tokens per CTA of the merge
constexpr int kAmOut = 16;                    // float4 outputs per CTA
constexpr int kAmGroups = kAmThreads / kAmOut;

struct AccumParams {
  FdecParams fd;
  const float* mass_in;   // [Hkv][T]
  float* mass_out;        // [Hkv][T], may be mass_in
  float decay;
};

// grid (max(token chunks, output slices), listed heads, sequences)
template <int D, int NT>
__global__ void __launch_bounds__(kAmThreads) accum_merge_kernel(const AccumParams ap) {
  grid_dep_wait();
  constexpr int NQP = NT * 8;
  const FdecParams& p = ap.fd;
  extern __shared__ __align__(16) uint8_t am_smem[];
  float* sml = reinterpret_cast<float*>(am_smem);  // [nsplit][NQP][2]: (m, l), then (w, l)
  __shared__ float sM[NQP], sInv[NQP], s_part[kAmThreads];
  __shared__ float4 sred[kAmGroups][kAmOut];
  const int tid = threadIdx.x, b = blockIdx.z, y = blockIdx.y, g = p.heads[y];
  const int row_id = b * gridDim.y + y;
  int off;
  const int L = seq_length(p.offsets, p.lengths, b, false, &off);
  const int nsplit = (L + p.chunk - 1) / p.chunk;
  const int n_out = p.NQ * (D / 4), o0 = blockIdx.x * kAmOut, t0 = blockIdx.x * kAmTokens;
  if (nsplit == 0 || (o0 >= n_out && t0 >= L)) return;  // no position: the gather wrote zero rows
  const float* rml = p.part_ml + (int64_t)row_id * p.max_splits * NQP * 2;
  for (int e = tid; e < nsplit * NQP * 2; e += kAmThreads) sml[e] = __ldcg(rml + e);
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
    const float* mi = ap.mass_in ? ap.mass_in + (int64_t)g * p.T + off : nullptr;
    float* mo = ap.mass_out + (int64_t)g * p.T + off;
    const float* lg = p.logits + ((int64_t)g * p.T + off) * p.logit_pitch;
    for (int t = t0 + tid; t < t1; t += kAmThreads) {
      const float2* row = reinterpret_cast<const float2*>(lg + (int64_t)t * p.logit_pitch);
      float s = 0.f;
      for (int q = 0; q < p.NQ; q += 2) {
        const float2 x = __ldcg(row + (q >> 1));
        s += exp2f(x.x - sM[q]) * sInv[q];
        if (q + 1 < p.NQ) s += exp2f(x.y - sM[q + 1]) * sInv[q + 1];
      }
      mo[t] = mi ? fmaf(ap.decay, mi[t], s) : s;
    }
  }

  // the outputs: slices of kAmOut float4, kAmGroups threads over the splits of each
  if (o0 < n_out) {
    const int ol = tid % kAmOut, s0 = tid / kAmOut, o = o0 + ol;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    const int qr = o / (D / 4), dd = (o % (D / 4)) * 4;
    if (o < n_out) {
      const float* col = p.part_acc + (int64_t)row_id * p.max_splits * NQP * D + (int64_t)qr * D + dd;
      for (int s = s0; s < nsplit; s += kAmGroups) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(col + (int64_t)s * NQP * D));
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
