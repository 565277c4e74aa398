// Scored routing: softmax or sigmoid scores, a selection bias per expert, expert groups,
// top-k, renormalised and scaled weights, then the stable (expert, adapter) sort.
//
// A router sends each token to its most relevant experts ([vLLM MoE-LoRA page],
// "Entendendo os Modelos MoE"); scores, bias, groups and scaling are the generic forms of
// that choice.
#include "common.cuh"
#include "kernels.h"
#include "prof.h"

#include <cfloat>

namespace mlb {

// One warp chooses the experts of one token.  Lane l holds experts l, l + 32, ... (E <= 256,
// eight at most), its selection scores in c[8] (-inf for a NaN: below every number, since
// infinite logits and biases are clamped to the largest finite float first).
//
// The scores are computed in 64 bits: two experts whose 32-bit scores are equal or off by a
// rounding would otherwise be ordered by the rounding.

constexpr int kScWarps = 8;

__device__ __forceinline__ float clamp_finite(float v) { return fminf(fmaxf(v, -FLT_MAX), FLT_MAX); }  // NaN: FLT_MAX or -FLT_MAX, checked apart

__device__ __forceinline__ void warp_argmax(double& v, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ov = __shfl_xor_sync(0xffffffffu, v, o);
    const int oe = __shfl_xor_sync(0xffffffffu, e, o);
    if (ov > v || (ov == v && oe < e)) {
      v = ov;
      e = oe;
    }
  }
}

__global__ void __launch_bounds__(kScWarps * 32) score_topk_kernel(const float* __restrict__ logits,
                                                                  const float* __restrict__ score_bias,
                                                                  const RouteArgs a, const ScoreFormat f) {
  __shared__ double s_c[kScWarps][256];
  __shared__ double s_s[kScWarps][256];
  __shared__ int s_id[kScWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kScWarps + warp;
  if (t >= a.M) return;
  const int E = a.E, k = a.k;
  float l[8];
  bool bad = false;
  unsigned nan_mask = 0u, alive = 0u;
  float mx = -FLT_MAX;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    l[i] = -FLT_MAX;
    if (e < E) {
      alive |= 1u << i;
      const float v = logits[static_cast<size_t>(t) * E + e];
      if (v != v) nan_mask |= 1u << i;
      else l[i] = clamp_finite(v);
      mx = fmaxf(mx, l[i]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  double s[8], sum = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = 0.0;
    if (!((alive & ~nan_mask) >> i & 1u)) continue;
    s[i] = f.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l[i]))) : exp(static_cast<double>(l[i]) - mx);
    sum += s[i];
  }
  if (!f.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((alive & ~nan_mask) >> i & 1u) s[i] /= sum;
  }
  double c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    c[i] = -INFINITY;
    if (e >= E) continue;
    const float b = score_bias ? score_bias[e] : 0.f;
    if ((nan_mask >> i & 1u) || b != b) {
      bad = true;
      continue;
    }
    c[i] = f.by_logit ? static_cast<double>(l[i]) : s[i] + static_cast<double>(clamp_finite(b));
  }

  if (f.n_group > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < E) {
        s_c[warp][lane + 32 * i] = c[i];
        s_s[warp][lane + 32 * i] = s[i];
      }
    __syncwarp();
    // group scores: lane g holds groups g, g + 32, ...
    double gs[8];
    unsigned galive = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane + 32 * i;
      gs[i] = -INFINITY;
      if (g >= f.n_group) continue;
      galive |= 1u << i;
      double m1 = -INFINITY, m2 = -INFINITY;
      int e1 = g * f.group_size, e2 = e1;
      for (int j = 0; j < f.group_size; ++j) {
        const int e = g * f.group_size + j;
        const double v = s_c[warp][e];
        if (v > m1) {
          m2 = m1;
          e2 = e1;
          m1 = v;
          e1 = e;
        } else if (v > m2) {
          m2 = v;
          e2 = e;
        }
      }
      gs[i] = m1;
      // scores and biases summed apart, so that groups whose two best have the same scores
      // and the same sum of biases tie, whatever the roundings
      if (f.top2 && f.group_size > 1)
        gs[i] = m2 == -INFINITY ? m2
                                : (s_s[warp][e1] + s_s[warp][e2]) +
                                      (score_bias ? static_cast<double>(clamp_finite(score_bias[e1])) +
                                                        static_cast<double>(clamp_finite(score_bias[e2]))
                                                  : 0.0);
    }
    unsigned keep = 0u;  // this lane's experts in a kept group
    for (int j = 0; j < f.topk_group; ++j) {
      double bv = -INFINITY;
      int bg = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((galive >> i & 1u) && (bg == 0x7fffffff || gs[i] > bv)) {
          bv = gs[i];
          bg = lane + 32 * i;
        }
      warp_argmax(bv, bg);
      if ((bg & 31) == lane) galive &= ~(1u << (bg >> 5));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((lane + 32 * i) / f.group_size == bg) keep |= 1u << i;
    }
    alive &= keep;
  }

  for (int j = 0; j < k; ++j) {
    double bv = -INFINITY;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((alive >> i & 1u) && (be == 0x7fffffff || c[i] > bv)) {
        bv = c[i];
        be = lane + 32 * i;
      }
    warp_argmax(bv, be);
    if ((be & 31) == lane) alive &= ~(1u << (be >> 5));
    if (lane == 0) s_id[warp][j] = be;
  }
  __syncwarp();

  // weights of the chosen, in 32 bits.  Renormalised: relative to the largest chosen logit
  // (at most 0 for sigmoids), so that scores below the smallest float keep their ratio.
  int ad = a.adapter_ids[t];
  if (ad < -1 || ad >= a.L) {
    bad = true;
    ad = -1;
  }
  const int ap = ad >= 0 ? ad : a.L;
  float top = -FLT_MAX;
  if (f.renorm) {
    for (int j = lane; j < k; j += 32) {
      const float v = logits[static_cast<size_t>(t) * E + s_id[warp][j]];
      if (v == v) top = fmaxf(top, clamp_finite(v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (f.sigmoid) top = fminf(top, 0.f);
  } else {
    top = f.sigmoid ? 0.f : mx;
  }
  float wsum = 0.f;
  for (int j = lane; j < k; j += 32) {
    const int e = s_id[warp][j];
    const float raw = logits[static_cast<size_t>(t) * E + e];
    const float v = clamp_finite(raw);
    float w = 0.f;
    if (raw == raw) {
      if (!f.sigmoid) w = expf(v - top);
      else w = v > 0.f ? 1.f / (1.f + expf(-v)) : expf(v - top) / (1.f + expf(v));
    }
    wsum += w;
    a.topk_ids[static_cast<size_t>(t) * k + j] = e;
    a.topk_w[static_cast<size_t>(t) * k + j] = w;
    atomicAdd(a.key_count + e * (a.L + 1) + ap, 1);
  }
  wsum = warp_sum(wsum);
  float mul = f.scale;
  if (f.renorm) mul = wsum > 0.f ? f.scale / wsum : 0.f;
  else if (!f.sigmoid) mul = f.scale / static_cast<float>(sum);
  for (int j = lane; j < k; j += 32) a.topk_w[static_cast<size_t>(t) * k + j] *= mul;
  if (lane == 0) a.a_key[t] = ap;
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(a.status, MOE_LORA_ERR_DEVICE_CHECK, t);
}

cudaError_t launch_route_scored(const RouteArgs& a, const ScoreFormat& f, const float* score_bias, cudaStream_t st) {
  const int nk = a.E * (a.L + 1);
  if (a.M == 0) return cudaMemsetAsync(a.seg_offsets, 0, sizeof(int32_t) * (nk + 1), st);
  cudaError_t err = cudaMemsetAsync(a.key_count, 0, sizeof(int32_t) * nk, st);
  if (err != cudaSuccess) return err;
  const float* lg = nullptr;
  err = launch_router_logits(a, &lg, st);
  if (err != cudaSuccess) return err;
  {
    ProfScope ps(K_ROUTE_SCORED, st);
    score_topk_kernel<<<(a.M + kScWarps - 1) / kScWarps, kScWarps * 32, 0, st>>>(lg, score_bias, a, f);
    count_launch();
  }
  return launch_sort_scatter(a, st);
}

}  // namespace mlb
