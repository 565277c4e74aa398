// y = act(x W^T + bias + c (x A) B) + residual: one dense projection with segmented
// multi-LoRA ([vLLM MoE-LoRA page], "O Papel da Multi-LoRA"; segments as in SGMV, [Punica
// review page], "提案手法"), everything behind the product fused into its epilogue
// ("Otimizações em Nível de Kernel").
#include "fused_tc.cuh"
#include "prof.h"

#include <algorithm>

namespace mlb {

// ---------------------------------------------------------------- fp32
// z_t = c x_t A_a(t) of fp32 adapters: a warp per (token, 4 ranks), lanes split h_in.  The call's
// first kernel: it also records each token's adapter for the projection, checks the segments
// and writes the status word.
__global__ void __launch_bounds__(256) fused_shrink_f32_kernel(const DenseFusedArgs a) {
  __shared__ int s_wrong;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();     // what ran ahead of the call is done, for the projection too
  pdl_trigger();  // which multiplies meanwhile
  if (blockIdx.x == 0) {
    if (tid == 0) s_wrong = 0x7fffffff;
    __syncthreads();
    int wrong = 0x7fffffff;
    for (int s = tid; s < a.S; s += 256)
      if (segment_wrong(a.seg_offsets[s], a.seg_offsets[s + 1], a.seg_adapter[s], a.T, a.L)) wrong = min(wrong, s);
    atomicMin(&s_wrong, wrong);
    __syncthreads();
    if (tid == 0) {
      a.status[0] = s_wrong != 0x7fffffff ? MOE_LORA_ERR_DEVICE_CHECK : MOE_LORA_OK;
      a.status[1] = s_wrong != 0x7fffffff ? s_wrong : 0;
    }
  }
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (tid >> 5);
  const int t = static_cast<int>(w / (a.r / 4)), i0 = static_cast<int>(w % (a.r / 4)) * 4;
  if (t >= a.T) return;
  const int s = segment_of(a.seg_offsets, a.S, t);
  int ad = s >= 0 ? a.seg_adapter[s] : -1;
  if (ad >= a.L || ad < 0) ad = -1;
  if (lane == 0 && i0 == 0) a.row_adapter[t] = ad;
  if (ad < 0) return;  // nobody reads its z
  const float4* x = reinterpret_cast<const float4*>(static_cast<const float*>(a.x) + static_cast<size_t>(t) * a.h_in);
  const float4* A = reinterpret_cast<const float4*>(static_cast<const float*>(a.lora_a) +
                                                    (static_cast<size_t>(ad) * a.r + i0) * a.h_in);
  const int h4 = a.h_in / 4;
  float acc[4] = {};
#pragma unroll 4
  for (int h = lane; h < h4; h += 32) {
    const float4 v = x[h];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 m = A[static_cast<size_t>(i) * h4 + h];
      acc[i] = fmaf(v.x, m.x, fmaf(v.y, m.y, fmaf(v.z, m.z, fmaf(v.w, m.w, acc[i]))));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v = warp_sum(acc[i]);
    if (lane == i) a.z[static_cast<size_t>(t) * a.r + i0 + i] = a.scale * v;
  }
}

// fp32 projection on CUDA cores: 64 tokens x 64 features per tile (both halves of a gated
// feature), 4 x 4 per thread from shared memory.  Few tiles leave SMs idle, so a cluster of C
// CTAs splits h_in for a tile and each finishes 64 / C tokens, their partial sums added up in
// rank order from the peers' shared memory (64 x 512 -> 512: 8 tiles, 64 CTAs, 9.9 us with
// adapters; two dependent launches and the K loop's latency bound it).
constexpr int kF32K = 32, kF32Pitch = 68;  // K step; floats per row, 16-byte aligned

template <bool GATED>
__global__ void __launch_bounds__(256) fused_f32_kernel(const DenseFusedArgs a, int C) {
  constexpr int NH = GATED ? 2 : 1;
  constexpr int kTile = kF32K * kF32Pitch;
  __shared__ alignas(16) float sm[(NH + 1) * kTile > NH * 64 * kF32Pitch ? (NH + 1) * kTile : NH * 64 * kF32Pitch];
  float* xs = sm;             // [kF32K][pitch], tokens along a row
  float* ws = sm + kTile;     // [NH][kF32K][pitch], features along a row
  float* part = sm;           // [NH][64 tokens][pitch], once the tiles are done
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int rank = static_cast<int>(blockIdx.x) % C, f0 = static_cast<int>(blockIdx.x) / C * 64;
  const int t0 = blockIdx.y * 64;
  if (a.r == 0) {  // the call's only kernel
    pdl_wait();
    if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) a.status[0] = 0;
  }
  const int nk = (a.h_in + kF32K - 1) / kF32K;
  const int k0 = static_cast<int>(static_cast<long long>(nk) * rank / C);
  const int k1 = static_cast<int>(static_cast<long long>(nk) * (rank + 1) / C);
  const float* x = static_cast<const float*>(a.x);
  const float* w = static_cast<const float*>(a.w);
  // a thread brings 4 K values of row tid % 64 twice per operand and K step
  const int row = tid & 63, kq = (tid >> 6) * 4;
  const float* xr = t0 + row < a.T ? x + static_cast<size_t>(t0 + row) * a.h_in : nullptr;
  const float* wr[NH];
#pragma unroll
  for (int h = 0; h < NH; ++h)
    wr[h] = f0 + row < a.h_out ? w + (static_cast<size_t>(h) * a.h_out + f0 + row) * a.h_in : nullptr;
  float4 nx[2], nw[NH][2];
  auto fetch = [&](int kb) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = kb * kF32K + kq + u * 16;
      const bool in = kb < k1 && k < a.h_in;  // (h_in is a multiple of 8)
      nx[u] = in && xr != nullptr ? __ldg(reinterpret_cast<const float4*>(xr + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int h = 0; h < NH; ++h)
        nw[h][u] = in && wr[h] != nullptr ? __ldg(reinterpret_cast<const float4*>(wr[h] + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  float acc[NH][4][4] = {};
  fetch(k0);
  for (int kb = k0; kb < k1; ++kb) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float* d = xs + (kq + u * 16) * kF32Pitch + row;
      d[0] = nx[u].x;
      d[kF32Pitch] = nx[u].y;
      d[2 * kF32Pitch] = nx[u].z;
      d[3 * kF32Pitch] = nx[u].w;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float* e = ws + h * kTile + (kq + u * 16) * kF32Pitch + row;
        e[0] = nw[h][u].x;
        e[kF32Pitch] = nw[h][u].y;
        e[2 * kF32Pitch] = nw[h][u].z;
        e[3 * kF32Pitch] = nw[h][u].w;
      }
    }
    __syncthreads();
    fetch(kb + 1);
#pragma unroll 8
    for (int k = 0; k < kF32K; ++k) {
      const float4 xv = *reinterpret_cast<const float4*>(xs + k * kF32Pitch + ty * 4);
      const float xa[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float4 wv = *reinterpret_cast<const float4*>(ws + h * kTile + k * kF32Pitch + tx * 4);
        const float wa[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(xa[i], wa[j], acc[h][i][j]);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(part + (h * 64 + ty * 4 + i) * kF32Pitch + tx * 4) =
          make_float4(acc[h][i][0], acc[h][i][1], acc[h][i][2], acc[h][i][3]);
  cluster_sync_all();
  pdl_trigger();  // a call behind this one may set itself up
  if (a.r) pdl_wait();  // z
  // tokens [rank 64 / C, ...): 16 threads per token, 4 features each
  for (int tok = rank * (64 / C) + ty; tok < (rank + 1) * (64 / C); tok += 16) {
    const int t = t0 + tok, f = f0 + tx * 4;
    if (t >= a.T || f >= a.h_out) continue;
    float v[NH][4];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const uint32_t at = smem_u32(part + (h * 64 + tok) * kF32Pitch + tx * 4);
      float4 p[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < C) p[c] = ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(c)));
      v[h][0] = p[0].x;
      v[h][1] = p[0].y;
      v[h][2] = p[0].z;
      v[h][3] = p[0].w;
#pragma unroll
      for (int c = 1; c < 8; ++c)
        if (c < C) {
          v[h][0] += p[c].x;
          v[h][1] += p[c].y;
          v[h][2] += p[c].z;
          v[h][3] += p[c].w;
        }
      if (a.bias != nullptr) {
        const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.bias) + h * a.h_out + f));
        v[h][0] += b.x;
        v[h][1] += b.y;
        v[h][2] += b.z;
        v[h][3] += b.w;
      }
    }
    const int ad = a.r ? a.row_adapter[t] : -1;
    if (ad >= 0) {
      const float* zr = a.z + static_cast<size_t>(t) * a.r;
      const float* bp = static_cast<const float*>(a.lora_b) + static_cast<size_t>(ad) * a.r * a.n + f;
#pragma unroll 8
      for (int i = 0; i < a.r; ++i) {
        const float zi = zr[i];
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const float4 b = __ldg(reinterpret_cast<const float4*>(bp + static_cast<size_t>(i) * a.n + h * a.h_out));
          v[h][0] = fmaf(zi, b.x, v[h][0]);
          v[h][1] = fmaf(zi, b.y, v[h][1]);
          v[h][2] = fmaf(zi, b.z, v[h][2]);
          v[h][3] = fmaf(zi, b.w, v[h][3]);
        }
      }
    }
    if (GATED) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[0][j] = silu(v[0][j]) * v[NH - 1][j];
    } else {
      act_apply<false>(a.act, v[0]);
    }
    const size_t at = static_cast<size_t>(t) * a.h_out + f;
    float4 o = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
    if (a.residual != nullptr) {
      const float4 res = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + at);
      o = make_float4(o.x + res.x, o.y + res.y, o.z + res.z, o.w + res.w);
    }
    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = o;
  }
  cluster_sync_all();  // the peers have read this CTA's partial sums
}

static cudaError_t launch_f32(const DenseFusedArgs& a, cudaStream_t st) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.r > 0) {
    ProfScope ps(K_FUSED_SHRINK, st);
    const long long warps = static_cast<long long>(a.T) * (a.r / 4);
    cfg.gridDim = dim3(static_cast<unsigned>((warps + 7) / 8));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fused_shrink_f32_kernel, a);
    count_launch();
    if (e != cudaSuccess) return e;
  }
  ProfScope ps(K_DENSE_FUSED, st);
  // splits of h_in: as many as keep two CTAs per SM, of two K steps at least
  const int ft = (a.h_out + 63) / 64, tt = (a.T + 63) / 64, nk = (a.h_in + kF32K - 1) / kF32K;
  int C = 8;
  while (C > 1 && (static_cast<long long>(ft) * tt * C > 2 * a.num_sms || nk / C < 2)) C /= 2;
  cfg.gridDim = dim3(ft * C, tt);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  const cudaError_t e = a.act == ML_ACT_SILU_AND_MUL ? cudaLaunchKernelEx(&cfg, fused_f32_kernel<true>, a, C)
                                                     : cudaLaunchKernelEx(&cfg, fused_f32_kernel<false>, a, C);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Up to here the adapters' shrink runs on CUDA cores (up to kFusedDecodeTokens where it is
// small: 203 x 2056 -> 1000 with 5 adapters of rank 8: 16.7 us in all, on the tensor cores 18.4)
constexpr int kSmallTokens = 64;

cudaError_t launch_dense_fused(const DenseFusedArgs& a, cudaStream_t st) {
  if (a.T <= 0) return cudaSuccess;
  if (!a.f32) {
    FusedTcArgs f{};
    f.a = a;
    f.z = reinterpret_cast<__nv_bfloat16*>(a.z);
    f.zc = static_cast<__nv_bfloat16*>(a.zc);
    f.zc_pitch = a.zc_pitch;
    f.tile_mask = a.tile_mask;
    f.bad_part = a.bad_part;
    f.scan_ctas = std::min(kFusedScanMax, 2 * a.num_sms);
    if (a.r > 0) {
      const bool simt = a.T <= kSmallTokens || (a.T <= kFusedDecodeTokens && fused_shrink_is_small(a));
      const cudaError_t e = simt ? launch_fused_shrink_simt(f, st)
                                                : launch_fused_shrink_tc(f, a.T > kFusedDecodeTokens, st);
      if (e != cudaSuccess) return e;
    }
    return a.T <= kFusedDecodeTokens ? launch_fused_decode_tc(f, st) : launch_fused_prefill_tc(f, st);
  }
  return launch_f32(a, st);
}

}  // namespace mlb
