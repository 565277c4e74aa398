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

// fp32 projection on CUDA cores: 64 tokens x 128 weight rows per tile (gated: 64 gate rows and
// the matching 64 up rows), 8 x 8 per thread from shared memory (4 x 8 waited for its loads:
// 512 x 2048 -> 2048 in 135 us), two rows per packed multiply-add.  Few tiles leave SMs idle, so a cluster of C CTAs splits h_in for a tile and
// each finishes 64 / C tokens, their partial sums added up in rank order from the peers' shared
// memory (64 x 512 -> 512: 4 tiles, 10.7 us with adapters; two dependent launches and the K
// loop's latency bound it.  468 x 1576 -> 864: 45 us; 512 x 2048 -> 2048: 106 us, 41 TFLOP/s).
constexpr int kF32Threads = 128, kF32K = 16, kF32Pitch = 68;  // K step; floats per token of the partial sums

// Shared tiles hold 64 rows per K value.  Four lanes bring 64 bytes of a row, so the runs of four
// rows are swapped by the K value's quarter: neither the stores nor the loads meet a bank twice.
__device__ __forceinline__ int f32_at(int k, int row4) { return k * 64 + ((row4 ^ (k / 4 * 2)) << 2); }

// d += a b, two fp32 fused multiply-adds
__device__ __forceinline__ void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ uint64_t twice(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}

template <bool GATED>
__global__ void __launch_bounds__(kF32Threads, 3) fused_f32_kernel(const DenseFusedArgs a, int C) {
  constexpr int kTile = kF32K * 64, kBuf = 3 * kTile;  // x, then the two halves of w
  __shared__ alignas(16) float sm[2 * kBuf > 128 * kF32Pitch ? 2 * kBuf : 128 * kF32Pitch];
  float* part = sm;  // [2 halves][64 tokens][pitch], once the tiles are done
  const int tid = threadIdx.x, warp = tid >> 5;
  // a warp has 32 tokens x one half's 64 rows, a lane runs of four of both, and four more 16
  // tokens or 32 rows on
  const int half_of = warp & 1, x4 = (warp >> 1) * 8 + ((tid >> 3) & 3), w4 = tid & 7;
  const int rank = static_cast<int>(blockIdx.x) % C;
  const int f0 = static_cast<int>(blockIdx.x) / C * (GATED ? 64 : 128);
  const int second = GATED ? a.h_out : 64;  // the second half's rows follow the first's by
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
  // a thread brings 4 K values of rows tid / 4 and 32 on of x and of both halves of w per K step
  const int row = tid >> 2, kq = (tid & 3) * 4;
  const float* from[3][2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int rr = row + 32 * u;
    from[0][u] = t0 + rr < a.T ? x + static_cast<size_t>(t0 + rr) * a.h_in : nullptr;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      from[1 + h][u] = f0 + rr + (GATED ? 0 : h * 64) < a.h_out
                           ? w + (static_cast<size_t>(f0) + rr + static_cast<size_t>(h) * second) * a.h_in
                           : nullptr;
  }
  float4 n[3][2];
  auto fetch = [&](int kb) {
    const int k = kb * kF32K + kq;
    const bool in = kb < k1 && k < a.h_in;  // (h_in is a multiple of 8)
#pragma unroll
    for (int o = 0; o < 3; ++o)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        n[o][u] = in && from[o][u] != nullptr ? __ldg(reinterpret_cast<const float4*>(from[o][u] + k))
                                              : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  auto store = [&](float* buf) {
#pragma unroll
    for (int o = 0; o < 3; ++o)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float* d = buf + o * kTile + f32_at(kq, (row >> 2) + 8 * u) + (row & 3);  // (one swap for all four)
        d[0] = n[o][u].x;
        d[64] = n[o][u].y;
        d[128] = n[o][u].z;
        d[192] = n[o][u].w;
      }
  };
  uint64_t acc[8][4] = {};  // [token][pair of rows]
  fetch(k0);
  store(sm);
  fetch(k0 + 1);
  __syncthreads();
  for (int kb = k0; kb < k1; ++kb) {
    const float* buf = sm + ((kb - k0) & 1) * kBuf;
#pragma unroll
    for (int k = 0; k < kF32K; ++k) {
      uint64_t wv[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(buf + (1 + half_of) * kTile + f32_at(k, w4 + 8 * u));
        wv[2 * u] = v.x;
        wv[2 * u + 1] = v.y;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float4 xv = *reinterpret_cast<const float4*>(buf + f32_at(k, x4 + 4 * u));
        const uint64_t xa[4] = {twice(xv.x), twice(xv.y), twice(xv.z), twice(xv.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) fma2(acc[4 * u + i][j], xa[i], wv[j]);
      }
    }
    store(sm + ((kb + 1 - k0) & 1) * kBuf);  // (everyone left that buffer a barrier ago)
    fetch(kb + 2);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int u = 0; u < 2; ++u)
      *reinterpret_cast<ulonglong2*>(part + (half_of * 64 + (x4 + i / 4 * 4) * 4 + i % 4) * kF32Pitch + (w4 + 8 * u) * 4) =
          make_ulonglong2(acc[i][2 * u], acc[i][2 * u + 1]);
  cluster_sync_all();
  pdl_trigger();  // a call behind this one may set itself up
  if (a.r) pdl_wait();  // z
  // tokens [rank 64 / C, ...): 16 threads per token and half (gated: both halves at once), 4
  // features each
  constexpr int NH = GATED ? 2 : 1;
  for (int o = tid; o < (64 / C) * (GATED ? 16 : 32); o += kF32Threads) {
    const int tok = rank * (64 / C) + o / (GATED ? 16 : 32), half = GATED ? 0 : (o >> 4) & 1;
    const int t = t0 + tok, f = f0 + half * 64 + (o & 15) * 4;
    if (t >= a.T || f >= a.h_out) continue;
    float v[NH][4];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const uint32_t at = smem_u32(part + ((half + h) * 64 + tok) * kF32Pitch + (o & 15) * 4);
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
      for (int j = 0; j < 4; ++j) v[0][j] = sigmoid_of<false>(v[0][j], v[0][j]) * v[NH - 1][j];
    } else {
      act_apply<false>(a.act, v[0]);
    }
    const size_t at = static_cast<size_t>(t) * a.h_out + f;
    float4 y = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
    if (a.residual != nullptr) {
      const float4 res = *reinterpret_cast<const float4*>(static_cast<const float*>(a.residual) + at);
      y = make_float4(y.x + res.x, y.y + res.y, y.z + res.z, y.w + res.w);
    }
    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = y;
  }
  __syncwarp();
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
  // splits of h_in, of four K steps at least: a CTA alone on its SM takes about 2.2 times, two
  // take 2.5 times its share of a full SM, and a split adds its exchange (about two K steps)
  const bool gated = a.act == ML_ACT_SILU_AND_MUL;
  const int ft = (a.h_out + (gated ? 63 : 127)) / (gated ? 64 : 128), tt = (a.T + 63) / 64;
  const int nk = (a.h_in + kF32K - 1) / kF32K;
  int C = 1;
  double best = 0.0;
  for (int c = 1; c <= 8 && (c == 1 || nk / c >= 4); c *= 2) {
    const long long per_sm = (static_cast<long long>(ft) * tt * c + a.num_sms - 1) / a.num_sms;
    const double cost = (per_sm == 1 ? 2.2 : per_sm == 2 ? 2.5 : static_cast<double>(per_sm)) * (static_cast<double>(nk) / c + 2.0);
    if (c == 1 || cost < best) {
      best = cost;
      C = c;
    }
  }
  cfg.blockDim = dim3(kF32Threads);
  cfg.gridDim = dim3(ft * C, tt);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  const cudaError_t e = gated ? cudaLaunchKernelEx(&cfg, fused_f32_kernel<true>, a, C)
                              : cudaLaunchKernelEx(&cfg, fused_f32_kernel<false>, a, C);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Up to here the adapters' shrink runs on CUDA cores (with more tokens of a split projection where it is
// small: 203 x 2056 -> 1000 with 5 adapters of rank 8: 15.7 us in all, on the tensor cores 19.4)
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
    const bool stream = a.T <= kFusedDecodeTokens || fused_decode_pays(a);
    if (stream) {
      if (a.r > 0) {
        const bool simt = a.T <= kSmallTokens || fused_shrink_is_small(a);
        const cudaError_t e = simt ? launch_fused_shrink_simt(f, st) : launch_fused_shrink_tc(f, false, 0, a.T, st);
        if (e != cudaSuccess) return e;
      }
      return launch_fused_decode_tc(f, st);
    }
    const int band = a.r > 0 ? fused_band(a.zc_pitch) : a.T;
    for (int t0 = 0; t0 < a.T; t0 += band) {
      const int t1 = std::min(a.T, t0 + band);
      cudaError_t e = a.r > 0 ? launch_fused_shrink_tc(f, true, t0, t1, st) : cudaSuccess;
      if (e == cudaSuccess) e = launch_fused_prefill_tc(f, t0, t1, st);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
  return launch_f32(a, st);
}

}  // namespace mlb
