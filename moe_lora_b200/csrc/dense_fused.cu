// y = act(x W^T + bias + c (x A) B) + residual: one dense projection with segmented
// multi-LoRA ([vLLM MoE-LoRA page], "O Papel da Multi-LoRA"; segments as in SGMV, [Punica
// review page], "提案手法"), everything behind the product fused into its epilogue
// ("Otimizações em Nível de Kernel").
#include "fused_tc.cuh"
#include "prof.h"

namespace mlb {

// ---------------------------------------------------------------- adapters of the rows
// Each row's adapter from the segments by binary search: the last segment that begins at or
// before the row and ends behind it.  Segments that run backwards or leave [0, T], and
// adapter ids outside [-1, L), are flagged; their rows count as without an adapter.
__global__ void __launch_bounds__(256) row_adapter_kernel(const int32_t* __restrict__ off,
                                                         const int32_t* __restrict__ ad, int S, int T, int L,
                                                         int32_t* __restrict__ row_adapter, int* status) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < S && (off[i] > off[i + 1] || off[i] < 0 || off[i + 1] > T || ad[i] < -1 || ad[i] >= L))
    set_status(status, MOE_LORA_ERR_DEVICE_CHECK, i);
  if (i >= T) return;
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= i) lo = mid;
    else hi = mid;
  }
  int a = -1;
  if (S > 0 && off[lo] <= i && i < off[lo + 1]) a = ad[lo];
  row_adapter[i] = (a >= 0 && a < L) ? a : -1;
}

// z[t] = c x_t A_a(t): a warp per (row, 4 ranks), lanes split h_in.
__global__ void __launch_bounds__(256) fused_shrink_simt(const DenseFusedArgs a) {
  const int lane = threadIdx.x & 31;
  const long long w = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = static_cast<int>(w / a.r), i = static_cast<int>(w % a.r);
  if (t >= a.T) return;
  const int ad = a.row_adapter[t];
  float s = 0.f;
  if (ad >= 0) {
    const float* x = static_cast<const float*>(a.x) + static_cast<size_t>(t) * a.h_in;
    const float* A = static_cast<const float*>(a.lora_a) + (static_cast<size_t>(ad) * a.r + i) * a.h_in;
    for (int h = lane; h < a.h_in; h += 32) s = fmaf(*(x + h), *(A + h), s);
    s = warp_sum(s);
  }
  if (lane == 0) a.z[static_cast<size_t>(t) * a.r + i] = a.scale * s;
}

// CUDA-core projection: 32 tokens x 64 features per CTA (both halves of a gated feature).
template <bool GATED>
__global__ void __launch_bounds__(256) fused_simt_kernel(const DenseFusedArgs a) {
  constexpr int NH = GATED ? 2 : 1;
  __shared__ float xs[32][33];
  __shared__ float ws[NH][64][33];
  const int tid = threadIdx.x;
  const int ty = tid >> 4, tx = tid & 15;
  const int t0 = blockIdx.y * 32, f0 = blockIdx.x * 64;
  const float* x = static_cast<const float*>(a.x);
  const float* w = static_cast<const float*>(a.w);
  float acc[NH][2][4] = {};
  for (int k0 = 0; k0 < a.h_in; k0 += 32) {
    for (int idx = tid; idx < 32 * 32; idx += 256) {
      const int rr = idx >> 5, kk = idx & 31;
      const int t = t0 + rr, k = k0 + kk;
      xs[rr][kk] = (t < a.T && k < a.h_in) ? *(x + static_cast<size_t>(t) * a.h_in + k) : 0.f;
    }
    for (int idx = tid; idx < NH * 64 * 32; idx += 256) {
      const int h = idx >> 11, rr = (idx >> 5) & 63, kk = idx & 31;
      const int f = f0 + rr, k = k0 + kk;
      ws[h][rr][kk] = (f < a.h_out && k < a.h_in) ? *(w + (static_cast<size_t>(h) * a.h_out + f) * a.h_in + k) : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int kk = 0; kk < 32; ++kk) {
      const float x0 = xs[ty * 2][kk], x1 = xs[ty * 2 + 1][kk];
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float wv = ws[h][tx * 4 + j][kk];
          acc[h][0][j] = fmaf(x0, wv, acc[h][0][j]);
          acc[h][1][j] = fmaf(x1, wv, acc[h][1][j]);
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int t = t0 + ty * 2 + u;
    if (t >= a.T) continue;
    const int ad = a.r ? a.row_adapter[t] : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int f = f0 + tx * 4 + j;
      if (f >= a.h_out) continue;
      float v[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        v[h] = acc[h][u][j];
        const int fh = f + h * a.h_out;
        if (a.bias != nullptr) v[h] += *(static_cast<const float*>(a.bias) + fh);
        if (ad >= 0) {
          const float* zr = a.z + static_cast<size_t>(t) * a.r;
          const float* bp = static_cast<const float*>(a.lora_b) + static_cast<size_t>(ad) * a.r * a.n + fh;
          for (int i = 0; i < a.r; ++i) v[h] = fmaf(zr[i], *(bp + static_cast<size_t>(i) * a.n), v[h]);
        }
      }
      float o;
      if (GATED) {
        o = silu(v[0]) * v[NH - 1];
      } else {
        act_apply<false>(a.act, v);
        o = v[0];
      }
      const size_t at = static_cast<size_t>(t) * a.h_out + f;
      if (a.residual != nullptr) o += *(static_cast<const float*>(a.residual) + at);
      static_cast<float*>(a.y)[at] = o;
    }
  }
}

static cudaError_t launch_simt(const DenseFusedArgs& a, cudaStream_t st) {
  if (a.r > 0) {
    ProfScope ps(K_FUSED_SHRINK, st);
    const long long warps = static_cast<long long>(a.T) * a.r;
    fused_shrink_simt<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, st>>>(a);
    count_launch();
  }
  ProfScope ps(K_DENSE_FUSED, st);
  const dim3 grid((a.h_out + 63) / 64, (a.T + 31) / 32);
  if (a.act == ML_ACT_SILU_AND_MUL) fused_simt_kernel<true><<<grid, 256, 0, st>>>(a);
  else fused_simt_kernel<false><<<grid, 256, 0, st>>>(a);
  count_launch();
  return cudaGetLastError();
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
    f.bad = reinterpret_cast<uint64_t*>(a.status + 32);  // in the status block
    f.bad_part = a.bad_part;
    if (a.r > 0) {
      const bool simt = a.T <= kSmallTokens || (a.T <= kFusedDecodeTokens && fused_shrink_is_small(a));
      const cudaError_t e = simt ? launch_fused_shrink_simt(f, st)
                                                : launch_fused_shrink_tc(f, a.T > kFusedDecodeTokens, st);
      if (e != cudaSuccess) return e;
    }
    return a.T <= kFusedDecodeTokens ? launch_fused_decode_tc(f, st) : launch_fused_prefill_tc(f, st);
  }
  if (a.r > 0) {
    ProfScope ps(K_FUSED_SHRINK, st);
    const int n = a.T > a.S ? a.T : a.S;
    row_adapter_kernel<<<(n + 255) / 256, 256, 0, st>>>(a.seg_offsets, a.seg_adapter, a.S, a.T, a.L, a.row_adapter,
                                                        a.status);
    count_launch();
  }
  return launch_simt(a, st);
}

}  // namespace mlb
