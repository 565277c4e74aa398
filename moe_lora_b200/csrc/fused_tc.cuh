// Pieces shared by the tensor-core kernels of dense_lora_fused and moe_lora_route_scored:
// activations, cluster shared memory, and the bounded wait of the pair barriers.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace mlb {

constexpr uint64_t kFtWaitNs = 2000000000ull;  // limit of every bounded wait: 2 s

__device__ __forceinline__ float act_apply(int act, float v) {
  switch (act) {
    case ML_ACT_RELU: return v > 0.f ? v : (v != v ? v : 0.f);
    case ML_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case ML_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
      return 0.5f * v * (1.f + tanhf(u));
    }
    case ML_ACT_SILU: return silu(v);
    default: return v;
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// arrive / wait whose release and acquire reach the whole cluster: for data that one CTA's
// threads wrote to its shared memory and the leader's MMA reads there
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                                  uint64_t limit_ns, int where) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *abort_flag = 1;
      set_status(status, MOE_LORA_ERR_TIMEOUT, where);
      return false;
    }
  }
}

// ------------------------------------------------------------------ adapters of a tile
// The adapters of a token tile as extra K of the product: h = [x, z] [W; B].  A group of 64
// K columns holds 64 / r adapters (half an adapter for r = 128); a token's z stands in its
// own adapter's columns, zeros elsewhere.  Walks the groups of a 64-bit adapter mask.
struct AdapterGroups {
  uint64_t rem;
  int r, half;
  int ids[8];  // adapters of the current group (-2: none)
  int na;      // how many
  __device__ __forceinline__ AdapterGroups(uint64_t mask, int rank) : rem(mask), r(rank), half(0), na(0) {}
  __device__ __forceinline__ static int count(uint64_t mask, int r) {
    const int n = __popcll(mask);
    return r > 64 ? 2 * n : (n * r + 63) / 64;
  }
  __device__ __forceinline__ bool next() {
    if (r > 64) {
      if (half == 0) {
        if (rem == 0) return false;
        ids[0] = __ffsll(static_cast<long long>(rem)) - 1;
        rem &= rem - 1;
        na = 1;
        half = 1;
      } else {
        half = 2;
      }
      if (half == 2) {
        half = 0;
        k0 = 64;
      } else {
        k0 = 0;
      }
      return true;
    }
    if (rem == 0) return false;
    const int cap = 64 / r;
    na = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      ids[q] = -2;
      if (q < cap && rem != 0) {
        ids[q] = __ffsll(static_cast<long long>(rem)) - 1;
        rem &= rem - 1;
        na = q + 1;
      }
    }
    return true;
  }
  int k0 = 0;  // first rank row of the group's adapter (r = 128)
};

// z rows [t0, t0 + rows) as the group's K-major tile (128-byte swizzle): row of 64 K columns,
// 16-byte chunk c at c ^ (row & 7).  Thread i of n.
__device__ __forceinline__ void write_z_tile(uint8_t* dst, const AdapterGroups& g, const __nv_bfloat16* z,
                                             const int32_t* row_adapter, int t0, int rows, int T, int r, int i, int n) {
  const int per = r >= 64 ? 64 : r;
  for (int e = i; e < rows * 8; e += n) {
    const int row = e >> 3, c = e & 7;
    const int t = t0 + row;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (t < T) {
      const int ad = row_adapter[t];
      const int q = (8 * c) / per;
      int want = -2;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j == q) want = g.ids[j];
      if (ad >= 0 && ad == want)
        v = *reinterpret_cast<const uint4*>(z + static_cast<size_t>(t) * r + g.k0 + (8 * c) % per);
    }
    *reinterpret_cast<uint4*>(dst + row * 128 + ((c ^ (row & 7)) << 4)) = v;
  }
}

// Host side: launches of the tensor-core projection.
struct FusedTcArgs {
  DenseFusedArgs a;
  __nv_bfloat16* z;        // [T][r]
  uint64_t* tile_mask;     // adapters of each 128-token tile
  uint64_t* bad;           // adapters whose B holds a value that is not finite
};
cudaError_t launch_fused_shrink_tc(const FusedTcArgs& p, cudaStream_t st);
cudaError_t launch_fused_decode_tc(const FusedTcArgs& p, cudaStream_t st);
cudaError_t launch_fused_prefill_tc(const FusedTcArgs& p, cudaStream_t st);

}  // namespace mlb
