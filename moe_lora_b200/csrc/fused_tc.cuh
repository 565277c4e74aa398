// Pieces shared by the tensor-core kernels of dense_lora_fused and moe_lora_route_scored:
// activations, cluster shared memory, and the bounded wait of the pair barriers.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace mlb {

constexpr uint64_t kFtWaitNs = 2000000000ull;  // limit of every bounded wait: 2 s

// Activations behind a projection.  The exponential's argument is at most 0, so that nothing
// overflows at either end.  Fp32 outputs take expf and an IEEE division; bf16 outputs (FAST),
// rounded to 2^-9 behind them, __expf (off by 2 + 1.2 |x| units of the last place) and
// __fdividef (2 units: the divisor lies in [1, 2]).  30000 x 512 -> 1024, bound by this epilogue,
// takes 122 us so and 130 with expf.
template <bool FAST>
__device__ __forceinline__ float sigmoid_of(float x, float v) {  // v / (1 + exp(-x))
  const float t = FAST ? __expf(-fabsf(x)) : expf(-fabsf(x)), n = x < 0.f ? v * t : v;
  if constexpr (FAST) return __fdividef(n, 1.f + t);
  return n / (1.f + t);
}

template <bool FAST, int N>
__device__ __forceinline__ void act_apply(int act, float (&h)[N]) {
  switch (act) {
    case ML_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) h[j] = h[j] > 0.f ? h[j] : (h[j] != h[j] ? h[j] : 0.f);
      break;
    case ML_ACT_GELU:
#pragma unroll
      for (int j = 0; j < N; ++j) h[j] = 0.5f * h[j] * (1.f + erff(h[j] * 0.70710678118654752f));
      break;
    case ML_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
#pragma unroll
      for (int j = 0; j < N; ++j)
        h[j] = sigmoid_of<FAST>(1.5957691216057308f * (h[j] + 0.044715f * h[j] * h[j] * h[j]), h[j]);
      break;
    case ML_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) h[j] = sigmoid_of<FAST>(h[j], h[j]);
      break;
    default: break;
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

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t cluster_addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// ------------------------------------------------------------------ adapters of a tile
// The adapters of a token tile as extra K of the product: h = [x, z] [W; B].  z = c x A is an fp32
// sum, given to the product as two bf16 numbers, the rounded value and what it left (2^-17 of z is
// lost; one bf16 would lose 2^-9, as much as the rounding of the output).  A group of 64 K columns
// covers 32 rank columns: 32 / r adapters, or 32 of one adapter's ranks.  Each 16 rank columns take
// 32 of K, values first, then remainders, both against the same 16 rows of B.  A token's z stands
// in its own adapter's columns, zeros elsewhere.
constexpr int kGroupRank = 32;

struct AdapterGroups {
  uint64_t rem;  // next(): adapters still to come
  int r, part = 0;
  int k0 = 0;   // first rank row of the group's adapter (r > 32)
  int ids[kGroupRank / 8];  // adapters of the current group (-2: none)
  int na = 0;   // how many
  __device__ __forceinline__ AdapterGroups(uint64_t mask, int rank) : rem(mask), r(rank) {}
  // groups of `cnt` adapters
  __device__ __forceinline__ int count(int cnt) const {
    return r > kGroupRank ? cnt * (r / kGroupRank) : (cnt + kGroupRank / r - 1) / (kGroupRank / r);
  }
  // rank rows per box of B
  __device__ __forceinline__ int box_rows() const { return min(r, kGroupRank); }
  // B boxes per 64 features: an odd adapter of rank 8 fills half an MMA step, so its rows come
  // once more and meet zeros of z
  __device__ __forceinline__ int boxes() const { return (r == 8 && (na & 1)) ? na + 1 : na; }
  // MMA steps of 16 K columns; step s takes rows 16 (s / 2) of B
  __device__ __forceinline__ int steps() const { return r > kGroupRank ? 4 : 2 * ((na * r + 15) / 16); }
  // group gi of the `cnt` adapters in `list`, in ascending order
  __device__ __forceinline__ void pick(const uint8_t* list, int cnt, int gi) {
    if (r > kGroupRank) {
      const int parts = r / kGroupRank;
      ids[0] = list[gi / parts];
      na = 1;
      k0 = gi % parts * kGroupRank;
      return;
    }
    const int cap = kGroupRank / r;
    na = min(cap, cnt - gi * cap);
#pragma unroll
    for (int q = 0; q < kGroupRank / 8; ++q) ids[q] = q < na ? list[gi * cap + q] : -2;
  }
  // the next group of the adapters in the mask
  __device__ __forceinline__ bool next() {
    if (r > kGroupRank) {
      if (part == 0) {
        if (rem == 0) return false;
        ids[0] = __ffsll(static_cast<long long>(rem)) - 1;
        rem &= rem - 1;
        na = 1;
      }
      k0 = part * kGroupRank;
      if (++part == r / kGroupRank) part = 0;
      return true;
    }
    if (rem == 0) return false;
    const int cap = kGroupRank / r;
    na = 0;
#pragma unroll
    for (int q = 0; q < kGroupRank / 8; ++q) {
      ids[q] = -2;
      if (q < cap && rem != 0) {
        ids[q] = __ffsll(static_cast<long long>(rem)) - 1;
        rem &= rem - 1;
        na = q + 1;
      }
    }
    return true;
  }
};

// Two values of z as pairs of bf16 numbers: rounded, and the remainders (0 where there is none:
// an infinity or NaN)
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2_bf16(a, b);
  const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xFFFF0000u);
  lo = pack2_bf16(fabsf(ra) < INFINITY ? ra : 0.f, fabsf(rb) < INFINITY ? rb : 0.f);
}

// Token t's segment: the last one that begins at or before it, if it ends behind it (-1: none).
// Every kernel of a call asks here, so that they agree even on segments out of order.
__device__ __forceinline__ int segment_of(const int32_t* off, int S, int t) {
  int lo = 0, hi = S;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid;
    else hi = mid;
  }
  return (off[lo] <= t && t < off[lo + 1]) ? lo : -1;
}

__device__ __forceinline__ bool segment_wrong(int lo, int hi, int a, int T, int L) {
  return lo > hi || lo < 0 || hi > T || a < -1 || a >= L;
}

// true if a bf16 of the eight is an infinity or NaN (exponent bits all ones)
__device__ __forceinline__ bool not_finite8(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  bool hit = false;
#pragma unroll
  for (int j = 0; j < 4; ++j) hit |= (w[j] & 0x7F80u) == 0x7F80u || (w[j] & 0x7F800000u) == 0x7F800000u;
  return hit;
}

// z rows [t0, t0 + N NT / 8) as a group's K-major tile (128-byte swizzle): a row
// holds 64 K columns, its 16-byte chunk c at c ^ (row & 7).  Thread i of NT takes chunk i & 7
// of rows i / 8 + j NT / 8, j < N: the rows' adapters once per tile, the z values ahead of
// the stage that takes them, so that only the shared-memory stores wait for it.
// z: [tokens][2][r], values and remainders.
template <int NT, int N>
struct ZTile {
  int ad[N];
  uint4 v[N];
  __device__ __forceinline__ void rows(const int32_t* row_adapter, int t0, int T, int i) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int t = t0 + (i >> 3) + j * (NT / 8);
      ad[j] = t < T ? row_adapter[t] : -1;
    }
  }
  __device__ __forceinline__ void load(const AdapterGroups& g, const __nv_bfloat16* z, int t0, int r, int i) {
    // chunk: 8 rank columns k, ..., their values (chunks 0, 1, 4, 5) or remainders
    const int k = (i & 4) * 4 + (i & 1) * 8, per = g.box_rows(), q = k / per;
    int want = -2;
#pragma unroll
    for (int e = 0; e < kGroupRank / 8; ++e)
      if (e == q) want = g.ids[e];
    const __nv_bfloat16* zp =
        z + static_cast<size_t>(t0 + (i >> 3)) * 2 * r + ((i & 2) ? r : 0) + g.k0 + k - q * per;
#pragma unroll
    for (int j = 0; j < N; ++j)
      v[j] = (ad[j] >= 0 && ad[j] == want)
                 ? *reinterpret_cast<const uint4*>(zp + static_cast<size_t>(j) * (NT / 8) * 2 * r)
                 : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void store(uint8_t* dst, int i) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int row = (i >> 3) + j * (NT / 8);
      *reinterpret_cast<uint4*>(dst + row * 128 + (((i & 7) ^ (row & 7)) << 4)) = v[j];
    }
  }
};

// a z value of the pair
__device__ __forceinline__ float z_value(const __nv_bfloat16* z, size_t t, int r, int i) {
  const __nv_bfloat16* at = z + t * 2 * r + i;
  return __bfloat162float(at[0]) + __bfloat162float(at[r]);
}

// Host side: launches of the tensor-core projection.
struct FusedTcArgs {
  DenseFusedArgs a;
  __nv_bfloat16* z;        // [T][2][r]: values and remainders
  __nv_bfloat16* zc;       // K columns of each 256-token tile's groups (see AdapterGroups): [a band][zc_pitch]
  int zc_pitch;
  uint64_t* tile_mask;     // ... those adapters
  uint64_t* bad_part;      // adapters whose B holds a value that is not finite, by CTA of the scan
  int scan_ctas;
};
cudaError_t launch_fused_shrink_simt(const FusedTcArgs& p, cudaStream_t st);
// the shrink on CUDA cores is two CTAs per SM at most
bool fused_shrink_is_small(const DenseFusedArgs& a);
// Tokens [t0, t1), t0 a multiple of 256.  operand: what launch_fused_prefill_tc asks for as well
// (zc, the masks; with the first tokens the scan)
cudaError_t launch_fused_shrink_tc(const FusedTcArgs& p, bool operand, int t0, int t1, cudaStream_t st);
cudaError_t launch_fused_decode_tc(const FusedTcArgs& p, cudaStream_t st);
// above kFusedDecodeTokens: few tiles, so that splitting h_in pays more than larger tiles
bool fused_decode_pays(const DenseFusedArgs& a);
cudaError_t launch_fused_prefill_tc(const FusedTcArgs& p, int t0, int t1, cudaStream_t st);

}  // namespace mlb
