// dense_lora_fused for few tokens (T <= 256, more where there are few tiles): y = act(x W^T + bias
// + z B) + residual.
//
// Bound by the weight stream from HBM (64 x 4096 -> 2 x 11008 gated: 180 MB at 6.4 TB/s while it
// lasts, 36 us for the call; 43 us with 22 adapters of rank 16).  As in the grouped GEMM the
// weight rows fill the MMA's M (128 rows; gated: 64 gate rows and the matching 64 up rows) and
// the tokens, up to 256, its N ([SageMaker MoE kernels page], first item: the large dimension as
// the first operand), so each weight is read once per 256 tokens.  h_out / 128 tiles are too few or too uneven for 148 SMs, so a
// cluster of C CTAs splits h_in for one tile: each streams its K range, then adds up every
// C-th token's partial sums from its peers' shared memory, in rank order (the same bits
// every time), and finishes those rows: bias, activation, residual, one rounding, 8-byte
// stores of 128 neighbouring features per warp.
//
// Adapters: h = [x, z] [W; B].  The tokens' adapters follow as extra K columns (see
// AdapterGroups), B_a^T read as the MN-major A operand straight from its storage order; the
// groups are dealt out over the cluster.  They wait for the shrink kernel, which this kernel
// overlaps (programmatic dependent launch): only the adapters' part needs z.
#include "fused_tc.cuh"
#include "prof.h"

#include <algorithm>
#include <atomic>

namespace mlb {

constexpr int kFdThreads = 192;
constexpr int kFdMaxStages = 8;
// K blocks between two groups of adapters, at most, and behind the last (64 x 4096 -> 2 x 11008
// with 22 adapters: 43.1 us; 2 between 44.2, none behind 43.7)
constexpr int kGroupStep = 4, kGroupTail = 2;
constexpr int kFdPitch = 132;  // floats per token row of partial sums (128 features)

struct FdParams {
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* y;
  const __nv_bfloat16* z;
  const __nv_bfloat16* lora_b;
  const int32_t* seg_offsets;
  const int32_t* seg_adapter;
  int* status;
  int S, T, K, h_out, n, r, L, act, gated, C, stages;
};

struct FdCore {
  uint64_t full[kFdMaxStages], empty[kFdMaxStages], zgo[kFdMaxStages], zfull[kFdMaxStages], tfull, rows;
  uint32_t tmem_base;
  int abort_flag;
  alignas(8) unsigned mask[2];    // adapters of the tokens
  uint8_t list[64];               // ... in ascending order
  // ... whose B rows of this tile hold a value that is not finite, by 32 rank rows
  alignas(8) unsigned broken[2 * (128 / kGroupRank)];
  int row_ad[256];
};

template <int BN>
struct FdCfg {
  static constexpr int kStageBytes = 128 * 128 + BN * 128;
  static constexpr int kTmemCols = BN < 32 ? 32 : BN;
  static constexpr int kPart = BN * kFdPitch * 4;
};

template <int BN>
__global__ void __launch_bounds__(kFdThreads, BN <= 64 ? 4 : BN <= 128 ? 2 : 1)
    fused_decode_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx,
                        const __grid_constant__ CUtensorMap tmb, const FdParams p) {
  using Cfg = FdCfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(ring);  // [BN][kFdPitch], once the ring is idle
  __shared__ FdCore sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.stages;
  volatile int* abort_flag = &sm.abort_flag;
  const int rank = static_cast<int>(blockIdx.x) % p.C;
  const int tile = static_cast<int>(blockIdx.x) / p.C;
  // this CTA's tokens: all, or up to BN of them
  const int t0 = static_cast<int>(blockIdx.y) * BN, T = min(BN, p.T - t0);
  const __nv_bfloat16* z = p.z + static_cast<size_t>(t0) * 2 * p.r;
  const __nv_bfloat16* residual = p.residual != nullptr ? p.residual + static_cast<size_t>(t0) * p.h_out : nullptr;
  __nv_bfloat16* y = p.y + static_cast<size_t>(t0) * p.h_out;
  const int f0 = tile * (p.gated ? 64 : 128);
  const int row1 = p.gated ? p.h_out + f0 : f0 + 64;  // the tile's second 64 weight rows
  const int nkb = (p.K + 63) / 64;
  const int kb0 = static_cast<int>(static_cast<long long>(nkb) * rank / p.C);
  const int kb1 = static_cast<int>(static_cast<long long>(nkb) * (rank + 1) / p.C);

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
      mbar_init(&sm.zgo[s], 1);
      mbar_init(&sm.zfull[s], 128);
    }
    mbar_init(&sm.tfull, 1);
    mbar_init(&sm.rows, 128);
    sm.abort_flag = 0;
    sm.mask[0] = sm.mask[1] = 0u;
    for (unsigned& b : sm.broken) b = 0u;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmw);
    tma_prefetch_desc(&tmx);
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, Cfg::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (p.r == 0) {  // the call's only kernel: what ran ahead is done
    pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) p.status[0] = 0;
  }

  // how many adapters the tokens have, looked up by the epilogue warps while the stream starts
  auto adapter_count = [&]() -> int {
    if (p.r == 0 || !mbar_wait(&sm.rows, 0, abort_flag, p.status, kFtWaitNs, 57)) return 0;
    return __popc(sm.mask[0]) + __popc(sm.mask[1]);
  };
  // The adapters' K columns come one group at a time between the last K blocks: late, for the
  // shrink kernel to be done, and a few blocks apart, so that the weight stream goes on while a
  // group's z is written.  This CTA's j-th group (group rank + j C) follows K block group_at(j);
  // not before kbz, where the roles look the tokens' adapters up.
  const int kbz = kb0 + (kb1 - kb0) / 4;
  int groups = 0, step = 1;
  auto deal = [&](const AdapterGroups& g, int cnt) {
    if (cnt > 0) groups = (g.count(cnt) + p.C - 1 - rank) / p.C;
    if (groups > 0) step = min(kGroupStep, (kb1 - kbz) / groups);
  };
  auto group_at = [&](int j) -> int { return max(kbz, kb1 - 1 - kGroupTail - step * (groups - 1 - j)); };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, parity_of = 0;
      bool ok = true;
      auto advance = [&]() {
        filled |= 1u << stage;
        parity_of = (parity_of & ~(1u << stage)) | (phase << stage);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      };
      AdapterGroups g(0ull, p.r);
      int j = 0, cnt = 0;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        ok = mbar_wait(&sm.empty[stage], phase ^ 1u, abort_flag, p.status, kFtWaitNs, 50);
        if (!ok) break;
        uint8_t* s = ring + stage * Cfg::kStageBytes;
        mbar_arrive_expect_tx(&sm.full[stage], Cfg::kStageBytes);
        tma_load_2d(s, &tmw, &sm.full[stage], kb * 64, f0);
        tma_load_2d(s + 64 * 128, &tmw, &sm.full[stage], kb * 64, row1);
        tma_load_2d(s + 128 * 128, &tmx, &sm.full[stage], kb * 64, t0);
        advance();
        if (kb < kbz) continue;
        if (kb == kbz) {
          cnt = adapter_count();
          deal(g, cnt);
        }
        for (; ok && j < groups && group_at(j) == kb; ++j) {
          g.pick(sm.list, cnt, rank + j * p.C);
          ok = mbar_wait(&sm.empty[stage], phase ^ 1u, abort_flag, p.status, kFtWaitNs, 51);
          if (!ok) break;
          mbar_arrive(&sm.zgo[stage]);  // the z tile may be written
          uint8_t* zs = ring + stage * Cfg::kStageBytes;
          const int rb = g.box_rows(), boxes = g.boxes();
          mbar_arrive_expect_tx(&sm.full[stage], static_cast<uint32_t>(2 * boxes * rb) * 128u);
#pragma unroll
          for (int q = 0; q < kGroupRank / 8; ++q) {
            if (q >= boxes) break;
            const int id = (q > 0 && q >= g.na) ? g.ids[q > 0 ? q - 1 : 0] : g.ids[q];
            tma_load_2d(zs + q * rb * 128, &tmb, &sm.full[stage], f0, id * p.r + g.k0);
            tma_load_2d(zs + 64 * 128 + q * rb * 128, &tmb, &sm.full[stage], row1, id * p.r + g.k0);
          }
          advance();
        }
      }
      if (*abort_flag)  // let our own copies land before the ring is reused
        for (int s = 0; s < S; ++s)
          if (filled & (1u << s)) {
            volatile int dummy = 0;
            mbar_wait(&sm.full[s], (parity_of >> s) & 1u, &dummy, nullptr, kFtWaitNs / 4, 0);
          }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, zi = 0;
      bool ok = true;
      const int n_mma = min(BN, (T + 15) & ~15);
      const uint32_t idesc = umma_idesc_bf16(128, n_mma);
      auto advance = [&]() {
        umma_commit(&sm.empty[stage]);
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      };
      const uint32_t zdesc = umma_idesc_bf16_amn(128, n_mma);
      AdapterGroups g(0ull, p.r);
      int j = 0, cnt = 0;
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        ok = mbar_wait(&sm.full[stage], phase, abort_flag, p.status, kFtWaitNs, 52);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s = smem_u32(ring + stage * Cfg::kStageBytes);
        const uint64_t ad = umma_desc_sw128(s), bd = umma_desc_sw128(s + 128 * 128);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
        advance();
        if (kb < kbz) continue;
        if (kb == kbz) {
          cnt = adapter_count();
          deal(g, cnt);
        }
        // adapters: A = B_a^T, MN-major (64-feature blocks 8 KB apart), 16 rank rows per two steps
        for (; ok && j < groups && group_at(j) == kb; ++j) {
          g.pick(sm.list, cnt, rank + j * p.C);
          ok = mbar_wait(&sm.full[stage], phase, abort_flag, p.status, kFtWaitNs, 53) &&
               mbar_wait(&sm.zfull[stage], static_cast<uint32_t>(zi >> stage) & 1u, abort_flag, p.status, kFtWaitNs, 54);
          if (!ok) break;
          tc_fence_after();
          const uint32_t zs = smem_u32(ring + stage * Cfg::kStageBytes);
          const uint64_t zad = umma_desc_mn_sw128(zs, 64 * 128), zbd = umma_desc_sw128(zs + 128 * 128);
          const int steps = g.steps();
          for (int k = 0; k < steps; ++k) umma_bf16(tmem, zad + 128 * (k >> 1), zbd + 2 * k, zdesc, 1u);
          zi ^= 1u << stage;  // parity of the stage's uses for adapters
          advance();
        }
      }
      umma_commit(&sm.tfull);
      volatile int dummy = 0;
      mbar_wait(&sm.tfull, 0, &dummy, nullptr, kFtWaitNs, 0);  // the MMAs are done with the ring
    }
    __syncwarp();
  } else {
    // the tokens' adapters, z tiles of this CTA's groups, then the accumulator -> partial sums
    const int e = tid - 64;
    if (p.r) {
      for (int t = e; t < BN; t += 128) {
        int a = -1;
        if (t < T) {
          const int s = segment_of(p.seg_offsets, p.S, t0 + t);
          if (s >= 0) a = p.seg_adapter[s];
          if (a < 0 || a >= p.L) a = -1;
          if (a >= 0) atomicOr(&sm.mask[a >> 5], 1u << (a & 31));
        }
        sm.row_ad[t] = a;
      }
      __syncwarp();
      named_bar_sync(1, 128);
      {
        const uint64_t mask = sm.mask[0] | (static_cast<uint64_t>(sm.mask[1]) << 32);
        if (e < 64 && (mask >> e & 1ull)) sm.list[__popcll(mask & ((1ull << e) - 1ull))] = static_cast<uint8_t>(e);
      }
      mbar_arrive(&sm.rows);
      AdapterGroups g(0ull, p.r);
      const int cnt = adapter_count();
      deal(g, cnt);
      uint32_t zi = 0;
      ZTile<128, BN / 16> zt;
      zt.rows(sm.row_ad, 0, BN, e);
      bool ok = true;
      if (groups > 0) pdl_wait();  // z comes from the shrink kernel
      for (int j = 0; ok && j < groups; ++j) {
        const int at = group_at(j) + 1 - kb0 + j;  // ring stages ahead of this one
        const int stage = at % S;
        const uint32_t lap = static_cast<uint32_t>(at / S) & 1u;
        g.pick(sm.list, cnt, rank + j * p.C);
        zt.load(g, z, 0, p.r, e);
        // (after zgo the barrier `full` is in this lap's phase)
        ok = mbar_wait(&sm.zgo[stage], zi >> stage & 1u, abort_flag, p.status, kFtWaitNs, 55) &&
             mbar_wait(&sm.full[stage], lap, abort_flag, p.status, kFtWaitNs, 58);
        __syncwarp();
        if (!named_bar_and(1, 128, ok)) {
          ok = false;
          break;
        }
        zi ^= 1u << stage;
        uint8_t* zs = ring + stage * Cfg::kStageBytes;
        zt.store(zs + 128 * 128, e);
        // B rows that are not finite would reach every token through its zeros: their adapter
        // leaves the product, the final rows add it for its own tokens alone
        const int per = g.box_rows(), used = g.boxes() * per * 8;  // 16-byte chunks of a block
        unsigned* broken = sm.broken + 2 * (g.k0 / kGroupRank);
        uint32_t hit = 0u;  // adapters of the group
        for (int c = e; c < used; c += 128) {
          const uint4* b = reinterpret_cast<const uint4*>(zs) + c;
          if (not_finite8(b[0]) || not_finite8(b[512])) hit |= 1u << min(c / 8 / per, g.na - 1);
        }
        hit = __reduce_or_sync(0xffffffffu, hit);
        if (!named_bar_and(1, 128, hit == 0u)) {
          if (hit != 0u && lane == 0) {
#pragma unroll
            for (int q = 0; q < kGroupRank / 8; ++q)
              if (hit >> q & 1u) atomicOr(&broken[g.ids[q] >> 5], 1u << (g.ids[q] & 31));
          }
          __syncwarp();
          named_bar_sync(1, 128);
          for (int c = e; c < used; c += 128) {
            const int q = min(c / 8 / per, g.na - 1);
            int id = 0;
#pragma unroll
            for (int j = 0; j < kGroupRank / 8; ++j)
              if (j == q) id = g.ids[j];
            if (broken[id >> 5] >> (id & 31) & 1u) {
              uint4* b = reinterpret_cast<uint4*>(zs) + c;
              b[0] = b[512] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&sm.zfull[stage]);
      }
    }
    bool got = mbar_wait(&sm.tfull, 0, abort_flag, p.status, kFtWaitNs, 56);
    __syncwarp();
    got = named_bar_and(1, 128, got);
    if (got) {
      tc_fence_after();
      const int g4 = warp & 3, m = g4 * 32 + lane;
      for (int c0 = 0; c0 < T; c0 += 32) {
        float v[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(g4 * 32) << 16) + c0, v);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (c0 + j < BN) part[(c0 + j) * kFdPitch + m] = v[j];
      }
      tc_fence_before();
    }
  }
  __syncwarp();
  cluster_sync_all();

  // tokens rank, rank + C, ...: a warp per token, 4 features per lane (gated: lanes 0-15 the
  // gate's 64 features, lanes 16-31 the up projection's)
  pdl_trigger();  // a call behind this one may set itself up
  if (p.r) pdl_wait();  // the call ends behind the shrink kernel, whatever the tokens need of it
  if (!*abort_flag) {
    const int col = p.gated ? ((lane < 16 ? 0 : p.h_out) + f0 + 4 * (lane & 15)) : f0 + 4 * lane;  // row of W
    const int feat = p.gated ? f0 + 4 * (lane & 15) : col;
    const bool in = feat < p.h_out;
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias != nullptr && in) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p.bias + col));
      b[0] = __uint_as_float(v.x << 16);
      b[1] = __uint_as_float(v.x & 0xFFFF0000u);
      b[2] = __uint_as_float(v.y << 16);
      b[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    // the tile's broken adapters, whichever CTA met them: a lane per CTA and 32 rank rows asks
    auto broken_at = [&](int i, int c) -> uint64_t {
      return ld_cluster_u64(mapa_shared(smem_u32(sm.broken + 2 * i), static_cast<uint32_t>(c)));
    };
    static_assert(8 * (128 / kGroupRank) <= 32, "eight CTAs' words for a warp");
    const int parts = (p.r + kGroupRank - 1) / kGroupRank;
    uint64_t bad = lane < p.C * parts ? broken_at(lane / p.C, lane % p.C) : 0ull;
    bad = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad)) |
          static_cast<uint64_t>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(bad >> 32))) << 32;
    // the next token's partial sums are on their way while one is finished
    const int t_step = p.C * (kFdThreads / 32);
    const bool writer = in && (!p.gated || lane < 16);
    float4 v[8];
    uint2 res_next = make_uint2(0u, 0u);
    auto fetch = [&](int t) {
      if (t >= T) return;
      const uint32_t at = smem_u32(part + t * kFdPitch + 4 * lane);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < p.C) v[c] = ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(c)));
      if (residual != nullptr && writer)
        res_next = *reinterpret_cast<const uint2*>(residual + static_cast<size_t>(t) * p.h_out + feat);
    };
    fetch(rank + p.C * warp);
    for (int t = rank + p.C * warp; t < T; t += t_step) {
      float h[4] = {b[0], b[1], b[2], b[3]};
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < p.C) {
          h[0] += v[c].x;
          h[1] += v[c].y;
          h[2] += v[c].z;
          h[3] += v[c].w;
        }
      const uint2 res = res_next;
      fetch(t + t_step);
      if (bad != 0) {  // an adapter with values that are not finite: its own tokens only
        const int ad = sm.row_ad[t];
        if (ad >= 0 && (bad >> ad & 1ull) && in)
          for (int i0 = 0; i0 < p.r; i0 += kGroupRank) {
            bool out = false;  // (else those rows are in the product)
            for (int c = 0; c < p.C; ++c) out |= broken_at(i0 / kGroupRank, c) >> ad & 1ull;
            if (!out) continue;
            for (int i = i0; i < min(i0 + kGroupRank, p.r); ++i) {
              const float zi = z_value(z, t, p.r, i);
              const __nv_bfloat16* br = p.lora_b + (static_cast<size_t>(ad) * p.r + i) * p.n + col;
#pragma unroll
              for (int j = 0; j < 4; ++j) h[j] = fmaf(zi, __bfloat162float(br[j]), h[j]);
            }
          }
      }
      if (p.gated) {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = sigmoid_of<true>(h[j], h[j]) * __shfl_down_sync(0xffffffffu, h[j], 16);
      } else {
        act_apply<true>(p.act, h);
      }
      h[0] += __uint_as_float(res.x << 16);
      h[1] += __uint_as_float(res.x & 0xFFFF0000u);
      h[2] += __uint_as_float(res.y << 16);
      h[3] += __uint_as_float(res.y & 0xFFFF0000u);
      if (writer)
        *reinterpret_cast<uint2*>(y + static_cast<size_t>(t) * p.h_out + feat) =
            make_uint2(pack2_bf16(h[0], h[1]), pack2_bf16(h[2], h[3]));
    }
  }
  __syncwarp();
  cluster_sync_all();  // the peers have read this CTA's partial sums
  if (warp == 1) tmem_dealloc(tmem, Cfg::kTmemCols);
}

static int weight_tiles(const DenseFusedArgs& a) {
  return a.act == ML_ACT_SILU_AND_MUL ? (a.h_out + 63) / 64 : (a.h_out + 127) / 128;
}

// Splitting h_in pays against 256 x 256 tiles when it takes more K blocks off each CTA than the
// exchange of partial sums costs: 300 x 2048 -> 1024 12.6 against 15.7 us (16 tiles of 128 rows x
// 256 tokens, 8 splits), 512 x 4096 -> 4096 25.8 against 26.0 (64 tiles, 2), with 16 adapters of
// rank 16 42 against 51, 400 x 11008 -> 1000 31 against 60; but 700 x 600 -> 2000 23.1 against 15.5
// (48 tiles, 3 splits of 10 K blocks).
bool fused_decode_pays(const DenseFusedArgs& a) {
  const long long tiles = static_cast<long long>(weight_tiles(a)) * ((a.T + 255) / 256);
  const long long splits = std::min<long long>(8, a.num_sms / tiles), nkb = (a.h_in + 63) / 64;
  return nkb * (splits - 1) >= 48;
}

template <int BN>
static cudaError_t launch_bn(const FusedTcArgs& f, cudaStream_t st) {
  using Cfg = FdCfg<BN>;
  const DenseFusedArgs& a = f.a;
  CUtensorMap tmw, tmx, tmb;
  if (encode_tmap_2d(&tmw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w, a.h_in, a.n, static_cast<uint64_t>(a.h_in) * 2, 64,
                     64, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tmap_2d(&tmx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.h_in, a.T, static_cast<uint64_t>(a.h_in) * 2, 64,
                     BN, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  tmb = tmx;
  if (a.r && encode_tmap_2d(&tmb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.lora_b, a.n, static_cast<uint64_t>(a.L) * a.r,
                            static_cast<uint64_t>(a.n) * 2, 64, std::min(a.r, kGroupRank),
                            CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  FdParams p{};
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.residual = static_cast<const __nv_bfloat16*>(a.residual);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.z = f.z;
  p.lora_b = static_cast<const __nv_bfloat16*>(a.lora_b);
  p.seg_offsets = a.seg_offsets;
  p.seg_adapter = a.seg_adapter;
  p.S = a.S;
  p.L = a.L;
  p.status = a.status;
  p.T = a.T;
  p.K = a.h_in;
  p.h_out = a.h_out;
  p.n = a.n;
  p.r = a.r;
  p.act = a.act;
  p.gated = a.act == ML_ACT_SILU_AND_MUL;
  const int wtiles = weight_tiles(a), ttiles = (a.T + BN - 1) / BN, tiles = wtiles * ttiles;
  // CTAs per SM and K splits.  As many splits as keep one wave (a second wave starts its stream
  // anew) and two K blocks per split: 1, 2, 4 and 8 splits take 73, 40, 24 and 22 us for 64 x
  // 11008 -> 4096 (32 tiles), 28, 19.5, 19.3 and 19.3 for one token 4096 -> 11008 (86 tiles, 3 at
  // most), 36, 21, 14 and 12 for 203 x 2056 -> 1000 (8 tiles);
  // of two or three CTAs per SM (one above 128 tokens) what has more of the ring in use (172
  // tiles: 42 us as 172 CTAs of two per SM, 36 as 344 of three).
  const int nkb = (a.h_in + 63) / 64, most = BN <= 64 ? 3 : BN <= 128 ? 2 : 1;
  long long in_use = -1;
  size_t smem = 0;
  for (int per_sm = BN <= 128 ? 2 : 1; per_sm <= most; ++per_sm) {
    const int budget = per_sm == 3 ? 72 * 1024 : per_sm == 2 ? 108 * 1024 : 200 * 1024;
    const int C = std::max(1, std::min(std::min(8, per_sm * a.num_sms / tiles), nkb / 2));
    const int stages = std::min(kFdMaxStages, budget / Cfg::kStageBytes);
    const long long bytes = std::min(tiles * C, per_sm * a.num_sms) * static_cast<long long>(stages);
    if (tiles * C > per_sm * a.num_sms && in_use >= 0) continue;
    if (bytes > in_use + in_use / 8) {
      in_use = bytes;
      p.C = C;
      p.stages = stages;
      smem = 1024 + std::max(stages * Cfg::kStageBytes, Cfg::kPart);
    }
  }
  static std::atomic<bool> attr_set[kMaxDevices];
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(fused_decode_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               1024 + (BN <= 128 ? 108 : 200) * 1024);
    if (e != cudaSuccess) return e;
    const cudaError_t c = cudaFuncSetAttribute(fused_decode_kernel<BN>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                               cudaSharedmemCarveoutMaxShared);
    if (c != cudaSuccess) return c;
    attr_set[dev].store(true, std::memory_order_release);
  }
  ProfScope ps(K_DENSE_FUSED, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(wtiles * p.C, ttiles);
  cfg.blockDim = dim3(kFdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fused_decode_kernel<BN>, tmw, tmx, tmb, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_fused_decode_tc(const FusedTcArgs& f, cudaStream_t st) {
  const int T = f.a.T;
  if (T <= 16) return launch_bn<16>(f, st);
  if (T <= 32) return launch_bn<32>(f, st);
  if (T <= 64) return launch_bn<64>(f, st);
  if (T <= 128) return launch_bn<128>(f, st);
  return launch_bn<256>(f, st);
}

}  // namespace mlb
