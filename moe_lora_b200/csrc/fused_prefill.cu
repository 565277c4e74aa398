// dense_lora_fused for many tokens: y = act(x W^T + bias + z B) + residual.
//
// Bound by the tensor pipe under the power cap (4096 x 4096 -> 11008: 260 us without adapters,
// 1.42 PFLOP/s over the call; 310 us with 16 of rank 64).  CTA pairs (tcgen05 cta_group::2, M = 256) compute tiles of 256
// tokens x 256 weight rows (gated: 128 gate rows and the matching 128 up rows): tokens in M,
// so that a thread of the epilogue holds one token's neighbouring features and bias,
// activation, residual and store work on whole 16-byte runs.  Each CTA stages its 128 tokens
// and half of the weight rows, 32 KB per 64 of h_in, six stages; two accumulators of 256
// columns fill TMEM, so the eight epilogue warps finish one tile under the next one's MMAs.
// Tiles are walked token tile by token tile for each strip of weight rows, so that the pairs
// in flight share the strip in L2.
//
// Adapters: h = [x, z] [W; B], the tokens' adapters as extra K columns (see AdapterGroups)
// behind each tile's K loop: the A operand is the tile's z as the shrink kernel laid it out
// (zero in other adapters' columns), the B operand B_a as stored (MN-major).  A role's first
// tile waits for the shrink kernel there (programmatic dependent launch).
#include "fused_tc.cuh"
#include "prof.h"

#include <algorithm>
#include <atomic>

namespace mlb {

constexpr int kFpThreads = 320;  // producer, MMA, 8 epilogue warps
constexpr int kFpStages = 6;
constexpr int kFpStageBytes = 2 * 128 * 128;
constexpr int kFpEpiWarps = 8;
constexpr int kFpBand = 16;  // token tiles per band

struct FpParams {
  const __nv_bfloat16* bias;
  const __nv_bfloat16* residual;
  __nv_bfloat16* y;
  const __nv_bfloat16* z;
  const __nv_bfloat16* lora_b;
  const int32_t* row_adapter;
  const uint64_t* tile_mask;
  const uint64_t* bad_part;
  int* status;
  int t_first, T;  // this launch's tokens: [t_first, T)
  int K, h_out, n, r, L, act, gated, scan_ctas;
  int tok_tiles, feat_tiles;
};

struct FpCore {
  uint64_t full[kFpStages], empty[kFpStages], tfull[2], tempty[2], tdone, scanned;
  uint64_t bad;  // adapters whose B holds a value that is not finite
  uint32_t tmem_base;
  int abort_flag;
};

// tile index -> (token tile, feature tile): bands of kFpBand token tiles, inside a band the
// token tiles of one feature tile follow each other
__device__ __forceinline__ void fp_tile(const FpParams& p, int t, int& tt, int& ft) {
  const int per_band = kFpBand * p.feat_tiles;
  const int band = t / per_band, in = t - band * per_band;
  const int width = min(kFpBand, p.tok_tiles - band * kFpBand);
  ft = in / width;
  tt = band * kFpBand + in - ft * width;
}

__global__ void __launch_bounds__(kFpThreads, 1)
    fused_prefill_kernel(const __grid_constant__ CUtensorMap tmw, const __grid_constant__ CUtensorMap tmx,
                         const __grid_constant__ CUtensorMap tmb, const __grid_constant__ CUtensorMap tmz,
                         const FpParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ FpCore sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sm.abort_flag;
  const uint32_t rank = cluster_ctarank();
  auto leader = [&](uint64_t* bar) -> uint32_t { return mapa_shared(smem_u32(bar), 0); };
  const int total = p.tok_tiles * p.feat_tiles;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int nk = (p.K + 63) / 64;

  if (tid == 0) {
    for (int s = 0; s < kFpStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.tfull[b], 1);
      mbar_init(&sm.tempty[b], 2 * kFpEpiWarps);
    }
    mbar_init(&sm.tdone, 1);
    mbar_init(&sm.scanned, 1);
    sm.abort_flag = 0;
    fence_mbarrier_init();
    tma_prefetch_desc(&tmw);
    tma_prefetch_desc(&tmx);
  }
  if (warp == 1) tmem_alloc_pair(&sm.tmem_base, 512);
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  if (p.r == 0) {  // the call's only kernel: what ran ahead is done
    pdl_wait();
    if (blockIdx.x == 0 && tid == 0) p.status[0] = 0;
  }

  // Adapters of a 256-token tile; every role that asks has waited for the kernels ahead.  From a
  // role's second tile on it asks ahead of the K loop, behind which the mask is needed.
  auto adapter_mask = [&](int tt) -> uint64_t {
    return p.r == 0 ? 0ull : *reinterpret_cast<const volatile uint64_t*>(p.tile_mask + tt);
  };

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, parity_of = 0;
      bool ok = true;
      auto advance = [&]() {
        filled |= 1u << stage;
        parity_of = (parity_of & ~(1u << stage)) | (phase << stage);
        if (++stage == kFpStages) {
          stage = 0;
          phase ^= 1u;
        }
      };
      for (int t = pair; ok && t < total; t += pairs) {
        int tt, ft;
        fp_tile(p, t, tt, ft);
        const int z0 = tt * 256 + static_cast<int>(rank) * 128, t0 = p.t_first + z0;
        const int wrow = p.gated ? static_cast<int>(rank) * p.h_out + ft * 128 : ft * 256 + static_cast<int>(rank) * 128;
        uint64_t mask = t != pair ? adapter_mask(tt) : 0ull;
        for (int kb = 0; kb < nk; ++kb) {
          ok = mbar_wait(&sm.empty[stage], phase ^ 1u, abort_flag, p.status, kFtWaitNs, 60);
          if (!ok) break;
          uint8_t* s = ring + stage * kFpStageBytes;
          const uint32_t fb = leader(&sm.full[stage]);
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[stage], 2u * kFpStageBytes);
          tma_load_2d_pair(s, &tmx, fb, kb * 64, t0);
          tma_load_2d_pair(s + 128 * 128, &tmw, fb, kb * 64, wrow);
          advance();
        }
        if (!ok || p.r == 0) continue;
        if (t == pair) {
          pdl_wait();
          mask = adapter_mask(tt);
          ok = mbar_wait(&sm.scanned, 0, abort_flag, p.status, kFtWaitNs, 65);
        }
        // An adapter that is not finite stays out of the product: its rows come from behind the
        // tensor, where they are zero, and the epilogue adds it for its own tokens.
        const uint64_t bad = sm.bad;
        AdapterGroups g(mask, p.r);
        for (int gi = 0; ok && g.next(); ++gi) {
          ok = mbar_wait(&sm.empty[stage], phase ^ 1u, abort_flag, p.status, kFtWaitNs, 61);
          if (!ok) break;
          uint8_t* s = ring + stage * kFpStageBytes;
          const uint32_t fb = leader(&sm.full[stage]);
          const int rb = g.box_rows(), boxes = g.boxes();
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[stage], 2u * 128u * 128u + static_cast<uint32_t>(4 * boxes * rb) * 128u);
          tma_load_2d_pair(s, &tmz, fb, gi * 64, z0);
          s += 128 * 128;
#pragma unroll
          for (int q = 0; q < kGroupRank / 8; ++q) {
            if (q >= boxes) break;
            const int id = (q > 0 && q >= g.na) ? g.ids[q > 0 ? q - 1 : 0] : g.ids[q];
            const int row = bad >> id & 1ull ? p.L * p.r : id * p.r + g.k0;
            tma_load_2d_pair(s + q * rb * 128, &tmb, fb, wrow, row);
            tma_load_2d_pair(s + 64 * 128 + q * rb * 128, &tmb, fb, wrow + 64, row);
          }
          advance();
        }
      }
      if (*abort_flag) {
        // let our own copies land before the CTA exits (the peer's complete on the leader's
        // barriers, so the peer gives them a fixed 50 us)
        if (rank != 0) {
          const uint64_t c0 = globaltimer_ns();
          while (globaltimer_ns() - c0 < 50000ull) {
          }
        } else {
          for (int s = 0; s < kFpStages; ++s)
            if (filled & (1u << s)) {
              volatile int dummy = 0;
              mbar_wait(&sm.full[s], (parity_of >> s) & 1u, &dummy, nullptr, kFtWaitNs / 4, 0);
            }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      int stage = 0, it = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto advance = [&]() {
        umma_commit_pair(&sm.empty[stage], 3);
        if (++stage == kFpStages) {
          stage = 0;
          phase ^= 1u;
        }
      };
      const uint32_t idesc = umma_idesc_bf16(256, 256);
      const uint32_t zidesc = idesc | (1u << 16);  // B operand MN-major
      for (int t = pair; ok && t < total; t += pairs, ++it) {
        int tt, ft;
        fp_tile(p, t, tt, ft);
        const int buf = it & 1;
        const uint32_t d = tmem + buf * 256;
        uint64_t mask = it != 0 ? adapter_mask(tt) : 0ull;
        ok = mbar_wait(&sm.tempty[buf], (static_cast<uint32_t>(it >> 1) & 1u) ^ 1u, abort_flag, p.status, kFtWaitNs, 62);
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < nk; ++kb) {
          ok = mbar_wait(&sm.full[stage], phase, abort_flag, p.status, kFtWaitNs, 63);
          if (!ok) break;
          tc_fence_after();
          const uint32_t s = smem_u32(ring + stage * kFpStageBytes);
          const uint64_t ad = umma_desc_sw128(s), bd = umma_desc_sw128(s + 128 * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16_pair(d, ad + 2 * k, bd + 2 * k, idesc, (kb != 0 || k != 0) ? 1u : 0u);
          advance();
        }
        if (ok && p.r) {
          if (it == 0) {
            pdl_wait();
            mask = adapter_mask(tt);
          }
          AdapterGroups g(mask, p.r);
          while (ok && g.next()) {
            ok = mbar_wait(&sm.full[stage], phase, abort_flag, p.status, kFtWaitNs, 64);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s = smem_u32(ring + stage * kFpStageBytes);
            const uint64_t ad = umma_desc_sw128(s), bd = umma_desc_mn_sw128(s + 128 * 128, 64 * 128);
            const int steps = g.steps();
            for (int k = 0; k < steps; ++k) umma_bf16_pair(d, ad + 2 * k, bd + 128 * (k >> 1), zidesc, 1u);
            advance();
          }
        }
        if (!ok) break;
        umma_commit_pair(&sm.tfull[buf], 3);
      }
      umma_commit_pair(&sm.tdone, 1);  // every MMA is done before TMEM is released
      volatile int dummy = 0;
      mbar_wait(&sm.tdone, 0, &dummy, nullptr, kFtWaitNs, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue: thread = token
    const int g4 = warp & 3;           // TMEM lane quarter this warp may access
    const int half = (warp - 2) >> 2;  // half of the tile's output features
    const int width = p.gated ? 64 : 128;
    if (p.r && warp == 2) {  // what the scan found
      pdl_wait();
      uint64_t b = 0ull;
      for (int i = lane; i < p.scan_ctas; i += 32) b |= *reinterpret_cast<const volatile uint64_t*>(p.bad_part + i);
      const unsigned lo = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(b));
      const unsigned hi = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(b >> 32));
      if (lane == 0) {
        sm.bad = lo | (static_cast<uint64_t>(hi) << 32);
        mbar_arrive(&sm.scanned);
      }
    }
    int it = 0;
    for (int t = pair; t < total; t += pairs, ++it) {
      int tt, ft;
      fp_tile(p, t, tt, ft);
      const int buf = it & 1;
      const bool got = mbar_wait(&sm.tfull[buf], static_cast<uint32_t>(it >> 1) & 1u, abort_flag, p.status, kFtWaitNs, 66);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const int tok = p.t_first + tt * 256 + static_cast<int>(rank) * 128 + g4 * 32 + lane;
      const bool row_ok = tok < p.T;
      int bad_ad = -1;
      if (p.r) {
        pdl_wait();
        mbar_wait(&sm.scanned, 0, abort_flag, p.status, kFtWaitNs, 67);
        const uint64_t bad = sm.bad;
        if (bad != 0 && row_ok) {
          const int ad = p.row_adapter[tok];
          if (ad >= 0 && (bad >> ad & 1ull)) bad_ad = ad;
        }
      }
      const uint32_t acc = tmem + (static_cast<uint32_t>(g4 * 32) << 16) + buf * 256;
      for (int c = half * width; c < (half + 1) * width; c += 32) {
        const int f = ft * 2 * width + c;  // first of 32 output features
        float h[32], u[32];
        __syncwarp();  // (rows behind the last token left the run before this one early)
        tmem_ld_32x32b_x32(acc + c, h);
        if (p.gated) tmem_ld_32x32b_x32(acc + 128 + c, u);
        if (c + 32 == (half + 1) * width) {  // the warp has read its last columns
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(leader(&sm.tempty[buf]));
        }
        if (!row_ok || f >= p.h_out) continue;
        if (bad_ad >= 0) {  // an adapter with values that are not finite: its own tokens only
          for (int i = 0; i < p.r; ++i) {
            const float zi = z_value(p.z, tok, p.r, i);
            const __nv_bfloat16* br = p.lora_b + (static_cast<size_t>(bad_ad) * p.r + i) * p.n + f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (f + j < p.h_out) {
                h[j] = fmaf(zi, __bfloat162float(br[j]), h[j]);
                if (p.gated) u[j] = fmaf(zi, __bfloat162float(br[p.h_out + j]), u[j]);
              }
          }
        }
        const size_t at = static_cast<size_t>(tok) * p.h_out + f;
        const int nq = min(4, (p.h_out - f) / 8);  // whole runs of 8 features (h_out is a multiple of 8)
        if (p.bias != nullptr) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= nq) break;
            float b[8];
            unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(p.bias + f) + q), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[8 * q + j] += b[j];
            if (p.gated) {
              unpack8_bf16(__ldg(reinterpret_cast<const uint4*>(p.bias + p.h_out + f) + q), b);
#pragma unroll
              for (int j = 0; j < 8; ++j) u[8 * q + j] += b[j];
            }
          }
        }
        if (p.gated) {
#pragma unroll
          for (int j = 0; j < 32; ++j) h[j] = sigmoid_of<true>(h[j], h[j]) * u[j];
        } else {
          act_apply<true>(p.act, h);
        }
        if (p.residual != nullptr) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q >= nq) break;
            float b[8];
            unpack8_bf16(*(reinterpret_cast<const uint4*>(p.residual + at) + q), b);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[8 * q + j] += b[j];
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (q >= nq) break;
          reinterpret_cast<uint4*>(p.y + at)[q] =
              make_uint4(pack2_bf16(h[8 * q], h[8 * q + 1]), pack2_bf16(h[8 * q + 2], h[8 * q + 3]),
                         pack2_bf16(h[8 * q + 4], h[8 * q + 5]), pack2_bf16(h[8 * q + 6], h[8 * q + 7]));
        }
      }
    }
  }

  pdl_trigger();  // a call behind this one may set itself up
  if (p.r) pdl_wait();
  tc_fence_before();
  __syncwarp();
  cluster_sync_all();  // no CTA leaves while its peer may still signal it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

cudaError_t launch_fused_prefill_tc(const FusedTcArgs& f, int t_first, int t_end, cudaStream_t st) {
  const DenseFusedArgs& a = f.a;
  CUtensorMap tmw, tmx, tmb, tmz;
  if (encode_tmap_2d(&tmw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w, a.h_in, a.n, static_cast<uint64_t>(a.h_in) * 2, 64,
                     128, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tmap_2d(&tmx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.h_in, a.T, static_cast<uint64_t>(a.h_in) * 2, 64,
                     128, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  tmb = tmz = tmx;
  if (a.r && encode_tmap_2d(&tmb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.lora_b, a.n, static_cast<uint64_t>(a.L) * a.r,
                            static_cast<uint64_t>(a.n) * 2, 64, std::min(a.r, kGroupRank),
                            CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  if (a.r && encode_tmap_2d(&tmz, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f.zc, f.zc_pitch, t_end - t_first,
                            static_cast<uint64_t>(f.zc_pitch) * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  FpParams p{};
  p.bias = static_cast<const __nv_bfloat16*>(a.bias);
  p.residual = static_cast<const __nv_bfloat16*>(a.residual);
  p.y = static_cast<__nv_bfloat16*>(a.y);
  p.z = f.z;
  p.lora_b = static_cast<const __nv_bfloat16*>(a.lora_b);
  p.row_adapter = a.row_adapter;
  p.tile_mask = f.tile_mask + t_first / 256;
  p.bad_part = f.bad_part;
  p.scan_ctas = f.scan_ctas;
  p.L = a.L;
  p.status = a.status;
  p.t_first = t_first;
  p.T = t_end;
  p.K = a.h_in;
  p.h_out = a.h_out;
  p.n = a.n;
  p.r = a.r;
  p.act = a.act;
  p.gated = a.act == ML_ACT_SILU_AND_MUL;
  p.tok_tiles = (t_end - t_first + 255) / 256;
  p.feat_tiles = p.gated ? (a.h_out + 127) / 128 : (a.h_out + 255) / 256;
  const long long total = static_cast<long long>(p.tok_tiles) * p.feat_tiles;
  const int grid = 2 * static_cast<int>(std::min<long long>(a.num_sms / 2, total));
  const size_t smem = 1024 + kFpStages * kFpStageBytes;
  static std::atomic<bool> attr_set[kMaxDevices];
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(fused_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  ProfScope ps(K_DENSE_FUSED, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fused_prefill_kernel, tmw, tmx, tmb, tmz, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mlb
