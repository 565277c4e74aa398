// Shrink of dense_lora_fused on the tensor cores: z_t = c x_t A_a(t), bf16
// ([vLLM MoE-LoRA page], "O Papel da Multi-LoRA"; split-K, "Otimizações em Nível de Kernel").
//
// A tile of 128 tokens fills the MMA's M; its N takes the rank rows of 256 / r of the tile's
// adapters at a time, so every token meets each of them and keeps the columns of its own.
// Ahead of the tiled projection z is also laid out as that kernel's operand: the K columns of a
// 256-token tile's adapters side by side (see AdapterGroups), zeros where a token has another one.
// A cluster of C CTAs splits h_in: each holds fp32 partial sums of all 128 tokens, then adds
// up 128 / C tokens' partials in rank order from its peers' shared memory (no atomics: the
// same bits every time).
//
// A launch beside it reads the B rows of the adapters in use and records which hold a value
// that is not finite: the projection keeps those out of its matrix product, where a zero times
// an infinity would reach other tenants' tokens.  The rows read stay in L2, where the
// projection finds them.
#include "fused_tc.cuh"
#include "prof.h"

#include <algorithm>
#include <atomic>

namespace mlb {

constexpr int kShThreads = 192;
constexpr int kShN = 256;
// The ring holds as many stages of a chunk's size as fit, at most kShStages: x is read from HBM
// once, so what counts is the bytes on their way (4096 tokens with one adapter of rank 64:
// 1036 cycles per 24 KB stage with three of them).
constexpr int kShRing = 147456, kShStages = 8;
constexpr int kShSegs = 512;  // segments kept in shared memory

struct ShParams {
  const int32_t* seg_offsets;
  const int32_t* seg_adapter;
  int S, T, L, r, K, n;
  float scale;
  int t_first;  // this launch's tokens: [t_first, t_end)
  const __nv_bfloat16* lora_b;
  __nv_bfloat16* z;
  __nv_bfloat16* zc;
  int zc_pitch;
  int32_t* row_adapter;
  uint64_t* tile_mask;
  uint64_t* bad_part;
  int* status;
  int C, P;
  int operand;  // the tiled projection follows: zc, row_adapter and tile_mask as well
  int t_end;
};

struct ShCore {
  uint64_t full[kShStages], empty[kShStages], tfull, tempty;
  uint32_t tmem_base;
  int abort_flag;
  unsigned mask[2], own[2];  // adapters of the 256-token tile (of the 128 without zc), of these 128 tokens
  int wrong;
  int ids[kShN / 8];  // adapters of the chunk
  int row_ad[128];
  int off[kShSegs + 1], ad[kShSegs];
};

// Which adapters in use have B rows that are not finite.  Each CTA leaves those that it found
// in a word of its own, so that no counter has to be cleared.  Launched behind the shrink
// kernel, which it overlaps and ends behind; the projection launched behind it waits for both.
constexpr int kScanThreads = 256;

__global__ void __launch_bounds__(kScanThreads) fused_scan_kernel(const ShParams p) {
  __shared__ unsigned s_mask[2], s_bad[2];
  __shared__ int s_ids[64];
  const int tid = threadIdx.x;
  pdl_trigger();
  if (tid < 2) s_mask[tid] = s_bad[tid] = 0u;
  __syncthreads();
  for (int s = tid; s < p.S; s += kScanThreads) {
    const int a = p.seg_adapter[s], lo = p.seg_offsets[s], hi = p.seg_offsets[s + 1];
    if (a >= 0 && a < p.L && hi > lo) atomicOr(&s_mask[a >> 5], 1u << (a & 31));
  }
  __syncthreads();
  const uint64_t mask = s_mask[0] | (static_cast<uint64_t>(s_mask[1]) << 32);
  const int cnt = __popcll(mask);
  if (tid < 64 && (mask >> tid & 1ull)) s_ids[__popcll(mask & ((1ull << tid) - 1ull))] = tid;
  __syncthreads();
  const size_t chunks = static_cast<size_t>(p.r) * p.n / 8;  // 16 bytes each
  const size_t step = static_cast<size_t>(gridDim.x) * kScanThreads;
  const uint4* b = reinterpret_cast<const uint4*>(p.lora_b);
  for (size_t i = static_cast<size_t>(blockIdx.x) * kScanThreads + tid; i < chunks; i += step) {
    for (int q = 0; q < cnt; q += 8) {  // eight adapters' loads in flight
      uint4 v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __ldg(b + s_ids[min(q + e, cnt - 1)] * chunks + i);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (not_finite8(v[e])) {
          const int a = s_ids[min(q + e, cnt - 1)];
          atomicOr(&s_bad[a >> 5], 1u << (a & 31));
        }
      }
    }
  }
  __syncthreads();
  // The launch ends behind the shrink kernel by one CTA; the others leave their SMs to the
  // projection, whose CTAs do not fit beside them (600 x 4096 -> 2 x 2048 with 16 adapters: 51.2
  // against 52.8 us with all of them waiting).
  if (blockIdx.x == 0) pdl_wait();
  if (tid == 0) p.bad_part[blockIdx.x] = s_bad[0] | (static_cast<uint64_t>(s_bad[1]) << 32);
}

__global__ void __launch_bounds__(kShThreads) fused_shrink_kernel(const __grid_constant__ CUtensorMap tmx,
                                                                 const __grid_constant__ CUtensorMap tma,
                                                                 const ShParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(ring + kShRing);  // [128][r + 4]
  __shared__ ShCore sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();     // what ran ahead of the call is done, for the kernels behind this one too
  pdl_trigger();  // the projection streams its weights meanwhile

  const int rank = static_cast<int>(blockIdx.x) % p.C;
  const int group = static_cast<int>(blockIdx.x) / p.C;  // cluster index
  const int tile = group / p.P, chunk0 = group % p.P;
  const int t0 = p.t_first + tile * 128;
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    for (int s = 0; s < kShStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.tfull, 1);
    mbar_init(&sm.tempty, 128);
    sm.abort_flag = 0;
    sm.mask[0] = sm.mask[1] = sm.own[0] = sm.own[1] = 0u;
    sm.wrong = 0x7fffffff;
    fence_mbarrier_init();
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, kShN);
  const bool near = p.S <= kShSegs;
  if (near) {
    for (int s = tid; s <= p.S; s += kShThreads) {
      sm.off[s] = p.seg_offsets[s];
      if (s < p.S) sm.ad[s] = p.seg_adapter[s];
    }
  }
  const int32_t* seg_off = near ? sm.off : p.seg_offsets;
  const int32_t* seg_ad = near ? sm.ad : p.seg_adapter;
  __syncthreads();
  if (blockIdx.x == 0 && p.t_first == 0) {  // the call's first kernel: its status word
    int wrong = 0x7fffffff;
    for (int s = tid; s < p.S; s += kShThreads)
      if (segment_wrong(seg_off[s], seg_off[s + 1], seg_ad[s], p.T, p.L)) wrong = min(wrong, s);
    atomicMin(&sm.wrong, wrong);
    __syncthreads();
    if (tid == 0) {
      p.status[0] = sm.wrong != 0x7fffffff ? MOE_LORA_ERR_DEVICE_CHECK : MOE_LORA_OK;
      p.status[1] = sm.wrong != 0x7fffffff ? sm.wrong : 0;
    }
  }
  const bool operand = p.operand != 0;
  for (int i = tid; i < (operand ? 256 : 128); i += kShThreads) {  // own tokens, then the other half's
    const int t = i < 128 ? t0 + i : (t0 ^ 128) + i - 128;
    int a = -1;
    if (t < p.t_end) {
      const int s = segment_of(seg_off, p.S, t);
      if (s >= 0) a = seg_ad[s];
      if (a >= p.L || a < 0) a = -1;
      if (operand && i < 128 && chunk0 == 0 && rank == 0) p.row_adapter[t] = a;
    }
    if (i < 128) sm.row_ad[i] = a;
    if (a >= 0) atomicOr(&sm.mask[a >> 5], 1u << (a & 31));
    if (a >= 0 && i < 128) atomicOr(&sm.own[a >> 5], 1u << (a & 31));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint64_t mask = sm.mask[0] | (static_cast<uint64_t>(sm.mask[1]) << 32);
  const uint64_t own = sm.own[0] | (static_cast<uint64_t>(sm.own[1]) << 32);
  if (operand && tid == 0 && chunk0 == 0 && rank == 0 && (tile & 1) == 0) p.tile_mask[t0 >> 8] = mask;
  const uint32_t tmem = sm.tmem_base;
  const int apc = kShN / p.r;  // adapters per chunk
  const int cnt = __popcll(mask);
  const int chunks = (cnt + apc - 1) / apc;
  const int nkb = (p.K + 63) / 64;
  const int kb0 = nkb * rank / p.C, kb1 = nkb * (rank + 1) / p.C;
  const int pitch = p.r + 4;  // floats per partial row: 16-byte aligned, rows on other banks
  uint32_t phase = 0;  // by stage: parity of its next use
  bool ok = true;
  uint32_t filled = 0;

  for (int ch = chunk0, it = 0; ch < chunks; ch += p.P) {
    // the chunk's adapters: bits [ch apc, ch apc + na) of the mask
    uint64_t rem = mask;
    for (int i = 0; i < ch * apc; ++i) rem &= rem - 1;
    const int na = min(apc, cnt - ch * apc);
    uint64_t here = rem;  // the chunk's adapters, and whether a token of this CTA has one
    for (int i = 0; i < na; ++i) here &= here - 1;
    here ^= rem;
    const bool work = (here & own) != 0ull;
    // (every chunk begins with an idle ring: the one before ended in a cluster barrier)
    const int stage_bytes = (128 + na * p.r) * 128, stages = min(kShStages, kShRing / stage_bytes);
    int stage = 0;
    auto advance = [&]() {
      phase ^= 1u << stage;
      if (++stage == stages) stage = 0;
    };
    if (tid < na) {
      uint64_t m = rem;
      for (int i = 0; i < tid; ++i) m &= m - 1;
      sm.ids[tid] = __ffsll(static_cast<long long>(m)) - 1;
    }
    if (!work) {
      // (the other half's adapters: zeros only)
    } else if (warp == 0) {
      if (lane == 0) {
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          ok = mbar_wait(&sm.empty[stage], (phase >> stage & 1u) ^ 1u, abort_flag, p.status, kFtWaitNs, 40);
          if (!ok) break;
          uint8_t* s = ring + stage * stage_bytes;
          mbar_arrive_expect_tx(&sm.full[stage], static_cast<uint32_t>(stage_bytes));
          tma_load_2d(s, &tmx, &sm.full[stage], kb * 64, t0);
          uint64_t m = rem;
          for (int q = 0; q < na; ++q, m &= m - 1) {
            const int a = __ffsll(static_cast<long long>(m)) - 1;
            tma_load_2d(s + 128 * 128 + q * p.r * 128, &tma, &sm.full[stage], kb * 64, a * p.r);
          }
          filled |= 1u << stage;
          advance();
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        const uint32_t idesc = umma_idesc_bf16(128, (na * p.r + 15) & ~15);
        ok = ok && mbar_wait(&sm.tempty, (static_cast<uint32_t>(it) & 1u) ^ 1u, abort_flag, p.status, kFtWaitNs, 41);
        tc_fence_after();
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          ok = mbar_wait(&sm.full[stage], phase >> stage & 1u, abort_flag, p.status, kFtWaitNs, 42);
          if (!ok) break;
          tc_fence_after();
          const uint32_t s = smem_u32(ring + stage * stage_bytes);
          const uint64_t ad = umma_desc_sw128(s), bd = umma_desc_sw128(s + 128 * 128);
#pragma unroll
          for (int k = 0; k < 4; ++k) umma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
          umma_commit(&sm.empty[stage]);
          advance();
        }
        umma_commit(&sm.tfull);
      }
      __syncwarp();
    } else {
      // this token's columns of its own adapter -> its partial row
      const int g4 = warp & 3, row = g4 * 32 + lane;
      bool got = mbar_wait(&sm.tfull, static_cast<uint32_t>(it) & 1u, abort_flag, p.status, kFtWaitNs, 43);
      __syncwarp();
      got = named_bar_and(1, 128, got);
      if (got && kb1 > kb0) {
        tc_fence_after();
        const int a = sm.row_ad[row];
        int mine = -1;  // this token's adapter among the chunk's
        if (a >= 0 && (rem >> a & 1ull)) {
          mine = __popcll(rem & ((1ull << a) - 1ull));
          if (mine >= na) mine = -1;
        }
        for (int c0 = 0; c0 < na * p.r; c0 += 32) {
          float v[32];
          __syncwarp();  // (lanes whose adapter is elsewhere stored nothing)
          tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(g4 * 32) << 16) + c0, v);
          // columns [c0, c0 + 32) against this token's [mine r, mine r + r)
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            const int i = c0 + j - mine * p.r;
            if (mine >= 0 && i >= 0 && i < p.r) {
              float4* d = reinterpret_cast<float4*>(part + row * pitch + i);
              d[0] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
              d[1] = make_float4(v[j + 4], v[j + 5], v[j + 6], v[j + 7]);
            }
          }
        }
        tc_fence_before();
      } else if (got) {  // no K block of its own: its share of the sum is zero
        for (int i = 0; i < p.r; ++i) part[row * pitch + i] = 0.f;
      }
      mbar_arrive(&sm.tempty);
    }
    if (work) ++it;
    __syncwarp();
    cluster_sync_all();
    // rows [rank 128 / C, ...): sum over the cluster in rank order
    const int rows = 128 / p.C, q4 = p.r / 4;
    if (operand) {
      const int r8 = p.r / 8, per_row = na * r8;
      for (int e = tid; e < rows * per_row; e += kShThreads) {
        const int row = rank * rows + e / per_row, q = e % per_row / r8, j = e % per_row % r8, a = sm.ids[q];
        const int t = t0 + row;
        if (t >= p.t_end) continue;
        uint4 o = make_uint4(0u, 0u, 0u, 0u), l = o;
        if (sm.row_ad[row] == a) {
          const uint32_t at = smem_u32(part + row * pitch + 8 * j);
          float s[8] = {};
          float4 v[2][8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < p.C) {
              v[0][c] = ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(c)));
              v[1][c] = ld_cluster_f4(mapa_shared(at + 16u, static_cast<uint32_t>(c)));
            }
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < p.C)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                s[4 * u] += v[u][c].x;
                s[4 * u + 1] += v[u][c].y;
                s[4 * u + 2] += v[u][c].z;
                s[4 * u + 3] += v[u][c].w;
              }
          split2(p.scale * s[0], p.scale * s[1], o.x, l.x);
          split2(p.scale * s[2], p.scale * s[3], o.y, l.y);
          split2(p.scale * s[4], p.scale * s[5], o.z, l.z);
          split2(p.scale * s[6], p.scale * s[7], o.w, l.w);
          uint4* zt = reinterpret_cast<uint4*>(p.z + static_cast<size_t>(t) * 2 * p.r + 8 * j);
          zt[0] = o;
          zt[r8] = l;
        }
        // rank column R of the tile's adapters: K columns 32 (R / 16) + R % 16 (values) and 16 on
        const int R = __popcll(mask & ((1ull << a) - 1ull)) * p.r + 8 * j;
        uint4* zt = reinterpret_cast<uint4*>(p.zc + static_cast<size_t>(t - p.t_first) * p.zc_pitch + 32 * (R >> 4) + (R & 15));
        zt[0] = o;
        zt[2] = l;
        // an odd adapter of rank 8 ends inside an MMA step
        if (p.r == 8 && !(R & 8) && R + 8 == cnt * 8) zt[1] = zt[3] = make_uint4(0u, 0u, 0u, 0u);
      }
    } else {
      for (int e = tid; e < rows * q4; e += kShThreads) {
        const int row = rank * rows + e / q4, i = (e % q4) * 4;
        const int a = sm.row_ad[row];
        if (a < 0 || !(rem >> a & 1ull) || __popcll(rem & ((1ull << a) - 1ull)) >= na) continue;
        const uint32_t at = smem_u32(part + row * pitch + i);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < p.C; ++c) {
          const float4 v = ld_cluster_f4(mapa_shared(at, static_cast<uint32_t>(c)));
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        uint2 o, l;
        split2(p.scale * s.x, p.scale * s.y, o.x, l.x);
        split2(p.scale * s.z, p.scale * s.w, o.y, l.y);
        __nv_bfloat16* zt = p.z + static_cast<size_t>(t0 + row) * 2 * p.r + i;
        *reinterpret_cast<uint2*>(zt) = o;
        *reinterpret_cast<uint2*>(zt + p.r) = l;
      }
    }
    __syncwarp();
    cluster_sync_all();  // the peers have read this CTA's partials
  }
  if (warp == 0 && lane == 0 && *abort_flag)  // let our own copies land before the CTA exits
    for (int s = 0; s < kShStages; ++s)
      if (filled & (1u << s)) {
        volatile int dummy = 0;
        mbar_wait(&sm.full[s], (phase >> s & 1u) ^ 1u, &dummy, nullptr, kFtWaitNs / 4, 0);  // (its last use)
      }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kShN);
}

// A launch that may start while what runs ahead ends (it waits for that itself).
template <typename... P, typename... A>
static cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_fused_shrink_tc(const FusedTcArgs& f, bool operand, int t_first, int t_end, cudaStream_t st) {
  const DenseFusedArgs& a = f.a;
  CUtensorMap tmx, tma;
  if (encode_tmap_2d(&tmx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.h_in, a.T, static_cast<uint64_t>(a.h_in) * 2, 64,
                     128, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tmap_2d(&tma, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.lora_a, a.h_in, static_cast<uint64_t>(a.L) * a.r,
                     static_cast<uint64_t>(a.h_in) * 2, 64, a.r, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  ShParams p{};
  p.seg_offsets = a.seg_offsets;
  p.seg_adapter = a.seg_adapter;
  p.S = a.S;
  p.T = a.T;
  p.L = a.L;
  p.r = a.r;
  p.K = a.h_in;
  p.n = a.n;
  p.scale = a.scale;
  p.lora_b = static_cast<const __nv_bfloat16*>(a.lora_b);
  p.z = f.z;
  p.row_adapter = a.row_adapter;
  p.zc = f.zc;
  p.zc_pitch = f.zc_pitch;
  p.tile_mask = f.tile_mask;
  p.bad_part = f.bad_part;
  p.status = a.status;
  // K splits: as many as keep one wave of CTAs (one per SM: 144 KB of ring each)
  const int tiles = (t_end - t_first + 127) / 128;
  p.C = 8;
  while (p.C > 1 && tiles * p.C > a.num_sms) p.C /= 2;
  // chunks of a tile side by side while SMs are left
  const int apc = kShN / a.r, most = (std::min(std::min(a.L, a.S), 128) + apc - 1) / apc;
  p.P = std::max(1, std::min(most, a.num_sms / (tiles * p.C)));
  p.operand = operand;
  p.t_first = t_first;
  p.t_end = t_end;
  const size_t smem = 1024 + kShRing + 128u * (a.r + 4) * 4;
  static std::atomic<bool> attr_set[kMaxDevices];
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(fused_shrink_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               1024 + kShRing + 128 * (128 + 4) * 4);
    if (e != cudaSuccess) return e;
    // (SMs that run the scan are split as the kernels behind it need them: see launch_small)
    const cudaError_t c = cudaFuncSetAttribute(fused_scan_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                               cudaSharedmemCarveoutMaxShared);
    if (c != cudaSuccess) return c;
    attr_set[dev].store(true, std::memory_order_release);
  }
  ProfScope ps(K_FUSED_SHRINK, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles * p.P * p.C);
  cfg.blockDim = dim3(kShThreads);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, fused_shrink_kernel, tmx, tma, p);
  count_launch();
  if (e == cudaSuccess && operand && t_first == 0) return launch_behind(fused_scan_kernel, dim3(f.scan_ctas), kScanThreads, st, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ---------------------------------------------------------------- few tokens
// z of a small batch on CUDA cores: latency counts, and CTAs that need no shared memory run
// beside the projection's, which starts meanwhile.  An item is up to 4 tokens of a segment; a
// CTA takes 4 rank rows of an item, its 8 warps split h_in.  Segments that are wrong may overlap
// without end, so there an item is one token, of the segment that every kernel finds for it.
constexpr int kSsTok = 4, kSsRank = 4, kSsThreads = 256;

template <int CTAS, int AHEAD>
__global__ void __launch_bounds__(kSsThreads, CTAS) fused_shrink_small_kernel(const ShParams p, const __nv_bfloat16* __restrict__ x,
                                                                       const __nv_bfloat16* __restrict__ lora_a) {
  __shared__ float s_red[8][kSsTok * kSsRank];
  __shared__ int s_item[3];  // first token, tokens (0: no such item), adapter
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();  // what ran ahead of the call is done, for the projection too
  pdl_trigger();
  const int i0 = blockIdx.y * kSsRank;
  for (int item = blockIdx.x;; item += gridDim.x) {
    if (warp == 0) {
      int base = 0, first_wrong = 0x7fffffff;
      if (lane == 0) s_item[1] = 0;
      __syncwarp();
      for (int s0 = 0; s0 < p.S; s0 += 32) {
        const int s = s0 + lane;
        int lo = 0, hi = 0, a = -1;
        if (s < p.S) {
          lo = p.seg_offsets[s];
          hi = p.seg_offsets[s + 1];
          a = p.seg_adapter[s];
          if (segment_wrong(lo, hi, a, p.T, p.L)) first_wrong = min(first_wrong, s);
          lo = max(lo, 0);
          hi = min(hi, p.T);
        }
        const int n = (a >= 0 && a < p.L && hi > lo) ? (hi - lo + kSsTok - 1) / kSsTok : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const int at = item - base - (incl - n);
        if (at >= 0 && at < n) {
          s_item[0] = lo + at * kSsTok;
          s_item[1] = min(kSsTok, hi - lo - at * kSsTok);
          s_item[2] = a;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
      first_wrong = __reduce_min_sync(0xffffffffu, first_wrong);
      __syncwarp();
      const bool wrong = first_wrong != 0x7fffffff;
      if (lane == 0) {
        if (wrong) {  // (without an adapter: some z that nobody reads)
          const int s = item < p.T ? segment_of(p.seg_offsets, p.S, item) : -1, a = s >= 0 ? p.seg_adapter[s] : 0;
          s_item[0] = item;
          s_item[1] = item < p.T ? 1 : 0;
          s_item[2] = a >= 0 && a < p.L ? a : 0;
        }
        if (blockIdx.x == 0 && blockIdx.y == 0 && item == 0) {  // the call's first kernel: its status word
          p.status[0] = wrong ? MOE_LORA_ERR_DEVICE_CHECK : MOE_LORA_OK;
          p.status[1] = wrong ? first_wrong : 0;
        }
      }
    }
    __syncthreads();
    const int t0 = s_item[0], nt = s_item[1], a = s_item[2];
    if (nt == 0) return;
    float acc[kSsRank][kSsTok] = {};
    const int h8 = p.K / 8;
    const uint4* A = reinterpret_cast<const uint4*>(lora_a) + (static_cast<size_t>(a) * p.r + i0) * h8;
    const uint4* X = reinterpret_cast<const uint4*>(x) + static_cast<size_t>(t0) * h8;
#pragma unroll AHEAD
    for (int c = tid; c < h8; c += kSsThreads) {
      uint4 av[kSsRank], xv[kSsTok];
#pragma unroll
      for (int i = 0; i < kSsRank; ++i) av[i] = __ldg(A + static_cast<size_t>(i) * h8 + c);
#pragma unroll
      for (int t = 0; t < kSsTok; ++t) xv[t] = __ldg(X + static_cast<size_t>(t < nt ? t : 0) * h8 + c);
#pragma unroll
      for (int t = 0; t < kSsTok; ++t)
        if (t < nt) {
#pragma unroll
          for (int i = 0; i < kSsRank; ++i) acc[i][t] += dot8_bf16(av[i], xv[t]);
        }
    }
#pragma unroll
    for (int i = 0; i < kSsRank; ++i)
#pragma unroll
      for (int t = 0; t < kSsTok; ++t) {
        const float v = warp_sum(acc[i][t]);
        if (lane == 0) s_red[warp][t * kSsRank + i] = v;
      }
    __syncthreads();
    if (tid < nt) {
      float s[kSsRank] = {};
#pragma unroll
      for (int w = 0; w < 8; ++w)
#pragma unroll
        for (int i = 0; i < kSsRank; ++i) s[i] += s_red[w][tid * kSsRank + i];
      uint2 o, l;
      split2(p.scale * s[0], p.scale * s[1], o.x, l.x);
      split2(p.scale * s[2], p.scale * s[3], o.y, l.y);
      __nv_bfloat16* zt = p.z + static_cast<size_t>(t0 + tid) * 2 * p.r + i0;
      *reinterpret_cast<uint2*>(zt) = o;
      *reinterpret_cast<uint2*>(zt + p.r) = l;
    }
    __syncthreads();
  }
}

// one item per segment and one per 4 more tokens
static int fused_shrink_items(const DenseFusedArgs& a) { return std::min(a.S, a.T) + a.T / kSsTok; }

bool fused_shrink_is_small(const DenseFusedArgs& a) {
  return static_cast<long long>(fused_shrink_items(a)) * (a.r / kSsRank) <= 2 * a.num_sms;
}

template <int CTAS, int AHEAD>
static cudaError_t launch_small(dim3 grid, cudaStream_t st, const ShParams& p, const __nv_bfloat16* x,
                                const __nv_bfloat16* lora_a) {
  // The projection's CTAs fill an SM's shared memory: an SM that runs this kernel has to be
  // split that way already, or it is drained first (64 x 11008 -> 4096: the last of them began
  // 7.6 us late).
  static std::atomic<bool> attr_set[kMaxDevices];
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e =
        cudaFuncSetAttribute(fused_shrink_small_kernel<CTAS, AHEAD>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  return launch_behind(fused_shrink_small_kernel<CTAS, AHEAD>, grid, kSsThreads, st, p, x, lora_a);
}

cudaError_t launch_fused_shrink_simt(const FusedTcArgs& f, cudaStream_t st) {
  const DenseFusedArgs& a = f.a;
  ShParams p{};
  p.seg_offsets = a.seg_offsets;
  p.seg_adapter = a.seg_adapter;
  p.S = a.S;
  p.T = a.T;
  p.L = a.L;
  p.r = a.r;
  p.K = a.h_in;
  p.scale = a.scale;
  p.z = f.z;
  p.status = a.status;
  ProfScope ps(K_FUSED_SHRINK, st);
  const dim3 grid(fused_shrink_items(a), a.r / kSsRank);
  // Up to two CTAs per SM: more loads in flight each (64 x 11008 -> 4096, one adapter: 26.0 us
  // against 28.0 with the other form); above, registers for a third (19 adapters of rank 64: 49
  // against 63 us).
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16*>(a.x), *la = static_cast<const __nv_bfloat16*>(a.lora_a);
  return fused_shrink_is_small(a) ? launch_small<2, 3>(grid, st, p, x, la) : launch_small<3, 2>(grid, st, p, x, la);
}

}  // namespace mlb
