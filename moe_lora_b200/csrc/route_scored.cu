// Scored routing: softmax or sigmoid scores, a selection bias per expert, expert groups,
// top-k, renormalised and scaled weights, then the stable (expert, adapter) sort.
//
// A router sends each token to its most relevant experts ([vLLM MoE-LoRA page],
// "Entendendo os Modelos MoE"); scores, bias, groups and scaling are the generic forms of
// that choice.
//
// One kernel makes logits, choice and weights: a cluster of C CTAs takes 128 tokens x all E
// experts (one tcgen05 tile: tokens in M, experts in N), splits H, and each CTA adds up the
// partial logits of 128 / C tokens from its peers' shared memory in rank order; its warps
// then choose those tokens' experts, a warp per token, the logits never leaving the SM.
// Batches that fill the SMs with 128 tokens each are bound by what the SMs read (x once, W_r
// once per tile): there CTA pairs (tcgen05 cta_group::2) share W_r, each reading half of it.
//
// 16384 tokens x 256 experts (H 7168) take 107 us (106 to 117 as calls among others): 47 us in which x streams (240 MB; 36 us at the
// copy rate), about 30 us of choice and weights (some 1000 instructions per token and warp),
// 10 us of sort.  One token in 12.6 us and 64 x 128 (H 7168) in 20.4 us are bound by latency: launch,
// copies, three cluster barriers and the choice follow each other at 1 to 2 us each.
//
// The sort needs no atomics on global memory: a CTA leaves one bit per (expert, token) and
// the running count of its pairs by expert.  Up to 128 tokens the cluster itself sorts (a
// warp per expert); above, a second kernel does, a CTA per expert.
#include "fused_tc.cuh"
#include "prof.h"

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>

namespace mlb {

constexpr int kRsThreads = 512;
constexpr int kRsWarps = kRsThreads / 32;
constexpr int kRsMaxStages = 8;
constexpr int kRsRing = 196608;  // bytes of the ring at most
constexpr int kRsBody = 128 * 260 * 4 + kRsWarps * 256 * 16;  // of its later use: logits, two words per warp and expert
static_assert(kRsBody >= kRsRing, "the dynamic shared memory of the largest case");

struct RsParams {
  const float* logits_in;
  const float* bias;
  const float* score_bias;
  const int32_t* adapter_ids;
  float* logits_out;
  int32_t* topk_ids;
  float* topk_w;
  int32_t* sorted_pairs;
  int32_t* seg_offsets;
  uint16_t* bitmap;  // [E][8 tiles]: bit t % 16 of word t / 16: token t chose the expert
  int32_t* before;   // [E][chunks]: the chunk's pairs of lower experts
  int32_t* flags;    // [chunks]: what the chunk has to report (kRsClean: nothing)
  int* status;
  int M, H, E, k, L;
  int tiles;  // of 128 tokens
  int C;      // CTAs that share a tile's tokens
  int wide;   // CTA pairs make the logits of two tiles (C = 1)
  int epad, stages;
  ScoreFormat f;
};

constexpr int kRsClean = INT_MAX;  // a token that failed a check: its index; a wait that ran out: < 0


// ------------------------------------------------------------------ the choice of one token
__device__ __forceinline__ float clamp_finite(float v) { return fminf(fmaxf(v, -FLT_MAX), FLT_MAX); }

// Order-preserving unsigned key of a finite float; both zeros alike.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
__device__ __forceinline__ float warp_max(float v) { return key_value(__reduce_max_sync(0xffffffffu, order_key(v))); }

// Selection scores as 23-bit fixed point q, so that q and the expert fit one word whose
// warp-wide maximum is one instruction, equal q going to the lower expert:
//   0 not a candidate, kQNan NaN, kQLow / kQHigh beyond the range, else kQMin + (v - lo) scale
// A fused multiply-add onto 2^23 leaves q in the mantissa.  An order is proved where q differs
// by more than `slack` (or the lower one is NaN); what is not proved is decided in 64 bits.
// Logits compared as such: every step is monotone, so any difference of q is a proof.
constexpr uint32_t kQNan = 1u, kQLow = 2u, kQHigh = (1u << 23) - 2u, kQMin = 16u;
constexpr float kQSpan = 8388576.f;  // 2^23 - 32
constexpr float kQOne = 8388608.f;   // 2^23: steps of one
constexpr float kBiasMost = 1024.f;  // larger biases leave the fixed-point range
constexpr float kLogitSpan = 32.f;   // logits further below the largest are kQLow

__device__ __forceinline__ bool proved(uint32_t above, uint32_t below, uint32_t slack) {
  return below <= kQNan || above > below + slack;
}

__device__ __forceinline__ float exp2_approx(float x) {  // within 2^-22 of the value
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {  // within a unit of the last place
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What the choice needs of the call.  One warp works it out for every expert while the copies
// are on their way, into shared memory; the others pick their lanes' experts up from there.
struct ExpertTable {
  float above[256];   // selection bias above the smallest one
  unsigned info[256];  // first lane of the expert's group | place among the groups' keys << 8 | kind << 28
  float range;        // of the biases: from the smallest to the largest
  int odd, exact;     // some expert is not just valid; every token in 64 bits
};
constexpr unsigned kValid = 1u, kNan = 2u, kLow = 4u, kHigh = 8u;  // kinds (a bias NaN, or out of the range)

struct RsCore {
  uint64_t full[kRsMaxStages], empty[kRsMaxStages], tfull;
  uint32_t tmem_base;
  int abort_flag;
  int flag;
  int next;  // token that no warp has taken yet
  int scan[kRsWarps];
  ExpertTable table;
  alignas(16) uint4 map[256];  // tokens of the tile (this CTA's: 128 / C of them) by expert
  uint8_t ids[kRsWarps][256];  // a token's choice
  alignas(16) uint8_t slot[256][16];  // up to 128 tokens: place of the expert among token i's choices
};

// lanes of a warp per group of experts
__device__ __forceinline__ int lanes_per_group(int n_group) {
  int per = 32;
  while (per > 1 && per * n_group > 32) per >>= 1;
  return per;
}

template <int NI>
__device__ __forceinline__ void make_table(const RsParams& p, ExpertTable& tab) {
  const int lane = threadIdx.x & 31, per = lanes_per_group(p.f.n_group);
  // a group's keys lie an odd number of words from the next one's (lanes meet other banks)
  const int pad = 1 - (p.f.group_size & 1);
  bool odd = false, exact = p.f.n_group > 32;
  float b[NI], bmin = FLT_MAX, bmax = -FLT_MAX;
  unsigned kind[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    kind[i] = 0u;
    b[i] = 0.f;
    if (e < p.E) {
      kind[i] = kValid;
      const float v = p.score_bias != nullptr ? p.score_bias[e] : 0.f;
      if (v != v) {
        kind[i] |= kNan;
      } else if (fabsf(v) > kBiasMost) {
        kind[i] |= v < 0.f ? kLow : kHigh;
        exact |= fabsf(v) < kBiasMost + 2.f;  // (a score is at most 1: it might cross over)
      } else {
        b[i] = v;
        bmin = fminf(bmin, v);
        bmax = fmaxf(bmax, v);
      }
    }
    odd |= kind[i] != kValid;
  }
  bmin = -warp_max(-bmin);
  bmax = warp_max(bmax);
  if (bmin > bmax) bmin = bmax = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    const int g = e < p.E && p.f.n_group > 1 ? e / p.f.group_size : 0;
    tab.above[e] = kind[i] == kValid ? b[i] - bmin : 0.f;
    tab.info[e] = static_cast<unsigned>(g * per & 31) | static_cast<unsigned>(e + g * pad) << 8 | kind[i] << 28;
  }
  odd = __any_sync(0xffffffffu, odd);
  exact = __any_sync(0xffffffffu, exact);
  if (lane == 0) {
    tab.range = bmax - bmin;
    tab.odd = odd;
    tab.exact = exact;
  }
}

// The table's part of a lane: experts lane, lane + 32, ...
template <int NI>
struct ChoiceSetup {
  float above[NI];
  unsigned group[NI];  // bit of the first lane of the expert's group
  int at[NI];
  int per, stride;     // lanes per group; words from a group's keys to the next one's
  float range;
  unsigned valid, nan, low, high;  // bit i: kind of expert lane + 32 i
  bool odd, exact;

  __device__ __forceinline__ void load(const RsParams& p, const ExpertTable& tab) {
    const int lane = threadIdx.x & 31;
    per = lanes_per_group(p.f.n_group);
    stride = p.f.group_size | 1;
    valid = nan = low = high = 0u;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const unsigned v = tab.info[lane + 32 * i];
      above[i] = tab.above[lane + 32 * i];
      group[i] = 1u << (v & 31u);
      at[i] = static_cast<int>(v >> 8 & 0xffffu);
      valid |= (v >> 28 & 1u) << i;
      nan |= (v >> 29 & 1u) << i;
      low |= (v >> 30 & 1u) << i;
      high |= (v >> 31 & 1u) << i;
    }
    range = tab.range;
    odd = tab.odd != 0;
    exact = tab.exact != 0;
  }
};

// The same for 64-bit scores: larger than 0, the key of "not a candidate".
__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// the warp's largest key, the smallest index of those that hold it
__device__ __forceinline__ int warp_argmax(uint64_t key, int at) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
  const bool same = static_cast<uint32_t>(key >> 32) == hi;
  const uint32_t lo = __reduce_max_sync(0xffffffffu, same ? static_cast<uint32_t>(key) : 0u);
  return static_cast<int>(
      __reduce_min_sync(0xffffffffu, same && static_cast<uint32_t>(key) == lo ? static_cast<uint32_t>(at) : 0xffffffffu));
}

// Scores in 64 bits.
__device__ __forceinline__ float row_max(const float* row, int E) {
  float mx = -FLT_MAX;
  for (int e = threadIdx.x & 31; e < E; e += 32)
    if (row[e] == row[e]) mx = fmaxf(mx, clamp_finite(row[e]));
  return warp_max(mx);
}

__device__ __noinline__ double exact_sum(const float* row, int E, float mx) {
  double sum = 0.0;
#pragma unroll 1
  for (int e = threadIdx.x & 31; e < E; e += 32)
    if (row[e] == row[e]) sum += exp(static_cast<double>(clamp_finite(row[e])) - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

__device__ __noinline__ double exact_score(float logit, int sigmoid, float mx, double sum) {
  const double l = clamp_finite(logit);
  const double x = exp(sigmoid ? -l : l - mx);
  return sigmoid ? 1.0 / (1.0 + x) : x / sum;
}

__device__ __forceinline__ double exact_selection(const float* row, const RsParams& p, int e, float mx, double sum) {
  const float b = p.score_bias ? p.score_bias[e] : 0.f;
  if (row[e] != row[e] || b != b) return -INFINITY;
  if (p.f.by_logit) return static_cast<double>(clamp_finite(row[e]));
  return exact_score(row[e], p.f.sigmoid, mx, sum) + static_cast<double>(clamp_finite(b));
}

// Up to 32 candidates, lane j holding expert e of the j-th (n of them): the first k in 64 bits.
__device__ __noinline__ void order_candidates(const float* row, const RsParams& p, int e, int n, uint8_t* ids) {
  const int lane = threadIdx.x & 31;
  const float mx = p.f.sigmoid || p.f.by_logit ? 0.f : row_max(row, p.E);
  const double sum = p.f.sigmoid || p.f.by_logit ? 1.0 : exact_sum(row, p.E, mx);
  const double c = lane < n ? exact_selection(row, p, e, mx, sum) : 0.0;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double o = __shfl_sync(0xffffffffu, c, i);
    const int oe = __shfl_sync(0xffffffffu, e, i);
    rank += (o > c || (o == c && oe < e)) ? 1 : 0;
  }
  if (lane < n && rank < p.k) ids[rank] = static_cast<uint8_t>(e);
  __syncwarp();
}

// The definition in 64 bits, for tokens whose 32-bit scores lie too close to prove an order.
// Few instructions rather than few steps: rarely run, its code is read from far.  c: a key of
// the warp per expert; g: a key per group (n_group > 1 only).
__device__ __noinline__ void choose_exact(const float* row, const RsParams& p, uint64_t* c, uint64_t* g, uint8_t* ids) {
  const int lane = threadIdx.x & 31;
  const ScoreFormat& f = p.f;
  const bool by_score = !f.sigmoid && !f.by_logit;
  const float mx = by_score ? row_max(row, p.E) : 0.f;
  const double sum = by_score ? exact_sum(row, p.E, mx) : 1.0;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) c[e] = order_key64(exact_selection(row, p, e, mx, sum));
  __syncwarp();
  // takes the largest of v[0, n), the first of equals
  auto take = [&](uint64_t* v, int n) -> int {
    uint64_t best = 0ull;
    int at = lane;
#pragma unroll 1
    for (int i = lane; i < n; i += 32)
      if (v[i] > best) {
        best = v[i];
        at = i;
      }
    at = warp_argmax(best, at);
    if ((at & 31) == lane) v[at] = 0ull;
    return at;
  };
  if (f.n_group > 1) {
#pragma unroll 1
    for (int q = lane; q < f.n_group; q += 32) {
      uint64_t m1 = 0ull, m2 = 0ull;
      int e1 = 0, e2 = 0;
#pragma unroll 1
      for (int e = q * f.group_size; e < (q + 1) * f.group_size; ++e) {
        const uint64_t v = c[e];
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
      // scores and biases summed apart, so that groups whose two best have the same scores
      // and the same sum of biases tie, whatever the roundings
      if (f.top2 && f.group_size > 1) {
        if (m2 == order_key64(-INFINITY)) {  // a NaN
          m1 = m2;
        } else {
          const double s1 = exact_score(row[e1], f.sigmoid, mx, sum), s2 = exact_score(row[e2], f.sigmoid, mx, sum);
          const double b1 = p.score_bias ? static_cast<double>(clamp_finite(p.score_bias[e1])) : 0.0;
          const double b2 = p.score_bias ? static_cast<double>(clamp_finite(p.score_bias[e2])) : 0.0;
          m1 = order_key64((s1 + s2) + (b1 + b2));
        }
      }
      g[q] = m1;
    }
    __syncwarp();
    unsigned out = 0xffffffffu;  // this lane's experts of groups that are not kept
#pragma unroll 1
    for (int j = 0; j < f.topk_group; ++j) {
      const int q = take(g, f.n_group);
#pragma unroll 1
      for (int i = 0; 32 * i + lane < p.E; ++i)
        if ((32 * i + lane) / f.group_size == q) out &= ~(1u << i);
    }
#pragma unroll 1
    for (int i = 0; 32 * i + lane < p.E; ++i)
      if (out >> i & 1u) c[32 * i + lane] = 0ull;
  }
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    const int e = take(c, p.E);
    if (lane == 0) ids[j] = static_cast<uint8_t>(e);
  }
  __syncwarp();
}

// The k experts of the token whose logits are row[0, E), in order, into ids; returns whether
// a NaN was met.  Also the row's largest logit and the sum of its exponentials (softmax).
// scratch: two 64-bit words of the warp per expert.
template <int NI>
__device__ __forceinline__ bool choose(const float* row, const RsParams& p, const ChoiceSetup<NI>& cs, float* copy_to,
                                       uint64_t* scratch, uint8_t* ids, float& mx, float& sum) {
  const int lane = threadIdx.x & 31;
  const ScoreFormat& f = p.f;
  float v[NI];       // logits, then scores (exponentials, for a softmax)
  uint32_t key[NI];  // q and 255 - expert
  unsigned unread = 0u;  // bit i: the logit of expert lane + 32 i is a NaN
  float probe = 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    v[i] = cs.valid >> i & 1u ? row[lane + 32 * i] : 0.f;
    if (copy_to != nullptr && (cs.valid >> i & 1u)) copy_to[lane + 32 * i] = v[i];
    probe = fmaf(v[i], 0.f, probe);
  }
  const bool odd = __any_sync(0xffffffffu, probe != probe) || cs.odd;
  if (odd) {  // infinities, NaN; no experts
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (v[i] != v[i]) unread |= 1u << i;
      v[i] = v[i] != v[i] || !(cs.valid >> i & 1u) ? -FLT_MAX : clamp_finite(v[i]);
    }
  }
  const unsigned nan = cs.nan | unread;
  mx = -FLT_MAX;
  sum = 1.f;
  if (!f.sigmoid || f.by_logit) {
#pragma unroll
    for (int i = 0; i < NI; ++i) mx = fmaxf(mx, v[i]);
    mx = warp_max(mx);
  }
  // q = v unit + above bias + base
  float unit = kQSpan / kLogitSpan, bias = 0.f, base = kQOne + kQMin + kQSpan, top = 1.f;
  if (!f.sigmoid && !(f.by_logit && f.renorm)) {
    float s[NI];
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      s[i] = cs.valid >> i & 1u ? expf(v[i] - mx) : 0.f;
      if (odd && unread >> i & 1u) s[i] = 0.f;
      sum += s[i];
    }
    sum = warp_sum(sum);
    if (!f.by_logit) {
      top = 1.f / sum;  // the largest score
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = s[i];
    }
  } else if (!f.by_logit) {
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = rcp_approx(1.f + exp2_approx(v[i] * -1.4426950408889634f));
  }
  // Error of a selection score in 2^-24: a sigmoid's exponential (s (1 - s) times 4 for the
  // value and 2 |l| for the argument) 2, its sum 1, its quotient 2; a softmax's exponential and
  // its argument 5, the sum of up to 256 of them (4 each, 13 roundings) 17, quotient and unit 3,
  // of the largest score; the bias above the smallest, the range.  In steps of range 2^-23, with
  // a step for the two roundings of q and one for `unit`; for two scores.
  uint32_t slack = 0u;
  if (f.by_logit) {
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] -= mx;
  } else {
    const float range = top + cs.range;
    bias = kQSpan / range;
    unit = bias * top;
    base = kQOne + kQMin;
    slack = static_cast<uint32_t>(2.f * (0.5f * ((f.sigmoid ? 5.f : 25.f * top) + range) / range + 2.f)) + 1u;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const float q = fmaxf(fmaf(v[i], unit, fmaf(cs.above[i], bias, base)), kQOne + kQLow);
    key[i] = __float_as_uint(q) * 256u + static_cast<uint32_t>(255 - 32 * i - lane);  // (drops the exponent)
  }
  if (odd) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint32_t tag = static_cast<uint32_t>(255 - 32 * i - lane);
      if (cs.low >> i & 1u) key[i] = kQLow << 8 | tag;
      if (cs.high >> i & 1u) key[i] = kQHigh << 8 | tag;
      if (nan >> i & 1u) key[i] = kQNan << 8 | tag;
      if (!(cs.valid >> i & 1u)) key[i] = 0u;
    }
  }
  bool exact = cs.exact;
  if (f.n_group > 1 && !exact) {
    uint32_t* keys = reinterpret_cast<uint32_t*>(scratch);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (cs.valid >> i & 1u) keys[cs.at[i]] = key[i];
    __syncwarp();
    // `per` lanes per group walk its experts and join their two largest
    const int per = cs.per, g = lane / per, sub = lane & (per - 1);
    const bool in = g < f.n_group;
    uint32_t m1 = 0u, m2 = 0u;
    if (in) {
      const uint32_t* from = keys + g * cs.stride;
#pragma unroll 8
      for (int j = sub; j < f.group_size; j += per) {
        const uint32_t o = from[j];
        m2 = max(m2, min(m1, o));
        m1 = max(m1, o);
      }
    }
    for (int o = 1; o < per; o <<= 1) {
      const uint32_t a1 = __shfl_xor_sync(0xffffffffu, m1, o), a2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = max(max(m2, a2), min(m1, a1));
      m1 = max(m1, a1);
    }
    m1 >>= 8;
    m2 >>= 8;
    uint32_t gk = m1, group_slack = slack;
    if (f.top2 && f.group_size > 1) {
      // (sums with a member beyond the range say nothing)
      exact = __any_sync(0xffffffffu, in && (m1 >= kQHigh || m2 == kQLow));
      gk = m2 <= kQNan ? kQNan : m1 + m2;
      group_slack *= 2u;
    }
    gk = gk << 5 | static_cast<uint32_t>(31 - g);
    int rank = 0;  // larger groups, and as large ones before
#pragma unroll 4
    for (int h = 0; h < f.n_group; ++h) rank += __shfl_sync(0xffffffffu, gk, h * per) > gk ? 1 : 0;
    const bool kept = in && rank < f.topk_group;
    const uint32_t last = __reduce_min_sync(0xffffffffu, kept ? gk : 0xffffffffu);
    const uint32_t first = __reduce_max_sync(0xffffffffu, in && !kept ? gk : 0u);
    exact |= !proved(last >> 5, first >> 5, group_slack);
    const unsigned keep = __ballot_sync(0xffffffffu, kept);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if ((keep & cs.group[i]) == 0u) key[i] = 0u;
  }
  if (!exact) {
    // each lane's three largest in order; the warp takes the largest of all, k times
    uint32_t a = 0u, b = 0u, c = 0u;
    auto refill = [&](uint32_t below) {
      a = b = c = 0u;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t o = key[i] < below ? key[i] : 0u, u = min(a, o), w = min(b, u);
        a = max(a, o);
        b = max(b, u);
        c = max(c, w);
      }
    };
    refill(0xffffffffu);
    int used = 0;
    auto next = [&]() -> uint32_t {
      const uint32_t m = __reduce_max_sync(0xffffffffu, a);
      if (a == m) {
        a = b;
        b = c;
        c = 0u;
        ++used;
      }
      if (used == 3) {
        refill(m);
        used = 0;
      }
      return m;
    };
    uint32_t prev = next(), gap = 0xffffffffu;
    uint32_t mine = prev;
    if (p.k > 32 && lane == 0) ids[0] = static_cast<uint8_t>(255u - (prev & 255u));
    for (int j = 1; j < p.k; ++j) {
      const uint32_t m = next();
      gap = min(gap, prev - m);
      prev = m;
      mine = lane == j ? m : mine;
      if (p.k > 32 && lane == 0) ids[j] = static_cast<uint8_t>(255u - (m & 255u));
    }
    uint32_t left = next();  // the first one left out
    gap = min(gap, prev - left);
    if (p.k <= 32 && lane < p.k) ids[lane] = static_cast<uint8_t>(255u - (mine & 255u));
    __syncwarp();
    if (gap <= slack * 256u + 256u) {  // (a difference of q above the slack is a larger gap)
      // with every expert that may belong to the first k
      int n = p.k;
      for (; n < 32 && !proved(prev >> 8, left >> 8, slack); ++n) {
        mine = lane == n ? left : mine;
        left = next();
      }
      exact = n > 32 || !proved(prev >> 8, left >> 8, slack);
      if (!exact) order_candidates(row, p, static_cast<int>(255u - (mine & 255u)), n, ids);
    }
  }
  if (exact) {
    __syncwarp();
    choose_exact(row, p, scratch, scratch + p.epad, ids);
    __syncwarp();
  }
  return __any_sync(0xffffffffu, nan != 0u);
}

// Weights of the chosen, in 32 bits.  Renormalised: relative to the largest chosen logit (at
// most 0 for sigmoids), so that scores below the smallest float keep their ratio.
__device__ __forceinline__ void weigh(const float* row, const RsParams& p, const uint8_t* ids, int t, float mx,
                                      float sum) {
  const int lane = threadIdx.x & 31;
  const ScoreFormat& f = p.f;
  float top = f.sigmoid ? 0.f : mx;
  if (f.renorm) {
    top = -FLT_MAX;
    for (int j = lane; j < p.k; j += 32) {
      const float v = row[ids[j]];
      if (v == v) top = fmaxf(top, clamp_finite(v));
    }
    top = key_value(__reduce_max_sync(0xffffffffu, order_key(top)));
    if (f.sigmoid) top = fminf(top, 0.f);
  }
  auto weight = [&](int e) -> float {
    const float raw = row[e], v = clamp_finite(raw);
    if (raw != raw) return 0.f;
    const float num = f.sigmoid && v > 0.f ? 1.f : expf(v - top);
    return f.sigmoid ? num / (1.f + expf(-fabsf(v))) : num;
  };
  float w = lane < p.k ? weight(ids[lane]) : 0.f, mul = f.scale;
  if (f.renorm) {
    float wsum = w;
    for (int j = lane + 32; j < p.k; j += 32) wsum += weight(ids[j]);
    wsum = warp_sum(wsum);
    mul = wsum > 0.f ? f.scale / wsum : 0.f;
  } else if (!f.sigmoid) {
    mul = sum > 0.f ? f.scale / sum : 0.f;
  }
  for (int j = lane; j < p.k; j += 32) {
    if (j >= 32) w = weight(ids[j]);
    p.topk_ids[static_cast<size_t>(t) * p.k + j] = ids[j];
    p.topk_w[static_cast<size_t>(t) * p.k + j] = w * mul;
  }
}

// ------------------------------------------------------------------ the stable sort
// Slot of expert e among token t's k choices (the token chose it); written by the kernel
// ahead.  No early exit: the loads of several calls overlap.
__device__ __forceinline__ int slot_of_expert(const int32_t* topk_ids, int t, int k, int e) {
  const int32_t* row = topk_ids + static_cast<size_t>(t) * k;
  int at = 0;
  if ((k & 3) == 0 && k <= 16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (4 * q >= k) break;
      const int4 v = __ldcg(reinterpret_cast<const int4*>(row) + q);
      at = v.x == e ? 4 * q : v.y == e ? 4 * q + 1 : v.z == e ? 4 * q + 2 : v.w == e ? 4 * q + 3 : at;
    }
    return at;
  }
#pragma unroll 8
  for (int j = 0; j < k; ++j)
    if (__ldcg(row + j) == e) at = j;
  return at;
}

__device__ __forceinline__ uint4 ld_cluster_u32x4(uint32_t cluster_addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// exclusive prefix sum over the CTA's 512 threads
__device__ __forceinline__ int block_prefix(int v, int* s_scan) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kRsWarps; ++w) base += w < warp ? s_scan[w] : 0;
  return base + incl - v;
}

// One warp's exclusive prefix over n <= 96 counters, in place; each result plus `base` also to
// off[i].  (run and off: shared and global.)
__device__ __forceinline__ void warp_offsets(int* run, int n, int base, int32_t* off) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = i0 + lane;
    const int v = i < n ? run[i] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (i < n) {
      run[i] = base + incl - v;
      off[i] = base + incl - v;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
}

// Places one warp's pairs of up to 32 tokens in token order (lane = token; chosen: it chose
// the expert, as `pair`): run[a] is the next free place of adapter a.
__device__ __forceinline__ void place32(const RsParams& p, bool chosen, int pair, int a, int* run) {
  const int lane = threadIdx.x & 31;
  const unsigned peers = __match_any_sync(0xffffffffu, chosen ? a : 128 + lane);
  const unsigned before = peers & ((1u << lane) - 1u);
  if (chosen) p.sorted_pairs[run[a] + __popc(before)] = pair;
  __syncwarp();
  if (chosen && before == 0u) run[a] += __popc(peers);
  __syncwarp();
}

// ------------------------------------------------------------------ logits, choice, weights
template <int NI>
__global__ void __launch_bounds__(kRsThreads, 1)
    route_scored_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmw,
                        const RsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ RsCore sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = p.C, TC = 128 / C;
  const int rank = static_cast<int>(blockIdx.x) % C, tile = static_cast<int>(blockIdx.x) / C;
  const int t0 = tile * 128, own0 = rank * TC;
  const int pitch = p.epad + 4;  // floats: rows 16-byte aligned, neighbours 4 banks apart
  const bool given = p.logits_in != nullptr;
  // logits: the tile's partial sums [128][pitch], or a row per warp of given ones
  float* part = reinterpret_cast<float*>(ring);
  uint64_t* scratch = reinterpret_cast<uint64_t*>(ring + static_cast<size_t>(given ? kRsWarps : 128) * pitch * 4) +
                    warp * 2 * p.epad;
  volatile int* abort_flag = &sm.abort_flag;

  if (tid == 0) {
    sm.abort_flag = 0;
    sm.flag = kRsClean;
    sm.next = kRsWarps;
    if (!given) {
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(&sm.full[s], 1);
        mbar_init(&sm.empty[s], 1);
      }
      mbar_init(&sm.tfull, 1);
      fence_mbarrier_init();
      tma_prefetch_desc(&tmx);
      tma_prefetch_desc(&tmw);
    }
  }
  pdl_wait();  // what ran ahead of the call is done
  if (p.tiles > 1) pdl_trigger();  // the sort may be launched
  if (tid < 256) {
    sm.map[tid] = make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t cols = 32;
  while (cols < static_cast<uint32_t>(p.epad)) cols <<= 1;
  if (!given && warp == 1) {
    if (p.wide) tmem_alloc_pair(&sm.tmem_base, cols);
    else tmem_alloc(&sm.tmem_base, cols);
  }
  tc_fence_before();
  __syncwarp();
  if (p.wide) cluster_sync_all();  // the pair's barriers are ready
  else __syncthreads();
  tc_fence_after();

  if (warp == 2) make_table<NI>(p, sm.table);
  if (given) __syncthreads();
  if (!given) {
    const uint32_t tmem = sm.tmem_base;
    const int nkb = (p.H + 63) / 64;
    const int kb0 = static_cast<int>(static_cast<long long>(nkb) * rank / C);
    const int kb1 = static_cast<int>(static_cast<long long>(nkb) * (rank + 1) / C);
    // pairs: M = 256 over both CTAs, each holding its own tokens and half of the experts' rows;
    // copies are counted and MMAs issued by the even CTA
    const int half = static_cast<int>(blockIdx.x) & 1, w_rows = p.wide ? p.epad / 2 : p.epad;
    const int stage_bytes = (128 + w_rows) * 128;
    if (warp == 0) {
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 0, filled = 0, parity_of = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&sm.empty[stage], phase ^ 1u, abort_flag, nullptr, kFtWaitNs, 70)) break;
          uint8_t* s = ring + stage * stage_bytes;
          if (p.wide) {
            const uint32_t fb = mapa_shared(smem_u32(&sm.full[stage]), 0);
            if (half == 0) mbar_arrive_expect_tx(&sm.full[stage], 2u * static_cast<uint32_t>(stage_bytes));
            tma_load_2d_pair(s, &tmx, fb, kb * 64, t0);
            tma_load_2d_pair(s + 128 * 128, &tmw, fb, kb * 64, half * w_rows);
          } else {
            mbar_arrive_expect_tx(&sm.full[stage], static_cast<uint32_t>(stage_bytes));
            tma_load_2d(s, &tmx, &sm.full[stage], kb * 64, t0);
            tma_load_2d(s + 128 * 128, &tmw, &sm.full[stage], kb * 64, 0);
          }
          filled |= 1u << stage;
          parity_of = (parity_of & ~(1u << stage)) | (phase << stage);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (*abort_flag) {  // let our own copies land before the ring is reused
          if (p.wide && half != 0) {  // (counted on the leader's barriers: a fixed 50 us)
            const uint64_t c0 = globaltimer_ns();
            while (globaltimer_ns() - c0 < 50000ull) {
            }
          } else {
            for (int s = 0; s < p.stages; ++s)
              if (filled & (1u << s)) {
                volatile int dummy = 0;
                mbar_wait(&sm.full[s], (parity_of >> s) & 1u, &dummy, nullptr, kFtWaitNs / 4, 0);
              }
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        if (!p.wide || half == 0) {
          int stage = 0;
          uint32_t phase = 0;
          const uint32_t idesc = umma_idesc_bf16(p.wide ? 256 : 128, p.epad);
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&sm.full[stage], phase, abort_flag, nullptr, kFtWaitNs, 71)) break;
            tc_fence_after();
            const uint32_t s = smem_u32(ring + stage * stage_bytes);
            const uint64_t ad = umma_desc_sw128(s), bd = umma_desc_sw128(s + 128 * 128);
            if (p.wide) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16_pair(tmem, ad + 2 * k, bd + 2 * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
              umma_commit_pair(&sm.empty[stage], 3);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16(tmem, ad + 2 * k, bd + 2 * k, idesc, (kb != kb0 || k != 0) ? 1u : 0u);
              umma_commit(&sm.empty[stage]);
            }
            if (++stage == p.stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (p.wide) umma_commit_pair(&sm.tfull, 3);
          else umma_commit(&sm.tfull);
        }
        if (!mbar_wait(&sm.tfull, 0, abort_flag, nullptr, kFtWaitNs, 72)) {  // (aborted: the MMAs issued end still)
          volatile int dummy = 0;
          mbar_wait(&sm.tfull, 0, &dummy, nullptr, kFtWaitNs, 0);
        }
      }
      __syncwarp();
    }
    __syncthreads();  // the ring is idle
    tc_fence_after();
    // accumulator -> partial sums: warps of a lane quarter take every fourth run of 32 experts
    const int q4 = warp & 3, m = q4 * 32 + lane;
    for (int c0 = (warp >> 2) * 32; c0 < p.epad; c0 += kRsWarps / 4 * 32) {
      float v[32];
      tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q4 * 32) << 16) + c0, v);
      if (kb1 == kb0) {  // no K block of its own: nothing was accumulated
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        if (c0 + j < p.epad)
          *reinterpret_cast<float4*>(part + m * pitch + c0 + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
    tc_fence_before();
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    tc_fence_after();
    if (!p.wide && warp == 1) tmem_dealloc(tmem, cols);
    // own tokens: the sum over the cluster in rank order, in place (no peer reads these rows)
    const int e4 = p.epad / 4;
    if (C > 1 || p.bias != nullptr)
      for (int i = tid; i < TC * e4; i += kRsThreads) {
        const int e = (i % e4) * 4;
        float* at = part + (own0 + i / e4) * pitch + e;
        float4 s;
        if (C == 1) {
          s = *reinterpret_cast<const float4*>(at);
        } else {
          const uint32_t addr = smem_u32(at);
          float4 v[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)  // all on their way before the first is added
            if (c < C) v[c] = ld_cluster_f4(mapa_shared(addr, static_cast<uint32_t>(c)));
          s = v[0];
#pragma unroll
          for (int c = 1; c < 8; ++c)
            if (c < C) {
              s.x += v[c].x;
              s.y += v[c].y;
              s.z += v[c].z;
              s.w += v[c].w;
            }
        }
        if (p.bias != nullptr) {
          s.x += e < p.E ? p.bias[e] : 0.f;
          s.y += e + 1 < p.E ? p.bias[e + 1] : 0.f;
          s.z += e + 2 < p.E ? p.bias[e + 2] : 0.f;
          s.w += e + 3 < p.E ? p.bias[e + 3] : 0.f;
        }
        *reinterpret_cast<float4*>(at) = s;
      }
    __syncthreads();
  }

  // ---- a warp per token
  ChoiceSetup<NI> cs;
  cs.load(p, sm.table);
  // (the next token goes to the first warp that is free: some take longer)
  for (int i = warp, after = 0; i < TC; i = __shfl_sync(0xffffffffu, after, 0)) {
    const int t = t0 + own0 + i;
    if (t >= p.M) break;
    if (lane == 0) after = TC > kRsWarps ? atomicAdd(&sm.next, 1) : TC;
    const float* row = part + (own0 + i) * pitch;
    const int a = p.adapter_ids[t];
    if (given) {
      float* mine = part + warp * pitch;
#pragma unroll
      for (int j = 0; j < NI; ++j)
        if (lane + 32 * j < p.E) mine[lane + 32 * j] = p.logits_in[static_cast<size_t>(t) * p.E + lane + 32 * j];
      row = mine;
      __syncwarp();
    }
    float mx, sum;
    bool bad = choose<NI>(row, p, cs, p.logits_out != nullptr ? p.logits_out + static_cast<size_t>(t) * p.E : nullptr,
                          scratch, sm.ids[warp], mx, sum);
    weigh(row, p, sm.ids[warp], t, mx, sum);
    bad |= a < -1 || a >= p.L;
    if (bad && lane == 0) atomicMin(&sm.flag, t);
    const int b = own0 + i;  // the token's bit
    for (int j = lane; j < p.k; j += 32) {
      const int e = sm.ids[warp][j];
      atomicOr(reinterpret_cast<unsigned*>(sm.map + e) + (b >> 5), 1u << (b & 31));
      if (p.tiles == 1) sm.slot[e][i] = static_cast<uint8_t>(j);  // (16 tokens per CTA then)
    }
    __syncwarp();
  }
  __syncthreads();
  if (tid == 0 && *abort_flag) sm.flag = -1;

  if (p.tiles > 1) {
    // ---- for the sort: the chunk's bits and its pairs of lower experts
    const int chunks = p.tiles * C, chunk = static_cast<int>(blockIdx.x);
    int n = 0;
    uint4 m = make_uint4(0u, 0u, 0u, 0u);
    if (tid < p.E) {
      m = sm.map[tid];
      n = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
    }
    const int before = block_prefix(n, sm.scan);
    if (tid < p.E) {
      p.before[static_cast<size_t>(tid) * chunks + chunk] = before;
      uint16_t* dst = p.bitmap + static_cast<size_t>(tid) * p.tiles * 8 + tile * 8 + own0 / 16;
      const uint32_t w[4] = {m.x, m.y, m.z, m.w};
      if (TC == 128) {
        *reinterpret_cast<uint4*>(dst) = m;
      } else if (TC == 64) {
        *reinterpret_cast<uint2*>(dst) = rank == 0 ? make_uint2(m.x, m.y) : make_uint2(m.z, m.w);
      } else if (TC == 32) {
        *reinterpret_cast<uint32_t*>(dst) = w[0] | w[1] | w[2] | w[3];  // one of them is this CTA's
      } else {
        const uint32_t v = w[0] | w[1] | w[2] | w[3];
        *dst = static_cast<uint16_t>(v | v >> 16);
      }
    }
    if (tid == 0) p.flags[chunk] = sm.flag;
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();  // the peers have read this CTA's partial sums
    tc_fence_after();
    if (p.wide && !given && warp == 1) tmem_dealloc_pair(sm.tmem_base, cols);
    return;
  }

  // ---- up to 128 tokens: the cluster sorts, a warp per expert
  pdl_trigger();  // a call behind this one may set itself up
  int* run = reinterpret_cast<int*>(scratch);            // next place by adapter, of this warp
  uint4* s_slot = reinterpret_cast<uint4*>(scratch + 64);  // slots of the tile's tokens, one expert
  int* s_base = reinterpret_cast<int*>(sm.ids);          // pairs of lower experts (the ids are done)
  uint8_t* s_ad = reinterpret_cast<uint8_t*>(sm.ids) + 1024;  // adapters of the tokens
  const int my_ad = tid < p.M ? p.adapter_ids[tid] : -1;      // (of the first 128 threads)
  __syncwarp();
  cluster_sync_all();
  uint4 m = make_uint4(0u, 0u, 0u, 0u);
  int n = 0;
  if (tid < p.E) {
    uint4 v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) v[c] = ld_cluster_u32x4(mapa_shared(smem_u32(sm.map + tid), static_cast<uint32_t>(c)));
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (c < C) m = make_uint4(m.x | v[c].x, m.y | v[c].y, m.z | v[c].z, m.w | v[c].w);
    n = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
  }
  if (rank == 0 && warp == kRsWarps - 1) {  // the call's status word
    int flag = lane < C ? ld_cluster_s32(mapa_shared(smem_u32(&sm.flag), static_cast<uint32_t>(lane))) : kRsClean;
    flag = __reduce_min_sync(0xffffffffu, flag);
    if (lane == 0) {
      p.status[0] = flag == kRsClean ? MOE_LORA_OK : flag < 0 ? MOE_LORA_ERR_TIMEOUT : MOE_LORA_ERR_DEVICE_CHECK;
      p.status[1] = flag == kRsClean || flag < 0 ? 0 : flag;
    }
  }
  uint4* s_map = reinterpret_cast<uint4*>(part);  // tokens by expert, of the whole tile
  const int base = block_prefix(n, sm.scan);
  if (tid < p.E) {
    s_base[tid] = base;
    s_map[tid] = m;
  }
  if (tid < 128) s_ad[tid] = static_cast<uint8_t>(my_ad >= 0 && my_ad < p.L ? my_ad : p.L);
  __syncthreads();
  const int LA = p.L + 1;
  for (int e = rank * kRsWarps + warp; e < p.E; e += C * kRsWarps) {
    const unsigned* w = reinterpret_cast<const unsigned*>(s_map + e);
    if (lane < C)  // the tokens' slots, 16 from every CTA
      s_slot[lane] = ld_cluster_u32x4(mapa_shared(smem_u32(sm.slot[e]), static_cast<uint32_t>(lane)));
    for (int a = lane; a < LA; a += 32) run[a] = 0;
    __syncwarp();
    int pair[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = q * 32 + lane;
      pair[q] = w[q] >> lane & 1u ? t * p.k + reinterpret_cast<const uint8_t*>(s_slot)[t] : -1;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (w[q] >> lane & 1u) atomicAdd(run + s_ad[q * 32 + lane], 1);
    __syncwarp();
    warp_offsets(run, LA, s_base[e], p.seg_offsets + e * LA);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (w[q] != 0u) place32(p, pair[q] >= 0, pair[q], s_ad[q * 32 + lane], run);
  }
  if (rank == 0 && tid == 0) p.seg_offsets[p.E * LA] = p.M * p.k;
  __syncwarp();
  cluster_sync_all();  // the peers have read this CTA's maps, slots and flag
}

// ------------------------------------------------------------------ sort of large batches
// A CTA per expert; its warps split the expert's words of 32 tokens and compact the set bits
// of up to 32 words at a time into a list, so that sparse experts cost loads for their own
// pairs only and an expert that every token chose is spread over the CTA.  Two walks: count
// by adapter, then place in token order.
constexpr int kRsList = 1024;  // tokens of 32 words

__global__ void __launch_bounds__(kRsThreads) route_scored_sort_kernel(const RsParams p) {
  extern __shared__ uint32_t s_lists[];  // [kRsWarps][kRsList]: token | slot << 10 | adapter << 18
  __shared__ int s_scan[kRsWarps];
  __shared__ int s_run[kRsWarps][65];
  __shared__ int s_off[65];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int e = blockIdx.x, LA = p.L + 1;
  const int words = p.tiles * 4, chunks = p.tiles * p.C;
  for (int i = tid; i < kRsWarps * 65; i += kRsThreads) (&s_run[0][0])[i] = 0;
  pdl_wait();
  // pairs of lower experts
  int part = 0;
  for (int c = tid; c < chunks; c += kRsThreads) part += p.before[static_cast<size_t>(e) * chunks + c];
  part = __reduce_add_sync(0xffffffffu, part);
  if (lane == 0) s_scan[warp] = part;
  if (e == 0 && warp == 0) {  // the call's status word
    int flag = kRsClean;
    for (int c = lane; c < chunks; c += 32) flag = min(flag, p.flags[c]);
    flag = __reduce_min_sync(0xffffffffu, flag);
    if (lane == 0) {
      p.status[0] = flag == kRsClean ? MOE_LORA_OK : flag < 0 ? MOE_LORA_ERR_TIMEOUT : MOE_LORA_ERR_DEVICE_CHECK;
      p.status[1] = flag == kRsClean || flag < 0 ? 0 : flag;
    }
  }
  const uint32_t* map = reinterpret_cast<const uint32_t*>(p.bitmap) + static_cast<size_t>(e) * words;
  const int w0 = static_cast<int>(static_cast<long long>(words) * warp / kRsWarps);
  const int w1 = static_cast<int>(static_cast<long long>(words) * (warp + 1) / kRsWarps);
  uint32_t* list = s_lists + warp * kRsList;
  int n = 0;
  // the tokens of words [r, min(r + 32, w1)) in order, with their slots and adapters
  auto compact = [&](int r) {
    uint32_t w = r + lane < w1 ? map[r + lane] : 0u;
    const int c = __popc(w);
    int incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    n = __shfl_sync(0xffffffffu, incl, 31);
    __syncwarp();
    for (int at = incl - c; w != 0u; ++at, w &= w - 1u) list[at] = static_cast<uint32_t>(lane * 32 + __ffs(w) - 1);
    __syncwarp();
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
      const int t = r * 32 + static_cast<int>(list[i]);
      const int a = p.adapter_ids[t];
      list[i] |= static_cast<uint32_t>(slot_of_expert(p.topk_ids, t, p.k, e)) << 10 |
                 static_cast<uint32_t>(a >= 0 && a < p.L ? a : p.L) << 18;
    }
    __syncwarp();
  };
  __syncthreads();
  int base = 0;
#pragma unroll
  for (int w = 0; w < kRsWarps; ++w) base += s_scan[w];
  for (int r = w0; r < w1; r += 32) {
    compact(r);
    for (int i = lane; i < n; i += 32) atomicAdd(&s_run[warp][list[i] >> 18], 1);
  }
  __syncthreads();
  if (tid < LA) {  // counts of the expert by adapter; s_run: the warps' exclusive prefix
    int acc = 0;
#pragma unroll
    for (int w = 0; w < kRsWarps; ++w) {
      const int c = s_run[w][tid];
      s_run[w][tid] = acc;
      acc += c;
    }
    s_off[tid] = acc;
  }
  __syncthreads();
  if (warp == 0) {
    warp_offsets(s_off, LA, base, p.seg_offsets + e * LA);
    if (e == p.E - 1 && lane == 0) p.seg_offsets[p.E * LA] = p.M * p.k;
  }
  __syncthreads();
  for (int a = lane; a < LA; a += 32) s_run[warp][a] += s_off[a];
  __syncwarp();
  pdl_trigger();  // a call behind this one may set itself up
  for (int r = w0; r < w1; r += 32) {
    if (w1 - w0 > 32) compact(r);
    for (int i0 = 0; i0 < n; i0 += 32) {
      const bool in = i0 + lane < n;
      const uint32_t o = in ? list[i0 + lane] : 0u;
      const int t = r * 32 + static_cast<int>(o & 1023u);
      place32(p, in, t * p.k + static_cast<int>(o >> 10 & 255u), static_cast<int>(o >> 18), s_run[warp]);
    }
  }
}

// ------------------------------------------------------------------ host
// CTAs per tile of 128 tokens: as many as keep one CTA per SM, 8 at most.  One: CTA pairs, an
// even count of tiles.  (The workspace's layout follows it and is sized without a device, so the
// B200's SMs are a constant here: on fewer the clusters queue.)
constexpr int kRsSms = 148;

static int scored_split(int M) {
  const int tiles = (M + 127) / 128;
  int C = 8;
  while (C > 1 && tiles * C > kRsSms) C /= 2;
  return C;
}

void route_scored_scratch(int M, int E, size_t* bitmap, size_t* before, size_t* flags) {
  const size_t tiles = M <= 128 ? 1 : (static_cast<size_t>(M) + 255) / 256 * 2;
  const size_t chunks = std::max<size_t>(tiles, std::min<size_t>(8 * tiles, kRsSms));  // or more: grows with M
  *bitmap = tiles > 1 ? E * tiles * 16 : 0;
  *before = tiles > 1 ? E * chunks * 4 : 0;
  *flags = tiles > 1 ? chunks * 4 : 0;
}

template <int NI>
static cudaError_t launch_choice(const RsParams& p, const CUtensorMap& tmx, const CUtensorMap& tmw, cudaStream_t st) {
  const int pitch = p.epad + 4;
  const size_t rows = p.logits_in ? kRsWarps : 128;
  size_t body = rows * pitch * 4 + static_cast<size_t>(kRsWarps) * p.epad * 16;
  if (!p.logits_in) body = std::max(body, static_cast<size_t>(p.stages) * (128 + p.epad / (p.wide ? 2 : 1)) * 128);
  static std::atomic<bool> attr_set[kMaxDevices];
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    const cudaError_t e = cudaFuncSetAttribute(route_scored_kernel<NI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               1024 + kRsBody);
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  ProfScope ps(K_ROUTE_SCORED, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.tiles * p.C);
  cfg.blockDim = dim3(kRsThreads);
  cfg.dynamicSmemBytes = 1024 + body;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.wide ? 2 : p.C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, route_scored_kernel<NI>, tmx, tmw, p);
  count_launch();
  return e;
}

cudaError_t launch_route_scored(const RouteScoredArgs& a, cudaStream_t st) {
  if (a.M == 0) {
    const cudaError_t e = cudaMemsetAsync(a.status, 0, 8, st);
    return e != cudaSuccess ? e : cudaMemsetAsync(a.seg_offsets, 0, sizeof(int32_t) * (a.E * (a.L + 1) + 1), st);
  }
  RsParams p{};
  p.logits_in = a.logits_in;
  p.bias = a.bias;
  p.score_bias = a.score_bias;
  p.adapter_ids = a.adapter_ids;
  p.logits_out = a.logits_out;
  p.topk_ids = a.topk_ids;
  p.topk_w = a.topk_w;
  p.sorted_pairs = a.sorted_pairs;
  p.seg_offsets = a.seg_offsets;
  p.bitmap = a.bitmap;
  p.before = a.before;
  p.flags = a.flags;
  p.status = a.status;
  p.M = a.M;
  p.H = a.H;
  p.E = a.E;
  p.k = a.k;
  p.L = a.L;
  p.C = scored_split(a.M);
  p.tiles = (a.M + 127) / 128;
  p.epad = std::max(48, (a.E + 15) / 16 * 16);  // (the sort's 65 counters and 128 slots fit a warp's scratch)
  p.wide = p.C == 1;
  if (p.wide) p.tiles = (p.tiles + 1) & ~1;
  p.stages = std::min(kRsMaxStages, kRsRing / ((128 + p.epad / (p.wide ? 2 : 1)) * 128));
  p.f = a.f;
  CUtensorMap tmx{}, tmw{};
  if (a.logits_in == nullptr &&
      (encode_tmap_2d(&tmx, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.x, a.H, a.M, static_cast<uint64_t>(a.H) * 2, 64, 128,
                      CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
       encode_tmap_2d(&tmw, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.w_router, a.H, a.E, static_cast<uint64_t>(a.H) * 2, 64,
                      p.wide ? p.epad / 2 : p.epad, CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS))
    return cudaErrorInvalidValue;
  cudaError_t e = a.E <= 64    ? launch_choice<2>(p, tmx, tmw, st)
                  : a.E <= 128 ? launch_choice<4>(p, tmx, tmw, st)
                               : launch_choice<8>(p, tmx, tmw, st);
  if (e != cudaSuccess || p.tiles == 1) return e != cudaSuccess ? e : cudaGetLastError();
  constexpr size_t sort_smem = sizeof(uint32_t) * kRsWarps * kRsList;
  static std::atomic<bool> attr_set[kMaxDevices];
  const int dev = current_device_index();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(route_scored_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(sort_smem));
    if (e != cudaSuccess) return e;
    attr_set[dev].store(true, std::memory_order_release);
  }
  ProfScope ps(K_SORT, st);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.E);
  cfg.blockDim = dim3(kRsThreads);
  cfg.dynamicSmemBytes = sort_smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, route_scored_sort_kernel, p);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mlb
