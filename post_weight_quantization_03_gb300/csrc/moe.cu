// Routing tokens to experts, and the weighted sum of what the experts give.
//
// Routing: s = softmax or sigmoid of a token's logits, c = s + bias, the best groups by the sum of
// their largest c, the top_k largest c among those; weights from s; then the assignments (token *
// top_k + place) sorted by expert.
//
// A warp takes a token; a lane holds `each` experts next to one another, so that a group is a run of
// lanes where its size allows.  Each of the top_k rounds is a maximum over the lane's own and one
// over the warp, of integers that are ordered as the c (redux; the lowest lane of equals has the
// lowest index).  c is taken in fp32, and where two that decide something lie nearer to one
// another than its error bound fp64 decides.  That is slow here (two operations a cycle and SM), so the
// bound is tight, and of sigmoids only the few in question are taken again, one in a lane; a softmax's
// need the sum, and so all (30 us for a token that meets it).  Without a bias the order of
// the c is that of the logits, which are compared themselves.  Between groups the bound is one for each,
// by the magnitudes of the c that it sums: these may cancel.
//
// The sort is a count by expert and chunk of tokens, then for each chunk the sum of the counts before
// it.  Within 64 tokens an assignment's place among its expert's is the number of lower bits in the
// expert's word of tokens, so that the result does not depend on how the GPU schedules it.  Two
// launches, or one for up to 32 tokens.
//
// Measured (GPU time): 1 token of 64 experts 4.2 us and 333 of 160 8.1, launches and latencies; 8192 of
// 256 16 us by logits and 23 by sigmoids with a bias and groups, by issue slots (1000 and 1610
// instructions a token, of which 450 are the eight rounds) and the order's latencies (5 us); 39 by a softmax
// with a bias and groups, whose tokens that fp32 does not tell are taken again whole.
//
// Combine: HBM-bound, one pass: 4096 x 8 rows of 4096 48 us, 6.9 TB/s of operands and outputs (some of which
// are still in L2 when it ends); one token 1.8 us.
#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

using fp8::kVec;
using fp8::Raw8;

constexpr int kMaxChunks = 152;       // of tokens: one for each SM of a GB300 (the workspace's size asks no device)
constexpr int kWord = 64;             // tokens that are sorted at once
constexpr int kPlanThreads = 1024;
constexpr int kOneTokens = 32;        // up to these, one CTA does everything

struct RouteParams {
  const void *logits; int dtype; int64_t ld;
  int64_t n_tokens; int n_experts, top_k;
  const float *bias;
  int sigmoid, groups, top_groups, group_top, renormalize;
  int size;                           // experts of a group
  int each;                           // experts of a lane
  int whole;                          // all lanes have VPL, in rows of 16-byte alignment
  int bias_whole;                     // so does the bias
  int lanes, shift;                   // lanes of a group, 1 << shift; 0: groups do not begin at lanes
  float scale;
  int32_t *ids; float *weights; int32_t *offsets, *order;
  uint32_t *counts;                   // [chunks, pairs]: of two neighbouring experts, 16 bits each (a
                                      // chunk has at most 2^22 / kMaxChunks tokens)
  int pairs;
  int chunk;                          // tokens of a chunk
  int chunks;
};

// Integers in the order of the numbers; none: 0, below all of them.
__device__ __forceinline__ uint32_t to_key(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);   // (-0 counts as 0)
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t to_key(double c) {
  const uint64_t b = (uint64_t)__double_as_longlong(c + 0.0);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double of_key(uint64_t k) {
  return __longlong_as_double((int64_t)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <typename C>
__device__ __forceinline__ C warp_sum(C v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint32_t warp_max_key(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// What a warp found for a token: lane j has the j-th chosen expert (-1: none).
struct Chosen {
  int id;
  float top, sum;   // largest logit; sum of exp(logit - top), where the weights need it
};

// (the type at run time: a kernel is a long one, and reads a few numbers a lane)
__device__ __forceinline__ float logit(const RouteParams &p, int64_t at) {
  if (p.dtype == GPTQ_F32) return ((const float *)p.logits)[at];
  if (p.dtype == GPTQ_F16) return to_f32(((const __half *)p.logits)[at]);
  return to_f32(((const __nv_bfloat16 *)p.logits)[at]);
}
// A sigmoid's c in fp64.
__device__ __forceinline__ double exact_c(const RouteParams &p, int64_t t, int id) {
  return 1.0 / (1.0 + exp(-(double)logit(p, t * p.ld + id))) + (p.bias ? (double)p.bias[id] : 0.0);
}

// The order of a few experts whose c, of sigmoids, are too near to one another: the first n lanes' `id`.
// In fp64, one in a lane.
__device__ __forceinline__ int sort_near(const RouteParams &p, int64_t t, int lane, int id, int n) {
  uint64_t key = 0;
  if (lane < n) {
    key = to_key(exact_c(p, t, id));
  }
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const uint64_t k = __shfl_sync(0xffffffffu, key, j);
    const int i = __shfl_sync(0xffffffffu, id, j);
    rank += k > key || (k == key && i < id);
  }
  int mine = -1;
  for (int j = 0; j < p.top_k; ++j) {
    const uint32_t who = __ballot_sync(0xffffffffu, lane < n && rank == j);
    const int i = __shfl_sync(0xffffffffu, id, who ? __ffs(who) - 1 : 0);
    if (lane == j && who) mine = i;
  }
  return mine;
}

// The groups that are looked at, of sigmoids, by values in fp64 of the group_top + 1 largest c of each
// (`score`: keys of this lane's c): one more than counts, and one in each of the group's lanes.  False
// where the next one may belong to these too.
template <int VPL>
__device__ __forceinline__ bool exact_groups(uint32_t (&score)[VPL], const RouteParams &p, int64_t t, int lane, float tau,
                                             uint32_t &open) {
  const int rank = lane & (p.lanes - 1), base = lane - rank, n = p.group_top + 1;
  const uint32_t group = (p.lanes == 32 ? 0xffffffffu : (1u << p.lanes) - 1) << base;
  int id[3] = {-1, -1, -1};
  float first = 0.0f, last = 0.0f;   // the largest c, and the last that counts
  bool told = true;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if (r > n) break;
    uint32_t mine = score[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) mine = max(mine, score[i]);
    uint32_t best = mine;
    for (int o = 1; o < p.lanes; o *= 2) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    const uint32_t who = __ballot_sync(0xffffffffu, best != 0 && mine == best) & group;
    int at = 0;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i) at = score[i] == best ? i : at;
    const int found = __shfl_sync(0xffffffffu, lane * p.each + at, who ? __ffs(who) - 1 : lane);
    if (who && lane == __ffs(who) - 1) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) score[i] = i == at ? 0 : score[i];
    }
    if (!who) continue;
    const float c = of_key(best);
    if (r == 0) first = c;
    if (r == p.group_top - 1) last = c;
    if (r < 3 && r < n) id[r] = found;
    if (r == n) told = last - c > tau + 0x1p-23f * fmaxf(fabsf(first), fabsf(c));
  }
  if (!__all_sync(0xffffffffu, told)) return false;
  uint64_t a = 0, b = 0;              // the two largest of the group
  for (int r0 = 0; r0 < n; r0 += p.lanes) {
    const int r = r0 + rank, mine = r == 0 ? id[0] : r == 1 ? id[1] : r == 2 && n > 2 ? id[2] : -1;
    const uint64_t k = mine >= 0 ? to_key(exact_c(p, t, mine)) : 0;
    b = max(b, min(a, k));
    a = max(a, k);
  }
  for (int o = 1; o < p.lanes; o *= 2) {
    const uint64_t oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    b = max(min(a, oa), max(b, ob));
    a = max(a, oa);
  }
  uint64_t value = p.group_top > 1 && b ? to_key(of_key(a) + of_key(b)) : a;
  if (rank != 0 || lane >= p.lanes * p.groups) value = 0;
  open = 0;
  for (int j = 0; j < p.top_groups; ++j) {
    const uint64_t best = warp_max_key(value);
    if (best == 0) break;
    const int w = __ffs(__ballot_sync(0xffffffffu, value == best)) - 1;
    open |= 1u << (w >> p.shift);
    if (lane == w) value = 0;
  }
  return true;
}

// A whole warp chooses token t's experts from its logits x (-inf: not to be chosen), c in type C; false
// where fp32 does not tell.  EXACT: not for groups of sigmoids that lie near to one another, which are
// then compared in fp64.
template <typename C, int VPL, bool EXACT = false>
__device__ __forceinline__ bool choose(const float (&x)[VPL], const RouteParams &p, int64_t t, int lane, Chosen &out) {
  using K = typename std::conditional<std::is_same<C, float>::value, uint32_t, uint64_t>::type;
  constexpr bool kSingle = std::is_same<C, float>::value;
  const bool by_logit = !p.bias;                        // the order of the c is that of the logits
  const bool scored = !by_logit || (p.groups > 1 && p.group_top > 1);
  bool sure = true;
  const int e0 = lane * p.each;
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) top = fmaxf(top, x[i]);
  top = warp_max(top);
  out.top = top;
  C c[VPL], sum = 0;
  if (!p.sigmoid && (scored || !p.renormalize)) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = x[i] > -INFINITY ? (C)exp((C)x[i] - (C)top) : (C)0;
      sum += c[i];
    }
    sum = warp_sum(sum);
  }
  out.sum = (float)sum;
  // Error of an fp32 c, both sides of a comparison.  A sigmoid's, from the quick functions: the
  // exponential's 2^-22 and what rounding its argument does, 1.44 |x| 2^-24, of which s (1 - s) gets
  // through: 2^-24 in all at most; the sum 2^-24, the reciprocal 2^-23.  A softmax's, relative to s, which
  // is at most 1 / sum: VPL + 5 additions, the exponential's 2^-22 and what rounding its argument x
  // does, x e^x <= 0.37, the reciprocal and the product.  And the addition of the bias, 2^-24 |c|.
  const float tau = p.sigmoid ? 4 * 0x1p-23f : (VPL + 15) * 0x1p-23f / (float)sum;
  if (scored) {
    const C inv = (C)1 / sum;
    float bias[VPL] = {};
    if (p.bias) {
      if (VPL % 4 == 0 && p.bias_whole) {
#pragma unroll
        for (int i = 0; i < VPL; i += 4) {
          const float4 b = *reinterpret_cast<const float4 *>(p.bias + e0 + i);
          bias[i] = b.x, bias[i + 1] = b.y, bias[i + 2] = b.z, bias[i + 3] = b.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPL; ++i) bias[i] = e0 + i < p.n_experts && i < p.each ? p.bias[e0 + i] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      C s;
      if constexpr (kSingle) s = p.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-x[i])) : c[i] * inv;
      else s = p.sigmoid ? 1.0 / (1.0 + exp(-(double)x[i])) : c[i] / sum;
      c[i] = x[i] > -INFINITY && fp8::finite(bias[i]) ? s + (C)bias[i] : -(C)INFINITY;
    }
  }
  K key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (by_logit) key[i] = x[i] > -INFINITY ? to_key((C)x[i]) : 0;
    else key[i] = c[i] > -(C)INFINITY ? to_key(c[i]) : 0;
  }
  if (p.groups > 1) {
    // the group's value in its first lane (or in the lane of its number); 0: nothing to choose in it
    const bool sums = p.group_top > 1;
    K value = 0;
    auto join = [&](K &a, K &b, K oa, K ob) {
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    };
    // with sums of scores the keys compared are the scores'; else those of the choice itself
    auto key_of = [&](int i) -> K { return !by_logit || !sums ? key[i] : key[i] ? to_key(c[i]) : 0; };
    auto value_of = [&](K a, K b) -> K { return sums && b ? to_key(of_key(a) + of_key(b)) : a; };
    // Error of a value in fp32: that of each c in it (tau / 2), and 2^-24 of their magnitudes for the
    // addition of the bias, of the sum, and of what is compared below.  Of the summands' magnitudes: where
    // biases of opposite signs cancel the sum's is far below what rounding them left.  (Finite, though
    // the sum may not be.)
    auto error_of = [&](K a, K b) -> float {
      constexpr float k = 0x1.9p-23f;   // (3 2^-24, and its own rounding)
      return (sums ? tau : 0.5f * tau) + k * fabsf((float)of_key(a)) + (sums && b ? k * fabsf((float)of_key(b)) : 0.0f);
    };
    float error = 0.0f;
    if (p.lanes > 0) {
      K a = 0, b = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) join(a, b, key_of(i), 0);
      for (int o = 1; o < p.lanes; o *= 2) join(a, b, __shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o));
      value = value_of(a, b);
      if constexpr (kSingle) error = error_of(a, b);
      if ((lane & (p.lanes - 1)) != 0 || lane >= p.lanes * p.groups) value = 0;
    } else {
      for (int g = 0; g < p.groups; ++g) {
        K a = 0, b = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (i < p.each && e0 + i >= g * p.size && e0 + i < (g + 1) * p.size) join(a, b, key_of(i), 0);
#pragma unroll
        for (int o = 16; o; o >>= 1) join(a, b, __shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o));
        if (lane == g) {
          value = value_of(a, b);
          if constexpr (kSingle) error = error_of(a, b);
        }
      }
    }
    uint32_t open = 0;
    const K valued = value;
    for (int j = 0; j < p.top_groups; ++j) {
      const K best = warp_max_key(value);
      if (best == 0) break;
      const int w = __ffs(__ballot_sync(0xffffffffu, value == best)) - 1;
      open |= 1u << (p.lanes > 0 ? w >> p.shift : w);
      if (lane == w) value = 0;
    }
    if constexpr (kSingle)
      if (!by_logit || sums) {
        // fp32 tells if the least that an open group may have is above the most of all others.  (A value
        // past fp32's range is at least, or at most, its largest number.)
        constexpr float kLargest = 0x1.fffffep127f;
        const float v = of_key(valued);
        const uint32_t least = valued && !value ? to_key(fminf(v, kLargest) - error) : 0xffffffffu;
        const uint32_t most = value ? to_key(fmaxf(v, -kLargest) + error) : 0;
        sure = __reduce_min_sync(0xffffffffu, least) > __reduce_max_sync(0xffffffffu, most);
      }
    if constexpr (EXACT)
      if (!sure && p.sigmoid && p.lanes > 0) {
        uint32_t score[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) score[i] = key_of(i);
        sure = exact_groups(score, p, t, lane, tau, open);
      }
    if (p.lanes > 0) {
      const bool in = open >> (lane >> p.shift) & 1;
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = in ? key[i] : 0;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (!(open >> ((e0 + i) / p.size & 31) & 1)) key[i] = 0;
    }
  }
  out.id = -1;
  if (!sure) return false;
  // fp32: rounds go on past top_k while the next is too near to the last, so that what is not among
  // these cannot be chosen
  const bool watch = kSingle && !by_logit;
  float last = 0.0f, gap = INFINITY, size = 0.0f;   // c of the round before; the least between two; the largest |c|
  const auto bound = [&]() { return tau + 0x1p-23f * size; };
  int j = 0;
  for (; j < (watch ? 32 : p.top_k); ++j) {
    K mine = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) mine = max(mine, key[i]);
    const K best = warp_max_key(mine);
    if (best == 0) break;
    if (watch) {
      const float c1 = (float)of_key(best);
      size = fmaxf(size, fabsf(c1));
      if (j > 0) {
        if (j >= p.top_k && last - c1 > bound()) break;
        gap = fminf(gap, last - c1);
      }
      last = c1;
    }
    const int w = __ffs(__ballot_sync(0xffffffffu, mine == best)) - 1;
    int at = 0;
    if (lane == w) {
      // the first of the lane's that has it is taken
#pragma unroll
      for (int i = VPL - 1; i >= 0; --i) at = key[i] == best ? i : at;
#pragma unroll
      for (int i = 0; i < VPL; ++i) key[i] = i == at ? 0 : key[i];
    }
    at = __shfl_sync(0xffffffffu, at, w);
    if (lane == j) out.id = w * p.each + at;
  }
  if (watch && (gap <= bound() || (j == 32 && p.n_experts > 32))) {
    if (!p.sigmoid || j == 32) return false;   // (32 rounds without an end may have left one out)
    out.id = sort_near(p, t, lane, out.id, j);
  }
  if (lane >= p.top_k) out.id = -1;
  return true;
}

// A lane's logits; -inf for what is not finite.
template <typename T, int VPL>
__device__ __forceinline__ void load_logits_of(float (&x)[VPL], const RouteParams &p, int64_t t, int lane) {
  const T *row = (const T *)p.logits + t * p.ld + lane * p.each;
  if (VPL % kVec == 0 && p.whole) {   // 16 bytes at a time
#pragma unroll
    for (int j = 0; j < VPL / kVec; ++j) {
      Raw8<T> q;
      q.load(row + kVec * j, kVec, 16);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[kVec * j + i] = q.get(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) x[i] = i < p.each && lane * p.each + i < p.n_experts ? to_f32(row[i]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) x[i] = fp8::finite(x[i]) ? x[i] : -INFINITY;
}
template <int VPL>
__device__ __forceinline__ void load_logits(float (&x)[VPL], const RouteParams &p, int64_t t, int lane) {
  if (p.dtype == GPTQ_F32) load_logits_of<float>(x, p, t, lane);
  else if (p.dtype == GPTQ_F16) load_logits_of<__half>(x, p, t, lane);
  else load_logits_of<__nv_bfloat16>(x, p, t, lane);
}

// The weight of this lane's chosen expert, whose logit is x.
__device__ __forceinline__ float weight_of(const Chosen &ch, float x, const RouteParams &p) {
  const bool any = ch.id >= 0;
  if (!p.renormalize) {
    const float s = p.sigmoid ? 1.0f / (1.0f + expf(-x)) : expf(x - ch.top) / ch.sum;
    return any ? s * p.scale : 0.0f;
  }
  // Relative to the largest chosen, so that not all can vanish: exactly so for a softmax; a
  // sigmoid of less than -60 is exp(x) to 2^-86.
  const float top = warp_max(any ? x : -INFINITY);
  const float s = !any ? 0.0f : (p.sigmoid && top > -60.0f) ? 1.0f / (1.0f + expf(-x)) : expf(x - top);
  const float sum = warp_sum(s);
  return any ? s / sum * p.scale : 0.0f;
}

// This lane's expert of the token (-1: none); -2 in all lanes, and nothing written, where fp32 does not
// tell, unless AGAIN.
template <int VPL, bool AGAIN>
__device__ __forceinline__ int route_token(const RouteParams &p, int64_t t, int lane) {
  float x[VPL];
  load_logits(x, p, t, lane);
  Chosen ch;
  if (!choose<float, VPL, AGAIN>(x, p, t, lane, ch)) {
    if constexpr (!AGAIN) return -2;
    const float sum = ch.sum;
    choose<double, VPL>(x, p, t, lane, ch);
    ch.sum = sum;
  }
  const float of = ch.id >= 0 ? logit(p, t * p.ld + ch.id) : 0.0f;
  const float w = weight_of(ch, of, p);
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = ch.id;
    p.weights[t * p.top_k + lane] = w;
  }
  return ch.id;
}

// The order of a chunk's assignments (kPlanThreads threads).
struct PlanSmem {
  uint32_t word[2][1024];       // of each expert: which of 64 tokens go to it
  int at[1024];                 // where its next assignment goes
  int part[4][kPlanThreads];    // of two neighbouring experts: all, those before
  int warp[32];
};

// The words of the assignments [i0, i1), which belong to the 64 tokens from t0 on; e: the expert of this
// thread's first.
__device__ __forceinline__ void fill_words(const RouteParams &p, const int *ids, int i0, int i1, int t0, int e, PlanSmem &sm) {
  for (int x = threadIdx.x; x < p.n_experts; x += kPlanThreads) sm.word[0][x] = sm.word[1][x] = 0;
  __syncthreads();
  for (int i = i0 + threadIdx.x; i < i1;) {
    const int t = i / p.top_k - t0;
    if (e >= 0) atomicOr(&sm.word[t >> 5][e], 1u << (t & 31));
    i += kPlanThreads;
    e = i < i1 ? ids[i] : -1;
  }
  __syncthreads();
}

__device__ __forceinline__ void plan(const RouteParams &p, int mine, const int *ids, PlanSmem &sm) {
  const int tid = threadIdx.x, lane = tid % 32;
  const int t0 = mine * p.chunk, t1 = min(t0 + p.chunk, (int)p.n_tokens);
  auto expert_of = [&](int i, int end) { return i < end ? ids[i] : -1; };
  // (asked for before the counts, all of which are asked for at once as far as they are a few: either
  // takes 0.5 us to come)
  const int end0 = min(t0 + kWord, t1) * p.top_k, e0 = expert_of(t0 * p.top_k + tid, end0);
  // an expert's assignments in all chunks, and in those before this one
  int span = 32;              // threads of a part: each has two experts, and every parts-th chunk
  while (span < p.pairs) span *= 2;
  const int parts = kPlanThreads / span, part = tid / span, e2 = tid % span;
  int all[2] = {0, 0}, pre[2] = {0, 0};
  if (p.chunks > 1 && e2 < p.pairs) {
    auto add_up = [&](auto batch) {
      constexpr int n = decltype(batch)::value;
      for (int c0 = part; c0 < p.chunks; c0 += n * parts) {
        const uint32_t *from = p.counts + c0 * p.pairs + e2;
        const int step = parts * p.pairs;
        uint32_t two[n];
#pragma unroll
        for (int i = 0; i < n; ++i) two[i] = c0 + i * parts < p.chunks ? from[i * step] : 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const uint32_t before = c0 + i * parts < mine ? two[i] : 0;
          all[0] += two[i] & 0xffffu;
          all[1] += two[i] >> 16;
          pre[0] += before & 0xffffu;
          pre[1] += before >> 16;
        }
      }
    };
    // (152 chunks by the 8 parts of 256 experts are 19; batches of 20 cost 1 us more where there are 3)
    if (p.chunks <= 4 * parts) add_up(std::integral_constant<int, 4>());
    else if (p.chunks <= 8 * parts) add_up(std::integral_constant<int, 8>());
    else add_up(std::integral_constant<int, 20>());
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    sm.part[h][tid] = all[h];
    sm.part[2 + h][tid] = pre[h];
  }
  fill_words(p, ids, t0 * p.top_k, end0, t0, e0, sm);   // (and waits for all)
  int sum = 0, before = 0;
  if (tid < p.n_experts) {
    if (p.chunks == 1) {
      sum = __popc(sm.word[0][tid]) + __popc(sm.word[1][tid]);
    } else {
      for (int q = 0; q < parts; ++q) {
        sum += sm.part[tid & 1][q * span + tid / 2];
        before += sm.part[2 + (tid & 1)][q * span + tid / 2];
      }
    }
  }
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sm.warp[tid / 32] = scan;
  __syncthreads();
  {
    const int w = sm.warp[lane];
    const int below = __reduce_add_sync(0xffffffffu, lane < tid / 32 ? w : 0);
    scan += below;
  }
  if (tid < p.n_experts) {
    sm.at[tid] = scan - sum + before;
    if (mine == 0) {
      p.offsets[tid] = scan - sum;
      if (tid == p.n_experts - 1) p.offsets[tid + 1] = scan;
    }
  }
  const int total = __reduce_add_sync(0xffffffffu, sm.warp[lane]);
  __syncthreads();
  for (int w0 = t0; w0 < t1; w0 += kWord) {
    const int i0 = w0 * p.top_k, i1 = min(w0 + kWord, t1) * p.top_k;
    if (w0 > t0) fill_words(p, ids, i0, i1, w0, expert_of(i0 + tid, i1), sm);
    for (int i = i0 + tid; i < i1; i += kPlanThreads) {
      const int e = ids[i], t = i / p.top_k - w0;
      if (e >= 0) {
        const uint32_t lo = sm.word[0][e];
        const int rank = t < 32 ? __popc(lo & ((1u << t) - 1)) : __popc(lo) + __popc(sm.word[1][e] & ((1u << (t - 32)) - 1));
        p.order[sm.at[e] + rank] = i;
      }
      if (i >= total) p.order[i] = -1;
    }
    __syncthreads();
    if (w0 + kWord < t1 && tid < p.n_experts) sm.at[tid] += __popc(sm.word[0][tid]) + __popc(sm.word[1][tid]);
    // (fill_words waits for all before the words are filled again)
  }
}

// A chunk of tokens for each CTA, a warp for each token in turn; the chunk's counts.
template <int VPL>
__global__ void __launch_bounds__(VPL <= 8 ? 1024 : 512) route_kernel(RouteParams p) {
  __shared__ int count[VPL * 32 + 2];
  for (int e = threadIdx.x; e < VPL * 32 + 2; e += blockDim.x) count[e] = 0;
  wait_for_grids();
  launch_dependents();
  __syncthreads();
  const int lane = threadIdx.x % 32;
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
  const int step = blockDim.x / 32, end = (int)min((int64_t)p.chunk, p.n_tokens - t0);
  for (int i0 = threadIdx.x / 32; i0 < end; i0 += 32 * step) {
    uint32_t again = 0;   // of the warp's next 32 tokens: those for fp64 (apart: its registers are not theirs)
    for (int k = 0; k < 32 && i0 + k * step < end; ++k) {
      const int id = route_token<VPL, false>(p, t0 + i0 + k * step, lane);
      if (id == -2) again |= 1u << k;
      else if (id >= 0) atomicAdd(&count[id], 1);
    }
    for (; again; again &= again - 1) {
      const int id = route_token<VPL, true>(p, t0 + i0 + (__ffs(again) - 1) * step, lane);
      if (id >= 0) atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.pairs; e += blockDim.x)
    p.counts[(int64_t)blockIdx.x * p.pairs + e] = (uint32_t)count[2 * e] | (uint32_t)count[2 * e + 1] << 16;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(RouteParams p) {
  __shared__ PlanSmem sm;
  wait_for_grids();
  launch_dependents();
  plan(p, blockIdx.x, p.ids, sm);
}

// Both, for a few tokens.
template <int VPL>
__global__ void __launch_bounds__(kPlanThreads) route_few_kernel(RouteParams p) {
  __shared__ PlanSmem sm;
  __shared__ int ids[kOneTokens * 32];
  wait_for_grids();
  launch_dependents();
  const int lane = threadIdx.x % 32, t = threadIdx.x / 32;
  if (t < p.n_tokens) {
    int id = route_token<VPL, false>(p, t, lane);
    if (id == -2) id = route_token<VPL, true>(p, t, lane);
    if (lane < p.top_k) ids[t * p.top_k + lane] = id;
  }
  __syncthreads();
  plan(p, 0, ids, sm);
}

int chunk_tokens(int64_t n_tokens, int threads) {
  int64_t c = ceil_div(n_tokens, kMaxChunks);
  if (c < threads / 32) c = threads / 32;   // (one for each warp)
  return (int)(c > kWord ? ceil_div(c, kWord) * kWord : c);
}
int route_threads(int64_t n_tokens, int n_experts) { return n_experts > 256 || n_tokens < 2048 ? 512 : 1024; }

template <int VPL>
gptq_status route_of(const RouteParams &p, int threads, cudaStream_t s) {
  if constexpr (VPL <= 8)
    if (p.n_tokens <= kOneTokens)
      return launch_early(route_few_kernel<VPL>, dim3(1), dim3(kPlanThreads), 0, 1, s, p);
  GPTQ_TRY(launch_early(route_kernel<VPL>, dim3((unsigned)p.chunks), dim3(threads), 0, 1, s, p));
  return launch_early(plan_kernel, dim3((unsigned)p.chunks), dim3(kPlanThreads), 0, 1, s, p);
}

// ---------------------------------------------------------------------------------------
// Combine
// ---------------------------------------------------------------------------------------
struct CombineParams {
  const void *y; int64_t ldy;
  const float *weights;
  const void *r; int64_t ldr;
  void *out; int64_t ldo;
  int64_t n_tokens, d;
  int top_k;
  int pieces;               // CTAs of a token
  int vy, vr, vo;           // alignment of each pointer's rows
};

// A thread has eight elements of a token's row; up to eight rows are asked for at once.
template <typename T>
__global__ void __launch_bounds__(256) combine_kernel(CombineParams p) {
  wait_for_grids();
  launch_dependents();
  const int64_t t = blockIdx.x / p.pieces;
  const int64_t c = ((int64_t)(blockIdx.x % p.pieces) * blockDim.x + threadIdx.x) * kVec, n = p.d - c;
  if (n <= 0) return;
  Raw8<T> r;
  if (p.r) r.load((const T *)p.r + t * p.ldr + c, n, p.vr);
  float v[kVec] = {};
  for (int j0 = 0; j0 < p.top_k; j0 += 8) {
    Raw8<T> y[8];
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = 0.0f;
      if (j0 + j < p.top_k) {
        y[j].load((const T *)p.y + (t * p.top_k + j0 + j) * p.ldy + c, n, p.vy);
        w[j] = p.weights[t * p.top_k + j0 + j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w[j] != 0.0f) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = fmaf(w[j], y[j].get(i), v[i]);
      }
  }
  if (p.r) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] += r.get(i);
  }
  Raw8<T> o;
  o.set(v);
  o.store((T *)p.out + t * p.ldo + c, n, p.vo);
}

}  // namespace

size_t moe_route_ws_bytes(int64_t n_tokens, int n_experts, int) {
  if (n_tokens <= kOneTokens && n_experts <= 256) return 256;
  const int chunk = chunk_tokens(n_tokens, route_threads(n_tokens, n_experts));
  return round_up(sizeof(uint32_t) * (size_t)ceil_div(n_tokens, chunk) * ((n_experts + 1) / 2) + 1, 256);
}

gptq_status launch_moe_route(const MoeRouteArgs &g, void *ws, cudaStream_t s) {
  if (g.n_tokens == 0) {
    GPTQ_CUDA_CHECK(cudaMemsetAsync(g.offsets, 0, sizeof(int32_t) * (g.n_experts + 1), s));
    return GPTQ_OK;
  }
  RouteParams p{};
  p.logits = g.logits; p.dtype = g.dtype; p.ld = g.ld;
  p.n_tokens = g.n_tokens; p.n_experts = g.n_experts; p.top_k = g.top_k;
  p.bias = g.bias;
  p.sigmoid = g.sigmoid; p.groups = g.groups; p.top_groups = g.top_groups; p.group_top = g.group_top;
  p.size = g.n_experts / g.groups;
  p.renormalize = g.renormalize; p.scale = g.scale;
  p.ids = g.ids; p.weights = g.weights; p.offsets = g.offsets; p.order = g.order;
  p.counts = (uint32_t *)ws;
  p.pairs = (g.n_experts + 1) / 2;
  p.each = (g.n_experts + 31) / 32;
  p.whole = p.each % kVec == 0 && (p.each & (p.each - 1)) == 0 && 32 * p.each == g.n_experts &&
            fp8::alignment(g.logits, g.ld * (g.dtype == GPTQ_F32 ? 4 : 2)) == 16;
  p.bias_whole = p.whole && fp8::alignment(g.bias, 0) == 16;
  // groups of whole lanes whose number is a power of two are joined by exchanges within them
  if (p.size % p.each == 0 && (p.size / p.each & (p.size / p.each - 1)) == 0) p.lanes = p.size / p.each;
  while (1 << p.shift < p.lanes) ++p.shift;
  const int threads = route_threads(g.n_tokens, g.n_experts);
  p.chunk = g.n_tokens <= kOneTokens && g.n_experts <= 256 ? kOneTokens : chunk_tokens(g.n_tokens, threads);
  p.chunks = (int)ceil_div(g.n_tokens, p.chunk);
  if (p.each == 1) return route_of<1>(p, threads, s);
  if (p.each == 2) return route_of<2>(p, threads, s);
  if (p.each <= 4) return route_of<4>(p, threads, s);
  if (p.each <= 8) return route_of<8>(p, threads, s);
  if (p.each <= 16) return route_of<16>(p, threads, s);
  return route_of<32>(p, threads, s);
}

gptq_status launch_moe_combine(const void *y, int dtype, int64_t ldy, int64_t n_tokens, int top_k,
                               int64_t d, const float *weights, const void *residual, int64_t ldr,
                               void *out, int64_t ldo, cudaStream_t s) {
  if (n_tokens == 0) return GPTQ_OK;
  CombineParams p{};
  p.y = y; p.ldy = ldy;
  p.weights = weights;
  p.r = residual; p.ldr = ldr;
  p.out = out; p.ldo = ldo;
  p.n_tokens = n_tokens; p.d = d; p.top_k = top_k;
  const int64_t es = dtype == GPTQ_F32 ? 4 : 2;
  p.vy = fp8::alignment(y, ldy * es);
  p.vr = fp8::alignment(residual, ldr * es);
  p.vo = fp8::alignment(out, ldo * es);
  const int64_t vecs = ceil_div(d, kVec), threads = vecs < 256 ? ceil_div(vecs, 32) * 32 : 256;
  p.pieces = (int)ceil_div(vecs, threads);
  const int64_t ctas = n_tokens * p.pieces;
  if (ctas > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas), block((unsigned)threads);
  switch (dtype) {
    case GPTQ_F32: return launch_early(combine_kernel<float>, grid, block, 0, 1, s, p);
    case GPTQ_F16: return launch_early(combine_kernel<__half>, grid, block, 0, 1, s, p);
    default: return launch_early(combine_kernel<__nv_bfloat16>, grid, block, 0, 1, s, p);
  }
}

}  // namespace gptq
