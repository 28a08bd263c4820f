// Routing tokens to experts, and the weighted sum of what the experts give.
//
// Routing: s = softmax or sigmoid of a token's logits, c = s + bias, the best groups by the sum of
// their largest c, the top_k largest c among those; weights from s; then the assignments (token *
// top_k + place) sorted by expert.
//
// A warp takes a token: lane l holds the experts l, l + 32, ...; each of the top_k rounds is a
// maximum over the lane's own and one over the warp (redux).  c is taken in fp32, and where two that
// decide something lie nearer to one another than its error bound the token is chosen again in
// fp64.  A softmax without bias and groups is monotone: the logits themselves are compared.
//
// The sort is a count by expert and chunk of tokens, then for each chunk the sum of the counts before
// it; a thread for each expert (or several, by parts) goes through the chunk's assignments in their
// order, so that the result does not depend on how the GPU schedules it.  Two launches, or
// one for up to 32 tokens.  A few bytes a token: bound by the latency of the launches.
//
// Combine: HBM-bound, one pass.
#include <type_traits>

#include "fp8.cuh"

namespace gptq {

namespace {

using fp8::kVec;
using fp8::Raw8;

constexpr int kMaxChunks = 128;       // of tokens, while a chunk's assignments fit kChunkIds
constexpr int kChunkIds = 8192;
constexpr int kPlanThreads = 1024;
constexpr int kOneTokens = 32;        // up to these, one CTA does everything

struct RouteParams {
  const void *logits; int64_t ld;
  int64_t n_tokens; int n_experts, top_k;
  const float *bias;
  int sigmoid, groups, top_groups, group_top, renormalize;
  int size;                           // experts of a group
  float scale;
  int32_t *ids; float *weights; int32_t *offsets, *order;
  uint16_t *counts;                   // [chunks, n_experts]
  int chunk;                          // tokens of a chunk
  int chunks;
};

template <typename C> __device__ __forceinline__ C minus_inf() { return -(C)INFINITY; }

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

// The largest c of the warp and the lowest index that has it (`e` of a lane without one: any).
__device__ __forceinline__ void warp_best(float &c, int &e) {
  const uint32_t b = __float_as_uint(c + 0.0f);  // (-0 counts as 0)
  const uint32_t key = b & 0x80000000u ? ~b : b | 0x80000000u;
  const uint32_t top = __reduce_max_sync(0xffffffffu, key);
  e = (int)__reduce_min_sync(0xffffffffu, key == top ? (uint32_t)e : 0xffffffffu);
  c = __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
}
__device__ __forceinline__ void warp_best(double &c, int &e) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const double oc = __shfl_xor_sync(0xffffffffu, c, o);
    const int oe = __shfl_xor_sync(0xffffffffu, e, o);
    if (oc > c || (oc == c && oe < e)) c = oc, e = oe;
  }
}

// What a warp found for a token: lane j has the j-th chosen expert (-1: none) and its logit.
struct Chosen {
  int id;
  float x;
  float top, sum;   // largest logit; sum of exp(logit - top), where it is asked for
};

// A whole warp chooses a token's experts, c in type C; false where fp32 does not tell.
template <typename C, int VPL>
__device__ __forceinline__ bool choose(const float (&x)[VPL], const RouteParams &p, int lane, Chosen &out) {
  const bool by_logit = !p.bias && p.groups == 1;
  bool sure = true;
  C c[VPL];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) top = fmaxf(top, fp8::finite(x[i]) ? x[i] : -INFINITY);
  top = warp_max(top);
  out.top = top;
  C sum = 0;
  if (!p.sigmoid && (!by_logit || !p.renormalize)) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      c[i] = fp8::finite(x[i]) ? (C)exp((C)x[i] - (C)top) : (C)0;
      sum += c[i];
    }
    sum = warp_sum(sum);
  }
  out.sum = (float)sum;
  // Error of c in fp32, both sides of a comparison: a sigmoid's is at most 4 2^-24 of max(1, |c|)
  // (exp 2 ulp, whose effect is a quarter; sum, quotient, addition of the bias), a softmax's has the
  // sum's (VPL + 5) 2^-24 too.
  const float tau = p.sigmoid ? 0x1p-20f : (VPL + 16) * 0x1p-23f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    if (by_logit) {
      c[i] = fp8::finite(x[i]) ? (C)x[i] : minus_inf<C>();
    } else {
      const C s = p.sigmoid ? (C)1 / ((C)1 + (C)exp(-(C)x[i])) : c[i] / sum;
      const float b = p.bias && e < p.n_experts ? p.bias[e] : 0.0f;
      c[i] = fp8::finite(x[i]) && fp8::finite(b) ? s + (C)b : minus_inf<C>();
    }
  }
  auto near = [&](C hi, C lo, float of) {
    return std::is_same<C, float>::value && !by_logit && lo > minus_inf<C>() &&
           (float)(hi - lo) <= of * tau * fmaxf(1.0f, fmaxf(fabsf((float)hi), fabsf((float)lo)));
  };
  if (p.groups > 1) {
    C mine = minus_inf<C>();
    for (int g = 0; g < p.groups; ++g) {
      C a = minus_inf<C>(), b = minus_inf<C>();
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = i * 32 + lane;
        if (e >= g * p.size && e < (g + 1) * p.size) {
          b = c[i] > a ? a : (c[i] > b ? c[i] : b);
          a = c[i] > a ? c[i] : a;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const C oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
        const C low = oa > a ? a : oa, high = ob > b ? ob : b;
        a = oa > a ? oa : a;
        b = low > high ? low : high;
      }
      if (lane == g) mine = p.group_top == 2 && b > minus_inf<C>() ? a + b : a;
    }
    uint32_t open = 0;
    C last = minus_inf<C>();
    for (int j = 0; j <= p.top_groups && j < p.groups; ++j) {
      C v = mine;
      int g = lane;
      warp_best(v, g);
      if (j == p.top_groups) {
        if (near(last, v, 2.0f)) sure = false;
      } else if (v > minus_inf<C>()) {
        open |= 1u << g;
        if (lane == g) mine = minus_inf<C>();
        last = v;
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!(open >> ((i * 32 + lane) / p.size & 31) & 1) || i * 32 + lane >= p.n_experts) c[i] = minus_inf<C>();
  }
  out.id = -1;
  out.x = 0.0f;
  C last = minus_inf<C>();
  for (int j = 0; j <= p.top_k; ++j) {
    if (j == p.top_k && (by_logit || !std::is_same<C, float>::value)) break;
    C best = c[0];
    int e = lane;
    float of = x[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i)
      if (c[i] > best) best = c[i], e = i * 32 + lane, of = x[i];
    const int own = e;
    warp_best(best, e);
    if (!(best > minus_inf<C>())) break;   // (the same in the whole warp)
    if (j > 0 && near(last, best, 1.0f)) sure = false;
    last = best;
    if (j == p.top_k) break;
    of = __shfl_sync(0xffffffffu, of, e & 31);
    if (lane == j) out.id = e, out.x = of;
    if (own == e) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i * 32 + lane == e) c[i] = minus_inf<C>();
    }
  }
  return sure;
}

template <typename T, int VPL>
__device__ __forceinline__ void load_logits(float (&x)[VPL], const RouteParams &p, int64_t t, int lane) {
  const T *row = (const T *)p.logits + t * p.ld;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    x[i] = e < p.n_experts ? to_f32(row[e]) : -INFINITY;
  }
}

// (apart, so that its registers are not those of every token)
template <typename T, int VPL>
__device__ __noinline__ void choose_again(const RouteParams &p, int64_t t, int lane, Chosen &out) {
  float x[VPL];
  load_logits<T, VPL>(x, p, t, lane);
  const float sum = out.sum;
  choose<double, VPL>(x, p, lane, out);
  out.sum = sum;
}

// The weight of this lane's chosen expert.
__device__ __forceinline__ float weight_of(const Chosen &ch, const RouteParams &p) {
  const bool any = ch.id >= 0;
  if (!p.renormalize) {
    const float s = p.sigmoid ? 1.0f / (1.0f + expf(-ch.x)) : expf(ch.x - ch.top) / ch.sum;
    return any ? s * p.scale : 0.0f;
  }
  // Relative to the largest chosen, so that not all can vanish: exactly so for a softmax; a
  // sigmoid of less than -60 is exp(x) to 2^-86.
  const float top = warp_max(any ? ch.x : -INFINITY);
  const float s = !any ? 0.0f : (p.sigmoid && top > -60.0f) ? 1.0f / (1.0f + expf(-ch.x)) : expf(ch.x - top);
  const float sum = warp_sum(s);
  return any ? s / sum * p.scale : 0.0f;
}

template <typename T, int VPL>
__device__ __forceinline__ int route_token(const RouteParams &p, int64_t t, int lane) {
  float x[VPL];
  load_logits<T, VPL>(x, p, t, lane);
  Chosen ch;
  if (!choose<float, VPL>(x, p, lane, ch)) choose_again<T, VPL>(p, t, lane, ch);
  const float w = weight_of(ch, p);
  if (lane < p.top_k) {
    p.ids[t * p.top_k + lane] = ch.id;
    p.weights[t * p.top_k + lane] = w;
  }
  return ch.id;
}

// A CTA's part of the order: the assignments of chunk `mine`, n of them, go to their places.  `ids`
// has them in shared memory, 16-byte aligned, -1 up to a multiple of four.  kPlanThreads threads, of
// which (part, e) counts and places expert e's in one of `parts` runs of them, and adds up one run of
// the chunks' counts.
struct PlanSmem {
  int a[kPlanThreads], b[kPlanThreads];
  int warp[32];
  int total;
};
__device__ __forceinline__ void plan(const RouteParams &p, int mine, const int *ids, int n, PlanSmem &sm) {
  int span = 32;
  while (span < p.n_experts) span *= 2;
  const int parts = kPlanThreads / span, tid = threadIdx.x, lane = tid % 32;
  const int part = tid / span, e = tid % span;
  const int first = mine * p.chunk * p.top_k;
  const int4 *quads = reinterpret_cast<const int4 *>(ids);
  const int n4 = (n + 3) / 4, q0 = n4 * part / parts, q1 = n4 * (part + 1) / parts;
  int here = 0, all = 0, before = 0;
  for (int q = q0; q < q1; ++q) {
    const int4 v = quads[q];
    here += (v.x == e) + (v.y == e) + (v.z == e) + (v.w == e);
  }
  if (p.chunks == 1) {
    all = here;
  } else if (e < p.n_experts) {
    const int c0 = p.chunks * part / parts, c1 = p.chunks * (part + 1) / parts;
#pragma unroll 16
    for (int c = c0; c < c1; ++c) {
      const int k = p.counts[(int64_t)c * p.n_experts + e];
      all += k;
      before += c < mine ? k : 0;
    }
  }
  sm.a[tid] = all;
  sm.b[tid] = before;
  __syncthreads();
  // threads of part 0: an expert's total, and the sum of those of the experts before it
  int sum = 0, base = 0;
  if (part == 0)
    for (int q = 0; q < parts; ++q) {
      sum += sm.a[q * span + e];
      base += sm.b[q * span + e];
    }
  int scan = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += v;
  }
  if (lane == 31) sm.warp[tid / 32] = scan;   // (warps of other parts: 0)
  __syncthreads();
  for (int w = 0; w < tid / 32 && part == 0; ++w) scan += sm.warp[w];
  if (part == 0) {
    base += scan - sum;
    if (mine == 0 && e < p.n_experts) {
      p.offsets[e] = scan - sum;
      if (e == p.n_experts - 1) p.offsets[e + 1] = scan;
    }
    if (e == p.n_experts - 1) sm.total = scan;
  }
  // where each part's run of an expert begins
  __syncthreads();
  sm.a[tid] = here;
  if (part == 0) sm.b[e] = base;
  __syncthreads();
  int at = sm.b[e];
  for (int q = 0; q < part; ++q) at += sm.a[q * span + e];
  if (here > 0)   // (-1 is nobody's)
    for (int q = q0; q < q1; ++q) {
      const int4 v = quads[q];
      if (v.x == e) p.order[at++] = first + 4 * q;
      if (v.y == e) p.order[at++] = first + 4 * q + 1;
      if (v.z == e) p.order[at++] = first + 4 * q + 2;
      if (v.w == e) p.order[at++] = first + 4 * q + 3;
    }
  for (int i = first + tid; i < first + n; i += kPlanThreads)
    if (i >= sm.total) p.order[i] = -1;
}

// A chunk of tokens for each CTA, a warp for each token in turn; the chunk's counts.
template <typename T, int VPL>
__global__ void __launch_bounds__(VPL <= 8 ? 1024 : 512) route_kernel(RouteParams p) {
  __shared__ int count[VPL * 32];
  for (int e = threadIdx.x; e < p.n_experts; e += blockDim.x) count[e] = 0;
  wait_for_grids();
  launch_dependents();
  __syncthreads();
  const int lane = threadIdx.x % 32;
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk;
  for (int i = threadIdx.x / 32; i < p.chunk && t0 + i < p.n_tokens; i += blockDim.x / 32) {
    const int id = route_token<T, VPL>(p, t0 + i, lane);
    if (id >= 0) atomicAdd(&count[id], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.n_experts; e += blockDim.x)
    p.counts[(int64_t)blockIdx.x * p.n_experts + e] = (uint16_t)count[e];
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(RouteParams p) {
  __shared__ PlanSmem sm;
  __shared__ __align__(16) int ids[kChunkIds];
  wait_for_grids();
  launch_dependents();
  const int64_t first = (int64_t)blockIdx.x * p.chunk * p.top_k, end = p.n_tokens * p.top_k;
  const int n = (int)min((int64_t)p.chunk * p.top_k, end - first);
  for (int i = threadIdx.x; i < ((n + 3) & ~3); i += kPlanThreads) ids[i] = i < n ? p.ids[first + i] : -1;
  __syncthreads();
  plan(p, blockIdx.x, ids, n, sm);
}

// Both, for a few tokens.
template <typename T, int VPL>
__global__ void __launch_bounds__(kPlanThreads) route_few_kernel(RouteParams p) {
  __shared__ PlanSmem sm;
  __shared__ __align__(16) int ids[kOneTokens * 32 + 4];
  wait_for_grids();
  launch_dependents();
  const int lane = threadIdx.x % 32, t = threadIdx.x / 32, n = (int)p.n_tokens * p.top_k;
  if (t < p.n_tokens) {
    const int id = route_token<T, VPL>(p, t, lane);
    if (lane < p.top_k) ids[t * p.top_k + lane] = id;
  }
  if (threadIdx.x < 3) ids[n + threadIdx.x] = -1;
  __syncthreads();
  plan(p, 0, ids, n, sm);
}

int chunk_tokens(int64_t n_tokens, int top_k, int threads) {
  int64_t c = ceil_div(n_tokens, kMaxChunks);
  if (c < threads / 32) c = threads / 32;   // (one for each warp)
  if (c * top_k > kChunkIds) c = kChunkIds / top_k;
  return (int)c;
}
int route_threads(int64_t n_tokens, int n_experts) { return n_experts > 256 || n_tokens < 2048 ? 512 : 1024; }

template <typename T, int VPL>
gptq_status route_of(const RouteParams &p, int threads, cudaStream_t s) {
  if constexpr (VPL <= 8)
    if (p.n_tokens <= kOneTokens)
      return launch_early(route_few_kernel<T, VPL>, dim3(1), dim3(kPlanThreads), 0, 1, s, p);
  GPTQ_TRY(launch_early(route_kernel<T, VPL>, dim3((unsigned)p.chunks), dim3(threads), 0, 1, s, p));
  return launch_early(plan_kernel, dim3((unsigned)p.chunks), dim3(kPlanThreads), 0, 1, s, p);
}
template <typename T>
gptq_status route(const RouteParams &p, int threads, cudaStream_t s) {
  const int e = p.n_experts;
  if (e <= 32) return route_of<T, 1>(p, threads, s);
  if (e <= 64) return route_of<T, 2>(p, threads, s);
  if (e <= 128) return route_of<T, 4>(p, threads, s);
  if (e <= 256) return route_of<T, 8>(p, threads, s);
  if (e <= 512) return route_of<T, 16>(p, threads, s);
  return route_of<T, 32>(p, threads, s);
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
      w[j] = j0 + j < p.top_k ? p.weights[t * p.top_k + j0 + j] : 0.0f;
      if (w[j] != 0.0f) y[j].load((const T *)p.y + (t * p.top_k + j0 + j) * p.ldy + c, n, p.vy);
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

size_t moe_route_ws_bytes(int64_t n_tokens, int n_experts, int top_k) {
  if (n_tokens <= kOneTokens && n_experts <= 256) return 256;
  const int chunk = chunk_tokens(n_tokens, top_k, route_threads(n_tokens, n_experts));
  return round_up(sizeof(uint16_t) * (size_t)ceil_div(n_tokens, chunk) * n_experts + 1, 256);
}

gptq_status launch_moe_route(const MoeRouteArgs &g, void *ws, cudaStream_t s) {
  if (g.n_tokens == 0) {
    GPTQ_CUDA_CHECK(cudaMemsetAsync(g.offsets, 0, sizeof(int32_t) * (g.n_experts + 1), s));
    return GPTQ_OK;
  }
  RouteParams p{};
  p.logits = g.logits; p.ld = g.ld;
  p.n_tokens = g.n_tokens; p.n_experts = g.n_experts; p.top_k = g.top_k;
  p.bias = g.bias;
  p.sigmoid = g.sigmoid; p.groups = g.groups; p.top_groups = g.top_groups; p.group_top = g.group_top;
  p.size = g.n_experts / g.groups;
  p.renormalize = g.renormalize; p.scale = g.scale;
  p.ids = g.ids; p.weights = g.weights; p.offsets = g.offsets; p.order = g.order;
  p.counts = (uint16_t *)ws;
  const int threads = route_threads(g.n_tokens, g.n_experts);
  p.chunk = g.n_tokens <= kOneTokens && g.n_experts <= 256 ? kOneTokens : chunk_tokens(g.n_tokens, g.top_k, threads);
  p.chunks = (int)ceil_div(g.n_tokens, p.chunk);
  switch (g.dtype) {
    case GPTQ_F32: return route<float>(p, threads, s);
    case GPTQ_F16: return route<__half>(p, threads, s);
    default: return route<__nv_bfloat16>(p, threads, s);
  }
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
