// What the attention kernels over the 8-bit cache share: the division of their work and the
// joining of its pieces.
//
// The rows of a (sequence, cache head) are its new tokens' queries of the group's heads, row r
// being token r / group and head r % group of the group.  An entry is a tile of up to kRows rows
// of one sequence, an item an entry with a head, and a unit one step along an item's cached
// tokens.  Units are numbered entry by entry, head by head.  For the division an item weighs its
// units and SETUP more, for what is done once for it: CTA w of n takes the weight [total w / n,
// total (w + 1) / n), a start inside an item's setup being its first unit.  An item inside one
// share is finished there; otherwise each share leaves a piece (acc, m, l) of it, in its CTA's
// first slot if the share begins with or inside the item and in the second otherwise, and
// join_kernel adds the pieces in order.
#pragma once

#include <type_traits>

#include "fp8.cuh"
#include "tc.cuh"

namespace gptq {
namespace kv8 {

constexpr int kTok = GPTQ_KV8_BLOCK;
constexpr int kMaxCtas = 160;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Terms of a sum of e4m3 numbers for operands of type T.
template <typename T>
constexpr int kTerms = std::is_same<T, __half>::value ? 3 : 2;

// x (two fp16 numbers, |x| <= 256) = term[0] + 2^-LOW (term[1] (+ term[2])), two codes each.  The
// first term leaves 8 at most, so LOW may be up to 5 where the lower terms' products are summed
// apart.  What is left out is 2^(-10 - LOW) at most, or the terms' 9 or 12 bits.
template <int NT, int LOW>
__device__ __forceinline__ void split(__half2 x, uint32_t (&term)[NT]) {
  const auto code = [](__half2 v) {
    return __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(v), __NV_SATFINITE, __NV_E4M3);
  };
  const auto value = [](__nv_fp8x2_storage_t c) {
    return __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3));
  };
  const __half2 up = __float2half2_rn((float)(1 << LOW)), down = __float2half2_rn(-(float)(1 << LOW));
  term[0] = code(x);
  x = __hfma2(value(term[0]), down, __hmul2(x, up));  // exact
  term[1] = code(x);
  if constexpr (NT == 3) term[2] = code(__hsub2(x, value(term[1])));
}

// Four numbers' terms, a word of codes each.
template <int NT, int LOW>
__device__ __forceinline__ void split4(__half2 ab, __half2 cd, uint32_t (&word)[NT]) {
  uint32_t lo[NT], hi[NT];
  split<NT, LOW>(ab, lo);
  split<NT, LOW>(cd, hi);
#pragma unroll
  for (int i = 0; i < NT; ++i) word[i] = lo[i] | (hi[i] << 16);
}
template <int NT, int LOW>
__device__ __forceinline__ void split4(float a, float b, float c, float d, uint32_t (&word)[NT]) {
  split4<NT, LOW>(__floats2half2_rn(a, b), __floats2half2_rn(c, d), word);
}

// Two fp16 numbers from the lower (upper) two codes of a word.
__device__ __forceinline__ uint32_t halves_lo(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(w));
  return h;
}

// Cached tokens of a sequence, inside the table.
__device__ __forceinline__ int seq_length(const Kv8AttentionArgs &g, int seq) {
  const int len = g.lengths[seq], cap = g.max_blocks * kTok;
  return len < 0 ? 0 : (len > cap ? cap : len);
}

// The exponent of a row's largest magnitude (0 for a row of zeros), by which queries are scaled
// into the range of the type that the tensor cores take.
__device__ __forceinline__ int row_exponent(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127;
  return amax == 0.0f ? 0 : (e < -110 ? -110 : e);
}

// Magnitudes as integers are in their order, infinities and NaN above all numbers.  A row with
// one of these has no softmax: scaled by NaN, all of it becomes NaN codes.
__device__ __forceinline__ float row_scale(float amax, int e) {
  return fp8::finite(amax) ? fp8::pow2(-e) : __uint_as_float(0x7FC00000u);
}

// Entries of ROWS rows whose units are UNIT cached tokens.
template <int ROWS, int UNIT, int SETUP>
struct Plan {
  static constexpr int kRows = ROWS, kSetup = SETUP;
  const Kv8AttentionArgs &g;
  int group, rows, tiles, entries;  // rows and row tiles of a sequence

  __device__ __forceinline__ explicit Plan(const Kv8AttentionArgs &a) : g(a) {
    group = a.n_heads / a.n_kv;
    rows = (int)a.n_new * group;
    tiles = (rows + ROWS - 1) / ROWS;
    entries = a.n_seq * tiles;
  }
  // Tokens that some row of [row0, row1) of a sequence with `length` tokens sees.
  __device__ __forceinline__ int seen(int length, int row0, int row1) const {
    if (row1 > rows) row1 = rows;
    if (row0 >= row1) return 0;
    const int n = g.causal ? length - (int)g.n_new + (row1 - 1) / group + 1 : length;
    return n < 0 ? 0 : n;
  }
  __device__ __forceinline__ int units(int entry) const {
    const int seq = entry / tiles, row0 = entry % tiles * ROWS;
    return (seen(seq_length(g, seq), row0, row0 + ROWS) + UNIT - 1) / UNIT;
  }
  // Whole warp: the weight of all items (the launch has checked that it fits 31 bits), or their
  // units.
  __device__ __forceinline__ int total(int setup = SETUP) const {
    int s = 0;
#pragma unroll 1
    for (int i = threadIdx.x % 32; i < entries; i += 32) {
      const int n = units(i);
      s += n > 0 ? n + setup : 0;
    }
    return __reduce_add_sync(0xffffffffu, s) * g.n_kv;
  }
};

// The CTAs that share the weight `total`, `turn` units of it at a time at least, and where share
// w starts.
__device__ __forceinline__ int shares(int total, int turn, int ctas) {
  const int n = total / turn + (total % turn != 0 ? 1 : 0);
  return n < ctas ? n : ctas;
}
__device__ __forceinline__ int share_start(int total, int n, int w) {
  const int q = total / n, r = total % n;
  return q * w + (w < r ? w : r);
}

// A unit: step `blk` of the `nblk` of an item.
struct Cursor {
  int entry, head, blk, nblk;
  template <typename P>
  __device__ __forceinline__ void next_item(const P &p) {
    blk = 0;
    if (++head < p.g.n_kv) return;
    head = 0;
#pragma unroll 1
    do ++entry; while (entry < p.entries && (nblk = p.units(entry)) == 0);
  }
  template <typename P>
  __device__ __forceinline__ void advance(const P &p, int by) {
#pragma unroll 1
    while (blk + by >= nblk && entry < p.entries) {
      by -= nblk - blk;
      next_item(p);
    }
    blk += by;
  }
  template <typename P>
  __device__ __forceinline__ void step(const P &p) {
    if (++blk >= nblk) next_item(p);
  }
};

// Whole warp: the cursor at weight v (0 <= v < total), the units before it and, in `start`, the
// weight at which its item starts.
template <typename P>
__device__ __forceinline__ Cursor cursor_at(const P &p, int v, int &unit, int &start) {
  const int lane = threadIdx.x % 32, kv = p.g.n_kv;
  unit = start = 0;
#pragma unroll 1
  for (int s0 = 0;; s0 += 32) {
    const int nb = s0 + lane < p.entries ? p.units(s0 + lane) : 0;
    int incl = nb > 0 ? (nb + P::kSetup) * kv : 0, units = nb * kv;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, incl, o), b = __shfl_up_sync(0xffffffffu, units, o);
      if (lane >= o) {
        incl += a;
        units += b;
      }
    }
    const unsigned past = __ballot_sync(0xffffffffu, start + incl > v);
    const int src = past ? __ffs(past) - 1 : 31;
    start += __shfl_sync(0xffffffffu, incl, src);
    unit += __shfl_sync(0xffffffffu, units, src);
    if (past == 0) continue;
    const int n = __shfl_sync(0xffffffffu, nb, src), weight = n + P::kSetup;
    start -= weight * kv;
    const int head = (v - start) / weight;
    start += head * weight;
    const int at = v - start - P::kSetup;
    const Cursor c{s0 + src, head, at < 0 ? 0 : at, n};
    unit += (head - kv) * n + c.blk;
    return c;
  }
}

// Whole warp: this CTA's share, as its first unit's cursor and the number of its units.
template <typename P>
__device__ __forceinline__ int my_share(const P &p, int turn, Cursor &first) {
  const int total = p.total(), n = shares(total, turn, gridDim.x);
  if ((int)blockIdx.x >= n) return 0;
  if constexpr (P::kSetup == 0) {  // weights are units
    const int v = share_start(total, n, blockIdx.x);
    int unit, start;
    first = cursor_at(p, v, unit, start);
    return share_start(total, n, blockIdx.x + 1) - v;
  }
  int u0 = 0, u1 = 0;
#pragma unroll 1
  for (int end = 0; end < 2; ++end) {  // one copy of the search for the share's two ends
    const int v = share_start(total, n, blockIdx.x + end);
    int start;
    u0 = u1;
    if (v == total) {
      u1 = p.total(0);
    } else {
      const Cursor c = cursor_at(p, v, u1, start);
      if (end == 0) first = c;
    }
  }
  return u1 - u0;
}

// The same with the items dealt whole: nothing is left to join.
template <typename P>
__device__ __forceinline__ int my_items(const P &p, Cursor &first) {
  const int items = p.entries * p.g.n_kv, n = items < (int)gridDim.x ? items : gridDim.x;
  if ((int)blockIdx.x >= n) return 0;
  const int i0 = share_start(items, n, blockIdx.x), i1 = share_start(items, n, blockIdx.x + 1);
  int count = 0;
#pragma unroll 1
  for (int i = i0; i < i1; ++i) count += p.units(i / p.g.n_kv);
  if (count == 0) return 0;
  first = Cursor{i0 / p.g.n_kv, i0 % p.g.n_kv, 0, p.units(i0 / p.g.n_kv)};
  if (first.nblk == 0) {
    first.head = p.g.n_kv - 1;  // on to the next entry that has units
    first.next_item(p);
  }
  return count;
}

// Where row `row` of a sequence's head goes.
template <typename T>
__device__ __forceinline__ T *out_row(const Kv8AttentionArgs &g, int group, int seq, int head,
                                      int row) {
  return (T *)g.out + seq * g.o_stride[0] + (row / group) * g.o_stride[1] +
         (int64_t)(head * group + row % group) * g.o_stride[2];
}

// All threads of a CTA: zeros for the entries that see nothing (no unit of theirs exists), the
// CTAs taking the entries in turn.
template <typename T, int D, typename P>
__device__ __forceinline__ void write_empty(const P &p, int thread, int threads) {
#pragma unroll 1
  for (int e = blockIdx.x; e < p.entries; e += gridDim.x) {
    if (p.units(e) > 0) continue;
    const int row0 = e % p.tiles * P::kRows, n = min(P::kRows, p.rows - row0);
#pragma unroll 1
    for (int i = thread; i < n * p.g.n_kv * D; i += threads)
      out_row<T>(p.g, p.group, e / p.tiles, i / D % p.g.n_kv, row0 + i / D / p.g.n_kv)[i % D] =
          from_f32<T>(0.0f);
  }
}

template <typename P, int D>
constexpr int kPiece = P::kRows *(D + 2);  // floats of a piece: acc [D / 4][rows][4], m, l

// Joins the pieces of the items that the start of share w cuts, w = blockIdx.x + 1, for 32 rows:
// out = sum_i 2^(m_i - m) acc_i / sum_i 2^(m_i - m) l_i.  A lane is a row (pieces keep the rows
// next to each other), a warp every fourth group of four channels; the rows leave through shared
// memory.  The kernel starts while the one before runs (which has waited for all before it, so
// the lengths are there) and waits for it where it reads the pieces; it waits also where there
// is nothing to join, since its end has to mean that the other's came.
template <typename T, int D, typename P>
__global__ void __launch_bounds__(128)
join_kernel(Kv8AttentionArgs g, const float *part, int turn, int ctas) {
  const P p(g);
  const int total = p.total(), n = shares(total, turn, ctas);
  const int w = blockIdx.x + 1;
  bool cut = w < n;
  Cursor at{};
  int last = w;
  bool late = false;
  if (cut) {
    int unit, first;
    const int v = share_start(total, n, w), before = share_start(total, n, w - 1);
    at = cursor_at(p, v, unit, first);
    // a later start in the same item leaves it to the first
    cut = at.blk > 0 && before <= first + P::kSetup;
    late = before < first;
#pragma unroll 1
    while (last + 1 < n && share_start(total, n, last + 1) < first + P::kSetup + at.nblk) ++last;
  }
  wait_for_grids();
  if (!cut) return;
  const int seq = at.entry / p.tiles, row0 = at.entry % p.tiles * P::kRows;
  const int rows = min(P::kRows, p.rows - row0), tile = blockIdx.y * 32;
  if (tile >= rows) return;
  constexpr int kGroups = D / 16;                 // groups of four channels of a thread
  __shared__ alignas(16) T stage[32][D + 8];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, row = tile + lane;
  const float *p0 = part + (int64_t)(2 * (w - 1) + (late ? 1 : 0)) * kPiece<P, D>;
  float m = -INFINITY, l = 0.0f;
  const float *q = p0;
#pragma unroll 2
  for (int i = w - 1; i <= last; ++i) {
    m = fmaxf(m, q[P::kRows * D + row]);
    q = part + (int64_t)(2 * (i + 1)) * kPiece<P, D>;
  }
  if (m == -INFINITY) m = 0.0f;
  float4 a[kGroups];
#pragma unroll
  for (int k = 0; k < kGroups; ++k) a[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  q = p0;
#pragma unroll 2
  for (int i = w - 1; i <= last; ++i) {
    float4 v[kGroups];
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
      v[k] = reinterpret_cast<const float4 *>(q)[(warp + 4 * k) * P::kRows + row];
    const float sc = ex2(q[P::kRows * D + row] - m);
    l = fmaf(q[P::kRows * (D + 1) + row], sc, l);
#pragma unroll
    for (int k = 0; k < kGroups; ++k) {
      a[k].x = fmaf(v[k].x, sc, a[k].x);
      a[k].y = fmaf(v[k].y, sc, a[k].y);
      a[k].z = fmaf(v[k].z, sc, a[k].z);
      a[k].w = fmaf(v[k].w, sc, a[k].w);
    }
    q = part + (int64_t)(2 * (i + 1)) * kPiece<P, D>;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    T *o = &stage[lane][4 * (warp + 4 * k)];
    o[0] = from_f32<T>(a[k].x * inv);
    o[1] = from_f32<T>(a[k].y * inv);
    o[2] = from_f32<T>(a[k].z * inv);
    o[3] = from_f32<T>(a[k].w * inv);
  }
  __syncthreads();
  constexpr int kLanes = D / 8;
#pragma unroll 1
  for (int r = threadIdx.x / kLanes; r < 32 && tile + r < rows; r += 128 / kLanes) {
    const int c = threadIdx.x % kLanes * 8;
    T *o = out_row<T>(g, p.group, seq, at.head, row0 + tile + r) + c;
    if (g.vec_o) {
      *reinterpret_cast<uint4 *>(o) = *reinterpret_cast<const uint4 *>(&stage[r][c]);
    } else {
      for (int j = 0; j < 8; ++j) o[j] = stage[r][c + j];
    }
  }
}

}  // namespace kv8

// What the kernels' 31-bit unit counts take; `rows` rows in tiles of `tile`, units of `blocks` blocks.
static inline bool kv8_plan_fits(const Kv8AttentionArgs &g, int64_t tile, int64_t blocks, int64_t setup) {
  const int64_t rows = g.n_new * (g.n_heads / g.n_kv), tiles = ceil_div(rows, tile);
  return rows < INT32_MAX / 2 &&
         (double)tiles * g.n_seq * g.n_kv * (double)(ceil_div(g.max_blocks, blocks) + setup) < INT32_MAX / 2;
}

// kv8_prompt.cu: many queries (prompts), on the tensor cores.
size_t kv8_prompt_ws_bytes(int n_seq, int64_t n_new, int n_heads, int n_kv, int dim,
                           int max_blocks);
gptq_status launch_kv8_prompt(const Kv8AttentionArgs &g, void *ws, cudaStream_t s);
gptq_status kv8_prompt_take_timeout(int *out, cudaStream_t s);

}  // namespace gptq
