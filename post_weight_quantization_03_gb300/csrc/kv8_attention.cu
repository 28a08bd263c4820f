// Attention over the 8-bit cache, few queries (a decoding step).
//
// Per (sequence, cache head) the queries of the group's heads and of the new tokens are the
// rows, at most 32, eight to an MMA tile; the keys and values stream past once.  HBM-bound for
// up to 16 rows or so: 2 D bytes a token and head, against 4 D operations a row.
//
//   products  e4m3 MMAs (m16n8k32, fp32 sums) straight on the cached codes.  The other operand
//             is a sum of e4m3 terms: with 4 bits of significand each, two terms hold a bf16
//             number exactly and three an fp16 one (down to 2^-22 of the row's maximum, to which
//             a row of queries is first scaled by a power of two).  An MMA has 16 rows: eight
//             rows' first terms and, below them, their lower terms times 2^5, so a thread finds
//             both halves of a score in its own accumulator.  Against fp16 MMAs on converted
//             codes: no conversions (512 a block and warp) and half the MMAs;
//   softmax   a block's key exponent is a factor of its scores, its value exponent lv is folded
//             into the exponential: with y = f s + lv, the running maximum m of y and a base b,
//               p = 2^(y - b),  acc += p vc,  l += p 2^(b - m - lv)   (out = 2^(b - m) acc / l),
//             so the block scales cost one addition per block; m, l, acc are fp32, and 2^8 p is
//             split into as many terms as the queries: 9 or 12 bits, but no finer than 2^-23 of
//             b.  What that leaves out stays in l and leaves acc, which shows behind a dominant
//             token of small value (a sink).  So b is not m but the maximum of the block at hand
//             (or up to kSlack above it), acc moving along, which costs nothing.  Within a block,
//             tokens below 2^-15 of b hold fewer than 8 bits.  Where the row's sums are not
//             large enough beside b for that to be lost in them, a second pass of products over
//             the block adds what the terms left out: the first blocks of wide histories, blocks
//             with a sink.  (Its code, mostly not run, costs 2 to 10 %: 48 sequences of up to
//             8000 tokens 109.0 -> 112.5 us, 32 of 4000 with 16 rows 72.2 -> 75.9; where scores
//             spread over tens of powers of two and it runs 124 and 91.  Scores taken again for
//             the pass, or the pass in a loop with the first: up to 2.3 times as long.)
//   layout    tokens are dealt to the score tiles' columns so that the 16 scores a thread owns
//             are 16 consecutive tokens: they are, unmoved, its operand of the second MMA, whose
//             other operand is 16 consecutive bytes of a V row (V is stored channel-major).
//
// Each CTA takes a contiguous share of all (sequence, head, block) units.  One warp looks the
// blocks up, 32 at a time and two batches ahead, and keeps the copies of K's and V's 64 x D bytes
// (contiguous) running; eight warps in groups of one warp per eight rows take the units in turn,
// each group through a ring of its own in shared memory, and meet at the end of an item.  An
// item that lies in one share is written there; pieces of others meet in a second small kernel,
// in order (repeatable).  Short histories are dealt whole, to CTAs or, where there are many, to
// groups.
//
// Measured: 48 sequences of up to 8000 tokens (8 cache heads of 128, 64 heads: 596 MB) 112.5 us,
// 5.3 TB/s; each further 100 MB takes 15.7 us (6.4 TB/s), the rest is the start of the copies and
// the joining kernel.  One sequence of 500 tokens, 32 heads: 7.5 us, latency.
#include "kv8.cuh"

namespace gptq {

namespace {

using namespace kv8;

constexpr int kRows = 32;                 // most rows of an item
using DecodePlan = Plan<kRows, kTok, 0>;  // a unit is one block
constexpr int kWarps = 8;                 // that compute
// Registers go by groups of four warps: two that compute, one with the look-up warp.  At launch
// 384 threads have 168 each (64,512); the split below is that many: 256 x 232 + 128 x 40.
constexpr int kThreads = 32 * (kWarps + 4);
constexpr int kList = 128;                // units that have been looked up
constexpr int kItem = 5;                  // an item's start and end, in blocks
constexpr int kLow = 5;                   // power of two of the lower terms
constexpr float kLowValue = 1.0f / (1 << kLow);
// In powers of two: how far a block's maximum may lie below the base of its products, and below
// the running maximum: acc cannot grow past fp32, and 2^20 blocks below that add 2^-14.
constexpr float kSlack = 1.0f, kFar = 40.0f;
// Of 2^8 p: the terms of what is smaller than kFew hold fewer than 8 bits, what is below kNone
// never counts.  What the terms of a number below kFew leave out is 2^-15 at most, so that times
// kRest it is a number for two terms again.
constexpr float kFew = 0x1p-7f, kNone = 0x1p-32f, kRest = 0x1p23f;
// What a block's terms leave out, up to 64 x 2^-15 x 56 with values' codes of middling size, over a
// row's sums is to be 2^-9 at most in the mean of the channels (so the sums count by their harmonic
// mean: by the plain one, tokens with values in a few channels would hide what the others lose).
constexpr float kHide = 64 * 0x1p-15f * 56 * 0x1p9f;
static_assert(kRows == 8 * 4, "row tiles: 1, 2 or 4");

__device__ int g_gave_up;  // a wait ran out since it was last asked for

template <int D>
struct Decode {
  static constexpr uint32_t kHalf = kTok * D;                 // bytes of K (or V) of a block
  static constexpr int kSlots = D == 128 ? 3 : 6;             // halves in flight per warp
  static constexpr uint32_t kRing = kWarps * kSlots * kHalf;  // 192 KB
  static constexpr int kWarpPart = 8 * D + 16;                // floats: acc, m, l of eight rows
  static constexpr size_t kSmem =
      128 + kRing + kWarps * kWarpPart * 4 + kList * 8 + 2 * kWarps * kSlots * 8;
  static constexpr int kPart = kPiece<DecodePlan, D>;
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c[i] += (sum of the terms) b[i] for N accumulators, the MMAs on one of them kept apart: the
// first two terms as the tile's two halves, a third one to the second's half.  x, y: the words of
// the first and second 16 elements of K.
template <int NT, int N>
__device__ __forceinline__ void mma_terms(float (&c)[N][4], const uint32_t (&x)[NT],
                                          const uint32_t (&y)[NT], const uint32_t (&b0)[N],
                                          const uint32_t (&b1)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) mma_e4m3(c[i], x[0], x[1], y[0], y[1], b0[i], b1[i]);
  if constexpr (NT == 3) {
#pragma unroll
    for (int i = 0; i < N; ++i) mma_e4m3(c[i], 0u, x[2], 0u, y[2], b0[i], b1[i]);
  }
}

// Queries of eight rows as MMA operands: thread (row = lane / 4, t = lane % 4) holds elements
// [t D/4, (t + 1) D/4), eight per K step.  f: factor that undoes the row's scaling, times the
// softmax scale in base 2.
template <typename T, int D>
__device__ __forceinline__ void load_queries(const Kv8AttentionArgs &g, int seq, int head, int r,
                                             int rows, int group,
                                             uint32_t (&qa)[D / 16][kTerms<T>], float &f) {
  const int t = threadIdx.x % 4;
  float v[D / 4];
  if (r < rows) {
    const T *q = (const T *)g.q + seq * g.q_stride[0] + (r / group) * g.q_stride[1] +
                 (int64_t)(head * group + r % group) * g.q_stride[2] + t * (D / 4);
    if (((uintptr_t)q & 15) == 0) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 w = reinterpret_cast<const uint4 *>(q)[i];
        const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * i + j] = to_f32(e[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < D / 4; ++i) v[i] = to_f32(q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 4; ++i) v[i] = 0.0f;
  }
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < D / 4; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
  most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
  const float amax = __uint_as_float(most);
  const int e = row_exponent(amax) - 7;  // the row's maximum in [128, 256)
  const float inv = row_scale(amax, e);
  f = fp8::pow2(e) * g.scale * kLog2e;
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    split4<kTerms<T>, kLow>(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv,
                            v[4 * i + 3] * inv, qa[i]);
}

// How the work is dealt: by units, items whole to CTAs (whose groups share an item's units), or
// items whole to the groups of a CTA in turn (each finishes its own; all of a CTA's units then fit
// the list).
enum Deal { kUnits, kItemsToCtas, kItemsToGroups };

// RT: row tiles, and warps of a group (1, 2 or 4).
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kThreads, 1)
decode_kernel(Kv8AttentionArgs g, int deal, float *part, DevStatus *st) {
  using C = Decode<D>;
  constexpr int NT = kTerms<T>;
  constexpr int G = kWarps / RT;             // groups
  constexpr int H = C::kSlots * RT;          // ring slots (halves of blocks) of a group
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 127) & ~(uintptr_t)127);
  float *spart = (float *)(smem + C::kRing);
  int2 *list = (int2 *)(spart + kWarps * C::kWarpPart);  // block and head (-1: none); exponents
  uint64_t *full = (uint64_t *)(list + kList), *empty = full + kWarps * C::kSlots;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const tc::Waits waits{st, &g_gave_up, g.wait_ns};
  if (threadIdx.x == 0) {
    for (int s = 0; s < G * H; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], RT);
    }
    tc::mbar_fence_init();
  }
  __syncthreads();
  wait_for_grids();
  launch_dependents();
  // the call's status; a wait that gives up writes it, two seconds from here or later
  if (blockIdx.x == 0 && threadIdx.x == 0) st->status = 0;

  const DecodePlan plan(g);
  const int group = plan.group, rows = plan.rows;
  write_empty<T, D>(plan, threadIdx.x, kThreads);
  Cursor at{};
  const int count = deal == kUnits ? my_share(plan, G, at) : my_items(plan, at);
  if (count == 0) return;
  const bool to_groups = deal == kItemsToGroups;
  const int item0 = at.entry * g.n_kv + at.head;
  auto owner = [&](const Cursor &c) { return (c.entry * g.n_kv + c.head - item0) % G; };

  if (warp >= kWarps) {
    // ---------------- look-up and copies ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp > kWarps) return;
    // Lane l looks up unit i0 + l of each batch of 32: table entries of the batch after the next
    // and exponents of the next are on their way while a batch is written to the list.
    Cursor c = at;
    c.advance(plan, lane);
    int page = -1, place = -1, exps = 0, head = 0, own = 0;  // of the batches after and next
    auto load_page = [&](int i) {
      page = -1;
      if (i < count) {
        page = g.table[c.entry * g.ld_table + c.blk];
        head = c.head;
        own = owner(c);
        if (i + 32 < count) c.advance(plan, 32);
      }
    };
    auto load_exps = [&]() {
      place = page < 0 || page >= g.n_blocks ? -1 : page * g.n_kv + head;
      exps = own << 16;
      if (place >= 0) exps |= (int)g.k_exps[place] | ((int)g.v_exps[place] << 8);
    };
    int filled = 0, soon = lane;
    load_page(soon);
    load_exps();
    load_page(soon += 32);
    // Lane q keeps group q's ring full: half hn of its blocks goes to slot hn % H.
    int i = to_groups ? 0 : lane, hn = 0;
    const int last = lane < G ? count : 0;
    uint64_t t0 = tc::global_ns();
    while (__any_sync(0xffffffffu, i < last)) {
      const int behind = __reduce_min_sync(0xffffffffu, i < last ? i : 0x7fffffff);
      while (filled < count && behind >= filled - 32) {
        list[(filled + lane) % kList] = make_int2(place, exps);
        load_exps();
        load_page(soon += 32);
        filled += 32;
        __syncwarp();
      }
      bool moved = false;
      if (to_groups)
        while (i < last && i < filled && list[i % kList].y >> 16 != lane) ++i;
      if (i < last && i < filled) {
        const int slot = lane * H + hn % H;
        if (hn < H || tc::mbar_try_wait(&empty[slot], (hn / H - 1) & 1)) {
          const int ph = list[i % kList].x;
          if (ph < 0) {
            tc::mbar_arrive(&full[slot]);
          } else if (hn != g.lost) {
            tc::mbar_arrive_expect_tx(&full[slot], C::kHalf);
            tc::bulk_load(smem + (size_t)slot * C::kHalf,
                          ((hn & 1) ? g.v : g.k) + (int64_t)ph * C::kHalf, C::kHalf, &full[slot]);
          }
          if (hn & 1) i += to_groups ? 1 : G;
          ++hn;
          moved = true;
        }
      }
      if (__any_sync(0xffffffffu, moved)) {
        t0 = tc::global_ns();
      } else if (tc::global_ns() - t0 > waits.ns) {
        tc::give_up(waits);
        break;
      }
    }
    // the copies have landed before the CTA leaves, also where nobody waits for them any more
    if (lane < G)
      for (int h = hn > H ? hn - H : 0; h < hn; ++h)
        if (h != g.lost) tc::mbar_wait_compact(&full[lane * H + h % H], (h / H) & 1, waits);
    return;
  }

  // ---------------- products ----------------
  asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
  const int t = lane % 4, grp = warp / RT, r = (warp % RT) * 8 + lane / 4;  // this thread's row
  uint8_t *ring = smem + (size_t)grp * H * C::kHalf;
  float *mine = spart + warp * C::kWarpPart;
  full += grp * H;
  empty += grp * H;
  int hn = 0;        // halves used
  // false once a wait has given up: the rest is skipped, and no slot is given back
  bool ok = true;
  auto arrived = [&]() {
    if (ok) ok = tc::mbar_wait_compact(&full[hn % H], (hn / H) & 1, waits);
    ok = __all_sync(0xffffffffu, ok);
  };
  auto release = [&]() {
    __syncwarp();
    if (lane == 0 && ok) tc::mbar_arrive(&empty[hn % H]);
    ++hn;
  };
  for (int i = grp, i0 = 0; i0 < count;) {
    const int i1 = i0 + at.nblk - at.blk < count ? i0 + at.nblk - at.blk : count;  // item's units
    if (to_groups) {
      i = i0;
      if (owner(at) != grp) {
        i0 = i1;
        if (i0 < count) at.next_item(plan);
        continue;
      }
    }
    const int length = seq_length(g, at.entry);
    const int limit = r >= rows ? 0 : (g.causal ? length - (int)g.n_new + r / group + 1 : length);
    uint32_t qa[D / 16][NT];
    // lift: 2^(b - m); hidden: the b up to which the row's sums hide what the terms leave out
    float f, m = -INFINITY, b = -INFINITY, lift = 0.0f, hidden = -INFINITY, l = 0.0f, acc[D / 8][4];
    load_queries<T, D>(g, at.entry, at.head, r, rows, group, qa, f);
#pragma unroll
    for (int q = 0; q < D / 8; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[q][j] = 0.0f;

#pragma unroll 1
    for (; i < i1; i += to_groups ? 1 : G) {
      arrived();
      const int2 what = list[i % kList];
      if (!ok || what.x < 0) {
        release();
        arrived();
        release();
        continue;
      }
      const float fk = f * fp8::exp_value((uint8_t)what.y);
      const int lv = (what.y >> 8 & 0xFF) - fp8::kBias;
      // column n of score tile j is token 16 (n / 2) + 2 j + n % 2 of the block
      const uint8_t *krow = ring + (size_t)(hn % H) * C::kHalf +
                            (16 * (lane / 8) + (lane / 4) % 2) * D + t * (D / 4);
      float s[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) s[j][q] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[4][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 w4 = *reinterpret_cast<const uint4 *>(krow + 2 * j * D + 16 * c);
          x[0][j] = w4.x; x[1][j] = w4.y; x[2][j] = w4.z; x[3][j] = w4.w;
        }
        mma_terms<NT, 8>(s, qa[4 * c], qa[4 * c + 1], x[0], x[1]);
        mma_terms<NT, 8>(s, qa[4 * c + 2], qa[4 * c + 3], x[2], x[3]);
      }
      release();
      // this thread's tokens of the block: 16 t + 2 j + {0, 1}
      const int first = (at.blk + i - i0) * kTok, tok = first + 16 * t;
      const bool cut = first + kTok > length - (g.causal ? (int)g.n_new - 1 : 0);
      const uint8_t *vrow = ring + (size_t)(hn % H) * C::kHalf + (lane / 4) * kTok + 16 * t;
      const int live = length - tok;  // of this thread's 16 tokens
      auto products = [&](const uint32_t (&p)[4][NT]) {  // acc += p V
#pragma unroll
        for (int q0 = 0; q0 < D / 8; q0 += 4) {
          uint32_t x[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 w4 = *reinterpret_cast<const uint4 *>(vrow + 8 * (q0 + q) * kTok);
            x[0][q] = w4.x; x[1][q] = w4.y; x[2][q] = w4.z; x[3][q] = w4.w;
          }
          if (cut && live < 16) {
            // bytes past the sequence may be NaN codes, and 0 x NaN is NaN
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int keep = live - 4 * j;
              const uint32_t mask = keep <= 0 ? 0u : (keep >= 4 ? ~0u : (1u << (8 * keep)) - 1u);
#pragma unroll
              for (int q = 0; q < 4; ++q) x[j][q] &= mask;
            }
          }
          float(&c)[4][4] = *reinterpret_cast<float(*)[4][4]>(&acc[q0]);
          mma_terms<NT, 4>(c, p[0], p[1], x[0], x[1]);
          mma_terms<NT, 4>(c, p[2], p[3], x[2], x[3]);
        }
      };
      auto scale_acc = [&](float by) {
#pragma unroll
        for (int q = 0; q < D / 8; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[q][j] *= by;
      };
      uint32_t pa[4][NT];
      {
        float y[16], mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          y[j] = fmaf(fmaf(s[j / 2][j % 2 + 2], kLowValue, s[j / 2][j % 2]), fk, (float)lv);
          if (cut && tok + j >= limit) y[j] = -INFINITY;
          mx = fmaxf(mx, y[j]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const bool move = mx > b || (mx < b - kSlack && mx >= m - kFar);
        if (__any_sync(0xffffffffu, move)) {
          const float to = move ? mx : b, by = move ? ex2(b - to) : 1.0f;  // 0 for the first block
          const float mn = fmaxf(m, to), unit = mn == -INFINITY ? 0.0f : mn;
          l *= ex2(m - unit);
          b = to;
          m = mn;
          lift = ex2(b - unit);
          scale_acc(by);
        }
        const float base = (b == -INFINITY ? 0.0f : b) - 8.0f;
        float sum = 0.0f;
        __half2 x[8];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          y[j] = ex2(y[j] - base);
          sum += y[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __floats2half2_rn(y[2 * j], y[2 * j + 1]);
        l = fmaf(sum * lift, 0x1p-8f * fp8::pow2(-lv), l);
        __half2 low = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) low = __hmin2(low, x[j]);
        low = __hmin2(low, __lowhigh2highlow(low));
        if (__builtin_expect(__any_sync(0xffffffffu, __low2float(low) < kFew && b > hidden), 0)) {
          bool few = false;  // without the zeros of masked tokens
#pragma unroll
          for (int j = 0; j < 16; ++j) few |= y[j] < kFew && y[j] >= kNone;
          few &= b > hidden;
          if (__any_sync(0xffffffffu, few)) {
            float inverse = 0.0f;  // of the row's sums: a sum of 0 hides nothing
#pragma unroll
            for (int q = 0; q < D / 8; ++q)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                inverse += __fdividef(1.0f, fabsf(fmaf(acc[q][j + 2], kLowValue, acc[q][j])));
            inverse += __shfl_xor_sync(0xffffffffu, inverse, 1);
            inverse += __shfl_xor_sync(0xffffffffu, inverse, 2);
            hidden = fmaxf(hidden, b - __log2f(inverse * (kHide / D)));
            few &= b > hidden;
          }
          if (__builtin_expect(__any_sync(0xffffffffu, few), 0)) {
            uint32_t rest[4][NT];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t term[NT];
              split4<NT, kLow>(x[2 * q], x[2 * q + 1], term);
              float left[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                float had = 0.0f;
#pragma unroll
                for (int i = NT - 1; i >= 0; --i)
                  had = fmaf(i == 0 ? kLowValue : 1.0f, had, fp8::unpack1((uint8_t)(term[i] >> (8 * j))));
                left[j] = y[4 * q + j] < kFew ? (y[4 * q + j] - had) * kRest : 0.0f;
              }
              split4<NT, kLow>(left[0], left[1], left[2], left[3], rest[q]);
            }
            scale_acc(kRest);
            arrived();
            products(rest);
            scale_acc(1.0f / kRest);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) split4<NT, kLow>(x[2 * q], x[2 * q + 1], pa[q]);
      }
      arrived();
      products(pa);
      release();
    }

    // the item's end, here or in the next share: join the groups
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float of_m = 0x1p-8f * lift;  // acc in units of 2^m
    if (to_groups) {
      if (r < rows) {
        const float inv = l == 0.0f ? 0.0f : of_m / l;
        T *o = out_row<T>(g, group, at.entry, at.head, r) + 2 * t;
#pragma unroll
        for (int q = 0; q < D / 8; ++q) {
          o[8 * q] = from_f32<T>(fmaf(acc[q][2], kLowValue, acc[q][0]) * inv);
          o[8 * q + 1] = from_f32<T>(fmaf(acc[q][3], kLowValue, acc[q][1]) * inv);
        }
      }
      i0 = i1;
      if (i0 < count) at.next_item(plan);
      continue;
    }
#pragma unroll
    for (int q = 0; q < D / 8; ++q)
      *reinterpret_cast<float2 *>(mine + (lane / 4) * D + 8 * q + 2 * t) =
          make_float2(fmaf(acc[q][2], kLowValue, acc[q][0]) * of_m, fmaf(acc[q][3], kLowValue, acc[q][1]) * of_m);
    if (t == 0) {
      mine[8 * D + lane / 4] = m;
      mine[8 * D + 8 + lane / 4] = l;
    }
    tc::named_barrier(1, 32 * kWarps);
    const bool all = at.blk == 0 && i1 - i0 == at.nblk;
    float *piece = part + (2 * (int64_t)blockIdx.x + (i0 > 0 ? 1 : 0)) * C::kPart;
    for (int e = threadIdx.x; e < rows * (D / 4); e += 32 * kWarps) {
      const int row = e / (D / 4), d = e % (D / 4) * 4;
      const float *p = spart + (row / 8) * C::kWarpPart;
      float mm = -INFINITY, ll = 0.0f;
#pragma unroll
      for (int q = 0; q < G; ++q) mm = fmaxf(mm, p[q * RT * C::kWarpPart + 8 * D + row % 8]);
      const float base = mm == -INFINITY ? 0.0f : mm;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < G; ++q, p += RT * C::kWarpPart) {
        const float sc = ex2(p[8 * D + row % 8] - base);
        const float4 v = *reinterpret_cast<const float4 *>(p + (row % 8) * D + d);
        ll = fmaf(p[8 * D + 8 + row % 8], sc, ll);
        a.x = fmaf(v.x, sc, a.x);
        a.y = fmaf(v.y, sc, a.y);
        a.z = fmaf(v.z, sc, a.z);
        a.w = fmaf(v.w, sc, a.w);
      }
      if (all) {
        const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
        T *o = out_row<T>(g, group, at.entry, at.head, row) + d;
        o[0] = from_f32<T>(a.x * inv);
        o[1] = from_f32<T>(a.y * inv);
        o[2] = from_f32<T>(a.z * inv);
        o[3] = from_f32<T>(a.w * inv);
      } else {
        // the share's first item, or (an item begun inside it) its last
        reinterpret_cast<float4 *>(piece)[d / 4 * kRows + row] = a;
        if (d == 0) {
          piece[kRows * D + row] = mm;
          piece[kRows * D + kRows + row] = ll;
        }
      }
    }
    tc::named_barrier(1, 32 * kWarps);  // the parts have been read
    i0 = i1;
    if (i0 < count) at.next_item(plan);
  }
}

int row_tiles(int64_t rows) { return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4); }

// Whether items are dealt whole: histories of at most two rounds of the groups.
bool stays_whole(int64_t rows, int64_t max_blocks) {
  return max_blocks <= 2 * kWarps / row_tiles(rows);
}

template <typename T, int D>
gptq_status run_decode(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  using C = Decode<D>;
  if (!kv8_plan_fits(g, kRows, 1, 0)) return GPTQ_ERR_UNSUPPORTED;
  const int64_t rows = g.n_new * (g.n_heads / g.n_kv);
  const int rt = row_tiles(rows);
  const auto kernel = rt == 1 ? decode_kernel<T, D, 1>
                              : (rt == 2 ? decode_kernel<T, D, 2> : decode_kernel<T, D, 4>);
  GPTQ_TRY(ensure_smem_attr((const void *)kernel, (int)C::kSmem));
  int sms = 0;
  GPTQ_TRY(device_sm_count(&sms));
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  float *part = (float *)((char *)ws + 256);
  // Short histories (two rounds of the groups) gain nothing from being cut, and uncut they need
  // no second kernel: 8.8 -> 7.7 us for one token of 500 with 32 heads.
  // More items than CTAs: a group an item leaves no group without blocks and joins nothing, where
  // the estimate in blocks says so (one token, 100 sequences of 60, 8 cache heads: 24.5 us by CTAs,
  // 11.0 by groups; 15 of 86, 32 cache heads: 21.9 and 11.5; but 8 of 500, 32 cache heads: 13.9
  // and 19.4).
  const int groups = kWarps / rt;
  int deal = stays_whole(rows, g.max_blocks) ? kItemsToCtas : kUnits;
  const int64_t items = ceil_div(g.n_seq * g.n_kv, ctas);  // of a CTA
  if (deal == kItemsToCtas && items * g.max_blocks <= kList &&
      ceil_div(items, groups) * (g.max_blocks + kItem) < items * (ceil_div(g.max_blocks, groups) + kItem))
    deal = kItemsToGroups;
  GPTQ_TRY(launch_early(kernel, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, 1, s, g, deal, part,
                        (DevStatus *)ws));
  if (deal != kUnits) return GPTQ_OK;
  return launch_early(join_kernel<T, D, DecodePlan>, dim3((unsigned)ctas - 1), dim3(128), 0, 1, s, g,
                      (const float *)part, kWarps / rt, ctas);
}

// Whether `rows` rows of a cache head go to the other kernel's 128-row tiles.  More than 32 always
// do; fewer where the products here (a pass of MMAs for each eight rows and three terms) outweigh
// the copies, and the history is long enough for that kernel's set-up (32 sequences of up to
// 4000 tokens of 8 cache heads, here and there):
//   17 to 32 rows   bf16 78 and 67 us with 64 channels (4 of 500: 14.8 and 10.2, 16 of 700: 18.3
//                   and 18.0), 124 and 80 with 128 (4 of 500: 19.7 and 12.5, 2 of 120: 9.5 and
//                   9.3); fp16 108 and 67, 222 and 84
//   9 to 16 rows    fp16, 128 channels 129 and 83 (8 of 1500: 29.5 and 23.3, 16 of 500: 16.4 and
//                   14.6); but fp16, 64 channels 65 and 67; bf16 48 and 66, 75 and 80
bool takes_tiles(int64_t rows, bool half, int dim, int64_t max_blocks) {
  if (rows > kRows) return true;
  if (rows > 16) return max_blocks > 6;
  return rows > 8 && half && dim == 128 && max_blocks > 20;
}

}  // namespace

size_t kv8_attention_ws_bytes(int n_seq, int64_t n_new, int n_heads, int n_kv, int dim,
                              int max_blocks) {
  const int64_t rows = n_new * (n_heads / n_kv);
  int64_t ctas = kMaxCtas;
  const int64_t units = (int64_t)n_seq * n_kv * max_blocks;
  if (units < ctas) ctas = units;
  const size_t here = rows > kRows ? 0
                      : stays_whole(rows, max_blocks)
                          ? 256  // the status alone
                          : 256 + (size_t)(2 * ctas) * kRows * (dim + 2) * 4;
  if (!takes_tiles(rows, true, dim, max_blocks)) return here;  // (with fp16 wherever with bf16)
  const size_t there = kv8_prompt_ws_bytes(n_seq, n_new, n_heads, n_kv, dim, max_blocks);
  return there > here ? there : here;
}

gptq_status kv8_attention_take_timeout(int *out, cudaStream_t s) {
  int prompt = 0;
  GPTQ_TRY(take_flag(g_gave_up, out, s));
  GPTQ_TRY(kv8_prompt_take_timeout(&prompt, s));
  if (prompt != 0) *out = prompt;
  return GPTQ_OK;
}

gptq_status launch_kv8_attention(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  if (g.n_seq == 0 || g.n_new == 0) {
    GPTQ_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
    return GPTQ_OK;
  }
  if (takes_tiles(g.n_new * (g.n_heads / g.n_kv), g.dtype == GPTQ_F16, g.dim, g.max_blocks))
    return launch_kv8_prompt(g, ws, s);
  if (g.dtype == GPTQ_F16)
    return g.dim == 64 ? run_decode<__half, 64>(g, ws, s) : run_decode<__half, 128>(g, ws, s);
  return g.dim == 64 ? run_decode<__nv_bfloat16, 64>(g, ws, s)
                     : run_decode<__nv_bfloat16, 128>(g, ws, s);
}

}  // namespace gptq
