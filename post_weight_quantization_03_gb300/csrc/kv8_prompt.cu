// Attention over the 8-bit cache, many queries (prompts and chunks of them).
//
// Bound by the tensor cores: 4 D operations a visible (row, token) pair, 2 D bytes a token and
// cache head for 256 rows.  The heads of a group and the new tokens are the rows; an item is 256
// rows of one cache head, two MMA tiles of 128 that share every key and value.
//
//   scores    kind::f8f6f4 straight on the cached codes, which TMA brings into the layout that the
//             MMA reads.  The queries are sums of two (bf16) or three (fp16) e4m3 terms, exact down
//             to 2^-17 of the row's maximum: as many MMAs as fp16 operands would take (half as
//             many again for fp16 queries), and the keys need no conversion.
//   outputs   kind::f16: a converter warp group turns the value codes into fp16 (exact), once for
//             256 rows.  (Splitting the probabilities into e4m3 terms instead costs the softmax
//             warps more than converting the values costs here.)
//   softmax   one row per thread, no exchange between threads.  A block's key exponent is a
//             factor of its scores, its value exponent lv goes into the exponential:
//             y = f s + lv,  p = 2^(y - b + 8),  O += p vc,  l += p 2^-lv;  out = O / l.
//             b is the maximum of y when it was last set.  It stays while a block's sum of p is
//             at most 2^15 (p within fp16's range), so that the maximum is looked for, and O (in
//             TMEM) and l are rescaled, only where the sum exceeds that: past a row's first
//             blocks rarely.  A maximum beside every block's exponentials takes two of the
//             twelve issue slots of a pair of scores (1 x 4096: 131 us, without 127).  p is rounded
//             to fp16 once and replaces the scores in TMEM, from where it is the second
//             product's A operand, a block of 64 tokens at a time.
//   overlap   while one tile's softmax runs, the tensor core multiplies for the other.
//
// Measured: 4096 tokens of 32 heads of 128 (8 in the cache, causal) 124 us, 1.1 PFLOP/s; 2 x 777
// of up to 16000 tokens, heads of 64, fp16 queries 240 us, 0.8 PFLOP/s of 4 D a pair (1.2 executed:
// a third term).  Neither the tensor core (49 and 43 % busy) nor the exponentials (26 and 35 %) are
// full: a block of 64 tokens of both tiles takes about the sum of its softmax and its MMAs (1900 and
// 1470 cycles), so that the two run nearly one after the other though two blocks of two tiles are in
// flight.  Which wait holds which role has not been measured.
//
// Warps: 0-3 and 4-7 softmax, a tile each; 8-11 copies and converters; 12 and 13 MMA issuers, a
// tile each (12 owns TMEM).
#include <cudaTypedefs.h>
#include <limits.h>
#include <string.h>

#include "kv8.cuh"

namespace gptq {

namespace {

using namespace kv8;

constexpr int kTile = 128;                      // rows of an MMA tile, tokens of a unit
// An item's set-up and end (queries in, outputs out, the first unit's scores with nothing beside
// them) weigh as much as five units of its 128 tokens: 1 x 4096 tokens take 204 us with 2, 161
// with 3, 143 with 4, 129 with 5 and 6, 132 with 8.
using PromptPlan = Plan<2 * kTile, kTile, 5>;
// Least weight of a share: cut finer, an item's set-ups and the joining of its pieces cost more
// than the units (2 sequences of 48 rows over up to 8588 tokens: 71 us with 1, 28 with 4 and 6,
// 30 with 10; 13 of 168 rows over up to 1149: 29.4, 27.0, 29.3, 34.6).
constexpr int kTurn = 4;
// Registers by warp group: 2 x 128 x 192 + 128 x 72 + 128 x 56 = 65,536, what 512 threads have
// at launch: a softmax thread holds its row's 128 scores.
constexpr int kThreads = 512;
constexpr int kInfo = 4;
constexpr float kMostSum = 0x1p15f;

constexpr int kKStages = 3, kVStages = 2;

__device__ int g_gave_up;  // a wait ran out since it was last asked for

template <int D, int NT>
struct Prompt {
  static constexpr uint32_t kTerm = kTile * D;                // a term of a tile of queries
  static constexpr uint32_t kQ = NT * kTerm;                  // its rows of 2 D bytes fit, too
  static constexpr uint32_t kK = kTile * D;                   // a unit's keys
  static constexpr uint32_t kV = D * kTile * 2;               // its values, fp16, channel-major
  static constexpr uint32_t kVChunk = D * 128;                // 64 tokens of them
  static constexpr uint32_t kHalf = kTok * D;                 // bytes of K (or V) of a block
  static constexpr size_t kSmem = 1024 + 2 * kQ + kKStages * kK + kVStages * kV + 2 * kHalf +
                                  kInfo * 32 + 2 * kTile * 4 + 256;
  static constexpr uint32_t kCols = 512;
  static constexpr uint32_t kO = 2 * kTile;                   // TMEM column of the first O
};

struct Info {   // of a unit's two blocks
  float ks[2];
  int lv[2];
  int there[2];
  int pad[2];
};

// D[tmem] (+)= A[tmem] B[smem]^T, kind::f16, one thread.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// D[tmem] (+)= A[smem] B[smem]^T, kind::f8f6f4 (e4m3), one thread.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of K-major rows of D bytes (64 or 128) with the swizzle of that width.
template <int D>
__device__ __forceinline__ uint64_t desc_rows(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
         ((uint64_t)(8 * D >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)(D == 128 ? 2 : 4) << 61);
}

// Two fp32 numbers at a time: a * b + c, a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The two elements of a word.
template <typename T>
__device__ __forceinline__ float2 pair(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  else
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) return pack_half2(a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Byte of element (row, 16-byte unit u) in a chunk of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int row, int u) {
  return (uint32_t)(row * 128 + ((u ^ (row & 7)) << 4));
}

// The same for rows of D bytes.
template <int D>
__host__ __device__ constexpr uint32_t swizzled_row(int row, int u) {
  return (uint32_t)(row * D + ((D == 128 ? u ^ (row & 7) : u ^ (row >> 1 & 3)) << 4));
}

// A tile of queries: byte of the 16-byte unit u of a row's term.
template <int D>
__host__ __device__ constexpr uint32_t query_byte(int row, int term, int u) {
  return (uint32_t)(term * kTile * D) + swizzled_row<D>(row, u);
}
// The same memory holds an item's outputs, rows of 2 D bytes: byte of the 16-byte unit u, in the
// row's own first two terms.
template <int D>
__host__ __device__ constexpr uint32_t output_byte(int row, int u) {
  return query_byte<D>(row, u / (D / 16), u % (D / 16));
}
// The four warps of a tile pass from an item's outputs to the next item's queries one by one, so
// the outputs of a warp's 32 rows may lie only where queries of these rows lie.
template <int D>
constexpr bool outputs_in_own_rows() {
  for (int row = 0; row < kTile; ++row)
    for (int u = 0; u < D / 8; ++u) {
      const uint32_t at = output_byte<D>(row, u), in_term = at % (uint32_t)(kTile * D);
      if (at / (uint32_t)(kTile * D) > 1 || in_term / (32 * D) != (uint32_t)(row / 32)) return false;
    }
  return true;
}
static_assert(outputs_in_own_rows<64>() && outputs_in_own_rows<128>(), "outputs in other warps' queries");

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ CUtensorMap mk, Kv8AttentionArgs g, int uncut, float *part,
              DevStatus *st) {
  constexpr int NT = kTerms<T>;
  using C = Prompt<D, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sq = smem, *sk = sq + 2 * C::kQ, *sv = sk + kKStages * C::kK;
  uint8_t *raw_v = sv + kVStages * C::kV;         // codes of a unit's values
  Info *info = (Info *)(raw_v + 2 * C::kHalf);
  float *factor = (float *)(info + kInfo);        // of each row's scores
  uint64_t *qfull = (uint64_t *)(factor + 2 * kTile);   // [2], by tile
  // by tile and block of a unit (a barrier has one phase a unit: its waiters never fall two behind)
  uint64_t *sfull = qfull + 2, *pfull = sfull + 4, *odone = pfull + 4;
  uint64_t *kfull = odone + 4, *kempty = kfull + kKStages;
  uint64_t *vfull = kempty + kKStages, *vempty = vfull + kVStages, *vraw = vempty + kVStages;
  uint64_t *mdone = vraw + 1;   // [2]: every MMA of the issuer's has completed
  uint32_t *tmem_slot = (uint32_t *)(mdone + 2);
  const tc::Waits waits{st, &g_gave_up, g.wait_ns};
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&qfull[b], 4);
      tc::mbar_init(&sfull[2 * b], 1);
      tc::mbar_init(&sfull[2 * b + 1], 1);
      tc::mbar_init(&pfull[2 * b], 4);
      tc::mbar_init(&pfull[2 * b + 1], 4);
      tc::mbar_init(&odone[2 * b], 1);
      tc::mbar_init(&odone[2 * b + 1], 1);
      tc::mbar_init(&vfull[b], 4);
      tc::mbar_init(&vempty[b], 2);
      tc::mbar_init(&mdone[b], 1);
    }
    for (int i = 0; i < kKStages; ++i) {
      tc::mbar_init(&kfull[i], 1);
      tc::mbar_init(&kempty[i], 2);
    }
    tc::mbar_init(vraw, 1);
    tc::mbar_fence_init();
  }
  if (warp == 12) tc::tmem_alloc(tmem_slot, C::kCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_grids();
  launch_dependents();
  // the call's status; a wait that gives up writes it, two seconds from here or later
  if (blockIdx.x == 0 && threadIdx.x == 0) st->status = 0;

  const PromptPlan plan(g);
  write_empty<T, D>(plan, threadIdx.x, kThreads);
  Cursor at{};
  const int count = uncut ? my_items(plan, at) : my_share(plan, kTurn, at);
  bool ok = true;  // false once a wait has given up: the rest passes without waiting

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < 14) {
      // ---------------- MMA issuers, one for each tile (the whole warp; one lane issues) ----------------
      const int b = warp - 12;
      constexpr uint32_t id_s = tc::instr_desc(0, 0, kTile, kTok, 0, 0);
      constexpr uint32_t id_o = tc::instr_desc(0, 0, kTile, D, 0, 0);
      // a descriptor holds its address in units of 16 bytes: offsets are added to it
      const uint64_t dq = desc_rows<D>(tc::smem_u32(sq)), dk = desc_rows<D>(tc::smem_u32(sk));
      const uint64_t dv = tc::smem_desc_sw128(tc::smem_u32(sv), 16, 1024);
      auto wait = [&](uint64_t *bar, int phase) {
        if (ok) ok = tc::mbar_wait_compact(bar, phase & 1, waits);
        ok = __all_sync(0xffffffffu, ok);
        tc::tc_fence_after();
      };
      auto commit = [&](uint64_t *bar) {
        if (ok && tc::elect_one()) tc::mma_commit(bar);
      };
      auto scores = [&](int u, int h) {               // of the unit's block h
        if (ok && tc::elect_one()) {
          const uint64_t q = dq + b * (C::kQ >> 4);
          const uint64_t k = dk + (u % kKStages * C::kK + h * C::kHalf >> 4);
#pragma unroll
          for (int i = 0; i < NT * (D / 32); ++i)
            mma_f8(tmem + b * kTile + h * kTok, q + ((i / (D / 32) * C::kTerm + i % (D / 32) * 32) >> 4),
                   k + 2 * (i % (D / 32)), id_s, i > 0);
          tc::mma_commit(&sfull[2 * b + h]);
        }
      };
      auto outputs = [&](int u, int h, bool first) {  // of the unit's block h
        if (ok && tc::elect_one()) {
          const uint64_t v = dv + ((u & 1) * C::kV + h * C::kVChunk >> 4);
          const uint32_t p = tmem + b * kTile + h * kTok;
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i)
            mma_f16_ts(tmem + C::kO + b * D, p + 8 * i, v + 2 * i, id_o, !first || i > 0);
          tc::mma_commit(&odone[2 * b + h]);
        }
      };
      int items = 0, done = 0;  // that the tile took part in: items; units multiplied
#pragma unroll 1
      for (int i0 = 0; i0 < count && ok;) {
        const int m = at.nblk - at.blk < count - i0 ? at.nblk - at.blk : count - i0;
        const int len = seq_length(g, at.entry / plan.tiles);
        const int row0 = at.entry % plan.tiles * 2 * kTile + b * kTile;
        // units of this item, counted from the share's first one, that the tile takes part in
        const int nb = (plan.seen(len, row0, row0 + kTile) + kTile - 1) / kTile - at.blk;
        const int to = nb < m ? (nb < 0 ? 0 : nb) : m;
        // step i: block by block, the outputs of unit i and then, where the scores were, those of
        // unit i + 1: they are there before the softmax is done with the other block
#pragma unroll 1
        for (int i = -1; i < m && ok; ++i) {
          const int u = i0 + i;
          if (i + 1 < m) wait(&kfull[(u + 1) % kKStages], (u + 1) / kKStages);
          if (i >= 0) wait(&vfull[u & 1], u >> 1);
          if (i < to && to > 0) {
            if (i < 0) wait(&qfull[b], items++);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (i >= 0) {
                wait(&pfull[2 * b + h], done);
                outputs(u, h, i == 0 && h == 0);
              }
              if (i + 1 < to) scores(u + 1, h);
            }
            if (i >= 0) ++done;
          }
          if (i >= 0) commit(&vempty[u & 1]);
          if (i + 1 < m) commit(&kempty[(u + 1) % kKStages]);
        }
        i0 += m;
        if (i0 < count) at.next_item(plan);
      }
      // nothing of these MMAs may still be running when the TMEM is released
      if (tc::elect_one()) tc::mma_commit(&mdone[b]);
      tc::mbar_wait_compact(&mdone[b], 0, waits);
    }
  } else if (warp >= 8) {
    // ---------------- copies and converters ----------------
    // One thread asks for a unit's keys (TMA) and value codes (contiguous copies); all turn pieces
    // of 16 value codes into fp16, one channel in every 32 a thread: four lanes take the 64 tokens
    // of a block, so that eight lanes' accesses of 16 bytes fall into different banks.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    const int ct = threadIdx.x - 256, x = ct % 4, r0 = ct / 4;
    Cursor c = at;              // of the unit whose blocks are looked up
    int pages[2], head = 0, len = 0, blk = 0, entry = -1;
    const int32_t *row = g.table;
    auto look_up = [&](int u) {
      pages[0] = pages[1] = -1;
      if (u >= count) return;
      if (c.entry != entry) {
        entry = c.entry;
        row = g.table + entry / plan.tiles * g.ld_table;
        len = seq_length(g, entry / plan.tiles);
      }
      head = c.head;
      blk = c.blk;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((2 * blk + h) * kTok < len) pages[h] = row[2 * blk + h];
      if (u + 1 < count) c.step(plan);
    };
    int place[2] = {-1, -1}, ex[2], left = 0;   // of the unit that is being copied
    auto locate = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        place[h] = pages[h] < 0 || pages[h] >= g.n_blocks ? -1 : pages[h] * g.n_kv + head;
        ex[h] = place[h] < 0 ? fp8::kBias * 257
                             : (int)g.k_exps[place[h]] | ((int)g.v_exps[place[h]] << 8);
      }
      left = len - blk * kTile;  // tokens of the unit that exist
    };
    const uint32_t at0 = swizzled(r0, 2 * x), at1 = swizzled(r0, 2 * x + 1);
    auto put = [&](uint8_t *rows, const uint4 &q) {
      *reinterpret_cast<uint4 *>(rows + at0) =
          make_uint4(halves_lo(q.x), halves_hi(q.x), halves_lo(q.y), halves_hi(q.y));
      *reinterpret_cast<uint4 *>(rows + at1) =
          make_uint4(halves_lo(q.z), halves_hi(q.z), halves_lo(q.w), halves_hi(q.w));
    };
    auto wait = [&](uint64_t *bar, int phase) {
      if (ok) ok = tc::mbar_wait_compact(bar, phase & 1, waits);
    };
    int keys = 0, codes = 0;  // units whose keys, value codes have been asked for; none once a wait gave up
    // step u: convert unit u, have unit u + 1 copied, look unit u + 2 up
#pragma unroll 1
    for (int u = count > 0 ? -2 : 0; u < count; ++u) {
      const int tokens = left, there = (place[0] >= 0 ? 1 : 0) | (place[1] >= 0 ? 2 : 0);
      const bool next = u >= -1 && u + 1 < count;
      uint32_t bytes = 0;
      if (u >= -1) locate();    // the next unit
      if (next && ct == 0) {
        // its keys, and what the softmax has to know of it (the unit four back has been read: the
        // keys of three units back were multiplied after the probabilities of four back)
        const int n = u + 1, s = n % kKStages;
        if (n >= kKStages) wait(&kempty[s], n / kKStages - 1);
        Info &f = info[n % kInfo];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f.ks[h] = fp8::exp_value((uint8_t)ex[h]);
          f.lv[h] = (ex[h] >> 8) - fp8::kBias;
          f.there[h] = place[h] >= 0;
          bytes += place[h] >= 0 ? C::kHalf : 0;
        }
        if (ok && n != g.lost) {
          tc::mbar_arrive_expect_tx(&kfull[s], bytes);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (place[h] >= 0)
              tc::tma_load_3d(sk + s * C::kK + h * C::kHalf, &mk, 0, 0, place[h], &kfull[s]);
        }
        keys += ok;
      }
      if (u >= 0) {
        // values; those past the sequence's end may be NaN codes and become zeros
        const int s = u % kVStages;
        wait(vraw, u);
        if (u >= kVStages) wait(&vempty[s], u / kVStages - 1);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {       // block; its channels r0 + 32 i
          const int live = tokens - h * kTok - x * 16;
          uint4 q[D / 32];
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            q[i] = there >> h & 1 ? *reinterpret_cast<const uint4 *>(raw_v + h * C::kHalf +
                                                                     (r0 + i * 32) * kTok + x * 16)
                                  : make_uint4(0, 0, 0, 0);
          if (live < 16) {
            auto mask = [&](int at) {
              return live <= at ? 0u : (live >= at + 4 ? ~0u : (1u << (8 * (live - at))) - 1u);
            };
            const uint4 m = make_uint4(mask(0), mask(4), mask(8), mask(12));
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
              q[i] = make_uint4(q[i].x & m.x, q[i].y & m.y, q[i].z & m.z, q[i].w & m.w);
          }
#pragma unroll
          for (int i = 0; i < D / 32; ++i) put(sv + s * C::kV + h * C::kVChunk + i * 32 * 128, q[i]);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&vfull[s]);
        tc::named_barrier(1, 128);  // the codes have been read
      }
      if (next && ct == 0 && ok) {
        codes = u + 2;
        tc::fence_proxy_async_smem();
        tc::mbar_arrive_expect_tx(vraw, bytes);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (place[h] >= 0)
            tc::bulk_load(raw_v + h * C::kHalf, g.v + (int64_t)place[h] * C::kHalf, C::kHalf, vraw);
      }
      look_up(u + 2);
    }
    if (ct == 0) {
      // the copies have landed before the CTA leaves, also where nobody waits for them any more
      for (int n = keys > kKStages ? keys - kKStages : 0; n < keys; ++n)
        if (n != g.lost) tc::mbar_wait_compact(&kfull[n % kKStages], (n / kKStages) & 1, waits);
      if (codes > 0) tc::mbar_wait_compact(vraw, (codes - 1) & 1, waits);
    }
  } else {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int b = warp / 4, row = threadIdx.x % kTile;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + lanes + b * kTile, to = tmem + lanes + C::kO + b * D;
    uint8_t *q_tile = sq + b * C::kQ;
    int seen = 0;  // units before this item: phases of sfull and odone
    auto wait = [&](uint64_t *bar, int phase) {
      if (ok) ok = tc::mbar_wait_compact(bar, phase & 1, waits);
      ok = __all_sync(0xffffffffu, ok);
      tc::tc_fence_after();
    };
    for (int i0 = 0; i0 < count && ok;) {
      const int m = at.nblk - at.blk < count - i0 ? at.nblk - at.blk : count - i0;
      const int seq = at.entry / plan.tiles, row0 = at.entry % plan.tiles * 2 * kTile + b * kTile;
      const int len = seq_length(g, seq), r = row0 + row;
      const int nb = (plan.seen(len, row0, row0 + kTile) + kTile - 1) / kTile;
      const int mine = nb - at.blk < m ? (nb - at.blk < 0 ? 0 : nb - at.blk) : m;
      // a row that does not exist is as good as one that sees everything
      const int limit = r < plan.rows ? plan.seen(len, r, r + 1) : INT_MAX;
      // Where this thread's row of queries starts, and of outputs (rows that do not exist: row 0).
      const int rq = r < plan.rows ? r / plan.group : 0, hq = r < plan.rows ? r % plan.group : 0;
      const int64_t q_at = seq * g.q_stride[0] + rq * g.q_stride[1] +
                           (int64_t)(at.head * plan.group + hq) * g.q_stride[2];
      const int64_t o_at = seq * g.o_stride[0] + rq * g.o_stride[1] +
                           (int64_t)(at.head * plan.group + hq) * g.o_stride[2];
      // Queries: 16 elements a lane, D / 16 lanes to a row, `kAt` rows of the warp's 32 at a time;
      // scaled to a maximum of [128, 256) and split into terms, K-major.  All loads in flight at
      // once, left in the lane's own slots; the rest in a small loop (code that runs once an item
      // costs its instructions' fetch).
      float f = 0.0f;
      if (mine > 0) {
        constexpr int kLanes = D / 16, kAt = 32 / kLanes;
        const int sub = lane / kLanes, piece16 = lane % kLanes, wrow = warp % 4 * 32;
        const T *q = (const T *)g.q + 16 * piece16;
        const int exist = plan.rows - row0 - wrow;  // of the warp's rows
        auto slot = [&](int mr, int term) {
          return reinterpret_cast<uint4 *>(q_tile + query_byte<D>(mr, term, piece16));
        };
        if (g.vec_q) {
          uint4 raw[2 * 32 / kAt];
#pragma unroll
          for (int i = 0; i < 32 / kAt; ++i) {
            const int mr = i * kAt + sub;
            const uint4 *at16 = reinterpret_cast<const uint4 *>(q + __shfl_sync(0xffffffffu, q_at, mr));
            raw[2 * i] = mr < exist ? at16[0] : make_uint4(0, 0, 0, 0);
            raw[2 * i + 1] = mr < exist ? at16[1] : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 32 / kAt; ++i) {
            *slot(wrow + i * kAt + sub, 0) = raw[2 * i];
            *slot(wrow + i * kAt + sub, 1) = raw[2 * i + 1];
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 64 / kAt; ++i) {
            const int mr = i / 2 * kAt + sub;
            const int64_t off = __shfl_sync(0xffffffffu, q_at, mr) + 8 * (i % 2);
            alignas(16) T e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = mr < exist ? q[off + j] : from_f32<T>(0.0f);
            *slot(wrow + mr, i % 2) = *reinterpret_cast<const uint4 *>(e);
          }
        }
#pragma unroll 2
        for (int i = 0; i < 32 / kAt; ++i) {
          const int mr = wrow + i * kAt + sub;
          const uint4 lo = *slot(mr, 0), hi = *slot(mr, 1);
          const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
          uint32_t most = 0;  // magnitudes of the even and of the odd elements
#pragma unroll
          for (int j = 0; j < 8; ++j) most = __vmaxu2(most, w[j] & 0x7FFF7FFFu);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1)
            most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
          const float amax = pair<T>(max(most & 0xFFFFu, most >> 16)).x;
          const int e = row_exponent(amax) - 7;
          const float scale = row_scale(amax, e), inv = g.scale < 0.0f ? -scale : scale;
          if (piece16 == 0) factor[b * kTile + mr] = fp8::pow2(e) * fabsf(g.scale) * kLog2e;
          uint32_t word[4][NT];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 a = pair<T>(w[2 * j]), c = pair<T>(w[2 * j + 1]);
            split4<NT, 0>(a.x * inv, a.y * inv, c.x * inv, c.y * inv, word[j]);
          }
#pragma unroll
          for (int term = 0; term < NT; ++term)
            *slot(mr, term) = make_uint4(word[0][term], word[1][term], word[2][term], word[3][term]);
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();  // O of the item before has been read
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&qfull[b]);
        f = factor[b * kTile + row];
      }
      float base = -INFINITY, l = 0.0f;  // the exponent that p is taken from; sum of p 2^-lv
      // Block by block: probabilities from the base as it is; where they are too large for it (rare
      // past a row's first blocks), the base is raised to the block's maximum, what the row has is
      // rescaled and the block's probabilities are taken again: 64 of 2^8 at most, below the limit.
#pragma unroll 1
      for (int i2 = 0; i2 < 2 * mine && ok; ++i2) {
        const int i = i2 >> 1, h = i2 & 1;
        wait(&sfull[2 * b + h], seen + i);
        const Info &in = info[(i0 + i) % kInfo];
        const float lv = (float)in.lv[h], ks = in.ks[h];
        const int left = in.there[h] ? limit - (at.blk + i) * kTile - h * kTok : 0;  // visible tokens
        const uint32_t tb = ts + h * kTok;
        uint32_t s[2][32];
        tc::tmem_ld32(tb, s[0]);
        tc::tmem_ld32(tb + 32, s[1]);
        // a factor of 0 would turn the masked -inf into NaN
        const float fk = fmaxf(f * ks, 1e-37f), back = 0x1p-8f * fp8::pow2(-in.lv[h]);
        tc::tmem_ld_wait();
        if (!__all_sync(0xffffffffu, left >= kTok)) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) s[c][j] = 32 * c + j < left ? s[c][j] : 0xFF800000u;
        }
        float2 sum[2];
#pragma unroll 1
        for (;;) {
          const float off = lv - (base == -INFINITY ? 0.0f : base) + 8.0f;
          const float2 fk2 = make_float2(fk, fk), off2 = make_float2(off, off);
          sum[0] = sum[1] = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 x = make_float2(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1]));
              float2 y = fma2(x, fk2, off2);
              y = make_float2(ex2(y.x), ex2(y.y));
              sum[j % 2] = add2(sum[j % 2], y);
              w[j] = pack_half2(y.x, y.y);
            }
            tmem_st16(tb + 16 * c, w);
          }
          sum[0] = add2(sum[0], sum[1]);
          const bool large = sum[0].x + sum[0].y > kMostSum || base == -INFINITY;
          if (!__any_sync(0xffffffffu, large)) break;
          float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              top[j / 2 % 2] = max3(top[j / 2 % 2], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
          const float high = fmaf(fmaxf(top[0], top[1]), fk, lv);
          const bool raise = large && high > base;
          if (!__any_sync(0xffffffffu, raise)) break;
          if (i2 > 0) {
            const float shrink = raise ? ex2(base - high) : 1.0f;
            l *= shrink;
            wait(&odone[2 * b + 1 - h], seen + i + h - 1);  // the block before
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(to + c, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink);
              tmem_st16(to + c, o);
            }
          }
          if (raise) base = high;
          tmem_st_wait();  // the probabilities are written again
        }
        l = fmaf(sum[0].x + sum[0].y, back, l);
        tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&pfull[2 * b + h]);
      }
      // the item's end, here or in the next share
      seen += mine;
      if (mine > 0) {
        wait(&odone[2 * b], seen - 1);
        wait(&odone[2 * b + 1], seen - 1);
      }
      const bool whole = at.blk == 0 && m == at.nblk;
      float *piece = part + (2 * (int64_t)blockIdx.x + (i0 > 0 ? 1 : 0)) * kPiece<PromptPlan, D>;
      const float inv = whole ? (l == 0.0f ? 0.0f : 0x1p-8f / l) : 0x1p-8f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t x[32];
        if (mine > 0) {
          tc::tmem_ld32(to + c, x);
          tc::tmem_ld_wait();
        }
#pragma unroll
        for (int j = 0; j < 32; ++j)
          x[j] = mine > 0 ? __float_as_uint(__uint_as_float(x[j]) * inv) : 0u;
        if (whole) {
          // through the tile of queries, whose products are done
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t e[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              e[q] = pack<T>(__uint_as_float(x[j + 2 * q]), __uint_as_float(x[j + 2 * q + 1]));
            *reinterpret_cast<uint4 *>(q_tile + output_byte<D>(row, (c + j) / 8)) =
                make_uint4(e[0], e[1], e[2], e[3]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            reinterpret_cast<uint4 *>(piece)[(c + j) / 4 * 2 * kTile + b * kTile + row] =
                make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        }
      }
      if (whole) {
        __syncwarp();  // a warp's rows are its own
        constexpr int kLanes = D / 8, kAt = 32 / kLanes;  // 16 bytes a lane
        const int sub = lane / kLanes, part8 = lane % kLanes, wrow = warp % 4 * 32;
        const int exist = plan.rows - row0 - wrow;
#pragma unroll 4
        for (int i = 0; i < 32; i += kAt) {
          const int64_t off = __shfl_sync(0xffffffffu, o_at, i + sub);
          if (i + sub >= exist) continue;
          const uint4 w = *reinterpret_cast<const uint4 *>(q_tile + output_byte<D>(wrow + i + sub, part8));
          T *o = (T *)g.out + off + 8 * part8;
          if (g.vec_o) {
            *reinterpret_cast<uint4 *>(o) = w;
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q] = reinterpret_cast<const T *>(&w)[q];
          }
        }
        __syncwarp();
      } else {
        piece[2 * kTile * D + b * kTile + row] = base;
        piece[2 * kTile * (D + 1) + b * kTile + row] = l;
      }
      i0 += m;
      if (i0 < count) at.next_item(plan);
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 12) tc::tmem_dealloc(tmem, C::kCols);
}

template <typename T, int D>
gptq_status run(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  using C = Prompt<D, kTerms<T>>;
  GPTQ_TRY(ensure_smem_attr((const void *)prompt_kernel<T, D>, (int)C::kSmem));
  int sms = 0;
  GPTQ_TRY(device_sm_count(&sms));
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  float *part = (float *)((char *)ws + 256);
  CUtensorMap mk;
  memset(&mk, 0, sizeof(mk));  // an empty cache is never read
  if (g.n_blocks > 0 && !tc::make_tmap_bytes_3d(&mk, g.k, g.n_blocks * g.n_kv, kTok, D))
    return GPTQ_ERR_UNSUPPORTED;
  // Short histories, with a CTA for each item, gain nothing from being cut, and uncut they need no
  // second kernel (37 sequences with 182 new tokens of up to 241: 22.4 us cut, 15.9 uncut; 500 of
  // 500 with 32 heads: 26.8 and 23.4).
  const int64_t rows = g.n_new * (g.n_heads / g.n_kv);
  const int uncut = g.max_blocks <= 8 && ceil_div(rows, 2 * kTile) * g.n_seq * g.n_kv <= ctas;
  GPTQ_TRY(launch_early(prompt_kernel<T, D>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, 1, s, mk,
                        g, uncut, part, (DevStatus *)ws));
  if (uncut) return GPTQ_OK;
  return launch_early(join_kernel<T, D, PromptPlan>, dim3((unsigned)ctas - 1, 8), dim3(128), 0, 1, s,
                      g, (const float *)part, kTurn, ctas);
}

}  // namespace

size_t kv8_prompt_ws_bytes(int n_seq, int64_t n_new, int n_heads, int n_kv, int dim,
                           int max_blocks) {
  int64_t ctas = kMaxCtas;
  const int64_t rows = n_new * (n_heads / n_kv);
  const int64_t weight = ceil_div(rows, 2 * kTile) * n_seq * n_kv *
                         (ceil_div(max_blocks, 2) + PromptPlan::kSetup);
  if (weight < ctas) ctas = weight;
  return 256 + (size_t)(2 * ctas) * (2 * kTile) * (dim + 2) * 4;
}

gptq_status kv8_prompt_take_timeout(int *out, cudaStream_t s) { return take_flag(g_gave_up, out, s); }

gptq_status launch_kv8_prompt(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  if (!kv8_plan_fits(g, 2 * kTile, 2, PromptPlan::kSetup)) return GPTQ_ERR_UNSUPPORTED;
  if (g.dtype == GPTQ_F16)
    return g.dim == 64 ? run<__half, 64>(g, ws, s) : run<__half, 128>(g, ws, s);
  return g.dim == 64 ? run<__nv_bfloat16, 64>(g, ws, s) : run<__nv_bfloat16, 128>(g, ws, s);
}

}  // namespace gptq
