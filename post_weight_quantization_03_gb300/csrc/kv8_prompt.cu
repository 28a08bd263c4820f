// Attention over the 8-bit cache, many queries (prompts and chunks of them).
//
// Bound by the tensor cores: 4 D operations a visible (row, token) pair, 2 D bytes a token and
// cache head for 256 rows.  The heads of a group and the new tokens are the rows; an item is 256
// rows of one cache head, two MMA tiles of 128 that share every key and value.
//
//   operands  kind::f16.  A converter warp group reads the codes, turns them into fp16 (exact)
//             and writes them to shared memory in the layout that the MMAs read: one conversion
//             of a key serves 256 rows.  (e4m3 MMAs would run at twice the rate, but a 16-bit
//             operand costs two or three e4m3 terms, and splitting the probabilities costs the
//             softmax warps more than converting the values costs here.)  A row of bf16 queries
//             is scaled by a power of two to a maximum of [1, 2); the scores are fp32 in TMEM.
//   softmax   one row per thread, no exchange between threads.  A block's key exponent is a
//             factor of its scores, its value exponent lv goes into the exponential:
//             y = f s + lv,  p = 2^(y - b + 8),  O += p vc,  l += p 2^-lv;  out = O / l.
//             b follows the maximum of y lazily: O (in TMEM) and l are rescaled only when y
//             exceeds b by 2^6 (p stays within fp16's range), which past a row's first tiles is
//             rare.  p is rounded to fp16 once and replaces the scores in TMEM, from where it is
//             the second product's A operand.
//   overlap   while one tile's softmax runs, the tensor core multiplies for the other.
//
// Warps: 0-3 and 4-7 softmax, a tile each; 8-11 converters; 12 MMA issuer and TMEM owner.
#include <cudaTypedefs.h>
#include <limits.h>
#include <string.h>

#include "kv8.cuh"

namespace gptq {

namespace {

using namespace kv8;

constexpr int kTile = 128;                      // rows of an MMA tile, tokens of a unit
using PromptPlan = Plan<2 * kTile, kTile, 2>;
// Registers by warp group: 2 x 128 x 192 + 128 x 72 + 128 x 56 = 65,536, what 512 threads have
// at launch: a softmax thread holds its row's 128 scores.
constexpr int kThreads = 512;
constexpr int kInfo = 4;
constexpr float kLazy = 6.0f;

template <int D>
struct Prompt {
  static constexpr uint32_t kChunk = kTile * 128;             // 128 rows of 128 bytes
  static constexpr uint32_t kQ = kTile * D * 2;               // a tile of queries (or keys)
  static constexpr uint32_t kV = D * kTile * 2;               // values, channel-major
  static constexpr uint32_t kVChunk = D * 128;                // 64 tokens of them
  static constexpr uint32_t kHalf = kTok * D;                 // bytes of K (or V) of a block
  static constexpr size_t kSmem =
      1024 + 2 * kQ + 2 * kQ + 2 * kV + 4 * kHalf + kInfo * 32 + 2 * kTile * 4 + 192;
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

// Byte of element (row, 16-byte unit u) in a chunk of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(int row, int u) {
  return (uint32_t)(row * 128 + ((u ^ (row & 7)) << 4));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(Kv8AttentionArgs g, float *part, DevStatus *st) {
  using C = Prompt<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sq = smem, *sk = sq + 2 * C::kQ, *sv = sk + 2 * C::kQ;
  uint8_t *raw_k = sv + 2 * C::kV, *raw_v = raw_k + 2 * C::kHalf;  // codes of a unit
  Info *info = (Info *)(raw_v + 2 * C::kHalf);
  float *factor = (float *)(info + kInfo);        // of each row's scores
  uint64_t *qfull = (uint64_t *)(factor + 2 * kTile);   // [2], by tile
  uint64_t *sfull = qfull + 2, *pfull = sfull + 2, *odone = pfull + 2;
  uint64_t *kfull = odone + 2, *kempty = kfull + 2, *vfull = kempty + 2, *vempty = vfull + 2;
  uint64_t *kraw = vempty + 2, *vraw = kraw + 1;
  uint32_t *tmem_slot = (uint32_t *)(vraw + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&qfull[b], 4);
      tc::mbar_init(&sfull[b], 1);
      tc::mbar_init(&pfull[b], 4);
      tc::mbar_init(&odone[b], 1);
      tc::mbar_init(&kfull[b], 4);
      tc::mbar_init(&kempty[b], 1);
      tc::mbar_init(&vfull[b], 4);
      tc::mbar_init(&vempty[b], 1);
    }
    tc::mbar_init(kraw, 1);
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
  const int count = my_share(plan, 1, at);
  bool ok = true;  // false once a wait has given up: the rest passes without waiting

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 12) {
      // ---------------- MMA issuer (the whole warp; one lane issues) ----------------
      constexpr uint32_t id_s = tc::instr_desc(0, 0, kTile, kTile, 0, 0);
      constexpr uint32_t id_o = tc::instr_desc(0, 0, kTile, D, 0, 0);
      // a descriptor holds its address in units of 16 bytes: offsets are added to it
      const uint64_t dq = tc::smem_desc_sw128(tc::smem_u32(sq), 16, 1024);
      const uint64_t dk = tc::smem_desc_sw128(tc::smem_u32(sk), 16, 1024);
      const uint64_t dv = tc::smem_desc_sw128(tc::smem_u32(sv), 16, 1024);
      auto wait = [&](uint64_t *bar, int phase) {
        if (ok) ok = tc::mbar_wait_compact(bar, phase & 1, st);
        ok = __all_sync(0xffffffffu, ok);
        tc::tc_fence_after();
      };
      auto commit = [&](uint64_t *bar) {
        if (tc::elect_one()) tc::mma_commit(bar);
      };
      auto scores = [&](int b, int u) {
        if (tc::elect_one()) {
          const uint64_t q = dq + b * (C::kQ >> 4), k = dk + (u & 1) * (C::kQ >> 4);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = ((uint32_t)(i / 4) * C::kChunk + (i % 4) * 32) >> 4;
            tc::mma_f16(tmem + b * kTile, q + off, k + off, id_s, i > 0);
          }
          tc::mma_commit(&sfull[b]);
        }
      };
      auto outputs = [&](int b, int u, bool first) {
        if (tc::elect_one()) {
          const uint64_t v = dv + (u & 1) * (C::kV >> 4);
#pragma unroll
          for (int i = 0; i < kTile / 16; ++i)
            mma_f16_ts(tmem + C::kO + b * D, tmem + b * kTile + 8 * i,
                       v + (((uint32_t)(i / 4) * C::kVChunk + (i % 4) * 32) >> 4), id_o,
                       !first || i > 0);
          tc::mma_commit(&odone[b]);
        }
      };
      // by tile: the items that it took part in, and the units multiplied
      int items0 = 0, items1 = 0, done0 = 0, done1 = 0;
#pragma unroll 1
      for (int i0 = 0; i0 < count && ok;) {
        const int m = at.nblk - at.blk < count - i0 ? at.nblk - at.blk : count - i0;
        const int len = seq_length(g, at.entry / plan.tiles), row0 = at.entry % plan.tiles * 2 * kTile;
        // units of this item, counted from the share's first one, that each tile takes part in
        auto part_of = [&](int b) {
          const int nb = (plan.seen(len, row0 + b * kTile, row0 + (b + 1) * kTile) + kTile - 1) / kTile;
          return nb - at.blk < m ? (nb - at.blk < 0 ? 0 : nb - at.blk) : m;
        };
        const int to0 = part_of(0), to1 = part_of(1);
        // step i: the outputs of unit i, then the scores of unit i + 1
#pragma unroll 1
        for (int i = -1; i < m && ok; ++i) {
          const int u = i0 + i;
          if (i >= 0) wait(&vfull[u & 1], u >> 1);
          if (i + 1 < m) wait(&kfull[(u + 1) & 1], (u + 1) >> 1);
#pragma unroll 1
          for (int b = 0; b < 2; ++b) {
            const int to = b ? to1 : to0;
            if (i >= to || to == 0) continue;
            if (i < 0) {
              wait(&qfull[b], b ? items1++ : items0++);
            } else {
              wait(&pfull[b], b ? done1++ : done0++);
              outputs(b, u, i == 0);
            }
            if (i + 1 < to) scores(b, u + 1);
          }
          if (i >= 0) commit(&vempty[u & 1]);
          if (i + 1 < m) commit(&kempty[(u + 1) & 1]);
        }
        i0 += m;
        if (i0 < count) at.next_item(plan);
      }
    }
  } else if (warp >= 8) {
    // ---------------- converters ----------------
    // Contiguous copies bring a unit's codes; each thread turns pieces of 16 into fp16, one row
    // of K (channel of V) in every 32: four lanes take 64 codes of a row, so that eight lanes'
    // accesses of 16 bytes fall into different banks.
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
    auto copy = [&](uint8_t *dst, const uint8_t *src, uint64_t *bar) {
      if (ct != 0) return;
      tc::fence_proxy_async_smem();
      tc::mbar_arrive_expect_tx(bar, (place[0] >= 0 ? C::kHalf : 0) + (place[1] >= 0 ? C::kHalf : 0));
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (place[h] >= 0)
          tc::bulk_load(dst + h * C::kHalf, src + (int64_t)place[h] * C::kHalf, C::kHalf, bar);
    };
    const uint32_t at0 = swizzled(r0, 2 * x), at1 = swizzled(r0, 2 * x + 1);
    auto put = [&](uint8_t *rows, const uint4 &q) {
      *reinterpret_cast<uint4 *>(rows + at0) =
          make_uint4(halves_lo(q.x), halves_hi(q.x), halves_lo(q.y), halves_hi(q.y));
      *reinterpret_cast<uint4 *>(rows + at1) =
          make_uint4(halves_lo(q.z), halves_hi(q.z), halves_lo(q.w), halves_hi(q.w));
    };
    auto wait = [&](uint64_t *bar, int phase) {
      if (ok) ok = tc::mbar_wait_compact(bar, phase & 1, st);
    };
    auto arrive = [&](uint64_t *bar) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    // step u: convert unit u, have unit u + 1 copied, look unit u + 2 up
#pragma unroll 1
    for (int u = count > 0 ? -2 : 0; u < count; ++u) {
      const int s = u & 1, tokens = left;
      const int there = (place[0] >= 0 ? 1 : 0) | (place[1] >= 0 ? 2 : 0);
      if (u >= 0) {
      // keys, and what the softmax has to know of the unit (four units back has been read: the
      // keys of two units back were multiplied after the probabilities of three units back)
      wait(kraw, u);
      if (u >= 2) wait(&kempty[s], (u - 2) >> 1);
      if (ct == 0) {
        Info &f = info[u % kInfo];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f.ks[h] = fp8::exp_value((uint8_t)ex[h]);
          f.lv[h] = (ex[h] >> 8) - fp8::kBias;
          f.there[h] = there >> h & 1;
        }
      }
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {       // block; its rows r0 + 32 i, odd rows the other chunk first
        uint4 q[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int ch = D == 128 ? (i / 2) ^ (r0 & 1) : 0;
          q[i] = there >> h & 1 ? *reinterpret_cast<const uint4 *>(
                                      raw_k + h * C::kHalf + (r0 + i % 2 * 32) * D + ch * 64 + x * 16)
                                : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const int ch = D == 128 ? (i / 2) ^ (r0 & 1) : 0;
          put(sk + s * C::kQ + ch * C::kChunk + (h * kTok + i % 2 * 32) * 128, q[i]);
        }
      }
      arrive(&kfull[s]);
      tc::named_barrier(1, 128);  // the codes have been read
      }
      if (u >= -1) {
        locate();                 // of the next unit
        if (u + 1 < count) copy(raw_k, g.k, kraw);
      }
      if (u >= 0) {
      // values; those past the sequence's end may be NaN codes and become zeros
      wait(vraw, u);
      if (u >= 2) wait(&vempty[s], (u - 2) >> 1);
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
      arrive(&vfull[s]);
      tc::named_barrier(1, 128);
      }
      if (u >= -1 && u + 1 < count) copy(raw_v, g.v, vraw);
      look_up(u + 2);
    }
  } else {
    // ---------------- softmax ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int b = warp / 4, row = threadIdx.x % kTile;
    const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
    const uint32_t ts = tmem + lanes + b * kTile, to = tmem + lanes + C::kO + b * D;
    uint8_t *q_tile = sq + b * C::kQ;
    int seen_s = 0, seen_o = 0;  // phases of sfull and odone that have been waited for
    auto wait = [&](uint64_t *bar, int phase) {
      if (ok) ok = tc::mbar_wait_compact(bar, phase & 1, st);
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
      // queries: scaled to a maximum of [1, 2), fp16, K-major
      // Where this thread's row of queries starts, and of outputs (rows that do not exist: row 0).
      const int rq = r < plan.rows ? r / plan.group : 0, hq = r < plan.rows ? r % plan.group : 0;
      const int64_t q_at = seq * g.q_stride[0] + rq * g.q_stride[1] +
                           (int64_t)(at.head * plan.group + hq) * g.q_stride[2];
      const int64_t o_at = seq * g.o_stride[0] + rq * g.o_stride[1] +
                           (int64_t)(at.head * plan.group + hq) * g.o_stride[2];
      // Rows move D / 8 lanes to a row, 16 bytes a lane; `kAt` rows of the warp's 32 at a time.
      constexpr int kLanes = D / 8, kAt = 32 / kLanes;
      const int sub = lane / kLanes, part8 = lane % kLanes, wrow = warp % 4 * 32;
      uint8_t *const mine8 = q_tile + part8 / 8 * C::kChunk;
      // Queries, scaled to a maximum of [1, 2), fp16, K-major; all loads in flight at once, the
      // rest in a small loop (code that runs once an item costs its instructions' fetch).
      float f = 0.0f;
      if (mine > 0) {
        const T *q = (const T *)g.q + 8 * part8;
        const int exist = plan.rows - row0 - wrow;  // of the warp's rows
        if (g.vec_q) {
#pragma unroll 1
          for (int i0 = 0; i0 < 32; i0 += 8 * kAt) {
            uint4 raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int mr = i0 + i * kAt + sub;
              const int64_t off = __shfl_sync(0xffffffffu, q_at, mr);
              raw[i] = mr < exist ? *reinterpret_cast<const uint4 *>(q + off) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4 *>(mine8 + swizzled(wrow + i0 + i * kAt + sub, part8 % 8)) = raw[i];
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < 32; i += kAt) {
            const int64_t off = __shfl_sync(0xffffffffu, q_at, i + sub);
            alignas(16) T e[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) e[j] = i + sub < exist ? q[off + j] : from_f32<T>(0.0f);
            *reinterpret_cast<uint4 *>(mine8 + swizzled(wrow + i + sub, part8 % 8)) =
                *reinterpret_cast<const uint4 *>(e);
          }
        }
#pragma unroll 4
        for (int i = 0; i < 32; i += kAt) {
          const int mr = wrow + i + sub;
          uint4 *const slot = reinterpret_cast<uint4 *>(mine8 + swizzled(mr, part8 % 8));
          uint4 w = *slot;
          float rf = fabsf(g.scale) * kLog2e;
          if constexpr (std::is_same<T, __half>::value) {  // as they are, but for a negative scale
            const uint32_t flip = g.scale < 0.0f ? 0x80008000u : 0u;
            w = make_uint4(w.x ^ flip, w.y ^ flip, w.z ^ flip, w.w ^ flip);
          } else {
            __nv_bfloat162 h[4];
            memcpy(h, &w, 16);
            const __nv_bfloat162 top = __hmax2(__hmax2(__habs2(h[0]), __habs2(h[1])),
                                               __hmax2(__habs2(h[2]), __habs2(h[3])));
            float amax = fmaxf(__low2float(top), __high2float(top));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1)
              amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int e = row_exponent(amax);
            const float inv = g.scale < 0.0f ? -fp8::pow2(-e) : fp8::pow2(-e);
            rf *= fp8::pow2(e);
            w = make_uint4(pack_half2(__low2float(h[0]) * inv, __high2float(h[0]) * inv),
                           pack_half2(__low2float(h[1]) * inv, __high2float(h[1]) * inv),
                           pack_half2(__low2float(h[2]) * inv, __high2float(h[2]) * inv),
                           pack_half2(__low2float(h[3]) * inv, __high2float(h[3]) * inv));
          }
          if (part8 == 0) factor[b * kTile + mr] = rf;
          *slot = w;
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();  // O of the item before has been read
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&qfull[b]);
        f = factor[b * kTile + row];
      }
      float base = -INFINITY, l = 0.0f;  // the exponent that p is taken from; sum of p 2^-lv
      for (int i = 0; i < mine && ok; ++i) {
        wait(&sfull[b], seen_s++);
        const Info &in = info[(i0 + i) % kInfo];
        const int tok = (at.blk + i) * kTile;
        const int there = in.there[0] | in.there[1] << 1;
        const bool cut = !__all_sync(0xffffffffu, tok + kTile <= limit) || there != 3;
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(ts + 32 * c, s[c]);
        tc::tmem_ld_wait();
        if (cut) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int seen = (there >> (c / 2)) & 1 ? limit - tok - 32 * c : 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) s[c][j] = j < seen ? s[c][j] : 0xFF800000u;
          }
        }
        float top = -INFINITY, fk[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) a[q] = __uint_as_float(s[2 * h + q / 2][q % 2 * 16]);
#pragma unroll
          for (int j = 1; j < 15; j += 2)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              a[q] = max3(a[q], __uint_as_float(s[2 * h + q / 2][q % 2 * 16 + j]),
                          __uint_as_float(s[2 * h + q / 2][q % 2 * 16 + j + 1]));
#pragma unroll
          for (int q = 0; q < 4; ++q)
            a[q] = fmaxf(a[q], __uint_as_float(s[2 * h + q / 2][q % 2 * 16 + 15]));
          // a factor of 0 would turn the masked -inf into NaN
          fk[h] = fmaxf(f * in.ks[h], 1e-37f);
          top = fmaxf(top, fmaf(fmaxf(max3(a[0], a[1], a[2]), a[3]), fk[h], (float)in.lv[h]));
        }
        const bool raise = top > base + kLazy || (base == -INFINITY && top > base);
        if (i > 0 && __any_sync(0xffffffffu, raise)) {
          const float shrink = raise ? ex2(base - top) : 1.0f;
          l *= shrink;
          wait(&odone[b], seen_o + i - 1);
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
        if (raise) base = top;
        const float ref = (base == -INFINITY ? 0.0f : base) - 8.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float off = (float)in.lv[h] - ref;
          const float2 fk2 = make_float2(fk[h], fk[h]), off2 = make_float2(off, off);
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int c = 2 * h; c < 2 * h + 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 y = fma2(make_float2(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1])),
                              fk2, off2);
              y = make_float2(ex2(y.x), ex2(y.y));
              sum[j % 2] = add2(sum[j % 2], y);
              w[j] = pack_half2(y.x, y.y);
            }
            tmem_st16(ts + 16 * c, w);
          }
          sum[0] = add2(sum[0], sum[1]);
          l = fmaf((sum[0].x + sum[0].y) * 0x1p-8f, fp8::pow2(-in.lv[h]), l);
        }
        tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&pfull[b]);
      }
      // the item's end, here or in the next share
      seen_o += mine;
      if (mine > 0) wait(&odone[b], seen_o - 1);
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
          // through the tile of queries, whose products are done: rows of 2 D bytes
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            alignas(16) T e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = from_f32<T>(__uint_as_float(x[j + q]));
            const int u = (c + j) / 8;
            *reinterpret_cast<uint4 *>(q_tile + u / 8 * C::kChunk + swizzled(row, u % 8)) =
                *reinterpret_cast<const uint4 *>(e);
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
        const int exist = plan.rows - row0 - wrow;
#pragma unroll 4
        for (int i = 0; i < 32; i += kAt) {
          const int64_t off = __shfl_sync(0xffffffffu, o_at, i + sub);
          if (i + sub >= exist) continue;
          const uint4 w = *reinterpret_cast<const uint4 *>(mine8 + swizzled(wrow + i + sub, part8 % 8));
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
  using C = Prompt<D>;
  GPTQ_TRY(ensure_smem_attr((const void *)prompt_kernel<T, D>, (int)C::kSmem));
  int sms = 0;
  GPTQ_TRY(device_sm_count(&sms));
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  float *part = (float *)((char *)ws + 256);
  GPTQ_TRY(launch_early(prompt_kernel<T, D>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, 1, s, g,
                        part, (DevStatus *)ws));
  return launch_early(join_kernel<T, D, PromptPlan>, dim3((unsigned)ctas - 1, 8), dim3(128), 0, 1, s,
                      g, (const float *)part, 1, ctas);
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

gptq_status launch_kv8_prompt(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  if (!kv8_plan_fits(g, 2 * kTile, 2, PromptPlan::kSetup)) return GPTQ_ERR_UNSUPPORTED;
  if (g.dtype == GPTQ_F16)
    return g.dim == 64 ? run<__half, 64>(g, ws, s) : run<__half, 128>(g, ws, s);
  return g.dim == 64 ? run<__nv_bfloat16, 64>(g, ws, s) : run<__nv_bfloat16, 128>(g, ws, s);
}

}  // namespace gptq
