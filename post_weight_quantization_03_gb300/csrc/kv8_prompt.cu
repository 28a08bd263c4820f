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
//             softmax warps more than converting the values costs here.)  A row of queries is
//             scaled by a power of two to a maximum of [1, 2); the scores are fp32 in TMEM.
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

#include "kv8.cuh"

namespace gptq {

namespace {

using namespace kv8;

constexpr int kTile = 128;                      // rows of an MMA tile, tokens of a unit
using PromptPlan = Plan<2 * kTile, kTile>;
// Registers by warp group: 2 x 128 x 192 + 128 x 80 + 128 x 40 = 64,512 of the 65,536 that 512
// threads have at launch.
constexpr int kThreads = 512;
constexpr int kInfo = 4;
constexpr float kLazy = 6.0f;

template <int D>
struct Prompt {
  static constexpr uint32_t kChunk = kTile * 128;             // 128 rows of 128 bytes
  static constexpr uint32_t kQ = kTile * D * 2;               // a tile of queries (or keys)
  static constexpr uint32_t kV = D * kTile * 2;               // values, channel-major
  static constexpr uint32_t kVChunk = D * 128;                // 64 tokens of them
  static constexpr size_t kSmem = 1024 + 2 * kQ + 2 * kQ + 2 * kV + kInfo * 32 + 256;
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t halves(uint32_t two) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
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
  Info *info = (Info *)(sv + 2 * C::kV);
  uint64_t *qfull = (uint64_t *)(info + kInfo);   // [2], by tile
  uint64_t *sfull = qfull + 2, *pfull = sfull + 2, *odone = pfull + 2;
  uint64_t *kfull = odone + 2, *kempty = kfull + 2, *vfull = kempty + 2, *vempty = vfull + 2;
  uint32_t *tmem_slot = (uint32_t *)(vempty + 2);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

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
  const int64_t total = plan.total();
  const int64_t n = shares(total, 1, gridDim.x);
  const int64_t u0 = blockIdx.x < n ? share_start(total, n, blockIdx.x) : 0;
  const int count = blockIdx.x < n ? (int)(share_start(total, n, blockIdx.x + 1) - u0) : 0;
  Cursor at{};
  if (count > 0) at = cursor_at(plan, u0);
  bool ok = true;  // false once a wait has given up: the rest passes without waiting

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 12 && lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t id_s = tc::instr_desc(0, 0, kTile, kTile, 0, 0);
      constexpr uint32_t id_o = tc::instr_desc(0, 0, kTile, D, 0, 0);
      const uint32_t q0 = tc::smem_u32(sq), k0 = tc::smem_u32(sk), v0 = tc::smem_u32(sv);
      auto wait = [&](uint64_t *bar, int phase) {
        if (ok) ok = tc::mbar_wait(bar, phase & 1, st);
        tc::tc_fence_after();
      };
      auto scores = [&](int b, int u) {
        const uint32_t q = q0 + b * C::kQ, k = k0 + (u & 1) * C::kQ;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t off = (uint32_t)(i / 4) * C::kChunk + (i % 4) * 32;
          tc::mma_f16(tmem + b * kTile, tc::smem_desc_sw128(q + off, 16, 1024),
                      tc::smem_desc_sw128(k + off, 16, 1024), id_s, i > 0);
        }
        tc::mma_commit(&sfull[b]);
      };
      auto outputs = [&](int b, int u, bool first) {
        const uint32_t v = v0 + (u & 1) * C::kV;
#pragma unroll
        for (int i = 0; i < kTile / 16; ++i)
          mma_f16_ts(tmem + C::kO + b * D, tmem + b * kTile + 8 * i,
                     tc::smem_desc_sw128(v + (uint32_t)(i / 4) * C::kVChunk + (i % 4) * 32, 16, 1024),
                     id_o, !first || i > 0);
        tc::mma_commit(&odone[b]);
      };
      int items[2] = {0, 0}, done[2] = {0, 0};  // by tile: items and units it took part in
      for (int i0 = 0; i0 < count && ok;) {
        const int m = at.nblk - at.blk < count - i0 ? at.nblk - at.blk : count - i0;
        const int len = seq_length(g, at.entry / plan.tiles), row0 = at.entry % plan.tiles * 2 * kTile;
        // units of this item, counted from the share's first one, that each tile takes part in
        int to[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int nb = (plan.seen(len, row0 + b * kTile, row0 + (b + 1) * kTile) + kTile - 1) / kTile;
          to[b] = nb - at.blk < m ? (nb - at.blk < 0 ? 0 : nb - at.blk) : m;
        }
        wait(&kfull[i0 & 1], i0 >> 1);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          if (to[b] == 0) continue;
          wait(&qfull[b], items[b]++);
          scores(b, i0);
        }
        tc::mma_commit(&kempty[i0 & 1]);
        for (int i = 0; i < m && ok; ++i) {
          const int u = i0 + i;
          wait(&vfull[u & 1], u >> 1);
          if (i + 1 < m) wait(&kfull[(u + 1) & 1], (u + 1) >> 1);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (i >= to[b]) continue;
            wait(&pfull[b], done[b]);
            outputs(b, u, i == 0);
            ++done[b];
            if (i + 1 < to[b]) scores(b, u + 1);
          }
          tc::mma_commit(&vempty[u & 1]);
          if (i + 1 < m) tc::mma_commit(&kempty[(u + 1) & 1]);
        }
        i0 += m;
        if (i0 < count) at.next_item(plan);
      }
    }
  } else if (warp >= 8) {
    // ---------------- converters ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    const int ct = threadIdx.x - 256;
    // K pieces of 16 codes: four lanes a row of 64, so that eight lanes' stores of 16 bytes fall
    // into different banks; V pieces: four lanes a channel of 64 tokens
    Cursor c = at;              // of the unit whose blocks are looked up
    int pages[2], head = 0, len = 0, blk = 0;
    auto look_up = [&](int u) {
      pages[0] = pages[1] = -1;
      if (u >= count) return;
      const int seq = c.entry / plan.tiles;
      const int32_t *row = g.table + seq * g.ld_table;
      head = c.head;
      len = seq_length(g, seq);
      blk = c.blk;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((2 * blk + h) * kTok < len) pages[h] = row[2 * blk + h];
      if (u + 1 < count) c.advance(plan, 1);
    };
    int place[2], ex[2], left;   // of the unit whose codes are on their way
    uint4 kq[D / 16], vq[D / 16];
    auto locate = [&]() {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        place[h] = pages[h] < 0 || pages[h] >= g.n_blocks ? -1 : pages[h] * g.n_kv + head;
        ex[h] = place[h] < 0 ? fp8::kBias * 257
                             : (int)g.k_exps[place[h]] | ((int)g.v_exps[place[h]] << 8);
      }
      left = len - blk * kTile;  // tokens of the unit that exist
    };
    constexpr int kPer = D / 16;          // pieces of K (of V) per thread
    constexpr int kColsOf = D / 64;       // 64-element chunks of a K row
    auto load_k = [&]() {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = ct + 128 * i, x = piece % 4, row = piece / 4 % kTile, ch = piece / (4 * kTile);
        const int h = row / kTok;
        kq[i] = place[h] < 0 ? make_uint4(0, 0, 0, 0)
                             : *reinterpret_cast<const uint4 *>(
                                   g.k + (int64_t)place[h] * (kTok * D) + (row % kTok) * D + ch * 64 + x * 16);
      }
    };
    auto load_v = [&]() {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = ct + 128 * i, x = piece % 4, d = piece / 4 % D, h = piece / (4 * D);
        vq[i] = place[h] < 0 ? make_uint4(0, 0, 0, 0)
                             : *reinterpret_cast<const uint4 *>(
                                   g.v + (int64_t)place[h] * (kTok * D) + d * kTok + x * 16);
      }
    };
    auto put = [&](uint8_t *chunk, int row, int x, const uint4 &q) {
      *reinterpret_cast<uint4 *>(chunk + swizzled(row, 2 * x)) =
          make_uint4(halves(q.x), halves(q.x >> 16), halves(q.y), halves(q.y >> 16));
      *reinterpret_cast<uint4 *>(chunk + swizzled(row, 2 * x + 1)) =
          make_uint4(halves(q.z), halves(q.z >> 16), halves(q.w), halves(q.w >> 16));
    };
    auto wait = [&](uint64_t *bar, int phase) {
      if (ok) ok = tc::mbar_wait(bar, phase & 1, st);
    };
    auto arrive = [&](uint64_t *bar) {
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar);
    };
    static_assert(kColsOf * 4 * kTile == kPer * 128, "K pieces");
    if (count > 0) {
      look_up(0);
      locate();
      load_k();
      load_v();
      look_up(1);
    }
    for (int u = 0; u < count && ok; ++u) {
      const int s = u & 1, tokens = left;
      // keys, and what the softmax has to know of the unit (four units back has been read: the
      // keys of two units back were multiplied after the probabilities of three units back)
      if (u >= 2) wait(&kempty[s], (u - 2) >> 1);
      if (ct == 0) {
        Info &f = info[u % kInfo];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f.ks[h] = fp8::exp_value((uint8_t)ex[h]);
          f.lv[h] = (ex[h] >> 8) - fp8::kBias;
          f.there[h] = place[h] >= 0;
        }
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = ct + 128 * i, x = piece % 4, row = piece / 4 % kTile, ch = piece / (4 * kTile);
        put(sk + s * C::kQ + ch * C::kChunk, row, x, kq[i]);
      }
      arrive(&kfull[s]);
      locate();                 // of the next unit
      if (u + 1 < count) load_k();
      // values; those past the sequence's end may be NaN codes and become zeros
      if (u >= 2) wait(&vempty[s], (u - 2) >> 1);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int piece = ct + 128 * i, x = piece % 4, d = piece / 4 % D, h = piece / (4 * D);
        const int live = tokens - h * kTok - x * 16;
        if (live < 16) {
          uint32_t e[4] = {vq[i].x, vq[i].y, vq[i].z, vq[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int keep = live - 4 * q;
            e[q] &= keep <= 0 ? 0u : (keep >= 4 ? ~0u : (1u << (8 * keep)) - 1u);
          }
          vq[i] = make_uint4(e[0], e[1], e[2], e[3]);
        }
        put(sv + s * C::kV + h * C::kVChunk, d, x, vq[i]);
      }
      arrive(&vfull[s]);
      if (u + 1 < count) load_v();
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
      if (ok) ok = tc::mbar_wait(bar, phase & 1, st);
      ok = __all_sync(0xffffffffu, ok);
      tc::tc_fence_after();
    };
    for (int i0 = 0; i0 < count && ok;) {
      const int m = at.nblk - at.blk < count - i0 ? at.nblk - at.blk : count - i0;
      const int seq = at.entry / plan.tiles, row0 = at.entry % plan.tiles * 2 * kTile + b * kTile;
      const int len = seq_length(g, seq), r = row0 + row;
      const int nb = (plan.seen(len, row0, row0 + kTile) + kTile - 1) / kTile;
      const int mine = nb - at.blk < m ? (nb - at.blk < 0 ? 0 : nb - at.blk) : m;
      const int limit = plan.seen(len, r, r + 1);
      // queries: scaled to a maximum of [1, 2), fp16, K-major
      float f = 0.0f;
      if (mine > 0) {
        const bool real = r < plan.rows;
        const T *q = (const T *)g.q + seq * g.q_stride[0] + (r / plan.group) * g.q_stride[1] +
                     (int64_t)(at.head * plan.group + r % plan.group) * g.q_stride[2];
        const bool vec = ((uintptr_t)q & 15) == 0;
        auto load = [&](int d, float(&v)[8]) {
          if (!real) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
          } else if (vec) {
            const uint4 w = *reinterpret_cast<const uint4 *>(q + d);
            const T *e = reinterpret_cast<const T *>(&w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f32(e[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f32(q[d + j]);
          }
        };
        float amax = 0.0f;
#pragma unroll
        for (int d = 0; d < D; d += 8) {
          float v[8];
          load(d, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fp8::finite_abs(v[j]));
        }
        const int e = row_exponent(amax);
        const float inv = g.scale < 0.0f ? -fp8::pow2(-e) : fp8::pow2(-e);
        f = fp8::pow2(e) * fabsf(g.scale) * kLog2e;
#pragma unroll
        for (int d = 0; d < D; d += 8) {
          float v[8];
          load(d, v);
          *reinterpret_cast<uint4 *>(q_tile + d / 64 * C::kChunk + swizzled(row, d % 64 / 8)) =
              make_uint4(pack_half2(v[0] * inv, v[1] * inv), pack_half2(v[2] * inv, v[3] * inv),
                         pack_half2(v[4] * inv, v[5] * inv), pack_half2(v[6] * inv, v[7] * inv));
        }
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();  // O of the item before has been read
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&qfull[b]);
      }
      float base = -INFINITY, l = 0.0f;  // the exponent that p is taken from; sum of p 2^-lv
      for (int i = 0; i < mine && ok; ++i) {
        wait(&sfull[b], seen_s++);
        const Info in = info[(i0 + i) % kInfo];
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc::tmem_ld32(ts + 32 * c, s[c]);
        tc::tmem_ld_wait();
        const int tok = (at.blk + i) * kTile;
        // a factor of 0 would turn the masked -inf into NaN
        const float fk[2] = {fmaxf(f * in.ks[0], 1e-37f), fmaxf(f * in.ks[1], 1e-37f)};
        if (!__all_sync(0xffffffffu, tok + kTile <= limit) || !in.there[0] || !in.there[1]) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (tok + 32 * c + j >= limit || !in.there[c / 2]) s[c][j] = 0xFF800000u;
        }
        float mx[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            a0 = fmaxf(a0, __uint_as_float(s[2 * h][j]));
            a1 = fmaxf(a1, __uint_as_float(s[2 * h + 1][j]));
          }
          mx[h] = fmaf(fmaxf(a0, a1), fk[h], (float)in.lv[h]);
        }
        const float top = fmaxf(mx[0], mx[1]);
        const bool raise = top > base + kLazy || (base == -INFINITY && top > base);
        if (i > 0 && __any_sync(0xffffffffu, raise)) {
          const float shrink = raise ? ex2(base - top) : 1.0f;
          l *= shrink;
          wait(&odone[b], seen_o + i - 1);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tc::tmem_ld32(to + c, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * shrink);
            tmem_st32(to + c, o);
          }
        }
        if (raise) base = top;
        const float ref = base == -INFINITY ? 0.0f : base;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float off = (float)in.lv[h] - ref + 8.0f;
          float sum0 = 0.0f, sum1 = 0.0f;
          uint32_t w[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float p0 = ex2(fmaf(__uint_as_float(s[2 * h + j / 16][2 * (j % 16)]), fk[h], off));
            const float p1 = ex2(fmaf(__uint_as_float(s[2 * h + j / 16][2 * (j % 16) + 1]), fk[h], off));
            sum0 += p0;
            sum1 += p1;
            w[j] = pack_half2(p0, p1);
          }
          tmem_st32(ts + 32 * h, w);
          l = fmaf((sum0 + sum1) * 0x1p-8f, fp8::pow2(-in.lv[h]), l);
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
      const bool real = r < plan.rows;
      T *o = out_row<T>(g, plan.group, seq, at.head, real ? r : 0);
      const bool vec = ((uintptr_t)o & 15) == 0;
      float *po = piece + (b * kTile + row) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t x[32];
        if (mine > 0) {
          tc::tmem_ld32(to + c, x);
          tc::tmem_ld_wait();
        }
        if (!real) continue;
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) y[j] = mine > 0 ? __uint_as_float(x[j]) * inv : 0.0f;
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(po + c + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
        } else if (vec) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            alignas(16) T e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = from_f32<T>(y[j + q]);
            *reinterpret_cast<uint4 *>(o + c + j) = *reinterpret_cast<const uint4 *>(e);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[c + j] = from_f32<T>(y[j]);
        }
      }
      if (!whole && real) {
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
  GPTQ_TRY(launch_early(prompt_kernel<T, D>, dim3((unsigned)ctas), dim3(kThreads), C::kSmem, s, g,
                        part, (DevStatus *)ws));
  return launch_early(join_kernel<T, D, PromptPlan>, dim3((unsigned)ctas - 1, 8), dim3(128), 0, s,
                      g, (const float *)part, 1, (int64_t)ctas);
}

}  // namespace

size_t kv8_prompt_ws_bytes(int n_seq, int64_t n_new, int n_heads, int n_kv, int dim,
                           int max_blocks) {
  int64_t ctas = kMaxCtas;
  const int64_t rows = n_new * (n_heads / n_kv);
  const int64_t units = ceil_div(rows, 2 * kTile) * n_seq * n_kv * ceil_div(max_blocks, 2);
  if (units < ctas) ctas = units;
  return 256 + (size_t)(2 * ctas) * (2 * kTile) * (dim + 2) * 4;
}

gptq_status launch_kv8_prompt(const Kv8AttentionArgs &g, void *ws, cudaStream_t s) {
  const int64_t rows = g.n_new * (g.n_heads / g.n_kv);
  if (rows > INT32_MAX / 2 || ceil_div(rows, 2 * kTile) * g.n_seq > INT32_MAX / 2)
    return GPTQ_ERR_UNSUPPORTED;
  if (g.dtype == GPTQ_F16)
    return g.dim == 64 ? run<__half, 64>(g, ws, s) : run<__half, 128>(g, ws, s);
  return g.dim == 64 ? run<__nv_bfloat16, 64>(g, ws, s) : run<__nv_bfloat16, 128>(g, ws, s);
}

}  // namespace gptq
