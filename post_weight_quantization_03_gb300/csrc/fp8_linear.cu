// Block-scaled e4m3 products with an epilogue, of one weight matrix or of one for each expert:
//   out = act(ra rw (A W^T) + bias) + residual                       (16 bits)
//   v = act(G) * U, G and U two such products of one A               (e4m3 codes by 1 x 128 blocks)
//
// The tile and the roles are those of the plain product (fp8_matmul.cu): the weights' 128 rows are
// the MMA's M, up to `tn` tokens its N, both block scales are applied in the tensor core.
//
//   warp 0     : TMA producer: (gate, up, tokens) of 128 bytes x rows per k-block
//   warp 1     : TMEM allocator + MMA issuer (one lane)
//   warps 2..9 : epilogue, two warps for each 32 weight rows, which take tokens in turn
//   warp 10    : scales
//   11..18     : copy token rows (the experts' gated product)
// (clusters that share a tile in the experts' gated product: 4 warps of epilogue, 4 that copy)
//
// Gated: a tile has 128 rows of both weights and two accumulators, so the 128 outputs that share an
// exponent are one column of the tile.  A warp turns 32 rows by 16 tokens around in shared memory, so
// that two lanes have a token's 32 outputs; their maximum meets those of three other warps.
//
// Experts: a tile is (expert, up to tn of its positions, 128 weight rows).  Each CTA counts the
// tiles from the offsets by itself.  The gated product takes its token rows by index, the other takes
// them as they lie and stores each where the order says, so that neither the rows nor the results
// are moved by a kernel of their own.  Rows by index are copied by eight warps, 16 bytes a lane, into the
// swizzle that the MMA reads: TMA's gather of four rows takes about 80 cycles, 2300 for a k-block whose
// MMAs take 770 (4096 tokens of 64 experts, 4096 x 1376: 709 us then).
//
// 16-bit outputs are turned around likewise, so that a store writes 64 contiguous bytes of four tokens.
//
// Few tokens leave few tiles; each cluster of up to 8 CTAs then has one, whose k-blocks they share, and
// their partial sums meet through distributed shared memory in rank order.
//
// Bounds, and what it measured (GPU time, tokens x n x k; TB/s: bytes of operands by time).  Few
// tokens: the weights' bytes, at 5.3 to 6.4 TB/s once under way, and 3.5 to 6 us for a CTA's set-up,
// the first copies and the end: linear 1 x 4096 x 11008 10.5 us (6.7 of them the bytes), gated 24 x
// 11008 x 4096 17.8 (13.6), experts gated 1 token of 6 of 64 x 1376 x 4096 16.8 (10.1), experts out 40
// tokens x 4096 x 1376 52.8, 6.8 TB/s.  Many: the tensor pipe, active in 69 % of the cycles of gated
// 4096 x 11008 x 4096: 238 us, 3.1 PFLOP/s (270 in a longer row of calls, at the power limit; what
// idles the pipe has not been found: a third fewer bytes from L2 changed 1 %).  The experts' tiles
// have fewer tokens for their weights' way from L2: gated 4096 tokens of 6 of 64 x 1376 x 4096 237 us,
// 2.3 PFLOP/s, 53 %.  linear 8192 x 11008 x 4096 234 us, 3.2 PFLOP/s, with a residual 252.  Short K:
// the epilogue, which takes as long however few the MMAs are: linear 24576 x 4096 x 1376 124 us (x
// 128: 98), experts out 4096 tokens x 4096 x 1376 170 (x 128: 138), gated 4096 x 11008 x 1024 109 (x
// 256: 98).
#include <cudaTypedefs.h>
#include <math.h>

#include "mx.cuh"
#include "per_device.cuh"

namespace gptq {

namespace {

using mx::BK;
using mx::BM;
using mx::copy_scales;
using mx::out_f32;

constexpr int kMaxTn = 240;
constexpr int kMaxTnGated = 112;            // two accumulators, for this tile and the next
constexpr int kScaleStages = 4;             // groups of four k-blocks in flight
// A group of scales in shared memory: weights, second weights, tokens 0..127, tokens 128..239.
__host__ __device__ constexpr uint32_t scale_bytes(int tn) { return tn > 128 ? 4 * 512 : 3 * 512; }
constexpr uint32_t kScaleCols = 16;         // TMEM columns of one group
constexpr int kMaxStages = 12;
constexpr int kBox = 64;                    // rows of A in a copy of the experts' plain product, at most
constexpr int64_t kAcross = 16;            // (about as many tiles along the tokens run with them)
constexpr uint32_t kTmemCols = 512;
constexpr int kTurnPitch = 36;              // (words in different banks along either way)
constexpr size_t kSmem = 227 * 1024;        // of a CTA alone on its SM
constexpr size_t kSmemTwo = 113 * 1024;     // of one of two
constexpr size_t kSmemLeast = 40 * 1024;
constexpr size_t kBarBytes = 512;
static_assert(2 * kMaxTn + 2 * kScaleCols <= kTmemCols, "TMEM columns");
static_assert(4 * kMaxTnGated + 2 * kScaleCols <= kTmemCols, "TMEM columns");

struct Params {
  const uint8_t *a; int64_t lda, K;
  const uint8_t *ae; int64_t ldae;
  const float *ra;
  const uint8_t *we[2]; int64_t ldwe[2], next_we[2];
  const float *rw[2], *bias[2];
  const void *residual; int64_t ldr;
  void *out; int64_t ldo;
  uint8_t *oe; int64_t ldoe;
  int64_t a_rows, M, N;
  int act;
  int kb;               // k-blocks
  int wide;             // rows of the output and the residual allow 8 bytes at a time
  int tn, stages;
  int box;              // rows of A that a copy takes (experts' plain product)
  int n_w, n_m;         // tiles along the weights; along the tokens (not of experts)
  int across;           // tiles along the weights that are gone through for all tokens before the next
  int splits;           // CTAs of a cluster that share a tile's k-blocks
  int acc_cols;         // columns of an accumulator
  int tmem_cols;
  uint32_t ring_bytes;
  const int32_t *offsets, *order;
  int n_experts, top_k;
  uint32_t per_tn, per_k;   // 2^32 / tn, / top_k, rounded up: quotients of numbers below 2^23
  uint64_t wait_ns;
  int lost;             // test hook: this copy of the producer's is left out
};

__device__ int g_gave_up;  // a wait ran out since it was last asked for

// (1 + exp(-x) overflows, or passes 2^126, only where x / that is below 2^-119 or so: 0)
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }
__device__ __forceinline__ float gelu(float x) { return 0.5f * x * (1.0f + erff(x * 0.70710678f)); }
__device__ __forceinline__ float relu(float x) { return x < 0.0f ? 0.0f : x; }
template <int N>
__device__ __forceinline__ void activate(float (&x)[N], int act) {
  if (act == GPTQ_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = silu(x[i]);
  } else if (act == GPTQ_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = gelu(x[i]);
  } else if (act == GPTQ_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = relu(x[i]);
  }
}

// a / b of a below 2^22, in a third of the instructions of the exact quotient of any (each tile starts
// with some in every role).
__device__ __forceinline__ int quotient(int a, int b) {
  int q = __float2int_rz(__fdividef((float)a, (float)b));
  const int r = a - q * b;
  return q + (r >= b) - (r < 0);
}

// k-blocks of this CTA: rank r of the cluster takes an even share of the groups of four.
__device__ __forceinline__ void k_range(const Params &p, int rank, int &k0, int &k1) {
  const int groups = (p.kb + 3) / 4;
  k0 = quotient(groups * rank, p.splits) * 4;
  k1 = min(quotient(groups * (rank + 1), p.splits) * 4, p.kb);
}

// Where the experts' positions and tiles begin, in shared memory.
struct Plan {
  int *at;      // [n_experts + 1] positions
  int *tiles;   // [n_experts + 1] tiles of tn positions
  const int *order;   // of all positions: where there are few in shared memory, so that copies of rows by
                      // index are not asked for after all of the weights' (they then came 4 us late)
};
constexpr int kFewPositions = 512;

struct Tile {
  int e, n;             // expert; tile along the weights
  int m0, cols;         // positions
};

// ONE: the grid is (CTAs of a cluster, tiles along the weights, along the tokens).
template <bool EXPERTS, bool ONE>
__device__ __forceinline__ Tile tile_of(const Params &p, const Plan &plan, int t) {
  Tile r;
  int m;
  if constexpr (EXPERTS) {
    m = ONE ? blockIdx.z : t < (1 << 22) ? quotient(t, p.n_w) : t / p.n_w;
    r.n = ONE ? blockIdx.y : t - m * p.n_w;
    int lo = 0, hi = p.n_experts;   // tiles[lo] <= m < tiles[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (plan.tiles[mid] <= m) lo = mid;
      else hi = mid;
    }
    // an expert's tiles are of even size, in whole groups of 16
    const int tiles = plan.tiles[lo + 1] - plan.tiles[lo], count = plan.at[lo + 1] - plan.at[lo];
    const int size = (quotient(count + tiles - 1, tiles) + 15) / 16 * 16, from = (m - plan.tiles[lo]) * size;
    r.e = lo;
    r.m0 = plan.at[lo] + from;
    r.cols = min(count - from, size);   // (above 0: size is at most tn)
  } else {
    if constexpr (ONE) {
      r.n = blockIdx.y;
      m = blockIdx.z;
    } else {
      // runs of `across` tiles along the weights, each for all tokens
      const int per_run = p.across * p.n_m, run = t < (1 << 22) ? quotient(t, per_run) : t / per_run;
      const int n0 = run * p.across, width = min(p.across, p.n_w - n0), in_run = t - n0 * p.n_m;
      m = in_run < (1 << 22) ? quotient(in_run, width) : in_run / width;
      r.n = n0 + in_run - m * width;
    }
    r.e = 0;
    r.m0 = m * p.tn;
    r.cols = (int)min(p.M - r.m0, (int64_t)p.tn);
  }
  return r;
}

// The word of a row's last one to three exponents.
__device__ __forceinline__ uint32_t last_exponents(const uint8_t *from, int n) {
  return (uint32_t)from[0] | (n > 1 ? (uint32_t)from[1] << 8 : 0u) | (n > 2 ? (uint32_t)from[2] << 16 : 0u);
}

// A's row of a position, a_rows (read as zeros) for none.
template <bool GATHER>
__device__ __forceinline__ int a_row(const Params &p, const Plan &plan, int pos) {
  if constexpr (GATHER) {
    const int o = plan.order[pos], row = o < 0 || p.top_k == 1 ? o : (int)__umulhi((uint32_t)o, p.per_k);
    return row >= 0 && row < p.a_rows ? row : (int)p.a_rows;
  }
  return pos;
}

// One warp: the plan from the offsets, which are limited to [0, M] and read as increasing.
__device__ __forceinline__ void make_plan(const Params &p, const Plan &plan, int lane) {
  const int each = (p.n_experts + 31) / 32, e0 = lane * each, e1 = min(e0 + each, p.n_experts);
  const int most = (int)p.M;
  int top = 0;   // the largest offset of this lane's
#pragma unroll 4
  for (int e = e0; e < e1; ++e) {
    const int o = min(p.offsets[e], most);
    plan.at[e] = o;
    top = max(top, o);
  }
  const int end = min(p.offsets[p.n_experts], most);
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, top, o);
    if (lane >= o) top = max(top, v);
  }
  const int all = max(__shfl_sync(0xffffffffu, top, 31), end);
  int at = __shfl_up_sync(0xffffffffu, top, 1);
  if (lane == 0) at = 0;
  int begin = all;   // of this lane's first expert
  for (int e = e0; e < e1; ++e) {
    plan.at[e] = at = max(at, plan.at[e]);
    if (e == e0) begin = at;
  }
  int next = __shfl_down_sync(0xffffffffu, begin, 1);
  if (lane == 31) next = all;
  auto tiles_of = [&](int e) {
    const int count = (e + 1 < e1 ? plan.at[e + 1] : next) - plan.at[e];
    return (int)__umulhi((uint32_t)(count + p.tn - 1), p.per_tn);
  };
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += tiles_of(e);
  int run = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  int tiles = run - sum;
  for (int e = e0; e < e1; ++e) {
    plan.tiles[e] = tiles;
    tiles += tiles_of(e);
  }
  if (lane == 31) {
    plan.at[p.n_experts] = all;
    plan.tiles[p.n_experts] = run;
  }
}

// Shared memory of the epilogue that goes from tile to tile.
__host__ __device__ constexpr size_t direct_bytes(int epilogue) {
  return 2 * 256 * 4 + epilogue * 16 * kTurnPitch * 4 + 2 * 2 * 4 * 16 * 4;
}

template <bool GATED, bool EXPERTS, bool ONE>
struct Warps {
  static constexpr int kEpilogue = ONE && GATED && EXPERTS ? 4 : 8;   // (registers of two CTAs an SM)
  static constexpr int kLoaders = ONE ? 4 : 8;   // copy rows by index, if there is such a thing
  static constexpr int kAll = 3 + kEpilogue + (GATED && EXPERTS ? kLoaders : 0);
};

// ONE: each cluster has one tile, whose k-blocks its CTAs share; their sums lie in shared memory, where
// a warp of one of them adds up and finishes a token's.  Two such CTAs can be on an SM, of one call or of two in a row,
// so that one sets itself up while the other ends.  Else a CTA goes from tile to tile, with a set of
// accumulators for the MMAs and one for the epilogue.  TO: type of the output, if it is not gated.
template <typename TO, bool GATED, bool EXPERTS, bool ONE>
__global__ void __launch_bounds__(32 * Warps<GATED, EXPERTS, ONE>::kAll, ONE ? 2 : 1)
linear_kernel(const __grid_constant__ CUtensorMap mw0, const __grid_constant__ CUtensorMap mw1,
              const __grid_constant__ CUtensorMap ma, Params p, DevStatus *st) {
  constexpr int W = GATED ? 2 : 1;
  constexpr bool GATHER = GATED && EXPERTS;
  constexpr int E = Warps<GATED, EXPERTS, ONE>::kEpilogue, kLoaders = Warps<GATED, EXPERTS, ONE>::kLoaders;
  constexpr int kSets = ONE ? 1 : 2;  // of accumulators
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sscale = ring + p.ring_bytes;
  uint64_t *full = (uint64_t *)(sscale + kScaleStages * scale_bytes(p.tn));
  uint64_t *empty = full + kMaxStages;
  uint64_t *sfull = empty + kMaxStages;
  uint64_t *sempty = sfull + kScaleStages;
  uint64_t *tfull = sempty + kScaleStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *mdone = tempty + 2;       // every MMA has completed
  uint32_t *tmem_slot = (uint32_t *)(mdone + 1);
  // not ONE: of each token (256) its factor and its row of the output (-1: none); the 16 tokens x 32
  // rows of each epilogue warp; [2 halves][2][4 warps][16 tokens]
  float *sra = (float *)((uint8_t *)full + kBarBytes);
  int *srow = (int *)(sra + 256);
  float *turned = (float *)(srow + 256), *smax = turned + E * 16 * kTurnPitch;
  int *plan_at = (int *)((uint8_t *)full + kBarBytes + (ONE ? 0 : direct_bytes(E)));
  int *few = plan_at + 2 * (p.n_experts + 4);   // [kFewPositions]
  const Plan plan{plan_at, plan_at + p.n_experts + 4, p.M <= kFewPositions ? few : p.order};
  const tc::Waits waits{st, &g_gave_up, p.wait_ns};

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t stage_bytes = (uint32_t)(W * BM + p.tn) * BK;
  const int rank = ONE ? blockIdx.x : 0;
  const int first = ONE ? blockIdx.z * p.n_w + blockIdx.y : blockIdx.x, step = ONE ? INT32_MAX / 2 : gridDim.x;
  int k0, k1;
  k_range(p, rank, k0, k1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(&full[s], GATHER ? 1 + 32 * kLoaders : 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kScaleStages; ++s) {
      tc::mbar_init(&sfull[s], 32);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&tfull[b], 1);
      tc::mbar_init(&tempty[b], E);
    }
    tc::mbar_init(mdone, 1);
    tc::mbar_fence_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, p.tmem_cols);
  if constexpr (EXPERTS) {
    wait_for_grids();
    if (warp == 0) make_plan(p, plan, lane);
    else if (p.M <= kFewPositions)
      for (int i = threadIdx.x - 32; i < (int)p.M; i += blockDim.x - 32) few[i] = p.order[i];
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if constexpr (!EXPERTS) wait_for_grids();
  launch_dependents();
  // The status of the call.  A wait that gives up writes it two seconds or more after its own
  // CTA started, so this store, by the first CTA to start, comes first.
  if (threadIdx.x == 0 && blockIdx.x == 0 && (!ONE || (blockIdx.y == 0 && blockIdx.z == 0))) st->status = 0;
  const int n_tiles = p.n_w * (EXPERTS ? plan.tiles[p.n_experts] : p.n_m);
  const uint32_t set_cols = (uint32_t)(W * p.acc_cols);          // accumulators of a tile
  const uint32_t sc_cols = tmem + kSets * set_cols;

  // ONE: what finishes this warp's token: the cluster's tokens are dealt to its CTAs in turn, a CTA's to
  // its warps, those of the epilogue first, which ask for all of it before the sums are there.  A lane
  // has four rows.
  constexpr int kAll = Warps<GATED, EXPERTS, ONE>::kAll;
  const int first_col = rank + (warp + kAll - 2) % kAll * p.splits;
  const Tile one = ONE && first < n_tiles ? tile_of<EXPERTS, ONE>(p, plan, first) : Tile{0, 0, 0, 0};
  const int64_t n4 = (int64_t)one.n * BM + lane * 4;
  float fin_rw[W][4], fin_bias[W][4], fin_ra = 1.0f;
  int64_t fin_row = -1;
  TO fin_res[4];
  auto ask_token = [&](int col) {
    if (col >= one.cols) return;
    const int pos = one.m0 + col, r = a_row<GATHER>(p, plan, pos);
    fin_ra = p.ra && r < p.a_rows ? p.ra[r] : 1.0f;
    fin_row = pos;
    if constexpr (EXPERTS && !GATED) {
      const int o = plan.order[pos];
      fin_row = o >= 0 && o < p.M ? o : -1;
    }
    if constexpr (!GATED)
      if (p.residual) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          fin_res[j] = n4 + j < p.N ? ((const TO *)p.residual)[fin_row * p.ldr + n4 + j] : out_f32<TO>(0.0f);
      }
  };
  auto ask_rows = [&]() {
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t at = (int64_t)one.e * p.N + n4 + j;
        fin_rw[w][j] = p.rw[w] && n4 + j < p.N ? p.rw[w][at] : 1.0f;
        fin_bias[w][j] = p.bias[w] && n4 + j < p.N ? p.bias[w][at] : 0.0f;
      }
    ask_token(first_col);
  };

  bool ok = true;                   // false once a wait has given up: the role ends
  int s = 0, n = 0;                 // producer and issuer: stage of the ring; copies
  uint32_t ph = 1;
  if (warp == 0) {
    // ---------------- producer ----------------
    if (tc::elect_one()) {
      tc::tma_prefetch_desc(&mw0);
      if constexpr (GATED) tc::tma_prefetch_desc(&mw1);
      if constexpr (!GATHER) tc::tma_prefetch_desc(&ma);
#pragma unroll 1
      for (int t = first; t < n_tiles && ok; t += step) {
        const Tile tile = tile_of<EXPERTS, ONE>(p, plan, t);
        // rows that the MMA reads: of experts, whole groups of 16
        const int rows = EXPERTS ? (tile.cols + 15) / 16 * 16 : p.tn;
        const int copied = GATHER ? 0 : EXPERTS ? (rows + p.box - 1) / p.box * p.box : rows;
        const uint32_t bytes = (uint32_t)(W * BM + copied) * BK;
        for (int kb = k0; kb < k1; ++kb) {
          ok = tc::mbar_wait_compact(&empty[s], ph, waits);
          if (!ok) break;
          uint8_t *base = ring + s * stage_bytes;
          // (a lost copy is one whose last bytes never arrive)
          tc::mbar_arrive_expect_tx(&full[s], bytes + (n++ == p.lost ? 16u : 0u));
          tc::tma_load_3d(base, &mw0, kb * BK, tile.n * BM, tile.e, &full[s]);
          if constexpr (GATED) tc::tma_load_3d(base + BM * BK, &mw1, kb * BK, tile.n * BM, tile.e, &full[s]);
          if constexpr (!EXPERTS) {
            tc::tma_load_2d(base + W * BM * BK, &ma, kb * BK, tile.m0, &full[s]);
          } else if constexpr (!GATHER) {
            for (int j = 0; j < copied; j += p.box)
              tc::tma_load_2d(base + (W * BM + j) * BK, &ma, kb * BK, tile.m0 + j, &full[s]);
          }
          if (++s == p.stages) s = 0, ph ^= 1;
        }
      }
    }
  } else if (GATHER && warp >= 3 + E) {
    // ---------------- token rows by index ----------------
    // A copy of a warp takes four rows of 128 bytes; the MMA's swizzle exchanges a row's 16-byte
    // pieces by its number modulo 8.  Zeros past K, and for positions that name no row.
    constexpr int kQuads = (kMaxTnGated / 4 + kLoaders - 1) / kLoaders;   // copies of a lane
    const int piece = lane % 8, sub = lane / 8;
    // where the lane's piece goes, of its first copy: quads are 512 bytes, which the warps take in turn
    const int row0 = (warp - 3 - E) * 4 + sub;
    const uint32_t to = tc::smem_u32(ring) + W * BM * BK + row0 * BK + (piece ^ (row0 & 7)) * 16;
    static_assert(kLoaders % 2 == 0, "a lane's rows are the same modulo 8");
#pragma unroll 1
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile tile = tile_of<EXPERTS, ONE>(p, plan, t);
      const int rows = (tile.cols + 15) / 16 * 16;
      const uint8_t *src[kQuads];
      bool there[kQuads];           // (zeros for what is not)
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int j = row0 + 4 * kLoaders * i;
        const int r = j < tile.cols ? a_row<GATHER>(p, plan, tile.m0 + j) : (int)p.a_rows;
        there[i] = r < p.a_rows;
        src[i] = p.a + (there[i] ? r * p.lda : 0) + piece * 16;
      }
#pragma unroll 1
      for (int kb = k0; kb < k1; ++kb) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait_compact(&empty[s], ph, waits));
        if (!ok) break;
        const uint32_t dst = to + s * stage_bytes;
        const int64_t k = (int64_t)kb * BK;
        if (k + BK <= p.K) {
#pragma unroll
          for (int i = 0; i < kQuads; ++i)
            if (row0 + 4 * kLoaders * i < rows)
              asm volatile(
                  "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %2, 0;\n\t"
                  "cp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst + 4 * kLoaders * BK * i),
                  "l"(src[i] + k), "r"((uint32_t)there[i])
                  : "memory");
        } else {
          const int64_t left = p.K - k - piece * 16;
          const int here = left <= 0 ? 0 : left < 16 ? (int)left : 16;
#pragma unroll
          for (int i = 0; i < kQuads; ++i)
            if (row0 + 4 * kLoaders * i < rows)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 4 * kLoaders * BK * i),
                           "l"(here > 0 ? src[i] + k : p.a), "r"(there[i] ? here : 0)
                           : "memory");
        }
        // arrives when the lane's copies have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(tc::smem_u32(&full[s])) : "memory");
        if (++s == p.stages) s = 0, ph ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp == 1 && tc::elect_one()) {
    // ---------------- MMA issuer ----------------
    const uint32_t ring0 = (tc::smem_u32(ring) >> 4) | (1u << 16), stage16 = stage_bytes >> 4;
    const uint32_t sc0 = tc::smem_u32(sscale);
    int g = 0, it = 0;
    uint32_t at = ring0;            // lower word of the stage's first descriptor
    ph = 0;
#pragma unroll 1
    for (int t = first; t < n_tiles && ok; t += step, ++it) {
      const int b = it & 1, use = it >> 1;   // accumulators in turn
      const int rows = EXPERTS ? (tile_of<EXPERTS, ONE>(p, plan, t).cols + 15) / 16 * 16 : p.tn;
      const uint32_t idesc = mx::instr_desc(rows);
      ok = tc::mbar_wait_compact(&tempty[b], (use & 1) ^ 1, waits);
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t acc = tmem + b * set_cols;
#pragma unroll 1
      for (int kb = k0; kb < k1 && ok; kb += 4, ++g) {
        const int q = g % kScaleStages;
        ok = tc::mbar_wait_compact(&sfull[q], (g / kScaleStages) & 1, waits);
        if (!ok) break;
        tc::tc_fence_after();
        // two groups of columns in turn: the scale warp's ring keeps a third group's copy from
        // starting before the first group's MMAs have completed
        const uint32_t sc = sc_cols + (uint32_t)(g & 1) * kScaleCols, sm = sc0 + q * scale_bytes(p.tn);
        copy_scales(sc, sm);
        if constexpr (GATED) copy_scales(sc + 4, sm + 512);
        copy_scales(sc + 8, sm + 1024);
        if (rows > 128) copy_scales(sc + 12, sm + 1536);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kb + j >= k1) break;
          ok = tc::mbar_wait_compact(&full[s], ph, waits);
          if (!ok) break;
          if constexpr (GATHER) tc::fence_proxy_async_smem();   // the rows were not written by TMA
          tc::tc_fence_after();
          const uint32_t id = idesc | ((uint32_t)j << 29) | ((uint32_t)j << 4);
#pragma unroll
          for (int w = 0; w < W; ++w)
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              mx::mma(acc + w * p.acc_cols, at + (w * BM * BK >> 4) + 2 * kk, at + (W * BM * BK >> 4) + 2 * kk,
                      id, sc + 4 * w, sc + 8, j > 0 || kk > 0 || kb > k0);
          tc::mma_commit(&empty[s]);
          at += stage16;
          if (++s == p.stages) s = 0, ph ^= 1, at = ring0;
        }
        tc::mma_commit(&sempty[q]);
      }
      if (ok) tc::mma_commit(&tfull[b]);
    }
  } else if (warp == 2 + E) {
    // ---------------- scales ----------------
    int g = 0;
    for (int t = first; t < n_tiles && ok; t += step) {
      const Tile tile = tile_of<EXPERTS, ONE>(p, plan, t);
      int64_t row[8];               // offsets of the lane's rows (-1: none)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        row[i] = -1;
        if (lane + 32 * i < tile.cols) {
          const int r = a_row<GATHER>(p, plan, tile.m0 + lane + 32 * i);
          if (r < p.a_rows) row[i] = r * p.ldae;
        }
      }
      const uint8_t *we[W];
#pragma unroll
      for (int w = 0; w < W; ++w) we[w] = p.we[w] + tile.e * p.next_we[w] + tile.n * p.ldwe[w];
#pragma unroll 1
      for (int sb = k0 / 4; 4 * sb < k1; ++sb, ++g) {
        uint32_t word[8], ww[W];
        if (4 * sb + 4 <= p.kb) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            word[i] = row[i] >= 0 ? *reinterpret_cast<const uint32_t *>(p.ae + row[i] + 4 * sb) : 0x7F7F7F7Fu;
#pragma unroll
          for (int w = 0; w < W; ++w) ww[w] = *reinterpret_cast<const uint32_t *>(we[w] + 4 * sb);
        } else {
          // what lies behind a row's last exponent need not be there (a matrix of one row has any pitch)
#pragma unroll
          for (int i = 0; i < 8; ++i) word[i] = row[i] >= 0 ? last_exponents(p.ae + row[i] + 4 * sb, p.kb - 4 * sb) : 0x7F7F7F7Fu;
#pragma unroll
          for (int w = 0; w < W; ++w) ww[w] = last_exponents(we[w] + 4 * sb, p.kb - 4 * sb);
        }
        const int q = g % kScaleStages;
        // two TMEM groups: wait for the MMAs of two groups back, not only for this slot's
        if (g >= 2) ok = tc::mbar_wait_compact(&sempty[(g - 2) % kScaleStages], ((g - 2) / kScaleStages) & 1, waits);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(sscale + q * scale_bytes(p.tn)) + lane;
#pragma unroll
        for (int w = 0; w < W; ++w) dst[32 * w] = make_uint4(ww[w], ww[w], ww[w], ww[w]);
        dst[64] = make_uint4(word[0], word[1], word[2], word[3]);
        if (p.tn > 128) dst[96] = make_uint4(word[4], word[5], word[6], word[7]);
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&sfull[q]);
      }
    }
  } else if (warp >= 2 && warp < 2 + E) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, lrow = q * 32 + lane, et = threadIdx.x - 64, half = (warp - 2) / 4;
    static_assert(ONE || 32 * E >= kMaxTn, "a thread has one token's factors");
    int it = 0, turn = 0;
    // factors of the next tile, asked for while this one is worked on: of token `et`, and of this row
    Tile next;
    float next_ra = 1.0f, next_rw[W], next_bias[W];
    int next_row = -1;
    auto fetch = [&](int t) {
      next = tile_of<EXPERTS, ONE>(p, plan, t);
      if (!ONE && et < next.cols) {
        const int pos = next.m0 + et, r = a_row<GATHER>(p, plan, pos);
        next_ra = p.ra && r < p.a_rows ? p.ra[r] : 1.0f;
        if constexpr (EXPERTS && !GATED) {
          const int o = plan.order[pos];
          next_row = o >= 0 && o < p.M ? o : -1;
        }
      }
      const int64_t nn = (int64_t)next.n * BM + lrow, at = (int64_t)next.e * p.N + nn;
#pragma unroll
      for (int w = 0; w < W && !ONE; ++w) {
        next_rw[w] = p.rw[w] && nn < p.N ? p.rw[w][at] : 1.0f;
        next_bias[w] = p.bias[w] && nn < p.N ? p.bias[w][at] : 0.0f;
      }
    };
    if (first < n_tiles) fetch(first);
    if constexpr (ONE) ask_rows();
    for (int t = first; t < n_tiles; t += step, ++it) {
      const int b = it & 1, use = it >> 1;   // accumulators in turn
      const Tile tile = next;
      const int64_t nn = (int64_t)tile.n * BM + lrow;
      const bool in = nn < p.N;
      // the warp's 32 rows are all there, and rows of the output allow 8 bytes at a time
      const bool wide = p.wide && (int64_t)tile.n * BM + q * 32 + 32 <= p.N;
      float rw[W], bias[W];
#pragma unroll
      for (int w = 0; w < W && !ONE; ++w) rw[w] = next_rw[w], bias[w] = next_bias[w];
      if constexpr (!ONE) {
        tc::named_barrier(2, 32 * E);  // the previous tile's factors have been read
        if (et < tile.cols) {
          sra[et] = next_ra;
          if constexpr (EXPERTS && !GATED) srow[et] = next_row;
        }
      }
      if (t + step < n_tiles) fetch(t + step);
      // the lane's four outputs of the tokens lane / 8, + 4, ... of a chunk; their residuals are asked
      // for a chunk ahead, and are the first to leave L2, which keeps operands that come again (8192 x
      // 11008 x 4096: 271 us without that)
      const int64_t n4 = (int64_t)tile.n * BM + q * 32 + lane % 8 * 4;
      uint2 res[8];
      auto ask = [&](int c) {
        if constexpr (!GATED && !ONE) {
          if (!wide || !p.residual) return;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + lane / 8 + 4 * i < tile.cols)
              res[i] = __ldcs(reinterpret_cast<const uint2 *>(
                  (const TO *)p.residual + (int64_t)(tile.m0 + c + lane / 8 + 4 * i) * p.ldr + n4));
        }
      };
      ask(32 * half);
      ok = tc::mbar_wait_compact(&tfull[b], use & 1, waits);
      if (!tc::named_barrier_and(1, 32 * E, ok)) break;
      tc::tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + b * set_cols;
      float *mine = turned + (warp - 2) * 16 * kTurnPitch;     // this warp's to turn
      if constexpr (ONE) {
        float *part = (float *)ring + lrow;
#pragma unroll 1
        for (int c = 16 * half; c < tile.cols; c += 4 * E) {
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t r[16];
            tc::tmem_ld16(acc + w * p.acc_cols + (uint32_t)c, r);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(w * p.tn + c + i) * BM] = __uint_as_float(r[i]);   // (tn: whole 16s)
          }
        }
      } else if constexpr (GATED) {
#pragma unroll 1
        for (int c = 16 * half; c < tile.cols; c += 32) {
          uint32_t r[W][16];
#pragma unroll
          for (int w = 0; w < W; ++w) tc::tmem_ld16(acc + w * p.acc_cols + (uint32_t)c, r[w]);
          tc::tmem_ld_wait();
          float v[16], u[16];
          const float4 *ra4 = reinterpret_cast<const float4 *>(sra + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = ra4[i];
            const float fs[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v[4 * i + j] = fmaf(__uint_as_float(r[0][4 * i + j]) * rw[0], fs[j], bias[0]);
              u[4 * i + j] = fmaf(__uint_as_float(r[W - 1][4 * i + j]) * rw[W - 1], fs[j], bias[W - 1]);
            }
          }
          activate(v, p.act);
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[i * kTurnPitch + lane] = in ? v[i] * u[i] : 0.0f;
          __syncwarp();
          // this lane's token, and 16 of the warp's 32 rows
          const int token = lane % 16, rows16 = lane / 16 * 16;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(&v[4 * i]) = *reinterpret_cast<const float4 *>(mine + token * kTurnPitch + rows16 + 4 * i);
          auto largest = [&]() {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));
            return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
          };
          float most = largest();
          if (__any_sync(0xffffffffu, most == INFINITY)) {
            // infinities become NaN, which a maximum passes over
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = fp8::inf_to_nan(v[i]);
            most = largest();
          }
          float *sm = smax + (half * 2 + (turn++ & 1)) * 64;
          if (lane < 16) sm[q * 16 + lane] = most;
          tc::named_barrier(3 + half, 128);
          most = fmaxf(fmaxf(sm[token], sm[16 + token]), fmaxf(sm[32 + token], sm[48 + token]));
          const int ex = fp8::block_exponent(most);
          const float inv = fp8::pow2(-ex);
          if (c + token < tile.cols) {
            const int64_t row = tile.m0 + c + token;
            const int64_t n16 = (int64_t)tile.n * BM + q * 32 + rows16;
            if (q == 0 && lane < 16) p.oe[row * p.ldoe + tile.n] = (uint8_t)(ex + fp8::kBias);
            uint4 codes;
            codes.x = fp8::pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            codes.y = fp8::pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
            codes.z = fp8::pack4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv);
            codes.w = fp8::pack4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv);
            uint8_t *o = (uint8_t *)p.out + row * p.ldo + n16;   // (rows of codes are 16-byte aligned)
            if (n16 + 16 <= p.N) {
              *reinterpret_cast<uint4 *>(o) = codes;
            } else {
              const uint32_t word[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (n16 + i < p.N) o[i] = (uint8_t)(word[i / 4] >> (8 * (i % 4)));
            }
          }
          __syncwarp();
        }
      } else {
#pragma unroll 1
        for (int c = 32 * half; c < tile.cols; c += 64) {
          uint32_t r[W][32];
          tc::tmem_ld32(acc + (uint32_t)c, r[0]);
          float v[32];
          const int left = tile.cols - c;                    // tokens of this chunk, if below 32
          const float4 *ra4 = reinterpret_cast<const float4 *>(sra + c);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 f = ra4[i];
            v[4 * i] = fmaf(__uint_as_float(r[0][4 * i]) * rw[0], f.x, bias[0]);
            v[4 * i + 1] = fmaf(__uint_as_float(r[0][4 * i + 1]) * rw[0], f.y, bias[0]);
            v[4 * i + 2] = fmaf(__uint_as_float(r[0][4 * i + 2]) * rw[0], f.z, bias[0]);
            v[4 * i + 3] = fmaf(__uint_as_float(r[0][4 * i + 3]) * rw[0], f.w, bias[0]);
          }
          activate(v, p.act);
          if (wide) {
            uint2 add[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) add[i] = res[i];
            ask(c + 64);
#pragma unroll
            for (int h = 0; h < 2; ++h) {                    // 16 tokens at a time
#pragma unroll
              for (int i = 0; i < 16; ++i) mine[i * kTurnPitch + lane] = v[16 * h + i];
              __syncwarp();
#pragma unroll
              for (int i = 4 * h; i < 4 * h + 4; ++i) {
                const int j = lane / 8 + 4 * i;
                const int64_t row = EXPERTS ? srow[c + j] : tile.m0 + c + j;
                if (j >= left || (EXPERTS && row < 0)) continue;
                float4 x = *reinterpret_cast<const float4 *>(mine + (j - 16 * h) * kTurnPitch + lane % 8 * 4);
                if (p.residual) {
                  const TO *r4 = reinterpret_cast<const TO *>(&add[i]);
                  x.x += to_f32(r4[0]);
                  x.y += to_f32(r4[1]);
                  x.z += to_f32(r4[2]);
                  x.w += to_f32(r4[3]);
                }
                alignas(8) const TO o[4] = {out_f32<TO>(x.x), out_f32<TO>(x.y), out_f32<TO>(x.z), out_f32<TO>(x.w)};
                *reinterpret_cast<uint2 *>((TO *)p.out + row * p.ldo + n4) = *reinterpret_cast<const uint2 *>(o);
              }
              __syncwarp();
            }
          } else if (in) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int64_t row = EXPERTS ? srow[c + i] : tile.m0 + c + i;
              if (i >= left || (EXPERTS && row < 0)) continue;
              const float x = p.residual ? v[i] + to_f32(((const TO *)p.residual)[row * p.ldr + nn]) : v[i];
              ((TO *)p.out)[row * p.ldo + nn] = out_f32<TO>(x);
            }
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&tempty[b]);
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  if (!__syncthreads_and(ok)) {
    // A wait has given up: what is in flight gets one more, bounded, to land or to complete before
    // the CTA leaves and the TMEM is released.
    if (warp == 0 && tc::elect_one()) {
      // stages before s are of this round of the ring, the others of the one before
#pragma unroll 1
      for (int i = 0; i < (n < p.stages ? s : p.stages); ++i)
        tc::mbar_wait_compact(&full[i], i < s ? ph ^ 1 : ph, waits);
    } else if (warp == 1 && tc::elect_one()) {
      tc::mma_commit(mdone);
      tc::mbar_wait_compact(mdone, 0, waits);
    }
    __syncwarp();
  }
  if (warp == 1) tc::tmem_dealloc(tmem, p.tmem_cols);
  if constexpr (ONE) {
    // the ring holds this CTA's partial sums [W][tn][128]
    if (warp < 2 || warp >= 2 + E) ask_rows();
    tc::cluster_sync();
    {
      const int64_t nn = n4;
      const bool pairs = (p.ldo & 1) == 0 && ((uintptr_t)p.out & 3) == 0 && nn + 3 < p.N;
#pragma unroll 1
      for (int col = first_col; col < one.cols; col += kAll * p.splits) {
        if (col != first_col) ask_token(col);
        const int64_t row = fin_row;
        float x[W][4];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t off = tc::smem_u32(ring) + (uint32_t)(w * p.tn + col) * BM * 4 + lane * 16;
          float4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = i < p.splits ? mx::ld_cluster_f32x4(tc::mapa_shared(off, (uint32_t)i)) : make_float4(0.f, 0.f, 0.f, 0.f);
          float4 sum = v[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) {
            sum.x += v[i].x;
            sum.y += v[i].y;
            sum.z += v[i].z;
            sum.w += v[i].w;
          }
          x[w][0] = fmaf(sum.x * fin_rw[w][0], fin_ra, fin_bias[w][0]);
          x[w][1] = fmaf(sum.y * fin_rw[w][1], fin_ra, fin_bias[w][1]);
          x[w][2] = fmaf(sum.z * fin_rw[w][2], fin_ra, fin_bias[w][2]);
          x[w][3] = fmaf(sum.w * fin_rw[w][3], fin_ra, fin_bias[w][3]);
        }
        activate(x[0], p.act);
        if constexpr (GATED) {
          float most = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[0][j] *= x[1][j];
            if (nn + j < p.N) most = fmaxf(most, fp8::finite_abs(x[0][j]));
          }
          most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
          const int ex = fp8::block_exponent(most);
          const float sc = fp8::pow2(-ex);
          const uint32_t four = fp8::pack4(fp8::inf_to_nan(x[0][0]) * sc, fp8::inf_to_nan(x[0][1]) * sc,
                                           fp8::inf_to_nan(x[0][2]) * sc, fp8::inf_to_nan(x[0][3]) * sc);
          uint8_t *dst = (uint8_t *)p.out + row * p.ldo + nn;   // (rows are 16-byte aligned)
          if (nn + 3 < p.N) {
            *reinterpret_cast<uint32_t *>(dst) = four;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (nn + j < p.N) dst[j] = (uint8_t)(four >> (8 * j));
          }
          if (lane == 0) p.oe[row * p.ldoe + one.n] = (uint8_t)(ex + fp8::kBias);
        } else if (row >= 0) {
          alignas(8) TO o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = out_f32<TO>(p.residual ? x[0][j] + to_f32(fin_res[j]) : x[0][j]);
          TO *dst = (TO *)p.out + row * p.ldo + nn;
          if (pairs) {
            reinterpret_cast<uint32_t *>(dst)[0] = reinterpret_cast<const uint32_t *>(o)[0];
            reinterpret_cast<uint32_t *>(dst)[1] = reinterpret_cast<const uint32_t *>(o)[1];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (nn + j < p.N) dst[j] = o[j];
          }
        }
      }
    }
    tc::cluster_sync();   // the others have read this CTA's sums
  }
}

// How a call's work is cut: tokens of a tile, CTAs that share its k-blocks, one tile a cluster or not,
// and what a CTA has of its SM.
struct Shape {
  int tn, splits, per_sm;
  bool one;
  int stages, tmem_cols;
  uint32_t ring_bytes;
  size_t smem;
};

// The ring of copies that fits; false where there is no room for three stages (or all k-blocks).
//
// A CTA that finds too little tensor memory free waits for it, and one of a cluster is waited for by
// others that hold some: two kernels' clusters on one SM could wait for one another in a ring.  So a CTA
// takes at least as large a share of an SM's shared memory as of its tensor memory, and more than the
// library's kernels with all of the tensor memory leave (193 KB and up); those that fit an SM together then
// all have theirs.
template <bool GATED, bool EXPERTS>
bool lay_out(Shape &h, int64_t groups, int n_experts) {
  constexpr int W = GATED ? 2 : 1;
  const size_t besides = 1024 + kScaleStages * scale_bytes(h.tn) + kBarBytes +
                         (EXPERTS ? round_up((2 * (n_experts + 4) + kFewPositions) * sizeof(int), 16) : 0) +
                         (h.one ? 0 : direct_bytes(Warps<GATED, EXPERTS, false>::kEpilogue));
  const size_t all = h.per_sm > 1 ? kSmemTwo : kSmem, room = all > besides ? all - besides : 0, stage = (size_t)(W * BM + h.tn) * BK;
  const int64_t blocks = 4 * ceil_div(groups, (int64_t)h.splits);   // of a CTA, at most
  int64_t stages = (int64_t)(room / stage);
  if (stages > kMaxStages) stages = kMaxStages;
  if (h.one && stages > blocks) stages = blocks;
  h.stages = (int)stages;
  h.ring_bytes = (uint32_t)(stages * stage);
  const size_t sums = h.one ? (size_t)W * h.tn * BM * 4 : 0;
  if (h.ring_bytes < sums) h.ring_bytes = (uint32_t)sums;
  h.smem = besides + h.ring_bytes;
  for (h.tmem_cols = 32; h.tmem_cols < (h.one ? 1 : 2) * W * h.tn + 2 * (int)kScaleCols;) h.tmem_cols *= 2;
  const size_t share = h.tmem_cols * (kSmemTwo / 256), least = share < kSmemLeast ? kSmemLeast : share;
  if (h.one && h.smem < least) h.smem = least;
  return h.smem <= all && (stages >= 3 || (h.one && stages == blocks));
}

// Clusters of `splits` CTAs, per_sm on an SM, that run at once.  They lie within groups of SMs, so
// there is room for fewer than SMs / splits.
template <typename TO, bool GATED, bool EXPERTS>
int clusters_at_once(int dev, int splits, int per_sm, int sms) {
  static PerDevice<18> known;
  return known.get(dev, splits + 9 * (per_sm - 1), [=]() {
    const auto kernel = linear_kernel<TO, GATED, EXPERTS, true>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(splits * sms));
    cfg.blockDim = dim3(32 * Warps<GATED, EXPERTS, true>::kAll);
    cfg.dynamicSmemBytes = per_sm > 1 ? kSmemTwo : kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (const void *)kernel, &cfg) == cudaSuccess) return n;
    (void)cudaGetLastError();
    return 0;
  }, per_sm * sms / splits * 7 / 8);
}

// The cut with the least of an estimate in SM cycles: a k-block of a tile takes the MMAs' time, that of
// their issue, or that of its operands' way from L2 (61 bytes a cycle and SM, as measured); the memory brings
// each operand once at 3500 bytes a cycle; a launch costs 6400, sums that meet 1400 + 8 a token.  Of experts the number
// of tiles is not known here: as many as if the rows were dealt evenly, or what there can be at most where
// each cluster has one.
template <typename TO, bool GATED, bool EXPERTS>
Shape choose(const Fp8LinearArgs &g, int dev, int sms) {
  constexpr int W = GATED ? 2 : 1;
  const int64_t n_w = ceil_div(g.N, (int64_t)BM), groups = ceil_div(ceil_div(g.K, (int64_t)BK), (int64_t)4);
  const int most = GATED ? kMaxTnGated : kMaxTn;
  // matrices in use, and rows of each
  const double used = EXPERTS ? g.n_experts * (1.0 - pow(1.0 - 1.0 / g.n_experts, (double)g.M)) : 1.0;
  const double rows = g.M / used;
  const double once = ((double)g.M + W * used * g.N) * g.K / 3500.0;
  Shape best{};
  double best_t = 1e30;
  for (int tn = 16; tn <= most; tn += EXPERTS && !GATED && tn >= kBox ? kBox : 16) {
    if (!EXPERTS && tn - 16 >= g.M) break;
    const double per = EXPERTS ? rows / tn + 0.5 : (double)ceil_div(g.M, (int64_t)tn);   // tiles along the tokens
    const double tiles = n_w * used * (per < 1.0 ? 1.0 : per);
    const int64_t at_most = n_w * (EXPERTS ? (g.n_experts < g.M ? g.n_experts : g.M) + g.M / tn : ceil_div(g.M, (int64_t)tn));
    const double mma = W * 3.45 * tn, issue = 300 + W * 1.7 * tn, feed = (W * BM + tn) * BK / 61.0;
    const double c = fmax(fmax(mma, issue), feed);
    for (int s = 1; s <= 8 && s <= groups; ++s) {   // 1: from tile to tile
      if (s > 1 && at_most * s > 2 * sms) break;
      Shape h{tn, s, 1, s > 1};
      if (h.one) {
        // alone on its SM, for copies in flight; or two, where there are that many
        auto fits = [&]() {
          return lay_out<GATED, EXPERTS>(h, groups, g.n_experts) &&
                 at_most <= clusters_at_once<TO, GATED, EXPERTS>(dev, s, h.per_sm, sms);
        };
        if (!fits()) {
          h.per_sm = 2;
          if (!fits()) continue;
        }
      } else if (!lay_out<GATED, EXPERTS>(h, groups, g.n_experts)) {
        continue;
      }
      const double busy = ceil(tiles * h.splits / sms);
      const double work = busy * 4 * ceil_div(groups, (int64_t)h.splits) * c;
      double t = sqrt(work * work + once * once);
      t += 6400.0 + (h.one ? 1400.0 + 8.0 * W * tn : 0.0) + (h.one ? 0.0 : 800.0 * (busy - 1));
      if (t < best_t) best_t = t, best = h;
    }
  }
  return best;
}

template <typename TO, bool GATED, bool EXPERTS, bool ONE>
gptq_status launch(const Shape &h, dim3 grid, cudaStream_t s, const CUtensorMap &mw0, const CUtensorMap &mw1,
                   const CUtensorMap &ma, const Params &p, DevStatus *st) {
  GPTQ_TRY(ensure_smem_attr((const void *)linear_kernel<TO, GATED, EXPERTS, ONE>, (int)kSmem));
  return launch_early(linear_kernel<TO, GATED, EXPERTS, ONE>, grid, dim3(32 * Warps<GATED, EXPERTS, ONE>::kAll),
                      h.smem, h.splits, s, mw0, mw1, ma, p, st);
}

template <typename TO, bool GATED, bool EXPERTS>
gptq_status run(const Fp8LinearArgs &g, DevStatus *st, cudaStream_t s) {
  constexpr int W = GATED ? 2 : 1;
  int sms = 0, dev = -1;
  GPTQ_TRY(device_sm_count(&sms));
  GPTQ_CUDA_CHECK(cudaGetDevice(&dev));
  // (set before the clusters that fit are asked for)
  GPTQ_TRY(ensure_smem_attr((const void *)linear_kernel<TO, GATED, EXPERTS, true>, (int)kSmem));
  const Shape h = choose<TO, GATED, EXPERTS>(g, dev, sms);
  Params p{};
  p.a = g.a; p.lda = g.lda; p.K = g.K;
  p.ae = g.ae; p.ldae = g.ldae;
  p.ra = g.ra;
  p.wide = fp8::alignment(g.out, 2 * g.ldo) >= 8 && (!g.residual || fp8::alignment(g.residual, 2 * g.ldr) >= 8);
  for (int w = 0; w < W; ++w) {
    p.we[w] = g.w[w].exps; p.ldwe[w] = g.w[w].ld_exps; p.next_we[w] = g.w[w].next_exps;
    p.rw[w] = g.w[w].scale;
    p.bias[w] = g.w[w].bias;
  }
  p.residual = g.residual; p.ldr = g.ldr;
  p.out = g.out; p.ldo = g.ldo;
  p.oe = g.oe; p.ldoe = g.ldoe;
  p.a_rows = g.a_rows; p.M = g.M; p.N = g.N;
  p.act = g.act;
  p.kb = (int)ceil_div(g.K, (int64_t)BK);
  p.tn = h.tn; p.stages = h.stages; p.splits = h.splits; p.ring_bytes = h.ring_bytes;
  p.box = h.tn < kBox ? h.tn : kBox;   // (tn is a multiple of it)
  p.n_w = (int)ceil_div(g.N, (int64_t)BM);
  p.n_m = (int)ceil_div(g.M, (int64_t)h.tn);
  p.across = (int)ceil_div(p.n_w, ceil_div(p.n_w, kAcross));
  const int64_t along = EXPERTS ? (g.n_experts < g.M ? g.n_experts : g.M) + g.M / h.tn : p.n_m;
  const int64_t tiles = p.n_w * along;   // at most
  if (tiles * 8 > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  p.acc_cols = h.tn;
  p.tmem_cols = h.tmem_cols;
  p.offsets = g.offsets; p.order = g.order;
  p.n_experts = g.n_experts; p.top_k = g.top_k;
  p.per_tn = (uint32_t)((0xFFFFFFFFull + h.tn) / h.tn);
  if (g.top_k > 1) p.per_k = (uint32_t)((0xFFFFFFFFull + g.top_k) / g.top_k);
  p.wait_ns = g.wait_ns;
  p.lost = (int)g.lost;
  const int64_t mats = EXPERTS ? g.n_experts : 1;
  CUtensorMap mw[2], ma;
  for (int w = 0; w < W; ++w)
    if (!tc::make_tmap_matrices(&mw[w], g.w[w].codes, mats, g.N, g.K, g.w[w].ld,
                                mats > 1 ? g.w[w].next_codes : g.N * g.w[w].ld, BM))
      return GPTQ_ERR_UNSUPPORTED;
  if (W == 1) mw[1] = mw[0];
  if (!tc::make_tmap_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a, g.a_rows, g.K, g.lda, BK,
                        EXPERTS ? p.box : h.tn))
    return GPTQ_ERR_UNSUPPORTED;
  return h.one ? launch<TO, GATED, EXPERTS, true>(h, dim3((unsigned)h.splits, (unsigned)p.n_w, (unsigned)along), s,
                                                  mw[0], mw[1], ma, p, st)
               : launch<TO, GATED, EXPERTS, false>(h, dim3((unsigned)(tiles < sms ? tiles : sms)), s, mw[0], mw[1],
                                                   ma, p, st);
}

}  // namespace

size_t fp8_linear_ws_bytes(int64_t, int64_t, int64_t) { return 256; }

gptq_status fp8_linear_take_timeout(int *out, cudaStream_t s) { return take_flag(g_gave_up, out, s); }

gptq_status launch_fp8_linear(const Fp8LinearArgs &g, void *ws, cudaStream_t s) {
  if (g.M == 0) {
    GPTQ_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
    return GPTQ_OK;
  }
  DevStatus *st = (DevStatus *)ws;
  using Half = __half;
  using Bf16 = __nv_bfloat16;
  if (g.n_experts > 0) {
    if (g.gated) return run<Bf16, true, true>(g, st, s);
    return g.odtype == GPTQ_F16 ? run<Half, false, true>(g, st, s) : run<Bf16, false, true>(g, st, s);
  }
  if (g.gated) return run<Bf16, true, false>(g, st, s);
  return g.odtype == GPTQ_F16 ? run<Half, false, false>(g, st, s) : run<Bf16, false, false>(g, st, s);
}

}  // namespace gptq
