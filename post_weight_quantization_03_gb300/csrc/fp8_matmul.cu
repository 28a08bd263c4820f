// The block-scaled e4m3 product
//   out[m, n] = ra_m rw_n sum_kb 2^(EA[m, kb] - 127) 2^(EW[n / 128, kb] - 127) sum_{k in kb} a w.
//
// tcgen05 kind::mxf8f6f4 takes a power-of-two scale byte per row and 32 elements of K, so both
// block scales are applied inside the tensor core and a tile is one uninterrupted fp32 sum in
// TMEM; the two row factors multiply it in the epilogue.
//
// The weights' 128 rows are the MMA's M and a tile of `tn` tokens is its N (any multiple of 16
// up to 240: two accumulators of 240 columns and the scales' columns fill the 512 of TMEM).  So
// a single token costs one 16-column MMA per 128 x 32 weights, which streams W at the memory's
// rate, and the lanes of an accumulator are consecutive outputs of one token (coalesced stores).
//
//   warp 0     : TMA producer (one lane): (W box, A box) of 128 bytes x rows per k-block
//   warp 1     : TMEM allocator + MMA issuer (one lane): copies the scales of four k-blocks to
//                TMEM, then four K = 32 MMAs per k-block, the byte chosen by the descriptor
//   warps 2..5 : epilogue, one weight row per thread
//   warp 6     : scales: gathers four k-blocks' bytes of each row (one 32-bit word) into the
//                32 x 16-byte arrangement that the copy to TMEM takes
//
// Few tokens leave few tiles; the k-blocks of a tile are then split over a cluster of up to 8
// CTAs, whose partial sums meet through distributed shared memory in rank order.
//
// Bounds, and what it measured (GPU time, m x n x k): up to a few hundred tokens W's bytes
// (1 x 4096 x 4096 5.7 us, of which 2.5 are the bytes; 24 x 11008 x 4096 11.3 us, 4.0 TB/s;
// 128 x 8192 x 28672 44 us, 5.4 TB/s), the rest of it being the launch, the first copies and the
// exchange of split sums.  Beyond, the tensor core: 515 x 4096 x 11008 25.5 us, 1.8 PFLOP/s;
// 8192 x 11008 x 4096 244 us, 3.0 PFLOP/s, the pipe busy 72 % of the time (281 us, 2.6 PFLOP/s, in a
// row of calls that the power limit holds back).
#include <cudaTypedefs.h>
#include <math.h>

#include "mx.cuh"
#include "per_device.cuh"

namespace gptq {

namespace {

using mx::BK;
using mx::BM;
using mx::copy_scales;
using mx::ld_cluster_f32x4;
using mx::out_f32;
constexpr int kMaxTn = 240;
constexpr int kThreads = 224;
constexpr int kScaleStages = 4;             // groups of four k-blocks in flight
constexpr uint32_t kScaleBytes = 3 * 512;   // W, tokens 0..127, tokens 128..239
constexpr uint32_t kScaleCols = 12;         // TMEM columns of one group
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 12;
constexpr uint32_t kRingBytes = 208 * 1024;      // one CTA on an SM
constexpr uint32_t kRingBytesTwo = 96 * 1024;    // two
constexpr size_t kSmemBesides = 1024 + kScaleStages * kScaleBytes + kMaxTn * 4 + 512;
static_assert(2 * kMaxTn + 2 * kScaleCols <= kTmemCols, "TMEM columns");
static_assert(2 * (kRingBytesTwo + kSmemBesides + 1024) <= 228 * 1024, "two CTAs on an SM");

struct MmParams {
  const uint8_t *ae; int64_t ldae;
  const uint8_t *we; int64_t ldwe;
  const float *ra, *rw;
  void *out; int64_t ldo;
  int64_t M, N;
  int kb;               // k-blocks
  int tn, stages;
  int n_w, n_tiles;     // tiles along the weights; tiles in all
  int splits;           // CTAs of a cluster that share a tile's k-blocks
  uint32_t ring_bytes;
  int acc_cols, tmem_cols;  // columns of an accumulator; allocated
  uint64_t wait_ns;
  int lost;             // test hook: this copy of the producer's is left out
};

__device__ int g_gave_up;  // a wait ran out since it was last asked for

// k-blocks of this CTA: rank r of the cluster takes an even share of the groups of four.
__device__ __forceinline__ void k_range(const MmParams &p, int rank, int &k0, int &k1) {
  const int groups = (p.kb + 3) / 4;
  k0 = groups * rank / p.splits * 4;
  k1 = min(groups * (rank + 1) / p.splits * 4, p.kb);
}

template <typename TO>
__global__ void __launch_bounds__(kThreads, 2)
matmul_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap ma,
              MmParams p, DevStatus *st) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t *sscale = ring + p.ring_bytes;
  float *sra = (float *)(sscale + kScaleStages * kScaleBytes);
  uint64_t *full = (uint64_t *)(sra + kMaxTn);
  uint64_t *empty = full + kMaxStages;
  uint64_t *sfull = empty + kMaxStages;
  uint64_t *sempty = sfull + kScaleStages;
  uint64_t *tfull = sempty + kScaleStages;
  uint64_t *tempty = tfull + 2;
  uint64_t *mdone = tempty + 2;       // every MMA has completed
  uint32_t *tmem_slot = (uint32_t *)(mdone + 1);
  const tc::Waits waits{st, &g_gave_up, p.wait_ns};

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  const uint32_t stage_bytes = (uint32_t)(BM + p.tn) * BK;
  const int rank = p.splits > 1 ? (int)tc::cluster_ctarank() : 0;
  const int first = blockIdx.x / p.splits, step = gridDim.x / p.splits;
  int k0, k1;
  k_range(p, rank, k0, k1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kScaleStages; ++s) {
      tc::mbar_init(&sfull[s], 32);
      tc::mbar_init(&sempty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&tfull[b], 1);
      tc::mbar_init(&tempty[b], 4);
    }
    tc::mbar_init(mdone, 1);
    tc::mbar_fence_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, p.tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_grids();
  launch_dependents();
  // The status of the call.  A wait that gives up writes it two seconds or more after its own
  // CTA started, so this store, by the first CTA to start, comes first.
  if (blockIdx.x == 0 && threadIdx.x == 0) st->status = 0;
  // with few tiles every CTA has one and a second accumulator is not allocated
  const uint32_t second = (uint32_t)p.acc_cols, sc_cols = tmem + (p.tmem_cols == (int)kTmemCols ? 2 : 1) * second;

  bool ok = true;                   // false once a wait has given up: the role ends
  int s = 0, n = 0;                 // producer and issuer: stage of the ring; copies
  uint32_t ph = 1;
  // (inside elect_one() one thread is known to run, and addresses stay in uniform registers)
  if (warp == 0 && tc::elect_one()) {
    // ---------------- producer ----------------
    tc::tma_prefetch_desc(&mw);
    tc::tma_prefetch_desc(&ma);
    for (int t = first; t < p.n_tiles && ok; t += step) {
      const int32_t n0 = (t % p.n_w) * BM, m0 = (t / p.n_w) * p.tn;
      for (int kb = k0; kb < k1; ++kb) {
        ok = tc::mbar_wait_compact(&empty[s], ph, waits);
        if (!ok) break;
        uint8_t *base = ring + s * stage_bytes;
        // (a lost copy is one whose last bytes never arrive)
        tc::mbar_arrive_expect_tx(&full[s], stage_bytes + (n++ == p.lost ? 16u : 0u));
        tc::tma_load_2d(base, &mw, kb * BK, n0, &full[s]);
        tc::tma_load_2d(base + BM * BK, &ma, kb * BK, m0, &full[s]);
        if (++s == p.stages) s = 0, ph ^= 1;
      }
    }
  } else if (warp == 1 && tc::elect_one()) {
    // ---------------- MMA issuer ----------------
    const uint32_t idesc = mx::instr_desc(p.tn);
    const uint32_t ring0 = (tc::smem_u32(ring) >> 4) | (1u << 16), stage16 = stage_bytes >> 4;
    const uint32_t sc0 = tc::smem_u32(sscale);
    int g = 0, it = 0;
    uint32_t at = ring0;            // lower word of the stage's first descriptor
    ph = 0;
#pragma unroll 1
    for (int t = first; t < p.n_tiles && ok; t += step, ++it) {
      const int b = it & 1;
      ok = tc::mbar_wait_compact(&tempty[b], ((it >> 1) & 1) ^ 1, waits);
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t acc = tmem + b * second;
#pragma unroll 1
      for (int kb = k0; kb < k1 && ok; kb += 4, ++g) {
        const int q = g % kScaleStages;
        ok = tc::mbar_wait_compact(&sfull[q], (g / kScaleStages) & 1, waits);
        if (!ok) break;
        tc::tc_fence_after();
        // two groups of columns in turn: the scale warp's ring keeps a third group's copy from
        // starting before the first group's MMAs have completed
        const uint32_t sc = sc_cols + (uint32_t)(g & 1) * kScaleCols, sm = sc0 + q * kScaleBytes;
        copy_scales(sc, sm);
        copy_scales(sc + 4, sm + 512);
        if (p.tn > 128) copy_scales(sc + 8, sm + 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kb + j >= k1) break;
          ok = tc::mbar_wait_compact(&full[s], ph, waits);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t id = idesc | ((uint32_t)j << 29) | ((uint32_t)j << 4);
#pragma unroll
          for (int kk = 0; kk < BK / 32; ++kk)
            mx::mma(acc, at + 2 * kk, at + (BM * BK >> 4) + 2 * kk, id, sc, sc + 4,
                    j > 0 || kk > 0 || kb > k0);
          tc::mma_commit(&empty[s]);
          at += stage16;
          if (++s == p.stages) s = 0, ph ^= 1, at = ring0;
        }
        tc::mma_commit(&sempty[q]);
      }
      if (ok) tc::mma_commit(&tfull[b]);
    }
  } else if (warp == 6) {
    // ---------------- scales ----------------
    int g = 0;
    for (int t = first; t < p.n_tiles && ok; t += step) {
      const int64_t m0 = (int64_t)(t / p.n_w) * p.tn;
      const uint8_t *we = p.we + (int64_t)(t % p.n_w) * p.ldwe;
#pragma unroll 1
      for (int sb = k0 / 4; 4 * sb < k1; ++sb, ++g) {
        uint32_t word[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t row = m0 + lane + 32 * i;
          word[i] = (lane + 32 * i < p.tn && row < p.M)
                        ? *reinterpret_cast<const uint32_t *>(p.ae + row * p.ldae + 4 * sb)
                        : 0x7F7F7F7Fu;
        }
        const uint32_t ww = *reinterpret_cast<const uint32_t *>(we + 4 * sb);
        const int q = g % kScaleStages;
        // two TMEM groups: wait for the MMAs of two groups back, not only for this slot's
        if (g >= 2) ok = tc::mbar_wait_compact(&sempty[(g - 2) % kScaleStages], ((g - 2) / kScaleStages) & 1, waits);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        uint4 *dst = reinterpret_cast<uint4 *>(sscale + q * kScaleBytes) + lane;
        dst[0] = make_uint4(ww, ww, ww, ww);
        dst[32] = make_uint4(word[0], word[1], word[2], word[3]);
        dst[64] = make_uint4(word[4], word[5], word[6], word[7]);
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&sfull[q]);
      }
    }
  } else if (warp >= 2 && warp < 6) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, row = q * 32 + lane, et = threadIdx.x - 64;
    int it = 0;
    for (int t = first; t < p.n_tiles; t += step, ++it) {
      const int b = it & 1;
      const int64_t n = (int64_t)(t % p.n_w) * BM + row, m0 = (int64_t)(t / p.n_w) * p.tn;
      const int cols = (int)(p.M - m0 < p.tn ? p.M - m0 : p.tn);
      if (p.splits == 1) {
        tc::named_barrier(2, 128);  // the previous tile's factors have been read
        for (int j = et; j < cols; j += 128) sra[j] = p.ra ? p.ra[m0 + j] : 1.0f;
      }
      const float rw = (p.rw && n < p.N) ? p.rw[n] : 1.0f;
      ok = tc::mbar_wait_compact(&tfull[b], (it >> 1) & 1, waits);
      if (!tc::named_barrier_and(1, 128, ok)) break;
      tc::tc_fence_after();
      TO *o = (TO *)p.out + m0 * p.ldo + n;
      float *part = (float *)ring + row;
#pragma unroll 1
      for (int c = 0; c < p.tn; c += 32) {
        uint32_t r[32];
        tc::tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + b * second + (uint32_t)c, r);
        tc::tmem_ld_wait();
        if (p.splits > 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < p.tn) part[(c + i) * BM] = __uint_as_float(r[i]);
        } else if (n < p.N) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (c + i < cols) o[(int64_t)(c + i) * p.ldo] = out_f32<TO>(__uint_as_float(r[i]) * rw * sra[c + i]);
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
    // the CTA leaves and the TMEM is released.  (In the regular course all of it has been waited
    // for; waiting here again costs a single token's product 0.3 us of 5.4.)
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
  if (p.splits > 1) {
    // one tile per cluster: the ring holds this CTA's partial sums [tn][128]
    tc::cluster_sync();
    const int64_t n0 = (int64_t)(first % p.n_w) * BM, m0 = (int64_t)(first / p.n_w) * p.tn;
    const int cols = (int)(p.M - m0 < p.tn ? p.M - m0 : p.tn);
    // this CTA's columns are rank, rank + splits, ...; a thread takes four rows of one
    const uint32_t base = tc::smem_u32(ring) + (threadIdx.x % 32) * 16;
    const int64_t n = n0 + threadIdx.x % 32 * 4;
    float rw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) rw[j] = p.rw && n + j < p.N ? p.rw[n + j] : 1.0f;
    const bool pairs = (p.ldo & 1) == 0 && ((uintptr_t)p.out & 3) == 0 && n + 3 < p.N;
#pragma unroll 2
    for (int col = rank + (threadIdx.x / 32) * p.splits; col < cols; col += kThreads / 32 * p.splits) {
      const uint32_t off = base + (uint32_t)col * BM * 4;
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        v[r] = r < p.splits ? ld_cluster_f32x4(tc::mapa_shared(off, (uint32_t)r))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 s = v[0];
#pragma unroll
      for (int r = 1; r < 8; ++r) {
        s.x += v[r].x;
        s.y += v[r].y;
        s.z += v[r].z;
        s.w += v[r].w;
      }
      const float ra = p.ra ? p.ra[m0 + col] : 1.0f;
      alignas(8) TO o[4] = {out_f32<TO>(s.x * rw[0] * ra), out_f32<TO>(s.y * rw[1] * ra),
                            out_f32<TO>(s.z * rw[2] * ra), out_f32<TO>(s.w * rw[3] * ra)};
      TO *dst = (TO *)p.out + (m0 + col) * p.ldo + n;
      if (pairs) {
        reinterpret_cast<uint32_t *>(dst)[0] = reinterpret_cast<const uint32_t *>(o)[0];
        reinterpret_cast<uint32_t *>(dst)[1] = reinterpret_cast<const uint32_t *>(o)[1];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < p.N) dst[j] = o[j];
      }
    }
    tc::cluster_sync();  // the others have read this CTA's sums
  }
}

// Tile of tokens, splits of K and CTAs on an SM: the least of an estimate in SM cycles, whose
// constants are fits to sweeps over all shapes at 1 to 2048 tokens.
//   - a k-block of a tile takes max(300 + 1.7 tn, 3.45 tn): the MMAs, below about 170 tokens the
//     issue of them and their waits;
//   - the busiest SM has `busy` tiles, together or one after another;
//   - the memory brings each operand once at 3500 bytes a cycle, L2 what the tiles fill again;
//     the two times overlap in part (root of the sum of squares);
//   - a launch costs 6400, splitting K 1400 + 8 tn (two cluster barriers and the exchange).
// Two CTAs on an SM cover each other's waits and ends, where the tile is small enough for three
// stages each.
struct Shape { int tn, splits, per_sm; };

// Clusters of `splits` CTAs, one on an SM, that run at once.  They lie within groups of SMs, so
// there is room for fewer than SMs / splits: 152 SMs take 46 clusters of three (52 x 6144 x 2896
// has 48 tiles of 64 tokens: split in three it took 13.7 us, in two rounds; now 8.8).
template <typename TO>
int clusters_at_once(int dev, int splits, int sms) {
  static PerDevice<9> known;
  return known.get(dev, splits, [splits, sms]() {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(splits * sms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kRingBytes + kSmemBesides;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (const void *)matmul_kernel<TO>, &cfg) == cudaSuccess) return n;
    (void)cudaGetLastError();
    return 0;
  }, sms / splits * 7 / 8);
}

template <typename TO>
Shape choose(int64_t M, int64_t N, int64_t K, int dev, int sms) {
  const int64_t n_w = ceil_div(N, BM), groups = ceil_div(ceil_div(K, BK), 4);
  const double once = (double)(M + N) * K / 3500.0;
  Shape best{16, 1, 1};
  double best_t = 1e30;
  const int64_t least = ceil_div(M, kMaxTn);
  for (int64_t mt = least; mt < least + 6; ++mt) {
    const int tn = (int)(ceil_div(ceil_div(M, mt), 16) * 16);
    const int64_t tiles = n_w * ceil_div(M, tn);
    const double c = tn < 172 ? 300 + 1.7 * tn : 3.45 * tn;
    const double fill = (double)tiles * K * (BM + tn) / 20000.0;
    for (int s = 1; s <= 8 && s <= groups; ++s) {
      for (int per = 1; per <= 2; ++per) {
        const int64_t ctas = tiles * s;
        if (per == 2 && ((uint32_t)(BM + tn) * BK * 3 > kRingBytesTwo || ctas <= sms || ctas > 2 * sms))
          continue;
        if (s > 1 && tiles > (int64_t)per * clusters_at_once<TO>(dev, s, sms)) continue;
        const int64_t busy = ceil_div(ctas, sms);
        const double work = (double)busy * 4 * ceil_div(groups, s) * c * (per == 2 ? 0.95 : 1.0);
        double t = sqrt(work * work + (once + fill) * (once + fill));
        t += 6400.0 + (s > 1 ? 1400.0 + 8.0 * tn : 0.0) + (per == 1 ? 800.0 * (busy - 1) : 0.0);
        if (t < best_t) best_t = t, best = Shape{tn, s, per};
      }
    }
    if (tn <= 32) break;
  }
  return best;
}

template <typename TO>
gptq_status run(const Fp8MatmulArgs &g, DevStatus *st, cudaStream_t s) {
  GPTQ_TRY(ensure_smem_attr((const void *)matmul_kernel<TO>, (int)(kRingBytes + kSmemBesides)));
  int sms = 0;
  GPTQ_TRY(device_sm_count(&sms));
  const int kb = (int)ceil_div(g.K, BK);
  int dev = -1;
  GPTQ_CUDA_CHECK(cudaGetDevice(&dev));
  const Shape sh = choose<TO>(g.M, g.N, g.K, dev, sms);
  MmParams p{};
  p.ae = g.ae; p.ldae = g.ldae;
  p.we = g.we; p.ldwe = g.ldwe;
  p.ra = g.ra; p.rw = g.rw;
  p.out = g.out; p.ldo = g.ldo;
  p.M = g.M; p.N = g.N;
  p.kb = kb;
  p.tn = sh.tn;
  p.n_w = (int)ceil_div(g.N, BM);
  const int64_t tiles = p.n_w * ceil_div(g.M, sh.tn);
  if (tiles * 8 > INT32_MAX) return GPTQ_ERR_UNSUPPORTED;
  p.n_tiles = (int)tiles;
  p.splits = sh.splits;
  p.wait_ns = g.wait_ns;
  p.lost = (int)g.lost;
  const bool one_tile = sh.splits > 1 || tiles <= (int64_t)sms * sh.per_sm;
  p.ring_bytes = sh.per_sm > 1 ? kRingBytesTwo : kRingBytes;
  const int fit = (int)(p.ring_bytes / (uint32_t)((BM + sh.tn) * BK));
  p.stages = fit < kMaxStages ? fit : kMaxStages;
  // an accumulator for the tile at hand and one for the next, or one and 256 columns at most
  p.acc_cols = one_tile && sh.tn <= 224 ? (sh.tn + 31) / 32 * 32 : kMaxTn;
  p.tmem_cols = kTmemCols;
  if (one_tile && sh.tn <= 224)
    for (p.tmem_cols = 64; p.tmem_cols < p.acc_cols + 2 * (int)kScaleCols;) p.tmem_cols *= 2;
  CUtensorMap mw, ma;
  if (!tc::make_tmap_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w, g.N, g.K, g.ldw, BK, BM) ||
      !tc::make_tmap_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a, g.M, g.K, g.lda, BK, sh.tn))
    return GPTQ_ERR_UNSUPPORTED;
  const int64_t slots = (int64_t)sms * sh.per_sm;
  const int64_t ctas = sh.splits > 1 ? tiles * sh.splits : (tiles < slots ? tiles : slots);
  return launch_early(matmul_kernel<TO>, dim3((unsigned)ctas), dim3(kThreads),
                      p.ring_bytes + kSmemBesides, sh.splits, s, mw, ma, p, st);
}

}  // namespace

size_t fp8_matmul_ws_bytes(int64_t, int64_t, int64_t) { return 256; }

gptq_status fp8_matmul_take_timeout(int *out, cudaStream_t s) { return take_flag(g_gave_up, out, s); }

gptq_status launch_fp8_matmul(const Fp8MatmulArgs &g, void *ws, cudaStream_t s) {
  if (g.M == 0) {
    GPTQ_CUDA_CHECK(cudaMemsetAsync(ws, 0, sizeof(DevStatus), s));
    return GPTQ_OK;
  }
  return g.odtype == GPTQ_F16 ? run<__half>(g, (DevStatus *)ws, s)
                              : run<__nv_bfloat16>(g, (DevStatus *)ws, s);
}

}  // namespace gptq
