// Product of two microscaled matrices on the fifth-generation tensor cores:
//
//   y[t][i] = sum_k 2^(ex[t][k] + ew[i][k]) sum_{j < 32} qx[t][32k + j] qw[i][32k + j]
//
// tcgen05 block-scaled MMA reads the codes as they are (two operands in 4 bits:
// kind::mxf4, K 64 an instruction; else kind::mxf8f6f4, K 32, 4-bit rows being
// widened to a byte per element by the TMA copy) and applies the scales of both
// operands itself, from tensor memory.  Sums are fp32.
//
// Both kernels fill a shared-memory ring by TMA in steps of 128 bytes of every
// row: 256 4-bit or 128 byte-wide elements of K, with the 512-byte scale tiles
// (128 rows x 128 elements) that belong to them.  tcgen05.cp brings those into
// tensor memory.  Roles (192 threads): warp 0 TMA producer; warp 1 tensor memory
// and the single-thread issue of scale copies and MMAs; warps 2-5 epilogue.
//
// Every wait is bounded; one that gives up records DBF_ERR_TIMEOUT in the
// workspace's status word and the kernel ends with y incomplete.
#include <algorithm>
#include <mutex>

#include "dbf_internal.h"
#include "mx_device.cuh"

namespace dbf {
namespace {

constexpr int kRows = 128;  // rows of P per tile (TMEM lanes)
constexpr int kThreads = 192;
constexpr int kRowBytes = 128;  // bytes of a row per stage
constexpr int kTileBytes = 512;  // a scale tile
constexpr size_t kStatusBytes = 256;

struct MxArgs {
  const uint8_t* p_scales;
  const uint8_t* q_scales;
  int64_t p_rows, q_rows;
  int64_t k4s;       // 128-element groups of K (scale tiles in a row of tiles)
  int steps_k;       // steps (128 bytes of a row) of the whole K range
  int p_tx, q_tx;    // bytes that a row of P, Q counts on its barrier
  uint32_t idesc;
  int w_static;      // the weights may be read before the PDL wait
  void* out;
  int64_t ld_out;
  int out_t;
  int* status;
};

__device__ __forceinline__ void store_out(void* out, int t, int64_t at, float v) {
  if (t == DBF_F32) {
    static_cast<float*>(out)[at] = v;
  } else if (t == DBF_F16) {
    static_cast<__half*>(out)[at] = __float2half_rn(v);
  } else {
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  }
}

// ---------------------------------------------------------------- few tiles: K split over a cluster
// Tiles of 128 weight rows (the tensor cores' M) by NT tokens (their N; up to NT
// tokens read as zero).  The K range of a tile is split over the CTAs of a
// cluster, each of which sends its fp32 partial sums of token group g to CTA
// g % size, which adds them in rank order.  With few tokens the weights'
// stream bounds it; a stage of the ring is U steps, because a stage costs some
// 250 cycles of waiting and signalling however little it multiplies (one token x
// 14336 x 4096, 8-bit tokens: 9.5 us with one step, 9.1 with two).
// Measured: 4-bit weights of 4096 x 4096 / 14336 x 4096, one token in 8 bits 4.6 /
// 9.0 us (the weights' DRAM time is 30 / 53% of that), in 4 bits 7.7 us for the wide
// one; 16 tokens 5.1 / 9.4 us; 128 tokens x 4096 x 4096 8.6 us.  The wide layer's 112
// tiles cannot be split by two over 148 SMs: 36 of them have no work, and the
// others read a whole row of tiles each.
template <int KA, int NT>
struct SplitCfg {
  static constexpr int U = NT <= 32 ? 2 : 1;
  static constexpr int kPBytes = kRows * kRowBytes;  // of a step
  static constexpr int kQBytes = NT * kRowBytes;
  static constexpr int kScaleBytes = U * KA * kTileBytes;  // of a stage and operand
  static constexpr int kStageBytes = U * (kPBytes + kQBytes) + 2 * kScaleBytes;
  static constexpr int kEpiBytes = (NT < 32 ? 32 : NT) * kRows * 4;  // the partial sums of the cluster
  static constexpr int kRoom = 227 * 1024 - 1024 - 512 - kEpiBytes;
  static constexpr int kStages = kRoom / kStageBytes < 8 ? kRoom / kStageBytes : 8;
  static constexpr int kEpiOffset = kStages * kStageBytes;
  static constexpr int kBarOffset = kEpiOffset + kEpiBytes;
  static constexpr int kSmemBytes = kBarOffset + 512 + 1024;
  // tensor memory: the accumulator, then each stage's scales (a copy may
  // overtake earlier MMAs, so a stage's place is its own as long as its slot of the ring is)
  static constexpr int kScaleCols = 2 * 4 * KA * U;
  static constexpr int kDCols = NT < 32 ? 32 : NT;
  static constexpr int kNeedCols = kDCols + kStages * kScaleCols;
  static constexpr int kTmemCols = kNeedCols <= 128 ? 128 : kNeedCols <= 256 ? 256 : 512;
  static_assert(kNeedCols <= 512, "accumulator and scales must fit in tensor memory");
  static_assert(kStages >= 2, "");
};

template <int KA, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    dbf_mx_gemm_split_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                             const MxArgs a) {
  using C = SplitCfg<KA, NT>;
  constexpr int S = C::kStages, U = C::U;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // operand rings first: their 128-byte swizzle counts from 1024-byte boundaries
  uint8_t* p_st = smem;
  uint8_t* q_st = smem + S * U * C::kPBytes;
  uint8_t* s_st = q_st + S * U * C::kQBytes;  // per stage: P's tiles, Q's tiles
  float* epi = reinterpret_cast<float*>(smem + C::kEpiOffset);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* mma_done = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ks = static_cast<int>(cluster_size());
  const int rank = static_cast<int>(cluster_rank());
  const int64_t p_tiles = (a.p_rows + kRows - 1) / kRows;
  const int64_t tile = blockIdx.x / ks;
  const int64_t p0 = (tile % p_tiles) * kRows, q0 = (tile / p_tiles) * NT;
  // this CTA's steps of K, and stages of U of them
  const int k0 = static_cast<int>(static_cast<int64_t>(a.steps_k) * rank / ks);
  const int k1 = static_cast<int>(static_cast<int64_t>(a.steps_k) * (rank + 1) / ks);
  const int stages = (k1 - k0 + U - 1) / U;

  // The producer's thread sets up the barriers and, if the weights may be read at
  // once, has the first ring's worth of them on its way before anyone meets.
  auto tiles_of = [&](int k) {  // 128-element groups of the stage that starts at step k
    return static_cast<int>(min(static_cast<int64_t>(min(U, k1 - k) * KA), a.k4s - static_cast<int64_t>(k) * KA));
  };
  auto load = [&](bool weights, int i) {
    const int k = k0 + i * U, s = i % S, tiles = tiles_of(k);
    const CUtensorMap* map = weights ? &p_map : &q_map;
    const uint8_t* scales = weights ? a.p_scales : a.q_scales;
    const int64_t row = weights ? p0 : q0;
    const int bytes = weights ? C::kPBytes : C::kQBytes;
    uint8_t* st = (weights ? p_st : q_st) + s * U * bytes;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u == 0 || k + u < k1) tma_load_2d(st + u * bytes, map, (k + u) * 128, static_cast<int>(row), &full[s]);
    bulk_load(s_st + (2 * s + (weights ? 0 : 1)) * C::kScaleBytes,
              scales + ((row >> 7) * a.k4s + static_cast<int64_t>(k) * KA) * kTileBytes, tiles * kTileBytes, &full[s]);
  };
  auto expect = [&](int i) {
    const int k = k0 + i * U;
    mbar_arrive_expect_tx(&full[i % S], min(U, k1 - k) * (kRows * a.p_tx + NT * a.q_tx) + 2 * tiles_of(k) * kTileBytes);
  };
  const int early = min(S, stages);
  if (tid == 0) {
    prefetch_tmap(&p_map);
    prefetch_tmap(&q_map);
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (a.w_static) {
      for (int i = 0; i < early; ++i) {
        expect(i);
        load(true, i);
      }
    }
  }
  __syncwarp();
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  // a rank's partial sums are written only after every CTA of its cluster has started
  cluster_arrive_relaxed();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (elect_one()) {
      pdl_wait();
      for (int i = 0; i < early; ++i) {
        if (!a.w_static) {
          expect(i);
          load(true, i);
        }
        load(false, i);
      }
      int it = early;
      for (; it < stages; ++it) {
        if (!mbar_wait_often<false>(&empty[it % S], (it / S - 1) & 1, abort_flag, a.status)) break;
        expect(it);
        load(true, it);
        load(false, it);
      }
      // after a wait that gave up: no copy may still be on its way when the CTA ends
      if (*abort_flag) {
        int never = 0;
        for (int i = max(0, it - S); i < it; ++i) (void)mbar_wait_often<false>(&full[i % S], (i / S) & 1, &never, a.status);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ scale copies and MMAs
    if (elect_one()) {
      pdl_wait();  // (the bounded waits start only when the kernel before has ended)
      bool ok = true;
      for (int it = 0; it < stages; ++it) {
        const int k = k0 + it * U, s = it % S;
        if (!mbar_wait_often<false>(&full[s], (it / S) & 1, abort_flag, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sc = smem_u32(s_st + 2 * s * C::kScaleBytes);
        const uint32_t sfp = tmem + C::kDCols + s * C::kScaleCols, sfq = sfp + 4 * KA * U;
        // K behind the last group of 128 elements is not multiplied: it has no scales
        const int64_t tiles = a.k4s - static_cast<int64_t>(k) * KA;
#pragma unroll
        for (int z = 0; z < KA * U; ++z) {
          if (z >= KA && k + z / KA >= k1) break;
          tc_copy_scales(sfp + 4 * z, smem_desc_rows16(sc + z * kTileBytes));
          tc_copy_scales(sfq + 4 * z, smem_desc_rows16(sc + C::kScaleBytes + z * kTileBytes));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (u > 0 && k + u >= k1) break;
          const uint32_t pa = smem_u32(p_st + (s * U + u) * C::kPBytes), qa = smem_u32(q_st + (s * U + u) * C::kQBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (KA == 2 && kk >= 2 && tiles <= 2 * u + 1) break;
            const uint32_t acc = it != 0 || u != 0 || kk != 0 ? 1u : 0u;
            const uint64_t pd = smem_desc_sw128_kmajor(pa + kk * 32), qd = smem_desc_sw128_kmajor(qa + kk * 32);
            if constexpr (KA == 2) {
              const uint32_t id = 2u * (kk & 1), at = 4 * (2 * u + (kk >> 1));
              tc_mma_mxf4(tmem, pd, qd, a.idesc | (id << 4) | (id << 29), sfp + at, sfq + at, acc);
            } else {
              tc_mma_mxf8f6f4(tmem, pd, qd,
                              a.idesc | (static_cast<uint32_t>(kk) << 4) | (static_cast<uint32_t>(kk) << 29), sfp + 4 * u,
                              sfq + 4 * u, acc);
            }
          }
        }
        tc_commit(&empty[s]);
      }
      if (ok) tc_commit(acc_full);
      tc_commit(mma_done);
    }
  } else {
    // ------------------------------------------------ epilogue
    pdl_wait();
    const int q = warp & 3;  // the TMEM lanes this warp may read
    const bool ok = __all_sync(0xffffffffu, mbar_wait_often<false>(acc_full, 0, abort_flag, a.status));
    tc_fence_after();
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const int64_t p_row = p0 + q * 32 + lane;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), a.q_rows - q0));
    if (ks == 1) {
      for (int c = 0; c < tokens && ok; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(acc + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < tokens && p_row < a.p_rows)
            store_out(a.out, a.out_t, (q0 + c + j) * a.ld_out + p_row, __uint_as_float(v[j]));
      }
    } else {
      // four tokens a store; token group g belongs to rank g % ks (ks a power
      // of two), which finds rank src's part at [src][g / ks][row]
      const int lg = 31 - __clz(ks), groups = (tokens + 3) / 4, per = (groups + ks - 1) >> lg;
      float4* parts = reinterpret_cast<float4*>(epi) + q * 32 + lane;
      const uint32_t mine = smem_u32(parts + (rank * per) * kRows);
      cluster_wait_acquire();
      for (int c = 0; c < tokens && ok; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(acc + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const int g = (c + j) >> 2;
          if (g < groups)
            st_cluster_v4f32(cluster_addr(mine + (g >> lg) * (kRows * 16), g & (ks - 1)), __uint_as_float(v[j]),
                             __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
        }
      }
      cluster_arrive_release();
      cluster_wait_acquire();
      for (int g = rank; g < groups && ok; g += ks) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int src = 0; src < ks; ++src) {
          const float4 t = parts[(src * per + (g >> lg)) * kRows];
          sum.x += t.x, sum.y += t.y, sum.z += t.z, sum.w += t.w;
        }
        if (p_row < a.p_rows) {
          const float out[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (4 * g + j < tokens) store_out(a.out, a.out_t, (q0 + 4 * g + j) * a.ld_out + p_row, out[j]);
        }
      }
    }
  }

  // ------------------------------------------------ teardown
  // every thread takes part in the cluster's barriers: the epilogue's two of a
  // split tile, or one to pair the first arrival
  __syncwarp();
  if (ks == 1) {
    cluster_wait_acquire();
  } else if (warp < 2) {
    cluster_wait_acquire();
    cluster_arrive_release();
    cluster_wait_acquire();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    int never = 0;  // the MMAs under way are waited for after a wait that gave up, too
    (void)mbar_wait_often<false>(mma_done, 0, &never, a.status);
    __syncwarp();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- many tiles: CTA pairs
// Tiles of 256 tokens x 256 weight rows, one per pair of CTAs (cta_group::2):
// each CTA holds its 128 tokens and half of the tile's weight rows, so a step
// costs it 32 KB where a CTA alone would fetch 48; the MMA reads both.  The
// pairs are persistent (one CTA per SM) and walk the work items, tokens fastest;
// the ring runs on across items.  Tiles that would leave most pairs idle (all of
// few, or the last round's) are cut into 2 or 4 items of 128 or 64 weight rows (which
// still fetch a whole tile's weight rows: a step of a quarter costs 0.25 us where a
// whole one costs 0.34).  Up to 128 tokens the odd CTA of a pair multiplies only
// rows behind the last token.
// Accumulators: tensor memory holds two of 256 columns that overlap in their
// last / first columns (both do not fit beside the scales), so the MMAs of an
// item wait only until the epilogue has read the shared columns of the one before.
// The epilogue writes through shared memory with TMA stores (rows of y on 16
// bytes), else row by row (n = 14335 fp16: 101 us where 14336 takes 50).
// The issue of a step's copies, MMAs and commit by one thread takes 590 cycles,
// its MMAs alone 512: that, the accumulators' hand-over (about 1000 cycles an
// item) and the clock under load bound it.  Loads, stores and the copies were
// taken out one at a time without effect.  Tried and slower: the scales written
// by other warps with tcgen05.st (220 us for 84: it waits behind the MMAs),
// copies by a second thread (93), 192 weight rows with no shared columns (95).
// Measured: 2048 x 14336 x 4096, everything in 4 bits, fp16 out 49.5 us (4.86
// PFLOP/s); 2048 x 4096 x 14336, tokens in 8 bits 82 us (2.9 PFLOP/s).
constexpr int kPairCols = 256;  // weight rows of a whole tile
template <int KA>
struct PairCfg {
  static constexpr int kQRows = kPairCols / 2;
  static constexpr int kQTiles = kPairCols / 128;  // scale tiles of a tile's weight rows
  static constexpr int kPBytes = kRows * kRowBytes;
  static constexpr int kQBytes = kQRows * kRowBytes;
  static constexpr int kScaleBytes = KA * (1 + kQTiles) * kTileBytes;
  static constexpr int kStageBytes = kPBytes + kQBytes + kScaleBytes;
  static constexpr int kWarpBuf = 32 * 128;  // 32 rows x 32 columns
  static constexpr int kBufs = 3;            // per epilogue warp
  static constexpr int kEpiBytes = 4 * kBufs * kWarpBuf;
  static constexpr int kRoom = 227 * 1024 - 1024 - 512 - kEpiBytes;
  static constexpr int kMost = 5;  // more would cost the accumulators' columns
  static constexpr int kStages = kRoom / kStageBytes < kMost ? kRoom / kStageBytes : kMost;
  static constexpr int kEpiOffset = kStages * (kPBytes + kQBytes);
  static constexpr int kScaleOffset = kEpiOffset + kEpiBytes;
  static constexpr int kBarOffset = kScaleOffset + kStages * kScaleBytes;
  static constexpr int kSmemBytes = kBarOffset + 512 + 1024;
  // scales in tensor memory: a copy may overtake the MMAs issued before it, so a
  // stage's place is its own as long as its slot of the ring is
  static constexpr int kScaleCols = 4 * KA * (1 + kQTiles);
  static constexpr int kScaleBase = 512 - kStages * kScaleCols;
  // the second accumulator starts where it still ends before the scales
  static constexpr int kAcc1 = (kScaleBase - kPairCols) / 32 * 32;
  static constexpr int kShared = kPairCols - kAcc1;  // columns both accumulators use
  static_assert(kShared % 32 == 0 && kShared <= 128, "");
};

struct PairArgs {
  int64_t p_rows, q_rows;
  int64_t k4s;
  int steps_k;
  int tx;  // bytes of a stage, both CTAs
  uint32_t idesc;  // without N
  int64_t whole;   // items that are whole tiles; the tiles behind them are cut
  int cut;         // into this many items each (1, 2 or 4)
  void* out;
  int64_t ld_out;
  int out_t;
  int tma_out;
  int* status;
};

// Rows of y that do not start on 16 bytes, from the swizzled 32 x 32 chunk in
// shared memory: a lane per column, sixteen rows under way together.
template <typename E>
__device__ __forceinline__ void store_rows(const uint8_t* src, E* out, int64_t ld, int rows, int lane) {
  constexpr int kLine = 32 * sizeof(E), kPer = 16 / sizeof(E);  // bytes of a row, elements of a 16-byte chunk
#pragma unroll
  for (int r0 = 0; r0 < 32; r0 += 16) {
    E e[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int rr = r0 + k, key = sizeof(E) == 4 ? rr & 7 : (rr >> 1) & 3;
      e[k] = *reinterpret_cast<const E*>(src + rr * kLine + (((lane / kPer) ^ key) << 4) + (lane % kPer) * sizeof(E));
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (r0 + k < rows) out[(r0 + k) * ld] = e[k];
  }
}

template <int KA>
__global__ void __launch_bounds__(kThreads, 1)
    dbf_mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                            const __grid_constant__ CUtensorMap ps_map, const __grid_constant__ CUtensorMap qs_map,
                            const __grid_constant__ CUtensorMap y_map, const PairArgs a) {
  using C = PairCfg<KA>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* p_st = smem;
  uint8_t* q_st = smem + S * C::kPBytes;
  uint8_t* epi_st = smem + C::kEpiOffset;
  uint8_t* s_st = smem + C::kScaleOffset;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);  // the even CTA's count both CTAs' bytes
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;   // one per accumulator
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* acc_shared = acc_empty + 2;  // the columns that the accumulators share have been read
  uint64_t* mma_done = acc_shared + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int64_t p_tiles = (a.p_rows + 255) / 256;
  const int64_t tiles = p_tiles * ((a.q_rows + kPairCols - 1) / kPairCols);
  const int64_t items = a.whole + (tiles - a.whole) * a.cut;
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  struct Item {
    int64_t p0, q0;  // first token, first weight row
    int cols;        // weight rows
  };
  auto item = [&](int64_t i) {
    const int64_t j = i - a.whole;
    const int64_t tile = j < 0 ? i : a.whole + j / a.cut;
    const int cols = j < 0 ? kPairCols : kPairCols / a.cut;
    return Item{(tile % p_tiles) * 256, (tile / p_tiles) * kPairCols + (j < 0 ? 0 : j % a.cut * cols), cols};
  };

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);  // the epilogue warps of both CTAs
      mbar_init(&acc_shared[i], 8);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&p_map);
    prefetch_tmap(&q_map);
    prefetch_tmap(&ps_map);
    prefetch_tmap(&qs_map);
    if (a.tma_out) prefetch_tmap(&y_map);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  // no copy, MMA or arrival reaches the other CTA before its barriers stand
  cluster_arrive_release();
  cluster_wait_acquire();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------ TMA producer (each CTA its own halves)
    if (elect_one()) {
      bool ok = true;
      uint32_t it = 0;
      pdl_wait();
      for (int64_t t = pair; t < items && ok; t += pairs) {
        const Item w = item(t);
        const int p0 = static_cast<int>(w.p0) + rank * kRows, q0 = static_cast<int>(w.q0);
        for (int kt = 0; kt < a.steps_k; ++kt, ++it) {
          const int s = static_cast<int>(it % S);
          if (it >= S && !mbar_wait_often<true>(&empty[s], (it / S - 1) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], a.tx);
          const uint32_t bar = map_to_rank(&full[s], 0);
          uint8_t* sc = s_st + s * C::kScaleBytes;
          tma_load_2d_pair(p_st + s * C::kPBytes, &p_map, kt * 128, p0, bar);
          tma_load_2d_pair(q_st + s * C::kQBytes, &q_map, kt * 128, q0 + rank * (w.cols / 2), bar);
          tma_load_2d_pair(sc, &ps_map, kt * 128 * KA, p0 >> 7, bar);
          tma_load_2d_pair(sc + KA * kTileBytes, &qs_map, kt * 128 * KA, q0 >> 7, bar);
        }
      }
      // after a wait that gave up: no copy may still be on its way when the CTAs
      // end.  The even CTA's barriers count both CTAs' bytes; the odd one gives its
      // copies, which take microseconds, a millisecond.
      if (*abort_flag) {
        int never = 0;
        if (rank == 0) {
          for (uint32_t i = it < S ? 0 : it - S; i < it; ++i)
            (void)mbar_wait_often<true>(&full[i % S], (i / S) & 1, &never, a.status);
        } else {
          const unsigned long long t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 1000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ scale copies and MMAs (the even CTA's, for both)
    if (rank == 0 && elect_one()) {
      pdl_wait();  // (the bounded waits start only when the kernel before has ended)
      bool ok = true;
      uint32_t it = 0, n = 0;
      for (int64_t t = pair; t < items && ok; t += pairs, ++n) {
        const uint32_t b = n & 1, use = n >> 1;
        // this accumulator's last tile has been read, and the tile before has
        // left the shared columns
        if (n >= 2) ok = mbar_wait_often<true>(&acc_empty[b], (use - 1) & 1, abort_flag, a.status);
        if (C::kShared > 0 && n >= 1 && ok)
          ok = mbar_wait_often<true>(&acc_shared[b ^ 1], ((n - 1) >> 1) & 1, abort_flag, a.status);
        if (!ok) break;
        const uint32_t d = tmem + b * C::kAcc1;
        const Item w = item(t);
        // where the item's first weight row lies in its scale tile (column 0 or 2)
        const uint32_t q_col = static_cast<uint32_t>(w.q0 & 127) >> 5;
        const uint32_t idesc = a.idesc | (static_cast<uint32_t>(w.cols >> 3) << 17);
        for (int kt = 0; kt < a.steps_k; ++kt, ++it) {
          const int s = static_cast<int>(it % S);
          ok = mbar_wait_often<true>(&full[s], (it / S) & 1, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sfa = tmem + C::kScaleBase + s * C::kScaleCols, sfb = sfa + 4 * KA;
          const uint32_t sc = smem_u32(s_st + s * C::kScaleBytes);
#pragma unroll
          for (int k = 0; k < KA; ++k) {
            tc_copy_scales_pair(sfa + 4 * k, smem_desc_rows16(sc + k * kTileBytes));
#pragma unroll
            for (int j = 0; j < C::kQTiles; ++j)
              tc_copy_scales_pair(sfb + 4 * (k * C::kQTiles + j), smem_desc_rows16(sc + (KA * (1 + j) + k) * kTileBytes));
          }
          const uint32_t pa = smem_u32(p_st + s * C::kPBytes), qa = smem_u32(q_st + s * C::kQBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t acc = kt != 0 || kk != 0 ? 1u : 0u;
            const uint64_t pd = smem_desc_sw128_kmajor(pa + kk * 32), qd = smem_desc_sw128_kmajor(qa + kk * 32);
            if constexpr (KA == 2) {
              const uint32_t id = 2u * (kk & 1);
              tc_mma_mxf4_pair(d, pd, qd, idesc | (id << 4) | (id << 29), sfa + 4 * (kk >> 1),
                               sfb + q_col + 4 * C::kQTiles * (kk >> 1), acc);
            } else {
              tc_mma_mxf8f6f4_pair(d, pd, qd,
                                   idesc | (static_cast<uint32_t>(kk) << 4) | (static_cast<uint32_t>(kk) << 29), sfa,
                                   sfb + q_col, acc);
            }
          }
          tc_commit_pair(&empty[s]);
        }
        if (ok) tc_commit_pair(&acc_full[b]);
      }
      tc_commit_pair(mma_done);
    }
  } else {
    // ------------------------------------------------ epilogue
    pdl_wait();
    const int q = warp & 3;  // the TMEM lanes this warp may read
    uint8_t* buf = epi_st + q * (C::kBufs * C::kWarpBuf);
    uint32_t n = 0, stores = 0;
    for (int64_t t = pair; t < items; t += pairs, ++n) {
      const uint32_t b = n & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_often<true>(&acc_full[b], (n >> 1) & 1, abort_flag, a.status))) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * C::kAcc1;
      const Item w = item(t);
      const int64_t row0 = w.p0 + rank * kRows + q * 32, q0 = w.q0;
      const int rows = static_cast<int>(max(int64_t{0}, min(int64_t{32}, a.p_rows - row0)));
      // 32 columns at a time; those shared with the other accumulator first, and
      // into registers all at once, so that its MMAs can start: the last ones of
      // accumulator 0, the first of accumulator 1
      auto column = [&](int i) { return b == 0 && C::kShared > 0 ? kPairCols - (i + 1) * 32 : i * 32; };
      auto signal = [&](uint64_t* bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_release(map_to_rank(bar, 0));
      };
      auto write = [&](int c0, const uint32_t (&v)[32]) {
        if (c0 >= w.cols) return;
        uint8_t* dst = buf + (stores % C::kBufs) * C::kWarpBuf;
        // the store that last used this buffer has read it
        if (lane == 0) bulk_wait_read<C::kBufs - 1>();
        __syncwarp();
        // the TMA map's swizzle: of a row's 16-byte chunks, chunk c lies at
        // c ^ (r & 7) of 128-byte rows, at c ^ (r / 2 & 3) of 64-byte rows
        if (a.out_t == DBF_F32) {
          uint8_t* line = dst + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(line + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          uint8_t* line = dst + lane * 64;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float lo = __uint_as_float(v[8 * j + 2 * e]), hi = __uint_as_float(v[8 * j + 2 * e + 1]);
              if (a.out_t == DBF_F16) {
                const __half2 p2 = __floats2half2_rn(lo, hi);
                h[e] = *reinterpret_cast<const uint32_t*>(&p2);
              } else {
                const __nv_bfloat162 p2 = __floats2bfloat162_rn(lo, hi);
                h[e] = *reinterpret_cast<const uint32_t*>(&p2);
              }
            }
            *reinterpret_cast<uint4*>(line + ((j ^ ((lane >> 1) & 3)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        if (a.tma_out) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (rows > 0 && q0 + c0 < a.q_rows) tma_store_2d(&y_map, dst, static_cast<int>(q0) + c0, static_cast<int>(row0));
            bulk_commit_group();
          }
          ++stores;
        } else {
          __syncwarp();
          const int64_t at = row0 * a.ld_out + q0 + c0 + lane;
          if (q0 + c0 + lane < a.q_rows) {
            if (a.out_t == DBF_F32) store_rows<uint32_t>(dst, static_cast<uint32_t*>(a.out) + at, a.ld_out, rows, lane);
            else store_rows<uint16_t>(dst, static_cast<uint16_t*>(a.out) + at, a.ld_out, rows, lane);
          }
          __syncwarp();
        }
      };
      constexpr int kFirst = C::kShared / 32;
      if constexpr (kFirst > 0) {
        uint32_t v[kFirst][32];
#pragma unroll
        for (int i = 0; i < kFirst; ++i) tmem_ld_32x32b_x32(acc + column(i), v[i]);
        tmem_ld_wait();
        signal(&acc_shared[b]);
#pragma unroll
        for (int i = 0; i < kFirst; ++i) write(column(i), v[i]);
      }
#pragma unroll 1
      for (int i = kFirst; i < kPairCols / 32; ++i) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(acc + column(i), v);
        tmem_ld_wait();
        if (i + 1 == kPairCols / 32) signal(&acc_empty[b]);
        write(column(i), v);
      }
    }
    if (lane == 0) bulk_wait_all<0>();
    __syncwarp();
  }

  // ------------------------------------------------ teardown
  // Warp 1 waits for the last MMAs: the even CTA's has issued them, the odd CTA's has
  // been here since the start and gets a wait's limit for each of its items (a barrier
  // with this CTA's other roles instead cost 0.4 us a launch).  After a wait that gave
  // up the MMAs under way are waited for all the same, with a limit of their own.
  __syncwarp();
  tc_fence_before();
  if (warp == 1) {
    bool done = false;
    if (rank == 1) {
      pdl_wait();
      for (int64_t t = pair; t < items && !done && !*abort_flag; t += pairs) {
        int never = 0;
        done = mbar_wait_often<true>(mma_done, 0, &never, nullptr);
      }
    }
    int never = 0;
    if (!done) (void)mbar_wait_often<true>(mma_done, 0, &never, a.status);
    __syncwarp();
  }
  // neither CTA ends while the other may still read its memory or signal it
  cluster_arrive_release();
  cluster_wait_acquire();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- host
struct Operand {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows;
  bool four;  // 4-bit codes
};

// The map of one operand's codes: 128-byte rows of the ring.  mxf4 copies the
// packed bytes; mxf8f6f4 copies bytes, or widens 16 4-bit elements to 16 bytes
// (8 of data, 8 unused).
bool operand_map(const Operand& o, int64_t pitch, bool packed, int box_rows, CUtensorMap* map) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const bool widen = o.four && !packed;
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(o.four ? pitch / 2 : pitch);
  const cuuint64_t dims[2] = {widen ? static_cast<cuuint64_t>(pitch) : row_bytes, static_cast<cuuint64_t>(o.rows)};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, widen ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                const_cast<uint8_t*>(o.codes), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs of a cluster that share a tile's K range: as many as the SMs hold, up to
// eight, with a step of K each at least.
int split_ways(int64_t tiles, int steps, int num_sms) {
  int ks = 1;
  while (ks < 8 && tiles * ks * 2 <= num_sms && ks * 2 <= steps) ks *= 2;
  return ks;
}

template <int KA, int NT>
dbf_status launch_split(const Operand& p, const Operand& q, MxArgs a, int64_t pitch, const DeviceInfo& dev,
                        cudaStream_t stream) {
  using C = SplitCfg<KA, NT>;
  auto kernel = dbf_mx_gemm_split_kernel<KA, NT>;
  const int64_t tiles = (p.rows + kRows - 1) / kRows * ((q.rows + NT - 1) / NT);
  int ks = split_ways(tiles, a.steps_k, dev.num_sms);
  static std::once_flag once[64];  // the attribute once per device
  static cudaError_t attr_err[64];
  std::call_once(once[dev.device], [&] {
    attr_err[dev.device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (attr_err[dev.device] != cudaSuccess) return DBF_ERR_CUDA;
  CUtensorMap p_map, q_map;
  if (!operand_map(p, pitch, KA == 2, kRows, &p_map) || !operand_map(q, pitch, KA == 2, NT, &q_map))
    return DBF_ERR_CUDA;
  a.p_scales = p.scales;
  a.q_scales = q.scales;
  a.p_rows = p.rows;
  a.q_rows = q.rows;
  // a widening copy counts the bytes it reads: half of what it fills
  a.p_tx = KA == 1 && p.four ? kRowBytes / 2 : kRowBytes;
  a.q_tx = KA == 1 && q.four ? kRowBytes / 2 : kRowBytes;
  a.idesc = KA == 2 ? idesc_block_scaled(kRows, NT, 1, 1) : idesc_block_scaled(kRows, NT, p.four ? 5 : 0, q.four ? 5 : 0);
  if (tiles * ks > 0x7fffffffLL) return DBF_ERR_UNSUPPORTED_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(ks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // No more clusters than the GPU holds at once (a GPC's SMs are no multiple of
  // eight): a second round would double the time.  16 tiles of 4096: 12.5 us over
  // eight CTAs each, 8.2 over four.
  while (ks > 1) {
    static std::once_flag asked[64][4];
    static int most[64][4];
    const int lg = ks == 2 ? 1 : ks == 4 ? 2 : 3;
    attr[1].val.clusterDim.x = static_cast<unsigned>(ks);
    cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms / ks * ks));
    std::call_once(asked[dev.device][lg], [&] {
      if (cudaOccupancyMaxActiveClusters(&most[dev.device][lg], kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        most[dev.device][lg] = 0;
      }
    });
    if (tiles <= most[dev.device][lg]) break;
    ks /= 2;
  }
  attr[1].val.clusterDim.x = static_cast<unsigned>(ks);
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * ks));
  return cudaLaunchKernelEx(&cfg, kernel, p_map, q_map, a) == cudaSuccess ? DBF_OK : DBF_ERR_CUDA;
}

// The map of one operand's scale tiles, as 32-bit words.
bool scale_map(const Operand& o, int64_t k4s, int ka, int box_tiles, CUtensorMap* map) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k4s * 128), static_cast<cuuint64_t>((o.rows + 127) / 128)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k4s * kTileBytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 * ka), static_cast<cuuint32_t>(box_tiles)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint8_t*>(o.scales), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The map of y for stores of 32 rows x 32 columns.
bool out_map(void* y, int out_t, int64_t rows, int64_t cols, CUtensorMap* map) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  const size_t e = dtype_size(out_t);
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * e};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapDataType t = out_t == DBF_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : out_t == DBF_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode(map, t, 2, y, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                e == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tiles of the last round (all of them where they fill no round) are cut
// into 2 or 4 items as long as every pair gets one at most.
struct PairPlan {
  int64_t whole, left;  // whole tiles in full rounds, tiles of the last round
  int cut;
};
PairPlan pair_plan(int64_t tokens, int64_t rows, int num_sms) {
  const int64_t tiles = (tokens + 255) / 256 * ((rows + kPairCols - 1) / kPairCols);
  const int64_t pairs = num_sms / 2, left = tiles % pairs;
  return {tiles - left, left, left * 4 <= pairs ? 4 : left * 2 <= pairs ? 2 : 1};
}

template <int KA>
dbf_status launch_pair(const Operand& x, const Operand& w, const MxArgs& m, int64_t pitch, const DeviceInfo& dev,
                       cudaStream_t stream) {
  using C = PairCfg<KA>;
  auto kernel = dbf_mx_gemm_pair_kernel<KA>;
  static std::once_flag once[64];  // the attribute once per device
  static cudaError_t attr_err[64];
  std::call_once(once[dev.device], [&] {
    attr_err[dev.device] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (attr_err[dev.device] != cudaSuccess) return DBF_ERR_CUDA;
  PairArgs a{};
  a.p_rows = x.rows;
  a.q_rows = w.rows;
  a.k4s = m.k4s;
  a.steps_k = m.steps_k;
  const int p_tx = KA == 1 && x.four ? kRowBytes / 2 : kRowBytes, q_tx = KA == 1 && w.four ? kRowBytes / 2 : kRowBytes;
  a.tx = 2 * (kRows * p_tx + C::kQRows * q_tx + C::kScaleBytes);
  a.idesc = KA == 2 ? idesc_block_scaled(256, 0, 1, 1) : idesc_block_scaled(256, 0, x.four ? 5 : 0, w.four ? 5 : 0);
  a.out = m.out;
  a.ld_out = m.ld_out;
  a.out_t = m.out_t;
  a.status = m.status;
  a.tma_out = m.ld_out * static_cast<int64_t>(dtype_size(m.out_t)) % 16 == 0;
  CUtensorMap p_map, q_map, ps_map, qs_map, y_map{};
  if (!operand_map(x, pitch, KA == 2, kRows, &p_map) || !operand_map(w, pitch, KA == 2, C::kQRows, &q_map) ||
      !scale_map(x, m.k4s, KA, 1, &ps_map) || !scale_map(w, m.k4s, KA, C::kQTiles, &qs_map) ||
      (a.tma_out && !out_map(m.out, m.out_t, x.rows, w.rows, &y_map)))
    return DBF_ERR_CUDA;
  const PairPlan plan = pair_plan(x.rows, w.rows, dev.num_sms);
  a.cut = plan.cut;
  a.whole = plan.whole;
  const int64_t items = plan.whole + plan.left * plan.cut, pairs = dev.num_sms / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(items, pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p_map, q_map, ps_map, qs_map, y_map, a) == cudaSuccess ? DBF_OK : DBF_ERR_CUDA;
}

template <int KA>
dbf_status launch_mx(const Operand& x, const Operand& w, const MxArgs& base, int64_t pitch, const DeviceInfo& dev,
                     cudaStream_t stream) {
  MxArgs a = base;
  a.steps_k = static_cast<int>((a.k4s + KA - 1) / KA);
  if (x.rows > 64) {
    // Estimated microseconds of both kernels: a step of K costs a CTA of the split
    // kernel 0.44 (4-bit operands, twice the K: 0.62), a pair 0.34 / 0.27 / 0.25
    // for 256 / 128 / 64 weight rows (4-bit: 0.39 / 0.32 / 0.30).  Both kernels timed
    // for 65 to 1024 tokens in both formats at 1024, 4096 and 14336 x 4096 and
    // 4096 x 14336 (56 points): the pairs take 0.89 to 1.29 of their estimate, the
    // split kernel 0.56 to 1.00, and the choice is the faster one or within 2.2% of
    // it at 49.  It loses 26 / 19% (4- / 8-bit tokens) for 65 tokens and 8 / 5% for
    // 128 at 14336 x 4096 (13.6 us on pairs, 10.8 split), 18% for 192 and 256 tokens
    // at 4096 x 14336 in 4 bits, 7% for 192 at 4096 x 4096 in 8.
    const bool four = KA == 2;
    const int64_t split_tiles = (w.rows + kRows - 1) / kRows * ((x.rows + 127) / 128);
    const int ks = split_ways(split_tiles, a.steps_k, dev.num_sms);
    const double split_rounds = static_cast<double>((split_tiles * ks + dev.num_sms - 1) / dev.num_sms);
    const double split_us = 3.5 + split_rounds * ((a.steps_k + ks - 1) / ks * (four ? 0.62 : 0.44) + 2.5);
    const PairPlan plan = pair_plan(x.rows, w.rows, dev.num_sms);
    const double cut_us = plan.left == 0 ? 0. : plan.cut == 1 ? (four ? 0.39 : 0.34) : plan.cut == 2 ? (four ? 0.32 : 0.27) : (four ? 0.30 : 0.25);
    const double pair_us = 4.5 + a.steps_k * (static_cast<double>(plan.whole / (dev.num_sms / 2)) * (four ? 0.39 : 0.34) + cut_us);
    // rows of y that do not start on 16 bytes cost the pairs' epilogue about 8 us a round
    const bool aligned = a.ld_out * static_cast<int64_t>(dtype_size(a.out_t)) % 16 == 0;
    const double store_us = aligned ? 0. : 8. * (static_cast<double>(plan.whole / (dev.num_sms / 2)) + (plan.left ? 1. / plan.cut : 0.));
    if (pair_us + store_us < split_us) return launch_pair<KA>(x, w, a, pitch, dev, stream);
    return launch_split<KA, 128>(w, x, a, pitch, dev, stream);
  }
  if (x.rows <= 16) return launch_split<KA, 16>(w, x, a, pitch, dev, stream);
  if (x.rows <= 32) return launch_split<KA, 32>(w, x, a, pitch, dev, stream);
  return launch_split<KA, 64>(w, x, a, pitch, dev, stream);
}

constexpr int64_t kMaxReduce = int64_t{1} << 20;

bool forward_shape_ok(int64_t n, int64_t m_in, int64_t batch) {
  return mx_shape_ok(n, m_in) && mx_shape_ok(batch, m_in) && m_in <= kMaxReduce;
}

}  // namespace
}  // namespace dbf

using namespace dbf;

extern "C" {

size_t dbf_mx_forward_workspace_bytes(int64_t n, int64_t m_in, int64_t batch) {
  return forward_shape_ok(n, m_in, batch) ? kStatusBytes : 0;
}

dbf_status dbf_mx_forward(const uint8_t* x_codes, const uint8_t* x_scales, dbf_mx_format x_fmt, const uint8_t* w_codes,
                          const uint8_t* w_scales, dbf_mx_format w_fmt, int64_t n, int64_t m_in, int64_t batch, void* y,
                          dbf_dtype y_t, void* workspace, size_t ws_bytes, uint32_t flags,
                          struct CUstream_st* stream) {
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return DBF_ERR_INVALID_ARG;
  if (!mx_format_ok(x_fmt) || !mx_format_ok(w_fmt) || !float_dtype_ok(y_t)) return DBF_ERR_INVALID_ARG;
  if (n < 1 || m_in < 1 || batch < 1 || (flags & ~static_cast<uint32_t>(DBF_FWD_WEIGHTS_STATIC)) != 0)
    return DBF_ERR_INVALID_ARG;
  if (!forward_shape_ok(n, m_in, batch)) return DBF_ERR_UNSUPPORTED_SHAPE;
  if (!aligned_to(x_codes, 32) || !aligned_to(w_codes, 32) || !aligned_to(x_scales, 16) || !aligned_to(w_scales, 16) ||
      !aligned_to(y, 16))
    return DBF_ERR_MISALIGNED;
  if (!workspace || !aligned_to(workspace, 16) || ws_bytes < dbf_mx_forward_workspace_bytes(n, m_in, batch))
    return DBF_ERR_WORKSPACE;
  DeviceInfo dev;
  const dbf_status st = current_device(&dev);
  if (st != DBF_OK) return st;
  MxArgs a{};
  a.k4s = mx_pitch(m_in) / 128;
  a.w_static = (flags & DBF_FWD_WEIGHTS_STATIC) != 0;
  a.out = y;
  a.ld_out = n;
  a.out_t = y_t;
  a.status = static_cast<int*>(workspace);
  const Operand x{x_codes, x_scales, batch, x_fmt == DBF_MX_E2M1}, w{w_codes, w_scales, n, w_fmt == DBF_MX_E2M1};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return x.four && w.four ? launch_mx<2>(x, w, a, mx_pitch(m_in), dev, s) : launch_mx<1>(x, w, a, mx_pitch(m_in), dev, s);
}

}  // extern "C"
