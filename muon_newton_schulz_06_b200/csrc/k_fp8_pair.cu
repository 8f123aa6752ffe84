// Block-scaled 8-bit products, 256 x 256 tiles by pairs of CTAs (tcgen05 cta_group::2), for
// results of many tiles.  The formula and the forms are those of k_fp8_gemm.cu.
//
// What bounds these products is the operands' way from L2 into shared memory: one SM takes
// about 50 B/clk (measured here on the 128 x 128 kernel, which asks for 128 B/clk at the
// tensor rate and stops at 1.7 PFLOP/s), so a CTA has to do more with each byte.  A pair's
// 256 x 256 tile asks for 64 B/clk per SM.
//
// Per CTA (384 threads, persistent over the pair's share of the tiles):
//   warp 0       TMA producer: 6-stage ring of 128 x 128 code tiles of A (this CTA's rows) and
//                B (this CTA's half of the columns); both CTAs' copies complete on the
//                leader's barrier
//   warp 1       tensor memory; in the leader the MMA issue (one thread)
//   warps 2, 3   scale words: this CTA's 128 rows of A, all 256 columns of B, per 512 codes
//   warps 4..11  epilogue of this CTA's 128 x 256 half, two warps per lane quadrant, each with
//                a 128 x 128 block's worth of columns: exactly one scale block of an 8-bit
//                result.  Results leave through 2 KB of shared memory per warp (32 rows x 64
//                bytes, 64-byte swizzle) and TMA stores.
//
// Tensor memory holds two accumulators that share 32 columns, [0, 256) and [224, 480), and two
// sets of scales in the rest: 512 columns have no room for two whole accumulators and scales.
// The epilogue reads the shared columns first and hands them over; the next tile's MMAs start
// then and overlap the rest of the epilogue.
//
// An 8-bit result needs its block's maximum before the first code: the four warps of a block
// read the accumulator twice (maximum; codes), keeping only the shared columns in registers.
// Every wait is bounded, the exchange of the maxima included.
#include <atomic>

#include "fp8_blocks.cuh"
#include "fp8_tc.cuh"

namespace muon {
namespace {

constexpr int kPStages8 = 6;
constexpr int kEpi = 8;
constexpr int kPairThreads = 128 + 32 * kEpi;
constexpr uint32_t kPOperand = 128 * kF8K;            // 16 KB
constexpr uint32_t kPStage = 2 * kPOperand;
constexpr uint32_t kPairTx = 2 * kPStage;
constexpr uint32_t kPSfSet = 3 * kF8SfBytes;          // A words, B words of both halves
constexpr int kPSfSets = 4;                           // in shared memory
constexpr uint32_t kOutStage = 2048;                  // 32 rows x 64 bytes per epilogue warp
constexpr uint32_t kPSmem =
    kPStages8 * kPStage + kEpi * kOutStage + kPSfSets * kPSfSet + 2 * kF8SlopeTable * 4 + 512 + 1024;
static_assert(kPSmem <= 232448, "shared memory per CTA");
constexpr uint32_t kAccStep = 224;  // first column of accumulator a: 224 a
constexpr uint32_t kPSfCol = 480;
constexpr uint32_t kPSfCols = 12;                     // per set in tensor memory, two sets
static_assert(kPSfSets % 2 == 0, "the scale warps take the sets in turn");
static_assert(kPSfCol + 2 * kPSfCols <= 512, "tensor memory columns");

struct PairTile {
  int gi, row, col, nkb;
};

// Tiles of a product in bands of 8 tile rows, columns outermost inside a band, so that the
// pairs running at one time share a compact rectangle of operands in L2.
template <typename Params>
__device__ __forceinline__ PairTile pair_tile(const Params& p, int t) {
  PairTile r;
  int gi = 0;
  while (gi + 1 < p.n && p.p[gi + 1].tile_begin <= t) ++gi;
  const F8Product& g = p.p[gi];
  const int local = t - g.tile_begin;
  const int band = local / (8 * g.tiles_n), rem = local - band * 8 * g.tiles_n;
  const int h = min(8, g.tiles_m - 8 * band);
  r.gi = gi;
  r.row = (8 * band + rem % h) * kF8PairTile;
  r.col = (rem / h) * kF8PairTile;
  r.nkb = (g.k + kF8K - 1) / kF8K;
  return r;
}

// 32 consecutive entries of one row of the addend.
__device__ __forceinline__ void add_c32(const F8Dense& c, int row, int col, int cols, float* v) {
  const int64_t at = (int64_t)row * c.ld + col;
  if (c.vec && col + 32 <= cols) {
    if (c.bf16) {
      const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(c.data) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = q[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] += __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
        }
      }
    } else {
      const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(c.data) + at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = q[i];
        v[4 * i] += x.x;
        v[4 * i + 1] += x.y;
        v[4 * i + 2] += x.z;
        v[4 * i + 3] += x.w;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (col + j < cols)
      v[j] += c.bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(c.data)[at + j])
                     : reinterpret_cast<const float*>(c.data)[at + j];
}

// Writes 16 bytes q of row `lane` of a staged block (64-byte swizzle).
__device__ __forceinline__ void stage16(uint8_t* blk, int lane, int q, uint4 x) {
  *reinterpret_cast<uint4*>(blk + lane * 64 + (((q ^ (lane >> 1)) & 3) << 4)) = x;
}

template <typename Params>
__global__ void __launch_bounds__(kPairThreads, 1) fp8_pair_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_smem = smem + kPStages8 * kPStage;
  uint8_t* sf_smem = out_smem + kEpi * kOutStage;
  float* slope = reinterpret_cast<float*>(sf_smem + kPSfSets * kPSfSet);  // e4m3's table, e5m2's
  uint64_t* full = reinterpret_cast<uint64_t*>(slope + 2 * kF8SlopeTable);
  uint64_t* empty = full + kPStages8;
  uint64_t* sf_full = empty + kPStages8;
  uint64_t* sf_empty = sf_full + kPSfSets;
  uint64_t* tfull = sf_empty + kPSfSets;
  uint64_t* tdone = tfull + 2;   // an accumulator has been read
  uint64_t* tover = tdone + 2;   // its columns shared with the other one have been read
  uint64_t* max_bar = tover + 2; // [2]: maxima of the two blocks
  uint64_t* drain = max_bar + 2;
  float* max_slot = reinterpret_cast<float*>(drain + 1);   // [2 turns][2 blocks][4 warps]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(max_slot + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;
  const int n_clusters = gridDim.x >> 1;

  if (p.backward) {
    f8_slope_init(slope, false, threadIdx.x, kPairThreads);
    f8_slope_init(slope + kF8SlopeTable, true, threadIdx.x, kPairThreads);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPStages8; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kPSfSets; ++a) {
      mbar_init(&sf_full[a], 2);  // a scale warp of both CTAs
      mbar_init(&sf_empty[a], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tdone[a], 2 * kEpi);
      mbar_init(&tover[a], kEpi);  // one block's warps of both CTAs
      mbar_init(&max_bar[a], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t peer_abort = peer_addr(smem_u32((const void*)abort_flag), rank ^ 1u);
  auto give_up = [&]() {
    *reinterpret_cast<volatile int*>(p.status) = kDevTimeout;  // page-locked host word
    __threadfence_system();
    *abort_flag = 1;
    remote_store_flag(peer_abort, 1);
  };

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer (both CTAs)
    if (elect_one()) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      const uint32_t ring = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t leader_full0 = peer_addr(full0, 0);
      for (int t = cluster; t < p.total_tiles && ok; t += n_clusters) {
        const PairTile tl = pair_tile(p, t);
        const CUtensorMap* ma = &p.map_a[tl.gi];
        const CUtensorMap* mb = &p.map_b[tl.gi];
        // coordinates (x, y) of each operand, one of which moves with k
        const bool a_mn = p.p[tl.gi].a_mn, b_mn = p.p[tl.gi].b_mn;
        const int row = tl.row + (int)rank * 128, col = tl.col + (int)rank * 128;
        int ax = a_mn ? row : 0, ay = a_mn ? 0 : row, bx = b_mn ? col : 0, by = b_mn ? 0 : col;
        const int adx = a_mn ? 0 : kF8K, ady = a_mn ? kF8K : 0, bdx = b_mn ? 0 : kF8K, bdy = b_mn ? kF8K : 0;
        for (int kb = 0; kb < tl.nkb; ++kb) {
          if (!bar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
          if (rank == 0) expect_tx_at(full0 + 8 * stage, kPairTx);
          const uint32_t a_dst = ring + stage * kPStage, bar = leader_full0 + 8 * stage;
          tma_load_2d_pair(a_dst, ma, bar, ax, ay);
          tma_load_2d_pair(a_dst + kPOperand, mb, bar, bx, by);
          ax += adx; ay += ady; bx += bdx; by += bdy;
          if (++stage == kPStages8) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok || *abort_flag) {
        give_up();
        spin_ns(kAbortGraceNs);  // copies already issued land within microseconds
      } else if (rank == 0) {
        for (uint32_t s = 0; s < kPStages8; ++s) {
          const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
          (void)mbar_wait(&full[s], par, nullptr);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issue (leader CTA)
    if (rank == 0 && elect_one()) {
      uint32_t stage = 0, phase = 0;
      uint32_t set = 0, sf_phase = 0;  // scale set of the next group
      int it = 0;
      bool ok = true;
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t sf_full0 = smem_u32(sf_full), sf_empty0 = smem_u32(sf_empty);
      const uint64_t ring_desc = sdesc(smem_u32(smem), 16, 1024);
      const uint64_t sf_desc = f8_sf_desc(smem_u32(sf_smem));
      for (int t = cluster; t < p.total_tiles && ok; t += n_clusters, ++it) {
        const PairTile tl = pair_tile(p, t);
        const F8Product& g = p.p[tl.gi];
        const int acc = it & 1;
        const uint32_t idesc = f8_idesc(g.a_e5m2, g.b_e5m2, g.a_mn, g.b_mn, kF8PairTile, kF8PairTile);
        const uint32_t a_step = (g.a_mn ? 4096 : 32) >> 4, b_step = (g.b_mn ? 4096 : 32) >> 4;
        if (!mbar_wait(&tdone[acc], (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag) ||
            (it > 0 && !mbar_wait(&tover[acc ^ 1], (uint32_t)(((it - 1) >> 1) & 1), abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)acc * kAccStep;
        uint32_t accumulate = 0;
        for (int kb = 0; kb < tl.nkb; kb += kF8Group) {
          // copies and products run in the order of their issue, so the two sets in tensor
          // memory need no barrier of their own
          const uint32_t sfa = tmem + kPSfCol + (set & 1u) * kPSfCols, sfb = sfa + 4;
          if (!bar_wait<true>(sf_full0 + 8 * set, sf_phase, abort_flag)) { ok = false; break; }
          const uint64_t src = sf_desc + (uint64_t)(set * (kPSfSet >> 4));
          f8_copy_sf_pair(sfa, src);
          f8_copy_sf_pair(sfb, src + (kF8SfBytes >> 4));
          f8_copy_sf_pair(sfb + 4, src + 2 * (kF8SfBytes >> 4));
          const int n = min(kF8Group, tl.nkb - kb);
#pragma unroll 1
          for (int q = 0; q < n; ++q) {
            if (!bar_wait(full0 + 8 * stage, phase, abort_flag)) { ok = false; break; }
            const uint64_t ad = ring_desc + (uint64_t)(stage * (kPStage >> 4)), bd = ad + (kPOperand >> 4);
            const uint32_t id = f8_idesc_sf(idesc, q);
            f8_mma_pair(d_tmem, ad, bd, id, sfa, sfb, accumulate);
            accumulate = 1;
#pragma unroll
            for (int k = 1; k < 4; ++k) f8_mma_pair(d_tmem, ad + k * a_step, bd + k * b_step, id, sfa, sfb, 1u);
            f8_commit_both_at(empty0 + 8 * stage);
            if (++stage == kPStages8) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          f8_commit_both_at(sf_empty0 + 8 * set);
          if (++set == kPSfSets) { set = 0; sf_phase ^= 1u; }
        }
        if (!ok) break;
        umma_commit_both(&tfull[acc]);
      }
      if (!ok) give_up();
      umma_commit_local(drain);
      (void)mbar_wait(drain, 0, nullptr);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------------ scale words (both CTAs)
    // warps 2 and 3 take the groups of 512 codes in turn, so that a group's bytes have the
    // time of two groups' products to arrive from L2
    const uint32_t mine = warp - 2;
    uint32_t turn = 0, set = mine, phase = 1;
    bool ok = true;
    const uint32_t leader_full0 = peer_addr(smem_u32(sf_full), 0);
    for (int t = cluster; t < p.total_tiles && ok; t += n_clusters) {
      const PairTile tl = pair_tile(p, t);
      const F8Product& g = p.p[tl.gi];
      for (int kb = 0; kb < tl.nkb; kb += kF8Group) {
        if ((turn++ & 1u) != mine) continue;
        const uint4 wa = f8_sf_words(g.sa, tl.row + (int)rank * 128, g.m, kb, tl.nkb, lane);
        const uint4 w0 = f8_sf_words(g.sb, tl.col, g.n, kb, tl.nkb, lane);
        const uint4 w1 = f8_sf_words(g.sb, tl.col + 128, g.n, kb, tl.nkb, lane);
        int got = 1;
        if (lane == 0) got = mbar_wait(&sf_empty[set], phase, abort_flag);
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        uint8_t* dst = sf_smem + set * kPSfSet + lane * 16;
        *reinterpret_cast<uint4*>(dst) = wa;
        *reinterpret_cast<uint4*>(dst + kF8SfBytes) = w0;
        *reinterpret_cast<uint4*>(dst + 2 * kF8SfBytes) = w1;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) remote_arrive(leader_full0 + 8 * set);
        if ((set += 2) >= kPSfSets) { set = mine; phase ^= 1u; }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const int ew = warp - 4;
    const int quad = warp & 3, half = ew >> 2;
    uint8_t* blk = out_smem + ew * kOutStage;
    const uint32_t leader_tdone = peer_addr(smem_u32(&tdone[0]), 0);
    const uint32_t leader_tover = peer_addr(smem_u32(&tover[0]), 0);
    uint32_t max_turn = 0;
    // one lane waits, so that the warp stays together when a wait runs out
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      int got = 1;
      if (lane == 0) got = mbar_wait(bar, parity, abort_flag);
      got = __shfl_sync(0xffffffffu, got, 0);
      __syncwarp();
      return got != 0;
    };
    int it = 0;
    bool ok = true;
    for (int t = cluster; t < p.total_tiles && ok; t += n_clusters, ++it) {
      const PairTile tl = pair_tile(p, t);
      const F8Product& g = p.p[tl.gi];
      const int acc = it & 1;
      const int row0 = tl.row + (int)rank * 128 + 32 * quad, row = row0 + lane;
      const int col0 = tl.col + 128 * half;
      const bool live = row < g.m;
      const int chunks = row0 < g.m ? max(0, min(4, (g.n - col0 + 31) / 32)) : 0;
      // the chunk in the columns shared with the other accumulator, -1 for the other block
      const int shared_c = acc == 0 ? (half == 1 ? 3 : -1) : (half == 0 ? 0 : -1);
      const bool backward = g.epi == kF8EpiRelu2Backward;

      // the checkpoint's 128 codes of this row, requested before the accumulator is waited for
      uint4 sv[8];
      float sv_scale = 0.f;
      const float* table = slope;
      if (backward) {
        const uint8_t* q = g.saved.codes + (int64_t)row * g.saved.ld + col0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          sv[i] = live && col0 + 16 * i < g.n ? *reinterpret_cast<const uint4*>(q + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t sb = live && col0 < g.n ? *f8_scale_at(g.saved, row, col0 / kFp8Block) : 127u;
        const int e = (int)sb - 127, parity = e & 1;
        sv_scale = sb == 255u ? __uint_as_float(0x7fc00000u) : f8_exp2((e - parity) / 2);
        table = slope + (g.saved.e5m2 ? kF8SlopeTable : 0) + 256 * parity;
      }

      if (!warp_wait(&tfull[acc], (uint32_t)((it >> 1) & 1))) { ok = false; break; }
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)acc * kAccStep + (uint32_t)(128 * half);

      // chunk c (32 columns) with addend, activation or its gradient; columns past n are 0
      auto finish = [&](int c, float* v) {
        const int col = col0 + 32 * c;
        if (g.c.data != nullptr && live) add_c32(g.c, row, col, g.n, v);
        if (g.epi == kF8EpiRelu2) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = f8_relu2(v[j]);
        } else if (backward) {
          uint4 x[2];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i == c) { x[0] = sv[2 * i]; x[1] = sv[2 * i + 1]; }
          const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = __fmul_rn(__fmul_rn(table[(w[j >> 2] >> (8 * (j & 3))) & 255u], sv_scale), v[j]);
        }
        if (col + 32 > g.n) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (col + j >= g.n) v[j] = 0.f;
        }
      };
      auto release_shared = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) remote_arrive(leader_tover + (uint32_t)(acc * sizeof(uint64_t)));
      };
      // A warp's staged block (32 rows x 64 bytes) goes to column `col` of the result.  TMA
      // stores clip at 16 bytes, not at an entry, so a block that ends inside 16 bytes of
      // the result's last columns (and rows that TMA cannot address) is written by the warp,
      // two bytes per lane.
      auto stage_begin = [&]() {
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
      };
      const int esz = g.out == kF8OutBf16 ? 2 : g.out == kF8OutF32 ? 4 : 1;
      const bool tma_ok = g.out == kF8OutCodes || g.d.vec;
      auto stage_store = [&](int col) {
        const int valid = min(64, (g.n - col) * esz);
        if (tma_ok && (valid & 15) == 0) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.map_d[tl.gi], smem_u32(blk), col, row0);
            bulk_commit();
          }
          return;
        }
        __syncwarp();
        uint8_t* dst = g.out == kF8OutCodes ? g.d8.codes + (int64_t)row0 * g.d8.ld + col
                                            : reinterpret_cast<uint8_t*>(g.d.data) + ((int64_t)row0 * g.d.ld + col) * esz;
        const int64_t pitch = g.out == kF8OutCodes ? g.d8.ld : g.d.ld * esz;
        const int off = 2 * lane;
        for (int r = 0; r < 32 && row0 + r < g.m; ++r) {
          const uint16_t x = *reinterpret_cast<const uint16_t*>(blk + r * 64 + ((((off >> 4) ^ (r >> 1)) & 3) << 4) + (off & 15));
          uint8_t* d = dst + r * pitch + off;
          if (off + 2 <= valid) *reinterpret_cast<uint16_t*>(d) = x;
          else if (off < valid) *d = (uint8_t)x;
        }
        __syncwarp();
      };

      if (shared_c >= 0 && shared_c >= chunks) release_shared();
      if (g.out != kF8OutCodes) {
        for (int k = 0; k < 4; ++k) {
          const int c = shared_c == 3 ? (k + 3) & 3 : k;
          if (c >= chunks) continue;
          float v[32];
          tmem_ld32(tbase + (uint32_t)(32 * c), v);
          if (c == shared_c) release_shared();
          finish(c, v);
          const int col = col0 + 32 * c;
          if (g.out == kF8OutBf16) {
            stage_begin();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 x;
              __nv_bfloat162* hh = reinterpret_cast<__nv_bfloat162*>(&x);
#pragma unroll
              for (int e = 0; e < 4; ++e) hh[e] = __floats2bfloat162_rn(v[8 * q + 2 * e], v[8 * q + 2 * e + 1]);
              stage16(blk, lane, q, x);
            }
            stage_store(col);
          } else {
#pragma unroll
            for (int hcol = 0; hcol < 2; ++hcol) {
              if (col + 16 * hcol >= g.n) break;
              stage_begin();
#pragma unroll
              for (int q = 0; q < 4; ++q)
                stage16(blk, lane, q,
                        make_uint4(__float_as_uint(v[16 * hcol + 4 * q]), __float_as_uint(v[16 * hcol + 4 * q + 1]),
                                   __float_as_uint(v[16 * hcol + 4 * q + 2]), __float_as_uint(v[16 * hcol + 4 * q + 3])));
              stage_store(col + 16 * hcol);
            }
          }
        }
      } else {
        // first reading: the maximum; the shared chunk stays in registers, finished
        float keep[32];
        float vmax = 0.f;
        for (int k = 0; k < 4; ++k) {
          const int c = shared_c == 3 ? (k + 3) & 3 : k;
          if (c >= chunks) continue;
          float v[32];
          tmem_ld32(tbase + (uint32_t)(32 * c), v);
          if (c == shared_c) release_shared();
          finish(c, v);
          if (live) {
#pragma unroll
            for (int j = 0; j < 32; ++j) vmax = fmaxf(vmax, fabsf(v[j]));
          }
          if (c == shared_c) {
#pragma unroll
            for (int j = 0; j < 32; ++j) keep[j] = v[j];
          }
        }
        // value of chunk c again
        auto again = [&](int c, float* v) {
          if (c == shared_c) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = keep[j];
          } else {
            tmem_ld32(tbase + (uint32_t)(32 * c), v);
            finish(c, v);
          }
        };
        // maximum over the block: row blocks are this thread's own row
        auto block_max = [&](float m, bool& good) {
          if (g.d8.row_blocks) return m;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          float* slot = max_slot + (max_turn & 1) * 8 + half * 4;
          if (lane == 0) {
            slot[quad] = m;
            mbar_arrive(&max_bar[half]);
          }
          good = warp_wait(&max_bar[half], max_turn & 1u);
          ++max_turn;
          volatile float* s = slot;
          return fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
        };
        bool good = true;
        float amax = block_max(vmax, good);
        if (!good) { ok = false; break; }
        bool inf = amax == kF8Inf;
        const bool any_inf = __any_sync(0xffffffffu, inf);
        if (any_inf) {  // once more over finite entries
          vmax = 0.f;
          for (int c = 0; c < chunks; ++c) {
            float v[32];
            again(c, v);
            if (live) {
#pragma unroll
              for (int j = 0; j < 32; ++j) vmax = fmaxf(vmax, f8_finite_abs(v[j]));
            }
          }
          amax = block_max(vmax, good);
          if (!good) { ok = false; break; }
        }
        const bool e5m2 = g.d8.e5m2;
        const int e = f8_exponent(amax, e5m2);
        const float inv = f8_exp2(-e);
        if (g.d8.row_blocks) {
          if (live && col0 < g.n) *f8_scale_at(g.d8, row, col0 / kFp8Block) = (uint8_t)(e + 127);
        } else if (quad == 0 && lane == 0 && live && col0 < g.n) {
          *f8_scale_at(g.d8, row, col0 / kFp8Block) = (uint8_t)(e + 127);
        }
        for (int c = 0; c < chunks; ++c) {
          float v[32];
          again(c, v);
          if ((c & 1) == 0) stage_begin();
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint2 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* vv = v + 16 * q + 8 * i;
              if (e5m2) {
                x[i] = f8_encode8<true>(vv, inv);
                if (any_inf) x[i] = f8_encode_inf8<true>(vv, x[i]);
              } else {
                x[i] = f8_encode8<false>(vv, inv);
                if (any_inf) x[i] = f8_encode_inf8<false>(vv, x[i]);
              }
            }
            stage16(blk, lane, 2 * (c & 1) + q, make_uint4(x[0].x, x[0].y, x[1].x, x[1].y));
          }
          if ((c & 1) == 1 || c == chunks - 1) stage_store(col0 + 64 * (c >> 1));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) remote_arrive(leader_tdone + (uint32_t)(acc * sizeof(uint64_t)));
    }
    if (!ok && lane == 0) give_up();
    if (lane == 0) bulk_wait_all();  // this warp's stores are complete and its staging is free
  }

  // both CTAs' MMAs, copies and stores are complete before either frees tensor memory or exits
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <typename Params>
cudaError_t launch_pair(const Params& p, int clusters, cudaStream_t st) {
  if (p.total_tiles == 0) return cudaSuccess;
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit) || bit == 0) {
    e = cudaFuncSetAttribute(fp8_pair_kernel<Params>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * clusters));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp8_pair_kernel<Params>, p);
}

}  // namespace

cudaError_t launch_fp8_gemm_pair(const F8PairParamsN<kF8FewProducts>& p, int clusters, cudaStream_t st) {
  return launch_pair(p, clusters, st);
}
cudaError_t launch_fp8_gemm_pair(const F8PairParamsN<kMaxF8Products>& p, int clusters, cudaStream_t st) {
  return launch_pair(p, clusters, st);
}

}  // namespace muon
