// Block-scaled 8-bit products, 256 x 256 tiles by pairs of CTAs (tcgen05 cta_group::2), for
// results of many tiles.  The formula and the forms are those of k_fp8_gemm.cu.
//
// What bounds these products is the operands' way into and out of shared memory. Per k-block of
// 512 tensor clocks a CTA's share of a 256 x 256 tile writes 32 KB (TMA) and reads 32 KB (MMA),
// 128 B/clk, all that a shared memory moves; a 128 x 128 tile per CTA needs twice that and stops
// at 1.8 PFLOP/s. 16384 x 12288 x 4096 takes 606-640 us (2.6-2.7 PFLOP/s, the chip at its power
// limit), 481 us without copies and epilogue. Not faster: 256 x 224 tiles with two whole
// accumulators (687 us) and 256 x 384 tiles as instructions of 256 and 128 columns (647 us),
// which read A twice.
//
// Per CTA (384 threads, persistent over the pair's share of the tiles):
//   warp 0       TMA producer: 6-stage ring of 128 x 128 code tiles of A (this CTA's rows) and
//                B (this CTA's half of the columns); both CTAs' copies complete on the
//                leader's barrier
//   warp 1       tensor memory; in the leader the MMA issue (one thread)
//   warps 2, 3   scale words: this CTA's 128 rows of A, all 256 columns of B, per 512 codes
//   warps 4..11  epilogue of this CTA's 128 x 256 half, two warps per lane quadrant, each with
//                a 128 x 128 block's worth of columns: exactly one scale block of an 8-bit
//                result.  A thread holds 32 consecutive entries of a row and stores them as
//                whole 32-byte sectors.
//
// Tensor memory holds two accumulators that share 32 columns, [0, 256) and [224, 480), and two
// sets of scales in the rest: 512 columns have no room for two whole accumulators and scales.
// The epilogue reads the shared columns first and hands them over; the next tile's MMAs start
// then and overlap the rest of the epilogue. 8192 x 6144 takes 4.3 us per k-block (11 rounds of
// tiles) and 16 us whatever its contraction: 6 us of these go without the epilogue (4 of them
// the stores), the rest are launch, handing over and the last round. Handing the columns over
// unread changes nothing.
//
// An 8-bit result needs its block's maximum before the first code: the four warps of a block
// read the accumulator twice (maximum; codes). The shared columns wait in shared memory for the
// second reading, the others in tensor memory, finished values in the place of sums. The
// backward epilogue's checkpoint block comes by TMA, requested a tile ahead (its lookups took
// 132 us per 8192 x 6144 x 1536 product with loads one chunk ahead and the shared columns in
// registers).
// The tensor cores truncate as they accumulate (1.2e-6 of the result's norm over 16384). A
// float32 result sums at most 4096 in tensor memory: a longer contraction goes tile by tile in
// segments, which each epilogue thread adds up in 128 registers; the sum goes back to tensor
// memory for the tile's end, so that nothing there needs the registers (6144 x 1536 x 16384:
// 120-125 us; 144 us when each segment went through the result; bf16, without segments, 113-115 us).
//
// Every wait is bounded, the exchange of the maxima included.
#include <type_traits>

#include "fp8_blocks.cuh"
#include "fp8_tc.cuh"

namespace muon {
namespace {

constexpr int kEpi = 8;
constexpr int kPairThreads = 128 + 32 * kEpi;
constexpr uint32_t kPOperand = 128 * kF8K;            // 16 KB
constexpr uint32_t kPStage = 2 * kPOperand;
constexpr uint32_t kPairTx = 2 * kPStage;
constexpr uint32_t kPSfSet = 3 * kF8SfBytes;          // A words, B words of both halves
constexpr int kPSfSets = 4;                           // in shared memory
constexpr uint32_t kOutStage = 1024;                  // 32 rows x 32 bytes per epilogue warp (unaligned rows)
constexpr uint32_t kKeep = 4096;                      // 32 x 32 fp32 of the shared columns, per lane quadrant
constexpr uint32_t kSaved = 4096;                     // 32 x 128 codes of the checkpoint, per epilogue warp

// Shared memory by kind of kernel (OUT, EPI as in the kernel, -1: decided per tile).
template <int OUT, int EPI>
struct PairSmem {
  static constexpr bool kHasKeep = OUT == kF8OutCodes || OUT < 0;
  static constexpr bool kHasSaved = EPI == kF8EpiRelu2Backward;
  static constexpr int kTables = EPI == kF8EpiRelu2Backward ? 1 : EPI < 0 ? 2 : 0;  // e4m3, e5m2
  static constexpr int kStages = kHasSaved || OUT < 0 ? 5 : 6;
  static constexpr uint32_t saved = kStages * kPStage;
  static constexpr uint32_t keep = saved + (kHasSaved ? kEpi * kSaved : 0);
  static constexpr uint32_t out = keep + (kHasKeep ? 4 * kKeep : 0);
  static constexpr uint32_t sf = out + kEpi * kOutStage;
  static constexpr uint32_t slope = sf + kPSfSets * kPSfSet;
  static constexpr uint32_t bars = slope + kTables * kF8SlopeTable * 4;
  static constexpr uint32_t bytes = bars + 512 + 1024;
  static_assert(bytes <= 232448, "shared memory per CTA");
};
constexpr uint32_t kAccStep = 224;  // first column of accumulator a: 224 a
constexpr uint32_t kPSfCol = 480;
constexpr uint32_t kPSfCols = 12;                     // per set in tensor memory, two sets
static_assert(kPSfSets % 2 == 0, "the scale warps take the sets in turn");
static_assert(kPSfCol + 2 * kPSfCols <= 512, "tensor memory columns");

struct PairTile {
  int gi, row, col, nkb;
  int seg_kb;  // k-blocks of a segment (a multiple of kF8Group, or all)
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
  r.seg_kb = g.seg_kb;
  return r;
}

// 32 bytes to an address that is 32-byte aligned: one whole sector.
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Rows that 16-byte accesses cannot address (and blocks that end inside 16 bytes) go through a
// warp's block in shared memory, 32 rows of 32 bytes, two or four bytes per lane.  Calls, so that the epilogue's loop stays small: with these inlined at every use the
// kernel had 260 KB of code and the epilogue ran at the speed of instruction fetch (18,000
// clocks per tile of 8-bit results in the place of 6,000).
// W: bytes per lane, 4 where every row starts at a multiple of 4 and holds whole words.
// Every load is issued before the first use (4001 x 1111 x 2000 into float32: 26.6 us; two bytes
// at a time, each stored as it was read, 38.7 us; 4000 x 1112, aligned, 21.2 us).
template <int W>
__device__ __noinline__ void rows_from_block(const uint8_t* blk, uint8_t* dst, int64_t pitch, int valid, int rows) {
  using T = std::conditional_t<W == 4, uint32_t, uint16_t>;
  const int lane = threadIdx.x & 31, off = W * (lane & (32 / W - 1)), first = lane / (32 / W);
  T x[32 / W];
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32 / W; ++i) {
    const int r = first + W * i;
    x[i] = *reinterpret_cast<const T*>(blk + r * 32 + ((off & 16) ^ ((r & 4) << 2)) + (off & 15));
  }
  __syncwarp();
  uint8_t* d = dst + first * pitch + off;
#pragma unroll
  for (int i = 0; i < 32 / W; ++i, d += W * pitch) {
    if (first + W * i >= rows) break;
    if (off + W <= valid) *reinterpret_cast<T*>(d) = x[i];
    else if (W == 2 && off < valid) *d = (uint8_t)x[i];
  }
}
template <int W>
__device__ __noinline__ void rows_to_block(uint8_t* blk, const uint8_t* src, int64_t pitch, int valid, int rows) {
  using T = std::conditional_t<W == 4, uint32_t, uint16_t>;
  const int lane = threadIdx.x & 31, off = W * (lane & (32 / W - 1)), first = lane / (32 / W);
  T x[32 / W];
  const uint8_t* q = src + first * pitch + off;
#pragma unroll
  for (int i = 0; i < 32 / W; ++i, q += W * pitch)
    x[i] = first + W * i < rows && off + W <= valid ? *reinterpret_cast<const T*>(q) : (T)0;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32 / W; ++i) {
    const int r = first + W * i;
    *reinterpret_cast<T*>(blk + r * 32 + ((off & 16) ^ ((r & 4) << 2)) + (off & 15)) = x[i];
  }
  __syncwarp();
}
// 16 bytes q (0, 1) of row `lane` of such a block.
__device__ __forceinline__ uint4* block16(uint8_t* blk, int lane, int q) {
  return reinterpret_cast<uint4*>(blk + lane * 32 + ((q << 4) ^ ((lane & 4) << 2)));
}
// Infinite values among 8, see f8_encode_inf8.
__device__ __noinline__ uint2 encode_inf8(float4 a, float4 b, uint2 c, bool e5m2) {
  const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  return e5m2 ? f8_encode_inf8<true>(v, c) : f8_encode_inf8<false>(v, c);
}

// The n codes at q (16-byte aligned) that lie before the row's end, at most 16.
__device__ __noinline__ uint4 codes_edge(const uint8_t* q, int n) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < n) w[j >> 2] |= (uint32_t)q[j] << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 32 consecutive entries of this thread's row of the addend (row0 + lane, col ..).
// VEC: whole 32 columns in rows that 16-byte loads can address.
template <bool BF16, bool VEC>
__device__ __forceinline__ void add_c32(const F8Dense& c, uint8_t* blk, int row0, int rows, int col, int cols,
                                        float (&v)[32]) {
  constexpr int kEsz = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(c.data) + ((int64_t)row0 * c.ld + col) * kEsz;
  const int64_t pitch = c.ld * kEsz;
  const bool live = row0 + lane < rows;
#pragma unroll
  for (int i = 0; i < kEsz; ++i) {  // 32 bytes of every row at a time
    const int valid = min(32, (cols - col) * kEsz - 32 * i);
    if (valid <= 0) break;
    uint4 x[2];
    if (VEC || (c.vec && valid == 32)) {
      const uint4* q = reinterpret_cast<const uint4*>(src + lane * pitch + 32 * i);
      x[0] = live ? q[0] : make_uint4(0u, 0u, 0u, 0u);
      x[1] = live ? q[1] : make_uint4(0u, 0u, 0u, 0u);
    } else {
      rows_to_block<kEsz>(blk, src + 32 * i, pitch, valid, rows - row0);
      x[0] = *block16(blk, lane, 0);
      x[1] = *block16(blk, lane, 1);
      __syncwarp();
    }
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (BF16) {
        v[16 * i + 2 * j] += __uint_as_float(w[j] << 16);
        v[16 * i + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
      } else {
        v[8 * i + j] += __uint_as_float(w[j]);
      }
    }
  }
}

// OUT, EPI: the launch's kind of result and epilogue where every product has the same, -1
// otherwise (decided per tile).  ADD: 0 where no product has an addend.  SEG: float32 results in
// segments.
template <typename Params, int OUT, int EPI, int ADD, bool SEG>
__global__ void __launch_bounds__(kPairThreads, 1) fp8_pair_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using L = PairSmem<OUT, EPI>;
  constexpr int kPStages8 = L::kStages;
  static_assert(!SEG || (OUT == kF8OutF32 && EPI == kF8EpiNone), "segments");
  uint8_t* sf_smem = smem + L::sf;
  float* slope = reinterpret_cast<float*>(smem + L::slope);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* empty = full + kPStages8;
  uint64_t* sf_full = empty + kPStages8;
  uint64_t* sf_empty = sf_full + kPSfSets;
  uint64_t* tfull = sf_empty + kPSfSets;
  uint64_t* tdone = tfull + 2;   // an accumulator has been read
  uint64_t* tover = tdone + 2;   // its columns shared with the other one have been read
  uint64_t* max_bar = tover + 2; // [2]: maxima of the two blocks
  uint64_t* drain = max_bar + 2;
  uint64_t* saved_bar = drain + 1;  // [kEpi]
  uint64_t* keep_bar = saved_bar + kEpi;  // [4]: a tile's use of a quadrant's kept columns is over
  float* max_slot = reinterpret_cast<float*>(keep_bar + 4);   // [2 turns][2 blocks][4 warps]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(max_slot + 16);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;
  const int n_clusters = gridDim.x >> 1;

  if (L::kTables > 0 && p.backward) {
    f8_slope_init(slope, false, threadIdx.x, kPairThreads);
    if (L::kTables > 1) f8_slope_init(slope + kF8SlopeTable, true, threadIdx.x, kPairThreads);
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
    for (int a = 0; a < kEpi; ++a) mbar_init(&saved_bar[a], 1);
    for (int a = 0; a < 4; ++a) mbar_init(&keep_bar[a], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane < p.n) {
    prefetch_map(&p.map_a[lane]);
    prefetch_map(&p.map_b[lane]);
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
  f8_grid_wait();
  const uint32_t peer_abort = peer_addr(smem_u32((const void*)abort_flag), rank ^ 1u);
  auto give_up = [&]() {
    f8_record_timeout(p.status);
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
          (void)bar_wait(smem_u32(&full[s]), par, nullptr);
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
      for (int t = cluster; t < p.total_tiles && ok; t += n_clusters) {
        const PairTile tl = pair_tile(p, t);
        const F8Product& g = p.p[tl.gi];
        const uint32_t idesc = f8_idesc(g.a_e5m2, g.b_e5m2, g.a_mn, g.b_mn, kF8PairTile, kF8PairTile);
        const uint32_t a_step = (g.a_mn ? 4096 : 32) >> 4, b_step = (g.b_mn ? 4096 : 32) >> 4;
        for (int seg = 0; seg < tl.nkb; seg += tl.seg_kb, ++it) {
          const int acc = it & 1, seg_end = min(tl.nkb, seg + tl.seg_kb);
          if (!bar_wait(smem_u32(&tdone[acc]), (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag) ||
              (it > 0 && !bar_wait(smem_u32(&tover[acc ^ 1]), (uint32_t)(((it - 1) >> 1) & 1), abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem + (uint32_t)acc * kAccStep;
          uint32_t accumulate = 0;
          for (int kb = seg; kb < seg_end; kb += kF8Group) {
            // copies and products run in the order of their issue, so the two sets in tensor
            // memory need no barrier of their own
            const uint32_t sfa = tmem + kPSfCol + (set & 1u) * kPSfCols, sfb = sfa + 4;
            if (!bar_wait(sf_full0 + 8 * set, sf_phase, abort_flag)) { ok = false; break; }
            const uint64_t src = sf_desc + (uint64_t)(set * (kPSfSet >> 4));
            f8_copy_sf_pair(sfa, src);
            f8_copy_sf_pair(sfb, src + (kF8SfBytes >> 4));
            f8_copy_sf_pair(sfb + 4, src + 2 * (kF8SfBytes >> 4));
            const int n = min(kF8Group, seg_end - kb);
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
      }
      if (!ok) give_up();
      umma_commit_local(drain);
      (void)bar_wait(smem_u32(drain), 0, nullptr);
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
        const F8SfWords wa = f8_sf_load(g.sa, tl.row + (int)rank * 128, g.m, kb, tl.nkb, lane);
        const F8SfWords w0 = f8_sf_load(g.sb, tl.col, g.n, kb, tl.nkb, lane);
        const F8SfWords w1 = f8_sf_load(g.sb, tl.col + 128, g.n, kb, tl.nkb, lane);
        int got = 1;
        if (lane == 0) got = bar_wait(smem_u32(&sf_empty[set]), phase, abort_flag);
        got = __shfl_sync(0xffffffffu, got, 0);
        if (!got) {
          if (lane == 0) give_up();
          ok = false;
          break;
        }
        uint8_t* dst = sf_smem + set * kPSfSet;
        f8_sf_store(dst, wa, lane);
        f8_sf_store(dst + kF8SfBytes, w0, lane);
        f8_sf_store(dst + 2 * kF8SfBytes, w1, lane);
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
    uint8_t* blk = smem + L::out + ew * kOutStage;
    uint8_t* keep = smem + L::keep + quad * kKeep;    // the two blocks' warps take turns, tile by tile
    uint8_t* saved = smem + L::saved + ew * kSaved;
    // the checkpoint's 32 rows x 128 codes of this warp's part of tile t
    auto request_block = [&](int t) {
      if (t < p.total_tiles && lane == 0) {
        const PairTile tl = pair_tile(p, t);
        fence_async_smem();
        mbar_arrive_expect_tx(&saved_bar[ew], kSaved);
        tma_load_2d_local(smem_u32(saved), &p.map_saved[tl.gi], &saved_bar[ew], tl.col + 128 * half,
                          tl.row + (int)rank * 128 + 32 * quad);
      }
    };
    if (L::kHasSaved) request_block(cluster);
    const uint32_t leader_tdone = peer_addr(smem_u32(&tdone[0]), 0);
    const uint32_t leader_tover = peer_addr(smem_u32(&tover[0]), 0);
    uint32_t max_turn = 0;
    // one lane waits, so that the warp stays together when a wait runs out
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
      int got = 1;
      if (lane == 0) got = bar_wait(smem_u32(bar), parity, abort_flag);
      got = __shfl_sync(0xffffffffu, got, 0);
      __syncwarp();
      return got != 0;
    };
    int it = 0;  // accumulations so far
    bool ok = true;
    for (int t = cluster; t < p.total_tiles && ok; t += n_clusters, ++it) {
      const PairTile tl = pair_tile(p, t);
      const F8Product& g = p.p[tl.gi];
      const int row0 = tl.row + (int)rank * 128 + 32 * quad, row = row0 + lane;
      const int col0 = tl.col + 128 * half;
      const bool live = row < g.m;
      const int chunks = row0 < g.m ? max(0, min(4, (g.n - col0 + 31) / 32)) : 0;
      // the chunk in the columns shared with the other accumulator, -1 for the other block
      auto shared_chunk = [&](int acc) { return acc == 0 ? (half == 1 ? 3 : -1) : (half == 0 ? 0 : -1); };
      auto columns = [&](int acc) {
        return tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)acc * kAccStep + (uint32_t)(128 * half);
      };
      auto release_shared = [&](int acc) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_tmem_free(leader_tover + (uint32_t)(acc * sizeof(uint64_t)));
      };
      if constexpr (SEG) {
        // the segments before the last one are added up in registers, and their sum to the last
        // one in tensor memory
        float part[4][32] = {};
        for (int seg = tl.seg_kb; ok; seg += tl.seg_kb, ++it) {
          const int acc = it & 1, shared_c = shared_chunk(acc);
          const bool last = seg >= tl.nkb;
          if (!warp_wait(&tfull[acc], (uint32_t)((it >> 1) & 1))) { ok = false; break; }
          tc_fence_after();
          if (!last && shared_c >= 0 && shared_c >= chunks) release_shared(acc);
          auto take = [&](auto chunk) {
            constexpr int c = decltype(chunk)::value;
            if (c >= chunks) return;
            float v[32];
            tmem_ld32(columns(acc) + (uint32_t)(32 * c), v);
            if (last) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += part[c][j];
              tmem_st32(columns(acc) + (uint32_t)(32 * c), v);
            } else {
              if (c == shared_c) release_shared(acc);
#pragma unroll
              for (int j = 0; j < 32; ++j) part[c][j] += v[j];
            }
          };
          if (shared_c != 0) take(std::integral_constant<int, 3>());
          take(std::integral_constant<int, 0>());
          take(std::integral_constant<int, 1>());
          take(std::integral_constant<int, 2>());
          if (shared_c == 0) take(std::integral_constant<int, 3>());
          if (last) break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_tmem_free(leader_tdone + (uint32_t)(acc * sizeof(uint64_t)));
        }
        if (!ok) break;
      }
      const int acc = it & 1;
      const int shared_c = shared_chunk(acc);

      const int out = OUT >= 0 ? OUT : g.out;
      const bool codes_out = out == kF8OutCodes;
      const int epi = EPI >= 0 ? EPI : g.epi;
      const bool backward = epi == kF8EpiRelu2Backward;
      const F8Dense& addend = g.c;
      const bool add = ADD == 0 ? false : addend.data != nullptr;
      const int rot = shared_c == 3 ? 3 : 0;  // the shared chunk comes first

      // the checkpoint's codes of this row: in shared memory, or requested one chunk ahead
      float sv_scale = 0.f;
      const float* table = slope;
      uint4 sv_next[2];
      auto request_saved = [&](auto plain, int c) {  // plain: see `finish`
        if (L::kHasSaved) return;
        const uint8_t* q = g.saved.codes + (int64_t)row * g.saved.ld + col0 + 32 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int left = live ? g.n - (col0 + 32 * c + 16 * i) : 0;
          if (decltype(plain)::value || left <= 0 || left >= 16)
            sv_next[i] = left > 0 ? *reinterpret_cast<const uint4*>(q + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
          else
            sv_next[i] = codes_edge(q + 16 * i, left);
        }
      };
      if (backward) {
        request_saved(std::false_type(), rot);
        const uint32_t sb = live && col0 < g.n ? *f8_scale_at(g.saved, row, col0 / kFp8Block) : 127u;
        const int e = (int)sb - 127, parity = e & 1;
        sv_scale = sb == 255u ? __uint_as_float(0x7fc00000u) : f8_exp2((e - parity) / 2);
        table = slope + (L::kTables > 1 && g.saved.e5m2 ? kF8SlopeTable : 0) + 256 * parity;
      }

      if (!warp_wait(&tfull[acc], (uint32_t)((it >> 1) & 1))) { ok = false; break; }
      if (L::kHasSaved && !warp_wait(&saved_bar[ew], (uint32_t)(it & 1))) { ok = false; break; }
      tc_fence_after();
      const uint32_t tbase = columns(acc);
      if (shared_c >= 0 && shared_c >= chunks) release_shared(acc);

      // addend, activation or its gradient
      // PLAIN: no chunk needs the calls for unaligned rows and edges.  The loops that most
      // tiles take hold no call at all: with the rare paths inside them an 8-bit tile's second
      // reading took 4,500 clocks.
      auto finish = [&](auto plain, int c, float (&v)[32]) {
        constexpr bool PLAIN = decltype(plain)::value;
        const int col = col0 + 32 * c;
        if (add) {
          if (addend.bf16) add_c32<true, PLAIN>(addend, blk, row0, g.m, col, g.n, v);
          else add_c32<false, PLAIN>(addend, blk, row0, g.m, col, g.n, v);
        }
        if (epi == kF8EpiRelu2) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = f8_relu2(v[j]);
        } else if (backward) {
          if (L::kHasSaved) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              sv_next[i] = *reinterpret_cast<const uint4*>(saved + lane * 128 + (((2 * c + i) ^ (lane & 7)) << 4));
          }
          const uint32_t w[8] = {sv_next[0].x, sv_next[0].y, sv_next[0].z, sv_next[0].w,
                                 sv_next[1].x, sv_next[1].y, sv_next[1].z, sv_next[1].w};
          request_saved(plain, (c + 1) & 3);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = __fmul_rn(__fmul_rn(table[(w[j >> 2] >> (8 * (j & 3))) & 255u], sv_scale), v[j]);
        }
      };
      // the sums of chunk c, finished: the first reading of the accumulator
      auto first = [&](auto plain, int c, float (&v)[32]) {
        tmem_ld32(tbase + (uint32_t)(32 * c), v);
        if (c == shared_c) release_shared(acc);
        finish(plain, c, v);
      };
      const bool write_back = epi != kF8EpiNone || add;
      // ... and the second, of 8-bit results
      auto again = [&](int c, float (&v)[32]) {
        if (c == shared_c) {  // the columns may hold the next tile's sums by now
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(keep + lane * 128 + ((q ^ (lane & 7)) << 4));
            v[4 * q] = x.x; v[4 * q + 1] = x.y; v[4 * q + 2] = x.z; v[4 * q + 3] = x.w;
          }
        } else {
          tmem_ld32(tbase + (uint32_t)(32 * c), v);
        }
      };
      // whole chunks in aligned rows
      const bool plain_tile = g.out_align >= 16 && col0 + 32 * chunks <= g.n && (!add || addend.vec);
      float inv = 1.f;
      bool any_inf = false;
      if (codes_out) {
        // largest magnitude; finished values wait for the codes
        auto maximum = [&](auto plain) {
          float vmax = 0.f;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            const int c = (k + rot) & 3;
            if (c >= chunks) {
              if (backward) request_saved(plain, (c + 1) & 3);
              continue;
            }
            float v[32];
            first(plain, c, v);
            if (c == shared_c) {
              // the other block's warp of this quadrant used the space for the tile before
              if (it > 0 && !warp_wait(&keep_bar[quad], (uint32_t)((it - 1) & 1))) {
                ok = false;
                break;
              }
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4*>(keep + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                    make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            } else if (write_back) {
              tmem_st32(tbase + (uint32_t)(32 * c), v);
            }
            if (decltype(plain)::value) {
              float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], fabsf(v[j]));
              vmax = fmaxf(vmax, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
            } else {
              const int lim = g.n - col0 - 32 * c;  // columns that count
#pragma unroll
              for (int j = 0; j < 32; ++j) vmax = fmaxf(vmax, j < lim ? fabsf(v[j]) : 0.f);
            }
          }
          return live ? vmax : 0.f;
        };
        // over the block's four warps; a row block is this thread's own row
        auto over_block = [&](float amax) {
          if (g.d8.row_blocks) return amax;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
          float* slot = max_slot + (max_turn & 1) * 8 + half * 4;
          if (lane == 0) {
            slot[quad] = amax;
            mbar_arrive(&max_bar[half]);
          }
          ok = warp_wait(&max_bar[half], max_turn & 1u) && ok;
          ++max_turn;
          volatile float* sl = slot;
          return fmaxf(fmaxf(sl[0], sl[1]), fmaxf(sl[2], sl[3]));
        };
        float amax = plain_tile ? maximum(std::true_type()) : maximum(std::false_type());
        if (!ok) break;
        if (L::kHasSaved) {  // every lane has read the checkpoint: the next tile's may come
          __syncwarp();
          request_block(t + n_clusters);
        }
        amax = over_block(amax);
        if (!ok) break;
        any_inf = __any_sync(0xffffffffu, amax == kF8Inf);
        if (any_inf) {  // once more over finite entries
          float vmax = 0.f;
#pragma unroll 1
          for (int c = 0; c < chunks; ++c) {
            float v[32];
            again(c, v);
            const int lim = live ? g.n - col0 - 32 * c : 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) vmax = fmaxf(vmax, j < lim ? f8_finite_abs(v[j]) : 0.f);
          }
          amax = over_block(vmax);
          if (!ok) break;
        }
        const int e = f8_exponent(amax, g.d8.e5m2);
        inv = f8_exp2(-e);
        if (live && col0 < g.n && (g.d8.row_blocks || (quad == 0 && lane == 0)))
          *f8_scale_at(g.d8, row, col0 / kFp8Block) = (uint8_t)(e + 127);
      }

      // to the result, 32 columns of this thread's row at a time, 32 bytes a store
      const int parts = codes_out ? 1 : out == kF8OutBf16 ? 2 : 4;
      uint8_t* const out0 = codes_out ? g.d8.codes : reinterpret_cast<uint8_t*>(g.d.data);
      const int64_t pitch = codes_out ? g.d8.ld : 2 * (parts / 2) * g.d.ld;
      uint8_t* const dst0 = out0 + row0 * pitch + (int64_t)col0 * parts;
      auto emit = [&](auto plain, auto e5m2) {
        constexpr bool PLAIN = decltype(plain)::value, E5M2 = decltype(e5m2)::value;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          const int c = (k + rot) & 3;
          if (c >= chunks) {
            if (backward && !codes_out) request_saved(plain, (c + 1) & 3);
            continue;
          }
          float v[32];
          if (codes_out) again(c, v);
          else first(plain, c, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i >= parts) break;
            uint32_t w[8];
            if (parts == 4) {
#pragma unroll
              for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * i + j]);
            } else if (parts == 2) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const __nv_bfloat162 hh = __floats2bfloat162_rn(v[(16 * i + 2 * j) & 31], v[(16 * i + 2 * j + 1) & 31]);
                w[j] = *reinterpret_cast<const uint32_t*>(&hh);
              }
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                uint2 x = f8_encode8<E5M2>(v + 8 * q, inv);
                if (!PLAIN && any_inf)
                  x = encode_inf8(make_float4(v[8 * q], v[8 * q + 1], v[8 * q + 2], v[8 * q + 3]),
                                  make_float4(v[8 * q + 4], v[8 * q + 5], v[8 * q + 6], v[8 * q + 7]), x, E5M2);
                w[2 * q] = x.x;
                w[2 * q + 1] = x.y;
              }
            }
            uint8_t* d = dst0 + (int64_t)(32 * c) * parts + 32 * i;
            const int valid = PLAIN ? 32 : min(32, (g.n - col0 - 32 * c) * parts - 32 * i);
            if (valid <= 0) break;
            if (PLAIN || (valid == 32 && g.out_align >= 16)) {
              d += lane * pitch;
              if (live) {
                if (g.out_align >= 32) {
                  st_global_32b(d, w);
                } else {
                  reinterpret_cast<uint4*>(d)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                  reinterpret_cast<uint4*>(d)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
              }
            } else {
              *block16(blk, lane, 0) = make_uint4(w[0], w[1], w[2], w[3]);
              *block16(blk, lane, 1) = make_uint4(w[4], w[5], w[6], w[7]);
              if (parts == 4) rows_from_block<4>(blk, d, pitch, valid, min(32, g.m - row0));
              else rows_from_block<2>(blk, d, pitch, valid, min(32, g.m - row0));
            }
          }
        }
      };
      if (codes_out && g.d8.e5m2) {
        if (plain_tile && !any_inf) emit(std::true_type(), std::true_type());
        else emit(std::false_type(), std::true_type());
      } else {
        if (plain_tile && !any_inf) emit(std::true_type(), std::false_type());
        else emit(std::false_type(), std::false_type());
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (L::kHasKeep && half == 1 - acc) {
        // Tiles hand the space over in order: a warp that had no use for it (a dense result, or a
        // chunk past the edge) still waits for the tile before. An arrival ahead of the other
        // block's would complete two phases, and the wait for the first of them would not end.
        if (it > 0 && !warp_wait(&keep_bar[quad], (uint32_t)((it - 1) & 1))) { ok = false; break; }
        if (lane == 0) mbar_arrive(&keep_bar[quad]);
      }
      if (lane == 0) arrive_tmem_free(leader_tdone + (uint32_t)(acc * sizeof(uint64_t)));
    }
    if (!ok && lane == 0) {
      give_up();
      if (L::kHasSaved) spin_ns(kAbortGraceNs);  // a requested block lands within microseconds
    }
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

template <typename Params, int OUT, int EPI, int ADD, bool SEG = false>
cudaError_t launch_variant(const Params& p, int clusters, cudaStream_t st) {
  const auto kernel = fp8_pair_kernel<Params, OUT, EPI, ADD, SEG>;
  constexpr uint32_t kSmem = PairSmem<OUT, EPI>::bytes;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = f8_allow_smem(reinterpret_cast<const void*>(kernel), kSmem, ready);
  if (e != cudaSuccess) return e;
  return f8_launch<Params>(kernel, p, 2 * clusters, kPairThreads, kSmem, 2, st);
}

}  // namespace

// The kinds of products that training steps issue have kernels of their own; the rest, and
// launches that mix kinds, take the one that decides per tile.
cudaError_t launch_fp8_gemm_pair(const F8PairParams& p, int clusters, cudaStream_t st) {
  using P = F8PairParams;
  if (p.total_tiles == 0) return cudaSuccess;
  const F8Product& g = p.p[0];
  bool same = true, same_add = true, any_add = false, segments = false;
  for (int i = 0; i < p.n; ++i) {
    const bool add = p.p[i].c.data != nullptr;
    same = same && p.p[i].out == g.out && p.p[i].epi == g.epi;
    same_add = same_add && add == (g.c.data != nullptr);
    any_add = any_add || add;
    segments = segments || p.p[i].seg_kb < (p.p[i].k + kF8K - 1) / kF8K;
  }
  const bool add = g.c.data != nullptr;
  // (the kernels with an addend do without one where a product has none)
  if (same && g.epi == kF8EpiNone && g.out == kF8OutBf16)
    return any_add ? launch_variant<P, kF8OutBf16, kF8EpiNone, 1>(p, clusters, st)
                   : launch_variant<P, kF8OutBf16, kF8EpiNone, 0>(p, clusters, st);
  if (segments) return launch_variant<P, kF8OutF32, kF8EpiNone, -1, true>(p, clusters, st);
  if (same && g.epi == kF8EpiNone && g.out == kF8OutF32)
    return any_add ? launch_variant<P, kF8OutF32, kF8EpiNone, 1>(p, clusters, st)
                   : launch_variant<P, kF8OutF32, kF8EpiNone, 0>(p, clusters, st);
  same = same && same_add;
  if (same && g.out == kF8OutCodes && !add) {
    if (g.epi == kF8EpiNone) return launch_variant<P, kF8OutCodes, kF8EpiNone, 0>(p, clusters, st);
    if (g.epi == kF8EpiRelu2) return launch_variant<P, kF8OutCodes, kF8EpiRelu2, 0>(p, clusters, st);
    bool e4m3 = true;
    for (int i = 0; i < p.n; ++i) e4m3 = e4m3 && !p.p[i].saved.e5m2;
    if (e4m3) return launch_variant<P, kF8OutCodes, kF8EpiRelu2Backward, 0>(p, clusters, st);
  }
  return launch_variant<P, -1, -1, -1>(p, clusters, st);
}

}  // namespace muon
