// Block-scaled 8-bit matrix products on tcgen05 (kind::mxf8f6f4):
//
//   D = epi(C + sum_kb 2^(ea + eb) sum_{k in block kb} qa qb)
//
// with one scale exponent per block of 128 along the contraction.  Scales are powers of
// two, so the instruction applies them itself and the sum over all blocks stays in tensor
// memory (fp32); no partial sum passes through registers.  Either operand may be stored
// with its contraction along rows (MN-major): weight and input gradients read the same
// 8-bit copies as the forward pass, untransposed.
//
// This file: one 128 x 128 tile per CTA, for results of few tiles, where latency counts
// (64 x 512 x 512: 5.3 us in a chain of calls, against 6.6 us by the persistent kernel of
// k_fp8_pair.cu and 9.7 us by one 256 x 256 tile per pair, which was not kept).  256 threads:
//   warp 0      TMA producer: ring of 128 x 128 code tiles of A and B (16 KB each)
//   warp 1      tensor memory, MMA issue (one thread)
//   warps 2, 3  scale words of both operands, one set per 512 codes, four sets in flight
//   all         epilogue: the fp32 tile goes through shared memory (the ring's space), then
//               half a warp per row finishes 8 columns per thread, as the block passes do
// With few tiles and a long contraction a cluster of 2 or 4 CTAs splits it: every CTA leaves
// its partial tile in its shared memory, and each finishes its share of the rows, adding the
// partial sums in rank order through distributed shared memory.  No workspace, no atomics,
// one launch, the same sums every time (2048 x 512 x 16384: 30.8 us whole, 20.7 us split in
// two; bound by shared memory, which would have to move 256 bytes per clock at the tensor
// rate).
//
// The tensor cores truncate as they accumulate, so the error grows with the length of a sum:
// 2.2e-7 of the result's norm over 4096, 1.2e-6 over 16384.  With the whole tensor memory at
// hand a CTA's share of the contraction goes to up to three accumulators, one per 2048, one after
// another, which the epilogue adds.  A float32 result may sum 4096 at most in one of them: where
// its share is longer than three of these (SEG), the three take segments of 4096 in turn, and the
// warps without a part in the loop above add each to a sum in registers while the next one runs.
//
// Every mbarrier wait is bounded; on expiry the kernel writes kDevTimeout to the status
// word, lets its copies and MMAs drain, frees tensor memory and returns.
#include "fp8_blocks.cuh"
#include "fp8_tc.cuh"

namespace muon {
namespace {

constexpr int kT = 128;  // rows of A and of B that a CTA holds
constexpr int kTThreads = 256;
constexpr uint32_t kTOperand = kT * kF8K;  // 16 KB
constexpr uint32_t kTStageBytes = 2 * kTOperand;
constexpr int kTMaxStages = 6;
constexpr int kTSfSets = 4;  // in shared memory; two in tensor memory

constexpr uint32_t kTSfSet = 2 * kF8SfBytes;   // A words, B words
// tensor memory: accumulators (one, or three where a CTA has an SM), then two sets of 8 columns
// of scales
constexpr int kTAccs = kF8TileAccs;
__device__ __forceinline__ uint32_t tile_tmem_cols(int accs) { return accs > 1 ? 512u : 256u; }
constexpr int kTPitch = kT + 4;                // floats per staged row
static_assert(kT * kTPitch * 4 <= 3 * (int)kTStageBytes, "the staged tile reuses the ring");
constexpr uint32_t tile_smem(int stages) {
  return (uint32_t)stages * kTStageBytes + kTSfSets * kTSfSet + kF8SlopeTable * 4 + 512 + 1024;
}
// one CTA of six stages per SM, or two of three
static_assert(tile_smem(kTMaxStages) <= 232448 && 2 * (tile_smem(3) + 1024) <= 233472, "shared memory");

__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// What follows the sum, for N groups of 8 consecutive entries at (row0 + i * step, col):
// addend, activation or its gradient.
template <int N>
__device__ __forceinline__ void f8_finish(const F8Product& g, const float* slope, int row0, int step, int row_end, int col,
                                          float (&v)[N][8]) {
  if (g.c.data != nullptr) {
    float c[N][8];
    f8_load_rows<N>(g.c, row0, step, row_end, col, g.n, c);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += c[i][j];
  }
  if (g.epi == kF8EpiRelu2) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = f8_relu2(v[i][j]);
  } else if (g.epi == kF8EpiRelu2Backward) {
    f8_times_slope<N>(g.saved, slope, row0, step, row_end, col, g.n, v);
  }
}

// Sum over a cluster's partial tiles, in rank order, of 8 columns at `addr` in each (all
// loads are issued before the first addition).
template <int S>
__device__ __forceinline__ void fetch_split(uint32_t addr, float* v) {
  float4 a[S], b[S];
#pragma unroll
  for (int r = 0; r < S; ++r) {
    const uint32_t at = peer_addr(addr, (uint32_t)r);
    a[r] = ld_cluster_f4(at);
    b[r] = ld_cluster_f4(at + 16);
  }
  v[0] = a[0].x; v[1] = a[0].y; v[2] = a[0].z; v[3] = a[0].w;
  v[4] = b[0].x; v[5] = b[0].y; v[6] = b[0].z; v[7] = b[0].w;
#pragma unroll
  for (int r = 1; r < S; ++r) {
    v[0] += a[r].x; v[1] += a[r].y; v[2] += a[r].z; v[3] += a[r].w;
    v[4] += b[r].x; v[5] += b[r].y; v[6] += b[r].z; v[7] += b[r].w;
  }
}

// SEG: segments as above, one CTA per SM.
template <typename Params, bool SEG>
__global__ void __launch_bounds__(kTThreads, SEG ? 1 : 2) fp8_tile_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t stages = (uint32_t)p.stages;
  uint8_t* sf_smem = smem + stages * kTStageBytes;
  float* slope = reinterpret_cast<float*>(sf_smem + kTSfSets * kTSfSet);
  uint64_t* full = reinterpret_cast<uint64_t*>(slope + kF8SlopeTable);
  uint64_t* empty = full + kTMaxStages;
  uint64_t* sf_full = empty + kTMaxStages;
  uint64_t* sf_empty = sf_full + kTSfSets;
  uint64_t* done = sf_empty + kTSfSets;
  uint64_t* seg_full = done + 1;            // [kTAccs] a segment is summed
  uint64_t* seg_free = seg_full + kTAccs;   // [kTAccs] and has been read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(seg_free + kTAccs);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* cta_max = reinterpret_cast<float*>(tmem_slot + 2);  // this CTA's maximum
  float* warp_max = cta_max + 1;                             // [8]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = (int)cluster_size();
  const int rank = (int)cluster_rank();
  const int tile = blockIdx.x / split;
  int gi = 0;
  while (gi + 1 < p.n && p.p[gi + 1].tile_begin <= tile) ++gi;
  const F8Product& g = p.p[gi];
  const int local = tile - g.tile_begin;
  const int tm = local % g.tiles_m, tn = local / g.tiles_m;
  const int row_t = tm * kT, col_t = tn * kT;
  const int nkb_all = (g.k + kF8K - 1) / kF8K;
  const int per = (nkb_all + split - 1) / split;
  const int kb_begin = min(nkb_all, rank * per), nkb = min(nkb_all, kb_begin + per) - kb_begin;
  // accumulators: all that fit, those used, and the k-blocks of each
  const int accs = SEG || stages == kTMaxStages ? kTAccs : 1;
  const int acc_used = min(accs, (nkb + 15) / 16);
  const int acc_kb = acc_used > 0 ? (nkb + acc_used - 1) / acc_used : 0;

  if (g.epi == kF8EpiRelu2Backward) f8_slope_init(slope, g.saved.e5m2, threadIdx.x, kTThreads);
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kTSfSets; ++s) {
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_empty[s], 1);
    }
    mbar_init(done, 1);
    for (int a = 0; SEG && a < kTAccs; ++a) {
      mbar_init(&seg_full[a], 1);
      mbar_init(&seg_free[a], 4);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x == 0 && nkb > 0) {
    prefetch_map(&p.map_a[gi]);
    prefetch_map(&p.map_b[gi]);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(tile_tmem_cols(accs))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  f8_grid_wait();

  auto give_up = [&]() {
    f8_record_timeout(p.status);
    *abort_flag = 1;
  };

  if (warp == 0) {
    if (elect_one()) {
      const CUtensorMap* ma = &p.map_a[gi];
      const CUtensorMap* mb = &p.map_b[gi];
      const uint32_t ring = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty);
      const int k0 = kb_begin * kF8K;
      int ax = g.a_mn ? row_t : k0, ay = g.a_mn ? k0 : row_t, bx = g.b_mn ? col_t : k0, by = g.b_mn ? k0 : col_t;
      const int adx = g.a_mn ? 0 : kF8K, ady = g.a_mn ? kF8K : 0, bdx = g.b_mn ? 0 : kF8K, bdy = g.b_mn ? kF8K : 0;
      uint32_t stage = 0, phase = 0;
      int issued = 0;
      bool ok = true;
      for (; issued < nkb; ++issued) {
        if (!bar_wait(empty0 + 8 * stage, phase ^ 1u, abort_flag)) { ok = false; break; }
        const uint32_t a_dst = ring + stage * kTStageBytes;
        expect_tx_at(full0 + 8 * stage, kTStageBytes);
        tma_load_2d_local(a_dst, ma, &full[stage], ax, ay);
        tma_load_2d_local(a_dst + kTOperand, mb, &full[stage], bx, by);
        ax += adx; ay += ady; bx += bdx; by += bdy;
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (!ok || *abort_flag) {
        give_up();
        spin_ns(kAbortGraceNs);  // copies already issued land within microseconds
      }
      // (without an abort the issuing thread has seen every copy land before `done`)
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = f8_idesc(g.a_e5m2, g.b_e5m2, g.a_mn, g.b_mn, kT, kT);
      const uint32_t a_step = (g.a_mn ? 4096 : 32) >> 4, b_step = (g.b_mn ? 4096 : 32) >> 4;
      const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty);
      const uint32_t sf_full0 = smem_u32(sf_full), sf_empty0 = smem_u32(sf_empty);
      const uint64_t ring_desc = sdesc(smem_u32(smem), 16, 1024);
      const uint64_t sf_desc = f8_sf_desc(smem_u32(sf_smem));
      uint32_t stage = 0, phase = 0, set = 0, sf_phase = 0, accumulate = 0;
      uint32_t d_tmem = tmem;
      int acc_left = acc_kb;
      uint32_t seg_acc = 0, seg_phase = 1;
      bool ok = true;
      for (int kb = 0; kb < nkb && ok; kb += kF8Group) {
        if (SEG && kb % kF8SegmentBlocks == 0) {
          if (!bar_wait(smem_u32(&seg_free[seg_acc]), seg_phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          d_tmem = tmem + 128 * seg_acc;
          accumulate = 0;
        }
        // copies and products run in the order of their issue, so the two sets in tensor memory
        // need no barrier of their own
        const uint32_t sfa = tmem + 128u * accs + (set & 1u) * 8, sfb = sfa + 4;
        if (!bar_wait(sf_full0 + 8 * set, sf_phase, abort_flag)) { ok = false; break; }
        const uint64_t src = sf_desc + (uint64_t)(set * (kTSfSet >> 4));
        f8_copy_sf(sfa, src);
        f8_copy_sf(sfb, src + (kF8SfBytes >> 4));
        const int n = min(kF8Group, nkb - kb);
#pragma unroll 1
        for (int q = 0; q < n; ++q) {
          if (!bar_wait(full0 + 8 * stage, phase, abort_flag)) { ok = false; break; }
          const uint64_t ad = ring_desc + (uint64_t)(stage * (kTStageBytes >> 4)), bd = ad + (kTOperand >> 4);
          const uint32_t id = f8_idesc_sf(idesc, q);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            f8_mma(d_tmem, ad + k * a_step, bd + k * b_step, id, sfa, sfb, k ? 1u : accumulate);
          accumulate = 1;
          if (!SEG && --acc_left == 0) {  // on to the next accumulator
            d_tmem += 128;
            accumulate = 0;
            acc_left = acc_kb;
          }
          f8_commit_at(empty0 + 8 * stage);
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        if (SEG && ok && ((kb + kF8Group) % kF8SegmentBlocks == 0 || kb + kF8Group >= nkb)) {
          f8_commit_at(smem_u32(&seg_full[seg_acc]));
          if (++seg_acc == kTAccs) { seg_acc = 0; seg_phase ^= 1u; }
        }
        f8_commit_at(sf_empty0 + 8 * set);
        if (++set == kTSfSets) { set = 0; sf_phase ^= 1u; }
      }
      if (!ok) give_up();
      f8_commit_at(smem_u32(done));  // arrives once everything issued here is complete
    }
  } else if (warp < 4) {
    // warps 2 and 3 take the groups of 512 codes in turn
    const int groups = (nkb + kF8Group - 1) / kF8Group;
    uint32_t set = warp - 2, phase = 1;
    for (int i = warp - 2; i < groups; i += 2) {
      const int kb = kb_begin + i * kF8Group;
      const F8SfWords wa = f8_sf_load(g.sa, row_t, g.m, kb, nkb_all, lane);
      const F8SfWords wb = f8_sf_load(g.sb, col_t, g.n, kb, nkb_all, lane);
      int ok = 1;
      if (lane == 0) ok = bar_wait(smem_u32(&sf_empty[set]), phase, abort_flag);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) give_up();
        break;
      }
      uint8_t* dst = sf_smem + set * kTSfSet;
      f8_sf_store(dst, wa, lane);
      f8_sf_store(dst + kF8SfBytes, wb, lane);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sf_full[set]);
      if ((set += 2) >= kTSfSets) { set = warp - 2; phase ^= 1u; }
    }
  }

  // warps 4 to 7: the segments' sum of row 32 (warp % 4) + lane
  float part[SEG ? 4 : 1][32];
  if constexpr (SEG) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) part[c][j] = 0.f;
    if (warp >= 4) {
      uint32_t acc = 0, phase = 0;
      for (int seg = 0; seg < nkb; seg += kF8SegmentBlocks) {
        int ok = 1;
        if (lane == 0) ok = bar_wait(smem_u32(&seg_full[acc]), phase, abort_flag);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) give_up();
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 128u * acc + 32u * c, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) part[c][j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_free[acc]);
        if (++acc == kTAccs) { acc = 0; phase ^= 1u; }
      }
    }
  }

  // the accumulator is final and the ring free once `done` completes
  if (lane == 0) (void)bar_wait(smem_u32(done), 0, nullptr);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  float* stage_f = reinterpret_cast<float*>(smem);
  if constexpr (SEG) {
    if (warp >= 4) {
      float* dst = stage_f + (32 * (warp & 3) + lane) * kTPitch;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(dst + 32 * c + 4 * j) =
              make_float4(part[c][4 * j], part[c][4 * j + 1], part[c][4 * j + 2], part[c][4 * j + 3]);
    }
  } else {
    const int quad = warp & 3, side = warp >> 2;
    constexpr int kChunks = 2;  // 32 columns each
    float* dst = stage_f + (32 * quad + lane) * kTPitch + 32 * kChunks * side;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float v[32];
      if (nkb > 0) {
        const uint32_t at = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(32 * kChunks * side + 32 * c);
        tmem_ld32(at, v);
        for (int a = 1; a * acc_kb < nkb; ++a) {
          float w[32];
          tmem_ld32(at + 128u * a, w);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += w[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(dst + 32 * c + 4 * j) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (split > 1) cluster_sync_all();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(tile_tmem_cols(accs)) : "memory");
  }

  // rows rank * 128/split ... of the tile; 16 threads x 8 columns per row
  const int rows_here = kT / split;
  const int iters = rows_here / 16;
  const int cl = (threadIdx.x & 15) * 8;
  const uint32_t stage_addr = smem_u32(stage_f);
  auto fetch = [&](int rl, float* v) {  // row rl of the tile
    if (split == 1) {
      const float4* q = reinterpret_cast<const float4*>(stage_f + rl * kTPitch + cl);
      const float4 a = q[0], b = q[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else if (split == 2) {
      fetch_split<2>(stage_addr + (uint32_t)(rl * kTPitch + cl) * 4, v);
    } else {
      fetch_split<4>(stage_addr + (uint32_t)(rl * kTPitch + cl) * 4, v);
    }
  };

  // rows of this CTA end at row_end
  const int row0 = row_t + rank * rows_here + (threadIdx.x >> 4);
  const int row_end = min(g.m, row_t + (rank + 1) * rows_here);
  const int col = col_t + cl;
  if (g.d8.codes == nullptr) {
    for (int i = 0; i < iters; ++i) {
      const int row = row0 + 16 * i;
      float v[1][8];
      fetch(row - row_t, v[0]);
      f8_finish<1>(g, slope, row, 16, row_end, col, v);
      if (g.d.vec) {
        if (row < row_end && col < g.n) f8_store8(g.d, row, col, g.n, v[0]);
      } else {  // through this CTA's own row of the staged tile, which no peer reads
        f8_store_rows_xch<1>(g.d, row, 16, row_end, col, g.n, v, stage_f + (row - row_t) * kTPitch);
      }
    }
  } else {
    // finished values go back to this CTA's own rows of the staged tile (no peer reads
    // those), a few rows per thread at a time, until the block's maximum is known
    auto put = [&](int rl, const float* v) {
      float4* q = reinterpret_cast<float4*>(stage_f + rl * kTPitch + cl);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    };
    auto get = [&](int rl, float* v) {
      const float4* q = reinterpret_cast<const float4*>(stage_f + rl * kTPitch + cl);
      const float4 x = q[0], y = q[1];
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    };
    constexpr int kC = 2;
    float vmax = 0.f;
    for (int i0 = 0; i0 < iters; i0 += kC) {
      float v[kC][8], rmax[kC];
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const int row = row0 + 16 * (i0 + i);
        if (row < row_end && col < g.n) {
          fetch(row - row_t, v[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j >= g.n) v[i][j] = 0.f;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        }
      }
      f8_finish<kC>(g, slope, row0 + 16 * i0, 16, row_end, col, v);
      if (g.d8.row_blocks) {
        f8_quantize_rows<kC>(g.d8, row0 + 16 * i0, 16, row_end, col, g.n, v);
      } else {
        f8_row_max<kC>(v, rmax);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          vmax = fmaxf(vmax, rmax[i]);
          if (row0 + 16 * (i0 + i) < row_end) put(row0 + 16 * (i0 + i) - row_t, v[i]);
        }
      }
    }
    if (!g.d8.row_blocks) {
      // maximum over the tile, then over the cluster
      auto tile_max = [&](float m) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        __syncthreads();
        if (lane == 0) warp_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kTThreads / 32; ++w) m = fmaxf(m, warp_max[w]);
        if (split > 1) {
          if (threadIdx.x == 0) *cta_max = m;
          __syncwarp();
          cluster_sync_all();
          for (int r = 0; r < split; ++r) m = fmaxf(m, ld_cluster_f1(peer_addr(smem_u32(cta_max), (uint32_t)r)));
          __syncwarp();
          cluster_sync_all();  // read everywhere before it is written again
        }
        return m;
      };
      float amax = tile_max(vmax);
      const bool inf = amax == kF8Inf;
      if (inf) {  // once more over finite entries
        vmax = 0.f;
        for (int i = 0; i < iters; ++i)
          if (row0 + 16 * i < row_end) {
            float v[8];
            get(row0 + 16 * i - row_t, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) vmax = fmaxf(vmax, f8_finite_abs(v[j]));
          }
        amax = tile_max(vmax);
      }
      const int e = f8_exponent(amax, g.d8.e5m2);
      if (threadIdx.x == 0 && rank == 0) *f8_scale_at(g.d8, row_t, tn) = (uint8_t)(e + 127);
      const float inv[1] = {f8_exp2(-e)};
      for (int i = 0; i < iters; ++i)
        if (row0 + 16 * i < row_end) {
          float v[1][8];
          get(row0 + 16 * i - row_t, v[0]);
          f8_store_rows<1>(g.d8, row0 + 16 * i, 16, row_end, col, g.n, v, inv, inf);
        }
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync_all();  // peers have read this CTA's partial tile and maxima
}

__global__ void fp8_wait_selftest_kernel(int* status, long long limit_clocks) {
  __shared__ uint64_t bar;
  mbar_init(&bar, 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  if (!bar_wait_slow(smem_u32(&bar), 0, nullptr, limit_clocks)) f8_record_timeout(status);
}

template <bool SEG, typename Params>
cudaError_t launch_tile(const Params& p, int split, cudaStream_t st) {
  if (p.total_tiles == 0) return cudaSuccess;
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e =
      f8_allow_smem(reinterpret_cast<const void*>(fp8_tile_kernel<Params, SEG>), tile_smem(kTMaxStages), ready);
  if (e != cudaSuccess) return e;
  return f8_launch(fp8_tile_kernel<Params, SEG>, p, p.total_tiles * split, kTThreads, tile_smem(p.stages), split, st);
}

}  // namespace

cudaError_t launch_fp8_wait_selftest(int* status, long long limit_clocks, cudaStream_t st) {
  fp8_wait_selftest_kernel<<<1, 1, 0, st>>>(status, limit_clocks);
  return cudaGetLastError();
}

cudaError_t launch_fp8_gemm_tile(const F8GemmParamsN<kF8FewProducts>& p, int split, bool segments, cudaStream_t st) {
  return segments ? launch_tile<true>(p, split, st) : launch_tile<false>(p, split, st);
}
cudaError_t launch_fp8_gemm_tile(const F8GemmParamsN<kMaxF8Products>& p, int split, bool segments, cudaStream_t st) {
  return segments ? launch_tile<true>(p, split, st) : launch_tile<false>(p, split, st);
}

}  // namespace muon
