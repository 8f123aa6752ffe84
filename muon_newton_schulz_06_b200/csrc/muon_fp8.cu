// Host side of the 8-bit operators: argument checks, kernel parameters and tensor maps,
// launches.  Nothing is kept between calls but the handle's status word.
#include <algorithm>
#include <tuple>
#include <vector>

#include <nvtx3/nvToolsExt.h>

#include "fp8_internal.h"
#include "muon_handle.h"

using namespace muon;

namespace {

constexpr int64_t kMaxDim8 = int64_t(1) << 24;
constexpr int kMaxItems = 65535;
// What one launch counts at most; a matrix above is refused before anything is enqueued.
constexpr int64_t kMaxBlocks = INT32_MAX / 2;  // of a pass (up to two CTAs each)
constexpr int64_t kMaxTiles = INT32_MAX / 8;   // of products (up to four CTAs each)

int64_t blocks_of(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }
bool empty(int64_t rows, int64_t cols) { return rows == 0 || cols == 0; }

// rows of `pitch` bytes reach no further than an address space does
bool addressable(int64_t rows, int64_t pitch) { return pitch <= (int64_t(1) << 47) / rows; }

// One buffer of a call as the overlap check sees it: rows x width bytes at pitch.
struct Span {
  uintptr_t lo;
  int64_t rows, width, pitch;  // bytes
  bool written;
  int item;
  uintptr_t hi() const { return lo + (uintptr_t)((rows - 1) * pitch + width); }
};

// Spans of one pitch that interleave without touching (column slices of one tensor). A single row
// has the pitch of the other span.
bool disjoint_columns(const Span& a, const Span& b) {
  if (a.rows < 1 || b.rows < 1 || (a.rows == 1 && b.rows == 1)) return false;
  const int64_t pitch = a.rows == 1 ? b.pitch : a.pitch;
  if (b.rows > 1 && b.pitch != pitch) return false;
  const uint64_t d = (b.lo >= a.lo ? b.lo - a.lo : a.lo - b.lo) % (uint64_t)pitch;
  const int64_t off = b.lo >= a.lo ? (int64_t)d : (d == 0 ? 0 : pitch - (int64_t)d);
  return off >= a.width && off + b.width <= pitch;
}

struct Call {
  muon_handle* h;
  std::vector<Span> spans;
  std::vector<const void*> ptrs;

  void add(const void* p, int64_t rows, int64_t width, int64_t pitch, bool written, int item) {
    ptrs.push_back(p);
    spans.push_back({(uintptr_t)p, rows, width, pitch, written, item});
  }

  muon_status dense(const muon_dense& x, const char* what, int item, bool written) {
    if (x.rows < 0 || x.cols < 0 || x.rows > kMaxDim8 || x.cols > kMaxDim8)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has shape %lld x %lld", item, what, (long long)x.rows,
                  (long long)x.cols);
    if (x.dtype != MUON_F32 && x.dtype != MUON_BF16)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has an unknown dtype", item, what);
    if (empty(x.rows, x.cols)) return MUON_OK;
    const int64_t esz = x.dtype == MUON_BF16 ? 2 : 4;
    if (!x.data) return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s is NULL", item, what);
    if ((uintptr_t)x.data % (uintptr_t)esz)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s is not aligned to its type", item, what);
    if (x.ld < x.cols || x.ld >= (int64_t(1) << 40) || !addressable(x.rows, x.ld * esz))
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has row pitch %lld for %lld columns", item, what,
                  (long long)x.ld, (long long)x.cols);
    add(x.data, x.rows, x.cols * esz, x.ld * esz, written, item);
    return MUON_OK;
  }

  muon_status fp8(const muon_fp8_matrix& x, const char* what, int item, bool written) {
    if (x.rows < 0 || x.cols < 0 || x.rows > kMaxDim8 || x.cols > kMaxDim8)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has shape %lld x %lld", item, what, (long long)x.rows,
                  (long long)x.cols);
    if (x.format != MUON_E4M3 && x.format != MUON_E5M2)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has an unknown format", item, what);
    if (x.blocks != MUON_BLOCK_SQUARE && x.blocks != MUON_BLOCK_ROW)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has an unknown block form", item, what);
    if (empty(x.rows, x.cols)) return MUON_OK;
    if (!x.codes || !x.scales) return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has a NULL pointer", item, what);
    if ((uintptr_t)x.codes & 15u)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has codes that are not 16-byte aligned", item, what);
    if (x.ld < x.cols || x.ld % 16 || x.ld >= (int64_t(1) << 40) || !addressable(x.rows, x.ld))
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: %s has row pitch %lld for %lld columns (a multiple of 16)", item,
                  what, (long long)x.ld, (long long)x.cols);
    const int64_t bc = blocks_of(x.cols);
    const int64_t ns = x.blocks == MUON_BLOCK_SQUARE ? blocks_of(x.rows) * bc : x.rows * bc;
    add(x.codes, x.rows, x.cols, x.ld, written, item);
    add(x.scales, 1, ns, ns, written, item);
    return MUON_OK;
  }

  // No written buffer may overlap another buffer; every pointer is memory of the device.
  muon_status check() {
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) {
      return std::tie(a.lo, a.written, a.rows, a.width, a.pitch) < std::tie(b.lo, b.written, b.rows, b.width, b.pitch);
    });
    // an operand that many items read counts once
    spans.erase(std::unique(spans.begin(), spans.end(),
                            [](const Span& a, const Span& b) {
                              return !a.written && !b.written &&
                                     std::tie(a.lo, a.rows, a.width, a.pitch) == std::tie(b.lo, b.rows, b.width, b.pitch);
                            }),
                spans.end());
    for (size_t i = 0; i < spans.size(); ++i)
      for (size_t j = i + 1; j < spans.size() && spans[j].lo < spans[i].hi(); ++j)
        if ((spans[i].written || spans[j].written) && !disjoint_columns(spans[i], spans[j]))
          return fail(h, MUON_ERR_INVALID_ARG, "buffers of items %d and %d overlap", spans[i].item, spans[j].item);
    for (size_t i = 0; i < ptrs.size(); ++i) {
      cudaPointerAttributes a;
      const cudaError_t e = cudaPointerGetAttributes(&a, ptrs[i]);
      if (e != cudaSuccess) cudaGetLastError();
      if (e != cudaSuccess || (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged) ||
          a.device != h->device)
        return fail(h, MUON_ERR_INVALID_ARG, "pointer %zu of the call (%p) is not device memory of device %d", i,
                    ptrs[i], h->device);
    }
    return MUON_OK;
  }
};

F8Dense kernel_dense(const muon_dense& x) {
  F8Dense d = {};
  d.data = empty(x.rows, x.cols) ? nullptr : x.data;
  d.ld = x.ld;
  d.bf16 = x.dtype == MUON_BF16;
  d.vec = ((uintptr_t)x.data & 15u) == 0 && (x.ld * (d.bf16 ? 2 : 4)) % 16 == 0;
  return d;
}

F8Mat kernel_fp8(const muon_fp8_matrix& x) {
  F8Mat m = {};
  if (empty(x.rows, x.cols)) return m;
  m.codes = static_cast<uint8_t*>(x.codes);
  m.scales = static_cast<uint8_t*>(x.scales);
  m.ld = x.ld;
  m.s_row = (int32_t)blocks_of(x.cols);
  m.s_col = (int32_t)x.rows;
  m.e5m2 = x.format == MUON_E5M2;
  m.row_blocks = x.blocks == MUON_BLOCK_ROW;
  return m;
}

// First call of a handle: the page-locked status word.  Allowed while the
// stream is being captured (no work is enqueued), hence the relaxed capture mode.
muon_status ensure_fp8(muon_handle* h) {
  if (h->fp8_status) return MUON_OK;
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  cudaThreadExchangeStreamCaptureMode(&mode);
  int* word = nullptr;
  cudaError_t e = cudaHostAlloc(&word, sizeof(int), cudaHostAllocMapped | cudaHostAllocPortable);
  if (e == cudaSuccess) {
    *word = kDevOk;
    void* dev = nullptr;
    e = cudaHostGetDevicePointer(&dev, word, 0);
    h->fp8_status_dev = static_cast<int*>(dev);
  }
  cudaThreadExchangeStreamCaptureMode(&mode);
  if (e != cudaSuccess) {
    if (word) cudaFreeHost(word);
    cudaGetLastError();
    return cuda_fail(h, e, "fp8 status set-up");
  }
  h->fp8_status = word;
  return MUON_OK;
}

// The mark for the end of this call's work on `st`, set up before anything is enqueued: that of the
// stream's last call, or one whose work is over, or a new one.  -1 under capture (captured work has
// none to wait for).
muon_status take_mark(muon_handle* h, cudaStream_t st, int* mark) {
  *mark = -1;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  cudaStreamIsCapturing(st, &cs);
  if (cs != cudaStreamCaptureStatusNone) return MUON_OK;
  unsigned long long id = 0;
  cudaError_t e = cudaStreamGetId(st, &id);
  if (e != cudaSuccess) return cuda_fail(h, e, "stream id");
  for (size_t i = 0; i < h->fp8_marks.size(); ++i)
    if (h->fp8_marks[i].stream == id) {
      *mark = (int)i;
      return MUON_OK;
    }
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;  // another stream may be in a capture
  cudaThreadExchangeStreamCaptureMode(&mode);
  for (size_t i = 0; i < h->fp8_marks.size() && *mark < 0; ++i)
    if (!h->fp8_marks[i].pending || cudaEventQuery(h->fp8_marks[i].event) == cudaSuccess) *mark = (int)i;
  cudaThreadExchangeStreamCaptureMode(&mode);
  cudaGetLastError();  // cudaErrorNotReady
  if (*mark < 0) {
    h->fp8_marks.reserve(h->fp8_marks.size() + 1);
    cudaEvent_t event = nullptr;
    if ((e = cudaEventCreateWithFlags(&event, cudaEventDisableTiming)) != cudaSuccess)
      return cuda_fail(h, e, "fp8 event set-up");
    *mark = (int)h->fp8_marks.size();
    h->fp8_marks.push_back({id, event, false});
  }
  h->fp8_marks[*mark].stream = id;
  h->fp8_marks[*mark].pending = false;
  return MUON_OK;
}

// Ends a call whose launches came to `s`: what was enqueued before an error is marked as well.
muon_status finish_fp8(muon_handle* h, cudaStream_t st, int mark, muon_status s) {
  if (mark < 0 || h->last_launches == 0) return s;
  const cudaError_t e = cudaEventRecord(h->fp8_marks[mark].event, st);
  if (e == cudaSuccess) h->fp8_marks[mark].pending = true;
  else if (s == MUON_OK) return cuda_fail(h, e, "fp8 event");
  return s;
}

struct NvtxScope {
  bool on;
  NvtxScope(bool o, const char* name) : on(o) {
    if (on) nvtxRangePushA(name);
  }
  ~NvtxScope() {
    if (on) nvtxRangePop();
  }
};

template <int N>
muon_status launch_passes(muon_handle* h, int op, int kind, const std::vector<F8Pass>& passes, int relu2,
                          cudaStream_t st) {
  F8PassParamsN<N> p;
  p.relu2 = relu2;
  for (size_t b = 0; b < passes.size();) {
    int64_t total = 0;
    p.n = 0;
    for (; b < passes.size() && p.n < N; ++b) {
      const int64_t nb = blocks_of(passes[b].rows) * (int64_t)passes[b].blocks_c;
      if (total + nb > kMaxBlocks) break;  // (one matrix always fits: run_passes)
      F8Pass& m = p.m[p.n++];
      m = passes[b];
      m.block_begin = (int32_t)total;
      total += nb;
    }
    p.total_blocks = (int)total;
    prof_begin(h, st, kFp8KindBase + kind);
    const cudaError_t e = launch_fp8_pass(op, p, st);
    prof_end(h, kFp8KindBase + kind, st);
    if (e != cudaSuccess) return cuda_fail(h, e, "8-bit pass launch");
    h->last_launches++;
  }
  return MUON_OK;
}

// Checks and then runs one list of block passes.
muon_status run_passes(Call& call, int op, int kind, const std::vector<F8Pass>& passes, muon_activation act,
                       cudaStream_t st) {
  muon_handle* h = call.h;
  muon_status s;
  int mark;
  if ((s = call.check())) return s;
  for (const F8Pass& m : passes)
    if (blocks_of(m.rows) * (int64_t)m.blocks_c > kMaxBlocks)
      return fail(h, MUON_ERR_UNSUPPORTED, "a matrix of %d x %d has too many blocks", m.rows, m.cols);
  if ((s = ensure_fp8(h))) return s;
  if ((s = poll_status(h, false, st))) return s;
  if ((s = take_mark(h, st, &mark))) return s;
  h->last_launches = 0;
  const int relu2 = act == MUON_ACT_RELU2;
  s = passes.size() <= kF8FewPasses ? launch_passes<kF8FewPasses>(h, op, kind, passes, relu2, st)
                                    : launch_passes<kMaxF8Passes>(h, op, kind, passes, relu2, st);
  return finish_fp8(h, st, mark, s);
}

F8Pass make_pass(int64_t rows, int64_t cols) {
  F8Pass m = {};
  m.rows = (int32_t)rows;
  m.cols = (int32_t)cols;
  m.blocks_c = (int32_t)blocks_of(cols);
  return m;
}

muon_status check_list(muon_handle* h, int n, const void* a, const void* b) {
  if (n < 0 || n > kMaxItems) return fail(h, MUON_ERR_INVALID_ARG, "n = %d outside 0..%d", n, kMaxItems);
  if (n > 0 && (!a || !b)) return fail(h, MUON_ERR_INVALID_ARG, "NULL array argument");
  return MUON_OK;
}

muon_status check_act(muon_handle* h, muon_activation act) {
  if (act != MUON_ACT_NONE && act != MUON_ACT_RELU2)
    return fail(h, MUON_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  return MUON_OK;
}

bool same_dense(const muon_dense& a, const muon_dense& b) {
  return a.data == b.data && a.ld == b.ld && a.dtype == b.dtype;
}

// ------------------------------------------------------------------ products

muon_status encode_codes(muon_handle* h, CUtensorMap* map, const muon_fp8_matrix& x, int box_rows = kFp8Block) {
  cuuint64_t dims[2] = {(cuuint64_t)x.cols, (cuuint64_t)x.rows};
  cuuint64_t strides[1] = {(cuuint64_t)x.ld};
  cuuint32_t box[2] = {(cuuint32_t)kFp8Block, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = h->encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, x.codes, dims, strides, box, estr,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(h, MUON_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MUON_OK;
}

// Scales of an operand; mn: stored with M / N along its columns (contraction over rows).
F8Scales scales_of(const muon_fp8_matrix& x, bool mn) {
  F8Scales s = {};
  s.s = static_cast<const uint8_t*>(x.scales);
  if (x.blocks == MUON_BLOCK_ROW) {
    s.by_row = 1;
    s.s_r = 1;
    s.s_k = (int32_t)x.rows;
  } else {
    const int32_t bc = (int32_t)blocks_of(x.cols);
    s.s_r = mn ? 1 : bc;
    s.s_k = mn ? bc : 1;
  }
  return s;
}

struct ProductSize {
  int32_t m, n, k;
};
ProductSize size_of(const muon_fp8_product& q) {
  return {(int32_t)(q.trans_a ? q.a.cols : q.a.rows), (int32_t)(q.trans_b ? q.b.rows : q.b.cols),
          (int32_t)(q.trans_a ? q.a.rows : q.a.cols)};
}

// A float32 result without an epilogue sums at most kF8SegmentBlocks k-blocks at a time on the
// tensor cores, wherever it is computed (the others' own rounding is far larger).
bool sums_in_parts(const muon_fp8_product& q) {
  return q.d.data && q.d.dtype == MUON_F32 && q.epilogue == MUON_EPI_NONE;
}
bool long_sum(const muon_fp8_product& q) { return sums_in_parts(q) && blocks_of(size_of(q).k) > kF8SegmentBlocks; }

// Products [b, end) of `live` in one launch: tiles of `tile` rows and columns.
template <typename Params>
muon_status fill_products(muon_handle* h, Params& p, const muon_fp8_product* products, const int* live, int count,
                          int tile, int64_t* total, int64_t* min_kb) {
  p.n = 0;
  p.backward = 0;
  p.status = h->fp8_status_dev;
  *total = 0;
  *min_kb = INT64_MAX;
  for (int i = 0; i < count; ++i) {
    const muon_fp8_product& q = products[live[i]];
    const ProductSize sz = size_of(q);
    F8Product g = {};
    g.m = sz.m;
    g.n = sz.n;
    g.k = sz.k;
    g.tiles_m = (g.m + tile - 1) / tile;
    g.tiles_n = (g.n + tile - 1) / tile;
    g.a_mn = q.trans_a ? 1 : 0;
    g.b_mn = q.trans_b ? 0 : 1;
    g.a_e5m2 = q.a.format == MUON_E5M2;
    g.b_e5m2 = q.b.format == MUON_E5M2;
    g.sa = scales_of(q.a, g.a_mn);
    g.sb = scales_of(q.b, g.b_mn);
    if (q.d.data) g.d = kernel_dense(q.d);
    else g.d8 = kernel_fp8(q.d8);
    g.out = !q.d.data ? kF8OutCodes : q.d.dtype == MUON_BF16 ? kF8OutBf16 : kF8OutF32;
    const uint64_t at = q.d.data ? (uintptr_t)q.d.data | (uint64_t)q.d.ld * (q.d.dtype == MUON_BF16 ? 2 : 4)
                                 : (uintptr_t)q.d8.codes | (uint64_t)q.d8.ld;
    g.out_align = at % 32 == 0 ? 32 : at % 16 == 0 ? 16 : 0;
    if (q.c.data) g.c = kernel_dense(q.c);
    g.epi = (int32_t)q.epilogue;
    g.seg_kb = long_sum(q) ? kF8SegmentBlocks : std::max<int32_t>(1, (int32_t)blocks_of(g.k));
    if (q.epilogue == MUON_EPI_RELU2_BACKWARD) {
      g.saved = kernel_fp8(q.saved);
      p.backward = 1;
    }
    g.tile_begin = (int32_t)*total;
    *total += (int64_t)g.tiles_m * g.tiles_n;
    *min_kb = std::min(*min_kb, blocks_of(g.k));
    muon_status s;
    if (g.k > 0 && ((s = encode_codes(h, &p.map_a[p.n], q.a)) || (s = encode_codes(h, &p.map_b[p.n], q.b)))) return s;
    p.p[p.n++] = g;
  }
  p.total_tiles = (int)*total;
  return MUON_OK;
}

muon_status launch_pair_products(muon_handle* h, const muon_fp8_product* products, const int* live, int count,
                                 cudaStream_t st) {
  F8PairParams p;
  int64_t tiles = 0, min_kb = 0;
  muon_status s = fill_products(h, p, products, live, count, kF8PairTile, &tiles, &min_kb);
  if (s) return s;
  for (int i = 0; i < count; ++i)
    if (p.p[i].epi == kF8EpiRelu2Backward && (s = encode_codes(h, &p.map_saved[i], products[live[i]].saved, 32))) return s;
  prof_begin(h, st, kFp8KindBase + MUON_FP8_KIND_MATMUL);
  const cudaError_t e = launch_fp8_gemm_pair(p, (int)std::min<int64_t>(tiles, h->sm_count / 2), st);
  prof_end(h, kFp8KindBase + MUON_FP8_KIND_MATMUL, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "8-bit product launch");
  h->last_launches++;
  return MUON_OK;
}

// How a run of products is launched.
struct Shape {
  bool persistent = false;  // 256 x 256 tiles by pairs of CTAs that take tile after tile
  int split = 1;            // otherwise a CTA per 128 x 128 tile: CTAs sharing its contraction
  int stages = 6;           // and its ring
};

// tiles: 128 x 128 tiles of all products; min_kb, mean_kb: shortest contraction in blocks of 128,
// and the mean over the tiles.
// Times in a chain of calls on one B200:
//   up to one tile per SM: a CTA per tile (64 x 512 x 512: 5.3 us, persistent 6.6; 1536 x 1536 x
//   4096: 12.6, 16.2), its contraction split while the SMs hold all parts and each keeps 8
//   blocks or more (128 x 1536 x 6144: whole 14.4, in two 10.9, in four 10.0; 2048 x 512 x
//   1024, parts of 4 blocks: whole 7.1, in two 8.0).
//   up to two per SM with short contractions: two CTAs per SM with half the ring (1536 x 2048 x
//   512: 7.6, persistent 8.3; at 2048 x 2048 x 4096: 19.4, 17.3).
//   more: persistent pairs (4096 x 4096 x 1024: 19.7, a CTA per tile 35).
//   Lists go by the mean over their tiles (1024 x 1024 x 128 beside 1280 x 1280 x 8192: pairs 26.5,
//   two CTAs per SM 29.3; 1280 x 1280 x 4096: 17.3, 18.0).
Shape choose_shape(int64_t tiles, int64_t min_kb, int64_t mean_kb, int sm_count) {
  Shape sh;
  if (tiles <= sm_count) {
    while (sh.split < 4 && tiles * sh.split * 2 <= sm_count && min_kb >= 16 * sh.split) sh.split *= 2;
    return sh;
  }
  sh.stages = 3;
  sh.persistent = min_kb > 0 && (tiles > 2 * sm_count || mean_kb >= 16);  // (pairs need a sum to wait for)
  return sh;
}

template <int N>
muon_status launch_tile_products(muon_handle* h, const muon_fp8_product* products, const int* live, int count,
                                 const Shape& sh, cudaStream_t st) {
  F8GemmParamsN<N> p;
  int64_t tiles = 0, min_kb = 0;
  const muon_status s =
      fill_products(h, p, products, live, count, kFp8Block, &tiles, &min_kb);
  if (s) return s;
  p.stages = sh.stages;
  bool segments = false;
  for (int i = 0; i < count; ++i) {
    const muon_fp8_product& q = products[live[i]];
    const int64_t share = (blocks_of(size_of(q).k) + sh.split - 1) / sh.split;
    segments = segments || (sums_in_parts(q) && share > kF8TileAccs * kF8SegmentBlocks);
  }
  prof_begin(h, st, kFp8KindBase + MUON_FP8_KIND_MATMUL);
  const cudaError_t e = launch_fp8_gemm_tile(p, sh.split, segments, st);
  prof_end(h, kFp8KindBase + MUON_FP8_KIND_MATMUL, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "8-bit product launch");
  h->last_launches++;
  return MUON_OK;
}

// The products products[live[..]], in launches of a few.
muon_status launch_run(muon_handle* h, const muon_fp8_product* products, const std::vector<int>& live,
                       cudaStream_t st) {
  for (size_t b = 0; b < live.size();) {
    int count = (int)std::min<size_t>(kMaxF8Products, live.size() - b);
    const int* items = live.data() + b;
    Shape sh;
    while (true) {
      int64_t tiles = 0, min_kb = INT64_MAX, work = 0;
      for (int i = 0; i < count; ++i) {
        const ProductSize z = size_of(products[items[i]]);
        const int64_t t = blocks_of(z.m) * blocks_of(z.n), kb = blocks_of(z.k);
        tiles += t;
        min_kb = std::min(min_kb, kb);
        work += t * kb;
      }
      sh = choose_shape(tiles, min_kb, work / tiles, h->sm_count);
      if (tiles > kMaxTiles) count = (count + 1) / 2;  // (one product always fits: matmul)
      else if (sh.persistent && count > kF8PairProducts) count = kF8PairProducts;
      else break;
    }
    const muon_status s = sh.persistent ? launch_pair_products(h, products, items, count, st)
                          : count <= kF8FewProducts
                              ? launch_tile_products<kF8FewProducts>(h, products, items, count, sh, st)
                              : launch_tile_products<kMaxF8Products>(h, products, items, count, sh, st);
    if (s) return s;
    b += (size_t)count;
  }
  return MUON_OK;
}

// All products of a call (independent of one another, so in any order). Where there are more tiles
// than SMs, the kernels for them sum a contraction in one accumulator or in segments, launch by
// launch, so long float32 sums go in launches of their own; and so do products of nothing, which
// the pairs do not take (128 x 256 x 0 beside 4096 x 4096 x 1024: 26.3 us, by a CTA per tile for
// both 36.8; beside 2560 x 2304 x 640: 16.5, 15.4). Fewer tiles share a launch: a CTA per tile has
// room for every kind.
muon_status launch_products(muon_handle* h, const muon_fp8_product* products, const std::vector<int>& live,
                            cudaStream_t st) {
  int64_t tiles = 0;
  for (int i : live) {
    const ProductSize z = size_of(products[i]);
    tiles += blocks_of(z.m) * blocks_of(z.n);
  }
  std::vector<int> runs[3];
  for (int i : live) {
    const muon_fp8_product& q = products[i];
    runs[tiles <= h->sm_count ? 0 : size_of(q).k == 0 ? 2 : long_sum(q) ? 1 : 0].push_back(i);
  }
  for (const std::vector<int>& run : runs) {
    const muon_status s = launch_run(h, products, run, st);
    if (s) return s;
  }
  return MUON_OK;
}

// ------------------------------------------------------------------ entry points

muon_status quantize(muon_handle_t h, const muon_dense* x, const muon_fp8_matrix* out, int n, muon_activation act,
                     void* cuda_stream) {
  if (!h) return MUON_ERR_INVALID_ARG;
  h->err.clear();
  muon_status s;
  if ((s = check_list(h, n, x, out)) || (s = check_act(h, act))) return s;
  if (n == 0) return MUON_OK;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(h, MUON_ERR_CUDA, "cannot select device %d", h->device);
  NvtxScope nv(h->nvtx, "muon_fp8_quantize");
  Call call{h};
  std::vector<F8Pass> passes;
  for (int i = 0; i < n; ++i) {
    if ((s = call.dense(x[i], "x", i, false)) || (s = call.fp8(out[i], "out", i, true))) return s;
    if (x[i].rows != out[i].rows || x[i].cols != out[i].cols)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: x and out differ in shape", i);
    if (empty(x[i].rows, x[i].cols)) continue;
    F8Pass m = make_pass(x[i].rows, x[i].cols);
    m.in = kernel_dense(x[i]);
    m.out8 = kernel_fp8(out[i]);
    passes.push_back(m);
  }
  return run_passes(call, kF8Quantize, MUON_FP8_KIND_QUANTIZE, passes, act, static_cast<cudaStream_t>(cuda_stream));
}

muon_status dequantize(muon_handle_t h, const muon_fp8_matrix* x, const muon_dense* out, int n, void* cuda_stream) {
  if (!h) return MUON_ERR_INVALID_ARG;
  h->err.clear();
  muon_status s;
  if ((s = check_list(h, n, x, out))) return s;
  if (n == 0) return MUON_OK;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(h, MUON_ERR_CUDA, "cannot select device %d", h->device);
  NvtxScope nv(h->nvtx, "muon_fp8_dequantize");
  Call call{h};
  std::vector<F8Pass> passes;
  for (int i = 0; i < n; ++i) {
    if ((s = call.fp8(x[i], "x", i, false)) || (s = call.dense(out[i], "out", i, true))) return s;
    if (x[i].rows != out[i].rows || x[i].cols != out[i].cols)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: x and out differ in shape", i);
    if (empty(x[i].rows, x[i].cols)) continue;
    F8Pass m = make_pass(x[i].rows, x[i].cols);
    m.saved = kernel_fp8(x[i]);
    m.out = kernel_dense(out[i]);
    passes.push_back(m);
  }
  return run_passes(call, kF8Dequantize, MUON_FP8_KIND_DEQUANTIZE, passes, MUON_ACT_NONE,
                    static_cast<cudaStream_t>(cuda_stream));
}

muon_status act_backward(muon_handle_t h, const muon_dense* dy, const muon_fp8_matrix* saved, const muon_dense* du,
                         const muon_fp8_matrix* du8, int n, muon_activation act, void* cuda_stream) {
  if (!h) return MUON_ERR_INVALID_ARG;
  h->err.clear();
  muon_status s;
  if ((s = check_list(h, n, dy, saved)) || (s = check_act(h, act))) return s;
  if (n == 0) return MUON_OK;
  if (!du && !du8) return fail(h, MUON_ERR_INVALID_ARG, "du and du8 are both NULL");
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(h, MUON_ERR_CUDA, "cannot select device %d", h->device);
  NvtxScope nv(h->nvtx, "muon_fp8_act_backward");
  Call call{h};
  std::vector<F8Pass> passes;
  for (int i = 0; i < n; ++i) {
    const int64_t rows = dy[i].rows, cols = dy[i].cols;
    if (saved[i].rows != rows || saved[i].cols != cols)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: dy and saved differ in shape", i);
    const bool to_dense = du && du[i].data, to_fp8 = du8 && du8[i].codes;
    if (!empty(rows, cols) && to_dense == to_fp8)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: give one of du and du8", i);
    if ((s = call.fp8(saved[i], "saved", i, false))) return s;
    if (to_dense) {
      if (du[i].rows != rows || du[i].cols != cols)
        return fail(h, MUON_ERR_INVALID_ARG, "item %d: dy and du differ in shape", i);
      // in place: the warp that writes an entry has read it before
      if (!same_dense(dy[i], du[i]) && (s = call.dense(dy[i], "dy", i, false))) return s;
      if ((s = call.dense(du[i], "du", i, true))) return s;
    } else {
      if ((s = call.dense(dy[i], "dy", i, false))) return s;
      if (to_fp8) {
        if (du8[i].rows != rows || du8[i].cols != cols)
          return fail(h, MUON_ERR_INVALID_ARG, "item %d: dy and du8 differ in shape", i);
        if ((s = call.fp8(du8[i], "du8", i, true))) return s;
      }
    }
    if (empty(rows, cols)) continue;
    F8Pass m = make_pass(rows, cols);
    m.in = kernel_dense(dy[i]);
    m.saved = kernel_fp8(saved[i]);
    if (to_dense) m.out = kernel_dense(du[i]);
    else m.out8 = kernel_fp8(du8[i]);
    passes.push_back(m);
  }
  return run_passes(call, kF8ActBackward, MUON_FP8_KIND_ACT_BACKWARD, passes, act,
                    static_cast<cudaStream_t>(cuda_stream));
}

muon_status selftest_timeout(muon_handle_t h, int64_t limit_ns, void* cuda_stream) {
  if (!h) return MUON_ERR_INVALID_ARG;
  h->err.clear();
  if (limit_ns < 0 || limit_ns > 10000000000ll) return fail(h, MUON_ERR_INVALID_ARG, "limit_ns out of range");
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(h, MUON_ERR_CUDA, "cannot select device %d", h->device);
  muon_status s;
  if ((s = ensure_fp8(h))) return s;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if ((s = poll_status(h, false, st))) return s;
  int mark;
  if ((s = take_mark(h, st, &mark))) return s;
  const cudaError_t e = launch_fp8_wait_selftest(h->fp8_status_dev, 2 * limit_ns, st);
  if (e != cudaSuccess) return cuda_fail(h, e, "self-test launch");
  h->last_launches = 1;
  return finish_fp8(h, st, mark, MUON_OK);
}

muon_status matmul(muon_handle_t h, const muon_fp8_product* products, int n, void* cuda_stream) {
  if (!h) return MUON_ERR_INVALID_ARG;
  h->err.clear();
  muon_status s;
  if ((s = check_list(h, n, products, products))) return s;
  if (n == 0) return MUON_OK;
  DeviceGuard dg(h->device);
  if (!dg.ok) return fail(h, MUON_ERR_CUDA, "cannot select device %d", h->device);
  NvtxScope nv(h->nvtx, "muon_fp8_matmul");
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  Call call{h};
  std::vector<int> live;
  for (int i = 0; i < n; ++i) {
    const muon_fp8_product& q = products[i];
    if ((s = call.fp8(q.a, "a", i, false)) || (s = call.fp8(q.b, "b", i, false))) return s;
    const int64_t m = q.trans_a ? q.a.cols : q.a.rows, k = q.trans_a ? q.a.rows : q.a.cols;
    const int64_t kb = q.trans_b ? q.b.cols : q.b.rows, nn = q.trans_b ? q.b.rows : q.b.cols;
    if (k != kb)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: op(A) has %lld columns, op(B) %lld rows", i, (long long)k,
                  (long long)kb);
    if ((q.trans_a && q.a.blocks != MUON_BLOCK_SQUARE) || (!q.trans_b && q.b.blocks != MUON_BLOCK_SQUARE))
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: an operand contracted over its rows needs square blocks", i);
    if (q.epilogue != MUON_EPI_NONE && q.epilogue != MUON_EPI_RELU2 && q.epilogue != MUON_EPI_RELU2_BACKWARD)
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: unknown epilogue %d", i, (int)q.epilogue);
    const bool to_dense = q.d.data != nullptr, to_fp8 = q.d8.codes != nullptr;
    if (!empty(m, nn) && to_dense == to_fp8) return fail(h, MUON_ERR_INVALID_ARG, "item %d: give one of d and d8", i);
    if (to_dense && (q.d.rows != m || q.d.cols != nn))
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: d is %lld x %lld, the product %lld x %lld", i,
                  (long long)q.d.rows, (long long)q.d.cols, (long long)m, (long long)nn);
    if (to_fp8 && (q.d8.rows != m || q.d8.cols != nn))
      return fail(h, MUON_ERR_INVALID_ARG, "item %d: d8 is %lld x %lld, the product %lld x %lld", i,
                  (long long)q.d8.rows, (long long)q.d8.cols, (long long)m, (long long)nn);
    if (to_dense && (s = call.dense(q.d, "d", i, true))) return s;
    if (to_fp8 && (s = call.fp8(q.d8, "d8", i, true))) return s;
    if (q.c.data) {
      if (q.c.rows != m || q.c.cols != nn)
        return fail(h, MUON_ERR_INVALID_ARG, "item %d: c is %lld x %lld, the product %lld x %lld", i,
                    (long long)q.c.rows, (long long)q.c.cols, (long long)m, (long long)nn);
      // c = d: the warp that writes an entry has read it before
      if (!(to_dense && same_dense(q.c, q.d)) && (s = call.dense(q.c, "c", i, false))) return s;
    }
    if (q.epilogue == MUON_EPI_RELU2_BACKWARD) {
      if (q.saved.rows != m || q.saved.cols != nn)
        return fail(h, MUON_ERR_INVALID_ARG, "item %d: saved is %lld x %lld, the product %lld x %lld", i,
                    (long long)q.saved.rows, (long long)q.saved.cols, (long long)m, (long long)nn);
      if ((s = call.fp8(q.saved, "saved", i, false))) return s;
    }
    if (blocks_of(m) * blocks_of(nn) > kMaxTiles)
      return fail(h, MUON_ERR_UNSUPPORTED, "item %d: the result has too many tiles", i);
    if (!empty(m, nn)) live.push_back(i);
  }
  int mark;
  if ((s = call.check())) return s;
  if ((s = ensure_fp8(h))) return s;
  if ((s = poll_status(h, false, st))) return s;
  if ((s = take_mark(h, st, &mark))) return s;
  h->last_launches = 0;
  return finish_fp8(h, st, mark, launch_products(h, products, live, st));
}

// No C++ exception (host memory that runs out) crosses the C boundary.
template <typename F>
muon_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return MUON_ERR_OOM;
  }
}

}  // namespace

extern "C" {

muon_status muon_fp8_quantize(muon_handle_t h, const muon_dense* x, const muon_fp8_matrix* out, int n,
                              muon_activation act, void* cuda_stream) {
  return guarded([&] { return quantize(h, x, out, n, act, cuda_stream); });
}

muon_status muon_fp8_dequantize(muon_handle_t h, const muon_fp8_matrix* x, const muon_dense* out, int n,
                                void* cuda_stream) {
  return guarded([&] { return dequantize(h, x, out, n, cuda_stream); });
}

muon_status muon_fp8_act_backward(muon_handle_t h, const muon_dense* dy, const muon_fp8_matrix* saved,
                                  const muon_dense* du, const muon_fp8_matrix* du8, int n, muon_activation act,
                                  void* cuda_stream) {
  return guarded([&] { return act_backward(h, dy, saved, du, du8, n, act, cuda_stream); });
}

muon_status muon_fp8_matmul(muon_handle_t h, const muon_fp8_product* products, int n, void* cuda_stream) {
  return guarded([&] { return matmul(h, products, n, cuda_stream); });
}

muon_status muon_selftest_fp8_timeout(muon_handle_t h, int64_t limit_ns, void* cuda_stream) {
  return guarded([&] { return selftest_timeout(h, limit_ns, cuda_stream); });
}

}  // extern "C"
