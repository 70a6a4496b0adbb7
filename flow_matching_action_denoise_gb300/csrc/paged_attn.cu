// Attention over a paged cache: which kernel, how its keys are divided, the join of splits, the entry points.

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "internal.h"
#include "kv.h"
#include "paged_tile.cuh"

namespace fm {

template cudaError_t tile_launch<Keys::kAll>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&, dim3, size_t,
                                             const LaunchOpts&);
template cudaError_t tile_configure<Keys::kAll>();

namespace {

// Joins the splits of the rows that they computed: an entry's (grid.y) first max_tokens tokens. All else keeps what it
// holds, the rows of an entry out of range too. Bound by latency, the shares come from L2: `warps` (1, 2, 4 or 8, a power
// of two) of a CTA's eight share a row, each every warps-th split, and are summed in warp order.
template <int DH>
__global__ void __launch_bounds__(256) combine_kernel(const AttnParams p, int warps) {
  constexpr int kPer = DH / 32;
  __shared__ float s_acc[8][DH];
  __shared__ float s_sum[8];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Entry en = entry_of(p, blockIdx.y, false);
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.H;   // of a split
  const int64_t in_entry = (blockIdx.x * 8ll + warp) / warps;
  const int sub = warp & (warps - 1);
  const bool live = in_entry < static_cast<int64_t>(min(en.nq, p.max_tokens)) * p.H;
  const int64_t row = static_cast<int64_t>(en.begin) * p.H + in_entry;
  float acc[kPer] = {};
  float sum = 0.f;
  if (live) {
    float top = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) top = fmaxf(top, p.part_ml[s * rows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 4
    for (int s = sub; s < p.splits; s += warps) {
      const float2 ml = p.part_ml[s * rows + row];   // one address for the warp
      // no keys: its share is not written. A NaN in the query has no maximum either, but its sum is NaN and so is the row
      if (ml.x == -INFINITY && ml.y == 0.f) continue;
      const float w = exp2f(ml.x - top);
      sum += ml.y * w;
      const float* src = p.part_o + (s * rows + row) * DH + lane * kPer;
      if constexpr (kPer == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] += w * v.x, acc[1] += w * v.y, acc[2] += w * v.z, acc[3] += w * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] += w * v.x, acc[1] += w * v.y;
      }
    }
  }
  if (warps > 1) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_acc[warp][lane * kPer + i] = acc[i];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (sub == 0) {
      for (int w = 1; w < warps; ++w) {
        sum += s_sum[warp + w];
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += s_acc[warp + w][lane * kPer + i];
      }
    }
  }
  if (!live || sub) return;
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  const int64_t token = in_entry / p.H;
  __nv_bfloat16* dst = p.out + (en.begin + token) * p.out_stride + (in_entry - token * p.H) * DH + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<false>(acc[0] * inv, acc[1] * inv), pack16<false>(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack16<false>(acc[0] * inv, acc[1] * inv);
}

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
    return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr)
                                                                : nullptr;
  }();
  return fn;
}

// Rows of one KV head's page block as a TMA source: (head dim, token, head, page).
bool kv_tmap(CUtensorMap* map, const fm_kv_cache& c, const void* base, bool decode) {
  const bool f8 = c.fmt == FM_FMT_FP8;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.Dh), static_cast<cuuint64_t>(c.page_tokens),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.pages)};
  // the stride of an extent of one is never used: any legal value
  const auto stride = [&](int64_t s, int extent) { return static_cast<cuuint64_t>((extent == 1 ? c.Dh : s) * (f8 ? 1 : 2)); };
  const cuuint64_t strides[3] = {stride(c.token_stride, c.page_tokens), stride(c.head_stride, c.Hkv),
                                 stride(c.page_stride, c.pages)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(f8 ? c.Dh : 64),
                             static_cast<cuuint32_t>(std::min(c.page_tokens, decode ? kDecodeKeys : kTileRows)), 1, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  // codes that are expanded in shared memory lie there in plain rows, all else is read by matrix instructions
  const CUtensorMapSwizzle swizzle = !f8                        ? CU_TENSOR_MAP_SWIZZLE_128B
                                     : !decode                  ? CU_TENSOR_MAP_SWIZZLE_NONE
                                     : c.Dh == 128              ? CU_TENSOR_MAP_SWIZZLE_128B
                                                                : CU_TENSOR_MAP_SWIZZLE_64B;
  const auto encode = tmap_encoder();
  return encode && encode(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base),
                          dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
  int decode, alt, splits, split_tiles, ring, raw_ring;
  int64_t row_blocks;
  int rows_first;
  size_t smem, workspace;
};

int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 152;
  }
  int v = cached[dev].load(std::memory_order_relaxed);
  if (v) return v;
  if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) {
    cudaGetLastError();
    v = 152;
  }
  cached[dev].store(v, std::memory_order_relaxed);
  return v;
}

// Keys that a CTA's tokens see together, and the tiles that they may lie in. With sinks the tokens are those of a block of
// `rows` rows, with a window alone all of an entry.
int64_t keys_of(const fm_kv_batch& b, int G, int rows, int window, int sinks) {
  const int64_t len = std::max(1, b.max_len);
  const int64_t tokens = sinks > 0 ? std::min<int64_t>(b.max_tokens, rows / G + 2) : b.max_tokens;
  return window > 0 ? std::min<int64_t>(len, static_cast<int64_t>(window) + tokens + sinks) : len;
}
int64_t tiles_of(int64_t keys, int tile, int window, int sinks) {
  return (keys + tile - 1) / tile + (window > 0) + (sinks > 0);
}

// The number of splits of a batch's keys. window 0: the one that the workspace is sized for.
int splits_of(const fm_kv_cache& c, const fm_kv_batch& b, int H, int window, int sinks) {
  const int64_t rows = static_cast<int64_t>(b.max_tokens) * (H / c.Hkv);
  const int sms = sm_count();
  const bool f8 = c.fmt == FM_FMT_FP8;
  const int G = H / c.Hkv;
  if (rows <= kDecodeRows) {
    const int64_t keys = keys_of(b, G, kDecodeRows, window, sinks);
    // As many CTAs as are resident at once: a second wave costs more than longer splits (64 units of 4096 keys: 25 us
    // in 256 CTAs, 31 us in 384). Splits of at least two tiles up to 8, which join in their cluster; beyond, where a
    // second kernel joins them, of at least four (32768 keys of one unit: 11.6 us in 64 splits, 20.7 us in 256), and
    // only where 8 would be long (4096 keys of one unit: 8.3 us in 8, 7.7 us in 24; 2000: 7.4 us in 8, 7.5 us in 16).
    const int64_t units = static_cast<int64_t>(c.Hkv) * std::max(1, b.n);
    const int64_t tiles = tiles_of(keys, kDecodeKeys, window, sinks);
    const int64_t slots = std::max<int64_t>(1, static_cast<int64_t>(sms) * decode_resident(c.Dh, f8, static_cast<int>(rows)) / units);
    const int64_t want = tiles > 40 ? std::min<int64_t>(std::min<int64_t>(slots, 64), (tiles + 3) / 4)
                                    : std::min<int64_t>(std::min<int64_t>(slots, 8), (tiles + 1) / 2);
    return static_cast<int>(std::max<int64_t>(1, want));
  }
  // One CTA an SM: waves x (start and end + tiles x time of a tile), in units of 0.1 us as measured, with the join of
  // splits (a kernel, and every share written and read) added. The number of splits with the least of it.
  const bool alt = rows <= kTileRows;
  const int64_t block_rows = alt ? kTileRows : 2 * kTileRows;
  const int64_t units = std::max<int64_t>(1, (rows + block_rows - 1) / block_rows * c.Hkv * b.n);
  const int64_t tiles = tiles_of(keys_of(b, G, static_cast<int>(block_rows), window, sinks), kTileRows, window, sinks);
  const int64_t fixed = f8 ? 85 : 70, each = alt ? (f8 ? 15 : 8) : (f8 ? 18 : 14);
  int64_t best = 0, splits = 1;
  // entries x splits are a dimension of the grid
  const int64_t most = std::min<int64_t>({64, std::max<int64_t>(1, tiles / 2), std::max(1, 65535 / std::max(1, b.n))});
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t waves = (units * s + sms - 1) / sms;
    const int64_t shares = s * b.tokens * H * c.Dh * 8;   // bytes, at 4 TB/s: 4e5 bytes in 0.1 us
    const int64_t cost = waves * (fixed + (tiles + s - 1) / s * each) + (s > 1 ? 25 + shares / 400000 : 0);
    if (s == 1 || cost < best) {
      best = cost;
      splits = s;
    }
  }
  return static_cast<int>(splits);
}

// The variant for a batch, by its bounds and the number of SMs alone. A window, which the workspace query does not
// know, only lowers the number of splits.
Plan plan_of(const fm_kv_cache& c, const fm_kv_batch& b, int H, int window, int sinks) {
  Plan pl = {};
  const int64_t rows = static_cast<int64_t>(b.max_tokens) * (H / c.Hkv);
  pl.splits = splits_of(c, b, H, 0, 0);
  if (window > 0) pl.splits = std::min(pl.splits, splits_of(c, b, H, window, sinks));
  pl.decode = rows <= kDecodeRows;
  if (!pl.decode) {
    pl.alt = rows <= kTileRows;
    const int block_rows = pl.alt ? kTileRows : 2 * kTileRows;
    const int64_t tiles = tiles_of(keys_of(b, H / c.Hkv, block_rows, window, sinks), kTileRows, window, sinks);
    pl.split_tiles = static_cast<int>((tiles + pl.splits - 1) / pl.splits);
    pl.row_blocks = (rows + block_rows - 1) / block_rows;
    // Where most of a sequence is new, a row block's place decides its keys, and CTAs start in the order of their work,
    // row blocks outermost, so that short ones fill the last wave (2048 tokens, 32 heads on 8 KV heads: 50.5 us with heads
    // outermost, 37.2 us; 4 x 2048 tokens of 16 on 2: 80.1 and 72.5 us). Else heads and entries are outermost: the entry's
    // length, which the host does not know, decides more. Splits are of equal length but the last.
    pl.rows_first = pl.splits == 1 && 2 * static_cast<int64_t>(b.max_tokens) >= b.max_len && pl.row_blocks <= 65535;
    const size_t tile = static_cast<size_t>(kTileRows) * c.Dh * 2;
    const size_t q = tile * (pl.alt ? 1 : 2);
    const size_t room = kSmemLimit - kCtlBytes - q;
    if (c.fmt == FM_FMT_FP8) {
      pl.ring = 4;
      pl.raw_ring = static_cast<int>(std::min<size_t>(kMaxRing, (room - pl.ring * tile) / (tile / 2)));
    } else {
      pl.ring = static_cast<int>(std::min<size_t>(kMaxRing, room / tile));
    }
    pl.smem = 1024 + q + pl.ring * tile + pl.raw_ring * (tile / 2) + kCtlBytes;
  }
  if (pl.splits > (pl.decode ? 8 : 1))
    pl.workspace = static_cast<size_t>(pl.splits) * b.tokens * H * (c.Dh * sizeof(float) + sizeof(float2));
  return pl;
}

// The kernels' shared-memory limits, once a device.
template <Keys K>
cudaError_t configure() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = tile_configure<K>();
  if (e == cudaSuccess) e = decode_configure<K>();
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

int check(const fm_kv_cache* c, const fm_kv_batch* b, int H) {
  int st = kv_check(c);
  if (st == FM_OK) st = kv_batch_check(c, b);
  if (st != FM_OK) return st;
  if (H <= 0 || H % c->Hkv) return record_error(FM_ERR_SHAPE, "H must be a positive multiple of the cache's Hkv");
  if (c->Dh != 64 && c->Dh != 128) return record_error(FM_ERR_SHAPE, "attention takes head dims of 64 or 128");
  const int64_t rows = static_cast<int64_t>(b->max_tokens) * (H / c->Hkv);
  if (rows > (int64_t(1) << 30)) return record_error(FM_ERR_SHAPE, "max_tokens * H / Hkv exceeds 2^30");
  return FM_OK;
}

template <Keys K>
int attend(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const uint16_t* q, int64_t q_stride, int H, float scale,
           int causal, int window, int sinks, uint16_t* out, int64_t out_stride, void* workspace, size_t workspace_bytes,
           void* stream) {
  const int st = check(c, b, H);
  if (st != FM_OK) return st;
  if (layer < 0 || layer >= c->layers) return record_error(FM_ERR_INVALID_ARG, "layer out of range");
  if (!(scale > 0.f) || !std::isfinite(scale)) return record_error(FM_ERR_INVALID_ARG, "scale must be positive and finite");
  if (window < 0) return record_error(FM_ERR_INVALID_ARG, "window must be 0 (none) or positive");
  if (b->n == 0 || b->tokens == 0 || b->max_tokens == 0) return FM_OK;
  if (!q || !out) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  const int64_t row = static_cast<int64_t>(H) * c->Dh;
  if (q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8)
    return record_error(FM_ERR_SHAPE, "token strides must be multiples of 8 elements and hold H * Dh");
  if (reinterpret_cast<uintptr_t>(q) % 16 || reinterpret_cast<uintptr_t>(out) % 16)
    return record_error(FM_ERR_ALIGN, "q and out must be 16-byte aligned");
  const fm_kv_batch bounded = bounded_batch(*b);
  b = &bounded;
  const Plan pl = plan_of(*c, *b, H, window, sinks);
  const size_t need = pl.workspace;
  if (need) {
    if (!workspace) return record_error(FM_ERR_INVALID_ARG, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(workspace) % 16) return record_error(FM_ERR_ALIGN, "workspace not 16-byte aligned");
    if (workspace_bytes < need)
      return record_error(FM_ERR_WORKSPACE, "workspace smaller than fm_paged_attention_workspace_size()");
  }
  const bool f8 = c->fmt == FM_FMT_FP8;
  const int64_t off = layer * c->layer_stride * (f8 ? 1 : 2);
  CUtensorMap tk, tv;
  if (!kv_tmap(&tk, *c, static_cast<const uint8_t*>(c->k) + off, pl.decode) ||
      !kv_tmap(&tv, *c, static_cast<const uint8_t*>(c->v) + off, pl.decode))
    return record_error(FM_ERR_CUDA, "cuTensorMapEncodeTiled (cache pages) failed");
  int* err = standalone_error_word();
  if (!err) return record_error(FM_ERR_CUDA, "no error word on the current device");
  cudaError_t e = configure<K>();
  if (e != cudaSuccess) return record_error(FM_ERR_CUDA, cudaGetErrorString(e));
  AttnParams p = {};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.start = b->start;
  p.seq = b->seq;
  p.lens = c->lens;
  p.table = c->table;
  p.n = b->n;
  p.tokens = b->tokens;
  p.max_tokens = b->max_tokens;
  p.seqs = c->seqs;
  p.table_stride = c->table_stride;
  p.pages = c->pages;
  p.page = c->page_tokens;
  while ((1 << p.page_shift) < c->page_tokens) ++p.page_shift;
  p.H = H;
  p.Hkv = c->Hkv;
  p.G = H / c->Hkv;
  p.causal = causal != 0;
  p.window = window;
  p.sinks = sinks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.k_scale = f8 ? c->k_scale + layer : nullptr;
  p.v_scale = f8 ? c->v_scale + layer : nullptr;
  p.alt = pl.alt;
  p.row_blocks = static_cast<int>(pl.row_blocks);
  p.rows_first = pl.rows_first;
  p.splits = pl.splits;
  p.split_tiles = pl.split_tiles;
  p.ring = pl.ring;
  p.raw_ring = pl.raw_ring;
  if (need) {
    p.part_o = static_cast<float*>(workspace);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(pl.splits) * b->tokens * H * c->Dh);
  }
  p.err = err;
  LaunchOpts o;
  o.stream = static_cast<cudaStream_t>(stream);
  o.pdl = true;
  if (pl.decode) {
    e = decode_launch<K>(p, c->Dh, f8, tk, tv, o);
  } else {
    const unsigned blocks = static_cast<unsigned>(pl.row_blocks), entries = static_cast<unsigned>(b->n * pl.splits);
    const dim3 grid = pl.rows_first ? dim3(c->Hkv, entries, blocks) : dim3(blocks, c->Hkv, entries);
    e = tile_launch<K>(p, c->Dh, f8, tk, tv, grid, pl.smem, o);
  }
  if (e == cudaSuccess && need) {
    // a warp takes up to four splits where there are few rows (256 splits of 8 rows took 45 us with a warp a row)
    int warps = 1;
    while (warps < 8 && pl.splits > 4 * warps) warps *= 2;
    const int64_t blocks = (static_cast<int64_t>(b->max_tokens) * H * warps + 7) / 8;
    auto join = c->Dh == 128 ? combine_kernel<128> : combine_kernel<64>;
    e = launch(join, dim3(static_cast<unsigned>(blocks), b->n), dim3(256), 0, o, p, warps);
  }
  return e == cudaSuccess ? FM_OK : record_error(FM_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace

}  // namespace fm

extern "C" int fm_paged_attention_workspace_size(const fm_kv_cache* c, const fm_kv_batch* b, int H, size_t* bytes) {
  if (!bytes) return fm::record_error(FM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = fm::check(c, b, H);
  if (st != FM_OK) return st;
  *bytes = b->n && b->tokens ? fm::plan_of(*c, fm::bounded_batch(*b), H, 0, 0).workspace : 0;
  return FM_OK;
}

extern "C" int fm_paged_attention(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const uint16_t* q,
                                  int64_t q_stride, int H, float scale, int causal, int window, uint16_t* out,
                                  int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  return fm::attend<fm::Keys::kAll>(c, layer, b, q, q_stride, H, scale, causal, window, 0, out, out_stride, workspace,
                                    workspace_bytes, stream);
}

extern "C" int fm_sink_attention(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const uint16_t* q, int64_t q_stride,
                                 int H, float scale, int causal, int window, int sinks, uint16_t* out, int64_t out_stride,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  using namespace fm;
  if (sinks < 0) return record_error(FM_ERR_INVALID_ARG, "sinks must not be negative");
  // without a window nothing is hidden, without first tokens nothing is kept: the same attention in one stretch of keys
  if (window <= 0 || sinks == 0)
    return attend<Keys::kAll>(c, layer, b, q, q_stride, H, scale, causal, window, 0, out, out_stride, workspace,
                              workspace_bytes, stream);
  return attend<Keys::kSinks>(c, layer, b, q, q_stride, H, scale, causal, window, sinks, out, out_stride, workspace,
                              workspace_bytes, stream);
}
