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
// in sources of their own
extern template cudaError_t tile_launch<Keys::kSinks>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&, dim3,
                                                      size_t, const LaunchOpts&);
extern template cudaError_t tile_configure<Keys::kSinks>();
extern template cudaError_t tile_launch<Keys::kPrefix>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&, dim3,
                                                       size_t, const LaunchOpts&);
extern template cudaError_t tile_configure<Keys::kPrefix>();

int tile_clusters(int size) {
  auto* kernel = &paged_attn_kernel<128, false, Keys::kAll, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, 1, size);
  cfg.blockDim = dim3(threads_of(false));
  cfg.dynamicSmemBytes = kSmemLimit;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = size;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  int n = 0;
  return tile_configure<Keys::kAll>() == cudaSuccess && cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
}

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
  int cluster;       // the tile kernel's splits that meet in their cluster (0: through the workspace)
  int64_t row_blocks;
  int rows_first;
  size_t smem, workspace;
};

// The tile kernel's buffers for keys and values, and its shared memory.
void rings_of(const fm_kv_cache& c, Plan& pl) {
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

// Clusters of `size` CTAs (1 to 8) that run at once: fewer CTAs than alone, since a cluster stays inside of a group of SMs (of
// the tile kernel, one CTA an SM, 76, 46, 36, 28, 23, 15 and 15 clusters of 2 to 8 on 152 SMs). kind: the kernel's variant.
template <typename Query>
int clusters_at_once(int kind, int size, int without, Query query) {
  static std::atomic<int> cached[64][16][9];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return std::max(1, without / size);
  }
  int v = cached[dev][kind][size].load(std::memory_order_relaxed);
  if (v) return v;
  v = query();
  if (v <= 0) {
    cudaGetLastError();
    v = std::max(1, without / size);
  }
  cached[dev][kind][size].store(v, std::memory_order_relaxed);
  return v;
}
int tile_clusters_at_once(int size) {
  return clusters_at_once(0, size, sm_count(), [=] { return tile_clusters(size); });
}
int decode_clusters_at_once(int Dh, bool f8, int rows, int size) {
  const int kind = 1 + (Dh == 128) + 2 * f8 + 4 * (rows > 8);
  return clusters_at_once(kind, size, sm_count() * decode_resident(Dh, f8, rows), [=] { return decode_clusters(Dh, f8, rows, size); });
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

// Time of a CTA of the tile kernel, in units of 0.1 us as measured: its start and end, and its tiles.
int64_t cta_time(bool f8, bool alt, int64_t tiles) { return (f8 ? 85 : 70) + tiles * (alt ? (f8 ? 15 : 8) : (f8 ? 18 : 14)); }

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
  // One CTA an SM: waves x the time of a CTA, with the join of splits (a kernel, and every share written and read) added.
  // The number of splits with the least of it.
  const bool alt = rows <= kTileRows;
  const int64_t block_rows = alt ? kTileRows : 2 * kTileRows;
  const int64_t units = std::max<int64_t>(1, (rows + block_rows - 1) / block_rows * c.Hkv * b.n);
  const int64_t tiles = tiles_of(keys_of(b, G, static_cast<int>(block_rows), window, sinks), kTileRows, window, sinks);
  int64_t best = 0, splits = 1;
  // entries x splits are a dimension of the grid
  const int64_t most = std::min<int64_t>({64, std::max<int64_t>(1, tiles / 2), std::max(1, 65535 / std::max(1, b.n))});
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t waves = (units * s + sms - 1) / sms;
    const int64_t shares = s * b.tokens * H * c.Dh * 8;   // bytes, at 4 TB/s: 4e5 bytes in 0.1 us
    const int64_t cost = waves * cta_time(f8, alt, (tiles + s - 1) / s) + (s > 1 ? 25 + shares / 400000 : 0);
    if (s == 1 || cost < best) {
      best = cost;
      splits = s;
    }
  }
  return static_cast<int>(splits);
}

// Time of the join of a plan's splits, in units of 0.1 us: in the cluster by the rows of a CTA, else a second kernel and the
// shares. An estimate of its own: splits_of, which chooses among up to 64 splits of a plain call, counts less for the same
// second kernel (2.5 us and the shares at 4 TB/s, here 5.5 us and 8 TB/s), and neither holds everywhere. Where a cluster is
// taken for it with first tokens, the workspace can be quicker: 1 x 30 tokens over 3000 keys, 8 heads on 1, Dh 128, window 2000
// + 100 take 16.5 us in a cluster of 7, all 3000 keys in 12 splits through the workspace 14.5 us.
int64_t join_time(const fm_kv_cache& c, const fm_kv_batch& b, int H, const Plan& pl) {
  if (pl.splits == 1) return 0;
  if (pl.cluster)
    return 5 + std::min<int64_t>(pl.alt ? kTileRows : 2 * kTileRows, static_cast<int64_t>(b.max_tokens) * (H / c.Hkv)) * 17 / 100;
  return 55 + static_cast<int64_t>(pl.splits) * b.tokens * H * c.Dh * 8 / 800000;
}

// Splits that meet in their cluster: up to 8, where the clusters take no more waves than CTAs alone would. A CTA reads its
// rows' parts from the others' shared memory: about 5 us for 256 rows and 2.5 us for 128, against a second kernel and the
// shares' way through L2, 4.5 us and more (6 entries x 20 tokens over 2000 keys, 6 heads of 64: 14.0 -> 10.2 us; 16 x up to 50 tokens
// over 4100, 16 heads of 128: 41.6 -> 39.0 us). With first tokens the number of splits is chosen for it (1 x 100 tokens, window
// 2000 + 100, 16 heads on 2: 36.4 us undivided, 22.1 in 4, 18.6 in 7); without them it stays what it is without a cluster.
void cluster_of(const fm_kv_cache& c, const fm_kv_batch& b, int H, int64_t tiles, bool sinks, Plan& pl) {
  const bool f8 = c.fmt == FM_FMT_FP8;
  const int64_t units = std::max<int64_t>(1, pl.row_blocks * c.Hkv * b.n);
  const auto waves = [](int64_t n, int64_t at_once) { return (n + at_once - 1) / at_once; };
  const auto time = [&](int s) { return cta_time(f8, pl.alt, (tiles + s - 1) / s); };   // 0.1 us
  if (!sinks) {
    if (pl.splits > 1 && pl.splits <= 8 && waves(units, tile_clusters_at_once(pl.splits)) <= waves(units * pl.splits, sm_count()))
      pl.cluster = pl.splits;
    return;
  }
  int64_t best = waves(units * pl.splits, sm_count()) * time(pl.splits) + join_time(c, b, H, pl);
  Plan with = pl;
  for (int s = 2; s <= std::min<int64_t>(8, tiles) && static_cast<int64_t>(b.n) * s <= 65535; ++s) {
    with.splits = with.cluster = s;
    const int64_t cost = waves(units, tile_clusters_at_once(s)) * time(s) + join_time(c, b, H, with);
    if (cost >= best) continue;
    best = cost;
    pl = with;
  }
}

// The variant for a batch, by its bounds and the number of SMs alone. A window, which the workspace query does not know, only
// lowers the number of splits that go through the workspace; with first tokens there may be more of them in clusters, which
// need none. meet: the tile kernel's splits may meet in clusters. fm_paged_attention's do not: its plan and its workspace are as
// they were before there were clusters for many rows, and the same calls without sharing through fm_shared_attention, which
// give the same bits, show what that costs (above).
Plan plan_of(const fm_kv_cache& c, const fm_kv_batch& b, int H, int window, int sinks, bool meet) {
  Plan pl = {};
  const int64_t rows = static_cast<int64_t>(b.max_tokens) * (H / c.Hkv);
  pl.splits = splits_of(c, b, H, 0, 0);
  if (window > 0) pl.splits = std::min(pl.splits, splits_of(c, b, H, window, sinks));
  pl.decode = rows <= kDecodeRows;
  if (pl.decode && sinks > 0 && pl.splits > 1 && pl.splits <= 8) {
    // Where the clusters do not all run at once, fewer splits, and some places are left free, since the last ones are not always
    // found: one of clusters of 2 and 4, which pack well, of the others one in 14. Window 2048 + 64, 8 heads on 1, keys from
    // HBM: E4M3, Dh 128: 148 of 148 clusters of 4 22.2 us, of 3 19.6; 146: 19.8, 19.5 (Dh 64: 11.8, 12.5); 112 of 117 of 5 20.0, of 4
    // 17.0; 108: 16.1, 16.7; 78 of 81 of 7 14.3, of 6 14.1; 75: 13.5, 13.9; bf16: 94 of 97 of 3 23.0, of 2 21.2; 89: 20.0, 20.3;
    // 35 of 36 of 8 12.4, of 7 11.5; 33: 11.3, 11.2. Over six kinds of calls and 358 counts, even and ragged, the choice is 0.7 % above the
    // better of the two sizes, without free places 4.6 %.
    const int64_t units = static_cast<int64_t>(c.Hkv) * b.n;
    const auto fits = [&](int s) {
      const int64_t places = decode_clusters_at_once(c.Dh, c.fmt == FM_FMT_FP8, static_cast<int>(rows), s);
      return units <= (s == 2 || s == 4 ? places - 1 : places * 13 / 14);
    };
    while (pl.splits > 1 && !fits(pl.splits)) --pl.splits;
  }
  if (!pl.decode) {
    pl.alt = rows <= kTileRows;
    const int block_rows = pl.alt ? kTileRows : 2 * kTileRows;
    const int64_t tiles = tiles_of(keys_of(b, H / c.Hkv, block_rows, window, sinks), kTileRows, window, sinks);
    pl.row_blocks = (rows + block_rows - 1) / block_rows;
    if (meet) cluster_of(c, b, H, tiles, sinks > 0, pl);
    pl.split_tiles = static_cast<int>((tiles + pl.splits - 1) / pl.splits);
    // Where most of a sequence is new, a row block's place decides its keys, and CTAs start in the order of their work,
    // row blocks outermost, so that short ones fill the last wave (2048 tokens, 32 heads on 8 KV heads: 50.5 us with heads
    // outermost, 37.2 us; 4 x 2048 tokens of 16 on 2: 80.1 and 72.5 us). Else heads and entries are outermost: the entry's
    // length, which the host does not know, decides more. Splits are of equal length but the last.
    pl.rows_first = pl.splits == 1 && 2 * static_cast<int64_t>(b.max_tokens) >= b.max_len && pl.row_blocks <= 65535;
    rings_of(c, pl);
  }
  if (pl.splits > (pl.decode ? 8 : 1) && !pl.cluster)
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
  // the groups' two kernels together
  e = tile_configure<K>();
  if (e == cudaSuccess) e = decode_configure<K == Keys::kPrefix ? Keys::kOwn : K>();
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

// What an attention call is given, checked and bounded; FM_OK with b = nullptr where there is nothing to do.
struct Call {
  const fm_kv_cache* c;
  int layer;
  const fm_kv_batch* b;
  const uint16_t* q;
  int64_t q_stride;
  int H;
  float scale;
  int causal;
  uint16_t* out;
  int64_t out_stride;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
};

int check_call(const Call& a) {
  const int st = check(a.c, a.b, a.H);
  if (st != FM_OK) return st;
  if (a.layer < 0 || a.layer >= a.c->layers) return record_error(FM_ERR_INVALID_ARG, "layer out of range");
  if (!(a.scale > 0.f) || !std::isfinite(a.scale)) return record_error(FM_ERR_INVALID_ARG, "scale must be positive and finite");
  return FM_OK;
}
bool nothing_to_do(const fm_kv_batch& b) { return b.n == 0 || b.tokens == 0 || b.max_tokens == 0; }
int check_tensors(const Call& a) {
  if (!a.q || !a.out) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  const int64_t row = static_cast<int64_t>(a.H) * a.c->Dh;
  if (a.q_stride < row || a.out_stride < row || a.q_stride % 8 || a.out_stride % 8)
    return record_error(FM_ERR_SHAPE, "token strides must be multiples of 8 elements and hold H * Dh");
  if (reinterpret_cast<uintptr_t>(a.q) % 16 || reinterpret_cast<uintptr_t>(a.out) % 16)
    return record_error(FM_ERR_ALIGN, "q and out must be 16-byte aligned");
  return FM_OK;
}
int check_workspace(const Call& a, size_t need, const char* too_small) {
  if (!need) return FM_OK;
  if (!a.workspace) return record_error(FM_ERR_INVALID_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(a.workspace) % 16) return record_error(FM_ERR_ALIGN, "workspace not 16-byte aligned");
  if (a.workspace_bytes < need) return record_error(FM_ERR_WORKSPACE, too_small);
  return FM_OK;
}

// The kernels' parameters but for the plan's; b: the batch, bounded. false: no error word.
bool params_of(const Call& a, const fm_kv_batch& b, AttnParams& p) {
  const fm_kv_cache& c = *a.c;
  const bool f8 = c.fmt == FM_FMT_FP8;
  p = {};
  p.q = reinterpret_cast<const __nv_bfloat16*>(a.q);
  p.out = reinterpret_cast<__nv_bfloat16*>(a.out);
  p.q_stride = a.q_stride;
  p.out_stride = a.out_stride;
  p.start = b.start;
  p.seq = b.seq;
  p.lens = c.lens;
  p.table = c.table;
  p.n = b.n;
  p.tokens = b.tokens;
  p.max_tokens = b.max_tokens;
  p.seqs = c.seqs;
  p.table_stride = c.table_stride;
  p.pages = c.pages;
  p.page = c.page_tokens;
  while ((1 << p.page_shift) < c.page_tokens) ++p.page_shift;
  p.H = a.H;
  p.Hkv = c.Hkv;
  p.G = a.H / c.Hkv;
  p.causal = a.causal != 0;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.k_scale = f8 ? c.k_scale + a.layer : nullptr;
  p.v_scale = f8 ? c.v_scale + a.layer : nullptr;
  p.err = standalone_error_word();
  return p.err != nullptr;
}

void shares_in(const Call& a, int places, int tokens, AttnParams& p) {
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(places) * tokens * a.H * a.c->Dh);
}

bool maps_of(const Call& a, bool decode, CUtensorMap* tk, CUtensorMap* tv) {
  const int64_t off = a.layer * a.c->layer_stride * (a.c->fmt == FM_FMT_FP8 ? 1 : 2);
  return kv_tmap(tk, *a.c, static_cast<const uint8_t*>(a.c->k) + off, decode) &&
         kv_tmap(tv, *a.c, static_cast<const uint8_t*>(a.c->v) + off, decode);
}

void use_plan(const Plan& pl, AttnParams& p) {
  p.alt = pl.alt;
  p.row_blocks = static_cast<int>(pl.row_blocks);
  p.rows_first = pl.rows_first;
  p.splits = pl.splits;
  p.split_tiles = pl.split_tiles;
  p.cluster = pl.cluster;
  p.ring = pl.ring;
  p.raw_ring = pl.raw_ring;
}

template <Keys K>
cudaError_t launch_tiles(const Call& a, const Plan& pl, int n, const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                         const LaunchOpts& o) {
  const unsigned blocks = static_cast<unsigned>(pl.row_blocks), entries = static_cast<unsigned>(n * pl.splits);
  const dim3 grid = pl.rows_first ? dim3(a.c->Hkv, entries, blocks) : dim3(blocks, a.c->Hkv, entries);
  LaunchOpts opts = o;
  if (pl.cluster > 1) opts.cluster = dim3(1, 1, pl.cluster);
  return tile_launch<K>(p, a.c->Dh, a.c->fmt == FM_FMT_FP8, tk, tv, grid, pl.smem, opts);
}

cudaError_t launch_join(const Call& a, const AttnParams& p, const LaunchOpts& o) {
  // a warp takes up to four splits where there are few rows (256 splits of 8 rows took 45 us with a warp a row)
  int warps = 1;
  while (warps < 8 && p.splits > 4 * warps) warps *= 2;
  const int64_t blocks = (static_cast<int64_t>(p.max_tokens) * a.H * warps + 7) / 8;
  auto join = a.c->Dh == 128 ? combine_kernel<128> : combine_kernel<64>;
  return launch(join, dim3(static_cast<unsigned>(blocks), p.n), dim3(256), 0, o, p, warps);
}

LaunchOpts opts_of(const Call& a) {
  LaunchOpts o;
  o.stream = static_cast<cudaStream_t>(a.stream);
  o.pdl = true;
  return o;
}

template <Keys K>
int attend(const Call& a, int window, int sinks, bool meet) {
  int st = check_call(a);
  if (st != FM_OK) return st;
  if (window < 0) return record_error(FM_ERR_INVALID_ARG, "window must be 0 (none) or positive");
  if (nothing_to_do(*a.b)) return FM_OK;
  st = check_tensors(a);
  if (st != FM_OK) return st;
  const fm_kv_batch b = bounded_batch(*a.b);
  const Plan pl = plan_of(*a.c, b, a.H, window, sinks, meet);
  st = check_workspace(a, pl.workspace, meet && K == Keys::kAll ? "workspace smaller than fm_shared_attention_workspace_size()"
                                                                : "workspace smaller than fm_paged_attention_workspace_size()");
  if (st != FM_OK) return st;
  CUtensorMap tk, tv;
  if (!maps_of(a, pl.decode, &tk, &tv)) return record_error(FM_ERR_CUDA, "cuTensorMapEncodeTiled (cache pages) failed");
  AttnParams p;
  if (!params_of(a, b, p)) return record_error(FM_ERR_CUDA, "no error word on the current device");
  cudaError_t e = configure<K>();
  if (e != cudaSuccess) return record_error(FM_ERR_CUDA, cudaGetErrorString(e));
  p.window = window;
  p.sinks = sinks;
  use_plan(pl, p);
  if (pl.workspace) shares_in(a, pl.splits, b.tokens, p);
  const LaunchOpts o = opts_of(a);
  e = pl.decode ? decode_launch<K>(p, a.c->Dh, a.c->fmt == FM_FMT_FP8, tk, tv, o) : launch_tiles<K>(a, pl, b.n, p, tk, tv, o);
  if (e == cudaSuccess && pl.workspace) e = launch_join(a, p, o);
  return e == cudaSuccess ? FM_OK : record_error(FM_ERR_CUDA, cudaGetErrorString(e));
}

// ---- groups of forks

int check_groups(const fm_kv_groups* g) {
  if (!g) return record_error(FM_ERR_INVALID_ARG, "NULL groups");
  if (g->n < 0 || g->max_entries < 0 || g->max_shared < 0)
    return record_error(FM_ERR_SHAPE, "the groups' counts must not be negative");
  if (g->n > 65535) return record_error(FM_ERR_SHAPE, "up to 65535 groups");
  if (g->n > 0 && (!g->first || !g->shared)) return record_error(FM_ERR_INVALID_ARG, "the groups have no first or no shared");
  return FM_OK;
}

// How a batch in groups is computed: the prefixes by the tile kernel and what is behind them by the kernel for few rows, or
// all keys of an entry together as without groups.
struct SharedPlan {
  bool split;        // prefixes by themselves
  Plan prefix;
  int own_splits;
  int tokens;        // of a group
  size_t workspace;
};

// A tile of 64 keys in the kernel for few rows, in units of 0.01 us: bf16 waits for its bytes however many CTAs share an SM,
// E4M3 with 16 rows for its own instructions.
int64_t decode_each(bool f8, int rows, int resident, int64_t ctas, int sms) {
  if (!f8) return rows <= 8 ? 55 : 60;
  return rows <= 8 ? 30 + 20 * std::min<int64_t>(resident, (ctas + sms - 1) / sms) : 110;
}

// Time of a batch without groups, in units of 0.1 us as splits_of takes it, from the same measurements.
int64_t cost_alone(const fm_kv_cache& c, const fm_kv_batch& b, int H, const Plan& pl) {
  const int sms = sm_count();
  const bool f8 = c.fmt == FM_FMT_FP8;
  const int64_t rows = static_cast<int64_t>(b.max_tokens) * (H / c.Hkv), len = std::max(1, b.max_len);
  if (pl.decode) {
    const int64_t ctas = static_cast<int64_t>(c.Hkv) * b.n * pl.splits, tiles = (len + kDecodeKeys - 1) / kDecodeKeys;
    const int resident = decode_resident(c.Dh, f8, static_cast<int>(rows));
    const int64_t waves = (ctas + static_cast<int64_t>(sms) * resident - 1) / (static_cast<int64_t>(sms) * resident);
    const int64_t each = decode_each(f8, static_cast<int>(rows), resident, ctas, sms);
    return (rows <= 8 ? 55 : 65) + waves * ((tiles + pl.splits - 1) / pl.splits) * each / 10 + (pl.splits > 8 ? 25 : 0);
  }
  const int64_t ctas = pl.row_blocks * c.Hkv * b.n * pl.splits;
  return (ctas + sms - 1) / sms * cta_time(f8, pl.alt, pl.split_tiles) + join_time(c, b, H, pl);
}

// Two kernels in a row cost 11 to 13 us with nothing to do, one 6 to 7, so sharing pays where entries x shared tokens are
// many: 96 single tokens of 16 heads on 2 KV heads (Dh 128, bf16) behind 2000 common keys take 14.8 us here and 24.3 us
// alone, 32 behind 8000 17.4 and 22.9 us; but 96 behind 500 13.1 and 11.3 us, 8 behind 8000 15.2 and 11.5 us. More than 128
// rows of an entry are not shared: own keys have the kernel for up to 16 rows alone, whose CTAs would all re-read them (16 x up to
// 50 tokens behind 4100: 43 us in two kernels, 39 alone).
SharedPlan shared_plan(const fm_kv_cache& c, const fm_kv_batch& b, const fm_kv_groups& g, int H) {
  SharedPlan sp = {};
  const int G = H / c.Hkv, sms = sm_count();
  const bool f8 = c.fmt == FM_FMT_FP8;
  const Plan alone = plan_of(c, b, H, 0, 0, true);
  sp.workspace = alone.workspace;
  sp.tokens = static_cast<int>(std::min<int64_t>(b.tokens, static_cast<int64_t>(g.max_entries) * b.max_tokens));
  const int64_t rows = static_cast<int64_t>(sp.tokens) * G, entry_rows = static_cast<int64_t>(b.max_tokens) * G;
  if (g.n == 0 || rows == 0 || g.max_shared == 0 || rows > (int64_t(1) << 30) || entry_rows > kTileRows) return sp;
  Plan& pre = sp.prefix;
  pre.alt = rows <= kTileRows;
  const int64_t block_rows = pre.alt ? kTileRows : 2 * kTileRows;
  pre.row_blocks = (rows + block_rows - 1) / block_rows;
  // blocks that have rows, by the packed rows: the bounds of one group or entry would count more
  const int64_t packed = static_cast<int64_t>(b.tokens) * G;
  const int64_t units = c.Hkv * std::min(pre.row_blocks * g.n, packed / block_rows + g.n);
  const int64_t tiles = (static_cast<int64_t>(g.max_shared) + kTileRows - 1) / kTileRows;
  const int block = entry_rows <= 8 ? 8 : kDecodeRows;
  const int64_t own_units = c.Hkv * std::min(b.n * ((entry_rows + block - 1) / block), packed / block + b.n);
  const int64_t own_tiles = (std::max<int64_t>({1, b.max_tokens, int64_t(b.max_len) - g.max_shared}) + kDecodeKeys - 1) / kDecodeKeys + 1;
  const int resident = own_resident(c.Dh, f8, block);
  const bool fewer_stages = resident > decode_resident(c.Dh, f8, block);
  if (c.Hkv > 8191) return sp;   // x blocks of an entry's rows are a dimension of the grid
  // The least of max(prefix, own keys) + the join + what of the second kernel finds no SM beside the first: its CTAs stay
  // until the prefix's shares are there, and those left over take their whole time behind it (8 us for 288 CTAs where 280
  // fit, 96 entries behind 500 keys). So neither takes more CTAs than it needs.
  const int64_t most = std::min<int64_t>({kMostPrefixSplits, tiles, std::max(1, 65535 / g.n)});
  int64_t best = 0;
  for (int64_t s = 1; s <= most; ++s) {
    const int64_t longest = (tiles + s - 1) / s;
    if (s > 1 && longest == (tiles + s - 2) / (s - 1)) continue;   // no shorter than with fewer
    const int64_t ctas = units * s, waves = (ctas + sms - 1) / sms, shares = s * b.tokens * H * c.Dh * 8;
    const int64_t prefix = waves * cta_time(f8, pre.alt, longest) + shares / 400000 + s * 6 / 10;
    const int64_t room = (waves * sms - ctas) * resident;
    for (int k = 1; k <= 8 && 2 * k <= own_tiles + 2; k *= 2) {   // own keys' splits: whole clusters find room
      const int64_t each = decode_each(f8, block, resident, own_units * k, sms) + (fewer_stages ? 20 : 0);
      const int64_t own = 55 + (own_tiles + k - 1) / k * each / 10, left = std::max<int64_t>(0, own_units * k - room);
      const int64_t cost = std::max(prefix, own) + 35 + (left + sms * resident - 1) / (sms * resident) * own;
      if (best == 0 || cost < best) {
        best = cost;
        pre.splits = static_cast<int>(s);
        sp.own_splits = k;
      }
    }
  }
  if (best * 11 / 10 >= cost_alone(c, b, H, alone)) return sp;   // 10 % that the estimate may be off
  pre.split_tiles = static_cast<int>((tiles + pre.splits - 1) / pre.splits);
  rings_of(c, pre);
  sp.split = true;
  // a place behind the shares' for the word between the two kernels: the size counts whole places
  sp.workspace = static_cast<size_t>(pre.splits + 1) * b.tokens * H * (c.Dh * sizeof(float) + sizeof(float2));
  return sp;
}

int attend_shared(const Call& a, const fm_kv_groups* g) {
  int st = check_call(a);
  if (st == FM_OK) st = check_groups(g);
  if (st != FM_OK) return st;
  if (nothing_to_do(*a.b)) return FM_OK;
  st = check_tensors(a);
  if (st != FM_OK) return st;
  const fm_kv_batch b = bounded_batch(*a.b);
  const SharedPlan sp = shared_plan(*a.c, b, *g, a.H);
  if (!sp.split) return attend<Keys::kAll>(a, 0, 0, true);
  st = check_workspace(a, sp.workspace, "workspace smaller than fm_shared_attention_workspace_size()");
  if (st != FM_OK) return st;
  CUtensorMap tk, tv, ok, ov;
  if (!maps_of(a, false, &tk, &tv) || !maps_of(a, true, &ok, &ov))
    return record_error(FM_ERR_CUDA, "cuTensorMapEncodeTiled (cache pages) failed");
  AttnParams p;
  if (!params_of(a, b, p)) return record_error(FM_ERR_CUDA, "no error word on the current device");
  cudaError_t e = configure<Keys::kPrefix>();
  if (e != cudaSuccess) return record_error(FM_ERR_CUDA, cudaGetErrorString(e));
  shares_in(a, sp.prefix.splits, b.tokens, p);
  p.seen = reinterpret_cast<uint64_t*>(p.part_ml + static_cast<size_t>(sp.prefix.splits) * b.tokens * a.H);
  p.g_first = g->first;
  p.g_shared = g->shared;
  p.g_n = g->n;
  p.g_tokens = sp.tokens;
  p.prefix_splits = sp.prefix.splits;
  const LaunchOpts o = opts_of(a);
  use_plan(sp.prefix, p);
  e = launch_tiles<Keys::kPrefix>(a, sp.prefix, g->n, p, tk, tv, o);
  if (e == cudaSuccess) {
    p.splits = sp.own_splits;
    e = decode_launch<Keys::kOwn>(p, a.c->Dh, a.c->fmt == FM_FMT_FP8, ok, ov, o);
  }
  return e == cudaSuccess ? FM_OK : record_error(FM_ERR_CUDA, cudaGetErrorString(e));
}

}  // namespace

}  // namespace fm

extern "C" int fm_paged_attention_workspace_size(const fm_kv_cache* c, const fm_kv_batch* b, int H, size_t* bytes) {
  if (!bytes) return fm::record_error(FM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = fm::check(c, b, H);
  if (st != FM_OK) return st;
  *bytes = b->n && b->tokens ? fm::plan_of(*c, fm::bounded_batch(*b), H, 0, 0, false).workspace : 0;
  return FM_OK;
}

extern "C" int fm_paged_attention(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const uint16_t* q,
                                  int64_t q_stride, int H, float scale, int causal, int window, uint16_t* out,
                                  int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  return fm::attend<fm::Keys::kAll>({c, layer, b, q, q_stride, H, scale, causal, out, out_stride, workspace, workspace_bytes, stream},
                                    window, 0, false);
}

extern "C" int fm_sink_attention(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const uint16_t* q, int64_t q_stride,
                                 int H, float scale, int causal, int window, int sinks, uint16_t* out, int64_t out_stride,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  using namespace fm;
  if (sinks < 0) return record_error(FM_ERR_INVALID_ARG, "sinks must not be negative");
  const Call a{c, layer, b, q, q_stride, H, scale, causal, out, out_stride, workspace, workspace_bytes, stream};
  // without a window nothing is hidden, without first tokens nothing is kept: the same attention in one stretch of keys
  return window <= 0 || sinks == 0 ? attend<Keys::kAll>(a, window, 0, false) : attend<Keys::kSinks>(a, window, sinks, true);
}

extern "C" int fm_shared_attention_workspace_size(const fm_kv_cache* c, const fm_kv_batch* b, const fm_kv_groups* g, int H,
                                                  size_t* bytes) {
  if (!bytes) return fm::record_error(FM_ERR_INVALID_ARG, "bytes is NULL");
  int st = fm::check(c, b, H);
  if (st == FM_OK) st = fm::check_groups(g);
  if (st != FM_OK) return st;
  *bytes = fm::nothing_to_do(*b) ? 0 : fm::shared_plan(*c, fm::bounded_batch(*b), *g, H).workspace;
  return FM_OK;
}

extern "C" int fm_shared_attention(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const fm_kv_groups* g,
                                   const uint16_t* q, int64_t q_stride, int H, float scale, int causal, uint16_t* out,
                                   int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  return fm::attend_shared({c, layer, b, q, q_stride, H, scale, causal, out, out_stride, workspace, workspace_bytes, stream}, g);
}

extern "C" int fm_test_paged_plan(const fm_kv_cache* c, const fm_kv_batch* b, const fm_kv_groups* g, int H, int window, int sinks,
                                  fm_paged_plan* plan) {
  using namespace fm;
  if (!plan) return record_error(FM_ERR_INVALID_ARG, "plan is NULL");
  int st = check(c, b, H);
  if (st == FM_OK && g) st = check_groups(g);
  if (st != FM_OK) return st;
  if (window < 0 || sinks < 0 || (g && (window || sinks)))
    return record_error(FM_ERR_INVALID_ARG, "window and sinks must not be negative, and 0 with groups");
  *plan = {};
  if (nothing_to_do(*b)) return FM_OK;
  const fm_kv_batch bounded = bounded_batch(*b);
  const bool first_tokens = window > 0 && sinks > 0;
  const SharedPlan sp = g ? shared_plan(*c, bounded, *g, H) : SharedPlan{};
  const Plan pl = sp.split ? sp.prefix : plan_of(*c, bounded, H, window, first_tokens ? sinks : 0, g || first_tokens);
  plan->few_rows = pl.decode;
  plan->row_tiles = pl.decode ? 0 : pl.alt ? 1 : 2;
  plan->splits = pl.splits;
  plan->cluster = pl.decode && pl.splits > 1 && !pl.workspace ? pl.splits : pl.cluster;
  if (plan->cluster)
    plan->clusters_at_once = pl.decode ? decode_clusters_at_once(c->Dh, c->fmt == FM_FMT_FP8, bounded.max_tokens * (H / c->Hkv), plan->cluster)
                                       : tile_clusters_at_once(plan->cluster);
  plan->own_splits = sp.split ? sp.own_splits : 0;
  return FM_OK;
}
