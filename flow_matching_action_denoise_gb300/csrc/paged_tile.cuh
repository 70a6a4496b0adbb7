// Attention of a chunk of new tokens over a paged cache: the kernel for many rows.
//
//   o[t, h] = sum_j p_j v_j,  p = softmax_j(scale q[t, h] . k_j),  key j of the token's sequence with
//   j < len, j <= pos(t) where causal, j > pos(t) - window where a window is set; a row without keys is zero.
//
// Work layout. The G = H / Hkv query heads of a KV head are stacked with the tokens into rows
// R = token * G + head, so that a key tile is read once for all of them. A CTA takes up to 256 rows of one
// entry and KV head and walks its keys in tiles of 128; S = Q K^T and O += P V run on tcgen05 tensor cores
// (M = 128) with both accumulators and P in tensor memory, one pass with the running maximum and sum.
// Two softmax warpgroups share the CTA. With more than 128 rows each owns a 128-row tile and both use every
// key tile; with up to 128 rows they own alternate key tiles of the same rows and merge at the end
// (`alt`), so that few rows keep two tiles in flight too (up to 16 rows have a kernel of their own). While one warpgroup exponentiates, the tensor cores
// work for the other. A long key axis with few rows is cut into splits of whole tiles, one CTA each, whose (max, sum, O)
// meet in their cluster's shared memory (up to 8) or in the workspace, where combine_kernel joins them in split order.
//
// Pages. One warp reads the page table and moves every page's rows by TMA straight into the swizzled tile the
// tensor cores read: values stay [token][head dim] and are read as an MN-major operand, so the cache needs no
// transpose. Pages outside the sequence are loaded from behind the pool's end, which TMA fills with zeros; the
// values behind the length inside the last page are zeroed in shared memory, since 0 * NaN is NaN.
//
// E4M3 cache. Four warps expand the codes to f16 (exact) into the same tile layout; q is scaled per row by a power
// of two that puts its largest element in [2^14, 2^15) and held in f16 (bf16's 8 significant bits are kept down to
// 2^-28 of that largest element), p is held in f16 times 2^6: finer than bf16 down to 2^-20 of the reference maximum's, below that in
// steps of 2^-30, which only shows where a row's largest p meet values of zero.
//
// Rounding: scores, statistics, P V sums and the splits' join are fp32; P is rounded to bf16 (f16 for the E4M3
// cache), the operand type of the second product; the output is rounded once to bf16. The running maximum moves
// only when it grows by more than 2^8 (in the exponent: 8), which makes rescaling O rare; the final division makes
// the result independent of that reference.
//
// Bounds and measurements. 4 Dh FLOP a head, query row and key on the tensor cores: 4096 tokens of 16 heads (2 KV heads,
// Dh 128) over 12288 keys, causal, take 253 us, 1.36 PFLOP/s, 70 % of the library's dense bf16 rate; E4M3 cache 269 us.
// What is missing: 256 CTAs fill 1.7 waves of 152, and inside a wave the tensor pipe is active for 60 % of the cycles
// (one wave of 256 rows over 4224 keys a CTA, 66 us): a tile's exponentials wait for its TMEM reads, which queue behind
// the other tile's MMAs. Small calls are bound by their ends: about 7 us a CTA from launch to the first scores and from
// the last products to the stored rows, 1.4 us a key tile of both query tiles between.

#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "kv.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace fm {

namespace {

constexpr int kTileRows = 128;    // rows of a query tile (MMA M) and keys of a key tile
// Warp roles behind the eight softmax warps: an MMA warp for each tile (one alone spent its time issuing: 16 MMAs, five
// waits and four commits a tile in sequence), TMA (and the tail's zeros), and with an E4M3 cache four that expand codes.
constexpr int kMmaWarp = 8, kTmaWarp = 10, kCvtWarp = 12, kCvtWarps = 4;
// Registers move to the softmax warpgroups, which keep 128 scores each: 384 x 168 = 256 x 224 + 128 x 56, 512 x 128 = 256 x 200 +
// 256 x 56 (8 fewer for them and 16 or 8 more for the others: 259.5 us against 254.5 for 4096 tokens over 12288 keys, E4M3 272.5
// against 269; 208 and 48 with E4M3 spill: 291 us).
constexpr int threads_of(bool f8) { return f8 ? 512 : 384; }
constexpr int kSmemLimit = 226 * 1024;
constexpr int kMaxRing = 8;
constexpr uint32_t kCtlBytes = 1024;

// Matrix descriptor of an MN-major operand in 128-byte-swizzled rows: rows along K (8-row groups 1024 bytes
// apart), 64 elements of MN per row, further blocks of 64 `block_bytes` apart.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t block_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(block_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// 16 bytes from global to shared memory, or 16 zero bytes (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool has) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(has ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint32_t swz(int r, int c) {   // 16-byte chunk c of row r of a 128-byte-row tile
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

// Every thread of the cluster: what one wrote before, in its shared memory, all can read behind.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Ctl {   // shared-memory control block
  uint64_t full[kMaxRing], empty[kMaxRing], rfull[kMaxRing], rempty[kMaxRing];
  uint64_t q_ready, s_full[2], p_full[2], o_done[2], turn[2], tail, drain[2];
  uint32_t tmem;
  float q_factor[kTileRows];   // E4M3 cache, alternate tiles: the scores' factor of every query row
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

// JOIN: the splits (p.cluster of them) meet in their cluster; as a variant of its own, since the join's registers cost all others
// 3 to 5 % with an E4M3 cache.
template <int DH, bool F8, Keys K, bool JOIN>
__global__ void __launch_bounds__(threads_of(F8), 1)
    paged_attn_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kHalves = DH / 64;                      // 128-byte blocks of a 16-bit row
  constexpr uint32_t kTileBytes = kTileRows * DH * 2;   // a 16-bit tile
  constexpr uint32_t kRawBytes = kTileRows * DH;        // a tile of E4M3 codes
  constexpr uint32_t kBlock = kTileRows * 128;          // one 128-byte-row block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int q_tiles = p.alt ? 1 : 2;
  uint8_t* sq = smem;
  uint8_t* sring = sq + q_tiles * kTileBytes;
  uint8_t* sraw = sring + p.ring * kTileBytes;
  Ctl& c = *reinterpret_cast<Ctl*>(sraw + (F8 ? p.raw_ring * kRawBytes : 0u));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // CTAs start in the order of their number. Row blocks go from the last one: with a causal mask it has most keys.
  const int g = p.rows_first ? blockIdx.x : blockIdx.y;
  const int row_block = p.row_blocks - 1 - static_cast<int>(p.rows_first ? blockIdx.z : blockIdx.x);
  const int place = p.rows_first ? blockIdx.y : blockIdx.z, entry = place / p.splits, split = place % p.splits;
  const int block_rows = q_tiles * kTileRows;

  // the CTA meets once, before anything is known of its entry; each role then goes as soon as its own data are there
  if (warp == kMmaWarp) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  } else if (warp == kTmaWarp) {
    if (elect_one()) {
      for (int i = 0; i < kMaxRing; ++i) {
        mbar_init(&c.full[i], F8 ? kCvtWarps : 1);
        mbar_init(&c.empty[i], p.alt ? 1 : 2);   // a key tile has one user, or both
        mbar_init(&c.rfull[i], 1);
        mbar_init(&c.rempty[i], kCvtWarps);
      }
      mbar_init(&c.q_ready, 8);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&c.s_full[t], 1);
        mbar_init(&c.p_full[t], 4);
        mbar_init(&c.o_done[t], 1);
      }
      mbar_init(&c.turn[0], 1);
      mbar_init(&c.turn[1], 1);
      mbar_init(&c.tail, 1);
      mbar_init(&c.drain[0], 1);
      mbar_init(&c.drain[1], 1);
      fence_mbar_init();
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
  }
  pdl_wait();
  if (K == Keys::kPrefix && tid == 0 && first_cta()) hand_inputs_on(p);

  // ---- the entry, its rows and its keys (the same in every thread)
  const bool report = tid == 0 && row_block == 0 && g == 0 && split == 0;
  const Entry en = K == Keys::kPrefix ? group_of(p, entry, report) : entry_of(p, entry, report);
  const bool shares = !JOIN && (K == Keys::kPrefix || p.splits > 1);   // the results go to the workspace
  const int begin = en.begin, nq = en.nq, len = en.len, sid = en.sid;
  const int rows = min(nq, K == Keys::kPrefix ? p.g_tokens : p.max_tokens) * p.G;   // <= 2^30
  const int row0 = row_block * block_rows;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // after TMEM is held
  const uint32_t tmem = c.tmem;
  if (row0 >= rows) {   // the same for the whole CTA
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    return;
  }

  const int past = len - nq;   // position of token i: past + i
  auto key_end = [&](int row) { return K == Keys::kPrefix ? len : last_key(p, past + row / p.G, len); };
  auto key_begin = [&](int row) { return K == Keys::kPrefix ? 0 : first_key(p, past + row / p.G); };
  const int last_row = min(rows, row0 + block_rows) - 1;
  const int hi_all = key_end(last_row);
  // t_lo, t_hi: places in the order of the key tiles
  const int t_first = key_begin(row0) / kTileRows;
  const Places<K> places(p, t_first, kTileRows);
  int t_lo = places.begin(t_first);
  int t_hi = places.place((hi_all + kTileRows - 1) / kTileRows);
  if (p.splits > 1) {
    t_lo += split * p.split_tiles;
    if (split < p.splits - 1) t_hi = min(t_hi, t_lo + p.split_tiles);   // the last one takes what is left
  }
  const int nt = max(0, t_hi - t_lo);   // key tiles of this CTA
  int n_of[2];
  if (p.alt) {
    n_of[0] = (nt + 1) / 2;
    n_of[1] = nt / 2;
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int lr = min(rows, row0 + (t + 1) * kTileRows) - 1;
      n_of[t] = lr < row0 + t * kTileRows
                    ? 0
                    : max(0, min(t_hi, places.place((key_end(lr) + kTileRows - 1) / kTileRows)) - t_lo);
    }
  }
  // Key tiles that some tile uses, and the tiles of each: n_of[0] <= n_of[1] except where tile 1 has no rows.
  const int n_keys = p.alt ? nt : max(n_of[0], n_of[1]);
  const int tail_tile = len % kTileRows ? places.place(len / kTileRows) - t_lo : -1;   // the tile that the length ends in

  [[maybe_unused]] float2* const cluster_ml = reinterpret_cast<float2*>(sq);   // JOIN: (log2 maximum, sum) of the rows, when the queries have been used
  const uint32_t ring_a = smem_u32(sring), raw_a = smem_u32(sraw), q_a = smem_u32(sq);

  // ---- the TMA warp's copies: one call moves the next key or value tile, a box for the rows of each page (at most
  // 128) and each 128-byte block.
  const int rows_box = min(p.page, kTileRows), boxes = kTileRows / rows_box;
  const int ring_n = F8 ? p.raw_ring : p.ring;
  uint64_t* const ring_full = F8 ? c.rfull : c.full;
  uint64_t* const ring_empty = F8 ? c.rempty : c.empty;
  constexpr uint32_t ring_bytes = F8 ? kRawBytes : kTileBytes;
  auto page_of = [&](int j) {   // lane x: the page of box x of key tile j; the pool's end where there is none
    const int key = places.tile(t_lo + j) * kTileRows + lane * rows_box;
    if (lane >= boxes || key >= len || j >= n_keys) return p.pages;
    const int pg = p.table[static_cast<int64_t>(sid) * p.table_stride + (key >> p.page_shift)];
    if (pg < 0 || pg >= p.pages) {
      atomicOr(p.err, kErrBadBatch);
      return p.pages;
    }
    return pg;
  };
  int copy_next = 0, copy_page = 0, copy_page_after = 0;
  Ring copy_at;
  auto copy_one = [&]() {
    const int j = copy_next >> 1, kv = copy_next & 1;
    if (kv == 0) {
      copy_page = copy_page_after;
      copy_page_after = page_of(j + 1);   // on its way while this tile's copies wait for their buffers
    }
    if (copy_next >= ring_n && !wait_for(&ring_empty[copy_at.b], copy_at.phase ^ 1)) return false;
    if (lane == 0) mbar_arrive_expect_tx(&ring_full[copy_at.b], ring_bytes);
    __syncwarp();
    // one lane issues all boxes: lanes that issue their own would be taken one after the other at twice the cost
    const CUtensorMap* map = kv ? &tm_v : &tm_k;
    const uint32_t dst = (F8 ? raw_a : ring_a) + copy_at.b * ring_bytes;
    for (int x = 0; x < boxes; ++x) {
      const int pg = __shfl_sync(0xffffffffu, copy_page, x);
      const int row_in = (places.tile(t_lo + j) * kTileRows + x * rows_box) & (p.page - 1);
      if (elect_one()) {
        if constexpr (F8) {
          tma_load_4d(dst + x * rows_box * DH, map, &ring_full[copy_at.b], 0, row_in, g, pg);
        } else {
#pragma unroll
          for (int h = 0; h < kHalves; ++h)
            tma_load_4d(dst + h * kBlock + x * rows_box * 128, map, &ring_full[copy_at.b], h * 64, row_in, g, pg);
        }
      }
      __syncwarp();
    }
    ++copy_next;
    copy_at.next(ring_n);
    return true;
  };

  // ---- the softmax warps' query rows: kRowChunks lanes a row, kStep rows a warp at a time
  constexpr int kRowChunks = DH / 8;          // 16-byte chunks of a 16-bit row
  constexpr int kStep = 32 / kRowChunks;
  constexpr int kSteps = 32 / kStep;
  const int t_of = (warp >> 2) & 1, wq = warp & 3;
  const int tile_row0 = row0 + (p.alt ? 0 : t_of * kTileRows);
  const int lane_row = lane / kRowChunks, lane_chunk = lane % kRowChunks;
  // Walks a lane's rows (every kStep-th) in an array [token][head][DH] by additions alone; G comes in opaque, so that
  // nothing of a walk is kept in registers for the next one. Elements are counted.
  struct Walk {
    int64_t at, step, wrap;   // the row's place, the way to the next, and more where that is another token
    int head, step_head, G;
    __device__ __forceinline__ Walk(int row, int group, int64_t tok_stride, int64_t from) : G(group) {
      asm volatile("" : "+r"(G));
      const int tok = row / G, step_tok = kStep / G;
      head = row - tok * G;
      step_head = kStep - step_tok * G;
      at = from + tok * tok_stride + head * DH;
      step = step_tok * tok_stride + step_head * DH;
      wrap = tok_stride - static_cast<int64_t>(G) * DH;
    }
    __device__ __forceinline__ void next() {
      at += step;
      head += step_head;
      if (head >= G) {
        head -= G;
        at += wrap;
      }
    }
  };
  // Byte offset of this lane's chunk of its i-th row inside a tile of 128-byte-row blocks (128-byte swizzle), and inside
  // a warp's 32 staged rows of DH * 2 bytes: kStep is 2 or 4, so that all but i is the lane's own.
  const uint32_t tile_lane = (lane_chunk >> 3) * kBlock + (wq * 32 + lane_row) * 128 + (((lane_chunk & 7) ^ lane_row) << 4);
  const uint32_t stage_lane = lane_row * (DH * 2) + ((lane_chunk ^ lane_row) << 4);
  auto tile_at = [&](int i) { return (tile_lane + i * kStep * 128) ^ (((i * kStep) & 7) << 4); };
  auto stage_at = [&](int i) { return (stage_lane + i * kStep * (DH * 2)) ^ (((i * kStep) & 7) << 4); };
  // What runs once a CTA: independent steps without divisions or clocks between them (as a loop of dependent ones the
  // 16 copies took 3000 cycles to issue).
  const uint32_t q_tile = q_a + (p.alt ? 0 : t_of * kTileBytes);
  if (warp < 8) {   // the rows go to their place in the swizzled tile; of one tile each warpgroup takes every other step
    Walk walk(tile_row0 + wq * 32 + lane_row, p.G, p.q_stride, begin * p.q_stride + g * p.G * DH + lane_chunk * 8);
    const int left = rows - tile_row0 - wq * 32 - lane_row;   // rows from this lane's first one on
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const bool has = i * kStep < left;
      if (!p.alt || (i & 1) == t_of) cp_async16_or_zero(q_tile + tile_at(i), p.q + (has ? walk.at : 0), has);
      walk.next();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  } else if (warp == kTmaWarp) {
    copy_page_after = page_of(0);
  }

  // one instruction for a whole warpgroup
  if (warp < 8) {
    if constexpr (F8)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  }

  if (warp < 8) {
    // ================================================= softmax warpgroups
    const int t = t_of;
    const int r = wq * 32 + lane;
    const int row = tile_row0 + r;
    const bool live = row < rows;
    const bool warp_live = row - lane < rows;
    asm volatile("cp.async.wait_all;" ::: "memory");
    float c_row = p.scale_log2;
    if constexpr (F8) {
      // Every thread turns its own row into f16, scaled by 2^(14 - exponent of its largest element): exact, and the
      // inverse goes into the scores' factor.
      __syncwarp();
      if (p.alt) asm volatile("bar.sync 1, 256;" ::: "memory");   // the other warpgroup's copies
      if ((!p.alt || t == 0) && warp_live) {
        uint4* mine = reinterpret_cast<uint4*>(sq + (p.alt ? 0 : t * kTileBytes) + r * 128);
        uint4 v[kRowChunks];
        uint32_t top = 0;   // largest |q| of the row as bf16 bits
#pragma unroll
        for (int ch = 0; ch < kRowChunks; ++ch) {
          v[ch] = mine[(ch >> 3) * (kBlock / 16) + ((ch & 7) ^ (r & 7))];
          const uint32_t w[4] = {v[ch].x, v[ch].y, v[ch].z, v[ch].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
        }
        const int ex = static_cast<int>(top >> 7);   // biased exponent (0: zero or subnormal; 255: not finite)
        const int sh = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -100), 100);   // 127 + 14 - ex
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        c_row *= __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * *p.k_scale;
#pragma unroll
        for (int ch = 0; ch < kRowChunks; ++ch) {
          uint32_t w[4] = {v[ch].x, v[ch].y, v[ch].z, v[ch].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack16<true>(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
          mine[(ch >> 3) * (kBlock / 16) + ((ch & 7) ^ (r & 7))] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      if (p.alt) {   // the other warpgroup's scores are of the same rows
        if (t == 0) c.q_factor[r] = c_row;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        c_row = c.q_factor[r];
      }
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.q_ready);
    // rows behind the last one need no mask: what they compute is not used
    const int my_end = live ? key_end(row) : 0x7fffffff, my_begin = live ? key_begin(row) : 0;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t t_s = t_lane + t * 128, t_o = t_lane + 256 + t * 128;
    const int n = n_of[t];
    float m = -INFINITY;                    // the reference maximum, in score units
    float m_grow = -INFINITY;               // a maximum above this moves it
    constexpr float kShift = F8 ? 6.0f : 0.0f;   // f16 probabilities are held 2^6 larger: subnormals begin lower
    float off = kShift;                     // -m in log2 units
    const float grow_by = kGrow / c_row;
    float2 sum2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      ok = wait_for(&c.s_full[t], i & 1);
      if (!ok) break;
      tc_fence_after();
      __syncwarp();
      if (!warp_live) {
        if (lane == 0) mbar_arrive(&c.p_full[t]);
        continue;
      }
      const int k0 = places.tile(t_lo + (p.alt ? 2 * i + t : i)) * kTileRows;
      float s[128];
      int lo = my_begin - k0;
      const int hi = my_end - k0;
      [[maybe_unused]] const int seen = p.sinks - k0;   // keys of the first tokens
      if (K == Keys::kSinks && seen >= kTileRows) lo = 0;
      const bool edge = __any_sync(0xffffffffu, lo > 0 || hi < kTileRows);
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld32_async(t_s + b * 32, s + b * 32);
      tmem_wait_ld();
      if (edge) {
        // One comparison an element where the warp's rows allow it: a window's tiles have mostly one kind of edge each (9 chunks
        // of up to 333 tokens, window 300 + first 37: 19.5 us with all comparisons everywhere, 16.0 with one).
        const bool low = __any_sync(0xffffffffu, lo > 0), high = __any_sync(0xffffffffu, hi < kTileRows);
        if (K == Keys::kSinks && seen > 0) {
          if (high || __any_sync(0xffffffffu, lo < kTileRows)) {
#pragma unroll
            for (int e = 0; e < 128; ++e) s[e] = (e >= lo || e < seen) && e < hi ? s[e] : -INFINITY;
          } else {
#pragma unroll
            for (int e = 0; e < 128; ++e) s[e] = e < seen ? s[e] : -INFINITY;
          }
        } else if (K == Keys::kAll || (low && high)) {
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] = e >= lo && e < hi ? s[e] : -INFINITY;
        } else if (low) {
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] = e >= lo ? s[e] : -INFINITY;
        } else {
#pragma unroll
          for (int e = 0; e < 128; ++e) s[e] = e < hi ? s[e] : -INFINITY;
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int e = 4; e < 124; e += 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmaxf(mx[j], s[e + j]), s[e + 4 + j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], s[124 + j]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      const bool grow = top > m_grow;
      if (__any_sync(0xffffffffu, grow)) {
        float f = 1.0f;
        if (grow) {
          f = ex2_approx((m - top) * c_row);   // 0 for a row's first keys
          m = top;
          m_grow = top + grow_by;
          off = kShift - m * c_row;
#pragma unroll
          for (int j = 0; j < 4; ++j) sum2[j].x *= f, sum2[j].y *= f;
        }
        // the P V product of the tile before has completed: these scores were issued after it
        if (i > 0) {
#pragma unroll 1
          for (int b = 0; b < DH; b += 16) {
            float o[16];
            tmem_ld16(t_o + b, o);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
            tmem_st16(t_o + b, w);
          }
        }
      }
      const float2 c2 = make_float2(c_row, c_row), off2 = make_float2(off, off);
      auto probabilities = [&](int from, int pairs, uint32_t* w) {
#pragma unroll
        for (int e = 0; e < pairs; ++e) {
          const int k = from + 2 * e;
          const float2 x = fma2(make_float2(s[k], s[k + 1]), c2, off2);
          s[k] = ex2_approx(x.x);
          s[k + 1] = ex2_approx(x.y);
          w[e] = pack16<F8>(s[k], s[k + 1]);
        }
      };
#pragma unroll
      for (int part = 0; part < (F8 ? 2 : 4); ++part) {   // narrow parts hold fewer registers (254.1 -> 252.4 us); E4M3: 269.4 -> 271.6
        if constexpr (F8) {
          uint32_t w[32];
          probabilities(part * 64, 32, w);
          tmem_st32(t_s + part * 32, w);
        } else {
          uint32_t w[16];
          probabilities(part * 32, 16, w);
          tmem_st16(t_s + part * 16, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.p_full[t]);
      // the sum is off the path of the tensor cores
#pragma unroll
      for (int e = 0; e < 128; e += 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sum2[j] = add2(sum2[j], make_float2(s[e + 2 * j], s[e + 2 * j + 1]));
      }
    }
    const float2 st = add2(add2(sum2[0], sum2[1]), add2(sum2[2], sum2[3]));
    float sum = st.x + st.y;
    float m2 = m > -INFINITY ? m * c_row : -INFINITY;   // log2 units
    // ---- the end: O complete, joined across the warpgroups (alternate tiles), stored
    if (p.alt) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (n_of[u] > 0) ok = wait_for(&c.o_done[u], 0) && ok;
    } else if (n > 0) {
      ok = wait_for(&c.o_done[t], 0) && ok;
    }
    tc_fence_after();
    __syncwarp();
    if (!ok && lane == 0) atomicOr(p.err, kErrPipelineTimeout);
    const float vs = F8 ? *p.v_scale : 1.0f;
    float* join = reinterpret_cast<float*>(sring);   // [128 or, for the cluster, 256][DH], chunks swizzled by row
    float2* join_ml = reinterpret_cast<float2*>(sring + kTileRows * DH * 4);
    if (JOIN && !p.alt) asm volatile("bar.sync 1, 256;" ::: "memory");   // the other tile's products, too, have read the ring
    auto load_o = [&](int b, float* o) {   // 32 of this row's sums
      if (n > 0) {
        tmem_ld32_async(t_o + b, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
      }
    };
    if (p.alt) {
      if (t == 1 && warp_live) {
        join_ml[r] = make_float2(m2, sum);
#pragma unroll 1
        for (int b = 0; b < DH; b += 32) {
          float o[32];
          load_o(b, o);
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(join + r * DH + ((((b + e) >> 2) ^ (r & 7)) << 2)) =
                make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
    }
    if ((!p.alt || t == 0) && warp_live) {
      float w0 = 1.0f, w1 = 0.0f;
      if (p.alt) {
        const float2 b = join_ml[r];
        const float top = fmaxf(m2, b.x);
        w0 = m2 > -INFINITY ? ex2_approx(m2 - top) : 0.f;
        w1 = b.x > -INFINITY ? ex2_approx(b.x - top) : 0.f;
        sum = sum * w0 + b.y * w1;
        m2 = top;
      }
      const int64_t split_row = static_cast<int64_t>(split) * p.tokens * p.H;
      if (JOIN || shares) {
        const float2 ml = make_float2(m2, sum);
        if (JOIN)
          cluster_ml[row - row0] = ml;
        else if (live)
          p.part_ml[split_row + static_cast<int64_t>(begin + row / p.G) * p.H + g * p.G + row % p.G] = ml;
        w0 *= vs;
        w1 *= vs;
      } else {
        const float inv = sum == 0.f ? 0.f : vs / sum;
        w0 *= inv;
        w1 *= inv;
      }
      // TMEM gives a lane one row: rows are staged in the query tile's 32 rows of this warp (its last reader has
      // completed) and leave kRowChunks lanes a row, whole 16-byte chunks. fp32 shares take two passes.
      const uint32_t stage = q_a + (p.alt ? 0 : t * kTileBytes) + wq * 32 * DH * 2;
      const int passes = JOIN ? 0 : !shares ? 1 : nt > 0 ? 2 : 0;
      if (JOIN && nt > 0) {   // this CTA's part of the rows, for the cluster
        const int x0 = row - row0;
#pragma unroll 1
        for (int b = 0; b < DH; b += 32) {
          float o[32];
          load_o(b, o);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4* at = reinterpret_cast<float4*>(join + x0 * DH + ((((b + e) >> 2) ^ (r & 7)) << 2));
            float4 x = make_float4(o[e] * w0, o[e + 1] * w0, o[e + 2] * w0, o[e + 3] * w0);
            if (p.alt) {
              const float4 y = *at;
              x = make_float4(o[e] * w0 + y.x * w1, o[e + 1] * w0 + y.y * w1, o[e + 2] * w0 + y.z * w1, o[e + 3] * w0 + y.w * w1);
            }
            *at = x;
          }
        }
      }
#pragma unroll 1
      for (int pass = 0; pass < passes; ++pass) {
        const int dims = shares ? DH / 2 : DH, d0 = pass * dims;
#pragma unroll 1
        for (int b = 0; b < dims; b += 32) {
          float o[32];
          load_o(d0 + b, o);
          if (p.alt) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(join + r * DH + ((((d0 + b + e) >> 2) ^ (r & 7)) << 2));
              o[e] = o[e] * w0 + x.x * w1;
              o[e + 1] = o[e + 1] * w0 + x.y * w1;
              o[e + 2] = o[e + 2] * w0 + x.z * w1;
              o[e + 3] = o[e + 3] * w0 + x.w * w1;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= w0;
          }
          if (shares) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              st_shared_v4(stage + lane * (DH * 2) + ((((b + e) >> 2) ^ (lane & 7)) << 4),
                           make_uint4(__float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                                      __float_as_uint(o[e + 3])));
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              st_shared_v4(stage + lane * (DH * 2) + ((((b + e) >> 3) ^ (lane & 7)) << 4),
                           make_uint4(pack16<false>(o[e], o[e + 1]), pack16<false>(o[e + 2], o[e + 3]),
                                      pack16<false>(o[e + 4], o[e + 5]), pack16<false>(o[e + 6], o[e + 7])));
          }
        }
        __syncwarp();
        const int left = rows - tile_row0 - wq * 32 - lane_row;
        const uint8_t* staged = sq + (p.alt ? 0 : t * kTileBytes) + wq * 32 * DH * 2;
        if (shares) {   // shares: [split][token][head][DH], this pass's half of the dims
          Walk walk(tile_row0 + wq * 32 + lane_row, p.G, static_cast<int64_t>(p.H) * DH,
                    (split_row + static_cast<int64_t>(begin) * p.H + g * p.G) * DH + d0 + lane_chunk * 4);
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            if (i * kStep < left) *reinterpret_cast<uint4*>(p.part_o + walk.at) = *reinterpret_cast<const uint4*>(staged + stage_at(i));
            walk.next();
          }
        } else {
          Walk walk(tile_row0 + wq * 32 + lane_row, p.G, p.out_stride, begin * p.out_stride + g * p.G * DH + lane_chunk * 8);
#pragma unroll
          for (int i = 0; i < kSteps; ++i) {
            if (i * kStep < left) *reinterpret_cast<uint4*>(p.out + walk.at) = *reinterpret_cast<const uint4*>(staged + stage_at(i));
            walk.next();
          }
        }
        __syncwarp();
      }
    }
    if constexpr (JOIN) {
      // ---- the cluster's splits are joined in split order, with the arithmetic of combine_kernel: rows go round the CTAs, 8 kPer
      // of them a step, a warp kPer at a time; R steps' loads from S splits are on their way together
      __syncwarp();
      cluster_meet();
      constexpr int kRowLanes = DH / 4, kPer = 32 / kRowLanes;
      const int rank = cluster_rank(), chunk = lane % kRowLanes, cs = p.cluster, n_rows = last_row - row0 + 1;
      const uint32_t o_a = smem_u32(sring), ml_a = smem_u32(cluster_ml);
      auto join_rows = [&](auto r_, auto s_) {
        constexpr int R = decltype(r_)::value, S = decltype(s_)::value;
        for (int base = (rank * 8 + warp) * kPer + lane / kRowLanes; base < n_rows; base += R * cs * 8 * kPer) {
          float2 ml[R][S];
          float w[R][S];
          float4 v[R][S];
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int x = base + i * cs * 8 * kPer;
#pragma unroll
            for (int s = 0; s < S; ++s) {
              ml[i][s] = make_float2(-INFINITY, 0.f);
              if (s < cs && x < n_rows)
                asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                             : "=f"(ml[i][s].x), "=f"(ml[i][s].y)
                             : "r"(map_dsmem(ml_a + x * 8, s)));
            }
          }
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int x = base + i * cs * 8 * kPer;
            float top = -INFINITY;
#pragma unroll
            for (int s = 0; s < S; ++s) top = fmaxf(top, ml[i][s].x);
#pragma unroll
            for (int s = 0; s < S; ++s) {
              // no keys: no share. A NaN in the query has no maximum either, but its sum is NaN and so is the row
              const bool none = ml[i][s].x == -INFINITY && ml[i][s].y == 0.f;
              w[i][s] = none ? 0.f : exp2f(ml[i][s].x - top);
              v[i][s] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (!none)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(v[i][s].x), "=f"(v[i][s].y), "=f"(v[i][s].z), "=f"(v[i][s].w)
                             : "r"(map_dsmem(o_a + x * DH * 4 + ((chunk ^ (x & 7)) << 4), s)));
            }
          }
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int x = base + i * cs * 8 * kPer;
            // four splits in a row, more by turns in two sums
            constexpr int kSums = S > 4 ? 2 : 1;
            float sum[2] = {0.f, 0.f};
            float4 acc[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
            for (int s = 0; s < S; ++s) {
              float4& a = acc[s % kSums];
              sum[s % kSums] = fmaf(ml[i][s].y, w[i][s], sum[s % kSums]);
              a = make_float4(fmaf(w[i][s], v[i][s].x, a.x), fmaf(w[i][s], v[i][s].y, a.y), fmaf(w[i][s], v[i][s].z, a.z),
                              fmaf(w[i][s], v[i][s].w, a.w));
            }
            if constexpr (kSums == 2) {
              sum[0] += sum[1];
              acc[0] = make_float4(acc[0].x + acc[1].x, acc[0].y + acc[1].y, acc[0].z + acc[1].z, acc[0].w + acc[1].w);
            }
            if (x >= n_rows) continue;
            const int in_entry = row0 + x, tok = in_entry / p.G;
            const int64_t token = begin + tok;
            const int head = g * p.G + in_entry - tok * p.G;
            const float inv = sum[0] == 0.f ? 0.f : 1.0f / sum[0];
            *reinterpret_cast<uint2*>(p.out + token * p.out_stride + head * DH + chunk * 4) =
                make_uint2(pack16<false>(acc[0].x * inv, acc[0].y * inv), pack16<false>(acc[0].z * inv, acc[0].w * inv));
          }
        }
      };
      using std::integral_constant;
      if (cs <= 2)
        join_rows(integral_constant<int, 4>{}, integral_constant<int, 2>{});
      else if (cs <= 4)
        join_rows(integral_constant<int, 2>{}, integral_constant<int, 4>{});
      else
        join_rows(integral_constant<int, 1>{}, integral_constant<int, 8>{});
      __syncwarp();
      cluster_arrive();   // behind this warp's reads: no CTA leaves while another still reads its part
      cluster_wait();
    }
  } else if (warp < kTmaWarp) {
    // ================================================= tensor cores, a warp for each tile
    // f32 accumulate; bf16 operands (code 1) or f16 (code 0); bit 16: the second operand MN-major
    constexpr uint32_t fmt = F8 ? 0u : ((1u << 7) | (1u << 10));
    constexpr uint32_t id_s = (1u << 4) | fmt | ((128u >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t id_o = (1u << 4) | fmt | (1u << 16) | ((static_cast<uint32_t>(DH) >> 3) << 17) | ((128u >> 4) << 24);
    const int t = warp - kMmaWarp;
    const int n = n_of[t];
    const uint32_t t_s = tmem + t * 128, t_o = tmem + 256 + t * 128;
    // Buffers alternate between the keys and the values of the key tiles in order. Tile t walks all of them, or every
    // other one. ks, vs: the next keys' and values' place in the ring.
    const int step = p.alt ? 4 : 2;
    Ring ks, vs;
    vs.next(p.ring);
    if (p.alt && t == 1) {
      for (int x = 0; x < 2; ++x) {
        ks.next(p.ring);
        vs.next(p.ring);
      }
    }
    const int tail_i = tail_tile < 0 ? -1 : (p.alt ? ((tail_tile & 1) == t ? tail_tile >> 1 : -1) : tail_tile);
    const uint64_t qd = sw128_kmajor_desc(q_a + (p.alt ? 0 : t * kTileBytes));
    bool ok = wait_for(&c.q_ready, 0);
    auto scores = [&](uint64_t kd) {
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x)   // descriptor addresses count 16 bytes
          tc_mma<false>(t_s, qd + ((h * kBlock + x * 32) >> 4), kd + ((h * kBlock + x * 32) >> 4), id_s, (h | x) ? 1u : 0u);
    };
    auto advance = [&](Ring& r) {
      for (int x = 0; x < step; ++x) r.next(p.ring);
    };
    if (n > 0) {
      ok = ok && wait_for(&c.full[ks.b], ks.phase);
      tc_fence_after();
      const uint64_t kd = sw128_kmajor_desc(ring_a + ks.b * kTileBytes);
      if (ok && elect_one()) {
        scores(kd);
        tc_commit(&c.s_full[t]);
        tc_commit(&c.empty[ks.b]);
      }
      __syncwarp();
      advance(ks);
    }
    // The two warps take turns on the tensor cores, a batch of P V and the next scores each: interleaved, both tiles'
    // products would end late and both warpgroups would then exponentiate at the same time. Everything a batch needs
    // is waited for before its turn, and the turn passes on before the commits, so that the queue of MMAs never drains.
    const int rounds = max(n_of[0], n_of[1]);
    for (int i = 0; i < rounds && ok; ++i) {
      const bool mine = i < n, more = i + 1 < n;
      if (mine)
        ok = wait_for(&c.full[vs.b], vs.phase) && (F8 || i != tail_i || wait_for(&c.tail, 0)) &&
             (F8 || !more || wait_for(&c.full[ks.b], ks.phase)) && wait_for(&c.p_full[t], i & 1);
      const uint64_t vd = sw128_mnmajor_desc(ring_a + vs.b * kTileBytes, kBlock);
      const uint64_t kd = sw128_kmajor_desc(ring_a + ks.b * kTileBytes);
      ok = ok && wait_for(&c.turn[t], t == 0 ? (i & 1) ^ 1 : i & 1);
      if (!ok) break;
      tc_fence_after();
      auto products = [&]() {
#pragma unroll
        for (int x = 0; x < 8; ++x) tc_mma_ts<false>(t_o, t_s + x * 8, vd + ((x * 2048) >> 4), id_o, (i | x) ? 1u : 0u);
      };
      if constexpr (F8) {
        // codes are expanded into four buffers only: the values' is given back before the next keys are waited for
        if (mine && elect_one()) {
          products();
          if (!more) tc_commit(&c.o_done[t]);
          tc_commit(&c.empty[vs.b]);
        }
        __syncwarp();
        if (more) {
          ok = wait_for(&c.full[ks.b], ks.phase);
          if (!ok) break;
          tc_fence_after();
        }
        if (elect_one()) {
          if (more) scores(kd);
          mbar_arrive(&c.turn[t ^ 1]);
          if (more) {
            tc_commit(&c.s_full[t]);
            tc_commit(&c.empty[ks.b]);
          }
        }
      } else if (elect_one()) {
        if (mine) {
          products();
          if (more) scores(kd);
        }
        mbar_arrive(&c.turn[t ^ 1]);
        if (mine) {
          if (more) {
            tc_commit(&c.s_full[t]);
            tc_commit(&c.empty[ks.b]);
          } else {
            tc_commit(&c.o_done[t]);
          }
          tc_commit(&c.empty[vs.b]);
        }
      }
      __syncwarp();
      if (mine) advance(vs);
      if (more) advance(ks);
      if (!mine && !p.alt) {   // a key tile that only the other one uses waits for this one's release all the same
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          Ring& at = kv ? vs : ks;
          ok = ok && wait_for(&c.full[at.b], at.phase);
          if (ok && lane == 0) mbar_arrive(&c.empty[at.b]);
          at.next(p.ring);
          at.next(p.ring);
        }
      }
    }
    if (!ok) {   // a wait ran out: let what was issued finish before the CTA leaves
      if (elect_one()) {
        atomicOr(p.err, kErrPipelineTimeout);
        tc_commit(&c.drain[t]);
      }
      __syncwarp();
      wait_for(&c.drain[t], 0);
    }
  } else if (warp == kTmaWarp) {
    // ================================================= page table and TMA
    bool ok = true;
    Ring last;   // the last copy's buffer
    while (copy_next < 2 * n_keys && ok) {
      last = copy_at;
      ok = copy_one();
    }
    if (!F8 && ok && tail_tile >= 0 && tail_tile == n_keys - 1) {
      // the values behind the length, in the last tile and so in the last buffer that was filled
      ok = wait_for(&c.full[last.b], last.phase);
      if (ok) {
        const int r0 = len % kTileRows;
        for (int x = lane; x < (kTileRows - r0) * 8 * kHalves; x += 32)
          st_shared_v4(ring_a + last.b * kTileBytes + (x % kHalves) * kBlock + r0 * 128 + (x / kHalves) * 16,
                       make_uint4(0, 0, 0, 0));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.tail);
      }
    }
    const int issued = copy_next, nb = ring_n;
    uint64_t* full = ring_full;
    if (!ok) {   // the copies in flight land before the CTA leaves
      if (lane == 0) atomicOr(p.err, kErrPipelineTimeout);
      for (int item = max(0, issued - nb); item < issued; ++item) wait_for(&full[item % nb], (item / nb) & 1);
    }
  } else if (F8 && warp >= kCvtWarp) {
    // ================================================= E4M3 codes -> f16 tiles
    const int ct = tid - kCvtWarp * 32;
    constexpr int kCvtThreads = kCvtWarps * 32;
    constexpr int kChunks = DH / 16;      // 16-code chunks of a row
    constexpr int kRowStep = kCvtThreads / kChunks;   // a multiple of 8: a thread's swizzle is the same in all its rows
    // this thread's rows cr, cr + kRowStep, ...; the two halves of a row write their two chunks in opposite orders, so
    // that eight lanes reach eight bank groups
    const int cr = ct / kChunks, ch = ct % kChunks, odd = (ch >> 2) & 1;
    const uint32_t dst = (ch >> 2) * kBlock;
    const uint32_t place0 = swz(cr, (ch & 3) * 2 + odd), place1 = swz(cr, (ch & 3) * 2 + 1 - odd);
    bool ok = true;
    Ring raw, out;
    for (int item = 0; item < 2 * n_keys && ok; ++item, raw.next(p.raw_ring), out.next(p.ring)) {
      const int rb = raw.b, b = out.b;
      ok = wait_for(&c.rfull[rb], raw.phase);
      if (ok && item >= p.ring) ok = wait_for(&c.empty[b], out.phase ^ 1);
      if (!ok) break;
      const int valid = len - places.tile(t_lo + (item >> 1)) * kTileRows;   // rows of the tile inside the length
      const uint4* src = reinterpret_cast<const uint4*>(sraw + rb * kRawBytes) + ct;
      constexpr int kIter = kTileRows / kRowStep;
      uint4 v[kIter];
#pragma unroll
      for (int x = 0; x < kIter; ++x) v[x] = src[x * kCvtThreads];
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.rempty[rb]);
      const uint32_t at = ring_a + b * kTileBytes + dst;
#pragma unroll
      for (int x = 0; x < kIter; ++x) {
        if (cr + x * kRowStep >= valid) v[x] = make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
        uint32_t h[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) expand4(w[e], h[2 * e], h[2 * e + 1]);
        const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), d = make_uint4(h[4], h[5], h[6], h[7]);
        st_shared_v4(at + x * kRowStep * 128 + place0, odd ? d : a);
        st_shared_v4(at + x * kRowStep * 128 + place1, odd ? a : d);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.full[b]);
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrPipelineTimeout);
  }
  __syncwarp();
  if (JOIN && warp >= 8) {   // the softmax warps' two meetings; these have read nothing of the others
    cluster_meet();
    cluster_arrive_relaxed();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

using TileKernel = void (*)(AttnParams, CUtensorMap, CUtensorMap);

template <Keys K, bool JOIN>
TileKernel tile_kernel(int Dh, bool f8) {
  return Dh == 128 ? (f8 ? paged_attn_kernel<128, true, K, JOIN> : paged_attn_kernel<128, false, K, JOIN>)
                   : (f8 ? paged_attn_kernel<64, true, K, JOIN> : paged_attn_kernel<64, false, K, JOIN>);
}

}  // namespace

// a prefix's shares are not joined here
template <Keys K>
constexpr bool kMayJoin = K != Keys::kPrefix;

template <Keys K>
cudaError_t tile_configure() {
  cudaError_t e = cudaSuccess;
  for (const int x : {0, 1, 2, 3})
    for (const bool join : {false, true}) {
      if (e != cudaSuccess || (join && !kMayJoin<K>)) continue;
      const auto kernel = join ? tile_kernel<K, kMayJoin<K>>(x & 1 ? 128 : 64, x & 2) : tile_kernel<K, false>(x & 1 ? 128 : 64, x & 2);
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit + 1024);
    }
  return e;
}

template <Keys K>
cudaError_t tile_launch(const AttnParams& p, int Dh, bool f8, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                        size_t smem, const LaunchOpts& o) {
  const auto kernel = p.cluster > 1 ? tile_kernel<K, kMayJoin<K>>(Dh, f8) : tile_kernel<K, false>(Dh, f8);
  return launch(kernel, grid, dim3(threads_of(f8)), smem, o, p, tk, tv);
}

}  // namespace fm
