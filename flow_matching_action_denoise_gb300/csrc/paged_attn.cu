// Attention of a chunk of new tokens over a paged cache (fm_paged_attention).
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
// work for the other. A long key axis with few rows is cut into splits of whole tiles, one CTA each, whose
// (max, sum, O) go to the workspace and are joined in split order by combine_kernel.
//
// Pages. One warp reads the page table and moves every page's rows by TMA straight into the swizzled tile the
// tensor cores read: values stay [token][head dim] and are read as an MN-major operand, so the cache needs no
// transpose. Pages outside the sequence are loaded from behind the pool's end, which TMA fills with zeros; the
// values behind the length inside the last page are zeroed in shared memory, since 0 * NaN is NaN.
//
// E4M3 cache. Four warps expand the codes to f16 (exact) into the same tile layout; q is scaled per row by a power
// of two that puts its largest element in [2^14, 2^15) and held in f16 (bf16's 8 significant bits are kept down to
// 2^-28 of that largest element), p is held in f16, so no rounding is coarser than for a 16-bit cache.
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

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

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

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
      "mov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// 16 bytes from global to shared memory, or 16 zero bytes (src is not read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool has) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(has ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint32_t swz(int r, int c) {   // 16-byte chunk c of row r of a 128-byte-row tile
  return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
}

struct Ctl {   // shared-memory control block
  uint64_t full[kMaxRing], empty[kMaxRing], rfull[kMaxRing], rempty[kMaxRing];
  uint64_t q_ready, s_full[2], p_full[2], o_done[2], turn[2], tail, drain[2];
  uint32_t tmem;
  float q_factor[kTileRows];   // E4M3 cache, alternate tiles: the scores' factor of every query row
};
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

template <int DH, bool F8>
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

  // ---- the entry, its rows and its keys (the same in every thread)
  const Entry en = entry_of(p, entry, tid == 0 && row_block == 0 && g == 0 && split == 0);
  const int begin = en.begin, nq = en.nq, len = en.len, sid = en.sid;
  const int rows = min(nq, p.max_tokens) * p.G;   // <= 2^30
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
  auto key_end = [&](int row) { return last_key(p, past + row / p.G, len); };
  auto key_begin = [&](int row) { return first_key(p, past + row / p.G); };
  const int last_row = min(rows, row0 + block_rows) - 1;
  const int hi_all = key_end(last_row);
  int t_lo = key_begin(row0) / kTileRows;
  int t_hi = (hi_all + kTileRows - 1) / kTileRows;
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
                    : max(0, min(t_hi, (key_end(lr) + kTileRows - 1) / kTileRows) - t_lo);
    }
  }
  // Key tiles that some tile uses, and the tiles of each: n_of[0] <= n_of[1] except where tile 1 has no rows.
  const int n_keys = p.alt ? nt : max(n_of[0], n_of[1]);
  const int tail_tile = len % kTileRows ? len / kTileRows - t_lo : -1;   // the tile that the length ends in

  const uint32_t ring_a = smem_u32(sring), raw_a = smem_u32(sraw), q_a = smem_u32(sq);

  // ---- the TMA warp's copies: one call moves the next key or value tile, a box for the rows of each page (at most
  // 128) and each 128-byte block.
  const int rows_box = min(p.page, kTileRows), boxes = kTileRows / rows_box;
  const int ring_n = F8 ? p.raw_ring : p.ring;
  uint64_t* const ring_full = F8 ? c.rfull : c.full;
  uint64_t* const ring_empty = F8 ? c.rempty : c.empty;
  constexpr uint32_t ring_bytes = F8 ? kRawBytes : kTileBytes;
  auto page_of = [&](int j) {   // lane x: the page of box x of key tile j; the pool's end where there is none
    const int key = (t_lo + j) * kTileRows + lane * rows_box;
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
      const int row_in = ((t_lo + j) * kTileRows + x * rows_box) & (p.page - 1);
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
      const int k0 = (t_lo + (p.alt ? 2 * i + t : i)) * kTileRows;
      float s[128];
      const int lo = my_begin - k0, hi = my_end - k0;
      const bool edge = __any_sync(0xffffffffu, lo > 0 || hi < kTileRows);
#pragma unroll
      for (int b = 0; b < 4; ++b) tmem_ld32_async(t_s + b * 32, s + b * 32);
      tmem_wait_ld();
      if (edge) {
#pragma unroll
        for (int e = 0; e < 128; ++e) s[e] = e >= lo && e < hi ? s[e] : -INFINITY;
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
    float* join = reinterpret_cast<float*>(sring);                        // [128][DH], chunks swizzled by row
    float2* join_ml = reinterpret_cast<float2*>(sring + kTileRows * DH * 4);
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
      if (p.splits > 1) {
        if (live) p.part_ml[split_row + static_cast<int64_t>(begin + row / p.G) * p.H + g * p.G + row % p.G] = make_float2(m2, sum);
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
      const int passes = p.splits == 1 ? 1 : nt > 0 ? 2 : 0;
#pragma unroll 1
      for (int pass = 0; pass < passes; ++pass) {
        const int dims = p.splits == 1 ? DH : DH / 2, d0 = pass * dims;
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
          if (p.splits > 1) {
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
        if (p.splits > 1) {   // shares: [split][token][head][DH], this pass's half of the dims
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
      const int valid = len - (t_lo + (item >> 1)) * kTileRows;   // rows of the tile inside the length
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
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

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

// The number of splits of a batch's keys. window 0: the one that the workspace is sized for.
int splits_of(const fm_kv_cache& c, const fm_kv_batch& b, int H, int window) {
  const int64_t rows = static_cast<int64_t>(b.max_tokens) * (H / c.Hkv);
  const int sms = sm_count();
  const bool f8 = c.fmt == FM_FMT_FP8;
  int64_t keys = std::max(1, b.max_len);
  if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + b.max_tokens);
  if (rows <= kDecodeRows) {
    // As many CTAs as are resident at once: a second wave costs more than longer splits (64 units of 4096 keys: 25 us
    // in 256 CTAs, 31 us in 384). Splits of at least two tiles up to 8, which join in their cluster; beyond, where a
    // second kernel joins them, of at least four (32768 keys of one unit: 11.6 us in 64 splits, 20.7 us in 256), and
    // only where 8 would be long (4096 keys of one unit: 8.3 us in 8, 7.7 us in 24; 2000: 7.4 us in 8, 7.5 us in 16).
    const int64_t units = static_cast<int64_t>(c.Hkv) * std::max(1, b.n);
    const int64_t tiles = (keys + kDecodeKeys - 1) / kDecodeKeys + (window > 0);
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
  const int64_t tiles = (keys + kTileRows - 1) / kTileRows + (window > 0);
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
Plan plan_of(const fm_kv_cache& c, const fm_kv_batch& b, int H, int window) {
  Plan pl = {};
  const int64_t rows = static_cast<int64_t>(b.max_tokens) * (H / c.Hkv);
  pl.splits = splits_of(c, b, H, 0);
  int64_t keys = std::max(1, b.max_len);
  if (window > 0) {
    pl.splits = std::min(pl.splits, splits_of(c, b, H, window));
    keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + b.max_tokens);
  }
  pl.decode = rows <= kDecodeRows;
  if (!pl.decode) {
    pl.alt = rows <= kTileRows;
    const int64_t tiles = (keys + kTileRows - 1) / kTileRows + (window > 0);
    pl.split_tiles = static_cast<int>((tiles + pl.splits - 1) / pl.splits);
    const int64_t block_rows = pl.alt ? kTileRows : 2 * kTileRows;
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

template <int DH, bool F8>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(paged_attn_kernel<DH, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSmemLimit + 1024);
}

// The kernels' shared-memory limits, once a device.
cudaError_t configure() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = configure_one<64, false>();
  if (e == cudaSuccess) e = configure_one<128, false>();
  if (e == cudaSuccess) e = configure_one<64, true>();
  if (e == cudaSuccess) e = configure_one<128, true>();
  if (e == cudaSuccess) e = decode_configure();
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

}  // namespace

}  // namespace fm

extern "C" int fm_paged_attention_workspace_size(const fm_kv_cache* c, const fm_kv_batch* b, int H, size_t* bytes) {
  if (!bytes) return fm::record_error(FM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = fm::check(c, b, H);
  if (st != FM_OK) return st;
  *bytes = b->n && b->tokens ? fm::plan_of(*c, fm::bounded_batch(*b), H, 0).workspace : 0;
  return FM_OK;
}

extern "C" int fm_paged_attention(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const uint16_t* q,
                                  int64_t q_stride, int H, float scale, int causal, int window, uint16_t* out,
                                  int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace fm;
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
  const Plan pl = plan_of(*c, *b, H, window);
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
  cudaError_t e = configure();
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
    e = decode_launch(p, c->Dh, f8, tk, tv, o);
  } else {
    auto kernel = c->Dh == 128 ? (f8 ? paged_attn_kernel<128, true> : paged_attn_kernel<128, false>)
                               : (f8 ? paged_attn_kernel<64, true> : paged_attn_kernel<64, false>);
    const unsigned blocks = static_cast<unsigned>(pl.row_blocks), entries = static_cast<unsigned>(b->n * pl.splits);
    const dim3 grid = pl.rows_first ? dim3(c->Hkv, entries, blocks) : dim3(blocks, c->Hkv, entries);
    e = launch(kernel, grid, dim3(threads_of(f8)), pl.smem, o, p, tk, tv);
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
