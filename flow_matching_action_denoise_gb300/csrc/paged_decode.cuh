// Attention over a paged cache for up to 16 stacked rows (tokens x query heads of a KV head): single tokens.
//
// Bound by reading the cache: 64 sequences of 8192 keys on 2 KV heads, Dh 128, take 46 us with an E4M3 cache (5.8 TB/s,
// 86 % of a plain copy's rate) and 80 us with bf16 (6.7 TB/s); 789 keys on one KV head take 4.9 us: three dependent loads
// and the first bytes 2.0, the keys 1.0, the joins of warps and cluster 1.2. A CTA takes one entry, KV head and split of its
// keys: a warp moves tiles of 64 keys by TMA into a three-stage ring, four warps take 16 keys each of every tile. Keys and head dims are the M = 16 of
// m16n8k16 tensor core instructions and the stacked rows their N, eight or sixteen: S^T = K Q^T, O^T = V^T P^T. So keys
// and values pass from shared memory straight into the fragments of one warp, and eight rows cost no padding (rows as
// M = 16 took twice the instructions and registers for eight). The big tensor cores would fill a sixteenth of their
// 128 rows and need E4M3 codes expanded in shared memory first: 32 KB of codes became 192 KB of traffic there, 1.2 us a
// 128-key tile and SM against 0.7 us at which HBM delivers them. Here codes are expanded in registers (exact, to f16).
// Every warp keeps its own running maximum, sum and O; the four are joined in shared memory, the splits of a key axis by
// their cluster (up to 8 splits: no workspace, no second kernel), whose CTAs send each other their shares by stores that the
// receiver's barrier counts; more splits meet in the workspace.
//
// E4M3 fragments. A 16-byte row piece holds 16 codes. Keys (M) x head dims (K): a lane's word is four consecutive dims
// of one key, taken as k pairs (2t, 2t + 1) and (2t + 8, 2t + 9); the query's fragments use the same order of dims, so
// the products meet. Values: the transposed load gives a lane [key, key + 1] x [dim, dim + 1], a byte permutation makes
// the pairs of keys of an even and of an odd dim: rows g and g + 8 of a 16-dim piece are its dims 2g and 2g + 1.

#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kv.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace fm {

namespace {

constexpr int kWarps = 4;
// CTAs an SM of a variant, by shared memory (16-bit tiles of 128 dims are 32 KB; two stages and three CTAs were slower:
// 28 us against 25 us for 32 sequences of 4096 keys) and registers.
template <int DH, bool F8, int NT>
constexpr int kResident = NT == 1 ? (F8 || DH == 64 ? 4 : 2) : (F8 || DH == 64 ? 3 : 2);
// Keys::kOwn, 16-bit rows of 128 dims: that more CTAs find room beside the prefix's counts for more than each one's speed
// (128 forks behind 8192 keys, 133 to 400 of their own: 29.1 -> 25.8 us).
template <int DH, bool F8, int NT, Keys K>
constexpr bool kMore = K == Keys::kOwn && NT == 1 && !F8 && DH == 128;
template <int DH, bool F8, int NT, Keys K>
constexpr int kStages = kMore<DH, F8, NT, K> ? 2 : 3;   // of the ring
constexpr int kThreads = (kWarps + 1) * 32;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The 8 x 8 matrix of 16-bit elements that the warp holds, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Byte offset of 16-byte piece c of row r in a tile of `row_bytes` rows (64: 64-byte swizzle, 128: 128-byte).
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  if constexpr (kRowBytes == 128)
    return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  else
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Shared memory: the ring, then the four warps' sums in its place; behind it, in a cluster, what a CTA receives.
constexpr int kPad = 8;   // floats between rows of sums
template <int DH, bool F8, int NT, Keys K>
constexpr size_t kWork = std::max<size_t>(static_cast<size_t>(kStages<DH, F8, NT, K>) * 2 * kDecodeKeys * DH * (F8 ? 1 : 2),
                                          static_cast<size_t>(8 * NT) * kWarps * (DH + kPad) * 4);
template <int DH, int NT>
constexpr size_t kReceived = (8 * NT * (DH / 4) + 8) * sizeof(float4) + 8 * 8 * NT * sizeof(float2);
template <int DH, bool F8, int NT, Keys K>
constexpr size_t smem_bytes(bool cluster) {
  return 1024 + kWork<DH, F8, NT, K> + (cluster ? kReceived<DH, NT> : 0);
}

// NT: row tiles of eight.
template <int DH, bool F8, int NT, Keys K>
__global__ void __launch_bounds__(kThreads, kResident<DH, F8, NT> + kMore<DH, F8, NT, K>)
    decode_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kDepth = kStages<DH, F8, NT, K>;
  constexpr int kRowBytes = F8 ? DH : 128;                 // bytes of a row in a block
  constexpr int kBlocks = F8 ? 1 : DH / 64;
  constexpr uint32_t kBlock = kDecodeKeys * kRowBytes;
  constexpr uint32_t kTile = kBlock * kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kDepth], empty[kDepth];
  __shared__ float2 s_ml[kWarps][8 * NT];                  // (log2 maximum, sum) of each warp
  // a cluster's splits: what every CTA has of this one's share of the rows' quads of sums, [split][share], and of the rows
  constexpr int kQuads = DH / 4;
  float4* got = reinterpret_cast<float4*>(smem + kWork<DH, F8, NT, K>);
  float2(*got_ml)[8 * NT] = reinterpret_cast<float2(*)[8 * NT]>(got + 8 * NT * kQuads + 8);
  __shared__ uint64_t landed;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, g = K == Keys::kOwn ? blockIdx.y % p.Hkv : blockIdx.y;
  if (tid == 0) {
    for (int i = 0; i < kDepth; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    mbar_init(&landed, 1);
    fence_mbar_init();
  }
  pdl_trigger();
  // Keys::kOwn starts when every CTA of the prefix's kernel has waited for what ran before it; it waits only for that kernel's
  // shares (and, rows or none, does not end before it)
  if constexpr (K == Keys::kOwn)
    see_inputs(p);
  else
    pdl_wait();
  [[maybe_unused]] auto prefix_done = [&] {
    pdl_wait();
    if (tid == 0 && first_cta()) take_word_back(p);
  };
  const Entry en = entry_of(p, blockIdx.z, tid == 0 && blockIdx.y == 0 && split == 0);
  // Keys::kOwn has any number of rows, a row block of 8 NT in each CTA
  const int row0 = K == Keys::kOwn ? blockIdx.y / p.Hkv * 8 * NT : 0;
  const int rows = min(max(min(en.nq, p.max_tokens) * p.G - row0, 0), 8 * NT);
  if (rows == 0) {   // the same in the whole cluster
    if constexpr (K == Keys::kOwn) prefix_done();
    return;
  }
  const int past = en.len - en.nq;
  int own = 0;   // Keys::kOwn: the first key
  if constexpr (K == Keys::kOwn) own = prefix_of(p, blockIdx.z, en);
  const int lo_all = K == Keys::kOwn ? own : first_key(p, past), hi_all = last_key(p, past + (row0 + rows - 1) / p.G, en.len);
  const int first = lo_all / kDecodeKeys;
  const Places<K> places(p, first, kDecodeKeys);
  const int begin = places.begin(first);   // t_lo: a place in the order of the key tiles
  const int all = max(0, places.place((hi_all + kDecodeKeys - 1) / kDecodeKeys) - begin);
  const int per = (all + p.splits - 1) / p.splits;
  const int t_lo = begin + split * per;
  const int nt = max(0, min(per, begin + all - t_lo));
  const bool clustered = p.splits > 1 && (K == Keys::kOwn || p.part_o == nullptr);
  const int total = rows * kQuads;   // quads of sums
  int share = total;                 // of a CTA of the cluster
  if (clustered) {
    share = (total + p.splits - 1) / p.splits;
    if (tid == 0) {
      const int x0 = min(total, split * share), x1 = min(total, x0 + share);
      const int touched = x1 > x0 ? (x1 - 1) / kQuads - x0 / kQuads + 1 : 0;   // rows
      mbar_arrive_expect_tx(&landed, p.splits * ((x1 - x0) * 16 + touched * 8));
    }
    __syncwarp();
    cluster_arrive_relaxed();   // paired with the wait before the first remote store
  }
  __syncthreads();

  // this lane's key (dim) g of eight, its quarter t of a row; its stacked rows are 8 x + 2 t and + 1
  const int q4 = lane & 3, g8 = lane >> 2;
  float o[NT][DH / 16][4];
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int i = 0; i < DH / 16; ++i) o[x][i][0] = o[x][i][1] = o[x][i][2] = o[x][i][3] = 0.f;
  float m[2 * NT], sum[2 * NT], c_row[2 * NT];
#pragma unroll
  for (int u = 0; u < 2 * NT; ++u) {
    m[u] = -INFINITY;
    sum[u] = 0.f;
    c_row[u] = p.scale_log2;
  }
  bool ok = true;
  if (warp == kWarps) {
    // ================================================= page table and TMA
    const int rows_box = min(p.page, kDecodeKeys), boxes = kDecodeKeys / rows_box;
    auto page_of = [&](int j) {
      const int key = places.tile(t_lo + j) * kDecodeKeys + lane * rows_box;
      if (lane >= boxes || key >= en.len || j >= nt) return p.pages;
      const int pg = p.table[static_cast<int64_t>(en.sid) * p.table_stride + (key >> p.page_shift)];
      if (pg < 0 || pg >= p.pages) {
        atomicOr(p.err, kErrBadBatch);
        return p.pages;
      }
      return pg;
    };
    int after = page_of(0);
    Ring at;
    int j = 0;
    for (; j < nt; ++j) {
      const int here = after;
      after = page_of(j + 1);
      if (j >= kDepth) ok = wait_for(&empty[at.b], at.phase ^ 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[at.b], 2 * kTile);
      __syncwarp();
      const uint32_t dst = smem_u32(smem) + at.b * 2 * kTile;
      for (int x = 0; x < boxes; ++x) {
        const int pg = __shfl_sync(0xffffffffu, here, x);
        const int row_in = (places.tile(t_lo + j) * kDecodeKeys + x * rows_box) & (p.page - 1);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < kBlocks; ++h) {
            tma_load_4d(dst + h * kBlock + x * rows_box * kRowBytes, &tm_k, &full[at.b], h * 64, row_in, g, pg);
            tma_load_4d(dst + kTile + h * kBlock + x * rows_box * kRowBytes, &tm_v, &full[at.b], h * 64, row_in, g, pg);
          }
        }
        __syncwarp();
      }
      at.next(kDepth);
    }
    if (!ok) {   // the copies in flight land before the CTA leaves
      if (lane == 0) atomicOr(p.err, kErrPipelineTimeout);
      for (int x = max(0, j - kDepth); x < j; ++x) wait_for(&full[x % kDepth], (x / kDepth) & 1);
    }
  } else {
    // ================================================= 16 keys of every tile
    uint32_t qf[NT][DH / 16][2];   // row 8 x + g
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int row = 8 * x + g8;
      const bool live = row < rows;
      const int tok = (row0 + row) / p.G, head = row0 + row - tok * p.G;
      const __nv_bfloat16* src = p.q + static_cast<int64_t>(en.begin + tok) * p.q_stride + (g * p.G + head) * DH;
#pragma unroll
      for (int c = 0; c < DH / 16; ++c) {
        if constexpr (F8) {   // dims 16 c + 4 t .. + 3
          const uint2 v = live ? *reinterpret_cast<const uint2*>(src + c * 16 + q4 * 4) : make_uint2(0, 0);
          qf[x][c][0] = v.x;
          qf[x][c][1] = v.y;
        } else {
          qf[x][c][0] = live ? *reinterpret_cast<const uint32_t*>(src + c * 16 + q4 * 2) : 0u;
          qf[x][c][1] = live ? *reinterpret_cast<const uint32_t*>(src + c * 16 + q4 * 2 + 8) : 0u;
        }
      }
      if constexpr (F8) {
        // rows into f16 by a power of two that puts the largest element in [2^14, 2^15); the inverse scales the scores
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < DH / 16; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) top = max(top, max(qf[x][c][y] & 0x7fffu, (qf[x][c][y] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = static_cast<int>(top >> 7);
        const int sh = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -100), 100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * *p.k_scale;
        // the scores' lanes own rows 2 t, 2 t + 1 of the eight
#pragma unroll
        for (int u = 0; u < 2; ++u) c_row[2 * x + u] *= __shfl_sync(0xffffffffu, down, (2 * q4 + u) * 4);
#pragma unroll
        for (int c = 0; c < DH / 16; ++c)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t w = qf[x][c][y];
            qf[x][c][y] = pack16<true>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
          }
      }
    }
    int my_lo[2 * NT], my_hi[2 * NT];
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u) {
      const int row = 8 * (u >> 1) + 2 * q4 + (u & 1), pos = past + (row0 + row) / p.G;
      my_lo[u] = K == Keys::kOwn ? own : row < rows ? first_key(p, pos) : 0;
      my_hi[u] = row < rows ? last_key(p, pos, en.len) : hi_all;
    }
    constexpr float kShift = F8 ? 6.0f : 0.0f;   // f16 probabilities are held 2^6 larger: subnormals begin lower
    float off[2 * NT], m_grow[2 * NT];
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u) {
      off[u] = kShift;
      m_grow[u] = -INFINITY;
    }
    // this lane's row of the matrices that ldmatrix moves: keys, and values transposed
    const int k_row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), k_sub = lane >> 4;
    const int v_row = warp * 16 + (lane >> 4) * 8 + (lane & 7), v_sub = (lane >> 3) & 1;
    const int f_row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), f_sub = lane >> 4;   // E4M3 values
    Ring at;
    for (int j = 0; j < nt; ++j) {
      ok = wait_for(&full[at.b], at.phase);
      if (!ok) break;
      const uint32_t kt = smem_u32(smem) + at.b * 2 * kTile, vt = kt + kTile;
      const int k0 = places.tile(t_lo + j) * kDecodeKeys + warp * 16;
      if (k0 < hi_all && (k0 + 16 > lo_all || (K == Keys::kSinks && k0 < p.sinks))) {
        // E4M3: two chains of dependent products (16.6 -> 15.9 us for 32 sequences of 4096 keys; no gain for bf16, which
        // waits for its bytes, nor with two row tiles, which have no registers left)
        constexpr bool kChains = F8 && NT == 1;
        float s[NT][4] = {}, s1[NT][4] = {};
        if constexpr (F8) {
#pragma unroll
          for (int c = 0; c < DH / 32; ++c) {
            uint32_t r[4];   // keys 0-7 and 8-15 of piece 2c, the same of piece 2c + 1
            ldsm4(r, kt + piece<kRowBytes>(k_row, 2 * c + k_sub));
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint32_t a[4];
              expand4(r[2 * y], a[0], a[2]);
              expand4(r[2 * y + 1], a[1], a[3]);
#pragma unroll
              for (int x = 0; x < NT; ++x) mma16816<true>(kChains && y ? s1[x] : s[x], a, qf[x][2 * c + y][0], qf[x][2 * c + y][1]);
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
            uint32_t a[4];
            ldsm4(a, kt + (c >> 2) * kBlock + piece<128>(k_row, 2 * (c & 3) + k_sub));
#pragma unroll
            for (int x = 0; x < NT; ++x) mma16816<false>(s[x], a, qf[x][c][0], qf[x][c][1]);
          }
        }
        if constexpr (kChains) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][e] += s1[0][e];
        }
        // s[x][0..1]: key g, rows 2 t, 2 t + 1 of tile x; s[x][2..3]: key g + 8
        bool edge = false, grow = false;
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) edge |= k0 + 16 > my_hi[u] || k0 < my_lo[u];
        if (__any_sync(0xffffffffu, edge)) {
#pragma unroll
          for (int u = 0; u < 2 * NT; ++u)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int key = k0 + 8 * y + g8;
              float& v = s[u >> 1][2 * y + (u & 1)];
              v = (key >= my_lo[u] || (K == Keys::kSinks && key < p.sinks)) && key < my_hi[u] ? v : -INFINITY;
            }
        }
        float top[2 * NT];
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u) {
          top[u] = fmaxf(s[u >> 1][u & 1], s[u >> 1][2 + (u & 1)]);
          grow |= top[u] > m_grow[u];
        }
        // the maximum over the keys is needed only where one of them moves it
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int u = 0; u < 2 * NT; ++u) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], d));
            if (!(top[u] > m_grow[u])) continue;
            const float f = ex2_approx((m[u] - top[u]) * c_row[u]);   // 0 for a row's first keys
            m[u] = top[u];
            m_grow[u] = top[u] + kGrow / c_row[u];
            off[u] = kShift - m[u] * c_row[u];
            sum[u] *= f;
#pragma unroll
            for (int i = 0; i < DH / 16; ++i) {
              o[u >> 1][i][u & 1] *= f;
              o[u >> 1][i][2 + (u & 1)] *= f;
            }
          }
        }
        uint32_t pf[NT][2];   // keys 2 t, 2 t + 1 (and + 8) of row g
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int u = 2 * x + (e & 1);
            s[x][e] = ex2_approx(fmaf(s[x][e], c_row[u], off[u]));
            sum[u] += s[x][e];
          }
          pf[x][0] = transpose8x8(pack16<F8>(s[x][0], s[x][1]));
          pf[x][1] = transpose8x8(pack16<F8>(s[x][2], s[x][3]));
        }
        // values behind the length may be anything, and 0 * NaN is NaN: masks of the pairs of keys (2t, 2t + 1) and + 8
        auto products = [&](auto tail) {
          constexpr bool kTail = decltype(tail)::value;
          const int in = en.len - k0 - 2 * q4;   // keys of the length from this lane's first one on
          const uint32_t k0m = in >= 2 ? 0xffffffffu : in == 1 ? 0x0000ffffu : 0u;
          const uint32_t k8m = in >= 10 ? 0xffffffffu : in == 9 ? 0x0000ffffu : 0u;
          if constexpr (F8) {
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
              uint32_t r[4];   // keys 0-7, 8-15 of piece 2c, the same of piece 2c + 1
              ldsm4_t(r, vt + piece<kRowBytes>(f_row, 2 * c + f_sub));
              if constexpr (kTail) r[0] &= k0m, r[1] &= k8m, r[2] &= k0m, r[3] &= k8m;
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                uint32_t a[4];   // dims 2 g and 2 g + 1, keys (2t, 2t + 1) and + 8
                expand4(__byte_perm(r[2 * y], 0, 0x3120), a[0], a[1]);
                expand4(__byte_perm(r[2 * y + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                for (int x = 0; x < NT; ++x) mma16816<true>(o[x][2 * c + y], a, pf[x][0], pf[x][1]);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < DH / 16; ++c) {
              uint32_t a[4];   // keys 0-7 of pieces 2c, 2c + 1, keys 8-15 of them
              ldsm4_t(a, vt + (c >> 2) * kBlock + piece<128>(v_row, 2 * (c & 3) + v_sub));
              if constexpr (kTail) a[0] &= k0m, a[1] &= k0m, a[2] &= k8m, a[3] &= k8m;
#pragma unroll
              for (int x = 0; x < NT; ++x) mma16816<false>(o[x][c], a, pf[x][0], pf[x][1]);
            }
          }
        };
        if (k0 + 16 > en.len)
          products(std::true_type{});
        else
          products(std::false_type{});
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[at.b]);
      at.next(kDepth);
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrPipelineTimeout);
  }
  __syncthreads();   // every tile has been used: the ring holds the warps' sums now

  // ---- join the four warps: [warp][row] sums, then the CTA's [row][DH]. Rows lie 8 floats apart in the banks.
  constexpr int kPitch = DH + kPad;
  float* sums = reinterpret_cast<float*>(smem);
  if (warp < kWarps) {
#pragma unroll
    for (int u = 0; u < 2 * NT; ++u) {
      float l = sum[u];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      const int row = 8 * (u >> 1) + 2 * q4 + (u & 1);
      if (g8 == 0) s_ml[warp][row] = make_float2(m[u] > -INFINITY ? m[u] * c_row[u] : -INFINITY, l);
      float* dst = sums + (warp * 8 * NT + row) * kPitch;
#pragma unroll
      for (int c = 0; c < DH / 16; ++c) {
        if constexpr (F8) {
          *reinterpret_cast<float2*>(dst + c * 16 + 2 * g8) = make_float2(o[u >> 1][c][u & 1], o[u >> 1][c][2 + (u & 1)]);
        } else {
          dst[c * 16 + g8] = o[u >> 1][c][u & 1];
          dst[c * 16 + 8 + g8] = o[u >> 1][c][2 + (u & 1)];
        }
      }
    }
  }
  __syncthreads();
  if constexpr (K == Keys::kOwn) prefix_done();   // its shares are there
  const float vs = F8 ? *p.v_scale : 1.0f;
  // Keys::kOwn: every split's weight in a row's sum over the prefix, under the prefix's maximum; that maximum, the total
  __shared__ float s_w[K == Keys::kOwn ? 8 * NT : 1][kMostPrefixSplits];
  __shared__ float2 s_pre[K == Keys::kOwn ? 8 * NT : 1];
  if constexpr (K == Keys::kOwn) {
    if (own > 0) {
      constexpr int kEach = kMostPrefixSplits / 32;
      for (int row = warp; row < rows; row += kWarps + 1) {
        const int64_t at = static_cast<int64_t>(en.begin + (row0 + row) / p.G) * p.H + g * p.G + (row0 + row) % p.G;
        float2 ml[kEach];
        float top = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int s = lane + 32 * i;
          ml[i] = s < p.prefix_splits ? p.part_ml[s * static_cast<int64_t>(p.tokens) * p.H + at] : make_float2(-INFINITY, 0.f);
          top = fmaxf(top, ml[i].x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          // no keys: no share. A NaN in the query has no maximum either, but its sum is NaN
          const bool none = ml[i].x == -INFINITY && ml[i].y == 0.f;
          const float w = ex2_approx(ml[i].x - top);
          s_w[row][lane + 32 * i] = none ? -1.0f : w;   // behind the last one, too
          if (!none) l += ml[i].y * w;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
        if (lane == 0) s_pre[row] = make_float2(top, l);
      }
      __syncthreads();
    }
  }
  // a row's quad of sums, under the maximum `top` and with their total l, as output; with the prefix's shares where the group
  // has some
  auto finish = [&](int row, int d, float top, float l, float4 acc) {
    const int tok = en.begin + (row0 + row) / p.G, head = g * p.G + (row0 + row) % p.G;
    float inv = vs;
    if constexpr (K == Keys::kOwn) {
      if (own > 0) {
        const int64_t rows_of = static_cast<int64_t>(p.tokens) * p.H, at = static_cast<int64_t>(tok) * p.H + head;
        const float2 pre = s_pre[row];
        const float all = fmaxf(top, pre.x);
        const float f = top > -INFINITY ? ex2_approx(top - all) : 0.f, fv = f * vs;
        const float fp = pre.x > -INFINITY ? ex2_approx(pre.x - all) : 0.f;
        l = l * f + pre.y * fp;
        float4 sum4 = make_float4(0.f, 0.f, 0.f, 0.f);
        // eight loads are on their way at a time (with a weight and a load by turns the join of 13 took 3 us more)
        for (int s0 = 0; s0 < p.prefix_splits; s0 += 8) {
          float4 v[8];
          float w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            w[i] = s_w[row][s0 + i];
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!(w[i] < 0.f)) v[i] = *reinterpret_cast<const float4*>(p.part_o + ((s0 + i) * rows_of + at) * DH + d);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum4.x += v[i].x * w[i], sum4.y += v[i].y * w[i], sum4.z += v[i].z * w[i], sum4.w += v[i].w * w[i];
        }
        acc.x = acc.x * fv + sum4.x * fp, acc.y = acc.y * fv + sum4.y * fp;
        acc.z = acc.z * fv + sum4.z * fp, acc.w = acc.w * fv + sum4.w * fp;
        inv = 1.0f;
      }
    }
    inv = l == 0.f ? 0.f : inv / l;
    *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + head * DH + d) =
        make_uint2(pack16<false>(acc.x * inv, acc.y * inv), pack16<false>(acc.z * inv, acc.w * inv));
  };
  if (clustered) cluster_wait();
  for (int x = tid; x < total; x += kThreads) {
    const int row = x / kQuads, d = (x % kQuads) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = s_ml[w][row];
      const float f = ml.x > -INFINITY ? ex2_approx(ml.x - top) : 0.f;
      const float4 v = *reinterpret_cast<const float4*>(sums + (w * 8 * NT + row) * kPitch + d);
      l += ml.y * f;
      acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    if (clustered) {
      const int owner = x / share;
      st_async_v4(map_dsmem(smem_u32(&got[split * share + x - owner * share]), owner), acc.x, acc.y, acc.z, acc.w,
                  map_dsmem(smem_u32(&landed), owner));
      if (d == 0) {   // to every CTA that has quads of the row
        for (int q = owner; q <= (x + kQuads - 1) / share; ++q)
          st_async_v2(map_dsmem(smem_u32(&got_ml[split][row]), q), top, l, map_dsmem(smem_u32(&landed), q));
      }
    } else if (p.splits > 1) {
      const int tok = en.begin + (row0 + row) / p.G, head = g * p.G + (row0 + row) % p.G;
      const int64_t at = (static_cast<int64_t>(split) * p.tokens + tok) * p.H + head;
      if (nt > 0) *reinterpret_cast<float4*>(p.part_o + at * DH + d) = make_float4(acc.x * vs, acc.y * vs, acc.z * vs, acc.w * vs);
      if (d == 0) p.part_ml[at] = make_float2(top, l);
    } else {
      finish(row, d, top, l, acc);
    }
  }
  if (!clustered) return;
  // ---- join the cluster's splits in split order: every CTA finishes a share of the quads, sent to it by all as they were done
  // (with the cluster's barrier before and after and the others' shared memory read between them a single token took 1 us more)
  __syncwarp();
  cluster_arrive_relaxed();
  if (warp == 0 && !wait_for_cluster(&landed, 0) && lane == 0) atomicOr(p.err, kErrPipelineTimeout);
  __syncthreads();   // one warp polls: others on the SM may still compute
  const int x0 = split * share;
  for (int x = x0 + tid; x < min(total, x0 + share); x += kThreads) {
    const int row = x / kQuads, d = (x % kQuads) * 4;
    float2 ml[8];
    float top = -INFINITY;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      ml[s] = s < p.splits ? got_ml[s][row] : make_float2(-INFINITY, 0.f);
      top = fmaxf(top, ml[s].x);
    }
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s >= p.splits) continue;
      const float f = ml[s].x > -INFINITY ? ex2_approx(ml[s].x - top) : 0.f;
      const float4 v = got[s * share + x - x0];
      l += ml[s].y * f;
      acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    finish(row, d, top, l, acc);
  }
  __syncwarp();
  cluster_wait();   // no CTA leaves while another still sends to it
}

template <int DH, bool F8, int NT, Keys K>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(decode_kernel<DH, F8, NT, K>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_bytes<DH, F8, NT, K>(true)));
}

template <int DH, bool F8, int NT, Keys K>
cudaError_t run(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const LaunchOpts& o) {
  const int blocks = K == Keys::kOwn ? (p.max_tokens * p.G + 8 * NT - 1) / (8 * NT) : 1;
  return launch(decode_kernel<DH, F8, NT, K>, dim3(p.splits, p.Hkv * blocks, p.n), dim3(kThreads),
                smem_bytes<DH, F8, NT, K>(o.cluster.x > 1), o, p, tk, tv);
}

template <int DH, bool F8, Keys K>
cudaError_t run_rows(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const LaunchOpts& o) {
  return p.max_tokens * p.G <= 8 ? run<DH, F8, 1, K>(p, tk, tv, o) : run<DH, F8, 2, K>(p, tk, tv, o);
}

template <int DH, bool F8, Keys K>
cudaError_t configure_rows() {
  const cudaError_t e = configure_one<DH, F8, 1, K>();
  return e == cudaSuccess ? configure_one<DH, F8, 2, K>() : e;
}

}  // namespace

template <Keys K>
cudaError_t decode_configure() {
  cudaError_t e = configure_rows<64, false, K>();
  if (e == cudaSuccess) e = configure_rows<128, false, K>();
  if (e == cudaSuccess) e = configure_rows<64, true, K>();
  if (e == cudaSuccess) e = configure_rows<128, true, K>();
  return e;
}

template <Keys K>
cudaError_t decode_launch(const AttnParams& p, int Dh, bool f8, const CUtensorMap& tk, const CUtensorMap& tv,
                          const LaunchOpts& opts) {
  LaunchOpts o = opts;
  if (p.splits > 1 && (K == Keys::kOwn || !p.part_o)) o.cluster = dim3(p.splits, 1, 1);
  if (Dh == 128) return f8 ? run_rows<128, true, K>(p, tk, tv, o) : run_rows<128, false, K>(p, tk, tv, o);
  return f8 ? run_rows<64, true, K>(p, tk, tv, o) : run_rows<64, false, K>(p, tk, tv, o);
}

}  // namespace fm
