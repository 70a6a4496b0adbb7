// Attention over a paged cache for up to 16 stacked rows (tokens x query heads of a KV head): single tokens.
//
// Bound by reading the cache. A CTA takes one entry, KV head and split of its keys: a warp moves tiles of 64 keys by
// TMA into a three-stage ring, four warps take 16 keys each of every tile. Rows are the M of m16n8k16 tensor core
// instructions, so that keys and values pass from shared memory straight into the fragments of one warp: the big
// tensor cores would fill an eighth of their 128 rows and need E4M3 codes expanded in shared memory first (32 KB of
// codes became 192 KB of traffic there: 1.5 us a 128-key tile and SM, against 0.7 us at which HBM delivers them).
// Here codes are expanded in registers (exact, to f16). Every warp keeps its own running maximum, sum and O; the four
// are joined in shared memory, the splits of a key axis by their cluster through distributed shared memory (up to 8
// splits: no workspace, no second kernel), more through the workspace.
//
// E4M3 fragments. A 16-byte row piece holds 16 codes. Keys (n) x head dims (k): a lane's word is four consecutive dims
// of one key, taken as k pairs (2t, 2t + 1) and (2t + 8, 2t + 9); the query's fragments use the same order of dims, so
// the products meet. Values: the transposed load gives a lane [key, key + 1] x [dim, dim + 1], two byte permutations
// make the pairs of keys of an even and of an odd dim: the two n tiles of a 16-dim piece are its even and its odd dims.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kv.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace fm {

namespace {

constexpr int kWarps = 4, kStages = 3;
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
// Two E4M3 codes (the low 16 bits) as f16 values.
__device__ __forceinline__ uint32_t expand2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

// Byte offset of 16-byte piece c of row r in a tile of `row_bytes` rows (64: 64-byte swizzle, 128: 128-byte).
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  if constexpr (kRowBytes == 128)
    return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  else
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

template <int DH, bool F8>
__global__ void __launch_bounds__(kThreads, 3)
    decode_kernel(const AttnParams p, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  constexpr int kRowBytes = F8 ? DH : 128;                 // bytes of a row in a block
  constexpr int kBlocks = F8 ? 1 : DH / 64;
  constexpr uint32_t kBlock = kDecodeKeys * kRowBytes;
  constexpr uint32_t kTile = kBlock * kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ float2 s_ml[kWarps + 1][kDecodeRows];         // (log2 maximum, sum) of each warp, and of the CTA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, g = blockIdx.y;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kWarps);
    }
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  const Entry en = entry_of(p, blockIdx.z, tid == 0 && g == 0 && split == 0);
  const int rows = min(min(en.nq, p.max_tokens) * p.G, kDecodeRows);
  if (rows == 0) return;   // the same in the whole cluster
  const int past = en.len - en.nq;
  const int lo_all = first_key(p, past), hi_all = last_key(p, past + (rows - 1) / p.G, en.len);
  const int first = lo_all / kDecodeKeys;
  const int all = max(0, (hi_all + kDecodeKeys - 1) / kDecodeKeys - first);
  const int per = (all + p.splits - 1) / p.splits;
  const int t_lo = first + split * per;
  const int nt = max(0, min(per, first + all - t_lo));
  __syncthreads();

  const int q4 = lane & 3, r0 = lane >> 2;   // this lane's rows r0 and r0 + 8, its quarter of a row
  float o[DH / 8][4];
#pragma unroll
  for (int i = 0; i < DH / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
  float c_row[2] = {p.scale_log2, p.scale_log2};
  bool ok = true;
  if (warp == kWarps) {
    // ================================================= page table and TMA
    const int rows_box = min(p.page, kDecodeKeys), boxes = kDecodeKeys / rows_box;
    auto page_of = [&](int j) {
      const int key = (t_lo + j) * kDecodeKeys + lane * rows_box;
      if (lane >= boxes || key >= en.len || j >= nt) return p.pages;
      const int pg = __ldg(p.table + static_cast<int64_t>(en.sid) * p.table_stride + (key >> p.page_shift));
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
      if (j >= kStages) ok = wait_for(&empty[at.b], at.phase ^ 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[at.b], 2 * kTile);
      __syncwarp();
      const uint32_t dst = smem_u32(smem) + at.b * 2 * kTile;
      for (int x = 0; x < boxes; ++x) {
        const int pg = __shfl_sync(0xffffffffu, here, x);
        const int row_in = ((t_lo + j) * kDecodeKeys + x * rows_box) & (p.page - 1);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < kBlocks; ++h) {
            tma_load_4d(dst + h * kBlock + x * rows_box * kRowBytes, &tm_k, &full[at.b], h * 64, row_in, g, pg);
            tma_load_4d(dst + kTile + h * kBlock + x * rows_box * kRowBytes, &tm_v, &full[at.b], h * 64, row_in, g, pg);
          }
        }
        __syncwarp();
      }
      at.next(kStages);
    }
    if (!ok) {   // the copies in flight land before the CTA leaves
      if (lane == 0) atomicOr(p.err, kErrPipelineTimeout);
      for (int x = max(0, j - kStages); x < j; ++x) wait_for(&full[x % kStages], (x / kStages) & 1);
    }
  } else {
    // ================================================= 16 keys of every tile
    uint32_t qf[DH / 16][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {   // rows r0, r0 + 8
      const int row = r0 + 8 * u;
      const bool live = row < rows;
      const int tok = row / p.G, head = row - tok * p.G;
      const __nv_bfloat16* src = p.q + static_cast<int64_t>(en.begin + tok) * p.q_stride + (g * p.G + head) * DH;
#pragma unroll
      for (int c = 0; c < DH / 16; ++c) {
        if constexpr (F8) {   // dims 16 c + 4 t .. + 3
          const uint2 v = live ? __ldg(reinterpret_cast<const uint2*>(src + c * 16 + q4 * 4)) : make_uint2(0, 0);
          qf[c][u] = v.x;
          qf[c][2 + u] = v.y;
        } else {
          qf[c][u] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + c * 16 + q4 * 2)) : 0u;
          qf[c][2 + u] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + c * 16 + q4 * 2 + 8)) : 0u;
        }
      }
      if constexpr (F8) {
        // rows into f16 by a power of two that puts the largest element in [2^14, 2^15); the inverse scales the scores
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < DH / 16; ++c)
#pragma unroll
          for (int x = 0; x < 2; ++x) top = max(top, max(qf[c][u + 2 * x] & 0x7fffu, (qf[c][u + 2 * x] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int ex = static_cast<int>(top >> 7);
        const int sh = ex == 0 || ex == 255 ? 0 : min(max(141 - ex, -100), 100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        c_row[u] *= __uint_as_float(static_cast<uint32_t>(127 - sh) << 23) * __ldg(p.k_scale);
#pragma unroll
        for (int c = 0; c < DH / 16; ++c)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t w = qf[c][u + 2 * x];
            qf[c][u + 2 * x] = pack16<true>(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
          }
      }
    }
    int my_lo[2], my_hi[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = r0 + 8 * u, pos = past + row / p.G;
      my_lo[u] = row < rows ? first_key(p, pos) : 0;
      my_hi[u] = row < rows ? last_key(p, pos, en.len) : hi_all;
    }
    constexpr float kShift = F8 ? 6.0f : 0.0f;   // f16 probabilities are held 2^6 larger: subnormals begin lower
    float off[2] = {kShift, kShift}, m_grow[2] = {-INFINITY, -INFINITY};
    const float grow_by[2] = {kGrow / c_row[0], kGrow / c_row[1]};
    // this lane's row of the matrices that ldmatrix moves: keys, and values transposed
    const int k_row = warp * 16 + (lane >> 4) * 8 + (lane & 7), k_sub = (lane >> 3) & 1;
    const int v_row = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), v_sub = lane >> 4;
    Ring at;
    for (int j = 0; j < nt; ++j) {
      ok = wait_for(&full[at.b], at.phase);
      if (!ok) break;
      const uint32_t kt = smem_u32(smem) + at.b * 2 * kTile, vt = kt + kTile;
      const int k0 = (t_lo + j) * kDecodeKeys + warp * 16;
      if (k0 < hi_all && k0 + 16 > lo_all) {
        float s[2][4] = {};
        if constexpr (F8) {
#pragma unroll
          for (int c = 0; c < DH / 32; ++c) {
            uint32_t r[4];   // keys 0-7 and 8-15 (r[0..1], r[2..3]) of two 16-dim pieces
            ldsm4(r, kt + piece<kRowBytes>(k_row, 2 * c + k_sub));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              mma16816<true>(s[0], qf[2 * c + x], expand2(r[x]), expand2(r[x] >> 16));
              mma16816<true>(s[1], qf[2 * c + x], expand2(r[2 + x]), expand2(r[2 + x] >> 16));
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
            uint32_t r[4];
            ldsm4(r, kt + (c >> 2) * kBlock + piece<128>(k_row, 2 * (c & 3) + k_sub));
            mma16816<false>(s[0], qf[c], r[0], r[1]);
            mma16816<false>(s[1], qf[c], r[2], r[3]);
          }
        }
        // s[x][0..1]: row r0, keys 8 x + 2 t, + 1; s[x][2..3]: row r0 + 8
        const bool edge = k0 + 16 > my_hi[0] || k0 + 16 > my_hi[1] || k0 < my_lo[0] || k0 < my_lo[1];
        if (__any_sync(0xffffffffu, edge)) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = k0 + 8 * x + 2 * q4 + (e & 1);
              s[x][e] = key >= my_lo[e >> 1] && key < my_hi[e >> 1] ? s[x][e] : -INFINITY;
            }
        }
        float top[2];
        bool grow = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          top[u] = fmaxf(fmaxf(s[0][2 * u], s[0][2 * u + 1]), fmaxf(s[1][2 * u], s[1][2 * u + 1]));
          top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 1));
          top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], 2));
          grow |= top[u] > m_grow[u];
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (!(top[u] > m_grow[u])) continue;
            const float f = ex2_approx((m[u] - top[u]) * c_row[u]);   // 0 for a row's first keys
            m[u] = top[u];
            m_grow[u] = top[u] + grow_by[u];
            off[u] = kShift - m[u] * c_row[u];
            sum[u] *= f;
#pragma unroll
            for (int i = 0; i < DH / 8; ++i) {
              o[i][2 * u] *= f;
              o[i][2 * u + 1] *= f;
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[x][e] = ex2_approx(fmaf(s[x][e], c_row[e >> 1], off[e >> 1]));
            sum[e >> 1] += s[x][e];
          }
        const uint32_t pf[4] = {pack16<F8>(s[0][0], s[0][1]), pack16<F8>(s[0][2], s[0][3]), pack16<F8>(s[1][0], s[1][1]),
                                pack16<F8>(s[1][2], s[1][3])};
        // values behind the length may be anything, and 0 * NaN is NaN: masks of the pairs of keys (2t, 2t + 1) and + 8
        const int in = en.len - k0 - 2 * q4;   // keys of the length from this lane's first one on
        if constexpr (F8) {
          const uint32_t k0m = in >= 2 ? 0xffffffffu : in == 1 ? 0x0000ffffu : 0u;
          const uint32_t k8m = in >= 10 ? 0xffffffffu : in == 9 ? 0x0000ffffu : 0u;
#pragma unroll
          for (int c = 0; c < DH / 32; ++c) {
            uint32_t r[4];   // keys 0-7, 8-15 of piece 2c, the same of piece 2c + 1
            ldsm4_t(r, vt + piece<kRowBytes>(v_row, 2 * c + v_sub));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t a = r[2 * x] & k0m, b = r[2 * x + 1] & k8m;
              const int i = (2 * c + x) * 2;
              mma16816<true>(o[i], pf, expand2(__byte_perm(a, 0, 0x4420)), expand2(__byte_perm(b, 0, 0x4420)));
              mma16816<true>(o[i + 1], pf, expand2(__byte_perm(a, 0, 0x4431)), expand2(__byte_perm(b, 0, 0x4431)));
            }
          }
        } else {
          const uint32_t k0m = in >= 2 ? 0xffffffffu : in == 1 ? 0x0000ffffu : 0u;
          const uint32_t k8m = in >= 10 ? 0xffffffffu : in == 9 ? 0x0000ffffu : 0u;
#pragma unroll
          for (int c = 0; c < DH / 16; ++c) {
            uint32_t r[4];
            ldsm4_t(r, vt + (c >> 2) * kBlock + piece<128>(v_row, 2 * (c & 3) + v_sub));
            mma16816<false>(o[2 * c], pf, r[0] & k0m, r[1] & k8m);
            mma16816<false>(o[2 * c + 1], pf, r[2] & k0m, r[3] & k8m);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[at.b]);
      at.next(kStages);
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrPipelineTimeout);
  }
  __syncthreads();   // every tile has been used: the ring holds the warps' sums now

  // ---- join the four warps: [warp][row][DH] sums, then the CTA's [row][DH]
  float* sums = reinterpret_cast<float*>(smem);
  float* cta = sums + kWarps * kDecodeRows * DH;
  if (warp < kWarps) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = sum[u];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int row = r0 + 8 * u;
      if (q4 == 0) s_ml[warp][row] = make_float2(m[u] > -INFINITY ? m[u] * c_row[u] : -INFINITY, l);
      float* dst = sums + (warp * kDecodeRows + row) * DH;
#pragma unroll
      for (int c = 0; c < DH / 16; ++c) {
        // E4M3: tiles 2c, 2c + 1 are the even and odd dims of a piece: a lane's four are consecutive
        if constexpr (F8) {
          *reinterpret_cast<float4*>(dst + c * 16 + q4 * 4) =
              make_float4(o[2 * c][2 * u], o[2 * c + 1][2 * u], o[2 * c][2 * u + 1], o[2 * c + 1][2 * u + 1]);
        } else {
          *reinterpret_cast<float2*>(dst + c * 16 + q4 * 2) = make_float2(o[2 * c][2 * u], o[2 * c][2 * u + 1]);
          *reinterpret_cast<float2*>(dst + c * 16 + 8 + q4 * 2) = make_float2(o[2 * c + 1][2 * u], o[2 * c + 1][2 * u + 1]);
        }
      }
    }
  }
  __syncthreads();
  const float vs = F8 ? __ldg(p.v_scale) : 1.0f;
  const bool clustered = p.splits > 1 && p.part_o == nullptr;
  constexpr int kQuads = DH / 4;
  for (int x = tid; x < rows * kQuads; x += kThreads) {
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
      const float4 v = *reinterpret_cast<const float4*>(sums + (w * kDecodeRows + row) * DH + d);
      l += ml.y * f;
      acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    const int tok = en.begin + row / p.G, head = g * p.G + row % p.G;
    if (clustered) {
      *reinterpret_cast<float4*>(cta + row * DH + d) = acc;
      if (d == 0) s_ml[kWarps][row] = make_float2(top, l);
    } else if (p.splits > 1) {
      const int64_t at = (static_cast<int64_t>(split) * p.tokens + tok) * p.H + head;
      if (nt > 0) *reinterpret_cast<float4*>(p.part_o + at * DH + d) = make_float4(acc.x * vs, acc.y * vs, acc.z * vs, acc.w * vs);
      if (d == 0) p.part_ml[at] = make_float2(top, l);
    } else {
      const float inv = l == 0.f ? 0.f : vs / l;
      *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + head * DH + d) =
          make_uint2(pack16<false>(acc.x * inv, acc.y * inv), pack16<false>(acc.z * inv, acc.w * inv));
    }
  }
  if (!clustered) return;
  // ---- join the cluster's splits in split order: every CTA finishes a share of the elements
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t rank = cluster_rank();
  const int total = rows * kQuads, share = (total + p.splits - 1) / p.splits;
  for (int x = rank * share + tid; x < min(total, static_cast<int>(rank + 1) * share); x += kThreads) {
    const int row = x / kQuads, d = (x % kQuads) * 4;
    float2 ml[8];
    float top = -INFINITY;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      ml[s] = make_float2(-INFINITY, 0.f);
      if (s < p.splits)
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(ml[s].x), "=f"(ml[s].y)
                     : "r"(map_dsmem(smem_u32(&s_ml[kWarps][row]), s)));
      top = fmaxf(top, ml[s].x);
    }
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      if (s >= p.splits) continue;
      const float f = ml[s].x > -INFINITY ? ex2_approx(ml[s].x - top) : 0.f;
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(map_dsmem(smem_u32(cta + row * DH + d), s)));
      l += ml[s].y * f;
      acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    const float inv = l == 0.f ? 0.f : vs / l;
    const int tok = en.begin + row / p.G, head = g * p.G + row % p.G;
    *reinterpret_cast<uint2*>(p.out + tok * p.out_stride + head * DH + d) =
        make_uint2(pack16<false>(acc.x * inv, acc.y * inv), pack16<false>(acc.z * inv, acc.w * inv));
  }
  // no CTA leaves while another still reads its share
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int DH, bool F8>
constexpr size_t smem_bytes() {
  const size_t ring = static_cast<size_t>(kStages) * 2 * kDecodeKeys * DH * (F8 ? 1 : 2);
  const size_t join = static_cast<size_t>(kWarps + 1) * kDecodeRows * DH * 4;
  return 1024 + (ring > join ? ring : join);
}

template <int DH, bool F8>
cudaError_t configure_one() {
  return cudaFuncSetAttribute(decode_kernel<DH, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem_bytes<DH, F8>()));
}

template <int DH, bool F8>
cudaError_t run(const AttnParams& p, const CUtensorMap& tk, const CUtensorMap& tv, const LaunchOpts& o) {
  return launch(decode_kernel<DH, F8>, dim3(p.splits, p.Hkv, p.n), dim3(kThreads), smem_bytes<DH, F8>(), o, p, tk, tv);
}

}  // namespace

cudaError_t decode_configure() {
  cudaError_t e = configure_one<64, false>();
  if (e == cudaSuccess) e = configure_one<128, false>();
  if (e == cudaSuccess) e = configure_one<64, true>();
  if (e == cudaSuccess) e = configure_one<128, true>();
  return e;
}

cudaError_t decode_launch(const AttnParams& p, int Dh, bool f8, const CUtensorMap& tk, const CUtensorMap& tv,
                          const LaunchOpts& opts) {
  LaunchOpts o = opts;
  if (p.splits > 1 && !p.part_o) o.cluster = dim3(p.splits, 1, 1);
  if (Dh == 128) return f8 ? run<128, true>(p, tk, tv, o) : run<128, false>(p, tk, tv, o);
  return f8 ? run<64, true>(p, tk, tv, o) : run<64, false>(p, tk, tv, o);
}

}  // namespace fm
