// Shared by the two attention kernels over a paged cache (paged_tile.cuh: many rows, paged_decode.cuh: up to 16).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.h"
#include "ptx.cuh"

namespace fm {

constexpr float kGrow = 8.0f;   // the running maximum moves when it grows by more than this power of two

// What a kernel's keys are: all that the mask leaves (one stretch of the axis), a window and the first tokens, or of a batch
// in groups the prefix that a group's entries share, for all its tokens at once, and what an entry has behind it.
enum class Keys { kAll, kSinks, kPrefix, kOwn };

struct AttnParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  int64_t q_stride, out_stride;   // elements between tokens
  const int32_t* start;
  const int32_t* seq;
  const int32_t* lens;
  const int32_t* table;
  int n, tokens, max_tokens, seqs, table_stride, pages, page, page_shift;
  int H, Hkv, G;
  int causal, window;
  int sinks;                      // first tokens that a window does not hide (Keys::kSinks)
  float scale_log2;               // scale * log2(e)
  const float* k_scale;
  const float* v_scale;
  int alt, splits, split_tiles;
  int row_blocks, rows_first;     // of paged_attn.cu's grid
  int ring, raw_ring;
  int cluster;                    // CTAs whose splits meet in their cluster (the tile kernel)
  const int32_t* g_first;         // groups: [g_n + 1] first entries
  const int32_t* g_shared;        // [g_n] tokens that a group's entries share
  int g_n, g_tokens;              // g_tokens: packed rows of a group that Keys::kPrefix takes
  int prefix_splits;              // shares of the prefix that Keys::kOwn joins
  uint64_t* seen;                 // the word between Keys::kPrefix and Keys::kOwn
  float* part_o;                  // [splits][tokens * H][Dh]
  float2* part_ml;                // [splits][tokens * H] (log2 maximum, sum)
  int* err;
};

// Both kernels are instantiated once for each Keys, in a source of their own; configure sets their shared-memory limits on
// the current device.
template <Keys K>
cudaError_t tile_launch(const AttnParams& p, int Dh, bool f8, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                        size_t smem, const LaunchOpts& o);
template <Keys K>
cudaError_t tile_configure();
int tile_clusters(int size);   // clusters of so many CTAs (of any variant: one is on an SM) at once

// The kernel for up to 16 stacked rows (max_tokens * G): p.splits CTAs an entry and KV head, joined inside a cluster
// where p.part_o is null, else through the workspace.
constexpr int kDecodeRows = 16;
constexpr int kDecodeKeys = 64;   // keys of a tile
constexpr int kMostPrefixSplits = 64;
template <Keys K>
cudaError_t decode_launch(const AttnParams& p, int Dh, bool f8, const CUtensorMap& tk, const CUtensorMap& tv,
                          const LaunchOpts& o);
template <Keys K>
cudaError_t decode_configure();
int decode_resident(int Dh, bool f8, int rows);   // CTAs of it on an SM at once
int own_resident(int Dh, bool f8, int rows);      // the same of Keys::kOwn
int decode_clusters(int Dh, bool f8, int rows, int size);   // clusters of so many of its CTAs at once

// An entry of the batch; one that is out of range has no tokens and no keys.
struct Entry {
  int begin, nq, sid, len;
};

__device__ __forceinline__ Entry entry_of(const AttnParams& p, int entry, bool report) {
  Entry e;
  e.begin = p.start[entry];
  e.nq = p.start[entry + 1] - e.begin;
  e.sid = p.seq ? p.seq[entry] : entry;
  e.len = 0;
  bool bad = e.begin < 0 || e.nq < 0 || e.begin > p.tokens || e.nq > p.tokens - e.begin || e.sid < 0 || e.sid >= p.seqs;
  if (bad) {
    e.nq = 0;
  } else {
    e.len = p.lens[e.sid];
    bad = e.len < 0 || e.len > p.table_stride * static_cast<int64_t>(p.page);
    if (bad) e.len = 0;
  }
  if (report && (bad || e.nq > p.max_tokens)) atomicOr(p.err, kErrBadBatch);
  return e;
}

// Group g as an entry: its packed rows from the first on, the pages of its first entry, the shared tokens as its length. One
// whose shared tokens are not all there has no keys.
__device__ __forceinline__ Entry group_of(const AttnParams& p, int g, bool report) {
  Entry e = {0, 0, 0, 0};
  const int f0 = p.g_first[g], f1 = p.g_first[g + 1], shared = p.g_shared[g];
  bool bad = f0 < 0 || f1 < f0 || f1 > p.n || shared < 0;
  if (!bad && f1 > f0) {
    e.begin = max(p.start[f0], 0);
    e.nq = min(max(min(p.start[f1], p.tokens), 0) - e.begin, p.g_tokens);
    e.sid = p.seq ? p.seq[f0] : f0;
    bad = e.sid < 0 || e.sid >= p.seqs || shared > p.lens[e.sid] || shared > p.table_stride * static_cast<int64_t>(p.page);
    if (!bad) e.len = shared;
    if (e.nq < 0) e.nq = 0;
  }
  if (report && bad) atomicOr(p.err, kErrBadBatch);
  return e;
}

// The tokens of an entry's prefix that its group's part covers, 0 where the entry has to see to all of its keys: without a
// (sound) group, with a token that does not see the whole prefix, or with rows behind those that the group's part takes.
// For whole warps.
__device__ __forceinline__ int prefix_of(const AttnParams& p, int entry, const Entry& e) {
  int lo = 0, hi = p.g_n;   // the last group that begins at or before the entry, 32 probes at a time
  for (int step = 32; step > 1;) {
    step = (hi - lo + 31) / 32;
    const int at = lo + static_cast<int>(threadIdx.x & 31) * step;
    const int before = __popc(__ballot_sync(0xffffffffu, at < hi && p.g_first[at] <= entry));
    if (before == 0) return 0;
    lo += (before - 1) * step;
    hi = min(hi, lo + step);
  }
  const int f0 = p.g_first[lo], f1 = p.g_first[lo + 1], shared = p.g_shared[lo];
  if (f0 < 0 || entry < f0 || entry >= f1 || f1 > p.n) return 0;
  const Entry group = group_of(p, lo, false);
  const int past = e.len - e.nq, end = e.begin + min(e.nq, p.max_tokens);
  const bool seen = past >= 0 && shared <= (p.causal ? past + 1 : e.len);
  return seen && group.len > 0 && e.begin >= group.begin && end <= group.begin + group.nq ? shared : 0;
}

// Keys::kOwn runs beside Keys::kPrefix and reads what kernels before both wrote (the batch, queries, keys, values). These
// writes are made visible to a grid that waits for the grids before it, as the prefix's does; for the other grid they are
// handed on by a word of the workspace. The prefix's first CTA stores kSeen (release) behind its wait and before it lets the
// other grid start; a thread there that finds kSeen (acquire) sees the inputs, and one that does not waits for the prefix to
// end, which is right as well, only later. Behind that wait Keys::kOwn's first CTA takes the word back, so that no call
// finds an earlier call's.
constexpr uint64_t kSeen = 0x5b1d93e6c7f0a42dull;
__device__ __forceinline__ bool first_cta() { return blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0; }
__device__ __forceinline__ void hand_inputs_on(const AttnParams& p) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p.seen), "l"(kSeen) : "memory");
}
__device__ __forceinline__ void see_inputs(const AttnParams& p) {
  uint64_t word;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(word) : "l"(p.seen) : "memory");
  if (word != kSeen) pdl_wait();
  asm volatile("fence.proxy.async.global;" ::: "memory");   // keys and values are read by TMA
}
__device__ __forceinline__ void take_word_back(const AttnParams& p) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p.seen), "l"(uint64_t(0)) : "memory");
}

// The keys [first_key, last_key) of a token at position pos.
__device__ __forceinline__ int last_key(const AttnParams& p, int pos, int len) {
  return pos < 0 ? 0 : (p.causal ? min(pos + 1, len) : len);
}
__device__ __forceinline__ int first_key(const AttnParams& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// The key tiles of a CTA in the order in which it takes them. With sinks these are the tiles of the first tokens up to the
// window's first tile, then the window's: place x of that order is tile x, or x + gap behind the first ones.
template <Keys K>
struct Places {
  int lead = 0, gap = 0;   // tiles of the first tokens alone, and those left out behind them
  // first: the window's first tile; keys: of a tile
  __device__ __forceinline__ Places(const AttnParams& p, int first, int keys) {
    if constexpr (K == Keys::kSinks) {
      lead = min((p.sinks - 1) / keys + 1, first);
      gap = first - lead;
    }
  }
  __device__ __forceinline__ int tile(int place) const {
    if constexpr (K == Keys::kSinks) return place < lead ? place : place + gap;
    return place;
  }
  // the place of a tile of the window (or of none: behind the last one)
  __device__ __forceinline__ int place(int tile) const {
    if constexpr (K == Keys::kSinks) return tile - gap;
    return tile;
  }
  __device__ __forceinline__ int begin(int first) const {
    if constexpr (K == Keys::kSinks) return 0;
    return first;
  }
};

// True once the phase with the given parity has completed; false after 2^22 polls (the hardware suspends the thread in
// each for a while): far beyond any legitimate wait. No clock is read between the polls, and no suspension time is
// asked for: with 20 us the E4M3 variant took 285 us instead of 270 for 4096 tokens over 12288 keys.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < (1 << 22); ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return false;
}

// The same for what other CTAs of the cluster have stored.
__device__ __forceinline__ bool wait_for_cluster(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < (1 << 22); ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.b32 %0, 1, 0, p;\n}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}

// One lane of a converged warp. Unlike a comparison with a lane number it tells the compiler that a single lane is
// active: tcgen05 instructions take their operands from the warp's uniform registers, and under a plain branch each
// MMA took about 100 cycles to issue (operands collected lane by lane), longer than it runs.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\t@p mov.s32 %0, 1;\n}" : "+r"(pred));
  return pred != 0;
}

// Position in a ring of buffers: the buffer and the parity of its barrier's phase.
struct Ring {
  int b = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++b == n) {
      b = 0;
      phase ^= 1;
    }
  }
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                            int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// The four E4M3 codes of a word as two pairs of f16 values (exact). The intrinsic takes and gives 16-bit halves, which
// costs three more instructions a pair.
__device__ __forceinline__ void expand4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

}  // namespace fm
