// Shared by the two attention kernels over a paged cache (paged_attn.cu: many rows, paged_decode.cu: up to 16).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv.h"
#include "ptx.cuh"

namespace fm {

constexpr float kGrow = 8.0f;   // the running maximum moves when it grows by more than this power of two

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
  float scale_log2;               // scale * log2(e)
  const float* k_scale;
  const float* v_scale;
  int alt, splits, split_tiles;
  int row_blocks, rows_first;     // of paged_attn.cu's grid
  int ring, raw_ring;
  float* part_o;                  // [splits][tokens * H][Dh]
  float2* part_ml;                // [splits][tokens * H] (log2 maximum, sum)
  int* err;
};

// The kernel for up to 16 stacked rows (max_tokens * G): p.splits CTAs an entry and KV head, joined inside a cluster
// where p.part_o is null, else through the workspace.
constexpr int kDecodeRows = 16;
constexpr int kDecodeKeys = 64;   // keys of a tile
cudaError_t decode_launch(const AttnParams& p, int Dh, bool f8, const CUtensorMap& tk, const CUtensorMap& tv,
                          const LaunchOpts& o);
cudaError_t decode_configure();
int decode_resident(int Dh, bool f8, int rows);   // CTAs of it on an SM at once

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

// The keys [first_key, last_key) of a token at position pos.
__device__ __forceinline__ int last_key(const AttnParams& p, int pos, int len) {
  return pos < 0 ? 0 : (p.causal ? min(pos + 1, len) : len);
}
__device__ __forceinline__ int first_key(const AttnParams& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// True once the phase with the given parity has completed; false after 2^22 polls (the hardware suspends the thread in
// each for a while): far beyond any legitimate wait. No clock is read between the polls, and no suspension time is
// asked for: with 20 us the E4M3 variant took 285 us instead of 270 for 4096 tokens over 12288 keys.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity) {
#pragma unroll 1
  for (int i = 0; i < (1 << 22); ++i)
    if (mbar_try_wait(bar, parity)) return true;
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
