// The paged prefix cache: its bookkeeping on the device (fm_kv_reserve, fm_kv_fork, fm_kv_release, fm_kv_compact),
// the rotary positions fused with the store of new keys and values (fm_rope_append), and the way from a sequence's
// pages into a policy's persistent prefix (prefix_from_pages_launch).
//
// Bookkeeping. A sequence is a row of the page table and a length; `refs` counts the rows that name a page, 0 = free.
// All of it lives on the device, so a serving step (fork, reserve, append, attend, release) needs no host round trip
// and can be captured into a graph. Calls are all or nothing: every entry is validated before a row or a length is
// written, and the two status words say why a call did nothing. Free pages are taken lowest index first, so the result of a
// call depends on its arguments alone. No kernel here waits on another CTA except through a cluster barrier.

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "kv.h"
#include "ptx.cuh"

namespace fm {

namespace {

constexpr int kBookThreads = 1024;   // of a bookkeeping CTA; 256 where entries and pages are few: barriers are cheaper
constexpr int kSmallThreads = 256, kSmallPages = 1024;
constexpr int kMaxEntries = 1024;   // sequences of one bookkeeping call: one thread each
constexpr int kForkCluster = 8;

// Device view of the bookkeeping.
struct Book {
  int32_t *table, *lens, *refs;
  int seqs, table_stride, pages, page, shift;
};

// Device view of the pools, in 16-byte units. The rows (token, head) of a page are taken as runs that are contiguous in
// memory: one run of all rows where heads lie inside of tokens without gaps, a run of the tokens of each head where
// tokens lie inside of heads, else a run a row.
enum Runs { kRunAll, kRunHead, kRunRow };
struct Pool {
  uint4 *k, *v;
  int64_t layer, pg, tok, head;   // strides
  int layers, Hkv, chunks;        // chunks: 16-byte units of a row
  Runs runs;
};

template <typename T>
__host__ __device__ constexpr T up(T a, int b) {
  return (a + b - 1) / b;
}

// Exclusive sum over the CTA's THREADS threads; *total receives the sum. Every thread calls it.
template <int THREADS>
__device__ __forceinline__ int block_exclusive(int v, int* warp_sums, int* total) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // warp_sums may still be read from an earlier call
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int s = lane < kWarps ? warp_sums[lane] : 0;   // every warp scans the sums for itself
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, kWarps - 1);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp ? before : 0) + x - v;
}

// Calls f(page, inside, refs) in ascending order within a warp's contiguous share of [0, pages); 32 pages a step,
// coalesced. The first steps' counts are loaded once and kept: most pools need no second load in a second walk.
template <int THREADS>
struct PageWalk {
  static constexpr int kKeep = 4;
  int lo, hi, kept[kKeep];
  __device__ __forceinline__ explicit PageWalk(const Book& b) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int share = up(up(b.pages, 32), THREADS / 32) * 32;
    lo = min(b.pages, warp * share);
    hi = min(b.pages, lo + share);
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int pg = lo + u * 32 + lane;
      kept[u] = pg < hi ? b.refs[pg] : -1;
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(const Book& b, F f) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int u = 0; u < kKeep; ++u) {
      const int pg = lo + u * 32 + lane;
      if (lo + u * 32 < hi) f(pg, pg < hi, kept[u]);   // warp-uniform
    }
    constexpr int kAhead = 4;   // 16: slower, most warps have few steps
    for (int p0 = lo + kKeep * 32; p0 < hi; p0 += kAhead * 32) {
      int r[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int pg = p0 + u * 32 + lane;
        r[u] = pg < hi ? b.refs[pg] : -1;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int pg = p0 + u * 32 + lane;
        if (p0 + u * 32 < hi) f(pg, pg < hi, r[u]);
      }
    }
  }
};

struct Copy {
  int src, dst, rows;
};

// A set of numbers >= 0 in shared memory, open addressing, at most half full: what the entries of a call have in common is
// found in a few steps each (compared pair by pair 1024 forks took 70 us).
constexpr int kSlotsPer = 2;   // slots an entry
template <int SLOTS>
struct Set {
  int key[SLOTS];
  __device__ __forceinline__ static unsigned home(int k) {   // Fibonacci hashing
    return (static_cast<unsigned>(k) * 2654435769u) >> 16 & (SLOTS - 1);
  }
  __device__ __forceinline__ void clear(int tid, int threads) {
    for (int x = tid; x < SLOTS; x += threads) key[x] = -1;
  }
  // the slot of k, which is put there if it is new
  __device__ __forceinline__ int put(int k, bool* old) {
    unsigned at = home(k);
    for (int x = 0; x < SLOTS; ++x, at = (at + 1) & (SLOTS - 1)) {
      const int was = atomicCAS(&key[at], -1, k);
      if (was == -1 || was == k) {
        *old = was == k;
        return static_cast<int>(at);
      }
    }
    *old = true;   // not reached: there are more slots than entries
    return 0;
  }
  __device__ __forceinline__ bool has(int k) const {
    unsigned at = home(k);
    for (int x = 0; x < SLOTS; ++x, at = (at + 1) & (SLOTS - 1)) {
      if (key[at] == k) return true;
      if (key[at] == -1) return false;
    }
    return false;
  }
};

// fm_kv_reserve. One CTA: the whole decision needs the order of the entries, and its work is a few hundred bytes an
// entry plus two passes over refs; a second kernel copies the shared last pages on all SMs. Bound by latency (one token more
// of 64 sequences in a pool of 2200 pages: 4.7 us with the copies' kernel, of 1024 in 40000: 10.4 us; new pages are dealt
// out a thread each, which finds its entry by bisection).
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) reserve_kernel(Book b, const int32_t* seq, const int32_t* count, int n,
                                                               int32_t* status, Copy* copies, int32_t* fresh) {
  constexpr int kSlots = kSlotsPer * THREADS;
  __shared__ int s_seq[THREADS], s_have[THREADS], s_off[THREADS], s_sums[32], s_bad;
  __shared__ Set<kSlots> seqs, lasts;               // the sequences, and their begun last pages:
  __shared__ int s_users[kSlots], s_keeper[kSlots];   // entries that write to one, and the last of them
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) s_bad = 0;
  seqs.clear(tid, THREADS);
  lasts.clear(tid, THREADS);
  for (int x = tid; x < kSlots; x += THREADS) s_users[x] = 0, s_keeper[x] = -1;
  __syncthreads();
  pdl_wait();
  const PageWalk<THREADS> walk(b);   // its loads are on their way while the entries are looked up
  int s = -1 - tid, len = 0, add = 0, last = -1, last_refs = 0, bad = 0;
  if (tid < n) {
    s = seq[tid];
    add = count[tid];
    if (s < 0 || s >= b.seqs || add < 0) {
      bad = FM_KV_BAD_ENTRY;
    } else {
      len = b.lens[s];
      const int64_t room = static_cast<int64_t>(b.table_stride) * b.page;
      if (len < 0 || len > room) {
        bad = FM_KV_BAD_ENTRY;
      } else if (len + static_cast<int64_t>(add) > room) {
        bad = FM_KV_ROW_FULL;
      } else if (add > 0 && (len & (b.page - 1))) {
        last = b.table[static_cast<int64_t>(s) * b.table_stride + (len >> b.shift)];
        if (last < 0 || last >= b.pages || (last_refs = b.refs[last]) < 1) {
          bad = FM_KV_BAD_ENTRY;
          last = -1;
        }
      }
    }
    s_seq[tid] = s;
  }
  int slot = 0;
  bool again = false;
  if (tid < n && s >= 0 && s < b.seqs) {
    seqs.put(s, &again);
    if (again) bad |= FM_KV_BAD_ENTRY;
  }
  if (last >= 0) {
    slot = lasts.put(last, &again);
    atomicAdd(&s_users[slot], 1);
    atomicMax(&s_keeper[slot], tid);
  }
  __syncthreads();
  // a shared last page: every entry that writes to it gets a copy, but the last one where no other row names it
  bool copied = false;
  if (last >= 0) {
    const int users = s_users[slot];
    if (users > last_refs) bad |= FM_KV_BAD_ENTRY;   // more rows than the page's count knows of
    copied = users < last_refs || s_keeper[slot] != tid;
  }
  const int have = (len >> b.shift) + ((len & (b.page - 1)) != 0);
  const int end = len + add;
  const int want = (end >> b.shift) + ((end & (b.page - 1)) != 0);
  const int need = bad || tid >= n ? 0 : want - have + copied;
  if (bad) atomicOr(&s_bad, bad);
  int total = 0;
  const int off = block_exclusive<THREADS>(need, s_sums, &total);
  if (tid < n) {
    s_off[tid] = off;
    s_have[tid] = have << 1 | copied;
  }
  // free pages: every warp counts its share, then writes its ranks below `total`
  int mine = 0;
  walk.each(b, [&](int, bool in, int refs) { mine += __popc(__ballot_sync(0xffffffffu, in && refs == 0)); });
  int all_free = 0;
  int rank = block_exclusive<THREADS>(lane == 0 ? mine : 0, s_sums, &all_free);
  rank = __shfl_sync(0xffffffffu, rank, 0);
  const int why = s_bad;
  if (why || total > all_free) {   // the same in every thread
    if (tid < n) copies[tid].rows = 0;
    if (tid == 0) {
      status[0] = why ? why : FM_KV_NO_PAGES;
      status[1] = why ? 0 : total - all_free;
    }
    return;
  }
  if (rank < total)
    walk.each(b, [&](int pg, bool in, int refs) {
      const unsigned m = __ballot_sync(0xffffffffu, in && refs == 0);
      const int at = rank + __popc(m & ((1u << lane) - 1));
      if (in && refs == 0 && at < total) fresh[at] = pg;
      rank += __popc(m);
    });
  __syncthreads();
  // the entries' changes: a copied page first, then the pages of the new tokens in order
  if (tid < n) {
    copies[tid].rows = copied ? len & (b.page - 1) : 0;
    if (copied) {
      const int to = fresh[off];
      copies[tid].src = last;
      copies[tid].dst = to;
      b.table[static_cast<int64_t>(s) * b.table_stride + (len >> b.shift)] = to;
      b.refs[to] = 1;
      atomicSub(&b.refs[last], 1);
    }
    b.lens[s] = end;
  }
  for (int x = tid; x < total; x += THREADS) {
    int lo = 0, hi = n;   // the last entry whose pages begin at or before x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_off[mid] <= x)
        lo = mid;
      else
        hi = mid;
    }
    const int at = x - s_off[lo] - (s_have[lo] & 1);   // -1: the copied page
    if (at < 0) continue;
    const int pg = fresh[x];
    b.table[static_cast<int64_t>(s_seq[lo]) * b.table_stride + (s_have[lo] >> 1) + at] = pg;
    b.refs[pg] = 1;
  }
  if (tid == 0) {
    status[0] = 0;
    status[1] = total;
  }
}

// Copies `rows` tokens of page src to page dst of one layer, K and V, 16 bytes a thread, four loads in flight.
__device__ __forceinline__ void copy_rows(const Pool& p, int layer, int src, int dst, int rows) {
  const int64_t base = layer * p.layer;
  const uint4 *ks = p.k + base + src * p.pg, *vs = p.v + base + src * p.pg;
  uint4 *kd = p.k + base + dst * p.pg, *vd = p.v + base + dst * p.pg;
  const int len = p.runs == kRunAll ? rows * p.Hkv * p.chunks : p.runs == kRunHead ? rows * p.chunks : p.chunks;
  const int runs = p.runs == kRunAll ? 1 : p.runs == kRunHead ? p.Hkv : rows * p.Hkv;
  const int total = len * runs;
  for (int x0 = threadIdx.x; x0 < total; x0 += blockDim.x * 2) {
    uint4 a[2], d[2];
    int64_t at[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int x = x0 + u * blockDim.x;
      if (x >= total) continue;
      at[u] = x;
      if (runs > 1) {
        const int y = x / len, c = x - y * len;
        at[u] = p.runs == kRunHead ? y * p.head + c : (y / p.Hkv) * p.tok + (y % p.Hkv) * p.head + c;
      }
      a[u] = __ldcs(ks + at[u]);
      d[u] = __ldcs(vs + at[u]);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (x0 + u * blockDim.x >= total) continue;
      kd[at[u]] = a[u];
      vd[at[u]] = d[u];
    }
  }
}

// The shared last pages of a reserve call: one CTA per entry and layer. Bound by HBM (67 MB read and written: 20.6 us,
// 6.5 TB/s).
__global__ void __launch_bounds__(256) copy_shared_kernel(Pool p, const Copy* copies) {
  pdl_trigger();
  pdl_wait();
  const Copy c = copies[blockIdx.x];
  if (c.rows > 0) copy_rows(p, blockIdx.y, c.src, c.dst, c.rows);
}

constexpr int kNone = INT32_MIN;   // nothing to do at a place
__device__ __forceinline__ int places_of(int tokens, const Book& b) {
  return (tokens >> b.shift) + ((tokens & (b.page - 1)) != 0);
}

// fm_kv_fork (kFork) and fm_kv_release: one CTA or one cluster. Every CTA validates all entries; the CTAs then share the
// places of their rows. A fork looks up the counts of the pages that it names before it changes any. A release takes its
// own off at once, since only the sum shows a page that two entries name and one row counts. The cluster meets, and either
// all of it goes on to the table and the lengths, or a release gives the counts back. Bound by latency: dependent loads,
// barriers, the cluster's start and the code's own way into the caches (with eight places a thread a single row takes
// 6.4 us, with one 4.5). A fork and its release together: 8 rows of 50 pages 5.1 us, 64 of 30 7.0 us, 1024 of 35 20.2 us, 4 of
// 8192 11.2 us; looking at the counts is 0.4, 1.1 and 3 us a call of it for 8, 64 and 1024 rows.
// kTake: 32-place parts that a warp takes at once, their loads on the way together.
template <bool kFork, int kTake>
__global__ void __launch_bounds__(kBookThreads)
    share_kernel(Book b, const int32_t* seq, const int32_t* other, int n, int32_t* status) {
  __shared__ int s_seq[kMaxEntries], s_oth[kMaxEntries], s_len[kMaxEntries], s_wrong;
  __shared__ Set<kSlotsPer * kMaxEntries> named;   // fork: the targets; release: the sequences
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), warps = static_cast<int>(blockDim.x >> 5);
  if (tid == 0) s_wrong = 0;
  named.clear(tid, blockDim.x);
  // the others may write to s_wrong once this CTA has arrived, which every warp's wait below sees
  if (gridDim.x > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  int s = -1, o = 0, len = 0;
  bool bad = false, again = false;
  if (tid < n) {
    s = seq[tid];
    o = other ? other[tid] : 0;
    bad = s < 0 || s >= b.seqs || o < 0 || (kFork && o >= b.seqs);
    if (bad) s = -1;
    s_seq[tid] = s;
    s_oth[tid] = o;
  }
  __syncthreads();
  // Warps take 32 places of a row each, up to kTake of them at once. The first are loaded beside the lengths.
  const int parts = up(b.table_stride, 32), step = gridDim.x * warps;
  const int64_t items = static_cast<int64_t>(n) * parts;   // up to 1024 rows of 2^21 parts
  int pg[kTake], e[kTake], x[kTake];   // the pages, their entries, their places
  const int64_t first = rank * warps + warp;
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int u = 0; u < kTake; ++u) {
      pg[u] = kNone;
      if (i0 + u * step >= items) continue;
      const uint32_t i = static_cast<uint32_t>(i0 + u * step);
      e[u] = i / parts;
      x[u] = (i - e[u] * parts) * 32 + lane;
      if (x[u] < b.table_stride && s_seq[e[u]] >= 0) pg[u] = b.table[static_cast<int64_t>(s_seq[e[u]]) * b.table_stride + x[u]];
    }
  };
  load(first);
  if (tid < n && !bad) {
    len = b.lens[s];
    bad = len < 0 || len > static_cast<int64_t>(b.table_stride) * b.page || (kFork && b.lens[o] != 0);
    s_len[tid] = len;
    // fork: a target appears once and is no source; release: a sequence appears once
    named.put(kFork ? o : s, &again);
    bad |= again;
  }
  __syncthreads();
  if (kFork && tid < n && s >= 0) bad |= named.has(s);
  int why = __syncthreads_or(bad) ? FM_KV_BAD_ENTRY : 0;   // the same in every CTA
  const bool sound = why == 0;
  // Calls f for each share of the places: of a fork's whole row, of a release's from the first one that it empties.
  const bool once = items <= kTake * step;
  auto every = [&](auto f, bool loaded) {
    for (int64_t i0 = first; i0 < items; i0 += kTake * step) {
      if (!loaded && !once) load(i0);
      loaded = false;
#pragma unroll
      for (int u = 0; u < kTake; ++u)
        if (pg[u] != kNone) pg[u] = kFork || x[u] >= places_of(min(s_len[e[u]], s_oth[e[u]]), b) ? max(pg[u], -1) : kNone;
      f();
    }
  };
  auto in_pool = [&](int p) { return p >= 0 && p < b.pages; };
  if (sound) {
    bool wrong = false;
    every([&] {
      int refs[kTake];
#pragma unroll
      for (int u = 0; u < kTake; ++u) {
        refs[u] = 1;
        if (in_pool(pg[u])) refs[u] = kFork ? b.refs[pg[u]] : atomicSub(&b.refs[pg[u]], 1);
      }
#pragma unroll
      for (int u = 0; u < kTake; ++u)
        wrong |= pg[u] != kNone && (refs[u] < 1 || pg[u] >= b.pages || (pg[u] < 0 && x[u] < places_of(s_len[e[u]], b)));
    }, true);
    why = __syncthreads_or(wrong) ? FM_KV_BAD_ENTRY : 0;
  }
  if (gridDim.x > 1) {   // what one CTA met all of them learn
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (why && tid < static_cast<int>(gridDim.x))
      asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(map_dsmem(smem_u32(&s_wrong), tid)), "r"(why) : "memory");
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    why |= *static_cast<volatile int*>(&s_wrong);
  }
  if (rank == 0 && tid == 0) {
    status[0] = why;
    status[1] = 0;
  }
  if (why == 0) {
    every([&] {   // a row's unused places are -1 and copied like the rest
#pragma unroll
      for (int u = 0; u < kTake; ++u) {
        if (pg[u] == kNone) continue;
        b.table[static_cast<int64_t>(kFork ? s_oth[e[u]] : s_seq[e[u]]) * b.table_stride + x[u]] = kFork ? pg[u] : -1;
        if (kFork && pg[u] >= 0) atomicAdd(&b.refs[pg[u]], 1);
      }
    }, false);
    for (int i = rank * blockDim.x + tid; i < n; i += gridDim.x * blockDim.x)
      b.lens[kFork ? s_oth[i] : s_seq[i]] = kFork ? s_len[i] : min(s_len[i], s_oth[i]);
  } else if (sound && !kFork) {
    every([&] {
#pragma unroll
      for (int u = 0; u < kTake; ++u)
        if (in_pool(pg[u])) atomicAdd(&b.refs[pg[u]], 1);
    }, false);
  }
}

// fm_kv_compact, the plan: live pages from n_live on move, in order, into the free ones below n_live, in order.
// One CTA, bound by latency: two walks over refs (held in registers up to 4096 pages).
// head: [0] n_live, [1] moves, [2] where they begin in src; src, dst: the moves; map: the new place of every page from n_live on (-1: free).
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) compact_plan_kernel(Book b, int32_t* status, int32_t* head, int32_t* src,
                                                                    int32_t* dst, int32_t* map) {
  __shared__ int s_sums[32], s_below;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const PageWalk<THREADS> walk(b);
  int mine = 0;
  walk.each(b, [&](int, bool in, int refs) { mine += __popc(__ballot_sync(0xffffffffu, in && refs > 0)); });
  int n_live = 0;
  int rank = __shfl_sync(0xffffffffu, block_exclusive<THREADS>(lane == 0 ? mine : 0, s_sums, &n_live), 0);
  if (tid == 0) s_below = n_live;
  __syncthreads();
  // with `at` live pages before it, a live page is the at-th of src, a free one below n_live the (pg - at)-th hole
  walk.each(b, [&](int pg, bool in, int refs) {
    const bool live = in && refs > 0;
    const unsigned m = __ballot_sync(0xffffffffu, live);
    const int at = rank + __popc(m & ((1u << lane) - 1));
    if (live && pg >= n_live) src[at] = pg;
    if (in && !live) {
      if (pg < n_live)
        dst[pg - at] = pg;
      else
        map[pg] = -1;
    }
    if (in && pg == n_live) s_below = at;
    rank += __popc(m);
  });
  __syncthreads();
  const int below = s_below, moves = n_live - below;   // live pages below n_live; as many free ones there as live above
  for (int i = tid; i < moves; i += THREADS) {
    const int from = src[below + i], to = dst[i];
    map[from] = to;
    b.refs[to] = b.refs[from];
    b.refs[from] = 0;
  }
  if (tid == 0) {
    head[0] = n_live;
    head[1] = moves;
    head[2] = below;
    status[0] = 0;
    status[1] = moves;
  }
}

// The moves (sources and targets are disjoint) and the table's new page numbers: 88 MB read and written in 25 us, 7 TB/s
// (part of what is written stays in L2).
__global__ void __launch_bounds__(256) compact_move_kernel(Pool p, Book b, const int32_t* head, const int32_t* src,
                                                           const int32_t* dst, const int32_t* map) {
  pdl_trigger();
  pdl_wait();
  const int n_live = head[0], moves = head[1];
  src += head[2];
  const int64_t items = static_cast<int64_t>(moves) * p.layers;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int m = static_cast<int>(i % moves);
    copy_rows(p, static_cast<int>(i / moves), src[m], dst[m], b.page);
  }
  const int64_t cells = static_cast<int64_t>(b.seqs) * b.table_stride;
  for (int64_t x = blockIdx.x * 256ll + threadIdx.x; x < cells; x += gridDim.x * 256ll) {
    const int pg = b.table[x];
    if (pg >= n_live && pg < b.pages) b.table[x] = map[pg];
  }
}

// ---------------------------------------------------------------- rotary positions and the store

struct AppendParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* q_out;
  int64_t qs, ks, vs, os;   // elements between tokens
  const int32_t *start, *seq, *lens, *table, *positions;
  const uint64_t* freq;     // turns per position * 2^64 of each pair
  float mag;
  int rot, interleaved;
  int tokens, max_tokens, seqs, table_stride, pages, page, shift;
  int H, Hkv, Dh;
  int toks, groups;         // tokens of a CTA, threads that share the heads of a token
  const float *q_gamma, *k_gamma;   // normalised heads: [Dh] or null
  float eps;
  void *kc, *vc;            // this layer
  int64_t pg, tok, head;    // strides in elements
  const float *k_scale, *v_scale;
  int* err;
};

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void unpack8(uint4 u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(bf2(f[0], f[1]), bf2(f[2], f[3]), bf2(f[4], f[5]), bf2(f[6], f[7]));
}
__device__ __forceinline__ uint2 codes8(const float* f, float rs) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(f[i] * rs, f[i + 1] * rs), __NV_SATFINITE, __NV_E4M3);
    w[i >> 2] |= c << (8 * (i & 2));
  }
  return make_uint2(w[0], w[1]);
}

// One CTA: `toks` tokens of an entry (grid.y), all heads. The angles of a token are computed once, a thread each, into
// shared memory: computed by every thread for its own pairs they were a third of the kernel's instructions. An angle is
// a fraction of a turn in 64-bit fixed point: position * freq modulo 2^64 drops whole turns exactly, at any position,
// without double precision. One thread: 16 elements (two 8-element chunks that hold whole pairs) of every groups-th
// head. Bound by HBM: q, k and v are read once and written once (9600 tokens of 16 + 2 x 4 heads of 128, half of each
// rotated, bf16 cache: 23.2 us, 5.1 TB/s; 32 single tokens: 2.5 us, launch).
// LANES > 0: every head of q and k is divided by its root mean square and multiplied by gamma before it turns. A head's threads
// are LANES neighbouring lanes, a power of two (some of them idle where Dh / 16 is none), which add their squares by shuffles.
// The same bytes as without the norm and, with 64 registers and shared memory free of conflicts, the same time: 23.0 us for
// those 9600 tokens, 5.1 TB/s (four heads' loads at once in 107 registers: 35 us; conflicts in the angles and gammas: 29 us).
template <bool F8, int LANES>
__global__ void __launch_bounds__(256, 4) append_kernel(const AppendParams p) {
  // [toks][rot / 2] (cos, sin) times magnitude; NORM: then [2][Dh] gammas, and both in the order in which neighbouring lanes
  // read 16 bytes each: [16-byte piece of a unit][unit] (in the order of the elements four lanes met in a bank)
  extern __shared__ float2 s_angle[];
  constexpr bool NORM = LANES > 0;
  pdl_trigger();
  const int units = p.Dh / 16, pairs = p.rot / 2, lanes = NORM ? LANES : units;
  const int unit = threadIdx.x % lanes, tok = (threadIdx.x / lanes) % p.toks, grp = threadIdx.x / (lanes * p.toks);
  const int entry = blockIdx.y;
  pdl_wait();
  const int begin = p.start[entry], nq = p.start[entry + 1] - begin;
  const int sid = p.seq ? p.seq[entry] : entry;
  const bool bad = begin < 0 || nq < 0 || begin > p.tokens || nq > p.tokens - begin || sid < 0 || sid >= p.seqs;
  const int len = bad ? 0 : p.lens[sid];
  const bool over = bad || nq > p.max_tokens || len < nq || len > p.table_stride * static_cast<int64_t>(p.page);
  if (over && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, kErrBadBatch);
  const int first = blockIdx.x * p.toks, end = min(nq, p.max_tokens);
  if (bad || first >= end) return;   // the same for the whole CTA
  const int past = len - nq;
  // chunks of this unit (in 8 elements): a rotated pair of chunks, or two that pass through
  const int rot_units = p.rot / 16;
  const bool turned = unit < rot_units, split = turned && !p.interleaved;
  const bool idle = NORM && unit >= units;   // takes part in the shuffles only; its places are those of unit 0
  const int c0 = idle ? 0 : (split ? unit : 2 * unit) * 8, c1 = idle ? 0 : (split ? unit + rot_units : 2 * unit + 1) * 8;
  struct Raw {   // a thread's part of a head
    uint4 a, b;
  };
  auto load = [&](const __nv_bfloat16* head) {
    Raw r = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (!idle) r = {*reinterpret_cast<const uint4*>(head + c0), *reinterpret_cast<const uint4*>(head + c1)};
    return r;
  };
  [[maybe_unused]] Raw ahead = {};   // NORM: the first query head, loaded while the angles are computed
  [[maybe_unused]] float* s_gamma = reinterpret_cast<float*>(s_angle + p.toks * pairs);
  if constexpr (NORM) {
    if (grp < p.groups && first + tok < end && grp < p.H)
      ahead = load(p.q + (begin + static_cast<int64_t>(first) + tok) * p.qs + grp * p.Dh);
    for (int x = threadIdx.x; x < 2 * p.Dh; x += 256) {
      const float* src = x < p.Dh ? p.q_gamma : p.k_gamma;
      const int el = x < p.Dh ? x : x - p.Dh, chunk = el / 8;
      const bool apart = !p.interleaved && chunk < 2 * rot_units;   // a unit's two chunks
      const int of = apart ? chunk % rot_units : chunk / 2, piece = (apart ? chunk / rot_units : chunk % 2) * 2 + el % 8 / 4;
      s_gamma[x - el + (piece * units + of) * 4 + el % 4] = src ? src[el] : 1.0f;
    }
  }
  for (int x = threadIdx.x; x < p.toks * pairs; x += 256) {
    const int i = x % pairs, w = first + x / pairs;
    if (w >= end) break;
    const int64_t at = p.positions ? p.positions[begin + w] : past + w;
    // the fraction of a turn as a signed 32-bit number: half turns in [-1, 1) for sincospif
    const uint64_t turn = p.freq[i] * static_cast<uint64_t>(at) + (1ull << 31);
    float2 a;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &a.y, &a.x);
    // a unit's eight pairs are four 16-byte pieces
    const int place = NORM ? x - i + (i % 8 / 2 * rot_units + i / 8) * 2 + i % 2 : x;
    s_angle[place] = make_float2(a.x * p.mag, a.y * p.mag);
  }
  const int within = first + tok;
  const bool mine = grp < p.groups && within < end;
  const int64_t token = begin + static_cast<int64_t>(within);
  const int64_t pos = static_cast<int64_t>(past) + within;   // place in the sequence
  int page = -1;
  if (mine && pos >= 0 && (pos >> p.shift) < p.table_stride)
    page = p.table[static_cast<int64_t>(sid) * p.table_stride + (pos >> p.shift)];
  if (page >= p.pages) page = -1;
  if (mine && page < 0 && unit == 0 && grp == 0) atomicOr(p.err, kErrBadBatch);
  __syncthreads();
  if (!mine) return;
  float2 ang[8];
  auto angles = [&] {
    const float4* src = reinterpret_cast<const float4*>(s_angle + tok * pairs + unit * (NORM ? 2 : 8));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[NORM ? i * rot_units : i];
      ang[2 * i] = make_float2(v.x, v.y);
      ang[2 * i + 1] = make_float2(v.z, v.w);
    }
  };
  if (!NORM && turned) angles();
  auto turn = [&](float* a, float* b) {
    if (!turned) return;
    if (NORM) angles();   // from shared memory every time: 16 registers fewer, more CTAs an SM
    if (p.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
        a[2 * i] = a0 * ang[i].x - a1 * ang[i].y;
        a[2 * i + 1] = a1 * ang[i].x + a0 * ang[i].y;
        b[2 * i] = b0 * ang[4 + i].x - b1 * ang[4 + i].y;
        b[2 * i + 1] = b1 * ang[4 + i].x + b0 * ang[4 + i].y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x0 = a[i], x1 = b[i];
        a[i] = x0 * ang[i].x - x1 * ang[i].y;
        b[i] = x1 * ang[i].x + x0 * ang[i].y;
      }
    }
  };
  if constexpr (NORM) {
    const uint32_t team = ((1u << LANES) - 1u) << (threadIdx.x & 31 & ~(LANES - 1));
    auto reduce = [&](float v, auto join) {   // over the head's lanes, in a fixed order, the same in all of them
#pragma unroll
      for (int o = LANES >> 1; o > 0; o >>= 1) v = join(v, __shfl_xor_sync(team, v, o));
      return v;
    };
    const float rdh = 1.0f / p.Dh;
    // two elements an instruction
    auto squares = [&](const float2* a, const float2* b) {
      float2 s = mul2(a[0], a[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s = fma2(a[e], a[e], s);
#pragma unroll
      for (int e = 0; e < 4; ++e) s = fma2(b[e], b[e], s);
      return reduce(s.x + s.y, [](float x, float y) { return x + y; });
    };
    auto normalise = [&](float2* a, float2* b, const float* gamma) {
      const float ms = fmaf(squares(a, b), rdh, p.eps);
      float rr = rsqrtf(ms);
      // Squares out of fp32's range, the same in all of the head's lanes: the head is taken times the power of two that puts
      // the larger of its maximum and sqrt(eps) into [2, 4). A head with a NaN or an infinity is NaN throughout.
      if (!(ms >= 0x1p-100f && ms < INFINITY)) {
        const auto larger = [](float x, float y) { return x > y || x != x ? x : y; };   // NaN if either is
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          top = larger(larger(larger(larger(top, fabsf(a[e].x)), fabsf(a[e].y)), fabsf(b[e].x)), fabsf(b[e].y));
        top = reduce(top, larger);
        const uint32_t ex = __float_as_uint(fmaxf(top, sqrtf(p.eps))) >> 23;
        const float f = __uint_as_float((255 - min(max(ex, 1u), 254u)) << 23);
        const float2 ff = make_float2(f, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = mul2(a[e], ff), b[e] = mul2(b[e], ff);
        const float scaled = squares(a, b) * rdh + p.eps * f * f;
        rr = !(top < INFINITY) ? NAN : scaled > 0.f ? 1.0f / sqrtf(scaled) : 0.f;
      }
      const float2 r2 = make_float2(rr, rr);
      const float4* g = reinterpret_cast<const float4*>(gamma) + (idle ? 0 : unit);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 v = g[e * units];
        float2* x = (e < 2 ? a : b) + (e & 1) * 2;
        x[0] = mul2(x[0], mul2(r2, make_float2(v.x, v.y)));
        x[1] = mul2(x[1], mul2(r2, make_float2(v.z, v.w)));
      }
    };
    auto normalised = [&](const Raw& r, const float* gamma, float* a, float* b) {
      unpack8(r.a, a);
      unpack8(r.b, b);
      normalise(reinterpret_cast<float2*>(a), reinterpret_cast<float2*>(b), gamma);
      turn(a, b);
    };
    {   // ---- queries: the next head is on its way while one is computed
      const __nv_bfloat16* src = p.q + token * p.qs + grp * p.Dh;
      __nv_bfloat16* dst = p.q_out + token * p.os + grp * p.Dh;
      const int step = p.groups * p.Dh;
#pragma unroll 1
      for (int h = grp; h < p.H; h += p.groups, dst += step) {
        const Raw r = ahead;
        src += step;
        if (h + p.groups < p.H) ahead = load(src);
        float a[8], b[8];
        normalised(r, s_gamma, a, b);
        if (idle) continue;
        *reinterpret_cast<uint4*>(dst + c0) = pack8(a);
        *reinterpret_cast<uint4*>(dst + c1) = pack8(b);
      }
    }
    if (page < 0) return;
    // ---- keys and values, the groups in turn where the queries' left off
    const int64_t cell = static_cast<int64_t>(page) * p.pg + (pos & (p.page - 1)) * p.tok;
    const float rk = F8 ? 1.0f / *p.k_scale : 1.0f, rv = F8 ? 1.0f / *p.v_scale : 1.0f;
    int h = grp - p.H % p.groups;
    if (h < 0) h += p.groups;
    auto row = [&](int x) { return x < p.Hkv ? p.k + token * p.ks + x * p.Dh : p.v + token * p.vs + (x - p.Hkv) * p.Dh; };
    if (h < 2 * p.Hkv) ahead = load(row(h));
#pragma unroll 1
    for (; h < 2 * p.Hkv; h += p.groups) {
      const bool is_v = h >= p.Hkv;
      const Raw r = ahead;
      if (h + p.groups < 2 * p.Hkv) ahead = load(row(h + p.groups));
      const int64_t at = cell + (is_v ? h - p.Hkv : h) * p.head;
      if (!F8 && is_v) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.vc) + at;
        if (idle) continue;
        *reinterpret_cast<uint4*>(dst + c0) = r.a;
        *reinterpret_cast<uint4*>(dst + c1) = r.b;
        continue;
      }
      float a[8], b[8];
      if (is_v) {
        unpack8(r.a, a);
        unpack8(r.b, b);
      } else {
        normalised(r, s_gamma + p.Dh, a, b);
      }
      if (idle) continue;
      if constexpr (F8) {
        uint8_t* dst = static_cast<uint8_t*>(is_v ? p.vc : p.kc) + at;
        *reinterpret_cast<uint2*>(dst + c0) = codes8(a, is_v ? rv : rk);
        *reinterpret_cast<uint2*>(dst + c1) = codes8(b, is_v ? rv : rk);
      } else {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.kc) + at;
        *reinterpret_cast<uint4*>(dst + c0) = pack8(a);
        *reinterpret_cast<uint4*>(dst + c1) = pack8(b);
      }
    }
    return;
  }
  {   // ---- queries
    const __nv_bfloat16* src = p.q + token * p.qs;
    __nv_bfloat16* dst = p.q_out + token * p.os;
#pragma unroll 4
    for (int h = grp; h < p.H; h += p.groups) {
      const uint4 u = *reinterpret_cast<const uint4*>(src + h * p.Dh + c0), w = *reinterpret_cast<const uint4*>(src + h * p.Dh + c1);
      if (!turned) {
        *reinterpret_cast<uint4*>(dst + h * p.Dh + c0) = u;
        *reinterpret_cast<uint4*>(dst + h * p.Dh + c1) = w;
        continue;
      }
      float a[8], b[8];
      unpack8(u, a);
      unpack8(w, b);
      turn(a, b);
      *reinterpret_cast<uint4*>(dst + h * p.Dh + c0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + h * p.Dh + c1) = pack8(b);
    }
  }
  if (page < 0) return;
  // ---- keys and values
  const int64_t cell = static_cast<int64_t>(page) * p.pg + (pos & (p.page - 1)) * p.tok;
  const float rk = F8 ? 1.0f / *p.k_scale : 1.0f, rv = F8 ? 1.0f / *p.v_scale : 1.0f;
  // heads go round the groups where the queries' left off, so that a small batch spreads over all of them
  int h = grp - p.H % p.groups;
  if (h < 0) h += p.groups;
#pragma unroll 2
  for (; h < 2 * p.Hkv; h += p.groups) {
    const bool is_v = h >= p.Hkv;
    const int hh = is_v ? h - p.Hkv : h;
    const __nv_bfloat16* src = (is_v ? p.v + token * p.vs : p.k + token * p.ks) + hh * p.Dh;
    const uint4 u = *reinterpret_cast<const uint4*>(src + c0), w = *reinterpret_cast<const uint4*>(src + c1);
    const int64_t at = cell + hh * p.head;
    if (!F8 && (is_v || !turned)) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(is_v ? p.vc : p.kc) + at;
      *reinterpret_cast<uint4*>(dst + c0) = u;
      *reinterpret_cast<uint4*>(dst + c1) = w;
      continue;
    }
    float a[8], b[8];
    unpack8(u, a);
    unpack8(w, b);
    if (!is_v) turn(a, b);
    if constexpr (F8) {
      uint8_t* dst = static_cast<uint8_t*>(is_v ? p.vc : p.kc) + at;
      *reinterpret_cast<uint2*>(dst + c0) = codes8(a, is_v ? rv : rk);
      *reinterpret_cast<uint2*>(dst + c1) = codes8(b, is_v ? rv : rk);
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.kc) + at;
      *reinterpret_cast<uint4*>(dst + c0) = pack8(a);
      *reinterpret_cast<uint4*>(dst + c1) = pack8(b);
    }
  }
}

// ---------------------------------------------------------------- pages -> a policy's prefix

struct PrefixParams {
  const uint8_t *k, *v;
  int f8;
  int64_t layer, pg, tok, head;   // bytes
  const float *k_scale, *v_scale;
  const int32_t *table, *lens;
  int seq, seq_tok, rows, table_stride, pages, page, shift, Hkv, Dh;
  __nv_bfloat16 *kcache, *vt;
  int P, p_pad, tok_begin;
  int* err;
};

constexpr int kPrefixTile = 64;

// 16-bit values of 8 elements of a page row.
__device__ __forceinline__ uint4 row_chunk(const uint8_t* row, int c, int f8, float scale) {
  if (!f8) return reinterpret_cast<const uint4*>(row)[c];
  const uint2 u = reinterpret_cast<const uint2*>(row)[c];
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? u.x : u.y;
    const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>((w >> (8 * (i & 3))) & 0xff), __NV_E4M3);
    f[i] = __half2float(__half(h)) * scale;
  }
  return pack8(f);
}

// One CTA: 64 tokens of one layer and head; keys are copied, values are read as rows and turned through shared memory, so
// that a warp stores 64 contiguous bytes along the tokens (two a lane: tok_begin may be odd). Bound by its launch, the chain
// length -> page -> row and these narrow stores: 788 tokens of 18 layers and one head of 128 take 4.4 us in a graph with bf16
// pages, 5.3 us with E4M3 (14.5 MB read and written: 2.1 us at HBM's rate).
__global__ void __launch_bounds__(256) prefix_kernel(const PrefixParams p) {
  extern __shared__ uint16_t s_v[];   // [64][Dh + 2]
  const int layer = blockIdx.z, g = blockIdx.y, t0 = blockIdx.x * kPrefixTile;
  const int len = p.lens[p.seq];
  const int chunks = p.Dh / 8, pitch = p.Dh + 2;
  const float ks = p.f8 ? p.k_scale[layer] : 1.f, vs = p.f8 ? p.v_scale[layer] : 1.f;
  for (int x = threadIdx.x; x < kPrefixTile * chunks; x += 256) {
    const int r = x / chunks, c = x % chunks, t = t0 + r;
    if (t >= p.rows) break;
    const int64_t pos = static_cast<int64_t>(p.seq_tok) + t;
    int page = -1;
    if (pos < len && (pos >> p.shift) < p.table_stride)
      page = p.table[static_cast<int64_t>(p.seq) * p.table_stride + (pos >> p.shift)];
    if (page >= p.pages) page = -1;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (page >= 0) {
      const int64_t off = layer * p.layer + page * p.pg + (pos & (p.page - 1)) * p.tok + g * p.head;
      k = row_chunk(p.k + off, c, p.f8, ks);
      v = row_chunk(p.v + off, c, p.f8, vs);
    } else if (c == 0) {
      atomicOr(p.err, kErrBadBatch);
    }
    reinterpret_cast<uint4*>(p.kcache + ((static_cast<int64_t>(layer) * p.P + p.tok_begin + t) * p.Hkv + g) * p.Dh)[c] = k;
    uint32_t* d = reinterpret_cast<uint32_t*>(s_v + r * pitch + c * 8);
    d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
  }
  __syncthreads();
  const int n = min(kPrefixTile, p.rows - t0);
  for (int x = threadIdx.x; x < kPrefixTile * p.Dh; x += 256) {
    const int r = x % kPrefixTile, d = x / kPrefixTile;
    if (r < n)
      reinterpret_cast<uint16_t*>(p.vt)[((static_cast<int64_t>(layer) * p.Hkv + g) * p.Dh + d) * p.p_pad + p.tok_begin +
                                        t0 + r] = s_v[r * pitch + d];
  }
}

int shift_of(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

Book book_of(const fm_kv_cache& c) {
  return Book{c.table, c.lens, c.refs, c.seqs, c.table_stride, c.pages, c.page_tokens, shift_of(c.page_tokens)};
}

Pool pool_of(const fm_kv_cache& c) {
  const int eb = c.fmt == FM_FMT_FP8 ? 1 : 2, per = 16 / eb;
  Pool p;
  p.k = static_cast<uint4*>(c.k);
  p.v = static_cast<uint4*>(c.v);
  p.layer = c.layer_stride / per;
  p.pg = c.page_stride / per;
  p.tok = c.token_stride / per;
  p.head = c.head_stride / per;
  p.layers = c.layers;
  p.Hkv = c.Hkv;
  p.chunks = c.Dh / per;
  const bool one = c.Hkv == 1;
  if ((one || c.head_stride == c.Dh) && c.token_stride == static_cast<int64_t>(c.Hkv) * c.Dh)
    p.runs = kRunAll;
  else if (c.token_stride == c.Dh)
    p.runs = kRunHead;
  else
    p.runs = kRunRow;
  return p;
}

size_t align16(size_t v) { return (v + 15) / 16 * 16; }
// Workspace: n copy records, then max(pages for a reserve's free list, the compaction's lists: head, src, dst, map).
size_t kv_workspace(const fm_kv_cache& c, int n) {
  return align16(n * sizeof(Copy)) + align16((4 + 3 * static_cast<size_t>(c.pages)) * sizeof(int32_t));
}

int page_call_check(const fm_kv_cache* c, int n, const void* status) {
  const int st = kv_check(c);
  if (st != FM_OK) return st;
  if (!c->refs || !status) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  if (n < 0 || n > kMaxEntries) return record_error(FM_ERR_SHAPE, "a call takes 0 to 1024 sequences");
  return FM_OK;
}

int workspace_check(const fm_kv_cache& c, int n, const void* ws, size_t bytes) {
  if (!ws) return record_error(FM_ERR_INVALID_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) % 16) return record_error(FM_ERR_ALIGN, "workspace not 16-byte aligned");
  if (bytes < kv_workspace(c, n)) return record_error(FM_ERR_WORKSPACE, "workspace smaller than fm_kv_workspace_size()");
  return FM_OK;
}

int done(cudaError_t e) { return e == cudaSuccess ? FM_OK : record_error(FM_ERR_CUDA, cudaGetErrorString(e)); }

LaunchOpts opts(void* stream) {
  LaunchOpts o;
  o.stream = static_cast<cudaStream_t>(stream);
  o.pdl = true;
  return o;
}

template <bool kFork>
int share(const fm_kv_cache* c, const int32_t* seq, const int32_t* other, int n, int32_t* status, void* stream) {
  LaunchOpts o = opts(stream);
  // A warp a part of 32 places while the cluster has enough of them; the CTAs that this needs, since barriers and a
  // cluster's start are most of a small call (a fork and its release of 8 rows of 50 pages: 5.1 us in one CTA, 6.3 in two).
  const int64_t items = static_cast<int64_t>(n) * up(c->table_stride, 32);
  const int threads = items <= kSmallThreads / 32 ? kSmallThreads : kBookThreads;
  int ctas = 1;
  while (ctas < kForkCluster && ctas * threads / 32 < items) ctas *= 2;
  o.cluster = dim3(ctas, 1, 1);
  // more parts than warps: four at once, eight where four would take a second round (512 rows of two parts: 12.5 us with
  // four, 14.1 with eight; 1024: 24.3 and 20.2)
  const int64_t each = up(items, ctas * threads / 32);
  auto kernel = each <= 1 ? share_kernel<kFork, 1> : each <= 4 ? share_kernel<kFork, 4> : share_kernel<kFork, 8>;
  return done(launch(kernel, dim3(ctas), dim3(threads), 0, o, book_of(*c), seq, other, n, status));
}

}  // namespace

int kv_check(const fm_kv_cache* c) {
  if (!c || !c->k || !c->v || !c->table || !c->lens) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  if (c->fmt != FM_FMT_BF16 && c->fmt != FM_FMT_FP8) return record_error(FM_ERR_INVALID_ARG, "cache format must be BF16 or FP8");
  if (c->fmt == FM_FMT_FP8 && (!c->k_scale || !c->v_scale))
    return record_error(FM_ERR_INVALID_ARG, "an FP8 cache needs its k_scale and v_scale");
  if (c->layers < 1 || c->pages < 1 || c->Hkv < 1 || c->seqs < 1 || c->table_stride < 1)
    return record_error(FM_ERR_SHAPE, "layers, pages, Hkv, seqs and table_stride must be positive");
  if (c->page_tokens < 16 || c->page_tokens > 256 || (c->page_tokens & (c->page_tokens - 1)))
    return record_error(FM_ERR_SHAPE, "page_tokens must be 16, 32, 64, 128 or 256");
  if (c->Dh < 16 || c->Dh > 256 || c->Dh % 16) return record_error(FM_ERR_SHAPE, "Dh must be a multiple of 16 up to 256");
  if (c->layers > 65535 || c->Hkv > 65535 || c->pages > (1 << 30))
    return record_error(FM_ERR_SHAPE, "layers and Hkv up to 65535, pages up to 2^30");
  if (static_cast<int64_t>(c->table_stride) * c->page_tokens > (1 << 30))
    return record_error(FM_ERR_SHAPE, "table_stride * page_tokens exceeds 2^30 tokens");
  // the pages that all rows together could ask for stay countable in 32 bits
  if (static_cast<int64_t>(c->table_stride) * c->seqs > INT32_MAX)
    return record_error(FM_ERR_SHAPE, "the table has more than 2^31 - 1 places");
  if (reinterpret_cast<uintptr_t>(c->k) % 16 || reinterpret_cast<uintptr_t>(c->v) % 16)
    return record_error(FM_ERR_ALIGN, "k and v must be 16-byte aligned");
  // rows must not overlap: each stride (of an extent above 1) spans all that is inside of it
  const int eb = c->fmt == FM_FMT_FP8 ? 1 : 2;
  struct { int64_t stride, extent; } d[4] = {{c->token_stride, c->page_tokens}, {c->head_stride, c->Hkv},
                                             {c->page_stride, c->pages}, {c->layer_stride, c->layers}};
  std::sort(d, d + 4, [](const auto& a, const auto& b) { return a.stride < b.stride; });
  int64_t span = c->Dh;
  for (const auto& x : d) {
    if (x.extent == 1) continue;
    if (x.stride < span || x.stride >= (int64_t(1) << 40) / eb) return record_error(FM_ERR_SHAPE, "cache strides overlap or are too large");
    if (x.stride * eb % 16) return record_error(FM_ERR_SHAPE, "cache strides must be multiples of 16 bytes");
    // nothing that the next dims' strides are held against, and no address, leaves 64 bits
    if (x.extent - 1 > ((int64_t(1) << 56) - span) / x.stride) return record_error(FM_ERR_SHAPE, "the cache exceeds 2^56 elements");
    span += x.stride * (x.extent - 1);
  }
  return FM_OK;
}

int kv_batch_check(const fm_kv_cache* c, const fm_kv_batch* b) {
  if (!b) return record_error(FM_ERR_INVALID_ARG, "NULL batch");
  if (b->n < 0 || b->tokens < 0 || b->max_tokens < 0 || b->max_len < 0)
    return record_error(FM_ERR_SHAPE, "a batch's counts must not be negative");
  if (b->n > 65535) return record_error(FM_ERR_SHAPE, "a batch takes up to 65535 entries");
  if (b->n > 0 && !b->start) return record_error(FM_ERR_INVALID_ARG, "the batch has no start");
  if (b->n > 0 && !b->seq && b->n > c->seqs)
    return record_error(FM_ERR_SHAPE, "without seq, entry i is sequence i: n must not exceed the cache's seqs");
  return FM_OK;
}

cudaError_t prefix_from_pages_launch(const fm_kv_cache& c, int seq, int seq_tok, int rows, __nv_bfloat16* kcache,
                                     __nv_bfloat16* vtcache, int P, int p_pad, int tok_begin, int* err, cudaStream_t st) {
  const int eb = c.fmt == FM_FMT_FP8 ? 1 : 2;
  PrefixParams p;
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.f8 = eb == 1;
  p.layer = c.layer_stride * eb;
  p.pg = c.page_stride * eb;
  p.tok = c.token_stride * eb;
  p.head = c.head_stride * eb;
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.table = c.table;
  p.lens = c.lens;
  p.seq = seq;
  p.seq_tok = seq_tok;
  p.rows = rows;
  p.table_stride = c.table_stride;
  p.pages = c.pages;
  p.page = c.page_tokens;
  p.shift = shift_of(c.page_tokens);
  p.Hkv = c.Hkv;
  p.Dh = c.Dh;
  p.kcache = kcache;
  p.vt = vtcache;
  p.P = P;
  p.p_pad = p_pad;
  p.tok_begin = tok_begin;
  p.err = err;
  LaunchOpts o;
  o.stream = st;
  return launch(prefix_kernel, dim3(up(rows, kPrefixTile), c.Hkv, c.layers), dim3(256),
                static_cast<size_t>(kPrefixTile) * (c.Dh + 2) * 2, o, p);
}

}  // namespace fm

using namespace fm;

extern "C" int fm_kv_workspace_size(const fm_kv_cache* c, int n, size_t* bytes) {
  if (!bytes) return record_error(FM_ERR_INVALID_ARG, "bytes is NULL");
  const int st = kv_check(c);
  if (st != FM_OK) return st;
  if (n < 0 || n > kMaxEntries) return record_error(FM_ERR_SHAPE, "a call takes 0 to 1024 sequences");
  *bytes = kv_workspace(*c, n);
  return FM_OK;
}

extern "C" int fm_kv_reserve(const fm_kv_cache* c, const int32_t* seq, const int32_t* count, int n, int32_t* status,
                             void* workspace, size_t workspace_bytes, void* stream) {
  int st = page_call_check(c, n, status);
  if (st != FM_OK) return st;
  if (n > 0 && (!seq || !count)) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  st = workspace_check(*c, n, workspace, workspace_bytes);
  if (st != FM_OK) return st;
  Copy* copies = static_cast<Copy*>(workspace);
  int32_t* fresh = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + align16(n * sizeof(Copy)));
  const LaunchOpts o = opts(stream);
  const bool small = n <= kSmallThreads && c->pages <= kSmallPages;
  cudaError_t e = launch(small ? reserve_kernel<kSmallThreads> : reserve_kernel<kBookThreads>, dim3(1),
                         dim3(small ? kSmallThreads : kBookThreads), 0, o, book_of(*c), seq, count, n, status, copies, fresh);
  if (e == cudaSuccess && n > 0)
    e = launch(copy_shared_kernel, dim3(n, c->layers), dim3(256), 0, o, pool_of(*c), static_cast<const Copy*>(copies));
  return done(e);
}

extern "C" int fm_kv_fork(const fm_kv_cache* c, const int32_t* src, const int32_t* dst, int n, int32_t* status, void* stream) {
  const int st = page_call_check(c, n, status);
  if (st != FM_OK) return st;
  if (n > 0 && (!src || !dst)) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  return share<true>(c, src, dst, n, status, stream);
}

extern "C" int fm_kv_release(const fm_kv_cache* c, const int32_t* seq, const int32_t* keep, int n, int32_t* status,
                             void* stream) {
  const int st = page_call_check(c, n, status);
  if (st != FM_OK) return st;
  if (n > 0 && !seq) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  return share<false>(c, seq, keep, n, status, stream);
}

extern "C" int fm_kv_compact(const fm_kv_cache* c, int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  int st = page_call_check(c, 0, status);
  if (st != FM_OK) return st;
  st = workspace_check(*c, 0, workspace, workspace_bytes);
  if (st != FM_OK) return st;
  int32_t* head = static_cast<int32_t*>(workspace);
  int32_t *src = head + 4, *dst = src + c->pages, *map = dst + c->pages;
  const LaunchOpts o = opts(stream);
  const bool small = c->pages <= kSmallPages;
  cudaError_t e = launch(small ? compact_plan_kernel<kSmallThreads> : compact_plan_kernel<kBookThreads>, dim3(1),
                         dim3(small ? kSmallThreads : kBookThreads), 0, o, book_of(*c), status, head, src, dst, map);
  if (e == cudaSuccess)
    e = launch(compact_move_kernel, dim3(152 * 8), dim3(256), 0, o, pool_of(*c), book_of(*c), static_cast<const int32_t*>(head),
               static_cast<const int32_t*>(src), static_cast<const int32_t*>(dst), static_cast<const int32_t*>(map));
  return done(e);
}

extern "C" int fm_rope_table(const fm_rope_config* r, uint64_t* freq, float* magnitude) {
  if (!r || !freq || !magnitude) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  if (r->rotary_dim < 16 || r->rotary_dim > 256 || r->rotary_dim % 16)
    return record_error(FM_ERR_SHAPE, "rotary_dim must be a multiple of 16 up to 256");
  if (!(r->theta > 1.0) || !std::isfinite(r->theta)) return record_error(FM_ERR_INVALID_ARG, "theta must exceed 1");
  if (r->scaling < FM_ROPE_PLAIN || r->scaling > FM_ROPE_BY_PARTS) return record_error(FM_ERR_INVALID_ARG, "unknown scaling");
  if (r->scaling != FM_ROPE_PLAIN && (!(r->factor >= 1.0) || !std::isfinite(r->factor)))
    return record_error(FM_ERR_INVALID_ARG, "factor must be at least 1");
  const double two_pi = 6.283185307179586476925286766559;
  const int d = r->rotary_dim;
  double theta = r->theta;
  if (r->scaling == FM_ROPE_BASE) theta *= std::pow(r->factor, d / (d - 2.0));
  double lo = 0, hi = 0;
  if (r->scaling == FM_ROPE_BY_PARTS) {
    if (!(r->original_len >= 1.0) || !std::isfinite(r->original_len) || !(r->beta_slow > 0.0) || !(r->beta_fast > r->beta_slow) ||
        !std::isfinite(r->beta_fast))
      return record_error(FM_ERR_INVALID_ARG, "by-parts scaling needs original_len >= 1 and beta_fast > beta_slow > 0");
    const auto where = [&](double turns) { return d * std::log(r->original_len / (turns * two_pi)) / (2 * std::log(theta)); };
    lo = std::max(std::floor(where(r->beta_fast)), 0.0);
    hi = std::min(std::ceil(where(r->beta_slow)), d - 1.0);
  }
  for (int i = 0; i < d / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / d);
    if (r->scaling == FM_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == FM_ROPE_BY_PARTS) {
      const double t = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 0.001)));
      f = f / r->factor * t + f * (1 - t);
    }
    // turns per position, below 0.16; 2^64 of them rounded to whole numbers (a double holds 53 bits of it)
    freq[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);
  }
  *magnitude = r->scaling == FM_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(r->factor) + 1.0) : 1.0f;
  return FM_OK;
}

namespace {

struct HeadNorm {
  const float *q_gamma, *k_gamma;
  float eps;
};

int append(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const fm_rope* rope, const uint16_t* q, int64_t q_stride,
           int H, const uint16_t* k, int64_t k_stride, const uint16_t* v, int64_t v_stride, uint16_t* q_out,
           int64_t q_out_stride, const HeadNorm* norm, const int32_t* positions, void* stream) {
  int st = kv_check(c);
  if (st == FM_OK) st = kv_batch_check(c, b);
  if (st != FM_OK) return st;
  if (!rope) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  if (layer < 0 || layer >= c->layers) return record_error(FM_ERR_INVALID_ARG, "layer out of range");
  if (rope->rotary_dim < 0 || rope->rotary_dim > c->Dh || rope->rotary_dim % 16)
    return record_error(FM_ERR_SHAPE, "rotary_dim must be a multiple of 16 up to Dh");
  if (rope->rotary_dim > 0 && !rope->freq) return record_error(FM_ERR_INVALID_ARG, "the rotary table is NULL");
  if (rope->layout != FM_ROPE_HALF && rope->layout != FM_ROPE_INTERLEAVED)
    return record_error(FM_ERR_INVALID_ARG, "unknown rotary layout");
  if (!std::isfinite(rope->magnitude)) return record_error(FM_ERR_INVALID_ARG, "magnitude must be finite");
  if (H < 0 || H > 65535) return record_error(FM_ERR_SHAPE, "H must be 0 to 65535");
  if (norm && (!(norm->eps >= 0.f) || !std::isfinite(norm->eps))) return record_error(FM_ERR_INVALID_ARG, "eps must not be negative");
  if (b->n == 0 || b->tokens == 0 || b->max_tokens == 0) return FM_OK;
  if (!k || !v || (H > 0 && (!q || !q_out))) return record_error(FM_ERR_INVALID_ARG, "NULL argument");
  const int64_t kv_row = static_cast<int64_t>(c->Hkv) * c->Dh, q_row = static_cast<int64_t>(H) * c->Dh;
  if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 || v_stride % 8 ||
      (H > 0 && (q_stride < q_row || q_out_stride < q_row || q_stride % 8 || q_out_stride % 8)))
    return record_error(FM_ERR_SHAPE, "token strides must be multiples of 8 elements and hold the token's heads");
  if (H > 0 && q == q_out && q_stride != q_out_stride && b->tokens > 1)
    return record_error(FM_ERR_SHAPE, "q_out in the place of q needs q's stride");
  for (const void* x : {static_cast<const void*>(k), static_cast<const void*>(v), static_cast<const void*>(q),
                        static_cast<const void*>(q_out)})
    if (reinterpret_cast<uintptr_t>(x) % 16) return record_error(FM_ERR_ALIGN, "q, k, v and q_out must be 16-byte aligned");
  if (norm && (reinterpret_cast<uintptr_t>(norm->q_gamma) % 4 || reinterpret_cast<uintptr_t>(norm->k_gamma) % 4))
    return record_error(FM_ERR_ALIGN, "q_gamma and k_gamma must be 4-byte aligned");
  int* err = standalone_error_word();
  if (!err) return record_error(FM_ERR_CUDA, "no error word on the current device");
  const fm_kv_batch bounded = bounded_batch(*b);
  b = &bounded;
  const bool f8 = c->fmt == FM_FMT_FP8;
  const int eb = f8 ? 1 : 2;
  AppendParams p = {};
  p.q = reinterpret_cast<const __nv_bfloat16*>(q);
  p.k = reinterpret_cast<const __nv_bfloat16*>(k);
  p.v = reinterpret_cast<const __nv_bfloat16*>(v);
  p.q_out = reinterpret_cast<__nv_bfloat16*>(q_out);
  p.qs = q_stride, p.ks = k_stride, p.vs = v_stride, p.os = q_out_stride;
  p.start = b->start, p.seq = b->seq, p.lens = c->lens, p.table = c->table, p.positions = positions;
  p.freq = rope->freq;
  p.mag = rope->magnitude;
  p.rot = rope->rotary_dim;
  p.interleaved = rope->layout == FM_ROPE_INTERLEAVED;
  p.tokens = b->tokens, p.max_tokens = b->max_tokens, p.seqs = c->seqs, p.table_stride = c->table_stride;
  p.pages = c->pages, p.page = c->page_tokens, p.shift = shift_of(c->page_tokens);
  p.H = H, p.Hkv = c->Hkv, p.Dh = c->Dh;
  p.kc = static_cast<uint8_t*>(c->k) + layer * c->layer_stride * eb;
  p.vc = static_cast<uint8_t*>(c->v) + layer * c->layer_stride * eb;
  p.pg = c->page_stride, p.tok = c->token_stride, p.head = c->head_stride;
  p.k_scale = f8 ? c->k_scale + layer : nullptr;
  p.v_scale = f8 ? c->v_scale + layer : nullptr;
  p.err = err;
  // A token has Dh / 16 threads a head group. As many tokens a CTA as leave two groups and three CTAs an SM (9000 tokens,
  // 24 heads of 128: 19.8 us with 16, 23.8 us with 4); a few tokens are spread over all threads of their CTAs.
  int lanes = c->Dh / 16;
  if (norm) {
    p.q_gamma = norm->q_gamma, p.k_gamma = norm->k_gamma, p.eps = norm->eps;
    lanes = lanes <= 4 ? 4 : lanes <= 8 ? 8 : 16;   // Dh is 256 at most
  }
  p.toks = 1;
  while (lanes * p.toks * 2 <= 128 && p.toks < b->max_tokens && b->tokens / (2 * p.toks) >= 152 * 3) p.toks *= 2;
  p.groups = 256 / (lanes * p.toks);
  const int blocks = (b->max_tokens - 1) / p.toks + 1;
  void (*kernel)(AppendParams) = !norm        ? (f8 ? append_kernel<true, 0> : append_kernel<false, 0>)
                                 : lanes == 4 ? (f8 ? append_kernel<true, 4> : append_kernel<false, 4>)
                                 : lanes == 8 ? (f8 ? append_kernel<true, 8> : append_kernel<false, 8>)
                                              : (f8 ? append_kernel<true, 16> : append_kernel<false, 16>);
  return done(launch(kernel, dim3(static_cast<unsigned>(blocks), b->n), dim3(256),
                     sizeof(float2) * p.toks * (p.rot / 2) + (norm ? sizeof(float) * 2 * c->Dh : 0), opts(stream), p));
}

}  // namespace

extern "C" int fm_rope_append(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const fm_rope* rope, const uint16_t* q,
                              int64_t q_stride, int H, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                              int64_t v_stride, uint16_t* q_out, int64_t q_out_stride, const int32_t* positions,
                              void* stream) {
  return append(c, layer, b, rope, q, q_stride, H, k, k_stride, v, v_stride, q_out, q_out_stride, nullptr, positions, stream);
}

extern "C" int fm_norm_rope_append(const fm_kv_cache* c, int layer, const fm_kv_batch* b, const fm_rope* rope,
                                   const uint16_t* q, int64_t q_stride, int H, const uint16_t* k, int64_t k_stride,
                                   const uint16_t* v, int64_t v_stride, uint16_t* q_out, int64_t q_out_stride,
                                   const float* q_gamma, const float* k_gamma, float eps, const int32_t* positions,
                                   void* stream) {
  const HeadNorm norm{q_gamma, k_gamma, eps};
  return append(c, layer, b, rope, q, q_stride, H, k, k_stride, v, v_stride, q_out, q_out_stride, &norm, positions, stream);
}
