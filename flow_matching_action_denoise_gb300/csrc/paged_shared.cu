// Attention of forks over a paged cache (fm_shared_attention), two kernels in a row:
//
//   the prefix: the tokens of a group's entries stacked into the rows of paged_tile.cuh's kernel, once over the keys that they
//   share: shares (m1, l1, o1) of every token and split of the prefix, to the workspace;
//   the own keys: paged_decode.cuh's kernel, up to 16 rows of an entry a CTA, over what the entry has behind its prefix, and the join
//   m = max(m1, m2), l = l1 e^(m1 - m) + l2 e^(m2 - m), o = (o1 e^(m1 - m) + o2 e^(m2 - m)) / l.
//
// An entry's keys and values meet its own rows only: with the own keys of many entries in one tile of stacked rows a NaN in
// one robot's values would reach all of them (0 x NaN). The second kernel starts once every CTA of the first is resident and
// works beside it on what SMs are free, on inputs that the first one hands on (see_inputs); it waits for the first before the join.
// 128 single tokens of 16 heads on 2 KV heads (Dh 128, bf16) behind 8192 common keys, 133 to 400 of their own: 25.8 us, 66 us as
// separate sequences. Bound by the chain: 18 us of prefix (7 us of them a CTA's ends), beside which the own CTAs have to find
// room (those that do not cost 8 us more, behind it), 3.5 us from the last share to the output.

#include "paged_decode.cuh"
#include "paged_tile.cuh"

namespace fm {

template cudaError_t tile_launch<Keys::kPrefix>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&, dim3,
                                                size_t, const LaunchOpts&);
template cudaError_t tile_configure<Keys::kPrefix>();
template cudaError_t decode_launch<Keys::kOwn>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&,
                                               const LaunchOpts&);
template cudaError_t decode_configure<Keys::kOwn>();

int own_resident(int Dh, bool f8, int rows) {
  return decode_resident(Dh, f8, rows) + (Dh == 128 && !f8 && rows <= 8 ? kMore<128, false, 1, Keys::kOwn> : 0);
}

}  // namespace fm
