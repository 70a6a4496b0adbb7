// Single-token attention over a paged cache, all keys that the mask leaves (the kernel: paged_decode.cuh).

#include "paged_decode.cuh"

namespace fm {

template cudaError_t decode_launch<Keys::kAll>(const AttnParams&, int, bool, const CUtensorMap&, const CUtensorMap&,
                                               const LaunchOpts&);
template cudaError_t decode_configure<Keys::kAll>();

int decode_resident(int Dh, bool f8, int rows) {
  if (Dh == 128) return rows <= 8 ? (f8 ? kResident<128, true, 1> : kResident<128, false, 1>)
                                  : (f8 ? kResident<128, true, 2> : kResident<128, false, 2>);
  return rows <= 8 ? (f8 ? kResident<64, true, 1> : kResident<64, false, 1>)
                   : (f8 ? kResident<64, true, 2> : kResident<64, false, 2>);
}

}  // namespace fm
