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

int decode_clusters(int Dh, bool f8, int rows, int size) {
  const auto query = [size](auto kernel, size_t smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n : 0;
  };
  if (decode_configure<Keys::kAll>() != cudaSuccess) return 0;
  constexpr Keys K = Keys::kAll;
  const auto of = [&](auto dh, auto f, auto nt) {
    constexpr int DH = decltype(dh)::value, NT = decltype(nt)::value;
    constexpr bool F8 = decltype(f)::value;
    return query(decode_kernel<DH, F8, NT, K>, smem_bytes<DH, F8, NT, K>(true));
  };
  const auto of_rows = [&](auto dh, auto f) {
    return rows <= 8 ? of(dh, f, std::integral_constant<int, 1>{}) : of(dh, f, std::integral_constant<int, 2>{});
  };
  const auto of_type = [&](auto dh) { return f8 ? of_rows(dh, std::true_type{}) : of_rows(dh, std::false_type{}); };
  return Dh == 128 ? of_type(std::integral_constant<int, 128>{}) : of_type(std::integral_constant<int, 64>{});
}

}  // namespace fm
