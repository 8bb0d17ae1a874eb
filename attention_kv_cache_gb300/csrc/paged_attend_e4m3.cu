// The paged attention kernels over 8-bit pools.
#include "paged_attend.cuh"

namespace kvsel {

PagedVariant paged_variant_e4m3(int d, int nt) {
  return d == 64 ? paged_variant<64, kE4m3>(nt) : paged_variant<128, kE4m3>(nt);
}

}  // namespace kvsel
