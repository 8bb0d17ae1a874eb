// The paged attention kernels over bf16 pools.
#include "paged_attend.cuh"

namespace kvsel {

PagedVariant paged_variant_bf16(int d, int nt) {
  return d == 64 ? paged_variant<64, kBf16>(nt) : paged_variant<128, kBf16>(nt);
}

}  // namespace kvsel
