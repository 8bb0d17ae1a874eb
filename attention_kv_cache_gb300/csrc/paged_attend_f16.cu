// The paged attention kernels over fp16 pools.
#include "paged_attend.cuh"

namespace kvsel {

PagedVariant paged_variant_f16(int d, int nt) {
  return d == 64 ? paged_variant<64, kF16>(nt) : paged_variant<128, kF16>(nt);
}

}  // namespace kvsel
