// Attention of many rows over a paged bf16 pool: its kernels.
#include "rows_attend.cuh"

namespace kvsel {

RowsVariant rows_variant_bf16(int d, bool split, bool scored) {
  return d == 64 ? rows_variant<64, kBf16>(split, scored) : rows_variant<128, kBf16>(split, scored);
}

}  // namespace kvsel
