// Attention of many rows over a paged f16 pool: its kernels.
#include "rows_attend.cuh"

namespace kvsel {

RowsVariant rows_variant_f16(int d, bool split, bool scored) {
  return d == 64 ? rows_variant<64, kF16>(split, scored) : rows_variant<128, kF16>(split, scored);
}

}  // namespace kvsel
