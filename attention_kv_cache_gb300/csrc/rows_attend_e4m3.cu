// Attention of many rows over a paged e4m3 pool: its kernels.
#include "rows_attend.cuh"

namespace kvsel {

RowsVariant rows_variant_e4m3(int d, bool split, bool scored) {
  return d == 64 ? rows_variant<64, kE4m3>(split, scored) : rows_variant<128, kE4m3>(split, scored);
}

}  // namespace kvsel
