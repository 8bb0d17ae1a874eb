// Attention of many rows over a paged e4m3 pool: its kernels.
#include "rows_attend.cuh"

namespace kvsel {

RowsVariant rows_variant_e4m3(int d, bool split) { return d == 64 ? rows_variant<64, kE4m3>(split) : rows_variant<128, kE4m3>(split); }

}  // namespace kvsel
