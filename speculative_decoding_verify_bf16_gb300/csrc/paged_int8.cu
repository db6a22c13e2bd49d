// paged_int8.cu -- attention over a paged cache of int8 numbers.
#include "paged_variants.cuh"

namespace specv {
PagedVariant paged_rows_int8(int dim, int64_t rows) { return paged_variant<SPEC_CACHE_INT8>(dim, rows); }
}  // namespace specv
