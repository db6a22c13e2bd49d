// paged_int8.cu -- attention over a paged cache of int8 numbers.
#include "paged_variants.cuh"

namespace specv {
PagedVariant paged_int8(int dim, int64_t rows, bool tiles, bool few) { return paged_variant<SPEC_CACHE_INT8>(dim, rows, tiles, few); }
}  // namespace specv
