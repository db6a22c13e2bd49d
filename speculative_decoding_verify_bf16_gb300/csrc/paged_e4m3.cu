// paged_e4m3.cu -- attention over a paged cache of e4m3 numbers.
#include "paged_variants.cuh"

namespace specv {
PagedVariant paged_e4m3(int dim, int64_t rows, bool tiles, bool few) { return paged_variant<SPEC_CACHE_E4M3>(dim, rows, tiles, few); }
}  // namespace specv
