// paged_bf16.cu -- attention over a paged cache of bf16 numbers.
#include "paged_variants.cuh"

namespace specv {
PagedVariant paged_bf16(int dim, int64_t rows, bool tiles, bool few) { return paged_variant<SPEC_CACHE_BF16>(dim, rows, tiles, few); }
}  // namespace specv
