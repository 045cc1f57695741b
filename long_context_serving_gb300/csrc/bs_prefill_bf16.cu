// New prompt tokens over bf16 caches.
#include "bs_rows_mma.cuh"

namespace bsi {

template <>
bs_status launch_rows_bf16<false>(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int rows, cudaStream_t cs) {
  return dispatch_rows<0, false>(a, p, maps, rows, cs);
}

}  // namespace bsi
