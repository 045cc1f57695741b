// New prompt tokens over 8-bit caches.
#include "bs_rows_mma.cuh"

namespace bsi {

template <>
bs_status launch_rows_quant<false>(const RowsArgs &a, const RowsPlan &p, const RowsMaps &maps, int rows, cudaStream_t cs) {
  return a.dims.kv_dtype == BS_INT8 ? dispatch_rows<2, false>(a, p, maps, rows, cs)
                                    : dispatch_rows<1, false>(a, p, maps, rows, cs);
}

}  // namespace bsi
