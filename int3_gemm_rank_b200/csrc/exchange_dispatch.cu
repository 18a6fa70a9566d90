// exchange_dispatch.cu -- milo_dispatch's kernels for rows that do not start on
// 16-byte boundaries: see exchange_rows.cuh.
#include "exchange_rows.cuh"

namespace milo {

cudaError_t launch_dispatch_rows(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s) {
    return run_rows_types<kXDispatch>(p, t, s);
}

}  // namespace milo
