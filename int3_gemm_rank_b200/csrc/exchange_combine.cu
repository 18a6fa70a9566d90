// exchange_combine.cu -- milo_combine's kernels (and milo_dispatch_backward's without weights): see exchange_rows.cuh.
#include "exchange_rows.cuh"

namespace milo {

cudaError_t launch_combine_rows(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s) {
    return run_rows_types<kXCombine>(p, t, s);
}

}  // namespace milo
