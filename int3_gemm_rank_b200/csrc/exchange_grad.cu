// exchange_grad.cu -- milo_combine_backward's kernels: see exchange_rows.cuh.
#include "exchange_rows.cuh"

namespace milo {

cudaError_t launch_combine_grad(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s) {
    return run_rows_types<kXCombineGrad>(p, t, s);
}

}  // namespace milo
