// exchange_dispatch_grad.cu -- milo_dispatch_backward's kernels with weights: see exchange_rows.cuh.
#include "exchange_rows.cuh"

namespace milo {

cudaError_t launch_dispatch_grad(const ExchangeParams& p, const ExchangeTypes& t, cudaStream_t s) {
    return run_rows_types<kXDispatchGrad>(p, t, s);
}

}  // namespace milo
