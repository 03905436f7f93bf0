// scan_bwd_f32.cu -- the selective scan's gradients for fp32 tensors (kernels in scan_bwd.cuh).
#include "scan_bwd.cuh"

namespace m2 {

cudaError_t scan_bwd_f32(const ScanArgs& a, const scan_bwd::BwdP& p, int KK, const float* init,
                         const float* dfinal, cudaStream_t st) {
    return scan_bwd::run_type<float>(a, p, KK, init, dfinal, st);
}

}  // namespace m2
