// scan_packed.hip -- instantiations of the packed scan (scan_packed.hpp).
#include <hip/hip_runtime.h>

#include "scan_packed.hpp"

namespace ssm {

namespace {
template <bool BF16, int N>
const ScanPackedKernels* kernels() {
  static const ScanPackedKernels k = {scan_packed_kernel<BF16, N, false>, scan_packed_kernel<BF16, N, true>};
  return &k;
}

template <bool BF16>
const ScanPackedKernels* find(int64_t dstate) {
  switch (dstate) {
    case 1: return kernels<BF16, 1>();
    case 2: return kernels<BF16, 2>();
    case 4: return kernels<BF16, 4>();
    case 8: return kernels<BF16, 8>();
    case 16: return kernels<BF16, 16>();
    case 32: return kernels<BF16, 32>();
    case 64: return kernels<BF16, 64>();
    default: return nullptr;
  }
}
}  // namespace

const ScanPackedKernels* scan_packed_kernels(bool bf16, int64_t dstate) {
  return bf16 ? find<true>(dstate) : find<false>(dstate);
}

}  // namespace ssm
