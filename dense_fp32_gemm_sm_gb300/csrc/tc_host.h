// tc_host.h -- host-side facts that the tensor-core units share: the driver's tensor-map
// encoder, the device error word of the bounded waits, and the testing hook's settings.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace fgemm {

// cuTensorMapEncodeTiled, or null when the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tc_encode_fn();
// Device address, in the current context, of the word that a kernel whose bounded wait ran
// out sets bits in (fgemm_device_status reads it); null on failure.
unsigned *tc_error_word();
// fgemm_debug_withhold_tensor_core: the k-block that producers withhold (-1: none), and the
// limit of every wait.
int tc_withheld_k_block();
unsigned long long tc_wait_limit_ns();

}  // namespace fgemm
