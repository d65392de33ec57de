// Status texts and the per-thread launch status of the operators of include/block_ops.h.
#include "host_checks.h"

namespace {
thread_local int g_last_cuda_error = 0;
}

namespace block_ops {
fn_status launch_status(int cuda_error) {
  if (cuda_error == 0) return FN_OK;
  g_last_cuda_error = cuda_error;
  return FN_ERR_CUDA;
}

fn_status wait_status(int* gave_up) {
  if (!__atomic_load_n(gave_up, __ATOMIC_RELAXED) || !__atomic_exchange_n(gave_up, 0, __ATOMIC_ACQ_REL)) return FN_OK;
  return launch_status(cudaErrorLaunchTimeout);
}
}  // namespace block_ops

extern "C" {

const char* block_ops_status_string(fn_status s) {
  switch (s) {
    case FN_OK: return "ok";
    case FN_ERR_INVALID_ARG: return "invalid argument";
    case FN_ERR_UNSUPPORTED: return "unsupported configuration (sizes outside the operator's range)";
    case FN_ERR_MISALIGNED: return "misaligned pointer or stride (16-byte rows required)";
    case FN_ERR_CUDA: return "CUDA launch error";
  }
  return "unknown status";
}

int block_ops_last_cuda_error(void) { return g_last_cuda_error; }

}  // extern "C"
