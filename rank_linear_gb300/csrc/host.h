// host.h -- host-side helpers shared by the files that implement the C ABI:
// error text, the device record, argument checks, launch accounting and the
// driver's tensor-map encoder.  Defined in lora_api.cu.
#pragma once

#include <cudaTypedefs.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "internal.h"
#include "lora_linear.h"

namespace lora {

struct DevInfo {
  bool init = false;
  int sms = 0, major = 0, minor = 0;
  unsigned *status = nullptr;  // the device status word
};

// Empties the calling thread's error text (first thing in an entry point).
void clear_error();
// Sets the calling thread's error text and returns st.
lora_status_t fail(lora_status_t st, const char *fmt, ...);
// The current device, which has to be one this library is built for.
lora_status_t device_info(DevInfo &out);
lora_status_t check_ptr(const void *p, const char *name, bool may_be_null = false);
lora_status_t check_ws(const void *ws, size_t have, size_t need);
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// The timing hook's events around a launch, and the launch count.  Returns
// the slot to hand to timing_after (-1: no hook).
lora_status_t timing_before(lora_kernel_kind_t kind, cudaStream_t s, const char *what, int *slot);
lora_status_t timing_after(int slot, cudaStream_t s, const char *what);

template <class F>
lora_status_t run(lora_kernel_kind_t kind, cudaStream_t s, const char *what, F &&launch) {
  int slot = -1;
  lora_status_t st = timing_before(kind, s, what, &slot);
  if (st != LORA_OK) return st;
  const cudaError_t e = launch();
  if (e != cudaSuccess) return fail(LORA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return timing_after(slot, s, what);
}

// out[row] = scale[row] * mul[0] (simt.cu): scales of rows that came quantised.
cudaError_t launch_scale_rows(const float *scale, const float *mul, int64_t rows, float *out,
                              cudaStream_t s);

inline int64_t rup(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline uint8_t *at(void *base, size_t off) { return static_cast<uint8_t *>(base) + off; }

// Launches a kernel with the programmatic-overlap attribute: the kernel has
// to begin with griddep_wait().
template <class... P, class... A>
cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       A &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Lets a kernel take `smem` bytes of dynamic shared memory on the current
// device; `done` keeps the devices that it has been said for.
template <class F>
cudaError_t allow_smem(F *kernel, size_t smem, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> (dev & 63) & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem));
  if (e == cudaSuccess) done.fetch_or(uint64_t(1) << (dev & 63), std::memory_order_relaxed);
  return e;
}

#define LORA_TRY(expr)                     \
  do {                                     \
    const lora_status_t st_ = (expr);      \
    if (st_ != LORA_OK) return st_;        \
  } while (0)

}  // namespace lora
