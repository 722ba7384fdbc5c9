// host.h -- host-side services of the library that its entry points in several source files share:
// argument checks, the device and stream of a call, the status word, tensor-map encoding.  Defined in
// packattn.cu (nothing here is exported from the library).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

struct pa_rope_axes_desc;

namespace pa {
namespace host {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// PA_OK with `*dev` set when every non-null pointer is memory of one GPU, else PA_ERR_NOT_DEVICE.
int common_device(std::initializer_list<const void*> ptrs, int* dev);

// One enqueueing call: holds the library's lock, makes the buffers' device current (the thread's own one is
// put back at the end) and finds the status word of (device, stream).  rc is not PA_OK when that failed.
class Call {
 public:
  Call(int dev, void* stream);
  ~Call();
  Call(const Call&) = delete;
  Call& operator=(const Call&) = delete;

  int rc;
  int sms = 0;
  cudaStream_t stream;
  int32_t* status = nullptr;
  uint64_t wait_limit_ns = 0;

 private:
  int prev_dev_ = -1;
};

// Tensor map of a bf16 [rows, heads * head_dim] matrix, box 64 columns x 128 rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* base, int32_t rows, int32_t heads, int32_t head_dim);

// Positions with several axes (rope_axes.cu): PA_OK or why a description is refused; the pairs of a head that belong
// to an axis; the (cos, sin) of every token and pair into `table`.
int check_rope_axes(const pa_rope_axes_desc* rope, int32_t head_dim);
int rope_turned(const pa_rope_axes_desc* rope);
int launch_rope_table(const float* pos, int32_t total, int32_t head_dim, const pa_rope_axes_desc* rope, void* table,
                      cudaStream_t stream);

inline int launch_status() { return cudaGetLastError() == cudaSuccess ? 0 : -8; }

// Launches a kernel that begins with griddepcontrol.wait as a programmatic dependent of the one before it in the
// stream: its blocks are placed, and what it does before that wait is done, while that one's last blocks run.
template <class P>
int launch_behind(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, params) == cudaSuccess ? launch_status() : -8;
}

}  // namespace host
}  // namespace pa
