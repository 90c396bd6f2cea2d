// shared_append.cu -- new rows of a shared-latent cache written into the page pool through a
// slot map, for sm_100a:  pool[slot_i] = [c_i (r values) | k^R_i (dr values)].
//
// A copy, bound by memory: 2 * (r + dr) bytes read and written a row.  Threads take 16-byte
// pieces; a row's pieces are neighbours, so both sides move whole lines.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"

namespace stief {

__global__ void __launch_bounds__(256) stief_shared_append_kernel(const SharedAppendArgs a) {
  const int w8 = (a.r + a.dr) / 8, r8 = a.r / 8;
  const long long total = (long long)a.N * w8, step = (long long)gridDim.x * blockDim.x;
  pdl_wait();
  pdl_launch_dependents();
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
    const int row = (int)(i / w8), c = (int)(i - (long long)row * w8);
    const int slot = __ldg(a.slots + row);
    if (slot < 0) continue;
    if (slot >= a.num_slots) {
      if (c == 0) report(a.dev_status, STIEF_DEV_CAPACITY_OVERFLOW);
      continue;
    }
    const uint16_t* src = c < r8 ? a.c + row * a.ld_c + c * 8 : a.pe + row * a.ld_pe + (c - r8) * 8;
    reinterpret_cast<uint4*>(a.pages)[(long long)slot * w8 + c] = __ldg(reinterpret_cast<const uint4*>(src));
  }
}

cudaError_t launch_shared_append(const SharedAppendArgs& a, int sms, cudaStream_t stream) {
  const long long pieces = (long long)a.N * ((a.r + a.dr) / 8);
  long long grid = (pieces + 255) / 256;
  if (grid > 8LL * sms) grid = 8LL * sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, stief_shared_append_kernel, a);
}

}  // namespace stief
