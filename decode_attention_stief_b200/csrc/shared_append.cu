// shared_append.cu -- new rows of a shared-latent cache written into the page pool through a
// slot map, for sm_100a:  pool[slot_i] = [c_i (r values) | k^R_i (dr values)].
//
// A copy, bound by memory: 2 * (r + dr) bytes read and written a row, each once.  A thread moves
// kPieces 16-byte pieces, all loads in flight before the first store; neighbouring threads take
// neighbouring pieces, so both sides move whole lines.  32768 rows of 576 values: 13.8 us, 5.5 TB/s, 0.79
// of a plain copy's rate; 64 rows: 1.6 us on the GPU.
#include <cstdint>

#include "shared_latent.h"
#include "stief_device.cuh"

namespace stief {

namespace {
constexpr int kThreads = 256;
}

template <int kPieces>
__global__ void __launch_bounds__(kThreads) stief_shared_append_kernel(const SharedAppendArgs a) {
  const unsigned w8 = (unsigned)(a.r + a.dr) / 8, r8 = (unsigned)a.r / 8;
  const long long total = (long long)a.N * w8;
  const long long first = (long long)blockIdx.x * (kThreads * kPieces) + threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  int row[kPieces], slot[kPieces];
  unsigned c[kPieces];
  uint4 x[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    const long long i = first + (long long)k * kThreads;
    slot[k] = -1;
    if (i < total) {
      row[k] = total <= 0xffffffffLL ? (int)((unsigned)i / w8) : (int)(i / w8);
      c[k] = (unsigned)(i - (long long)row[k] * w8);
      slot[k] = __ldg(a.slots + row[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    if (slot[k] >= 0) {  // (a skipped row is not read)
      const uint16_t* src = c[k] < r8 ? a.c + row[k] * a.ld_c + c[k] * 8 : a.pe + row[k] * a.ld_pe + (c[k] - r8) * 8;
      x[k] = __ldcs(reinterpret_cast<const uint4*>(src));
    }
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    if (slot[k] >= 0) {
      if (slot[k] < a.num_slots)
        reinterpret_cast<uint4*>(a.pages)[(long long)slot[k] * w8 + c[k]] = x[k];
      else if (c[k] == 0)
        report(a.dev_status, STIEF_DEV_CAPACITY_OVERFLOW);
    }
}

cudaError_t launch_shared_append(const SharedAppendArgs& a, int sms, cudaStream_t stream) {
  const long long pieces = (long long)a.N * ((a.r + a.dr) / 8);
  // Few rows: as many threads as pieces (latency); many: four pieces a thread.
  const bool many = pieces > 8LL * kThreads * sms;
  const long long per = kThreads * (many ? 4 : 1), grid = (pieces + per - 1) / per;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = many ? cudaLaunchKernelEx(&cfg, stief_shared_append_kernel<4>, a)
                             : cudaLaunchKernelEx(&cfg, stief_shared_append_kernel<1>, a);
  // (a pool without position values may be the per-head pool of one KV head: a paged decode that follows
  // must not request its rows before this kernel has written them)
  if (e == cudaSuccess) mark_stream_compress(a.device, stream, true);
  return e;
}

}  // namespace stief
