// A row of bf16 as a buffer of its own: what is read behind its end is 0, and what is written there is
// dropped (a row that is not there is a buffer of no bytes).  So no load or store of a row stands under a
// condition: behind one that may or may not have been issued, the compiler waits for all in flight, the
// loads for rows to come among them.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../csrc/device_common.hpp"

namespace lora {

struct RowBuffer {
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t r;
#endif
  // `width` values from row t on; all arguments are the same in all lanes of a wave
  __device__ __forceinline__ RowBuffer(const uint16_t* base, long ld, int t, int width, bool there) {
#if defined(__HIP_DEVICE_COMPILE__)
    r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base) + (there ? t * ld : 0), 0, there ? 2 * width : 0, 0x00020000);
#endif
  }
  __device__ __forceinline__ uint4 load(int at) const {
#if defined(__HIP_DEVICE_COMPILE__)
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, 2 * at, 0, 0));
#else
    return zero4();
#endif
  }
  __device__ __forceinline__ void store(int at, const uint4& v) const {
#if defined(__HIP_DEVICE_COMPILE__)
    typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, 2 * at, 0, 0);
#endif
  }
};

}  // namespace lora
