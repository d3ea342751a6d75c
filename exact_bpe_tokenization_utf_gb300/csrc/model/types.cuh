// The element types of the model's arrays (TOK_F32, TOK_F16, TOK_BF16), eight
// elements at a time, and checks that their entry points share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../tok_handle.cuh"

namespace tokgb {

inline size_t element_size(int dtype) { return dtype == TOK_F32 ? 4 : dtype == TOK_F16 || dtype == TOK_BF16 ? 2 : 0; }

// addresses come without a type: one that no element can have would fault on the device
inline bool lies_at(const void* p, size_t multiple) { return reinterpret_cast<uintptr_t>(p) % multiple == 0; }

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight elements that lie at a 16-byte boundary, as they are in memory.
template <class T> struct Eight {
  static constexpr int WORDS = sizeof(T) * 2;
  uint32_t w[WORDS];
  __device__ __forceinline__ void load(const T* p) {   // what the kernel writes, too
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void load_once(const T* p) {  // what nobody reads again
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < WORDS / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  __device__ __forceinline__ float get(int i) const;
  __device__ __forceinline__ void put_pair(int i, float a, float b);  // elements 2 i and 2 i + 1
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0;
  }
};
template <> __device__ __forceinline__ float Eight<float>::get(int i) const { return __uint_as_float(w[i]); }
template <> __device__ __forceinline__ float Eight<__half>::get(int i) const {
  const __half2 h = *reinterpret_cast<const __half2*>(&w[i >> 1]);
  return i & 1 ? __high2float(h) : __low2float(h);
}
template <> __device__ __forceinline__ float Eight<__nv_bfloat16>::get(int i) const {
  return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}
template <> __device__ __forceinline__ void Eight<float>::put_pair(int i, float a, float b) {
  w[2 * i] = __float_as_uint(a);
  w[2 * i + 1] = __float_as_uint(b);
}
template <> __device__ __forceinline__ void Eight<__half>::put_pair(int i, float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  w[i] = *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ void Eight<__nv_bfloat16>::put_pair(int i, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  w[i] = *reinterpret_cast<const uint32_t*>(&h);
}

// A kernel that launch_behind launched starts while the one before it in the stream
// ends, if that one lets it, and waits here until its results are there.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <class... Args>
cudaError_t launch_behind(void (*kernel)(Args...), unsigned ctas, unsigned threads, size_t smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// count of a batch of at most n whose number the device knows (p may be nullptr)
__device__ __forceinline__ uint32_t count_of(const long long* p, uint32_t n) {
  if (!p) return n;
  const long long m = *p;
  return m <= 0 ? 0u : m < (long long)n ? (uint32_t)m : n;
}

}  // namespace tokgb
