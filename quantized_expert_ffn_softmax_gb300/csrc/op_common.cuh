// What the stand-alone operators (norm.cu, linear.cu) share: argument checks
// of their entry points, launches that overlap the preceding kernel's tail,
// and bf16 helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "moe_internal.cuh"

namespace moe {
namespace op {

inline moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

inline moe_status cuda_fail(cudaError_t e, const char* what) {
  cudaGetLastError();
  return fail(e == cudaErrorMemoryAllocation ? MOE_ERR_OOM : MOE_ERR_CUDA, "%s: %s", what,
              cudaGetErrorString(e));
}

// A buffer argument of an entry point: [base, base + bytes).
struct Buf {
  const char* name;
  const void* p;
  size_t bytes;
  size_t align;
};

// b is device memory of device `dev` (or managed memory), aligned.
inline moe_status check_buf(const Buf& b, int dev) {
  if (!b.p) return fail(MOE_ERR_INVALID, "%s is NULL", b.name);
  if (reinterpret_cast<uintptr_t>(b.p) & (b.align - 1))
    return fail(MOE_ERR_INVALID, "%s is not %zu-byte aligned", b.name, b.align);
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, b.p) != cudaSuccess) {
    cudaGetLastError();
    return fail(MOE_ERR_INVALID, "%s is not device memory", b.name);
  }
  if (a.type == cudaMemoryTypeManaged) return MOE_OK;
  if (a.type != cudaMemoryTypeDevice || a.device != dev)
    return fail(MOE_ERR_INVALID, "%s is not memory of the current device", b.name);
  return MOE_OK;
}

inline bool overlap(const Buf& a, const Buf& b) {
  const char* x = static_cast<const char*>(a.p);
  const char* y = static_cast<const char*>(b.p);
  return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}

// Launch whose grid may become resident while the preceding kernel of the
// stream drains; the kernel itself orders its accesses with dep_wait().
template <typename... KA, typename... A>
cudaError_t launch_overlapped(void (*kernel)(KA...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, KA(args)...);
}

// Every thread of an overlapped kernel calls dep_wait() before its first
// access to memory that another kernel may have written or may still read,
// and, but for kernels that say why not, only then lets the next kernel in with
// dep_release(): a kernel that is let in therefore starts after everything
// before the current one is done, so no line of a reused buffer can sit in an
// L1 from an older reader.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A float that the kernel before may have written while this one was already
// resident: never through the read-only path, which takes it to be constant
// over the kernel's lifetime.
__device__ __forceinline__ float ld_f32(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// The same, past L1.
__device__ __forceinline__ float ld_l2_f32(const float* p) {
  float v;
  asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}

// The two bf16 values of a word as floats, and back (round to nearest even).
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace op
}  // namespace moe
