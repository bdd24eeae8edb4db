// What the translation units of the paged K/V cache share.
#pragma once
#include <atomic>

#include "fm_internal.h"

namespace fm {

constexpr int kMaxTokenIndex = 1 << 30;   // tokens of a row (32-bit positions)
constexpr int kMaxPoolPages = (1 << 23) - 1;
constexpr int kMaxHeads = 65535;

// Sizes of `c` that every cache entry point needs; `pools`: its pools' too.
fm_status check_cache(const fm_cache* c, bool pools);
// The same of a cache of e4m3 codes, and its pools and scales.
fm_status check_cache8(const fm_cache* c, const void* k_pool, const void* v_pool, const void* k_scale,
                       const void* v_scale);

__device__ __forceinline__ void flag(int* status, int bit) {
  if (status) atomicOr(status, bit);
}

// Context length of packed sequence b (tokens before its new ones), or -1 if
// its lens or cu entries are out of range; n: its new tokens.
__device__ __forceinline__ int context_of(const int32_t* lens, const int32_t* cu, int b, int total,
                                          int max_tokens, int& n) {
  const int c0 = cu[b], c1 = cu[b + 1], len = lens[b];
  n = c1 - c0;
  if (c0 < 0 || c1 < c0 || c1 > total || len > max_tokens || len < n) return -1;
  return len - n;
}

inline fm_status done(cudaError_t e) { return e == cudaSuccess ? FM_OK : FM_ERR_CUDA; }

inline int page_shift(int page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
}

inline bool aligned_to(const void* p, uintptr_t n) {
  return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

// [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const char* x = static_cast<const char*>(a);
  const char* y = static_cast<const char*>(b);
  return x < y + nb && y < x + na;
}

// Sets a kernel's shared memory on the current device at its first launch
// there (two runtime calls, some 1.5 us, that every later launch is spared);
// min_regs: registers per thread that it must have been compiled with.
template <typename K>
inline fm_status prepare_kernel(K* kern, int smem, int min_regs, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FM_ERR_CUDA;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return FM_OK;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return FM_ERR_CUDA;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return FM_ERR_CUDA;
  if (fa.numRegs < min_regs) return FM_ERR_UNSUPPORTED;
  done.fetch_or(bit, std::memory_order_release);
  return FM_OK;
}

// Division by a number that the host knows, of values below 2^31: one high
// product, one add and one shift in place of some forty instructions.
struct FastDiv {
  uint32_t d, mul, shift;
  static FastDiv of(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = static_cast<uint32_t>(((1ull << f.shift) - d) * (1ull << 32) / d + 1);
    return f;
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};

// A launch that may start while the kernel before it in the stream still
// runs (it calls grid_dependency_wait() before it touches memory).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                                    cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace fm
