// Dropout with a mask that is never stored (rib_dropout):
//   y[i] = bits16(i) >= threshold ? x[i] / keep : 0
// with the random bits of philox.cuh. The backward is the same call on the
// upstream gradient.
//
// What bounds it: memory, 2 * n * size bytes (x once, y once). One thread owns
// one Philox block of eight elements: 16 bytes of a 16-bit type, 32 of fp32.
// A call of ten rounds is 20 wide multiplies and 20 three-input xors for eight
// elements, under half of the issue slots that the memory time leaves.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "philox.cuh"
#include "rib_internal.h"
#include "sm100.cuh"

namespace rib {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerThread = 2;   // Philox blocks of a thread, loaded before any is used

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }

// A dropped element is 0 whatever x holds (a selection, not a product).
// x and y may be the same buffer: each element is read and written by one thread.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T* x, T* y, size_t n, DropRng rng) {
  constexpr int W = sizeof(T) * 8 / 16;   // 16-byte words of a block
  const uint64_t stream = rng.offset + (rng.step ? *rng.step : 0ull);
  const size_t blocks = (n + 7) / 8;
  const size_t first = static_cast<size_t>(blockIdx.x) * kThreads * kBlocksPerThread + threadIdx.x;
  union Pack {
    uint4 w[W];
    T e[8];
  };
  Pack in[kBlocksPerThread];
#pragma unroll
  for (int k = 0; k < kBlocksPerThread; ++k) {
    const size_t b = first + static_cast<size_t>(k) * kThreads;
    if (b >= blocks) continue;
    if (VEC && b * 8 + 8 <= n) {
#pragma unroll
      for (int i = 0; i < W; ++i) in[k].w[i] = reinterpret_cast<const uint4*>(x + b * 8)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) in[k].e[i] = b * 8 + i < n ? x[b * 8 + i] : from_f<T>(0.f);
    }
  }
#pragma unroll
  for (int k = 0; k < kBlocksPerThread; ++k) {
    const size_t b = first + static_cast<size_t>(k) * kThreads;
    if (b >= blocks) continue;
    const uint4 bits = philox4x32_10(b, stream, rng.seed);
    Pack out;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      out.e[i] = from_f<T>(drop_bits(bits, i) >= rng.threshold ? to_f(in[k].e[i]) * rng.up : 0.f);
    if (VEC && b * 8 + 8 <= n) {
#pragma unroll
      for (int i = 0; i < W; ++i) reinterpret_cast<uint4*>(y + b * 8)[i] = out.w[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (b * 8 + i < n) y[b * 8 + i] = out.e[i];
    }
  }
}

template <typename T>
cudaError_t launch_dropout(const void* x, void* y, size_t n, const DropRng& rng, cudaStream_t stream) {
  const size_t per_cta = static_cast<size_t>(kThreads) * kBlocksPerThread * 8;
  const size_t ctas = (n + per_cta - 1) / per_cta;
  if (ctas > 0x7FFFFFFFull) return cudaErrorInvalidConfiguration;
  const bool vec = (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % 16 == 0;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (vec) dropout_kernel<T, true><<<grid, kThreads, 0, stream>>>(static_cast<const T*>(x), static_cast<T*>(y), n, rng);
  else dropout_kernel<T, false><<<grid, kThreads, 0, stream>>>(static_cast<const T*>(x), static_cast<T*>(y), n, rng);
  return cudaGetLastError();
}

}  // namespace

bool make_drop_rng(float p, uint64_t seed, uint64_t offset, const uint64_t* step, DropRng* rng) {
  if (!(p >= 0.f && p <= 1.f)) return false;
  const uint32_t thr = static_cast<uint32_t>(std::floor(static_cast<double>(p) * 65536.0 + 0.5));
  rng->threshold = thr;
  rng->up = thr < 65536u ? static_cast<float>(65536.0 / (65536u - thr)) : 0.f;
  rng->seed = seed;
  rng->offset = offset;
  rng->step = step;
  return true;
}

}  // namespace rib

using namespace rib;

extern "C" rib_status rib_dropout(const void* x, void* y, rib_dtype dtype, size_t n, float p, uint64_t seed,
                                  uint64_t offset, const uint64_t* step, cudaStream_t stream) {
  if (dtype != RIB_BF16 && dtype != RIB_F32 && dtype != RIB_F16)
    return fail(RIB_ERR_INVALID_ARG, "rib_dropout: dtype must be RIB_BF16, RIB_F32 or RIB_F16");
  DropRng rng{};
  if (!make_drop_rng(p, seed, offset, step, &rng)) return fail(RIB_ERR_INVALID_ARG, "rib_dropout: p must be in [0, 1]");
  if ((!x || !y) && n) return fail(RIB_ERR_INVALID_ARG, "rib_dropout: null pointer");
  const size_t size = dtype == RIB_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % size || reinterpret_cast<uintptr_t>(y) % size || reinterpret_cast<uintptr_t>(step) % 8)
    return fail(RIB_ERR_ALIGNMENT, "rib_dropout: x and y need their element's alignment, step 8 bytes");
  if (n > (size_t(1) << 42)) return fail(RIB_ERR_UNSUPPORTED, "rib_dropout: n above 2^42");
  if (n == 0) return RIB_OK;
  cudaError_t e = dtype == RIB_F32   ? launch_dropout<float>(x, y, n, rng, stream)
                  : dtype == RIB_F16 ? launch_dropout<__half>(x, y, n, rng, stream)
                                     : launch_dropout<__nv_bfloat16>(x, y, n, rng, stream);
  if (e != cudaSuccess) return cuda_fail(e, "rib_dropout launch");
  return RIB_OK;
}
