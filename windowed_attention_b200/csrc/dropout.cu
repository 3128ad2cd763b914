// Dropout with a mask that is never stored (rib_dropout):
//   y[i] = bits16(i) >= threshold ? x[i] / keep : 0
// with the random bits of philox.cuh. The backward is the same call on the
// upstream gradient.
//
// One thread owns Philox blocks of eight elements: 16 bytes of a 16-bit type, 32
// of fp32; a block takes 20 wide multiplies and 20 three-input xors, and the
// selection works on word halves without taking them apart. 41.5 M bf16
// elements: 33-35 us, where their 166 MB take 25 at 6.54 TB/s; with one block a
// thread 39, with four 37 us. In fp32 (332 MB, 51 us) 50 us. In 16 bits nothing
// is full: issue 73 %, the pipe of the wide multiplies 63 %, ALU 59 %, memory
// 71 % of a copy's rate; for 11 % of the time, at the grid's start and end, SMs
// are idle.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "philox.cuh"
#include "rib_internal.h"
#include "sm100.cuh"

namespace rib {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerThread = 2;   // Philox blocks of a thread, loaded before any is used

// A dropped element is 0 whatever x holds (a selection, not a product).
// x and y may be the same buffer: each element is read and written by one thread.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T* x, T* y, size_t n, DropRng rng) {
  constexpr int W = sizeof(T) * 8 / 16;   // 16-byte words of a block
  const uint64_t stream = rng.offset + (rng.step ? *rng.step : 0ull);
  const size_t blocks = (n + 7) / 8;
  // thresholds up to 65535 in a word's high half; 65536 drops everything
  const uint32_t least = rng.threshold << 16;
  const bool all_dropped = rng.threshold > 65535u;
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
      for (int i = 0; i < 8; ++i) in[k].e[i] = b * 8 + i < n ? x[b * 8 + i] : T(0.f);
    }
  }
#pragma unroll
  for (int k = 0; k < kBlocksPerThread; ++k) {
    const size_t b = first + static_cast<size_t>(k) * kThreads;
    if (b >= blocks) continue;
    const uint4 bits = philox4x32_10(b, stream, rng.seed);
    const uint32_t words[4] = {bits.x, bits.y, bits.z, bits.w};
    Pack out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // elements 2 i and 2 i + 1 own the low and the high half of a word; both are compared in the high half's place
      const bool low = (words[i] << 16) >= least, high = words[i] >= least;
      if constexpr (sizeof(T) == 4) {
        out.e[2 * i] = low ? in[k].e[2 * i] * rng.up : T(0);
        out.e[2 * i + 1] = high ? in[k].e[2 * i + 1] * rng.up : T(0);
      } else {
        const uint32_t v = reinterpret_cast<const uint32_t*>(in[k].w)[i];
        const uint64_t up = f2_pack(rng.up, rng.up);
        float a, c;
        uint32_t r;
        if constexpr (std::is_same<T, __half>::value) {
          f2_unpack(f2_mul(f2_pack(f16_lo(v), f16_hi(v)), up), a, c);
          const __half2 h = __floats2half2_rn(a, c);
          r = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          f2_unpack(f2_mul(f2_pack(bf16_lo(v), bf16_hi(v)), up), a, c);
          r = pack_bf16x2(a, c);
        }
        reinterpret_cast<uint32_t*>(out.w)[i] = (low ? r & 0xFFFFu : 0u) | (high ? r & 0xFFFF0000u : 0u);
      }
    }
    if (all_dropped)
#pragma unroll
      for (int i = 0; i < W; ++i) out.w[i] = make_uint4(0u, 0u, 0u, 0u);
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
