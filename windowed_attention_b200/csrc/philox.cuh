// Counter-based random bits for dropout: Philox4x32-10 (Salmon, Moraes, Dror
// and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011). One call
// turns a 128-bit counter and a 64-bit key into 128 random bits; eight
// elements take 16 bits each. An element is kept where its 16 bits are at
// least the threshold round(65536 p), so the mask is a function of (element,
// seed, offset) alone: the backward draws it again and nothing is stored.
//
// 16 bits an element halve the integer products per element against 32 (the
// ten rounds are 20 wide multiplies a call); p is then a multiple of 2^-16,
// and the scale 65536 / (65536 - threshold) is that of the p in use, so the
// mean is exact.
#pragma once
#include <cstdint>

namespace rib {

struct DropRng {
  uint32_t threshold;     // 0: no dropout
  float up;               // 1 / (kept share); 0 when nothing is kept
  uint64_t seed, offset;
  const uint64_t* step;   // device word added to offset, or null
};

__device__ __forceinline__ uint4 philox4x32_10(uint64_t block, uint64_t stream, uint64_t seed) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = static_cast<uint32_t>(stream), c3 = static_cast<uint32_t>(stream >> 32);
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

}  // namespace rib
