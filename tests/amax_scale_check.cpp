// a/448 and 448/a as the kernels work them out (amax_scale, taken from csrc/block.hpp as it stands)
// against the two divisions, for every float from 2^lo up to 2^hi, with the hardware's
// reciprocal, which is within one unit in the last place, taken as the nearest float and its two
// neighbours. Usage: amax_scale_check lo hi
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <thread>
#include <vector>

#define __device__
#define __forceinline__ inline __attribute__((always_inline))

static float from_bits(uint32_t u) {
  float f;
  std::memcpy(&f, &u, 4);
  return f;
}
static uint32_t bits(float f) {
  uint32_t u;
  std::memcpy(&u, &f, 4);
  return u;
}

template <int kOff>
struct Check {
  static float reciprocal(float x) { return from_bits(bits(1.0f / x) + kOff); }
#define __builtin_amdgcn_rcpf reciprocal
#define AMAX_SCALE static
#include "amax_scale.inc"
  // Mismatches among the floats whose bit patterns are first .. last - 1.
  static uint64_t wrong(uint32_t first, uint32_t last) {
    uint32_t n = 0;
    for (uint32_t u = first; u < last; ++u) {
      const float a = from_bits(u);
      float s, r;
      amax_scale(a, s, r);
      n += bits(s) != bits(a / 448.0f);
      n += bits(r) != bits(448.0f / a);
    }
    return n;
  }
};

int main(int argc, char** argv) {
  if (argc != 3) return 2;
  const int lo = std::atoi(argv[1]), hi = std::atoi(argv[2]);
  if (lo < -119 || hi > 128 || lo >= hi) return 2;
  uint64_t wrong = 0;
  std::vector<std::thread> pool;
  std::vector<uint64_t> part(8, 0);
  for (int t = 0; t < 8; ++t)
    pool.emplace_back([&, t] {
      for (int e = lo + t; e < hi; e += 8) {  // one binade at a time
        const uint32_t u = static_cast<uint32_t>(e + 127) << 23, v = u + (1u << 23);
        part[t] += Check<-1>::wrong(u, v) + Check<0>::wrong(u, v) + Check<1>::wrong(u, v);
      }
    });
  for (auto& p : pool) p.join();
  for (uint64_t n : part) wrong += n;
  std::printf("%llu wrong of %d binades\n", static_cast<unsigned long long>(wrong), hi - lo);
  return wrong == 0 ? 0 : 1;
}
