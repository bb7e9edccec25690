// host_warp.h — enough of the device language for the CPU: a warp's lanes are threads, and its
// collectives exchange their values through a barrier. Device headers are included behind it.
#pragma once

#include <barrier>
#include <cstdint>
#include <cstring>
#include <thread>
#include <vector>

#include <cuda_runtime.h>

struct HostDim {
  unsigned x, y, z;
};
inline thread_local HostDim threadIdx{}, blockIdx{}, blockDim{}, gridDim{};

namespace host_warp {
inline std::barrier<> gate(32);
inline uint64_t slot[32];

template <class T>
T exchange(T v, int from) {  // what lane `from` gave
  uint64_t w = 0;
  std::memcpy(&w, &v, sizeof(T));
  slot[threadIdx.x & 31] = w;
  gate.arrive_and_wait();
  w = slot[from & 31];
  gate.arrive_and_wait();
  std::memcpy(&v, &w, sizeof(T));
  return v;
}
template <class T, class F>
T reduce(T v, F f) {
  slot[threadIdx.x & 31] = static_cast<uint64_t>(v);
  gate.arrive_and_wait();
  T r = static_cast<T>(slot[0]);
  for (int i = 1; i < 32; ++i) r = f(r, static_cast<T>(slot[i]));
  gate.arrive_and_wait();
  return r;
}
// f(lane) by 32 threads.
template <class F>
void warp(F f) {
  std::vector<std::thread> t;
  for (unsigned i = 0; i < 32; ++i)
    t.emplace_back([&f, i] {
      threadIdx.x = i;
      f(static_cast<int>(i));
    });
  for (auto& x : t) x.join();
}
}  // namespace host_warp

template <class T>
T __shfl_sync(unsigned, T v, int from) { return host_warp::exchange(v, from); }
template <class T>
T __shfl_up_sync(unsigned, T v, int off) {
  const int lane = threadIdx.x & 31;
  return host_warp::exchange(v, lane >= off ? lane - off : lane);
}
template <class T>
T __shfl_xor_sync(unsigned, T v, int mask) { return host_warp::exchange(v, (threadIdx.x & 31) ^ mask); }
inline unsigned __reduce_add_sync(unsigned, unsigned v) { return host_warp::reduce(v, [](unsigned a, unsigned b) { return a + b; }); }
inline int __reduce_max_sync(unsigned, int v) {
  return host_warp::reduce(v, [](int a, int b) { return a > b ? a : b; });
}
inline unsigned __ballot_sync(unsigned, bool p) {
  return host_warp::reduce(p ? 1u << (threadIdx.x & 31) : 0u, [](unsigned a, unsigned b) { return a | b; });
}
inline int __ffs(unsigned v) { return __builtin_ffs(static_cast<int>(v)); }
inline unsigned __umulhi(unsigned a, unsigned b) { return static_cast<unsigned>((static_cast<uint64_t>(a) * b) >> 32); }
inline float __uint_as_float(unsigned v) {
  float f;
  std::memcpy(&f, &v, 4);
  return f;
}
inline float __int_as_float(int v) { return __uint_as_float(static_cast<unsigned>(v)); }
inline unsigned __vminu4(unsigned a, unsigned b) {
  unsigned r = 0;
  for (int i = 0; i < 32; i += 8) {
    const unsigned x = a >> i & 255u, y = b >> i & 255u;
    r |= (x < y ? x : y) << i;
  }
  return r;
}
template <class T>
T __ldcg(const T* p) { return *p; }
template <class T>
T __ldg(const T* p) { return *p; }
inline size_t __cvta_generic_to_shared(const void* p) { return reinterpret_cast<size_t>(p); }
inline int atomicOr(int* p, int v) { return __atomic_fetch_or(p, v, __ATOMIC_RELAXED); }
template <class T>
T min(T a, T b) { return a < b ? a : b; }
template <class T>
T max(T a, T b) { return a > b ? a : b; }
