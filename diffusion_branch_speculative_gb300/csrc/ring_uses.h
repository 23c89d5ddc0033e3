// The uses of a ring of buffers.  Plain C++: the tests compile it for the host.
#pragma once

#ifdef __CUDACC__
#define SF_RING __host__ __device__ __forceinline__
#else
#define SF_RING inline
#endif

namespace sf {

// f(slot, parity) for the last use of every slot of a ring whose uses 0 .. last have begun
// (-1: none); use i has slot i % ring and completes the phase i / ring of its barrier.
template <typename F>
SF_RING void each_last_use(int last, int ring, F f) {
  for (int i = last >= ring ? last - ring + 1 : 0; i <= last; ++i) f(i % ring, static_cast<unsigned>(i / ring) & 1u);
}

}  // namespace sf
