// Order in which a thread's asynchronous stores take its N staging buffers.  Plain C++, so that a host program
// can walk it too.
#pragma once

#ifdef __CUDACC__
#define MLA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MLA_HOST_DEVICE inline
#endif

namespace mla {

// One store group is committed per take().  A wait that leaves at most N - 1 groups pending, in front of
// writing the buffer taken, covers that buffer's last store: the N - 1 newest groups hold the other buffers.  That
// needs the turns to go on over the whole life of the thread; a count that starts again (with every output
// tile, say) breaks it wherever the number of stores in between is no multiple of N.
template <int N>
struct StoreRing {
  static_assert(N > 0 && (N & (N - 1)) == 0, "a power of two: the count may wrap");
  unsigned turn = 0;
  MLA_HOST_DEVICE int take() { return (int)(turn++ % N); }
};

}  // namespace mla
