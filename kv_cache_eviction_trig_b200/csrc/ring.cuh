// Shared-memory places that copies fill in turn, each with an mbarrier whose phases count the
// place's fills.  Plain C++, so that it compiles for the host too.
#pragma once

#ifdef __CUDACC__
#define TRIA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define TRIA_HOST_DEVICE inline
#endif

namespace tria {

// Waits for the last of `issued` copies in every place of a ring that has seen any.  The parity of
// that fill is needed: of a barrier's two parities one always tests as complete, that of
// the phase before the current one, whether or not a copy is under way.
template <class Await>
TRIA_HOST_DEVICE void drain_ring(int issued, int places, Await await) {
  for (int s = 0; s < places && s < issued; ++s) await(s, (unsigned)((issued - 1 - s) / places) & 1u);
}

}  // namespace tria
