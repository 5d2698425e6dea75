// Which copies of a ring of shared-memory stages are in flight, for the path on which a wait ran out.
//
// Copy n goes into stage n % stages and completes phase n / stages of that stage's barrier.  The first `stages`
// copies are issued ahead, and copy n + stages only after copy n has landed; so when the wait for copy `landed`
// runs out, copies [landed, ring_end) are in flight, at most one in a stage.
// Plain integers, so that the bookkeeping also compiles and is tested on the host.
#pragma once

#ifdef __CUDACC__
#define DSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DSA_HOST_DEVICE inline
#endif

namespace dsa {

DSA_HOST_DEVICE int ring_stage(int n, int stages) { return n % stages; }
DSA_HOST_DEVICE unsigned ring_parity(int n, int stages) { return static_cast<unsigned>(n / stages) & 1u; }
DSA_HOST_DEVICE int ring_end(int landed, int stages, int copies) { return copies - landed < stages ? copies : landed + stages; }

}  // namespace dsa
