// Which pipeline stages a producer has copies in flight to, so that a CTA whose
// bounded wait ran out does not end before they have landed.
//
// A parity wait on an mbarrier succeeds while the phase of that parity is the
// last completed one: of the two parities exactly one succeeds at any time.  So
// a stage's barrier is asked for the parity of the phase that its last copy
// completes, never for either of the two.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ARMT_COPIES_FN __device__ __forceinline__
#else
#define ARMT_COPIES_FN inline
#endif

namespace armt {

struct CopiesInFlight {
  uint32_t stages = 0;   // bit s: a copy was issued to stage s
  uint32_t parity = 0;   // bit s: parity of the phase that the last one completes

  ARMT_COPIES_FN void issued(int s, uint32_t phase_parity) {
    stages |= 1u << s;
    parity = (parity & ~(1u << s)) | (phase_parity & 1u) << s;
  }

  // Those of these copies that `other`, the pair's other CTA, has not issued.
  ARMT_COPIES_FN CopiesInFlight beyond(const CopiesInFlight& other) const {
    CopiesInFlight r;
    r.stages = stages & ~(other.stages & ~(parity ^ other.parity));
    r.parity = parity;
    return r;
  }

  // In one word, for at most 16 stages.
  ARMT_COPIES_FN uint32_t word() const { return (stages & 0xffffu) | parity << 16; }
  ARMT_COPIES_FN static CopiesInFlight of(uint32_t word) {
    CopiesInFlight r;
    r.stages = word & 0xffffu;
    r.parity = word >> 16;
    return r;
  }

  // landed(s, parity): whether that phase of stage s is complete; late(): whether
  // the limit is over.  True once every copy has landed.
  template <class Landed, class Late>
  ARMT_COPIES_FN bool drain(Landed landed, Late late) const {
    for (int s = 0; s < 32 && stages >> s; ++s) {
      if (!(stages >> s & 1u)) continue;
      while (!landed(s, parity >> s & 1u))
        if (late()) return false;
    }
    return true;
  }
};

}  // namespace armt
