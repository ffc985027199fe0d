// A warp's waits in a kernel whose warps hand tiles to one another through mbarriers.
//
// mbar_wait gives up after its limit lane by lane: lanes that saw the phase in time and lanes that
// did not would part, and the first would reach the warp's shuffles and matrix instructions without
// the others.  Here all lanes take the same answer, and a warp that gave up once never waits
// again, however many tiles are left: a kernel in which a copy or an arrival is missing ends after
// one limit for each link of the chain, not for each tile.
#pragma once

#include <stdint.h>

namespace skv {

struct WarpWait {
  unsigned int* err;
  bool ok = true;  // no wait of this warp has given up

  __device__ __forceinline__ explicit WarpWait(unsigned int* e) : err(e) {}

  // The whole warp calls it.  False, without waiting, once a wait has given up.
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, unsigned int code) {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, err, code)) != 0;
    return ok;
  }
};

}  // namespace skv
