// What the decode kernels (decode.cu, decode_mx.cu) share: the per-stage record the producer
// warp hands its consumers, the ring's barriers, and the voted, bounded wait.
#pragma once

#include <cstdint>

#include "device_utils.cuh"
#include "pva_internal.h"

namespace pva {
namespace {

struct StageInfo {
    int32_t unit, group, k, k1;
    int32_t tok0, ntok, qpos0, nsplit;
    int32_t pbase, split, flags, hb;
    int32_t nparts;
    int32_t index;  // decode_mx.cu: the stage's number in its unit
    int32_t pad1, pad2;
};
constexpr int kFirst = 1, kLast = 2, kEnd = 4;

template <int I>
struct IntTag {
    static constexpr int value = I;
};

struct DecSmemHead {
    uint64_t full[8];
    uint64_t empty[8];
    StageInfo info[8];
    int32_t abort_flag;
};

__device__ __forceinline__ void abort_cta(DecSmemHead* sh, uint32_t* err) {
    sh->abort_flag = 1;
    dev::set_error(err, kErrTimeout);
}

// A work wait of one whole warp (every lane calls it, converged): the lanes' results are
// voted, so the warp leaves together or not at all (its next steps -- warp MMAs, fragment
// loads, warp syncs -- need every lane); lane 0 records the abort.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit, DecSmemHead* sh,
                                          uint32_t* err) {
    if (__all_sync(0xffffffffu, dev::mbar_wait(bar, parity, limit))) return true;
    if ((threadIdx.x & 31) == 0) abort_cta(sh, err);
    __syncwarp();
    return false;
}

}  // namespace
}  // namespace pva
