// The distribution each drafted token was drawn from: row t of a sequence is
// the softmax of the pair scores of the token chosen at t - 1, over the K
// candidates ("DFlash 2: Keep Drafting Parallel", section "A Lightweight Path
// Selector": sampling draws from the same scores; rejection sampling needs
// the whole row to draw from what is left of the target).
//
// One wave a position, a lane a candidate.  Maximum, exponentials and the sum
// in rank order are those of the sampling walk's draw, so that the drawn
// token's entry is the walk's q bit for bit.
#pragma once

#include "common.hpp"

namespace df2 {

struct DraftArgs {
    const float* S;             // [B, P, K, K]
    const int32_t* cand;        // [B, P, K]
    const int32_t* path;        // [B, P]
    int32_t* out_cand;          // [B, P, K] or NULL
    float* out_rows;            // [B, P, K]
    int P, K;
    float inv_tau;
};

__global__ __launch_bounds__(64) void k_draft_rows(DraftArgs a) {
    const int lane = lane_id(), K = a.K;
    const int64_t pos = blockIdx.x;
    const int t = (int)(pos % a.P);
    int i = 0;
    if (t > 0) {
        // the rank of the token chosen one step earlier (0 if it is none)
        const int32_t before = a.path[pos - 1];
        const int32_t id = a.cand[(pos - 1) * K + min(lane, K - 1)];
        const uint64_t hit = __ballot(lane < K && id == before);
        i = hit ? __builtin_ctzll(hit) : 0;
    }
    const float v = a.S[(pos * K + i) * K + min(lane, K - 1)];
    const float m = wave_max_f32(v);
    const float e = lane < K ? expf((v - m) * a.inv_tau) : 0.f;
    float z = 0.f;
    for (int k = 0; k < K; ++k) z += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(e), k));
    if (lane < K) {
        a.out_rows[pos * K + lane] = e / z;
        if (a.out_cand) a.out_cand[pos * K + lane] = a.cand[pos * K + lane];
    }
}

}  // namespace df2
