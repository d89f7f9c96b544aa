// heavy.cuh -- arguments of the attention over a heavy-hitter draft cache (heavy.cu, heavy_tc.cu).
#pragma once

#include "common.cuh"

namespace magicdec {

struct HeavyParams {
    const uint16_t *q;
    const uint16_t *v;               // of the tensor map, for values that are not finite
    uint16_t *out;
    float *weight;
    int32_t *pos;
    const int32_t *len, *next_pos;
    int *err;
    int B, H_q, H_kv, G, n, cap, R;
    int stride;                      // floats between two query rows' scores
    int stages;                      // of the ring (both: heavy.cu's way only)
    float scale_log2;                // log2(e) / sqrt(d)
};

double heavy_time(long long pairs, int cap, int C, int keys, double each, double way);
// By up to 32 query rows of a KV head, the scores of all but a stretch's last tiles computed twice.
magicdec_status launch_heavy_tc(const HeavyParams &p, int D, const uint16_t *k, const uint16_t *v, cudaStream_t st);

}  // namespace magicdec
