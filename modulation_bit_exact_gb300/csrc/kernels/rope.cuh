// rope.cuh -- the angles of rotary positions on several axes.
#pragma once

#include "rowgroup.cuh"

namespace mbx {

// cos and sin of 2*pi*turns.
__device__ __forceinline__ float2 cos_sin_turns(double turns) {
    const double q = turns * 4.0, r = rint(q);
    const int quadrant = (int)(long long)r & 3;
    float s, c;
    sincospif((float)(q - r) * 0.5f, &s, &c);  // |argument| <= 1/4
    const float cc = (quadrant & 1) ? -s : c, ss = (quadrant & 1) ? c : s;
    return (quadrant & 2) ? make_float2(-cc, -ss) : make_float2(cc, ss);
}

// cos and sin of the angle by which pair j of a token turns: `tok` is the token's
// index in the batch, `s` that in its sequence.
__device__ __forceinline__ float2 token_cos_sin(const RopeParams& p, unsigned tok, unsigned s, int j) {
    int a = 0;
    while (a < p.axes - 1 && j >= p.axis_end[a]) ++a;
    const int64_t prow = p.pos_batched ? tok : s;
    const double pos = p.pos_f32 ? (double)static_cast<const float*>(p.pos)[prow * p.pos_stride + a]
                                 : (double)static_cast<const int*>(p.pos)[prow * p.pos_stride + a];
    float2 v = cos_sin_turns(pos * (p.freqs[j] * 0.15915494309189533577));  // 1 / (2 pi)
    if (p.inverse) v.y = -v.y;
    return v;
}

}  // namespace mbx
