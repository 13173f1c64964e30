// rope.cuh -- norm and position rotation of one head row, shared by the kernels
// that write rotated queries and keys (rope.cu).
//
//   y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
//
// A row of D channels is held by D / 8 neighbouring lanes, two runs of four
// channels each.  The runs are chosen so that both partners of every rotated pair
// sit in one lane, so the rotation needs no exchange: with half-split pairs
// (i, i + R/2) lane l < R/8 holds 4l .. 4l+3 and R/2 + 4l .. R/2 + 4l+3, with
// interleaved pairs (2i, 2i + 1) it holds 8l .. 8l+7; lanes from R/8 on hold eight
// channels that are not rotated.  Either way lane l needs the four angles
// 4l .. 4l+3 of its token, one 16-byte load of cosines and one of sines.
// Everything is fp32 with explicit roundings (so every kernel gives the same bits)
// and is rounded to bf16 once, at the end.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace spd {

struct RopeLane {
    int o0, o1;   // first channel of the lane's two runs
    bool turned;  // the lane's channels are rotated
};

template <int D>
__device__ __forceinline__ RopeLane rope_lane(int l, int rot, int interleaved) {
    RopeLane r;
    r.turned = l < (rot >> 3);
    if (r.turned && !interleaved) {
        r.o0 = 4 * l;
        r.o1 = (rot >> 1) + 4 * l;
    } else {
        r.o0 = 8 * l;
        r.o1 = 8 * l + 4;
    }
    return r;
}

__device__ __forceinline__ void unpack4(const uint2& u, float* x) {
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

__device__ __forceinline__ uint2 pack4(const float* x) {
    return make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

// The lane's weights, or ones.
__device__ __forceinline__ void rope_weights(const uint16_t* w, const RopeLane& r, float* wt) {
    if (w) {
        unpack4(__ldg(reinterpret_cast<const uint2*>(w + r.o0)), wt);
        unpack4(__ldg(reinterpret_cast<const uint2*>(w + r.o1)), wt + 4);
    }
}

// Normalises (when `norm`) and rotates the lane's eight channels in place.  cs and
// sn are the lane's four angles (read only when turned).  By whole warps.
template <int D>
__device__ __forceinline__ void rope_row(float* x, bool norm, const float* wt, float eps, const RopeLane& r,
                                         int interleaved, const float4& cs, const float4& sn) {
    if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __fmaf_rn(x[i], x[i], ss);
#pragma unroll
        for (int off = 1; off < D / 8; off <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
        const float inv = rsqrtf(__fmaf_rn(ss, 1.f / D, eps));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), wt[i]);
    }
    if (r.turned) {
        const float c[4] = {cs.x, cs.y, cs.z, cs.w}, s[4] = {sn.x, sn.y, sn.z, sn.w};
        auto turn = [](float& a, float& b, float co, float si) {
            const float a0 = a;
            a = __fmaf_rn(a0, co, -__fmul_rn(b, si));
            b = __fmaf_rn(b, co, __fmul_rn(a0, si));
        };
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], c[i], s[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) turn(x[i], x[i + 4], c[i], s[i]);
        }
    }
}

}  // namespace spd
