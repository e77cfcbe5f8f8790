// Rotation of keys and queries by position on their way out of the projection.
#pragma once

#include <hip/hip_runtime.h>

#include "kv_common.h"

namespace mbd {
namespace kv {

struct Turn {
    const float* table;                  // [n_positions][rot]
    const int32_t* positions;
    const void* q;
    uint16_t* q_out;
    int64_t q_stride, q_out_stride;
    int32_t n_positions, rot, n_q_heads;
    bool pairs;
};

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
}

// The slot that a token goes to: none where its position has no row in the table.
template <bool TURN>
__device__ __forceinline__ int32_t slot_at(const int32_t* slots, const Turn& u, int32_t t) {
    const int32_t s = slots[t];
    if constexpr (TURN) {
        const int32_t p = u.positions[t];
        if (p < 0 || p >= u.n_positions) return -1;
    }
    return s;
}

// Channels d .. d+4 of a head whose channel 0 is at `head`, turned by a row of the table.  rot / 2
// is a multiple of 4, so the four have their partners side by side as well.  Products and sums
// are rounded one by one: the codes that come of them are the same wherever they are computed.
template <class T>
__device__ __forceinline__ f32x4 turned(const Turn& u, const T* head, const float* row, int d) {
#pragma clang fp contract(off)
    const f32x4 x = load4(head + d);
    if (d >= u.rot) return x;
    const int half = u.rot / 2;
    if (u.pairs) {
        const f32x2 c = *reinterpret_cast<const f32x2*>(row + d / 2), s = *reinterpret_cast<const f32x2*>(row + half + d / 2);
        return f32x4{x[0] * c[0] - x[1] * s[0], x[1] * c[0] + x[0] * s[0], x[2] * c[1] - x[3] * s[1], x[3] * c[1] + x[2] * s[1]};
    }
    const bool second = d >= half;
    const int j = second ? d - half : d;
    const f32x4 y = load4(head + (second ? j : d + half)), c = load4(row + j), s = load4(row + half + j);
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = x[i] * c[i], b = y[i] * s[i];
        r[i] = second ? a + b : a - b;
    }
    return r;
}

// Eight channels (octet `o` of a token's row of queries) turned and rounded to bf16.
template <class T>
__device__ __forceinline__ void turn_query(const Turn& u, int32_t token, int o, int head_dim) {
    const int32_t p = u.positions[token];
    if (p < 0 || p >= u.n_positions) return;
    const int h = o / (head_dim / 8), d = (o - h * (head_dim / 8)) * 8;
    const T* head = static_cast<const T*>(u.q) + token * u.q_stride + int64_t(h) * head_dim;
    const float* row = u.table + int64_t(p) * u.rot;
    const f32x4 a = turned(u, head, row, d), b = turned(u, head, row, d + 4);
    *reinterpret_cast<u32x4*>(u.q_out + token * u.q_out_stride + int64_t(h) * head_dim + d) =
        u32x4{pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(b[0], b[1]), pack_bf16(b[2], b[3])};
}

}  // namespace kv
}  // namespace mbd
