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

// What turns channels d .. d+4 of any head of a token: x becomes x c + y s, where y are their partners.
// Products and sums are rounded one by one: the codes that come of them are the same wherever they are
// computed.  rot / 2 is a multiple of 4, so the four have their partners side by side as well.
struct Angles {
    f32x4 c, s;
    int partner;                         // first channel of the partners; d itself: in the four; -1: not turned

    __device__ __forceinline__ void load(const Turn& u, const float* row, int d) {
        const int half = u.rot / 2;
        partner = -1;
        if (d >= u.rot) return;
        if (u.pairs) {
            const f32x2 a = *reinterpret_cast<const f32x2*>(row + d / 2), b = *reinterpret_cast<const f32x2*>(row + half + d / 2);
            c = f32x4{a[0], a[0], a[1], a[1]};
            s = f32x4{-b[0], b[0], -b[1], b[1]};
            partner = d;
            return;
        }
        const bool second = d >= half;
        const int j = second ? d - half : d;
        c = load4(row + j);
        s = load4(row + half + j);
        if (!second) s = -s;
        partner = second ? j : d + half;
    }
    __device__ __forceinline__ f32x4 turn(const f32x4 x, const f32x4 y) const {
#pragma clang fp contract(off)
        const f32x4 a = x * c, b = y * s;
        return a + b;
    }
};

// Channels d .. d+4 of a head whose channel 0 is at `head`, turned by a row of the table.
template <class T>
__device__ __forceinline__ f32x4 turned(const Turn& u, const T* head, const float* row, int d) {
    const f32x4 x = load4(head + d);
    Angles a;
    a.load(u, row, d);
    if (a.partner < 0) return x;
    return a.turn(x, a.partner == d ? f32x4{x[1], x[0], x[3], x[2]} : load4(head + a.partner));
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
