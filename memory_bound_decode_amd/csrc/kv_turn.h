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

__device__ __forceinline__ bool has_row(const Turn& u, int32_t t) {
    const int32_t p = u.positions[t];
    return p >= 0 && p < u.n_positions;
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

// Eight channels as loaded, all from one address or each four from its own.
template <class T> struct Eight;
template <> struct Eight<float> {
    f32x4 a, b;
    __device__ void load(const float* p) { load(p, p + 4); }
    __device__ void load(const float* p, const float* q) { a = load4(p), b = load4(q); }
    __device__ f32x4 low() const { return a; }
    __device__ f32x4 high() const { return b; }
};
template <> struct Eight<uint16_t> {
    u32x4 w;
    static __device__ f32x4 four(uint32_t x, uint32_t y) {
        return f32x4{__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u), __uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u)};
    }
    __device__ void load(const uint16_t* p) { w = *reinterpret_cast<const u32x4*>(p); }
    __device__ void load(const uint16_t* p, const uint16_t* q) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(p), y = *reinterpret_cast<const u32x2*>(q);
        w = u32x4{x[0], x[1], y[0], y[1]};
    }
    __device__ f32x4 low() const { return four(w[0], w[1]); }
    __device__ f32x4 high() const { return four(w[2], w[3]); }
};

// A wave takes 8 tokens x 8 octets (64 channels) of several heads, one after the other, which are turned by
// the same angles: prompts of 19.5k tokens x (32 + 8) heads x 128 in bf16 into 4 bits 161 us with the angles read for each
// head, 88 so, which is the rate of a plain copy.  (With an octet and its partners in one lane, so that both are
// read once: 89, and one token 4.8 us for 4.1.)
constexpr int kTurnRows = 8;             // tokens of a wave
constexpr int kTurnHeads = 4;            // heads whose loads are in flight together

// put(h, x0, x1) for channels d .. d+8 of heads h0 .. h1 of the token whose heads begin at `from`.
template <bool TURN, class T, class Put>
__device__ __forceinline__ void each_head(const Turn& u, const T* from, int d, int head_dim, int h0, int h1, const Angles& a0, const Angles& a1, Put&& put) {
    const bool whole = TURN && u.rot % 16 == 0;              // an octet's partners are an octet
    const bool pairs = TURN && u.pairs;
    for (int hb = h0; hb < h1; hb += kTurnHeads) {
        Eight<T> x[kTurnHeads], y[kTurnHeads];
#pragma unroll
        for (int i = 0; i < kTurnHeads; ++i) {
            if (hb + i >= h1) break;
            const T* head = from + int64_t(hb + i) * head_dim;
            x[i].load(head + d);
            if (TURN && !pairs) {                            // (channels that are not turned load themselves)
                const int p = a0.partner < 0 ? d : a0.partner, q = a1.partner < 0 ? d + 4 : a1.partner;
                if (whole) y[i].load(head + p);
                else y[i].load(head + p, head + q);
            }
        }
#pragma unroll
        for (int i = 0; i < kTurnHeads; ++i) {
            if (hb + i >= h1) break;
            f32x4 x0 = x[i].low(), x1 = x[i].high();
            if (TURN) {
                const f32x4 y0 = pairs ? f32x4{x0[1], x0[0], x0[3], x0[2]} : y[i].low(), y1 = pairs ? f32x4{x1[1], x1[0], x1[3], x1[2]} : y[i].high();
                if (a0.partner >= 0) x0 = a0.turn(x0, y0);
                if (a1.partner >= 0) x1 = a1.turn(x1, y1);
            }
            put(hb + i, x0, x1);
        }
    }
}

// Eight channels of queries, rounded to bf16.
__device__ __forceinline__ void store_query(const Turn& u, int64_t token, int64_t at, const f32x4 x0, const f32x4 x1) {
    *reinterpret_cast<u32x4*>(u.q_out + token * u.q_out_stride + at) =
        u32x4{pack_bf16(x0[0], x0[1]), pack_bf16(x0[2], x0[3]), pack_bf16(x1[0], x1[1]), pack_bf16(x1[2], x1[3])};
}

// The queries of a wave's 8 tokens from t0 on, channels 64 column .. +64 of heads h0 .. h1.
template <class T>
__device__ __forceinline__ void turn_queries(const Turn& u, int64_t t0, int32_t tokens, int column, int h0, int h1, int head_dim) {
    const int lane = threadIdx.x & 63, d = column * 64 + (lane & 7) * 8;
    const int64_t token = t0 + (lane >> 3);
    if (token >= tokens) return;
    const int32_t p = u.positions[token];
    if (p < 0 || p >= u.n_positions) return;
    const float* row = u.table + int64_t(p) * u.rot;
    Angles a0, a1;
    a0.load(u, row, d);
    a1.load(u, row, d + 4);
    each_head<true>(u, static_cast<const T*>(u.q) + token * u.q_stride, d, head_dim, h0, h1, a0, a1,
                    [&](int h, const f32x4 x0, const f32x4 x1) { store_query(u, token, int64_t(h) * head_dim + d, x0, x1); });
}

}  // namespace kv
}  // namespace mbd
