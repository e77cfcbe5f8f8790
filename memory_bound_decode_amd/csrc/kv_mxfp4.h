// Append to and read-back of the 4-bit KV cache (MBD_KV_MXFP4).
//
// A token's codes depend on that token alone, so there is nothing to share between its rows: a
// lane takes eight channels of one token (an octet), four lanes a group of 32, whose maximum
// gives the exponent.  What costs is where the bytes lie: a tile of 16 tokens keeps a token's codes
// in pieces of 16 bytes (keys) and 4 (values), so the lanes of a wave are laid over (tokens,
// octets) such that its stores fill whole lines where tokens follow each other in a tile: keys 16
// tokens x one group, values 4 tokens x 16 octets.
#pragma once

#include <hip/hip_runtime.h>

#include "kv_turn.h"

namespace mbd {
namespace kv {

constexpr int kRows4 = 16;               // tokens of a workgroup's window

struct Cache4Args {
    uint8_t *codes[2], *scales[2];
    const int32_t* slots;
    int32_t n_slots, T, n_heads, shift;
};

// A token's place in one side of the cache.
template <int DQ>
struct Place4 {
    int64_t tile;                        // of 16 tokens x one head
    int t;                               // token in the tile
    __device__ Place4(const Cache4Args& a, int32_t slot, int head) {
        const int64_t bh = int64_t(slot >> a.shift) * a.n_heads + head;
        tile = (bh << (a.shift - 4)) + ((slot & ((1 << a.shift) - 1)) >> 4);
        t = slot & 15;
    }
    __device__ int64_t scale(int d) const { return tile * (32 * DQ) + d / 32 * 16 + t; }
    __device__ int64_t key(int d) const { return tile * (512 * DQ) + d / 32 * 256 + t * 16 + d % 32 / 2; }
    // an octet of values: 4 bytes, or in a last half slab 2, and 2 more 8 bytes further on
    __device__ static bool halved(int d) { return DQ % 2 && d >= DQ / 2 * 128; }
    __device__ int64_t value(int d) const {
        const int64_t at = tile * (512 * DQ) + d / 128 * 1024;
        if (halved(d)) return at + t / 4 * 128 + d % 64 / 4 * 8 + t % 4 * 2;
        return at + t / 4 * 256 + d % 128 / 8 * 16 + t % 4 * 4;
    }
};

struct Append4Args {
    Cache4Args c;
    const void* x[2];
    int64_t stride[2];
    int32_t k_tasks, v_tasks, tasks;     // of waves; what follows the keys' and the values' are the queries'
    Turn turn;
};

// Largest of the four lanes of a group.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xb1, 0xf, 0xf, false)));    // quad_perm 1 0 3 2
    return max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4e, 0xf, 0xf, false))); // quad_perm 2 3 0 1
}

// The smallest e with amax <= 7 * 2^e, from amax's bits: 7 = 1.75 * 2^2.
__device__ __forceinline__ int exponent4(uint32_t amax) {
    return min(max(int(amax >> 23) - 129 + ((amax & 0x7fffffu) > 0x600000u), -100), 125);
}

// Eight codes, and the byte of their group's exponent.  The conversion rounds x / 2^e to the
// nearest, ties to even, and saturates.
__device__ __forceinline__ uint32_t encode4(const f32x4 x0, const f32x4 x1, int* e) {
    float x[8] = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
        top = max(top, b < 0x7f800000u ? b : 0u);
        x[i] = x[i] == x[i] ? x[i] : 0.f;
    }
    *e = exponent4(quad_max(top)) + 127;
    const float s = __uint_as_float(uint32_t(*e) << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
}

template <int DQ, class T, bool TURN>
__global__ __launch_bounds__(256) void append4_kernel(Append4Args a) {
    constexpr int D = 64 * DQ;
    const int lane = threadIdx.x & 63;
    const int task = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (task >= a.tasks) return;
    const bool keys = task < a.k_tasks, queries = TURN && task >= a.k_tasks + a.v_tasks;
    const int side = keys ? 0 : 1, spread = queries ? task - a.k_tasks - a.v_tasks : task - a.k_tasks;
    const int row = keys ? lane >> 2 : (spread & 3) * 4 + (lane >> 4);
    const int octet = keys ? task * 4 + (lane & 3) : (spread >> 2) * 16 + (lane & 15);
    const int octets = (queries ? a.turn.n_q_heads : a.c.n_heads) * (D / 8);
    if (octet >= octets) return;
    const int head = octet / (D / 8), d = (octet - head * (D / 8)) * 8;
    for (int64_t w0 = int64_t(blockIdx.y) * kRows4; w0 < a.c.T; w0 += int64_t(gridDim.y) * kRows4) {
        const int64_t token = w0 + row;
        if (token >= a.c.T) continue;
        if (queries) {
            if constexpr (TURN) turn_query<T>(a.turn, int32_t(token), octet, D);
            continue;
        }
        const int32_t slot = slot_at<TURN>(a.c.slots, a.turn, int32_t(token));
        if (slot < 0 || slot >= a.c.n_slots) continue;
        const T* from = static_cast<const T*>(a.x[side]) + token * a.stride[side] + int64_t(head) * D;
        f32x4 x0, x1;
        if (TURN && keys) {
            const float* angles = a.turn.table + int64_t(a.turn.positions[token]) * a.turn.rot;
            x0 = turned(a.turn, from, angles, d);
            x1 = turned(a.turn, from, angles, d + 4);
        } else {
            x0 = load4(from + d);
            x1 = load4(from + d + 4);
        }
        int e;
        const uint32_t codes = encode4(x0, x1, &e);
        const Place4<DQ> at(a.c, slot, head);
        if ((lane & 3) == 0) a.c.scales[side][at.scale(d)] = uint8_t(e);
        if (keys) {
            *reinterpret_cast<uint32_t*>(a.c.codes[0] + at.key(d)) = codes;
        } else if (Place4<DQ>::halved(d)) {
            uint16_t* to = reinterpret_cast<uint16_t*>(a.c.codes[1] + at.value(d));
            to[0] = uint16_t(codes);
            to[4] = uint16_t(codes >> 16);
        } else {
            *reinterpret_cast<uint32_t*>(a.c.codes[1] + at.value(d)) = codes;
        }
    }
}

// Eight codes and the scale's bits as fp32.
__device__ __forceinline__ void decode4(uint32_t w, uint32_t e, f32x4* x0, f32x4* x1) {
    const float s = __uint_as_float(e << 23);
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    *x0 = f32x4{a[0], a[1], b[0], b[1]};
    *x1 = f32x4{c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ void stream8(float* p, const f32x4 x0, const f32x4 x1) {
    __builtin_nontemporal_store(x0, reinterpret_cast<f32x4*>(p));
    __builtin_nontemporal_store(x1, reinterpret_cast<f32x4*>(p + 4));
}
__device__ __forceinline__ void stream8(uint16_t* p, const f32x4 x0, const f32x4 x1) {
    __builtin_nontemporal_store(u32x4{pack_bf16(x0[0], x0[1]), pack_bf16(x0[2], x0[3]), pack_bf16(x1[0], x1[1]), pack_bf16(x1[2], x1[3])},
                                reinterpret_cast<u32x4*>(p));
}

constexpr int kGather4 = 2;              // tokens of one thread

// 16 octets x 16 tokens, twice, of keys and values: a line of codes holds 8 tokens of one group, or
// 4 of 64 channels, all of them read by this workgroup.
template <int DQ, class T>
__global__ __launch_bounds__(256) void gather4_kernel(Cache4Args a, T* k_out, T* v_out) {
    constexpr int D = 64 * DQ;
    const int row = threadIdx.x >> 4, octet = blockIdx.x * 16 + (threadIdx.x & 15), octets = a.n_heads * (D / 8);
    if (octet >= octets) return;
    const int head = octet / (D / 8), d = (octet - head * (D / 8)) * 8;
    for (int64_t w0 = int64_t(blockIdx.y) * (16 * kGather4); w0 < a.T; w0 += int64_t(gridDim.y) * (16 * kGather4)) {
        int32_t slot[kGather4];
        uint32_t kw[kGather4], vw[kGather4], ke[kGather4], ve[kGather4];
#pragma unroll
        for (int i = 0; i < kGather4; ++i) {
            const int64_t token = w0 + 16 * i + row;
            slot[i] = token < a.T ? a.slots[token] : -1;
            if (slot[i] >= a.n_slots) slot[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < kGather4; ++i)
            if (slot[i] >= 0) {
                const Place4<DQ> at(a, slot[i], head);
                kw[i] = *reinterpret_cast<const uint32_t*>(a.codes[0] + at.key(d));
                if (Place4<DQ>::halved(d)) {
                    const uint16_t* from = reinterpret_cast<const uint16_t*>(a.codes[1] + at.value(d));
                    vw[i] = from[0] | uint32_t(from[4]) << 16;
                } else {
                    vw[i] = *reinterpret_cast<const uint32_t*>(a.codes[1] + at.value(d));
                }
                ke[i] = a.scales[0][at.scale(d)];
                ve[i] = a.scales[1][at.scale(d)];
            }
#pragma unroll
        for (int i = 0; i < kGather4; ++i)
            if (slot[i] >= 0) {
                const int64_t to = (w0 + 16 * i + row) * (int64_t(a.n_heads) * D) + int64_t(octet) * 8;
                f32x4 x0, x1;
                decode4(kw[i], ke[i], &x0, &x1);
                stream8(k_out + to, x0, x1);
                decode4(vw[i], ve[i], &x0, &x1);
                stream8(v_out + to, x0, x1);
            }
    }
}

inline Cache4Args cache4_args(const mbd_kv_cache* c, const int32_t* slots, int32_t T) {
    return Cache4Args{{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->v_codes)},
                      {static_cast<uint8_t*>(c->k_scale), static_cast<uint8_t*>(c->v_scale)},
                      slots, int32_t(c->n_blocks * c->block_size), T, c->n_heads, log2_of(c->block_size)};
}

template <int DQ, class T>
void launch_append4(const Append4Args& a, dim3 grid, hipStream_t s) {
    if (a.turn.table) hipLaunchKernelGGL((append4_kernel<DQ, T, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((append4_kernel<DQ, T, false>), grid, dim3(256), 0, s, a);
}

template <class T>
void append4(const mbd_kv_cache* c, const Turn& turn, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
             const int32_t* slots, int32_t T_, hipStream_t s) {
    Append4Args a{cache4_args(c, slots, T_), {k, v}, {k_stride, v_stride}, 0, 0, 0, turn};
    const int dq = c->head_dim / 64;
    a.k_tasks = c->n_heads * 2 * dq;
    a.v_tasks = (c->n_heads * 8 * dq + 15) / 16 * 4;
    a.tasks = a.k_tasks + a.v_tasks + (turn.table ? (turn.n_q_heads * 8 * dq + 15) / 16 * 4 : 0);
    const dim3 grid(unsigned((a.tasks + 3) / 4), unsigned(T_ / kRows4 < 65535 ? (T_ + kRows4 - 1) / kRows4 : 65535));
    if (dq == 1) launch_append4<1, T>(a, grid, s);
    else if (dq == 2) launch_append4<2, T>(a, grid, s);
    else if (dq == 3) launch_append4<3, T>(a, grid, s);
    else launch_append4<4, T>(a, grid, s);
}

template <class T>
void gather4(const mbd_kv_cache* c, const int32_t* slots, int32_t n, void* k_out, void* v_out, hipStream_t s) {
    const Cache4Args a = cache4_args(c, slots, n);
    T *k = static_cast<T*>(k_out), *v = static_cast<T*>(v_out);
    const int dq = c->head_dim / 64, per = 16 * kGather4;
    const dim3 grid(unsigned((c->n_heads * 8 * dq + 15) / 16), unsigned(n / per < 65535 ? (n + per - 1) / per : 65535));
    if (dq == 1) hipLaunchKernelGGL((gather4_kernel<1, T>), grid, dim3(256), 0, s, a, k, v);
    else if (dq == 2) hipLaunchKernelGGL((gather4_kernel<2, T>), grid, dim3(256), 0, s, a, k, v);
    else if (dq == 3) hipLaunchKernelGGL((gather4_kernel<3, T>), grid, dim3(256), 0, s, a, k, v);
    else hipLaunchKernelGGL((gather4_kernel<4, T>), grid, dim3(256), 0, s, a, k, v);
}

}  // namespace kv
}  // namespace mbd
