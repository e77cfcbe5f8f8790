// Append to and read-back of the 4-bit KV cache (MBD_KV_MXFP4).
//
// A token's codes depend on that token alone, so there is nothing to share between its rows: a
// lane takes eight channels of one token (an octet), four lanes a group of 32, whose maximum
// gives the exponent.  What costs is where the bytes lie: a tile of 16 tokens keeps a token's codes
// in pieces of 16 bytes (keys) and 4 (values).  A wave takes 8 tokens x 8 octets: a line of 64 bf16
// channels in, and where the tokens follow each other in a tile whole lines of codes out; and the same of
// several heads one after the other, which are turned by the same angles.
// Prompts of 19.5k tokens (32 + 8 heads x 128, bf16, turned: 250 MB in, 181 out) take 86 us, 5.0 TB/s, the rate of a copy;
// one token 4.5, which is a launch and a chain of four loads (position, angles and keys, slot).  Without rotation the prompts' keys
// and values, 101 MB, take 23.9 us, 4.2 TB/s, from fp32, 181 MB, 43.6; one token 3.2.
#pragma once

#include <hip/hip_runtime.h>

#include "kv_turn.h"

namespace mbd {
namespace kv {

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
        if (halved(d)) return at + t / 4 * 128 + d % 64 / 4 * 8 + t % 4 * 2 + d % 4 / 2;
        return at + t / 4 * 256 + d % 128 / 8 * 16 + t % 4 * 4 + d % 8 / 2;
    }
};

struct Append4Args {
    Cache4Args c;
    const void* x[2];
    int64_t stride[2];
    int32_t heads;                       // of one wave's task
    int32_t kv_tasks, tasks;             // of the keys, as many of the values; and all
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
    const int side = task < a.kv_tasks ? 0 : TURN && task >= 2 * a.kv_tasks ? 2 : 1;     // keys, values, queries
    const int mine = task - side * a.kv_tasks, d = mine % DQ * 64 + (lane & 7) * 8;
    const int h0 = mine / DQ * a.heads, h1 = min(h0 + a.heads, side == 2 ? a.turn.n_q_heads : a.c.n_heads);
    const bool turns = TURN && side != 1;
    const T* rows = static_cast<const T*>(side == 2 ? a.turn.q : a.x[side & 1]);
    const int64_t stride = side == 2 ? a.turn.q_stride : a.stride[side & 1];
    for (int64_t w0 = int64_t(blockIdx.y) * kTurnRows; w0 < a.c.T; w0 += int64_t(gridDim.y) * kTurnRows) {
        const int64_t token = w0 + (lane >> 3);
        if (token >= a.c.T) continue;
        const T* from = rows + token * stride;
        Angles a0, a1;
        if constexpr (TURN) {
            const int32_t p = a.turn.positions[token];
            if (p < 0 || p >= a.turn.n_positions) continue;
            a0.partner = a1.partner = -1;
            if (turns) {
                const float* row = a.turn.table + int64_t(p) * a.turn.rot;
                a0.load(a.turn, row, d);
                a1.load(a.turn, row, d + 4);
            }
        }
        const int32_t slot = side == 2 ? 0 : a.c.slots[token];
        if (slot < 0 || slot >= a.c.n_slots) continue;
        auto put = [&](int h, const f32x4 x0, const f32x4 x1) {
            if (TURN && side == 2) return store_query(a.turn, token, int64_t(h) * D + d, x0, x1);
            int e;
            const uint32_t codes = encode4(x0, x1, &e);
            const Place4<DQ> at(a.c, slot, h);
            uint8_t* to = a.c.codes[side & 1] + (side ? at.value(d) : at.key(d));
            if ((lane & 3) == 0) a.c.scales[side & 1][at.scale(d)] = uint8_t(e);
            if (side && Place4<DQ>::halved(d)) {
                *reinterpret_cast<uint16_t*>(to) = uint16_t(codes);
                *reinterpret_cast<uint16_t*>(to + 8) = uint16_t(codes >> 16);
            } else {
                *reinterpret_cast<uint32_t*>(to) = codes;
            }
        };
        each_head<TURN>(a.turn, from, d, D, h0, h1, a0, a1, put);
    }
}

constexpr int kGather4 = 4;              // tokens of one thread

// A thread writes 16 bytes (8 bf16 or 4 fp32 channels), a wave 4 tokens x 256 bytes of keys and as much of values;
// a line of codes, which holds 8 tokens of one group or 4 of 64 channels, is read by this workgroup alone.
// The outputs are not read again here: streamed past the caches.
// 32768 tokens x 8 heads x 128 to bf16 (36 MB in, 134 out): 26.1 us, 6.5 TB/s; to fp32 19.7k tokens 33.7, 5.4 TB/s.
template <int DQ, class T>
__global__ __launch_bounds__(256) void gather4_kernel(Cache4Args a, T* k_out, T* v_out) {
    constexpr int D = 64 * DQ, C = 16 / sizeof(T);
    const int row = threadIdx.x >> 4, unit = blockIdx.x * 16 + (threadIdx.x & 15), units = a.n_heads * (D / C);
    if (unit >= units) return;
    const int head = unit / (D / C), d = (unit - head * (D / C)) * C;
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
                const uint8_t *k = a.codes[0] + at.key(d), *v = a.codes[1] + at.value(d);
                if constexpr (C == 4) {
                    kw[i] = *reinterpret_cast<const uint16_t*>(k);
                    vw[i] = *reinterpret_cast<const uint16_t*>(v);
                } else {
                    kw[i] = *reinterpret_cast<const uint32_t*>(k);
                    if (Place4<DQ>::halved(d)) vw[i] = *reinterpret_cast<const uint16_t*>(v) | uint32_t(*reinterpret_cast<const uint16_t*>(v + 8)) << 16;
                    else vw[i] = *reinterpret_cast<const uint32_t*>(v);
                }
                ke[i] = a.scales[0][at.scale(d)];
                ve[i] = a.scales[1][at.scale(d)];
            }
#pragma unroll
        for (int i = 0; i < kGather4; ++i)
            if (slot[i] >= 0) {
                const int64_t to = (w0 + 16 * i + row) * (int64_t(a.n_heads) * D) + int64_t(unit) * C;
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    const uint32_t w = side ? vw[i] : kw[i];
                    const float s = __uint_as_float((side ? ve[i] : ke[i]) << 23);
                    const f32x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
                    u32x4 r;
                    if constexpr (C == 4) {
                        r = __builtin_bit_cast(u32x4, f32x4{p0[0], p0[1], p1[0], p1[1]});
                    } else {
                        const f32x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
                        r = u32x4{pack_bf16(p0[0], p0[1]), pack_bf16(p1[0], p1[1]), pack_bf16(p2[0], p2[1]), pack_bf16(p3[0], p3[1])};
                    }
                    __builtin_nontemporal_store(r, reinterpret_cast<u32x4*>((side ? v_out : k_out) + to));
                }
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
    const int dq = c->head_dim / 64;
    const int64_t windows = (int64_t(T_) + kTurnRows - 1) / kTurnRows;
    // heads of a task: as many as leave 4096 waves
    int heads = 1;
    while (heads < 8 && windows * dq * (2 * int64_t(c->n_heads) + turn.n_q_heads) / (2 * heads) >= 4096) heads *= 2;
    const int kv_tasks = (c->n_heads + heads - 1) / heads * dq, q_tasks = turn.table ? (turn.n_q_heads + heads - 1) / heads * dq : 0;
    const Append4Args a{cache4_args(c, slots, T_), {k, v}, {k_stride, v_stride}, heads, kv_tasks, 2 * kv_tasks + q_tasks, turn};
    const dim3 grid(unsigned((a.tasks + 3) / 4), unsigned(windows < 65535 ? windows : 65535));
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
    const dim3 grid(unsigned((int64_t(c->n_heads) * 64 * dq * int64_t(sizeof(T)) / 16 + 15) / 16), unsigned(n / per < 65535 ? (n + per - 1) / per : 65535));
    if (dq == 1) hipLaunchKernelGGL((gather4_kernel<1, T>), grid, dim3(256), 0, s, a, k, v);
    else if (dq == 2) hipLaunchKernelGGL((gather4_kernel<2, T>), grid, dim3(256), 0, s, a, k, v);
    else if (dq == 3) hipLaunchKernelGGL((gather4_kernel<3, T>), grid, dim3(256), 0, s, a, k, v);
    else hipLaunchKernelGGL((gather4_kernel<4, T>), grid, dim3(256), 0, s, a, k, v);
}

}  // namespace kv
}  // namespace mbd
