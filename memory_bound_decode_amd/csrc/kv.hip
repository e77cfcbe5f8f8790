// The paged 8-bit KV cache around its attention: block tables and slot maps from
// request lengths, the append that quantises new keys and values, and the read-back.
// A decode step's time is the bytes that it reads ([Bolt] background); beside the
// weights those are the cached keys and values, halved here against bf16.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv_common.h"

namespace mbd {
namespace kv {

// ---------------------------------------------------------------- slots

constexpr int kSlotThreads = 1024;
constexpr int kPer = kMaxSeqs / kSlotThreads;   // requests of one thread, neighbours

struct SlotArgs {
    const int32_t *add, *lens, *held, *n_free;
    int32_t *table, *free_blocks;
    int32_t *seq_start, *slots, *positions, *lens_out, *held_out, *n_free_out, *status;
    int32_t n, shift, max_blocks, n_blocks, T;
    bool map_here;
};

// Exclusive sums of two values over the workgroup's threads, and the totals.
struct Sums { int64_t u, v, all_u, all_v; };

__device__ __forceinline__ Sums block_scan(int64_t u, int64_t v, int64_t (*wave_sums)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    int64_t iu = u, iv = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t pu = __shfl_up(iu, d), pv = __shfl_up(iv, d);
        if (lane >= d) { iu += pu; iv += pv; }
    }
    if (lane == 63) { wave_sums[wave][0] = iu; wave_sums[wave][1] = iv; }
    __syncthreads();
    Sums s{iu - u, iv - v, 0, 0};
    for (int w = 0; w < waves; ++w) {
        const int64_t wu = wave_sums[w][0], wv = wave_sums[w][1];
        if (w < wave) { s.u += wu; s.v += wv; }
        s.all_u += wu;
        s.all_v += wv;
    }
    return s;
}

// The last i in [0, n] with start[i] <= x; start[0] <= x, start does not fall.
__device__ __forceinline__ int owner(const int32_t* start, int n, int32_t x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int32_t capped(int64_t v) { return v > 0x7fffffff ? 0x7fffffff : int32_t(v); }

constexpr int kMapTokens = 1024;   // of one workgroup of slot_map_kernel
constexpr int kBatch = 4;

__device__ __forceinline__ void map_token(const SlotArgs& a, const int32_t* start, const int32_t* from, int32_t e) {
    const int i = owner(start, a.n, e);
    int32_t slot = -1, pos = -1;
    if (i < a.n && from[i] >= 0) {
        pos = from[i] + (e - start[i]);
        const int32_t id = a.table[int64_t(i) * a.max_blocks + (pos >> a.shift)];
        if (id >= 0 && id < a.n_blocks) slot = (id << a.shift) + (pos & ((1 << a.shift) - 1));
    }
    a.slots[e] = slot;
    if (a.positions) a.positions[e] = pos;
}

// One workgroup: every request's place in the step's token batch, in the blocks that
// come back and in the blocks that are taken is a prefix sum over the requests; the
// entries behind each sum are then written flat over the threads, each finding its
// request by bisection of the sums in LDS.  A decode step's work is a few KB, so the time
// is that of the dependent loads (lengths, free stack, tables) and of two scans: 4.6 us for 32
// requests.  250 requests with 30 prompts (66k tokens, 4k new blocks) take 10.7 us, and 6.0 more
// for their slot map over the chip, which one workgroup would write in 50.
__global__ __launch_bounds__(kSlotThreads) void slots_kernel(SlotArgs a) {
    __shared__ int64_t sums[2][kSlotThreads / 64][2];
    __shared__ int32_t start[kMaxSeqs + 1], back_at[kMaxSeqs + 1], take_at[kMaxSeqs + 1];
    __shared__ int32_t from[kMaxSeqs];       // position of the first new token, -1: not served
    __shared__ int32_t first_new[kMaxSeqs];  // the first column that is not held
    __shared__ int32_t taken_all;
    const int t = threadIdx.x, n = a.n;
    const int per = (n + int(blockDim.x) - 1) / int(blockDim.x);
    const int bs = 1 << a.shift;
    int32_t add[kPer], len[kPer], held[kPer], st[kPer];
    int64_t want[kPer], my_add = 0, my_back = 0;
    if (t == 0) taken_all = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = t * per + j;
        add[j] = len[j] = held[j] = st[j] = 0;
        want[j] = 0;
        if (j < per && i < n) {
            add[j] = a.add[i];
            len[j] = a.lens[i];
            held[j] = a.held[i];
            if (len[j] < 0 || held[j] < 0 || held[j] > a.max_blocks || len[j] > (int64_t(held[j]) << a.shift)) st[j] = 4;
            if (add[j] > 0) my_add += add[j];
            if (add[j] < 0 && st[j] == 0) my_back += held[j];
        }
    }
    const int32_t n_free = min(max(*a.n_free, 0), a.n_blocks);
    const Sums of_add = block_scan(my_add, my_back, sums[0]);
    const int64_t all_add = of_add.all_u, all_back = of_add.all_v;
    int64_t at_add = of_add.u, at_back = of_add.v;
    const int64_t top = min(n_free + all_back, int64_t(a.n_blocks));
    int64_t my_need = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = t * per + j;
        if (j < per && i < n) {
            start[i] = int32_t(min(at_add, int64_t(a.T)));
            back_at[i] = capped(at_back);
            if (add[j] > 0) {
                at_add += add[j];
                const int64_t blocks = (int64_t(len[j]) + add[j] + bs - 1) >> a.shift;
                if (st[j] == 0) st[j] = blocks > a.max_blocks ? 2 : at_add > a.T ? 3 : 0;
                if (st[j] == 0 && blocks > held[j]) want[j] = blocks - held[j];
                my_need += want[j];
            } else if (add[j] < 0 && st[j] == 0) {
                at_back += held[j];
            }
        }
    }
    const Sums of_need = block_scan(my_need, 0, sums[1]);
    const int64_t all_need = of_need.all_u;
    int64_t at_need = of_need.u;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = t * per + j;
        if (j < per && i < n) {
            take_at[i] = capped(at_need);
            at_need += want[j];
            if (want[j] > 0 && at_need > top) { st[j] = 1; want[j] = 0; }
            if (want[j] > 0) atomicMax(&taken_all, int32_t(at_need));
            const bool ended = add[j] < 0 && st[j] == 0;
            from[i] = add[j] > 0 && st[j] == 0 ? len[j] : -1;
            first_new[i] = held[j];
            a.status[i] = st[j];
            a.lens_out[i] = ended ? 0 : st[j] == 0 ? len[j] + max(add[j], 0) : len[j];
            a.held_out[i] = ended ? 0 : held[j] + int32_t(want[j]);
            a.seq_start[i] = start[i];
        }
    }
    if (t == 0) {
        start[n] = int32_t(min(all_add, int64_t(a.T)));
        back_at[n] = capped(all_back);
        take_at[n] = capped(all_need);
        a.seq_start[n] = start[n];
    }
    __syncthreads();
    const int32_t taken = taken_all;
    if (t == 0) *a.n_free_out = int32_t(top) - taken;
    // Entries behind the sums, a batch of each thread's at a time: their reads are in flight together.
    const int32_t step = blockDim.x;
    for (int32_t e0 = t; e0 < int32_t(top) - n_free; e0 += kBatch * step) {
        int32_t id[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t e = e0 + k * step;
            if (e < int32_t(top) - n_free) {
                const int i = owner(back_at, n, e);
                id[k] = a.table[int64_t(i) * a.max_blocks + (e - back_at[i])];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (e0 + k * step < int32_t(top) - n_free) a.free_blocks[n_free + e0 + k * step] = id[k];
    }
    __syncthreads();
    for (int32_t e0 = t; e0 < taken; e0 += kBatch * step) {
        int32_t id[kBatch];
        int64_t to[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t e = e0 + k * step;
            if (e < taken) {
                id[k] = a.free_blocks[int32_t(top) - 1 - e];
                const int i = owner(take_at, n, e);
                to[k] = int64_t(i) * a.max_blocks + first_new[i] + (e - take_at[i]);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (e0 + k * step < taken) a.table[to[k]] = id[k];
    }
    __syncthreads();
    if (!a.map_here) return;
    for (int32_t e = t; e < a.T; e += blockDim.x) map_token(a, start, from, e);
}

// The slot map of many tokens, over the chip: the first kernel's outputs, in LDS.
__global__ __launch_bounds__(256) void slot_map_kernel(SlotArgs a) {
    __shared__ int32_t start[kMaxSeqs + 1], from[kMaxSeqs];
    for (int i = threadIdx.x; i <= a.n; i += 256) {
        start[i] = a.seq_start[i];
        if (i < a.n) {                   // a served request's tokens end at its new length
            const int32_t count = a.seq_start[i + 1] - a.seq_start[i];
            from[i] = count > 0 && a.status[i] == 0 ? a.lens_out[i] - count : -1;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMapTokens / 256; ++k) {
        const int64_t e = int64_t(blockIdx.x) * kMapTokens + 256 * k + threadIdx.x;
        if (e < a.T) map_token(a, start, from, int32_t(e));
    }
}

// ---------------------------------------------------------------- append

struct AppendArgs {
    uint8_t* codes[2];
    float* scales[2];
    const void* x[2];
    int64_t stride[2];
    const int32_t* slots;
    int32_t n_slots;      // slots of the cache
    int32_t T, window, n_heads, head_dim, shift;
};

template <bool E4M3>
__device__ __forceinline__ float wanted_scale(float amax) {
    if (!(amax > 0.f)) return 0.f;
    if constexpr (E4M3) {
        int e;
        const float f = frexpf(amax, &e);          // 448 = 0.875 * 2^9
        return ldexpf(1.f, max(e - (f <= 0.875f ? 9 : 8), -126));
    }
    return amax * (1.0f / 127.0f);
}

// Four scaled values as one word of codes; any values.
template <bool E4M3>
__device__ __forceinline__ uint32_t encode(const float v[4]) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float lim = E4M3 ? 448.f : 127.f;
        c[i] = v[i] == v[i] ? fminf(fmaxf(v[i], -lim), lim) : 0.f;
    }
    if constexpr (E4M3) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true));
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= (uint32_t(int32_t(rintf(c[i]))) & 255u) << (8 * i);
    return w;
}

// Sixteen values x over a scale, as the codes of one unit.  r is the scale's reciprocal,
// correctly rounded.  E4M3: where the scale is a power of two, the product is the quotient.  INT8:
// Markstein's theorem (IBM J. Res. Dev. 34, 1990): for such an r and a q within an ulp of
// x / s, q + r (x - q s) with fused operations rounds correctly; three operations where a
// division without r takes ten and more.  Adding 1.5 * 2^23 then rounds to a whole number,
// ties to even, whose low byte is the code.  (The bare product x r will not do: a value of half
// the block's maximum is a tie, 63.5, which is found in two of three waves.)
template <bool E4M3>
__device__ __forceinline__ u32x4 encode_unit(const float x[16], float div, float r, bool any_values) {
    u32x4 w;
    if (!any_values) {
        if constexpr (E4M3) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * q] * r, x[4 * q + 1] * r, 0, false);
                w[q] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(x[4 * q + 2] * r, x[4 * q + 3] * r, lo, true));
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v = x[4 * q + i], near = v * r;
                    c[i] = __float_as_uint(__builtin_fmaf(__builtin_fmaf(-near, div, v), r, near) + 12582912.f);
                }
                w[q] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400), __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400), 0x05040100);
            }
        }
        return w;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float v[4] = {x[4 * q] / div, x[4 * q + 1] / div, x[4 * q + 2] / div, x[4 * q + 3] / div};
        w[q] = encode<E4M3>(v);
    }
    return w;
}

template <bool E4M3>
__device__ __forceinline__ u32x4 rescale_unit(const u32x4 w, float ratio) {
    u32x4 res;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float v[4] = {code_value<E4M3, 0>(w[q]) * ratio, code_value<E4M3, 1>(w[q]) * ratio, code_value<E4M3, 2>(w[q]) * ratio,
                            code_value<E4M3, 3>(w[q]) * ratio};
        res[q] = encode<E4M3>(v);
    }
    return res;
}

// Four neighbouring channels of one token, as loaded.
template <class T> struct Quad;
template <> struct Quad<float> {
    f32x4 v;
    __device__ void load(const float* p) { v = *reinterpret_cast<const f32x4*>(p); }
    __device__ void clear() { v = f32x4{0.f, 0.f, 0.f, 0.f}; }
    __device__ float at(int j) const { return v[j]; }
    // the largest |bits|: above every finite value's where one is infinite or NaN
    typedef uint32_t Top;
    static __device__ uint32_t bits(Top t) { return t; }
    __device__ void raise(Top& t) const {
        const u32x4 b = __builtin_bit_cast(u32x4, v) & 0x7fffffffu;
        t = max(max(t, max(b.x, b.y)), max(b.z, b.w));
    }
};
template <> struct Quad<uint16_t> {
    u32x2 v;
    __device__ void load(const uint16_t* p) { v = *reinterpret_cast<const u32x2*>(p); }
    __device__ void clear() { v = u32x2{0, 0}; }
    __device__ float at(int j) const { return __uint_as_float(j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16); }
    typedef uint16_t Top __attribute__((ext_vector_type(2)));
    static __device__ uint32_t bits(Top t) { return uint32_t(max(t.x, t.y)) << 16; }
    __device__ void raise(Top& t) const {
        t = __builtin_elementwise_max(t, __builtin_bit_cast(Top, v.x & 0x7fff7fffu));
        t = __builtin_elementwise_max(t, __builtin_bit_cast(Top, v.y & 0x7fff7fffu));
    }
};

// The tokens of one block that the call brings, places [fill, end), for one head's keys
// or values, by THREADS threads (a wave, or a workgroup of 256), each with KEEP units in
// registers between the maximum and the codes (more are read again).  A unit is 16
// bytes of a code tile: lane (g, m) of slab s holds, of a key tile, token m and channels
// 64s + 16g .. +16; of a value tile, tokens 4g .. +4 and channels 64s + 4m .. +4.
template <bool E4M3, bool V, class T, int THREADS, int KEEP>
__device__ __forceinline__ void append_run(const AppendArgs& a, int32_t token, int64_t block, int fill, int end, int head, uint32_t* lds) {
    const int tid = THREADS == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, m = lane & 15;
    const int D = a.head_dim, slabs = D / 64;
    const int64_t bh = block * a.n_heads + head;
    uint8_t* codes = a.codes[V] + ((bh * D) << a.shift);
    const int64_t stride = a.stride[V];
    const T* row0 = static_cast<const T*>(a.x[V]) + int64_t(token) * stride + int64_t(head) * D;
    const float old_scale = fill > 0 ? a.scales[V][bh] : 0.f;
    const int tile0 = fill / kTok, chunks = ((end - 1) / kTok + 1 - tile0) * slabs;   // 64 units each

    Quad<T> x[KEEP][4];
    u32x4 old[THREADS == 64 ? KEEP : 1];
    auto first_token = [&](int tile) { return tile * kTok + (V ? 4 * g : m); };
    auto unit_at = [&](int tile, int s) { return reinterpret_cast<u32x4*>(codes + int64_t(tile) * kTok * D + s * 1024 + lane * 16); };
    auto all_new = [&](int tile) { return tile * kTok >= fill && (tile + 1) * kTok <= end; };     // in every lane
    // a unit that also holds tokens of before, or bytes behind the last
    auto boundary = [&](bool in, int tile, int s) {
        const int first = first_token(tile);
        u32x4 w = {0, 0, 0, 0};
        if (in && first < end && (first < fill || (V && first + 4 > end))) w = *unit_at(tile, s);
        return w;
    };
    auto load = [&](int c0) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int c = c0 + i * (THREADS / 64) + wave;
            const int tile = tile0 + c / slabs, s = c % slabs, first = first_token(tile);
            const T* from = row0 + (first - fill) * stride + 64 * s + (V ? 4 * m : 16 * g);
            if (c < chunks && all_new(tile)) {
#pragma unroll
                for (int k = 0; k < 4; ++k) x[i][k].load(from + (V ? k * stride : 4 * k));
                continue;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tok = V ? first + k : first;
                x[i][k].clear();
                if (c < chunks && tok >= fill && tok < end) x[i][k].load(from + (V ? k * stride : 4 * k));
            }
            if constexpr (THREADS == 64) old[i] = boundary(c < chunks, tile, s);   // early: few waves, so latency counts
        }
    };
    constexpr int round = KEEP * (THREADS / 64);
    const bool once = chunks <= round;
    typename Quad<T>::Top most{};
    for (int c0 = 0; c0 < chunks; c0 += round) {
        load(c0);
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k].raise(most);
    }
    auto reduce = [&](uint32_t v) {
#pragma unroll
        for (int d = 32; d; d >>= 1) v = max(v, uint32_t(__shfl_xor(int(v), d)));
        if constexpr (THREADS > 64) {
            __syncthreads();
            if (lane == 0) lds[wave] = v;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < THREADS / 64; ++w) v = max(v, lds[w]);
        }
        return uint32_t(__builtin_amdgcn_readfirstlane(int(v)));
    };
    uint32_t top = reduce(Quad<T>::bits(most));
    const bool finite = top < 0x7f800000u;
    if (!finite) {                       // the largest of the finite values
        top = 0;
        for (int c0 = 0; c0 < chunks; c0 += round) {
            load(c0);
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t b = __float_as_uint(x[i][k].at(j)) & 0x7fffffffu;
                        if (b < 0x7f800000u) top = max(top, b);
                    }
        }
        top = reduce(top);
    }
    const float wanted = wanted_scale<E4M3>(__uint_as_float(top));
    const bool grew = wanted > old_scale;
    const float now = grew ? wanted : old_scale, div = now > 0.f ? now : 1.f;
    const float r = 1.f / div, ratio = old_scale / div;
    // a smaller scale's remainders lose bits; an e4m3 scale of a cache filled elsewhere may be no power of two
    const bool any_values = !finite || !(div >= 0x1p-100f) || (E4M3 && (__float_as_uint(div) & 0x7fffffu));
    if (tid == 0 && (grew || fill == 0)) a.scales[V][bh] = now;
    for (int c0 = 0; c0 < chunks; c0 += round) {
        if (!once) load(c0);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            const int c = c0 + i * (THREADS / 64) + wave;
            if (c >= chunks) break;
            const int tile = tile0 + c / slabs, s = c % slabs, first = first_token(tile);
            float v[16];
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) v[V ? 4 * j + k : 4 * k + j] = x[i][k].at(j);
            const u32x4 fresh = encode_unit<E4M3>(v, div, r, any_values);
            if (all_new(tile)) {
                *unit_at(tile, s) = fresh;
                continue;
            }
            if (first >= end || (!grew && first + (V ? 4 : 1) <= fill)) continue;
            uint32_t mask = 0;           // bytes of a word whose tokens are new
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tok = V ? first + k : first;
                if (tok >= fill && tok < end) mask |= 255u << (8 * k);
            }
            u32x4 kept;
            if constexpr (THREADS == 64) kept = old[i];
            else kept = boundary(true, tile, s);
            if (grew && fill > 0) kept = rescale_unit<E4M3>(kept, ratio);
            *unit_at(tile, s) = (fresh & mask) | (kept & ~mask);
        }
    }
    if (grew)                            // tiles that hold old tokens alone
        for (int c = wave; c < tile0 * slabs; c += THREADS / 64) {
            u32x4* unit = unit_at(c / slabs, c % slabs);
            *unit = rescale_unit<E4M3>(*unit, ratio);
        }
}

// What a wave sees of the slots from token t0 on: lane l holds token t0 + l's; a bit of
// `starts` is a token that begins a run, of `more[0]`, `more[1]` one of the first 128 that
// goes on with its predecessor's run (the next place of the same block).
struct Look {
    int32_t slot;
    uint64_t starts, more[2];
};

__device__ __forceinline__ Look look_at(const AppendArgs& a, int32_t t0) {
    const int lane = threadIdx.x & 63, in_block = (1 << a.shift) - 1;
    int32_t slot[2], prev[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t t = t0 + 64 * h + lane;
        slot[h] = t < a.T ? a.slots[t] : -1;
        prev[h] = t < a.T && t > 0 ? a.slots[t - 1] : -2;
    }
    Look k;
    k.slot = slot[0];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool good = slot[h] >= 0 && slot[h] < a.n_slots, goes_on = good && prev[h] == slot[h] - 1 && (slot[h] & in_block) != 0;
        k.more[h] = __ballot(goes_on);
        if (h == 0) k.starts = __ballot(good && !goes_on && lane < a.window);
    }
    return k;
}

// Tokens of the run that begins at bit l, `first` its slot.
__device__ __forceinline__ int run_length(const AppendArgs& a, const Look& k, int32_t t0, int l, int32_t first) {
    const uint64_t rest = l < 63 ? k.more[0] >> (l + 1) : 0;
    int count = 1 + __builtin_ctzll(~rest);            // a shift leaves a zero at the top
    if (count < 64 - l) return count;
    count = 64 - l + (~k.more[1] ? __builtin_ctzll(~k.more[1]) : 64);
    if (count < 128 - l) return count;
    const int lane = threadIdx.x & 63, most = (1 << a.shift) - (first & ((1 << a.shift) - 1));
    for (int at = count; at < most; at += 64) {        // a long run of a large block
        const int i = at + lane;
        const uint64_t off = ~__ballot(i < most && t0 + l + i < a.T && a.slots[t0 + l + i] == first + i);
        count = at + (off ? __builtin_ctzll(off) : 64);
        if (off) break;
    }
    return count;
}

// Few tokens: a wave for each (token, head, keys or values), busy where the token begins
// a run.  The waves of a workgroup take neighbouring heads, which lie side by side.  Bound by
// its chain of loads (slots -> values, old codes, scale): one token 5.2 us, a verify step of 48
// requests x 0..9 tokens (fp32, 236 rows) 7.7 us.
template <bool E4M3, class T>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    const int hw = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (hw >= 2 * a.n_heads) return;
    const int head = hw % a.n_heads;
    const int32_t t0 = int32_t(blockIdx.y);
    const Look k = look_at(a, t0);
    if (!k.starts) return;
    const int32_t first = __builtin_amdgcn_readfirstlane(k.slot);
    const int fill = first & ((1 << a.shift) - 1), end = fill + run_length(a, k, t0, 0, first);
    if (hw >= a.n_heads) append_run<E4M3, true, T, 64, 4>(a, t0, first >> a.shift, fill, end, head, nullptr);
    else append_run<E4M3, false, T, 64, 4>(a, t0, first >> a.shift, fill, end, head, nullptr);
}

// Many tokens: a workgroup for each (window of tokens, head, keys or values).  Long runs
// are taken by the whole workgroup, so that prompts are read once and all their loads are
// in flight together; short ones (a wave's units at most) by one wave each.  13 prompts of
// 19.5k tokens (8 heads x 128, bf16 to int8, 120 MB) take 33.6 us, 3.6 TB/s, from fp32 (200 MB) 48.6
// us, 4.1 TB/s: the vector units work 42% of that, the rest is the chain of a workgroup's loads.
template <bool E4M3, class T>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 ? 6 : 4))) void append_window_kernel(AppendArgs a) {
    __shared__ uint32_t lds[4];
    constexpr int kept = 2;            // fewer registers, more workgroups in flight
    const int wave = threadIdx.x >> 6;
    const int head = blockIdx.x % uint32_t(a.n_heads);
    const bool values = int(blockIdx.x) >= a.n_heads;
    for (int64_t at = int64_t(blockIdx.y) * a.window; at < a.T; at += int64_t(gridDim.y) * a.window) {
        const int32_t t0 = int32_t(at);
        const Look k = look_at(a, t0);                     // the same in every wave
        uint64_t todo = k.starts;
        for (int turn = 0; todo; ++turn) {
            const int l = __builtin_ctzll(todo);
            todo &= todo - 1;
            const int32_t first = __builtin_amdgcn_readlane(k.slot, l), token = t0 + l;
            const int fill = first & ((1 << a.shift) - 1), end = fill + run_length(a, k, t0, l, first);
            if (((end - 1) / kTok + 1 - fill / kTok) * a.head_dim > 64 * kept) {
                if (values) append_run<E4M3, true, T, 256, kept>(a, token, first >> a.shift, fill, end, head, lds);
                else append_run<E4M3, false, T, 256, kept>(a, token, first >> a.shift, fill, end, head, lds);
            } else if (turn % 4 == wave) {
                if (values) append_run<E4M3, true, T, 64, kept>(a, token, first >> a.shift, fill, end, head, nullptr);
                else append_run<E4M3, false, T, 64, kept>(a, token, first >> a.shift, fill, end, head, nullptr);
            }
        }
    }
}

// ---------------------------------------------------------------- gather

struct GatherArgs {
    const uint8_t* codes[2];
    const float* scales[2];
    void* out[2];
    const int32_t* slots;
    int32_t n_slots, T, n_heads, head_dim, shift;
};

__device__ __forceinline__ void store4(float* p, const f32x4 v) { __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(p)); }
__device__ __forceinline__ void store4(uint16_t* p, const f32x4 v) {
    __builtin_nontemporal_store(u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, reinterpret_cast<u32x2*>(p));
}

constexpr int kGatherTokens = 4;   // tokens of one thread

// A thread writes four neighbouring channels, so that a workgroup's stores are whole rows of a
// head, and neighbouring workgroups take a token's other heads: the outputs fill front to back
// (32768 tokens of 8 heads x 128 to fp32, 336 MB, four fifths of it writes, in 49 us, 6.9 TB/s, what a
// plain fill reaches; to bf16, 201 MB, 31 us; with the tokens of one head side by side 63-75 for
// 49).  They are not read again here: streamed past the caches (77 us if kept).
// The four tokens of a value word are read by four threads: the repeats hit L1.
template <bool E4M3, class T>
__global__ __launch_bounds__(256) void gather_kernel(GatherArgs a) {
    const int quads = a.head_dim / 4, rows = 256 / quads;
    const int row = threadIdx.x / quads, quad = threadIdx.x - row * quads;
    if (row >= rows) return;
    const int head = blockIdx.x, D = a.head_dim;
    for (int64_t group = blockIdx.y; group * rows * kGatherTokens < a.T; group += gridDim.y) {
        const int32_t t0 = int32_t(group) * rows * kGatherTokens + row;
        int32_t slot[kGatherTokens];
        uint32_t kw[kGatherTokens];
        u32x4 vw[kGatherTokens];
        float ks[kGatherTokens], vs[kGatherTokens];
#pragma unroll
        for (int i = 0; i < kGatherTokens; ++i) {
            const int32_t t = t0 + i * rows;
            slot[i] = t < a.T ? a.slots[t] : -1;
            if (slot[i] >= a.n_slots) slot[i] = -1;
        }
        const int slab = quad / 16, m = quad % 16;
#pragma unroll
        for (int i = 0; i < kGatherTokens; ++i)
            if (slot[i] >= 0) {
                const int64_t bh = int64_t(slot[i] >> a.shift) * a.n_heads + head;
                const int place = slot[i] & ((1 << a.shift) - 1), tok = place % kTok;
                const int64_t tile = ((bh * D) << a.shift) + int64_t(place / kTok) * kTok * D + slab * 1024;
                kw[i] = *reinterpret_cast<const uint32_t*>(a.codes[0] + tile + (m / 4) * 256 + tok * 16 + (m % 4) * 4);
                vw[i] = *reinterpret_cast<const u32x4*>(a.codes[1] + tile + (tok / 4) * 256 + m * 16);
                ks[i] = a.scales[0][bh];
                vs[i] = a.scales[1][bh];
            }
#pragma unroll
        for (int i = 0; i < kGatherTokens; ++i)
            if (slot[i] >= 0) {
                const int64_t at = (int64_t(t0 + i * rows) * a.n_heads + head) * D + quad * 4;
                const int sh = (slot[i] & 3) * 8;
                store4(static_cast<T*>(a.out[0]) + at, f32x4{code_value<E4M3, 0>(kw[i]) * ks[i], code_value<E4M3, 1>(kw[i]) * ks[i],
                                                             code_value<E4M3, 2>(kw[i]) * ks[i], code_value<E4M3, 3>(kw[i]) * ks[i]});
                f32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = code_value<E4M3, 0>(vw[i][j] >> sh) * vs[i];
                store4(static_cast<T*>(a.out[1]) + at, v);
            }
    }
}

// Host checks of the token-wise calls.
static mbd_status check_tokens(const void* k, const void* v, int32_t dtype, const int32_t* slots, int32_t T) {
    if (dtype != MBD_BF16 && dtype != MBD_F32) return fail(MBD_EINVAL, "unknown dtype %d", dtype);
    if (T < 0 || T > (1 << 24)) return fail(MBD_ESHAPE, "T %d outside [0, 2^24]", T);
    if (T == 0) return MBD_OK;
    if (!k || !v || !slots) return fail(MBD_EINVAL, "NULL argument");
    if (!aligned(k, 16) || !aligned(v, 16)) return fail(MBD_EALIGN, "keys and values must be 16-byte aligned");
    if (!aligned(slots, 4)) return fail(MBD_EALIGN, "slots must be 4-byte aligned");
    return MBD_OK;
}

}  // namespace kv
}  // namespace mbd

using namespace mbd;

extern "C" {

mbd_status mbd_kv_slots(const mbd_kv_pool* pool, const int32_t* new_tokens, const int32_t* lens, const int32_t* held,
                        const int32_t* n_free, int32_t T, int32_t* seq_start, int32_t* slots, int32_t* positions,
                        int32_t* lens_out, int32_t* held_out, int32_t* n_free_out, int32_t* status, void* stream) {
    hip_clear();
    if (!pool) return fail(MBD_EINVAL, "NULL pool");
    if (pool->n_seqs < 1 || pool->n_seqs > kv::kMaxSeqs) return fail(MBD_ESHAPE, "n_seqs %d outside [1, %d]", pool->n_seqs, kv::kMaxSeqs);
    if (!kv::block_size_ok(pool->block_size)) return fail(MBD_ESHAPE, "block_size %d is not 16, 32, 64, 128 or 256", pool->block_size);
    if (pool->max_blocks < 1) return fail(MBD_ESHAPE, "max_blocks %d below 1", pool->max_blocks);
    if (pool->n_blocks < 1 || int64_t(pool->n_blocks) * pool->block_size >= (int64_t(1) << 31))
        return fail(MBD_ESHAPE, "n_blocks * block_size outside [1, 2^31)");
    if (int64_t(pool->max_blocks) * pool->block_size >= (int64_t(1) << 31)) return fail(MBD_ESHAPE, "max_blocks * block_size is 2^31 or more");
    if (T < 0) return fail(MBD_ESHAPE, "T %d below 0", T);
    const void* every[] = {pool->block_table, pool->free_blocks, new_tokens, lens, held, n_free, seq_start, lens_out, held_out, n_free_out, status};
    for (const void* p : every) {
        if (!p) return fail(MBD_EINVAL, "NULL argument");
        if (!kv::aligned(p, 4)) return fail(MBD_EALIGN, "int32 arrays must be 4-byte aligned");
    }
    if (T > 0 && !slots) return fail(MBD_EINVAL, "NULL argument");
    if (!kv::aligned(slots, 4) || !kv::aligned(positions, 4)) return fail(MBD_EALIGN, "int32 arrays must be 4-byte aligned");
    kv::SlotArgs a{new_tokens, lens, held, n_free, pool->block_table, pool->free_blocks, seq_start, slots, positions, lens_out, held_out,
                   n_free_out, status, pool->n_seqs, kv::log2_of(pool->block_size), pool->max_blocks, pool->n_blocks, T,
                   T <= 8192};
    // Up to 8192 tokens the one workgroup writes the slot map in less time than a second launch takes:
    // 64 requests with 2168, 4281 and 8976 tokens 8.9, 10.2 and 13.3 us against 12.0, 12.1 and 12.1, two
    // with 6001 and 12001 8.6 and 10.8 against 9.8 and 9.9, 4000 that decode 30 against 46.
    // A step that decodes has few entries behind its sums: fewer waves meet at the barriers sooner
    // (32 requests 5.1 us, with 1024 threads 7.0; 64 with 525 tokens 7.7 either way, with 1228 9.0 and 8.3).
    const int threads = pool->n_seqs <= 256 && T <= 256 ? 256 : kv::kSlotThreads;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(kv::slots_kernel, dim3(1), dim3(threads), 0, s, a);
    if (!a.map_here)
        hipLaunchKernelGGL(kv::slot_map_kernel, dim3(unsigned((int64_t(T) + kv::kMapTokens - 1) / kv::kMapTokens)), dim3(256), 0, s, a);
    return hip_check("slots launch");
}

mbd_status mbd_kv_append(const mbd_kv_cache* cache, const void* k, const void* v, int32_t dtype, int64_t k_stride, int64_t v_stride,
                         const int32_t* slots, int32_t T, void* stream) {
    hip_clear();
    mbd_status st = kv::check_cache(cache, true);
    if (st == MBD_OK) st = kv::check_tokens(k, v, dtype, slots, T);
    if (st != MBD_OK) return st;
    const int64_t row = int64_t(cache->n_heads) * cache->head_dim;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return fail(MBD_ESHAPE, "token strides must be multiples of 8 and at least n_heads * head_dim");
    if (T == 0) return MBD_OK;
    // A wave a token up to 4096 waves: above, those that find no run cost more than windows do
    // (8 heads x 128, waves against windows: 256 requests x 1 token 17.8 and 21.3 us, 128 x 4 21.3 and
    // 15.2, 128 x 8 fp32 50 and 19, one prompt of 512 12.9 and 10.8).  A window takes the runs that begin in it,
    // so narrow ones start workgroups that find none; they widen down to 2048 workgroups: one prompt of
    // 4096 tokens 20.0 us, with 4096 of them 25.4; 512 requests x 8 46.0 and 45.3, with 1024 49.3.
    const int64_t waves = int64_t(T) * 2 * cache->n_heads;
    int32_t window = 1;
    while (window < 64 && waves / window > 2048) window *= 2;
    const bool few = waves <= 4096;
    if (few) window = 1;
    kv::AppendArgs a{{static_cast<uint8_t*>(cache->k_codes), static_cast<uint8_t*>(cache->v_codes)}, {cache->k_scale, cache->v_scale},
                     {k, v}, {k_stride, v_stride}, slots, int32_t(cache->n_blocks * cache->block_size), T, window, cache->n_heads,
                     cache->head_dim, kv::log2_of(cache->block_size)};
    const dim3 grid(unsigned(few ? (2 * cache->n_heads + 3) / 4 : 2 * cache->n_heads), unsigned(std::min((T + window - 1) / window, 65535)));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool wide = dtype == MBD_F32;
    const auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a); };
    if (cache->fmt == MBD_KV_E4M3) {
        if (few) wide ? run(kv::append_kernel<true, float>) : run(kv::append_kernel<true, uint16_t>);
        else wide ? run(kv::append_window_kernel<true, float>) : run(kv::append_window_kernel<true, uint16_t>);
    } else {
        if (few) wide ? run(kv::append_kernel<false, float>) : run(kv::append_kernel<false, uint16_t>);
        else wide ? run(kv::append_window_kernel<false, float>) : run(kv::append_window_kernel<false, uint16_t>);
    }
    return hip_check("append launch");
}

mbd_status mbd_kv_gather(const mbd_kv_cache* cache, const int32_t* slots, int32_t T, int32_t dtype, void* k_out, void* v_out,
                         void* stream) {
    hip_clear();
    mbd_status st = kv::check_cache(cache, true);
    if (st == MBD_OK) st = kv::check_tokens(k_out, v_out, dtype, slots, T);
    if (st != MBD_OK || T == 0) return st;
    kv::GatherArgs a{{static_cast<const uint8_t*>(cache->k_codes), static_cast<const uint8_t*>(cache->v_codes)},
                     {cache->k_scale, cache->v_scale}, {k_out, v_out}, slots, int32_t(cache->n_blocks * cache->block_size), T,
                     cache->n_heads, cache->head_dim, kv::log2_of(cache->block_size)};
    const int per = 256 / (cache->head_dim / 4) * kv::kGatherTokens;
    const dim3 grid(unsigned(cache->n_heads), unsigned(std::min((T + per - 1) / per, 65535)));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool e4m3 = cache->fmt == MBD_KV_E4M3, wide = dtype == MBD_F32;
    if (e4m3 && wide) hipLaunchKernelGGL((kv::gather_kernel<true, float>), grid, dim3(256), 0, s, a);
    else if (e4m3) hipLaunchKernelGGL((kv::gather_kernel<true, uint16_t>), grid, dim3(256), 0, s, a);
    else if (wide) hipLaunchKernelGGL((kv::gather_kernel<false, float>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv::gather_kernel<false, uint16_t>), grid, dim3(256), 0, s, a);
    return hip_check("gather launch");
}

}  // extern "C"
