// The paged 8-bit KV cache around its attention: block tables and slot maps from
// request lengths, the append that quantises new keys and values, and the read-back.
// A decode step's time is the bytes that it reads ([Bolt] background); beside the
// weights those are the cached keys and values, halved here against bf16.
#include <hip/hip_runtime.h>

#include "kv_common.h"

namespace mbd {
namespace kv {

// ---------------------------------------------------------------- slots

constexpr int kMaxSeqs = 4096;
constexpr int kSlotThreads = 1024;
constexpr int kPer = kMaxSeqs / kSlotThreads;   // requests of one thread, neighbours

struct SlotArgs {
    const int32_t *add, *lens, *held, *n_free;
    int32_t *table, *free_blocks;
    int32_t *seq_start, *slots, *positions, *lens_out, *held_out, *n_free_out, *status;
    int32_t n, shift, max_blocks, n_blocks, T;
};

// Exclusive sum over the workgroup's threads, and the total.
template <class V>
__device__ __forceinline__ V block_scan(V v, V* wave_sums, V* total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    V inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const V up = __shfl_up(inc, d);
        if (lane >= d) inc += up;
    }
    if (lane == 63) wave_sums[wave] = inc;
    __syncthreads();
    V before = 0, all = 0;
    for (int w = 0; w < waves; ++w) {
        const V s = wave_sums[w];
        if (w < wave) before += s;
        all += s;
    }
    __syncthreads();
    *total = all;
    return before + inc - v;
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

// One workgroup: every request's place in the step's token batch, in the blocks that
// come back and in the blocks that are taken is a prefix sum over the requests; the
// entries behind each sum are then written flat over the threads, each finding its
// request by bisection of the sums in LDS.  Work is a few KB, so the time is that of
// the dependent loads (lengths, free stack, tables) and of two scans.
__global__ __launch_bounds__(kSlotThreads) void slots_kernel(SlotArgs a) {
    __shared__ int64_t sums[2][kSlotThreads / 64];
    __shared__ int32_t start[kMaxSeqs + 1], back_at[kMaxSeqs + 1], take_at[kMaxSeqs + 1];
    __shared__ int32_t from[kMaxSeqs];       // position of the first new token, -1: not served
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
    int64_t all_add, all_back;
    int64_t at_add = block_scan(my_add, sums[0], &all_add);
    int64_t at_back = block_scan(my_back, sums[1], &all_back);
    const int32_t n_free = min(max(*a.n_free, 0), a.n_blocks);
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
    int64_t all_need;
    int64_t at_need = block_scan(my_need, sums[0], &all_need);
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
    for (int32_t e = t; e < int32_t(top) - n_free; e += blockDim.x) {
        const int i = owner(back_at, n, e);
        a.free_blocks[n_free + e] = a.table[int64_t(i) * a.max_blocks + (e - back_at[i])];
    }
    __syncthreads();
    for (int32_t e = t; e < taken; e += blockDim.x) {
        const int i = owner(take_at, n, e);
        // the first column that is not held: lens_out, held_out may be lens, held
        const int64_t blocks = a.held_out[i] - (take_at[i + 1] - take_at[i]);
        a.table[int64_t(i) * a.max_blocks + blocks + (e - take_at[i])] = a.free_blocks[int32_t(top) - 1 - e];
    }
    __syncthreads();
    for (int32_t e = t; e < a.T; e += blockDim.x) {
        const int i = owner(start, n, e);
        int32_t slot = -1, pos = -1;
        if (i < n && from[i] >= 0) {
            pos = from[i] + (e - start[i]);
            const int32_t id = a.table[int64_t(i) * a.max_blocks + (pos >> a.shift)];
            if (id >= 0 && id < a.n_blocks) slot = (id << a.shift) + (pos & (bs - 1));
        }
        a.slots[e] = slot;
        if (a.positions) a.positions[e] = pos;
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

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

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

// Four scaled values as one word of codes.
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

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p);
    return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                 __uint_as_float(w.y & 0xffff0000u)};
}

// A 16-byte unit of a code tile: lane (g, m) of slab s holds, of a key tile, token m and
// channels 64s + 16g .. +16; of a value tile, tokens 4g .. +4 and channels 64s + 4m .. +4.
// x[i] is the value of byte i, 0 where the byte's token is not among the call's (new_at).
template <bool V, class T>
__device__ __forceinline__ void load_unit(float x[16], const T* row0, int64_t stride, int tile, int s, int g, int m,
                                          int fill, int end) {
    if constexpr (V) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int tok = tile * kTok + 4 * g + k;
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if (tok >= fill && tok < end) v = load4(row0 + (tok - fill) * stride + 64 * s + 4 * m);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * j + k] = v[j];
        }
    } else {
        const int tok = tile * kTok + m;
        const bool in = tok >= fill && tok < end;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f32x4 v = {0.f, 0.f, 0.f, 0.f};
            if (in) v = load4(row0 + (tok - fill) * stride + 64 * s + 16 * g + 4 * k);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * k + j] = v[j];
        }
    }
}

// One wave, one (run, head, keys or values): a run is the tokens of one block that the
// call brings, places [fill, end).
template <bool E4M3, bool V, class T>
__device__ __forceinline__ void append_run(const AppendArgs& a, int32_t token, int64_t block, int fill, int end, int head) {
    const int lane = threadIdx.x & 63, g = lane >> 4, m = lane & 15;
    const int D = a.head_dim, slabs = D / 64;
    const int64_t bh = block * a.n_heads + head;
    uint8_t* codes = a.codes[V] + ((bh * D) << a.shift);
    const int64_t stride = a.stride[V];
    const T* row0 = static_cast<const T*>(a.x[V]) + int64_t(token) * stride + int64_t(head) * D;
    const float old = fill > 0 ? a.scales[V][bh] : 0.f;
    float amax = 0.f;
    for (int tile = fill / kTok; tile * kTok < end; ++tile)
        for (int s = 0; s < slabs; ++s) {
            float x[16];
            load_unit<V>(x, row0, stride, tile, s, g, m, fill, end);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = fabsf(x[i]);
                amax = v <= 3.4028235e38f ? fmaxf(amax, v) : amax;      // NaN and infinities do not count
            }
        }
    const float wanted = wanted_scale<E4M3>(wave_max(amax));
    const bool grew = wanted > old;
    const float now = grew ? wanted : old, div = now > 0.f ? now : 1.f;
    const float ratio = old / div;
    if (lane == 0 && (grew || fill == 0)) a.scales[V][bh] = now;
    for (int tile = grew ? 0 : fill / kTok; tile * kTok < end; ++tile)
        for (int s = 0; s < slabs; ++s) {
            const int first = tile * kTok + (V ? 4 * g : m), last = first + (V ? 4 : 1);   // the unit's tokens
            if (first >= end || (!grew && last <= fill)) continue;
            u32x4* unit = reinterpret_cast<u32x4*>(codes + int64_t(tile) * kTok * D + s * 1024 + lane * 16);
            u32x4 w = {0, 0, 0, 0};
            if (first < fill || last > end) w = *unit;
            float x[16];
            load_unit<V>(x, row0, stride, tile, s, g, m, fill, end);
            u32x4 res;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float fresh[4], kept[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) fresh[k] = x[4 * q + k] / div;
                kept[0] = code_value<E4M3, 0>(w[q]) * ratio;
                kept[1] = code_value<E4M3, 1>(w[q]) * ratio;
                kept[2] = code_value<E4M3, 2>(w[q]) * ratio;
                kept[3] = code_value<E4M3, 3>(w[q]) * ratio;
                const uint32_t nw = encode<E4M3>(fresh), ow = grew ? encode<E4M3>(kept) : w[q];
                uint32_t mask = 0;                  // bytes whose tokens are new
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = V ? first + k : first;
                    if (tok >= fill && tok < end) mask |= 255u << (8 * k);
                }
                res[q] = (nw & mask) | (ow & ~mask);
            }
            *unit = res;
        }
}

// Each wave looks through a window of tokens for the first token of a run and takes the
// runs that begin there; the waves of a workgroup take neighbouring (head, keys or
// values), which lie side by side in the tokens' rows.
template <bool E4M3, class T>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int hw = blockIdx.y * 4 + wave;
    if (hw >= 2 * a.n_heads) return;
    const int head = hw % a.n_heads;
    const bool values = hw >= a.n_heads;
    const int bs = 1 << a.shift;
    const int32_t t0 = int32_t(blockIdx.x) * a.window;
    const int32_t mine = t0 + lane;
    const int32_t slot = mine < a.T ? a.slots[mine] : -1;
    const int32_t prev = mine < a.T && mine > 0 ? a.slots[mine - 1] : -2;
    const bool good = slot >= 0 && slot < a.n_slots;
    const bool leads = good && lane < a.window && (prev != slot - 1 || (slot & (bs - 1)) == 0);
    uint64_t todo = __ballot(leads);
    while (todo) {
        const int l = __builtin_ctzll(todo);
        todo &= todo - 1;
        const int32_t first = __shfl(slot, l), token = t0 + l;
        const int fill = first & (bs - 1);
        int count = 1;
        for (int at = 1; at < bs - fill; at += 64) {
            const int k = at + lane;
            const bool on = k < bs - fill && token + k < a.T && a.slots[token + k] == first + k;
            const uint64_t off = ~__ballot(on);
            count = at + (off ? __builtin_ctzll(off) : 64);
            if (off) break;
        }
        if (values) append_run<E4M3, true, T>(a, token, first >> a.shift, fill, fill + count, head);
        else append_run<E4M3, false, T>(a, token, first >> a.shift, fill, fill + count, head);
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

__device__ __forceinline__ void store4(float* p, const f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, const f32x4 v) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

constexpr int kGatherTokens = 4;   // tokens of one thread

// A thread writes four neighbouring channels, so that a workgroup's stores are whole
// rows.  The four tokens of a value word are read by four threads: the repeats hit L1.
template <bool E4M3, class T>
__global__ __launch_bounds__(256) void gather_kernel(GatherArgs a) {
    const int quads = a.head_dim / 4, rows = 256 / quads;
    const int row = threadIdx.x / quads, quad = threadIdx.x - row * quads;
    if (row >= rows) return;
    const int head = blockIdx.y, D = a.head_dim;
    const int32_t t0 = int32_t(blockIdx.x) * rows * kGatherTokens + row;
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
                   n_free_out, status, pool->n_seqs, kv::log2_of(pool->block_size), pool->max_blocks, pool->n_blocks, T};
    hipLaunchKernelGGL(kv::slots_kernel, dim3(1), dim3(kv::kSlotThreads), 0, reinterpret_cast<hipStream_t>(stream), a);
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
    // Waves look through windows of tokens: one token each while that gives no more waves than
    // the chip holds twice over, longer windows beyond, so that idle waves do not add up.
    const int64_t waves = int64_t(T) * 2 * cache->n_heads;
    int32_t window = 1;
    while (window < 64 && waves / window > 16384) window *= 2;
    kv::AppendArgs a{{static_cast<uint8_t*>(cache->k_codes), static_cast<uint8_t*>(cache->v_codes)}, {cache->k_scale, cache->v_scale},
                     {k, v}, {k_stride, v_stride}, slots, int32_t(cache->n_blocks * cache->block_size), T, window, cache->n_heads,
                     cache->head_dim, kv::log2_of(cache->block_size)};
    const dim3 grid(unsigned((T + window - 1) / window), unsigned((2 * cache->n_heads + 3) / 4));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool e4m3 = cache->fmt == MBD_KV_E4M3, wide = dtype == MBD_F32;
    if (e4m3 && wide) hipLaunchKernelGGL((kv::append_kernel<true, float>), grid, dim3(256), 0, s, a);
    else if (e4m3) hipLaunchKernelGGL((kv::append_kernel<true, uint16_t>), grid, dim3(256), 0, s, a);
    else if (wide) hipLaunchKernelGGL((kv::append_kernel<false, float>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv::append_kernel<false, uint16_t>), grid, dim3(256), 0, s, a);
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
    const dim3 grid(unsigned((T + per - 1) / per), unsigned(cache->n_heads));
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    const bool e4m3 = cache->fmt == MBD_KV_E4M3, wide = dtype == MBD_F32;
    if (e4m3 && wide) hipLaunchKernelGGL((kv::gather_kernel<true, float>), grid, dim3(256), 0, s, a);
    else if (e4m3) hipLaunchKernelGGL((kv::gather_kernel<true, uint16_t>), grid, dim3(256), 0, s, a);
    else if (wide) hipLaunchKernelGGL((kv::gather_kernel<false, float>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((kv::gather_kernel<false, uint16_t>), grid, dim3(256), 0, s, a);
    return hip_check("gather launch");
}

}  // extern "C"
