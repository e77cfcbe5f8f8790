// What the attention kernels over every cache format share: a call's arguments, how its work is cut into
// parts for the workgroups, and small wave helpers.
#pragma once

#include <type_traits>

#include <hip/hip_runtime.h>

#include "kv_common.h"

namespace mbd {
namespace kv {

constexpr int kStep = 2;               // tiles of one step: 32 tokens, the k of an MFMA
constexpr int kRefill = 64 / kStep;    // steps whose block ids and scales one lane each holds
constexpr int kMaxWaves = 4;           // most waves of a workgroup; they take its steps in turn
constexpr int kCus = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Workgroups a CU (waves a SIMD) that a variant's registers are held to, in either kernel: enough loads in
// flight for the memory, and as many parts as there are places for them.  (With a second
// buffer for a step's codes int8 at head_dim 128 took 213 registers, two waves, and 212 us
// for the 1.08 GB of the largest decode step.  At head_dim 64 and one row tile the registers would let
// in a fifth wave; counted as places they make shorter parts.  8 bits, five and four: 4 requests of 8000 tokens 18.1 and
// 15.7 us, a verify step of 8 x 5 15.4 and 13.9, 32 of up to 8192 32.4 and 32.3; 4 bits: 4 of 8000 15.6 and 14.4, 16 of
// 2500 17.1 and 14.4, one of 100001 24.0 and 23.3, 32 of up to 8192 27.0 and 26.7, of 16384 66 and 69.)
constexpr int per_cu(int dq, int nt) { return nt == 1 ? (dq <= 2 ? 4 : dq == 3 ? 3 : 2) : (dq == 1 ? 4 : dq == 2 ? 3 : 2); }

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
template <int N> using Const = std::integral_constant<int, N>;

// A tile of a request's query rows whose tokens are cut into parts, for what joins them;
// parts = 0 behind the last.
struct Split {
    int32_t parts, slot, stride;         // slot of its first partial result, slots from one to the next
    int32_t row0, r0, rows;              // the request's first row of q; the tile's first row, and how many
};

struct AttnArgs {
    const uint8_t *k, *v;
    const void *k_scale, *v_scale;       // fp32, or bytes in 4 bits
    const uint16_t* q;
    const int32_t *seq_start, *lens, *table;
    uint16_t* out;
    float *lse, *part_o, *part_ml;
    Split* splits;                       // [n_splits]
    const float* slopes;
    int64_t q_stride, out_stride;
    uint32_t per_group;                  // ceil(2^32 / group)
    int32_t n_blocks, n_seqs, max_blocks, T, max_new, window, shift, n_kv, group, row_shift, min_part, places, unit, n_splits, n_parts;
    bool split;                          // whether requests may be cut into parts
    float to_score, softcap;             // product to score in the log2 domain (or over the cap); the cap there
    int32_t most_ks;                     // 8 bits: largest key scale whose product with to_score is finite, as bits
    uint32_t flip;                       // 4 bits: sign bits of the queries where the scale is negative; to_score is its magnitude
};

// Token of a query row: r / group, exact for r * group below 2^32.
__device__ __forceinline__ int token_of(const AttnArgs& a, int r) { return a.group == 1 ? r : int(__umulhi(uint32_t(r), a.per_group)); }

// ---------------------------------------------------------------- shares of the work

// A request as its workgroups see it.
struct Seq {
    int32_t row0, n_new, rows;   // first row of q, new tokens, rows a KV head (up to max_new tokens)
    int32_t p0;                  // position of its first new token (below 0: before its start)
    int32_t lo, hi;              // tiles that any of its queries sees
    int32_t len;
};

__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int i) {
    Seq s;
    s.row0 = min(max(a.seq_start[i], 0), a.T);
    s.n_new = min(max(a.seq_start[i + 1], s.row0), a.T) - s.row0;
    s.len = min(max(a.lens[i], 0), a.max_blocks << a.shift);
    const int32_t tokens = min(s.n_new, a.max_new);
    s.rows = tokens * a.group;
    s.p0 = s.len - s.n_new;
    const int32_t end = max(s.p0 + tokens, 0);
    s.lo = a.window > 0 ? max(max(s.p0, 0) - a.window + 1, 0) / kTok : 0;
    s.hi = (end + kTok - 1) / kTok;
    return s;
}

// Inclusive sum over the wave's lanes, by row shifts and row broadcasts (no LDS trips).
template <int CTRL, int ROWS>
__device__ __forceinline__ int plus_dpp(int v) { return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false); }

__device__ __forceinline__ int wave_scan(int v) {
    v = plus_dpp<0x111, 0xf>(v);       // row_shr 1, 2, 4, 8
    v = plus_dpp<0x112, 0xf>(v);
    v = plus_dpp<0x114, 0xf>(v);
    v = plus_dpp<0x118, 0xf>(v);
    v = plus_dpp<0x142, 0xa>(v);       // row_bcast 15 into rows 1 and 3
    return plus_dpp<0x143, 0xc>(v);    // row_bcast 31 into rows 2 and 3
}

// The lengths are known on the device alone, so the workgroups cut the work up themselves: in 8 bits every wave
// for itself, by find_item; in 4 bits one wave for its workgroup, up to 64 requests by find_item_64, above by
// find_item.  The work of a request is its tiles of tokens times its tiles of query rows; all of it over the
// places that the chip has for a head's workgroups is a chunk of tokens, a request is cut into
// ceil(tokens / chunk) even parts, and the workgroup's (request, part, row tile) follows from
// the prefix sums of their counts.  One round of workgroups: two or four rounds of shorter
// ones, which end more evenly, lost more on the way to their first product (with an earlier form,
// 32 requests of 32768 tokens 201 and 207 us against 193, one of 131072 64 and 77 against 57).
__device__ __forceinline__ int tiles_of(const Seq& s) { return s.n_new < 1 ? 0 : max(s.hi - s.lo, 1); }
__device__ __forceinline__ int row_tiles_of(const AttnArgs& a, const Seq& s) { return (s.rows + (1 << a.row_shift) - 1) >> a.row_shift; }

struct Item {
    int32_t seq, parts, index;           // index: among the request's, row tiles fastest
    int32_t slot, split;                 // of the request's first partial result; split row tiles before it
};

__device__ __forceinline__ int32_t even_part(int tiles, int parts) {     // tiles of a part, whole steps
    return ((tiles - 1) / parts + kStep) / kStep * kStep;
}

// Item `want` (seq is -1 if there is none), its request, and how many row tiles are split, for any number of requests.
__device__ __forceinline__ Item find_item(const AttnArgs& a, int32_t want, Seq* sq, int* splits) {
    const int lane = threadIdx.x & 63;
    // Request 64 j + l is lane l's in turn j: a turn's loads are whole lines.  (With a run of
    // neighbours a lane each load met 64 lines, and 1000 requests of up to 600 tokens took 169 us
    // against 103.)
    const Seq first = load_seq(a, min(lane, a.n_seqs - 1));     // turn 0, read once
    const int n0 = lane < a.n_seqs ? tiles_of(first) : 0, rt0 = n0 ? row_tiles_of(a, first) : 0;
    // f(tiles, row tiles) of the lane's requests; the loads of four turns are in flight at once
    auto each = [&](auto&& f) {
        f(n0, rt0);
#pragma unroll 4
        for (int i = 64 + lane; i < a.n_seqs; i += 64) {
            const Seq s = load_seq(a, i);
            const int n = tiles_of(s);
            f(n, n ? row_tiles_of(a, s) : 0);
        }
    };
    // in units that keep the sum within 32 bits, rounded up
    int work = 0, used = 0;
    each([&](int n, int rt) {
        work += int((uint64_t(uint32_t(n)) * uint32_t(rt) + (uint64_t(1) << a.unit) - 1) >> a.unit);
        used += rt;
    });
    work = max(__builtin_amdgcn_readlane(wave_scan(work), 63), 1);
    used = __builtin_amdgcn_readlane(wave_scan(used), 63);
    // With chunks of work / room, the parts times row tiles add up to between room and
    // room + used: the smallest of three chunks whose items fit the places, of which the
    // last always does, unless there are as many row tiles as places: then only what is longer
    // than two places' share is cut (prompt slices cut at one share each: 58 us, 12 of them the
    // join; not cut 51).  No chunk is below work / places, so the items of split requests
    // number less than twice the places.
    uint32_t chunk = 0x7fffffff;
    int cut = 0;                                   // split row tiles
    auto parts_of = [&](int n) { return int((uint32_t(n) + chunk - 1) / chunk); };
#pragma unroll 1
    for (int tries = 0; tries < 3; ++tries) {
        if (a.split) {
            const int room = a.places - (tries * used + 1) / 2;
            const uint64_t share = uint64_t(uint32_t(work - 1) / uint32_t(room > 0 ? room : (a.places + 1) / 2) + 1) << a.unit;
            chunk = uint32_t(min(max(share, uint64_t(a.min_part)), uint64_t(1) << 30));
        }
        int items = 0;
        cut = 0;
        each([&](int n, int rt) {
            const int p = parts_of(n);
            items += p * rt;
            cut += p > 1 ? rt : 0;
        });
        if (!a.split || __builtin_amdgcn_readlane(wave_scan(items), 63) <= a.places) break;
    }
    *splits = __builtin_amdgcn_readlane(wave_scan(cut), 63);

    Seq s = first;
    int items = 0, slots = 0, cuts = 0;            // of earlier turns
#pragma unroll 1
    for (int turn = 0; turn < a.n_seqs; turn += 64) {
        Seq next = s;
        if (turn + 64 < a.n_seqs) next = load_seq(a, min(turn + 64 + lane, a.n_seqs - 1));
        const int n = turn + lane < a.n_seqs ? tiles_of(s) : 0, rt = n ? row_tiles_of(a, s) : 0, p = parts_of(n);
        const int mine = p * rt, my_slots = p > 1 ? mine : 0, my_cuts = p > 1 ? rt : 0;
        const int end = items + wave_scan(mine), slots_end = slots + wave_scan(my_slots), cuts_end = cuts + wave_scan(my_cuts);
        const uint64_t who = __ballot(want >= end - mine && want < end);
        if (who) {
            const int l = __builtin_ctzll(who);
            auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            *sq = {of(s.row0), of(s.n_new), of(s.rows), of(s.p0), of(s.lo), of(s.hi), of(s.len)};
            return {turn + l, of(p), want - of(end - mine), of(slots_end - my_slots), of(cuts_end - my_cuts)};
        }
        items = __builtin_amdgcn_readlane(end, 63);
        slots = __builtin_amdgcn_readlane(slots_end, 63);
        cuts = __builtin_amdgcn_readlane(cuts_end, 63);
        s = next;
    }
    return {-1, 0, 0, 0, 0};
}

// Maximum over the four lanes of a query row (lane % 16): the rows of 16 lanes swap places.
__device__ __forceinline__ float lane_max(float v) {
    const uint32_t x = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    const float m = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
    const uint32_t y = __float_as_uint(m);
    const auto r = __builtin_amdgcn_permlane16_swap(y, y, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Bytes of a value word (tokens tok .. tok+4) whose tokens exist; the rest may be anything
// in memory, NaN codes included, and a zero weight does not silence those.
__device__ __forceinline__ uint32_t live_bytes(int tok, int len) {
    const int n = min(max(len - tok, 0), 4);
    return n == 4 ? 0xffffffffu : (1u << (8 * n)) - 1u;
}

// Near 0, where 1 - 2 / (1 + e^2x) would cancel, the series (next term below 2^-26 of it).
__device__ __forceinline__ float tanh_of(float x) {
    const float y = x * x;
    const float near = x * (1.f + y * (-1.f / 3 + y * (2.f / 15 + y * (-17.f / 315 + y * (62.f / 2835)))));
    const float far = 1.f - 2.f * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * (2.f * kLog2e)));
    return y < 0.0625f ? near : far;
}

// Codes unpacked far ahead of their product would cost a wave or two a SIMD in registers.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ float lane_float(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

}  // namespace kv
}  // namespace mbd
