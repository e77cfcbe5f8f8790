// Attention over the paged 8-bit KV cache ([Bolt] background: a decode step's time is
// the bytes it reads; next to the weights those are the cached keys and values).
//
// Per KV head the query rows of one request (its new tokens times the query heads that
// share the head) are the columns of both matrix products, the cached tokens the rows:
//   S^T [tokens][rows] = K [tokens][d] Q^T,  O^T [d][rows] += V^T [d][tokens] P^T
// with v_mfma_f32_16x16x32_bf16.  A lane's accumulators of S^T (4 tokens of a 16-token
// tile, for one row) are then its own B operand of the second product, two tiles being
// one k step of 32: nothing crosses lanes but the row maxima.  The cache stores each
// tile as the lanes' A operands, so a wave reads whole KBs, and codes become bf16
// (exact for int8 and e4m3) on their way into the product; the block's scale is one
// factor of the 16 x 16 scores, or of the weights.
//
// A decode step is bound by the codes it streams: 32 requests of 32768 tokens (64 / 4 heads
// x 128, int8, 1.08 GB) take 180 us, 6.0 of the 6.5 TB/s that a plain read of 4 GiB reaches, and 5 us
// to join the parts; 32 requests of 1 to 8192 tokens (32 / 8 heads, e4m3, 277 MB) 49 + 5 us, 5.6 TB/s.
// Short calls are bound by the way to the first product (lengths -> table -> scales and codes,
// a memory latency each): one request of 2048 tokens takes 6 + 4 us.  Many query rows are bound
// by the vector units (scores and unpacking take three times the matrix units' cycles) and by how
// the row tiles fill the chip: four prompt slices of 90 to 300 tokens, 22.5 GFLOP, are 113 row tiles
// a head on 96 places and take 58 + 5 us, 52 in a row of such calls.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "kv_common.h"

namespace mbd {
namespace kv {

constexpr int kStep = 2;               // tiles of one step: 32 tokens, the k of an MFMA
constexpr int kRefill = 64 / kStep;    // steps whose block ids and scales one lane each holds
constexpr int kMaxWaves = 4;           // most waves of a workgroup; they take its steps in turn
constexpr int kCus = 256;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// A tile of a request's query rows whose tokens are cut into parts, for what joins them;
// parts = 0 behind the last.
struct Split {
    int32_t parts, slot, stride;         // slot of its first partial result, slots from one to the next
    int32_t row0, r0, rows;              // the request's first row of q; the tile's first row, and how many
};

struct AttnArgs {
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
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
    int32_t most_ks;                     // largest key scale whose product with to_score is finite, as bits
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

// The lengths are known on the device alone, so every wave cuts the work up itself.  The
// work of a request is its tiles of tokens times its tiles of query rows; all of it over the
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

// Item `want` (seq is -1 if there is none), its request, and how many row tiles are split.
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

// ---------------------------------------------------------------- operands

// Eight codes as the bf16 values they stand for before scaling.
template <bool E4M3>
__device__ __forceinline__ bf16x8 operand(uint32_t w0, uint32_t w1) {
    u32x4 r;
    if constexpr (E4M3) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true));
    } else {
        // |code| <= 127 leaves the low half of its fp32 form zero: the high halves are the bf16s
        // (the empty asm keeps the words whole until here: taken apart at their loads, each byte
        // would hold a register of its own while the step is in flight)
        asm("" : "+v"(w0), "+v"(w1));
        const uint32_t w[2] = {w0, w1};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t f0 = __float_as_uint(code_value<false, 0>(w[h])), f1 = __float_as_uint(code_value<false, 1>(w[h]));
            const uint32_t f2 = __float_as_uint(code_value<false, 2>(w[h])), f3 = __float_as_uint(code_value<false, 3>(w[h]));
            r[2 * h] = __builtin_amdgcn_perm(f1, f0, 0x07060302);
            r[2 * h + 1] = __builtin_amdgcn_perm(f3, f2, 0x07060302);
        }
    }
    return __builtin_bit_cast(bf16x8, r);
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

// Workgroups a CU (waves a SIMD) that a variant's registers are held to: enough loads in
// flight for the memory, and as many parts as there are places for them.  (With a second
// buffer for a step's codes int8 at head_dim 128 took 213 registers, two waves, and 212 us
// for the 1.08 GB of the largest decode step.  At head_dim 64 and one row tile the registers would let
// in a fifth wave; counted as places they make shorter parts: 4 requests of 8000 tokens 18.1 us against
// 15.7, a verify step of 8 x 5 15.4 against 13.9, 32 of up to 8192 32.4 against 32.3.)
constexpr int per_cu(int dq, int nt) { return nt == 1 ? (dq <= 2 ? 4 : dq == 3 ? 3 : 2) : (dq == 1 ? 4 : dq == 2 ? 3 : 2); }

// DQ = head_dim / 64, NT = tiles of 16 query rows, EXT: cap, window or distance bias, WAVES: four
// to a part, or one, which waits for no other and finds its share alone, where the requests
// outnumber the places that parts of four waves have.  Four waves against one there:
// 1000 requests of up to 600 tokens (64 / 4 heads x 128, e4m3) 167 and 103 us, 256 of up to 1000
// (32 / 8 x 128, int8) 68 and 64.5, 160 of up to 8192 (e4m3) 241 and 237, 40 of up to 600 with 32 / 32
// heads 27.9 and 28.8; with fewer requests, 100 of up to 600 (32 / 8) 22.8 and 25.7, 64 of 2000 to 4000
// 79.4 and 78.7.
template <bool E4M3, int DQ, int NT, bool EXT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(per_cu(DQ, NT)))) void attn_kernel(AttnArgs a) {
    constexpr int D = 64 * DQ, ROWS = 16 * NT, PITCH = 68;
    __shared__ float merge[WAVES][ROWS][PITCH];     // pitch: rows 4 banks apart
    __shared__ float merge_m[WAVES][ROWS], merge_l[WAVES][ROWS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, n = lane & 15;
    const int in_block = (1 << a.shift) - 1;
    // Heads side by side: workgroups go round the XCDs, so that of 8 heads each has an XCD, in
    // whose L2 a request's row tiles find each other's codes.
    const int want = blockIdx.x / uint32_t(a.n_kv), head = blockIdx.x - want * a.n_kv;
    Seq sq;
    int splits;
    const Item it = find_item(a, want, &sq, &splits);
    if (head == 0 && threadIdx.x == 0 && want >= splits && want < a.n_splits) a.splits[want] = Split{0, 0, 0, 0, 0, 0};
    if (it.seq < 0) return;
    const int row_tiles = row_tiles_of(a, sq), part = it.index / row_tiles;
    const int row_tile = row_tiles - 1 - (it.index - part * row_tiles);       // the last rows, which see most, first
    const int r0 = row_tile * ROWS, slot = it.slot + row_tile;
    const int rows = min(ROWS, sq.rows - r0);
    // what the first and the last row see bounds what any row sees
    const int pos_first = sq.p0 + token_of(a, r0), pos_last = sq.p0 + token_of(a, r0 + rows - 1);
    const int all_end = pos_first + 1, all_begin = a.window > 0 ? max(pos_last, 0) - a.window + 1 : 0;
    int t0 = sq.lo, t1 = min(sq.hi, (max(pos_last + 1, 0) + kTok - 1) / kTok);
    if (it.parts > 1) {
        // (starts that fall, which no request can have, could count rows twice; in range all the same)
        if (it.split + row_tile >= a.n_splits || slot + int64_t(it.parts - 1) * row_tiles >= a.n_parts) return;
        const int size = even_part(tiles_of(sq), it.parts);
        t0 += part * size;
        t1 = min(t1, t0 + size);
        if (head == 0 && threadIdx.x == 0 && part == 0) a.splits[it.split + row_tile] = Split{it.parts, slot, row_tiles, sq.row0, r0, rows};
    }
    if (a.window > 0) t0 = max(t0, max(max(pos_first, 0) - a.window + 1, 0) / kTok);

    const int steps = (max(t1 - t0, 0) + kStep - 1) / kStep;
    const int mine = steps > wave ? (steps - wave + WAVES - 1) / WAVES : 0;
    auto tile_of = [&](int k) { return t0 + kStep * (wave + WAVES * k); };
    // lane l looks up tile l % 2 of step k0 + l / 2; the first look is on its way before the queries
    const int32_t* table = a.table + int64_t(it.seq) * a.max_blocks;
    auto look_up = [&](int k0) {
        const int tile = tile_of(k0 + lane / kStep) + lane % kStep;
        return tile < t1 ? table[(tile * kTok) >> a.shift] : -1;
    };
    int32_t next_id = look_up(0);

    // Two row tiles' queries would hold as many registers as a third wave a SIMD needs: they lie
    // in LDS, in the lanes' order, and every wave reads them there.
    constexpr bool kQueryLds = NT > 1;
    __shared__ u32x4 queries[kQueryLds ? NT * 2 * DQ : 1][64];
    u32x4 held[kQueryLds ? 1 : NT][kQueryLds ? 1 : 2 * DQ];
    int pos[NT];
    float slope[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = r0 + 16 * t + n;
        const bool in = r < sq.rows;
        const int j = token_of(a, r), qh = head * a.group + (r - j * a.group);
        pos[t] = in ? sq.p0 + j : -1;
        slope[t] = 0.f;
        if (EXT && a.slopes && in) slope[t] = a.slopes[qh] * kLog2e;
        const uint16_t* row = a.q + int64_t(sq.row0 + j) * a.q_stride + int64_t(qh) * D + 16 * g;
#pragma unroll
        for (int c = 0; c < 2 * DQ; ++c) {
            if (kQueryLds && c % WAVES != wave) continue;
            u32x4 w = {0, 0, 0, 0};
            if (in) w = *reinterpret_cast<const u32x4*>(row + 64 * (c / 2) + 8 * (c % 2));
            if constexpr (kQueryLds) queries[t * 2 * DQ + c][lane] = w;
            else held[t][c] = w;
        }
    }
    if (kQueryLds) __syncthreads();
    auto query = [&](int t, int c) {
        if constexpr (kQueryLds) return __builtin_bit_cast(bf16x8, queries[t * 2 * DQ + c][lane]);
        else return __builtin_bit_cast(bf16x8, held[t][c]);
    };

    f32x4 acc[DQ][4][NT];
    float top[NT], sum[NT];          // base of the weights (log2 domain); this lane's share of their sum
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        top[t] = -INFINITY;
        sum[t] = 0.f;
#pragma unroll
        for (int c = 0; c < DQ; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[c][j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    int32_t my_id = -1;
    float my_ks = 0.f, my_vs = 0.f;

    u32x4 kc[kStep][DQ], vc[kStep][DQ];      // one step's codes
    auto load = [&](u32x4 (&to)[kStep][DQ], const uint8_t* codes, int tile, int l) {
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
            const int32_t id = max(__builtin_amdgcn_readlane(my_id, l + h), 0);
            const uint8_t* from = codes + ((((int64_t(id) * a.n_kv + head) << a.shift) + (((tile + h) * kTok) & in_block)) * D);
#pragma unroll
            for (int c = 0; c < DQ; ++c) {
                const u32x4* p = reinterpret_cast<const u32x4*>(from + c * 1024 + lane * 16);
                // one tile of query rows is all there is: the codes are read once and streamed (32 x
                // 8192 tokens 70 -> 66 us); with several, the other tiles find them in L2 (prompt
                // slices 88 us, streamed 100)
                to[h][c] = NT == 1 ? __builtin_nontemporal_load(p) : *p;
            }
        }
    };

    // The next step's keys are asked for as soon as this one's are used up, and so the values:
    // each load has the other product and the softmax to arrive in.  A second buffer, asked for a
    // whole step ahead, measured the same (prompt slices 55 us) and costs a wave a SIMD.
    auto step = [&](int tile, int l, int next_tile, bool more) {
        if (kQueryLds) asm volatile("" ::: "memory");      // the queries are read again in each step
        f32x4 s[kStep][NT];
        bool whole = tile * kTok >= all_begin && (tile + kStep) * kTok <= all_end;
        float ks[kStep], vs[kStep];
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
            // the factor stays finite: past fp32 a zero score would become 0 * inf, where any other only
            // meets the cap (scales are not negative, so their bits compare as they do)
            ks[h] = __int_as_float(min(__builtin_amdgcn_readlane(__float_as_int(my_ks), l + h), a.most_ks)) * a.to_score;
            vs[h] = lane_float(my_vs, l + h);
            whole = whole && __builtin_amdgcn_readlane(my_id, l + h) >= 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) s[h][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int c = 0; c < DQ; ++c) {
            keep_order();
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int h = 0; h < kStep; ++h) {
                    const bf16x8 kf = operand<E4M3>(kc[h][c][2 * e], kc[h][c][2 * e + 1]);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        s[h][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, query(t, 2 * c + e), s[h][t], 0, 0, 0);
                }
        }
        keep_order();
        if (more) load(kc, a.k, next_tile, l + kStep);
        keep_order();
        bf16x8 pf[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float u[kStep][4];
            const float away = float(tile * kTok + 4 * g - pos[t]);
#pragma unroll
            for (int h = 0; h < kStep; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = s[h][t][i] * ks[h];
                    if (EXT && a.softcap > 0.f) x = a.softcap * tanh_of(x);
                    if (EXT) x += slope[t] * (away + float(h * kTok + i));
                    u[h][i] = x;
                }
            if (!whole) {
#pragma unroll
                for (int h = 0; h < kStep; ++h) {
                    const bool id_ok = __builtin_amdgcn_readlane(my_id, l + h) >= 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int tok = (tile + h) * kTok + 4 * g + i;
                        bool sees = id_ok && tok <= pos[t];
                        if (EXT && a.window > 0) sees = sees && pos[t] - tok < a.window;
                        u[h][i] = sees ? u[h][i] : -INFINITY;
                    }
                }
            }
            float m = fmaxf(fmaxf(fmaxf(u[0][0], u[0][1]), fmaxf(u[0][2], u[0][3])),
                            fmaxf(fmaxf(u[1][0], u[1][1]), fmaxf(u[1][2], u[1][3])));
            m = lane_max(m);
            // the base of the weights need not be the maximum, only near it: it moves where a
            // weight would pass 2^8, so most steps leave the sums as they are
            if (__ballot(m > top[t] + 8.f)) {
                m = fmaxf(m, top[t]);
                const float f = __builtin_amdgcn_exp2f(top[t] - (m == -INFINITY ? 0.f : m));
                sum[t] *= f;
#pragma unroll
                for (int c = 0; c < DQ; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[c][j][t] *= f;
                top[t] = m;
            }
            const float base = top[t] == -INFINITY ? 0.f : top[t];
            float p[kStep][4];
#pragma unroll
            for (int h = 0; h < kStep; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[h][i] = __builtin_amdgcn_exp2f(u[h][i] - base);
                    sum[t] += p[h][i];
                    p[h][i] *= vs[h];
                }
            // The matrix unit takes bf16: a weight times its value scale is off by at most 2^-8 of
            // itself, and so is o where one token has the weight, or where equal weights share a block's scale
            // and so their rounding; over many tokens of unlike weights the errors mostly cancel (o off by
            // 2.1e-3 to 2.3e-3 in the mean, its own rounding to bf16 among it, which alone is 1.65e-3).
            // With what is left of each weight as a second operand that is all, for prompt slices of 61 us
            // instead of 53, verify steps of 16 x 8 41 instead of 38, single tokens 0 to 2% more, and
            // scratch memory in six variants.  The sums are of the weights before it.
            const u32x4 w = {pack_bf16(p[0][0], p[0][1]), pack_bf16(p[0][2], p[0][3]), pack_bf16(p[1][0], p[1][1]), pack_bf16(p[1][2], p[1][3])};
            pf[t] = __builtin_bit_cast(bf16x8, w);
        }
        if (!whole) {
#pragma unroll
            for (int h = 0; h < kStep; ++h) {
                const bool id_ok = __builtin_amdgcn_readlane(my_id, l + h) >= 0;
                const uint32_t live = id_ok ? live_bytes((tile + h) * kTok + 4 * g, sq.len) : 0u;
#pragma unroll
                for (int c = 0; c < DQ; ++c) vc[h][c] &= live;
            }
        }
#pragma unroll
        for (int c = 0; c < DQ; ++c) {
            keep_order();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 vf = operand<E4M3>(vc[0][c][j], vc[1][c][j]);
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[c][j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[t], acc[c][j][t], 0, 0, 0);
            }
        }
        keep_order();
        if (more) load(vc, a.v, next_tile, l + kStep);
    };

    for (int k0 = 0; k0 < mine; k0 += kRefill) {
        my_id = next_id >= 0 && next_id < a.n_blocks ? next_id : -1;
        my_ks = my_vs = 0.f;
        if (my_id >= 0) {
            my_ks = a.k_scale[int64_t(my_id) * a.n_kv + head];
            my_vs = a.v_scale[int64_t(my_id) * a.n_kv + head];
        }
        const int end = min(mine - k0, kRefill);
        load(kc, a.k, tile_of(k0), 0);
        load(vc, a.v, tile_of(k0), 0);
        next_id = look_up(k0 + kRefill);
        for (int k = 0; k < end; ++k) step(tile_of(k0 + k), kStep * k, tile_of(k0 + k + 1), k + 1 < end);
    }

    // A row's four channels from d on: final, from their weighted sum, and the row's sum of weights.
    auto put = [&](int r, int d, const f32x4 o, float m, float l) {
        const int j = token_of(a, r0 + r), qh = head * a.group + (r0 + r - j * a.group);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* to = a.out + int64_t(sq.row0 + j) * a.out_stride + int64_t(qh) * D + d;
        *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
        if (d == 0 && a.lse) a.lse[int64_t(sq.row0 + j) * (a.n_kv * a.group) + qh] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    };
    // Join the waves: a common maximum a row, then sums slab by slab through LDS.
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        sum[t] += __shfl_xor(sum[t], 16);
        sum[t] += __shfl_xor(sum[t], 32);
        if (g == 0) {
            merge_m[wave][16 * t + n] = top[t];
            merge_l[wave][16 * t + n] = sum[t];
        }
    }
    __syncthreads();
    float f[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) m = fmaxf(m, merge_m[w][16 * t + n]);
        f[t] = __builtin_amdgcn_exp2f(top[t] - (m == -INFINITY ? 0.f : m));
    }
#pragma unroll
    for (int c = 0; c < DQ; ++c) {
        if (c) __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)      // register i of product j is channel 16g + 4i + j
                *reinterpret_cast<f32x4*>(&merge[wave][16 * t + n][16 * g + 4 * i]) =
                    f32x4{acc[c][0][t][i], acc[c][1][t][i], acc[c][2][t][i], acc[c][3][t][i]} * f[t];
        __syncthreads();
        for (int e = threadIdx.x; e < rows * 16; e += 64 * WAVES) {
            const int r = e >> 4, d = (e & 15) * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) m = fmaxf(m, merge_m[w][r]);
            const float base = m == -INFINITY ? 0.f : m;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                l += merge_l[w][r] * __builtin_amdgcn_exp2f(merge_m[w][r] - base);
                o += *reinterpret_cast<const f32x4*>(&merge[w][r][d]);
            }
            if (it.parts == 1) {
                put(r, 64 * c + d, o, m, l);
            } else {
                const int64_t to = ((slot + int64_t(part) * row_tiles) * a.n_kv + head) * ROWS + r;
                *reinterpret_cast<f32x4*>(a.part_o + to * D + 64 * c + d) = o;
                if (c == 0 && d == 0) *reinterpret_cast<f32x2*>(a.part_ml + to * 2) = f32x2{m, l};
            }
        }
    }
}

// The parts of the split row tiles: a workgroup for each four query rows of a tile and head,
// WAVES waves a row; lanes over channels, waves over parts.
// A second launch: joining in the last workgroup to arrive needs partial results that
// pass the XCDs' L2s and a counter, which took longer (with an earlier form of the kernel above, one
// request of 2048 tokens 10.5 against 8.9 us, one of 131072 84 against 57).
constexpr int kJoinRows = 4, kJoinAhead = 8;

template <int DQ, int WAVES>
__global__ __launch_bounds__(64 * kJoinRows * WAVES) void join_kernel(AttnArgs a, int rows_of_tile) {
    constexpr int D = 64 * DQ;
    __shared__ float joined[kJoinRows][WAVES][D], top[kJoinRows][WAVES], sum[kJoinRows][WAVES];
    const int lane = threadIdx.x & 63, row = threadIdx.x / (64 * WAVES), wave = (threadIdx.x >> 6) % WAVES;
    const Split sp = a.splits[blockIdx.x];
    const int head = blockIdx.y;
    // the attention kernel's own words, unless another call shares the workspace at the same time:
    // then results are lost, but nothing is read or written out of range
    if (sp.parts < 2) return;
    if (sp.rows > rows_of_tile || sp.slot < 0 || sp.stride < 1 || sp.slot + int64_t(sp.parts - 1) * sp.stride >= a.n_parts || sp.row0 < 0 ||
        sp.r0 < 0 || sp.r0 >= (1 << 24) || int64_t(sp.row0) + token_of(a, sp.r0 + sp.rows - 1) >= a.T)
        return;
    for (int pass = blockIdx.z; pass * kJoinRows < sp.rows; pass += gridDim.z) {
        const int in_tile = pass * kJoinRows + row;
        if (pass != int(blockIdx.z)) __syncthreads();          // the last pass's sums are read
        const bool mine = in_tile < sp.rows;
        const int r = sp.r0 + in_tile;
        auto row_of = [&](int p) { return ((sp.slot + int64_t(p) * sp.stride) * a.n_kv + head) * rows_of_tile + (mine ? in_tile : 0); };
        float m = -INFINITY, l = 0.f, o[DQ] = {};
        for (int p0 = wave; p0 < sp.parts; p0 += kJoinAhead * WAVES) {
            f32x2 ml[kJoinAhead];
            float x[kJoinAhead][DQ];
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k) {
                const int64_t at = row_of(min(p0 + k * WAVES, sp.parts - 1));
                ml[k] = *reinterpret_cast<const f32x2*>(a.part_ml + at * 2);
#pragma unroll
                for (int c = 0; c < DQ; ++c) x[k][c] = a.part_o[at * D + 64 * c + lane];
            }
            float most = m;
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (p0 + k * WAVES < sp.parts) most = fmaxf(most, ml[k][0]);
            const float base = most == -INFINITY ? 0.f : most, f0 = __builtin_amdgcn_exp2f(m - base);
            m = most;
            l *= f0;
#pragma unroll
            for (int c = 0; c < DQ; ++c) o[c] *= f0;
#pragma unroll
            for (int k = 0; k < kJoinAhead; ++k)
                if (p0 + k * WAVES < sp.parts) {
                    const float f = __builtin_amdgcn_exp2f(ml[k][0] - base);
                    l += ml[k][1] * f;
#pragma unroll
                    for (int c = 0; c < DQ; ++c) o[c] += x[k][c] * f;
                }
        }
        if (WAVES > 1 && lane == 0) top[row][wave] = m;
        if (WAVES > 1) {
            __syncthreads();
            float most = top[row][0];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) most = fmaxf(most, top[row][w]);
            const float f = __builtin_amdgcn_exp2f(m - (most == -INFINITY ? 0.f : most));
            m = most;
            l *= f;
#pragma unroll
            for (int c = 0; c < DQ; ++c) o[c] *= f;
        }
        if (lane == 0) sum[row][wave] = l;
#pragma unroll
        for (int c = 0; c < DQ; ++c) joined[row][wave][64 * c + lane] = o[c];
        __syncthreads();
        if (!mine) continue;
        l = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) l += sum[row][w];
        const int j = token_of(a, r), qh = head * a.group + (r - j * a.group);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t token = sp.row0 + j;
        const int first = (threadIdx.x % (64 * WAVES)) * 2;
        for (int d = first; d < D; d += 128 * WAVES) {
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                x0 += joined[row][w][d];
                x1 += joined[row][w][d + 1];
            }
            *reinterpret_cast<uint32_t*>(a.out + token * a.out_stride + int64_t(qh) * D + d) = pack_bf16(x0 * inv, x1 * inv);
        }
        if (first == 0 && a.lse) a.lse[token * (a.n_kv * a.group) + qh] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    }
}

// How a call is laid out; the same for the workspace's size and the launch.
struct Plan {
    int32_t group, nt, waves, row_tiles, places, unit;
    bool split;
    int64_t longest;         // parts of a request at most
    uint64_t parts;          // partial results of a head, of nt * 16 rows
    uint64_t splits;         // row tiles that they can come from
    uint64_t bytes;
};

// Workgroups of a head that the chip holds.
static int places_of(const mbd_kv_cache* c, int nt, int waves) {
    return std::max(1, kCus * per_cu(c->head_dim / 64, nt) * kMaxWaves / waves / c->n_heads);
}

// The parts and their memory, for tiles of p->nt * 16 query rows and parts of p->waves waves.
static void lay_out(const mbd_kv_cache* c, int64_t tiles, int64_t seq_tiles, Plan* p) {
    p->places = places_of(c, p->nt, p->waves);
    // tiles of a part: a step a wave (with two, three: one request of 2048 tokens 11.4, 12.7 us against
    // 10.2, a verify step of 8 x 5 13.5, 13.5 against 13.9, 8 of up to 4096 13.4, 13.7 against 13.9)
    const int64_t least = p->waves * kStep;
    p->longest = (seq_tiles + least - 1) / least;
    p->split = p->longest > 1 && p->places > 1;
    p->parts = p->split ? std::min<int64_t>(2 * p->places, tiles * p->longest) : 0;
    p->splits = std::min<int64_t>(p->parts / 2, tiles);
    p->bytes = p->parts * c->n_heads * (16u * p->nt) * (c->head_dim + 2) * sizeof(float) + p->splits * sizeof(Split);
}

static mbd_status plan_of(const mbd_kv_cache* c, int32_t n_heads, int32_t n_seqs, int32_t max_new, int32_t max_blocks, Plan* p) {
    if (n_heads < 1 || n_heads % c->n_heads) return fail(MBD_ESHAPE, "n_heads %d is not a multiple of the cache's %d", n_heads, c->n_heads);
    if (n_seqs < 1 || n_seqs > kMaxSeqs) return fail(MBD_ESHAPE, "n_seqs %d outside [1, %d]", n_seqs, kMaxSeqs);
    if (max_blocks < 1 || int64_t(max_blocks) * c->block_size > (int64_t(1) << 30))
        return fail(MBD_ESHAPE, "max_blocks * block_size outside [1, 2^30]");
    const int64_t seq_tiles = int64_t(max_blocks) * (c->block_size / kTok);
    if (seq_tiles * n_seqs >= (int64_t(1) << 31)) return fail(MBD_ESHAPE, "n_seqs * max_blocks * block_size / 16 is 2^31 or more");
    p->group = n_heads / c->n_heads;
    if (p->group > 256) return fail(MBD_ESHAPE, "%d query heads a KV head, more than 256", p->group);
    if (max_new < 1 || int64_t(max_new) * p->group >= (int64_t(1) << 24)) return fail(MBD_ESHAPE, "max_new * query heads a KV head outside [1, 2^24)");
    const int32_t rows = max_new * p->group;
    p->nt = rows <= 16 ? 1 : 2;
    p->row_tiles = (rows + 16 * p->nt - 1) / (16 * p->nt);
    const int64_t tiles = int64_t(n_seqs) * p->row_tiles;                  // of query rows
    if (tiles > (int64_t(1) << 28)) return fail(MBD_ESHAPE, "n_seqs times tiles of max_new tokens' query rows above 2^28");
    p->unit = 0;
    while (((seq_tiles * p->row_tiles) >> p->unit) + 1 >= (int64_t(1) << 31) / n_seqs) ++p->unit;
    p->waves = p->nt == 1 && tiles > places_of(c, 1, kMaxWaves) ? 1 : kMaxWaves;
    lay_out(c, tiles, seq_tiles, p);
    return MBD_OK;
}

// The workspace that this call and every one with fewer requests, tokens or blocks needs: up to
// 16 query rows parts are of one wave or of four, above that of two row tiles, and the places,
// which bound the partial results, are most numerous where the rows are few.
static uint64_t largest_workspace(const mbd_kv_cache* c, int32_t n_seqs, int32_t max_blocks, const Plan& own) {
    const int64_t seq_tiles = int64_t(max_blocks) * (c->block_size / kTok);
    uint64_t bytes = own.bytes;
    if (own.group > 16) return bytes;          // a single token has two row tiles
    Plan p{};
    p.nt = 1;
    for (int waves : {kMaxWaves, 1}) {
        const int64_t fours = places_of(c, 1, kMaxWaves);
        if (waves == 1 && n_seqs <= fours) break;
        p.waves = waves;
        lay_out(c, waves == 1 ? n_seqs : std::min<int64_t>(n_seqs, fours), seq_tiles, &p);
        bytes = std::max(bytes, p.bytes);
    }
    return bytes;
}

template <bool E4M3, int DQ, int NT, int WAVES>
static void launch(const AttnArgs& a, const Plan& p, int64_t items, bool ext, hipStream_t s) {
    const dim3 grid(unsigned(items) * unsigned(a.n_kv)), block(64 * WAVES);
    if (ext) hipLaunchKernelGGL((attn_kernel<E4M3, DQ, NT, true, WAVES>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attn_kernel<E4M3, DQ, NT, false, WAVES>), grid, block, 0, s, a);
    if (a.n_splits) {
        const int rows = std::min(16 * NT, a.max_new * a.group);
        // (at most four workgroups a tile: where few tiles are split, most find nothing to do)
        const dim3 joins(unsigned(a.n_splits), unsigned(a.n_kv), unsigned(std::min((rows + kJoinRows - 1) / kJoinRows, 4)));
        // few row tiles can have many parts each: more waves over them (four against one, one request of
        // 131072 tokens 58.8 and 69.3 us, 8 of up to 4096 13.9 and 14.8, one of 500 10.0 and 8.9; with more row
        // tiles, 32 of up to 8192 54.9 and 53.7, a verify step of 8 x 5 15.3 and 14.2)
        if (a.n_seqs * int64_t(p.row_tiles) * 8 < p.places)
            hipLaunchKernelGGL((join_kernel<DQ, 4>), joins, dim3(64 * kJoinRows * 4), 0, s, a, 16 * NT);
        else
            hipLaunchKernelGGL((join_kernel<DQ, 1>), joins, dim3(64 * kJoinRows), 0, s, a, 16 * NT);
    }
}

template <bool E4M3, int DQ>
static void launch_rows(const AttnArgs& a, const Plan& p, int64_t items, bool ext, hipStream_t s) {
    if (p.nt == 2) launch<E4M3, DQ, 2, 4>(a, p, items, ext, s);
    else if (p.waves == 4) launch<E4M3, DQ, 1, 4>(a, p, items, ext, s);
    else launch<E4M3, DQ, 1, 1>(a, p, items, ext, s);
}

template <bool E4M3>
static void launch_dim(const AttnArgs& a, const Plan& p, int64_t items, int dq, bool ext, hipStream_t s) {
    if (dq == 1) launch_rows<E4M3, 1>(a, p, items, ext, s);
    else if (dq == 2) launch_rows<E4M3, 2>(a, p, items, ext, s);
    else if (dq == 3) launch_rows<E4M3, 3>(a, p, items, ext, s);
    else launch_rows<E4M3, 4>(a, p, items, ext, s);
}

}  // namespace kv
}  // namespace mbd

using namespace mbd;

extern "C" {

mbd_status mbd_kv_attn_workspace_bytes(const mbd_kv_cache* cache, int32_t n_heads, int32_t n_seqs, int32_t max_new,
                                       int32_t max_blocks, uint64_t* bytes) {
    if (!bytes) return fail(MBD_EINVAL, "NULL argument");
    kv::Plan p;
    mbd_status st = kv::check_cache(cache, false);
    if (st == MBD_OK) st = kv::plan_of(cache, n_heads, n_seqs, max_new, max_blocks, &p);
    if (st == MBD_OK) *bytes = kv::largest_workspace(cache, n_seqs, max_blocks, p);
    return st;
}

mbd_status mbd_kv_attn(const mbd_kv_cache* cache, const mbd_kv_attn_args* args, const uint16_t* q, const int32_t* seq_start,
                       const int32_t* lens, const int32_t* block_table, uint16_t* out, float* lse, void* ws, uint64_t ws_bytes,
                       void* stream) {
    hip_clear();
    kv::Plan p;
    mbd_status st = kv::check_cache(cache, true);
    if (st != MBD_OK) return st;
    if (!args) return fail(MBD_EINVAL, "NULL argument");
    st = kv::plan_of(cache, args->n_heads, args->n_seqs, args->max_new, args->max_blocks, &p);
    if (st != MBD_OK) return st;
    if (args->T < 0 || args->T > (1 << 24)) return fail(MBD_ESHAPE, "T %d outside [0, 2^24]", args->T);
    if (args->window < 0) return fail(MBD_EINVAL, "window %d below 0", args->window);
    if (!(std::fabs(args->scale) <= 0x1p64f)) return fail(MBD_EINVAL, "scale outside [-2^64, 2^64]");
    if (args->softcap != 0 && !(args->softcap >= 0x1p-64f && args->softcap <= 0x1p64f))
        return fail(MBD_EINVAL, "softcap is neither 0 nor in [2^-64, 2^64]");
    if (args->softcap > 0 && std::fabs(args->scale) / double(args->softcap) > 0x1p126)
        return fail(MBD_EINVAL, "|scale| / softcap above 2^126");
    const int64_t row = int64_t(args->n_heads) * cache->head_dim;
    if (args->q_stride < row || args->out_stride < row || args->q_stride % 8 || args->out_stride % 8)
        return fail(MBD_ESHAPE, "row strides must be multiples of 8 and at least n_heads * head_dim");
    if (!seq_start || !lens || !block_table) return fail(MBD_EINVAL, "NULL argument");
    if (!kv::aligned(seq_start, 4) || !kv::aligned(lens, 4) || !kv::aligned(block_table, 4) || !kv::aligned(lse, 4) ||
        !kv::aligned(args->slopes, 4))
        return fail(MBD_EALIGN, "int32 and fp32 arrays must be 4-byte aligned");
    // a head's items: places, and the row tiles that the sums may pass them by; T bounds those
    const int64_t used = std::min<int64_t>(int64_t(args->n_seqs) * p.row_tiles, int64_t(args->T) * p.group / (16 * p.nt) + args->n_seqs);
    const int64_t items = p.split ? std::min(p.places + used, used * p.longest) : used;
    if (items * cache->n_heads >= (int64_t(1) << 24)) return fail(MBD_ESHAPE, "KV heads times tiles of query rows is 2^24 or more");
    if (args->T == 0) return MBD_OK;
    if (!q || !out) return fail(MBD_EINVAL, "NULL argument");
    if (!kv::aligned(q, 16) || !kv::aligned(out, 16)) return fail(MBD_EALIGN, "q and out must be 16-byte aligned");
    if (p.bytes) {
        if (!ws || ws_bytes < p.bytes) return fail(MBD_EINVAL, "workspace of %llu bytes needed", static_cast<unsigned long long>(p.bytes));
        if (!kv::aligned(ws, 16)) return fail(MBD_EALIGN, "workspace must be 16-byte aligned");
    }
    kv::AttnArgs a{};
    a.k = static_cast<const uint8_t*>(cache->k_codes);
    a.v = static_cast<const uint8_t*>(cache->v_codes);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.q = q;
    a.seq_start = seq_start;
    a.lens = lens;
    a.table = block_table;
    a.out = out;
    a.lse = lse;
    a.part_o = static_cast<float*>(ws);
    a.part_ml = a.part_o + p.parts * cache->n_heads * (16u * p.nt) * cache->head_dim;
    a.splits = reinterpret_cast<kv::Split*>(a.part_ml + p.parts * cache->n_heads * (16u * p.nt) * 2);
    a.slopes = args->slopes;
    a.q_stride = args->q_stride;
    a.out_stride = args->out_stride;
    a.n_blocks = int32_t(cache->n_blocks);
    a.n_seqs = args->n_seqs;
    a.max_blocks = args->max_blocks;
    a.T = args->T;
    a.max_new = args->max_new;
    a.window = args->window < args->max_blocks * cache->block_size ? args->window : 0;   // else it hides nothing
    a.shift = kv::log2_of(cache->block_size);
    a.n_kv = cache->n_heads;
    a.group = p.group;
    a.per_group = uint32_t(((uint64_t(1) << 32) + p.group - 1) / p.group);
    a.row_shift = p.nt == 1 ? 4 : 5;
    a.min_part = p.waves * kv::kStep;
    a.places = p.places;
    a.unit = p.unit;
    a.n_splits = int32_t(std::min<int64_t>(p.splits, used));
    a.n_parts = int32_t(p.parts);
    a.split = p.split;
    a.to_score = args->softcap > 0 ? args->scale / args->softcap : kv::kLog2e * args->scale;
    // (the margin is for this rounding and the product's)
    const float most = float(double(FLT_MAX) * (1 - 0x1p-22) / std::max(double(std::fabs(a.to_score)), 1.0));
    a.most_ks = __builtin_bit_cast(int32_t, most);
    a.softcap = args->softcap * kv::kLog2e;
    const bool ext = a.window > 0 || args->softcap > 0 || args->slopes;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    if (cache->fmt == MBD_KV_E4M3) kv::launch_dim<true>(a, p, items, cache->head_dim / 64, ext, s);
    else kv::launch_dim<false>(a, p, items, cache->head_dim / 64, ext, s);
    return hip_check("attention launch");
}

}  // extern "C"
