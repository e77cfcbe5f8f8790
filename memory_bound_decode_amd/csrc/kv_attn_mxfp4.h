// Attention over the 4-bit KV cache (MBD_KV_MXFP4): the products of kv_attn.hip,
//   S^T [tokens][rows] = K [tokens][d] Q^T,  O^T [d][rows] += V^T [d][tokens] P^T
// on bf16 matrix instructions, with the same sharing of the work.
//
// Keys: a lane holds 32 channels of one token, which is a group with one exponent; v_cvt_scalef32_pk_bf16_fp4 makes
// two of them the exact bf16 values of an operand.  Values: the pairs of a byte are two channels of one token, and the
// sum runs over tokens, whose exponents differ; so the pairs of eight tokens are sorted into operands by
// byte permutes.
//
// (v_mfma_scale_f32_16x16x128_f8f6f4 would take the keys as they are stored, and the queries as the sum of two e4m3.  But
// it cuts products some 17 bits below the largest of a sum, exponents of groups included: scores were off by
// 1e-5 where these are by 1e-7, and that is what a log-sum-exp loses.)
//
// One query row tile and long contexts: bound by HBM, 32 requests of 32768 tokens (64 / 4 heads x 128, 572 MB) in 94 us,
// 6.1 TB/s, and 5 of the join.  Short ones: by the way to the first product (4 us: share, block ids, codes) and the join's
// launch (4 us).  Two row tiles (prompts): by the vector units, two thirds of the time busy, since they unpack for 32
// rows at a time, and the matrix units, a third; 22.5 GFLOP of prompt slices in 55 us.
#pragma once

#include <hip/hip_runtime.h>

#include "kv_attn_share.h"

namespace mbd {
namespace kv {

// Channels 2 B and 2 B + 1 of a word of codes as bf16; of the scale its exponent bits alone count.
template <int B>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, uint32_t scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(scale), B));
}

// Eight channels of a token as an operand.
__device__ __forceinline__ bf16x8 key_operand(uint32_t w, uint32_t scale) {
    return __builtin_bit_cast(bf16x8, u32x4{value_pair<0>(w, scale), value_pair<1>(w, scale), value_pair<2>(w, scale), value_pair<3>(w, scale)});
}

// Token i's byte of a word of four exponents, in the place of an fp32's exponent; what else stays in
// the word has no meaning to value_pair.
__device__ __forceinline__ uint32_t exponent_of(uint32_t w, int i) { return i == 3 ? w >> 1 : w << (23 - 8 * i); }

// Two channels (low and high halves of t[..]) of eight tokens as the operands of two products.
__device__ __forceinline__ void pair_up(const uint32_t (&t)[8], bf16x8* even, bf16x8* odd) {
    u32x4 e, o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x05040100);
        o[i] = __builtin_amdgcn_perm(t[2 * i + 1], t[2 * i], 0x07060302);
    }
    *even = __builtin_bit_cast(bf16x8, e);
    *odd = __builtin_bit_cast(bf16x8, o);
}

// ceil(n / chunk), 0 for 0: exact where the quotient is below 2^20, as a reciprocal's errors then move
// it by less than one.
__device__ __forceinline__ int parts_in(int n, int chunk, float inverse) {
    int q = int(float(n - 1) * inverse);
    const int rest = n - 1 - q * chunk;
    q += rest >= chunk ? 1 : rest < 0 ? -1 : 0;
    return n > 0 ? q + 1 : 0;
}

// find_item for up to 64 requests, one a lane.  The way to a workgroup's first load goes through here, so it
// is kept short: four chunks are tried at once, two counts to a word, and the smallest that fits is
// taken.  (Parts and row tiles add up to about work / chunk + used / 2, so that is where the candidates stand; the
// last always fits.)
// Where there are more items than places, those of the longest parts come first, in four classes: the
// last ones to start then end early.
__device__ __forceinline__ Item find_item_64(const AttnArgs& a, int32_t want, Seq* sq, int* splits) {
    const int lane = threadIdx.x & 63;
    const Seq s = load_seq(a, min(lane, a.n_seqs - 1));
    const int n = lane < a.n_seqs ? tiles_of(s) : 0, rt = n ? row_tiles_of(a, s) : 0;
    auto total = [](int scan) { return __builtin_amdgcn_readlane(scan, 63); };
    auto uniform = [](int v, int l) { return __builtin_amdgcn_readlane(v, l); };
    int chunk = 0x3fffffff;
    float inverse = 0x1p-30f;
    if (a.split) {
        const int units = a.unit ? int((uint64_t(uint32_t(n)) * uint32_t(rt) + (uint64_t(1) << a.unit) - 1) >> a.unit) : n * rt;
        const int work = max(total(wave_scan(units)), 1), used = total(wave_scan(rt));
        // lane k's candidate: at least work / room, as the reciprocal's and the roundings' errors are below 2^-21
        const int eighths = lane == 0 ? 3 : lane == 1 ? 4 : lane == 2 ? 5 : 8;
        const int room = used < a.places ? a.places - (eighths * used + 7) / 8 : (a.places + 1) / 2;
        const uint32_t share = uint32_t(float(work) * __builtin_amdgcn_rcpf(float(room)) * (1 + 0x1p-20f)) + 1;
        const int mine = int(min(max(uint64_t(share) << a.unit, uint64_t(a.min_part)), uint64_t(1) << 30));     // (no request has as many)
        const float one_over = __builtin_amdgcn_rcpf(float(mine));
        int best = 3;
        if (used < a.places) {
            uint32_t count[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                auto items = [&](int t) { return parts_in(n, uniform(mine, t), __int_as_float(uniform(__float_as_int(one_over), t))) * rt; };
                count[k] = wave_scan(items(2 * k) | items(2 * k + 1) << 16);     // below 2^14 each: up to room + used
            }
            const int last = total(count[1]), first = total(count[0]);
            best = (first & 0xffff) <= a.places ? 0 : (first >> 16) <= a.places ? 1 : (last & 0xffff) <= a.places ? 2 : 3;
        }
        chunk = uniform(mine, best);
        inverse = __int_as_float(uniform(__float_as_int(one_over), best));
    }
    const int p = parts_in(n, chunk, inverse);
    const int mine = p * rt, my_slots = p > 1 ? mine : 0, my_cuts = p > 1 ? rt : 0;
    int end = wave_scan(mine);
    const int slots_end = wave_scan(my_slots), cuts_end = wave_scan(my_cuts);
    *splits = total(cuts_end);
    if (total(end) > a.places) {
        const int length = p > 0 ? int(float(n) * __builtin_amdgcn_rcpf(float(p))) : 0;
        float longest = lane_max(float(length));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) longest = fmaxf(longest, __shfl_xor(longest, d));
        const int four = 4 * length, most = int(longest), kind = four > 3 * most ? 0 : four > 2 * most ? 1 : four > most ? 2 : 3;
        int before = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int in = wave_scan(kind == k ? mine : 0);
            if (kind == k) end = before + in;
            before += total(in);
        }
    }
    const uint64_t who = __ballot(want >= end - mine && want < end);
    if (!who) return {-1, 0, 0, 0, 0};
    const int l = __builtin_ctzll(who);
    auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
    *sq = {of(s.row0), of(s.n_new), of(s.rows), of(s.p0), of(s.lo), of(s.hi), of(s.len)};
    return {l, of(p), want - of(end - mine), of(slots_end - my_slots), of(cuts_end - my_cuts)};
}

// What a workgroup does, from the wave that found out.
struct Share {
    Item it;
    Seq sq;
    int32_t splits;
    __device__ __forceinline__ void read(const Share& from) {      // into scalar registers
        constexpr int words = sizeof(Share) / 4;
        static_assert(words <= 64, "a word a lane");
        const int32_t mine = reinterpret_cast<const int32_t*>(&from)[min(int(threadIdx.x & 63), words - 1)];
        int32_t all[words];
#pragma unroll
        for (int i = 0; i < words; ++i) all[i] = __builtin_amdgcn_readlane(mine, i);
        *this = __builtin_bit_cast(Share, all);
    }
};

// (NaN if one is: fmaxf spends an instruction on each operand for those that are signalling)
__device__ __forceinline__ float max3(float a, float b, float c) { return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c); }

// DQ = head_dim / 64, NT = tiles of 16 query rows, EXT: cap, window, distance bias, or a factor of scores
// near 0; WAVES: of a part (as attn_kernel).  DIRECT: a workgroup takes a whole request, its own number, of one row
// tile: nothing to look for, nothing to join.
template <int DQ, int NT, bool EXT, int WAVES, bool DIRECT>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(WAVES == 16 ? 4 : per_cu(DQ, NT)))) void attn4_kernel(AttnArgs a) {
    constexpr int D = 64 * DQ, ROWS = 16 * NT, F = DQ / 2, H = DQ % 2, S = F + H;   // slabs of 128 channels, of 64
    // The waves' sums are joined in LDS, of one row tile all at once, of two 64 channels at a time.  Pitch: rows 4 banks apart.
    constexpr int SLABS = NT == 1 ? DQ : 1, PITCH = 64 * SLABS + 4;
    __shared__ float merge[WAVES][ROWS][PITCH];
    __shared__ float merge_m[WAVES][ROWS], merge_l[WAVES][ROWS];
    __shared__ Share share;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, n = lane & 15;
    const int in_block = (1 << a.shift) - 1;
    const int want = blockIdx.x / uint32_t(a.n_kv), head = blockIdx.x - want * a.n_kv;
    // One wave looks for the workgroup's share (some hundred operations: in every wave at once they kept the
    // vector units busy for the longer part of the start); not always the same, whose SIMD would have it all.
    Share sh;
    if (DIRECT) {
        sh = {{want, 1, 0, 0, 0}, load_seq(a, want), 0};
        if (sh.sq.n_new < 1) return;
    } else if (WAVES == 1 || wave == int(blockIdx.x / kCus % WAVES)) {
        sh.it = a.n_seqs <= 64 ? find_item_64(a, want, &sh.sq, &sh.splits) : find_item(a, want, &sh.sq, &sh.splits);
        if (WAVES > 1 && lane == 0) share = sh;
    }
    if (WAVES > 1 && !DIRECT) {
        __syncthreads();
        sh.read(share);
    }
    const Item it = sh.it;
    const Seq sq = sh.sq;
    const int splits = sh.splits;
    if (!DIRECT && head == 0 && threadIdx.x == 0 && want >= splits && want < a.n_splits) a.splits[want] = Split{0, 0, 0, 0, 0, 0};
    if (it.seq < 0) return;
    const int row_tiles = DIRECT ? 1 : row_tiles_of(a, sq), part = DIRECT ? 0 : it.index / row_tiles;
    const int row_tile = row_tiles - 1 - (it.index - part * row_tiles);       // the last rows, which see most, first
    const int r0 = row_tile * ROWS, slot = it.slot + row_tile;
    const int rows = min(ROWS, sq.rows - r0);
    // what the first and the last row see bounds what any row sees
    const int pos_first = sq.p0 + token_of(a, r0), pos_last = sq.p0 + token_of(a, r0 + rows - 1);
    const int all_end = pos_first + 1, all_begin = a.window > 0 ? max(pos_last, 0) - a.window + 1 : 0;
    int t0 = sq.lo, t1 = min(sq.hi, (max(pos_last + 1, 0) + kTok - 1) / kTok);
    if (!DIRECT && it.parts > 1) {
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

    // Lane (g, n) holds row n's channels 32 g .. +32 of a slab of 128, four operands; of one of 64 the 16 from 32 (g % 2) +
    // 16 (g / 2) on, two.  Two row tiles' lie in LDS, in the lanes' order.  Rows past the last repeat its
    // queries (where masks are applied they see nothing); nothing of them is kept.
    constexpr bool kQueryLds = NT > 1, kLean = EXT || DQ > 2;
    __shared__ u32x4 queries[kQueryLds ? NT * 2 * DQ : 1][64];
    u32x4 held[kQueryLds ? 1 : 2 * DQ];
    int pos[NT];
    float slope[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int r = min(r0 + 16 * t + n, sq.rows - 1), j = token_of(a, r), qh = head * a.group + (r - j * a.group);
        pos[t] = r0 + 16 * t + n < sq.rows ? sq.p0 + j : -1;
        slope[t] = EXT && a.slopes ? a.slopes[qh] * kLog2e : 0.f;
        const uint16_t* row = a.q + int64_t(sq.row0 + j) * a.q_stride + int64_t(qh) * D;
#pragma unroll
        for (int c = 0; c < 2 * DQ; ++c) {
            if (kQueryLds && c % WAVES != wave) continue;
            const int d = c < 4 * F ? c / 4 * 128 + 32 * g + c % 4 * 8 : F * 128 + g % 2 * 32 + g / 2 * 16 + c % 4 * 8;
            const u32x4 w = *reinterpret_cast<const u32x4*>(row + d);
            if constexpr (kQueryLds) queries[t * 2 * DQ + c][lane] = w ^ a.flip;
            else held[c] = w;
        }
    }
    auto query = [&](int t, int c) {
        if constexpr (kQueryLds) return __builtin_bit_cast(bf16x8, queries[t * 2 * DQ + c][lane]);
        else return __builtin_bit_cast(bf16x8, held[c]);
    };

    // The first step's codes are on their way while the queries come.
    int32_t my_id = -1;
    u32x4 kc[kStep][S], vc[kStep][S];    // one step's codes (of a half slab two words)
    uint32_t ks[kStep][S], vs[kStep][S]; // and exponents: of the lane's key, of four tokens' values
    auto tile_at = [&](int tile, int l) {
        const int32_t id = max(__builtin_amdgcn_readlane(my_id, l), 0);
        return ((int64_t(id) * a.n_kv + head) << (a.shift - 4)) + (((tile * kTok) & in_block) >> 4);
    };
    // A wave's base and a lane's offset of 32 bits are the loads' own address form; the empty asms keep the
    // compiler from widening the offsets ahead of the loop (five registers, and two operations a load).
    const uint32_t lane16 = lane * 16, lane8 = lane * 8, key8 = lane % 32 * 16 + lane / 32 * 8;
    const uint32_t scales_at = n / 4 * 16 + 4 * g, half_scales_at = n / 8 * 16 + 4 * g;
    auto here = [](uint32_t off) {
        asm("" : "+v"(off));
        return off;
    };
    // one tile of query rows is all there is: the codes are read once and streamed; with several, the
    // other tiles find them in L2
    auto read = [&](auto* from) { return NT == 1 ? __builtin_nontemporal_load(from) : *from; };
    auto load_keys = [&](int tile, int l) {
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
            const int64_t at = tile_at(tile + h, l + h);
            const uint8_t *codes = a.k + at * (512 * DQ), *scales = static_cast<const uint8_t*>(a.k_scale) + at * (32 * DQ);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (s < F) {
                    kc[h][s] = read(reinterpret_cast<const u32x4*>(codes + s * 1024 + here(lane16)));
                } else {
                    const u32x2 w = read(reinterpret_cast<const u32x2*>(codes + s * 1024 + here(key8)));
                    kc[h][s] = u32x4{w.x, w.y, 0, 0};
                }
                ks[h][s] = (scales + s * 64)[here(s < F ? uint32_t(lane) : uint32_t(lane % 32))];
            }
        }
    };
    auto load_values = [&](int tile, int l) {
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
            const int64_t at = tile_at(tile + h, l + h);
            const uint8_t *codes = a.v + at * (512 * DQ), *scales = static_cast<const uint8_t*>(a.v_scale) + at * (32 * DQ);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (s < F) {
                    vc[h][s] = read(reinterpret_cast<const u32x4*>(codes + s * 1024 + here(lane16)));
                } else {
                    const u32x2 w = read(reinterpret_cast<const u32x2*>(codes + s * 1024 + here(lane8)));
                    vc[h][s] = u32x4{w.x, w.y, 0, 0};
                }
                vs[h][s] = *reinterpret_cast<const uint32_t*>(scales + s * 64 + here(s < F ? scales_at : half_scales_at));
            }
        }
    };

    auto refill = [&](int k0) {
        my_id = next_id >= 0 && next_id < a.n_blocks ? next_id : -1;
        if (k0 < mine) {
            load_keys(tile_of(k0), 0);
            load_values(tile_of(k0), 0);
        }
        next_id = look_up(k0 + kRefill);
    };
    refill(0);

    if constexpr (kQueryLds) __syncthreads();
    else
#pragma unroll
        for (int c = 0; c < 2 * DQ; ++c) held[c] ^= a.flip;

    f32x4 acc[4 * DQ][NT];               // 8 products of a slab of 128 channels, 4 of one of 64
    float top[NT], sum[NT];              // base of the weights (log2 domain); this lane's share of their sum
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        top[t] = -INFINITY;
        sum[t] = 0.f;
#pragma unroll
        for (int c = 0; c < 4 * DQ; ++c) acc[c][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    auto step = [&](int tile, int l, int next_tile, bool more) {
        if (kQueryLds) asm volatile("" ::: "memory");      // the queries are read again in each step
        f32x4 s[kStep][NT];
        bool whole = tile * kTok >= all_begin && (tile + kStep) * kTok <= all_end;
#pragma unroll
        for (int h = 0; h < kStep; ++h) {
            whole = whole && __builtin_amdgcn_readlane(my_id, l + h) >= 0;
#pragma unroll
            for (int t = 0; t < NT; ++t) s[h][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int c = 0; c < S; ++c)
#pragma unroll
            for (int j = 0; j < (c < F ? 4 : 2); ++j) {
                keep_order();
#pragma unroll
                for (int h = 0; h < kStep; ++h) {
                    const bf16x8 kf = key_operand(kc[h][c][j], ks[h][c] << 23);
#pragma unroll
                    for (int t = 0; t < NT; ++t) s[h][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, query(t, 4 * c + j), s[h][t], 0, 0, 0);
                }
            }
        // (the products stay here: behind the loads, old and new codes would be held at once)
#pragma unroll
        for (int h = 0; h < kStep; ++h)
#pragma unroll
            for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(s[h][t]));
        keep_order();
        if (more) load_keys(next_tile, l + kStep);
        keep_order();
        bf16x8 pf[NT], rest[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float u[kStep][4];
            const float away = float(tile * kTok + 4 * g - pos[t]);
#pragma unroll
            for (int h = 0; h < kStep; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x = s[h][t][i];
                    if (EXT) {
                        x *= a.to_score;
                        if (a.softcap > 0.f) x = a.softcap * tanh_of(x);
                        x += slope[t] * (away + float(h * kTok + i));
                    }
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
            float m = lane_max(max3(max3(u[0][0], u[0][1], u[0][2]), max3(u[0][3], u[1][0], u[1][1]), max3(u[1][2], u[1][3], u[1][3])));
            if (!EXT) m *= a.to_score;
            // the base of the weights need not be the maximum, only near it: it moves where a
            // weight would pass 2^8, so most steps leave the sums as they are
            if (__ballot(m > top[t] + 8.f)) {
                m = fmaxf(m, top[t]);
                const float f = __builtin_amdgcn_exp2f(top[t] - (m == -INFINITY ? 0.f : m));
                sum[t] *= f;
#pragma unroll
                for (int c = 0; c < 4 * DQ; ++c) acc[c][t] *= f;
                top[t] = m;
            }
            const float base = top[t] == -INFINITY ? 0.f : top[t];
            float p[kStep][4];
#pragma unroll
            for (int h = 0; h < kStep; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[h][i] = __builtin_amdgcn_exp2f(EXT ? u[h][i] - base : __builtin_fmaf(u[h][i], a.to_score, -base));
                    sum[t] += p[h][i];
                }
            // The matrix unit takes bf16: a weight goes in as the nearest one, and what that leaves of it as a second operand,
            // off by 2^-16 of itself together, so that o is off by its own rounding to bf16 alone (1.65e-3 in the mean; with the
            // first operand alone 1.9e-3 to 2.1e-3, and up to 2^-8 of the weighted |v| where few tokens have the weight).  The
            // first alone and both: 32 requests of 32768 tokens 98.0 and 100 us, of up to 8192 34.3 and 35.2, prompt slices 47.2
            // and 52.8, one prompt of 4000 tokens 184 and 215, of which 20 are the products; put off behind the next two
            // channels' conversions, or with the remainder from a dot product of pairs, they take as long.
            u32x4 w, r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = p[i / 2][i % 2 * 2], y = p[i / 2][i % 2 * 2 + 1];
                w[i] = pack_bf16(x, y);
                r[i] = pack_bf16(x - __uint_as_float(w[i] << 16), y - __uint_as_float(w[i] & 0xffff0000u));
            }
            pf[t] = __builtin_bit_cast(bf16x8, w);
            rest[t] = __builtin_bit_cast(bf16x8, r);
        }
        if (!whole) {
            // tokens that do not exist may have any codes and exponents, and a zero weight does not silence a
            // NaN: 0 * 2^-127 instead
#pragma unroll
            for (int h = 0; h < kStep; ++h) {
                const bool id_ok = __builtin_amdgcn_readlane(my_id, l + h) >= 0;
                const int tok = (tile + h) * kTok + 4 * g;
                const uint32_t live = id_ok ? live_bytes(tok, sq.len) : 0u;
#pragma unroll
                for (int c = 0; c < S; ++c) {
                    vs[h][c] &= live;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (c < F) vc[h][c][i] = id_ok && tok + i < sq.len ? vc[h][c][i] : 0u;
                        else if (i < 2) vc[h][c][i] &= (live >> (16 * i) & 1 ? 0xffffu : 0u) | (live >> (16 * i + 8) & 1 ? 0xffff0000u : 0u);
                    }
                }
            }
        }
#pragma unroll
        for (int c = 0; c < S; ++c) {
            auto exponent = [&](int h, int i) { return exponent_of(vs[h][c], i); };
            auto two = [&](auto byte) {                  // two channels: the products 2 B and 2 B + 1 of the slab
                constexpr int B = decltype(byte)::value;
                keep_order();
                // (where registers are short, the eight exponents are made anew for each two channels)
                if (kLean) asm("" : "+v"(vs[0][c]), "+v"(vs[1][c]));
                uint32_t t8[8];
#pragma unroll
                for (int h = 0; h < kStep; ++h)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        t8[4 * h + i] = c < F ? value_pair<B>(vc[h][c][i], exponent(h, i))
                                              : (i % 2 ? value_pair<(B + 2) % 4>(vc[h][c][i / 2], exponent(h, i)) : value_pair<B>(vc[h][c][i / 2], exponent(h, i)));
                bf16x8 even, odd;
                pair_up(t8, &even, &odd);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[8 * c + 2 * B][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, pf[t], acc[8 * c + 2 * B][t], 0, 0, 0);
                    acc[8 * c + 2 * B + 1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, pf[t], acc[8 * c + 2 * B + 1][t], 0, 0, 0);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    acc[8 * c + 2 * B][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even, rest[t], acc[8 * c + 2 * B][t], 0, 0, 0);
                    acc[8 * c + 2 * B + 1][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd, rest[t], acc[8 * c + 2 * B + 1][t], 0, 0, 0);
                }
            };
            two(Const<0>{});
            two(Const<1>{});
            if (c < F) {
                two(Const<2>{});
                two(Const<3>{});
            }
        }
        keep_order();
        if (more) load_values(next_tile, l + kStep);
    };

    // Of waves that wait alike the oldest goes first, and the youngest workgroup of a CU ended 16% after the oldest.
    // So a wave's priority falls with what it has done: 32 requests of 32768 tokens 107 -> 103.6 us, 32 of up to 8192 38.7
    // -> 38.1, one of 100001 29.6 either way.  (With two row tiles, which are not bound by loads, prompts of an earlier form 62 -> 65.)
    constexpr bool kEven = NT == 1 && !DIRECT;
    const int quarter = max(mine / 4, 1);
    if (kEven) __builtin_amdgcn_s_setprio(3);
    for (int k0 = 0; k0 < mine;) {
        const int end = min(mine - k0, kRefill);
        for (int k = 0; k < end; ++k) {
            if (kEven && k0 + k == quarter) __builtin_amdgcn_s_setprio(2);
            if (kEven && k0 + k == 2 * quarter) __builtin_amdgcn_s_setprio(1);
            if (kEven && k0 + k == 3 * quarter) __builtin_amdgcn_s_setprio(0);
            step(tile_of(k0 + k), kStep * k, tile_of(k0 + k + 1), k + 1 < end);
        }
        k0 += kRefill;
        if (k0 < mine) refill(k0);
    }

    // A row's four channels from d on: final, from their weighted sum, and the row's sum of weights.
    auto put = [&](int r, int d, const f32x4 o, float m, float l) {
        const int j = token_of(a, r0 + r), qh = head * a.group + (r0 + r - j * a.group);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t* to = a.out + int64_t(sq.row0 + j) * a.out_stride + int64_t(qh) * D + d;
        *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
        if (d == 0 && a.lse) a.lse[int64_t(sq.row0 + j) * (a.n_kv * a.group) + qh] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
    };
    // Join the waves: a common maximum a row, then sums four products at a time through LDS.
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
    for (int c0 = 0; c0 < DQ; c0 += SLABS) {
        if (c0) __syncthreads();
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (16 * t + n < rows)
#pragma unroll
                for (int c = c0; c < c0 + SLABS; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)  // register i of product j: channel j of the octet (in a half slab, the four) 4 g + i
                        *reinterpret_cast<f32x4*>(&merge[wave][16 * t + n][64 * (c - c0) + 16 * g + 4 * i]) =
                            f32x4{acc[4 * c][t][i], acc[4 * c + 1][t][i], acc[4 * c + 2][t][i], acc[4 * c + 3][t][i]} * f[t];
        __syncthreads();
        for (int e = threadIdx.x; e < rows * 16 * SLABS; e += 64 * WAVES) {
            const int r = e / (16 * SLABS), at = e % (16 * SLABS), c = c0 + at / 16, unit = at & 15;
            const int d = c < 2 * F ? c / 2 * 128 + unit * 8 + c % 2 * 4 : F * 128 + unit * 4;
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) m = fmaxf(m, merge_m[w][r]);
            const float base = m == -INFINITY ? 0.f : m;
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                l += merge_l[w][r] * __builtin_amdgcn_exp2f(merge_m[w][r] - base);
                o += *reinterpret_cast<const f32x4*>(&merge[w][r][at * 4]);
            }
            if (DIRECT || it.parts == 1) {
                put(r, d, o, m, l);
            } else {
                const int64_t to = ((slot + int64_t(part) * row_tiles) * a.n_kv + head) * ROWS + r;
                *reinterpret_cast<f32x4*>(a.part_o + to * D + d) = o;
                if (d == 0) *reinterpret_cast<f32x2*>(a.part_ml + to * 2) = f32x2{m, l};
            }
        }
    }
}

}  // namespace kv
}  // namespace mbd
