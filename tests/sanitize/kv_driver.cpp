// Host-only driver of the KV-cache calls for an AddressSanitizer + UndefinedBehavior-
// Sanitizer build of their HIP sources' host passes: every call fails validation or has
// nothing to do, so no device work is enqueued and the fake pointers are never
// dereferenced.  Exit status 0 and no sanitizer report is the pass condition.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "mbd.h"

namespace {

int failures = 0;

void expect(mbd_status got, mbd_status want, const char* what) {
    if (got != want) {
        std::fprintf(stderr, "FAILED: %s: status %d, expected %d (%s)\n", what, int(got), int(want), mbd_last_error());
        ++failures;
    }
}

void* fake(uintptr_t a) { return reinterpret_cast<void*>(a); }

mbd_kv_cache cache() {
    return mbd_kv_cache{MBD_KV_INT8, 16, 2, 128, 8, fake(0x1000), fake(0x1000), static_cast<float*>(fake(0x1000)), static_cast<float*>(fake(0x1000))};
}

mbd_kv_attn_args args() { return mbd_kv_attn_args{8, 2, 4, 2, 1, 0, 0.1f, 0.f, nullptr, 1024, 1024}; }

void sizes() {
    // the extremes that the plan's products and shifts meet
    uint64_t bytes = 0;
    for (int32_t dim : {64, 128, 192, 256})
        for (int32_t heads : {1, 2, 65535})
            for (int32_t seqs : {1, 7, 4096})
                for (int32_t fresh : {1, 2, 1 << 10, (1 << 24) - 1, INT32_MAX})
                    for (int32_t blocks : {1, 4097, 1 << 22, 1 << 26, INT32_MAX}) {
                        mbd_kv_cache c = cache();
                        c.head_dim = dim;
                        c.n_heads = heads;
                        const mbd_status st = mbd_kv_attn_workspace_bytes(&c, heads, seqs, fresh, blocks, &bytes);
                        if (st != MBD_OK && st != MBD_ESHAPE) expect(st, MBD_OK, "workspace size");
                        if (st == MBD_OK && bytes > (uint64_t(1) << 32)) expect(MBD_ERANGE, MBD_OK, "workspace below 4 GiB");
                        mbd_kv_attn_args a = args();
                        a.n_heads = heads;
                        a.n_seqs = seqs;
                        a.max_new = fresh;
                        a.max_blocks = blocks;
                        a.q_stride = a.out_stride = int64_t(heads) * dim;
                        a.T = 0;                                    // reaches the layout of the launch, enqueues nothing
                        const mbd_status run = mbd_kv_attn(&c, &a, nullptr, static_cast<int32_t*>(fake(16)), static_cast<int32_t*>(fake(16)),
                                                           static_cast<int32_t*>(fake(16)), nullptr, nullptr, nullptr, 0, nullptr);
                        if (run != MBD_OK && run != MBD_ESHAPE) expect(run, MBD_OK, "empty attention");
                    }
}

void refusals() {
    auto* i = static_cast<int32_t*>(fake(0x2000));
    auto* q = static_cast<uint16_t*>(fake(0x2000));
    mbd_kv_cache c = cache();
    mbd_kv_attn_args a = args();
    uint64_t bytes = 0;
    expect(mbd_kv_attn_workspace_bytes(nullptr, 8, 2, 1, 4, &bytes), MBD_EINVAL, "workspace of no cache");
    expect(mbd_kv_attn_workspace_bytes(&c, 8, 2, 1, 4, nullptr), MBD_EINVAL, "workspace to nowhere");
    expect(mbd_kv_attn(nullptr, &a, q, i, i, i, q, nullptr, nullptr, 0, nullptr), MBD_EINVAL, "no cache");
    expect(mbd_kv_attn(&c, nullptr, q, i, i, i, q, nullptr, nullptr, 0, nullptr), MBD_EINVAL, "no arguments");
    a.max_blocks = 512;                                             // long enough to be cut into parts
    expect(mbd_kv_attn(&c, &a, q, i, i, i, q, nullptr, nullptr, 0, nullptr), MBD_EINVAL, "no workspace");
    a.scale = std::nanf("");
    expect(mbd_kv_attn(&c, &a, q, i, i, i, q, nullptr, nullptr, 0, nullptr), MBD_EINVAL, "scale NaN");
    a = args();
    a.softcap = INFINITY;
    expect(mbd_kv_attn(&c, &a, q, i, i, i, q, nullptr, nullptr, 0, nullptr), MBD_EINVAL, "softcap infinite");
    a = args();
    a.T = INT32_MAX;
    expect(mbd_kv_attn(&c, &a, q, i, i, i, q, nullptr, nullptr, 0, nullptr), MBD_ESHAPE, "too many rows");
    c.n_blocks = INT64_MAX;
    expect(mbd_kv_append(&c, q, q, MBD_BF16, 256, 256, i, 1, nullptr), MBD_ESHAPE, "too many blocks");
    c = cache();
    expect(mbd_kv_append(&c, q, q, MBD_BF16, INT64_MIN, 256, i, 1, nullptr), MBD_ESHAPE, "negative stride");
    expect(mbd_kv_append(&c, q, q, MBD_BF16, 256, INT64_MAX, i, 1, nullptr), MBD_ESHAPE, "odd stride");
    expect(mbd_kv_append(&c, q, q, 0, 256, 256, i, 1, nullptr), MBD_EINVAL, "no type");
    expect(mbd_kv_append(&c, q, q, MBD_F32, 256, 256, i, 0, nullptr), MBD_OK, "nothing to append");
    expect(mbd_kv_gather(&c, i, INT32_MAX, MBD_F32, q, q, nullptr), MBD_ESHAPE, "too many tokens");
    expect(mbd_kv_gather(&c, i, 0, MBD_F32, nullptr, nullptr, nullptr), MBD_OK, "nothing to read");
    mbd_kv_pool pool{4, 16, INT32_MAX, 100, i, i};
    expect(mbd_kv_slots(&pool, i, i, i, i, 4, i, i, i, i, i, i, i, nullptr), MBD_ESHAPE, "table too wide");
    pool.max_blocks = 8;
    pool.n_blocks = INT32_MAX;
    expect(mbd_kv_slots(&pool, i, i, i, i, 4, i, i, i, i, i, i, i, nullptr), MBD_ESHAPE, "pool too large");
    pool.n_blocks = 100;
    expect(mbd_kv_slots(&pool, i, i, i, i, INT32_MIN, i, i, i, i, i, i, i, nullptr), MBD_ESHAPE, "negative rows");
    expect(mbd_kv_slots(&pool, i, i, nullptr, i, 4, i, i, i, i, i, i, i, nullptr), MBD_EINVAL, "no held blocks");
    expect(mbd_kv_slots(&pool, i, i, i, i, 4, i, static_cast<int32_t*>(fake(0x2002)), i, i, i, i, i, nullptr), MBD_EALIGN, "odd slots");
}

}  // namespace

int main() {
    sizes();
    refusals();
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
