// Host-only driver of the 4-bit cache's calls and of the append with rotation for an
// AddressSanitizer + UndefinedBehaviorSanitizer build of their HIP sources' host passes: every
// call fails validation or has nothing to do, so no device work is enqueued and the fake
// pointers are never dereferenced.  Exit status 0 and no sanitizer report is the pass condition.
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
int32_t* ints() { return static_cast<int32_t*>(fake(0x2000)); }

mbd_kv_cache cache() { return mbd_kv_cache{MBD_KV_MXFP4, 16, 2, 128, 8, fake(0x1000), fake(0x1000), fake(0x1000), fake(0x1000)}; }

mbd_rope rope() {
    return mbd_rope{static_cast<float*>(fake(0x3000)), 64, 128, 0, 8, fake(0x4000), static_cast<uint16_t*>(fake(0x5000)), 1024, 1024};
}

void sizes() {
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
                        mbd_kv_attn_args a{heads, seqs, blocks, 0, fresh, 0, 0.1f, 0.f, nullptr, int64_t(heads) * dim, int64_t(heads) * dim};
                        const mbd_status run = mbd_kv_attn(&c, &a, nullptr, ints(), ints(), ints(), nullptr, nullptr, nullptr, 0, nullptr);
                        if (run != MBD_OK && run != MBD_ESHAPE) expect(run, MBD_OK, "empty attention");
                    }
}

void appends() {
    for (int32_t fmt : {MBD_KV_INT8, MBD_KV_E4M3, MBD_KV_MXFP4}) {
        mbd_kv_cache c = cache();
        c.fmt = fmt;
        auto call = [&](const mbd_rope* r, int32_t T, const int32_t* pos) {
            return mbd_kv_append_rope(&c, r, fake(0x1000), fake(0x1000), MBD_BF16, 256, 256, ints(), pos, T, nullptr);
        };
        mbd_rope r = rope();
        expect(call(nullptr, 1, ints()), MBD_EINVAL, "no rotation");
        expect(call(&r, 0, nullptr), MBD_OK, "no tokens");
        expect(call(&r, 1, nullptr), MBD_EINVAL, "no positions");
        expect(call(&r, INT32_MIN, ints()), MBD_ESHAPE, "T below 0");
        for (int32_t rot : {INT32_MIN, -8, 0, 7, 136, INT32_MAX}) {
            r = rope();
            r.rot_dim = rot;
            expect(call(&r, 1, ints()), MBD_ESHAPE, "rot_dim");
        }
        for (int32_t heads : {INT32_MIN, -1, 65536, INT32_MAX}) {
            r = rope();
            r.n_q_heads = heads;
            expect(call(&r, 1, ints()), MBD_ESHAPE, "n_q_heads");
        }
        for (int64_t stride : {INT64_MIN, int64_t(-8), int64_t(0), int64_t(1023), int64_t(1028)}) {
            r = rope();
            r.q_stride = stride;
            expect(call(&r, 1, ints()), MBD_ESHAPE, "q_stride");
            r = rope();
            r.q_out_stride = stride;
            expect(call(&r, 1, ints()), MBD_ESHAPE, "q_out_stride");
        }
        r = rope();
        r.q_out = static_cast<uint16_t*>(fake(0x4000));
        expect(call(&r, 1, ints()), MBD_EINVAL, "q_out is q");
        r = rope();
        r.table = static_cast<float*>(fake(0x3004));
        expect(call(&r, 1, ints()), MBD_EALIGN, "table alignment");
        expect(mbd_kv_append(&c, fake(0x1000), fake(0x1000), MBD_F32, 256, 256, ints(), 0, nullptr), MBD_OK, "empty append");
        expect(mbd_kv_gather(&c, ints(), 0, MBD_F32, nullptr, nullptr, nullptr), MBD_OK, "empty gather");
        c.block_size = 24;
        expect(call(&r, 1, ints()), MBD_ESHAPE, "block size");
    }
}

}  // namespace

int main() {
    sizes();
    appends();
    if (failures) return 1;
    std::puts("ok");
    return 0;
}
