// The KV cache's addresses and codes, shared by its HIP sources.
#pragma once

#include <hip/hip_runtime.h>

#include "hip_check.h"
#include "mbd_internal.h"

namespace mbd {
namespace kv {

constexpr int kTok = 16;         // tokens of one code tile
constexpr int kMaxSeqs = 4096;   // requests of a call

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

inline bool block_size_ok(int32_t b) { return b == 16 || b == 32 || b == 64 || b == 128 || b == 256; }

inline int log2_of(int32_t b) { return __builtin_ctz(unsigned(b)); }

// Checks shared by every call that takes a cache; device memory is not looked at.
inline mbd_status check_cache(const mbd_kv_cache* c, bool pointers) {
    if (!c) return fail(MBD_EINVAL, "NULL cache");
    if (c->fmt != MBD_KV_INT8 && c->fmt != MBD_KV_E4M3 && c->fmt != MBD_KV_MXFP4) return fail(MBD_EINVAL, "unknown cache format %d", c->fmt);
    if (!block_size_ok(c->block_size)) return fail(MBD_ESHAPE, "block_size %d is not 16, 32, 64, 128 or 256", c->block_size);
    if (c->head_dim < 64 || c->head_dim > 256 || c->head_dim % 64)
        return fail(MBD_ESHAPE, "head_dim %d is not 64, 128, 192 or 256", c->head_dim);
    if (c->n_heads < 1 || c->n_heads > 65535) return fail(MBD_ESHAPE, "n_heads %d outside [1, 65535]", c->n_heads);
    if (c->n_blocks < 1 || c->n_blocks >= (int64_t(1) << 31) / c->block_size)
        return fail(MBD_ESHAPE, "n_blocks * block_size outside [1, 2^31)");
    if (!pointers) return MBD_OK;
    if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return fail(MBD_EINVAL, "NULL cache pointer");
    if ((reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes)) & 15)
        return fail(MBD_EALIGN, "cache codes must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3)
        return fail(MBD_EALIGN, "cache scales must be 4-byte aligned");
    return MBD_OK;
}

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// bf16 nearest even; the compiler's conversion is one v_cvt_pk_bf16_f32 per pair.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// Byte B of a word of codes, as the value it stands for before scaling.
template <bool E4M3, int B>
__device__ __forceinline__ float code_value(uint32_t w) {
    if constexpr (E4M3) return __builtin_amdgcn_cvt_f32_fp8(int(w), B);
    return float(int8_t(w >> (8 * B)));
}

}  // namespace kv
}  // namespace mbd
