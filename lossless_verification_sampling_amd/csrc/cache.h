// cache.h -- the paged key/value cache: layout, checks and conversions shared
// by the kernels that write, read, attend over and move its rows (internal).
#pragma once

#include "common.h"

namespace sv {

constexpr float kE4m3Max = 448.0f;                 // largest finite e4m3 value
constexpr float kMinScale = 1.17549435e-38f;       // 2^-126, so that x / scale is finite

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
// (vector types of the language, not the runtime's structs: arrays of those
// end up in scratch memory)
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// One layer's pages.  Token t of request r: page table[r * max_pages + (t >>
// shift)], offset t & (size - 1); the row of head h starts at element
// ((page * heads + h) * size + offset) * D.
struct Pages {
    void *k, *v;             // [num_pages][heads][size][D]
    float *k_scale, *v_scale;  // [num_pages][heads][size] (e4m3 only)
    const int32_t *table;    // [R][max_pages]
    int num_pages, max_pages, heads, size, shift;
};

// The two halves of a 32-bit word as bf16, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    f32x2_t v;
    v.x = lo;
    v.y = hi;
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}
// Four fp32 values (|x| <= 448) as e4m3 codes, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
// Two e4m3 codes (the low or the high half of w) as packed bf16: exact.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3_bf16(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// Whether count tokens from first lie inside the page table, and far enough
// below 2^31 for token numbers a few steps ahead to be 32-bit ones.
__device__ __forceinline__ bool in_table(int first, int count, int max_pages, int shift) {
    return first >= 0 && count >= 0 &&
           (int64_t)first + count <= min((int64_t)max_pages << shift, (int64_t)0x7ffff000);
}

// Workgroups of kBlock threads along one axis of a launch: threads count in 32 bits.
constexpr int64_t kMaxBlocks = (1ll << 32) / kBlock - 1;

// Host checks of a cache's arguments that every entry point shares; 0 or a
// negative spec_status.  (A missing page table is looked for once it is known
// that the call has anything to do.)
inline int check_pages(const void *k, const void *v, int dtype, const float *ks, const float *vs,
                       int num_pages, int page_size, int max_pages, int Hkv, int D) {
    if (num_pages < 1 || max_pages < 0 || Hkv < 1 || D < 1 || page_size < 1) return SPEC_EINVAL;
    if (dtype != SPEC_BF16 && dtype != SPEC_E4M3) return SPEC_EDTYPE;
    if (D != 64 && D != 128 && D != 256) return SPEC_EUNSUPPORTED;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return SPEC_EUNSUPPORTED;
    if (!k || !v) return SPEC_EINVAL;
    if (dtype == SPEC_E4M3 && (!ks || !vs)) return SPEC_EINVAL;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)ks | (uintptr_t)vs) & 15u) return SPEC_EINVAL;
    return SPEC_OK;
}

inline Pages make_pages(const void *k, const void *v, const float *ks, const float *vs,
                        int num_pages, int page_size, const int32_t *table, int max_pages,
                        int Hkv) {
    Pages c{};
    c.k = const_cast<void *>(k);
    c.v = const_cast<void *>(v);
    c.k_scale = const_cast<float *>(ks);
    c.v_scale = const_cast<float *>(vs);
    c.table = table;
    c.num_pages = num_pages;
    c.max_pages = max_pages;
    c.heads = Hkv;
    c.size = page_size;
    c.shift = __builtin_ctz((unsigned)page_size);
    return c;
}

inline bool bad_workspace(const void *ws, size_t bytes, size_t need) {
    return !ws || ((uintptr_t)ws & 255u) || bytes < need;
}

}  // namespace sv
