// kv_common.cuh -- what the kernels of the quantised key/value cache share:
// the stored format, page lookups and the unit's status word.
//
// A token's key (or value) head of D elements is stored as D codes of 4 or 8
// bits and D / 32 fp16 scales; element d has the value scale[d / 32] * code.
// Codes are offset binary (code + 8, code + 128).  The codes of a row are not
// in dimension order but in the order in which the lanes of a tensor-core
// fragment take them (include/row_norm.h gives both orders), so that a lane's
// share of a row is one run of bytes and every instruction's elements belong
// to one scale group.
#pragma once

#include <type_traits>

#include "rn_common.cuh"
#include "rn_host.h"

namespace rn {

constexpr int kKvGroup = 32;  // elements of one scale

template <int D, int BITS>
struct KvFormat {
    static constexpr int kGroups = D / kKvGroup;      // scales of a row
    static constexpr int kRow = D * BITS / 8;         // bytes of a row's codes
    static constexpr int kQ = BITS == 4 ? 7 : 127;    // largest code
    static constexpr int kZero = BITS == 4 ? 8 : 128; // stored form of code 0
};

// The scale of a group that held a NaN or an infinity: every element reads as
// NaN.  As a signed 16-bit integer it is -1, so a signed maximum over scales passes
// it by.
constexpr uint16_t kKvNanScale = 0xFFFFu;

// Where the cache's parts lie.  Pages are [2, Hkv, P, row]: head h of page p
// starts at row ((p * 2 + which) * Hkv + h) * P of its tensor.
struct KvCache {
    uint8_t *codes;
    uint16_t *scales;
    int64_t num_pages;
    int Hkv;
    int log2_page;

    __device__ __forceinline__ int64_t row(int64_t page, int which, int head, int off) const {
        return ((((page * 2 + which) * Hkv + head)) << log2_page) + off;
    }
};

__device__ __forceinline__ float half_bits_to_float(uint16_t h) {
    return __half2float(__ushort_as_half(h));
}

// Two fp32 operations an instruction: r = x * b + c and r = x + c, each rounded once.
__device__ __forceinline__ void fma2(float &r0, float &r1, float x0, float x1, float b, float c) {
    asm("{\n\t.reg .b64 x, b, c, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 c, {%5, %5};\n\t"
        "fma.rn.f32x2 r, x, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r0), "=f"(r1) : "f"(x0), "f"(x1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float &r0, float &r1, float x0, float x1, float c) {
    asm("{\n\t.reg .b64 x, c, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\t"
        "add.rn.f32x2 r, x, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(r0), "=f"(r1) : "f"(x0), "f"(x1), "f"(c));
}

struct KvWriteArgs {
    const uint16_t *kv;    // first key element of token 0
    int64_t stride;        // elements from one token to the next
    const int64_t *slots;
    uint32_t tokens;       // T
    uint32_t parts;        // groups of kHeads heads of a token
    int64_t num_slots;
    KvCache cache;
};

// log2 of a page size the cache takes (16, 32, 64, 128 or 256), else -1.
inline int kv_log2_page(int page_size) {
    for (int l = 4; l <= 8; ++l)
        if (page_size == 1 << l) return l;
    return -1;
}

// Sizes every cache entry point checks the same way: RN_OK, RN_ERR_ARG for an
// unknown format, RN_ERR_SHAPE.
inline int kv_check_sizes(int format, int Hkv, int D, int page_size, int64_t num_pages) {
    if (format != RN_KV_INT4 && format != RN_KV_INT8) return RN_ERR_ARG;
    if (D != 64 && D != 128 && D != 256) return RN_ERR_SHAPE;
    if (Hkv < 1 || Hkv > 16384) return RN_ERR_SHAPE;  // a page's codes stay under 4 GB
    if (kv_log2_page(page_size) < 0) return RN_ERR_SHAPE;
    if (num_pages < 1 || num_pages > INT32_MAX) return RN_ERR_SHAPE;
    return RN_OK;
}

// Calls f with the compile-time head size and bits of a checked (D, format).
template <typename Fn>
inline auto kv_dispatch(int D, int format, Fn &&f) {
    if (format == RN_KV_INT4) {
        if (D == 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
        if (D == 128) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
        return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
    }
    if (D == 64) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
    if (D == 128) return f(std::integral_constant<int, 128>(), std::integral_constant<int, 8>());
    return f(std::integral_constant<int, 256>(), std::integral_constant<int, 8>());
}

// Reads (and optionally clears) a translation unit's status word.
template <typename Sym>
inline int kv_status_word(Sym &symbol, unsigned int *out, int clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, symbol, sizeof v) != cudaSuccess) {
        cudaGetLastError();
        return RN_ERR_DEVICE;
    }
    if (clear && v != 0) {
        const unsigned int zero = 0;
        if (cudaMemcpyToSymbol(symbol, &zero, sizeof zero) != cudaSuccess) {
            cudaGetLastError();
            return RN_ERR_DEVICE;
        }
    }
    *out = v;
    return RN_OK;
}

}  // namespace rn
