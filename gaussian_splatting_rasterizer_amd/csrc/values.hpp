// values.hpp -- runs of eight values of one type in registers (device code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gsr {

// 16 and 8 bytes at any element's address.
typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t Words2 __attribute__((ext_vector_type(2), aligned(2)));

// Eight values as they lie in memory.  Rows of odd length and views start anywhere, and the memory system takes 16-byte
// accesses at any element's address, so a whole run is always one (float32: two) of them; only the last run of a row
// goes element by element.
template <class T>
struct Run8 {
    T v[8];
    // n values from p; the rest zero.  STREAM, here and in store: not kept in the caches for longer than other data
    template <bool STREAM = false>
    __device__ __forceinline__ void load(const T* p, int n) {
        if (n >= 8) {
            if constexpr (STREAM) {
#pragma unroll
                for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
                    const Words4 w = __builtin_nontemporal_load((const Words4*)p + i);
                    __builtin_memcpy((char*)v + 16 * i, &w, 16);
                }
            } else {
                __builtin_memcpy(v, p, sizeof(v));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : (T)0.f;
        }
    }
    template <bool STREAM = false>
    __device__ __forceinline__ void store(T* p, int n) const {
        if (n >= 8) {
            if constexpr (STREAM) {
#pragma unroll
                for (int i = 0; i < (int)sizeof(v) / 16; ++i) {
                    Words4 w;
                    __builtin_memcpy(&w, (const char*)v + 16 * i, 16);
                    __builtin_nontemporal_store(w, (Words4*)p + i);
                }
            } else {
                __builtin_memcpy(p, v, sizeof(v));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) p[e] = v[e];
        }
    }
    __device__ __forceinline__ float get(int e) const { return (float)v[e]; }
    __device__ __forceinline__ void set(int e, float x) { v[e] = (T)x; }
};

// The largest value of the nearest 8-bit type (4 exponent bits, 3 fraction bits, no infinities) and its smallest step.
constexpr float kF8Max = 448.f, kF8Min = 0x1p-9f;

// Magnitudes as integers: their order is the floats', and NaN lies above infinity, so a maximum keeps it.
__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }

// Scale of a group whose largest magnitude is top; a group without a value above zero has scale 1.
__device__ __forceinline__ float f8_scale(float top) { return top > 0.f ? top * (1.f / kF8Max) : 1.f; }

// Four codes in a word, rounded to nearest even.
__device__ __forceinline__ uint32_t pack_f8(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

}  // namespace gsr
