// rowvec.cuh — V consecutive elements of a row as one memory access, held as
// they are stored (bf16 pairs stay packed) until they are used.  Shared by the
// gated linear recurrence (scan.cuh) and the row norms (norm.cuh).
#pragma once

#include "device.cuh"

namespace la {

template <typename T, int V>
struct RowVec;

template <>
struct RowVec<float, 4> {
    float4 r;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }
    __device__ __forceinline__ void load(const float *p) { r = __ldg(reinterpret_cast<const float4 *>(p)); }
    static __device__ __forceinline__ void store(float *p, const float *v) {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
    __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct RowVec<float, 1> {
    float r;
    __device__ __forceinline__ float get(int) const { return r; }
    __device__ __forceinline__ void load(const float *p) { r = __ldg(p); }
    static __device__ __forceinline__ void store(float *p, const float *v) { *p = v[0]; }
    __device__ __forceinline__ void zero() { r = 0.f; }
};
template <>
struct RowVec<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t u = (i >> 1) == 0 ? r.x : (i >> 1) == 1 ? r.y : (i >> 1) == 2 ? r.z : r.w;
        return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const uint4 *>(p)); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                   pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
    __device__ __forceinline__ void zero() { r = make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct RowVec<__nv_bfloat16, 4> {
    uint2 r;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t u = (i >> 1) == 0 ? r.x : r.y;
        return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
    }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const uint2 *>(p)); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
    __device__ __forceinline__ void zero() { r = make_uint2(0u, 0u); }
};
template <>
struct RowVec<__nv_bfloat16, 2> {
    uint32_t r;
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(i ? (r & 0xffff0000u) : (r << 16)); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const uint32_t *>(p)); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) {
        *reinterpret_cast<uint32_t *>(p) = pack_bf16x2(v[0], v[1]);
    }
    __device__ __forceinline__ void zero() { r = 0u; }
};
template <>
struct RowVec<__nv_bfloat16, 1> {
    unsigned short r;
    __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)r << 16); }
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { r = __ldg(reinterpret_cast<const unsigned short *>(p)); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) { *p = __float2bfloat16_rn(v[0]); }
    __device__ __forceinline__ void zero() { r = 0; }
};

// Whether every access of V elements of `esize` bytes at p + row * k is aligned.
inline bool vec_ok(const void *p, int64_t row, int esize, int V) {
    return !p || ((reinterpret_cast<uintptr_t>(p) % (size_t)(esize * V)) == 0 && row % V == 0);
}

}  // namespace la
