// Four elements of an input at a time, bf16 or fp32, shared by the packed
// forward (gdn_packed.hip), linear attention (gdn_linear.hip) and the query and
// key norm (gdn_qk_norm.hip).  Internal to libgdn.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdn_mfma_common.h"

namespace gdn {
namespace {

// four consecutive input-typed elements, as loaded and as fp32
template <int DT>
using R4 = std::conditional_t<DT == GDN_BF16, u32x2, f32x4>;
template <int DT>
__device__ __forceinline__ R4<DT> ldr(const void* base, int64_t i) {
    if constexpr (DT == GDN_BF16) return *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(base) + i);
    else return *reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + i);
}
template <int DT>
__device__ __forceinline__ f32x4 cvt(const R4<DT>& u) {
    if constexpr (DT == GDN_BF16)
        return f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xFFFF0000u), __uint_as_float(u[1] << 16),
                     __uint_as_float(u[1] & 0xFFFF0000u)};
    else return u;
}
template <int DT>
__device__ __forceinline__ f32x4 ld4e(const void* p, int64_t i) {
    return cvt<DT>(ldr<DT>(p, i));
}
__device__ __forceinline__ float dot4e(const f32x4& x, const f32x4& y) {
    return x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
}
template <int DT>
__device__ __forceinline__ void st_out(void* out, int64_t i, float x) {
    if constexpr (DT == GDN_F32) static_cast<float*>(out)[i] = x;
    else static_cast<uint16_t*>(out)[i] = (uint16_t)pack_bf16(x, 0.f);
}

}  // namespace
}  // namespace gdn
