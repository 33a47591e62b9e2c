// kda_mla_cache.cu -- the paged latent cache: writing new tokens (quantised for e4m3) and reading tokens
// back.
//
// Per token: 512 latent channels and 64 positional ones.  e4m3: with a = max |c|, the scale is s = 2^k,
// k = the least integer with a <= 448 2^k, clamped to [-64, 120]; codes are e4m3(c / s).  A power of two
// makes c / s and code * s exact, so the only rounding is the one to e4m3 (half a step of 2^-4) and a value
// read back is exact in bf16 too.
//
// Both directions are bound by memory (a token moves 1152 B on the packed side and 644 or 1152 B on the
// cache's).  One warp takes a token: lane l holds channels 16 l .. 16 l + 15 of the latent (the e4m3 codes of
// a lane are then one 16-byte store, a row is one contiguous 512-byte or 1024-byte piece) and channels 2 l,
// 2 l + 1 of the positional key; the maximum is five shuffles.
#include <cuda_fp8.h>

#include "kda_mla_common.cuh"

namespace kda {
namespace {

constexpr int WARPS = 8;

// 16 consecutive values of the packed side, as fp32
__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(p) + i);
        v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 x = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        __stcs(reinterpret_cast<float4*>(p) + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                       pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
}
__device__ __forceinline__ float2 load2(const float* p) { return __ldcs(reinterpret_cast<const float2*>(p)); }
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
    const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(p));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void store2(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v.x, v.y);
}

__device__ __forceinline__ float pow2(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// The exponent k of a token's scale from its largest magnitude a >= 0 (448 = 1.75 * 2^8).
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t bits = __float_as_uint(a);
    const int e = static_cast<int>(bits >> 23) - 127;
    const int k = (bits & 0x7FFFFFu) > 0x600000u ? e - 7 : e - 8;
    return min(max(k, -64), 120);
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(WARPS * 32) mla_cache_write_kernel(MlaCacheCopyArgs a) {
    if (blockIdx.x == 0) mla::check_cu(a.cu_seqlens, a.T, a.B, a.flags);
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    // the loads do not depend on where the token goes: they are in flight during the search
    float v[16];
    load16(static_cast<const T*>(a.latent) + t * kMlaLatent + lane * 16, v);
    const float2 pe = load2(static_cast<const T*>(a.pe) + t * kMlaPe + lane * 2);

    const int b = mla::seq_of_row(a.cu_seqlens, a.T, a.B, t);
    if (b >= a.B) return;  // behind the last sequence
    int64_t first;
    const int n = mla::seq_rows(a.cu_seqlens, a.T, a.B, b, first, a.flags);
    if (t < first || t >= first + n) return;
    const int len = a.lens[b];
    if (len < n || len > mla::table_reach(a.cache)) {
        raise_flag(a.flags, KDA_DEVFLAG_SEQ_LENS);
        return;
    }
    const int64_t row = mla::pool_row(a.cache, b, len - n + static_cast<int>(t - first), a.flags);
    if (row < 0) return;

    if (E4M3) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]));  // fmaxf passes over NaN
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const int k = scale_exponent(m);
        const float inv = pow2(-k);
        uint4 codes;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv),
                                                         __NV_SATFINITE, __NV_E4M3);
            w[i] = lo | (hi << 16);
        }
        codes = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.cache.latent) + row * kMlaLatent)[lane] = codes;
        if (lane == 0) a.cache.scale[row] = pow2(k);
    } else {
        store16(static_cast<__nv_bfloat16*>(a.cache.latent) + row * kMlaLatent + lane * 16, v);
    }
    store2(static_cast<__nv_bfloat16*>(a.cache.pe) + row * kMlaPe + lane * 2, pe);
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(WARPS * 32) mla_cache_read_kernel(MlaCacheCopyArgs a) {
    if (blockIdx.x == 0) mla::check_cu(a.cu_seqlens, a.T, a.B, a.flags);
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int b = mla::seq_of_row(a.cu_seqlens, a.T, a.B, t);
    if (b >= a.B) return;
    int64_t first;
    const int n = mla::seq_rows(a.cu_seqlens, a.T, a.B, b, first, a.flags);
    if (t < first || t >= first + n) return;
    const int start = a.lens ? a.lens[b] : 0;
    if (start < 0 || static_cast<int64_t>(start) + n > mla::table_reach(a.cache)) {
        raise_flag(a.flags, KDA_DEVFLAG_SEQ_LENS);
        return;
    }
    const int64_t row = mla::pool_row(a.cache, b, start + static_cast<int>(t - first), a.flags);
    if (row < 0) return;

    float v[16];
    if (E4M3) {
        const uint4 codes = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.cache.latent) +
                                                                  row * kMlaLatent) + lane);
        const float s = a.cache.scale[row];
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> ((i & 1) * 16)), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
        }
    } else {
        load16(static_cast<const __nv_bfloat16*>(a.cache.latent) + row * kMlaLatent + lane * 16, v);
    }
    const float2 pe = load2(static_cast<const __nv_bfloat16*>(a.cache.pe) + row * kMlaPe + lane * 2);
    store16(static_cast<T*>(a.latent) + t * kMlaLatent + lane * 16, v);
    store2(static_cast<T*>(a.pe) + t * kMlaPe + lane * 2, pe);
}

}  // namespace

cudaError_t launch_mla_cache_write(const MlaCacheCopyArgs& a) {
    const dim3 grid(static_cast<unsigned>((a.T + WARPS - 1) / WARPS)), block(WARPS * 32);
    if (a.fp32) {
        if (a.cache.e4m3) mla_cache_write_kernel<float, true><<<grid, block, 0, a.stream>>>(a);
        else mla_cache_write_kernel<float, false><<<grid, block, 0, a.stream>>>(a);
    } else {
        if (a.cache.e4m3) mla_cache_write_kernel<__nv_bfloat16, true><<<grid, block, 0, a.stream>>>(a);
        else mla_cache_write_kernel<__nv_bfloat16, false><<<grid, block, 0, a.stream>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_mla_cache_read(const MlaCacheCopyArgs& a) {
    const dim3 grid(static_cast<unsigned>((a.T + WARPS - 1) / WARPS)), block(WARPS * 32);
    if (a.fp32) {
        if (a.cache.e4m3) mla_cache_read_kernel<float, true><<<grid, block, 0, a.stream>>>(a);
        else mla_cache_read_kernel<float, false><<<grid, block, 0, a.stream>>>(a);
    } else {
        if (a.cache.e4m3) mla_cache_read_kernel<__nv_bfloat16, true><<<grid, block, 0, a.stream>>>(a);
        else mla_cache_read_kernel<__nv_bfloat16, false><<<grid, block, 0, a.stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kda
