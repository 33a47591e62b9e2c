// kda_mla_cache.cu -- the paged latent cache: writing new tokens (quantised for e4m3) and reading tokens
// back.
//
// Per token: 512 latent channels and 64 positional ones.  e4m3: with a = max |c|, the scale is s = 2^k,
// k = the least integer with a <= 448 2^k, clamped to [-64, 120]; codes are e4m3(c / s).  A power of two
// makes c / s and code * s exact, so the only rounding is the one to e4m3 (half a step of 2^-4) and a value
// read back is exact in bf16 too.  One end: with s = 2^120 a code of 256 or more stands for 2^128 or more, which
// fp32 and bf16 read as infinity (|c| from 248 x 2^120 = 3.30e38 on: the largest bf16, 3.39e38, and infinity itself).
//
// Both directions are bound by memory (a token moves 1152 B on the packed side and 644 or 1152 B on the cache's).  A warp
// takes a token, or several with all their loads in flight: lane l holds channels 8 l .. 8 l + 7 and 256 + 8 l .. of the
// latent, so that every access of the warp, 16 bytes a lane in bf16 and 8 in e4m3, is one contiguous piece, and
// channels 2 l, 2 l + 1 of the positional key; the maximum is five shuffles.
#include <cuda_fp8.h>

#include <type_traits>

#include "kda_mla_common.cuh"

namespace kda {
namespace {

constexpr int WARPS = 8;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// Eight neighbouring values as they lie in memory, and as fp32.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 raw;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <> struct Eight<float> {
    float4 raw[2];
    __device__ __forceinline__ void load(const float* p) {
        raw[0] = __ldcs(reinterpret_cast<const float4*>(p));
        raw[1] = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        v[0] = raw[0].x; v[1] = raw[0].y; v[2] = raw[0].z; v[3] = raw[0].w;
        v[4] = raw[1].x; v[5] = raw[1].y; v[6] = raw[1].z; v[7] = raw[1].w;
    }
};
struct EightCodes {  // e4m3
    uint2 raw;
    __device__ __forceinline__ void load(const uint8_t* p) { raw = __ldcs(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        const uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> ((i & 1) * 16)), __NV_E4M3);
            const float2 f = __half22float2(__half2(h));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8]) {  // as e4m3
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(v[2 * i], v[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
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

// The pool rows of a warp's N consecutive packed rows t0 .. (-1: nothing to do there: behind the last sequence, a
// skipped sequence, a bad page).  `lens`: seq_lens, of which the packed rows are the last (write), or the first
// positions, NULL for 0 (read).  Mostly all N belong to the sequence that the first one's search has found.
template <int N, bool WRITE>
__device__ __forceinline__ void find_rows(const MlaCacheCopyArgs& a, int64_t t0, int64_t (&row)[N]) {
    int b = -1, base = 0;  // position of the packed row `first`
    int64_t first = 0, end = 0;
    bool good = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = t0 + i;
        row[i] = -1;
        if (t >= a.T) continue;
        if (b < 0 || t >= end) {
            b = mla::seq_of_row(a.cu_seqlens, a.T, a.B, t);
            if (b >= a.B) {
                end = a.T;
                good = false;
                continue;
            }
            const int n = mla::seq_rows(a.cu_seqlens, a.T, a.B, b, first, a.flags);
            end = first + n;
            base = a.lens ? a.lens[b] - (WRITE ? n : 0) : 0;
            good = base >= 0 && static_cast<int64_t>(base) + n <= mla::table_reach(a.cache);
            if (!good) raise_flag(a.flags, KDA_DEVFLAG_SEQ_LENS);
            good = good && t >= first && t < end;
        }
        if (good) row[i] = mla::pool_row(a.cache, b, base + static_cast<int>(t - first), a.flags);
    }
}

// Packed rows per warp: several, their loads in flight at once, where there are enough rows to fill the SMs all the same.
// 1, 2, 3, 4: 16 prompts of 1,024 to 8,192 tokens written in e4m3 in 26.7, 25.5, 26.9, 27.6 us (4.7 TB/s), as many read in
// 24.7, 20.4, 21.0, 21.4 us (5.6 TB/s).
constexpr int ROWS = 2;
constexpr int64_t kManyRows = 148 * 32 * ROWS;

template <typename T, bool E4M3, int N>
__global__ void __launch_bounds__(WARPS * 32) mla_cache_write_kernel(const __grid_constant__ MlaCacheCopyArgs a) {
    using C = std::conditional_t<E4M3, uint8_t, __nv_bfloat16>;
    mla::after_previous();
    if (blockIdx.x == 0) mla::check_cu(a.cu_seqlens, a.T, a.B, a.flags);
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5)) * N;
    if (t0 >= a.T) return;
    // the loads do not depend on where the tokens go: they are in flight during the search
    Eight<T> in[N][2];
    float2 pe[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t t = min(t0 + i, a.T - 1);
#pragma unroll
        for (int g = 0; g < 2; ++g) in[i][g].load(static_cast<const T*>(a.latent) + t * kMlaLatent + g * 256 + lane * 8);
        pe[i] = load2(static_cast<const T*>(a.pe) + t * kMlaPe + lane * 2);
    }
    int64_t row[N];
    find_rows<N, true>(a, t0, row);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (row[i] < 0) continue;  // the same for the whole warp
        float v[2][8];
        in[i][0].values(v[0]);
        in[i][1].values(v[1]);
        if (E4M3) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(v[0][j]), fabsf(v[1][j])));  // fmaxf passes over NaN
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            const int k = scale_exponent(m);
            const float inv = pow2(-k);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[0][j] *= inv;
                v[1][j] *= inv;
            }
            if (lane == 0) a.cache.scale[row[i]] = pow2(k);
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) store8(static_cast<C*>(a.cache.latent) + row[i] * kMlaLatent + g * 256 + lane * 8, v[g]);
        store2(static_cast<__nv_bfloat16*>(a.cache.pe) + row[i] * kMlaPe + lane * 2, pe[i]);
    }
}

template <typename T, bool E4M3, int N>
__global__ void __launch_bounds__(WARPS * 32) mla_cache_read_kernel(const __grid_constant__ MlaCacheCopyArgs a) {
    using C = std::conditional_t<E4M3, uint8_t, __nv_bfloat16>;
    mla::after_previous();
    if (blockIdx.x == 0) mla::check_cu(a.cu_seqlens, a.T, a.B, a.flags);
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5)) * N;
    if (t0 >= a.T) return;
    int64_t row[N];
    find_rows<N, false>(a, t0, row);
    std::conditional_t<E4M3, EightCodes, Eight<__nv_bfloat16>> in[N][2];
    float2 pe[N];
    float scale[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (row[i] < 0) continue;
#pragma unroll
        for (int g = 0; g < 2; ++g) in[i][g].load(static_cast<const C*>(a.cache.latent) + row[i] * kMlaLatent + g * 256 + lane * 8);
        if (E4M3) scale[i] = a.cache.scale[row[i]];
        pe[i] = load2(static_cast<const __nv_bfloat16*>(a.cache.pe) + row[i] * kMlaPe + lane * 2);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (row[i] < 0) continue;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            float v[8];
            in[i][g].values(v);
            if (E4M3) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] *= scale[i];
            }
            store8(static_cast<T*>(a.latent) + (t0 + i) * kMlaLatent + g * 256 + lane * 8, v);
        }
        store2(static_cast<T*>(a.pe) + (t0 + i) * kMlaPe + lane * 2, pe[i]);
    }
}

template <bool WRITE, typename T, bool E4M3>
cudaError_t launch(const MlaCacheCopyArgs& a) {
    const bool many = a.T >= kManyRows;
    const int64_t per = WARPS * (many ? ROWS : 1);
    const dim3 grid(static_cast<unsigned>((a.T + per - 1) / per)), block(WARPS * 32);
    constexpr auto one = WRITE ? mla_cache_write_kernel<T, E4M3, 1> : mla_cache_read_kernel<T, E4M3, 1>;
    constexpr auto several = WRITE ? mla_cache_write_kernel<T, E4M3, ROWS> : mla_cache_read_kernel<T, E4M3, ROWS>;
    return launch_early(many ? several : one, grid, block, 0, a.stream, a);
}

template <bool WRITE>
cudaError_t dispatch(const MlaCacheCopyArgs& a) {
    if (a.fp32) return a.cache.e4m3 ? launch<WRITE, float, true>(a) : launch<WRITE, float, false>(a);
    return a.cache.e4m3 ? launch<WRITE, __nv_bfloat16, true>(a) : launch<WRITE, __nv_bfloat16, false>(a);
}

}  // namespace

cudaError_t launch_mla_cache_write(const MlaCacheCopyArgs& a) { return dispatch<true>(a); }
cudaError_t launch_mla_cache_read(const MlaCacheCopyArgs& a) { return dispatch<false>(a); }

}  // namespace kda
