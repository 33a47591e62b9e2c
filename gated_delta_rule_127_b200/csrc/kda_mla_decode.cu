// kda_mla_decode.cu -- absorbed latent attention over the paged cache.
//
// Simple form: one warp per (sequence, token, head) walks the keys with a running maximum and sum; lane l holds
// channels 16 l .. 16 l + 15 of the latent and 2 l, 2 l + 1 of the positional part.
#include <cuda_fp8.h>

#include "kda_mla_common.cuh"

namespace kda {
namespace {

template <bool E4M3, typename TO>
__global__ void __launch_bounds__(128) mla_decode_rows(MlaDecodeArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (r >= static_cast<int64_t>(a.B) * a.S * a.H) return;
    const int b = static_cast<int>(r / (a.S * a.H)), s = static_cast<int>(r % (a.S * a.H)) / a.H;
    float q[16], o[16] = {};
    const __nv_bfloat16* ql = static_cast<const __nv_bfloat16*>(a.q_latent) + r * kMlaLatent + lane * 16;
    for (int i = 0; i < 16; ++i) q[i] = __bfloat162float(ql[i]);
    const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q_pe) + r * kMlaPe + lane * 2;
    const float p0 = __bfloat162float(qp[0]), p1 = __bfloat162float(qp[1]);
    int len = a.seq_lens[b];
    if (len < 0 || len > mla::table_reach(a.cache)) {
        raise_flag(a.flags, KDA_DEVFLAG_SEQ_LENS);
        len = 0;
    }
    const int see = len - (a.S - 1 - s);
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < see; ++j) {
        const int64_t row = mla::pool_row(a.cache, b, j, a.flags);
        if (row < 0) continue;
        float c[16], x = 0.f;
        if (E4M3) {
            const uint8_t* p = static_cast<const uint8_t*>(a.cache.latent) + row * kMlaLatent + lane * 16;
            const float sc = a.cache.scale[row];
            for (int i = 0; i < 16; ++i)
                c[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(p[i], __NV_E4M3))) * sc;
        } else {
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.cache.latent) + row * kMlaLatent + lane * 16;
            for (int i = 0; i < 16; ++i) c[i] = __bfloat162float(p[i]);
        }
        const __nv_bfloat16* pe = static_cast<const __nv_bfloat16*>(a.cache.pe) + row * kMlaPe + lane * 2;
        for (int i = 0; i < 16; ++i) x += q[i] * c[i];
        x += p0 * __bfloat162float(pe[0]) + p1 * __bfloat162float(pe[1]);
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= a.scale;
        const float mn = fmaxf(m, x), f = mn == -INFINITY ? 1.f : expf(m - mn), e = expf(x - mn);
        l = l * f + e;
        for (int i = 0; i < 16; ++i) o[i] = o[i] * f + e * c[i];
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    TO* out = static_cast<TO*>(a.o) + r * kMlaLatent + lane * 16;
    for (int i = 0; i < 16; ++i) out[i] = from_f32<TO>(o[i] * inv);
    if (a.lse && lane == 0) a.lse[r] = m + logf(l);
}

}  // namespace

size_t mla_decode_workspace_size(int, int, int) { return 0; }

cudaError_t launch_mla_decode(const MlaDecodeArgs& a) {
    const int64_t rows = static_cast<int64_t>(a.B) * a.S * a.H;
    const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
    if (a.cache.e4m3) {
        if (a.o_fp32) mla_decode_rows<true, float><<<grid, 128, 0, a.stream>>>(a);
        else mla_decode_rows<true, __nv_bfloat16><<<grid, 128, 0, a.stream>>>(a);
    } else {
        if (a.o_fp32) mla_decode_rows<false, float><<<grid, 128, 0, a.stream>>>(a);
        else mla_decode_rows<false, __nv_bfloat16><<<grid, 128, 0, a.stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace kda
