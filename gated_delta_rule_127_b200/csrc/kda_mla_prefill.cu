// kda_mla_prefill.cu -- expanded latent attention over a packed batch.
//
// Simple form: one warp per (query, head) walks its keys with a running maximum and sum; lane l holds channels
// 4 l .. 4 l + 3 of the 128 and 2 l, 2 l + 1 of the 64 positional ones.
#include "kda_mla_common.cuh"

namespace kda {
namespace {

template <typename TO>
__global__ void __launch_bounds__(128) mla_prefill_rows(MlaPrefillArgs a) {
    if (blockIdx.x == 0) {
        mla::check_cu(a.cu_q, a.Tq, a.B, a.flags);
        mla::check_cu(a.cu_k, a.Tk, a.B, a.flags);
    }
    const int lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (r >= a.Tq * a.H) return;
    const int64_t t = r / a.H;
    const int h = static_cast<int>(r % a.H);
    const int b = mla::seq_of_row(a.cu_q, a.Tq, a.B, t);
    if (b >= a.B) return;
    int64_t q0, k0;
    const int nq = mla::seq_rows(a.cu_q, a.Tq, a.B, b, q0, a.flags);
    const int nk = mla::seq_rows(a.cu_k, a.Tk, a.B, b, k0, a.flags);
    const int i = static_cast<int>(t - q0);
    const int see = nq <= i ? 0 : a.causal ? min(nk, i + 1 + nk - nq) : nk;
    float q[4], p[2], o[4] = {};
    const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + r * kMlaQk;
    for (int c = 0; c < 4; ++c) q[c] = __bfloat162float(qr[lane * 4 + c]);
    for (int c = 0; c < 2; ++c) p[c] = __bfloat162float(qr[kMlaNope + lane * 2 + c]);
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < see; ++j) {
        const __nv_bfloat16* kv = static_cast<const __nv_bfloat16*>(a.kv) + ((k0 + j) * a.H + h) * kMlaKv + lane * 4;
        const __nv_bfloat16* pe = static_cast<const __nv_bfloat16*>(a.k_pe) + (k0 + j) * kMlaPe + lane * 2;
        float x = 0.f;
        for (int c = 0; c < 4; ++c) x += q[c] * __bfloat162float(kv[c]);
        for (int c = 0; c < 2; ++c) x += p[c] * __bfloat162float(pe[c]);
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        x *= a.scale;
        const float mn = fmaxf(m, x), f = mn == -INFINITY ? 1.f : expf(m - mn), e = expf(x - mn);
        l = l * f + e;
        for (int c = 0; c < 4; ++c) o[c] = o[c] * f + e * __bfloat162float(kv[kMlaNope + c]);
        m = mn;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    TO* out = static_cast<TO*>(a.o) + r * kMlaV + lane * 4;
    for (int c = 0; c < 4; ++c) out[c] = from_f32<TO>(o[c] * inv);
    if (a.lse && lane == 0) a.lse[r] = m + logf(l);
}

}  // namespace

cudaError_t launch_mla_prefill(const MlaPrefillArgs& a) {
    const dim3 grid(static_cast<unsigned>((a.Tq * a.H + 3) / 4));
    if (a.o_fp32) mla_prefill_rows<float><<<grid, 128, 0, a.stream>>>(a);
    else mla_prefill_rows<__nv_bfloat16><<<grid, 128, 0, a.stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
