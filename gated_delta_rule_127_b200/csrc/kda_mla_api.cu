// kda_mla_api.cu -- the latent-attention entry points: host-side validation and launch.
#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <initializer_list>

#include "kda.h"
#include "kda_internal.h"

namespace kda {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool plain_dtype(kda_dtype d) { return d == KDA_BF16 || d == KDA_FP32; }
bool given16(const void* p) { return p && aligned16(p); }

// Rows and positions are 32-bit numbers in the kernels, also those just past a last tile of 256.
constexpr int64_t kMostRows = 0x7fffff00;

// An array of a call.  Kernels read inputs while others of their blocks write, so an output may lie over nothing else.
struct Span {
    const void* p;
    int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}
bool apart(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
    for (const Span* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Span* other = outputs.begin(); other != o; ++other)
            if (overlap(*o, *other)) return false;
        for (const Span& i : inputs)
            if (overlap(*o, i)) return false;
    }
    return true;
}
int64_t size_of(kda_dtype d) { return d == KDA_FP32 ? 4 : d == KDA_BF16 ? 2 : 1; }

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

// Sizes, types and pointers of the paged cache; `used` false: a call without tokens reads no pointer.
kda_status check_cache(const void* latent, const void* pe, const float* scale, const int32_t* page_table,
                       int d_latent, int d_pe, int64_t num_pages, int page_size, int max_pages,
                       kda_dtype dtype_cache, bool used, MlaCache* c) {
    if (d_latent <= 0 || d_pe <= 0 || num_pages < 0 || page_size <= 0 || max_pages < 0) return KDA_ERR_INVALID_ARG;
    if (dtype_cache != KDA_BF16 && dtype_cache != KDA_E4M3)
        return dtype_cache == KDA_FP32 ? KDA_ERR_UNSUPPORTED : KDA_ERR_INVALID_ARG;
    if (d_latent != kMlaLatent || d_pe != kMlaPe) return KDA_ERR_UNSUPPORTED;
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return KDA_ERR_UNSUPPORTED;
    if (num_pages > kMostRows / page_size || static_cast<int64_t>(max_pages) * page_size > kMostRows)
        return KDA_ERR_UNSUPPORTED;
    const bool e4m3 = dtype_cache == KDA_E4M3;
    if (used) {
        if (num_pages > 0 && (!given16(latent) || !given16(pe))) return KDA_ERR_INVALID_ARG;
        if (num_pages > 0 && e4m3 && !given16(scale)) return KDA_ERR_INVALID_ARG;
        if (max_pages > 0 && (!page_table || !aligned4(page_table))) return KDA_ERR_INVALID_ARG;
    }
    c->latent = const_cast<void*>(latent);
    c->pe = const_cast<void*>(pe);
    c->scale = e4m3 ? const_cast<float*>(scale) : nullptr;
    c->page_table = page_table;
    c->num_pages = num_pages;
    c->page_size = page_size;
    c->page_shift = 0;
    while ((1 << c->page_shift) < page_size) ++c->page_shift;
    c->max_pages = max_pages;
    c->e4m3 = e4m3;
    return KDA_OK;
}

Span latent_of(const MlaCache& c) { return {c.latent, c.num_pages * c.page_size * kMlaLatent * (c.e4m3 ? 1 : 2)}; }
Span pe_of(const MlaCache& c) { return {c.pe, c.num_pages * c.page_size * kMlaPe * 2}; }
Span scale_of(const MlaCache& c) { return {c.scale, c.num_pages * c.page_size * 4}; }
Span table_of(const MlaCache& c, int B) { return {c.page_table, static_cast<int64_t>(B) * c.max_pages * 4}; }

kda_status cache_copy(bool write, const void* latent, const void* pe, const int32_t* cu_seqlens, const int32_t* lens,
                      int64_t T, int B, kda_dtype dtype, const MlaCache& cache, void* stream) {
    if (T == 0) return KDA_OK;
    if (!given16(latent) || !given16(pe)) return KDA_ERR_INVALID_ARG;
    if ((write && !lens) || !aligned4(lens) || !aligned4(cu_seqlens)) return KDA_ERR_INVALID_ARG;
    const Span rows{latent, T * kMlaLatent * size_of(dtype)}, keys{pe, T * kMlaPe * size_of(dtype)};
    const Span cu{cu_seqlens, (static_cast<int64_t>(B) + 1) * 4}, each{lens, static_cast<int64_t>(B) * 4};
    const Span cl = latent_of(cache), cp = pe_of(cache), cs = scale_of(cache), table = table_of(cache, B);
    if (write ? !apart({cl, cp, cs}, {rows, keys, cu, each, table}) : !apart({rows, keys}, {cl, cp, cs, cu, each, table}))
        return KDA_ERR_INVALID_ARG;
    MlaCacheCopyArgs a{};
    a.cache = cache;
    a.latent = const_cast<void*>(latent);
    a.pe = const_cast<void*>(pe);
    a.cu_seqlens = cu_seqlens;
    a.lens = lens;
    a.T = T;
    a.B = B;
    a.fp32 = dtype == KDA_FP32;
    a.stream = static_cast<cudaStream_t>(stream);
    if (const kda_status st = status_of(device_flags_ptr(&a.flags)); st != KDA_OK) return st;
    NvtxRange range(write ? "kda_mla_cache_write" : "kda_mla_cache_read");
    return status_of(write ? launch_mla_cache_write(a) : launch_mla_cache_read(a));
}

}  // namespace
}  // namespace kda

extern "C" {

kda_status kda_mla_cache_write(const void* latent, const void* pe, const int32_t* cu_seqlens,
                               const int32_t* seq_lens, int64_t T, int B, int d_latent, int d_pe,
                               kda_dtype dtype_in, kda_dtype dtype_cache, void* cache_latent, void* cache_pe,
                               float* cache_scale, const int32_t* page_table, int64_t num_pages, int page_size,
                               int max_pages, void* stream) {
    using namespace kda;
    if (T < 0 || B <= 0 || !plain_dtype(dtype_in)) return KDA_ERR_INVALID_ARG;
    MlaCache c{};
    const kda_status st = check_cache(cache_latent, cache_pe, cache_scale, page_table, d_latent, d_pe, num_pages,
                                      page_size, max_pages, dtype_cache, T > 0, &c);
    if (st != KDA_OK) return st;
    if (T > kMostRows) return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens && T % B != 0) return KDA_ERR_INVALID_ARG;
    return cache_copy(true, latent, pe, cu_seqlens, seq_lens, T, B, dtype_in, c, stream);
}

kda_status kda_mla_cache_read(const void* cache_latent, const void* cache_pe, const float* cache_scale,
                              const int32_t* page_table, const int32_t* cu_seqlens, const int32_t* starts, int64_t T,
                              int B, int d_latent, int d_pe, int64_t num_pages, int page_size, int max_pages,
                              kda_dtype dtype_cache, kda_dtype dtype_o, void* latent, void* pe, void* stream) {
    using namespace kda;
    if (T < 0 || B <= 0 || !plain_dtype(dtype_o)) return KDA_ERR_INVALID_ARG;
    MlaCache c{};
    const kda_status st = check_cache(cache_latent, cache_pe, cache_scale, page_table, d_latent, d_pe, num_pages,
                                      page_size, max_pages, dtype_cache, T > 0, &c);
    if (st != KDA_OK) return st;
    if (T > kMostRows) return KDA_ERR_UNSUPPORTED;
    if (!cu_seqlens && T % B != 0) return KDA_ERR_INVALID_ARG;
    return cache_copy(false, latent, pe, cu_seqlens, starts, T, B, dtype_o, c, stream);
}

size_t kda_mla_decode_workspace_size(int B, int S, int H, int d_latent, int d_pe) {
    if (B <= 0 || S <= 0 || H <= 0 || static_cast<int64_t>(S) * H > 65535 || d_latent != kda::kMlaLatent ||
        d_pe != kda::kMlaPe)
        return 0;
    return kda::mla_decode_workspace_size(B, S, H);
}

kda_status kda_mla_decode(const void* q_latent, const void* q_pe, const void* cache_latent, const void* cache_pe,
                          const float* cache_scale, const int32_t* page_table, const int32_t* seq_lens, int B, int S,
                          int H, int d_latent, int d_pe, int64_t num_pages, int page_size, int max_pages,
                          float softmax_scale, kda_dtype dtype_q, kda_dtype dtype_cache, kda_dtype dtype_o, void* o,
                          float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace kda;
    if (B < 0 || S <= 0 || H <= 0 || !plain_dtype(dtype_q) || !plain_dtype(dtype_o) || !std::isfinite(softmax_scale))
        return KDA_ERR_INVALID_ARG;
    MlaCache c{};
    const kda_status st = check_cache(cache_latent, cache_pe, cache_scale, page_table, d_latent, d_pe, num_pages,
                                      page_size, max_pages, dtype_cache, B > 0, &c);
    if (st != KDA_OK) return st;
    if (dtype_q != KDA_BF16 || static_cast<int64_t>(S) * H > 65535 || static_cast<int64_t>(B) * S * H > 0x7fffffffLL)
        return KDA_ERR_UNSUPPORTED;
    if (B == 0) return KDA_OK;
    if (!given16(q_latent) || !given16(q_pe) || !given16(o) || !aligned4(lse)) return KDA_ERR_INVALID_ARG;
    if (!seq_lens || !aligned4(seq_lens)) return KDA_ERR_INVALID_ARG;
    const bool have_ws = workspace != nullptr && workspace_bytes > 0;
    if (have_ws && (!aligned16(workspace) || workspace_bytes < mla_decode_workspace_size(B, S, H)))
        return KDA_ERR_INVALID_ARG;
    const int64_t q_rows = static_cast<int64_t>(B) * S * H;
    if (!apart({{o, q_rows * kMlaLatent * size_of(dtype_o)}, {lse, q_rows * 4},
                {have_ws ? workspace : nullptr, static_cast<int64_t>(mla_decode_workspace_size(B, S, H))}},
               {{q_latent, q_rows * kMlaLatent * 2}, {q_pe, q_rows * kMlaPe * 2}, latent_of(c), pe_of(c), scale_of(c),
                table_of(c, B), {seq_lens, static_cast<int64_t>(B) * 4}}))
        return KDA_ERR_INVALID_ARG;
    MlaDecodeArgs a{};
    a.q_latent = q_latent;
    a.q_pe = q_pe;
    a.cache = c;
    a.seq_lens = seq_lens;
    a.B = B; a.S = S; a.H = H;
    a.scale = softmax_scale;
    a.o_fp32 = dtype_o == KDA_FP32;
    a.o = o;
    a.lse = lse;
    a.workspace = have_ws ? workspace : nullptr;
    a.wait_polls = consumer_wait_polls();
    a.stream = static_cast<cudaStream_t>(stream);
    if (const kda_status st = status_of(device_flags_ptr(&a.flags)); st != KDA_OK) return st;
    NvtxRange range("kda_mla_decode");
    return status_of(launch_mla_decode(a));
}

kda_status kda_mla_prefill(const void* q, const void* kv, const void* k_pe, const int32_t* cu_seqlens_q,
                           const int32_t* cu_seqlens_k, int64_t Tq, int64_t Tk, int B, int H, int d_nope, int d_pe,
                           int dv, int causal, float softmax_scale, kda_dtype dtype_qkv, kda_dtype dtype_o, void* o,
                           float* lse, void* stream) {
    using namespace kda;
    if (Tq < 0 || Tk < 0 || B <= 0 || H <= 0 || d_nope <= 0 || d_pe <= 0 || dv <= 0 || (causal != 0 && causal != 1) ||
        !plain_dtype(dtype_qkv) || !plain_dtype(dtype_o) || !std::isfinite(softmax_scale))
        return KDA_ERR_INVALID_ARG;
    if (d_nope != kMlaNope || d_pe != kMlaPe || dv != kMlaV || dtype_qkv != KDA_BF16 || H > 65535 ||
        Tq > kMostRows || Tk > kMostRows)
        return KDA_ERR_UNSUPPORTED;
    if ((!cu_seqlens_q && Tq % B != 0) || (!cu_seqlens_k && Tk % B != 0)) return KDA_ERR_INVALID_ARG;
    if (Tq == 0) return KDA_OK;
    if (!given16(q) || !given16(o) || !aligned4(lse) || !aligned4(cu_seqlens_q) || !aligned4(cu_seqlens_k))
        return KDA_ERR_INVALID_ARG;
    if (Tk > 0 && (!given16(kv) || !given16(k_pe))) return KDA_ERR_INVALID_ARG;
    const int64_t cu_bytes = (static_cast<int64_t>(B) + 1) * 4;
    if (!apart({{o, Tq * H * kMlaV * size_of(dtype_o)}, {lse, Tq * H * 4}},
               {{q, Tq * H * kMlaQk * 2}, {kv, Tk * H * kMlaKv * 2}, {k_pe, Tk * kMlaPe * 2}, {cu_seqlens_q, cu_bytes},
                {cu_seqlens_k, cu_bytes}}))
        return KDA_ERR_INVALID_ARG;
    MlaPrefillArgs a{};
    a.q = q; a.kv = kv; a.k_pe = k_pe;
    a.cu_q = cu_seqlens_q; a.cu_k = cu_seqlens_k;
    a.Tq = Tq; a.Tk = Tk;
    a.B = B; a.H = H;
    a.causal = causal != 0;
    a.scale = softmax_scale;
    a.o_fp32 = dtype_o == KDA_FP32;
    a.o = o;
    a.lse = lse;
    a.wait_polls = consumer_wait_polls();
    a.stream = static_cast<cudaStream_t>(stream);
    if (const kda_status st = status_of(device_flags_ptr(&a.flags)); st != KDA_OK) return st;
    NvtxRange range("kda_mla_prefill");
    return status_of(launch_mla_prefill(a));
}

}  // extern "C"
