// kda_internal.h -- launchers shared between the host API (kda_api.cu) and the kernel files.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "kda.h"

namespace kda {

// The status of a CUDA call.  An error is taken off the runtime's record, where the next launch's check would find it.
inline kda_status status_of(cudaError_t err) {
    if (err == cudaSuccess) return KDA_OK;
    cudaGetLastError();
    return KDA_ERR_CUDA;
}

struct ChunkArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* log_alpha;
    const void* beta;
    const float* initial_state;
    const int32_t* cu_seqlens;  // may be NULL: equal lengths T_total / N
    int64_t T_total;
    int N, H, dk, dv;
    kda_dtype dtype_qkv, dtype_gate, dtype_o;
    void* o;
    float* final_state;
    void* workspace;
    size_t workspace_bytes;
    unsigned int* flags;  // device address of the sticky flag word
    cudaStream_t stream;
    bool scalar_gate;     // log_alpha is [T_total, H] (Gated DeltaNet), broadcast over dk
    bool l2norm_qk;       // q, k raw: divided by their L2 norm per (token, head) in the kernels
    bool beta_logits;     // beta holds logits: sigmoid applied in the kernels
    bool epilogue;        // o <- o / rms(o) * norm_weight * sigmoid(out_gate) per (token, head)
    const void* out_gate; // [T_total, H, dv], dtype_qkv
    const float* norm_weight;  // [dv]
    float norm_eps;
    uint32_t wait_polls;  // polls before a consumer-side bounded wait gives up (consumer_wait_polls())
};

struct DecodeArgs {
    const void* q;
    const void* k;
    const void* v;
    const void* log_alpha;
    const void* beta;
    float* state;
    int B, H, dk, dv;
    kda_dtype dtype_qkv, dtype_gate, dtype_o;
    void* o;
    unsigned int* flags;
    cudaStream_t stream;
    bool scalar_gate;  // log_alpha is [B, H] (Gated DeltaNet), broadcast over dk
    bool l2norm_qk;    // q, k raw: divided by their L2 norm per (b, h) in the kernel
    bool beta_logits;  // beta holds logits: sigmoid applied in the kernel
    bool epilogue;     // o <- o / rms(o) * norm_weight * sigmoid(out_gate) per (b, h)
    const void* out_gate;  // [B, H, dv], dtype_qkv
    const float* norm_weight;  // [dv]
    float norm_eps;
};

// The bf16 dk = dv = 128 tensor-core prefill runs exactly when this holds; it is the only prefill
// path that reads a workspace (T_total = 0 has no tile to describe and goes to the CUDA-core path,
// which passes the states through).
inline bool chunk_tc_path(int64_t T_total, kda_dtype dtype_qkv, int dk, int dv) {
    return dtype_qkv == KDA_BF16 && dk == 128 && dv == 128 && T_total > 0 && T_total < (int64_t(1) << 31);
}

// Polls before a bounded wait of a consumer (a role waiting for another role's data) gives up:
// kDefaultWaitPolls unless kda_testing_set_wait_limit changed it.  Waits that drain work already in
// flight on an abort keep kDefaultWaitPolls.  Either way each wait also ends after 2 s of wall time.
constexpr uint32_t kDefaultWaitPolls = 1u << 26;
uint32_t consumer_wait_polls();

// Each launcher returns cudaSuccess or the launch error.
cudaError_t launch_decode(const DecodeArgs& a);
cudaError_t launch_chunk_simt(const ChunkArgs& a);
// bf16, dk = dv = 128 with a workspace of chunk_wy_workspace_size bytes: the chunk-local kernel
// (launch_chunk_prep) writes every chunk's record, then the scan (launch_chunk_scan) walks them.
size_t chunk_wy_workspace_size(int64_t T_total, int N, int H, int dk, int dv);
// The scan's part of that workspace, after the records: two fp32 [N, H, dk, dv] state arrays.
size_t chunk_scan_state_bytes(int N, int H);
cudaError_t launch_chunk_prep(const ChunkArgs& a);
cudaError_t launch_chunk_scan(const ChunkArgs& a);
// The output epilogue as its own pass over o, for the prefill paths that do not fuse it (the scan
// does): o <- o / rms(o) * norm_weight * sigmoid(out_gate), one warp per (token, head).
cudaError_t launch_output_epilogue(const ChunkArgs& a);

// ---- latent attention (kda_mla_api.cu checks the arguments, kda_mla_*.cu hold the kernels)

// Device address of the current device's sticky flag word (looked up once per device).
cudaError_t device_flags_ptr(unsigned int** out);

constexpr int kMlaLatent = 512, kMlaPe = 64;             // cached channels per token
constexpr int kMlaNope = 128, kMlaV = 128;               // per-head channels of the expanded form
constexpr int kMlaQk = kMlaNope + kMlaPe, kMlaKv = kMlaNope + kMlaV;

// The paged latent cache and the sequences' places in it.
struct MlaCache {
    void* latent;       // [num_pages, page_size, 512] bf16 or e4m3
    void* pe;           // [num_pages, page_size, 64] bf16
    float* scale;       // [num_pages, page_size], e4m3 only
    const int32_t* page_table;  // [B, max_pages]
    int64_t num_pages;
    int page_size, page_shift, max_pages;
    bool e4m3;
};

struct MlaCacheCopyArgs {  // kda_mla_cache_write and kda_mla_cache_read
    MlaCache cache;
    void* latent;  // [T, 512] of the packed side, fp32 or bf16
    void* pe;      // [T, 64]
    const int32_t* cu_seqlens;  // may be NULL: equal lengths T / B
    const int32_t* lens;        // write: seq_lens; read: starts (may be NULL)
    int64_t T;
    int B;
    bool fp32;  // the packed side's type
    unsigned int* flags;
    cudaStream_t stream;
};

struct MlaDecodeArgs {
    const void* q_latent;
    const void* q_pe;
    MlaCache cache;
    const int32_t* seq_lens;
    int B, S, H;
    float scale;
    bool o_fp32;
    void* o;
    float* lse;  // may be NULL
    void* workspace;  // NULL: no sequence is split
    unsigned int* flags;
    uint32_t wait_polls;
    cudaStream_t stream;
};

struct MlaPrefillArgs {
    const void* q;
    const void* kv;
    const void* k_pe;
    const int32_t* cu_q;  // may be NULL: equal lengths
    const int32_t* cu_k;
    int64_t Tq, Tk;
    int B, H;
    bool causal;
    float scale;
    bool o_fp32;
    void* o;
    float* lse;  // may be NULL
    unsigned int* flags;
    uint32_t wait_polls;
    cudaStream_t stream;
};

// Lets `kernel` use `bytes` of dynamic shared memory on the current device, once per device (a bit each in `allowed`).
template <typename K>
inline cudaError_t allow_shared(K kernel, int bytes, std::atomic<uint64_t>& allowed) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (allowed.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    return err;
}

// Launches a kernel that may start while the one before it in the stream ends: it sets itself up and waits for that
// one's memory itself (mla::after_previous()).  Takes 2 us off a kda_mla_decode that follows another kernel.
template <typename... P, typename... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t shared, cudaStream_t stream,
                                A&&... args) {
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

cudaError_t launch_mla_cache_write(const MlaCacheCopyArgs& a);
cudaError_t launch_mla_cache_read(const MlaCacheCopyArgs& a);
size_t mla_decode_workspace_size(int B, int S, int H);
cudaError_t launch_mla_decode(const MlaDecodeArgs& a);
cudaError_t launch_mla_prefill(const MlaPrefillArgs& a);

}  // namespace kda
