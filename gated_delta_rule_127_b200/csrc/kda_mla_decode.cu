// kda_mla_decode.cu -- absorbed latent attention over the paged cache, on the tensor cores.
//
// Per sequence, R query rows (new token, head) at a time against tiles of 64 cached tokens:
//
//     S^T [64 tokens, R]   = C Q_c^T + P Q_p^T      (C [64, 512] latents, P [64, 64] positional keys)
//     W^T                  = 2^(scale log2(e) S^T - m)   (m: running reference per row)
//     O^T [512, R]        += C^T W
//
// Tokens are the M side of the first product and latent channels the M side of the second, so few query rows (R =
// 32 or 64, the N side) still fill the tensor core's M, and the one shared-memory copy of C serves both: as the
// K-major A operand first and as the MN-major A operand (C^T) second.  Each cached byte is read once from
// memory; per tile of 72 KB (bf16) an SM's tensor core needs about 1,100 cycles for R = 32, its share of the
// memory bandwidth about 3,100.
//
// e4m3: the codes are multiplied as they are (kind::f8f6f4).  Queries and weights enter as two e4m3 parts,
// hi = e4m3(x) and lo = e4m3(16 (x - hi)), as 2 R columns of one product whose halves are added (hi + lo / 16) in
// fp32: 4 + 4 significant bits, as many as bf16, without a pass that turns codes into bf16.  A token's scale s
// multiplies its scores after the product and its weight before it; the reference m is the maximum of
// x + log2(s) less 4, so the weights w s that enter the product lie in [0, 2^8.5].
//
// The reference moves only when a new maximum exceeds it by 8 (bf16) or 4.5 + 4 (e4m3) in log2 units; then the
// accumulated output and sums are multiplied by 2^(old - new).  Until then weights above 1 are as exact as any.
//
// Work split: all tiles of all sequences, in order, are cut into G equal ranges, one per CTA (per row tile); a
// sequence that a cut falls into leaves partial (m, l, O) in the workspace, which mla_combine_kernel joins in a
// fixed order.  The cuts are found on the device from seq_lens, so a captured call follows new lengths.
//
// Roles of a CTA's 6 warps: 0-3 softmax, rescaling and output (thread = token, then channel), 4 loads (TMA), 5
// issues the products.
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_mla_common.cuh"
#include "kda_mla_sm100.cuh"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace sm100;

constexpr int TOK = 64;          // tokens per tile
constexpr int THREADS = 192;
constexpr int GROUPS = 148;      // CTAs the work is cut for (one per SM)
constexpr int kSmemMax = 227 * 1024;

template <int R, bool E4M3>
struct Shape {
    static constexpr int NQ = E4M3 ? 2 * R : R;            // columns of the latent products (two parts for e4m3)
    static constexpr int BLOCKS = E4M3 ? 4 : 8;            // 128-byte column blocks of a latent row
    static constexpr int BLK = TOK * 128;                  // one block of a tile
    static constexpr int STAGE = (BLOCKS + 1) * BLK;       // latents, then the positional keys
    static constexpr int STAGES = E4M3 ? 4 : 2;
    static constexpr int QBUFS = !E4M3 && R == 32 ? 2 : 1;
    static constexpr int QBYTES = BLOCKS * NQ * 128 + R * 128;
    static constexpr int PBYTES = NQ * 128;                // rows of 64 tokens (e4m3 uses half of each row)
    static constexpr int OFF_Q = STAGES * STAGE;
    static constexpr int OFF_P = OFF_Q + QBUFS * QBYTES;
    static constexpr int OFF_CTL = OFF_P + PBYTES;
    // tensor memory columns
    static constexpr int S_COLS = E4M3 ? NQ + R : R;       // one score buffer: latent part(s), positional part
    static constexpr int COL_O = 2 * S_COLS;               // four chunks of 128 channels
    static_assert(COL_O + 4 * NQ <= 512, "tensor memory");
};

template <int R, bool E4M3>
struct Ctl {
    uint64_t kv_full[4], kv_empty[4], q_full[2], q_empty[2], s_full[2], p_full, pv_done, drain_bar;
    uint32_t tmem;
    uint32_t abort_word;
    uint32_t bad[4];          // per stage: page slots of the tile with a bad page number
    long long scan[8];        // partial sums of the start search
    int b0, t0;
    long long count, total;
    alignas(16) float scale[E4M3 ? 4 : 1][TOK];  // e4m3: the tokens' scales, per stage
    float qscale[E4M3 ? R : 1];                  // e4m3: the query rows' scales
    float red[2][4][R];       // per tile parity, warp and row: maxima; at a segment's end sums
    alignas(16) float factor[R];                 // per row: rescaling factor; at a segment's end 1 / l
};
template <int R, bool E4M3>
constexpr int kSmemBytes = Shape<R, E4M3>::OFF_CTL + static_cast<int>(sizeof(Ctl<R, E4M3>));
static_assert(kSmemBytes<64, false> <= kSmemMax && kSmemBytes<32, false> <= kSmemMax && kSmemBytes<32, true> <= kSmemMax,
              "shared memory");

// A sequence's cached tokens; a bad length raises the flag and counts as none.
__device__ __forceinline__ int cached_len(const MlaDecodeArgs& a, int b) {
    const int len = a.seq_lens[b];
    if (len < 0 || len > mla::table_reach(a.cache)) {
        raise_flag(a.flags, KDA_DEVFLAG_SEQ_LENS);
        return 0;
    }
    return len;
}
// Tiles of a sequence; an empty one still gets a tile, so that its rows are written.
__device__ __forceinline__ int tiles_of(int len) { return len > 0 ? (len + TOK - 1) / TOK : 1; }

// The workspace: for each CTA, which split sequence starts in it (sequence, last group; -1: none), and two
// partial results (0: of a sequence begun in an earlier group, 1: of one begun here and left unfinished).
struct Part {
    int2* meta;   // [ctas]
    float* m;     // [ctas][2][R]
    float* l;     // [ctas][2][R]
    float* o;     // [ctas][2][R][512]
};
__host__ __device__ inline size_t part_bytes(int ctas, int R) {
    return (static_cast<size_t>(ctas) * sizeof(int2) + 15) / 16 * 16 +
           static_cast<size_t>(ctas) * 2 * R * (2 + kMlaLatent) * sizeof(float);
}
__host__ __device__ inline Part part_of(void* ws, int ctas, int R) {
    Part p;
    p.meta = static_cast<int2*>(ws);
    p.o = reinterpret_cast<float*>(static_cast<char*>(ws) + (static_cast<size_t>(ctas) * sizeof(int2) + 15) / 16 * 16);
    p.m = p.o + static_cast<size_t>(ctas) * 2 * R * kMlaLatent;
    p.l = p.m + static_cast<size_t>(ctas) * 2 * R;
    return p;
}

// A CTA's walk over its range of tiles: one segment per sequence it touches.
struct Walk {
    int b, t, nt, len;       // sequence, first tile of the segment, tiles of the sequence, cached tokens
    int n;                   // tiles of the segment
    long long left;          // tiles of the range from the segment's first on
    __device__ __forceinline__ void open(const MlaDecodeArgs& a) {
        len = cached_len(a, b);
        nt = tiles_of(len);
        n = static_cast<int>(min(static_cast<long long>(nt - t), left));
    }
    __device__ __forceinline__ bool next(const MlaDecodeArgs& a) {
        left -= n;
        if (left <= 0) return false;
        ++b;
        t = 0;
        open(a);
        return true;
    }
};

// Transposed reduction over the 16 lanes of a half warp: on return v[0 .. HH/16) hold the results of heads
// (lane % 16) * (HH / 16) + i, each lane having kept half of its values at every step.
template <int HH, bool MAX>
__device__ __forceinline__ void reduce16(float (&v)[HH], int lane) {
#pragma unroll
    for (int d = 8, n = HH / 2; d > 0; d >>= 1, n >>= 1) {
        const bool up = (lane & d) != 0;
#pragma unroll
        for (int i = 0; i < HH / 2; ++i) {
            if (i < n) {
                const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                const float got = __shfl_xor_sync(0xffffffffu, send, d);
                v[i] = MAX ? fmaxf(keep, got) : keep + got;
            }
        }
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// x as two e4m3 parts each: codes of hi and of 16 (x - hi) for two values
__device__ __forceinline__ void split_e4m3(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
    const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(hi), __NV_E4M3)));
    lo = __nv_cvt_float2_to_fp8x2(make_float2(16.f * (x - h.x), 16.f * (y - h.y)), __NV_SATFINITE, __NV_E4M3);
}

template <int R, bool E4M3, typename TO>
__global__ void __launch_bounds__(THREADS, 1)
mla_decode_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_qp,
                  const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_pe,
                  const __grid_constant__ MlaDecodeArgs a, int row_tiles, int groups) {
    using SH = Shape<R, E4M3>;
    constexpr int HH = R / 2;
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl<R, E4M3>& c = *reinterpret_cast<Ctl<R, E4M3>*>(smem + SH::OFF_CTL);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = blockIdx.x / row_tiles, row0 = (blockIdx.x % row_tiles) * R;
    const int rows = a.S * a.H;

    // ---- the range of this CTA: every thread sums its share of the sequences, then the one that holds the first
    // tile of the range finds its sequence
    {
        const int per = (a.B + THREADS - 1) / THREADS, lo = min(tid * per, a.B), hi = min(lo + per, a.B);
        long long mine = 0;
        for (int b = lo; b < hi; ++b) mine += tiles_of(cached_len(a, b));
        long long upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) c.scan[warp] = upto;
        if (tid == 0) {
            c.abort_word = 0u;
            c.count = 0;
            for (int i = 0; i < SH::STAGES; ++i) {
                mbar_init(&c.kv_full[i], 1);
                mbar_init(&c.kv_empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&c.q_full[i], E4M3 ? 128 : 1);
                mbar_init(&c.q_empty[i], 1);
                mbar_init(&c.s_full[i], 1);
            }
            mbar_init(&c.p_full, 128);
            mbar_init(&c.pv_done, 1);
            mbar_init(&c.drain_bar, 1);
            fence_mbar_init();
        }
        if (warp == 5) tmem_alloc(&c.tmem, 512);
        __syncthreads();
        long long total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) upto += c.scan[w];
            total += c.scan[w];
        }
        // no more ranges than tiles, so that none of those between a split sequence's first and last is empty
        if (total < groups) groups = static_cast<int>(total);
        const long long first = total * group / groups;
        const long long end = group < groups ? total * (group + 1) / groups : first;
        long long at = upto - mine;
        if (a.workspace) {  // cuts fall anywhere
            if (first < end && at <= first && first < upto) {
                int b = lo;
                while (first >= at + tiles_of(cached_len(a, b))) at += tiles_of(cached_len(a, b++));
                c.b0 = b;
                c.t0 = static_cast<int>(first - at);
                c.count = end - first;
            }
        } else if (at < end && upto > first) {  // whole sequences: those whose first tile lies in the range
            int b = lo;
            while (b < hi && at < first) at += tiles_of(cached_len(a, b++));
            // the earliest such sequence opens the range; only the thread whose share it lies in sees it as first
            long long before = at;
            if (b < hi && at < end && (at == 0 || at - (b > 0 ? tiles_of(cached_len(a, b - 1)) : 0) < first)) {
                c.b0 = b;
                c.t0 = 0;
                int e = b;
                while (e < a.B && before < end) before += tiles_of(cached_len(a, e++));
                c.count = before - at;
            }
        }
        if (tid == 0) c.total = total;
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    const uint32_t tmem = c.tmem;
    const RoleWait wait{a.wait_polls, &c.abort_word, a.flags};
    if (a.workspace && tid == 0) part_of(a.workspace, gridDim.x, R).meta[blockIdx.x] = make_int2(-1, -1);

    if (c.count > 0) {
        Walk w;
        w.b = c.b0;
        w.t = c.t0;
        w.left = c.count;
        w.open(a);

        if (warp == 4) {
            // ---------------------------------------------------------------- loads
            const int shift = min(a.cache.page_shift, 6), prow = 1 << shift;     // tokens per box
            const int boxes = TOK >> shift;                                       // page slots of a tile
            uint32_t g = 0, seg = 0, queries = 0;  // tiles and query tiles issued
            bool ok = true;
            do {
                if (!E4M3) {  // the segment's queries
                    const uint32_t qb = seg % SH::QBUFS, qn = seg / SH::QBUFS;
                    ok = wait(&c.q_empty[qb], (qn & 1) ^ 1);
                    if (!ok) break;
                    if (lane == 0) {
                        unsigned char* q = smem + SH::OFF_Q + qb * SH::QBYTES;
                        mbar_arrive_expect_tx(&c.q_full[qb], SH::QBYTES);
                        tma_load_4d(q, &tm_q, 0, row0, 0, w.b, &c.q_full[qb]);
                        tma_load_4d(q + SH::BLOCKS * SH::NQ * 128, &tm_qp, 0, row0, 0, w.b, &c.q_full[qb]);
                    }
                    ++queries;
                    __syncwarp();
                }
                const int32_t* table = a.cache.page_table + static_cast<int64_t>(w.b) * a.cache.max_pages;
                for (int i = 0; i < w.n; ++i, ++g) {
                    const uint32_t st = g % SH::STAGES;
                    const int pos = (w.t + i) * TOK + lane * prow;                // first token of this lane's box
                    bool use = lane < boxes && pos < w.len;
                    int page = use ? table[pos >> a.cache.page_shift] : 0;
                    bool bad = use && (page < 0 || page >= a.cache.num_pages);
                    if (bad) raise_flag(a.flags, KDA_DEVFLAG_PAGE_TABLE);
                    const uint32_t bads = __ballot_sync(0xffffffffu, bad);
                    use = use && !bad;
                    const uint32_t used = __ballot_sync(0xffffffffu, use);
                    ok = wait(&c.kv_empty[st], ((g / SH::STAGES) & 1) ^ 1);
                    if (!ok) break;
                    unsigned char* kv = smem + st * SH::STAGE;
                    if (lane == 0) {
                        c.bad[st] = bads;
                        mbar_arrive_expect_tx(&c.kv_full[st], static_cast<uint32_t>(__popc(used)) * prow *
                                                                  ((SH::BLOCKS + 1) * 128 + (E4M3 ? 4 : 0)));
                    }
                    __syncwarp();
                    if (use) {
                        const int row = static_cast<int>((static_cast<int64_t>(page) << a.cache.page_shift) +
                                                         (pos & (a.cache.page_size - 1)));
                        unsigned char* dst = kv + lane * prow * 128;
                        if (prow == TOK) {  // the whole tile in one box
                            tma_load_3d(dst, &tm_kv, 0, row, 0, &c.kv_full[st]);
                        } else {
#pragma unroll
                            for (int k = 0; k < SH::BLOCKS; ++k)
                                tma_load_3d(dst + k * SH::BLK, &tm_kv, 0, row, k, &c.kv_full[st]);
                        }
                        tma_load_3d(dst + SH::BLOCKS * SH::BLK, &tm_pe, 0, row, 0, &c.kv_full[st]);
                        if (E4M3) bulk_load(&c.scale[st][lane * prow], a.cache.scale + row, prow * 4, &c.kv_full[st]);
                    }
                    __syncwarp();
                }
                ++seg;
            } while (ok && w.next(a));
            if (!ok) {  // let what is in flight land before the block ends
                for (uint32_t i = g > SH::STAGES ? g - SH::STAGES : 0; i < g; ++i)
                    drain(&c.kv_full[i % SH::STAGES], (i / SH::STAGES) & 1);
                for (uint32_t i = queries > SH::QBUFS ? queries - SH::QBUFS : 0; i < queries; ++i)
                    drain(&c.q_full[i % SH::QBUFS], (i / SH::QBUFS) & 1);
            }
        } else if (warp == 5) {
            // ---------------------------------------------------------------- products
            const uint32_t base = smem_u32(smem), qs = base + SH::OFF_Q, ps = base + SH::OFF_P;
            constexpr uint32_t idesc_s = E4M3 ? idesc_e4m3(64, SH::NQ, false, false) : idesc_bf16(64, R, false, false);
            constexpr uint32_t idesc_sp = idesc_bf16(64, R, false, false);
            constexpr uint32_t idesc_o = E4M3 ? idesc_e4m3(128, SH::NQ, true, false) : idesc_bf16(128, R, true, false);
            bool ok = true;
            uint32_t seg = 0;
            // scores of tile number g of the CTA (of segment sg); `last`: the segment's last tile
            auto scores = [&](uint32_t g, uint32_t sg, bool first, bool last) -> bool {
                const uint32_t st = g % SH::STAGES, qb = sg % SH::QBUFS;
                if (first && !wait(&c.q_full[qb], (sg / SH::QBUFS) & 1)) return false;
                if (!wait(&c.kv_full[st], (g / SH::STAGES) & 1)) return false;
                tc_fence_after_sync();
                if (lane == 0) {
                    const uint32_t kv = base + st * SH::STAGE, q = qs + qb * SH::QBYTES;
                    const uint32_t d = tmem + (g & 1) * SH::S_COLS;
#pragma unroll
                    for (int k = 0; k < SH::BLOCKS; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t da = sw128_desc(kv + k * SH::BLK + j * 32, 16, 1024);
                            const uint64_t db = sw128_desc(q + k * SH::NQ * 128 + j * 32, 16, 1024);
                            if (E4M3) mma_f8(d, da, db, idesc_s, k + j > 0);
                            else mma_f16(d, da, db, idesc_s, k + j > 0);
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16(E4M3 ? d + SH::NQ : d, sw128_desc(kv + SH::BLOCKS * SH::BLK + j * 32, 16, 1024),
                                sw128_desc(q + SH::BLOCKS * SH::NQ * 128 + j * 32, 16, 1024), idesc_sp,
                                E4M3 ? j > 0 : 1);
                    mma_commit(&c.s_full[g & 1]);
                    if (last) mma_commit(&c.q_empty[qb]);
                }
                __syncwarp();
                return true;
            };
            uint32_t g = 0;
            bool issued = scores(0, 0, true, w.n == 1);
            ok = issued;
            while (ok) {
                // the next tile's scores go first, so that its softmax overlaps this tile's second product; across
                // segments only where the queries have a buffer of their own
                bool more = true;
                for (int i = 0; i < w.n && ok; ++i, ++g) {
                    Walk nx = w;
                    const bool inside = i + 1 < w.n;
                    more = inside || nx.next(a);
                    if (inside) ok = scores(g + 1, seg, false, i + 2 == w.n);
                    else if (more && SH::QBUFS == 2) ok = scores(g + 1, seg + 1, true, nx.n == 1);
                    if (!ok || !wait(&c.p_full, g & 1)) { ok = false; break; }
                    tc_fence_after_sync();
                    if (lane == 0) {
                        const uint32_t st = g % SH::STAGES, kv = base + st * SH::STAGE;
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch)
#pragma unroll
                            for (int k = 0; k < (E4M3 ? 2 : 4); ++k) {
                                const uint32_t d = tmem + SH::COL_O + ch * SH::NQ;
                                const uint64_t db = sw128_desc(ps + k * 32, 16, 1024);
                                if (E4M3)  // 32 tokens of 128 channels: four groups of 8 tokens, 1024 bytes each
                                    mma_f8(d, sw128_desc(kv + ch * SH::BLK + k * 4096, SH::BLK, 1024), db, idesc_o,
                                           i > 0 || k > 0);
                                else       // 16 tokens of 2 x 64 channels
                                    mma_f16(d, sw128_desc(kv + 2 * ch * SH::BLK + k * 2048, SH::BLK, 1024), db, idesc_o,
                                            i > 0 || k > 0);
                            }
                        mma_commit(&c.kv_empty[st]);
                        mma_commit(&c.pv_done);
                    }
                    __syncwarp();
                    if (!inside && more && SH::QBUFS == 1) ok = scores(g + 1, seg + 1, true, nx.n == 1);
                }
                ++seg;
                if (!ok || !w.next(a)) break;
            }
            if (!ok) {  // let issued products finish before the block ends
                if (lane == 0) mma_commit(&c.drain_bar);
                drain(&c.drain_bar, 0);
            }
        } else {
            // ---------------------------------------------------------------- softmax, rescaling, output
            const int tok = warp * 16 + (lane & 15), half = lane >> 4;
            const float sl2 = a.scale * 1.4426950408889634f;
            const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
            unsigned char* p_tile = smem + SH::OFF_P;
            uint32_t g = 0;
            // ok: this warp's waits so far; stop: some warp's have failed, known to all four at the same barrier
            bool ok = true, stop = false;

            // e4m3: a segment's queries as two e4m3 parts with a power-of-two scale per row; thread = (row, quarter)
            auto load_queries = [&](int b) {
                const int r = tid >> 2, part = tid & 3;
                unsigned char* q = smem + SH::OFF_Q;
                const bool real = row0 + r < rows;
                const int64_t row = static_cast<int64_t>(b) * rows + row0 + r;
                uint4 v[16];
                float m = 0.f;
                bool finite = true;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    v[i] = real ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_latent) +
                                                                 row * kMlaLatent)[part + 4 * i]
                                : make_uint4(0, 0, 0, 0);
                uint4 pe[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    pe[i] = real ? reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_pe) +
                                                                  row * kMlaPe)[2 * part + i]
                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float lo = __uint_as_float(x[j] << 16), hi = __uint_as_float(x[j] & 0xFFFF0000u);
                        finite = finite && isfinite(lo) && isfinite(hi);
                        m = fmaxf(m, fmaxf(fabsf(lo), fabsf(hi)));
                    }
                }
                if (!finite) m = INFINITY;
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // the least k with m <= 448 2^k (448 = 1.75 * 2^8); a row that is not finite gives NaN scores
                const uint32_t bits = __float_as_uint(m);
                int k = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7FFFFFu) > 0x600000u ? 7 : 8);
                k = min(max(k, -100), 120);
                const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                if (part == 0)
                    c.qscale[r] = m == INFINITY ? __uint_as_float(0x7FC00000u)
                                                : __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        split_e4m3(__uint_as_float(x[j] << 16) * inv, __uint_as_float(x[j] & 0xFFFF0000u) * inv, h[j], l[j]);
                    const int ch = (part + 4 * i) * 8;  // first of 8 channels
                    unsigned char* blk = q + (ch >> 7) * SH::NQ * 128;
                    *reinterpret_cast<uint2*>(blk + sw128_byte(r, ch & 127)) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                    *reinterpret_cast<uint2*>(blk + sw128_byte(R + r, ch & 127)) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    *reinterpret_cast<uint4*>(q + SH::BLOCKS * SH::NQ * 128 + sw128_byte(r, (2 * part + i) * 16)) = pe[i];
                fence_async_smem();
                mbar_arrive(&c.q_full[0]);
            };
            if (E4M3) {
                load_queries(w.b);
                group_sync(1, 128);
            }

            while (true) {
                float m[HH], l[HH];
#pragma unroll
                for (int i = 0; i < HH; ++i) { m[i] = -INFINITY; l[i] = 0.f; }
                for (int t = 0; t < w.n; ++t, ++g) {
                    const uint32_t st = g % SH::STAGES;
                    ok = ok && wait(&c.s_full[g & 1], (g >> 1) & 1) && wait(&c.kv_full[st], (g / SH::STAGES) & 1);
                    tc_fence_after_sync();
                    float x[HH];
                    const uint32_t s_at = tmem + lane_base + (g & 1) * SH::S_COLS;
                    float ts = 1.f, ls = 0.f;   // the token's scale and its log2
                    const int pos = (w.t + t) * TOK + tok;
                    const uint32_t bads = c.bad[st];
                    const bool seen = pos < w.len &&
                                      !(bads >> (tok >> min(a.cache.page_shift, 6)) & 1u);
                    if constexpr (E4M3) {
                        float lo[HH], pe[HH];
                        tmem_ld16_x2<HH>(s_at, x);
                        tmem_ld16_x2<HH>(s_at + R, lo);
                        tmem_ld16_x2<HH>(s_at + SH::NQ, pe);
                        if (seen) {
                            ts = c.scale[st][tok];
                            ls = log2f(ts);
                        }
#pragma unroll
                        for (int i = 0; i < HH; ++i)
                            x[i] = sl2 * fmaf((x[i] + 0.0625f * lo[i]) * ts, c.qscale[half * HH + i], pe[i]);
                    } else {
                        if constexpr (R == 32) tmem_ld16_x2<HH>(s_at, x);
                        else tmem_ld32_x2<HH>(s_at, x);
#pragma unroll
                        for (int i = 0; i < HH; ++i) x[i] *= sl2;
                    }
                    const bool edge = (w.t + t + 1) * TOK > w.len - (a.S - 1) || bads != 0u;
                    if (edge) {
#pragma unroll
                        for (int i = 0; i < HH; ++i) {
                            const int s = min((row0 + half * HH + i) / a.H, a.S - 1);
                            if (!seen || pos >= w.len - (a.S - 1 - s)) x[i] = -INFINITY;
                        }
                        // rows of the tile that no query sees hold whatever lay there: zero them, so that their
                        // weight of 0 meets no NaN in the second product (the first one is done with them)
                        if (!seen && half == 0) {
#pragma unroll 1
                            for (int k = 0; k < SH::BLOCKS; ++k)
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    *reinterpret_cast<uint4*>(smem + st * SH::STAGE + k * SH::BLK + tok * 128 + j * 16) =
                                        make_uint4(0, 0, 0, 0);
                        }
                    }
                    // the tile's maximum of each row (e4m3: of x + log2 s)
                    float v[HH];
#pragma unroll
                    for (int i = 0; i < HH; ++i) v[i] = x[i] + ls;
                    reduce16<HH, true>(v, lane);
#pragma unroll
                    for (int i = 0; i < HH / 16; ++i) c.red[g & 1][warp][half * HH + (lane & 15) * (HH / 16) + i] = v[i];
                    stop = group_sync_or(1, 128, !ok);
                    if (stop) break;
                    constexpr float kOver = E4M3 ? 8.5f : 8.f, kBelow = E4M3 ? 4.f : 0.f;
                    bool move = false;
                    float top[HH];
#pragma unroll
                    for (int i = 0; i < HH; ++i) {
                        const int h = half * HH + i;
                        const auto& red = c.red[g & 1];
                        top[i] = fmaxf(fmaxf(red[0][h], red[1][h]), fmaxf(red[2][h], red[3][h]));
                        move = move || top[i] > m[i] + kOver;
                    }
                    move = __any_sync(0xffffffffu, move);
                    // this tile's weights overwrite the last one's, and the output moves: the last product must be done
                    if (g > 0) ok = ok && wait(&c.pv_done, (g - 1) & 1);
                    tc_fence_after_sync();
                    if (move) {  // the same for all 128 threads: every warp has seen the same maxima
#pragma unroll
                        for (int i = 0; i < HH; ++i) {
                            float f = 1.f;
                            if (top[i] > m[i] + kOver) {
                                f = ex2(m[i] - (top[i] - kBelow));
                                m[i] = top[i] - kBelow;
                                l[i] *= f;
                            }
                            if (tid == 0 || tid == 16) c.factor[half * HH + i] = f;
                        }
                        group_sync(1, 128);
                        if (t > 0) {
#pragma unroll 1
                            for (int k = 0; k < 4 * SH::NQ / 32; ++k) {
                                float o[32];
                                const uint32_t at = tmem + lane_base + SH::COL_O + k * 32;
                                tmem_ld32(at, o);
                                const float4* f = reinterpret_cast<const float4*>(c.factor + (k * 32) % R);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4 q = f[i];
                                    o[4 * i] *= q.x; o[4 * i + 1] *= q.y; o[4 * i + 2] *= q.z; o[4 * i + 3] *= q.w;
                                }
                                tmem_st32(at, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    // weights, into the second product's B operand [rows][64 tokens]
                    if constexpr (E4M3) {
#pragma unroll
                        for (int i = 0; i < HH; i += 2) {
                            float e[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                e[j] = ex2(x[i + j] - (m[i + j] == -INFINITY ? 0.f : m[i + j]));
                                l[i + j] += e[j];
                            }
                            uint32_t hi, lo;
                            split_e4m3(e[0] * ts, e[1] * ts, hi, lo);
                            const int r = half * HH + i;
                            p_tile[sw128_byte(r, tok)] = static_cast<unsigned char>(hi);
                            p_tile[sw128_byte(r + 1, tok)] = static_cast<unsigned char>(hi >> 8);
                            p_tile[sw128_byte(R + r, tok)] = static_cast<unsigned char>(lo);
                            p_tile[sw128_byte(R + r + 1, tok)] = static_cast<unsigned char>(lo >> 8);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < HH; ++i) {
                            const float e = ex2(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
                            l[i] += e;
                            *reinterpret_cast<__nv_bfloat16*>(p_tile + sw128_byte(half * HH + i, tok * 2)) = __float2bfloat16_rn(e);
                        }
                    }
                    fence_async_smem();
                    tc_fence_before_sync();
                    mbar_arrive(&c.p_full);
                }
                if (stop) break;

                // ---- the segment's end: sums over its tokens, then the output from tensor memory
                const Walk seg_w = w;
                const bool more = w.next(a);
                if (E4M3 && more) load_queries(w.b);  // while the last product runs
                reduce16<HH, false>(l, lane);
                group_sync(1, 128);  // the last tile's maxima have been read by all
#pragma unroll
                for (int i = 0; i < HH / 16; ++i) c.red[0][warp][half * HH + (lane & 15) * (HH / 16) + i] = l[i];
                ok = ok && wait(&c.pv_done, (g - 1) & 1);
                tc_fence_after_sync();
                if (tid == 0 || tid == 16) {
#pragma unroll
                    for (int i = 0; i < HH; ++i) c.factor[half * HH + i] = m[i];
                }
                stop = group_sync_or(1, 128, !ok);
                if (stop) break;
                const bool whole = seg_w.n == seg_w.nt;
                const Part part = part_of(a.workspace, gridDim.x, R);
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg_w.t == 0 ? 1 : 0);
                if (tid < R) {
                    const auto& red = c.red[0];
                    const float sum = (red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid]);
                    const float mm = c.factor[tid];
                    const int r = row0 + tid;
                    if (whole) {
                        if (a.lse && r < rows)
                            a.lse[static_cast<int64_t>(seg_w.b) * rows + r] = (mm + log2f(sum)) * 0.6931471805599453f;
                    } else {
                        part.m[slot * R + tid] = mm;
                        part.l[slot * R + tid] = sum;
                    }
                    c.factor[tid] = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                }
                if (!whole && tid == 0 && seg_w.t == 0) {  // which groups share this sequence
                    // its first tile is number `x - n + 1`..; the range of group k is [total k / G, total (k + 1) / G)
                    const long long last = c.total * (group + 1) / groups - seg_w.n + seg_w.nt - 1;
                    part.meta[blockIdx.x] = make_int2(seg_w.b, static_cast<int>(((last + 1) * groups - 1) / c.total));
                }
                group_sync(1, 128);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
#pragma unroll 1
                    for (int j = 0; j < R; j += 32) {
                        float o[32];
                        tmem_ld32(tmem + lane_base + SH::COL_O + k * SH::NQ + j, o);
                        if (E4M3) {
                            float lo[32];
                            tmem_ld32(tmem + lane_base + SH::COL_O + k * SH::NQ + R + j, lo);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = fmaf(0.0625f, lo[i], o[i]);
                        }
                        const int ch = k * 128 + warp * 32 + lane;
                        if (whole) {
                            TO* out = static_cast<TO*>(a.o) + (static_cast<int64_t>(seg_w.b) * rows + row0 + j) * kMlaLatent + ch;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (row0 + j + i < rows) out[i * kMlaLatent] = from_f32<TO>(o[i] * c.factor[j + i]);
                        } else {
                            float* out = part.o + (slot * R + j) * kMlaLatent + ch;
#pragma unroll
                            for (int i = 0; i < 32; ++i) out[i * kMlaLatent] = o[i];
                        }
                    }
                }
                tc_fence_before_sync();
                group_sync(1, 128);  // factor and red are free again
                if (!more) break;
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial results of the sequences that the cuts split: block = (CTA of the main kernel in which the
// sequence starts, row), thread = 4 channels.  The parts are added in the order of their groups.
template <typename TO>
__global__ void __launch_bounds__(128) mla_combine_kernel(MlaDecodeArgs a, int R, int row_tiles, int ctas) {
    const Part p = part_of(a.workspace, ctas, R);
    const int cta = blockIdx.x, group = cta / row_tiles, rt = cta % row_tiles, i = blockIdx.y;
    const int rows = a.S * a.H, r = rt * R + i;
    if (r >= rows) return;
    const int2 meta = p.meta[cta];
    if (meta.x < 0) return;
    const int n = meta.y - group + 1;
    auto index = [&](int k) {  // row of part k
        return ((static_cast<int64_t>(group + k) * row_tiles + rt) * 2 + (k == 0 ? 1 : 0)) * R + i;
    };
    __shared__ float wgt[GROUPS];
    __shared__ float red[4];
    const int tid = threadIdx.x;
    float m = -INFINITY;
    for (int k = tid; k < n; k += 128) m = fmaxf(m, p.m[index(k)]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    for (int k = tid; k < n; k += 128) {
        const float mk = p.m[index(k)];
        wgt[k] = mk == -INFINITY ? 0.f : ex2(mk - m);
    }
    __syncthreads();
    float l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const float f = wgt[k];
        const float4 v = *reinterpret_cast<const float4*>(p.o + index(k) * kMlaLatent + tid * 4);
        l = fmaf(f, p.l[index(k)], l);
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    }
    const int64_t row = static_cast<int64_t>(meta.x) * rows + r;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    TO* out = static_cast<TO*>(a.o) + row * kMlaLatent + tid * 4;
    out[0] = from_f32<TO>(o.x * inv); out[1] = from_f32<TO>(o.y * inv);
    out[2] = from_f32<TO>(o.z * inv); out[3] = from_f32<TO>(o.w * inv);
    if (a.lse && tid == 0) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
}

// Query rows per CTA: 32, or 64 where a sequence has more rows than 32 and the cache is bf16 (the e4m3 form needs the
// tensor memory for its two parts).
int tile_rows(int S, int H, bool e4m3) { return !e4m3 && S * H > 32 ? 64 : 32; }

struct Grid { int R, row_tiles, groups; };
Grid grid_of(int S, int H, bool e4m3) {
    Grid g;
    g.R = tile_rows(S, H, e4m3);
    g.row_tiles = (S * H + g.R - 1) / g.R;
    g.groups = g.row_tiles >= GROUPS ? 1 : GROUPS / g.row_tiles;
    return g;
}

bool encode(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
    auto fn = tma_encode_fn();
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return fn && fn(m, dt, rank, const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [B, rows, d] as {64 channels, rows, d / 64 blocks, B}: one box is a row tile of one sequence, block after
// block; rows past the sequence's own read as zero.
bool encode_q(CUtensorMap* m, const void* q, int d, int rows, int B, int R) {
    const cuuint64_t dims[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(d / 64),
                                static_cast<cuuint64_t>(B)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, 128, static_cast<cuuint64_t>(d) * 2 * rows};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(R), static_cast<cuuint32_t>(d / 64), 1};
    return encode(m, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims, strides, box);
}

// A cache array [pool rows, row_bytes] as {128 bytes, pool rows, blocks}.
bool encode_pool(CUtensorMap* m, const void* base, int esize, int64_t pool_rows, int blocks, int box_rows,
                 int box_blocks) {
    const cuuint64_t inner = static_cast<cuuint64_t>(128 / esize);
    const cuuint64_t dims[3] = {inner, static_cast<cuuint64_t>(pool_rows), static_cast<cuuint64_t>(blocks)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(blocks) * 128, 128};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(inner), static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(box_blocks)};
    return encode(m, base, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims,
                  strides, box);
}

template <int R, bool E4M3, typename TO>
cudaError_t launch(const MlaDecodeArgs& a, const Grid& g) {
    using SH = Shape<R, E4M3>;
    constexpr int smem = kSmemBytes<R, E4M3>;
    auto kernel = mla_decode_kernel<R, E4M3, TO>;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    CUtensorMap q, qp, kv, pe;
    const int rows = a.S * a.H, box = a.cache.page_size < TOK ? a.cache.page_size : TOK;
    // a cache without pages is never loaded from (every page number is out of range): any valid map serves
    const bool none = a.cache.num_pages == 0;
    const int64_t pool = none ? 1 : a.cache.num_pages * a.cache.page_size;
    const void* latent = none ? a.q_latent : a.cache.latent;
    const void* cpe = none ? a.q_pe : a.cache.pe;
    if (!encode_q(&q, a.q_latent, kMlaLatent, rows, a.B, R) || !encode_q(&qp, a.q_pe, kMlaPe, rows, a.B, R) ||
        !encode_pool(&kv, latent, E4M3 ? 1 : 2, pool, SH::BLOCKS, box, box == TOK ? SH::BLOCKS : 1) ||
        !encode_pool(&pe, cpe, 2, pool, 1, box, 1))
        return cudaErrorInvalidValue;
    const int ctas = g.groups * g.row_tiles;
    kernel<<<ctas, THREADS, smem, a.stream>>>(q, qp, kv, pe, a, g.row_tiles, g.groups);
    err = cudaGetLastError();
    if (err != cudaSuccess || !a.workspace) return err;
    mla_combine_kernel<TO><<<dim3(ctas, R), 128, 0, a.stream>>>(a, R, g.row_tiles, ctas);
    return cudaGetLastError();
}

template <typename TO>
cudaError_t dispatch(const MlaDecodeArgs& a) {
    const Grid g = grid_of(a.S, a.H, a.cache.e4m3);
    MlaDecodeArgs b = a;
    if (g.groups == 1) b.workspace = nullptr;  // nothing is split
    if (a.cache.e4m3) return launch<32, true, TO>(b, g);
    return g.R == 64 ? launch<64, false, TO>(b, g) : launch<32, false, TO>(b, g);
}

}  // namespace

size_t mla_decode_workspace_size(int, int S, int H) {
    size_t most = 0;
    for (const bool e4m3 : {false, true}) {
        const Grid g = grid_of(S, H, e4m3);
        if (g.groups > 1) most = std::max(most, part_bytes(g.groups * g.row_tiles, g.R));
    }
    return most;
}

cudaError_t launch_mla_decode(const MlaDecodeArgs& a) {
    return a.o_fp32 ? dispatch<float>(a) : dispatch<__nv_bfloat16>(a);
}

}  // namespace kda
