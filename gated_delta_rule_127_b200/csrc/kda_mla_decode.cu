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
// memory bandwidth about 3,000: memory is the bound, and the rings keep as much of it in flight as shared memory holds.
//
// e4m3: the codes are multiplied as they are (kind::f8f6f4).  Queries and weights enter as two e4m3 parts,
// hi = e4m3(x) and lo = e4m3(16 (x - hi)), as 2 R columns of one product whose halves are added (hi + lo / 16) in
// fp32: 4 + 4 significant bits, as many as bf16 (down to 2^-6), without a pass that turns codes into bf16.  A token's scale s
// multiplies its scores after the product and its weight before it; the reference m is the maximum of
// x + log2(s) less 4, so the weights w s that enter the product lie in [0, 2^8.5].
//
// The reference rises only when a new maximum exceeds it by 8 (bf16) or 4.5 + 4 (e4m3) in log2 units; then the
// accumulated output and sums are multiplied by 2^(old - new).  Until then weights above 1 are as exact as any.
//
// e4m3: it falls, too.  The two parts end at 2^-13: a small w s is off by up to 2^-14, and below that it is 0.  Under a
// reference that only rises, one heavy token (2^4) takes the tail of a long sequence out of the output while l still
// counts it: 5% of the output for 131,072 tokens 13 nats below the first one.  So every 8 tiles (and once early, as the
// heavy token is mostly the first) each row looks at what the tokens since the last look weigh, e = sum w s.  From 8 on, their
// 512 x 2^-14 are 2^-8 of that at most, as much as the rounding of a bf16 weight.  Below, the reference falls to where they
// would have weighed 16 to 32: then what they have lost is at most 2^-9 of the heavy token's 2^4, each time a quarter of the
// time before.  At most 20 below its highest place: there 2^30 tokens that weigh nothing are 2^-8 of that token, and O and l
// stay far from fp32's end.  A look takes some 300 cycles beside a tile's 1,800: with looks at every 4th, 8th and 16th tile
// one sequence of 1,000,001 tokens took 141, 138 and 137 us, without any 136.
//
// Work split: all tiles of all sequences, in order, are cut into G equal ranges, one per CTA (per row tile), with a
// few tiles' worth added before each sequence for what it costs to begin and end one (queries, first maxima, output:
// about 8,000 cycles against 1,800 per e4m3 tile, 6,000 against 3,200 per bf16 tile; without it the CTAs with
// the most sequences finished 20% after the median of a batch of 128).  A sequence that a cut falls into leaves
// partial (m, l, O) in the workspace, which mla_combine_kernel joins in a fixed order.  The cuts are found on the device
// from seq_lens, so a captured call follows new lengths.
//
// Bound by memory.  Measured, calls in a row: one sequence of 1,000,001 tokens, 32 heads, bf16 184 us (6.3 TB/s); 64 of
// 1,024 to 16,384 tokens 125 us (5.6 TB/s; 5.9 while this kernel runs); 128 of 1 to 8,000 tokens, 2 x 16 rows, e4m3, pages
// of 16 80 us (4.4 TB/s).  A call alone on new inputs and a cold L2 takes 207, 133 and 95 us.  What is over the copy rate: 4 us until the first loads, 8,000 cycles where a CTA passes from one sequence to
// the next and its rings stand full, 7 us from the first CTA's end to the joined result.
//
// Roles of a CTA's 11 warps: 0-3 and 4-7 softmax, rescaling and output, each group of four for half of the rows and
// independent of the other (thread = token, then channel); 8 loads (TMA); 9 issues the first products, 10 the second
// ones (issuing 16 to 36 of them takes as long as they run: one warp for both would keep a tile's finished weights
// waiting behind the next tile's scores).
#include <cuda_fp8.h>

#include <algorithm>

#include "kda_mla_common.cuh"
#include "kda_mla_sm100.cuh"
#include "kda_mla_split.h"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace sm100;
using mla::group_of;
using mla::scaled;

constexpr int TOK = 64;          // tokens per tile
constexpr int THREADS = 352;
constexpr int GROUPS = 148;      // CTAs the work is cut for (one per SM)
constexpr int kSmemMax = 227 * 1024;

template <int R, bool E4M3>
struct Shape {
    static constexpr int NQ = E4M3 ? 2 * R : R;            // columns of the latent products (two parts for e4m3)
    static constexpr int BLOCKS = E4M3 ? 4 : 8;            // 128-byte column blocks of a latent row
    static constexpr int BLK = TOK * 128;                  // one block of a tile
    // Four blocks of latents, the ring's unit, as 8 groups of 8 tokens with 4 blocks of 1 KB each: then one box brings the
    // four blocks of a page of any size, and 8-token groups lie evenly apart for the products.  (As four blocks of 64
    // tokens, a tile of 16-token pages took 24 copies.)
    static constexpr int PIECE = 4 * BLK;
    static constexpr int ATOM = 1024, GROUP = 4 * ATOM;
    static constexpr int NP = BLOCKS / 4;                  // pieces of a tile
    static constexpr int PIECES = R == 32 ? 5 : 4;
    static constexpr int PES = R == 32 ? 3 : 2;            // tiles of positional keys
    static constexpr int SLOTS = (PIECES + NP - 1) / NP;   // tiles in flight, the one being freed included
    static constexpr int QBYTES = BLOCKS * NQ * 128 + R * 128;
    static constexpr int PROW = E4M3 ? NQ : NQ * 2;        // weights: one row of all columns per token, 64 or 128 bytes
    static constexpr int PBYTES = TOK * PROW;
    static constexpr int OFF_PE = PIECES * PIECE;
    static constexpr int OFF_Q = OFF_PE + PES * BLK;
    static constexpr int OFF_P = OFF_Q + QBYTES;
    static constexpr int OFF_CTL = OFF_P + PBYTES;
    // tensor memory columns
    static constexpr int S_COLS = E4M3 ? NQ + R : R;       // one score buffer: latent part(s), positional part
    static constexpr int COL_O = 2 * S_COLS;               // four chunks of 128 channels
    static constexpr int LEAD = E4M3 ? 4 : 2;              // tiles that a sequence costs besides its own
    static_assert(COL_O + 4 * NQ <= 512, "tensor memory");
};

template <int R, bool E4M3>
struct Ctl {
    uint64_t kv_full[5], kv_empty[5], pe_empty[3], q_full, q_empty, s_full[2], s_empty[2], p_full, pv_done, drain_bar[2];
    uint32_t tmem;
    uint32_t abort_word;
    uint32_t bad[5];          // per tile in flight: page slots of the tile with a bad page number
    long long scan[THREADS / 32];  // partial sums of the start search
    int b0, t0;
    long long first, end, left, total;  // the range of this CTA, the tiles of it from t0 on (and later leads), all
    alignas(16) float scale[E4M3 ? Shape<R, E4M3>::SLOTS : 1][TOK];  // e4m3: the tokens' scales, per tile in flight
    alignas(16) float qscale[E4M3 ? R : 4];      // e4m3: the query rows' scales
    alignas(16) float red[4][R];          // per warp and row: maxima; at a segment's end sums
    alignas(16) float factor[R];                 // per row: rescaling factor; at a segment's end 1 / l
    alignas(16) float mass[4][E4M3 ? R : 4];     // e4m3, per warp and row: what a window's tokens weigh
    alignas(16) float lowest[E4M3 ? R : 4];      // e4m3, per row: where the reference may fall to
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

// The workspace: two partial results per CTA (0: of a sequence begun in an earlier group, 1: of one begun here and
// left unfinished), and for each of them its sequence (-1: none) and the first and last group that share it.
struct Part {
    int4* meta;   // [ctas][2]
    float* m;     // [ctas][2][R]
    float* l;     // [ctas][2][R]
    float* o;     // [ctas][2][R][512]
};
__host__ __device__ inline size_t part_bytes(int ctas, int R) {
    return static_cast<size_t>(ctas) * 2 * (sizeof(int4) + R * (2 + kMlaLatent) * sizeof(float));
}
__host__ __device__ inline Part part_of(void* ws, int ctas, int R) {
    Part p;
    p.meta = static_cast<int4*>(ws);
    p.o = reinterpret_cast<float*>(p.meta + static_cast<size_t>(ctas) * 2);
    p.m = p.o + static_cast<size_t>(ctas) * 2 * R * kMlaLatent;
    p.l = p.m + static_cast<size_t>(ctas) * 2 * R;
    return p;
}

// A CTA's walk over its range of tiles: one segment per sequence it touches.
template <int LEAD>
struct Walk {
    int b, t, nt, len;       // sequence, first tile of the segment, tiles of the sequence, cached tokens
    int n;                   // tiles of the segment
    long long left;          // what is left of the range from the segment's first tile on
    __device__ __forceinline__ void open(const MlaDecodeArgs& a) {
        len = cached_len(a, b);
        nt = tiles_of(len);
        n = static_cast<int>(min(static_cast<long long>(nt - t), left));
    }
    __device__ __forceinline__ bool next(const MlaDecodeArgs& a) {
        left -= n + LEAD;
        if (left <= 0) return false;
        ++b;
        t = 0;
        open(a);
        return true;
    }
};

// Transposed reduction over the 16 lanes of a half warp, each lane keeping half of its values at every step: on return
// v[i] is the result of row (lane % 16) * HH / 16 + i (HH = 8: two lanes have the same row).
template <int HH, bool MAX>
__device__ __forceinline__ void reduce16(float (&v)[HH], int lane) {
#pragma unroll
    for (int d = 8, n = HH / 2; d > 0; d >>= 1, n >>= 1) {
        const bool up = (lane & d) != 0;
        if (n == 0) {
            const float got = __shfl_xor_sync(0xffffffffu, v[0], d);
            v[0] = MAX ? fmaxf(v[0], got) : v[0] + got;
        }
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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
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
    constexpr int HH = R / 4;  // rows per softmax thread
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl<R, E4M3>& c = *reinterpret_cast<Ctl<R, E4M3>*>(smem + SH::OFF_CTL);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = blockIdx.x / row_tiles, row0 = (blockIdx.x % row_tiles) * R;
    const int rows = a.S * a.H;

    // ---- the range of this CTA: every thread sums its share of the sequences, then the one that holds the range's
    // first place finds its sequence
    {
        if (tid == 0) {
            c.abort_word = 0u;
            c.left = 0;
            for (int i = 0; i < 5; ++i) {
                mbar_init(&c.kv_full[i], SH::NP);
                mbar_init(&c.kv_empty[i], 1);
            }
            for (int i = 0; i < 3; ++i) mbar_init(&c.pe_empty[i], 1);
            mbar_init(&c.q_full, E4M3 ? 8 : 1);
            mbar_init(&c.q_empty, 1);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&c.s_full[i], 1);
                mbar_init(&c.s_empty[i], 8);
            }
            mbar_init(&c.p_full, 8);
            mbar_init(&c.pv_done, 1);
            mbar_init(&c.drain_bar[0], 1);
            mbar_init(&c.drain_bar[1], 1);
            fence_mbar_init();
        }
        if (warp == 9) tmem_alloc(&c.tmem, 512);
        if (warp == 8 && lane < 4) tma_prefetch_desc(lane == 0 ? &tm_kv : lane == 1 ? &tm_pe : lane == 2 ? &tm_q : &tm_qp);
        mla::after_previous();
        const int per = (a.B + THREADS - 1) / THREADS, lo = min(tid * per, a.B), hi = min(lo + per, a.B);
        const auto places = [&](int b) { return tiles_of(cached_len(a, b)) + SH::LEAD; };
        long long mine = 0;
        for (int b = lo; b < hi; ++b) mine += places(b);
        long long upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) c.scan[warp] = upto;
        __syncthreads();
        long long total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) upto += c.scan[w];
            total += c.scan[w];
        }
        // no more ranges than tiles, so that none of those between a split sequence's first and last is empty
        if (total < groups) groups = static_cast<int>(total);
        const long long first = scaled(total, group, groups);
        const long long end = group < groups ? scaled(total, group + 1, groups) : first;
        long long at = upto - mine;
        if (a.workspace) {  // cuts fall anywhere
            if (first < end && at <= first && first < upto) {
                int b = lo;
                while (first >= at + places(b)) at += places(b++);
                const long long in = first - at;  // places of the sequence before the cut
                c.b0 = b;
                c.t0 = static_cast<int>(max(in - SH::LEAD, 0LL));
                c.left = end - max(first, at + SH::LEAD);
            }
        } else if (at < end && upto > first) {  // whole sequences: those whose first place lies in the range
            int b = lo;
            while (b < hi && at < first) at += places(b++);
            // the earliest such sequence opens the range; only the thread whose share it lies in sees it as first
            if (b < hi && at < end && (b == 0 || at - places(b - 1) < first)) {
                c.b0 = b;
                c.t0 = 0;
                long long upto_b = at;
                for (int e = b; e < a.B && upto_b < end; ++e) upto_b += places(e);
                c.left = upto_b - at - SH::LEAD;
            }
        }
        if (tid == 0) {
            c.first = first;
            c.end = end;
            c.total = total;
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    // the joining kernel may be set up now; it waits for this one's end itself
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const uint32_t tmem = c.tmem;
    const RoleWait wait{a.wait_polls, &c.abort_word, a.flags};
    if (a.workspace && tid == 0)
        for (int i = 0; i < 2; ++i) part_of(a.workspace, gridDim.x, R).meta[blockIdx.x * 2 + i] = make_int4(-1, 0, 0, 0);

    if (c.left > 0) {
        Walk<SH::LEAD> w;
        w.b = c.b0;
        w.t = c.t0;
        w.left = c.left;
        w.open(a);

        if (warp == 8) {
            // ---------------------------------------------------------------- loads
            // A tile's copies: per page slot of up to 64 tokens the latent blocks (a box of four), the positional keys and
            // the scales, each as soon as its place in the ring is free.  A tile's page numbers are read, by all lanes
            // alike, a tile ahead.  (One lane per slot and shuffles took 1,500 cycles a tile, as shuffles queue behind the
            // other warps' shared-memory traffic, and bound the e4m3 form.)
            const int shift = min(a.cache.page_shift, 6), prow = 1 << shift, slots = TOK >> shift;
            uint32_t g = 0, n = 0;  // tiles and pieces issued
            bool ok = true;
            do {
                const int32_t* table = a.cache.page_table + static_cast<int64_t>(w.b) * a.cache.max_pages;
                const auto fetch = [&](int (&page)[4], int i) {
                    const int pos = (w.t + i) * TOK;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        page[x] = x < slots && i < w.n && pos + x * prow < w.len
                                      ? __ldg(table + ((pos + x * prow) >> a.cache.page_shift))
                                      : 0;
                };
                int page[4];
                fetch(page, 0);
                for (int i = 0; i < w.n; ++i, ++g) {
                    const uint32_t slot = g % SH::SLOTS;
                    const int pos = (w.t + i) * TOK;
                    uint32_t bads = 0u, used = 0u;
                    int row[4];  // pool row of each slot's first token
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const bool real = x < slots && pos + x * prow < w.len;
                        const bool good = page[x] >= 0 && page[x] < a.cache.num_pages;
                        bads |= real && !good ? 1u << x : 0u;
                        used |= real && good ? 1u << x : 0u;
                        row[x] = static_cast<int>((static_cast<uint32_t>(page[x]) << a.cache.page_shift) +
                                                  ((pos + x * prow) & (a.cache.page_size - 1)));
                    }
                    if (bads) raise_flag(a.flags, KDA_DEVFLAG_PAGE_TABLE);
                    fetch(page, i + 1);
                    const uint32_t tokens = static_cast<uint32_t>(__popc(used)) * prow, at_pe = g % SH::PES;
                    int done = 0;  // arrivals for the tile
                    for (; done < SH::NP; ++done, ++n) {
                        const uint32_t at = n % SH::PIECES, turn = ((n / SH::PIECES) & 1) ^ 1;
                        ok = done == 0 ? wait.both(&c.kv_empty[at], turn, &c.pe_empty[at_pe], ((g / SH::PES) & 1) ^ 1)
                                       : wait(&c.kv_empty[at], turn);
                        if (!ok) break;
                        unsigned char* kv = smem + at * SH::PIECE;
                        if (elect_one()) {
                            if (done == 0) c.bad[slot] = bads;
                            mbar_arrive_expect_tx(&c.kv_full[slot], tokens * (512 + (done == 0 ? 128 + (E4M3 ? 4 : 0) : 0)));
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                if (used >> x & 1u) {
                                    tma_load_4d(kv + x * prow * 512, &tm_kv, 0, 0, done * 4, row[x] >> 3, &c.kv_full[slot]);
                                    if (done == 0) {
                                        tma_load_3d(smem + SH::OFF_PE + at_pe * SH::BLK + x * prow * 128, &tm_pe, 0, row[x], 0,
                                                    &c.kv_full[slot]);
                                        if (E4M3)
                                            bulk_load(&c.scale[slot][x * prow], a.cache.scale + row[x], prow * 4, &c.kv_full[slot]);
                                    }
                                }
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) {  // the rest of the tile stays empty
                        if (lane == 0)
                            for (; done < SH::NP; ++done) mbar_arrive(&c.kv_full[slot]);
                        __syncwarp();
                        ++g;
                        break;
                    }
                }
            } while (ok && w.next(a));
            if (!ok) {  // let what is in flight land before the block ends
                for (uint32_t i = g > SH::SLOTS ? g - SH::SLOTS : 0; i < g; ++i)
                    drain(&c.kv_full[i % SH::SLOTS], (i / SH::SLOTS) & 1);
            }
        } else if (warp == 9) {
            // ---------------------------------------------------------------- first products: scores
            const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0), qs = base + SH::OFF_Q;
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            constexpr uint32_t idesc_s = E4M3 ? idesc_e4m3(64, SH::NQ, false, false) : idesc_bf16(64, R, false, false);
            constexpr uint32_t idesc_p = idesc_bf16(64, R, false, false);
            uint32_t g = 0, seg = 0;
            bool ok = true;
            do {
                if (!E4M3) {  // the segment's queries, once the last one's scores are done
                    ok = wait(&c.q_empty, (seg & 1) ^ 1);
                    if (!ok) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&c.q_full, SH::QBYTES);
                        tma_load_4d(smem + SH::OFF_Q, &tm_q, 0, row0, 0, w.b, &c.q_full);
                        tma_load_4d(smem + SH::OFF_Q + SH::BLOCKS * SH::NQ * 128, &tm_qp, 0, row0, 0, w.b, &c.q_full);
                    }
                    __syncwarp();
                }
                ok = wait(&c.q_full, seg & 1);
                if (!E4M3 && !ok) drain(&c.q_full, seg & 1);
                for (int i = 0; i < w.n && ok; ++i) {
                    ok = wait.both(&c.s_empty[g & 1], ((g >> 1) & 1) ^ 1, &c.kv_full[g % SH::SLOTS], (g / SH::SLOTS) & 1);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t d = tm + (g & 1) * SH::S_COLS;
                    const uint64_t q0 = sw128_desc(qs, 16, 1024), p0 = sw128_desc(base + SH::OFF_PE + g % SH::PES * SH::BLK, 16, 1024);
                    uint64_t k0[SH::NP];
#pragma unroll
                    for (int h = 0; h < SH::NP; ++h)
                        k0[h] = sw128_desc(base + (g * SH::NP + h) % SH::PIECES * SH::PIECE, 16, SH::GROUP);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < SH::BLOCKS; ++k)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint64_t da = k0[k / 4] + ((k % 4 * SH::ATOM + j * 32) >> 4);
                                const uint64_t db = q0 + ((k * SH::NQ * 128 + j * 32) >> 4);
                                if (E4M3) mma_f8(d, da, db, idesc_s, k + j > 0);
                                else mma_f16(d, da, db, idesc_s, k + j > 0);
                            }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_f16(E4M3 ? d + SH::NQ : d, p0 + ((j * 32) >> 4),
                                    q0 + ((SH::BLOCKS * SH::NQ * 128 + j * 32) >> 4), idesc_p, E4M3 ? j > 0 : 1);
                        mma_commit(&c.s_full[g & 1]);
                        mma_commit(&c.pe_empty[g % SH::PES]);
                        if (!E4M3 && i + 1 == w.n) mma_commit(&c.q_empty);
                    }
                    __syncwarp();
                    ++g;
                }
                ++seg;
            } while (ok && w.next(a));
            if (!ok) {  // let issued products finish before the block ends
                if (elect_one()) mma_commit(&c.drain_bar[0]);
                __syncwarp();
                drain(&c.drain_bar[0], 0);
            }
        } else if (warp == 10) {
            // ---------------------------------------------------------------- second products: weighted latents
            const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint64_t ps = SH::PROW == 128 ? sw128_desc(base + SH::OFF_P, 16, 1024) : sw64_desc(base + SH::OFF_P, 16, 512);
            constexpr uint32_t idesc_o = E4M3 ? idesc_e4m3(128, SH::NQ, true, true) : idesc_bf16(128, R, true, true);
            uint32_t g = 0;
            bool ok = true;
            do {
                for (int i = 0; i < w.n; ++i) {
                    ok = wait(&c.p_full, g & 1);
                    if (!ok) break;
                    tc_fence_after_sync();
                    uint32_t at[SH::NP];
                    uint64_t v0[SH::NP];
#pragma unroll
                    for (int h = 0; h < SH::NP; ++h) {
                        at[h] = (g * SH::NP + h) % SH::PIECES;
                        v0[h] = sw128_desc(base + at[h] * SH::PIECE, SH::ATOM, SH::GROUP);
                    }
                    if (elect_one()) {
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch) {
#pragma unroll
                            for (int k = 0; k < (E4M3 ? 2 : 4); ++k) {
                                const uint32_t d = tm + SH::COL_O + ch * SH::NQ;
                                const uint64_t pk = ps + ((k * (E4M3 ? 32 : 16) * SH::PROW) >> 4);
                                if (E4M3)  // 32 tokens of 128 channels
                                    mma_f8(d, v0[0] + ((ch * SH::ATOM + k * 4 * SH::GROUP) >> 4), pk, idesc_o, i > 0 || k > 0);
                                else       // 16 tokens of 2 x 64 channels
                                    mma_f16(d, v0[ch / (4 / SH::NP)] + ((ch % 2 * 2 * SH::ATOM + k * 2 * SH::GROUP) >> 4), pk, idesc_o, i > 0 || k > 0);
                            }
                            if (ch % (4 / SH::NP) == 4 / SH::NP - 1) mma_commit(&c.kv_empty[at[ch / (4 / SH::NP)]]);
                        }
                        mma_commit(&c.pv_done);
                    }
                    __syncwarp();
                    ++g;
                }
            } while (ok && w.next(a));
            if (!ok) {
                if (elect_one()) mma_commit(&c.drain_bar[1]);
                __syncwarp();
                drain(&c.drain_bar[1], 0);
            }
        } else {
            // ---------------------------------------------------------------- softmax, rescaling, output
            // a warp reads the accumulators' lanes 32 (warp % 4) ..; of a score tile's 64 tokens that is 16, so its halves
            // take a quarter of the rows each
            const int wg = warp >> 2, sub = warp & 3, tok = sub * 16 + (lane & 15), half = lane >> 4;
            const int bar = 1 + wg, h0 = wg * (R / 2) + half * HH;  // named barrier, first row of this thread
            const bool writer = sub == 0 && (lane & 15) == 0;
            const float sl2 = a.scale * 1.4426950408889634f;
            constexpr float kOver = E4M3 ? 8.5f : 8.f, kBelow = E4M3 ? 4.f : 0.f, kFall = 20.f;
            constexpr int kWindow = 8;  // e4m3: tiles between two looks at what the tokens weigh
            const uint32_t lane_base = static_cast<uint32_t>(sub * 32) << 16;
            unsigned char* p_tile = smem + SH::OFF_P;
            // this thread's first row: new token and head (rows past the sequence's own are never stored)
            const int new0 = (row0 + h0) / a.H, head0 = (row0 + h0) % a.H;
            uint32_t g = 0;
            // ok: this warp's waits so far; stop: some warp's have failed, known to all four at the same barrier
            bool ok = true, stop = false;

            // e4m3: a segment's queries as two e4m3 parts with a power-of-two scale per row; thread = (row, eighth)
            auto load_queries = [&](int b) {
                const int r = tid >> 3, part = tid & 7;
                unsigned char* q = smem + SH::OFF_Q;
                const bool real = row0 + r < rows;
                const int64_t row = static_cast<int64_t>(b) * rows + row0 + r;
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = real ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_latent) +
                                                                       row * kMlaLatent) + part + 8 * i)
                                : make_uint4(0, 0, 0, 0);
                const uint4 pe = real ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q_pe) +
                                                                             row * kMlaPe) + part)
                                      : make_uint4(0, 0, 0, 0);
                __nv_bfloat162 top = __nv_bfloat162(__float2bfloat16(0.f), __float2bfloat16(0.f));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&x[j])));
                }
                const float t0 = __low2float(top), t1 = __high2float(top);
                float m = isfinite(t0) && isfinite(t1) ? fmaxf(t0, t1) : INFINITY;
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                // the least k with m <= 448 2^k (448 = 1.75 * 2^8); a row that is not finite gives NaN scores
                const uint32_t bits = __float_as_uint(m);
                int k = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7FFFFFu) > 0x600000u ? 7 : 8);
                k = min(max(k, -100), 120);
                const float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
                if (part == 0)
                    c.qscale[r] = m == INFINITY ? __uint_as_float(0x7FC00000u)
                                                : __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t h[4], l[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        split_e4m3(__uint_as_float(x[j] << 16) * inv, __uint_as_float(x[j] & 0xFFFF0000u) * inv, h[j], l[j]);
                    const int ch = (part + 8 * i) * 8;  // first of 8 channels
                    unsigned char* blk = q + (ch >> 7) * SH::NQ * 128;
                    *reinterpret_cast<uint2*>(blk + sw128_byte(r, ch & 127)) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
                    *reinterpret_cast<uint2*>(blk + sw128_byte(R + r, ch & 127)) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
                }
                *reinterpret_cast<uint4*>(q + SH::BLOCKS * SH::NQ * 128 + sw128_byte(r, part * 16)) = pe;
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.q_full);
            };
            if (E4M3) {
                load_queries(w.b);
                group_sync(bar, 128);
            }

            while (true) {
                float m[HH], l[HH], e[E4M3 ? HH : 1] = {};  // e: what the tokens since the last look weigh
#pragma unroll
                for (int i = 0; i < HH; ++i) { m[i] = -INFINITY; l[i] = 0.f; }
                if (E4M3 && writer)
#pragma unroll
                    for (int i = 0; i < HH; ++i) c.lowest[h0 + i] = -INFINITY;
                if (E4M3 && w.left > w.n + SH::LEAD && row0 + (tid >> 3) < rows)  // the next segment's queries, into L2
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(
                        static_cast<const __nv_bfloat16*>(a.q_latent) +
                        (static_cast<int64_t>(w.b + 1) * rows + row0 + (tid >> 3)) * kMlaLatent + (tid & 7) * 64));
                for (int t = 0; t < w.n; ++t, ++g) {
                    const uint32_t slot = g % SH::SLOTS;
                    ok = ok && wait.both(&c.kv_full[slot], (g / SH::SLOTS) & 1, &c.s_full[g & 1], (g >> 1) & 1);
                    tc_fence_after_sync();
                    float x[HH];
                    const uint32_t s_at = tmem + lane_base + (g & 1) * SH::S_COLS + wg * (R / 2);
                    float ts = 1.f, ls = 0.f;   // the token's scale and its log2
                    const int pos = (w.t + t) * TOK + tok;
                    const uint32_t bads = c.bad[slot];
                    const bool seen = pos < w.len && !(bads >> (tok >> min(a.cache.page_shift, 6)) & 1u);
                    if constexpr (E4M3) {
                        uint32_t hi[HH], lo[HH], pe[HH];
                        tmem_ld8_x2_nw<HH>(s_at, hi);
                        tmem_ld8_x2_nw<HH>(s_at + R, lo);
                        tmem_ld8_x2_nw<HH>(s_at + SH::NQ, pe);
                        if (seen) {
                            ts = c.scale[slot][tok];
                            ls = __log2f(ts);
                        }
                        tmem_ld_wait();
                        after_ld_wait(hi);
                        after_ld_wait(lo);
                        after_ld_wait(pe);
                        const float4* qs = reinterpret_cast<const float4*>(c.qscale + h0);
#pragma unroll
                        for (int i = 0; i < HH; i += 4) {
                            const float4 q4 = qs[i / 4];
                            const float q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                x[i + j] = sl2 * fmaf(fmaf(0.0625f, __uint_as_float(lo[i + j]), __uint_as_float(hi[i + j])) * ts,
                                                      q[j], __uint_as_float(pe[i + j]));
                        }
                    } else {
                        uint32_t raw[HH];
                        if constexpr (R == 32) tmem_ld8_x2_nw<HH>(s_at, raw);
                        else tmem_ld16_x2_nw<HH>(s_at, raw);
                        tmem_ld_wait();
                        after_ld_wait(raw);
#pragma unroll
                        for (int i = 0; i < HH; ++i) x[i] = sl2 * __uint_as_float(raw[i]);
                    }
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.s_empty[g & 1]);
                    const bool edge = (w.t + t + 1) * TOK > w.len - (a.S - 1) || bads != 0u;
                    if (edge) {
                        int ends = w.len - (a.S - 1) + new0, head = head0;  // what row i sees ends there
#pragma unroll
                        for (int i = 0; i < HH; ++i) {
                            if (!seen || pos >= ends) x[i] = -INFINITY;
                            if (++head == a.H) {
                                head = 0;
                                ++ends;
                            }
                        }
                        // rows of the tile that no query sees hold whatever lay there: zero them, so that their
                        // weight of 0 meets no NaN in the second product (the first one is done with them)
                        if (!seen && half == 0) {
#pragma unroll 1
                            for (int k = wg; k < SH::BLOCKS; k += 2) {
                                unsigned char* at = smem + (g * SH::NP + k / 4) % SH::PIECES * SH::PIECE + (tok >> 3) * SH::GROUP + k % 4 * SH::ATOM;
#pragma unroll
                                for (int j = 0; j < 8; ++j)  // neighbouring tokens' stores in different banks
                                    *reinterpret_cast<uint4*>(at + (tok & 7) * 128 + ((j + lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
                            }
                        }
                    }
                    // Does some score exceed its row's reference by too much?  Seldom; only then are the tile's maxima
                    // needed at all (e4m3: of x + log2 s).
                    bool over = false;
#pragma unroll
                    for (int i = 0; i < HH; ++i) over = over || x[i] + ls > m[i] + kOver;
                    // (A failed wait takes the same way, to the barrier at which all four warps stop.)  e4m3: the vote is also the
                    // barrier of a look's sums.
                    const bool look = E4M3 && t > 0 && (t % kWindow == 0 || t == 3);
                    if constexpr (E4M3) {
                        if (look) {
                            reduce16<HH, false>(e, lane);
                            c.mass[sub][h0 + (lane & 15) * HH / 16] = e[0];
                        }
                    }
                    bool move = group_sync_or(bar, 128, over || !ok);
                    [[maybe_unused]] uint32_t fall[2] = {0u, 0u};  // e4m3, a byte per row: by how much its reference falls
                    if constexpr (E4M3) {
                        static_assert(HH == 8 && kWindow == 8, "rows in `fall`, exponents below");
                        if (look) {  // tiles 1 and 2: below 2, to 4 .. 8; kWindow tiles: below 8, to 16 .. 32
                            const int most = 127 + (t == 3 ? 2 : 4);
#pragma unroll
                            for (int i = 0; i < HH; i += 4) {
                                float4 r[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) r[k] = *reinterpret_cast<const float4*>(&c.mass[k][h0 + i]);
                                const float mass[4] = {(r[0].x + r[1].x) + (r[2].x + r[3].x), (r[0].y + r[1].y) + (r[2].y + r[3].y),
                                                       (r[0].z + r[1].z) + (r[2].z + r[3].z), (r[0].w + r[1].w) + (r[2].w + r[3].w)};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int by = most - static_cast<int>(__float_as_uint(mass[k]) >> 23);
                                    if (by > 1) fall[i / 4] |= static_cast<uint32_t>(by) << (8 * k);
                                }
                            }
                            move = __any_sync(0xffffffffu, (fall[0] | fall[1]) != 0u) || move;  // the same in all four warps
                        }
                        if (look || t == 1) {
#pragma unroll
                            for (int i = 0; i < HH; ++i) e[i] = 0.f;
                        }
                    }
                    if (move) {
                        float v[HH];
#pragma unroll
                        for (int i = 0; i < HH; ++i) v[i] = x[i] + ls;
                        reduce16<HH, true>(v, lane);
#pragma unroll
                        for (int i = 0; i < (HH + 15) / 16; ++i) c.red[sub][h0 + (lane & 15) * HH / 16 + i] = v[i];
                        stop = group_sync_or(bar, 128, !ok);
                        if (stop) break;
#pragma unroll
                        for (int i = 0; i < HH; i += 4) {
                            float to[4] = {m[i], m[i + 1], m[i + 2], m[i + 3]};
                            if constexpr (E4M3) {
                                const float4 low = *reinterpret_cast<const float4*>(c.lowest + h0 + i);
                                const float least[4] = {low.x, low.y, low.z, low.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k)  // (a row that has seen nothing has both at -infinity)
                                    if (to[k] > least[k]) to[k] = fmaxf(to[k] - static_cast<float>(fall[i / 4] >> (8 * k) & 255u), least[k]);
                            }
                            float4 r[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) r[k] = *reinterpret_cast<const float4*>(&c.red[k][h0 + i]);
                            const float top[4] = {fmaxf(fmaxf(r[0].x, r[1].x), fmaxf(r[2].x, r[3].x)),
                                                  fmaxf(fmaxf(r[0].y, r[1].y), fmaxf(r[2].y, r[3].y)),
                                                  fmaxf(fmaxf(r[0].z, r[1].z), fmaxf(r[2].z, r[3].z)),
                                                  fmaxf(fmaxf(r[0].w, r[1].w), fmaxf(r[2].w, r[3].w))};
                            float f[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if (top[k] > to[k] + kOver) to[k] = top[k] - kBelow;
                                f[k] = 1.f;
                                if (to[k] != m[i + k]) {
                                    f[k] = ex2(m[i + k] - to[k]);
                                    m[i + k] = to[k];
                                    l[i + k] *= f[k];
                                    if constexpr (E4M3) e[i + k] *= f[k];
                                }
                            }
                            if (writer)
                                *reinterpret_cast<float4*>(c.factor + h0 + i) = make_float4(f[0], f[1], f[2], f[3]);
                        }
                        group_sync(bar, 128);
                        if (E4M3 && writer)  // read only before that barrier
#pragma unroll
                            for (int i = 0; i < HH; ++i) c.lowest[h0 + i] = fmaxf(c.lowest[h0 + i], m[i] - kFall);
                        if (t > 0) {
                            // the accumulated output moves too: the last product must be done with it
                            ok = ok && wait(&c.pv_done, (g - 1) & 1);
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int k = 0; k < 4 * SH::NQ / R; ++k) {  // chunk and part: this group's half of the rows
                                float o[R / 2];
                                const uint32_t at = tmem + lane_base + SH::COL_O + k * R + wg * (R / 2);
                                if constexpr (R == 32) tmem_ld16(at, o);
                                else tmem_ld32(at, o);
                                const float4* f = reinterpret_cast<const float4*>(c.factor + wg * (R / 2));
#pragma unroll
                                for (int i = 0; i < R / 8; ++i) {
                                    const float4 q = f[i];
                                    o[4 * i] *= q.x; o[4 * i + 1] *= q.y; o[4 * i + 2] *= q.z; o[4 * i + 3] *= q.w;
                                }
                                if constexpr (R == 32) tmem_st16(at, o);
                                else tmem_st32(at, o);
                            }
                            tmem_st_wait();
                        }
                    }
                    // weights, one row of all columns per token (the second product's MN-major B operand): this thread
                    // has HH neighbouring columns of its token, of each part
#pragma unroll
                    for (int i = 0; i < HH; ++i) {
                        x[i] = ex2(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
                        l[i] += x[i];
                        if constexpr (E4M3) e[i] = fmaf(x[i], ts, e[i]);
                    }
                    uint32_t pk[HH / 2];  // bf16: pairs of columns; e4m3: pairs of the high parts, then of the low ones
                    if constexpr (E4M3) {
#pragma unroll
                        for (int i = 0; i < HH / 4; ++i) {
                            uint32_t h[2], lo[2];
#pragma unroll
                            for (int j = 0; j < 2; ++j) split_e4m3(x[4 * i + 2 * j] * ts, x[4 * i + 2 * j + 1] * ts, h[j], lo[j]);
                            pk[i] = h[0] | h[1] << 16;
                            pk[HH / 4 + i] = lo[0] | lo[1] << 16;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < HH / 2; ++i) pk[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
                    }
                    // they overwrite the last tile's: that product must be done
                    if (g > 0) ok = ok && wait(&c.pv_done, (g - 1) & 1);
                    if constexpr (E4M3) {
                        *reinterpret_cast<uint2*>(p_tile + sw64_byte(tok, h0)) = make_uint2(pk[0], pk[1]);
                        *reinterpret_cast<uint2*>(p_tile + sw64_byte(tok, R + h0)) = make_uint2(pk[2], pk[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < HH / 8; ++i)
                            *reinterpret_cast<uint4*>(p_tile + (SH::PROW == 128 ? sw128_byte(tok, h0 * 2 + i * 16)
                                                                               : sw64_byte(tok, h0 * 2 + i * 16))) =
                                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                    }
                    fence_async_smem();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.p_full);
                }
                if (stop) break;

                // ---- the segment's end: sums over its tokens, then the output from tensor memory
                const Walk<SH::LEAD> seg_w = w;
                const bool more = w.next(a);
                if (E4M3 && more) load_queries(w.b);  // while the last product runs
                reduce16<HH, false>(l, lane);
#pragma unroll
                for (int i = 0; i < (HH + 15) / 16; ++i) c.red[sub][h0 + (lane & 15) * HH / 16 + i] = l[i];
                ok = ok && wait(&c.pv_done, (g - 1) & 1);
                tc_fence_after_sync();
                if (writer) {
#pragma unroll
                    for (int i = 0; i < HH; ++i) c.factor[h0 + i] = m[i];
                }
                stop = group_sync_or(bar, 128, !ok);
                if (stop) break;
                const bool whole = seg_w.n == seg_w.nt;
                const Part part = part_of(a.workspace, gridDim.x, R);
                const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg_w.t == 0 ? 1 : 0);
                if ((tid & 127) < R / 2) {
                    const int h = wg * (R / 2) + (tid & 127), r = row0 + h;
                    const float sum = (c.red[0][h] + c.red[1][h]) + (c.red[2][h] + c.red[3][h]), mm = c.factor[h];
                    if (whole) {
                        if (a.lse && r < rows)
                            a.lse[static_cast<int64_t>(seg_w.b) * rows + r] = (mm + log2f(sum)) * 0.6931471805599453f;
                    } else {
                        part.m[slot * R + h] = mm;
                        part.l[slot * R + h] = sum;
                    }
                    c.factor[h] = sum == 0.f ? 0.f : 1.f / sum;
                }
                group_sync(bar, 128);
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {  // 128 channels of this group's rows; thread = channel
                    constexpr int N = R / 2;
                    const int j = wg * N, ch = k * 128 + sub * 32 + lane;
                    const uint32_t at = tmem + lane_base + SH::COL_O + k * SH::NQ + j;
                    uint32_t raw[N];
                    float o[N];
                    if constexpr (N == 16) tmem_ld16_nw(at, raw);
                    else tmem_ld32_nw(at, raw);
                    if constexpr (E4M3) {
                        uint32_t lo[N];
                        tmem_ld16_nw(at + R, lo);
                        tmem_ld_wait();
                        after_ld_wait(raw);
                        after_ld_wait(lo);
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = fmaf(0.0625f, __uint_as_float(lo[i]), __uint_as_float(raw[i]));
                    } else {
                        tmem_ld_wait();
                        after_ld_wait(raw);
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = __uint_as_float(raw[i]);
                    }
                    if (whole) {
                        const float4* f = reinterpret_cast<const float4*>(c.factor + j);
#pragma unroll
                        for (int i = 0; i < N / 4; ++i) {
                            const float4 q = f[i];
                            o[4 * i] *= q.x; o[4 * i + 1] *= q.y; o[4 * i + 2] *= q.z; o[4 * i + 3] *= q.w;
                        }
                        const int have = rows - (row0 + j);  // rows of this sequence among the N
                        TO* out = static_cast<TO*>(a.o) + (static_cast<int64_t>(seg_w.b) * rows + row0 + j) * kMlaLatent;
                        if constexpr (sizeof(TO) == 2) {
                            // neighbouring lanes swap halves of their rows, so that a lane stores two channels at once:
                            // an even lane those of the first half of the rows, an odd one of the second
                            const bool odd = lane & 1;
                            out += (odd ? N / 2 * kMlaLatent : 0) + (ch & ~1);
#pragma unroll
                            for (int i = 0; i < N / 2; ++i) {
                                const float got = __shfl_xor_sync(0xffffffffu, odd ? o[i] : o[i + N / 2], 1);
                                const uint32_t v = odd ? pack_bf16(got, o[i + N / 2]) : pack_bf16(o[i], got);
                                if (i + (odd ? N / 2 : 0) < have) *reinterpret_cast<uint32_t*>(out + i * kMlaLatent) = v;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < N; ++i)
                                if (i < have) out[i * kMlaLatent + ch] = o[i];
                        }
                    } else {
                        float* out = part.o + (slot * R + j) * kMlaLatent + ch;
#pragma unroll
                        for (int i = 0; i < N; ++i) out[i * kMlaLatent] = o[i];
                    }
                }
                if (!whole && tid == 0) {  // which groups share this sequence (group k's range begins at total k / groups)
                    const long long x = seg_w.t == 0 ? c.end - seg_w.n : c.first - seg_w.t;  // its first tile's place
                    part.meta[slot] = make_int4(seg_w.b, group_of(x, groups, c.total),
                                                group_of(x + seg_w.nt - 1, groups, c.total), 0);
                }
                tc_fence_before_sync();
                group_sync(bar, 128);  // factor and red are free again
                if (!more) break;
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the partial results of the sequences that the cuts split.  Blocks: (CTA of the main kernel, 128 of the 512
// channels, which of its two results); the n groups that share a sequence share its rows, n apart.  A warp adds up one
// row (a lane has 4 channels); of a sequence cut into more than 32 parts the block adds up one row, its warps taking
// every eighth part.  Every sum has a fixed order.  The time is latency, so loads that do not depend on the
// weights are issued before them.  The grid is launched while the main kernel runs and waits for its end.
constexpr int COMBINE = 256;

template <int R, typename TO>
__global__ void __launch_bounds__(COMBINE) mla_combine_kernel(const __grid_constant__ MlaDecodeArgs a, int row_tiles,
                                                              int ctas) {
    static_assert(GROUPS <= COMBINE, "a thread per part");
    constexpr int WARPS = COMBINE / 32, AHEAD = 4;
    mla::after_previous();
    const Part p = part_of(a.workspace, ctas, R);
    const int4 meta = p.meta[blockIdx.x * 2 + blockIdx.z];  // sequence, first and last group
    if (meta.x < 0) return;
    const int group = blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles, rows = min(a.S * a.H - rt * R, R);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = blockIdx.y * 128 + lane * 4;
    const int n = meta.z - meta.y + 1, first = group - meta.y;
    const int64_t base = (static_cast<int64_t>(meta.y) * row_tiles + rt) * 2 * R;
    auto index = [&](int k, int i) { return base + (static_cast<int64_t>(k) * row_tiles * 2 + (k == 0 ? 1 : 0)) * R + i; };
    auto load = [&](int k, int i) { return __ldcg(reinterpret_cast<const float4*>(p.o + index(k, i) * kMlaLatent + ch)); };
    auto add = [](float4& o, float f, float4 v) {
        o.x = fmaf(f, v.x, o.x); o.y = fmaf(f, v.y, o.y); o.z = fmaf(f, v.z, o.z); o.w = fmaf(f, v.w, o.w);
    };
    auto store = [&](int i, float4 o, float inv, float m, float l) {
        const int64_t row = static_cast<int64_t>(meta.x) * a.S * a.H + rt * R + i;
        TO* out = static_cast<TO*>(a.o) + row * kMlaLatent + ch;
        if constexpr (sizeof(TO) == 2)
            *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        else
            *reinterpret_cast<float4*>(out) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (a.lse && blockIdx.y == 0 && lane == 0) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
    };
    auto warp_max = [](float v) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    };
    auto warp_sum = [](float v) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    };
    if (n <= 32) {
        for (int i = first + warp * n; i < rows; i += WARPS * n) {
            const float mk = lane < n ? p.m[index(lane, i)] : -INFINITY, lk = lane < n ? p.l[index(lane, i)] : 0.f;
            float4 v[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) v[k] = k < n ? load(k, i) : make_float4(0.f, 0.f, 0.f, 0.f);
            const float m = warp_max(mk), f = mk == -INFINITY ? 0.f : ex2(mk - m), l = warp_sum(f * lk);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k) add(o, __shfl_sync(0xffffffffu, f, k), v[k]);
#pragma unroll 4
            for (int k = AHEAD; k < n; ++k) add(o, __shfl_sync(0xffffffffu, f, k), load(k, i));
            store(i, o, l == 0.f ? 0.f : 1.f / l, m, l);
        }
        return;
    }
    __shared__ float wgt[GROUPS], red[2][WARPS];
    __shared__ float4 acc[WARPS][32];
    for (int i = first; i < rows; i += n) {
        const int k0 = threadIdx.x;  // this thread's part, for the weights
        const float mk = k0 < n ? p.m[index(k0, i)] : -INFINITY, lk = k0 < n ? p.l[index(k0, i)] : 0.f;
        float4 v[AHEAD];  // n > 32 = AHEAD * WARPS
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) v[k] = load(warp + k * WARPS, i);
        float m = warp_max(mk);
        if (lane == 0) red[0][warp] = m;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < WARPS; ++k) m = fmaxf(m, red[0][k]);
        const float f = mk == -INFINITY ? 0.f : ex2(mk - m);
        if (k0 < n) wgt[k0] = f;
        float l = warp_sum(f * lk);
        if (lane == 0) red[1][warp] = l;
        __syncthreads();
        l = 0.f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) l += red[1][k];
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) add(o, wgt[warp + k * WARPS], v[k]);
#pragma unroll 8
        for (int k = warp + AHEAD * WARPS; k < n; k += WARPS) add(o, wgt[k], load(k, i));
        acc[warp][lane] = o;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int k = 1; k < WARPS; ++k) add(o, 1.f, acc[k][lane]);
            store(i, o, l == 0.f ? 0.f : 1.f / l, m, l);
        }
        __syncthreads();
    }
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

// Cached latents [pool rows, blocks of 128 bytes] as {128 bytes, 8 rows, blocks, pool rows / 8}: one box is four blocks of
// box_rows tokens, 8 tokens after another.
bool encode_latent(CUtensorMap* m, const void* base, int esize, int64_t pool_rows, int blocks, int box_rows) {
    const cuuint64_t inner = static_cast<cuuint64_t>(128 / esize), row = static_cast<cuuint64_t>(blocks) * 128;
    const cuuint64_t dims[4] = {inner, 8, static_cast<cuuint64_t>(blocks), static_cast<cuuint64_t>(pool_rows / 8)};
    const cuuint64_t strides[3] = {row, 128, row * 8};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), 8, 4, static_cast<cuuint32_t>(box_rows / 8)};
    return encode(m, base, esize == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims,
                  strides, box);
}

// Cached positional keys [pool rows, 64] as {64, pool rows, 1}.
bool encode_pe(CUtensorMap* m, const void* base, int64_t pool_rows, int box_rows) {
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(pool_rows), 1}, strides[2] = {128, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    return encode(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, strides, box);
}

template <int R, bool E4M3, typename TO>
cudaError_t launch(const MlaDecodeArgs& a, const Grid& g) {
    using SH = Shape<R, E4M3>;
    constexpr int smem = kSmemBytes<R, E4M3>;
    auto kernel = mla_decode_kernel<R, E4M3, TO>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kernel, smem, allowed);
    if (err != cudaSuccess) return err;
    CUtensorMap q, qp, kv, pe;
    const int rows = a.S * a.H, box = a.cache.page_size < TOK ? a.cache.page_size : TOK;
    // a cache without pages is never loaded from (every page number is out of range): any valid map serves
    const bool none = a.cache.num_pages == 0;
    const int64_t pool = none ? 8 : a.cache.num_pages * a.cache.page_size;
    const void* latent = none ? a.q_latent : a.cache.latent;
    const void* cpe = none ? a.q_pe : a.cache.pe;
    if (!encode_q(&q, a.q_latent, kMlaLatent, rows, a.B, R) || !encode_q(&qp, a.q_pe, kMlaPe, rows, a.B, R) ||
        !encode_latent(&kv, latent, E4M3 ? 1 : 2, pool, SH::BLOCKS, box) ||
        !encode_pe(&pe, cpe, pool, box))
        return cudaErrorInvalidValue;
    const int ctas = g.groups * g.row_tiles;
    err = launch_early(kernel, dim3(ctas), dim3(THREADS), smem, a.stream, q, qp, kv, pe, a, g.row_tiles, g.groups);
    if (err != cudaSuccess || !a.workspace) return err;
    return launch_early(mla_combine_kernel<R, TO>, dim3(ctas, kMlaLatent / 128, 2), dim3(COMBINE), 0, a.stream, a,
                        g.row_tiles, ctas);
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
