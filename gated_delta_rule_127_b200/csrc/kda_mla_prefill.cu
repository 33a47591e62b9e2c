// kda_mla_prefill.cu -- expanded latent attention over a packed batch, on the tensor cores.
//
// A CTA has 256 queries of one head, as two sides of 128, and walks the sequence's keys in tiles of 128:
//
//     S = Q_nope K^T + Q_pe P^T        [128, 128], 192 channels     (P: positional keys, one copy for all heads)
//     W = 2^(scale log2(e) S - m),  l += sum W                      (m: running reference per row)
//     O += W V                         [128, 128]
//
// The sides take turns on the tensor core: while one side's scores become weights (four warps, thread = row, its 128
// scores in registers), the other side's products run.  Scores and outputs of both sides fill the 512 columns of
// tensor memory; the weights are written over the scores they come from, in bf16, and are the second product's A
// operand there.  Per tile and side the tensor core needs 1,280 cycles (128 x 128 x (192 + 128) products at 4,096 a
// cycle), the exponentials 1,024 cycles of the special-function units, so the two are meant to overlap.
//
// The reference moves only when a row's maximum exceeds it by 8 in log2 units; then the warp's 32 rows of O and l
// are multiplied by 2^(old - new).  Until then weights above 1 are as exact as any.
//
// Keys and values come through a ring of eight 16 KB pieces (64 channels of 128 keys; 128 channels of 64 values): a tile
// is three pieces of keys and two of values, and a piece is free as soon as both sides have used it.
//
// A thread per side issues its products, in turns: O += W V of a tile and the scores of the next one, then the other
// thread the same for its side.  Without turns the sides' products mix on the tensor core, both sides' scores come
// late and together, and the sides fall into step (6,180 cycles a tile).  A look at a barrier costs 250 cycles while the
// softmax warps keep the special-function units' queue full, and the tensor core idles meanwhile; so a step looks at two:
// `go` for half of its weights, this tile's values and the other side's turn, `p_full` for the other half and the next
// tile's keys.  A warp of its own reports the loads there (4,100 cycles with a look at each barrier).
//
// Roles of the 12 warps: 0-3 and 4-7 the sides' softmax and output, 8 loads (TMA), 9 and 10 issue the sides' products, 11
// reports the loads' arrival.  Registers: 384 threads at 168 when launched, of which the last four warps give up 96 each so that the softmax
// warps have 216 (a row's 128 scores): 256 x 216 + 128 x 72 = 384 x 168.
#include <algorithm>

#include "kda_mla_common.cuh"
#include "kda_mla_sm100.cuh"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace sm100;

constexpr int ROWS = 128;              // queries per side, keys per tile
constexpr int THREADS = 384;
constexpr int PIECE = 16384, PIECES = 8, PER_TILE = 5;
constexpr int OFF_RING = 2 * 3 * PIECE;                   // after both sides' queries (three blocks of 64 channels each)
constexpr int OFF_CTL = OFF_RING + PIECES * PIECE;
constexpr uint32_t COL_S = 0, COL_O = 256;                // tensor memory: per side 128 columns of each

struct Ctl {
    uint64_t k_full[2], v_full[2], empty[PIECES], q_full[2], s_full[2], go[2], p_full[2], o_full[2], drain_bar[2];
    uint32_t tmem, abort_word;
    long long scan[THREADS / 32];
    int b, pair;                       // this CTA's sequence (-1: none) and pair of query tiles
};
constexpr int SMEM_BYTES = OFF_CTL + static_cast<int>(sizeof(Ctl));
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}

template <typename TO>
__global__ void __launch_bounds__(THREADS, 1)
mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pe,
                   const __grid_constant__ MlaPrefillArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl& c = *reinterpret_cast<Ctl*>(smem + OFF_CTL);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, head = blockIdx.y;

    // ---- which 256 queries: pairs of query tiles are numbered over the sequences, the last pair of each (which sees the
    // most keys) first
    {
        const int per = (a.B + THREADS - 1) / THREADS, lo = min(tid * per, a.B), hi = min(lo + per, a.B);
        const auto pairs = [&](int b) {
            int64_t first;
            return (mla::seq_rows(a.cu_q, a.Tq, a.B, b, first, a.flags) + 2 * ROWS - 1) / (2 * ROWS);
        };
        long long mine = 0;
        for (int b = lo; b < hi; ++b) mine += pairs(b);
        long long upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, upto, d);
            if (lane >= d) upto += v;
        }
        if (lane == 31) c.scan[warp] = upto;
        if (tid == 0) {
            c.abort_word = 0u;
            c.b = -1;
            for (int i = 0; i < PIECES; ++i) mbar_init(&c.empty[i], 2);
            for (int i = 0; i < 2; ++i) {
                mbar_init(&c.q_full[i], 1);
                mbar_init(&c.s_full[i], 1);
                mbar_init(&c.go[i], 6);
                mbar_init(&c.p_full[i], 5);
                mbar_init(&c.o_full[i], 1);
                mbar_init(&c.k_full[i], 1);
                mbar_init(&c.v_full[i], 1);
                mbar_init(&c.drain_bar[i], 1);
            }
            fence_mbar_init();
        }
        if (warp == 9) tmem_alloc(&c.tmem, 512);
        if (warp == 8 && lane < 4) tma_prefetch_desc(lane == 0 ? &tm_q : lane == 1 ? &tm_k : lane == 2 ? &tm_v : &tm_pe);
        __syncthreads();
        for (int w = 0; w < warp; ++w) upto += c.scan[w];
        long long at = upto - mine;
        if (at <= blockIdx.x && blockIdx.x < upto) {
            int b = lo;
            while (blockIdx.x >= at + pairs(b)) at += pairs(b++);
            c.b = b;
            c.pair = pairs(b) - 1 - static_cast<int>(blockIdx.x - at);
        }
        tc_fence_before_sync();
        __syncthreads();
        tc_fence_after_sync();
    }
    const uint32_t tmem = c.tmem;
    const RoleWait wait{a.wait_polls, &c.abort_word, a.flags};

    if (c.b >= 0) {
        int64_t q0, k0;
        const int nq = mla::seq_rows(a.cu_q, a.Tq, a.B, c.b, q0, a.flags);
        const int nk = mla::seq_rows(a.cu_k, a.Tk, a.B, c.b, k0, a.flags);
        const int i0 = c.pair * 2 * ROWS;
        // keys that the last query of a side sees, and tiles of them
        const auto tiles = [&](int side) {
            const int first = i0 + side * ROWS, last = min(first + ROWS, nq) - 1;
            if (first >= nq) return 0;
            const int see = a.causal ? min(max(last + 1 + nk - nq, 0), nk) : nk;
            return (see + ROWS - 1) / ROWS;
        };
        const int n0 = tiles(0), n1 = tiles(1), most = max(n0, n1);

        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            // ---------------------------------------------------------------- softmax and output of one side
            const int s = warp >> 2, n = s == 0 ? n0 : n1;
            const int i = i0 + s * ROWS + (warp & 3) * 32 + lane;  // this thread's query
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t at_s = tmem + lanes + COL_S + s * 128, at_o = tmem + lanes + COL_O + s * 128;
            // the last key that the query sees, and a scale that is never 0 or negative (scores are negated instead)
            const int see = i < nq ? (a.causal ? min(i + nk - nq, nk - 1) : nk - 1) : -1;
            const int warp_see = __reduce_min_sync(0xffffffffu, see);  // by the warp's query that sees least
            const float sl2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
            const bool negate = a.scale < 0.f;
            float m = -INFINITY, l = 0.f;
            // the tile that the sequence ends in, if any (then it is the side's last): all four warps meet there, once,
            // also those whose waits have failed
            const int ending = n * ROWS > nk ? n - 1 : -1;
            bool ok = true, met = ending < 0;
            for (int j = 0; j < n; ++j) {
                ok = wait(&c.s_full[s], j & 1);
                if (!ok) break;
                tc_fence_after_sync();
                uint32_t raw[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld32_nw(at_s + k * 32, raw[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 4; ++k) after_ld_wait(raw[k]);
                float x[ROWS];
#pragma unroll
                for (int k = 0; k < ROWS; ++k) x[k] = __uint_as_float(raw[k >> 5][k & 31]);
                if (negate) {
#pragma unroll
                    for (int k = 0; k < ROWS; ++k) x[k] = -x[k];
                }
                const bool edge = j * ROWS + ROWS - 1 > warp_see;  // some query of the warp does not see the whole tile
                if (edge) {
                    const int left = see - j * ROWS;   // the last column this one sees
#pragma unroll
                    for (int k = 0; k < ROWS; ++k)
                        if (k > left) x[k] = -INFINITY;
                }
                if (j == ending) {
                    // rows of V past the sequence's end hold whatever lies there: zero them, so that their weight of 0
                    // meets no NaN (both sides do, each before its own product)
                    const uint32_t g = j * PER_TILE + 3;
                    ok = wait(&c.v_full[j & 1], (j >> 1) & 1);
                    const int r = (warp & 3) * 32 + lane;  // a key of the tile
                    if (ok && r >= nk - j * ROWS) {
                        unsigned char* v = smem + OFF_RING + ((g + (r >> 6)) % PIECES) * PIECE + (r & 63) * 128;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            *reinterpret_cast<uint4*>(v + (k >> 3) * (PIECE / 2) + (k & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    ok = !group_sync_or(1 + s, 128, !ok);  // zeroed before any warp's weights are announced
                    met = true;
                    if (!ok) break;
                }
                float t[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
                for (int k = 4; k < ROWS; ++k) t[k & 3] = fmaxf(t[k & 3], x[k]);
                const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * sl2;
                const bool move = top > m + 8.f;
                if (__any_sync(0xffffffffu, move)) {
                    float f = 1.f;
                    if (move) {
                        f = ex2(m - top);
                        m = top;
                        l *= f;
                    }
                    if (j > 0) {  // the last second product is done: it was issued before this tile's scores
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            float o[32];
                            tmem_ld32(at_o + k * 32, o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= f;
                            tmem_st32(at_o + k * 32, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float u = ex2(fmaf(x[k * 32 + e], sl2, -ref)), v = ex2(fmaf(x[k * 32 + e + 1], sl2, -ref));
                        sum[e & 2] += u;
                        sum[(e & 2) + 1] += v;
                        w[e / 2] = pack_bf16(u, v);
                    }
                    if (k == 3) tmem_st16_nw(at_s + k * 16, w);
                    if (k >= 2) {  // the first half is announced when the third quarter has been computed: its stores have landed
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(k == 2 ? &c.go[s] : &c.p_full[s]);
                    }
                    if (k < 3) tmem_st16_nw(at_s + k * 16, w);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            if (!met) group_sync_or(1 + s, 128, true);
            if (n > 0 && ok) ok = wait(&c.o_full[s], 0);
            if (ok && i0 + s * ROWS < nq) {
                tc_fence_after_sync();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int64_t row = (q0 + i) * a.H + head;
                TO* out = static_cast<TO*>(a.o) + row * kMlaV;
#pragma unroll 1
                for (int k = 0; k < 4; ++k) {
                    float o[32];
                    if (n > 0) {
                        tmem_ld32(at_o + k * 32, o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                    if (i < nq) {
                        if constexpr (sizeof(TO) == 2) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                reinterpret_cast<uint4*>(out + k * 32)[e] =
                                    make_uint4(pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                               pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv), pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                reinterpret_cast<float4*>(out + k * 32)[e] =
                                    make_float4(o[4 * e] * inv, o[4 * e + 1] * inv, o[4 * e + 2] * inv, o[4 * e + 3] * inv);
                        }
                    }
                }
                if (a.lse && i < nq) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
            }
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            if (warp == 8) {
                // ---------------------------------------------------------------- loads
                uint32_t g = 0;
                bool ok = true;
                if (most > 0 && elect_one()) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if ((s == 0 ? n0 : n1) == 0) continue;
                        mbar_arrive_expect_tx(&c.q_full[s], 3 * PIECE);
#pragma unroll
                        for (int k = 0; k < 3; ++k)
                            tma_load_3d(smem + (s * 3 + k) * PIECE, &tm_q, k * 64, head, static_cast<int>(q0) + i0 + s * ROWS,
                                        &c.q_full[s]);
                    }
                }
                __syncwarp();
                for (int j = 0; j < most && ok; ++j) {
                    const int row = static_cast<int>(k0) + j * ROWS;
                    uint64_t *kb = &c.k_full[j & 1], *vb = &c.v_full[j & 1];
#pragma unroll
                    for (int k = 0; k < PER_TILE; ++k) {
                        const uint32_t slot = g % PIECES;
                        ok = wait(&c.empty[slot], ((g / PIECES) & 1) ^ 1);
                        if (!ok) break;
                        if (elect_one()) {
                            unsigned char* dst = smem + OFF_RING + slot * PIECE;
                            if (k == 0) mbar_arrive_expect_tx(kb, 3 * PIECE);
                            if (k == 3) mbar_arrive_expect_tx(vb, 2 * PIECE);
                            if (k < 2) {
                                tma_load_3d(dst, &tm_k, k * 64, head, row, kb);
                            } else if (k == 2) {
                                tma_load_3d(dst, &tm_pe, 0, 0, row, kb);
                            } else {
                                tma_load_3d(dst, &tm_v, kMlaNope, head, row + (k - 3) * 64, vb);
                                tma_load_3d(dst + PIECE / 2, &tm_v, kMlaNope + 64, head, row + (k - 3) * 64, vb);
                            }
                        }
                        __syncwarp();
                        ++g;
                    }
                }
                if (!ok) {
                    // let what is in flight land before the block ends; first what a begun group of pieces still lacks, or its
                    // barrier would never complete
                    const int j = g / PER_TILE, k = g % PER_TILE;
                    if (k != 0 && k != 3 && elect_one()) {
                        const int row = static_cast<int>(k0) + j * ROWS;
                        for (int i = k; i < (k < 3 ? 3 : 5); ++i) {
                            uint64_t* b = k < 3 ? &c.k_full[j & 1] : &c.v_full[j & 1];
                            unsigned char* dst = smem + OFF_RING + (g - k + i) % PIECES * PIECE;
                            tma_load_3d(dst, &tm_pe, 0, 0, row, b);  // any piece of this size: nobody reads it
                        }
                    }
                    __syncwarp();
                    const int last_k = j - (k > 0 ? 0 : 1), last_v = j - (k > 3 ? 0 : 1);  // last tiles begun
                    for (int i = max(last_k - 1, 0); i <= last_k; ++i) drain(&c.k_full[i & 1], (i >> 1) & 1);
                    for (int i = max(last_v - 1, 0); i <= last_v; ++i) drain(&c.v_full[i & 1], (i >> 1) & 1);
                    if (n0 > 0) drain(&c.q_full[0], 0);
                    if (n1 > 0) drain(&c.q_full[1], 0);
                }
            } else if (warp == 9 || warp == 10) {
                // ---------------------------------------------------------------- products of one side
                const int s = warp - 9, n = s == 0 ? n0 : n1;
                const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
                const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
                const uint32_t d_s = tm + COL_S + s * 128, d_o = tm + COL_O + s * 128;
                const uint64_t q = sw128_desc(base + s * 3 * PIECE, 16, 1024);
                constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false), idesc_o = idesc_bf16(128, 128, false, true);
                if (elect_one()) {
                    const auto scores = [&](uint32_t g) {
                        tc_fence_after_sync();
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const uint64_t kd = sw128_desc(base + OFF_RING + (g + k) % PIECES * PIECE, 16, 1024);
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                mma_f16(d_s, q + ((k * PIECE + i * 32) >> 4), kd + i * 2, idesc_s, k + i > 0);
                        }
                        mma_commit(&c.s_full[s]);
                    };
                    const auto release = [&](uint32_t g, int count) {
                        for (int k = 0; k < count; ++k) mma_commit(&c.empty[(g + k) % PIECES]);
                    };
                    bool ok = n == 0 || (wait.alone(&c.q_full[s], 0) && wait.alone(&c.k_full[0], 0));
                    if (ok && n > 0) {
                        scores(0);
                        release(0, 3);
                    }
                    uint32_t g = 0;
                    for (int j = 0; j < n && ok; ++j, g += PER_TILE) {
                        if (s == 0 ? j == 0 || j > n1 : j >= n0) mbar_arrive(&c.go[s]);  // no other side to wait for
                        ok = wait.alone(&c.go[s], j & 1);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (k == 1) ok = ok && wait.alone(&c.p_full[s], j & 1);
                            if (!ok) break;
                            tc_fence_after_sync();
                            const uint64_t vd = sw128_desc(base + OFF_RING + (g + 3 + k) % PIECES * PIECE, PIECE / 2, 1024);
#pragma unroll
                            for (int i = 0; i < 4; ++i)  // 16 keys of 2 x 64 channels
                                mma_f16_ts(d_o, d_s + k * 32 + i * 8, vd + ((i * 2048) >> 4), idesc_o, j > 0 || k + i > 0);
                            release(g + 3 + k, 1);  // before the scores: what a commit reports is all that came before it
                        }
                        if (!ok) break;
                        if (j + 1 < n) scores(g + PER_TILE);
                        if (s == 0 ? j < n1 : j + 1 < n0) mbar_arrive(&c.go[s ^ 1]);  // the other side's turn
                        if (j + 1 < n) release(g + PER_TILE, 3);
                        else mma_commit(&c.o_full[s]);
                    }
                    for (int j = n; j < most && ok; ++j, g += PER_TILE) {  // keys that only the other side sees
                        ok = wait.alone(&c.k_full[j & 1], (j >> 1) & 1);
                        for (int k = 0; k < 3 && ok; ++k) mbar_arrive(&c.empty[(g + k) % PIECES]);
                        ok = ok && wait.alone(&c.v_full[j & 1], (j >> 1) & 1);
                        for (int k = 3; k < PER_TILE && ok; ++k) mbar_arrive(&c.empty[(g + k) % PIECES]);
                    }
                    if (!ok) {  // let issued products finish before the block ends
                        mma_commit(&c.drain_bar[s]);
                        drain(&c.drain_bar[s], 0);
                    }
                }
                __syncwarp();
            } else {
                // ---------------------------------------------------------------- arrivals: tells the sides' steps of them
                if (elect_one()) {
                    bool ok = true;
                    for (int j = 0; j < most && ok; ++j) {
                        ok = wait.alone(&c.v_full[j & 1], (j >> 1) & 1);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {  // one step at a time, here and below
                            if (j >= (s == 0 ? n0 : n1)) continue;
                            ok = ok && (j == 0 || wait.alone(&c.go[s], (j - 1) & 1));
                            if (ok) mbar_arrive(&c.go[s]);
                        }
                        if (j + 1 < most) ok = ok && wait.alone(&c.k_full[(j + 1) & 1], ((j + 1) >> 1) & 1);
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (j >= (s == 0 ? n0 : n1)) continue;
                            ok = ok && (j == 0 || wait.alone(&c.p_full[s], (j - 1) & 1));
                            if (ok) mbar_arrive(&c.p_full[s]);
                        }
                    }
                }
                __syncwarp();
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

template <typename TO>
cudaError_t launch(const MlaPrefillArgs& a) {
    auto kernel = mla_prefill_kernel<TO>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t err = allow_shared(kernel, SMEM_BYTES, allowed);
    if (err != cudaSuccess) return err;
    // without keys nothing is loaded: any valid maps serve
    const bool none = a.Tk == 0;
    const void* kv = none ? a.q : a.kv;
    const void* pe = none ? a.q : a.k_pe;
    const uint64_t tk = none ? 1 : static_cast<uint64_t>(a.Tk), kw = none ? kMlaQk : kMlaKv;
    CUtensorMap mq, mk, mv, mp;
    const auto enc = [](CUtensorMap* m, const void* base, uint64_t d, uint64_t H, uint64_t T, uint32_t rows) {
        return tma_encode_thd(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d, H, T, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    if (!enc(&mq, a.q, kMlaQk, a.H, a.Tq, ROWS) || !enc(&mk, kv, kw, none ? 1 : a.H, tk, ROWS) ||
        !enc(&mv, kv, kw, none ? 1 : a.H, tk, 64) || !enc(&mp, pe, 64, 1, tk, ROWS))
        return cudaErrorInvalidValue;
    // at most this many pairs of query tiles, wherever the sequences end
    const int64_t pairs = a.cu_q ? a.Tq / (2 * ROWS) + std::min<int64_t>(a.B, a.Tq)
                                 : a.B * ((a.Tq / a.B + 2 * ROWS - 1) / (2 * ROWS));
    kernel<<<dim3(static_cast<unsigned>(pairs), a.H), THREADS, SMEM_BYTES, a.stream>>>(mq, mk, mv, mp, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mla_prefill(const MlaPrefillArgs& a) { return a.o_fp32 ? launch<float>(a) : launch<__nv_bfloat16>(a); }

}  // namespace kda
