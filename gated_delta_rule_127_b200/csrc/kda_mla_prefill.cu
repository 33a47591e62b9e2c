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
// tensor memory; the weights are written over scores that have been read, in bf16, and are the second product's A
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
// late and together, and the sides fall into step (2 to 25% slower, most over long keys).  A look at a barrier costs 250
// cycles while the softmax warps keep the special-function units' queue full, and the tensor core idles meanwhile; so a
// step looks at two: `go` for half of its weights, this tile's values and the other side's turn, `p_full` for the other
// half and the next tile's keys.  A warp of its own reports the loads there.
//
// A CTA takes one item, 256 queries of a head, after another: the loads of the next one begin while the last tiles of
// this one are computed, and its first scores while this one's output is written (about 14,000 cycles of an item that
// would stand alone).  The grid has a block for every item; a running CTA takes over blocks that have not begun yet
// (cluster launch control), which balances them; the blocks' order puts the large items first.
//
// Bound by the tensor core and the power that it draws.  Measured, causal, 32 heads, calls in a row: 8,192 tokens 585 us
// (1,170 TFLOP/s, 71% of what a library's matrix product reaches in a burst, 84% of what it sustains), eight prompts of 63
// to 2,500 tokens 301 us, 2,048 queries over up to 32,048 keys 1,149 us (1,130 TFLOP/s).  A call alone on new inputs and a
// cold L2 takes 642, 362 and 1,207 us.
//
// Roles of the 12 warps: 0-3 and 4-7 the sides' softmax and output, 8 finds the items and loads (TMA), 9 and 10 issue the
// sides' products, 11 reports the loads' arrival.
#include <algorithm>

#include "kda_mla_common.cuh"
#include "kda_mla_sm100.cuh"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace sm100;

constexpr int ROWS = 128;              // queries per side, keys per tile
constexpr int THREADS = 384;
// Steps in which the work is ordered by size.  In turn on the same inputs after a flush of L2: 1, one head after another,
// 629 us for 8,192 tokens, 337 for the eight prompts; 4: 563, 311; 16: 552, 337, as heads' keys and values are shared less.
// The long keys are in one order whatever the steps, all pairs seeing about as many tiles (1,055, 1,055, 1,067 us).
constexpr int LEVELS = 4;
constexpr int PIECE = 16384, PIECES = 8, PER_TILE = 5;
constexpr int OFF_RING = 2 * 3 * PIECE;                   // after both sides' queries (three blocks of 64 channels each)
constexpr int OFF_CTL = OFF_RING + PIECES * PIECE;
constexpr uint32_t COL_S = 0, COL_O = 256;                // tensor memory: per side 128 columns of each

__device__ __forceinline__ int pairs_of(int queries) { return queries / (2 * ROWS) + (queries % (2 * ROWS) > 0); }

struct Item {                          // 256 queries of a head
    int real;                          // 0: there are no more
    int q0, k0, nq, nk;                // first rows and numbers of the sequence's queries and keys
    int i0, head;                      // the first of the queries
    // keys that the last query of a side sees, in tiles
    __device__ __forceinline__ int tiles(int side, bool causal) const {
        const int first = i0 + side * ROWS, last = min(first + ROWS, nq) - 1;
        if (first >= nq) return 0;
        const int see = causal ? min(max(last + 1 + nk - nq, 0), nk) : nk;
        return (see + ROWS - 1) / ROWS;
    }
};
struct Ctl {
    alignas(16) uint4 taken;           // the answer of the launch control
    uint64_t taken_full, item_full[2], item_empty[2];
    uint64_t k_full[2], v_full[2], empty[PIECES], q_full[2], q_empty[2], s_full[2], go[2], p_full[2], zeroed[2], o_full[2],
        o_empty[2], drain_bar[2];
    Item item[2];
    uint32_t tmem, abort_word;
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

// Asks for a block of the grid that has not begun (the answer, 16 bytes, is counted on `bar`), and reads the answer:
// true and its coordinates, or false, after which nothing is asked any more.
__device__ __forceinline__ void ask_for_block(void* answer, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(answer)),
                 "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ bool block_taken(const void* answer, uint32_t& x, uint32_t& y) {
    uint32_t got;
    asm volatile(
        "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 z, w;\n\t"
        "ld.shared.b128 h, [%3];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %2, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, %1, z, w}, h;\n\t}\n"
        : "+r"(x), "+r"(y), "=r"(got)
        : "r"(smem_u32(answer))
        : "memory");
    return got != 0u;
}

template <typename TO>
__global__ void __launch_bounds__(THREADS, 1)
mla_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_pe,
                   const __grid_constant__ MlaPrefillArgs a) {
    extern __shared__ __align__(1024) unsigned char smem[];
    Ctl& c = *reinterpret_cast<Ctl*>(smem + OFF_CTL);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        c.abort_word = 0u;
        mbar_init(&c.taken_full, 1);
        for (int i = 0; i < PIECES; ++i) mbar_init(&c.empty[i], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.item_full[i], 1);
            mbar_init(&c.item_empty[i], 11);  // all warps but the one that loads
            mbar_init(&c.k_full[i], 1);
            mbar_init(&c.v_full[i], 1);
            mbar_init(&c.q_full[i], 1);
            mbar_init(&c.q_empty[i], 1);
            mbar_init(&c.s_full[i], 1);
            mbar_init(&c.go[i], 6);
            mbar_init(&c.p_full[i], 5);
            mbar_init(&c.zeroed[i], 4);
            mbar_init(&c.o_full[i], 1);
            mbar_init(&c.o_empty[i], 4);
            mbar_init(&c.drain_bar[i], 1);
        }
        fence_mbar_init();
    }
    if (warp == 9) tmem_alloc(&c.tmem, 512);
    if (warp == 8 && lane < 4) tma_prefetch_desc(lane == 0 ? &tm_q : lane == 1 ? &tm_k : lane == 2 ? &tm_v : &tm_pe);
    if (blockIdx.x == 0) {
        mla::check_cu(a.cu_q, a.Tq, a.B, a.flags);
        mla::check_cu(a.cu_k, a.Tk, a.B, a.flags);
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = c.tmem;
    const RoleWait wait{a.wait_polls, &c.abort_word, a.flags};

    // Every role counts on across the items: tiles (jt), steps of a side (st), its items with keys (outs).  Phases of a
    // barrier are numbered by these counts.
    if (warp < 8) {
        // -------------------------------------------------------------------- softmax and output of one side
        const int s = warp >> 2;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t at_s = tmem + lanes + COL_S + s * 128, at_o = tmem + lanes + COL_O + s * 128;
        // the scale in log2 units, never 0, so that a hidden score (-infinity) gives a weight of 0; where it is negative the
        // products are formed with -Q
        const float sl2 = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-30f);
        uint32_t it = 0, jt = 0, st = 0, outs = 0, ends = 0;
        bool ok = true;
        while (true) {
            ok = wait(&c.item_full[it & 1], (it >> 1) & 1);
            if (!ok) break;
            const Item w = c.item[it & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.item_empty[it & 1]);
            ++it;
            if (!w.real) break;
            const int n0 = w.tiles(0, a.causal), n1 = w.tiles(1, a.causal), n = s == 0 ? n0 : n1, nk = w.nk;
            const int i = w.i0 + s * ROWS + (warp & 3) * 32 + lane;  // this thread's query
            // the last key that the query sees (one past the sequence's end, never stored, as the last query does)
            const int see = a.causal ? min(i + nk - w.nq, nk - 1) : nk - 1;
            const int warp_see = __reduce_min_sync(0xffffffffu, see);  // by the warp's query that sees least
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < n; ++j, ++st) {
                ok = wait(&c.s_full[s], st & 1);
                if (!ok) break;
                tc_fence_after_sync();
                // The 128 scores in two passes: for the maximum all at once, for the weights in quarters, each read again
                // from tensor memory while the one before is worked on, in a loop that stays one.  (With the weights of
                // all four unrolled from registers the code outgrows the instruction caches: 8% slower.)
                uint32_t xa[32], xb[32];
                if (j * ROWS + ROWS - 1 > warp_see) {  // some query of the warp does not see the whole tile: hide scores
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const int left = see - j * ROWS - k * 32;  // the last column that this query sees
                        tmem_ld32_nw(at_s + k * 32, xa);
                        tmem_ld_wait();
                        after_ld_wait(xa);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (e > left) xa[e] = 0xFF800000u;
                        tmem_st32_nw(at_s + k * 32, xa);
                    }
                    tmem_st_wait();
                }
                float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                {
                    uint32_t rest[3][32];
                    tmem_ld32_nw(at_s, xa);  // stays for the second pass
#pragma unroll
                    for (int k = 0; k < 3; ++k) tmem_ld32_nw(at_s + 32 + k * 32, rest[k]);
                    tmem_ld_wait();
                    after_ld_wait(xa);
#pragma unroll
                    for (int k = 0; k < 3; ++k) after_ld_wait(rest[k]);
#pragma unroll
                    for (int k = 0; k < 32; ++k) t[k & 3] = fmaxf(t[k & 3], __uint_as_float(xa[k]));
#pragma unroll
                    for (int k = 0; k < 96; ++k) t[k & 3] = fmaxf(t[k & 3], __uint_as_float(rest[k >> 5][k & 31]));
                }
                if (j * ROWS + ROWS > nk) {
                    // rows of V past the sequence's end hold whatever lies there: zero them, so that their weight of 0
                    // meets no NaN (both sides do, each before its own product, all four warps before any of them
                    // announces weights)
                    const uint32_t g = (jt + j) * PER_TILE + 3;
                    ok = wait(&c.v_full[(jt + j) & 1], ((jt + j) >> 1) & 1);
                    if (!ok) break;
                    const int r = (warp & 3) * 32 + lane;  // a key of the tile
                    if (r >= nk - j * ROWS) {
                        unsigned char* v = smem + OFF_RING + ((g + (r >> 6)) % PIECES) * PIECE + (r & 63) * 128;
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            *reinterpret_cast<uint4*>(v + (k >> 3) * (PIECE / 2) + (k & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.zeroed[s]);
                    ok = wait(&c.zeroed[s], ends & 1);
                    ++ends;
                    if (!ok) break;
                }
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
                uint32_t w16[16];
                const auto weigh = [&](const uint32_t (&x)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float u = ex2(fmaf(__uint_as_float(x[e]), sl2, -ref)), v = ex2(fmaf(__uint_as_float(x[e + 1]), sl2, -ref));
                        sum[e & 2] += u;
                        sum[(e & 2) + 1] += v;
                        w16[e / 2] = pack_bf16(u, v);
                    }
                };
                const auto announce = [&](uint64_t* bar) {
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar);
                };
                // a quarter's weights go over scores that have been read: columns 16 k .. of quarter k / 2
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    tmem_ld32_nw(at_s + h * 64 + 32, xb);
                    weigh(xa);
                    if (h == 1) announce(&c.go[s]);  // the first half: its stores have long landed
                    tmem_st16_nw(at_s + h * 32, w16);
                    tmem_ld_wait();
                    after_ld_wait(xb);
                    if (h == 0) tmem_ld32_nw(at_s + 64, xa);
                    weigh(xb);
                    tmem_st16_nw(at_s + h * 32 + 16, w16);
                    if (h == 0) {
                        tmem_ld_wait();
                        after_ld_wait(xa);
                    }
                }
                announce(&c.p_full[s]);
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            if (!ok) break;
            if (n > 0) {
                ok = wait(&c.o_full[s], outs & 1);
                if (!ok) break;
                ++outs;
                tc_fence_after_sync();
            }
            if (w.i0 + s * ROWS < w.nq) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const int64_t row = (static_cast<int64_t>(w.q0) + i) * a.H + w.head;
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
                    if (n > 0 && k == 3) {  // read: the next item's first product may overwrite it
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c.o_empty[s]);
                    }
                    if (i < w.nq) {
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
                if (a.lse && i < w.nq) a.lse[row] = (m + log2f(l)) * 0.6931471805599453f;
            }
            jt += max(n0, n1);
        }
    } else {
        if (warp == 8) {
            // ---------------------------------------------------------------- items and loads
            uint32_t it = 0, g = 0, asked = 0, answered = 0, qn[2] = {0, 0};
            uint32_t x = blockIdx.x, unused;
            int row = 0;                    // of the tile being loaded
            // 32 sequences at a time, one to a lane: the first of them, the blocks before theirs, their lengths, the most
            // tiles that one of their queries sees and their number of pairs of query tiles
            int scan_b = 0, nqs = 0, nks = 0, deepest = 0;
            uint32_t scan_at = 0, all = 0;
            bool ok = true, more = true;
            const auto look_at = [&](int b) {
                int64_t first;
                scan_b = b;
                nqs = b + lane < a.B ? mla::seq_rows(a.cu_q, a.Tq, a.B, b + lane, first, a.flags) : 0;
                nks = b + lane < a.B ? mla::seq_rows(a.cu_k, a.Tk, a.B, b + lane, first, a.flags) : 0;
                deepest = __reduce_max_sync(0xffffffffu, (nks + ROWS - 1) / ROWS);
                all = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(pairs_of(nqs)));
            };
            // of this lane's sequence, the pairs that see v tiles or more; they are its last ones
            const auto pairs_with = [&](int v) {
                if (v == 0) return pairs_of(nqs);
                const int64_t keys = static_cast<int64_t>(v - 1) * ROWS;  // more than these
                if (!a.causal) return nks > keys ? pairs_of(nqs) : 0;
                const int64_t t = keys - nks + nqs;  // a pair's end must lie behind query t
                return t >= nqs ? 0 : pairs_of(nqs) - static_cast<int>(max(t, static_cast<int64_t>(0)) / (2 * ROWS));
            };
            look_at(0);
            while (ok) {
                // The blocks are, for 32 sequences at a time, their pairs of query tiles and heads in LEVELS steps by the tiles
                // that a pair sees, most first, so that what is left to the end is short (with one head after another CTAs
                // stood idle for a tenth of 8,192 x 32 heads); in a step a head's pairs follow one another, as they share
                // keys and values.  The grid may have more blocks than there are pairs.
                Item w{};
                while (more && x >= scan_at + all * a.H && scan_b + 32 < a.B) {
                    scan_at += all * a.H;
                    look_at(scan_b + 32);
                }
                const uint32_t in = x - scan_at;
                if (more && in < all * a.H) {
                    const int step = max(1, (deepest + LEVELS - 1) / LEVELS);
                    int v = step * (LEVELS - 1) + 1, later = 0;  // the step's least tiles; the sequence's pairs that see more
                    uint32_t before = 0, upto;                   // pairs of all sequences before it, and with it
                    while (true) {
                        upto = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(pairs_with(v)));
                        if (in < upto * a.H || v == 0) break;
                        before = upto;
                        later = pairs_with(v);
                        v = max(v - step, 0);
                    }
                    const uint32_t n = upto - before, at = (in - before * a.H) % n;  // of n pairs of each head
                    const int p = pairs_with(v) - later;
                    int sum = p;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int u = __shfl_up_sync(0xffffffffu, sum, d);
                        if (lane >= d) sum += u;
                    }
                    const int l = __ffs(__ballot_sync(0xffffffffu, at < static_cast<uint32_t>(sum))) - 1;
                    const int i = pairs_of(nqs) - 1 - later - (static_cast<int>(at) - (sum - p));
                    int64_t first;
                    w.real = 1;
                    w.head = static_cast<int>((in - before * a.H) / n);
                    w.i0 = __shfl_sync(0xffffffffu, i, l) * 2 * ROWS;
                    w.nq = mla::seq_rows(a.cu_q, a.Tq, a.B, scan_b + l, first, a.flags);
                    w.q0 = static_cast<int>(first);
                    w.nk = mla::seq_rows(a.cu_k, a.Tk, a.B, scan_b + l, first, a.flags);
                    w.k0 = static_cast<int>(first);
                }
                if (w.real || !more) {  // told to the other roles: an item, or that there are no more
                    ok = wait(&c.item_empty[it & 1], ((it >> 1) & 1) ^ 1);
                    if (!ok) break;
                    if (!more) w.real = 0;
                    if (lane == 0) {
                        c.item[it & 1] = w;
                        mbar_arrive(&c.item_full[it & 1]);
                    }
                    __syncwarp();
                    ++it;
                }
                if (!more) break;
                if (elect_one()) ask_for_block(&c.taken, &c.taken_full);
                __syncwarp();
                ++asked;
                if (w.real) {
                    const int n0 = w.tiles(0, a.causal), n1 = w.tiles(1, a.causal), most = max(n0, n1);
                    const auto queries = [&](int s) {
                        if (!wait(&c.q_empty[s], (qn[s] & 1) ^ 1)) return false;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&c.q_full[s], 3 * PIECE);
#pragma unroll
                            for (int k = 0; k < 3; ++k)
                                tma_load_3d(smem + (s * 3 + k) * PIECE, &tm_q, k * 64, w.head, w.q0 + w.i0 + s * ROWS, &c.q_full[s]);
                        }
                        __syncwarp();
                        ++qn[s];
                        return true;
                    };
                    if (n0 > 0) ok = queries(0);
                    for (int j = 0; j < most && ok; ++j) {
                        const uint32_t jt = g / PER_TILE;
                        row = w.k0 + j * ROWS;
                        uint64_t *kb = &c.k_full[jt & 1], *vb = &c.v_full[jt & 1];
#pragma unroll 1
                        for (int k = 0; k < PER_TILE; ++k) {
                            const uint32_t slot = g % PIECES;
                            // the second side is half a step behind: its queries come after the first keys
                            if (k == 3 && j == 0 && n1 > 0) ok = queries(1);
                            ok = ok && wait(&c.empty[slot], ((g / PIECES) & 1) ^ 1);
                            if (!ok) break;
                            if (elect_one()) {
                                unsigned char* dst = smem + OFF_RING + slot * PIECE;
                                if (k == 0) mbar_arrive_expect_tx(kb, 3 * PIECE);
                                if (k == 3) mbar_arrive_expect_tx(vb, 2 * PIECE);
                                if (k < 2) {
                                    tma_load_3d(dst, &tm_k, k * 64, w.head, row, kb);
                                } else if (k == 2) {
                                    tma_load_3d(dst, &tm_pe, 0, 0, row, kb);
                                } else {
                                    tma_load_3d(dst, &tm_v, kMlaNope, w.head, row + (k - 3) * 64, vb);
                                    tma_load_3d(dst + PIECE / 2, &tm_v, kMlaNope + 64, w.head, row + (k - 3) * 64, vb);
                                }
                            }
                            __syncwarp();
                            ++g;
                        }
                    }
                }
                ok = ok && wait(&c.taken_full, answered & 1);
                if (!ok) break;
                ++answered;
                more = block_taken(&c.taken, x, unused);
                if (more && x < scan_at) {
                    scan_at = 0;
                    look_at(0);
                }
                fence_async_smem();  // read before the next answer is written there
                __syncwarp();
            }
            if (!ok) {
                // let what is in flight land before the block ends; first what a begun group of pieces still lacks, or its
                // barrier would never complete
                const int j = g / PER_TILE, k = g % PER_TILE;
                if (k != 0 && k != 3 && elect_one()) {
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
                for (int s = 0; s < 2; ++s)
                    if (qn[s] > 0) drain(&c.q_full[s], (qn[s] - 1) & 1);
                if (asked > answered) drain(&c.taken_full, answered & 1);
            }
        } else if (warp == 9 || warp == 10) {
            // ---------------------------------------------------------------- products of one side
            const int s = warp - 9;
            const uint32_t base = __shfl_sync(0xffffffffu, smem_u32(smem), 0);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t d_s = tm + COL_S + s * 128, d_o = tm + COL_O + s * 128;
            const uint64_t q = sw128_desc(base + s * 3 * PIECE, 16, 1024);
            constexpr uint32_t idesc_o = idesc_bf16(128, 128, false, true);
            const uint32_t idesc_s = idesc_bf16(128, 128, false, false) | (a.scale < 0.f ? 1u << 13 : 0u);  // negated A
            // Whole warps wait, one lane issues.
            const auto scores = [&](uint32_t g, bool last) {
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const uint64_t kd = sw128_desc(base + OFF_RING + (g + k) % PIECES * PIECE, 16, 1024);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_f16(d_s, q + ((k * PIECE + i * 32) >> 4), kd + i * 2, idesc_s, k + i > 0);
                }
                mma_commit(&c.s_full[s]);
                if (last) mma_commit(&c.q_empty[s]);
            };
            const auto release = [&](uint32_t g, int count) {
                for (int k = 0; k < count; ++k) mma_commit(&c.empty[(g + k) % PIECES]);
            };
            uint32_t it = 0, jt = 0, st = 0, outs = 0;
            bool ok = true;
            while (true) {
                ok = wait(&c.item_full[it & 1], (it >> 1) & 1);
                if (!ok) break;
                const Item w = c.item[it & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.item_empty[it & 1]);
                ++it;
                if (!w.real) break;
                const int n0 = w.tiles(0, a.causal), n1 = w.tiles(1, a.causal), n = s == 0 ? n0 : n1, most = max(n0, n1);
                uint32_t g = jt * PER_TILE;
                if (n > 0) {
                    ok = wait(&c.q_full[s], outs & 1) && wait(&c.k_full[jt & 1], (jt >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
                        scores(g, n == 1);
                        release(g, 3);
                    }
                    __syncwarp();
                    ok = outs == 0 || wait(&c.o_empty[s], (outs - 1) & 1);  // the last item's output has been read
                    ++outs;
                }
                for (int j = 0; j < n && ok; ++j, ++st, g += PER_TILE) {
                    if ((s == 0 ? j == 0 || j > n1 : j >= n0) && lane == 0) mbar_arrive(&c.go[s]);  // no other side to wait for
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        ok = wait(k == 0 ? &c.go[s] : &c.p_full[s], st & 1);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint64_t vd = sw128_desc(base + OFF_RING + (g + 3 + k) % PIECES * PIECE, PIECE / 2, 1024);
                        if (elect_one()) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)  // 16 keys of 2 x 64 channels
                                mma_f16_ts(d_o, d_s + k * 32 + i * 8, vd + ((i * 2048) >> 4), idesc_o, j > 0 || k + i > 0);
                            release(g + 3 + k, 1);  // before the scores: what a commit reports is all that came before it
                            if (k == 1) {
                                if (j + 1 < n) scores(g + PER_TILE, j + 2 == n);
                                if (s == 0 ? j < n1 : j + 1 < n0) mbar_arrive(&c.go[s ^ 1]);  // the other side's turn
                                if (j + 1 < n) release(g + PER_TILE, 3);
                                else mma_commit(&c.o_full[s]);
                            }
                        }
                        __syncwarp();
                    }
                }
                for (int j = n; j < most && ok; ++j, g += PER_TILE) {  // keys that only the other side sees
                    const uint32_t t = jt + j;
                    ok = wait(&c.k_full[t & 1], (t >> 1) & 1);
                    if (ok && lane < 3) mbar_arrive(&c.empty[(g + lane) % PIECES]);
                    ok = ok && wait(&c.v_full[t & 1], (t >> 1) & 1);
                    if (ok && lane < 2) mbar_arrive(&c.empty[(g + 3 + lane) % PIECES]);
                    __syncwarp();
                }
                if (!ok) break;
                jt += most;
            }
            if (!ok) {  // let issued products finish before the block ends
                if (elect_one()) mma_commit(&c.drain_bar[s]);
                __syncwarp();
                drain(&c.drain_bar[s], 0);
            }
        } else {
            // ---------------------------------------------------------------- arrivals: tells the sides' steps of them
            uint32_t it = 0, jt = 0, st[2] = {0, 0};
            bool ok = true;
            while (true) {
                ok = wait(&c.item_full[it & 1], (it >> 1) & 1);
                if (!ok) break;
                const Item w = c.item[it & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.item_empty[it & 1]);
                ++it;
                if (!w.real) break;
                const int n0 = w.tiles(0, a.causal), n1 = w.tiles(1, a.causal), most = max(n0, n1);
                for (int j = 0; j < most && ok; ++j, ++jt) {
                    ok = wait(&c.v_full[jt & 1], (jt >> 1) & 1);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {  // one step at a time, here and below
                        if (j >= (s == 0 ? n0 : n1)) continue;
                        ok = ok && (st[s] == 0 || wait(&c.go[s], (st[s] - 1) & 1));
                        if (ok && lane == 0) mbar_arrive(&c.go[s]);
                    }
                    if (j + 1 < most) ok = ok && wait(&c.k_full[(jt + 1) & 1], ((jt + 1) >> 1) & 1);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (j >= (s == 0 ? n0 : n1)) continue;
                        ok = ok && (st[s] == 0 || wait(&c.p_full[s], (st[s] - 1) & 1));
                        if (ok && lane == 0) mbar_arrive(&c.p_full[s]);
                        ++st[s];
                    }
                }
                if (!ok) break;
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
    if (pairs * a.H > INT32_MAX) return cudaErrorInvalidConfiguration;  // more queries than memory holds
    kernel<<<static_cast<unsigned>(pairs * a.H), THREADS, SMEM_BYTES, a.stream>>>(mq, mk, mv, mp, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_mla_prefill(const MlaPrefillArgs& a) { return a.o_fp32 ? launch<float>(a) : launch<__nv_bfloat16>(a); }

}  // namespace kda
