// Attention of many query tokens over one sequence of a cache: the prefix that a batch shares, read (and, in a
// coded cache, rebuilt) once for all of them.
//
// The library's own operator (the LoopVQ paper decodes every sequence over its own cache).  For the R = rows *
// Hq / Hkv query rows of a KV head, O = softmax(scale Q K^T) V over the prefix's tokens: two matrix products, so
// both run on the tensor cores with accumulators in tensor memory.
//
// One CTA per (token split, KV head, up to 2 x 128 query rows).  Its warps:
//   0-3, 4-7  softmax of stream 0 and stream 1: thread = query row = tensor-memory lane
//   8, 9      bf16 cache: one thread issues every product, one copies K and V tiles by TMA
//   8-15, 16-18  coded cache: eight warps rebuild K tiles, one thread issues every product, two warps rebuild V tiles
// A step is one product pair S = Q K^T, O += P V of 128 rows by one tile of tokens.  Steps alternate between two
// streams, each with its own S, O, maximum and sum, so that the products of one stream run under the softmax of
// the other: with up to 128 rows the streams take the tiles in turn (and give two partial results), with more
// they take the two halves of the rows (and share every tile).
//
// Precision: the library returns fp32, so P is not rounded to bf16 once but split into two bf16 parts (the
// remainder of the first rounding in the second, which leaves 2^-17 of P at most), two products into the same
// accumulator, or three where tokens are few (FINE); a rebuilt, rotated key is split the same way.  bf16 queries, keys
// and values are exact.
//
// The tensor cores cut their fp32 sums toward zero at every product, so values of one sign come out low by as much as there
// are products: 256 tiles in a row (2000 query rows, 32768 tokens) 2.2e-4.  Every 4096 tokens a stream therefore adds its O
// to a sum in the workspace and starts afresh (RUNS): 1.9e-5 there, in 639 us instead of 620.
//
// P overwrites S in place, 16 score columns becoming 8 + 8 columns of packed pairs (one product's tokens; a third part
// has columns of its own).  The running maximum moves only when a tile passes it by 2^8 (any reference is exact; it
// bounds P), so O is rarely rescaled.
//
// What bounds it: over a bf16 prefix the products and, with few tiles a CTA, its set-up and exchange (16347 tokens, 64
// queries, 4 KV / 16 query heads: 26 us with the merge, tensor pipe busy 33% of 24); over a coded one the shared-memory
// pipe, which gathers, tile stores and the products' operands share (32768 tokens, 32 queries, 16 heads: 77 us, the pipe
// busy 73% of it).
#pragma once

#include "shared_rows.cuh"

namespace loopvq {

struct SharedArgs {
    const uint16_t *q;       // [rows][Hq][D]
    const int32_t *start;    // of the sequence, or null
    const int32_t *len;
    float *ws_o;             // [nsplit][Hkv][D / 4][R][4]: a warp's 32 rows write 512 bytes in a run
    float2 *ws_ml;           // [nsplit][Hkv][R]: maximum reference (log2 units), sum
    int rows, Hkv, Hq, R, qpk, max_len, nsplit;
    int qshift;              // log2 of qpk
    float qscale;            // scale * log2(e)
    unsigned int *fault;
    unsigned long long wait_ns;
    // bf16 cache: rows of the sequence's tensor map per KV head
    int head_rows;
    // coded cache
    const uint32_t *idx;     // of (layer, block, sequence, h = 0)
    size_t idx_head;         // words per KV head
    const uint16_t *slk, *slv;
    const float *rope;
    int K;
    // tiles of a stream after which O leaves tensor memory (run), and where it is summed: [CTA][stream][D / 4][128][4]
    int run;
    float4 *ws_run;
    // one split: the kernel writes the result itself, merged with the other part (null where there is none)
    const float *other_out, *other_lse;
    float *out, *lse;        // out null: records for the merge; lse may be null
};

// Shared-memory and tensor-memory plan.  NT tokens per tile, KP bf16 parts per key, PARTS of P.
// FINE: P and rebuilt keys in three parts, all of an fp32 value, where one CTA writes the result of few tokens.
// bf16 cache: the queries lie in shared memory (S and O fill the tensor memory at 128-token tiles).
// Coded cache: 64-token tiles leave tensor memory for the queries, so the products read only the tiles from shared
// memory, whose bandwidth they share with the rebuilding.
template <int D, int MB, int C, bool PG, bool FINE>
struct Plan {
    static constexpr bool coded = C != 0;
    static constexpr int NT = coded || FINE ? 64 : 128;
    static constexpr int KP = coded ? (FINE ? 3 : 2) : 1;
    static constexpr int PARTS = FINE ? 3 : 2;
    static constexpr int kPanel = NT * 128;                          // 64 channels of a tile
    static constexpr int kTile = (D / 64) * kPanel;
    static constexpr int kStage = (KP + 1) * kTile;                  // K parts, then V
    static constexpr int kQ = coded ? 0 : (D / 64) * 128 * 128;      // one row block
    static constexpr int ST = D == 64 ? 4 : coded ? (FINE ? 2 : 4) : FINE ? 4 : MB == 1 ? 3 : 2;
    static constexpr int kTable = coded && !PG ? kTableBytes : 0;    // K slice, then V slice
    static constexpr int offQ = 0;
    static constexpr int offStage = MB * kQ;
    static constexpr int offTable = offStage + ST * kStage;
    static constexpr int offTurn = offTable + 2 * kTable;            // rope row 64: the turn from tile to tile
    static constexpr int offBar = offTurn + (coded ? D * 4 : 0);
    static constexpr int kBars = 4 * ST + 7;
    static constexpr int offTmem = offBar + kBars * 8;
    static constexpr int kUsed = offTmem + 16;
    static constexpr int kAlloc = kUsed + 1024;
    static constexpr int kThreads = coded ? 20 * 32 : 320;
    static constexpr int kMma = coded ? 16 : 8;                      // warps: products;
    static constexpr int kCopy = coded ? 16 : 9;                     // copies (and the barriers' set-up);
    [[maybe_unused]] static constexpr int kRebuild = 8, kValues = 17;                 // the first of those that rebuild keys, values
    static constexpr int colS = NT;                                  // S of stream w at w * colS
    [[maybe_unused]] static constexpr int colP3 = 192;                // FINE: third part of P of stream w at 192 + 32 w
    static_assert(!FINE || MB == 1, "Q of a second row block lies there");
    [[maybe_unused]] static constexpr int colQ = coded ? 128 : 0;                     // coded: Q of row block w at 128 + 64 w
    static_assert(kAlloc <= 232448, "shared memory");
    static_assert(ST * kStage >= 128 * D * 4, "the streams' exchange reuses the tiles");
};

constexpr int kTmemCols = 512;                                       // O of stream w at 256 + 128 w

// The running softmax of one query row of one stream, and what its thread does with a tile's scores.
template <int D, int NT, int PARTS>
struct RowSoftmax {
    float m, l;                                                      // maximum reference (log2 units), sum
    bool far;                                                        // some row of the warp's is past kExact
    float carry;                                                     // factor that brings the sum of earlier runs to m
    static constexpr float kExact = 16777216.f;                      // scores up to here are held to 2 log2 units

    // S columns at ts (a third part of P goes to tp); tokens [lo, hi) of the tile count; O columns at to.  first: O holds
    // nothing yet.
    // odone: barrier (parity) of the stream's previous O += P V.
    __device__ __forceinline__ bool tile(uint32_t ts, uint32_t tp, uint32_t to, int lo, int hi, float qs, bool first, uint32_t odone,
                                         uint32_t odone_parity, uint64_t limit, volatile int *dead) {
        // 32 scores at a time, read from tensor memory once for the maximum and once for the exponentials: a tile's
        // scores in registers spill, and loops keep the code small enough for the instruction cache (a call of few
        // tiles spent most of its time fetching the unrolled form: 3400 clocks for its first tile)
        const bool edge = lo > 0 || hi < NT;
        auto load = [&](uint32_t (&x)[32], int c) {
            tc::tmem_ld32(ts + c, x);
            tc::tmem_wait_ld(x);
            if (edge) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (c + k < lo || c + k >= hi) x[k] = 0xff800000u;
            }
        };
        float a0 = -CUDART_INF_F, a1 = a0, a2 = a0, a3 = a0;
#pragma unroll 1
        for (int c = 0; c < NT; c += 32) {
            uint32_t x[32];
            load(x, c);
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                a0 = fmaxf(a0, __uint_as_float(x[k]));
                a1 = fmaxf(a1, __uint_as_float(x[k + 1]));
                a2 = fmaxf(a2, __uint_as_float(x[k + 2]));
                a3 = fmaxf(a3, __uint_as_float(x[k + 3]));
            }
        }
        const float mt = fmaxf(fmaxf(a0, a1), fmaxf(a2, a3)) * qs;
        const bool up = mt > m + 8.f;
        if (__any_sync(0xffffffffu, up)) {
            const float corr = up ? ex2(m - mt) : 1.f;
            if (up) m = mt;
            l *= corr;
            carry *= corr;
            far = __any_sync(0xffffffffu, fabsf(m) > kExact && m != -CUDART_INF_F);
            if (!first) {
                const bool ok = tc::mbar_wait_or_dead(odone, odone_parity, limit, dead);
                if (!__all_sync(0xffffffffu, ok)) return false;
                tc::tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tc::tmem_ld32(to + c, o);
                    tc::tmem_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * corr);
                    tc::tmem_st32(to + c, o);
                }
            }
        }
        float nm = m == -CUDART_INF_F ? 0.f : -m;
        if (far) {
            // a reference that cannot hold fractions of its scores: the difference of two rounded numbers, which is 0 at the
            // maximum, takes the place of the scores, instead of an exact product less a rounded one
#pragma unroll 1
            for (int c = 0; c < NT; c += 32) {
                uint32_t x[32];
                tc::tmem_ld32(ts + c, x);
                tc::tmem_wait_ld(x);
#pragma unroll
                for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(x[k]), qs), nm));
                tc::tmem_st32(ts + c, x);
            }
            tc::tmem_wait_st();
            qs = 1.f;
            nm = 0.f;
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll 1
        for (int c = 0; c < NT; c += 32) {
            uint32_t x[32];
            load(x, c);
            [[maybe_unused]] uint32_t w3[16];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float p0 = ex2(fmaf(__uint_as_float(x[half * 16 + 2 * k]), qs, nm));
                    const float p1 = ex2(fmaf(__uint_as_float(x[half * 16 + 2 * k + 1]), qs, nm));
                    s0 += p0;
                    s1 += p1;
                    const uint32_t hi2 = cvt_bf16x2(p1, p0);
                    w[k] = hi2;
                    const float d0 = p0 - bf16lo(hi2), d1 = p1 - bf16hi(hi2);
                    w[8 + k] = cvt_bf16x2(d1, d0);
                    if constexpr (PARTS == 3) w3[half * 8 + k] = cvt_bf16x2(d1 - bf16hi(w[8 + k]), d0 - bf16lo(w[8 + k]));
                }
                tc::tmem_st16(ts + c + half * 16, w);
            }
            if constexpr (PARTS == 3) tc::tmem_st16(tp + c / 2, w3);
        }
        l += s0 + s1;
        tc::tmem_wait_st();
        return true;
    }

    // O at `to` is added to the sum of the runs before (more) at `sum`, in fp32 rounded to nearest; the next product starts
    // O afresh.  Where the maximum has not moved since (carry 1 in the whole warp) the memory does the addition and nothing
    // waits for it: an element has one thread, so the order is fixed.
    __device__ __forceinline__ void end_run(uint32_t to, float4 *sum, bool more) {
        const bool moved = __any_sync(0xffffffffu, carry != 1.f);
#pragma unroll 1
        for (int k0 = 0; k0 < D; k0 += 32) {
            uint32_t o[32];
            tc::tmem_ld32(to + k0, o);
            tc::tmem_wait_ld(o);
            if (more && !moved) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(sum + (k0 / 4 + k) * 128),
                                 "f"(__uint_as_float(o[4 * k])), "f"(__uint_as_float(o[4 * k + 1])),
                                 "f"(__uint_as_float(o[4 * k + 2])), "f"(__uint_as_float(o[4 * k + 3])) : "memory");
                continue;
            }
            if (more) add_runs(o, sum, k0);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sum[(k0 / 4 + k) * 128] = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                      __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
        }
        carry = 1.f;
    }
    __device__ __forceinline__ void add_runs(uint32_t (&o)[32], const float4 *sum, int k0) const {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 y = __ldcg(sum + (k0 / 4 + k) * 128);           // (the additions are made in L2)
            o[4 * k] = __float_as_uint(fmaf(y.x, carry, __uint_as_float(o[4 * k])));
            o[4 * k + 1] = __float_as_uint(fmaf(y.y, carry, __uint_as_float(o[4 * k + 1])));
            o[4 * k + 2] = __float_as_uint(fmaf(y.z, carry, __uint_as_float(o[4 * k + 2])));
            o[4 * k + 3] = __float_as_uint(fmaf(y.w, carry, __uint_as_float(o[4 * k + 3])));
        }
    }
};

// D channels (64 or 128), MB blocks of 128 query rows per CTA, C = 0 for a bf16 cache or the channels per code of
// a coded one; PG: one codebook per channel group, whose slices (128 bytes per entry and more) do not fit beside
// the tiles and are gathered from L2.  RUNS: O leaves tensor memory every a.run tiles of a stream (as a test of a.run in one
// kernel for both: 16347 tokens, 64 grouped queries 26.4 us against 26.0).
template <int D, int MB, int C, bool PG, bool FINE, bool RUNS>
__global__ void __launch_bounds__(Plan<D, MB, C, PG, FINE>::kThreads, 1)
    shared_attn_kernel(const SharedArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    using P = Plan<D, MB, C, PG, FINE>;
    constexpr bool coded = C != 0;
    constexpr int NT = P::NT, KP = P::KP, ST = P::ST, NPAN = D / 64;

    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (base - tc::smem_u32(smem_raw));
    const uint32_t sQ = base + P::offQ, sStage = base + P::offStage, bars = base + P::offBar;
    auto kfull = [&](int s) { return bars + 8u * s; };
    auto vfull = [&](int s) { return bars + 8u * (ST + s); };
    auto kempty = [&](int s) { return bars + 8u * (2 * ST + s); };
    auto vempty = [&](int s) { return bars + 8u * (3 * ST + s); };
    auto sfull = [&](int w) { return bars + 8u * (4 * ST + w); };
    auto pfull = [&](int w) { return bars + 8u * (4 * ST + 2 + w); };
    auto odone = [&](int w) { return bars + 8u * (4 * ST + 4 + w); };
    const uint32_t drain = bars + 8u * (4 * ST + 6);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + P::offTmem);
    volatile int *dead = reinterpret_cast<volatile int *>(smem + P::offTmem + 4);

    const int tid = threadIdx.x, lane = tid & 31, warp = tc::uniform_warp();
    const int split = blockIdx.x, h = blockIdx.y;
    const int r0 = blockIdx.z * (MB * 128);                          // first query row of this CTA

    grid_trigger();
    grid_wait();
    const int len = min(max(word(a.len), 0), a.max_len);
    const int st = a.start ? min(max(word(a.start), 0), len) : 0;
    const int tok0 = coded ? (st & ~3) : st;                         // index words come in tiles of 4 tokens
    const int tiles_all = len > st ? (len - tok0 + NT - 1) / NT : 0;
    const int t_first = (int)((long long)split * tiles_all / a.nsplit);
    const int ntiles = (int)((long long)(split + 1) * tiles_all / a.nsplit) - t_first;
    const int tok_first = tok0 + t_first * NT;
    const int nsteps = ntiles * MB;                                  // step i: stream i & 1
    const size_t rec = ((size_t)split * a.Hkv + h) * a.R;            // this split's records of the head

    const bool whole = a.out != nullptr;                             // no other split, no merge
    auto result_row = [&](int r) {
        return (size_t)(r >> a.qshift) * a.Hq + h * a.qpk + (r & (a.qpk - 1));
    };
    if (ntiles == 0 && whole) {                                      // no tokens: the other part, or zeros
        const int rows = min(MB * 128, a.R - r0);
        for (int it = tid; it < rows * (D / 4); it += P::kThreads) {
            const size_t row = result_row(r0 + it / (D / 4));
            const float ol = a.other_lse ? a.other_lse[row] : -CUDART_INF_F;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (ol != -CUDART_INF_F) x = *reinterpret_cast<const float4 *>(a.other_out + row * D + it % (D / 4) * 4);
            if (!(fabsf(ol) < CUDART_INF_F) && ol != -CUDART_INF_F) x = make_float4(ol - ol, ol - ol, ol - ol, ol - ol);
            *reinterpret_cast<float4 *>(a.out + row * D + it % (D / 4) * 4) = x;
            if (a.lse != nullptr && it % (D / 4) == 0) a.lse[row] = ol == CUDART_INF_F ? ol - ol : ol;
        }
        return;
    }
    if (ntiles == 0) {                                               // nothing in this split
        for (int r = r0 + tid; r < min(r0 + MB * 128, a.R); r += P::kThreads) a.ws_ml[rec + r] = f2(-CUDART_INF_F, 0.f);
        return;
    }

    // ---- set-up: barriers and the first copies, tensor memory, queries (and the slices of a coded cache)
    auto issue_k = [&](int t) {
        const int s = t % ST;
        tc::mbar_expect_tx(kfull(s), P::kTile);
#pragma unroll
        for (int p = 0; p < NPAN; ++p)
            tc::tma_load_2d(sStage + s * P::kStage + p * P::kPanel, &kmap, p * 64, h * a.head_rows + tok_first + t * NT,
                            kfull(s));
    };
    auto issue_v = [&](int t) {
        const int s = t % ST;
        tc::mbar_expect_tx(vfull(s), P::kTile);
#pragma unroll
        for (int p = 0; p < NPAN; ++p)
            tc::tma_load_2d(sStage + s * P::kStage + KP * P::kTile + p * P::kPanel, &vmap, p * 64,
                            h * a.head_rows + tok_first + t * NT, vfull(s));
    };
    int issued = 0;                                                  // tiles copied by the producer thread
    if (warp == P::kCopy && lane == 0) {
        for (int s = 0; s < ST; ++s) {
            tc::mbar_init(kfull(s), coded ? 8 : 1);
            tc::mbar_init(vfull(s), coded ? 2 : 1);
            tc::mbar_init(kempty(s), 1);
            tc::mbar_init(vempty(s), 1);
        }
        for (int w = 0; w < 2; ++w) {
            tc::mbar_init(sfull(w), 1);
            tc::mbar_init(pfull(w), 128);
            tc::mbar_init(odone(w), 1);
        }
        tc::mbar_init(drain, 1);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if constexpr (!coded) {
            for (; issued < ntiles && issued < ST; ++issued) {
                issue_k(issued);
                issue_v(issued);
            }
        }
    }
    if (warp == P::kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(tmem_slot)),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // queries: rows of warps that have a real one (the others' lanes are never read), padding rows zero
    auto q_row = [&](int r) {
        return a.q + ((size_t)((r0 + r) >> a.qshift) * a.Hq + h * a.qpk + ((r0 + r) & (a.qpk - 1))) * D;
    };
    uint4 qv[coded ? D / 8 : 1];                                     // coded: this thread's query row
    const int q_rows = min(MB * 128, (a.R - r0 + 31) & ~31);
    if constexpr (!coded) {
        for (int it = tid; it < q_rows * (D / 8); it += P::kThreads) {
            const int r = it / (D / 8), ch = it % (D / 8);
            const uint32_t dst = sQ + (r / 128) * P::kQ + (ch / 8) * (128 * 128) + sw128(r % 128, ch % 8);
            const bool real = r0 + r < a.R;
            cp_async16_zfill(dst, real ? q_row(r) + ch * 8 : a.q, real);
        }
        cp_async_commit();
    } else {
        if (tid < q_rows) {
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                qv[c] = r0 + tid < a.R ? *reinterpret_cast<const uint4 *>(q_row(tid) + c * 8) : make_uint4(0, 0, 0, 0);
        }
        for (int i = tid; i < D; i += P::kThreads)                   // used from the second tile on: row 64 is there
            reinterpret_cast<float *>(smem + P::offTurn)[i] = ntiles > 1 ? a.rope[(size_t)64 * D + i] : 0.f;
    }
    if constexpr (coded && !PG)
        fill_tables<C>(smem + P::offTable, a.slk + (size_t)h * a.K * C, a.slv + (size_t)h * a.K * C, a.K, P::kThreads);
    cp_async_wait<0>();
    tc::fence_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if constexpr (coded) {
        if (warp * 32 < q_rows) {                                    // the queries into tensor memory
            uint32_t x[32];
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 v = qv[c / 4 + k];
                    x[4 * k] = v.x;
                    x[4 * k + 1] = v.y;
                    x[4 * k + 2] = v.z;
                    x[4 * k + 3] = v.w;
                }
                tc::tmem_st32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + P::colQ + (warp >> 2) * 64 + c, x);
            }
            tc::tmem_wait_st();
        }
        tc::tc_fence_before();
        __syncthreads();
        tc::tc_fence_after();
    }

    if (warp < 8) {
        // ---- softmax of stream w: 128 threads, one query row each
        // 20 warps are launched with 96 registers each; the running cosines and sines of the warps that rebuild keys need
        // more and the softmax less: 256 x 80 + 256 x 112 + 128 x 96 = 640 x 96
        if constexpr (coded) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int w = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lane_base + w * P::colS, to = tmem + lane_base + 256 + w * 128;
        const int rq = r0 + (MB == 2 ? w * 128 : 0) + row;           // query row of this thread
        const bool any = __any_sync(0xffffffffu, rq < a.R);          // warps of padding only keep step
        RowSoftmax<D, NT, P::PARTS> sm{-CUDART_INF_F, 0.f, false, 1.f};
        bool ok = true;
        int j = 0, in_run = 0;                                       // tiles of the stream, and of its O
        [[maybe_unused]] float4 *runs = a.ws_run + ((((size_t)blockIdx.z * a.Hkv + h) * a.nsplit + split) * 2 + w) * (D / 4) * 128 + row;
        for (int i = w; i < nsteps; i += 2, ++j, ++in_run) {
            const int t = MB == 2 ? j : i;
            ok = __all_sync(0xffffffffu, tc::mbar_wait_or_dead(sfull(w), j & 1, a.wait_ns, dead));
            if (!ok) break;
            tc::tc_fence_after();
            if constexpr (RUNS) {
                if (in_run == a.run) {                               // (S of this step is behind the last product of O)
                    if (any) sm.end_run(to, runs, j > in_run);
                    in_run = 0;
                }
            }
            if (any) {
                const int n0 = tok_first + t * NT;
                ok = sm.tile(ts, tmem + lane_base + P::colP3 + w * 32, to, st - n0, len - n0, a.qscale, in_run == 0, odone(w),
                             (j - 1) & 1, a.wait_ns, dead);
                if (!ok) break;
            }
            tc::tc_fence_before();
            tc::mbar_arrive(pfull(w));
        }
        if (ok && j > 0) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait_or_dead(odone(w), (j - 1) & 1, a.wait_ns, dead));
            tc::tc_fence_after();
        }
        // with two streams of one row block, stream 1 hands its part to stream 0 through the tiles' memory, free by
        // now (every product of both streams is done once both have waited): 16 bytes of 32 rows in a run
        float c0 = 1.f, c1 = 0.f;
        float4 *ex = reinterpret_cast<float4 *>(smem + P::offStage);
        if constexpr (MB == 1) {
            float *mls = reinterpret_cast<float *>(smem + P::offStage);   // first the rows' (m, l)
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (w == 1) {
                mls[row] = !ok ? 0.f : j > 0 ? sm.m : -CUDART_INF_F;
                mls[128 + row] = !ok ? CUDART_NAN_F : j > 0 ? sm.l : 0.f;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (w == 0) {
                const float m1 = mls[row], l1 = mls[128 + row];
                if (j == 0) sm.m = -CUDART_INF_F;
                const float top = fmaxf(sm.m, m1);
                c0 = top == -CUDART_INF_F ? 0.f : ex2(sm.m - top);
                c1 = top == -CUDART_INF_F ? 0.f : ex2(m1 - top);
                sm.l = sm.l * c0 + l1 * c1;
                sm.m = top;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (w == 1 && any) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    if (j > 0) {
                        tc::tmem_ld32(to + c, o);
                        tc::tmem_wait_ld(o);
                        if (RUNS && j > in_run) sm.add_runs(o, runs, c);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0u;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        ex[(c / 4 + k) * 128 + row] =
                            make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                        __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
        // the factors of this thread's O and of the other part in the result, where the kernel writes it
        const size_t dst = rq < a.R ? result_row(rq) : 0;
        float f_own = 1.f, f_other = 0.f;
        if (whole && rq < a.R && (MB == 2 || w == 0)) {
            const float ol = a.other_lse ? a.other_lse[dst] * 1.44269504088896340736f : -CUDART_INF_F;
            const float top = fmaxf(sm.m, ol);
            float l2 = -CUDART_INF_F;
            f_own = 0.f;
            if (top != -CUDART_INF_F) {
                const float eo = ex2(sm.m - top), ex = ex2(ol - top), total = sm.l * eo + ex;
                l2 = top + log2f(total);
                f_own = eo / total;
                f_other = ex / total;
            }
            if (!ok || sm.l != sm.l || ol != ol) f_own = f_other = l2 = CUDART_NAN_F;
            if (a.lse != nullptr) a.lse[dst] = l2 == -CUDART_INF_F ? l2 : l2 * 0.69314718055994530942f;
        }
        if (any && (MB == 2 || w == 0)) {
            // (a maximum passes NaN over: a row of nothing but NaN must not look like one without tokens)
            if (!whole && rq < a.R) a.ws_ml[rec + rq] = ok && sm.l == sm.l ? f2(sm.m, sm.l) : f2(0.f, CUDART_NAN_F);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc::tmem_ld32(to + c, o);
                tc::tmem_wait_ld(o);
                if (RUNS && j > in_run) sm.add_runs(o, runs, c);
                if (rq < a.R) {
                    float4 *rec_o = reinterpret_cast<float4 *>(a.ws_o) + (rec / a.R * (D / 4) + c / 4) * a.R + rq;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float4 x = make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                               __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
                        if constexpr (MB == 1) {
                            const float4 y = ex[(c / 4 + k) * 128 + row];
                            x.x = x.x * c0 + y.x * c1;
                            x.y = x.y * c0 + y.y * c1;
                            x.z = x.z * c0 + y.z * c1;
                            x.w = x.w * c0 + y.w * c1;
                        }
                        if (whole) {
                            const size_t at = dst * D + c + 4 * k;
                            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);   // (factors of NaN make the row NaN)
                            if (a.other_lse && f_other != 0.f) y = *reinterpret_cast<const float4 *>(a.other_out + at);
                            x = f_own != 0.f ? make_float4(x.x * f_own, x.y * f_own, x.z * f_own, x.w * f_own)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
                            if (f_other != 0.f)
                                x = make_float4(x.x + y.x * f_other, x.y + y.y * f_other, x.z + y.z * f_other, x.w + y.w * f_other);
                            *reinterpret_cast<float4 *>(a.out + at) = x;
                        } else {
                            rec_o[(size_t)k * a.R] = x;
                        }
                    }
                }
            }
        }
        tc::tc_fence_before();
    } else if (warp == P::kMma) {
        // ---- products
        constexpr uint32_t id_qk = tc::idesc_bf16(128, NT);
        constexpr uint32_t id_pv = tc::idesc_bf16(128, D) | (1u << 16);        // B: channels contiguous
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait_or_dead(bar, parity, a.wait_ns, dead));
            return ok;
        };
        auto qk = [&](int i) {                                       // S of step i
            const int t = MB == 2 ? i >> 1 : i, s = t % ST;
            if (!wait(kfull(s), (t / ST) & 1)) return;
            tc::tc_fence_after();
            constexpr uint32_t hi = tc::desc_hi(1024, 2);
            const uint32_t sd = tc::uniform(tmem + (i & 1) * P::colS);
            const uint32_t k_lo = tc::uniform(tc::desc_lo(sStage + s * P::kStage, 16));
            const uint32_t q_lo = tc::uniform(tc::desc_lo(sQ + (MB == 2 ? (i & 1) * P::kQ : 0), 16));
            const uint32_t q_tm = tc::uniform(tmem + P::colQ + (MB == 2 ? (i & 1) * 64 : 0));
            if (tc::elect_one()) {
#pragma unroll
                for (int part = 0; part < KP; ++part)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {               // 16 channels per product: 32 bytes of a row
                        const uint32_t at = k_lo + (part * P::kTile + (k / 4) * P::kPanel + (k % 4) * 32) / 16;
                        if constexpr (coded)
                            tc::mma_ts(sd, q_tm + k * 8, at, hi, id_qk, part + k > 0);
                        else
                            tc::mma_ss(sd, q_lo + ((k / 4) * (128 * 128) + (k % 4) * 32) / 16, hi, at, hi, id_qk, part + k > 0);
                    }
                if ((MB == 1 || (i & 1)) && t + ST < ntiles) tc::mma_commit(kempty(s));
                tc::mma_commit(sfull(i & 1));
            }
            __syncwarp();
        };
        int in_run = 0;                                              // tiles in the O of this step's stream
        qk(0);
        if (ok && nsteps > 1) qk(1);
        for (int i = 0; ok && i < nsteps; ++i) {
            const int t = MB == 2 ? i >> 1 : i, s = t % ST, w = i & 1;
            const uint32_t vb = sStage + s * P::kStage + KP * P::kTile;
            if (!wait(vfull(s), (t / ST) & 1)) break;
            if constexpr (!coded) {
                // rows behind the last token may hold anything: 0 x that has to be 0
                const int end = len - (tok_first + t * NT);
                if (end < NT && (MB == 1 || w == 0)) {
                    for (int it = lane; it < (NT - end) * (D / 8); it += 32) {
                        const int n = end + it / (D / 8), ch = it % (D / 8);
                        sts128(vb + (ch / 8) * P::kPanel + n * 128 + (ch % 8) * 16, make_uint4(0, 0, 0, 0));
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                }
            }
            if (!wait(pfull(w), (i >> 1) & 1)) break;
            tc::tc_fence_after();
            const uint32_t od = tc::uniform(tmem + 256 + w * 128), pa = tc::uniform(tmem + w * P::colS);
            [[maybe_unused]] const uint32_t pz = tc::uniform(tmem + P::colP3 + w * 32);
            const uint32_t v_lo = tc::uniform(tc::desc_lo(vb, P::kPanel)), more = tc::uniform(in_run != 0);
            if (tc::elect_one()) {
#pragma unroll
                for (int part = 0; part < P::PARTS; ++part)
#pragma unroll
                    for (int k = 0; k < NT / 16; ++k)                // 16 tokens per product: 8 packed columns
                        tc::mma_ts(od, part < 2 ? pa + k * 16 + part * 8 : pz + k * 8, v_lo + k * 128, tc::desc_hi(1024, 2), id_pv,
                                   part + k > 0 ? 1u : more);
                if ((MB == 1 || w == 1) && t + ST < ntiles) tc::mma_commit(vempty(s));
                tc::mma_commit(odone(w));
            }
            __syncwarp();
            if (w == 1 && ++in_run == a.run && RUNS) in_run = 0;
            if (i + 2 < nsteps) qk(i + 2);
        }
    } else if constexpr (!coded) {
        // ---- copies
        if (lane == 0) {
            bool ok = true;
            for (int t = issued; t < ntiles; ++t) {
                const int s = t % ST;
                const uint32_t par = (t / ST - 1) & 1;
                if (!(ok = tc::mbar_wait_or_dead(kempty(s), par, a.wait_ns, dead))) break;
                issue_k(t);
                if (!(ok = tc::mbar_wait_or_dead(vempty(s), par, a.wait_ns, dead))) {
                    // the drain below waits for both halves of every issued tile
                    issue_v(t);
                    ++issued;
                    break;
                }
                issue_v(t);
                ++issued;
            }
        }
    } else {
        // ---- rebuilding
        RebuildArgs b;
        b.idx = a.idx + (size_t)h * a.idx_head;
        b.slk = a.slk + (size_t)h * a.K * (PG ? D : C);
        b.slv = a.slv + (size_t)h * a.K * (PG ? D : C);
        b.rope = a.rope;
        b.table = smem + P::offTable;
        b.turn = smem + P::offTurn;
        b.stages = sStage;
        b.kfull = kfull(0);
        b.vfull = vfull(0);
        b.kempty = kempty(0);
        b.vempty = vempty(0);
        b.K = a.K;
        b.wait_ns = a.wait_ns;
        b.dead = dead;
        if (warp < P::kRebuild + 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
            rebuild_keys<D, C, PG, ST, KP>(b, warp - P::kRebuild, tok_first, ntiles, st, len);
        } else if (warp < P::kValues + 2) {
            rebuild_values<D, C, PG, ST, KP>(b, warp - P::kValues, tok_first, ntiles, st, len);
        }
    }

    // ---- all done (or given up): free the tensor memory
    __syncthreads();
    if (*dead) {
        if (tid == 0) atomicOr(a.fault, kFaultAttnWait);
        if (!coded && warp == P::kCopy && lane == 0)                        // copies still in flight
            for (int t = issued > ST ? issued - ST : 0; t < issued; ++t) {
                tc::mbar_wait_bounded(kfull(t % ST), (t / ST) & 1, tc::kDrainNs);
                tc::mbar_wait_bounded(vfull(t % ST), (t / ST) & 1, tc::kDrainNs);
            }
        if (warp == P::kMma && tc::elect_one()) {                    // products still in flight, of the thread that issued them
            tc::mma_commit(drain);
            tc::mbar_wait_bounded(drain, 0, tc::kDrainNs);
        }
        __syncthreads();
    }
    tc::tc_fence_after();
    if (warp == P::kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

}  // namespace loopvq
