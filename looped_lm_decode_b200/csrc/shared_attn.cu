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
// remainder of the first rounding in the second, which leaves 2^-17 of P at most), two products into the same accumulator; a
// rebuilt, rotated key is split the same way.  bf16 queries, keys and values are exact.
//
// P overwrites S in place, 16 score columns becoming 8 + 8 columns of packed pairs (one product's tokens).  The running maximum moves
// only when a tile passes it by 2^8 (any reference is exact; it bounds P), so O is rarely rescaled.
#include <cuda.h>

#include <atomic>

#include "shared_rows.cuh"

namespace loopvq {

namespace {

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
};

// Shared-memory and tensor-memory plan.  NT tokens per tile, KP bf16 parts per key.
// bf16 cache: the queries lie in shared memory (S and O fill the tensor memory at 128-token tiles).
// Coded cache: 64-token tiles leave tensor memory for the queries, so the products read only the tiles from shared
// memory, whose bandwidth they share with the rebuilding.
template <int D, int MB, int C, bool PG>
struct Plan {
    static constexpr bool coded = C != 0;
    static constexpr int NT = coded ? 64 : 128;
    static constexpr int KP = coded ? 2 : 1;
    static constexpr int kPanel = NT * 128;                          // 64 channels of a tile
    static constexpr int kTile = (D / 64) * kPanel;
    static constexpr int kStage = (KP + 1) * kTile;                  // K parts, then V
    static constexpr int kQ = coded ? 0 : (D / 64) * 128 * 128;      // one row block
    static constexpr int ST = D == 64 || coded ? 4 : MB == 1 ? 3 : 2;
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
    static constexpr int kRebuild = 8, kValues = 17;                 // the first of those that rebuild keys, values
    static constexpr int colS = coded ? 64 : 128;                    // S of stream w at w * colS
    static constexpr int colQ = coded ? 128 : 0;                     // coded: Q of row block w at 128 + 64 w
    static_assert(kAlloc <= 232448, "shared memory");
    static_assert(ST * kStage >= 128 * D * 4, "the streams' exchange reuses the tiles");
};

constexpr int kTmemCols = 512;                                       // O of stream w at 256 + 128 w

// The running softmax of one query row of one stream, and what its thread does with a tile's scores.
template <int D, int NT>
struct RowSoftmax {
    float m, l;                                                      // maximum reference (log2 units), sum

    // S columns at ts; tokens [lo, hi) of the tile count; O columns at to.  first: O holds nothing yet.
    // odone: barrier (parity) of the stream's previous O += P V.
    __device__ __forceinline__ bool tile(uint32_t ts, uint32_t to, int lo, int hi, float qs, bool first, uint32_t odone,
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
        const float nm = m == -CUDART_INF_F ? 0.f : -m;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll 1
        for (int c = 0; c < NT; c += 32) {
            uint32_t x[32];
            load(x, c);
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
                    w[8 + k] = cvt_bf16x2(p1 - bf16hi(hi2), p0 - bf16lo(hi2));
                }
                tc::tmem_st16(ts + c + half * 16, w);
            }
        }
        l += s0 + s1;
        tc::tmem_wait_st();
        return true;
    }
};

// D channels (64 or 128), MB blocks of 128 query rows per CTA, C = 0 for a bf16 cache or the channels per code of
// a coded one; PG: one codebook per channel group, whose slices (128 bytes per entry and more) do not fit beside
// the tiles and are gathered from L2.
template <int D, int MB, int C, bool PG>
__global__ void __launch_bounds__(Plan<D, MB, C, PG>::kThreads, 1)
    shared_attn_kernel(const SharedArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    using P = Plan<D, MB, C, PG>;
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
    const int len = min(max(__ldg(a.len), 0), a.max_len);
    const int st = a.start ? min(max(__ldg(a.start), 0), len) : 0;
    const int tok0 = coded ? (st & ~3) : st;                         // index words come in tiles of 4 tokens
    const int tiles_all = len > st ? (len - tok0 + NT - 1) / NT : 0;
    const int t_first = (int)((long long)split * tiles_all / a.nsplit);
    const int ntiles = (int)((long long)(split + 1) * tiles_all / a.nsplit) - t_first;
    const int tok_first = tok0 + t_first * NT;
    const int nsteps = ntiles * MB;                                  // step i: stream i & 1
    const size_t rec = ((size_t)split * a.Hkv + h) * a.R;            // this split's records of the head

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
        RowSoftmax<D, NT> sm{-CUDART_INF_F, 0.f};
        bool ok = true;
        int j = 0;
        for (int i = w; i < nsteps; i += 2, ++j) {
            const int t = MB == 2 ? j : i;
            ok = __all_sync(0xffffffffu, tc::mbar_wait_or_dead(sfull(w), j & 1, a.wait_ns, dead));
            if (!ok) break;
            tc::tc_fence_after();
            if (any) {
                const int n0 = tok_first + t * NT;
                ok = sm.tile(ts, to, st - n0, len - n0, a.qscale, j == 0, odone(w), (j - 1) & 1, a.wait_ns, dead);
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
        if (any && (MB == 2 || w == 0)) {
            if (rq < a.R) a.ws_ml[rec + rq] = ok ? f2(sm.m, sm.l) : f2(0.f, CUDART_NAN_F);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tc::tmem_ld32(to + c, o);
                tc::tmem_wait_ld(o);
                if (rq < a.R) {
                    float4 *dst = reinterpret_cast<float4 *>(a.ws_o) + (rec / a.R * (D / 4) + c / 4) * a.R + rq;
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
                        dst[(size_t)k * a.R] = x;
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
            const uint32_t v_lo = tc::uniform(tc::desc_lo(vb, P::kPanel)), more = tc::uniform(i > 1);
            if (tc::elect_one()) {
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int k = 0; k < NT / 16; ++k)                // 16 tokens per product: 8 packed columns
                        tc::mma_ts(od, pa + k * 16 + part * 8, v_lo + k * 128, tc::desc_hi(1024, 2), id_pv,
                                   part + k > 0 ? 1u : more);
                if ((MB == 1 || w == 1) && t + ST < ntiles) tc::mma_commit(vempty(s));
                tc::mma_commit(odone(w));
            }
            __syncwarp();
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
            rebuild_keys<D, C, PG, ST>(b, warp - P::kRebuild, tok_first, ntiles, st, len);
        } else if (warp < P::kValues + 2) {
            rebuild_values<D, C, PG, ST>(b, warp - P::kValues, tok_first, ntiles, st, len);
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
        if (warp == P::kMma && lane == 0) {                          // products still in flight
            tc::mma_commit(drain);
            tc::mbar_wait_bounded(drain, 0, tc::kDrainNs);
        }
        __syncthreads();
    }
    tc::tc_fence_after();
    if (warp == P::kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
}

struct MergeArgs {
    const float *ws_o;
    const float2 *ws_ml;
    int Hkv, Hq, R, qshift, nrec;
};

// Log-sum-exp merge of the records of every query row, and of another part over other tokens.  A KV head has R * D / 4
// elements of 16 bytes in each of nrec records, row fastest or (ROWS) channels fastest; a CTA takes 32 of them, its 8 warps a share of
// the splits each (all loads of a warp in flight at once: the merge is a chain of latencies, not of bytes), joined
// through shared memory.  Row r of KV head h is query token r / qpk, head h * qpk + r % qpk.
template <int D, bool ROWS>
__global__ void __launch_bounds__(256) shared_merge_kernel(const MergeArgs a, const float *other_out,
                                                           const float *other_lse, float *out, float *lse) {
    constexpr int W = 8, BATCH = 5;
    __shared__ float4 s_acc[W][32];
    __shared__ float2 s_ml[W][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t per_head = (size_t)a.R * (D / 4);
    const size_t id = (size_t)blockIdx.x * 32 + lane;
    const bool live = id < per_head * a.Hkv;
    const int h = live ? (int)(id / per_head) : 0, e = live ? (int)(id % per_head) : 0;
    const int c4 = ROWS ? e % (D / 4) : e / a.R, r = ROWS ? e / (D / 4) : e % a.R;
    const int qpk = 1 << a.qshift;
    const size_t dst = (size_t)(r >> a.qshift) * a.Hq + h * qpk + (r & (qpk - 1));
    grid_wait();
    const float2 *ml = a.ws_ml + (size_t)h * a.R + r;
    const float4 *o = reinterpret_cast<const float4 *>(a.ws_o) + (size_t)h * per_head + e;
    const size_t step = (size_t)a.Hkv * a.R;                         // elements of the next record
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float mx = -CUDART_INF_F, sum = 0.f;
    if (live) {
        for (int i0 = warp; i0 < a.nrec; i0 += W * BATCH) {
            float2 x[BATCH];
            float4 y[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const size_t i = (size_t)min(i0 + k * W, a.nrec - 1) * step;
                x[k] = ml[i];
                y[k] = o[i * (D / 4)];
            }
            float top = mx;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (i0 + k * W >= a.nrec) x[k] = f2(-CUDART_INF_F, 0.f);
                top = fmaxf(top, x[k].x);
            }
            if (top == -CUDART_INF_F) continue;
            const float corr = ex2(mx - top);
            mx = top;
            sum *= corr;
            acc = make_float4(acc.x * corr, acc.y * corr, acc.z * corr, acc.w * corr);
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                if (x[k].x == -CUDART_INF_F) continue;               // a record without tokens has no O
                const float w = ex2(x[k].x - top);
                sum += w * x[k].y;
                acc.x += w * y[k].x;
                acc.y += w * y[k].y;
                acc.z += w * y[k].z;
                acc.w += w * y[k].w;
            }
        }
    }
    s_acc[warp][lane] = acc;
    s_ml[warp][lane] = f2(mx, sum);
    __syncthreads();
    if (warp != 0 || !live) return;
    const float ol = other_lse ? other_lse[dst] * 1.44269504088896340736f : -CUDART_INF_F;
    float top = ol;
#pragma unroll
    for (int k = 0; k < W; ++k) top = fmaxf(top, s_ml[k][lane].x);
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    if (top != -CUDART_INF_F) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float w = ex2(s_ml[k][lane].x - top);              // of no record: 0
            const float4 y = s_acc[k][lane];
            total += w * s_ml[k][lane].y;
            acc.x += w * y.x;
            acc.y += w * y.y;
            acc.z += w * y.z;
            acc.w += w * y.w;
        }
        const float wo = ex2(ol - top);
        if (wo > 0.f) {
            const float4 y = *reinterpret_cast<const float4 *>(other_out + dst * D + c4 * 4);
            total += wo;
            acc.x += wo * y.x;
            acc.y += wo * y.y;
            acc.z += wo * y.z;
            acc.w += wo * y.w;
        }
    }
    const float inv = total != 0.f ? 1.f / total : 0.f;              // no tokens at all: zeros
    *reinterpret_cast<float4 *>(out + dst * D + c4 * 4) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (lse != nullptr && c4 == 0)
        lse[dst] = total == 0.f ? -CUDART_INF_F : (top + log2f(total)) * 0.69314718055994530942f;
}

// Query rows of a KV head up to which tokens are the products' long side (shared_rows.cuh).
constexpr int kFewRows = 32, kFewRowsCoded = 16;

struct SharedPlan {
    bool few;                // shared_rows_kernel; else shared_attn_kernel with mb blocks of 128 rows
    bool direct;             // one CTA per KV head, which writes the result itself
    int mb, nsplit, nz, nrec;
};

// Splits: a CTA owns an SM (its tiles fill shared memory), so the splits that fill whole waves of 148 CTAs are
// compared by waves x (tiles per split + set-up), the set-up and drain of a CTA counted as two tiles.
SharedPlan plan_shared(int Hkv, int R, int max_len, bool coded) {
    SharedPlan p{};
    const int nt = coded ? 64 : 128;                                 // tokens per tile
    p.few = R <= (coded ? kFewRowsCoded : kFewRows);
    p.mb = R > 128 ? 2 : 1;
    p.nz = (R + p.mb * 128 - 1) / (p.mb * 128);
    const long units = (long)Hkv * p.nz, tiles = (max_len + nt - 1) / nt;
    long best = -1;
    p.nsplit = 1;
    for (int w = 1; w <= 4; ++w) {
        long ns = 148L * w / units;
        ns = ns < 1 ? 1 : ns > tiles ? (tiles > 0 ? tiles : 1) : ns;
        const long waves = (units * ns + 147) / 148;
        const long cost = waves * ((tiles + ns - 1) / ns + 2);
        if (best < 0 || cost < best) {
            best = cost;
            p.nsplit = (int)ns;
        }
    }
    // few tiles: a head on one CTA takes about as long as its tiles on several and the merge of their records, and has
    // one launch and no workspace
    p.direct = p.few && tiles <= kDirectTiles;
    p.nrec = p.direct ? 0 : p.few ? 2 * p.nsplit : p.nsplit;         // a CTA's two streams write a record each
    return p;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t ws_bytes(const SharedPlan &p, size_t RT, int D) {
    return p.nrec == 0 ? 0 : align256(p.nrec * RT * D * sizeof(float)) + p.nrec * RT * sizeof(float2);
}

// cuTensorMapEncodeTiled through the runtime: the library does not link the driver.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_tiled_fn(EncodeTiled *out) {
    static std::atomic<void *> fn{nullptr};
    void *p = fn.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult found;
        cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess || p == nullptr) return cudaErrorNotSupported;
        fn.store(p, std::memory_order_release);
    }
    *out = reinterpret_cast<EncodeTiled>(p);
    return cudaSuccess;
}

// Map of one sequence's rows [rows][D]: boxes of 128 tokens x 64 channels, rows of 128 bytes swizzled.
cudaError_t make_map(CUtensorMap *m, const uint16_t *p, size_t rows, int D, int nt) {
    EncodeTiled enc;
    cudaError_t e = encode_tiled_fn(&enc);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)nt}, es[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(p), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int MB, int C, bool PG>
cudaError_t launch_t(const SharedArgs &a, const SharedPlan &p, const CUtensorMap &km, const CUtensorMap &vm,
                     cudaStream_t s) {
    using PL = Plan<D, MB, C, PG>;
    auto kern = shared_attn_kernel<D, MB, C, PG>;
    cudaError_t e = ensure_dynamic_smem((const void *)kern, PL::kAlloc);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.nsplit, a.Hkv, p.nz), PL::kThreads, PL::kAlloc, s, a, km, vm);
}

template <int D, int NR, int C, bool PG, bool SCORES, bool DIRECT>
cudaError_t launch_rows_t(const RowsArgs &a, const CUtensorMap &km, const CUtensorMap &vm, cudaStream_t s) {
    using PL = RowsPlan<D, NR, C, PG>;
    auto kern = shared_rows_kernel<D, NR, C, PG, SCORES, DIRECT>;
    cudaError_t e = ensure_dynamic_smem((const void *)kern, PL::kAlloc);
    if (e != cudaSuccess) return e;
    const unsigned grid = DIRECT ? (unsigned)(a.seqs * a.Hkv) : a.nsplit > 0 ? (unsigned)(a.Hkv * a.nsplit) : kRowCtas;
    return launch_pdl(kern, dim3(grid), PL::kThreads, PL::kAlloc, s, a, km, vm);
}

RowsArgs rows_args(const SharedArgs &a, const SharedOther &o, float *out, float *lse) {
    RowsArgs r{};
    r.other_out = o.out;
    r.other_lse = o.lse;
    r.out = out;
    r.lse = lse;
    r.q = a.q;
    r.starts = a.start;
    r.lens = a.len;
    r.ws_o = a.ws_o;
    r.ws_ml = a.ws_ml;
    r.seqs = 1;
    r.Hkv = a.Hkv;
    r.Hq = a.Hq;
    r.R = a.R;
    r.qshift = a.qshift;
    r.max_len = a.max_len;
    r.nsplit = a.nsplit;
    r.sh = (size_t)a.R;
    r.ss = (size_t)a.Hkv * a.R;
    r.qscale = a.qscale;
    r.fault = a.fault;
    r.wait_ns = a.wait_ns;
    r.head_rows = a.head_rows;
    r.idx = a.idx;
    r.idx_head = a.idx_head;
    r.slk = a.slk;
    r.slv = a.slv;
    r.rope = a.rope;
    r.K = a.K;
    return r;
}

template <int D, int C, bool PG>
cudaError_t launch_p(const SharedArgs &a, const SharedPlan &p, const CUtensorMap &km, const CUtensorMap &vm,
                     const SharedOther &o, float *out, float *lse, cudaStream_t s) {
    if (p.few) {
        const RowsArgs r = rows_args(a, o, out, lse);
        if (a.R <= 16)
            return p.direct ? launch_rows_t<D, 16, C, PG, false, true>(r, km, vm, s)
                            : launch_rows_t<D, 16, C, PG, false, false>(r, km, vm, s);
        if constexpr (C == 0)
            return p.direct ? launch_rows_t<D, 32, C, PG, false, true>(r, km, vm, s)
                            : launch_rows_t<D, 32, C, PG, false, false>(r, km, vm, s);
    }
    return p.mb == 2 ? launch_t<D, 2, C, PG>(a, p, km, vm, s) : launch_t<D, 1, C, PG>(a, p, km, vm, s);
}

template <int C, bool PG>
cudaError_t launch_d(int D, const SharedArgs &a, const SharedPlan &p, const CUtensorMap &km, const CUtensorMap &vm,
                     const SharedOther &o, float *out, float *lse, cudaStream_t s) {
    if (D == 128) return launch_p<128, C, PG>(a, p, km, vm, o, out, lse, s);
    if (D == 64) return launch_p<64, C, PG>(a, p, km, vm, o, out, lse, s);
    return cudaErrorInvalidValue;
}

cudaError_t finish(const SharedArgs &a, const SharedPlan &p, int D, const SharedOther &o, float *out, float *lse,
                   cudaStream_t s) {
    const unsigned blocks = (unsigned)(((size_t)a.rows * a.Hq * (D / 4) + 31) / 32);
    const MergeArgs m{a.ws_o, a.ws_ml, a.Hkv, a.Hq, a.R, a.qshift, p.nrec};
    auto kern = D == 128 ? (p.few ? shared_merge_kernel<128, true> : shared_merge_kernel<128, false>)
                         : (p.few ? shared_merge_kernel<64, true> : shared_merge_kernel<64, false>);
    return launch_pdl(kern, dim3(blocks), 256, 0, s, m, o.out, o.lse, out, lse);
}

SharedArgs common_args(int rows, int Hkv, int Hq, int D, const SharedPlan &p, const uint16_t *q, const int32_t *start,
                       const int32_t *len, int max_len, float scale, void *workspace) {
    SharedArgs a{};
    a.q = q;
    a.start = start;
    a.len = len;
    a.rows = rows;
    a.Hkv = Hkv;
    a.Hq = Hq;
    a.qpk = Hq / Hkv;
    while ((1 << a.qshift) < a.qpk) ++a.qshift;
    a.R = rows * a.qpk;
    a.max_len = max_len;
    a.nsplit = p.nsplit;
    a.qscale = scale * 1.44269504088896340736f;
    a.ws_o = reinterpret_cast<float *>(workspace);
    a.ws_ml = reinterpret_cast<float2 *>(reinterpret_cast<char *>(workspace) +
                                         align256(p.nrec * (size_t)rows * Hq * D * sizeof(float)));
    a.wait_ns = wait_limit_ns();
    return a;
}

}  // namespace

// Decode attention of every sequence's one query token on the rows kernel, scores kept.  ws_o null: DIRECT, which also
// writes out, lse and the scores; else records of pieces (two streams of Hq / Hkv rows each) and scores in log2 units
// for the caller's merge.
cudaError_t launch_rows_scored(const loopvq_bf16_cache &c, const uint16_t *q, const int32_t *starts, const int32_t *lens,
                               int max_len, float qscale, const Bf16Scored &sc, float *out, float *lse, float *ws_o,
                               float2 *ws_ml, float *ws_s, int sstride, cudaStream_t s) {
    RowsArgs a{};
    a.q = q;
    a.starts = starts;
    a.lens = lens;
    a.ws_o = ws_o;
    a.ws_ml = ws_ml;
    a.ws_s = ws_s;
    a.sstride = sstride;
    a.seqs = c.B;
    a.Hkv = c.Hkv;
    a.Hq = c.Hq;
    a.R = c.Hq / c.Hkv;
    while ((1 << a.qshift) < a.R) ++a.qshift;
    a.max_len = max_len;
    a.ss = (size_t)a.R;
    a.qscale = qscale;
    a.wait_ns = wait_limit_ns();
    a.head_rows = c.Nmax;
    a.seq_rows = c.Hkv * c.Nmax;
    a.other_out = sc.other_out;
    a.other_lse = sc.other_lse;
    a.out = out;
    a.lse = lse;
    a.score_in = sc.score_in;
    a.score_out = sc.score_out;
    cudaError_t e = fault_word_for_current_device(&a.fault);
    if (e != cudaSuccess) return e;
    CUtensorMap km, vm;
    const size_t rows = (size_t)c.B * c.Hkv * c.Nmax;
    e = make_map(&km, c.k, rows, c.D, 128);
    if (e == cudaSuccess) e = make_map(&vm, c.v, rows, c.D, 128);
    if (e != cudaSuccess) return e;
    if (ws_o == nullptr)
        return c.D == 128 ? launch_rows_t<128, 16, 0, false, true, true>(a, km, vm, s)
                          : launch_rows_t<64, 16, 0, false, true, true>(a, km, vm, s);
    return c.D == 128 ? launch_rows_t<128, 16, 0, false, true, false>(a, km, vm, s)
                      : launch_rows_t<64, 16, 0, false, true, false>(a, km, vm, s);
}

size_t shared_ws_bytes(int Hkv, int Hq, int D, int rows, int max_len, bool coded) {
    return ws_bytes(plan_shared(Hkv, rows * (Hq / Hkv), max_len, coded), (size_t)rows * Hq, D);
}

cudaError_t launch_bf16_shared(const loopvq_bf16_cache &c, int seq, const uint16_t *q, int rows, const int32_t *starts,
                               const int32_t *lens, int max_len, float scale, const SharedOther &other, float *out,
                               float *lse, void *workspace, cudaStream_t s) {
    const SharedPlan p = plan_shared(c.Hkv, rows * (c.Hq / c.Hkv), max_len, false);
    SharedArgs a = common_args(rows, c.Hkv, c.Hq, c.D, p, q, starts ? starts + seq : nullptr, lens + seq, max_len, scale,
                               workspace);
    cudaError_t e = fault_word_for_current_device(&a.fault);
    if (e != cudaSuccess) return e;
    a.head_rows = c.Nmax;
    const size_t at = (size_t)seq * c.Hkv * c.Nmax * c.D, map_rows = (size_t)c.Hkv * c.Nmax;
    CUtensorMap km, vm;
    e = make_map(&km, c.k + at, map_rows, c.D, 128);
    if (e == cudaSuccess) e = make_map(&vm, c.v + at, map_rows, c.D, 128);
    if (e == cudaSuccess) e = launch_d<0, false>(c.D, a, p, km, vm, other, out, lse, s);
    if (e != cudaSuccess || p.direct) return e;
    return finish(a, p, c.D, other, out, lse, s);
}

cudaError_t launch_shared(const loopvq_cache &cc, int layer, int t, int seq, const uint16_t *q, int rows,
                          const int32_t *starts, const int32_t *lens, int max_len, float scale,
                          const SharedOther &other, float *out, float *lse, void *workspace, cudaStream_t s) {
    const SharedPlan p = plan_shared(cc.Hkv, rows * (cc.Hq / cc.Hkv), max_len, true);
    SharedArgs a = common_args(rows, cc.Hkv, cc.Hq, cc.D, p, q, starts ? starts + seq : nullptr, lens + seq, max_len,
                               scale, workspace);
    cudaError_t e = fault_word_for_current_device(&a.fault);
    if (e != cudaSuccess) return e;
    a.idx = cc.idx + idx_base(cc, layer, t / cc.Tc, seq, 0);
    a.idx_head = idx_words_per_bh(cc.Nmax, cc.D, cc.c);
    a.slk = cc.slices + slice_base(cc, layer, t, 0, 0);
    a.slv = cc.slices + slice_base(cc, layer, t, 1, 0);
    a.rope = cc.rope;
    a.K = cc.K;
    CUtensorMap none{};
    const bool pg = ncb_of(cc) > 1;
    switch (cc.c) {
        case 4: e = pg ? launch_d<4, true>(cc.D, a, p, none, none, other, out, lse, s) : launch_d<4, false>(cc.D, a, p, none, none, other, out, lse, s); break;
        case 8: e = pg ? launch_d<8, true>(cc.D, a, p, none, none, other, out, lse, s) : launch_d<8, false>(cc.D, a, p, none, none, other, out, lse, s); break;
        case 16: e = pg ? launch_d<16, true>(cc.D, a, p, none, none, other, out, lse, s) : launch_d<16, false>(cc.D, a, p, none, none, other, out, lse, s); break;
        case 32: e = pg ? launch_d<32, true>(cc.D, a, p, none, none, other, out, lse, s) : launch_d<32, false>(cc.D, a, p, none, none, other, out, lse, s); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess || p.direct) return e;
    return finish(a, p, cc.D, other, out, lse, s);
}

}  // namespace loopvq
