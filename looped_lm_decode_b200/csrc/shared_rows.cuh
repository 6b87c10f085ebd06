// Attention of few query rows over one sequence's tokens with the tokens along the tensor cores' long side.
//
// A tensor-core product has 128 rows (M) whether they are used or not, and its time goes with its columns (N).  For up
// to 32 query rows of a KV head the tokens are the rows and the queries the columns:
//   S^T [tokens x rows] = K Q^T,   O^T [channels x rows] = V^T P^T,
// so that a tile of 128 tokens costs products of 16 or 32 columns instead of 128, and the softmax of a tile is spread
// over 128 threads (thread = token = tensor-memory lane) instead of one thread per row.
//
// What differs from the kernel with rows as M:
//  - P^T is an operand from shared memory: every thread writes its token's row of 16 or 32 probabilities, each in three
//    bf16 parts (24 bits, all of an fp32 probability), side by side as columns.  The parts meet the same values in one
//    product and have accumulators of their own, added when the result is read: V is read once for all of them, and the
//    small parts are not cut to the large one's last place.
//  - A row's maximum would be a reduction over lanes.  Any reference is exact, and fp32 and bf16 have 8 exponent bits, so
//    the reference only has to keep exp2 in range: it is the score of a stream's first token (a first score of -inf or far
//    from 0: the lowest number) and moves, to the tile's maximum, only when some score passes it by 2^40, which the warps of
//    a stream agree on with one barrier vote per tile.
//  - Sums are kept per (thread, row) and added over the lanes at the end (a product of ones and P would give them too, at
//    8 more products a tile; every product takes 46 clocks or more, however few its columns).
//
// A CTA works through items (sequence, KV head, split) with its copies running ahead across them, so that a batch of
// ragged sequences keeps every SM's copies in flight.  Warps: 0-3 and 4-7 softmax of the two streams that take the tiles
// in turn; then two that issue the products, the copying one (bf16 cache: TMA; coded cache: eight warps that rebuild
// keys, two that rebuild values) and one that loads the queries.
//
// What bounds it: long bf16 prefixes the HBM (32768 tokens, 8 queries, 16 heads: 268 MB in 47 us with the merge, 5.7 TB/s,
// 87% of a copy; 16 ragged sequences of up to 16384 tokens with scores: 305 MB in 56 us and 8 us of merge), short ones the
// chain of a tile through copy, product, softmax and product (1000 tokens, 3 queries, 16 heads, one launch: 10.1 us).
#pragma once

#include <cfloat>

#include <cuda.h>

#include "shared_rebuild.cuh"

namespace loopvq {

struct RowsArgs {
    const uint16_t *q;               // [sequence][query token][Hq][D]
    const int32_t *starts, *lens;    // of the sequences (starts may be null)
    float *ws_o;                     // [record][D]
    float2 *ws_ml;                   // [record]: maximum reference (log2 units), sum
    float *ws_s;                     // scores in log2 units [sequence][Hq][sstride], or null
    int sstride;
    int seqs, Hkv, Hq, R, qshift;    // R = query rows per (sequence, KV head)
    int max_len;
    int nsplit;                      // one sequence: its tiles in nsplit equal shares per KV head.  0: the tiles of all
                                     // (KV head, sequence) segments end to end, in equal shares per CTA (RowTiles)
    // record of stream w of split x (or, with nsplit = 0, of piece x), row r: (2 * x + w) * ss + h * sh + r (sh = 0 then)
    size_t sh, ss;
    float qscale;                    // scale * log2(e)
    unsigned int *fault;
    unsigned long long wait_ns;
    int head_rows, seq_rows;         // bf16 cache: rows of the tensor maps per KV head and per sequence
    // written by the kernel itself where a CTA has all tokens of its rows (DIRECT)
    const float *other_out, *other_lse;
    float *out, *lse;                // lse may be null
    const float *score_in;           // [sequence][Hkv][head_rows], or null for zeros
    float *score_out;
    const uint32_t *idx;             // coded cache: as in SharedArgs
    size_t idx_head;
    const uint16_t *slk, *slv;
    const float *rope;
    int K;
};

// The tile space of a batch of ragged sequences: segment s = h * B + b holds the 128-token tiles of sequence b from its
// start; all segments lie end to end and CTA c of G = min(CTAs, T) takes tiles [c T / G, (c + 1) T / G), so that every
// CTA has the same work whatever the lengths, and the others none.  The part of segment s in CTA c is piece s + c (both
// only rise along the space, so no two pieces share a number), and the pieces of a segment are consecutive.
struct RowTiles {
    long long per_head, before;      // tiles of a KV head; those of the sequences before b
};
__device__ __forceinline__ int row_tiles(const int32_t *starts, const int32_t *lens, int max_len, int b) {
    const int len = min(max(word(lens + b), 0), max_len);
    const int st = starts ? min(max(word(starts + b), 0), len) : 0;
    return (len - st + 127) >> 7;
}
__device__ __forceinline__ RowTiles row_space(const int32_t *starts, const int32_t *lens, int max_len, int seqs, int lane,
                                              int b) {               // one warp
    RowTiles r{0, 0};
    for (int i = lane; i < seqs; i += 32) {
        const int t = row_tiles(starts, lens, max_len, i);
        r.per_head += t;
        r.before += i < b ? t : 0;
    }
    r.per_head = warp_sum64(r.per_head);
    r.before = warp_sum64(r.before);
    return r;
}

// NT tokens per tile; KP bf16 parts per key (three hold a rebuilt, rotated key's fp32 values whole: calls of one launch are
// bound by latency, and what a third part costs does not show); NR columns; three parts of P.
template <int D, int NR, int C, bool PG>
struct RowsPlan {
    static constexpr bool coded = C != 0;
    static constexpr int NT = coded ? 64 : 128;
    static constexpr int KP = coded ? 3 : 1;
    static constexpr int PARTS = 3;
    static constexpr int kPanel = NT * 128;
    static constexpr int kTile = (D / 64) * kPanel;
    static constexpr int kStage = (KP + 1) * kTile;
    static constexpr int kPart = NT * NR * 2;                        // one part of P
    static constexpr int kP = PARTS * kPart;                         // of one stream
    static constexpr int kQ = (D / 64) * NR * 128;
    static constexpr int NQ = coded ? 1 : 2;                         // buffers of queries
    static constexpr int ST = D == 64 ? 4 : !coded && NR == 16 ? 3 : 2;
    static constexpr int kTable = coded && !PG ? kTableBytes : 0;
    static constexpr int offStage = 0;
    static constexpr int offP = ST * kStage;
    static constexpr int offQ = offP + 2 * kP;
    static constexpr int offTable = offQ + NQ * kQ;
    static constexpr int offTurn = offTable + 2 * kTable;
    static constexpr int offRef = offTurn + (coded ? D * 4 : 0);     // per stream: references, their moves, maxima
    static constexpr int kRef = 6 * NR * 4 + 16;
    static constexpr int offZero = offRef + 2 * kRef;                // NR zeros
    static constexpr int offInfo = offZero + NR * 4;                 // this CTA's first piece
    static constexpr int offBar = offInfo + 32;
    static constexpr int kBars = 4 * ST + 2 * NQ + 7;
    static constexpr int offTmem = offBar + kBars * 8;
    static constexpr int kUsed = offTmem + 16;
    static constexpr int kAlloc = kUsed + 1024;
    [[maybe_unused]] static constexpr int kMma = coded ? 16 : 8, kCopy = 9, kRebuild = 8, kValues = 17, kQuery = coded ? 19 : 10,
                         kPv = coded ? kQuery : 11;
    static constexpr int kThreads = (kPv + 1) * 32;
    static constexpr int kCols = 256;                                // stream w: S at 32 w, O at 64 + 96 w
    static_assert(kAlloc <= 232448, "shared memory");
    static_assert(offStage % 1024 == 0 && offP % 1024 == 0 && offQ % 1024 == 0 && kP % 512 == 0, "swizzle atoms");
    static_assert(PARTS * NR <= 96, "tensor memory");
    static_assert(2 * kP >= NR * D * 4, "the streams' merge");
};

// The row of P^T of token n: 16-byte chunk c of NR columns, swizzled by rows of 32 (NR = 16) or 64 (NR = 32) bytes.
template <int NR>
__device__ __forceinline__ uint32_t p_chunk(int n, int c) {
    if constexpr (NR == 16) return (uint32_t)n * 32u + ((uint32_t)(c ^ ((n >> 2) & 1)) << 4);
    else return (uint32_t)n * 64u + ((uint32_t)(c ^ ((n >> 1) & 3)) << 4);
}

// Barrier over the 128 threads of a stream, with a vote.
__device__ __forceinline__ bool stream_any(int id, bool p) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r) : "r"((uint32_t)p), "r"(id) : "memory");
    return r != 0;
}
__device__ __forceinline__ void both_sync() { asm volatile("barrier.cta.sync 3, 256;" ::: "memory"); }
__device__ __forceinline__ void stream_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// fp32 bits as signed integers of the same order
__device__ __forceinline__ int ordered(float x) {
    const int i = __float_as_int(x);
    return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }

// Tiles up to which a CTA takes all tokens of its rows.
constexpr int kDirectTiles = 8;

// Tiles of a stream after which O moves from tensor memory into registers: the tensor cores cut what they add to 24 bits
// instead of rounding it, always toward zero, so a long run of additions drifts (32768 tokens, 16 heads: off by 2e-6
// without the moves and 6e-7 with them, in the same time).
constexpr int kFlush = 4;
static_assert(kDirectTiles / 2 <= kFlush, "direct calls keep O in tensor memory");

// SCORES: every attended token's scores are kept (NR = 16 only).
// DIRECT: grid = sequences x KV heads; a CTA has all tokens of its rows, merges its two streams and the other part, writes
// out and lse, and (SCORES) adds the weights of the tokens, whose scores stayed in registers: no records, no second launch.
template <int D, int NR, int C, bool PG, bool SCORES, bool DIRECT>
__global__ void __launch_bounds__(RowsPlan<D, NR, C, PG>::kThreads, 1)
    shared_rows_kernel(const RowsArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
    using P = RowsPlan<D, NR, C, PG>;
    constexpr bool coded = C != 0;
    static_assert(!coded || DIRECT, "over a coded cache only calls of one launch");
    constexpr int NT = P::NT, KP = P::KP, ST = P::ST, NQ = P::NQ, PARTS = P::PARTS, NPAN = D / 64;
    constexpr float kFar = 40.f;                                     // log2 units a score may pass the reference by
    constexpr float kExact = 16777216.f;                             // scores up to here are held to 2 log2 units

    extern __shared__ unsigned char smem_raw[];
    const uint32_t base = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (base - tc::smem_u32(smem_raw));
    const uint32_t sStage = base + P::offStage, bars = base + P::offBar;
    auto kfull = [&](int s) { return bars + 8u * s; };
    auto vfull = [&](int s) { return bars + 8u * (ST + s); };
    auto kempty = [&](int s) { return bars + 8u * (2 * ST + s); };
    auto vempty = [&](int s) { return bars + 8u * (3 * ST + s); };
    auto qfull = [&](int b) { return bars + 8u * (4 * ST + b); };
    auto qempty = [&](int b) { return bars + 8u * (4 * ST + NQ + b); };
    auto sfull = [&](int w) { return bars + 8u * (4 * ST + 2 * NQ + w); };
    auto pfull = [&](int w) { return bars + 8u * (4 * ST + 2 * NQ + 2 + w); };
    auto odone = [&](int w) { return bars + 8u * (4 * ST + 2 * NQ + 4 + w); };
    const uint32_t drain = bars + 8u * (4 * ST + 2 * NQ + 6);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + P::offTmem);
    volatile int *dead = reinterpret_cast<volatile int *>(smem + P::offTmem + 4);
    const int tid = threadIdx.x, lane = tid & 31, warp = tc::uniform_warp();

    grid_trigger();
    if (!coded && warp == P::kCopy && lane == 0) {
        tc::prefetch_map(&kmap);
        tc::prefetch_map(&vmap);
    }
    if (tid < NR) reinterpret_cast<float *>(smem + P::offZero)[tid] = 0.f;
    if (warp == P::kMma) {
        if (lane == 0) {
            for (int s = 0; s < ST; ++s) {
                tc::mbar_init(kfull(s), coded ? 8 : 1);
                tc::mbar_init(vfull(s), coded ? 2 : 1);
                tc::mbar_init(kempty(s), 1);
                tc::mbar_init(vempty(s), 1);
            }
            for (int b = 0; b < NQ; ++b) {
                tc::mbar_init(qfull(b), 1);
                tc::mbar_init(qempty(b), 1);
            }
            for (int w = 0; w < 2; ++w) {
                tc::mbar_init(sfull(w), 1);
                tc::mbar_init(pfull(w), 128);
                tc::mbar_init(odone(w), 1);
            }
            tc::mbar_init(drain, 2);
            *dead = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
    }
    grid_wait();
    if (warp == P::kMma) {                                           // behind the wait: a CTA that waits holds no tensor
                                                                     // memory that the kernel before could want
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(tmem_slot)),
                     "r"(P::kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if constexpr (coded) {                                           // an item's KV head is this CTA's: one item per CTA
        if constexpr (!PG) {
            const int h = blockIdx.x % a.Hkv;
            fill_tables<C>(smem + P::offTable, a.slk + (size_t)h * a.K * C, a.slv + (size_t)h * a.K * C, a.K, P::kThreads);
        }
        for (int i = tid; i < D; i += P::kThreads)                   // row 64 is there when a second tile is
            reinterpret_cast<float *>(smem + P::offTurn)[i] = a.max_len > 64 ? a.rope[(size_t)64 * D + i] : 0.f;
    }
    // ---- items of this CTA, the same walk in every role: one split, or the pieces of its share of the tile space
    struct Item {
        int b, h, st, len, tok_first, ntiles;
        size_t rec;                                                  // of stream 0, row 0
        long long left;                                              // tiles of the CTA from this item on
    };
    auto item_of = [&](int b, int h, long long skip, long long most) {
        Item x;
        x.b = b;
        x.h = h;
        x.len = min(max(word(a.lens + b), 0), a.max_len);
        x.st = a.starts ? min(max(word(a.starts + b), 0), x.len) : 0;
        const int tok0 = coded ? (x.st & ~3) : x.st;                 // index words come in tiles of 4 tokens
        const int tiles = x.len > x.st ? (x.len - tok0 + NT - 1) / NT : 0;
        x.tok_first = tok0 + (int)skip * NT;
        x.ntiles = (int)min((long long)tiles - skip, most);
        x.left = most;
        x.rec = (size_t)(h * a.seqs + b + (int)blockIdx.x) * 2 * a.ss;
        return x;
    };
    Item item0;
    if constexpr (DIRECT) {
        item0 = item_of(blockIdx.x / a.Hkv, blockIdx.x % a.Hkv, 0, INT32_MAX);
        item0.left = item0.ntiles;
    } else if (a.nsplit > 0) {
        const int split = blockIdx.x % a.nsplit, h = blockIdx.x / a.nsplit;
        item0 = item_of(0, h, 0, INT32_MAX);
        const long long tiles = item0.ntiles;
        const int t0 = (int)(split * tiles / a.nsplit);
        item0.ntiles = (int)((split + 1) * tiles / a.nsplit) - t0;
        item0.left = item0.ntiles;
        item0.tok_first += t0 * NT;
        item0.rec = (size_t)(2 * split) * a.ss + h * a.sh;
    } else if (warp == 0) {
        const RowTiles sp = row_space(a.starts, a.lens, a.max_len, a.seqs, lane, 0);
        const long long T = sp.per_head * a.Hkv, G = min((long long)gridDim.x, T);
        const bool any = blockIdx.x < G;
        const long long x0 = any ? cta_first_tile(blockIdx.x, T, G) : 0, x1 = any ? cta_first_tile(blockIdx.x + 1, T, G) : 0;
        long long *info = reinterpret_cast<long long *>(smem + P::offInfo);
        if (lane == 0) info[0] = x1 - x0;
        if (x0 < x1) {
            const long long h = x0 / sp.per_head, r = x0 - h * sp.per_head;
            long long carry = 0;
            for (int b0 = 0; b0 < a.seqs; b0 += 32) {                // the sequence that holds tile r of the head
                const long long t = b0 + lane < a.seqs ? row_tiles(a.starts, a.lens, a.max_len, b0 + lane) : 0;
                long long inc = t;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                inc += carry;
                const unsigned hit = __ballot_sync(0xffffffffu, inc > r);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        info[1] = (h << 32) | (long long)(b0 + lane);
                        info[2] = r - (inc - t);
                    }
                    break;
                }
                carry = __shfl_sync(0xffffffffu, inc, 31);
            }
        }
    }
    tc::fence_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!DIRECT && a.nsplit == 0) {
        const long long *info = reinterpret_cast<const long long *>(smem + P::offInfo);
        item0.ntiles = 0;
        item0.left = info[0];
        if (info[0] > 0) item0 = item_of((int)(info[1] & 0xffffffff), (int)(info[1] >> 32), info[2], info[0]);
    }
    // the next item with tiles; false behind the last
    auto advance = [&](Item &x) {
        const long long left = x.left - x.ntiles;
        if (DIRECT || left <= 0) return false;
        int b = x.b, h = x.h;
        do {
            if (++b == a.seqs) {
                b = 0;
                ++h;
            }
            x = item_of(b, h, 0, left);
        } while (x.ntiles == 0);
        return true;
    };

    if (warp < 8) {
        // ---- softmax of stream w: 128 threads, one token of a tile each
        if constexpr (coded) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int w = warp >> 2, wq = warp & 3, bar = 1 + w;
        // tile row and channel of this thread's lane: products of 64 rows use the first 16 lanes of every 32
        const int token = NT == 128 ? wq * 32 + lane : lane < 16 ? wq * 16 + lane : -1;
        const int chan = D == 128 ? wq * 32 + lane : lane < 16 ? wq * 16 + lane : -1;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t ts = lanes + w * 32, to = lanes + 64 + w * 96;
        const uint32_t sp = base + P::offP + w * P::kP;
        float *ref = reinterpret_cast<float *>(smem + P::offRef + w * P::kRef);   // a row's reference, negated
        float *corr = ref + NR;
        float *wmax = ref + 2 * NR;                                  // [4][NR]: a warp's maxima, later its sums
        volatile int *wok = reinterpret_cast<volatile int *>(ref + 6 * NR);
        // 16 rows of O from their three accumulators
        auto read_o = [](uint32_t at, int c, float (&v)[16]) {
            uint32_t o[16], y[16], z[16];
            tc::tmem_ld16(at + c, o);
            tc::tmem_ld16(at + NR + c, y);
            tc::tmem_ld16(at + 2 * NR + c, z);
            tc::tmem_wait_ld16(o);
            tc::tmem_wait_ld16(y);
            tc::tmem_wait_ld16(z);
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(o[k]) + (__uint_as_float(y[k]) + __uint_as_float(z[k]));
        };
        const int cols = (a.R + 15) & ~15;                           // columns in use (padding rows: zero queries)
        int g = 0;                                                   // tiles of this CTA so far
        bool ok = true;
        Item x = item0;
        for (bool more = DIRECT || a.nsplit > 0 || x.left > 0; more; more = advance(x)) {
            const size_t rec = x.rec + w * a.ss;
            float l[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) l[r] = 0.f;
            float osum[DIRECT ? 1 : NR] = {};                        // this channel's O of the tiles before the last move
            float kept[SCORES && DIRECT ? kDirectTiles / 2 : 1][8] = {};   // this token's scores in the stream's tiles
            int j = 0;                                               // tiles of this stream in the item
            bool far = false;                                        // some reference is past kExact (the stream's threads alike)
            for (int t = 0; ok && t < x.ntiles; ++t, ++g) {
                if ((g & 1) != w) continue;
                // S of this step; and P of the stream's step before is read, O written
                bool came = tc::mbar_wait_or_dead(sfull(w), (g >> 1) & 1, a.wait_ns, dead);
                if (g >= 2) came = came && tc::mbar_wait_or_dead(odone(w), ((g >> 1) - 1) & 1, a.wait_ns, dead);
                ok = __all_sync(0xffffffffu, came);
                tc::tc_fence_after();
                const int n = x.tok_first + t * NT + token;
                const bool in = token >= 0 && n >= x.st && n < x.len;
                if constexpr (!DIRECT) {
                    if (ok && j > 0 && j % kFlush == 0) {            // the next product starts O afresh
#pragma unroll
                        for (int c = 0; c < NR; c += 16) {
                            if (c < cols) {
                                float o[16];
                                read_o(to, c, o);
#pragma unroll
                                for (int k = 0; k < 16; ++k) osum[c + k] += o[k];
                            }
                        }
                    }
                }
                // 16 columns in the exponent's units relative to the reference
                float qs = a.qscale;
                const float *nref = ref;
                auto load = [&](int c, float (&v)[16]) {
                    uint32_t s[16];
                    tc::tmem_ld16(ts + c, s);
                    tc::tmem_wait_ld16(s);
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 nr = *reinterpret_cast<const float4 *>(nref + c + k);
                        v[k] = fmaf(__uint_as_float(s[k]), qs, nr.x);
                        v[k + 1] = fmaf(__uint_as_float(s[k + 1]), qs, nr.y);
                        v[k + 2] = fmaf(__uint_as_float(s[k + 2]), qs, nr.z);
                        v[k + 3] = fmaf(__uint_as_float(s[k + 3]), qs, nr.w);
                    }
                };
                if (j == 0) {
                    // an item's first tile: its first attended token gives the reference.  Where that is -inf, or far, the
                    // lowest number does, which any other score passes (and exp2 of -inf is 0 against it)
                    if (ok && wq == 0) {
#pragma unroll 1
                        for (int c = 0; c < cols; c += 16) {
                            uint32_t s[16];
                            tc::tmem_ld16(ts + c, s);
                            tc::tmem_wait_ld16(s);
                            if (token == max(x.st - (x.tok_first + t * NT), 0)) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) {
                                    const float v = __uint_as_float(s[k]) * a.qscale;
                                    ref[c + k] = fabsf(v) <= kExact ? -v : FLT_MAX;
                                }
                            }
                        }
                    }
                    stream_sync(bar);
                }
                float top = 0.f;
                if (ok) {
#pragma unroll
                    for (int c = 0; c < NR; c += 16) {
                        if (c < cols) {
                            float v[16];
                            load(c, v);
#pragma unroll
                            for (int k = 0; k < 16; ++k) top = fmaxf(top, v[k]);
                        }
                    }
                }
                if (stream_any(bar, !ok || far || (in && top > kFar))) {
                    // rare: move the references to the maxima of this tile, and what was summed with them.  Maxima of the scores
                    // themselves: relative to a reference far below they have lost their last places
                    if (lane == 0) wok[wq] = ok;
                    if (ok) {
#pragma unroll 1
                        for (int c = 0; c < cols; c += 16) {
                            uint32_t s[16];
                            tc::tmem_ld16(ts + c, s);
                            tc::tmem_wait_ld16(s);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const int m = __reduce_max_sync(0xffffffffu, ordered(in ? __uint_as_float(s[k]) * a.qscale : -FLT_MAX));
                                if (lane == 0) wmax[wq * NR + c + k] = unordered(m);
                            }
                        }
                    }
                    stream_sync(bar);
                    ok = wok[0] && wok[1] && wok[2] && wok[3];
                    if (!ok) break;                                  // every warp of the stream alike
                    const int r = tid % 128;
                    if (r < cols) {                                  // how far the row's reference rises
                        const float was = -ref[r];
                        const float now = fmaxf(was, fmaxf(fmaxf(wmax[r], wmax[NR + r]), fmaxf(wmax[2 * NR + r], wmax[3 * NR + r])));
                        corr[r] = ex2(was - now);
                        ref[r] = -now;
                    }
                    stream_sync(bar);
#pragma unroll
                    for (int r2 = 0; r2 < NR; ++r2)
                        if (r2 < cols) {
                            l[r2] *= corr[r2];
                            if constexpr (!DIRECT) osum[r2] *= corr[r2];
                        }
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < PARTS * NR; c += 16) {
                            uint32_t o[16];
                            tc::tmem_ld16(to + c, o);
                            tc::tmem_wait_ld16(o);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * corr[(c + k) % NR]);
                            tc::tmem_st16(to + c, o);
                        }
                        tc::tmem_wait_st();
                    }
                    // a reference that cannot hold fractions of its scores: the difference of two rounded numbers, which is 0
                    // at the maximum, takes the place of the scores, instead of an exact product less a rounded one
                    far = false;
                    for (int r2 = 0; r2 < cols; ++r2) far = far || (fabsf(ref[r2]) > kExact && ref[r2] != FLT_MAX);
                    if (far) {
#pragma unroll 1
                        for (int c = 0; c < cols; c += 16) {
                            uint32_t s[16];
                            tc::tmem_ld16(ts + c, s);
                            tc::tmem_wait_ld16(s);
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                s[k] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(s[k]), qs), ref[c + k]));
                            tc::tmem_st16(ts + c, s);
                        }
                        tc::tmem_wait_st();
                        qs = 1.f;
                        nref = reinterpret_cast<const float *>(smem + P::offZero);
                    }
                }
                if constexpr (SCORES) {
                    uint32_t s[16];
                    tc::tmem_ld16(ts, s);
                    tc::tmem_wait_ld16(s);
                    if (far) {                                       // they were replaced above
#pragma unroll
                        for (int k = 0; k < 8; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) - ref[k]);
                    }
                    if constexpr (DIRECT) {
#pragma unroll
                        for (int q = 0; q < kDirectTiles / 2; ++q)
                            if (j == q) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) kept[q][k] = __uint_as_float(s[k]) * qs;
                            }
                    } else {
                        float *sc = a.ws_s + ((size_t)x.b * a.Hq + x.h * a.R) * a.sstride + n;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (in && k < a.R) sc[(size_t)k * a.sstride] = __uint_as_float(s[k]) * qs;
                    }
                }
#pragma unroll
                for (int c = 0; c < NR; c += 16) {
                    if (c < cols) {
                        float v[16];
                        load(c, v);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t p1[4], p2[4], p3[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                float2 p = f2(ex2(v[half * 8 + 2 * k]), ex2(v[half * 8 + 2 * k + 1]));
                                if (!in) p = f2(0.f, 0.f);
                                l[c + half * 8 + 2 * k] += p.x;
                                l[c + half * 8 + 2 * k + 1] += p.y;
                                p1[k] = cvt_bf16x2(p.y, p.x);
                                const float2 d = f2(p.x - bf16lo(p1[k]), p.y - bf16hi(p1[k]));
                                p2[k] = cvt_bf16x2(d.y, d.x);
                                p3[k] = cvt_bf16x2(d.y - bf16hi(p2[k]), d.x - bf16lo(p2[k]));
                            }
                            if (token >= 0) {
                                const uint32_t at = sp + p_chunk<NR>(token, c / 8 + half);
                                sts128(at, make_uint4(p1[0], p1[1], p1[2], p1[3]));
                                sts128(at + P::kPart, make_uint4(p2[0], p2[1], p2[2], p2[3]));
                                sts128(at + 2 * P::kPart, make_uint4(p3[0], p3[1], p3[2], p3[3]));
                            }
                        }
                    }
                }
                tc::fence_async_smem();
                tc::tc_fence_before();
                tc::mbar_arrive(pfull(w));
                ++j;
            }
            if (ok && j > 0) {
                // the item's last step of this stream: g counts tiles of both
                const int last = (g - 1 - (((g - 1) & 1) != w)) >> 1;
                ok = __all_sync(0xffffffffu, tc::mbar_wait_or_dead(odone(w), last & 1, a.wait_ns, dead));
                tc::tc_fence_after();
            }
            // sums over the lanes, scattered so that lane r ends with row r; then the records: (reference, sum), and
            // channels in runs of 128 bytes
#pragma unroll
            for (int o = NR / 2; o >= 1; o >>= 1) {
#pragma unroll
                for (int r = 0; r < o; ++r) {
                    const bool up = (lane & o) != 0;
                    const float keep = up ? l[o + r] : l[r], give = up ? l[r] : l[o + r];
                    l[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
            }
            if constexpr (NR == 16) l[0] += __shfl_xor_sync(0xffffffffu, l[0], 16);
            if (lane < NR) wmax[wq * NR + lane] = l[0];
            if (lane == 0) wok[wq] = ok;
            stream_sync(bar);
            const bool all_ok = wok[0] && wok[1] && wok[2] && wok[3];
            if constexpr (DIRECT) {
                // ---- merge of the streams: stream 1 hands its part over through the memory of both P, which every
                // product has read by now
                float *part = reinterpret_cast<float *>(smem + P::offP);           // [NR][D]
                const float *ref1 = reinterpret_cast<const float *>(smem + P::offRef + P::kRef);
                float *coef = reinterpret_cast<float *>(smem + P::offRef) + 2 * NR;  // c0, c1, other's; joint log2-sum-exp2
                if (tid % 128 < a.R) {
                    const int r = tid % 128;
                    const float sum = wmax[r] + wmax[NR + r] + wmax[2 * NR + r] + wmax[3 * NR + r];
                    corr[r] = !all_ok ? CUDART_NAN_F : j > 0 ? sum : 0.f;
                }
                both_sync();
                if (w == 1 && j > 0) {
#pragma unroll 1
                    for (int c = 0; c < cols; c += 16) {
                        float o[16];
                        read_o(to, c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (chan >= 0 && c + k < a.R) part[(c + k) * D + chan] = o[k];
                    }
                }
                auto dst = [&](int r) {
                    return (size_t)(x.b * (a.R >> a.qshift) + (r >> a.qshift)) * a.Hq + (x.h << a.qshift) +
                           (r & ((1 << a.qshift) - 1));
                };
                if (w == 0 && tid < a.R) {
                    const int r = tid;
                    const float s0 = corr[r], s1 = ref1[NR + r];
                    const float m0 = s0 != 0.f ? -ref[r] : -CUDART_INF_F, m1 = s1 != 0.f ? -ref1[r] : -CUDART_INF_F;
                    const float ol = a.other_lse ? a.other_lse[dst(r)] * 1.44269504088896340736f : -CUDART_INF_F;
                    const float top = fmaxf(fmaxf(m0, m1), ol);
                    float c0 = 0.f, c1 = 0.f, co = 0.f, l2 = -CUDART_INF_F;
                    if (top != -CUDART_INF_F) {
                        c0 = ex2(m0 - top);
                        c1 = ex2(m1 - top);
                        co = ex2(ol - top);
                        const float total = s0 * c0 + s1 * c1 + co;
                        l2 = top + log2f(total);
                        c0 /= total;
                        c1 /= total;
                        co /= total;
                    }
                    if (s0 + s1 != s0 + s1 || ol != ol) c0 = c1 = co = l2 = CUDART_NAN_F;   // a stream gave up, or NaN inputs
                    coef[r] = c0;
                    coef[NR + r] = c1;
                    coef[2 * NR + r] = co;
                    coef[3 * NR + r] = l2;
                    if (a.lse != nullptr)
                        a.lse[dst(r)] = l2 == -CUDART_INF_F ? -CUDART_INF_F : l2 * 0.69314718055994530942f;
                }
                both_sync();
                if (w == 0) {
#pragma unroll 1
                    for (int c = 0; c < cols; c += 16) {
                        float o[16];
                        if (j > 0) read_o(to, c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int r = c + k;
                            if (chan >= 0 && r < a.R) {
                                float v = j > 0 ? o[k] * coef[r] : 0.f;
                                if (coef[NR + r] != 0.f) v += part[r * D + chan] * coef[NR + r];
                                if (coef[2 * NR + r] > 0.f) v += a.other_out[dst(r) * D + chan] * coef[2 * NR + r];
                                if (coef[r] != coef[r]) v = coef[r];
                                a.out[dst(r) * D + chan] = v;
                            }
                        }
                    }
                }
                if constexpr (SCORES) {
                    const size_t row = ((size_t)x.b * a.Hkv + x.h) * a.head_rows;
                    float l2[8];                                     // a head without weight gives none: exp2(-inf - inf)
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        l2[k] = coef[3 * NR + k];
                        if (l2[k] == -CUDART_INF_F) l2[k] = CUDART_INF_F;
                    }
#pragma unroll
                    for (int q = 0; q < kDirectTiles / 2; ++q) {
                        const int n = x.tok_first + (2 * q + w) * NT + token;
                        if (q < j && n < x.len) {
                            float sum = 0.f;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (k < a.R) sum += ex2(kept[q][k] - l2[k]);
                            a.score_out[row + n] = (a.score_in ? a.score_in[row + n] : 0.f) + sum;
                        }
                    }
                }
            } else {
                if (tid % 128 < a.R) {
                    const int r = tid % 128;
                    const float sum = wmax[r] + wmax[NR + r] + wmax[2 * NR + r] + wmax[3 * NR + r];
                    // (a row whose every score is -inf has no weight)
                    a.ws_ml[rec + r] = !all_ok             ? f2(0.f, CUDART_NAN_F)
                                       : j > 0 && sum != 0.f ? f2(-ref[r], sum)
                                                           : f2(-CUDART_INF_F, 0.f);
                }
                if (all_ok && j > 0) {
#pragma unroll
                    for (int c = 0; c < NR; c += 16) {
                        if (c < cols) {
                            float o[16];
                            read_o(to, c, o);
                            float *dst = a.ws_o + (rec + c) * D + chan;
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                if (chan >= 0 && c + k < a.R) dst[k * D] = o[k] + osum[c + k];
                        }
                    }
                }
            }
            tc::tc_fence_before();
            stream_sync(bar);                                        // the next item writes ref again
            ok = all_ok;
            if (!DIRECT && !ok) {                                    // the records of the items left: NaN
                while (advance(x))
                    if (tid % 128 < a.R) a.ws_ml[x.rec + w * a.ss + tid % 128] = f2(0.f, CUDART_NAN_F);
                break;
            }
        }
    } else if (warp == P::kMma) {
        // ---- S^T = K Q^T.  The two kinds of products have a warp each: a product takes 46 clocks and more to issue, and
        // one that waits for its copy must not hold up another whose tile, once read, makes room for the next
        constexpr uint32_t id_qk = tc::idesc_bf16(NT, NR), hi = tc::desc_hi(1024, 2);
        Item x = item0;
        int it = 0, t = 0;                                           // the item's number, its tile
        for (long long g64 = 0, total = item0.left; g64 < total; ++g64) {
            const int g = (int)g64, sg = g % ST, w = g & 1;
            bool came = t > 0 || tc::mbar_wait_or_dead(qfull(it % NQ), (it / NQ) & 1, a.wait_ns, dead);
            came = came && tc::mbar_wait_or_dead(kfull(sg), (g / ST) & 1, a.wait_ns, dead);
            if (g >= 2) came = came && tc::mbar_wait_or_dead(pfull(w), ((g >> 1) - 1) & 1, a.wait_ns, dead);   // S is read
            if (!__all_sync(0xffffffffu, came)) break;
            tc::tc_fence_after();
            const bool last = t + 1 == x.ntiles;
            const uint32_t k_lo = tc::uniform(tc::desc_lo(sStage + sg * P::kStage, 16));
            const uint32_t q_lo = tc::uniform(tc::desc_lo(base + P::offQ + (it % NQ) * P::kQ, 16));
            const uint32_t sd = tc::uniform(tmem + w * 32);
            if (tc::elect_one()) {
#pragma unroll
                for (int part = 0; part < KP; ++part)
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)                 // 16 channels per product: 32 bytes of a row
                        tc::mma_ss(sd, k_lo + (part * P::kTile + (k / 4) * P::kPanel + (k % 4) * 32) / 16, hi,
                                   q_lo + ((k / 4) * (NR * 128) + (k % 4) * 32) / 16, hi, id_qk, part + k > 0);
                tc::mma_commit(sfull(w));
                if (g + ST < total) tc::mma_commit(kempty(sg));      // what will not be used again is not freed
                if (last && g + 1 < total) tc::mma_commit(qempty(it % NQ));
            }
            __syncwarp();
            ++t;
            if (last && advance(x)) {
                t = 0;
                ++it;
            }
        }
    } else if (warp == P::kQuery || warp == P::kPv) {
        if (warp == P::kQuery) {
            // ---- queries: NR rows (those past R zero), swizzled rows of 64 channels
            int it = 0;
            Item x = item0;
            for (bool more = x.left > 0; more; more = advance(x)) {
                if (it >= NQ &&
                    !__all_sync(0xffffffffu, tc::mbar_wait_or_dead(qempty(it % NQ), (it / NQ - 1) & 1, a.wait_ns, dead)))
                    break;
                const uint32_t qb = base + P::offQ + (it % NQ) * P::kQ;
                const int tokens = a.R >> a.qshift, qpk = 1 << a.qshift;
                for (int e = lane; e < NR * (D / 8); e += 32) {
                    const int r = e / (D / 8), ch = e % (D / 8);
                    const bool real = r < a.R;
                    const uint16_t *src =
                        a.q + (((size_t)x.b * tokens + (r >> a.qshift)) * a.Hq + x.h * qpk + (r & (qpk - 1))) * D + ch * 8;
                    cp_async16_zfill(qb + (ch / 8) * (NR * 128) + sw128(r, ch % 8), real ? src : a.q, real);
                }
                cp_async_commit();
                cp_async_wait<0>();
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(qfull(it % NQ));
                ++it;
            }
        }
        if (warp == P::kPv) {
            // ---- O^T += V^T P^T
            constexpr uint32_t id_pv = tc::idesc_bf16(D, PARTS * NR) | (1u << 15) | (1u << 16);   // both: contraction outside
            Item x = item0;
            int t = 0;
            for (long long g64 = 0, total = item0.left; g64 < total; ++g64) {
                const int g = (int)g64, sg = g % ST, w = g & 1;
                const uint32_t vb = sStage + sg * P::kStage + KP * P::kTile;
                bool came = tc::mbar_wait_or_dead(vfull(sg), (g / ST) & 1, a.wait_ns, dead);
                if constexpr (!coded) {
                    // rows behind the last token may hold anything: 0 x that has to be 0
                    const int end = x.len - (x.tok_first + t * NT);
                    if (end < NT && __all_sync(0xffffffffu, came)) {
                        for (int it = lane; it < (NT - end) * (D / 8); it += 32) {
                            const int n = end + it / (D / 8), ch = it % (D / 8);
                            sts128(vb + (ch / 8) * P::kPanel + n * 128 + (ch % 8) * 16, make_uint4(0, 0, 0, 0));
                        }
                        tc::fence_async_smem();
                        __syncwarp();
                    }
                }
                came = came && tc::mbar_wait_or_dead(pfull(w), (g >> 1) & 1, a.wait_ns, dead);
                if (!__all_sync(0xffffffffu, came)) break;
                tc::tc_fence_after();
                const uint32_t p_lo = tc::uniform(tc::desc_lo(base + P::offP + w * P::kP, P::kPart));
                const uint32_t v_lo = tc::uniform(tc::desc_lo(vb, P::kPanel)), od = tc::uniform(tmem + 64 + w * 96);
                const uint32_t more = tc::uniform((t >> 1) % kFlush != 0);   // else O of this stream holds nothing to keep
                if (tc::elect_one()) {
#pragma unroll
                    for (int k = 0; k < NT / 16; ++k)                    // 16 tokens per product
                        tc::mma_ss(od, v_lo + k * 128, tc::desc_hi(1024, 2), p_lo + k * (2 * NR),
                                   tc::desc_hi(8 * NR * 2, NR == 16 ? 6 : 4), id_pv, k > 0 ? 1u : more);
                    tc::mma_commit(odone(w));
                    if (g + ST < total) tc::mma_commit(vempty(sg));
                }
                __syncwarp();
                if (++t == x.ntiles && advance(x)) t = 0;
            }
        }
    } else if constexpr (!coded) {
        // ---- copies
        if (lane == 0) {
            int g = 0;
            bool ok = true;
            Item x = item0;
            for (bool more = x.left > 0; ok && more; more = advance(x)) {
                const int y = x.b * a.seq_rows + x.h * a.head_rows + x.tok_first;
                for (int t = 0; t < x.ntiles; ++t, ++g) {
                    const int sg = g % ST;
                    const uint32_t kb = sStage + sg * P::kStage, vb = kb + KP * P::kTile;
                    if (g >= ST && !(ok = tc::mbar_wait_or_dead(kempty(sg), (g / ST - 1) & 1, a.wait_ns, dead))) break;
                    tc::mbar_expect_tx(kfull(sg), P::kTile);
#pragma unroll
                    for (int c = 0; c < NPAN; ++c) tc::tma_load_2d(kb + c * P::kPanel, &kmap, c * 64, y + t * NT, kfull(sg));
                    if (g >= ST) ok = tc::mbar_wait_or_dead(vempty(sg), (g / ST - 1) & 1, a.wait_ns, dead);
                    tc::mbar_expect_tx(vfull(sg), P::kTile);         // also when giving up: the drain waits for both
#pragma unroll
                    for (int c = 0; c < NPAN; ++c) tc::tma_load_2d(vb + c * P::kPanel, &vmap, c * 64, y + t * NT, vfull(sg));
                    if (!ok) {
                        ++g;
                        break;
                    }
                }
            }
            *reinterpret_cast<volatile int *>(smem + P::offTmem + 8) = g;          // tiles copied, for the drain
        }
    } else {
        // ---- rebuilding
        RebuildArgs b;
        b.idx = a.idx + (size_t)item0.h * a.idx_head;
        b.slk = a.slk + (size_t)item0.h * a.K * (PG ? D : C);
        b.slv = a.slv + (size_t)item0.h * a.K * (PG ? D : C);
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
            rebuild_keys<D, C, PG, ST, KP>(b, warp - P::kRebuild, item0.tok_first, item0.ntiles, item0.st, item0.len);
        } else {
            rebuild_values<D, C, PG, ST, KP>(b, warp - P::kValues, item0.tok_first, item0.ntiles, item0.st, item0.len);
        }
    }

    // ---- all done (or given up): free the tensor memory
    __syncthreads();
    if (*dead) {
        if (tid == 0) atomicOr(a.fault, kFaultAttnWait);
        if (!coded && warp == P::kCopy && lane == 0) {               // copies still in flight
            const int n = *reinterpret_cast<volatile int *>(smem + P::offTmem + 8);
            for (int t = n > ST ? n - ST : 0; t < n; ++t) {
                tc::mbar_wait_bounded(kfull(t % ST), (t / ST) & 1, tc::kDrainNs);
                tc::mbar_wait_bounded(vfull(t % ST), (t / ST) & 1, tc::kDrainNs);
            }
        }
        if ((warp == P::kMma || warp == P::kPv) && tc::elect_one()) {   // products still in flight, of the threads that issued them
            tc::mma_commit(drain);
            tc::mbar_wait_bounded(drain, 0, tc::kDrainNs);
        }
        __syncthreads();
    }
    tc::tc_fence_after();
    if (warp == P::kMma)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P::kCols));
}

}  // namespace loopvq
