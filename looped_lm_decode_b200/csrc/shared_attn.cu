// Shared-prefix attention: plans, launches over bf16 caches, the merge of the kernels' records, and the rows kernel's
// launch for the scored decode.  The kernels are in shared_rows.cuh (few query rows of a KV head) and shared_mma.cuh (any).
#include <atomic>

#include "shared_launch.cuh"

namespace loopvq {

namespace {

struct MergeArgs {
    const float *ws_o;
    const float2 *ws_ml;
    int Hkv, Hq, R, qshift, nrec;
};

// Log-sum-exp merge of the records of every query row, and of another part over other tokens.  A KV head has R * D / 4
// elements of 16 bytes in each of nrec records, row fastest or (ROWS) channels fastest; a CTA takes 32 of them, its 8
// warps a share of the splits each (all loads of a warp in flight at once: the merge is a chain of latencies, not of
// bytes), joined through shared memory.  Row r of KV head h is query token r / qpk, head h * qpk + r % qpk.
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
        if (wo != 0.f) {
            const float4 y = *reinterpret_cast<const float4 *>(other_out + dst * D + c4 * 4);
            total += wo;
            acc.x += wo * y.x;
            acc.y += wo * y.y;
            acc.z += wo * y.z;
            acc.w += wo * y.w;
        }
    }
    if (ol != ol) total = ol;                                        // passed over by fmaxf above
    const float inv = total != 0.f ? 1.f / total : 0.f;              // no tokens at all: zeros
    *reinterpret_cast<float4 *>(out + dst * D + c4 * 4) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (lse != nullptr && c4 == 0)
        lse[dst] = total == 0.f ? -CUDART_INF_F : (top + log2f(total)) * 0.69314718055994530942f;
}

// Query rows of a KV head up to which tokens are the products' long side (shared_rows.cuh).  On a bf16 cache that takes 47
// us where the other kernel takes 56 (32768 tokens, 16 heads, 8 rows); on a coded cache, which is bound by the
// rebuilding, 77 where the other takes 69, so there it only serves calls of one launch.
constexpr int kFewRows = 32, kFewRowsCoded = 16;

// Tiles up to which a CTA of the kernel with rows as M takes all tokens of its rows and writes the result itself: one launch
// and no records, but tile after tile.  Calls in a graph / made one by one, us, one launch against two, 64 queries, 16
// heads: bf16 3 tiles 12.3 / 12.5 against 11.0 / 16.1, 6 tiles 14.1 / 14.4 (P in two parts) against 11.4 / 16.4; coded 4
// tiles 14.9 / 15.0 against 13.7 / 16.7, 8 tiles 17.1 / 17.2 (two parts) against 14.3 / 16.7.  Records of many rows cost
// more than the tiles: 200 queries, 16 heads: bf16 4 tiles 15.4 against 17.0, 8 tiles 18.0 against 18.8; coded 8 tiles 22.1
// against 22.5.
constexpr int kDirectTilesM = 3, kDirectTilesCoded = 4, kManyRows = 2048;

// Tokens up to which such calls hold P and rebuilt keys in three bf16 parts.  Few tokens average little out: 52 coded
// tokens are off by 2.9e-6 with two parts, 5.8e-7 with three (3 bf16 tiles 12.3 us against 10.8, 4 coded ones 14.9 / 13.1).
constexpr int kFineTokens = 512;

// Tokens that a stream of the kernel with rows as M adds into one O before that moves to a sum in the workspace.  Values of
// one sign (1 + N(0, 0.1)) are off by, and 2000 queries, 16 heads, 32768 tokens take: 1024 tokens
// 3.8e-6, 689 us; 2048 7.9e-6, 656; 4096 1.9e-5, 639; never 2.2e-4, 620.  200 queries, whose CTAs have 3700 tokens: 1024
// 3.0e-6, 99.1 us; 2048 6.5e-6, 96.1; 4096 and never 1.55e-5, 90.2.
constexpr int kRunTokens = 4096;

// Splits: a CTA owns an SM (its tiles fill shared memory), so the splits that fill whole waves of 148 CTAs are
// compared by waves x (tiles per split + set-up), the set-up and drain of a CTA counted as two tiles.
SharedPlan plan_shared(int Hkv, int R, int max_len, bool coded) {
    SharedPlan p{};
    const int nt = coded ? 64 : 128;                                 // tokens per tile
    p.few = coded ? R <= kFewRowsCoded && max_len <= kDirectTiles * nt : R <= kFewRows;
    const long tiles = (max_len + nt - 1) / nt;
    // Few tiles: a head on one CTA, in one launch without a workspace, instead of its tiles on several and a merge: 1000
    // tokens, 3 queries, 16 heads 14 us against 19 where calls are made one by one (10 against 8 in a graph).
    p.direct = tiles <= (p.few || (long)Hkv * R >= kManyRows ? kDirectTiles : coded ? kDirectTilesCoded : kDirectTilesM);
    // More than 128 rows: two blocks on a CTA share its tiles, or are CTAs of their own with twice the tiles.  A coded tile
    // is rebuilt once for both (direct calls with SMs to spare rebuild it twice: 4 tiles, 200 queries, 16 heads 15.1 us
    // against 19.7, keys in two parts); a bf16 tile's second read is L2's, and pays off while a CTA has few tiles (us with two
    // blocks / one: 16347 tokens, 4 heads, 256 rows 24.1 / 23.9, 4096, 16 heads 30.6 / 28.7; 32768, 16 heads, 200 rows
    // 93.2 / 111.7).
    const bool share = coded ? !(p.direct && (long)Hkv * ((R + 127) / 128) <= 148) : tiles * Hkv * ((R + 255) / 256) >= 8 * 148;
    p.mb = R > 128 && share ? 2 : 1;
    p.nz = (R + p.mb * 128 - 1) / (p.mb * 128);
    const long units = (long)Hkv * p.nz;
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
    if (p.direct) p.nsplit = 1;
    if (!p.few && p.nsplit == 1) p.direct = true;                    // enough rows to fill the SMs: nothing to merge
    p.fine = !p.few && p.direct && p.mb == 1 && tiles * nt <= kFineTokens;
    p.nrec = p.direct ? 0 : p.few ? 2 * p.nsplit : p.nsplit;         // a CTA's two streams write a record each
    const long most = (tiles + p.nsplit - 1) / p.nsplit;             // tiles of a CTA; with one block of rows its streams share them
    p.run = !p.few && (p.mb == 2 ? most : (most + 1) / 2) > kRunTokens / nt ? kRunTokens / nt : 0;
    return p;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Records (O, then maxima and sums), then the sums of runs.
size_t record_bytes(const SharedPlan &p, size_t RT, int D) {
    return p.nrec == 0 ? 0 : align256(p.nrec * RT * D * sizeof(float)) + align256(p.nrec * RT * sizeof(float2));
}
size_t ws_bytes(const SharedPlan &p, int Hkv, size_t RT, int D) {
    return record_bytes(p, RT, D) + (p.run == 0 ? 0 : (size_t)p.nsplit * Hkv * p.nz * 2 * 128 * D * sizeof(float));
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

// Map of one sequence's rows [rows][D]: boxes of nt tokens x 64 channels, rows of 128 bytes swizzled.
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
    a.run = p.run > 0 ? p.run : INT32_MAX;
    a.ws_run = reinterpret_cast<float4 *>(reinterpret_cast<char *>(workspace) + record_bytes(p, (size_t)rows * Hq, D));
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
    return ws_bytes(plan_shared(Hkv, rows * (Hq / Hkv), max_len, coded), Hkv, (size_t)rows * Hq, D);
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
    const int nt = p.fine ? 64 : 128;                                // rows of a copy
    e = make_map(&km, c.k + at, map_rows, c.D, nt);
    if (e == cudaSuccess) e = make_map(&vm, c.v + at, map_rows, c.D, nt);
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
    const bool pg = ncb_of(cc) > 1;
    switch (cc.c) {
        case 4: e = launch_shared_c4(pg, cc.D, a, p, other, out, lse, s); break;
        case 8: e = launch_shared_c8(pg, cc.D, a, p, other, out, lse, s); break;
        case 16: e = launch_shared_c16(pg, cc.D, a, p, other, out, lse, s); break;
        case 32: e = launch_shared_c32(pg, cc.D, a, p, other, out, lse, s); break;
        default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess || p.direct) return e;
    return finish(a, p, cc.D, other, out, lse, s);
}

}  // namespace loopvq
