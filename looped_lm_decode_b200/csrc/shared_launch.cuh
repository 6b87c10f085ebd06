// Launches of the shared-prefix attention kernels for the instantiating units: shared_attn.cu (bf16 caches) and
// shared_coded_c*.cu (coded caches, one unit per channels per code, so that they compile side by side).
#pragma once

#include "shared_mma.cuh"

namespace loopvq {

struct SharedPlan {
    bool few;                // shared_rows_kernel; else shared_attn_kernel with mb blocks of 128 rows
    bool direct;             // one CTA per KV head (and block of rows), which writes the result itself
    bool fine;               // shared_attn_kernel with P and rebuilt keys in three bf16 parts, tiles of 64 tokens
    int mb, nsplit, nz, nrec;
    int run;                 // tiles of a stream after which its O leaves tensor memory; 0: never
};

template <int D, int MB, int C, bool PG, bool FINE, bool RUNS>
inline cudaError_t launch_t(const SharedArgs &a, const SharedPlan &p, const CUtensorMap &km, const CUtensorMap &vm,
                     cudaStream_t s) {
    using PL = Plan<D, MB, C, PG, FINE>;
    auto kern = shared_attn_kernel<D, MB, C, PG, FINE, RUNS>;
    cudaError_t e = ensure_dynamic_smem((const void *)kern, PL::kAlloc);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(p.nsplit, a.Hkv, p.nz), PL::kThreads, PL::kAlloc, s, a, km, vm);
}

template <int D, int NR, int C, bool PG, bool SCORES, bool DIRECT>
inline cudaError_t launch_rows_t(const RowsArgs &a, const CUtensorMap &km, const CUtensorMap &vm, cudaStream_t s) {
    using PL = RowsPlan<D, NR, C, PG>;
    auto kern = shared_rows_kernel<D, NR, C, PG, SCORES, DIRECT>;
    cudaError_t e = ensure_dynamic_smem((const void *)kern, PL::kAlloc);
    if (e != cudaSuccess) return e;
    const unsigned grid = DIRECT ? (unsigned)(a.seqs * a.Hkv) : a.nsplit > 0 ? (unsigned)(a.Hkv * a.nsplit) : kRowCtas;
    return launch_pdl(kern, dim3(grid), PL::kThreads, PL::kAlloc, s, a, km, vm);
}

inline RowsArgs rows_args(const SharedArgs &a, const SharedOther &o, float *out, float *lse) {
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
inline cudaError_t launch_p(const SharedArgs &a, const SharedPlan &p, const CUtensorMap &km, const CUtensorMap &vm,
                     const SharedOther &o, float *out, float *lse, cudaStream_t s) {
    if (p.few) {
        const RowsArgs r = rows_args(a, o, out, lse);
        if constexpr (C != 0)
            return launch_rows_t<D, 16, C, PG, false, true>(r, km, vm, s);
        else if (a.R <= 16)
            return p.direct ? launch_rows_t<D, 16, C, PG, false, true>(r, km, vm, s)
                            : launch_rows_t<D, 16, C, PG, false, false>(r, km, vm, s);
        else
            return p.direct ? launch_rows_t<D, 32, C, PG, false, true>(r, km, vm, s)
                            : launch_rows_t<D, 32, C, PG, false, false>(r, km, vm, s);
    }
    SharedArgs x = a;
    if (p.direct) {
        x.other_out = o.out;
        x.other_lse = o.lse;
        x.out = out;
        x.lse = lse;
    }
    if (p.fine) return launch_t<D, 1, C, PG, true, false>(x, p, km, vm, s);
    if (p.run > 0)
        return p.mb == 2 ? launch_t<D, 2, C, PG, false, true>(x, p, km, vm, s) : launch_t<D, 1, C, PG, false, true>(x, p, km, vm, s);
    return p.mb == 2 ? launch_t<D, 2, C, PG, false, false>(x, p, km, vm, s) : launch_t<D, 1, C, PG, false, false>(x, p, km, vm, s);
}

template <int C, bool PG>
inline cudaError_t launch_d(int D, const SharedArgs &a, const SharedPlan &p, const CUtensorMap &km, const CUtensorMap &vm,
                     const SharedOther &o, float *out, float *lse, cudaStream_t s) {
    if (D == 128) return launch_p<128, C, PG>(a, p, km, vm, o, out, lse, s);
    if (D == 64) return launch_p<64, C, PG>(a, p, km, vm, o, out, lse, s);
    return cudaErrorInvalidValue;
}

// The coded caches' units: per_group: one codebook per channel group.
#define LQ_DECLARE_CODED(C)                                                                                          \
    cudaError_t launch_shared_c##C(bool per_group, int D, const SharedArgs &a, const SharedPlan &p, const SharedOther &o, \
                                   float *out, float *lse, cudaStream_t s)
LQ_DECLARE_CODED(4);
LQ_DECLARE_CODED(8);
LQ_DECLARE_CODED(16);
LQ_DECLARE_CODED(32);
#define LQ_DEFINE_CODED(C)                                                                                           \
    LQ_DECLARE_CODED(C) {                                                                                            \
        const CUtensorMap none{};                                                                                    \
        return per_group ? launch_d<C, true>(D, a, p, none, none, o, out, lse, s)                                    \
                         : launch_d<C, false>(D, a, p, none, none, o, out, lse, s);                                  \
    }

}  // namespace loopvq
