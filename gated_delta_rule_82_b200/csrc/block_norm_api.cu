// block_norm_api.cu -- the C ABI of the block norms: argument validation and dispatch (host only).
#include <math.h>

#include "block_norm.cuh"

using namespace ckda;

namespace {

struct Buf { const void* p; size_t n; };
bool overlap(const Buf& a, const Buf& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool group_ok(int W, int D) {
    return W == 0 || W == D || ((W == 16 || W == 32 || W == 64 || W == 128) && D % W == 0);
}

ckda_status check(const void* y, const void* gate, long long rows, int D, const ckda_norm_flags& f,
                  ckda_dtype dtype) {
    if (!y) return CKDA_ERR_NULL;
    if (dtype != CKDA_F32 && dtype != CKDA_BF16) return CKDA_ERR_UNSUPPORTED;
    if (rows < 1 || D < 1 || rows > (1ll << 40) / D) return CKDA_ERR_SHAPE;
    if (D > CKDA_BLOCK_NORM_MAX_D || !group_ok(f.post_group, D)) return CKDA_ERR_UNSUPPORTED;
    if (f.gate_act < 0 || f.gate_act > 2 || (f.gate_act != 0) != (gate != nullptr)) return CKDA_ERR_ARG;
    if (!(f.eps > 0.f) || !isfinite(f.eps) || !isfinite(f.res_scale)) return CKDA_ERR_ARG;
    return CKDA_OK;
}

BlockNormArgs make_args(const void* y, const void* gate, const void* residual,
                        const float* post_weight, const float* res_vector, const float* pre_weight,
                        void* h, void* n, long long rows, int D, const ckda_norm_flags& f) {
    BlockNormArgs a;
    a.y = y; a.gate = gate; a.x = residual;
    a.w_post = f.post_group ? post_weight : nullptr;
    a.w_pre = pre_weight; a.r = res_vector;
    a.h = h; a.n = n;
    a.rows = rows; a.D = D; a.W = f.post_group;
    a.act = f.gate_act;
    a.scale = f.res_scale; a.eps = f.eps;
    return a;
}

}  // namespace

extern "C" {

ckda_status ckda_block_norm(const void* y, const void* gate, const void* residual,
                            const float* post_weight, const float* res_vector,
                            const float* pre_weight, void* h, void* n, long long rows, int D,
                            ckda_norm_flags flags, ckda_dtype dtype, ckda_stream_t stream) {
    if (!h) return CKDA_ERR_NULL;
    const ckda_status st = check(y, gate, rows, D, flags, dtype);
    if (st != CKDA_OK) return st;
    for (const void* p : {y, gate, residual, (const void*)h, (const void*)n})
        if (!aligned(p, 16)) return CKDA_ERR_ALIGN;
    for (const float* p : {post_weight, res_vector, pre_weight})
        if (!aligned(p, 4)) return CKDA_ERR_ALIGN;
    const size_t nb = (size_t)rows * D * (dtype == CKDA_BF16 ? 2 : 4);
    // element by element in place is fine (a row is read before it is written); h is written
    // before n, so an array that both would touch is not
    const Buf rowsin[] = {{y, nb}, {gate, nb}, {residual, nb}};
    const Buf vecs[] = {{post_weight, (size_t)flags.post_group * 4}, {res_vector, (size_t)D * 4},
                        {pre_weight, (size_t)D * 4}};
    for (void* o : {h, n}) {
        for (const Buf& in : rowsin)
            if (o != in.p && overlap({o, nb}, in)) return CKDA_ERR_ARG;
        for (const Buf& in : vecs)
            if (overlap({o, nb}, in)) return CKDA_ERR_ARG;
    }
    if (overlap({h, nb}, {n, nb})) return CKDA_ERR_ARG;
    const cudaError_t e = launch_block_norm(
        make_args(y, gate, residual, post_weight, res_vector, pre_weight, h, n, rows, D, flags),
        dtype, (cudaStream_t)stream);
    return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

size_t ckda_block_norm_bwd_workspace_bytes(long long rows, int D, int post_group) {
    if (rows < 1 || D < 1 || D > CKDA_BLOCK_NORM_MAX_D || rows > (1ll << 40) / D ||
        !group_ok(post_group, D))
        return (size_t)-1;
    return block_norm_bwd_partial_floats(rows, D, post_group) * sizeof(float);
}

ckda_status ckda_block_norm_bwd(const void* y, const void* gate, const void* residual,
                                const float* post_weight, const float* res_vector,
                                const float* pre_weight, const void* dh, const void* dn, void* dy,
                                void* dgate, void* dresidual, float* dpost_weight,
                                float* dres_vector, float* dpre_weight, long long rows, int D,
                                ckda_norm_flags flags, ckda_dtype dtype, void* workspace,
                                size_t workspace_bytes, ckda_stream_t stream) {
    if (!dy || (!dh && !dn)) return CKDA_ERR_NULL;
    const ckda_status st = check(y, gate, rows, D, flags, dtype);
    if (st != CKDA_OK) return st;
    if (gate && !dgate) return CKDA_ERR_NULL;
    if (!gate && dgate) return CKDA_ERR_ARG;
    if (dpost_weight && !flags.post_group) return CKDA_ERR_ARG;
    if (dpre_weight && !dn) return CKDA_ERR_ARG;
    for (const void* p : {y, gate, residual, dh, dn, (const void*)dy, (const void*)dgate,
                          (const void*)dresidual, (const void*)workspace})
        if (!aligned(p, 16)) return CKDA_ERR_ALIGN;
    for (const float* p : {post_weight, res_vector, pre_weight, (const float*)dpost_weight,
                           (const float*)dres_vector, (const float*)dpre_weight})
        if (!aligned(p, 4)) return CKDA_ERR_ALIGN;
    const bool sums = dpost_weight || dres_vector || dpre_weight;
    const size_t need = sums ? ckda_block_norm_bwd_workspace_bytes(rows, D, flags.post_group) : 0;
    if (need && (!workspace || workspace_bytes < need)) return CKDA_ERR_WORKSPACE;
    const size_t nb = (size_t)rows * D * (dtype == CKDA_BF16 ? 2 : 4);
    const size_t wb = (size_t)flags.post_group * 4, db = (size_t)D * 4;
    const Buf rowsin[] = {{y, nb}, {gate, nb}, {residual, nb}, {dh, nb}, {dn, nb}};
    const Buf rowsout[] = {{dy, nb}, {dgate, nb}, {dresidual, nb}};
    const Buf vecsin[] = {{post_weight, wb}, {res_vector, db}, {pre_weight, db}};
    const Buf vecsout[] = {{dpost_weight, wb}, {dres_vector, db}, {dpre_weight, db},
                           {need ? workspace : nullptr, need}};
    for (const Buf& o : rowsout) {
        for (const Buf& in : rowsin)
            if (o.p != in.p && overlap(o, in)) return CKDA_ERR_ARG;
        for (const Buf& in : vecsin)
            if (overlap(o, in)) return CKDA_ERR_ARG;
        for (const Buf& o2 : rowsout)
            if (&o != &o2 && overlap(o, o2)) return CKDA_ERR_ARG;
        for (const Buf& o2 : vecsout)
            if (overlap(o, o2)) return CKDA_ERR_ARG;
    }
    for (const Buf& o : vecsout) {
        for (const Buf& in : rowsin)
            if (overlap(o, in)) return CKDA_ERR_ARG;
        for (const Buf& in : vecsin)
            if (overlap(o, in)) return CKDA_ERR_ARG;
        for (const Buf& o2 : vecsout)
            if (&o != &o2 && overlap(o, o2)) return CKDA_ERR_ARG;
    }
    BlockNormGrads g;
    g.dh = dh; g.dn = dn;
    g.dx = dresidual; g.dy = dy; g.dgate = dgate;
    g.dw_post = dpost_weight; g.dw_pre = dpre_weight; g.dr = dres_vector;
    g.partial = static_cast<float*>(workspace);
    const cudaError_t e = launch_block_norm_bwd(
        make_args(y, gate, residual, post_weight, res_vector, pre_weight, nullptr, nullptr, rows, D,
                  flags),
        g, dtype, (cudaStream_t)stream);
    return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
