// linattn_api.cu -- the C ABI of the decayed linear attention: argument validation and dispatch.
// Everything here runs on the host before any launch; nothing is allocated.
#include <math.h>

#include "linattn.cuh"

using namespace ckda;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool supported_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
size_t elem_size(ckda_dtype t) { return t == CKDA_BF16 ? 2 : 4; }
ckda_status from_cuda(cudaError_t e) { return e == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA; }

struct Buf { const void* p; size_t n; };
bool overlap(const Buf& a, const Buf& b) {
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.n && y < x + a.n;
}

// The token axis: B rows of T tokens, or n packed sequences.
struct Tokens {
    int n, T;              // sequences; tokens of a row (batched) or of the axis (packed)
    long long total, longest;
    int empty;             // a packed sequence has no tokens
};
ckda_status read_tokens(int B, int T, const int* cu_host, int n_seqs, int H, Tokens* t) {
    if (!cu_host) {
        if (B < 1 || T < 1 || H < 1) return CKDA_ERR_SHAPE;
        *t = Tokens{B, T, (long long)B * T, T, 0};
    } else {
        if (n_seqs < 1 || H < 1) return CKDA_ERR_SHAPE;
        if (cu_host[0] != 0) return CKDA_ERR_ARG;
        long long longest = 0;
        int empty = 0;
        for (int s = 0; s < n_seqs; ++s) {
            const long long len = (long long)cu_host[s + 1] - cu_host[s];
            if (len < 0) return CKDA_ERR_ARG;
            longest = len > longest ? len : longest;
            empty |= len == 0;
        }
        *t = Tokens{n_seqs, cu_host[n_seqs], (long long)cu_host[n_seqs], longest, empty};
    }
    // (grid sizes and chunk numbers stay below 2^31, byte counts below 2^48)
    if (t->longest > 0x7fffff00ll) return CKDA_ERR_SHAPE;   // (rounded up to whole chunks below 2^31)
    if ((t->total / kLaChunk + 2ll * t->n + 1) * H > 0x7fffffll * 16) return CKDA_ERR_SHAPE;
    if (t->total > (1ll << 40) / 128 / H) return CKDA_ERR_SHAPE;
    return CKDA_OK;
}

// Units that run side by side.  On tcgen05 (bf16, 128 x 128) a CTA fills an SM; in the backward its
// longest launch holds two runs (16 heads, 2 x 2048 tokens, caches flushed: 158 us, with 100 units 182,
// with 148 156; 2 x 1000 tokens: 94, 113, 100).
// The warp tiles take a warp for 16 output channels: several narrow heads fit an SM, and a unit
// leaves its SM waiting for longer than it takes to start another (4096 x 16 heads of 64 x 64:
// forward 97 us with 148 units, 58 with 296; backward 405 with 74, 224 with 148, 192 with 296; fp32
// backward of 128 x 128 806 with 74, 680 with 148).  All of these are square heads; for others the wider
// side counts, which leaves SMs idle where the output is the narrow one (128 x 16: a warp a CTA).
int unit_slots(int dk, int dv, ckda_dtype dtype, bool backward) {
    if (dtype == CKDA_BF16 && dk == 128 && dv == 128) return backward ? 74 : 148;
    return 148 * (128 / (dk > dv ? dk : dv));
}

LaSplit make_split(const Tokens& t, const int* cu, const int* cu_host, int H, int slots) {
    LaSplit sp;
    sp.cu = cu;
    sp.n = t.n;
    sp.T = t.T;
    sp.H = H;
    sp.empty = t.empty;
    sp.L = la_unit_len(t.total, t.longest, H, slots);
    sp.units = (int)la_units(cu_host, t.n, t.T, sp.L);
    return sp;
}

ckda_status check_flags(const ckda_flags& f, int H, int* G) {
    // the rotation, the norm and gate logits belong to the CKDA recurrence and its prologue
    if (f.l2norm || f.rope_theta > 0.f || f.gate_logits) return CKDA_ERR_ARG;
    if (f.qk_heads < 0 || (f.qk_heads > 0 && H % f.qk_heads != 0)) return CKDA_ERR_ARG;
    *G = f.qk_heads > 0 ? H / f.qk_heads : 1;
    return CKDA_OK;
}
float resolve_scale(const ckda_flags& f, int dk) {
    return f.scale != 0.f ? f.scale : (float)(1.0 / sqrt((double)dk));
}

}  // namespace

extern "C" {

size_t ckda_linattn_fwd_workspace_bytes(int B, int T, const int* cu_seqlens_host, int n_seqs,
                                        int H, int dk, int dv) {
    Tokens t;
    if (!supported_dim(dk) || !supported_dim(dv)) return (size_t)-1;
    if (read_tokens(B, T, cu_seqlens_host, n_seqs, H, &t) != CKDA_OK) return (size_t)-1;
    size_t need = 0;                    // of either type
    for (ckda_dtype type : {CKDA_F32, CKDA_BF16}) {
        const LaSplit sp =
            make_split(t, nullptr, cu_seqlens_host, H, unit_slots(dk, dv, type, false));
        const size_t n = la_fwd_workspace(sp, t.longest, dk, dv);
        need = n > need ? n : need;
    }
    return need;
}

ckda_status ckda_linattn_fwd_chunked(const void* q, const void* k, const void* v,
                                     const float* log_decay, int per_token, const float* h0,
                                     void* out, float* hT, int B, int T, const int* cu_seqlens,
                                     const int* cu_seqlens_host, int n_seqs, int H, int dk, int dv,
                                     ckda_flags flags, ckda_dtype dtype, void* workspace,
                                     size_t workspace_bytes, ckda_stream_t stream) {
    if (!cu_seqlens != !cu_seqlens_host) return CKDA_ERR_NULL;
    if (dtype != CKDA_F32 && dtype != CKDA_BF16) return CKDA_ERR_UNSUPPORTED;
    Tokens t;
    ckda_status st = read_tokens(B, T, cu_seqlens_host, n_seqs, H, &t);
    if (st != CKDA_OK) return st;
    if (t.total > 0 && (!q || !k || !v || !out)) return CKDA_ERR_NULL;
    if ((t.total > 0 || !per_token) && !log_decay) return CKDA_ERR_NULL;
    if (!supported_dim(dk) || !supported_dim(dv)) return CKDA_ERR_UNSUPPORTED;
    if (per_token != 0 && per_token != 1) return CKDA_ERR_ARG;
    int G;
    if ((st = check_flags(flags, H, &G)) != CKDA_OK) return st;
    const void* ptrs[] = {q, k, v, h0, out, hT, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return CKDA_ERR_ALIGN;
    if (!aligned4(cu_seqlens) || !aligned4(log_decay)) return CKDA_ERR_ALIGN;
    const LaSplit sp =
        make_split(t, cu_seqlens, cu_seqlens_host, H, unit_slots(dk, dv, dtype, false));
    const size_t need = la_fwd_workspace(sp, t.longest, dk, dv);
    if (need > 0 && (!workspace || workspace_bytes < need)) return CKDA_ERR_WORKSPACE;
    const size_t es = elem_size(dtype), tok = (size_t)t.total, nst = (size_t)t.n * H * dk * dv * 4;
    const Buf ins[] = {{q, tok * (H / G) * dk * es}, {k, tok * (H / G) * dk * es},
                       {v, tok * H * dv * es}, {log_decay, (per_token ? tok * H : H) * 4},
                       {h0, nst}, {cu_seqlens, ((size_t)t.n + 1) * 4}};
    const Buf outs[] = {{out, tok * H * dv * es}, {hT, nst}, {need ? workspace : nullptr, need}};
    for (int i = 0; i < 3; ++i) {
        for (const Buf& in : ins)
            if (!(i == 1 && in.p == h0 && hT == h0) && overlap(outs[i], in)) return CKDA_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return CKDA_ERR_ARG;
    }
    const LaFwdArgs a{q, k, v, log_decay, h0, out, hT, per_token, G, resolve_scale(flags, dk), sp};
    return from_cuda(launch_la_fwd(a, t.longest, dk, dv, dtype, workspace, (cudaStream_t)stream));
}

size_t ckda_linattn_bwd_workspace_bytes(int B, int T, const int* cu_seqlens_host, int n_seqs,
                                        int H, int qk_heads, int dk, int dv) {
    Tokens t;
    if (!supported_dim(dk) || !supported_dim(dv)) return (size_t)-1;
    if (read_tokens(B, T, cu_seqlens_host, n_seqs, H, &t) != CKDA_OK) return (size_t)-1;
    if (qk_heads < 0 || (qk_heads > 0 && H % qk_heads != 0)) return (size_t)-1;
    size_t need = 0;                    // of either type
    for (ckda_dtype type : {CKDA_F32, CKDA_BF16}) {
        const LaSplit sp =
            make_split(t, nullptr, cu_seqlens_host, H, unit_slots(dk, dv, type, true));
        const size_t n =
            la_bwd_workspace(sp, t.longest, t.total, qk_heads > 0 ? H / qk_heads : 1, dk, dv);
        need = n > need ? n : need;
    }
    return need;
}

ckda_status ckda_linattn_bwd_chunked(const void* q, const void* k, const void* v,
                                     const float* log_decay, int per_token, const float* h0,
                                     const void* dout, const float* dhT, void* dq, void* dk,
                                     void* dv, float* dlog_decay, float* dh0, int B, int T,
                                     const int* cu_seqlens, const int* cu_seqlens_host, int n_seqs,
                                     int H, int dk_, int dv_, ckda_flags flags, ckda_dtype dtype,
                                     void* workspace, size_t workspace_bytes,
                                     ckda_stream_t stream) {
    if (!cu_seqlens != !cu_seqlens_host) return CKDA_ERR_NULL;
    if (dtype != CKDA_F32 && dtype != CKDA_BF16) return CKDA_ERR_UNSUPPORTED;
    Tokens t;
    ckda_status st = read_tokens(B, T, cu_seqlens_host, n_seqs, H, &t);
    if (st != CKDA_OK) return st;
    if (t.total > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)) return CKDA_ERR_NULL;
    if ((t.total > 0 || !per_token) && !log_decay) return CKDA_ERR_NULL;
    if (!supported_dim(dk_) || !supported_dim(dv_)) return CKDA_ERR_UNSUPPORTED;
    if (per_token != 0 && per_token != 1) return CKDA_ERR_ARG;
    int G;
    if ((st = check_flags(flags, H, &G)) != CKDA_OK) return st;
    const void* ptrs[] = {q, k, v, h0, dout, dhT, dq, dk, dv, dh0, workspace};
    for (const void* p : ptrs)
        if (p && !aligned16(p)) return CKDA_ERR_ALIGN;
    if (!aligned4(cu_seqlens) || !aligned4(log_decay) || !aligned4(dlog_decay))
        return CKDA_ERR_ALIGN;
    const LaSplit sp =
        make_split(t, cu_seqlens, cu_seqlens_host, H, unit_slots(dk_, dv_, dtype, true));
    const size_t need = la_bwd_workspace(sp, t.longest, t.total, G, dk_, dv_);
    if (!workspace || workspace_bytes < need) return CKDA_ERR_WORKSPACE;
    const size_t es = elem_size(dtype), tok = (size_t)t.total;
    const size_t nst = (size_t)t.n * H * dk_ * dv_ * 4, ng = (per_token ? tok * H : H) * 4;
    const size_t nqk = tok * (H / G) * dk_ * es, nv = tok * H * dv_ * es;
    const Buf ins[] = {{q, nqk}, {k, nqk}, {v, nv}, {log_decay, ng}, {h0, nst}, {dout, nv},
                       {dhT, nst}, {cu_seqlens, ((size_t)t.n + 1) * 4}};
    const Buf outs[] = {{dq, nqk}, {dk, nqk}, {dv, nv}, {dlog_decay, ng}, {dh0, nst},
                        {workspace, need}};
    for (int i = 0; i < 6; ++i) {
        for (const Buf& in : ins)
            if (overlap(outs[i], in)) return CKDA_ERR_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], outs[j])) return CKDA_ERR_ARG;
    }
    LaBwdArgs a;
    a.q = q; a.k = k; a.v = v; a.g = log_decay; a.h0 = h0; a.dout = dout; a.dhT = dhT;
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dlog_decay; a.dh0 = dh0;
    a.per_token = per_token;
    a.G = G;
    a.scale = resolve_scale(flags, dk_);
    a.sp = sp;
    a.tokens = t.total;
    a.chunks = (int)la_units(cu_seqlens_host, t.n, t.T, kLaChunk);
    return from_cuda(launch_la_bwd(a, t.longest, dk_, dv_, dtype, workspace,
                                   (cudaStream_t)stream));
}

ckda_status ckda_linattn_decode_step(const void* q, const void* k, const void* v,
                                     const float* log_decay, int per_token, float* state,
                                     void* out, int N, int H, int dk, int dv, ckda_flags flags,
                                     ckda_dtype dtype, ckda_stream_t stream) {
    if (!q || !k || !v || !log_decay || !state || !out) return CKDA_ERR_NULL;
    if (dtype != CKDA_F32 && dtype != CKDA_BF16) return CKDA_ERR_UNSUPPORTED;
    if (N < 1 || H < 1) return CKDA_ERR_SHAPE;
    if ((long long)N * H > (1ll << 26)) return CKDA_ERR_SHAPE;
    if (!supported_dim(dk) || !supported_dim(dv)) return CKDA_ERR_UNSUPPORTED;
    if (per_token != 0 && per_token != 1) return CKDA_ERR_ARG;
    int G;
    ckda_status st = check_flags(flags, H, &G);
    if (st != CKDA_OK) return st;
    const void* ptrs[] = {q, k, v, state, out};
    for (const void* p : ptrs)
        if (!aligned16(p)) return CKDA_ERR_ALIGN;
    if (!aligned4(log_decay)) return CKDA_ERR_ALIGN;
    const size_t es = elem_size(dtype), n = N;
    const Buf ins[] = {{q, n * (H / G) * dk * es}, {k, n * (H / G) * dk * es}, {v, n * H * dv * es},
                       {log_decay, (per_token ? n * H : H) * 4}};
    const Buf o{out, n * H * dv * es}, s{state, n * H * dk * dv * 4};
    for (const Buf& in : ins)
        if (overlap(o, in) || overlap(s, in)) return CKDA_ERR_ARG;
    if (overlap(o, s)) return CKDA_ERR_ARG;
    return from_cuda(launch_la_decode(q, k, v, log_decay, per_token, state, out, N, H, G, dk, dv,
                                      resolve_scale(flags, dk), dtype, (cudaStream_t)stream));
}

}  // extern "C"
