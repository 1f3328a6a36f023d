// linattn_ops.cu -- the linear attention's forward and backward as sequences of runs
// (linattn.cuh), and what the backward needs beside them: the gradient of the log decays, and the
// sums over the value heads that share a q/k head.
#include "linattn.cuh"

namespace ckda {

namespace {

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

struct Carve {
    unsigned char* base;
    size_t at = 0;
    explicit Carve(void* p) : base(static_cast<unsigned char*>(p)) {}
    template <typename T>
    T* take(size_t n) {
        T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
        at += align_up(n * sizeof(T));
        return p;
    }
};

LaRun blank_run() {
    LaRun r = {};
    r.xg = r.yg = r.zg = r.dg = 1;
    r.p_scale = r.u_scale = r.o_scale = 1.f;
    return r;
}

// ----------------------------------------------------------------- gradient of the log decays
// dg_t = <dhT, hT> + sum over s >= t of (q_s.dq_s - k_s.dk_s), per sequence and head: the runs
// leave the row products and their sums per chunk; the sums behind every chunk, then the rows.
// Sums in fp64: a gradient is a small difference of long sums.

__global__ void __launch_bounds__(256)
la_dg_suffix_kernel(LaSplit sp, double* sq, double* __restrict__ sk,
                    const double* __restrict__ dot, int parts, long long clear_to) {
    la_let_next_start();
    la_wait_before();
    const int w = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (w >= sp.n * sp.H) return;
    const int seq = w / sp.H, h = w - seq * sp.H;
    long long start = (long long)seq * sp.T;
    int len = sp.T;
    if (sp.cu) {
        start = min(max(sp.cu[seq], 0), sp.T);
        len = min(max(sp.cu[seq + 1], (int)start), sp.T) - (int)start;
    }
    const int count = (len + kLaChunk - 1) / kLaChunk;
    const long long id0 = la_chunk_id(start, seq, 0);
    if (clear_to) {       // numbers between this sequence's last chunk and the next one's first
        const long long next = seq + 1 < sp.n ? la_chunk_id(start + len, seq + 1, 0) : clear_to;
        for (long long id = id0 + count + lane; id < next && id < clear_to; id += 32)
            sq[(size_t)id * sp.H + h] = 0.0;
    }
    double behind = 0.0;
    if (dot)
        for (int p = 0; p < parts; ++p) behind += dot[(size_t)w * parts + p];
    for (int c0 = count - 1; c0 >= 0; c0 -= 32) {      // 32 chunks at a time, from the last
        const int c = c0 - lane;
        double own = 0.0;
        const size_t at = c >= 0 ? (size_t)(id0 + c) * sp.H + h : 0;
        if (c >= 0) own = sq[at] - sk[at];
        double upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (c >= 0) sk[at] = behind + upto - own;      // what lies behind the chunk
        behind += __shfl_sync(0xffffffffu, upto, 31);
    }
}

// One chunk per CTA, 32 heads at a time (lanes), 8 tokens per warp.  sp.L is the chunk here.
__global__ void __launch_bounds__(256)
la_dg_rows_kernel(LaSplit sp, const float* __restrict__ g, int per_token,
                  const double* __restrict__ rq, const double* __restrict__ rk,
                  const double* __restrict__ behind, float* __restrict__ dg,
                  double* __restrict__ sums) {
    __shared__ double part[8][32];
    la_let_next_start();
    la_wait_before();
    const UnitAt u = find_unit(sp, blockIdx.x);
    if (!u.ok) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long id = la_chunk_id(u.tok - (long long)u.index * sp.L, u.seq, u.index);
    for (int h0 = 0; h0 < sp.H; h0 += 32) {
        const int h = h0 + lane;
        double d[8], s = 0.0;
#pragma unroll
        for (int j = 7; j >= 0; --j) {
            const int t = warp * 8 + j;
            if (t < u.len && h < sp.H) {
                const size_t at = (size_t)(u.tok + t) * sp.H + h;
                s += rq[at] - rk[at];
            }
            d[j] = s;
        }
        __syncthreads();
        part[warp][lane] = s;
        __syncthreads();
        double after = h < sp.H ? behind[(size_t)id * sp.H + h] : 0.0;
        for (int w = warp + 1; w < 8; ++w) after += part[w][lane];
        double total = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int t = warp * 8 + j;
            if (t < u.len && h < sp.H) {
                const size_t at = (size_t)(u.tok + t) * sp.H + h;
                // nothing passes a decay of zero: no rounding error of the sums is left there
                const float gv = per_token ? g[at] : g[h];
                const double x = gv * 1.4426950408889634 < -150.0 ? 0.0 : d[j] + after;
                if (per_token) dg[at] = (float)x;
                total += x;
            }
        }
        if (!per_token) {
            __syncthreads();
            part[warp][lane] = total;
            __syncthreads();
            if (warp == 0 && h < sp.H) {
                double t = 0.0;
                for (int w = 0; w < 8; ++w) t += part[w][lane];
                sums[(size_t)id * sp.H + h] = t;
            }
        }
    }
}

// Fixed decays: the sum over every chunk.  One CTA per head; chunk numbers that no chunk has were
// cleared by la_dg_suffix_kernel.
__global__ void __launch_bounds__(256)
la_dg_head_kernel(const double* __restrict__ sums, long long ids, int H, float* __restrict__ dg) {
    __shared__ double part[8];
    la_wait_before();
    double s = 0.0;
    for (long long i = threadIdx.x; i < ids; i += 256) s += sums[(size_t)i * H + blockIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
        for (int w = 0; w < 8; ++w) t += part[w];
        dg[blockIdx.x] = (float)t;
    }
}

// Gradients of shared q/k heads: the sum over the G value heads that read them.
template <typename T>
__global__ void __launch_bounds__(256)
la_group_sum_kernel(const float* __restrict__ dqf, const float* __restrict__ dkf, T* dq, T* dk,
                    long long vecs, int G, int dim) {
    la_let_next_start();
    la_wait_before();
    const float* src = blockIdx.y ? dkf : dqf;
    T* dst = blockIdx.y ? dk : dq;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;   // four elements of the result
    if (i >= vecs) return;
    const int per = dim / 4;
    const long long row = i / per;                                   // token * q/k heads + head
    const int c = (int)(i - row * per) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < G; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(src + ((size_t)row * G + j) * dim + c);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    T* p = dst + (size_t)row * dim + c;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = s;
    } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(s.x, s.y), b = __floats2bfloat162_rn(s.z, s.w);
        uint2 w = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
        *reinterpret_cast<uint2*>(p) = w;
    }
}

}  // namespace

// ------------------------------------------------------------------------------------ forward

namespace {
struct FwdWs { float* states; double* decay; size_t bytes; };
FwdWs fwd_ws(void* ws, bool split, long long units, int H, int dk, int dv) {
    Carve c(ws);
    FwdWs w = {};
    if (split) {
        w.states = c.take<float>((size_t)units * H * dk * dv);
        w.decay = c.take<double>((size_t)units * H);
    }
    w.bytes = c.at;
    return w;
}
}  // namespace

size_t la_fwd_workspace(const LaSplit& sp, long long longest, int dk, int dv) {
    return fwd_ws(nullptr, la_is_split(longest, sp.L), sp.units, sp.H, dk, dv).bytes;
}

cudaError_t launch_la_fwd(const LaFwdArgs& f, long long longest, int dk, int dv, ckda_dtype dtype,
                          void* ws, cudaStream_t s) {
    const bool split = la_is_split(longest, f.sp.L);
    const FwdWs w = fwd_ws(ws, split, f.sp.units, f.sp.H, dk, dv);
    LaArgs a = {};
    a.sp = f.sp;
    a.g = f.g;
    a.per_token = f.per_token;
    a.runs = 1;
    LaRun r = blank_run();
    r.x = f.q; r.y = f.k; r.z = f.v;
    r.xg = r.yg = f.G;
    r.out = f.out;
    r.init = f.h0;
    r.fin = f.hT;
    r.p_scale = r.o_scale = f.scale;
    r.unit_state = w.states;
    r.unit_decay = w.decay;
    // (every unit reads h0 then, and the last one writes hT: not when they are the same)
    r.fold = la_folds(longest, f.sp.L, kLaFoldUnits) && f.hT != f.h0;
    a.run[0] = r;
    cudaError_t e;
    if (f.sp.empty && f.hT && (!split || r.fold))
        if ((e = launch_la_empty(a, dk, dv, s)) != cudaSuccess) return e;
    if (split) {
        if ((e = launch_la_summary(a, dk, dv, dtype, s)) != cudaSuccess) return e;
        a.after = 1;
        if (!r.fold && (e = launch_la_scan(a, dk, dv, s)) != cudaSuccess) return e;
    }
    return launch_la_run(a, dk, dv, false, dtype, s);
}

// ----------------------------------------------------------------------------------- backward

namespace {
struct BwdWs {
    float *S, *R, *dqf, *dkf;
    double *decS, *decR, *rq, *rk, *sq, *sk, *dot;
    size_t bytes;
};
BwdWs bwd_ws(void* ws, bool split, const LaSplit& sp, long long tokens, int G, int dk, int dv) {
    Carve c(ws);
    BwdWs w = {};
    const size_t H = sp.H, uh = (size_t)sp.units * H, th = (size_t)tokens * H;
    if (split) {
        w.S = c.take<float>(uh * dk * dv);
        w.R = c.take<float>(uh * dk * dv);
        w.decS = c.take<double>(uh);
        w.decR = c.take<double>(uh);
    }
    w.rq = c.take<double>(th);
    w.rk = c.take<double>(th);
    w.sq = c.take<double>(la_chunk_ids(tokens, sp.n) * H);
    w.sk = c.take<double>(la_chunk_ids(tokens, sp.n) * H);
    w.dot = c.take<double>((size_t)sp.n * H * la_scan_parts(dk * dv));
    if (G > 1) {
        w.dqf = c.take<float>(th * dk);
        w.dkf = c.take<float>(th * dk);
    }
    w.bytes = c.at;
    return w;
}
}  // namespace

size_t la_bwd_workspace(const LaSplit& sp, long long longest, long long tokens, int G, int dk,
                        int dv) {
    return bwd_ws(nullptr, la_is_split(longest, sp.L), sp, tokens, G, dk, dv).bytes;
}

cudaError_t launch_la_bwd(const LaBwdArgs& b, long long longest, int dk, int dv, ckda_dtype dtype,
                          void* ws, cudaStream_t s) {
    const LaSplit& sp = b.sp;
    const bool split = la_is_split(longest, sp.L);
    const int H = sp.H, G = b.G;
    const BwdWs w = bwd_ws(ws, split, sp, b.tokens, G, dk, dv);
    cudaError_t e;
    LaArgs a = {};
    a.sp = sp;
    a.g = b.g;
    a.per_token = b.per_token;

    // states S forwards and their gradients R backwards, per unit
    LaRun rs = blank_run(), rr = blank_run();
    rs.y = b.k; rs.yg = G; rs.z = b.v;
    rs.init = b.h0;
    rr.y = b.q; rr.yg = G; rr.z = b.dout;
    rr.init = b.dhT;
    rr.fin = b.dh0;
    rr.reverse = 1;
    rr.u_scale = b.scale;
    const bool want_dot = b.dg && b.dhT;
    // (the tcgen05 run of dq reads its summaries a thread a row, which a scan in coalesced reads beats
    // from three units on: 256 tokens x 16 heads in four 52 -> 42 us; 2 x 2048 tokens in two units 147
    // us, with a scan 151)
    const bool tc = dtype == CKDA_BF16 && dk == 128 && dv == 128;
    const bool fold = la_folds(longest, sp.L, tc ? 2 : kLaFoldUnits), scan = split && !fold;
    int parts = 1;
    if (sp.empty && b.dh0 && !scan) {
        a.run[0] = rr;
        a.runs = 1;
        if ((e = launch_la_empty(a, dk, dv, s)) != cudaSuccess) return e;
    }
    if (split) {
        rs.unit_state = w.S; rs.unit_decay = w.decS;
        rr.unit_state = w.R; rr.unit_decay = w.decR;
        if (scan && want_dot) { rs.fin_dot = b.dhT; rs.fin_dot_out = w.dot; parts = la_scan_parts(dk * dv); }
        a.run[0] = rs;
        a.run[1] = rr;
        a.runs = 2;
        if ((e = launch_la_summary(a, dk, dv, dtype, s)) != cudaSuccess) return e;
        a.after = 1;
        if (scan && (e = launch_la_scan(a, dk, dv, s)) != cudaSuccess) return e;
    }

    LaRun q = blank_run(), k = blank_run(), v = blank_run();
    q.x = b.dout; q.y = b.v; q.z = b.k; q.zg = G;
    q.out = G > 1 ? (void*)w.dqf : b.dq;
    q.transposed = 1;
    q.p_scale = q.o_scale = b.scale;
    q.init = b.h0;
    q.unit_state = w.S; q.unit_decay = w.decS;
    q.fold = k.fold = v.fold = fold;
    if (!scan && want_dot) { q.fin_dot = b.dhT; q.fin_dot_out = w.dot; }
    k.x = b.v; k.y = b.dout; k.z = b.q; k.zg = G;
    k.out = G > 1 ? (void*)w.dkf : b.dk;
    k.transposed = 1;
    k.reverse = 1;
    k.p_scale = k.u_scale = b.scale;
    k.init = b.dhT;
    k.unit_state = w.R; k.unit_decay = w.decR;
    q.out_f32 = k.out_f32 = G > 1;
    if (b.dg) {
        q.dot = b.q; k.dot = b.k;
        q.dg = k.dg = G;
        q.dot_out = w.rq; k.dot_out = w.rk;
        q.dot_sum = w.sq; k.dot_sum = w.sk;
    }
    v.x = b.k; v.xg = G; v.y = b.q; v.yg = G; v.z = b.dout;
    v.out = b.dv;
    v.reverse = 1;
    v.p_scale = v.u_scale = b.scale;
    v.init = b.dhT;
    v.unit_state = w.R; v.unit_decay = w.decR;
    if (!scan) v.fin = b.dh0;
    a.run[0] = q;
    a.run[1] = k;
    a.run[2] = v;
    // dq and dk in full precision: the decay gradient is made of small differences of q.dq and k.dk,
    // and asking for it changes neither (two terms without it: 16 heads x 2 x 2048 tokens 112 us, not 134).
    // Three runs of the same kernel go in one launch, side by side.
    const bool one = dk == dv && dtype == CKDA_F32;
    a.runs = one ? 3 : 2;
    if ((e = launch_la_run(a, dv, dk, true, dtype, s)) != cudaSuccess) return e;
    if (!one) {
        a.run[0] = v;
        a.runs = 1;
        a.after = 1;      // (nothing of it depends on the run before: they only follow each other)
        if ((e = launch_la_run(a, dk, dv, false, dtype, s)) != cudaSuccess) return e;
    }

    if (G > 1 && b.tokens > 0) {
        const long long vecs = b.tokens * (H / G) * (dk / 4);
        const dim3 grid((unsigned)((vecs + 255) / 256), 2);
        e = dtype == CKDA_BF16
                ? la_launch_after(la_group_sum_kernel<__nv_bfloat16>, grid, 256, 0, s, w.dqf, w.dkf,
                                  (__nv_bfloat16*)b.dq, (__nv_bfloat16*)b.dk, vecs, G, dk)
                : la_launch_after(la_group_sum_kernel<float>, grid, 256, 0, s, w.dqf, w.dkf,
                                  (float*)b.dq, (float*)b.dk, vecs, G, dk);
        if (e != cudaSuccess) return e;
    }
    if (b.dg) {
        const long long ids = (long long)la_chunk_ids(b.tokens, sp.n);
        e = la_launch_after(la_dg_suffix_kernel, dim3((unsigned)((sp.n * H + 7) / 8)), 256, 0, s, sp,
                            w.sq, w.sk, want_dot ? w.dot : nullptr, parts, b.per_token ? 0ll : ids);
        if (e != cudaSuccess) return e;
        // (w.sq has been read: it takes the chunks' sums of a fixed decay's gradient)
        LaSplit rows = sp;
        rows.L = kLaChunk;
        rows.units = b.chunks;
        if (rows.units > 0 &&
            (e = la_launch_after(la_dg_rows_kernel, dim3((unsigned)rows.units), 256, 0, s, rows, b.g,
                                 b.per_token, w.rq, w.rk, w.sk, b.dg, w.sq)) != cudaSuccess)
            return e;
        if (!b.per_token && (e = la_launch_after(la_dg_head_kernel, dim3((unsigned)H), 256, 0, s, w.sq,
                                                 ids, H, b.dg)) != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace ckda
