// linattn.cu -- chunked linear attention with a decay for each head (every head size and type).
//
// A run carries the state M = S^T (rows: output channels, columns: contracted channels) through
// the chunks of one unit of tokens.  With G the running sum of the log decays inside the chunk
// and P_ij = (x_i . y_j) exp(G_i - G_j) for j <= i:
//     out_i = p P_i z + o exp(G_i) M x_i,     M <- exp(G_C) M + u sum_j exp(G_C - G_j) z_j y_j^T
// (a backward run mirrors this: j >= i, out takes exp(G_C - G_i), the update exp(G_j)).  Only
// differences of G with a non-positive sign are ever exponentiated, so nothing overflows however
// strong the decay.
//
// Layout: one warp owns 16 output channels for the whole unit, and keeps its 16 rows of M in
// registers as fp32 accumulators.  The accumulator layout of M is the operand layout of the
// read-out product, so M never passes through shared memory; z is loaded once per 16 x 16 tile
// and serves both the product with P and (weighted, as the left operand) the update.  The warps
// share only P, which they form together (16 x 16 tiles on or below the diagonal).
//
// Precision: every value enters the products as a sum of bf16 terms: one for a bf16 input
// (exact), three for an fp32 one (8 bits each, 24 in all; the products of terms below 2^-24 are
// left out).  The weighted z of the state update always has three, so states are fp32-grade
// whatever the input type; P and M as operands have three when `exact` asks for it, else two, which
// leave 2^-18 of a value, far below a bf16 output's own rounding.  (With one term of M outputs were
// 1.24 times as far off as their rounding, with one of P too 1.6 times.)
//
// What bounds it: latency.  A warp holds a state and its operands in 200 registers, so an SM has 8 to
// 12 warps, 0.27 instructions a cycle and scheduler, the mma.sync pipe 20 to 30 % busy; an fp32 chunk
// takes six products of terms for one.  16 heads x 4096 tokens, calls one after the other: bf16 64 x 64
// forward 65 us, backward 198; fp32 128 x 128 forward 247 us, backward 709; fp32 3 x 333 tokens x 6 heads
// backward 52 us.
#include "linattn.cuh"

namespace ckda {

namespace {

constexpr int C = kLaChunk;

// ------------------------------------------------------------------------------ small pieces

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void ldsm4(uint32_t r[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t r[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
    const int n = live ? 16 : 0;   // (0 source bytes: the destination is zero-filled)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // a in the low half
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
// a, b as sums of N bf16 terms (round to nearest, then the remainders: each has 8 bits more).
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t t[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = pack2(a, b);
        if (i + 1 < N) { a -= lo_f(t[i]); b -= hi_f(t[i]); }
    }
}

// ------------------------------------------------------------------------------- the run kernel

template <typename T>
struct Terms { static constexpr int value = sizeof(T) == 2 ? 1 : 3; };

template <typename T, int DC, int DO, bool kSummary, int NP>
struct RunShape {
    static constexpr int NW = DO / 16;                 // warps: 16 output channels each
    static constexpr int THREADS = NW * 32;
    static constexpr int NI = Terms<T>::value;         // bf16 planes of an input
    static constexpr int STAGES = NI == 1 ? 2 : 1;
    static constexpr int LC = DC + 8, LO = DO + 8, LP = C + 8;   // row pitches: 16 bytes of padding
    static constexpr int XY = C * LC, Z = C * LO;      // (elements; keeps ldmatrix conflict-free)
    static constexpr int STAGE = NI * (XY * (kSummary ? 1 : 2) + Z);
    static constexpr int PP = kSummary ? 0 : NP * C * LP;
    static constexpr size_t SMEM = (size_t)(STAGES * STAGE + PP) * 2 + 2 * (4 * C + 8) * 4 +
                                   (kSummary ? 0 : NW * C * 8);
};

__device__ __forceinline__ float2 pair_of(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 pair_of(const __nv_bfloat16* p) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(lo_f(w), hi_f(w));
}

// Running sums of the chunk's log2 decays (fp64, kept as two floats), and the two weights of
// every token.  One warp.
struct GateBuf {
    float hi[C], lo[C], out[C], upd[C];
    float total;    // exp2 of the chunk's sum
    float pad;
    double sum;     // that sum, log2
    double pad2[2];
};
static_assert(sizeof(GateBuf) == (4 * C + 8) * 4, "gate buffer size");

__device__ void chunk_gates(GateBuf* b, double g0, double g1, bool reverse, float u_scale) {
    const int lane = threadIdx.x & 31;
    double s = g0 + g1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    const double all = __shfl_sync(0xffffffffu, s, 31);
    const double G[2] = {s - g1, s};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * lane + e;
        const float hi = (float)G[e];
        const float up = exp2f((float)(all - G[e])), down = exp2f(hi);
        b->hi[t] = hi;
        b->lo[t] = (float)(G[e] - (double)hi);
        b->out[t] = reverse ? up : down;
        b->upd[t] = (reverse ? down : up) * u_scale;
    }
    if (lane == 0) {
        b->total = exp2f((float)all);
        b->sum = all;
    }
}

// One operand's chunk: D channels of up to C tokens, zero behind the last one.  bf16: asynchronous.
template <typename T, int D, int THREADS>
__device__ __forceinline__ void load_rows(__nv_bfloat16* dst, const T* src, long long tok, int live,
                                          int stride, int head) {
    constexpr int LD = D + 8, V = D / 8;
    for (int i = threadIdx.x; i < C * V; i += THREADS) {
        const int r = i / V, c = (i % V) * 8;
        const bool in = r < live;
        cp16(smem_addr(dst + r * LD + c),
             src + ((size_t)(tok + (in ? r : 0)) * stride + head) * D + c, in);
    }
}
// fp32: every request is on its way before the first value is split (a chunk's latency is one
// memory round trip, not one per 16 bytes).
template <int D, int THREADS>
struct Fetch {
    static constexpr int V = D / 4, N = C * V / THREADS;
    float4 x[N];
    __device__ __forceinline__ void request(const float* src, long long tok, int live, int stride,
                                            int head) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * THREADS, r = i / V, c = (i % V) * 4;
            x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < live)
                x[k] = __ldg(reinterpret_cast<const float4*>(
                    src + ((size_t)(tok + r) * stride + head) * D + c));
        }
    }
    __device__ __forceinline__ void store(__nv_bfloat16* dst) const {
        constexpr int LD = D + 8;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = threadIdx.x + k * THREADS, r = i / V, c = (i % V) * 4;
            uint32_t a[3], b[3];
            split2<3>(x[k].x, x[k].y, a);
            split2<3>(x[k].z, x[k].w, b);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<uint2*>(dst + p * C * LD + r * LD + c) = make_uint2(a[p], b[p]);
        }
    }
};

// acc += A B for the leading terms, low += A B for the other pairs whose product is not below the
// precision kept.  Two accumulators, because the tensor core's sums do not round to nearest: what
// is lost then is a part of the few leading products only.  With three terms those are added in fp32
// one tile at a time, so that no loss carries on (errors of fp32 results 2.0e-7 -> 1.2e-7, about half the
// plain fp32 form's; 4096 x 16 heads 128 x 128 forward 224 -> 237 us, 64 x 64 backward 276 -> 281).
template <int NA, int NB>
__device__ __forceinline__ void mma_terms(float acc[4], float low[4], const uint32_t (*a)[4],
                                          const uint32_t (*b)[2]) {
    constexpr int N = NA > NB ? NA : NB;
#pragma unroll
    for (int s = N - 1; s > 0; --s)      // smallest terms first
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = s - i;
            if (j >= 0 && j < NB) mma(low, a[i], b[j][0], b[j][1]);
        }
    if constexpr (N == 3) {
        float f[4] = {};
        mma(f, a[0], b[0][0], b[0][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += f[k];
    } else {
        mma(acc, a[0], b[0][0], b[0][1]);
    }
}

template <typename T, int DC, int DO, bool kSummary, int NP>
__global__ void __launch_bounds__(DO * 2)
la_run_kernel(const LaArgs a) {
    using S = RunShape<T, DC, DO, kSummary, NP>;
    constexpr int NW = S::NW, NI = S::NI, LC = S::LC, LO = S::LO, LP = S::LP;
    constexpr int KC = DC / 16;                 // 16-deep steps over the contracted channels
    constexpr int NU = 3;                       // terms of the weighted z
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __nv_bfloat16* stages = reinterpret_cast<__nv_bfloat16*>(smem_raw);
    __nv_bfloat16* sP = stages + S::STAGES * S::STAGE;
    GateBuf* gates = reinterpret_cast<GateBuf*>(sP + S::PP);
    double* sDot = reinterpret_cast<double*>(gates + 2);

    const LaRun& R = a.run[blockIdx.y];
    const int H = a.sp.H;
    const int unit = blockIdx.x / H, h = blockIdx.x - unit * H;
    const UnitAt u = find_unit(a.sp, unit);
    la_let_next_start();
    la_wait_before();       // (returns at once in the first launch of a call)
    if (!u.ok) return;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gr = lane >> 2, gc = (lane & 3) * 2;          // fragment row, column pair
    const int r0 = warp * 16;                               // this warp's output channels
    const bool rev = R.reverse;
    const T* x = static_cast<const T*>(R.x);
    const T* y = static_cast<const T*>(R.y);
    const T* z = static_cast<const T*>(R.z);
    const int nch = (u.len + C - 1) / C;

    auto chunk_at = [&](int i) { return rev ? nch - 1 - i : i; };
    auto load = [&](int i) {
        const int c = chunk_at(i), live = min(C, u.len - c * C);
        const long long tok = u.tok + (long long)c * C;
        __nv_bfloat16* st = stages + (i % S::STAGES) * S::STAGE;
        if constexpr (sizeof(T) == 2) {
            load_rows<T, DC, S::THREADS>(st, y, tok, live, H / R.yg, h / R.yg);
            load_rows<T, DO, S::THREADS>(st + NI * S::XY, z, tok, live, H / R.zg, h / R.zg);
            if constexpr (!kSummary)
                load_rows<T, DC, S::THREADS>(st + NI * (S::XY + S::Z), x, tok, live, H / R.xg,
                                             h / R.xg);
        } else {
            // (x with y and z, or after them in y's registers where y alone takes over 8 requests a
            // thread.  Few output channels leave few threads: 128 x 16 asks for 64 at once, and spills)
            Fetch<DC, S::THREADS> fy;
            Fetch<DO, S::THREADS> fz;
            fy.request(y, tok, live, H / R.yg, h / R.yg);
            fz.request(z, tok, live, H / R.zg, h / R.zg);
            if constexpr (!kSummary && Fetch<DC, S::THREADS>::N <= 8) {
                Fetch<DC, S::THREADS> fx;
                fx.request(x, tok, live, H / R.xg, h / R.xg);
                fy.store(st);
                fz.store(st + NI * S::XY);
                fx.store(st + NI * (S::XY + S::Z));
            } else {
                fy.store(st);
                fz.store(st + NI * S::XY);
                if constexpr (!kSummary) {
                    fy.request(x, tok, live, H / R.xg, h / R.xg);
                    fy.store(st + NI * (S::XY + S::Z));
                }
            }
        }
    };
    auto gate_pair = [&](int i, double* g0, double* g1) {
        const int c = chunk_at(i);
        const long long tok = u.tok + (long long)c * C;
        const int left = u.len - c * C;
        *g0 = log2_decay(a.g, a.per_token, tok + 2 * lane, H, h, 2 * lane < left);
        *g1 = log2_decay(a.g, a.per_token, tok + 2 * lane + 1, H, h, 2 * lane + 1 < left);
    };

    auto load_z = [&](uint32_t f[4], const __nv_bfloat16* z, int kk) {
        ldsm4t(f, smem_addr(z + (kk * 16 + (lane >> 4) * 8 + (lane & 7)) * LO + r0 + ((lane >> 3) & 1) * 8));
    };

    // The state: rows r0 + gr (+ 8), columns 8 n + gc (+ 1).
    float M[DC / 8][4];
    const int rs = R.transposed ? DC : 1, cs = R.transposed ? 1 : DO;
    const int own = (r0 + gr) * rs + gc * cs;
    const size_t st_size = (size_t)DC * DO;
    const size_t seq_state = ((size_t)u.seq * H + h) * st_size;
    const size_t unit_state = ((size_t)unit * H + h) * st_size;
    const bool fold = !kSummary && R.fold && R.unit_state;
    const float* init = nullptr;
    if (!kSummary) {
        if (R.unit_state && !fold) init = R.unit_state + unit_state;
        else if (R.init) init = R.init + seq_state;
    }
#pragma unroll
    for (int n = 0; n < DC / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            M[n][e] = init ? init[own + (e >> 1) * 8 * rs + (8 * n + (e & 1)) * cs] : 0.f;
    if (fold) {                               // the units ahead of this one, in the run's order
        const int ahead = la_units_ahead(fold, rev, unit, u.index, u.count, a.sp.units);
#pragma unroll 1
        for (int k = 0; k < ahead; ++k) {
            const size_t un = (size_t)(rev ? unit + ahead - k : unit - ahead + k) * H + h;
            const float w = exp2f((float)R.unit_decay[un]);
            const float* E = R.unit_state + un * st_size + own;
#pragma unroll
            for (int n = 0; n < DC / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    M[n][e] = fmaf(M[n][e], w, E[(e >> 1) * 8 * rs + (8 * n + (e & 1)) * cs]);
        }
    }
    double decay = 0.0;

    if (warp == 0) {
        double g0, g1;
        gate_pair(0, &g0, &g1);
        chunk_gates(&gates[0], g0, g1, rev, R.u_scale);
    }
    if constexpr (S::STAGES == 2) load(0);
    asm volatile("cp.async.commit_group;");

    for (int i = 0; i < nch; ++i) {
        const int c = chunk_at(i), live = min(C, u.len - c * C);
        const long long tok = u.tok + (long long)c * C;
        if constexpr (S::STAGES == 1) {
            if (i > 0) __syncthreads();   // the last chunk's operands are done with
            load(i);
        }
        double g0 = 0.0, g1 = 0.0;
        if (warp == 0 && i + 1 < nch) gate_pair(i + 1, &g0, &g1);
        asm volatile("cp.async.wait_group 0;");
        __syncthreads();
        if constexpr (S::STAGES == 2) {
            if (i + 1 < nch) load(i + 1);
            asm volatile("cp.async.commit_group;");
        }
        const GateBuf& gb = gates[i & 1];
        const __nv_bfloat16* sY = stages + (i % S::STAGES) * S::STAGE;
        const __nv_bfloat16* sZ = sY + NI * S::XY;
        const __nv_bfloat16* sX = sZ + NI * S::Z;

        float acc[4][2][4], low[4][2][4];     // (low stays zero, and free, without lower terms)
        if constexpr (!kSummary) {
            // 1. this warp's tiles of P (16 x 16; on the kept side of the diagonal)
            // (rolled where registers allow it: unrolled throughout, the code is 100 KB, which no
            // instruction cache keeps from one chunk to the next)
#pragma unroll 1
            for (int t = warp; t < 16; t += NW) {
                const int mi = t & 3, nj = t >> 2;
                if (rev ? mi > nj : mi < nj) continue;
                float p[2][4] = {}, pl[2][4] = {};
#pragma unroll 1
                for (int kk = 0; kk < KC; ++kk) {
                    uint32_t fa[NI][4], fb[NI][4];
#pragma unroll
                    for (int q = 0; q < NI; ++q) {
                        ldsm4(fa[q], smem_addr(sX + q * S::XY + (mi * 16 + (lane & 15)) * LC +
                                               kk * 16 + (lane >> 4) * 8));
                        ldsm4(fb[q], smem_addr(sY + q * S::XY +
                                               (nj * 16 + (lane >> 4) * 8 + (lane & 7)) * LC +
                                               kk * 16 + ((lane >> 3) & 1) * 8));
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        uint32_t b[NI][2];
#pragma unroll
                        for (int q = 0; q < NI; ++q) {
                            b[q][0] = fb[q][2 * n];
                            b[q][1] = fb[q][2 * n + 1];
                        }
                        mma_terms<NI, NI>(p[n], pl[n], fa, b);
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        const int row = mi * 16 + gr + e2 * 8, col = nj * 16 + n * 8 + gc;
                        float w[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float d = (gb.hi[row] - gb.hi[col + e]) +
                                            (gb.lo[row] - gb.lo[col + e]);
                            const bool keep = rev ? row <= col + e : row >= col + e;
                            w[e] = keep ? (p[n][2 * e2 + e] + pl[n][2 * e2 + e]) * exp2f(rev ? -d : d) * R.p_scale : 0.f;
                        }
                        uint32_t t3[NP];
                        split2<NP>(w[0], w[1], t3);
#pragma unroll
                        for (int q = 0; q < NP; ++q)
                            *reinterpret_cast<uint32_t*>(sP + q * C * LP + row * LP + col) = t3[q];
                    }
            }
            // 2. read-out of the entering state: X M^T, rows scaled by the decay since then
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[m][n][e] = low[m][n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KC; ++kk) {
                uint32_t b[2][NP][2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    uint32_t t0[NP], t1[NP];
                    split2<NP>(M[2 * kk][2 * n], M[2 * kk][2 * n + 1], t0);
                    split2<NP>(M[2 * kk + 1][2 * n], M[2 * kk + 1][2 * n + 1], t1);
#pragma unroll
                    for (int q = 0; q < NP; ++q) { b[n][q][0] = t0[q]; b[n][q][1] = t1[q]; }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t fa[NI][4];
#pragma unroll
                    for (int q = 0; q < NI; ++q)
                        ldsm4(fa[q], smem_addr(sX + q * S::XY + (m * 16 + (lane & 15)) * LC +
                                               kk * 16 + (lane >> 4) * 8));
                    mma_terms<NI, NP>(acc[m][0], low[m][0], fa, b[0]);
                    mma_terms<NI, NP>(acc[m][1], low[m][1], fa, b[1]);
                }
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const float w = gb.out[m * 16 + gr + e2 * 8] * R.o_scale;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        acc[m][n][2 * e2] *= w;
                        acc[m][n][2 * e2 + 1] *= w;
                        low[m][n][2 * e2] *= w;
                        low[m][n][2 * e2 + 1] *= w;
                    }
                }
            __syncthreads();              // P is complete
        }
        if constexpr (!kSummary) {
            // 3. the chunk's own products, 16 tokens of z at a time.  z^T tile: registers 0, 2 are
            // channels 0-7, 1, 3 channels 8-15; 2, 3 tokens 8-15
#pragma unroll 1
            for (int kk = 0; kk < C / 16; ++kk) {
                uint32_t fz[NI][4], b[2][NI][2];
#pragma unroll
                for (int q = 0; q < NI; ++q) {
                    load_z(fz[q], sZ + q * S::Z, kk);
#pragma unroll
                    for (int n = 0; n < 2; ++n) { b[n][q][0] = fz[q][n]; b[n][q][1] = fz[q][n + 2]; }
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (rev ? m > kk : m < kk) continue;
                    uint32_t fp[NP][4];
#pragma unroll
                    for (int q = 0; q < NP; ++q)
                        ldsm4(fp[q], smem_addr(sP + q * C * LP + (m * 16 + (lane & 15)) * LP +
                                               kk * 16 + (lane >> 4) * 8));
                    mma_terms<NP, NI>(acc[m][0], low[m][0], fp, b[0]);
                    mma_terms<NP, NI>(acc[m][1], low[m][1], fp, b[1]);
                }
            }
        }
        decay += gb.sum;
        if constexpr (!kSummary) {
            // 4. the outputs: rows m 16 + gr (+ 8), channels r0 + 8 n + gc (+ 1)
            const size_t at0 = ((size_t)tok * H + h) * DO + r0 + gc, ostep = (size_t)H * DO;
            const int Hd = H / R.dg;
            const T* w0 = R.dot ? static_cast<const T*>(R.dot) + ((size_t)tok * Hd + h / R.dg) * DO + r0 + gc
                                : nullptr;
            const bool f32 = sizeof(T) == 4 || R.out_f32;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2) {
                    const int row = m * 16 + gr + e2 * 8;
                    float2 v[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        v[n] = make_float2(acc[m][n][2 * e2] + low[m][n][2 * e2],
                                           acc[m][n][2 * e2 + 1] + low[m][n][2 * e2 + 1]);
                    if (row < live) {
                        const size_t at = at0 + row * ostep;
                        if (f32) {
                            float* o = static_cast<float*>(R.out) + at;
                            *reinterpret_cast<float2*>(o) = v[0];
                            *reinterpret_cast<float2*>(o + 8) = v[1];
                        } else {
                            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(R.out) + at;
                            *reinterpret_cast<uint32_t*>(o) = pack2(v[0].x, v[0].y);
                            *reinterpret_cast<uint32_t*>(o + 8) = pack2(v[1].x, v[1].y);
                        }
                    }
                    if (w0) {
                        double dot = 0.0;
                        if (row < live) {
                            const T* w = w0 + (size_t)row * Hd * DO;
                            const float2 a = pair_of(w), b = pair_of(w + 8);
                            dot = (double)v[0].x * a.x + (double)v[0].y * a.y + (double)v[1].x * b.x + (double)v[1].y * b.y;
                        }
                        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
                        dot += __shfl_xor_sync(0xffffffffu, dot, 2);
                        if ((lane & 3) == 0) sDot[warp * C + row] = dot;
                    }
                }
            if (R.dot) {
                __syncthreads();
                if (warp == 0) {
                    double sum = 0.0;
#pragma unroll
                    for (int e = 0; e < C / 32; ++e) {
                        const int r = lane + 32 * e;
                        double s = 0.0;
#pragma unroll
                        for (int w = 0; w < NW; ++w) s += sDot[w * C + r];
                        if (r < live) {
                            R.dot_out[(size_t)(tok + r) * H + h] = s;
                            sum += s;
                        }
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    if (lane == 0)
                        R.dot_sum[(size_t)la_chunk_id(u.tok - (long long)u.index * a.sp.L, u.seq,
                                                      u.index * (a.sp.L / C) + c) * H + h] = sum;
                }
            }
        }
        // 5. the state update: the chunk's sum on its own (fp32 accumulators from zero), then added
        const float total = gb.total;
        uint32_t wz[C / 16][NU][4];
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk) {
            uint32_t fz[NI][4];
#pragma unroll
            for (int q = 0; q < NI; ++q) load_z(fz[q], sZ + q * S::Z, kk);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = kk * 16 + gc + (r >> 1) * 8;
                float v0 = 0.f, v1 = 0.f;
#pragma unroll
                for (int q = NI - 1; q >= 0; --q) { v0 += lo_f(fz[q][r]); v1 += hi_f(fz[q][r]); }
                uint32_t t3[NU];
                split2<NU>(v0 * gb.upd[t], v1 * gb.upd[t + 1], t3);
#pragma unroll
                for (int q = 0; q < NU; ++q) wz[kk][q][r] = t3[q];
            }
        }
#pragma unroll
        for (int n = 0; n < DC / 16; ++n) {
            float sum[2][4] = {}, less[2][4] = {};
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk) {
                uint32_t fy[NI][4];
#pragma unroll
                for (int q = 0; q < NI; ++q)
                    ldsm4t(fy[q], smem_addr(sY + q * S::XY +
                                            (kk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * LC +
                                            n * 16 + (lane >> 4) * 8));
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t b[NI][2];
#pragma unroll
                    for (int q = 0; q < NI; ++q) { b[q][0] = fy[q][2 * e]; b[q][1] = fy[q][2 * e + 1]; }
                    mma_terms<NU, NI>(sum[e], less[e], wz[kk], b);
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    M[2 * n + e][k] = fmaf(M[2 * n + e][k], total, sum[e][k] + less[e][k]);
        }
        if (warp == 0 && i + 1 < nch) chunk_gates(&gates[(i + 1) & 1], g0, g1, rev, R.u_scale);
    }

    // the state after the unit: a summary, or (one unit per sequence) the final state
    // (the run's last unit of a sequence, where no scan has formed it)
    const bool last = !R.unit_state || (fold && u.index == (rev ? 0 : u.count - 1));
    float* fin = kSummary ? R.unit_state + unit_state : (last && R.fin ? R.fin + seq_state : nullptr);
    if (fin) {
#pragma unroll
        for (int n = 0; n < DC / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                fin[own + (e >> 1) * 8 * rs + (8 * n + (e & 1)) * cs] = M[n][e];
    }
    if (kSummary && tid == 0) R.unit_decay[(size_t)unit * H + h] = decay;
    if (!kSummary && last && R.fin_dot) {
        double d = 0.0;
#pragma unroll
        for (int n = 0; n < DC / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                d += (double)M[n][e] *
                     (double)R.fin_dot[seq_state + own + (e >> 1) * 8 * rs + (8 * n + (e & 1)) * cs];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        __syncthreads();                  // (the gate buffers are free)
        double* sd = reinterpret_cast<double*>(gates);
        if (lane == 0) sd[warp] = d;
        __syncthreads();
        if (tid == 0) {
            double s = 0.0;
            for (int w = 0; w < NW; ++w) s += sd[w];
            R.fin_dot_out[(size_t)u.seq * H + h] = s;
        }
    }
}

// Units of a sequence, in the run's order: entering state of each from the summaries, in place.
// One thread per four state elements.
constexpr int kScanThreads = 256;
__global__ void __launch_bounds__(kScanThreads)
la_scan_kernel(const LaArgs a, int elems, int parts) {
    la_let_next_start();
    la_wait_before();
    const LaRun& R = a.run[blockIdx.y];
    const int H = a.sp.H;
    const int sh = blockIdx.x / parts, part = blockIdx.x - sh * parts;
    const int seq = sh / H, h = sh - seq * H;
    int first, count;
    seq_units(a.sp, seq, &first, &count);
    const int e = (part * kScanThreads + threadIdx.x) * 4;
    const bool in = e < elems;
    double d = 0.0;
    if (in) {
        const size_t at = (size_t)sh * elems + e;
        float4 S = R.init ? *reinterpret_cast<const float4*>(R.init + at)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int AHEAD = 4;      // summaries requested before the first is used
        for (int i0 = 0; i0 < count; i0 += AHEAD) {
            float4 E[AHEAD];
            float w[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (i0 + j < count) {
                    const int un = first + (R.reverse ? count - 1 - i0 - j : i0 + j);
                    E[j] = *reinterpret_cast<const float4*>(R.unit_state +
                                                            ((size_t)un * H + h) * elems + e);
                    w[j] = exp2f((float)R.unit_decay[(size_t)un * H + h]);
                }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (i0 + j < count) {
                    const int un = first + (R.reverse ? count - 1 - i0 - j : i0 + j);
                    *reinterpret_cast<float4*>(R.unit_state + ((size_t)un * H + h) * elems + e) = S;
                    S.x = fmaf(S.x, w[j], E[j].x);
                    S.y = fmaf(S.y, w[j], E[j].y);
                    S.z = fmaf(S.z, w[j], E[j].z);
                    S.w = fmaf(S.w, w[j], E[j].w);
                }
        }
        if (R.fin) *reinterpret_cast<float4*>(R.fin + at) = S;
        if (R.fin_dot) {
            const float4 f = *reinterpret_cast<const float4*>(R.fin_dot + at);
            d = (double)S.x * f.x + (double)S.y * f.y + (double)S.z * f.z + (double)S.w * f.w;
        }
    }
    if (R.fin_dot) {
        __shared__ double sd[kScanThreads / 32];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
        if ((threadIdx.x & 31) == 0) sd[threadIdx.x >> 5] = d;
        __syncthreads();
        if (threadIdx.x == 0) {
            double s = 0.0;
            for (int w = 0; w < kScanThreads / 32; ++w) s += sd[w];
            R.fin_dot_out[(size_t)sh * parts + part] = s;
        }
    }
}

// Final states of sequences without tokens (no unit carries them).
__global__ void __launch_bounds__(kScanThreads)
la_empty_kernel(const LaArgs a, int elems) {
    const LaRun& R = a.run[blockIdx.y];
    const int seq = blockIdx.x / a.sp.H;
    if (!R.fin || a.sp.cu[seq + 1] > a.sp.cu[seq]) return;
    const size_t at = (size_t)blockIdx.x * elems;
    for (int e = threadIdx.x; e < elems; e += kScanThreads)
        R.fin[at + e] = R.init ? R.init[at + e] : 0.f;
}

// ------------------------------------------------------------------------------ launch helpers

template <typename T, int DC, int DO, bool kSummary, int NP>
cudaError_t launch_t(const LaArgs& a, cudaStream_t s) {
    using S = RunShape<T, DC, DO, kSummary, NP>;
    auto kern = la_run_kernel<T, DC, DO, kSummary, NP>;
    // (set on every call: the attribute belongs to the current device)
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)S::SMEM);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)(a.sp.units * a.sp.H), a.runs);
    if (a.after) return la_launch_after(kern, grid, S::THREADS, S::SMEM, s, a);
    kern<<<grid, S::THREADS, S::SMEM, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int DC, int DO>
cudaError_t launch_do(const LaArgs& a, bool summary, bool exact, cudaStream_t s) {
    if (summary) return launch_t<T, DC, DO, true, 2>(a, s);
    if constexpr (sizeof(T) == 2)
        if (!exact) return launch_t<T, DC, DO, false, 2>(a, s);
    return launch_t<T, DC, DO, false, 3>(a, s);
}

template <typename T, int DC>
cudaError_t launch_dc(const LaArgs& a, int dout, bool summary, bool exact, cudaStream_t s) {
    switch (dout) {
        case 16: return launch_do<T, DC, 16>(a, summary, exact, s);
        case 32: return launch_do<T, DC, 32>(a, summary, exact, s);
        case 64: return launch_do<T, DC, 64>(a, summary, exact, s);
        case 128:
            // (bf16 heads of 128 x 128 run on tcgen05)
            if constexpr (!(sizeof(T) == 2 && DC == 128))
                return launch_do<T, DC, 128>(a, summary, exact, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_type(const LaArgs& a, int dc, int dout, bool summary, bool exact,
                        cudaStream_t s) {
    switch (dc) {
        case 16: return launch_dc<T, 16>(a, dout, summary, exact, s);
        case 32: return launch_dc<T, 32>(a, dout, summary, exact, s);
        case 64: return launch_dc<T, 64>(a, dout, summary, exact, s);
        case 128: return launch_dc<T, 128>(a, dout, summary, exact, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_la_summary(const LaArgs& a, int dc, int dout, ckda_dtype dtype,
                              cudaStream_t s) {
    if (a.sp.units == 0) return cudaSuccess;
    if (dtype == CKDA_BF16 && dc == 128 && dout == 128) return launch_la_tc_summary(a, s);
    return dtype == CKDA_BF16 ? launch_type<__nv_bfloat16>(a, dc, dout, true, false, s)
                              : launch_type<float>(a, dc, dout, true, false, s);
}

cudaError_t launch_la_run(const LaArgs& a, int dc, int dout, bool exact, ckda_dtype dtype,
                          cudaStream_t s) {
    if (a.sp.units == 0) return cudaSuccess;
    if (dtype == CKDA_BF16 && dc == 128 && dout == 128) return launch_la_tc_run(a, exact, s);
    return dtype == CKDA_BF16 ? launch_type<__nv_bfloat16>(a, dc, dout, false, exact, s)
                              : launch_type<float>(a, dc, dout, false, true, s);
}

int la_scan_parts(int elems) { return (elems / 4 + kScanThreads - 1) / kScanThreads; }

cudaError_t launch_la_scan(const LaArgs& a, int dk, int dv, cudaStream_t s) {
    const int elems = dk * dv, parts = la_scan_parts(elems);
    return la_launch_after(la_scan_kernel, dim3((unsigned)(a.sp.n * a.sp.H * parts), a.runs),
                           kScanThreads, 0, s, a, elems, parts);
}

cudaError_t launch_la_empty(const LaArgs& a, int dk, int dv, cudaStream_t s) {
    la_empty_kernel<<<dim3((unsigned)(a.sp.n * a.sp.H), a.runs), kScanThreads, 0, s>>>(a, dk * dv);
    return cudaGetLastError();
}

}  // namespace ckda
