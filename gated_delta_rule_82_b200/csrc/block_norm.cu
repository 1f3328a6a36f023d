// block_norm.cu -- the norms around a block, fused with its gate, its scale and the residual add.
//
// For rows of D channels (s = scale * r[channel], groups of W channels):
//     u = y rsqrt(mean_W y^2 + eps) w_post        (group norm after the block; W = 0: u = y)
//     m = u act(gate),   h = x + s m              (gate, residual x and r optional)
//     n = h rsqrt(mean_D h^2 + eps) w_pre         (norm before the next block, optional)
// and the reverse mode, which forms all of that again from the inputs (no statistics are stored):
//     dH = dh + r2 (dn w_pre - hhat mean_D(dn w_pre hhat)),    dx = dH,   dr = sum_rows scale dH m
//     du = s dH act(gate),   dgate = s dH u act'(gate)
//     dy = r1 (du w_post - yhat mean_W(du w_post yhat))
//     dw_pre = sum_rows dn hhat,   dw_post = sum_rows and groups du yhat
//
// Bound by HBM: every array crosses once.  A row lives in the registers of 32 .. 1024 threads
// (8 channels each, 16-byte accesses for 2-byte types), so one pass serves both norms; sums are
// fp32.  The weight gradients are kept per thread over the rows its CTA takes, written once per
// CTA and added up by a second launch in a fixed order (no atomics).
// Forward, 65536 x 2048 bf16 with all parts: 226 us, 91 % of the measured copy rate; 4096 rows with the
// head norm and a gate 13.3 us.  The backward holds four to six arrays of a row in registers: two
// CTAs of 256 threads an SM (128 registers), 54 us + 6 for 4096 x 2048, 36 % of the copy rate, bound
// by the latency of loads and sums (4 channels a thread 66 us; three CTAs an SM, with spills, 89).
#include "common.cuh"
#include "block_norm.cuh"
#include "linattn.cuh"        // la_launch_after

namespace ckda {

namespace {

constexpr int E = 8;      // channels per thread

enum { kActNone = 0, kActSigmoid = 1, kActSilu = 2 };

// 8 consecutive channels as they lie in memory, so that a row that is requested ahead costs few
// registers.  kVec: rows start on 16-byte boundaries and D is a multiple of 8.
template <typename T, bool kVec>
struct Raw {
    static constexpr int N = kVec ? 8 * (int)sizeof(T) / 16 : 1;
    uint4 w[N];
    T e[kVec ? 1 : E];

    __device__ __forceinline__ void load(const void* base, size_t at, int left) {
        const T* p = static_cast<const T*>(base) + at;
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                w[i] = left > 0 ? *reinterpret_cast<const uint4*>(p + i * (16 / (int)sizeof(T)))
                                : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) e[i] = i < left ? p[i] : from_f32<T>(0.f);
        }
    }
    __device__ __forceinline__ void clear() {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) e[i] = from_f32<T>(0.f);
        }
    }
    // channel i (a constant after unrolling)
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (!kVec) return to_f32(e[i]);
        if constexpr (kVec && sizeof(T) == 4) {
            const uint4& q = w[i >> 2];
            return __uint_as_float((i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w);
        }
        if constexpr (kVec && sizeof(T) == 2) {
            const uint4& q = w[0];
            const uint32_t x = (i >> 1) == 0 ? q.x : (i >> 1) == 1 ? q.y : (i >> 1) == 2 ? q.z : q.w;
            return __uint_as_float(i & 1 ? x & 0xffff0000u : x << 16);
        }
        return 0.f;
    }
};
template <typename T, bool kVec>
__device__ __forceinline__ void store_e(void* base, size_t at, int left, const float v[E]) {
    T* p = static_cast<T*>(base) + at;
    if constexpr (kVec) {
        if (left > 0) {
            if constexpr (sizeof(T) == 2) {
                Vec16<T, 8>::store(p, v);
            } else {
                Vec16<T, 4>::store(p, v);
                Vec16<T, 4>::store(p + 4, v + 4);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (i < left) p[i] = from_f32<T>(v[i]);
    }
}

// Sums over the threads of one row, one or two values at a time.  TPR threads hold a row; rows of up
// to 32 threads stay in a warp, longer ones meet in shared memory (one slot per warp, two buffers in
// turn).
template <int TPR>
struct RowSum {
    float2* slots;    // [2][warps of the CTA]
    int turn = 0;
    __device__ __forceinline__ float2 both(float2 x) {
        x.x = group_sum<TPR < 32 ? TPR : 32>(x.x);
        x.y = group_sum<TPR < 32 ? TPR : 32>(x.y);
        if constexpr (TPR > 32) {
            constexpr int WPR = TPR / 32;
            const int warp = threadIdx.x >> 5;
            float2* s = slots + turn * (blockDim.x >> 5);
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) s[warp] = x;
            __syncthreads();
            const int w0 = warp / WPR * WPR;
            x = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WPR; ++w) {
                const float2 y = s[w0 + w];
                x.x += y.x;
                x.y += y.y;
            }
        }
        return x;
    }
    __device__ __forceinline__ float operator()(float x) {
        x = group_sum<TPR < 32 ? TPR : 32>(x);
        if constexpr (TPR > 32) {
            constexpr int WPR = TPR / 32;
            const int warp = threadIdx.x >> 5;
            float* s = reinterpret_cast<float*>(slots + turn * (blockDim.x >> 5));
            turn ^= 1;
            if ((threadIdx.x & 31) == 0) s[warp] = x;
            __syncthreads();
            const int w0 = warp / WPR * WPR;
            x = 0.f;
#pragma unroll
            for (int w = 0; w < WPR; ++w) x += s[w0 + w];
        }
        return x;
    }
};
// Sums over groups of W channels: W / 8 neighbouring threads (W = 16 .. 128), or the row.
template <int TPR>
__device__ __forceinline__ float group_w_sum(float x, int W, int D, RowSum<TPR>& row) {
    if (W == D) return row(x);
    for (int o = W / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// 2^x and 1 / x of the special function unit (about 2^-22 relative): with the exact forms the gate
// took 40 of 67 instructions per channel, and the kernel was bound by them, not by memory.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp(-z).  For fp32 results the product z log2(e) is kept in two parts: its rounding, |z| 2^-24,
// would be the largest error.
template <typename T>
__device__ __forceinline__ float exp_neg(float z) {
    const float kL = -1.44269504f;
    const float h = z * kL;
    if constexpr (sizeof(T) == 2) return ex2(h);
    // (-inf and overflow: nothing to correct)
    const float l = fmaf(z, kL, -h), e = ex2(h);
    return fabsf(h) < 120.f ? fmaf(e, l * 0.693147181f, e) : e;
}
// logistic(z)
template <typename T>
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + exp_neg<T>(z)); }
// logistic(z) and 1 - logistic(z), neither by cancellation
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float z) {
    const float e = exp_neg<T>(fabsf(z)), inv = rcp(1.f + e);
    return z >= 0.f ? make_float2(inv, e * inv) : make_float2(e * inv, inv);
}

// Weight vectors (fp32) in shared memory: [post][pre][s], the post weight once per row group of the
// row, ones where a vector is missing; loaded by the whole CTA.
struct Weights {
    float *post, *pre, *s;
    __device__ __forceinline__ void load(const BlockNormArgs& p, float* base) {
        const int D = p.D;
        post = base;
        pre = post + (p.W ? D : 0);
        s = pre + (p.w_pre ? D : 0);
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            if (p.W) post[c] = p.w_post ? __ldg(p.w_post + (p.W == D ? c : c & (p.W - 1))) : 1.f;
            if (p.w_pre) pre[c] = __ldg(p.w_pre + c);
            if (p.r) s[c] = __ldg(p.r + c) * p.scale;
        }
        __syncthreads();
    }
};
size_t weights_floats(const BlockNormArgs& p) {
    return (size_t)p.D * ((p.W != 0) + (p.w_pre != nullptr) + (p.r != nullptr));
}
// channel c + i of a vector in shared memory (rows of 8: two 16-byte reads)
template <bool kVec>
__device__ __forceinline__ void take(const float* v, int c, int left, float w[E]) {
    if constexpr (kVec) {
        if (left > 0) {
            Vec16<float, 4>::load(v + c, w);
            Vec16<float, 4>::load(v + c + 4, w + 4);
            return;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = i < left ? v[c + i] : 0.f;
    }
}

// The gate's factor.
template <typename T, int kAct>
__device__ __forceinline__ float gate_of(float z) {
    const float g = sigmoid<T>(z);
    return kAct == kActSilu ? z * g : g;
}

// The root of the first norm for this thread's group, and m (the gated value) of its 8 channels.
template <typename T, int TPR, bool kVec>
__device__ __forceinline__ float first_norm(const BlockNormArgs& p, const Raw<T, kVec>& y, float inv_w,
                                            RowSum<TPR>& row) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) ss += y[i] * y[i];
    return rsqrtf(group_w_sum<TPR>(ss, p.W, p.D, row) * inv_w + p.eps);
}

template <int TPR>
constexpr int threads_of() { return TPR < 128 ? 128 : TPR; }
// CTAs per SM that the register budget is set for: the kernels live on loads in flight
template <int TPR>
constexpr int fwd_ctas() { return 1024 / threads_of<TPR>(); }
template <int TPR>
constexpr int bwd_ctas() { return TPR >= 1024 ? 1 : 512 / threads_of<TPR>(); }

template <typename T, int TPR, bool kVec, int kAct>
__global__ void __launch_bounds__(threads_of<TPR>(), fwd_ctas<TPR>())
block_norm_kernel(const BlockNormArgs p) {
    constexpr int THREADS = threads_of<TPR>(), RPC = THREADS / TPR;
    extern __shared__ __align__(16) float sw[];
    __shared__ float2 slots[2 * THREADS / 32];
    RowSum<TPR> row_sum{slots};
    const int D = p.D, sub = threadIdx.x / TPR, c = (threadIdx.x % TPR) * E, left = D - c;
    const float inv_w = 1.f / (float)(p.W ? p.W : 1), inv_d = 1.f / (float)D;
    const long long step = (long long)gridDim.x * RPC;
    long long r = (long long)blockIdx.x * RPC + sub;
    // the first row is requested before the weights are waited for, every other one a row ahead
    Raw<T, kVec> y, z, x;
    auto request = [&](long long row, Raw<T, kVec>& y, Raw<T, kVec>& z, Raw<T, kVec>& x) {
        const int l = row < p.rows ? left : 0;
        const size_t at = (size_t)(row < p.rows ? row : 0) * D + c;
        y.load(p.y, at, l);
        if constexpr (kAct != kActNone) z.load(p.gate, at, l);
        if (p.x) x.load(p.x, at, l);
    };
    z.clear();
    x.clear();
    request(r, y, z, x);
    Weights w;
    w.load(p, sw);
    // (every thread of a CTA goes through the same number of rows: sums synchronise)
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < p.rows; r0 += step, r += step) {
        const int l = r < p.rows ? left : 0;
        const size_t at = (size_t)(r < p.rows ? r : 0) * D + c;
        Raw<T, kVec> ny, nz, nx;
        nz.clear();
        nx.clear();
        if (r0 + step < p.rows) request(r + step, ny, nz, nx);
        float h[E], v[E];
        if (p.W) {
            const float r1 = first_norm<T, TPR, kVec>(p, y, inv_w, row_sum);
            take<kVec>(w.post, c, left, v);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] = y[i] * r1 * v[i];
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] = y[i];
        }
        if constexpr (kAct != kActNone) {
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] *= gate_of<T, kAct>(z[i]);
        }
        if (p.r) {
            take<kVec>(w.s, c, left, v);
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] = x[i] + v[i] * h[i];
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) h[i] = x[i] + p.scale * h[i];
        }
        store_e<T, kVec>(p.h, at, l, h);
        if (p.n) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) ss += h[i] * h[i];
            const float r2 = rsqrtf(row_sum(ss) * inv_d + p.eps);
            if (p.w_pre) {
                take<kVec>(w.pre, c, left, v);
#pragma unroll
                for (int i = 0; i < E; ++i) h[i] *= r2 * v[i];
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) h[i] *= r2;
            }
            store_e<T, kVec>(p.n, at, l, h);
        }
        y = ny;
        z = nz;
        x = nx;
    }
}

template <typename T, int TPR, bool kVec, int kAct>
__global__ void __launch_bounds__(threads_of<TPR>(), bwd_ctas<TPR>())
block_norm_bwd_kernel(const BlockNormArgs p, const BlockNormGrads g) {
    la_let_next_start();
    constexpr int THREADS = threads_of<TPR>(), RPC = THREADS / TPR;
    extern __shared__ __align__(16) float sw[];
    __shared__ float2 slots[2 * THREADS / 32];
    RowSum<TPR> row_sum{slots};
    const int D = p.D, sub = threadIdx.x / TPR, c = (threadIdx.x % TPR) * E, left = D - c;
    const float inv_w = 1.f / (float)(p.W ? p.W : 1), inv_d = 1.f / (float)D;
    float dwp[E], dwn[E], dr[E];
#pragma unroll
    for (int i = 0; i < E; ++i) dwp[i] = dwn[i] = dr[i] = 0.f;
    Weights w;
    w.load(p, sw);
    const long long step = (long long)gridDim.x * RPC;
    // (2-byte types: the next row's arrays wait in 20 registers while this one is worked on)
    constexpr bool kAhead = sizeof(T) == 2 && kVec;
    constexpr bool kGate = kAct != kActNone, silu = kAct == kActSilu;
    Raw<T, kVec> y, z, x, rh, rn, ny, nz, nx, nrh, nrn;
    auto request = [&](long long row, Raw<T, kVec>& y, Raw<T, kVec>& z, Raw<T, kVec>& x, Raw<T, kVec>& rh,
                       Raw<T, kVec>& rn) {
        const int l = row < p.rows ? left : 0;
        const size_t at = (size_t)(row < p.rows ? row : 0) * D + c;
        y.load(p.y, at, l);
        if constexpr (kGate) z.load(p.gate, at, l);
        if (g.dn) rn.load(g.dn, at, l);
        if (g.dn && p.x) x.load(p.x, at, l);
        if (g.dh) rh.load(g.dh, at, l);
    };
    z.clear(); x.clear(); rh.clear(); rn.clear();
    nz.clear(); nx.clear(); nrh.clear(); nrn.clear();
    if constexpr (kAhead) request((long long)blockIdx.x * RPC + sub, ny, nz, nx, nrh, nrn);
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < p.rows; r0 += step) {
        const long long r = r0 + sub;
        const int l = r < p.rows ? left : 0;
        const size_t at = (size_t)(r < p.rows ? r : 0) * D + c;
        if constexpr (kAhead) {
            y = ny; z = nz; x = nx; rh = nrh; rn = nrn;
            if (r0 + step < p.rows) request(r + step, ny, nz, nx, nrh, nrn);
        } else {
            request(r, y, z, x, rh, rn);
        }
        // the forward's values again: yhat, the gate's logistic and its complement, s
        float r1 = 1.f, yh[E], sg[E], sm[E], s[E], v[E], dh[E];
        if (p.W) {
            r1 = first_norm<T, TPR, kVec>(p, y, inv_w, row_sum);
#pragma unroll
            for (int i = 0; i < E; ++i) yh[i] = y[i] * r1;
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) yh[i] = y[i];
        }
        float wp[E];
        if (p.W) {
            take<kVec>(w.post, c, left, wp);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) wp[i] = 1.f;
        }
        if (p.r) {
            take<kVec>(w.s, c, left, s);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) s[i] = p.scale;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) {
            dh[i] = rh[i];
            const float2 g2 = kGate ? sigmoid2<T>(z[i]) : make_float2(1.f, 0.f);
            sg[i] = g2.x;
            sm[i] = g2.y;
        }
        if (g.dn) {
            float h[E];
            float2 t = make_float2(0.f, 0.f);                     // h^2, dn w h
            if (p.w_pre) {
                take<kVec>(w.pre, c, left, v);
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < E; ++i) {
                v[i] *= rn[i];
                h[i] = x[i] + s[i] * (yh[i] * wp[i] * (silu ? z[i] * sg[i] : sg[i]));
                t.x += h[i] * h[i];
                t.y += v[i] * h[i];
            }
            t = row_sum.both(t);
            const float r2 = rsqrtf(t.x * inv_d + p.eps), mean = t.y * r2 * inv_d;   // of dn w hhat
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float hhat = h[i] * r2;
                dh[i] += r2 * (v[i] - hhat * mean);
                dwn[i] += rn[i] * hhat;
            }
        }
        if (g.dx) store_e<T, kVec>(g.dx, at, l, dh);
        // dh becomes the gradient of u; the gate's gradient goes out on the way
        float dd = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float u = yh[i] * wp[i], f = silu ? z[i] * sg[i] : sg[i];
            dr[i] += dh[i] * (u * f);
            dh[i] *= s[i];
            if constexpr (kGate) v[i] = dh[i] * u * (silu ? sg[i] + f * sm[i] : sg[i] * sm[i]);
            dh[i] *= f;
            dd += dh[i] * wp[i] * yh[i];
        }
        if constexpr (kGate) store_e<T, kVec>(g.dgate, at, l, v);
        if (p.W) {
            const float mean = group_w_sum<TPR>(dd, p.W, D, row_sum) * inv_w;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                dwp[i] += dh[i] * yh[i];
                dh[i] = r1 * (dh[i] * wp[i] - yh[i] * mean);
            }
        }
        store_e<T, kVec>(g.dy, at, l, dh);
    }
    // this CTA's sums: [CTA][W], [CTA][D], [CTA][D] for the weights that want one
    __syncthreads();
    float* fold = sw;         // (the weights are done with; the launch leaves room for both)
    float* to = g.partial;
    auto put = [&](const float v[E], int width) {
        __syncthreads();
        Vec16<float, 4>::store(fold + threadIdx.x * E, v);
        Vec16<float, 4>::store(fold + threadIdx.x * E + 4, v + 4);
        __syncthreads();
        for (int k = threadIdx.x; k < width; k += THREADS) {
            float t = 0.f;
            for (int r = 0; r < RPC; ++r)
                for (int j = k; j < D; j += width) t += fold[r * TPR * E + j];
            to[(size_t)blockIdx.x * width + k] = t;
        }
        to += (size_t)gridDim.x * width;
    };
    if (g.dw_post) put(dwp, p.W);
    if (g.dw_pre) put(dwn, D);
    if (g.dr) {
#pragma unroll
        for (int i = 0; i < E; ++i) dr[i] *= p.scale;
        put(dr, D);
    }
}

// Column sums of the partials, [rows][cols] each: 32 columns per CTA, a warp per row in turn.
struct ReduceArgs {
    const float* src[3];
    float* dst[3];
    int cols[3], rows;
};
__global__ void __launch_bounds__(1024)
block_norm_reduce_kernel(const ReduceArgs a) {
    la_wait_before();
    __shared__ float part[32][33];
    const int k = blockIdx.y, cols = a.cols[k];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    if (blockIdx.x * 32 >= cols) return;
    float s = 0.f;
    if (c < cols) {
        const float* p = a.src[k] + c;
        int r = ty;
        for (; r + 96 < a.rows; r += 128) {       // four rows in flight
            const float a0 = p[(size_t)r * cols], a1 = p[(size_t)(r + 32) * cols];
            const float a2 = p[(size_t)(r + 64) * cols], a3 = p[(size_t)(r + 96) * cols];
            s += (a0 + a1) + (a2 + a3);
        }
        for (; r < a.rows; r += 32) s += p[(size_t)r * cols];
    }
    part[ty][tx] = s;
    __syncthreads();
    s = warp_sum(part[tx][ty]);
    if (tx == 0 && blockIdx.x * 32 + ty < cols) a.dst[k][blockIdx.x * 32 + ty] = s;
}

// Threads per row: a power of two that covers D with 8 channels each.
int threads_per_row(int D) {
    int t = 32;
    while (t * E < D) t *= 2;
    return t;
}

int rows_per_cta(int D) {
    const int t = threads_per_row(D);
    return t < 128 ? 128 / t : 1;
}

// Dynamic shared memory above the default needs the attribute, per kernel and device.  Always for the
// most that rows of TPR threads can ask for (three weight vectors): set to a call's own need, it fell
// below that of a call that another host thread was about to launch.
template <int TPR, typename K>
cudaError_t room(K kern) {
    constexpr int kMost = 3 * TPR * E * (int)sizeof(float);
    return kMost > 40 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost)
                             : cudaSuccess;
}

template <typename T, int TPR, bool kVec>
cudaError_t fwd_t(const BlockNormArgs& p, cudaStream_t s) {
    constexpr int THREADS = threads_of<TPR>(), RPC = THREADS / TPR;
    const long long ctas = (p.rows + RPC - 1) / RPC, most = 148ll * fwd_ctas<TPR>();
    const size_t smem = weights_floats(p) * sizeof(float);
    auto kern = p.act == kActSilu      ? block_norm_kernel<T, TPR, kVec, kActSilu>
                : p.act == kActSigmoid ? block_norm_kernel<T, TPR, kVec, kActSigmoid>
                                       : block_norm_kernel<T, TPR, kVec, kActNone>;
    const cudaError_t e = room<TPR>(kern);
    if (e != cudaSuccess) return e;
    kern<<<(int)(ctas < most ? ctas : most), THREADS, smem, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int TPR, bool kVec>
cudaError_t bwd_t(const BlockNormArgs& p, const BlockNormGrads& g, int grid, cudaStream_t s) {
    constexpr int THREADS = threads_of<TPR>();
    const size_t wb = weights_floats(p) * sizeof(float), fb = (size_t)THREADS * E * sizeof(float);
    const size_t smem = wb > fb ? wb : fb;
    auto kern = p.act == kActSilu      ? block_norm_bwd_kernel<T, TPR, kVec, kActSilu>
                : p.act == kActSigmoid ? block_norm_bwd_kernel<T, TPR, kVec, kActSigmoid>
                                       : block_norm_bwd_kernel<T, TPR, kVec, kActNone>;
    const cudaError_t e = room<TPR>(kern);
    if (e != cudaSuccess) return e;
    kern<<<grid, THREADS, smem, s>>>(p, g);
    return cudaGetLastError();
}

template <typename T, bool kVec>
cudaError_t launch_fwd(const BlockNormArgs& p, cudaStream_t s) {
    switch (threads_per_row(p.D)) {
        case 32: return fwd_t<T, 32, kVec>(p, s);
        case 64: return fwd_t<T, 64, kVec>(p, s);
        case 128: return fwd_t<T, 128, kVec>(p, s);
        case 256: return fwd_t<T, 256, kVec>(p, s);
        case 512: return fwd_t<T, 512, kVec>(p, s);
        default: return fwd_t<T, 1024, kVec>(p, s);
    }
}

template <typename T, bool kVec>
cudaError_t launch_bwd(const BlockNormArgs& p, const BlockNormGrads& g, int grid, cudaStream_t s) {
    switch (threads_per_row(p.D)) {
        case 32: return bwd_t<T, 32, kVec>(p, g, grid, s);
        case 64: return bwd_t<T, 64, kVec>(p, g, grid, s);
        case 128: return bwd_t<T, 128, kVec>(p, g, grid, s);
        case 256: return bwd_t<T, 256, kVec>(p, g, grid, s);
        case 512: return bwd_t<T, 512, kVec>(p, g, grid, s);
        default: return bwd_t<T, 1024, kVec>(p, g, grid, s);
    }
}

}  // namespace

// CTAs of the backward: each keeps the weight gradients of the rows it takes, so there are only
// as many as run side by side.
int block_norm_bwd_grid(long long rows, int D) {
    const int threads = threads_per_row(D) < 128 ? 128 : threads_per_row(D);
    const long long most = 148ll * (threads >= 1024 ? 1 : 512 / threads);
    const long long need = (rows + rows_per_cta(D) - 1) / rows_per_cta(D);
    return (int)(need < most ? need : most);
}

size_t block_norm_bwd_partial_floats(long long rows, int D, int W) {
    return (size_t)block_norm_bwd_grid(rows, D) * (W + 2 * D);
}

cudaError_t launch_block_norm(const BlockNormArgs& p, ckda_dtype dtype, cudaStream_t s) {
    const bool vec = p.D % E == 0;
    if (dtype == CKDA_BF16)
        return vec ? launch_fwd<__nv_bfloat16, true>(p, s) : launch_fwd<__nv_bfloat16, false>(p, s);
    return vec ? launch_fwd<float, true>(p, s) : launch_fwd<float, false>(p, s);
}

cudaError_t launch_block_norm_bwd(const BlockNormArgs& p, const BlockNormGrads& g,
                                  ckda_dtype dtype, cudaStream_t s) {
    const int grid = block_norm_bwd_grid(p.rows, p.D);
    const bool vec = p.D % E == 0;
    cudaError_t e;
    if (dtype == CKDA_BF16)
        e = vec ? launch_bwd<__nv_bfloat16, true>(p, g, grid, s)
                : launch_bwd<__nv_bfloat16, false>(p, g, grid, s);
    else
        e = vec ? launch_bwd<float, true>(p, g, grid, s) : launch_bwd<float, false>(p, g, grid, s);
    if (e != cudaSuccess) return e;
    ReduceArgs r = {};
    r.rows = grid;
    int k = 0, widest = 0;
    const float* src = g.partial;
    auto add = [&](float* dst, int cols) {
        if (!dst) return;
        r.src[k] = src;
        r.dst[k] = dst;
        r.cols[k] = cols;
        widest = cols > widest ? cols : widest;
        ++k;
        src += (size_t)grid * cols;
    };
    add(g.dw_post, p.W);
    add(g.dw_pre, p.D);
    add(g.dr, p.D);
    if (k == 0) return cudaSuccess;
    // (it starts as the backward's CTAs leave; before that they fill the SMs)
    return la_launch_after(block_norm_reduce_kernel, dim3((widest + 31) / 32, k), 1024, 0, s, r);
}

}  // namespace ckda
