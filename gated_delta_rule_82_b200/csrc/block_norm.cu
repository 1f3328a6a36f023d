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
#include "common.cuh"
#include "block_norm.cuh"

namespace ckda {

namespace {

constexpr int E = 8;      // channels per thread

enum { kActNone = 0, kActSigmoid = 1, kActSilu = 2 };

// 8 consecutive channels.  kVec: the row starts on a 16-byte boundary and D is a multiple of 8.
template <typename T, bool kVec>
__device__ __forceinline__ void load_e(const T* p, int left, float v[E]) {
    if constexpr (kVec) {
        if (left > 0) {
            if constexpr (sizeof(T) == 2) {
                Vec16<T, 8>::load(p, v);
            } else {
                Vec16<T, 4>::load(p, v);
                Vec16<T, 4>::load(p + 4, v + 4);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = i < left ? to_f32(p[i]) : 0.f;
    }
}
template <typename T, bool kVec>
__device__ __forceinline__ void store_e(T* p, int left, const float v[E]) {
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

// Sums over the threads of one row.  TPR threads hold a row; rows of up to 32 threads stay in a
// warp, longer ones meet in shared memory (one slot per warp, two buffers in turn).
template <int TPR>
struct RowSum {
    float* slots;     // [2][warps of the CTA]
    int turn = 0;
    __device__ __forceinline__ float operator()(float x) {
        x = group_sum<TPR < 32 ? TPR : 32>(x);
        if constexpr (TPR > 32) {
            constexpr int WPR = TPR / 32;
            const int warp = threadIdx.x >> 5;
            float* s = slots + turn * (blockDim.x >> 5);
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

// logistic(z) and 1 - logistic(z), neither by cancellation
__device__ __forceinline__ float2 sigmoid2(float z) {
    const float e = expf(-fabsf(z)), inv = 1.f / (1.f + e);
    return z >= 0.f ? make_float2(inv, e * inv) : make_float2(e * inv, inv);
}

struct Pieces {           // of the forward, per channel
    float yhat[E], u[E], a[E], m[E], h[E];
    float r1;
};

// u, m, h of 8 channels from the loaded rows.
template <int TPR>
__device__ __forceinline__ void forward_row(const BlockNormArgs& p, int D, const float y[E],
                                            const float z[E], const float x[E], const float wp[E],
                                            const float s[E], RowSum<TPR>& row, Pieces& f) {
    if (p.W) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) ss += y[i] * y[i];
        f.r1 = rsqrtf(group_w_sum<TPR>(ss, p.W, D, row) / (float)p.W + p.eps);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
        f.yhat[i] = p.W ? y[i] * f.r1 : y[i];
        f.u[i] = p.W ? f.yhat[i] * wp[i] : y[i];
        f.a[i] = 1.f;
        if (p.gate) {
            const float g = sigmoid2(z[i]).x;
            f.a[i] = p.act == kActSilu ? z[i] * g : g;
        }
        f.m[i] = f.u[i] * f.a[i];
        f.h[i] = x[i] + s[i] * f.m[i];
    }
}

// The per-channel vectors (fp32; their length need not be a multiple of 8).
__device__ __forceinline__ void load_vec(const float* p, int c, int left, int wrap, float dflt,
                                         float v[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i)
        v[i] = p && i < left ? __ldg(p + (wrap ? (c + i) % wrap : c + i)) : dflt;
}

template <typename T, int TPR, bool kVec>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
block_norm_kernel(const BlockNormArgs p) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR, RPC = THREADS / TPR;
    __shared__ float slots[2 * THREADS / 32];
    RowSum<TPR> row_sum{slots};
    const int D = p.D, sub = threadIdx.x / TPR, c = (threadIdx.x % TPR) * E, left = D - c;
    float wp[E], wn[E], s[E];
    load_vec(p.w_post, c, left, p.W, 1.f, wp);
    load_vec(p.w_pre, c, left, 0, 1.f, wn);
    load_vec(p.r, c, left, 0, 1.f, s);
#pragma unroll
    for (int i = 0; i < E; ++i) s[i] *= p.scale;
    // (every thread of a CTA goes through the same number of rows: sums synchronise)
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < p.rows; r0 += (long long)gridDim.x * RPC) {
        const long long r = r0 + sub;
        const bool in = r < p.rows;
        const int l = in ? left : 0;
        const size_t at = (size_t)(in ? r : 0) * D + c;
        float y[E], z[E], x[E];
        load_e<T, kVec>((const T*)p.y + at, l, y);
        load_e<T, kVec>((const T*)p.gate + at, p.gate ? l : 0, z);
        load_e<T, kVec>((const T*)p.x + at, p.x ? l : 0, x);
        Pieces f;
        forward_row<TPR>(p, D, y, z, x, wp, s, row_sum, f);
        store_e<T, kVec>((T*)p.h + at, l, f.h);
        if (p.n) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) ss += i < left ? f.h[i] * f.h[i] : 0.f;
            const float r2 = rsqrtf(row_sum(ss) / (float)D + p.eps);
            float n[E];
#pragma unroll
            for (int i = 0; i < E; ++i) n[i] = f.h[i] * r2 * wn[i];
            store_e<T, kVec>((T*)p.n + at, l, n);
        }
    }
}

template <typename T, int TPR, bool kVec>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
block_norm_bwd_kernel(const BlockNormArgs p, const BlockNormGrads g) {
    constexpr int THREADS = TPR < 128 ? 128 : TPR, RPC = THREADS / TPR;
    __shared__ float slots[2 * THREADS / 32];
    RowSum<TPR> row_sum{slots};
    const int D = p.D, sub = threadIdx.x / TPR, c = (threadIdx.x % TPR) * E, left = D - c;
    float wp[E], wn[E], s[E], dwp[E], dwn[E], dr[E];
    load_vec(p.w_post, c, left, p.W, 1.f, wp);
    load_vec(p.w_pre, c, left, 0, 1.f, wn);
    load_vec(p.r, c, left, 0, 1.f, s);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        s[i] *= p.scale;
        dwp[i] = dwn[i] = dr[i] = 0.f;
    }
    for (long long r0 = (long long)blockIdx.x * RPC; r0 < p.rows; r0 += (long long)gridDim.x * RPC) {
        const long long r = r0 + sub;
        const bool in = r < p.rows;
        const int l = in ? left : 0;
        const size_t at = (size_t)(in ? r : 0) * D + c;
        float y[E], z[E], x[E], dh[E], dn[E];
        load_e<T, kVec>((const T*)p.y + at, l, y);
        load_e<T, kVec>((const T*)p.gate + at, p.gate ? l : 0, z);
        load_e<T, kVec>((const T*)p.x + at, p.x && g.dn ? l : 0, x);
        load_e<T, kVec>((const T*)g.dh + at, g.dh ? l : 0, dh);
        load_e<T, kVec>((const T*)g.dn + at, g.dn ? l : 0, dn);
        Pieces f;
        forward_row<TPR>(p, D, y, z, x, wp, s, row_sum, f);
        if (g.dn) {
            float ss = 0.f, dd = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                ss += i < left ? f.h[i] * f.h[i] : 0.f;
                dd += dn[i] * wn[i] * f.h[i];
            }
            const float r2 = rsqrtf(row_sum(ss) / (float)D + p.eps);
            const float mean = row_sum(dd) * r2 / (float)D;       // mean of dn w hhat
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float hhat = f.h[i] * r2;
                dh[i] += r2 * (dn[i] * wn[i] - hhat * mean);
                dwn[i] += dn[i] * hhat;
            }
        }
        if (g.dx) store_e<T, kVec>((T*)g.dx + at, l, dh);
        float du[E], dz[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (l > 0) dr[i] += dh[i] * f.m[i];
            const float dm = dh[i] * s[i];
            du[i] = dm * f.a[i];
            dz[i] = 0.f;
            if (p.gate) {
                const float2 sg = sigmoid2(z[i]);
                const float slope = p.act == kActSilu ? sg.x * (1.f + z[i] * sg.y) : sg.x * sg.y;
                dz[i] = dm * f.u[i] * slope;
            }
        }
        if (p.gate) store_e<T, kVec>((T*)g.dgate + at, l, dz);
        if (p.W) {
            float dd = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) dd += du[i] * wp[i] * f.yhat[i];
            const float mean = group_w_sum<TPR>(dd, p.W, D, row_sum) / (float)p.W;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                dwp[i] += du[i] * f.yhat[i];
                du[i] = f.r1 * (du[i] * wp[i] - f.yhat[i] * mean);
            }
        }
        store_e<T, kVec>((T*)g.dy + at, l, du);
    }
    // this CTA's sums: [CTA][W], [CTA][D], [CTA][D] for the weights that want one
    __shared__ float fold[THREADS * E];
    float* to = g.partial;
    auto put = [&](const float v[E], int width) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < E; ++i) fold[threadIdx.x * E + i] = v[i];
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
    __shared__ float part[32][33];
    const int k = blockIdx.y, cols = a.cols[k];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
    if (blockIdx.x * 32 >= cols) return;
    float s = 0.f;
    if (c < cols)
        for (int r = ty; r < a.rows; r += 32) s += a.src[k][(size_t)r * cols + c];
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

template <typename T, bool kVec>
cudaError_t launch_fwd(const BlockNormArgs& p, int grid, cudaStream_t s) {
    switch (threads_per_row(p.D)) {
        case 32: block_norm_kernel<T, 32, kVec><<<grid, 128, 0, s>>>(p); break;
        case 64: block_norm_kernel<T, 64, kVec><<<grid, 128, 0, s>>>(p); break;
        case 128: block_norm_kernel<T, 128, kVec><<<grid, 128, 0, s>>>(p); break;
        case 256: block_norm_kernel<T, 256, kVec><<<grid, 256, 0, s>>>(p); break;
        case 512: block_norm_kernel<T, 512, kVec><<<grid, 512, 0, s>>>(p); break;
        default: block_norm_kernel<T, 1024, kVec><<<grid, 1024, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

template <typename T, bool kVec>
cudaError_t launch_bwd(const BlockNormArgs& p, const BlockNormGrads& g, int grid, cudaStream_t s) {
    switch (threads_per_row(p.D)) {
        case 32: block_norm_bwd_kernel<T, 32, kVec><<<grid, 128, 0, s>>>(p, g); break;
        case 64: block_norm_bwd_kernel<T, 64, kVec><<<grid, 128, 0, s>>>(p, g); break;
        case 128: block_norm_bwd_kernel<T, 128, kVec><<<grid, 128, 0, s>>>(p, g); break;
        case 256: block_norm_bwd_kernel<T, 256, kVec><<<grid, 256, 0, s>>>(p, g); break;
        case 512: block_norm_bwd_kernel<T, 512, kVec><<<grid, 512, 0, s>>>(p, g); break;
        default: block_norm_bwd_kernel<T, 1024, kVec><<<grid, 1024, 0, s>>>(p, g); break;
    }
    return cudaGetLastError();
}

}  // namespace

// CTAs of the backward: each keeps the weight gradients of the rows it takes, so there are only
// as many as run side by side (2048 threads per SM at most, and half that by registers).
int block_norm_bwd_grid(long long rows, int D) {
    const int threads = threads_per_row(D) < 128 ? 128 : threads_per_row(D);
    const long long most = 148ll * (threads >= 1024 ? 1 : 1024 / threads);
    const long long need = (rows + rows_per_cta(D) - 1) / rows_per_cta(D);
    return (int)(need < most ? need : most);
}

size_t block_norm_bwd_partial_floats(long long rows, int D, int W) {
    return (size_t)block_norm_bwd_grid(rows, D) * (W + 2 * D);
}

cudaError_t launch_block_norm(const BlockNormArgs& p, ckda_dtype dtype, cudaStream_t s) {
    const long long ctas = (p.rows + rows_per_cta(p.D) - 1) / rows_per_cta(p.D);
    const int threads = threads_per_row(p.D) < 128 ? 128 : threads_per_row(p.D);
    const long long most = 148ll * 2048 / threads;   // (as many as run side by side)
    const int grid = (int)(ctas < most ? ctas : most);
    const bool vec = p.D % E == 0;
    if (dtype == CKDA_BF16)
        return vec ? launch_fwd<__nv_bfloat16, true>(p, grid, s)
                   : launch_fwd<__nv_bfloat16, false>(p, grid, s);
    return vec ? launch_fwd<float, true>(p, grid, s) : launch_fwd<float, false>(p, grid, s);
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
    block_norm_reduce_kernel<<<dim3((widest + 31) / 32, k), 1024, 0, s>>>(r);
    return cudaGetLastError();
}

}  // namespace ckda
