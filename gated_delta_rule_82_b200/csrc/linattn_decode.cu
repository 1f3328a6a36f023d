// linattn_decode.cu -- single-token step of the linear attention, in place on an fp32 state.
//
//     S <- exp(g) S + k v^T,     o = scale * S^T q
//
// Bound by HBM: 8 bytes of state moved per element for 5 flops.  Every output column needs only
// its own column of the state, so a head is cut into strips of up to 32 columns (128-byte row
// pieces) that different groups of threads, and CTAs, work on independently: one sequence of a
// few heads still spreads over the SMs.  A thread holds 8 rows x 4 columns in registers between
// the one read and the one write; the sum over rows goes through shuffles and one shared row per
// warp.  256 sequences x 32 heads of 128 x 128: 157.5 us, 105 % of the measured copy rate (part of
// the state is still in L2); one sequence of 16 heads 2.4 us.
#include "linattn.cuh"

namespace ckda {

namespace {

constexpr int kThreads = 256;
constexpr int R = 8;                                   // state rows per thread

template <int DK, int DV>
struct StepShape {
    static constexpr int CW = DV < 32 ? DV : 32;       // columns per strip
    static constexpr int C4 = CW / 4;                  // threads across a strip
    static constexpr int RG = DK / R;                  // row groups
    static constexpr int TPS = C4 * RG;                // threads per strip: 8 .. 128
    static constexpr int SPC = kThreads / TPS;         // strips per CTA
    static constexpr int PER = DV / CW;                // strips per head
};

__device__ __forceinline__ float4 ld_stream(const float* p) {
    float4 v;
    asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ void st_stream(float* p, float4 v) {
    asm volatile("st.global.cs.v4.f32 [%0], {%1, %2, %3, %4};"
                 :: "l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void load8(const float* p, float x[8]) {
    Vec16<float, 4>::load(p, x);
    Vec16<float, 4>::load(p + 4, x + 4);
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float x[8]) {
    Vec16<__nv_bfloat16, 8>::load(p, x);
}
__device__ __forceinline__ float4 load4(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}

template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kThreads)
la_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const float* __restrict__ g, int per_token, float* __restrict__ state,
                 T* __restrict__ out, long long strips, int H, int G, float scale) {
    using S = StepShape<DK, DV>;
    constexpr int C4 = S::C4, RG = S::RG, TPS = S::TPS;
    const int tid = threadIdx.x, th = tid % TPS, c4 = th % C4, rg = th / C4;
    const long long strip = (long long)blockIdx.x * S::SPC + tid / TPS;
    const bool live = strip < strips;
    const long long head = live ? strip / S::PER : 0;             // sequence * H + head
    const int col = (int)(live ? strip % S::PER : 0) * S::CW + c4 * 4;
    const int h = (int)(head % H);
    float* sp = state + (size_t)head * DK * DV + (size_t)(rg * R) * DV + col;

    float4 s[R];
    if (live) {
#pragma unroll
        for (int j = 0; j < R; ++j) s[j] = ld_stream(sp + (size_t)j * DV);
    }
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live) {
        const long long hq = G == 1 ? head : head / G;            // (H is a multiple of G)
        float qv[R], kv[R];
        load8(q + (size_t)hq * DK + rg * R, qv);
        load8(k + (size_t)hq * DK + rg * R, kv);
        const float4 vv = load4(v + (size_t)head * DV + col);
        const float a = expf(per_token ? g[head] : g[h]);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            s[j].x = fmaf(s[j].x, a, kv[j] * vv.x);
            s[j].y = fmaf(s[j].y, a, kv[j] * vv.y);
            s[j].z = fmaf(s[j].z, a, kv[j] * vv.z);
            s[j].w = fmaf(s[j].w, a, kv[j] * vv.w);
            st_stream(sp + (size_t)j * DV, s[j]);
            y.x = fmaf(s[j].x, qv[j], y.x);
            y.y = fmaf(s[j].y, qv[j], y.y);
            y.z = fmaf(s[j].z, qv[j], y.z);
            y.w = fmaf(s[j].w, qv[j], y.w);
        }
    }
    // sum over the row groups: those of this warp by shuffles, then one partial per warp
    constexpr int IN_WARP = TPS < 32 ? RG : 32 / C4;              // row groups of a strip in a warp
#pragma unroll
    for (int o = C4 * IN_WARP / 2; o >= C4; o >>= 1) {
        y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
        y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
        y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
        y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
    }
    if constexpr (TPS > 32) {
        __shared__ float4 part[kThreads / 32][C4];
        const int lane = tid & 31, warp = tid >> 5;
        if (lane < C4) part[warp][lane] = y;
        __syncthreads();
        if (rg != 0) return;
        const int w0 = (tid / TPS) * (TPS / 32);
        y = part[w0][c4];
#pragma unroll
        for (int w = 1; w < TPS / 32; ++w) {
            const float4 p = part[w0 + w][c4];
            y.x += p.x; y.y += p.y; y.z += p.z; y.w += p.w;
        }
    }
    if (live && rg == 0) {
        T* o = out + (size_t)head * DV + col;
        o[0] = from_f32<T>(scale * y.x);
        o[1] = from_f32<T>(scale * y.y);
        o[2] = from_f32<T>(scale * y.z);
        o[3] = from_f32<T>(scale * y.w);
    }
}

template <typename T, int DK, int DV>
cudaError_t step_t(const void* q, const void* k, const void* v, const float* g, int per_token,
                   float* state, void* out, int N, int H, int G, float scale, cudaStream_t s) {
    using S = StepShape<DK, DV>;
    const long long strips = (long long)N * H * S::PER;
    la_decode_kernel<T, DK, DV><<<(unsigned)((strips + S::SPC - 1) / S::SPC), kThreads, 0, s>>>(
        (const T*)q, (const T*)k, (const T*)v, g, per_token, state, (T*)out, strips, H, G, scale);
    return cudaGetLastError();
}

template <typename T, int DK>
cudaError_t step_dv(int dv, const void* q, const void* k, const void* v, const float* g,
                    int per_token, float* state, void* out, int N, int H, int G, float scale,
                    cudaStream_t s) {
    switch (dv) {
        case 16: return step_t<T, DK, 16>(q, k, v, g, per_token, state, out, N, H, G, scale, s);
        case 32: return step_t<T, DK, 32>(q, k, v, g, per_token, state, out, N, H, G, scale, s);
        case 64: return step_t<T, DK, 64>(q, k, v, g, per_token, state, out, N, H, G, scale, s);
        case 128: return step_t<T, DK, 128>(q, k, v, g, per_token, state, out, N, H, G, scale, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t step_dk(int dk, int dv, const void* q, const void* k, const void* v, const float* g,
                    int per_token, float* state, void* out, int N, int H, int G, float scale,
                    cudaStream_t s) {
    switch (dk) {
        case 16: return step_dv<T, 16>(dv, q, k, v, g, per_token, state, out, N, H, G, scale, s);
        case 32: return step_dv<T, 32>(dv, q, k, v, g, per_token, state, out, N, H, G, scale, s);
        case 64: return step_dv<T, 64>(dv, q, k, v, g, per_token, state, out, N, H, G, scale, s);
        case 128: return step_dv<T, 128>(dv, q, k, v, g, per_token, state, out, N, H, G, scale, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_la_decode(const void* q, const void* k, const void* v, const float* g,
                             int per_token, float* state, void* out, int N, int H, int G, int dk,
                             int dv, float scale, ckda_dtype dtype, cudaStream_t s) {
    return dtype == CKDA_BF16
               ? step_dk<__nv_bfloat16>(dk, dv, q, k, v, g, per_token, state, out, N, H, G, scale, s)
               : step_dk<float>(dk, dv, q, k, v, g, per_token, state, out, N, H, G, scale, s);
}

}  // namespace ckda
