// linattn.cuh -- linear attention with a decay for each head: shared declarations.
//
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t       (S in R^{dk x dv})
//
// and its gradients, which are three more runs of the same recurrence (with R_t the gradient with
// respect to S_t, carried backwards in time):
//     dq_t = scale S_t do_t              a forward run  with (q, k, v) -> (do, v, k), state S^T
//     dv_t = R_t^T k_t                   a backward run with (q, k, v) -> (k, q, do), state R
//     dk_t = R_t v_t                     a backward run with (q, k, v) -> (v, do, q), state R^T
//     R_t  = exp(g_{t+1}) R_{t+1} + scale q_t do_t^T
//     dg_t = <R_t, exp(g_t) S_{t-1}>,    dg_t - dg_{t+1} = q_t.dq_t - k_t.dk_t
#pragma once

#include "common.cuh"
#include "linattn_units.h"

namespace ckda {

// Launch with programmatic stream serialisation: the grid may start while its predecessor in the
// stream still runs, and calls la_wait_before() ahead of everything that the predecessor wrote (or
// still reads).  The first launch of a call is an ordinary one, so the inputs are complete by then.
template <typename... P, typename... A>
cudaError_t la_launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                            A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kern, args...);
}
__device__ __forceinline__ void la_let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void la_wait_before() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// How the token axis is cut: sequences (batched rows of T tokens, or packed ones) into units of
// at most L tokens (a multiple of kLaChunk) that are worked on side by side.
struct LaSplit {
    const int* cu;       // device token offsets [n + 1] of packed sequences, or nullptr
    int n;               // sequences
    int T;               // tokens of one batched row (cu == nullptr), else of the token axis
    int L;               // tokens per unit
    int units;           // units of all sequences (from the host's offsets)
    int H;               // value heads
    int empty;           // a packed sequence has no tokens
};

// One run of the recurrence.  x, y, z play q, k, v: [token][heads][dim], value head h reads head
// h / group of an operand.  The state is addressed in its [dk][dv] layout, row = output dim,
// column = contracted dim.
struct LaRun {
    const void *x, *y, *z;
    int xg, yg, zg;              // value heads per head of the operand
    void* out;                   // [token][H][output dim]
    int out_f32;                 // out is fp32 whatever the input type
    const float* init;           // state entering the run per (sequence, head), or nullptr (zero)
    float* fin;                  // state leaving it, or nullptr
    const float* fin_dot;        // per (sequence, head) state to multiply the leaving state with
    double* fin_dot_out;         // <fin_dot, leaving state> per (sequence, head)
    float* unit_state;           // per (unit, head): summary, then the entering state; or nullptr
    double* unit_decay;          // per (unit, head): sum of log2 decays
    int fold;                    // unit_state holds summaries: a run adds up those ahead of its unit
    int transposed;              // output dim is dk (rows of the state in memory), not dv
    int reverse;                 // runs from the last token to the first
    float p_scale, u_scale, o_scale;   // on the chunk's own products, the state update, the read-out
    const void* dot;             // rows [token][H / dg][output dim] whose products with the output
    int dg;                      // rows are written to dot_out[token][H], or nullptr
    double* dot_out;
    double* dot_sum;             // sums of those products over every chunk, by la_chunk_id
};
constexpr int kLaMaxRuns = 3;

struct LaArgs {
    LaSplit sp;
    const float* g;              // log decays [token][H], or [H]
    int per_token;
    LaRun run[kLaMaxRuns];
    int runs;
    int after;                   // not the first launch of the call (la_launch_after)
};

// Where a unit lies: its sequence, its first token on the token axis, its length.
struct UnitAt {
    int seq, len, index, count;     // index: number among the sequence's `count` units
    long long tok;
    bool ok;
};
// Packed sequences: a warp counts units 32 sequences at a time.  Offsets are taken from device
// memory but clamped to the token axis, and a unit that they do not yield is skipped, so that
// offsets that differ from the host's cannot lead outside the arrays.
__device__ inline UnitAt find_unit(const LaSplit& sp, int unit) {
    UnitAt u{0, 0, 0, 0, 0, false};
    if (!sp.cu) {
        const int per = (sp.T + sp.L - 1) / sp.L;
        u.seq = unit / per;
        u.index = unit - u.seq * per;
        u.tok = (long long)u.seq * sp.T + (long long)u.index * sp.L;
        u.len = min(sp.L, sp.T - u.index * sp.L);
        u.count = per;
        u.ok = true;
        return u;
    }
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int s0 = 0; s0 < sp.n; s0 += 32) {
        int a = 0, b = 0;
        if (s0 + lane < sp.n) {
            a = min(max(sp.cu[s0 + lane], 0), sp.T);
            b = min(max(sp.cu[s0 + lane + 1], a), sp.T);
        }
        const int mine = (b - a + sp.L - 1) / sp.L;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const bool here = unit >= before + upto - mine && unit < before + upto;
        const unsigned who = __ballot_sync(0xffffffffu, here);
        if (who) {
            const int w = __ffs(who) - 1;
            u.seq = s0 + w;
            u.index = unit - before - __shfl_sync(0xffffffffu, upto - mine, w);
            const int a0 = __shfl_sync(0xffffffffu, a, w), b0 = __shfl_sync(0xffffffffu, b, w);
            u.tok = (long long)a0 + (long long)u.index * sp.L;
            u.len = (int)min((long long)sp.L, b0 - u.tok);
            u.count = (b0 - a0 + sp.L - 1) / sp.L;
            u.ok = true;
            return u;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return u;
}
// First unit and unit count of a sequence (all threads of a warp call it).
__device__ inline void seq_units(const LaSplit& sp, int seq, int* first, int* count) {
    if (!sp.cu) {
        *count = (sp.T + sp.L - 1) / sp.L;
        *first = seq * *count;
        return;
    }
    const int lane = threadIdx.x & 31;
    int before = 0, own = 0;
    for (int s0 = 0; s0 <= seq; s0 += 32) {
        const int s = s0 + lane;
        int m = 0;
        if (s <= seq) {
            const int a = min(max(sp.cu[s], 0), sp.T), b = min(max(sp.cu[s + 1], a), sp.T);
            m = (b - a + sp.L - 1) / sp.L;
        }
        if (s == seq) own = m;
        if (s < seq) before = la_add_units(before, m, sp.units);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        before = la_add_units(before, __shfl_xor_sync(0xffffffffu, before, o), sp.units);
        own += __shfl_xor_sync(0xffffffffu, own, o);
    }
    *first = before;
    *count = min(own, sp.units - before);
}

// Number of a sequence's chunk among all chunks: distinct for every (sequence, chunk), because
// a sequence has at most floor(end / 64) - floor(start / 64) + 1 chunks, and a one is added per
// sequence.  Below la_chunk_ids().
__device__ __forceinline__ long long la_chunk_id(long long seq_start, int seq, int chunk) {
    return seq_start / kLaChunk + seq + chunk;
}
inline size_t la_chunk_ids(long long tokens, int n) { return (size_t)(tokens / kLaChunk + n + 1); }

// log2 of a token's decay.  exp(g) below 2^-160 is zero in fp32; the floor keeps -inf (a reset)
// out of the differences.
constexpr double kLaMinLog2 = -160.0;
__device__ __forceinline__ double log2_decay(const float* g, int per_token, long long tok, int H,
                                             int h, bool live) {
    if (!live) return 0.0;
    const double x = (double)(per_token ? g[(size_t)tok * H + h] : g[h]) * 1.4426950408889634;
    return x < kLaMinLog2 ? kLaMinLog2 : x;     // (NaN stays NaN)
}

// Summaries of every unit, then the states entering every unit (needs unit_state), then the runs.
// exact: operands that are formed in fp32 (decayed scores, states) enter the products in full
// precision; otherwise rounded once to bf16 (bf16 inputs only).
cudaError_t launch_la_summary(const LaArgs& a, int dc, int dout, ckda_dtype dtype, cudaStream_t s);
// The same summaries and runs on the tcgen05 tensor cores: bf16, 128 x 128 heads (linattn_tc.cu).
// A wait of theirs that runs out is kept as kLaStatusWait on the current device, until la_status_move hands
// it to a status word that holds no other.
constexpr int kLaStatusWait = 4;
cudaError_t launch_la_tc_summary(const LaArgs& a, cudaStream_t s);
cudaError_t launch_la_tc_run(const LaArgs& a, bool exact, cudaStream_t s);
cudaError_t la_status_move(int* word, cudaStream_t stream);

// Up to this many units a sequence, a run forms its entering state itself (from a few 64 KB summaries
// in L2) instead of a launch of its own for the scan: 4 units of 512 tokens 41.1 -> 38.8 us, 8 units
// of 192 tokens in fp32 60 -> 72 us.
constexpr int kLaFoldUnits = 4;

int la_scan_parts(int elems);    // partial sums of fin_dot per (sequence, head)
cudaError_t launch_la_scan(const LaArgs& a, int dk, int dv, cudaStream_t s);
// Final states of sequences without tokens (packed sequences in one unit each).
cudaError_t launch_la_empty(const LaArgs& a, int dk, int dv, cudaStream_t s);
cudaError_t launch_la_run(const LaArgs& a, int dc, int dout, bool exact, ckda_dtype dtype,
                          cudaStream_t s);

struct LaFwdArgs {
    const void *q, *k, *v;
    const float *g, *h0;
    void* out;
    float* hT;
    int per_token, G;
    float scale;
    LaSplit sp;
};
// (longest: tokens of the longest sequence)
size_t la_fwd_workspace(const LaSplit& sp, long long longest, int dk, int dv);
cudaError_t launch_la_fwd(const LaFwdArgs& a, long long longest, int dk, int dv, ckda_dtype dtype,
                          void* ws, cudaStream_t s);

struct LaBwdArgs {
    const void *q, *k, *v;
    const float *g, *h0;
    const void* dout;
    const float* dhT;
    void *dq, *dk, *dv;
    float *dg, *dh0;
    int per_token, G;
    float scale;
    LaSplit sp;
    long long tokens;
    int chunks;                  // chunks of all sequences
};
size_t la_bwd_workspace(const LaSplit& sp, long long longest, long long tokens, int G, int dk,
                        int dv);
cudaError_t launch_la_bwd(const LaBwdArgs& a, long long longest, int dk, int dv, ckda_dtype dtype,
                          void* ws, cudaStream_t s);

cudaError_t launch_la_decode(const void* q, const void* k, const void* v, const float* g,
                             int per_token, float* state, void* out, int N, int H, int G, int dk,
                             int dv, float scale, ckda_dtype dtype, cudaStream_t s);

}  // namespace ckda
