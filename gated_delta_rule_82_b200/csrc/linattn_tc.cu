// linattn_tc.cu -- chunked linear attention on the tcgen05 tensor cores (bf16, 128 x 128 heads).
//
// The runs of linattn.cuh for one unit of tokens per CTA, 64-token chunks, everything transposed
// so that an output channel sits in a TMEM lane (M = 128) and 64 tokens in the columns:
//     Sc  = X Y^T                        (64 x 64)    scores of the chunk
//     O1^T = S^T X^T                     (128 x 64)   read-out of the entering state
//     O2^T = Z^T P^T                     (128 x 64)   P: scores x decay, on the kept side
//     U^T = (w Z)^T Y                    (128 x 128)  what the chunk adds to the state
//     out_i = o exp(G_i) O1_i + O2_i,    S <- exp(G_C) S + U      (fp32, in registers)
// X, Y, Z arrive by TMA as 128-byte-swizzled tiles; one tile serves as K-major and as MN-major
// operand.  The state lives in the registers of eight warps (a row of 64 channels per thread) and
// goes to the tensor core as a bf16 operand through TMEM; the weighted Z as well, in three bf16
// terms (24 bits, 32 columns each), so that states are fp32-grade.  P and the state have NP terms where
// they are read: two leave 2^-18 of a value, far below an output's own rounding to bf16 (one term of
// the state, the output's own precision, made outputs 1.24 times as far off); three are fp32-grade.
// The state's lower terms lie in shared memory, half of the second one at NP = 2 in TMEM's last columns.
//
// Roles (one CTA per SM, all of TMEM): warps 0-7 weight Z; 8-15 carry the state and write the
// outputs; 16-19 turn scores into P; then one warp each for the decays, the products U, Sc (and
// TMA), and O1 with O2 (a poll of a barrier takes 80 cycles even when it is complete, so one warp
// that issued all of them would be the slowest part).  They meet on mbarriers only, so a chunk's
// products overlap the neighbours' element work: per chunk the tensor pipe needs 256 (Sc) + 768 (U)
// + 530 (O1) + 400 (O2) cycles at NP = 2.
// What bounds it: the element work of a chunk, about 3800 cycles in the state warps (read U, decay,
// write the state as an operand, outputs to memory) where HBM alone would allow 2700; tensor pipe 31 %
// busy, 0.47 instructions a cycle and scheduler.  16 heads: 2 x 2048 tokens, forward 43.0 us a call (with
// one term of the state 38.7), 65536 tokens 409 (355), the summary's launch 16 and 131 of them.
// Every wait is bounded; one that runs out is recorded (ckda_last_device_status) and ends the CTA
// once its copies and products have landed.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "linattn.cuh"
#include "tc_sm100.cuh"

namespace ckda {

namespace {

constexpr int C = kLaChunk;
constexpr int D = 128;                    // contracted and output channels
constexpr int kTile = C * D * 2;          // bytes of one operand tile
constexpr int kBlock = C * 128;           // 64 channels of it
constexpr int kGateRing = 4;
constexpr int kPolls = 1 << 20;

// TMEM columns
constexpr uint32_t kColU = 0, kColS = 128, kColO1 = 192, kColO2 = 256, kColSc = 320, kColSlo = 480;

__device__ int g_la_status;               // 0, or kLaStatusWait since the host last read it

struct TcArgs {
    LaArgs a;
    CUtensorMap map[kLaMaxRuns][3];       // x, y, z of every run
    CUtensorMap out[kLaMaxRuns];          // bf16 outputs
};

// A chunk's decays, as log2 sums over its 16-token blocks that start or end at a block's edge: the decay
// between two tokens of different blocks is r (to the end of the block) + whole blocks + l (from the start
// of the block), each a factor of at most one; that between two tokens of a block is the difference of
// their l, which is kept in two floats: a reset adds kLaMinLog2 to the sums, and behind it differences
// of single floats were off by 2e-4.  Summed in fp64.
struct GateSlot {
    float l[C], r[C];        // up to and including the token; behind the token
    float lo[C];             // what l leaves of its sum
    float out[C], upd[C];    // weights of the read-out and of the update, with their scales
    float block[4];          // whole blocks
    float total, pad[3];     // exp2 of the chunk's sum
};

// Position in a ring of N slots: the slot, and the parity of the phase that its n-th use completes.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) { slot = 0; phase ^= 1; }
    }
};

template <int NP, bool kSummary>
struct TcShape {
    static constexpr int STAGES = kSummary ? 4 : NP == 2 ? 3 : 2;
    static constexpr int STAGE = kSummary ? 2 * kTile : 3 * kTile;       // Y, Z, X
    static constexpr int P = kSummary ? 0 : NP * kBlock;
    static constexpr int OUT = kSummary ? 0 : 2 * kTile;                 // outputs on their way out
    static constexpr int SLO = kSummary ? 0 : NP == 2 ? D * D : (NP - 1) * D * D * 2;  // lower terms of the state
    static constexpr int GATES = STAGES * STAGE + P + SLO + OUT;
    static constexpr int DOT = GATES + kGateRing * (int)sizeof(GateSlot);
    static constexpr int BARS = DOT + (NP == 3 ? kGateRing * 4 * C * 4 : 0);
    static constexpr int SMEM = BARS + 512 + 1024;                       // (+ alignment of the base)
    static constexpr int EXTRA = kSummary ? 16 : 20;                     // first of the single warps
    static constexpr int THREADS = (EXTRA + (kSummary ? 3 : 4)) * 32;
    static constexpr uint32_t WZ = kSummary ? 256 : 384;                  // its first column
    static constexpr int UB = kSummary ? 2 : 1;      // buffers of U and of the weighted Z in TMEM
};

struct Bars {
    uint64_t full[4], empty[4], gfull[kGateRing], gempty[kGateRing];
    uint64_t sc_full, sc_empty, p_full, p_empty, wz_full[2], wz_empty[2];
    uint64_t u_full[2], u_empty[2], s_full, s_empty, o_full, o_empty, dot_full[kGateRing], dot_empty[kGateRing], fin_full, tail, drain[3];
    double fin[8];
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// Bounded wait of a converged warp: false when it has run out (a poll sleeps for up to about 4 us,
// so after some 4 s at most).  Short and in line: the roles' hot code together has to stay in
// the instruction cache (at 50 KB the element warps spent most of their time on instruction
// fetches), and calls do not go with the warpgroups' register shares.
__device__ __forceinline__ bool wait(Bars& b, uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n"
        "POLL:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\tsub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra POLL;\n"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(tc::smem_u32(bar)), "r"(parity), "n"(kPolls) : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    b.abort = 1;
    return false;
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // a in the low half
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The thread's number, read anew: what is derived from it is formed where it is used and holds no
// register over the chunks (the state's warps have none to spare).
__device__ __forceinline__ int thread_again() {
    int t;
    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(t));
    return t;
}

// Registers per thread of this warpgroup (all four warps).  A run launches with 80 (24 warps); the
// shares below add up to 6 x 80, so every raise finds what the others gave back.
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
constexpr int kRegsZ = 64, kRegsState = 120, kRegsP = 64, kRegsSingle = 48;
static_assert(2 * kRegsZ + 2 * kRegsState + kRegsP + kRegsSingle == 6 * 80, "register shares");

// One lane of a converged warp.  A group of products issued by it in one unrolled run keeps the
// tensor pipe fed (34 cycles per 128 x 64 x 16, 66 per 128 x 128 x 16); a loop of single products
// takes 77 cycles each whatever their size, and twice that beside busy warps.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// log2 of a decay exp(g), floored as kLaMinLog2 (a NaN stays one)
__device__ __forceinline__ double log2_decay(float g) {
    const double x = (double)g * 1.4426950408889634;
    return x < kLaMinLog2 ? kLaMinLog2 : x;
}

// ---- two fp32 values at a time
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
    return *reinterpret_cast<float2*>(&r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r)
        : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
          "l"(*reinterpret_cast<unsigned long long*>(&c)));
    return *reinterpret_cast<float2*>(&r);
}
// The leading 8 bits of both values as a bf16 pair; x keeps the rest.  Cutting (not rounding)
// leaves at most 16, then 8 significant bits, so three terms hold the 24 bits exactly.
__device__ __forceinline__ uint32_t cut2(float2& x) {
    const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
    const uint32_t t = __byte_perm(a, b, 0x7632);
    const float2 minus = make_float2(-1.f, -1.f);
    x = fma2(make_float2(__uint_as_float(a & 0xffff0000u), __uint_as_float(b & 0xffff0000u)), minus, x);
    return t;
}

// Both values rounded to bf16, as a pair; x keeps the rest (at most 2^-9 of it).
__device__ __forceinline__ uint32_t round2(float2& x) {
    const uint32_t t = pack2(x.x, x.y);
    x = fma2(make_float2(lo_f(t), hi_f(t)), make_float2(-1.f, -1.f), x);
    return t;
}

// ---- TMEM in 16-lane pieces whose elements are spread over the warp like mma fragments
// 16 lanes x 32 columns of packed bf16: v[2 j + e] is lane l / 4 + 8 e, column 4 j + l % 4.
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
        "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
        "r"(v[15]) : "memory");
}
// 32 lanes x 4 or 8 columns, a lane per thread.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]),
                 "r"(v[6]), "r"(v[7]) : "memory");
}
// 16 lanes x 32 columns of fp32: v[2 j + e] holds lane l / 4 + 8 e, columns 8 j + 2 (l % 4) and
// the one behind it.  No wait.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float2* v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
// A wait that the values depend on, so that no use of them is scheduled before it.
__device__ __forceinline__ void ld_wait(float2* v, float2* w) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0].x), "+f"(v[0].y), "+f"(v[1].x), "+f"(v[1].y), "+f"(v[2].x), "+f"(v[2].y),
                   "+f"(v[3].x), "+f"(v[3].y), "+f"(v[4].x), "+f"(v[4].y), "+f"(v[5].x), "+f"(v[5].y),
                   "+f"(v[6].x), "+f"(v[6].y), "+f"(v[7].x), "+f"(v[7].y),
                   "+f"(w[0].x), "+f"(w[0].y), "+f"(w[1].x), "+f"(w[1].y), "+f"(w[2].x), "+f"(w[2].y),
                   "+f"(w[3].x), "+f"(w[3].y), "+f"(w[4].x), "+f"(w[4].y)
                 :: "memory");
    asm volatile("" : "+f"(w[5].x), "+f"(w[5].y), "+f"(w[6].x), "+f"(w[6].y), "+f"(w[7].x), "+f"(w[7].y));
}
// 16 lanes x 16 columns in the same layout; no wait.
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, float2* v) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                   "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
__device__ __forceinline__ void tmem_ld_wait4(float2* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0].x), "+f"(v[0].y), "+f"(v[1].x), "+f"(v[1].y), "+f"(v[2].x), "+f"(v[2].y),
                   "+f"(v[3].x), "+f"(v[3].y)
                 :: "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t r[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t a, const uint32_t r[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// 16-byte piece of a 128-byte row of a swizzled tile; row: the address of its piece 0.  (Formed at the
// store: addresses held over the loop cost more registers than the state's warps have.)
__device__ __forceinline__ void st_piece(uint32_t row, uint32_t piece, const uint32_t v[4]) {
    asm volatile("{\n\t.reg .b32 a;\n\txor.b32 a, %0, %1;\n\tst.shared.v4.b32 [a], {%2, %3, %4, %5};\n\t}"
                 ::"r"(row), "r"(piece << 4), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
// The output warps' staging: 32 tokens x 32 channels of bf16 per warp, 16-byte pieces swizzled so
// that eight neighbouring tokens lie in different banks.
__device__ __forceinline__ uint32_t stage_at(uint32_t tok, uint32_t piece) {
    return tok * 64 + ((piece ^ ((tok >> 1) & 3)) << 4);
}

// kF32: the outputs are fp32 (gradients that are still to be summed over a group of heads).
// kDots: the output rows are multiplied with LaRun::dot.
template <int NP, bool kSummary, bool kF32, bool kDots>
__global__ void __launch_bounds__(TcShape<NP, kSummary>::THREADS, 1)
la_tc_kernel(const __grid_constant__ TcArgs args) {
    using S = TcShape<NP, kSummary>;
    constexpr int NS = S::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sP = sm + NS * S::STAGE;
    uint8_t* sSlo = sP + S::P;
    GateSlot* gates = reinterpret_cast<GateSlot*>(sm + S::GATES);
    float* sDot = reinterpret_cast<float*>(sm + S::DOT);
    Bars& b = *reinterpret_cast<Bars*>(sm + S::BARS);

    const LaArgs& a = args.a;
    const LaRun& R = a.run[blockIdx.y];
    const int H = a.sp.H, unit = blockIdx.x / H, h = blockIdx.x - unit * H;
    const UnitAt u = find_unit(a.sp, unit);
    if (!u.ok) {
        la_wait_before();       // (no grid of a call ends before the one ahead of it)
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
    const bool rev = R.reverse;
    const int n = (u.len + C - 1) / C;
    auto chunk_at = [&](int i) { return rev ? n - 1 - i : i; };
    auto live_of = [&](int i) { return min(C, u.len - chunk_at(i) * C); };

    if (warp == S::EXTRA + 1) {
        tc::tmem_alloc(&b.tmem, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&b.full[i], 1);
            tc::mbar_init(&b.empty[i], kSummary ? 9 : 11);  // the products; eight warps that read Z
        }
        for (int i = 0; i < kGateRing; ++i) {
            tc::mbar_init(&b.gfull[i], 1);
            tc::mbar_init(&b.gempty[i], S::EXTRA);    // every element warp
            tc::mbar_init(&b.dot_full[i], 8);
            tc::mbar_init(&b.dot_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&b.wz_full[i], 8);
            tc::mbar_init(&b.wz_empty[i], 1);
        }
        tc::mbar_init(&b.p_full, 4);
        tc::mbar_init(&b.p_empty, 1);
        tc::mbar_init(&b.sc_full, 1);
        tc::mbar_init(&b.sc_empty, 4);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&b.u_full[i], 1);
            tc::mbar_init(&b.u_empty[i], 8);
        }
        tc::mbar_init(&b.s_full, 8);
        tc::mbar_init(&b.s_empty, 1);
        tc::mbar_init(&b.o_full, 1);
        tc::mbar_init(&b.o_empty, 8);
        tc::mbar_init(&b.fin_full, 8);
        tc::mbar_init(&b.tail, 1);
        for (int i = 0; i < 3; ++i) tc::mbar_init(&b.drain[i], 1);
        b.abort = 0;
        tc::fence_mbar_init();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = b.tmem;
    la_let_next_start();
    if constexpr (!kSummary) {        // (one instruction per warpgroup)
        if (warp < 8) regs_down<kRegsZ>();
        else if (warp < 16) regs_up<kRegsState>();
        else if (warp < 20) regs_down<kRegsP>();
        else regs_down<kRegsSingle>();
    }

    if (warp < 8) {
        // --------------------------------------------- weighted Z: 16 output channels a warp.
        // ldmatrix leaves the transposed tile in the layout that the 16-lane TMEM store takes.
        const int m = lane >> 3, e = warp >> 2;
        const uint32_t zat = ((m >> 1) * 8 + (lane & 7)) * 128 + (quarter >> 1) * kBlock +
                             ((((quarter & 1) * 4 + 2 * e + (m & 1)) ^ (lane & 7)) << 4);
        const uint32_t to = tc::tmem_addr(tmem, 32 * quarter + 16 * e, S::WZ);
        const bool packed = a.sp.cu != nullptr;
        Ring<NS> at;
        Ring<kGateRing> gp;
        Ring<S::UB> wz;
        const uint32_t z0 = tc::smem_u32(sm) + kTile + zat;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (!wait(b, &b.full[at.slot], at.phase) || !wait(b, &b.gfull[gp.slot], gp.phase)) break;
            if (packed && live_of(i) < C && !wait(b, &b.tail, 0)) break;
            const uint32_t z = z0 + at.slot * S::STAGE;
            const float* upd = gates[gp.slot].upd + 2 * (lane & 3);
            uint32_t p[16];                     // [4 tb + m]: tokens 16 tb + 8 (m / 2) ..
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) ldsm4t(&p[4 * tb], z + tb * 2048);
            float2 v[16];
#pragma unroll
            for (int g = 0; g < 8; ++g) {       // 8 tokens
                const float2 w = *reinterpret_cast<const float2*>(upd + 8 * g);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    v[2 * g + k] = mul2(make_float2(lo_f(p[2 * g + k]), hi_f(p[2 * g + k])), w);
            }
            arrive_warp(&b.empty[at.slot]);
            arrive_warp(&b.gempty[gp.slot]);
            at.next();
            gp.next();
            if (i >= S::UB && !wait(b, &b.wz_empty[wz.slot], wz.phase ^ 1)) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 3; ++k) {
                uint32_t t[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) t[j] = cut2(v[j]);
                tmem_st_16x32(to + 96 * wz.slot + 32 * k, t);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            arrive_warp(&b.wz_full[wz.slot]);
            wz.next();
        }
    } else if (warp < 16) {
        // ------------------------------------------ the state: 64 contracted channels of one row
        const int row = 32 * quarter + lane, half = (warp - 8) >> 2, col0 = 64 * half;
        const int rs = R.transposed ? D : 1, cs = R.transposed ? 1 : D;
        const size_t seq_state = ((size_t)u.seq * H + h) * (D * D);
        const size_t unit_state = ((size_t)unit * H + h) * (D * D);
        const size_t own = (size_t)row * rs + (size_t)col0 * cs;
        const bool fold = !kSummary && R.fold && R.unit_state;
        const float* init = nullptr;
        if (!kSummary) {
            if (R.unit_state && !fold) init = R.unit_state + unit_state;
            else if (R.init) init = R.init + seq_state;
        }
        // (of what a run reads, only the entering states and the outputs' places are the business of
        // the launches before it; the inputs are complete)
        if constexpr (!kSummary) la_wait_before();
        float2 st[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) st[j] = make_float2(0.f, 0.f);
        // the entering state, then (folded) the units ahead of this one, in the run's order.  Where a
        // thread's channels lie one after the other it takes four at a time (a layer's backward with
        // h0 and dhT: 176 us with single ones)
        const int ahead = la_units_ahead(fold, rev, unit, u.index, u.count, a.sp.units);
#pragma unroll 1
        for (int k = init ? -1 : 0; k < ahead; ++k) {
            const size_t un = (size_t)(rev ? unit + ahead - k : unit - ahead + k) * H + h;
            const float w = k < 0 ? 0.f : exp2f((float)R.unit_decay[un]);
            const float* E = (k < 0 ? init : R.unit_state + un * (D * D)) + own;
            const float2 w2 = make_float2(w, w);
            if (R.transposed) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(E + 4 * j);
                    st[2 * j] = fma2(st[2 * j], w2, make_float2(x.x, x.y));
                    st[2 * j + 1] = fma2(st[2 * j + 1], w2, make_float2(x.z, x.w));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    st[j] = fma2(st[j], w2, make_float2(E[(size_t)(2 * j) * D], E[(size_t)(2 * j + 1) * D]));
            }
        }
        bool ok = true;
        auto again = [&]() { return NP == 2 ? thread_again() : tid; };
        auto put_state = [&](int i) {             // the state entering chunk i, as an operand
            const int tid = again(), lane = tid & 31, quarter = (tid >> 5) & 3, half = (tid >> 7) & 1;
            const int row = 32 * quarter + lane;
            // this row of its lower terms (NP = 2: channels 64-127 only)
            const uint32_t slo = tc::smem_u32(sSlo) + (NP == 3 ? half * (D * 128) : 0) + row * 128 + ((row & 7) << 4);
            if (i > 0 && !wait(b, &b.s_empty, (i - 1) & 1)) return false;
            tc::tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t t[8];
                if constexpr (NP == 2) {
                    // the second term: of channels 0-63 through TMEM too, of the others through shared memory
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t m[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 x = st[8 * k + 4 * q + j];
                            const uint32_t hi = pack2(x.x, x.y);
                            m[j] = pack2(x.x - lo_f(hi), x.y - hi_f(hi));
                            t[4 * q + j] = hi;
                        }
                        if (half == 0)
                            tmem_st4(tc::tmem_addr(tmem, 32 * quarter, kColSlo + 8 * k + 4 * q), m);
                        else
                            st_piece(slo, 2 * k + q, m);
                    }
                } else {
                    // three terms: the first through TMEM, the others through shared memory
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t m[4], l[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float2 x = st[8 * k + 4 * q + j];
                            t[4 * q + j] = cut2(x);
                            m[j] = cut2(x);
                            l[j] = __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
                        }
                        st_piece(slo, 2 * k + q, m);
                        st_piece(slo + D * D * 2, 2 * k + q, l);
                    }
                }
                tmem_st8(tc::tmem_addr(tmem, 32 * quarter, kColS + 32 * half + 8 * k), t);
            }
            tc::tmem_st_wait();
            if (NP == 3 || half == 1) tc::fence_proxy_async_smem();
            tc::tc_fence_before();
            arrive_warp(&b.s_full);
            return true;
        };
        constexpr bool dots = kDots;
        // The rows that the outputs are multiplied with, into the staging area, long before their use.
        auto fetch_rows = [&](int i) {
            const int tid = again(), warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
            const int ch0 = 32 * quarter, tq = 32 * ((warp >> 2) & 1);
            const int tr = lane >> 2, tp = lane & 3;             // row and 16-byte piece, 8 rows a time
            const int Hd = H / R.dg, live = live_of(i) - tq;
            const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(R.dot) +
                                       ((size_t)(u.tok + chunk_at(i) * C + tq) * Hd + h / R.dg) * D + ch0 + 8 * tp;
            uint8_t* sOut = sSlo + S::SLO + (warp - 8) * (kTile / 8) + (i & 1) * kTile;
            if (lane == 0) tc::bulk_wait_read<1>();              // (what was last stored from it)
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 8 * k + tr;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                             ::"r"(tc::smem_u32(sOut + stage_at(t, tp))),
                               "l"(src + (t < live ? (size_t)t * Hd * D : 0)), "r"(t < live ? 16 : 0) : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Outputs: this warp's 32 channels, 32 of the chunk's tokens; two staging areas, a tile apart
        auto put_out = [&](int i) {
            const int tid = again(), warp = tid >> 5, lane = tid & 31, quarter = warp & 3;
            const int ch0 = 32 * quarter, tq = 32 * ((warp >> 2) & 1);
            const int tr = lane >> 2, tp = lane & 3;             // row and 16-byte piece, 8 rows a time
            const int gr = lane >> 2, gc = 2 * (lane & 3);
            const int m4 = lane >> 3;                            // matrix of an x4 access
            const int gs = i % kGateRing, c = chunk_at(i), live = live_of(i) - tq;
            const long long tok = u.tok + (long long)c * C + tq;
            uint8_t* sOut = sSlo + S::SLO + (warp - 8) * (kTile / 8) + (i & 1) * kTile;
            if constexpr (dots) {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            } else if (lane == 0) {
                tc::bulk_wait_read<1>();                         // the staging area is free again
            }
            __syncwarp();
            if (!wait(b, &b.o_full, i & 1)) return false;
            tc::tc_fence_after();
            float2 dot[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dot[j] = make_float2(0.f, 0.f);
            float2 x[8], y[8];
            const uint32_t o1 = tc::tmem_addr(tmem, 32 * quarter, kColO1 + tq), o2 = o1 + (kColO2 - kColO1);
            tmem_ld_16x32(o1, x);
            tmem_ld_16x32(o2, y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {                        // 16 channels
                ld_wait(x, y);
                if (e == 1) {
                    tc::tc_fence_before();
                    arrive_warp(&b.o_empty);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 w = *reinterpret_cast<const float2*>(gates[gs].out + tq + 8 * j + gc);
                    x[2 * j] = fma2(x[2 * j], w, y[2 * j]);
                    x[2 * j + 1] = fma2(x[2 * j + 1], w, y[2 * j + 1]);
                }
                const uint32_t at0 = tc::smem_u32(sOut) + stage_at(8 * (m4 >> 1) + (lane & 7), 2 * e + (m4 & 1));
                if constexpr (dots) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {                // 16 tokens: four 8 x 8 matrices
                        uint32_t d[4];
                        ldsm4t(d, at0 + 1024 * j);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            dot[2 * j + (k >> 1)] = fma2(x[4 * j + k], make_float2(lo_f(d[k]), hi_f(d[k])),
                                                         dot[2 * j + (k >> 1)]);
                    }
                    __syncwarp();
                }
                if constexpr (!kF32) {
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = pack2(x[j].x, x[j].y);
                    if (e == 0) {                                // (in flight while this half is stored)
                        tmem_ld_16x32(o1 + (16u << 16), x);
                        tmem_ld_16x32(o2 + (16u << 16), y);
                    }
                    stsm4t(at0, o);
                    stsm4t(at0 + 1024, o + 4);
                } else {
                    float* dst = static_cast<float*>(R.out) + ((size_t)tok * H + h) * D + ch0 + 16 * e + gr;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = 8 * (j >> 1) + gc;
                        float* at = dst + (size_t)t * H * D + 8 * (j & 1);
                        if (t < live) at[0] = x[j].x;
                        if (t + 1 < live) at[(size_t)H * D] = x[j].y;
                    }
                    if (e == 0) {
                        tmem_ld_16x32(o1 + (16u << 16), x);
                        tmem_ld_16x32(o2 + (16u << 16), y);
                    }
                }
            }
            arrive_warp(&b.gempty[gs]);
            if constexpr (!kF32) {
                if (a.sp.cu && live < 32) {       // (the rows behind are another sequence's)
                    __syncwarp();
                    __nv_bfloat16* dst =
                        static_cast<__nv_bfloat16*>(R.out) + ((size_t)tok * H + h) * D + ch0 + 8 * tp;
                    for (int t = tr; t < live; t += 8)
                        *reinterpret_cast<uint4*>(dst + (size_t)t * H * D) =
                            *reinterpret_cast<const uint4*>(sOut + stage_at(t, tp));
                } else if (live > 0) {
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tc::tma_store_4d(&args.out[blockIdx.y], sOut, ch0, h,
                                         (a.sp.cu ? (int)u.tok : u.index * a.sp.L) + c * C + tq,
                                         a.sp.cu ? 0 : u.seq);
                        tc::bulk_commit();
                    }
                }
            }
            if constexpr (dots) {
                // sum over the lanes that hold other channels
#pragma unroll
                for (int s = 2; s > 0; s >>= 1)
#pragma unroll
                    for (int j = 0; j < s; ++j) {
                        const bool up = lane & (8 * s);
                        const float2 send = up ? dot[j] : dot[j + s], keep = up ? dot[j + s] : dot[j];
                        dot[j].x = keep.x + __shfl_xor_sync(0xffffffffu, send.x, 8 * s);
                        dot[j].y = keep.y + __shfl_xor_sync(0xffffffffu, send.y, 8 * s);
                    }
                dot[0].x += __shfl_xor_sync(0xffffffffu, dot[0].x, 4);
                dot[0].y += __shfl_xor_sync(0xffffffffu, dot[0].y, 4);
                if (i >= kGateRing && !wait(b, &b.dot_empty[gs], (i / kGateRing - 1) & 1)) return false;
                if (!(lane & 4))
                    *reinterpret_cast<float2*>(sDot + (4 * gs + quarter) * C + tq + 8 * (lane >> 3) + gc) = dot[0];
                arrive_warp(&b.dot_full[gs]);
            }
            return true;
        };
        // In the order in which nothing is waited for: O1 and O2 of a chunk run beside the next
        // update, and O1 of the next chunk beside the outputs of this one.
        if constexpr (!kSummary) ok = put_state(0);
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
            const int gs = i % kGateRing;
            if constexpr (dots) fetch_rows(i);
            const int ub = kSummary ? i & 1 : 0;
            if (!(ok = wait(b, &b.u_full[ub], (kSummary ? i >> 1 : i) & 1))) break;
            tc::tc_fence_after();
            // (U was formed from the chunk's decays: they are there)
            const float2 total = make_float2(gates[gs].total, gates[gs].total);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float x[16];
                tc::tmem_ld16_sync(tc::tmem_addr(tmem, 32 * quarter, kColU + D * ub + col0 + 16 * q), x);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    st[8 * q + j] = fma2(st[8 * q + j], total, make_float2(x[2 * j], x[2 * j + 1]));
            }
            tc::tc_fence_before();
            arrive_warp(&b.u_empty[ub]);
            if constexpr (kSummary) arrive_warp(&b.gempty[gs]);
            if constexpr (!kSummary) {
                if (i + 1 < n && !(ok = put_state(i + 1))) break;
                if (!(ok = put_out(i))) break;
            }
        }
        if (!kSummary && lane == 0) tc::bulk_wait_all();
        if (ok) {
            // the run's last unit of a sequence leaves the final state (where no scan has formed it)
            const bool last = !R.unit_state || (fold && u.index == (rev ? 0 : u.count - 1));
            float* fin = kSummary ? R.unit_state + unit_state : (last && R.fin ? R.fin + seq_state : nullptr);
            if (fin) {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    fin[own + (size_t)(2 * j) * cs] = st[j].x;
                    fin[own + (size_t)(2 * j + 1) * cs] = st[j].y;
                }
            }
            if (!kSummary && last && R.fin_dot) {
                // (the run of dq, which holds its rows one channel after the other)
                const float* f = R.fin_dot + seq_state + own;
                double d = 0.0, d2 = 0.0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float4 x = *reinterpret_cast<const float4*>(f + 4 * j);
                    d += (double)st[2 * j].x * x.x + (double)st[2 * j].y * x.y;
                    d2 += (double)st[2 * j + 1].x * x.z + (double)st[2 * j + 1].y * x.w;
                }
                d += d2;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
                if (lane == 0) b.fin[warp - 8] = d;
                arrive_warp(&b.fin_full);
                if (warp == 8 && wait(b, &b.fin_full, 0) && lane == 0) {
                    double s = 0.0;
                    for (int w = 0; w < 8; ++w) s += b.fin[w];
                    R.fin_dot_out[(size_t)u.seq * H + h] = s;
                }
            }
        }
    } else if (!kSummary && warp < S::EXTRA) {
        // -------------------------------------------------------------------- P from the scores
        const int gr = lane >> 2, gc = 2 * (lane & 3);
        const float p_scale = R.p_scale;
        // P is zero beyond the diagonal: those 16 x 8 tiles are cleared once and stay
        for (int k = 0; k < NP; ++k)
            for (int w = lane; w < 16 * 8; w += 32) {
                const int row = 16 * quarter + (w >> 3), c8 = w & 7;
                if (rev ? c8 < 2 * quarter : c8 > 2 * quarter + 1)
                    *reinterpret_cast<uint4*>(sP + k * kBlock + row * 128 + ((c8 ^ (row & 7)) << 4)) =
                        make_uint4(0, 0, 0, 0);
            }
        // 16 x 16 tiles: 16 tokens (this warp's rows) against the 16 tokens from c0
        auto put = [&](uint8_t* p, int c0, float2 w[4]) {     // w[2 j + e]: columns 8 j, rows 8 e
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t at = ((((uint32_t)c0 >> 3) + j) ^ gr) << 4;
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int q = 0; q < NP; ++q)       // (two terms: both rounded, three: cut)
                        *reinterpret_cast<uint32_t*>(p + q * kBlock + e * 1024 + at) =
                            NP == 3  ? cut2(w[2 * j + e])
                            : q == 0 ? round2(w[2 * j + e])
                                     : pack2(w[2 * j + e].x, w[2 * j + e].y);
            }
        };
        auto make_p = [&](int i) {
            const int gs = i % kGateRing;
            if (!wait(b, &b.gfull[gs], (i / kGateRing) & 1)) return false;
            const GateSlot& g = gates[gs];
            const int r0 = 16 * quarter + gr;
            // Tiles off the diagonal: the decay between row and column passes the edge of this
            // warp's 16 rows, so it is a row factor times a column factor, both at most one.
            const float* edge = rev ? g.r : g.l;
            const float* far = rev ? g.l : g.r;
            float ra[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) ra[e] = ex2(edge[r0 + 8 * e]) * p_scale;
            const float rl[2] = {g.l[r0], g.l[r0 + 8]}, rlo[2] = {g.lo[r0], g.lo[r0 + 8]};
            const float sg = rev ? -1.f : 1.f;
            if (!wait(b, &b.sc_full, i & 1)) return false;
            if (i > 0 && !wait(b, &b.p_empty, (i - 1) & 1)) return false;
            tc::tc_fence_after();
            const uint32_t sc = tc::tmem_addr(tmem, 32 * quarter, kColSc);
            uint8_t* p = sP + r0 * 128 + gc * 2;
            float2 x[4], nx[4];
            tmem_ld_16x16(sc + 16 * quarter, x);
            // the diagonal tile, while the first of the others is on its way (outwards from it)
            const int dt = rev ? 1 : -1, end = rev ? 4 : -1;
            int t = quarter + dt;
            float mid = 0.f;                                     // whole blocks in between
            tmem_ld_wait4(x);
            if (t != end) tmem_ld_16x16(sc + 16 * t, nx);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = 16 * quarter + 8 * j + gc;
                const float2 cl = *reinterpret_cast<const float2*>(g.l + c);
                const float2 clo = *reinterpret_cast<const float2*>(g.lo + c);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = r0 + 8 * e;
                    float2& w = x[2 * j + e];
                    w.x = (rev ? row <= c : row >= c) ? w.x * ex2(sg * ((rl[e] - cl.x) + (rlo[e] - clo.x))) * p_scale : 0.f;
                    w.y = (rev ? row <= c + 1 : row >= c + 1) ? w.y * ex2(sg * ((rl[e] - cl.y) + (rlo[e] - clo.y))) * p_scale : 0.f;
                }
            }
            put(p, 16 * quarter, x);
#pragma unroll 1
            for (; t != end; t += dt) {
                tmem_ld_wait4(nx);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = nx[j];
                if (t + dt != end) tmem_ld_16x16(sc + 16 * (t + dt), nx);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = 16 * t + 8 * j + gc;
                    const float2 cf = *reinterpret_cast<const float2*>(far + c);
                    const float2 cb = make_float2(ex2(cf.x + mid), ex2(cf.y + mid));
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        x[2 * j + e] = mul2(mul2(x[2 * j + e], cb), make_float2(ra[e], ra[e]));
                }
                mid += g.block[t];
                put(p, 16 * t, x);
            }
            tc::tc_fence_before();
            arrive_warp(&b.sc_empty);
            arrive_warp(&b.gempty[gs]);
            tc::fence_proxy_async_smem();
            arrive_warp(&b.p_full);
            return true;
        };
        for (int i = 0; i < n; ++i)
            if (!make_p(i)) break;
    } else if (warp == S::EXTRA) {
        // -------------------------------------------------------------------------- the decays
        // (and the output rows' products: their sums over the channel groups, and over the chunk)
        constexpr bool dots = kDots;
        auto dot_rows = [&](int i) {
            const int slot = i % kGateRing;
            const float* d = sDot + 4 * slot * C;
            if (!wait(b, &b.dot_full[slot], (i / kGateRing) & 1)) return false;
            const int c = chunk_at(i), live = live_of(i);
            const long long tok = u.tok + (long long)c * C;
            double sum = 0.0;      // (a gradient is a small difference of these sums)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 32 * e + lane;
                const double s = ((double)d[t] + d[C + t]) + ((double)d[2 * C + t] + d[3 * C + t]);
                if (t < live) {
                    R.dot_out[(size_t)(tok + t) * H + h] = s;
                    sum += s;
                }
            }
            arrive_warp(&b.dot_empty[slot]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0)
                R.dot_sum[(size_t)la_chunk_id(u.tok - (long long)u.index * a.sp.L, u.seq,
                                              u.index * (a.sp.L / C) + c) * H + h] = sum;
            return true;
        };
        const float u_scale = R.u_scale, o_scale = R.o_scale;
        // The raw decays are requested a chunk ahead (and stay requested there: volatile), clamped to
        // the unit and unconditional, so that nothing depends on them before they are used.
        const float* gp = a.g + h + (a.per_token ? (size_t)u.tok * H : 0);
        const size_t gstep = a.per_token ? H : 0;
        auto load = [&](int t) {
            float x;
            asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(gp + min(t, u.len - 1) * gstep));
            return x;
        };
        int t0 = chunk_at(0) * C + 2 * lane;
        float2 cur = make_float2(load(t0), load(t0 + 1)), next;
        double decay = 0.0;
        for (int i = 0; i < n; ++i, cur = next) {
            const int gs = i % kGateRing, live = live_of(i);
            t0 = chunk_at(min(i + 1, n - 1)) * C + 2 * lane;
            next = make_float2(load(t0), load(t0 + 1));
            const double g0 = 2 * lane < live ? log2_decay(cur.x) : 0.0;
            const double g1 = 2 * lane + 1 < live ? log2_decay(cur.y) : 0.0;
            double upto = g0 + g1;                                // since the start of the chunk
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += x;
            }
            const double all = __shfl_sync(0xffffffffu, upto, 31);
            if constexpr (kSummary) decay += all;
            if (i >= kGateRing && !wait(b, &b.gempty[gs], (i / kGateRing - 1) & 1)) break;
            GateSlot& g = gates[gs];
            const double G0 = upto - g1;
            const float2 down = make_float2(ex2((float)G0), ex2((float)upto));                  // since the start
            const float2 up = make_float2(ex2((float)(all - G0)), ex2((float)(all - upto)));    // to the end
            const float2 w = rev ? down : up;
            const int t = 2 * lane;
            *reinterpret_cast<float2*>(g.upd + t) =
                make_float2(t < live ? w.x * u_scale : 0.f, t + 1 < live ? w.y * u_scale : 0.f);
            if constexpr (!kSummary) {
                const double end = __shfl_sync(0xffffffffu, upto, lane | 7);    // of this lane's block
                double start = __shfl_sync(0xffffffffu, upto, max((lane & ~7) - 1, 0));
                if (lane < 8) start = 0.0;
                const double l0 = G0 - start, l1 = upto - start;
                const float2 l = make_float2((float)l0, (float)l1);
                *reinterpret_cast<float2*>(g.l + t) = l;
                *reinterpret_cast<float2*>(g.lo + t) = make_float2((float)(l0 - l.x), (float)(l1 - l.y));
                *reinterpret_cast<float2*>(g.r + t) = make_float2((float)(end - G0), (float)(end - upto));
                if ((lane & 7) == 7) g.block[lane >> 3] = l.y;
                const float2 o = rev ? up : down;
                *reinterpret_cast<float2*>(g.out + t) = make_float2(o.x * o_scale, o.y * o_scale);
            }
            if (lane == 0) g.total = ex2((float)all);
            arrive_warp(&b.gfull[gs]);
            // (three chunks behind, so that the element warps never wait for this)
            if constexpr (dots)
                if (i >= 3 && !dot_rows(i - 3)) break;
        }
        if constexpr (dots)
            for (int i = max(n - 3, 0); i < n; ++i)
                if (!dot_rows(i)) break;
        if (kSummary && lane == 0) R.unit_decay[(size_t)unit * H + h] = decay;
    } else {
        // ---------------------------------------------- tcgen05.mma: U (+ 1), Sc (+ 2), O (+ 3)
        const int role = warp - S::EXTRA - 1;
        const bool packed = a.sp.cu != nullptr;
        Ring<NS> at;                                      // of the chunk being worked on
        // a chunk's tiles are in place; packed: rows behind the sequence's end belong to the next
        // one and must not reach a product even as 0 x NaN, so the first role clears them
        auto tiles = [&](int i) {
            if (!wait(b, &b.full[at.slot], at.phase)) return false;
            if (packed && live_of(i) < C) {
                if (role == 0) {
                    uint8_t* s = sm + at.slot * S::STAGE;
                    const int live = live_of(i), words = (C - live) * 8;   // 16-byte words per block
#pragma unroll 1
                    for (int k = 0; k < 2 * (S::STAGE / kTile); ++k)
#pragma unroll 1
                        for (int w = lane; w < words; w += 32)
                            *reinterpret_cast<uint4*>(s + k * kBlock + live * 128 + w * 16) =
                                make_uint4(0, 0, 0, 0);
                    tc::fence_proxy_async_smem();
                    arrive_warp(&b.tail);           // (one such chunk in a unit)
                } else {
                    if (!wait(b, &b.tail, 0)) return false;
                    tc::fence_proxy_async_smem();
                }
            }
            return true;
        };
        // TMA: the role that needs a chunk first requests the one that takes a freed stage
        const CUtensorMap* map = args.map[blockIdx.y];
        const int hx = h / R.xg, hy = h / R.yg, hz = h / R.zg, brow = packed ? 0 : u.seq;
        const int tok0 = packed ? (int)u.tok : u.index * a.sp.L;
        Ring<NS> req;
        int sent = 0;
        auto request = [&](int i) {
            if (i >= NS && !wait(b, &b.empty[req.slot], req.phase ^ 1)) return false;
            if (elect_one()) {
                uint64_t* full = &b.full[req.slot];
                uint8_t* dst = sm + req.slot * S::STAGE;
                const int t = tok0 + chunk_at(i) * C;
                tc::mbar_arrive_expect_tx(full, S::STAGE);
#pragma unroll 1
                for (int k = 0; k < 2; ++k, dst += kBlock) {
                    tc::tma_load_4d(dst, &map[1], 64 * k, hy, t, brow, full);
                    tc::tma_load_4d(dst + kTile, &map[2], 64 * k, hz, t, brow, full);
                    if constexpr (!kSummary)
                        tc::tma_load_4d(dst + 2 * kTile, &map[0], 64 * k, hx, t, brow, full);
                }
            }
            __syncwarp();
            req.next();
            sent = i + 1;
            return true;
        };
        bool ok = true;
        if (role == 0) {
            constexpr uint32_t id_u = tc::idesc_bf16_f32(128, 128, 0, 1);
            const uint64_t yd0 = tc::smem_desc_sw128(tc::smem_u32(sm), kBlock, 1024);
            Ring<S::UB> ub;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                if (!(ok = tiles(i))) break;
                if (i >= S::UB && !(ok = wait(b, &b.u_empty[ub.slot], ub.phase ^ 1))) break;
                const uint64_t yd = tc::desc_add(yd0, at.slot * S::STAGE);
                if (!(ok = wait(b, &b.wz_full[ub.slot], ub.phase))) break;
                tc::tc_fence_after();
                if (elect_one()) {
#pragma unroll 1
                    for (int k = 2; k >= 0; --k)        // the smallest term of the weighted Z first:
#pragma unroll                                          // fewer roundings at the full size
                        for (int ks = 0; ks < 4; ++ks)
                            mma_tmem_a(tmem + kColU + D * ub.slot,
                                       tmem + S::WZ + 96 * ub.slot + 32 * k + 8 * ks,
                                       tc::desc_add(yd, ks * 2048), id_u, k < 2 || ks > 0);
                    tc::mma_commit(&b.wz_empty[ub.slot]);
                    tc::mma_commit(&b.u_full[ub.slot]);
                    tc::mma_commit(&b.empty[at.slot]);
                }
                __syncwarp();
                at.next();
                ub.next();
            }
        } else if (kSummary) {
#pragma unroll 1
            for (int i = 0; i < n; ++i)
                if (!(ok = request(i))) break;
        } else if (role == 1) {
            constexpr uint32_t id_sc = tc::idesc_bf16_f32(64, 64, 0, 0);
            const uint64_t d0 = tc::smem_desc_sw128(tc::smem_u32(sm), 16, 1024);
#pragma unroll 1
            for (int i = 1 - NS; i < n; ++i) {
                if (i >= 0) {
                    if (!(ok = tiles(i))) break;
                    if (i > 0 && !(ok = wait(b, &b.sc_empty, (i - 1) & 1))) break;
                    tc::tc_fence_after();
                    const uint64_t yd = tc::desc_add(d0, at.slot * S::STAGE), xd = tc::desc_add(yd, 2 * kTile);
                    if (elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t off = (ks >> 2) * kBlock + (ks & 3) * 32;
                            tc::mma_bf16(tmem + kColSc, tc::desc_add(xd, off), tc::desc_add(yd, off), id_sc,
                                         ks > 0);
                        }
                        tc::mma_commit(&b.sc_full);
                        tc::mma_commit(&b.empty[at.slot]);
                    }
                    __syncwarp();
                    at.next();
                }
                if (i + NS - 1 < n && !(ok = request(i + NS - 1))) break;
            }
        } else {
            constexpr uint32_t id_o1 = tc::idesc_bf16_f32(128, 64, 0, 0);
            constexpr uint32_t id_o2 = tc::idesc_bf16_f32(128, 64, 1, 0);
            const uint64_t xd0 = tc::smem_desc_sw128(tc::smem_u32(sm) + 2 * kTile, 16, 1024);
            const uint64_t zd0 = tc::smem_desc_sw128(tc::smem_u32(sm) + kTile, kBlock, 1024);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                if (!(ok = tiles(i))) break;
                if (i > 0 && !(ok = wait(b, &b.o_empty, (i - 1) & 1))) break;
                // O1: the entering state read by X
                if (!(ok = wait(b, &b.s_full, i & 1))) break;
                tc::tc_fence_after();
                const uint64_t xd = tc::desc_add(xd0, at.slot * S::STAGE);
                if (elect_one()) {
                    if constexpr (NP == 2) {
                        const uint64_t sd = tc::smem_desc_sw128(tc::smem_u32(sSlo), 16, 1024);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            mma_tmem_a(tmem + kColO1, tmem + kColSlo + 8 * ks, tc::desc_add(xd, ks * 32),
                                       id_o1, ks > 0);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16(tmem + kColO1, tc::desc_add(sd, ks * 32),
                                         tc::desc_add(xd, kBlock + ks * 32), id_o1, 1);
                    } else {
#pragma unroll 1
                        for (int q = NP - 2; q >= 0; --q) {
                            const uint64_t sd =
                                tc::smem_desc_sw128(tc::smem_u32(sSlo) + q * D * D * 2, 16, 1024);
#pragma unroll
                            for (int ks = 0; ks < 8; ++ks)
                                tc::mma_bf16(tmem + kColO1,
                                             tc::desc_add(sd, (ks >> 2) * (D * 128) + (ks & 3) * 32),
                                             tc::desc_add(xd, (ks >> 2) * kBlock + (ks & 3) * 32), id_o1,
                                             q < NP - 2 || ks > 0);
                        }
                    }
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_tmem_a(tmem + kColO1, tmem + kColS + 8 * ks,
                                   tc::desc_add(xd, (ks >> 2) * kBlock + (ks & 3) * 32), id_o1, 1);
                    tc::mma_commit(&b.s_empty);
                }
                __syncwarp();
                // O2: the chunk's own scores
                if (!(ok = wait(b, &b.p_full, i & 1))) break;
                tc::tc_fence_after();
                const uint64_t zd = tc::desc_add(zd0, at.slot * S::STAGE);
                if (elect_one()) {
#pragma unroll 1
                    for (int q = NP - 1; q >= 0; --q) {
                        const uint64_t pd =
                            tc::smem_desc_sw128(tc::smem_u32(sP) + q * kBlock, 16, 1024);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16(tmem + kColO2, tc::desc_add(zd, ks * 2048),
                                         tc::desc_add(pd, ks * 32), id_o2, q < NP - 1 || ks > 0);
                    }
                    tc::mma_commit(&b.p_empty);
                    tc::mma_commit(&b.o_full);
                    tc::mma_commit(&b.empty[at.slot]);
                }
                __syncwarp();
                at.next();
            }
        }
        // every copy has landed and every product finished before the memory is given back
#pragma unroll 1
        for (int i = sent > NS ? sent - NS : 0; i < sent; ++i) wait(b, &b.full[i % NS], (i / NS) & 1);
        uint64_t* drain = &b.drain[role];
        if (elect_one()) tc::mma_commit(drain);
        __syncwarp();
        wait(b, drain, 0);
        __syncwarp();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (b.abort && tid == 0) atomicCAS(&g_la_status, 0, kLaStatusWait);
    if (warp == S::EXTRA + 1) tc::tmem_dealloc(tmem, 512);
}

__global__ void la_status_move_kernel(int* word) {
    const int v = atomicExch(&g_la_status, 0);
    if (v != 0) atomicCAS(word, 0, v);
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// [rows][T][heads][128] bf16 as {channel, head, token, row}; boxes of 64 channels x 64 tokens of
// one head.  Tokens behind T read as zeros.  Stores: 32 x 32, tokens behind T are not written.
bool encode(CUtensorMap* m, const void* base, int heads, int T, int rows, bool store = false) {
    auto enc = encoder();
    if (!enc) return false;
    const cuuint64_t dims[4] = {D, (cuuint64_t)heads, (cuuint64_t)T, (cuuint64_t)rows};
    const cuuint64_t row = D * 2;
    const cuuint64_t strides[3] = {row, row * heads, row * heads * T};
    const cuuint32_t box[4] = {store ? 32u : 64u, 1, store ? 32u : (cuuint32_t)C, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, store ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NP, bool kSummary, bool kF32, bool kDots>
cudaError_t launch(const LaArgs& a, cudaStream_t s) {
    using S = TcShape<NP, kSummary>;
    TcArgs t;
    t.a = a;
    const int H = a.sp.H, rows = a.sp.cu ? 1 : a.sp.n;
    for (int r = 0; r < a.runs; ++r) {
        const LaRun& u = a.run[r];
        if ((!kSummary && !encode(&t.map[r][0], u.x, H / u.xg, a.sp.T, rows)) ||
            !encode(&t.map[r][1], u.y, H / u.yg, a.sp.T, rows) ||
            !encode(&t.map[r][2], u.z, H / u.zg, a.sp.T, rows))
            return cudaErrorInvalidValue;
        if (!kSummary && !kF32 && !encode(&t.out[r], u.out, H, a.sp.T, rows, true))
            return cudaErrorInvalidValue;
    }
    auto kern = la_tc_kernel<NP, kSummary, kF32, kDots>;
    // (an attribute of the kernel on the current device: set once for each)
    static std::atomic<unsigned long long> set{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(set.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        set.fetch_or(bit, std::memory_order_relaxed);
    }
    const dim3 grid((unsigned)(a.sp.units * H), a.runs);
    if (a.after) return la_launch_after(kern, grid, S::THREADS, S::SMEM, s, t);
    kern<<<grid, S::THREADS, S::SMEM, s>>>(t);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_tc_summary(const LaArgs& a, cudaStream_t s) {
    return launch<2, true, false, false>(a, s);
}
// (the runs of one launch agree in out_f32 and in having rows to multiply with; both go with exact ones)
cudaError_t launch_la_tc_run(const LaArgs& a, bool exact, cudaStream_t s) {
    const bool f32 = a.run[0].out_f32, dots = a.run[0].dot != nullptr;
    if (dots) return f32 ? launch<3, false, true, true>(a, s) : launch<3, false, false, true>(a, s);
    if (exact) return f32 ? launch<3, false, true, false>(a, s) : launch<3, false, false, false>(a, s);
    return launch<2, false, false, false>(a, s);
}

cudaError_t la_status_move(int* word, cudaStream_t stream) {
    la_status_move_kernel<<<1, 1, 0, stream>>>(word);
    return cudaGetLastError();
}

}  // namespace ckda
