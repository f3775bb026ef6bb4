// k_gdr_chunk_tc.cu — the gated delta rule over whole sequences in chunks of
// 32 tokens, on the 5th-generation tensor cores (bf16 inputs).
//
// With h the state entering a chunk (S x H), G the log decay summed from the
// chunk's start and K, Q, V its rows, the corrections w_i = beta_i (v_i - (state
// before token i, decayed)^T k_i) of
//     h_t = e^{g_t} h_{t-1} + k_t w_t^T,   y_t = scale h_t^T q_t
// solve a unit lower triangular system, and everything else is products:
//     A_ij = beta_i e^{G_i - G_j} (k_i . k_j)   (j < i),      N = (I + A)^-1
//     X = diag(beta) (V - diag(e^G) K h),                     W = N X
//     y = scale (diag(e^G) Q h + P W),  P_ij = e^{G_i - G_j} (q_i . k_j)  (j <= i)
//     h <- e^{G_last} h + K^T diag(e^{G_last - G}) W.
// q and k rows that are to be normalised stay as they are in shared memory:
// their norms are factors of rows and columns of the products above.
//
// GB300 design.  One CTA owns one head of up to 128 columns (or two heads of up to 64
// columns of one q/k group, NV = 2; smaller states and heads are filled up with zeros:
// 4 x 1024 tokens of 24 heads of 96 columns, S 96, 124 us, token by token 367) and
// walks the chunks; the carried state and every intermediate stay on the chip, so q,
// k, v, g, beta are read once and y is written once.  All products of the chain run
// transposed, with the head's columns as the 128 rows of the MMA: the fp32 state h^T
// lives in tensor memory, and what is fed back (h, X, W) is read from there,
// converted, and written back to tensor memory as the next product's left operand,
// while K, Q, N and P are right operands in shared memory, straight from the TMA or as
// the scores' warps wrote them.
//   warps 0-15   chain: h -> two bf16 parts and e^{G_last} h;  R = K h -> X;  W ->
//                its parts (four per TMEM lane quadrant, a quarter of the columns
//                each)
//   warps 16-19  output: y from Q h and P W
//   warps 20-23  G, k's norms, A and N's diagonal blocks of the next chunks, while the
//                chain runs on this one
//   warps 24-27  the rest of N, q's norms and P
//   warps 28-31  TMA producer of K and Q; TMA producer of V; issuers of the chain's
//                products and of P W (a product takes its issuer 46 cycles or more
//                however small it is, so P W would hold up the chain's)
// What bounds it is the chain from state to state: three dependent products and three
// conversions a chunk, about 3.5 us with two heads to a CTA and 3.0 with one, whatever
// the memory could do.  4 x 8192 tokens of 64 heads of 64 columns, S 128, 16 q/k
// groups: 907 us (0.93 TB/s of what has to move, 114 TFLOP/s of the recurrence's
// arithmetic); 4 x 4096 of 32 heads of 128: 406 us (1.04 TB/s; DRAM 10 %, tensor pipe
// 15 %, 0.56 instructions a cycle and scheduler); 1237 tokens alone: 119 us
// (before Q h took h's second part, 902, 395 and 119, and in some runs of the same binary
// 1004 and 429 for the first two; why is not shown).
//
// Precision.  What enters the fp32 state is as good as fp32: N, X and W take part in its
// products as three bf16 parts each (24 bits), h in the correction R as two (16 bits; R's
// share of an error decays with the state's). With two parts throughout, the state was 1e-6 to
// 3e-6 off on ordinary inputs and 2e-3 where keys agree and beta is 2 (N's entries are
// +-2 there and W's sums cancel).  The final state is 4e-7 to 6e-7 off, and up to
// 1.1e-6 in heads that hardly decay (fp32 2e-7 to 4e-7): a third part of h brought
// that to 0.7e-6 and cost 15 % of the time (4 x 4096, when it was tried: 396 -> 457 us),
// the rest is the tensor cores' accumulation, which rounds towards zero.  P, W and h enter y as
// two parts.  With keys that agree, P W sums corrections that cancel, and one part lost 1.8
// % of y's largest value; and P W cancels against Q h where a token overwrites a larger
// value, so Q h takes the h that R took (with h's high part alone, y of a token that
// overwrites one 100 times its size was 10 % off; both parts cost 1 to 3 % of the time).
// y is off by its rounding to bf16 alone, 1.658e-3 by norm.
//
// Chunks of 32 and not 64: N and P cost a chunk's square on the CUDA cores, and
// with 64 tokens N (about 12000 cycles a chunk for four warps) held up a chain of
// 8000.
//
// The scores K K^T and Q K^T are 16 x 16 pieces that are masked, scaled and fed on
// in registers; they use the warp-level mma, whose accumulators are registers.  N
// goes by blocks of 16: the diagonal blocks by forward substitution, then
// N_10 = -N_11 A_10 N_00, all in fp32.  Forward substitution by blocks is stable
// for any A; a product of powers of A would not be (equal keys make A all ones
// below the diagonal).
//
// G is summed in fixed point and kept as an integer and a fraction, so that
// G_i - G_j is good to 2^-22 even behind a token that forgets everything.
// A token's g is clamped to +-112 (162 in log2), beyond which e^g is 0 or infinity in
// fp32.
#include "gated_delta.cuh"
#include "tc_ptx.cuh"
#include "tmap_host.cuh"

namespace m2 {
namespace {

constexpr int kT = 32;  // tokens per chunk
constexpr int kChainWarps = 16, kOutWarps = 4, kNWarp0 = 20, kNWarps = 4, kPWarp0 = 24, kPWarps = 4;
constexpr int kTmaWarp = 28, kVWarp = 29, kMmaWarp = 30, kPwWarp = 31;
constexpr int kThreads = 32 * 32;    // 64 registers each
constexpr uint32_t kBox = kT * 128;  // one box: the chunk's tokens x 64 columns of bf16
constexpr int kMaxStages = 4, kMaxVStages = 4;
constexpr int kBufs = 4;  // of scalars and scratch: how far N's makers may be ahead of the outputs
constexpr int kSmemLimit = 232448;

struct Tok {       // what the scores need of a token
    float gi, gf;  // G in log2 units: integer part, fraction
    float rk;      // 1 / norm of k
    float beta;
};
// The block below the diagonal takes its decays from its rows' first token r,
// e^{G_i - G_j} = e^{G_i - G_r} e^{G_r - G_j}: both factors are at most 1 and one
// exponential serves a row or a column of the block.
struct Scalars {  // one head's, per chunk
    Tok tok[kT];
    float cb[kT], cr[kT];  // X = cb v + cr R
    float d[kT];           // W's share of the state
    float gam[kT];         // e^G
    float oq[kT];          // y = oq (gam Q h + P W)
    float g_last;          // e^{G_last}
    float pad[3];
};

// A head's results of the scores: N's three and P's two planes of 32 rows of 128
// bytes (the first 64 of each used), in one buffer each (they are needed late in
// a chunk, and written when the chunk before has used them), the scalars in kBufs.
constexpr uint32_t kPlane = kT * 128;
constexpr uint32_t kNPlanes = 3, kPPlanes = 2;
constexpr uint32_t kScalBytes = sizeof(Scalars);
static_assert(kScalBytes % 16 == 0, "scalars");

struct NScratch {           // one head's, per chunk, in fp32
    float diag[2][16][20];  // A's diagonal blocks, then N's, a column in a row
    float n10[16][20];      // N's block (1, 0) (behind the others: see its use)
    float low[16][20];      // A's block (1, 0)
    float4 fac[3][2][32];   // rk_j e^{G_i - G_j} of the blocks, as the mma's threads hold them: A's and P's factors
};

enum : int {
    kBarFull = 0,                         // [stages] K and Q
    kBarFree = kBarFull + kMaxStages,     // [stages] every reader of the stage is done
    kBarVFull = kBarFree + kMaxStages,    // [V stages]
    kBarVFree = kBarVFull + kMaxVStages,  // [V stages]
    kBarSFull = kBarVFree + kMaxVStages,  // [bufs] scalars but oq (and K's rows past the end cleared)
    kBarSFree = kBarSFull + kBufs,        // [bufs] scalars and scratch
    kBarDFull = kBarSFree + kBufs,        // [bufs] scratch: A's block and N's diagonal blocks, factors
    kBarHReady = kBarDFull + kBufs,        // h's parts are written; y's sum of the chunk before has been read
    kBarRDone,                            // R and Q h
    kBarXReady,                           // X's parts and N are written, h is decayed
    kBarWDone,
    kBarWReady,  // W's parts for the state
    kBarHDone,
    kBarPReady,  // P, oq and W's parts for y are written, Q h is scaled
    kBarPDone,   // P W
    kBarDrain,  // [2] issuers
    kNumBars = kBarDrain + 2
};

struct SharedCtl {
    uint32_t tmem_base;
    int abort;
    int never;  // stays 0: for drain waits, which no abort cuts short
};

struct GdrTcParams {
    Geom g;
    int nst, nvst;  // stages
    uint32_t off_v, off_n, off_p, off_scal, off_scratch, off_bar;
    const float* gate;
    const float* beta;
    const int32_t* lengths;
    const float* init;
    __nv_bfloat16* y;
    float* final_state;
    unsigned int* status;
    float scale, l2_eps;
    int l2norm;
};

__device__ __forceinline__ void set_abort(SharedCtl* ctl, unsigned int* status) {
    ctl->abort = 1;
    if (status) atomicExch(status, kStatusTimeout);
}

// A barrier of `threads` threads that also tells each whether all of them came
// with `ok`.
__device__ __forceinline__ bool bar_sync_and(int id, int threads, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "bar.red.and.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

// Waits for a phase: true once it has completed; false if the kernel was
// aborted, or after about 2 s.  A waiting thread costs the working warps issue
// slots with every look (looks with a clock and an abort flag beside them took
// half of all issued instructions), so a round of looks is a bare loop, and
// roles off the chain (SLEEP) sleep between looks.
template <bool SLEEP>
__device__ __forceinline__ bool thread_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const long long c0 = clock64();
    for (;;) {
#pragma unroll 1
        for (int i = 0; i < 64; ++i) {
            if (SLEEP) __nanosleep(40);
            if (tc::mbar_try_wait(bar, parity)) return true;
        }
        if (*abort != 0 || clock64() - c0 > tc::kWaitLimitCycles) return false;
    }
}
// A whole warp's wait: all lanes look (each sees the phase complete for itself)
// and leave with one answer.
template <bool SLEEP = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, thread_wait<SLEEP>(bar, parity, abort));
}

// Byte offset of 16-byte piece `ch` (of 8) of row `row` in a box of 128-byte
// rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw(uint32_t row, uint32_t ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d (16 x 8, fp32) += a (16 x 16) b (16 x 8)
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 4 columns of this warp's lanes (packed bf16 pairs).
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    tc::tmem_ld8_nowait(taddr, r);
    tc::tmem_wait_ld8(r);
}

// Four rows of a 16 x 16 block times a column: o += B[4 rows][16] x, with the
// block's columns at col(k) as float4 of these rows.
template <class Col>
__device__ __forceinline__ void block_times(float2 (&o)[2], const float (&x)[16], Col col) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float4 b = col(k);
        const float2 xk = make_float2(x[k], x[k]);
        o[0] = tc::fma_f32x2(make_float2(b.x, b.y), xk, o[0]);
        o[1] = tc::fma_f32x2(make_float2(b.z, b.w), xk, o[1]);
    }
}
// The 16 values of a column of which each of four neighbouring lanes has four.
__device__ __forceinline__ void gather(float (&x)[16], const float2 (&o)[2], int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x[4 * q] = __shfl_sync(0xffffffffu, o[0].x, (lane & ~3) | q);
        x[4 * q + 1] = __shfl_sync(0xffffffffu, o[0].y, (lane & ~3) | q);
        x[4 * q + 2] = __shfl_sync(0xffffffffu, o[1].x, (lane & ~3) | q);
        x[4 * q + 3] = __shfl_sync(0xffffffffu, o[1].y, (lane & ~3) | q);
    }
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// e^{G_i - G_j}
__device__ __forceinline__ float decay(const Tok& i, const Tok& j) { return ex2((i.gi - j.gi) + (i.gf - j.gf)); }

// A pair of fp32 values as its high bf16 parts, and what they leave.
__device__ __forceinline__ uint32_t high(float2& v) {
    const uint32_t hi = tc::pack_bf16x2(v.x, v.y);
    v = tc::fma_f32x2(make_float2(tc::bf16_lo(hi), tc::bf16_hi(hi)), make_float2(-1.f, -1.f), v);
    return hi;
}
// As its two bf16 parts, and as three.
__device__ __forceinline__ void split2(float2 v, uint32_t& hi, uint32_t& lo) {
    hi = high(v);
    lo = tc::pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ void split3(float2 v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = high(v);
    split2(v, mid, lo);
}
__device__ __forceinline__ float2 as_f2(const uint32_t* r) {
    return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// The 16 x 16 products of rows 16 i .. of tile x with rows 16 j .. of tile k (K
// or Q of a stage), summed over the S columns.
template <int S>
__device__ __forceinline__ void score_block(uint32_t x, uint32_t k, int i, int j, int lane, float (&acc)[2][4]) {
    float part[S / 64][2][4] = {};  // a chain of four for each box
    // pieces 2 ks, 2 ks + 1 of a row: the swizzled place of the first, with 2 ks' bits flipped
    const uint32_t xa = x + sw(16 * i + (lane & 15), lane >> 4);
    const uint32_t kb = k + sw(16 * j + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
#pragma unroll
    for (int box = 0; box < S / 64; ++box) {
        uint32_t a[4][4], b[4][4];
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            ldsm4((xa ^ (ks << 5)) + box * 2 * kBox, a[ks]);
            ldsm4((kb ^ (ks << 5)) + box * 2 * kBox, b[ks]);
        }
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            mma16(part[box][0], a[ks], b[ks][0], b[ks][1]);
            mma16(part[box][1], a[ks], b[ks][2], b[ks][3]);
        }
    }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = S == 128 ? part[0][nt][e] + part[S / 64 - 1][nt][e] : part[0][nt][e];
}

// 1 / sqrt(x + eps) of a block's diagonal, handed to put(row, value).
template <class Put>
__device__ __forceinline__ void diag_norm(const float (&acc)[2][4], int lane, float eps, Put put) {
    const int gid = lane >> 2, tig = lane & 3;
    if (gid >> 1 != tig) return;  // rows gid, gid + 8 meet their columns 2 tig, 2 tig + 1 here
    put(gid, __frsqrt_rn((gid & 1 ? acc[0][1] : acc[0][0]) + eps));
    put(gid + 8, __frsqrt_rn((gid & 1 ? acc[1][3] : acc[1][2]) + eps));
}

// S x H: the state's size, or with PAD what its size is filled up to.
template <int S, int H, int NV, bool PAD>
__global__ void __launch_bounds__(kThreads, 1)
k_gdr_chunk_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const GdrTcParams p) {
    constexpr int kBoxes = S / 64, kVBoxes = NV * H / 64;
    // A stage: K's and Q's boxes in turn, so that 32 rows of K and 32 of Q are one operand of 64.  V has
    // stages of its own (it is needed late and not for long).
    constexpr uint32_t kStage = 2 * kBoxes * kBox, kVStage = kVBoxes * kBox;
    static_assert((S == 64 || S == 128) && (NV == 1 ? (H == 64 || H == 128) : H == 64), "shapes");
    // Tensor memory columns (128 lanes = the head's columns; NV = 2: 64 of each head): h and its two parts,
    // R | Q h (then W | y's sum), the second head's W and y's sum (products with N and P cover all lanes,
    // and each head has its own), X's parts, W's parts for the state and for y.
    constexpr uint32_t cH = 0, cHi = S, cLo = S + S / 2, cR = 2 * S, cO = 2 * S + 32, cR2 = 2 * S + 64,
                       cO2 = 2 * S + 96, cX = 2 * S + 128, cU = 2 * S + 176, cW = 2 * S + 224;
    static_assert(cW + 32 <= 512, "tensor memory");

    // (aligned by an offset, so that the compiler still knows it for shared memory)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);
    const Geom& g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int h0 = NV * blockIdx.x;
    // Ragged batches: blocks are started in order, so the longest rows come first (16 rows of 0 to 1024
    // tokens, 16 heads of 128: 157 -> 130 us when it was added, 114 now).  A row's place is the number of rows before it.
    __shared__ int s_row;
    int64_t b = blockIdx.y;
    if (p.lengths && g.batch <= kThreads) {
        const int t = threadIdx.x, count = (int)g.batch;
        if (t < count) {
            const int64_t mine = row_length(p.lengths, t, g.seqlen);
            int before = 0;
            for (int i = 0; i < count; ++i) {
                const int64_t other = row_length(p.lengths, i, g.seqlen);
                before += other > mine || (other == mine && i < t);
            }
            if (before == (int)blockIdx.y) s_row = t;
        }
        __syncthreads();
        b = s_row;
    }
    const int grp = (int)(h0 / g.heads_per_group);
    const int64_t L = g.seqlen, n = row_length(p.lengths, b, L);
    const int nc = (int)((n + kT - 1) / kT);

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.off_bar);
    SharedCtl* ctl = reinterpret_cast<SharedCtl*>(smem + p.off_bar + kNumBars * 8);
    // head hv's N and P (planes of falling weight) and scalars
    auto n_of = [&](int hv) -> uint8_t* { return smem + p.off_n + hv * kNPlanes * kPlane; };
    auto p_of = [&](int hv) -> uint8_t* { return smem + p.off_p + hv * kPPlanes * kPlane; };
    auto scal_of = [&](int buf, int hv) -> Scalars* {
        return reinterpret_cast<Scalars*>(smem + p.off_scal + (buf * NV + hv) * kScalBytes);
    };
    auto scratch_of = [&](int buf, int hv) -> NScratch* {
        return reinterpret_cast<NScratch*>(smem + p.off_scratch) + buf * NV + hv;
    };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            tc::mbar_init(&bars[kBarFull + i], 1);
            tc::mbar_init(&bars[kBarFree + i], 1 + kPWarps);
        }
        for (int i = 0; i < kMaxVStages; ++i) {
            tc::mbar_init(&bars[kBarVFull + i], 1);
            tc::mbar_init(&bars[kBarVFree + i], kChainWarps);
        }
        for (int i = 0; i < kBufs; ++i) {
            tc::mbar_init(&bars[kBarSFull + i], kNWarps);
            tc::mbar_init(&bars[kBarSFree + i], 1 + kOutWarps + kPWarps);
            tc::mbar_init(&bars[kBarDFull + i], kNWarps);
        }
        for (int i = 0; i < 2; ++i) tc::mbar_init(&bars[kBarDrain + i], 1);
        tc::mbar_init(&bars[kBarHReady], kChainWarps + kOutWarps);
        tc::mbar_init(&bars[kBarRDone], 1);
        tc::mbar_init(&bars[kBarXReady], kChainWarps + kPWarps);
        tc::mbar_init(&bars[kBarWDone], 1);
        tc::mbar_init(&bars[kBarWReady], kChainWarps);
        tc::mbar_init(&bars[kBarHDone], 1);
        tc::mbar_init(&bars[kBarPReady], kChainWarps + kOutWarps + kPWarps);
        tc::mbar_init(&bars[kBarPDone], 1);
        ctl->abort = 0;
        ctl->never = 0;
        tc::fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&ctl->tmem_base, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = ctl->tmem_base;
    volatile int* abort_flag = &ctl->abort;
    volatile int* never = &ctl->never;
    bool ok = true;

    if (warp < kChainWarps) {
        // ============================== chain ==============================
        const int q = warp & 3, part = warp >> 2;
        const int hv = NV == 2 ? q >> 1 : 0;
        const int colh = 32 * (NV == 2 ? (q & 1) : q) + lane;  // column of its head
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const int rows = PAD ? (int)g.dstate : S, cols = PAD ? (int)g.headdim : H;
        const bool live = colh < cols;
        const int64_t sbase = (b * g.nheads + h0 + hv) * (int64_t)rows * cols + colh;
        const int s0 = part * (S / 4), i0 = part * (kT / 4);  // this warp's state rows and tokens
        const uint32_t w_at = tl + (hv ? cR2 : cR) + i0;       // W of its head
        // this thread's column of V in a stage: 16-byte piece and place in it
        const uint32_t vch = (32 * (q & 1) + lane) >> 3, vin = (lane & 7) * 2;
        uint8_t* v_at = smem + p.off_v + (q >> 1) * kBox + vin;
#pragma unroll 1
        for (int s = s0; s < s0 + S / 4; s += 16) {
            uint32_t r[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
                r[j] = live && p.init && (!PAD || s + j < rows) ? __float_as_uint(p.init[sbase + (int64_t)(s + j) * cols])
                                                                : 0u;
            tc::tmem_st16(tl + cH + s, r);
        }
        tc::tmem_wait_st();
        int vs = 0;
        uint32_t v_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c % kBufs;
            const uint32_t ph = c & 1;
            const Scalars* sc = scal_of(buf, hv);
            if (!warp_wait(&bars[kBarSFull + buf], (c / kBufs) & 1, abort_flag)) { ok = false; break; }
            const float g_last = sc->g_last;
            if (c > 0 && !warp_wait(&bars[kBarHDone], ph ^ 1, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            // h's parts
#pragma unroll 1
            for (int s = s0; s < s0 + S / 4; s += 16) {
                uint32_t r[16], hi[8], lo[8];
                tc::tmem_ld16(tl + cH + s, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) split2(as_f2(&r[2 * j]), hi[j], lo[j]);
                tc::tmem_st8(tl + cHi + s / 2, hi);
                tc::tmem_st8(tl + cLo + s / 2, lo);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarHReady]);
            // while R = K h runs: h decayed to the chunk's end, and V
#pragma unroll 1
            for (int s = s0; s < s0 + S / 4; s += 16) {
                uint32_t r[16];
                tc::tmem_ld16(tl + cH + s, r);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 v = tc::mul_f32x2(as_f2(&r[j]), make_float2(g_last, g_last));
                    r[j] = __float_as_uint(v.x);
                    r[j + 1] = __float_as_uint(v.y);
                }
                tc::tmem_st16(tl + cH + s, r);
            }
            if (!warp_wait(&bars[kBarVFull + vs], v_phase, abort_flag)) { ok = false; break; }
            float2 bv[4];
            {
                const uint8_t* sv = v_at + vs * kVStage + i0 * 128;
                const int64_t left = n - (int64_t)c * kT - i0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint32_t v = *reinterpret_cast<const uint16_t*>(sv + j * 128 + ((vch ^ j) << 4));
                    const float x = left > j ? tc::bf16_lo(v) * sc->cb[i0 + j] : 0.f;  // past the end, whatever is there
                    if (j & 1) bv[j / 2].y = x;
                    else bv[j / 2].x = x;
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarVFree + vs]);
            if (++vs == p.nvst) {
                vs = 0;
                v_phase ^= 1u;
            }
            if (!warp_wait(&bars[kBarRDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            // X (in lanes that have no column, whatever comes: nothing reads them)
            {
                uint32_t r[8], x0[4], x1[4], x2[4];
                tmem_ld8(tl + cR + i0, r);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    split3(tc::fma_f32x2(*reinterpret_cast<const float2*>(&sc->cr[i0 + 2 * j]), as_f2(&r[2 * j]), bv[j]),
                           x0[j], x1[j], x2[j]);
                tmem_st4(tl + cX + i0 / 2, x0);
                tmem_st4(tl + cX + 16 + i0 / 2, x1);
                tmem_st4(tl + cX + 32 + i0 / 2, x2);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarXReady]);

            // W = N X, decayed to the chunk's end for the state, then as it is for y
            if (!warp_wait(&bars[kBarWDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            {
                uint32_t r[8], x0[4], x1[4], x2[4];
                tmem_ld8(w_at, r);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    split3(tc::mul_f32x2(*reinterpret_cast<const float2*>(&sc->d[i0 + 2 * j]), as_f2(&r[2 * j])), x0[j],
                           x1[j], x2[j]);
                tmem_st4(tl + cU + i0 / 2, x0);
                tmem_st4(tl + cU + 16 + i0 / 2, x1);
                tmem_st4(tl + cU + 32 + i0 / 2, x2);
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[kBarWReady]);
#pragma unroll
                for (int j = 0; j < 4; ++j) split2(as_f2(&r[2 * j]), x0[j], x1[j]);
                tmem_st4(tl + cW + i0 / 2, x0);
                tmem_st4(tl + cW + 16 + i0 / 2, x1);
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[kBarPReady]);
            }
        }
        if (ok && nc > 0) ok = warp_wait(&bars[kBarHDone], (nc - 1) & 1, abort_flag);
        if (ok && p.final_state) {
            tc::tc_fence_after();
#pragma unroll 1
            for (int s = s0; s < s0 + S / 4; s += 16) {
                uint32_t r[16];
                tc::tmem_ld16(tl + cH + s, r);
                if (live) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (!PAD || s + j < rows) p.final_state[sbase + (int64_t)(s + j) * cols] = __uint_as_float(r[j]);
                }
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else if (warp < kNWarp0) {
        // ============================== output ==============================
        const int q = warp & 3;
        const int hv = NV == 2 ? q >> 1 : 0;
        const int colh = 32 * (NV == 2 ? (q & 1) : q) + lane;
        const int cols = PAD ? (int)g.headdim : H;
        const bool live = colh < cols;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const uint32_t o_at = tl + (hv ? cO2 : cO);
        const int64_t row = (int64_t)g.nheads * cols;
        const int odd = lane & 1;
        // lanes meet in pairs: the even one stores both columns of token i, the odd one of i + 1
        __nv_bfloat16* y = p.y + (b * L + odd) * row + (int64_t)(h0 + hv) * cols + (colh & ~1);
        if (lane == 0 && nc > 0) tc::mbar_arrive(&bars[kBarHReady]);  // no sum to be read yet
        for (int c = 0; c < nc; ++c) {
            const int buf = c % kBufs;
            const uint32_t ph = c & 1;
            const Scalars* sc = scal_of(buf, hv);
            // Q h -> e^G Q h, onto which P W is summed (the second head's in a place of its own)
            if (!warp_wait<true>(&bars[kBarSFull + buf], (c / kBufs) & 1, abort_flag)) { ok = false; break; }
            if (!warp_wait<true>(&bars[kBarRDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
#pragma unroll 1
            for (int m = 0; m < kT; m += 16) {
                uint32_t r[16];
                tc::tmem_ld16(tl + cO + m, r);
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float2 a = tc::mul_f32x2(*reinterpret_cast<const float2*>(&sc->gam[m + j]), as_f2(&r[j]));
                    r[j] = __float_as_uint(a.x);
                    r[j + 1] = __float_as_uint(a.y);
                }
                tc::tmem_st16(o_at + m, r);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarPReady]);
            if (!warp_wait<true>(&bars[kBarPDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            const int64_t nleft = n - (int64_t)c * kT, lleft = L - (int64_t)c * kT;
            const int nv = nleft < kT ? (int)nleft : kT, lv = live ? (lleft < kT ? (int)lleft : kT) : 0;
            __nv_bfloat16* yc = y + c * kT * row;
            // (all of it into registers: the next chunk's R | Q h waits for the place)
            uint32_t r[2][16];
            tc::tmem_ld16_nowait(o_at, r[0]);
            tc::tmem_ld16_nowait(o_at + 16, r[1]);
            tc::tmem_wait_ld16(r[0]);
            tc::tmem_tie16(r[1]);
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0 && c + 1 < nc) tc::mbar_arrive(&bars[kBarHReady]);
#pragma unroll
            for (int i = 0; i < kT; i += 2) {
                float2 a = tc::mul_f32x2(*reinterpret_cast<const float2*>(&sc->oq[i]), as_f2(&r[i >> 4][i & 15]));
                if (nv < kT) a = make_float2(i < nv ? a.x : 0.f, i + 1 < nv ? a.y : 0.f);
                const uint32_t both = tc::pack_bf16x2(a.x, a.y);  // this column of tokens i, i + 1
                const uint32_t other = __shfl_xor_sync(0xffffffffu, both, 1);
                const uint32_t pair = odd ? __byte_perm(other, both, 0x7632) : __byte_perm(both, other, 0x5410);
                if (i + odd < lv) *reinterpret_cast<uint32_t*>(yc) = pair;
                yc += 2 * row;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarSFree + buf]);
        }
        if (!ok) set_abort(ctl, p.status);
        if (ok && live)
            for (int64_t t = (int64_t)nc * kT; t + odd < L; t += 2) *reinterpret_cast<uint32_t*>(y + t * row) = 0u;
    } else if (warp < kPWarp0) {
        // ============== G, k's norms, A and N's diagonal blocks ==============
        // K K^T's blocks (0, 0), (1, 1), (1, 0) on warps 0 to 2, for all heads; warp 3: G and the scalars
        const int w = warp - kNWarp0;
        const int gid = lane >> 2, tig = lane & 3;
        const int64_t gbase = b * L * g.nheads + h0;
        // warp 3's lanes hold the next chunk's g and beta, a token each
        float gn[NV], bn[NV];
        auto fetch = [&](int c) {
            const int64_t t = (int64_t)c * kT + lane;
#pragma unroll
            for (int hv = 0; hv < NV; ++hv) {
                gn[hv] = t < n ? p.gate[gbase + t * g.nheads + hv] : 0.f;
                bn[hv] = t < n ? p.beta[gbase + t * g.nheads + hv] : 0.f;
            }
        };
        if (w == 3 && nc > 0) fetch(0);
        int st = 0;
        uint32_t full_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c % kBufs;
            // every warp comes to the barrier below, whatever its waits said
            if (ok && c >= kBufs) ok = warp_wait<true>(&bars[kBarSFree + buf], (c / kBufs - 1) & 1, abort_flag);
            if (w == 3 && ok) {
#pragma unroll
                for (int hv = 0; hv < NV; ++hv) {
                    // log2 decays as an integer and a fraction in units of 2^-24, summed apart
                    constexpr float kL = 1.44269502162933349609375f, kLrest = 1.925963033500011e-8f;  // log2 e
                    const float lim = fminf(fmaxf(gn[hv], -112.f), 112.f);  // |log2 decay| < 162
                    const float x = lim * kL, rest = fmaf(lim, kL, -x) + lim * kLrest, whole = floorf(x);
                    int si = (int)whole, sf = __float2int_rn(((x - whole) + rest) * 16777216.f);
#pragma unroll
                    for (int m = 1; m < 32; m <<= 1) {
                        const int oi = __shfl_up_sync(0xffffffffu, si, m), of = __shfl_up_sync(0xffffffffu, sf, m);
                        if (lane >= m) si += oi, sf += of;
                    }
                    Tok* t = &scal_of(buf, hv)->tok[lane];
                    t->gi = (float)(si + (sf >> 24));
                    t->gf = (float)(sf & 0xffffff) * 5.9604644775390625e-8f;
                    t->beta = gn[hv] != gn[hv] ? gn[hv] : bn[hv];  // a NaN decay shows in the token's correction
                }
                if (c + 1 < nc) fetch(c + 1);
            }
            if (ok) ok = warp_wait<true>(&bars[kBarFull + st], full_phase, abort_flag);
            uint8_t* sK = smem + st * kStage;
            const uint32_t aK = tc::smem_u32(sK);
            const int64_t left = n - (int64_t)c * kT;
            const int nv = left < kT ? (int)left : kT;
            if (ok && nv < kT && w < 2) {
                // past the row's end: K enters the state's product and has to be 0
                const int r = 16 * w + (lane >> 1);
                if (r >= nv)
                    for (int i = 0; i < S / 16; ++i)
                        *reinterpret_cast<uint4*>(sK + (S == 128 ? (lane & 1) * 2 * kBox + sw(r, i)
                                                                 : sw(r, 4 * (lane & 1) + i))) = make_uint4(0, 0, 0, 0);
                __syncwarp();
            }
            // The norms are K K^T's diagonal: summed by the same instructions as the rest, so that
            // rk_i rk_j (k_i . k_j) is 1 to rounding where keys agree.
            const int bi = w == 0 ? 0 : 1, bj = w == 1 ? 1 : 0;
            float acc[2][4];
            if (ok && w < 3) score_block<S>(aK, aK, bi, bj, lane, acc);
            if (ok && w < 2) {
#pragma unroll
                for (int hv = 0; hv < NV; ++hv) {
                    Tok* tok = scal_of(buf, hv)->tok + 16 * w;
                    if (p.l2norm) diag_norm(acc, lane, p.l2_eps, [&](int r, float f) { tok[r].rk = f; });
                    else if (lane < 16) tok[lane].rk = 1.f;
                }
            }
            ok = bar_sync_and(1, 32 * kNWarps, ok);
            if (!ok) break;
            if (w == 3) {
#pragma unroll
                for (int hv = 0; hv < NV; ++hv) {
                    Scalars* sc = scal_of(buf, hv);
                    const Tok t = sc->tok[lane], last = sc->tok[kT - 1];
                    const float e = ex2(t.gi) * ex2(t.gf);
                    sc->cb[lane] = t.beta;
                    sc->cr[lane] = -t.beta * e * t.rk;
                    sc->gam[lane] = e;
                    sc->d[lane] = ex2(last.gi - t.gi) * ex2(last.gf - t.gf) * t.rk;
                    if (lane == kT - 1) sc->g_last = e;
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarSFull + buf]);
            // A = beta rk rk decay (K K^T); rows past the end: 0, whatever their products are
            if (w < 3) {
                const bool in0 = 16 * bi + gid < nv, in1 = 16 * bi + gid + 8 < nv;
#pragma unroll 1
                for (int hv = 0; hv < NV; ++hv) {
                    const Tok* tok = scal_of(buf, hv)->tok;
                    NScratch* scr = scratch_of(buf, hv);
                    const Tok ti0 = tok[16 * bi + gid], ti1 = tok[16 * bi + gid + 8], tr = tok[16 * bi];
                    const float f0 = in0 ? ti0.beta * ti0.rk : 0.f, f1 = in1 ? ti1.beta * ti1.rk : 0.f;
                    const float e0 = decay(ti0, tr), e1 = decay(ti1, tr);
                    float(*a)[20] = w < 2 ? scr->diag[w] : scr->low;
#pragma unroll 1
                    for (int nt = 0; nt < 2; ++nt) {
                        float c[2][2], s[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[x] = nt ? acc[1][x] : acc[0][x];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int jj = 8 * nt + 2 * tig + x;
                            const Tok tj = tok[16 * bj + jj];
                            if (w < 2) {
                                c[0][x] = tj.rk * decay(ti0, tj);
                                c[1][x] = tj.rk * decay(ti1, tj);
                            } else {
                                const float cj = tj.rk * decay(tr, tj);
                                c[0][x] = e0 * cj;
                                c[1][x] = e1 * cj;
                            }
                            a[jj][gid] = in0 && (w == 2 || jj < gid) ? s[x] * (f0 * c[0][x]) : 0.f;
                            a[jj][gid + 8] = in1 && (w == 2 || jj < gid + 8) ? s[2 + x] * (f1 * c[1][x]) : 0.f;
                        }
                        scr->fac[w][nt][lane] = make_float4(c[0][0], c[0][1], c[1][0], c[1][1]);
                    }
                }
            }
            __syncwarp();
            // N's diagonal blocks, a column per lane; the warp's halves take the two heads (or the same one)
            if (w < 2) {
                const int l = lane & 15;
                float(*a)[20] = scratch_of(buf, NV == 2 ? lane >> 4 : 0)->diag[w];
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = i == l ? 1.f : 0.f;
#pragma unroll
                for (int m = 0; m < 15; ++m) {
#pragma unroll
                    for (int i4 = (m + 1) / 4; i4 < 4; ++i4) {
                        const float4 v = *reinterpret_cast<const float4*>(&a[m][4 * i4]);
                        if (4 * i4 > m) x[4 * i4] = fmaf(-v.x, x[m], x[4 * i4]);
                        if (4 * i4 + 1 > m) x[4 * i4 + 1] = fmaf(-v.y, x[m], x[4 * i4 + 1]);
                        if (4 * i4 + 2 > m) x[4 * i4 + 2] = fmaf(-v.z, x[m], x[4 * i4 + 2]);
                        if (4 * i4 + 3 > m) x[4 * i4 + 3] = fmaf(-v.w, x[m], x[4 * i4 + 3]);
                    }
                }
                __syncwarp();
                if (NV == 2 || lane < 16)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4*>(&a[l][i]) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarDFull + buf]);
            if (++st == p.nst) {
                st = 0;
                full_phase ^= 1u;
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else if (warp < kTmaWarp) {
        // ==================== the rest of N, q's norms and P ====================
        // Q K^T's blocks (0, 0), (1, 1), (1, 0) on warps 0 to 2, for all heads; warp 3: Q Q^T's diagonal
        const int w = warp - kPWarp0;
        const int gid = lane >> 2, tig = lane & 3;
        int st = 0;
        uint32_t full_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c % kBufs;
            // N's place is free once the last chunk's W is done
            ok = warp_wait<true>(&bars[kBarFull + st], full_phase, abort_flag) &&
                 warp_wait<true>(&bars[kBarDFull + buf], (c / kBufs) & 1, abort_flag) &&
                 (c == 0 || warp_wait<true>(&bars[kBarWDone], (c - 1) & 1, abort_flag));
            if (!ok) break;
            // N_10 = -N_11 A_10 N_00 and all of N into its planes, eight columns (of a head's half) to a
            // warp, four lanes to a column, four rows each
            if (w < 2 * NV) {
                const int hv = w >> 1, col = 8 * (w & 1) + (lane >> 2), r4 = lane & 3;
                const NScratch& m = *scratch_of(buf, hv);
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(&m.diag[0][col][i]);
                    x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
                }
                float2 o[2];
#pragma unroll (NV)
                for (int f = 0; f < 2; ++f) {  // A_10's product, then N_11's
                    const float(*blk)[20] = f ? m.diag[1] : m.low;
                    o[0] = o[1] = make_float2(0.f, 0.f);
                    block_times(o, x, [&](int k) { return *reinterpret_cast<const float4*>(&blk[k][4 * r4]); });
                    gather(x, o, lane);
                }
                NScratch& to = *scratch_of(buf, hv);
                *reinterpret_cast<float4*>(&to.n10[col][4 * r4]) = make_float4(-o[0].x, -o[0].y, -o[1].x, -o[1].y);
                const uint32_t at = p.off_n + hv * kNPlanes * kPlane + 2 * (col & 7);
#pragma unroll 1
                for (int blk = 0; blk < 3; ++blk) {  // (0, 0), (1, 1), (1, 0), one behind the other in the scratch
                    const float4 f = *reinterpret_cast<const float4*>(&to.diag[0][0][0] + blk * 320 + col * 20 + 4 * r4);
                    const int row = (blk ? 16 : 0) + 4 * r4, ch = (blk == 1 ? 2 : 0) + (col >> 3);
                    float2 v0 = make_float2(f.x, f.y), v1 = make_float2(f.z, f.w);
#pragma unroll
                    for (uint32_t pl = 0; pl < kNPlanes; ++pl) {
                        const uint32_t t0 = high(v0), t1 = high(v1);
                        uint8_t* dst = smem + at + pl * kPlane;
                        *reinterpret_cast<uint16_t*>(dst + sw(row, ch)) = (uint16_t)t0;
                        *reinterpret_cast<uint16_t*>(dst + sw(row + 1, ch)) = (uint16_t)(t0 >> 16);
                        *reinterpret_cast<uint16_t*>(dst + sw(row + 2, ch)) = (uint16_t)t1;
                        *reinterpret_cast<uint16_t*>(dst + sw(row + 3, ch)) = (uint16_t)(t1 >> 16);
                    }
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarXReady]);
            const uint32_t aK = tc::smem_u32(smem + st * kStage), aQ = aK + kBox;
#pragma unroll 1
            for (int r = 0; r < (w == 3 ? 2 : 1); ++r) {
                const int bi = w == 3 ? r : (w == 0 ? 0 : 1), bj = w == 3 ? r : (w == 1 ? 1 : 0), i0 = 16 * bi + gid;
                float acc[2][4];
                if (w < 3 || p.l2norm) score_block<S>(aQ, w == 3 ? aQ : aK, bi, bj, lane, acc);
                // P's place is free once the last chunk's P W is done
                if (c > 0) ok = warp_wait<true>(&bars[kBarPDone], (c - 1) & 1, abort_flag);
                if (!ok) break;
                if (w == 3) {
                    if (p.l2norm) {
                        diag_norm(acc, lane, p.l2_eps, [&](int r16, float f) {
#pragma unroll
                            for (int hv = 0; hv < NV; ++hv) scal_of(buf, hv)->oq[16 * bi + r16] = p.scale * f;
                        });
                    } else if (lane < 16) {
#pragma unroll
                        for (int hv = 0; hv < NV; ++hv) scal_of(buf, hv)->oq[16 * bi + lane] = p.scale;
                    }
                    continue;
                }
#pragma unroll 1
                for (int t = 0; t < 2 * NV; ++t) {
                    const int hv = t >> 1, nt = t & 1, j0 = 16 * bj + 8 * nt + 2 * tig;
                    uint8_t* sP = p_of(hv);
                    const float4 f = scratch_of(buf, hv)->fac[w][nt][lane];
                    float2 a0 = nt ? make_float2(acc[1][0], acc[1][1]) : make_float2(acc[0][0], acc[0][1]);
                    float2 a1 = nt ? make_float2(acc[1][2], acc[1][3]) : make_float2(acc[0][2], acc[0][3]);
                    a0 = tc::mul_f32x2(make_float2(f.x, f.y), a0);
                    a1 = tc::mul_f32x2(make_float2(f.z, f.w), a1);
                    // (in block (1, 0) every j is below every i)
                    a0 = make_float2(j0 <= i0 ? a0.x : 0.f, j0 + 1 <= i0 ? a0.y : 0.f);
                    a1 = make_float2(j0 <= i0 + 8 ? a1.x : 0.f, j0 + 1 <= i0 + 8 ? a1.y : 0.f);
                    const uint32_t o0 = sw(i0, 2 * bj + nt) + 4 * tig;
                    uint32_t hi, lo;
                    split2(a0, hi, lo);
                    *reinterpret_cast<uint32_t*>(sP + o0) = hi;
                    *reinterpret_cast<uint32_t*>(sP + kPlane + o0) = lo;
                    split2(a1, hi, lo);
                    *reinterpret_cast<uint32_t*>(sP + o0 + 1024) = hi;
                    *reinterpret_cast<uint32_t*>(sP + kPlane + o0 + 1024) = lo;
                }
            }
            if (!ok) break;
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&bars[kBarPReady]);
                tc::mbar_arrive(&bars[kBarSFree + buf]);
                tc::mbar_arrive(&bars[kBarFree + st]);
            }
            if (++st == p.nst) {
                st = 0;
                full_phase ^= 1u;
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else {
        if (warp == kTmaWarp) {
            // ============================ TMA producer ============================
            if (lane == 0) {
                tc::tma_prefetch_desc(&tm_q);
                tc::tma_prefetch_desc(&tm_k);
                int fills[kMaxStages] = {};
                int st = 0;
                uint32_t free_phase = 1;
                for (int c = 0; c < nc; ++c) {
                    if (c >= p.nst && !thread_wait<true>(&bars[kBarFree + st], free_phase, abort_flag)) { ok = false; break; }
                    uint8_t* s = smem + st * kStage;
                    uint64_t* full = &bars[kBarFull + st];
                    tc::mbar_arrive_expect_tx(full, kStage);
#pragma unroll
                    for (int x = 0; x < kBoxes; ++x) {
                        tc::tma_load_4d(s + 2 * x * kBox, &tm_k, full, 64 * x, grp, c * kT, (int)b);
                        tc::tma_load_4d(s + (2 * x + 1) * kBox, &tm_q, full, 64 * x, grp, c * kT, (int)b);
                    }
                    ++fills[st];
                    if (++st == p.nst) {
                        st = 0;
                        free_phase ^= 1u;
                    }
                }
                if (!ok) set_abort(ctl, p.status);
                // no copy may still be landing when the CTA exits
    #pragma unroll
                for (int i = 0; i < kMaxStages; ++i)
                    if (fills[i] > 0) (void)tc::mbar_wait(&bars[kBarFull + i], (fills[i] - 1) & 1, never);
            }
        } else if (warp == kVWarp) {
            // ========================= TMA producer of V =========================
            if (lane == 0) {
                tc::tma_prefetch_desc(&tm_v);
                int fills[kMaxVStages] = {};
                int vs = 0;
                uint32_t free_phase = 1;
                for (int c = 0; c < nc; ++c) {
                    if (c >= p.nvst && !thread_wait<true>(&bars[kBarVFree + vs], free_phase, abort_flag)) {
                        ok = false;
                        break;
                    }
                    uint64_t* full = &bars[kBarVFull + vs];
                    tc::mbar_arrive_expect_tx(full, kVStage);
#pragma unroll
                    for (int x = 0; x < kVBoxes; ++x)
                        tc::tma_load_4d(smem + p.off_v + vs * kVStage + x * kBox, &tm_v, full, NV == 2 ? 0 : 64 * x,
                                        NV == 2 ? h0 + x : h0, c * kT, (int)b);
                    ++fills[vs];
                    if (++vs == p.nvst) {
                        vs = 0;
                        free_phase ^= 1u;
                    }
                }
                if (!ok) set_abort(ctl, p.status);
#pragma unroll
                for (int i = 0; i < kMaxVStages; ++i)
                    if (fills[i] > 0) (void)tc::mbar_wait(&bars[kBarVFull + i], (fills[i] - 1) & 1, never);
            }
        } else if (warp == kMmaWarp) {
            // ==================== issuer of the chain's products ====================
            if (lane == 0 && nc > 0) {
                constexpr uint32_t id_t = tc::idesc_bf16(128, kT, false, false);       // N = tokens
                constexpr uint32_t id_rq = tc::idesc_bf16(128, 2 * kT, false, false);  // of K and of Q
                constexpr uint32_t id_s = tc::idesc_bf16(128, S, false, true);         // N = state rows
                const uint64_t dN = tc::sdesc_sw128(tc::smem_u32(smem + p.off_n), 16, 1024);
                int st = 0;
                for (int c = 0; c < nc; ++c) {
                    const int buf = c % kBufs;
                    const uint32_t ph = c & 1;
                    const uint32_t aK = tc::smem_u32(smem + st * kStage);
                    const uint64_t dK = tc::sdesc_sw128(aK, 16, 1024);
                    const uint64_t dKt = tc::sdesc_sw128(aK, 2 * kBox, 1024);
                    // R | Q h from h's high part, then from its low part (Q h too: P W, made from this R, cancels
                    // against it).  (The chain has waited for the scalars, and their makers for K and Q; K's rows
                    // past the end they cleared.)
                    if (!thread_wait<false>(&bars[kBarHReady], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 2 * kBoxes; ++x) {
                        const uint32_t box = x < kBoxes ? x : x - kBoxes;
                        const uint64_t d = dK + box * (2 * kBox >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            tc::mma_bf16_ts(tmem + cR, tmem + cHi + 32 * x + 8 * ks, d + 2 * ks, id_rq,
                                            x > 0 || ks > 0);
                    }
                    tc::mma_commit(&bars[kBarRDone]);
                    // W = N X, N's parts times X's down to 2^-16 of hi hi; N's second block column only has
                    // rows from 16 on
                    if (!thread_wait<false>(&bars[kBarXReady], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 2 * NV; ++x) {
                        const int kb = x & 1, hv = x >> 1;
                        const uint32_t a = tmem + cX + 8 * kb, d = tmem + (hv ? cR2 : cR) + 16 * kb;
                        const uint32_t id = id_t - (static_cast<uint32_t>(2 * kb) << 17);  // N = 32 - 16 kb
                        const uint64_t at = dN + hv * (kNPlanes * kPlane >> 4) + ((2048 >> 4) + 2) * kb;
                        tc::mma_bf16_ts(d, a, at, id, kb);
                        tc::mma_bf16_ts(d, a, at + (kPlane >> 4), id, 1);
                        tc::mma_bf16_ts(d, a, at + 2 * (kPlane >> 4), id, 1);
                        tc::mma_bf16_ts(d, a + 16, at, id, 1);
                        tc::mma_bf16_ts(d, a + 16, at + (kPlane >> 4), id, 1);
                        tc::mma_bf16_ts(d, a + 32, at, id, 1);
                    }
                    tc::mma_commit(&bars[kBarWDone]);
                    // h += K^T W
                    if (!thread_wait<false>(&bars[kBarWReady], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
#pragma unroll
                    for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            tc::mma_bf16_ts(tmem + cH, tmem + cU + 16 * part + 8 * kt, dKt + 128 * kt, id_s, 1);
                    }
                    tc::mma_commit(&bars[kBarHDone]);
                    tc::mma_commit(&bars[kBarSFree + buf]);
                    tc::mma_commit(&bars[kBarFree + st]);
                    if (++st == p.nst) st = 0;
                }
                if (!ok) set_abort(ctl, p.status);
                // no product may still run when the tensor memory is freed
                tc::mma_commit(&bars[kBarDrain]);
                (void)tc::mbar_wait(&bars[kBarDrain], 0, never);
            }
        } else if (warp == kPwWarp) {
            // ========================= issuer of P W =========================
            if (lane == 0 && nc > 0) {
                constexpr uint32_t id_t = tc::idesc_bf16(128, kT, false, false);
                const uint64_t dP = tc::sdesc_sw128(tc::smem_u32(smem + p.off_p), 16, 1024);
                for (int c = 0; c < nc; ++c) {
                    // onto the scaled Q h: hi hi + hi lo + lo hi
                    if (!thread_wait<true>(&bars[kBarPReady], c & 1, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int x = 0; x < 2 * NV; ++x) {
                        const int kb = x & 1, hv = x >> 1;
                        const uint32_t a = tmem + cW + 8 * kb, d = tmem + (hv ? cO2 : cO) + 16 * kb;
                        const uint32_t id = id_t - (static_cast<uint32_t>(2 * kb) << 17);
                        const uint64_t at = dP + hv * (kPPlanes * kPlane >> 4) + ((2048 >> 4) + 2) * kb;
                        tc::mma_bf16_ts(d, a, at, id, 1);
                        tc::mma_bf16_ts(d, a, at + (kPlane >> 4), id, 1);
                        tc::mma_bf16_ts(d, a + 16, at, id, 1);
                    }
                    tc::mma_commit(&bars[kBarPDone]);
                }
                if (!ok) set_abort(ctl, p.status);
                tc::mma_commit(&bars[kBarDrain + 1]);
                (void)tc::mbar_wait(&bars[kBarDrain + 1], 0, never);
            }
        }
    }

    tc::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        __syncwarp();
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

bool aligned16(const void* p, int64_t stride) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride % 8 == 0; }

template <int S, int H, int NV, bool PAD>
cudaError_t launch_k(const GdrArgs& a, cudaStream_t st) {
    const Geom& g = a.g;
    GdrTcParams p{};
    p.g = g;
    p.gate = a.gate;
    p.beta = a.beta;
    p.lengths = a.lengths;
    p.init = a.init;
    p.y = static_cast<__nv_bfloat16*>(a.y);
    p.final_state = a.final_state;
    p.status = device_status_word();
    p.scale = a.scale;
    p.l2_eps = a.l2_eps;
    p.l2norm = a.l2norm;
    constexpr uint32_t stage = 2 * (S / 64) * kBox, vstage = NV * H / 64 * kBox;
    constexpr uint32_t rest = kMaxVStages * vstage + NV * ((kNPlanes + kPPlanes) * kPlane + kBufs * kScalBytes) +
                              kBufs * NV * (uint32_t)sizeof(NScratch) + kNumBars * 8 + (uint32_t)sizeof(SharedCtl) + 1024;
    static_assert(kMaxStages * stage + rest <= (uint32_t)kSmemLimit, "shared memory");
    p.nst = kMaxStages;
    p.nvst = kMaxVStages;
    p.off_v = kMaxStages * stage;
    p.off_n = p.off_v + kMaxVStages * vstage;
    p.off_p = p.off_n + NV * kNPlanes * kPlane;
    p.off_scal = p.off_p + NV * kPPlanes * kPlane;
    p.off_scratch = p.off_scal + kBufs * NV * kScalBytes;
    p.off_bar = p.off_scratch + kBufs * NV * (uint32_t)sizeof(NScratch);
    const int smem = (int)(kMaxStages * stage + rest);

    CUtensorMap tm_q, tm_k, tm_v;
    const uint64_t L = g.seqlen, B = g.batch;
    const uint32_t box[4] = {64, 1, kT, 1};
    auto map = [&](CUtensorMap* m, const void* base, uint64_t width, uint64_t count, uint64_t stride) {
        const uint64_t dims[4] = {width, count, L, B};
        const uint64_t strides[3] = {width * 2, stride * 2, L * stride * 2};
        return make_tmap_bf16(m, base, 4, dims, strides, box);
    };
    if (!map(&tm_q, a.q, g.dstate, g.ngroups, a.q_stride) || !map(&tm_k, a.k, g.dstate, g.ngroups, a.k_stride) ||
        !map(&tm_v, a.v, g.headdim, g.nheads, a.v_stride))
        return cudaErrorInvalidValue;
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(k_gdr_chunk_tc<S, H, NV, PAD>), smem);
    if (e != cudaSuccess) return e;
    k_gdr_chunk_tc<S, H, NV, PAD><<<dim3((unsigned)(g.nheads / NV), (unsigned)g.batch), kThreads, smem, st>>>(tm_q, tm_k, tm_v, p);
    return cudaGetLastError();
}

template <bool PAD>
cudaError_t launch_shape(const GdrArgs& a, bool wide, bool pairs, cudaStream_t st) {
    if (a.g.dstate > 64) {
        if (wide) return launch_k<128, 128, 1, PAD>(a, st);
        return pairs ? launch_k<128, 64, 2, PAD>(a, st) : launch_k<128, 64, 1, PAD>(a, st);
    }
    if (wide) return launch_k<64, 128, 1, PAD>(a, st);
    return pairs ? launch_k<64, 64, 2, PAD>(a, st) : launch_k<64, 64, 1, PAD>(a, st);
}

}  // namespace

// bf16 shapes the kernel covers: states and heads of up to 128 rows and columns, filled up
// to 64 or 128 with zeros by the TMA, which wants every row of q, k and v (and every head
// of a row) on a 16-byte boundary.
bool gdr_chunk_tc_fits(const GdrArgs& a) {
    const Geom& g = a.g;
    if (g.dstate > 128 || g.headdim > 128 || g.dstate % 8 != 0 || g.headdim % 8 != 0) return false;
    if (g.seqlen >= ((int64_t)1 << 30) || g.nheads > 65535) return false;
    return aligned16(a.q, a.q_stride) && aligned16(a.k, a.k_stride) && aligned16(a.v, a.v_stride);
}

// Two heads of up to 64 columns to a CTA where there are more heads than SMs: a chunk of
// two takes a sixth longer than one of one head (1024 tokens, S 128, us with one head to a CTA
// / two: 64 heads 120 / 135, 128 heads 123 / 135, 256 heads 240 / 140).
cudaError_t launch_gdr_chunk_tc(const GdrArgs& a, cudaStream_t st) {
    const int sms = sm_count();
    const bool wide = a.g.headdim > 64;
    const bool pairs = !wide && a.g.heads_per_group % 2 == 0 && a.g.batch * a.g.nheads > (sms > 0 ? sms : 152);
    const bool pad = a.g.dstate % 64 != 0 || a.g.headdim % 64 != 0;
    return pad ? launch_shape<true>(a, wide, pairs, st) : launch_shape<false>(a, wide, pairs, st);
}

}  // namespace m2
