// k_gdr_chunk_tc.cu — the gated delta rule over whole sequences in chunks of
// 64 tokens, on the 5th-generation tensor cores (bf16 inputs).
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
// GB300 design.  One CTA owns one head of up to 128 columns (or two heads of 64
// columns of one q/k group, NV = 2) and walks the chunks; the carried state and
// every intermediate stay on the chip, so q, k, v, g, beta are read once and y
// is written once.  All products of the chain run transposed, with the head's
// columns as the 128 rows of the MMA: the fp32 state h^T lives in tensor memory,
// and what is fed back (h, X, W) is read from there, converted, and written back
// to tensor memory as the next product's left operand, while K, Q, N and P are
// right operands in shared memory, straight from the TMA or as the scores' warps
// wrote them.
//   warps 0-7    chain: h -> two bf16 parts and e^{G_last} h;  R = K h -> X;  W ->
//                its parts (two per TMEM lane quadrant, half of the columns each)
//   warps 8-11   output: y from Q h and P W
//   then 4 NV    G, k's norms, A and N of the next chunk, while the chain runs on
//                this one (four warps to a head)
//   then 4       q's norms and P
//   then 1, 1    TMA producer; tcgen05.mma issuer
// What bounds it is the chain from state to state: three dependent products and
// three conversions a chunk.  What enters the fp32 state is as good as fp32: N, X
// and W take part in its products as three bf16 parts each (24 bits), h in the
// correction R as two (16 bits; R's share of an error decays with the state's).
// With two parts throughout, the state was 1e-6 to 3e-6 off on ordinary inputs
// and 2e-3 where keys agree and beta is 2 (N's entries are +-2 there and W's sums
// cancel).  P and W enter y as two parts: with keys that agree, P W sums
// corrections that cancel, and one part lost 1.8 % of y's largest value.  Q h
// takes h's high part.
//
// The scores K K^T and Q K^T and N's off-diagonal blocks are 16 x 16 pieces that
// are masked, scaled and fed on in registers; they use the warp-level mma, whose
// accumulators are registers, and leave the tensor memory (all 512 columns of it)
// to the chain.  N = (I + A)^-1 goes by blocks of 16: the diagonal blocks by
// forward substitution in fp32, then N_ij = -N_ii sum_{j <= m < i} A_im N_mj
// below them, in products of tf32 parts (two of 11 bits each: three products).
// Forward substitution by blocks is stable for any A; a product of powers of A
// would not be (equal keys make A all ones below the diagonal).
//
// G is summed in fixed point and kept as an integer and a fraction, so that
// G_i - G_j is good to 2^-22 even behind a token that forgets everything.
// Log2 decays of a token are clamped to +-160, beyond which fp32 has only 0 and
// infinity.
#include "gated_delta.cuh"
#include "tc_ptx.cuh"
#include "tmap_host.cuh"

namespace m2 {
namespace {

constexpr int kT = 64;             // tokens per chunk
constexpr int kChainWarps = 8, kOutWarp0 = 8, kOutWarps = 4, kNWarp0 = 12, kPWarps = 4;
// whole warpgroups, for the register split: the last one is TMA, MMA and two idle warps
constexpr int threads_of(int nv) { return (kNWarp0 + 4 * nv + kPWarps + 4) * 32; }
constexpr uint32_t kBox = kT * 128;  // one box: 64 tokens x 64 columns of bf16
constexpr int kMaxStages = 3;
constexpr int kSmemLimit = 232448;

struct Tok {       // what the scores need of a token
    float gi, gf;  // G in log2 units: integer part, fraction
    float rk;      // 1 / norm of k
    float beta;
};
// Blocks below the diagonal take their decays from the first token r of their
// rows' block, e^{G_i - G_j} = e^{G_i - G_r} e^{G_r - G_j}: both factors are at
// most 1 and one exponential serves a row or a column of the block.
struct Scalars {  // one head's, per chunk
    Tok tok[kT];
    float cb[kT], cr[kT];  // X = cb v + cr R
    float d[kT];           // W's share of the state
    float gam[kT];         // e^G
    float oq[kT];          // y = oq (gam Q h + P W)
    float el[kT];          // e^{G_i - G_r}
    float ea[kT];          // beta_i rk_i e^{G_i - G_r}
    float g_last;          // e^{G_last}
    float pad[3];
};

// A head's results of the scores: N's three and P's two planes of 64 rows of
// 128 bytes, in one buffer each (they are needed late in a chunk, and written
// when the chunk before has used them), the scalars in two.
constexpr uint32_t kPlane = kT * 128;
constexpr uint32_t kNPlanes = 3, kPPlanes = 2;
constexpr uint32_t kScalBytes = sizeof(Scalars);
static_assert(kScalBytes % 16 == 0, "scalars");

struct NScratch {           // one head's
    float diag[4][16][20];  // A's diagonal blocks, [column][row]; then N's, [row][column]
    float2 low[6][16][8];   // A's blocks below the diagonal, see low_at
};
// Place of columns 2 c2, 2 c2 + 1 of row r in a block of `low` (spread over the
// banks for eight rows by four pairs).
__device__ __forceinline__ int low_at(int r, int c2) { return c2 ^ (((r >> 1) & 1) << 2); }
__device__ __forceinline__ int low_block(int i, int m) { return i * (i - 1) / 2 + m; }

// The ten 16 x 16 blocks (i, j) of a lower triangle, in rounds of four warps:
// block t = 4 round + warp, the diagonal first.
__device__ __forceinline__ int tri_i(int t) { return (0x3323213210 >> (4 * t)) & 15; }
__device__ __forceinline__ int tri_j(int t) { return (0x0102103210 >> (4 * t)) & 15; }

enum : int {
    kBarFull = 0,                        // [stages] TMA
    kBarFree = kBarFull + kMaxStages,    // [stages] every reader of the stage is done
    kBarSFull = kBarFree + kMaxStages,   // [2] scalars but out (and K's rows past the end cleared)
    kBarSFree = kBarSFull + 2,           // [2]
    kBarNFull = kBarSFree + 2,           // N; free again with kBarWDone
    kBarPFull,                           // P and the scalars' out
    kBarPFree,
    kBarHReady,  // h's parts are written, h is decayed
    kBarRDone,   // R and Q h
    kBarXReady,
    kBarWDone,
    kBarWReady,   // W's parts for the state
    kBarWyReady,  // and for y
    kBarHDone,
    kBarO1Read,
    kBarO2Done,  // P W
    kBarO2Read,
    kBarDrain,
    kNumBars
};

struct SharedCtl {
    uint32_t tmem_base;
    int abort;
    int never;  // stays 0: for drain waits, which no abort cuts short
};

struct GdrTcParams {
    Geom g;
    int nst;  // stages
    uint32_t off_n, off_p, off_y, off_scal, off_scratch, off_bar;
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

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// bar_sync that also tells every thread whether all of them came with `ok`.
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

// A whole warp's wait for a phase: true once it has completed; false if the
// kernel was aborted, or after about 2 s.  try_wait suspends the warp in
// hardware, so a waiting warp takes few issue slots from working ones.  All
// lanes leave with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    bool done = tc::mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, done)) {
        const long long c0 = clock64();
        bool give_up = false;
        do {
            done = tc::mbar_try_wait(bar, parity);
            give_up = *abort != 0 || clock64() - c0 > tc::kWaitLimitCycles;
            done = __all_sync(0xffffffffu, done);
            give_up = __any_sync(0xffffffffu, give_up);
        } while (!done && !give_up);
    }
    return done;
}

// Registers per thread of the calling warpgroup from here on.  A block is
// launched with threads_of(NV) x 80 (NV = 2: x 72) registers; the groups'
// shares (chain twice) sum to 480 and 504 a thread of a warpgroup, six times 80
// and seven times 72.
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
__device__ __forceinline__ void stsm4_trans(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
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

// d (16 x 8) += a (16 x 8) b (8 x 8) of fp32 values, each as two tf32 parts
// (hi hi + hi lo + lo hi).  The order of the contracted index is free, and is
// chosen so that an accumulator is a left operand as it is: a thread's
// positions t and t + 4 are columns 2 t and 2 t + 1.  b is transposed: b.x, b.y
// are row g's (n) columns 2 t, 2 t + 1.
__device__ __forceinline__ uint32_t tf32_rn(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// d += a b over 16 columns of fp32 values: a an accumulator block (as above),
// b(row n, pair of columns) b's float2.
template <class B>
__device__ __forceinline__ void mma_block(float (&d)[2][4], const float (&a)[2][4], int gid, int tig, B b) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
        uint32_t ah[4], al[4], bh[2][2], bl[2][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = a[kk][((i & 1) << 1) | (i >> 1)];
            ah[i] = tf32_rn(v);
            al[i] = tf32_rn(v - __uint_as_float(ah[i]));
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const float2 v = b(8 * nt + gid, 4 * kk + tig);
            bh[nt][0] = tf32_rn(v.x);
            bh[nt][1] = tf32_rn(v.y);
            bl[nt][0] = tf32_rn(v.x - __uint_as_float(bh[nt][0]));
            bl[nt][1] = tf32_rn(v.y - __uint_as_float(bh[nt][1]));
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma8(d[nt], ah, bh[nt]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma8(d[nt], ah, bl[nt]);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma8(d[nt], al, bh[nt]);
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

// 32 fp32 columns of this warp's lanes.
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t (&a)[16], uint32_t (&b)[16]) {
    tc::tmem_ld16_nowait(addr, a);
    tc::tmem_ld16_nowait(addr + 16, b);
    tc::tmem_wait_ld16(a);
    tc::tmem_tie16(b);
}

// The 16 x 16 products of rows 16 i .. of tile x with rows 16 j .. of tile k (K
// or Q of a stage), summed over the S columns.
template <int S>
__device__ __forceinline__ void score_block(uint32_t x, uint32_t k, int i, int j, int lane, float (&acc)[2][4]) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
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
            mma16(acc[0], a[ks], b[ks][0], b[ks][1]);
            mma16(acc[1], a[ks], b[ks][2], b[ks][3]);
        }
    }
}

// 1 / sqrt(x + eps) of a block's diagonal, handed to put(row, value).
template <class Put>
__device__ __forceinline__ void diag_norm(const float (&acc)[2][4], int lane, float eps, Put put) {
    const int gid = lane >> 2, tig = lane & 3;
    if (gid >> 1 != tig) return;  // rows gid, gid + 8 meet their columns 2 tig, 2 tig + 1 here
    put(gid, __frsqrt_rn((gid & 1 ? acc[0][1] : acc[0][0]) + eps));
    put(gid + 8, __frsqrt_rn((gid & 1 ? acc[1][3] : acc[1][2]) + eps));
}

template <int S, int H, int NV>
__global__ void __launch_bounds__(threads_of(NV), 1)
k_gdr_chunk_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_y,
               const GdrTcParams p) {
    constexpr int kNWarps = 4 * NV, kPWarp0 = kNWarp0 + kNWarps, kTmaWarp = kPWarp0 + kPWarps, kMmaWarp = kTmaWarp + 1;
    constexpr int kBoxes = S / 64, kVBoxes = NV * H / 64;
    // A stage: K's and Q's boxes in turn, so that 64 rows of K and 64 of Q are one operand of 128; then V's
    constexpr uint32_t kOffV = 2 * kBoxes * kBox, kStage = kOffV + kVBoxes * kBox;
    static_assert((S == 64 || S == 128) && (NV == 1 ? (H == 64 || H == 128) : H == 64), "shapes");
    // Tensor memory columns (128 lanes = the head's columns; NV = 2: 64 of each head)
    constexpr uint32_t cH = 0, cHi = S, cLo = S + S / 2, cR = 2 * S, cO = 2 * S + 64, cX = 2 * S + 128,
                       cW2 = 2 * S + 192;
    // cR: R, then W.  cO: Q h, then y's sum.  cX: X's parts (96 columns), then W's parts for y (64).  cU: the second head's X
    // parts, then W's parts for the state (96 each), over h's parts, which are done with by then (S = 64:
    // behind the rest).  cW2: the second head's W parts for y.  An operand of one of two heads has zeros in
    // the other one's rows.
    constexpr uint32_t cU = S == 128 ? cHi : 2 * S + 256;

    // (aligned by an offset, so that the compiler still knows it for shared memory)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-tc::smem_u32(smem_raw) & 1023u);
    const Geom& g = p.g;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int h0 = NV * blockIdx.x;
    const int64_t b = blockIdx.y;
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

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            tc::mbar_init(&bars[kBarFull + i], 1);
            tc::mbar_init(&bars[kBarFree + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars[kBarSFull + i], kNWarps);
            tc::mbar_init(&bars[kBarSFree + i], 1 + kOutWarps + kPWarps);
        }
        tc::mbar_init(&bars[kBarNFull], kNWarps);
        tc::mbar_init(&bars[kBarPFull], kPWarps);
        tc::mbar_init(&bars[kBarPFree], 1);
        tc::mbar_init(&bars[kBarHReady], kChainWarps);
        tc::mbar_init(&bars[kBarRDone], 1);
        tc::mbar_init(&bars[kBarXReady], kChainWarps);
        tc::mbar_init(&bars[kBarWDone], 1);
        tc::mbar_init(&bars[kBarWReady], kChainWarps);
        tc::mbar_init(&bars[kBarWyReady], kChainWarps);
        tc::mbar_init(&bars[kBarHDone], 1);
        tc::mbar_init(&bars[kBarO1Read], kOutWarps);
        tc::mbar_init(&bars[kBarO2Done], 1);
        tc::mbar_init(&bars[kBarO2Read], kOutWarps);
        tc::mbar_init(&bars[kBarDrain], 1);
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
        more_registers<NV == 2 ? 80 : 88>();
        // ============================== chain ==============================
        const int q = warp & 3, hf = warp >> 2;
        const int hv = NV == 2 ? q >> 1 : 0;
        const int colh = 32 * (NV == 2 ? (q & 1) : q) + lane;  // column of its head
        const bool live = colh < H;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const int64_t sbase = (b * g.nheads + h0 + hv) * (int64_t)S * H + colh;
        // this thread's column of V in a stage: 16-byte piece and place in it
        const uint32_t vch = (32 * (q & 1) + lane) >> 3, vin = (lane & 7) * 2;
        const uint32_t v_off = kOffV + (q >> 1) * kBox + vin;
        {
#pragma unroll 1
            for (int s = hf * (S / 2); s < (hf + 1) * (S / 2); s += 16) {
                uint32_t r[16];
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    r[j] = (live && p.init) ? __float_as_uint(p.init[sbase + (int64_t)(s + j) * H]) : 0u;
                tc::tmem_st16(tl + cH + s, r);
            }
            if (NV == 2) {  // the rows of the other head's operands: zeros, never written again
                uint32_t z[16] = {};
                tc::tmem_st16(tl + (hv ? cX : cW2) + 32 * hf, z);
                tc::tmem_st16(tl + (hv ? cX : cW2) + 32 * hf + 16, z);
            }
            tc::tmem_wait_st();
        }
        int st = 0;
        uint32_t full_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c & 1;
            const uint32_t ph = c & 1;
            if (!warp_wait(&bars[kBarSFull + buf], (c >> 1) & 1, abort_flag)) { ok = false; break; }
            const Scalars* sc = scal_of(buf, hv);
            const float g_last = sc->g_last;
            if (c > 0 && !warp_wait(&bars[kBarHDone], ph ^ 1, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            // h's parts
#pragma unroll 1
            for (int s = hf * (S / 2); s < (hf + 1) * (S / 2); s += 32) {
                uint32_t r[2][16], hi[16], lo[16];
                ld32(tl + cH + s, r[0], r[1]);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    split2(as_f2(&r[j >> 3][(2 * j) & 15]), hi[j], lo[j]);
                }
                tc::tmem_st16(tl + cHi + s / 2, hi);
                tc::tmem_st16(tl + cLo + s / 2, lo);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarHReady]);
            // while R = K h runs: h decayed to the chunk's end, and V from the stage (it has landed: the
            // scores waited for the same copy)
#pragma unroll 1
            for (int s = hf * (S / 2); s < (hf + 1) * (S / 2); s += 32) {
                uint32_t r[2][16];
                ld32(tl + cH + s, r[0], r[1]);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint32_t* x = &r[j >> 3][(2 * j) & 15];
                    const float2 v = tc::mul_f32x2(as_f2(x), make_float2(g_last, g_last));
                    x[0] = __float_as_uint(v.x);
                    x[1] = __float_as_uint(v.y);
                }
                tc::tmem_st16(tl + cH + s, r[0]);
                tc::tmem_st16(tl + cH + s + 16, r[1]);
            }
            if (!warp_wait(&bars[kBarFull + st], full_phase, abort_flag)) { ok = false; break; }
            const int i0 = 32 * hf;  // this warp's tokens: i0 .. i0 + 31
            uint32_t v2[16];         // their V, two to a register
            {
                const int64_t left = n - (int64_t)c * kT;
                const int nv = left < kT ? (int)left : kT;
                const uint8_t* sv = smem + st * kStage + v_off;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int k = i0 + 2 * j;
                    const uint32_t a0 = *reinterpret_cast<const uint16_t*>(sv + k * 128 + ((vch ^ (2 * j & 7)) << 4));
                    const uint32_t a1 =
                        *reinterpret_cast<const uint16_t*>(sv + k * 128 + 128 + ((vch ^ ((2 * j + 1) & 7)) << 4));
                    v2[j] = a0 | (a1 << 16);
                }
                if (nv < kT || !live) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int k = i0 + 2 * j;
                        v2[j] = !live || k >= nv ? 0u : (k + 1 >= nv ? v2[j] & 0xffffu : v2[j]);
                    }
                }
            }
            if (!warp_wait(&bars[kBarRDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            // X
            {
                const uint32_t mine = hv ? cU : cX;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int i1 = i0 + 16 * m;
                    uint32_t r[16], x0[8], x1[8], x2[8];
                    tc::tmem_ld16(tl + cR + i1, r);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 cb = *reinterpret_cast<const float4*>(&sc->cb[i1 + j]);
                        const float4 cr = *reinterpret_cast<const float4*>(&sc->cr[i1 + j]);
                        const uint32_t va = v2[8 * m + j / 2], vb = v2[8 * m + j / 2 + 1];
                        const float2 bv0 = tc::mul_f32x2(make_float2(cb.x, cb.y),
                                                         make_float2(tc::bf16_lo(va), tc::bf16_hi(va)));
                        const float2 bv1 = tc::mul_f32x2(make_float2(cb.z, cb.w),
                                                         make_float2(tc::bf16_lo(vb), tc::bf16_hi(vb)));
                        split3(tc::fma_f32x2(make_float2(cr.x, cr.y), as_f2(&r[j]), bv0), x0[j / 2], x1[j / 2],
                               x2[j / 2]);
                        split3(tc::fma_f32x2(make_float2(cr.z, cr.w), as_f2(&r[j + 2]), bv1), x0[j / 2 + 1],
                               x1[j / 2 + 1], x2[j / 2 + 1]);
                    }
                    tc::tmem_st8(tl + mine + i1 / 2, x0);
                    tc::tmem_st8(tl + mine + 32 + i1 / 2, x1);
                    tc::tmem_st8(tl + mine + 64 + i1 / 2, x2);
                }
                if (NV == 2) {  // zeros in the other head's X: all of it, or the columns that held W
                    uint32_t z[16] = {};
                    if (hv == 0) {
                        tc::tmem_st16(tl + cU + i0 / 2, z);
                        tc::tmem_st16(tl + cU + 32 + i0 / 2, z);
                        tc::tmem_st16(tl + cU + 64 + i0 / 2, z);
                    } else {
                        tc::tmem_st16(tl + cX + 64 + i0 / 2, z);
                    }
                }
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarXReady]);

            // W = N X, decayed to the chunk's end for the state, then as it is for y
            if (!warp_wait(&bars[kBarWDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            uint32_t r[2][16];
            ld32(tl + cR + i0, r[0], r[1]);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                uint32_t u0[8], u1[8], u2[8];
                const int i1 = i0 + 16 * m;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 d = *reinterpret_cast<const float4*>(&sc->d[i1 + j]);
                    const uint32_t* x = &r[m][j];
                    split3(tc::mul_f32x2(make_float2(d.x, d.y), as_f2(x)), u0[j / 2], u1[j / 2], u2[j / 2]);
                    split3(tc::mul_f32x2(make_float2(d.z, d.w), as_f2(x + 2)), u0[j / 2 + 1], u1[j / 2 + 1],
                           u2[j / 2 + 1]);
                }
                tc::tmem_st8(tl + cU + i1 / 2, u0);
                tc::tmem_st8(tl + cU + 32 + i1 / 2, u1);
                tc::tmem_st8(tl + cU + 64 + i1 / 2, u2);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarWReady]);
            {
                const uint32_t mine = hv ? cW2 : cX;
                uint32_t w0[16], w1[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    split2(as_f2(&r[j >> 3][(2 * j) & 15]), w0[j], w1[j]);
                }
                tc::tmem_st16(tl + mine + i0 / 2, w0);
                tc::tmem_st16(tl + mine + 32 + i0 / 2, w1);
                if (NV == 2 && hv == 0) {  // the second head's W: the columns that held X
                    uint32_t z[16] = {};
                    tc::tmem_st16(tl + cW2 + i0 / 2, z);
                }
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarWyReady]);
            if (++st == p.nst) {
                st = 0;
                full_phase ^= 1u;
            }
        }
        if (ok && nc > 0) ok = warp_wait(&bars[kBarHDone], (nc - 1) & 1, abort_flag);
        if (ok && p.final_state) {
            tc::tc_fence_after();
#pragma unroll 1
            for (int s = hf * (S / 2); s < (hf + 1) * (S / 2); s += 16) {
                uint32_t r[16];
                tc::tmem_ld16(tl + cH + s, r);
                if (live) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) p.final_state[sbase + (int64_t)(s + j) * H] = __uint_as_float(r[j]);
                }
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else if (warp < kOutWarp0 + kOutWarps) {
        fewer_registers<NV == 2 ? 64 : 72>();
        // ============================== output ==============================
        const int q = warp & 3;
        const int hv = NV == 2 ? q >> 1 : 0;
        const int colh = 32 * (NV == 2 ? (q & 1) : q) + lane;
        const bool live = colh < H;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const bool storer = threadIdx.x == kOutWarp0 * 32;
        // this thread's column of the staged y
        const uint32_t ych = (32 * (q & 1) + lane) >> 3;
        uint8_t* sy = smem + p.off_y + (q >> 1) * kBox + (lane & 7) * 2;
        for (int c = 0; c < nc; ++c) {
            const int buf = c & 1;
            const uint32_t ph = c & 1;
            const Scalars* sc = scal_of(buf, hv);
            // Q h -> e^G Q h, onto which P W is summed
            ok = warp_wait(&bars[kBarRDone], ph, abort_flag);
            if (ok) {
                tc::tc_fence_after();
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t r[16];
                    tc::tmem_ld16(tl + cO + 16 * m, r);
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&sc->gam[16 * m + j]);
                        const float2 a0 = tc::mul_f32x2(make_float2(f.x, f.y), as_f2(&r[j]));
                        const float2 a1 = tc::mul_f32x2(make_float2(f.z, f.w), as_f2(&r[j + 2]));
                        r[j] = __float_as_uint(a0.x), r[j + 1] = __float_as_uint(a0.y);
                        r[j + 2] = __float_as_uint(a1.x), r[j + 3] = __float_as_uint(a1.y);
                    }
                    tc::tmem_st16(tl + cO + 16 * m, r);
                }
                tc::tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bars[kBarO1Read]);
                ok = warp_wait(&bars[kBarPFull], ph, abort_flag) && warp_wait(&bars[kBarO2Done], ph, abort_flag);
            }
            if (storer) tc::bulk_wait_read_all();  // the last chunk's y has left its place
            ok = bar_sync_and(3, 32 * kOutWarps, ok);
            if (!ok) break;
            tc::tc_fence_after();
            const int64_t left = n - (int64_t)c * kT;
            const int nv = left < kT ? (int)left : kT;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t r[16];
                tc::tmem_ld16(tl + cO + 16 * m, r);
                if (m == 3) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars[kBarO2Read]);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const int i = 16 * m + j;
                    const float4 f = *reinterpret_cast<const float4*>(&sc->oq[i]);
                    const float2 a0 = tc::mul_f32x2(make_float2(f.x, f.y), as_f2(&r[j]));
                    const float2 a1 = tc::mul_f32x2(make_float2(f.z, f.w), as_f2(&r[j + 2]));
                    uint32_t y2[2] = {tc::pack_bf16x2(a0.x, a0.y), tc::pack_bf16x2(a1.x, a1.y)};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t v = e & 1 ? y2[e >> 1] >> 16 : y2[e >> 1] & 0xffffu;
                        if (live)
                            *reinterpret_cast<uint16_t*>(sy + (i + e) * 128 + ((ych ^ ((i + e) & 7)) << 4)) =
                                (uint16_t)(nv == kT || i + e < nv ? v : 0u);
                    }
                }
            }
            tc::fence_proxy_async_smem();
            bar_sync(3, 32 * kOutWarps);
            if (storer) {  // rows past L are clipped
#pragma unroll
                for (int x = 0; x < kVBoxes; ++x)
                    tc::tma_store_4d(&tm_y, smem + p.off_y + x * kBox, NV == 2 ? 0 : 64 * x, NV == 2 ? h0 + x : h0,
                                     c * kT, (int)b);
                tc::bulk_commit();
            }
            if (lane == 0) tc::mbar_arrive(&bars[kBarSFree + buf]);
        }
        if (storer) tc::bulk_wait_all();
        if (!ok) set_abort(ctl, p.status);
        if (ok && live) {
            __nv_bfloat16* y = p.y + (b * L * g.nheads + h0 + hv) * (int64_t)H + colh;
            for (int64_t t = (int64_t)nc * kT; t < L; ++t) y[t * g.nheads * H] = __float2bfloat16_rn(0.f);
        }
    } else if (warp < kPWarp0) {
        more_registers<NV == 2 ? 88 : 120>();
        // ======================= G, k's norms, A and N =======================
        const int hv = (warp - kNWarp0) >> 2, w = (warp - kNWarp0) & 3;
        const int tid = w * 32 + lane;
        const int gid = lane >> 2, tig = lane & 3;
        NScratch* scr = reinterpret_cast<NScratch*>(smem + p.off_scratch) + hv;
        const int64_t gbase = b * L * g.nheads + h0 + hv;
        // warp 0's lanes hold the next chunk's g and beta of tokens 2 lane, 2 lane + 1
        float gn[2], bn[2];
        auto fetch = [&](int c) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t t = (int64_t)c * kT + 2 * lane + r;
                gn[r] = t < n ? p.gate[gbase + t * g.nheads] : 0.f;
                bn[r] = t < n ? p.beta[gbase + t * g.nheads] : 0.f;
            }
        };
        if (w == 0 && nc > 0) fetch(0);
        int st = 0;
        uint32_t full_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c & 1;
            Scalars* sc = scal_of(buf, hv);
            // every warp of the head comes to the barrier below, whatever its waits said
            if (c >= 2) ok = warp_wait(&bars[kBarSFree + buf], ((c >> 1) - 1) & 1, abort_flag);
            if (w == 0 && ok) {
                // log2 decays as an integer and a fraction in units of 2^-24, summed apart
                int gi[2], gf[2];
                float be[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    constexpr float kL = 1.44269502162933349609375f, kLrest = 1.925963033500011e-8f;  // log2 e
                    const float lim = fminf(fmaxf(gn[r], -112.f), 112.f);  // |log2 decay| < 162
                    const float x = lim * kL, rest = fmaf(lim, kL, -x) + lim * kLrest, whole = floorf(x);
                    gi[r] = (int)whole;
                    gf[r] = __float2int_rn(((x - whole) + rest) * 16777216.f);
                    be[r] = gn[r] != gn[r] ? gn[r] : bn[r];  // a NaN decay shows in the token's correction
                }
                int si = gi[0] + gi[1], sf = gf[0] + gf[1];
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const int oi = __shfl_up_sync(0xffffffffu, si, m), of = __shfl_up_sync(0xffffffffu, sf, m);
                    if (lane >= m) si += oi, sf += of;
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int ti = r ? si : si - gi[1], tf = r ? sf : sf - gf[1];
                    sc->tok[2 * lane + r].gi = (float)(ti + (tf >> 24));
                    sc->tok[2 * lane + r].gf = (float)(tf & 0xffffff) * 5.9604644775390625e-8f;
                    sc->tok[2 * lane + r].beta = be[r];
                }
                if (c + 1 < nc) fetch(c + 1);
            }
            if (ok) ok = warp_wait(&bars[kBarFull + st], full_phase, abort_flag);
            uint8_t* sK = smem + st * kStage;
            const uint32_t aK = tc::smem_u32(sK);
            const int64_t left = n - (int64_t)c * kT;
            const int nv = left < kT ? (int)left : kT;
            // the diagonal block of K K^T, whose diagonal gives the norms: summed by the same
            // instructions as the rest, so that rk_i rk_j (k_i . k_j) is 1 to rounding where keys agree
            float acc[2][4];
            if (ok) {
                if (nv < kT) {
                    // past the row's end: K enters the state's product and has to be 0
                    const int r = 16 * w + (lane >> 1);
                    if (r >= nv) {
#pragma unroll
                        for (int i = 0; i < S / 16; ++i)
                            *reinterpret_cast<uint4*>(sK + (S == 128 ? (lane & 1) * 2 * kBox + sw(r, i)
                                                                     : sw(r, 4 * (lane & 1) + i))) =
                                make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                score_block<S>(aK, aK, w, w, lane, acc);
                if (p.l2norm)
                    diag_norm(acc, lane, p.l2_eps, [&](int i, float f) { sc->tok[16 * w + i].rk = f; });
                else if (lane < 16)
                    sc->tok[16 * w + lane].rk = 1.f;
            }
            ok = bar_sync_and(1 + hv, 128, ok);
            if (!ok) break;
            if (tid < kT) {
                const Tok t = sc->tok[tid], last = sc->tok[kT - 1];
                const float e = ex2(t.gi) * ex2(t.gf);
                sc->cb[tid] = t.beta;
                sc->cr[tid] = -t.beta * e * t.rk;
                sc->gam[tid] = e;
                sc->d[tid] = ex2(last.gi - t.gi) * ex2(last.gf - t.gf) * t.rk;
                const float el = decay(t, sc->tok[tid & ~15]);
                sc->el[tid] = el;
                sc->ea[tid] = t.beta * t.rk * el;
                if (tid == kT - 1) sc->g_last = e;
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarSFull + buf]);
            // A's diagonal block, by columns
            {
                const Tok ti0 = sc->tok[16 * w + gid], ti1 = sc->tok[16 * w + gid + 8];
                const float f0 = ti0.beta * ti0.rk, f1 = ti1.beta * ti1.rk;
                const bool in0 = 16 * w + gid < nv, in1 = 16 * w + gid + 8 < nv;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int jj = 8 * nt + 2 * tig + e;
                        const Tok tj = sc->tok[16 * w + jj];
                        scr->diag[w][jj][gid] = in0 && jj < gid ? acc[nt][e] * (f0 * tj.rk * decay(ti0, tj)) : 0.f;
                        scr->diag[w][jj][gid + 8] =
                            in1 && jj < gid + 8 ? acc[nt][2 + e] * (f1 * tj.rk * decay(ti1, tj)) : 0.f;
                    }
            }
            // and one or two below
#pragma unroll 1
            for (int t = w + 4; t < 10; t += 4) {
                const int i = tri_i(t), j = tri_j(t);
                score_block<S>(aK, aK, i, j, lane, acc);
                // (rows past the end: 0, whatever their products are)
                const float f0 = 16 * i + gid < nv ? sc->ea[16 * i + gid] : 0.f;
                const float f1 = 16 * i + gid + 8 < nv ? sc->ea[16 * i + gid + 8] : 0.f;
                const Tok tr = sc->tok[16 * i];
                float2 (*low)[8] = scr->low[low_block(i, j)];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int jj = 8 * nt + 2 * tig;
                    const Tok t0 = sc->tok[16 * j + jj], t1 = sc->tok[16 * j + jj + 1];
                    const float2 cj = make_float2(t0.rk * decay(tr, t0), t1.rk * decay(tr, t1));
                    const float2 c0 = tc::mul_f32x2(cj, make_float2(f0, f0)), c1 = tc::mul_f32x2(cj, make_float2(f1, f1));
                    low[gid][low_at(gid, jj / 2)] = tc::mul_f32x2(c0, make_float2(acc[nt][0], acc[nt][1]));
                    low[gid + 8][low_at(gid + 8, jj / 2)] = tc::mul_f32x2(c1, make_float2(acc[nt][2], acc[nt][3]));
                }
            }
            __syncwarp();
            // the diagonal block of N, a column per lane (both halves of the warp the same)
            {
                const int l = lane & 15;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = i == l ? 1.f : 0.f;
#pragma unroll
                for (int m = 0; m < 15; ++m) {
#pragma unroll
                    for (int i4 = (m + 1) / 4; i4 < 4; ++i4) {
                        const float4 a = *reinterpret_cast<const float4*>(&scr->diag[w][m][4 * i4]);
                        if (4 * i4 > m) x[4 * i4] = fmaf(-a.x, x[m], x[4 * i4]);
                        if (4 * i4 + 1 > m) x[4 * i4 + 1] = fmaf(-a.y, x[m], x[4 * i4 + 1]);
                        if (4 * i4 + 2 > m) x[4 * i4 + 2] = fmaf(-a.z, x[m], x[4 * i4 + 2]);
                        if (4 * i4 + 3 > m) x[4 * i4 + 3] = fmaf(-a.w, x[m], x[4 * i4 + 3]);
                    }
                }
                __syncwarp();
                if (lane < 16) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) scr->diag[w][i][l] = x[i];
                }
            }
            bar_sync(1 + hv, 128);
            // N's block column w, transposed: N_ij^T = -(sum_m N_mj^T A_im^T) N_ii^T, as accumulator
            // fragments nf[d] (i = w + d), which are also left operands
            {
                float nf[4][2][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int r = 8 * nt + 2 * tig;
                    nf[0][nt][0] = scr->diag[w][r][gid];
                    nf[0][nt][1] = scr->diag[w][r + 1][gid];
                    nf[0][nt][2] = scr->diag[w][r][gid + 8];
                    nf[0][nt][3] = scr->diag[w][r + 1][gid + 8];
                }
#pragma unroll
                for (int d = 1; d < 4; ++d) {
                    if (w + d > 3) break;
                    const int i = w + d;
                    float x[2][4] = {};
#pragma unroll
                    for (int m = 0; m < d; ++m) {
                        const float2 (*low)[8] = scr->low[low_block(i, w + m)];
                        mma_block(x, nf[m], gid, tig, [&](int r, int c2) { return low[r][low_at(r, c2)]; });
                    }
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[nt][e] = -x[nt][e], nf[d][nt][e] = 0.f;
                    mma_block(nf[d], x, gid, tig, [&](int r, int c2) {
                        return *reinterpret_cast<const float2*>(&scr->diag[i][r][2 * c2]);
                    });
                }
                // the last chunk's N has been used
                if (c > 0) ok = warp_wait(&bars[kBarWDone], (c - 1) & 1, abort_flag);
                const uint32_t tr = (lane & 7) + ((lane >> 4) << 3), tch = (lane >> 3) & 1;
                const uint32_t aN = tc::smem_u32(n_of(hv));
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    if (w + d > 3 || !ok) break;
                    const uint32_t at = aN + sw(16 * (w + d) + tr, 2 * w + tch);
#pragma unroll
                    for (int pl = 0; pl < (int)kNPlanes; ++pl) {
                        uint32_t r[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float* v = &nf[d][x >> 1][2 * (x & 1)];
                            float2 f = make_float2(v[0], v[1]);
                            r[x] = high(f);
                            v[0] = f.x;
                            v[1] = f.y;
                        }
                        stsm4_trans(at + pl * kPlane, r);
                    }
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(&bars[kBarNFull]);
            if (++st == p.nst) {
                st = 0;
                full_phase ^= 1u;
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else if (warp < kPWarp0 + kPWarps) {
        fewer_registers<NV == 2 ? 56 : 64>();
        // ========================= q's norms and P =========================
        const int w = warp - kPWarp0;
        const int gid = lane >> 2, tig = lane & 3;
        int st = 0;
        uint32_t full_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c & 1;
            ok = warp_wait(&bars[kBarFull + st], full_phase, abort_flag) &&
                 warp_wait(&bars[kBarSFull + buf], (c >> 1) & 1, abort_flag);
            const uint32_t aK = tc::smem_u32(smem + st * kStage), aQ = aK + kBox;
            float acc[2][4];
            if (ok && p.l2norm) {
                // 1 / norm into oq's place
                score_block<S>(aQ, aQ, w, w, lane, acc);
                diag_norm(acc, lane, p.l2_eps, [&](int i, float f) { scal_of(buf, 0)->oq[16 * w + i] = f; });
                __syncwarp();
            }
            if (ok && lane < 16) {  // a row per lane
                const int i = 16 * w + lane;
                const float oq = p.l2norm ? p.scale * scal_of(buf, 0)->oq[i] : p.scale;
#pragma unroll
                for (int hv = 0; hv < NV; ++hv) scal_of(buf, hv)->oq[i] = oq;
            }
#pragma unroll 1
            for (int t = w; t < 10; t += 4) {
                const int i = tri_i(t), j = tri_j(t), i0 = 16 * i + gid;
                if (ok) score_block<S>(aQ, aK, i, j, lane, acc);
                // the last chunk's P has been used
                if (ok && t < 4 && c > 0) ok = warp_wait(&bars[kBarPFree], (c - 1) & 1, abort_flag);
                if (!ok) break;
#pragma unroll
                for (int hv = 0; hv < NV; ++hv) {
                    const Scalars* sc = scal_of(buf, hv);
                    uint8_t* sP = p_of(hv);
                    // (the diagonal block takes its decays exactly)
                    const bool below = i > j;
                    const Tok tr = sc->tok[16 * i], ti0 = sc->tok[i0], ti1 = sc->tok[i0 + 8];
                    const float f0 = sc->el[i0], f1 = sc->el[i0 + 8];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int j0 = 16 * j + 8 * nt + 2 * tig;
                        const Tok t0 = sc->tok[j0], t1 = sc->tok[j0 + 1];
                        float2 c0, c1;
                        if (below) {
                            const float2 cj = make_float2(t0.rk * decay(tr, t0), t1.rk * decay(tr, t1));
                            c0 = tc::mul_f32x2(cj, make_float2(f0, f0));
                            c1 = tc::mul_f32x2(cj, make_float2(f1, f1));
                        } else {
                            c0 = make_float2(t0.rk * decay(ti0, t0), t1.rk * decay(ti0, t1));
                            c1 = make_float2(t0.rk * decay(ti1, t0), t1.rk * decay(ti1, t1));
                        }
                        float2 a0 = tc::mul_f32x2(c0, make_float2(acc[nt][0], acc[nt][1]));
                        float2 a1 = tc::mul_f32x2(c1, make_float2(acc[nt][2], acc[nt][3]));
                        if (!below) {
                            a0 = make_float2(j0 <= i0 ? a0.x : 0.f, j0 + 1 <= i0 ? a0.y : 0.f);
                            a1 = make_float2(j0 <= i0 + 8 ? a1.x : 0.f, j0 + 1 <= i0 + 8 ? a1.y : 0.f);
                        }
                        const uint32_t o0 = sw(i0, 2 * j + nt) + 4 * tig;
                        uint32_t hi, lo;
                        split2(a0, hi, lo);
                        *reinterpret_cast<uint32_t*>(sP + o0) = hi;
                        *reinterpret_cast<uint32_t*>(sP + kPlane + o0) = lo;
                        split2(a1, hi, lo);
                        *reinterpret_cast<uint32_t*>(sP + o0 + 1024) = hi;
                        *reinterpret_cast<uint32_t*>(sP + kPlane + o0 + 1024) = lo;
                    }
                }
            }
            if (!ok) break;
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&bars[kBarPFull]);
                tc::mbar_arrive(&bars[kBarSFree + buf]);
            }
            if (++st == p.nst) {
                st = 0;
                full_phase ^= 1u;
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else {
        fewer_registers<48>();
        if (warp == kTmaWarp) {
            // ============================ TMA producer ============================
            if (lane == 0) {
                tc::tma_prefetch_desc(&tm_q);
                tc::tma_prefetch_desc(&tm_k);
                tc::tma_prefetch_desc(&tm_v);
                tc::tma_prefetch_desc(&tm_y);
                int fills[kMaxStages] = {};
                int st = 0;
                uint32_t free_phase = 1;
                for (int c = 0; c < nc; ++c) {
                    if (c >= p.nst && !tc::mbar_wait(&bars[kBarFree + st], free_phase, abort_flag)) { ok = false; break; }
                    uint8_t* s = smem + st * kStage;
                    uint64_t* full = &bars[kBarFull + st];
                    tc::mbar_arrive_expect_tx(full, kStage);
    #pragma unroll
                    for (int x = 0; x < kBoxes; ++x) {
                        tc::tma_load_4d(s + 2 * x * kBox, &tm_k, full, 64 * x, grp, c * kT, (int)b);
                        tc::tma_load_4d(s + (2 * x + 1) * kBox, &tm_q, full, 64 * x, grp, c * kT, (int)b);
                    }
    #pragma unroll
                    for (int x = 0; x < kVBoxes; ++x)
                        tc::tma_load_4d(s + kOffV + x * kBox, &tm_v, full, NV == 2 ? 0 : 64 * x, NV == 2 ? h0 + x : h0,
                                        c * kT, (int)b);
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
        } else if (warp == kMmaWarp) {
            // ============================= MMA issuer =============================
            if (lane == 0 && nc > 0) {
                constexpr uint32_t id_t = tc::idesc_bf16(128, kT, false, false);       // N = tokens
                constexpr uint32_t id_rq = tc::idesc_bf16(128, 2 * kT, false, false);  // of K and of Q
                constexpr uint32_t id_s = tc::idesc_bf16(128, S, false, true);    // N = state rows
                int st = 0;
                uint32_t full_phase = 0;
                for (int c = 0; c < nc; ++c) {
                    const int buf = c & 1;
                    const uint32_t ph = c & 1;
                    const uint32_t aK = tc::smem_u32(smem + st * kStage);
                    const uint64_t dK = tc::sdesc_sw128(aK, 16, 1024);
                    const uint64_t dKt = tc::sdesc_sw128(aK, 2 * kBox, 1024);
                    if (!tc::mbar_wait(&bars[kBarFull + st], full_phase, abort_flag)) { ok = false; break; }
                    if (!tc::mbar_wait(&bars[kBarSFull + buf], (c >> 1) & 1, abort_flag)) { ok = false; break; }
                    if (!tc::mbar_wait(&bars[kBarHReady], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
                    // R | Q h from h's high part, once y's sum of the chunk before has been read; R from its low part
                    if (c > 0 && !tc::mbar_wait(&bars[kBarO2Read], ph ^ 1, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < S / 16; ++ks)
                        tc::mma_bf16_ts(tmem + cR, tmem + cHi + 8 * ks,
                                        dK + (((ks >> 2) * 2 * kBox + (ks & 3) * 32) >> 4), id_rq, ks > 0);
#pragma unroll
                    for (int ks = 0; ks < S / 16; ++ks)
                        tc::mma_bf16_ts(tmem + cR, tmem + cLo + 8 * ks,
                                        dK + (((ks >> 2) * 2 * kBox + (ks & 3) * 32) >> 4), id_t, 1);
                    tc::mma_commit(&bars[kBarRDone]);
                    // W = N X, N's parts times X's down to 2^-16 of hi hi; block column kb of N only has rows from its
                    // own block on
                    if (!tc::mbar_wait(&bars[kBarNFull], ph, abort_flag)) { ok = false; break; }
                    if (!tc::mbar_wait(&bars[kBarXReady], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
    #pragma unroll
                    for (int hv = 0; hv < NV; ++hv) {
                        const uint32_t x = tmem + (hv ? cU : cX);
                        const uint64_t dN = tc::sdesc_sw128(tc::smem_u32(n_of(hv)), 16, 1024);
    #pragma unroll
                        for (int kb = 0; kb < 4; ++kb) {
                            const uint32_t d = tmem + cR + 16 * kb, id = tc::idesc_bf16(128, kT - 16 * kb, false, false);
                            const uint64_t at = dN + (2048 >> 4) * kb + 2 * kb;
                            tc::mma_bf16_ts(d, x + 8 * kb, at, id, hv > 0 || kb > 0);
                            tc::mma_bf16_ts(d, x + 8 * kb, at + (kPlane >> 4), id, 1);
                            tc::mma_bf16_ts(d, x + 8 * kb, at + 2 * (kPlane >> 4), id, 1);
                            tc::mma_bf16_ts(d, x + 32 + 8 * kb, at, id, 1);
                            tc::mma_bf16_ts(d, x + 32 + 8 * kb, at + (kPlane >> 4), id, 1);
                            tc::mma_bf16_ts(d, x + 64 + 8 * kb, at, id, 1);
                        }
                    }
                    tc::mma_commit(&bars[kBarWDone]);
                    // h += K^T W
                    if (!tc::mbar_wait(&bars[kBarWReady], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
    #pragma unroll
                    for (int kt = 0; kt < 4; ++kt) {
                        tc::mma_bf16_ts(tmem + cH, tmem + cU + 8 * kt, dKt + 128 * kt, id_s, 1);
                        tc::mma_bf16_ts(tmem + cH, tmem + cU + 32 + 8 * kt, dKt + 128 * kt, id_s, 1);
                        tc::mma_bf16_ts(tmem + cH, tmem + cU + 64 + 8 * kt, dKt + 128 * kt, id_s, 1);
                    }
                    tc::mma_commit(&bars[kBarHDone]);
                    // P W onto the scaled Q h: hi hi + hi lo + lo hi
                    if (!tc::mbar_wait(&bars[kBarPFull], ph, abort_flag)) { ok = false; break; }
                    if (!tc::mbar_wait(&bars[kBarWyReady], ph, abort_flag)) { ok = false; break; }
                    if (!tc::mbar_wait(&bars[kBarO1Read], ph, abort_flag)) { ok = false; break; }
                    tc::tc_fence_after();
    #pragma unroll
                    for (int hv = 0; hv < NV; ++hv) {
                        const uint32_t wp = tmem + (hv ? cW2 : cX);
                        const uint64_t dP = tc::sdesc_sw128(tc::smem_u32(p_of(hv)), 16, 1024);
    #pragma unroll
                        for (int kb = 0; kb < 4; ++kb) {
                            const uint32_t d = tmem + cO + 16 * kb, id = tc::idesc_bf16(128, kT - 16 * kb, false, false);
                            const uint64_t at = dP + (2048 >> 4) * kb + 2 * kb;
                            tc::mma_bf16_ts(d, wp + 8 * kb, at, id, 1);
                            tc::mma_bf16_ts(d, wp + 8 * kb, at + (kPlane >> 4), id, 1);
                            tc::mma_bf16_ts(d, wp + 32 + 8 * kb, at, id, 1);
                        }
                    }
                    tc::mma_commit(&bars[kBarO2Done]);
                    tc::mma_commit(&bars[kBarSFree + buf]);
                    tc::mma_commit(&bars[kBarPFree]);
                    tc::mma_commit(&bars[kBarFree + st]);
                    if (++st == p.nst) {
                        st = 0;
                        full_phase ^= 1u;
                    }
                }
                if (!ok) set_abort(ctl, p.status);
                // no product may still run when the tensor memory is freed
                tc::mma_commit(&bars[kBarDrain]);
                (void)tc::mbar_wait(&bars[kBarDrain], 0, never);
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

template <int S, int H, int NV>
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
    constexpr uint32_t stage = (2 * (S / 64) + NV * H / 64) * kBox;
    constexpr uint32_t scratch = NV * (uint32_t)sizeof(NScratch);
    constexpr uint32_t rest =
        NV * ((kNPlanes + kPPlanes) * kPlane + H / 64 * kBox + 2 * kScalBytes) + scratch + kNumBars * 8 + (uint32_t)sizeof(SharedCtl) + 1024;
    constexpr int fit = (kSmemLimit - (int)rest) / (int)stage;
    static_assert(fit >= 2, "two stages at least");
    p.nst = fit < kMaxStages ? fit : kMaxStages;
    p.off_n = p.nst * stage;
    p.off_p = p.off_n + NV * kNPlanes * kPlane;
    p.off_y = p.off_p + NV * kPPlanes * kPlane;
    p.off_scal = p.off_y + NV * H / 64 * kBox;
    p.off_scratch = p.off_scal + 2 * NV * kScalBytes;
    p.off_bar = p.off_scratch + scratch;
    const int smem = (int)(p.nst * stage + rest);

    CUtensorMap tm_q, tm_k, tm_v, tm_y;
    const uint64_t L = g.seqlen, B = g.batch;
    const uint32_t box[4] = {64, 1, kT, 1};
    auto map = [&](CUtensorMap* m, const void* base, uint64_t width, uint64_t count, uint64_t stride) {
        const uint64_t dims[4] = {width, count, L, B};
        const uint64_t strides[3] = {width * 2, stride * 2, L * stride * 2};
        return make_tmap_bf16(m, base, 4, dims, strides, box);
    };
    if (!map(&tm_q, a.q, S, g.ngroups, a.q_stride) || !map(&tm_k, a.k, S, g.ngroups, a.k_stride) ||
        !map(&tm_v, a.v, H, g.nheads, a.v_stride) || !map(&tm_y, a.y, H, g.nheads, (uint64_t)(g.nheads * H)))
        return cudaErrorInvalidValue;
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(k_gdr_chunk_tc<S, H, NV>), smem);
    if (e != cudaSuccess) return e;
    k_gdr_chunk_tc<S, H, NV><<<dim3((unsigned)(g.nheads / NV), (unsigned)g.batch), threads_of(NV), smem, st>>>(tm_q, tm_k, tm_v, tm_y, p);
    return cudaGetLastError();
}

}  // namespace

// bf16 shapes the kernel covers; TMA wants every row of q, k and v on a 16-byte
// boundary.
bool gdr_chunk_tc_fits(const GdrArgs& a) {
    const Geom& g = a.g;
    if ((g.dstate != 64 && g.dstate != 128) || (g.headdim != 64 && g.headdim != 128)) return false;
    if (g.seqlen >= ((int64_t)1 << 30) || g.nheads > 65535) return false;
    return aligned16(a.q, a.q_stride) && aligned16(a.k, a.k_stride) && aligned16(a.v, a.v_stride);
}

cudaError_t launch_gdr_chunk_tc(const GdrArgs& a, cudaStream_t st) {
    const bool pairs = a.g.headdim == 64 && a.g.heads_per_group % 2 == 0;
    if (a.g.dstate == 128) {
        if (a.g.headdim == 128) return launch_k<128, 128, 1>(a, st);
        return pairs ? launch_k<128, 64, 2>(a, st) : launch_k<128, 64, 1>(a, st);
    }
    if (a.g.headdim == 128) return launch_k<64, 128, 1>(a, st);
    return pairs ? launch_k<64, 64, 2>(a, st) : launch_k<64, 64, 1>(a, st);
}

}  // namespace m2
