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
//   then 4 NV    scores: G, norms, A, P and N of the next chunk, while the
//                chain runs on this one
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
// G is summed in 32.32 fixed point and kept as an integer and a fraction, so
// that G_i - G_j is good to 2^-23 even behind a token that forgets everything.
// Log2 decays of a token are clamped to +-160, beyond which fp32 has only 0 and
// infinity.
#include "gated_delta.cuh"
#include "tc_ptx.cuh"
#include "tmap_host.cuh"

namespace m2 {
namespace {

constexpr int kT = 64;             // tokens per chunk
constexpr int kChainWarps = 8, kOutWarp0 = 8, kOutWarps = 4, kScoreWarp0 = 12;
constexpr uint32_t kBox = kT * 128;  // one box: 64 tokens x 64 columns of bf16
constexpr int kMaxStages = 3;
constexpr int kSmemLimit = 232448;

struct TokScore {  // what the scores need of a token
    float gi, gf;  // G in log2 units: integer part, fraction
    float rk;      // 1 / norm of k
    float beta;
};
struct TokChain {
    float cb, cr, d, pad;  // X = cb v - cr R;  W's share of the state: d
};
struct Scalars {  // one head's, per chunk
    TokChain chain[kT];
    float2 out[kT];  // y = x Qh + y PW
    float g_last;    // e^{G_last}
    float pad[7];
};

// A head's results of the scores: N's three and P's two planes of 64 rows of
// 128 bytes, in one buffer each (they are needed late in a chunk, and written
// when the chunk before has used them), the scalars in two.
constexpr uint32_t kPlane = kT * 128;
constexpr uint32_t kNPlanes = 3, kPPlanes = 2;
constexpr uint32_t kScalBytes = 3072;
static_assert(sizeof(Scalars) <= kScalBytes, "scalars");

struct ScoreScratch {       // one head's
    float diag[4][16][20];  // A's diagonal blocks, [column][row]; then N's, [row][column]
    float2 low[6][16][8];   // A's blocks below the diagonal, see low_at
    TokScore tok[kT];
    float rq[kT];
};
// Place of columns 2 c2, 2 c2 + 1 of row r in a block of `low` (spread over the
// banks for eight rows by four pairs).
__device__ __forceinline__ int low_at(int r, int c2) { return c2 ^ (((r >> 1) & 1) << 2); }
__device__ __forceinline__ int low_block(int i, int m) { return i * (i - 1) / 2 + m; }

enum : int {
    kBarFull = 0,                        // [stages] TMA
    kBarFree = kBarFull + kMaxStages,    // [stages] every reader of the stage is done
    kBarSFull = kBarFree + kMaxStages,   // [2] scalars (and K's rows past the end cleared)
    kBarSFree = kBarSFull + 2,           // [2]
    kBarNFull = kBarSFree + 2,           // N; free again with kBarWDone
    kBarPFull,
    kBarPFree,
    kBarHReady,  // h's parts are written, h is decayed
    kBarRDone,
    kBarXReady,
    kBarWDone,
    kBarWReady,
    kBarHDone,
    kBarO1Done,  // Q h
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
    uint32_t off_n, off_p, off_scal, off_scratch, off_bar;
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

// A whole warp's wait: all lanes leave with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort));
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
__device__ __forceinline__ void mma_tf32x3(float (&d)[4], const float (&a)[4], float2 b) {
    const float av[4] = {a[0], a[2], a[1], a[3]}, bv[2] = {b.x, b.y};
    uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        ah[i] = tf32_rn(av[i]);
        al[i] = tf32_rn(av[i] - __uint_as_float(ah[i]));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        bh[i] = tf32_rn(bv[i]);
        bl[i] = tf32_rn(bv[i] - __uint_as_float(bh[i]));
    }
    mma8(d, ah, bh);
    mma8(d, ah, bl);
    mma8(d, al, bh);
}

// A pair of fp32 values as its two bf16 parts.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = tc::pack_bf16x2(a, b);
    lo = tc::pack_bf16x2(a - tc::bf16_lo(hi), b - tc::bf16_hi(hi));
}

// And as three.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = tc::pack_bf16x2(a, b);
    split2(a - tc::bf16_lo(hi), b - tc::bf16_hi(hi), mid, lo);
}

// 32 fp32 columns of this warp's lanes.
__device__ __forceinline__ void ld32(uint32_t addr, uint32_t (&a)[16], uint32_t (&b)[16]) {
    tc::tmem_ld16_nowait(addr, a);
    tc::tmem_ld16_nowait(addr + 16, b);
    tc::tmem_wait_ld16(a);
    tc::tmem_tie16(b);
}

// 16 rows (from row0 of tile x) against the rows of blocks jmin .. jmax of tile
// k, summed over the S columns: acc[jb] is the 16 x 16 product with block jb.
template <int S>
__device__ __forceinline__ void score_rows(uint32_t x, uint32_t k, int row0, int jmin, int jmax, int lane,
                                           float (&acc)[4][2][4]) {
#pragma unroll
    for (int jb = 0; jb < 4; ++jb)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[jb][nt][e] = 0.f;
    const uint32_t ar = row0 + (lane & 15), ac = lane >> 4;
    const uint32_t br = (lane & 7) + ((lane >> 4) << 3), bc = (lane >> 3) & 1;
#pragma unroll
    for (int ks = 0; ks < S / 16; ++ks) {
        const uint32_t box = (ks >> 2) * kBox, ch = (ks & 3) * 2;
        uint32_t a[4];
        ldsm4(x + box + sw(ar, ch + ac), a);
#pragma unroll
        for (int jb = 0; jb < 4; ++jb) {
            if (jb > jmax) break;
            if (jb < jmin) continue;
            uint32_t b[4];
            ldsm4(k + box + sw(16 * jb + br, ch + bc), b);
            mma16(acc[jb][0], a, b[0], b[1]);
            mma16(acc[jb][1], a, b[2], b[3]);
        }
    }
}

// 1 / sqrt(x + eps) of the diagonal of block jb, handed to put(row, value).
template <class Put>
__device__ __forceinline__ void diag_norm(const float (&acc)[4][2][4], int jb, int lane, float eps, Put put) {
    const int gid = lane >> 2, tig = lane & 3;
    if (gid >> 1 != tig) return;  // rows gid, gid + 8 meet their columns 2 tig, 2 tig + 1 here
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        if (b == jb) {
            d0 = gid & 1 ? acc[b][0][1] : acc[b][0][0];
            d1 = gid & 1 ? acc[b][1][3] : acc[b][1][2];
        }
    put(gid, __frsqrt_rn(d0 + eps));
    put(gid + 8, __frsqrt_rn(d1 + eps));
}

template <int S, int H, int NV>
__global__ void __launch_bounds__((kScoreWarp0 + 4 * NV + 2) * 32, 1)
k_gdr_chunk_tc(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
               const __grid_constant__ CUtensorMap tm_v, const GdrTcParams p) {
    constexpr int kScoreWarps = 4 * NV, kTmaWarp = kScoreWarp0 + kScoreWarps, kMmaWarp = kTmaWarp + 1;
    constexpr int kBoxes = S / 64, kVBoxes = NV * H / 64;
    constexpr uint32_t kOffQ = kBoxes * kBox, kOffV = 2 * kOffQ, kStage = kOffV + kVBoxes * kBox;
    static_assert((S == 64 || S == 128) && (NV == 1 ? (H == 64 || H == 128) : H == 64), "shapes");
    // Tensor memory columns (128 lanes = the head's columns; NV = 2: 64 of each head)
    constexpr uint32_t cH = 0, cHi = S, cLo = S + S / 2, cR = 2 * S, cX = 2 * S + 64, cW2 = 2 * S + 128,
                       cO = 2 * S + 192;
    // R holds R, then W.  cX: X's parts (96 columns), then W's parts for y (64).  cU: the second head's X
    // parts, then W's parts for the state (96 each), over h's parts, which are done with by then (S = 64:
    // behind the rest).  cW2: the second head's W parts for y.  An operand of one of two heads has zeros in
    // the other one's rows.
    constexpr uint32_t cU = S == 128 ? cHi : 2 * S + 256;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
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
            tc::mbar_init(&bars[kBarSFull + i], kScoreWarps);
            tc::mbar_init(&bars[kBarSFree + i], 1 + kOutWarps);
        }
        tc::mbar_init(&bars[kBarNFull], kScoreWarps);
        tc::mbar_init(&bars[kBarPFull], kScoreWarps);
        tc::mbar_init(&bars[kBarPFree], 1);
        tc::mbar_init(&bars[kBarHReady], kChainWarps);
        tc::mbar_init(&bars[kBarRDone], 1);
        tc::mbar_init(&bars[kBarXReady], kChainWarps);
        tc::mbar_init(&bars[kBarWDone], 1);
        tc::mbar_init(&bars[kBarWReady], kChainWarps);
        tc::mbar_init(&bars[kBarHDone], 1);
        tc::mbar_init(&bars[kBarO1Done], 1);
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
            // h: its parts, and itself decayed to the chunk's end
#pragma unroll 1
            for (int s = hf * (S / 2); s < (hf + 1) * (S / 2); s += 32) {
                uint32_t r[2][16], hi[16], lo[16];
                ld32(tl + cH + s, r[0], r[1]);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint32_t* x = &r[j >> 3][(2 * j) & 15];
                    const float a0 = __uint_as_float(x[0]), a1 = __uint_as_float(x[1]);
                    split2(a0, a1, hi[j], lo[j]);
                    x[0] = __float_as_uint(g_last * a0);
                    x[1] = __float_as_uint(g_last * a1);
                }
                tc::tmem_st16(tl + cHi + s / 2, hi);
                tc::tmem_st16(tl + cLo + s / 2, lo);
                tc::tmem_st16(tl + cH + s, r[0]);
                tc::tmem_st16(tl + cH + s + 16, r[1]);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarHReady]);

            // R = K h -> X (the stage's V has landed: the scores waited for the same copy)
            if (!warp_wait(&bars[kBarFull + st], full_phase, abort_flag)) { ok = false; break; }
            if (!warp_wait(&bars[kBarRDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            const int i0 = 32 * hf;  // this warp's tokens: i0 .. i0 + 31
            const int64_t left = n - (int64_t)c * kT;
            const int nv = left < kT ? (int)left : kT;
            const uint8_t* sv = smem + st * kStage + v_off;
            // (Q h, which follows R, also reads what X may overwrite)
            if (NV == 2 && S == 128 && !warp_wait(&bars[kBarO1Done], ph, abort_flag)) { ok = false; break; }
            {
                const uint32_t mine = hv ? cU : cX;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int i1 = i0 + 16 * m;
                    uint32_t r[16], x0[8], x1[8], x2[8];
                    tc::tmem_ld16(tl + cR + i1, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float x[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int k = 2 * j + e;
                            const float4 t = *reinterpret_cast<const float4*>(&sc->chain[i1 + k]);
                            float v = __bfloat162float(
                                *reinterpret_cast<const __nv_bfloat16*>(sv + (i1 + k) * 128 + ((vch ^ (k & 7)) << 4)));
                            v = (live && i1 + k < nv) ? v : 0.f;
                            x[e] = fmaf(-t.y, __uint_as_float(r[k]), t.x * v);
                        }
                        split3(x[0], x[1], x0[j], x1[j], x2[j]);
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

            // W = N X: its parts for y, and decayed to the chunk's end for the state
            if (!warp_wait(&bars[kBarWDone], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            {
                const uint32_t mine = hv ? cW2 : cX;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t r[16], w0[8], w1[8], u0[8], u1[8], u2[8];
                    const int i1 = i0 + 16 * m;
                    tc::tmem_ld16(tl + cR + i1, r);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float a0 = __uint_as_float(r[2 * j]), a1 = __uint_as_float(r[2 * j + 1]);
                        split2(a0, a1, w0[j], w1[j]);
                        split3(sc->chain[i1 + 2 * j].d * a0, sc->chain[i1 + 2 * j + 1].d * a1, u0[j], u1[j], u2[j]);
                    }
                    tc::tmem_st8(tl + cU + i1 / 2, u0);
                    tc::tmem_st8(tl + cU + 32 + i1 / 2, u1);
                    tc::tmem_st8(tl + cU + 64 + i1 / 2, u2);
                    tc::tmem_st8(tl + mine + i1 / 2, w0);
                    tc::tmem_st8(tl + mine + 32 + i1 / 2, w1);
                }
                if (NV == 2 && hv == 0) {  // the second head's W: the columns that held X
                    uint32_t z[16] = {};
                    tc::tmem_st16(tl + cW2 + i0 / 2, z);
                }
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarWReady]);
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
        // ============================== output ==============================
        const int q = warp & 3;
        const int hv = NV == 2 ? q >> 1 : 0;
        const int colh = 32 * (NV == 2 ? (q & 1) : q) + lane;
        const bool live = colh < H;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const int64_t row = (int64_t)g.nheads * H;
        const int odd = lane & 1;
        // lanes meet in pairs: the even one stores both columns of token i, the odd one of i + 1
        __nv_bfloat16* y = p.y + (b * L + odd) * row + (int64_t)(h0 + hv) * H + (colh & ~1);
        for (int c = 0; c < nc; ++c) {
            const int buf = c & 1;
            const uint32_t ph = c & 1;
            const Scalars* sc = scal_of(buf, hv);
            if (!warp_wait(&bars[kBarSFull + buf], (c >> 1) & 1, abort_flag)) { ok = false; break; }
            if (!warp_wait(&bars[kBarO1Done], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            uint32_t o1[4][16];
#pragma unroll
            for (int m = 0; m < 4; ++m) tc::tmem_ld16_nowait(tl + cO + 16 * m, o1[m]);
            tc::tmem_wait_ld16(o1[0]);
            tc::tmem_tie16(o1[1]);
            tc::tmem_tie16(o1[2]);
            tc::tmem_tie16(o1[3]);
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarO1Read]);
            if (!warp_wait(&bars[kBarO2Done], ph, abort_flag)) { ok = false; break; }
            tc::tc_fence_after();
            const int64_t t0 = (int64_t)c * kT;
            const int64_t nleft = n - t0, lleft = L - t0;
            const int nv = nleft < kT ? (int)nleft : kT, lv = lleft < kT ? (int)lleft : kT;
            __nv_bfloat16* yc = y + t0 * row;
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t o2[16];
                tc::tmem_ld16(tl + cO + 16 * m, o2);
                if (m == 3) {
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bars[kBarO2Read]);
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const int i = 16 * m + j;
                    const float2 f0 = sc->out[i], f1 = sc->out[i + 1];
                    float a0 = fmaf(f0.x, __uint_as_float(o1[m][j]), f0.y * __uint_as_float(o2[j]));
                    float a1 = fmaf(f1.x, __uint_as_float(o1[m][j + 1]), f1.y * __uint_as_float(o2[j + 1]));
                    a0 = i < nv ? a0 : 0.f;
                    a1 = i + 1 < nv ? a1 : 0.f;
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
                    const uint32_t pair = odd ? tc::pack_bf16x2(got, a1) : tc::pack_bf16x2(a0, got);
                    if (live && i + odd < lv) *reinterpret_cast<uint32_t*>(yc + i * row) = pair;
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarSFree + buf]);
        }
        if (!ok) set_abort(ctl, p.status);
        if (ok && live)
            for (int64_t t = (int64_t)nc * kT; t + odd < L; t += 2) *reinterpret_cast<uint32_t*>(y + t * row) = 0u;
    } else if (warp < kScoreWarp0 + kScoreWarps) {
        // ============================== scores ==============================
        const int hv = (warp - kScoreWarp0) >> 2, w = (warp - kScoreWarp0) & 3;  // head, block of 16 rows
        const int tid = w * 32 + lane;
        const int gid = lane >> 2, tig = lane & 3;
        ScoreScratch* scr = reinterpret_cast<ScoreScratch*>(smem + p.off_scratch) + hv;
        const int64_t gbase = b * L * g.nheads + h0 + hv;
        // warp 0's lanes hold the next chunk's g and beta of tokens lane, lane + 32
        float gn[2], bn[2];
        auto fetch = [&](int c) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t t = (int64_t)c * kT + lane + 32 * r;
                gn[r] = t < n ? p.gate[gbase + t * g.nheads] : 0.f;
                bn[r] = t < n ? p.beta[gbase + t * g.nheads] : 0.f;
            }
        };
        if (w == 0 && nc > 0) fetch(0);
        int st = 0;
        uint32_t full_phase = 0;
        for (int c = 0; c < nc; ++c) {
            const int buf = c & 1;
            if (w == 0) {
                long long f[2];
                float be[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float lim = fminf(fmaxf(gn[r], -112.f), 112.f);  // |log2 decay| < 162
                    f[r] = __double2ll_rn((double)lim * 1.4426950408889634 * 4294967296.0);
                    be[r] = gn[r] != gn[r] ? gn[r] : bn[r];  // a NaN decay shows in the token's correction
                }
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const long long o = __shfl_up_sync(0xffffffffu, f[r], m);
                        if (lane >= m) f[r] += o;
                    }
                }
                f[1] += __shfl_sync(0xffffffffu, f[0], 31);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    TokScore* t = &scr->tok[lane + 32 * r];
                    t->gi = (float)(int)(f[r] >> 32);
                    t->gf = (float)(uint32_t)f[r] * 2.3283064365386963e-10f;
                    t->beta = be[r];
                }
                if (c + 1 < nc) fetch(c + 1);
            }
            // every warp of the head comes to the barrier below, whatever its waits said
            ok = warp_wait(&bars[kBarFull + st], full_phase, abort_flag);
            if (ok && c >= 2) ok = warp_wait(&bars[kBarSFree + buf], ((c >> 1) - 1) & 1, abort_flag);
            uint8_t* sK = smem + st * kStage;
            const uint32_t aK = tc::smem_u32(sK), aQ = aK + kOffQ;
            const int64_t left = n - (int64_t)c * kT;
            const int nv = left < kT ? (int)left : kT;
            // K K^T; the norms are its diagonal and Q Q^T's (summed by the same instructions, so that
            // rk_i rk_j (k_i . k_j) is 1 to rounding where keys agree)
            float acc[4][2][4];
            if (ok) {
                if (nv < kT) {
                    // past the row's end: K enters the state's product and has to be 0
                    const int r = 16 * w + (lane >> 1);
                    if (r >= nv) {
#pragma unroll
                        for (int i = 0; i < S / 16; ++i)
                            *reinterpret_cast<uint4*>(sK + (S == 128 ? (lane & 1) * kBox + sw(r, i)
                                                                     : sw(r, 4 * (lane & 1) + i))) =
                                make_uint4(0, 0, 0, 0);
                    }
                    __syncwarp();
                }
                if (p.l2norm) {
                    score_rows<S>(aQ, aQ, 16 * w, w, w, lane, acc);
                    diag_norm(acc, w, lane, p.l2_eps, [&](int i, float f) { scr->rq[16 * w + i] = f; });
                }
                score_rows<S>(aK, aK, 16 * w, 0, w, lane, acc);
                if (p.l2norm) {
                    diag_norm(acc, w, lane, p.l2_eps, [&](int i, float f) { scr->tok[16 * w + i].rk = f; });
                } else if (lane < 16) {
                    scr->tok[16 * w + lane].rk = 1.f;
                    scr->rq[16 * w + lane] = 1.f;
                }
            }
            ok = bar_sync_and(1 + hv, 128, ok);
            if (!ok) break;
            if (tid < kT) {
                const TokScore t = scr->tok[tid], last = scr->tok[kT - 1];
                Scalars* sc = scal_of(buf, hv);
                const float e = exp2f(t.gi) * exp2f(t.gf);
                const float d = exp2f(last.gi - t.gi) * exp2f(last.gf - t.gf);
                const float oq = p.scale * scr->rq[tid];
                *reinterpret_cast<float4*>(&sc->chain[tid]) = make_float4(t.beta, t.beta * e * t.rk, d * t.rk, 0.f);
                sc->out[tid] = make_float2(oq * e, oq);
                if (tid == kT - 1) sc->g_last = e;
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[kBarSFull + buf]);
            const TokScore ti0 = scr->tok[16 * w + gid], ti1 = scr->tok[16 * w + gid + 8];
            // A, in fp32: blocks below the diagonal, and the diagonal block by columns
            {
                const float f0 = ti0.beta * ti0.rk, f1 = ti1.beta * ti1.rk;
                const bool in0 = 16 * w + gid < nv, in1 = 16 * w + gid + 8 < nv;
#pragma unroll
                for (int jb = 0; jb < 4; ++jb) {
                    if (jb > w) break;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int jj = 8 * nt + 2 * tig, j = 16 * jb + jj;
                        const TokScore t0 = scr->tok[j], t1 = scr->tok[j + 1];
                        float (&a)[4] = acc[jb][nt];
                        a[0] = in0 ? a[0] * (f0 * t0.rk * exp2f((ti0.gi - t0.gi) + (ti0.gf - t0.gf))) : 0.f;
                        a[1] = in0 ? a[1] * (f0 * t1.rk * exp2f((ti0.gi - t1.gi) + (ti0.gf - t1.gf))) : 0.f;
                        a[2] = in1 ? a[2] * (f1 * t0.rk * exp2f((ti1.gi - t0.gi) + (ti1.gf - t0.gf))) : 0.f;
                        a[3] = in1 ? a[3] * (f1 * t1.rk * exp2f((ti1.gi - t1.gi) + (ti1.gf - t1.gf))) : 0.f;
                        if (jb < w) {
                            float2 (*low)[8] = scr->low[low_block(w, jb)];
                            low[gid][low_at(gid, jj / 2)] = make_float2(a[0], a[1]);
                            low[gid + 8][low_at(gid + 8, jj / 2)] = make_float2(a[2], a[3]);
                        } else {
                            scr->diag[w][jj][gid] = jj < gid ? a[0] : 0.f;
                            scr->diag[w][jj + 1][gid] = jj + 1 < gid ? a[1] : 0.f;
                            scr->diag[w][jj][gid + 8] = jj < gid + 8 ? a[2] : 0.f;
                            scr->diag[w][jj + 1][gid + 8] = jj + 1 < gid + 8 ? a[3] : 0.f;
                        }
                    }
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
            // fragments nf[d] (i = w + d), which are also left operands (see mma_tf32x3)
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
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt)
                                mma_tf32x3(x[nt], nf[m][kk], low[8 * nt + gid][low_at(gid, 4 * kk + tig)]);
                    }
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[nt][e] = -x[nt][e], nf[d][nt][e] = 0.f;
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
                            mma_tf32x3(nf[d][nt], x[kk],
                                       *reinterpret_cast<const float2*>(&scr->diag[i][8 * nt + gid][8 * kk + 2 * tig]));
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
                            r[x] = tc::pack_bf16x2(v[0], v[1]);
                            v[0] -= tc::bf16_lo(r[x]);
                            v[1] -= tc::bf16_hi(r[x]);
                        }
                        stsm4_trans(at + pl * kPlane, r);
                    }
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(&bars[kBarNFull]);
            // P, once the last chunk's has been used
            {
                score_rows<S>(aQ, aK, 16 * w, 0, w, lane, acc);
                if (ok && c > 0) ok = warp_wait(&bars[kBarPFree], (c - 1) & 1, abort_flag);
                uint8_t* sP = p_of(hv);
#pragma unroll
                for (int jb = 0; jb < 4; ++jb) {
                    if (jb > w || !ok) break;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int j = 16 * jb + 8 * nt + 2 * tig, i0 = 16 * w + gid;
                        const TokScore t0 = scr->tok[j], t1 = scr->tok[j + 1];
                        const float (&a)[4] = acc[jb][nt];
                        const float e0 = t0.rk * exp2f((ti0.gi - t0.gi) + (ti0.gf - t0.gf));
                        const float e1 = t1.rk * exp2f((ti0.gi - t1.gi) + (ti0.gf - t1.gf));
                        const float e2 = t0.rk * exp2f((ti1.gi - t0.gi) + (ti1.gf - t0.gf));
                        const float e3 = t1.rk * exp2f((ti1.gi - t1.gi) + (ti1.gf - t1.gf));
                        const uint32_t o0 = sw(i0, 2 * jb + nt) + 4 * tig;
                        uint32_t hi, lo;
                        split2(j <= i0 ? a[0] * e0 : 0.f, j + 1 <= i0 ? a[1] * e1 : 0.f, hi, lo);
                        *reinterpret_cast<uint32_t*>(sP + o0) = hi;
                        *reinterpret_cast<uint32_t*>(sP + kPlane + o0) = lo;
                        split2(j <= i0 + 8 ? a[2] * e2 : 0.f, j + 1 <= i0 + 8 ? a[3] * e3 : 0.f, hi, lo);
                        *reinterpret_cast<uint32_t*>(sP + o0 + 1024) = hi;
                        *reinterpret_cast<uint32_t*>(sP + kPlane + o0 + 1024) = lo;
                    }
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) tc::mbar_arrive(&bars[kBarPFull]);
            ok = bar_sync_and(1 + hv, 128, ok);  // the tokens' scalars have been read
            if (!ok) break;
            if (++st == p.nst) {
                st = 0;
                full_phase ^= 1u;
            }
        }
        if (!ok) set_abort(ctl, p.status);
    } else if (warp == kTmaWarp) {
        // ============================ TMA producer ============================
        if (lane == 0) {
            tc::tma_prefetch_desc(&tm_q);
            tc::tma_prefetch_desc(&tm_k);
            tc::tma_prefetch_desc(&tm_v);
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
                    tc::tma_load_4d(s + x * kBox, &tm_k, full, 64 * x, grp, c * kT, (int)b);
                    tc::tma_load_4d(s + kOffQ + x * kBox, &tm_q, full, 64 * x, grp, c * kT, (int)b);
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
    } else {
        // ============================= MMA issuer =============================
        if (lane == 0 && nc > 0) {
            constexpr uint32_t id_t = tc::idesc_bf16(128, kT, false, false);  // N = tokens
            constexpr uint32_t id_s = tc::idesc_bf16(128, S, false, true);    // N = state rows
            int st = 0;
            uint32_t full_phase = 0;
            for (int c = 0; c < nc; ++c) {
                const int buf = c & 1;
                const uint32_t ph = c & 1;
                const uint32_t aK = tc::smem_u32(smem + st * kStage);
                const uint64_t dK = tc::sdesc_sw128(aK, 16, 1024), dQ = tc::sdesc_sw128(aK + kOffQ, 16, 1024);
                const uint64_t dKt = tc::sdesc_sw128(aK, kBox, 1024);
                if (!tc::mbar_wait(&bars[kBarFull + st], full_phase, abort_flag)) { ok = false; break; }
                if (!tc::mbar_wait(&bars[kBarSFull + buf], (c >> 1) & 1, abort_flag)) { ok = false; break; }
                if (!tc::mbar_wait(&bars[kBarHReady], ph, abort_flag)) { ok = false; break; }
                tc::tc_fence_after();
                // R = K h, from h's two parts
#pragma unroll
                for (int ks = 0; ks < S / 16; ++ks)
                    tc::mma_bf16_ts(tmem + cR, tmem + cHi + 8 * ks, dK + (((ks >> 2) * kBox + (ks & 3) * 32) >> 4), id_t,
                                    ks > 0);
#pragma unroll
                for (int ks = 0; ks < S / 16; ++ks)
                    tc::mma_bf16_ts(tmem + cR, tmem + cLo + 8 * ks, dK + (((ks >> 2) * kBox + (ks & 3) * 32) >> 4), id_t,
                                    1);
                tc::mma_commit(&bars[kBarRDone]);
                // Q h, once the outputs of the chunk before have been read
                if (c > 0 && !tc::mbar_wait(&bars[kBarO2Read], ph ^ 1, abort_flag)) { ok = false; break; }
                tc::tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < S / 16; ++ks)
                    tc::mma_bf16_ts(tmem + cO, tmem + cHi + 8 * ks, dQ + (((ks >> 2) * kBox + (ks & 3) * 32) >> 4), id_t,
                                    ks > 0);
                tc::mma_commit(&bars[kBarO1Done]);
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
                // P W, once Q h has been read: hi hi + hi lo + lo hi
                if (!tc::mbar_wait(&bars[kBarPFull], ph, abort_flag)) { ok = false; break; }
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
                        tc::mma_bf16_ts(d, wp + 8 * kb, at, id, hv > 0 || kb > 0);
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
    constexpr uint32_t scratch = (NV * (uint32_t)sizeof(ScoreScratch) + 15) / 16 * 16;
    constexpr uint32_t rest =
        NV * ((kNPlanes + kPPlanes) * kPlane + 2 * kScalBytes) + scratch + kNumBars * 8 + (uint32_t)sizeof(SharedCtl) + 1024;
    constexpr int fit = (kSmemLimit - (int)rest) / (int)stage;
    static_assert(fit >= 2, "two stages at least");
    p.nst = fit < kMaxStages ? fit : kMaxStages;
    p.off_n = p.nst * stage;
    p.off_p = p.off_n + NV * kNPlanes * kPlane;
    p.off_scal = p.off_p + NV * kPPlanes * kPlane;
    p.off_scratch = p.off_scal + 2 * NV * kScalBytes;
    p.off_bar = p.off_scratch + scratch;
    const int smem = (int)(p.nst * stage + rest);

    CUtensorMap tm_q, tm_k, tm_v;
    const uint64_t L = g.seqlen, B = g.batch;
    const uint32_t box[4] = {64, 1, kT, 1};
    auto map = [&](CUtensorMap* m, const void* base, uint64_t width, uint64_t count, uint64_t stride) {
        const uint64_t dims[4] = {width, count, L, B};
        const uint64_t strides[3] = {width * 2, stride * 2, L * stride * 2};
        return make_tmap_bf16(m, base, 4, dims, strides, box);
    };
    if (!map(&tm_q, a.q, S, g.ngroups, a.q_stride) || !map(&tm_k, a.k, S, g.ngroups, a.k_stride) ||
        !map(&tm_v, a.v, H, g.nheads, a.v_stride))
        return cudaErrorInvalidValue;
    const cudaError_t e = ensure_max_dynamic_smem(reinterpret_cast<const void*>(k_gdr_chunk_tc<S, H, NV>), smem);
    if (e != cudaSuccess) return e;
    k_gdr_chunk_tc<S, H, NV><<<dim3((unsigned)(g.nheads / NV), (unsigned)g.batch), (kScoreWarp0 + 4 * NV + 2) * 32,
                               smem, st>>>(tm_q, tm_k, tm_v, p);
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
