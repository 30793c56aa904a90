// Linear attention with a decay for each head on tensor cores: a walk (layer.h, linattn.cu)
// over chunks of 128 tokens, bf16 operands, fp32 state.
//
// In a chunk of n tokens with the state S entering it, lam = e^{log_decay} and the rows a, k, v
// of its tokens, a forward walk is (a reverse walk is its mirror image)
//     o_i = read (sum_{j <= i} lam^{i-j} (a_i . k_j) write v_j + lam^{i+1} a_i S)
//     S'  = lam^n S + sum_j k_j (write lam^{n-1-j} v_j)^T
// four products with M = 128 on tcgen05: the scores A K^T, P V with the decayed, masked scores P
// (bf16, in tensor memory), A S (S rounded to bf16) and K^T V'.  S itself stays in registers in
// fp32.  Its update must not lose the 24 bits: V' = write lam^{n-1-j} v is split exactly into
// three bf16 parts (truncations: 8 bits each), side by side as one operand of 192 columns so that
// K is read once; each chunk's sums start from zero in tensor memory and are added to S in fp32.
// P and the S of the readout are rounded to bf16 once, half a step of 2^-8 on terms of an output
// that is itself stored as bf16.
//
// A block walks one segment of one (batch row, head), 64 columns of v and the state: per
// chunk 80 KB come in by TMA and 16 KB go out.  One block an SM, its 20 warps with a role each:
//     warp 0       TMA loads, two chunks ahead, each tile again as soon as its last reader is done
//     warp 1       all MMAs, per chunk: A K^T, K^T V', A S, P V
//     warps 4-11   P from the scores, and the output (a thread a token and half of the columns)
//     warps 12-15  the state (a thread a state row, 64 values in registers)
//     warps 16-19  V'
// so that P is made while K^T V' and A S run, and V', the state and the output of one chunk
// beside the products of the next.
#include <atomic>

#include "chunk_common.cuh"
#include "layer.h"

namespace ssm {

// Device word raised by the bounded waits of these kernels (0 = no error).
__device__ int ssm_la_error_word;

namespace la {

using namespace umma;
using chunkc::WAIT_LIMIT;

constexpr int C = 128;                   // tokens of a chunk
constexpr int THREADS = 640;
constexpr uint32_t TILE = 16384;         // 128 rows x 128 bytes (64 bf16), 128-byte swizzle
constexpr uint32_t ST_A = 0, ST_K = 2 * TILE, ST_V = 4 * TILE, STAGE = 5 * TILE;
constexpr uint32_t SM_VP = 2 * STAGE;    // V' in three parts
constexpr uint32_t SM_S = SM_VP + 3 * TILE;   // S as the bf16 operand of the readout
constexpr uint32_t SM_F32 = SM_S + TILE;
constexpr int F_PW = 0;                  // [129] lam^m
constexpr int F_W = 132;                 // [160] read write lam^m at 32 + m, zero below
constexpr int F_UP = F_W + 160;          // [32] lam^u
constexpr int F_DOWN = F_UP + 32;        // [32] lam^{31 - u}
constexpr int F_END = F_DOWN + 32;
constexpr uint32_t SM_BAR = SM_F32 + F_END * 4;
constexpr uint32_t SMEM_BYTES = SM_BAR + 224 + 1024;
static_assert(F_UP % 4 == 0 && F_DOWN % 4 == 0, "16-byte rows");
static_assert(SM_BAR % 8 == 0 && SMEM_BYTES <= 232448, "one block an SM");
// tensor memory columns
constexpr uint32_t TM_SC = 0;            // 128: scores
constexpr uint32_t TM_OI = 128;          // 64: P V
constexpr uint32_t TM_OS = 192;          // 64: A S
constexpr uint32_t TM_KV = 256;          // 3 x 64: K^T V', a part each
constexpr uint32_t TM_P = 448;           // 64: P, two bf16 a column
constexpr uint32_t TM_COLS = 512;

struct Maps {
    CUtensorMap a, k, v;
};
struct Args {
    LaArgs p;
    int o32[3];      // the output takes 32-byte stores
    float *seg[3];   // [segment][b H + h][da][dc]: what a segment adds, then its entering state
    int nseg, G;     // segments of G chunks
    int slices;      // 64-column slices, the most of all walks
};

// Descriptor (umma.cuh, sdesc) of 128-byte-swizzled rows with leading offset LBO, at an address
// in 16-byte units: only its low word is not constant.
template <uint32_t LBO> __device__ __forceinline__ uint64_t desc(uint32_t units) {
    constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | LAYOUT_SW128 << 29;
    return (uint64_t)hi << 32 | (units | (LBO >> 4) << 16);
}
// One lane of a converged warp, known to the compiler to be one.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(one));
    return one != 0;
}
// D[tmem] (+)= A[tmem] * B[smem]; issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
#define LA_R16(r) \
    "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), \
    "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
// 32 columns of the thread's lane; the values are there after tmem_wait_ld
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : LA_R16(a), LA_R16(b)
        : "r"(taddr));
}
// (the values pass through, so that nothing reads them before)
#define LA_IO16(r) \
    "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), \
    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" : LA_IO16(a), LA_IO16(b)::"memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&r)[8], uint32_t (&q)[8], uint32_t (&t)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(q[0]), "+r"(q[1]), "+r"(q[2]), "+r"(q[3]), "+r"(q[4]), "+r"(q[5]), "+r"(q[6]), "+r"(q[7]),
                   "+r"(t[0]), "+r"(t[1]), "+r"(t[2]), "+r"(t[3]), "+r"(t[4]), "+r"(t[5]), "+r"(t[6]), "+r"(t[7])
                 :: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&r);
}
// the bf16 parts (high halves) of two floats as one word
__device__ __forceinline__ uint32_t high2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// (a.x b.x, a.y b.y) in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(reinterpret_cast<uint64_t &>(r))
        : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
    return r;
}
__device__ __forceinline__ void st32(void *p, uint4 a, uint4 b) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

struct Bars {
    uint64_t a_full[2], k_full[2], v_full[2];   // tiles loaded
    uint64_t a_free[2], k_free[2], v_free[2];   // tiles read by their last product
    uint64_t sc, kv, o;                         // products done: scores; K^T V'; A S and P V
    uint64_t p, vp, s;                          // operands written: P, V', S
    uint64_t kv_read, o_read;                   // results fetched from tensor memory
    uint64_t end;
    uint32_t tslot;
    int abort;
};
static_assert(sizeof(Bars) <= 224, "barrier space");

// Bounded wait for the completion number `n` (from 0) of a barrier; false, with the error word
// and the block's abort flag raised, when it does not come or another role has given up.  The
// hint lets the hardware keep the thread suspended: polls of 16 waiting warps would take the
// issue slots that the others need.
constexpr uint32_t POLL_NS = 20000, POLLS = 1u << 15;   // about half a second
__device__ __forceinline__ bool await(Bars *B, uint64_t *bar, uint32_t n) {
#pragma unroll 1
    for (uint32_t i = 0; i < POLLS; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(n & 1u), "r"(POLL_NS)
            : "memory");
        if (ok) return true;
        if (*reinterpret_cast<volatile int *>(&B->abort)) return false;
    }
    *reinterpret_cast<volatile int *>(&B->abort) = 1;
    atomicCAS(&ssm_la_error_word, 0, 1);
    return false;
}
// The same for a whole warp, all lanes alike.
__device__ __forceinline__ bool await_warp(Bars *B, uint64_t *bar, uint32_t n) {
    return __all_sync(0xffffffffu, await(B, bar, n));
}
// One arrival a warp, after all its lanes are done.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// STATE: only the state is walked (no scores, no output).
template <bool STATE>
__global__ void __launch_bounds__(THREADS, 1)
k_la_walk(const __grid_constant__ Maps m0, const __grid_constant__ Maps m1,
          const __grid_constant__ Maps m2, const __grid_constant__ Args A) {
    const LaArgs &p = A.p;
    const int BH = p.B * p.H;
    int id = blockIdx.x;
    const int slice = id % A.slices;
    id /= A.slices;
    const int bh = id % BH;
    id /= BH;
    const int sg = id % A.nseg, wi = id / A.nseg;
    const LaWalk &w = p.w[wi];
    const Maps *maps = wi == 0 ? &m0 : wi == 1 ? &m1 : &m2;
    const int c0 = 64 * slice;
    if (c0 >= w.dc) return;
    const int b = bh / p.H, h = bh - b * p.H;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
    const int first = sg * A.G, nch = min(A.G, (len + C - 1) / C - first);   // chunks; may be <= 0
    const bool rev = w.rev;

    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *f32 = reinterpret_cast<float *>(sm + SM_F32);
    Bars *B = reinterpret_cast<Bars *>(sm + SM_BAR);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i)
            for (uint64_t *q : {&B->a_full[i], &B->k_full[i], &B->v_full[i], &B->a_free[i], &B->k_free[i], &B->v_free[i]})
                mbar_init(q, 1);
        for (uint64_t *q : {&B->sc, &B->kv, &B->o, &B->end}) mbar_init(q, 1);
        for (uint64_t *q : {&B->vp, &B->s, &B->kv_read}) mbar_init(q, 4);    // an arrival a warp
        for (uint64_t *q : {&B->p, &B->o_read}) mbar_init(q, 8);
        B->abort = 0;
        mbar_fence_init();
    }
    if (warp == 1) tmem_alloc(&B->tslot, TM_COLS);
    {   // powers of lam from its logarithm in 64 bits: every one right to half a step
        double g = (double)p.log_decay[h];
        if (g < -1e6) g = -1e6;   // -inf: lam^0 stays 1
        const double rw = (double)w.read * (double)w.write;
        for (int i = tid; i < 129 + 160 + 64; i += THREADS) {
            if (i < 129) f32[F_PW + i] = (float)exp(g * i);
            else if (i < 289) f32[F_W + i - 129] = i < 161 ? 0.f : (float)(rw * exp(g * (i - 161)));
            else if (i < 321) f32[F_UP + i - 289] = (float)exp(g * (i - 289));
            else f32[F_DOWN + i - 321] = (float)exp(g * (352 - i));
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = B->tslot;
    const uint32_t lane_q = (uint32_t)(32 * (warp & 3)) << 16;
    const int row = 32 * (warp & 3) + lane;      // token, or state row, of the thread
    // chunk number c of the walk: its first token and its tokens
    auto chunk = [&](int c) { return C * (first + (rev ? nch - 1 - c : c)); };
    auto ntok = [&](int t0) { return min(C, len - t0); };
    // rows of the chunk's tiles that are other tokens (TMA fills those past L with zeros)
    auto dirty = [&](int t0, int n) { return n < C && t0 + n < p.L; };

    if (warp == 0) {
        if (lane == 0) {
            const int nboxa = (w.da + 63) / 64, ha = h / w.rep_a, hk = h / w.rep_k, hv = h / w.rep_v;
            uint32_t got_a = 0, got_k = 0, got_v = 0;   // loads issued
#pragma unroll 1
            for (int c = 0; c < nch; ++c) {
                const int s = c & 1, t0 = chunk(c);
                const uint32_t n = (uint32_t)(c >> 1) - 1u;
                unsigned char *st = sm + s * STAGE;
                if (c >= 2 && !await(B, &B->k_free[s], n)) break;
                mbar_expect_tx(&B->k_full[s], 2 * TILE);
                tma_load_4d(st + ST_K, &maps->k, &B->k_full[s], 0, hk, t0, b);
                // a second box past the head is zeros: state rows that are not there
                tma_load_4d(st + ST_K + TILE, &maps->k, &B->k_full[s], 64, hk, t0, b);
                ++got_k;
                if (!STATE) {
                    if (c >= 2 && !await(B, &B->a_free[s], n)) break;
                    mbar_expect_tx(&B->a_full[s], TILE * nboxa);
                    for (int i = 0; i < nboxa; ++i)
                        tma_load_4d(st + ST_A + i * TILE, &maps->a, &B->a_full[s], 64 * i, ha, t0, b);
                    ++got_a;
                }
                if (c >= 2 && !await(B, &B->v_free[s], n)) break;
                mbar_expect_tx(&B->v_full[s], TILE);
                tma_load_4d(st + ST_V, &maps->v, &B->v_full[s], c0, hv, t0, b);
                ++got_v;
            }
            // no copy is in flight when the block ends
            for (uint32_t i = 0; i < 2; ++i) {
                if (got_a > i) mbar_wait(&B->a_full[(got_a - 1 - i) & 1], ((got_a - 1 - i) >> 1) & 1u, WAIT_LIMIT);
                if (got_k > i) mbar_wait(&B->k_full[(got_k - 1 - i) & 1], ((got_k - 1 - i) >> 1) & 1u, WAIT_LIMIT);
                if (got_v > i) mbar_wait(&B->v_full[(got_v - 1 - i) & 1], ((got_v - 1 - i) >> 1) & 1u, WAIT_LIMIT);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t base = smem_u32(sm);
            constexpr uint32_t id_sc = idesc_bf16(128, 128, false, false), id_n = idesc_bf16(128, 64, false, true);
            constexpr uint32_t id_kv = idesc_bf16(128, 192, true, true);
            // descriptors: their address field counts 16-byte units; along a row, 16 values are 2 of them
            const uint32_t u0 = base >> 4;
            auto kmaj = [&](uint32_t tile, int s) { return desc<16u>(u0 + (tile >> 4) + (s >> 2) * (TILE >> 4) + (s & 3) * 2u); };
            auto mnmaj = [&](uint32_t tile, int s) { return desc<TILE>(u0 + (tile >> 4) + 128u * s); };
            const int ks = (w.da + 15) / 16;
#pragma unroll 1
            for (int c = 0; c < nch; ++c) {
                const uint32_t st = (c & 1) ? STAGE : 0u;
                const uint32_t half = (uint32_t)c >> 1;
                if (!await(B, &B->k_full[c & 1], half)) break;
                if (!STATE) {
                    if (!await(B, &B->a_full[c & 1], half)) break;
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        if (s < ks) mma_bf16(tm + TM_SC, kmaj(st + ST_A, s), kmaj(st + ST_K, s), id_sc, s > 0);
                    mma_commit(&B->sc);
                }
                if (!await(B, &B->vp, (uint32_t)c)) break;
                if (c > 0 && !await(B, &B->kv_read, (uint32_t)c - 1u)) break;
                fence_after_sync();
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_bf16(tm + TM_KV, mnmaj(st + ST_K, s), mnmaj(SM_VP, s), id_kv, s > 0);
                mma_commit(&B->kv);
                mma_commit(&B->k_free[c & 1]);
                if (!STATE) {
                    if (!await(B, &B->s, (uint32_t)c)) break;
                    if (c > 0 && !await(B, &B->o_read, (uint32_t)c - 1u)) break;
                    fence_after_sync();
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        if (s < ks) mma_bf16(tm + TM_OS, kmaj(st + ST_A, s), mnmaj(SM_S, s), id_n, s > 0);
                    mma_commit(&B->a_free[c & 1]);
                    if (!await(B, &B->p, (uint32_t)c)) break;
                    fence_after_sync();
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ts(tm + TM_OI, tm + TM_P + 8u * s, mnmaj(st + ST_V, s), id_n, s > 0);
                    mma_commit(&B->o);
                }
                mma_commit(&B->v_free[c & 1]);
            }
            mma_commit(&B->end);   // every MMA is over before tensor memory goes
            mbar_wait(&B->end, 0u, WAIT_LIMIT);
        }
        __syncwarp();
    } else if (!STATE && warp >= 4 && warp < 12) {
        const int half = (warp - 4) >> 2, qd = warp & 3;
        const long long ob = b * w.so[0] + h * w.so[2] + c0 + 32 * half;
        const int nq = min(4, (w.dc - c0 - 32 * half) / 8);   // 8-column pieces of the output (<= 0: none)
        const bool wide = A.o32[wi] && nq == 4;
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
            const int t0 = chunk(c), n = ntok(t0);
            if (!await_warp(B, &B->sc, (uint32_t)c)) break;
            fence_after_sync();
            // P[i][j] = read write lam^{|i - j|} (a_i . k_j) on one side of the diagonal, 32 columns
            // at a time
#pragma unroll 1
            for (int z = 0; z < 2; ++z) {
                const int jb = 2 * half + z;
                uint32_t o[16];
                if (rev ? jb < qd : jb > qd) {   // masked
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = 0u;
                } else {
                    uint32_t x[16], y[16];
                    tmem_ld32(tm + TM_SC + lane_q + 32u * jb, x, y);
                    const int left = n - 32 * jb;   // columns of this sequence
                    if (jb == qd || left < 32) {
                        // the diagonal, and the sequence's end: tokens past it are not read, whatever they hold
                        const int at = rev ? 32 * jb - row : row - 32 * jb, d = rev ? 1 : -1;
                        float wv[32];
#pragma unroll
                        for (int u = 0; u < 32; ++u) wv[u] = f32[F_W + 32 + at + d * u];
                        tmem_wait_ld(x, y);
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            o[u] = pack2(2 * u < left ? __uint_as_float(x[2 * u]) * wv[2 * u] : 0.f,
                                         2 * u + 1 < left ? __uint_as_float(x[2 * u + 1]) * wv[2 * u + 1] : 0.f);
                            o[8 + u] = pack2(16 + 2 * u < left ? __uint_as_float(y[2 * u]) * wv[16 + 2 * u] : 0.f,
                                             17 + 2 * u < left ? __uint_as_float(y[2 * u + 1]) * wv[17 + 2 * u] : 0.f);
                        }
                    } else {
                        // off it the weight is a factor of the row times one of the column
                        const float r = f32[F_W + 32 + (rev ? 32 * jb - row : row - 32 * jb - 31)];
                        const float4 *cw = reinterpret_cast<const float4 *>(f32 + (rev ? F_UP : F_DOWN));
                        const float2 rr = make_float2(r, r);
                        tmem_wait_ld(x, y);
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float4 f = cw[u];
                            const uint32_t *s4 = u < 4 ? x + 4 * u : y + 4 * (u - 4);
                            const float2 e0 = mul2(mul2(make_float2(__uint_as_float(s4[0]), __uint_as_float(s4[1])), rr), make_float2(f.x, f.y));
                            const float2 e1 = mul2(mul2(make_float2(__uint_as_float(s4[2]), __uint_as_float(s4[3])), rr), make_float2(f.z, f.w));
                            o[2 * u] = pack2(e0.x, e0.y);
                            o[2 * u + 1] = pack2(e1.x, e1.y);
                        }
                    }
                }
                tmem_st16(tm + TM_P + lane_q + 16u * jb, o);
            }
            tmem_wait_st();
            fence_before_sync();
            warp_arrive(&B->p);
            if (!await_warp(B, &B->o, (uint32_t)c)) break;
            fence_after_sync();
            uint32_t x[16], y[16], u[16], v[16];
            tmem_ld32(tm + TM_OI + lane_q + 32u * half, x, y);
            tmem_ld32(tm + TM_OS + lane_q + 32u * half, u, v);
            const float e = w.read * f32[F_PW + max(0, rev ? n - 1 - row : row + 1)];
            tmem_wait_ld(x, y);
            tmem_wait_ld(u, v);
            fence_before_sync();
            warp_arrive(&B->o_read);
            float o[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                o[j] = fmaf(e, __uint_as_float(u[j]), __uint_as_float(x[j]));
                o[16 + j] = fmaf(e, __uint_as_float(v[j]), __uint_as_float(y[j]));
            }
            if (row < n) {
                const long long at = ob + (long long)(t0 + row) * w.so[1];
                if (w.o_f32) {
                    float4 *dst = reinterpret_cast<float4 *>(reinterpret_cast<float *>(w.o) + at);
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (q < 2 * nq) dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(w.o) + at);
                    uint4 r[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        r[q] = make_uint4(pack2(o[8 * q], o[8 * q + 1]), pack2(o[8 * q + 2], o[8 * q + 3]),
                                          pack2(o[8 * q + 4], o[8 * q + 5]), pack2(o[8 * q + 6], o[8 * q + 7]));
                    if (wide) {
                        st32(dst, r[0], r[1]);
                        st32(dst + 2, r[2], r[3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (q < nq) dst[q] = r[q];
                    }
                }
            }
        }
    } else if (warp >= 12 && warp < 16) {
        float S[64];
        const bool live = row < w.da;
        const float *src = STATE && A.nseg > 1 ? nullptr   // a segment's own sum
                         : A.nseg > 1 ? A.seg[wi] + ((long long)sg * BH + bh) * w.da * w.dc
                         : w.s_in ? w.s_in + (long long)bh * w.da * w.dc : nullptr;
        const int sta = A.nseg > 1 ? w.dc : w.st_a, stc = A.nseg > 1 ? 1 : w.st_c;
        const long long at = (long long)row * sta + (long long)c0 * stc;
        const int cols = live ? w.dc - c0 : 0;
        {
            const float *q = src + at;
            const int n = src ? cols : 0;
#pragma unroll
            for (int j = 0; j < 64; ++j, q += stc) S[j] = j < n ? *q : 0.f;
        }
        auto operand = [&]() {   // S in bf16, the layout of a V tile
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint4 v = make_uint4(pack2(S[8 * q], S[8 * q + 1]), pack2(S[8 * q + 2], S[8 * q + 3]),
                                           pack2(S[8 * q + 4], S[8 * q + 5]), pack2(S[8 * q + 6], S[8 * q + 7]));
                *reinterpret_cast<uint4 *>(sm + SM_S + row * 128 + ((q ^ (row & 7)) << 4)) = v;
            }
            fence_proxy_async();
            warp_arrive(&B->s);
        };
        if (!STATE) operand();
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
            const float E = f32[F_PW + ntok(chunk(c))];
            if (!await_warp(B, &B->kv, (uint32_t)c)) break;
            fence_after_sync();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint32_t x[8], y[8], z[8];
                tmem_ld8(tm + TM_KV + lane_q + 8u * q, x);
                tmem_ld8(tm + TM_KV + lane_q + 64u + 8u * q, y);
                tmem_ld8(tm + TM_KV + lane_q + 128u + 8u * q, z);
                tmem_wait_ld8(x, y, z);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    S[8 * q + j] = fmaf(E, S[8 * q + j],
                                        __uint_as_float(x[j]) + (__uint_as_float(y[j]) + __uint_as_float(z[j])));
            }
            fence_before_sync();
            warp_arrive(&B->kv_read);
            if (!STATE && c + 1 < nch) {
                // A S of this chunk has read the operand
                if (!await_warp(B, &B->a_free[c & 1], (uint32_t)c >> 1)) break;
                operand();
            }
        }
        float *dst = A.nseg > 1 ? (STATE ? A.seg[wi] + ((long long)sg * BH + bh) * w.da * w.dc : nullptr)
                                : w.s_out ? w.s_out + (long long)bh * w.da * w.dc : nullptr;
        if (dst) {
            float *q = dst + at;
#pragma unroll
            for (int j = 0; j < 64; ++j, q += stc)
                if (j < cols) *q = S[j];
        }
    } else if (warp >= 16) {
        const int t = tid - 512;
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
            unsigned char *st = sm + (c & 1) * STAGE;
            const int t0 = chunk(c), n = ntok(t0);
            const bool fix = dirty(t0, n);
            if (!await_warp(B, &B->v_full[c & 1], (uint32_t)c >> 1)) break;
            if (c > 0 && !await_warp(B, &B->kv, (uint32_t)c - 1u)) break;   // V' has been read
            if (fix && !await_warp(B, &B->k_full[c & 1], (uint32_t)c >> 1)) break;
            if (fix && !STATE && !await_warp(B, &B->sc, (uint32_t)c)) break;   // the scores have read K
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
                const int ch = t + 128 * q, r = ch >> 3;   // 16-byte piece of row r
                const uint32_t off = (uint32_t)ch * 16u;
                uint4 x = *reinterpret_cast<const uint4 *>(st + ST_V + off);
                if (fix && r >= n) {
                    x = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(st + ST_V + off) = x;
                    *reinterpret_cast<uint4 *>(st + ST_K + off) = x;
                    *reinterpret_cast<uint4 *>(st + ST_K + TILE + off) = x;
                }
                const float f = w.write * f32[F_PW + (rev ? r + 1 : max(0, n - 1 - r))];
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[3][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a = lo_f(u[i]) * f, bb = hi_f(u[i]) * f;
#pragma unroll
                    for (int z = 0; z < 3; ++z) {
                        o[z][i] = high2(a, bb);
                        a -= hi_f(__float_as_uint(a));
                        bb -= hi_f(__float_as_uint(bb));
                    }
                }
#pragma unroll
                for (int z = 0; z < 3; ++z)
                    *reinterpret_cast<uint4 *>(sm + SM_VP + z * TILE + off) = make_uint4(o[z][0], o[z][1], o[z][2], o[z][3]);
            }
            fence_proxy_async();
            warp_arrive(&B->vp);
        }
    }
    fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        fence_after_sync();
        tmem_dealloc(tm, TM_COLS);
    }
}

// The state entering every segment, in place of what the segment adds, and the state that
// leaves the walk: a thread an element, the segments in the walk's order.
__global__ void __launch_bounds__(256) k_la_segments(const __grid_constant__ Args A) {
    const LaArgs &p = A.p;
    const LaWalk &w = p.w[blockIdx.y];
    const int BH = p.B * p.H, bh = blockIdx.x % BH, b = bh / p.H, h = bh - b * p.H;
    const int e = blockIdx.x / BH * 256 + threadIdx.x, a = e / w.dc, c = e - a * w.dc;
    if (a >= w.da) return;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
    double g = (double)p.log_decay[h];
    if (g < -1e6) g = -1e6;
    const long long at = (long long)bh * w.da * w.dc, ext = at + (long long)a * w.st_a + (long long)c * w.st_c;
    float E = w.s_in ? w.s_in[ext] : 0.f;
    for (int i = 0; i < A.nseg; ++i) {
        const int s = w.rev ? A.nseg - 1 - i : i;
        const int n = min(max(len - s * A.G * C, 0), A.G * C);   // its tokens
        float *q = A.seg[blockIdx.y] + (long long)s * BH * w.da * w.dc + at + e;
        const float add = *q;
        *q = E;
        E = fmaf((float)exp(g * n), E, add);
    }
    if (w.s_out) w.s_out[ext] = E;
}

bool make_map(CUtensorMap *m, const void *base, int d, int heads, const LaArgs &p, const long long *s) {
    chunkc::EncodeTiledFn fn = chunkc::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)p.L, (cuuint64_t)p.B};
    // the stride of a dimension of one is not used, and need not be a valid one
    cuuint64_t st[3] = {(cuuint64_t)(heads > 1 ? s[2] * 2 : 16), (cuuint64_t)(p.L > 1 ? s[1] * 2 : 16),
                        (cuuint64_t)(p.B > 1 ? s[0] * 2 : 16)};
    cuuint32_t box[4] = {64, 1, C, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, st, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Allows the walks their shared memory, once a device.
cudaError_t set_smem() {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    if ((e = cudaFuncSetAttribute(k_la_walk<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES)) ||
        (e = cudaFuncSetAttribute(k_la_walk<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES)))
        return e;
    if (dev < 64) done.fetch_or(1ull << dev);
    return cudaSuccess;
}

}  // namespace la

// Walks that may take the tensor cores by their sizes.
bool la_chunked_sizes(int bf16, int da, int dc) { return bf16 && da <= 128 && da % 8 == 0 && dc % 8 == 0; }

// Segments of the sequences (of `L` tokens; `items` blocks without segments): the count with
// the shortest estimate, where a chunk's walk takes 1 and its state alone 1/2, 148 blocks run
// at a time, and the two more launches take 4.
int la_segments(long long L, long long items) {
    const long long nc = (L + la::C - 1) / la::C;
    double best = 0;
    int pick = 1;
    for (long long n = 1; n <= nc && n <= 64; ++n) {
        const long long g = (nc + n - 1) / n, seg = (nc + g - 1) / g, waves = (items * seg + 147) / 148;
        const double t = (double)(waves * g) * (seg > 1 ? 1.5 : 1.0) + (seg > 1 ? 4 : 0);
        if (seg == n && (n == 1 || t < 0.95 * best)) {
            best = t;
            pick = (int)n;
        }
    }
    return pick;
}

// The walks of `p` on tensor cores with `nseg` segments and their states in seg[]; false (and
// nothing done) where the tensors' alignment does not allow it.
bool la_chunked(const LaArgs &p, int nseg, float *const *seg, cudaStream_t st, cudaError_t *err) {
    using namespace la;
    Maps m[3] = {};
    Args A = {};
    A.p = p;
    A.slices = 0;
    for (int i = 0; i < p.nwalk; ++i) {
        const LaWalk &w = p.w[i];
        auto ok = [](const void *q, const long long *s, int el) {
            return ((uintptr_t)q & 15) == 0 && s[0] % el == 0 && s[1] % el == 0 && s[2] % el == 0;
        };
        if (!la_chunked_sizes(p.bf16, w.da, w.dc) || !ok(w.a, w.sa, 8) || !ok(w.k, w.sk, 8) ||
            !ok(w.v, w.sv, 8) || (w.o && !ok(w.o, w.so, w.o_f32 ? 4 : 8)))
            return false;
        if (!make_map(&m[i].a, w.a, w.da, p.H / w.rep_a, p, w.sa) ||
            !make_map(&m[i].k, w.k, w.da, p.H / w.rep_k, p, w.sk) ||
            !make_map(&m[i].v, w.v, w.dc, p.H / w.rep_v, p, w.sv))
            return false;
        const int sl = (w.dc + 63) / 64;
        A.slices = sl > A.slices ? sl : A.slices;
        A.seg[i] = seg[i];
        A.o32[i] = w.o && !w.o_f32 && ((uintptr_t)w.o & 31) == 0 && w.so[0] % 16 == 0 && w.so[1] % 16 == 0 && w.so[2] % 16 == 0;
    }
    const int nc = (p.L + C - 1) / C;
    A.G = (nc + nseg - 1) / nseg;
    A.nseg = (nc + A.G - 1) / A.G;
    const bool state_only = p.nwalk == 1 && !p.w[0].o;
    const long long items = (long long)p.nwalk * A.nseg * p.B * p.H * A.slices;
    if ((*err = set_smem()) != cudaSuccess) return true;
    if (A.nseg > 1 || state_only) {
        k_la_walk<true><<<(unsigned)items, THREADS, SMEM_BYTES, st>>>(m[0], m[1], m[2], A);
        profile_mark(st, "k_la_walk_state");
        if ((*err = cudaGetLastError()) != cudaSuccess) return true;
    }
    if (A.nseg > 1) {
        int n = 0;
        for (int i = 0; i < p.nwalk; ++i) n = p.w[i].da * p.w[i].dc > n ? p.w[i].da * p.w[i].dc : n;
        k_la_segments<<<dim3((n + 255) / 256 * p.B * p.H, p.nwalk), 256, 0, st>>>(A);
        profile_mark(st, "k_la_segments");
        if ((*err = cudaGetLastError()) != cudaSuccess) return true;
    }
    if (!state_only) {
        k_la_walk<false><<<(unsigned)items, THREADS, SMEM_BYTES, st>>>(m[0], m[1], m[2], A);
        profile_mark(st, "k_la_walk");
    }
    *err = cudaGetLastError();
    return true;
}

// Read and clear the device error word of these kernels.
int la_error_take() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, ssm_la_error_word, sizeof(int)) != cudaSuccess) return -1;
    if (v) cudaMemcpyToSymbol(ssm_la_error_word, &zero, sizeof(int));
    return v;
}

}  // namespace ssm
