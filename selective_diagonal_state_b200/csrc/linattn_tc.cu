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
// chunk 80 KB come in by TMA and 16 KB go out.  One block an SM, its 28 warps with a role each:
//     warp 0       TMA loads, two chunks ahead, each tile again as soon as its last reader is done
//     warps 1, 3   MMAs: K^T V'; and A S, P V, then the next chunk's A K^T (one warp for all of them
//                  spent half of a chunk's time in its waits between the products)
//     warp 2       TMA stores of the output, which is laid over the chunk's V tile (fp32: A tiles)
//     warps 4-11   P from the scores, and the output (a thread a token and half of the columns)
//     warps 12-19  the state (a thread a state row and half of the columns, in registers)
//     warps 20-27  V', in halves of 64 tokens, v straight from L2
// so that P, V', the state and the output of one chunk are made beside the products of others.
//
// On one B200, 4 x 16384 tokens of 16 heads of 128 / 128: 319 us, 1.08 GB (3.4 TB/s) and 0.5
// PFLOP/s (384 us call behind call for two seconds: at 1000 W the SMs run at 1550 MHz); 4 x 4096 tokens of 16 heads over 4: 87 us, the gradient 312; 1 x 257: 14 us.  What bounds
// it is none of the units (tensor pipe 26 %, issue 47 %, HBM 26 %) but the steps of a chunk handed on
// from role to role, 2.5 us a chunk: scores, P, P V, output, and K^T V', state, A S.  Taking the
// output off the first of these chains (P a chunk ahead of it, two accumulators) was no faster, 328 us.
// Steps that counted:
// the roles' own warps (a block of 20 warps with all of a chunk's MMAs in one took 351 us);
// v from L2 by registers instead of out of the V tile (403 to 351); two warps for the MMAs (327).
// Every role runs its own code once a chunk, so the walk is compiled for each direction and kind of
// output and its loops stay rolled: instruction fetch was what bound a kernel of the same
// structure with unrolled, run-time variants (185 KB of code, 613 us; 72 KB, 412 us).
#include <atomic>

#include "chunk_common.cuh"
#include "layer.h"

namespace ssm {

// Device word raised by the bounded waits of these kernels (0 = no error).
__device__ int ssm_la_error_word;

namespace la {

using namespace umma;

constexpr int C = 128;                   // tokens of a chunk
constexpr int THREADS = 896;
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
constexpr uint32_t SMEM_BYTES = SM_BAR + 256 + 1024;
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
    CUtensorMap a, k, v, o;
};
struct Args {
    LaArgs p;
    float *seg[3];   // [segment][b H + h][da][dc]: what a segment adds, then its entering state
    int nseg, G;     // segments of G chunks
    int slices;      // 64-column slices, the most of all walks
    uint32_t polls;  // of a wait of a role for another (await)
};

// Descriptor (umma.cuh, sdesc) of 128-byte-swizzled rows with leading offset LBO, at an address
// in 16-byte units: only its low word is not constant.
template <uint32_t LBO> __device__ __forceinline__ uint64_t desc(uint32_t units) {
    constexpr uint32_t hi = (1024u >> 4) | 1u << 14 | LAYOUT_SW128 << 29;
    return (uint64_t)hi << 32 | (units | (LBO >> 4) << 16);
}
// 16 bytes that stay out of L1, or zeros; one statement, so that nothing waits for the load but
// the values' use (behind a branch, the choice of the value does).
__device__ __forceinline__ uint4 ld_once(const void *p, bool on) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}\n"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)on));
    return v;
}
// Prefetch of a tile into L2.
__device__ __forceinline__ void tma_prefetch_4d(const void *tmap, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];\n" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
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
// Loads from tensor memory write their registers at any time up to the wait, behind the
// compiler's back: a copy or a reuse of one of them in between reads or destroys a value.
// So each load and its wait are one statement.  Columns of the thread's lane:
#define LA_OUT8(r, k) \
    "=&r"(r[k]), "=&r"(r[k + 1]), "=&r"(r[k + 2]), "=&r"(r[k + 3]), "=&r"(r[k + 4]), "=&r"(r[k + 5]), "=&r"(r[k + 6]), "=&r"(r[k + 7])
// 32 columns
__device__ __forceinline__ void tmem_get32(uint32_t t, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : LA_OUT8(a, 0), LA_OUT8(a, 8), LA_OUT8(b, 0), LA_OUT8(b, 8)
        : "r"(t)
        : "memory");
}
// 16 columns at each of two places
__device__ __forceinline__ void tmem_get16x2(uint32_t t, uint32_t u, uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%32];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%33];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : LA_OUT8(a, 0), LA_OUT8(a, 8), LA_OUT8(b, 0), LA_OUT8(b, 8)
        : "r"(t), "r"(u)
        : "memory");
}
// 8 columns at each of two places
__device__ __forceinline__ void tmem_get8x2(uint32_t t, uint32_t u, uint32_t (&a)[8], uint32_t (&b)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : LA_OUT8(a, 0), LA_OUT8(b, 0)
        : "r"(t), "r"(u)
        : "memory");
}
__device__ __forceinline__ void tmem_get8(uint32_t t, uint32_t (&a)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : LA_OUT8(a, 0)
        : "r"(t)
        : "memory");
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
// two products, sums or both in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 asf2(uint32_t a, uint32_t b) { return make_float2(__uint_as_float(a), __uint_as_float(b)); }
// A wait tests a barrier's parity, so it is right only if the completion before the one waited
// for has happened (else it passes too early) and the one after it cannot happen yet (else it is
// missed).  The first holds because a role waits for every completion of a barrier in turn, or
// has waited for what needs the earlier one (a tile's place is free once its products have read
// it); the second because what completes a barrier again needs an arrival, or a tile's place, that
// the waiter gives afterwards.  The V' warps do not follow a, v and the scores from chunk to
// chunk, so for the one chunk whose tiles they touch they have a barrier of its own, `taken`.
struct Bars {
    uint64_t a_full[2], k_full[2], v_full[2];   // tiles loaded
    uint64_t a_free[2], k_free[2], v_free[2];   // tiles read by their last product
    uint64_t sc, kv[2], as, o;                  // products done: scores; K^T V' (halves of the tokens); A S; P V
    uint64_t p, vp[2], s;                       // operands written: P, V' (halves), S
    uint64_t kv_read, o_read;                   // results fetched from tensor memory
    uint64_t o_tile[2];                         // the output in shared memory, or stored
    uint64_t taken, fixed;                      // one chunk of a walk at most: its tiles have come and its scores have
                                                // read them; its rows of other tokens are zeros
    uint64_t end[2];
    uint32_t tslot;
    int failed;
};
static_assert(sizeof(Bars) <= 256, "barrier space");

// Bounded wait for the completion number `n` (from 0) of a barrier; false when it does not
// come, and every role that waits for one that has given up gives up too, the block's error
// raised at its end.  The hint lets the hardware keep the thread suspended between polls.
// A role's waits poll as often as the call says (at most POLLS times, ssm_scan_set_wait_limit);
// those for a warp's own copies and products, at its end, always POLLS times.
constexpr uint32_t POLL_NS = 20000, POLLS = 1u << 15;   // about half a second
__device__ __forceinline__ bool await(uint64_t *bar, uint32_t n, uint32_t polls) {
    const uint32_t a = smem_u32(bar);
#pragma unroll 1
    for (uint32_t i = 0; i < polls; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok)
            : "r"(a), "r"(n & 1u), "r"(POLL_NS)
            : "memory");
        if (ok) return true;
    }
    return false;
}
// The same for a whole warp, all lanes alike.
__device__ __forceinline__ bool await_warp(uint64_t *bar, uint32_t n, uint32_t polls) {
    return __all_sync(0xffffffffu, await(bar, n, polls));
}
// One arrival a warp, after all its lanes are done.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The walk of a block.  STATE: only the state (no scores, no output).  REV: reverse.  OUT: the
// output is bf16 (0) or fp32 (1).
template <bool STATE, bool REV, int OUT>
__device__ __forceinline__ void walk(const Args &A, const Maps &maps, const LaWalk &w, int wi, int slice, int bh, int sg,
                                     unsigned char *sm) {
    const LaArgs &p = A.p;
    const int c0 = 64 * slice, BH = p.B * p.H;
    const int b = bh / p.H, h = bh - b * p.H;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
    const int first = sg * A.G, nch = min(A.G, (len + C - 1) / C - first);   // chunks; may be <= 0
    float *f32 = reinterpret_cast<float *>(sm + SM_F32);
    Bars *B = reinterpret_cast<Bars *>(sm + SM_BAR);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t polls = A.polls;
    // chunk number c of the walk: its first token and its tokens
    auto chunk = [&](int c) { return C * (first + (REV ? nch - 1 - c : c)); };
    // the chunk that the sequence ends in, if it is a short one, and its tokens
    const bool ends = nch > 0 && (first + nch) * C > len;
    const int ragged = ends ? (REV ? 0 : nch - 1) : -1, rest = len - C * (first + nch - 1);
    auto ntok = [&](int c) { return c == ragged ? rest : C; };
    // the chunk, if any, whose tiles hold rows of other tokens (TMA fills those past L with zeros)
    const int shared = len < p.L ? ragged : -1;
    auto dirty = [&](int c) { return c == shared; };
    const int nboxa = (w.da + 63) / 64, ha = h / w.rep_a, hk = h / w.rep_k, hv = h / w.rep_v;
    auto load_k = [&](int c) {
        unsigned char *st = sm + (c & 1) * STAGE + ST_K;
        mbar_expect_tx(&B->k_full[c & 1], 2 * TILE);
        tma_load_4d(st, &maps.k, &B->k_full[c & 1], 0, hk, chunk(c), b);
        // a second box past the head is zeros: state rows that are not there
        tma_load_4d(st + TILE, &maps.k, &B->k_full[c & 1], 64, hk, chunk(c), b);
    };
    auto load_a = [&](int c) {
        mbar_expect_tx(&B->a_full[c & 1], TILE * nboxa);
        for (int i = 0; i < nboxa; ++i)
            tma_load_4d(sm + (c & 1) * STAGE + ST_A + i * TILE, &maps.a, &B->a_full[c & 1], 64 * i, ha, chunk(c), b);
    };
    auto load_v = [&](int c) {
        mbar_expect_tx(&B->v_full[c & 1], TILE);
        tma_load_4d(sm + (c & 1) * STAGE + ST_V, &maps.v, &B->v_full[c & 1], c0, hv, chunk(c), b);
    };
    {   // powers of lam from its logarithm in 64 bits: every one right to half a step
        double g = (double)p.log_decay[h];
        if (g < -1e6) g = -1e6;   // -inf: lam^0 stays 1
        const double rw = (double)w.read * (double)w.write;
        if (tid < 129 + 160 + 64) {
            const int m = tid < 129 ? tid : tid < 289 ? tid - 161 : tid < 321 ? tid - 289 : 352 - tid;
            const double e = exp(g * m);
            f32[tid < 129 ? F_PW + tid : tid < 289 ? F_W + tid - 129 : tid < 321 ? F_UP + tid - 289 : F_DOWN + tid - 321] =
                m < 0 ? 0.f : (float)(tid >= 129 && tid < 289 ? rw * e : e);
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = B->tslot;
    // a role that leaves its loop early says so
    auto over = [&](bool all) {
        if (!all) B->failed = 1;
    };
    const uint32_t lane_q = (uint32_t)(32 * (warp & 3)) << 16;
    const int row = 32 * (warp & 3) + lane;      // token, or state row, of the thread

    if (warp == 0) {
        if (lane == 0) {
            uint32_t got_a = 0, got_k = 0, got_v = 0;   // loads issued
            int c = 0;
#pragma unroll 1
            for (; c < nch; ++c) {
                const uint32_t n = (uint32_t)(c >> 1) - 1u;
                if (c + 2 < nch) {   // what comes into these slots next, on its way into L2
                    const int tn = chunk(c + 2);
#pragma unroll 1
                    for (int i = 0; i < nboxa; ++i) {
                        tma_prefetch_4d(&maps.k, 64 * i, hk, tn, b);
                        if (!STATE) tma_prefetch_4d(&maps.a, 64 * i, ha, tn, b);
                    }
                    tma_prefetch_4d(&maps.v, c0, hv, tn, b);
                }
                if (c >= 2 && !await(&B->k_free[c & 1], n, polls)) break;
                load_k(c);
                ++got_k;
                if (STATE) continue;
                if (c >= 2 && !await(&B->a_free[c & 1], n, polls)) break;
                load_a(c);
                ++got_a;
                if (c >= 2 && !await(&B->v_free[c & 1], n, polls)) break;
                load_v(c);
                ++got_v;
            }
            over(c >= nch);
            // no copy is in flight when the block ends
#pragma unroll 1
            for (uint32_t i = 0; i < 6; ++i) {
                const uint32_t got = i < 2 ? got_a : i < 4 ? got_k : got_v, back = 1 + (i & 1);
                uint64_t *full = i < 2 ? B->a_full : i < 4 ? B->k_full : B->v_full;
                if (got >= back) await(&full[(got - back) & 1], (got - back) >> 1, POLLS);
            }
        }
        __syncwarp();
    } else if (warp == 1 || (!STATE && warp == 3)) {
        if (elect_one()) {
            constexpr uint32_t id_sc = idesc_bf16(128, 128, false, false), id_n = idesc_bf16(128, 64, false, true);
            constexpr uint32_t id_kv = idesc_bf16(128, 192, true, true);
            // descriptors: their address field counts 16-byte units; along a row, 16 values are 2 of them
            const uint32_t u0 = smem_u32(sm) >> 4;
            constexpr uint32_t HALF = TILE >> 4, STEP = 2048 >> 4;   // the next 64 values of the rows; the next 16 rows
            auto kmaj = [](uint32_t u, int s) { return desc<16u>(u + s * 2u); };
            auto mnmaj = [](uint32_t u, int s) { return desc<TILE>(u + STEP * s); };
            int c = 0;
            if (warp == 1) {   // K^T V', the smallest part of V' in the last columns
#pragma unroll 1
                for (; c < nch; ++c) {
                    const uint32_t st = u0 + ((c & 1) ? STAGE >> 4 : 0u);
                    if (!await(&B->k_full[c & 1], (uint32_t)c >> 1, polls)) break;
                    if (c > 0 && !await(&B->kv_read, (uint32_t)c - 1u, polls)) break;
                    int z = 0;
#pragma unroll 1
                    for (; z < 2; ++z) {
                        if (!await(&B->vp[z], (uint32_t)c, polls)) break;
                        fence_after_sync();
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_bf16(tm + TM_KV, mnmaj(st + (ST_K >> 4) + 4 * STEP * z, s), mnmaj(u0 + (SM_VP >> 4) + 4 * STEP * z, s),
                                     id_kv, s > 0 || z > 0);
                        mma_commit(&B->kv[z]);
                    }
                    if (z < 2) break;
                    mma_commit(&B->k_free[c & 1]);
                }
            } else {
                // a chunk's product over the head dimension, 64 values at a time (heads padded with the
                // tiles' zeros): rolled to one MMA the loop took 130 cycles an MMA, and all of them
                // in a row are more code than the fetch keeps up with
                auto over_head = [&](uint32_t d, uint32_t a, uint32_t bb, uint32_t id, bool kb) {
#pragma unroll 1
                    for (int q = 0; q < nboxa; ++q)
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            mma_bf16(d, kmaj(a + HALF * q, s), kb ? kmaj(bb + HALF * q, s) : mnmaj(bb + 4 * STEP * q, s), id, s > 0 || q > 0);
                };
#pragma unroll 1
                for (c = -1; c < nch; ++c) {
                    const uint32_t st = u0 + ((c & 1) ? STAGE >> 4 : 0u);
                    if (c >= 0) {
                        if (!await(&B->s, (uint32_t)c, polls)) break;
                        if (c > 0 && !await(&B->o_read, (uint32_t)c - 1u, polls)) break;
                        fence_after_sync();
                        over_head(tm + TM_OS, st + (ST_A >> 4), u0 + (SM_S >> 4), id_n, false);
                        mma_commit(&B->as);
                        if (OUT == 0) mma_commit(&B->a_free[c & 1]);   // else warp 2, when the output has left the tile
                        if (!await(&B->v_full[c & 1], (uint32_t)c >> 1, polls) || !await(&B->p, (uint32_t)c, polls)) break;
                        if (dirty(c)) {   // P is there, so the scores are done
                            mbar_arrive(&B->taken);
                            if (!await(&B->fixed, 0u, polls)) break;
                        }
                        fence_after_sync();
#pragma unroll 1
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int s = 0; s < 4; ++s)
                                mma_bf16_ts(tm + TM_OI, tm + TM_P + 32u * q + 8u * s, mnmaj(st + (ST_V >> 4) + 4 * STEP * q, s), id_n, s > 0 || q > 0);
                        mma_commit(&B->o);
                        if (OUT == 1) mma_commit(&B->v_free[c & 1]);
                    }
                    if (c + 1 < nch) {   // the scores of the next chunk; P's warps have fetched this one's
                        const uint32_t sn = u0 + ((c & 1) ? 0u : STAGE >> 4), n = (uint32_t)(c + 1) >> 1;
                        if (!await(&B->k_full[(c + 1) & 1], n, polls) || !await(&B->a_full[(c + 1) & 1], n, polls)) break;
                        fence_after_sync();
                        over_head(tm + TM_SC, sn + (ST_A >> 4), sn + (ST_K >> 4), id_sc, true);
                        mma_commit(&B->sc);
                        mma_commit(&B->k_free[(c + 1) & 1]);
                    }
                }
            }
            over(c >= nch);
            uint64_t *end = &B->end[warp >> 1];
            mma_commit(end);   // every MMA is over before tensor memory goes
            await(end, 0u, POLLS);
        }
        __syncwarp();
    } else if (!STATE && warp == 2) {
        if (lane == 0) {
            int c = 0;
#pragma unroll 1
            for (; c < nch; ++c) {
                const int t0 = chunk(c);
                if (!await(&B->o_tile[c & 1], (uint32_t)c >> 1, polls)) break;
                // what is past L or the head is not written
                if (OUT == 1) {   // (rows behind the sequence hold nothing that is read)
                    const unsigned char *at = sm + (c & 1) * STAGE + ST_A;
                    tma_store_4d(&maps.o, at, c0, h, t0, b);
                    if (c0 + 32 < w.dc) tma_store_4d(&maps.o, at + TILE, c0 + 32, h, t0, b);
                } else if (!dirty(c)) {
                    tma_store_4d(&maps.o, sm + (c & 1) * STAGE + ST_V, c0, h, t0, b);
                }
                bulk_commit();
                bulk_wait_read_all();
                mbar_arrive(OUT == 1 ? &B->a_free[c & 1] : &B->v_free[c & 1]);
            }
            over(c >= nch);
        }
        __syncwarp();
    } else if (!STATE && warp >= 4 && warp < 12) {
        const int half = (warp - 4) >> 2, qd = warp & 3;
        const long long ob = b * w.so[0] + h * w.so[2] + c0 + 32 * half;
        const int nq = min(4, (w.dc - c0 - 32 * half) / 8);   // 8-column pieces of the output (<= 0: none)
        int c = 0;
#pragma unroll 1
        for (; c < nch; ++c) {
            const int t0 = chunk(c), n = ntok(c);
            if (!await_warp(&B->sc, (uint32_t)c, polls)) break;
            fence_after_sync();
            // P[i][j] = read write lam^{|i - j|} (a_i . k_j) on one side of the diagonal, 32 columns
            // at a time
#pragma unroll 1
            for (int z = 0; z < 2; ++z) {
                const int jb = 2 * half + z;
                uint32_t o[16];
                const bool zero = REV ? jb < qd : jb > qd;   // masked
                uint32_t x[16], y[16];
                if (!zero) {
                    tmem_get32(tm + TM_SC + lane_q + 32u * jb, x, y);
                }
                if (zero) {
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = 0u;
                } else if (jb == qd) {   // the diagonal
                    const int d = REV ? 1 : -1;
                    const float *wv = f32 + F_W + 32 + (REV ? 32 * jb - row : row - 32 * jb);
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        const float2 e = mul2(u < 8 ? asf2(x[2 * u], x[2 * u + 1]) : asf2(y[2 * u - 16], y[2 * u - 15]),
                                              make_float2(wv[0], wv[d]));
                        wv += 2 * d;
                        o[u] = pack2(e.x, e.y);
                    }
                } else {   // off it the weight is a factor of the row times one of the column
                    const float r = f32[F_W + 32 + (REV ? 32 * jb - row : row - 32 * jb - 31)];
                    const float4 *cw = reinterpret_cast<const float4 *>(f32 + (REV ? F_UP : F_DOWN));
                    const float2 rr = make_float2(r, r);
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const float4 f = cw[u];
                        const uint32_t *s4 = u < 4 ? x + 4 * u : y + 4 * (u - 4);
                        const float2 e0 = mul2(mul2(asf2(s4[0], s4[1]), rr), make_float2(f.x, f.y));
                        const float2 e1 = mul2(mul2(asf2(s4[2], s4[3]), rr), make_float2(f.z, f.w));
                        o[2 * u] = pack2(e0.x, e0.y);
                        o[2 * u + 1] = pack2(e1.x, e1.y);
                    }
                }
                const int left = n - 32 * jb;   // columns of this sequence
                if (__builtin_expect(left < 32, 0)) {   // tokens past it do not count, whatever they hold
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[u] = 2 * u + 1 < left ? o[u] : 2 * u < left ? o[u] & 0xffffu : 0u;
                }
                tmem_st16(tm + TM_P + lane_q + 16u * jb, o);
            }
            tmem_wait_st();
            fence_before_sync();
            warp_arrive(&B->p);
            if (!await_warp(&B->o, (uint32_t)c, polls)) break;
            fence_after_sync();
            const float e = w.read * f32[F_PW + max(0, REV ? n - 1 - row : row + 1)];
            const float2 ee = make_float2(e, e);
            // 16 columns at a time: over the chunk's V tile (fp32: its A tiles), from where warp 2 stores
            // whole chunks, or, where rows behind the sequence must stay as they are, straight to memory
            const bool tile = OUT == 0 && !dirty(c);
            unsigned char *vt = sm + (c & 1) * STAGE + ST_V + row * 128;
            unsigned char *at32 = sm + (c & 1) * STAGE + ST_A + half * TILE + row * 128;
            const long long at = ob + (long long)(t0 + row) * w.so[1];
#pragma unroll 1
            for (int z = 0; z < 2; ++z) {
                uint32_t x[16], u[16];
                tmem_get16x2(tm + TM_OI + lane_q + 32u * half + 16u * z, tm + TM_OS + lane_q + 32u * half + 16u * z, x, u);
                float2 o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fma2(ee, asf2(u[2 * j], u[2 * j + 1]), asf2(x[2 * j], x[2 * j + 1]));
                if (OUT == 1) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<float4 *>(at32 + (((4 * z + q) ^ (row & 7)) << 4)) =
                            make_float4(o[2 * q].x, o[2 * q].y, o[2 * q + 1].x, o[2 * q + 1].y);
                    continue;
                }
                const uint4 r0 = make_uint4(pack2(o[0].x, o[0].y), pack2(o[1].x, o[1].y), pack2(o[2].x, o[2].y), pack2(o[3].x, o[3].y));
                const uint4 r1 = make_uint4(pack2(o[4].x, o[4].y), pack2(o[5].x, o[5].y), pack2(o[6].x, o[6].y), pack2(o[7].x, o[7].y));
                if (__builtin_expect(tile, 1)) {
                    const int q = 4 * half + 2 * z;
                    *reinterpret_cast<uint4 *>(vt + ((q ^ (row & 7)) << 4)) = r0;
                    *reinterpret_cast<uint4 *>(vt + (((q + 1) ^ (row & 7)) << 4)) = r1;
                } else if (row < n) {
                    uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(w.o) + at) + 2 * z;
                    if (nq > 2 * z) dst[0] = r0;
                    if (nq > 2 * z + 1) dst[1] = r1;
                }
            }
            fence_before_sync();
            warp_arrive(&B->o_read);
            fence_proxy_async();
            warp_arrive(&B->o_tile[c & 1]);
        }
        over(c >= nch);
    } else if (warp >= 20) {
        // V' = write lam^.. v, from memory by way of registers a chunk ahead: it does not wait
        // for a free V tile, nor hold one.  A thread takes 8 columns of two rows of each half.
        const int t = tid - 640, col = 8 * (t & 7);
        const float2 minus = make_float2(-1.f, -1.f);
        // the rows of each half have registers of their own: a move would wait for the load
        const bool mine = c0 + col < w.dc;
        const long long by = 64 * w.sv[1];   // bytes from a row to the 32nd after it
        const char *vg = reinterpret_cast<const char *>(reinterpret_cast<const __nv_bfloat16 *>(w.v) + b * w.sv[0] + hv * w.sv[2] +
                                                        c0 + col + (long long)(chunk(0) + (t >> 3)) * w.sv[1]);
        uint4 cur[2], lo[2] = {}, hi[2] = {};
        int hh = -2;
#pragma unroll 1
        for (; hh < 2 * nch; ++hh) {
            const int c = hh >> 1, z = hh & 1, live = c + 1 < nch && mine ? ntok(c + 1) - (t >> 3) : 0;   // rows of the next chunk
            if (z == 0) {
                cur[0] = lo[0];
                cur[1] = lo[1];
                lo[0] = ld_once(vg, live > 0);
                lo[1] = ld_once(vg + by, live > 32);
            } else {
                cur[0] = hi[0];
                cur[1] = hi[1];
                hi[0] = ld_once(vg + 2 * by, live > 64);
                hi[1] = ld_once(vg + 3 * by, live > 96);
                vg += REV ? -4 * by : 4 * by;
            }
            if (c < 0) continue;
            unsigned char *st = sm + (c & 1) * STAGE;
            const int n = ntok(c);
            const bool fix = dirty(c);
            if (__builtin_expect(fix, 0)) {
                // behind `taken` the tiles are the chunk's and stay so until they are fixed; a walk of
                // the state alone has waited for K^T V' of two chunks ago, the last reader of K's place
                if (!STATE && !await_warp(&B->taken, 0u, polls)) break;
                if (!await_warp(&B->k_full[c & 1], (uint32_t)c >> 1, polls)) break;
                if (!STATE && !await_warp(&B->v_full[c & 1], (uint32_t)c >> 1, polls)) break;
            }
            if (c > 0 && !await_warp(&B->kv[z], (uint32_t)c - 1u, polls)) break;   // this half has been read
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                const int r = (t >> 3) + 64 * z + 32 * i;
                const uint32_t off = (uint32_t)r * 128u + (uint32_t)((col / 8) ^ (r & 7)) * 16u;
                const uint4 x = cur[0];
                cur[0] = cur[1];
                if (__builtin_expect(fix && r >= n, 0)) {
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                    if (!STATE) *reinterpret_cast<uint4 *>(st + ST_V + off) = zero;
                    *reinterpret_cast<uint4 *>(st + ST_K + off) = zero;
                    *reinterpret_cast<uint4 *>(st + ST_K + TILE + off) = zero;
                }
                const float f = w.write * f32[F_PW + (REV ? r + 1 : max(0, n - 1 - r))];
                const float2 ff = make_float2(f, f);
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                uint32_t o[3][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 a = mul2(make_float2(lo_f(u[k]), hi_f(u[k])), ff);
#pragma unroll
                    for (int q = 0; q < 3; ++q) {
                        o[q][k] = high2(a.x, a.y);
                        a = fma2(make_float2(hi_f(__float_as_uint(a.x)), hi_f(__float_as_uint(a.y))), minus, a);
                    }
                }
#pragma unroll
                for (int q = 0; q < 3; ++q)
                    *reinterpret_cast<uint4 *>(sm + SM_VP + q * TILE + off) = make_uint4(o[q][0], o[q][1], o[q][2], o[q][3]);
            }
            fence_proxy_async();
            warp_arrive(&B->vp[z]);
            if (__builtin_expect(fix && z == 1, 0)) warp_arrive(&B->fixed);
        }
        over(hh >= 2 * nch);
    } else if (warp >= 12) {
        float2 S[16];
        const int half = (warp - 12) >> 2, col = c0 + 32 * half;   // the thread's first column
        const bool seg = A.nseg > 1;
        // where the state comes from and goes to: the caller's, or the segment's slot (a segment
        // that only adds starts from zero; the states that leave are k_la_segments' work)
        float *slot = seg ? A.seg[wi] + ((long long)sg * BH + bh) * w.da * w.dc : nullptr;
        const long long outside = (long long)bh * w.da * w.dc;
        const float *src = seg ? (STATE ? nullptr : slot) : w.s_in ? w.s_in + outside : nullptr;
        float *dst = seg ? (STATE ? slot : nullptr) : w.s_out ? w.s_out + outside : nullptr;
        const int stc = seg ? 1 : w.st_c, cols = row < w.da ? w.dc - col : 0;
        const long long at = (long long)row * (seg ? w.dc : w.st_a) + (long long)col * stc;
        // Where a row of the state lies along its columns, a warp's 32 rows pass, 16 columns at a time,
        // through 2 KB of the operand's place, so that memory is read and written in whole sectors
        // (a thread with a row of its own took 5 us for a head of 128 x 128); transposed, the lanes
        // are neighbours already.
        float *tile = reinterpret_cast<float *>(sm + SM_S) + 512 * (warp - 12);
        auto place = [&](int r, int q) { return tile + 16 * r + ((q ^ ((r >> 1) & 3)) << 2); };   // 4 columns q of row r
        const int sub = lane >> 4, sc = lane & 15;   // a lane's row of two, and its column
        const int rs = seg ? w.dc : w.st_a, rows0 = (row - lane + sub) * rs + col + sc;
        const int dense_rows = w.da - (row - lane) - sub;   // of the lane's rows, those of the state
        if (!src) {
#pragma unroll
            for (int i = 0; i < 16; ++i) S[i] = make_float2(0.f, 0.f);
        } else if (stc == 1) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const float *q = src + rows0 + 16 * z;
                const bool mine = col + 16 * z + sc < w.dc;
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 16) {
                    float x[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) x[r] = mine && r0 + 2 * r < dense_rows ? q[(r0 + 2 * r) * rs] : 0.f;
#pragma unroll
                    for (int r = 0; r < 8; ++r) place(r0 + 2 * r + sub, sc >> 2)[sc & 3] = x[r];
                }
                __syncwarp();
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const float4 v = *reinterpret_cast<const float4 *>(place(lane, q4));
                    S[8 * z + 2 * q4] = make_float2(v.x, v.y);
                    S[8 * z + 2 * q4 + 1] = make_float2(v.z, v.w);
                }
                __syncwarp();
            }
            asm volatile("bar.sync 8, 256;\n" ::: "memory");   // the operand may be written
        } else {
            const float *q = src + at;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                S[i].x = 2 * i < cols ? q[2 * i * stc] : 0.f;
                S[i].y = 2 * i + 1 < cols ? q[(2 * i + 1) * stc] : 0.f;
            }
        }
        int c = 0;
#pragma unroll 1
        for (; c < nch; ++c) {
            if (!STATE) {   // S in bf16, the layout of a V tile; A S of the chunk before has read it
                if (c > 0 && !await_warp(&B->as, (uint32_t)c - 1u, polls)) break;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint4 v = make_uint4(pack2(S[4 * q].x, S[4 * q].y), pack2(S[4 * q + 1].x, S[4 * q + 1].y),
                                               pack2(S[4 * q + 2].x, S[4 * q + 2].y), pack2(S[4 * q + 3].x, S[4 * q + 3].y));
                    *reinterpret_cast<uint4 *>(sm + SM_S + row * 128 + (((q + 4 * half) ^ (row & 7)) << 4)) = v;
                }
                fence_proxy_async();
                warp_arrive(&B->s);
            }
            const float E = f32[F_PW + ntok(c)];
            const float2 EE = make_float2(E, E);
            const uint32_t tk = tm + TM_KV + lane_q + 32u * half;
            if (!await_warp(&B->kv[1], (uint32_t)c, polls)) break;
            fence_after_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t x[8], y[8];
                tmem_get8x2(tk + 64u + 8u * q, tk + 128u + 8u * q, x, y);
                float2 small[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) small[k] = add2(asf2(x[2 * k], x[2 * k + 1]), asf2(y[2 * k], y[2 * k + 1]));
                tmem_get8(tk + 8u * q, x);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    S[4 * q + k] = fma2(EE, S[4 * q + k], add2(asf2(x[2 * k], x[2 * k + 1]), small[k]));
            }
            fence_before_sync();
            warp_arrive(&B->kv_read);
        }
        over(c >= nch);
        if (dst) {
            if (!STATE && c >= nch && nch > 0) await_warp(&B->as, (uint32_t)nch - 1u, polls);   // A S has read the operand
            if (stc == 1) {
#pragma unroll
                for (int z = 0; z < 2; ++z) {
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        *reinterpret_cast<float4 *>(place(lane, q4)) =
                            make_float4(S[8 * z + 2 * q4].x, S[8 * z + 2 * q4].y, S[8 * z + 2 * q4 + 1].x, S[8 * z + 2 * q4 + 1].y);
                    __syncwarp();
                    float *q = dst + rows0 + 16 * z;
                    if (col + 16 * z + sc < w.dc)
#pragma unroll 1
                        for (int r = 0; r < min(32, dense_rows); r += 2) q[r * rs] = place(r + sub, sc >> 2)[sc & 3];
                    __syncwarp();
                }
            } else {
                float *q = dst + at;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (2 * i < cols) q[2 * i * stc] = S[i].x;
                    if (2 * i + 1 < cols) q[(2 * i + 1) * stc] = S[i].y;
                }
            }
        }
    }
}

template <bool STATE>
__global__ void __launch_bounds__(THREADS, 1)
k_la_walk(const __grid_constant__ Maps m0, const __grid_constant__ Maps m1,
          const __grid_constant__ Maps m2, const __grid_constant__ Args A) {
    const int BH = A.p.B * A.p.H;
    int id = blockIdx.x;
    const int slice = id % A.slices;
    id /= A.slices;
    const int bh = id % BH;
    id /= BH;
    const int sg = id % A.nseg, wi = id / A.nseg;
    const LaWalk w = A.p.w[wi];   // by value: with the index unknown, every use would load from memory
    const Maps &maps = wi == 0 ? m0 : wi == 1 ? m1 : m2;
    if (64 * slice >= w.dc) return;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *B = reinterpret_cast<Bars *>(sm + SM_BAR);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i)
            for (uint64_t *q : {&B->a_full[i], &B->k_full[i], &B->v_full[i], &B->a_free[i], &B->k_free[i], &B->v_free[i]})
                mbar_init(q, q == &B->k_free[i] && !STATE ? 2 : 1);   // K has two readers
        for (uint64_t *q : {&B->sc, &B->kv[0], &B->kv[1], &B->as, &B->o, &B->taken, &B->end[0], &B->end[1]}) mbar_init(q, 1);
        // an arrival a warp
        for (uint64_t *q : {&B->vp[0], &B->vp[1], &B->s, &B->kv_read, &B->fixed, &B->p, &B->o_read, &B->o_tile[0], &B->o_tile[1]}) mbar_init(q, 8);
        B->failed = 0;
        mbar_fence_init();
    }
    if (threadIdx.x / 32 == 1) tmem_alloc(&B->tslot, TM_COLS);
    if (STATE || !w.o_f32)
        w.rev ? walk<STATE, true, 0>(A, maps, w, wi, slice, bh, sg, sm) : walk<STATE, false, 0>(A, maps, w, wi, slice, bh, sg, sm);
    else
        w.rev ? walk<STATE, true, 1>(A, maps, w, wi, slice, bh, sg, sm) : walk<STATE, false, 1>(A, maps, w, wi, slice, bh, sg, sm);
    fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && B->failed) atomicCAS(&ssm_la_error_word, 0, 1);
    if (threadIdx.x / 32 == 1) {
        fence_after_sync();
        tmem_dealloc(B->tslot, TM_COLS);
    }
}

// The state entering every segment, in place of what the segment adds, and the state that
// leaves the walk: a thread an element, the segments in the walk's order, eight loads at a time.
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
    const long long step = (long long)BH * w.da * w.dc;
    float *slot = A.seg[blockIdx.y] + at + e;
    float E = w.s_in ? w.s_in[ext] : 0.f;
    const float whole = (float)exp(g * (A.G * C));   // the decay of a whole segment
    for (int i0 = 0; i0 < A.nseg; i0 += 8) {
        float add[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int s = w.rev ? A.nseg - 1 - i0 - k : i0 + k;
            add[k] = i0 + k < A.nseg ? slot[s * step] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + k >= A.nseg) break;
            const int s = w.rev ? A.nseg - 1 - i0 - k : i0 + k;
            const int n = min(max(len - s * A.G * C, 0), A.G * C);   // its tokens
            slot[s * step] = E;
            E = fmaf(n == A.G * C ? whole : (float)exp(g * n), E, add[k]);
        }
    }
    if (w.s_out) w.s_out[ext] = E;
}

// bf16, boxes of 64 values, or fp32, boxes of 32: 128 bytes either way
bool make_map(CUtensorMap *m, const void *base, int d, int heads, const LaArgs &p, const long long *s, bool f32 = false) {
    chunkc::EncodeTiledFn fn = chunkc::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)p.L, (cuuint64_t)p.B};
    // the stride of a dimension of one is not used, and need not be a valid one
    const int e = f32 ? 4 : 2;
    cuuint64_t st[3] = {(cuuint64_t)(heads > 1 ? s[2] * e : 16), (cuuint64_t)(p.L > 1 ? s[1] * e : 16),
                        (cuuint64_t)(p.B > 1 ? s[0] * e : 16)};
    cuuint32_t box[4] = {(cuuint32_t)(128 / e), 1, C, 1}, es[4] = {1, 1, 1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, st, box, es,
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
// the shortest estimate, in chunks of a walk (about 2.5 us): a block takes 3 to begin and end,
// a chunk whose state alone is walked 0.7, the pass over the segments' states and its launch
// 3, and a block an SM runs at a time.
int la_segments(long long L, long long items) {
    const long long nc = (L + la::C - 1) / la::C;
    double best = 0;
    int pick = 1;
    for (long long n = 1; n <= nc && n <= 64; ++n) {
        const long long g = (nc + n - 1) / n, seg = (nc + g - 1) / g, waves = (items * seg + SMS - 1) / SMS;
        const double t = waves * (g + 3.0) + (seg > 1 ? waves * (0.7 * g + 3.0) + 3.0 : 0.0);
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
    const long long limit = abi_wait_limit();
    A.polls = limit < POLLS ? (uint32_t)limit : POLLS;
    for (int i = 0; i < p.nwalk; ++i) {
        const LaWalk &w = p.w[i];
        auto ok = [](const void *q, const long long *s, int el) {
            return ((uintptr_t)q & 15) == 0 && s[0] % el == 0 && s[1] % el == 0 && s[2] % el == 0;
        };
        if (!la_chunked_sizes(p.bf16, w.da, w.dc) || !ok(w.a, w.sa, 8) || !ok(w.k, w.sk, 8) ||
            !ok(w.v, w.sv, 8) || (w.o && !ok(w.o, w.so, w.o_f32 ? 4 : 8)))
            return false;
        m[i].o = CUtensorMap{};
        if (w.o && !make_map(&m[i].o, w.o, w.dc, p.H, p, w.so, w.o_f32)) return false;
        if (!make_map(&m[i].a, w.a, w.da, p.H / w.rep_a, p, w.sa) ||
            !make_map(&m[i].k, w.k, w.da, p.H / w.rep_k, p, w.sk) ||
            !make_map(&m[i].v, w.v, w.dc, p.H / w.rep_v, p, w.sv))
            return false;
        const int sl = (w.dc + 63) / 64;
        A.slices = sl > A.slices ? sl : A.slices;
        A.seg[i] = seg[i];
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
