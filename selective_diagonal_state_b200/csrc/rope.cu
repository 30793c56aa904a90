// Rotary positions of queries and keys, and the gradient through them (the opposite
// rotation): pair j of every head at position m turns by m freq[j],
//     (a, b) -> magnitude (a cos - b sin, a sin + b cos).
// The angle is taken in 64 bits, in half turns, and reduced to (-1, 1] there, so that
// sincospi of its fp32 rest is right for any position.  Bound by memory, each value read and
// written once, as long as the rest is kept small: the 64-bit steps of an angle are taken
// once a block, a thread keeps a piece's sines and its addresses for up to eight heads, and has
// four of them on their way.  On one B200, 65536 tokens of 32 heads of 128 (bf16, all
// of a head turned): 165 us, 6.5 TB/s; with two heads on their way 173, with four heads a
// thread 211, with the angles taken by every thread that needs them 190.
#include "common.cuh"
#include "layer.h"

namespace ssm {
namespace {

struct RopeArgs {
    const void *q, *k;
    void *qo, *ko;
    const double *freq;
    const int64_t *pos;
    long long sq[3], sk[3], sqo[3], sko[3], sp[2];
    long long tokens;   // batch * seqlen
    int L, hq, hk, dim, rot;
    int units;          // pieces a token: rotated ones, then copied ones
    int urot, share;    // rotated pieces; threads that share the heads of a piece
    int per_block;      // tokens of a block
    int pairs;          // layout (2 i, 2 i + 1)
    float mag, sign;
};

__device__ __forceinline__ void turn(double angle_halfturns, float mag, float sign, float &c,
                                     float &s) {
    const double r = angle_halfturns - 2.0 * rint(angle_halfturns * 0.5);
    float sn, cs;
    sincospif((float)r, &sn, &cs);
    c = mag * cs;
    s = mag * sign * sn;
}

constexpr int TURNS = 4096;   // pairs whose sines a block may hold
constexpr int EACH = 8;       // heads a thread turns at most
constexpr int NB = 4;         // of which it has so many on their way at once
constexpr double INV_PI = 0.31830988618379067154;

template <bool BF16> __device__ __forceinline__ void unpack(const uint4 &w, float *v) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        } else {
            v[i] = __uint_as_float(u[i]);
        }
    }
}
template <bool BF16> __device__ __forceinline__ uint4 pack(const float *v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&r);
        } else {
            u[i] = __float_as_uint(v[i]);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// Pieces of N values (16 bytes): dense and 16-byte aligned heads.  A block takes p.per_block
// tokens: its threads first take the sines of all their pairs, one each, into shared
// memory, then turn the pieces, a thread the same piece of some of the token's heads.
template <bool BF16, bool PAIRS>
__global__ void __launch_bounds__(256) k_rope(const RopeArgs p) {
    constexpr int N = BF16 ? 8 : 4, ES = 16 / N, NP = PAIRS ? N / 2 : N;
    extern __shared__ float2 turns[];   // [token of the block][pair] (cosine, sine)
    const int tid = threadIdx.x, np = p.rot / 2;
    const long long t0 = (long long)blockIdx.x * p.per_block, b0 = t0 / p.L;
    const uint32_t first = (uint32_t)(t0 - b0 * p.L);   // the block's first token in its batch row
    const int nt = (int)min((long long)p.per_block, p.tokens - t0), items = nt * p.units * p.share;
    for (int i = tid; i < nt * np; i += 256) {
        const int l = i / np;
        const uint32_t at = first + l, rows = at / p.L, t = at - rows * p.L;
        const double m = p.pos ? (double)p.pos[(b0 + rows) * p.sp[0] + t * p.sp[1]] : (double)t;
        float2 w;
        turn(m * (p.freq[i - l * np] * INV_PI), p.mag, p.sign, w.x, w.y);
        turns[i] = w;
    }
    __syncthreads();
    for (int e = tid; e < items; e += 256) {
        const int u = e % p.units, r = e / p.units, tl = r / p.share;
        int h = r - tl * p.share;
        const uint32_t at = first + tl, rows = at / p.L, t = at - rows * p.L;
        const long long b = b0 + rows;
        const bool rotated = u < p.urot;
        const int e0 = rotated ? u * N : p.rot + (u - p.urot) * N;
        const int across = np * ES;   // bytes from a piece to its partner in the half layout
        float2 w[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) w[i] = rotated ? turns[tl * np + (PAIRS ? e0 / 2 : e0) + i] : make_float2(1.f, 0.f);
        // q's heads, then k's
#pragma unroll 1
        for (int op = 0; op < 2; ++op) {
            const int n = op ? p.hk : p.hq;
            const long long *si = op ? p.sk : p.sq, *so = op ? p.sko : p.sqo;
            const char *in = reinterpret_cast<const char *>(op ? p.k : p.q) + (b * si[0] + t * si[1] + h * si[2] + e0) * ES;
            char *out = reinterpret_cast<char *>(op ? p.ko : p.qo) + (b * so[0] + t * so[1] + h * so[2] + e0) * ES;
            const long long di = p.share * si[2] * ES, dn = p.share * so[2] * ES;
#pragma unroll 1
            for (; h < n; h += NB * p.share) {
                uint4 lo[NB], hi[NB];
#pragma unroll
                for (int i = 0; i < NB; ++i, in += di) {
                    if (h + i * p.share >= n) continue;
                    lo[i] = *reinterpret_cast<const uint4 *>(in);
                    if (!PAIRS && rotated) hi[i] = *reinterpret_cast<const uint4 *>(in + across);
                }
#pragma unroll
                for (int i = 0; i < NB; ++i, out += dn) {
                    if (h + i * p.share >= n) continue;
                    if (rotated) {
                        float x[N], y[N];
                        unpack<BF16>(lo[i], x);
                        if (PAIRS) {
#pragma unroll
                            for (int k = 0; k < NP; ++k) {
                                const float a = x[2 * k], c = x[2 * k + 1];
                                x[2 * k] = a * w[k].x - c * w[k].y;
                                x[2 * k + 1] = a * w[k].y + c * w[k].x;
                            }
                        } else {
                            unpack<BF16>(hi[i], y);
#pragma unroll
                            for (int k = 0; k < NP; ++k) {
                                const float a = x[k], c = y[k];
                                x[k] = a * w[k].x - c * w[k].y;
                                y[k] = a * w[k].y + c * w[k].x;
                            }
                            *reinterpret_cast<uint4 *>(out + across) = pack<BF16>(y);
                        }
                        lo[i] = pack<BF16>(x);
                    }
                    *reinterpret_cast<uint4 *>(out) = lo[i];
                }
            }
            h = (h - n) % p.share;   // k's heads go on where q's end
        }
    }
}

// Any alignment and width: a pair, or one copied value, a thread.
template <bool BF16>
__global__ void __launch_bounds__(256) k_rope_any(const RopeArgs p) {
    const long long id = blockIdx.x * 256ll + threadIdx.x;
    const long long tok = id / p.units;
    if (tok >= p.tokens) return;
    const int u = (int)(id - tok * p.units);
    const long long b = tok / p.L, t = tok - b * p.L;
    const bool rotated = u < p.urot;
    float c = 1.f, s = 0.f;
    if (rotated) {
        const double m = p.pos ? (double)p.pos[b * p.sp[0] + t * p.sp[1]] : (double)t;
        turn(m * (p.freq[u] * INV_PI), p.mag, p.sign, c, s);
    }
    const int e0 = !rotated ? p.rot + u - p.urot : p.pairs ? 2 * u : u;
    const int e1 = p.pairs ? e0 + 1 : e0 + p.rot / 2;
    for (int hh = 0; hh < p.hq + p.hk; ++hh) {
        const bool isk = hh >= p.hq;
        const int h = isk ? hh - p.hq : hh;
        const long long *si = isk ? p.sk : p.sq, *so = isk ? p.sko : p.sqo;
        const void *in = isk ? p.k : p.q;
        void *out = isk ? p.ko : p.qo;
        const long long i = b * si[0] + t * si[1] + h * si[2], o = b * so[0] + t * so[1] + h * so[2];
        const float x = ld_io(in, i + e0, BF16);
        if (!rotated) {
            st_io(out, o + e0, x, BF16);
            continue;
        }
        const float y = ld_io(in, i + e1, BF16);
        st_io(out, o + e0, x * c - y * s, BF16);
        st_io(out, o + e1, x * s + y * c, BF16);
    }
}

}  // namespace

cudaError_t rope_rotate(const ssm_rope_desc_t &d, const void *q, const void *k, const double *freq,
                        const int64_t *positions, void *q_out, void *k_out, float sign,
                        cudaStream_t st) {
    const bool bf16 = d.dtype_io == SSM_BF16;
    const int n = bf16 ? 8 : 4;
    RopeArgs a = {};
    a.q = q;
    a.k = k;
    a.qo = q_out;
    a.ko = k_out;
    a.freq = freq;
    a.pos = positions;
    bool vec = true;
    auto ok = [&](const void *p, const int64_t *s) {
        return !p || (((uintptr_t)p & 15) == 0 && s[0] % n == 0 && s[1] % n == 0 && s[2] % n == 0);
    };
    vec = ok(q, d.stride_q) && ok(k, d.stride_k) && ok(q_out, d.stride_q_out) &&
          ok(k_out, d.stride_k_out);
    for (int i = 0; i < 3; ++i) {
        a.sq[i] = d.stride_q[i];
        a.sk[i] = d.stride_k[i];
        a.sqo[i] = d.stride_q_out[i];
        a.sko[i] = d.stride_k_out[i];
    }
    a.sp[0] = d.stride_pos[0];
    a.sp[1] = d.stride_pos[1];
    a.tokens = d.batch * d.seqlen;
    a.L = (int)d.seqlen;
    a.hq = q ? (int)d.nheads_q : 0;
    a.hk = k ? (int)d.nheads_k : 0;
    a.dim = (int)d.headdim;
    a.rot = (int)d.rot_dim;
    a.pairs = d.layout == SSM_ROPE_PAIRS;
    a.mag = d.magnitude;
    a.sign = sign;
    // values past rot_dim stay where they are when both outputs are their inputs
    auto in_place = [](const void *i, const void *o, const int64_t *si, const int64_t *so) {
        return !i || (i == o && si[0] == so[0] && si[1] == so[1] && si[2] == so[2]);
    };
    const bool still = in_place(q, q_out, d.stride_q, d.stride_q_out) &&
                       in_place(k, k_out, d.stride_k, d.stride_k_out);
    const int rest = still ? 0 : a.dim - a.rot;
    vec = vec && a.rot / 2 <= TURNS && a.dim % n == 0 && (a.pairs ? a.rot % n : a.rot % (2 * n)) == 0;
    if (vec) {
        a.urot = a.pairs ? a.rot / n : a.rot / (2 * n);
        a.units = a.urot + rest / n;
    } else {
        a.urot = a.rot / 2;
        a.units = a.urot + rest;
    }
    if (a.units == 0) return cudaSuccess;
    if (!vec) {
        const unsigned grid = (unsigned)((a.tokens * a.units + 255) / 256);
        bf16 ? k_rope_any<true><<<grid, 256, 0, st>>>(a) : k_rope_any<false><<<grid, 256, 0, st>>>(a);
        profile_mark(st, "k_rope_any");
        return cudaGetLastError();
    }
    // fewer heads a thread until the card has eight warps a scheduler: 8192 tokens of 27 heads of
    // 64 took 11.4 us with eight heads a thread and 15.7 with four, 8 tokens of 20 heads of 128 3.9
    const long long heads = a.hq + a.hk, threads = (long long)sm_count() * 1024;
    int each = EACH;
    while (each > 1 && a.tokens * a.units * ((heads + each - 1) / each) < threads) each /= 2;
    a.share = (int)((heads + each - 1) / each);
    const long long fit = 256 / ((long long)a.units * a.share), spread = a.tokens / sm_count(), room = TURNS / (a.rot / 2);
    a.per_block = (int)max(1ll, min(fit, min(spread, room)));
    const size_t smem = sizeof(float2) * a.per_block * (a.rot / 2);
    const unsigned grid = (unsigned)((a.tokens + a.per_block - 1) / a.per_block);
    if (bf16)
        a.pairs ? k_rope<true, true><<<grid, 256, smem, st>>>(a) : k_rope<true, false><<<grid, 256, smem, st>>>(a);
    else
        a.pairs ? k_rope<false, true><<<grid, 256, smem, st>>>(a) : k_rope<false, false><<<grid, 256, smem, st>>>(a);
    profile_mark(st, "k_rope");
    return cudaGetLastError();
}

}  // namespace ssm
