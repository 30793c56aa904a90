// Rotary positions of queries and keys, and the gradient through them (the opposite
// rotation): pair j of every head at position m turns by m freq[j],
//     (a, b) -> magnitude (a cos - b sin, a sin + b cos).
// The angle is taken in 64 bits, in half turns, and reduced to (-1, 1] there, so that
// sincospi of its fp32 rest is right for any position.  Bound by memory (each value read
// and written once): a thread takes one 16-byte piece of pairs of a token (two pieces in
// the half layout) and turns it for all, or a share of, the heads of q and k with one
// set of sines; the values past rot_dim are copied piece by piece.
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

// Pieces of N values (16 bytes): dense and 16-byte aligned heads.
template <bool BF16, bool PAIRS>
__global__ void __launch_bounds__(256) k_rope(const RopeArgs p) {
    constexpr int N = BF16 ? 8 : 4, ES = 16 / N, NP = PAIRS ? N / 2 : N;
    const long long per_token = (long long)p.units * p.share;
    const long long id = blockIdx.x * 256ll + threadIdx.x;
    const long long tok = id / per_token;
    if (tok >= p.tokens) return;
    const int rest = (int)(id - tok * per_token);
    const int h0 = rest / p.units, u = rest - h0 * p.units;
    const long long b = tok / p.L, t = tok - b * p.L;
    const bool rotated = u < p.urot;
    float c[NP], s[NP];
    if (rotated) {
        const double m = p.pos ? (double)p.pos[b * p.sp[0] + t * p.sp[1]] : (double)t;
#pragma unroll
        for (int i = 0; i < NP; ++i)
            turn(m * (p.freq[u * NP + i] * INV_PI), p.mag, p.sign, c[i], s[i]);
    }
    // first value of the piece in its head, and of its partner in the half layout
    const int e0 = rotated ? u * N : p.rot + (u - p.urot) * N, e1 = e0 + p.rot / 2;
    const int heads = p.hq + p.hk;
#pragma unroll 4
    for (int hh = h0; hh < heads; hh += p.share) {
        const bool isk = hh >= p.hq;
        const int h = isk ? hh - p.hq : hh;
        const long long *si = isk ? p.sk : p.sq, *so = isk ? p.sko : p.sqo;
        const char *in = reinterpret_cast<const char *>(isk ? p.k : p.q) +
                         (b * si[0] + t * si[1] + h * si[2] + e0) * ES;
        char *out = reinterpret_cast<char *>(isk ? p.ko : p.qo) +
                    (b * so[0] + t * so[1] + h * so[2] + e0) * ES;
        const uint4 w = *reinterpret_cast<const uint4 *>(in);
        if (!rotated) {
            *reinterpret_cast<uint4 *>(out) = w;
            continue;
        }
        float x[N];
        unpack<BF16>(w, x);
        if (PAIRS) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float a = x[2 * i], bb = x[2 * i + 1];
                x[2 * i] = a * c[i] - bb * s[i];
                x[2 * i + 1] = a * s[i] + bb * c[i];
            }
        } else {
            float y[N];
            unpack<BF16>(*reinterpret_cast<const uint4 *>(in + (e1 - e0) * ES), y);
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const float a = x[i], bb = y[i];
                x[i] = a * c[i] - bb * s[i];
                y[i] = a * s[i] + bb * c[i];
            }
            *reinterpret_cast<uint4 *>(out + (e1 - e0) * ES) = pack<BF16>(y);
        }
        *reinterpret_cast<uint4 *>(out) = pack<BF16>(x);
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
    vec = vec && a.dim % n == 0 && (a.pairs ? a.rot % n : a.rot % (2 * n)) == 0;
    if (vec) {
        a.urot = a.pairs ? a.rot / n : a.rot / (2 * n);
        a.units = a.urot + rest / n;
    } else {
        a.urot = a.rot / 2;
        a.units = a.urot + rest;
    }
    if (a.units == 0) return cudaSuccess;
    // share the heads among more threads until the card has a few warps a scheduler
    a.share = 1;
    const long long want = (long long)sm_count() * 1024;
    while (vec && 2 * a.share <= a.hq + a.hk && a.tokens * a.units * a.share < want) a.share *= 2;
    const long long threads = a.tokens * a.units * a.share;
    const unsigned grid = (unsigned)((threads + 255) / 256);
    if (vec && bf16)
        a.pairs ? k_rope<true, true><<<grid, 256, 0, st>>>(a) : k_rope<true, false><<<grid, 256, 0, st>>>(a);
    else if (vec)
        a.pairs ? k_rope<false, true><<<grid, 256, 0, st>>>(a) : k_rope<false, false><<<grid, 256, 0, st>>>(a);
    else
        bf16 ? k_rope_any<true><<<grid, 256, 0, st>>>(a) : k_rope_any<false><<<grid, 256, 0, st>>>(a);
    profile_mark(st, "k_rope");
    return cudaGetLastError();
}

}  // namespace ssm
