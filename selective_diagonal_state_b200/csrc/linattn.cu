// Linear attention with a decay for each head, token by token: the recurrence for whole
// sequences (any type, head dims up to 256, any alignment), the sum over shared heads of
// the gradients, and the single-token step.
//
// The output and all gradients are one kind of walk (LaWalk).  With lam = e^{log_decay},
//     S_t = lam S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t          walk (q, k, v) forward
//     dq_t = scale S_t do_t                                         walk (do, v, k) forward, on S^T
//     G_t = scale q_t do_t^T + lam G_{t+1}  (the adjoint of S_t)
//     dk_t = G_t v_t                                                walk (v, do, q) in reverse, on G^T
//     dv_t = G_t^T k_t                                              walk (k, q, do) in reverse, on G
// and the reverse walks leave lam G_0 = dstate_in, having entered with dstate_out.
#include <type_traits>

#include "common.cuh"
#include "layer.h"

namespace ssm {
namespace {

// lam as a pair of floats: lam itself, and what its rounding leaves, so that the weight of
// a token n steps back is not n roundings off.
__device__ __forceinline__ void decay_pair(float g, float &hi, float &lo) {
    const double l = exp((double)g);
    hi = (float)l;
    lo = (float)(l - (double)hi);
}

// a value as it lies in memory, converted only when it is used: a load whose value is
// converted at once is waited for at once
template <bool BF16> struct Raw {
    using T = float;
    static __device__ __forceinline__ float f(T x) { return x; }
};
template <> struct Raw<true> {
    using T = unsigned short;
    static __device__ __forceinline__ float f(T x) { return __uint_as_float((uint32_t)x << 16); }
};

// Columns 32 bx .. of one (batch row, head, walk): lane = column, warp w of W holds the state rows
// [w NR, (w + 1) NR) in registers.  TT tokens at a time are staged in shared memory as fp32,
// the next ones waiting in registers; then every token costs a warp 4 NR FMAs, and the W
// warps' partial outputs are added once a tile.  Bound by the latency of a
// token's steps and, for wide heads, by shared memory, which gives every lane all of k and a: on
// one B200, a token costs 0.075 us for heads of 16, 0.11 for 64 and 0.2 for 128 (fp32, 2 x 300 tokens of
// 4 heads of 16 / 24: 25 us; 2 x 2048 of 8 heads of 64: 227 us; tiles of 16 tokens: 29 and 246).
template <int NR, int TT, bool BF16, int W = 8>
__global__ void __launch_bounds__(32 * W) k_la_recurrent(const LaArgs p, int slices) {
    constexpr int DA = W * NR, THREADS = 32 * W;
    using R = Raw<BF16>;
    using T = typename R::T;
    __shared__ __align__(16) float sa[TT][DA], sk[TT][DA];
    __shared__ float sv[TT][32], part[TT][W][32];
    const LaWalk w = p.w[blockIdx.y];
    const int bh = blockIdx.x / slices, c0 = 32 * (blockIdx.x - bh * slices);
    if (c0 >= w.dc) return;
    const int b = bh / p.H, h = bh - b * p.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, col = c0 + lane;
    const int n = p.lengths ? min(max(p.lengths[b], 0), p.L) : p.L;
    const T *pa = reinterpret_cast<const T *>(w.a) + b * w.sa[0] + (h / w.rep_a) * w.sa[2];
    const T *pk = reinterpret_cast<const T *>(w.k) + b * w.sk[0] + (h / w.rep_k) * w.sk[2];
    const T *pv = reinterpret_cast<const T *>(w.v) + b * w.sv[0] + (h / w.rep_v) * w.sv[2];
    const long long bo = b * w.so[0] + h * w.so[2];
    constexpr int NA = TT * DA / THREADS, NV = TT * 32 / THREADS;
    T xa[NA], xk[NA], xv[NV];
    auto fetch = [&](int i0) {
        const int m = min(TT, n - i0);
#pragma unroll
        for (int u = 0; u < NA; ++u) {
            const int e = tid + THREADS * u, i = e / DA, a = e - i * DA;
            const long long t = w.rev ? n - 1 - i0 - i : i0 + i;
            const bool on = i < m && a < w.da;
            xa[u] = xk[u] = 0;
            if (on && w.o) xa[u] = pa[t * w.sa[1] + a];
            if (on) xk[u] = pk[t * w.sk[1] + a];
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int e = tid + THREADS * u, i = e >> 5, c = c0 + (e & 31);
            const long long t = w.rev ? n - 1 - i0 - i : i0 + i;
            xv[u] = 0;
            if (i < m && c < w.dc) xv[u] = pv[t * w.sv[1] + c];
        }
    };
    if (n > 0) fetch(0);
    float lam, lam_lo;
    decay_pair(p.log_decay[h], lam, lam_lo);
    const long long sbase = (long long)bh * w.da * w.dc;
    float S[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int a = warp * NR + r;
        S[r] = (w.s_in && a < w.da && col < w.dc)
                   ? w.s_in[sbase + (long long)a * w.st_a + (long long)col * w.st_c] : 0.f;
    }
    // a token of the tile; `rev`: the decay comes behind it
    auto token = [&](int i, auto rev) {
        const float v = sv[i][lane];
        float o = 0.f;
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
            const float4 k4 = *reinterpret_cast<const float4 *>(&sk[i][warp * NR + r]);
            const float4 a4 = *reinterpret_cast<const float4 *>(&sa[i][warp * NR + r]);
            const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, aa[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float s = S[r + q];
                if (!decltype(rev)::value) s = fmaf(lam, s, fmaf(lam_lo, s, kk[q] * v));
                else s = fmaf(kk[q], v, s);
                o = fmaf(aa[q], s, o);
                S[r + q] = decltype(rev)::value ? fmaf(lam, s, lam_lo * s) : s;
            }
        }
        part[i][warp][lane] = o;
    };
    for (int i0 = 0; i0 < n; i0 += TT) {
        const int m = min(TT, n - i0);
        // every warp is past the tile before (the barrier in front of its sums)
#pragma unroll
        for (int u = 0; u < NA; ++u) {
            const int e = tid + THREADS * u;
            (&sa[0][0])[e] = R::f(xa[u]);
            (&sk[0][0])[e] = R::f(xk[u]);
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) (&sv[0][0])[tid + THREADS * u] = R::f(xv[u]) * w.write;
        __syncthreads();
        if (i0 + TT < n) fetch(i0 + TT);
        if (w.rev) {
#pragma unroll(NR == 4 ? 8 : 4)
            for (int i = 0; i < m; ++i) token(i, std::true_type{});
        } else {
#pragma unroll(NR == 4 ? 8 : 4)
            for (int i = 0; i < m; ++i) token(i, std::false_type{});
        }
        __syncthreads();
        if (w.o)
            for (int e = tid; e < m * 32; e += THREADS) {
                const int i = e >> 5, c = e & 31;
                if (c0 + c >= w.dc) continue;
                float o = part[i][0][c];
#pragma unroll
                for (int q = 1; q < W; ++q) o += part[i][q][c];
                const long long t = w.rev ? n - 1 - i0 - i : i0 + i;
                st_io(w.o, bo + t * w.so[1] + c0 + c, o * w.read, BF16 && !w.o_f32);
            }
    }
    if (w.s_out && col < w.dc)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int a = warp * NR + r;
            if (a < w.da) w.s_out[sbase + (long long)a * w.st_a + (long long)col * w.st_c] = S[r];
        }
}

__global__ void __launch_bounds__(256)
k_la_group_sum(const float *in, void *out, long long s0, long long s1, long long s2, int B, int L,
               int H, int rep, int d, const int *lengths, int bf16) {
    const int G = H / rep;
    const long long total = (long long)B * L * G * d;
    for (long long e = blockIdx.x * 256ll + threadIdx.x; e < total; e += gridDim.x * 256ll) {
        const int c = (int)(e % d);
        const long long r = e / d;
        const int g = (int)(r % G);
        const long long bt = r / G;
        const int b = (int)(bt / L), t = (int)(bt - (long long)b * L);
        if (lengths && t >= lengths[b]) continue;
        const float *src = in + (bt * H + (long long)g * rep) * d + c;
        float s = src[0];
        for (int k = 1; k < rep; ++k) s += src[(long long)k * d];
        st_io(out, b * s0 + t * s1 + g * s2 + c, s, bf16);
    }
}

// The same, 16 bytes of bf16 or fp32 sums a thread: dense fp32 rows, 16-byte aligned outputs.
__global__ void __launch_bounds__(256)
k_la_group_sum16(const float4 *in, void *out, long long s0, long long s1, long long s2, int L, int H, int rep, int d,
                 const int *lengths, int bf16, long long total) {
    const long long e = blockIdx.x * 256ll + threadIdx.x;
    if (e >= total) return;
    const int G = H / rep, per = bf16 ? 8 : 4, nv = d / per, f4 = per / 4;
    const long long r = e / nv;
    const int c = (int)(e - r * nv);
    const long long bt = r / G;
    const int g = (int)(r - bt * G), b = (int)(bt / L), t = (int)(bt - (long long)b * L);
    if (lengths && t >= lengths[b]) return;
    const float4 *src = in + ((bt * H + (long long)g * rep) * d + (long long)c * per) / 4;
    const long long step = d / 4;
    float4 s[2] = {src[0], f4 == 2 ? src[1] : make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k = 1; k < rep; ++k)
        for (int i = 0; i < f4; ++i) {
            const float4 x = src[k * step + i];
            s[i].x += x.x;
            s[i].y += x.y;
            s[i].z += x.z;
            s[i].w += x.w;
        }
    const long long at = b * s0 + t * s1 + g * s2 + (long long)c * per;
    if (bf16) {
        const __nv_bfloat162 v[4] = {__floats2bfloat162_rn(s[0].x, s[0].y), __floats2bfloat162_rn(s[0].z, s[0].w),
                                     __floats2bfloat162_rn(s[1].x, s[1].y), __floats2bfloat162_rn(s[1].z, s[1].w)};
        *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(out) + at) = *reinterpret_cast<const uint4 *>(v);
    } else {
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + at) = s[0];
    }
}

struct StepArgs {
    const void *q, *k, *v;
    const float *log_decay;
    float *state;
    void *o;
    long long sq0, sq2, sk0, sk2, sv0, sv2, so0, so2;
    int H, rep, dk, dv, bf16;
    float scale;
};

// One token: bound by reading and writing the state.  A block takes 32 columns of a head's
// state, 16 rows at a time, eight lanes a row with four columns each (VEC), or a lane a
// column; the partial products with q are added over the rows at the end.  64 rows of 16 heads of
// 128 x 128 (137 MB there and back): 25.8 us on one B200, 5.2 TB/s, the launch among it.
template <bool VEC>
__global__ void __launch_bounds__(128) k_la_step(const StepArgs p, int slices) {
    __shared__ float sq[LA_MAX_DIM], sk[LA_MAX_DIM], red[4][32], decay[2];
    const int bh = blockIdx.x / slices, c0 = 32 * (blockIdx.x - bh * slices);
    const int b = bh / p.H, h = bh - b * p.H, hk = h / p.rep;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int a = tid; a < p.dk; a += 128) {
        sq[a] = ld_io(p.q, b * p.sq0 + h * p.sq2 + a, p.bf16) * p.scale;
        sk[a] = ld_io(p.k, b * p.sk0 + hk * p.sk2 + a, p.bf16);
    }
    if (tid == 127) decay_pair(p.log_decay[h], decay[0], decay[1]);
    float *S = p.state + (long long)bh * p.dk * p.dv;
    const long long vb = b * p.sv0 + hk * p.sv2;
    if constexpr (VEC) {
        const int r0 = tid >> 3, c = c0 + 4 * (lane & 7);
        float v[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
        const bool on = c < p.dv;
        float4 x[8];
        auto load = [&](int a0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int a = a0 + r0 + 16 * i;
                if (on && a < p.dk) x[i] = *reinterpret_cast<const float4 *>(S + (long long)a * p.dv + c);
            }
        };
        load(0);   // on its way beside the decay
        if (on)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ld_io(p.v, vb + c + j, p.bf16);
        __syncthreads();
        const float lam = decay[0], lam_lo = decay[1];
        for (int a0 = 0; a0 < p.dk; a0 += 128) {
            if (a0) load(a0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int a = a0 + r0 + 16 * i;
                if (!on || a >= p.dk) continue;
                const float k = sk[a], q = sq[a];
                x[i].x = fmaf(lam, x[i].x, fmaf(lam_lo, x[i].x, k * v[0]));
                x[i].y = fmaf(lam, x[i].y, fmaf(lam_lo, x[i].y, k * v[1]));
                x[i].z = fmaf(lam, x[i].z, fmaf(lam_lo, x[i].z, k * v[2]));
                x[i].w = fmaf(lam, x[i].w, fmaf(lam_lo, x[i].w, k * v[3]));
                o[0] = fmaf(q, x[i].x, o[0]);
                o[1] = fmaf(q, x[i].y, o[1]);
                o[2] = fmaf(q, x[i].z, o[2]);
                o[3] = fmaf(q, x[i].w, o[3]);
                *reinterpret_cast<float4 *>(S + (long long)a * p.dv + c) = x[i];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o[j] += __shfl_xor_sync(0xffffffffu, o[j], 8);
            o[j] += __shfl_xor_sync(0xffffffffu, o[j], 16);
            if (lane < 8) red[warp][4 * lane + j] = o[j];
        }
    } else {
        const int c = c0 + lane;
        float o = 0.f, x[16];
        auto load = [&](int a0) {   // 16 rows on their way at once
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c < p.dv && a0 + 4 * i < p.dk) x[i] = S[(long long)(a0 + 4 * i) * p.dv + c];
        };
        load(warp);
        const float v = c < p.dv ? ld_io(p.v, vb + c, p.bf16) : 0.f;
        __syncthreads();
        const float lam = decay[0], lam_lo = decay[1];
        if (c < p.dv) {
            for (int a0 = warp; a0 < p.dk; a0 += 64) {
                if (a0 > warp) load(a0);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int a = a0 + 4 * i;
                    if (a >= p.dk) break;
                    x[i] = fmaf(lam, x[i], fmaf(lam_lo, x[i], sk[a] * v));
                    o = fmaf(sq[a], x[i], o);
                    S[(long long)a * p.dv + c] = x[i];
                }
            }
        }
        red[warp][lane] = o;
    }
    __syncthreads();
    if (tid < 32 && c0 + tid < p.dv)
        st_io(p.o, b * p.so0 + h * p.so2 + c0 + tid,
              red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid], p.bf16);
}

}  // namespace

cudaError_t la_recurrent(const LaArgs &p, cudaStream_t st) {
    int da = 0, dc = 0;
    for (int i = 0; i < p.nwalk; ++i) {
        da = p.w[i].da > da ? p.w[i].da : da;
        dc = p.w[i].dc > dc ? p.w[i].dc : dc;
    }
    const int slices = (dc + 31) / 32;
    const dim3 grid((unsigned)((long long)p.B * p.H * slices), p.nwalk);
    auto go = [&](auto kern, int threads = 256) { kern<<<grid, threads, 0, st>>>(p, slices); };
    if (da <= 16) p.bf16 ? go(k_la_recurrent<4, 32, true, 4>, 128) : go(k_la_recurrent<4, 32, false, 4>, 128);
    else if (da <= 32) p.bf16 ? go(k_la_recurrent<4, 32, true>) : go(k_la_recurrent<4, 32, false>);
    else if (da <= 64) p.bf16 ? go(k_la_recurrent<8, 24, true>) : go(k_la_recurrent<8, 24, false>);
    else if (da <= 128) p.bf16 ? go(k_la_recurrent<16, 16, true>) : go(k_la_recurrent<16, 16, false>);
    else p.bf16 ? go(k_la_recurrent<32, 8, true>) : go(k_la_recurrent<32, 8, false>);
    profile_mark(st, "k_la_recurrent");
    return cudaGetLastError();
}

cudaError_t la_group_sum(const float *in, void *out, const long long *so, int B, int L, int H,
                         int rep, int d, const int *lengths, int bf16, cudaStream_t st) {
    const long long total = (long long)B * L * (H / rep) * d;
    const int per = bf16 ? 8 : 4;
    if (d % per == 0 && ((uintptr_t)out & 15) == 0 && so[0] % per == 0 && so[1] % per == 0 && so[2] % per == 0) {
        const long long n = total / per;
        k_la_group_sum16<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(reinterpret_cast<const float4 *>(in), out, so[0], so[1],
                                                                     so[2], L, H, rep, d, lengths, bf16, n);
        profile_mark(st, "k_la_group_sum16");
        return cudaGetLastError();
    }
    long long blocks = (total + 255) / 256;
    if (blocks > sm_count() * 16ll) blocks = sm_count() * 16ll;
    k_la_group_sum<<<(unsigned)blocks, 256, 0, st>>>(in, out, so[0], so[1], so[2], B, L, H, rep, d,
                                                     lengths, bf16);
    profile_mark(st, "k_la_group_sum");
    return cudaGetLastError();
}

cudaError_t la_step(const ssm_linattn_desc_t &d, const void *q, const void *k, const void *v,
                    const float *log_decay, float *state, void *o, cudaStream_t st) {
    StepArgs a = {q, k, v, log_decay, state, o, d.stride_q[0], d.stride_q[2], d.stride_k[0],
                  d.stride_k[2], d.stride_v[0], d.stride_v[2], d.stride_o[0], d.stride_o[2],
                  (int)d.nheads, (int)(d.nheads / d.nheads_kv), (int)d.dim_k, (int)d.dim_v,
                  d.dtype_io == SSM_BF16, d.scale};
    const int slices = (int)((d.dim_v + 31) / 32);
    const unsigned grid = (unsigned)(d.batch * d.nheads * slices);
    if (d.dim_v % 4 == 0 && ((uintptr_t)state & 15) == 0)
        k_la_step<true><<<grid, 128, 0, st>>>(a, slices);
    else
        k_la_step<false><<<grid, 128, 0, st>>>(a, slices);
    profile_mark(st, "k_la_step");
    return cudaGetLastError();
}

}  // namespace ssm
