// Root-mean-square norm with the residual's addition, 8-bit output with scales, and its
// gradient:
//     r = x + residual,  rstd = (mean(r^2) + eps)^{-1/2},  y = r rstd w,
//     dx = rstd (w dy - xhat mean(w dy xhat)) + dr,  xhat = r rstd,  dw = sum_rows dy xhat.
// Bound by memory: a row is read once, kept in registers (V 16-byte pieces a thread) while the
// team of T threads that holds it sums its squares, and written once.  Sums are fp32.  r is
// rounded to the I/O type before its norm is taken, so that the norm is that of the stored
// residual stream, which the backward reads.
//
// With many rows a team is a warp (rows up to 2048 bf16 values): no barriers, and 8 x 16
// bytes a lane and tensor in flight.  On one B200, 65536 x 2048 bf16 with a residual: 160 us without
// codes (1.07 GB, 6.7 TB/s), 152 with a row scale (0.94 GB, 6.2 TB/s; 206 with a block a
// row), 178 with block scales, whose maxima go through shuffles; the gradient 232 us
// (1.07 GB, 4.6 TB/s: three tensors and the sums of dweight take all of a thread's 128 registers and, at four
// pieces of bf16, 200 bytes of spills, so that one block of 16 warps is on an SM, a quarter of its warps).
// With few rows, a decoding step's, a block takes a row, for the shortest chain (8 x 2048: 2.4 us).
#include <cuda_fp8.h>

#include "common.cuh"
#include "layer.h"

namespace ssm {
namespace {

constexpr float E4M3_MAX = 448.f;

template <bool BF16> struct Io;
template <> struct Io<true> {
    static constexpr int N = 8;   // values in 16 bytes
    static __device__ __forceinline__ void unpack(const uint4 &w, float *v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 r = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&r);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Io<false> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float *v) {
        v[0] = __uint_as_float(w.x);
        v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z);
        v[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};

// the larger of two magnitudes; a NaN stays
__device__ __forceinline__ float top(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// What codes are values times, 448 / amax, and what values are codes times.  Both stay finite for the
// smallest blocks, and each other's inverse: 2^127 and 2^-127 there.  A block of zeros has codes and scale 0.
__device__ __forceinline__ float code_scale(float amax) { return fminf(E4M3_MAX / amax, 0x1p127f); }
__device__ __forceinline__ float value_scale(float amax) {
    return top(amax / E4M3_MAX, amax > 0.f ? 0x1p-127f : 0.f);
}
__device__ __forceinline__ uint16_t e4m3x2(float a, float b) {
    return (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Team reduction: T threads (a power of two) of a block, consecutive; `buf` has a float a
// warp.  Every thread of the team calls it.
template <int T, bool MAX>
__device__ __forceinline__ float team_reduce(float v, float *buf) {
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? top(v, u) : v + u;
    }
    if constexpr (T > 32) {
        const int warp = threadIdx.x >> 5, first = warp & ~(T / 32 - 1);
        const int bar = 1 + threadIdx.x / T;   // the team's own barrier
        asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "n"(T) : "memory");   // the buffer's last use is over
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        asm volatile("bar.sync %0, %1;\n" ::"r"(bar), "n"(T) : "memory");
        v = buf[first];
#pragma unroll
        for (int i = 1; i < T / 32; ++i) v = MAX ? top(v, buf[first + i]) : v + buf[first + i];
    }
    return v;
}

struct FwdArgs {
    const void *x, *res;
    const float *w;
    void *r, *y;
    unsigned char *y8;
    float *scales, *rstd;
    long long rows, sx, sres, sr, sy, sy8;
    int dim, quant;
    float eps;
};

template <bool BF16, int V, int T, int QUANT>
__global__ void __launch_bounds__(T < 256 ? 256 : T) k_rmsnorm_fwd(const FwdArgs p) {
    constexpr int BLOCK = T < 256 ? 256 : T;
    using I = Io<BF16>;
    constexpr int N = I::N, ES = 16 / N;
    __shared__ float buf[BLOCK / 32];
    const int lane = threadIdx.x % T;
    const long long row = blockIdx.x * (long long)(BLOCK / T) + threadIdx.x / T;
    const bool live = row < p.rows;
    const int nv = p.dim / N;
    auto at = [&](const void *base, long long stride, int v) {
        return reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) +
                                               row * stride * ES) + v;
    };
    uint4 raw[V], rs[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * T;
        raw[k] = make_uint4(0, 0, 0, 0);
        if (live && v < nv) raw[k] = *at(p.x, p.sx, v);
    }
    if (p.res) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * T;
            rs[k] = make_uint4(0, 0, 0, 0);
            if (live && v < nv) rs[k] = *at(p.res, p.sres, v);
        }
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        float a[N];
        I::unpack(raw[k], a);
        if (p.res) {
            float b[N];
            I::unpack(rs[k], b);
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] += b[i];
            raw[k] = I::pack(a);   // the stored sum is the one that is normalised
            I::unpack(raw[k], a);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(a[i], a[i], ss);
        const int v = lane + k * T;
        if (p.r && live && v < nv) *const_cast<uint4 *>(at(p.r, p.sr, v)) = raw[k];
    }
    ss = team_reduce<T, false>(ss, buf);
    const float rstd = rsqrtf(ss / (float)p.dim + p.eps);
    if (p.rstd && live && lane == 0) p.rstd[row] = rstd;
    // the norm of piece k, in fp32
    auto value = [&](int k, float *a) {
        const int v = lane + k * T;
        I::unpack(raw[k], a);
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] *= rstd;
        if (p.w && v < nv) {
            float w[N];
#pragma unroll
            for (int q = 0; q < N / 4; ++q)
                *reinterpret_cast<float4 *>(w + 4 * q) =
                    __ldg(reinterpret_cast<const float4 *>(p.w) + (long long)v * (N / 4) + q);
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] *= w[i];
        }
    };
    if (QUANT == SSM_QUANT_NONE) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * T;
            float a[N];
            value(k, a);
            if (live && v < nv) *const_cast<uint4 *>(at(p.y, p.sy, v)) = I::pack(a);
        }
        return;
    }
    float y[V][N];
    float whole = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * T;
        value(k, y[k]);
        if (p.y && live && v < nv) *const_cast<uint4 *>(at(p.y, p.sy, v)) = I::pack(y[k]);
        if (QUANT == SSM_QUANT_ROW)
#pragma unroll
            for (int i = 0; i < N; ++i) whole = top(whole, fabsf(y[k][i]));
    }
    if (QUANT == SSM_QUANT_ROW) {
        whole = team_reduce<T, true>(whole, buf);
        if (live && lane == 0) p.scales[row] = value_scale(whole);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * T;
        float m = whole;
        if (QUANT == SSM_QUANT_BLOCK) {   // 128 columns: 128 / N neighbouring lanes
#pragma unroll
            for (int i = 0; i < N; ++i) m = top(m, fabsf(y[k][i]));
#pragma unroll
            for (int o = 64 / N; o > 0; o >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (live && v < nv && v % (128 / N) == 0)
                p.scales[row * (p.dim / 128) + v / (128 / N)] = value_scale(m);
        }
        const float c = code_scale(m);
        if (live && v < nv) {
            unsigned char *dst = p.y8 + row * p.sy8 + (long long)v * N;
            const uint32_t lo = e4m3x2(y[k][0] * c, y[k][1] * c) | (uint32_t)e4m3x2(y[k][2] * c, y[k][3] * c) << 16;
            if constexpr (N == 8) {
                const uint32_t hi =
                    e4m3x2(y[k][4] * c, y[k][5] * c) | (uint32_t)e4m3x2(y[k][6] * c, y[k][7] * c) << 16;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(lo, hi);
            } else {
                *reinterpret_cast<uint32_t *>(dst) = lo;
            }
        }
    }
}

// Any alignment, stride and width: a block a row, the row read again for each pass
// (from r once it is stored).
template <bool BF16>
__global__ void __launch_bounds__(256) k_rmsnorm_fwd_any(const FwdArgs p) {
    __shared__ float buf[8];
    const long long row = blockIdx.x;
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.dim; i += 256) {
        float a = ld_io(p.x, row * p.sx + i, BF16);
        if (p.res) {
            a += ld_io(p.res, row * p.sres + i, BF16);
            if (BF16) a = __bfloat162float(__float2bfloat16_rn(a));
        }
        if (p.r) st_io(p.r, row * p.sr + i, a, BF16);
        ss = fmaf(a, a, ss);
    }
    ss = team_reduce<256, false>(ss, buf);
    const float rstd = rsqrtf(ss / (float)p.dim + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    const void *src = p.r ? p.r : p.x;
    const long long ss_ = p.r ? p.sr : p.sx;
    auto value = [&](int i) {   // this thread wrote the values it reads
        const float a = ld_io(src, row * ss_ + i, BF16) * rstd;
        return p.w ? a * p.w[i] : a;
    };
    float whole = 0.f;
    if (p.quant == SSM_QUANT_ROW) {
        for (int i = threadIdx.x; i < p.dim; i += 256) whole = top(whole, fabsf(value(i)));
        whole = team_reduce<256, true>(whole, buf);
        if (threadIdx.x == 0) p.scales[row] = value_scale(whole);
    }
    if (p.quant == SSM_QUANT_BLOCK) {   // a warp a block
        for (int b = threadIdx.x / 32; b < p.dim / 128; b += 8) {
            // the row's values of other threads: r is stored by now (barrier above)
            float a[4], m = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] = value(128 * b + 32 * j + (threadIdx.x & 31));
                m = top(m, fabsf(a[j]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = top(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((threadIdx.x & 31) == 0) p.scales[row * (p.dim / 128) + b] = value_scale(m);
            const float c = code_scale(m);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p.y8[row * p.sy8 + 128 * b + 32 * j + (threadIdx.x & 31)] =
                    (unsigned char)(e4m3x2(a[j] * c, 0.f) & 0xff);
        }
        __syncthreads();   // y below may overwrite what a block's warp reads
    }
    const float c = code_scale(whole);
    for (int i = threadIdx.x; i < p.dim; i += 256) {
        const float a = value(i);
        if (p.quant == SSM_QUANT_ROW)
            p.y8[row * p.sy8 + i] = (unsigned char)(e4m3x2(a * c, 0.f) & 0xff);
        if (p.y) st_io(p.y, row * p.sy + i, a, BF16);
    }
}

struct BwdArgs {
    const void *dy, *r, *dr;
    const float *w, *rstd;
    void *dx;
    float *part;   // [gridDim.x][dim] partial sums of dweight (null: not wanted)
    long long rows, sdy, sr, sdr, sdx;
    int dim;
};

// A team of T threads walks rows with the grid's stride; dweight's partial sums stay in
// its registers, are added over the block's teams in team order, and leave once.
constexpr int BWD_BLOCK = 512;
template <bool BF16, int V, int T>
__global__ void __launch_bounds__(BWD_BLOCK) k_rmsnorm_bwd(const BwdArgs p) {
    using I = Io<BF16>;
    constexpr int BLOCK = BWD_BLOCK, N = I::N, ES = 16 / N, TEAMS = BLOCK / T;
    __shared__ float buf[BLOCK / 32];
    __shared__ float add[TEAMS > 1 ? T * N : 1];
    const int lane = threadIdx.x % T, team = threadIdx.x / T;
    const int nv = p.dim / N;
    float dw[V][N];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) dw[k][i] = 0.f;
    auto weight = [&](int v, float *w) {
#pragma unroll
        for (int q = 0; q < N / 4; ++q)
            *reinterpret_cast<float4 *>(w + 4 * q) =
                p.w && v < nv ? __ldg(reinterpret_cast<const float4 *>(p.w) + (long long)v * (N / 4) + q)
                              : make_float4(1.f, 1.f, 1.f, 1.f);
    };
    const long long step = (long long)gridDim.x * TEAMS;
    const long long rounds = (p.rows + step - 1) / step;
    for (long long it = 0; it < rounds; ++it) {
        const long long row = it * step + (long long)blockIdx.x * TEAMS + team;
        const bool live = row < p.rows;
        auto at = [&](const void *base, long long stride, int v) {
            return reinterpret_cast<const uint4 *>(reinterpret_cast<const char *>(base) +
                                                   row * stride * ES) + v;
        };
        uint4 g4[V], r4[V], d4[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * T;
            g4[k] = r4[k] = d4[k] = make_uint4(0, 0, 0, 0);
            if (live && v < nv) {
                g4[k] = *at(p.dy, p.sdy, v);
                r4[k] = *at(p.r, p.sr, v);
                if (p.dr) d4[k] = *at(p.dr, p.sdr, v);
            }
        }
        const float rstd = live ? p.rstd[row] : 0.f;
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * T;
            float g[N], r[N], w[N];
            I::unpack(g4[k], g);
            I::unpack(r4[k], r);
            weight(v, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float xh = r[i] * rstd;
                dw[k][i] = fmaf(g[i], xh, dw[k][i]);
                dot = fmaf(w[i] * g[i], xh, dot);
            }
        }
        dot = team_reduce<T, false>(dot, buf) / (float)p.dim;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * T;
            if (!live || v >= nv) continue;
            float g[N], r[N], d[N], w[N];
            I::unpack(g4[k], g);
            I::unpack(r4[k], r);
            I::unpack(d4[k], d);
            weight(v, w);
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = fmaf(rstd, w[i] * g[i] - r[i] * rstd * dot, d[i]);
            *const_cast<uint4 *>(at(p.dx, p.sdx, v)) = I::pack(g);
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * T;
        if constexpr (TEAMS > 1) {
            for (int t = 0; t < TEAMS; ++t) {
                __syncthreads();
                if (t == team) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (t) dw[k][i] += add[lane * N + i];
                        add[lane * N + i] = dw[k][i];
                    }
                }
            }
            __syncthreads();
        }
        if (team == TEAMS - 1 && v < nv) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                p.part[(long long)blockIdx.x * p.dim + (long long)v * N + i] = dw[k][i];
        }
    }
}

// Any alignment, stride and width: a block a row for dx.
template <bool BF16>
__global__ void __launch_bounds__(256) k_rmsnorm_bwd_any(const BwdArgs p) {
    __shared__ float buf[8];
    const long long row = blockIdx.x;
    const float rstd = p.rstd[row];
    float dot = 0.f;
    for (int i = threadIdx.x; i < p.dim; i += 256)
        dot = fmaf((p.w ? p.w[i] : 1.f) * ld_io(p.dy, row * p.sdy + i, BF16),
                   ld_io(p.r, row * p.sr + i, BF16) * rstd, dot);
    dot = team_reduce<256, false>(dot, buf) / (float)p.dim;
    for (int i = threadIdx.x; i < p.dim; i += 256) {
        const float g = ld_io(p.dy, row * p.sdy + i, BF16) * (p.w ? p.w[i] : 1.f);
        const float xh = ld_io(p.r, row * p.sr + i, BF16) * rstd;
        const float d = p.dr ? ld_io(p.dr, row * p.sdr + i, BF16) : 0.f;
        st_io(p.dx, row * p.sdx + i, fmaf(rstd, g - xh * dot, d), BF16);
    }
}
// Its dweight partials, before dx may overwrite dy: block y takes the rows y, y + gridDim.y, ...
template <bool BF16>
__global__ void __launch_bounds__(256) k_rmsnorm_dw_any(const BwdArgs p) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= p.dim) return;
    float s = 0.f;
    for (long long row = blockIdx.y; row < p.rows; row += gridDim.y)
        s = fmaf(ld_io(p.dy, row * p.sdy + i, BF16), ld_io(p.r, row * p.sr + i, BF16) * p.rstd[row], s);
    p.part[(long long)blockIdx.y * p.dim + i] = s;
}

// dweight[i] = sum over the partials, 32 columns a block, eight threads a column, each
// over its own share and the shares added in order.
__global__ void __launch_bounds__(256) k_rmsnorm_dw(const float *part, float *dw, int dim, int n) {
    __shared__ float sh[8][33];
    const int c = threadIdx.x & 31, q = threadIdx.x >> 5, i = blockIdx.x * 32 + c;
    float s = 0.f;
    if (i < dim)
        for (int k = q; k < n; k += 8) s += part[(long long)k * dim + i];
    sh[q][c] = s;
    __syncthreads();
    if (q == 0 && i < dim) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += sh[k][c];
        dw[i] = s;
    }
}

bool al16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Pieces a thread and threads a row for rows of nv 16-byte pieces; v 0: the kernels for any
// row.  Forward: a warp a row while eight pieces a lane suffice, wider teams above; a block a row where
// there are too few rows for that to fill the card (four warps an SM): 591 x 2048 with block scales took 4.2 us
// so and 8.0 with a warp a row, 8 x 2048 4.2 and 6.3 (in a graph), 3999 x 1024 12.4 and 8.3.
struct Shape {
    int v, t;
};
Shape fwd_team(int nv, long long rows) {
    if (rows < SMS * 4 && nv > 32) {
        if (nv <= 256) return {1, 256};
        if (nv <= 512) return {2, 256};
        if (nv <= 1024) return {4, 256};
    }
    if (nv <= 32) return {1, 32};
    if (nv <= 64) return {2, 32};
    if (nv <= 128) return {4, 32};
    if (nv <= 256) return {8, 32};
    if (nv <= 512) return {8, 64};
    if (nv <= 1024) return {8, 128};
    if (nv <= 2048) return {8, 256};
    return {0, 0};
}
// Backward: three tensors and the sums of dweight are in registers, so half of that.  Four pieces of
// bf16 spill; where three do (129 to 192 of them), 8191 rows of 1032 to 1536 take 20.6 to 22.7 us, 65536 110 to 122,
// against 33 to 37 and 192 to 214 with four.
Shape bwd_team(int nv) {
    if (nv <= 32) return {1, 32};
    if (nv <= 64) return {2, 32};
    if (nv <= 128) return {4, 32};
    if (nv <= 192) return {3, 64};
    if (nv <= 256) return {4, 64};
    if (nv <= 512) return {4, 128};
    if (nv <= 1024) return {4, 256};
    if (nv <= 2048) return {4, 512};
    return {0, 0};
}

constexpr int DW_BLOCKS = SMS;   // partial sums of dweight: a block an SM

int bwd_blocks(const ssm_rmsnorm_desc_t &d) {
    const int n = d.dtype_io == SSM_BF16 ? 8 : 4;
    const Shape s = bwd_team((int)((d.dim + n - 1) / n));
    const long long teams = s.v ? BWD_BLOCK / s.t : 1;   // rows a block takes at once
    const long long b = (d.rows + teams - 1) / teams;
    return (int)(b < DW_BLOCKS ? b : DW_BLOCKS);
}

template <bool BF16, int QUANT>
cudaError_t fwd(const FwdArgs &a, bool vec, cudaStream_t st) {
    constexpr int N = Io<BF16>::N;
    const Shape s = vec ? fwd_team(a.dim / N, a.rows) : Shape{0, 0};
    auto go = [&](auto kern, int t) {
        const int block = t < 256 ? 256 : t;
        const long long per = block / t, grid = (a.rows + per - 1) / per;
        kern<<<(unsigned)grid, block, 0, st>>>(a);
    };
    if (s.t == 32 && s.v == 1) go(k_rmsnorm_fwd<BF16, 1, 32, QUANT>, 32);
    else if (s.t == 32 && s.v == 2) go(k_rmsnorm_fwd<BF16, 2, 32, QUANT>, 32);
    else if (s.t == 32 && s.v == 4) go(k_rmsnorm_fwd<BF16, 4, 32, QUANT>, 32);
    else if (s.t == 32) go(k_rmsnorm_fwd<BF16, 8, 32, QUANT>, 32);
    else if (s.t == 64) go(k_rmsnorm_fwd<BF16, 8, 64, QUANT>, 64);
    else if (s.t == 128) go(k_rmsnorm_fwd<BF16, 8, 128, QUANT>, 128);
    else if (s.t == 256 && s.v == 1) go(k_rmsnorm_fwd<BF16, 1, 256, QUANT>, 256);
    else if (s.t == 256 && s.v == 2) go(k_rmsnorm_fwd<BF16, 2, 256, QUANT>, 256);
    else if (s.t == 256 && s.v == 4) go(k_rmsnorm_fwd<BF16, 4, 256, QUANT>, 256);
    else if (s.t == 256) go(k_rmsnorm_fwd<BF16, 8, 256, QUANT>, 256);
    else k_rmsnorm_fwd_any<BF16><<<(unsigned)a.rows, 256, 0, st>>>(a);
    profile_mark(st, "k_rmsnorm_fwd");
    return cudaGetLastError();
}
template <bool BF16>
cudaError_t fwd(const FwdArgs &a, bool vec, cudaStream_t st) {
    return a.quant == SSM_QUANT_ROW     ? fwd<BF16, SSM_QUANT_ROW>(a, vec, st)
           : a.quant == SSM_QUANT_BLOCK ? fwd<BF16, SSM_QUANT_BLOCK>(a, vec, st)
                                        : fwd<BF16, SSM_QUANT_NONE>(a, vec, st);
}

template <bool BF16>
cudaError_t bwd(const BwdArgs &a, bool vec, int blocks, float *dweight, cudaStream_t st) {
    constexpr int N = Io<BF16>::N;
    const Shape s = vec ? bwd_team(a.dim / N) : Shape{0, 0};
    cudaError_t e;
    auto go = [&](auto kern) { kern<<<blocks, BWD_BLOCK, 0, st>>>(a); };
    if (s.t == 32 && s.v == 1) go(k_rmsnorm_bwd<BF16, 1, 32>);
    else if (s.t == 32 && s.v == 2) go(k_rmsnorm_bwd<BF16, 2, 32>);
    else if (s.t == 32) go(k_rmsnorm_bwd<BF16, 4, 32>);
    else if (s.t == 64 && s.v == 3) go(k_rmsnorm_bwd<BF16, 3, 64>);
    else if (s.t == 64) go(k_rmsnorm_bwd<BF16, 4, 64>);
    else if (s.t == 128) go(k_rmsnorm_bwd<BF16, 4, 128>);
    else if (s.t == 256) go(k_rmsnorm_bwd<BF16, 4, 256>);
    else if (s.t == 512) go(k_rmsnorm_bwd<BF16, 4, 512>);
    else {
        if (a.part) {
            k_rmsnorm_dw_any<BF16><<<dim3((a.dim + 255) / 256, blocks), 256, 0, st>>>(a);
            profile_mark(st, "k_rmsnorm_dw_any");
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
        }
        k_rmsnorm_bwd_any<BF16><<<(unsigned)a.rows, 256, 0, st>>>(a);
    }
    profile_mark(st, "k_rmsnorm_bwd");
    if ((e = cudaGetLastError()) != cudaSuccess || !a.part) return e;
    k_rmsnorm_dw<<<(a.dim + 31) / 32, 256, 0, st>>>(a.part, dweight, a.dim, blocks);
    profile_mark(st, "k_rmsnorm_dw");
    return cudaGetLastError();
}

}  // namespace

cudaError_t rmsnorm_forward(const ssm_rmsnorm_desc_t &d, const void *x, const void *residual,
                            const float *weight, void *r, void *y, void *y8, float *scales,
                            float *rstd, cudaStream_t st) {
    const bool bf16 = d.dtype_io == SSM_BF16;
    const int n = bf16 ? 8 : 4;
    FwdArgs a = {x, residual, weight, r, y, (unsigned char *)y8, scales, rstd, d.rows, d.stride_x,
                 d.stride_residual, d.stride_r, d.stride_y, d.stride_y8, (int)d.dim, d.quant, d.eps};
    auto ok = [&](const void *p, int64_t s) { return !p || (al16(p) && s % n == 0); };
    const bool vec = d.dim % n == 0 && ok(x, d.stride_x) && ok(residual, d.stride_residual) &&
                     ok(r, d.stride_r) && ok(y, d.stride_y) && al16(weight) &&
                     (!y8 || ((uintptr_t)y8 % n == 0 && d.stride_y8 % n == 0));
    return bf16 ? fwd<true>(a, vec, st) : fwd<false>(a, vec, st);
}

size_t rmsnorm_bwd_bytes(const ssm_rmsnorm_desc_t &d) {
    return (((size_t)bwd_blocks(d) * (size_t)d.dim * 4) + 255) & ~(size_t)255;
}

cudaError_t rmsnorm_backward(const ssm_rmsnorm_desc_t &d, const void *dy, const void *r,
                             const float *weight, const float *rstd, const void *dr, void *dx,
                             float *dweight, float *ws, cudaStream_t st) {
    const bool bf16 = d.dtype_io == SSM_BF16;
    const int n = bf16 ? 8 : 4;
    BwdArgs a = {dy, r, dr, weight, rstd, dx, dweight ? ws : nullptr, d.rows, d.stride_dy,
                 d.stride_r, d.stride_dr, d.stride_dx, (int)d.dim};
    auto ok = [&](const void *p, int64_t s) { return !p || (al16(p) && s % n == 0); };
    const bool vec = d.dim % n == 0 && ok(dy, d.stride_dy) && ok(r, d.stride_r) &&
                     ok(dr, d.stride_dr) && ok(dx, d.stride_dx) && al16(weight);
    const int blocks = bwd_blocks(d);
    return bf16 ? bwd<true>(a, vec, blocks, dweight, st) : bwd<false>(a, vec, blocks, dweight, st);
}

}  // namespace ssm
