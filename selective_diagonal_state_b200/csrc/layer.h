// Host-side declarations shared by the operators around the mixer (rmsnorm.cu, rope.cu,
// linattn*.cu) and their C entry points (abi_layer.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ssm_scan.h"

namespace ssm {

// Streaming multiprocessors of a B200, in the rules that also size workspaces: those must give the same
// whichever device is current when a caller asks for the size.  Grids alone go by sm_count().
constexpr int SMS = 148;
int sm_count();
void profile_mark(cudaStream_t st, const char *name);
long long abi_wait_limit();   // ssm_scan_set_wait_limit's

cudaError_t rmsnorm_forward(const ssm_rmsnorm_desc_t &d, const void *x, const void *residual,
                            const float *weight, void *r, void *y, void *y8, float *scales,
                            float *rstd, cudaStream_t st);
size_t rmsnorm_bwd_bytes(const ssm_rmsnorm_desc_t &d);
cudaError_t rmsnorm_backward(const ssm_rmsnorm_desc_t &d, const void *dy, const void *r,
                             const float *weight, const float *rstd, const void *dr, void *dx,
                             float *dweight, float *ws, cudaStream_t st);

// sign: +1 the rotation, -1 the opposite one
cudaError_t rope_rotate(const ssm_rope_desc_t &d, const void *q, const void *k, const double *freq,
                        const int64_t *positions, void *q_out, void *k_out, float sign,
                        cudaStream_t st);

// ---- linear attention ------------------------------------------------------------------
// One walk along the sequences: for every batch row and head, with lam = e^{log_decay},
//   forward:  S <- lam S + write k v^T,  o = read a S        (tokens first to last)
//   reverse:  S <- S + write k v^T,  o = read a S,  S <- lam S   (last to first)
// The output and every gradient of the operator is such a walk (see linattn.cu).
struct LaWalk {
    const void *a, *k, *v;            // [B][L][heads][da], [da], [dc]
    void *o;                          // [B][L][heads][dc]; null: state only
    long long sa[3], sk[3], sv[3], so[3];   // batch, time, head
    int rep_a, rep_k, rep_v;          // heads that share one of the operand's
    int da, dc;
    const float *s_in;                // entering state (null: zero) and leaving state (may
    float *s_out;                     // be null), element (a, c) at a * st_a + c * st_c
    int st_a, st_c;                   // from (b H + h) da dc
    float read, write;
    int rev, o_f32;                   // o_f32: o is fp32 whatever the I/O type
};
struct LaArgs {
    int B, L, H, bf16;
    const float *log_decay;
    const int *lengths;
    int nwalk;
    LaWalk w[3];
};
cudaError_t la_recurrent(const LaArgs &p, cudaStream_t st);
// the walks on tensor cores (linattn_tc.cu)
bool la_chunked_sizes(int bf16, int da, int dc);
int la_segments(long long L, long long items);
bool la_chunked(const LaArgs &p, int nseg, float *const *seg, cudaStream_t st, cudaError_t *err);
int la_error_take();
// sum of the `rep` heads that share a key / value head, fp32 [B][L][H][d] -> out
cudaError_t la_group_sum(const float *in, void *out, const long long *so, int B, int L, int H,
                         int rep, int d, const int *lengths, int bf16, cudaStream_t st);
cudaError_t la_step(const ssm_linattn_desc_t &d, const void *q, const void *k, const void *v,
                    const float *log_decay, float *state, void *o, cudaStream_t st);
constexpr int LA_MAX_DIM = 256;

}  // namespace ssm
