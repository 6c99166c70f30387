// Normalisation of q and k per token and head with the position rotation, and its
// gradients (declared in include/gdn.h): one warp per row, the row in shared memory.
#include <cmath>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kMaxD = 256, kWarps = 8, kSlots = 592;

struct QkParams {
    int64_t tokens;
    int32_t T, d, rot, norm, interleaved;
    float c, eps;
    const int32_t *pos;
    const float *inv_freq;
    // [0]: q, [1]: k
    int32_t heads[2];
    int64_t xs[2], ys[2], dxs[2];
    const void *x[2], *dy[2];
    const float *w[2];
    void *y[2], *dx[2];
    float *dw[2], *part;
};

__device__ __forceinline__ float ld(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p, int64_t i) {
    return __bfloat162float(p[i]);
}
__device__ __forceinline__ void st(float *p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, int64_t i, float x) {
    p[i] = __float2bfloat16_rn(x);
}

__device__ __forceinline__ float total(float s) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    return s;
}

// cos and sin of pos * freq: the angle in turns in 64 bits, its fraction in 32.
__device__ __forceinline__ void turn(int32_t pos, float freq, float *c, float *s) {
    const double t = (double)pos * (double)freq * 0.15915494309189533577;
    sincospif(2.f * (float)(t - rint(t)), s, c);
}

// Value i of the row: its pair's other value, its angle's index (-1: not turned) and the
// sign of sin at the other value.
__device__ __forceinline__ void partner(const QkParams &p, int i, int *j, int *f, float *sign) {
    const int half = p.rot / 2;
    *f = -1, *j = i, *sign = 0.f;
    if (i >= p.rot) return;
    const bool first = p.interleaved ? !(i & 1) : i < half;
    *j = p.interleaved ? i ^ 1 : first ? i + half : i - half;
    *f = p.interleaved ? i / 2 : first ? i : i - half;
    *sign = first ? -1.f : 1.f;
}

__device__ __forceinline__ float scale_of(const QkParams &p, float sum) {
    if (p.norm == GDN_NORM_NONE) return 1.f;
    const float m = fmaf(p.c, sum, p.eps);
    return m > 0.f ? 1.f / sqrtf(m) : m == 0.f ? 0.f : m;
}

template <typename T, bool BWD>
__global__ void __launch_bounds__(32 * kWarps) qk_kernel(QkParams p) {
    __shared__ float rows[kWarps][kMaxD], sums[kWarps][kMaxD];
    const int l = threadIdx.x & 31, wi = threadIdx.x >> 5, which = blockIdx.y;
    const int64_t n = p.tokens * p.heads[which];
    const T *x = static_cast<const T *>(p.x[which]), *dy = static_cast<const T *>(p.dy[which]);
    T *out = static_cast<T *>(BWD ? p.dx[which] : p.y[which]);
    const int64_t os = BWD ? p.dxs[which] : p.ys[which];
    const float *w = p.w[which];
    float *row = rows[wi], acc[kMaxD / 32] = {};
    for (int64_t r = (int64_t)blockIdx.x * kWarps + wi; r < n; r += (int64_t)gridDim.x * kWarps) {
        const int64_t tok = r / p.heads[which];
        const int h = (int)(r % p.heads[which]);
        const int32_t pos = p.pos ? p.pos[tok] : (int32_t)(tok % p.T);
        const T *xr = x + tok * p.xs[which] + (int64_t)h * p.d;
        float s = 0.f;
        for (int i = l; i < p.d; i += 32) s = fmaf(ld(xr, i), ld(xr, i), s);
        const float inv = scale_of(p, total(s));
        for (int i = l; i < p.d; i += 32)
            row[i] = BWD ? ld(dy, tok * p.ys[which] + (int64_t)h * p.d + i)
                         : ld(xr, i) * inv * (w ? w[i] : 1.f);
        __syncwarp();
        T *o = out + tok * os + (int64_t)h * p.d;
        float u[kMaxD / 32], dot = 0.f;
        for (int i = l, m = 0; i < p.d; i += 32, ++m) {
            int j, f;
            float sign, c = 1.f, sn = 0.f;
            partner(p, i, &j, &f, &sign);
            if (f >= 0) turn(pos, p.inv_freq[f], &c, &sn);
            if (BWD) {
                u[m] = fmaf(row[j], -sign * sn, row[i] * c);
                const float xn = ld(xr, i) * inv;
                acc[m] = fmaf(u[m], xn, acc[m]);
                u[m] *= w ? w[i] : 1.f;
                dot = fmaf(u[m], xn, dot);
            } else {
                st(o, i, fmaf(row[j], sign * sn, row[i] * c));
            }
        }
        if (BWD) {
            dot = p.norm == GDN_NORM_NONE ? 0.f : p.c * total(dot);
            for (int i = l, m = 0; i < p.d; i += 32, ++m)
                st(o, i, inv * fmaf(-(ld(xr, i) * inv), dot, u[m]));
        }
        __syncwarp();
    }
    if (BWD && p.dw[which]) {
        for (int i = l, m = 0; i < p.d; i += 32, ++m) sums[wi][i] = acc[m];
        __syncthreads();
        for (int i = threadIdx.x; i < p.d; i += 32 * kWarps) {
            float s = 0.f;
            for (int k = 0; k < kWarps; ++k) s += sums[k][i];
            p.part[((int64_t)which * kSlots + blockIdx.x) * kMaxD + i] = s;
        }
    }
}

__global__ void __launch_bounds__(kMaxD) qk_dw_kernel(QkParams p, int blocks) {
    const int i = threadIdx.x, which = blockIdx.x;
    if (i >= p.d || !p.dw[which]) return;
    float s = 0.f;
    for (int b = 0; b < blocks; ++b) s += p.part[((int64_t)which * kSlots + b) * kMaxD + i];
    p.dw[which][i] = s;
}

template <typename T>
cudaError_t launch(const QkParams &p, bool bwd, cudaStream_t s) {
    const int64_t most = p.tokens * (p.heads[0] > p.heads[1] ? p.heads[0] : p.heads[1]);
    const int64_t want = (most + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)(want < 1 ? 1 : want < kSlots ? want : kSlots), 2);
    if (!bwd) {
        if (p.tokens) GDN_LAUNCH(kKQkRope, s, qk_kernel<T, false><<<grid, 32 * kWarps, 0, s>>>(p));
        return cudaSuccess;
    }
    if (p.tokens || p.dw[0] || p.dw[1])
        GDN_LAUNCH(kKQkRopeBwd, s, qk_kernel<T, true><<<grid, 32 * kWarps, 0, s>>>(p));
    if (p.dw[0] || p.dw[1])
        GDN_LAUNCH(kKQkRopeDw, s, qk_dw_kernel<<<2, kMaxD, 0, s>>>(p, (int)grid.x));
    return cudaSuccess;
}

size_t workspace_bytes_needed() { return sizeof(float) * 2 * kSlots * kMaxD; }

// Checks that need no pointers; fills the sizes and strides.
gdn_status describe(const gdn_qk_desc *d, QkParams *p) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->dtype != GDN_BF16 && d->dtype != GDN_FP32) return GDN_ERR_UNSUPPORTED;
    if (d->norm < GDN_NORM_NONE || d->norm > GDN_NORM_RMS) return GDN_ERR_UNSUPPORTED;
    if (d->d < 2 || d->d > kMaxD || d->d % 2) return GDN_ERR_UNSUPPORTED;
    if (d->rot < 0 || d->rot > d->d || d->rot % 2) return GDN_ERR_INVALID_ARG;
    if (d->flags & ~GDN_QK_INTERLEAVED) return GDN_ERR_INVALID_ARG;
    if (!(d->eps >= 0.f) || std::isinf(d->eps)) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->Hq < 1 || d->Hq > 65535 || d->Hk < 1 || d->Hk > 65535)
        return GDN_ERR_INVALID_ARG;
    // range checks before any product is formed (no signed overflow on huge inputs)
    constexpr int64_t kLim = int64_t(1) << 31;
    if (d->B >= kLim || d->T >= kLim || d->T >= kLim / d->B) return GDN_ERR_INVALID_ARG;
    const int64_t heads[] = {d->Hq, d->Hk};
    const int64_t in[][2] = {{d->q_stride, d->k_stride}, {d->qo_stride, d->ko_stride},
                             {d->dq_stride, d->dk_stride}};
    int64_t *out[] = {p->xs, p->ys, p->dxs};
    for (int j = 0; j < 3; ++j)
        for (int i = 0; i < 2; ++i) {
            const int64_t width = heads[i] * d->d;
            if (in[j][i] != 0 && (in[j][i] < width || in[j][i] >= kLim)) return GDN_ERR_INVALID_ARG;
            out[j][i] = in[j][i] ? in[j][i] : width;
        }
    p->tokens = d->B * d->T;
    p->T = (int32_t)d->T;
    p->d = (int32_t)d->d;
    p->rot = (int32_t)d->rot;
    p->norm = d->norm;
    p->interleaved = d->flags & GDN_QK_INTERLEAVED;
    p->c = d->norm == GDN_NORM_RMS ? 1.f / (float)d->d : 1.f;
    p->eps = d->eps;
    p->heads[0] = (int32_t)d->Hq;
    p->heads[1] = (int32_t)d->Hk;
    return GDN_OK;
}

bool mis(const void *p, size_t a = 16) { return p && (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_qk_norm_rope_fwd(const gdn_qk_desc *desc, const void *q, const void *k,
                                const int32_t *positions, const float *inv_freq,
                                const float *q_weight, const float *k_weight, void *qo, void *ko,
                                void *stream) {
    using namespace gdn;
    QkParams p{};
    gdn_status st = describe(desc, &p);
    if (st != GDN_OK) return st;
    if (p.tokens > 0 && (!q || !k || !qo || !ko)) return GDN_ERR_INVALID_ARG;
    if (p.rot > 0 && !inv_freq) return GDN_ERR_INVALID_ARG;
    const void *wide[] = {q, k, qo, ko}, *narrow[] = {positions, inv_freq, q_weight, k_weight};
    for (const void *a : wide)
        if (mis(a)) return GDN_ERR_ALIGNMENT;
    for (const void *a : narrow)
        if (mis(a, 4)) return GDN_ERR_ALIGNMENT;
    p.pos = positions, p.inv_freq = inv_freq;
    p.x[0] = q, p.x[1] = k, p.y[0] = qo, p.y[1] = ko, p.w[0] = q_weight, p.w[1] = k_weight;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    arm_planted_failure();
    const cudaError_t e = desc->dtype == GDN_BF16 ? launch<__nv_bfloat16>(p, false, s)
                                                  : launch<float>(p, false, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_rope_bwd_workspace_size(const gdn_qk_desc *desc) {
    gdn::QkParams p{};
    return gdn::describe(desc, &p) == GDN_OK ? gdn::workspace_bytes_needed() : 0;
}

gdn_status gdn_qk_norm_rope_bwd(const gdn_qk_desc *desc, const void *q, const void *k,
                                const int32_t *positions, const float *inv_freq,
                                const float *q_weight, const float *k_weight, const void *dqo,
                                const void *dko, void *dq, void *dk, float *dq_weight,
                                float *dk_weight, void *workspace, size_t workspace_bytes,
                                void *stream) {
    using namespace gdn;
    QkParams p{};
    gdn_status st = describe(desc, &p);
    if (st != GDN_OK) return st;
    if (p.tokens > 0 && (!q || !k || !dqo || !dko || !dq || !dk)) return GDN_ERR_INVALID_ARG;
    if (p.rot > 0 && !inv_freq) return GDN_ERR_INVALID_ARG;
    const void *wide[] = {q, k, dqo, dko, dq, dk};
    const void *narrow[] = {positions, inv_freq, q_weight, k_weight, dq_weight, dk_weight};
    for (const void *a : wide)
        if (mis(a)) return GDN_ERR_ALIGNMENT;
    for (const void *a : narrow)
        if (mis(a, 4)) return GDN_ERR_ALIGNMENT;
    if (dq_weight || dk_weight) {
        if (!workspace) return GDN_ERR_WORKSPACE;
        if (mis(workspace, 256)) return GDN_ERR_ALIGNMENT;
        if (workspace_bytes < workspace_bytes_needed()) return GDN_ERR_WORKSPACE;
    }
    p.pos = positions, p.inv_freq = inv_freq;
    p.x[0] = q, p.x[1] = k, p.dy[0] = dqo, p.dy[1] = dko, p.dx[0] = dq, p.dx[1] = dk;
    p.w[0] = q_weight, p.w[1] = k_weight, p.dw[0] = dq_weight, p.dw[1] = dk_weight;
    p.part = static_cast<float *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    arm_planted_failure();
    const cudaError_t e = desc->dtype == GDN_BF16 ? launch<__nv_bfloat16>(p, true, s)
                                                  : launch<float>(p, true, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
