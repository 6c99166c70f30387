// Gated linear recurrence, forward, backward and one-token form (declared in
// include/gdn.h): one thread per sequence and channel, token after token.
#include <vector>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kTile = 128;  // tokens between two saved states

struct LinrecParams {
    int64_t T, BT, D, N;
    int64_t xs, gs, os, dxs, dgs;
    const int32_t *cu;
    const void *x, *g, *dy;
    const float *h0, *dhT;
    void *o, *dx, *dg;
    float *hT, *dh0, *states;
};

__device__ __forceinline__ float ld(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p, int64_t i) {
    return __bfloat162float(p[i]);
}
__device__ __forceinline__ void st(float *p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, int64_t i, float x) {
    p[i] = __float2bfloat16_rn(x);
}

// Tokens [t0, t1) of sequence n, inside the buffers whatever cu holds.
__device__ __forceinline__ void bounds(const LinrecParams &p, int64_t n, int64_t *t0, int64_t *t1) {
    if (!p.cu) {
        *t0 = n * p.T;
        *t1 = *t0 + p.T;
        return;
    }
    const int64_t a = p.cu[n], b = p.cu[n + 1];
    *t0 = a < 0 ? 0 : a > p.BT ? p.BT : a;
    *t1 = b < *t0 ? *t0 : b > p.BT ? p.BT : b;
}

// Saved states: one for every 128 tokens, counted from the start of a dense row or of the
// packed row.  `tile0` is the index of the first one of the row that starts at token `row0`.
__device__ __forceinline__ void tiles(const LinrecParams &p, int64_t n, int64_t *row0, int64_t *tile0) {
    *row0 = p.cu ? 0 : n * p.T;
    *tile0 = p.cu ? 0 : n * ((p.T + kTile - 1) / kTile);
}

template <bool COMP>
__device__ __forceinline__ void gate(float g, float *a, float *w) {
    *a = expf(g);
    *w = COMP ? -expm1f(g) : 1.f;
}

template <typename T, typename G, bool COMP>
__global__ void __launch_bounds__(128) linrec_fwd_kernel(LinrecParams p) {
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x, n = blockIdx.x;
    if (c >= p.D) return;
    int64_t t0, t1;
    bounds(p, n, &t0, &t1);
    int64_t row0, tile0;
    tiles(p, n, &row0, &tile0);
    const T *x = static_cast<const T *>(p.x);
    const G *g = static_cast<const G *>(p.g);
    T *o = static_cast<T *>(p.o);
    float h = p.h0 ? p.h0[n * p.D + c] : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        if (p.states && t > t0 && (t - row0) % kTile == 0)
            p.states[(tile0 + (t - row0) / kTile) * p.D + c] = h;
        float a, w;
        gate<COMP>(ld(g, t * p.gs + c), &a, &w);
        h = fmaf(a, h, w * ld(x, t * p.xs + c));
        if (o) st(o, t * p.os + c, h);
    }
    if (p.hT) p.hT[n * p.D + c] = h;
}

template <typename T, typename G, bool COMP>
__global__ void __launch_bounds__(128) linrec_bwd_kernel(LinrecParams p) {
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x, n = blockIdx.x;
    if (c >= p.D) return;
    int64_t t0, t1;
    bounds(p, n, &t0, &t1);
    int64_t row0, tile0;
    tiles(p, n, &row0, &tile0);
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    const G *g = static_cast<const G *>(p.g);
    T *dx = static_cast<T *>(p.dx);
    G *dg = static_cast<G *>(p.dg);
    float carry = p.dhT ? p.dhT[n * p.D + c] : 0.f;  // gradient of the state after the token
    float before[kTile];                             // states entering a tile's tokens
    for (int64_t end = t1; end > t0;) {
        const int64_t tile = (end - 1 - row0) / kTile;
        int64_t begin = row0 + tile * kTile;
        if (begin < t0) begin = t0;
        float h = begin == t0 ? (p.h0 ? p.h0[n * p.D + c] : 0.f) : p.states[(tile0 + tile) * p.D + c];
        float a, w;
        for (int64_t t = begin; t < end; ++t) {
            before[t - begin] = h;
            gate<COMP>(ld(g, t * p.gs + c), &a, &w);
            h = fmaf(a, h, w * ld(x, t * p.xs + c));
        }
        for (int64_t t = end - 1; t >= begin; --t) {
            gate<COMP>(ld(g, t * p.gs + c), &a, &w);
            const float e = ld(dy, t * p.os + c) + carry;
            carry = a * e;
            st(dx, t * p.dxs + c, w * e);
            st(dg, t * p.dgs + c,
               carry * (COMP ? before[t - begin] - ld(x, t * p.xs + c) : before[t - begin]));
        }
        end = begin;
    }
    if (p.dh0) p.dh0[n * p.D + c] = carry;
}

template <typename T, typename G, bool COMP>
__global__ void __launch_bounds__(128) linrec_decode_kernel(LinrecParams p, float *state) {
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x, n = blockIdx.x;
    if (c >= p.D) return;
    const T *x = static_cast<const T *>(p.x);
    const G *g = static_cast<const G *>(p.g);
    T *o = static_cast<T *>(p.o);
    float h = state[n * p.D + c];
    for (int64_t t = n * p.T; t < (n + 1) * p.T; ++t) {
        float a, w;
        gate<COMP>(ld(g, t * p.gs + c), &a, &w);
        h = fmaf(a, h, w * ld(x, t * p.xs + c));
        st(o, t * p.os + c, h);
    }
    state[n * p.D + c] = h;
}

enum class Pass { kFwd, kBwd, kDecode };

template <typename T, typename G, bool COMP>
cudaError_t launch_typed(const LinrecParams &p, Pass pass, float *state, cudaStream_t s) {
    const dim3 grid((unsigned)p.N, (unsigned)((p.D + 127) / 128));
    if (pass == Pass::kFwd)
        GDN_LAUNCH(kKLinrecFwd, s, linrec_fwd_kernel<T, G, COMP><<<grid, 128, 0, s>>>(p));
    else if (pass == Pass::kBwd)
        GDN_LAUNCH(kKLinrecBwd, s, linrec_bwd_kernel<T, G, COMP><<<grid, 128, 0, s>>>(p));
    else
        GDN_LAUNCH(kKLinrecDecode, s, linrec_decode_kernel<T, G, COMP><<<grid, 128, 0, s>>>(p, state));
    return cudaSuccess;
}

template <typename T, typename G>
cudaError_t launch_comp(const LinrecParams &p, bool comp, Pass pass, float *state, cudaStream_t s) {
    return comp ? launch_typed<T, G, true>(p, pass, state, s)
                : launch_typed<T, G, false>(p, pass, state, s);
}

cudaError_t launch(const gdn_linrec_desc *d, const LinrecParams &p, Pass pass, float *state,
                   cudaStream_t s) {
    const bool comp = d->flags & GDN_LINREC_COMPLEMENT;
    if (d->dtype == GDN_FP32) return launch_comp<float, float>(p, comp, pass, state, s);
    if (d->g_dtype == GDN_FP32) return launch_comp<__nv_bfloat16, float>(p, comp, pass, state, s);
    return launch_comp<__nv_bfloat16, __nv_bfloat16>(p, comp, pass, state, s);
}

// Checks that need no pointers; fills the sizes and strides.
gdn_status describe(const gdn_linrec_desc *d, LinrecParams *p) {
    if (!d) return GDN_ERR_INVALID_ARG;
    if (d->B < 1 || d->T < 0 || d->D < 1 || d->n_seqs < 0) return GDN_ERR_INVALID_ARG;
    if (d->dtype != GDN_BF16 && d->dtype != GDN_FP32) return GDN_ERR_UNSUPPORTED;
    if (d->g_dtype != GDN_FP32 && d->g_dtype != d->dtype) return GDN_ERR_UNSUPPORTED;
    if (d->reserved != 0 || (d->flags & ~GDN_LINREC_COMPLEMENT)) return GDN_ERR_INVALID_ARG;
    if (d->n_seqs > 0 && d->B != 1) return GDN_ERR_INVALID_ARG;
    // range checks before any product is formed (no signed overflow on huge inputs)
    constexpr int64_t kLim = int64_t(1) << 31;
    if (d->B >= kLim || d->T >= kLim || d->T >= kLim / d->B || d->D > (1 << 20) ||
        d->n_seqs >= kLim)
        return GDN_ERR_INVALID_ARG;
    p->T = d->T;
    p->BT = d->B * d->T;
    p->D = d->D;
    p->N = d->n_seqs > 0 ? d->n_seqs : d->B;
    const int64_t in[] = {d->x_stride, d->g_stride, d->o_stride, d->dx_stride, d->dg_stride};
    int64_t *out[] = {&p->xs, &p->gs, &p->os, &p->dxs, &p->dgs};
    for (int i = 0; i < 5; ++i) {
        if (in[i] != 0 && (in[i] < d->D || in[i] >= kLim)) return GDN_ERR_INVALID_ARG;
        *out[i] = in[i] ? in[i] : d->D;
    }
    return GDN_OK;
}

bool mis(const void *p, size_t a = 16) { return p && (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// Rows of at most 128 tokens need none: every sequence starts within its tile.
size_t states_bytes(const LinrecParams &p) {
    const size_t rows = p.T > kTile ? (size_t)(p.BT / p.T) : 0;
    const size_t b = rows * ((p.T + kTile - 1) / kTile) * p.D * sizeof(float);
    return b < 256 ? 256 : (b + 255) / 256 * 256;
}

// Host-side check of cu_seqlens (the rules of gdn_fwd).
gdn_status check_seqlens(const gdn_linrec_desc *d, const int32_t *cu_dev, const int32_t *cu_host,
                         cudaStream_t s) {
    if (d->n_seqs == 0) return cu_dev || cu_host ? GDN_ERR_INVALID_ARG : GDN_OK;
    if (!cu_dev) return GDN_ERR_INVALID_ARG;
    if (mis(cu_dev, 4)) return GDN_ERR_ALIGNMENT;
    std::vector<int32_t> copy;
    if (!cu_host) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) return GDN_ERR_CUDA;
        if (cap != cudaStreamCaptureStatusNone) return GDN_ERR_INVALID_ARG;
        copy.resize((size_t)d->n_seqs + 1);
        if (cudaMemcpyAsync(copy.data(), cu_dev, sizeof(int32_t) * copy.size(),
                            cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return GDN_ERR_CUDA;
        cu_host = copy.data();
    }
    if (cu_host[0] != 0 || cu_host[d->n_seqs] != d->T) return GDN_ERR_INVALID_ARG;
    for (int64_t n = 0; n < d->n_seqs; ++n)
        if (cu_host[n + 1] < cu_host[n]) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" {

size_t gdn_linrec_states_size(const gdn_linrec_desc *desc) {
    gdn::LinrecParams p{};
    return gdn::describe(desc, &p) == GDN_OK ? gdn::states_bytes(p) : 0;
}

gdn_status gdn_linrec_fwd(const gdn_linrec_desc *desc, const void *x, const void *g,
                          const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                          const float *h0, void *o, float *hT, float *states, void *stream) {
    using namespace gdn;
    LinrecParams p{};
    gdn_status st = describe(desc, &p);
    if (st != GDN_OK) return st;
    if (p.BT > 0 && (!x || !g || !o)) return GDN_ERR_INVALID_ARG;
    if (hT && hT == h0) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, g, h0, o, hT, states};
    for (const void *q : ptrs)
        if (mis(q)) return GDN_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = check_seqlens(desc, cu_seqlens, cu_seqlens_host, s)) != GDN_OK) return st;
    p.cu = desc->n_seqs > 0 ? cu_seqlens : nullptr;
    p.x = x, p.g = g, p.h0 = h0, p.o = o, p.hT = hT, p.states = states;
    arm_planted_failure();
    return launch(desc, p, Pass::kFwd, nullptr, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linrec_bwd(const gdn_linrec_desc *desc, const void *x, const void *g,
                          const int32_t *cu_seqlens, const int32_t *cu_seqlens_host,
                          const float *h0, const void *do_, const float *dhT, void *dx, void *dg,
                          float *dh0, const float *states, void *workspace,
                          size_t workspace_bytes, void *stream) {
    using namespace gdn;
    LinrecParams p{};
    gdn_status st = describe(desc, &p);
    if (st != GDN_OK) return st;
    if (p.BT > 0 && (!x || !g || !do_ || !dx || !dg)) return GDN_ERR_INVALID_ARG;
    if (dh0 && dh0 == dhT) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, g, h0, do_, dhT, dx, dg, dh0, states};
    for (const void *q : ptrs)
        if (mis(q)) return GDN_ERR_ALIGNMENT;
    if (!states) {
        if (!workspace) return GDN_ERR_WORKSPACE;
        if (mis(workspace, 256)) return GDN_ERR_ALIGNMENT;
        if (workspace_bytes < states_bytes(p)) return GDN_ERR_WORKSPACE;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((st = check_seqlens(desc, cu_seqlens, cu_seqlens_host, s)) != GDN_OK) return st;
    p.cu = desc->n_seqs > 0 ? cu_seqlens : nullptr;
    p.x = x, p.g = g, p.h0 = h0, p.dy = do_, p.dhT = dhT, p.dx = dx, p.dg = dg, p.dh0 = dh0;
    p.states = const_cast<float *>(states);
    arm_planted_failure();
    if (!states && p.T > kTile) {
        p.states = static_cast<float *>(workspace);
        if (launch(desc, p, Pass::kFwd, nullptr, s) != cudaSuccess) return GDN_ERR_CUDA;
    }
    return launch(desc, p, Pass::kBwd, nullptr, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_linrec_decode(const gdn_linrec_desc *desc, const void *x, const void *g,
                             float *state, void *o, void *stream) {
    using namespace gdn;
    LinrecParams p{};
    gdn_status st = describe(desc, &p);
    if (st != GDN_OK) return st;
    if (desc->T < 1 || desc->n_seqs != 0) return GDN_ERR_INVALID_ARG;
    if (!x || !g || !state || !o) return GDN_ERR_INVALID_ARG;
    const void *ptrs[] = {x, g, state, o};
    for (const void *q : ptrs)
        if (mis(q)) return GDN_ERR_ALIGNMENT;
    p.x = x, p.g = g, p.o = o;
    arm_planted_failure();
    return launch(desc, p, Pass::kDecode, state, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
