// Gated linear recurrence, forward, backward and one-token form (declared in
// include/gdn.h).
//
// A sequence's map over any span of tokens is affine per channel, h' = A h + X with
// A the product of the span's factors, and the reverse map of the gradients is
// r' = A r + Y with the same A; spans join by (A2, X2)(A1, X1) = (A2 A1, A2 X1 + X2).
// So a CTA takes 64 channels (two per lane) and 64 tokens at a time, 8 tokens per warp in
// registers: each warp forms its span's A and X (and Y), the 8 spans are joined in
// shared memory, and the warp then runs its tokens from the state that enters them.  A
// cluster of up to 16 CTAs takes consecutive tiles of the same channels and joins the
// tiles' maps over distributed shared memory, one cluster barrier per step; every CTA
// folds all of them, so each keeps the state that enters the next step.  Joins go in
// token order from the state itself, so results do not depend on the cluster's size or
// on timing.  The data is read once: the next steps' tiles are already on their way by
// cp.async, each warp copying the rows it will use.
//
// A start of a sequence inside a span drops what comes before it by selection (not by a
// factor of 0), so that no infinity or NaN crosses; padded tokens are zeros (factor
// exp(0) = 1, input 0), which is the identity map in both directions.
//
// The backward runs the tiles from the last to the first.  It needs the states that
// enter each token: the forward leaves the state entering every 64th token (4 / 64 bytes
// per element), from which a tile recomputes its own.
#include <atomic>
#include <vector>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kSpan = 8;               // tokens per warp
constexpr int kWarps = 8;
constexpr int kTile = kSpan * kWarps;  // tokens per CTA and step, and between saved states
constexpr int kCh = 64;                // channels per CTA
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 16;
constexpr int kSms = 148, kPerSm = 2;
constexpr size_t kSmemSm = 227 * 1024, kSmemMax = 196 * 1024, kSmemStatic = 31 * 1024;  // dynamic, static and reserved

struct LinrecParams {
    int64_t T, BT, D, N;
    int64_t xs, gs, os, dxs, dgs;
    int64_t streams, rows_per_stream, tiles;  // a stream: one dense row, several short ones, or the packed row
    int32_t slabs, cluster, stages, wide, even;
    const int32_t *cu;
    const void *x, *g, *dy;
    const float *h0, *dhT;
    void *o, *dx, *dg;
    float *hT, *dh0, *states;
};

// ---------------------------------------------------------------- small pieces
__device__ __forceinline__ float2 load2(const float *p, int lane) {
    return reinterpret_cast<const float2 *>(p)[lane];
}
__device__ __forceinline__ float2 load2(const __nv_bfloat16 *p, int lane) {
    return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(p)[lane]);
}
__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put2(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void put2(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(v);
}
// Two adjacent channels of a row; n of them (0, 1 or 2) exist.
template <bool EVEN, typename E>
__device__ __forceinline__ void store_pair(E *p, float2 v, int n) {
    if (EVEN) {
        if (n) put2(p, v);
    } else {
        if (n > 0) put(p, v.x);
        if (n > 1) put(p + 1, v.y);
    }
}
// A row of states ([...][D] fp32, any alignment); zeros for a NULL array.
__device__ __forceinline__ float2 load_state(const float *p, int64_t at, int n) {
    float2 v = make_float2(0.f, 0.f);
    if (p && n > 0) v.x = p[at];
    if (p && n > 1) v.y = p[at + 1];
    return v;
}
__device__ __forceinline__ void store_state(float *p, int64_t at, float2 v, int n) {
    if (p && n > 0) p[at] = v.x;
    if (p && n > 1) p[at + 1] = v.y;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }

// a = exp(g), and the write strength 1 or 1 - a; the latter without the cancellation.
template <bool COMP>
__device__ __forceinline__ void gate(float2 g, float2 *a, float2 *w) {
    *a = make_float2(__expf(g.x), __expf(g.y));
    *w = COMP ? make_float2(-expm1f(g.x), -expm1f(g.y)) : make_float2(1.f, 1.f);
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
template <int N>  // copies `bytes` (0 .. N) of N, the rest zeros
__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes) {
    if (N == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `pending` of this thread's groups are unfinished.
__device__ __forceinline__ void copy_wait(int pending) {
    switch (pending) {
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    case 7: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    }
}

// A warp's copy of 8 tokens x 64 channels; `rows` and `cols` of them exist, the rest become
// zeros.  wide: 16-byte pieces (rows 16-byte aligned; the last piece may be partial), else 4
// bytes (fp32, or bf16 with even rows), else one bf16 after another.
template <typename E>
__device__ __forceinline__ void copy_rows(E *dst, const E *src, int64_t stride, int rows, int cols,
                                          int wide, int even, int lane) {
    if (wide) {
        constexpr int kPer = 16 / sizeof(E), kPieces = kCh / kPer, kRows = 32 / kPieces;
        const int c = lane % kPieces * kPer;
        const int here = (cols - c) * (int)sizeof(E), bytes = here < 0 ? 0 : here > 16 ? 16 : here;
#pragma unroll
        for (int i = 0; i < kSpan; i += kRows) {
            const int r = i + lane / kPieces, n = r < rows ? bytes : 0;
            copy_async<16>(dst + r * kCh + c, n ? src + r * stride + c : src, n);
        }
    } else if (sizeof(E) == 4 || even) {
        constexpr int kPer = 4 / sizeof(E);
#pragma unroll
        for (int r = 0; r < kSpan; ++r)
#pragma unroll
            for (int c = lane * kPer; c < kCh; c += 32 * kPer) {
                const bool in = r < rows && c < cols;
                copy_async<4>(dst + r * kCh + c, in ? src + r * stride + c : src, in ? 4 : 0);
            }
    } else {
        E v[kSpan][2];
#pragma unroll
        for (int r = 0; r < kSpan; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = lane + 32 * j;
                v[r][j] = r < rows && c < cols ? src[r * stride + c] : E(0.f);
            }
#pragma unroll
        for (int r = 0; r < kSpan; ++r)
#pragma unroll
            for (int j = 0; j < 2; ++j) dst[r * kCh + lane + 32 * j] = v[r][j];
    }
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void cluster_store(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ void cluster_store(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// ---------------------------------------------------------------- sequences of a stream
// The sequence that holds a token, for a whole warp: index n, tokens [beg, end) of the stream.
struct Seq {
    int64_t n;
    int beg, end;
};

// Moves s to the sequence that holds token t (0 <= t < S).  Packed: the largest n with cu[n]
// <= t, searched near s first and then 33 ways at a time.  Only cu[1 .. N - 1] are trusted as
// far as indices go; the bounds are forced around t whatever they hold.
__device__ __forceinline__ void seek(const LinrecParams &p, int64_t first, int S, int t, int lane, Seq *s) {
    if (t >= s->beg && t < s->end) return;
    if (!p.cu) {
        const int T = (int)p.T, k = t / T;
        s->n = first + k, s->beg = k * T, s->end = s->beg + T;
        return;
    }
    int lo = 0, hi = (int)p.N;  // cu[lo] <= t < cu[hi]
    int step = 1;
    if (t >= s->end) {
        lo = (int)s->n;
    } else {
        hi = s->n > 0 ? (int)s->n : 1;
        const int at = hi - 1 - lane;
        const bool after = at > lo && p.cu[at] > t;
        const int cnt = __ffs(~__ballot_sync(0xffffffffu, after)) - 1;  // -1: all 32
        if (cnt >= 0) {
            hi -= cnt;
            lo = hi - 1;
        } else {
            hi -= 32;
            step = (hi - lo + 32) / 33;
        }
    }
    while (hi - lo > 1) {
        const int64_t at = lo + (int64_t)(lane + 1) * step;
        const bool before = at < hi && p.cu[at] <= t;
        const uint32_t b = __ballot_sync(0xffffffffu, before);
        const int cnt = b == 0xffffffffu ? 32 : __ffs(~b) - 1;
        const int64_t end = lo + (int64_t)(cnt + 1) * step;
        lo += cnt * step;
        if (cnt < 32 && end < hi) hi = (int)end;
        step = (hi - lo + 32) / 33;
    }
    const int b = lo > 0 ? p.cu[lo] : 0, e = lo + 1 < (int)p.N ? p.cu[lo + 1] : S;
    s->n = lo;
    s->beg = b < 0 ? 0 : b > t ? t : b;
    s->end = e > S ? S : e <= t ? t + 1 : e;
}

// What begins and ends among the tokens [t0, t1) of a span: bit i of `starts` (`ends`): token
// t0 + i is the first (last) of its sequence, whose index is start_of[i] (end_of[i]).  s holds
// the sequence of t0 afterwards.
struct Marks {
    uint32_t starts, ends;
};
__device__ __forceinline__ Marks mark(const LinrecParams &p, int64_t first, int S, int t0, int t1, int lane,
                                      Seq *s, int *start_of, int *end_of) {
    Marks m = {0, 0};
    if (t0 >= t1) return m;
    seek(p, first, S, t0, lane, s);
    Seq q = *s;
    if (q.beg == t0) {
        m.starts = 1;
        if (lane == 0) start_of[0] = (int)q.n;
    }
    while (true) {
        const int e = q.end;
        if (e <= t1) {
            m.ends |= 1u << (e - 1 - t0);
            if (lane == 0) end_of[e - 1 - t0] = (int)q.n;
        }
        if (e >= t1) break;
        seek(p, first, S, e, lane, &q);
        m.starts |= 1u << (e - t0);
        if (lane == 0) start_of[e - t0] = (int)q.n;
    }
    return m;
}

// What a CTA works on.
struct Unit {
    int64_t first;  // first sequence of the stream (dense)
    int64_t tok0;   // the stream's first token
    int64_t tile0;  // its first saved state
    int S, steps;   // its tokens, and the cluster's steps over them
    int64_t c0;
    int cols, mine;  // channels of the CTA, and of this lane (0, 1 or 2)
    int rank;
};
__device__ __forceinline__ Unit unit_of(const LinrecParams &p, int lane) {
    Unit u;
    u.rank = blockIdx.x % p.cluster;
    const int64_t i = blockIdx.x / p.cluster, stream = i / p.slabs;
    u.c0 = i % p.slabs * kCh;
    u.cols = p.D - u.c0 < kCh ? (int)(p.D - u.c0) : kCh;
    const int left = u.cols - 2 * lane;
    u.mine = left < 0 ? 0 : left > 2 ? 2 : left;
    u.first = stream * p.rows_per_stream;
    if (p.cu) {
        u.tok0 = 0;
        u.S = (int)p.BT;
    } else {
        const int64_t rows = p.N - u.first < p.rows_per_stream ? p.N - u.first : p.rows_per_stream;
        u.tok0 = u.first * p.T;
        u.S = (int)(rows * p.T);
    }
    u.tile0 = stream * p.tiles;
    u.steps = (int)((u.S + (int64_t)kTile * p.cluster - 1) / ((int64_t)kTile * p.cluster));
    return u;
}

// States of empty documents pass through: to[n] = from[n].
__device__ __forceinline__ void pass_empty(const LinrecParams &p, const Unit &u, const float *from, float *to,
                                           int warp, int lane) {
    if (!p.cu || !to) return;
    const int64_t warps = (int64_t)p.cluster * kWarps;
    for (int64_t n0 = 32 * ((int64_t)u.rank * kWarps + warp); n0 < p.N; n0 += 32 * warps) {
        const int64_t n = n0 + lane;
        uint32_t empty = __ballot_sync(0xffffffffu, n < p.N && p.cu[n] == p.cu[n + 1]);
        while (empty) {
            const int64_t at = (n0 + __ffs(empty) - 1) * p.D + u.c0 + 2 * lane;
            empty &= empty - 1;
            store_state(to, at, load_state(from, at, u.mine), u.mine);
        }
    }
}

// ---------------------------------------------------------------- forward
template <typename T, typename G, bool COMP, bool EVEN>
__global__ void __launch_bounds__(32 * kWarps, 2) linrec_fwd_kernel(const __grid_constant__ LinrecParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float4 spans[2][kWarps][32], tiles[2][kMaxCluster][32];  // (A, X) of two channels
    __shared__ int span_cut[2][kWarps], tile_cut[2][kMaxCluster];       // 1: what comes before does not count
    __shared__ int start_of[kWarps][kSpan], end_of[kWarps][kSpan];
    constexpr int kRowsX = kSpan * kCh * sizeof(T), kRows = kRowsX + kSpan * kCh * sizeof(G);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = p.cluster, stages = p.stages;
    const Unit u = unit_of(p, lane);
    unsigned char *mine = smem + (size_t)warp * stages * kRows;
    const T *x = static_cast<const T *>(p.x) + u.tok0 * p.xs + u.c0;
    const G *g = static_cast<const G *>(p.g) + u.tok0 * p.gs + u.c0;
    T *o = static_cast<T *>(p.o);
    if (o) o += u.tok0 * p.os + u.c0 + 2 * lane;
    const auto first_token = [&](int step) { return (int64_t)(step * (int64_t)cluster + u.rank) * kTile + warp * kSpan; };
    const auto fetch = [&](int step, int stage) {
        const int64_t t0 = first_token(step);
        if (step < u.steps) {
            const int rows = t0 >= u.S ? 0 : u.S - t0 < kSpan ? (int)(u.S - t0) : kSpan;
            unsigned char *to = mine + stage * kRows;
            copy_rows(reinterpret_cast<T *>(to), rows ? x + t0 * p.xs : x, p.xs, rows, u.cols, p.wide, p.even, lane);
            copy_rows(reinterpret_cast<G *>(to + kRowsX), rows ? g + t0 * p.gs : g, p.gs, rows, u.cols, p.wide, p.even, lane);
        }
        copy_commit();
    };
    for (int i = 0; i < stages; ++i) fetch(i, i);
    if (cluster > 1) cluster_sync();  // the others run: their shared memory may be written

    Seq seq = {0, 0, 0};
    float2 carry = make_float2(0.f, 0.f);  // the state that enters the cluster's step
    for (int step = 0, stage = 0; step < u.steps; ++step, stage = stage + 1 == stages ? 0 : stage + 1) {
        const int buf = step & 1;
        const int64_t at = first_token(step);
        const int t0 = at < u.S ? (int)at : u.S, t1 = u.S - t0 < kSpan ? u.S : t0 + kSpan;
        __syncwarp();
        const Marks m = mark(p, u.first, u.S, t0, t1, lane, &seq, start_of[warp], end_of[warp]);
        copy_wait(stages - 1);
        __syncwarp();
        // the span's map
        float2 a[kSpan], v[kSpan], A = make_float2(1.f, 1.f), X = make_float2(0.f, 0.f);
        const T *xr = reinterpret_cast<const T *>(mine + stage * kRows);
        const G *gr = reinterpret_cast<const G *>(mine + stage * kRows + kRowsX);
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
            float2 w;
            gate<COMP>(load2(gr + i * kCh, lane), &a[i], &w);
            v[i] = load2(xr + i * kCh, lane);
            if (COMP) v[i] = mul2(w, v[i]);
        }
        __syncwarp();
        fetch(step + stages, stage);
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
            if (m.starts >> i & 1) X = load_state(p.h0, start_of[warp][i] * p.D + u.c0 + 2 * lane, u.mine);
            X = fma2(a[i], X, v[i]);
            A = mul2(A, a[i]);
        }
        spans[buf][warp][lane] = make_float4(A.x, X.x, A.y, X.y);
        if (lane == 0) span_cut[buf][warp] = m.starts != 0;
        __syncthreads();
        // the maps of the spans before this one, and of the tile
        float2 PA, PX, QA = make_float2(1.f, 1.f), QX = make_float2(0.f, 0.f), h;
        int pcut, qcut = 0;
#pragma unroll
        for (int j = 0; j < kWarps; ++j) {
            if (j == warp) PA = QA, PX = QX, pcut = qcut;
            const float4 s = spans[buf][j][lane];
            if (span_cut[buf][j]) qcut = 1, QX = make_float2(0.f, 0.f);
            QX = make_float2(fmaf(s.x, QX.x, s.y), fmaf(s.z, QX.y, s.w));
            QA = make_float2(QA.x * s.x, QA.y * s.z);
        }
        // the state that enters the span, and the next step
        if (cluster == 1) {
            h = pcut ? PX : fma2(PA, carry, PX);
            carry = qcut ? QX : fma2(QA, carry, QX);
        } else {
            for (int r = warp; r < cluster; r += kWarps) {
                cluster_store(cluster_addr(&tiles[buf][u.rank][lane], r), make_float4(QA.x, QX.x, QA.y, QX.y));
                if (lane == 0) cluster_store(cluster_addr(&tile_cut[buf][u.rank], r), qcut);
            }
            cluster_sync();
            for (int j = 0; j < cluster; ++j) {
                if (j == u.rank) h = pcut ? PX : fma2(PA, carry, PX);
                const float4 s = tiles[buf][j][lane];
                carry = tile_cut[buf][j] ? make_float2(s.y, s.w) : make_float2(fmaf(s.x, carry.x, s.y), fmaf(s.z, carry.y, s.w));
            }
        }
        // the span's tokens
        if (p.states && warp == 0 && t0 < t1 && p.tiles > 1)
            store_state(p.states, (u.tile0 + t0 / kTile) * p.D + u.c0 + 2 * lane, h, u.mine);
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
            if (m.starts >> i & 1) h = load_state(p.h0, start_of[warp][i] * p.D + u.c0 + 2 * lane, u.mine);
            h = fma2(a[i], h, v[i]);
            if (o && t0 + i < t1) store_pair<EVEN>(o + (t0 + i) * p.os, h, u.mine);
            if (m.ends >> i & 1) store_state(p.hT, end_of[warp][i] * p.D + u.c0 + 2 * lane, h, u.mine);
        }
    }
    pass_empty(p, u, p.h0, p.hT, warp, lane);
}

// ---------------------------------------------------------------- backward
template <typename T, typename G, bool COMP, bool EVEN>
__global__ void __launch_bounds__(32 * kWarps, 2) linrec_bwd_kernel(const __grid_constant__ LinrecParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float4 spans[2][kWarps][32], tiles[2][kMaxCluster][32];  // (A, X), (A, Y) of two channels
    __shared__ float2 grads[2][kWarps][32];                             // Y
    __shared__ int span_cut[2][kWarps], tile_cut[2][kMaxCluster];       // bit 0: forward, bit 1: backward
    __shared__ int start_of[kWarps][kSpan], end_of[kWarps][kSpan];
    constexpr int kRowsX = kSpan * kCh * sizeof(T), kRows = 2 * kRowsX + kSpan * kCh * sizeof(G);

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = p.cluster, stages = p.stages;
    const Unit u = unit_of(p, lane);
    unsigned char *mine = smem + (size_t)warp * stages * kRows;
    const T *x = static_cast<const T *>(p.x) + u.tok0 * p.xs + u.c0;
    const T *dy = static_cast<const T *>(p.dy) + u.tok0 * p.os + u.c0;
    const G *g = static_cast<const G *>(p.g) + u.tok0 * p.gs + u.c0;
    T *dx = static_cast<T *>(p.dx) + u.tok0 * p.dxs + u.c0 + 2 * lane;
    G *dg = static_cast<G *>(p.dg) + u.tok0 * p.dgs + u.c0 + 2 * lane;
    // steps count from the stream's end
    const auto first_token = [&](int step) {
        return ((int64_t)(u.steps - 1 - step) * cluster + u.rank) * kTile + warp * kSpan;
    };
    const auto fetch = [&](int step, int stage) {
        if (step < u.steps) {
            const int64_t t0 = first_token(step);
            const int rows = t0 >= u.S ? 0 : u.S - t0 < kSpan ? (int)(u.S - t0) : kSpan;
            unsigned char *to = mine + stage * kRows;
            copy_rows(reinterpret_cast<T *>(to), rows ? x + t0 * p.xs : x, p.xs, rows, u.cols, p.wide, p.even, lane);
            copy_rows(reinterpret_cast<T *>(to + kRowsX), rows ? dy + t0 * p.os : dy, p.os, rows, u.cols, p.wide, p.even, lane);
            copy_rows(reinterpret_cast<G *>(to + 2 * kRowsX), rows ? g + t0 * p.gs : g, p.gs, rows, u.cols, p.wide, p.even, lane);
        }
        copy_commit();
    };
    for (int i = 0; i < stages; ++i) fetch(i, i);
    if (cluster > 1) cluster_sync();

    Seq seq = {0, 0, 0};
    float2 carry = make_float2(0.f, 0.f);  // gradient of the state that leaves the cluster's step
    for (int step = 0, stage = 0; step < u.steps; ++step, stage = stage + 1 == stages ? 0 : stage + 1) {
        const int buf = step & 1;
        const int64_t at = first_token(step);
        const int t0 = at < u.S ? (int)at : u.S, t1 = u.S - t0 < kSpan ? u.S : t0 + kSpan;
        // the state that enters the tile (the first tile starts a sequence)
        const int64_t tile = (at - warp * kSpan) / kTile;
        float2 h = make_float2(0.f, 0.f);
        if (tile > 0 && tile < p.tiles) h = load_state(p.states, (u.tile0 + tile) * p.D + u.c0 + 2 * lane, u.mine);
        __syncwarp();
        const Marks m = mark(p, u.first, u.S, t0, t1, lane, &seq, start_of[warp], end_of[warp]);
        copy_wait(stages - 1);
        __syncwarp();
        const T *xr = reinterpret_cast<const T *>(mine + stage * kRows);
        const T *dr = reinterpret_cast<const T *>(mine + stage * kRows + kRowsX);
        const G *gr = reinterpret_cast<const G *>(mine + stage * kRows + 2 * kRowsX);
        // the span's maps
        float2 a[kSpan], w[kSpan], A = make_float2(1.f, 1.f), X = make_float2(0.f, 0.f), Y = X;
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
            gate<COMP>(load2(gr + i * kCh, lane), &a[i], &w[i]);
            if (m.starts >> i & 1) X = load_state(p.h0, start_of[warp][i] * p.D + u.c0 + 2 * lane, u.mine);
            const float2 v = load2(xr + i * kCh, lane);
            X = fma2(a[i], X, COMP ? mul2(w[i], v) : v);
            A = mul2(A, a[i]);
        }
#pragma unroll
        for (int i = kSpan - 1; i >= 0; --i) {
            if (m.ends >> i & 1) Y = load_state(p.dhT, end_of[warp][i] * p.D + u.c0 + 2 * lane, u.mine);
            const float2 d = load2(dr + i * kCh, lane);
            Y = mul2(a[i], make_float2(d.x + Y.x, d.y + Y.y));
        }
        spans[buf][warp][lane] = make_float4(A.x, X.x, A.y, X.y);
        grads[buf][warp][lane] = Y;
        if (lane == 0) span_cut[buf][warp] = (m.starts != 0) | (m.ends != 0) << 1;
        __syncthreads();
        // the state that enters the span
        for (int j = 0; j < warp; ++j) {
            const float4 s = spans[buf][j][lane];
            if (span_cut[buf][j] & 1) h = make_float2(0.f, 0.f);
            h = make_float2(fmaf(s.x, h.x, s.y), fmaf(s.z, h.y, s.w));
        }
        // the reverse maps of the spans after this one, and of the tile
        float2 PA, PY, QA = make_float2(1.f, 1.f), QY = make_float2(0.f, 0.f), r;
        int pcut, qcut = 0;
#pragma unroll
        for (int j = kWarps - 1; j >= 0; --j) {
            if (j == warp) PA = QA, PY = QY, pcut = qcut;
            const float4 s = spans[buf][j][lane];
            const float2 y = grads[buf][j][lane];
            if (span_cut[buf][j] & 2) qcut = 1, QY = make_float2(0.f, 0.f);
            QY = make_float2(fmaf(s.x, QY.x, y.x), fmaf(s.z, QY.y, y.y));
            QA = make_float2(QA.x * s.x, QA.y * s.z);
        }
        // the gradient of the state that leaves the span, and the next step
        if (cluster == 1) {
            r = pcut ? PY : fma2(PA, carry, PY);
            carry = qcut ? QY : fma2(QA, carry, QY);
        } else {
            for (int k = warp; k < cluster; k += kWarps) {
                cluster_store(cluster_addr(&tiles[buf][u.rank][lane], k), make_float4(QA.x, QY.x, QA.y, QY.y));
                if (lane == 0) cluster_store(cluster_addr(&tile_cut[buf][u.rank], k), qcut);
            }
            cluster_sync();
            for (int j = cluster - 1; j >= 0; --j) {
                if (j == u.rank) r = pcut ? PY : fma2(PA, carry, PY);
                const float4 s = tiles[buf][j][lane];
                carry = tile_cut[buf][j] ? make_float2(s.y, s.w) : make_float2(fmaf(s.x, carry.x, s.y), fmaf(s.z, carry.y, s.w));
            }
        }
        // the span's tokens: the states before them, then the gradients from the last to the first
        float2 before[kSpan];
#pragma unroll
        for (int i = 0; i < kSpan; ++i) {
            if (m.starts >> i & 1) h = load_state(p.h0, start_of[warp][i] * p.D + u.c0 + 2 * lane, u.mine);
            const float2 v = load2(xr + i * kCh, lane);
            before[i] = COMP ? make_float2(h.x - v.x, h.y - v.y) : h;
            h = fma2(a[i], h, COMP ? mul2(w[i], v) : v);
        }
#pragma unroll
        for (int i = kSpan - 1; i >= 0; --i) {
            if (m.ends >> i & 1) r = load_state(p.dhT, end_of[warp][i] * p.D + u.c0 + 2 * lane, u.mine);
            const float2 d = load2(dr + i * kCh, lane), e = make_float2(d.x + r.x, d.y + r.y);
            r = mul2(a[i], e);
            if (t0 + i < t1) {
                store_pair<EVEN>(dx + (t0 + i) * p.dxs, COMP ? mul2(w[i], e) : e, u.mine);
                store_pair<EVEN>(dg + (t0 + i) * p.dgs, mul2(r, before[i]), u.mine);
            }
            if (m.starts >> i & 1) store_state(p.dh0, start_of[warp][i] * p.D + u.c0 + 2 * lane, r, u.mine);
        }
        __syncwarp();
        fetch(step + stages, stage);
    }
    pass_empty(p, u, p.dhT, p.dh0, warp, lane);
}

// ---------------------------------------------------------------- one-token form
__device__ __forceinline__ float ld(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p, int64_t i) { return __bfloat162float(p[i]); }

template <typename T, typename G, bool COMP>
__global__ void __launch_bounds__(128) linrec_decode_kernel(LinrecParams p, float *state) {
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x, n = blockIdx.x;
    if (c >= p.D) return;
    const T *x = static_cast<const T *>(p.x);
    const G *g = static_cast<const G *>(p.g);
    T *o = static_cast<T *>(p.o);
    float h = state[n * p.D + c];
    for (int64_t t = n * p.T; t < (n + 1) * p.T; ++t) {
        const float gt = ld(g, t * p.gs + c), xt = ld(x, t * p.xs + c);
        h = fmaf(__expf(gt), h, COMP ? -expm1f(gt) * xt : xt);
        put(o + t * p.os + c, h);
    }
    state[n * p.D + c] = h;
}

// ---------------------------------------------------------------- launches
enum class Pass { kFwd, kBwd, kDecode };

// A kernel of `smem` bytes of dynamic shared memory on p's clusters.  The two attributes are set
// once per device and kernel.
cudaError_t launch_cluster(void (*kernel)(LinrecParams), std::atomic<uint64_t> *ready, const LinrecParams &p,
                           size_t smem, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev > 63 || !(ready->load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        ready->fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.streams * p.slabs * p.cluster));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, typename G, bool COMP, bool EVEN>
cudaError_t launch_typed(LinrecParams p, Pass pass, cudaStream_t s) {
    static std::atomic<uint64_t> ready[2];
    const size_t rows = (size_t)kTile * kCh * (pass == Pass::kFwd ? sizeof(T) + sizeof(G) : 2 * sizeof(T) + sizeof(G));
    // CTAs: as many as give every SM kPerSm of them, in clusters no longer than the stream
    const int64_t units = p.streams * p.slabs;
    p.cluster = 1;
    while (p.cluster < kMaxCluster && 2 * p.cluster <= p.tiles && units * p.cluster * 2 <= kSms * kPerSm) p.cluster *= 2;
    // stages: what the SM's shared memory holds for the CTAs that it gets, up to the steps there are
    const int64_t per_sm = (units * p.cluster + kSms - 1) / kSms;
    const int64_t steps = (p.tiles + p.cluster - 1) / p.cluster;
    const size_t room = kSmemSm / (per_sm < 1 ? 1 : per_sm > kPerSm ? kPerSm : per_sm) - kSmemStatic;
    int64_t stages = (int64_t)((room < kSmemMax ? room : kSmemMax) / rows);
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages > steps) stages = steps;
    p.stages = stages < 1 ? 1 : (int32_t)stages;
    const size_t smem = rows * p.stages;
    cudaError_t err = cudaSuccess;
    if (pass == Pass::kFwd)
        GDN_LAUNCH(kKLinrecFwd, s, (err = launch_cluster(linrec_fwd_kernel<T, G, COMP, EVEN>, &ready[0], p, smem, s)));
    else
        GDN_LAUNCH(kKLinrecBwd, s, (err = launch_cluster(linrec_bwd_kernel<T, G, COMP, EVEN>, &ready[1], p, smem, s)));
    return err;
}

template <typename T, typename G, bool COMP>
cudaError_t launch_even(const LinrecParams &p, Pass pass, float *state, cudaStream_t s) {
    if (pass == Pass::kDecode) {
        const dim3 grid((unsigned)p.N, (unsigned)((p.D + 127) / 128));
        GDN_LAUNCH(kKLinrecDecode, s, linrec_decode_kernel<T, G, COMP><<<grid, 128, 0, s>>>(p, state));
        return cudaSuccess;
    }
    return p.even ? launch_typed<T, G, COMP, true>(p, pass, s) : launch_typed<T, G, COMP, false>(p, pass, s);
}

template <typename T, typename G>
cudaError_t launch_comp(const LinrecParams &p, bool comp, Pass pass, float *state, cudaStream_t s) {
    return comp ? launch_even<T, G, true>(p, pass, state, s) : launch_even<T, G, false>(p, pass, state, s);
}

cudaError_t launch(const gdn_linrec_desc *d, LinrecParams p, Pass pass, float *state, cudaStream_t s) {
    // 16-byte copies need rows that start on 16 bytes; pairs of channels need even rows
    const int es = d->dtype == GDN_BF16 ? 2 : 4, ges = d->g_dtype == GDN_BF16 ? 2 : 4;
    const int64_t in[] = {p.xs * es, p.gs * ges, pass == Pass::kBwd ? p.os * es : 0};
    p.wide = 1;
    for (int64_t b : in)
        if (b % 16) p.wide = 0;
    p.even = (p.D | p.xs | p.gs | p.os) % 2 == 0 && (pass != Pass::kBwd || (p.dxs | p.dgs) % 2 == 0);
    const bool comp = d->flags & GDN_LINREC_COMPLEMENT;
    if (d->dtype == GDN_FP32) return launch_comp<float, float>(p, comp, pass, state, s);
    if (d->g_dtype == GDN_FP32) return launch_comp<__nv_bfloat16, float>(p, comp, pass, state, s);
    return launch_comp<__nv_bfloat16, __nv_bfloat16>(p, comp, pass, state, s);
}

// The states of no token: to[n] = from[n] for every sequence.
cudaError_t pass_all(const LinrecParams &p, const float *from, float *to, cudaStream_t s) {
    if (!to) return cudaSuccess;
    const size_t bytes = (size_t)p.N * p.D * sizeof(float);
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
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
    // streams: the packed row, a dense row, or as many short dense rows as fill a tile
    p->rows_per_stream = d->n_seqs > 0 ? 1 : p->T > 0 && p->T < kTile ? kTile / p->T : 1;
    p->streams = d->n_seqs > 0 ? 1 : (p->N + p->rows_per_stream - 1) / p->rows_per_stream;
    p->tiles = (p->rows_per_stream * p->T + kTile - 1) / kTile;
    p->slabs = (int32_t)((p->D + kCh - 1) / kCh);
    if (p->streams * p->slabs >= kLim / kMaxCluster) return GDN_ERR_INVALID_ARG;
    const int64_t in[] = {d->x_stride, d->g_stride, d->o_stride, d->dx_stride, d->dg_stride};
    int64_t *out[] = {&p->xs, &p->gs, &p->os, &p->dxs, &p->dgs};
    for (int i = 0; i < 5; ++i) {
        if (in[i] != 0 && (in[i] < d->D || in[i] >= kLim)) return GDN_ERR_INVALID_ARG;
        *out[i] = in[i] ? in[i] : d->D;
    }
    return GDN_OK;
}

bool mis(const void *p, size_t a = 16) { return p && (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// A stream of one tile needs none: every sequence starts within it.
size_t states_bytes(const LinrecParams &p) {
    const size_t b = p.tiles > 1 ? (size_t)p.streams * p.tiles * p.D * sizeof(float) : 0;
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
    const cudaError_t e = p.BT == 0 ? pass_all(p, h0, hT, s) : launch(desc, p, Pass::kFwd, nullptr, s);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
    if (p.BT == 0) return pass_all(p, dhT, dh0, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    if (!states && p.tiles > 1) {
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
