// Gated linear recurrence, forward, backward and one-token form (declared in
// include/gdn.h).
//
// A sequence's map over any span of tokens is affine per channel, h' = A h + X with
// A the product of the span's factors, and the reverse map of the gradients is
// r' = A r + Y with the same A; spans join by (A2, X2)(A1, X1) = (A2 A1, A2 X1 + X2).
// A CTA takes 64 channels (two per lane) and a tile of adjacent tokens at a time, split into
// one span per warp, whose factors and inputs stay in registers.  Each of eight warps forms its
// span's map and joins the maps of the spans before it; the last one, which thereby has the
// tile's map, carries the state.  A cluster of up to 16 CTAs takes consecutive tiles of the
// same channels: the carrying warps send their tile's map to all of them (st.async through
// distributed shared memory, counted by an mbarrier: a release would wait for the outputs
// still being stored) and each folds them in order, so each holds the state that enters its
// tile and the next step.  The data is read from memory once, by cp.async into a ring of tiles
// that runs ahead of the steps, each warp copying its own rows.
//
// Measured on a B200, bf16 inputs and fp32 gates (of the measured copy rate, 6.56 TB/s): 16 x 4096 x
// 2048 forward 170 us (96%) and backward 337 us (85%); 4 x 4096 x 2048 54 us (75%) and 99 us (72%),
// where the rows' channels alone do not fill the GPU: the first stall there is a step's two barriers, with
// the exchange between them (a warp scheduler issues in 48 and 52% of the cycles, DRAM runs at 56 and 38% of its
// peak); one row of 262144 x 1024 506 us (65%) and 1037 us (55%), where an exchange takes about 2600
// cycles of a step of 6000.  bf16 gates at 16 x 4096 x 2048, with no exchange: 157 us (78%) and 307 us
// (67%), 23 and 46 instructions per element, issued in 62 and 61% of the cycles; the rest is waits of
// an instruction for the one before it, with the 16 warps that the registers allow.  The write
// strength 1 - a costs 15 to 20% more.  Three CTAs per SM in the backward, tiles twice as long or
// 16 warps with one CTA per SM, and one step ahead were slower.  The registers are at the limit of
// two CTAs per SM: some kernels of rows off 16 bytes or in fp32 spill 4 to 28 bytes.
//
// A start of a sequence inside a span drops what comes before it by selection (not by a
// factor of 0), so that no infinity or NaN crosses; padded tokens are zeros (factor
// exp(0) = 1, input 0), which is the identity map in both directions.
//
// The backward runs the tiles from the last to the first.  It needs the states that
// enter each token: the forward leaves the state entering every 64th token (4 / 64 bytes per
// element), from which a tile recomputes its own.
#include <atomic>
#include <memory>
#include <mutex>
#include <new>

#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCh = 64;        // channels per CTA
constexpr int kSaved = 64;     // tokens between two saved states
constexpr int kMaxSpan = 16, kMaxStages = 8, kMaxCluster = 16;
constexpr int kPerSm = 2;      // CTAs that an SM's registers hold
constexpr size_t kSmemSm = 227 * 1024;  // of an SM
constexpr int kSms = 148;
constexpr int kCuKept = 256;                // offsets of documents that a CTA keeps

// Tokens per warp: 16 in the forward of bf16 inputs; 8 where the tiles are larger, and in the
// backward, which has more to keep in registers.
template <typename T> constexpr int kFwdSpan = sizeof(T) == 2 ? 16 : 8;
constexpr int kBwdSpan = 8;

struct LinrecParams {
    int64_t T, BT, D, N;
    int64_t xs, gs, os, dxs, dgs;
    int64_t streams, rows_per_stream;  // a stream: one dense row, several short ones, or the packed row
    int64_t saved;                            // saved states of a stream
    int32_t slabs, cluster, stages, aligned, even;
    // bytes from a token to the next, and from a step of the cluster to the next
    int64_t x_row, g_row, dy_row, o_row, dx_row, dg_row;
    int64_t x_step, g_step, dy_step, o_step, dx_step, dg_step;
    uint32_t wait_limit;
    int32_t test_hook;
    int32_t slot;    // of g_gave_up
    int32_t single;  // every stream is one sequence
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
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// exp, to 2 ulp and the rounding of g log2(e).
__device__ __forceinline__ float exp_fast(float g) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(g * 1.44269504088896341f));
    return y;
}

// a = exp(g), and the write strength w = 1 or 1 - a (COMP).  A factor near 1 acts over many tokens,
// over which an error of one sign adds up, and exp_fast is about a third of an ulp low; so for
// small |g| the factor comes from the Taylor polynomial, rounded once: to g^5 for |g| <= 1/8 (the
// next term is below 2^-27), and where 1 - a is wanted without its cancellation to g^8 for |g| <=
// 1/2 (the next term is below 2^-26 of the sum).  With factors around 0.986 the last of 262144
// states is then below 1e-6 off, and above it with exp_fast alone.  The polynomials take two
// channels per instruction; elsewhere packed operations cost more in moves than they save (the
// forward of 16 x 4096 x 2048: 176 us so, 201 us all packed, 198 us not at all).
template <bool COMP>
__device__ __forceinline__ void gate(float2 g, float2 *a, float2 *w) {
    const float2 e = make_float2(exp_fast(g.x), exp_fast(g.y));
    if (COMP) {
        float2 s = both(-1.f / 40320);
        s = __ffma2_rn(s, g, both(-1.f / 5040));
        s = __ffma2_rn(s, g, both(-1.f / 720));
        s = __ffma2_rn(s, g, both(-1.f / 120));
        s = __ffma2_rn(s, g, both(-1.f / 24));
        s = __ffma2_rn(s, g, both(-1.f / 6));
        s = __ffma2_rn(s, g, both(-1.f / 2));
        s = __ffma2_rn(s, g, both(-1.f));
        s = __fmul2_rn(s, g);
        const bool x = fabsf(g.x) <= 0.5f, y = fabsf(g.y) <= 0.5f;
        *a = make_float2(x ? 1.f - s.x : e.x, y ? 1.f - s.y : e.y);
        *w = make_float2(x ? s.x : 1.f - e.x, y ? s.y : 1.f - e.y);
    } else {
        float2 s = both(1.f / 120);
        s = __ffma2_rn(s, g, both(1.f / 24));
        s = __ffma2_rn(s, g, both(1.f / 6));
        s = __ffma2_rn(s, g, both(1.f / 2));
        s = __ffma2_rn(s, g, both(1.f));
        s = __ffma2_rn(s, g, both(1.f));
        *a = make_float2(fabsf(g.x) <= 0.125f ? s.x : e.x, fabsf(g.y) <= 0.125f ? s.y : e.y);
        *w = both(1.f);
    }
}

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes) {  // 4, or 4 zeros
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async16(void *dst, const void *src, int bytes) {  // and 16 - bytes zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
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

// The copies of whole spans whose rows start on 16 bytes: a lane copies 16 bytes (the last ones maybe
// in part, the rest become zeros) of every kAtOnce-th row, from a pointer that moves with the steps.
template <int kSpan, typename E>
struct Copies {
    static constexpr int kPer = 16 / sizeof(E), kPieces = kCh / kPer, kAtOnce = 32 / kPieces;
    const char *src;  // the lane's piece of the span's first rows
    int bytes, at;    // how much of it exists, and where it goes in a span
    __device__ __forceinline__ void start(const void *base, int64_t tok, int64_t row, const int c0, int cols, int lane) {
        const int c = lane % kPieces * kPer, r = lane / kPieces, here = (cols - c) * (int)sizeof(E);
        bytes = here < 0 ? 0 : here > 16 ? 16 : here;
        at = r * kCh + c;
        src = static_cast<const char *>(base) + (tok + r) * row + (c0 + (bytes ? c : 0)) * (int64_t)sizeof(E);
    }
    __device__ __forceinline__ void span(E *dst, int64_t row) const {
#pragma unroll
        for (int i = 0; i < kSpan; i += kAtOnce) copy_async16(dst + at + i * kCh, src + i * row, bytes);
    }
};

// A span's tokens x 64 channels; `rows` and `cols` of them exist, the rest become zeros.  Rows that
// start on 16 bytes: 16 at a time; fp32, or bf16 with even rows: 4 at a time; else one bf16 after
// another.
template <int kSpan, bool ALIGNED, typename E>
__device__ __forceinline__ void copy_rows(E *dst, const E *src, int64_t stride, int rows, int cols,
                                          int even, int lane) {
    if (ALIGNED) {
        constexpr int kPer = 16 / sizeof(E), kPieces = kCh / kPer, kAtOnce = 32 / kPieces;
        const int c = lane % kPieces * kPer, r = lane / kPieces;
        const int here = (cols - c) * (int)sizeof(E), bytes = here < 0 ? 0 : here > 16 ? 16 : here;
        dst += r * kCh + c;
#pragma unroll
        for (int i = 0; i < kSpan; i += kAtOnce) {
            const int n = i + r < rows ? bytes : 0;
            copy_async16(dst + i * kCh, n ? src + (i + r) * stride + c : src, n);
        }
    } else if (sizeof(E) == 4 || even) {
        constexpr int kPer = 4 / sizeof(E);
#pragma unroll
        for (int r = 0; r < kSpan; ++r)
#pragma unroll
            for (int c = lane * kPer; c < kCh; c += 32 * kPer) {
                const bool in = r < rows && c < cols;
                copy_async(dst + r * kCh + c, in ? src + r * stride + c : src, in ? 4 : 0);
            }
    } else {
#pragma unroll 1
        for (int i = 0; i < kSpan; i += 8) {
            E v[8][2];
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = lane + 32 * j;
                    v[r][j] = i + r < rows && c < cols ? src[(i + r) * stride + c] : E(0.f);
                }
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) dst[(i + r) * kCh + lane + 32 * j] = v[r][j];
        }
    }
}

__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
// Stores 16 bytes into a CTA of the cluster; they count down its mbarrier.
__device__ __forceinline__ void send(uint32_t to, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(to), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar) : "memory");
}

// Waits of this device's calls that gave up (gdn_linrec_status), counted by the stream of the call, so that no
// stream's calls are taken for another's (two of 4095 may fall together); slot 0: captured calls, which replay
// on any stream.  Counts are never cleared: what one reader is told is not lost to the others.
constexpr int kSlots = 4096;
__device__ uint32_t g_gave_up[kSlots];

// ---------------------------------------------------------------- sequences of a stream
// The sequence that holds a token, for a whole warp: index n, tokens [beg, end) of the stream.
struct Seq {
    int n, beg, end;
};

// Moves s to the sequence that holds token t (0 <= t < S).  Packed: the largest n with cu[n]
// <= t, searched near s first and then 33 ways at a time.  Only cu[1 .. N - 1] are trusted as
// far as indices go; the bounds are forced around t whatever they hold.
__device__ __forceinline__ void seek(const LinrecParams &p, const int32_t *cu, int first, int S, int t, int lane, Seq *s) {
    if (t >= s->beg && t < s->end) return;
    if (!cu) {
        const int T = (int)p.T, k = t / T;
        s->n = first + k, s->beg = k * T, s->end = s->beg + T;
        return;
    }
    int lo = 0, hi = (int)p.N;  // cu[lo] <= t < cu[hi]
    int step = 1;
    if (t >= s->end) {
        lo = s->n;
    } else {
        hi = s->n > 0 ? s->n : 1;
        const int at = hi - 1 - lane;
        const bool after = at > lo && cu[at] > t;
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
        const bool before = at < hi && cu[at] <= t;
        const uint32_t b = __ballot_sync(0xffffffffu, before);
        const int cnt = b == 0xffffffffu ? 32 : __ffs(~b) - 1;
        const int64_t end = lo + (int64_t)(cnt + 1) * step;
        lo += cnt * step;
        if (cnt < 32 && end < hi) hi = (int)end;
        step = (hi - lo + 32) / 33;
    }
    const int b = lo > 0 ? cu[lo] : 0, e = lo + 1 < (int)p.N ? cu[lo + 1] : S;
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
__device__ __forceinline__ Marks mark(const LinrecParams &p, const int32_t *cu, int first, int S, int t0, int t1, int lane,
                                      Seq *s, int *start_of, int *end_of) {
    Marks m = {0, 0};
    if (t0 >= t1) return m;
    if (p.single) {
        m.starts = t0 == 0;
        m.ends = t1 == S ? 1u << (t1 - 1 - t0) : 0;
        if (lane == 0) {
            if (m.starts) start_of[0] = first;
            if (m.ends) end_of[t1 - 1 - t0] = first;
        }
        return m;
    }
    seek(p, cu, first, S, t0, lane, s);
    Seq q = *s;
    if (q.beg == t0) {
        m.starts = 1;
        if (lane == 0) start_of[0] = q.n;
    }
    while (true) {
        const int e = q.end;
        if (e <= t1) {
            m.ends |= 1u << (e - 1 - t0);
            if (lane == 0) end_of[e - 1 - t0] = q.n;
        }
        if (e >= t1) break;
        seek(p, cu, first, S, e, lane, &q);
        m.starts |= 1u << (e - t0);
        if (lane == 0) start_of[e - t0] = q.n;
    }
    return m;
}

// What a CTA works on.
struct Unit {
    int first;   // first sequence of the stream (dense)
    int tok0;    // the stream's first token
    int saved0;  // its first saved state
    int S, steps;  // its tokens, and the cluster's steps over them
    int c0;
    int cols, mine;  // channels of the CTA, and of this lane (0, 1 or 2)
    int rank;
};
__device__ __forceinline__ Unit unit_of(const LinrecParams &p, int tile, int lane) {
    Unit u;
    u.rank = blockIdx.x % p.cluster;
    const int i = blockIdx.x / p.cluster, stream = i / p.slabs;
    u.c0 = i % p.slabs * kCh;
    u.cols = p.D - u.c0 < kCh ? (int)(p.D - u.c0) : kCh;
    const int left = u.cols - 2 * lane;
    u.mine = left < 0 ? 0 : left > 2 ? 2 : left;
    u.first = stream * (int)p.rows_per_stream;
    if (p.cu) {
        u.tok0 = 0;
        u.S = (int)p.BT;
    } else {
        const int left_rows = (int)p.N - u.first, rows = left_rows < p.rows_per_stream ? left_rows : (int)p.rows_per_stream;
        u.tok0 = u.first * (int)p.T;
        u.S = rows * (int)p.T;
    }
    u.saved0 = stream * (int)p.saved;
    u.steps = (int)((u.S + (int64_t)tile * p.cluster - 1) / ((int64_t)tile * p.cluster));
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

// ---------------------------------------------------------------- the carrying warp
// A tile's map (A, X of each lane's two channels); a step's maps, and those of the step before it, are
// in each CTA of the cluster.  Factors are not negative, so the sign of the first one says that
// what comes before the tile does not count.
struct __align__(16) Map {
    float4 m[32];
};
// Shared memory of a CTA, beside its tiles and the cluster's maps.
struct Shared {
    float4 spans[kWarps][32];               // a span's map (A, X) of the lane's two channels; backward: (A, Y)
    float2 starts[kWarps][32];              // backward: X
    float2 enter[32];                       // what enters the CTA's tile
    uint64_t bar[2];                        // arrivals of the cluster's maps (even, odd steps)
    int cut[kWarps];                        // bit 0: a start in the span, bit 1: an end
    int start_of[kWarps][kMaxSpan], end_of[kWarps][kMaxSpan];
    int dead;                               // the step in which a wait ran out, counted from 1 (0: none)
    int sent[kMaxCluster];                  // steps whose maps each CTA sends: all, or what one that gave up says
    int32_t cu[kCuKept];                    // the offsets of few documents: crossing one costs no global loads
};
constexpr size_t kSmemCta = sizeof(Shared) + 1024;  // of a CTA beside tiles and maps (1 KB is the system's)

__device__ __forceinline__ float2 join(float4 s, bool cut, float2 h) {
    return cut ? make_float2(s.y, s.w) : fma2(make_float2(s.x, s.z), h, make_float2(s.y, s.w));
}

// Waits (up to `limit` polls) for the phase of this parity.
__device__ __forceinline__ bool arrived(uint64_t *bar, uint32_t parity, uint32_t limit) {
    for (uint32_t i = 0; i < limit; ++i) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred q;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
        if (ok) return true;
        if (i > 64) __nanosleep(32);
    }
    return false;
}
__device__ __forceinline__ void give_up(const LinrecParams &p, Shared &sh, int step) {
    sh.dead = step + 1;
    atomicAdd(&g_gave_up[p.slot], 1u);
}

// Whether the planted failure makes this CTA wait for 16 bytes that no one sends.
__device__ __forceinline__ bool stalls(const LinrecParams &p, int step) {
    return p.test_hook == GDN_TEST_STALL_COPY && blockIdx.x == 0 && step == 0;
}

// Makes the mbarriers ready in every CTA of the cluster before anyone sends.
__device__ __forceinline__ void cluster_begin(const LinrecParams &p, Shared &sh, int cluster, int steps) {
    if (p.cu && p.N < kCuKept)
        for (int i = threadIdx.x; i <= p.N; i += kThreads) sh.cu[i] = p.cu[i];
    if (threadIdx.x == 0) {
        sh.dead = 0;
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&sh.bar[i], 1);
        for (int i = 0; i < kMaxCluster; ++i) sh.sent[i] = steps;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if (cluster > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_ready(int cluster) {
    if (cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// No CTA leaves while a map may still arrive in it.  One that has made all its steps has seen all maps.  One that
// gave up in a step has sent its maps up to that step's, which it tells the others before the barrier; behind the
// barrier it knows how many maps come, makes up for those that do not, and waits (up to `limit` polls) for the rest.
__device__ __forceinline__ void count_maps(Shared &sh, int cluster, int step, uint32_t extra, uint32_t limit) {
    uint32_t now = 0, next = 0;  // maps of this step and, of CTAs that went on, of the one after it
    for (int r = 0; r < cluster; ++r) now += sh.sent[r] > step, next += sh.sent[r] > step + 1;
    const uint32_t missing = (cluster - now) * (uint32_t)sizeof(Map) + extra;
    uint64_t *bar = &sh.bar[step & 1], *other = &sh.bar[(step + 1) & 1];
    if (missing)
        asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(missing) : "memory");
    if (next) ptx::mbar_arrive_expect_tx(other, next * (uint32_t)sizeof(Map));
    arrived(bar, (step >> 1) & 1, limit);
    if (next) arrived(other, (step + 1) >> 1 & 1, limit);
}
__device__ __forceinline__ void cluster_end(const LinrecParams &p, Shared &sh, int cluster) {
    if (cluster == 1) return;
    const int sent = sh.dead;
    if (!sent) {
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        return;
    }
    const int i = threadIdx.x;
    if (i < cluster)
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr(&sh.sent[blockIdx.x % p.cluster], i)), "r"(sent) : "memory");
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (i == 0) count_maps(sh, cluster, sent - 1, stalls(p, sent - 1) ? 16 : 0, kWaitLimit);
}

// The carrying warp's part of a step, between the CTA's two barriers: sends the tile's map q to
// the cluster, forms what enters the tile from all tiles of the step, and the new carry.  REV:
// from the last rank to the first.
__device__ __forceinline__ void send_map(const LinrecParams &p, Shared &sh, Map *maps, int rank, int step, int lane, float4 q, bool cut) {
    if (p.cluster == 1) return;
    const int buf = step & 1;
    if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&sh.bar[buf], p.cluster * (uint32_t)sizeof(Map) + (stalls(p, step) ? 16 : 0));
    }
    q.x = __uint_as_float((__float_as_uint(q.x) & 0x7fffffffu) | (cut ? 0x80000000u : 0u));
    const Map *to = maps + buf * p.cluster + rank;
    for (int i = 1; i <= p.cluster; ++i) {  // to the neighbour first, so that no CTA is everyone's first
        const int r = rank + i < p.cluster ? rank + i : rank + i - p.cluster;
        send(cluster_addr(&to->m[lane], r), q, cluster_addr(&sh.bar[buf], r));
    }
}
template <bool REV>
__device__ __forceinline__ void carry_on(const LinrecParams &p, Shared &sh, const Map *maps, int rank, int step, int lane, float4 q, bool cut, float2 *carry) {
    if (p.cluster == 1) {
        sh.enter[lane] = *carry;
        *carry = join(q, cut, *carry);
        return;
    }
    const int buf = step & 1;
    if (!__all_sync(0xffffffffu, arrived(&sh.bar[buf], (step >> 1) & 1, p.wait_limit))) {
        if (lane == 0) give_up(p, sh, step);
        return;
    }
    const Map *from = maps + buf * p.cluster;
    float2 c = *carry;
    for (int i0 = 0; i0 < p.cluster; i0 += 4) {  // four loads at a time
        float4 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = i0 + i < p.cluster ? i0 + i : 0;
            f[i] = from[REV ? p.cluster - 1 - k : k].m[lane];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i0 + i >= p.cluster) break;
            if ((REV ? p.cluster - 1 - (i0 + i) : i0 + i) == rank) sh.enter[lane] = c;
            c = join(f[i], signbit(f[i].x), c);
        }
    }
    *carry = c;
}

// A warp's span of a step.
struct Span {
    int count;  // tokens (0 .. kSpan)
    Marks m;
    bool plain;  // nothing starts or ends in it, and nothing is missing
};
template <int kSpan>
__device__ __forceinline__ Span span_at(const LinrecParams &p, Shared &sh, const Unit &u, uint32_t t0, int warp, int lane, Seq *seq) {
    Span s = {kSpan, {0, 0}, true};
    // strictly inside a sequence?
    if (p.single ? t0 > 0 && t0 + kSpan < (uint32_t)u.S : (int)t0 > seq->beg && t0 + kSpan < (uint32_t)seq->end) return s;
    s.count = t0 >= (uint32_t)u.S ? 0 : u.S - t0 < kSpan ? u.S - t0 : kSpan;
    __syncwarp();
    if (s.count) s.m = mark(p, p.N < kCuKept && p.cu ? sh.cu : p.cu, u.first, u.S, (int)t0, (int)t0 + s.count, lane, seq, sh.start_of[warp], sh.end_of[warp]);
    s.plain = !(s.m.starts | s.m.ends) && s.count == kSpan;
    __syncwarp();
    return s;
}

// A state that a span reads, asked for before the span's copies are waited for: that of the first
// start (or last end) in it.
struct Early {
    int i;  // the token in the span, -1: none
    float2 v;
};
__device__ __forceinline__ Early early(const float *p, const LinrecParams &q, const Unit &u, int i, const int *of, int c) {
    Early e = {i, both(0.f)};
    if (i >= 0) e.v = load_state(p, of[i] * q.D + c, u.mine);
    return e;
}
__device__ __forceinline__ float2 state_at(const Early &e, const float *p, const LinrecParams &q, const Unit &u, int i, const int *of, int c) {
    return i == e.i ? e.v : load_state(p, of[i] * q.D + c, u.mine);
}

// ---------------------------------------------------------------- forward
// A span's map.  PLAIN: no sequence starts in it.
template <bool PLAIN, int kSpan>
__device__ __forceinline__ float4 map_span(const LinrecParams &p, const Unit &u, const float2 (&a)[kSpan],
                                           const float2 (&v)[kSpan], uint32_t starts, const Early &e, const int *start_of, int c) {
    float2 A = a[0], X = v[0];
    if (!PLAIN && (starts & 1)) X = fma2(a[0], state_at(e, p.h0, p, u, 0, start_of, c), v[0]);
#pragma unroll
    for (int i = 1; i < kSpan; ++i) {
        if (!PLAIN && (starts >> i & 1)) X = state_at(e, p.h0, p, u, i, start_of, c);
        X = fma2(a[i], X, v[i]);
        A = mul2(A, a[i]);
    }
    return make_float4(A.x, X.x, A.y, X.y);
}

// Runs the span's tokens from h; `mine` channels are stored (0: only the states are wanted).
template <bool PLAIN, bool EVEN, int kSpan, typename T>
__device__ __forceinline__ void run_span(const LinrecParams &p, const Unit &u, const float2 (&a)[kSpan],
                                         const float2 (&v)[kSpan], float2 h, const Span &s, int mine,
                                         const Early &e, const int *start_of, const int *end_of, int c, T *o) {
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        if (!PLAIN && (s.m.starts >> i & 1)) h = state_at(e, p.h0, p, u, i, start_of, c);
        h = fma2(a[i], h, v[i]);
        if (PLAIN || i < s.count) store_pair<EVEN>(o, h, mine);
        o = reinterpret_cast<T *>(reinterpret_cast<char *>(o) + p.o_row);
        if (!PLAIN && (s.m.ends >> i & 1)) store_state(p.hT, end_of[i] * p.D + c, h, u.mine);
    }
}

// ALIGNED: rows start on 16 bytes, and pairs of channels can be stored at once.
template <int kSpan, typename T, typename G, bool COMP, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, kPerSm) linrec_fwd_kernel(const __grid_constant__ LinrecParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Shared sh;
    constexpr int kTile = kSpan * kWarps;
    constexpr int kBytesX = kSpan * kCh * sizeof(T), kBytes = kBytesX + kSpan * kCh * sizeof(G);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = p.cluster, stages = p.stages;
    const Unit u = unit_of(p, kTile, lane);
    const int c = u.c0 + 2 * lane;
    unsigned char *mine = smem + warp * stages * kBytes;
    Map *maps = reinterpret_cast<Map *>(smem + kWarps * stages * kBytes);
    const int *start_of = sh.start_of[warp], *end_of = sh.end_of[warp];
    cluster_begin(p, sh, cluster, u.steps);

    uint32_t t0 = u.rank * kTile + warp * kSpan, ahead = t0;  // the warp's first token of a step, and of the next copies
    Copies<kSpan, T> cx;
    Copies<kSpan, G> cg;
    if (ALIGNED) {
        cx.start(p.x, (int64_t)u.tok0 + ahead, p.x_row, u.c0, u.cols, lane);
        cg.start(p.g, (int64_t)u.tok0 + ahead, p.g_row, u.c0, u.cols, lane);
    }
    const auto fetch = [&](int stage) {
        const int rows = ahead >= (uint32_t)u.S ? 0 : u.S - ahead < kSpan ? u.S - ahead : kSpan;
        unsigned char *to = mine + stage * kBytes;
        if (ALIGNED && rows == kSpan) {
            cx.span(reinterpret_cast<T *>(to), p.x_row);
            cg.span(reinterpret_cast<G *>(to + kBytesX), p.g_row);
        } else if (rows) {
            const int64_t tok = (int64_t)u.tok0 + ahead;
            copy_rows<kSpan, ALIGNED>(reinterpret_cast<T *>(to), static_cast<const T *>(p.x) + tok * p.xs + u.c0, p.xs, rows, u.cols, p.even, lane);
            copy_rows<kSpan, ALIGNED>(reinterpret_cast<G *>(to + kBytesX), static_cast<const G *>(p.g) + tok * p.gs + u.c0, p.gs, rows, u.cols, p.even, lane);
        }
        copy_commit();
        ahead += cluster * kTile;
        if (ALIGNED) cx.src += p.x_step, cg.src += p.g_step;
    };
    for (int i = 0; i < stages; ++i) fetch(i);
    cluster_ready(cluster);

    Seq seq = {0, 0, 0};
    float2 carry = both(0.f);  // the state that enters the cluster's step (the last warp's)
    char *o = static_cast<char *>(p.o) + ((int64_t)u.tok0 + t0) * p.o_row + c * (int64_t)sizeof(T);
    const int stored = p.o ? u.mine : 0;
    for (int step = 0, stage = 0; step < u.steps; ++step, t0 += cluster * kTile, o += p.o_step) {
        const Span s = span_at<kSpan>(p, sh, u, t0, warp, lane, &seq);
        const Early e = early(p.h0, p, u, __ffs(s.m.starts) - 1, start_of, c);
        copy_wait(stages - 1);
        __syncwarp();
        float2 a[kSpan], v[kSpan];
        {
            const T *x = reinterpret_cast<const T *>(mine + stage * kBytes);
            const G *g = reinterpret_cast<const G *>(mine + stage * kBytes + kBytesX);
#pragma unroll
            for (int i = 0; i < kSpan; ++i) {
                const float2 gi = load2(g + i * kCh, lane);
                float2 w;
                gate<COMP>(gi, &a[i], &w);
                v[i] = load2(x + i * kCh, lane);
                if (COMP) v[i] = mul2(w, v[i]);
            }
        }
        __syncwarp();
        fetch(stage);
        if (++stage == stages) stage = 0;
        float4 own;
        if (s.plain) {
            own = map_span<true>(p, u, a, v, 0, e, nullptr, c);
        } else {
#pragma unroll
            for (int i = 0; i < kSpan; ++i)
                if (i >= s.count) a[i] = both(1.f), v[i] = both(0.f);
            own = map_span<false>(p, u, a, v, s.m.starts, e, start_of, c);
        }
        const bool cuts = s.m.starts != 0;
        sh.spans[warp][lane] = own;
        if (lane == 0) sh.cut[warp] = cuts;
        const bool any = __syncthreads_or(cuts);
        // the map of the spans before this one
        float2 PA = both(1.f), PX = both(0.f);
        bool cut = false;
        if (!any) {
#pragma unroll
            for (int j = 0; j < kWarps - 1; ++j)
                if (j < warp) {
                    const float4 f = sh.spans[j][lane];
                    PX = fma2(make_float2(f.x, f.z), PX, make_float2(f.y, f.w));
                    PA = mul2(PA, make_float2(f.x, f.z));
                }
        } else {
#pragma unroll 1
            for (int j = 0; j < warp; ++j) {
                const float4 f = sh.spans[j][lane];
                const bool here = sh.cut[j] & 1;
                PX = join(f, here, PX);
                PA = mul2(PA, make_float2(f.x, f.z));
                cut |= here;
            }
        }
        if (warp == kWarps - 1) {
            const float2 X = join(own, cuts, PX);
            const float4 q = make_float4(PA.x * own.x, X.x, PA.y * own.z, X.y);
            send_map(p, sh, maps, u.rank, step, lane, q, cut || cuts);
            carry_on<false>(p, sh, maps, u.rank, step, lane, q, cut || cuts, &carry);
        }
        __syncthreads();
        if (sh.dead) break;
        const float2 h = cut ? PX : fma2(PA, sh.enter[lane], PX);
        if (p.states && t0 % kSaved == 0 && s.count)
            store_state(p.states, (int64_t)(u.saved0 + t0 / kSaved) * p.D + c, h, u.mine);
        if (s.plain)
            run_span<true, ALIGNED>(p, u, a, v, h, s, stored, e, start_of, end_of, c, reinterpret_cast<T *>(o));
        else
            run_span<false, ALIGNED>(p, u, a, v, h, s, stored, e, start_of, end_of, c, reinterpret_cast<T *>(o));
    }
    copy_wait(0);
    pass_empty(p, u, p.h0, p.hT, warp, lane);
    cluster_end(p, sh, cluster);
}

// ---------------------------------------------------------------- backward
// A token's two channels as they are kept in registers.
__device__ __forceinline__ float2 raw(const float *p, int lane) { return load2(p, lane); }
__device__ __forceinline__ __nv_bfloat162 raw(const __nv_bfloat16 *p, int lane) {
    return reinterpret_cast<const __nv_bfloat162 *>(p)[lane];
}
__device__ __forceinline__ float2 value(float2 v) { return v; }
__device__ __forceinline__ float2 value(__nv_bfloat162 v) { return __bfloat1622float2(v); }

// The reverse map of a span; d: its tokens' gradients.
template <bool PLAIN, int kSpan, typename R>
__device__ __forceinline__ float2 map_back(const LinrecParams &p, const Unit &u, const float2 (&a)[kSpan], const R (&d)[kSpan],
                                           const Span &s, const Early &l, const int *end_of, int c) {
    float2 Y = both(0.f);
#pragma unroll
    for (int i = kSpan - 1; i >= 0; --i) {
        if (!PLAIN && (s.m.ends >> i & 1)) Y = state_at(l, p.dhT, p, u, i, end_of, c);
        if (PLAIN || i < s.count) Y = mul2(a[i], add2(value(d[i]), Y));
    }
    return Y;
}

// The span's tokens: the states before them (minus x, COMP) in place of x, then the gradients from the
// last to the first.
template <bool PLAIN, bool COMP, bool EVEN, int kSpan, typename R, typename T, typename G>
__device__ __forceinline__ void run_back(const LinrecParams &p, const Unit &u, const float2 (&a)[kSpan],
                                         const float2 (&w)[kSpan], float2 (&x)[kSpan], const R (&d)[kSpan], float2 h, float2 r,
                                         const Span &s, const Early &e, const Early &l, const int *start_of, const int *end_of, int c, T *dx, G *dg) {
#pragma unroll
    for (int i = 0; i < kSpan; ++i) {
        if (!PLAIN && (s.m.starts >> i & 1)) h = state_at(e, p.h0, p, u, i, start_of, c);
        const float2 v = x[i];
        x[i] = COMP ? make_float2(h.x - v.x, h.y - v.y) : h;
        h = fma2(a[i], h, COMP ? mul2(w[i], v) : v);
    }
    char *px = reinterpret_cast<char *>(dx) + (kSpan - 1) * p.dx_row, *pg = reinterpret_cast<char *>(dg) + (kSpan - 1) * p.dg_row;
#pragma unroll
    for (int i = kSpan - 1; i >= 0; --i) {
        if (!PLAIN && (s.m.ends >> i & 1)) r = state_at(l, p.dhT, p, u, i, end_of, c);
        if (PLAIN || i < s.count) {
            const float2 y = add2(value(d[i]), r);
            r = mul2(a[i], y);
            store_pair<EVEN>(reinterpret_cast<T *>(px), COMP ? mul2(w[i], y) : y, u.mine);
            store_pair<EVEN>(reinterpret_cast<G *>(pg), mul2(r, x[i]), u.mine);
        }
        px -= p.dx_row;
        pg -= p.dg_row;
        if (!PLAIN && (s.m.starts >> i & 1)) store_state(p.dh0, start_of[i] * p.D + c, r, u.mine);
    }
}

template <int kSpan, typename T, typename G, bool COMP, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, kPerSm) linrec_bwd_kernel(const __grid_constant__ LinrecParams p) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Shared sh;
    constexpr int kTile = kSpan * kWarps;
    static_assert(kTile == kSaved, "a tile starts from a saved state");
    constexpr int kBytesX = kSpan * kCh * sizeof(T), kBytes = 2 * kBytesX + kSpan * kCh * sizeof(G);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = p.cluster, stages = p.stages;
    const Unit u = unit_of(p, kTile, lane);
    const int c = u.c0 + 2 * lane;
    unsigned char *mine = smem + warp * stages * kBytes;
    Map *maps = reinterpret_cast<Map *>(smem + kWarps * stages * kBytes);
    const int *start_of = sh.start_of[warp], *end_of = sh.end_of[warp];
    cluster_begin(p, sh, cluster, u.steps);

    // steps go from the stream's end
    uint32_t t0 = ((uint32_t)(u.steps - 1) * cluster + u.rank) * kTile + warp * kSpan, ahead = t0;
    int left = u.steps;  // steps whose copies are still to be made
    Copies<kSpan, T> cx, cd;
    Copies<kSpan, G> cg;
    if (ALIGNED) {
        cx.start(p.x, (int64_t)u.tok0 + ahead, p.x_row, u.c0, u.cols, lane);
        cd.start(p.dy, (int64_t)u.tok0 + ahead, p.dy_row, u.c0, u.cols, lane);
        cg.start(p.g, (int64_t)u.tok0 + ahead, p.g_row, u.c0, u.cols, lane);
    }
    const auto fetch = [&](int stage) {
        const int rows = left <= 0 || ahead >= (uint32_t)u.S ? 0 : u.S - ahead < kSpan ? u.S - ahead : kSpan;
        unsigned char *to = mine + stage * kBytes;
        if (ALIGNED && rows == kSpan) {
            cx.span(reinterpret_cast<T *>(to), p.x_row);
            cd.span(reinterpret_cast<T *>(to + kBytesX), p.dy_row);
            cg.span(reinterpret_cast<G *>(to + 2 * kBytesX), p.g_row);
        } else if (rows) {
            const int64_t tok = (int64_t)u.tok0 + ahead;
            copy_rows<kSpan, ALIGNED>(reinterpret_cast<T *>(to), static_cast<const T *>(p.x) + tok * p.xs + u.c0, p.xs, rows, u.cols, p.even, lane);
            copy_rows<kSpan, ALIGNED>(reinterpret_cast<T *>(to + kBytesX), static_cast<const T *>(p.dy) + tok * p.os + u.c0, p.os, rows, u.cols, p.even, lane);
            copy_rows<kSpan, ALIGNED>(reinterpret_cast<G *>(to + 2 * kBytesX), static_cast<const G *>(p.g) + tok * p.gs + u.c0, p.gs, rows, u.cols, p.even, lane);
        }
        copy_commit();
        ahead -= cluster * kTile;
        --left;
        if (ALIGNED) cx.src -= p.x_step, cd.src -= p.dy_step, cg.src -= p.g_step;
    };
    // the state that enters a step's tile (the stream's first tile starts a sequence)
    const auto saved = [&](uint32_t t) {
        const uint32_t tile = t - warp * kSpan;
        return tile > 0 && tile < (uint32_t)u.S ? load_state(p.states, (int64_t)(u.saved0 + tile / kSaved) * p.D + c, u.mine) : both(0.f);
    };
    for (int i = 0; i < stages; ++i) fetch(i);
    cluster_ready(cluster);

    Seq seq = {0, 0, 0};
    float2 carry = both(0.f);  // the gradient of the state that leaves the step (the first warp's)
    char *dx = static_cast<char *>(p.dx) + ((int64_t)u.tok0 + t0) * p.dx_row + c * (int64_t)sizeof(T);
    char *dg = static_cast<char *>(p.dg) + ((int64_t)u.tok0 + t0) * p.dg_row + c * (int64_t)sizeof(G);
    for (int step = 0, stage = 0; step < u.steps; ++step, t0 -= cluster * kTile, dx -= p.dx_step, dg -= p.dg_step) {
        float2 h = saved(t0);
        const Span s = span_at<kSpan>(p, sh, u, t0, warp, lane, &seq);
        const Early e = early(p.h0, p, u, __ffs(s.m.starts) - 1, start_of, c), l = early(p.dhT, p, u, 31 - __clz(s.m.ends), end_of, c);
        copy_wait(stages - 1);
        __syncwarp();
        float2 a[kSpan], w[kSpan], x[kSpan];
        decltype(raw(static_cast<const T *>(nullptr), 0)) d[kSpan];
        {
            const T *xs = reinterpret_cast<const T *>(mine + stage * kBytes), *ds = reinterpret_cast<const T *>(mine + stage * kBytes + kBytesX);
            const G *gs = reinterpret_cast<const G *>(mine + stage * kBytes + 2 * kBytesX);
#pragma unroll
            for (int i = 0; i < kSpan; ++i) {
                gate<COMP>(load2(gs + i * kCh, lane), &a[i], &w[i]);
                x[i] = load2(xs + i * kCh, lane);
                d[i] = raw(ds + i * kCh, lane);
            }
        }
        __syncwarp();
        fetch(stage);
        if (++stage == stages) stage = 0;
        // the span's maps in both directions
        if (!s.plain) {
#pragma unroll
            for (int i = 0; i < kSpan; ++i)
                if (i >= s.count) a[i] = both(1.f), x[i] = both(0.f);
        }
        float2 Y;
        float4 f;
        {
            float2 v[kSpan];
#pragma unroll
            for (int i = 0; i < kSpan; ++i) v[i] = COMP ? mul2(w[i], x[i]) : x[i];
            if (s.plain) {
                f = map_span<true>(p, u, a, v, 0, e, nullptr, c);
                Y = map_back<true>(p, u, a, d, s, l, end_of, c);
            } else {
                f = map_span<false>(p, u, a, v, s.m.starts, e, start_of, c);
                Y = map_back<false>(p, u, a, d, s, l, end_of, c);
            }
        }
        const bool ends = s.m.ends != 0;
        const float4 own = make_float4(f.x, Y.x, f.z, Y.y);
        sh.spans[warp][lane] = own;
        sh.starts[warp][lane] = make_float2(f.y, f.w);
        if (lane == 0) sh.cut[warp] = (s.m.starts != 0) | ends << 1;
        const bool any = __syncthreads_or(s.m.starts | s.m.ends);
        // the reverse map of the spans after this one, and the state that enters the span
        float2 PA = both(1.f), PY = both(0.f);
        bool cut = false;
        if (!any) {
#pragma unroll
            for (int j = kWarps - 1; j > 0; --j)
                if (j > warp) {
                    const float4 m = sh.spans[j][lane];
                    PY = fma2(make_float2(m.x, m.z), PY, make_float2(m.y, m.w));
                    PA = mul2(PA, make_float2(m.x, m.z));
                }
        } else {
#pragma unroll 1
            for (int j = kWarps - 1; j > warp; --j) {
                const float4 m = sh.spans[j][lane];
                const bool here = sh.cut[j] & 2;
                PY = join(m, here, PY);
                PA = mul2(PA, make_float2(m.x, m.z));
                cut |= here;
            }
        }
        float4 q;
        if (warp == 0) {
            const float2 R = join(own, ends, PY);
            q = make_float4(PA.x * own.x, R.x, PA.y * own.z, R.y);
            send_map(p, sh, maps, u.rank, step, lane, q, cut || ends);
        }
        if (!any) {
#pragma unroll
            for (int j = 0; j < kWarps - 1; ++j)
                if (j < warp) {
                    const float4 m = sh.spans[j][lane];
                    h = fma2(make_float2(m.x, m.z), h, sh.starts[j][lane]);
                }
        } else {
#pragma unroll 1
            for (int j = 0; j < warp; ++j) {
                const float4 m = sh.spans[j][lane];
                const float2 X = sh.starts[j][lane];
                h = sh.cut[j] & 1 ? X : fma2(make_float2(m.x, m.z), h, X);
            }
        }
        if (warp == 0) carry_on<true>(p, sh, maps, u.rank, step, lane, q, cut || ends, &carry);
        __syncthreads();
        if (sh.dead) break;
        const float2 r = cut ? PY : fma2(PA, sh.enter[lane], PY);
        if (s.plain)
            run_back<true, COMP, ALIGNED>(p, u, a, w, x, d, h, r, s, e, l, start_of, end_of, c, reinterpret_cast<T *>(dx), reinterpret_cast<G *>(dg));
        else
            run_back<false, COMP, ALIGNED>(p, u, a, w, x, d, h, r, s, e, l, start_of, end_of, c, reinterpret_cast<T *>(dx), reinterpret_cast<G *>(dg));
    }
    copy_wait(0);
    pass_empty(p, u, p.dhT, p.dh0, warp, lane);
    cluster_end(p, sh, cluster);
}

// ---------------------------------------------------------------- one-token form
// C adjacent channels per thread (4 where rows and states allow 16-byte state accesses, else 1), the
// state in registers over the T tokens.  Bound by the state's bytes for many rows, by the launch
// for few: back to back 1.7 us for 256 x 2048 bf16 (3.5 us with a channel per thread), 1.1 us for 1 x 2048.
template <int C>
__device__ __forceinline__ void load_some(const float *p, float (&v)[C]) {
    if (C == 4) {
        const float4 t = *reinterpret_cast<const float4 *>(p);
        v[0] = t.x, v[1 % C] = t.y, v[2 % C] = t.z, v[3 % C] = t.w;
    } else {
        v[0] = *p;
    }
}
template <int C>
__device__ __forceinline__ void load_some(const __nv_bfloat16 *p, float (&v)[C]) {
    if (C == 4) {
        const uint2 t = *reinterpret_cast<const uint2 *>(p);
        v[0] = __uint_as_float(t.x << 16), v[1 % C] = __uint_as_float(t.x & 0xffff0000u);
        v[2 % C] = __uint_as_float(t.y << 16), v[3 % C] = __uint_as_float(t.y & 0xffff0000u);
    } else {
        v[0] = __bfloat162float(*p);
    }
}
template <typename T, typename G, bool COMP, int C>
__global__ void __launch_bounds__(128) linrec_decode_kernel(const __grid_constant__ LinrecParams p, float *state) {
    const int64_t c = ((int64_t)blockIdx.y * 128 + threadIdx.x) * C, n = blockIdx.x;
    if (c >= p.D) return;
    const T *x = static_cast<const T *>(p.x) + n * p.T * p.xs + c;
    const G *g = static_cast<const G *>(p.g) + n * p.T * p.gs + c;
    T *o = static_cast<T *>(p.o) + n * p.T * p.os + c;
    float h[C];
    load_some<C>(state + n * p.D + c, h);
    for (int64_t t = 0; t < p.T; ++t, x += p.xs, g += p.gs, o += p.os) {
        float xt[C], gt[C];
        load_some<C>(x, xt);
        load_some<C>(g, gt);
#pragma unroll
        for (int i = 0; i < C; i += 2) {
            float2 a, w;
            gate<COMP>(make_float2(gt[i], gt[(i + 1) % C]), &a, &w);
            h[i] = fmaf(a.x, h[i], COMP ? w.x * xt[i] : xt[i]);
            if (C > 1) h[(i + 1) % C] = fmaf(a.y, h[(i + 1) % C], COMP ? w.y * xt[(i + 1) % C] : xt[(i + 1) % C]);
        }
        if (C > 1) {
#pragma unroll
            for (int i = 0; i < C; i += 2) put2(o + i, make_float2(h[i], h[(i + 1) % C]));
        } else {
            put(o, h[0]);
        }
    }
    float *to = state + n * p.D + c;
    if (C == 4)
        *reinterpret_cast<float4 *>(to) = make_float4(h[0], h[1 % C], h[2 % C], h[3 % C]);
    else
        *to = h[0];
}

// ---------------------------------------------------------------- launches
enum class Pass { kFwd, kBwd, kDecode };

using Kernel = void (*)(LinrecParams);

// Clusters of each size (1 .. 16 CTAs) that a device runs at once: they stay
// within a group of SMs, so long ones fit less well (two CTAs per SM on a B200: 296 CTAs singly,
// 264 in clusters of 8, 224 in clusters of 16).  Asked for once per kernel and device, with the
// attributes that its launches need.
constexpr int kDevices = 64;
constexpr size_t kDynamic = (kSmemSm / kPerSm - kSmemCta) / 128 * 128;
struct Fit {
    std::atomic<int32_t> known{0};
    int16_t clusters[kMaxCluster + 1];
};
cudaError_t fit_of(Kernel kernel, Fit *fits, const Fit **out) {
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    Fit &fit = fits[dev];
    *out = &fit;
    if (fit.known.load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu);
    if (fit.known.load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDynamic);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (int k = 1; k <= kMaxCluster && e == cudaSuccess; ++k) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = k;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(k);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kDynamic;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        fit.clusters[k] = (int16_t)n;
    }
    if (e == cudaSuccess) fit.known.store(1, std::memory_order_release);
    return e;
}

bool capturing(cudaStream_t s) {
    cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) {  // cap says nothing; what comes next on the stream fails
        cudaGetLastError();
        return false;
    }
    return cap != cudaStreamCaptureStatusNone;
}
int stream_slot(cudaStream_t s) {
    return 1 + (int)((reinterpret_cast<uintptr_t>(s) * 0x9E3779B97F4A7C15ull >> 32) % (kSlots - 1));
}
int slot_of(cudaStream_t s) { return capturing(s) ? 0 : stream_slot(s); }

// Whether this host thread has not been told of this count yet.  It remembers the captured calls' of every
// device, and those of the last 64 streams it asked for.
bool is_news(int device, int slot, uint32_t count) {
    struct Told {
        int device, slot;  // slot 0 where unused
        uint32_t count;
    };
    constexpr int kTold = 64;
    thread_local Told told[kTold];
    thread_local uint32_t captured[kDevices];
    thread_local int next = 0;
    uint32_t *at = slot == 0 ? &captured[device] : nullptr;
    for (int i = 0; i < kTold && !at; ++i)
        if (told[i].slot == slot && told[i].device == device) at = &told[i].count;
    if (!at) {
        told[next] = {device, slot, 0};
        at = &told[next].count;
        next = (next + 1) % kTold;
    }
    const bool news = *at != count;
    *at = count;
    return news;
}

// A kernel of `smem` bytes of dynamic shared memory on p's clusters.
cudaError_t launch_cluster(Kernel kernel, const LinrecParams &p, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.streams * p.slabs * p.cluster));
    cfg.blockDim = dim3(kThreads);
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

template <typename T, typename G, bool COMP, bool ALIGNED>
cudaError_t launch_typed(LinrecParams p, Pass pass, cudaStream_t s) {
    static Fit fits[2][kDevices];
    const bool fwd = pass == Pass::kFwd;
    const int tile = kWarps * (fwd ? kFwdSpan<T> : kBwdSpan);
    const size_t bytes = (size_t)tile * kCh * (fwd ? sizeof(T) + sizeof(G) : 2 * sizeof(T) + sizeof(G));
    const int64_t tiles = (p.rows_per_stream * p.T + tile - 1) / tile, units = p.streams * p.slabs;
    // the longest clusters that can all run at once, and that the stream fills
    const Kernel kernel = fwd ? linrec_fwd_kernel<kFwdSpan<T>, T, G, COMP, ALIGNED> : linrec_bwd_kernel<kBwdSpan, T, G, COMP, ALIGNED>;
    const Fit *fit = nullptr;
    cudaError_t err = fit_of(kernel, fits[fwd ? 0 : 1], &fit);
    if (err != cudaSuccess) return err;
    p.cluster = 1;
    for (int k = 2; k <= kMaxCluster && k <= tiles; ++k)
        if (units <= fit->clusters[k]) p.cluster = k;
    // a ring of as many tiles as the shared memory holds, up to the steps there are
    const int64_t steps = (tiles + p.cluster - 1) / p.cluster;
    const size_t maps = p.cluster > 1 ? 2 * p.cluster * sizeof(Map) : 0;
    int64_t stages = (int64_t)((kSmemSm / kPerSm - kSmemCta - maps) / bytes);
    if (stages > kMaxStages) stages = kMaxStages;
    if (stages > steps) stages = steps;
    p.stages = stages < 1 ? 1 : (int32_t)stages;
    const size_t smem = bytes * p.stages + maps;
    const int64_t es = sizeof(T), ges = sizeof(G), tokens = (int64_t)p.cluster * tile;
    p.x_row = p.xs * es, p.g_row = p.gs * ges, p.dy_row = p.o_row = p.os * es, p.dx_row = p.dxs * es, p.dg_row = p.dgs * ges;
    p.x_step = tokens * p.x_row, p.g_step = tokens * p.g_row, p.dy_step = p.o_step = tokens * p.o_row;
    p.dx_step = tokens * p.dx_row, p.dg_step = tokens * p.dg_row;
    p.wait_limit = call_wait_limit();
    p.test_hook = call_test_hook();
    p.slot = slot_of(s);
    GDN_LAUNCH(fwd ? kKLinrecFwd : kKLinrecBwd, s, (err = launch_cluster(kernel, p, smem, s)));
    return err;
}

template <typename T, typename G, bool COMP>
cudaError_t launch_even(const LinrecParams &p, Pass pass, float *state, cudaStream_t s) {
    if (pass == Pass::kDecode) {
        const bool fours = (p.D | p.xs | p.gs | p.os) % 4 == 0;
        const int64_t width = fours ? 512 : 128;
        const dim3 grid((unsigned)p.N, (unsigned)((p.D + width - 1) / width));
        if (fours)
            GDN_LAUNCH(kKLinrecDecode, s, linrec_decode_kernel<T, G, COMP, 4><<<grid, 128, 0, s>>>(p, state));
        else
            GDN_LAUNCH(kKLinrecDecode, s, linrec_decode_kernel<T, G, COMP, 1><<<grid, 128, 0, s>>>(p, state));
        return cudaSuccess;
    }
    return p.aligned ? launch_typed<T, G, COMP, true>(p, pass, s) : launch_typed<T, G, COMP, false>(p, pass, s);
}

template <typename T, typename G>
cudaError_t launch_comp(const LinrecParams &p, bool comp, Pass pass, float *state, cudaStream_t s) {
    return comp ? launch_even<T, G, true>(p, pass, state, s) : launch_even<T, G, false>(p, pass, state, s);
}

cudaError_t launch(const gdn_linrec_desc *d, LinrecParams p, Pass pass, float *state, cudaStream_t s) {
    // 16-byte copies need rows that start on 16 bytes; pairs of channels even rows.
    const bool bwd = pass == Pass::kBwd;
    const int es = d->dtype == GDN_BF16 ? 2 : 4, ges = d->g_dtype == GDN_BF16 ? 2 : 4;
    p.even = (p.D | p.xs | p.gs | p.os) % 2 == 0 && (!bwd || (p.dxs | p.dgs) % 2 == 0);
    p.aligned = p.even && p.xs * es % 16 == 0 && p.gs * ges % 16 == 0 && (!bwd || p.os * es % 16 == 0);
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
    // streams: the packed row, a dense row, or several rows of less than 64 tokens: as many as fill 64,
    // or as leave every SM two CTAs if that is twice as many (1024 x 16 x 2048 bf16: 78 us forward and
    // 138 us backward, 155 and 147 us when they only fill 64; 300 x 7 x 1024 with 16 instead of 9:
    // 14 and 21 us, 16 and 16 us.  Rows of 100 tokens lose, 64 x 100 x 2048: backward 66 us, singly 59 us)
    p->slabs = (int32_t)((p->D + kCh - 1) / kCh);
    p->rows_per_stream = 1;
    if (d->n_seqs == 0 && p->T > 0 && p->T < kSaved) {
        const int64_t fill = kSaved / p->T, share = p->N * p->slabs / (2 * kSms);
        const int64_t rows = share >= 2 * fill ? share : fill;
        p->rows_per_stream = rows > p->N ? p->N : rows;
    }
    p->streams = d->n_seqs > 0 ? 1 : (p->N + p->rows_per_stream - 1) / p->rows_per_stream;
    p->single = d->n_seqs > 0 ? d->n_seqs == 1 : p->rows_per_stream == 1;
    if (p->streams * p->slabs >= kLim / kMaxCluster) return GDN_ERR_INVALID_ARG;
    p->saved = (p->rows_per_stream * p->T + kSaved - 1) / kSaved;
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
    const size_t b = p.saved > 1 ? (size_t)p.streams * p.saved * p.D * sizeof(float) : 0;
    return b < 256 ? 256 : (b + 255) / 256 * 256;
}

// Host-side check of cu_seqlens (the rules of gdn_fwd).
gdn_status check_seqlens(const gdn_linrec_desc *d, const int32_t *cu_dev, const int32_t *cu_host,
                         cudaStream_t s) {
    if (d->n_seqs == 0) return cu_dev || cu_host ? GDN_ERR_INVALID_ARG : GDN_OK;
    if (!cu_dev) return GDN_ERR_INVALID_ARG;
    if (mis(cu_dev, 4)) return GDN_ERR_ALIGNMENT;
    std::unique_ptr<int32_t[]> copy;
    if (!cu_host) {
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(s, &cap) != cudaSuccess) return GDN_ERR_CUDA;
        if (cap != cudaStreamCaptureStatusNone) return GDN_ERR_INVALID_ARG;
        const size_t n = (size_t)d->n_seqs + 1;
        copy.reset(new (std::nothrow) int32_t[n]);  // no exception leaves a C entry
        if (!copy) return GDN_ERR_CUDA;
        if (cudaMemcpyAsync(copy.get(), cu_dev, sizeof(int32_t) * n,
                            cudaMemcpyDeviceToHost, s) != cudaSuccess ||
            cudaStreamSynchronize(s) != cudaSuccess)
            return GDN_ERR_CUDA;
        cu_host = copy.get();
    }
    if (cu_host[0] != 0 || cu_host[d->n_seqs] != d->T) return GDN_ERR_INVALID_ARG;
    for (int64_t n = 0; n < d->n_seqs; ++n)
        if (cu_host[n + 1] < cu_host[n]) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

extern "C" {

gdn_status gdn_linrec_status(void *stream) {
    using namespace gdn;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (capturing(s)) return GDN_ERR_INVALID_ARG;
    int device = 0;
    void *at = nullptr;
    if (cudaGetDevice(&device) != cudaSuccess || device >= kDevices || cudaGetSymbolAddress(&at, g_gave_up) != cudaSuccess)
        return GDN_ERR_CUDA;
    const uint32_t *counts = static_cast<const uint32_t *>(at);
    const int slot = stream_slot(s);
    uint32_t own = 0, captured = 0;
    if (cudaMemcpyAsync(&own, counts + slot, sizeof(own), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemcpyAsync(&captured, counts, sizeof(captured), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return GDN_ERR_CUDA;
    const bool one = is_news(device, slot, own), two = is_news(device, 0, captured);
    return one || two ? GDN_ERR_TIMEOUT : GDN_OK;
}

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
    p.x = x, p.g = g, p.h0 = h0, p.o = o, p.hT = hT, p.states = p.saved > 1 ? states : nullptr;
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
    if (!states && p.saved > 1) {
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
