// Normalisation of q and k per token and head with the position rotation, and its
// gradients (declared in include/gdn.h).
//
// A row (one token and head) is split into units of two 16-byte chunks that turn into
// each other: the values i .. i + V and their partners i + rot / 2 .., or two adjacent chunks
// where pairs are adjacent or nothing turns.  A lane holds one unit, so norm and rotation
// need no exchange but the sum of squares over the row's lanes (8 lanes of a bf16 row of
// 128), and 32 / lanes heads of a token run side by side in a warp.  A warp walks the heads
// of its tokens, asking for the next row before it works on one; the angles of a token are formed
// once per warp (64-bit product and reduction, sincospi of the fraction) and shared through
// shared memory by all its heads.  Bound by HBM: every row is read and written once.  The
// weights' gradients are summed in registers over a block's rows, written once per block, and
// added in block order by a second kernel.
//
// Measured for 4 x 4096 tokens of 16 + 16 heads x 128: bf16 52 us forward and 77 us backward (78% and
// 79% of the measured copy rate), fp32 88 and 133 us (93% and 92%).  With a warp per row and shared
// memory between the passes: 335 and 560 us; with a row's loads behind the one before it 56 and 90 us.
// With few heads a token's angles and addresses weigh more than its rows (32 angles cost about 75
// instructions, a row 250, the step to another token 150): 8 + 2 heads x 64 bf16 20 and 24 us (31% and
// 40%).  Three blocks per SM in the forward: 53 us, fp32 92 us; with 8 + 1 heads 27 us, four 28 us.
// Adjacent pairs: 55 and 81 us.  fp32 rows of adjacent pairs that are taken value by value spill 20 to 52 bytes.
#include <cmath>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kMaxD = 256, kWarps = 8, kThreads = 32 * kWarps;
// Blocks of an SM.  Rows that are turned in part take more registers (56 us forward and 80 us backward for
// half of 4 x 4096 x 32 rows of 128 bf16; with four blocks 62 us).
constexpr int kSms = 148, kPerSm = 4, kPartPerSm = 3, kBwdPerSm = 2;
constexpr int kSlots = kSms * kPerSm;  // blocks at most, of both tensors
constexpr int kAngles = 288;           // angles that a warp keeps, those of its tokens

struct QkParams {
    int64_t tokens;
    int32_t T, d, rot, norm, interleaved;
    int32_t lanes, lanes_log2;  // lanes of a row
    int32_t whole;              // every lane has both chunks of its units
    int32_t blocks[2];          // blocks of q and of k
    int32_t per[2], parts[2];   // rows (times 32 / lanes) of a warp's item, and items of a token
    int32_t group[2];           // tokens side by side in a warp, where it has lanes for all their heads
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

// ---------------------------------------------------------------- small pieces
// V values of a row: as loaded, and in fp32.  VEC: one load of V values, else one by one.
template <typename T, int V, bool VEC>
struct Chunk;
template <int V, bool VEC>
struct Chunk<float, V, VEC> {
    float r[V];
    __device__ __forceinline__ void load(const float *p) {
        if (VEC && V == 4) {
            const float4 t = __ldcs(reinterpret_cast<const float4 *>(p));
            r[0] = t.x, r[1 % V] = t.y, r[2 % V] = t.z, r[3 % V] = t.w;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = p[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = 0.f;
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = r[i];
    }
    static __device__ __forceinline__ void store(float *p, const float (&x)[V]) {
        if (VEC && V == 4) {
            *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1 % V], x[2 % V], x[3 % V]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = x[i];
        }
    }
};
template <int V, bool VEC>
struct Chunk<__nv_bfloat16, V, VEC> {
    static constexpr int kWords = (V + 1) / 2;
    uint32_t r[kWords];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        if (VEC && V == 8) {
            const uint4 t = __ldcs(reinterpret_cast<const uint4 *>(p));
            r[0] = t.x, r[1 % kWords] = t.y, r[2 % kWords] = t.z, r[3 % kWords] = t.w;
        } else if (VEC && V == 4) {
            const uint2 t = __ldcs(reinterpret_cast<const uint2 *>(p));
            r[0] = t.x, r[1 % kWords] = t.y;
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                r[i / 2] = __bfloat16_as_ushort(p[i]);
                if (i + 1 < V) r[i / 2] |= (uint32_t)__bfloat16_as_ushort(p[i + 1]) << 16;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) r[i] = 0;
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = __uint_as_float(i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float (&x)[V]) {
        if (VEC) {
            uint32_t t[kWords];
#pragma unroll
            for (int i = 0; i < V; i += 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[i], x[(i + 1) % V]);
                t[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
            }
            if (V == 8)
                *reinterpret_cast<uint4 *>(p) = make_uint4(t[0], t[1 % kWords], t[2 % kWords], t[3 % kWords]);
            else
                *reinterpret_cast<uint2 *>(p) = make_uint2(t[0], t[1 % kWords]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = __float2bfloat16_rn(x[i]);
        }
    }
};

// 1 / sqrt(c |x|^2 + eps), 0 for 0.
__device__ __forceinline__ float scale_of(const QkParams &p, float sum) {
    if (p.norm == GDN_NORM_NONE) return 1.f;
    const float m = fmaf(p.c, sum, p.eps);
    return m > 0.f ? rsqrtf(m) : m;
}

// Where value i of chunk e of unit j is among the weights in shared memory: fours of neighbouring
// units side by side, so that a row's lanes read adjacent 16 bytes.
template <int V>
__device__ __forceinline__ int weight_at(int n, int j, int e, int i) {
    return V % 4 ? (e * V + i) * n + j : ((e * (V / 4) + i / 4) * n + j) * 4 + i % 4;
}
template <int V>
__device__ __forceinline__ void weights_of(const float *from, int n, int j, int e, float (&w)[V]) {
    if (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(from + weight_at<V>(n, j, e, i));
            w[i] = t.x, w[(i + 1) % V] = t.y, w[(i + 2) % V] = t.z, w[(i + 3) % V] = t.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = from[weight_at<V>(n, j, e, i)];
    }
}

// Two values per instruction where V is even: d = a b + c, and a b.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
template <int V>
__device__ __forceinline__ void fma_into(float (&c)[V], const float (&a)[V], const float (&b)[V]) {
    if (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const int j = (i + 1) % V;
            const float2 t = __ffma2_rn(make_float2(a[i], a[j]), make_float2(b[i], b[j]), make_float2(c[i], c[j]));
            c[i] = t.x, c[j] = t.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = fmaf(a[i], b[i], c[i]);
    }
}
// The same summed into s.
template <int V>
__device__ __forceinline__ void dot_into(float2 &s, const float (&a)[V], const float (&b)[V]) {
    if (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) s = __ffma2_rn(make_float2(a[i], a[(i + 1) % V]), make_float2(b[i], b[(i + 1) % V]), s);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) s.x = fmaf(a[i], b[i], s.x);
    }
}
template <int V>
__device__ __forceinline__ void times(float (&a)[V], const float (&b)[V]) {
    if (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const int j = (i + 1) % V;
            const float2 t = __fmul2_rn(make_float2(a[i], a[j]), make_float2(b[i], b[j]));
            a[i] = t.x, a[j] = t.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] *= b[i];
    }
}
template <int V>
__device__ __forceinline__ void times(float (&a)[V], float r) {
    float b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = r;
    times<V>(a, b);
}

// A warp's angles: pairs of a unit's angles side by side and neighbouring units next to each other, so
// that a row's lanes read adjacent 16 bytes: two cosines and two sines (adjacent pairs: cosine and
// sine of each).  n: units and one for what is not turned.
template <int V>
__device__ __forceinline__ int angle_at(int n, int j, int i) {
    return V % 2 ? n * i + j : 2 * (n * (i / 2) + j) + i % 2;
}
template <int V, bool ADJ>
__device__ __forceinline__ void put_angle(float2 *angles, int n, int j, int i, float2 cs) {
    if (V % 2 || ADJ) {
        angles[angle_at<V>(n, j, i)] = cs;
    } else {
        float *to = reinterpret_cast<float *>(angles + angle_at<V>(n, j, i - i % 2)) + i % 2;
        to[0] = cs.x, to[2] = cs.y;
    }
}

// A pair of chunks turned by the first `some` of a unit's angles (BACK: turned back; halves: by all or
// none).  The others are not even turned by 0, so that no infinity crosses.  Adjacent pairs: the first V / 2
// angles are the first chunk's.
template <int V, bool ADJ, bool BACK>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float2 *angles, int n, int some) {
    if (some <= 0) return;
    if (V % 2 == 0 && !ADJ) {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const int f = (e + 1) % V;
            const float4 t = *reinterpret_cast<const float4 *>(angles + angle_at<V>(n, 0, e));
            const float2 c = make_float2(t.x, t.y), s = make_float2(t.z, t.w);
            const float2 u = make_float2(a[e], a[f]), v = make_float2(b[e], b[f]), m = __fmul2_rn(BACK ? u : v, both(-1.f));
            const float2 x = __ffma2_rn(u, c, __fmul2_rn(BACK ? v : m, s)), y = __ffma2_rn(v, c, __fmul2_rn(BACK ? m : u, s));
            a[e] = x.x, a[f] = x.y, b[e] = y.x, b[f] = y.y;
        }
        return;
    }
    float2 cs[V];
    if (V % 2 == 0) {  // two angles per load
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float4 t = *reinterpret_cast<const float4 *>(angles + angle_at<V>(n, 0, e));
            cs[e] = make_float2(t.x, t.y), cs[(e + 1) % V] = make_float2(t.z, t.w);
        }
    } else {
        cs[0] = angles[0];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float c = cs[e].x, sn = BACK ? -cs[e].y : cs[e].y;
        if (!ADJ) {
            const float u = a[e], v = b[e];
            a[e] = fmaf(u, c, -v * sn);
            b[e] = fmaf(u, sn, v * c);
        } else {
            float(&t)[V] = e < V / 2 ? a : b;
            const int i = 2 * (e % (V / 2 ? V / 2 : 1));
            const float u = t[i], v = t[(i + 1) % V];
            t[i] = e < some ? fmaf(u, c, -v * sn) : u;
            t[(i + 1) % V] = e < some ? fmaf(u, sn, v * c) : v;
        }
    }
}

// A warp's way through its rows: items (a token's heads, or a part of them, or a group's) and the rows
// of an item.  tok: the token, or the group of tokens.
// row, drow: where this lane's row is, for reading (x, dy) or writing.
template <typename P>
struct Way {
    uint32_t item, tok;
    int it, end;
    int32_t pos;
    P row, drow;
};

// ---------------------------------------------------------------- the kernel
// NU units per lane.  VEC: whole chunks are loaded and stored at once.  GROUP: q or k has few heads, so
// that a warp takes several tokens at once.  FULL: whole rows are turned.
template <typename T, int V, int NU, bool VEC, bool ADJ, bool BWD, bool GROUP, bool FULL>
__global__ void __launch_bounds__(kThreads, BWD ? kBwdPerSm : FULL ? kPerSm : kPartPerSm) qk_kernel(const __grid_constant__ QkParams p) {
    // rows on their way while a warp works on one: one, but two in the backward of fp32 rows (4 x 4096 tokens of
    // 16 + 16 heads x 128: 134 against 139 us), whose bytes are twice as many
    constexpr int kUnroll = BWD && sizeof(T) == 4 && NU == 1 && !GROUP ? 2 : 1;
    __shared__ __align__(16) float2 angles[kWarps][GROUP ? kAngles : kMaxD / 2 + 8];  // (cos, sin), see angle_at
    __shared__ float sums[BWD ? kWarps : 1][kMaxD];
    __shared__ __align__(16) float weights[kMaxD];
    const int l = threadIdx.x & 31, wi = threadIdx.x >> 5;
    const int which = blockIdx.x >= p.blocks[0], block = blockIdx.x - (which ? p.blocks[0] : 0);
    const int H = p.heads[which], half = p.rot / 2, d = p.d;
    const int side = 32 >> p.lanes_log2, sub = l >> p.lanes_log2, unit = l & (p.lanes - 1);
    const T *x = static_cast<const T *>(p.x[which]), *dy = static_cast<const T *>(p.dy[which]);
    T *out = static_cast<T *>(BWD ? p.dx[which] : p.y[which]);
    const int64_t xs = p.xs[which], ys = p.ys[which], os = BWD ? p.dxs[which] : ys;
    const int its = (H + side - 1) / side, per = p.per[which], parts = p.parts[which];
    const int group = GROUP ? p.group[which] : 1, slot = GROUP ? sub / H : 0, head = GROUP ? sub - slot * H : sub;
    const uint32_t tokens = (uint32_t)p.tokens, items = GROUP && group > 1 ? (tokens + group - 1) / group : tokens * parts;
    const uint32_t warps = p.blocks[which] * kWarps;

    const int units = NU * p.lanes + 1, table = units * V;
    // this lane's units: where their chunks are (-1: nowhere) and whose angles they take
    int at[NU][2], angle[NU];
    float acc[NU][2][V];
#pragma unroll
    for (int k = 0; k < NU; ++k) {
        const int j = unit + k * p.lanes;
        if (ADJ || j * V < half) {
            at[k][0] = ADJ ? 2 * j * V : j * V;
            at[k][1] = at[k][0] + (ADJ ? V : half);
            angle[k] = j;
        } else {  // behind the turned values
            at[k][0] = p.rot + 2 * (j * V - half);
            at[k][1] = at[k][0] + V;
            angle[k] = units - 1;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (at[k][e] >= d) at[k][e] = -1;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                acc[k][e][i] = 0.f;
                if (wi == 0 && sub == 0)
                    weights[weight_at<V>(units - 1, j, e, i)] = p.w[which] && at[k][e] >= 0 ? p.w[which][at[k][e] + i] : 1.f;
            }
        }
    }
    for (int i = half + l; i < table; i += 32)
        for (int g = 0; g < group; ++g) put_angle<V, ADJ>(angles[wi] + g * table, units, i / V, i % V, make_float2(1.f, 0.f));
    const float2 *turns = angles[wi] + (GROUP && group > 1 && slot < group ? slot * table : 0);

    __syncthreads();
    // whole: every lane has both chunks of its units, and every row of lanes a head
    const bool whole = VEC && NU == 1 && (GROUP && group > 1 ? H * group == side && tokens % group == 0 : H % side == 0) && p.whole;
    const int64_t step = (int64_t)side * d;
    const auto offset = [&](const auto &y, int64_t stride) {
        if (GROUP && group > 1) return (y.tok * group + slot) * stride + (int64_t)head * d;
        return y.tok * stride + (int64_t)(y.it * side + sub) * d;
    };
    const auto enter = [&](auto &y, auto base, int64_t stride) {
        y.tok = parts == 1 ? y.item : y.item / parts;
        y.it = (y.item - y.tok * parts) * per;
        y.end = y.it + per < its ? y.it + per : its;
        y.row = base + offset(y, stride);
    };
    // whether this lane's row is one
    const auto is_row = [&](const auto &y) {
        return whole || (GROUP && group > 1 ? slot < group && y.tok * group + slot < tokens : y.it * side + sub < H);
    };
    Chunk<T, V, VEC> rx[kUnroll][NU][2], rd[BWD ? kUnroll : 1][NU][2];
    int32_t pos[kUnroll];
    Way<const T *> ahead = {(uint32_t)(block * kWarps + wi), 0, 0, 0, 0, nullptr, nullptr};
    Way<T *> go = {ahead.item, 0, 0, 0, 0, nullptr, nullptr};
    // to the next item; with one per token (or group) by a fixed jump
    const int64_t skip = (int64_t)warps * group, back = its * step;
    const auto next = [&](auto &y, auto base, int64_t stride) {
        y.item += warps;
        if (parts == 1) {
            y.tok = y.item;
            y.it = 0;
            y.row += skip * stride - back;
        } else if (y.item < items) {
            enter(y, base, stride);
        }
    };
    const int32_t turn_over = p.T ? (int32_t)((uint32_t)skip % (uint32_t)p.T) : 0;
    const auto find_pos = [&](bool first) {
        if (ahead.item >= items) return;
        uint32_t tok = ahead.tok;
        if (GROUP && group > 1) {  // lane i: the i-th token's
            tok = tok * group + l % group;
            if (tok >= tokens) tok = tokens - 1;
        }
        if (p.pos) {
            ahead.pos = p.pos[tok];
        } else if (first || parts != 1) {
            ahead.pos = (int32_t)(tok % (uint32_t)p.T);
        } else {
            ahead.pos = ahead.pos >= p.T - turn_over ? ahead.pos - (p.T - turn_over) : ahead.pos + turn_over;
        }
    };
    if (ahead.item < items) {
        enter(ahead, x, xs);
        if (BWD) ahead.drow = dy + offset(ahead, ys);
        find_pos(true);
    }
    // loads the row that `ahead` is at, and moves on
    const auto load = [&](int u) {
        if (ahead.item >= items) return;
        pos[u] = ahead.pos;
        const bool in = is_row(ahead);
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (whole) {
                    rx[u][k][e].load(ahead.row + at[k][e]);
                    if (BWD) rd[u][k][e].load(ahead.drow + at[k][e]);
                } else {
                    const bool here = in && at[k][e] >= 0;
                    rx[u][k][e].zero();
                    if (here) rx[u][k][e].load(ahead.row + at[k][e]);
                    if (BWD) {
                        rd[u][k][e].zero();
                        if (here) rd[u][k][e].load(ahead.drow + at[k][e]);
                    }
                }
            }
        ahead.row += step;
        if (BWD) ahead.drow += step;
        if (++ahead.it == ahead.end) {
            next(ahead, x, xs);
            if (BWD) ahead.drow = parts == 1 ? ahead.drow + (skip * ys - back) : dy + offset(ahead, ys);
            find_pos(false);
        }
    };

    if (go.item < items) enter(go, out, os);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) load(u);
    uint32_t angles_of = ~0u;  // token whose angles are at hand
    while (go.item < items) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (go.item >= items) break;
            if (angles_of != go.tok) {
                angles_of = go.tok;
                __syncwarp();
                const auto form = [&](int i, int32_t at_pos, float2 *to) {
                    const double t = (double)at_pos * ((double)p.inv_freq[i] * 0.15915494309189533577);
                    float2 cs;
                    sincospif(2.f * (float)(t - rint(t)), &cs.y, &cs.x);
                    put_angle<V, ADJ>(to, units, i / V, i % V, cs);
                };
                if (GROUP && group > 1) {
                    int i = l, g = 0;  // angle i of token g
                    for (int first = 0; first < half * group; first += 32, i += 32) {
                        while (i >= half) i -= half, ++g;
                        const int32_t at_pos = __shfl_sync(0xffffffffu, pos[u], g);
                        if (g < group) form(i, at_pos, angles[wi] + g * table);
                    }
                } else {
                    for (int i = l; i < half; i += 32) form(i, pos[u], angles[wi]);
                }
                __syncwarp();
            }
            float a[NU][2][V], g[NU][2][V];
            float2 s2 = both(0.f), dot2 = both(0.f);
            const bool in = is_row(go);
#pragma unroll
            for (int k = 0; k < NU; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    rx[u][k][e].get(a[k][e]);
                    if (BWD) rd[u][k][e].get(g[k][e]);
                }
            if (kUnroll == 1) load(u);  // at once, so that it overlaps the row's arithmetic
#pragma unroll
            for (int k = 0; k < NU; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) dot_into<V>(s2, a[k][e], a[k][e]);
                if (BWD) {
                    turn<V, ADJ, true>(g[k][0], g[k][1], turns + angle_at<V>(units, angle[k], 0), units, FULL ? V : half - angle[k] * V);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float w[V];
                        weights_of<V>(weights, units - 1, unit + k * p.lanes, e, w);
                        times<V>(w, g[k][e]);
                        dot_into<V>(dot2, w, a[k][e]);
                    }
                }
            }
            if (kUnroll > 1) load(u);
            float s = s2.x + s2.y, dot = dot2.x + dot2.y;
            for (int off = p.lanes >> 1; off > 0; off >>= 1) {
                s += __shfl_xor_sync(0xffffffffu, s, off);
                if (BWD) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            }
            const float r = scale_of(p, s);
            const float cd = p.norm == GDN_NORM_NONE ? 0.f : p.c * (r * dot);
#pragma unroll
            for (int k = 0; k < NU; ++k) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float w[V];
                    weights_of<V>(weights, units - 1, unit + k * p.lanes, e, w);
                    times<V>(a[k][e], r);
                    if (BWD) {
                        float cds[V];
#pragma unroll
                        for (int i = 0; i < V; ++i) cds[i] = -cd;
                        fma_into<V>(acc[k][e], g[k][e], a[k][e]);
                        times<V>(w, g[k][e]);
                        if (p.norm != GDN_NORM_NONE) fma_into<V>(w, a[k][e], cds);
                        times<V>(w, r);
#pragma unroll
                        for (int i = 0; i < V; ++i) a[k][e][i] = w[i];
                    } else {
                        times<V>(a[k][e], w);
                    }
                }
                if (!BWD) turn<V, ADJ, false>(a[k][0], a[k][1], turns + angle_at<V>(units, angle[k], 0), units, FULL ? V : half - angle[k] * V);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (whole || (in && at[k][e] >= 0)) Chunk<T, V, VEC>::store(go.row + at[k][e], a[k][e]);
            }
            go.row += step;
            if (++go.it == go.end) next(go, out, os);
        }
    }
    if (BWD && p.dw[which]) {
        // over the heads side by side, then over the block's warps
#pragma unroll
        for (int k = 0; k < NU; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float t = acc[k][e][i];
                    for (int off = 16; off >= p.lanes; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
                    if (sub == 0 && at[k][e] >= 0) sums[wi][at[k][e] + i] = t;
                }
        __syncthreads();
        for (int i = threadIdx.x; i < d; i += kThreads) {
            float t = 0.f;
            for (int k = 0; k < kWarps; ++k) t += sums[k][i];
            p.part[(int64_t)blockIdx.x * kMaxD + i] = t;
        }
    }
}

// The weights' gradients from the blocks' sums: 32 values per block of 32 x 32 threads.
__global__ void __launch_bounds__(1024) qk_dw_kernel(const __grid_constant__ QkParams p) {
    __shared__ float sums[32][33];
    const int which = blockIdx.y, i = blockIdx.x * 32 + threadIdx.x;
    if (!p.dw[which]) return;
    const float *part = p.part + (which ? (int64_t)p.blocks[0] * kMaxD : 0);
    float s = 0.f;
    if (i < p.d)
        for (int b = threadIdx.y; b < p.blocks[which]; b += 32) s += part[(int64_t)b * kMaxD + i];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && i < p.d) {
        s = 0.f;
        for (int b = 0; b < 32; ++b) s += sums[b][threadIdx.x];
        p.dw[which][i] = s;
    }
}

// ---------------------------------------------------------------- launches
template <typename T, int V, int NU, bool VEC, bool ADJ>
cudaError_t launch_units(QkParams p, bool bwd, cudaStream_t s) {
    const bool full = NU == 1 && p.rot == p.d;
    // lanes of a row: a power of two that its units fit
    const int half = p.rot / 2, units = ADJ ? (p.d + 2 * V - 1) / (2 * V) : half / V + (p.d - p.rot + 2 * V - 1) / (2 * V);
    p.lanes_log2 = 0;
    while ((1 << p.lanes_log2) < (units + NU - 1) / NU) ++p.lanes_log2;
    p.lanes = 1 << p.lanes_log2;
    p.whole = NU == 1 && p.lanes * 2 * V == p.d;
    const int side = 32 >> p.lanes_log2, most = kSms * (bwd ? kBwdPerSm : full ? kPerSm : kPartPerSm);
    // a warp takes all heads of a token, or fewer where that leaves warps without work, or several tokens
    // where their heads fit its lanes and every warp has some.  16384 tokens, bf16, without and with: 4 + 4
    // heads x 64 forward 20.5 and 18.3 us, backward 28.1 and 22.0 us; 8 + 2 x 64 backward 28.1 and 24.5 us.
    // The forward does so for both tensors or none (8 + 1 x 128: 27.1 us, 29.2 us with k alone)
    int64_t rows[2], items[2], blocks[2];
    for (int i = 0; i < 2; ++i) {
        rows[i] = (p.heads[i] + side - 1) / side;
        p.group[i] = 1;
        if (NU == 1 && p.tokens >= 2 * most * kWarps)
            while ((p.group[i] + 1) * p.heads[i] <= side && (p.group[i] + 1) * (p.lanes + 1) * V <= kAngles) ++p.group[i];
    }
    if (!bwd && (p.group[0] == 1 || p.group[1] == 1)) p.group[0] = p.group[1] = 1;
    for (int i = 0; i < 2; ++i) items[i] = (p.tokens + p.group[i] - 1) / p.group[i];
    const int64_t fair = (items[0] * rows[0] + items[1] * rows[1]) / (most * kWarps);  // rows per warp if all had some
    for (int i = 0; i < 2; ++i) {
        p.per[i] = (int32_t)(fair < 1 ? 1 : fair < rows[i] ? fair : rows[i]);
        p.parts[i] = (int32_t)((rows[i] + p.per[i] - 1) / p.per[i]);
        blocks[i] = (items[i] * p.parts[i] + kWarps - 1) / kWarps;
        if (blocks[i] < 1) blocks[i] = 1;
    }
    if (blocks[0] + blocks[1] > most) {
        // walk, with shares by the instructions: about 250 for a row (backward 430), 100 for an item and 60
        // for every 32 angles
        int64_t work[2];
        for (int i = 0; i < 2; ++i) work[i] = items[i] * (rows[i] * (bwd ? 14 : 8) + 3 + 2 * ((half * p.group[i] + 31) / 32));
        int64_t q = most * work[0] / (work[0] + work[1]);
        q = q < 1 ? 1 : q > most - 1 ? most - 1 : q;
        if (q < blocks[0]) blocks[0] = q;
        if (most - q < blocks[1]) blocks[1] = most - q;
    }
    p.blocks[0] = (int32_t)blocks[0];
    p.blocks[1] = (int32_t)blocks[1];
    const unsigned grid = (unsigned)(blocks[0] + blocks[1]);
    constexpr bool kVariants = NU == 1;
    const bool group = kVariants && (p.group[0] > 1 || p.group[1] > 1);
    using Kernel = void (*)(QkParams);
    const Kernel kernel = !bwd ? !group ? full ? qk_kernel<T, V, NU, VEC, ADJ, false, false, kVariants>
                                               : qk_kernel<T, V, NU, VEC, ADJ, false, false, false>
                                        : full ? qk_kernel<T, V, NU, VEC, ADJ, false, kVariants, kVariants>
                                               : qk_kernel<T, V, NU, VEC, ADJ, false, kVariants, false>
                               : !group ? full ? qk_kernel<T, V, NU, VEC, ADJ, true, false, kVariants>
                                               : qk_kernel<T, V, NU, VEC, ADJ, true, false, false>
                                        : full ? qk_kernel<T, V, NU, VEC, ADJ, true, kVariants, kVariants>
                                               : qk_kernel<T, V, NU, VEC, ADJ, true, kVariants, false>;
    if (!bwd) {
        if (p.tokens) GDN_LAUNCH(group ? kKQkRopeGroup : kKQkRope, s, kernel<<<grid, kThreads, 0, s>>>(p));
        return cudaSuccess;
    }
    if (p.tokens || p.dw[0] || p.dw[1]) GDN_LAUNCH(group ? kKQkRopeBwdGroup : kKQkRopeBwd, s, kernel<<<grid, kThreads, 0, s>>>(p));
    if (p.dw[0] || p.dw[1])
        GDN_LAUNCH(kKQkRopeDw, s, qk_dw_kernel<<<dim3((p.d + 31) / 32, 2), dim3(32, 32), 0, s>>>(p));
    return cudaSuccess;
}

// Whether rows split into whole, aligned chunks of v values.
bool chunks(const QkParams &p, bool bwd, int v) {
    int64_t all = p.d | p.xs[0] | p.xs[1] | p.ys[0] | p.ys[1];
    if (bwd) all |= p.dxs[0] | p.dxs[1];
    if (!p.interleaved) all |= p.rot / 2;
    return all % v == 0;
}

template <typename T>
cudaError_t launch(const QkParams &p, bool bwd, cudaStream_t s) {
    // 16-byte chunks; bf16 rows whose halves or strides are multiples of 4 only: 8-byte ones; other
    // rows value by value
    constexpr int kWide = 16 / sizeof(T);
    if (chunks(p, bwd, kWide))
        return p.interleaved ? launch_units<T, kWide, 1, true, true>(p, bwd, s) : launch_units<T, kWide, 1, true, false>(p, bwd, s);
    if (sizeof(T) == 2 && chunks(p, bwd, 4))
        return p.interleaved ? launch_units<T, 4, 1, true, true>(p, bwd, s) : launch_units<T, 4, 1, true, false>(p, bwd, s);
    return p.interleaved ? launch_units<T, 2, 4, false, true>(p, bwd, s) : launch_units<T, 1, 4, false, false>(p, bwd, s);
}

size_t workspace_bytes_needed() { return sizeof(float) * kSlots * kMaxD; }

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
