// Queries, keys and values between the product that makes them and the
// attention: the norm of each head with the position rotation in the same
// pass, its gradients, and a cache of keys and values in MXFP4 that is
// quantized as it is written.
//
// Per head x of d channels of a token at position p, in fp32:
//   s = 1 / sqrt(sum x^2 / d + eps), n = x s w,
//   (n_a, n_b) -> amp (n_a cos t - n_b sin t, n_b cos t + n_a sin t), t = p f_i,
// for the pairs i < r / 2 of the first r channels; the others are n.
//
// The angle is reduced in 64 bits: p f / (2 pi) less its nearest whole number is
// off by 2^-52 of itself, so by 2e-8 turns at 10^8 turns, where 32 bits would
// leave nothing of it past a few million. Sine and cosine of the rest are taken
// in 32 bits.
//
// A head is held by LG neighbouring lanes. A lane has U units of it, each two
// pieces of V neighbouring channels: for pairs (i, i + r / 2) the two pieces are
// partners, and pairs (2 i, 2 i + 1) lie inside a piece, so a rotation never
// leaves its lane. V is 8 or 4 channels (16-byte or 8-byte accesses) where sizes
// and alignment allow, else 1.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>

#include "kq.h"
#include "kq_chunk.hpp"
#include "kq_cvt.hpp"
#include "kq_device.hpp"
#include "kq_host.hpp"
#include "kq_lanesum.hpp"

namespace kq {
namespace heads {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kBackThreads = 512, kBackWaves = kBackThreads / 64;

struct Rope {
    const int64_t *pos;  // [m][axes]
    const double *freq;  // [half], radians per position
    float amp;
    int axes, upto[4];   // pairs below upto[a] (and not below upto[a - 1]) turn with axis a
    int d, half;         // channels per head, rotated pairs
};

// Rows are the heads of `tokens` tokens of a workgroup, heads of a token side by side.
struct Geom {
    int64_t m;
    int heads, second;  // heads per token; those from `second` on take the second weight
    int tokens;         // per workgroup (a block of them)
    int split_rows;     // forward: rows per workgroup of a block
    int norm;
    float eps;
};

// V neighbouring elements as they are loaded.
template <class T, int V>
struct Piece {
    static constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t q[kWords];
    __device__ __forceinline__ void load(const T *p) { __builtin_memcpy(q, __builtin_assume_aligned(p, kWords > 2 ? 16 : 4 * kWords), 4 * kWords); }
    __device__ __forceinline__ void widen(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if (sizeof(T) == 2) {
                x[2 * i] = bf16_lo(q[i]);
                x[2 * i + 1] = bf16_hi(q[i]);
            } else {
                x[i] = __uint_as_float(q[i]);
            }
        }
    }
};
template <>
struct Piece<uint16_t, 1> {
    uint32_t q;
    __device__ __forceinline__ void load(const uint16_t *p) { q = *p; }
    __device__ __forceinline__ void widen(float (&x)[1]) const { x[0] = bf16_lo(q); }
};

template <int V>
__device__ __forceinline__ void store_values(float *p, const float (&x)[V]) {
    if constexpr (V == 1) {
        *p = x[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) *reinterpret_cast<floatx4_t *>(p + i) = floatx4_t{x[i], x[i + 1], x[i + 2], x[i + 3]};
    }
}
template <int V>
__device__ __forceinline__ void store_values(uint16_t *p, const float (&x)[V]) {
    if constexpr (V == 1) {
        store1(p, x[0]);
    } else {
        typedef uint32_t words_t __attribute__((ext_vector_type(V / 2)));
        words_t q;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) q[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        *reinterpret_cast<words_t *>(p) = q;
    }
}

// Sum over the LG lanes of a head (all lanes of the wave take part).
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
    if (LG >= 2) v += moved<0xB1>(v);
    if (LG >= 4) v += moved<0x4E>(v);
    if (LG >= 8) v += moved<0x141>(v);
    if (LG >= 16) v += moved<0x140>(v);
    if (LG >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (LG >= 64) {
        const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        v = __uint_as_float(q[0]) + __uint_as_float(q[1]);
    }
    return v;
}

// Where unit u of a head lies: its first piece at channel a, its second at b, and whether they exist and are rotated.
struct Place {
    int a, b;
    bool in_a, in_b, rot_a, rot_b;
};
template <int V, bool INTER>
__device__ __forceinline__ Place place_of(int u, int d, int half) {
    const int r = 2 * half;
    Place p;
    if (INTER && V > 1) {
        const int n = d / V, h = (n + 1) / 2;
        p.in_a = u < h;
        p.in_b = u + h < n && p.in_a;
        p.a = V * u;
        p.b = V * (u + h);
        p.rot_a = p.a < r;
        p.rot_b = p.b < r;
    } else if (u < half / V) {
        p.a = INTER ? 2 * u : V * u;
        p.b = INTER ? 2 * u + 1 : half + V * u;
        p.in_a = p.in_b = p.rot_a = p.rot_b = true;
    } else {
        const int n = (d - r) / V, h = (n + 1) / 2, w = u - half / V;
        p.in_a = w < h;
        p.in_b = w + h < n && p.in_a;
        p.a = r + V * w;
        p.b = r + V * (w + h);
        p.rot_a = p.rot_b = false;
    }
    // a missing piece reads the head's first (and counts for nothing)
    if (!p.in_a) p.a = 0, p.rot_a = false;
    if (!p.in_b) p.b = 0, p.rot_b = false;
    return p;
}

// (amp cos t, amp sin t) of the block's tokens in LDS, token by token, and after the last V times (1, 0), what
// the channels that are not rotated use.
__device__ __forceinline__ void fill_table(float2 *table, const Rope &rope, int64_t t0, int tokens, int tid, int threads) {
    const int n = tokens * rope.half;
    for (int i = tid; i < n; i += threads) {
        const int t = i / rope.half, j = i - t * rope.half;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < 3; ++a) axis += a + 1 < rope.axes && j >= rope.upto[a];
        const double turns = (double)rope.pos[(t0 + t) * rope.axes + axis] * (rope.freq[j] * 0.15915494309189534);
        const float x = 2.0f * (float)(turns - rint(turns));
        float s, c;
        sincospif(x, &s, &c);
        table[i] = make_float2(c * rope.amp, s * rope.amp);
    }
    if (tid < 8) table[n + tid] = make_float2(1.0f, 0.0f);
}

// The pieces (a, b) of one unit turned by their angles, BACK: by the opposite ones.
template <int V, bool INTER, bool BACK>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float2 *table, int token, int none,
                                     const Place &p, const Rope &rope) {
    const float2 *ta, *tb;
    if (INTER && V > 1) {
        ta = table + (p.rot_a ? token * rope.half + p.a / 2 : none);
        tb = table + (p.rot_b ? token * rope.half + p.b / 2 : none);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 ca = ta[e / 2], cb = tb[e / 2];
            const float sa = BACK ? -ca.y : ca.y, sb = BACK ? -cb.y : cb.y;
            const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
            a[e] = fmaf(a0, ca.x, -(a1 * sa));
            a[e + 1] = fmaf(a1, ca.x, a0 * sa);
            b[e] = fmaf(b0, cb.x, -(b1 * sb));
            b[e + 1] = fmaf(b1, cb.x, b0 * sb);
        }
    } else {
        ta = table + (p.rot_a ? token * rope.half + (INTER ? p.a / 2 : p.a) : none);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 c = ta[e];
            const float s = BACK ? -c.y : c.y, x = a[e], y = b[e];
            a[e] = fmaf(x, c.x, -(y * s));
            b[e] = fmaf(y, c.x, x * s);
        }
    }
}

// X and Y may be the same memory: a lane has read all of its pieces before it writes any of them.
// A workgroup takes the heads of a few tokens; a wave 64 / LG of them at a time, the next ones' loads in flight
// while these are finished. The table of angles is made once per token and read back by every head.
template <class T, int V, int LG, int U, bool INTER>
__global__ __launch_bounds__(kThreads) void forward_kernel(const T *X, int64_t ldx, int64_t hsx,
                                                           const float *__restrict__ w0, const float *__restrict__ w1,
                                                           Geom g, Rope rope, T *Y, int64_t ldy,
                                                           int64_t hsy) {
    extern __shared__ float2 table[];
    constexpr int HP = 64 / LG, G = U > 1 ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sub = lane % LG, slot = lane / LG;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens);
    const int row0 = (int)blockIdx.y * g.split_rows;
    const int row1 = min(row0 + g.split_rows, tokens * g.heads);
    if (row0 >= row1) return;
    const float inv_heads = 1.0f / (float)g.heads, inv_d = 1.0f / (float)rope.d;
    const int none = tokens * rope.half;

    Place at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = place_of<V, INTER>(sub + LG * u, rope.d, rope.half);
    struct Row {
        Piece<T, V> a[U], b[U];
    };
    // row r's token (of the block) and head
    auto split = [&](int r, int &t, int &h) {
        t = (int)(((float)r + 0.5f) * inv_heads);
        h = r - t * g.heads;
    };
    auto fetch = [&](Row (&to)[G], int first) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
            int t, h;
            split(min(first + kWaves * HP * i + slot, row1 - 1), t, h);
            const T *x = X + (t0 + t) * ldx + h * hsx;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                to[i].a[u].load(x + at[u].a);
                to[i].b[u].load(x + at[u].b);
            }
        }
    };
    Row now[G], next[G];
    int first = row0 + wave * HP;
    fetch(next, first);
    float wv[2][U][2][V];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float *w = k ? w1 : w0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                wv[k][u][0][e] = g.norm && w ? w[at[u].a + e] : 1.0f;
                wv[k][u][1][e] = g.norm && w ? w[at[u].b + e] : 1.0f;
            }
    }
    fill_table(table, rope, t0, tokens, tid, kThreads);
    __syncthreads();
    for (; first < row1; first += kWaves * HP * G) {
#pragma unroll
        for (int i = 0; i < G; ++i) now[i] = next[i];
        if (first + kWaves * HP * G < row1) fetch(next, first + kWaves * HP * G);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int r = first + kWaves * HP * i + slot;
            int t, h;
            split(min(r, row1 - 1), t, h);
            float a[U][V], b[U][V], s = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                now[i].a[u].widen(a[u]);
                now[i].b[u].widen(b[u]);
                float sa = 0.f, sb = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sa = fmaf(a[u][e], a[u][e], sa);
                    sb = fmaf(b[u][e], b[u][e], sb);
                }
                s += (at[u].in_a ? sa : 0.f) + (at[u].in_b ? sb : 0.f);
            }
            if (g.norm) {
                const float rs = __builtin_amdgcn_rsqf(fmaf(group_sum<LG>(s), inv_d, g.eps));
                const bool second = h >= g.second;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        a[u][e] = a[u][e] * rs * (second ? wv[1][u][0][e] : wv[0][u][0][e]);
                        b[u][e] = b[u][e] * rs * (second ? wv[1][u][1][e] : wv[0][u][1][e]);
                    }
            }
            T *y = Y + (t0 + t) * ldy + h * hsy;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                turn<V, INTER, false>(a[u], b[u], table, t, none, at[u], rope);
                if (r < row1 && at[u].in_a) store_values(y + at[u].a, a[u]);
                if (r < row1 && at[u].in_b) store_values(y + at[u].b, b[u]);
            }
        }
    }
}

// Gradients. With e the gradient turned back, h = x s and g = e w:
//   dx = s (g - h sum(g h) / d), dw = sum of e h over the rows of that weight.
// Workgroup p of `parts` takes the blocks of tokens p, p + parts, ...; its lanes keep their channels of both dw in
// registers, and row p of the partial sums gets them at the end, the waves joined in their order.
template <class T, int V, int LG, int U, bool INTER>
__global__ __launch_bounds__(kBackThreads) void backward_kernel(const T *dY, int64_t lddy, int64_t hsdy,
                                                                const T *X, int64_t ldx, int64_t hsx,
                                                                const float *__restrict__ w0,
                                                                const float *__restrict__ w1, Geom g, Rope rope,
                                                                T *dX, int64_t lddx, int64_t hsdx,
                                                                int parts, float *__restrict__ p0,
                                                                float *__restrict__ p1) {
    extern __shared__ float2 table[];
    constexpr int HP = 64 / LG;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sub = lane % LG, slot = lane / LG;
    const float inv_heads = 1.0f / (float)g.heads, inv_d = 1.0f / (float)rope.d;
    Place at[U];
    float wv[2][U][2][V], acc[2][U][2][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        at[u] = place_of<V, INTER>(sub + LG * u, rope.d, rope.half);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float *w = k ? w1 : w0;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                wv[k][u][0][e] = g.norm && w ? w[at[u].a + e] : 1.0f;
                wv[k][u][1][e] = g.norm && w ? w[at[u].b + e] : 1.0f;
                acc[k][u][0][e] = acc[k][u][1][e] = 0.f;
            }
        }
    }
    struct Row {
        Piece<T, V> a[U], b[U], da[U], db[U];
    };
    auto split = [&](int r, int &t, int &h) {
        t = (int)(((float)r + 0.5f) * inv_heads);
        h = r - t * g.heads;
    };
    const int64_t blocks = (g.m + g.tokens - 1) / g.tokens;
    int par = 0;
    for (int64_t block = blockIdx.x; block < blocks; block += parts, par ^= 1) {
        const int64_t t0 = block * g.tokens;
        const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens), rows = tokens * g.heads;
        const int none = tokens * rope.half;
        // two tables in turn: one is written again only after the next block's barrier
        float2 *tab = table + par * (g.tokens * rope.half + 8);
        Row now, next;
        auto fetch = [&](int first) {
            int t, h;
            split(min(first + slot, rows - 1), t, h);
            const T *dy = dY + (t0 + t) * lddy + h * hsdy;
            const T *x = X + (t0 + t) * ldx + h * hsx;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                next.da[u].load(dy + at[u].a);
                next.db[u].load(dy + at[u].b);
                if (g.norm) {
                    next.a[u].load(x + at[u].a);
                    next.b[u].load(x + at[u].b);
                }
            }
        };
        int first = wave * HP;
        fetch(first);
        fill_table(tab, rope, t0, tokens, tid, kBackThreads);
        __syncthreads();
        for (; first < rows; first += kBackWaves * HP) {
            now = next;
            if (first + kBackWaves * HP < rows) fetch(first + kBackWaves * HP);
            const int r = first + slot;
            int t, h;
            split(min(r, rows - 1), t, h);
            const bool second = h >= g.second;
            T *dx = dX + (t0 + t) * lddx + h * hsdx;
            float ea[U][V], eb[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                now.da[u].widen(ea[u]);
                now.db[u].widen(eb[u]);
                turn<V, INTER, true>(ea[u], eb[u], tab, t, none, at[u], rope);
            }
            if (g.norm) {
                float xa[U][V], xb[U][V], s = 0.f, q = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    now.a[u].widen(xa[u]);
                    now.b[u].widen(xb[u]);
                    float sa = 0.f, sb = 0.f, qa = 0.f, qb = 0.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        sa = fmaf(xa[u][e], xa[u][e], sa);
                        sb = fmaf(xb[u][e], xb[u][e], sb);
                        qa = fmaf(xa[u][e] * (second ? wv[1][u][0][e] : wv[0][u][0][e]), ea[u][e], qa);
                        qb = fmaf(xb[u][e] * (second ? wv[1][u][1][e] : wv[0][u][1][e]), eb[u][e], qb);
                    }
                    s += (at[u].in_a ? sa : 0.f) + (at[u].in_b ? sb : 0.f);
                    q += (at[u].in_a ? qa : 0.f) + (at[u].in_b ? qb : 0.f);
                }
                const float rs = __builtin_amdgcn_rsqf(fmaf(group_sum<LG>(s), inv_d, g.eps));
                const float c = group_sum<LG>(q) * rs * inv_d;
                const bool in0 = r < rows && !second, in1 = r < rows && second;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float ha = xa[u][e] * rs, hb = xb[u][e] * rs;
                        const float va = ea[u][e] * ha, vb = eb[u][e] * hb;
                        acc[0][u][0][e] += in0 ? va : 0.f;
                        acc[0][u][1][e] += in0 ? vb : 0.f;
                        acc[1][u][0][e] += in1 ? va : 0.f;
                        acc[1][u][1][e] += in1 ? vb : 0.f;
                        ea[u][e] = rs * fmaf(-ha, c, ea[u][e] * (second ? wv[1][u][0][e] : wv[0][u][0][e]));
                        eb[u][e] = rs * fmaf(-hb, c, eb[u][e] * (second ? wv[1][u][1][e] : wv[0][u][1][e]));
                    }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r < rows && at[u].in_a) store_values(dx + at[u].a, ea[u]);
                if (r < rows && at[u].in_b) store_values(dx + at[u].b, eb[u]);
            }
        }
    }
    if (!p0 && !p1) return;
    // the rows side by side in a wave, then the waves, in their order
    constexpr int kWave = LG * U * 2 * V;
    float *join = reinterpret_cast<float *>(table);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float v = acc[k][u][b][e];
#pragma unroll
                    for (int o = LG; o < 64; o *= 2) v += __shfl_xor(v, o);
                    if (slot == 0) join[(wave * 2 + k) * kWave + ((u * 2 + b) * V + e) * LG + sub] = v;
                }
    __syncthreads();
    for (int i = tid; i < 2 * kWave; i += kBackThreads) {
        const int k = i / kWave, j = i % kWave, s = j % LG, e = j / LG % V, b = j / (LG * V) % 2, u = j / (LG * V * 2);
        float *part = k ? p1 : p0;
        const Place p = place_of<V, INTER>(s + LG * u, rope.d, rope.half);
        if (!part || !(b ? p.in_b : p.in_a)) continue;
        float v = join[k * kWave + j];
#pragma unroll
        for (int w = 1; w < kBackWaves; ++w) v += join[(w * 2 + k) * kWave + j];
        part[(int64_t)blockIdx.x * rope.d + (b ? p.b : p.a) + e] = v;
    }
}

// Keys and values of a block of tokens into the cache: rows are a token's key heads, normed and turned as above, then
// its value heads, as they are. A wave's rows meet in LDS, where four lanes take each block of 32 channels.
struct Cache {
    const int64_t *slots;  // [m]
    int64_t n;             // slots of the cache
    int keys, values;      // heads of each per token
    uint8_t *codes[2], *scales[2];
};
template <class T, int V, int LG, int U, bool INTER>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(const T *__restrict__ K, int64_t ldk, int64_t hsk,
                                                               const T *__restrict__ Vx, int64_t ldv, int64_t hsv,
                                                               const float *__restrict__ w, Geom g, Rope rope,
                                                               Cache cache, int stage_at) {
    extern __shared__ float2 table[];
    constexpr int HP = 64 / LG;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sub = lane % LG, slot = lane / LG;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens);
    const int row0 = (int)blockIdx.y * g.split_rows;
    const int row1 = min(row0 + g.split_rows, tokens * g.heads);
    if (row0 >= row1) return;
    const float inv_heads = 1.0f / (float)g.heads, inv_d = 1.0f / (float)rope.d;
    const int none = tokens * rope.half, d = rope.d;
    float *stage = reinterpret_cast<float *>(table) + stage_at + wave * HP * d;

    Place at[U];
    float wv[U][2][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        at[u] = place_of<V, INTER>(sub + LG * u, d, rope.half);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            wv[u][0][e] = g.norm && w ? w[at[u].a + e] : 1.0f;
            wv[u][1][e] = g.norm && w ? w[at[u].b + e] : 1.0f;
        }
    }
    auto split = [&](int r, int &t, int &h) {
        t = (int)(((float)r + 0.5f) * inv_heads);
        h = r - t * g.heads;
    };
    struct Row {
        Piece<T, V> a[U], b[U];
    } now, next;
    auto fetch = [&](int first) {
        int t, h;
        split(min(first + slot, row1 - 1), t, h);
        const T *x = h < cache.keys ? K + (t0 + t) * ldk + h * hsk : Vx + (t0 + t) * ldv + (h - cache.keys) * hsv;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            next.a[u].load(x + at[u].a);
            next.b[u].load(x + at[u].b);
        }
    };
    int first = row0 + wave * HP;
    fetch(first);
    fill_table(table, rope, t0, tokens, tid, kThreads);
    __syncthreads();
    for (; first < row1; first += kWaves * HP) {
        now = next;
        if (first + kWaves * HP < row1) fetch(first + kWaves * HP);
        int t, h;
        split(min(first + slot, row1 - 1), t, h);
        const bool key = h < cache.keys;
        float a[U][V], b[U][V], s = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            now.a[u].widen(a[u]);
            now.b[u].widen(b[u]);
            float sa = 0.f, sb = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                sa = fmaf(a[u][e], a[u][e], sa);
                sb = fmaf(b[u][e], b[u][e], sb);
            }
            s += (at[u].in_a ? sa : 0.f) + (at[u].in_b ? sb : 0.f);
        }
        if (g.norm) {
            const float rs = __builtin_amdgcn_rsqf(fmaf(group_sum<LG>(s), inv_d, g.eps));
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    a[u][e] = key ? a[u][e] * rs * wv[u][0][e] : a[u][e];
                    b[u][e] = key ? b[u][e] * rs * wv[u][1][e] : b[u][e];
                }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Place p = at[u];
            p.rot_a = p.rot_a && key;
            p.rot_b = p.rot_b && key;
            turn<V, INTER, false>(a[u], b[u], table, t, none, p, rope);
            if (p.in_a) store_values(stage + slot * d + p.a, a[u]);
            if (p.in_b) store_values(stage + slot * d + p.b, b[u]);
        }
        // a wave's LDS accesses stay in order; nothing may move across this point
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int pieces = d / 8, rows = min(HP, row1 - first);
        for (int i = lane; i < rows * pieces; i += 64) {
            const int q = i / pieces, c = i - q * pieces;
            split(first + q, t, h);
            const int64_t to = cache.slots[t0 + t];
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const floatx4_t v = *reinterpret_cast<const floatx4_t *>(stage + q * d + 8 * c + e);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[e + j] = v[j];
            }
            uint32_t sbyte;
            const uint32_t code = quantize_quad_f32(x, sbyte);
            if (to < 0 || to >= cache.n) continue;
            const int which = h < cache.keys ? 0 : 1;
            const int64_t row = which ? to * cache.values + (h - cache.keys) : to * cache.keys + h;
            *reinterpret_cast<uint32_t *>(cache.codes[which] + row * (d / 2) + 4 * c) = code;
            if ((lane & 3) == 0) cache.scales[which][row * (d / 32) + c / 4] = (uint8_t)sbyte;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

// Rows of the cache decoded: a lane takes 8 channels (a dword of codes) at a time. A row whose slot lies outside the
// cache is zeros.
template <class T>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(const int64_t *__restrict__ slots, int64_t m, int64_t n,
                                                              const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, int heads, int d,
                                                              T *__restrict__ Y, int64_t ldy, int64_t hsy, int vec) {
    const int pieces = d / 8, row = heads * pieces;
    for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < m * row; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / row;
        const int at = (int)(i - t * row), h = at / pieces, c = at - h * pieces;
        const int64_t from = slots[t];
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (from >= 0 && from < n) {
            const int64_t r = from * heads + h;
            const uint32_t code = *reinterpret_cast<const uint32_t *>(codes + r * (d / 2) + 4 * c);
            const uint32_t s = scales[r * (d / 32) + c / 4];
            const bf16x8_t v = decode_fp4x8_bf16_cvt(code, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
        }
        T *y = Y + t * ldy + h * hsy + 8 * c;
        if (vec) {
            store_values(y, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) store1(y + e, x[e]);
        }
    }
}

}  // namespace heads
}  // namespace kq

// ===========================================================================
// Host side
// ===========================================================================
namespace {

using kq::heads::Geom;
using kq::heads::Rope;
using kqhost::aligned;
using kqhost::launched;
using kqhost::sizes_fit;

bool good_type(int type) { return type == KQ_F32 || type == KQ_BF16; }

// A tensor [m][heads][d] with unit channel stride; strides of one token or one head do not matter.
struct Tensor {
    const void *p;
    int64_t ld, hs;
    Tensor(const void *p_, int64_t ld_, int64_t hs_, int64_t m, int64_t heads)
        : p(p_), ld(m > 1 ? ld_ : 0), hs(heads > 1 ? hs_ : 0) {}
};

// Whether rows of d elements at these strides do not overlap: heads inside tokens or tokens inside heads.
bool apart(int64_t m, int64_t heads, int64_t d, int64_t ld, int64_t hs) {
    if (m == 0 || heads == 0 || d == 0 || (m == 1 && heads == 1)) return true;
    if (m <= 1) return hs >= d;
    if (heads <= 1) return ld >= d;
    return (hs >= d && ld >= (heads - 1) * hs + d) || (ld >= d && hs >= (m - 1) * ld + d);
}

// The rotation's arguments (host); NULL: none.
kq_status read_rope(const kq_rope *r, int64_t m, int64_t d, Rope &out) {
    out = Rope{nullptr, nullptr, 1.0f, 1, {0, 0, 0, 0}, (int)d, 0};
    if (!r || r->rot == 0) return KQ_OK;
    if (r->rot < 0 || r->rot > d || r->rot % 2 != 0) return KQ_ERR_SHAPE;
    if (r->axes < 1 || r->axes > 4) return KQ_ERR_UNSUPPORTED;
    int64_t sum = 0;
    for (int a = 0; a < r->axes; ++a) {
        if (r->axis_pairs[a] < 0 || r->axis_pairs[a] > r->rot / 2) return KQ_ERR_SHAPE;
        sum += r->axis_pairs[a];
        out.upto[a] = (int)sum;
    }
    if (sum != r->rot / 2) return KQ_ERR_SHAPE;
    if (m > 0 && (!r->positions || !r->freq)) return KQ_ERR_NULL;
    if (!aligned(r->positions, 8) || !aligned(r->freq, 8)) return KQ_ERR_ALIGN;
    out.pos = r->positions;
    out.freq = r->freq;
    out.amp = r->amplitude;
    out.axes = r->axes;
    out.half = (int)(r->rot / 2);
    return KQ_OK;
}

// Channels per piece: 8 or 4 where the halves of the rotated part (the whole of it with neighbouring pairs), the head
// and every address are multiples of it.
int piece_width(int es, const Rope &rope, bool inter, std::initializer_list<Tensor> tensors) {
    for (int v = 8; v >= 4; v /= 2) {
        const int bytes = v * es < 16 ? v * es : 16;
        bool ok = rope.d % v == 0 && (inter ? 2 * rope.half : rope.half) % v == 0;
        for (const Tensor &t : tensors)
            ok = ok && aligned(t.p, bytes) && t.ld * es % bytes == 0 && t.hs * es % bytes == 0;
        if (ok) return v;
    }
    return 1;
}

int units_of(const Rope &rope, bool inter, int v) {
    if (inter && v > 1) return (rope.d / v + 1) / 2;
    return rope.half / v + ((rope.d - 2 * rope.half) / v + 1) / 2;
}

// f(V, LG, U): the smallest group of lanes that holds a head, more units a lane where 64 do not.
template <int V, int LG, int U>
struct Form {
    static constexpr int kV = V, kLG = LG, kU = U;
};
template <class F>
void choose_form(int v, int units, F f) {
    if (v == 8) {
        if (units <= 4) f(Form<8, 4, 1>());
        else if (units <= 8) f(Form<8, 8, 1>());
        else if (units <= 16) f(Form<8, 16, 1>());
        else if (units <= 32) f(Form<8, 32, 1>());
        else f(Form<8, 64, 1>());
    } else if (v == 4) {
        if (units <= 8) f(Form<4, 8, 1>());
        else if (units <= 16) f(Form<4, 16, 1>());
        else if (units <= 32) f(Form<4, 32, 1>());
        else if (units <= 64) f(Form<4, 64, 1>());
        else f(Form<4, 64, 2>());
    } else {
        if (units <= 16) f(Form<1, 16, 1>());
        else if (units <= 64) f(Form<1, 64, 1>());
        else if (units <= 128) f(Form<1, 64, 2>());
        else if (units <= 256) f(Form<1, 64, 4>());
        else f(Form<1, 64, 8>());
    }
}

constexpr int kTable = 2048;  // angles of a block of tokens, 16 KB of LDS

// Tokens per workgroup and, for few of them, the parts that a block's rows are split into: four passes a
// wave where that leaves four workgroups per compute unit.
struct Plan {
    int tokens, split_rows;
    int64_t blocks, splits;
};
Plan plan_of(int64_t m, int64_t heads, int half, int hp) {
    const int64_t waves = kq::heads::kWaves, cus = kqhost::compute_units();
    int64_t t = (4 * waves * hp + heads - 1) / heads;
    if (half > 0 && t * half > kTable) t = kTable / half;
    if (t > m / (4 * cus)) t = m / (4 * cus);
    if (t < 1) t = 1;
    Plan p;
    p.tokens = (int)t;
    p.blocks = (m + t - 1) / t;
    const int64_t passes = (t * heads + hp - 1) / hp;
    int64_t s = (passes + waves - 1) / waves;
    const int64_t want = (2 * cus + p.blocks - 1) / p.blocks;
    if (s > want) s = want;
    const int64_t per = (passes + s - 1) / s;
    p.split_rows = (int)(per * hp);
    p.splits = (passes + per - 1) / per;
    return p;
}

template <class T>
kq_status launch_forward(const Tensor &x, const Tensor &y, const float *w0, const float *w1, Geom g, const Rope &rope,
                         bool inter, kq_stream_t stream) {
    const int v = piece_width(sizeof(T), rope, inter, {x, y});
    kq_status status = KQ_OK;
    choose_form(v, units_of(rope, inter, v), [&](auto form) {
        constexpr int V = decltype(form)::kV, LG = decltype(form)::kLG, U = decltype(form)::kU;
        const Plan p = plan_of(g.m, g.heads, rope.half, 64 / LG);
        if (p.blocks >= (int64_t)1 << 24) {
            status = KQ_ERR_UNSUPPORTED;
            return;
        }
        g.tokens = p.tokens;
        g.split_rows = p.split_rows;
        const size_t lds = (size_t)(p.tokens * rope.half + 8) * sizeof(float2);
        auto go = [&](auto I) {
            hipLaunchKernelGGL((kq::heads::forward_kernel<T, V, LG, U, I()>), dim3((unsigned)p.blocks, (unsigned)p.splits),
                               dim3(kq::heads::kThreads), lds, (hipStream_t)stream, (const T *)x.p, x.ld, x.hs, w0, w1, g,
                               rope, (T *)const_cast<void *>(y.p), y.ld, y.hs);
        };
        if (inter) go(std::true_type());
        else go(std::false_type());
        status = launched();
    });
    return status;
}

template <class T>
kq_status launch_backward(const Tensor &dy, const Tensor &x, const Tensor &dx, const float *w0, const float *w1, Geom g,
                          const Rope &rope, bool inter, int parts, float *p0, float *p1, kq_stream_t stream) {
    const int v = g.norm ? piece_width(sizeof(T), rope, inter, {dy, x, dx}) : piece_width(sizeof(T), rope, inter, {dy, dx});
    kq_status status = KQ_OK;
    choose_form(v, units_of(rope, inter, v), [&](auto form) {
        constexpr int V = decltype(form)::kV, LG = decltype(form)::kLG, U = decltype(form)::kU;
        constexpr int waves = kq::heads::kBackWaves, HP = 64 / LG;
        // a part's tokens in as many whole blocks as give each wave about four passes
        const int64_t per = (g.m + parts - 1) / parts;
        int64_t want = (4 * waves * HP + g.heads - 1) / g.heads;
        if (rope.half > 0 && want * rope.half > kTable) want = kTable / rope.half;
        if (want < 1) want = 1;
        const int64_t rounds = per > want ? (per + want - 1) / want : 1;
        g.tokens = (int)((per + rounds - 1) / rounds);
        const size_t tables = 2 * (size_t)(g.tokens * rope.half + 8) * sizeof(float2);
        const size_t join = (size_t)waves * 2 * LG * U * 2 * V * sizeof(float);
        auto go = [&](auto I) {
            hipLaunchKernelGGL((kq::heads::backward_kernel<T, V, LG, U, I()>), dim3((unsigned)parts),
                               dim3(kq::heads::kBackThreads), tables > join ? tables : join, (hipStream_t)stream,
                               (const T *)dy.p, dy.ld, dy.hs, (const T *)x.p, x.ld, x.hs, w0, w1, g, rope,
                               (T *)const_cast<void *>(dx.p), dx.ld, dx.hs, parts, p0, p1);
        };
        if (inter) go(std::true_type());
        else go(std::false_type());
        status = launched();
    });
    return status;
}

template <class T>
kq_status launch_write(const Tensor &k, const Tensor &v_, const float *w, Geom g, const Rope &rope, bool inter,
                       const kq::heads::Cache &cache, kq_stream_t stream) {
    const int v = piece_width(sizeof(T), rope, inter, {k, v_});
    kq_status status = KQ_OK;
    choose_form(v, units_of(rope, inter, v), [&](auto form) {
        constexpr int V = decltype(form)::kV, LG = decltype(form)::kLG, U = decltype(form)::kU;
        const Plan p = plan_of(g.m, g.heads, rope.half, 64 / LG);
        if (p.blocks >= (int64_t)1 << 24) {
            status = KQ_ERR_UNSUPPORTED;
            return;
        }
        g.tokens = p.tokens;
        g.split_rows = p.split_rows;
        const int stage_at = (2 * (p.tokens * rope.half + 8) + 3) / 4 * 4;  // in floats, 16-byte aligned
        const size_t lds = (size_t)(stage_at + kq::heads::kWaves * (64 / LG) * rope.d) * sizeof(float);
        auto go = [&](auto I) {
            hipLaunchKernelGGL((kq::heads::cache_write_kernel<T, V, LG, U, I()>),
                               dim3((unsigned)p.blocks, (unsigned)p.splits), dim3(kq::heads::kThreads), lds,
                               (hipStream_t)stream, (const T *)k.p, k.ld, k.hs, (const T *)v_.p, v_.ld, v_.hs, w, g, rope,
                               cache, stage_at);
        };
        if (inter) go(std::true_type());
        else go(std::false_type());
        status = launched();
    });
    return status;
}

bool good_eps(float eps) { return eps >= 0.f && eps <= 3.4e38f; }

constexpr int64_t kMostChannels = 1024, kMostHeads = 65536;

}  // namespace

extern "C" {

kq_status kq_rope_frequencies(int64_t rot, double base, int scaling, double factor, double original, double low,
                              double high, double *freq) {
    if (rot < 0 || rot % 2 != 0 || !(base > 0) || !(base < HUGE_VAL)) return KQ_ERR_SHAPE;
    if (scaling < KQ_ROPE_PLAIN || scaling > KQ_ROPE_PARTS) return KQ_ERR_UNSUPPORTED;
    if (scaling != KQ_ROPE_PLAIN && (!(factor > 0) || !(factor < HUGE_VAL))) return KQ_ERR_SHAPE;
    if (scaling == KQ_ROPE_PARTS && (!(original > 0) || !(original < HUGE_VAL) || !(low < high) || !(low > -HUGE_VAL) || !(high < HUGE_VAL)))
        return KQ_ERR_SHAPE;
    if (rot == 0) return KQ_OK;
    if (!freq) return KQ_ERR_NULL;
    if (scaling == KQ_ROPE_BASE && rot > 2) base *= pow(factor, (double)rot / (double)(rot - 2));
    for (int64_t i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * (double)i / (double)rot);
        if (scaling == KQ_ROPE_LINEAR) f /= factor;
        if (scaling == KQ_ROPE_PARTS) {
            const double turns = original * f * 0.15915494309189535;
            double keep = (turns - low) / (high - low);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = keep * f + (1 - keep) * (f / factor);
        }
        freq[i] = f;
    }
    return KQ_OK;
}

kq_status kq_headnorm_rope(const void *X, int type, int64_t m, int64_t heads, int64_t d, int64_t ldx, int64_t hsx,
                           int norm, const float *weight_q, const float *weight_k, int64_t q_heads, float eps,
                           const kq_rope *rope, void *Y, int64_t ldy, int64_t hsy, kq_stream_t stream) {
    if (m < 0 || heads < 0 || d < 0 || q_heads < 0 || q_heads > heads || ldx < 0 || hsx < 0 || ldy < 0 || hsy < 0 ||
        !good_eps(eps))
        return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, heads, d, ldx, hsx, ldy, hsy}) || d > kMostChannels || heads > kMostHeads)
        return KQ_ERR_UNSUPPORTED;
    if (!apart(m, heads, d, ldy, hsy)) return KQ_ERR_SHAPE;
    Rope r;
    const kq_status s = read_rope(rope, m, d, r);
    if (s != KQ_OK) return s;
    if (m == 0 || heads == 0 || d == 0) return KQ_OK;
    if (!X || !Y) return KQ_ERR_NULL;
    const uintptr_t es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(X, es) || !aligned(Y, es) || !aligned(weight_q, 4) || !aligned(weight_k, 4)) return KQ_ERR_ALIGN;
    const Geom g{m, (int)heads, (int)q_heads, 0, 0, norm != 0, eps};
    const Tensor x(X, ldx, hsx, m, heads), y(Y, ldy, hsy, m, heads);
    const bool inter = r.half > 0 && rope->interleaved != 0;
    return type == KQ_BF16 ? launch_forward<uint16_t>(x, y, weight_q, weight_k, g, r, inter, stream)
                           : launch_forward<float>(x, y, weight_q, weight_k, g, r, inter, stream);
}

kq_status kq_headnorm_rope_backward_workspace_bytes(int64_t m, int64_t d, int64_t *bytes) {
    if (!bytes) return KQ_ERR_NULL;
    *bytes = 0;
    if (m < 0 || d < 0) return KQ_ERR_SHAPE;
    if (!sizes_fit({m, d}) || d > kMostChannels) return KQ_ERR_UNSUPPORTED;
    const int64_t parts = kqhost::row_parts(m);
    if (parts > 1) *bytes = parts * 2 * d * 4;
    return KQ_OK;
}

kq_status kq_headnorm_rope_backward(const void *dY, int64_t lddy, int64_t hsdy, const void *X, int64_t ldx, int64_t hsx,
                                    int type, int64_t m, int64_t heads, int64_t d, int norm, const float *weight_q,
                                    const float *weight_k, int64_t q_heads, float eps, const kq_rope *rope, void *dX,
                                    int64_t lddx, int64_t hsdx, float *dweight_q, float *dweight_k, void *workspace,
                                    int64_t workspace_bytes, kq_stream_t stream) {
    if (m < 0 || heads < 0 || d < 0 || q_heads < 0 || q_heads > heads || lddy < 0 || hsdy < 0 || ldx < 0 || hsx < 0 ||
        lddx < 0 || hsdx < 0 || !good_eps(eps))
        return KQ_ERR_SHAPE;
    if (!norm && (dweight_q || dweight_k)) return KQ_ERR_SHAPE;
    if (!norm) ldx = hsx = 0;
    if (!good_type(type) || !sizes_fit({m, heads, d, lddy, hsdy, ldx, hsx, lddx, hsdx}) || d > kMostChannels ||
        heads > kMostHeads)
        return KQ_ERR_UNSUPPORTED;
    if (!apart(m, heads, d, lddx, hsdx)) return KQ_ERR_SHAPE;
    Rope r;
    kq_status s = read_rope(rope, m, d, r);
    if (s != KQ_OK) return s;
    if (d == 0) return KQ_OK;
    if (!aligned(dweight_q, 4) || !aligned(dweight_k, 4)) return KQ_ERR_ALIGN;
    const bool params = dweight_q || dweight_k;
    if (m == 0 || heads == 0) return params ? kqhost::reduce_parts(nullptr, nullptr, 0, d, dweight_q, dweight_k, stream) : KQ_OK;
    if (!dY || !dX || (norm && !X)) return KQ_ERR_NULL;
    const uintptr_t es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(dY, es) || !aligned(dX, es) || (norm && !aligned(X, es)) || !aligned(weight_q, 4) || !aligned(weight_k, 4))
        return KQ_ERR_ALIGN;
    const int64_t parts = kqhost::row_parts(m);
    float *p0 = dweight_q, *p1 = dweight_k;
    if (params && parts > 1) {
        if (!workspace) return KQ_ERR_NULL;
        if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
        if (workspace_bytes < parts * 2 * d * 4) return KQ_ERR_SHAPE;
        p0 = static_cast<float *>(workspace);
        p1 = p0 + parts * d;
    }
    const Geom g{m, (int)heads, (int)q_heads, 0, 0, norm != 0, eps};
    const Tensor dy(dY, lddy, hsdy, m, heads), x(X, ldx, hsx, m, heads), dx(dX, lddx, hsdx, m, heads);
    const bool inter = r.half > 0 && rope->interleaved != 0;
    s = type == KQ_BF16
            ? launch_backward<uint16_t>(dy, x, dx, weight_q, weight_k, g, r, inter, (int)parts, p0, p1, stream)
            : launch_backward<float>(dy, x, dx, weight_q, weight_k, g, r, inter, (int)parts, p0, p1, stream);
    if (s != KQ_OK) return s;
    if (params && parts > 1) return kqhost::reduce_parts(p0, p1, parts, d, dweight_q, dweight_k, stream);
    return KQ_OK;
}

kq_status kq_cache_write_mxfp4(const void *K, int64_t ldk, int64_t hsk, int64_t k_heads, const void *V, int64_t ldv,
                               int64_t hsv, int64_t v_heads, int type, int64_t m, int64_t d, int norm,
                               const float *weight, float eps, const kq_rope *rope, const int64_t *slots,
                               int64_t cache_slots, uint8_t *codes_k, uint8_t *scales_k, uint8_t *codes_v,
                               uint8_t *scales_v, kq_stream_t stream) {
    if (m < 0 || d < 0 || d % 32 != 0 || k_heads < 0 || v_heads < 0 || cache_slots < 0 || !good_eps(eps) ||
        (k_heads && (ldk < 0 || hsk < 0)) || (v_heads && (ldv < 0 || hsv < 0)))
        return KQ_ERR_SHAPE;
    if (!k_heads) ldk = hsk = 0;
    if (!v_heads) ldv = hsv = 0;
    if (!good_type(type) || !sizes_fit({m, d, k_heads, v_heads, cache_slots, ldk, hsk, ldv, hsv}) || d > kMostChannels ||
        k_heads + v_heads > kMostHeads)
        return KQ_ERR_UNSUPPORTED;
    Rope r;
    const kq_status s = read_rope(k_heads ? rope : nullptr, m, d, r);
    if (s != KQ_OK) return s;
    if (m == 0 || d == 0 || k_heads + v_heads == 0 || cache_slots == 0) return KQ_OK;
    if (!slots || (k_heads && (!K || !codes_k || !scales_k)) || (v_heads && (!V || !codes_v || !scales_v)))
        return KQ_ERR_NULL;
    const uintptr_t es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(slots, 8) || !aligned(weight, 4) || (k_heads && (!aligned(K, es) || !aligned(codes_k, 4))) ||
        (v_heads && (!aligned(V, es) || !aligned(codes_v, 4))))
        return KQ_ERR_ALIGN;
    const Geom g{m, (int)(k_heads + v_heads), (int)k_heads, 0, 0, norm != 0 && k_heads, eps};
    const kq::heads::Cache cache{slots, cache_slots, (int)k_heads, (int)v_heads, {codes_k, codes_v}, {scales_k, scales_v}};
    // a missing tensor takes the other's place in the choice of the access width
    const Tensor k(k_heads ? K : V, k_heads ? ldk : ldv, k_heads ? hsk : hsv, m, k_heads ? k_heads : v_heads);
    const Tensor v(v_heads ? V : K, v_heads ? ldv : ldk, v_heads ? hsv : hsk, m, v_heads ? v_heads : k_heads);
    const bool inter = r.half > 0 && rope->interleaved != 0;
    return type == KQ_BF16 ? launch_write<uint16_t>(k, v, weight, g, r, inter, cache, stream)
                           : launch_write<float>(k, v, weight, g, r, inter, cache, stream);
}

kq_status kq_cache_read_mxfp4(const int64_t *slots, int64_t m, const uint8_t *codes, const uint8_t *scales,
                              int64_t cache_slots, int64_t heads, int64_t d, int type, void *Y, int64_t ldy, int64_t hsy,
                              kq_stream_t stream) {
    if (m < 0 || heads < 0 || d < 0 || d % 32 != 0 || cache_slots < 0 || ldy < 0 || hsy < 0) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, heads, d, cache_slots, ldy, hsy}) || d > kMostChannels || heads > kMostHeads)
        return KQ_ERR_UNSUPPORTED;
    if (!apart(m, heads, d, ldy, hsy)) return KQ_ERR_SHAPE;
    if (m == 0 || heads == 0 || d == 0) return KQ_OK;
    if (!slots || !Y || (cache_slots > 0 && (!codes || !scales))) return KQ_ERR_NULL;
    const int es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(slots, 8) || !aligned(codes, 4) || !aligned(Y, es)) return KQ_ERR_ALIGN;
    const Tensor y(Y, ldy, hsy, m, heads);
    const int vec = aligned(Y, 16) && y.ld * es % 16 == 0 && y.hs * es % 16 == 0;
    const int64_t total = m * heads * (d / 8), groups = (total + kq::heads::kThreads - 1) / kq::heads::kThreads;
    const int64_t most = (int64_t)kqhost::compute_units() * 32;
    const dim3 grid((unsigned)(groups < most ? groups : most)), block(kq::heads::kThreads);
    if (type == KQ_BF16)
        hipLaunchKernelGGL((kq::heads::cache_read_kernel<uint16_t>), grid, block, 0, (hipStream_t)stream, slots, m,
                           cache_slots, codes, scales, (int)heads, (int)d, (uint16_t *)Y, y.ld, y.hs, vec);
    else
        hipLaunchKernelGGL((kq::heads::cache_read_kernel<float>), grid, block, 0, (hipStream_t)stream, slots, m,
                           cache_slots, codes, scales, (int)heads, (int)d, (float *)Y, y.ld, y.hs, vec);
    return launched();
}

}  // extern "C"
