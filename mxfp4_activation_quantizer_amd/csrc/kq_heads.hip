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
// The angle is reduced in 64 bits: p f / (2 pi), less its nearest whole number. The
// constant, its product with f, that with p and p itself are rounded: off by 2^-51 of
// itself at most (1.2 2^-52 measured, 1.6 for p past 2^53), so by 4e-8 turns at 10^8
// turns, where 32 bits would leave nothing of it past a few million. Sine and cosine of
// the rest are taken in 32 bits, to 1.5 units in the last place (kq_turn.hpp).
//
// A head is held by LG neighbouring lanes. A lane has U units of it, each two
// pieces of V neighbouring channels: for pairs (i, i + r / 2) the two pieces are
// partners, and pairs (2 i, 2 i + 1) lie inside a piece, so a rotation never
// leaves its lane. V is 8 or 4 channels (16-byte or 8-byte accesses) where sizes
// and alignment allow, else 1.
//
// A wave takes its heads in passes of 64 / LG: heads of one token, or all of a
// few tokens where a token has fewer. Heads of one kind (queries, keys, values)
// at a time, so that what they need (weights, sums, whether they are rotated) is
// the same for the wave; a pass's place is in scalar registers and a lane's
// offset in it never changes. What a lane does not have (a piece past the head, a
// head past the last) is an offset past the buffer's record count: it loads
// zeros, which add nothing to a sum, and its stores are dropped. (With heads
// dealt to the lanes one by one, each with its own address, weight and kind,
// half of the instructions were those: 8192 x 16 x 128 bf16 into the cache 14.6
// us instead of 11.4, one token of 40 x 128 4.5 instead of 3.5.)
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
#include "kq_turn.hpp"

namespace kq {
namespace heads {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kBackThreads = 512, kBackWaves = kBackThreads / 64;
constexpr uint32_t kNone = 0x80000000u;

struct Rope {
    const int64_t *pos;  // [m][axes]
    const double *freq;  // [half], radians per position
    float amp;
    int axes, upto[4];   // pairs below upto[a] (and not below upto[a - 1]) turn with axis a
    int d, half;         // channels per head, rotated pairs
};

// x / n for the n and magic = floor(2^32 / n) + 1 of the host, x n < 2^32.
struct Divisor {
    int n;
    uint32_t magic;
    __device__ __forceinline__ int of(int x) const { return n == 1 ? x : (int)__umulhi((uint32_t)x, magic); }
};

// Heads of one kind: a pass takes all of them of `group` tokens, or, where they are more than a wave holds, one of
// the `per` parts of a token's.
struct Kind {
    int heads, first;
    Divisor group, per;
};
struct Geom {
    int64_t m;
    Kind kind[2];
    int tokens;  // per workgroup (a block of them)
    int norm;
    float eps;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t whole_rsrc(const void *p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)kNone, 0x00020000);
}

// V neighbouring elements as they are loaded; NT: non-temporal.
template <class T, int V>
struct Piece {
    static constexpr int kWords = V == 1 ? 1 : V * (int)sizeof(T) / 4;
    uint32_t q[kWords];
    template <bool NT>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
        constexpr int aux = NT ? 2 : 0;
        if constexpr (V == 1 && sizeof(T) == 2) {
            q[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, aux) << 16;
        } else if constexpr (V == 1) {
            q[0] = __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, aux);
        } else if constexpr (kWords == 2) {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(r, at, 0, aux);
            q[0] = v[0];
            q[1] = v[1];
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, at + 4 * i, 0, aux);
#pragma unroll
                for (int k = 0; k < 4; ++k) q[i + k] = v[k];
            }
        }
    }
    __device__ __forceinline__ void widen(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            if constexpr (V > 1 && sizeof(T) == 2) {
                x[2 * i] = bf16_lo(q[i]);
                x[2 * i + 1] = bf16_hi(q[i]);
            } else {
                x[i] = __uint_as_float(q[i]);
            }
        }
    }
};

// V values to neighbouring elements.
template <class T, int V, bool NT>
__device__ __forceinline__ void store_piece(__amdgpu_buffer_rsrc_t r, uint32_t at, const float (&x)[V]) {
    constexpr int aux = NT ? 2 : 0, words = V * (int)sizeof(T) / 4;
    if constexpr (V == 1 && sizeof(T) == 2) {
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)x[0]), r, at, 0, aux);
    } else if constexpr (V == 1) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(x[0]), r, at, 0, aux);
    } else {
        uint32_t q[words];
#pragma unroll
        for (int i = 0; i < words; ++i) {
            if constexpr (sizeof(T) == 2) q[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            else q[i] = __float_as_uint(x[i]);
        }
        if constexpr (words == 2) {
            typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
            __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{q[0], q[1]}, r, at, 0, aux);
        } else {
#pragma unroll
            for (int i = 0; i < words; i += 4)
                __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{q[i], q[i + 1], q[i + 2], q[i + 3]}, r, at + 4 * i, 0, aux);
        }
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

// Where unit u of a head lies: its first piece at channel a, its second at b, whether they exist, and the pairs that
// they (each by itself, for pairs inside a piece) start with; -1 for none.
struct Place {
    int a, b, pair_a, pair_b;
    bool in_a, in_b;
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
        p.pair_a = p.in_a && p.a < r ? p.a / 2 : -1;
        p.pair_b = p.in_b && p.b < r ? p.b / 2 : -1;
    } else if (u < half / V) {
        p.a = INTER ? 2 * u : V * u;
        p.b = INTER ? 2 * u + 1 : half + V * u;
        p.in_a = p.in_b = true;
        p.pair_a = p.pair_b = V * u;
    } else {
        const int n = (d - r) / V, h = (n + 1) / 2, w = u - half / V;
        p.in_a = w < h;
        p.in_b = w + h < n && p.in_a;
        p.a = r + V * w;
        p.b = r + V * (w + h);
        p.pair_a = p.pair_b = -1;
    }
    // a missing piece's weight is read where the head's first is
    if (!p.in_a) p.a = 0;
    if (!p.in_b) p.b = 0;
    return p;
}

// The table of angles in LDS: (amp cos t, amp sin t) of every pair of every token of a block, a token's row V longer than
// its pairs, so that the rows' first entries are not all in one bank.
template <int V>
__device__ __forceinline__ int table_row(const Rope &rope) { return rope.half + V; }
template <int V>
__device__ __forceinline__ void fill_table(float2 *table, const Rope &rope, int64_t t0, int tokens, int tid, int threads) {
    const float inv = 1.0f / (float)rope.half;
    for (int i = tid; i < tokens * rope.half; i += threads) {
        const int t = (int)(((float)i + 0.5f) * inv), j = i - t * rope.half;
        int axis = 0;
#pragma unroll
        for (int a = 0; a < 3; ++a) axis += a + 1 < rope.axes && j >= rope.upto[a];
        // in quarter turns
        const double x = (double)rope.pos[(t0 + t) * rope.axes + axis] * (rope.freq[j] * 0.63661977236758134);
        const double n = rint(x);
        float2 v = quarter_turn(x - n);
        const int64_t k = (int64_t)n;
        if (k & 1) v = make_float2(-v.y, v.x);
        if (k & 2) v = make_float2(-v.x, -v.y);
        v.x *= rope.amp;
        v.y *= rope.amp;
        table[t * table_row<V>(rope) + j] = v;
    }
}

// The pieces (a, b) of one unit turned by their angles, BACK: by the opposite ones; a piece that no pair is in is left as it
// is, to the sign of its zeros. `row`: the token's row of the table.
template <int V, bool INTER, bool BACK>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float2 *row, const Place &p) {
    if (INTER && V > 1) {
        const float2 *ta = row + (p.pair_a < 0 ? 0 : p.pair_a), *tb = row + (p.pair_b < 0 ? 0 : p.pair_b);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 ca = ta[e / 2], cb = tb[e / 2];
            const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
            const float s0 = fmaf(a0, ca.x, BACK ? a1 * ca.y : -(a1 * ca.y));
            const float s1 = fmaf(a1, ca.x, BACK ? -(a0 * ca.y) : a0 * ca.y);
            const float t0 = fmaf(b0, cb.x, BACK ? b1 * cb.y : -(b1 * cb.y));
            const float t1 = fmaf(b1, cb.x, BACK ? -(b0 * cb.y) : b0 * cb.y);
            a[e] = p.pair_a < 0 ? a0 : s0;
            a[e + 1] = p.pair_a < 0 ? a1 : s1;
            b[e] = p.pair_b < 0 ? b0 : t0;
            b[e + 1] = p.pair_b < 0 ? b1 : t1;
        }
    } else {
        if (p.pair_a < 0) return;
        const float2 *ta = row + p.pair_a;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 c = ta[e];
            const float x = a[e], y = b[e];
            a[e] = fmaf(x, c.x, BACK ? y * c.y : -(y * c.y));
            b[e] = fmaf(y, c.x, BACK ? -(x * c.y) : x * c.y);
        }
    }
}

// A pass of one kind, the same for the wave: its first token (of the block) and head, and the lanes' limit.
struct Pass {
    int token, head, limit;
};
__device__ __forceinline__ int passes_of(const Kind &k, int tokens) {
    return k.heads ? k.group.of(tokens + k.group.n - 1) * k.per.n : 0;
}
// Past the last pass: the last one, with no heads. (Loads without a branch: where paths with more and with fewer of
// them meet, the compiler waits for as many as the shorter one leaves.)
template <int LG>
__device__ __forceinline__ Pass pass_of(const Kind &k, int p, int passes, int tokens) {
    const int q = p < passes ? p : passes - 1, group = k.per.of(q), part = q - group * k.per.n;
    Pass r;
    r.token = group * k.group.n;
    r.head = part * (64 / LG);
    r.limit = p >= passes ? 0 : k.heads < 64 / LG ? tokens - r.token : k.heads - r.head;
    return r;
}
// Which pass of the second kind is a wave's first where the two kinds' passes are dealt out in one turn: from p on,
// every step-th, the first kind's `passes` first.
__device__ __forceinline__ int next_turn(int p, int passes, int step) {
    const int n = passes - p;
    return n <= 0 ? -n : (step - n % step) % step;
}
// A lane's part in the passes of a kind: the token of the pass's group that its head belongs to, its place among the
// pass's heads of a token, and the number that has to be below a pass's limit for the head to exist (one of the two).
template <int LG>
struct Lane {
    int token, head, bound;
    __device__ __forceinline__ void set(const Kind &k, int slot) {
        const bool grouped = k.heads < 64 / LG && k.heads > 0;
        token = grouped ? (int)(((float)slot + 0.5f) * (1.0f / (float)k.heads)) : 0;
        bound = !grouped ? slot : token < k.group.n ? token : 1 << 30;
        head = slot - token * k.heads;
    }
    // byte offset of channel c from a pass's place in a tensor of these strides
    __device__ __forceinline__ uint32_t offset(bool in, int c, int64_t ld, int64_t hs, int es) const {
        return in ? (uint32_t)((token * ld + head * hs + c) * es) : kNone;
    }
    // what an offset is joined with: past the record count where the head does not exist
    __device__ __forceinline__ uint32_t mask(const Pass &s) const { return bound < s.limit ? 0u : kNone; }
    // the lane's token of the block, the pass's first where its head does not exist
    __device__ __forceinline__ int row_of(const Pass &s) const { return s.token + (bound < s.limit ? token : 0); }
};

// The weights of a lane's pieces (1 without any); asked for and taken apart, since the table is made in between.
template <int V, int U>
struct Weights {
    Piece<float, V> q[U][2];
    float v[U][2][V];
    __device__ __forceinline__ void ask(const float *w, const Place (&at)[U], int d) {
        const auto r = row_rsrc(w, w ? 4 * d : 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            q[u][0].template load<false>(r, 4 * (uint32_t)at[u].a);
            q[u][1].template load<false>(r, 4 * (uint32_t)at[u].b);
        }
    }
    __device__ __forceinline__ void take(const float *w) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                q[u][b].widen(v[u][b]);
#pragma unroll
                for (int e = 0; e < V; ++e) v[u][b][e] = w ? v[u][b][e] : 1.0f;
            }
    }
};

// X and Y may be the same memory: a lane has read all of its pieces before it writes any of them.
// A workgroup takes the heads of a few tokens, a wave G passes in turn, each one's next loads asked for when it is
// done. The table of angles is made once per token and read back by every head.
//
// Bound by HBM once it is large: 8192 x 40 x 128 bf16 31.5 us (168 MB, 5.3 TB/s; a 1 GiB copy 4.7 to 5.0), fp32 59.7, 37.4
// where half of the channels are turned (bf16); one token of 40 x 128 3.4, a launch and the latency of its positions,
// frequencies and heads. A head that does not fill its lanes leaves some idle: 4096 x 32 x 72 fp32 (9 of 16 lanes) 15.3 us,
// 4.9 TB/s. One by one (d = 65) 4096 x 32 takes 31.2 us in bf16 and 31.9 in fp32, 1.1 and 2.1 TB/s: a load and a store of 2 or 4
// bytes for each channel of each lane.
template <class T, int V, int LG, int U, bool INTER, bool NT>
__global__ __launch_bounds__(kThreads) void forward_kernel(const T *X, int64_t ldx, int64_t hsx,
                                                           const float *__restrict__ w0, const float *__restrict__ w1,
                                                           Geom g, Rope rope, T *Y, int64_t ldy, int64_t hsy) {
    extern __shared__ float2 table[];
    constexpr int G = U * V > 8 ? 1 : 2, es = (int)sizeof(T);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sub = lane % LG, slot = lane / LG;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens);
    const int passes0 = passes_of(g.kind[0], tokens), passes1 = passes_of(g.kind[1], tokens);
    const int step = kWaves * (int)gridDim.y, p0 = (int)blockIdx.y * kWaves + wave;
    if ((int)blockIdx.y * kWaves >= passes0 + passes1) return;  // the whole workgroup
    const float inv_d = 1.0f / (float)rope.d;
    Place at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = place_of<V, INTER>(sub + LG * u, rope.d, rope.half);
    struct Row {
        Piece<T, V> a[U], b[U];
    };
    bool made = false;  // the table
    // the passes of one kind, from the wave's first on
    auto run = [&](const Kind &kind, const float *w, int passes, int p) {
        if (passes == 0) return;
        Lane<LG> in;
        in.set(kind, slot);
        uint32_t xo[U][2], yo[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xo[u][0] = in.offset(at[u].in_a, at[u].a, ldx, hsx, es);
            xo[u][1] = in.offset(at[u].in_b, at[u].b, ldx, hsx, es);
            yo[u][0] = in.offset(at[u].in_a, at[u].a, ldy, hsy, es);
            yo[u][1] = in.offset(at[u].in_b, at[u].b, ldy, hsy, es);
        }
        Row rows[G];
        auto fetch = [&](Row &row, int q) {
            const Pass s = pass_of<LG>(kind, q, passes, tokens);
            const auto from = whole_rsrc(X + (t0 + s.token) * ldx + (kind.first + s.head) * hsx);
            const uint32_t none = in.mask(s);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                row.a[u].template load<NT>(from, xo[u][0] | none);
                row.b[u].template load<NT>(from, xo[u][1] | none);
            }
        };
#pragma unroll
        for (int i = 0; i < G; ++i) fetch(rows[i], p + step * i);
        Weights<V, U> wv;
        wv.ask(w, at, rope.d);
        if (!made) {
            fill_table<V>(table, rope, t0, tokens, tid, kThreads);
            __syncthreads();
            made = true;
        }
        wv.take(w);
        for (; p < passes; p += step * G) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int q = p + step * i;
                if (i > 0 && q >= passes) break;
                const Pass s = pass_of<LG>(kind, q, passes, tokens);
                float a[U][V], b[U][V], sum = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    rows[i].a[u].widen(a[u]);
                    rows[i].b[u].widen(b[u]);
                }
                fetch(rows[i], q + step * G);
                if (g.norm) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float sa = 0.f, sb = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            sa = fmaf(a[u][e], a[u][e], sa);
                            sb = fmaf(b[u][e], b[u][e], sb);
                        }
                        sum += sa + sb;
                    }
                    const float rs = __builtin_amdgcn_rsqf(fmaf(group_sum<LG>(sum), inv_d, g.eps));
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            a[u][e] = a[u][e] * rs * wv.v[u][0][e];
                            b[u][e] = b[u][e] * rs * wv.v[u][1][e];
                        }
                }
                const auto to = whole_rsrc(Y + (t0 + s.token) * ldy + (kind.first + s.head) * hsy);
                const float2 *turns = table + in.row_of(s) * table_row<V>(rope);
                const uint32_t none = in.mask(s);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    turn<V, INTER, false>(a[u], b[u], turns, at[u]);
                    store_piece<T, V, NT>(to, yo[u][0] | none, a[u]);
                    store_piece<T, V, NT>(to, yo[u][1] | none, b[u]);
                }
            }
        }
    };
    // the second kind's passes follow the first's in the waves' turns
    run(g.kind[0], w0, passes0, p0);
    run(g.kind[1], w1, passes1, next_turn(p0, passes0, step));
}

// Gradients. With e the gradient turned back, h = x s and g = e w:
//   dx = s (g - h sum(g h) / d), dw = sum of e h over the rows of that weight.
// Workgroup p of `parts` takes the blocks of tokens p, p + parts, ...; its lanes keep their channels of both dw in
// registers, and row p of the partial sums gets them at the end, the waves joined in their order. dX may be dY or X.
//
// Bound by HBM: 8192 x 40 x 128 bf16 53 us and 4 for the partial sums' (252 MB, 4.7 TB/s), fp32 97 and 4, 4096 x 32 x 72 fp32
// 25 and 4; one by one (4096 x 32 x 65) 44 in bf16 and 46 in fp32.
// Parts of 512 threads (768 are level, 1024 take 120 us) with one pass of each kind in flight (two and three are
// level). Both dweights cost 1.9 us at one token (the joins) and 4 where a second launch adds the parts.
template <class T, int V, int LG, int U, bool INTER, bool NT>
__global__ __launch_bounds__(kBackThreads) void backward_kernel(const T *dY, int64_t lddy, int64_t hsdy, const T *X,
                                                                int64_t ldx, int64_t hsx,
                                                                const float *__restrict__ w0,
                                                                const float *__restrict__ w1, Geom g, Rope rope, T *dX,
                                                                int64_t lddx, int64_t hsdx, int parts,
                                                                float *__restrict__ p0, float *__restrict__ p1) {
    extern __shared__ float2 table[];
    constexpr int es = (int)sizeof(T);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sub = lane % LG, slot = lane / LG;
    const float inv_d = 1.0f / (float)rope.d;
    Place at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = place_of<V, INTER>(sub + LG * u, rope.d, rope.half);
    struct Row {
        Piece<T, V> a[U], b[U], da[U], db[U];
    };
    // what the lane keeps for the heads of one kind
    struct Side {
        Lane<LG> in;
        uint32_t yo[U][2], xo[U][2], zo[U][2];
        Weights<V, U> w;
        float acc[U][2][V];
    } sides[2];
    float (&acc0)[U][2][V] = sides[0].acc, (&acc1)[U][2][V] = sides[1].acc;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        Side &s = sides[k];
        s.in.set(g.kind[k], slot);
        s.w.ask(k ? w1 : w0, at, rope.d);
        s.w.take(k ? w1 : w0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const bool is = b ? at[u].in_b : at[u].in_a;
                const int c = b ? at[u].b : at[u].a;
                s.yo[u][b] = s.in.offset(is, c, lddy, hsdy, es);
                s.xo[u][b] = s.in.offset(is, c, ldx, hsx, es);
                s.zo[u][b] = s.in.offset(is, c, lddx, hsdx, es);
#pragma unroll
                for (int e = 0; e < V; ++e) s.acc[u][b][e] = 0.f;
            }
    }
    const int64_t blocks = (g.m + g.tokens - 1) / g.tokens;
    int par = 0;
    for (int64_t block = blockIdx.x; block < blocks; block += parts, par ^= 1) {
        const int64_t t0 = block * g.tokens;
        const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens);
        const int passes0 = passes_of(g.kind[0], tokens), passes1 = passes_of(g.kind[1], tokens);
        // two tables in turn: one is written again only after the next block's barrier
        float2 *tab = table + par * (g.tokens * table_row<V>(rope));
        auto fetch = [&](Row &row, const Kind &kind, const Side &side, int p, int passes) {
            const Pass s = pass_of<LG>(kind, p, passes, tokens);
            const auto fy = whole_rsrc(dY + (t0 + s.token) * lddy + (kind.first + s.head) * hsdy);
            const auto fx = whole_rsrc(X + (t0 + s.token) * ldx + (kind.first + s.head) * hsx);
            const uint32_t none = side.in.mask(s), none_x = g.norm ? none : kNone;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                row.da[u].template load<NT>(fy, side.yo[u][0] | none);
                row.db[u].template load<NT>(fy, side.yo[u][1] | none);
                row.a[u].template load<NT>(fx, side.xo[u][0] | none_x);
                row.b[u].template load<NT>(fx, side.xo[u][1] | none_x);
            }
        };
        auto run = [&](Row &row, const Kind &kind, Side &side, int p, int passes) {
            for (; p < passes; p += kBackWaves) {
                const Pass s = pass_of<LG>(kind, p, passes, tokens);
                const float2 *turns = tab + side.in.row_of(s) * table_row<V>(rope);
                float ea[U][V], eb[U][V], xa[U][V], xb[U][V];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    row.da[u].widen(ea[u]);
                    row.db[u].widen(eb[u]);
                    row.a[u].widen(xa[u]);
                    row.b[u].widen(xb[u]);
                }
                fetch(row, kind, side, p + kBackWaves, passes);
#pragma unroll
                for (int u = 0; u < U; ++u) turn<V, INTER, true>(ea[u], eb[u], turns, at[u]);
                if (g.norm) {
                    float sum = 0.f, dot = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float sa = 0.f, sb = 0.f, qa = 0.f, qb = 0.f;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            sa = fmaf(xa[u][e], xa[u][e], sa);
                            sb = fmaf(xb[u][e], xb[u][e], sb);
                            qa = fmaf(xa[u][e] * side.w.v[u][0][e], ea[u][e], qa);
                            qb = fmaf(xb[u][e] * side.w.v[u][1][e], eb[u][e], qb);
                        }
                        sum += sa + sb;
                        dot += qa + qb;
                    }
                    sum = group_sum<LG>(sum);
                    dot = group_sum<LG>(dot);
                    // a head that is not there is all zeros: with eps = 0 the root's reciprocal would be infinite
                    const float rs = side.in.bound < s.limit ? __builtin_amdgcn_rsqf(fmaf(sum, inv_d, g.eps)) : 0.f;
                    const float c = dot * rs * inv_d;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float ha = xa[u][e] * rs, hb = xb[u][e] * rs;
                            side.acc[u][0][e] = fmaf(ea[u][e], ha, side.acc[u][0][e]);
                            side.acc[u][1][e] = fmaf(eb[u][e], hb, side.acc[u][1][e]);
                            ea[u][e] = rs * fmaf(-ha, c, ea[u][e] * side.w.v[u][0][e]);
                            eb[u][e] = rs * fmaf(-hb, c, eb[u][e] * side.w.v[u][1][e]);
                        }
                }
                const auto to = whole_rsrc(dX + (t0 + s.token) * lddx + (kind.first + s.head) * hsdx);
                const uint32_t none = side.in.mask(s);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    store_piece<T, V, NT>(to, side.zo[u][0] | none, ea[u]);
                    store_piece<T, V, NT>(to, side.zo[u][1] | none, eb[u]);
                }
            }
        };
        // the second kind's first pass is in flight beside the first kind's
        Row row, other;
        const int p1 = next_turn(wave, passes0, kBackWaves);
        if (passes0) fetch(row, g.kind[0], sides[0], wave, passes0);
        if (passes1) fetch(other, g.kind[1], sides[1], p1, passes1);
        fill_table<V>(tab, rope, t0, tokens, tid, kBackThreads);
        __syncthreads();
        if (passes0) run(row, g.kind[0], sides[0], wave, passes0);
        if (passes1) run(other, g.kind[1], sides[1], p1, passes1);
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
                    const float v = slots_sum<LG>(k ? acc1[u][b][e] : acc0[u][b][e]);
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

// Keys and values of a block of tokens into the cache: keys normed and turned as above, values as they are. QUADS:
// every four lanes' first pieces, and their second ones, are a block of 32 channels each (V = 8, and the two pieces of
// a unit a multiple of 32 channels apart), so they are quantized where they are. Otherwise a wave's heads meet in LDS,
// where four lanes take each block.
//
// 8192 x (8 + 8) x 128 bf16 takes 11.6 us (42 MB, 3.7 TB/s, into slots in any order) and 9.0 of them with no slot to write to:
// what bounds it is reading, 34 MB at 3.8 TB/s with one pass of loads a wave in flight, and not the stores. fp32 15.6; staged,
// d = 96 16.8 and d = 160 23.7; 64 tokens 4.2 by themselves, 3.3 one call after another. The values' first loads beside the keys'
// are slower (11.7 to 11.0).
struct Cache {
    const int64_t *slots;  // [m]
    int64_t n;             // slots of the cache
    uint8_t *codes[2], *scales[2];  // of keys and of values
};
template <class T, int V, int LG, int U, bool INTER, bool QUADS>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(const T *__restrict__ K, int64_t ldk, int64_t hsk,
                                                               const T *__restrict__ Vx, int64_t ldv, int64_t hsv,
                                                               const float *__restrict__ w, Geom g, Rope rope,
                                                               Cache cache, int stage_at) {
    extern __shared__ float2 table[];
    static_assert(!QUADS || (V == 8 && LG >= 4 && U == 1), "blocks of 32 channels in four lanes");
    constexpr int HP = 64 / LG, es = (int)sizeof(T);
    __shared__ int64_t row_of[kWaves][HP];  // row of the cache, -1 for none
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int sub = lane % LG, slot = lane / LG, d = rope.d;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens);
    const int passes0 = passes_of(g.kind[0], tokens), passes1 = passes_of(g.kind[1], tokens);
    const int step = kWaves * (int)gridDim.y, p0 = (int)blockIdx.y * kWaves + wave;
    if ((int)blockIdx.y * kWaves >= passes0 + passes1) return;  // the whole workgroup
    const float inv_d = 1.0f / (float)d;
    float *stage = reinterpret_cast<float *>(table) + stage_at + wave * HP * d;
    Place at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = place_of<V, INTER>(sub + LG * u, d, rope.half);
    struct Row {
        Piece<T, V> a[U], b[U];
        int64_t to;
    };
    // the passes of keys (k = 0) or values, from the wave's first on
    auto run = [&](auto which, const T *X, int64_t ld, int64_t hs, int passes, int p) {
        constexpr int k = decltype(which)::value;
        const Kind &kind = g.kind[k];
        if (passes == 0) return;
        Lane<LG> in;
        in.set(kind, slot);
        uint32_t xo[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            xo[u][0] = in.offset(at[u].in_a, at[u].a, ld, hs, es);
            xo[u][1] = in.offset(at[u].in_b, at[u].b, ld, hs, es);
        }
        Row next;
        auto fetch = [&](Row &row, int q) {
            const Pass s = pass_of<LG>(kind, q, passes, tokens);
            const auto from = whole_rsrc(X + (t0 + s.token) * ld + s.head * hs);
            const uint32_t none = in.mask(s);
            row.to = cache.slots[t0 + in.row_of(s)];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                row.a[u].template load<false>(from, xo[u][0] | none);
                row.b[u].template load<false>(from, xo[u][1] | none);
            }
        };
        fetch(next, p);
        Weights<V, U> wv;
        if (k == 0) {
            wv.ask(w, at, d);
            fill_table<V>(table, rope, t0, tokens, tid, kThreads);
            __syncthreads();
            wv.take(w);
        }
        for (; p < passes; p += step) {
            const Pass s = pass_of<LG>(kind, p, passes, tokens);
            float a[U][V], b[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                next.a[u].widen(a[u]);
                next.b[u].widen(b[u]);
            }
            const int64_t slot_of = next.to;
            fetch(next, p + step);
            if (k == 0 && g.norm) {
                float sum = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float sa = 0.f, sb = 0.f;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        sa = fmaf(a[u][e], a[u][e], sa);
                        sb = fmaf(b[u][e], b[u][e], sb);
                    }
                    sum += sa + sb;
                }
                const float rs = __builtin_amdgcn_rsqf(fmaf(group_sum<LG>(sum), inv_d, g.eps));
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        a[u][e] = a[u][e] * rs * wv.v[u][0][e];
                        b[u][e] = b[u][e] * rs * wv.v[u][1][e];
                    }
            }
            if (k == 0) {
                const float2 *turns = table + in.row_of(s) * table_row<V>(rope);
#pragma unroll
                for (int u = 0; u < U; ++u) turn<V, INTER, false>(a[u], b[u], turns, at[u]);
            }
            const bool is = in.bound < s.limit && slot_of >= 0 && slot_of < cache.n;
            const int64_t to = is ? slot_of * kind.heads + (s.head + in.head) : -1;
            if constexpr (QUADS) {
                uint32_t sa, sb;
                const uint32_t ca = quantize_quad_f32(a[0], sa), cb = quantize_quad_f32(b[0], sb);
                uint8_t *codes = cache.codes[k] + to * (d / 2), *scales = cache.scales[k] + to * (d / 32);
                if (is && at[0].in_a) {
                    *reinterpret_cast<uint32_t *>(codes + at[0].a / 2) = ca;
                    if ((lane & 3) == 0) scales[at[0].a / 32] = (uint8_t)sa;
                }
                if (is && at[0].in_b) {
                    *reinterpret_cast<uint32_t *>(codes + at[0].b / 2) = cb;
                    if ((lane & 3) == 0) scales[at[0].b / 32] = (uint8_t)sb;
                }
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        if (at[u].in_a) stage[slot * d + at[u].a + e] = a[u][e];
                        if (at[u].in_b) stage[slot * d + at[u].b + e] = b[u][e];
                    }
                if (sub == 0) row_of[wave][slot] = to;
                // a wave's LDS accesses stay in order; nothing may move across this point
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const int pieces = d / 8;
                for (int j = lane; j < HP * pieces; j += 64) {
                    const int row = j / pieces, c = j - row * pieces;
                    const int64_t at_row = row_of[wave][row];
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const floatx4_t v = *reinterpret_cast<const floatx4_t *>(stage + row * d + 8 * c + e);
#pragma unroll
                        for (int n = 0; n < 4; ++n) x[e + n] = v[n];
                    }
                    uint32_t sbyte;
                    const uint32_t code = quantize_quad_f32(x, sbyte);
                    if (at_row < 0) continue;
                    *reinterpret_cast<uint32_t *>(cache.codes[k] + at_row * (d / 2) + 4 * c) = code;
                    if ((lane & 3) == 0) cache.scales[k][at_row * (d / 32) + c / 4] = (uint8_t)sbyte;
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        }
    };
    // the values' passes follow the keys' in the waves' turns
    run(std::integral_constant<int, 0>(), K, ldk, hsk, passes0, p0);
    run(std::integral_constant<int, 1>(), Vx, ldv, hsv, passes1, next_turn(p0, passes0, step));
}

// Rows of the cache decoded: a lane takes 8 channels (a dword of codes) of R places of the workgroup's tokens (or
// of its part of one token), all of whose loads are in flight together. A row whose slot lies outside the cache is
// zeros.
// Eight places hide the two dependent loads (slot, then codes and scale): 131072 x 8 x 128 bf16 50 us (340 MB, 6.8 TB/s
// with the cache partly in the Infinity Cache), 97 with one; in fp32 246 (608 MB, 2.5 TB/s): a lane's two stores of 16 bytes take
// the lines that its neighbours write too. One place for calls that would not fill the card: 509 tokens 2.6.
struct Read {
    int64_t m, n;             // tokens, slots
    int tokens, pieces;       // tokens per workgroup; 8-channel pieces of a token
    int per_head;             // pieces of a head
    uint32_t by_token, by_head;  // floor(2^32 / n) + 1 for n = pieces and per_head: the high half of its product with
                                 // i is i / n for i n < 2^32
};
template <class T, bool NT>
__device__ __forceinline__ void store_values(T *p, const float (&x)[8]) {
    constexpr int words = 2 * (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < words; i += 4) {
        u32x4_t q;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 2) q[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
            else q[k] = __float_as_uint(x[i + k]);
        }
        u32x4_t *to = reinterpret_cast<u32x4_t *>(p) + i / 4;
        if (NT) __builtin_nontemporal_store(q, to);
        else *to = q;
    }
}
template <class T, int R, bool VEC, bool NT>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(const int64_t *__restrict__ slots,
                                                              const uint8_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales, Read g,
                                                              T *__restrict__ Y, int64_t ldy, int64_t hsy) {
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens;
    const int tokens = (int)(g.m - t0 < g.tokens ? g.m - t0 : g.tokens);
    const int first = (int)blockIdx.y * (R * kThreads) + (int)threadIdx.x, count = tokens * g.pieces;
    int64_t from[R];
    int token[R], at[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int j = first + i * kThreads, jj = j < count ? j : 0;
        token[i] = g.tokens > 1 ? (int)__umulhi((uint32_t)jj, g.by_token) : 0;
        at[i] = jj - token[i] * g.pieces;
        from[i] = slots[t0 + token[i]];
    }
    uint32_t code[R], scale[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool in = from[i] >= 0 && from[i] < g.n && first + i * kThreads < count;
        const int64_t piece = in ? from[i] * g.pieces + at[i] : 0;
        code[i] = in ? reinterpret_cast<const uint32_t *>(codes)[piece] : 0;
        scale[i] = in ? scales[piece >> 2] : 127;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        if (first + i * kThreads >= count) break;
        const int h = (int)__umulhi((uint32_t)at[i], g.by_head), c = at[i] - h * g.per_head;
        const bf16x8_t v = decode_fp4x8_bf16_cvt(code[i], scale[i]);
        T *y = Y + (t0 + token[i]) * ldy + h * hsy + 8 * c;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
        if (VEC) {
            store_values<T, NT>(y, x);
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

// Channels per piece, at most `most`: 8 or 4 where the halves of the rotated part (the whole of it with neighbouring
// pairs), the head and every address are multiples of it.
int piece_width(int most, int es, const Rope &rope, bool inter, std::initializer_list<Tensor> tensors) {
    for (int v = most; v >= 4; v /= 2) {
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
template <int MOST, class F>
void choose_form(int v, int units, F f) {
    if constexpr (MOST == 8) {
        if (v == 8) {
            if (units <= 4) f(Form<8, 4, 1>());
            else if (units <= 8) f(Form<8, 8, 1>());
            else if (units <= 16) f(Form<8, 16, 1>());
            else if (units <= 32) f(Form<8, 32, 1>());
            else f(Form<8, 64, 1>());
            return;
        }
    }
    if (v == 4) {
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

constexpr int kTable = 2048, kBackTable = 4096;  // entries of a block of tokens' angles, 8 bytes of LDS each

// Heads of one kind in passes of hp.
kq::heads::Kind kind_of(int64_t heads, int64_t first, int hp) {
    auto divisor = [](int64_t n) { return kq::heads::Divisor{(int)n, (uint32_t)(((uint64_t)1 << 32) / (uint64_t)n + 1)}; };
    return kq::heads::Kind{(int)heads, (int)first, divisor(heads > 0 && heads < hp ? hp / heads : 1),
                           divisor(heads > hp ? (heads + hp - 1) / hp : 1)};
}
int64_t passes_of(const kq::heads::Kind &k, int64_t tokens) {
    return k.heads ? (tokens + k.group.n - 1) / k.group.n * k.per.n : 0;
}

// Whether a lane's offset inside a pass fits 31 bits: heads of one token, or of a group of tokens.
bool offsets_fit(const kq::heads::Kind &k, int hp, int d, int es, std::initializer_list<Tensor> tensors) {
    const int64_t heads = k.heads < hp ? k.heads : hp;
    for (const Tensor &t : tensors)
        if (((k.group.n - 1) * t.ld + (heads > 0 ? heads - 1 : 0) * t.hs + d) * es >= (int64_t)1 << 31) return false;
    return true;
}

// f(V, LG, U) for these tensors, a first kind of n0 heads and a second of n1: the fastest form of pieces of at most MOST
// channels whose offsets fit. A whole wave per head has none but its own channels'.
template <int MOST, class F>
kq_status choose(int es, const Rope &rope, bool inter, int64_t n0, int64_t n1, std::initializer_list<Tensor> tensors, F f) {
    const int v = piece_width(MOST, es, rope, inter, tensors), units = units_of(rope, inter, v);
    kq_status status = KQ_OK;
    auto go = [&](auto form) {
        constexpr int hp = 64 / decltype(form)::kLG;
        status = f(form, kind_of(n0, 0, hp), kind_of(n1, n0, hp));
    };
    bool fits = true;
    choose_form<MOST>(v, units, [&](auto form) {
        constexpr int hp = 64 / decltype(form)::kLG;
        fits = offsets_fit(kind_of(n0, 0, hp), hp, rope.d, es, tensors) && offsets_fit(kind_of(n1, n0, hp), hp, rope.d, es, tensors);
    });
    choose_form<MOST>(v, fits || units > 64 ? units : 64, go);
    return status;
}

// Tokens per workgroup and, for few of them, the workgroups that share a block's passes: four passes a
// wave where that leaves four workgroups per compute unit.
struct Plan {
    int tokens;
    int64_t blocks, splits;
};
Plan plan_of(int64_t m, const kq::heads::Kind &a, const kq::heads::Kind &b, int half, int hp) {
    const int64_t waves = kq::heads::kWaves, cus = kqhost::compute_units(), heads = a.heads + b.heads;
    int64_t t = (4 * waves * hp + heads - 1) / heads;
    if (t * (half + 8) > kTable) t = kTable / (half + 8);
    if (t > m / (4 * cus)) t = m / (4 * cus);
    // whole groups of tokens
    const int64_t group = a.group.n > b.group.n ? a.group.n : b.group.n;
    if (t > group) t -= t % group;
    if (t < 1) t = 1;
    Plan p;
    p.tokens = (int)t;
    p.blocks = (m + t - 1) / t;
    const int64_t passes = passes_of(a, t) + passes_of(b, t);
    const int64_t want = (2 * cus + p.blocks - 1) / p.blocks, most = (passes + waves - 1) / waves;
    p.splits = most < want ? most : want;
    if (p.splits > 65535) p.splits = 65535;
    return p;
}

// Pieces of 16 bytes: two loads side by side for one of 32 take each line twice (fp32 8192 x 40 x 128 71.0 us with 8
// channels and 64.2 with 4, its gradients 112 and 107; 4096 x 32 x 72 19.7 and 18.4, 32.5 and 27.6), and past the caches
// their non-temporal form (59.6, 101).
template <class T>
constexpr int kMost = 16 / (int)sizeof(T);

template <class T>
kq_status launch_forward(const Tensor &x, const Tensor &y, const float *w0, const float *w1, int64_t heads, int64_t q_heads,
                         Geom g, const Rope &rope, bool inter, kq_stream_t stream) {
    return choose<kMost<T>>(sizeof(T), rope, inter, q_heads, heads - q_heads, {x, y}, [&](auto form, auto a, auto b) {
        constexpr int V = decltype(form)::kV, LG = decltype(form)::kLG, U = decltype(form)::kU;
        const Plan p = plan_of(g.m, a, b, rope.half, 64 / LG);
        if (p.blocks >= (int64_t)1 << 24) return KQ_ERR_UNSUPPORTED;
        g.kind[0] = a;
        g.kind[1] = b;
        g.tokens = p.tokens;
        const size_t lds = (size_t)p.tokens * (rope.half + V) * sizeof(float2);
        auto go = [&](auto I, auto NT) {
            hipLaunchKernelGGL((kq::heads::forward_kernel<T, V, LG, U, I(), V * sizeof(T) == 16 && NT()>),
                               dim3((unsigned)p.blocks, (unsigned)p.splits), dim3(kq::heads::kThreads), lds,
                               (hipStream_t)stream, (const T *)x.p, x.ld, x.hs, w0, w1, g, rope,
                               (T *)const_cast<void *>(y.p), y.ld, y.hs);
        };
        const bool nt = kq::streamed_once(2 * g.m * heads * rope.d * (int64_t)sizeof(T));
        if (inter && nt) go(std::true_type(), std::true_type());
        else if (inter) go(std::true_type(), std::false_type());
        else if (nt) go(std::false_type(), std::true_type());
        else go(std::false_type(), std::false_type());
        return launched();
    });
}

template <class T>
kq_status launch_backward(const Tensor &dy, const Tensor &x, const Tensor &dx, const float *w0, const float *w1,
                          int64_t heads, int64_t q_heads, Geom g, const Rope &rope, bool inter, int parts, float *p0,
                          float *p1, kq_stream_t stream) {
    const Tensor &x_or = g.norm ? x : dy;
    return choose<kMost<T>>(sizeof(T), rope, inter, q_heads, heads - q_heads, {dy, x_or, dx}, [&](auto form, auto a, auto b) {
        constexpr int V = decltype(form)::kV, LG = decltype(form)::kLG, U = decltype(form)::kU;
        constexpr int waves = kq::heads::kBackWaves;
        // a part's tokens in as few blocks as two tables of 32 KB allow (one of 32 tokens is level with four of 8)
        const int64_t per = (g.m + parts - 1) / parts;
        int64_t want = kBackTable / (rope.half + V);
        // a block's passes times `per` stay below 2^32 (Divisor)
        const int64_t per_token = a.per.n > b.per.n ? a.per.n : b.per.n;
        if (want * per_token > ((int64_t)1 << 32) / per_token) want = ((int64_t)1 << 32) / (per_token * per_token);
        if (want < 1) want = 1;
        const int64_t rounds = per > want ? (per + want - 1) / want : 1;
        g.tokens = (int)((per + rounds - 1) / rounds);
        g.kind[0] = a;
        g.kind[1] = b;
        const size_t tables = 2 * (size_t)g.tokens * (rope.half + V) * sizeof(float2);
        const size_t join = (size_t)waves * 2 * LG * U * 2 * V * sizeof(float);
        auto go = [&](auto I, auto NT) {
            hipLaunchKernelGGL((kq::heads::backward_kernel<T, V, LG, U, I(), V * sizeof(T) == 16 && NT()>), dim3((unsigned)parts),
                               dim3(kq::heads::kBackThreads), tables > join ? tables : join, (hipStream_t)stream,
                               (const T *)dy.p, dy.ld, dy.hs, (const T *)x.p, x.ld, x.hs, w0, w1, g, rope,
                               (T *)const_cast<void *>(dx.p), dx.ld, dx.hs, parts, p0, p1);
        };
        const bool nt = kq::streamed_once((g.norm ? 3 : 2) * g.m * heads * rope.d * (int64_t)sizeof(T));
        if (inter && nt) go(std::true_type(), std::true_type());
        else if (inter) go(std::true_type(), std::false_type());
        else if (nt) go(std::false_type(), std::true_type());
        else go(std::false_type(), std::false_type());
        return launched();
    });
}

template <class T>
kq_status launch_write(const Tensor &k, const Tensor &v, const float *w, int64_t k_heads, int64_t v_heads, Geom g,
                       const Rope &rope, bool inter, const kq::heads::Cache &cache, kq_stream_t stream) {
    return choose<8>(sizeof(T), rope, inter, k_heads, v_heads, {k, v}, [&](auto form, auto a, auto b) {
        constexpr int V = decltype(form)::kV, LG = decltype(form)::kLG, U = decltype(form)::kU;
        const Plan p = plan_of(g.m, a, b, rope.half, 64 / LG);
        if (p.blocks >= (int64_t)1 << 24) return KQ_ERR_UNSUPPORTED;
        g.kind[0] = a;
        g.kind[1] = b;
        g.tokens = p.tokens;
        // the pieces of a unit lie a multiple of 32 channels apart, and units of unlike kinds start at multiples of four
        const int r = 2 * rope.half;
        const bool quads = V == 8 && (inter ? rope.d % 64 == 0 : rope.half % 32 == 0 && (rope.d - r) % 64 == 0);
        const int stage_at = (2 * p.tokens * (rope.half + V) + 3) / 4 * 4;  // in floats, 16-byte aligned
        const size_t lds = (size_t)(stage_at + (quads ? 0 : kq::heads::kWaves * (64 / LG) * rope.d)) * sizeof(float);
        auto go = [&](auto I, auto Q) {
            hipLaunchKernelGGL((kq::heads::cache_write_kernel<T, V, LG, U, I(), V == 8 && Q()>),
                               dim3((unsigned)p.blocks, (unsigned)p.splits), dim3(kq::heads::kThreads), lds,
                               (hipStream_t)stream, (const T *)k.p, k.ld, k.hs, (const T *)v.p, v.ld, v.hs, w, g, rope,
                               cache, stage_at);
        };
        if (inter && quads) go(std::true_type(), std::true_type());
        else if (inter) go(std::true_type(), std::false_type());
        else if (quads) go(std::false_type(), std::true_type());
        else go(std::false_type(), std::false_type());
        return launched();
    });
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
    const Geom g{m, {}, 0, norm != 0, eps};
    const Tensor x(X, ldx, hsx, m, heads), y(Y, ldy, hsy, m, heads);
    const bool inter = r.half > 0 && rope->interleaved != 0;
    return type == KQ_BF16 ? launch_forward<uint16_t>(x, y, weight_q, weight_k, heads, q_heads, g, r, inter, stream)
                           : launch_forward<float>(x, y, weight_q, weight_k, heads, q_heads, g, r, inter, stream);
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
    const Geom g{m, {}, 0, norm != 0, eps};
    const Tensor dy(dY, lddy, hsdy, m, heads), x(X, ldx, hsx, m, heads), dx(dX, lddx, hsdx, m, heads);
    const bool inter = r.half > 0 && rope->interleaved != 0;
    s = type == KQ_BF16
            ? launch_backward<uint16_t>(dy, x, dx, weight_q, weight_k, heads, q_heads, g, r, inter, (int)parts, p0, p1,
                                          stream)
            : launch_backward<float>(dy, x, dx, weight_q, weight_k, heads, q_heads, g, r, inter, (int)parts, p0, p1,
                                          stream);
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
    const Geom g{m, {}, 0, norm != 0 && k_heads, eps};
    const kq::heads::Cache cache{slots, cache_slots, {codes_k, codes_v}, {scales_k, scales_v}};
    // a missing tensor takes the other's place in the choice of the access width
    const Tensor k(k_heads ? K : V, k_heads ? ldk : ldv, k_heads ? hsk : hsv, m, k_heads ? k_heads : v_heads);
    const Tensor v(v_heads ? V : K, v_heads ? ldv : ldk, v_heads ? hsv : hsk, m, v_heads ? v_heads : k_heads);
    const bool inter = r.half > 0 && rope->interleaved != 0;
    return type == KQ_BF16 ? launch_write<uint16_t>(k, v, weight, k_heads, v_heads, g, r, inter, cache, stream)
                           : launch_write<float>(k, v, weight, k_heads, v_heads, g, r, inter, cache, stream);
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
    const bool vec = aligned(Y, 16) && y.ld * es % 16 == 0 && y.hs * es % 16 == 0;
    const int64_t pieces = heads * (d / 8), per_head = d / 8;
    const bool nt = kq::streamed_once(m * heads * d * es);
    kq_status status = KQ_OK;
    auto go = [&](auto type0, auto R, auto VEC, auto NT) {
        typedef decltype(type0) T;
        constexpr int64_t places = R() * kq::heads::kThreads;
        // with several tokens a workgroup, i < places and n <= 1024; at < 2^23 and per_head <= 128
        const int64_t tokens = pieces <= 1024 && pieces < places ? places / pieces : 1, splits = (tokens * pieces + places - 1) / places;
        const int64_t blocks = (m + tokens - 1) / tokens;
        if (splits > 65535 || blocks * splits >= (int64_t)1 << 24) {  // work-items are counted in 32 bits
            status = KQ_ERR_UNSUPPORTED;
            return;
        }
        const kq::heads::Read g{m, cache_slots, (int)tokens, (int)pieces, (int)per_head,
                                (uint32_t)(((uint64_t)1 << 32) / pieces + 1), (uint32_t)(((uint64_t)1 << 32) / per_head + 1)};
        hipLaunchKernelGGL((kq::heads::cache_read_kernel<T, R(), VEC(), NT()>), dim3((unsigned)blocks, (unsigned)splits),
                           dim3(kq::heads::kThreads), 0, (hipStream_t)stream, slots, codes, scales, g, (T *)Y, y.ld, y.hs);
        status = launched();
    };
    typedef std::integral_constant<int, 8> Many;
    typedef std::integral_constant<int, 1> One;
    auto go_type = [&](auto type0) {
        const bool few = m * pieces <= (int64_t)kqhost::compute_units() * 8 * kq::heads::kThreads;
        if (vec && nt) go(type0, Many(), std::true_type(), std::true_type());
        else if (vec && few) go(type0, One(), std::true_type(), std::false_type());
        else if (vec) go(type0, Many(), std::true_type(), std::false_type());
        else go(type0, Many(), std::false_type(), std::false_type());
    };
    if (type == KQ_BF16) go_type((uint16_t)0);
    else go_type(0.f);
    return status;
}

}  // extern "C"
