// Layer norm in front of the quantized layers: forward, backward with the
// reduction of its parameters' gradients, and forward straight into the
// Kronecker transform and MXFP4 quantizer (KroQuant, arXiv 2607.21446v1,
// Sec. 1 Eq. 1, Sec. 3.1-3.2).
//
// Per row x of d values, in fp32:
//   mean = sum x / d, rstd = 1 / sqrt(sum (x - mean)^2 / d + eps),
//   y = (x - mean) rstd w + b.
// The mean is summed in 64 bits: a mean near zero is what is left of values
// that cancel, and 32 bits would leave it with the rounding of the largest. It
// is kept as c + off (c its fp32 rounding, off the rest), so that the rounding
// of the mean itself (2^-24 |mean|, 1000 times the rest for a mean of 3000
// beside a deviation of 1) never enters y: with v = x - c,
//   sum (x - mean)^2 = sum v^2 - d off^2,  (x - mean) rstd = v rstd - off rstd,
// one subtraction and two multiply-adds per element.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>
#include <type_traits>
#include <utility>

#include "kq.h"
#include "kq_chunk.hpp"
#include "kq_device.hpp"
#include "kq_host.hpp"
#include "kq_lanesum.hpp"

namespace kq {
namespace norm {

constexpr int kThreads = 256;

// Sum over a workgroup of 4 waves, in every thread.
template <class V>
__device__ __forceinline__ V block_sum(V v) {
    __shared__ V red[kThreads / 64];
    v = wave_sum(v);
    __syncthreads();  // the previous call's values have been read
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return (red[0] + red[1]) + (red[2] + red[3]);
}

// A row's statistics.
struct Stats {
    float c, off, rstd, shift;
    __device__ __forceinline__ float normed(float x) const { return fmaf(x - c, rstd, shift); }
    __device__ __forceinline__ void set_mean(double sum, double inv) {
        const double mean = sum * inv;
        c = (float)mean;
        off = (float)(mean - c);
    }
    __device__ __forceinline__ void set_rstd(float squares, double inv, float eps) {  // sum (x - c)^2
        const float var = fmaf(squares, (float)inv, -off * off);
        rstd = __builtin_amdgcn_rsqf((var < 0.f ? 0.f : var) + eps);  // 1 ulp; NaN stays NaN
        shift = -off * rstd;
    }
};

// Statistics of a row by a workgroup that reads it element by element.
template <class T>
__device__ __forceinline__ Stats row_stats(const T *x, int64_t d, float eps) {
    Stats st;
    const double inv = 1.0 / (double)d;
    double s = 0.0;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) s += (double)load1(x + c);
    st.set_mean(block_sum(s), inv);
    float q = 0.f;
    for (int64_t c = threadIdx.x; c < d; c += kThreads) {
        const float v = load1(x + c) - st.c;
        q = fmaf(v, v, q);
    }
    st.set_rstd(block_sum(q), inv, eps);
    return st;
}

// Forward of rows wider than registers hold; one workgroup per row, the row read three times
// (twice from the caches).
template <class T>
__global__ __launch_bounds__(kThreads) void forward_any_kernel(const T *__restrict__ X, int64_t m, int64_t d,
                                                               int64_t ldx, const float *__restrict__ w,
                                                               const float *__restrict__ b, float eps,
                                                               T *__restrict__ Y, int64_t ldy,
                                                               float *__restrict__ mean, float *__restrict__ rstd) {
    for (int64_t i = blockIdx.x; i < m; i += gridDim.x) {
        const T *x = X + i * ldx;
        const Stats st = row_stats(x, d, eps);
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float h = st.normed(load1(x + c));
            store1(Y + i * ldy + c, fmaf(h, w ? w[c] : 1.0f, b ? b[c] : 0.0f));
        }
        if (threadIdx.x == 0) {
            if (mean) mean[i] = st.c;
            if (rstd) rstd[i] = st.rstd;
        }
    }
}

// Backward of such rows, dx: one workgroup per row.
template <class T>
__global__ __launch_bounds__(kThreads) void backward_dx_any_kernel(const T *__restrict__ dY, int64_t lddy,
                                                                   const T *__restrict__ X, int64_t ldx, int64_t m,
                                                                   int64_t d, const float *__restrict__ w,
                                                                   const float *__restrict__ mean,
                                                                   const float *__restrict__ rstd,
                                                                   T *__restrict__ dX, int64_t lddx) {
    for (int64_t i = blockIdx.x; i < m; i += gridDim.x) {
        const float mu = mean[i], rs = rstd[i], inv = 1.0f / (float)d;
        float a = 0.f, b = 0.f;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float g = load1(dY + i * lddy + c) * (w ? w[c] : 1.0f);
            const float h = (load1(X + i * ldx + c) - mu) * rs;
            a += g;
            b = fmaf(g, h, b);
        }
        a = block_sum(a) * inv;
        b = block_sum(b) * inv;
        for (int64_t c = threadIdx.x; c < d; c += kThreads) {
            const float g = load1(dY + i * lddy + c) * (w ? w[c] : 1.0f);
            const float h = (load1(X + i * ldx + c) - mu) * rs;
            store1(dX + i * lddx + c, rs * (fmaf(-h, b, g - a)));
        }
    }
}

// Backward of such rows, the parameters' gradients: workgroup (x, p) sums 256 columns over
// the rows p, p + parts, ... into row p of the partial sums.
template <class T>
__global__ __launch_bounds__(kThreads) void backward_params_any_kernel(
    const T *__restrict__ dY, int64_t lddy, const T *__restrict__ X, int64_t ldx, int64_t m, int64_t d,
    const float *__restrict__ mean, const float *__restrict__ rstd, int parts, float *__restrict__ pw,
    float *__restrict__ pb) {
    const int64_t c = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (c >= d) return;
    const int p = (int)blockIdx.y;
    float sw = 0.f, sb = 0.f;
    for (int64_t i = p; i < m; i += parts) {
        const float dy = load1(dY + i * lddy + c);
        sw = fmaf(dy, (load1(X + i * ldx + c) - mean[i]) * rstd[i], sw);
        sb += dy;
    }
    if (pw) pw[p * d + c] = sw;
    if (pb) pb[p * d + c] = sb;
}

// out[c] = sum over p of part[p][c]: 32 columns per workgroup (one cache line of a part), half
// wave w adds the parts w, w + 32, ... in turn, then four of them the 32 sums in order and the
// first those four; y = 0 for the first output, 1 for the second. Few columns make few
// workgroups, so the parts are spread as wide as one has threads (256 parts of 2 x 1152
// columns: 2.4 us).
constexpr int kColumns = 32, kChains = 32;
__global__ __launch_bounds__(kColumns *kChains) void reduce_parts_kernel(const float *__restrict__ part0,
                                                                         const float *__restrict__ part1, int parts,
                                                                         int64_t d, float *__restrict__ out0,
                                                                         float *__restrict__ out1) {
    __shared__ float red[kChains][kColumns + 1];
    const float *part = blockIdx.y ? part1 : part0;
    float *out = blockIdx.y ? out1 : out0;
    if (!out) return;
    const int col = threadIdx.x % kColumns, w = threadIdx.x / kColumns;
    for (int64_t c0 = (int64_t)blockIdx.x * kColumns; c0 < d; c0 += (int64_t)gridDim.x * kColumns) {
        const int64_t c = c0 + col;
        float s = 0.f;
        if (c < d) {
#pragma unroll 8
            for (int p = w; p < parts; p += kChains) s += part[p * d + c];
        }
        red[w][col] = s;
        __syncthreads();
        if (w < 4) {
            s = red[8 * w][col];
#pragma unroll
            for (int i = 1; i < 8; ++i) s += red[8 * w + i][col];
        }
        __syncthreads();
        if (w < 4) red[w][col] = s;
        __syncthreads();
        if (w == 0 && c < d) out[c] = (red[0][col] + red[1][col]) + (red[2][col] + red[3][col]);
        __syncthreads();
    }
}

// Layer norm, transform and quantizer of rows wider than registers hold: one
// workgroup per row, a quad of lanes per 32-channel block, the row read three times.
template <class T>
__global__ __launch_bounds__(kThreads) void quantize_wide_kernel(const T *__restrict__ X, int64_t m, int64_t d,
                                                            int64_t ldx, const float *__restrict__ w,
                                                            const float *__restrict__ b, float eps,
                                                            const float *__restrict__ factors,
                                                            uint8_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales, int packed,
                                                            float *__restrict__ y_debug, float *__restrict__ mean,
                                                            float *__restrict__ rstd) {
    const int sub = threadIdx.x & 3;
    const int nblk = (int)(d / 32);
    for (int64_t i = blockIdx.x; i < m; i += gridDim.x) {
        const T *x = X + i * ldx;
        const Stats st = row_stats(x, d, eps);
        for (int j = threadIdx.x >> 2; j < nblk; j += kThreads / 4) {
            const int c = 32 * j + 8 * sub;
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = st.normed(load1(x + c + e));
                y[e] = fmaf(h, w ? w[c + e] : 1.0f, b ? b[c + e] : 0.0f);
            }
            if (factors) {
                KronLane L;
                kron_lane_setup(factors + (int64_t)j * 20, sub, L);
                kron_apply8(y, L);
            }
            uint32_t sbyte;
            const uint32_t q = quantize_quad_f32(y, sbyte);
            *reinterpret_cast<uint32_t *>(codes + i * (d / 2) + c / 2) = q;
            if (sub == 0) {
                if (packed) scales[((int64_t)(j >> 3) * m + i) * 8 + 4 * (j & 1) + ((j & 7) >> 1)] = (uint8_t)sbyte;
                else scales[i * nblk + j] = (uint8_t)sbyte;
            }
            if (y_debug) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y_debug[i * d + c + e] = y[e];
            }
        }
        if (threadIdx.x == 0) {
            if (mean) mean[i] = st.c;
            if (rstd) rstd[i] = st.rstd;
        }
    }
}

// ---------------------------------------------------------------------------
// Rows of up to 16384 channels, held in registers from one read. A row belongs
// to W waves; wave w holds the C pieces of 512 channels W c + w, c < C, 8 of them
// in each lane (Lanes: neighbours in rows of whole 16-byte pieces, every 64th
// otherwise), so every access of a wave is one contiguous run. Only piece C - 1
// can lie past the row's end, whole or in part: there it reads zeros and its
// stores are dropped (record counts of the row's bytes), and its centred values
// are left out of the sum of squares.
// Rows are walked by a persistent grid, so the parameters (fp32, four times the
// bytes of a bf16 row) are loaded once per workgroup, and the next row's loads
// are in flight while a row is summed. With W = 1 a workgroup's waves walk
// rows of their own and there is no barrier in the loop.
//
// Bound by memory where there are many rows (us on the device; the bytes of one
// read and one write): forward 8192 x 4608 bf16 28 (5.4 TB/s), 4096 x 16384 bf16
// 45 (5.9), 8192 x 4609 bf16, element by element, 35 (4.3), 29412 x 716 17.5 (4.8);
// backward 16384 x 4096 fp32 141 (5.7), 4096 x 1152 bf16 9.5 and 2.2 for the sum of
// its parts. By the launch and two dependent latencies where there are few: one row
// of 4096 2.3.
// ---------------------------------------------------------------------------
// Parameters of a lane's chunk (fp32; `none` where there are none or past d).
template <bool VEC = true>
__device__ __forceinline__ void load_params(const float *p, int64_t ch, int64_t d, float none, float v[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = none;
    if (!VEC) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (p && ch + 64 * e < d) v[e] = p[ch + 64 * e];
    } else if (p && ch < d) {
        const float4 a = *reinterpret_cast<const float4 *>(p + ch), b = *reinterpret_cast<const float4 *>(p + ch + 4);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// Sum of v over the W waves of a row, in every lane; `red` belongs to this sum alone and
// is written again only after another row_sum's barrier.
template <int W, class V>
__device__ __forceinline__ V row_sum(V v, V *red, int wave) {
    v = wave_sum(v);
    if (W == 1) return v;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    V s = red[0];
#pragma unroll
    for (int w = 1; w < W; ++w) s += red[w];
    return s;
}

template <int W>
constexpr int kGroupThreads = W == 1 ? 256 : 64 * W;

// A row's statistics from its chunks; `ch`: the last chunk's first channel.
template <int W, class T, bool VEC, int C>
__device__ __forceinline__ Stats chunk_stats(const Chunk<T, VEC> (&raw)[C], uint32_t ch, int64_t d, double inv, float eps,
                                             double *red_sum, float *red_sq, int wave) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float x[8];
        raw[c].widen(x);
        // each value widened first: eight bf16 values whose exponents differ by 13 or more do not add up
        // exactly in fp32, and a mean that is left of large ones cancelling would show it (with the eight
        // summed in fp32: norm into codes 8192 x 4096 24.1 us, 24.9; norm 8192 x 4608 27.7, 27.9)
        auto pair = [&](int e) { return (double)x[e] + (double)x[e + 1]; };
        s += (pair(0) + pair(2)) + (pair(4) + pair(6));
    }
    Stats st;
    st.set_mean(row_sum<W>(s, red_sum, wave), inv);
    float q = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float x[8], qc = 0.f;
        raw[c].widen(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float v = VEC || c < C - 1 || ch + 64 * e < d ? x[e] - st.c : 0.f;
            qc = fmaf(v, v, qc);
        }
        q += !VEC || c < C - 1 || ch < d ? qc : 0.f;
    }
    st.set_rstd(row_sum<W>(q, red_sq, wave), inv, eps);
    return st;
}

template <class T, int W, int C, bool NT, bool VEC>
__global__ __launch_bounds__(kGroupThreads<W>) void forward_kernel(const T *__restrict__ X, int64_t m, int64_t d,
                                                                   int64_t ldx, const float *__restrict__ w,
                                                                   const float *__restrict__ b, float eps,
                                                                   T *__restrict__ Y, int64_t ldy,
                                                                   float *__restrict__ mean,
                                                                   float *__restrict__ rstd) {
    __shared__ double red_sum[W];
    __shared__ float red_sq[W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = W == 1 ? 0 : wave;  // this wave's place in its row
    constexpr int R = W == 1 ? 4 : 1;  // rows a workgroup has at a time
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t row = (int64_t)blockIdx.x * R + (W == 1 ? wave : 0);
    if (row >= m) return;  // whole waves, and with W > 1 whole workgroups
    uint32_t ch[C];
    float pw[C][8], pb[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        ch[c] = Lanes<VEC>::first(W * c + wr, lane);
        load_params<VEC>(w, ch[c], d, 1.0f, pw[c]);
        load_params<VEC>(b, ch[c], d, 0.0f, pb[c]);
    }
    const double inv = 1.0 / (double)d;
    const int64_t bytes = d * (int)sizeof(T);
    Chunk<T, VEC> raw[C], next[C];
#pragma unroll
    for (int c = 0; c < C; ++c) next[c].template load<NT>(row_rsrc(X + row * ldx, bytes), ch[c]);
    for (; row < m; row += step) {
#pragma unroll
        for (int c = 0; c < C; ++c) raw[c] = next[c];
        // past the last row: no records, so no access
        const auto ahead = row_rsrc(X + (row + step < m ? row + step : row) * ldx, row + step < m ? bytes : 0);
#pragma unroll
        for (int c = 0; c < C; ++c) next[c].template load<NT>(ahead, ch[c]);
        const Stats st = chunk_stats<W>(raw, ch[C - 1], d, inv, eps, red_sum, red_sq, wr);
        const auto out = row_rsrc(Y + row * ldy, bytes);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float x[8];
            raw[c].widen(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(st.normed(x[e]), pw[c][e], pb[c][e]);
            store8<NT, VEC>(out, ch[c], x, Y);
        }
        if (lane == 0 && wr == 0) {
            if (mean) mean[row] = st.c;
            if (rstd) rstd[row] = st.rstd;
        }
    }
}

// Workgroup p of `parts` in the backward pass walks the p-th run of rows, or, where the rows
// stream from memory (NT), the rows p, p + parts, ..., so that all workgroups together read one
// stretch of it (16384 x 8192 bf16 152 us, 167 with runs; from the caches, runs are faster: 1024 x
// 4096 12.4 us, 13.1 without). With W = 1, each of its R waves takes every R-th of them. It writes
// their dx and keeps its lanes' columns of dweight and dbias in registers; row p of the partial
// sums gets them at the end.
template <class T, int W, int C, int R, bool NT, bool VEC>
__global__ __launch_bounds__(64 * W * R) void backward_kernel(const T *__restrict__ dY, int64_t lddy,
                                                                    const T *__restrict__ X, int64_t ldx, int64_t m,
                                                                    int64_t d, const float *__restrict__ w,
                                                                    const float *__restrict__ mean,
                                                                    const float *__restrict__ rstd,
                                                                    T *__restrict__ dX, int64_t lddx, int parts,
                                                                    float *__restrict__ pw, float *__restrict__ pb) {
    __shared__ float red[2][2][W];
    __shared__ float4 join[R][W == 1 ? C : 1][2][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = W == 1 ? 0 : wave;
    static_assert(W == 1 || R == 1, "rows side by side have a wave each");
    // 1024 threads have 128 registers each, too few for the next row beside two chunks of 32-bit values
    constexpr bool kAhead = W < 16 || C < 2 || (VEC && sizeof(T) == 2);
    const int64_t p = blockIdx.x, run = (m + parts - 1) / parts;
    const int64_t apart = NT ? parts : 1, step = R * apart;
    const int64_t end = NT || m - p * run < run ? m : (p + 1) * run;
    int64_t row = (NT ? p : p * run) + (W == 1 ? apart * wave : 0);
    uint32_t ch[C];
    float wv[C][8], aw[C][8], ab[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        ch[c] = Lanes<VEC>::first(W * c + wr, lane);
        load_params<VEC>(w, ch[c], d, 1.0f, wv[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[c][e] = ab[c][e] = 0.f;
    }
    const float inv = 1.0f / (float)d;
    const int64_t bytes = d * (int)sizeof(T);
    Chunk<T, VEC> x[C], dy[C], nx[C], ndy[C];
    float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;
    auto fetch = [&](int64_t r) {
        const bool in = r < end;
        const int64_t rr = in ? r : 0;
        const auto rx = row_rsrc(X + rr * ldx, in ? bytes : 0), rd = row_rsrc(dY + rr * lddy, in ? bytes : 0);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            nx[c].template load<NT>(rx, ch[c]);
            ndy[c].template load<NT>(rd, ch[c]);
        }
        nmu = mean[rr];
        nrs = rstd[rr];
    };
    if (kAhead) fetch(row);
    for (int par = 0; row < end; row += step, par ^= 1) {
        if (!kAhead) fetch(row);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            x[c] = nx[c];
            dy[c] = ndy[c];
        }
        mu = nmu;
        rs = nrs;
        if (kAhead) fetch(row + step);
        float g[C][8], h[C][8], a = 0.f, b = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float v[8], t[8];
            x[c].widen(v);
            dy[c].widen(t);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[c][e] = (v[e] - mu) * rs;
                g[c][e] = t[e] * wv[c][e];
                aw[c][e] = fmaf(t[e], h[c][e], aw[c][e]);
                ab[c][e] += t[e];
                a += g[c][e];
                b = fmaf(g[c][e], h[c][e], b);
            }
        }
        a = wave_sum(a);
        b = wave_sum(b);
        if (W > 1) {
            // two sets in turn: a set is written again only after the next row's barrier
            if (lane == 0) {
                red[par][0][wr] = a;
                red[par][1][wr] = b;
            }
            __syncthreads();
            a = red[par][0][0];
            b = red[par][1][0];
#pragma unroll
            for (int i = 1; i < W; ++i) {
                a += red[par][0][i];
                b += red[par][1][i];
            }
        }
        a *= inv;
        b *= inv;
        const auto out = row_rsrc(dX + row * lddx, bytes);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = rs * fmaf(-h[c][e], b, g[c][e] - a);
            store8<false, VEC>(out, ch[c], t, dX);
        }
    }
    // with W = 1, the R waves' columns meet in LDS, in wave order
    auto put = [&](float (&v)[C][8], float *to) {
        if (!to) return;
        to += p * d;
        if (W > 1 && !VEC) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (ch[c] + 64 * e < d) to[ch[c] + 64 * e] = v[c][e];
            return;
        }
        if (W > 1) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (ch[c] < d) {
                    *reinterpret_cast<float4 *>(to + ch[c]) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
                    *reinterpret_cast<float4 *>(to + ch[c] + 4) = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
                }
            return;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < C; ++c) {
            join[wave][c][0][lane] = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
            join[wave][c][1][lane] = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
        }
        __syncthreads();
        for (int i = wave; i < 2 * C; i += R) {
            float4 s = join[0][i >> 1][i & 1][lane];
#pragma unroll
            for (int k = 1; k < R; ++k) {
                const float4 o = join[k][i >> 1][i & 1][lane];
                s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
            }
            const uint32_t cc = Lanes<VEC>::first(i >> 1, lane) + 4 * (i & 1) * Lanes<VEC>::kStep;
            if (VEC) {
                if (cc < d) *reinterpret_cast<float4 *>(to + cc) = s;
            } else {
                const float one[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (cc + 64 * e < d) to[cc + 64 * e] = one[e];
            }
        }
    };
    put(aw, pw);
    put(ab, pb);
}

// Layer norm, transform and quantizer (lanes with 8 neighbours). A quad of lanes holds a 32-channel block and a wave's
// chunk 16 of them (the segments of the fused transform kernels), for which every lane keeps
// its block's 16 coefficients and its channels' parameters over all rows of the workgroup.
// (bf16 with 3 chunks and fewer than 8 waves: held to the 168 registers of three waves per SIMD:
// 8192 x 1152 11.8 us, 14.3 without, 8192 x 4608 28.9 and 29.7. fp32 spills there: 8192 x 4608 44, 42
// without, 2048 x 12288 68 and 33.)
// 8192 x 4096 bf16 takes 25 to 28 us, its bytes 17 at 5.1 TB/s. Neither memory nor the vector units
// alone bound it (profiles/counters_norm_into_codes.md): 340 vector instructions per wave and row
// (statistics, norm, five transform stages, quantizer) keep the units busy 71% of the time; the
// waves wait for a row or at the two barriers of its sums 31% of theirs, and for their turn to issue
// another 31%. The sums on the matrix unit cost registers and gained nothing.
template <class T, int W, int C>
__global__ __launch_bounds__(kGroupThreads<W>, sizeof(T) == 2 && C == 3 && W < 8 ? 3 : 1) void quantize_kernel(
    const T *__restrict__ X, int64_t m, int64_t d, int64_t ldx, const float *__restrict__ w,
    const float *__restrict__ b, float eps, const float *__restrict__ factors, uint8_t *__restrict__ codes,
    uint8_t *__restrict__ scales, int packed, float *__restrict__ y_debug, float *__restrict__ mean,
    float *__restrict__ rstd) {
    __shared__ double red_sum[W];
    __shared__ float red_sq[W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = W == 1 ? 0 : wave, sub = lane & 3;
    constexpr int R = W == 1 ? 4 : 1;
    const int64_t step = (int64_t)gridDim.x * R;
    int64_t row = (int64_t)blockIdx.x * R + (W == 1 ? wave : 0);
    if (row >= m) return;
    uint32_t ch[C], scale_at[C];
    float pw[C][8], pb[C][8], coef[C][16];
    bool shear[C];
    const double inv = 1.0 / (double)d;
    const int64_t bytes = d * (int)sizeof(T);
    Chunk<T> raw[C], next[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        ch[c] = 8u * (64u * (W * c + wr) + lane);
        next[c].load(row_rsrc(X + row * ldx, bytes), ch[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        load_params(w, ch[c], d, 1.0f, pw[c]);
        load_params(b, ch[c], d, 0.0f, pb[c]);
        // the block's scale byte from its row's first, stored by the quad's first lane; the others and
        // the blocks past d are past every record count
        const uint32_t j = ch[c] / 32;
        scale_at[c] = sub || ch[c] >= d ? 0xFFFFFFF0u
                      : packed          ? (uint32_t)((j >> 3) * m * 8) + 4 * (j & 1) + ((j & 7) >> 1)
                                        : j;
        shear[c] = true;
#pragma unroll
        for (int i = 0; i < 16; ++i) coef[c][i] = 0.f;
        if (factors) {
            const bool in = ch[c] < d;
            float f[20];
            SetupLane S;
            S.shear = true;
            if (in) {
                load_factors20(factors + (int64_t)(ch[c] / 32) * 20, f);
                setup_ratios(f, S);
            }
            shear[c] = __builtin_amdgcn_ballot_w64(!S.shear) == 0;
            if (in) {
                if (shear[c]) write_shear_coefs(f, S, sub, coef[c]);
                else write_general_coefs(f, sub, coef[c]);
            }
        }
    }
    // one row in `now` while the next one comes into `ahead`
    auto one = [&](Chunk<T> (&now)[C], Chunk<T> (&ahead)[C]) {
        const auto rx = row_rsrc(X + (row + step < m ? row + step : row) * ldx, row + step < m ? bytes : 0);
#pragma unroll
        for (int c = 0; c < C; ++c) ahead[c].load(rx, ch[c]);
        const Stats st = chunk_stats<W>(now, ch[C - 1], d, inv, eps, red_sum, red_sq, wr);
        const auto rc = row_rsrc(codes + row * (d / 2), d / 2);
        const auto rs = packed ? row_rsrc(scales + 8 * row, m * (d / 32) - 8 * row) : row_rsrc(scales + row * (d / 32), d / 32);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float y[8];
            now[c].widen(y);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(st.normed(y[e]), pw[c][e], pb[c][e]);
            if (factors) {
                if (shear[c]) apply_coefs<true>(y, coef[c]);
                else apply_coefs<false>(y, coef[c]);
            }
            uint32_t sbyte;
            const uint32_t q = quantize_quad_f32(y, sbyte);
            __builtin_amdgcn_raw_buffer_store_b32(q, rc, ch[c] / 2, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)sbyte, rs, scale_at[c], 0, 0);
            if (y_debug) store8(row_rsrc(y_debug + row * d, 4 * d), ch[c], y, y_debug);
        }
        if (lane == 0 && wr == 0) {
            if (mean) mean[row] = st.c;
            if (rstd) rstd[row] = st.rstd;
        }
    };
    // two sets in turn: no register is copied
    for (;;) {
        one(next, raw);
        row += step;
        if (row >= m) break;
        one(raw, next);
        row += step;
        if (row >= m) break;
    }
}

}  // namespace norm
}  // namespace kq

// ===========================================================================
// Host side
// ===========================================================================
namespace {

using kqhost::aligned;
using kqhost::launched;
using kqhost::sizes_fit;

bool good_eps(float eps) { return eps >= 0.f && eps <= 3.4e38f; }
bool good_type(int type) { return type == KQ_F32 || type == KQ_BF16; }
uintptr_t size_of(int type) { return type == KQ_BF16 ? 2 : 4; }

// Workgroups that walk m rows: enough to fill the chip, the rest by stride.
unsigned row_grid(int64_t m) { return (unsigned)(m < 65536 ? m : 65536); }

// Whether every row is whole 16-byte pieces and so are the parameters.
bool vector_rows(int type, int64_t d, std::initializer_list<const void *> ptrs, std::initializer_list<int64_t> lds,
                 std::initializer_list<const float *> params) {
    if (d % 8 != 0) return false;
    for (const void *p : ptrs)
        if (!aligned(p, 16)) return false;
    for (const int64_t ld : lds)
        if (ld % (type == KQ_BF16 ? 8 : 4) != 0) return false;
    for (const float *p : params)
        if (!aligned(p, 16)) return false;
    return true;
}

// Waves per row and chunks of 8 channels per lane for a row of `pieces` 512-channel pieces: the
// first entry W, C of a kernel's list that holds it, f(W, C); false if none does.
template <class F>
bool first_shape(int64_t, std::integer_sequence<int>, F) {
    return false;
}
template <int W, int C, int... Rest, class F>
bool first_shape(int64_t pieces, std::integer_sequence<int, W, C, Rest...>, F f) {
    if (pieces > W * C) return first_shape(pieces, std::integer_sequence<int, Rest...>(), f);
    f(std::integral_constant<int, W>(), std::integral_constant<int, C>());
    return true;
}

// In each list, an entry is reached only by rows of more than W (C - 1) pieces, so that no chunk but
// the last has places past the row's end.
// Many rows: few waves per row, so that a wave has work between its sums, with as few empty
// places as the lists allow (us at 8192 x 1152: norm 8.8 with 1 x 3, 10.7 with 2 x 2, 12.7 with
// 4 x 1; norm and quantizer 11.8, 14.6, 16.2).
// Above three waves, multiples of four: a workgroup's waves are dealt to the four SIMDs from
// the first on, so 5 waves take a second place on one of them in every workgroup. 3 x 3 is for
// rows of 9 pieces (norm and quantizer 8192 x 4608: 28.9 us, 33.1 with 4 x 3, 41.0 with 8 x 2; the norm
// 28.1, 28.3 and 30.4). Rows of 5 and 6 pieces take 4 x 2, with up to three of its eight places
// empty; 3 x 2 was not measured for them.
using Many = std::integer_sequence<int, 1, 1, 1, 2, 1, 3, 2, 2, 4, 2, 3, 3, 4, 3, 8, 2, 8, 3, 8, 4>;
// Fewer rows than compute units: one chunk per lane where 16 waves reach, so that a row's time
// is one memory latency.
using Few = std::integer_sequence<int, 1, 1, 2, 1, 4, 1, 8, 1, 16, 1, 16, 2>;
// Backward: at most one workgroup per compute unit (the parts of the parameters' sums), so
// as many waves as the row has pieces, from 2048 channels on.
using Backward = std::integer_sequence<int, 1, 1, 1, 2, 1, 3, 4, 1, 8, 1, 8, 2, 8, 3, 16, 2>;

int64_t pieces_of(int64_t d) { return (d + 511) / 512; }

// Workgroups of `waves` waves (4 rows at a time when waves == 1) that keep `per_cu` waves on
// every compute unit, or one per row where there are fewer.
unsigned persistent_grid(int64_t m, int waves, int per_cu) {
    const int64_t rows = waves == 1 ? 4 : 1, need = (m + rows - 1) / rows;
    const int64_t fill = (int64_t)kqhost::compute_units() * per_cu / (waves == 1 ? 4 : waves);
    return (unsigned)(need < fill ? need : fill);
}

template <class T>
kq_status launch_forward(const void *X, int64_t m, int64_t d, int64_t ldx, const float *weight, const float *bias,
                         float eps, void *Y, int64_t ldy, float *mean, float *rstd, bool vec, kq_stream_t stream) {
    const bool few = m < kqhost::compute_units();
    auto go = [&](auto W, auto C, auto NT, auto VEC) {
        // one resident round, by the registers that the shapes of more chunks leave (us, 1000 x 16384 bf16
        // 13.5, 16.9 in two rounds); two for fp32 rows of 16-byte pieces (8192 x 16384 249, 267 in one)
        constexpr int per_cu = W() == 8 && C() == 4 && (sizeof(T) == 2 || !VEC()) ? 8
                               : C() == 3 && !VEC() ? (W() == 8 ? 8 : W() == 3 ? 9 : 12)
                               : W() == 3           ? 12
                                                    : 16;
        hipLaunchKernelGGL((kq::norm::forward_kernel<T, W(), C(), NT(), VEC()>), dim3(persistent_grid(m, W(), per_cu)),
                           dim3(kq::norm::kGroupThreads<W()>), 0, (hipStream_t)stream, (const T *)X, m, d, ldx, weight,
                           bias, eps, (T *)Y, ldy, mean, rstd);
    };
    auto go_plain = [&](auto W, auto C) {
        if (vec) go(W, C, std::false_type(), std::true_type());
        else go(W, C, std::false_type(), std::false_type());
    };
    auto go_nt = [&](auto W, auto C) {
        if (vec) go(W, C, std::true_type(), std::true_type());
        else go(W, C, std::true_type(), std::false_type());
    };
    if (d > 16384 || !(few ? first_shape(pieces_of(d), Few(), go_plain)
                  : kq::streamed_once(2 * m * d * (int)sizeof(T)) ? first_shape(pieces_of(d), Many(), go_nt)
                                                                  : first_shape(pieces_of(d), Many(), go_plain)))
        hipLaunchKernelGGL((kq::norm::forward_any_kernel<T>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const T *)X, m, d, ldx, weight, bias, eps, (T *)Y, ldy, mean, rstd);
    return launched();
}

template <class T>
kq_status launch_backward(const void *dY, int64_t lddy, const void *X, int64_t ldx, int64_t m, int64_t d,
                          const float *weight, const float *mean, const float *rstd, void *dX, int64_t lddx,
                          int64_t parts, float *pw, float *pb, bool params, bool vec, kq_stream_t stream) {
    auto go = [&](auto W, auto C, auto NT, auto VEC) {
        // Rows of one wave: eight at a time, so that a compute unit has two waves per SIMD (us, bf16 with 4
        // and 8: 32768 x 512 36.5, 25.3; 29412 x 716 49.8, 36.2; 4096 x 1152 12.1, 11.6); four where the
        // registers allow two anyway (fp32 by 16 bytes, three chunks: 4096 x 1152 14.8, 15.9)
        constexpr int R = W() > 1 ? 1 : C() == 3 && sizeof(T) == 4 && VEC() ? 4 : 8;
        hipLaunchKernelGGL((kq::norm::backward_kernel<T, W(), C(), R, NT(), VEC()>), dim3((unsigned)parts),
                           dim3(64 * W() * R), 0, (hipStream_t)stream, (const T *)dY, lddy, (const T *)X, ldx, m, d,
                           weight, mean, rstd, (T *)dX, lddx, (int)parts, pw, pb);
    };
    auto go_plain = [&](auto W, auto C) {
        if (vec) go(W, C, std::false_type(), std::true_type());
        else go(W, C, std::false_type(), std::false_type());
    };
    auto go_nt = [&](auto W, auto C) {
        if (vec) go(W, C, std::true_type(), std::true_type());
        else go(W, C, std::true_type(), std::false_type());
    };
    if (d <= 16384 && (kq::streamed_once(3 * m * d * (int)sizeof(T)) ? first_shape(pieces_of(d), Backward(), go_nt)
                                                              : first_shape(pieces_of(d), Backward(), go_plain)))
        return launched();
    hipLaunchKernelGGL((kq::norm::backward_dx_any_kernel<T>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                       (hipStream_t)stream, (const T *)dY, lddy, (const T *)X, ldx, m, d, weight, mean, rstd, (T *)dX,
                       lddx);
    if (params)
        hipLaunchKernelGGL((kq::norm::backward_params_any_kernel<T>), dim3((unsigned)((d + 255) / 256), (unsigned)parts),
                           dim3(kq::norm::kThreads), 0, (hipStream_t)stream, (const T *)dY, lddy, (const T *)X, ldx, m,
                           d, mean, rstd, (int)parts, pw, pb);
    return launched();
}

template <class T>
kq_status launch_quantize(const void *X, int64_t m, int64_t d, int64_t ldx, const float *weight, const float *bias,
                          float eps, const float *factors, uint8_t *codes, uint8_t *scales, int packed, float *y_debug,
                          float *mean, float *rstd, kq_stream_t stream) {
    auto go = [&](auto W, auto C) {
        // one resident round: bf16 rows of three chunks leave registers for three waves per SIMD, fp32 ones
        // and eight waves a workgroup for two (us, 8192 x 12288 bf16 71, 92 in 1.5 rounds; 4096 x 10240 37, 49);
        // with one wave per row the coefficients' setup weighs more and 8 waves per
        // compute unit are faster (8192 x 512 5.9 us, 6.0 with 16)
        constexpr int per_cu = W() == 8 && C() >= 3       ? 8
                               : C() == 3 && sizeof(T) == 4 ? (W() == 3 ? 6 : 8)
                               : C() == 3                   ? 12
                               : W() == 1                   ? 8
                                                            : 16;
        hipLaunchKernelGGL((kq::norm::quantize_kernel<T, W(), C()>), dim3(persistent_grid(m, W(), per_cu)),
                           dim3(kq::norm::kGroupThreads<W()>), 0, (hipStream_t)stream, (const T *)X, m, d, ldx, weight,
                           bias, eps, factors, codes, scales, packed, y_debug, mean, rstd);
    };
    if (d > 16384 || !(m < kqhost::compute_units() ? first_shape(pieces_of(d), Few(), go)
                                                   : first_shape(pieces_of(d), Many(), go)))
        hipLaunchKernelGGL((kq::norm::quantize_wide_kernel<T>), dim3(row_grid(m)), dim3(kq::norm::kThreads), 0,
                           (hipStream_t)stream, (const T *)X, m, d, ldx, weight, bias, eps, factors, codes, scales,
                           packed, y_debug, mean, rstd);
    return launched();
}

}  // namespace

namespace kqhost {

kq_status reduce_parts(const float *part0, const float *part1, int64_t parts, int64_t d, float *out0, float *out1,
                       kq_stream_t stream) {
    const int64_t groups = (d + kq::norm::kColumns - 1) / kq::norm::kColumns;
    hipLaunchKernelGGL(kq::norm::reduce_parts_kernel, dim3((unsigned)(groups < 65536 ? groups : 65536), out1 ? 2 : 1),
                       dim3(kq::norm::kColumns * kq::norm::kChains), 0, (hipStream_t)stream, part0, part1, (int)parts, d, out0, out1);
    return launched();
}

}  // namespace kqhost

extern "C" {

kq_status kq_layernorm(const void *X, int type, int64_t m, int64_t d, int64_t ldx, const float *weight,
                       const float *bias, float eps, void *Y, int64_t ldy, float *mean, float *rstd,
                       kq_stream_t stream) {
    if (m < 0 || d < 0 || ldx < d || ldy < d || !good_eps(eps)) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, d, ldx, ldy})) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || d == 0) return KQ_OK;
    if (!X || !Y) return KQ_ERR_NULL;
    const uintptr_t es = size_of(type);
    if (!aligned(X, es) || !aligned(Y, es) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KQ_ERR_ALIGN;
    const bool vec = vector_rows(type, d, {X, Y}, {ldx, ldy}, {weight, bias});
    return type == KQ_BF16
               ? launch_forward<uint16_t>(X, m, d, ldx, weight, bias, eps, Y, ldy, mean, rstd, vec, stream)
               : launch_forward<float>(X, m, d, ldx, weight, bias, eps, Y, ldy, mean, rstd, vec, stream);
}

kq_status kq_layernorm_backward_workspace_bytes(int64_t m, int64_t d, int64_t *bytes) {
    if (!bytes) return KQ_ERR_NULL;
    *bytes = 0;
    if (m < 0 || d < 0) return KQ_ERR_SHAPE;
    if (!sizes_fit({m, d})) return KQ_ERR_UNSUPPORTED;
    const int64_t parts = kqhost::row_parts(m);
    if (parts > 1) *bytes = parts * 2 * d * 4;
    return KQ_OK;
}

kq_status kq_layernorm_backward(const void *dY, int64_t lddy, const void *X, int64_t ldx, int type, int64_t m,
                                int64_t d, const float *weight, const float *mean, const float *rstd, void *dX,
                                int64_t lddx, float *dweight, float *dbias, void *workspace, int64_t workspace_bytes,
                                kq_stream_t stream) {
    if (m < 0 || d < 0 || ldx < d || lddy < d || lddx < d) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, d, ldx, lddy, lddx})) return KQ_ERR_UNSUPPORTED;
    if (d == 0) return KQ_OK;
    if (!aligned(dweight, 4) || !aligned(dbias, 4)) return KQ_ERR_ALIGN;
    const bool params = dweight || dbias;
    if (m == 0) return params ? kqhost::reduce_parts(nullptr, nullptr, 0, d, dweight, dbias, stream) : KQ_OK;
    if (!dY || !X || !mean || !rstd || !dX) return KQ_ERR_NULL;
    const uintptr_t es = size_of(type);
    if (!aligned(dY, es) || !aligned(X, es) || !aligned(dX, es) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KQ_ERR_ALIGN;
    const int64_t parts = kqhost::row_parts(m);
    float *pw = dweight, *pb = dbias;
    if (params && parts > 1) {
        if (!workspace) return KQ_ERR_NULL;
        if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
        if (workspace_bytes < parts * 2 * d * 4) return KQ_ERR_SHAPE;
        pw = static_cast<float *>(workspace);
        pb = pw + parts * d;
    }
    const bool vec = vector_rows(type, d, {dY, X, dX}, {lddy, ldx, lddx}, {weight, pw, pb});
    const kq_status s =
        type == KQ_BF16 ? launch_backward<uint16_t>(dY, lddy, X, ldx, m, d, weight, mean, rstd, dX, lddx, parts, pw,
                                                    pb, params, vec, stream)
                        : launch_backward<float>(dY, lddy, X, ldx, m, d, weight, mean, rstd, dX, lddx, parts, pw, pb,
                                                 params, vec, stream);
    if (s != KQ_OK) return s;
    if (params && parts > 1) return kqhost::reduce_parts(pw, pb, parts, d, dweight, dbias, stream);
    return KQ_OK;
}

kq_status kq_layernorm_quantize_mxfp4(const void *X, int type, int64_t m, int64_t d, int64_t ldx, const float *weight,
                                      const float *bias, float eps, const float *factors, uint8_t *codes,
                                      uint8_t *scales, int packed, float *y_debug, float *mean, float *rstd,
                                      kq_stream_t stream) {
    if (m < 0 || d < 0 || ldx < d || d % 32 != 0 || (packed && d % 256 != 0) || !good_eps(eps)) return KQ_ERR_SHAPE;
    if (!good_type(type) || !sizes_fit({m, d, ldx}) || d > 32768) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || d == 0) return KQ_OK;
    if (packed && m > (((int64_t)1 << 31) - 16) / (d / 32)) return KQ_ERR_UNSUPPORTED;
    if (!X || !codes || !scales) return KQ_ERR_NULL;
    if (!aligned(X, 16) || ldx % (type == KQ_BF16 ? 8 : 4) != 0 || !aligned(weight, 16) || !aligned(bias, 16) ||
        !aligned(factors, 16) || !aligned(codes, 16) || !aligned(y_debug, 16) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KQ_ERR_ALIGN;
    return type == KQ_BF16
               ? launch_quantize<uint16_t>(X, m, d, ldx, weight, bias, eps, factors, codes, scales, packed, y_debug,
                                           mean, rstd, stream)
               : launch_quantize<float>(X, m, d, ldx, weight, bias, eps, factors, codes, scales, packed, y_debug, mean,
                                        rstd, stream);
}

}  // extern "C"
