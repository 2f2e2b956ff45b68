// The W4A4 product with a linear layer's epilogue,
//   z = deq(A) deq(W)^T + bias,  O = act(z) + residual
// (KroQuant, arXiv 2607.21446v1, Sec. 1 Eq. 2 for the product), and the
// gradients of that epilogue: here the kernels for few rows and for few tiles
// and the choice between them and the 256 x 256 one (kq_gemm256.hip).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "kq.h"
#include "kq_choice.hpp"
#include "kq_device.hpp"
#include "kq_dma.hpp"
#include "kq_epilogue.hpp"
#include "kq_host.hpp"
#include "kq_lanesum.hpp"
#include "kq_tileorder.hpp"

namespace kq {
namespace linear {

typedef float floatx16_t __attribute__((ext_vector_type(16)));

struct Geom {
    int kbytes, kblocks;  // k / 2, k / 32
    int stages;           // ceil(k / 256)
    int tiles_n, tiles_m;
};

// How an operand's scales are read: byte by byte from the MX layout (any k % 32 == 0), or a
// row's eight bytes of a 256-k stage at once, from the MX layout (k % 256 == 0, 8-byte
// aligned) or the packed one.
enum Scales { kBytes = 0, kRows8 = 1, kPacked8 = 2 };

// A workgroup of WK waves computes 16 MF rows x 16 NF columns of O, each wave every
// WK-th 256-k stage of the whole tile on v_mfma_scale_f32_16x16x128_f8f6f4, operands
// straight from memory into registers (a stage of a row is 128 code bytes, one cache
// line) D stages ahead, and the waves' sums meet in LDS in wave order. The
// instruction's A operand is a W fragment and its B operand an A fragment: lane l
// supplies row l % 16 of each and k group l / 16 (one MX block: 16 code bytes, one
// scale byte), and receives O row l % 16, columns 4 (l / 16) + 0..3 of the fragment.
// Rows past m or n and k groups past k are past a record count (or pushed past it) and
// read zero codes.
//
// Why: with few rows a product is its weights' bytes, and a tile's time the latency of its
// stages one after the other, so k is split over the waves and the tiles are as small as the
// instruction. 1 x 4096 x 4096 takes 5.0 us (W and its scales, 8.9 MB, from the Infinity
// Cache: launch, two dependent latencies, the joined sums), 1 x 16384 x 8192 with W from HBM
// 19.2 (71 MB, 3.7 TB/s). Deeper prefetch (D of 2, 4) is level or slower.
template <int F>
struct Stage {
    u32x4_t code[2][F];
    uint32_t scl[2][F];
};

// With GatedEpi a workgroup multiplies the same rows of A by as many of both weights: the second's fragments and
// sums stand behind the first's.
template <class E>
constexpr bool kGated = std::is_same<E, GatedEpi>::value;

template <class T, int SC, int MF, int NF, int WK, int D, class E>
__global__ __launch_bounds__(64 * WK) void product_kernel(const uint8_t *__restrict__ ca,
                                                          const uint8_t *__restrict__ sa,
                                                          const uint8_t *__restrict__ cw,
                                                          const uint8_t *__restrict__ sw, Geom g, E ep) {
    constexpr int NW = kGated<E> ? 2 : 1;
    __shared__ float4 red[WK][NW * MF * NF][64];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int tn = (int)(blockIdx.x % (unsigned)g.tiles_n), tm = (int)(blockIdx.x / (unsigned)g.tiles_n);
    const int64_t m0 = (int64_t)tm * (16 * MF), n0 = (int64_t)tn * (16 * NF);
    const int rows_a = (int)(ep.m - m0 < 16 * MF ? ep.m - m0 : 16 * MF);
    const int rows_w = (int)(ep.n - n0 < 16 * NF ? ep.n - n0 : 16 * NF);
    const int row = lane & 15, grp = lane >> 4;

    auto rsrc = [](const uint8_t *p, int64_t bytes) {
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), (short)0, (int)bytes, 0x00020000);
    };
    const auto rca = rsrc(ca + m0 * g.kbytes, (int64_t)rows_a * g.kbytes);
    const auto rcw = rsrc(cw + n0 * g.kbytes, (int64_t)rows_w * g.kbytes);
    // packed: a padding row reads a neighbour's or a later stage's byte, or zero past the
    // array; its codes are zero and its outputs are not stored
    const auto rsa = SC == kPacked8 ? rsrc(sa + 8 * m0, (int64_t)g.stages * 8 * ep.m - 8 * m0)
                                    : rsrc(sa + m0 * g.kblocks, (int64_t)rows_a * g.kblocks);
    const auto rsw = SC == kPacked8 ? rsrc(sw + 8 * n0, (int64_t)g.stages * 8 * ep.n - 8 * n0)
                                    : rsrc(sw + n0 * g.kblocks, (int64_t)rows_w * g.kblocks);
    const uint8_t *cu = cw, *su = sw;
    if constexpr (kGated<E>) cu = ep.cu, su = ep.su;
    const auto rcu = rsrc(cu + n0 * g.kbytes, (int64_t)rows_w * g.kbytes);
    const auto rsu = SC == kPacked8 ? rsrc(su + 8 * n0, (int64_t)g.stages * 8 * ep.n - 8 * n0)
                                    : rsrc(su + n0 * g.kblocks, (int64_t)rows_w * g.kblocks);
    constexpr uint32_t kNone = 0x80000000u;

    floatx4_t acc[NW][NF][MF];
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int b = 0; b < NF; ++b)
#pragma unroll
            for (int a = 0; a < MF; ++a) acc[w][b][a] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    // stage s of the F fragments of one operand of `rows` rows
    auto fetch = [&](auto &S, __amdgpu_buffer_rsrc_t rc, __amdgpu_buffer_rsrc_t rs, int64_t rows, int s) {
        constexpr int F = sizeof(S.code) / sizeof(u32x4_t) / 2;
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const int r = 16 * f + row;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kb = 8 * s + 4 * h + grp;
                const bool in = kb < g.kblocks;
                S.code[h][f] = __builtin_amdgcn_raw_buffer_load_b128(
                    rc, in ? (uint32_t)(r * g.kbytes + 16 * kb) : kNone, 0, 0);
                if (SC == kBytes)
                    S.scl[h][f] = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? (uint32_t)(r * g.kblocks + kb) : kNone,
                                                                     0, 0);
            }
            if (SC != kBytes) {
                const uint32_t off = SC == kPacked8 ? (uint32_t)(8 * rows * s) + 8 * r : (uint32_t)(r * g.kblocks + 8 * s);
                const auto q = __builtin_amdgcn_raw_buffer_load_b64(rs, s < g.stages ? off : kNone, 0, 0);
                S.scl[0][f] = q[0];
                S.scl[1][f] = q[1];
            }
        }
    };
    // the lane's scale of half h, in byte 0 (packed, half 1: in byte 2)
    auto scale = [&](const auto &S, int h, int f) -> int {
        if (SC == kBytes) return (int)S.scl[h][f];
        if (SC == kRows8) return (int)(S.scl[h][f] >> (8 * grp));
        return (int)((grp & 1 ? S.scl[1][f] : S.scl[0][f]) >> (8 * (grp >> 1)));
    };
    constexpr int kSel1 = SC == kPacked8 ? 2 : 0;

    Stage<MF> A[D];
    Stage<NF> B[D][NW];
    auto fetch_w = [&](int i, int s) {
        fetch(B[i][0], rcw, rsw, ep.n, s);
        if constexpr (kGated<E>) fetch(B[i][1], rcu, rsu, ep.n, s);
    };
#pragma unroll
    for (int i = 0; i < D; ++i) {
        fetch(A[i], rca, rsa, ep.m, wave + WK * i);
        fetch_w(i, wave + WK * i);
    }
    for (int s = wave; s < g.stages; s += WK * D) {
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if (s + WK * i < g.stages) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int wb = 0; wb < NW * NF; ++wb) {
                        const int w = wb / NF, b = wb % NF;
                        const u32x4_t w4 = B[i][w].code[h][b];
                        const i32x8_t fw = {(int)w4[0], (int)w4[1], (int)w4[2], (int)w4[3], 0, 0, 0, 0};
                        const int xw = scale(B[i][w], h, b);
#pragma unroll
                        for (int a = 0; a < MF; ++a) {
                            const u32x4_t a4 = A[i].code[h][a];
                            const i32x8_t fa = {(int)a4[0], (int)a4[1], (int)a4[2], (int)a4[3], 0, 0, 0, 0};
                            if (h == 0)
                                acc[w][b][a] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    fw, fa, acc[w][b][a], 4, 4, 0, xw, 0, scale(A[i], h, a));
                            else
                                acc[w][b][a] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                    fw, fa, acc[w][b][a], 4, 4, kSel1, xw, kSel1, scale(A[i], h, a));
                        }
                    }
            }
            fetch(A[i], rca, rsa, ep.m, s + WK * (i + D));
            fetch_w(i, s + WK * (i + D));
        }
    }
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int b = 0; b < NF; ++b)
#pragma unroll
            for (int a = 0; a < MF; ++a)
                red[wave][(w * NF + b) * MF + a][lane] =
                    make_float4(acc[w][b][a][0], acc[w][b][a][1], acc[w][b][a][2], acc[w][b][a][3]);
    __syncthreads();
    // group q of four columns: row q / (4 NF) of the tile, columns 4 (q % (4 NF)) ..
    for (int q = t; q < 64 * MF * NF; q += 64 * WK) {
        const int r = q / (4 * NF), c4 = q % (4 * NF);
        const int f = (c4 >> 2) * MF + (r >> 4), l = (c4 & 3) * 16 + (r & 15);
        float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float4 v = red[w][f][l];
            z[0] += v.x; z[1] += v.y; z[2] += v.z; z[3] += v.w;
        }
        if constexpr (kGated<E>) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                const float4 v = red[w][MF * NF + f][l];
                y[0] += v.x; y[1] += v.y; y[2] += v.z; y[3] += v.w;
            }
            if (r < rows_a && 4 * c4 < rows_w) {
                const int64_t i = m0 + r, j = n0 + 4 * c4;
                float b[4], bu[4];
                load_bias(ep.bias, ep.n, j, b);
                load_bias(ep.bias_u, ep.n, j, bu);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    z[e] += b[e];
                    y[e] += bu[e];
                }
                if (ep.align >= 4 * (int)sizeof(T) && j + 4 <= ep.n) {
                    finish_gated<T>(z, y, ep, i, j);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j + e < ep.n) finish_gated1<T>(z[e], y[e], ep, i, j + e);
                }
            }
        } else if (r < rows_a && 4 * c4 < rows_w) {
            const int64_t i = m0 + r, j = n0 + 4 * c4;
            float b[4];
            load_bias(ep, j, b);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] += b[e];
            if (ep.align >= 4 * (int)sizeof(T) && j + 4 <= ep.n) {
                float add[4];
                load_residual<T>(ep, i, j, add);
                finish<T>(z, add, ep, i, j);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < ep.n) finish1<T>(z[e], load_residual1<T>(ep, i, j + e), ep, i, j + e);
            }
        }
    }
}

// Between a few rows and many: 64 FA x 64 FB tiles through LDS. Four waves multiply, each
// 32 FA x 32 FB on the 32 x 32 x 64 scaled instruction (layouts as the 256 x 256 kernel:
// swapped operands, chunk c of staged row r at slot c ^ swz8(r)); they move the codes of
// the 256-k stages straight into LDS, N - 1 stages ahead of the one multiplied, waiting only
// for the oldest. A fifth wave brings the scales, whose layout (packed, or MX rows of any
// length and alignment) needs them in registers on the way: eight bytes per row and stage,
// even blocks first, zero past k. One barrier a stage.
//
// Why: the 256 x 256 kernel takes as long for one tile as for one on every compute unit
// (22 us at k = 4096), so products of fewer tiles than that are faster in smaller ones.
// Bound by the lines in flight: a compute unit takes in about 55 GB/s whatever N is (128 x 4096
// x 4096 8.3 us; two sets of waves on halves of a stage, or scales asked for 8 stages ahead, are
// level).
//
// With GatedEpi (FB = 2) half of the staged rows of W are the first weight's and half the second's, and each wave
// multiplies one fragment of both, so that both sums of an output are the same lane's. One token of n = 11008, k = 4096
// takes 11.4 us so (47.9 MB of weights, 4.2 TB/s), 256 rows 32.2 with four stages and 26.6 with two.
template <class T, int FA, int FB, int N, class E>
__global__ __launch_bounds__(320, 3) void tile_kernel(const uint8_t *__restrict__ ca, const uint8_t *__restrict__ sa,
                                                   const uint8_t *__restrict__ cw, const uint8_t *__restrict__ sw,
                                                   int packed, Geom g, E ep) {
    constexpr int TM = 64 * FA, TN = 64 * FB, kRowsAll = TM + TN;
    constexpr bool GATED = kGated<E>;
    static_assert(!GATED || FB == 2, "64 rows of each weight");
    constexpr int TC = GATED ? TN / 2 : TN;  // columns of the output
    constexpr int kOffScl = kRowsAll * 128, kStage = kRowsAll * 136;
    constexpr int kLoads = kRowsAll / 32;  // code loads (8 rows each) per wave and stage
    static_assert(kLoads * (N - 2) <= 63 && N >= 2, "the wait counts at most 63 loads");
    static_assert(N * kStage >= TM * TN * 4, "the output is staged in the same LDS");
    __shared__ __attribute__((aligned(16))) uint8_t smem[N * kStage];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    // an XCD's workgroups take a run of tiles, walked in bands of kBand rows of tiles (kq_tileorder.hpp)
    constexpr int kBand = 4;
    const int u = g256::tile_work((int)blockIdx.x, g256::TileOrder{g.tiles_m * g.tiles_n, 0, 0, 0}).tile;
    const int band = u / (kBand * g.tiles_n), within = u % (kBand * g.tiles_n);
    const int band_rows = g.tiles_m - band * kBand < kBand ? g.tiles_m - band * kBand : kBand;
    const int tm = band * kBand + within % band_rows, tn = within / band_rows;
    const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TC;
    const int rows_a = (int)(ep.m - m0 < TM ? ep.m - m0 : TM), rows_w = (int)(ep.n - n0 < TC ? ep.n - n0 : TC);
    const uint8_t *cu = cw, *su = sw;
    if constexpr (GATED) cu = ep.cu, su = ep.su;

    if (w == 4) {
        // Rows lane + 64 i of the tile: A's first, then W's. A padding row takes the last row's
        // scales (its codes are zero and its outputs are not stored), so no load has a condition.
        constexpr int R = FA + FB;
        const uint8_t *at[R];
        int64_t step[R];  // packed: bytes from a stage to the next
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const bool is_a = i < FA;
            const int row = lane + 64 * (is_a ? i : GATED ? 0 : i - FA), last = (is_a ? rows_a : rows_w) - 1;
            const int64_t g_row = (is_a ? m0 : n0) + (row < last ? row : last);
            at[i] = (is_a ? sa : GATED && i > FA ? su : sw) + g_row * (packed ? 8 : g.kblocks);
            step[i] = 8 * (is_a ? ep.m : ep.n);
        }
        // this slot held stage s - N, whose reads ended before the barrier of stage s - N + 1
        auto publish = [&](int slot, const uint2 (&v)[R]) {
            uint8_t *to = smem + slot * kStage + kOffScl + 8 * lane;
#pragma unroll
            for (int i = 0; i < R; ++i) *reinterpret_cast<uint2 *>(to + 512 * i) = v[i];
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        };
        if (packed) {
            uint2 ring[4][R];
            auto fetch = [&](uint2 (&v)[R], int s) {
                const int sc = s < g.stages ? s : g.stages - 1;
#pragma unroll
                for (int i = 0; i < R; ++i) v[i] = *reinterpret_cast<const uint2 *>(at[i] + sc * step[i]);
            };
            if (g.stages > 0) {
#pragma unroll
                for (int q = 0; q < 4; ++q) fetch(ring[q], q);
            }
            for (int s0 = 0; s0 < g.stages; s0 += 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (s0 + q >= g.stages) break;
                    publish(q % N, ring[q]);
                    fetch(ring[q], s0 + q + 4);
                }
            }
        } else {
            // Four stages at a time: a row's 32 bytes of them lie in one cache line with nothing else that
            // the tile needs now (fetched eight at a time, the scales cost as many lines as the codes and
            // a product 1.5 x the time).
            struct Group {
                uint4 u[R][2];
            };
            Group now, next;
            auto fetch = [&](Group &v, int s0) {
                const int left = g.kblocks - 8 * s0;
                if (left >= 32) {
#pragma unroll
                    for (int i = 0; i < R; ++i) __builtin_memcpy(v.u[i], at[i] + 8 * s0, 32);
                } else {
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        uint64_t x[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            if (left >= 8 * q + 8) {
                                __builtin_memcpy(&x[q], at[i] + 8 * (s0 + q), 8);
                            } else {
                                for (int b = 8 * q; b < left; ++b) x[q] |= (uint64_t)at[i][8 * s0 + b] << (8 * (b - 8 * q));
                            }
                        }
                        __builtin_memcpy(v.u[i], x, 32);
                    }
                }
            };
            fetch(now, 0);
            fetch(next, 4);
            for (int s0 = 0; s0 < g.stages; s0 += 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (s0 + q >= g.stages) break;
                    uint2 v[R];
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const uint4 u = now.u[i][q >> 1];
                        const uint32_t x = q & 1 ? u.z : u.x, y = q & 1 ? u.w : u.y;
                        v[i] = make_uint2(__builtin_amdgcn_perm(y, x, 0x06040200u),
                                          __builtin_amdgcn_perm(y, x, 0x07050301u));
                    }
                    publish(q % N, v);
                }
                now = next;
                fetch(next, s0 + 8);
            }
        }
        static_assert(4 % N == 0, "a stage's slot is its place in a group of four, modulo N");
        asm volatile("s_barrier" ::: "memory");  // the one in front of the output's staging
        return;
    }

    const i32x4_t dca = sdesc(ca + m0 * g.kbytes, (uint32_t)(rows_a * g.kbytes));
    const i32x4_t dcw = sdesc(cw + n0 * g.kbytes, (uint32_t)(rows_w * g.kbytes));
    const i32x4_t dcu = sdesc(cu + n0 * g.kbytes, (uint32_t)(rows_w * g.kbytes));
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
    // load j of wave w: staged rows 8 (kLoads w + j) + lane / 8 (A's TM rows, then W's), slot lane % 8
    const int chunk[2] = {(lane & 7) ^ swz8(lane >> 3), (lane & 7) ^ swz8(8 + (lane >> 3))};
    uint32_t voff[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int r0 = 8 * (kLoads * w + j);
        const int row = (r0 < TM ? r0 : GATED && r0 >= TM + TC ? r0 - TM - TC : r0 - TM) + (lane >> 3);
        voff[j] = (uint32_t)(row * g.kbytes) + 16u * (uint32_t)chunk[j & 1];
    }
    // Past k (whole stages too): past the record count, zeros. The scalar offset stays below that count: 0 for the
    // stages past the last.
    auto issue = [&](int s, int slot) {
        const bool in[2] = {128 * s + 16 * chunk[0] < g.kbytes, 128 * s + 16 * chunk[1] < g.kbytes};
        const int kb = s < g.stages ? 128 * s : 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r0 = 8 * (kLoads * w + j);
            const uint32_t off = in[j & 1] ? voff[j] : 0x80000000u;
            i32x4_t dw = dcw;
            if (GATED) {
                dw.x = __builtin_amdgcn_readfirstlane(r0 >= TM + TC ? dcu.x : dcw.x);
                dw.y = __builtin_amdgcn_readfirstlane(r0 >= TM + TC ? dcu.y : dcw.y);
            }
            dma16(r0 < TM ? dca : dw, lds0 + (uint32_t)(slot * kStage + r0 * 128), off, (uint32_t)kb);
        }
    };
    const int r = lane & 31, hi = lane >> 5;
    const int wm = (w >> 1) * (TM / 2), wn = (w & 1) * (TC / 2);
    // staged row of W at which the wave's fragment b starts
    auto frag = [&](int b) { return wn + (GATED ? TC * b : 32 * b); };
    int rdo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) rdo[j] = r * 128 + 16 * ((2 * j + hi) ^ swz8(r & 15));

    floatx16_t acc[FA][FB];
#pragma unroll
    for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int b = 0; b < FB; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

#pragma unroll
    for (int i = 0; i < N - 1; ++i) issue(i, i);
    for (int s0 = 0; s0 < g.stages; s0 += N) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int s = s0 + i;
            if (s >= g.stages) break;
            // stage s has landed (the N - 2 younger ones may be in flight), and every wave is done
            // with stage s - 1, whose slot takes stage s + N - 1
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads * (N - 2)) : "memory");
            issue(s + N - 1, (i + N - 1) % N);
            const uint8_t *st = smem + i * kStage;
            uint32_t xa[FA], xw[FB];
#pragma unroll
            for (int a = 0; a < FA; ++a)
                xa[a] = *reinterpret_cast<const uint32_t *>(st + kOffScl + 8 * (wm + 32 * a + r) + 4 * hi);
#pragma unroll
            for (int b = 0; b < FB; ++b)
                xw[b] = *reinterpret_cast<const uint32_t *>(st + kOffScl + 8 * (TM + frag(b) + r) + 4 * hi);
            auto step = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                i32x8_t fa[FA], fw[FB];
#pragma unroll
                for (int a = 0; a < FA; ++a) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(st + (wm + 32 * a) * 128 + rdo[j]);
                    fa[a] = i32x8_t{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
                }
#pragma unroll
                for (int b = 0; b < FB; ++b) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(st + (TM + frag(b)) * 128 + rdo[j]);
                    fw[b] = i32x8_t{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
                }
#pragma unroll
                for (int a = 0; a < FA; ++a)
#pragma unroll
                    for (int b = 0; b < FB; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fw[b], fa[a], acc[a][b], 4, 4, j,
                                                                                    (int)xw[b], j, (int)xa[a]);
            };
            step(std::integral_constant<int, 0>());
            step(std::integral_constant<int, 1>());
            step(std::integral_constant<int, 2>());
            step(std::integral_constant<int, 3>());
        }
    }

    constexpr int WM = TM / 2, WN = TN / 2, CH = WN / 4;
    Bias<T, WM, WN> bias;
    Residual<T, WM, WN> add;
    if constexpr (!GATED) {
        bias.load(ep, n0 + wn);
        add.load(ep, m0 + wm, rows_a - wm, n0 + wn, 0);
    }
    // every load into LDS has landed (the ones past k too) and every wave is done with the stages
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    // Each wave stages its block in fp32 in its own region, rows of 32 FB columns with 16-byte chunk c
    // at c ^ (row % CH), and reads it back row by row.
    uint8_t *reg = smem + w * (WM * WN * 4);
#pragma unroll
    for (int a = 0; a < FA; ++a)
#pragma unroll
        for (int b = 0; b < FB; ++b)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = 32 * a + r, c = 8 * b + 2 * q + hi;
                *reinterpret_cast<floatx4_t *>(reg + row * (WN * 4) + 16 * (c ^ (row & (CH - 1)))) =
                    floatx4_t{acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
            }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if constexpr (GATED) finish_gated_staged<T, WM>(reg, ep, m0 + wm, rows_a - wm, n0 + wn);
    else finish_staged(reg, ep, m0 + wm, rows_a - wm, n0 + wn, bias, add);
}

// Backward of the epilogue: wave w of workgroup (x, p) takes 512
// columns (8 per lane: 1 KB of a bf16 row) of every fourth of the p-th `group_rows` rows, U of
// them in flight; the waves' column sums meet in LDS in wave order. Bound by HBM: two reads and a
// write per element against about 25 vector operations of 39 T/s for gelu_tanh (131 us without
// an activation too at 8192 x 16384 bf16: 6.1 TB/s; with every parts-th row instead 140). gelu has
// more operations than fit under that: 142.
template <class T, bool NT, bool VEC>
__global__ __launch_bounds__(256) void backward_kernel(const T *__restrict__ dO, int64_t lddo,
                                                       const T *__restrict__ Z, int64_t ldz, int64_t m, int64_t n,
                                                       int act, T *__restrict__ dZ, int64_t lddz, int64_t group_rows,
                                                       float *__restrict__ part) {
    // element by element, rows past the last cost their loads' issue (us, bf16 silu with 8 and 4: 1000 x
    // 4001 19.9, 14.8; 301 x 4607 10.5, 8.3; 8192 x 4609 58, 60)
    constexpr int U = VEC ? 8 : 4;
    __shared__ float4 join[4][2][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)blockIdx.x * 512, left = n - c0 < 512 ? n - c0 : 512;
    const int64_t bytes = left * (int)sizeof(T);
    const uint32_t ch = Lanes<VEC>::first(0, lane);
    const int p = (int)blockIdx.y;
    const bool reads_z = act != KQ_ACT_NONE;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int64_t end = m - p * group_rows < group_rows ? m : (p + 1) * group_rows;
    for (int64_t i = p * group_rows + wave; i < end; i += 4 * U) {
        Chunk<T, VEC> d[U], z[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = i + 4 * u;
            const bool in = row < end;
            d[u].template load<NT>(row_rsrc(dO + (in ? row : i) * lddo + c0, in ? bytes : 0), ch);
            if (reads_z) z[u].template load<NT>(row_rsrc(Z + (in ? row : i) * ldz + c0, in ? bytes : 0), ch);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = i + 4 * u;
            if (row >= end) break;
            float v[8], x[8];
            d[u].widen(v);
            if (reads_z) {
                z[u].widen(x);
                activate_grad(v, x, act);
            }
            if (dZ) store8<NT, VEC>(row_rsrc(dZ + row * lddz + c0, bytes), ch, v, dZ);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += v[e];
        }
    }
    if (!part) return;
    join[wave][0][lane] = make_float4(s[0], s[1], s[2], s[3]);
    join[wave][1][lane] = make_float4(s[4], s[5], s[6], s[7]);
    __syncthreads();
    if (wave < 2) {
        float4 a = join[0][wave][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 o = join[w][wave][lane];
            a.x += o.x; a.y += o.y; a.z += o.z; a.w += o.w;
        }
        const int64_t c = c0 + ch + 4 * wave * Lanes<VEC>::kStep;
        if (VEC) {
            if (c < n) *reinterpret_cast<float4 *>(part + p * n + c) = a;
        } else {
            const float one[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c + 64 * e < n) part[p * n + c + 64 * e] = one[e];
        }
    }
}

// V neighbouring elements, one or whole 16 bytes of them.
template <class T, int V>
__device__ __forceinline__ void load_some(const T *p, float (&x)[V]) {
    if constexpr (V > 1) load_piece(p, x);
    else if constexpr (sizeof(T) == 2) x[0] = bf16_lo(*p);
    else x[0] = *p;
}
template <class T, int V>
__device__ __forceinline__ void store_some(T *p, const float (&x)[V]) {
    if constexpr (V == 1) store1(p, x[0]);
    else if constexpr (sizeof(T) == 4) *reinterpret_cast<floatx4_t *>(p) = floatx4_t{x[0], x[1], x[2], x[3]};
    else *reinterpret_cast<u32x4_t *>(p) = u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
}

// Backward of the gated epilogue, as backward_kernel: three reads and two writes per element, and both biases' sums.
// The outputs may be inputs: a lane has read an element of each before it writes any.
// 8192 x 11008 bf16 silu 158 us (902 MB, 5.7 TB/s) and 6 for the sums of 256 parts.
template <class T, bool NT, bool VEC>
__global__ __launch_bounds__(256) void gated_backward_kernel(const T *dO, int64_t lddo,
                                                             const T *G, int64_t ldg,
                                                             const T *U, int64_t ldu, int64_t m, int64_t n,
                                                             int act, T *dG, int64_t lddg,
                                                             T *dU, int64_t lddu, int64_t group_rows,
                                                             float *__restrict__ part_g, float *__restrict__ part_u) {
    constexpr int R = 4;  // rows in flight per wave
    __shared__ float4 join[4][4][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)blockIdx.x * 512, left = n - c0 < 512 ? n - c0 : 512;
    const int64_t bytes = left * (int)sizeof(T);
    const uint32_t ch = Lanes<VEC>::first(0, lane);
    const int p = (int)blockIdx.y;
    float s[2][8] = {};
    const int64_t end = m - p * group_rows < group_rows ? m : (p + 1) * group_rows;
    for (int64_t i = p * group_rows + wave; i < end; i += 4 * R) {
        Chunk<T, VEC> d[R], g[R], u[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = i + 4 * k < end ? i + 4 * k : i, some = i + 4 * k < end ? bytes : 0;
            d[k].template load<NT>(row_rsrc(dO + row * lddo + c0, some), ch);
            g[k].template load<NT>(row_rsrc(G + row * ldg + c0, some), ch);
            u[k].template load<NT>(row_rsrc(U + row * ldu + c0, some), ch);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t row = i + 4 * k;
            if (row >= end) break;
            float v[8], x[8], y[8];
            d[k].widen(v);
            g[k].widen(x);
            u[k].widen(y);
            activate_gated_grad(v, y, x, act);
            if (dG) store8<NT, VEC>(row_rsrc(dG + row * lddg + c0, bytes), ch, v, dG);
            if (dU) store8<NT, VEC>(row_rsrc(dU + row * lddu + c0, bytes), ch, y, dU);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0][e] += v[e];
                s[1][e] += y[e];
            }
        }
    }
    if (!part_g && !part_u) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        join[wave][2 * k][lane] = make_float4(s[k][0], s[k][1], s[k][2], s[k][3]);
        join[wave][2 * k + 1][lane] = make_float4(s[k][4], s[k][5], s[k][6], s[k][7]);
    }
    __syncthreads();
    // wave w: half w % 2 of the columns of the gate's (w < 2) or the other's sums
    float *part = wave < 2 ? part_g : part_u;
    if (!part) return;
    float4 a = join[0][wave][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
        const float4 o = join[w][wave][lane];
        a.x += o.x; a.y += o.y; a.z += o.z; a.w += o.w;
    }
    const int64_t c = c0 + ch + 4 * (wave & 1) * Lanes<VEC>::kStep;
    if (VEC) {
        if (c < n) *reinterpret_cast<float4 *>(part + p * n + c) = a;
    } else {
        const float one[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (c + 64 * e < n) part[p * n + c + 64 * e] = one[e];
    }
}

// The same for few rows: a workgroup owns all rows of 32 columns, so that the sums need no second launch (nor partial sums):
// V neighbouring columns a lane, the rows dealt to the lanes' groups in turn, the waves joined in their order. Bound by the
// latency of its few loads and, with more rows, by what a compute unit takes in: 64 x 4608 bf16 3.5 us, 301 x 4607 fp32, element
// by element, 10.4 (27.7 MB, 2.7 TB/s on 144 of 256 compute units).
template <class T, int V, int THREADS>
__global__ __launch_bounds__(THREADS) void gated_strip_kernel(const T *dO, int64_t lddo, const T *G, int64_t ldg, const T *U,
                                                              int64_t ldu, int64_t m, int64_t n, int act, T *dG, int64_t lddg,
                                                              T *dU, int64_t lddu, float *__restrict__ dbias_g,
                                                              float *__restrict__ dbias_u) {
    constexpr int C = 32, LR = C / V, step = THREADS / LR, K = 4, kWaves = THREADS / 64;
    __shared__ float join[2][kWaves][C];
    const int tid = threadIdx.x, c = tid % LR * V;
    const int64_t col = (int64_t)blockIdx.x * C + c;
    const bool in = col < n;
    float s[2][V] = {};
    for (int64_t i = tid / LR; in && i < m; i += K * step) {
        float d[K][V], z[K][V], u[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t row = i + k * step < m ? i + k * step : i;
            load_some(dO + row * lddo + col, d[k]);
            load_some(G + row * ldg + col, z[k]);
            load_some(U + row * ldu + col, u[k]);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t row = i + k * step;
            if (row >= m) break;
            activate_gated_grad(d[k], u[k], z[k], act);
            if (dG) store_some(dG + row * lddg + col, d[k]);
            if (dU) store_some(dU + row * lddu + col, u[k]);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                s[0][e] += d[k][e];
                s[1][e] += u[k][e];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float v = slots_sum<LR>(s[k][e]);
            if (tid % 64 < LR) join[k][tid / 64][c + e] = v;
        }
    __syncthreads();
    if (tid >= 2 * C) return;
    const int k = tid / C, j = tid % C;
    float *out = k ? dbias_u : dbias_g;
    if (!out || (int64_t)blockIdx.x * C + j >= n) return;
    float v = join[k][0][j];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += join[k][w][j];
    out[(int64_t)blockIdx.x * C + j] = v;
}

}  // namespace linear
}  // namespace kq

// ===========================================================================
// Host side
// ===========================================================================
namespace kqhost {
kq_status gemm256_linear(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_w,
                         const uint8_t *scales_w, int packed, int64_t k, int type, const kq::Epi &ep,
                         kq_stream_t stream);  // kq_gemm256.hip
kq_status gated256_bf16(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_g, const uint8_t *scales_g,
                        int packed, int64_t k, const kq::GatedEpi &ep, kq_stream_t stream);  // kq_gated256_bf16.hip
kq_status gated256_f32(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_g, const uint8_t *scales_g,
                       int packed, int64_t k, const kq::GatedEpi &ep, kq_stream_t stream);  // kq_gated256_f32.hip
}

namespace {

using kqhost::aligned;
using kqhost::launched;
using kqhost::sizes_fit;

bool good_type(int type) { return type == KQ_F32 || type == KQ_BF16; }
bool good_act(int act) { return act >= KQ_ACT_NONE && act <= KQ_ACT_GELU_TANH; }

// Parts of the bias gradient's sum: those of m rows, at most as many as give 8192 workgroups of
// 512 columns; none of no columns.
int64_t column_parts(int64_t m, int64_t n) {
    if (n == 0) return 0;
    const int64_t strips = (n + 511) / 512, most = 8192 / (strips < 128 ? strips : 128), p = kqhost::row_parts(m);
    return p < most ? p : most;
}

template <class T>
void launch_backward(const void *dO, int64_t lddo, const void *Z, int64_t ldz, int64_t m, int64_t n, int act, void *dZ,
                     int64_t lddz, int64_t parts, float *part, bool vec, kq_stream_t stream) {
    const int64_t rows = (m + parts - 1) / parts;
    const dim3 grid((unsigned)((n + 511) / 512), (unsigned)parts);
    auto go = [&](auto NT, auto VEC) {
        hipLaunchKernelGGL((kq::linear::backward_kernel<T, NT(), VEC()>), grid, dim3(256), 0, (hipStream_t)stream,
                           (const T *)dO, lddo, (const T *)Z, ldz, m, n, act, (T *)dZ, lddz, rows, part);
    };
    const bool nt = kq::streamed_once(3 * m * n * (int)sizeof(T));
    if (vec && nt) go(std::true_type(), std::true_type());
    else if (vec) go(std::false_type(), std::true_type());
    else if (nt) go(std::true_type(), std::false_type());
    else go(std::false_type(), std::false_type());
}

// The launch's work-items are counted in 32 bits.
bool groups_fit(int64_t groups, int threads) { return groups <= (int64_t)0xFFFFFFFF / threads; }

template <class T, int SC, int MF, int NF, int WK, int D, class E>
kq_status launch_product(const uint8_t *ca, const uint8_t *sa, const uint8_t *cw, const uint8_t *sw,
                         kq::linear::Geom g, const E &ep, kq_stream_t stream) {
    const int64_t tiles_m = (ep.m + 16 * MF - 1) / (16 * MF), tiles_n = (ep.n + 16 * NF - 1) / (16 * NF);
    g.tiles_n = (int)tiles_n;
    if (!groups_fit(tiles_m * tiles_n, 64 * WK)) return KQ_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((kq::linear::product_kernel<T, SC, MF, NF, WK, D, E>), dim3((unsigned)(tiles_m * tiles_n)),
                       dim3(64 * WK), 0, (hipStream_t)stream, ca, sa, cw, sw, g, ep);
    return launched();
}

template <class T, int FA, int FB, int N, class E>
kq_status launch_tiles(const uint8_t *ca, const uint8_t *sa, const uint8_t *cw, const uint8_t *sw, int packed,
                       kq::linear::Geom g, const E &ep, kq_stream_t stream) {
    constexpr int cols = kq::linear::kGated<E> ? 32 * FB : 64 * FB;
    const int64_t tiles_m = (ep.m + 64 * FA - 1) / (64 * FA), tiles_n = (ep.n + cols - 1) / cols;
    g.tiles_n = (int)tiles_n;
    g.tiles_m = (int)tiles_m;
    if (!groups_fit(tiles_m * tiles_n, 320)) return KQ_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((kq::linear::tile_kernel<T, FA, FB, N, E>), dim3((unsigned)(tiles_m * tiles_n)), dim3(320), 0,
                       (hipStream_t)stream, ca, sa, cw, sw, packed, g, ep);
    return launched();
}

using kq::linear::Kernel;
using kq::linear::kProduct11;
using kq::linear::kProduct12;
using kq::linear::kProduct22;
using kq::linear::kTile256;
using kq::linear::kTile64;
using kq::linear::kTile64Deep;

template <class T, int MF, int NF, int WK, class E>
kq_status launch_any_product(const uint8_t *ca, const uint8_t *sa, const uint8_t *cw, const uint8_t *sw, int packed,
                             const kq::linear::Geom &g, const E &ep, kq_stream_t stream) {
    if (packed) return launch_product<T, kq::linear::kPacked8, MF, NF, WK, 1, E>(ca, sa, cw, sw, g, ep, stream);
    bool rows8 = g.kblocks % 8 == 0 && aligned(sa, 8) && aligned(sw, 8);
    if constexpr (kq::linear::kGated<E>) rows8 = rows8 && aligned(ep.su, 8);
    if (rows8)
        return launch_product<T, kq::linear::kRows8, MF, NF, WK, 1, E>(ca, sa, cw, sw, g, ep, stream);
    return launch_product<T, kq::linear::kBytes, MF, NF, WK, 1, E>(ca, sa, cw, sw, g, ep, stream);
}

template <class T>
kq_status launch_linear(Kernel k, const uint8_t *ca, const uint8_t *sa, const uint8_t *cw, const uint8_t *sw,
                        int packed, const kq::linear::Geom &g, const kq::Epi &ep, kq_stream_t stream) {
    switch (k) {
        case kProduct11: return launch_any_product<T, 1, 1, 8>(ca, sa, cw, sw, packed, g, ep, stream);
        case kProduct12: return launch_any_product<T, 1, 2, 4>(ca, sa, cw, sw, packed, g, ep, stream);
        case kProduct22: return launch_any_product<T, 2, 2, 4>(ca, sa, cw, sw, packed, g, ep, stream);
        case kTile64Deep: return launch_tiles<T, 1, 1, 4>(ca, sa, cw, sw, packed, g, ep, stream);
        case kTile64: return launch_tiles<T, 1, 1, 2>(ca, sa, cw, sw, packed, g, ep, stream);
        default: return launch_tiles<T, 2, 2, 2>(ca, sa, cw, sw, packed, g, ep, stream);
    }
}

using kq::linear::GatedKernel;
using kq::linear::kGatedProduct1;
using kq::linear::kGatedProduct2;
using kq::linear::kGatedTile256;
using kq::linear::kGatedTile64;
using kq::linear::kGatedTile64Deep;

template <class T>
kq_status launch_gated(GatedKernel k, const uint8_t *ca, const uint8_t *sa, const uint8_t *cg, const uint8_t *sg,
                       int packed, const kq::linear::Geom &g, const kq::GatedEpi &ep, kq_stream_t stream) {
    switch (k) {
        case kGatedProduct1: return launch_any_product<T, 1, 1, 4>(ca, sa, cg, sg, packed, g, ep, stream);
        case kGatedProduct2: return launch_any_product<T, 2, 1, 4>(ca, sa, cg, sg, packed, g, ep, stream);
        case kGatedTile64Deep: return launch_tiles<T, 1, 2, 4>(ca, sa, cg, sg, packed, g, ep, stream);
        case kGatedTile64: return launch_tiles<T, 1, 2, 2>(ca, sa, cg, sg, packed, g, ep, stream);
        default: return launch_tiles<T, 2, 2, 2>(ca, sa, cg, sg, packed, g, ep, stream);
    }
}

// Rows up to which the gated gradients are taken in strips of columns, in one launch, by rows and by strips (us, both biases,
// silu):
//   bf16                       64        128        256        384        512         1024 rows
//     4608 columns        5.6 3.5    6.5 4.0    8.2 6.6    9.8 8.6  11.4 10.5    15.4 16.7
//     11008               7.4 4.3    9.2 7.3  12.6 10.6  15.7 14.6
//     28672              12.1 8.7  15.6 13.2  23.1 21.5  32.9 38.0      42 50
//   fp32, by element
//     4607                6.3 3.9    8.2 5.7   11.0 8.7  13.0 11.7
//     11009               9.3 6.4   12.1 9.7  17.9 17.2  23.3 25.3      32 42
// One number for all of them, so that the workspace's size is a function of the sizes alone: at 257 to 384 rows of the
// widest ones the strips are up to 15% slower. 256 threads for 16-byte pieces (1024: 301 x 28672 25.5 and 34.9), 1024 for
// elements (256: 301 x 4607 9.0 and 16.7).
constexpr int64_t kStripRows = 384;
bool in_strips(int64_t m, int64_t n) { return m <= kStripRows && groups_fit((n + 31) / 32, 1024); }

template <class T>
void launch_gated_strips(const void *dO, int64_t lddo, const void *G, int64_t ldg, const void *U, int64_t ldu, int64_t m,
                         int64_t n, int act, void *dG, int64_t lddg, void *dU, int64_t lddu, float *dbias_g,
                         float *dbias_u, bool vec, kq_stream_t stream) {
    auto go = [&](auto V, auto THREADS) {
        hipLaunchKernelGGL((kq::linear::gated_strip_kernel<T, V(), THREADS()>), dim3((unsigned)((n + 31) / 32)),
                           dim3(THREADS()), 0, (hipStream_t)stream, (const T *)dO, lddo, (const T *)G, ldg, (const T *)U,
                           ldu, m, n, act, (T *)dG, lddg, (T *)dU, lddu, dbias_g, dbias_u);
    };
    if (vec) go(std::integral_constant<int, 16 / (int)sizeof(T)>(), std::integral_constant<int, 256>());
    else go(std::integral_constant<int, 1>(), std::integral_constant<int, 1024>());
}

template <class T>
void launch_gated_backward(const void *dO, int64_t lddo, const void *G, int64_t ldg, const void *U, int64_t ldu, int64_t m,
                           int64_t n, int act, void *dG, int64_t lddg, void *dU, int64_t lddu, int64_t parts,
                           float *part_g, float *part_u, bool vec, kq_stream_t stream) {
    const int64_t rows = (m + parts - 1) / parts;
    const dim3 grid((unsigned)((n + 511) / 512), (unsigned)parts);
    auto go = [&](auto NT, auto VEC) {
        hipLaunchKernelGGL((kq::linear::gated_backward_kernel<T, NT(), VEC()>), grid, dim3(256), 0, (hipStream_t)stream,
                           (const T *)dO, lddo, (const T *)G, ldg, (const T *)U, ldu, m, n, act, (T *)dG, lddg, (T *)dU,
                           lddu, rows, part_g, part_u);
    };
    const bool nt = kq::streamed_once(5 * m * n * (int)sizeof(T));
    if (vec && nt) go(std::true_type(), std::true_type());
    else if (vec) go(std::false_type(), std::true_type());
    else if (nt) go(std::true_type(), std::false_type());
    else go(std::false_type(), std::false_type());
}

}  // namespace

extern "C" {

kq_status kq_mxfp4_linear(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_w,
                          const uint8_t *scales_w, int packed, int64_t m, int64_t n, int64_t k, const float *bias,
                          int act, int type, const void *residual, int64_t ldr, void *O, int64_t ldo, void *Z,
                          int64_t ldz, kq_stream_t stream) {
    if (m < 0 || n < 0 || k < 0 || k % 32 != 0 || (packed && k % 256 != 0) || ldo < n || (residual && ldr < n) ||
        (Z && ldz < n))
        return KQ_ERR_SHAPE;
    if (!residual) ldr = 0;
    if (!Z) ldz = 0;
    if (!good_type(type) || !good_act(act) || !sizes_fit({m, n, k, ldr, ldo, ldz})) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return KQ_OK;
    if (!O || (k > 0 && (!codes_a || !scales_a || !codes_w || !scales_w))) return KQ_ERR_NULL;
    const int es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(codes_a, 16) || !aligned(codes_w, 16) || (packed && (!aligned(scales_a, 8) || !aligned(scales_w, 8))) ||
        !aligned(bias, 4) || !aligned(residual, es) || !aligned(O, es) || !aligned(Z, es))
        return KQ_ERR_ALIGN;
    // buffer record counts and offsets are 32-bit
    const int64_t lim = (int64_t)1 << 31;
    if (256 * (k / 2) >= lim || m * (k / 32) >= lim || n * (k / 32) >= lim || (255 * ldo + n) * es >= lim ||
        (255 * ldr + n) * es >= lim || (255 * ldz + n) * es >= lim)
        return KQ_ERR_UNSUPPORTED;
    kq::Epi ep{bias, residual, O, Z, m, n, ldr, ldo, ldz, act, 16, m * n * es >= (int64_t)256 << 20};
    while (ep.align > es && (!aligned(O, ep.align) || !aligned(residual, ep.align) || !aligned(Z, ep.align) ||
                             ((ldo | ldr | ldz) * es) % ep.align != 0))
        ep.align /= 2;
    const kq::linear::Geom g{(int)(k / 2), (int)(k / 32), (int)((k + 255) / 256), 0, 0};
    // without scales their layout does not matter, and the packed record counts (stages 8 m - 8 m0) would
    // be below zero, so past every guard, for all tiles but the first
    if (k == 0) packed = 0;
    const bool big = k > 0 && (packed ? aligned(scales_a, 16) && aligned(scales_w, 16)
                                      : k % 128 == 0 && aligned(scales_a, 4) && aligned(scales_w, 4));
    const Kernel kernel = kq::linear::choose_kernel(m, n, g.stages, packed != 0, big, kqhost::compute_units());
    if (kernel == kTile256)
        return kqhost::gemm256_linear(codes_a, scales_a, codes_w, scales_w, packed, k, type, ep, stream);
    return type == KQ_BF16
               ? launch_linear<uint16_t>(kernel, codes_a, scales_a, codes_w, scales_w, packed, g, ep, stream)
               : launch_linear<float>(kernel, codes_a, scales_a, codes_w, scales_w, packed, g, ep, stream);
}

kq_status kq_mxfp4_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t *bytes) {
    if (!bytes) return KQ_ERR_NULL;
    *bytes = 0;
    if (m < 0 || n < 0) return KQ_ERR_SHAPE;
    if (!sizes_fit({m, n})) return KQ_ERR_UNSUPPORTED;
    const int64_t parts = column_parts(m, n);
    if (parts > 1) *bytes = parts * n * 4;
    return KQ_OK;
}

kq_status kq_mxfp4_linear_backward(const void *dO, int64_t lddo, const void *Z, int64_t ldz, int type, int64_t m,
                                   int64_t n, int act, void *dZ, int64_t lddz, float *dbias, void *workspace,
                                   int64_t workspace_bytes, kq_stream_t stream) {
    const bool reads_z = act != KQ_ACT_NONE;
    if (m < 0 || n < 0 || lddo < n || (reads_z && ldz < n) || (dZ && lddz < n)) return KQ_ERR_SHAPE;
    if (!reads_z) ldz = 0;
    if (!dZ) lddz = 0;
    if (!good_type(type) || !good_act(act) || !sizes_fit({m, n, lddo, ldz, lddz})) return KQ_ERR_UNSUPPORTED;
    if (n == 0) return KQ_OK;
    if (!aligned(dbias, 4)) return KQ_ERR_ALIGN;
    if (m == 0) return dbias ? kqhost::reduce_parts(nullptr, nullptr, 0, n, dbias, nullptr, stream) : KQ_OK;
    if (!dO || (reads_z && !Z) || (!dZ && !dbias)) return KQ_ERR_NULL;
    const uintptr_t es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(dO, es) || (reads_z && !aligned(Z, es)) || !aligned(dZ, es)) return KQ_ERR_ALIGN;
    const int64_t parts = column_parts(m, n);
    float *part = dbias;
    if (dbias && parts > 1) {
        if (!workspace) return KQ_ERR_NULL;
        if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
        if (workspace_bytes < parts * n * 4) return KQ_ERR_SHAPE;
        part = static_cast<float *>(workspace);
    }
    const int64_t per16 = 16 / es;
    const bool vec = n % 8 == 0 && aligned(dO, 16) && lddo % per16 == 0 && (!reads_z || (aligned(Z, 16) && ldz % per16 == 0)) &&
                     aligned(dZ, 16) && lddz % per16 == 0 && aligned(part, 16);
    if (type == KQ_BF16) launch_backward<uint16_t>(dO, lddo, Z, ldz, m, n, act, dZ, lddz, parts, part, vec, stream);
    else launch_backward<float>(dO, lddo, Z, ldz, m, n, act, dZ, lddz, parts, part, vec, stream);
    const kq_status s = launched();
    if (s != KQ_OK) return s;
    if (dbias && parts > 1) return kqhost::reduce_parts(part, nullptr, parts, n, dbias, nullptr, stream);
    return KQ_OK;
}

kq_status kq_mxfp4_gated_linear(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_g,
                                const uint8_t *scales_g, const uint8_t *codes_u, const uint8_t *scales_u, int packed,
                                int64_t m, int64_t n, int64_t k, const float *bias_g, const float *bias_u, int act,
                                int type, void *O, int64_t ldo, void *G, int64_t ldg, void *U, int64_t ldu,
                                kq_stream_t stream) {
    if (m < 0 || n < 0 || k < 0 || k % 32 != 0 || (packed && k % 256 != 0) || ldo < n || (G && ldg < n) || (U && ldu < n))
        return KQ_ERR_SHAPE;
    if (!G) ldg = 0;
    if (!U) ldu = 0;
    if (!good_type(type) || !good_act(act) || !sizes_fit({m, n, k, ldo, ldg, ldu})) return KQ_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return KQ_OK;
    if (!O || (k > 0 && (!codes_a || !scales_a || !codes_g || !scales_g || !codes_u || !scales_u))) return KQ_ERR_NULL;
    const int es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(codes_a, 16) || !aligned(codes_g, 16) || !aligned(codes_u, 16) ||
        (packed && (!aligned(scales_a, 8) || !aligned(scales_g, 8) || !aligned(scales_u, 8))) || !aligned(bias_g, 4) ||
        !aligned(bias_u, 4) || !aligned(O, es) || !aligned(G, es) || !aligned(U, es))
        return KQ_ERR_ALIGN;
    // buffer record counts and offsets are 32-bit
    const int64_t lim = (int64_t)1 << 31;
    if (256 * (k / 2) >= lim || m * (k / 32) >= lim || n * (k / 32) >= lim || (255 * ldo + n) * es >= lim ||
        (255 * ldg + n) * es >= lim || (255 * ldu + n) * es >= lim)
        return KQ_ERR_UNSUPPORTED;
    kq::GatedEpi ep{bias_g, bias_u, O, G, U, m, n, ldo, ldg, ldu, act, 16, codes_u, scales_u};
    while (ep.align > es && (!aligned(O, ep.align) || !aligned(G, ep.align) || !aligned(U, ep.align) ||
                             ((ldo | ldg | ldu) * es) % ep.align != 0))
        ep.align /= 2;
    const kq::linear::Geom g{(int)(k / 2), (int)(k / 32), (int)((k + 255) / 256), 0, 0};
    if (k == 0) packed = 0;  // as kq_mxfp4_linear
    const int s_align = packed ? 16 : 4;
    const bool big = k > 256 && (packed || k % 128 == 0) && aligned(scales_a, s_align) && aligned(scales_g, s_align) &&
                     aligned(scales_u, s_align);
    const GatedKernel kernel = kq::linear::choose_gated_kernel(m, n, g.stages, packed != 0, big, kqhost::compute_units());
    if (kernel == kGatedTile256)
        return type == KQ_BF16 ? kqhost::gated256_bf16(codes_a, scales_a, codes_g, scales_g, packed, k, ep, stream)
                               : kqhost::gated256_f32(codes_a, scales_a, codes_g, scales_g, packed, k, ep, stream);
    return type == KQ_BF16 ? launch_gated<uint16_t>(kernel, codes_a, scales_a, codes_g, scales_g, packed, g, ep, stream)
                           : launch_gated<float>(kernel, codes_a, scales_a, codes_g, scales_g, packed, g, ep, stream);
}

kq_status kq_mxfp4_gated_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t *bytes) {
    if (!bytes) return KQ_ERR_NULL;
    *bytes = 0;
    if (m < 0 || n < 0) return KQ_ERR_SHAPE;
    if (!sizes_fit({m, n})) return KQ_ERR_UNSUPPORTED;
    const int64_t parts = column_parts(m, n);
    if (!in_strips(m, n)) *bytes = parts > 1 ? parts * 2 * n * 4 : 0;
    return KQ_OK;
}

kq_status kq_mxfp4_gated_linear_backward(const void *dO, int64_t lddo, const void *G, int64_t ldg, const void *U,
                                         int64_t ldu, int type, int64_t m, int64_t n, int act, void *dG, int64_t lddg,
                                         void *dU, int64_t lddu, float *dbias_g, float *dbias_u, void *workspace,
                                         int64_t workspace_bytes, kq_stream_t stream) {
    if (m < 0 || n < 0 || lddo < n || ldg < n || ldu < n || (dG && lddg < n) || (dU && lddu < n)) return KQ_ERR_SHAPE;
    if (!dG) lddg = 0;
    if (!dU) lddu = 0;
    if (!good_type(type) || !good_act(act) || !sizes_fit({m, n, lddo, ldg, ldu, lddg, lddu})) return KQ_ERR_UNSUPPORTED;
    if (n == 0) return KQ_OK;
    if (!aligned(dbias_g, 4) || !aligned(dbias_u, 4)) return KQ_ERR_ALIGN;
    const bool sums = dbias_g || dbias_u;
    if (m == 0) return sums ? kqhost::reduce_parts(nullptr, nullptr, 0, n, dbias_g, dbias_u, stream) : KQ_OK;
    if (!dO || !G || !U || (!dG && !dU && !sums)) return KQ_ERR_NULL;
    const uintptr_t es = type == KQ_BF16 ? 2 : 4;
    if (!aligned(dO, es) || !aligned(G, es) || !aligned(U, es) || !aligned(dG, es) || !aligned(dU, es)) return KQ_ERR_ALIGN;
    const int64_t per16 = 16 / es;
    bool vec = n % 8 == 0 && aligned(dO, 16) && aligned(G, 16) && aligned(U, 16) && aligned(dG, 16) && aligned(dU, 16) &&
               (lddo | ldg | ldu | lddg | lddu) % per16 == 0;
    if (sums && in_strips(m, n)) {
        if (type == KQ_BF16)
            launch_gated_strips<uint16_t>(dO, lddo, G, ldg, U, ldu, m, n, act, dG, lddg, dU, lddu, dbias_g, dbias_u, vec, stream);
        else
            launch_gated_strips<float>(dO, lddo, G, ldg, U, ldu, m, n, act, dG, lddg, dU, lddu, dbias_g, dbias_u, vec, stream);
        return launched();
    }
    const int64_t parts = column_parts(m, n);
    float *part_g = dbias_g, *part_u = dbias_u;
    if (sums && parts > 1) {
        if (!workspace) return KQ_ERR_NULL;
        if (!aligned(workspace, 16)) return KQ_ERR_ALIGN;
        if (workspace_bytes < parts * 2 * n * 4) return KQ_ERR_SHAPE;
        part_g = static_cast<float *>(workspace);
        part_u = part_g + parts * n;
    }
    vec = vec && aligned(part_g, 16) && aligned(part_u, 16);
    if (type == KQ_BF16)
        launch_gated_backward<uint16_t>(dO, lddo, G, ldg, U, ldu, m, n, act, dG, lddg, dU, lddu, parts, part_g, part_u, vec, stream);
    else
        launch_gated_backward<float>(dO, lddo, G, ldg, U, ldu, m, n, act, dG, lddg, dU, lddu, parts, part_g, part_u, vec, stream);
    const kq_status s = launched();
    if (s != KQ_OK) return s;
    if (sums && parts > 1) return kqhost::reduce_parts(part_g, part_u, parts, n, dbias_g, dbias_u, stream);
    return KQ_OK;
}

}  // extern "C"
