// The two products of a gated feed-forward block (KroQuant, arXiv 2607.21446v1, Sec. 1 Eq. 2 for each) and their
// gate on large tiles: 256 rows of A by 128 columns of both weights per workgroup, on the scheme of the 256 x 256
// kernel (kq_gemm256.hip has the layouts of the stages, the fragments and the order of the tiles). A stage's 256
// staged rows of W are 128 of the first weight's and then 128 of the second's, as are their scales; a wave's
// fragments are of the two weights in turn, so that both sums of an output are the same lane's.
//
// A product of k = 4096 spends 1.6 us a 256-k stage at 96% of the matrix rate, and in a launch of one tile per
// workgroup another 9 us a tile on starting, the first stage's latency and the epilogue: a quarter of its
// time. So the workgroups here are persistent: the first stage of the next tile is loaded like one more
// stage of this one, into the buffer that its last stage leaves free, and its second when every wave has read that last
// stage; the epilogue, on outputs gated in registers and staged once, in their own type, has a little LDS of its own.
// Stores are counted with the loads and come back in their order, so that a wait for a load waits for the stores before
// it: with both stages asked for in front of them, an epilogue's stores have two stages' time to leave. Where no tile of
// the same kind follows, those loads have no records and no scalar offset. Halves of a tile without a column inside n
// are passed over.
//
// 8192 x 11008 x 4096 bf16 silu, packed scales: 337 to 367 us with the clock the board settles at (4.0 to 4.4 PFLOP/s; FP4
// matrix instructions alone 5.5), 410 as one launch of a workgroup per tile. In one run: 365 us, fp32 outputs 372, with both
// biases 388 (their loads come back behind the next tile's two stages), g and u kept 406, both 431, fp32 with g and u 463,
// scales in the MX layout 420 (four loads of 4 bytes a lane each stage where the packed ones take one of 16). What is left
// over the matrix unit's time is 4 us of epilogue a tile, 32 outputs gated per lane and 4 KB block with nothing to cover
// them: a second set of sums does not fit the registers. Cached stores in place of non-temporal ones: 374 us.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "kq.h"
#include "kq_device.hpp"
#include "kq_dma.hpp"
#include "kq_epilogue.hpp"
#include "kq_host.hpp"
#include "kq_tileorder.hpp"

namespace kq {
namespace gated256 {

using g256::TileOrder;
using g256::TileWork;

constexpr int kThreads = 256, kTile = 256, kGroupM = 4, kLoadSteps = 2;
// a stage: A codes [256][128], W codes [256][128], A scales [256][8], W scales [2][128][8]
constexpr int kOffW = kTile * 128, kOffSA = 2 * kTile * 128, kOffSW = kOffSA + kTile * 8, kStage = kOffSW + kTile * 8;
// after two of them, for each wave: 4 KB to stage outputs in, and two times 64 columns' bias
constexpr int kOffStage = 2 * kStage, kOffBias = kOffStage + 4 * 4096, kLds = kOffBias + 4 * 512;

typedef float floatx16_t __attribute__((ext_vector_type(16)));

struct Geom {
    int kbytes, stages;
    int tiles_m, tiles_n;
    TileOrder order;
};

// One tile's place and operands.
struct Place {
    int64_t m0, n0;
    int rows;
    i32x4_t a, w;   // this wave's descriptors of codes
    i32x4_t s;      // and of scales
    uint32_t s_at;  // the lane's offset into the scales
    uint32_t step;  // scalar offset of stage 1: 0 where there is nothing to load
};

// Values of one output in the matrix layout (16 neighbouring rows' worth of a lane: groups q of columns 8 q + 4 hi ..)
// to their place in the wave's staging block of 32 NP columns.
template <class T, int NP>
__device__ __forceinline__ void stage16(uint8_t *reg, const float (&v)[16], int row, int p, int hi) {
    constexpr int es = (int)sizeof(T), pitch = 32 * NP * es, chunks = pitch / 16;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (es == 2) {
            typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
            *reinterpret_cast<u32x2_t *>(reg + row * pitch + 16 * ((4 * p + q) ^ (row & (chunks - 1))) + 8 * hi) =
                u32x2_t{pack_bf16(v[4 * q], v[4 * q + 1]), pack_bf16(v[4 * q + 2], v[4 * q + 3])};
        } else {
            *reinterpret_cast<floatx4_t *>(reg + row * pitch + 16 * ((8 * p + 2 * q + hi) ^ (row & (chunks - 1)))) =
                floatx4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        }
    }
}

// 32 staged rows of 32 NP columns to rows i0 .. (those < rows) and columns j0 .. of out: whole 16-byte pieces, or
// element by element where those are not aligned or not all inside n.
template <class T, int NP>
__device__ __forceinline__ void flush(const uint8_t *reg, void *out, int64_t ld, int64_t i0, int rows, int64_t j0, int64_t n,
                                      bool whole) {
    // an output that is not wanted has no record: its stores are dropped
    constexpr int es = (int)sizeof(T), cols = 32 * NP, pitch = cols * es, chunks = pitch / 16, kRows = 64 / chunks, ROWS = 32;
    if (rows <= 0 || j0 >= n) return;
    // a new value for each block, so that the offsets of all blocks' elements are not kept side by side
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int left = (int)(n - j0 < cols ? n - j0 : cols);
    const auto ro = out ? block_rsrc<T>(out, ld, i0, rows, j0, left) : row_rsrc(out, 0);
    const uint32_t step = (uint32_t)ld * es;
    if (whole && left == cols) {
        const int c = lane % chunks, r0 = lane / chunks;
#pragma unroll
        for (int i = 0; i < ROWS / kRows; ++i) {
            const int row = kRows * i + r0;
            const u32x4_t v = *reinterpret_cast<const u32x4_t *>(reg + row * pitch + 16 * (c ^ (row & (chunks - 1))));
            __builtin_amdgcn_raw_buffer_store_b128(v, ro, (uint32_t)row * step + 16u * c, 0, 2);
        }
        return;
    }
    const int c = lane % cols, r0 = lane / cols;
    if (c >= left) return;
    for (int row = r0; row < ROWS; row += 64 / cols) {
        const uint8_t *at = reg + row * pitch + 16 * ((c * es / 16) ^ (row & (chunks - 1))) + c * es % 16;
        if (es == 2) __builtin_amdgcn_raw_buffer_store_b16(*reinterpret_cast<const uint16_t *>(at), ro, (uint32_t)row * step + 2 * c, 0, 0);
        else __builtin_amdgcn_raw_buffer_store_b32(*reinterpret_cast<const uint32_t *>(at), ro, (uint32_t)row * step + 4 * c, 0, 0);
    }
}

// NS: scales in the MX layout [rows][k / 32] instead of packed; its last stage may be part of one. A kernel of its own
// for each activation (ACT; none and relu share one, below which `low` is put in) and for whether g and u are wanted
// (PRE): with branches between them the sums of all were moved in front of the branch, into registers that spilled.
template <class T, bool NS, int ACT, bool PRE>
struct Tile {
    const uint8_t *ca, *sa;
    const uint8_t *cw, *sw;  // this wave's weight: waves 0 and 1 load the first's codes, 2 and 3 the second's; wave 2 the first's scales, 3 the second's
    Geom g;
    const GatedEpi &ep;
    uint8_t *smem;
    int lane, w;
    uint32_t lds0;
    float low;  // none: -inf, relu: 0

    // The row and column tile of work i of the order, and its half (0: whole, 1, 2), in one number. Some hundred
    // instructions with their divisions: every lane takes another work, the wave reads them one by one.
    __device__ __forceinline__ uint64_t tile_of(int i) const {
        const TileWork work = g256::tile_work(i, g.order);
        const int u = work.tile, band = u / (kGroupM * g.tiles_n), within = u % (kGroupM * g.tiles_n);
        const int gm = min(kGroupM, g.tiles_m - band * kGroupM);
        return (uint64_t)(uint32_t)(band * kGroupM + within % gm) << 32 | (uint32_t)(within / gm) << 2 | (uint32_t)(work.half + 1);
    }

    // Whether a work, a whole tile or a half, has a column inside n.
    __device__ __forceinline__ bool some(uint32_t tn_half) const {
        return g256::gated_cols((int)(tn_half >> 2), (int)(tn_half & 3) - 1, ep.n).count > 0;
    }

    // TN: staged rows of W, 256 or, for a half tile, 128. none: nothing to load.
    template <int TN>
    __device__ __forceinline__ Place place(uint32_t tm, uint32_t tn_half, bool none) const {
        Place p;
        const g256::GatedCols c = g256::gated_cols((int)(tn_half >> 2), TN == 256 ? -1 : (int)(tn_half & 3) - 1, ep.n);
        p.m0 = (int64_t)tm * kTile;
        p.n0 = c.first;
        p.rows = (int)min<int64_t>(kTile, ep.m - p.m0);
        const g256::CodeSpan a = g256::code_span(p.m0, none ? 0 : p.rows, g.kbytes);
        const g256::CodeSpan w_ = g256::code_span(p.n0, none ? 0 : c.count, g.kbytes);
        p.a = sdesc(ca + a.first, a.bytes);
        p.w = sdesc(cw + w_.first, w_.bytes);
        p.step = a.step;
        // scales: the whole array, so that every read stays inside it (a padding row past m or n reads a later stage's
        // bytes, or zero past the last: its codes are zero and its outputs are not stored)
        const int kblocks = NS ? g.kbytes / 16 : 8 * g.stages;
        const bool is_a = w < 2;
        p.s = sdesc(is_a ? sa : sw, none ? 0u : (uint32_t)(kblocks * (is_a ? ep.m : ep.n)));
        const int64_t row0 = is_a ? p.m0 + 128 * (w & 1) : p.n0;
        p.s_at = NS ? (uint32_t)((row0 + (lane >> 1)) * kblocks) + 4u * (uint32_t)(lane & 1)
                    : (uint32_t)(8 * (row0 + 2 * lane));
        return p;
    }

    static constexpr int kScl = NS ? 4 : 1;
    template <int TN>
    static constexpr int kLoads = 8 + TN / 32 + kScl;

    // Stores of a wave for O where all of its columns leave in whole pieces.
    template <int TN>
    static constexpr int kStores = 128 * (TN / 4) * (int)sizeof(T) / 1024;

    // One tile. `buf`: the buffer of its stage 0; warm: that stage and the next are on their way; stores: and kStores stores
    // or more were issued after them. Returns whether this tile has issued so many. Loads stages 0 and 1 of `next`, from
    // the buffer after the last stage's on (without a branch, which would hold the accumulators' registers twice).
    template <int TN>
    __device__ __forceinline__ bool run(const Place p, int buf, bool warm, bool stores, const Place next) const {
        constexpr int TC = TN / 2, NB = TN / 64, NP = NB / 2, LW = TN / 32;
        // computed for each tile: kept over all of them, the offsets of both kinds of tiles would not fit the registers
        int lane = this->lane;
        asm volatile("" : "+v"(lane));
        const int r = lane & 31, hi = lane >> 5;
        const int wm = (w >> 1) * 128, wn = (w & 1) * (TC / 2);
        // code load j of A and of W: 8 rows, lane & 7 the slot
        uint32_t offa[8], offw[LW];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int row = 64 * w + 8 * j + (lane >> 3);
            offa[j] = (uint32_t)(row * g.kbytes) + 16u * (uint32_t)((lane & 7) ^ swz8(row & 15));
        }
#pragma unroll
        for (int j = 0; j < LW; ++j) {
            const int row = (TN / 4) * (w & 1) + 8 * j + (lane >> 3);
            offw[j] = (uint32_t)(row * g.kbytes) + 16u * (uint32_t)((lane & 7) ^ swz8(row & 15));
        }
        // the chunk of k of an even and of an odd load (their rows start at multiples of 8)
        const int chunk[2] = {(lane & 7) ^ swz8(lane >> 3), (lane & 7) ^ swz8(8 + (lane >> 3))};
        // Load l of stage s, kb bytes of k on, of tile q into buffer `to`: 0 .. 7 A's codes, .. 7 + LW W's, then the scales.
        auto issue = [&](const Place &q, int s, uint32_t kb, int to, int l) {
            const uint32_t st = lds0 + (uint32_t)(to * kStage);
            // chunks past k are pushed past the record count
            auto in = [&](uint32_t off, int j) { return !NS || 128 * s + 16 * chunk[j & 1] < g.kbytes ? off : 0x80000000u; };
            if (l < 8) {
                dma16(q.a, st + (uint32_t)((64 * w + 8 * l) * 128), in(offa[l], l), kb);
            } else if (l < 8 + LW) {
                const int j = l - 8;
                dma16(q.w, st + (uint32_t)(kOffW + ((TN / 4) * w + 8 * j) * 128), in(offw[j], j), kb);
            } else {
                const uint32_t at = st + (uint32_t)(w < 2 ? kOffSA + 1024 * w : kOffSW + 1024 * (w - 2));
                if (NS) {
                    const int j = l - (8 + LW), kblocks = g.kbytes / 16;
                    const bool past = 8 * s + 4 * (lane & 1) >= kblocks;
                    dma4(q.s, at + 256u * (uint32_t)j, past ? 0x80000000u : q.s_at + (uint32_t)(32 * j * kblocks + 8 * s));
                } else {
                    dma16(q.s, at, q.s_at + (uint32_t)(8 * (w < 2 ? ep.m : ep.n)) * (uint32_t)s, 0u);
                }
            }
        };
        auto frag = [&](int b) { return wn + TC * (b & 1) + 32 * (b >> 1); };
        auto frag_scl = [&](int b) { return wn + 128 * (b & 1) + 32 * (b >> 1); };
        int rdo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) rdo[j] = r * 128 + 16 * ((2 * j + hi) ^ swz8(r & 15));
        struct Frag {
            i32x8_t a[4], b[NB];
        };
        struct Scl {
            uint32_t sa[4], sb[NB];
        };
        const uint32_t ns_sel = hi ? 0x07050301u : 0x06040200u;
        auto read_scl = [&](int to, Scl &S) {
            if constexpr (NS) {
                const uint8_t *sc = smem + to * kStage + 8 * r;
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const uint2 d = *reinterpret_cast<const uint2 *>(sc + kOffSA + 8 * (wm + 32 * a));
                    S.sa[a] = __builtin_amdgcn_perm(d.y, d.x, ns_sel);
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint2 d = *reinterpret_cast<const uint2 *>(sc + kOffSW + 8 * frag_scl(b));
                    S.sb[b] = __builtin_amdgcn_perm(d.y, d.x, ns_sel);
                }
            } else {
                const uint8_t *sc = smem + to * kStage + 4 * hi + 8 * r;
#pragma unroll
                for (int a = 0; a < 4; ++a) S.sa[a] = *reinterpret_cast<const uint32_t *>(sc + kOffSA + 8 * (wm + 32 * a));
#pragma unroll
                for (int b = 0; b < NB; ++b) S.sb[b] = *reinterpret_cast<const uint32_t *>(sc + kOffSW + 8 * frag_scl(b));
            }
        };
        auto read_frags = [&](int to, int j, Frag &F) {
            const uint8_t *st = smem + to * kStage;
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const uint4 q = *reinterpret_cast<const uint4 *>(st + (wm + 32 * a) * 128 + rdo[j]);
                F.a[a] = i32x8_t{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 q = *reinterpret_cast<const uint4 *>(st + kOffW + frag(b) * 128 + rdo[j]);
                F.b[b] = i32x8_t{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
            }
        };
        floatx16_t acc[4][NB];
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;
        auto mma = [&](const Frag &F, const Scl &S, auto jc, int a, int b) {
            constexpr int j = decltype(jc)::value;
            acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(F.b[b], F.a[a], acc[a][b], 4, 4, j, (int)S.sb[b], j,
                                                                        (int)S.sa[a]);
        };
        // keeps the instruction that wrote acc[a][b] in front of the loads issued after it (it emits nothing)
        auto pin = [&](int a, int b) { asm volatile("" : "+a"(acc[a][b])); };
        using J0 = std::integral_constant<int, 0>;
        using J1 = std::integral_constant<int, 1>;
        using J2 = std::integral_constant<int, 2>;
        using J3 = std::integral_constant<int, 3>;

        constexpr int kAll = kLoads<TN>, kPerStep = (kAll + kLoadSteps - 1) / kLoadSteps;
        static_assert(kPerStep <= 4 * NB && kLoadSteps <= 3, "every load of a stage needs a slot before the wait");
        // step j with the loads kPerStep j .. of stage s of tile q, one after each matrix instruction
        auto step_loading = [&](const Frag &F, const Scl &S, auto jc, const Place &q, int s, int to) {
            constexpr int j = decltype(jc)::value;
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int l = kPerStep * j + NB * a + b;
                    mma(F, S, jc, a, b);
                    if (j < kLoadSteps && NB * a + b < kPerStep && l < kAll) {
                        pin(a, b);
                        issue(q, s, 128u * (uint32_t)s, to, l);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
        };
        auto step = [&](const Frag &F, const Scl &S, auto jc) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b) mma(F, S, jc, a, b);
        };
        if (!warm) {
            // what the tile before loaded for none to follow it
            asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
            for (int l = kAll - 1; l >= 0; --l) issue(p, 0, 0u, buf, l);
#pragma unroll
            for (int l = kAll - 1; l >= 0; --l) issue(p, 1, p.step, buf ^ 1, l);
        }
        // Stage 0 has landed in every wave's part. After it came the loads of stage 1 and, of the tile before, the stores.
        auto landed = [&](auto younger) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(younger)::value) : "memory");
        };
        static_assert(kAll + kStores<TN> <= 63, "the wait counts at most 63");
        if (stores) landed(std::integral_constant<int, kAll + kStores<TN>>());
        else landed(std::integral_constant<int, kAll>());
        Frag F0, F1;
        Scl S, Sn;
        read_scl(buf, S);
        read_frags(buf, 0, F0);
        // The last steps of a stage: the wait makes the next one's loads visible and ends every wave's reads of this one.
        auto end = [&](auto wait) {
            read_frags(buf, 3, F1);
            __builtin_amdgcn_sched_barrier(0);
            step(F0, S, J2());
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int a = 0; a < 3; ++a)
#pragma unroll
                for (int b = 0; b < NB; ++b) mma(F1, S, J3(), a, b);
            __builtin_amdgcn_sched_barrier(0);
            wait();
            buf ^= 1;
            read_scl(buf, Sn);
            read_frags(buf, 0, F0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma(F1, S, J3(), 3, b);
            __builtin_amdgcn_sched_barrier(0);
            S = Sn;
        };
        // Stage 0: stage 1 is on its way. Stage s from 1 on (s + 1 < stages): the other buffer held stage s - 1, whose last
        // reads came before the previous barrier, so stage s + 1's loads go out during steps 0 .. kLoadSteps - 1.
        read_frags(buf, 1, F1);
        __builtin_amdgcn_sched_barrier(0);
        step(F0, S, J0());
        read_frags(buf, 2, F0);
        __builtin_amdgcn_sched_barrier(0);
        step(F1, S, J1());
        __builtin_amdgcn_sched_barrier(0);
        end([&] {
            if (stores) landed(std::integral_constant<int, kStores<TN>>());
            else landed(std::integral_constant<int, 0>());
        });
        static_assert(kLoadSteps == 2, "the loads of a stage go out in its first two steps");
        for (int s = 1; s + 1 < g.stages; ++s) {
            read_frags(buf, 1, F1);
            __builtin_amdgcn_sched_barrier(0);
            step_loading(F0, S, J0(), p, s + 1, buf ^ 1);
            read_frags(buf, 2, F0);
            __builtin_amdgcn_sched_barrier(0);
            step_loading(F1, S, J1(), p, s + 1, buf ^ 1);
            __builtin_amdgcn_sched_barrier(0);
            end([&] { landed(std::integral_constant<int, 0>()); });
        }
        read_frags(buf, 1, F1);
        __builtin_amdgcn_sched_barrier(0);
        step_loading(F0, S, J0(), next, 0, buf ^ 1);
        read_frags(buf, 2, F0);
        __builtin_amdgcn_sched_barrier(0);
        step_loading(F1, S, J1(), next, 0, buf ^ 1);
        __builtin_amdgcn_sched_barrier(0);
        read_frags(buf, 3, F1);
        step(F0, S, J2());
        step(F1, S, J3());

        // the fragments' registers end here (the compiler would carry matrix instructions into the epilogue, and spill)
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) pin(a, b);
        __builtin_amdgcn_sched_barrier(0);
        // every wave has read the last stage: its buffer takes the next tile's stage 1
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int l = 0; l < kAll; ++l) issue(next, 1, next.step, buf, l);

        // Epilogue: the wave's 128 rows x 32 NP columns, 4 KB at a time.
        const int64_t i0 = p.m0 + wm, j0 = p.n0 + wn;
        const int rows = p.rows - wm;
        // both biases of the wave's columns through LDS (in registers, 64 of them spilled)
        const bool biased = ep.bias || ep.bias_u;
        float *const bias = reinterpret_cast<float *>(smem + kOffBias + 512 * w);
        if (biased) {
            const int64_t j = j0 + (lane & (32 * NP - 1));
            bias[lane] = ep.bias && j < ep.n ? ep.bias[j] : 0.f;
            bias[64 + lane] = ep.bias_u && j < ep.n ? ep.bias_u[j] : 0.f;
        }
        // staged in blocks of 32 rows x 32 CB columns
        constexpr int CB = sizeof(T) == 2 ? NP : 1;
        uint8_t *reg = smem + kOffStage + 4096 * w;
        const bool whole = ep.align >= 16;
        // every block of an output: `value(a, c, v)` gives 32 x 32 of it
        auto put = [&](void *out, int64_t ld, auto value) {
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int c0 = 0; c0 < NP; c0 += CB) {
#pragma unroll
                    for (int c = c0; c < c0 + CB; ++c) {
                        float v[16];
                        if constexpr (PRE) {
                            // a new value for each output, so that one's sums are not kept for the next
                            pin(a, 2 * c);
                            pin(a, 2 * c + 1);
                        }
                        value(a, c, v);
                        stage16<T, CB>(reg, v, r, c - c0, hi);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    // the wave reads back only what it wrote (its LDS operations complete in order)
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    flush<T, CB>(reg, out, ld, i0 + 32 * a, rows - 32 * a, j0 + 32 * c0, ep.n, whole);
                    asm volatile("" ::: "memory");
                }
        };
        auto sums = [&](int a, int c, int of, float (&v)[16]) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = acc[a][2 * c + of][e];
            if (biased) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const floatx4_t x = *reinterpret_cast<const floatx4_t *>(bias + 64 * of + 32 * c + 8 * q + 4 * hi);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * q + e] += x[e];
                }
            }
        };
        auto first = [&](int a, int c, float (&v)[16]) { sums(a, c, 0, v); };
        auto second = [&](int a, int c, float (&v)[16]) { sums(a, c, 1, v); };
        if constexpr (PRE) {
            put(ep.G, ep.ldg, first);
            put(ep.U, ep.ldu, second);
        }
        put(ep.O, ep.ldo, [&](int a, int c, float (&v)[16]) {
            float u[16];
            first(a, c, v);
            second(a, c, u);
            if constexpr (ACT == KQ_ACT_SILU || ACT == KQ_ACT_GELU_TANH) {
                // z s(z), all sixteen one step at a time: with one wave per SIMD nothing else covers a chain of them
                float x[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = ACT == KQ_ACT_SILU ? -kLog2e * v[e] : gelu_tanh_exponent(v[e], v[e] * v[e]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = exp2_hw(x[e]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = 1.0f + x[e];
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = rcp_hw(x[e]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = v[e] * x[e];
            } else if constexpr (ACT == KQ_ACT_GELU) {
                activate<T>(v, ACT);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = v[e] < low ? low : v[e];
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] *= u[e];
        });
        return whole && rows > 96 && j0 + 32 * NP <= ep.n;
    }
};

// Workgroup b takes the works b, b + gridDim.x, ... of the order.
template <class T, bool NS, int ACT, bool PRE>
__global__ __launch_bounds__(kThreads) void gated256_kernel(const uint8_t *__restrict__ ca, const uint8_t *__restrict__ sa,
                                                            const uint8_t *__restrict__ cg, const uint8_t *__restrict__ sg,
                                                            Geom g, GatedEpi ep, int works, float low) {
    __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
    const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const Tile<T, NS, ACT, PRE> t{ca, sa, w < 2 ? cg : ep.cu, w < 3 ? sg : ep.su, g, ep, smem, (int)threadIdx.x & 63, w,
                        (uint32_t)(uintptr_t)smem, low};
    int buf = 0, n = 0;  // n: this workgroup's work
    const int count = (works - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    bool warm = false, stores = false;
    // lane l: work 64 (n / 64) + l
    uint64_t tiles = 0;
    auto work = [&](int k, uint32_t &tm, uint32_t &tn_half) {
        tm = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(tiles >> 32), k & 63);
        tn_half = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)tiles, k & 63);
    };
    auto look = [&](int k) {
        const int mine = (k & ~63) + t.lane;
        tiles = t.tile_of((int)blockIdx.x + (mine < count ? mine : 0) * (int)gridDim.x);
    };
    // n: the next work, from it on, that has a column inside n; `count` for none
    uint32_t tm = 0, tn_half = 0;
    auto seek = [&] {
        for (; n < count; ++n) {
            if ((n & 63) == 0) look(n);
            work(n, tm, tn_half);
            if (t.some(tn_half)) return;
        }
    };
    // works of one kind, whole or half tiles, as long as they follow each other
    auto all = [&](auto TN) {
        Place here = t.template place<TN()>(tm, tn_half, false);
        for (;;) {
            ++n;
            seek();
            const bool ahead = n < count && ((tn_half & 3) == 0) == (TN() == 256);
            const Place next = t.template place<TN()>(ahead ? tm : 0, ahead ? tn_half : TN() == 256 ? 0 : 1, !ahead);
            stores = t.template run<TN()>(here, buf, warm, warm && stores, next);
            // the buffer after the last stage's, where the next tile's first one is
            buf = (buf + g.stages) & 1;
            warm = ahead;
            if (!ahead) break;
            here = next;
        }
    };
    seek();
    while (n < count) {
        if ((tn_half & 3) == 0) all(std::integral_constant<int, 256>());
        else all(std::integral_constant<int, 128>());
    }
    // the loads for none to follow
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

}  // namespace gated256
}  // namespace kq

namespace kqhost {
// kq_mxfp4_gated_linear on these tiles for outputs of type T; its arguments are checked by the caller. Packed scales
// 16-byte aligned and k % 256 == 0, or MX-layout scales 4-byte aligned and k % 128 == 0; k > 256 (two stages).
template <class T>
kq_status launch_gated256(const uint8_t *codes_a, const uint8_t *scales_a, const uint8_t *codes_g, const uint8_t *scales_g,
                          int packed, int64_t k, const kq::GatedEpi &ep, kq_stream_t stream) {
    const int64_t tiles_m = (ep.m + 255) / 256, tiles_n = (ep.n + 127) / 128;
    if (tiles_m * tiles_n >= (int64_t)1 << 23) return KQ_ERR_UNSUPPORTED;
    const int cus = compute_units();
    kq::gated256::Geom g;
    g.kbytes = (int)(k / 2);
    g.stages = (int)((k + 255) / 256);
    g.tiles_m = (int)tiles_m;
    g.tiles_n = (int)tiles_n;
    g.order = kq::g256::make_tile_order((int)(tiles_m * tiles_n), cus);
    const int works = kq::g256::tile_order_groups(g.order);
    const float low = ep.act == KQ_ACT_RELU ? 0.f : -__builtin_huge_valf();
    auto go = [&](auto NS, auto ACT, auto PRE) {
        hipLaunchKernelGGL((kq::gated256::gated256_kernel<T, NS(), ACT(), PRE()>), dim3((unsigned)(works < cus ? works : cus)),
                           dim3(kq::gated256::kThreads), 0, (hipStream_t)stream, codes_a, scales_a, codes_g, scales_g, g, ep,
                           works, low);
    };
    auto go_layout = [&](auto ACT, auto PRE) {
        if (packed) go(std::false_type(), ACT, PRE);
        else go(std::true_type(), ACT, PRE);
    };
    auto go_act = [&](auto PRE) {
        switch (ep.act) {
            case KQ_ACT_SILU: go_layout(std::integral_constant<int, KQ_ACT_SILU>(), PRE); break;
            case KQ_ACT_GELU: go_layout(std::integral_constant<int, KQ_ACT_GELU>(), PRE); break;
            case KQ_ACT_GELU_TANH: go_layout(std::integral_constant<int, KQ_ACT_GELU_TANH>(), PRE); break;
            default: go_layout(std::integral_constant<int, KQ_ACT_NONE>(), PRE); break;
        }
    };
    if (ep.G || ep.U) go_act(std::true_type());
    else go_act(std::false_type());
    return launched();
}
}  // namespace kqhost
