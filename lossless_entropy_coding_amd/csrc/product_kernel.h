// Kernels of the matrix products, for the files that launch them.
#pragma once

#include "ffn_common.h"

namespace ec {
namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) f32x2 lds_f32x2;

// ------------------------------------------------------------- tiled product
//
// A workgroup of WI x WJ waves makes a TI x TJ tile of D, each wave a block
// of 32 x 32 tiles of the matrix units.  The contraction is walked in stages
// of 64 bytes (32 bf16 or 64 e4m3 values); S stages of both factors lie in
// LDS and are filled by loads that bypass the registers.  The fragments of a
// stage are read while the products of the one before run.
//
// What bounds it: every value of a tile's rows passes the CU's load path, 64
// bytes a clock, once a tile, so large tiles halve that (256 x 256: half of
// the matrix units' time at their full rate, 128 x 128: all of it), and the
// power limit, which brings the clock under full load from 2.4 to 1.6 - 2.0
// GHz (the same product of zeros runs 1.25 times as fast).  Eight waves of
// 128 x 64 keep two waves a SIMD (four of 128 x 128 need all registers: Wide).
// 4096 x 16384 x 2048 bf16 with GELU and e4m3 output: 306 us (0.90
// PFLOP/s; 300 to 315 by card); 4096 x 2048 x 16384 e4m3: 224 us with the join
// (1.2); backward of 2048 x 16384 x 2048: 288 us (0.95).  One workgroup a CU
// leaves its first loads and its epilogue exposed: 30% of the waves' time is
// waiting.  Asking for lines ahead of their stage, or loading two stages at
// a time (whole 128-byte lines), was slower where the weights come from HBM.
template <int TI_, int TJ_, int WI_, int WJ_, int S_, int PER_CU_>
struct Shape {
    static constexpr int TI = TI_, TJ = TJ_, WI = WI_, WJ = WJ_, S = S_;
    static constexpr int PER_CU = PER_CU_;              // workgroups whose LDS fits a CU
    static constexpr int NI = TI / WI / 32, NJ = TJ / WJ / 32, W = WI * WJ, THREADS = 64 * W;
    static constexpr int kStage = (TI + TJ) * 64;
};

using Huge = Shape<256, 256, 2, 4, 4, 1>;
using Even = Shape<128, 128, 2, 2, 4, 2>;
using Small = Shape<64, 64, 2, 2, 6, 3>;
using Tall = Shape<256, 128, 4, 2, 4, 1>;               // of the operators beside ec_linear_op's

enum ShapeId { kHuge, kEven, kSmall, kTall, kFew };

constexpr int kStageBytes = 64;            // of the contraction
constexpr uint32_t kOutside = 0x80000000u; // an offset past every buffer: reads as zero

__device__ __forceinline__ constexpr uint32_t unit_order(uint32_t c, uint32_t T) {
    return (2 * (c & 3) + ((c >> 1) & 1)) & (T / 16 - 1);
}

// One factor's tile of T rows (i or j) by one stage.
//
// Rows contiguous along the contraction: the tile holds row r at r * 64, its
// four 16-byte chunks in the order chunk ^ (r / 4 % 4), so that 16 rows' equal
// chunks cover all 64 banks.  Contraction outermost (OUTER): the tile
// holds stage row c at c * 2 T, its 32-byte units in the order unit ^ h(c),
// h = 2 (c % 4) + c / 2 % 2 (modulo the units of a row), so that the four rows of a transposed read fall
// into different banks.  A load writes 1 KB of consecutive LDS per wave; the
// order is made by which address each lane reads.
//
// HALF (the gated product): the tile's rows are HALF of one range of rows and
// HALF of a second one by turns.  A load's 16 rows lie in one range, the same
// one in all loads of a wave, whose first row the wave is given.
template <int T, bool OUTER, int ES, int W, int HALF = 0>
struct Factor {
    static_assert(!HALF || (!OUTER && HALF % 16 == 0 && W * 16 % (2 * HALF) == 0));
    static constexpr int kBytes = T * kStageBytes, kInstr = kBytes / 1024, kLoads = (kInstr + W - 1) / W;
    static constexpr int kDepth = kStageBytes / ES;     // contraction values a stage
    static constexpr int kRowsPer = 1024 / (T * 2);     // OUTER: stage rows a load
    uint32_t off[kLoads];                               // per lane
    uint64_t base;                                      // of the stage
    int64_t left;                                       // bytes from base to the end of what may be read
    uint64_t step;
    i32x4 d;                                            // the buffer of the stage being loaded
    uint32_t out;                                       // kOutside on the lanes past the contraction's end

    // rows: of the tile that exist; stride in elements; first and count along the contraction
    __device__ __forceinline__ void init(const void *p, uint64_t stride, uint64_t row0, uint32_t rows, uint32_t c0,
                                         uint32_t c1, uint32_t wave, uint32_t lane) {
        const uint64_t sb = stride * ES;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const uint32_t q = (n * W + wave) % kInstr;
            if constexpr (OUTER) {
                constexpr uint32_t kLane = 64 / kRowsPer;
                const uint32_t c = q * kRowsPer + lane / kLane, pos = lane % kLane;
                const uint32_t h = unit_order(c, T);
                off[n] = c * (uint32_t)sb + ((((pos >> 1) ^ h) << 1) | (pos & 1)) * 16;
            } else {
                const uint32_t r = q * 16 + (lane >> 2);
                uint32_t row = r;
                if constexpr (HALF) row = r / (2 * HALF) * HALF + r % HALF;
                off[n] = row * (uint32_t)sb + ((lane & 3) ^ ((r >> 2) & 3)) * 16;
            }
        }
        if constexpr (OUTER) {
            base = (uint64_t)p + c0 * sb + row0 * ES;
            left = ((int64_t)(c1 - c0) - 1) * (int64_t)sb + rows * ES;
            step = kDepth * sb;
        } else {
            base = (uint64_t)p + row0 * sb + (uint64_t)c0 * ES;
            left = ((int64_t)rows - 1) * (int64_t)sb + (int64_t)(c1 - c0) * ES;
            step = kStageBytes;
        }
        left = (left + 3) & ~3ll;           // whole dwords: the last one holds valid elements
    }

    // Makes the next stage the one to load; `rest` is what remains of the
    // contraction, in bytes of a row (not OUTER): chunks past it read as zero.
    __device__ __forceinline__ void next(uint32_t rest, uint32_t lane) {
        // by halves: the scalar unit does not compare 64 bits with a sign
        const int32_t high = (int32_t)(left >> 32);
        const uint32_t low = (uint32_t)left, n = high < 0 ? 0 : high > 0 || low > 0x7FFFFFFFu ? 0x7FFFFFFFu : low;
        d[0] = __builtin_amdgcn_readfirstlane((int)base);
        d[1] = __builtin_amdgcn_readfirstlane((int)(base >> 32) & 0xFFFF);
        d[2] = __builtin_amdgcn_readfirstlane((int)(rest ? n : 0));
        d[3] = 0x00027000;
        out = 0;
        if constexpr (!OUTER) out = ((lane & 3) ^ ((lane >> 4) & 3)) * 16 < rest ? 0 : kOutside;
        base += step;
        left -= (int64_t)step;
    }

    // Load k of that stage, to the stage's place in LDS (in m0).  The compiler
    // may make d with vector instructions, after which a memory instruction
    // needs five wait states, and it does not count them for inline assembly.
    __device__ __forceinline__ void load(int k, uint32_t at, uint32_t wave) {
        const uint32_t q = (k * W + wave) % kInstr;
        asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off[k] | out), "s"(d),
                     "{m0}"(at + q * 1024)
                     : "memory");
    }
};

// A wave's fragments of one factor: N tiles of 32 rows by the two halves of a stage.
template <int T, int N, bool OUTER>
struct Fragments {
    // per-lane LDS offsets within a stage of the factor
    static __device__ __forceinline__ uint32_t at(uint32_t wave_row, int t, uint32_t lane) {
        if constexpr (OUTER) {
            const uint32_t c = 8 * (lane >> 5) + ((lane & 15) >> 2), h = unit_order(c, T);
            const uint32_t unit = wave_row / 16 + t * 2 + ((lane >> 4) & 1);
            return c * (2 * T) + (unit ^ h) * 32 + (lane & 3) * 8;
        } else {
            return (wave_row + t * 32 + (lane & 31)) * 64 + ((lane >> 5) ^ ((lane >> 2) & 3)) * 16;
        }
    }

    // Half s of tile t.
    static __device__ __forceinline__ void read(u32x4 (&f)[N][2], lds_char *stage, const uint32_t *offs, int t, int s) {
        if constexpr (OUTER) {
            union {
                s16x4 h[2];
                u32x4 w;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(stage + offs[t] + s * 16 * 2 * T));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(stage + offs[t] + (s * 16 + 4) * 2 * T));
            f[t][s] = u.w;
        } else {
            f[t][s] = *(lds_u32x4 *)(stage + (offs[0] ^ (s * 32)) + t * 2048);
        }
    }
};

// A stage's products, in the order of the fragments' halves; between(g) is
// called before each of kGroups groups of them, for what goes on beside them.
template <int NI, int NJ, bool E4M3>
struct Multiply {
    static constexpr int kGroups = E4M3 ? 4 : 2 * NI;

    template <class F>
    static __device__ __forceinline__ void run(f32x16 (&acc)[NI][NJ], const u32x4 (&a)[NI][2], const u32x4 (&b)[NJ][2],
                                               F between) {
        if constexpr (E4M3) {
            // e4m3 values are exact in bf16, and the products of bf16 are added in
            // 32 bits.  The e4m3 instructions are not used: they cut the products
            // they add to a few bits below the largest (measured: sums of 16
            // products of random bytes off by up to 2^-11.2 of the sum of
            // magnitudes, against 2^-22.3 here), where sums are to be held in 32
            // bits.
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                between(s);
                bf16x8 fa[NI], fb[NJ];
#pragma unroll
                for (int x = 0; x < NI; ++x)
                    fa[x] = e4m3_to_bf16x8(a[x][s >> 1][2 * (s & 1)], a[x][s >> 1][2 * (s & 1) + 1]);
#pragma unroll
                for (int y = 0; y < NJ; ++y)
                    fb[y] = e4m3_to_bf16x8(b[y][s >> 1][2 * (s & 1)], b[y][s >> 1][2 * (s & 1) + 1]);
#pragma unroll
                for (int x = 0; x < NI; ++x)
#pragma unroll
                    for (int y = 0; y < NJ; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[y], fa[x], acc[x][y], 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int x = 0; x < NI; ++x) {
                    between(s * NI + x);
#pragma unroll
                    for (int y = 0; y < NJ; ++y)
                        acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b[y][s]),
                                                                            __builtin_bit_cast(bf16x8, a[x][s]),
                                                                            acc[x][y], 0, 0, 0);
                }
        }
    }
};

// ----------------------------------------------------------------- epilogue

// The wave's accumulators hold, of each 32 x 32 tile, row i = lane % 32 and
// columns 8 g + 4 (lane / 32) + r in register 4 g + r.  32 rows at a time go
// through the wave's part of LDS (fp32, 16-byte chunks in the order chunk ^
// row), so that a lane has eight consecutive columns, the same ones in every
// row, and the lanes of a row side by side read and write whole lines.
template <int NJ>
struct Turn {
    static constexpr int kLanes = NJ * 4, kRows = 64 / kLanes, kBytes = 32 * NJ * 128;  // lanes a row, rows at a time

    static __device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t chunk) {
        return row * (NJ * 128) + (chunk ^ (NJ == 1 ? row >> 1 & 7 : row & (NJ * 8 - 1))) * 16;
    }

    static __device__ __forceinline__ void put(lds_char *mem, const f32x16 (&acc)[NJ], uint32_t lane) {
#pragma unroll
        for (int y = 0; y < NJ; ++y)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *(lds_f32x4 *)(mem + chunk_at(lane & 31, y * 8 + g * 2 + (lane >> 5))) =
                    f32x4{acc[y][4 * g], acc[y][4 * g + 1], acc[y][4 * g + 2], acc[y][4 * g + 3]};
    }

    static __device__ __forceinline__ void get(lds_char *mem, uint32_t row, uint32_t lane, float *v) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 w = *(lds_f32x4 *)(mem + chunk_at(row, lane % kLanes * 2 + h));
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * h + r] = w[r];
        }
    }
};

template <int NI, int NJ, int OP, int ACT>
__device__ __forceinline__ void finish_tiles(const ProductArgs &p, f32x16 (&acc)[NI][NJ], uint32_t g, uint32_t i0,
                                             uint32_t i1, uint32_t j0, bool zero, lds_char *mem) {
    using R = Turn<NJ>;
    constexpr int kSteps = 32 / R::kRows;
    const uint32_t lane = threadIdx.x & 63, j = j0 + lane % R::kLanes * 8;
    const float os = OP == EC_LINEAR_FORWARD && p.out_scale ? *p.out_scale : 1.0f;
    const Columns c = load_columns<OP>(p, g, j);
    // The residual, or the activation's input, of all rows is asked for at
    // once, since every turn of 32 rows would wait for HBM anew (1023 x 2050:
    // 26.1 -> 23.9 us); the forward pass's large tiles have no registers left
    // for that (spilled, 4096 x 16384 x 2048 takes 6% longer).
    constexpr bool kSide = OP == EC_LINEAR_FORWARD || (OP == EC_LINEAR_GRAD_INPUT && ACT != EC_ACT_NONE);
    const uint16_t *const from = OP == EC_LINEAR_FORWARD ? p.residual : p.preact;
    const uint64_t stride = OP == EC_LINEAR_FORWARD ? p.residual_stride : p.preact_stride;
    constexpr bool kAll = kSide && (OP != EC_LINEAR_FORWARD || NI * NJ < 8);
    u32x4 side[kAll ? NI : 1][kSteps];
    const auto load_sides = [&](int x) {
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const uint32_t i = i0 + x * 32 + t * R::kRows + lane / R::kLanes;
            u32x4 w = {0, 0, 0, 0};
            if (from && i < i1 && c.left >= 8) w = ((const AnyU32x4 *)(from + i * stride + j))->v;
            side[kAll ? x : 0][t] = w;
        }
    };
    if constexpr (kAll) {
#pragma unroll
        for (int x = 0; x < NI; ++x) load_sides(x);
    }
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        R::put(mem, acc[x], lane);
        if constexpr (kSide && !kAll) load_sides(x);
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const uint32_t row = t * R::kRows + lane / R::kLanes, i = i0 + x * 32 + row;
            float v[8], extra[8], xs = 1.0f;
            R::get(mem, row, lane, v);
            if (i >= i1) continue;
            if (OP == EC_LINEAR_FORWARD && p.x_scale) xs = p.x_scale[p.x_scales > 1 ? i : 0];
            if constexpr (kSide) {
                if (c.left >= 8) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        extra[2 * q] = __uint_as_float(side[kAll ? x : 0][t][q] << 16);
                        extra[2 * q + 1] = __uint_as_float(side[kAll ? x : 0][t][q] & 0xFFFF0000u);
                    }
                } else {
                    load_side<OP>(p, i, j, c.left, extra);
                }
            }
            finish8<OP, ACT>(p, g, i, j, v, c, extra, xs, os, zero);
        }
    }
}

// The gated product's: of a wave's NJ * 32 columns the first half are the
// gate's, the second half what it is multiplied by, of the same NJ * 16 columns
// of the output; a lane has eight of them.
struct GatedColumns {
    Columns gate, rest;
    uint32_t left;
};

__device__ __forceinline__ GatedColumns load_gated_columns(const ProductArgs &p, uint32_t g, uint32_t j) {
    GatedColumns c;
    c.left = p.J > j ? p.J - j : 0;
    const uint64_t at = (uint64_t)g * 2 * p.J + j;
    if (p.w_scale) {
        // not in a branch of its own, for which the compiler keeps the address in scratch memory
        const float one = p.w_scale[p.w_scales > 1 ? (uint64_t)g * 2 * p.J : g];
#pragma unroll
        for (int q = 0; q < 8; ++q) c.gate.w_scale[q] = c.rest.w_scale[q] = one;
        if (p.w_scales > 1) {
            load8(p.w_scale, EC_FP32, at, c.left, c.gate.w_scale);
            load8(p.w_scale, EC_FP32, at + p.J, c.left, c.rest.w_scale);
        }
    }
    if (p.bias) {
        load8(p.bias, p.bias_dtype, at, c.left, c.gate.bias);
        load8(p.bias, p.bias_dtype, at + p.J, c.left, c.rest.bias);
    }
    return c;
}

// Finishes and stores eight columns of row i: y = act(gate) rest.
template <int ACT>
__device__ __forceinline__ void finish8_gated(const ProductArgs &p, uint32_t i, uint32_t j, float *gate, float *rest,
                                              const GatedColumns &c, float x_scale, float out_scale, bool zero) {
    if (!c.left) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        if (p.x_scale) {
            gate[q] *= x_scale;
            rest[q] *= x_scale;
        }
        if (p.w_scale) {
            gate[q] *= c.gate.w_scale[q];
            rest[q] *= c.rest.w_scale[q];
        }
        if (p.bias) {
            gate[q] += c.gate.bias[q];
            rest[q] += c.rest.bias[q];
        }
        if (zero) gate[q] = rest[q] = 0.0f;
    }
    if (p.preact) {
        store8(p.preact, EC_BF16, i * p.preact_stride + j, c.left, gate);
        store8(p.preact, EC_BF16, i * p.preact_stride + p.J + j, c.left, rest);
    }
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        v[q] = act_value<ACT>(gate[q]) * rest[q];
        if (p.out_scale) v[q] *= out_scale;
    }
    store8(p.out, p.out_dtype, i * p.out_stride + j, c.left, v);
}

template <int NI, int NJ, int ACT>
__device__ __forceinline__ void finish_gated(const ProductArgs &p, f32x16 (&acc)[NI][NJ], uint32_t g, uint32_t i0,
                                             uint32_t i1, uint32_t j0, bool zero, lds_char *mem) {
    using R = Turn<NJ>;
    constexpr int kLanes = NJ * 2, kRows = 64 / kLanes;
    const uint32_t lane = threadIdx.x & 63, j = j0 + lane % kLanes * 8;
    const float os = p.out_scale ? *p.out_scale : 1.0f;
    const GatedColumns c = load_gated_columns(p, g, j);
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        R::put(mem, acc[x], lane);
        // not unrolled for the large tiles: what follows is long, and the sums must stay in registers
        constexpr int kUnroll = NI * NJ < 8 ? 32 / kRows : 1;
#pragma unroll kUnroll
        for (int t = 0; t < 32 / kRows; ++t) {
            const uint32_t row = t * kRows + lane / kLanes, i = i0 + x * 32 + row;
            float gate[8], rest[8], xs = 1.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const f32x4 a = *(lds_f32x4 *)(mem + R::chunk_at(row, lane % kLanes * 2 + h));
                const f32x4 b = *(lds_f32x4 *)(mem + R::chunk_at(row, NJ * 4 + lane % kLanes * 2 + h));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    gate[4 * h + r] = a[r];
                    rest[4 * h + r] = b[r];
                }
            }
            if (i >= i1) continue;
            if (p.x_scale) xs = p.x_scale[p.x_scales > 1 ? i : 0];
            finish8_gated<ACT>(p, i, j, gate, rest, c, xs, os, zero);
        }
    }
}

// The gradient of the cross entropy at eight logits of a row, columns j ..
// j + 7 of the piece: (exp(logit - lse) - [target]) times the loss's gradient;
// zeros past the last column, so that rows are whole 16-byte chunks.  Rounded
// to bf16 for the matrix units, as every factor of the backward products is.
__device__ __forceinline__ void finish8_logits(const ProductArgs &p, uint32_t i, uint32_t j, float *v, float2 row,
                                               int32_t target) {
    const uint32_t at = (uint32_t)target - (p.first + j);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = __builtin_amdgcn_exp2f((v[q] - row.x) * kLog2E) * row.y;
    if (at < 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] -= q == (int)at ? row.y : 0.0f;
    }
    if (j + 8 > p.J) {
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = j + q < p.J ? v[q] : 0.0f;
    }
    store8(p.out, EC_BF16, i * p.out_stride + j, 8, v);
}

template <int NI, int NJ>
__device__ __forceinline__ void finish_logits(const ProductArgs &p, f32x16 (&acc)[NI][NJ], uint32_t i0, uint32_t i1,
                                              uint32_t j0, lds_char *mem) {
    using R = Turn<NJ>;
    const uint32_t lane = threadIdx.x & 63, j = j0 + lane % R::kLanes * 8;
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        R::put(mem, acc[x], lane);
#pragma unroll
        for (int t = 0; t < 32 / R::kRows; ++t) {
            const uint32_t row = t * R::kRows + lane / R::kLanes, i = i0 + x * 32 + row;
            float v[8];
            R::get(mem, row, lane, v);
            if (i < i1 && j < p.J) finish8_logits(p, i, j, v, p.row[i], p.row_target[i]);
        }
    }
}

// With an activation known when compiled.
template <int NI, int NJ, int OP, int ACT>
__device__ __forceinline__ void finish_act(const ProductArgs &p, f32x16 (&acc)[NI][NJ], uint32_t g, uint32_t i0,
                                           uint32_t i1, uint32_t j0, bool zero, lds_char *mem) {
    if constexpr (OP == kOpLogitGrad)
        finish_logits<NI, NJ>(p, acc, i0, i1, j0, mem);
    else if constexpr (OP == kOpGated)
        finish_gated<NI, NJ, ACT>(p, acc, g, i0, i1, j0, zero, mem);
    else
        finish_tiles<NI, NJ, OP, ACT>(p, acc, g, i0, i1, j0, zero, mem);
}

// Whether an operator's epilogue has an activation.
template <int OP>
constexpr bool kActs = OP == EC_LINEAR_FORWARD || OP == EC_LINEAR_GRAD_INPUT || OP == kOpGated;

template <int NI, int NJ, int OP>
__device__ __forceinline__ void finish(const ProductArgs &p, f32x16 (&acc)[NI][NJ], uint32_t g, uint32_t i0,
                                       uint32_t i1, uint32_t j0, bool zero, lds_char *mem) {
    if constexpr (!kActs<OP>) {
        finish_act<NI, NJ, OP, EC_ACT_NONE>(p, acc, g, i0, i1, j0, zero, mem);
    } else {
        switch (p.act) {
            case EC_ACT_GELU: finish_act<NI, NJ, OP, EC_ACT_GELU>(p, acc, g, i0, i1, j0, zero, mem); break;
            case EC_ACT_SILU: finish_act<NI, NJ, OP, EC_ACT_SILU>(p, acc, g, i0, i1, j0, zero, mem); break;
            case EC_ACT_RELU: finish_act<NI, NJ, OP, EC_ACT_RELU>(p, acc, g, i0, i1, j0, zero, mem); break;
            default: finish_act<NI, NJ, OP, EC_ACT_NONE>(p, acc, g, i0, i1, j0, zero, mem);
        }
    }
}

// -------------------------------------------------------------- tile order
//
// Workgroups go round the 8 XCDs in turn; each XCD gets a run of consecutive
// tiles, taken in bands of kBand row tiles, the row fastest, so that what an
// XCD works on at a time shares rows of both factors in its L2.
constexpr uint32_t kBand = 8;

__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t total) {
    const uint32_t x = b & 7, per = total >> 3, rem = total & 7;
    return x * per + min(x, rem) + (b >> 3);
}

__device__ __forceinline__ void band_order(uint32_t t, uint32_t tiles_i, uint32_t tiles_j, uint32_t *ti, uint32_t *tj) {
    const uint32_t band = t / (kBand * tiles_j), r = t - band * (kBand * tiles_j);
    const uint32_t h = min(kBand, tiles_i - band * kBand);
    *tj = r / h;
    *ti = band * kBand + (r - *tj * h);
}

// Row tiles of a product that is not ragged.
template <class T, int OP>
__device__ __forceinline__ uint32_t row_tiles(const ProductArgs &p) {
    if constexpr (counts_rows(OP) && !contracts_a_rows(OP))
        return (min(p.I, (uint32_t)__builtin_amdgcn_readfirstlane((int)*p.used)) + T::TI - 1) / T::TI;
    else
        return p.tiles_i;
}

// Whether the contraction may be split (a kernel joins the sums).
template <int OP>
constexpr bool kJoins = OP != kOpRowStats && OP != kOpLogitGrad;

struct Place {
    uint32_t i0, i1, j0, c0, c1, group, split, tile;
    bool zero, none;
};

template <class T, int OP>
__device__ __forceinline__ Place find_place(const ProductArgs &p, uint32_t block) {
    constexpr uint32_t TJ = OP == kOpGated ? T::TJ / 2 : T::TJ;      // columns of the output
    Place q = {};
    uint32_t ti, tj;
    q.c1 = p.C;
    if constexpr (counts_rows(OP)) {
        const uint32_t used = (uint32_t)__builtin_amdgcn_readfirstlane((int)*p.used);
        const uint32_t tiles_i = row_tiles<T, OP>(p), tiles = tiles_i * p.tiles_j;
        const uint32_t total = tiles * (kJoins<OP> ? p.splits : 1);
        q.none = block >= total;
        if (q.none) return q;
        const uint32_t t = xcd_order(block, total);
        q.split = t / tiles;
        q.tile = t - q.split * tiles;
        band_order(q.tile, tiles_i, p.tiles_j, &ti, &tj);
        q.i0 = ti * T::TI;
        q.i1 = min(p.I, q.i0 + T::TI);
        if constexpr (contracts_a_rows(OP))
            q.c1 = min(p.C, used);
        else
            q.i1 = min(q.i1, used);
    } else if (p.groups && OP != EC_LINEAR_GRAD_WEIGHT) {
        const uint32_t rows = (uint32_t)__builtin_amdgcn_readfirstlane(
            (int)count_row_tiles(p.offsets, p.groups, p.I, T::TI));
        const uint64_t total = (uint64_t)rows * p.tiles_j;
        q.none = block >= total;
        if (q.none) return q;
        band_order(xcd_order(block, (uint32_t)total), rows, p.tiles_j, &ti, &tj);
        const RowTile r = find_row_tile(p.offsets, p.groups, p.I, T::TI, ti);
        q.i0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)r.row);
        q.i1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)r.end);
        q.group = (uint32_t)__builtin_amdgcn_readfirstlane((int)r.group);
        q.zero = __builtin_amdgcn_readfirstlane((int)r.zero);
        if (q.zero) q.c1 = 0;
    } else {
        const uint32_t tiles = p.tiles_i * p.tiles_j, t = xcd_order(block, gridDim.x);
        const uint32_t z = t / tiles;
        q.tile = t - z * tiles;
        band_order(q.tile, p.tiles_i, p.tiles_j, &ti, &tj);
        q.i0 = ti * T::TI;
        q.i1 = min(p.I, q.i0 + T::TI);
        if (p.groups) {
            q.group = z;
            group_range(p.offsets, p.C, z, &q.c0, &q.c1);
            q.c0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)q.c0);
            q.c1 = (uint32_t)__builtin_amdgcn_readfirstlane((int)q.c1);
        } else {
            q.split = z;
        }
    }
    q.j0 = tj * TJ;
    return q;
}

// Tile (x, y) of a wave's sums, laid out by tiles or by pairs of columns of them.
template <int NI, int NJ>
__device__ __forceinline__ f32x16 &tile_of(f32x16 (&acc)[NI][NJ], int x, int y) {
    return acc[x][y];
}

template <int NI>
__device__ __forceinline__ f32x16 &tile_of(f32x16 (&acc)[2][NI][2], int x, int y) {
    return acc[y / 2][x][y % 2];
}

// Of the tile's columns, each row's maximum and the sum of the exponentials
// from it, and the logit of the row's target where that is among them.  A
// wave's accumulators hold row lane % 32 and half of the columns of a 32 x 32
// tile; the waves side by side are joined in LDS.  A maximum of -inf counts as
// 0 in the exponent, so that columns of -inf add nothing.
template <class T, class ACC>
__device__ __forceinline__ void finish_stats(const ProductArgs &p, ACC &acc, const Place &q, uint32_t wi, uint32_t wave,
                                             lds_char *at_mem) {
    constexpr int NI = T::NI, NJ = T::NJ;
    lds_f32x2 *const mem = (lds_f32x2 *)at_mem;
    const uint32_t lane = threadIdx.x & 63, wj = wave % T::WJ, j0 = q.j0 + wj * (NJ * 32);
    const uint32_t columns = p.J > j0 ? p.J - j0 : 0, half = 4 * (lane >> 5);
#pragma unroll
    for (int x = 0; x < NI; ++x) {
        const uint32_t row = wi + x * 32 + (lane & 31), i = q.i0 + row;
        int64_t at = -1;
        if (i < q.i1) at = p.target_bytes == 8 ? ((const int64_t *)p.target)[i] : (int64_t)((const int32_t *)p.target)[i];
        at -= (int64_t)j0;
        const uint32_t place = at >= 0 && at < (int64_t)min(columns, NJ * 32u) ? (uint32_t)at : ~0u;
        if (columns < NJ * 32) {            // the vocabulary's end
#pragma unroll
            for (int y = 0; y < NJ; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (y * 32 + 8 * (r >> 2) + half + (r & 3) >= columns) tile_of(acc, x, y)[r] = -__builtin_inff();
        }
        float hit = 0.0f;
        if (__ballot(place != ~0u)) {       // seldom, of a large one
#pragma unroll
            for (int y = 0; y < NJ; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    hit = y * 32 + 8 * (r >> 2) + half + (r & 3) == place ? tile_of(acc, x, y)[r] : hit;
        }
        // four sums side by side, so that none waits for the one before
        float tops[4], sums[4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k) tops[k] = tile_of(acc, x, 0)[k];
#pragma unroll
        for (int y = 0; y < NJ; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) tops[r & 3] = fmaxf(tops[r & 3], tile_of(acc, x, y)[r]);
        float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        top = fmaxf(top, -__builtin_inff());                            // of NaN only
        top = fmaxf(top, __shfl_xor(top, 32));
        const float from = top == -__builtin_inff() ? 0.0f : top;
#pragma unroll
        for (int y = 0; y < NJ; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                sums[r & 3] += __builtin_amdgcn_exp2f((tile_of(acc, x, y)[r] - from) * kLog2E);
        float sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
        sum += __shfl_xor(sum, 32);
        if (place != ~0u && (place & 4) == half) p.hit[i] = hit;
        if (lane < 32) mem[wj * T::TI + row] = f32x2{top, sum};
    }
    __syncthreads();
    const uint32_t t = threadIdx.x, i = q.i0 + t;       // as many threads as rows, or more
    static_assert(T::THREADS >= T::TI);
    if (t >= T::TI || i >= q.i1) return;
    float2 s = {mem[t][0], mem[t][1]};
#pragma unroll
    for (int k = 1; k < T::WJ; ++k) s = join_stats(s, float2{mem[k * T::TI + t][0], mem[k * T::TI + t][1]});
    p.stats[(uint64_t)i * p.tiles_j + q.j0 / T::TJ] = s;
}

__device__ __forceinline__ float sum8(const u32x4 &w) {
    float s[4];
#pragma unroll
    for (int d = 0; d < 4; ++d) s[d] = __uint_as_float(w[d] << 16) + __uint_as_float(w[d] & 0xFFFF0000u);
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// SUM (grad weight): db too.  The branch costs the loop a tenth, so it is not
// in the kernel of a large dense product, whose dy is little to read again
// (2048 x 16384 x 2048: 127 us and 10 us for the sums, 141 us together);
// 16 groups of 8192 rows by 2048 columns: 69 us and 16 us, 76 us together.
template <class T, int OP, bool E4M3, bool SUM>
__global__ __launch_bounds__(T::THREADS, 2) void product_kernel(ProductArgs p) {
    constexpr bool kOuterA = contracts_a_rows(OP), kOuterB = contracts_b_rows(OP), kGated = OP == kOpGated;
    constexpr int kES = E4M3 ? 1 : 2, kDepth = kStageBytes / kES;
    constexpr int NI = T::NI, NJ = T::NJ, S = T::S;
    using FA = Factor<T::TI, kOuterA, kES, T::W>;
    using FB = Factor<T::TJ, kOuterB, kES, T::W, kGated ? NJ * 16 : 0>;
    using RA = Fragments<T::TI, NI, kOuterA>;
    using RB = Fragments<T::TJ, NJ, kOuterB>;
    __shared__ __attribute__((aligned(1024))) char lds[S * T::kStage];

    if (!counts_rows(OP) && p.groups && blockIdx.x == 0 && threadIdx.x < 64)
        check_offsets(p.offsets, p.groups, kOuterA ? p.C : p.I, p.status);
    const Place q = find_place<T, OP>(p, blockIdx.x);
    if (q.none) return;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t wi = wave / T::WJ * (NI * 32), wj = wave % T::WJ * (NJ * 32);

    // the split's range of stages
    uint32_t c0 = q.c0, c1 = q.c1;
    if (kJoins<OP> && p.splits > 1) {
        const uint32_t stages = (c1 + kDepth - 1) / kDepth;
        c0 = (uint32_t)((uint64_t)stages * q.split / p.splits) * kDepth;
        c1 = min(c1, (uint32_t)((uint64_t)stages * (q.split + 1) / p.splits) * kDepth);
    }
    f32x16 acc[NI][NJ];
#pragma unroll
    for (int x = 0; x < NI; ++x)
#pragma unroll
        for (int y = 0; y < NJ; ++y)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[x][y][r] = 0.0f;
    // db, the sum of A over the contraction: the first tile of a row of tiles
    // adds up its fragments, a wave those of one of its NI tiles of 32 rows
    // (the waves side by side hold the same ones).
    float db = 0.0f;

    if (c1 > c0) {
        const uint32_t n = (c1 - c0 + kDepth - 1) / kDepth;
        const void *a = p.a;
        const void *b = (const char *)p.b + (kOuterA ? 0 : q.group * p.b_group * kES);
        FA fa;
        FB fb;
        fa.init(a, kOuterA ? p.a_c : p.a_i, q.i0, q.i1 - q.i0, c0, c1, wave, lane);
        if constexpr (kGated) {
            const uint64_t half = wave * 16 / (NJ * 16) & 1;
            fb.init(b, p.b_j, half * p.J + q.j0, min((uint32_t)T::TJ / 2, p.J - q.j0), c0, c1, wave, lane);
        } else {
            fb.init(b, kOuterB ? p.b_c : p.b_j, q.j0, min((uint32_t)T::TJ, p.J - q.j0), c0, c1, wave, lane);
        }
        lds_char *const mem = (lds_char *)lds;
        const uint32_t mem_at = (uint32_t)(uintptr_t)mem;
        uint32_t rest = (c1 - c0) * kES;      // below 2^32
        uint32_t ao[NI], bo[NJ];
#pragma unroll
        for (int x = 0; x < NI; ++x) ao[x] = RA::at(wi, x, lane);
#pragma unroll
        for (int y = 0; y < NJ; ++y) bo[y] = T::TI * kStageBytes + RB::at(wj, y, lane);

        constexpr int kLoads = FA::kLoads + FB::kLoads, kReads = 2 * (NI + NJ);
        uint32_t fill_at = 0, read_at = 0;
        const auto load = [&](int k) {      // of kLoads
            if (k == 0) fa.next(rest, lane);
            if (k == FA::kLoads) fb.next(rest, lane);
            const uint32_t at = mem_at + fill_at * T::kStage;
            if (k < FA::kLoads)
                fa.load(k, at, wave);
            else
                fb.load(k - FA::kLoads, at + FA::kBytes, wave);
            if (k == kLoads - 1) {
                fill_at = fill_at + 1 == S ? 0 : fill_at + 1;
                rest = rest > kStageBytes ? rest - kStageBytes : 0;
            }
        };
        u32x4 af[2][NI][2], bf[2][NJ][2];
        const auto read = [&](int r, int to, uint32_t stage) {      // in the order of their use
            const int s = r / (NI + NJ), t = r % (NI + NJ);
            if (t < NJ)
                RB::read(bf[to], mem + stage * T::kStage, bo, t, s);
            else
                RA::read(af[to], mem + stage * T::kStage, ao, t - NJ, s);
        };
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) load(k);
        // stage 0 has arrived, everywhere
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((S - 1) * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
#pragma unroll
        for (int r = 0; r < kReads; ++r) read(r, 0, 0);
        // Stage k: its fragments are in registers (or on the way).  Once every
        // wave has them, its LDS takes stage k + S, and stage k + 1 is read.
        // The loads are spread over the products of stage k (a wave whose load
        // finds the queue full issues no products either), the reads over
        // their first half, so that the wait for the last one is short.
        const bool sum = SUM && q.j0 == 0;
        const auto step = [&](int now) {
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((S - 2) * kLoads) : "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            read_at = read_at + 1 == S ? 0 : read_at + 1;
            using M = Multiply<NI, NJ, E4M3>;
            M::run(acc, af[now], bf[now], [&](int g) {
                constexpr int G = M::kGroups;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int r = 0; r < kReads; ++r)
                    if (r >= 2 * g * kReads / G && r < 2 * (g + 1) * kReads / G) read(r, 1 - now, read_at);
#pragma unroll
                for (int k = 0; k < kLoads; ++k)
                    if (k >= g * kLoads / G && k < (g + 1) * kLoads / G) load(k);
            });
            if constexpr (SUM) {
                if (sum) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        u32x4 f = af[now][0][s];
#pragma unroll
                        for (int x = 1; x < NI; ++x)
#pragma unroll
                            for (int d = 0; d < 4; ++d) f[d] = wave % T::WJ == (uint32_t)x ? af[now][x][s][d] : f[d];
                        db += sum8(f);
                    }
                }
            }
        };
        for (uint32_t k = 0;;) {
            step(0);
            if (++k >= n) break;
            step(1);
            if (++k >= n) break;
        }
        // nothing is left in flight into this workgroup's LDS
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    if constexpr (SUM) {
        // The lane's two halves of the contraction; row lane % 32 of the wave's tile x.
        db += __shfl_xor(db, 32);
        const uint32_t x = wave % T::WJ, i = q.i0 + wi + x * 32 + lane;
        if (q.j0 == 0 && x < (uint32_t)NI && lane < 32 && i < q.i1) p.db[(uint64_t)q.group * p.I + i] = db;
    }
    if (kJoins<OP> && p.splits > 1) {
        float *o = p.partial + ((uint64_t)q.split * (row_tiles<T, OP>(p) * p.tiles_j) + q.tile) * (T::TI * T::TJ);
        o += wave * (NI * NJ * 1024) + lane * 4;
#pragma unroll
        for (int x = 0; x < NI; ++x)
#pragma unroll
            for (int y = 0; y < NJ; ++y)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x4 v = {acc[x][y][4 * r], acc[x][y][4 * r + 1], acc[x][y][4 * r + 2], acc[x][y][4 * r + 3]};
                    *(f32x4 *)(o + ((x * NJ + y) * 4 + r) * 256) = v;
                }
        return;
    }
    __syncthreads();                        // every wave has read its last stage
    static_assert(T::W * Turn<NJ>::kBytes <= S * T::kStage, "the turned tiles fit the stages' LDS");
    if constexpr (OP == kOpRowStats)
        finish_stats<T>(p, acc, q, wi, wave, (lds_char *)lds);
    else
        finish<NI, NJ, OP>(p, acc, q.group, q.i0 + wi, q.i1, q.j0 + (kGated ? wj / 2 : wj), q.zero,
                           (lds_char *)lds + wave * Turn<NJ>::kBytes);
}

// ------------------------------------------------------------- wide stages
//
// 256 x 256 tiles of bf16 by four waves of 128 x 128, the only ones of their
// SIMDs: all 512 registers, half of them sums.  A stage is 128 bytes of the
// contraction, whole lines of either factor; A has two stages in LDS, B, which
// may come from HBM, three.  The waves read 128 KB of LDS for the 64 KB of a stage
// (eight waves of 128 x 64: 192); LDS gives 128 bytes a clock, and with what is
// written the matrix units' full rate would take all of that from eight waves.
// Logits of 4096 x 32768 x 8192, maxima and sums only: 1.36 PFLOP/s (1.99 of
// zeros, without the power limit), by eight waves 1.23 (1.59).  What is left is
// the first loads and the epilogue, some 10 us a tile (4096 x 32768 x 2048: 1.17,
// of zeros 1.65).  One workgroup a CU that goes from tile to tile, the next one's
// first stages on the way during the epilogue, was slower by 5 to 10%: what it
// has to decide stands between the matrix instructions of the one wave of a SIMD.
//
// The matrix instructions are inline assembly, since the compiler moves the sums
// between registers where it may choose them; a wait follows the last one.  One
// or two other instructions go between two of them, spread by hand.
struct Wide {
    static constexpr int TI = 256, TJ = 256, WI = 2, WJ = 2, NI = 4, NJ = 4, W = 4, THREADS = 64 * W;
    static constexpr int kSlot = 256 * 128;             // a factor's stage
    static constexpr int kSlotsA = 2, kSlotsB = 3, kBAt = kSlotsA * kSlot;
    static constexpr int kDepth = 64, kLoads = 8;       // of the contraction; a wave's loads of a factor's stage
};

// One factor.  Rows contiguous along the contraction: row r at r * 128, its
// eight 16-byte chunks in the order chunk ^ (r / 2 % 8).  Contraction
// outermost: as in Factor.  GATED: 32 rows of the first half of B and 32 of the
// second by turns, a load's rows in one of them.
template <bool OUTER, bool GATED>
struct WideFactor {
    static constexpr int kHalves = GATED ? 2 : 1;
    uint32_t off[Wide::kLoads];                         // per lane
    uint64_t step, base[kHalves];
    int64_t left[kHalves];
    i32x4 d[kHalves];
    uint32_t rest, out;                                 // rest: bytes of a row to come

    // the tile's first row and rows, where the second half begins, and the contraction's range
    __device__ __forceinline__ void init(const void *p, uint64_t stride, uint64_t row0, uint64_t second, uint32_t rows,
                                         uint32_t c0, uint32_t c1, uint32_t wave, uint32_t lane) {
        const uint64_t sb = stride * 2;
        step = OUTER ? Wide::kDepth * sb : 128;
        rest = (c1 - c0) * 2;
#pragma unroll
        for (int n = 0; n < Wide::kLoads; ++n) {
            const uint32_t q = n * Wide::W + wave;
            if constexpr (OUTER) {
                const uint32_t c = q * 2 + (lane >> 5), pos = lane & 31, h = unit_order(c, 256);
                off[n] = c * (uint32_t)sb + ((((pos >> 1) ^ h) << 1) | (pos & 1)) * 16;
            } else {
                const uint32_t r = q * 8 + (lane >> 3), row = GATED ? r / 64 * 32 + r % 32 : r;
                off[n] = row * (uint32_t)sb + ((lane & 7) ^ ((r >> 1) & 7)) * 16;
            }
        }
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const uint64_t row = row0 + (h ? second : 0);
            base[h] = (uint64_t)p + (OUTER ? c0 * sb + row * 2 : row * sb + (uint64_t)c0 * 2);
            left[h] = OUTER ? ((int64_t)(c1 - c0) - 1) * (int64_t)sb + rows * 2
                            : ((int64_t)rows - 1) * (int64_t)sb + (int64_t)(c1 - c0) * 2;
            left[h] = (left[h] + 3) & ~3ll;
        }
    }

    // Makes the next stage the one to load, in two parts of a few instructions each and a half.
    __device__ __forceinline__ void next(int part, uint32_t wave, uint32_t lane) {
        const int h = part / 2 % kHalves;
        if (part % 2 == 0) {
            const int32_t high = (int32_t)(left[h] >> 32);
            const uint32_t low = (uint32_t)left[h], n = high < 0 ? 0 : high > 0 || low > 0x7FFFFFFFu ? 0x7FFFFFFFu : low;
            d[h][2] = __builtin_amdgcn_readfirstlane((int)(rest ? n : 0));
            left[h] -= (int64_t)step;
        } else {
            d[h][0] = __builtin_amdgcn_readfirstlane((int)base[h]);
            d[h][1] = __builtin_amdgcn_readfirstlane((int)(base[h] >> 32) & 0xFFFF);
            d[h][3] = 0x00027000;
            base[h] += step;
            if (h == kHalves - 1) {
                out = 0;
                if constexpr (!OUTER) out = ((lane & 7) ^ ((wave * 4 + (lane >> 4)) & 7)) * 16 < rest ? 0 : kOutside;
                rest = rest > 128 ? rest - 128 : 0;
            }
        }
    }

    // Load k of the stage, to `at` in LDS.  The descriptor was made five
    // instructions before, or more; m0 needs one wait.
    __device__ __forceinline__ void load(int k, uint32_t at, uint32_t wave) {
        const uint32_t q = k * Wide::W + wave;
        const i32x4 &from = d[GATED ? k & 1 : 0];
        asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off[k] | out), "s"(from),
                     "{m0}"(at + q * 1024)
                     : "memory");
    }

    __device__ __forceinline__ void load_all(uint32_t at, uint32_t wave, uint32_t lane) {
#pragma unroll
        for (int part = 0; part < 2 * kHalves; ++part) next(part, wave, lane);
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 4" ::: "memory");
#pragma unroll
        for (int k = 0; k < Wide::kLoads; ++k) load(k, at, wave);
    }
};

template <bool OUTER>
struct WideFragments {
    static __device__ __forceinline__ uint32_t at(uint32_t wave_row, int t, uint32_t lane) {
        if constexpr (OUTER)
            return Fragments<256, 4, true>::at(wave_row, t, lane);
        else
            return (wave_row + t * 32 + (lane & 31)) * 128 + ((lane >> 5) ^ ((lane >> 1) & 7)) * 16;
    }

    // Quarter s of tile t.
    static __device__ __forceinline__ u32x4 read(lds_char *stage, const uint32_t *offs, int t, int s) {
        if constexpr (OUTER) {
            union {
                s16x4 h[2];
                u32x4 w;
            } u;
            u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(stage + offs[t] + s * 16 * 512));
            u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(stage + offs[t] + (s * 16 + 4) * 512));
            return u.w;
        } else {
            return *(lds_u32x4 *)(stage + (offs[0] ^ (s * 32)) + t * 4096);
        }
    }
};

template <int OP, int ACT>
__global__ __launch_bounds__(Wide::THREADS, 1) void wide_kernel(ProductArgs p) {
    using T = Wide;
    constexpr bool kOuterA = contracts_a_rows(OP), kOuterB = contracts_b_rows(OP), kGated = OP == kOpGated;
    using FA = WideFactor<kOuterA, false>;
    using FB = WideFactor<kOuterB, kGated>;
    using RA = WideFragments<kOuterA>;
    using RB = WideFragments<kOuterB>;
    __shared__ __attribute__((aligned(1024))) char lds[(T::kSlotsA + T::kSlotsB) * T::kSlot];
    if (!counts_rows(OP) && p.groups && blockIdx.x == 0 && threadIdx.x < 64)
        check_offsets(p.offsets, p.groups, kOuterA ? p.C : p.I, p.status);
    const Place q = find_place<T, OP>(p, blockIdx.x);
    if (q.none) return;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t wi = wave / 2 * 128, wj = wave % 2 * 128;
    lds_char *const mem = (lds_char *)lds;
    // the split's range, in stages of the other tiles, so that its sums are theirs
    uint32_t c0 = q.c0, c1 = q.c1;
    if (kJoins<OP> && p.splits > 1) {
        const uint32_t stages = (c1 + 31) / 32;
        c0 = (uint32_t)((uint64_t)stages * q.split / p.splits) * 32;
        c1 = min(c1, (uint32_t)((uint64_t)stages * (q.split + 1) / p.splits) * 32);
    }
    f32x16 acc[2][4][2];                                // [64 columns][32 rows][32 columns]
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[h][x][y][r] = 0.0f;
    if (c1 > c0) {
        const uint32_t n = (c1 - c0 + T::kDepth - 1) / T::kDepth, mem_at = (uint32_t)(uintptr_t)mem;
        FA fa;
        FB fb;
        fa.init(p.a, kOuterA ? p.a_c : p.a_i, q.i0, 0, q.i1 - q.i0, c0, c1, wave, lane);
        fb.init((const char *)p.b + (kOuterA ? 0 : q.group * p.b_group * 2), kOuterB ? p.b_c : p.b_j, q.j0, p.J,
                min(kGated ? 128u : 256u, p.J - q.j0), c0, c1, wave, lane);
        uint32_t ao[4], bo[4], a_read = 0, b_read = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            ao[t] = RA::at(wi, t, lane);
            bo[t] = T::kBAt + RB::at(wj, t, lane);
        }
        u32x4 af[2][2][4], bf[2][2][4];                 // [half of a stage][quarter of it][tile]
        const auto read = [&](int r, int half) __attribute__((always_inline)) {     // of 16, in the order of their use
            const int s = r / 8, t = r % 8;
            if (t < 4)
                bf[half][s][t] = RB::read(mem + b_read, bo, t, half * 2 + s);
            else
                af[half][s][t - 4] = RA::read(mem + a_read, ao, t - 4, half * 2 + s);
        };
        fa.load_all(mem_at, wave, lane);
        fb.load_all(mem_at + T::kBAt, wave, lane);
        fb.load_all(mem_at + T::kBAt + T::kSlot, wave, lane);
        fa.load_all(mem_at + T::kSlot, wave, lane);
        fb.load_all(mem_at + T::kBAt + 2 * T::kSlot, wave, lane);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * T::kLoads) : "memory");     // the first stage has arrived, everywhere
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int r = 0; r < 16; ++r) read(r, 0);
        // A stage: in its first half its second half's fragments are read;
        // then, when every wave has them, its slots take the stages two (A) and
        // three (B) later, and the next stage's first fragments are read.  At
        // that point all loads but the last eight, of B two stages ahead, must
        // have arrived.
        for (uint32_t k = 0; k < n; ++k) {
            const uint32_t a_fill = mem_at + a_read, b_fill = mem_at + T::kBAt + b_read;
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int g = 0; g < 64; ++g) {
                const int half = g / 32, s = g / 16 % 2, x = g / 4 % 4, y = g % 4;
                if (g == 32) {
                    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(T::kLoads) : "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    a_read ^= T::kSlot;
                    b_read = b_read == 2 * T::kSlot ? 0 : b_read + T::kSlot;
                    __builtin_amdgcn_sched_barrier(0);
                }
                asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0"
                             : "+a"(acc[y / 2][x][y % 2])
                             : "v"(bf[half][s][y]), "v"(af[half][s][x]));
                if (g % 32 < 16) read(g % 32, 1 - half);
                if (g == 16 || g == 17) fa.next(g - 16, wave, lane);
                if (g >= 18 && g < 18 + 2 * FB::kHalves) fb.next(g - 18, wave, lane);
                if (g >= 32 && g % 2 == 1) {
                    const int l = (g - 33) / 2;
                    if (l < T::kLoads)
                        fa.load(l, a_fill, wave);
                    else
                        fb.load(l - T::kLoads, b_fill, wave);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // nothing is left in flight into this workgroup's LDS; the last products' results
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) asm volatile("" : "+a"(acc[h][x][y]));
    if (kJoins<OP> && p.splits > 1) {
        float *o = p.partial + ((uint64_t)q.split * (row_tiles<T, OP>(p) * p.tiles_j) + q.tile) * (T::TI * T::TJ);
        o += wave * (16 * 1024) + lane * 4;
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const f32x16 &v = acc[y / 2][x][y % 2];
                    *(f32x4 *)(o + ((x * 4 + y) * 4 + r) * 256) = f32x4{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
                }
        return;
    }
    __syncthreads();                                    // every wave has read its last stage
    if constexpr (OP == kOpRowStats) {
        finish_stats<T>(p, acc, q, wi, wave, mem);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            finish_act<4, 2, OP, ACT>(p, acc[h], q.group, q.i0 + wi, q.i1, q.j0 + (kGated ? wj / 2 + h * 32 : wj + h * 64), q.zero,
                                      mem + wave * Turn<2>::kBytes);
    }
}

// Adds the splits' sums in their order and finishes: a workgroup takes one
// 32 x 32 tile of each of the four waves of a tile.
template <class T, int OP>
__global__ __launch_bounds__(T::THREADS) void join_kernel(ProductArgs p) {
    constexpr int NI = T::NI, NJ = T::NJ;
    __shared__ __attribute__((aligned(1024))) char lds[T::W * Turn<1>::kBytes];
    const uint32_t tile = blockIdx.x / (NI * NJ), xy = blockIdx.x - tile * (NI * NJ), x = xy / NJ, y = xy - x * NJ;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t tiles_i = row_tiles<T, OP>(p);
    const uint64_t tiles = (uint64_t)tiles_i * p.tiles_j;
    if (tile >= tiles) return;
    uint32_t ti, tj;
    band_order(tile, tiles_i, p.tiles_j, &ti, &tj);
    f32x16 acc[1][1] = {};
    const float *o = p.partial + (uint64_t)tile * (T::TI * T::TJ) + wave * (NI * NJ * 1024) + xy * 1024 + lane * 4;
#pragma unroll 4                            // loads of four splits on the way
    for (uint32_t s = 0; s < p.splits; ++s, o += tiles * (T::TI * T::TJ))
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const f32x4 v = *(const f32x4 *)(o + r * 256);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[0][0][4 * r + k] += v[k];
        }
    const uint32_t i0 = ti * T::TI, wi = wave / T::WJ * (NI * 32) + x * 32, wj = wave % T::WJ * (NJ * 32) + y * 32;
    uint32_t end = p.I;
    if constexpr (counts_rows(OP) && !contracts_a_rows(OP)) end = min(end, *p.used);
    finish<1, 1, OP>(p, acc, 0, i0 + wi, min(end, i0 + T::TI), tj * T::TJ + wj, false,
                      (lds_char *)lds + wave * Turn<1>::kBytes);
}

// The same for the gated product: of each wave the 32 rows of one NI, with the
// columns of the gate and those it is multiplied by.
template <class T>
__global__ __launch_bounds__(T::THREADS) void join_gated_kernel(ProductArgs p) {
    constexpr int NI = T::NI, N = T::NJ > 2 ? 2 : T::NJ, PAIRS = T::NJ / N;    // 32 x 32 tiles taken at a time
    __shared__ __attribute__((aligned(1024))) char lds[T::W * Turn<N>::kBytes];
    const uint32_t part = blockIdx.x % (NI * PAIRS), tile = blockIdx.x / (NI * PAIRS), x = part / PAIRS, pair = part % PAIRS;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t tiles = (uint64_t)p.tiles_i * p.tiles_j;
    uint32_t ti, tj;
    band_order(tile, p.tiles_i, p.tiles_j, &ti, &tj);
    f32x16 acc[1][N] = {};
    const float *o = p.partial + (uint64_t)tile * (T::TI * T::TJ) + wave * (NI * T::NJ * 1024) +
                     (x * T::NJ + pair * N) * 1024 + lane * 4;
#pragma unroll 2                            // loads of two splits on the way
    for (uint32_t s = 0; s < p.splits; ++s, o += tiles * (T::TI * T::TJ))
#pragma unroll
        for (int y = 0; y < N; ++y)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const f32x4 v = *(const f32x4 *)(o + y * 1024 + r * 256);
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[0][y][4 * r + k] += v[k];
            }
    const uint32_t i0 = ti * T::TI, wi = wave / T::WJ * (NI * 32) + x * 32, wj = (wave % T::WJ * T::NJ + pair * N) * 16;
    finish<1, N, kOpGated>(p, acc, 0, i0 + wi, min(p.I, i0 + T::TI), tj * (T::TJ / 2) + wj, false,
                           (lds_char *)lds + wave * Turn<N>::kBytes);
}

// ------------------------------------------------------------------ few rows
//
// Up to 32 rows (of a group): the time is that of reading B once, so nothing
// is staged.  A workgroup takes 16 columns and RT x 16 rows, its W waves a
// part of the contraction each; a lane loads 16 bytes of its column's row of
// B, and of its rows of A, at a time, 64 bytes of a row in a wave's load, and
// the waves' sums are joined in LDS in the waves' order.  One row by 16384 x
// 2048 bf16 weights: 13.6 us (4.9 TB/s); 64 rows over 32 experts of 1024 x
// 2048: 26.8 us (5.0 TB/s); 17 rows by 2048 x 16384 e4m3 weights: 18.3 us, the
// latency of 256 workgroups' loads.
template <int RT, int W>
struct Few {
    static constexpr int TI = RT * 16, TJ = 16;
    static constexpr int kAtOnce = 8;                   // loads of B on the way in a lane
};

// The first n < 16 / ES values at p, and zeros.
template <int ES>
__device__ __forceinline__ u32x4 few_values(const char *p, uint32_t n) {
    u32x4 w = {};
    for (uint32_t k = 0; k < n; ++k) {
        const uint32_t v = ES == 1 ? (uint32_t)((const uint8_t *)p)[k] : (uint32_t)((const uint16_t *)p)[k];
        const uint32_t bit = k * ES * 8;
#pragma unroll
        for (uint32_t d = 0; d < 4; ++d) w[d] |= d == bit / 32 ? v << (bit & 31) : 0;
    }
    return w;
}

template <int RT, bool E4M3>
__device__ __forceinline__ void few_multiply(f32x4 (&acc)[RT], const u32x4 &b, const u32x4 (&a)[RT]) {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if constexpr (E4M3) {
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_to_bf16x8(b[0], b[1]), e4m3_to_bf16x8(a[t][0], a[t][1]),
                                                             acc[t], 0, 0, 0);
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3_to_bf16x8(b[2], b[3]), e4m3_to_bf16x8(a[t][2], a[t][3]),
                                                             acc[t], 0, 0, 0);
        } else {
            acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a[t]),
                                                             acc[t], 0, 0, 0);
        }
    }
}

// The eight sums of a thread's row and columns, over the waves in their order.
template <int RT>
__device__ __forceinline__ void few_sums(const float *sums, uint32_t waves, float *v) {
    const uint32_t t = threadIdx.x;
    for (uint32_t w = 0; w < waves; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 s = *(const f32x4 *)(sums + (w * (RT * 16) + (t >> 1)) * 20 + (t & 1) * 8 + h * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * h + r] += s[r];
        }
}

template <int RT, int ACT>
__device__ __forceinline__ void few_finish(const ProductArgs &p, const Place &q, const float *sums, uint32_t waves) {
    const uint32_t t = threadIdx.x, i = q.i0 + (t >> 1), j = q.j0 + (t & 1) * 8;
    if (t >= RT * 32 || i >= q.i1) return;
    const Columns c = load_columns<EC_LINEAR_FORWARD>(p, q.group, j);
    float side[8], v[8] = {};
    load_side<EC_LINEAR_FORWARD>(p, i, j, c.left, side);
    const float xs = p.x_scale ? p.x_scale[p.x_scales > 1 ? i : 0] : 1.0f, os = p.out_scale ? *p.out_scale : 1.0f;
    few_sums<RT>(sums, waves, v);
    finish8<EC_LINEAR_FORWARD, ACT>(p, q.group, i, j, v, c, side, xs, os, q.zero);
}

template <int RT>
__device__ __forceinline__ void few_stats(const ProductArgs &p, const Place &q, const float *sums, uint32_t waves) {
    const uint32_t t = threadIdx.x, i = q.i0 + (t >> 1), j = q.j0 + (t & 1) * 8;
    if (t >= RT * 32 || i >= q.i1) return;              // both threads of a row
    float v[8] = {};
    few_sums<RT>(sums, waves, v);
    const int64_t at =
        (p.target_bytes == 8 ? ((const int64_t *)p.target)[i] : (int64_t)((const int32_t *)p.target)[i]) - (int64_t)j;
    float2 s = {-__builtin_inff(), 0.0f};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        if (j + c >= p.J) v[c] = -__builtin_inff();
        s.x = fmaxf(s.x, v[c]);
        if (c == at && j + c < p.J) p.hit[i] = v[c];
    }
    const float from = s.x == -__builtin_inff() ? 0.0f : s.x;
#pragma unroll
    for (int c = 0; c < 8; ++c) s.y += __builtin_amdgcn_exp2f((v[c] - from) * kLog2E);
    const float2 other = {__shfl_xor(s.x, 1), __shfl_xor(s.y, 1)};
    if (!(t & 1)) p.stats[(uint64_t)i * p.tiles_j + q.j0 / 16] = join_stats(s, other);
}

template <int RT>
__device__ __forceinline__ void few_logits(const ProductArgs &p, const Place &q, const float *sums, uint32_t waves) {
    const uint32_t t = threadIdx.x, i = q.i0 + (t >> 1), j = q.j0 + (t & 1) * 8;
    if (t >= RT * 32 || i >= q.i1 || j >= p.J) return;
    float v[8] = {};
    few_sums<RT>(sums, waves, v);
    finish8_logits(p, i, j, v, p.row[i], p.row_target[i]);
}

template <int RT, int W, bool E4M3, int OP = EC_LINEAR_FORWARD>
__global__ __launch_bounds__(W * 64) void few_rows_kernel(ProductArgs p) {
    using T = Few<RT, W>;
    constexpr int ES = E4M3 ? 1 : 2, U = T::kAtOnce;
    __shared__ __attribute__((aligned(16))) float sums[W * RT * 16 * 20];   // [wave][row][16 columns and a gap]
    if (OP == EC_LINEAR_FORWARD && p.groups && blockIdx.x == 0 && threadIdx.x < 64)
        check_offsets(p.offsets, p.groups, p.I, p.status);
    const Place q = find_place<T, OP>(p, blockIdx.x);
    if (q.none) return;
    const uint32_t lane = threadIdx.x & 63, row = lane & 15, part = (lane >> 4) * 16;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    // rows and columns that do not exist repeat the last one: their sums are not stored
    const char *b = (const char *)p.b + (q.group * p.b_group + min(q.j0 + row, p.J - 1) * p.b_j) * ES + part;
    const char *a[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) a[t] = (const char *)p.a + min(q.i0 + t * 16 + row, q.i1 - 1) * p.a_i * ES + part;
    const uint64_t bytes = (uint64_t)(q.c1 - q.c0) * ES;
    const uint32_t steps = (uint32_t)((bytes + 63) / 64), whole = (uint32_t)(bytes / 64);
    uint32_t s = (uint32_t)((uint64_t)steps * wave / W);
    const uint32_t s1 = (uint32_t)((uint64_t)steps * (wave + 1) / W);
    f32x4 acc[RT] = {};
    for (; s + U <= min(s1, whole); s += U) {
        u32x4 vb[U], va[U][RT];
#pragma unroll
        for (int u = 0; u < U; ++u) vb[u] = ((const AnyByteU32x4 *)(b + (uint64_t)(s + u) * 64))->v;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int t = 0; t < RT; ++t) va[u][t] = ((const AnyByteU32x4 *)(a[t] + (uint64_t)(s + u) * 64))->v;
#pragma unroll
        for (int u = 0; u < U; ++u) few_multiply<RT, E4M3>(acc, vb[u], va[u]);
    }
    for (; s < s1; ++s) {
        u32x4 vb = {}, va[RT] = {};
        const uint64_t at = (uint64_t)s * 64 + part;
        if (at + 16 <= bytes) {
            vb = ((const AnyByteU32x4 *)(b + (uint64_t)s * 64))->v;
#pragma unroll
            for (int t = 0; t < RT; ++t) va[t] = ((const AnyByteU32x4 *)(a[t] + (uint64_t)s * 64))->v;
        } else if (at < bytes) {                        // the row's last values
            const uint32_t n = (uint32_t)(bytes - at) / ES;
            vb = few_values<ES>(b + (uint64_t)s * 64, n);
#pragma unroll
            for (int t = 0; t < RT; ++t) va[t] = few_values<ES>(a[t] + (uint64_t)s * 64, n);
        }
        few_multiply<RT, E4M3>(acc, vb, va);
    }
    // the accumulators hold row lane % 16, columns 4 (lane / 16) + r
#pragma unroll
    for (int t = 0; t < RT; ++t) *(f32x4 *)(sums + (wave * (RT * 16) + t * 16 + row) * 20 + (lane >> 4) * 4) = acc[t];
    __syncthreads();
    if constexpr (OP == kOpRowStats) {
        few_stats<RT>(p, q, sums, W);
        return;
    } else if constexpr (OP == kOpLogitGrad) {
        few_logits<RT>(p, q, sums, W);
        return;
    }
    switch (p.act) {
        case EC_ACT_GELU: few_finish<RT, EC_ACT_GELU>(p, q, sums, W); break;
        case EC_ACT_SILU: few_finish<RT, EC_ACT_SILU>(p, q, sums, W); break;
        case EC_ACT_RELU: few_finish<RT, EC_ACT_RELU>(p, q, sums, W); break;
        default: few_finish<RT, EC_ACT_NONE>(p, q, sums, W);
    }
}

}  // namespace

// How a product is launched: tiles or few rows, splits of the contraction, copied factors.
struct Plan {
    uint32_t shape, splits, tiles_i, tiles_j;
    uint32_t row_tiles, waves;              // kFew
    uint64_t blocks;
    uint32_t a_pitch, b_pitch;              // elements; 0: read in place
    bool none;                              // rows too long, or tiles too many, for every shape
    uint64_t a_at, b_at, partial_at, bytes; // workspace
};

inline uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
inline uint64_t round_up(uint64_t a, uint64_t b) { return ceil_div(a, b) * b; }

// A launch has fewer than 2^32 threads; of one with more, only the rest by
// 2^32 would run, without an error.
inline bool launchable(uint64_t blocks, uint64_t threads) { return blocks * threads < (1ull << 32); }

Plan make_plan(const ProductArgs &a);

// Copies the factors that the plan has copied and fills in what it decides.
hipError_t place_product(ProductArgs &a, const Plan &q, void *workspace, hipStream_t s);

namespace {

// Whether the tiles of 256 x 256 are Wide's: where the contraction of a
// workgroup is long, since four waves take longer for what surrounds it.  Gated
// 2048 x 2 x 16384 by a contraction of 1024 165.5 us so and 158.5 by eight
// waves, 1280 191.9 and 191.5, 1536 212.5 and 218.9, 2048 260.6 and 268.4; loss
// with gradients of M x 65536 x 2048, where M is the weight gradient's: 1024
// 1015 and 990, 1536 1551 and 1542, 2048 1835 and 1843.  An epilogue that stores
// nothing does not weigh: maxima and sums of 1023 x 50001 x 1000 logits 152 and
// 164 us, 4096 x 131072 x 2048 1902 and 2027.  Where the contraction is outermost
// a stage's 64 rows must be within 2 GiB, twice what the other tiles' 32 need.
// The plan's costs are those of the eight waves: it chooses the tiles, not these.
inline bool runs_wide(const ProductArgs &a, const Plan &q) {
    const uint32_t parts = contracts_a_rows(a.op) && a.groups ? a.groups : q.splits;
    const auto far = [](uint64_t stride) { return Wide::kDepth * stride * 2 + 65536 >= 1ull << 31; };
    if ((contracts_a_rows(a.op) && far(a.a_c)) || (contracts_b_rows(a.op) && far(a.b_c))) return false;
    return q.shape == kHuge && a.dtype == EC_BF16 && (a.op == kOpRowStats || a.C / parts >= 1536);
}

template <int OP, int ACT>
void launch_wide(const ProductArgs &a, const Plan &q, hipStream_t s) {
    wide_kernel<OP, ACT><<<(uint32_t)q.blocks, Wide::THREADS, 0, s>>>(a);
    if constexpr (OP == kOpGated) {
        if (q.splits > 1) join_gated_kernel<Wide><<<q.tiles_i * q.tiles_j * 8, Wide::THREADS, 0, s>>>(a);
    } else if constexpr (kJoins<OP>) {
        if (q.splits > 1) join_kernel<Wide, OP><<<q.tiles_i * q.tiles_j * 16, Wide::THREADS, 0, s>>>(a);
    }
}

}  // namespace

}  // namespace ec
