// Matrix products with a fused epilogue, dense and grouped by expert.
#include <string.h>

#include "ffn_common.h"

namespace ec {
namespace {

typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

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
// 128 x 64 keep two waves a SIMD; four of 128 x 128 need all registers and
// spill.  4096 x 16384 x 2048 bf16 with GELU and e4m3 output: 306 us (0.90
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
template <int T, bool OUTER, int ES, int W>
struct Factor {
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
                off[n] = r * (uint32_t)sb + ((lane & 3) ^ ((r >> 2) & 3)) * 16;
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

template <int NI, int NJ, int OP>
__device__ __forceinline__ void finish(const ProductArgs &p, f32x16 (&acc)[NI][NJ], uint32_t g, uint32_t i0,
                                       uint32_t i1, uint32_t j0, bool zero, lds_char *mem) {
    if constexpr (OP == EC_LINEAR_GRAD_WEIGHT) {
        finish_tiles<NI, NJ, OP, EC_ACT_NONE>(p, acc, g, i0, i1, j0, zero, mem);
    } else {
        switch (p.act) {
            case EC_ACT_GELU: finish_tiles<NI, NJ, OP, EC_ACT_GELU>(p, acc, g, i0, i1, j0, zero, mem); break;
            case EC_ACT_SILU: finish_tiles<NI, NJ, OP, EC_ACT_SILU>(p, acc, g, i0, i1, j0, zero, mem); break;
            case EC_ACT_RELU: finish_tiles<NI, NJ, OP, EC_ACT_RELU>(p, acc, g, i0, i1, j0, zero, mem); break;
            default: finish_tiles<NI, NJ, OP, EC_ACT_NONE>(p, acc, g, i0, i1, j0, zero, mem);
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

struct Place {
    uint32_t i0, i1, j0, c0, c1, group, split, tile;
    bool zero, none;
};

template <class T, int OP>
__device__ __forceinline__ Place find_place(const ProductArgs &p, uint32_t block) {
    Place q = {};
    uint32_t ti, tj;
    q.c1 = p.C;
    if (p.groups && OP != EC_LINEAR_GRAD_WEIGHT) {
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
    q.j0 = tj * T::TJ;
    return q;
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
    constexpr bool kOuterA = OP == EC_LINEAR_GRAD_WEIGHT, kOuterB = OP != EC_LINEAR_FORWARD;
    constexpr int kES = E4M3 ? 1 : 2, kDepth = kStageBytes / kES;
    constexpr int NI = T::NI, NJ = T::NJ, S = T::S;
    using FA = Factor<T::TI, kOuterA, kES, T::W>;
    using FB = Factor<T::TJ, kOuterB, kES, T::W>;
    using RA = Fragments<T::TI, NI, kOuterA>;
    using RB = Fragments<T::TJ, NJ, kOuterB>;
    __shared__ __attribute__((aligned(1024))) char lds[S * T::kStage];

    if (p.groups && blockIdx.x == 0 && threadIdx.x < 64)
        check_offsets(p.offsets, p.groups, OP == EC_LINEAR_GRAD_WEIGHT ? p.C : p.I, p.status);
    const Place q = find_place<T, OP>(p, blockIdx.x);
    if (q.none) return;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t wi = wave / T::WJ * (NI * 32), wj = wave % T::WJ * (NJ * 32);

    // the split's range of stages
    uint32_t c0 = q.c0, c1 = q.c1;
    if (p.splits > 1) {
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
        const void *b = (const char *)p.b + (OP == EC_LINEAR_GRAD_WEIGHT ? 0 : q.group * p.b_group * kES);
        FA fa;
        FB fb;
        fa.init(a, kOuterA ? p.a_c : p.a_i, q.i0, q.i1 - q.i0, c0, c1, wave, lane);
        fb.init(b, kOuterB ? p.b_c : p.b_j, q.j0, min((uint32_t)T::TJ, p.J - q.j0), c0, c1, wave, lane);
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
    if (p.splits > 1) {
        float *o = p.partial + ((uint64_t)q.split * (p.tiles_i * p.tiles_j) + q.tile) * (T::TI * T::TJ);
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
    finish<NI, NJ, OP>(p, acc, q.group, q.i0 + wi, q.i1, q.j0 + wj, q.zero, (lds_char *)lds + wave * Turn<NJ>::kBytes);
}

// Adds the splits' sums in their order and finishes: a workgroup takes one
// 32 x 32 tile of each of the four waves of a tile.
template <class T, int OP>
__global__ __launch_bounds__(T::THREADS) void join_kernel(ProductArgs p) {
    constexpr int NI = T::NI, NJ = T::NJ;
    __shared__ __attribute__((aligned(1024))) char lds[T::W * Turn<1>::kBytes];
    const uint32_t tile = blockIdx.x / (NI * NJ), xy = blockIdx.x - tile * (NI * NJ), x = xy / NJ, y = xy - x * NJ;
    const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t tiles = (uint64_t)p.tiles_i * p.tiles_j;
    uint32_t ti, tj;
    band_order(tile, p.tiles_i, p.tiles_j, &ti, &tj);
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
    finish<1, 1, OP>(p, acc, 0, i0 + wi, min(p.I, i0 + T::TI), tj * T::TJ + wj, false,
                      (lds_char *)lds + wave * Turn<1>::kBytes);
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

template <int RT, int ACT>
__device__ __forceinline__ void few_finish(const ProductArgs &p, const Place &q, const float *sums, uint32_t waves) {
    const uint32_t t = threadIdx.x, i = q.i0 + (t >> 1), j = q.j0 + (t & 1) * 8;
    if (t >= RT * 32 || i >= q.i1) return;
    const Columns c = load_columns<EC_LINEAR_FORWARD>(p, q.group, j);
    float side[8], v[8] = {};
    load_side<EC_LINEAR_FORWARD>(p, i, j, c.left, side);
    const float xs = p.x_scale ? p.x_scale[p.x_scales > 1 ? i : 0] : 1.0f, os = p.out_scale ? *p.out_scale : 1.0f;
    for (uint32_t w = 0; w < waves; ++w)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x4 s = *(const f32x4 *)(sums + (w * (RT * 16) + (t >> 1)) * 20 + (t & 1) * 8 + h * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * h + r] += s[r];
        }
    finish8<EC_LINEAR_FORWARD, ACT>(p, q.group, i, j, v, c, side, xs, os, q.zero);
}

template <int RT, int W, bool E4M3>
__global__ __launch_bounds__(W * 64) void few_rows_kernel(ProductArgs p) {
    using T = Few<RT, W>;
    constexpr int ES = E4M3 ? 1 : 2, U = T::kAtOnce;
    __shared__ __attribute__((aligned(16))) float sums[W * RT * 16 * 20];   // [wave][row][16 columns and a gap]
    if (p.groups && blockIdx.x == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.I, p.status);
    const Place q = find_place<T, EC_LINEAR_FORWARD>(p, blockIdx.x);
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
    switch (p.act) {
        case EC_ACT_GELU: few_finish<RT, EC_ACT_GELU>(p, q, sums, W); break;
        case EC_ACT_SILU: few_finish<RT, EC_ACT_SILU>(p, q, sums, W); break;
        case EC_ACT_RELU: few_finish<RT, EC_ACT_RELU>(p, q, sums, W); break;
        default: few_finish<RT, EC_ACT_NONE>(p, q, sums, W);
    }
}

// ------------------------------------------------------- rows made readable
//
// The loads above take rows at 16-byte addresses whose contraction is a whole
// number of 16-byte chunks.  Any other factor is copied first: rows padded
// with zeros to 16 bytes, one after the other.
struct RowCopy {
    const void *p;
    uint64_t stride, group_stride, total;  // elements; total: 16-byte chunks of all groups
    uint32_t rows, cols, pitch;            // pitch of the copy's rows, elements
    void *out;
    uint32_t blocks;                       // 0: none
};

// Both factors in one launch: the first a.blocks workgroups copy a's.
template <typename E>
__global__ __launch_bounds__(256) void copy_rows_kernel(RowCopy a, RowCopy b) {
    constexpr uint32_t V = 16 / sizeof(E);
    const bool first = blockIdx.x < a.blocks;
    const RowCopy &k = first ? a : b;
    const uint32_t chunks = k.pitch / V;
    const uint64_t q = (uint64_t)(blockIdx.x - (first ? 0 : a.blocks)) * 256 + threadIdx.x;
    if (q >= k.total) return;
    uint64_t row, g;
    if (k.total >> 32) {
        row = q / chunks;
        g = row / k.rows;
    } else {                                // the same in short divisions
        row = (uint32_t)q / chunks;
        g = (uint32_t)row / k.rows;
    }
    const uint32_t c = (uint32_t)(q - row * chunks) * V;
    const E *in = (const E *)k.p + g * k.group_stride + (row - g * k.rows) * k.stride + c;
    union {
        E e[V];
        u32x4 w;
    } u;
    if (c + V <= k.cols) {
        u.w = ((const AnyByteU32x4 *)in)->v;
    } else {
        u.w = u32x4{0, 0, 0, 0};
#pragma unroll
        for (uint32_t n = 0; n < V; ++n)
            if (c + n < k.cols) u.e[n] = in[n];
    }
    ((u32x4 *)k.out)[q] = u.w;
}

// ---------------------------------------------------------------- column sums
//
// db[n] = sum of dy's rows.  A workgroup takes 128 columns of one part of a
// group's rows, 16 threads of eight columns by 16 rows; where that alone does
// not fill the card the rows are cut into parts, added in their order after.
constexpr uint32_t kSumCols = 128;

__global__ __launch_bounds__(256) void column_sum_kernel(ColumnSumArgs p, float *out, uint32_t parts) {
    __shared__ float sh[16][kSumCols + 4];
    const uint32_t g = blockIdx.y, part = blockIdx.z;
    uint32_t lo = 0, hi = p.m;
    if (p.groups) {
        if (blockIdx.x == 0 && g == 0 && part == 0 && threadIdx.x < 64) check_offsets(p.offsets, p.groups, p.m, p.status);
        group_range(p.offsets, p.m, g, &lo, &hi);
    }
    const uint64_t len = hi - lo;
    hi = lo + (uint32_t)(len * (part + 1) / parts);
    lo += (uint32_t)(len * part / parts);
    const uint32_t x = (threadIdx.x & 15) * 8, y = threadIdx.x >> 4, n = blockIdx.x * kSumCols + x;
    const uint32_t left = p.n > n ? p.n - n : 0;
    float s[8] = {};
    if (left) {
        uint32_t i = lo + y;
        for (; i + 48 < hi; i += 64) {      // four rows on the way at a time
            float v[4][8];
#pragma unroll
            for (int k = 0; k < 4; ++k) load8_bf16(p.dy, (uint64_t)(i + 16 * k) * p.dy_stride + n, left, v[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int q = 0; q < 8; ++q) s[q] += v[k][q];
        }
        for (; i < hi; i += 16) {
            float v[8];
            load8_bf16(p.dy, (uint64_t)i * p.dy_stride + n, left, v);
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q] += v[q];
        }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) sh[y][x + q] = s[q];
    __syncthreads();
    const uint32_t c = blockIdx.x * kSumCols + threadIdx.x;
    if (threadIdx.x >= kSumCols || c >= p.n) return;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += sh[k][threadIdx.x];
    out[((uint64_t)part * gridDim.y + g) * p.n + c] = t;
}

__global__ __launch_bounds__(256) void column_join_kernel(const float *in, float *db, uint64_t n, uint32_t parts) {
    const uint64_t c = (uint64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= n) return;
    float s = 0.0f;
#pragma unroll 8                            // loads of eight parts on the way
    for (uint32_t q = 0; q < parts; ++q) s += in[q * n + c];
    db[c] = s;
}

// For a grouped product that has nothing to compute.
__global__ __launch_bounds__(64) void check_offsets_kernel(const int32_t *offsets, uint32_t groups, uint32_t m,
                                                           uint32_t *status) {
    check_offsets(offsets, groups, m, status);
}

// ---------------------------------------------------------------------- plan

using Huge = Shape<256, 256, 2, 4, 4, 1>;
using Even = Shape<128, 128, 2, 2, 4, 2>;
using Small = Shape<64, 64, 2, 2, 6, 3>;

enum ShapeId { kHuge, kEven, kSmall, kFew };

// What a plan's time is made of, measured on whole runs (us): a stage of one
// workgroup alone on its CU, a stage per workgroup where every CU is full, and
// what a workgroup costs besides its stages; bf16 and e4m3.  The full rates
// are 1.25, 0.87 and 0.51 PFLOP/s in bf16.
struct ShapeCost {
    uint32_t TI, TJ, threads, per_cu;
    float alone[2], full[2], fixed;
};
constexpr ShapeCost kCost[] = {{256, 256, Huge::THREADS, 1, {0.55f, 1.1f}, {0.86f, 1.5f}, 10.0f},
                               {128, 128, Even::THREADS, 2, {0.25f, 0.43f}, {0.31f, 0.45f}, 5.0f},
                               {64, 64, Small::THREADS, 3, {0.17f, 0.28f}, {0.133f, 0.18f}, 6.0f}};
constexpr uint64_t kCUs = 256;

struct Plan {
    uint32_t shape, splits, tiles_i, tiles_j;
    uint32_t row_tiles, waves;              // kFew
    uint64_t blocks;
    uint32_t a_pitch, b_pitch;              // elements; 0: read in place
    bool none;                              // rows too long, or tiles too many, for every shape
    uint64_t a_at, b_at, partial_at, bytes; // workspace
};

uint64_t ceil_div(uint64_t a, uint64_t b) { return (a + b - 1) / b; }
uint64_t round_up(uint64_t a, uint64_t b) { return ceil_div(a, b) * b; }

bool aligned(const void *p, uint64_t stride, uint64_t group, uint64_t cols, uint32_t es, bool outer) {
    return !((((uintptr_t)p | (stride * es) | (group * es)) & 15) || (!outer && (cols * es & 15)));
}

// Whether the offsets of a stage's rows fit 31 bits: T rows of a tile where
// they are contiguous along the contraction, or the stage's rows of it.
bool reachable(uint64_t T, uint64_t stride, uint32_t es, bool outer) {
    return (outer ? kStageBytes / es : T) * stride * es + 65536 < (1ull << 31);
}

// A launch has fewer than 2^32 threads; of one with more, only the rest by
// 2^32 would run, without an error.
bool launchable(uint64_t blocks, uint64_t threads) { return blocks * threads < (1ull << 32); }

Plan make_plan(const ProductArgs &a) {
    Plan q;
    memset(&q, 0, sizeof(q));
    const uint32_t es = a.dtype == EC_E4M3 ? 1 : 2;
    const bool outer_a = a.op == EC_LINEAR_GRAD_WEIGHT, outer_b = a.op != EC_LINEAR_FORWARD;
    const bool ragged = a.groups && !outer_a;
    const uint64_t groups = a.groups ? a.groups : 1;
    q.splits = 1;
    // Row tiles of a ragged product: at most one begun a group besides the whole ones.
    const auto most_tiles = [&](uint64_t tile) {
        return ragged ? a.I / tile + (a.I < groups + 2 ? a.I : groups + 2) : ceil_div(a.I, tile);
    };
    const auto few = [&](uint32_t row_tiles) {          // reads rows at any address, of any length
        q.shape = kFew;
        q.tiles_j = (uint32_t)ceil_div(a.J, 16);
        q.row_tiles = row_tiles;
        q.tiles_i = (uint32_t)most_tiles(16 * q.row_tiles);
        // Waves that share a contraction: with 1024 tiles four are enough
        // (16.4 us; 16.2 with eight), with 128 eight are better (13.4, 16.1).
        q.waves = (ragged ? groups : q.tiles_i) * q.tiles_j >= 2 * kCUs ? 4 : 8;
        q.blocks = (uint64_t)q.tiles_i * q.tiles_j;
        return launchable(q.blocks, q.waves * 64);
    };
    // Few rows a group, forward: one row by 16384 x 2048 weights takes 13.5 us
    // so, 20 us in tiles with a split contraction and its join.  17 to 32 rows:
    // one tile of 32 reads the weights once, but two of 16 use twice as many
    // CUs, so that the tiles of 16 columns must be enough for them all (17 rows:
    // 16384 columns 24 against 32 us, 2048 columns of 16384 e4m3 values 22
    // against 18), twice over by group, where rows are uneven (20 rows by 1024 x
    // 2048 a group, 32 groups: 50 us against 64, e4m3 22 against 38; uneven 61
    // against 58, e4m3 30 against 34; four uneven groups 13.7 against 12.3).
    // The average decides, since the host does not know the offsets: 1024 rows
    // of which 962 are in one of 32 groups take 90 us so and 45 in tiles.
    const uint64_t rows = ragged ? ceil_div(a.I, groups) : a.I;
    if (a.op == EC_LINEAR_FORWARD && rows <= 32) {
        const bool fill = ceil_div(a.J, 16) * groups >= (ragged ? 2 : 1) * kCUs;
        if (few(rows > 16 && fill ? 2 : 1)) return q;
    }
    // The tiles and the number of splits with the least time, of the shapes
    // whose tiles reach their rows: where these lie, or else in a copy.
    const uint64_t a_rows = outer_a ? a.C : a.I, a_cols = outer_a ? a.I : a.C, a_stride = outer_a ? a.a_c : a.a_i;
    const uint64_t b_rows = outer_b ? a.C : a.J, b_cols = outer_b ? a.J : a.C, b_stride = outer_b ? a.b_c : a.b_j;
    const uint64_t a_pitch = round_up(a_cols, 16 / es), b_pitch = round_up(b_cols, 16 / es);
    const bool a_aligned = aligned(a.a, a_stride, 0, a_cols, es, outer_a);
    const bool b_aligned = aligned(a.b, b_stride, outer_a ? 0 : a.b_group, b_cols, es, outer_b);
    const uint64_t a_bytes = round_up(a_rows * a_pitch * es, 256);
    const uint64_t b_bytes = round_up((outer_a ? 1 : groups) * b_rows * b_pitch * es, 256);
    const uint64_t stages = ceil_div((outer_a ? ceil_div(a.C, groups) : (uint64_t)a.C) * es, kStageBytes);
    float best = 0.0f;
    for (uint32_t id = kHuge; id <= kSmall; ++id) {
        const ShapeCost &c = kCost[id];
        float copies = 0.0f;                            // what this shape has copied and another need not, at 4 TB/s
        bool copy_a = false, copy_b = false;
        if (a.C) {
            copy_a = !a_aligned || !reachable(c.TI, a_stride, es, outer_a);
            copy_b = !b_aligned || !reachable(c.TJ, b_stride, es, outer_b);
            if ((copy_a && !reachable(c.TI, a_pitch, es, outer_a)) || (copy_b && !reachable(c.TJ, b_pitch, es, outer_b)))
                continue;
            if (!launchable(((copy_a ? a_bytes : 0) + (copy_b ? b_bytes : 0)) / 16 + 512, 1)) continue;
            copies = ((copy_a && a_aligned ? a_bytes : 0) + (copy_b && b_aligned ? b_bytes : 0)) * 0.5e-6f;
        }
        const uint64_t ti = ragged ? a.I / c.TI + (groups + 1) / 2 : ceil_div(a.I, c.TI);
        const uint64_t tiles = ti * ceil_div(a.J, c.TJ) * (outer_a ? groups : 1);
        if (!launchable(most_tiles(c.TI) * ceil_div(a.J, c.TJ) * (outer_a ? groups : 1), c.threads)) continue;
        for (uint32_t n = 1; n == 1 || (!a.groups && n <= 32 && stages / n >= 8 && launchable(tiles * n, c.threads));
             n *= 2) {
            const uint64_t rounds = ceil_div(tiles * n, kCUs * c.per_cu), each = ceil_div(stages, n);
            const float alone = rounds * c.alone[es == 1], full = ceil_div(tiles * n, kCUs) * c.full[es == 1];
            float t = (alone > full ? alone : full) * each + c.fixed * rounds + copies;
            if (n > 1) t += 4.0f + (float)n * a.I * a.J * 1e-6f;      // the partial sums' bytes at 4 TB/s
            if (!best || t < best) {
                best = t;
                q.shape = id;
                q.splits = n;
                q.a_pitch = copy_a ? (uint32_t)a_pitch : 0;
                q.b_pitch = copy_b ? (uint32_t)b_pitch : 0;
            }
        }
    }
    if (!best) {                                        // rows of more than 32 MiB
        q.none = a.op != EC_LINEAR_FORWARD || !few(2);
        return q;
    }
    uint64_t at = q.a_pitch ? a_bytes : 0;
    q.b_at = at;
    if (q.b_pitch) at += b_bytes;
    const uint32_t TI = kCost[q.shape].TI, TJ = kCost[q.shape].TJ;
    const uint64_t ti = most_tiles(TI);
    q.tiles_i = (uint32_t)ti;
    q.tiles_j = (uint32_t)ceil_div(a.J, TJ);
    q.blocks = ti * q.tiles_j * (outer_a ? groups : 1);
    q.partial_at = at;
    if (q.splits > 1) {
        at += q.splits * q.blocks * TI * TJ * 4;
        q.blocks *= q.splits;
    }
    q.bytes = at;
    return q;
}

template <class T, int OP, bool E4M3, bool SUM = false>
void launch_shape(const ProductArgs &a, const Plan &q, hipStream_t s) {
    product_kernel<T, OP, E4M3, SUM><<<(uint32_t)q.blocks, T::THREADS, 0, s>>>(a);
    if (q.splits > 1) join_kernel<T, OP><<<q.tiles_i * q.tiles_j * T::NI * T::NJ, T::THREADS, 0, s>>>(a);
}

template <class T>
void launch_op(const ProductArgs &a, const Plan &q, hipStream_t s) {
    if (a.op == EC_LINEAR_GRAD_INPUT)
        launch_shape<T, EC_LINEAR_GRAD_INPUT, false>(a, q, s);
    else if (a.op == EC_LINEAR_GRAD_WEIGHT)
        a.db ? launch_shape<T, EC_LINEAR_GRAD_WEIGHT, false, true>(a, q, s)
             : launch_shape<T, EC_LINEAR_GRAD_WEIGHT, false>(a, q, s);
    else if (a.dtype == EC_E4M3)
        launch_shape<T, EC_LINEAR_FORWARD, true>(a, q, s);
    else
        launch_shape<T, EC_LINEAR_FORWARD, false>(a, q, s);
}

template <int RT, bool E4M3>
void launch_few(const ProductArgs &a, const Plan &q, hipStream_t s) {
    const uint32_t n = (uint32_t)q.blocks;
    if (q.waves == 4)
        few_rows_kernel<RT, 4, E4M3><<<n, 256, 0, s>>>(a);
    else
        few_rows_kernel<RT, 8, E4M3><<<n, 512, 0, s>>>(a);
}

RowCopy row_copy(const void *p, uint64_t stride, uint64_t group_stride, uint64_t groups, uint64_t rows, uint64_t cols,
                 uint32_t es, void *out, uint32_t pitch) {
    RowCopy c = {p, stride, group_stride, groups * rows * (pitch * es / 16), (uint32_t)rows, (uint32_t)cols, pitch, out, 0};
    const uint64_t blocks = ceil_div(c.total, 256);
    c.blocks = blocks > 0x7FFFFFFF ? 0xFFFFFFFFu : (uint32_t)blocks;
    return c;
}

}  // namespace

hipError_t launch_check_offsets(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t *status, hipStream_t s) {
    if (!groups || !status) return hipSuccess;
    check_offsets_kernel<<<1, 64, 0, s>>>(offsets, groups, m, status);
    return hipGetLastError();
}

bool product_sums_columns(const ProductArgs &a) {
    // The second launch and its join cost 8 - 10 us, the sums a tenth of the
    // product: up to 1024 rows that is less (see product_kernel).
    return a.op == EC_LINEAR_GRAD_WEIGHT && a.I && a.J && (a.groups || (a.C <= 1024 && make_plan(a).splits == 1));
}

bool product_fits(const ProductArgs &a) { return !a.I || !a.J || !make_plan(a).none; }

uint64_t product_workspace(const ProductArgs &a) {
    if (!a.I || !a.J) return 0;
    return make_plan(a).bytes;
}

hipError_t launch_product(ProductArgs a, void *workspace, hipStream_t s) {
    if (!a.I || !a.J)
        return launch_check_offsets(a.offsets, a.groups, a.op == EC_LINEAR_GRAD_WEIGHT ? a.C : a.I, a.status, s);
    const Plan q = make_plan(a);
    if (q.none) return hipErrorInvalidValue;
    const uint32_t es = a.dtype == EC_E4M3 ? 1 : 2;
    const bool outer_a = a.op == EC_LINEAR_GRAD_WEIGHT, outer_b = a.op != EC_LINEAR_FORWARD;
    char *ws = (char *)workspace;
    RowCopy ca = {}, cb = {};
    if (q.a_pitch) {
        const uint64_t rows = outer_a ? a.C : a.I, cols = outer_a ? a.I : a.C;
        ca = row_copy(a.a, outer_a ? a.a_c : a.a_i, 0, 1, rows, cols, es, ws + q.a_at, q.a_pitch);
        a.a = ws + q.a_at;
        (outer_a ? a.a_c : a.a_i) = q.a_pitch;
    }
    if (q.b_pitch) {
        const uint64_t rows = outer_b ? a.C : a.J, cols = outer_b ? a.J : a.C, groups = !outer_a && a.groups ? a.groups : 1;
        cb = row_copy(a.b, outer_b ? a.b_c : a.b_j, a.b_group, groups, rows, cols, es, ws + q.b_at, q.b_pitch);
        a.b = ws + q.b_at;
        (outer_b ? a.b_c : a.b_j) = q.b_pitch;
        a.b_group = rows * q.b_pitch;
    }
    const uint64_t copies = (uint64_t)ca.blocks + cb.blocks;
    if (!launchable(copies, 256)) return hipErrorInvalidValue;
    if (copies && es == 1)
        copy_rows_kernel<uint8_t><<<(uint32_t)copies, 256, 0, s>>>(ca, cb);
    else if (copies)
        copy_rows_kernel<uint16_t><<<(uint32_t)copies, 256, 0, s>>>(ca, cb);
    a.tiles_i = q.tiles_i;
    a.tiles_j = q.tiles_j;
    a.splits = q.splits;
    a.partial = (float *)(ws + q.partial_at);
    switch (q.shape) {
        case kHuge: launch_op<Huge>(a, q, s); break;
        case kEven: launch_op<Even>(a, q, s); break;
        case kSmall: launch_op<Small>(a, q, s); break;
        default:
            if (a.dtype == EC_E4M3)
                q.row_tiles == 1 ? launch_few<1, true>(a, q, s) : launch_few<2, true>(a, q, s);
            else
                q.row_tiles == 1 ? launch_few<1, false>(a, q, s) : launch_few<2, false>(a, q, s);
    }
    return hipGetLastError();
}

static uint32_t column_parts(const ColumnSumArgs &a) {
    const uint64_t groups = a.groups ? a.groups : 1, blocks = ceil_div(a.n, kSumCols) * groups;
    uint64_t parts = ceil_div(1024, blocks), most = ceil_div(a.m, groups * 64);
    if (parts > most) parts = most;
    return (uint32_t)(parts < 1 ? 1 : parts > 32 ? 32 : parts);
}

uint64_t column_sum_workspace(const ColumnSumArgs &a) {
    const uint32_t parts = a.n ? column_parts(a) : 1;
    return parts > 1 ? (uint64_t)parts * (a.groups ? a.groups : 1) * a.n * 4 : 0;
}

hipError_t launch_column_sum(const ColumnSumArgs &a, float *workspace, hipStream_t s) {
    if (!a.n) return launch_check_offsets(a.offsets, a.groups, a.m, a.status, s);
    const uint32_t parts = column_parts(a), groups = a.groups ? a.groups : 1;
    const uint64_t n = (uint64_t)groups * a.n;
    if (!launchable(ceil_div(a.n, kSumCols), 256) || (parts > 1 && !launchable(ceil_div(n, 256), 256)))
        return hipErrorInvalidValue;
    column_sum_kernel<<<dim3((uint32_t)ceil_div(a.n, kSumCols), groups, parts), 256, 0, s>>>(a, parts > 1 ? workspace : a.db,
                                                                                           parts);
    if (parts > 1) column_join_kernel<<<(uint32_t)ceil_div(n, 256), 256, 0, s>>>(workspace, a.db, n, parts);
    return hipGetLastError();
}

}  // namespace ec
