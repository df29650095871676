// AdamW over many tensors at once, states in fp32 or e4m3.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2            (g times *grad_scale)
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// The states of all tensors lie in one array, in blocks of 256 values; every
// tensor begins a block.  In e4m3 a block has a scale, the least power of two
// that takes its values to at most 448.  v is held as its root, which halves
// the exponents it spans.
//
// Rounding to e4m3 is random: to the nearest value a moving average stops
// where its steps fall below half a step of the type, a sixteenth of its value
// (v with b2 = 0.999 after some ten steps).  m goes up or down by its place
// between two values of the type, the root of v by v's place between the
// squares of two, so that the means of m and of v are kept.  The 16 random bits
// of each come from a hash of (seed, step, place), so that the same call gives
// the same bits.
//
// A v held as 0 says only that it was below the least square of its block, the
// square of 2^-9 scales, while the m beside it may be held as a whole step: m /
// sqrt(v) would then be anything (hundreds of lr where a value's gradients are
// 1e-5 of its block's largest or less; those of exact states are within 7.3 of 0
// with b1 = 0.9, b2 = 0.999).  The change of p therefore takes sqrt(b2) times
// that least root where v's own is below it: at least what any v held as more
// than 0 leaves, and never less than what v stood for.  v itself stays as it is.
//
// Bound by HBM: one pass, 28 bytes a value with fp32 states, bf16 gradients and
// a bf16 copy, 16 with e4m3 states.
#include "ffn_common.h"
#include "train_common.h"

namespace ec {
namespace {

constexpr uint32_t kBlock = 256;            // values with one scale; a wave's float4 a lane
constexpr int kPerWave = 4;                 // blocks a wave has on the way
constexpr int kWaves = 4, kAloneWaves = 16; // a workgroup's
// Workgroups of a launch; more take several chunks a wave.  A layer of 45
// million values with fp32 states: 185 us with 4096, 180 with 8192, 186 with
// 16384.
constexpr uint32_t kMostBlocks = 8192;
// Chunks up to which one workgroup does a step alone, and moves the step's number
// on, which takes a launch of its own after several workgroups.  18 chunks: 7 us
// alone; in several workgroups 7 us and 5 for the number.
constexpr uint32_t kAloneChunks = 32;

// At any address that suits their elements.  Params and states are read and
// written past the caches (non-temporal), since a step's do not stay there till
// the next one; the copies, which the next layer reads, are not.  45 million
// values with fp32 states: 216 us without, 180 with, 191 with the copies too.
typedef f32x4 AnyFloats __attribute__((aligned(4)));
typedef u32x2 AnyHalves __attribute__((aligned(2)));
constexpr int kLeastScale = -60;            // exponent
constexpr float kRootMax = 448.0f * 448.0f;

// A 32-bit hash by xor-shifts and multiplications (the constants are the
// published ones of C. Wellons' search for low-bias mixers).
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x = (x ^ (x >> 16)) * 0x7FEB352Du;
    x = (x ^ (x >> 15)) * 0x846CA68Bu;
    return x ^ (x >> 16);
}

// 2^e for e in the normal range.
__device__ __forceinline__ float power(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// The exponent e of the least 2^e with top <= most 2^e; top is finite and not
// negative.  Of values below fp32's normal range only that they are small
// counts.
__device__ __forceinline__ int scale_exponent(float top, float most) {
    const uint32_t t = __float_as_uint(top), w = __float_as_uint(most);
    return (int)(t >> 23) - (int)(w >> 23) + ((t & 0x7FFFFF) > (w & 0x7FFFFF) ? 1 : 0);
}

// The distance of e4m3 values around a in [0, 448] (powers of two, from bits), and its inverse.
__device__ __forceinline__ void grid(float a, float *step, float *inverse) {
    const uint32_t binade = max(__float_as_uint(a) & 0x7F800000u, 121u << 23) - (3u << 23);
    *step = __uint_as_float(binade);
    *inverse = __uint_as_float((254u << 23) - binade);
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

// sqrt to 2 u, below the normal range too, where the instruction gives zero.
__device__ __forceinline__ float root_of(float v) {
    const bool small = v < 0x1p-100f;
    return __builtin_amdgcn_sqrtf(v * (small ? 0x1p64f : 1.0f)) * (small ? 0x1p-32f : 1.0f);
}

// 1 - e^x for x <= 0, to a few u of itself: the series near 0 (what is left out
// is below 2^-30 of it), the difference elsewhere.
__device__ __forceinline__ float one_minus_exp(float x) {
    float s = 1.0f / 40320.0f;
    s = __builtin_fmaf(s, x, 1.0f / 5040.0f);
    s = __builtin_fmaf(s, x, 1.0f / 720.0f);
    s = __builtin_fmaf(s, x, 1.0f / 120.0f);
    s = __builtin_fmaf(s, x, 1.0f / 24.0f);
    s = __builtin_fmaf(s, x, 1.0f / 6.0f);
    s = __builtin_fmaf(s, x, 0.5f);
    s = __builtin_fmaf(s, x, 1.0f);
    return x > -0.35f ? -x * s : 1.0f - __builtin_amdgcn_exp2f(x * 1.44269504f);
}

// Values of the type, or NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(const float (&v)[4]) {
    const int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], r, true);
}

// Eight values of a lane, each to be joined over the wave by the maximum: by
// halves, so that ten exchanges do for the eight.  Returns the maxima of
// values 0 .. 7 at lanes 0, 8, .. 56 and beside.
__device__ __forceinline__ uint32_t maxima(const uint32_t (&v)[8]) {
    const uint32_t lane = threadIdx.x & 63;
    uint32_t a[4], b[2], c;
#pragma unroll
    for (int k = 0; k < 4; ++k) {           // lanes of the upper half keep values 4 .. 7
        const uint32_t mine = lane & 32 ? v[4 + k] : v[k], give = lane & 32 ? v[k] : v[4 + k];
        a[k] = max(mine, (uint32_t)__shfl_xor((int)give, 32));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t mine = lane & 16 ? a[2 + k] : a[k], give = lane & 16 ? a[k] : a[2 + k];
        b[k] = max(mine, (uint32_t)__shfl_xor((int)give, 16));
    }
    {
        const uint32_t mine = lane & 8 ? b[1] : b[0], give = lane & 8 ? b[0] : b[1];
        c = max(mine, (uint32_t)__shfl_xor((int)give, 8));
    }
#pragma unroll
    for (int d = 4; d; d >>= 1) c = max(c, (uint32_t)__shfl_xor((int)c, d));
    return c;
}

// What a step's formulas take besides the tensors.
struct Step {
    float scale, rate, widen, keep;         // keep: 1 - lr decay, of the tensor
    float least;                            // e4m3: v's root at the least, over its block's scale
    uint32_t key;
};

template <bool E4M3, bool BF16, bool COPY>
__device__ __forceinline__ void step_blocks(const AdamArgs &a, const AdamTensor &t, const Step &c, uint64_t first) {
#pragma clang fp contract(off)              // m and v round as written, wherever they are computed
    const uint32_t lane = threadIdx.x & 63;
    float p[kPerWave][4], g[kPerWave][4];
    f32x4 m[kPerWave], v[kPerWave];
    uint32_t mc[kPerWave], vc[kPerWave];
    float ms[kPerWave], vs[kPerWave];
    int left[kPerWave];                     // values of the lane that exist
#pragma unroll
    for (int k = 0; k < kPerWave; ++k) {
        const uint64_t at = (first + k) * kBlock + lane * 4, state = t.block * kBlock + at;
        left[k] = at >= t.n ? 0 : t.n - at < 4 ? (int)(t.n - at) : 4;
#pragma unroll
        for (int q = 0; q < 4; ++q) p[k][q] = g[k][q] = 0.0f;
        m[k] = v[k] = f32x4{0, 0, 0, 0};
        mc[k] = vc[k] = 0;
        ms[k] = vs[k] = 1.0f;
        if ((first + k) * kBlock >= t.n) continue;
        if constexpr (E4M3) {
            mc[k] = __builtin_nontemporal_load((const uint32_t *)a.m + state / 4);
            vc[k] = __builtin_nontemporal_load((const uint32_t *)a.v + state / 4);
            ms[k] = a.m_scale[t.block + first + k];
            vs[k] = a.v_scale[t.block + first + k];
        } else if (left[k]) {
            m[k] = __builtin_nontemporal_load((const f32x4 *)((const float *)a.m + state));
            v[k] = __builtin_nontemporal_load((const f32x4 *)((const float *)a.v + state));
        }
        if (left[k] == 4) {
            const f32x4 w = __builtin_nontemporal_load((const AnyFloats *)(t.p + at));
#pragma unroll
            for (int q = 0; q < 4; ++q) p[k][q] = w[q];
            if constexpr (BF16) {
                const u32x2 h = __builtin_nontemporal_load((const AnyHalves *)((const uint16_t *)t.g + at));
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    g[k][q] = __uint_as_float(q & 1 ? h[q >> 1] & 0xFFFF0000u : h[q >> 1] << 16);
            } else {
                const f32x4 h = __builtin_nontemporal_load((const AnyFloats *)((const float *)t.g + at));
#pragma unroll
                for (int q = 0; q < 4; ++q) g[k][q] = h[q];
            }
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < left[k]) {
                    p[k][q] = t.p[at + q];
                    g[k][q] = BF16 ? bf16_to_f32(((const uint16_t *)t.g)[at + q]) : ((const float *)t.g)[at + q];
                }
        }
    }

    uint32_t top[8] = {};                   // of |m| and of v; what is past the tensor's end is zero
#pragma unroll
    for (int k = 0; k < kPerWave; ++k) {
        if constexpr (E4M3) {
            const f32x2 m0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[k], false), m1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)mc[k], true);
            const f32x2 v0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[k], false), v1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)vc[k], true);
            m[k] = f32x4{m0[0], m0[1], m1[0], m1[1]};
            v[k] = f32x4{v0[0], v0[1], v1[0], v1[1]};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                m[k][q] = m[k][q] * ms[k];
                const float root = v[k][q] * vs[k];
                v[k][q] = root * root;
            }
        }
        const float least = E4M3 ? vs[k] * c.least : 0.0f;
        float most[2] = {0.0f, 0.0f};       // without NaN
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float d = g[k][q] * c.scale;
            m[k][q] = m[k][q] * a.b1 + d * a.rest1;
            v[k][q] = v[k][q] * a.b2 + (d * d) * a.rest2;
            float root = root_of(v[k][q]);
            if constexpr (E4M3) root = root < least ? least : root;         // NaN stays
            const float below = root * c.widen + a.eps;
            p[k][q] = p[k][q] * c.keep - c.rate * m[k][q] * __builtin_amdgcn_rcpf(below);
            most[0] = fmaxf(most[0], fabsf(m[k][q]));
            most[1] = fmaxf(most[1], v[k][q]);
        }
        top[k] = __float_as_uint(most[0]);
        top[kPerWave + k] = __float_as_uint(most[1]);
    }
    uint32_t all = 0;
    bool infinite = false;
    if constexpr (E4M3) {
        static_assert(kPerWave == 4, "eight maxima");
        all = maxima(top);
        if (__ballot(all == 0x7F800000u)) { // seldom: the largest of those that are finite
            infinite = true;
#pragma unroll
            for (int k = 0; k < kPerWave; ++k) {
                top[k] = top[kPerWave + k] = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (finite(m[k][q])) top[k] = max(top[k], __float_as_uint(fabsf(m[k][q])));
                    if (finite(v[k][q])) top[kPerWave + k] = max(top[kPerWave + k], __float_as_uint(v[k][q]));
                }
            }
            all = maxima(top);
        }
    }
#pragma unroll
    for (int k = 0; k < kPerWave; ++k) {
        if ((first + k) * kBlock >= t.n) continue;
        const uint64_t at = (first + k) * kBlock + lane * 4, state = t.block * kBlock + at;
        if (left[k] == 4) {
            __builtin_nontemporal_store((AnyFloats){p[k][0], p[k][1], p[k][2], p[k][3]}, (AnyFloats *)(t.p + at));
            if constexpr (COPY)
                ((AnyU32x2 *)(t.copy + at))->v = u32x2{f32_to_bf16x2(p[k][0], p[k][1]), f32_to_bf16x2(p[k][2], p[k][3])};
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (q < left[k]) {
                    t.p[at + q] = p[k][q];
                    if constexpr (COPY) t.copy[at + q] = f32_to_bf16(p[k][q]);
                }
        }
        if constexpr (!E4M3) {
            // past the tensor's end a block holds zeros: their values stay
            if (left[k]) {
                __builtin_nontemporal_store(m[k], (f32x4 *)((float *)a.m + state));
                __builtin_nontemporal_store(v[k], (f32x4 *)((float *)a.v + state));
            }
        } else {
            const float m_top = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)all, k * 8));
            const float v_top = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)all, (kPerWave + k) * 8));
            const int em = max(scale_exponent(m_top, 448.0f), kLeastScale);
            const int e2 = scale_exponent(v_top, kRootMax), ev = max((e2 + (e2 & 1)) / 2, kLeastScale);
            const float m_inverse = power(-em), v_inverse = power(-2 * ev);
            const uint32_t base = mix((uint32_t)(state >> 32) ^ c.key);
            float mq[4], vq[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t r = mix(((uint32_t)state + q) ^ base);
                const float um = (float)(r & 0xFFFF) * 0x1p-16f, uv = (float)(r >> 16) * 0x1p-16f;
                float step, inverse;
                const float x = fabsf(m[k][q]) * m_inverse;
                grid(x, &step, &inverse);
                // the product is exact, a step being a power of two
                mq[q] = __builtin_copysignf(floorf(__builtin_fmaf(x, inverse, um)) * step, m[k][q]);
                // A root next to a value of the grid may fall on either side of
                // it: the comparison with v itself then leads to that value.
                const float b = v[k][q] * v_inverse, root = __builtin_amdgcn_sqrtf(b);
                grid(root, &step, &inverse);
                const float low = floorf(root * inverse);
                const bool up = uv * __builtin_fmaf(2.0f, low, 1.0f) < __builtin_fmaf(-low, low, b * (inverse * inverse));
                vq[q] = (up ? low + 1.0f : low) * step;
                if (infinite) {
                    if (!finite(m[k][q])) mq[q] = __builtin_nanf("");
                    if (!finite(v[k][q])) vq[q] = __builtin_nanf("");
                }
            }
            __builtin_nontemporal_store(to_e4m3x4(mq), (uint32_t *)a.m + state / 4);
            __builtin_nontemporal_store(to_e4m3x4(vq), (uint32_t *)a.v + state / 4);
            if (lane == 0) {
                a.m_scale[t.block + first + k] = power(em);
                a.v_scale[t.block + first + k] = power(ev);
            }
        }
    }
}

// A wave takes kPerWave blocks of a tensor at a time, the waves of the launch
// one after the other.  ALONE: the launch is one workgroup, which moves the
// step's number on itself.
template <bool E4M3, int WAVES, bool ALONE>
__global__ __launch_bounds__(WAVES * 64) void adamw_kernel(AdamPart part) {
    const AdamArgs &a = part.a;
    const uint32_t lane = threadIdx.x & 63;
    const int32_t now = *a.steps + 1;
    Step c;
    c.scale = a.grad_scale ? *a.grad_scale : 1.0f;
    const float lr = a.lr_at ? *a.lr_at : a.lr;
    c.rate = lr / one_minus_exp((float)now * a.log_b1);
    c.widen = 1.0f / sqrtf(one_minus_exp((float)now * a.log_b2));
    c.least = sqrtf(a.b2) * 0x1p-9f;
    c.key = mix((uint32_t)now ^ mix(a.seed));
    if constexpr (ALONE) {
        __syncthreads();                    // every wave has the number
        if (threadIdx.x == 0) *a.steps = now;
    }
    const uint32_t begins = lane < part.count ? part.first[lane] : 0xFFFFFFFFu;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    for (uint32_t i = blockIdx.x * WAVES + wave; i < part.chunks; i += gridDim.x * WAVES) {
        // the last tensor that begins at or before i
        const uint32_t k = (uint32_t)__builtin_amdgcn_readfirstlane(63 - __clzll((long long)__ballot(begins <= i)));
        const AdamTensor &t = part.t[k];
        const uint64_t first = (uint64_t)(i - part.first[k]) * kPerWave;
        c.keep = 1.0f - lr * t.decay;
        if (t.grad_bf16)
            t.copy ? step_blocks<E4M3, true, true>(a, t, c, first) : step_blocks<E4M3, true, false>(a, t, c, first);
        else
            t.copy ? step_blocks<E4M3, false, true>(a, t, c, first) : step_blocks<E4M3, false, false>(a, t, c, first);
    }
}

__global__ void advance_kernel(int32_t *steps) { *steps += 1; }

template <bool E4M3>
void launch_part(const AdamPart &part, bool alone, hipStream_t s) {
    if (alone)
        adamw_kernel<E4M3, kAloneWaves, true><<<1, kAloneWaves * 64, 0, s>>>(part);
    else {
        const uint32_t need = (part.chunks + kWaves - 1) / kWaves;
        adamw_kernel<E4M3, kWaves, false><<<need < kMostBlocks ? need : kMostBlocks, kWaves * 64, 0, s>>>(part);
    }
}

}  // namespace

uint64_t adamw_blocks(uint64_t n) { return (n + kBlock - 1) / kBlock; }

hipError_t AdamBatch::launch(bool alone) {
    if (!part.count) return hipSuccess;
    part.a.e4m3 ? launch_part<true>(part, alone, stream) : launch_part<false>(part, alone, stream);
    launched = true;
    part.count = part.chunks = 0;
    return hipGetLastError();
}

hipError_t AdamBatch::add(const AdamTensor &t) {
    if (!t.n) return hipSuccess;
    if (part.count == kAdamTensors) {
        const hipError_t e = launch(false);
        if (e != hipSuccess) return e;
    }
    part.t[part.count] = t;
    part.first[part.count++] = part.chunks;
    part.chunks += (uint32_t)((adamw_blocks(t.n) + kPerWave - 1) / kPerWave);
    return hipSuccess;
}

hipError_t AdamBatch::finish() {
    const bool alone = !launched && part.count && part.chunks <= kAloneChunks;
    const hipError_t e = launch(alone);
    if (e != hipSuccess || alone) return e;
    advance_kernel<<<1, 1, 0, stream>>>(part.a.steps);
    return hipGetLastError();
}

}  // namespace ec
