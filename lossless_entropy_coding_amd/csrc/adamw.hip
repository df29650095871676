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
// Bound by HBM: one pass, 28 bytes a value with fp32 states, bf16 gradients and
// a bf16 copy, 16 with e4m3 states.
#include "ffn_common.h"
#include "train_common.h"

namespace ec {
namespace {

constexpr uint32_t kBlock = 256;            // values with one scale; a wave's float4 a lane
constexpr int kWaves = 4, kPerWave = 4;     // blocks a wave has on the way
constexpr uint32_t kChunk = kWaves * kPerWave;
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

// The exponent e of the least 2^e with top <= most 2^e, kLeastScale at least;
// top is finite and not negative.  Of values below fp32's normal range only
// that they are small counts.
__device__ __forceinline__ int scale_exponent(float top, float most) {
    const uint32_t t = __float_as_uint(top), w = __float_as_uint(most);
    return (int)(t >> 23) - (int)(w >> 23) + ((t & 0x7FFFFF) > (w & 0x7FFFFF) ? 1 : 0);
}

// The distance of e4m3 values around a in [0, 448], and its inverse.
__device__ __forceinline__ void grid(float a, float *step, float *inverse) {
    const int e = max((int)(__float_as_uint(a) >> 23) - 127, -6) - 3;
    *step = power(e);
    *inverse = power(-e);
}

__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u; }

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

template <bool E4M3, bool BF16, bool COPY>
__device__ __forceinline__ void step_blocks(const AdamPart &part, const AdamTensor &t, uint32_t chunk) {
#pragma clang fp contract(off)              // m and v round as written, wherever they are computed
    const AdamArgs &a = part.a;
    const uint32_t lane = threadIdx.x & 63;
    const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint64_t first = (uint64_t)chunk * kChunk + wave * kPerWave;      // block of the tensor
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
            mc[k] = ((const uint32_t *)a.m)[state / 4];
            vc[k] = ((const uint32_t *)a.v)[state / 4];
            ms[k] = a.m_scale[t.block + first + k];
            vs[k] = a.v_scale[t.block + first + k];
        } else if (left[k]) {
            m[k] = *(const f32x4 *)((const float *)a.m + state);
            v[k] = *(const f32x4 *)((const float *)a.v + state);
        }
        if (left[k] == 4) {
            const f32x4 w = ((const AnyF32x4 *)(t.p + at))->v;
#pragma unroll
            for (int q = 0; q < 4; ++q) p[k][q] = w[q];
            if constexpr (BF16) {
                const u32x2 h = ((const AnyU32x2 *)((const uint16_t *)t.g + at))->v;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    g[k][q] = __uint_as_float(q & 1 ? h[q >> 1] & 0xFFFF0000u : h[q >> 1] << 16);
            } else {
                const f32x4 h = ((const AnyF32x4 *)((const float *)t.g + at))->v;
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

    const int32_t now = *a.steps + 1;
    const float scale = a.grad_scale ? *a.grad_scale : 1.0f, lr = a.lr_at ? *a.lr_at : a.lr;
    // 1 - b^t without the difference of near values
    const float c1 = -expm1f((float)now * a.log_b1), c2 = -expm1f((float)now * a.log_b2);
    const float rate = lr / c1, widen = 1.0f / sqrtf(c2), keep = 1.0f - lr * t.decay;
    uint32_t top[8] = {};                   // of |m| and of v, the finite ones
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
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float d = g[k][q] * scale;
            m[k][q] = m[k][q] * a.b1 + d * a.rest1;
            v[k][q] = v[k][q] * a.b2 + (d * d) * a.rest2;
            p[k][q] = p[k][q] * keep - rate * m[k][q] / (sqrtf(v[k][q]) * widen + a.eps);
            if constexpr (E4M3) {
                if (q < left[k]) {
                    if (finite(m[k][q])) top[k] = max(top[k], __float_as_uint(fabsf(m[k][q])));
                    if (finite(v[k][q])) top[kPerWave + k] = max(top[kPerWave + k], __float_as_uint(v[k][q]));
                }
            }
        }
    }
    uint32_t all = 0, key = 0;
    if constexpr (E4M3) {
        static_assert(kPerWave == 4, "eight maxima");
        all = maxima(top);
        key = mix((uint32_t)now ^ mix(a.seed));
    }
#pragma unroll
    for (int k = 0; k < kPerWave; ++k) {
        if ((first + k) * kBlock >= t.n) continue;
        const uint64_t at = (first + k) * kBlock + lane * 4, state = t.block * kBlock + at;
        if (left[k] == 4) {
            ((AnyF32x4 *)(t.p + at))->v = f32x4{p[k][0], p[k][1], p[k][2], p[k][3]};
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
                *(f32x4 *)((float *)a.m + state) = m[k];
                *(f32x4 *)((float *)a.v + state) = v[k];
            }
        } else {
            const float m_top = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)all, k * 8));
            const float v_top = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)all, (kPerWave + k) * 8));
            const int em = max(scale_exponent(m_top, 448.0f), kLeastScale);
            const int e2 = scale_exponent(v_top, kRootMax), ev = max((e2 + (e2 & 1)) / 2, kLeastScale);
            const float m_inverse = power(-em), v_inverse = power(-2 * ev);
            const uint32_t base = mix((uint32_t)(state >> 32) ^ key);
            float mq[4], vq[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t r = mix(((uint32_t)state + q) ^ base);
                const float um = (float)(r & 0xFFFF) * 0x1p-16f, uv = (float)(r >> 16) * 0x1p-16f;
                float step, inverse;
                const float x = fabsf(m[k][q]) * m_inverse;
                grid(x, &step, &inverse);
                mq[q] = __builtin_copysignf(floorf(x * inverse + um) * step, m[k][q]);
                const float b = v[k][q] * v_inverse, root = sqrtf(b);
                grid(root, &step, &inverse);
                const float low = floorf(root * inverse);
                const float up = uv * (2.0f * low + 1.0f) < b * inverse * inverse - low * low ? 1.0f : 0.0f;
                vq[q] = (low + up) * step;
                if (!finite(m[k][q])) mq[q] = __builtin_nanf("");
                if (!finite(v[k][q])) vq[q] = __builtin_nanf("");
                if (q >= left[k]) mq[q] = vq[q] = 0.0f;
            }
            ((uint32_t *)a.m)[state / 4] = f32_to_e4m3x4(mq[0], mq[1], mq[2], mq[3]);
            ((uint32_t *)a.v)[state / 4] = f32_to_e4m3x4(vq[0], vq[1], vq[2], vq[3]);
            if (lane == 0) {
                a.m_scale[t.block + first + k] = power(em);
                a.v_scale[t.block + first + k] = power(ev);
            }
        }
    }
}

template <bool E4M3>
__global__ __launch_bounds__(kWaves * 64) void adamw_kernel(AdamPart part) {
    // the tensor of this workgroup: the last that begins at or before it
    const uint32_t lane = threadIdx.x & 63;
    const uint64_t mask = __ballot(lane < part.count && part.first[lane] <= blockIdx.x);
    const uint32_t k = (uint32_t)__builtin_amdgcn_readfirstlane(63 - __clzll((long long)mask));
    const AdamTensor &t = part.t[k];
    const uint32_t chunk = blockIdx.x - part.first[k];
    if (t.grad_bf16)
        t.copy ? step_blocks<E4M3, true, true>(part, t, chunk) : step_blocks<E4M3, true, false>(part, t, chunk);
    else
        t.copy ? step_blocks<E4M3, false, true>(part, t, chunk) : step_blocks<E4M3, false, false>(part, t, chunk);
}

__global__ void advance_kernel(int32_t *steps) { *steps += 1; }

}  // namespace

uint64_t adamw_blocks(uint64_t n) { return (n + kBlock - 1) / kBlock; }

hipError_t AdamBatch::launch() {
    if (!part.count) return hipSuccess;
    if (part.a.e4m3)
        adamw_kernel<true><<<part.blocks, kWaves * 64, 0, stream>>>(part);
    else
        adamw_kernel<false><<<part.blocks, kWaves * 64, 0, stream>>>(part);
    part.count = part.blocks = 0;
    return hipGetLastError();
}

hipError_t AdamBatch::add(AdamTensor t) {
    constexpr uint32_t kMost = 1u << 22;    // workgroups a launch: 2^30 threads
    while (t.n) {                           // a tensor of more than a launch's workgroups is cut at a block
        if (part.count == kAdamTensors || part.blocks == kMost) {
            const hipError_t e = launch();
            if (e != hipSuccess) return e;
        }
        const uint64_t chunks = (adamw_blocks(t.n) + kChunk - 1) / kChunk, room = kMost - part.blocks;
        const uint64_t now = chunks < room ? chunks : room, values = now * kChunk * kBlock;
        AdamTensor &to = part.t[part.count];
        to = t;
        if (to.n > values) to.n = values;
        part.first[part.count++] = part.blocks;
        part.blocks += (uint32_t)now;
        t.p += to.n;
        t.g = (const char *)t.g + to.n * (t.grad_bf16 ? 2 : 4);
        if (t.copy) t.copy += to.n;
        t.block += now * kChunk;
        t.n -= to.n;
    }
    return hipSuccess;
}

hipError_t AdamBatch::finish() {
    const hipError_t e = launch();
    if (e != hipSuccess) return e;
    advance_kernel<<<1, 1, 0, stream>>>(part.a.steps);
    return hipGetLastError();
}

}  // namespace ec
