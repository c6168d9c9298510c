// Writing and reading a KV cache held in 4 bits.
//
// A row of d values is held as d / 16 blocks: per block one scale s in e4m3 and sixteen
// codes c in e2m1 (values 0, 1/2, 1, 3/2, 2, 3, 4, 6 with a sign), value = c s 2^exp:
//   s = e4m3(max |x| 2^-exp / 6),  c = e2m1(x 2^-exp / s),
// each rounded to nearest, ties to even, and saturating at 448 and 6; s = 0 leaves codes
// of zero.  exp is a power of two for the whole tensor, which moves the range of the
// scales (2^-9 .. 448) to the tensor's; it keeps every product exact.  Two codes a byte,
// the earlier element in the low nibble: (1/2 + 1/16) d bytes a row.
//
// Both roundings are those of the exact quotients.  max |x| / 6 and x / s are correctly
// rounded: q0 = x r, q = q0 + (x - q0 s) r with r the correctly rounded reciprocal of the
// divisor, where x - q0 s is exact in an fma (the remainder step of Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).  A
// correctly rounded quotient of fp32 values lies on a halfway point of either grid (at
// most 5 significant bits) only if the exact one does.
//
// Bound by HBM when the instructions a value takes are few (about 230 a byte-time of an SM
// for 16 values): writing, a lane takes a block of 16 values, its row's address formed
// once for several rows; reading, a lane takes 8 values, so that a warp's 16-byte stores
// are whole lines.  (Writing with two lanes a block, whole lines but the divisions twice:
// 8K prompts of 64 heads written and read back 248 us.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "internal.h"

namespace ba {
namespace {

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// max(|a|, |b|, c), NaN when one is.
__device__ __forceinline__ float absmax3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(c));
    return d;
}

// Two quotients v / s rounded correctly (see above), r = 1 / s.
__device__ __forceinline__ float2 quotients(float v0, float v1, float s, float r) {
    float2 q;
    asm("{\n\t.reg .b64 v, s, r, q, n;\n\tmov.b64 v, {%2, %3};\n\tmov.b64 s, {%4, %4};\n\tmov.b64 r, {%5, %5};\n\t"
        "mul.rn.f32x2 q, v, r;\n\tfma.rn.f32x2 n, q, s, v;\n\tfma.rn.f32x2 q, n, r, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
        : "=f"(q.x), "=f"(q.y)
        : "f"(v0), "f"(v1), "f"(-s), "f"(r));
    return q;
}

__device__ __forceinline__ uint2 codes16(const float (&x)[16], float s) {
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = quotients(x[8 * k + 2 * i], x[8 * k + 2 * i + 1], s, r);
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(w[k])
            : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
    }
    return make_uint2(w[0], w[1]);
}

// Sixteen values to their codes (the first value in the lowest nibble) and scale byte; up = 2^exp.
__device__ __forceinline__ uint2 quantise16(float (&x)[16], float up, float six, float sixth, uint32_t &scale) {
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) big = absmax3(x[i], x[i + 1], big);
    // scale: want = max / (6 up), rounded once (up is a power of two)
    const float top = big <= 3.0e38f ? big : 3.0e38f;
    float want = top * sixth;
    want = fmaf(fmaf(-want, six, top), sixth, want);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(fminf(want, 448.f)));
    scale = two & 0xffu;
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    const float s = __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu))) * up;
    if (!(big <= 3.0e38f && want <= 448.f)) {
        // a block that the largest scale does not hold, or with infinities or NaN: quotients
        // are kept within +-8 (which saturates), NaN as the largest value
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] != x[i] ? 8.f * s : fminf(fmaxf(x[i], -8.f * s), 8.f * s);
    }
    return codes16(x, s);
}

// Sixteen values as they are loaded.
struct Raw16b {   // bf16
    uint4 u[2];
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
        u[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        u[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
                x[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};
struct Raw16f {   // fp32
    float4 u[4];
    __device__ __forceinline__ void load(const float *p) {
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = __ldg(reinterpret_cast<const float4 *>(p) + k);
    }
    __device__ __forceinline__ void get(float (&x)[16]) const {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[4 * k] = u[k].x;
            x[4 * k + 1] = u[k].y;
            x[4 * k + 2] = u[k].z;
            x[4 * k + 3] = u[k].w;
        }
    }
};
template <typename T>
struct RawOf {
    using type = Raw16b;
};
template <>
struct RawOf<float> {
    using type = Raw16f;
};

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&z);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
        __stcs(reinterpret_cast<float4 *>(p) + k, make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
}

constexpr int KV_THREADS = 256, KV_ROUNDS = 4;

// First row of this thread's group of lanes (LPR lanes a row): row t of (tensor w, b, h).
// FLAT: one row, of all heads' rows in one sequence; else blockIdx.y is (w, b, h) and the
// rows t, t + KV_THREADS / LPR, .. (KV_ROUNDS of them).  false: there is none.
template <int LPR, bool FLAT>
__device__ __forceinline__ bool first_row(const Kv4Args &a, int &w, int &b, int &h, int &t) {
    constexpr int RPB = KV_THREADS / LPR;
    const int place = threadIdx.x / LPR;
    unsigned whb;
    if constexpr (FLAT) {
        const unsigned long long e = (unsigned long long)blockIdx.x * RPB + place;
        if (e >= 2ull * a.B * a.H * a.T) return false;
        if (e >> 32) {
            t = (int)(e % (unsigned)a.T);
            whb = (unsigned)(e / (unsigned)a.T);
        } else {
            t = (int)((unsigned)e % (unsigned)a.T);
            whb = (unsigned)e / (unsigned)a.T;
        }
    } else {
        t = (int)blockIdx.x * (RPB * KV_ROUNDS) + place;
        whb = blockIdx.y;
    }
    h = (int)(whb % (unsigned)a.H);
    whb /= (unsigned)a.H;
    b = (int)(whb % (unsigned)a.B);
    w = (int)(whb / (unsigned)a.B);
    return t < a.T;
}

template <typename T, int D, bool FLAT>
__global__ void __launch_bounds__(KV_THREADS) kv4_append_kernel(const Kv4Args a) {
    constexpr int LPR = D / 16, RPB = KV_THREADS / LPR, N = FLAT ? 1 : KV_ROUNDS;
    int w, b, h, t;
    if (!first_row<LPR, FLAT>(a, w, b, h, t)) return;
    const int l = threadIdx.x % LPR;   // the lane's block of a row
    const long long start = a.start ? (long long)a.start[b] : (long long)a.first;
    int rows = a.counts ? min(a.T, a.counts[b]) : a.T;
    rows = (int)min((long long)rows, (long long)a.S - start);   // rows behind the cache are dropped
    const int skip = start < 0 ? (int)min(-start, (long long)a.T) : 0;   // as are rows before it
    const T *x = static_cast<const T *>(a.x[w]) + b * a.xsB[w] + h * a.xsH[w] + t * a.xsT[w] + l * 16;
    const long long xs = RPB * a.xsT[w];
    typename RawOf<T>::type raw[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int tu = t + u * RPB;
        if (tu < rows && tu >= skip) raw[u].load(x + u * xs);
    }
    const float up = pow2(a.exp[w]), six = 6.f * up, sixth = __frcp_rn(six);
    const long long slot = start + t;
    uint8_t *c = static_cast<uint8_t *>(a.codes[w]) + b * a.csB[w] + h * a.csH[w] + slot * a.csT[w] + l * 8;
    uint8_t *s = static_cast<uint8_t *>(a.scales[w]) + b * a.ssB[w] + h * a.ssH[w] + slot * a.ssT[w] + l;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int tu = t + u * RPB;
        if (tu >= rows || tu < skip) continue;
        float v[16];
        raw[u].get(v);
        uint32_t scale;
        const uint2 codes = quantise16(v, up, six, sixth, scale);
        *reinterpret_cast<uint2 *>(c + u * (RPB * a.csT[w])) = codes;
        s[u * (RPB * a.ssT[w])] = (uint8_t)scale;
    }
}

template <typename T, int D, bool FLAT>
__global__ void __launch_bounds__(KV_THREADS) kv4_read_kernel(const Kv4Args a) {
    constexpr int LPR = D / 8, RPB = KV_THREADS / LPR, N = FLAT ? 1 : KV_ROUNDS;
    int w, b, h, t;
    if (!first_row<LPR, FLAT>(a, w, b, h, t)) return;
    const int l = threadIdx.x % LPR;   // the lane's eight values of a row
    const long long slot = (long long)a.first + t;
    const uint8_t *c = static_cast<const uint8_t *>(a.codes[w]) + b * a.csB[w] + h * a.csH[w] + slot * a.csT[w] + l * 4;
    const uint8_t *s = static_cast<const uint8_t *>(a.scales[w]) + b * a.ssB[w] + h * a.ssH[w] + slot * a.ssT[w] + (l >> 1);
    T *y = static_cast<T *>(a.y[w]) + (((long long)b * a.H + h) * a.T + t) * D + l * 8;
    uint32_t codes[N], sb[N];
#pragma unroll
    for (int u = 0; u < N; ++u)
        if (t + u * RPB < a.T) {
            codes[u] = __ldg(reinterpret_cast<const uint32_t *>(c + u * (RPB * a.csT[w])));
            sb[u] = __ldg(s + u * (RPB * a.ssT[w]));
        }
    const float up = pow2(a.exp[w]);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (t + u * RPB >= a.T) continue;
        uint32_t s2, f[4];
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)sb[u]));
        const float sc = __half2float(__ushort_as_half((unsigned short)(s2 & 0xffffu))) * up;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
            : "r"(codes[u]));
        float v[8];   // exact: 2 + 4 significant bits
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 z = __half22float2(*reinterpret_cast<__half2 *>(&f[i]));
            v[2 * i] = z.x * sc;
            v[2 * i + 1] = z.y * sc;
        }
        store8(y + (long long)u * RPB * D, v);
    }
}

// Launches the append (APPEND) or the read.
template <bool APPEND, typename T, int D>
int launch(const Kv4Args &a, cudaStream_t s) {
    constexpr int RPB = KV_THREADS / (APPEND ? D / 16 : D / 8);
    const long long heads = 2LL * a.B * a.H, chunks = ((long long)a.T + RPB * KV_ROUNDS - 1) / (RPB * KV_ROUNDS);
    if (a.T >= RPB * KV_ROUNDS && heads <= 65535) {
        const dim3 grid((unsigned)chunks, (unsigned)heads);
        if constexpr (APPEND)
            kv4_append_kernel<T, D, false><<<grid, KV_THREADS, 0, s>>>(a);
        else
            kv4_read_kernel<T, D, false><<<grid, KV_THREADS, 0, s>>>(a);
    } else {
        const long long blocks = (heads * a.T + RPB - 1) / RPB;
        if (blocks > 0x7fffffffLL || heads > 0xffffffffLL) return BA_ERR_SHAPE;
        if constexpr (APPEND)
            kv4_append_kernel<T, D, true><<<(unsigned)blocks, KV_THREADS, 0, s>>>(a);
        else
            kv4_read_kernel<T, D, true><<<(unsigned)blocks, KV_THREADS, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

template <bool APPEND>
int launch_any(const Kv4Args &a, cudaStream_t s) {
    if ((long long)a.B * a.H * a.T == 0) return BA_OK;
    if (a.dtype == BA_BF16)
        return a.d == 128 ? launch<APPEND, __nv_bfloat16, 128>(a, s) : launch<APPEND, __nv_bfloat16, 64>(a, s);
    return a.d == 128 ? launch<APPEND, float, 128>(a, s) : launch<APPEND, float, 64>(a, s);
}

}  // namespace

int launch_kv4_append(const Kv4Args &a, cudaStream_t s) { return launch_any<true>(a, s); }
int launch_kv4_read(const Kv4Args &a, cudaStream_t s) { return launch_any<false>(a, s); }

}  // namespace ba
