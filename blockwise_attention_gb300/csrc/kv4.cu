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
// Both roundings are those of the exact quotients.  max |x| / 6 is a correctly rounded
// division; a quotient of an fp32 value that is not itself halfway between two e4m3
// values (5 significant bits) does not round to such a point.  x / s is formed as
// q0 = x r, q = q0 + (x - q0 s) r with r = 1 / s correctly rounded: x - q0 s is exact in
// an fma and q is the correctly rounded quotient (the remainder step of Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990),
// and again no quotient off a halfway point of the e2m1 grid rounds onto one.
//
// Bound by HBM: one thread per block of 16, 32 (or 64) bytes in and 9 out; the reverse
// for reading.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "internal.h"

namespace ba {
namespace {

__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Sixteen values to their codes (two words, the first element in the lowest nibble) and scale byte.
__device__ __forceinline__ uint2 quantise16(float (&x)[16], float down, uint32_t &scale) {
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] *= down;
        big = max(big, __float_as_uint(x[i]) & 0x7fffffffu);
    }
    if (big >= 0x7f800000u) {   // infinities and NaN: saturate (NaN as the largest value)
        big = 0x7f7fffffu;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = x[i] != x[i] ? 3.0e38f : fminf(fmaxf(x[i], -3.0e38f), 3.0e38f);
    }
    const float want = fminf(__fdiv_rn(__uint_as_float(big), 6.f), 448.f);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.f), "f"(want));
    scale = two & 0xffu;
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    const float s = __half2float(__ushort_as_half((unsigned short)(h2 & 0xffffu)));
    const float r = s > 0.f ? __frcp_rn(s) : 0.f;
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float q0 = x[i] * r;
        q[i] = fmaf(fmaf(-q0, s, x[i]), r, q0);
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(w[k])
            : "f"(q[8 * k]), "f"(q[8 * k + 1]), "f"(q[8 * k + 2]), "f"(q[8 * k + 3]), "f"(q[8 * k + 4]), "f"(q[8 * k + 5]),
              "f"(q[8 * k + 6]), "f"(q[8 * k + 7]));
    return make_uint2(w[0], w[1]);
}

template <typename T>
__device__ __forceinline__ void load16(const T *p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, float (&x)[16]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[8 * k + 2 * i] = __uint_as_float(w[i] << 16);
            x[8 * k + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <>
__device__ __forceinline__ void load16(const float *p, float (&x)[16]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 u = __ldcs(reinterpret_cast<const float4 *>(p) + k);
        x[4 * k] = u.x;
        x[4 * k + 1] = u.y;
        x[4 * k + 2] = u.z;
        x[4 * k + 3] = u.w;
    }
}

// Block `blk` of row t of (tensor w, b, h) for flat index e (blocks fastest).  I: the
// index type, 32 bits when the count allows (a third of the 64-bit divisions' time).
template <typename I>
struct Where {
    int w, b, h, t, blk;
    __device__ __forceinline__ Where(I e, const Kv4Args &a, int nb_log2) {
        blk = (int)(e & ((1u << nb_log2) - 1u));
        e >>= nb_log2;
        t = (int)(e % (I)a.T);
        e /= (I)a.T;
        h = (int)(e % (I)a.H);
        e /= (I)a.H;
        b = (int)(e % (I)a.B);
        w = (int)(e / (I)a.B);
    }
};

template <typename T, typename I>
__global__ void __launch_bounds__(128) kv4_append_kernel(const Kv4Args a, int nb_log2) {
    const long long e = (long long)blockIdx.x * 128 + threadIdx.x;
    if (e >= 2LL * a.B * a.H * a.T << nb_log2) return;
    const Where<I> at((I)e, a, nb_log2);
    if (a.counts && at.t >= a.counts[at.b]) return;
    const long long slot = (a.start ? (long long)a.start[at.b] : (long long)a.first) + at.t;
    if (slot < 0 || slot >= a.S) return;   // behind the cache: dropped
    float x[16];
    load16(static_cast<const T *>(a.x[at.w]) + at.b * a.xsB[at.w] + at.h * a.xsH[at.w] + at.t * a.xsT[at.w] + at.blk * 16, x);
    uint32_t scale;
    const uint2 codes = quantise16(x, pow2(-a.exp[at.w]), scale);
    uint8_t *c = static_cast<uint8_t *>(a.codes[at.w]) + at.b * a.csB[at.w] + at.h * a.csH[at.w] + slot * a.csT[at.w];
    reinterpret_cast<uint2 *>(c)[at.blk] = codes;
    uint8_t *s = static_cast<uint8_t *>(a.scales[at.w]) + at.b * a.ssB[at.w] + at.h * a.ssH[at.w] + slot * a.ssT[at.w];
    s[at.blk] = (uint8_t)scale;
}

template <typename T, typename I>
__global__ void __launch_bounds__(128) kv4_read_kernel(const Kv4Args a, int nb_log2) {
    const long long e = (long long)blockIdx.x * 128 + threadIdx.x;
    if (e >= 2LL * a.B * a.H * a.T << nb_log2) return;
    const Where<I> at((I)e, a, nb_log2);
    const long long slot = (long long)a.first + at.t;
    const uint8_t *c =
        static_cast<const uint8_t *>(a.codes[at.w]) + at.b * a.csB[at.w] + at.h * a.csH[at.w] + slot * a.csT[at.w];
    const uint2 codes = __ldcs(reinterpret_cast<const uint2 *>(c) + at.blk);
    const uint32_t sb = static_cast<const uint8_t *>(
        a.scales[at.w])[at.b * a.ssB[at.w] + at.h * a.ssH[at.w] + slot * a.ssT[at.w] + at.blk];
    uint32_t s2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)(sb | sb << 8)));
    const float up = pow2(a.exp[at.w]);
    float v[16];
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t f[4];
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
            : "r"(w[k]));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t p;   // exact: 2 + 4 significant bits
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(p) : "r"(f[i]), "r"(s2));
            const float2 y = __half22float2(*reinterpret_cast<__half2 *>(&p));
            v[8 * k + 2 * i] = y.x * up;
            v[8 * k + 2 * i + 1] = y.y * up;
        }
    }
    T *y = static_cast<T *>(a.y[at.w]) + (e - ((long long)at.w * a.B * a.H * a.T << nb_log2)) * 16;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 z = __floats2bfloat162_rn(v[8 * k + 2 * i], v[8 * k + 2 * i + 1]);
                p[i] = *reinterpret_cast<const uint32_t *>(&z);
            }
            __stcs(reinterpret_cast<uint4 *>(y) + k, make_uint4(p[0], p[1], p[2], p[3]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            __stcs(reinterpret_cast<float4 *>(y) + k, make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
    }
}

}  // namespace

static int grid_of(const Kv4Args &a, int &nb_log2, bool &wide, unsigned &blocks) {
    nb_log2 = a.d == 128 ? 3 : 2;
    const long long n = 2LL * a.B * a.H * a.T << nb_log2;
    if ((n + 127) / 128 > 0x7fffffffLL) return BA_ERR_SHAPE;
    wide = n > 0xffffffffLL;
    blocks = (unsigned)((n + 127) / 128);
    return BA_OK;
}

int launch_kv4_append(const Kv4Args &a, int, cudaStream_t s) {
    int lg;
    bool wide;
    unsigned n;
    const int rc = grid_of(a, lg, wide, n);
    if (rc || n == 0) return rc;
    if (a.dtype == BA_BF16) {
        if (wide)
            kv4_append_kernel<__nv_bfloat16, unsigned long long><<<n, 128, 0, s>>>(a, lg);
        else
            kv4_append_kernel<__nv_bfloat16, unsigned><<<n, 128, 0, s>>>(a, lg);
    } else {
        if (wide)
            kv4_append_kernel<float, unsigned long long><<<n, 128, 0, s>>>(a, lg);
        else
            kv4_append_kernel<float, unsigned><<<n, 128, 0, s>>>(a, lg);
    }
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

int launch_kv4_read(const Kv4Args &a, int, cudaStream_t s) {
    int lg;
    bool wide;
    unsigned n;
    const int rc = grid_of(a, lg, wide, n);
    if (rc || n == 0) return rc;
    if (a.dtype == BA_BF16) {
        if (wide)
            kv4_read_kernel<__nv_bfloat16, unsigned long long><<<n, 128, 0, s>>>(a, lg);
        else
            kv4_read_kernel<__nv_bfloat16, unsigned><<<n, 128, 0, s>>>(a, lg);
    } else {
        if (wide)
            kv4_read_kernel<float, unsigned long long><<<n, 128, 0, s>>>(a, lg);
        else
            kv4_read_kernel<float, unsigned><<<n, 128, 0, s>>>(a, lg);
    }
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

}  // namespace ba
