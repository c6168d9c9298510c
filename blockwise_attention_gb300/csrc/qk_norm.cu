// Norms of queries and keys per head with the position rotation in the same pass, and
// their gradients.
//
// For a row x of d values (one head at one position m) with weights w:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  z = n w,
//   (y_2c, y_2c+1) = (z_2c cos a_c - z_2c+1 sin a_c, z_2c sin a_c + z_2c+1 cos a_c),
//   a_c = m base^(-2c/d)  (the rotation of rope_apply).
// Backward: dz = the rotation's transpose of dy, dw = sum over rows of dz n, dn = dz w,
//   dx = r (dn - n mean(dn n)).
//
// Bound by HBM: x (and dy) in, y (or dx) out, once each.  Lanes own 16 bytes of a row
// (LPR lanes a row); a thread keeps its place (position, columns) and walks the heads of
// both tensors, so that the angles of its pairs are formed once for all heads (and for
// all sequences, when they share their positions), and the weights' gradients stay in
// registers until the end.  Four rows' loads are in flight per thread, kept as loaded.
// Angles: a turn's fraction is m times base^(-2c/d) / 2 pi held as a 64-bit fraction,
// modulo 2^64: exact integer arithmetic, so that far positions cost no accuracy (the
// fraction's own error is 2^-53 relative, times m) and no fp64 instruction, of which an
// SM has few; then sincospi in fp32.  (Product and reduction in fp64, and one block of
// positions a CTA: 8K positions, 2 sequences, 20 heads, forward 54 us.)
// dw: every block writes its sums, a second launch adds the blocks' in a fixed order (no
// atomics), in fp64.
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "internal.h"

namespace ba {
namespace {

constexpr int QN_THREADS = 256;
constexpr int QN_ROWS = 4;   // rows in flight per thread
#ifndef QN_WANT
#define QN_WANT 12
#endif

template <typename T>
struct Lane;   // a lane's 16 bytes of a row of T
template <>
struct Lane<__nv_bfloat16> {
    static constexpr int N = 8;
};
template <>
struct Lane<float> {
    static constexpr int N = 4;
};

// N consecutive values of T as they are loaded (16-byte words when VEC, else one by one).
template <typename T, int N, bool VEC>
struct Raw {
    static constexpr int WORDS = N * (int)sizeof(T) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < WORDS / 4; ++i) {
                const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = u.x;
                w[4 * i + 1] = u.y;
                w[4 * i + 2] = u.z;
                w[4 * i + 3] = u.w;
            }
            if constexpr (WORDS % 4 == 2) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p));
                w[0] = u.x;
                w[1] = u.y;
            }
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i)
                w[i] = (uint32_t)__bfloat16_as_ushort(p[2 * i]) | (uint32_t)__bfloat16_as_ushort(p[2 * i + 1]) << 16;
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = __float_as_uint(p[i]);
        }
    }
    __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            if constexpr (sizeof(T) == 2) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
};

__device__ __forceinline__ void store_n(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&z);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store_n(float *p, const float (&x)[4]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0], x[1], x[2], x[3]));
}

__device__ __forceinline__ float weight(const void *w, int f32, int c) {
    return f32 ? static_cast<const float *>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]);
}

// T: type of x and y (dx); G: type of dy; LPR: lanes a row.
template <typename T, typename G, int LPR, bool BWD, bool VEC>
__global__ void __launch_bounds__(QN_THREADS, BWD ? 2 : 3) qk_norm_kernel(const QkNormArgs a) {
    constexpr int N = Lane<T>::N, TP = QN_THREADS / LPR, D = LPR * N;
    const int place = threadIdx.x / LPR, gl = threadIdx.x % LPR, c0 = gl * N;
    const int HT = a.H[0] + a.H[1];
    const int rows = a.nb * HT;   // of a place: (sequence, head), the queries' heads first
    // blocks: the splits of a block of places side by side, so that its memory is read at one time
    const int gx = gridDim.x / a.splits, bx = blockIdx.x / a.splits, by = blockIdx.x - bx * a.splits;
    const int per = (rows + a.splits - 1) / a.splits, r_begin = by * per, r_end = min(rows, r_begin + per);
    float wq[N], wk[N], dwq[N], dwk[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        wq[e] = a.H[0] ? weight(a.w[0], a.w_f32, c0 + e) : 0.f;
        wk[e] = a.H[1] ? weight(a.w[1], a.w_f32, c0 + e) : 0.f;
        dwq[e] = dwk[e] = 0.f;
    }
    for (long long p0 = (long long)bx * TP; p0 < a.places; p0 += (long long)gx * TP) {
        // (lanes behind the last place stay for the shuffles: they repeat the last place and store nothing)
        const bool valid = p0 + place < a.places;
        const long long at = valid ? p0 + place : a.places - 1;
        const int b0 = a.nb == 1 && a.places != a.T ? (int)(at / a.T) : 0, t = (int)(at - (long long)b0 * a.T);
        const int m = a.positions ? a.positions[(long long)b0 * a.pos_ld + t] : t;
        float cs[N / 2], sn[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const int turns = (int)(((unsigned long long)(long long)m * a.turn[c0 / 2 + i]) >> 32);   // [-1/2, 1/2) turns
            sincospif((float)turns * 0x1p-31f, &sn[i], &cs[i]);
        }
        // runs of heads of one tensor and sequence
        for (int r = r_begin; r < r_end;) {
            const int bi = r / HT, hh = r - bi * HT, i = hh >= a.H[0] ? 1 : 0, h = hh - (i ? a.H[0] : 0), b = b0 + bi;
            const int n = min(r_end - r, a.H[i] - h);
            r += n;
            const T *px = static_cast<const T *>(a.x[i]) + b * a.sB[i] + h * a.sH[i] + t * a.sT[i] + c0;
            const G *pg = BWD ? static_cast<const G *>(a.g[i]) + b * a.gB[i] + h * a.gH[i] + t * a.gT[i] + c0 : nullptr;
            T *py = static_cast<T *>(a.y[i]) + (((long long)b * a.H[i] + h) * a.T + t) * D + c0;
            const long long sx = a.sH[i], sg = BWD ? a.gH[i] : 0, sy = (long long)a.T * D;
            float w[N], dw[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                w[e] = i ? wk[e] : wq[e];
                dw[e] = 0.f;
            }
            for (int k = 0; k < n; k += QN_ROWS) {
                Raw<T, N, VEC> rx[QN_ROWS];
                Raw<G, N, VEC> rg[BWD ? QN_ROWS : 1];
#pragma unroll
                for (int u = 0; u < QN_ROWS; ++u) {
                    const int ku = min(k + u, n - 1);
                    rx[u].load(px + ku * sx);
                    if constexpr (BWD) rg[u].load(pg + ku * sg);
                }
#pragma unroll
                for (int u = 0; u < QN_ROWS; ++u) {
                    if (k + u >= n) break;   // (the same for the whole block)
                    float x[N], y[N], ss = 0.f;
                    rx[u].get(x);
#pragma unroll
                    for (int e = 0; e < N; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, LPR);
                    const float rn = rsqrtf(fmaf(ss, 1.f / D, a.eps));
                    if constexpr (!BWD) {
#pragma unroll
                        for (int e = 0; e < N; e += 2) {
                            const float z0 = x[e] * rn * w[e], z1 = x[e + 1] * rn * w[e + 1];
                            y[e] = fmaf(z0, cs[e / 2], -z1 * sn[e / 2]);
                            y[e + 1] = fmaf(z0, sn[e / 2], z1 * cs[e / 2]);
                        }
                    } else {
                        float g[N], dn[N], dot = 0.f;
                        rg[u].get(g);
#pragma unroll
                        for (int e = 0; e < N; e += 2) {
                            const float dz0 = fmaf(g[e], cs[e / 2], g[e + 1] * sn[e / 2]);
                            const float dz1 = fmaf(g[e + 1], cs[e / 2], -g[e] * sn[e / 2]);
                            x[e] *= rn;
                            x[e + 1] *= rn;
                            dw[e] = fmaf(dz0, x[e], dw[e]);
                            dw[e + 1] = fmaf(dz1, x[e + 1], dw[e + 1]);
                            dn[e] = dz0 * w[e];
                            dn[e + 1] = dz1 * w[e + 1];
                            dot = fmaf(dn[e], x[e], fmaf(dn[e + 1], x[e + 1], dot));
                        }
#pragma unroll
                        for (int off = LPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off, LPR);
                        dot *= 1.f / D;
#pragma unroll
                        for (int e = 0; e < N; ++e) y[e] = rn * fmaf(-x[e], dot, dn[e]);
                    }
                    if (valid) store_n(py + (k + u) * sy, y);
                }
            }
            if (BWD && valid) {
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    if (i)
                        dwk[e] += dw[e];
                    else
                        dwq[e] += dw[e];
                }
            }
        }
    }
    if constexpr (BWD) {
        // sum over the block's places, then one row of partials: [block][tensor][column]
        __shared__ float sm[QN_THREADS / 32][2][D];
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float v = i ? dwk[e] : dwq[e];
#pragma unroll
                for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                if (lane < LPR) sm[warp][i][c0 + e] = v;
            }
        __syncthreads();
        const long long block = blockIdx.x;
        for (int j = threadIdx.x; j < 2 * D; j += QN_THREADS) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < QN_THREADS / 32; ++k) v += sm[k][j / D][j % D];
            a.part[block * 2 * D + j] = v;
        }
    }
}

// dw[j] = the blocks' partials of column j, one warp a column group: 32 columns by 8
// strided runs of blocks, in fp64, joined in a fixed order.
__global__ void __launch_bounds__(256) qk_norm_sum_kernel(const float *part, int n_blocks, int d, float *dwq, float *dwk) {
    __shared__ double sm[8][32];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    double v = 0.0;
    if (j < 2 * d)
        for (int b = run; b < n_blocks; b += 8) v += (double)part[(long long)b * 2 * d + j];
    sm[run][lane] = v;
    __syncthreads();
    if (run == 0 && j < 2 * d) {
#pragma unroll
        for (int k = 1; k < 8; ++k) v += sm[k][lane];
        float *dst = j < d ? dwq : dwk;
        if (dst) dst[j < d ? j : j - d] = (float)v;
    }
}

template <typename T, typename G, int LPR, bool BWD>
int launch_v(const QkNormArgs &a, const dim3 &grid, bool vec, cudaStream_t s) {
    if (vec)
        qk_norm_kernel<T, G, LPR, BWD, true><<<grid, QN_THREADS, 0, s>>>(a);
    else
        qk_norm_kernel<T, G, LPR, BWD, false><<<grid, QN_THREADS, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

template <typename T, typename G, bool BWD>
int launch_l(const QkNormArgs &a, const dim3 &grid, bool vec, cudaStream_t s) {
    switch (a.d / Lane<T>::N) {
        case 2: return launch_v<T, G, 2, BWD>(a, grid, vec, s);
        case 4: return launch_v<T, G, 4, BWD>(a, grid, vec, s);
        case 8: return launch_v<T, G, 8, BWD>(a, grid, vec, s);
        case 16: return launch_v<T, G, 16, BWD>(a, grid, vec, s);
        case 32:
            if constexpr (sizeof(T) == 4) return launch_v<T, G, 32, BWD>(a, grid, vec, s);
        default: return BA_ERR_SHAPE;
    }
}

}  // namespace

// Grid of a launch: blocks of places times splits of the rows, about `want` CTAs in all (a
// few waves); the blocks of places loop when there are more of them.
void qk_norm_grid(long long places, int rows, int d, int dtype, int num_sms, int &gx, int &gy) {
    const int tp = QN_THREADS / (d / (dtype == BA_BF16 ? 8 : 4));
    const long long blocks = (places + tp - 1) / tp, want = (long long)QN_WANT * num_sms;
    gx = (int)(blocks < want ? (blocks > 0 ? blocks : 1) : want);
    long long y = (want + gx - 1) / gx;
    const int most = (rows + QN_ROWS - 1) / QN_ROWS;
    if (y > most) y = most;
    gy = (int)(y < 1 ? 1 : y);
}

int launch_qk_norm(QkNormArgs a, bool bwd, int g_dtype, bool vec, int num_sms, float *dwq, float *dwk,
                   cudaStream_t s) {
    int gx, gy;
    qk_norm_grid(a.places, a.nb * (a.H[0] + a.H[1]), a.d, a.dtype, num_sms, gx, gy);
    a.splits = gy;
    const dim3 grid(gx * gy);
    if (!bwd)
        return a.dtype == BA_BF16 ? launch_l<__nv_bfloat16, float, false>(a, grid, vec, s)
                                  : launch_l<float, float, false>(a, grid, vec, s);
    int rc;
    if (a.dtype == BA_F32)
        rc = launch_l<float, float, true>(a, grid, vec, s);
    else if (g_dtype == BA_F32)
        rc = launch_l<__nv_bfloat16, float, true>(a, grid, vec, s);
    else
        rc = launch_l<__nv_bfloat16, __nv_bfloat16, true>(a, grid, vec, s);
    if (rc) return rc;
    qk_norm_sum_kernel<<<(2 * a.d + 31) / 32, 256, 0, s>>>(a.part, gx * gy, a.d, dwq, dwk);
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

}  // namespace ba
