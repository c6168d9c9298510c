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
// registers until the end.  Four rows' loads are in flight per thread.
// Angles: m theta / 2 pi in fp64 less its nearest integer (exact for |m| < 2^31 but for
// the 2^-53 of the product), then sincospi in fp32: far positions cost no accuracy.
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

// N consecutive values of T from p: 16-byte loads when VEC, else one by one.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void load_n(const T *p, float (&x)[N]) {
    if constexpr (VEC && sizeof(T) == 2) {
        static_assert(N % 8 == 0 || N == 4, "16- or 8-byte pieces");
        if constexpr (N == 4) {
            const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p));
            x[0] = __uint_as_float(u.x << 16);
            x[1] = __uint_as_float(u.x & 0xffff0000u);
            x[2] = __uint_as_float(u.y << 16);
            x[3] = __uint_as_float(u.y & 0xffff0000u);
        } else {
            const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    } else if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 u = __ldcs(reinterpret_cast<const float4 *>(p) + i);
            x[4 * i] = u.x;
            x[4 * i + 1] = u.y;
            x[4 * i + 2] = u.z;
            x[4 * i + 3] = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 2)
                x[i] = __bfloat162float(p[i]);
            else
                x[i] = p[i];
        }
    }
}

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
__global__ void __launch_bounds__(QN_THREADS) qk_norm_kernel(const QkNormArgs a) {
    constexpr int N = Lane<T>::N, TP = QN_THREADS / LPR, D = LPR * N;
    const int place = threadIdx.x / LPR, gl = threadIdx.x % LPR, c0 = gl * N;
    const int HT = a.H[0] + a.H[1];
    const int rows = a.nb * HT;   // of a place: (sequence, head), the queries' heads first
    const int per = (rows + gridDim.y - 1) / gridDim.y, r_begin = blockIdx.y * per, r_end = min(rows, r_begin + per);
    float w[2][N], dw[2][N];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            w[i][e] = a.H[i] ? weight(a.w[i], a.w_f32, c0 + e) : 0.f;
            dw[i][e] = 0.f;
        }
    for (long long p0 = (long long)blockIdx.x * TP; p0 < a.places; p0 += (long long)gridDim.x * TP) {
        // (lanes behind the last place stay for the shuffles: they repeat the last place and store nothing)
        const bool valid = p0 + place < a.places;
        const long long at = valid ? p0 + place : a.places - 1;
        const int t = (int)(at % a.T), b0 = (int)(at / a.T);   // b0 = 0 when the sequences share their positions
        const double m = (a.positions ? (double)a.positions[(long long)b0 * a.pos_ld + t] : (double)t) * a.pos_scale;
        float cs[N / 2], sn[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const double turns = m * a.turn[c0 / 2 + i];
            sincospif((float)(2.0 * (turns - rint(turns))), &sn[i], &cs[i]);
        }
        for (int r0 = r_begin; r0 < r_end; r0 += QN_ROWS) {
            float x[QN_ROWS][N], g[BWD ? QN_ROWS : 1][N];
            int ti[QN_ROWS];
            long long out[QN_ROWS];
#pragma unroll
            for (int u = 0; u < QN_ROWS; ++u) {
                const int r = min(r0 + u, r_end - 1), bi = r / HT, hh = r % HT, b = b0 + bi;
                ti[u] = hh >= a.H[0];
                const int i = ti[u], h = hh - (i ? a.H[0] : 0);
                load_n<T, N, VEC>(static_cast<const T *>(a.x[i]) + b * a.sB[i] + h * a.sH[i] + t * a.sT[i] + c0, x[u]);
                if constexpr (BWD)
                    load_n<G, N, VEC>(static_cast<const G *>(a.g[i]) + b * a.gB[i] + h * a.gH[i] + t * a.gT[i] + c0, g[u]);
                out[u] = (((long long)b * a.H[i] + h) * a.T + t) * D + c0;
            }
#pragma unroll
            for (int u = 0; u < QN_ROWS; ++u) {
                const bool live = valid && r0 + u < r_end;
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < N; ++e) ss = fmaf(x[u][e], x[u][e], ss);
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, LPR);
                const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
                float y[N];
                if constexpr (!BWD) {
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float z0 = x[u][e] * r * (ti[u] ? w[1][e] : w[0][e]);
                        const float z1 = x[u][e + 1] * r * (ti[u] ? w[1][e + 1] : w[0][e + 1]);
                        y[e] = fmaf(z0, cs[e / 2], -z1 * sn[e / 2]);
                        y[e + 1] = fmaf(z0, sn[e / 2], z1 * cs[e / 2]);
                    }
                } else {
                    float dn[N], dot = 0.f;
#pragma unroll
                    for (int e = 0; e < N; e += 2) {
                        const float dz0 = fmaf(g[u][e], cs[e / 2], g[u][e + 1] * sn[e / 2]);
                        const float dz1 = fmaf(g[u][e + 1], cs[e / 2], -g[u][e] * sn[e / 2]);
                        x[u][e] *= r;
                        x[u][e + 1] *= r;
                        if (live) {
                            const float a0 = dz0 * x[u][e], a1 = dz1 * x[u][e + 1];
                            if (ti[u]) {
                                dw[1][e] += a0;
                                dw[1][e + 1] += a1;
                            } else {
                                dw[0][e] += a0;
                                dw[0][e + 1] += a1;
                            }
                        }
                        dn[e] = dz0 * (ti[u] ? w[1][e] : w[0][e]);
                        dn[e + 1] = dz1 * (ti[u] ? w[1][e + 1] : w[0][e + 1]);
                        dot = fmaf(dn[e], x[u][e], fmaf(dn[e + 1], x[u][e + 1], dot));
                    }
#pragma unroll
                    for (int off = LPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off, LPR);
                    dot *= 1.f / D;
#pragma unroll
                    for (int e = 0; e < N; ++e) y[e] = r * fmaf(-x[u][e], dot, dn[e]);
                }
                if (live) store_n(static_cast<T *>(a.y[ti[u]]) + out[u], y);
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
                float v = dw[i][e];
#pragma unroll
                for (int off = LPR; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
                if (lane < LPR) sm[warp][i][c0 + e] = v;
            }
        __syncthreads();
        const long long block = (long long)blockIdx.y * gridDim.x + blockIdx.x;
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

// Grid of a launch: blocks of places times splits of the rows, about `want` blocks in
// all; the blocks of places loop when there are more of them.
void qk_norm_grid(long long places, int rows, int d, int dtype, int num_sms, int &gx, int &gy) {
    const int tp = QN_THREADS / (d / (dtype == BA_BF16 ? 8 : 4));
    const long long blocks = (places + tp - 1) / tp, want = 6LL * num_sms;
    gx = (int)(blocks < want ? (blocks > 0 ? blocks : 1) : want);
    long long y = want / gx;
    const int most = (rows + QN_ROWS - 1) / QN_ROWS;
    if (y > most) y = most;
    gy = (int)(y < 1 ? 1 : y);
}

int launch_qk_norm(const QkNormArgs &a, bool bwd, int g_dtype, bool vec, int num_sms, float *dwq, float *dwk,
                   cudaStream_t s) {
    int gx, gy;
    qk_norm_grid(a.places, a.nb * (a.H[0] + a.H[1]), a.d, a.dtype, num_sms, gx, gy);
    const dim3 grid(gx, gy);
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
