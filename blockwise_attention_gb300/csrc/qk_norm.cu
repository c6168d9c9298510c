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
// registers until the end.  The next rows' loads are in flight while a thread works.
// Angles: a turn's fraction is m times base^(-2c/d) / 2 pi held as a 64-bit fraction,
// modulo 2^64: exact integer arithmetic, so that far positions cost no accuracy (the
// fraction's own error is 2^-53 relative, times m) and no fp64 instruction, of which an
// SM has few; then sincospi in fp32.  (Product and reduction in fp64, and one block of
// positions a CTA: 8K positions, 2 sequences, 20 heads, forward 54 us.)
// dw: every block writes its sums, a second launch adds the blocks' in a fixed order (no
// atomics).
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "internal.h"

namespace ba {
namespace {

constexpr int QN_THREADS = 256;
constexpr int QN_ROWS = 4;   // least rows of a CTA's share

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
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i)
                w[i] = (uint32_t)__bfloat16_as_ushort(p[2 * i]) | (uint32_t)__bfloat16_as_ushort(p[2 * i + 1]) << 16;
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) w[i] = __float_as_uint(p[i]);
        }
    }
    __device__ __forceinline__ void put(const uint4 *at, int step) {   // from shared memory, 16-byte words `step` apart
#pragma unroll
        for (int i = 0; i < WORDS / 4; ++i) {
            const uint4 u = at[i * step];
            w[4 * i] = u.x;
            w[4 * i + 1] = u.y;
            w[4 * i + 2] = u.z;
            w[4 * i + 3] = u.w;
        }
    }
    __device__ __forceinline__ void get(float2 (&x)[N / 2]) const {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            if constexpr (sizeof(T) == 2)
                x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else
                x[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
};

__device__ __forceinline__ void store_n(__nv_bfloat16 *p, const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 z = __floats2bfloat162_rn(x[i].x, x[i].y);
        w[i] = *reinterpret_cast<const uint32_t *>(&z);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
__device__ __forceinline__ void store_n(float *p, const float2 (&x)[2]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(x[0].x, x[0].y, x[1].x, x[1].y));
}

// Two fp32 lanes an instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
// v.x m0 + v.y m1 (one lane at a time: the packed form would first have to copy v.x and v.y)
__device__ __forceinline__ float2 turn(float2 v, float2 m0, float2 m1) {
    return make_float2(fmaf(v.x, m0.x, v.y * m1.x), fmaf(v.x, m0.y, v.y * m1.y));
}

__device__ __forceinline__ float weight(const void *w, int f32, int c) {
    return f32 ? static_cast<const float *>(w)[c] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Rows in the ring.
template <bool BWD>
constexpr int ring_rows = BWD ? 6 : 8;

// T: type of x and y (dx); G: type of dy; LPR: lanes a row.
template <typename T, typename G, int LPR, bool BWD, bool VEC>
__global__ void __launch_bounds__(QN_THREADS, 3) qk_norm_kernel(const QkNormArgs a) {
    constexpr int NS = ring_rows<BWD>;
    constexpr int N = Lane<T>::N, P = N / 2, TP = QN_THREADS / LPR, D = LPR * N;
    const int place = threadIdx.x / LPR, gl = threadIdx.x % LPR, c0 = gl * N;
    const int HT = a.H[0] + a.H[1];
    const int rows = a.nb * HT;   // of a place: (sequence, head), the queries' heads first
    int r_begin = 0, r_end = 0;   // of the block of places at work
    __shared__ float2 sw[2][D / 2];   // the weights
    float2 dwq[BWD ? P : 1], dwk[BWD ? P : 1];
#pragma unroll
    for (int e = 0; e < (BWD ? P : 1); ++e) dwq[e] = dwk[e] = both(0.f);

    // Rows come through a ring in shared memory, ring_rows ahead of the row at work: every
    // lane copies its own 16 bytes (32 of an fp32 dy beside bf16 rows) with cp.async and
    // reads them back itself, so that tens of KB are in flight per SM without registers
    // or barriers.  Rows that 16-byte copies cannot read are loaded where they are used.
    extern __shared__ __align__(16) uint4 ring[];
    constexpr int GW = BWD ? Raw<G, N, VEC>::WORDS / 4 : 0, WORDS = 1 + GW;   // 16-byte words a row and lane
    const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
    struct Cursor {
        const T *px;
        const G *pg;
        T *py;
        long long sx, sg;
        int r, i, left;   // row, tensor, rows of the same tensor and sequence from this one on
    };
    int b0 = 0, t = 0;
    auto open = [&](Cursor &q, int r) {
        const int bi = r / HT, hh = r - bi * HT, b = b0 + bi;
        q.r = r;
        q.i = hh >= a.H[0] ? 1 : 0;
        const int h = hh - (q.i ? a.H[0] : 0);
        q.left = a.H[q.i] - h;
        q.sx = a.sH[q.i];
        q.px = static_cast<const T *>(a.x[q.i]) + b * a.sB[q.i] + h * q.sx + t * a.sT[q.i] + c0;
        if constexpr (BWD) {
            q.sg = a.gH[q.i];
            q.pg = static_cast<const G *>(a.g[q.i]) + b * a.gB[q.i] + h * q.sg + t * a.gT[q.i] + c0;
        }
        q.py = static_cast<T *>(a.y[q.i]) + (((long long)b * a.H[q.i] + h) * a.T + t) * D + c0;
    };
    const long long sy = (long long)a.T * D;
    auto next = [&](Cursor &q) {
        if (q.left == 1) {
            if (q.r + 1 < r_end)
                open(q, q.r + 1);
            else
                ++q.r;
            return;
        }
        ++q.r;
        --q.left;
        q.px += q.sx;
        if constexpr (BWD) q.pg += q.sg;
        q.py += sy;
    };
    auto issue = [&](Cursor &q, int slot) {   // the row at q into a slot, and q to the next
        if (q.r < r_end) {
            const uint32_t at = mine + slot * (WORDS * QN_THREADS * 16);
            cp16(at, q.px);
            if constexpr (BWD) {
#pragma unroll
                for (int k = 0; k < GW; ++k) cp16(at + (1 + k) * (QN_THREADS * 16), q.pg + k * (16 / (int)sizeof(G)));
            }
            next(q);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");   // a group each time, so that the count below holds
    };
    bool valid = false;
    float cs[P], sn[P];
    // (v0, v1) -> v0 m0 + v1 m1: the weighted rotation (forward), or the transposed rotation
    // of dy, before the weights w (backward); of tensor `of`
    float2 m0[P], m1[P], w[BWD ? P : 1];
    int of = -1;
    auto work = [&](const Cursor &q, const Raw<T, N, VEC> &dx, const Raw<G, N, VEC> &dg) {
        if (q.i != of) {   // (the same for the whole block)
            of = q.i;
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float2 v = sw[of][c0 / 2 + e];
                if constexpr (BWD) {
                    w[e] = v;
                    m0[e] = make_float2(cs[e], -sn[e]);
                    m1[e] = make_float2(sn[e], cs[e]);
                } else {
                    m0[e] = make_float2(v.x * cs[e], v.x * sn[e]);
                    m1[e] = make_float2(-v.y * sn[e], v.y * cs[e]);
                }
            }
        }
            float2 x[P], y[P], s2 = both(0.f);
            dx.get(x);
#pragma unroll
            for (int e = 0; e < P; ++e) s2 = fma2(x[e], x[e], s2);
            float ss = s2.x + s2.y;
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off, LPR);
            const float2 rn2 = both(rsqrtf(fmaf(ss, 1.f / D, a.eps)));
            if constexpr (!BWD) {
#pragma unroll
                for (int e = 0; e < P; ++e) y[e] = mul2(turn(x[e], m0[e], m1[e]), rn2);
            } else {
                float2 g[P], d2 = both(0.f);
                dg.get(g);
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const float2 dz = turn(g[e], m0[e], m1[e]);
                    x[e] = mul2(x[e], rn2);
                    if (valid) {
                        if (q.i)
                            dwk[e] = fma2(dz, x[e], dwk[e]);
                        else
                            dwq[e] = fma2(dz, x[e], dwq[e]);
                    }
                    y[e] = mul2(dz, w[e]);
                    d2 = fma2(y[e], x[e], d2);
                }
                float dot = d2.x + d2.y;
#pragma unroll
                for (int off = LPR / 2; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off, LPR);
                const float2 dot2 = both(dot * (-1.f / D));
#pragma unroll
                for (int e = 0; e < P; ++e) y[e] = mul2(fma2(x[e], dot2, y[e]), rn2);
            }
            if (valid) store_n(q.py, y);
    };
    bool weights_there = false;
    // The CTA's run: units (block of places, row), rows fastest, an equal share of all.
    const long long units = (a.places + TP - 1) / TP * rows, u1 = min(units, (blockIdx.x + 1LL) * a.run);
    for (long long u0 = (long long)blockIdx.x * a.run; u0 < u1; u0 += r_end - r_begin) {
        const long long p0 = u0 / rows * TP;
        r_begin = (int)(u0 % rows);
        r_end = (int)min((long long)rows, r_begin + (u1 - u0));
        // (lanes behind the last place stay for the shuffles: they repeat the last place and store nothing)
        valid = p0 + place < a.places;
        const long long at = valid ? p0 + place : a.places - 1;
        b0 = a.nb == 1 && a.places != a.T ? (int)(at / a.T) : 0;
        t = (int)(at - (long long)b0 * a.T);
        Cursor q, ahead;
        open(q, r_begin);
        if constexpr (VEC) {
            ahead = q;
            for (int k = 0; k < NS - 1; ++k) issue(ahead, k);
        }
        if (!weights_there) {
            for (int j = threadIdx.x; j < D; j += QN_THREADS) {
                const int i = j / (D / 2), c = j % (D / 2) * 2;
                sw[i][c / 2] = a.H[i] ? make_float2(weight(a.w[i], a.w_f32, c), weight(a.w[i], a.w_f32, c + 1)) : both(0.f);
            }
            __syncthreads();
            weights_there = true;
        }
        const int m = a.positions ? a.positions[(long long)b0 * a.pos_ld + t] : t;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int turns = (int)(((unsigned long long)(long long)m * a.turn[c0 / 2 + i]) >> 32);   // [-1/2, 1/2) turns
            sincospif((float)turns * 0x1p-31f, &sn[i], &cs[i]);
        }
        of = -1;
        for (int slot = 0; q.r < r_end;) {
            Raw<T, N, VEC> dx;
            Raw<G, N, VEC> dg;
            if constexpr (VEC) {
                issue(ahead, slot == 0 ? NS - 1 : slot - 1);   // into the slot read a step ago
                asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
                const uint4 *at = ring + slot * (WORDS * QN_THREADS) + threadIdx.x;
                dx.put(at, QN_THREADS);
                if constexpr (BWD) dg.put(at + QN_THREADS, QN_THREADS);
                slot = slot == NS - 1 ? 0 : slot + 1;
            } else {
                dx.load(q.px);
                if constexpr (BWD) dg.load(q.pg);
            }
            work(q, dx, dg);
            next(q);
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
                const float2 pair = i ? dwk[e / 2] : dwq[e / 2];
                float v = e % 2 ? pair.y : pair.x;
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

// dw[j] = the sum of the blocks' partials of column j, in a fixed order: 32 columns a block,
// 32 runs of blocks beside each other with eight loads in flight each, then the runs.  In
// fp32: a column's chain is n_blocks / 32 + 32 additions of partials that are sums
// themselves (in fp64, of which an SM has few units: 13 us).
__global__ void __launch_bounds__(1024) qk_norm_sum_kernel(const float *part, int n_blocks, int d, float *dwq, float *dwk) {
    __shared__ float sm[32][33];
    const int lane = threadIdx.x & 31, run = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (j < 2 * d) {
        const float *p = part + j;
        for (int b0 = run; b0 < n_blocks; b0 += 256) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = b0 + 32 * k < n_blocks ? __ldcg(p + (long long)(b0 + 32 * k) * 2 * d) : 0.f;
            v += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        }
    }
    sm[run][lane] = v;
    __syncthreads();
    // warp `run` joins column `run`: its lanes the runs
    v = sm[lane][run];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    const int c = blockIdx.x * 32 + run;
    if (lane == 0 && c < 2 * d) {
        float *dst = c < d ? dwq : dwk;
        if (dst) dst[c < d ? c : c - d] = v;
    }
}

template <typename T, typename G, int LPR, bool BWD>
int launch_v(const QkNormArgs &a, const dim3 &grid, bool vec, cudaStream_t s) {
    constexpr size_t ring = (size_t)ring_rows<BWD> * (1 + (BWD ? Lane<T>::N * sizeof(G) / 16 : 0)) * QN_THREADS * 16;
    if (vec) {
        auto kern = qk_norm_kernel<T, G, LPR, BWD, true>;
        static std::atomic<unsigned long long> allowed{0};
        if (!allow_smem(allowed, reinterpret_cast<const void *>(kern), (int)ring)) return BA_ERR_CUDA;
        kern<<<grid, QN_THREADS, ring, s>>>(a);
    } else
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

// CTAs of a launch and the rows (of a block of places) that each takes: one wave of three
// an SM, every CTA the same number (a run may end one block of places and begin the next),
// but no fewer than four.  (Whole blocks of places instead, 512 of them on 456 places of a
// wave: 8K positions, the slowest CTAs took twice the others.)
void qk_norm_grid(long long places, int rows, int d, int dtype, int num_sms, int &ctas, int &run) {
    const int tp = QN_THREADS / (d / (dtype == BA_BF16 ? 8 : 4));
    const long long units = (places + tp - 1) / tp * rows, most = 3LL * num_sms;
    long long n = (units + most - 1) / most;
    if (n < QN_ROWS) n = QN_ROWS;
    run = (int)n;
    ctas = (int)((units + n - 1) / n);
    if (ctas < 1) ctas = 1;
}

int launch_qk_norm(QkNormArgs a, bool bwd, int g_dtype, bool vec, int num_sms, float *dwq, float *dwk,
                   cudaStream_t s) {
    int ctas;
    qk_norm_grid(a.places, a.nb * (a.H[0] + a.H[1]), a.d, a.dtype, num_sms, ctas, a.run);
    const dim3 grid(ctas);
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
    qk_norm_sum_kernel<<<(2 * a.d + 31) / 32, 1024, 0, s>>>(a.part, ctas, a.d, dwq, dwk);
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

}  // namespace ba
