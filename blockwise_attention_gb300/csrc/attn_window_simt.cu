// Windowed attention with sinks on the CUDA cores, fp32 arithmetic throughout: fp32
// inputs, bf16 with head dimension 16 or 32, and strides that TMA cannot read.
//
// O_i = sum_j p_ij v_j / l_i with the running (max, l, O) of an online softmax; see
// attn_window_fwd for the visible pairs.  What bounds it is the fp32 FMA rate: 2 d FMAs a
// pair.  A block of 128 threads takes 32 queries of one head and walks their keys (the
// sinks, then the window) 64 at a time; both products are register-tiled, 4 x 4 scores and
// 4 rows x d / 16 columns of O a thread, with the contracted index leading in shared
// memory (Q and K transposed, P transposed, V as it is), so that a step reads two (or
// three) 16-byte words for 16 (or 4 d / 16) FMAs.  32 rows a block rather than 64: a
// chunk of a prompt has few tiles, and twice the blocks fill the SMs more evenly.
#include <cuda_bf16.h>

#include "internal.h"

namespace ba {
namespace {

constexpr int WM = 32, WN = 64, WT = 128;   // queries and keys of a tile, threads
constexpr int KLD = WN + 4, QLD = WM + 4;    // leading dimensions (16-byte rows; the transposing stores run along them)

template <typename T>
__device__ __forceinline__ float4 load4(const T *p, bool vec);
template <>
__device__ __forceinline__ float4 load4(const float *p, bool vec) {
    return vec ? __ldg(reinterpret_cast<const float4 *>(p)) : make_float4(p[0], p[1], p[2], p[3]);
}
template <>
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p, bool vec) {
    if (!vec)
        return make_float4(__bfloat162float(p[0]), __bfloat162float(p[1]), __bfloat162float(p[2]), __bfloat162float(p[3]));
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

// N consecutive columns of O a thread: 1, 2, 4, or 8 as two runs of 4 (64 apart, so that
// the 16 threads of a row read 256 consecutive bytes of V at a time).
template <int N>
__device__ __forceinline__ int o_col(int tx, int c) {
    return N == 8 ? (c < 4 ? tx * 4 + c : 64 + tx * 4 + c - 4) : tx * N + c;
}

template <int D>
constexpr size_t window_simt_smem() {
    return sizeof(float) * ((size_t)D * QLD + (size_t)D * KLD + (size_t)WN * D + (size_t)WN * QLD) + WN;
}

template <int D, typename T>
__global__ void __launch_bounds__(WT) window_simt_kernel(const AttnArgs a, int vec) {
    constexpr int NC = D / 16;
    extern __shared__ __align__(16) float wsm[];
    float *Qt = wsm, *Kt = Qt + D * QLD, *Vs = Kt + D * KLD, *Pt = Vs + WN * D;   // [d][row], [d][key], [key][d], [key][row]
    uint8_t *hide = reinterpret_cast<uint8_t *>(Pt + WN * QLD);
    const Geom &g = a.g;
    const int tiles = (g.Lq + WM - 1) / WM;
    const int tile = tiles - 1 - (int)(blockIdx.x % tiles);   // the longest walks first
    const int bh = blockIdx.x / tiles, b = bh / g.H, h = bh % g.H, hk = h / g.kv_group;
    const int r0 = tile * WM, nr = min(WM, g.Lq - r0);
    const long long p0 = g.q_off + r0;   // position of the first row
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const T *qb = static_cast<const T *>(a.q) + (long long)b * a.qsB + (long long)h * a.qsH;
    const T *kb = static_cast<const T *>(a.k) + (long long)b * a.ksB + (long long)hk * a.ksH;
    const T *vb = static_cast<const T *>(a.v) + (long long)b * a.vsB + (long long)hk * a.vsH;

    for (int e = t; e < WM * (D / 4); e += WT) {
        const int r = e % WM, c = e / WM * 4;
        const float4 x = r < nr ? load4(qb + (long long)(r0 + r) * a.qsT + c, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        Qt[c * QLD + r] = x.x;
        Qt[(c + 1) * QLD + r] = x.y;
        Qt[(c + 2) * QLD + r] = x.z;
        Qt[(c + 3) * QLD + r] = x.w;
    }
    float m[4], l[4], o[4][NC];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
    }
    const long long p_last = p0 + nr - 1;
    const int end = (int)min(p_last + 1, (long long)g.Lk);
    const int lo = (int)max(0LL, p0 - g.window + 1), first = lo > g.sinks ? min(g.sinks, end) : 0;
    // chunk 0: the sinks [0, first); chunk 1: the window's keys
    for (int chunk = first > 0 ? 0 : 1; chunk < 2; ++chunk) {
        const int c0 = chunk == 0 ? 0 : (lo > g.sinks ? lo : 0), c1 = chunk == 0 ? first : end;
        for (int j0 = c0; j0 < c1; j0 += WN) {
            const int nk = min(WN, c1 - j0);
            __syncthreads();   // the previous tile is read
            if (t < WN) hide[t] = t >= nk || (g.kpm && g.kpm[(long long)b * g.kpm_ld + j0 + t]);
            __syncthreads();
            // (hidden keys are not read: what they hold has no effect)
            for (int e = t; e < WN * (D / 4); e += WT) {
                const int j = e % WN, c = e / WN * 4;
                const float4 x = hide[j] ? make_float4(0.f, 0.f, 0.f, 0.f) : load4(kb + (long long)(j0 + j) * a.ksT + c, vec);
                Kt[c * KLD + j] = x.x;
                Kt[(c + 1) * KLD + j] = x.y;
                Kt[(c + 2) * KLD + j] = x.z;
                Kt[(c + 3) * KLD + j] = x.w;
            }
            for (int e = t; e < WN * (D / 4); e += WT) {
                const int j = e / (D / 4), c = e % (D / 4) * 4;
                *reinterpret_cast<float4 *>(Vs + j * D + c) =
                    hide[j] ? make_float4(0.f, 0.f, 0.f, 0.f) : load4(vb + (long long)(j0 + j) * a.vsT + c, vec);
            }
            __syncthreads();
            float s[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 8
            for (int c = 0; c < D; ++c) {
                const float4 q4 = *reinterpret_cast<const float4 *>(Qt + c * QLD + ty * 4);
                const float4 k4 = *reinterpret_cast<const float4 *>(Kt + c * KLD + tx * 4);
                const float qv[4] = {q4.x, q4.y, q4.z, q4.w}, kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = fmaf(qv[i], kv[j], s[i][j]);
            }
            // every pair of the tile visible: the last key before the first row, the first
            // one inside the last row's window (or all of them sinks), none hidden
            const bool whole = nk == WN && j0 + WN - 1 <= p0 && (j0 > p_last - g.window || j0 + WN <= g.sinks) && !g.kpm;
            const int hid = *reinterpret_cast<const int *>(hide + tx * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long long p = p0 + ty * 4 + i;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int key = j0 + tx * 4 + j;
                    s[i][j] *= a.scale_log2;
                    if (!whole && ((hid >> (8 * j) & 0xff) || key > p || (key <= p - g.window && key >= g.sinks)))
                        s[i][j] = -INFINITY;
                    mx = fmaxf(mx, s[i][j]);
                }
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off, 16));
                const float m_new = fmaxf(m[i], mx), base = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m[i] - base);   // 0 before the first key
                m[i] = m_new;
                l[i] *= alpha;
#pragma unroll
                for (int c = 0; c < NC; ++c) o[i][c] *= alpha;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[i][j] = exp2f(s[i][j] - base);
                    l[i] += s[i][j];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4 *>(Pt + (tx * 4 + j) * QLD + ty * 4) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
            __syncwarp();   // a warp's rows of P are its own: 8 rows, all keys
            for (int j = 0; j < nk; ++j) {
                const float4 p4 = *reinterpret_cast<const float4 *>(Pt + j * QLD + ty * 4);
                const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
                float vv[NC];
                if constexpr (NC >= 4) {
#pragma unroll
                    for (int c = 0; c < NC; c += 4) {
                        const float4 v4 = *reinterpret_cast<const float4 *>(Vs + j * D + o_col<NC>(tx, c));
                        vv[c] = v4.x;
                        vv[c + 1] = v4.y;
                        vv[c + 2] = v4.z;
                        vv[c + 3] = v4.w;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < NC; ++c) vv[c] = Vs[j * D + tx * NC + c];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < NC; ++c) o[i][c] = fmaf(pv[i], vv[c], o[i][c]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sum = l[i];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off, 16);
        const int r = ty * 4 + i;
        if (r >= nr) continue;
        const long long row = (long long)bh * g.Lq + r0 + r;
        const float inv = m[i] == -INFINITY ? 0.f : 1.f / sum;   // a row without keys: zeros
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const long long at = row * D + o_col<NC>(tx, c);
            if (a.out_dtype == BA_BF16)
                static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(o[i][c] * inv);
            else
                static_cast<float *>(a.out)[at] = o[i][c] * inv;
        }
        if (tx == 0) a.lse[row] = m[i] == -INFINITY ? -INFINITY : (m[i] + log2f(sum)) * LN2;
    }
}

template <int D, typename T>
int launch_t(const AttnArgs &a, long long blocks, cudaStream_t s) {
    constexpr size_t smem = window_simt_smem<D>();
    auto kern = window_simt_kernel<D, T>;
    static std::atomic<unsigned long long> allowed{0};
    if (!allow_smem(allowed, reinterpret_cast<const void *>(kern), (int)smem)) return BA_ERR_CUDA;
    // rows read four elements at a time where every row is aligned for it
    const long long step = 4;
    auto fits = [&](const void *p, long long sB, long long sH, long long sT) {
        return reinterpret_cast<uintptr_t>(p) % (step * sizeof(T)) == 0 && sB % step == 0 && sH % step == 0 && sT % step == 0;
    };
    const int vec = fits(a.q, a.qsB, a.qsH, a.qsT) && fits(a.k, a.ksB, a.ksH, a.ksT) && fits(a.v, a.vsB, a.vsH, a.vsT);
    kern<<<(unsigned)blocks, WT, smem, s>>>(a, vec);
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

template <int D>
int launch_d(const AttnArgs &a, long long blocks, cudaStream_t s) {
    return a.dtype == BA_F32 ? launch_t<D, float>(a, blocks, s) : launch_t<D, __nv_bfloat16>(a, blocks, s);
}

}  // namespace

int launch_window_simt(const AttnArgs &a, cudaStream_t s) {
    const long long blocks = (long long)((a.g.Lq + WM - 1) / WM) * a.g.B * a.g.H;
    if (blocks == 0) return BA_OK;
    if (blocks > 0x7fffffffLL) return BA_ERR_SHAPE;
    switch (a.g.d) {
        case 16: return launch_d<16>(a, blocks, s);
        case 32: return launch_d<32>(a, blocks, s);
        case 64: return launch_d<64>(a, blocks, s);
        case 128: return launch_d<128>(a, blocks, s);
        default: return BA_ERR_SHAPE;
    }
}

}  // namespace ba
