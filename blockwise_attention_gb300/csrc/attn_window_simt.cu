// Windowed attention with sinks on the CUDA cores, fp32 arithmetic throughout: fp32
// inputs, bf16 with head dimension 16 or 32, and strides that TMA cannot read.
//
// O_i = sum_j p_ij v_j / l_i with the running (max, l, O) of an online softmax; see
// attn_window_fwd for the visible pairs.  What bounds it is the fp32 FMA rate: 2 d FMAs a
// pair.  A block of 128 threads takes 32 queries of one head and walks their keys (the
// sinks and the window as one range) 64 at a time; both products are register-tiled, 4 x 4
// scores and 4 rows x d / 16 columns of O a thread, with the contracted index leading in
// shared memory (Q and K transposed, P transposed, V as it is), so that a step reads two (or
// three) 16-byte words for 16 (or 4 d / 16) FMAs.  32 rows a block rather than 64: a
// chunk of a prompt has few tiles, and twice the blocks fill the SMs more evenly.
// 2 x 765 queries behind 259, 8 heads of 64, window 257: 47.5 us (a thread a row: 258; the
// sinks as a tile of their own and K read a row a lane: 59; K and V loaded where they are
// needed instead of ahead: 55).  2.5 blocks of four warps an SM hide little of the rest of
// what they wait for in shared memory.
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

// Row and column of a thread's four values when R rows are read and stored transposed: a warp
// takes 8 rows of 64 bytes (fp32), 16 lines instead of the 32 of a row a lane, and its
// stores meet two to a bank.
template <int R>
__device__ __forceinline__ void transposed_place(int e, int &row, int &col) {
    const int lane = e & 31, w = e >> 5;
    row = w % (R / 8) * 8 + (lane & 7);
    col = (w / (R / 8) * 4 + (lane >> 3)) * 4;
}

template <int D>
constexpr size_t window_simt_smem() {
    return sizeof(float) * ((size_t)D * QLD + (size_t)D * KLD + (size_t)WN * D + (size_t)WN * QLD) + 2 * WN;
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
        int r, c;
        transposed_place<WM>(e, r, c);
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
    // The keys that the rows see as one range without a gap: the sinks before the window, then its keys.
    const int shift = lo > g.sinks ? lo - first : 0, n = lo > g.sinks ? first + max(0, end - lo) : end;
    auto key_at = [&](int i) { return i < first ? i : i + shift; };
    // The next tile's K is loaded into registers while this one is worked on, V (fp32) by
    // cp.async while the scores are formed.  Hidden keys are not read: what they hold has no effect.
    constexpr int KN = D * WN / 4 / WT;
    const bool async = sizeof(T) == 4 && vec;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 next[KN];
    auto mark = [&](int j0, uint8_t *hd) {
        if (t < WN) hd[t] = j0 + t >= n || (g.kpm && g.kpm[(long long)b * g.kpm_ld + key_at(j0 + t)]);
    };
    auto fetch = [&](int j0, const uint8_t *hd) {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            int j, c;
            transposed_place<WN>(t + i * WT, j, c);
            next[i] = hd[j] ? zero : load4(kb + (long long)key_at(j0 + j) * a.ksT + c, vec);
        }
    };
    mark(0, hide);
    __syncthreads();
    fetch(0, hide);
    for (int j0 = 0; j0 < n; j0 += WN) {
        const int nk = min(WN, n - j0);
        uint8_t *hd = hide + (j0 / WN & 1) * WN, *hd_next = hide + (~(j0 / WN) & 1) * WN;
        __syncthreads();   // the previous tile is read
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            int j, c;
            transposed_place<WN>(t + i * WT, j, c);
            Kt[c * KLD + j] = next[i].x;
            Kt[(c + 1) * KLD + j] = next[i].y;
            Kt[(c + 2) * KLD + j] = next[i].z;
            Kt[(c + 3) * KLD + j] = next[i].w;
        }
        for (int e = t; e < WN * (D / 4); e += WT) {
            const int j = e / (D / 4), c = e % (D / 4) * 4;
            const T *from = vb + (long long)(hd[j] ? 0 : key_at(j0 + j)) * a.vsT + c;
            if (async)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(Vs + j * D + c)),
                             "l"(from), "r"(hd[j] ? 0 : 16)
                             : "memory");
            else
                *reinterpret_cast<float4 *>(Vs + j * D + c) = hd[j] ? zero : load4(from, vec);
        }
        if (j0 + WN < n) mark(j0 + WN, hd_next);
        __syncthreads();
        if (j0 + WN < n) fetch(j0 + WN, hd_next);
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
        const int k_lo = key_at(j0), k_hi = key_at(j0 + WN - 1);
        const bool whole = nk == WN && k_hi <= p0 && (k_lo > p_last - g.window || k_hi < g.sinks) && !g.kpm;
        const int hid = *reinterpret_cast<const int *>(hd + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long p = p0 + ty * 4 + i;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int key = key_at(j0 + tx * 4 + j);
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
        if (async) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();   // V
        } else {
            __syncwarp();   // a warp's rows of P are its own: 8 rows, all keys
        }
        const int nk8 = (nk + 7) / 8 * 8;   // (P and V are zero behind nk)
#pragma unroll 8
        for (int j = 0; j < nk8; ++j) {
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

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------

// dS = P * (dO V^T - D) with P = exp(S - lse); dV = P^T dO, dK = scale dS^T Q, dQ = scale dS K.
// A block holds 32 rows of one side (of a key head: K, V; of a query head: Q, dO) and walks
// the rows of the other that its window reaches, NY at a time: both score products, then
// the products into its own rows' sums, all register-tiled as in the forward (4 rows x NY / 16
// scores, 4 rows x d / 16 sums a thread).  Rows lie as they are in shared memory, padded by 16
// bytes, so the score products read four columns of a row at a time.  The key side's blocks
// take their query rows once for each head of the group; a key tile that holds sinks is seen by
// every later query, whose rows are cut into chunks with a partial each (launch_sink_sum).
// Both sides in one launch: short sequences have few blocks of either.  fp32 FMAs bound it,
// 4 d a pair on the key side and 3 d on the query side, and the length of a key block's walk
// where there are few: 2 x 24 query and 3 key heads, 346 tokens, d = 128, window 125: 541 us
// (the kernels of attn_block_bwd over the window's spans, four scores a thread: 1725);
// 4 heads, 900 tokens, d = 64, window 100: 46 us (172).
constexpr int BM = WINDOW_SIMT_ROWS;

template <int D>
constexpr int NY = D == 128 ? 32 : 64;   // (64 rows of 128 would leave one block on an SM)

template <int D>
constexpr size_t window_bwd_smem() {
    return sizeof(float) * ((size_t)2 * BM * (D + 4) + (size_t)2 * NY<D> * (D + 4) + (size_t)2 * NY<D> * (BM + 4) + 2 * NY<D>) +
           NY<D>;
}

template <typename T>
__device__ __forceinline__ const T *row_of(const TensorRef &t, int b, int h, long long row) {
    return static_cast<const T *>(t.p) + (long long)b * t.sB + (long long)h * t.sH + row * t.sT;
}

__device__ __forceinline__ void put(const BwdArgs &a, void *base, long long i, float v) {   // rounded once, if at all
    if (a.grad_bf16)
        static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(base)[i] = v;
}

__device__ __forceinline__ float dot4(const float4 &x, const float4 &y, float acc) {
    return fmaf(x.w, y.w, fmaf(x.z, y.z, fmaf(x.y, y.y, fmaf(x.x, y.x, acc))));
}

template <int D, typename T, bool KEYS>
__device__ __forceinline__ void window_bwd_block(const BwdArgs &a, int item, bool vec, float *sm) {
    constexpr int LD = D + 4, SLD = BM + 4, N = NY<D>, NJ = N / 16, NC = D / 16;
    float *X1 = sm, *X2 = X1 + BM * LD, *Y1 = X2 + BM * LD, *Y2 = Y1 + N * LD;   // rows: K, V | Q, dO and the other side's
    float *Ps = Y2 + N * LD, *Ss = Ps + N * SLD, *yl = Ss + N * SLD, *yd = yl + N;
    uint8_t *hide = reinterpret_cast<uint8_t *>(yd + N);
    const int t = threadIdx.x, tx = t & 15, ty = t >> 4;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);

    // the block's rows, and the ranges of the other side's
    const int tiles = (int)(((KEYS ? a.Lk : a.Lq) + (long long)BM - 1) / BM);
    int tile, part = -1, bh;
    if (KEYS) {
        const int parts = a.n_sink_tiles * a.n_sink_parts, items = tiles - a.n_sink_tiles + parts;
        bh = item / items;
        tile = item % items;
        if (tile < parts) {
            part = tile % a.n_sink_parts;
            tile /= a.n_sink_parts;
        } else {
            tile += a.n_sink_tiles - parts;
        }
    } else {
        bh = item / tiles;
        tile = tiles - 1 - item % tiles;   // the longest walks first
    }
    const int heads = KEYS ? a.Hkv : a.H, b = bh / heads, h = bh % heads;
    const int r0 = tile * BM, nr = min(BM, (KEYS ? a.Lk : a.Lq) - r0);
    // (query side: the keys as one range without a gap, as in the forward)
    long long lo = 0, hi, first = 0, shift = 0;
    if (KEYS) {
        lo = r0 - a.q_off;
        hi = (long long)r0 + nr - 1 + a.window - a.q_off;
        if (part >= 0) {
            lo = max(lo, (long long)part * a.sink_rows);
            hi = (long long)(part + 1) * a.sink_rows;
        } else if (r0 < a.sinks) {
            hi = a.Lq;   // one chunk covers every query
        }
        lo = max(lo, 0LL);
        hi = min(hi, (long long)a.Lq);
    } else {
        const long long p0 = a.q_off + r0, end = min(p0 + nr, (long long)a.Lk), from = max(0LL, p0 - a.window + 1);
        if (from > a.sinks) {
            first = min((long long)a.sinks, end);
            shift = from - first;
            hi = first + max(0LL, end - from);
        } else {
            hi = end;
        }
    }
    auto at = [&](long long y) { return KEYS || y < first ? y : y + shift; };
    auto hidden = [&](long long key) { return a.kpm && a.kpm[(long long)b * a.kpm_ld + key]; };
    for (int e = t; e < BM * (D / 4); e += WT) {   // (a hidden key's rows may hold anything and are not read)
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        const bool in = r < nr && !(KEYS && hidden(r0 + r));
        *reinterpret_cast<float4 *>(X1 + r * LD + c) = in ? load4(row_of<T>(KEYS ? a.k : a.q, b, h, r0 + r) + c, vec) : zero;
        *reinterpret_cast<float4 *>(X2 + r * LD + c) = in ? load4(row_of<T>(KEYS ? a.v : a.dout, b, h, r0 + r) + c, vec) : zero;
    }
    bool in[4];
    float xl[4], xd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        in[i] = r < nr && !(KEYS && hidden(r0 + r));
        xl[i] = xd[i] = 0.f;
        if (!KEYS && in[i]) {
            const long long row = ((long long)b * a.H + h) * a.Lq + r0 + r;
            xl[i] = a.lse[row];
            xd[i] = a.D[row];
            in[i] = xl[i] != -INFINITY;
            xl[i] *= LOG2E;
        }
    }
    float acc1[4][NC], acc2[4][NC];   // dK and dV, or dQ
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            acc1[i][c] = 0.f;
            if (KEYS) acc2[i][c] = 0.f;
        }
    const float sl2 = a.scale * LOG2E;

    for (int step = 0; step < (KEYS ? a.kv_group : 1); ++step) {
        const int hy = KEYS ? h * a.kv_group + step : h / a.kv_group;   // the other side's head
        for (long long y0 = lo; y0 < hi; y0 += N) {
            const int ny = (int)min((long long)N, hi - y0);
            __syncthreads();   // the previous rows are read
            if (t < N) {
                if (KEYS) {
                    const long long row = ((long long)b * a.H + hy) * a.Lq + y0 + t;
                    const float l = t < ny ? a.lse[row] : -INFINITY;
                    hide[t] = l == -INFINITY;
                    yl[t] = l * LOG2E;
                    yd[t] = t < ny ? a.D[row] : 0.f;
                } else {
                    hide[t] = t >= ny || hidden(at(y0 + t));
                }
            }
            __syncthreads();
            for (int e = t; e < N * (D / 4); e += WT) {
                const int y = e / (D / 4), c = e % (D / 4) * 4;
                const bool use = !hide[y];
                *reinterpret_cast<float4 *>(Y1 + y * LD + c) = use ? load4(row_of<T>(KEYS ? a.q : a.k, b, hy, at(y0 + y)) + c, vec) : zero;
                *reinterpret_cast<float4 *>(Y2 + y * LD + c) =
                    use ? load4(row_of<T>(KEYS ? a.dout : a.v, b, hy, at(y0 + y)) + c, vec) : zero;
            }
            __syncthreads();
            float s[4][NJ], g[4][NJ];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) s[i][j] = g[i][j] = 0.f;
#pragma unroll 2
            for (int c = 0; c < D; c += 4) {
                float4 x[4], y[NJ];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(X1 + (ty * 4 + i) * LD + c);
#pragma unroll
                for (int j = 0; j < NJ; ++j) y[j] = *reinterpret_cast<const float4 *>(Y1 + (tx + 16 * j) * LD + c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4 *>(X2 + (ty * 4 + i) * LD + c);
#pragma unroll
                for (int j = 0; j < NJ; ++j) y[j] = *reinterpret_cast<const float4 *>(Y2 + (tx + 16 * j) * LD + c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) g[i][j] = dot4(x[i], y[j], g[i][j]);
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int y = tx + 16 * j;
                const bool use = !hide[y];
                const float l = KEYS ? yl[y] : 0.f, dd = KEYS ? yd[y] : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long p = a.q_off + (KEYS ? y0 + y : (long long)r0 + ty * 4 + i);
                    const long long key = KEYS ? (long long)r0 + ty * 4 + i : at(y0 + y);
                    float pr = 0.f, ds = 0.f;
                    if (use && in[i] && key <= p && (key > p - a.window || key < a.sinks)) {
                        pr = exp2f(fmaf(s[i][j], sl2, -(KEYS ? l : xl[i])));
                        ds = pr * (g[i][j] - (KEYS ? dd : xd[i]));
                    }
                    s[i][j] = pr;
                    g[i][j] = ds;
                }
                *reinterpret_cast<float4 *>(Ss + y * SLD + ty * 4) = make_float4(g[0][j], g[1][j], g[2][j], g[3][j]);
                if (KEYS) *reinterpret_cast<float4 *>(Ps + y * SLD + ty * 4) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
            }
            __syncwarp();   // a warp's rows of P and dS are its own: 8 rows, the chunk's columns
            auto add = [&](float(&acc)[4][NC], const float *w, const float *row) {
                const float4 w4 = *reinterpret_cast<const float4 *>(w);
                const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
                float v[NC];
                if constexpr (NC >= 4) {
#pragma unroll
                    for (int c = 0; c < NC; c += 4) {
                        const float4 v4 = *reinterpret_cast<const float4 *>(row + o_col<NC>(tx, c));
                        v[c] = v4.x;
                        v[c + 1] = v4.y;
                        v[c + 2] = v4.z;
                        v[c + 3] = v4.w;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < NC; ++c) v[c] = row[tx * NC + c];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int c = 0; c < NC; ++c) acc[i][c] = fmaf(wv[i], v[c], acc[i][c]);
            };
            const int ny4 = (ny + 3) / 4 * 4;   // (dS, P and the rows are zero behind ny)
#pragma unroll 4
            for (int y = 0; y < ny4; ++y) {
                add(acc1, Ss + y * SLD + ty * 4, Y1 + y * LD);
                if constexpr (KEYS) add(acc2, Ps + y * SLD + ty * 4, Y2 + y * LD);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= nr) continue;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int col = o_col<NC>(tx, c);
            if constexpr (!KEYS) {
                put(a, a.dq, ((long long)bh * a.Lq + r0 + r) * D + col, acc1[i][c] * a.scale);
            } else if (part >= 0) {   // dV, then dK of the chunk's partial
                float *dst = a.part + ((((long long)bh * a.n_sink_tiles + tile) * a.n_sink_parts + part) * 2 * BM + r) * (long long)D;
                dst[col] = acc2[i][c];
                dst[(long long)BM * D + col] = acc1[i][c] * a.scale;
            } else {
                const long long to = ((long long)bh * a.Lk + r0 + r) * D + col;
                put(a, a.dv, to, acc2[i][c]);
                put(a, a.dk, to, acc1[i][c] * a.scale);
            }
        }
    }
}

// The key side's blocks first: their walks are the longer ones.
template <int D, typename T>
__global__ void __launch_bounds__(WT) window_bwd_simt_kernel(const BwdArgs a, int key_items, int vec) {
    extern __shared__ __align__(16) float wsm[];
    if ((int)blockIdx.x < key_items)
        window_bwd_block<D, T, true>(a, blockIdx.x, vec, wsm);
    else
        window_bwd_block<D, T, false>(a, blockIdx.x - key_items, vec, wsm);
}

template <int D, typename T>
int launch_bwd_t(const BwdArgs &a, int key_items, long long blocks, cudaStream_t s) {
    constexpr size_t smem = window_bwd_smem<D>();
    auto kern = window_bwd_simt_kernel<D, T>;
    static std::atomic<unsigned long long> allowed{0};
    if (!allow_smem(allowed, reinterpret_cast<const void *>(kern), (int)smem)) return BA_ERR_CUDA;
    bool vec = true;
    for (const TensorRef *t : {&a.q, &a.k, &a.v, &a.dout})
        vec = vec && reinterpret_cast<uintptr_t>(t->p) % (4 * sizeof(T)) == 0 && t->sB % 4 == 0 && t->sH % 4 == 0 && t->sT % 4 == 0;
    kern<<<(unsigned)blocks, WT, smem, s>>>(a, key_items, vec);
    return cudaGetLastError() == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

template <int D>
int launch_bwd_d(const BwdArgs &a, int key_items, long long blocks, cudaStream_t s) {
    return a.dtype == BA_F32 ? launch_bwd_t<D, float>(a, key_items, blocks, s)
                             : launch_bwd_t<D, __nv_bfloat16>(a, key_items, blocks, s);
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

int launch_attn_window_bwd(const BwdArgs &a, int num_sms, cudaStream_t s) {
    int rc = launch_window_pre(a, num_sms, s);
    if (rc) return rc;
    const long long key_items = ((a.Lk + (long long)BM - 1) / BM - a.n_sink_tiles + (long long)a.n_sink_tiles * a.n_sink_parts) *
                                a.B * a.Hkv;
    const long long blocks = key_items + (a.Lq + (long long)BM - 1) / BM * a.B * a.H;
    if (blocks > 0x7fffffffLL) return BA_ERR_SHAPE;
    switch (a.d) {
        case 16: rc = launch_bwd_d<16>(a, (int)key_items, blocks, s); break;
        case 32: rc = launch_bwd_d<32>(a, (int)key_items, blocks, s); break;
        case 64: rc = launch_bwd_d<64>(a, (int)key_items, blocks, s); break;
        case 128: rc = launch_bwd_d<128>(a, (int)key_items, blocks, s); break;
        default: rc = BA_ERR_SHAPE;
    }
    return rc ? rc : launch_sink_sum(a, BM, num_sms, s);
}

}  // namespace ba
