// Single-token attention with grouped heads: a window with sinks over a bf16 or fp32
// cache (attn_window_decode_fwd), and the whole cache or a window over a cache held in
// 4 bits (attn_decode_kv4_fwd).
//
// Sequence b holds len = lengths[b] keys and its query is at position len - 1.  The
// keys it sees, [0, s) and [lo, len) with lo = len - window behind the s = sinks first
// ones (all of [0, len) when lo <= sinks), are numbered 0 .. n - 1 without a gap; the
// softmax does not mind the order.
//
// Division of the work: the ranges of all (sequence, key head) pairs, cut into units of
// one step of a CTA, lie one behind the other as one row of units, and every CTA takes
// an equal run of it (one wave of CTAs, whatever the lengths are: they are read on the
// device).  A run covers parts of one or more pairs; a part that is its pair's whole
// range writes the result, any other its (O, m, l), which a second, small launch joins
// by the rule of attn_merge.  Up to 16 query heads share the reading of their key head.
// (Splits of a fixed length, 512 keys, took 113 us where this takes 97: 8 sequences of 32K
// to 64K 4-bit keys, 32 query and 8 key heads, d = 128.)
//
// decode_mma_kernel (bf16 cache with d = 64, 128; 4-bit cache).  What bounds it is HBM:
//   a key costs 4 G d flop for 4 d bytes (bf16) or 1.125 d bytes (4 bits), G <= 16.  On
//   the CUDA cores that would be 2 G d FMAs a key, beyond the fp32 rate from about G = 4
//   at 6.8 TB/s; the products therefore run as mma.sync m16n8k16.  (tcgen05.mma needs its
//   operands in shared memory in its own layout, which for the 4-bit cache would mean
//   writing every unpacked value back to shared memory; here the fragments are unpacked in
//   the registers that loaded them.)  The keys are M of S^T = K q^T, the d's M of O^T =
//   V^T P^T, eight query heads N: no row of a fragment is empty at G = 8, and O takes half
//   the registers that it takes with the heads as M.  P passes from one product to the
//   other by two 8 x 8 transposes a tile.
//   A warp works alone on tiles of 16 keys, which it brings in with cp.async through a
//   ring of its own in shared memory: every lane copies exactly the bytes that it will use
//   and reads them back itself, so the loop has no block barrier.
//   Fragments: the order of d inside the contraction q . k and that of the rows of O^T are
//   free, so a lane (g = lane / 4, t = lane % 4) takes contiguous runs: of the keys g and
//   g + 8 the d's of t for K, and of the keys 2t, 2t+1, 2t+8, 2t+9 the d's of g for V; the
//   pairs of keys that V^T's fragment wants side by side are put together with byte
//   permutes (bf16), or by joining two keys' nibbles before the conversion (4 bits).
//   4 bits: a code times its e4m3 scale has 6 significant bits, so the unpacked values are
//   exact in fp16; q is scaled by a power of two to at most 2 in magnitude before its
//   conversion (bf16 values keep their 8 bits down to 2^-14 of the largest), and p is
//   kept times 2^11 in fp16 (relative 2^-11, absolute 2^-36 of the row's largest).
//   bf16: p is rounded to bf16 for P V, as in the prompt kernels.  l sums unrounded p.
//
// decode_simt_kernel (fp32, and bf16 with d = 16, 32): lanes own 16 bytes of a key row,
//   fp32 arithmetic, up to four query heads at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "internal.h"

namespace ba {
namespace {

constexpr int DG_WARPS = 4;
constexpr float P_BIAS = 11.f;      // 4-bit cache: p is kept times 2^P_BIAS
constexpr float LAZY = 4.f;         // the reference maximum moves when exceeded by 2^LAZY

// The visible keys of one sequence as a gapless range of n indices.
struct KeyRange {
    int n, s;          // indices; the first s are the slots 0 .. s - 1
    long long shift;   // slot of index i >= s: i + shift
    __device__ __forceinline__ long long slot(int i) const { return i < s ? i : i + shift; }
};

__device__ __forceinline__ KeyRange key_range(const DecodeGroupArgs &a, int b) {
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.S) : a.S;
    KeyRange r;
    const int lo = a.window > 0 ? len - a.window : 0;
    if (lo <= a.sinks) {
        r.n = len;
        r.s = 0;
        r.shift = 0;
    } else {
        r.s = a.sinks;
        r.n = a.sinks + len - lo;
        r.shift = lo - a.sinks;
    }
    return r;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool in) {
        // (with the hint to bring 256 bytes into L2: 64 sequences x 4K bf16 keys 208 -> 203 us)
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void *src, bool in) {   // 4 or 8 bytes
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(in ? N : 0), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds4b(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds2b(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds1b(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), 16-bit operands of one type.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight e2m1 codes of a word as four fp16 pairs (the low nibble of a byte in the low half).
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}
// Two e4m3 scales (low byte first) as an fp16 pair.
__device__ __forceinline__ uint32_t scales2(uint32_t two) {
    uint32_t o;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o) : "h"((uint16_t)two));
    return o;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t o;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
    return o;
}
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool f16) {
    uint32_t o;
    if (f16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
    return o;
}
// An 8 x 8 matrix of 16-bit values across the warp (lane (g, t): row g, columns 2t, 2t + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The row of units: UNIT keys each, sequences in order, in each its HS segments (key head,
// group of 16 query heads).  The host bounds their number below 2^31.  Every function is
// run by whole warps.
struct Plan {
    int HS;      // segments per sequence
    int total;   // units in all
    int run;     // units per CTA
};

template <int UNIT>
__device__ __forceinline__ int units_of(const DecodeGroupArgs &a, int b) {
    return (key_range(a, b).n + UNIT - 1) / UNIT;
}

__device__ __forceinline__ int warp_sum(int n) { return __reduce_add_sync(0xffffffffu, n); }

template <int UNIT>
__device__ __forceinline__ Plan make_plan(const DecodeGroupArgs &a) {
    Plan p;
    p.HS = a.Hkv * ((a.G + 15) / 16);
    int n = 0;
    for (int b = threadIdx.x & 31; b < a.B; b += 32) n += units_of<UNIT>(a, b);
    p.total = warp_sum(n) * p.HS;
    p.run = (p.total + a.n_ctas - 1) / a.n_ctas;
    return p;
}

// The sequence of unit u (0 <= u < total) and the first unit of that sequence.
template <int UNIT>
__device__ __forceinline__ void find_unit(const DecodeGroupArgs &a, const Plan &p, int u, int &b, int &base) {
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
        const int v = b0 + lane < a.B ? units_of<UNIT>(a, b0 + lane) : 0;
        int incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, (before + incl) * p.HS > u);
        if (hit || b0 + 32 >= a.B) {
            const int first = hit ? __ffs(hit) - 1 : 31;
            b = b0 + first;
            base = (before + __shfl_sync(0xffffffffu, incl - v, first)) * p.HS;
            return;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// First unit of sequence b.
template <int UNIT>
__device__ __forceinline__ int first_unit(const DecodeGroupArgs &a, const Plan &p, int b) {
    int n = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) n += units_of<UNIT>(a, i);
    return warp_sum(n) * p.HS;
}

// A part of one segment: keys [v0, v1) of sequence b for the query heads q0 .. q0 + nh - 1
// of key head hk.  part: its place among the partial results (CTAs and segments both
// ascend along the row, so CTA + segment is one place each), or -1 for a whole segment.
struct Part {
    int b, hk, q0, nh, v0, v1, part;
};

// Calls body(Part) for each part of this CTA's run.
template <int UNIT, typename F>
__device__ __forceinline__ void for_parts(const DecodeGroupArgs &a, F body) {
    const Plan p = make_plan<UNIT>(a);
    const int cta = blockIdx.x;
    if ((long long)cta * p.run >= p.total) return;
    int u = cta * p.run, left = min(p.run, p.total - u), b, base;
    find_unit<UNIT>(a, p, u, b, base);
    while (left > 0) {
        const KeyRange kr = key_range(a, b);
        const int per = (kr.n + UNIT - 1) / UNIT;   // units of a segment of this sequence
        if (per > 0) {
            const int seg = (u - base) / per, off = (u - base) - seg * per;
            const int take = min(left, per - off);
            Part x;
            x.b = b;
            const int chunks = p.HS / a.Hkv;
            x.hk = seg / chunks;
            const int h0 = (seg - x.hk * chunks) * 16;
            x.q0 = x.hk * a.G + h0;
            x.nh = min(16, a.G - h0);
            x.v0 = off * UNIT;
            x.v1 = min(kr.n, (off + take) * UNIT);
            x.part = off == 0 && take == per ? -1 : cta + b * p.HS + seg;
            body(x);
            u += take;
            left -= take;
            if (seg + 1 < p.HS || off + take < per) continue;
        }
        base += per * p.HS;
        ++b;
    }
}

// What a part found for element d of its query head q0 + row: the reference maximum ref
// (log2 units), the sum L and the weighted sum acc relative to it.
__device__ __forceinline__ void store_part(const DecodeGroupArgs &a, const Part &x, int row, int d, float ref, float L,
                                           float acc) {
    if (x.part >= 0) {
        const long long at = (long long)x.part * a.part_rows + row;
        a.part_o[at * a.d + d] = acc;
        if (d == 0) a.part_ml[at] = make_float2(ref, L);
        return;
    }
    const long long at = (long long)x.b * a.Hkv * a.G + x.q0 + row;
    const float y = L > 0.f ? acc / L * a.out_mul : (L != L ? L : 0.f);
    if (a.out_dtype == BA_BF16)
        static_cast<__nv_bfloat16 *>(a.out)[at * a.d + d] = __float2bfloat16_rn(y);
    else
        static_cast<float *>(a.out)[at * a.d + d] = y;
    if (d == 0) a.lse[at] = L == 0.f ? -INFINITY : (ref + log2f(L)) * LN2;
}

// One stage of a warp's ring: SUB tiles of 16 keys, in the order in which the lanes read
// them.  bf16: K of a tile as [key half][chunk of 32 d's][lane], V as [key 0..3 of the
// lane][chunk of 64 d's][lane], 16 bytes each.  4 bits: K as [key half][lane] (D / 8
// bytes), V as [key 0..3][lane] (D / 16 bytes); then the stage's scales, K's and V's, key by key.
template <int D, bool KV4>
struct Ring {
    static constexpr int SUB = KV4 ? 2 : 1, KEYS = 16 * SUB;
    static constexpr int K_BYTES = KV4 ? 2 * 32 * (D / 8) : 2 * (D / 32) * 512;
    static constexpr int V_BYTES = KV4 ? 4 * 32 * (D / 16) : 4 * (D / 64) * 512;
    static constexpr int TILE16 = K_BYTES + V_BYTES;
    static constexpr int SC_ROW = D / 16, SC_OFF = SUB * TILE16;
    static constexpr int STAGE = SC_OFF + (KV4 ? 2 * KEYS * SC_ROW : 0);
    static constexpr int NS = KV4 && D == 128 ? 2 : 3;   // (4 bits, d = 128: 3 stages 101 us, 2 stages 99 us)
    static constexpr int BYTES = DG_WARPS * NS * STAGE;
    static constexpr int UNIT = DG_WARPS * KEYS;
};

// CTAs of a kernel that an SM holds (registers and shared memory).
constexpr int mma_places(int d, bool kv4, int nh) {
    return kv4 ? (d == 128 ? (nh == 1 ? 4 : 2) : (nh == 1 ? 6 : 4)) : (d == 128 ? 2 : (nh == 1 ? 4 : 4));
}

// NH: groups of 8 query heads (G <= 8 NH).
template <int D, bool KV4, int NH>
__device__ __forceinline__ void mma_part(const DecodeGroupArgs &a, const Part &part) {
    using R = Ring<D, KV4>;
    constexpr int MT = D / 16;   // row tiles of O^T
    constexpr int KS = D / 16;   // steps of the contraction over d
    extern __shared__ __align__(128) uint8_t dg_smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int b = part.b, hk = part.hk, nh = part.nh, v0 = part.v0, v1 = part.v1;
    const KeyRange kr = key_range(a, b);

    const uint32_t ring = smem_u32(dg_smem) + (uint32_t)warp * R::NS * R::STAGE;
    const uint8_t *kb = static_cast<const uint8_t *>(a.k) + (long long)b * a.ksB + (long long)hk * a.ksH;
    const uint8_t *vb = static_cast<const uint8_t *>(a.v) + (long long)b * a.vsB + (long long)hk * a.vsH;
    const uint8_t *ksb = KV4 ? static_cast<const uint8_t *>(a.k_scales) + (long long)b * a.kcB + (long long)hk * a.kcH : nullptr;
    const uint8_t *vsb = KV4 ? static_cast<const uint8_t *>(a.v_scales) + (long long)b * a.vcB + (long long)hk * a.vcH : nullptr;

    // Stage i of this warp: indices v0 + KEYS (warp + DG_WARPS i) ..; keys behind v1 are
    // not read (their bytes arrive as zeros).
    const int stages = v1 > v0 ? (v1 - v0 + R::KEYS - 1) / R::KEYS : 0;
    const int mine = stages > warp ? (stages - warp + DG_WARPS - 1) / DG_WARPS : 0;
    // the lane's part of a key's row: its bytes from row + k_part (v_part) on
    const int k_part = KV4 ? t * (D / 8) : t * 16, v_part = KV4 ? g * (D / 16) : g * 16;
    const long long k_lane = g * a.ksT + k_part, k8 = 8 * a.ksT, v_lane = 2 * t * a.vsT + v_part, v8 = 8 * a.vsT;
    const long long ks_lane = lane * a.kcT, vs_lane = lane * a.vcT;
    auto copy_k = [&](uint32_t dst, const uint8_t *at, bool in) {
        if constexpr (KV4 && D == 128)
            cp16(dst + lane * 16, at, in);
        else if constexpr (KV4)
            cp_small<8>(dst + lane * 8, at, in);
        else
            for (int c = 0; c < D / 32; ++c) cp16(dst + (c * 32 + lane) * 16, at + c * 64, in);
    };
    auto copy_v = [&](uint32_t dst, const uint8_t *at, bool in) {
        if constexpr (KV4)
            cp_small<D / 16>(dst + lane * (D / 16), at, in);
        else
            for (int c = 0; c < D / 64; ++c) cp16(dst + (c * 32 + lane) * 16, at + c * 128, in);
    };
    auto issue = [&](int i) {
        if (i < mine) {
            const uint32_t st = ring + (uint32_t)(i % R::NS) * R::STAGE;
            const int i0 = v0 + R::KEYS * (warp + DG_WARPS * i);
            // Whole stages on one side of the gap between sinks and window: rows at a fixed
            // distance from the first, addressed by additions.  Others (the gap, the end):
            // slot by slot.
            if (i0 + R::KEYS <= v1 && (i0 >= kr.s || i0 + R::KEYS <= kr.s)) {
                const long long slot0 = kr.slot(i0);
                const uint8_t *k0 = kb + slot0 * a.ksT + k_lane, *w0 = vb + slot0 * a.vsT + v_lane;
#pragma unroll
                for (int u = 0; u < R::SUB; ++u) {
                    copy_k(st + u * R::TILE16, k0, true);
                    copy_k(st + u * R::TILE16 + R::K_BYTES / 2, k0 + k8, true);
                    const uint32_t dv = st + u * R::TILE16 + R::K_BYTES;
                    copy_v(dv, w0, true);
                    copy_v(dv + R::V_BYTES / 4, w0 + a.vsT, true);
                    copy_v(dv + R::V_BYTES / 2, w0 + v8, true);
                    copy_v(dv + 3 * (R::V_BYTES / 4), w0 + v8 + a.vsT, true);
                    if (u + 1 < R::SUB) {
                        k0 += 2 * k8;
                        w0 += 2 * v8;
                    }
                }
                if constexpr (KV4) {   // lane = key of the stage
                    cp_small<R::SC_ROW>(st + R::SC_OFF + lane * R::SC_ROW, ksb + slot0 * a.kcT + ks_lane, true);
                    cp_small<R::SC_ROW>(st + R::SC_OFF + (R::KEYS + lane) * R::SC_ROW, vsb + slot0 * a.vcT + vs_lane, true);
                }
            } else {
#pragma unroll 1
                for (int u = 0; u < R::SUB; ++u) {
#pragma unroll 1
                    for (int n = 0; n < 2; ++n) {
                        const int r = i0 + 16 * u + 8 * n + g;
                        copy_k(st + u * R::TILE16 + n * (R::K_BYTES / 2), kb + kr.slot(min(r, v1 - 1)) * a.ksT + k_part, r < v1);
                    }
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        const int r = i0 + 16 * u + 2 * t + (x & 1) + 8 * (x >> 1);
                        copy_v(st + u * R::TILE16 + R::K_BYTES + x * (R::V_BYTES / 4),
                               vb + kr.slot(min(r, v1 - 1)) * a.vsT + v_part, r < v1);
                    }
                }
                if constexpr (KV4) {
                    const bool in = i0 + lane < v1;
                    const long long slot = kr.slot(min(i0 + lane, v1 - 1));
                    cp_small<R::SC_ROW>(st + R::SC_OFF + lane * R::SC_ROW, ksb + slot * a.kcT, in);
                    cp_small<R::SC_ROW>(st + R::SC_OFF + (R::KEYS + lane) * R::SC_ROW, vsb + slot * a.vcT, in);
                }
            }
        }
        cp_commit();   // a group each time, so that the counts below hold
    };
#pragma unroll
    for (int i = 0; i < R::NS - 1; ++i) issue(i);

    // q fragments (B of S^T = K q^T): the d's that lane t contracts, in the order of its K
    // words, of head g of each group.  4 bits: times a power of two that brings the head's
    // largest magnitude into [1, 2).  sl2: of the heads 2t, 2t + 1 of each group.
    uint32_t qb[NH][2 * KS];
    float sl2[NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x) {
        const int head = g + 8 * x;
        const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + (long long)b * a.qsB +
                                  (long long)(part.q0 + min(head, nh - 1)) * a.qsH;
        float mul = a.scale_log2;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(qp + (KV4 ? t * (D / 4) + c * 8 : c * 32 + t * 8)));
            qb[x][4 * c] = u.x;
            qb[x][4 * c + 1] = u.y;
            qb[x][4 * c + 2] = u.z;
            qb[x][4 * c + 3] = u.w;
        }
        if constexpr (KV4) {
            uint32_t big = 0;   // largest magnitude, as bits
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) big = max(big, max(qb[x][i] & 0x7fffu, (qb[x][i] >> 16) & 0x7fffu));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const int e = min(max((int)(big >> 7), 1), 253);   // biased exponent
            const float down = __uint_as_float((uint32_t)(254 - e) << 23);
            mul *= __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i)
                qb[x][i] = pack16(__uint_as_float(qb[x][i] << 16) * down, __uint_as_float(qb[x][i] & 0xffff0000u) * down, true);
        }
        if (head >= nh) {
#pragma unroll
            for (int i = 0; i < 2 * KS; ++i) qb[x][i] = 0u;
        }
        sl2[x][0] = __shfl_sync(0xffffffffu, mul, 8 * t);
        sl2[x][1] = __shfl_sync(0xffffffffu, mul, 8 * t + 4);
    }

    float o[NH][MT][4], m[NH][2], l[NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x) {
        m[x][0] = m[x][1] = -INFINITY;
        l[x][0] = l[x][1] = 0.f;
#pragma unroll
        for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][n][e] = 0.f;
    }

    for (int i = 0; i < mine; ++i) {
        issue(i + R::NS - 1);     // into the stage of step i - 1, which every lane has read (__syncwarp below)
        cp_wait<R::NS - 1>();     // stage i has arrived
        __syncwarp();             // for every lane: the scales are shared
        const uint32_t st = ring + (uint32_t)(i % R::NS) * R::STAGE;
        const int i0 = v0 + R::KEYS * (warp + DG_WARPS * i);
        float s[R::SUB][NH][4];   // [key g, heads 2t, 2t + 1; key g + 8, the same]
#pragma unroll
        for (int u = 0; u < R::SUB; ++u) {
            uint32_t kw[2][2 * KS];   // A fragments: the lane's words of the keys g and g + 8
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint32_t at = st + u * R::TILE16 + n * (R::K_BYTES / 2);
                if constexpr (KV4) {
                    uint32_t code[D / 32], sc[2];   // sc: the scale of each 16 codes of the lane, twice in a word
                    const uint32_t sc_at = st + R::SC_OFF + (16 * u + 8 * n + g) * R::SC_ROW;
                    if constexpr (D == 128) {
                        const uint4 w = lds16(at + lane * 16);
                        code[0] = w.x;
                        code[1] = w.y;
                        code[2] = w.z;
                        code[3] = w.w;
                        const uint32_t p = scales2(lds2b(sc_at + 2 * t));
                        sc[0] = __byte_perm(p, p, 0x1010);
                        sc[1] = __byte_perm(p, p, 0x3232);
                    } else {
                        const uint2 w = lds8(at + lane * 8);
                        code[0] = w.x;
                        code[1] = w.y;
                        const uint32_t p = scales2(lds1b(sc_at + t));
                        sc[0] = sc[1] = __byte_perm(p, p, 0x1010);
                    }
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t f[4];
                        unpack8(code[c], f);
#pragma unroll
                        for (int e = 0; e < 4; ++e) kw[n][4 * c + e] = hmul2(f[e], sc[c >> 1]);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        const uint4 w = lds16(at + (c * 32 + lane) * 16);
                        kw[n][4 * c] = w.x;
                        kw[n][4 * c + 1] = w.y;
                        kw[n][4 * c + 2] = w.z;
                        kw[n][4 * c + 3] = w.w;
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < NH; ++x) {
                s[u][x][0] = s[u][x][1] = s[u][x][2] = s[u][x][3] = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    mma16816<KV4>(s[u][x], kw[0][2 * k], kw[1][2 * k], kw[0][2 * k + 1], kw[1][2 * k + 1], qb[x][2 * k],
                                  qb[x][2 * k + 1]);
            }
        }
        // Scores in log2 units; indices behind the range take no part.  The reference
        // maximum of a head moves, and O and l with it, only when one of its scores
        // passes it by more than 2^LAZY: until then p stays below 2^LAZY and no lane has
        // to know another's scores.
        const bool inside = i0 + R::KEYS <= v1;
        bool move = false;
        float mx[NH][2];
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mx[x][e] = -INFINITY;
#pragma unroll
                for (int u = 0; u < R::SUB; ++u)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float &y = s[u][x][2 * n + e];
                        y *= sl2[x][e];
                        if (!inside && i0 + 16 * u + 8 * n + g >= v1) y = -INFINITY;
                        mx[x][e] = fmaxf(mx[x][e], y);
                    }
                move = move || mx[x][e] > m[x][e] + LAZY;
            }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int x = 0; x < NH; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = mx[x][e];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                    const float m_new = fmaxf(m[x][e], v);
                    const float alpha = m_new == -INFINITY ? 1.f : ex2(m[x][e] - m_new);
                    m[x][e] = m_new;
                    l[x][e] *= alpha;
#pragma unroll
                    for (int n = 0; n < MT; ++n) {
                        o[x][n][e] *= alpha;
                        o[x][n][2 + e] *= alpha;
                    }
                }
        }
#pragma unroll
        for (int u = 0; u < R::SUB; ++u) {
            uint32_t pb[NH][2];   // B fragments of O^T += V^T P^T: keys 2t, 2t + 1 (+ 8) of head g
#pragma unroll
            for (int x = 0; x < NH; ++x) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float base = (m[x][e] == -INFINITY ? 0.f : m[x][e]) - (KV4 ? P_BIAS : 0.f);
                    p[e] = ex2(s[u][x][e] - base);
                    p[2 + e] = ex2(s[u][x][2 + e] - base);
                    l[x][e] += p[e] + p[2 + e];
                }
                pb[x][0] = transpose8(pack16(p[0], p[1], KV4));
                pb[x][1] = transpose8(pack16(p[2], p[3], KV4));
            }
            const uint32_t at = st + u * R::TILE16 + R::K_BYTES;
            if constexpr (KV4) {
                constexpr int VW = D / 64;   // words of codes per key and lane
                uint32_t vw[4][VW], vs[2];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (VW == 2) {
                        const uint2 w = lds8(at + (x * 32 + lane) * 8);
                        vw[x][0] = w.x;
                        vw[x][1] = w.y;
                    } else {
                        vw[x][0] = lds4b(at + (x * 32 + lane) * 4);
                    }
                }
                const uint32_t sc_at = st + R::SC_OFF + (R::KEYS + 16 * u) * R::SC_ROW + (D == 128 ? g : g >> 1);
#pragma unroll
                for (int n = 0; n < 2; ++n)   // scales of the keys 2t + 8n, 2t + 1 + 8n
                    vs[n] = scales2(lds1b(sc_at + (2 * t + 8 * n) * R::SC_ROW) |
                                    lds1b(sc_at + (2 * t + 1 + 8 * n) * R::SC_ROW) << 8);
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    uint32_t even[2][4], odd[2][4];   // [key half]: (key 2t, key 2t + 1) of the word's even and odd d's
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const uint32_t p = vw[2 * n][w], q = vw[2 * n + 1][w];
                        unpack8((p & 0x0f0f0f0fu) | ((q << 4) & 0xf0f0f0f0u), even[n]);
                        unpack8(((p >> 4) & 0x0f0f0f0fu) | (q & 0xf0f0f0f0u), odd[n]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a0 = hmul2(even[0][e], vs[0]), a1 = hmul2(odd[0][e], vs[0]);
                        const uint32_t a2 = hmul2(even[1][e], vs[1]), a3 = hmul2(odd[1][e], vs[1]);
#pragma unroll
                        for (int x = 0; x < NH; ++x) mma16816<true>(o[x][4 * w + e], a0, a1, a2, a3, pb[x][0], pb[x][1]);
                    }
                }
            } else {
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t vw[4][4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 w = lds16(at + ((x * (D / 64) + c) * 32 + lane) * 16);
                        vw[x][0] = w.x;
                        vw[x][1] = w.y;
                        vw[x][2] = w.z;
                        vw[x][3] = w.w;
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a0 = __byte_perm(vw[0][e], vw[1][e], 0x5410), a1 = __byte_perm(vw[0][e], vw[1][e], 0x7632);
                        const uint32_t a2 = __byte_perm(vw[2][e], vw[3][e], 0x5410), a3 = __byte_perm(vw[2][e], vw[3][e], 0x7632);
#pragma unroll
                        for (int x = 0; x < NH; ++x) mma16816<false>(o[x][4 * c + e], a0, a1, a2, a3, pb[x][0], pb[x][1]);
                    }
                }
            }
        }
        __syncwarp();   // the stage may be refilled
    }
    cp_wait<0>();
    __syncthreads();   // every warp is done with its ring: the merge area overlays it

    // Join the warps: each head's (m, l) and O of each warp, then one weighted sum.
    float *mo = reinterpret_cast<float *>(dg_smem);                     // [warp][8 NH][D]
    float *mm = mo + DG_WARPS * 8 * NH * D, *ml = mm + DG_WARPS * 16;   // [warp][16]
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = 8 * x + 2 * t + e;
            float sum = l[x][e];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (g == 0) {
                mm[warp * 16 + row] = m[x][e];
                ml[warp * 16 + row] = sum;
            }
            float *dst = mo + (warp * 8 * NH + row) * D;
#pragma unroll
            for (int n = 0; n < MT; ++n) {   // rows g and g + 8 of tile n: an even d of lane group g and the next one
                const int d = KV4 ? g * (D / 8) + 2 * n : (n >> 2) * 64 + g * 8 + 2 * (n & 3);
                *reinterpret_cast<float2 *>(dst + d) = make_float2(o[x][n][e], o[x][n][2 + e]);
            }
        }
    __syncthreads();
    for (int y = threadIdx.x; y < nh * D; y += DG_WARPS * 32) {
        const int row = y / D, d = y % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < DG_WARPS; ++w) M = fmaxf(M, mm[w * 16 + row]);
        float L = 0.f, acc = 0.f;
        if (M != -INFINITY) {
#pragma unroll
            for (int w = 0; w < DG_WARPS; ++w) {
                const float wt = ex2(mm[w * 16 + row] - M);
                L += wt * ml[w * 16 + row];
                acc += wt * mo[(w * 8 * NH + row) * D + d];
            }
        }
        store_part(a, part, row, d, M - (KV4 ? P_BIAS : 0.f), L, acc);
    }
    __syncthreads();   // the merge area becomes the next part's ring
}

template <int D, bool KV4, int NH>
__global__ void __launch_bounds__(DG_WARPS * 32, mma_places(D, KV4, NH)) decode_mma_kernel(const DecodeGroupArgs a) {
    for_parts<Ring<D, KV4>::UNIT>(a, [&](const Part &x) { mma_part<D, KV4, NH>(a, x); });
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may be placed now
}

// fp32 arithmetic: a group of LPK lanes owns a key, each lane 16 bytes of its row; HC query
// heads share the loads.  The groups of the CTA are joined in
// shared memory.
template <typename T>
struct Row16;   // 16 bytes of T, unpacked to fp32
template <>
struct Row16<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void load(const void *p, float (&x)[8]) {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Row16<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void load(const void *p, float (&x)[4]) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(p));
        x[0] = u.x;
        x[1] = u.y;
        x[2] = u.z;
        x[3] = u.w;
    }
};

constexpr int SIMT_UNIT = 64;
constexpr int SIMT_PLACES = 4;

template <typename T, int D, int HC>
__device__ __forceinline__ void simt_part(const DecodeGroupArgs &a, const Part &part) {
    constexpr int EPL = Row16<T>::N, LPK = D / EPL, GROUPS = 128 / LPK, GPW = 32 / LPK, UN = 4;
    __shared__ float sm_o[GROUPS][HC][D];
    __shared__ float sm_m[GROUPS][HC], sm_l[GROUPS][HC];
    const int b = part.b, hk = part.hk, v0 = part.v0, v1 = part.v1;
    const KeyRange kr = key_range(a, b);
    const int grp = threadIdx.x / LPK, gl = threadIdx.x % LPK;
    const int warp = threadIdx.x / 32, gw = (threadIdx.x % 32) / LPK;

    for (int h0 = 0; h0 < part.nh; h0 += HC) {   // HC query heads at a time (the next ones' keys come from L1 / L2)
        const int nh = min(HC, part.nh - h0);
        float q[HC][EPL], o[HC][EPL], m[HC], l[HC];
#pragma unroll
        for (int h = 0; h < HC; ++h) {
            const T *qp = static_cast<const T *>(a.q) + (long long)b * a.qsB +
                          (long long)(part.q0 + h0 + min(h, nh - 1)) * a.qsH;
            Row16<T>::load(qp + gl * EPL, q[h]);
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int e = 0; e < EPL; ++e) o[h][e] = 0.f;
        }
        const uint8_t *kb = static_cast<const uint8_t *>(a.k) + (long long)b * a.ksB + (long long)hk * a.ksH + gl * 16;
        const uint8_t *vb = static_cast<const uint8_t *>(a.v) + (long long)b * a.vsB + (long long)hk * a.vsH + gl * 16;

        // The loop runs on a warp-uniform base (the shuffles span the warp); keys behind the
        // range are masked and their loads clamped into it.
        for (int jb = v0 + warp * GPW * UN; jb < v1; jb += 4 * GPW * UN) {
            const int j0 = jb + gw * UN;
            float kx[UN][EPL], vx[UN][EPL];
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const long long slot = kr.slot(min(j0 + u, v1 - 1));
                Row16<T>::load(kb + slot * a.ksT, kx[u]);
                Row16<T>::load(vb + slot * a.vsT, vx[u]);
                if (j0 + u >= v1) {   // a repeated key: no part of it may enter the sums
#pragma unroll
                    for (int e = 0; e < EPL; ++e) vx[u][e] = 0.f;
                }
            }
#pragma unroll
            for (int h = 0; h < HC; ++h) {
                float s[UN], mx = -INFINITY;
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    float acc = 0.f;
#pragma unroll
                    for (int e = 0; e < EPL; ++e) acc = fmaf(q[h][e], kx[u][e], acc);
#pragma unroll
                    for (int off = LPK / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off, LPK);
                    s[u] = j0 + u < v1 ? acc * a.scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[u]);
                }
                const float m_new = fmaxf(m[h], mx);
                const float alpha = m[h] == -INFINITY ? 0.f : exp2f(m[h] - m_new);
                l[h] *= alpha;
#pragma unroll
                for (int e = 0; e < EPL; ++e) o[h][e] *= alpha;
#pragma unroll
                for (int u = 0; u < UN; ++u) {
                    const float p = s[u] == -INFINITY ? 0.f : exp2f(s[u] - m_new);
                    l[h] += p;
#pragma unroll
                    for (int e = 0; e < EPL; ++e) o[h][e] = fmaf(p, vx[u][e], o[h][e]);
                }
                m[h] = m_new;
            }
        }
#pragma unroll
        for (int h = 0; h < HC; ++h) {
#pragma unroll
            for (int e = 0; e < EPL; ++e) sm_o[grp][h][gl * EPL + e] = o[h][e];
            if (gl == 0) {
                sm_m[grp][h] = m[h];
                sm_l[grp][h] = l[h];
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < nh * D; x += 128) {
            const int h = x / D, d = x % D;
            float M = -INFINITY, L = 0.f, acc = 0.f;
            for (int g = 0; g < GROUPS; ++g) M = fmaxf(M, sm_m[g][h]);
            if (M != -INFINITY) {
                for (int g = 0; g < GROUPS; ++g) {
                    const float w = exp2f(sm_m[g][h] - M);
                    L += w * sm_l[g][h];
                    acc += w * sm_o[g][h][d];
                }
            }
            store_part(a, part, h0 + h, d, M, L, acc);
        }
        __syncthreads();
    }
}

template <typename T, int D, int HC>
__global__ void __launch_bounds__(128) decode_simt_kernel(const DecodeGroupArgs a) {
    for_parts<SIMT_UNIT>(a, [&](const Part &x) { simt_part<T, D, HC>(a, x); });
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The join of a row's parts: O = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s.  One block per
// (b, query head); it is launched while the parts are still computed (programmatic
// launch) and waits for them, so that its start is hidden.  Rows of one part are done;
// rows without keys are written here.
template <int UNIT>
__global__ void __launch_bounds__(128) decode_join_kernel(const DecodeGroupArgs a) {
    __shared__ float wt[128], red[4];
    const int Hq = a.Hkv * a.G, b = blockIdx.x / Hq, h = blockIdx.x % Hq, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long row = blockIdx.x;
    const Plan p = make_plan<UNIT>(a);
    const int per = units_of<UNIT>(a, b), hk = h / a.G, seg = hk * (p.HS / a.Hkv) + (h % a.G) / 16;
    const int s0 = first_unit<UNIT>(a, p, b) + seg * per;
    int c0 = 0, used = 0;
    if (per > 0) {
        c0 = s0 / p.run;
        used = (s0 + per - 1) / p.run - c0 + 1;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // also where nothing is left to do: what follows
    if (used == 1) return;                               // this launch must follow the parts' as well
    float M = -INFINITY, L = 0.f, acc = 0.f;
    const long long first = ((long long)c0 + b * p.HS + seg) * a.part_rows + (h % a.G) % 16;
    const float2 *ml = a.part_ml + first;
    const float *po = a.part_o + first * a.d;
    for (int i0 = 0; i0 < used; i0 += 128) {   // in rounds of 128 parts, carrying (M, L, acc)
        const int here = min(128, used - i0);
        const float2 x =
            threadIdx.x < here ? __ldcg(ml + (long long)(i0 + threadIdx.x) * a.part_rows) : make_float2(-INFINITY, 0.f);
        float v = x.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
        __syncthreads();
        if (lane == 0) red[warp] = v;
        __syncthreads();
        const float M_new = fmaxf(fmaxf(M, fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
        const float carry = M == -INFINITY ? 0.f : exp2f(M - M_new);
        const float w = x.x == -INFINITY ? 0.f : exp2f(x.x - M_new);
        float lw = w * x.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, off);
        __syncthreads();
        wt[threadIdx.x] = w;
        if (lane == 0) red[warp] = lw;
        __syncthreads();
        L = L * carry + ((red[0] + red[1]) + (red[2] + red[3]));
        if (threadIdx.x < a.d) {
            acc *= carry;
#pragma unroll 8
            for (int i = 0; i < here; ++i)
                acc = fmaf(wt[i], __ldcg(po + (long long)(i0 + i) * a.part_rows * a.d + threadIdx.x), acc);
        }
        M = M_new;
    }
    if (threadIdx.x < a.d) {
        const float y = L > 0.f ? acc / L * a.out_mul : (L != L ? L : 0.f);
        if (a.out_dtype == BA_BF16)
            static_cast<__nv_bfloat16 *>(a.out)[row * a.d + threadIdx.x] = __float2bfloat16_rn(y);
        else
            static_cast<float *>(a.out)[row * a.d + threadIdx.x] = y;
        if (threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * LN2;
    }
}

template <int UNIT>
int launch_join(const DecodeGroupArgs &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.Hkv * a.G));
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_join_kernel<UNIT>, a) == cudaSuccess ? BA_OK : BA_ERR_CUDA;
}

template <int D, bool KV4, int NH>
int launch_mma(const DecodeGroupArgs &a, cudaStream_t s) {
    auto kern = decode_mma_kernel<D, KV4, NH>;
    using R = Ring<D, KV4>;
    constexpr int merge = DG_WARPS * (8 * NH * D + 32) * 4;
    constexpr int smem = R::BYTES > merge ? R::BYTES : merge;
    static_assert(mma_places(D, KV4, NH) * (smem + 1024) <= 233472, "shared memory of an SM");
    static std::atomic<unsigned long long> allowed{0};
    if (!allow_smem(allowed, reinterpret_cast<const void *>(kern), smem)) return BA_ERR_CUDA;
    kern<<<a.n_ctas, DG_WARPS * 32, smem, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return BA_ERR_CUDA;
    return launch_join<R::UNIT>(a, s);
}

template <typename T, int D>
int launch_simt(const DecodeGroupArgs &a, cudaStream_t s) {
    if (a.G >= 3)
        decode_simt_kernel<T, D, 4><<<a.n_ctas, 128, 0, s>>>(a);
    else if (a.G == 2)
        decode_simt_kernel<T, D, 2><<<a.n_ctas, 128, 0, s>>>(a);
    else
        decode_simt_kernel<T, D, 1><<<a.n_ctas, 128, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return BA_ERR_CUDA;
    return launch_join<SIMT_UNIT>(a, s);
}

template <typename T>
int launch_simt_t(const DecodeGroupArgs &a, cudaStream_t s) {
    switch (a.d) {
        case 16: return launch_simt<T, 16>(a, s);
        case 32: return launch_simt<T, 32>(a, s);
        case 64: return launch_simt<T, 64>(a, s);
        case 128: return launch_simt<T, 128>(a, s);
        default: return BA_ERR_SHAPE;
    }
}

// The tensor-core kernel's case (else the CUDA-core one).
bool on_mma(int dtype, int d, bool kv4) { return kv4 || (dtype == BA_BF16 && (d == 64 || d == 128)); }

}  // namespace

// CTAs of a launch over B sequences of up to n_max keys.  4 bits: one wave, so that a CTA's
// start and its joins are paid once (8 sequences of 32K to 64K keys: 97 us; four waves of
// shorter runs 111 us).  16 or 32 bits: up to eight waves of runs of at least 16 units,
// because there the SMs' unequal shares of the bandwidth cost more than the starts (64
// sequences of 4K keys: 198 us; one wave 203 us).  At least a CTA for each SM, when there
// are units for them: a single sequence is bound by the time of one run.
int decode_group_ctas(int B, int Hkv, int G, long long n_max, int dtype, int d, bool kv4, int num_sms) {
    const bool mma = on_mma(dtype, d, kv4);
    const int unit = mma ? (kv4 ? Ring<128, true>::UNIT : Ring<128, false>::UNIT) : SIMT_UNIT;
    const long long units = (long long)B * Hkv * ((G + 15) / 16) * ((n_max + unit - 1) / unit);
    if (units > 0x7fffffffLL - 0x10000) return -1;
    const long long most = (long long)(kv4 ? 1 : 8) * num_sms * (mma ? mma_places(d, kv4, G > 8 ? 2 : 1) : SIMT_PLACES);
    long long n = units / (kv4 ? 4 : 16);
    if (n > most) n = most;
    if (n < num_sms) n = units < num_sms ? units : num_sms;
    return (int)(n < 1 ? 1 : n);
}

int launch_decode_group(const DecodeGroupArgs &a, cudaStream_t s) {
    const bool kv4 = a.k_scales != nullptr;
    if (!on_mma(a.dtype, a.d, kv4))
        return a.dtype == BA_BF16 ? launch_simt_t<__nv_bfloat16>(a, s) : launch_simt_t<float>(a, s);
    const bool two = a.G > 8;
    if (kv4)
        return a.d == 128 ? (two ? launch_mma<128, true, 2>(a, s) : launch_mma<128, true, 1>(a, s))
                          : (two ? launch_mma<64, true, 2>(a, s) : launch_mma<64, true, 1>(a, s));
    return a.d == 128 ? (two ? launch_mma<128, false, 2>(a, s) : launch_mma<128, false, 1>(a, s))
                      : (two ? launch_mma<64, false, 2>(a, s) : launch_mma<64, false, 1>(a, s));
}

}  // namespace ba
