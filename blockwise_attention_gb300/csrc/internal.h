// Host-side interface between the C-ABI entry points (api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

namespace ba {

// The dynamic shared memory that a kernel may use, set once for each device (`done`: a
// bit for each, kept by the caller beside the kernel; a second setting by another thread
// does no harm).
inline bool allow_smem(std::atomic<unsigned long long> &done, const void *kernel, int bytes) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
}

// Arguments of one attention launch (block or ring geometry).
struct AttnArgs {
    Geom g;
    const void *q, *k, *v;               // base pointers, dtype `dtype`
    long long qsB, qsH, qsT;             // element strides (d contiguous)
    long long ksB, ksH, ksT;
    long long vsB, vsH, vsT;
    int dtype;                           // BA_F32 / BA_BF16
    float scale_log2;                    // softmax scale * log2(e)
    void *out;                           // (B, H, rows, d) contiguous, out_dtype
    int out_dtype;
    int tma_out;                         // tensor-core kernel: full tiles stored by TMA (map `o`)
    float *lse;                          // (B, H, rows) natural-log LSE
    long long rows;                      // rows of out/lse per (b, h): Lq or T
    const float *acc_o;                  // nullable fp32 (B, H, rows, d) partial to merge with
    const float *acc_lse;                // nullable fp32 (B, H, rows)
    unsigned *err;                       // device error word
    unsigned *sched;                     // nullable zeroed item counter (dynamic scheduling); null = round-robin
    unsigned long long wait_limit_ns;    // bounded-wait limit
};

// A (B, H, rows, d) tensor with element strides, d contiguous.
struct TensorRef {
    const void *p;
    long long sB, sH, sT;
};

// Arguments of the attention backward (block or ring geometry).  Rows of
// q/out/dout and of k/v are positions - off in block mode and token positions
// in ring mode (global token order).
struct BwdArgs {
    int B, H, d, dtype;
    int ring;                            // 0: one block (Lq x Lk at q_off / k_off)
    int Lq, Lk;
    long long q_off, k_off;
    int T, P, zigzag, CL, NC, s_begin, s_end;   // ring geometry and the steps to cover
    int causal;
    const uint8_t *kpm;
    long long kpm_ld;
    const uint8_t *am;
    long long am_ld;
    TensorRef q, k, v, out, dout;
    const float *lse;                    // (B, H, Lq) natural-log LSE of the whole row
    float *D;                            // (B, H, Lq) dout . out, written by the pre-pass
    float scale;
    float *dq, *dk, *dv;                 // fp32 (B, H, L, d) contiguous
    int accumulate;                      // add into dq / dk / dv instead of overwriting
    unsigned *err;                       // device error word (tensor-core kernels)
    unsigned long long wait_limit_ns;    // bounded-wait limit (tensor-core kernels)
    unsigned *sched;                     // 2 zeroed item counters (dK/dV kernel, dQ kernel), tensor-core kernels
    int heads_per_group;                 // (b, h) pairs whose items run side by side (L2 reuse)
    // Sliding window with sinks (window > 0: block geometry with k_off = 0, causal).
    int window, sinks;                   // visible keys (p - window, p] and [0, sinks)
    int Hkv, kv_group;                   // key heads; query heads per key head
    int grad_bf16;                       // gradients stored as bf16 (else fp32)
    int n_sink_tiles;                    // key tiles that hold sinks: their queries are split into
    int n_sink_parts, sink_rows;         //   n_sink_parts chunks of sink_rows query rows, one partial each
    float *part;                         // (B, Hkv, n_sink_tiles, n_sink_parts, dV / dK, tile rows, d) partials
};

// TMA descriptors of q, k, v and dout for the tensor-core backward.
struct BwdMaps {
    CUtensorMap q, k, v, dout;
};

int launch_attn_bwd(const BwdArgs &a, int num_sms, cudaStream_t s);
int launch_bwd_pre(const BwdArgs &a, int num_sms, cudaStream_t s);
constexpr int WINDOW_SIMT_ROWS = 32;   // rows of a block of the CUDA-core windowed backward
int launch_attn_window_bwd(const BwdArgs &a, int num_sms, cudaStream_t s);
int launch_attn_window_bwd_tc(const BwdArgs &a, const BwdMaps &m, int num_sms, cudaStream_t s);
int launch_window_pre(const BwdArgs &a, int num_sms, cudaStream_t s);
int launch_sink_sum(const BwdArgs &a, int tile_rows, int num_sms, cudaStream_t s);
bool bwd_tc_supported(int dtype, int d);
int launch_attn_bwd_tc(const BwdArgs &a, const BwdMaps &m, int num_sms, cudaStream_t s);

// One Ulysses exchange: the token-split stacked array (P, H, B, Tl, d),
// contiguous, against a strided (B, H, T = P Tl, d) view of the head side.
struct UlyssesArgs {
    void *tok;                // token-split array
    void *head;               // head-side view base
    long long sB, sH, sT;     // head-side element strides (d contiguous)
    int P, H, B, Tl;
    long long row_bytes;      // d * elem_bytes
    int elem_bytes;
    int to_head;              // 1: token-split -> head side, 0: head side -> token-split
};

int launch_ulysses_a2a(const UlyssesArgs &a, int num_sms, cudaStream_t s);

// Decode attention of one query per (b, h) against a KV cache, in key splits.
struct DecodeArgs {
    int B, H, S, d, dtype;
    const void *q, *k, *v;               // q: (B, H, 1, d); k, v: (B, H, S, d), element strides
    long long qsB, qsH;
    long long ksB, ksH, ksT, vsB, vsH, vsT;
    const int32_t *lengths;              // (B) valid cache lengths, or nullptr = S
    float scale;
    int split_len, n_splits;
    float *part_o, *part_lse;            // (B*H, n_splits, d), (B*H, n_splits) fp32 partials
    void *out;                           // (B, H, 1, d) contiguous, out_dtype
    int out_dtype;
    float *lse;                          // (B, H, 1)
};

int launch_decode(const DecodeArgs &a, cudaStream_t s);

// Decode attention of grouped heads over a window with sinks or a 4-bit cache, in key splits.
struct DecodeGroupArgs {
    int B, Hkv, G, S, d, dtype;          // Hkv G query heads; dtype of q (and of a cache that is not 4-bit)
    const void *q, *k, *v;               // q: (B, Hkv G, 1, d), element strides; k, v: rows of the cache, BYTE strides
    long long qsB, qsH;
    long long ksB, ksH, ksT, vsB, vsH, vsT;
    const void *k_scales, *v_scales;     // 4-bit cache: e4m3 scales, byte strides (null: k, v hold dtype)
    long long kcB, kcH, kcT, vcB, vcH, vcT;
    const int32_t *lengths;              // (B) valid cache lengths, or nullptr = S
    int window, sinks;                   // window 0: every key
    float scale_log2;                    // softmax scale * log2(e) (times the 4-bit keys' power of two)
    float out_mul;                       // factor of the outputs (the 4-bit values' power of two)
    int n_ctas;                          // CTAs that share the work
    int part_rows;                       // query heads of a part: min(G, 16)
    float *part_o;                       // (n_ctas + segments, part_rows, d) weighted sums
    float2 *part_ml;                     // (n_ctas + segments, part_rows) reference maximum (log2 units) and sum
    void *out;                           // (B, Hq, 1, d) contiguous, out_dtype
    int out_dtype;
    float *lse;                          // (B, Hq, 1)
};

int decode_group_ctas(int B, int Hkv, int G, long long n_max, int dtype, int d, bool kv4, int num_sms);
int launch_decode_group(const DecodeGroupArgs &a, cudaStream_t s);

// Writing and reading a cache held in 4 bits.
struct Kv4Args {
    int B, H, T, S, d, dtype;            // T new rows per (b, h); dtype of x (append) or y (read)
    const void *x[2];                    // K and V rows (append), element strides
    long long xsB[2], xsH[2], xsT[2];
    void *y[2];                          // contiguous (B, H, T, d) outputs (read)
    void *codes[2], *scales[2];          // cache: byte strides
    long long csB[2], csH[2], csT[2], ssB[2], ssH[2], ssT[2];
    const int32_t *start;                // (B) first slot, or nullptr = first
    const int32_t *counts;               // (B) rows to write, or nullptr = T
    int first;
    int exp[2];                          // a stored value is code * scale * 2^exp
};

int launch_kv4_append(const Kv4Args &a, cudaStream_t s);
int launch_kv4_read(const Kv4Args &a, cudaStream_t s);

// Norm per head and rotation of queries ([0]) and keys ([1]), forward or backward.
struct QkNormArgs {
    int B, T, d, dtype, H[2];
    const void *x[2], *w[2];
    long long sB[2], sH[2], sT[2];       // element strides of x
    const void *g[2];                    // dy (backward)
    long long gB[2], gH[2], gT[2];
    int w_f32;                           // weights fp32 (else dtype)
    void *y[2];                          // y, or dx: contiguous (B, H, T, d)
    const int32_t *positions;            // nullptr: t
    long long pos_ld;                    // entries between sequences (0: shared)
    unsigned long long turn[64];         // pos_scale base^(-2c/d) / (2 pi), its fraction times 2^64
    float eps;
    long long places;                    // T, or B T when each sequence has its own positions
    int nb;                              // sequences of a place: B, or 1
    int run;                             // rows of blocks of places per CTA
    float *part;                         // backward: (blocks, 2, d) sums of dz n
};

void qk_norm_grid(long long places, int rows, int d, int dtype, int num_sms, int &ctas, int &run);
int launch_qk_norm(QkNormArgs a, bool bwd, int g_dtype, bool vec, int num_sms, float *dwq, float *dwk,
                   cudaStream_t s);

// TMA descriptors of Q, K, V (loads) and out (stores, boxes of 32 rows) for
// the tensor-core kernel.
struct TmaMaps {
    CUtensorMap q, k, v, o;
};

int launch_attn_simt(const AttnArgs &a, cudaStream_t s);
int launch_window_simt(const AttnArgs &a, cudaStream_t s);
int launch_attn_tc(const AttnArgs &a, const TmaMaps &maps, int num_sms, cudaStream_t s);
bool tc_supported(int dtype, int d);
size_t tc_smem_bytes(int d);

}  // namespace ba
