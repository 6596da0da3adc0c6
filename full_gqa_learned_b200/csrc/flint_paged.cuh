// Definitions shared by the kernels of the paged key/value cache
// (flint_paged.cu: append, read back, the plan of an attention call and the
// host side; flint_paged_step.cu: attention of few new tokens per sequence).
//
// Position p of sequence b lives in page table[b][p / ps], slot p mod ps, of
// pools laid out [num_pages, ng, ps, 128] (ng KV heads, ps slots a page), so
// the slots of one (page, head) are consecutive rows.  16-bit pages hold the
// normalised, rotated keys in FP16 and the values in BF16.  8-bit pages hold
// E4M3 codes with one scale 2^e per token and head (E8M0: the byte e + 127).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "../../include/flint_attn.h"
#include "flint_common.cuh"

namespace flint {

// Exponent range of the 8-bit pages' scales.  Below 2^-24 nothing is left of
// a normalised key or of a value that a BF16 model works with; the upper end
// keeps 448 x 2^e finite in the FP32 arithmetic of the readers (larger values
// saturate).
constexpr int kPagedEMin = -24;
constexpr int kPagedEMax = 40;

struct PagedCache {
    const int* table;            // [B, max_pages]
    const int* len;              // [B] positions cached before this call
    const int* cu;               // [B + 1] packed rows of the sequences
    int B, T, max_pages, num_pages;
    int ps_log2;                 // log2 of the slots per page
    int ng;
};

// Row of the pools that holds (page, head g, slot).
__device__ __forceinline__ size_t paged_row(const PagedCache& c, int page, int g, int slot) {
    return (((size_t)page * c.ng + g) << c.ps_log2) + slot;
}

// Last b in [0, n) with a[b] <= x, for a non-decreasing a with a[0] <= x;
// warp-wide (x uniform): 32 probes a step.  Any other a gives some index in
// [0, n), so callers check what they read there.
template <typename I, typename X>
__device__ __forceinline__ int warp_last_leq(const I* a, int n, X x) {
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lane * step;
        const bool le = at < n && (X)a[lo + at] <= x;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Rotation of pair f at position pos as rope_cos_sin gives it, to FP32's last
// places: the angle is reduced in double and what its rounding to float
// leaves out is put back by a first-order term.  Used where the result is
// rounded once into the cache.
__device__ __forceinline__ void rope_cos_sin_exact(int pos, double inv_freq, float* c, float* s) {
    const double two_pi_hi = 6.283185307179586, two_pi_lo = 2.4492935982947064e-16;
    const double a = (double)pos * inv_freq;
    const double k = rint(a * 0.15915494309189535);
    double r = fma(-k, two_pi_hi, a);
    r = fma(-k, two_pi_lo, r);
    const float rf = (float)r;
    const float d = (float)(r - (double)rf);
    float s0, c0;
    sincosf(rf, &s0, &c0);
    *c = fmaf(-s0, d, c0);
    *s = fmaf(c0, d, s0);
}

// 2^e as the readers apply it: the byte of an E8M0 scale is the biased FP32
// exponent (0 stands for 2^-127, a subnormal; 255 for NaN).
__device__ __forceinline__ float paged_scale(uint32_t byte) {
    return byte == 0 ? __uint_as_float(0x00400000u) : byte == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23);
}

// ---- attention of new tokens ------------------------------------------------
struct PagedAttnParams {
    const __nv_bfloat16* q;      // [T, 8 ng, 128]
    const float* q_norm_w;
    const float* sinks;          // [8 ng]
    const void* k_pages;
    const void* v_pages;
    const uint8_t* k_scales;     // null: 16-bit pages
    const uint8_t* v_scales;
    __nv_bfloat16* out;          // [T, 8 ng x 128]
    float* lse;                  // [8 ng, T] or null
    char* ws;
    PagedCache c;
    int max_new, window, use_rope;
    int ctas;                    // CTAs of the step kernel
    float rope_theta, eps;
};

// A row group of the step kernel: up to NT consecutive new tokens of one
// sequence; its tiles are runs of positions from the 16-aligned start of what
// its rows see.
struct PagedGroup { int b, row0, nrows, tiles; };

struct PagedPlanHeader {
    int status;                  // device-side status (0 = ok)
    int n_groups;                // row groups of the step kernel
    long long tiles;             // the sum of their tiles (of one KV head)
    int pad[60];
};
static_assert(sizeof(PagedPlanHeader) == 256, "plan header");

// Workspace of an attention call.
struct PagedWs {
    size_t header, inv, groups, prefix, arrive, part, total;
};
__host__ __device__ inline PagedWs paged_ws(int T, int ng, int ctas) {
    PagedWs L;
    size_t o = 256;
    L.header = 0;
    L.inv = o;    o += 64 * sizeof(double);
    L.groups = o; o = ws_align(o + sizeof(PagedGroup) * (size_t)T, 256);
    L.prefix = o; o = ws_align(o + sizeof(long long) * ((size_t)T + 1), 256);
    L.arrive = o; o = ws_align(o + sizeof(int) * (size_t)T * ng, 256);
    // two partials a CTA (its first and its last segment), up to 16 rows each
    L.part = o;   o = ws_align(o + sizeof(float) * (size_t)ctas * 2 * 16 * (kHD + 2), 256);
    L.total = o;
    return L;
}

}  // namespace flint
