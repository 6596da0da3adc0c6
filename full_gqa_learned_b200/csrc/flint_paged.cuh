// Definitions shared by the kernels of the paged key/value cache
// (flint_paged.cu: append, read back and the host side; flint_paged_step.cu with
// flint_paged_walk.cuh: attention of few new tokens per sequence;
// flint_paged_chunk.cu: of many).
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
// Keys are read back and multiplied in FP16: 448 x 2^7 is the largest multiple
// that no rounding takes out of its range.
constexpr int kPagedKeyEMax = 7;

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

// A word of the call's arrays (read-only while its kernels run).
__host__ __device__ __forceinline__ int paged_ld(const int* p) {
#ifdef __CUDA_ARCH__
    return __ldg(p);
#else
    return *p;
#endif
}

// Last b in [0, n) with a[b] <= x, for a non-decreasing a with a[0] <= x;
// warp-wide (x uniform): 32 probes a step.  Any other a gives some index in
// [0, n), so callers check what they read there.  On the host one thread makes
// the same probes.
template <typename I, typename X>
__host__ __device__ __forceinline__ int warp_last_leq(const I* a, int n, X x) {
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        int k = 0;
#ifdef __CUDA_ARCH__
        const int at = (int)(threadIdx.x & 31) * step;
        const bool le = at < n && (X)a[lo + at] <= x;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        if (m) k = 31 - __clz(m);
#else
        for (int l = 0; l < 32 && l * step < n; ++l)
            if ((X)a[lo + l * step] <= x) k = l;
#endif
        lo += k * step;
        const int rest = n - k * step;
        n = step < rest ? step : rest;
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

// The two E4M3 codes in the low half of a word as two FP16 values (exact).
__device__ __forceinline__ uint32_t e4m3_f16(uint32_t codes) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(codes));
    return r;
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
    int step_ctas, chunk_ctas;   // CTAs of the two kernels (chunk: 0 where it is not run)
    int stage_rows;              // positions a sequence has room to expand to 16 bits (0: none)
    float rope_theta, eps;
    // > 0: test hook.  The step kernel's consumers first wait this many
    // nanoseconds on a barrier nothing arrives on (FLINT_ERR_TIMEOUT, abort).
    unsigned long long test_wait_ns;
};

// A row group: consecutive new tokens of one sequence that a kernel takes
// together (at most `nt` of its list).  Its tiles are runs of positions from
// the aligned start of what its rows see.
struct PagedGroup {
    int b, nrows, tiles;
    int p0;                      // position of its first row
    int row;                     // packed row of its first row
    int krow;                    // expanded row of its first chunk's first position
};

// The work of one kernel: the tiles of all (group, KV head) pairs in a row,
// group by group, head by head.  Every CTA takes a run of them, so it holds at
// most two pairs in part.  The step kernel's CTA c of G takes tiles [W c / G,
// W (c + 1) / G) of the W = tiles x heads and works that out itself; for the
// chunk kernel a plan kernel writes the groups and where every CTA starts.
struct PagedPlanHeader {
    int status;                  // device-side status (0 = ok)
    int pad[63];
};
static_assert(sizeof(PagedPlanHeader) == 256, "plan header");

// Where a chunk CTA's share starts: tile x of all, tile off of pair (gi, head).
struct PagedStart {
    long long x;
    int gi, head, off, pad;
};

// SMs that a call's shares are cut for.  The workspace does not depend on the
// device: room for a full B200's CTAs.
constexpr int kPagedMaxSms = 148;
constexpr int kChunkTok = 32;            // new tokens of a chunk kernel's group
constexpr int kPagedStepRows = 16;       // query rows of a step partial
// floats of a step partial: m[16], l[16], O[16][128]; of a chunk partial:
// m[256], l[256], O[32][256][4] (channel quads outermost)
constexpr size_t kStepPart = (size_t)kPagedStepRows * (kHD + 2);
constexpr size_t kChunkPart = (size_t)8 * kChunkTok * (kHD + 2);

// The CTA that owns tile x.
__device__ __forceinline__ long long paged_owner(long long W, long long G, long long x) { return ((x + 1) * G - 1) / W; }
// The CTAs cf .. cl that hold parts of the pair whose first tile is tile seg
// of all W, and where they left them: a CTA's first pair in slot 2 c, a later
// one (its last) in 2 c + 1.  Every CTA but cf begins inside the pair.
struct PagedParts {
    int cf, cl;
    bool second;                 // in cf's share it is not the first pair
    __device__ __forceinline__ size_t slot(int x) const { return 2 * (size_t)x + (x == cf && second ? 1 : 0); }
};
__device__ __forceinline__ PagedParts paged_parts(long long W, long long G, long long seg, int tiles) {
    PagedParts r;
    r.cf = (int)paged_owner(W, G, seg);
    r.cl = (int)paged_owner(W, G, seg + tiles - 1);
    r.second = W * r.cf / G < seg;
    return r;
}

// 32 bytes by one store (p 32-byte aligned): two of 16 leave half a sector each.
__device__ __forceinline__ void st_32(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}

// What a CTA leaves for the kernel that folds the parts.
struct PagedNote {
    int status;                  // the CTA's (step kernel)
    int fold;                    // 1: its share is the first to begin inside a pair; the pair:
    PagedParts parts;
    int row, head, rows;         // packed row of its first token, KV head, query rows
    int pad;
};

// Workspace of an attention call: of the step kernel (chunk_ctas == 0) a note
// and two partials a CTA, of the chunk kernel the plan and two partials a CTA.
struct PagedWs {
    size_t header, notes, spart, inv, starts, groups, prefix, cpart, stage_k, stage_v, total;
};
// Row groups of a chunk call at most.
__host__ __device__ inline size_t paged_groups(int B, int T) { return (size_t)T / kChunkTok + (B < T ? B : T); }
__host__ __device__ inline PagedWs paged_ws(int B, int T, int ng, int step_ctas, int chunk_ctas, int stage_rows) {
    PagedWs L;
    size_t o = 256;
    L.header = 0;
    L.notes = L.spart = L.inv = L.starts = L.groups = L.prefix = L.cpart = L.stage_k = L.stage_v = o;
    if (chunk_ctas == 0) {
        o = ws_align(o + sizeof(PagedNote) * (size_t)step_ctas, 256);
        L.spart = o; o = ws_align(o + sizeof(float) * 2 * (size_t)step_ctas * kStepPart, 256);
    } else {
        const size_t n = paged_groups(B, T);
        o = ws_align(o + sizeof(PagedNote) * (size_t)chunk_ctas, 256);
        L.inv = o;    o += 64 * sizeof(double);
        L.starts = o; o = ws_align(o + sizeof(PagedStart) * ((size_t)chunk_ctas + 1), 256);
        L.groups = o; o = ws_align(o + sizeof(PagedGroup) * n, 256);
        L.prefix = o; o = ws_align(o + sizeof(long long) * (n + 1), 256);
        L.cpart = o;  o = ws_align(o + sizeof(float) * 2 * (size_t)chunk_ctas * kChunkPart, 256);
        if (stage_rows > 0) {
            L.stage_k = o; o += (size_t)B * stage_rows * ng * kHD * 2;
            L.stage_v = o; o += (size_t)B * stage_rows * ng * kHD * 2;
        }
    }
    L.total = o;
    return L;
}

// New tokens of the sequence whose packed rows are [a, z) at positions len ..;
// -1 where its entries are ill-formed.
__host__ __device__ __forceinline__ int paged_new(const PagedCache& c, int max_new, int a, int z, int len) {
    if (a < 0 || z < a || z > c.T || len < 0 || len > FLINT_MAX_TOKENS) return -1;
    const int n = z - a;
    const long long end = (long long)len + n;
    if (n > max_new) return -1;
    return n > 0 && (end > FLINT_MAX_TOKENS || end > ((long long)c.max_pages << c.ps_log2)) ? -1 : n;
}

// Joins the sink to a row's running state (M, L in log2 units, O in units of
// 2^M): the output is O x *scale.  A sink that has no log2 in FP32 (infinite, or
// finite from 2.36e38 on) takes all the weight.
__device__ __forceinline__ void paged_finish(float M, float L, float sink, float* scale, float* lse) {
    const float s2 = sink * 1.4426950408889634f;
    if (s2 == INFINITY) {
        *scale = 0.f;
        *lse = sink;
        return;
    }
    const float m = fmaxf(M, s2);
    const float a = M > -INFINITY ? exp2f(M - m) : 0.f;
    const float l = L * a + (s2 == -INFINITY ? 0.f : exp2f(s2 - m));
    // l == 0: nothing seen and no sink; NaN (of a sink, or of L) goes through
    *scale = l == 0.f ? 0.f : a / l;
    *lse = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// A chunk CTA's share, walked pair by pair.
struct PagedShare {
    int gi, head, off;           // the next pair; off: tile of it that the share enters at
    int left;                    // tiles left in the share
};
struct PagedSeg {
    PagedGroup g;
    int head, t0, t1;            // tiles [t0, t1) of the group's pair with this head
    bool whole;                  // all of it
};
__device__ __forceinline__ bool paged_share_begin(PagedShare& s, const PagedStart* starts, int cta) {
    const PagedStart at = starts[cta];
    s.gi = at.gi;
    s.head = at.head;
    s.off = at.off;
    s.left = (int)(starts[cta + 1].x - at.x);
    return s.left > 0;
}
__device__ __forceinline__ bool paged_share_next(PagedShare& s, const PagedGroup* groups, int ng, PagedSeg& g) {
    if (s.left <= 0) return false;
    g.g = groups[s.gi];
    g.head = s.head;
    g.t0 = s.off;
    g.t1 = min(g.g.tiles, s.off + s.left);
    g.whole = g.t0 == 0 && g.t1 == g.g.tiles;
    s.left -= g.t1 - g.t0;
    s.off = 0;
    if (++s.head == ng) { s.head = 0; ++s.gi; }
    return true;
}
}  // namespace flint
