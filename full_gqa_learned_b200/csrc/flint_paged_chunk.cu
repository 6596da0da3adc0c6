// Attention of prompts' chunks over paged keys and values (sm_100a: TMA,
// tcgen05, TMEM): the operation of flint_paged_step.cu for sequences with many
// new tokens, where 8 query heads x 32 tokens share every key and the tensor
// cores, not memory, are the limit (4 x 128 FLOP a query row and key; a key
// and value of 512 bytes serve 256 rows).
//
// * A group is 32 new tokens of one sequence, a tile 16 tokens x 8 query heads
//   = 128 rows; chunks of 128 positions start at the page that holds the
//   first position any row sees, so a chunk is a whole number of pages.
//   Persistent CTAs share the chunks of all (group, KV head) pairs so that
//   each has the same work (PagedShare): a pair inside one CTA is written at
//   once, the two pairs a CTA may hold in part leave (m, l, O) in FP32, folded
//   in CTA order by the combine kernel.  Few long sequences fill the GPU as
//   well as many short ones, and the last CTA ends with the first.
// * Warp 0 loads the raw query tiles and, for 16-bit pages, K by TMA, warp 3 V:
//   a page's slots of one head are consecutive rows, so a box is a page (64
//   channels x ps slots) and 128 / ps boxes fill a chunk's half tile.  Pages
//   past the last position are not loaded.  Warp 2 writes zeros over the V
//   rows that hold no position of the group (stale slots may hold NaN, and
//   0 x NaN would reach every row); masked columns of S need no such care.
// * 8-bit pages: where the workspace has room, a kernel in front expands the
//   positions the call reads (codes x 2^e: V in BF16, exact; K in FP16, exact from
//   e = -15 on, below that rounded to FP16's subnormals) into rows of their own,
//   loaded like pages of any size.  Otherwise a third
//   warpgroup does the same chunk by chunk, into the swizzled layout that the
//   tensor core reads; it does so again for every group of 32 tokens, and four
//   warps need 5 to 7 us a chunk where the products and the softmax take 3 to 4
//   (their 120 registers hold a chunk's codes on the way: with 104, 766 us for 128
//   sequences of 1 to 16 tokens over up to 6,000 positions, with 120, 566).
// * Warp 1 issues S = Q K^T and O += P V per chunk and tile; warps 4-7 and
//   8-11 are the softmax warpgroups of the two tiles (one thread a row): RMS
//   norm and rotation of the queries in place as FP16 when a tile lands, then
//   the online softmax, P in BF16 over S in tensor memory (the product wants
//   P in V's type, and V in BF16 holds what FP16's range does not; a second, low
//   part of P would double the products, for an output that BF16 rounds by as
//   much: 2.4e-3 from the exact one instead of 1.7e-3).  The two tiles
//   alternate, so one's softmax runs under the other's products.  Interior
//   chunks after the first skip the row max while the row sum of their terms
//   stays within 2^8.  A group of at most 16 rows runs on one tile alone.
// Every wait is bounded (FLINT_ERR_TIMEOUT in the status word, abort, drain).
// The softmax warps spill 244 to 460 bytes a thread (stores; on-chip conversion
// most); states kept elsewhere were slower.
//
// Measured: 2,048 tokens over 32,049 positions, 16-bit pages: 1,179 us, 883 TF/s,
// 0.53 of the measured bf16 rate, as the forward kernel (its softmax and tensor
// pipe take turns); four chunks of 257 to 512 tokens over up to 8,703 positions of
// 8-bit pages 255 us, of which the expansion, the plan and the combine are 20.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cmath>

#include "flint_host.cuh"
#include "flint_paged.cuh"
#include "sm100.cuh"

namespace flint {

constexpr uint32_t kPcTile = 128 * kHD * 2;          // 128 rows x 128 channels x 16 bits
constexpr uint32_t kPcHalf = kPcTile / 2;            // one 64-channel swizzled half
constexpr uint32_t kPcQ = 0;                         // 2 query tiles
constexpr uint32_t kPcK = kPcQ + 2 * kPcTile;        // 2 K stages
constexpr uint32_t kPcV = kPcK + 2 * kPcTile;        // 2 V stages
constexpr uint32_t kPcStage = kPcV + 2 * kPcTile;    // output staging (and RoPE table), 4 KiB a softmax warp
constexpr uint32_t kPcStageBytes = 32 * 128;
constexpr uint32_t kPcBar = kPcStage + 8 * kPcStageBytes;
constexpr uint32_t kPcMisc = kPcBar + 32 * 8;
constexpr uint32_t kPcWq = kPcMisc + 64;             // q_norm weight (128 floats)
constexpr uint32_t kPcWalk = kPcWq + kHD * 4;         // the converting warps' places in the share
constexpr uint32_t kPcSmem = kPcWalk + 4 * 16 + 1024; // + alignment slack
static_assert(kPcSmem <= 232448, "shared memory per block");
// RoPE table of a softmax warp's 4 tokens: per token 32 frequency pairs {cos,
// cos, sin, sin} (16 bytes), then 32 pairs {-sin, -sin}; rows padded
constexpr uint32_t kPcTabCs = 32 * 16;
constexpr uint32_t kPcTabStride = kPcTabCs + 32 * 8 + 16;
static_assert(kPcTabStride % 16 == 0 && 4 * kPcTabStride <= kPcStageBytes, "RoPE table fits the staging block");

enum : uint32_t {
    PC_Q_FULL = 0, PC_Q_EMPTY = 2, PC_Q_READY = 4,
    PC_K_FULL = 6, PC_K_EMPTY = 8, PC_V_FULL = 10, PC_V_EMPTY = 12, PC_V_OK = 14,
    PC_S_FULL = 16, PC_P_FULL = 18, PC_O_FULL = 20, PC_DRAIN = 22
};

struct PcMisc {
    uint32_t tmem_base;
    int abort_flag;
    float logit_scale;   // log2(e) / sqrt(128) x 2^-eq
    float q_scale;       // 2^eq
};

// Threads and registers: 384 threads x 168 launched (8-bit pages: 512 x 128);
// the control warps give theirs to the softmax warpgroups.
// Where a chunk's keys and values come from.
enum PcSource { kPcPages, kPcCodes, kPcStaged };
template <bool FP8> struct PcShape {
    static constexpr int threads = FP8 ? 512 : 384;
    static constexpr uint32_t control = FP8 ? 40 : 80, softmax = FP8 ? 176 : 208, convert = 120;
};
static_assert(128 * 80 + 256 * 208 <= 384 * 168, "register split");
static_assert(128 * 40 + 128 * 120 + 256 * 176 <= 512 * 128, "register split, 8-bit pages");
static_assert(PcShape<true>::convert <= 128, "setmaxnreg.dec cannot raise the launch's 128");

__device__ __forceinline__ float pc_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Packed FP32 pairs: one instruction acts on both halves of a 64-bit register.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float pc_max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ uint32_t pc_pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 bf16_pair(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// ---------------------------------------------------------------- plan
// Exclusive prefix of v over the (1,024 threads') block; the block's total in *total.
template <typename I>
__device__ __forceinline__ I plan_scan(I v, I* sh, I* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    I x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    if (warp == 0) {
        I w = sh[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        sh[lane] = w;
    }
    __syncthreads();
    const I r = x - v + (warp ? sh[warp - 1] : 0);
    *total = sh[31];
    __syncthreads();
    return r;
}

// Sequence b's new tokens; 0 (and *bad) where its entries are ill-formed.
__device__ __forceinline__ int plan_new(const PagedAttnParams& p, int b, bool* bad) {
    const int n = paged_new(p.c, p.max_new, p.c.cu[b], p.c.cu[b + 1], p.c.len[b]);
    if (n < 0) *bad = true;
    return max(n, 0);
}

// One block: checks the boundaries and lengths, writes the groups, where every
// CTA's share of their chunks starts and the combine's notes, and leaves the
// rotation frequencies.
// Group offsets of the sequences are kept in shared memory; past kPlanSeqs
// sequences only every `every`-th is, and the rest is walked.
constexpr int kPlanThreads = 1024;
constexpr int kPlanSeqs = 4096;
// A chunk takes about 3 us, a pair's query prologue and epilogue 5 to 6; a pair
// held in part costs both again, 128 KiB of partial results and the combine, so
// a boundary near a pair's end moves there: within a chunk, or with two pairs a
// CTA or more a 16th of a share, at most 4 chunks.  24 sequences with 1 to 384
// new tokens over up to 40,000 positions: window 513, 8-bit (2,049, 16-bit):
// shares by chunks alone 160 us (331), by chunks and pairs 146 (281), moved by
// a chunk 123 (270), by the rule 123 (257); twice the sequences 260 -> 232.  Where
// there are 1.3 pairs of 33 chunks a CTA, moving by 2 costs 4 us of 257.
constexpr long long kCostChunk = 2, kCostPair = 3;
constexpr int kSnapPart = 16, kSnapMost = 4;
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedAttnParams p) {
    griddep_launch_dependents();
    __shared__ int s_bad, sh_i[32], off[kPlanSeqs];
    __shared__ long long sh_l[32], sh_prefix[kPlanThreads], sh_start[kPagedMaxSms + 1];
    const int tid = threadIdx.x;
    const PagedCache& c = p.c;
    const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, p.chunk_ctas, p.stage_rows);
    PagedPlanHeader* hdr = reinterpret_cast<PagedPlanHeader*>(p.ws + L.header);
    double* inv = reinterpret_cast<double*>(p.ws + L.inv);
    PagedGroup* groups = reinterpret_cast<PagedGroup*>(p.ws + L.groups);
    long long* prefix = reinterpret_cast<long long*>(p.ws + L.prefix);
    PagedStart* starts = reinterpret_cast<PagedStart*>(p.ws + L.starts);
    PagedNote* notes = reinterpret_cast<PagedNote*>(p.ws + L.notes);
    if (tid == 0) s_bad = (c.cu[0] != 0 || c.cu[c.B] > c.T) ? 1 : 0;
    if (p.use_rope && tid < 64) inv[tid] = exp2(-(double)tid / 64.0 * log2((double)p.rope_theta));
    __syncthreads();
    const int every = (c.B + kPlanSeqs - 1) / kPlanSeqs;
    const int page_mask = (1 << c.ps_log2) - 1;
    // ill-formed boundaries can name the same rows again and again; the groups
    // have room for each row once (counts stop one above it)
    const int most = (int)paged_groups(c.B, c.T);
    int n_groups = 0;
    for (int b0 = 0; b0 < c.B; b0 += kPlanThreads * every) {
        const int b1 = b0 + tid * every;
        int cnt = 0;
        bool bad = false;
        for (int b = b1; b < min(b1 + every, c.B); ++b) cnt = min(cnt + (plan_new(p, b, &bad) + kChunkTok - 1) / kChunkTok, most + 1);
        if (bad) s_bad = 1;
        int tot;
        const int ex = plan_scan(cnt, sh_i, &tot);
        if (b1 < c.B) off[b1 / every] = n_groups + ex;
        n_groups = min(n_groups + tot, most + 1);
    }
    if (n_groups > most) {
        n_groups = most;
        s_bad = 1;
    }
    __syncthreads();
    const int n_off = (c.B + every - 1) / every;
    long long tiles = 0;
    for (int g0 = 0; g0 < n_groups; g0 += kPlanThreads) {
        const int g = g0 + tid;
        PagedGroup r = {};
        if (g < n_groups) {
            int lo = 0, hi = n_off - 1;                       // last entry with off <= g
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (off[mid] <= g) lo = mid; else hi = mid - 1;
            }
            int at = off[lo];
            bool bad = false;
            for (int b = lo * every; b < c.B; ++b) {          // one step where every == 1
                const int n = plan_new(p, b, &bad), k = (n + kChunkTok - 1) / kChunkTok;
                if (g < at + k) {
                    const int row0 = (g - at) * kChunkTok;
                    r.b = b;
                    r.nrows = min(kChunkTok, n - row0);
                    r.p0 = c.len[b] + row0;
                    r.row = c.cu[b] + row0;
                    const int first = p.window > 0 ? max(0, r.p0 - p.window + 1) : 0;
                    r.tiles = (r.p0 + r.nrows - (first & ~page_mask) + kKeyChunk - 1) / kKeyChunk;
                    if (p.stage_rows > 0) {
                        const int seq_first = p.window > 0 ? max(0, c.len[b] - p.window + 1) : 0;
                        r.krow = b * p.stage_rows + (first & ~page_mask) - (seq_first & ~page_mask);
                    }
                    break;
                }
                at += k;
            }
        }
        long long tot;
        const long long ex = plan_scan((long long)r.tiles, sh_l, &tot);
        if (g < n_groups) {
            groups[g] = r;
            prefix[g] = tiles + ex;
        }
        if (g0 == 0) sh_prefix[tid] = ex;
        tiles += tot;
    }
    if (tid == 0) {
        prefix[n_groups] = tiles;
        hdr->status = s_bad ? kStatusInvalid : kStatusOk;
    }
    __syncthreads();
    // Where the CTAs start.  Where shares are too short for every CTA to get a
    // chunk by the rule above, chunks alone count (a constant start takes at
    // most (2 snap + 1) a + o of the cost).
    const long long all = tiles * c.ng;
    long long W = c.ng * (kCostChunk * tiles + kCostPair * n_groups), a = kCostChunk, o = kCostPair, G = p.chunk_ctas;
    int snap = (long long)n_groups * c.ng < 2 * G ? 1 : max(1, min(kSnapMost, (int)(all / (kSnapPart * G))));
    if (W / G < (2 * snap + 2) * a + 2 * o) {
        snap = 0;
        W = all;
        a = 1;
        o = 0;
        G = min(W, G);
    }
    for (int x = tid; x <= p.chunk_ctas; x += kPlanThreads) {
        PagedStart st = {all, n_groups, 0, 0, 0};
        const long long pos = x < G ? W * x / G : W;
        if (pos < W) {
            auto pre = [&](int g) { return g == n_groups ? tiles : n_groups <= kPlanThreads ? sh_prefix[g] : prefix[g]; };
            int lo = 0, hi = n_groups - 1;                    // last group that starts at or before pos
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (c.ng * (a * pre(mid) + o * mid) <= pos) lo = mid; else hi = mid - 1;
            }
            const long long g0 = pre(lo), k = pre(lo + 1) - g0, in = pos - c.ng * (a * g0 + o * lo), w = a * k + o;
            const int head = (int)(in / w);
            long long off = max(in - head * w - o + a - 1, 0ll) / a;             // a chunk belongs to whose share holds its first unit
            off = off <= snap ? 0 : k - off <= snap ? k : off;
            st.x = g0 * c.ng + head * k + off;
            st.gi = lo;
            st.head = head;
            st.off = (int)off;
            if (off == k) {                                   // the next pair's first
                st.off = 0;
                if (++st.head == c.ng) {
                    st.head = 0;
                    ++st.gi;
                }
            }
        }
        starts[x] = st;
        sh_start[x] = st.x;
    }
    __syncthreads();
    // A pair that a share begins inside of is held in part by the CTAs before,
    // too: the first CTA of those leaves the combine a note.
    for (int x = tid; x < p.chunk_ctas; x += kPlanThreads) {
        const PagedStart st = starts[x];
        PagedNote n = {};
        if (sh_start[x + 1] > st.x && st.off > 0) {
            const PagedGroup g = groups[st.gi];
            auto owner = [&](long long tile) {                // the CTA that holds it
                int lo = 0, hi = p.chunk_ctas - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (sh_start[mid] <= tile) lo = mid; else hi = mid - 1;
                }
                return lo;
            };
            const long long seg = st.x - st.off;
            n.parts.cf = owner(seg);
            n.parts.cl = owner(seg + g.tiles - 1);
            n.parts.second = sh_start[n.parts.cf] < seg;
            n.fold = n.parts.cf == x - 1;
            n.row = g.row;
            n.head = st.head;
            n.rows = kGroup * g.nrows;
        }
        notes[x] = n;
    }
}

// ---------------------------------------------------------------- expansion of 8-bit pages
// A warp takes 16 positions of one sequence and KV head: eight lanes a row, 16
// codes a lane, four rows at once.  Rows without a position are not written (the chunk kernel
// masks them and clears their values).  Sequence b's rows start at b x
// stage_rows.  It moves 258 bytes in and 512 out per position and head.
constexpr int kExpandThreads = 256;
__global__ void __launch_bounds__(kExpandThreads) paged_expand_kernel(const PagedAttnParams p) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, rl = lane >> 3, sub = lane & 7;
    const PagedCache& c = p.c;
    const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, p.chunk_ctas, p.stage_rows);
    PagedPlanHeader* hdr = reinterpret_cast<PagedPlanHeader*>(p.ws + L.header);
    __half* ks = reinterpret_cast<__half*>(p.ws + L.stage_k);
    __nv_bfloat16* vs = reinterpret_cast<__nv_bfloat16*>(p.ws + L.stage_v);
    const uint8_t* kp = static_cast<const uint8_t*>(p.k_pages);
    const uint8_t* vp = static_cast<const uint8_t*>(p.v_pages);
    const int blocks = p.stage_rows / 16, n = c.B * blocks * c.ng, warps = gridDim.x * (kExpandThreads / 32);
    bool bad = false;
    for (int w = blockIdx.x * (kExpandThreads / 32) + (threadIdx.x >> 5); w < n; w += warps) {
        const int b = w / (blocks * c.ng), x = w / c.ng % blocks, g = w % c.ng;
        const int len = c.len[b], a = c.cu[b], z = c.cu[b + 1], nn = paged_new(c, p.max_new, a, z, len);
        const int end = len + nn, lo = p.window > 0 ? max(0, len - p.window + 1) : 0;
        const int pos = (lo & ~((1 << c.ps_log2) - 1)) + 16 * x;
        if (nn <= 0 || pos >= end || pos + 16 <= lo) continue;
        const int page = __ldg(c.table + (size_t)b * c.max_pages + (pos >> c.ps_log2));
        if (page < 0 || page >= c.num_pages) {
            bad = true;
            continue;
        }
        const size_t src = paged_row(c, page, g, pos & ((1 << c.ps_log2) - 1)), dst = ((size_t)g * c.B + b) * p.stage_rows + 16 * x;
        uint4 kc[4], vc[4];
        uint32_t sk[4], sv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * i + rl;
            if (pos + r < lo || pos + r >= end) continue;
            kc[i] = __ldg(reinterpret_cast<const uint4*>(kp + (src + r) * kHD) + sub);
            vc[i] = __ldg(reinterpret_cast<const uint4*>(vp + (src + r) * kHD) + sub);
            sk[i] = __ldg(p.k_scales + src + r);
            sv[i] = __ldg(p.v_scales + src + r);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * i + rl;
            if (pos + r < lo || pos + r >= end) continue;
            const __half2 ks2 = __float2half2_rn(paged_scale(sk[i]));
            const float vsf = paged_scale(sv[i]);
            const uint32_t kw[4] = {kc[i].x, kc[i].y, kc[i].z, kc[i].w}, vw[4] = {vc[i].x, vc[i].y, vc[i].z, vc[i].w};
            uint32_t ko[8], vo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t kh = e4m3_f16(kw[e >> 1] >> (16 * (e & 1))), vh = e4m3_f16(vw[e >> 1] >> (16 * (e & 1)));
                const __half2 kk = __hmul2(*reinterpret_cast<const __half2*>(&kh), ks2);
                const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&vh));
                ko[e] = *reinterpret_cast<const uint32_t*>(&kk);
                vo[e] = pc_pack_bf16(vf.x * vsf, vf.y * vsf);
            }
            st_32(ks + (dst + r) * kHD + 16 * sub, make_uint4(ko[0], ko[1], ko[2], ko[3]), make_uint4(ko[4], ko[5], ko[6], ko[7]));
            st_32(vs + (dst + r) * kHD + 16 * sub, make_uint4(vo[0], vo[1], vo[2], vo[3]), make_uint4(vo[4], vo[5], vo[6], vo[7]));
        }
    }
    // nothing above needs the plan; it writes the status word, and who waits
    // for this grid waits for it, too
    griddep_wait();
    if (bad && lane == 0) atomicCAS(&hdr->status, 0, kStatusInvalid);
}

// ---------------------------------------------------------------- chunk kernel
// What a group sees of its cache, and its chunks.
struct PcGroup {
    int p0, hi;          // position of its first row; one past its last row's
    int kb;              // first position of chunk 0, a page's first
    int lo;              // first position any row sees
    int row;             // packed row of its first token
};
__device__ __forceinline__ PcGroup pc_group(const PagedAttnParams& p, const PagedGroup& g) {
    PcGroup r;
    r.p0 = g.p0;
    r.hi = r.p0 + g.nrows;
    r.lo = p.window > 0 ? max(0, r.p0 - p.window + 1) : 0;
    r.kb = r.lo & ~((1 << p.c.ps_log2) - 1);
    r.row = g.row;
    return r;
}
// Columns of the chunk that starts at ks: up to the group's last position,
// rounded up to the MMA's step of 16.
__device__ __forceinline__ int pc_cols(int ks, int hi) { return min(kKeyChunk, (hi - ks + 15) & ~15); }

template <PcSource SRC>
__global__ void __launch_bounds__(PcShape<SRC == kPcCodes>::threads, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                   const __grid_constant__ CUtensorMap tm_o1, const PagedAttnParams p) {
    constexpr bool FP8 = SRC == kPcCodes;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + kPcBar;
    auto bar = [&](uint32_t i) { return bar0 + 8u * i; };
    PcMisc* misc = reinterpret_cast<PcMisc*>(smem + kPcMisc);
    volatile int* abort_flag = &misc->abort_flag;
    const PagedCache& c = p.c;
    const int ng = c.ng;
    const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, p.chunk_ctas, p.stage_rows);
    PagedPlanHeader* hdr = reinterpret_cast<PagedPlanHeader*>(p.ws + L.header);
    int* status = &hdr->status;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---------------------------------------------------------------- setup
    griddep_launch_dependents();
    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(bar(PC_Q_FULL + t), 1);
            mbar_init(bar(PC_Q_EMPTY + t), 1);
            mbar_init(bar(PC_Q_READY + t), 128);       // every softmax thread of tile t
            mbar_init(bar(PC_K_FULL + t), FP8 ? 4 : 1);   // the converting warps, or the loads
            mbar_init(bar(PC_K_EMPTY + t), 1);
            mbar_init(bar(PC_V_FULL + t), FP8 ? 4 : 1);
            mbar_init(bar(PC_V_EMPTY + t), 1);
            mbar_init(bar(PC_V_OK + t), 1);
            mbar_init(bar(PC_S_FULL + t), 1);
            mbar_init(bar(PC_P_FULL + t), 128);
            mbar_init(bar(PC_O_FULL + t), 1);
        }
        mbar_init(bar(PC_DRAIN), 1);
        misc->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tm_q);
        if (!FP8) {
            tma_prefetch_desc(&tm_k);
            tma_prefetch_desc(&tm_v);
        }
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&misc->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 2) {
        const int eq = prescale_exponent(warp_max_abs128(p.q_norm_w));
        if (lane == 0) {
            misc->logit_scale = ldexpf(1.4426950408889634f * 0.08838834764831845f, -eq);
            misc->q_scale = ldexpf(1.f, eq);
        }
    }
    if (warp == 3) {
        float* wq = reinterpret_cast<float*>(smem + kPcWq);
#pragma unroll
        for (int i = 0; i < 4; ++i) wq[lane + 32 * i] = p.q_norm_w[lane + 32 * i];
    }
    // the plan is read only after its kernel completed
    griddep_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc->tmem_base;
    PagedShare share;
    PagedSeg sg;
    bool first = true;
    const PagedStart* starts = reinterpret_cast<const PagedStart*>(p.ws + L.starts);
    const PagedGroup* groups = reinterpret_cast<const PagedGroup*>(p.ws + L.groups);
    const bool work = paged_share_begin(share, starts, blockIdx.x);

    if (!work) {
        // nothing in flight: straight to the end
    } else if (warp < 4) {
      regs_dec<PcShape<FP8>::control>();
      if (warp == 0 || warp == 3) {
        // ============================================================ producers: queries and K (warp 0), V (warp 3)
        // (one warp for both would hold K back behind a V stage in use)
        const bool is_k = warp == 0;
        const uint32_t full = is_k ? PC_K_FULL : PC_V_FULL, empty = is_k ? PC_K_EMPTY : PC_V_EMPTY;
        const uint32_t tile = sbase + (is_k ? kPcK : kPcV);
        uint32_t qph[2] = {0u, 0u}, st = 0, ph = 0, narm_q[2] = {0u, 0u}, narm = 0;
        bool ok = true;
        while (ok && paged_share_next(share, groups, ng, sg)) {
            const PcGroup gr = pc_group(p, sg.g);
            const int ntile = !is_k ? 0 : sg.g.nrows > kTokPerTile ? 2 : 1;
            for (int t = 0; t < ntile && ok; ++t) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(PC_Q_EMPTY + t), qph[t] ^ 1, abort_flag, status));
                if (!ok) break;
                if (lane == 0) {
                    const uint32_t dst = sbase + kPcQ + t * kPcTile;
                    mbar_expect_tx(bar(PC_Q_FULL + t), kPcTile);
                    tma_load_3d(dst, &tm_q, bar(PC_Q_FULL + t), 0, kGroup * sg.head, gr.row + kTokPerTile * t);
                    tma_load_3d(dst + kPcHalf, &tm_q, bar(PC_Q_FULL + t), 64, kGroup * sg.head, gr.row + kTokPerTile * t);
                }
                ++narm_q[t];
                qph[t] ^= 1;
            }
            if (FP8 || !ok) continue;
            // lane i < 128 / ps loads page i of each chunk; its table entry is
            // fetched a chunk ahead.  Expanded rows: one box.
            const int ps = SRC == kPcStaged ? kKeyChunk : 1 << c.ps_log2, npg = SRC == kPcStaged ? 1 : kKeyChunk >> c.ps_log2;
            const int* table = c.table + (size_t)sg.g.b * c.max_pages;
            auto entry = [&](int ch) -> int {
                if (SRC == kPcStaged) return lane == 0 ? 0 : -2;
                const int pos = gr.kb + kKeyChunk * ch + lane * ps;
                return lane < npg && pos < gr.hi ? max(__ldg(table + (pos >> c.ps_log2)), -1) : -2;
            };
            int pg = entry(sg.t0);
            for (int ch = sg.t0; ch < sg.t1; ++ch) {
                const bool live = pg >= 0 && pg < c.num_pages;
                if (!live && pg != -2) atomicCAS(status, 0, kStatusInvalid);
                const int page = pg;
                pg = ch + 1 < sg.t1 ? entry(ch + 1) : -2;
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * ps * kHD * 2;
                const int y = SRC == kPcStaged ? sg.g.krow + kKeyChunk * ch : 0;
                const int z = SRC == kPcStaged ? sg.head : live ? page * ng + sg.head : 0;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(empty + st), ph ^ 1, abort_flag, status));
                if (!ok) break;
                if (lane == 0) mbar_expect_tx(bar(full + st), bytes);
                __syncwarp();
                const uint32_t dst = tile + st * kPcTile + lane * ps * 128;
                if (live) {
                    tma_load_3d(dst, is_k ? &tm_k : &tm_v, bar(full + st), 0, y, z);
                    tma_load_3d(dst + kPcHalf, is_k ? &tm_k : &tm_v, bar(full + st), 64, y, z);
                }
                ++narm;
                st ^= 1; if (st == 0) ph ^= 1;
            }
        }
        // drain: every armed load has landed before shared memory is released
        volatile int never = 0;
        const unsigned long long lim = 100ull * 1000ull * 1000ull;
        for (uint32_t t = 0; t < 2; ++t) {
            if (narm_q[t]) mbar_wait(bar(PC_Q_FULL + t), (narm_q[t] - 1) & 1, &never, nullptr, lim);
            const uint32_t n = (narm + 1 - t) / 2;     // stage t received loads number t, t + 2, ...
            if (n) mbar_wait(bar(full + t), (n - 1) & 1, &never, nullptr, lim);
        }
      } else if (warp == 1) {
        // ============================================================ MMA issuer
        const uint32_t idesc_pv = idesc_f16(1, 1, 1, 128);
        const uint64_t dq0 = smem_desc_sw128(sbase + kPcQ, 16, 1024);
        const uint64_t dk0 = smem_desc_sw128(sbase + kPcK, 16, 1024);
        const uint64_t dv0 = smem_desc_sw128(sbase + kPcV, kPcHalf, 1024);
        const uint32_t q_lo = (uint32_t)dq0, q_hi = (uint32_t)(dq0 >> 32);
        const uint32_t k_lo = (uint32_t)dk0, k_hi = (uint32_t)(dk0 >> 32);
        const uint32_t v_lo = (uint32_t)dv0, v_hi = (uint32_t)(dv0 >> 32);
        constexpr uint32_t kStep = kPcTile >> 4;
        constexpr uint32_t kVReady = FP8 ? PC_V_FULL : PC_V_OK;
        auto issue_s = [&](uint32_t t, uint32_t stage, int ncols) {
            const uint32_t idesc = idesc_f16(0, 0, 0, (uint32_t)ncols);
            const uint32_t qa = q_lo + t * kStep, kb = k_lo + stage * kStep, d = tmem + 128u * t;
#pragma unroll
            for (uint32_t kk = 0; kk < kHD / 16; ++kk) {
                const uint32_t off = (kk >> 2) * (kPcHalf >> 4) + (kk & 3) * 2;
                mma_ss_w(d, qa + off, q_hi, kb + off, k_hi, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit(bar(PC_S_FULL + t));
        };
        auto issue_pv = [&](uint32_t t, uint32_t stage, int ncols, bool acc) {
            const uint32_t vb = v_lo + stage * kStep, d = tmem + 256u + 128u * t, pa = tmem + 128u * t;
            const int nk = ncols >> 4;
            mma_ts_w(d, pa, vb, v_hi, idesc_pv, acc ? 1u : 0u);
#pragma unroll
            for (int kk = 1; kk < 8; ++kk)
                if (kk < nk) mma_ts_w(d, pa + 8u * kk, vb + kk * (2048 >> 4), v_hi, idesc_pv, 1u);
        };
        // the whole warp walks the share; lane 0 waits and issues, the others
        // follow its outcome
        uint32_t kst = 0, kph = 0, vst = 0, vph = 0, qrph[2] = {0u, 0u}, pph[2] = {0u, 0u};
        bool ok = true;
        while (ok && paged_share_next(share, groups, ng, sg)) {
            if (lane == 0) {
                const PcGroup gr = pc_group(p, sg.g);
                const int ntile = sg.g.nrows > kTokPerTile ? 2 : 1, n = sg.t1 - sg.t0;
                const int ks0 = gr.kb + kKeyChunk * sg.t0;
                auto wait = [&](uint32_t b, uint32_t parity) {
                    if (ok) ok = mbar_wait(bar(b), parity, abort_flag, status);
                    return ok;
                };
                auto step_k = [&]() { kst ^= 1; if (kst == 0) kph ^= 1; };
                int nc = pc_cols(ks0, gr.hi);
                if (wait(PC_K_FULL + kst, kph)) {
                    for (int t = 0; t < ntile; ++t) {
                        if (!wait(PC_Q_READY + t, qrph[t])) break;
                        qrph[t] ^= 1;
                        tc_fence_after();
                        issue_s(t, kst, nc);
                        if (n == 1) mma_commit(bar(PC_Q_EMPTY + t));
                    }
                    if (ok) {
                        mma_commit(bar(PC_K_EMPTY + kst));
                        step_k();
                    }
                }
                for (int i = 0; i < n && ok; ++i) {
                    const bool more = i + 1 < n;
                    const int nn = more ? pc_cols(ks0 + kKeyChunk * (i + 1), gr.hi) : 0;
                    if (!wait(kVReady + vst, vph)) break;
                    for (int t = 0; t < ntile; ++t) {
                        if (!wait(PC_P_FULL + t, pph[t])) break;
                        pph[t] ^= 1;
                        tc_fence_after();
                        issue_pv(t, vst, nc, i > 0);
                        if (t == ntile - 1) mma_commit(bar(PC_V_EMPTY + vst));
                        if (more) {
                            if (t == 0 && !wait(PC_K_FULL + kst, kph)) break;
                            tc_fence_after();
                            issue_s(t, kst, nn);
                            if (i + 2 == n) mma_commit(bar(PC_Q_EMPTY + t));
                        } else {
                            mma_commit(bar(PC_O_FULL + t));
                        }
                    }
                    if (!ok) break;
                    if (more) {
                        mma_commit(bar(PC_K_EMPTY + kst));
                        step_k();
                    }
                    vst ^= 1; if (vst == 0) vph ^= 1;
                    nc = nn;
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        if (lane == 0) {
            // drain: every MMA issued so far has completed
            mma_commit(bar(PC_DRAIN));
            volatile int never = 0;
            mbar_wait(bar(PC_DRAIN), 0, &never, nullptr, 100ull * 1000ull * 1000ull);
        }
        __syncwarp();
      } else if (warp == 2 && !FP8) {
        // ============================================================ V rows without a position
        uint32_t st = 0, ph = 0;
        bool ok = true;
        while (ok && paged_share_next(share, groups, ng, sg)) {
            const PcGroup gr = pc_group(p, sg.g);
            for (int ch = sg.t0; ch < sg.t1; ++ch) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(PC_V_FULL + st), ph, abort_flag, status));
                if (!ok) break;
                const int ks = gr.kb + kKeyChunk * ch;
                if (ks < gr.lo || ks + kKeyChunk > gr.hi) {
                    const int r0 = max(0, gr.lo - ks), r1 = min(kKeyChunk, gr.hi - ks), nc = pc_cols(ks, gr.hi);
                    uint8_t* v = smem + kPcV + st * kPcTile;
                    // 16 lanes a row: 8 x 16 bytes of each channel half
                    for (int r = lane >> 4; r < nc; r += 2) {
                        if (r >= r0 && r < r1) continue;
                        *reinterpret_cast<uint4*>(v + ((lane >> 3) & 1) * kPcHalf + r * 128 + (lane & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(bar(PC_V_OK + st));
                st ^= 1; if (st == 0) ph ^= 1;
            }
        }
      }
    } else if (FP8 && warp >= 12) {
        regs_dec<PcShape<FP8>::convert>();
        // ============================================================ 8-bit pages: codes and scales -> FP16 K, BF16 V
        // Warp w takes rows 32 w .. 32 w + 31 of each chunk, four at a time:
        // lane (a, b, s) = bits (4-3, 2, 1-0) holds codes 16 sub .. + 15, sub =
        // 4 (a / 2) + s, of row 2 (a % 2) + b, so that the eight lanes of a
        // store phase, rows of both parities, meet no bank twice.  K's and V's
        // codes are fetched one chunk ahead of their conversion.  Rows without
        // a position become zeros.
        const int w = warp - 12, sub = 4 * (lane >> 4) + (lane & 3), rl = 2 * ((lane >> 3) & 1) + ((lane >> 2) & 1);
        const uint8_t* kp = static_cast<const uint8_t*>(p.k_pages);
        const uint8_t* vp = static_cast<const uint8_t*>(p.v_pages);
        uint32_t st = 0, ph = 0;
        bool ok = true;
        // the place in the share is kept in shared memory: the codes on their
        // way take the registers
        PagedShare* walk = reinterpret_cast<PagedShare*>(smem + kPcWalk) + w;
        if (lane == 0) *walk = share;
        __syncwarp();
        auto next_pair = [&]() -> bool {
            PagedShare sh = *walk;
            __syncwarp();
            const bool more = paged_share_next(sh, groups, ng, sg);
            if (lane == 0) *walk = sh;
            __syncwarp();
            return more;
        };
        while (ok && next_pair()) {
            const PcGroup gr = pc_group(p, sg.g);
            const int* table = c.table + (size_t)sg.g.b * c.max_pages;
            // Pages of the warp's 32 positions of chunk ch, lane l's position
            // ks + l: -1 none, -2 no position.
            auto page_of = [&](int ch) -> int {
                const int pos = gr.kb + kKeyChunk * ch + 32 * w + lane;
                return ch < sg.t1 && pos >= gr.lo && pos < gr.hi ? max(__ldg(table + (pos >> c.ps_log2)), -1) : -2;
            };
            // Row of the pools, or -1.
            auto row_of = [&](int page, int ch) -> long long {
                if (page == -2) return -1;
                if (page < 0 || page >= c.num_pages) {
                    atomicCAS(status, 0, kStatusInvalid);
                    return -1;
                }
                const int pos = gr.kb + kKeyChunk * ch + 32 * w + lane;
                return (long long)paged_row(c, page, sg.head, pos & ((1 << c.ps_log2) - 1));
            };
            auto load = [&](const uint8_t* pages, long long row, uint4* x) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const long long r = __shfl_sync(0xffffffffu, row, 4 * i + rl);
                    x[i] = r >= 0 ? __ldg(reinterpret_cast<const uint4*>(pages + r * kHD) + sub) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            auto place = [&](uint32_t tile, int r, const uint32_t* h) {
                uint8_t* d = smem + tile + (sub >> 2) * kPcHalf + r * 128;
                const int c0 = 2 * (sub & 3);
                *reinterpret_cast<uint4*>(d + ((c0 ^ (r & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(d + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
            };
            long long row = row_of(page_of(sg.t0), sg.t0);
            uint4 xk[8], xv[8];
            load(kp, row, xk);
            load(vp, row, xv);
            uint32_t sk = row >= 0 ? __ldg(p.k_scales + row) : 127u, sv = row >= 0 ? __ldg(p.v_scales + row) : 127u;
            int pg = page_of(sg.t0 + 1);
            for (int ch = sg.t0; ch < sg.t1; ++ch) {
                const long long next = row_of(pg, ch + 1);
                pg = page_of(ch + 2);
                ok = __all_sync(0xffffffffu, mbar_wait(bar(PC_K_EMPTY + st), ph ^ 1, abort_flag, status));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const __half2 s2 = __float2half2_rn(paged_scale(__shfl_sync(0xffffffffu, sk, 4 * i + rl)));
                    const uint32_t cw[4] = {xk[i].x, xk[i].y, xk[i].z, xk[i].w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t v = e4m3_f16(cw[e >> 1] >> (16 * (e & 1)));
                        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&v), s2);
                        h[e] = *reinterpret_cast<const uint32_t*>(&y);
                    }
                    place(kPcK + st * kPcTile, 32 * w + 4 * i + rl, h);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(PC_K_FULL + st));
                load(kp, next, xk);
                sk = next >= 0 ? __ldg(p.k_scales + next) : 127u;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(PC_V_EMPTY + st), ph ^ 1, abort_flag, status));
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = paged_scale(__shfl_sync(0xffffffffu, sv, 4 * i + rl));
                    const uint32_t cw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
                    uint32_t h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t v = e4m3_f16(cw[e >> 1] >> (16 * (e & 1)));
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
                        h[e] = pc_pack_bf16(f.x * s, f.y * s);
                    }
                    place(kPcV + st * kPcTile, 32 * w + 4 * i + rl, h);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(PC_V_FULL + st));
                load(vp, next, xv);
                sv = next >= 0 ? __ldg(p.v_scales + next) : 127u;
                st ^= 1; if (st == 0) ph ^= 1;
            }
        }
    } else {
        regs_inc<PcShape<FP8>::softmax>();
        // ============================================================ softmax
        const int t = (warp - 4) >> 2;               // tile 0 or 1
        const int r = tid - 128 - 128 * t;           // row = TMEM lane, 0..127
        const int tl = r >> 3, hl = r & 7;           // token within tile, head within group
        const uint32_t lane_base = (uint32_t)(warp & 3) * 32u;
        const uint32_t t_s = tmem + (lane_base << 16) + 128u * t;
        const uint32_t t_o = tmem + (lane_base << 16) + 256u + 128u * t;
        const float C = misc->logit_scale;
        uint32_t s_ph = 0, oph = 0, qph = 0;
        uint8_t* stg = smem + kPcStage + (warp - 4) * kPcStageBytes;
        const uint32_t stg_s = sbase + kPcStage + (warp - 4) * kPcStageBytes;
        // The next pair this tile takes part in, in few registers (the softmax
        // needs them): its first chunk's start, chunks, one past its last
        // position, the tile's first position and packed row; rows, head,
        // whole and first.
        struct Work { int ks, n, hi, pos0, row, info; };
        auto fetch = [&](Work& w) -> bool {
            while (paged_share_next(share, groups, ng, sg)) {
                const bool f = first;
                first = false;
                if (t != 0 && sg.g.nrows <= kTokPerTile) continue;
                const PcGroup g = pc_group(p, sg.g);
                w.ks = g.kb + kKeyChunk * sg.t0;
                w.n = sg.t1 - sg.t0;
                w.hi = g.hi;
                w.pos0 = g.p0 + kTokPerTile * t;
                w.row = g.row + kTokPerTile * t;
                w.info = (sg.g.nrows - kTokPerTile * t) << 8 | sg.head << 2 | (sg.whole ? 2 : 0) | (f ? 1 : 0);
                return true;
            }
            return false;
        };
        // Query prologue: thread r normalises row r of the tile in place
        // (weight-form RMSNorm), rotates channel pairs (f, f + 64) by pos x
        // theta^(-f/64) and leaves FP16 x 2^eq.
        auto prepare_q = [&](const int pos0) -> bool {
            if (!__all_sync(0xffffffffu, mbar_wait(bar(PC_Q_FULL + t), qph, abort_flag, status))) return false;
            qph ^= 1;
            const uint8_t* tab = stg + (lane >> 3) * kPcTabStride;
            if (p.use_rope) {
                // this warp's 4 tokens x 32 frequency pairs; the block is free
                // once lane 0's earlier output stores have read it
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
                const int pos = pos0 + tl;
                const double* inv = reinterpret_cast<const double*>(p.ws + L.inv);
                uint8_t* tw = stg + (lane >> 3) * kPcTabStride;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int pp = 4 * hl + e;                       // pair (2 pp, 2 pp + 1)
                    float c0, s0, c1, s1;
                    rope_cos_sin(pos, inv[2 * pp], &c0, &s0);
                    rope_cos_sin(pos, inv[2 * pp + 1], &c1, &s1);
                    *reinterpret_cast<float4*>(tw + 16 * pp) = make_float4(c0, c1, s0, s1);
                    *reinterpret_cast<float2*>(tw + kPcTabCs + 8 * pp) = make_float2(-s0, -s1);
                }
                __syncwarp();
            }
            uint8_t* qrow = smem + kPcQ + t * kPcTile + r * 128;
            const int swz = r & 7;
            uint64_t ss2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const uint4 a = *reinterpret_cast<const uint4*>(qrow + (x >> 3) * kPcHalf + (((x & 7) ^ swz) << 4));
                const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = bf16_pair(av[j]);
                    const uint64_t v2 = f2(f.x, f.y);
                    ss2[j] = f2_fma(v2, v2, ss2[j]);
                }
            }
            const float2 sst = f2_get(f2_add(f2_add(ss2[0], ss2[1]), f2_add(ss2[2], ss2[3])));
            const float rn = rsqrtf((sst.x + sst.y) * (1.f / kHD) + p.eps) * misc->q_scale;
            const uint64_t rn2 = f2(rn, rn);
            const float* wq = reinterpret_cast<const float*>(smem + kPcWq);
#pragma unroll 2
            for (int x = 0; x < 8; ++x) {
                uint8_t* pa = qrow + ((x ^ swz) << 4);
                uint8_t* pb = pa + kPcHalf;
                const uint4 a = *reinterpret_cast<const uint4*>(pa);
                const uint4 b = *reinterpret_cast<const uint4*>(pb);
                const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
                uint32_t h0[4], h1[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 fa = bf16_pair(av[e]), fb = bf16_pair(bv[e]);
                    const float2 wa = *reinterpret_cast<const float2*>(wq + 8 * x + 2 * e);
                    const float2 wb = *reinterpret_cast<const float2*>(wq + 64 + 8 * x + 2 * e);
                    uint64_t n0 = f2_mul(f2(fa.x, fa.y), f2(wa.x, wa.y));
                    uint64_t n1 = f2_mul(f2(fb.x, fb.y), f2(wb.x, wb.y));
                    if (p.use_rope) {
                        const int pp = 4 * x + e;
                        const float4 cs = *reinterpret_cast<const float4*>(tab + 16 * pp);
                        const float2 ns = *reinterpret_cast<const float2*>(tab + kPcTabCs + 8 * pp);
                        const uint64_t cc = f2(cs.x, cs.y), sn = f2(cs.z, cs.w), nsn = f2(ns.x, ns.y);
                        const uint64_t y0 = f2_fma(n1, nsn, f2_mul(n0, cc));   // n0 cos - n1 sin
                        const uint64_t y1 = f2_fma(n0, sn, f2_mul(n1, cc));    // n1 cos + n0 sin
                        n0 = y0;
                        n1 = y1;
                    }
                    const float2 g0 = f2_get(f2_mul(n0, rn2)), g1 = f2_get(f2_mul(n1, rn2));
                    const __half2 lo = __floats2half2_rn(g0.x, g0.y), hi = __floats2half2_rn(g1.x, g1.y);
                    h0[e] = *reinterpret_cast<const uint32_t*>(&lo);
                    h1[e] = *reinterpret_cast<const uint32_t*>(&hi);
                }
                *reinterpret_cast<uint4*>(pa) = make_uint4(h0[0], h0[1], h0[2], h0[3]);
                *reinterpret_cast<uint4*>(pb) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
            }
            fence_proxy_async_smem();                  // generic writes -> the tensor core's reads
            mbar_arrive(bar(PC_Q_READY + t));
            return true;
        };
        Work wk = {};
        bool have = fetch(wk);
        if (have) have = prepare_q(wk.pos0);
        while (have) {
            const int pos0 = wk.pos0, pos = pos0 + tl;               // the tile's first position, this row's
            const int wlo = p.window > 0 ? pos - p.window + 1 : -(1 << 30);
            float m = -INFINITY, l = 0.f;                            // the sink joins at the end
            bool alive = true;
            for (int ch = 0; ch < wk.n; ++ch) {
                const bool first_ch = ch == 0;
                const int ks = wk.ks + kKeyChunk * ch;
                const int nc = pc_cols(ks, wk.hi);
                const int nblk = (nc + 31) >> 5;
                if (!__all_sync(0xffffffffu, mbar_wait(bar(PC_S_FULL + t), s_ph, abort_flag, status))) { alive = false; break; }
                s_ph ^= 1;
                tc_fence_after();
                const bool boundary = ks + kKeyChunk - 1 > pos0 || (p.window > 0 && ks < pos0 + kTokPerTile - p.window);
                const bool fastp = !boundary && !first_ch && __all_sync(0xffffffffu, m > -INFINITY && m < INFINITY);
                uint32_t sv[128];
                tmem_ld32(t_s, sv);
                if (nblk > 1) tmem_ld32(t_s + 32u, sv + 32);
                if (fastp) tmem_wait_ld();
                if (nblk > 2) tmem_ld32(t_s + 64u, sv + 64);
                if (nblk > 3) tmem_ld32(t_s + 96u, sv + 96);
                if (!fastp) tmem_wait_ld();
                // row r sees columns jlo .. jhi; each block of 32 columns is
                // full, empty or partial for the whole warp
                const int jlo = wlo - ks, jhi = min(pos - ks, nc - 1);
                uint32_t fullm = 0xFu, emptym = 0u;
                if (boundary) {
                    const int lo_max = __reduce_max_sync(0xffffffffu, jlo), lo_min = __reduce_min_sync(0xffffffffu, jlo);
                    const int hi_max = __reduce_max_sync(0xffffffffu, jhi), hi_min = __reduce_min_sync(0xffffffffu, jhi);
                    fullm = 0u;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (lo_max <= 32 * b && hi_min >= 32 * b + 31) fullm |= 1u << b;
                        else if (hi_max < 32 * b || lo_min > 32 * b + 31) emptym |= 1u << b;
                    }
                }
                auto row_max = [&]() -> float {
                    float mxp[8];
#pragma unroll
                    for (int k8 = 0; k8 < 8; ++k8) mxp[k8] = -INFINITY;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (fullm & (1u << b)) {
#pragma unroll
                            for (int j = 32 * b; j < 32 * b + 32; j += 2)
                                mxp[(j >> 1) & 7] = pc_max3(mxp[(j >> 1) & 7], __uint_as_float(sv[j]), __uint_as_float(sv[j + 1]));
                        } else if (!(emptym & (1u << b))) {
#pragma unroll
                            for (int j = 32 * b; j < 32 * b + 32; j += 2) {
                                const float x0 = ((j >= jlo) && (j <= jhi)) ? __uint_as_float(sv[j]) : -INFINITY;
                                const float x1 = ((j + 1 >= jlo) && (j + 1 <= jhi)) ? __uint_as_float(sv[j + 1]) : -INFINITY;
                                sv[j] = __float_as_uint(x0);
                                sv[j + 1] = __float_as_uint(x1);
                                mxp[(j >> 1) & 7] = pc_max3(mxp[(j >> 1) & 7], x0, x1);
                            }
                        }
                    }
                    return pc_max3(pc_max3(mxp[0], mxp[1], mxp[2]), pc_max3(mxp[3], mxp[4], mxp[5]), fmaxf(mxp[6], mxp[7]));
                };
                // Raise the running max to cover mx (on the first chunk to mx
                // itself, later only by more than 2^8); rescale l and O.
                // Whether any row of the warp did.
                auto raise_to = [&](float mx) -> bool {
                    const float m_new = fmaxf(m, mx * C);
                    const bool raise = first_ch ? (m_new > m) : (m_new > m + 8.f);
                    float alpha = 1.f;
                    if (raise) {
                        alpha = pc_ex2(m - m_new);
                        l *= alpha;
                    }
                    const bool any = __any_sync(0xffffffffu, raise);
                    if (!first_ch && any) {
#pragma unroll 1
                        for (int b = 0; b < 8; ++b) {
                            uint32_t v[16];
                            tmem_ld16(t_o + 16u * b, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
                            tmem_st16(t_o + 16u * b, v);
                        }
                    }
                    if (raise) m = m_new;
                    return any;
                };
                // P = 2^(s C - m) -> BF16 over S; the row sum.  Blocks b0 ..
                // b1 - 1 of an unmasked chunk, free of branches:
                auto exp_block = [&](const int b, uint64_t C2, uint64_t negm2, uint64_t* lp) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = f2_get(f2_fma(f2(__uint_as_float(sv[32 * b + 2 * j]),
                                                          __uint_as_float(sv[32 * b + 2 * j + 1])), C2, negm2));
                        const float e0 = pc_ex2(x.x), e1 = pc_ex2(x.y);
                        lp[j & 3] = f2_add(lp[j & 3], f2(e0, e1));
                        pk[j] = pc_pack_bf16(e0, e1);
                    }
                    tmem_st16(t_s + 16u * b, pk);
                };
                auto exp_sum = [&](const uint64_t* lp) -> float {
                    const float2 ls = f2_get(f2_add(f2_add(lp[0], lp[1]), f2_add(lp[2], lp[3])));
                    return ls.x + ls.y;
                };
                auto exp_part = [&](const int b0, const int b1) -> float {
                    uint64_t lp[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int b = b0; b < b1; ++b) exp_block(b, f2(C, C), f2(-m, -m), lp);
                    return exp_sum(lp);
                };
                // and with masks (masked columns are -inf already), empty
                // blocks as zeros
                auto exp_masked = [&]() -> float {
                    const float negm = m == -INFINITY ? 0.f : -m;
                    uint64_t lp[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (b >= nblk) continue;
                        if (emptym & (1u << b)) {
                            uint32_t z[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j) z[j] = 0u;
                            tmem_st16(t_s + 16u * b, z);
                        } else {
                            exp_block(b, f2(C, C), f2(negm, negm), lp);
                        }
                    }
                    return exp_sum(lp);
                };
                float lsum = 0.f;
                if (fastp) {
                    // against the current m without a row max: every term is
                    // at most the row sum, so a sum within 2^8 keeps each
                    // inside the lazy bound; a larger one (rare) takes the
                    // exact max and recomputes if some row moved
#pragma unroll 1
                    for (int attempt = 0; attempt < 2; ++attempt) {
                        lsum = exp_part(0, 2);
                        tmem_wait_ld();                    // columns 64..127 (no-op when recomputing)
                        lsum += exp_part(2, 4);
                        if (attempt == 1 || !__any_sync(0xffffffffu, !(lsum <= 256.f))) break;
                        if (!raise_to(row_max())) break;   // first attempt stands
                        tmem_wait_st();                    // its P stores land before the new ones
                    }
                } else {
                    raise_to(row_max());
                    lsum = exp_masked();
                }
                l += lsum;
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(PC_P_FULL + t));
            }
            if (!alive) break;

            // ---- the next pair's queries, under this one's last products
            const int row0 = wk.row, info = wk.info;
            const int nrows = info >> 8, head = info >> 2 & 63;      // of this tile
            have = fetch(wk);
            if (have && !prepare_q(wk.pos0)) break;

            // ---- epilogue
            if (!__all_sync(0xffffffffu, mbar_wait(bar(PC_O_FULL + t), oph, abort_flag, status))) break;
            oph ^= 1;
            tc_fence_after();
            if (!(info & 2)) {
                // partial: m, l and O in FP32, channel quads outermost so that
                // the rows of a warp are consecutive
                tc_fence_before();
                if (4 * (warp & 3) >= nrows) continue;    // none of the warp's rows is a new token's
                float* dst = reinterpret_cast<float*>(p.ws + L.cpart) + (2 * (size_t)blockIdx.x + (info & 1 ? 0 : 1)) * kChunkPart;
                const int row = 128 * t + r;
                dst[row] = m;
                dst[256 + row] = l;
                float4* o4 = reinterpret_cast<float4*>(dst + 512) + row;
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    uint32_t v[32];
                    tmem_ld32(t_o + 32u * b, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o4[(size_t)(8 * b + j) * 256] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                                                    __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
                }
                tc_fence_before();
                continue;
            }
            float lse, scale;
            const int h = kGroup * head + hl;
            paged_finish(m, l, p.sinks[h], &scale, &lse);
            // Valid tokens of this warp's 4: rows behind the sequence's last
            // new token are other sequences' or nobody's
            const int wt0 = 4 * (warp & 3);
            const int nvw = max(0, min(4, nrows - wt0));
            const int sw = lane & 7;
#pragma unroll 1
            for (int hb = 0; hb < 2; ++hb) {
                uint32_t pk[32];
                {
                    uint32_t v[64];
                    tmem_ld32(t_o + 64u * hb, v);
                    tmem_ld32(t_o + 64u * hb + 32u, v + 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        pk[j] = pc_pack_bf16(__uint_as_float(v[2 * j]) * scale, __uint_as_float(v[2 * j + 1]) * scale);
                }
                // the staging block is free once lane 0's earlier stores have read it
                if (lane == 0) bulk_wait_group_read0();
                __syncwarp();
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4*>(stg + lane * 128 + ((x ^ sw) << 4)) =
                        make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && nvw > 0) {
                    if (nvw == 4) {
                        tma_store_3d(&tm_o, stg_s, 64 * hb, kGroup * head, row0 + wt0);
                    } else {
                        for (int k = 0; k < nvw; ++k)
                            tma_store_3d(&tm_o1, stg_s + 1024u * k, 64 * hb, kGroup * head, row0 + wt0 + k);
                    }
                    bulk_commit_group();
                }
            }
            if (tl < nrows && p.lse) p.lse[(size_t)h * c.T + row0 + tl] = lse;
            tc_fence_before();
        }
    }

    // ---------------------------------------------------------------- teardown
    if (warp >= 4 && warp < 12 && lane == 0) bulk_wait_group0();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Folds the partials of the pairs that several CTAs hold (in CTA order): block
// (x, y) what CTA x + 1's note says, rows 32 y .. 32 y + 31 (a lane a row, a
// warp eight channel quads).
__global__ void __launch_bounds__(128) paged_combine_kernel(const PagedAttnParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const PagedCache& c = p.c;
    const int nh = kGroup * c.ng;
    const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, p.chunk_ctas, p.stage_rows);
    const float* part = reinterpret_cast<const float*>(p.ws + L.cpart);
    griddep_wait();
    const PagedNote n = reinterpret_cast<const PagedNote*>(p.ws + L.notes)[blockIdx.x + 1];
    const int row = 32 * blockIdx.y + lane;
    if (!n.fold || 32 * (int)blockIdx.y >= n.rows) return;
    const PagedParts pp = n.parts;
    // two parts a round (most pairs have two), their loads all on their way
    // at once; the running max of a later round rescales what is there
    float M = -INFINITY, l = 0.f;
    float4 o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x = pp.cf; x <= pp.cl; x += 2) {
        const bool two = x + 1 <= pp.cl;
        const float* b0 = part + pp.slot(x) * kChunkPart;
        const float* b1 = two ? part + pp.slot(x + 1) * kChunkPart : b0;
        const float m0 = __ldcg(b0 + row), m1 = two ? __ldcg(b1 + row) : -INFINITY;
        const float l0 = __ldcg(b0 + 256 + row), l1 = two ? __ldcg(b1 + 256 + row) : 0.f;
        const float4* p0 = reinterpret_cast<const float4*>(b0 + 512) + (size_t)(8 * warp) * 256 + row;
        const float4* p1 = reinterpret_cast<const float4*>(b1 + 512) + (size_t)(8 * warp) * 256 + row;
        float4 v0[8], v1[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v0[j] = __ldcg(p0 + (size_t)j * 256);
            v1[j] = __ldcg(p1 + (size_t)j * 256);
        }
        const float Mn = fmaxf(M, fmaxf(m0, m1));
        const float ab = M > -INFINITY ? exp2f(M - Mn) : 0.f;
        const float a0 = m0 > -INFINITY ? exp2f(m0 - Mn) : 0.f, a1 = m1 > -INFINITY ? exp2f(m1 - Mn) : 0.f;
        M = Mn;
        l = l * ab + l0 * a0 + l1 * a1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            o[j].x = o[j].x * ab + v0[j].x * a0 + v1[j].x * a1;
            o[j].y = o[j].y * ab + v0[j].y * a0 + v1[j].y * a1;
            o[j].z = o[j].z * ab + v0[j].z * a0 + v1[j].z * a1;
            o[j].w = o[j].w * ab + v0[j].w * a0 + v1[j].w * a1;
        }
    }
    if (row >= n.rows) return;
    const int h = kGroup * n.head + (row & 7);
    float scale, lse;
    paged_finish(M, l, p.sinks[h], &scale, &lse);
    const size_t t = (size_t)(n.row + (row >> 3));
    uint4* dst = reinterpret_cast<uint4*>(p.out + (t * nh + h) * kHD + 32 * warp);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        dst[j] = make_uint4(pc_pack_bf16(o[2 * j].x * scale, o[2 * j].y * scale), pc_pack_bf16(o[2 * j].z * scale, o[2 * j].w * scale),
                            pc_pack_bf16(o[2 * j + 1].x * scale, o[2 * j + 1].y * scale),
                            pc_pack_bf16(o[2 * j + 1].z * scale, o[2 * j + 1].w * scale));
    if (warp == 0 && p.lse) p.lse[(size_t)h * c.T + t] = lse;
}

// ============================================================================ host
namespace {

// dims (128, d1, d2) of 16-bit elements, rows of 256 bytes, d1 rows a block of
// the outermost dimension; box (64, b1, b2), 128-byte swizzle.
flint_status_t pc_map(EncodeTiledFn enc, CUtensorMap* m, CUtensorMapDataType dt, const void* base, cuuint64_t d1,
                      cuuint64_t d2, cuuint32_t b1, cuuint32_t b2) {
    cuuint64_t dims[3] = {(cuuint64_t)kHD, d1, d2};
    cuuint64_t strides[2] = {(cuuint64_t)kHD * 2, d1 * kHD * 2};
    cuuint32_t box[3] = {64, b1, b2}, estr[3] = {1, 1, 1};
    const CUresult r = enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FLINT_ERR_CUDA, "cuTensorMapEncodeTiled (paged attention) failed (%d)", (int)r);
    return FLINT_OK;
}

template <PcSource SRC>
cudaError_t launch_chunk(const CUtensorMap* m, const PagedAttnParams& p, cudaStream_t s) {
    static bool set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!set[dev & 63]) {
        const cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<SRC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPcSmem);
        if (e != cudaSuccess) return e;
        set[dev & 63] = true;
    }
    // each launch a programmatic dependent of the one before it
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaSuccess;
    if (SRC == kPcStaged) {
        // a warp for 16 positions of a head, at most eight blocks an SM
        const int n = (p.c.B * (p.stage_rows / 16) * p.c.ng + kExpandThreads / 32 - 1) / (kExpandThreads / 32);
        cfg.gridDim = dim3(n < 8 * p.chunk_ctas ? n : 8 * p.chunk_ctas);
        cfg.blockDim = dim3(kExpandThreads);
        e = cudaLaunchKernelEx(&cfg, paged_expand_kernel, p);
        if (e != cudaSuccess) return e;
    }
    cfg.gridDim = dim3(p.chunk_ctas);
    cfg.blockDim = dim3(PcShape<SRC == kPcCodes>::threads);
    cfg.dynamicSmemBytes = kPcSmem;
    e = cudaLaunchKernelEx(&cfg, paged_chunk_kernel<SRC>, m[0], m[1], m[2], m[3], m[4], p);
    if (e != cudaSuccess || p.chunk_ctas < 2) return e;
    cfg.gridDim = dim3(p.chunk_ctas - 1, 8 * kChunkTok / 32);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, paged_combine_kernel, p);
}

}  // namespace

flint_status_t launch_paged_chunk(const PagedAttnParams& p, cudaStream_t s) {
    EncodeTiledFn enc = nullptr;
    flint_status_t st = get_encoder(&enc);
    if (st != FLINT_OK) return st;
    const PagedCache& c = p.c;
    const bool fp8 = p.k_scales != nullptr;
    const cuuint64_t nh = (cuuint64_t)kGroup * c.ng, ps = 1u << c.ps_log2, rows = (cuuint64_t)c.num_pages * c.ng;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap m[5];
    st = pc_map(enc, &m[0], bf, p.q, nh, c.T, kGroup, kTokPerTile);
    const CUtensorMapDataType f16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    if (p.stage_rows > 0) {
        const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, p.chunk_ctas, p.stage_rows);
        if (st == FLINT_OK) st = pc_map(enc, &m[1], f16, p.ws + L.stage_k, (cuuint64_t)c.B * p.stage_rows, c.ng, kKeyChunk, 1);
        if (st == FLINT_OK) st = pc_map(enc, &m[2], bf, p.ws + L.stage_v, (cuuint64_t)c.B * p.stage_rows, c.ng, kKeyChunk, 1);
    } else if (!fp8) {
        if (st == FLINT_OK) st = pc_map(enc, &m[1], f16, p.k_pages, ps, rows, (cuuint32_t)ps, 1);
        if (st == FLINT_OK) st = pc_map(enc, &m[2], bf, p.v_pages, ps, rows, (cuuint32_t)ps, 1);
    } else {
        m[1] = m[2] = m[0];                         // not used
    }
    if (st == FLINT_OK) st = pc_map(enc, &m[3], bf, p.out, nh, c.T, kGroup, 4);
    if (st == FLINT_OK) st = pc_map(enc, &m[4], bf, p.out, nh, c.T, kGroup, 1);
    if (st != FLINT_OK) return st;
    paged_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
    if (cudaGetLastError() != cudaSuccess) return fail(FLINT_ERR_CUDA, "paged attention launch: plan");
    const cudaError_t e = p.stage_rows > 0 ? launch_chunk<kPcStaged>(m, p, s)
                          : fp8            ? launch_chunk<kPcCodes>(m, p, s)
                                           : launch_chunk<kPcPages>(m, p, s);
    if (e != cudaSuccess) return fail(FLINT_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
    return FLINT_OK;
}

}  // namespace flint
