// Attention of few new tokens per sequence over paged keys and values.
//
// For new row i of sequence b at position p = len[b] + i and query head h of
// KV head g = h / 8 (FlintAttention.forward on the NeMo AutoModel
// "flint.layers" API page, restricted to the new rows):
//   z_j = q~ . K_j / sqrt(128) over max(0, p - W + 1) <= j <= p
//   out = sum e^{z_j} V_j / (e^sink + sum e^{z_j}),  lse = ln(e^sink + sum e^{z_j})
// with the learned sink as a zero-value column (HF discussion #26 on
// RecursiveSI/flint).
//
// A position's keys and values are read once per row group (up to NT new
// tokens x 8 query heads), 4 NT multiply-adds a byte: the kernel is bound by
// HBM.  So the matrix instructions are the warp-level ones
// (mma.m16n8k16): N = 8 is exactly a KV head's 8 query heads, and scores and
// outputs stay in registers, where a tcgen05 tile of 128 slots goes through
// tensor memory, barriers and four roles for the same 16 KFLOP a slot.
//
// * Work is the 64-position (8-bit pages: 128) tiles of all (group, head)
//   pairs in a row; CTA c takes tiles [W c / G, W (c + 1) / G), whatever
//   sequences they belong to, so every CTA streams the same number of bytes
//   for any mix of lengths.  Each CTA works its share out from the lengths
//   (no planning launch in front).  A (group, head) inside one CTA is written
//   at once; otherwise its CTAs leave partials (m, l, O), folded in CTA order
//   by the kernel behind (results do not depend on timing).  Folding by the
//   last CTA to finish, with counters cleared by a kernel in front, took 3 to
//   6 us a call longer.
// * A producer warp streams the tiles by TMA (three stages of 32 KiB, two CTAs
//   an SM), across the pairs of its share: interior tiles in boxes as tall as
//   a page and tile allow, a pair's edges in boxes of 16 slots, so that next
//   to nothing outside the window is read.  (Sixteen-byte cp.async copies by
//   the consuming lanes, with the products left out, took as long as with
//   them: 94 us for 450 MB, 4.8 TB/s.)  It also brings the next pair's
//   queries to L2 and copies the scales of 8-bit pages.
// * Four consumer warps take 16 (32) positions of each tile each; nothing but
//   a pair's end joins them.  Fragments come from the 128-byte-swizzled tiles
//   without bank conflicts:
//     K (A operand, 16 keys x 16 channels): lane (j, i) = (lane / 4,
//     lane % 4) reads 16-byte chunks 2 i and 2 i + 1 of each 128 bytes of
//     rows j and j + 8; the channel order that gives is used for q~ (B
//     operand) too.
//     V (A operand of O^T += V^T P^T, 16 channels x 16 keys): lane (j, i)
//     reads chunk j of rows 2 i, 2 i + 1, 2 i + 8, 2 i + 9 and interleaves
//     pairs of rows; rows of the product are the channels of its chunks.
// * S^T = K Q^T has the head pairs (2 i, 2 i + 1) of keys j and j + 8 in lane
//   (j, i): the softmax needs no exchange as long as the running max stands.
//   It is raised only when a score passes it by 2^8 (a vote a block).
//   movmatrix turns P^T into the next B operand.
// * q~ is FP16, as in the forward; P for BF16 values is split into high and
//   low parts (both multiplied), so its rounding does not show.  8-bit
//   values: the codes are exact in FP16 and the scale 2^e joins the exponent,
//   p' = 2^(z + e - m + 7), with m the running maximum of z + e, while l sums
//   p' 2^-e.  The 7 put the largest P' at 2^15, the top of FP16 (the lazy
//   maximum may be passed by 2^8): it keeps 11 bits down to 2^-21 of the
//   largest term, and what is less is off by 2^-32 of it at most, so that
//   tokens far below one with a large value scale still count.
// Every wait is bounded (FLINT_ERR_TIMEOUT in the status word).
//
// Measured: one token each of 2 sequences over 100,003 to 131,071 positions,
// 16-bit pages: 75 to 77 us for 450 MB, 6.0 TB/s, 0.91 of the measured copy rate (82 us
// with both launches); 128 sequences at a window of 513 37 us for 137 MB; 64
// sequences of up to 4,096 on 8-bit pages 40 us for 112 MB.  About 11 us of a
// call are its start (launch, lengths, page table, first tile) and the fold.
#include <cuda.h>
#include <cuda_runtime.h>

#include "flint_host.cuh"
#include "flint_paged_walk.cuh"
#include "sm100.cuh"

namespace flint {

flint_status_t launch_paged_chunk(const PagedAttnParams& p, cudaStream_t s);

constexpr int kStepWarps = 4;                            // consumer warps
// Threads: the consumers and the producer.  Two tokens a group (NT = 2) take
// more registers than two CTAs an SM leave each of 160 threads (168: they
// spill), so there the producer is a warpgroup of one busy warp that gives its
// registers to the consumers' (drafts of 2 to 6 tokens 55 us, 60 without; one
// token a group has no use for it: 36 us become 38).
template <int NT> struct StepShape {
    static constexpr int threads = 32 * kStepWarps + (NT == 1 ? 32 : 128);
    static constexpr uint32_t producer = 56, consumer = 200;
};
static_assert(128 * 56 + 128 * 200 <= 256 * 128, "register split");
constexpr uint32_t kStepStages = 3;
constexpr uint32_t kStepHalf = 16384;                    // a tile's keys, or values
constexpr uint32_t kStepStage = 2 * kStepHalf;
constexpr int kStepCtasPerSm = 2;
// Scores of 8-bit values are held 2^7 above the running maximum's unit.
template <bool FP8> constexpr float kStepLift = FP8 ? 7.f : 0.f;

// Positions of a warp's block and of a tile; 16-position pieces of a tile.
template <bool FP8> struct StepTile {
    static constexpr int block = FP8 ? 32 : 16, tile = block * kStepWarps, pieces = tile / 16;
};

// ---------------------------------------------------------------- step kernel
__device__ __forceinline__ float st_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
    return r;
}
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t reg4(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

struct StepPlanSmem { long long scan[8]; int at[4]; };
template <int NT>
struct StepSmem {
    static constexpr int rows = 8 * NT;
    static constexpr uint32_t ring = 0;                                                // K, V of a tile; stages
    static constexpr uint32_t scales = kStepStages * kStepStage;                       // 8 pieces x (K, V) x 16 bytes a stage
    static constexpr uint32_t q = scales + kStepStages * 256;                          // q~ in FP16
    static constexpr uint32_t ml = q + rows * kHD * 2;                                 // [warp][rows] m, then l
    static constexpr uint32_t plan = ml;                                               // the plan's, before the pairs
    static constexpr uint32_t fin = ml + 2 * kStepWarps * rows * 4;                    // [rows] output scale
    static constexpr uint32_t inv = (fin + rows * 4 + 15) / 16 * 16;                   // rotation frequencies
    static constexpr uint32_t w = inv + 64 * 8;                                        // q_norm weight
    static constexpr uint32_t sink = w + kHD * 4;                                      // the learned sinks
    static constexpr uint32_t bar = sink + kHQ * 4;                                    // full, empty, consumers, test
    static constexpr uint32_t misc = bar + 8 * 8;                                      // abort flag, CTA status
    static constexpr uint32_t total = misc + 16 + 1024;                                // and alignment slack
    // the warps' parts of a pair meet in the stage read last
    static_assert(kStepWarps * rows * kHD * 4 <= kStepStage, "the warps' outputs fit a stage");
    static_assert(plan >= kStepStages * kStepStage && plan % 8 == 0 && sizeof(StepPlanSmem) <= fin - plan,
                  "plain accesses only: the plan stays off what TMA writes");
};
static_assert(2 * (StepSmem<2>::total + 1024) <= 233472, "two CTAs share an SM");
// ST_TEST: nothing arrives here, the timeout test hook waits on it
enum : uint32_t { ST_FULL = 0, ST_EMPTY = 3, ST_CONS = 6, ST_TEST = 7 };

// The share of CTA `cta` of `ctas`; *W, *G: tiles of all pairs, CTAs that
// share them; *bad: ill-formed boundaries or lengths.  Every thread of the
// block calls it; false: no share.
template <int NT>
__device__ bool step_plan(const PagedAttnParams& p, int tile, int cta, int ctas, StepPlanSmem* sm, StepWalk& w, long long* W,
                          long long* G, bool* bad) {
    const PagedCache& c = p.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // a run of sequences a thread
    constexpr int kThreads = StepShape<NT>::threads;
    const int per = (c.B + kThreads - 1) / kThreads, b0 = min(tid * per, c.B), b1 = min(b0 + per, c.B);
    bool ill = false;
    long long sum = 0;
    if (b0 < b1) {
        int a = paged_ld(c.cu + b0);
        if (b0 == 0) ill = a != 0;
        for (int b = b0; b < b1; ++b) {
            const int len = paged_ld(c.len + b), z = paged_ld(c.cu + b + 1);
            sum += step_seq_tiles<NT>(p, a, z, len, tile, &ill);   // a last boundary past T as well
            a = z;
        }
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) sm->scan[warp] = inc;
    *bad = __syncthreads_or(ill);
    long long before = inc - sum, total = 0;
#pragma unroll
    for (int x = 0; x < kThreads / 32; ++x) {
        if (x < warp) before += sm->scan[x];
        total += sm->scan[x];
    }
    *W = total * c.ng;
    *G = *W < (long long)ctas ? *W : (long long)ctas;
    if (cta >= *G) return false;
    const long long t = *W * cta / *G, end = *W * (cta + 1) / *G;
    if (t >= before * c.ng && t < (before + sum) * c.ng) {
        // the share begins in this thread's run
        step_place<NT>(p, b0, b1, t - before * c.ng, tile, sm->at);
    }
    __syncthreads();
    step_begin(p, w, sm->at, (int)(end - t), *bad);
    return true;
}

// Maps of the pools: k, v in boxes of min(page, tile) slots; k16, v16 of 16.
struct StepMaps { CUtensorMap k, v, k16, v16; };

template <int NT, bool FP8>
__global__ void __launch_bounds__(StepShape<NT>::threads, kStepCtasPerSm)
paged_step_kernel(const __grid_constant__ StepMaps maps, const PagedAttnParams p) {
    using S = StepSmem<NT>;
    using TL = StepTile<FP8>;
    constexpr int kSub = FP8 ? 2 : 1;                    // 16-position parts of a warp's block
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = lane >> 2, i = lane & 3;
    const PagedCache& c = p.c;
    const int ng = c.ng, nh = kGroup * ng;
    const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, 0, 0);
    float* part = reinterpret_cast<float*>(p.ws + L.spart);
    PagedNote* note = reinterpret_cast<PagedNote*>(p.ws + L.notes) + blockIdx.x;
    float* s_m = reinterpret_cast<float*>(smem + S::ml);
    float* s_l = s_m + kStepWarps * S::rows;
    float* s_fin = reinterpret_cast<float*>(smem + S::fin);
    float* s_w = reinterpret_cast<float*>(smem + S::w);
    float* s_sink = reinterpret_cast<float*>(smem + S::sink);
    double* s_inv = reinterpret_cast<double*>(smem + S::inv);
    volatile int* abort_flag = reinterpret_cast<int*>(smem + S::misc);
    int* s_status = reinterpret_cast<int*>(smem + S::misc) + 1;
    auto bar = [&](uint32_t x) { return sb + S::bar + 8 * x; };

    griddep_launch_dependents();                         // the fold kernel, which waits for this one
    StepWalk walk;
    long long W, G;
    bool bad;
    const bool work = step_plan<NT>(p, TL::tile, blockIdx.x, gridDim.x, reinterpret_cast<StepPlanSmem*>(smem + S::plan), walk, &W, &G, &bad);
    if (!work) {
        if (tid == 0) *note = PagedNote{bad ? kStatusInvalid : kStatusOk};
        return;
    }
    if (tid == 0) {
        // a whole note first: the fold kernel reads it even where a wait ran
        // out before the first pair, and the workspace holds anything
        *note = PagedNote{};
        for (uint32_t x = 0; x < kStepStages; ++x) {
            mbar_init(bar(ST_FULL + x), 1);
            mbar_init(bar(ST_EMPTY + x), kStepWarps);
        }
        mbar_init(bar(ST_CONS), 32 * kStepWarps);
        mbar_init(bar(ST_TEST), 1);
        *abort_flag = 0;
        *s_status = bad ? kStatusInvalid : kStatusOk;
        fence_mbar_init();
    }
    __syncthreads();                                     // the barriers are set, the plan's memory is read
    auto see = [&](const StepSeg& g, int* lo, int* hi) {
        *lo = p.window > 0 ? max(0, g.p0 - p.window + 1) : 0;
        *hi = g.p0 + g.nrows;
    };

    if (warp >= kStepWarps) {
        // ============================================================ producer (a whole warp)
        if constexpr (NT > 1) {
            regs_dec<StepShape<NT>::producer>();
            if (warp > kStepWarps) {
                __syncthreads();
                return;
            }
        }
        // Lane l < pieces holds piece l (16 positions) of a tile: its page, and
        // for 8-bit pages its scales, both fetched ahead.
        struct Tile { int key, lo, hi, head, page; bool any; };
        const int box = min(1 << c.ps_log2, TL::tile), slot_mask = (1 << c.ps_log2) - 1;
        constexpr uint32_t kPiece = FP8 ? 2048 : 4096;   // bytes of a piece's keys, or values
        int left = 0, key = 0, lo = 0, hi = 0, head = 0;
        const int* table = nullptr;
        auto next_tile = [&]() -> Tile {
            Tile t = {};
            if (left == 0) {
                StepSeg sg;
                if (!step_next<NT>(p, walk, sg, TL::tile)) return t;
                see(sg, &lo, &hi);
                left = sg.t1 - sg.t0;
                head = sg.head;
                key = step_base(p, lo, TL::tile) + sg.t0 * TL::tile;
                table = c.table + (size_t)sg.b * c.max_pages;
                if (lane < sg.nrows) bulk_prefetch_l2(p.q + ((size_t)(sg.row + lane) * nh + kGroup * head) * kHD, kGroup * kHD * 2);
            }
            t.any = true;
            t.key = key;
            t.lo = lo;
            t.hi = hi;
            t.head = head;
            const int k = key + 16 * lane;
            t.page = lane < TL::pieces && k < hi && k + 16 > lo ? max(__ldg(table + (k >> c.ps_log2)), -1) : -2;
            key += TL::tile;
            --left;
            return t;
        };
        auto row_of = [&](const Tile& t) -> long long {   // pool row of the lane's piece, -1 where it has none
            if (t.page < 0 || t.page >= c.num_pages) return -1;
            return (long long)paged_row(c, t.page, t.head, (t.key + 16 * lane) & slot_mask);
        };
        uint4 ks = {}, vs = {};
        auto load_scales = [&](const Tile& t) {
            const long long r = t.any ? row_of(t) : -1;
            if (FP8 && r >= 0) {
                ks = __ldg(reinterpret_cast<const uint4*>(p.k_scales + r));
                vs = __ldg(reinterpret_cast<const uint4*>(p.v_scales + r));
            }
        };
        Tile cur = next_tile(), nxt = next_tile();
        load_scales(cur);
        uint32_t st = 0, ph = 0, n = 0;
        while (cur.any) {
            const uint4 k0 = ks, v0 = vs;
            load_scales(nxt);
            const Tile after = next_tile();
            if (!__all_sync(0xffffffffu, mbar_wait(bar(ST_EMPTY + st), ph ^ 1, abort_flag, s_status))) break;
            const bool live = row_of(cur) >= 0;
            if (!live && cur.page != -2) *s_status = kStatusInvalid;
            if (FP8 && live) {
                uint4* d = reinterpret_cast<uint4*>(smem + S::scales + st * 256) + 2 * lane;
                d[0] = k0;
                d[1] = v0;
            }
            const uint32_t bytes = 2 * kPiece * __popc(__ballot_sync(0xffffffffu, live));
            __syncwarp();
            if (lane == 0) mbar_expect_tx(bar(ST_FULL + st), bytes);
            __syncwarp();
            const uint32_t dst = sb + S::ring + st * kStepStage + lane * 2048;
            const int slot = (cur.key + 16 * lane) & slot_mask, z = cur.page * ng + cur.head;
            const bool inside = cur.key >= cur.lo && cur.key + TL::tile <= cur.hi;   // every row of the tile is seen
            if (inside ? live && (16 * lane & (box - 1)) == 0 : live) {
                const CUtensorMap* mk = inside ? &maps.k : &maps.k16;
                const CUtensorMap* mv = inside ? &maps.v : &maps.v16;
                if constexpr (FP8) {
                    tma_load_3d(dst, mk, bar(ST_FULL + st), 0, slot, z);
                    tma_load_3d(dst + kStepHalf, mv, bar(ST_FULL + st), 0, slot, z);
                } else {
                    // the channel halves of a tile are 8 KiB apart
                    tma_load_3d(dst, mk, bar(ST_FULL + st), 0, slot, z);
                    tma_load_3d(dst + kStepHalf / 2, mk, bar(ST_FULL + st), 64, slot, z);
                    tma_load_3d(dst + kStepHalf, mv, bar(ST_FULL + st), 0, slot, z);
                    tma_load_3d(dst + kStepHalf + kStepHalf / 2, mv, bar(ST_FULL + st), 64, slot, z);
                }
            }
            ++n;
            if (++st == kStepStages) { st = 0; ph ^= 1; }
            cur = nxt;
            nxt = after;
        }
        // every armed load has landed before shared memory is released
        volatile int never = 0;
        for (uint32_t x = 0; x < kStepStages; ++x) {
            const uint32_t nl = (n + kStepStages - 1 - x) / kStepStages;     // loads number x, x + 3, ..
            if (nl) mbar_wait(bar(ST_FULL + x), (nl - 1) & 1, &never, nullptr, 100ull * 1000ull * 1000ull);
        }
        __syncthreads();
        if (lane == 0) note->status = *reinterpret_cast<volatile int*>(s_status);
        return;
    }

    // ================================================================ consumers
    // (their constants are fetched while the first tiles are on their way)
    if constexpr (NT > 1) regs_inc<StepShape<NT>::consumer>();
    const int eq = prescale_exponent(warp_max_abs128(p.q_norm_w));
    const float C = ldexpf(1.4426950408889634f * 0.08838834764831845f, -eq);   // log2(e) / sqrt(128)
    const float qscale = ldexpf(1.f, eq);
    s_w[tid] = p.q_norm_w[tid];
    if (tid < nh) s_sink[tid] = p.sinks[tid];
    if (p.use_rope && tid < 64) s_inv[tid] = exp2(-(double)tid / 64.0 * log2((double)p.rope_theta));
    uint32_t cph = 0, stage = 0, fph = 0;
    auto csync = [&]() -> bool {                         // a bounded barrier of the consumer warps
        mbar_arrive(bar(ST_CONS));
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(ST_CONS), cph, abort_flag, s_status));
        cph ^= 1;
        return ok;
    };
    StepSeg sg;
    bool alive = (p.test_wait_ns == 0 || mbar_wait(bar(ST_TEST), 0, abort_flag, s_status, p.test_wait_ns)) && csync();
    for (bool first = true; alive && step_next<NT>(p, walk, sg, TL::tile); first = false) {
        const int head = sg.head, p0 = sg.p0, nrows = sg.nrows;
        int lo, hi;
        see(sg, &lo, &hi);
        if (first && tid == 0 && sg.t0 > 0) {
            // a pair that the share begins inside of is held in part by the
            // CTAs before, too: the first CTA of those leaves the fold a note
            const PagedParts parts = paged_parts(W, G, W * blockIdx.x / G - sg.t0, sg.tiles);
            note->fold = parts.cf == (int)blockIdx.x - 1;
            note->parts = parts;
            note->row = sg.row;
            note->head = head;
            note->rows = kGroup * nrows;
        }

        // ---- q~ of the group's rows: warp w takes heads 4 (w % 2) .. + 3 of row w / 2
        if (warp < 2 * NT) {
            const int nt = warp >> 1, sub = lane & 7, hh = 4 * (warp & 1) + (lane >> 3);
            const bool have = nt < nrows;
            const int pos = p0 + (have ? nt : 0);
            const __nv_bfloat16* src = p.q + ((size_t)(sg.row + (have ? nt : 0)) * nh + kGroup * head + hh) * kHD;
            const uint4 a = *reinterpret_cast<const uint4*>(src + 8 * sub);
            const uint4 b = *reinterpret_cast<const uint4*>(src + 64 + 8 * sub);
            float x0[8], x1[8], ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t aw = reg4(a, e >> 1), bw = reg4(b, e >> 1);
                x0[e] = (e & 1) ? __uint_as_float(aw & 0xffff0000u) : __uint_as_float(aw << 16);
                x1[e] = (e & 1) ? __uint_as_float(bw & 0xffff0000u) : __uint_as_float(bw << 16);
                ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
            }
            ss += __shfl_xor_sync(0xffffffffu, ss, 1);
            ss += __shfl_xor_sync(0xffffffffu, ss, 2);
            ss += __shfl_xor_sync(0xffffffffu, ss, 4);
            const float rn = qscale * rsqrtf(ss * (1.f / kHD) + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x0[e] *= rn * s_w[8 * sub + e];
                x1[e] *= rn * s_w[64 + 8 * sub + e];
            }
            if (p.use_rope) {
                float c0, s0, c1, s1;
                rope_cos_sin(pos, s_inv[2 * lane], &c0, &s0);
                rope_cos_sin(pos, s_inv[2 * lane + 1], &c1, &s1);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int f = 8 * sub + e;
                    const float cc = __shfl_sync(0xffffffffu, (e & 1) ? c1 : c0, f >> 1);
                    const float sn = __shfl_sync(0xffffffffu, (e & 1) ? s1 : s0, f >> 1);
                    const float y0 = x0[e] * cc - x1[e] * sn, y1 = x1[e] * cc + x0[e] * sn;
                    x0[e] = y0;
                    x1[e] = y1;
                }
            }
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                h[e] = have ? pack2_f16(x0[2 * e], x0[2 * e + 1]) : 0u;
                h[4 + e] = have ? pack2_f16(x1[2 * e], x1[2 * e + 1]) : 0u;
            }
            uint8_t* qd = smem + S::q + ((nt * kGroup + hh) * kHD + 8 * sub) * 2;
            *reinterpret_cast<uint4*>(qd) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(qd + 128) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        if (!csync()) break;
        // B fragments of q~ (head j, the lane's channels)
        uint32_t qf[NT][16];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                // 16-bit: chunk 2 i + x % 2 of half x / 2; 8-bit: the x % 2 half of chunk 2 i + x / 2
                const int ch = FP8 ? (2 * i + (x >> 1)) * 16 + (x & 1) * 8 : (x >> 1) * 64 + (2 * i + (x & 1)) * 8;
                const uint4 v = lds16(sb + S::q + ((nt * kGroup + j) * kHD + ch) * 2);
                qf[nt][4 * x] = v.x;
                qf[nt][4 * x + 1] = v.y;
                qf[nt][4 * x + 2] = v.z;
                qf[nt][4 * x + 3] = v.w;
            }

        // ---- the stream
        float acc[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 8; ++x) acc[nt][x][0] = acc[nt][x][1] = acc[nt][x][2] = acc[nt][x][3] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }
        int key0 = step_base(p, lo, TL::tile) + sg.t0 * TL::tile + warp * TL::block;
        for (int it = sg.t0; it < sg.t1; ++it, key0 += TL::tile) {
            if (!__all_sync(0xffffffffu, mbar_wait(bar(ST_FULL + stage), fph, abort_flag, s_status))) { alive = false; break; }
            const uint32_t src = sb + S::ring + stage * kStepStage + warp * TL::block * 128;
            const uint8_t* ssc = smem + S::scales + stage * 256 + warp * kSub * 32;
            // the last tile's stage is given back at the pair's end
            auto release = [&]() {
                if (it + 1 == sg.t1) return;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(ST_EMPTY + stage));
                if (++stage == kStepStages) { stage = 0; fph ^= 1; }
            };
            if (key0 >= hi || key0 + TL::block <= lo) {
                release();
                continue;
            }
            // byte offset of 16-byte chunk x of row r of the warp's rows
            auto at = [&](int r, int x) -> uint32_t { return src + r * 128 + ((x ^ (r & 7)) << 4); };
            // scores: s[u][nt][0..3] = (key j, heads 2i, 2i + 1), (key j + 8, the same)
            float s[kSub][NT][4];
            float ev[kSub][2];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                float s2[NT][4];                          // two chains of products
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[u][nt][e] = s2[nt][e] = 0.f;
                if constexpr (!FP8) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t k = at(j, 2 * i + (x & 1)) + (x >> 1) * (kStepHalf / 2);
                        const uint4 a = lds16(k), b = lds16(k + 1024);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(s[u][nt], a.x, b.x, a.y, b.y, qf[nt][4 * x], qf[nt][4 * x + 1]);
                            mma_f16(s2[nt], a.z, b.z, a.w, b.w, qf[nt][4 * x + 2], qf[nt][4 * x + 3]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[u][nt][e] = (s[u][nt][e] + s2[nt][e]) * C;
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t k = at(j, 2 * i + x) + u * 2048;
                        const uint4 a = lds16(k), b = lds16(k + 1024);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t aw = reg4(a, r), bw = reg4(b, r);
                            const uint32_t a0 = e4m3_f16(aw), a2 = e4m3_f16(aw >> 16);
                            const uint32_t a1 = e4m3_f16(bw), a3 = e4m3_f16(bw >> 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16((r & 1) ? s2[nt] : s[u][nt], a0, a1, a2, a3, qf[nt][8 * x + 2 * r], qf[nt][8 * x + 2 * r + 1]);
                        }
                    }
                    const float k0 = paged_scale(ssc[u * 32 + j]) * C, k1 = paged_scale(ssc[u * 32 + j + 8]) * C;
                    ev[u][0] = (float)((int)ssc[u * 32 + 16 + j] - 127);
                    ev[u][1] = (float)((int)ssc[u * 32 + 24 + j] - 127);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[u][nt][e] = fmaf(s[u][nt][e] + s2[nt][e], e < 2 ? k0 : k1, ev[u][e >> 1]);
                }
            }
            // masks: only where some row does not see the whole block
            const bool edge = key0 < lo || key0 + TL::block > p0 + 1 || (p.window > 0 && key0 < hi - p.window);
            if (edge) {
#pragma unroll
                for (int u = 0; u < kSub; ++u) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const int pos = p0 + nt, wl = p.window > 0 ? max(0, pos - p.window + 1) : 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int k = key0 + 16 * u + j + (e >> 1) * 8;
                            if (k > pos || k < wl) s[u][nt][e] = -INFINITY;
                        }
                    }
                    // slots that hold no key of this call have any scale
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = key0 + 16 * u + j + 8 * e;
                        if (k < lo || k >= hi) ev[u][e] = 0.f;
                    }
                }
            }
            // values in slots that hold no key: anything, NaN included
            auto drop = [&](uint4& v0, uint4& v1, uint4& v2, uint4& v3, int u) {
                const int k = key0 + 16 * u + 2 * i;
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                if (k < lo || k >= hi) v0 = z;
                if (k + 1 < lo || k + 1 >= hi) v1 = z;
                if (k + 8 < lo || k + 8 >= hi) v2 = z;
                if (k + 9 < lo || k + 9 >= hi) v3 = z;
            };
            // raise the running max where a score passes it by 2^8
            bool up = false;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) up = up || fmaxf(s[u][nt][e], s[u][nt][2 + e]) > m[nt][e] + 8.f;
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float mx = fmaxf(s[0][nt][h], s[0][nt][2 + h]);
                        if (kSub == 2) mx = fmaxf(mx, fmaxf(s[kSub - 1][nt][h], s[kSub - 1][nt][2 + h]));
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const float mn = fmaxf(m[nt][h], mx);
                        const float al = m[nt][h] > -INFINITY ? st_ex2(m[nt][h] - mn) : 0.f;
                        m[nt][h] = mn;
                        l[nt][h] *= al;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            acc[nt][x][h] *= al;
                            acc[nt][x][2 + h] *= al;
                        }
                    }
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float pr[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mm = m[nt][e & 1];
                        pr[e] = st_ex2(s[u][nt][e] - (mm > -INFINITY ? mm - kStepLift<FP8> : 0.f));
                    }
                    if constexpr (!FP8) {
                        l[nt][0] += pr[0] + pr[2];
                        l[nt][1] += pr[1] + pr[3];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t h = pack2_bf16(pr[2 * e], pr[2 * e + 1]);
                            ph[nt][e] = transpose8(h);
                            pl[nt][e] = transpose8(pack2_bf16(pr[2 * e] - __uint_as_float(h << 16),
                                                              pr[2 * e + 1] - __uint_as_float(h & 0xffff0000u)));
                        }
                    } else {
                        // l in units of 2^m: the scale's exponent taken back
                        const float i0 = __uint_as_float((uint32_t)(127 - (int)ev[u][0]) << 23);
                        const float i1 = __uint_as_float((uint32_t)(127 - (int)ev[u][1]) << 23);
                        l[nt][0] += pr[0] * i0 + pr[2] * i1;
                        l[nt][1] += pr[1] * i0 + pr[3] * i1;
                        ph[nt][0] = transpose8(pack2_f16(pr[0], pr[1]));
                        ph[nt][1] = transpose8(pack2_f16(pr[2], pr[3]));
                    }
                }
                if constexpr (!FP8) {
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint32_t va = at(2 * i, j) + kStepHalf + hh * (kStepHalf / 2), vb = at(2 * i + 1, j) + kStepHalf + hh * (kStepHalf / 2);
                        uint4 v0 = lds16(va), v1 = lds16(vb), v2 = lds16(va + 1024), v3 = lds16(vb + 1024);
                        if (edge) drop(v0, v1, v2, v3, u);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t a0 = __byte_perm(reg4(v0, r), reg4(v1, r), 0x5410);
                            const uint32_t a1 = __byte_perm(reg4(v0, r), reg4(v1, r), 0x7632);
                            const uint32_t a2 = __byte_perm(reg4(v2, r), reg4(v3, r), 0x5410);
                            const uint32_t a3 = __byte_perm(reg4(v2, r), reg4(v3, r), 0x7632);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_bf16(acc[nt][hh * 4 + r], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                                mma_bf16(acc[nt][hh * 4 + r], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
                            }
                        }
                    }
                } else {
                    const uint32_t va = at(2 * i, j) + kStepHalf + u * 2048, vb = at(2 * i + 1, j) + kStepHalf + u * 2048;
                    uint4 v0 = lds16(va), v1 = lds16(vb), v2 = lds16(va + 1024), v3 = lds16(vb + 1024);
                    if (edge) drop(v0, v1, v2, v3, u);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t x0 = __byte_perm(reg4(v0, r), reg4(v1, r), 0x5140);
                        const uint32_t x1 = __byte_perm(reg4(v0, r), reg4(v1, r), 0x7362);
                        const uint32_t y0 = __byte_perm(reg4(v2, r), reg4(v3, r), 0x5140);
                        const uint32_t y1 = __byte_perm(reg4(v2, r), reg4(v3, r), 0x7362);
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const uint32_t xx = hf ? x1 : x0, yy = hf ? y1 : y0;
                            const uint32_t a0 = e4m3_f16(xx), a1 = e4m3_f16(xx >> 16);
                            const uint32_t a2 = e4m3_f16(yy), a3 = e4m3_f16(yy >> 16);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_f16(acc[nt][2 * r + hf], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                        }
                    }
                }
            }
            release();
        }
        if (!alive) break;

        // ---- the four warps' states into one, in warp order, in the stage
        // they read last (the tiles on their way are in the others)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], o);
                m[nt][h] -= kStepLift<FP8>;                // l and acc are in units of 2^m again
                if (j == 0) {
                    s_m[warp * S::rows + nt * kGroup + 2 * i + h] = m[nt][h];
                    s_l[warp * S::rows + nt * kGroup + 2 * i + h] = l[nt][h];
                }
            }
        if (!csync()) break;
        float* bufs = reinterpret_cast<float*>(smem + S::ring + stage * kStepStage);
        constexpr int kBufStep = S::rows * kHD;
        float* buf = bufs + warp * kBufStep;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = nt * kGroup + 2 * i + h;
                float M = s_m[row];
#pragma unroll
                for (int w = 1; w < kStepWarps; ++w) M = fmaxf(M, s_m[w * S::rows + row]);
                const float a = m[nt][h] > -INFINITY ? st_ex2(m[nt][h] - M) : 0.f;
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const int ch = FP8 ? 16 * j + 2 * x : (x >> 2) * 64 + 8 * j + 2 * (x & 3);
                    *reinterpret_cast<float2*>(buf + row * kHD + ch) = make_float2(acc[nt][x][h] * a, acc[nt][x][2 + h] * a);
                }
            }
        const int rows = kGroup * nrows;
        const size_t out_row = (size_t)sg.row;
        float* dst = part + (2 * (size_t)blockIdx.x + (first ? 0 : 1)) * kStepPart;   // where the pair is held in part
        if (tid < rows) {
            float M = s_m[tid], l4 = 0.f;
#pragma unroll
            for (int w = 1; w < kStepWarps; ++w) M = fmaxf(M, s_m[w * S::rows + tid]);
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) {
                const float mw = s_m[w * S::rows + tid];
                l4 += s_l[w * S::rows + tid] * (mw > -INFINITY ? st_ex2(mw - M) : 0.f);
            }
            if (sg.whole) {
                const int h = kGroup * head + (tid & 7);
                float v;
                paged_finish(M, l4, s_sink[h], &s_fin[tid], &v);
                if (p.lse) p.lse[(size_t)h * c.T + out_row + (tid >> 3)] = v;
            } else {
                dst[tid] = M;
                dst[kPagedStepRows + tid] = l4;
            }
        }
        if (!csync()) break;
        // warp w: rows w, w + 4, ..; a lane four channels
#pragma unroll
        for (int r0 = 0; r0 < S::rows; r0 += kStepWarps) {
            const int r = r0 + warp;
            if (r >= rows) break;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kStepWarps; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(bufs + w * kBufStep + r * kHD + 4 * lane);
                o.x += v.x;
                o.y += v.y;
                o.z += v.z;
                o.w += v.w;
            }
            if (sg.whole) {
                const float sc = s_fin[r];
                *reinterpret_cast<uint2*>(p.out + ((out_row + (r >> 3)) * nh + kGroup * head + (r & 7)) * kHD + 4 * lane) =
                    make_uint2(pack2_bf16(o.x * sc, o.y * sc), pack2_bf16(o.z * sc, o.w * sc));
            } else {
                *reinterpret_cast<float4*>(dst + 2 * kPagedStepRows + r * kHD + 4 * lane) = o;
            }
        }
        // the parts are read: the stage goes back (the producer's copies into
        // it follow these generic accesses)
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(ST_EMPTY + stage));
        if (++stage == kStepStages) { stage = 0; fph ^= 1; }
    }
    __syncthreads();                                     // the producer records the CTA's status
}

// Folds the parts of the pairs that several CTAs hold, in CTA order: block
// (x, y) what CTA x + 1's note says, rows 8 y .. 8 y + 7.  A warp takes a row, a
// lane four channels and every 32nd CTA's weight.  Block (0, 0) also collects
// the CTAs' statuses.
constexpr int kFoldThreads = 256;
__global__ void __launch_bounds__(kFoldThreads, 2) paged_fold_kernel(const PagedAttnParams p) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const PagedCache& c = p.c;
    const int nh = kGroup * c.ng;
    const PagedWs L = paged_ws(c.B, c.T, c.ng, p.step_ctas, 0, 0);
    const PagedNote* notes = reinterpret_cast<const PagedNote*>(p.ws + L.notes);
    const float* part = reinterpret_cast<const float*>(p.ws + L.spart);
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        int any = kStatusOk;
        for (int x = tid; x < p.step_ctas; x += kFoldThreads) any = max(any, notes[x].status);
        const bool timeout = __syncthreads_or(any == kStatusTimeout), invalid = __syncthreads_or(any != kStatusOk);
        if (tid == 0) *reinterpret_cast<int*>(p.ws + L.header) = timeout ? kStatusTimeout : invalid ? kStatusInvalid : kStatusOk;
    }
    if ((int)blockIdx.x + 1 >= p.step_ctas) return;
    const PagedNote n = notes[blockIdx.x + 1];
    const int r = (kFoldThreads / 32) * blockIdx.y + warp;    // the warp's row
    if (!n.fold || r >= n.rows) return;
    const PagedParts pp = n.parts;
    // thirty-two parts a round, their weights a lane each; the running max
    // (rounds after the first) rescales what is there
    float M = -INFINITY, lsum = 0.f;
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = pp.cf; x0 <= pp.cl; x0 += 32) {
        const int xl = min(x0 + lane, pp.cl), cnt = min(32, pp.cl - x0 + 1);
        const float mx = __ldcg(part + pp.slot(xl) * kStepPart + r);
        const float lx = __ldcg(part + pp.slot(xl) * kStepPart + kPagedStepRows + r);
        float4 v[16];                                        // sixteen parts on their way at once
        auto load = [&](int k0) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
                if (k0 + k < cnt)
                    v[k] = __ldcg(reinterpret_cast<const float4*>(part + pp.slot(x0 + k0 + k) * kStepPart +
                                                                  2 * kPagedStepRows + r * kHD) + lane);
        };
        load(0);
        float Mn = fmaxf(M, mx);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Mn = fmaxf(Mn, __shfl_xor_sync(0xffffffffu, Mn, o));
        const float back = M > -INFINITY ? exp2f(M - Mn) : 0.f;
        M = Mn;
        lsum *= back;
        o4.x *= back;
        o4.y *= back;
        o4.z *= back;
        o4.w *= back;
        const float a = mx > -INFINITY && lane < cnt ? exp2f(mx - M) : 0.f;
        lsum += lx * a;
        for (int k0 = 0; k0 < cnt; k0 += 16) {
            if (k0) load(k0);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const float ak = __shfl_sync(0xffffffffu, a, k0 + k);
                if (k0 + k < cnt) {
                    o4.x += v[k].x * ak;
                    o4.y += v[k].y * ak;
                    o4.z += v[k].z * ak;
                    o4.w += v[k].w * ak;
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
    const int h = kGroup * n.head + (r & 7);
    const size_t row = (size_t)n.row + (r >> 3);
    float sc, v;
    paged_finish(M, lsum, p.sinks[h], &sc, &v);
    *reinterpret_cast<uint2*>(p.out + (row * nh + h) * kHD + 4 * lane) =
        make_uint2(pack2_bf16(o4.x * sc, o4.y * sc), pack2_bf16(o4.z * sc, o4.w * sc));
    if (lane == 0 && p.lse) p.lse[(size_t)h * c.T + row] = v;
}

// ============================================================================ host
namespace {

// dims (128, ps, rows) of 16-bit elements, or codes; box (128 bytes, slots, 1),
// 128-byte swizzle.
flint_status_t step_map(EncodeTiledFn enc, CUtensorMap* m, CUtensorMapDataType dt, int bytes, const void* base, cuuint64_t ps,
                        cuuint64_t rows, int slots) {
    cuuint64_t dims[3] = {(cuuint64_t)kHD, ps, rows};
    cuuint64_t strides[2] = {(cuuint64_t)kHD * bytes, ps * kHD * bytes};
    cuuint32_t box[3] = {(cuuint32_t)(128 / bytes), (cuuint32_t)slots, 1}, estr[3] = {1, 1, 1};
    const CUresult r = enc(m, dt, 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(FLINT_ERR_CUDA, "cuTensorMapEncodeTiled (paged step) failed (%d)", (int)r);
    return FLINT_OK;
}

template <int NT, bool FP8>
cudaError_t launch_step(const StepMaps& maps, const PagedAttnParams& p, cudaStream_t s) {
    static bool set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (!set[dev & 63]) {
        const cudaError_t e = cudaFuncSetAttribute(paged_step_kernel<NT, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (int)StepSmem<NT>::total);
        if (e != cudaSuccess) return e;
        set[dev & 63] = true;
    }
    paged_step_kernel<NT, FP8><<<p.step_ctas, StepShape<NT>::threads, StepSmem<NT>::total, s>>>(maps, p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.step_ctas > 1 ? p.step_ctas - 1 : 1, kGroup * NT / (kFoldThreads / 32));
    cfg.blockDim = dim3(kFoldThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_fold_kernel, p);
}

// Calls whose sequences all have at most this many new tokens run the step
// kernel, others the chunk kernel: the step kernel reads a sequence's keys and
// values once per two tokens, the chunk kernel once per 32 but with more to set
// up.  Measured, 16 sequences on two heads over 700 to 16,383 positions, step /
// chunk: 9 tokens 98 / 75 us, 12 117 / 73, 16 150 / 75 (8-bit pages: 9 88 / 97,
// 16 125 / 97); 25 sequences of 4 to 9 tokens over none 20 / 26.
constexpr int kStepMaxNew = 8;

// Positions a sequence has room for where the chunk kernel's calls on 8-bit
// pages expand them to 16 bits: the window of its new tokens, from a page's
// start; 0 where all sequences' would take more than 512 MiB.  Expanding is
// faster wherever there is room (expanded / on chip: 16 sequences over 700 to
// 16,383 positions, 9 new tokens each 97 / 115 us, 64 145 / 226, 128 223 / 424);
// the limit keeps the workspace from outgrowing the cache it saves.
int stage_rows(int B, int max_new, int max_pages, int page_size, int ng, int window) {
    long long span = (long long)max_pages * page_size;
    if (span > FLINT_MAX_TOKENS) span = FLINT_MAX_TOKENS;
    if (window > 0 && span > (long long)window + max_new + page_size) span = (long long)window + max_new + page_size;
    span = (span + 15) / 16 * 16;
    return span * B * ng * kHD * 4 <= 512LL << 20 ? (int)span : 0;
}

}  // namespace

size_t paged_attn_workspace(int B, int T, int max_new, int max_pages, int page_size, int ng, int window, bool fp8) {
    const bool chunk = max_new > kStepMaxNew;
    return paged_ws(B, T, ng, kPagedMaxSms * kStepCtasPerSm, chunk ? kPagedMaxSms : 0,
                    chunk && fp8 ? stage_rows(B, max_new, max_pages, page_size, ng, window) : 0).total;
}

flint_status_t launch_paged_attn(const PagedAttnParams& in, const PagedCache& c, int sms, size_t workspace_bytes,
                                 cudaStream_t s) {
    PagedAttnParams p = in;
    if (sms > kPagedMaxSms) sms = kPagedMaxSms;
    p.step_ctas = sms * kStepCtasPerSm;
    p.chunk_ctas = p.max_new > kStepMaxNew ? sms : 0;
    const bool fp8 = p.k_scales != nullptr;
    p.stage_rows = 0;
    if (p.chunk_ctas) {
        // 8-bit pages: expanded first where the caller gave room for it
        const int rows = fp8 ? stage_rows(c.B, p.max_new, c.max_pages, 1 << c.ps_log2, c.ng, p.window) : 0;
        if (rows && paged_ws(c.B, c.T, c.ng, p.step_ctas, p.chunk_ctas, rows).total <= workspace_bytes) p.stage_rows = rows;
        return launch_paged_chunk(p, s);
    }
    p.test_wait_ns = test_stall_once();
    EncodeTiledFn enc = nullptr;
    flint_status_t st = get_encoder(&enc);
    if (st != FLINT_OK) return st;
    StepMaps m;
    const cuuint64_t ps = 1u << c.ps_log2, rows = (cuuint64_t)c.num_pages * c.ng;
    const int tile = fp8 ? StepTile<true>::tile : StepTile<false>::tile, box = (int)ps < tile ? (int)ps : tile, bytes = fp8 ? 1 : 2;
    const CUtensorMapDataType tk = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const CUtensorMapDataType tv = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    st = step_map(enc, &m.k, tk, bytes, p.k_pages, ps, rows, box);
    if (st == FLINT_OK) st = step_map(enc, &m.v, tv, bytes, p.v_pages, ps, rows, box);
    if (st == FLINT_OK) st = step_map(enc, &m.k16, tk, bytes, p.k_pages, ps, rows, 16);
    if (st == FLINT_OK) st = step_map(enc, &m.v16, tv, bytes, p.v_pages, ps, rows, 16);
    if (st != FLINT_OK) return st;
    const cudaError_t e = p.max_new > 1 ? (fp8 ? launch_step<2, true>(m, p, s) : launch_step<2, false>(m, p, s))
                                        : (fp8 ? launch_step<1, true>(m, p, s) : launch_step<1, false>(m, p, s));
    if (e != cudaSuccess) return fail(FLINT_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
    return FLINT_OK;
}

}  // namespace flint
