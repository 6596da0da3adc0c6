// The paged key/value cache: writing new tokens into it, reading positions
// back out of it, and the host side of its entry points.
//
// Append (one warp takes four (token, KV head) rows, eight lanes each): the
// key gets the prologue of FlintAttention.forward (NeMo AutoModel
// "flint.layers" API page; weight-form RMSNorm, then NeoX RoPE on sliding
// layers), in FP32 with one rounding at the end, and goes with its value to
// the slot the page table names.  8-bit pages: with a the row's largest
// magnitude, e is the smallest integer in [-24, 40] (keys: to 7, so that FP16
// holds them) with a <= 448 x 2^e (448: the largest E4M3 number), the codes are
// E4M3(x 2^-e).  A power of two makes
// the scaling exact, so the code's rounding (half a step, 2^-4 relative) is
// the only one, and what is read back is exact in BF16, and in FP16 from a scale
// of 2^-15 on.  An arbitrary
// scale would not round better: E4M3 is a floating format.
//
// Both kernels move bytes: 512 read and 512 or 258 written per token and head
// (append), the reverse for reading.  Measured (launch included): appending
// 21,455 tokens to 8-bit pages 18 us (3.6 TB/s), reading 103,592 back 57 us
// (5.6 TB/s; a copy of as many bytes 50); 128 tokens, or 4,096 read, 8 us, which
// is launch and four dependent loads.
#include <cuda.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cmath>

#include "flint_host.cuh"
#include "flint_paged.cuh"
#include "sm100.cuh"

namespace flint {

constexpr int kPagedThreads = 256;

// One block checks what the rows' warps only step over: the packed boundaries,
// the lengths, and every page table entry the call uses.  It writes the
// status word itself, so no launch has to clear it.  `keep_none`: the entry
// -1 is allowed (append: the token is not kept).
__device__ void paged_check_block(const PagedCache& c, int* status, bool keep_none) {
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    __syncthreads();
    bool bad = false;
    // threads per sequence: a power of two, so that the entries of few long
    // sequences and those of many short ones are both read in parallel
    int per = 1;
    while (per < 32 && c.B * per * 2 <= (int)blockDim.x) per *= 2;
    const int sub = threadIdx.x % per;
    if (threadIdx.x == 0 && (c.cu[0] != 0 || c.cu[c.B] > c.T)) bad = true;
    for (int b = threadIdx.x / per; b < c.B; b += blockDim.x / per) {
        const int a = c.cu[b], n = c.cu[b + 1] - a, L = c.len[b];
        if (a < 0 || n < 0 || n > c.T || L < 0 || L > FLINT_MAX_TOKENS) { bad = true; continue; }
        if (n == 0) continue;
        const long long end = (long long)L + n;
        if (end > FLINT_MAX_TOKENS || end > ((long long)c.max_pages << c.ps_log2)) { bad = true; continue; }
        const int p1 = (int)((end - 1) >> c.ps_log2);
        for (int i = (L >> c.ps_log2) + sub; i <= p1; i += per) {
            const int pg = c.table[(size_t)b * c.max_pages + i];
            if (pg >= c.num_pages || pg < (keep_none ? -1 : 0)) bad = true;
        }
    }
    if (bad) s_bad = 1;
    __syncthreads();
    if (threadIdx.x == 0) *status = s_bad ? kStatusInvalid : kStatusOk;
}

// Places of the warp's tokens t0 .. t0 + n - 1 (n <= 32): lane i holds token
// t0 + i's position and page, page -1 where it has none or belongs to nobody
// (`own`: it belongs to a sequence's run).  One search a warp, and one a lane
// past its sequence's end.
struct PagedPlace { int pos, page; bool own; };
__device__ __forceinline__ PagedPlace paged_locate(const PagedCache& c, int t0, int n) {
    const int t = t0 + (threadIdx.x & 31);
    PagedPlace r = {0, -1, false};
    int b = warp_last_leq(c.cu, c.B, t0);
    if ((int)(threadIdx.x & 31) >= n || t >= c.T) return r;
    if (t >= __ldg(c.cu + b + 1)) {
        // the last sequence that starts at t or before
        int hi = c.B - 1;
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if (__ldg(c.cu + mid) <= t) b = mid; else hi = mid - 1;
        }
    }
    const int a = __ldg(c.cu + b), z = __ldg(c.cu + b + 1);
    const int L = __ldg(c.len + b);
    r.own = t < __ldg(c.cu + c.B);
    if (t < a || t >= z || L < 0) return r;
    const long long p = (long long)L + (t - a);
    if (p >= FLINT_MAX_TOKENS || (p >> c.ps_log2) >= c.max_pages) return r;
    r.pos = (int)p;
    const int page = __ldg(c.table + (size_t)b * c.max_pages + (int)(p >> c.ps_log2));
    r.page = page < c.num_pages ? max(page, -1) : -1;
    return r;
}

// Tokens a warp takes: eight on long calls, so that one look-up serves many
// rows; fewer where a call of few tokens would leave SMs idle.  Measured on four
// heads (fewer heads take the same tokens, so fewer rows, a warp):
// appending 78,523 tokens to 8-bit (16-bit) pages 49 us (55), with 16 tokens a warp
// 55 (59).
__host__ __device__ inline int paged_tokens_per_warp(int T) { return T >= 16384 ? 8 : T >= 4096 ? 4 : T >= 2048 ? 2 : 1; }
// Reading, the longest calls take 32: fewer rows on their way at once keep the
// memory's reads and writes in longer runs (more resident blocks or smaller ones
// are slower, too).  Measured: 103,592 tokens of 8-bit (16-bit) pages 57 us (74),
// with 8 tokens a warp 70 (82); 42,772 tokens 26 (31), with 32 33 (35).
constexpr int kReadThreads = 256;
__host__ __device__ inline int paged_read_tokens(int T) { return T >= 65536 ? 32 : paged_tokens_per_warp(T); }

// E8M0 exponent e of a row whose largest magnitude is a.
__device__ __forceinline__ int paged_exponent(float a, int most) {
    const uint32_t u = __float_as_uint(a);
    const int E = (int)(u >> 23) - 127;                       // a = 1.m x 2^E
    const int e = E - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);   // 448 = 1.75 x 2^8
    return min(max(e, kPagedEMin), most);
}

// Eight values x 2^-e as E4M3 codes (round to nearest even, saturating).
__device__ __forceinline__ uint2 paged_codes8(const float* x, float inv) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

struct AppendParams {
    PagedCache c;
    const __nv_bfloat16* k;      // [T, ng, 128]
    const __nv_bfloat16* v;
    const float* k_norm_w;
    void* k_pages;
    void* v_pages;
    uint8_t* k_scales;           // null: 16-bit pages
    uint8_t* v_scales;
    int* status;
    int use_rope;
    float rope_theta, eps;
};

template <int NG, bool FP8>
__global__ void __launch_bounds__(kPagedThreads) paged_append_kernel(const AppendParams p) {
    if (blockIdx.x == 0) {                             // first, so that no wave of the others is before it
        paged_check_block(p.c, p.status, true);
        return;
    }
    __shared__ double s_inv[64];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int grp = lane >> 3, sub = lane & 7;
    if (p.use_rope) {
        if (tid < 64) s_inv[tid] = exp2(-(double)tid / 64.0 * log2((double)p.rope_theta));
        __syncthreads();
    }
    float w0[8], w1[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w0[e] = p.k_norm_w[8 * sub + e];
        w1[e] = p.k_norm_w[64 + 8 * sub + e];
    }
    // a pass: 4 / NG tokens, four rows of eight lanes
    constexpr int kTok = 4 / NG;
    const int per = max(kTok, paged_tokens_per_warp(p.c.T));
    const long long t0 = (long long)((blockIdx.x - 1) * (kPagedThreads >> 5) + warp) * per;
    if (t0 < p.c.T) {
      const PagedPlace place = paged_locate(p.c, (int)t0, per);
#pragma unroll 2
      for (int i = 0; i < per; i += kTok) {
        const int tok = i + grp / NG, head = grp % NG;
        const bool in = t0 + tok < p.c.T;
        const size_t src = ((size_t)(in ? t0 + tok : t0) * NG + head) * kHD;
        const uint4 ka = *reinterpret_cast<const uint4*>(p.k + src + 8 * sub);
        const uint4 kb = *reinterpret_cast<const uint4*>(p.k + src + 64 + 8 * sub);
        const uint4 va = *reinterpret_cast<const uint4*>(p.v + src + 8 * sub);
        const uint4 vb = *reinterpret_cast<const uint4*>(p.v + src + 64 + 8 * sub);
        const int pos = __shfl_sync(0xffffffffu, place.pos, tok), page = __shfl_sync(0xffffffffu, place.page, tok);
        const bool ok = in && page >= 0;
        float x0[8], x1[8];
        const uint32_t aw[4] = {ka.x, ka.y, ka.z, ka.w}, bw[4] = {kb.x, kb.y, kb.z, kb.w};
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x0[e] = (e & 1) ? __uint_as_float(aw[e >> 1] & 0xffff0000u) : __uint_as_float(aw[e >> 1] << 16);
            x1[e] = (e & 1) ? __uint_as_float(bw[e >> 1] & 0xffff0000u) : __uint_as_float(bw[e >> 1] << 16);
            ss = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], ss));
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        ss += __shfl_xor_sync(0xffffffffu, ss, 4);
        const float rn = 1.f / sqrtf(ss * (1.f / kHD) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x0[e] = x0[e] * rn * w0[e];
            x1[e] = x1[e] * rn * w1[e];
        }
        if (p.use_rope) {
            // a token's 64 rotations are shared by its NG heads: 8 / NG each
            // lane, exchanged by shuffles
            constexpr int kPer = 8 / NG;
            const int li = lane & (8 * NG - 1), base = lane & ~(8 * NG - 1);
            float mc[kPer], ms[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) rope_cos_sin_exact(pos, s_inv[kPer * li + e], &mc[e], &ms[e]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int f = 8 * sub + e;
                const float c = __shfl_sync(0xffffffffu, mc[e % kPer], base + f / kPer);
                const float s = __shfl_sync(0xffffffffu, ms[e % kPer], base + f / kPer);
                const float y0 = x0[e] * c - x1[e] * s;
                const float y1 = x1[e] * c + x0[e] * s;
                x0[e] = y0;
                x1[e] = y1;
            }
        }
        const size_t row = ok ? paged_row(p.c, page, head, pos & ((1 << p.c.ps_log2) - 1)) : 0;
        if constexpr (!FP8) {
            if (ok) {
                // |k~| <= sqrt(128) max|w|: only weights above 5,789 reach the clamp; NaN stays
                const __half2 top = __float2half2_rn(65504.f), low = __float2half2_rn(-65504.f);
                __half2 h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = __hmin2_nan(__hmax2_nan(__floats2half2_rn(x0[2 * e], x0[2 * e + 1]), low), top);
                    h[4 + e] = __hmin2_nan(__hmax2_nan(__floats2half2_rn(x1[2 * e], x1[2 * e + 1]), low), top);
                }
                __half* kd = static_cast<__half*>(p.k_pages) + row * kHD + 8 * sub;
                __nv_bfloat16* vd = static_cast<__nv_bfloat16*>(p.v_pages) + row * kHD + 8 * sub;
                *reinterpret_cast<uint4*>(kd) = *reinterpret_cast<uint4*>(&h[0]);
                *reinterpret_cast<uint4*>(kd + 64) = *reinterpret_cast<uint4*>(&h[4]);
                *reinterpret_cast<uint4*>(vd) = va;
                *reinterpret_cast<uint4*>(vd + 64) = vb;
            }
        } else {
            float y0[8], y1[8];
            const uint32_t cw[4] = {va.x, va.y, va.z, va.w}, dw[4] = {vb.x, vb.y, vb.z, vb.w};
            float ak = 0.f, av = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y0[e] = (e & 1) ? __uint_as_float(cw[e >> 1] & 0xffff0000u) : __uint_as_float(cw[e >> 1] << 16);
                y1[e] = (e & 1) ? __uint_as_float(dw[e >> 1] & 0xffff0000u) : __uint_as_float(dw[e >> 1] << 16);
                ak = fmaxf(ak, fmaxf(fabsf(x0[e]), fabsf(x1[e])));
                av = fmaxf(av, fmaxf(fabsf(y0[e]), fabsf(y1[e])));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                ak = fmaxf(ak, __shfl_xor_sync(0xffffffffu, ak, o));
                av = fmaxf(av, __shfl_xor_sync(0xffffffffu, av, o));
            }
            const int ek = paged_exponent(ak, kPagedKeyEMax), ev = paged_exponent(av, kPagedEMax);
            const float ik = __uint_as_float((uint32_t)(127 - ek) << 23), iv = __uint_as_float((uint32_t)(127 - ev) << 23);
            if (ok) {
                uint8_t* kd = static_cast<uint8_t*>(p.k_pages) + row * kHD + 8 * sub;
                uint8_t* vd = static_cast<uint8_t*>(p.v_pages) + row * kHD + 8 * sub;
                *reinterpret_cast<uint2*>(kd) = paged_codes8(x0, ik);
                *reinterpret_cast<uint2*>(kd + 64) = paged_codes8(x1, ik);
                *reinterpret_cast<uint2*>(vd) = paged_codes8(y0, iv);
                *reinterpret_cast<uint2*>(vd + 64) = paged_codes8(y1, iv);
                if (sub == 0) {
                    p.k_scales[row] = (uint8_t)(ek + 127);
                    p.v_scales[row] = (uint8_t)(ev + 127);
                }
            }
        }
      }
    }
}

struct ReadParams {
    PagedCache c;                // len: first position of each sequence's run
    const void* k_pages;
    const void* v_pages;
    const uint8_t* k_scales;     // null: 16-bit pages
    const uint8_t* v_scales;
    __half* k;                   // [T, ng, 128]
    __nv_bfloat16* v;
    int* status;
};

__device__ __forceinline__ float2 paged_decode2(uint32_t codes) {
    const uint32_t h = e4m3_f16(codes);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int NG, bool FP8>
__global__ void __launch_bounds__(kReadThreads) paged_read_kernel(const ReadParams p) {
    if (blockIdx.x == 0) {
        paged_check_block(p.c, p.status, false);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int grp = lane >> 3, sub = lane & 7;
    constexpr int kTok = 4 / NG;
    const int per = max(kTok, paged_read_tokens(p.c.T));
    const long long t0 = (long long)((blockIdx.x - 1) * (kReadThreads >> 5) + warp) * per;
    if (t0 < p.c.T) {
      const PagedPlace place = paged_locate(p.c, (int)t0, per);
      const bool wide = ((reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 31) == 0;
      // four passes' loads on their way at once
      for (int i0 = 0; i0 < per; i0 += 4 * kTok) {
        uint4 ka[4], kb[4], va[4], vb[4];
        uint32_t sk[4], sv[4];
        bool mine[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int tok = (i0 + y * kTok + grp / NG) & 31;
            const int pos = __shfl_sync(0xffffffffu, place.pos, tok), page = __shfl_sync(0xffffffffu, place.page, tok);
            mine[y] = __shfl_sync(0xffffffffu, (int)place.own, tok) != 0 && i0 + y * kTok < per;
            // a row without a page reads as zeros
            ka[y] = kb[y] = va[y] = vb[y] = make_uint4(0, 0, 0, 0);
            sk[y] = sv[y] = 127;
            if (!mine[y] || page < 0) continue;
            const size_t row = paged_row(p.c, page, grp % NG, pos & ((1 << p.c.ps_log2) - 1));
            if constexpr (!FP8) {
                const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.k_pages) + row * kHD);
                const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.v_pages) + row * kHD);
                ka[y] = __ldg(ks + sub); kb[y] = __ldg(ks + 8 + sub);
                va[y] = __ldg(vs + sub); vb[y] = __ldg(vs + 8 + sub);
            } else {
                ka[y] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.k_pages) + row * kHD) + sub);
                va[y] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.v_pages) + row * kHD) + sub);
                sk[y] = __ldg(p.k_scales + row);
                sv[y] = __ldg(p.v_scales + row);
            }
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (!mine[y]) continue;                           // rows behind the last sequence stay as they were
            const size_t r = (size_t)(t0 + i0 + y * kTok + grp / NG) * NG + grp % NG;
            if constexpr (!FP8) {
                uint4* kd = reinterpret_cast<uint4*>(p.k + r * kHD);
                uint4* vd = reinterpret_cast<uint4*>(p.v + r * kHD);
                kd[sub] = ka[y]; kd[8 + sub] = kb[y];
                vd[sub] = va[y]; vd[8 + sub] = vb[y];
            } else {
                const float fk = paged_scale(sk[y]), fv = paged_scale(sv[y]);
                const uint32_t kw[4] = {ka[y].x, ka[y].y, ka[y].z, ka[y].w}, vw[4] = {va[y].x, va[y].y, va[y].z, va[y].w};
                __half2 ko[8];
                __nv_bfloat162 vo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 a = paged_decode2(kw[i >> 1] >> (16 * (i & 1)));
                    const float2 b = paged_decode2(vw[i >> 1] >> (16 * (i & 1)));
                    ko[i] = __floats2half2_rn(a.x * fk, a.y * fk);
                    vo[i] = __floats2bfloat162_rn(b.x * fv, b.y * fv);
                }
                uint4* kd = reinterpret_cast<uint4*>(p.k + r * kHD + 16 * sub);
                uint4* vd = reinterpret_cast<uint4*>(p.v + r * kHD + 16 * sub);
                const uint4 k0 = *reinterpret_cast<uint4*>(&ko[0]), k1 = *reinterpret_cast<uint4*>(&ko[4]);
                const uint4 v0 = *reinterpret_cast<uint4*>(&vo[0]), v1 = *reinterpret_cast<uint4*>(&vo[4]);
                if (wide) {
                    st_32(kd, k0, k1);
                    st_32(vd, v0, v1);
                } else {
                    kd[0] = k0; kd[1] = k1;
                    vd[0] = v0; vd[1] = v1;
                }
            }
        }
      }
    }
}

// ============================================================================ host
flint_status_t launch_paged_attn(const PagedAttnParams& p, const PagedCache& c, int sms, size_t workspace_bytes,
                                 cudaStream_t s);
size_t paged_attn_workspace(int B, int T, int max_new, int max_pages, int page_size, int ng, int window, bool fp8);

namespace {

bool al(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    explicit Range(const char* name) { nvtxRangePushA(name); }
    ~Range() { nvtxRangePop(); }
};

// What the three entry points check alike; fills c.
flint_status_t check_cache(PagedCache* c, const void* k_pages, const void* v_pages, const void* k_scales,
                           const void* v_scales, const int32_t* table, const int32_t* len, const int32_t* cu,
                           int32_t B, int32_t T, int32_t max_pages, int32_t num_pages, int32_t page_size,
                           int32_t kv_heads) {
    fail(FLINT_OK, "%s", "");
    if (B < 0 || B > FLINT_MAX_DECODE_BATCH)
        return fail(FLINT_ERR_INVALID_ARG, "B=%d outside [0, %d]", B, FLINT_MAX_DECODE_BATCH);
    if (T < 0 || T > FLINT_MAX_TOKENS)
        return fail(FLINT_ERR_INVALID_ARG, "T=%d outside [0, %d]", T, FLINT_MAX_TOKENS);
    if (kv_heads != 1 && kv_heads != 2 && kv_heads != 4)
        return fail(FLINT_ERR_INVALID_ARG, "kv_heads=%d: 1, 2 or 4", kv_heads);
    if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
        return fail(FLINT_ERR_UNSUPPORTED, "page_size=%d: 16, 32, 64 or 128 slots", page_size);
    if ((k_scales == nullptr) != (v_scales == nullptr))
        return fail(FLINT_ERR_INVALID_ARG, "give k_scales and v_scales (8-bit pages) or neither (16-bit pages)");
    if (B == 0 || T == 0) return FLINT_OK;
    if (max_pages < 1 || max_pages > FLINT_MAX_TOKENS)
        return fail(FLINT_ERR_INVALID_ARG, "max_pages=%d outside [1, %d]", max_pages, FLINT_MAX_TOKENS);
    if (num_pages < 1 || (long long)num_pages * kv_heads > 0x7fffffffLL)
        return fail(FLINT_ERR_INVALID_ARG, "num_pages=%d", num_pages);
    if (!k_pages || !v_pages || !table || !len || !cu) return fail(FLINT_ERR_INVALID_ARG, "null tensor pointer");
    if (!al(k_pages, 16) || !al(v_pages, 16) || !al(k_scales, 16) || !al(v_scales, 16))
        return fail(FLINT_ERR_INVALID_ARG, "the pages and their scales must be 16-byte aligned");
    if (!al(table, 4) || !al(len, 4) || !al(cu, 4)) return fail(FLINT_ERR_INVALID_ARG, "misaligned 32-bit array");
    c->table = table;
    c->len = len;
    c->cu = cu;
    c->B = B;
    c->T = T;
    c->max_pages = max_pages;
    c->num_pages = num_pages;
    c->ps_log2 = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
    c->ng = kv_heads;
    return FLINT_OK;
}

flint_status_t check_prologue(int32_t use_rope, float rope_theta, float eps) {
    if (use_rope != 0 && use_rope != 1) return fail(FLINT_ERR_INVALID_ARG, "use_rope must be 0 or 1");
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(FLINT_ERR_INVALID_ARG, "eps must be > 0");
    if (use_rope && (!(rope_theta > 1.f) || !std::isfinite(rope_theta)))
        return fail(FLINT_ERR_INVALID_ARG, "rope_theta must be > 1");
    return FLINT_OK;
}

flint_status_t check_workspace(const void* workspace, size_t have, size_t need) {
    if (!workspace || !al(workspace, 256))
        return fail(FLINT_ERR_WORKSPACE, "workspace missing or not 256-byte aligned");
    if (have < need) return fail(FLINT_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", have, need);
    return FLINT_OK;
}

// Blocks of a row kernel whose warps take per tokens (at least four rows), and
// the checking block.
int row_blocks(const PagedCache& c, int per, int threads) {
    if (per < 4 / c.ng) per = 4 / c.ng;
    const long long warps = ((long long)c.T + per - 1) / per;
    return (int)((warps + threads / 32 - 1) / (threads / 32)) + 1;
}

template <bool FP8>
void launch_append(const AppendParams& p, int grid, cudaStream_t s) {
    if (p.c.ng == 4) paged_append_kernel<4, FP8><<<grid, kPagedThreads, 0, s>>>(p);
    else if (p.c.ng == 2) paged_append_kernel<2, FP8><<<grid, kPagedThreads, 0, s>>>(p);
    else paged_append_kernel<1, FP8><<<grid, kPagedThreads, 0, s>>>(p);
}
template <bool FP8>
void launch_read(const ReadParams& p, int grid, cudaStream_t s) {
    if (p.c.ng == 4) paged_read_kernel<4, FP8><<<grid, kReadThreads, 0, s>>>(p);
    else if (p.c.ng == 2) paged_read_kernel<2, FP8><<<grid, kReadThreads, 0, s>>>(p);
    else paged_read_kernel<1, FP8><<<grid, kReadThreads, 0, s>>>(p);
}

}  // namespace
}  // namespace flint

using namespace flint;

extern "C" {

flint_status_t flint_paged_append(const void* k, const void* v, const float* k_norm_w, void* k_pages,
                                  void* v_pages, void* k_scales, void* v_scales, const int32_t* page_table,
                                  const int32_t* cache_len, const int32_t* cu_new, int32_t B, int32_t T,
                                  int32_t max_pages, int32_t num_pages, int32_t page_size, int32_t kv_heads,
                                  int32_t use_rope, float rope_theta, float eps, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    Range r("flint_paged_append");
    AppendParams p = {};
    flint_status_t st = check_cache(&p.c, k_pages, v_pages, k_scales, v_scales, page_table, cache_len, cu_new, B, T,
                                    max_pages, num_pages, page_size, kv_heads);
    if (st == FLINT_OK) st = check_prologue(use_rope, rope_theta, eps);
    if (st != FLINT_OK || B == 0 || T == 0) return st;
    if (!k || !v || !k_norm_w) return fail(FLINT_ERR_INVALID_ARG, "null tensor pointer");
    if (!al(k, 16) || !al(v, 16)) return fail(FLINT_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    if (!al(k_norm_w, 4)) return fail(FLINT_ERR_INVALID_ARG, "misaligned 32-bit array");
    st = check_workspace(workspace, workspace_bytes, FLINT_PAGED_STATUS_BYTES);
    if (st != FLINT_OK) return st;
    int sms = 0;
    st = device_setup(&sms);
    if (st != FLINT_OK) return st;
    p.k = static_cast<const __nv_bfloat16*>(k);
    p.v = static_cast<const __nv_bfloat16*>(v);
    p.k_norm_w = k_norm_w;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = static_cast<uint8_t*>(k_scales);
    p.v_scales = static_cast<uint8_t*>(v_scales);
    p.status = static_cast<int*>(workspace);
    p.use_rope = use_rope;
    p.rope_theta = rope_theta;
    p.eps = eps;
    const int grid = row_blocks(p.c, paged_tokens_per_warp(p.c.T), kPagedThreads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k_scales) launch_append<true>(p, grid, s);
    else launch_append<false>(p, grid, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FLINT_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
    return FLINT_OK;
}

flint_status_t flint_paged_read(const void* k_pages, const void* v_pages, const void* k_scales,
                                const void* v_scales, const int32_t* page_table, const int32_t* start,
                                const int32_t* cu_out, int32_t B, int32_t T, int32_t max_pages,
                                int32_t num_pages, int32_t page_size, int32_t kv_heads, void* k, void* v,
                                void* workspace, size_t workspace_bytes, void* stream) {
    Range r("flint_paged_read");
    ReadParams p = {};
    flint_status_t st = check_cache(&p.c, k_pages, v_pages, k_scales, v_scales, page_table, start, cu_out, B, T,
                                    max_pages, num_pages, page_size, kv_heads);
    if (st != FLINT_OK || B == 0 || T == 0) return st;
    if (!k || !v) return fail(FLINT_ERR_INVALID_ARG, "null tensor pointer");
    if (!al(k, 16) || !al(v, 16)) return fail(FLINT_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    st = check_workspace(workspace, workspace_bytes, FLINT_PAGED_STATUS_BYTES);
    if (st != FLINT_OK) return st;
    int sms = 0;
    st = device_setup(&sms);
    if (st != FLINT_OK) return st;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = static_cast<const uint8_t*>(k_scales);
    p.v_scales = static_cast<const uint8_t*>(v_scales);
    p.k = static_cast<__half*>(k);
    p.v = static_cast<__nv_bfloat16*>(v);
    p.status = static_cast<int*>(workspace);
    const int grid = row_blocks(p.c, paged_read_tokens(p.c.T), kReadThreads);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k_scales) launch_read<true>(p, grid, s);
    else launch_read<false>(p, grid, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return fail(FLINT_ERR_CUDA, "read launch: %s", cudaGetErrorString(e));
    return FLINT_OK;
}

size_t flint_attn_paged_workspace_bytes(int32_t B, int32_t T, int32_t max_new, int32_t max_pages, int32_t page_size,
                                        int32_t kv_heads, int32_t window, int32_t eight_bit) {
    if (B < 0 || B > FLINT_MAX_DECODE_BATCH || T < 0 || T > FLINT_MAX_TOKENS || max_new < 0 || max_pages < 1 ||
        max_pages > FLINT_MAX_TOKENS || window < 0 || (kv_heads != 1 && kv_heads != 2 && kv_heads != 4) ||
        (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128))
        return 0;
    return paged_attn_workspace(B, T, max_new, max_pages, page_size, kv_heads, window, eight_bit != 0);
}

flint_status_t flint_attn_paged(const void* q, const float* q_norm_w, const float* sinks, const void* k_pages,
                                const void* v_pages, const void* k_scales, const void* v_scales,
                                const int32_t* page_table, const int32_t* cache_len, const int32_t* cu_new,
                                int32_t B, int32_t T, int32_t max_new, int32_t max_pages, int32_t num_pages,
                                int32_t page_size, int32_t kv_heads, int32_t window, int32_t use_rope,
                                float rope_theta, float eps, void* out, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
    Range r("flint_attn_paged");
    PagedCache c = {};
    flint_status_t st = check_cache(&c, k_pages, v_pages, k_scales, v_scales, page_table, cache_len, cu_new, B, T,
                                    max_pages, num_pages, page_size, kv_heads);
    if (st == FLINT_OK) st = check_prologue(use_rope, rope_theta, eps);
    if (st != FLINT_OK) return st;
    if (window < 0) return fail(FLINT_ERR_INVALID_ARG, "window=%d < 0", window);
    if (max_new < 0) return fail(FLINT_ERR_INVALID_ARG, "max_new=%d < 0", max_new);
    if (B == 0 || T == 0) return FLINT_OK;
    if (!q || !q_norm_w || !sinks || !out) return fail(FLINT_ERR_INVALID_ARG, "null tensor pointer");
    if (!al(q, 16) || !al(out, 16)) return fail(FLINT_ERR_INVALID_ARG, "q and out must be 16-byte aligned");
    if (!al(q_norm_w, 4) || !al(sinks, 4) || !al(lse, 4)) return fail(FLINT_ERR_INVALID_ARG, "misaligned 32-bit array");
    // the least: 8-bit pages converted on chip
    st = check_workspace(workspace, workspace_bytes,
                         paged_attn_workspace(B, T, max_new, max_pages, page_size, kv_heads, window, false));
    if (st != FLINT_OK) return st;
    int sms = 0;
    st = device_setup(&sms);
    if (st != FLINT_OK) return st;
    PagedAttnParams p = {};
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.q_norm_w = q_norm_w;
    p.sinks = sinks;
    p.k_pages = k_pages;
    p.v_pages = v_pages;
    p.k_scales = static_cast<const uint8_t*>(k_scales);
    p.v_scales = static_cast<const uint8_t*>(v_scales);
    p.out = static_cast<__nv_bfloat16*>(out);
    p.lse = lse;
    p.ws = static_cast<char*>(workspace);
    p.c = c;
    p.max_new = max_new;
    p.window = window;
    p.use_rope = use_rope;
    p.rope_theta = rope_theta;
    p.eps = eps;
    return launch_paged_attn(p, c, sms, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
