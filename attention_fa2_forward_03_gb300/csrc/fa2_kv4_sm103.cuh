// A paged KV cache held in 4 bits: the kernels that plan its pages, write it,
// read it back and attend over it (sm_103a).
//
// The cache is [num_pages, H_kv, 2, page * (D/2 + D/16)] bytes: of a page and
// KV head first the keys, then the values of `page` tokens, each part as the
// e2m1 codes [page, D/2] followed by one e4m3 scale per 16 elements
// [page, D/16]. Element = code * scale * descale[head]. A product code * scale
// has at most six significant bits and lies in [2^-10, 2688], so it is exact in
// fp16: both matrix products of the attention run on fp16 operands whatever
// the type of q, and the cache costs no precision beyond its own rounding.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fa2.h"
#include "fa2_fwd_sm103.cuh"
#include "ptx_sm103.cuh"

namespace fa2 {
namespace kv4 {

// Sites of the status word for page ids, slots and lengths that point outside
// the cache or the table. These checks are in every build: the ids come from
// device memory, so the host cannot make them, and an id that fails is
// skipped, never followed.
enum Site : int { kSitePage = 48, kSiteSlot = 49, kSiteLength = 50, kSitePool = 51 };

__device__ __forceinline__ void report(int site) { atomicCAS(&g_fa2_status, 0, FA2_ERR_BOUNDS | (site << 8)); }

// Bytes of one part (keys or values) of a page of one head.
template <int D>
__host__ __device__ constexpr int part_bytes(int page) {
    return page * (D / 2 + D / 16);
}

// ------------------------------------------------------------------ conversions

// Four bytes of e2m1 pairs to four fp16 pairs (low four bits of a byte in the
// low half).
__device__ __forceinline__ void e2m1_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 bytes (low byte in the low half) to an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Eight fp32 values to eight e2m1 codes, the first in the lowest four bits:
// nearest, ties to even, at most 6 in magnitude.
__device__ __forceinline__ uint32_t pack8_e2m1(const float* x) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// ------------------------------------------------------------------ append

struct AppendParams {
    const void* x[2];          // keys, values
    long long sb[2], sh[2], sn[2];  // strides in elements: request, head, token
    const float* descale[2];   // [hkv]
    const int* slots;          // [B, N]
    uint8_t* cache;
    int rows;                  // B * hkv * N
    int hkv, n, page, log2_page;
    int num_slots;             // num_pages * page
};

// One thread quantises 16 elements of a key and of a value: the unit of a
// scale, 32 bytes read and 9 written for each.
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) fa2_kv4_append_kernel(const AppendParams p) {
    constexpr int kGroups = D / 16;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = i / kGroups;
    const int grp = static_cast<int>(i % kGroups);
    if (row >= p.rows) return;
    const unsigned bh = static_cast<unsigned>(row) / static_cast<unsigned>(p.n);
    const unsigned n = static_cast<unsigned>(row) - bh * static_cast<unsigned>(p.n);
    const unsigned b = bh / static_cast<unsigned>(p.hkv), h = bh - b * static_cast<unsigned>(p.hkv);
    const int slot = p.slots[static_cast<long long>(b) * p.n + n];
    if (slot < 0) return;
    if (slot >= p.num_slots) {
        report(kSiteSlot);
        return;
    }
    const int pg = slot >> p.log2_page, at = slot & (p.page - 1);
    uint4 in[2][2];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        const uint16_t* src = static_cast<const uint16_t*>(p.x[part]) + b * p.sb[part] + h * p.sh[part] +
                              n * p.sn[part] + grp * 16;
        in[part][0] = reinterpret_cast<const uint4*>(src)[0];
        in[part][1] = reinterpret_cast<const uint4*>(src)[1];
    }
    uint8_t* blk = p.cache + (static_cast<long long>(pg) * p.hkv + h) * 2 * part_bytes<D>(p.page);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        float x[16];
        const uint32_t* w = reinterpret_cast<const uint32_t*>(in[part]);
#pragma unroll
        for (int j = 0; j < 8; ++j) ptx::unpack2<kBf16>(w[j], x[2 * j], x[2 * j + 1]);
        // The largest magnitude by its bits, which order NaN above infinity
        // above every finite value.
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        const float descale = p.descale[part][h];
        uint32_t s8 = 0x7F;   // e4m3 NaN: a block that holds a NaN or an infinity reads back as NaN
        uint32_t codes[2] = {0, 0};
        if (top < 0x7F800000u) {
            const float want = __fdiv_rn(__uint_as_float(top), 6.0f * descale);
            asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %1, %1;\n\tcvt.u32.u16 %0, a;\n\t}"
                : "=r"(s8)
                : "f"(want));
            s8 &= 0xFF;
            float s, other;
            ptx::unpack2<false>(e4m3_to_f16(s8), s, other);
            const float t = __fmul_rn(s, descale);
            if (t > 0.0f) {
                // True quotients: a tie between two codes (common, as inputs
                // and scales have few bits) has to be seen as one.
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = __fdiv_rn(x[j], t);
                codes[0] = pack8_e2m1(x);
                codes[1] = pack8_e2m1(x + 8);
            }
        }
        uint8_t* dst = blk + part * part_bytes<D>(p.page);
        *reinterpret_cast<uint2*>(dst + at * (D / 2) + grp * 8) = make_uint2(codes[0], codes[1]);
        dst[p.page * (D / 2) + at * kGroups + grp] = static_cast<uint8_t>(s8);
    }
}

// ------------------------------------------------------------------ gather

struct GatherParams {
    const uint8_t* cache;
    const int* block_table;    // [B, max_pages]
    const int* seq_lens;       // [B]
    const int* starts;         // [B] or NULL (0)
    const float* descale[2];   // [hkv]
    void* out[2];              // [B, hkv, N, D]
    int rows;                  // B * hkv * N
    int hkv, n, page, log2_page, max_pages, num_pages;
};

// One thread reads 16 elements of a key and of a value: 9 bytes read and 32
// written for each. Rows at or past a request's length are zeros.
template <int D, bool kBf16>
__global__ void __launch_bounds__(256) fa2_kv4_gather_kernel(const GatherParams p) {
    constexpr int kGroups = D / 16;
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long row = i / kGroups;
    const int grp = static_cast<int>(i % kGroups);
    if (row >= p.rows) return;
    const unsigned bh = static_cast<unsigned>(row) / static_cast<unsigned>(p.n);
    const unsigned n = static_cast<unsigned>(row) - bh * static_cast<unsigned>(p.n);
    const unsigned b = bh / static_cast<unsigned>(p.hkv), h = bh - b * static_cast<unsigned>(p.hkv);
    const long long pos = static_cast<long long>(p.starts ? p.starts[b] : 0) + n;
    const uint8_t* blk = nullptr;
    int at = 0;
    if (pos >= 0 && pos < p.seq_lens[b]) {
        const long long entry = pos >> p.log2_page;
        const int pg = entry < p.max_pages ? p.block_table[static_cast<long long>(b) * p.max_pages + entry] : -1;
        at = static_cast<int>(pos & (p.page - 1));
        if (pg >= 0 && pg < p.num_pages)
            blk = p.cache + (static_cast<long long>(pg) * p.hkv + h) * 2 * part_bytes<D>(p.page);
        else
            report(kSitePage);
    }
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        uint32_t out[8] = {};
        if (blk) {
            const uint8_t* src = blk + part * part_bytes<D>(p.page);
            const uint2 codes = *reinterpret_cast<const uint2*>(src + at * (D / 2) + grp * 8);
            float s, other;
            ptx::unpack2<false>(e4m3_to_f16(src[p.page * (D / 2) + at * kGroups + grp]), s, other);
            const float t = __fmul_rn(s, p.descale[part][h]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t c[4];
                e2m1_to_f16(j ? codes.y : codes.x, c);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    ptx::unpack2<false>(c[e], lo, hi);
                    out[4 * j + e] = ptx::pack2<kBf16>(__fmul_rn(lo, t), __fmul_rn(hi, t));
                }
            }
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[part]) + row * D + grp * 16);
        dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
        dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
}

// ------------------------------------------------------------------ plan

struct PlanParams {
    const int* seq_lens;       // [B]
    const int* new_lens;       // [B]; negative: the request ends
    int* block_table;          // [B, max_pages]
    int* free_pages;           // [num_pages], a ring
    const int* free_state;     // {first, count}
    int* seq_lens_out;         // [B], may be seq_lens
    int* accepted;             // [B]
    int* slots;                // [B, N]
    int* free_state_out;       // {first, count}, may be free_state
    int B, n, max_pages, page, log2_page, num_pages;
};

constexpr int kPlanThreads = 1024;

// Exclusive prefix sums of (a, r) over the block's threads, and the totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& r, long long& a_all, long long& r_all,
                                            long long (*sm)[kPlanThreads / 32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ir = r;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long ta = __shfl_up_sync(~0u, ia, o), tr = __shfl_up_sync(~0u, ir, o);
        if (lane >= o) {
            ia += ta;
            ir += tr;
        }
    }
    __syncthreads();
    if (lane == 31) {
        sm[0][warp] = ia;
        sm[1][warp] = ir;
    }
    __syncthreads();
    long long ba = 0, br = 0;
    a_all = r_all = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) {
            ba = a_all;
            br = r_all;
        }
        a_all += sm[0][w];
        r_all += sm[1][w];
    }
    a = ba + ia - a;
    r = br + ir - r;
}

// Pages, lengths and the free ring, by one block: a scan over the requests in
// order, 1024 at a time. A request gets its pages iff the pages wanted up to
// and including it are free (or it needs none); pages of requests that end
// join the ring behind its last page and are not handed out by this call.
__global__ void __launch_bounds__(kPlanThreads) fa2_kv4_plan_kernel(const PlanParams p) {
    __shared__ long long sm[2][kPlanThreads / 32];
    int first = p.free_state[0], count = p.free_state[1];
    if (first < 0 || first >= p.num_pages || count < 0 || count > p.num_pages) {
        if (threadIdx.x == 0) report(kSitePool);
        first = 0;
        count = 0;
    }
    const long long room = static_cast<long long>(p.max_pages) << p.log2_page;
    long long want = 0, back = 0;   // pages wanted by, and returned by, the requests before this chunk
    long long taken = 0;            // pages this thread's requests got
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int len = 0, add = 0;
        bool in = b < p.B, ends = false, fits = false;
        if (in) {
            len = p.seq_lens[b];
            add = p.new_lens[b];
            if (len < 0 || len > room) {
                report(kSiteLength);
                len = 0;
            }
            ends = add < 0;
            fits = !ends && add <= p.n && static_cast<long long>(len) + add <= room;
        }
        const int have = (len + p.page - 1) >> p.log2_page;
        const int need = fits ? static_cast<int>(((static_cast<long long>(len) + add + p.page - 1) >> p.log2_page) - have) : 0;
        const int rel = in && ends ? have : 0;
        long long a = need, r = rel, a_all, r_all;
        block_scan2(a, r, a_all, r_all, sm);
        const bool granted = fits && (need == 0 || want + a + need <= count);
        if (in) {
            int* row = p.block_table + static_cast<long long>(b) * p.max_pages;
            if (granted) {
                taken += need;
                for (int j = 0; j < need; ++j) row[have + j] = p.free_pages[(first + want + a + j) % p.num_pages];
            }
            for (int j = 0; j < rel; ++j) p.free_pages[(first + static_cast<long long>(count) + back + r + j) % p.num_pages] = row[j];
            p.seq_lens_out[b] = ends ? 0 : len + (granted ? add : 0);
            p.accepted[b] = granted ? add : 0;
        }
        want += a_all;
        back += r_all;
    }
    long long zero = 0, all, unused;
    block_scan2(taken, zero, all, unused, sm);
    if (threadIdx.x == 0) {
        long long left = count - all + back;
        if (left > p.num_pages) {   // more pages came back than were out
            report(kSitePool);
            left = p.num_pages;
        }
        p.free_state_out[0] = static_cast<int>((first + all) % p.num_pages);
        p.free_state_out[1] = static_cast<int>(left);
    }
}

// Slots of the accepted tokens, -1 in the other places.
__global__ void __launch_bounds__(256) fa2_kv4_slots_kernel(const PlanParams p) {
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= static_cast<long long>(p.B) * p.n) return;
    const int b = static_cast<int>(i / p.n), j = static_cast<int>(i - static_cast<long long>(b) * p.n);
    const int add = p.accepted[b];
    int slot = -1;
    if (j < add) {
        const int pos = p.seq_lens_out[b] - add + j;
        const int pg = p.block_table[static_cast<long long>(b) * p.max_pages + (pos >> p.log2_page)];
        if (pg >= 0 && pg < p.num_pages) slot = (pg << p.log2_page) + (pos & (p.page - 1));
        else report(kSitePage);
    }
    p.slots[i] = slot;
}

// ------------------------------------------------------------------ attention

constexpr int kTile = 32;      // tokens a warp takes at a time
constexpr int kWarps = 4;
constexpr int kFwdThreads = 32 * kWarps;
constexpr int kMaxCtas = 640;  // workspace is sized for this many

struct FwdParams {
    const void* q;             // [B, H_q, N_q, D]: `rows` contiguous rows a KV head
    const uint8_t* cache;
    const float* k_descale;    // [hkv]
    const float* v_descale;
    const int* seq_lens;       // [B]
    const int* block_table;    // [B, max_pages]
    void* o;
    float* lse;
    float* part_o;             // [2 * ctas, 8 NR, D]
    float* part_ml;            // [2 * ctas, 8 NR, 2]
    int B, hkv, nq, rows, rblocks;   // rows = group * N_q; rblocks = ceil(rows / (8 NR))
    int max_pages, max_tokens, page, log2_page, num_pages;
    int causal;
    int ctas;                  // CTAs that take work
    float scale_log2;
};

// fp32 accumulators += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// The work: the tiles of every (request, KV head, row block), in that order,
// as one line of units cut into equal runs, one a CTA. A run may end inside a
// segment (the tiles of one row block); its CTAs then leave partial results.
struct Cursor {
    long long u, end;          // next unit, end of the run
    int b, hr, tile, tiles;    // request, head * rblocks + row block, next tile of the segment, its tiles
};

__device__ __forceinline__ int tiles_of(const FwdParams& p, int b) {
    const int len = min(max(p.seq_lens[b], 0), p.max_tokens);
    return (len >> 5) + ((len & 31) != 0);
}

// Finds unit `u` of the line for the caller's whole block: per = units a CTA,
// total = all units. Uses shared memory `sm` (kFwdThreads / 32 + 4 values).
// first_run: u = blockIdx.x * per, else u = (blockIdx.x + 1) * per - 1.
__device__ __forceinline__ bool locate(const FwdParams& p, bool last, long long* sm, long long& per, long long& total,
                                       Cursor& cur) {
    const int tid = threadIdx.x, nt = blockDim.x;
    const int chunk = (p.B + nt - 1) / nt;
    const int b0 = min(tid * chunk, p.B), b1 = min(b0 + chunk, p.B);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of(p, b);
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(~0u, inc, o);
        if ((tid & 31) >= o) inc += t;
    }
    if ((tid & 31) == 31) sm[tid >> 5] = inc;
    if (tid == 0) sm[nt / 32] = -1;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < nt / 32; ++w) {
        if (w == (tid >> 5)) before = total;
        total += sm[w];
    }
    const int hrs = p.hkv * p.rblocks;
    total *= hrs;
    per = (total + p.ctas - 1) / p.ctas;
    per = (per + kWarps - 1) / kWarps * kWarps;
    const long long u = last ? (blockIdx.x + 1) * per - 1 : blockIdx.x * per;
    long long at = (before + inc - mine) * hrs;   // first unit of request b0
    if (u < total && u >= at && u < at + mine * hrs) {
        int b = b0;
        long long t = tiles_of(p, b) * static_cast<long long>(hrs);
        while (u >= at + t) {
            at += t;
            ++b;
            t = tiles_of(p, b) * static_cast<long long>(hrs);
        }
        sm[nt / 32] = b;
        sm[nt / 32 + 1] = u - at;
    }
    __syncthreads();
    if (u >= total) return false;
    cur.u = u;
    cur.end = min(total, u + per);
    cur.b = static_cast<int>(sm[nt / 32]);
    cur.tiles = tiles_of(p, cur.b);
    const long long rem = sm[nt / 32 + 1];
    cur.hr = static_cast<int>(rem / cur.tiles);
    cur.tile = static_cast<int>(rem - static_cast<long long>(cur.hr) * cur.tiles);
    return true;
}

// Past the current segment's tiles of this run.
__device__ __forceinline__ void next_segment(const FwdParams& p, Cursor& c, int n) {
    c.u += n;
    c.tile = 0;
    if (c.u >= c.end) return;
    if (++c.hr == p.hkv * p.rblocks) {
        c.hr = 0;
        do {
            ++c.b;
            c.tiles = tiles_of(p, c.b);
        } while (c.tiles == 0);
    }
}

template <int D, int NR>
struct FwdSmem {
    static constexpr int kRows = 8 * NR;
    static constexpr int kStride = D + 4;    // floats a row of the merge buffer
    uint2 q[D / 16][NR][32];                 // B fragments of q
    float c[kRows];                          // log2(e) * scale * descale, with q's power of two taken out
    float o[kWarps][kRows * kStride];
    float ml[kWarps][kRows][2];
    long long scan[kFwdThreads / 32 + 4];
};

// Rows of q as B fragments of Q^T (k = d, n = row), in fp16. A bf16 row is
// scaled by the power of two that brings its largest magnitude into
// [2^14, 2^15): its 8 bits are kept exactly but for elements below 2^-29 of
// that magnitude. Thread (g, t) of a warp takes row g and elements
// [t D/4, (t + 1) D/4): the order of d inside a product is free, and this one
// lets a thread read a key's codes as one piece.
template <int D, int NR, bool kBf16>
__device__ __forceinline__ void stage_q(const FwdParams& p, FwdSmem<D, NR>& sm, int b, int hr) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int h = hr / p.rblocks, rb = hr - h * p.rblocks;
    const float c0 = p.scale_log2 * p.k_descale[h];
    for (int nr = warp; nr < NR; nr += kWarps) {
        const int r = (rb * NR + nr) * 8 + g;
        uint32_t w[D / 8];
        if (r < p.rows) {
            const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                                  ((static_cast<long long>(b) * p.hkv + h) * p.rows + r) * D + t * (D / 4);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint4 v = reinterpret_cast<const uint4*>(src)[j];
                w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) w[j] = 0;
        }
        float c = c0;
        if constexpr (kBf16) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const int e = static_cast<int>(top >> 7);   // biased exponent of the largest magnitude
            const int k = e == 255 ? 0 : min(14 + 127 - e, 126);
            const float f = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
            c *= __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                float lo, hi;
                ptx::unpack2<true>(w[j], lo, hi);
                w[j] = ptx::pack2<false>(lo * f, hi * f);
            }
        }
#pragma unroll
        for (int s = 0; s < D / 16; ++s) sm.q[s][nr][lane] = make_uint2(w[2 * s], w[2 * s + 1]);
        if (t == 0) sm.c[nr * 8 + g] = c;
    }
}

// What a warp carries along a segment: unnormalised O^T as accumulators
// (thread (g, t): d in [g D/8, (g + 1) D/8), rows 2t and 2t + 1 of each eight)
// and per row the reference of the exponentials.
template <int D, int NR>
struct Acc {
    float o[NR][D / 16][4];
    float m[NR][2];        // running maximum of the raw scores, -inf before the first
    float thr[NR][2];      // a score above this moves the reference
    float ref[NR][2];      // exponentials are 2^(s c - ref)
    float l[NR][2];        // this thread's part of the row sums
    float c[NR][2];
    int lim[NR][2];        // first key the row may not see
};

// Exponentials reach 2^15 at most (fp16 holds 65504): 2^7 at the running
// maximum, and scores may pass that by 2^8 before the reference moves, which
// spares most tiles the exchange of maxima and the rescaling.
constexpr float kLift = 7.0f, kSlack = 8.0f;

// 32 tokens from `tok0`: kc[u], ks[u], vc[u], vs[u] point at the codes and
// scales of the 16 tokens of half u. `kMask`: some row may not see all of
// them, or half u is past the sequence or on a bad page (n_ok[u] < 16 tokens
// of it are usable).
//
// Token order inside a half: position kk of a product is token (kk >> 1) +
// 4 (kk & 1) + (kk & 8), so a warp reads four neighbouring tokens at once.
template <int D, int NR, bool kMask>
__device__ __forceinline__ void tile_step(Acc<D, NR>& acc, const uint2 (*qs)[NR][32], const uint8_t* const (&kc)[2],
                                          const uint8_t* const (&ks)[2], const uint8_t* const (&vc)[2],
                                          const uint8_t* const (&vs)[2], int tok0, const int (&n_ok)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tg = (g >> 1) + 4 * (g & 1);
    float s[NR][2][4];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nr][u][e] = 0.0f;

    // S^T = K Q^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t w[2][D / 32];   // codes of tokens tg and 8 + tg, elements [t D/4, (t+1) D/4)
        uint32_t sc[2][2];       // their scales, twice each
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint8_t* src = kc[u] + (tg + 8 * x) * (D / 2) + t * (D / 8);
            const uint8_t* ss = ks[u] + (tg + 8 * x) * (D / 16) + t * (D / 64);
            if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                w[x][0] = v.x; w[x][1] = v.y; w[x][2] = v.z; w[x][3] = v.w;
                const uint32_t two = e4m3_to_f16(*reinterpret_cast<const uint16_t*>(ss));
                sc[x][0] = __byte_perm(two, 0, 0x1010);
                sc[x][1] = __byte_perm(two, 0, 0x3232);
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                w[x][0] = v.x; w[x][1] = v.y;
                sc[x][0] = sc[x][1] = e4m3_to_f16(*ss * 0x0101u);
            }
        }
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint32_t a[2][4];
            e2m1_to_f16(w[0][i], a[0]);
            e2m1_to_f16(w[1][i], a[1]);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) a[x][e] = mul_f16x2(a[x][e], sc[x][D == 128 ? i / 2 : 0]);
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    const uint2 q = qs[2 * i + y][nr][lane];
                    mma_f16(s[nr][u], a[0][2 * y], a[1][2 * y], a[0][2 * y + 1], a[1][2 * y + 1], q.x, q.y);
                }
        }
    }

    if constexpr (kMask) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = tg + 4 * (e & 2);
                    if (j >= n_ok[u] || tok0 + 16 * u + j >= acc.lim[nr][e & 1]) s[nr][u][e] = -INFINITY;
                }
    }

    // Running maximum: exchanged and moved only when some score passes its
    // row's threshold.
    bool up = false;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float mx = fmaxf(fmaxf(s[nr][0][r], s[nr][0][r + 2]), fmaxf(s[nr][1][r], s[nr][1][r + 2]));
            up = up || mx > acc.thr[nr][r];
        }
    if (__any_sync(~0u, up)) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            float alpha[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(s[nr][0][r], s[nr][0][r + 2]), fmaxf(s[nr][1][r], s[nr][1][r + 2]));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                mx = fmaxf(mx, acc.m[nr][r]);
                const float ref = mx == -INFINITY ? 0.0f : mx * acc.c[nr][r] - kLift;
                // before a row's first score o and l are 0 and have no reference
                alpha[r] = acc.m[nr][r] == -INFINITY ? 1.0f : ptx::ex2_approx(acc.ref[nr][r] - ref);
                acc.m[nr][r] = mx;
                acc.thr[nr][r] = mx == -INFINITY ? -INFINITY : mx + kSlack / acc.c[nr][r];
                acc.ref[nr][r] = ref;
                acc.l[nr][r] *= alpha[r];
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.o[nr][i][e] *= alpha[e & 1];
        }
    }

    uint32_t pb[NR][2][2];   // P^T as B fragments (k = token, n = row)
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                pr[e] = ptx::ex2_approx(fmaf(s[nr][u][e], acc.c[nr][e & 1], -acc.ref[nr][e & 1]));
                if (kMask && s[nr][u][e] == -INFINITY) pr[e] = 0.0f;
                acc.l[nr][e & 1] += pr[e];
            }
            pb[nr][u][0] = transpose8(ptx::pack2<false>(pr[0], pr[1]));
            pb[nr][u][1] = transpose8(ptx::pack2<false>(pr[2], pr[3]));
        }

    // O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t w[4][D / 64];   // codes of tokens t, 4 + t, 8 + t, 12 + t, elements [g D/8, (g+1) D/8)
        uint32_t sb[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint8_t* src = vc[u] + (t + 4 * x) * (D / 2) + g * (D / 16);
            if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                w[x][0] = v.x; w[x][1] = v.y;
            } else {
                w[x][0] = *reinterpret_cast<const uint32_t*>(src);
            }
            sb[x] = vs[u][(t + 4 * x) * (D / 16) + (D == 128 ? g : g / 2)];
        }
        if constexpr (kMask) {
            // Whatever lies behind the sequence must not enter the product,
            // where 0 * NaN is NaN; and a NaN that some rows see but others
            // do not has to reach only those that do.
            uint32_t nan = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (t + 4 * x >= n_ok[u]) sb[x] = 0;
                if ((sb[x] & 0x7F) == 0x7F) {
                    nan |= 1u << (t + 4 * x);
                    sb[x] = 0;
                }
            }
            nan |= __shfl_xor_sync(~0u, nan, 1);
            nan |= __shfl_xor_sync(~0u, nan, 2);
            if (nan) {
                const int first = tok0 + 16 * u + __ffs(nan) - 1;
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (first < acc.lim[nr][e & 1]) acc.o[nr][i][e] = NAN;
            }
        }
        const uint32_t s01 = e4m3_to_f16(sb[0] | sb[1] << 8), s23 = e4m3_to_f16(sb[2] | sb[3] << 8);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            // Pairs of tokens side by side: even elements, then odd ones.
            uint32_t a[4][4];
            e2m1_to_f16((w[0][i] & 0x0F0F0F0Fu) | ((w[1][i] << 4) & 0xF0F0F0F0u), a[0]);
            e2m1_to_f16(((w[0][i] >> 4) & 0x0F0F0F0Fu) | (w[1][i] & 0xF0F0F0F0u), a[1]);
            e2m1_to_f16((w[2][i] & 0x0F0F0F0Fu) | ((w[3][i] << 4) & 0xF0F0F0F0u), a[2]);
            e2m1_to_f16(((w[2][i] >> 4) & 0x0F0F0F0Fu) | (w[3][i] & 0xF0F0F0F0u), a[3]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t a0 = mul_f16x2(a[0][e], s01), a1 = mul_f16x2(a[1][e], s01);
                const uint32_t a2 = mul_f16x2(a[2][e], s23), a3 = mul_f16x2(a[3][e], s23);
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    mma_f16(acc.o[nr][4 * i + e], a0, a1, a2, a3, pb[nr][u][0], pb[nr][u][1]);
            }
        }
    }
}

// Writes a row's result: o / l * descale and the natural-log sum.
template <int D, bool kBf16>
__device__ __forceinline__ void store_row8(const FwdParams& p, long long row, int d0, const float (&o)[8], float m,
                                           float l, float v_descale) {
    const float f = l == 0.0f ? 0.0f : v_descale / l;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = l == 0.0f ? 0u : ptx::pack2<kBf16>(o[2 * j] * f, o[2 * j + 1] * f);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + row * D + d0) = make_uint4(w[0], w[1], w[2], w[3]);
    if (d0 == 0)
        p.lse[row] = l == 0.0f ? -INFINITY
                               : static_cast<float>((static_cast<double>(m) + static_cast<double>(log2f(l))) * 0.69314718055994530942);
}

template <int D, int NR, bool kBf16>
__global__ void __launch_bounds__(kFwdThreads, NR == 1 ? 4 : 2) fa2_kv4_fwd_kernel(const FwdParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    FwdSmem<D, NR>& sm = *reinterpret_cast<FwdSmem<D, NR>*>(raw);
    constexpr int kRows = 8 * NR;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

    // Requests without a key: O = 0, LSE = -inf.
    for (int b = blockIdx.x; b < p.B; b += gridDim.x)
        if (p.seq_lens[b] <= 0) {
            const long long r0 = static_cast<long long>(b) * p.hkv * p.rows;
            const float none[8] = {};
            for (int i = tid; i < p.hkv * p.rows * (D / 8); i += kFwdThreads)
                store_row8<D, kBf16>(p, r0 + i / (D / 8), i % (D / 8) * 8, none, 0.0f, 0.0f, 0.0f);
        } else if (p.seq_lens[b] > p.max_tokens && tid == 0) {
            report(kSiteLength);
        }

    long long per, total;
    Cursor cur;
    if (!locate(p, false, sm.scan, per, total, cur)) return;

    while (cur.u < cur.end) {
        const int n = static_cast<int>(min(cur.end - cur.u, static_cast<long long>(cur.tiles - cur.tile)));
        const int h = cur.hr / p.rblocks, rb = cur.hr - h * p.rblocks;
        const int len = min(p.seq_lens[cur.b], p.max_tokens);
        stage_q<D, NR, kBf16>(p, sm, cur.b, cur.hr);
        __syncthreads();

        Acc<D, NR> acc;
        int low = len;   // the first key that some row may not see
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.o[nr][i][e] = 0.0f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                acc.m[nr][r] = acc.thr[nr][r] = -INFINITY;
                acc.ref[nr][r] = acc.l[nr][r] = 0.0f;
                acc.c[nr][r] = sm.c[nr * 8 + 2 * t + r];
                const int row = rb * kRows + nr * 8 + 2 * t + r;
                acc.lim[nr][r] = p.causal && row < p.rows ? len - p.nq + row % p.nq + 1 : len;
                low = min(low, acc.lim[nr][r]);
            }
        }
        low = __reduce_min_sync(~0u, low);

        const int* table = p.block_table + static_cast<long long>(cur.b) * p.max_pages;
        for (int i = warp; i < n; i += kWarps) {
            const int tok0 = (cur.tile + i) * kTile;
            const uint8_t *kc[2], *ks[2], *vc[2], *vs[2];
            int n_ok[2];
            bool whole = tok0 + kTile <= low;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int tok = tok0 + 16 * u;
                int pg = -1;
                n_ok[u] = min(16, len - tok);
                if (n_ok[u] > 0) {
                    pg = table[tok >> p.log2_page];
                    if (pg < 0 || pg >= p.num_pages) {
                        report(kSitePage);
                        pg = -1;
                    }
                }
                if (pg < 0) {   // read some page's bytes instead, and use none of them
                    n_ok[u] = 0;
                    whole = false;
                    pg = 0;
                }
                const int at = tok & (p.page - 1);
                kc[u] = p.cache + (static_cast<long long>(pg) * p.hkv + h) * 2 * part_bytes<D>(p.page) + at * (D / 2);
                ks[u] = kc[u] - at * (D / 2) + p.page * (D / 2) + at * (D / 16);
                vc[u] = kc[u] + part_bytes<D>(p.page);
                vs[u] = ks[u] + part_bytes<D>(p.page);
            }
            if (whole) tile_step<D, NR, false>(acc, sm.q, kc, ks, vc, vs, tok0, n_ok);
            else tile_step<D, NR, true>(acc, sm.q, kc, ks, vc, vs, tok0, n_ok);
        }

        // Join the warps' results.
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = acc.l[nr][r];
                l += __shfl_xor_sync(~0u, l, 4);
                l += __shfl_xor_sync(~0u, l, 8);
                l += __shfl_xor_sync(~0u, l, 16);
                const int row = nr * 8 + 2 * t + r;
                if (g == 0) {
                    sm.ml[warp][row][0] = l == 0.0f ? -INFINITY : isnan(acc.ref[nr][r]) ? 0.0f : acc.ref[nr][r];
                    sm.ml[warp][row][1] = l;
                }
                float* dst = &sm.o[warp][row * FwdSmem<D, NR>::kStride + g * (D / 8)];
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    *reinterpret_cast<float2*>(dst + 2 * i) = make_float2(acc.o[nr][i][r], acc.o[nr][i][r + 2]);
            }
        __syncthreads();
        const bool starts = cur.tile == 0, ends = cur.tile + n == cur.tiles;
        const int slot = 2 * blockIdx.x + (starts ? 1 : 0);
        for (int i = tid; i < kRows * (D / 8); i += kFwdThreads) {
            const int row = i / (D / 8), d0 = i % (D / 8) * 8;
            float m = -INFINITY, l = 0.0f, o[8] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.ml[w][row][0]);
            if (m != -INFINITY) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = ptx::ex2_approx(sm.ml[w][row][0] - m);
                    l += f * sm.ml[w][row][1];
                    const float* src = &sm.o[w][row * FwdSmem<D, NR>::kStride + d0];
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = fmaf(f, src[j], o[j]);
                }
            }
            const int r = rb * kRows + row;
            if (starts && ends) {
                if (r < p.rows)
                    store_row8<D, kBf16>(p, (static_cast<long long>(cur.b) * p.hkv + h) * p.rows + r, d0, o, m, l,
                                         p.v_descale[h]);
            } else {
                float* dst = p.part_o + (static_cast<long long>(slot) * kRows + row) * D + d0;
                *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
                if (d0 == 0)
                    *reinterpret_cast<float2*>(p.part_ml + (static_cast<long long>(slot) * kRows + row) * 2) =
                        make_float2(m, l);
            }
        }
        __syncthreads();
        next_segment(p, cur, n);
    }
}

// Joins the partial results of the segments that several CTAs took: block c
// does the segment that starts in CTA c's run and goes on behind its end.
template <int D, int NR, bool kBf16>
__global__ void __launch_bounds__(kFwdThreads) fa2_kv4_join_kernel(const FwdParams p) {
    __shared__ long long scan[kFwdThreads / 32 + 4];
    constexpr int kRows = 8 * NR;
    long long per, total;
    Cursor cur;   // at the last unit of CTA blockIdx.x's run
    if (!locate(p, true, scan, per, total, cur)) return;
    const long long seg0 = cur.u - cur.tile, seg1 = seg0 + cur.tiles;
    const long long run0 = blockIdx.x * per;
    if (seg0 < run0 || seg1 <= run0 + per) return;
    const int c1 = static_cast<int>((seg1 - 1) / per);
    const int h = cur.hr / p.rblocks, rb = cur.hr - h * p.rblocks;
    for (int i = threadIdx.x; i < kRows * (D / 8); i += kFwdThreads) {
        const int row = i / (D / 8), d0 = i % (D / 8) * 8, r = rb * kRows + row;
        if (r >= p.rows) continue;
        float m = -INFINITY, l = 0.0f, o[8] = {};
        for (int c = blockIdx.x; c <= c1; ++c) {
            const int slot = 2 * c + (c == static_cast<int>(blockIdx.x) ? 1 : 0);
            m = fmaxf(m, p.part_ml[(static_cast<long long>(slot) * kRows + row) * 2]);
        }
        if (m != -INFINITY) {
            for (int c = blockIdx.x; c <= c1; ++c) {
                const int slot = 2 * c + (c == static_cast<int>(blockIdx.x) ? 1 : 0);
                const float* ml = p.part_ml + (static_cast<long long>(slot) * kRows + row) * 2;
                const float f = ptx::ex2_approx(ml[0] - m);
                l += f * ml[1];
                const float* src = p.part_o + (static_cast<long long>(slot) * kRows + row) * D + d0;
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = fmaf(f, src[j], o[j]);
            }
        }
        store_row8<D, kBf16>(p, (static_cast<long long>(cur.b) * p.hkv + h) * p.rows + r, d0, o, m, l, p.v_descale[h]);
    }
}

}  // namespace kv4
}  // namespace fa2
