// A paged KV cache held in 4 bits: the kernels that plan its pages, write it,
// read it back and attend over it (sm_103a).
//
// The cache is [num_pages, H_kv, 2, page * (D/2 + D/16)] bytes: of a page and
// KV head first the keys, then the values of `page` tokens, each part as the
// e2m1 codes [page, D/2] followed by one e4m3 scale per 16 elements
// [page, D/16]. Element = code * scale * descale[head]. A product code * scale
// has at most six significant bits and lies in [2^-10, 2688], so it is exact in
// fp16: both matrix products of the attention run on fp16 operands whatever
// the type of q, and the cache costs no precision beyond its own rounding. The
// softmax's weights are the other operand of the second product and become fp16
// too, 2^-11 of each (bf16 would be 2^-8): as fp32 they would take a second
// product for their lower bits.
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

// The kernels of this file are launched so that one may take its place on the
// SMs while the one before it in the stream still runs (programmatic
// dependent launch). Nothing of global memory is touched before that one is
// done and its writes can be seen.
__device__ __forceinline__ void enter_stream_order() {
    asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
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

// For each 16 elements: scale s = e4m3(max|x| / (6 descale)), t = s descale,
// code = e2m1(x / t). A row is 2 D bytes in and 9 D / 16 out. 262112 rows of 128
// of keys and of values (4 prompts of 8191 tokens, 8 heads) take 42 us, 4.1 TB/s,
// 60% of a plain copy's rate: what bounds it is instructions, about 130 for the eight
// elements that a lane has of one part (24 of them quotients), in 71% of the issue
// slots.
struct AppendParams {
    const void* x[2];          // keys, values
    int sb[2], sh[2], sn[2];   // strides in elements: request, head, token
    const float* descale[2];   // [hkv]
    const int* slots;          // [B, N]
    uint8_t* cache;
    int rows;                  // B * hkv * N
    int hkv, n, page, log2_page;
    int num_slots;             // num_pages * page
};

// Eight elements a lane, so that a warp's loads and stores are contiguous:
// 16 bytes of a row, two lanes to a scale. A thread has P rows of keys and of
// values in flight: four where there are enough rows, one where that would
// leave SMs idle.
template <int D, int P>
struct Copy {
    static constexpr int kLanes = D / 8;             // lanes of a row
    static constexpr int kRowsPass = 256 / kLanes;
    static constexpr int kPasses = P;
    static constexpr int kRows = kRowsPass * kPasses;   // rows of a block
};

// Row (b, h, n) of [B, hkv, n], and the row `k` on.
struct Row {
    unsigned b, h, n;
    __device__ __forceinline__ Row(unsigned row, unsigned hkv, unsigned len) {
        const unsigned bh = row / len;
        n = row - bh * len;
        b = bh / hkv;
        h = bh - b * hkv;
    }
    __device__ __forceinline__ void step(unsigned k, unsigned hkv, unsigned len) {
        n += k;
        if (n >= len) {   // most rows are followed by rows of their own sequence: divisions are rare
            const unsigned q = n / len;
            n -= q * len;
            h += q;
            if (h >= hkv) {
                const unsigned r = h / hkv;
                h -= r * hkv;
                b += r;
            }
        }
    }
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Quotients rounded to nearest by Markstein's correction (IBM J. Res. Dev. 34,
// 1990): with r the nearest to 1 / t, q the nearest to x r, and the remainder
// x - q t, which an fma gives exactly, q + remainder * r rounds to the nearest
// of x / t. A tie between two codes (or scales) is common, as inputs and scales
// have few bits, and has to be seen as one. It holds where no step leaves the
// normal numbers: `plain` says so for a divisor and the largest numerator of
// its block, smaller ones giving codes near 0, far from a tie. The divider
// takes the rest.
__device__ __forceinline__ bool plain(float t, float top) {
    return t > 1e-18f && t < 1e18f && top > 1e-18f && top < 1e18f;
}
__device__ __forceinline__ float quotient(float x, float t, float r) {
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, t, x), r, q);
}

template <int D, bool kBf16, int P>
__global__ void __launch_bounds__(256, 4) fa2_kv4_append_kernel(const AppendParams p) {
    enter_stream_order();
    using C = Copy<D, P>;
    const int lane = threadIdx.x % C::kLanes;
    const long long row0 = static_cast<long long>(blockIdx.x) * C::kRows + threadIdx.x / C::kLanes;
    uint4 in[C::kPasses][2];
    int slot[C::kPasses];
    unsigned head[C::kPasses];
    long long at[C::kPasses][2];
    Row r(static_cast<unsigned>(row0), p.hkv, p.n);
#pragma unroll
    for (int i = 0; i < C::kPasses; ++i) {
        slot[i] = -1;
        if (row0 + i * C::kRowsPass < p.rows) slot[i] = p.slots[static_cast<long long>(r.b) * p.n + r.n];
        head[i] = r.h;
#pragma unroll
        for (int part = 0; part < 2; ++part)
            at[i][part] = static_cast<long long>(static_cast<int>(r.b)) * p.sb[part] +
                          static_cast<long long>(static_cast<int>(r.h)) * p.sh[part] +
                          static_cast<long long>(static_cast<int>(r.n)) * p.sn[part] + lane * 8;
        r.step(C::kRowsPass, p.hkv, p.n);
    }
#pragma unroll
    for (int i = 0; i < C::kPasses; ++i) {
        if (slot[i] >= p.num_slots) {
            if (lane == 0) report(kSiteSlot);
            slot[i] = -1;
        }
        in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
        if (slot[i] >= 0)
#pragma unroll
            for (int part = 0; part < 2; ++part)
                in[i][part] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x[part]) + at[i][part]);
    }
    float scales[2], six[2], six_r[2];   // of the head at hand: descale, 6 descale and its reciprocal
    unsigned at_head = ~0u;
#pragma unroll
    for (int i = 0; i < C::kPasses; ++i) {
        if (slot[i] >= 0 && head[i] != at_head) {
            at_head = head[i];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
                scales[part] = p.descale[part][at_head];
                six[part] = 6.0f * scales[part];
                six_r[part] = __frcp_rn(six[part]);
            }
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            const uint4 w = in[i][part];
            // The largest magnitude by its bits, which order NaN above
            // infinity above every finite value.
            uint32_t pair = max_u16x2(max_u16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                                      max_u16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
            pair = max_u16x2(pair, __shfl_xor_sync(~0u, pair, 1));
            if (slot[i] < 0) continue;
            float lo, hi;
            ptx::unpack2<kBf16>(pair, lo, hi);
            const float top = __uint_as_float(max(__float_as_uint(lo), __float_as_uint(hi)));
            const float descale = scales[part];
            uint32_t s8 = 0x7F;   // e4m3 NaN: 16 elements that hold a NaN or an infinity read back as NaN
            uint32_t codes = 0;
            if (__float_as_uint(top) < 0x7F800000u) {
                const float want = plain(six[part], top) ? quotient(top, six[part], six_r[part]) : __fdiv_rn(top, six[part]);
                asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %1, %1;\n\tcvt.u32.u16 %0, a;\n\t}"
                    : "=r"(s8)
                    : "f"(want));
                s8 &= 0xFF;
                float s, other;
                ptx::unpack2<false>(e4m3_to_f16(s8), s, other);
                const float t = __fmul_rn(s, descale);
                if (t > 0.0f) {
                    float x[8];
                    ptx::unpack2<kBf16>(w.x, x[0], x[1]);
                    ptx::unpack2<kBf16>(w.y, x[2], x[3]);
                    ptx::unpack2<kBf16>(w.z, x[4], x[5]);
                    ptx::unpack2<kBf16>(w.w, x[6], x[7]);
                    if (plain(t, top)) {
                        const float r = __frcp_rn(t);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = quotient(x[j], t, r);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], t);
                    }
                    codes = pack8_e2m1(x);
                }
            }
            const int pg = slot[i] >> p.log2_page, off = slot[i] & (p.page - 1);
            uint8_t* dst = p.cache + ((static_cast<long long>(pg) * p.hkv + head[i]) * 2 + part) * part_bytes<D>(p.page);
            *reinterpret_cast<uint32_t*>(dst + off * (D / 2) + lane * 4) = codes;
            if (lane % 2 == 0) dst[p.page * (D / 2) + off * (D / 16) + lane / 2] = static_cast<uint8_t>(s8);
        }
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

// value = code * (scale * descale), rounded once. Bound by memory: 2 x 65536
// tokens of 8 heads of 128 (up to, 105 us) move at 6.1 TB/s, 90% of a plain
// copy's rate. Rows at or past a request's length are zeros.
template <int D, bool kBf16, int P>
__global__ void __launch_bounds__(256) fa2_kv4_gather_kernel(const GatherParams p) {
    enter_stream_order();
    using C = Copy<D, P>;
    const int lane = threadIdx.x % C::kLanes;
    const long long row0 = static_cast<long long>(blockIdx.x) * C::kRows + threadIdx.x / C::kLanes;
    uint32_t codes[C::kPasses][2], scale[C::kPasses][2];
    unsigned head[C::kPasses];
    Row next(static_cast<unsigned>(row0), p.hkv, p.n);
#pragma unroll
    for (int i = 0; i < C::kPasses; ++i) {
        const Row r = next;
        next.step(C::kRowsPass, p.hkv, p.n);
        codes[i][0] = codes[i][1] = scale[i][0] = scale[i][1] = 0;   // reads as zeros
        head[i] = r.h;
        if (row0 + i * C::kRowsPass >= p.rows) continue;
        const long long pos = static_cast<long long>(p.starts ? p.starts[r.b] : 0) + r.n;
        if (pos < 0 || pos >= p.seq_lens[r.b]) continue;
        const long long entry = pos >> p.log2_page;
        const int pg = entry < p.max_pages ? p.block_table[static_cast<long long>(r.b) * p.max_pages + entry] : -1;
        if (pg < 0 || pg >= p.num_pages) {
            if (lane == 0) report(kSitePage);
            continue;
        }
        const int at = static_cast<int>(pos & (p.page - 1));
        const uint8_t* src = p.cache + (static_cast<long long>(pg) * p.hkv + r.h) * 2 * part_bytes<D>(p.page);
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            codes[i][part] = *reinterpret_cast<const uint32_t*>(src + at * (D / 2) + lane * 4);
            scale[i][part] = src[p.page * (D / 2) + at * (D / 16) + lane / 2];
            src += part_bytes<D>(p.page);
        }
    }
#pragma unroll
    for (int i = 0; i < C::kPasses; ++i) {
        const long long row = row0 + i * C::kRowsPass;
        if (row >= p.rows) break;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            float s, other;
            ptx::unpack2<false>(e4m3_to_f16(scale[i][part]), s, other);
            const float t = __fmul_rn(s, p.descale[part][min(head[i], static_cast<unsigned>(p.hkv) - 1)]);
            uint32_t c[4], out[4];
            e2m1_to_f16(codes[i][part], c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo, hi;
                ptx::unpack2<false>(c[e], lo, hi);
                out[e] = ptx::pack2<kBf16>(__fmul_rn(lo, t), __fmul_rn(hi, t));
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[part]) + row * D + lane * 8) =
                make_uint4(out[0], out[1], out[2], out[3]);
        }
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
    int in_place;              // outputs are inputs: the grid is one cluster
};

constexpr int kPlanCtas = 8;   // of a cluster, where there is much to write in place

// Exclusive prefix sums of (a, r) over the block's T threads, and the totals.
template <int T>
__device__ __forceinline__ void block_scan2(long long& a, long long& r, long long& a_all, long long& r_all,
                                            long long (*sm)[T / 32]) {
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
    if (lane == 31) {
        sm[0][warp] = ia;
        sm[1][warp] = ir;
    }
    __syncthreads();
    // every warp scans the warps' sums for itself
    const long long wa = lane < T / 32 ? sm[0][lane] : 0, wr = lane < T / 32 ? sm[1][lane] : 0;
    long long sa = wa, sr = wr;
#pragma unroll
    for (int o = 1; o < T / 32; o <<= 1) {
        const long long ta = __shfl_up_sync(~0u, sa, o), tr = __shfl_up_sync(~0u, sr, o);
        if (lane >= o) {
            sa += ta;
            sr += tr;
        }
    }
    a_all = __shfl_sync(~0u, sa, T / 32 - 1);
    r_all = __shfl_sync(~0u, sr, T / 32 - 1);
    a = __shfl_sync(~0u, sa - wa, warp) + ia - a;
    r = __shfl_sync(~0u, sr - wr, warp) + ir - r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Where in the ring the page lies that comes `at` places behind page 0's.
__device__ __forceinline__ int ring_place(long long at, int num_pages) {
    if (at >= num_pages) at -= num_pages;   // below 3 num_pages in a sane ring
    if (at >= num_pages) at -= num_pages;
    if (at >= num_pages) at %= num_pages;
    return static_cast<int>(at);
}

// Writes the pages of the n requests at table row `rows` that end into the ring from
// place `behind` on without the ids outside the cache among them, the pages
// behind such an id moving up; returns how many pages there are. A call of its
// own, for a table that holds such an id. s_page is unused by requests that end.
template <int T>
__device__ __noinline__ long long release_usable(const int* rows, int* free_pages, int max_pages, int log2_page, int num_pages, int n,
                                                 const int* s_len, const int* s_add, int* s_page, int* s_back,
                                                 long long (*sm)[T / 32], long long behind) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int pass = 0; pass < 2; ++pass) {   // counts them, then writes them
        for (int q = warp; q < n; q += T / 32) {
            if (s_add[q] >= 0) continue;
            const int have = (s_len[q] + (1 << log2_page) - 1) >> log2_page;
            const int* row = rows + static_cast<long long>(q) * max_pages;
            int kept = 0;
            for (int j = lane; j < (have + 31) / 32 * 32; j += 32) {
                const int id = j < have ? row[j] : -1;
                const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(num_pages);
                const unsigned mask = __ballot_sync(~0u, good);
                if (pass && good)
                    free_pages[ring_place(static_cast<long long>(s_back[q]) + kept + __popc(mask & ((1u << lane) - 1)), num_pages)] = id;
                kept += __popc(mask);
            }
            if (!pass && lane == 0) s_page[q] = kept;
        }
        if (pass) break;
        __syncthreads();
        long long kept = tid < n && s_add[tid] < 0 ? s_page[tid] : 0, none = 0, all, unused;
        block_scan2<T>(kept, none, all, unused, sm);
        s_back[tid] = ring_place(behind + kept, num_pages);
        __syncthreads();
        if (tid == 0) sm[0][0] = all;   // every thread's copy need not live through the second pass
    }
    __syncthreads();
    return sm[0][0];
}

// Every CTA scans the requests in order, T at a time, so that each knows where
// every request's pages lie in the ring; then they share the writing. Where
// outputs are the inputs the CTAs are one cluster, whose barrier lies between. A
// request gets its pages iff the pages wanted up to and including it are free
// (or it needs none); pages of requests that end join the ring behind its last
// page and are not handed out by this call. Bound by latency, three dependent
// reads, and by the launch: 2.9 us for a step of 256 requests, 5.1 us where 6% of
// them end; 5.2 us for 48 prompts of 16384 tokens (3.4 MB), 20.9 us in place.
template <int T>
__global__ void __launch_bounds__(T) fa2_kv4_plan_kernel(const PlanParams p) {
    __shared__ long long sm[2][T / 32];
    __shared__ int s_len[T], s_add[T], s_page[T], s_back[T];
    enter_stream_order();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = blockIdx.x, ranks = gridDim.x;
    int first = p.free_state[0], count = p.free_state[1];
    if (first < 0 || first >= p.num_pages || count < 0 || count > p.num_pages) {
        if (tid == 0 && rank == 0) report(kSitePool);
        first = 0;
        count = 0;
    }
    const long long room = static_cast<long long>(p.max_pages) << p.log2_page;
    // pages wanted by the requests before this chunk, handed out to them, and returned by them
    long long want = 0, taken = 0, back = 0;
    for (int b0 = 0; b0 < p.B; b0 += T) {
        const int n = min(T, p.B - b0), b = b0 + tid;
        int len = 0, add = 0;
        const bool in = tid < n;
        if (in) {
            len = p.seq_lens[b];
            add = p.new_lens[b];
            if (len < 0 || len > room) {
                if (rank == 0) report(kSiteLength);
                len = 0;
            }
        }
        const bool ends = in && add < 0;
        const bool fits = in && !ends && add <= p.n && static_cast<long long>(len) + add <= room;
        const int have = (len + p.page - 1) >> p.log2_page;
        const int need = fits ? static_cast<int>((static_cast<long long>(len) + add + p.page - 1) >> p.log2_page) - have : 0;
        long long a = need, r = ends ? have : 0, a_all, r_all;
        block_scan2<T>(a, r, a_all, r_all, sm);
        const bool granted = fits && (need == 0 || want + a + need <= count);
        s_len[tid] = len;
        s_add[tid] = ends ? -1 : granted ? add : 0;
        s_page[tid] = granted ? static_cast<int>(first + want + a) : 0;   // of its first new page in the ring; < 2 num_pages if it has one
        s_back[tid] = ring_place(first + static_cast<long long>(count) + back + r, p.num_pages);
        // those that got pages are the first of those that wanted any
        taken = want + a_all <= count ? want + a_all : taken;
        const bool cut = want <= count && want + a_all > count;
        if (cut) {
            long long got = granted ? need : 0, none = 0, unused;
            __syncthreads();
            block_scan2<T>(got, none, taken, unused, sm);
            taken += want;
        }
        want += a_all;
        __syncthreads();
        if (p.in_place) cluster_sync();

        if (rank == 0 && in) {
            p.seq_lens_out[b] = ends ? 0 : len + (granted ? add : 0);
            p.accepted[b] = granted ? add : 0;
        }
        // Slots, and the table entries of the pages that begin among them. A
        // slot's page comes from the table, or from the ring if it is new.
        int* slots = p.slots + static_cast<long long>(b0) * p.n;
        auto page_at = [&](int rb, int len, int entry) -> const int* {
            const int had = (len + p.page - 1) >> p.log2_page;
            if (entry < had) return p.block_table + static_cast<long long>(b0 + rb) * p.max_pages + entry;
            const int k = s_page[rb] + entry - had;
            return p.free_pages + (k >= p.num_pages ? k - p.num_pages : k);
        };
        if (p.n >= 256) {
            // Long rows: a warp takes 256 slots of one request. They lie in 17
            // pages at most, whose ids the lanes read and then pass around.
            const unsigned pieces = (p.n + 255) / 256, all = n * pieces;
            for (unsigned q = rank * (T / 32) + warp; q < all; q += ranks * (T / 32)) {
                const int rb = q / pieces, i0 = (q - rb * pieces) * 256, got = s_add[rb] - i0, start = s_len[rb] + i0;
                const int entry0 = start >> p.log2_page;
                int pg = -1;
                if (got > 0 && entry0 + lane <= (start + min(got, 256) - 1) >> p.log2_page) {
                    pg = *page_at(rb, s_len[rb], entry0 + lane);
                    // a page that begins behind the cached tokens is a new one
                    if ((entry0 + lane) << p.log2_page >= start)
                        p.block_table[static_cast<long long>(b0 + rb) * p.max_pages + entry0 + lane] = pg;
                    if (pg < 0 || pg >= p.num_pages) {
                        report(kSitePage);
                        pg = -1;
                    }
                }
                int* to = slots + static_cast<long long>(rb) * p.n + i0;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int i = 32 * j + lane, pos = start + i;
                    const int page_of = __shfl_sync(~0u, pg, ((pos >> p.log2_page) - entry0) & 31);
                    if (i0 + i < p.n)
                        to[i] = i < got && page_of >= 0 ? (page_of << p.log2_page) + (pos & (p.page - 1)) : -1;
                }
            }
        } else {
            const unsigned total = static_cast<unsigned>(n) * static_cast<unsigned>(p.n);
            const unsigned stride = ranks * T, sb = stride / p.n, si = stride - sb * p.n;
            unsigned e = rank * T + tid, rb = e / p.n, i = e - rb * p.n;
            for (; e < total; e += stride) {
                int slot = -1;
                if (static_cast<int>(i) < s_add[rb]) {
                    const int pos = s_len[rb] + static_cast<int>(i), off = pos & (p.page - 1), entry = pos >> p.log2_page;
                    const int pg = *page_at(rb, s_len[rb], entry);
                    if (off == 0) p.block_table[static_cast<long long>(b0 + rb) * p.max_pages + entry] = pg;
                    if (pg >= 0 && pg < p.num_pages) slot = (pg << p.log2_page) + off;
                    else report(kSitePage);
                }
                slots[e] = slot;
                rb += sb;
                i += si;
                if (i >= static_cast<unsigned>(p.n)) {
                    i -= p.n;
                    ++rb;
                }
            }
        }
        // Pages of requests that end, a warp each, by the CTA that also writes
        // the ring's state. An id outside the cache is reported and does not join the
        // ring; it is seen when the others have been written, which is then done again.
        bool odd = false;
        if (r_all > 0 && rank == 0) {
            unsigned seen = 0, turn = warp;   // requests that end, so far; the next that is this warp's
            for (int q0 = 0; q0 < n; q0 += 32) {
                unsigned who = __ballot_sync(~0u, q0 + lane < n && s_add[min(q0 + lane, T - 1)] < 0);
                for (; who; who &= who - 1, ++seen) {
                    if (seen != turn) continue;
                    turn += T / 32;
                    const int q = q0 + __ffs(who) - 1, have_q = (s_len[q] + p.page - 1) >> p.log2_page;
                    const int* row = p.block_table + static_cast<long long>(b0 + q) * p.max_pages;
                    for (int j0 = lane; j0 < have_q; j0 += 128) {
                        int pg[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j0 + 32 * j < have_q) pg[j] = row[j0 + 32 * j];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j0 + 32 * j < have_q) {
                                int k = s_back[q] + j0 + 32 * j;
                                if (k >= p.num_pages) k -= p.num_pages;
                                if (k >= p.num_pages) k %= p.num_pages;   // more pages than there are
                                p.free_pages[k] = pg[j];
                                odd |= static_cast<unsigned>(pg[j]) >= static_cast<unsigned>(p.num_pages);
                            }
                    }
                }
            }
        }
        if (__syncthreads_or(odd)) {
            if (tid == 0) report(kSitePage);
            r_all = release_usable<T>(p.block_table + static_cast<long long>(b0) * p.max_pages, p.free_pages, p.max_pages, p.log2_page,
                                      p.num_pages, n, s_len, s_add, s_page, s_back, sm, first + static_cast<long long>(count) + back);
            __syncthreads();
        }
        back += r_all;
    }
    if (tid == 0 && rank == 0) {
        long long left = count - taken + back;
        if (left > p.num_pages) {   // more pages came back than were out
            report(kSitePool);
            left = p.num_pages;
        }
        p.free_state_out[0] = static_cast<int>(first + taken >= p.num_pages ? first + taken - p.num_pages : first + taken);
        p.free_state_out[1] = static_cast<int>(left);
    }
}

// ------------------------------------------------------------------ attention

constexpr int kTile = 32;      // tokens a warp takes at a time
constexpr int kMaxCtas = 320;  // workspace is sized for this many
// Tiles of 32 that a CTA's run has at least. With 64, one request of 4096 tokens and
// 8 heads takes 15.8 us instead of 12.2. With 16, one of 2304 takes 10.0 us instead of
// 14.6, but one of 8192 with 64 rows a head 41.7 instead of 37.6, and 16 requests of up
// to 2304 with 64 rows 56 instead of 44.
constexpr int kMinRun = 32;
// Tiles by which a run may grow so that no segment is split. With none, 256 segments of
// up to 2304 tokens, heads of 64, take 20.7 us instead of 15.7, and 128 with 20 rows
// 34 instead of 22.7; a few segments pay for it: 8 of 2304 tokens take 14.6 us, 12.0
// with none. With 96, 8 of 4096 take 22 us instead of 12.2.
constexpr int kSpare = 40;
// Partial results that are joined at once. With 6, ten parts of 20 rows (16 heads of
// 65536 tokens) take 64.0 us instead of 62.2; with 24, 19 parts (8 heads) 40.5 instead of
// 39.0, although of 8 rows (16 heads) 36.4 instead of 37.3.
constexpr int kJoinAtOnce = 12;

// Attention for up to 24 query rows a KV head, NR blocks of eight: both
// products on mma.sync, transposed (S^T = K Q^T, O^T += V^T P^T), so that tokens
// and elements of d fill the 16 rows of an instruction and the query rows its 8
// columns. The codes become fp16 in registers, a lane reading those that its own
// fragments hold, and no other lane's: nothing goes back to shared memory. Each
// warp has tiles of its own and runs its own online softmax (l, reference); warps
// and CTAs are joined at the end of a segment.
//
// What bounds it: at 8 rows memory. 64 sequences of 32768 tokens, 8 heads of 128 (as
// drawn, 1.56 GB) take 253 us, 6.15 TB/s, 91% of a plain copy's rate; issue slots
// are 64% busy. Above, the issue of instructions that wait for one another:
// 38 sequences of 8192 tokens (358 MB) take 63, 89 and 110 us for 8, 16 and 24 rows,
// where the tensor pipe is busy for 27, 37 and 44% of the time with 16, 8 and 8
// warps an SM, which is what the accumulators leave registers for. Twelve warps
// spill and are slower; two warps on one tile, half of d each, take 111 us
// for 16 rows; both halves of a tile one after the other are slower too.

// Warps a CTA and CTAs an SM by the rows a pass over the keys serves: what
// the accumulators leave room for in the registers.
template <int NR>
struct Shape {
    static constexpr int kWarps = 8;
    static constexpr int kCtas = NR == 1 ? 2 : 1;
    static constexpr int kThreads = 32 * kWarps;
};

struct FwdParams {
    const void* q;             // [B, H_q, N_q, D]: `rows` contiguous rows a KV head
    const uint8_t* cache;
    const float* k_descale;    // [hkv]
    const float* v_descale;
    const int* seq_lens;       // [B]
    const int* block_table;    // [B, max_pages]
    void* o;
    float* lse;
    float* part_o;             // [2 * ctas, rows of a block, D]
    float* part_ml;            // [2 * ctas, rows of a block, 2]: reference, sum
    unsigned long long* arrived;  // [2 ctas]: of a segment by its first CTA, of a group of CTAs by its first
    unsigned long long nonce;  // of this launch, low 16 bits 0
    int B, hkv, nq, rows, rblocks;   // rows = group * N_q; rblocks: blocks of them
    int max_pages, max_tokens, page, log2_page, num_pages;
    int part, page_bytes;      // bytes of keys (or values) of a head's page, of a page of all heads
    int causal;
    int ctas;                  // CTAs that take work
    int idle;                  // CTAs that write the zeros of a request without a key
    float scale_log2;
    long long wait_limit_ns;   // of a wait for the tensor cores
    int debug_flags;
};

// fp32 accumulators += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into accumulators that were zero.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// The transpose of an 8 x 8 matrix of 16-bit elements held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Shared-memory loads at 32-bit addresses.
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The work: the tiles of every (request, KV head, row block), in that order,
// as one line of units cut into equal runs, one a CTA: every CTA has the same
// amount whatever the lengths, which only the device knows. A run may end
// inside a segment (the tiles of one row block); its CTAs then leave partial
// results, and the last of them to finish joins them. Where the segments are
// so few that each CTA can begin one at its own run's start, the segments are
// padded to whole runs (`pad` = per, else 1), so that no CTA has two.
struct Cursor {
    int u, end;                // first unit of the segment's part in this run, end of the run
    int b, hr, tile;           // request, head * rblocks + row block, first tile of the part
    int len, tiles;            // the request's tokens and tiles
};

__device__ __forceinline__ int length_of(const FwdParams& p, int b) { return min(max(p.seq_lens[b], 0), p.max_tokens); }
// Tiles of 2^L tokens.
template <int L>
__device__ __forceinline__ int tiles_in(int len) {
    return (len >> L) + ((len & ((1 << L) - 1)) != 0);
}
// `tiles` rounded up to whole runs of `pad`, of which there are fewer than
// 2^20; inv = 1 / pad.
__device__ __forceinline__ int padded(int tiles, int pad, float inv) {
    if (pad == 1) return tiles;
    int n = static_cast<int>(static_cast<float>(tiles) * inv);   // off by one at most
    n += n * pad < tiles;
    n -= (n - 1) * pad >= tiles;
    return n * pad;
}
__device__ __forceinline__ int padded(int tiles, int pad) { return (tiles + pad - 1) / pad * pad; }

__device__ __forceinline__ int warp_scan(int x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

// The start of this CTA's run; false if it has none. Every warp finds it for
// itself, a lane looking at its share of the requests: no barrier.
template <int W, int L>
__device__ __forceinline__ bool locate(const FwdParams& p, Cursor& cur, int& per, int& pad) {
    const int lane = threadIdx.x & 31;
    const int chunk = (p.B + 31) >> 5;
    const int b0 = min(lane * chunk, p.B), b1 = min(b0 + chunk, p.B);
    const int hrs = p.hkv * p.rblocks;
    int mine = 0, longest = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
        const int t = tiles_in<L>(length_of(p, b));
        mine += t;
        longest = max(longest, t);
    }
    int to = warp_scan(mine);
    int total = __shfl_sync(~0u, to, 31) * hrs;
    if (total == 0) return false;
    longest = __reduce_max_sync(~0u, longest);
    per = max((total + p.ctas - 1) / p.ctas, kMinRun >> (L - 5));
    per = (per + W - 1) / W * W;
    pad = 1;
    float inv = 1.0f;
    if (p.B * hrs <= p.ctas) {
        // Every segment could have a CTA of its own, which is worth a
        // somewhat longer run: nothing to join, no second segment.
        if (longest <= per + (kSpare >> (L - 5))) per = max(per, (longest + W - 1) / W * W);
        inv = 1.0f / static_cast<float>(per);
        int mine_p = 0;
        for (int b = b0; b < b1; ++b) mine_p += padded(tiles_in<L>(length_of(p, b)), per, inv);
        const int to_p = warp_scan(mine_p), total_p = __shfl_sync(~0u, to_p, 31) * hrs;
        if (total_p <= p.ctas * per) {
            pad = per;
            total = total_p;
            to = to_p;
            mine = mine_p;
        } else {
            inv = 1.0f;
        }
    }
    const int u = static_cast<int>(blockIdx.x) * per;
    if (u >= total) return false;
    int at = (to - mine) * hrs, b = b0, len = 0;   // the lane's first unit
    const bool here = u >= at && u < to * hrs;
    if (here) {
        while (true) {
            len = length_of(p, b);
            const int t = padded(tiles_in<L>(len), pad, inv) * hrs;
            if (u < at + t) break;
            at += t;
            ++b;
        }
    }
    const int from = __ffs(__ballot_sync(~0u, here)) - 1;
    cur.u = u;
    cur.end = min(total, u + per);
    cur.b = __shfl_sync(~0u, b, from);
    cur.len = __shfl_sync(~0u, len, from);
    cur.tiles = tiles_in<L>(cur.len);
    const int rem = u - __shfl_sync(~0u, at, from), seg = padded(cur.tiles, pad, inv);
    cur.hr = rem / seg;
    cur.tile = rem - cur.hr * seg;
    return true;
}

// Units and tiles of the cursor's part of its segment.
__device__ __forceinline__ int part_units(const Cursor& c, int pad) {
    return min(c.end - c.u, (pad == 1 ? c.tiles : padded(c.tiles, pad)) - c.tile);
}
__device__ __forceinline__ int part_tiles(const Cursor& c) { return min(c.end - c.u, c.tiles - c.tile); }

// To the next segment of the run; at its end, to a place without tiles.
template <int L>
__device__ __forceinline__ void next_segment(const FwdParams& p, Cursor& c, int pad) {
    c.u += part_units(c, pad);
    c.tile = 0;
    if (c.u >= c.end) return;
    if (++c.hr == p.hkv * p.rblocks) {
        c.hr = 0;
        do {
            c.len = length_of(p, ++c.b);
        } while (c.len == 0);
        c.tiles = tiles_in<L>(c.len);
    }
}

// A tile of 32 tokens in shared memory: key codes, value codes, key scales,
// value scales. Rows of value codes are placed so that the four rows two
// apart that a warp reads at once (values of tokens 2t, t = 0 .. 3) lie in
// different banks: rows in natural order would put all of them into the same.
template <int D>
struct Tile {
    static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / 16;
    static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales;
    // Place of 16-byte piece c of value row r.
    static __device__ __forceinline__ int v_at(int r, int c) {
        if constexpr (D == 128) {
            const int line = r >> 1;
            return line * 128 + (((r & 1) ^ (line & 1)) * 64) + ((c ^ (line & 2)) * 16);
        } else {
            const int line = r >> 2;
            return line * 128 + (((r & 3) ^ (line & 1)) * 32) + c * 16;
        }
    }
};

template <int D, int NR>
struct FwdSmem {
    static constexpr int kWarps = Shape<NR>::kWarps;
    static constexpr int kRows = 8 * NR;
    static constexpr int kStages = NR == 1 ? 2 : 3;
    static constexpr int kStride = D + 4;    // floats a row of the merge buffer
    alignas(16) uint8_t ring[kWarps][kStages][Tile<D>::kBytes];
    float o[kWarps][8 * kStride];            // eight rows of every warp's result; the join's weights
    uint4 raw[kRows][D / 8 + 1];             // the next segment's rows of q, as they are; padded against bank conflicts
    uint2 q[D / 16][NR][32];                 // B fragments of q
    float c[kRows];                          // log2(e) * scale * descale, with q's power of two taken out
    int off[kRows];                          // keys at the sequence's end that the row may not see
    float ml[kWarps][kRows][2];
    float row_ml[kRows][2];
    unsigned long long seen[2];              // the segment's and the group's counter, as they were when the segment began
    int last;
};

// Queues the copy of a segment's rows of q (rows that do not exist: zeros).
template <int D, int NR>
__device__ __forceinline__ void load_q(const FwdParams& p, FwdSmem<D, NR>& sm, int b, int hr) {
    const int h = hr / p.rblocks, r0 = (hr - h * p.rblocks) * 8 * NR;
    const uint8_t* src = static_cast<const uint8_t*>(p.q) + ((static_cast<long long>(b) * p.hkv + h) * p.rows + r0) * (2 * D);
    for (int i = threadIdx.x; i < 8 * NR * (D / 8); i += Shape<NR>::kThreads) {
        const int r = i / (D / 8), c = i % (D / 8);
        if (r0 + r < p.rows) copy16(ptx::smem_addr(&sm.raw[r][c]), src + r * (2 * D) + c * 16);
        else sm.raw[r][c] = make_uint4(0, 0, 0, 0);
    }
}

// Rows of q as B fragments of Q^T (k = d, n = row), in fp16. A bf16 row is
// scaled by the power of two that brings its largest magnitude into
// [2^14, 2^15): its elements' 8 bits stay as they are down to 2^-17, 2^-31 of that
// magnitude; below they become multiples of 2^-24, off by 2^-39 of it at most.
// Thread (g, t) of a warp takes row g and elements
// [t D/4, (t + 1) D/4): the order of d inside a product is free, and this one
// lets a thread read a key's codes as one piece.
template <int D, int NR, bool kBf16>
__device__ __forceinline__ void stage_q(const FwdParams& p, FwdSmem<D, NR>& sm, int hr, float k_descale) {
    const int nr = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (nr >= NR) return;
    uint32_t w[D / 8];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
        const uint4 v = sm.raw[nr * 8 + g][t * (D / 32) + j];
        w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
    }
    float c = p.scale_log2 * k_descale;
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
    if (t == 0) {
        const int row = hr % p.rblocks * 8 * NR + nr * 8 + g;
        sm.c[nr * 8 + g] = c;
        sm.off[nr * 8 + g] = p.causal && row < p.rows ? p.nq - 1 - row % p.nq : 0;
    }
}

// Where a thread (g, t) finds its pieces of a tile: byte offsets of keys g,
// values 2t and 2t + 1 and their scales, each with those of the other tokens
// a fixed distance away; and the addresses of its q fragments and row factors.
template <int D>
struct Lane {
    uint32_t k, ks, v[2], vs, q, c;
    template <int NR>
    __device__ __forceinline__ void set(const FwdSmem<D, NR>& sm) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        k = g * (D / 2) + t * (D / 8);
        ks = Tile<D>::kKs + g * (D / 16) + t * (D / 64);
#pragma unroll
        for (int x = 0; x < 2; ++x)
            v[x] = Tile<D>::kV + Tile<D>::v_at(2 * t + x, g * (D / 16) / 16) + g * (D / 16) % 16;
        vs = Tile<D>::kVs + 2 * t * (D / 16) + (D == 128 ? g : g / 2);
        q = ptx::smem_addr(&sm.q[0][0][lane]);
        c = ptx::smem_addr(&sm.c[2 * t]);
    }
};

// What a warp carries along a segment: unnormalised O^T as accumulators
// (thread (g, t): d in [g D/8, (g + 1) D/8), rows 2t and 2t + 1 of each eight)
// and per row the reference of the exponentials.
template <int D, int NR>
struct Acc {
    float o[NR][D / 16][4];
    float ref[NR][2];      // exponentials are 2^(s c - ref); -inf before the first score
    float l[NR][2];        // this thread's part of the row sums
};

// Exponentials reach 2^15 at most (fp16 holds 65504): 2^7 at the maximum that
// set the reference, and scores may pass that by 2^8 before it moves, which
// spares most tiles the exchange of maxima and the rescaling.
constexpr float kLift = 7.0f, kTop = 15.0f;

// One tile of 32 tokens from `tok0`, in shared memory at `tile`. kMask: some
// row may not see all of them, or a half's tokens are not all usable (it ends
// behind the sequence or lies on a bad page): n_ok[u] of its 16 are.
template <int D, int NR, bool kMask>
__device__ __forceinline__ void tile_step(Acc<D, NR>& acc, const FwdSmem<D, NR>& sm, const Lane<D>& ln, uint32_t tile,
                                          int tok0, int len, const int (&n_ok)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[NR][2][4];

    // S^T = K Q^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t w[2][D / 32];   // codes of tokens g and 8 + g, elements [t D/4, (t+1) D/4)
        uint32_t sc[2][2];       // their scales, twice each
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t at = tile + ln.k + (16 * u + 8 * x) * (D / 2), sat = tile + ln.ks + (16 * u + 8 * x) * (D / 16);
            if constexpr (D == 128) {
                const uint4 v = lds128(at);
                w[x][0] = v.x; w[x][1] = v.y; w[x][2] = v.z; w[x][3] = v.w;
                const uint32_t two = e4m3_to_f16(lds16(sat));
                sc[x][0] = __byte_perm(two, 0, 0x1010);
                sc[x][1] = __byte_perm(two, 0, 0x3232);
            } else {
                const uint2 v = lds64(at);
                w[x][0] = v.x; w[x][1] = v.y;
                sc[x][0] = sc[x][1] = e4m3_to_f16(__byte_perm(lds8(sat), 0, 0x4400));
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
                    const uint2 q = lds64(ln.q + ((2 * i + y) * NR + nr) * 256);
                    if (i == 0 && y == 0)
                        mma_f16_first(s[nr][u], a[0][0], a[1][0], a[0][1], a[1][1], q.x, q.y);
                    else
                        mma_f16(s[nr][u], a[0][2 * y], a[1][2 * y], a[0][2 * y + 1], a[1][2 * y + 1], q.x, q.y);
                }
        }
    }

    // Exponents; the reference moves only when some score passes it by too much.
    float c[NR][2];
    bool hide[NR][2][4];
    float top = -INFINITY;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
        const uint2 two = lds64(ln.c + nr * 32);
        c[nr][0] = __uint_as_float(two.x);
        c[nr][1] = __uint_as_float(two.y);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kMask) {
                    const int j = g + 4 * (e & 2);
                    hide[nr][u][e] = j >= n_ok[u] || tok0 + 16 * u + j >= len - sm.off[nr * 8 + 2 * t + (e & 1)];
                    if (hide[nr][u][e]) s[nr][u][e] = -INFINITY;
                }
                const float x = fmaf(s[nr][u][e], c[nr][e & 1], -acc.ref[nr][e & 1]);
                if (!kMask || !hide[nr][u][e]) top = fmaxf(top, x);
            }
    }
    if (__any_sync(~0u, top > kTop)) {
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            float alpha[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float mx = fmaxf(fmaxf(s[nr][0][r], s[nr][0][r + 2]), fmaxf(s[nr][1][r], s[nr][1][r + 2]));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 16));
                const float old = acc.ref[nr][r];
                const float ref = mx == -INFINITY ? old : fmaxf(old, fmaf(mx, c[nr][r], -kLift));
                // before a row's first score o and l are 0 and have no reference
                alpha[r] = old == -INFINITY ? 1.0f : ptx::ex2_approx(old - ref);
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
                pr[e] = ptx::ex2_approx(fmaf(s[nr][u][e], c[nr][e & 1], -acc.ref[nr][e & 1]));
                if (kMask && hide[nr][u][e]) pr[e] = 0.0f;
                acc.l[nr][e & 1] += pr[e];
            }
            pb[nr][u][0] = transpose8(ptx::pack2<false>(pr[0], pr[1]));
            pb[nr][u][1] = transpose8(ptx::pack2<false>(pr[2], pr[3]));
        }

    // O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t w[4][D / 64];   // codes of tokens 2t, 2t + 1, 2t + 8, 2t + 9, elements [g D/8, (g+1) D/8)
        uint32_t sb[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const uint32_t at = tile + ln.v[x & 1] + (16 * u + 8 * (x >> 1)) * (D / 2);
            if constexpr (D == 128) {
                const uint2 v = lds64(at);
                w[x][0] = v.x; w[x][1] = v.y;
            } else {
                w[x][0] = lds32(at);
            }
            sb[x] = lds8(tile + ln.vs + (16 * u + 8 * (x >> 1) + (x & 1)) * (D / 16));
        }
        if constexpr (kMask) {
            // Whatever lies behind the sequence must not enter the product,
            // where 0 * NaN is NaN; and a NaN that some rows see but others
            // do not has to reach only those that do.
            uint32_t nan = 0;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int j = 8 * (x >> 1) + 2 * t + (x & 1);
                if (j >= n_ok[u]) sb[x] = 0;
                if ((sb[x] & 0x7F) == 0x7F) {
                    nan |= 1u << j;
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
                            if (first < len - sm.off[nr * 8 + 2 * t + (e & 1)]) acc.o[nr][i][e] = NAN;
            }
        }
        const uint32_t s01 = e4m3_to_f16(__byte_perm(sb[0], sb[1], 0x5540)), s23 = e4m3_to_f16(__byte_perm(sb[2], sb[3], 0x5540));
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

// Writes four elements of a row's result, o / l * descale, and the
// natural-log sum.
template <int D, bool kBf16>
__device__ __forceinline__ void store_row4(const FwdParams& p, long long row, int d0, const float4& o, float m, float l,
                                           float v_descale) {
    const float f = v_descale / l;
    uint2 w = make_uint2(0, 0);
    if (l != 0.0f) w = make_uint2(ptx::pack2<kBf16>(o.x * f, o.y * f), ptx::pack2<kBf16>(o.z * f, o.w * f));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + d0) = w;
    if (d0 == 0) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

// Requests without a key: O = 0, LSE = -inf, by the T threads of `idle` CTAs a
// request. Lengths behind the table's end are reported here too. A call, so
// that the registers of the tiles' loop are not chosen with this in sight: 152
// sequences of 8192 tokens take 231 us either way, one of 512 tokens 7.2 us, inlined
// 6.8 us.
template <int D, bool kBf16, int T>
__device__ __noinline__ void idle_requests(const FwdParams& p) {
    for (int w = blockIdx.x; w < p.B * p.idle; w += gridDim.x) {
        const int b = p.idle == 1 ? w : w / p.idle, share = w - b * p.idle;
        const int len = p.seq_lens[b];
        if (len <= 0) {
            const long long rows = static_cast<long long>(p.hkv) * p.rows;
            for (long long i = share * T + threadIdx.x; i < rows * (D / 4); i += p.idle * T)
                store_row4<D, kBf16>(p, b * rows + i / (D / 4), static_cast<int>(i % (D / 4)) * 4, make_float4(0, 0, 0, 0),
                                     0.0f, 0.0f, 0.0f);
        } else if (len > p.max_tokens && threadIdx.x == 0) {
            report(kSiteLength);
        }
    }
}

__device__ __forceinline__ void axpy4(float4& y, float a, const float4& x) {
    y.x = fmaf(a, x.x, y.x);
    y.y = fmaf(a, x.y, y.y);
    y.z = fmaf(a, x.z, y.z);
    y.w = fmaf(a, x.w, y.w);
}

// A warp's tiles of a segment, loaded ahead of the computation into its own
// ring; the first of the next segment are on their way while the results of
// one are joined. Page ids are read one tile ahead of the copies that need
// them. A copy's lanes take neighbouring 16-byte pieces; the addresses of a
// half's 16 tokens differ by constants.
template <int D, int W>
struct Loader {
    const uint8_t* codes;      // cache + the head's offset inside a page + the lane's piece of its codes
    const uint8_t* scales;     // the same for the piece of scales that the lane copies
    const int* table;          // the request's row
    uint32_t k_dst, v_dst, s_dst;   // places of the lane's pieces in a tile
    int tile, end, len;        // the warp's next tile, end of the part, the request's tokens
    int pg[2];                 // pages of its halves

    static constexpr int kEach = Tile<D>::kScales / 16;   // pieces of a tile's key scales

    __device__ __forceinline__ void start() {
        const int lane = threadIdx.x & 31;
        constexpr int kPieces = D / 32;   // of a token's codes
        k_dst = lane * 16;
        v_dst = Tile<D>::kV + Tile<D>::v_at(lane / kPieces, lane % kPieces);
        s_dst = Tile<D>::kKs + lane * 16;
    }

    __device__ __forceinline__ void enter(const FwdParams& p, const Cursor& c) {
        const int lane = threadIdx.x & 31;
        codes = p.cache + static_cast<long long>(c.hr / p.rblocks) * 2 * p.part;
        scales = codes + (lane >= kEach ? p.part : 0) + p.page * (D / 2) + lane % kEach * 16;
        codes += lane * 16;
        table = p.block_table + static_cast<long long>(c.b) * p.max_pages;
        len = c.len;
        tile = c.tile + (threadIdx.x >> 5);
        end = c.tile + part_tiles(c);
        look(p);
    }

    __device__ __forceinline__ void look(const FwdParams& p) {
        if (tile < end) {
            const int at = tile * kTile;
            pg[0] = table[at >> p.log2_page];
            if (p.page < kTile) pg[1] = at + 16 < len ? table[(at + 16) >> p.log2_page] : -1;
        }
    }

    // Queues the copies of the next tile (none behind the last) and closes
    // the group. Returns one bit a half whose page can be used; the others
    // take some page's bytes, which nobody uses. With pages of 32 tokens or
    // more both halves lie in one page.
    __device__ __forceinline__ int issue(const FwdParams& p, uint32_t dst) {
        int ok = 0;
        if (tile < end) {
            constexpr int kHalf = 16 * (D / 2), kIts = kHalf / 512;   // bytes of a half's codes, copies for them
            const int lane = threadIdx.x & 31;
            const int at = (tile * kTile) & (p.page - 1);
            const bool ok0 = static_cast<unsigned>(pg[0]) < static_cast<unsigned>(p.num_pages);
            const long long page0 = static_cast<long long>(ok0 ? pg[0] : 0) * p.page_bytes;
            const uint8_t* from = codes + page0 + at * (D / 2);
            const uint8_t* from_v = from + p.part;
            const uint8_t* from_s = scales + page0 + at * (D / 16);
            ok = ok0 ? 3 : 0;
            long long more = 0;   // from where the second half would follow the first to where it is
            if (p.page < kTile) {
                const bool ok1 = static_cast<unsigned>(pg[1]) < static_cast<unsigned>(p.num_pages);
                ok = (ok0 ? 1 : 0) | (ok1 ? 2 : 0);
                more = static_cast<long long>(ok1 ? pg[1] : 0) * p.page_bytes - page0;
                if (lane % kEach >= kEach / 2) from_s += more - kHalf / 8;
                more -= kHalf;
                if (!ok1 && tile * kTile + 16 < len) report(kSitePage);
            }
            if (!ok0) report(kSitePage);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int it = 0; it < kIts; ++it) {
                    copy16(dst + k_dst + u * kHalf + it * 512, from + u * kHalf + it * 512);
                    copy16(dst + v_dst + u * kHalf + it * 512, from_v + u * kHalf + it * 512);
                }
                from += more;
                from_v += more;
            }
            if (D == 128 || lane < 2 * kEach) copy16(dst + s_dst, from_s);
            tile += W;
            look(p);
        }
        copy_commit();
        return ok;
    }
};

// The counter of a segment that several CTAs share counts those that are
// done. It needs no clearing beforehand: a word that does not carry this
// launch's nonce is replaced by the nonce before anyone counts on it, and the
// last CTA leaves 0, so that a replayed launch finds none of its own.
__device__ __forceinline__ int count_in(unsigned long long* word, unsigned long long seen, unsigned long long nonce) {
    unsigned long long old;
    if ((seen & ~0xFFFFULL) != nonce) atomicCAS(word, seen, nonce);   // in vain if someone else did it since
    asm volatile("atom.acq_rel.gpu.global.add.u64 %0, [%1], 1;" : "=l"(old) : "l"(word) : "memory");
    return static_cast<int>(old & 0xFFFF) + 1;
}

// A segment's CTAs c0 .. c1, and how their partial results are joined: at once
// by the last of them to be done, or, where there are many, those of `group`
// neighbours by the last of these (level 0), and the groups' results by the last
// of all (level 1): one request of 262139 tokens, 4 heads, takes 38 us (41 us with
// 74 parts joined at once), with 40 rows a head 85 us (125 us).
struct Split {
    int c0, parts, group, first, in_group;   // first CTA of CTA `cta`'s group, CTAs in it
    __host__ __device__ __forceinline__ Split(int begin, int end, int cta) : c0(begin), parts(end - begin + 1) {
        group = parts;
        if (parts > kJoinAtOnce) {
            group = 4;
            while (group * group < parts) ++group;
        }
        first = c0 + (cta - c0) / group * group;
        in_group = c0 + parts - first < group ? c0 + parts - first : group;
    }
    __host__ __device__ __forceinline__ bool tree() const { return group < parts; }
    __host__ __device__ __forceinline__ int groups() const { return (parts + group - 1) / group; }
    // The level at which the CTA begins, the counter of a level, and the
    // count at which all are done. A group of one has its result in place and is
    // not counted: its CTA may begin the next segment, whose first group would
    // count on the same word. Any other group's first CTA goes on to the next
    // CTA within the segment, and so does c0, which no two segments can: each
    // word has one segment.
    __host__ __device__ __forceinline__ int begins() const { return tree() && in_group > 1 ? 0 : 1; }
    __host__ __device__ __forceinline__ int word(int level, int ctas) const { return level ? c0 : ctas + first; }
    __host__ __device__ __forceinline__ int count(int level) const { return !level ? in_group : tree() ? groups() : parts; }
};

// Joins `n` partial results of a row block, those of CTAs from, from + step, ..,
// by the first T threads of a CTA, with `sync` as their barrier: into the block's
// output, or into the first one's place. wt: room for 32 weights a row.
template <int D, int kRows, int T, bool kBf16, typename Sync>
__device__ __forceinline__ void join_parts(const FwdParams& p, float* wt, float (*row_ml)[2], int c0, int from, int step, int n,
                                           bool final, int rows, long long row0, float v_descale, Sync sync) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // CTA c0 has the segment in its second place
    const long long at0 = 2LL * from + (from == c0 ? 1 : 0);
    auto at = [&](int i) { return i == 0 ? at0 : 2LL * (from + i * step); };
    constexpr int kEach = (kRows + T / 32 - 1) / (T / 32);   // rows of a warp; a lane has a part
    float2 ml[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int row = warp + k * (T / 32);
        ml[k] = make_float2(-INFINITY, 0.0f);
        if (lane < n && row < rows) ml[k] = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (at(lane) * kRows + row) * 2));
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int row = warp + k * (T / 32);
        if (row >= rows) break;
        float m = ml[k].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        const float f = m == -INFINITY ? 0.0f : ptx::ex2_approx(ml[k].x - m);
        if (lane < n) wt[lane * kRows + row] = f;
        float l = f * ml[k].y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
        if (lane == 0) {
            row_ml[row][0] = m;
            row_ml[row][1] = l;
        }
    }
    sync();
    // Two of the thread's items at a time, but for the kernel on tcgen05, whose
    // loop would spill (64 rows: 197 us against 169 us).
    constexpr int kItems = (kRows * (D / 4) + T - 1) / T, kPair = kItems > 1 && kRows <= 24 ? 2 : 1;
#pragma unroll 1
    for (int k = 0; k < kItems; k += kPair) {
        const int i = tid + k * T, d0 = i % (D / 4) * 4;   // T is a multiple of D / 4
        const float* src = p.part_o + (2LL * from * kRows + i / (D / 4)) * D + d0;
        const long long next = 2LL * step * kRows * D;
        constexpr int kDown = T / (D / 4);   // rows from one item to the next
        int row[kPair];
        bool in[kPair];
        float4 o[kPair];
#pragma unroll
        for (int e = 0; e < kPair; ++e) {
            row[e] = i / (D / 4) + e * kDown;
            in[e] = row[e] < rows;
            o[e] = make_float4(0, 0, 0, 0);
        }
        auto add = [&](const float* at, int j) {
            float4 x[kPair];
#pragma unroll
            for (int e = 0; e < kPair; ++e)
                if (in[e]) x[e] = __ldcg(reinterpret_cast<const float4*>(at + e * kDown * D));
#pragma unroll
            for (int e = 0; e < kPair; ++e)
                if (in[e]) axpy4(o[e], wt[j * kRows + row[e]], x[e]);
        };
        if (in[0]) {
            add(src + (from == c0 ? kRows * D : 0), 0);
#pragma unroll 4
            for (int j = 1; j < n; ++j) add(src + j * next, j);
        }
#pragma unroll
        for (int e = 0; e < kPair; ++e) {
            if (!in[e]) continue;
            if (final) {
                store_row4<D, kBf16>(p, row0 + row[e], d0, o[e], row_ml[row[e]][0], row_ml[row[e]][1], v_descale);
            } else {
                *reinterpret_cast<float4*>(p.part_o + (at0 * kRows + row[e]) * D + d0) = o[e];
                if (d0 == 0)
                    *reinterpret_cast<float2*>(p.part_ml + (at0 * kRows + row[e]) * 2) = make_float2(row_ml[row[e]][0], row_ml[row[e]][1]);
            }
        }
    }
}

// Counts this CTA's partial results of a segment in and joins what is complete.
// seen: the words as they were when the segment began, of the segment and of
// the group.
template <int D, int kRows, int T, bool kBf16, typename Sync>
__device__ __forceinline__ void finish_part(const FwdParams& p, int c0, int c1, const unsigned long long (&seen)[2], int& last,
                                            float* wt, float (*row_ml)[2], int rows, long long row0, float v_descale, Sync sync) {
    const Split s(c0, c1, static_cast<int>(blockIdx.x));
    for (int level = s.begins(); level < 2; ++level) {
        unsigned long long* word = p.arrived + s.word(level, p.ctas);
        const int n = s.count(level);
        if (threadIdx.x == 0) {
            last = count_in(word, seen[level ? 0 : 1], p.nonce) == n;
            if (last) *word = 0;
        }
        sync();
        if (!last) return;
        join_parts<D, kRows, T, kBf16>(p, wt, row_ml, s.c0, level ? s.c0 : s.first, level && s.tree() ? s.group : 1, n, level == 1, rows,
                                       row0, v_descale, sync);
        sync();
    }
}

template <int D, int NR, bool kBf16>
__global__ void __launch_bounds__(Shape<NR>::kThreads, Shape<NR>::kCtas) fa2_kv4_fwd_kernel(const FwdParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    using Smem = FwdSmem<D, NR>;
    Smem& sm = *reinterpret_cast<Smem*>(smem);
    constexpr int W = Shape<NR>::kWarps, T = Shape<NR>::kThreads;
    constexpr int kRows = 8 * NR, kStages = Smem::kStages, kStride = Smem::kStride;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

    enter_stream_order();
    Cursor cur;
    int per = 0, pad = 1;
    if (locate<W, 5>(p, cur, per, pad)) {
        load_q<D, NR>(p, sm, cur.b, cur.hr);
        float k_descale = p.k_descale[cur.hr / p.rblocks];
        Loader<D, W> ld;
        ld.start();
        ld.enter(p, cur);
        uint32_t oks = 0;   // two bits a stage
        const uint32_t ring = ptx::smem_addr(sm.ring[warp]);
        Lane<D> ln;
        ln.set(sm);
#pragma unroll
        for (int st = 0; st < kStages - 1; ++st) oks |= ld.issue(p, ring + st * Tile<D>::kBytes) << (2 * st);
        copy_wait<kStages - 2>();   // q went with the first tile
        __syncthreads();
        stage_q<D, NR, kBf16>(p, sm, cur.hr, k_descale);
        __syncthreads();

        int st = 0;
        while (true) {
            const int n = part_tiles(cur), units = part_units(cur, pad);
            const int h = cur.hr / p.rblocks, rb = cur.hr - h * p.rblocks;
            const int seg0 = cur.u - cur.tile, seg1 = seg0 + (pad == 1 ? cur.tiles : padded(cur.tiles, pad));
            const bool split = seg0 < static_cast<int>(blockIdx.x) * per || seg1 > cur.end;
            const int c0 = split ? seg0 / per : 0, c1 = split ? (seg1 - 1) / per : 0;
            if (split && tid < 2)   // read ahead; in place when the tiles are done
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_addr(&sm.seen[tid])),
                             "l"(p.arrived + Split(c0, c1, static_cast<int>(blockIdx.x)).word(1 - tid, p.ctas))
                             : "memory");
            const float v_descale = p.v_descale[h];
            Cursor nxt = cur;
            next_segment<5>(p, nxt, pad);
            const bool more = nxt.u < nxt.end;
            if (more) {
                load_q<D, NR>(p, sm, nxt.b, nxt.hr);
                k_descale = p.k_descale[nxt.hr / p.rblocks];
            }

            Acc<D, NR> acc;
            const int low = p.causal ? cur.len - p.nq + 1 : cur.len;   // keys before it are seen by every row
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc.o[nr][i][e] = 0.0f;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    acc.ref[nr][r] = -INFINITY;
                    acc.l[nr][r] = 0.0f;
                }
            }

            for (int i = warp; i < n; i += W) {
                copy_wait<kStages - 2>();
                __syncwarp();   // every lane's copies of this tile have landed, and all are done with the one before
                const int into = st == 0 ? kStages - 1 : st - 1;
                const uint32_t ok = (oks >> (2 * st)) & 3;
                oks = (oks & ~(3u << (2 * into))) |
                      static_cast<uint32_t>(ld.issue(p, ring + into * Tile<D>::kBytes)) << (2 * into);
                const int tok0 = (cur.tile + i) * kTile;
                const int n_ok[2] = {ok & 1 ? cur.len - tok0 : 0, ok & 2 ? cur.len - tok0 - 16 : 0};
                const uint32_t tile = ring + st * Tile<D>::kBytes;
                if (ok == 3 && tok0 + kTile <= low) tile_step<D, NR, false>(acc, sm, ln, tile, tok0, cur.len, n_ok);
                else tile_step<D, NR, true>(acc, sm, ln, tile, tok0, cur.len, n_ok);
                st = st + 1 == kStages ? 0 : st + 1;
            }
            copy_wait_all();   // the next rows of q
            if (more) {
                ld.enter(p, nxt);
                oks = 0;
                st = 0;
#pragma unroll
                for (int i = 0; i < kStages - 1; ++i) oks |= ld.issue(p, ring + i * Tile<D>::kBytes) << (2 * i);
            }

            // Join the warps' results, eight rows at a time.
            const long long row0 = (static_cast<long long>(cur.b) * p.hkv + h) * p.rows + rb * kRows;
            const int rows = min(kRows, p.rows - rb * kRows);
            const int slot = 2 * blockIdx.x + (c0 == static_cast<int>(blockIdx.x) ? 1 : 0);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                if (nr > 0) __syncthreads();
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float l = acc.l[nr][r];
                    l += __shfl_xor_sync(~0u, l, 4);
                    l += __shfl_xor_sync(~0u, l, 8);
                    l += __shfl_xor_sync(~0u, l, 16);
                    const int row = 2 * t + r;
                    if (g == 0) {
                        sm.ml[warp][nr * 8 + row][0] = l == 0.0f ? -INFINITY : acc.ref[nr][r] == -INFINITY ? 0.0f : acc.ref[nr][r];
                        sm.ml[warp][nr * 8 + row][1] = l;
                    }
                    float* dst = &sm.o[warp][row * kStride + g * (D / 8)];
#pragma unroll
                    for (int i = 0; i < D / 16; i += 2)
                        *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(acc.o[nr][i][r], acc.o[nr][i][r + 2],
                                                                              acc.o[nr][i + 1][r], acc.o[nr][i + 1][r + 2]);
                }
                __syncthreads();
                for (int i = tid; i < min(8, rows - nr * 8) * (D / 4); i += T) {
                    const int in = i / (D / 4), row = nr * 8 + in, d0 = i % (D / 4) * 4;
                    float m = -INFINITY, l = 0.0f;
                    float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int w = 0; w < W; ++w) m = fmaxf(m, sm.ml[w][row][0]);
                    if (m != -INFINITY) {
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const float f = ptx::ex2_approx(sm.ml[w][row][0] - m);
                            l = fmaf(f, sm.ml[w][row][1], l);
                            axpy4(o, f, *reinterpret_cast<const float4*>(&sm.o[w][in * kStride + d0]));
                        }
                    }
                    if (!split) {
                        store_row4<D, kBf16>(p, row0 + row, d0, o, m, l, v_descale);
                    } else {
                        const long long at = static_cast<long long>(slot) * kRows + row;
                        *reinterpret_cast<float4*>(p.part_o + at * D + d0) = o;
                        if (d0 == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m, l);
                    }
                }
            }
            if (more) stage_q<D, NR, kBf16>(p, sm, nxt.hr, k_descale);
            __syncthreads();

            if (split)
                finish_part<D, kRows, T, kBf16>(p, c0, c1, sm.seen, sm.last, sm.o[0], sm.row_ml, rows, row0, v_descale,
                                                [] { __syncthreads(); });
            if (!more) break;
            cur = nxt;
        }
    }

    idle_requests<D, kBf16, T>(p);
}

}  // namespace kv4
}  // namespace fa2
