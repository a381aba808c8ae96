// Attention of new tokens over a paged KV cache held in 16 bits (sm_103a): one
// token a request (decoding), a chunk of a prompt, or both in one call.
//
// The cache is [num_pages, H_kv, 2, page, D] 16-bit elements: of a page and KV
// head first the keys, then the values of `page` tokens. Request b has q_lens[b]
// new tokens, rows q_starts[b] .. of q [T, H_q, D], and seq_lens[b] cached ones,
// its own among them.
//
// How. The tiles are those of the forward kernel: 128 query rows (tokens times
// the G query heads that share a KV head, heads next to each other) against 128
// keys, S = Q K^T and O += P V on tcgen05 with S and O in tensor memory, keys
// and values by TMA, a box for each page of a tile. A block of query rows is up
// to two tiles; both read the same keys (`pair`). A block of one tile, such as a
// decoding request's few rows, uses the second S and O for every other tile of
// keys instead (`single`): two softmax streams over the same rows, whose results
// the epilogue adds up, so that one's exponentials overlap the other's products.
//
// Lengths are known on the device only. The key tiles of all (request, KV head,
// row block) are one line of units that is cut into equal runs, one a CTA. A run
// may begin and end inside a row block; its CTAs then leave partial results in
// fp32, which a second, small kernel joins in a fixed order. A warp of each CTA
// finds the run and hands its parts, row block by row block, to the others.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "fa2.h"
#include "fa2_fwd_sm103.cuh"
#include "fa2_kv4_sm103.cuh"
#include "fa2_kv4_tc_sm103.cuh"
#include "ptx_sm103.cuh"

namespace fa2 {
namespace kv16 {

using kv4::report;

// Sites of the status word (page ids and lengths as for the 4-bit cache).
enum Site : int { kSiteRows = 53, kSitePart = 54, kSiteGuard = 55 };

constexpr int kMaxCtas = 160;
constexpr int kSchedWarp = 14, kGuardWarp = 15;
// Units. A tile of keys counts kPairUnits for two query tiles and kSingleUnits
// for one, and every row block kStart more for its start and its end. Single calls with
// caches cold (32 / 8 heads of 128): a step of 24 decoding requests and 3 chunks up to 512
// tokens, contexts up to 8192, takes 166 us (218 with pages of 16); with 4, 3 and 5 units
// 172 (214), with 2, 1 and 2 173 (253). A prompt of 4096 tokens, whose row blocks are of
// all lengths, takes 136 us; 144 with kStart = 2, 134 with 8, which costs two such prompts
// with 32 / 32 heads of 64 190 us instead of 187.
constexpr int kPairUnits = 3, kSingleUnits = 2, kStart = 4;
constexpr int kMinRun = 4;        // units of a run at least
// Registers a thread. What spills is waited for as long as keys are: the cache
// that shared memory leaves is small. With 176 and 104 for the softmax and the
// epilogue the prompt takes 140 us instead of 136, with 184 and 88 141, and a chunk of 2048
// tokens over 32768 713 and 718 instead of 704.
constexpr uint32_t kRegSoft = 168, kRegOut = 120, kRegRest = 56;
static_assert(2 * kRegSoft + kRegOut + kRegRest == 65536 / 128 && kRegSoft >= 128 && kRegOut <= 128 && kRegRest <= 128,
              "shares of the 128 registers a thread that the launch has");
constexpr int kParts = 4;         // parts on their way from the scheduling warp
constexpr int kPartUsers = 15;    // warps that read a part
constexpr int kJoinY = 4, kJoinThreads = 256;

struct Begun {                    // the row block that begins in a CTA's run and ends behind it
    int parts;                    // CTAs that share it; 0: none
    int q0, ntok, h;
};

struct Params {
    const int* q_starts;          // [B]
    const int* q_lens;            // [B]
    const int* seq_lens;          // [B]
    const int* block_table;       // [B, max_pages]
    void* o;                      // [T, hq, D]
    float* lse;                   // [T, hq]
    float* part_o;                // [2 ctas, part_rows, D]: a CTA's part of a block that began before its run, of one that begins in it
    float* part_ml;               // [2 ctas, part_rows, 2]: running maximum (log2 units) and sum
    Begun* begun;                 // [ctas]
    int B, T, hq, hkv, group;
    int tok_tile;                 // tokens of a tile of query rows: 128 / group
    int part_rows;
    int max_pages, max_tokens, page, log2_page, num_pages;
    int causal, ctas;
    int debug_flags;
    float scale_log2;
    long long wait_limit_ns;
};

// A part: the key tiles jb .. jb + n of one row block that this CTA works on.
struct __align__(16) Part {
    int kind;                     // 0: no more, 1: two tiles of query rows, 2: one
    int steps0, steps1;           // key tiles of each softmax stream
    int jb, n;
    int len, b, h;
    int q0, ntok;                 // first token (row of q) of the block, its tokens
    int vis0;                     // keys that its first token sees
    int buffer;                   // of partial results, or -1: the whole block
    int qslot;                    // single: the place of its query tile
    int jmask0, jmask1;           // first key tile that some row of the stream does not see whole
    int ring;                     // entry of the ring that its first tile has, modulo 16

    __device__ __forceinline__ int steps(int t) const { return t ? steps1 : steps0; }
    __device__ __forceinline__ int jmask(int t) const { return t ? jmask1 : jmask0; }
};
static_assert(sizeof(Part) == 64, "four 16-byte loads");
constexpr int kPair = 1, kSingle = 2;

template <int D>
struct Lay {
    static constexpr int kBlkBytes = Layout<D>::kBlkBytes;
    static constexpr int kTileBytes = Layout<D>::kTileBytes;
    static constexpr int kStages = Layout<D>::kStages;
    static constexpr int kQOff = 0;
    static constexpr int kRingOff = 2 * kTileBytes;
    static constexpr int kBarOff = kRingOff + kStages * kTileBytes;
    // q_full[2] q_empty[2] kv_full[S] kv_empty[S] s_full[2] alpha[2] stats[2] p_full[2] o_full[2] mma_done
    // stats_free[2] part_full[4] part_empty[4] p_rest[2]
    static constexpr int kNumBars = 2 * kStages + 19 + 2 * kParts;
    static constexpr int kRowOff = kBarOff + (kNumBars * 8 + 15) / 16 * 16;   // alpha[2][128], m[2][128], l[2][128]
    static constexpr int kPartOff = kRowOff + 6 * kBM * 4;
    static constexpr int kIdOff = kPartOff + kParts * static_cast<int>(sizeof(Part));   // page ids [4][32]
    static constexpr int kFirstOff = kIdOff + 4 * 32 * 4;   // page ids of the first two tiles of a part [kParts][16]
    // Of a part (modulo 8): whether a value that is not finite was taken out, and
    // in each column the positions of the first +inf and of the first -inf [8][2][D] (a
    // NaN counts as both).
    static constexpr int kFlagOff = kFirstOff + kParts * 16 * 4;
    static constexpr int kBadOff = kFlagOff + 8 * 4;
    static constexpr int kMiscOff = kBadOff + 8 * 2 * D * 4;
    static constexpr int kSmemBytes = kMiscOff + 32 + 1024;   // + TMEM address, abort flag, the guard's counters
    static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
};

template <int D>
struct BarSet : Bars<D> {
    static constexpr int S = Layout<D>::kStages;
    __device__ uint32_t part_full(int s) const { return this->base + 8 * (17 + 2 * S + s); }
    __device__ uint32_t part_empty(int s) const { return this->base + 8 * (17 + 2 * S + kParts + s); }
    // P in two halves: p_full is for the weights of a tile's first 64 keys (and a rescaled O), p_rest for the others'.
    __device__ uint32_t p_rest(int t) const { return this->base + 8 * (17 + 2 * S + 2 * kParts + t); }
};

// Where a tile's 128 keys lie in a place of the ring: in order, groups of eight
// (which the swizzle and the products' descriptors go by) behind one another, of a
// group first the first 64 columns, then the others. So a page is one box of
// [groups][D / 64][8][64] elements. (A box costs the copies about 100 cycles whatever
// its size: with one for each 64 columns, 64 requests of up to 16384 tokens in pages of
// 16 take 554 us, 472 so.)
template <int D>
struct Tiles {
    static constexpr int kBlkBytes = 1024;                  // from a block of 64 columns to the next
    static constexpr int kGroupBytes = D / 64 * kBlkBytes;  // from a group of eight keys to the next
    static constexpr int kHalfBytes = 8 * kGroupBytes;      // from the first 64 keys to the others
    static __device__ __forceinline__ int row_bytes(int r) { return (r >> 3) * kGroupBytes + (r & 7) * 128; }
};

// 5-D tiled copy global -> shared.
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, int x, int y, int z, int u, int v, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
        : "memory");
}

// One arrival for the warp, behind what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// O (+)= P V over one half of a tile's keys, in four steps of 16: P from TMEM
// (8 columns a step), V MN-major (kStep * 16 bytes a step).
template <int kStep>
__device__ __forceinline__ void mma_half(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred e, p0, pt;\n\t.reg .b32 blo, bhi, t0, t1;\n\t.reg .b64 b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p0, %4, 0;\n\t"
        "setp.eq.b32 pt, %4, %4;\n\t"
        "mov.b64 {blo, bhi}, %2;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p0;\n\t"
        "add.u32 t0, %1, 8;\n\tadd.u32 t1, blo, %5;\n\tmov.b64 b, {t1, bhi};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
        "add.u32 t0, %1, 16;\n\tadd.u32 t1, blo, %6;\n\tmov.b64 b, {t1, bhi};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
        "add.u32 t0, %1, 24;\n\tadd.u32 t1, blo, %7;\n\tmov.b64 b, {t1, bhi};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
        "}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(acc), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep)
        : "memory");
}

// ---------------------------------------------------------------- the line of units

// A request as the call may use it: what points outside q or the table counts
// as nothing and is reported.
struct Request {
    int start, n, len, blocks;
};

__device__ __forceinline__ Request request(const Params& p, int start, int n, int len) {
    Request r{start, n, len, 0};
    if (r.n < 0 || r.start < 0 || r.start > p.T - max(r.n, 0)) {
        if (blockIdx.x == 0 && r.n != 0) report(kSiteRows);
        r.n = 0;
    }
    if (r.len < 0 || r.len > p.max_tokens) {
        if (blockIdx.x == 0 && r.n > 0) report(kv4::kSiteLength);
        r.len = min(max(r.len, 0), p.max_tokens);
    }
    r.blocks = r.n <= p.tok_tile ? (r.n > 0) : (r.n + 2 * p.tok_tile - 1) / (2 * p.tok_tile);
    return r;
}
__device__ __forceinline__ Request request(const Params& p, int b) { return request(p, p.q_starts[b], p.q_lens[b], p.seq_lens[b]); }

__device__ __forceinline__ int tiles_in(int keys) { return keys <= 0 ? 0 : (keys + kBN - 1) / kBN; }

// Tiles of keys of n row blocks, where the first sees `keys` keys (1 or more) and each
// next one `step` more (even, up to 256). A block of x keys has (x + r) / kBN tiles with r = -x
// mod kBN, the places of its last tile that it leaves empty, so the sum is that of the
// keys (an arithmetic series) and of the r. These repeat: with g, the largest
// power of two in step and kBN, a period is kBN / g blocks, and its r are e, e + g, ..
// (e below g), kBN (period - 1) / 2 + period e together.
__device__ __forceinline__ int tiles_of_blocks(int n, int keys, int step) {
    const int g = min(step & -step, kBN), e = -keys & (g - 1);
    const int periods = n >> __popc(kBN / g - 1), whole = periods * (kBN / g);
    long long sum = static_cast<long long>(n) * keys + static_cast<long long>(n) * (n - 1) / 2 * step;
    sum += static_cast<long long>(whole) * e + static_cast<long long>(whole - periods) * (kBN / 2);
    for (int i = whole, r = -keys & (kBN - 1); i < n; ++i, r = (r - step) & (kBN - 1)) sum += r;
    return static_cast<int>(sum / kBN);
}

// The first row block in which some row sees a key (len > 0).
__device__ __forceinline__ int first_block(const Params& p, const Request& r) {
    return p.causal && r.n > r.len ? (r.n - r.len) / (2 * p.tok_tile) : 0;
}

// A row block's units: kStart, then its tiles' (none without a tile).
__device__ __forceinline__ int weight(const Params& p, int ntok) { return ntok > p.tok_tile ? kPairUnits : kSingleUnits; }
__device__ __forceinline__ int block_units(int tiles, int w) { return tiles > 0 ? kStart + tiles * w : 0; }

// Units of the first x row blocks of one head (below 2^30: the host's bound).
__device__ __forceinline__ int units_before(const Params& p, const Request& r, int x) {
    if (x <= 0 || r.len == 0) return 0;
    const int step = 2 * p.tok_tile, full = min(x, r.blocks - 1), k0 = first_block(p, r);
    int sum = 0;
    if (full > k0) {
        int tiles = (full - k0) * tiles_in(r.len);
        // block k's last row sees len - n + (k + 1) step keys
        if (p.causal) tiles = tiles_of_blocks(full - k0, r.len - r.n + (k0 + 1) * step, step);
        sum = (full - k0) * kStart + kPairUnits * tiles;
    }
    if (x >= r.blocks) sum += block_units(tiles_in(r.len), weight(p, r.n - (r.blocks - 1) * step));   // its last row sees every key
    return sum;
}

// The scheduling warp: finds this CTA's run and hands out its parts.
template <int D>
__device__ __forceinline__ void scheduler(const Params& p, uint8_t* smem, const BarSet<D>& bars, const Waiter& w) {
    const int lane = threadIdx.x & 31;
    const uint32_t slots = ptx::smem_addr(smem + Lay<D>::kPartOff);
    int n_part = 0;
    bool ok = true;
    int* first_ids = reinterpret_cast<int*>(smem + Lay<D>::kFirstOff);
    const int pages = kBN >> p.log2_page;   // of a tile
    auto put = [&](const Part& x) {
        const int s = n_part % kParts;
        // The page ids that its loads begin with, on their way before the place is free.
        const int entry = x.jb * pages + lane;
        int id = -1;
        if (lane < pages * min(x.n, 2) && entry < (x.len + p.page - 1) >> p.log2_page)
            id = p.block_table[static_cast<long long>(x.b) * p.max_pages + entry];
        ok = __all_sync(~0u, w.wait(bars.part_empty(s), ((n_part / kParts) & 1) ^ 1, kSitePart));
        if (!ok) return;
        if (lane < 16) first_ids[16 * s + lane] = id;
        __syncwarp();
        if (lane == 0) {
            const uint32_t to = slots + s * static_cast<int>(sizeof(Part));
            ptx::st_shared_v4(to, x.kind, x.steps0, x.steps1, x.jb);
            ptx::st_shared_v4(to + 16, x.n, x.len, x.b, x.h);
            ptx::st_shared_v4(to + 32, x.q0, x.ntok, x.vis0, x.buffer);
            ptx::st_shared_v4(to + 48, x.qslot, x.jmask0, x.jmask1, x.ring);
            ptx::mbar_arrive(bars.part_full(s));
        }
        __syncwarp();
        ++n_part;
    };

    // The request at which the run begins: units in front of each lane's share
    // of the requests; then the same within the share that has the run's start.
    int total = 0, per = kMinRun, u = 0, end = 0;
    int at = 0, each = 0, b = 0;   // units in front of the request, of one of its heads, its number
    Request r{};
    for (int lo = 0, hi = p.B, chunk = 0; chunk != 1;) {
        chunk = (hi - lo + 31) / 32;
        const int b0 = min(lo + lane * chunk, hi), b1 = min(b0 + chunk, hi);
        int mine = 0;
        long long rows = 0;
        for (int i = b0; i < b1; i += 4) {   // four requests' numbers are read at once
            int s[4], n[4], len[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[e] = n[e] = len[e] = 0;
                if (i + e < b1) {
                    s[e] = p.q_starts[i + e];
                    n[e] = p.q_lens[i + e];
                    len[e] = p.seq_lens[i + e];
                }
            }
#pragma unroll 1
            for (int e = 0; e < min(4, b1 - i); ++e) {
                r = request(p, s[0], n[0], len[0]);
                each = units_before(p, r, r.blocks);
                mine += each * p.hkv;
                rows += r.n;
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    s[k] = s[k + 1];
                    n[k] = n[k + 1];
                    len[k] = len[k + 1];
                }
            }
        }
        int to = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, to, o);
            if (lane >= o) to += y;
            rows += __shfl_xor_sync(~0u, rows, o);
        }
        if (total == 0) {   // all requests
            total = __shfl_sync(~0u, to, 31);   // below 2^30 if no row has two requests
            if (rows > p.T) {
                if (blockIdx.x == 0 && lane == 0) report(kSiteRows);
                total = 0;
            }
            per = max((total + p.ctas - 1) / p.ctas, kMinRun);
            u = static_cast<int>(blockIdx.x) * per;
            end = min(total, u + per);
            if (u >= end) break;
        }
        const int from = __ffs(__ballot_sync(~0u, u >= at + to - mine && u < at + to)) - 1;
        at += __shfl_sync(~0u, to - mine, from);
        lo = b = __shfl_sync(~0u, b0, from);
        hi = min(lo + chunk, hi);
        each = __shfl_sync(~0u, each, from);
        r = Request{__shfl_sync(~0u, r.start, from), __shfl_sync(~0u, r.n, from), __shfl_sync(~0u, r.len, from),
                    __shfl_sync(~0u, r.blocks, from)};
    }
    const int begin = u;
    Begun begun{0, 0, 0, 0};
    if (u < end) {
        int h = (u - at) / each, inside = u - at - h * each, rb = 0;
        // the row block: 32 candidates at a time
        int before = 0;
        for (int hi = r.blocks; hi - rb > 1;) {
            const int step = (hi - rb + 31) / 32, x = rb + lane * step, units = units_before(p, r, x);
            const int top = 31 - __clz(__ballot_sync(~0u, x < hi && units <= inside));
            before = __shfl_sync(~0u, units, top);
            rb += top * step;
            hi = min(hi, rb + step);
        }
        inside -= before;
        int first = first_block(p, r);
        int singles = 0, ring = 0;
        while (ok) {
            const int tok0 = rb * 2 * p.tok_tile, ntok = min(2 * p.tok_tile, r.n - tok0);
            const int vis0 = p.causal ? r.len - r.n + tok0 + 1 : r.len;
            const int more = p.causal ? 1 : 0;
            const int tiles = tiles_in(vis0 + more * (ntok - 1)), wt = weight(p, ntok), units = block_units(tiles, wt);
            auto over = [&](int a) { return wt == kPairUnits ? a / kPairUnits : a / kSingleUnits; };
            const int seg0 = u - inside, upto = min(end - seg0, units);
            // Tile j is that of the run with unit kStart + j wt of the block.
            Part x;
            x.jb = over(max(inside - kStart + wt - 1, 0));
            x.n = over(max(upto - kStart + wt - 1, 0)) - x.jb;
            x.kind = ntok > p.tok_tile ? kPair : kSingle;
            x.len = r.len;
            x.b = b;
            x.h = h;
            x.q0 = r.start + tok0;
            x.ntok = ntok;
            x.vis0 = vis0;
            x.buffer = -1;
            x.qslot = 0;
            const int tile0 = seg0 + kStart, tile1 = tile0 + (tiles - 1) * wt;   // units of the first and the last tile
            if (tile0 < begin || tile1 >= end) {
                x.buffer = 2 * static_cast<int>(blockIdx.x) + (tile0 >= begin ? 1 : 0);
                if (x.jb == 0 && x.n > 0) begun = Begun{tile1 / per - static_cast<int>(blockIdx.x) + 1, x.q0, ntok, h};
            }
            x.jmask0 = max(vis0, 0) / kBN;
            if (x.kind == kPair) {
                x.steps0 = max(min(x.jb + x.n, tiles_in(vis0 + more * (p.tok_tile - 1))) - x.jb, 0);
                x.steps1 = x.n;
                x.jmask1 = max(vis0 + more * p.tok_tile, 0) / kBN;
            } else {
                x.steps0 = (x.n + 1) / 2;
                x.steps1 = x.n / 2;
                x.jmask1 = x.jmask0;
                if (x.n > 0) x.qslot = singles++ & 1;
            }
            x.ring = ring & 15;
            ring += 2 * x.n;
            if (x.n > 0) put(x);
            u = seg0 + upto;
            inside = 0;
            if (u >= end) break;
            if (++rb == r.blocks) {
                if (++h == p.hkv) {
                    h = 0;
                    do {
                        r = request(p, ++b);
                    } while (r.n == 0 || r.len == 0);
                    first = first_block(p, r);
                }
                rb = first;
            }
        }
    }
    if (lane == 0) p.begun[blockIdx.x] = begun;
    Part x{};
    if (ok) put(x);
}

// The next part; false behind the last one or if the CTA is aborting (`ok`).
// `before`: what else is read of its place.
struct Nothing {
    __device__ __forceinline__ void operator()(int) const {}
};
template <int D, typename Before = Nothing>
__device__ __forceinline__ bool next_part(uint8_t* smem, const BarSet<D>& bars, const Waiter& w, int& n_part, Part& x, bool& ok,
                                          Before before = Before{}) {
    const int s = n_part % kParts;
    ok = __all_sync(~0u, w.wait(bars.part_full(s), (n_part / kParts) & 1, kSitePart));
    if (!ok) return false;
    const uint32_t at = ptx::smem_addr(smem + Lay<D>::kPartOff + s * static_cast<int>(sizeof(Part)));
    uint4* to = reinterpret_cast<uint4*>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = ptx::ld_shared_v4(at + 16 * i);
    before(s);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bars.part_empty(s));
    ++n_part;
    return x.kind != 0;
}

// ---------------------------------------------------------------- producer

// Order of a part's tiles in the ring, the order of their use. Pair: K_0 V_0
// K_1 V_1 ..; single: K_0 K_1 V_0 K_2 V_1 .. V_{n-2} V_{n-1}.
__device__ __forceinline__ void ring_entry(bool pair, int n, int k, int& value, int& tile) {
    if (pair) {
        value = k & 1;
        tile = k >> 1;
    } else if (k == 2 * n - 1) {
        value = 1;
        tile = n - 1;
    } else if (k < 2) {
        value = 0;
        tile = k;
    } else {
        value = (k & 1) ^ 1;
        tile = value ? (k - 2) / 2 : (k + 1) / 2;
    }
}
__device__ __forceinline__ int value_entry(bool pair, int n, int tile) { return pair ? 2 * tile + 1 : min(2 + 2 * tile, 2 * n - 1); }

// A query tile's place: loads of a part's tiles, and what an aborting CTA waits for.
template <int D>
struct Queries {
    uint32_t phase = 0, ever = 0;   // a bit for each place: loads modulo 2, any load

    static __device__ __forceinline__ bool has(const Part& x, int t) { return x.kind == kPair ? x.steps(t) > 0 : t == x.qslot; }

    __device__ __forceinline__ bool free_now(const Part& x, const BarSet<D>& bars) const {
        bool yes = true;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            if (has(x, t)) yes = yes && ptx::mbar_test_wait(bars.q_empty(t), ((phase >> t) & 1) ^ 1);
        return __all_sync(~0u, yes);
    }
    __device__ __forceinline__ bool load(const CUtensorMap* tm, const Params& p, const Part& x, uint32_t sbase, const BarSet<D>& bars,
                                         const Waiter& w) {
        using L = Lay<D>;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            if (!has(x, t)) continue;
            if (!__all_sync(~0u, w.wait(bars.q_empty(t), ((phase >> t) & 1) ^ 1, kSiteQEmpty))) return false;
            if (!(p.debug_flags & 1) && (threadIdx.x & 31) == 0) {   // test hook: no query tiles
                ptx::mbar_arrive_expect_tx(bars.q_full(t), p.tok_tile * p.group * (D * 2));
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    ptx::tma_load_3d(sbase + L::kQOff + t * L::kTileBytes + c * L::kBlkBytes, tm, c * 64, x.h * p.group,
                                     x.q0 + (x.kind == kPair ? t * p.tok_tile : 0), bars.q_full(t));
            }
            phase ^= 1u << t;
            ever |= 1u << t;
        }
        return true;
    }
    __device__ __forceinline__ void drain(const Params& p, const BarSet<D>& bars, const Waiter& w) const {
        if (p.debug_flags & 1) return;
        for (int t = 0; t < 2; ++t)
            if ((ever >> t) & 1) w.drain(bars.q_full(t), ((phase >> t) & 1) ^ 1);
    }
};

// A box for each page, each by a lane of its own.
template <int D>
__device__ __forceinline__ void producer(const CUtensorMap* tmQ, const CUtensorMap* tmKV, const Params& p, uint8_t* smem,
                                         uint32_t sbase, const BarSet<D>& bars, const Waiter& w) {
    using L = Lay<D>;
    constexpr int S = L::kStages;
    const int lane = threadIdx.x & 31;
    const int pages = kBN >> p.log2_page;          // of a tile
    const int page_at = lane;
    const bool loads = page_at < pages;
    const uint32_t box = page_at * (p.page * D * 2);
    int* ids = reinterpret_cast<int*>(smem + L::kIdOff) + lane;   // of the lane's page, tile modulo 4
    const int nothing = p.num_pages * p.hkv * 2;   // past the tensor: a box of zeros
    int ring = 0, n_part = 0;
    Queries<D> queries;
    const int* first_ids = reinterpret_cast<const int*>(smem + L::kFirstOff);
    int ahead[2];   // page ids of the next two tiles of keys
    bool ok = true;
    Part x;
    while (next_part<D>(smem, bars, w, n_part, x, ok, [&](int s) {
        if (loads)
#pragma unroll
            for (int e = 0; e < 2; ++e) ahead[e] = *const_cast<const volatile int*>(first_ids + 16 * s + e * pages + page_at);
    })) {
        const bool pair = x.kind == kPair;
        const int* table = p.block_table + static_cast<long long>(x.b) * p.max_pages;
        const int used = (x.len + p.page - 1) >> p.log2_page;   // pages of the request
        const int entry0 = x.jb * pages + page_at;
        auto look = [&](int tile) {
            const int e = entry0 + tile * pages;
            return loads && tile < x.n && e < used ? __ldg(table + e) : -1;
        };
        auto load_kv = [&](int k) {
            int value, tile;
            ring_entry(pair, x.n, k, value, tile);
            const int s = ring % S;
            ok = __all_sync(~0u, w.wait(bars.kv_empty(s), ((ring / S) & 1) ^ 1, kSiteKvEmpty));
            if (!ok) return;
            int z;
            if (value) {
                z = ids[32 * (tile & 3)];
                z = z < 0 ? nothing : z + 1;
            } else {
                const int id = ahead[0];
                const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(p.num_pages);
                if (!good && loads && entry0 + tile * pages < used) report(kv4::kSitePage);
                z = good ? (id * p.hkv + x.h) * 2 : -1;
                ids[32 * (tile & 3)] = z;
                z = good ? z : nothing;
                ahead[0] = ahead[1];
                ahead[1] = look(tile + 2);
            }
            if (lane == 0) ptx::mbar_arrive_expect_tx(bars.kv_full(s), L::kTileBytes);
            __syncwarp();
            const uint32_t dst = sbase + L::kRingOff + s * L::kTileBytes + box;
            if (loads) tma_load_5d(dst, tmKV, 0, 0, 0, 0, z, bars.kv_full(s));
            ++ring;
        };
        // Query tiles whose places are free go before the keys, whose page ids are
        // on their way; others behind the first tile, for which there is room earlier.
        const int when = queries.free_now(x, bars) ? 0 : 1;
#pragma unroll 1
        for (int k = 0; k < 2 * x.n && ok; ++k) {
            if (k == when && !(ok = queries.load(tmQ, p, x, sbase, bars, w))) break;
            load_kv(k);
        }
        if (!ok) break;
    }
    if (!ok) {   // aborting: every copy that this CTA started lands before it exits
        const int first = ring > S ? ring - S : 0;
        for (int r = first; r < ring; ++r) w.drain(bars.kv_full(r % S), (r / S) & 1);
        queries.drain(p, bars, w);
    }
    __syncwarp();
}

// ---------------------------------------------------------------- guard

// The guard and the softmax: a stream's first warp lets the guard go on to a tile
// when it has seen the tile's scores, or of a pair the scores before (then the values' place in the ring holds no
// older tile that could be taken for them), and waits for the guard before it hands
// over the tile's first weights. Tiles are counted, those of all parts.
struct Gate {
    uint32_t at;   // in shared memory: go of each stream, done
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < 3; ++i) asm volatile("st.shared.b32 [%0], 0;" ::"r"(at + 4 * i) : "memory");
    }
    __device__ __forceinline__ int read(int i) const {
        int v;
        asm volatile("ld.acquire.cta.shared.b32 %0, [%1];" : "=r"(v) : "r"(at + 4 * i) : "memory");
        return v;
    }
    __device__ __forceinline__ void set(int i, int v) const { asm volatile("st.release.cta.shared.b32 [%0], %1;" ::"r"(at + 4 * i), "r"(v) : "memory"); }
    __device__ __forceinline__ void set_go(int t, int n) const { set(t, n); }
    __device__ __forceinline__ void set_done(int n) const { set(2, n); }
    template <typename Done>
    __device__ __forceinline__ bool spin(const Waiter& w, Done done) const {
        bool ok = true;
        const uint64_t t0 = ptx::globaltimer_ns();
        while (!done()) {
            if (*w.abort_flag) ok = false;
            if (static_cast<long long>(ptx::globaltimer_ns() - t0) > w.limit_ns) {
                *w.abort_flag = 1;
                atomicCAS(&g_fa2_status, 0, FA2_ERR_TIMEOUT | (kSiteGuard << 8));
                ok = false;
            }
            if (!ok) break;
        }
        return __all_sync(~0u, ok);
    }
    __device__ __forceinline__ bool wait_go(int n, const Waiter& w) const { return spin(w, [&] { return max(read(0), read(1)) >= n; }); }
    __device__ __forceinline__ bool wait_done(int n, const Waiter& w) const { return spin(w, [&] { return read(2) >= n; }); }
};

// A weight of 0 does not keep out a value that is not finite: 0 * NaN is NaN. So
// the values of tiles that some row does not see whole are gone over before they
// are used. What lies behind the request's end, of whoever had the page before,
// becomes zeros. Values that are not finite behind the first row's last key
// become zeros too, and the epilogue adds them to the rows that do see them: an
// infinity whatever its weight, +inf and -inf for a NaN.
// Where all rows of a block see the same keys (one token, or no mask), only
// the end is to be seen to, which the softmax does itself: it is there sooner.
__device__ __forceinline__ bool rows_differ(const Params& p, const Part& x) { return p.causal && x.ntok > 1; }
__device__ __forceinline__ int guarded_from(const Params& p, const Part& x) {   // first tile of the part that the guard goes over
    return rows_differ(p, x) ? max(x.jmask0 - x.jb, 0) : x.n;
}

// sum + 0 * x for a pair.
template <bool kBf16>
__device__ __forceinline__ uint32_t zero_times(uint32_t x, uint32_t sum) {
    uint32_t r;
    if constexpr (kBf16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(sum));
    return r;
}

template <int D, bool kBf16>
__device__ __forceinline__ void guard(const Params& p, uint8_t* smem, uint32_t sbase, const BarSet<D>& bars, const Waiter& w, const Gate& gate) {
    using L = Lay<D>;
    using T = Tiles<D>;
    constexpr int S = L::kStages, kPieces = D / 8, kRows = 32 / kPieces;   // pieces of 16 bytes of a row, rows at a time
    constexpr uint32_t kInf = kBf16 ? 0x7F80u : 0x7C00u;
    const int lane = threadIdx.x & 31, piece = lane % kPieces;
    int n_part = 0, ring = 0, seen = 0;   // seen: tiles
    bool ok = true;
    Part x;
    while (next_part<D>(smem, bars, w, n_part, x, ok)) {
        // Eight parts back the epilogue is done: part n + 4 is not handed out before it has taken part n.
        volatile int* flag = reinterpret_cast<int*>(smem + L::kFlagOff) + (n_part & 7);
        int* first_bad = reinterpret_cast<int*>(smem + L::kBadOff) + (n_part & 7) * (2 * D);
        if (lane == 0) *flag = 0;
        __syncwarp();
        const int ring0 = ring;
        ring += 2 * x.n;
        for (int j = guarded_from(p, x); j < x.n; ++j) {
            const int r = ring0 + value_entry(x.kind == kPair, x.n, j), at = (x.jb + j) * kBN;
            ok = gate.wait_go(++seen, w);
            ok = __all_sync(~0u, ok && w.wait(bars.kv_full(r % S), (r / S) & 1, kSiteKvFull));
            if (!ok) break;
            const int valid = x.len - at;
            const uint32_t tile = sbase + L::kRingOff + (r % S) * L::kTileBytes + (piece / 8) * T::kBlkBytes;
            auto place = [&](int row) { return tile + T::row_bytes(row) + (((piece ^ row) & 7) << 4); };
            for (int row = valid / kRows * kRows + lane / kPieces; row < kBN; row += kRows)
                if (row >= valid) ptx::st_shared_v4(place(row), 0, 0, 0, 0);
            __syncwarp();
            // Rows that the first row sees are seen by all. 0 * x is a zero where x is finite.
            const int low = max(x.vis0 - at, 0), high = min(valid, kBN);
            uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll 1
            for (int row0 = low / (8 * kRows) * (8 * kRows); row0 < high; row0 += 8 * kRows) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint4 v = ptx::ld_shared_v4(place(row0 + e * kRows + lane / kPieces));
                    sum[0] = zero_times<kBf16>(v.x, sum[0]);
                    sum[1] = zero_times<kBf16>(v.y, sum[1]);
                    sum[2] = zero_times<kBf16>(v.z, sum[2]);
                    sum[3] = zero_times<kBf16>(v.w, sum[3]);
                }
            }
            if (__any_sync(~0u, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7FFF7FFFu) != 0)) {
                if (*flag == 0) {
                    for (int c = lane; c < 2 * D; c += 32) first_bad[c] = 0x7FFFFFFF;
                    __syncwarp();
                    if (lane == 0) *flag = 1;
                }
                __syncwarp();
                for (int row = low + lane / kPieces; row < high; row += kRows) {
                    uint4 v = ptx::ld_shared_v4(place(row));
                    uint32_t* word = reinterpret_cast<uint32_t*>(&v);
#pragma unroll 1
                    for (int half = 0; half < 2; ++half) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t y = word[k] & 0xFFFFu;
                            if ((y & kInf) == kInf) {
                                int* first = first_bad + piece * 8 + 2 * k + half;
                                if (y != (kInf | 0x8000u)) atomicMin(first, at + row);
                                if (y != kInf) atomicMin(first + D, at + row);
                                y = 0;
                            }
                            word[k] = word[k] >> 16 | y << 16;
                        }
                    }
                    ptx::st_shared_v4(place(row), v.x, v.y, v.z, v.w);
                }
                __syncwarp();
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) gate.set_done(seen);
        }
        if (!ok) break;
    }
    __syncwarp();
}

// ---------------------------------------------------------------- MMA issuer

template <int D, bool kBf16>
__device__ __forceinline__ void mma_issuer(const Params& p, uint8_t* smem, uint32_t sbase, uint32_t tmem, const BarSet<D>& bars,
                                           const Waiter& w) {
    using L = Lay<D>;
    constexpr int S = L::kStages;
    constexpr uint32_t kAB = kBf16 ? 1u : 0u;
    using T = Tiles<D>;
    constexpr uint32_t kIdS = ptx::idesc_f16(kAB, 0, 0, kBM, kBN);
    constexpr uint32_t kIdO = ptx::idesc_f16(kAB, 0, 1, kBM, D);
    // Descriptors of the ring's first place as keys and as values, and of the
    // query tiles' first; others lie kTileBytes / 16 further on.
    constexpr uint32_t kNext = L::kTileBytes >> 4;
    const uint64_t keys = ptx::desc_sw128(sbase + L::kRingOff, 16, T::kGroupBytes),
                   values = ptx::desc_sw128(sbase + L::kRingOff, T::kBlkBytes, T::kGroupBytes),
                   query = ptx::desc_sw128(sbase + L::kQOff, 16, 1024);
    auto wait_u = [&](uint32_t bar, uint32_t parity, int site) { return __all_sync(~0u, w.wait(bar, parity, site)); };
    constexpr uint32_t kQ = L::kBlkBytes >> 4, kK = T::kBlkBytes >> 4;   // from 64 columns to the next
    auto issue_qk = [&](int t, uint64_t qd, uint64_t kd) {
        if constexpr (D == 128)
            ptx::mma_ss_kloop<2, 4, 6, kQ, kQ + 2, kQ + 4, kQ + 6, 2, 4, 6, kK, kK + 2, kK + 4, kK + 6, 8>(tmem + Layout<D>::col_s(t), qd, kd, kIdS, 0u);
        else
            ptx::mma_ss_kloop<2, 4, 6, 0, 0, 0, 0, 2, 4, 6, 0, 0, 0, 0, 4>(tmem + Layout<D>::col_s(t), qd, kd, kIdS, 0u);
        ptx::tc_commit_elect(bars.s_full(t));
    };
    // P V of a tile whose p_full has completed: its halves as their weights are there.
    auto issue_pv = [&](int t, uint64_t vd, bool acc, uint32_t parity) {
        ptx::tc_fence_after();
        mma_half<T::kGroupBytes / 8>(tmem + Layout<D>::col_o(t), tmem + Layout<D>::col_s(t), vd, kIdO, acc ? 1u : 0u);
        if (!wait_u(bars.p_rest(t), parity, kSitePFull)) return false;
        ptx::tc_fence_after();
        mma_half<T::kGroupBytes / 8>(tmem + Layout<D>::col_o(t), tmem + Layout<D>::col_s(t) + 32, vd + (T::kHalfBytes >> 4), kIdO, 1u);
        return true;
    };
    // The same in loops of four products, for one query tile, where copies bound the
    // time: what is executed now and then has to fit the instruction cache beside the
    // rest. (For two, whose products are waited for, these are slower: a chunk of 2048
    // tokens over 32768 takes 782 us instead of 704.)
    auto issue_qk_single = [&](int t, uint64_t qd, uint64_t kd) {
#pragma unroll 1
        for (int blk = 0; blk < D / 64; ++blk)
            ptx::mma_ss_kloop<2, 4, 6, 0, 0, 0, 0, 2, 4, 6, 0, 0, 0, 0, 4>(tmem + Layout<D>::col_s(t), qd + blk * kQ, kd + blk * kK, kIdS, blk);
        ptx::tc_commit_elect(bars.s_full(t));
    };
    auto issue_pv_single = [&](int t, uint64_t vd, bool acc, uint32_t parity) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            if (h && !wait_u(bars.p_rest(t), parity, kSitePFull)) return false;
            ptx::tc_fence_after();
            mma_half<T::kGroupBytes / 8>(tmem + Layout<D>::col_o(t), tmem + Layout<D>::col_s(t) + 32 * h, vd + h * (T::kHalfBytes >> 4),
                                         kIdO, acc || h ? 1u : 0u);
        }
        return true;
    };
    auto release = [&](int r) { ptx::tc_commit_elect(bars.kv_empty(r % S)); };
    // Waits for two entries of the ring and one more barrier together.
    auto wait_three = [&](int r0, int r1, uint32_t bar, uint32_t parity) {
        const uint32_t wb[3] = {bars.kv_full(r0 % S), bars.kv_full(r1 % S), bar};
        const uint32_t wp[3] = {static_cast<uint32_t>((r0 / S) & 1), static_cast<uint32_t>((r1 / S) & 1), parity & 1};
        return __all_sync(~0u, w.wait_all<3>(wb, wp, kSiteKvFull));
    };

    int ring = 0, n_part = 0;
    uint32_t nq = 0, np = 0;   // a bit for each place: query tiles used, P tiles consumed, modulo 2
    bool ok = true;
    Part x;
    while (next_part<D>(smem, bars, w, n_part, x, ok)) {
        if (x.kind == kPair) {
            // As the forward kernel's general mode: at key tile j the streams with
            // j < steps(t) take part, stream 1 in all.
            if (x.steps0 > 0) ok = wait_u(bars.q_full(0), nq & 1, kSiteQFull);
            if (!ok || !(ok = wait_three(ring, ring, bars.q_full(1), nq >> 1))) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                if (x.steps(t) == 0) continue;
                issue_qk(t, query + t * kNext, keys + (ring % S) * kNext);
                if (x.steps(t) == 1) ptx::tc_commit_elect(bars.q_empty(t));
            }
            release(ring++);
            for (int j = 0; j < x.n; ++j) {
                const bool more = j + 1 < x.n;
                const int v_ring = ring++, k_ring = more ? ring++ : v_ring;
                const uint64_t vd = values + (v_ring % S) * kNext, kd = keys + (k_ring % S) * kNext;
                const int t0 = j < x.steps0 ? 0 : 1;
                // V_j, K_{j+1} and the first stream's first weights are waited for together.
                if (!(ok = wait_three(v_ring, k_ring, bars.p_full(t0), np >> t0))) break;
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    if (t < t0) continue;
                    if (t != t0 && !(ok = wait_u(bars.p_full(t), (np >> t) & 1, kSitePFull))) break;
                    if (!(ok = issue_pv(t, vd, j > 0, (np >> t) & 1))) break;
                    np ^= 1u << t;
                    if (t == 1) release(v_ring);
                    if (j + 1 < x.steps(t)) {
                        issue_qk(t, query + t * kNext, kd);
                        if (j + 2 == x.steps(t)) ptx::tc_commit_elect(bars.q_empty(t));
                        if (t == 1) release(k_ring);
                    } else {
                        ptx::tc_commit_elect(bars.o_full(t));
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            nq ^= x.steps0 > 0 ? 3u : 2u;
        } else {
            // Every other tile of keys for each stream: QK of tile j + 2 follows PV of
            // tile j; the first two, behind no PV, count as steps -2 and -1.
            const uint64_t qd = query + x.qslot * kNext;
            for (int j = -2; j < x.n; ++j) {
                const bool first = j < 0, more = j + 2 < x.n;
                if (first && !more) continue;   // n = 1
                const int t = j & 1, v_ring = first ? ring : ring++, k_ring = more ? ring++ : v_ring;
                const uint64_t vd = values + (v_ring % S) * kNext, kd = keys + (k_ring % S) * kNext;
                if (!(ok = wait_three(v_ring, k_ring, first ? bars.q_full(x.qslot) : bars.p_full(t), first ? nq >> x.qslot : np >> t))) break;
                ptx::tc_fence_after();
                if (!first) {
                    if (!(ok = issue_pv_single(t, vd, j > 1, (np >> t) & 1))) break;
                    np ^= 1u << t;
                    release(v_ring);
                }
                if (more) {
                    issue_qk_single(t, qd, kd);
                    if (j + 3 == x.n) ptx::tc_commit_elect(bars.q_empty(x.qslot));
                    release(k_ring);
                } else {
                    ptx::tc_commit_elect(bars.o_full(t));
                }
            }
            if (!ok) break;
            nq ^= 1u << x.qslot;
        }
    }
    // Every MMA issued above finishes before the CTA frees its TMEM.
    ptx::tc_commit_elect(bars.mma_done());
    w.drain(bars.mma_done(), 0);
    __syncwarp();
}

// ---------------------------------------------------------------- softmax

// Tokens of the tile that a stream's rows belong to.
__device__ __forceinline__ int stream_tokens(const Params& p, const Part& x, int t) {
    return x.kind == kPair ? min(x.ntok - t * p.tok_tile, p.tok_tile) : x.ntok;
}

// r / group for r < 128: inv = ceil(2^16 / group), which is off by less than
// group / 2^16 of a quotient, so r / group by less than 1 / group.
__device__ __forceinline__ int by_group(int r, uint32_t inv) { return static_cast<int>((static_cast<uint32_t>(r) * inv) >> 16); }

template <int D, bool kBf16>
__device__ __forceinline__ void softmax_role(const Params& p, uint32_t tmem, uint8_t* smem, const BarSet<D>& bars, const Waiter& w,
                                             const Gate& gate, int t) {
    using L = Lay<D>;
    using T = Tiles<D>;
    constexpr int S = L::kStages;
    const uint32_t ring0 = ptx::smem_addr(smem + L::kRingOff);
    const int row = threadIdx.x & 127;          // row of the query tile = TMEM lane
    const uint32_t row_addr = tmem + (static_cast<uint32_t>(row & ~31) << 16);
    const uint32_t colS = Layout<D>::col_s(t);
    float* alpha_buf = reinterpret_cast<float*>(smem + L::kRowOff) + t * kBM;
    float* m_buf = alpha_buf + 2 * kBM;
    float* l_buf = m_buf + 2 * kBM;
    const float c = p.scale_log2;
    const uint64_t c2 = ptx::f2_pack(c, c);
    const int tok = by_group(row, (65536u + p.group - 1) / p.group);   // the row's token in the tile

    uint32_t n_s = 0, n_item = 0;   // parities: steps, parts of the stream
    int n_part = 0, guarded = 0;    // guarded: tiles that the guard goes over, of the parts so far
    bool ok = true;
    Part x;
    while (next_part<D>(smem, bars, w, n_part, x, ok)) {
        const bool pair = x.kind == kPair;
        const int steps = x.steps(t), g0 = guarded_from(p, x);
        guarded += max(x.n - g0, 0);
        if (steps == 0) continue;
        // The stream's step i is the part's tile i (pair) or 2 i + t (single).
        const int every = pair ? 1 : 2, from = x.jb + (pair ? 0 : t);
        int tile = guarded - x.n + from - x.jb + 1;   // the step's, as the guard counts
        const bool live = (row & ~31) < stream_tokens(p, x, t) * p.group;   // of the warp: some row is a query's
        // Keys of the step's tile that the row sees, and the first step at which that may be fewer than all.
        int lim = min(x.len, x.vis0 + (p.causal ? tok + (pair ? t * p.tok_tile : 0) : 0)) - from * kBN;
        const int mask_from = (x.jmask(t) - from + every - 1) / every;
        const bool gated = rows_differ(p, x);
        // Without a guard: the step in whose tile the request ends, if it has it; the tile's V, and how many keys it has.
        int tail_step = -1, tail = 0;
        if (!gated && x.len % kBN != 0) {
            const int last = x.len / kBN - from;
            if (last >= 0 && last % every == 0) {
                tail_step = last / every;
                tail = (x.ring + value_entry(pair, x.n, last + from - x.jb)) * kBN + x.len % kBN;
            }
        }
        float m = -INFINITY;  // running row max of the scaled scores, log2 units
        float l = 0.0f;       // running sum of exp2(s*c - m)
        for (int i = 0; i < steps; ++i, n_s ^= 1, lim -= every * kBN, tile += every) {
            ok = w.wait(bars.s_full(t), n_s, kSiteSFull);
            if (!__all_sync(~0u, ok)) {
                ok = false;
                break;
            }
            if (i == tail_step) {   // zeros behind the end; two streams that share the tile write the same
                const int r = tail / kBN;
                ok = w.wait(bars.kv_full(r % S), (r / S) & 1, kSiteKvFull);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                if (row >= tail % kBN) {
                    const uint32_t at = ring0 + (r % S) * L::kTileBytes + T::row_bytes(row);
#pragma unroll 4
                    for (int k = 0; k < D / 8; ++k)
                        ptx::st_shared_v4(at + (k / 8) * T::kBlkBytes + (((k ^ row) & 7) << 4), 0, 0, 0, 0);
                }
                ptx::fence_proxy_async_smem();
            }
            if (!live) {   // no row of this warp is a query's: its lanes of P and O may hold anything
                if (i > 0) warp_arrive(bars.alpha_ready(t));
                if (i + 1 == steps) {
                    ok = w.wait(bars.stats_free(t), n_item ^ 1, kSiteStats);
                    if (!__all_sync(~0u, ok)) {
                        ok = false;
                        break;
                    }
                    warp_arrive(bars.stats_ready(t));
                }
                warp_arrive(bars.p_full(t));
                warp_arrive(bars.p_rest(t));
                continue;
            }
            ptx::tc_fence_after();
            const bool masked = i >= mask_from;   // some row does not see all of these keys
            if (gated && row == 0) {
                // A pair's scores of a tile are behind the values of the tile before the last: the next one's place is seen to.
                if (pair && i + 1 >= mask_from && i + 1 < steps) gate.set_go(t, tile + 1);
                else if (masked) gate.set_go(t, tile);
            }
            // The last 64 scores are read for the maximum and, when the first 64
            // weights are done, once more: all 128 and the rest of the state do not
            // fit the registers.
            uint32_t s[kBN / 2];
            float m_tile;
            {
                uint32_t s2[kBN / 2];
                float mq[4];
                ptx::tmem_ld32_max_at<0>(row_addr + colS + 64, s2, mq[2]);
                ptx::tmem_ld32_max_at<32>(row_addr + colS + 96, s2, mq[3]);
                ptx::tmem_ld32_max_at<0>(row_addr + colS + 0, s, mq[0]);
                ptx::tmem_ld32_max_at<32>(row_addr + colS + 32, s, mq[1]);
                ptx::tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mq[k] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < kBN / 2; k += 2) {
                        s[k] = k < lim ? s[k] : 0xFF800000u;
                        s[k + 1] = k + 1 < lim ? s[k + 1] : 0xFF800000u;
                        mq[k / 2 % 2] = ptx::max3(mq[k / 2 % 2], __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
                        mq[2 + k / 2 % 2] = ptx::max3(mq[2 + k / 2 % 2], k + 64 < lim ? __uint_as_float(s2[k]) : -INFINITY,
                                                      k + 65 < lim ? __uint_as_float(s2[k + 1]) : -INFINITY);
                    }
                }
                m_tile = fmaxf(ptx::max3(mq[0], mq[1], mq[2]), mq[3]) * c;
            }
            const float m_new = fmaxf(m, m_tile);
            if (i > 0) {
                const float alpha = m_new == m ? 1.0f : ptx::ex2_approx(m - m_new);
                alpha_buf[row] = alpha;
                warp_arrive(bars.alpha_ready(t));
                l *= alpha;
            }
            m = m_new;
            // A row with no key so far keeps m = -inf; its weights are exp2(-inf - 0) = 0.
            const float m_use = m == -INFINITY ? 0.0f : m;
            const uint64_t nm2 = ptx::f2_pack(-m_use, -m_use);
            uint64_t acc[4] = {0, 0, 0, 0};
            // The products take 16-bit operands, so a weight is rounded to the cache's type, half a step
            // of it (bf16 2^-8, fp16 2^-11): O is off by 0.0021 to 0.0023 in bf16, with fp32 weights by
            // 0.0017, in fp16 by 0.00026 to 0.00028 instead of 0.0002. The sum is of the unrounded ones.
            auto weights = [&](const uint32_t (&v)[kBN / 2], uint32_t (&pk)[32], int k0) {   // of v's scores k0 .. k0 + 32
#pragma unroll
                for (int k = k0 / 2; k < k0 / 2 + 16; ++k) {
                    float x0, x1;
                    ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), c2, nm2), x0, x1);
                    x0 = ptx::ex2_approx(x0);
                    x1 = ptx::ex2_approx(x1);
                    acc[k & 3] = ptx::f2_add(acc[k & 3], ptx::f2_pack(x0, x1));
                    pk[k] = ptx::pack2<kBf16>(x0, x1);
                }
            };
            uint32_t pk[32];
            weights(s, pk, 0);
            uint32_t s2[kBN / 2];
            ptx::tmem_ld32_at<0>(row_addr + colS + 64, s2);
            weights(s, pk, 32);
            ptx::tmem_ld32_at<32>(row_addr + colS + 96, s2);
            ptx::tmem_st32_at<0>(row_addr + colS, pk);
            ptx::tmem_wait_ld();
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            if (masked && gated && row < 32 && !(ok = gate.wait_done(tile, w))) break;
            warp_arrive(bars.p_full(t));
            if (masked) {
#pragma unroll
                for (int k = 0; k < kBN / 2; ++k) s2[k] = k + 64 < lim ? s2[k] : 0xFF800000u;
            }
            weights(s2, pk, 0);
            weights(s2, pk, 32);
            ptx::tmem_st32_at<0>(row_addr + colS + 32, pk);
            float a0, a1;
            ptx::f2_unpack(ptx::f2_add(ptx::f2_add(acc[0], acc[1]), ptx::f2_add(acc[2], acc[3])), a0, a1);
            l += a0 + a1;
            if (i + 1 == steps) {
                // the epilogue has read the stream's last m and l
                ok = w.wait(bars.stats_free(t), n_item ^ 1, kSiteStats);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                m_buf[row] = m;
                l_buf[row] = l;
                warp_arrive(bars.stats_ready(t));
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            warp_arrive(bars.p_rest(t));
        }
        if (!ok) break;
        n_item ^= 1;
    }
}

// ---------------------------------------------------------------- correction + epilogue

// 32 bytes to global memory, one sector; as two stores where the output is
// aligned to 16 bytes only.
__device__ __forceinline__ void store32(char* to, bool wide, const uint32_t* v) {
    if (wide)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

template <int D, bool kBf16>
__device__ __forceinline__ void correction_role(const Params& p, uint32_t tmem, uint8_t* smem, uint32_t sbase, const BarSet<D>& bars,
                                                const Waiter& w) {
    using L = Lay<D>;
    const int q = (threadIdx.x / 32) & 3;
    const int lane = threadIdx.x & 31;
    const int row = 32 * q + lane;
    const uint32_t row_addr = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const float* rowbuf = reinterpret_cast<const float*>(smem + L::kRowOff);  // alpha | m | l
    const int row_tok = by_group(row, (65536u + p.group - 1) / p.group);   // the row's token in its tile,
    const int row_line = row_tok * p.hq + (row - row_tok * p.group);       // its line in o, from the tile's first on
    const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;

    uint32_t n_s = 0, n_items = 0;   // a bit for each stream: steps, parts, modulo 2
    int n_part = 0;
    bool ok = true;
    Part x;
    // At a part's first step O is overwritten, not rescaled: what the PV product
    // waits for is that the O of the stream's last part has been read. That
    // arrival is made here and, from then on, by the epilogue.
    for (int t = 0; t < 2; ++t) warp_arrive(bars.p_full(t));
    while (next_part<D>(smem, bars, w, n_part, x, ok)) {
        const bool pair = x.kind == kPair;
        const int most = max(x.steps0, x.steps1);
        for (int i = 1; i < most && ok; ++i) {
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
                if (i >= x.steps(t)) continue;
                ok = w.wait(bars.alpha_ready(t), (n_s >> t) & 1, kSiteAlpha);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                n_s ^= 1u << t;
                const bool live = 32 * q < stream_tokens(p, x, t) * p.group;
                const float alpha = live ? rowbuf[t * kBM + row] : 1.0f;
                if (__any_sync(~0u, alpha != 1.0f)) {
                    ptx::tc_fence_after();
                    const uint32_t colO = Layout<D>::col_o(t);
                    const uint64_t a2 = ptx::f2_pack(alpha, alpha);
#pragma unroll 1
                    for (int h = 0; h < D; h += 32) {
                        uint32_t o[32];
                        ptx::tmem_ld32_at<0>(row_addr + colO + h, o);
                        ptx::tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float o0, o1;
                            ptx::f2_unpack(
                                ptx::f2_mul(ptx::f2_pack(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1])), a2), o0, o1);
                            o[2 * k] = __float_as_uint(o0);
                            o[2 * k + 1] = __float_as_uint(o1);
                        }
                        ptx::tmem_st32_at<0>(row_addr + colO + h, o);
                    }
                    ptx::tmem_wait_st();
                }
                ptx::tc_fence_before();
                warp_arrive(bars.p_full(t));
            }
        }
        // Epilogue.
#pragma unroll 1
        for (int tile = 0; tile < (pair ? 2 : 1) && ok; ++tile) {
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};   // of the streams that have this tile's rows
            bool has[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = pair ? tile : e;
                has[e] = (!pair || e == 0) && x.steps(t) > 0;
                if (!has[e]) continue;
                ok = ok && w.wait(bars.stats_ready(t), (n_items >> t) & 1, kSiteStats) &&
                     w.wait(bars.o_full(t), (n_items >> t) & 1, kSiteOFull);
                if (!__all_sync(~0u, ok)) {
                    ok = false;
                    break;
                }
                n_items ^= 1u << t;
                m[e] = rowbuf[(2 + t) * kBM + row];
                l[e] = rowbuf[(4 + t) * kBM + row];
                warp_arrive(bars.stats_free(t));
            }
            if (!ok) break;
            ptx::tc_fence_after();
            const int rows = stream_tokens(p, x, tile) * p.group;
            // The next part's first PV products may overwrite the streams' O.
            auto release = [&] {
                ptx::tc_fence_before();
                if (pair) {
                    if (has[0]) warp_arrive(bars.p_full(tile));
                } else {
                    warp_arrive(bars.p_full(0));
                    if (has[1]) warp_arrive(bars.p_full(1));
                }
            };
            if (32 * q >= rows) {
                release();
                continue;
            }
            float mm = m[0], ll = l[0], f[2] = {1.0f, 0.0f};
            if (has[1]) {
                mm = fmaxf(m[0], m[1]);
                const float ref = mm == -INFINITY ? 0.0f : mm;
                f[0] = ptx::ex2_approx(m[0] - ref);
                f[1] = ptx::ex2_approx(m[1] - ref);
                ll = f[0] * l[0] + f[1] * l[1];
            }
            const uint32_t col0 = Layout<D>::col_o(pair ? tile : 0);
            if (x.buffer < 0) {
                // l = 0 only for a row without a key: O = 0, LSE = -inf.
                const float inv = ll != 0.0f ? ptx::rcp_approx(ll) : 0.0f;
                f[0] *= inv;
                f[1] *= inv;
            }
            // The guard was here before the products with the tiles that it goes over; else its flag may be an old one.
            const bool bad = guarded_from(p, x) < x.n && reinterpret_cast<const volatile int*>(smem + L::kFlagOff)[n_part & 7] != 0;
            const bool whole = x.buffer < 0;
            const long long line = whole ? static_cast<long long>(x.q0 + (pair ? tile * p.tok_tile : 0)) * p.hq + x.h * p.group + row_line
                                         : static_cast<long long>(x.buffer) * p.part_rows + tile * kBM + row;
            char* to = whole ? static_cast<char*>(p.o) + line * (2 * D) : reinterpret_cast<char*>(p.part_o) + line * (4 * D);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {   // columns of the tile's stream, or of both
                uint32_t v[32];
                ptx::tmem_ld32_at<0>(row_addr + col0 + c, v);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f[0]);
                if (has[1]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8) {
                        uint32_t u[8];
                        kv4::tc::tmem_ld8(row_addr + Layout<D>::col_o(1) + c + e, u);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[e + k] = __float_as_uint(fmaf(__uint_as_float(u[k]), f[1], __uint_as_float(v[e + k])));
                    }
                }
                if (c + 32 >= D) release();
                if (ll == 0.0f) {   // no key, whatever the values hold
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = 0;
                }
                if (row < rows) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t y[8];
#pragma unroll
                            for (int s = 0; s < 8; ++s)
                                y[s] = ptx::pack2<kBf16>(__uint_as_float(v[16 * e + 2 * s]), __uint_as_float(v[16 * e + 2 * s + 1]));
                            store32(to + 2 * c + 32 * e, wide, y);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) store32(to + 4 * c + 32 * e, true, v + 8 * e);
                    }
                }
                __syncwarp();
            }
            // Values that are not finite, added to what is written: rare, so a small loop.
            if (bad && row < rows && ll != 0.0f) {
                const volatile int* first_bad = reinterpret_cast<const volatile int*>(smem + L::kBadOff) + (n_part & 7) * (2 * D);
                const int seen = x.vis0 + row_tok + (pair ? tile * p.tok_tile : 0);   // the guard is for causal rows only
#pragma unroll 1
                for (int c = 0; c < D; ++c) {
                    const bool up = seen > first_bad[c], down = seen > first_bad[D + c];
                    if (!up && !down) continue;
                    const float add = up && down ? NAN : up ? INFINITY : -INFINITY;
                    if (whole) {
                        uint16_t* y = reinterpret_cast<uint16_t*>(to) + c;
                        float y0, y1;
                        ptx::unpack2<kBf16>(*y, y0, y1);
                        *y = static_cast<uint16_t>(ptx::pack2<kBf16>(y0 + add, 0.0f));
                    } else {
                        reinterpret_cast<float*>(to)[c] += add;
                    }
                }
            }
            if (row < rows) {
                if (whole) p.lse[line] = ll != 0.0f ? (mm + ptx::lg2_approx(ll)) * 0.69314718055994530942f : -INFINITY;
                else *reinterpret_cast<float2*>(p.part_ml + 2 * line) = make_float2(mm, ll);
            }
        }
        if (!ok) break;
    }
}

// ---------------------------------------------------------------- kernels

template <int D, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    fa2_kv16_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmKV, const Params p) {
    using L = Lay<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = ptx::smem_addr(smem);
    BarSet<D> bars;
    bars.base = sbase + L::kBarOff;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
    const Gate gate{sbase + L::kMiscOff + 8};
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bars.q_full(t), 1);
            ptx::mbar_init(bars.q_empty(t), 1);
            ptx::mbar_init(bars.s_full(t), 1);
            ptx::mbar_init(bars.alpha_ready(t), 4);   // a warp's arrival each
            ptx::mbar_init(bars.stats_ready(t), 4);
            ptx::mbar_init(bars.stats_free(t), 4);
            ptx::mbar_init(bars.p_full(t), 8);
            ptx::mbar_init(bars.p_rest(t), 4);
            ptx::mbar_init(bars.o_full(t), 1);
        }
#pragma unroll 1
        for (int s = 0; s < L::kStages; ++s) {
            ptx::mbar_init(bars.kv_full(s), 1);
            ptx::mbar_init(bars.kv_empty(s), 1);
        }
#pragma unroll 1
        for (int s = 0; s < kParts; ++s) {
            ptx::mbar_init(bars.part_full(s), 1);
            ptx::mbar_init(bars.part_empty(s), kPartUsers);
        }
        ptx::mbar_init(bars.mma_done(), 1);
        *abort_flag = 0;
        gate.init();
        ptx::fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        ptx::tma_prefetch_desc(&tmQ);
        ptx::tma_prefetch_desc(&tmKV);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), Layout<D>::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    kv4::enter_stream_order();
    const uint32_t tmem = *tmem_slot;
    const Waiter w{abort_flag, p.wait_limit_ns};

    // The roles' loops share an instruction cache that their program does not fit, so their
    // order counts: a prompt of 4096 tokens takes 136 us in this one, two with heads of 64
    // 186; 136 to 157 and 191 to 206 in eight others of the last four.
    if (warp < kCorrWarp0) {
        ptx::setmaxnreg_inc<kRegSoft>();
        softmax_role<D, kBf16>(p, tmem, smem, bars, w, gate, warp / 4);
    } else if (warp < kLoadWarp) {
        ptx::setmaxnreg_dec<kRegOut>();
        correction_role<D, kBf16>(p, tmem, smem, sbase, bars, w);
    } else {
        ptx::setmaxnreg_dec<kRegRest>();
        if (warp == kSchedWarp) scheduler<D>(p, smem, bars, w);
        else if (warp == kLoadWarp) producer<D>(&tmQ, &tmKV, p, smem, sbase, bars, w);
        else if (warp == kMmaWarp) mma_issuer<D, kBf16>(p, smem, sbase, tmem, bars, w);
        else guard<D, kBf16>(p, smem, sbase, bars, w, gate);
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, Layout<D>::kTmemCols);
    }
}

// Joins the partial results of the row blocks that several CTAs share, and
// writes the rows that no key is visible to where a whole block has none
// (O = 0, LSE = -inf). Block (c, y) has a share of the rows that CTA c began. D / 8
// lanes take a row, eight elements each: 256 rows of two parts in each of 152
// blocks take 13 us by itself with caches cold, 2.8 M warp instructions (17 us and 9.5 M
// with a warp a row and four elements a lane).
template <int D, bool kBf16>
__global__ void __launch_bounds__(kJoinThreads) fa2_kv16_join_kernel(const Params p) {
    constexpr int kLanes = D / 8, kGroups = kJoinThreads / kLanes;
    __shared__ float acc[kGroups][D];
    __shared__ float2 stat[kGroups];
    kv4::enter_stream_order();
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes;
    const int c = blockIdx.x;
    const Begun begun = p.begun[c];
    const uint32_t inv_group = (65536u + p.group - 1) / p.group;
    struct Row {
        float m, l, o[8];
        __device__ __forceinline__ void clear() {
            m = -INFINITY;
            l = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0.0f;
        }
    };
    // Adds parts i, i + step, .. of line r of the buffers, U at a time.
    auto add = [&](auto at_once, Row& x, int r, int i, int step) {
        constexpr int U = decltype(at_once)::value;
        for (; i < begun.parts; i += U * step) {
            float2 ml[U];
            float v[U][8];
#pragma unroll
            for (int e = 0; e < U; ++e) {
                const int part = i + e * step;
                ml[e] = make_float2(-INFINITY, 0.0f);
                if (part >= begun.parts) continue;
                const long long line = (2LL * (c + part) + (part == 0 ? 1 : 0)) * p.part_rows + r;
                ml[e] = *reinterpret_cast<const float2*>(p.part_ml + 2 * line);
                asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                             : "=f"(v[e][0]), "=f"(v[e][1]), "=f"(v[e][2]), "=f"(v[e][3]), "=f"(v[e][4]), "=f"(v[e][5]), "=f"(v[e][6]),
                               "=f"(v[e][7])
                             : "l"(p.part_o + line * D + 8 * lane));
            }
            float top = x.m;
#pragma unroll
            for (int e = 0; e < U; ++e) top = fmaxf(top, ml[e].x);
            const float ref = top == -INFINITY ? 0.0f : top, f0 = ptx::ex2_approx(x.m - ref);
            x.m = top;
            x.l *= f0;
#pragma unroll
            for (int k = 0; k < 8; ++k) x.o[k] *= f0;
#pragma unroll
            for (int e = 0; e < U; ++e) {
                if (ml[e].x == -INFINITY && ml[e].y == 0.0f) continue;   // it saw no key
                const float f = ptx::ex2_approx(ml[e].x - ref);
                x.l = fmaf(f, ml[e].y, x.l);
#pragma unroll
                for (int k = 0; k < 8; ++k) x.o[k] = fmaf(f, v[e][k], x.o[k]);
            }
        }
    };
    auto out_line = [&](int r) {   // in o
        const int tok = by_group(r % kBM, inv_group);
        return static_cast<long long>(begun.q0 + r / kBM * p.tok_tile + tok) * p.hq + begun.h * p.group + (r % kBM - tok * p.group);
    };
    auto finish = [&](const Row& x, int r) {
        const long long line = out_line(r);
        const float inv = x.l != 0.0f ? ptx::rcp_approx(x.l) : 0.0f;
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = ptx::pack2<kBf16>(x.o[2 * k] * inv, x.o[2 * k + 1] * inv);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + line * D + 8 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
        if (lane == 0) p.lse[line] = x.l != 0.0f ? (x.m + ptx::lg2_approx(x.l)) * 0.69314718055994530942f : -INFINITY;
    };
    // Line r of a buffer has a row of the block (lines of the second tile follow the first 128).
    auto there = [&](int r) { return r % kBM < min(begun.ntok - r / kBM * p.tok_tile, p.tok_tile) * p.group; };
    const int lines = begun.ntok > p.tok_tile ? 2 * kBM : kBM;
    Row x;
    if (begun.parts > kGroups) {   // many parts: all groups share those of a row
        for (int r = blockIdx.y; r < lines; r += kJoinY) {
            if (!there(r)) continue;
            x.clear();
            add(std::integral_constant<int, 2>{}, x, r, group, kGroups);
            float4* to = reinterpret_cast<float4*>(&acc[group][8 * lane]);
            to[0] = make_float4(x.o[0], x.o[1], x.o[2], x.o[3]);
            to[1] = make_float4(x.o[4], x.o[5], x.o[6], x.o[7]);
            if (lane == 0) stat[group] = make_float2(x.m, x.l);
            __syncthreads();
            if (threadIdx.x < D / 2) {   // two elements a thread
                float top = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
                for (int e = 0; e < kGroups; ++e) top = fmaxf(top, stat[e].x);
                const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
                for (int e = 0; e < kGroups; ++e) {
                    const float f = ptx::ex2_approx(stat[e].x - ref);
                    const float2 u = *reinterpret_cast<const float2*>(&acc[e][2 * threadIdx.x]);
                    l = fmaf(f, stat[e].y, l);
                    o0 = fmaf(f, u.x, o0);
                    o1 = fmaf(f, u.y, o1);
                }
                const float inv = l != 0.0f ? ptx::rcp_approx(l) : 0.0f;
                const long long line = out_line(r);
                *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + line * D + 2 * threadIdx.x) = ptx::pack2<kBf16>(o0 * inv, o1 * inv);
                if (threadIdx.x == 0) p.lse[line] = l != 0.0f ? (top + ptx::lg2_approx(l)) * 0.69314718055994530942f : -INFINITY;
            }
            __syncthreads();
        }
    } else if (begun.parts > 0) {
        for (int r = blockIdx.y * kGroups + group; r < lines; r += kJoinY * kGroups) {
            if (!there(r)) continue;
            x.clear();
            if (begun.parts <= 2) add(std::integral_constant<int, 2>{}, x, r, 0, 1);
            else add(std::integral_constant<int, 4>{}, x, r, 0, 1);
            finish(x, r);
        }
    }
    // Blocks of rows without a key.
    for (int b = c; b < p.B; b += gridDim.x) {
        const Request r = request(p, b);
        const int none = r.n == 0 ? 0 : r.len == 0 ? r.n : min(r.n, first_block(p, r) * 2 * p.tok_tile);
        const long long lines0 = static_cast<long long>(none) * p.hq, line0 = static_cast<long long>(r.start) * p.hq;
        for (long long i = blockIdx.y * kJoinThreads + threadIdx.x; i < lines0 * (D / 8); i += kJoinY * kJoinThreads)
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + line0 * D)[i] = make_uint4(0, 0, 0, 0);
        for (long long i = blockIdx.y * kJoinThreads + threadIdx.x; i < lines0; i += kJoinY * kJoinThreads) p.lse[line0 + i] = -INFINITY;
    }
}

}  // namespace kv16
}  // namespace fa2
