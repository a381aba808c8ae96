// Attention over the 4-bit cache for many query rows a KV head (drafted tokens,
// large groups, chunks of prompts): both products on tcgen05.
//
// Transposed, as in fa2_kv4_sm103.cuh: S^T = K Q^T and O^T += V^T P^T, so that
// the long axis (128 tokens, 128 elements of d) is the M of the instruction and
// the few query rows its N (16 to 64). What bounds it is turning codes into
// fp16, about one instruction an element whatever N is; mma.sync needs the same
// and, at a quarter of the rate, as much time again for the products of 24 rows.
//   K   codes -> fp16 in registers -> tensor memory, a thread a token: the A
//       operand of S^T from there, so that shared memory does not carry it
//   V   codes -> fp16 -> shared memory [token][d], read as an MN-major A
//   Q   [row][d] in shared memory, a K-major B
//   P^T [token][row] in shared memory, an MN-major B
// A thread holds one token's scores of half the rows, so the maximum of a row
// runs over threads; it is looked for only when some score passes the row's
// reference by 2^8 (kTop), as in the other kernel.
//
// Two CTAs an SM; in each eight warps do this work, one issues the products and
// one the copies. Products run while operands are made: S^T of the next tile,
// which has a place of its own, while this tile's values and weights are; O^T
// while the next but one's keys are.
//
// 38 sequences of 8192 tokens, 8 KV heads of 128 (358 MB): 121, 138 and 169 us
// for 32, 48 and 64 rows, where the kernel on mma.sync takes 138 us for 32. Without
// the conversions and weights the same loop takes 68 us, without V's alone 90 us,
// without K's 105 us: issue slots are 59% busy, 4245 instructions a tile of 128
// tokens (1920 of them conversions and their multiplications at the least), and
// the tensor pipe 14%.
#pragma once

#include <type_traits>

#include "fa2_kv4_sm103.cuh"

namespace fa2 {
namespace kv4 {
namespace tc {

constexpr int kLog = 7, kTok = 1 << kLog;   // tokens of a tile
constexpr int kThreads = 256;               // of the eight working warps
constexpr int kAll = kThreads + 64;         // with the one that issues products and the one that loads
constexpr int kSiteTc = 52;                 // a wait for the tensor cores

// Tensor memory: K (fp16 pairs), S^T of two tiles, O^T. Two CTAs an SM.
constexpr uint32_t kColK = 0, kColS = 64, kColO = 192, kCols = 256;

template <int D, int N>
struct Smem {
    static constexpr int kCodes = kTok * D / 2, kScales = kTok * D / 16;
    static constexpr int kV = kCodes, kKs = 2 * kCodes, kVs = 2 * kCodes + kScales, kStage = 2 * kCodes + 2 * kScales;
    alignas(1024) uint8_t v[2][kTok * 128];      // two blocks of 64 elements of d; zeros in the second for D = 64
    alignas(1024) uint8_t p[kTok * 128];
    alignas(1024) uint8_t q[D / 64][N * 128];
    alignas(16) uint8_t code[2][kStage];
    alignas(16) float cref[N / 2][4];            // of two rows: factors, negative references
    float alpha[N], l[N];
    float row_ml[N][2];
    int off[N], mx[N];
    int nan_first[D / 16];                       // first token with a NaN among its values, by scale group
    alignas(8) uint32_t ok[4][2];                // usable 16-token blocks of the last tiles loaded: the first bit of each byte
    unsigned long long bar[12], seen[2];         // seen: as in the other kernel
    uint32_t tmem;
    int abort, last;
};

// Barriers: products done, their operands ready, places of codes (of keys, of
// values; two each) full and free.
enum Bar { kBarS = 0, kBarO = 1, kBarK = 2, kBarP = 3, kBarFull = 4, kBarFree = 8 };

// Barrier of the working warps, and one that also joins a condition.
__device__ __forceinline__ void work_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ bool work_sync_or(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}

// Eight columns of the thread's lane of tensor memory, waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(a));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(a), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// D = A B^T with A from tensor memory (8 columns a step of K = 16) and B
// K-major in shared memory (32 bytes a step, then the next block of 64):
// D / 16 steps, the first of which does not accumulate.
template <int D, uint32_t kBlock>
__device__ __forceinline__ void mma_scores(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc) {
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred e, pf, pt;\n\t.reg .b32 blo, bhi, t0, t1;\n\t.reg .b64 b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pf, %3, %3;\n\tsetp.eq.b32 pt, %3, %3;\n\t"
            "mov.b64 {blo, bhi}, %2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pf;\n\t"
            "add.u32 t0, %1, 8;\n\tadd.u32 t1, blo, 2;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 16;\n\tadd.u32 t1, blo, 4;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 24;\n\tadd.u32 t1, blo, 6;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 32;\n\tadd.u32 t1, blo, %4;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 40;\n\tadd.u32 t1, blo, %5;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 48;\n\tadd.u32 t1, blo, %6;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 56;\n\tadd.u32 t1, blo, %7;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "n"(kBlock), "n"(kBlock + 2), "n"(kBlock + 4),
            "n"(kBlock + 6)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, pf, pt;\n\t.reg .b32 blo, bhi, t0, t1;\n\t.reg .b64 b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 pf, %3, %3;\n\tsetp.eq.b32 pt, %3, %3;\n\t"
            "mov.b64 {blo, bhi}, %2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, pf;\n\t"
            "add.u32 t0, %1, 8;\n\tadd.u32 t1, blo, 2;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 16;\n\tadd.u32 t1, blo, 4;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "add.u32 t0, %1, 24;\n\tadd.u32 t1, blo, 6;\n\tmov.b64 b, {t1, bhi};\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t0], b, %3, pt;\n\t"
            "}" ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc)
            : "memory");
    }
}

// 16-byte piece c of row r of a tile's codes: rows lie one after another, and
// the pieces are swapped so that eight rows' pieces of one place, which a warp
// reads at once, lie in different banks.
template <int D>
__device__ __forceinline__ int code_at(int r, int c) {
    if constexpr (D == 128) return r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
    else return r * 32 + ((c ^ ((r >> 2) & 1)) * 16);
}

// The loading warp: the run's tiles one after another; keys a tile ahead of
// values, as they are used. Eight lanes take a block of 16 tokens (of one page),
// 128 bytes of codes at a time, and every lane has two blocks, so that all
// addresses of a tile are two and constants from them. Page ids are read a tile
// ahead.
template <int D, int N>
__device__ __forceinline__ void load_tiles(const FwdParams& p, Smem<D, N>& sm, Cursor c, int pad, const Waiter& wait) {
    using Sm = Smem<D, N>;
    constexpr int kLines = D / 16, kPieces = D / 32;   // 128-byte lines of a block's codes, 16-byte pieces of a token's
    const int lane = threadIdx.x & 31, piece = lane & 7;
    const uint32_t bars = ptx::smem_addr(sm.bar), block = (lane >> 3) * 8 * D, sblock = (lane >> 3) * D + piece * 16;
    bool ok = !(p.debug_flags & 1);   // test hook: nothing is loaded, and the waits run out
    struct Place {
        const uint8_t* codes[2];   // of the lane's piece in its blocks, keys
        const uint8_t* scales[2];
        bool good[2];
    };

    // One part (0 keys, 1 values) of the run's k-th tile, once there is room.
    auto load = [&](int part, uint32_t k, const Place& x) {
        const int st = 2 * part + (k & 1);
        ok = __all_sync(~0u, wait.wait(bars + 8 * (kBarFree + st), ((k >> 1) & 1) ^ 1, kSiteTc));
        if (!ok) return;
        const uint32_t stage = ptx::smem_addr(sm.code[k & 1]);
        const uint32_t dst = stage + (part ? Sm::kV : 0) + block, dst_s = stage + (part ? Sm::kVs : Sm::kKs) + sblock;
        const int off = part ? p.part : 0;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (x.good[u]) {
#pragma unroll
                for (int j = 0; j < kLines; ++j)   // placed as code_at says
                    copy16(dst + u * (32 * D) + j * 128 + ((piece ^ (j & (kPieces - 1))) * 16), x.codes[u] + off + j * 128);
                if (piece < D / 16) copy16(dst_s + u * (4 * D), x.scales[u] + off);
            }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bars + 8 * (kBarFull + st)) : "memory");
        if (lane == 0) ptx::mbar_arrive(bars + 8 * (kBarFull + st));
    };
    uint32_t k = 0;
    Place now, was;   // was: of the tile whose values are still to be loaded
    while (c.u < c.end && ok) {
        const uint8_t* head = p.cache + static_cast<long long>(c.hr / p.rblocks) * 2 * p.part + piece * 16;
        const int* table = p.block_table + static_cast<long long>(c.b) * p.max_pages;
        const int end = c.tile + part_tiles(c);
        int id[2], mine = c.tile * kTok + (lane >> 3) * 16;
#pragma unroll
        for (int u = 0; u < 2; ++u) id[u] = mine + 64 * u < c.len ? table[(mine + 64 * u) >> p.log2_page] : -1;
        for (int tile = c.tile; tile < end && ok; ++tile, ++k, mine += kTok) {
            uint32_t usable[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                now.good[u] = static_cast<unsigned>(id[u]) < static_cast<unsigned>(p.num_pages);
                if (!now.good[u] && mine + 64 * u < c.len && piece == 0) report(kSitePage);
                usable[u] = __ballot_sync(~0u, now.good[u]);
                const int at = (mine + 64 * u) & (p.page - 1);
                const uint8_t* from = head + static_cast<long long>(id[u]) * p.page_bytes;
                now.codes[u] = from + at * (D / 2);
                now.scales[u] = from + p.page * (D / 2) + at * (D / 16);
            }
            if (tile + 1 < end)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    id[u] = mine + kTok + 64 * u < c.len ? table[(mine + kTok + 64 * u) >> p.log2_page] : -1;
            if (lane == 0) *reinterpret_cast<uint2*>(sm.ok[k & 3]) = make_uint2(usable[0], usable[1]);
            load(0, k, now);
            if (k > 0 && ok) load(1, k - 1, was);
            was = now;
        }
        next_segment<kLog>(p, c, pad);
    }
    if (k > 0 && ok) load(1, k - 1, was);
    copy_wait_all();
}

// The issuing warp: S^T of a segment's first tile, then S^T of each next tile
// and O^T of the one before it, as their operands get ready.
template <int D, int N>
__device__ __forceinline__ void issue_products(const FwdParams& p, Smem<D, N>& sm, Cursor c, int pad, uint32_t tmem,
                                               const Waiter& wait) {
    const uint32_t bars = ptx::smem_addr(sm.bar);
    const uint64_t qdesc = ptx::desc_sw128(ptx::smem_addr(sm.q[0]), 16, 1024);
    const uint64_t vdesc = ptx::desc_sw128(ptx::smem_addr(sm.v[0]), kTok * 128, 1024);
    const uint64_t pdesc = ptx::desc_sw128(ptx::smem_addr(sm.p), kTok * 128, 1024);
    constexpr uint32_t kIdS = ptx::idesc_f16(0, 0, 0, 128, N), kIdO = ptx::idesc_f16(0, 1, 1, 128, N);
    uint32_t n_k = 0, n_p = 0;
    bool ok = true;
    auto scores = [&] {
        ok = __all_sync(~0u, wait.wait(bars + 8 * kBarK, n_k & 1, kSiteTc));
        if (!ok) return;
        ptx::tc_fence_after();
        mma_scores<D, N * 8>(tmem + kColS + (n_k & 1) * 64, tmem + kColK, qdesc, kIdS);
        ptx::tc_commit_elect(bars + 8 * kBarS);
        ++n_k;
    };
    while (c.u < c.end && ok) {
        const int n = part_tiles(c);
        scores();
        for (int i = 0; i < n && ok; ++i) {
            if (i + 1 < n) scores();
            if (!ok) break;
            ok = __all_sync(~0u, wait.wait(bars + 8 * kBarP, n_p & 1, kSiteTc));
            if (!ok) break;
            ++n_p;
            ptx::tc_fence_after();
            ptx::mma_ss_kloop<128, 256, 384, 512, 640, 768, 896, 128, 256, 384, 512, 640, 768, 896, 8>(
                tmem + kColO, vdesc, pdesc, kIdO, i > 0);
            ptx::tc_commit_elect(bars + 8 * kBarO);
        }
        next_segment<kLog>(p, c, pad);
    }
    if (!ok) {   // a wait ran out: let what is in flight finish, as far as it does
        if (n_k) wait.drain(bars + 8 * kBarS, (n_k - 1) & 1);
        if (n_p) wait.drain(bars + 8 * kBarO, (n_p - 1) & 1);
    }
}

// A thread's token and half of d: its codes as fp16 pairs in order, D / 4 of
// them, each multiplied by its scale. nan: groups of 16 whose scale is a NaN,
// which are read as zeros.
template <int D, int N>
__device__ __forceinline__ void decode(uint32_t (&r)[D / 4], uint32_t stage, int part, int tk, int half, bool live, uint32_t& nan) {
    using Sm = Smem<D, N>;
    uint32_t w[D / 16], sb;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint4 v = lds128(stage + (part ? Sm::kV : 0) + code_at<D>(tk, half * (D / 64) + c));
        w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
    }
    const uint32_t sat = stage + (part ? Sm::kVs : Sm::kKs) + tk * (D / 16) + half * (D / 32);
    sb = D == 128 ? lds32(sat) : lds16(sat);
    if (!live) sb = 0;
    nan = 0;
    if (part) {
        nan = ((sb & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;   // bytes 0x7F and 0xFF
        if (nan) sb &= ~((nan >> 7) * 0xFFu);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {   // groups of 16
        const uint32_t sc = e4m3_to_f16(__byte_perm(sb, 0, i * 0x11));
        uint32_t a[4], b[4];
        e2m1_to_f16(w[2 * i], a);
        e2m1_to_f16(w[2 * i + 1], b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            r[8 * i + e] = mul_f16x2(a[e], sc);
            r[8 * i + 4 + e] = mul_f16x2(b[e], sc);
        }
    }
}

// Keys of a tile into tensor memory: column c of a token's lane holds
// elements 2c and 2c + 1.
template <int D, int N>
__device__ __forceinline__ void put_keys(uint32_t tmem_lane, uint32_t stage, int tk, int half) {
    uint32_t r[D / 4], nan;
    decode<D, N>(r, stage, 0, tk, half, true, nan);
    if constexpr (D == 128) ptx::tmem_st32_at<0>(tmem_lane + kColK + half * 32, r);
    else ptx::tmem_st16(tmem_lane + kColK + half * 16, r);
    ptx::tmem_wait_st();
}

// Values of a tile into shared memory: rows of 64 elements, 128-byte swizzle.
template <int D, int N>
__device__ __forceinline__ void put_values(Smem<D, N>& sm, uint32_t stage, int tk, int half, bool live, int pos) {
    uint32_t r[D / 4], nan;
    decode<D, N>(r, stage, 1, tk, half, live, nan);
    if (nan)
        for (int i = 0; i < D / 32; ++i)
            if (nan >> (8 * i + 7) & 1) atomicMin(&sm.nan_first[half * (D / 32) + i], pos);
    const uint32_t row = ptx::smem_addr(sm.v[D == 128 ? half : 0]) + tk * 128;
    const int c0 = D == 128 ? 0 : half * 4;
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
        ptx::st_shared_v4(row + (((c0 + c) ^ (tk & 7)) * 16), r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
}

__device__ __forceinline__ int ordered(float x) {   // order-preserving, for integer maxima
    const int i = __float_as_int(x);
    return i >= 0 ? i : i ^ 0x7FFFFFFF;
}
__device__ __forceinline__ float unordered(int i) { return __int_as_float(i >= 0 ? i : i ^ 0x7FFFFFFF); }

// Rows of q as fp16 (scaled as in the other kernel's stage_q), K-major with
// the 128-byte swizzle, and the rows' factors.
template <int D, int N, bool kBf16>
__device__ __forceinline__ void stage_q(const FwdParams& p, Smem<D, N>& sm, const Cursor& c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3;
    const int h = c.hr / p.rblocks, r0 = (c.hr - h * p.rblocks) * N;
    const float c0 = p.scale_log2 * p.k_descale[h];
    for (int r = warp * 8 + (lane >> 2); r < N; r += kThreads / 4) {
        uint32_t w[D / 8];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) w[j] = 0;
        if (r0 + r < p.rows) {
            const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                                  ((static_cast<long long>(c.b) * p.hkv + h) * p.rows + r0 + r) * D + t * (D / 4);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                const uint4 v = reinterpret_cast<const uint4*>(src)[j];
                w[4 * j] = v.x; w[4 * j + 1] = v.y; w[4 * j + 2] = v.z; w[4 * j + 3] = v.w;
            }
        }
        float f = c0;
        if constexpr (kBf16) {
            const uint32_t quad = 0xFu << (lane & 28);   // the lanes of this row
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
            top = max(top, __shfl_xor_sync(quad, top, 1));
            top = max(top, __shfl_xor_sync(quad, top, 2));
            const int e = static_cast<int>(top >> 7);   // biased exponent of the largest magnitude
            const int k = e == 255 ? 0 : min(14 + 127 - e, 126);
            const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
            f *= __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                float lo, hi;
                ptx::unpack2<true>(w[j], lo, hi);
                w[j] = ptx::pack2<false>(lo * up, hi * up);
            }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
            const int piece = t * (D / 32) + j;   // 8 elements
            ptx::st_shared_v4(ptx::smem_addr(sm.q[piece >> 3]) + r * 128 + (((piece & 7) ^ (r & 7)) * 16), w[4 * j], w[4 * j + 1],
                              w[4 * j + 2], w[4 * j + 3]);
        }
        if (t == 0) {
            sm.cref[r / 2][r & 1] = f;
            sm.cref[r / 2][2 + (r & 1)] = INFINITY;
            sm.off[r] = p.causal && r0 + r < p.rows ? p.nq - 1 - (r0 + r) % p.nq : 0;
            sm.mx[r] = ordered(-INFINITY);
        }
    }
    if (threadIdx.x < D / 16) sm.nan_first[threadIdx.x] = 0x7FFFFFFF;
}

template <int D, int N, bool kBf16>
__global__ void __launch_bounds__(kAll, 2) fa2_kv4_fwd_tc_kernel(const FwdParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using Sm = Smem<D, N>;
    Sm& sm = *reinterpret_cast<Sm*>(smem + ((1024 - (ptx::smem_addr(smem) & 1023)) & 1023));
    constexpr int H = N / 2;   // rows a thread works on
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int half = warp >> 2, tk = (warp & 3) * 32 + lane;   // half of d (or of the rows); token, or element of d

    enter_stream_order();
    Cursor cur;
    int per = 0, pad = 1;
    if (locate<1, kLog>(p, cur, per, pad)) {
        const uint32_t bars = ptx::smem_addr(sm.bar);
        if (tid == 0) {
            ptx::mbar_init(bars + 8 * kBarS, 1);
            ptx::mbar_init(bars + 8 * kBarO, 1);
            ptx::mbar_init(bars + 8 * kBarK, kThreads / 32);
            ptx::mbar_init(bars + 8 * kBarP, kThreads / 32);
            for (int s = 0; s < 4; ++s) {
                ptx::mbar_init(bars + 8 * (kBarFull + s), 33);   // the lanes' copies, and what they left out
                ptx::mbar_init(bars + 8 * (kBarFree + s), kThreads / 32);
            }
            sm.abort = 0;
            ptx::fence_mbar_init();
        }
        if (warp == 0) {
            ptx::tmem_alloc(ptx::smem_addr(&sm.tmem), kCols);
            ptx::tmem_relinquish();
        }
        if (D == 64)
            for (int i = tid; i < kTok * 8; i += kAll) reinterpret_cast<uint4*>(sm.v[1])[i] = make_uint4(0, 0, 0, 0);
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        const uint32_t tmem = sm.tmem;
        const uint32_t lane_at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const Waiter wait{&sm.abort, p.wait_limit_ns};
        uint32_t n_s = 0, n_o = 0;   // products waited for so far
        uint32_t k = 0;              // tiles so far: the places of the next, and how often they were used
        // the token's row of weights; a row's place in it is chosen by exclusive or
        const uint32_t p_row = ptx::smem_addr(sm.p) + tk * 128 + (tk & 7) * 16;
        bool ok = true;
        auto arrive = [&](int bar) {   // one arrival a warp, behind all its lanes' writes
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bars + 8 * bar);
        };

        if (warp == kThreads / 32) issue_products<D, N>(p, sm, cur, pad, tmem, wait);
        else if (warp > kThreads / 32) load_tiles<D, N>(p, sm, cur, pad, wait);
        else while (true) {
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
            next_segment<kLog>(p, nxt, pad);
            const bool more = nxt.u < nxt.end;
            const int low = p.causal ? cur.len - p.nq + 1 : cur.len;   // keys before it are seen by every row

            // Keys of the run's k-th tile, as soon as its codes are there
            auto keys = [&](uint32_t k) {
                ok = wait.wait(bars + 8 * (kBarFull + (k & 1)), (k >> 1) & 1, kSiteTc) && ok;
                put_keys<D, N>(lane_at, ptx::smem_addr(sm.code[k & 1]), tk, half);
                ptx::tc_fence_before();
                arrive(kBarK);
                arrive(kBarFree + (k & 1));
            };
            stage_q<D, N, kBf16>(p, sm, cur);
            ptx::fence_proxy_async_smem();
            work_sync();   // row factors
            keys(k);
            uint64_t l[H / 2];   // the thread's tokens' part of the row sums, two rows a register pair
#pragma unroll
            for (int j = 0; j < H / 2; ++j) l[j] = 0;

            for (int i = 0; i < n; ++i, ++k) {
                const int tok0 = (cur.tile + i) * kTok, pos = tok0 + tk;
                const bool live = pos < cur.len && (sm.ok[k & 3][tk >> 6] >> (tk >> 4 & 3) * 8 & 1);
                const uint32_t s_at = lane_at + kColS + (k & 1) * 64 + half * H;
                ok = wait.wait(bars + 8 * kBarS, n_s & 1, kSiteTc) && ok;
                ++n_s;
                ptx::tc_fence_after();
                if (i + 1 < n) keys(k + 1);   // their product runs while this tile's weights are made
                if (i > 0) {   // the values' place is free when the last product with them is done
                    ok = wait.wait(bars + 8 * kBarO, n_o & 1, kSiteTc) && ok;
                    ++n_o;
                    ptx::tc_fence_after();
                }
                ok = wait.wait(bars + 8 * (kBarFull + 2 + (k & 1)), (k >> 1) & 1, kSiteTc) && ok;
                put_values<D, N>(sm, ptx::smem_addr(sm.code[k & 1]), tk, half, live, pos);
                arrive(kBarFree + 2 + (k & 1));

                // The thread's token and its half of the rows: exponents, then
                // weights, which go to shared memory and into the row sums.
                uint64_t x[H / 2];
                auto exponents = [&](auto masked) {
                    float top = -INFINITY;
#pragma unroll
                    for (int j0 = 0; j0 < H; j0 += 8) {
                        uint32_t s[8];
                        tmem_ld8(s_at + j0, s);
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            const int row = half * H + j0 + j;
                            const uint4 cr = lds128(ptx::smem_addr(sm.cref[row / 2]));
                            uint64_t x2 = ptx::f2_fma(ptx::f2_pack(__uint_as_float(s[j]), __uint_as_float(s[j + 1])),
                                                      ptx::f2_pack(__uint_as_float(cr.x), __uint_as_float(cr.y)),
                                                      ptx::f2_pack(__uint_as_float(cr.z), __uint_as_float(cr.w)));
                            float x0, x1;
                            ptx::f2_unpack(x2, x0, x1);
                            if constexpr (decltype(masked)::value) {
                                if (!live || pos >= cur.len - sm.off[row]) x0 = -INFINITY;
                                if (!live || pos >= cur.len - sm.off[row + 1]) x1 = -INFINITY;
                                x2 = ptx::f2_pack(x0, x1);
                            }
                            top = ptx::max3(top, x0, x1);
                            x[(j0 + j) / 2] = x2;
                        }
                    }
                    return top;
                };
                auto weights = [&](bool add) {
#pragma unroll
                    for (int j0 = 0; j0 < H; j0 += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float p0, p1;
                            ptx::f2_unpack(x[j0 / 2 + j], p0, p1);
                            p0 = ptx::ex2_approx(p0);
                            p1 = ptx::ex2_approx(p1);
                            w[j] = ptx::pack2<false>(p0, p1);
                            if (add) l[j0 / 2 + j] = ptx::f2_add(l[j0 / 2 + j], ptx::f2_pack(p0, p1));
                        }
                        ptx::st_shared_v4(p_row ^ ((half * H + j0) * 2), w[0], w[1], w[2], w[3]);
                    }
                };
                const bool all = __all_sync(~0u, live) && tok0 + kTok <= low;
                const float top = all ? exponents(std::false_type{}) : exponents(std::true_type{});
                const bool up = __any_sync(~0u, top > kTop);
                weights(!up);   // those past the reference may be infinite, and are done again
                ptx::fence_proxy_async_smem();
                ptx::tc_fence_before();
                if (work_sync_or(up || !ok)) {
                    if (work_sync_or(*static_cast<volatile int*>(&sm.abort) != 0)) {   // all or none
                        ok = false;
                        break;
                    }
                    // Rarely: the rows' maxima over the tile, new references, results rescaled.
#pragma unroll
                    for (int j0 = 0; j0 < H; j0 += 8) {
                        uint32_t s[8];
                        tmem_ld8(s_at + j0, s);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int row = half * H + j0 + j;
                            const bool hide = !live || pos >= cur.len - sm.off[row];
                            const float v = __uint_as_float(s[j]);
                            const int mx = __reduce_max_sync(~0u, ordered(hide || isnan(v) ? -INFINITY : v));
                            if (lane == 0) atomicMax(&sm.mx[row], mx);
                        }
                    }
                    work_sync();
                    if (tid < N) {
                        float* cr = sm.cref[tid / 2] + (tid & 1);
                        const float was = -cr[2], mx = unordered(sm.mx[tid]);
                        const float ref = mx == -INFINITY ? was : fmaxf(was, fmaf(mx, cr[0], -kLift));
                        // before a row's first score its sums are 0 and have no reference
                        sm.alpha[tid] = was == -INFINITY ? 1.0f : ptx::ex2_approx(was - ref);
                        cr[2] = -ref;
                        sm.mx[tid] = ordered(-INFINITY);
                    }
                    work_sync();
#pragma unroll
                    for (int j0 = 0; j0 < H; j0 += 8) {
                        if (i > 0) {
                            uint32_t o[8];
                            tmem_ld8(lane_at + kColO + half * H + j0, o);
#pragma unroll
                            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sm.alpha[half * H + j0 + j]);
                            tmem_st8(lane_at + kColO + half * H + j0, o);
                        }
#pragma unroll
                        for (int j = 0; j < 8; j += 2)
                            l[(j0 + j) / 2] = ptx::f2_mul(l[(j0 + j) / 2], ptx::f2_pack(sm.alpha[half * H + j0 + j], sm.alpha[half * H + j0 + j + 1]));
                    }
                    ptx::tmem_wait_st();
                    // What a warp without such a score added is right after the rescaling.
                    exponents(std::true_type{});
                    weights(up);
                    ptx::fence_proxy_async_smem();
                    ptx::tc_fence_before();
                    work_sync();
                }
                arrive(kBarP);
            }
            if (ok) {
                ok = wait.wait(bars + 8 * kBarO, n_o & 1, kSiteTc);
                ++n_o;
            }
            copy_wait_all();   // the segment's counter
            if (work_sync_or(!ok)) break;
            ptx::tc_fence_after();

            // Row sums over the tokens: every warp adds up its 32.
            float* sums = reinterpret_cast<float*>(sm.p);   // [4][N]
#pragma unroll
            for (int j = 0; j < H / 2; ++j) {
                float x0, x1;
                ptx::f2_unpack(l[j], x0, x1);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    x0 += __shfl_xor_sync(~0u, x0, o);
                    x1 += __shfl_xor_sync(~0u, x1, o);
                }
                if (lane == 0) {
                    sums[(warp & 3) * N + half * H + 2 * j] = x0;
                    sums[(warp & 3) * N + half * H + 2 * j + 1] = x1;
                }
            }
            work_sync();
            const long long row0 = (static_cast<long long>(cur.b) * p.hkv + h) * p.rows + rb * N;
            const int rows = min(N, p.rows - rb * N);
            const int slot = 2 * blockIdx.x + (c0 == static_cast<int>(blockIdx.x) ? 1 : 0);
            if (tid < N) {
                const float sum = (sums[tid] + sums[N + tid]) + (sums[2 * N + tid] + sums[3 * N + tid]);
                const float ref = -sm.cref[tid / 2][2 + (tid & 1)], m = sum == 0.0f ? -INFINITY : ref == -INFINITY ? 0.0f : ref;
                sm.l[tid] = sum;
                if (tid < rows) {
                    if (split)
                        *reinterpret_cast<float2*>(p.part_ml + (static_cast<long long>(slot) * N + tid) * 2) = make_float2(m, sum);
                    else
                        p.lse[row0 + tid] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
                }
            }
            work_sync();
            // O^T: the thread's element of d for its half of the rows
            const int nan_at = tk < D ? sm.nan_first[min(tk, D - 1) / 16] : 0x7FFFFFFF;
#pragma unroll
            for (int j0 = 0; j0 < H; j0 += 8) {
                uint32_t o[8];
                tmem_ld8(lane_at + kColO + half * H + j0, o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int row = half * H + j0 + j;
                    if (row < rows && tk < D) {
                        float x = __uint_as_float(o[j]);
                        if (nan_at < cur.len - sm.off[row]) x = NAN;
                        const float sum = sm.l[row];
                        if (split) {
                            p.part_o[(static_cast<long long>(slot) * N + row) * D + tk] = x;
                        } else {
                            const uint32_t w = ptx::pack2<kBf16>(sum == 0.0f ? 0.0f : x * (v_descale / sum), 0.0f);
                            static_cast<uint16_t*>(p.o)[(row0 + row) * D + tk] = static_cast<uint16_t>(w);
                        }
                    }
                }
            }
            ptx::tc_fence_before();
            work_sync();

            if (split)
                finish_part<D, N, kThreads, kBf16>(p, c0, c1, sm.seen, sm.last, reinterpret_cast<float*>(sm.v[0]), sm.row_ml, rows,
                                                   row0, v_descale, [] { work_sync(); });
            if (!more) break;
            cur = nxt;
        }
        ptx::tc_fence_before();
        __syncthreads();
        if (warp == 0) {
            ptx::tc_fence_after();
            ptx::tmem_dealloc(tmem, kCols);
        }
    }

    idle_requests<D, kBf16, kAll>(p);
}

}  // namespace tc
}  // namespace kv4
}  // namespace fa2
