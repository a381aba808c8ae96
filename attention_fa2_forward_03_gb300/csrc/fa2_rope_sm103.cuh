// Rotary positions with several axes, and the append to a paged 16-bit KV
// cache that applies them on the way (sm_103a).
//
// Of a head's d elements the first R are rotated, as R / 2 pairs (x1, x2): pair
// i by the angle positions[axis of i] * inv_freq[i],
//     y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin,
// in fp32, rounded once. The gradient is the rotation by the opposite angle.
//
// Angles. Far positions leave few of an fp32 product's 24 bits for the angle in
// a turn, and fp64 is slow here, so angles are integers: a frequency is kept
// as u = inv_freq / (2 pi) turns in units of 2^-64, its whole turns dropped
// (24 bits of inv_freq times 64 bits of 1 / (2 pi), shifted), and u * position
// mod 2^64 is the angle in a turn, off by |position| (1 + |inv_freq|) 2^-64 turns
// at most, for any int32 position. sincospif takes it from there.
//
// What bounds it: memory, each element read and written once. An angle is
// made once a token and pair, in shared memory, and serves all heads.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "fa2.h"
#include "fa2_kv4_sm103.cuh"
#include "ptx_sm103.cuh"

namespace fa2 {
namespace rope {

constexpr int kSiteAxis = 56;   // an entry of `axes` outside 0 .. n_axes - 1
constexpr int kThreads = 256;
// Tokens of a block where there are many, items (32 bytes) of a thread in flight
// and blocks an SM. 8191 tokens of 48 heads, one call behind another, take 33 us; 36 with
// 8, 4 and 3 (what 80 registers allow), 34.7 with 2, 2 and 5; 4, 3 and 4 take as long, but 9.2
// us for 2000 tokens instead of 8.5 (2, 2 and 5: 7.7).
constexpr int kTokens = 4, kBatch = 2, kBlocks = 5;

struct Params {
    const void* in[3];          // queries, keys, values (values: the append alone)
    void* out[3];               // of the append: rotated queries; keys and values go to the cache
    int in_b[3], in_h[3], in_n[3];      // strides in elements: batch entry, head, token
    int out_b[2], out_h[2], out_n[2];
    int heads[3];
    const int* positions;       // [n_axes, tokens]
    const float* inv_freq;      // [rot / 2]
    const int* axes;            // [rot / 2] or NULL: all 0
    int tokens, n;              // batch entries times n; tokens of one
    int n_axes, rot;            // rot 0: nothing is rotated
    int interleaved;            // pairs of neighbours, else of halves
    int inverse;
    const int* slots;           // [tokens]: the append alone
    void* cache;                // [num_pages, hkv, 2, page, D]
    int page, log2_page, num_slots;
};

// inv_freq / (2 pi) turns in units of 2^-64, mod 2^64.
__device__ __forceinline__ uint64_t turns_of(float f) {
    constexpr uint64_t kInv2Pi = 0x28BE60DB9391054AULL;   // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(f), field = (bits >> 23) & 255u;
    const uint64_t m = (bits & 0x7FFFFFu) | (field ? 0x800000u : 0u);   // |f| = m 2^e
    const int e = static_cast<int>(field ? field : 1u) - 150;
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    uint64_t u;
    if (e >= 0) u = e < 64 ? lo << e : 0;
    else if (e > -64) u = (lo >> -e) | (hi << (64 + e));
    else u = e > -128 ? hi >> (-e - 64) : 0;
    return bits >> 31 ? 0 - u : u;
}

// The rows of one block: kTok tokens of every head. An item is 16 elements of
// a row: the eight pairs that share a table entry, or 16 neighbours behind R.
template <int D, bool kBf16, bool kCache, int kTok>
__global__ void __launch_bounds__(kThreads, kBlocks) fa2_rope_kernel(const Params p) {
    constexpr int kItems = D / 16;   // of a row
    __shared__ float4 table[kTok][4][kItems];   // cos, sin of pairs 8c + 2k and 8c + 2k + 1 at [k][c]
    __shared__ int2 place[kTok];                // batch entry and token of it
    __shared__ int slot_of[kTok];               // -1: no keys and values to write
    kv4::enter_stream_order();
    const int t0 = blockIdx.x * kTok;
    const int here = min(kTok, p.tokens - t0);
    const int tid = threadIdx.x;

    if (tid < kTok) {
        const int t = t0 + min(tid, here - 1);
        const int b = t / p.n;
        place[tid] = make_int2(b, t - b * p.n);
        if constexpr (kCache) {
            int s = p.slots[t];
            if (s >= p.num_slots) {
                kv4::report(kv4::kSiteSlot);
                s = -1;
            }
            slot_of[tid] = s;
        }
    }
    const int pair = tid % (D / 2);
    if (pair < p.rot / 2) {
        const uint64_t u = turns_of(p.inv_freq[pair]);
        int axis = p.axes ? p.axes[pair] : 0;
        const bool good = static_cast<unsigned>(axis) < static_cast<unsigned>(p.n_axes);
        if (!good && blockIdx.x == 0) kv4::report(kSiteAxis);
#pragma unroll
        for (int i = 0; i < (kTok * D / 2 + kThreads - 1) / kThreads; ++i) {
            const int t = tid / (D / 2) + i * (kThreads / (D / 2));
            if (t >= here) break;
            const long long pos = good ? p.positions[static_cast<long long>(axis) * p.tokens + t0 + t] : 0;
            // signed: a turn is -2^63 .. 2^63, which sincospif takes as -1 .. 1 half turns
            float s, c;
            sincospif(__ll2float_rn(static_cast<long long>(u * static_cast<uint64_t>(pos))) * 0x1p-63f, &s, &c);
            float2* at = reinterpret_cast<float2*>(&table[t][pair % 8 / 2][pair / 8]) + pair % 2;
            *at = make_float2(c, p.inverse ? -s : s);
        }
    }
    __syncthreads();

    const int rows = (p.heads[0] + p.heads[1] + p.heads[2]) * kTok;
    const int c = tid % kItems;
    const bool turned = 16 * c < p.rot;
    // the two vectors of eight elements
    const int a0 = turned && !p.interleaved ? 8 * c : 16 * c;
    const int a1 = turned && !p.interleaved ? p.rot / 2 + 8 * c : 16 * c + 8;
    constexpr int kStep = kThreads / kItems;
    for (int r0 = tid / kItems; r0 < rows; r0 += kBatch * kStep) {
        uint4 x[kBatch][2];
        uint16_t* to[kBatch];
        int which[kBatch];   // token of the block; -1: nothing to do, bit 30: not rotated
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int row = r0 + i * kStep, t = row % kTok;
            int h = row / kTok;
            which[i] = -1;
            if (row >= rows || t >= here) continue;
            int part = 0;
            if (h >= p.heads[0]) {
                h -= p.heads[0];
                part = 1;
                if (kCache && h >= p.heads[1]) {
                    h -= p.heads[1];
                    part = 2;
                }
            }
            const int2 at = place[t];
            if (kCache && part > 0) {
                const int s = slot_of[t];
                if (s < 0) continue;
                const long long line = ((static_cast<long long>(s >> p.log2_page) * p.heads[1] + h) * 2 + (part - 1)) * p.page +
                                       (s & (p.page - 1));
                to[i] = static_cast<uint16_t*>(p.cache) + line * D;
            } else {
                to[i] = static_cast<uint16_t*>(p.out[part]) + static_cast<long long>(at.x) * p.out_b[part] +
                        static_cast<long long>(h) * p.out_h[part] + static_cast<long long>(at.y) * p.out_n[part];
            }
            const uint16_t* from = static_cast<const uint16_t*>(p.in[part]) + static_cast<long long>(at.x) * p.in_b[part] +
                                   static_cast<long long>(h) * p.in_h[part] + static_cast<long long>(at.y) * p.in_n[part];
            which[i] = t | (part == 2 ? 1 << 30 : 0);
            x[i][0] = *reinterpret_cast<const uint4*>(from + (part == 2 ? 16 * c : a0));
            x[i][1] = *reinterpret_cast<const uint4*>(from + (part == 2 ? 16 * c + 8 : a1));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (which[i] < 0) continue;
            const bool plain = which[i] >> 30;
            if (turned && !plain) {
                const int t = which[i];
                uint32_t w[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {   // pairs 8c + 2k and 8c + 2k + 1
                    const float4 cs = table[t][k][c];
                    float u0, u1, v0, v1;
                    if (p.interleaved) {
                        ptx::unpack2<kBf16>(w[2 * k], u0, v0);
                        ptx::unpack2<kBf16>(w[2 * k + 1], u1, v1);
                    } else {
                        ptx::unpack2<kBf16>(w[k], u0, u1);
                        ptx::unpack2<kBf16>(w[k + 4], v0, v1);
                    }
                    const float y0 = u0 * cs.x - v0 * cs.y, z0 = v0 * cs.x + u0 * cs.y;
                    const float y1 = u1 * cs.z - v1 * cs.w, z1 = v1 * cs.z + u1 * cs.w;
                    if (p.interleaved) {
                        w[2 * k] = ptx::pack2<kBf16>(y0, z0);
                        w[2 * k + 1] = ptx::pack2<kBf16>(y1, z1);
                    } else {
                        w[k] = ptx::pack2<kBf16>(y0, y1);
                        w[k + 4] = ptx::pack2<kBf16>(z0, z1);
                    }
                }
                x[i][0] = make_uint4(w[0], w[1], w[2], w[3]);
                x[i][1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            *reinterpret_cast<uint4*>(to[i] + (plain ? 16 * c : a0)) = x[i][0];
            *reinterpret_cast<uint4*>(to[i] + (plain ? 16 * c + 8 : a1)) = x[i][1];
        }
    }
}

}  // namespace rope
}  // namespace fa2
