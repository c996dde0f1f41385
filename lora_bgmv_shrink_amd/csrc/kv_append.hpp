// A row of an append: its place in the cache, the rotation of its heads, and
// the writing of them in a type of the matrix cores (kv.hip; the queries of a
// cache in 8 bits, kv_q8.hip).
#pragma once

#include "kv_internal.hpp"

namespace lora {
namespace {

constexpr int KA_WAVES = 4;    // waves per workgroup, each with a row of its own
constexpr int KA_BATCH = 4;    // items a lane has in flight

// eight consecutive elements, as fp32
template <typename T> struct Eight;
template <> struct Eight<bf16> {
    uint4 u;
    __device__ __forceinline__ void load(const bf16* p) { u = *(const uint4*)p; }
    __device__ __forceinline__ float get(int e) const {
        const uint32_t w = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
        return __uint_as_float((e & 1) ? (w & 0xffff0000u) : (w << 16));
    }
};
template <> struct Eight<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = *(const float4*)p;
        b = *(const float4*)(p + 4);
    }
    __device__ __forceinline__ float get(int e) const {
        const float4& w = e < 4 ? a : b;
        return (e & 3) == 0 ? w.x : (e & 3) == 1 ? w.y : (e & 3) == 2 ? w.z : w.w;
    }
};
__device__ __forceinline__ void store8(bf16* p, const float (&f)[8]) {
    union { uint4 u; bf16 e[8]; } t;
#pragma unroll
    for (int e = 0; e < 8; ++e) t.e[e] = f32_to_bf16(f[e]);
    *(uint4*)p = t.u;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    *(float4*)p = float4{f[0], f[1], f[2], f[3]};
    *(float4*)(p + 4) = float4{f[4], f[5], f[6], f[7]};
}

// A wave takes one row and a run of `it` * 64 items; an item is 16 elements of
// one head in two pieces of 8: for a head rotated in halves, piece c and the
// piece that holds its partners; otherwise two neighbouring pieces.  64 is a
// multiple of a head's items, so a lane keeps the same place in every head it
// visits and loads its cosines and sines once.
// EARLY: the row's elements are requested before its place is looked up, and
// the lookup takes fewer steps.
template <typename TI, typename TO, int D, bool EARLY>
__device__ __forceinline__ void append_row(const AppendArgs& a, int it, int block_row, int run) {
    constexpr int IPH = D / 16;   // items per head
    const int lane = threadIdx.x & 63;
    const int row = __builtin_amdgcn_readfirstlane(block_row * KA_WAVES + (threadIdx.x >> 6));
    const KvBatchDev& B = a.B;
    if (row >= B.n_rows) return;
    const int heads = a.n_q_heads + 2 * a.C.n_kv_heads;
    const int n_items = heads * IPH;

    // pieces of this lane's items inside a head
    const int c = lane & (IPH - 1);
    const int rot = a.cos ? 2 * a.half : 0;
    int e0, e1, p0 = 0;   // first elements of the pieces, first pair
    bool turn = c * 16 < rot;
    const bool halves = turn && !a.interleaved;
    if (halves) {
        p0 = c * 8;
        e0 = c * 8;
        e1 = e0 + a.half;
    } else {
        p0 = c * 8;
        e0 = c * 16;
        e1 = e0 + 8;
    }

    const int end = min(n_items, (int)(run + 1) * it * 64), begin = run * it * 64 + lane;
    Eight<TI> x0[KA_BATCH], x1[KA_BATCH];
    auto request = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < KA_BATCH; ++u) {
            const int i = i0 + u * 64;
            if (i >= end) break;
            const int h = i / IPH;
            const TI* src;
            if (h < a.n_q_heads) src = (const TI*)a.q + (int64_t)row * a.ldq + h * D;
            else if (h < a.n_q_heads + a.C.n_kv_heads)
                src = (const TI*)a.k + (int64_t)row * a.ldk + (h - a.n_q_heads) * D;
            else src = (const TI*)a.v + (int64_t)row * a.ldv + (h - a.n_q_heads - a.C.n_kv_heads) * D;
            const bool plain = h >= a.n_q_heads + a.C.n_kv_heads && halves;
            x0[u].load(src + (plain ? c * 16 : e0));
            x1[u].load(src + (plain ? c * 16 + 8 : e1));
        }
    };
    if (EARLY && begin < end) request(begin);

    // the row's place: sequence, index among its own tokens, page
    int s, r0 = 0, r1 = 0, len = 0;
    bool ok;
    if constexpr (EARLY) {
        ok = wave_find_seq(B, row, lane, [](int, int off) { return off; }, s, r0, r1, len);
    } else {
        s = wave_find_run(B.row_off, B.n_seqs, row, lane);
        ok = s < B.n_seqs;
    }
    int pos = 0;
    int64_t slot = 0;
    if (ok) {
        if constexpr (!EARLY) {
            r1 = B.row_off[s + 1];
            len = B.kv_len[s];
        }
        const int t = len - (r1 - row);
        int before = 0;
        if (B.n_groups) {
            const int g = wave_find_run(B.group_off, B.n_groups, s, lane);
            if (g < B.n_groups) before = max(B.prefix_len[g], 0);
        }
        const int pg = t >> a.C.page_shift;
        ok = t >= 0 && pg < B.ldp;
        const int page = ok ? B.pages[(int64_t)s * B.ldp + pg] : -1;
        pos = before + t;
        ok = ok && page >= 0 && page < a.C.n_pages && (!a.cos || (pos >= 0 && pos < a.n_pos));
        slot = (int64_t)page * a.C.page_stride + (int64_t)(t & ((1 << a.C.page_shift) - 1)) * a.C.token_stride;
        if (!ok && lane == 0 && run == 0 && a.status) flag_bad_id(a.status);
    }
    float cs[8], sn[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        cs[e] = 1.f;
        sn[e] = 0.f;
    }
    if (ok && turn) {
        Eight<float> cv, sv;
        cv.load(a.cos + (int64_t)pos * a.ldr + p0);
        sv.load(a.sin + (int64_t)pos * a.ldr + p0);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cs[e] = cv.get(e);
            sn[e] = sv.get(e);
        }
    }

    for (int i0 = begin; i0 < end; i0 += KA_BATCH * 64) {
        if (!EARLY || i0 != begin) request(i0);
#pragma unroll
        for (int u = 0; u < KA_BATCH; ++u) {
            const int i = i0 + u * 64;
            if (i >= end) break;
            const int h = i / IPH;
            const bool is_q = h < a.n_q_heads;
            const bool is_v = h >= a.n_q_heads + a.C.n_kv_heads;
            float y0[8], y1[8];
            if (is_v || !turn) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    y0[e] = x0[u].get(e);
                    y1[e] = x1[u].get(e);
                }
            } else if (halves) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = x0[u].get(e), q = x1[u].get(e);
                    y0[e] = p * cs[e] - q * sn[e];
                    y1[e] = p * sn[e] + q * cs[e];
                }
            } else {   // neighbouring pairs: piece 0 holds pairs 0..3, piece 1 pairs 4..7
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float p = x0[u].get(2 * e), q = x0[u].get(2 * e + 1);
                    y0[2 * e] = p * cs[e] - q * sn[e];
                    y0[2 * e + 1] = p * sn[e] + q * cs[e];
                    const float r = x1[u].get(2 * e), w = x1[u].get(2 * e + 1);
                    y1[2 * e] = r * cs[e + 4] - w * sn[e + 4];
                    y1[2 * e + 1] = r * sn[e + 4] + w * cs[e + 4];
                }
            }
            TO* dst;
            if (is_q) {
                dst = (TO*)a.q_out + (int64_t)row * a.ldqo + h * D;
                if (!ok) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) y0[e] = y1[e] = 0.f;
                }
            } else {
                if (!ok) continue;
                const int hk = h - a.n_q_heads - (is_v ? a.C.n_kv_heads : 0);
                dst = (TO*)(is_v ? a.C.v : a.C.k) + slot + (int64_t)hk * a.C.head_stride;
            }
            const bool plain = is_v && halves;
            store8(dst + (plain ? c * 16 : e0), y0);
            store8(dst + (plain ? c * 16 + 8 : e1), y1);
        }
    }
}

}  // namespace
}  // namespace lora
