// Attention over a paged cache in 8 bits: the few-column form and the launches.
// The mathematics, and the tiled form, are attn_common.hpp's: a key or value,
// e4m3 times a power of two, is a bf16 number, and from there on this is
// attention over a bf16 cache.
#include "attn_common.hpp"

namespace lora {
namespace {

// A wave's staged values: 64 rows of D bytes as they lie in the cache, 16-byte
// pieces permuted inside a row so that a transposed read (16 bytes of each of
// 32 rows) takes distinct banks.
template <int D>
struct Bytes {
    static constexpr int LPR = D / 16;   // pieces of a row
    static __device__ __forceinline__ constexpr int x(int key) {
        return D == 64 ? (key >> 2) & 3 : D == 128 ? (key >> 1) & 7 : key & 15;
    }
    static __device__ __forceinline__ int at(int key, int piece) { return key * D + ((piece ^ x(key)) << 4); }
};
template <int D>
struct FewStageQ8 {   // LDS of a wave: values and 64 scales of keys and of values, or O and its statistics
    static constexpr int VALUES = 64 * D, KEYS = VALUES + 2 * 64 * 4, OUT = 16 * (D + 4) * 4 + 128;
    static constexpr int WAVE = KEYS > OUT ? KEYS : OUT;
};
__device__ __forceinline__ bool has_nan(const u32x4_t& v) {   // e4m3: seven bits set
    auto bad = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
    return (bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w)) != 0;
}

// Up to 16 columns.  Reading keys and values bounds it, at half the bytes of
// bf16, so a wave takes 64 keys at a time where the bf16 form takes 32, with as
// many bytes in flight.
//
// A product's sum may run in any order, so a lane takes 16 neighbouring numbers
// of a key, as one load gives them, for two steps of it (the queries are laid
// out alike): keys go from memory to the matrix cores without passing LDS, and
// the widening multiplies them by their scale.  Values pass LDS in 8 bits, for
// the transposed reading, and are widened behind it; there a lane holds eight
// keys of one dimension, so their scales go into the weights, which are a
// power of two times what they were and lose nothing by it.  (Both products in 8
// bits would spare the widening, but a query or weight then takes two numbers:
// twice the products for K, and splitting a weight costs more than widening a
// value.  A widening is an ordinary vector instruction, 4.5 cycles a SIMD.)
//
// bf16 queries, 8 key heads of 128, 8 sequences of 16 k to 60 k tokens: 99 us,
// 0.57 GB, 5.7 TB/s, and 6 for the join; 32 sequences of up to 2047 tokens 21.5
// us, 57 MB: a (problem, key head) is on one CU, which takes in no more than some
// 32 KB at a time (31 bytes a ns at a latency of 1 us), so the longest sequence's
// 0.5 MB are 17 us of it.  256 sequences of up to 1000 tokens 104 us, 270 MB: at
// 237 registers a CU holds eight waves, one workgroup, whose chain of loads (its
// problem, its queries and pages, its keys) and end nothing else covers.
template <int D, bool PAGED, int NW>
__device__ __forceinline__ void attn_few_q8(const AttnArgs& a, int kind, int block, int blocks, uint8_t* stage, int* sh) {
    using BT = Bytes<D>;
    using O = Op<bf16>;
    constexpr int KW = ATTN_WAVE_KEYS_Q8;       // keys of a wave's unit
    constexpr int KEYS = NW * KW;
    constexpr int G = KW / 16;                  // groups of 16
    constexpr int KC = D / 64;                  // pieces of a lane's key
    constexpr int NV = BT::LPR;                 // pieces of values per lane
    constexpr int RPL = 64 / BT::LPR;           // keys one load of values covers
    constexpr int WB = FewStageQ8<D>::WAVE;
    static_assert(KW == 64, "a key per lane");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    uint8_t* mine_at = stage + wave * WB;
    float* scales_at = (float*)(mine_at + FewStageQ8<D>::VALUES);   // of keys, then of values
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    const float slack = slack_of(c);
    // this lane's places among the staged values: of the piece it stores, of
    // its eight bytes in a transposed read (keys 4 g4 .. + 3 of two groups)
    const int vst = BT::at(lane / BT::LPR, lane % BT::LPR);
    const int vop = BT::at(((l16 >> 1) & 3) + 4 * g4 + 16 * (l16 >> 3), 0) + (l16 & 1) * 8;

    // m, l of this lane's column (l: this lane's keys only, until the end)
    float m, l;
    f32x4_t acc[D / 16];
    auto work = [&](const Prob& P, const Range& R, int h, int i, int n) __attribute__((always_inline)) {
        bf16x8_t qf[KC][2];
        int col_pos = -1;   // position of this lane's column, -1: no column
        {
            const int j = l16 / a.share;
            const bool there = l16 < P.nr * a.share;
            const bf16* q = (const bf16*)a.q + (int64_t)(P.r0 + j) * a.ldq + (int64_t)(h * a.share + l16 - j * a.share) * D;
#pragma unroll
            for (int s = 0; s < KC; ++s)
#pragma unroll
                for (int e = 0; e < 2; ++e) qf[s][e] = there ? O::load(q + g4 * (D / 4) + s * 16 + e * 8) : O::zero();
            int seq_rows;
            if (there) col_pos = kind == 0 ? P.pos0 + j : a.window > 0 ? row_position(a, P.r0 + j, seq_rows) : P.pos1;
        }
        // the least position of the columns, from which a window reaches back
        int lo_pos = P.pos0;
        if (kind == 1 && a.window > 0) {
            lo_pos = l16 < P.nr * a.share ? col_pos : 0x7fffffff;
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) lo_pos = min(lo_pos, __shfl_xor(lo_pos, x, 64));
            lo_pos = __builtin_amdgcn_readfirstlane(lo_pos);
        }
        auto base_of = [&](int x) __attribute__((always_inline)) { return R.tile(x) * KEYS + wave * KW; };
        // A wave leaves out units at the range's ends of whose keys its rows see
        // none (with a wave of 64 keys, most of a short sequence's).
        auto unseen = [&](int x) __attribute__((always_inline)) {
            const int key = base_of(x), at = P.key0 + key;
            return key >= P.len || at > P.pos1 ||
                   (a.window > 0 && at + KW - 1 <= lo_pos - a.window && at >= a.n_sink);
        };
        while (n > 0 && unseen(i + n - 1)) --n;
        while (n > 0 && unseen(i)) {
            ++i;
            --n;
        }
        // page number of key `lane` of the wave's unit x, -1: none
        auto load_id = [&](int x) __attribute__((always_inline)) {
            const int key = base_of(x) + lane;
            return key < P.len ? P.tbl[key >> a.C.page_shift] : -1;
        };
        // bit k says whether any column sees key k of unit x; place and scale:
        // where key `lane` and its scales are read from (in page 0 where its
        // page number is no good)
        auto seen_of = [&](int x, int id, int64_t& place, int64_t& scale) __attribute__((always_inline)) {
            const int key = base_of(x) + lane, at = P.key0 + key;
            const bool page_ok = id >= 0 && id < a.C.n_pages;
            bool seen = key < P.len && at <= P.pos1;
            if (a.window > 0) seen = seen && (at > lo_pos - a.window || at < a.n_sink);
            if (seen && !page_ok && a.status) flag_bad_id(a.status);
            place = place_of(a, page_ok ? id : 0, key, h);
            scale = scale_at(a, page_ok ? id : 0, key, h);
            return (uint64_t)__ballot(seen && page_ok);
        };
        // Keys through the caches, since two loads share a line (past them the
        // second fetches it again: 32 requests of up to 2047 tokens 25 us, so
        // 21.5); values, whole lines, past them (8 requests of 16 k to 60 k tokens
        // 99 us, both tensors through the caches 107).
        u32x4_t rk[G][KC], rv[NV];
        float ks, vs;   // scales of key `lane`
        auto request_k = [&](int64_t place) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const int64_t off = PAGED ? lane_of(place, 16 * j) : __shfl(place, 16 * j + l16, 64);
                const uint32_t in = (uint32_t)((PAGED ? l16 * (int)a.C.token_stride : 0) + g4 * (D / 4));
#pragma unroll
                for (int s = 0; s < KC; ++s) rk[j][s] = *(const u32x4_t*)((const uint8_t*)a.C.k + off + in + s * 16);
            }
        };
        auto request_v = [&](int64_t place) __attribute__((always_inline)) {
            const int row = lane / BT::LPR;
            const uint32_t in = (uint32_t)((PAGED ? row * (int)a.C.token_stride : 0) + (lane % BT::LPR) * 16);
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                const int64_t off = PAGED ? lane_of(place, j * RPL) : __shfl(place, j * RPL + row, 64);
                rv[j] = piece_at((const uint8_t*)a.C.v + off + in);
            }
        };

        // Walks the wave's units.  NaN among values that some rows do not see
        // (0 times it is NaN) is looked for in the units that rows see in
        // part; where there is some (the answer) the walk is made again with
        // ODD, which leaves it out of the product and adds it to the columns
        // that see it.  One row sees just what `bits` says.
        auto walk = [&](auto ODD) __attribute__((always_inline)) {
            m = -kInf;
            l = 0.f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            bool odd = false;
            if (n == 0) return false;
            // Loads return in order, and a wait is for a number of loads that may
            // still be out: page numbers and scales are requested before the
            // pieces that stay in flight when they are waited for, here as in
            // the loop.
            const int id0 = load_id(i);
            int id = load_id(min(i + 1, i + n - 1));
            int64_t place, scale;
            uint64_t bits = seen_of(i, id0, place, scale);
            ks = a.S.k_scale[scale];
            vs = a.S.v_scale[scale];
            __builtin_amdgcn_sched_barrier(0);
            request_k(place);
            __builtin_amdgcn_sched_barrier(0);
            request_v(place);
            __builtin_amdgcn_sched_barrier(0);
            for (int x = i; x < i + n; ++x) {
                const int next = min(x + 1, i + n - 1);   // after the last unit that one again: nothing branches
                const int lo = P.key0 + base_of(x);
                const uint64_t bits_x = bits;
                const bool all_see = bits_x == ~0ull && lo + KW - 1 <= P.pos0 &&
                                     (a.window == 0 || lo > P.pos1 - a.window);
                scales_at[lane] = power_of(ks);
                scales_at[64 + lane] = power_of(vs);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                // element r of s[j]: key 16 j + 4 g4 + r, this lane's column
                f32x4_t s[G];
                float by[G];
#pragma unroll
                for (int j = 0; j < G; ++j) {
                    by[j] = scales_at[16 * j + l16];
                    s[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
                // (the groups' sums in turn: a product waits for the one before it)
#pragma unroll
                for (int t = 0; t < KC; ++t) {
#pragma unroll
                    for (int j = 0; j < G; ++j) s[j] = O::mma16(widen(rk[j][t].x, rk[j][t].y, by[j]), qf[t][0], s[j]);
#pragma unroll
                    for (int j = 0; j < G; ++j) s[j] = O::mma16(widen(rk[j][t].z, rk[j][t].w, by[j]), qf[t][1], s[j]);
                }
                bits = seen_of(next, id, place, scale);
                id = load_id(min(x + 2, i + n - 1));
                ks = a.S.k_scale[scale];
                vs = a.S.v_scale[scale];
                __builtin_amdgcn_sched_barrier(0);
                request_k(place);
                __builtin_amdgcn_sched_barrier(0);
                if (!all_see) {
                    asm volatile("");
                    hide_rows<NV>(rv, bits_x, here(lane) / BT::LPR, RPL);
                    if (!ODD && P.nr > 1) {
#pragma unroll
                        for (int j = 0; j < NV; ++j) odd |= has_nan(rv[j]);
                    }
                }
                {
                    const int to = here(vst);
#pragma unroll
                    for (int j = 0; j < NV; ++j)
                        *(u32x4_t*)(mine_at + j * RPL * D + (to ^ (BT::x(j * RPL) << 4))) = rv[j];
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                request_v(place);
                if (!all_see) {
                    asm volatile("");   // a branch: most units need no mask
                    const uint64_t mine = sees(a, col_pos, lo, bits_x) >> here(4 * g4);
#pragma unroll
                    for (int j = 0; j < G; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) s[j][r] = (mine >> (16 * j + r)) & 1u ? s[j][r] : -kInf;
                }
                float top = s[0][0];
#pragma unroll
                for (int e = 1; e < 4 * G; ++e) top = max_of(top, s[e >> 2][e & 3]);
                top = max_of(top, __shfl_xor(top, 16, 64));
                top = max_of(top, __shfl_xor(top, 32, 64));
                if (__ballot(top > m + slack)) {
                    const bool up = top > m + slack;   // a column's own matter: its neighbours do not change its bits
                    const float f = up ? exp2_fast((m - top) * c) : 1.f;   // from -infinity: 0
                    l *= f;
#pragma unroll
                    for (int t = 0; t < D / 16; ++t) acc[t] *= f;
                    if (up) m = top;
                }
                const float ref = m == -kInf ? 0.f : m;
                bf16x8_t pf[G / 2];
#pragma unroll
                for (int u = 0; u < G / 2; ++u) {
                    f32x8_t w;
                    float4 by[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) by[e] = *(const float4*)(scales_at + 64 + 16 * (2 * u + e) + 4 * g4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        w[e] = exp2_fast((s[2 * u + (e >> 2)][e & 3] - ref) * c);
                        if (ODD) s[2 * u + (e >> 2)][e & 3] = w[e];
                    }
                    l += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
                    w *= f32x8_t{by[0].x, by[0].y, by[0].z, by[0].w, by[1].x, by[1].y, by[1].z, by[1].w};
                    pf[u] = O::round(w);
                }
                const int va = here(vop);
                const bool clean = ODD && !all_see;
                // values of dimensions 16 t .. and keys 32 u ..: read AHEAD products before they are multiplied
                constexpr int AHEAD = 8, NP = G / 2 * (D / 16);
                typedef int i32x2_t __attribute__((ext_vector_type(2)));
                i32x2_t b[AHEAD];
                auto read = [&](int p) __attribute__((always_inline)) {
                    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t*)(
                        mine_at + 32 * (p / (D / 16)) * D + (va ^ ((p % (D / 16)) << 4))));
                };
#pragma unroll
                for (int p = 0; p < AHEAD; ++p) b[p] = read(p);
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    bf16x8_t vf = widen((uint32_t)b[p % AHEAD].x, (uint32_t)b[p % AHEAD].y, 1.f);
                    if (p + AHEAD < NP) b[p % AHEAD] = read(p + AHEAD);
                    if (clean) O::clean(vf);
                    acc[p % (D / 16)] = O::mma16(vf, pf[p / (D / 16)], acc[p % (D / 16)]);
                }
                if constexpr (!ODD) {
                    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
                        if (p + AHEAD < NP) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    }
                }
                if (clean) {
                    const uint64_t seen = sees(a, col_pos, lo, bits_x);
                    for (int k = 0; k < KW; ++k) {
                        const int e = (k & 3) + 4 * (k >> 4);
                        float wk = 0.f;
#pragma unroll
                        for (int y = 0; y < 4 * G; ++y)
                            if (y == e) wk = s[y >> 2][y & 3];
                        wk = __shfl(wk, ((k >> 2) & 3) * 16 + l16, 64);
                        if (!((seen >> k) & 1)) continue;
#pragma unroll
                        for (int t = 0; t < D / 16; ++t)
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                const int dim = t * 16 + g4 * 4 + y;
                                if ((mine_at[BT::at(k, t) + (dim & 15)] & 0x7f) == 0x7f) acc[t][y] += wk * __builtin_nanf("");
                            }
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
            return __ballot(odd) != 0;
        };
        if (walk(Int<0>{})) walk(Int<1>{});
    };
    few_pieces<KEYS, NW>(a, kind, block, blocks, sh, tid, lane, work,
                                 [&](const Prob& P, int h, bool whole, int slot) __attribute__((always_inline)) {
                                     few_finish<bf16, D, WB, NW>(a, kind, P, h, whole, slot, stage, wave, lane, m, l, acc);
                                 });
}

template <int D_, bool PAGED_, bool TOGETHER>
struct InBytes {
    using T = bf16;
    using TL = Tile<T, D_>;
    static constexpr int D = D_, FEW_WAVES = few_waves_q8(D, TOGETHER), FEW_KEYS = FEW_WAVES * ATTN_WAVE_KEYS_Q8;
    static constexpr int FEW_STAGE = FewStageQ8<D>::WAVE;
    static constexpr int WAVES = D <= 128 ? 2 : 1;
    static constexpr bool PAGED = PAGED_, Q8 = true;
    static __device__ __forceinline__ void few(const AttnArgs& a, int kind, int block, int blocks, uint8_t* stage, int* sh) {
        attn_few_q8<D, PAGED, FEW_WAVES>(a, kind, block, blocks, stage, sh);
    }
};
template <int D>
struct InBytesOf {
    template <bool PAGED, bool TOGETHER> using F = InBytes<D, PAGED, TOGETHER>;
};

}  // namespace

hipError_t launch_attn_q8(const AttnArgs& a, int32_t head_dim, hipStream_t stream) {
    const bool paged = a.C.page_shift >= 4;   // 16 keys of a load
    switch (head_dim) {
        case 64: return launch_form<InBytesOf<64>::template F>(a, paged, stream);
        case 128: return launch_form<InBytesOf<128>::template F>(a, paged, stream);
        default: return launch_form<InBytesOf<256>::template F>(a, paged, stream);
    }
}

}  // namespace lora
