// Attention over a paged cache in bf16 or fp32: the few-column form, the plan
// of a batch and the launches.  The mathematics and the tiled form:
// attn_common.hpp.
#include "attn_common.hpp"

namespace lora {
namespace {

// ---------------------------------------------------------------------------
// Few query columns (decode): the keys are split
// ---------------------------------------------------------------------------

// Up to 16 columns (query heads of one key head, times the sequence's rows).
// Reading the visible keys and values bounds it: 4 * 16 columns * D flop per
// 4 D bytes of bf16 keep the matrix cores below a quarter of their rate.
//
// A work unit is 128 keys of one (problem, key head); each of the four waves
// takes 32 of them through LDS of its own (no barrier; values take the keys'
// place once those are multiplied), with the next unit's pieces in flight in
// registers and the unit after's page numbers before them.  At 128 dimensions
// that is 253 registers a lane, two workgroups a CU (and 149 scalar registers
// kept in vector lanes); at 64, three.  Shared form (few = 2): the units of
// all problems are dealt to the workgroups in equal runs, whatever the
// lengths; a run's first and last (problem, head) may be partial and go to
// slots that the join adds.  Otherwise a workgroup takes one (problem, head)
// whole.
//
// bf16, 8 key heads of 128, 8 sequences of 16 k to 60 k tokens: 189 us, 1.14
// GB, 6.0 TB/s (a plain read of this shape: 6.5); 256 sequences that see 1024
// tokens and 4 sinks: 180 us, 0.94 GB seen and, in whole units, 1.14 GB read,
// 6.3 TB/s; 32 sequences of up to 2048 tokens: 32 us, 4.2 TB/s, of which some
// 6 us are a piece's beginning (its problem, its q, its first keys: loads that
// depend on one another) and its end.
template <typename T, int D>
struct FewStage {   // LDS of a wave: 32 keys, or 16 columns of O and their statistics
    static constexpr int KEYS = ATTN_FEW_KEYS / 4 * Tile<T, D>::RB, OUT = 16 * (D + 4) * 4 + 128;
    static constexpr int WAVE = KEYS > OUT ? KEYS : OUT;
};
template <typename T, int D, bool PAGED>
__device__ __forceinline__ void attn_few(const AttnArgs& a, int kind, int block, int blocks, uint8_t* stage, int* sh) {
    using TL = Tile<T, D>;
    using O = Op<T>;
    constexpr int KW = ATTN_FEW_KEYS / 4;            // keys of a wave's unit
    constexpr int NL = KW * TL::LPR / 64;            // pieces per lane, of K and of V
    constexpr int RPL = 64 / TL::LPR;                // rows one load covers
    constexpr int WB = FewStage<T, D>::WAVE;         // LDS bytes of a wave
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    uint8_t* mine_at = stage + wave * WB;   // keys, and then values in their place
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    const float slack = slack_of(c);
    // this lane's places in its stage: of the pieces it stores, of its operands
    const int kst = TL::k_at(lane / TL::LPR, lane % TL::LPR), vst = TL::v_at(lane / TL::LPR, lane % TL::LPR);
    const int kop = TL::k_at(l16, TL::piece_of(g4 * 8)), vop = TL::v_base(4 * g4, 0, l16);

    // m, l of this lane's column (l: this lane's keys only, until the end)
    float m, l;
    f32x4_t acc[D / 16];
    auto work = [&](const Prob& P, const Range& R, int h, int i, int n) __attribute__((always_inline)) {
        typename O::frag qf[D / 32];
        int col_pos = -1;   // position of this lane's column, -1: no column
        {
            const int j = l16 / a.share;
            const bool there = l16 < P.nr * a.share;
            const T* q = (const T*)a.q + (int64_t)(P.r0 + j) * a.ldq + (int64_t)(h * a.share + l16 - j * a.share) * D;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) qf[s] = there ? O::load(q + s * 32 + g4 * 8) : O::zero();
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

        // page number of key `lane` of the wave's unit x (lanes 0 .. 31), -1: none
        auto load_id = [&](int x) __attribute__((always_inline)) {
            const int key = R.tile(x) * ATTN_FEW_KEYS + wave * KW + lane;
            return lane < KW && key < P.len ? P.tbl[key >> a.C.page_shift] : -1;
        };
        u32x4_t rk[NL], rv[NL];
        auto base_of = [&](int x) __attribute__((always_inline)) { return R.tile(x) * ATTN_FEW_KEYS + wave * KW; };
        // bit k says whether any column sees key k of unit x; place: where key
        // `lane` is read from (in page 0 where its page number is no good)
        auto seen_of = [&](int x, int id, int64_t& place) __attribute__((always_inline)) {
            const int key = base_of(x) + lane, at = P.key0 + key;
            const bool page_ok = id >= 0 && id < a.C.n_pages;
            bool seen = lane < KW && key < P.len && at <= P.pos1;
            if (a.window > 0) seen = seen && (at > lo_pos - a.window || at < a.n_sink);
            if (seen && !page_ok && a.status) flag_bad_id(a.status);
            place = place_of(a, page_ok ? id : 0, key, h);
            return (uint32_t)__ballot(seen && page_ok);
        };
        auto stored = [&](const u32x4_t (&r)[NL], int at, auto x) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < NL; ++j) *(u32x4_t*)(mine_at + j * RPL * TL::RB + (at ^ (x(j * RPL) << 4))) = r[j];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        };
        // one unit, whose keys are staged; `values` stages its values
        auto compute = [&](int x, uint32_t bits, bool all_see, auto values, auto ODD) __attribute__((always_inline)) {
            const uint8_t* sk = mine_at;
            const uint8_t* sv = mine_at;
            f32x4_t s[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
            const int ka = here(kop), va = here(vop);
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                const int at = ka ^ (TL::piece_of(ks * 32) << 4);
                s[0] = O::mma16(TL::k_frag(sk, at), qf[ks], s[0]);
                s[1] = O::mma16(TL::k_frag(sk + 16 * TL::RB, at), qf[ks], s[1]);
            }
            values();
            // element r of s[t]: key 16 t + 4 g4 + r, this lane's column
            const int lo = P.key0 + base_of(x);
            if (!all_see) {
                asm volatile("");   // a branch: most tiles need no mask
                const uint32_t mine = (uint32_t)sees(a, col_pos, lo, bits) >> here(4 * g4);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[t][r] = (mine >> (16 * t + r)) & 1u ? s[t][r] : -kInf;
            }
            float top = max_of(max_of(max_of(s[0][0], s[0][1]), max_of(s[0][2], s[0][3])),
                               max_of(max_of(s[1][0], s[1][1]), max_of(s[1][2], s[1][3])));
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
            f32x8_t w;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[r] = exp2_fast((s[0][r] - ref) * c);
                w[4 + r] = exp2_fast((s[1][r] - ref) * c);
            }
            l += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
            const typename O::frag pf = O::round(w);
            if (!ODD || all_see) {
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
                    acc[t] = O::mma16(TL::template v_frag<0, 16>(sv + (va ^ (TL::piece_of(t * 16) << 4))), pf, acc[t]);
                return;
            }
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                typename O::frag vf = TL::template v_frag<0, 16>(sv + (va ^ (TL::piece_of(t * 16) << 4)));
                O::clean(vf);
                acc[t] = O::mma16(vf, pf, acc[t]);
            }
            const uint32_t seen = (uint32_t)sees(a, col_pos, lo, bits);
            for (int k = 0; k < KW; ++k) {
                const int r = (k & 3) + 4 * (k >> 4);
                float wk = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e == r) wk = w[e];
                wk = __shfl(wk, ((k >> 2) & 3) * 16 + l16, 64);
                if (!((seen >> k) & 1)) continue;
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = TL::v_one(sv, k, t * 16 + g4 * 4 + e);
                        if (non_finite(y)) acc[t][e] += wk * y;
                    }
            }
        };

        // Walks the wave's units.  Infinities or NaN among values that some
        // rows do not see (0 times them is NaN) are looked for in the units
        // that rows see in part; where there are some (the answer) the walk is
        // made again with ODD, which leaves them out of the product and adds
        // them to the columns that see them.  One row sees just what `bits`
        // says.
        auto walk = [&](auto ODD) __attribute__((always_inline)) {
            m = -kInf;
            l = 0.f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            bool odd = false;
            if (n == 0) return false;
            int id = load_id(i);
            int64_t place;
            uint32_t bits = seen_of(i, id, place);
            request<T, D, NL, RPL, PAGED>(a, a.C.k, place, lane, rk);
            request<T, D, NL, RPL, PAGED>(a, a.C.v, place, lane, rv);
            id = load_id(min(i + 1, i + n - 1));
            for (int x = i; x < i + n; ++x) {
                const int next = min(x + 1, i + n - 1);   // after the last unit that one again: nothing branches
                const int lo = P.key0 + base_of(x);
                const uint32_t bits_x = bits;
                const bool all_see = bits_x == 0xffffffffu && lo + KW - 1 <= P.pos0 &&
                                     (a.window == 0 || lo > P.pos1 - a.window);
                stored(rk, here(kst), [](int row) { return TL::kx(row); });
                bits = seen_of(next, id, place);
                id = load_id(min(x + 2, i + n - 1));
                request<T, D, NL, RPL, PAGED>(a, a.C.k, place, lane, rk);
                compute(x, bits_x, all_see, [&]() __attribute__((always_inline)) {
                    if (!all_see) {
                        asm volatile("");
                        hide_rows<NL>(rv, bits_x, here(lane) / TL::LPR, RPL);
                        if (!ODD && P.nr > 1) {
#pragma unroll
                            for (int j = 0; j < NL; ++j) odd |= odd_piece<T>(rv[j]);
                        }
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                    stored(rv, here(vst), [](int row) { return TL::vx(row); });
                    request<T, D, NL, RPL, PAGED>(a, a.C.v, place, lane, rv);
                }, ODD);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
            return __ballot(odd) != 0;
        };
        if (walk(Int<0>{})) walk(Int<1>{});

    };
    few_pieces<ATTN_FEW_KEYS, 4>(a, kind, block, blocks, sh, tid, lane, work,
                              [&](const Prob& P, int h, bool whole, int slot) __attribute__((always_inline)) {
                                  few_finish<T, D, WB, 4>(a, kind, P, h, whole, slot, stage, wave, lane, m, l, acc);
                              });
}

template <typename T_, int D_, bool PAGED_>
struct Plain {
    using T = T_;
    using TL = Tile<T, D_>;
    static constexpr int D = D_, FEW_KEYS = ATTN_FEW_KEYS, FEW_STAGE = FewStage<T, D>::WAVE;
    static constexpr int FEW_WAVES = 4;
    static constexpr int WAVES = sizeof(T) * D <= 256 ? 2 : 1;
    static constexpr bool PAGED = PAGED_, Q8 = false;
    static __device__ __forceinline__ void few(const AttnArgs& a, int kind, int block, int blocks, uint8_t* stage, int* sh) {
        attn_few<T, D, PAGED>(a, kind, block, blocks, stage, sh);
    }
};
template <typename T, int D>
struct PlainOf {
    template <bool PAGED, bool> using F = Plain<T, D, PAGED>;
};
template <typename T, int D>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
    return launch_form<PlainOf<T, D>::template F>(a, (1 << a.C.page_shift) >= 64 / Tile<T, D>::LPR, stream);
}

}  // namespace

void plan_attn(AttnPlan& P, int32_t head_dim, int32_t elem_bytes, const int32_t (&n_prob)[2], const int32_t (&max_rows)[2],
               const int32_t (&max_len)[2], bool in_8_bits) {
    // The workspace's parts grow with every bound and do not rest on the
    // window (with one there are fewer keys, so fewer shared units and no more
    // splits), so that one allocation serves every smaller batch.
    AttnArgs& a = P.a;
    const int hkv = a.C.n_kv_heads;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = align_up(at + bytes, 256);
        return o;
    };
    a.join = n_prob[1] > 0 ? 1 : 0;
    a.need_join = a.join;
    const int64_t cols[2] = {(int64_t)max_rows[0] * a.share, (int64_t)max_rows[1] * a.share};   // of a problem, at most
    // 256 columns a tile (8 waves) halve what a column's keys cost to stage;
    // with fewer columns than that half of the waves would have none, longer
    // rows do not leave the registers (kWide), and where the wide tiles would
    // not fill the card narrow ones go twice as far (twelve prompts behind
    // three prefixes 103 us, in wide tiles 111).
    a.decode = cols[0] <= ATTN_FEW_COLS;
    const int64_t wide_items = ((int64_t)a.B.n_rows * a.share / 256 + std::min(n_prob[0], a.B.n_rows)) * hkv;
    a.tile_cols = (a.join && a.decode) || head_dim * elem_bytes > 256 || wide_items < 256 ||
                          std::max(cols[0], n_prob[1] > 0 ? cols[1] : 0) <= 128 ? 128 : 256;
    // Both forms in one launch where both have work and tiles of 128 columns
    // do: 32 requests behind a prefix of 4096 tokens 31 us, in two launches
    // 43; a few fp32 rows and a short prompt 21 us, in two launches 30.
    const bool tiles = (n_prob[0] > 0 && cols[0] > ATTN_FEW_COLS) || (n_prob[1] > 0 && cols[1] > ATTN_FEW_COLS);
    a.together = a.tile_cols == 128 && tiles && (n_prob[0] > 0 || n_prob[1] > 0) && a.share <= ATTN_FEW_COLS && a.B.n_rows > 0;
    const int few_waves = in_8_bits ? few_waves_q8(head_dim, a.together) : 4;
    const int few_keys = in_8_bits ? few_waves * ATTN_WAVE_KEYS_Q8 : ATTN_FEW_KEYS;
    for (int k = 0; k < 2; ++k) {
        AttnPart& W = a.part[k];
        W = AttnPart{};
        W.max_rows = max_rows[k];
        W.max_len = max_len[k];
        for (size_t& o : P.off[k]) o = 0;
        if (n_prob[k] <= 0) continue;
        // the keys that a problem's tiles span
        int64_t reach = max_len[k];
        if (a.window > 0) reach = std::min<int64_t>(reach, (int64_t)a.window + max_rows[k] + a.n_sink + 256);
        if (a.share <= ATTN_FEW_COLS) {
            const int64_t units = ceil_div(reach, few_keys);
            const int64_t heads = (int64_t)n_prob[k] * hkv;
            // Whole (problem, head) pairs per workgroup, or equal shares of
            // all units.  A pair's chain takes 1.7 us a unit, whatever the
            // others do; shares cost the join and their own ends, some 12
            // us beyond the reads.  So pairs up to 16 units where there are
            // 8 pairs a unit, and up to 4 units always (us, whole pairs /
            // shares, lengths spread up to the longest, 8 key heads of 128):
            //     requests    640 tokens   1024         2048        4096
            //     1           12 / 14      17 / 14      27 / 16
            //     8           13 / 17      17 / 18      28 / 25
            //     16          13 / 17      18 / 25      28 / 31
            //     31          13 / 24      18 / 31      31 / 44
            //     32          13 / 25      18 / 30      30 / 42     58 / 66
            //     64          21 / 36      27 / 45      56 / 69     104 / 111
            // One request of 2048 among 31 short ones: 27 / 19; of 4096, 49 /
            // 23, which is why longer ones are shared though even lengths
            // would gain (32 of 4096: 83 / 93).  With thousands of pairs the
            // hardware's own order evens them out (512 of up to 8000: 1381 /
            // 1404), and there the shares' table would grow.
            // In 8 bits, units of 512 keys (lengths spread as above; whole / shares):
            //     requests    1024         2048        4096        8192
            //     1           13 / 16      17 / 16     26 / 17     51 / 21
            //     8           13 / 17      21 / 20     32 / 29     54 / 34
            //     16          15 / 19      21 / 28     33 / 32     56 / 47
            //     32          17 / 28      23 / 36     38 / 48     70 / 79
            //     64          29 / 38      42 / 53     74 / 82     132 / 135
            // The same rule for units of 256 keys: heads of 256 (whole / shares),
            //     requests    512       768       1024      2048      4096      8192
            //     1           16 / 19   20 / 19   23 / 19   38 / 21   63 / 26   111 / 35
            //     8           16 / 20   20 / 22   25 / 22   41 / 38   70 / 54   116 / 64
            //     16          17 / 22   22 / 35   25 / 36   41 / 56   68 / 64   120 / 94
            //     32          19 / 35   23 / 46   27 / 52   40 / 63   74 / 95   132 / 136
            //     64          34 / 53   41 / 62   48 / 67   84 / 105  137 / 147
            // and of 128 beside a prompt of 40 rows, in one launch:
            //     1           15 / 17   15 / 17   15 / 17   21 / 18   34 / 20   61 / 25
            //     8           15 / 17   15 / 18   16 / 19   24 / 29   37 / 36   63 / 42
            //     16          13 / 18   13 / 19   14 / 19   21 / 34   34 / 37   61 / 54
            //     32          26 / 30   28 / 41   31 / 42   37 / 50   52 / 64   85 / 94
            //     64          36 / 40   39 / 50   43 / 53   57 / 68   89 / 98
            auto direct = [in_8_bits](int64_t u, int64_t pairs) {
                if (in_8_bits) return u <= 3 || (u <= 16 && pairs >= 16 * u) || pairs >= 4096;
                return u <= 4 || (u <= 16 && pairs >= 8 * u) || pairs >= 4096;
            };
            W.few = direct(units, heads) ? 1 : 2;
            W.few_grid = W.few == 1 ? n_prob[k] * hkv : ATTN_FEW_WGS * 4 / few_waves;
            if (W.few == 2) a.need_join = 1;
            // (a smaller batch may have both forms in one launch, with smaller units)
            const int least = in_8_bits ? few_waves_q8(head_dim, true) * ATTN_WAVE_KEYS_Q8 : few_keys;
            if (!direct(ceil_div(max_len[k], least), hkv)) {   // of a single sequence or group
                P.off[k][0] = take((size_t)n_prob[k] * hkv * sizeof(int2));
                P.off[k][1] = take((size_t)2 * ATTN_FEW_WGS * 16 * head_dim * 4);
                P.off[k][2] = take((size_t)2 * ATTN_FEW_WGS * 16 * sizeof(float2));
            }
        }
        if ((int64_t)max_rows[k] * a.share > ATTN_FEW_COLS) {
            const int64_t nct = (int64_t)a.B.n_rows * a.share / a.tile_cols + std::min(n_prob[k], a.B.n_rows);
            int64_t tiles = ceil_div(reach, ATTN_TILE_KEYS) + 1;
            int64_t most_tiles = ceil_div(max_len[k], ATTN_TILE_KEYS) + 1;
            if (k == 0 && n_prob[1] > 0) {   // its sequences walk their prefixes too
                tiles += ceil_div(max_len[1], ATTN_TILE_KEYS) + 1;
                most_tiles += ceil_div(max_len[1], ATTN_TILE_KEYS) + 1;
            }
            // Key tiles are split among workgroups only where column tiles and
            // heads alone leave half the card or more without work; a split
            // costs its partial results, so it has at least four tiles.
            // Prefixes, whose lengths differ and which run beside other work,
            // are split to four items per workgroup slot pair (256 requests
            // behind eight prefixes of 1000 to 8000 tokens: 230 us, at 256
            // items 248).
            const int64_t items = nct * hkv, want = k == 1 ? 1024 : 256;
            const int64_t most = std::max<int64_t>(1, std::min(want / items, most_tiles / 4));
            const int64_t ns_want = std::max<int64_t>(1, std::min(most, tiles / 4));
            W.spl = (int32_t)std::min<int64_t>(ceil_div(tiles, ns_want), 1 << 30);
            const int64_t ns = ceil_div(tiles, W.spl);
            W.tile_grid = (int32_t)(items * ns);
            W.slots = ns > 1 ? 1 : 0;
            if (W.slots) a.need_join = 1;
            // Room for the partial results of any smaller batch too: it splits
            // min(want / items, most_tiles / 4) ways into at most `want` items
            // and at most most_tiles / 4 times its own, in narrow tiles where
            // this one's are.  Sequences in wide tiles are `want` items or
            // more and never split.
            if (most_tiles >= 8) {
                auto columns = [&](int tc) {
                    const int64_t most_items = ((int64_t)a.B.n_rows * a.share / tc + std::min(n_prob[k], a.B.n_rows)) * hkv;
                    return std::min(want, most_items * (most_tiles / 4)) * tc;
                };
                const size_t cols = (size_t)std::max(columns(128), k == 1 && a.tile_cols == 256 ? columns(256) : 0);
                P.off[k][3] = take((size_t)n_prob[k] * sizeof(int4));
                P.off[k][4] = take(cols * head_dim * 4);
                P.off[k][5] = take(cols * sizeof(float2));
            }
        }
    }
    if (a.join) {
        for (int k = 0; k < 2; ++k) {
            P.off[k][6] = take((size_t)a.B.n_rows * a.n_q_heads * ((size_t)head_dim * 4 + sizeof(float2)));
        }
    }
    P.bytes = at;
}

hipError_t launch_attn(const AttnArgs& a, lora_dtype_t dt, int32_t head_dim, hipStream_t stream) {
    if (dt == LORA_BF16) {
        switch (head_dim) {
            case 64: return launch_d<bf16, 64>(a, stream);
            case 128: return launch_d<bf16, 128>(a, stream);
            default: return launch_d<bf16, 256>(a, stream);
        }
    }
    return head_dim == 64 ? launch_d<float, 64>(a, stream) : launch_d<float, 128>(a, stream);
}

}  // namespace lora
