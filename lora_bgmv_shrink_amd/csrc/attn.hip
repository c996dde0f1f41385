// Attention over a paged key/value cache:
//
//     o = sum_k softmax_k(scale q . k) v,    lse = log sum_k exp(scale q . k)
//
// a row at position p seeing key k when k <= p and, with a window, when
// k > p - window or k < n_sink.
//
// Both kernels form the transposed products: S^T = K Q^T, then O^T = V^T P^T.
// The matrix cores' output layout puts one query column in each lane, so the
// running maximum and sum of the softmax are one register a lane, a column's
// scores are folded by one or two lane exchanges, and the rounded weights are
// already the operand of the second product: they never leave registers.
// (An output lane holds keys 4g .. 4g + 3 of a block, not eight neighbours;
// a product's sum may run in any order, so V is read in that same order, by
// LDS transpose reads.)  Scores, the statistics and O are fp32; the weights
// P are rounded to the cache's type for the second product, each by at most
// 2^-9 of itself in bf16, the rounding o itself gets at the end.
#include "kv_internal.hpp"

namespace lora {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;

// Operand fragments: eight elements of the summed index per lane.
//   mma16: 16 x 16 output, lane l supplies row l % 16, k = 8 (l / 16) .. + 8;
//          output element r: row 4 (l / 16) + r, column l % 16
//   mma32: 32 x 32 output, lane l supplies row l % 32, k = 8 (l / 32) .. + 8;
//          output element r: row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32
template <typename T> struct Op;
template <> struct Op<bf16> {
    using frag = bf16x8_t;
    static __device__ __forceinline__ f32x4_t mma16(const frag& a, const frag& b, f32x4_t c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16_t mma32(const frag& a, const frag& b, f32x16_t c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ frag zero() { return __builtin_bit_cast(frag, uint4{0u, 0u, 0u, 0u}); }
    static __device__ __forceinline__ frag load(const bf16* p) { return *(const frag*)p; }
    static __device__ __forceinline__ frag round(f32x8_t v) { return __builtin_convertvector(v, frag); }
    // 0 in the place of infinities and NaN; says whether there was one
    static __device__ __forceinline__ bool clean(frag& f) {
        union { frag v; bf16 e[8]; } t;
        t.v = f;
        bool any = false;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if ((t.e[e] & 0x7f80u) == 0x7f80u) {
                t.e[e] = 0;
                any = true;
            }
        f = t.v;
        return any;
    }
};
template <> struct Op<float> {
    using frag = f32x8_t;
    static __device__ __forceinline__ f32x4_t mma16(const frag& a, const frag& b, f32x4_t c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ f32x16_t mma32(const frag& a, const frag& b, f32x16_t c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ frag zero() { return frag{0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}; }
    static __device__ __forceinline__ frag load(const float* p) {
        const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
        return frag{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    }
    static __device__ __forceinline__ frag round(f32x8_t v) { return v; }
    static __device__ __forceinline__ bool clean(frag& f) {
        bool any = false;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if ((__float_as_uint(f[e]) & 0x7f800000u) == 0x7f800000u) {
                f[e] = 0.f;
                any = true;
            }
        return any;
    }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// the larger of two, the other one if one is NaN (fmaxf would first quiet
// both operands, an instruction each, for products of the matrix cores)
__device__ __forceinline__ float max_of(float a, float b) {
    return __builtin_amdgcn_fmed3f(a, b, __builtin_inff());
}
// The softmax's reference score m is not the largest score so far but one
// that no score exceeds by more than this (in log2 units): weights stay below
// 2^8, where fp32 and bf16 are as exact as below 1, and most tiles need no
// rescaling of O.
constexpr float kSlack = 8.f;

// A staged tile of keys or values: rows of D elements as they lie, 16-byte
// pieces permuted inside a row (or a pair of rows when a row is 128 bytes) so
// that the lanes of one LDS access fall in distinct banks.
template <typename T, int D>
struct Tile {
    static constexpr int RB = D * (int)sizeof(T);   // bytes of a row
    static constexpr int LPR = RB / 16;             // pieces of a row
    // keys: 16 lanes read one piece of 16 neighbouring rows
    static __device__ __forceinline__ int k_at(int key, int piece) {
        const int x = RB == 128 ? (key >> 1) & 7 : key & 15;
        return key * RB + ((piece ^ x) << 4);
    }
    // values, bf16: a transpose read takes 32 bytes of each of 4 rows per 16
    // lanes, 8 or 16 rows in all; fp32: 64 or 128 neighbouring bytes of rows 4 apart
    static __device__ __forceinline__ int v_at(int key, int piece) {
        const int x = sizeof(T) == 4 ? ((key >> 2) & 1) << 2 : RB == 128 ? ((key >> 1) & 3) << 1 : (key & 7) << 1;
        return key * RB + ((piece ^ x) << 4);
    }
    static __device__ __forceinline__ int v_elem(int key, int dim) {
        const int byte = dim * (int)sizeof(T);
        return v_at(key, byte >> 4) + (byte & 15);
    }
    // The operand holding, for one dimension per lane (this lane's row of
    // V^T), four keys from k + K0 and four from k + K1 (K0, K1 multiples of
    // 8), k = the lane's first key: v_base gives the lane's offset for k and
    // dimensions dim0 .. dim0 + 15, the rest is an immediate.  l16: lane % 16.
    static __device__ __forceinline__ int v_base(int k, int dim0, int l16) {
        if constexpr (sizeof(T) == 2) return v_elem(k + (l16 >> 2), dim0 + (l16 & 3) * 4);
        else return v_elem(k, dim0 + l16);
    }
    template <int K0, int K1>
    static __device__ __forceinline__ typename Op<T>::frag v_frag(const uint8_t* at) {
        static_assert(K0 % 8 == 0 && K1 % 8 == 0, "the permutation repeats every 8 keys");
        if constexpr (sizeof(T) == 2) {
            const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(at + K0 * RB));
            const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t*)(at + K1 * RB));
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            f32x8_t f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = *(const float*)(at + (K0 + e) * RB);
                f[e + 4] = *(const float*)(at + (K1 + e) * RB);
            }
            return f;
        }
    }
    static __device__ __forceinline__ float v_one(const uint8_t* sv, int key, int dim) {
        return to_f32(*(const T*)(sv + v_elem(key, dim)));
    }
    // eight elements of the summed index (dims d0 .. d0 + 7) of one key
    static __device__ __forceinline__ typename Op<T>::frag k_frag(const uint8_t* sk, int key, int d0) {
        const int piece = d0 * (int)sizeof(T) / 16;
        if constexpr (sizeof(T) == 2) {
            return *(const bf16x8_t*)(sk + k_at(key, piece));
        } else {
            const float4 a = *(const float4*)(sk + k_at(key, piece)), b = *(const float4*)(sk + k_at(key, piece + 1));
            return f32x8_t{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        }
    }
};

__device__ __forceinline__ bool non_finite(float v) { return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u; }

// ---------------------------------------------------------------------------
// Problems and their key tiles
// ---------------------------------------------------------------------------

struct Prob {
    int r0, nr;     // query rows
    int len;        // keys that the page table covers
    int key0;       // position of key 0
    int pos0;       // position of row r0 (kind 1: the least position any row can have)
    int pos1;       // position of the last row (kind 1: the largest)
    const int32_t* tbl;
};

// number of i in 1 .. n with off[i] <= key (one thread)
__device__ inline int find_run(const int32_t* __restrict__ off, int n, int key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (off[m] <= key) lo = m;
        else hi = m - 1;
    }
    return lo;
}

__device__ __forceinline__ int table_keys(int len, int64_t ld, int shift) {
    return (int)max((int64_t)0, min((int64_t)len, min(ld << shift, (int64_t)0x7fffff00)));
}

__device__ inline Prob load_prob(const AttnArgs& a, int kind, int p) {
    const KvBatchDev& B = a.B;
    Prob P;
    int r0, r1;
    if (kind == 0) {
        r0 = B.row_off[p];
        r1 = B.row_off[p + 1];
    } else {
        const int s0 = min(max(B.group_off[p], 0), B.n_seqs), s1 = min(max(B.group_off[p + 1], s0), B.n_seqs);
        r0 = B.row_off[s0];
        r1 = B.row_off[s1];
    }
    P.r0 = min(max(r0, 0), B.n_rows);
    const int nr = min(max(r1, P.r0), B.n_rows) - P.r0;
    P.nr = min(nr, a.part[kind].max_rows);
    P.key0 = 0;
    if (kind == 0) {
        const int n = max(B.kv_len[p], 0);
        if (B.n_groups) {
            const int g = find_run(B.group_off, B.n_groups, p);
            if (g < B.n_groups) P.key0 = max(B.prefix_len[g], 0);
        }
        P.len = table_keys(min(n, a.part[0].max_len), B.ldp, a.C.page_shift);
        P.pos0 = P.key0 + n - nr;
        P.pos1 = P.pos0 + P.nr - 1;
        P.tbl = B.pages + (int64_t)p * B.ldp;
    } else {
        const int n = max(B.prefix_len[p], 0);
        P.len = table_keys(min(n, a.part[1].max_len), B.ldpp, a.C.page_shift);
        P.pos0 = n;
        P.pos1 = 0x7ffffffe;
        P.tbl = B.prefix_pages + (int64_t)p * B.ldpp;
    }
    return P;
}
__device__ __forceinline__ int problems(const AttnArgs& a, int kind) { return kind == 0 ? a.B.n_seqs : a.B.n_groups; }
__device__ __forceinline__ bool is_few(const AttnArgs& a, const Prob& P) {
    return (int64_t)P.nr * a.share <= ATTN_FEW_COLS;
}

// Tiles of KB keys that rows at positions p_lo .. p_hi see some key of: tiles
// 0 .. ns - 1 hold the first tokens, tiles `first` on the window.
struct Range {
    int ns, first, n;
    __device__ __forceinline__ int tile(int i) const { return i < ns ? i : first + i - ns; }
};
template <int KB>
__device__ __forceinline__ Range key_tiles(const AttnArgs& a, const Prob& P, int p_lo, int p_hi) {
    Range R{0, 0, 0};
    const int e = min(P.len, p_hi - P.key0 + 1);
    if (e <= 0) return R;
    const int te = (e + KB - 1) / KB;
    if (a.window > 0) {
        const int lo = p_lo - a.window + 1 - P.key0;
        if (lo > 0) R.first = min(lo / KB, te);
        const int sk = min(e, a.n_sink - P.key0);
        if (sk > 0) R.ns = min((sk + KB - 1) / KB, R.first);
    }
    R.n = R.ns + te - R.first;
    return R;
}

// Position of query row `row` (kind 1 rows lie in several sequences); -1 for none.
__device__ inline int row_position(const AttnArgs& a, int row) {
    const KvBatchDev& B = a.B;
    const int s = find_run(B.row_off, B.n_seqs, row);
    if (s >= B.n_seqs) return -1;
    int before = 0;
    if (B.n_groups) {
        const int g = find_run(B.group_off, B.n_groups, s);
        if (g < B.n_groups) before = max(B.prefix_len[g], 0);
    }
    return before + max(B.kv_len[s], 0) - (B.row_off[s + 1] - row);
}

// Inclusive scan over 256 threads; *total: their sum.  sh: 4 ints.
__device__ inline int block_scan(int v, int tid, int* sh, int* total) {
    int x = wave_incl_scan(v, tid & 63);
    __syncthreads();
    if ((tid & 63) == 63) sh[tid >> 6] = x;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < (tid >> 6)) x += sh[w];
        sum += sh[w];
    }
    *total = sum;
    return x;
}

// The problem that work unit u lies in, units numbered problem by problem
// (units(p) each): its number, the unit's place in it and the units before
// it.  All 256 threads; false past the last unit.
template <class F>
__device__ inline bool locate(int n, int u, F units, int tid, int* sh, int& p_out, int& base_out) {
    int before = 0;
    for (int p0 = 0; p0 < n; p0 += 256) {
        const int v = p0 + tid < n ? units(p0 + tid) : 0;
        int total;
        const int incl = before + block_scan(v, tid, sh, &total);
        if (u < before + total) {
            if (u < incl && u >= incl - v) {
                sh[4] = p0 + tid;
                sh[5] = incl - v;
            }
            __syncthreads();
            p_out = __builtin_amdgcn_readfirstlane(sh[4]);
            base_out = __builtin_amdgcn_readfirstlane(sh[5]);
            return true;
        }
        before += total;
    }
    return false;
}
template <class F>
__device__ inline int64_t sum_units(int n, F units, int tid, int* sh) {
    int64_t all = 0;
    for (int p0 = 0; p0 < n; p0 += 256) {
        int total;
        block_scan(p0 + tid < n ? units(p0 + tid) : 0, tid, sh, &total);
        all += total;
    }
    return all;
}

// unnormalised o of one (row, head), elements d .. d + N - 1, to its output
template <int N>
__device__ __forceinline__ void put_out(const AttnArgs& a, int row, int head, int D, int d, const float (&v)[N], float l) {
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // nothing seen: 0; NaN stays
    const int64_t at = (int64_t)row * a.ldo + (int64_t)head * D + d;
    if (a.o_bf16) {
        union { bf16 e[N]; uint2 u2[(N + 3) / 4]; uint32_t u1; } t;
#pragma unroll
        for (int i = 0; i < N; ++i) t.e[i] = f32_to_bf16(v[i] * inv);
        bf16* o = (bf16*)a.o + at;
        if constexpr (N >= 4) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) ((uint2*)o)[i] = t.u2[i];
        } else if constexpr (N == 2) {
            *(uint32_t*)o = t.u1;
        } else {
            static_assert(N == 1, "element counts a lane can own");
            *o = t.e[0];
        }
    } else {
        float* o = (float*)a.o + at;
        if constexpr (N >= 4) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                *(float4*)(o + i) = float4{v[i] * inv, v[i + 1] * inv, v[i + 2] * inv, v[i + 3] * inv};
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = v[i] * inv;
        }
    }
}
template <int N>
__device__ __forceinline__ void put_raw(float* o, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *(float4*)(o + i) = float4{v[i], v[i + 1], v[i + 2], v[i + 3]};
}
// log of the sum of exponentials, from the largest raw score and the sum
__device__ __forceinline__ float lse_of(const AttnArgs& a, float m, float l) {
    return l == 0.f ? -__builtin_inff() : m * a.scale + logf(l);
}

// ---------------------------------------------------------------------------
// Requests of keys and values
// ---------------------------------------------------------------------------

// 16 bytes; ONCE: no other workgroup reads them, so they pass the caches by
// (a read stream of this shape reaches 6.5 TB/s so, and 5.9 through L2)
template <bool ONCE>
__device__ __forceinline__ u32x4_t piece_at(const void* p) {
    if constexpr (ONCE) return __builtin_nontemporal_load((const u32x4_t*)p);
    return *(const u32x4_t*)p;
}

// Where the wave-wide loads of N x `rows` neighbouring keys start: page number
// `id` holds that of key `lane` of the tile (page 0 in the place of none).
// PAGED: a load's rows lie in one page (page_size >= the rows of a load), so
// its base is scalar; otherwise every lane follows its own key's page.
template <typename T, int D, int NL, int STEP, bool PAGED, bool ONCE>
__device__ __forceinline__ void request(const AttnArgs& a, int id, int base, int row0, int h, int lane, u32x4_t (&rk)[NL],
                                        u32x4_t (&rv)[NL]) {
    using TL = Tile<T, D>;
    const int mask = (1 << a.C.page_shift) - 1;
    const int r = lane / TL::LPR, piece = (lane % TL::LPR) * (16 / (int)sizeof(T));
    const int64_t hs = (int64_t)h * a.C.head_stride;
    if constexpr (PAGED) {
        const uint32_t lo = (uint32_t)(r * (int)a.C.token_stride + piece);
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = row0 + j * STEP;   // uniform
            const int64_t page = __builtin_amdgcn_readlane(id, row);
            const int64_t off = page * a.C.page_stride + (int64_t)(((base + row) & mask) * (int)a.C.token_stride) + hs;
            rk[j] = piece_at<ONCE>((const T*)a.C.k + off + lo);
            rv[j] = piece_at<ONCE>((const T*)a.C.v + off + lo);
        }
    } else {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = row0 + j * STEP + r;
            const int64_t off = (int64_t)__shfl(id, row, 64) * a.C.page_stride +
                                (int64_t)((base + row) & mask) * a.C.token_stride + hs + piece;
            rk[j] = piece_at<ONCE>((const T*)a.C.k + off);
            rv[j] = piece_at<ONCE>((const T*)a.C.v + off);
        }
    }
}
template <int NL>
__device__ __forceinline__ void hide_rows(u32x4_t (&rv)[NL], uint64_t bits, int row0, int step) {
#pragma unroll
    for (int j = 0; j < NL; ++j)
        if (!((bits >> (row0 + j * step)) & 1)) rv[j] = u32x4_t{0u, 0u, 0u, 0u};
}
template <typename T>
__device__ __forceinline__ bool odd_piece(const u32x4_t& v) {
    if constexpr (sizeof(T) == 4) {
        auto bad = [](uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u; };
        return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
    } else {
        auto bad = [](uint32_t w) { return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u; };
        return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
    }
}

// Whether a lane's column sees key k of a tile: `see` and `from` are the last
// and first such k by position (first tokens: k < sink), bit k of `bits` is
// set for keys that exist.
struct Sees {
    int see, from, sink;
    __device__ __forceinline__ Sees(const AttnArgs& a, int col_pos, int lo) {
        see = col_pos - lo;
        from = a.window > 0 ? see - a.window + 1 : -0x7fffffff;
        sink = a.window > 0 ? a.n_sink - lo : 0;
    }
    // (no branches: one test after the other would make a jump of each)
    __device__ __forceinline__ bool at(int k) const { return (k <= see) & ((k >= from) | (k < sink)); }
};

// ---------------------------------------------------------------------------
// Few query columns (decode): the keys are split
// ---------------------------------------------------------------------------

// Up to 16 columns (query heads of one key head, times the sequence's rows).
// Reading the visible keys and values bounds it: 4 * 16 columns * D flop per
// 4 D bytes of bf16 keep the matrix cores below a quarter of their rate.
//
// A work unit is 128 keys of one (problem, key head); each of the four waves
// takes 32 of them through LDS of its own (no barrier), with the next unit's
// pieces in flight in registers and the unit after's page numbers before
// them.  Shared form (few = 2): the units of all problems are dealt to the
// workgroups in equal runs, whatever the lengths; a run's first and last
// (problem, head) may be partial and go to slots that the join adds.
// Otherwise a workgroup takes one (problem, head) whole.
template <typename T, int D, bool PAGED>
__device__ __forceinline__ void attn_few(const AttnArgs& a, int kind, int block, int blocks, uint8_t* stage, int* sh) {
    using TL = Tile<T, D>;
    using O = Op<T>;
    constexpr int KW = ATTN_FEW_KEYS / 4;            // keys of a wave's unit
    constexpr int NL = KW * TL::LPR / 64;            // pieces per lane, of K and of V
    constexpr int RPL = 64 / TL::LPR;                // rows one load covers
    constexpr int WB = 2 * KW * TL::RB;              // LDS bytes of a wave
    constexpr int OP = D + 4;                        // fp32 pitch of a wave's O at the end
    static_assert(16 * OP * 4 + 128 <= WB, "O and its statistics fit the wave's stage");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int hkv = a.C.n_kv_heads;
    const AttnPart& W = a.part[kind];
    const bool shared = W.few == 2;
    const int n_prob = problems(a, kind);
    uint8_t* sk = stage + wave * WB;
    uint8_t* sv = sk + KW * TL::RB;
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    const float slack = kSlack / c;
    int vb[D / 16];   // this lane's place in the stage of values, per 16 dimensions
#pragma unroll
    for (int t = 0; t < D / 16; ++t) vb[t] = TL::v_base(4 * g4, t * 16, l16);

    auto range_of = [&](const Prob& P) __attribute__((always_inline)) {
        if (P.nr == 0 || !is_few(a, P)) return Range{0, 0, 0};
        return key_tiles<ATTN_FEW_KEYS>(a, P, P.pos0, P.pos1);
    };

    int p, h, i;    // the piece worked on: problem, key head, first unit of it
    Prob P;
    Range R;
    int u = 0, u1;  // this workgroup's units [u, u1)
    int64_t total = 0, wgs = 1;   // all units, and the workgroups that have some
    if (shared) {
        auto units = [&](int q) { return range_of(load_prob(a, kind, q)).n * hkv; };
        total = sum_units(n_prob, units, tid, sh);
        wgs = min((int64_t)blocks, total);   // no run between a first and a last one is empty
        if (block >= wgs) return;
        u = (int)(block * total / wgs);
        u1 = (int)((block + 1) * total / wgs);
        int base = 0;
        if (!locate(n_prob, u, units, tid, sh, p, base)) return;
        P = load_prob(a, kind, p);
        R = range_of(P);
        h = (u - base) / R.n;
        i = u - base - h * R.n;
    } else {
        p = block / hkv;
        h = block - p * hkv;
        i = 0;
        P = load_prob(a, kind, p);
        if (P.nr == 0 || !is_few(a, P)) return;   // no rows, or the tiled form's
        R = range_of(P);
        u1 = R.n;
    }

    const int first = u;
    while (true) {
        const int n = min(R.n - i, u1 - u);   // units of this piece (0: rows that see no key)
        // m, l of this lane's column (l: this lane's keys only, until the end)
        float m = -kInf, l = 0.f;
        f32x4_t acc[D / 16];
#pragma unroll
        for (int t = 0; t < D / 16; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        typename O::frag qf[D / 32];
        int col_pos = -1;   // position of this lane's column, -1: no column
        {
            const int j = l16 / a.share;
            const bool there = l16 < P.nr * a.share;
            const T* q = (const T*)a.q + (int64_t)(P.r0 + j) * a.ldq + (int64_t)(h * a.share + l16 - j * a.share) * D;
#pragma unroll
            for (int s = 0; s < D / 32; ++s) qf[s] = there ? O::load(q + s * 32 + g4 * 8) : O::zero();
            if (there) col_pos = kind == 0 ? P.pos0 + j : a.window > 0 ? row_position(a, P.r0 + j) : P.pos1;
        }

        // page number of key `lane` of the wave's unit x (lanes 0 .. 31), -1: none
        auto load_id = [&](int x) __attribute__((always_inline)) {
            const int key = R.tile(x) * ATTN_FEW_KEYS + wave * KW + lane;
            return lane < KW && key < P.len ? P.tbl[key >> a.C.page_shift] : -1;
        };
        u32x4_t rk[NL], rv[NL];
        // requests the wave's pieces of unit x; the answer's bit k says whether
        // any column sees key k (the others are read from page 0 and not used)
        auto load_kv = [&](int x, int id) __attribute__((always_inline)) {
            const int base = R.tile(x) * ATTN_FEW_KEYS + wave * KW;
            const int key = base + lane, at = P.key0 + key;
            const bool page_ok = id >= 0 && id < a.C.n_pages;
            bool seen = lane < KW && key < P.len && at <= P.pos1;
            if (a.window > 0) seen = seen && (at > P.pos0 - a.window || at < a.n_sink);
            if (seen && !page_ok && a.status) flag_bad_id(a.status);
            request<T, D, NL, RPL, PAGED, true>(a, page_ok ? id : 0, base, 0, h, lane, rk, rv);
            return (uint32_t)__ballot(seen && page_ok);
        };
        auto compute = [&](int x, uint32_t bits, bool all_see, bool odd) __attribute__((always_inline)) {
            f32x4_t s[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                s[0] = O::mma16(TL::k_frag(sk, l16, ks * 32 + g4 * 8), qf[ks], s[0]);
                s[1] = O::mma16(TL::k_frag(sk, 16 + l16, ks * 32 + g4 * 8), qf[ks], s[1]);
            }
            // element r of s[t]: key 16 t + 4 g4 + r, this lane's column
            const int lo = P.key0 + R.tile(x) * ATTN_FEW_KEYS + wave * KW;
            if (!all_see) {
                asm volatile("");   // a branch: most tiles need no mask
                const Sees S(a, col_pos, lo + 4 * g4);
                const uint32_t mine = bits >> (4 * g4);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s[t][r] = S.at(16 * t + r) & ((mine >> (16 * t + r)) & 1u) ? s[t][r] : -kInf;
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
            const float mc = m == -kInf ? 0.f : m * c;
            f32x8_t w;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[r] = exp2_fast(s[0][r] * c - mc);
                w[4 + r] = exp2_fast(s[1][r] * c - mc);
            }
            l += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
            const typename O::frag pf = O::round(w);
            if (!odd) {
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
                    acc[t] = O::mma16(TL::template v_frag<0, 16>(sv + vb[t]), pf, acc[t]);
                return;
            }
            asm volatile("");
            // Infinities or NaN among values that some rows do not see: they
            // are left out of the product (0 times them is NaN) and added to
            // the columns that see them.
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
                typename O::frag vf = TL::template v_frag<0, 16>(sv + vb[t]);
                O::clean(vf);
                acc[t] = O::mma16(vf, pf, acc[t]);
                __builtin_amdgcn_sched_barrier(0);
            }
            const Sees S(a, col_pos, lo);
            for (int k = 0; k < KW; ++k) {
                const int r = (k & 3) + 4 * (k >> 4);
                float wk = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e == r) wk = w[e];
                wk = __shfl(wk, ((k >> 2) & 3) * 16 + l16, 64);
                if (!S.at(k) || !((bits >> k) & 1)) continue;
#pragma unroll
                for (int t = 0; t < D / 16; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = TL::v_one(sv, k, t * 16 + g4 * 4 + e);
                        if (non_finite(y)) acc[t][e] += wk * y;
                    }
            }
        };

        if (n > 0) {
            uint32_t bits = load_kv(i, load_id(i));
            int id = n > 1 ? load_id(i + 1) : -1;
            for (int x = i; x < i + n; ++x) {
                const int lo = P.key0 + R.tile(x) * ATTN_FEW_KEYS + wave * KW;
                const bool all_see = bits == 0xffffffffu && lo + KW - 1 <= P.pos0 &&
                                     (a.window == 0 || lo > P.pos1 - a.window);
                bool odd = false;
                if (bits != 0xffffffffu) hide_rows<NL>(rv, bits, lane / TL::LPR, RPL);
                if (!all_see && P.nr > 1) {
#pragma unroll
                    for (int j = 0; j < NL; ++j) odd |= odd_piece<T>(rv[j]);
                    odd = __ballot(odd) != 0;
                }
#pragma unroll
                for (int j = 0; j < NL; ++j) {
                    const int row = j * RPL + lane / TL::LPR, piece = lane % TL::LPR;
                    *(u32x4_t*)(sk + TL::k_at(row, piece)) = rk[j];
                    *(u32x4_t*)(sv + TL::v_at(row, piece)) = rv[j];
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                const uint32_t bits_x = bits;
                if (x + 1 < i + n) {
                    const int id_x = id;
                    if (x + 2 < i + n) id = load_id(x + 2);
                    bits = load_kv(x + 1, id_x);
                }
                if (bits_x) compute(x, bits_x, all_see, odd);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
        }

        // joins the four waves' results and writes them
        bool whole = true;
        int slot = 0;
        if (shared) {
            const int ra = u - i, rb = ra + R.n;   // the units of (p, h)
            const bool starts = ra >= first;
            whole = starts && rb <= u1;
            slot = 2 * block + (starts ? 1 : 0);
            if (starts && tid == 0) W.rec[p * hkv + h] = int2{block, (int)((rb * wgs - 1) / total)};
        }
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        float* so = (float*)sk;
        float* stat = so + 16 * OP;   // 16 largest scores, 16 sums
        if (lane < 16) {
            stat[lane] = m;
            stat[16 + lane] = l;
        }
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
            *(float4*)(so + l16 * OP + t * 16 + g4 * 4) = float4{acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
        __syncthreads();
        {
            constexpr int N = D / 16;   // elements per thread, of column tid / 16
            constexpr int WF = WB / 4;  // floats of a wave's stage
            const int col = tid >> 4, d = (tid & 15) * N;
            const float* all = (const float*)stage;
            float mw[4], M = -kInf, sum = 0.f, v[N];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                mw[w] = all[w * WF + 16 * OP + col];
                M = fmaxf(M, mw[w]);
            }
            const float Mc = M == -kInf ? 0.f : M * c;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                mw[w] = exp2_fast(mw[w] * c - Mc);
                sum += mw[w] * all[w * WF + 16 * OP + 16 + col];
            }
#pragma unroll
            for (int e = 0; e < N; e += 4) {
                float4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float4 y = *(const float4*)(all + w * WF + col * OP + d + e);
                    x.x += mw[w] * y.x;
                    x.y += mw[w] * y.y;
                    x.z += mw[w] * y.z;
                    x.w += mw[w] * y.w;
                }
                v[e] = x.x;
                v[e + 1] = x.y;
                v[e + 2] = x.z;
                v[e + 3] = x.w;
            }
            if (!whole) {
                put_raw<N>(W.few_o + ((int64_t)slot * 16 + col) * D + d, v);
                if ((tid & 15) == 0) W.few_ml[slot * 16 + col] = float2{M, sum};
            } else if (col < P.nr * a.share) {
                const int j = col / a.share;
                const int row = P.r0 + j, head = h * a.share + (col - j * a.share);
                const int64_t rh = (int64_t)row * a.n_q_heads + head;
                if (a.join) {
                    put_raw<N>(W.row_o + rh * D + d, v);
                    if ((tid & 15) == 0) W.row_ml[rh] = float2{M, sum};
                } else {
                    put_out<N>(a, row, head, D, d, v, sum);
                    if (a.lse && (tid & 15) == 0) a.lse[rh] = lse_of(a, M, sum);
                }
            }
        }
        u += n;
        if (u >= u1) break;
        __syncthreads();
        i = 0;
        if (++h == hkv) {
            h = 0;
            do {   // in bounds: units remain
                P = load_prob(a, kind, ++p);
                R = range_of(P);
            } while (R.n == 0 && p + 1 < n_prob);
        }
    }
}

// ---------------------------------------------------------------------------
// Many query columns (prompts, shared prefixes): the columns are split
// ---------------------------------------------------------------------------

// A workgroup owns 128 columns of one key head, 32 a wave, and walks tiles of
// 64 keys staged in LDS, two buffers, the next tile's pieces in flight in
// registers meanwhile: one barrier a tile.  Each staged byte feeds 128
// columns, 4 D flop per key and column, so the matrix cores bound it.  Items
// (problem, column tile, key head, run of key tiles) are numbered with the
// key head fastest, so that the columns of one head meet in one XCD's L2, and
// later column tiles (more keys under the causal mask) first.
template <typename T, int D, bool PAGED>
__device__ __forceinline__ void attn_tile(const AttnArgs& a, int kind, int block, uint8_t* stage, int* sh) {
    using TL = Tile<T, D>;
    using O = Op<T>;
    constexpr int KB = ATTN_TILE_KEYS, TC = ATTN_TILE_COLS;
    constexpr int NL = KB * TL::LPR / 256;     // pieces per thread, of K and of V
    constexpr int RPL = 256 / TL::LPR;         // rows one load of the workgroup covers
    constexpr int TB = KB * TL::RB;            // bytes of a staged tile
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, h2 = lane >> 5, l16 = lane & 15, d16 = (lane >> 4) & 1;
    const int hkv = a.C.n_kv_heads;
    const AttnPart& W = a.part[kind];
    const int n_prob = problems(a, kind);
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    const float slack = kSlack / c;
    int vb[D / 32];   // this lane's place in the stage of values, per 32 dimensions
#pragma unroll
    for (int t = 0; t < D / 32; ++t) vb[t] = TL::v_base(4 * h2, t * 32 + d16 * 16, l16);

    auto splits_of = [&](const Prob& Q, int& nct) __attribute__((always_inline)) {
        const int64_t cols = (int64_t)Q.nr * a.share;
        nct = cols > ATTN_FEW_COLS ? (int)((cols + TC - 1) / TC) : 0;
        const int n = key_tiles<KB>(a, Q, Q.pos0, Q.pos1).n;
        return n > W.spl ? (n + W.spl - 1) / W.spl : 1;
    };
    int p, base;
    if (!locate(n_prob, block,
                [&](int q) {
                    int nct;
                    const int ns = splits_of(load_prob(a, kind, q), nct);
                    return nct * ns * hkv;
                },
                tid, sh, p, base))
        return;
    const Prob P = load_prob(a, kind, p);
    int nct;
    const int nsplit = splits_of(P, nct);
    int rem = block - base;
    const int h = rem % hkv;
    rem /= hkv;
    const int split = rem / nct;
    const int ct = nct - 1 - rem % nct;
    if (rem == 0 && h == 0 && tid == 0 && W.slots) W.item[p] = int4{base, nct, nsplit, 0};

    // the workgroup's rows, its key tiles and this split's run of them
    const int j_lo = ct * TC / a.share, j_hi = min(P.nr - 1, (ct * TC + TC - 1) / a.share);
    const int wg_lo = kind == 0 ? P.pos0 + j_lo : P.pos0, wg_hi = kind == 0 ? P.pos0 + j_hi : P.pos1;
    const Range R = key_tiles<KB>(a, P, wg_lo, wg_hi);
    const int i0 = split * W.spl, i1 = min(R.n, i0 + W.spl);
    if (split > 0 && i0 >= R.n) return;

    // this lane's column
    const int64_t n_cols = (int64_t)P.nr * a.share;
    const int col = ct * TC + wave * 32 + l32;
    const bool there = col < n_cols;
    const int j = there ? col / a.share : 0;
    const int row = P.r0 + j, head = h * a.share + (there ? col - j * a.share : 0);
    const bool wave_there = ct * TC + wave * 32 < n_cols;
    int col_pos = -1;
    if (there) col_pos = kind == 0 ? P.pos0 + j : a.window > 0 ? row_position(a, row) : P.pos1;
    // least and largest position of the wave's columns
    const int wv_lo = kind == 0 ? P.pos0 + (ct * TC + wave * 32) / a.share : P.pos0;
    const int wv_hi = kind == 0 ? min(P.pos1, P.pos0 + (ct * TC + wave * 32 + 31) / a.share) : P.pos1;

    typename O::frag qf[D / 16];
    {
        const T* q = (const T*)a.q + (int64_t)row * a.ldq + (int64_t)head * D;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = there ? O::load(q + s * 16 + h2 * 8) : O::zero();
    }
    float m = -kInf, l = 0.f;
    f32x16_t acc[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;

    // page number of key `lane` of tile i, -1: none
    auto load_id = [&](int i) __attribute__((always_inline)) {
        const int key = R.tile(i) * KB + lane;
        return key < P.len ? P.tbl[key >> a.C.page_shift] : -1;
    };
    u32x4_t rk[NL], rv[NL];
    auto load_kv = [&](int i, int id) __attribute__((always_inline)) {
        const int base_k = R.tile(i) * KB;
        const int key = base_k + lane, at = P.key0 + key;
        const bool page_ok = id >= 0 && id < a.C.n_pages;
        bool seen = key < P.len && at <= wg_hi;
        if (a.window > 0) seen = seen && (at > wg_lo - a.window || at < a.n_sink);
        if (seen && !page_ok && a.status) flag_bad_id(a.status);
        request<T, D, NL, RPL, PAGED, false>(a, page_ok ? id : 0, base_k, wave * (64 / TL::LPR), h, lane, rk, rv);
        return (uint64_t)__ballot(seen && page_ok);
    };
    // sh[6 + buffer]: some value of a tile that columns see in part is not finite
    if (tid == 0) sh[6] = sh[7] = 0;

    uint64_t bits = 0;
    int id = -1;
    if (i0 < i1) {
        bits = load_kv(i0, load_id(i0));
        if (i0 + 1 < i1) id = load_id(i0 + 1);
    }
    __syncthreads();
    for (int i = i0; i < i1; ++i) {
        const int buf = (i - i0) & 1;
        uint8_t* sk = stage + buf * 2 * TB;
        uint8_t* sv = sk + TB;
        const int lo = P.key0 + R.tile(i) * KB;
        const int r0 = tid / TL::LPR, piece = tid % TL::LPR;
        if (bits != ~0ull) hide_rows<NL>(rv, bits, r0, RPL);
        const bool wg_all = bits == ~0ull && lo + KB - 1 <= wg_lo && (a.window == 0 || lo > wg_hi - a.window);
        if (!wg_all) {
            bool odd = false;
#pragma unroll
            for (int n = 0; n < NL; ++n) odd |= odd_piece<T>(rv[n]);
            if (__ballot(odd) && lane == 0) sh[6 + buf] = 1;
        }
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            *(u32x4_t*)(sk + TL::k_at(n * RPL + r0, piece)) = rk[n];
            *(u32x4_t*)(sv + TL::v_at(n * RPL + r0, piece)) = rv[n];
        }
        __syncthreads();
        const uint64_t bits_i = bits;
        if (i + 1 < i1) {
            const int id_i = id;
            if (i + 2 < i1) id = load_id(i + 2);
            bits = load_kv(i + 1, id_i);
        }
        if (!wave_there || lo > wv_hi) continue;
        const bool all_see = bits_i == ~0ull && lo + KB - 1 <= wv_lo && (a.window == 0 || lo > wv_hi - a.window);
        const bool odd = !wg_all && *(volatile int*)(sh + 6 + buf) != 0;
        // element r of s[kb]: key 32 kb + 8 (r / 4) + 4 h2 + r % 4
        f32x16_t s[2];
#pragma unroll
        for (int r = 0; r < 16; ++r) s[0][r] = s[1][r] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            s[0] = O::mma32(TL::k_frag(sk, l32, ks * 16 + h2 * 8), qf[ks], s[0]);
            s[1] = O::mma32(TL::k_frag(sk + 32 * TL::RB, l32, ks * 16 + h2 * 8), qf[ks], s[1]);
        }
        if constexpr (sizeof(T) == 2) {
            // K's operands are requested four products ahead of their use
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int n = 0; n < D / 16 - 2; ++n) {
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
        }
        if (!all_see) {
            asm volatile("");   // a branch: most tiles need no mask
            const Sees S(a, col_pos, lo + 4 * h2);
            const uint64_t mine = bits_i >> (4 * h2);
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int k = 32 * kb + 8 * (r >> 2) + (r & 3);
                    s[kb][r] = S.at(k) & ((uint32_t)(mine >> k) & 1u) ? s[kb][r] : -kInf;
                }
        }
        float top = max_of(s[0][0], s[1][0]);
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, max_of(s[0][r], s[1][r]));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        if (__ballot(top > m + slack)) {
            const bool up = top > m + slack;   // a column's own matter: its neighbours do not change its bits
            const float f = up ? exp2_fast((m - top) * c) : 1.f;   // from -infinity: 0
            l *= f;
#pragma unroll
            for (int t = 0; t < D / 32; ++t) acc[t] *= f;
            if (up) m = top;
        }
        const float mc = m == -kInf ? 0.f : m * c;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                s[kb][r] = exp2_fast(s[kb][r] * c - mc);
                part[r & 3] += s[kb][r];
            }
        l += (part[0] + part[1]) + (part[2] + part[3]);
        typename O::frag pf[2][2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x8_t x;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s[kb][8 * t + e];
                pf[kb][t] = O::round(x);
            }
        // the four 16-key steps of the second product
        auto each_step = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<0, 8>(sv + vb[t]), pf[0][0], t);
#pragma unroll
            for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<16, 24>(sv + vb[t]), pf[0][1], t);
#pragma unroll
            for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<32, 40>(sv + vb[t]), pf[1][0], t);
#pragma unroll
            for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<48, 56>(sv + vb[t]), pf[1][1], t);
        };
        if (!odd) {
            each_step([&](const typename O::frag& vf, const typename O::frag& w, int t)
                          __attribute__((always_inline)) { acc[t] = O::mma32(vf, w, acc[t]); });
            if constexpr (sizeof(T) == 2) {
                // V's operands are requested four products ahead of their use
                constexpr int NM = 4 * (D / 32);
                __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
#pragma unroll
                for (int n = 0; n < NM - 4; ++n) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                }
                __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);
            }
            continue;
        }
        asm volatile("");
        // Infinities or NaN among values that some columns do not see: they
        // are left out of the product (0 times them is NaN) and added to the
        // columns that see them.
        each_step([&](typename O::frag vf, const typename O::frag& w, int t) __attribute__((always_inline)) {
            O::clean(vf);
            acc[t] = O::mma32(vf, w, acc[t]);
            __builtin_amdgcn_sched_barrier(0);
        });
        const Sees S(a, col_pos, lo);
        for (int k = 0; k < KB; ++k) {
            const int e = ((k >> 3) & 3) * 4 + (k & 3);
            float w = 0.f;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (r == e) w = k < 32 ? s[0][r] : s[1][r];
            w = __shfl(w, ((k >> 2) & 1) * 32 + l32, 64);
            if (!S.at(k) || !((bits_i >> k) & 1)) continue;
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float x = TL::v_one(sv, k, t * 32 + 8 * (r >> 2) + 4 * h2 + (r & 3));
                    if (non_finite(x)) acc[t][r] += w * x;
                }
        }
    }

    l += __shfl_xor(l, 32, 64);
    if (!there) return;
    const bool whole = nsplit == 1;
    const int64_t rh = (int64_t)row * a.n_q_heads + head;
    const int64_t sc = (int64_t)block * TC + wave * 32 + l32;
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float v[4] = {acc[t][4 * x], acc[t][4 * x + 1], acc[t][4 * x + 2], acc[t][4 * x + 3]};
            const int d = t * 32 + x * 8 + h2 * 4;
            if (!whole) put_raw<4>(W.tile_o + sc * D + d, v);
            else if (a.join) put_raw<4>(W.row_o + rh * D + d, v);
            else put_out<4>(a, row, head, D, d, v, l);
        }
    if (h2 == 0) {
        if (!whole) W.tile_ml[sc] = float2{m, l};
        else if (a.join) W.row_ml[rh] = float2{m, l};
        else if (a.lse) a.lse[rh] = lse_of(a, m, l);
    }
}

// Both forms, over own tokens and shared prefixes, in one launch: a
// workgroup's number says which.  Tiled items come first (the longest ones);
// the few-column workgroups, bound by memory, run beside and after them.
template <typename T, int D, bool PAGED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(sizeof(T) * D <= 256 ? 2 : 1)))
void k_attn(AttnArgs a) {
    // a staged tile pair, twice: two buffers of 64 keys, or four waves' 32 keys
    __shared__ __attribute__((aligned(16))) uint8_t stage[4 * ATTN_TILE_KEYS * Tile<T, D>::RB];
    __shared__ int sh[8];
    int b = blockIdx.x;
#pragma unroll 1
    for (int kind = 1; kind >= 0; --kind) {
        if (b < a.part[kind].tile_grid) {
            attn_tile<T, D, PAGED>(a, kind, b, stage, sh);
            return;
        }
        b -= a.part[kind].tile_grid;
    }
#pragma unroll 1
    for (int kind = 1; kind >= 0; --kind) {
        const int n = a.part[kind].few_grid;
        if (b < n) {
            attn_few<T, D, PAGED>(a, kind, b, n, stage, sh);
            return;
        }
        b -= n;
    }
}

// ---------------------------------------------------------------------------
// Join
// ---------------------------------------------------------------------------

// Adds the partial results of a row's own keys and of its shared prefix, each
// scaled to the largest reference score, in their fixed order.  A wave takes
// one row and four query heads, 16 lanes each (the row's lookups, a chain of
// dependent loads, are most of a small join's time and are shared by the
// four); every partial result is read once.
//
// by_row: all rows (a shared prefix, or split tiled items).  Otherwise only
// rows of few-column sequences can have partial results, and the waves are
// numbered by (sequence, row in it) so that a prompt's rows cost nothing.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a, int by_row, int rows_of_few) {
    constexpr int N = D / 16;   // elements per lane
    const int lane = threadIdx.x & 63, sub = lane >> 4, sl = lane & 15;
    const KvBatchDev& B = a.B;
    const int blocks = (a.n_q_heads + 3) / 4;   // of four heads
    const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t at_row = unit / blocks;
    const int head = (int)(unit - at_row * blocks) * 4 + sub;
    int s, row;
    if (by_row) {
        if (at_row >= B.n_rows) return;
        row = (int)at_row;
        s = wave_find_run(B.row_off, B.n_seqs, row, lane);
        if (s >= B.n_seqs) return;
    } else {
        s = (int)(at_row / rows_of_few);
        if (s >= B.n_seqs) return;
        row = -1;
    }
    const Prob P = load_prob(a, 0, s);
    const int j = by_row ? row - P.r0 : (int)(at_row - (int64_t)s * rows_of_few);
    if (j < 0 || j >= P.nr) return;
    row = P.r0 + j;
    const bool few = is_few(a, P);
    const bool mine = head < a.n_q_heads;
    const int hd = mine ? head : a.n_q_heads - 1;
    const int h = hd / a.share, hkv = a.C.n_kv_heads;
    const int col = j * a.share + (hd - h * a.share);
    const int64_t rh = (int64_t)row * a.n_q_heads + hd;

    // where problem Q's partial results of column x lie: n of them, the i-th
    // at places place(i) of o and ml (0: none)
    struct Parts {
        const float* o;
        const float2* ml;
        int n, first, step;     // places first + i * step, and
        int other, last;        // the 0-th at `other`; places end at `last`
    };
    auto parts_of = [&](int kind, const Prob& Q, int q, int x) __attribute__((always_inline)) {
        const AttnPart& W = a.part[kind];
        const Parts one{W.row_o, W.row_ml, a.join ? 1 : 0, (int)rh, 0, (int)rh, (int)rh};
        Parts r{W.few_o, W.few_ml, 0, 0, 0, 0, 0};
        if (is_few(a, Q)) {
            if (W.few == 1) return one;
            if (key_tiles<ATTN_FEW_KEYS>(a, Q, Q.pos0, Q.pos1).n == 0) return r;
            const int2 b = W.rec[q * hkv + h];
            if (b.x == b.y) return one;
            r.n = min(b.y - b.x + 1, ATTN_FEW_WGS);
            r.first = 2 * b.x * 16 + x;
            r.step = 32;
            r.other = r.first + 16;
            r.last = 2 * ATTN_FEW_WGS * 16 - 1;
            return r;
        }
        const int4 it = W.slots ? W.item[q] : int4{0, 1, 1, 0};
        if (it.z == 1) return one;
        const int ct = x / ATTN_TILE_COLS;
        const int j_lo = ct * ATTN_TILE_COLS / a.share;
        const int j_hi = min(Q.nr - 1, (ct * ATTN_TILE_COLS + ATTN_TILE_COLS - 1) / a.share);
        const int n = key_tiles<ATTN_TILE_KEYS>(a, Q, kind == 0 ? Q.pos0 + j_lo : Q.pos0,
                                                kind == 0 ? Q.pos0 + j_hi : Q.pos1).n;
        r.o = W.tile_o;
        r.ml = W.tile_ml;
        r.n = min(max(1, (n + W.spl - 1) / W.spl), W.tile_grid);
        r.first = r.other = (it.x + (it.y - 1 - ct) * hkv + h) * ATTN_TILE_COLS + x % ATTN_TILE_COLS;
        r.step = it.y * hkv * ATTN_TILE_COLS;
        r.last = W.tile_grid * ATTN_TILE_COLS - 1;
        return r;
    };

    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    float M = -kInf, L = 0.f, v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 0.f;
    auto add = [&](const Parts& R) __attribute__((always_inline)) {
        // whatever the batch's offsets say, places stay inside the workspace
        auto at = [&](int i) { return min(max(i == 0 ? R.other : R.first + i * R.step, 0), R.last); };
        for (int i0 = 0; __ballot(i0 < R.n); i0 += 16) {
            const int here = min(16, R.n - i0);
            const float2 x = sl < here ? R.ml[at(i0 + sl)] : float2{-kInf, 0.f};
            float top = x.x;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
            const float m_new = fmaxf(M, top);
            const float mc = m_new == -kInf ? 0.f : m_new * c;
            const float f = exp2_fast(M * c - mc);
            const float w = exp2_fast(x.x * c - mc);
            float sum = sl < here ? w * x.y : 0.f;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) sum += __shfl_xor(sum, d, 64);
            L = L * f + sum;
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] *= f;
            M = m_new;
            for (int i1 = 0; __ballot(i1 < here); i1 += 4) {
                float4 y[4][N / 4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = i1 + u < here ? i0 + i1 + u : 0;
                    const float* src = R.o + (int64_t)at(i) * D + sl * N;
#pragma unroll
                    for (int e = 0; e < N / 4; ++e)
                        if (i1 + u < here) y[u][e] = *(const float4*)(src + 4 * e);
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float wi = __shfl(w, (i1 + u) & 15, 16);
                    if (i1 + u < here) {
#pragma unroll
                        for (int e = 0; e < N / 4; ++e) {
                            v[4 * e] += wi * y[u][e].x;
                            v[4 * e + 1] += wi * y[u][e].y;
                            v[4 * e + 2] += wi * y[u][e].z;
                            v[4 * e + 3] += wi * y[u][e].w;
                        }
                    }
                }
            }
        }
    };

    Parts own = parts_of(0, P, s, col);
    bool write = mine;
    if (!a.join) {   // whole results are in place already
        if (few && a.part[0].few == 1) return;
        const bool partial = own.n > 0 || (few && key_tiles<ATTN_FEW_KEYS>(a, P, P.pos0, P.pos1).n == 0);
        write = write && partial;
        if (!__ballot(write)) return;
    }
    if (P.pos0 + j < P.key0) {   // more rows than tokens: this row has no place and sees nothing
        own.n = 0;
    } else if (a.join && B.n_groups) {
        const int g = wave_find_run(B.group_off, B.n_groups, s, lane);
        if (g < B.n_groups) {
            const Prob G = load_prob(a, 1, g);
            const int gj = row - G.r0;
            if (gj >= 0 && gj < G.nr && G.len > 0) add(parts_of(1, G, g, gj * a.share + (hd - h * a.share)));
        }
    }
    add(own);
    if (!write) return;
    put_out<N>(a, row, head, D, sl * N, v, L);
    if (a.lse && sl == 0) a.lse[rh] = lse_of(a, M, L);
}

template <typename T, int D>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
    const int64_t grid = (int64_t)a.part[0].tile_grid + a.part[1].tile_grid + a.part[0].few_grid + a.part[1].few_grid;
    const bool paged = (1 << a.C.page_shift) >= 64 / Tile<T, D>::LPR;
    if (paged) hipLaunchKernelGGL((k_attn<T, D, true>), dim3((unsigned)grid), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_attn<T, D, false>), dim3((unsigned)grid), dim3(256), 0, stream, a);
    if (a.need_join) {
        const int by_row = a.join || a.part[0].slots;
        const int few_rows = std::max(1, std::min(ATTN_FEW_COLS / a.share, a.part[0].max_rows));
        const int64_t rows = by_row ? a.B.n_rows : (int64_t)a.B.n_seqs * few_rows;
        hipLaunchKernelGGL((k_attn_join<D>), dim3((unsigned)ceil_div(rows * ceil_div(a.n_q_heads, 4), 4)), dim3(256), 0,
                           stream, a, by_row, few_rows);
    }
    return hipGetLastError();
}

}  // namespace

void plan_attn(AttnPlan& P, int32_t head_dim, const int32_t (&n_prob)[2], const int32_t (&max_rows)[2],
               const int32_t (&max_len)[2]) {
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
    for (int k = 0; k < 2; ++k) {
        AttnPart& W = a.part[k];
        W = AttnPart{};
        W.max_rows = max_rows[k];
        W.max_len = max_len[k];
        for (size_t& o : P.off[k]) o = 0;
        if (n_prob[k] <= 0) continue;
        // the keys that a problem's tiles span.  The workspace does not rest on
        // the window: with one there are fewer keys, so fewer shared units, and
        // no more splits than the bound `most` below.
        int64_t reach = max_len[k];
        if (a.window > 0) reach = std::min<int64_t>(reach, (int64_t)a.window + max_rows[k] + a.n_sink + 256);
        if (a.share <= ATTN_FEW_COLS) {
            const int64_t units = ceil_div(reach, ATTN_FEW_KEYS);
            W.few = units <= 2 ? 1 : 2;
            W.few_grid = W.few == 1 ? n_prob[k] * hkv : ATTN_FEW_WGS;
            if (W.few == 2) a.need_join = 1;
            if (ceil_div(max_len[k], ATTN_FEW_KEYS) > 2) {
                P.off[k][0] = take((size_t)n_prob[k] * hkv * sizeof(int2));
                P.off[k][1] = take((size_t)2 * ATTN_FEW_WGS * 16 * head_dim * 4);
                P.off[k][2] = take((size_t)2 * ATTN_FEW_WGS * 16 * sizeof(float2));
            }
        }
        if ((int64_t)max_rows[k] * a.share > ATTN_FEW_COLS) {
            const int64_t nct = (int64_t)a.B.n_rows * a.share / ATTN_TILE_COLS + std::min(n_prob[k], a.B.n_rows);
            const int64_t tiles = ceil_div(reach, ATTN_TILE_KEYS) + 1;
            const int64_t spl = std::max<int64_t>(8, ceil_div(tiles * nct * hkv, 1024));
            W.spl = (int32_t)std::min<int64_t>(spl, 1 << 30);
            const int64_t ns = std::max<int64_t>(1, ceil_div(tiles, W.spl));
            W.tile_grid = (int32_t)(nct * hkv * ns);
            W.slots = ns > 1 ? 1 : 0;
            if (W.slots) a.need_join = 1;
            const int64_t most = std::min(ceil_div(1024, nct * hkv),
                                          ceil_div(ceil_div(max_len[k], ATTN_TILE_KEYS) + 1, 8));
            if (most > 1) {
                P.off[k][3] = take((size_t)n_prob[k] * sizeof(int4));
                P.off[k][4] = take((size_t)(nct * hkv * most) * ATTN_TILE_COLS * head_dim * 4);
                P.off[k][5] = take((size_t)(nct * hkv * most) * ATTN_TILE_COLS * sizeof(float2));
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
