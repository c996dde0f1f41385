// Attention over a paged key/value cache: what its forms share (attn.hip: bf16
// and fp32, attn_q8.hip: 8 bits).
//
//     o = sum_k softmax_k(scale q . k) v,    lse = log sum_k exp(scale q . k)
//
// a row at position p seeing key k when k <= p and, with a window, when
// k > p - window or k < n_sink.
//
// Both forms (few query columns, many) make the transposed products: S^T = K Q^T, then O^T = V^T P^T.
// The matrix cores' output layout puts one query column in each lane, so the
// running maximum and sum of the softmax are one register a lane, a column's
// scores are folded by one or two lane exchanges, and the rounded weights are
// already the operand of the second product: they never leave registers.
// (An output lane holds keys 4g .. 4g + 3 of a block, not eight neighbours;
// a product's sum may run in any order, so V is read in that same order, by
// LDS transpose reads.)  Scores, the statistics and O are fp32; the weights
// P are rounded to the cache's type for the second product, each by at most
// 2^-8 of itself in bf16, the rounding o itself gets at the end; they are
// summed for the softmax before they are rounded.
#pragma once

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
// that scores may exceed: weights up to 2^20 are as exact in fp32 and bf16 as
// weights below 1, and almost no tile needs a rescaling of O.  The reference
// is raised by a score that exceeds it by more; such a weight is noticed in the
// sum of a lane's weights.
constexpr float kSlackLog2 = 20.f, kSlack = 1048576.f;
// A weight is exp2((s - m) c).  The tiled form takes it as s c - m c, one
// operation with m c rounded before; all weights of a column carry that
// rounding alike and it drops out, unless m c is so large that 2 to its
// rounding is not near 1 (and for 2^31 no number).  From 2^20 on, where a
// score in fp32 is known to 2^-4 at best, the difference is taken first.
constexpr float kLargeLog2 = 1048576.f;
// as a raw score; finite where c is next to nothing, so that a first score
// still exceeds -infinity by more
__device__ __forceinline__ float slack_of(float c) { return fminf(kSlackLog2 / c, 3.402823466e38f); }

// A staged tile of keys or values: rows of D elements as they lie, 16-byte
// pieces permuted inside a row (or a pair of rows when a row is 128 bytes) so
// that the lanes of one LDS access fall in distinct banks.
template <typename T, int D>
struct Tile {
    static constexpr int RB = D * (int)sizeof(T);   // bytes of a row
    static constexpr int LPR = RB / 16;             // pieces of a row
    // what a row's pieces are permuted with (XOR).  Keys: 16 lanes read one
    // piece of 16 neighbouring rows.
    static __device__ __forceinline__ constexpr int kx(int key) { return RB == 128 ? (key >> 1) & 7 : key & 15; }
    // Values, bf16: a transpose read takes 32 bytes of each of 4 rows per 16
    // lanes, 8 or 16 rows in all; fp32: 64 or 128 neighbouring bytes of rows 4
    // apart.
    static __device__ __forceinline__ constexpr int vx(int key) {
        return sizeof(T) == 4 ? ((key >> 2) & 1) << 2 : RB == 128 ? ((key >> 1) & 3) << 1 : (key & 7) << 1;
    }
    static __device__ __forceinline__ int k_at(int key, int piece) { return key * RB + ((piece ^ kx(key)) << 4); }
    static __device__ __forceinline__ int v_at(int key, int piece) { return key * RB + ((piece ^ vx(key)) << 4); }
    // Both distribute over XOR where the parts share no bits, so a lane keeps
    // one offset and reaches its other rows and pieces with constants:
    //   at(r0 + r, piece) = r0 * RB + (at(r, piece) ^ x(r0) << 4)
    //   at(r, p0 + piece) = at(r, piece) ^ p0 << 4
    static __device__ __forceinline__ int v_elem(int key, int dim) {
        const int byte = dim * (int)sizeof(T);
        return v_at(key, byte >> 4) + (byte & 15);
    }
    static constexpr int piece_of(int dim) { return dim * (int)sizeof(T) / 16; }
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
    // eight neighbouring elements of one key, from the offset of the first's piece
    static __device__ __forceinline__ typename Op<T>::frag k_frag(const uint8_t* sk, int at) {
        if constexpr (sizeof(T) == 2) {
            return *(const bf16x8_t*)(sk + at);
        } else {
            const float4 a = *(const float4*)(sk + at), b = *(const float4*)(sk + (at ^ 16));
            return f32x8_t{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        }
    }
};

// v, but computed from here on: what is derived from it (in a rarely taken
// branch, or cheaply) is then not kept in registers through a whole loop.
__device__ __forceinline__ int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

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

// The length of the prefix before sequence s, and its group (n_groups: none).
// Called by a whole wave with a uniform s: one round of loads up to 64 groups.
__device__ inline int prefix_of(const KvBatchDev& B, int s, int lane, int& g) {
    if (B.n_groups <= 64) {
        const int end = lane < B.n_groups ? B.group_off[lane + 1] : 0x7fffffff;
        const int len = lane < B.n_groups ? B.prefix_len[lane] : 0;
        g = __popcll(__ballot(end <= s));
        return g < B.n_groups ? max(__builtin_amdgcn_readlane(len, g), 0) : 0;
    }
    g = wave_find_run(B.group_off, B.n_groups, s, lane);
    return g < B.n_groups ? max(B.prefix_len[g], 0) : 0;
}

// WAVE: p is uniform and a whole wave calls (its loads then go out together);
// otherwise every thread has its own p.
template <bool WAVE>
__device__ inline Prob load_prob(const AttnArgs& a, int kind, int p, int lane = 0) {
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
            int g;
            if constexpr (WAVE) {
                P.key0 = prefix_of(B, p, lane, g);
            } else {
                g = find_run(B.group_off, B.n_groups, p);
                if (g < B.n_groups) P.key0 = max(B.prefix_len[g], 0);
            }
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
__device__ __forceinline__ Range key_tiles(const AttnArgs& a, int len, int key0, int p_lo, int p_hi) {
    Range R{0, 0, 0};
    const int e = min(len, p_hi - key0 + 1);
    if (e <= 0) return R;
    const int te = (e + KB - 1) / KB;
    if (a.window > 0) {
        const int lo = p_lo - a.window + 1 - key0;
        if (lo > 0) R.first = min(lo / KB, te);
        const int sk = min(e, a.n_sink - key0);
        if (sk > 0) R.ns = min((sk + KB - 1) / KB, R.first);
    }
    R.n = R.ns + te - R.first;
    return R;
}

template <int KB>
__device__ __forceinline__ Range key_tiles(const AttnArgs& a, const Prob& P, int p_lo, int p_hi) {
    return key_tiles<KB>(a, P.len, P.key0, p_lo, p_hi);
}

// The keys of a tiled problem: a sequence of many columns walks its prefix
// and its own tokens in one go (each of its column tiles feeds the matrix
// cores by itself, so reading the prefix once per group would save nothing
// that bounds it, and its results need no join); a group's problem has only
// its prefix, for the rows of its few-column sequences.
struct Before {
    int len;              // 0: none
    const int32_t* tbl;
};
template <bool WAVE>
__device__ inline Before prefix_keys(const AttnArgs& a, int kind, int p, int lane = 0) {
    const KvBatchDev& B = a.B;
    Before F{0, nullptr};
    if (kind != 0 || B.n_groups == 0) return F;
    int g, len;
    if constexpr (WAVE) {
        len = prefix_of(B, p, lane, g);
    } else {
        g = find_run(B.group_off, B.n_groups, p);
        len = g < B.n_groups ? max(B.prefix_len[g], 0) : 0;
    }
    F.len = table_keys(min(len, a.part[1].max_len), B.ldpp, a.C.page_shift);
    F.tbl = B.prefix_pages + (int64_t)min(g, B.n_groups - 1) * B.ldpp;
    return F;
}
// Tiles of both, the prefix's first, that rows at positions lo .. hi see some key of.
struct Walk {
    Range pre, own;
    __device__ __forceinline__ int n() const { return pre.n + own.n; }
};
template <int KB>
__device__ __forceinline__ Walk walk_of(const AttnArgs& a, const Before& F, const Prob& P, int lo, int hi) {
    return Walk{key_tiles<KB>(a, F.len, 0, lo, hi), key_tiles<KB>(a, P, lo, hi)};
}
// The lowest position of rows from j on: -1 where a row has no place (more
// rows than tokens) and sees nothing.
__device__ __forceinline__ int lowest(const Prob& P, int j) {
    const int at = P.pos0 + j;
    return at < P.key0 ? -1 : at;
}

// Position of query row `row` (kind 1 rows lie in several sequences); -1 for none.
// seq_rows: the rows of its sequence.
__device__ inline int row_position(const AttnArgs& a, int row, int& seq_rows) {
    const KvBatchDev& B = a.B;
    const int s = find_run(B.row_off, B.n_seqs, row);
    seq_rows = 0;
    if (s >= B.n_seqs) return -1;
    seq_rows = min(B.row_off[s + 1] - B.row_off[s], a.part[0].max_rows);
    int before = 0;
    if (B.n_groups) {
        const int g = find_run(B.group_off, B.n_groups, s);
        if (g < B.n_groups) before = max(B.prefix_len[g], 0);
    }
    return before + max(B.kv_len[s], 0) - (B.row_off[s + 1] - row);
}

// Inclusive scan over the workgroup's NW waves; *total: their sum.  sh: NW ints.
template <int NW>
__device__ inline int block_scan(int v, int tid, int* sh, int* total) {
    int x = wave_incl_scan(v, tid & 63);
    __syncthreads();
    if ((tid & 63) == 63) sh[tid >> 6] = x;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < (tid >> 6)) x += sh[w];
        sum += sh[w];
    }
    *total = sum;
    return x;
}

// The problem that work unit pick(total) lies in, units numbered problem by
// problem (units(p) each): its number and the units before it.  All threads;
// false where the pick is past the last unit.  sh: NW + 2 ints.
template <int NW, class F, class G>
__device__ inline bool locate(int n, F units, G pick, int tid, int* sh, int& p_out, int& base_out) {
    int total = 0, v = 0, incl = 0;
    for (int p0 = 0; p0 < n; p0 += 64 * NW) {   // one round where the problems are no more than the threads
        v = p0 + tid < n ? units(p0 + tid) : 0;
        int sum;
        incl = total + block_scan<NW>(v, tid, sh, &sum);
        total += sum;
    }
    const int u = pick(total);
    if (u >= total) return false;
    for (int p0 = 0, before = 0; p0 < n; p0 += 64 * NW) {
        int sum = total;
        if (n > 64 * NW) {
            v = p0 + tid < n ? units(p0 + tid) : 0;
            incl = before + block_scan<NW>(v, tid, sh, &sum);
        }
        if (u < before + sum) {
            if (u < incl && u >= incl - v) {
                sh[NW] = p0 + tid;
                sh[NW + 1] = incl - v;
            }
            break;
        }
        before += sum;
    }
    __syncthreads();
    p_out = __builtin_amdgcn_readfirstlane(sh[NW]);
    base_out = __builtin_amdgcn_readfirstlane(sh[NW + 1]);
    return true;
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

// 16 bytes that no other workgroup reads: they pass the caches by (a read
// stream of this shape reaches 6.5 TB/s so, and 5.9 through L2)
__device__ __forceinline__ u32x4_t piece_at(const void* p) { return __builtin_nontemporal_load((const u32x4_t*)p); }

// Where key `key` of head h lies in the cache, in elements.
__device__ __forceinline__ int64_t place_of(const AttnArgs& a, int page, int key, int h) {
    return (int64_t)page * a.C.page_stride + (int64_t)((key & ((1 << a.C.page_shift) - 1)) * (int)a.C.token_stride) +
           (int64_t)h * a.C.head_stride;
}
// the value of lane l, uniform
__device__ __forceinline__ int64_t lane_of(int64_t v, int l) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)v, l), hi = __builtin_amdgcn_readlane((int)(v >> 32), l);
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// Requests 16-byte pieces of NL x STEP neighbouring keys of one tensor: load j
// covers keys j * STEP .. of the tile.  `place`: where key `lane` of the tile
// lies.  PAGED: a load's keys lie in one page (page_size >= the keys of a
// load), so its base is scalar; otherwise every lane follows its own key.
template <typename T, int D, int NL, int STEP, bool PAGED>
__device__ __forceinline__ void request(const AttnArgs& a, const void* from, int64_t place, int lane, u32x4_t (&r)[NL]) {
    using TL = Tile<T, D>;
    const int row = lane / TL::LPR, piece = (lane % TL::LPR) * (16 / (int)sizeof(T));
    const uint32_t in = (uint32_t)((PAGED ? row * (int)a.C.token_stride : 0) + piece);
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const int64_t off = PAGED ? lane_of(place, j * STEP) : __shfl(place, j * STEP + row, 64);
        r[j] = piece_at((const T*)from + off + in);
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

template <int V>
struct Int {
    __device__ constexpr operator int() const { return V; }
};

// Keeps the computation of a value above this point.
__device__ __forceinline__ void stay(bf16x8_t& v) {
    u32x4_t x = __builtin_bit_cast(u32x4_t, v);
    asm volatile("" : "+v"(x));
    v = __builtin_bit_cast(bf16x8_t, x);
}
__device__ __forceinline__ void stay(f32x8_t&) {}

// Order of a block of bf16 matrix products: AHEAD operand reads from LDS, then
// after each of N products READS more of them, VALU vector operations and
// TRANS exponentials, so that the wave's matrix and vector work overlap.
// (fp32 products take 16 times as long and hide everything else.)
template <typename T, int AHEAD, int N, int READS, int VALU, int TRANS>
__device__ __forceinline__ void sched_mix() {
    if constexpr (sizeof(T) == 2) {
        __builtin_amdgcn_sched_group_barrier(0x100, AHEAD * READS, 0);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (n + AHEAD < N) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
            if (TRANS) __builtin_amdgcn_sched_group_barrier(0x400, TRANS, 0);
            if (VALU) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
        }
    }
}

// Direct loads from memory to LDS: lane i's 16 bytes go to `to` + 16 i.  The
// staged tile lies in rows of the pieces' permuted order, so a lane asks for
// the piece that belongs at its place.  M0 names the place; it is the
// compiler's register, and put back at once.  landed() waits for them; the compiler
// does not count them, and its own waits, which count fewer loads than are
// out, come out later and never earlier than they must.
__device__ __forceinline__ void lds_load(const void* base, uint32_t off, uint32_t to) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)base);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uintptr_t)base >> 32));
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "v"(off), "s"(((uint64_t)hi << 32) | lo), "s"(__builtin_amdgcn_readfirstlane(to))
                 : "memory");
}
__device__ __forceinline__ void lds_load(const void* at, uint32_t to) {
    uint32_t m0;
    asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "v"(at), "s"(__builtin_amdgcn_readfirstlane(to))
                 : "memory");
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint32_t lds_offset(const uint8_t* p) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)p);
}

// A workgroup's request of a tile of 64 keys: load n of K and of V, of NL.
template <typename T, int D, bool PAGED, int NW>
struct TileRequest {
    using TL = Tile<T, D>;
    static constexpr int RPW = 64 / TL::LPR;    // rows of a wave's load
    static constexpr int ALL = NW * RPW;        // rows of the workgroup's
    static constexpr int NL = ATTN_TILE_KEYS / ALL;
    static constexpr int NX = ALL < 16 ? 16 / ALL : 1;
    // bytes from a load's first row to this lane's piece.  The piece is the
    // one whose permuted place is the lane's; the permutations are their own
    // inverses and repeat every 16 rows, so with fewer rows than that to a
    // load every other load has its own.
    uint32_t pk[NX], pv[NX];
    __device__ __forceinline__ TileRequest(const AttnArgs& a, int wave, int lane) {
        const int r = lane / TL::LPR;
#pragma unroll
        for (int x = 0; x < NX; ++x) {
            const int row = x * ALL + wave * RPW + r;
            const uint32_t in = PAGED ? (uint32_t)(r * (int)a.C.token_stride) * (uint32_t)sizeof(T) : 0u;
            pk[x] = in + ((TL::k_at(row, lane % TL::LPR) >> 4) % TL::LPR) * 16;
            pv[x] = in + ((TL::v_at(row, lane % TL::LPR) >> 4) % TL::LPR) * 16;
        }
    }
    // `place`: where key `lane` of the tile lies
    __device__ __forceinline__ void load(const AttnArgs& a, int n, int64_t place, int wave, int lane, uint32_t to_k,
                                         uint32_t to_v) const {
        const int row0 = n * ALL + wave * RPW, x = n % NX;
        const uint32_t tk = to_k + row0 * TL::RB, tv = to_v + row0 * TL::RB;
        if constexpr (PAGED) {
            const int64_t off = lane_of(place, row0);
            lds_load((const T*)a.C.k + off, pk[x], tk);
            lds_load((const T*)a.C.v + off, pv[x], tv);
        } else {
            const int64_t off = __shfl(place, row0 + lane / TL::LPR, 64);
            lds_load((const uint8_t*)((const T*)a.C.k + off) + pk[x], tk);
            lds_load((const uint8_t*)((const T*)a.C.v + off) + pv[x], tv);
        }
    }
};

// Numbers in 8 bits: a scale as the widening takes it (a power of two, whatever
// the word holds), and eight neighbouring e4m3 numbers times it as bf16, which
// holds them exactly.
__device__ __forceinline__ float power_of(float scale) {
    const int e = (__float_as_uint(scale) >> 23) & 255;
    return __int_as_float(min(max(e, Q8_LEAST + 127), Q8_MOST + 127) << 23);
}
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi, float scale) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    union { bf16x2_t p[4]; bf16x8_t v; } t;
    t.p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    t.p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    t.p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    t.p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return t.v;
}
// Where the scale of key `key` of head h lies, in elements.
__device__ __forceinline__ int64_t scale_at(const AttnArgs& a, int page, int key, int h) {
    const int block = (key & ((1 << a.C.page_shift) - 1)) >> a.S.block_shift;
    return (int64_t)page * a.S.page_stride + (int64_t)(block * (int)a.S.block_stride) + (int64_t)h * a.S.head_stride;
}

// A workgroup's request of a tile of 64 keys in 8 bits: NT pieces of 16 numbers
// a thread, keys' and then values', in registers until they are widened into
// the staged tile of bf16 (so a number is widened once for all waves), after
// the tile's products: stores to LDS before them would keep the compiler from
// reading their operands ahead.  A prompt of 8192 tokens, 32 heads on 8 of 128:
// 585 us, as over a bf16 cache (580).  Pieces that wait in LDS instead cost 8 %
// more, and so do lane exchanges for places and scales.
template <int D, bool PAGED, int NW>
struct TileRequestQ8 {
    using TL = Tile<bf16, D>;
    static constexpr int LPR = D / 16;                                 // pieces of a key
    static constexpr int RPL = 64 / LPR;                               // keys of a wave's load
    static constexpr int NT = 2 * ATTN_TILE_KEYS * LPR / (64 * NW);    // loads, LPR waves' for each tensor
    u32x4_t r[NT];
    float s[NT];    // scales
    int at[NT];     // places in the staged tile
    __device__ __forceinline__ TileRequestQ8(int wave, int lane) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int L = n * NW + wave, row = (L % LPR) * RPL + lane / LPR, piece = 2 * (lane % LPR);
            at[n] = L < LPR ? TL::k_at(row, piece) : ATTN_TILE_KEYS * TL::RB + TL::v_at(row, piece);
        }
    }
    // place, scales: where key `lane` of the tile and its scales lie
    __device__ __forceinline__ void load(const AttnArgs& a, int64_t place, int64_t scales, int wave, int lane) {
        const int row = lane / LPR;
        // keys of a load start at a multiple of RPL: their blocks follow from the first one's
        const int block = PAGED ? (row >> a.S.block_shift) * (int)a.S.block_stride : 0;
        const uint32_t in = (uint32_t)((PAGED ? row * (int)a.C.token_stride : 0) + (lane % LPR) * 16);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int L = n * NW + wave, row0 = (L % LPR) * RPL;
            const int64_t off = PAGED ? lane_of(place, row0) : __shfl(place, row0 + row, 64);
            const int64_t sc = PAGED ? lane_of(scales, row0) : __shfl(scales, row0 + row, 64);
            s[n] = ((L < LPR ? a.S.k_scale : a.S.v_scale) + sc)[block];
            r[n] = *(const u32x4_t*)((const uint8_t*)(L < LPR ? a.C.k : a.C.v) + off + in);
        }
    }
    __device__ __forceinline__ void store(uint8_t* to) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float by = power_of(s[n]);
            *(bf16x8_t*)(to + at[n]) = widen(r[n].x, r[n].y, by);
            *(bf16x8_t*)(to + (at[n] ^ 16)) = widen(r[n].z, r[n].w, by);
        }
    }
};

// Which of the keys of a tile that starts at position lo a row at position
// col_pos sees, one bit each, of those that exist (`bits`).
__device__ __forceinline__ uint64_t sees(const AttnArgs& a, int col_pos, int lo, uint64_t bits) {
    auto below = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : ~0ull >> (64 - n); };   // keys 0 .. n - 1
    const int last = col_pos - lo;
    uint64_t v = bits & below(last + 1);
    if (a.window > 0) v &= ~below(last + 1 - a.window) | below(a.n_sink - lo);
    return v;
}

// ---------------------------------------------------------------------------
// Few query columns (decode): pieces of the keys
// ---------------------------------------------------------------------------

// Deals the units, FK keys of one (problem, key head) each: of every piece (a
// run of units of one problem P and key head h) of this workgroup's, calls
// work(P, R, h, i, n) with its n units from the i-th of the range R on (n = 0:
// rows that see no key) and finish(P, h, whole, slot): the piece is all of (P,
// h), or its results are partial and go to `slot`.  Shared form (few = 2): the units of
// all problems are dealt to the workgroups in equal runs, whatever the
// lengths; a run's first and last (problem, head) may be partial and go to
// slots that the join adds.  Otherwise a workgroup takes one (problem, head)
// whole.
template <int FK, int NW, class WORK, class FINISH>
__device__ __forceinline__ void few_pieces(const AttnArgs& a, int kind, int block, int blocks, int* sh, int tid, int lane,
                                           WORK work, FINISH finish) {
    const int hkv = a.C.n_kv_heads;
    const AttnPart& W = a.part[kind];
    const bool shared = W.few == 2;
    const int n_prob = problems(a, kind);
    auto range_of = [&](const Prob& P) __attribute__((always_inline)) {
        if (P.nr == 0 || !is_few(a, P)) return Range{0, 0, 0};
        return key_tiles<FK>(a, P, P.pos0, P.pos1);
    };

    int p, h, i;    // the piece worked on: problem, key head, first unit of it
    Prob P;
    Range R;
    int u = 0, u1;  // this workgroup's units [u, u1)
    uint32_t total = 0, wgs = 1;   // all units, and the workgroups that have some
    // a * b / d, in 32 bits where that holds
    auto share_of = [](uint32_t a, uint32_t b, uint32_t d) {
        return b < (1u << 20) ? a * b / d : (uint32_t)((uint64_t)a * b / d);
    };
    static_assert(ATTN_FEW_WGS <= 1 << 12, "share_of's products stay below 2^32");
    if (shared) {
        auto units = [&](int q) { return range_of(load_prob<false>(a, kind, q)).n * hkv; };
        auto pick = [&](int all) {
            total = all;
            wgs = min((uint32_t)blocks, total);   // no run between a first and a last one is empty
            if ((uint32_t)block >= wgs) return 0x7fffffff;
            u = (int)share_of(block, total, wgs);
            u1 = (int)share_of(block + 1, total, wgs);
            return u;
        };
        int base = 0;
        if (!locate<NW>(n_prob, units, pick, tid, sh, p, base)) return;
        P = load_prob<true>(a, kind, p, lane);
        R = range_of(P);
        h = (u - base) / R.n;
        i = u - base - h * R.n;
    } else {
        p = block / hkv;
        h = block - p * hkv;
        i = 0;
        P = load_prob<true>(a, kind, p, lane);
        if (P.nr == 0 || !is_few(a, P)) return;   // no rows, or the tiled form's
        R = range_of(P);
        u1 = R.n;
    }

    const int first = u;
    while (true) {
        const int n = min(R.n - i, u1 - u);
        work(P, R, h, i, n);
        bool whole = true;
        int slot = 0;
        if (shared) {
            const int ra = u - i, rb = ra + R.n;   // the units of (p, h)
            const bool starts = ra >= first;
            whole = starts && rb <= u1;
            slot = 2 * block + (starts ? 1 : 0);
            if (starts && tid == 0) W.rec[p * hkv + h] = int2{block, (int)(((uint64_t)rb * wgs - 1) / total)};
        }
        finish(P, h, whole, slot);
        u += n;
        if (u >= u1) break;
        __syncthreads();
        i = 0;
        if (++h == hkv) {
            h = 0;
            do {   // in bounds: units remain
                P = load_prob<true>(a, kind, ++p, lane);
                R = range_of(P);
            } while (R.n == 0 && p + 1 < n_prob);
        }
    }
}

// Joins the NW waves' results of a piece and writes them: to their place, or
// as partial results.  WB: LDS bytes of a wave's stage.  m, l and acc are a
// lane's largest score, sum of its weights and elements of O.
template <typename T, int D, int WB, int NW>
__device__ __forceinline__ void few_finish(const AttnArgs& a, int kind, const Prob& P, int h, bool whole, int slot,
                                           uint8_t* stage, int wave, int lane, float m, float l,
                                           const f32x4_t (&acc)[D / 16]) {
    constexpr int OP = D + 4;   // fp32 pitch of a wave's O
    const AttnPart& W = a.part[kind];
    const int tid = threadIdx.x, l16 = lane & 15, g4 = lane >> 4;
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    uint8_t* mine_at = stage + wave * WB;
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    float* so = (float*)mine_at;
    float* stat = so + 16 * OP;   // 16 largest scores, 16 sums
    if (lane < 16) {
        stat[lane] = m;
        stat[16 + lane] = l;
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
        *(float4*)(so + l16 * OP + t * 16 + g4 * 4) = float4{acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
    __syncthreads();
    if (NW == 4 || tid < 256) {
        constexpr int N = D / 16;   // elements per thread, of column tid / 16
        constexpr int WF = WB / 4;  // floats of a wave's stage
        const int col = tid >> 4, d = (tid & 15) * N;
        const float* all = (const float*)stage;
        float mw[NW], M = -kInf, sum = 0.f, v[N];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            mw[w] = all[w * WF + 16 * OP + col];
            M = fmaxf(M, mw[w]);
        }
        const float ref = M == -kInf ? 0.f : M;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            mw[w] = exp2_fast((mw[w] - ref) * c);
            sum += mw[w] * all[w * WF + 16 * OP + 16 + col];
        }
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            float4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
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
}

// ---------------------------------------------------------------------------
// Many query columns (prompts, shared prefixes): the columns are split
// ---------------------------------------------------------------------------

// A workgroup owns 128 or 256 columns of one key head, 32 a wave, and walks
// tiles of 64 keys that its waves load straight into LDS: two buffers, one
// barrier a tile, the next tile's loads spread over this one's products.  Each
// staged byte feeds all columns, 4 D flop per key and column, so the matrix
// cores bound it; a wave's two halves of 32 keys let them work on one half
// while the vector units make weights of the other.  Items (problem, column
// tile, key head, run of key tiles) are numbered with the key head fastest,
// so that the columns of one head meet in one XCD's L2, and later column
// tiles (more keys under the causal mask) first.
//
// bf16, 32 heads on 8 of 128, a prompt of 8192 tokens: 570 us, 965 TFLOP/s of
// the 1273 that a large matrix product reaches.  A tile of 64 keys by 256
// columns takes 2.2 us of a CU, of them 0.9 at the matrix cores' peak; the
// rest is LDS reads' latency, the waves' skew at the barrier and the softmax's
// vector work.  Beside 16 decode rows, 4 prompt pieces of 512 rows, 64 heads
// on 8, in windows of 2048 with 4 sinks (8.6e10 flop): 169 us in three
// launches one after another, this one 136, the few-column form 33, the join
// 6.  Its 512 items have 2 to 35 tiles and take 49 in a row on 256 CUs (43 if
// they were even), 2.8 us each: the tiles at the window's ends are masked,
// their values looked over behind a second barrier, and the sinks cost one
// tile more.  Over a prefix with a window (kind 1) every tile goes that way,
// since what a window's row sees is not known from its place in the group.
//
// Only rows of up to 256 bytes leave the registers for tiles of 256 columns.
template <typename T, int D> constexpr bool kWide = sizeof(T) * D <= 256;
template <class FORM, int NW>
__device__ __forceinline__ void attn_tile(const AttnArgs& a, int kind, int block, uint8_t* stage, int* sh) {
    using T = typename FORM::T;
    constexpr int D = FORM::D;
    constexpr bool PAGED = FORM::PAGED;
    using TL = Tile<T, D>;
    using O = Op<T>;
    constexpr int KB = ATTN_TILE_KEYS, TC = 32 * NW;
    constexpr int NL = KB * TL::LPR / (64 * NW);   // loads per wave, of K and of V
    constexpr int RPL = 64 * NW / TL::LPR;         // rows one load of the workgroup covers
    constexpr int TB = KB * TL::RB;            // bytes of a staged tile
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, h2 = lane >> 5, l16 = lane & 15, d16 = (lane >> 4) & 1;
    const int hkv = a.C.n_kv_heads;
    const AttnPart& W = a.part[kind];
    const int n_prob = problems(a, kind);
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();
    const float slack = slack_of(c);
    // this lane's operands in a staged tile of keys and of values
    const int kop = TL::k_at(l32, TL::piece_of(h2 * 8)), vop = TL::v_base(4 * h2, d16 * 16, l16);

    auto splits_of = [&](const Before& F, const Prob& Q, int& nct) __attribute__((always_inline)) {
        const int64_t cols = (int64_t)Q.nr * a.share;
        nct = cols > ATTN_FEW_COLS ? (int)((cols + TC - 1) / TC) : 0;
        const int n = walk_of<KB>(a, F, Q, Q.pos0, Q.pos1).n();
        return n > W.spl ? (n + W.spl - 1) / W.spl : 1;
    };
    int p, base;
    if (!locate<NW>(
            n_prob,
            [&](int q) {
                int nct;
                const int ns = splits_of(prefix_keys<false>(a, kind, q), load_prob<false>(a, kind, q), nct);
                return nct * ns * hkv;
            },
            [&](int) { return block; }, tid, sh, p, base))
        return;
    const Prob P = load_prob<true>(a, kind, p, lane);
    const Before F = prefix_keys<true>(a, kind, p, lane);
    int nct;
    const int nsplit = splits_of(F, P, nct);
    int rem = block - base;
    const int h = rem % hkv;
    rem /= hkv;
    const int split = rem / nct;
    const int ct = nct - 1 - rem % nct;
    if (rem == 0 && h == 0 && tid == 0 && W.slots) W.item[p] = int4{base, nct, nsplit, 0};

    // the workgroup's rows, its key tiles and this split's run of them
    const int j_lo = ct * TC / a.share, j_hi = min(P.nr - 1, (ct * TC + TC - 1) / a.share);
    int wg_lo = kind == 0 ? lowest(P, j_lo) : P.pos0;
    const int wg_hi = kind == 0 ? P.pos0 + j_hi : P.pos1;
    const Walk R = walk_of<KB>(a, F, P, kind == 0 ? P.pos0 + j_lo : P.pos0, wg_hi);
    const int i0 = split * W.spl, i1 = min(R.n(), i0 + W.spl);
    if (split > 0 && i0 >= R.n()) return;
    // a tile: its first key in its page table, that key's position, the
    // table's keys and the table
    struct At {
        int key, pos, len;
        const int32_t* tbl;
    };
    auto tile_at = [&](int i) __attribute__((always_inline)) {
        const bool pre = i < R.pre.n;
        const int key = KB * (pre ? R.pre.tile(i) : R.own.tile(i - R.pre.n));
        return At{key, pre ? key : key + P.key0, pre ? F.len : P.len, pre ? F.tbl : P.tbl};
    };

    // this lane's column
    const int64_t n_cols = (int64_t)P.nr * a.share;
    const int col = ct * TC + wave * 32 + l32;
    bool there = col < n_cols;
    const int j = there ? col / a.share : 0;
    const int row = P.r0 + j, head = h * a.share + (there ? col - j * a.share : 0);
    int col_pos = -1;
    if (there) col_pos = kind == 0 ? lowest(P, j) : P.pos1;
    if (kind == 1 && there && (a.window > 0 || !a.decode)) {
        int seq_rows;
        const int at = row_position(a, row, seq_rows);
        if (a.window > 0) col_pos = at;
        there = (int64_t)seq_rows * a.share <= ATTN_FEW_COLS;   // the others walk the prefix themselves
    }
    if (kind == 1 && !a.decode && !__syncthreads_or(there)) return;
    if (kind == 1 && a.window > 0) {   // the least position that a window reaches back from
        int lo = there ? col_pos : 0x7fffffff;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) lo = min(lo, __shfl_xor(lo, x, 64));
        if (lane == 0) sh[wave] = lo;
        __syncthreads();
        wg_lo = sh[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) wg_lo = min(wg_lo, sh[w]);
        wg_lo = __builtin_amdgcn_readfirstlane(wg_lo);
    }
    const bool wave_there = __ballot(there) != 0;
    // least and largest position of the wave's columns
    const int wv_lo = kind == 0 ? lowest(P, (ct * TC + wave * 32) / a.share) : P.pos0;
    const int wv_hi = kind == 0 ? min(P.pos1, P.pos0 + (ct * TC + wave * 32 + 31) / a.share) : P.pos1;

    typename O::frag qf[D / 16];
    {
        const T* q = (const T*)a.q + (int64_t)row * a.ldq + (int64_t)head * D;
#pragma unroll
        for (int s = 0; s < D / 16; ++s) qf[s] = there ? O::load(q + s * 16 + h2 * 8) : O::zero();
    }
    float m, l;
    f32x16_t acc[D / 32];

    // page number of key `lane` of a tile, -1: none
    auto load_id = [&](const At& X) __attribute__((always_inline)) {
        const int key = X.key + lane;
        return key < X.len ? X.tbl[key >> a.C.page_shift] : -1;
    };
    // bit k says whether any column sees key k of a tile; place: where key
    // `lane` is read from (in page 0 where its page number is no good)
    // (and, in 8 bits, where its scale lies)
    auto seen_of = [&](const At& X, int id, int64_t& place, int64_t& scales) __attribute__((always_inline)) {
        const int at = X.pos + lane;
        const bool page_ok = id >= 0 && id < a.C.n_pages;
        bool seen = X.key + lane < X.len && at <= wg_hi;
        if (a.window > 0) seen = seen && (at > wg_lo - a.window || at < a.n_sink);
        if (seen && !page_ok && a.status) flag_bad_id(a.status);
        place = place_of(a, page_ok ? id : 0, X.key + lane, h);
        if constexpr (FORM::Q8) scales = scale_at(a, page_ok ? id : 0, X.key + lane, h);
        return (uint64_t)__ballot(seen && page_ok);
    };
    auto request = [&]() __attribute__((always_inline)) {
        if constexpr (FORM::Q8) return TileRequestQ8<D, PAGED, NW>(wave, lane);
        else return TileRequest<T, D, PAGED, NW>(a, wave, lane);
    }();
    const uint32_t stage_at = lds_offset(stage);
    // the loads from..to - 1 of a tile into a buffer; in 8 bits all of them
    // with the first, into registers
    auto load = [&](int from, int to, int64_t place, int64_t scales, int buf) __attribute__((always_inline)) {
        if constexpr (FORM::Q8) {
            if (from == 0) request.load(a, place, scales, wave, lane);
        } else {
            const uint32_t at = stage_at + buf * 2 * TB;
#pragma unroll
            for (int n = from; n < to; ++n) request.load(a, n, place, wave, lane, at, at + TB);
        }
    };
    // what was loaded in 8 bits goes into its buffer, which nobody reads any more
    auto stash = [&](int buf) __attribute__((always_inline)) {
        if constexpr (FORM::Q8) request.store(stage + buf * 2 * TB);
    };
    constexpr int Q1 = (NL + 3) / 4, Q2 = (NL + 1) / 2, Q3 = (3 * NL + 3) / 4;   // a quarter each

    // Walks the tiles.  Infinities or NaN among values that some columns do
    // not see (0 times them is NaN) are looked for in the tiles that columns
    // see in part; where there are some (sh[NW + 2]) the walk is made again with
    // ODD, which leaves them out of the product and adds them to the columns
    // that see them.
    if (tid == 0) sh[NW + 2] = 0;
    auto walk = [&](auto ODD) __attribute__((always_inline)) {
        m = there ? -kInf : 0.f;   // (no column: q is 0, nothing ever asks for a reference)
        l = 0.f;
#pragma unroll
        for (int t = 0; t < D / 32; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[t][r] = 0.f;
        if (i0 >= i1) return;
        At cur = tile_at(i0), nxt = cur, aft = tile_at(min(i0 + 1, i1 - 1));   // tiles i, i + 1, i + 2
        int id = load_id(cur);
        int64_t place, scales = 0;
        uint64_t bits = seen_of(cur, id, place, scales), bits_i = 0;
        load(0, NL, place, scales, 0);
        stash(0);
        id = load_id(aft);
        // tile i is there: requests the next one (the first quarter of it, or
        // all; after the last one that one again, so that nothing branches)
        auto arrive = [&](int i, int quarters) __attribute__((always_inline)) {
            const int buf = (i - i0) & 1;
            if constexpr (!FORM::Q8) landed();
            __syncthreads();   // and nobody reads the other buffer any more
            bits_i = bits;
            cur = nxt;
            nxt = aft;
            aft = tile_at(min(i + 2, i1 - 1));
            bits = seen_of(nxt, id, place, scales);
            id = load_id(aft);
            load(0, quarters == 1 ? Q1 : NL, place, scales, buf ^ 1);
            const int lo = cur.pos;
            if (bits_i != ~0ull || lo + KB - 1 > wg_lo || (a.window != 0 && lo <= wg_hi - a.window)) {
                // values that no column sees are cleared; are the others finite?
                uint8_t* sv = stage + buf * 2 * TB + TB;
                const int me = here(tid);
                bool odd = false;
#pragma unroll
                for (int n = 0; n < NL; ++n) {
                    const int r = n * RPL + me / TL::LPR;
                    u32x4_t* at = (u32x4_t*)(sv + r * TL::RB + (me % TL::LPR) * 16);
                    if ((bits_i >> r) & 1) odd |= odd_piece<T>(*at);
                    else *at = u32x4_t{0u, 0u, 0u, 0u};
                }
                if (__ballot(odd) && lane == 0) sh[NW + 2] = 1;
                __syncthreads();
            }
        };
        // the wave's own end: later tiles hold only keys past its rows
        int iw = i0;
        if (wave_there) {
            iw = i1;
            while (iw > i0 && tile_at(iw - 1).pos > wv_hi) --iw;
        }
        for (int i = i0; i < iw; ++i) {
            const int buf = (i - i0) & 1;
            const uint8_t* sk = stage + buf * 2 * TB;
            const uint8_t* sv = sk + TB;
            arrive(i, 1);
            const int lo = cur.pos;
            const bool all_see = bits_i == ~0ull && lo + KB - 1 <= wv_lo && (a.window == 0 || lo > wv_hi - a.window);

            // Two halves of 32 keys, so that the matrix cores work on one
            // while the vector units turn the other's scores into weights.
            // Element r of w[kb]: key 32 kb + 8 (r / 4) + 4 h2 + r % 4.
            f32x16_t w[2];
            typename O::frag pf[2][2];
            float sum[2];
            const int ka = here(kop), va = here(vop);
            auto scores = [&](auto kb) __attribute__((always_inline)) {
#pragma unroll
                for (int r = 0; r < 16; ++r) w[kb][r] = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    w[kb] = O::mma32(TL::k_frag(sk + kb * 32 * TL::RB, ka ^ (TL::piece_of(ks * 16) << 4)), qf[ks], w[kb]);
            };
            auto weights = [&](auto kb, auto LARGE) __attribute__((always_inline)) {
                const float mc = m == -kInf ? 0.f : m * c;
                const bool large = LARGE && !(fabsf(mc) < kLargeLog2);
                const float ref = large ? m : 0.f, rest = large ? 0.f : mc;
                float part[4];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    w[kb][r] = exp2_fast(LARGE ? (w[kb][r] - ref) * c - rest : w[kb][r] * c - mc);
                    part[r & 3] = r < 4 ? w[kb][r] : part[r & 3] + w[kb][r];
                }
                sum[kb] = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    f32x8_t v;
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = w[kb][8 * x + e];
                    pf[kb][x] = O::round(v);
                }
            };
            constexpr Int<0> h0{};
            constexpr Int<1> h1{};
            // Every key seen and every column with a reference that is not
            // large: no branch until the weights are there.
            bool done = all_see && !__ballot(!(fabsf(m * c) < kLargeLog2));
            if (done) {
                scores(h0);
                sched_mix<T, 4, D / 16, 1, 0, 0>();
                load(Q1, Q2, place, scales, buf ^ 1);
                scores(h1);
                weights(h0, h0);
                sched_mix<T, 4, D / 16, 1, 4, 2>();
                stay(pf[0][0]);
                stay(pf[0][1]);
                load(Q2, Q3, place, scales, buf ^ 1);
                weights(h1, h0);
                load(Q3, NL, place, scales, buf ^ 1);
                done = !__ballot(fmaxf(sum[0], sum[1]) > kSlack);
            } else {
                load(Q1, NL, place, scales, buf ^ 1);
            }
            if (!done) {
                asm volatile("");
                scores(h0);
                scores(h1);
                if (!all_see) {
                    const uint64_t v = sees(a, col_pos, lo, bits_i) >> here(4 * h2);
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            w[kb][r] = (uint32_t)(v >> (32 * kb)) & (1u << (8 * (r >> 2) + (r & 3))) ? w[kb][r] : -kInf;
                }
                // A reference is a column's own matter: it is set by the first
                // tile with a key that the column sees and raised by a score
                // that exceeds it by the slack, whatever the neighbours do.
                float top = max_of(w[0][0], w[1][0]);
#pragma unroll
                for (int r = 1; r < 16; ++r) top = fmaxf(top, max_of(w[0][r], w[1][r]));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const bool up = top > m + slack;
                const float f = up ? exp2_fast((m - top) * c) : 1.f;   // from -infinity: 0
                m = up ? top : m;
                l *= f;
#pragma unroll
                for (int t = 0; t < D / 32; ++t) acc[t] *= f;
                weights(h0, h1);
                weights(h1, h1);
            }
            l += sum[0] + sum[1];

            // the 16-key steps of the second product
            auto products = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
                for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<0, 8>(sv + (va ^ (TL::piece_of(t * 32) << 4))), pf[0][0], t);
#pragma unroll
                for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<16, 24>(sv + (va ^ (TL::piece_of(t * 32) << 4))), pf[0][1], t);
#pragma unroll
                for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<32, 40>(sv + (va ^ (TL::piece_of(t * 32) << 4))), pf[1][0], t);
#pragma unroll
                for (int t = 0; t < D / 32; ++t) f(TL::template v_frag<48, 56>(sv + (va ^ (TL::piece_of(t * 32) << 4))), pf[1][1], t);
            };
            if constexpr (!ODD) {
                products([&](const typename O::frag& vf, const typename O::frag& x, int t)
                             __attribute__((always_inline)) { acc[t] = O::mma32(vf, x, acc[t]); });
                sched_mix<T, 4, D / 8, 2, 0, 0>();
            } else {
                products([&](typename O::frag vf, const typename O::frag& x, int t) __attribute__((always_inline)) {
                    O::clean(vf);
                    acc[t] = O::mma32(vf, x, acc[t]);
                });
                const uint64_t seen = sees(a, col_pos, lo, bits_i);
                for (int k = 0; k < KB; ++k) {
                    const int e = ((k >> 3) & 3) * 4 + (k & 3);
                    float x = 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (r == e) x = k < 32 ? w[0][r] : w[1][r];
                    x = __shfl(x, ((k >> 2) & 1) * 32 + l32, 64);
                    if (!((seen >> k) & 1)) continue;
#pragma unroll
                    for (int t = 0; t < D / 32; ++t)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float y = TL::v_one(sv, k, t * 32 + 8 * (r >> 2) + 4 * h2 + (r & 3));
                            if (non_finite(y)) acc[t][r] += x * y;
                        }
                }
            }
            stash(buf ^ 1);
        }
        for (int i = iw; i < i1; ++i) {
            arrive(i, 4);
            stash(((i - i0) & 1) ^ 1);
        }
        if constexpr (!FORM::Q8) landed();
    };
    walk(Int<0>{});
    __syncthreads();
    if (sh[NW + 2]) walk(Int<1>{});

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
            else if (kind == 1) put_raw<4>(W.row_o + rh * D + d, v);
            else put_out<4>(a, row, head, D, d, v, l);
        }
    if (h2 == 0) {
        if (!whole) W.tile_ml[sc] = float2{m, l};
        else if (kind == 1) W.row_ml[rh] = float2{m, l};
        else if (a.lse) a.lse[rh] = lse_of(a, m, l);
    }
}

// A FORM of the kernels says:
//   T, TL, D        the matrix cores' operands, their staged tile, the head dimension
//   Q8              the cache is in 8 bits;  PAGED: a load's keys lie in one page
//   few(), FEW_WAVES, FEW_KEYS, FEW_STAGE   the few-column function, its waves, keys of
//                   a unit, LDS of a wave
//   WAVES           of a SIMD that share its registers

// One launch of a form over own tokens and shared prefixes: a workgroup's
// number says which.
template <class FORM>
__global__ __launch_bounds__(64 * FORM::FEW_WAVES) __attribute__((amdgpu_waves_per_eu(FORM::WAVES)))
void k_attn_few(AttnArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t stage[FORM::FEW_WAVES * FORM::FEW_STAGE];
    __shared__ int sh[FORM::FEW_WAVES + 4];
    const int n0 = a.part[0].few_grid, b = blockIdx.x;
    const int kind = b < n0 ? 0 : 1;
    FORM::few(a, kind, kind ? b - n0 : b, a.part[kind].few_grid, stage, sh);
}
template <class FORM, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(FORM::WAVES)))
void k_attn_tile(AttnArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t stage[4 * ATTN_TILE_KEYS * FORM::TL::RB];   // K and V, twice
    __shared__ int sh[NW + 4];
    const int n1 = a.part[1].tile_grid, b = blockIdx.x;
    const int kind = b < n1 ? 1 : 0;
    attn_tile<FORM, NW>(a, kind, kind ? b : b - n1, stage, sh);
}
// Both forms in one launch, side by side (decode rows behind a shared prefix:
// the tiled form over the prefix, the few-column form over the rows' own
// tokens): their workgroups alternate, eight by eight so that each kind still
// goes round the XCDs, and the one's matrix products run beside the other's
// reads.  256 requests behind eight prefixes of 1000 to 8000 tokens, 64 heads
// on 8: 226 us with the join, 0.72 GB and 5.0e10 flop (3.4 TB/s: a CU holds two
// workgroups of either form, so beside a tile half as many reads are in
// flight as beside another reader).
template <class FORM>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(FORM::WAVES)))
void k_attn_both(AttnArgs a) {
    constexpr int TILES = 4 * ATTN_TILE_KEYS * FORM::TL::RB, FEW = 4 * FORM::FEW_STAGE;
    __shared__ __attribute__((aligned(16))) uint8_t stage[TILES > FEW ? TILES : FEW];
    __shared__ int sh[8];
    const int tiles = a.part[0].tile_grid + a.part[1].tile_grid, n0 = a.part[0].few_grid;
    const int few = n0 + a.part[1].few_grid;
    const int pairs = min(tiles, few) / 8;   // of eight workgroups each
    int b = blockIdx.x;
    bool tile;
    if (b < pairs * 16) {
        tile = (b & 8) == 0;
        b = (b >> 4) * 8 + (b & 7);
    } else {
        b -= pairs * 8;
        tile = b < tiles;
        if (!tile) b -= tiles - pairs * 8;
    }
    if (tile) {
        const int n1 = a.part[1].tile_grid;
        const int kind = b < n1 ? 1 : 0;
        attn_tile<FORM, 4>(a, kind, kind ? b : b - n1, stage, sh);
    } else {
        const int kind = b < n0 ? 0 : 1;
        FORM::few(a, kind, kind ? b - n0 : b, a.part[kind].few_grid, stage, sh);
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
// by_row: all rows (split tiled items).  Otherwise only rows of few-column
// sequences can have partial results, and the waves are numbered by
// (sequence, row in it) so that a prompt's rows cost nothing.
// 32 rows of 32 heads: 9 us with its launch, nearly all of it latency.
template <int D, int FK>
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
    const Prob P = load_prob<true>(a, 0, s, lane);
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
            if (key_tiles<FK>(a, Q, Q.pos0, Q.pos1).n == 0) return r;
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
        if (it.z == 1) return kind == 1 ? one : r;   // a sequence's is in place already
        const int ct = x / a.tile_cols;
        const int j_lo = ct * a.tile_cols / a.share;
        const int j_hi = min(Q.nr - 1, (ct * a.tile_cols + a.tile_cols - 1) / a.share);
        const Before F = prefix_keys<true>(a, kind, q, lane);
        const int n = walk_of<ATTN_TILE_KEYS>(a, F, Q, kind == 0 ? Q.pos0 + j_lo : Q.pos0,
                                              kind == 0 ? Q.pos0 + j_hi : Q.pos1).n();
        r.o = W.tile_o;
        r.ml = W.tile_ml;
        r.n = min(max(1, (n + W.spl - 1) / W.spl), W.tile_grid);
        r.first = r.other = (it.x + (it.y - 1 - ct) * hkv + h) * a.tile_cols + x % a.tile_cols;
        r.step = it.y * hkv * a.tile_cols;
        r.last = W.tile_grid * a.tile_cols - 1;
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
            const float ref = m_new == -kInf ? 0.f : m_new;
            const float f = exp2_fast((M - ref) * c);
            const float w = exp2_fast((x.x - ref) * c);
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
    if (!few || !a.join) {   // whole results are in place already
        if (few && a.part[0].few == 1) return;
        const bool partial = own.n > 0 || (few && key_tiles<FK>(a, P, P.pos0, P.pos1).n == 0);
        write = write && partial;
        if (!__ballot(write)) return;
    } else if (P.pos0 + j < P.key0) {   // more rows than tokens: this row has no place and sees nothing
        own.n = 0;
    } else if (B.n_groups) {
        int g;
        prefix_of(B, s, lane, g);
        if (g < B.n_groups) {
            const Prob G = load_prob<true>(a, 1, g, lane);
            const int gj = row - G.r0;
            if (gj >= 0 && gj < G.nr && G.len > 0) add(parts_of(1, G, g, gj * a.share + (hd - h * a.share)));
        }
    }
    add(own);
    if (!write) return;
    put_out<N>(a, row, head, D, sl * N, v, L);
    if (a.lse && sl == 0) a.lse[rh] = lse_of(a, M, L);
}

// FORM<PAGED, TOGETHER>: the form for pages that hold a load's keys, or less;
// for both forms in one launch, or in two.
template <template <bool, bool> class FORM>
hipError_t launch_form(const AttnArgs& a, bool paged, hipStream_t stream) {
    using T = typename FORM<true, false>::T;
    constexpr int D = FORM<true, false>::D;
    const unsigned tiles = a.part[0].tile_grid + a.part[1].tile_grid, few = a.part[0].few_grid + a.part[1].few_grid;
    if (a.together) {
        if (paged) hipLaunchKernelGGL((k_attn_both<FORM<true, true>>), dim3(tiles + few), dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((k_attn_both<FORM<false, true>>), dim3(tiles + few), dim3(256), 0, stream, a);
    }
    if (tiles && !a.together) {
        const dim3 grid(tiles), block(2 * a.tile_cols);
        bool wide = false;
        if constexpr (kWide<T, D>) {
            wide = a.tile_cols == 256;
            if (wide && paged) hipLaunchKernelGGL((k_attn_tile<FORM<true, false>, 8>), grid, block, 0, stream, a);
            else if (wide) hipLaunchKernelGGL((k_attn_tile<FORM<false, false>, 8>), grid, block, 0, stream, a);
        }
        if (!wide) {
            if (paged) hipLaunchKernelGGL((k_attn_tile<FORM<true, false>, 4>), grid, block, 0, stream, a);
            else hipLaunchKernelGGL((k_attn_tile<FORM<false, false>, 4>), grid, block, 0, stream, a);
        }
    }
    if (few && !a.together) {
        if (paged) hipLaunchKernelGGL((k_attn_few<FORM<true, false>>), dim3(few), dim3(64 * FORM<true, false>::FEW_WAVES), 0, stream, a);
        else hipLaunchKernelGGL((k_attn_few<FORM<false, false>>), dim3(few), dim3(64 * FORM<true, false>::FEW_WAVES), 0, stream, a);
    }
    if (a.need_join) {
        const int by_row = a.part[0].slots;
        const int few_rows = std::max(1, std::min(ATTN_FEW_COLS / a.share, a.part[0].max_rows));
        const int64_t rows = by_row ? a.B.n_rows : (int64_t)a.B.n_seqs * few_rows;
        const dim3 grid((unsigned)ceil_div(rows * ceil_div(a.n_q_heads, 4), 4));
        constexpr int ALONE = FORM<true, false>::FEW_KEYS, BESIDE = FORM<true, true>::FEW_KEYS;
        if (a.together) hipLaunchKernelGGL((k_attn_join<D, BESIDE>), grid, dim3(256), 0, stream, a, by_row, few_rows);
        else hipLaunchKernelGGL((k_attn_join<D, ALONE>), grid, dim3(256), 0, stream, a, by_row, few_rows);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace lora
