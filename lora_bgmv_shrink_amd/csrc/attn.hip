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
    // lanes, 8 or 16 rows in all; fp32: 64 neighbouring bytes of rows 4 apart
    static __device__ __forceinline__ int v_at(int key, int piece) {
        const int x = sizeof(T) == 4 ? ((key >> 2) & 3) << 2 : RB == 128 ? ((key >> 1) & 3) << 1 : (key & 7) << 1;
        return key * RB + ((piece ^ x) << 4);
    }
    static __device__ __forceinline__ int v_elem(int key, int dim) {
        const int byte = dim * (int)sizeof(T);
        return v_at(key, byte >> 4) + (byte & 15);
    }
    // the operand holding, for dimension `dim` (this lane's row of V^T), keys
    // k0 .. k0 + 3 and k1 .. k1 + 3.  l16: lane % 16; dim is dim0 + l16.
    static __device__ __forceinline__ typename Op<T>::frag v_frag(const uint8_t* sv, int k0, int k1, int dim0, int l16) {
        if constexpr (sizeof(T) == 2) {
            const int r = l16 >> 2, dim = dim0 + (l16 & 3) * 4;
            const i16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) i16x4_t*)(sv + v_elem(k0 + r, dim)));
            const i16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) i16x4_t*)(sv + v_elem(k1 + r, dim)));
            return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            f32x8_t f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f[e] = *(const float*)(sv + v_elem(k0 + e, dim0 + l16));
                f[e + 4] = *(const float*)(sv + v_elem(k1 + e, dim0 + l16));
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

template <int KIND>
__device__ inline Prob load_prob(const AttnArgs& a, int p) {
    const KvBatchDev& B = a.B;
    Prob P;
    int r0, r1;
    if (KIND == 0) {
        r0 = B.row_off[p];
        r1 = B.row_off[p + 1];
    } else {
        const int s0 = min(max(B.group_off[p], 0), B.n_seqs), s1 = min(max(B.group_off[p + 1], s0), B.n_seqs);
        r0 = B.row_off[s0];
        r1 = B.row_off[s1];
    }
    P.r0 = min(max(r0, 0), B.n_rows);
    const int nr = min(max(r1, P.r0), B.n_rows) - P.r0;
    P.nr = min(nr, a.part[KIND].max_rows);
    if (KIND == 0) {
        const int n = max(B.kv_len[p], 0);
        P.key0 = 0;
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
        P.key0 = 0;
        P.len = table_keys(min(n, a.part[1].max_len), B.ldpp, a.C.page_shift);
        P.pos0 = n;
        P.pos1 = 0x7ffffffe;
        P.tbl = B.prefix_pages + (int64_t)p * B.ldpp;
    }
    return P;
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
// Few query columns (decode): the keys are split
// ---------------------------------------------------------------------------

// Up to 16 columns (query heads of one key head, times the sequence's rows).
// Reading the visible keys and values bounds it: 4 * 16 columns * D flop per
// 4 D bytes of bf16 keep the matrix cores below a quarter of their rate.
//
// A work unit is 128 keys of one (problem, key head); each of the four waves
// takes 32 of them through LDS of its own (no barrier), with the next unit's
// pieces in flight in registers and the unit after's page numbers behind
// them.  SHARED: the units of all problems are dealt to the workgroups in
// equal runs, whatever the lengths; a run's first and last (problem, head)
// may be partial and go to slots that the join adds.  Otherwise a workgroup
// takes one (problem, head) whole.
template <typename T, int D, int KIND, bool SHARED>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(sizeof(T) * D <= 256 ? 2 : 1)))
void k_attn_few(AttnArgs a) {
    using TL = Tile<T, D>;
    using O = Op<T>;
    constexpr int KW = ATTN_FEW_KEYS / 4;            // keys of a wave's unit
    constexpr int NL = KW * TL::LPR / 64;            // pieces per lane, of K and of V
    constexpr int RPL = 64 / TL::LPR;                // rows one load covers
    constexpr int WB = 2 * KW * TL::RB;              // LDS bytes of a wave
    constexpr int OP = D + 4;                        // fp32 pitch of a wave's O at the end
    static_assert(16 * OP * 4 <= WB, "O fits the wave's stage");
    __shared__ __attribute__((aligned(16))) uint8_t stage[4 * WB];
    __shared__ float sM[4][16], sL[4][16];
    __shared__ int sh[8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int hkv = a.C.n_kv_heads;
    const AttnPart& W = a.part[KIND];
    const int n_prob = KIND == 0 ? a.B.n_seqs : a.B.n_groups;
    uint8_t* sk = stage + wave * WB;
    uint8_t* sv = sk + KW * TL::RB;
    const float c = a.scale * kLog2e;

    // units of a problem, per key head
    auto range_of = [&](const Prob& P) __attribute__((always_inline)) {
        if (P.nr == 0 || P.nr * a.share > ATTN_FEW_COLS) return Range{0, 0, 0};
        return key_tiles<ATTN_FEW_KEYS>(a, P, P.pos0, P.pos1);
    };

    struct At {
        int p, h, i;
        Prob P;
        Range R;
    } L;
    int u, u1;      // this workgroup's units [u, u1)
    int64_t total = 0, wgs = 1;   // all units, and the workgroups that have some
    if (SHARED) {
        auto units = [&](int p) { return range_of(load_prob<KIND>(a, p)).n * hkv; };
        total = sum_units(n_prob, units, tid, sh);
        wgs = min((int64_t)gridDim.x, total);   // no run between a first and a last one is empty
        if (blockIdx.x >= wgs) return;
        u = (int)(blockIdx.x * total / wgs);
        u1 = (int)((blockIdx.x + 1) * total / wgs);
        int base = 0;
        if (!locate(n_prob, u, units, tid, sh, L.p, base)) return;
        L.P = load_prob<KIND>(a, L.p);
        L.R = range_of(L.P);
        const int rem = u - base;
        L.h = rem / L.R.n;
        L.i = rem - L.h * L.R.n;
    } else {
        L.p = blockIdx.x / hkv;
        L.h = blockIdx.x - L.p * hkv;
        L.i = 0;
        L.P = load_prob<KIND>(a, L.p);
        L.R = range_of(L.P);
        u = 0;
        u1 = L.R.n;
        if (L.P.nr == 0 || L.P.nr * a.share > ATTN_FEW_COLS) return;   // no rows, or the tiled kernel's
    }

    // m, l of this lane's column (l: this lane's keys only, until the end)
    float m = -__builtin_inff(), l = 0.f;
    f32x4_t acc[D / 16];
    typename O::frag qf[D / 32];

    // Joins the four waves' results for (p, h) and writes them.
    auto finish = [&](const At& X, bool whole, int slot) __attribute__((always_inline)) {
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (lane < 16) {
            sM[wave][lane] = m;
            sL[wave][lane] = l;
        }
        float* so = (float*)sk;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
            *(float4*)(so + l16 * OP + t * 16 + g4 * 4) = float4{acc[t][0], acc[t][1], acc[t][2], acc[t][3]};
        __syncthreads();
        constexpr int N = D / 16;   // elements per thread, of column tid / 16
        const int col = tid >> 4, d = (tid & 15) * N;
        float M = sM[0][col], f[4], sum = 0.f, v[N];
#pragma unroll
        for (int w = 1; w < 4; ++w) M = fmaxf(M, sM[w][col]);
        const float Mc = M == -__builtin_inff() ? 0.f : M * c;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            f[w] = exp2_fast(sM[w][col] * c - Mc);
            sum += f[w] * sL[w][col];
        }
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            float4 x{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 y = *(const float4*)((const float*)(stage + w * WB) + col * OP + d + e);
                x.x += f[w] * y.x;
                x.y += f[w] * y.y;
                x.z += f[w] * y.z;
                x.w += f[w] * y.w;
            }
            v[e] = x.x;
            v[e + 1] = x.y;
            v[e + 2] = x.z;
            v[e + 3] = x.w;
        }
        if (!whole) {
            put_raw<N>(W.few_o + ((int64_t)slot * 16 + col) * D + d, v);
            if ((tid & 15) == 0) W.few_ml[slot * 16 + col] = float2{M, sum};
        } else if (col < X.P.nr * a.share) {
            const int j = col / a.share;
            const int row = X.P.r0 + j, head = X.h * a.share + (col - j * a.share);
            const int64_t rh = (int64_t)row * a.n_q_heads + head;
            if (a.join) {
                put_raw<N>(W.row_o + rh * D + d, v);
                if ((tid & 15) == 0) W.row_ml[rh] = float2{M, sum};
            } else {
                put_out<N>(a, row, head, D, d, v, sum);
                if (a.lse && (tid & 15) == 0) a.lse[rh] = lse_of(a, M, sum);
            }
        }
        __syncthreads();
    };
    auto clear = [&]() __attribute__((always_inline)) {
        m = -__builtin_inff();
        l = 0.f;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
    if (!SHARED && u1 == 0) {   // rows that see no key
        clear();
        finish(L, true, 0);
        return;
    }

    int col_pos = -1;   // position of this lane's column, -1: no column
    auto begin = [&](const At& X) __attribute__((always_inline)) {
        const int j = l16 / a.share;
        const bool there = l16 < X.P.nr * a.share;
        const T* q = (const T*)a.q + (int64_t)(X.P.r0 + j) * a.ldq + (int64_t)(X.h * a.share + l16 - j * a.share) * D;
#pragma unroll
        for (int s = 0; s < D / 32; ++s) qf[s] = there ? O::load(q + s * 32 + g4 * 8) : O::zero();
        if (KIND == 0) col_pos = there ? X.P.pos0 + j : -1;
        else if (a.window > 0) col_pos = there ? row_position(a, X.P.r0 + j) : -1;
        else col_pos = there ? X.P.pos1 : -1;
        clear();
    };
    // page number of key `lane` of the wave's unit (lanes 0 .. 31), -1: none
    auto load_id = [&](const At& X) __attribute__((always_inline)) {
        const int key = X.R.tile(X.i) * ATTN_FEW_KEYS + wave * KW + lane;
        return lane < KW && key < X.P.len ? X.P.tbl[key >> a.C.page_shift] : -1;
    };
    uint4 rk[NL], rv[NL];
    // requests the wave's pieces of unit X; the answer's bit k says whether
    // any column sees key k (the others are read from page 0 and not used)
    auto load_kv = [&](const At& X, int id) __attribute__((always_inline)) {
        const int base = X.R.tile(X.i) * ATTN_FEW_KEYS + wave * KW;
        const int key = base + lane, at = X.P.key0 + key;
        const bool page_ok = id >= 0 && id < a.C.n_pages;
        bool seen = lane < KW && key < X.P.len && at <= X.P.pos1;
        if (a.window > 0) seen = seen && (at > X.P.pos0 - a.window || at < a.n_sink);
        if (seen && !page_ok && a.status) flag_bad_id(a.status);
        seen = seen && page_ok;
        const uint32_t bits = (uint32_t)__ballot(seen);
        const int page = page_ok ? id : 0;
        const int mask = (1 << a.C.page_shift) - 1;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = j * RPL + lane / TL::LPR;
            const int64_t off = (int64_t)__shfl(page, row, 64) * a.C.page_stride +
                                (int64_t)((base + row) & mask) * a.C.token_stride + (int64_t)X.h * a.C.head_stride +
                                (lane % TL::LPR) * (16 / (int)sizeof(T));
            rk[j] = *(const uint4*)((const T*)a.C.k + off);
            rv[j] = *(const uint4*)((const T*)a.C.v + off);
        }
        return bits;
    };
    auto store_kv = [&](uint32_t bits) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = j * RPL + lane / TL::LPR, piece = lane % TL::LPR;
            *(uint4*)(sk + TL::k_at(row, piece)) = rk[j];
            if (bits != 0xffffffffu && !((bits >> row) & 1)) rv[j] = uint4{0u, 0u, 0u, 0u};
            *(uint4*)(sv + TL::v_at(row, piece)) = rv[j];
        }
    };
    auto compute = [&](const At& X, uint32_t bits) __attribute__((always_inline)) {
        f32x4_t s[2] = {f32x4_t{0.f, 0.f, 0.f, 0.f}, f32x4_t{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) {
            s[0] = O::mma16(TL::k_frag(sk, l16, ks * 32 + g4 * 8), qf[ks], s[0]);
            s[1] = O::mma16(TL::k_frag(sk, 16 + l16, ks * 32 + g4 * 8), qf[ks], s[1]);
        }
        // element r of s[t]: key 16 t + 4 g4 + r, this lane's column
        const int lo = X.P.key0 + X.R.tile(X.i) * ATTN_FEW_KEYS + wave * KW;
        const bool all_see = lo + KW - 1 <= X.P.pos0 && (a.window == 0 || lo > X.P.pos1 - a.window);
        const bool masked = bits != 0xffffffffu || !all_see;
        auto sees = [&](int k) __attribute__((always_inline)) {
            const int at = lo + k;
            return ((bits >> k) & 1) && at <= col_pos && (a.window == 0 || at > col_pos - a.window || at < a.n_sink);
        };
        if (masked) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!sees(16 * t + 4 * g4 + r)) s[t][r] = -__builtin_inff();
        }
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float m_new = fmaxf(m, top);
        const float mc = m_new == -__builtin_inff() ? 0.f : m_new * c;
        if (__ballot(m_new != m)) {
            const float f = exp2_fast(m * c - mc);
            l *= f;
#pragma unroll
            for (int t = 0; t < D / 16; ++t) acc[t] *= f;
            m = m_new;
        }
        f32x8_t p;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            p[r] = exp2_fast(s[0][r] * c - mc);
            p[4 + r] = exp2_fast(s[1][r] * c - mc);
        }
        l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
        const typename O::frag pf = O::round(p);
        // A key that some rows see and others do not may hold infinities or
        // NaN: 0 times those must not reach the rows that do not see it.
        const bool mixed = !all_see && X.P.nr > 1;
        bool odd = false;
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            typename O::frag vf = TL::v_frag(sv, 4 * g4, 16 + 4 * g4, t * 16, l16);
            if (mixed) odd |= O::clean(vf);
            acc[t] = O::mma16(vf, pf, acc[t]);
        }
        if (mixed && __ballot(odd)) {
            for (int k = 0; k < KW; ++k) {
                const int r = k & 3, t = k >> 4;
                float w = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e == t * 4 + r) w = p[e];
                w = __shfl(w, ((k >> 2) & 3) * 16 + l16, 64);
                if (!sees(k)) continue;
#pragma unroll
                for (int q = 0; q < D / 16; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = TL::v_one(sv, k, q * 16 + g4 * 4 + e);
                        if (non_finite(x)) acc[q][e] += w * x;
                    }
            }
        }
    };
    auto step = [&](At& X) __attribute__((always_inline)) {
        if (++X.i < X.R.n) return;
        X.i = 0;
        if (++X.h < hkv) return;
        X.h = 0;
        do {   // in bounds: called only while units remain
            X.P = load_prob<KIND>(a, ++X.p);
            X.R = range_of(X.P);
        } while (X.R.n == 0 && X.p + 1 < n_prob);
    };

    // C: the unit worked on, L: the unit whose pieces are requested, N: the
    // one whose page numbers are
    const int first = u;
    At C = L;
    uint32_t bits = load_kv(L, load_id(L));
    int id = -1;
    if (u + 1 < u1) {
        step(L);
        id = load_id(L);
    }
    begin(C);
    while (true) {
        store_kv(bits);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const uint32_t bits_c = bits;
        At N = L;
        if (u + 1 < u1) {
            bits = load_kv(L, id);
            if (u + 2 < u1) {
                step(N);
                id = load_id(N);
            }
        }
        if (bits_c) compute(C, bits_c);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const bool last = u + 1 == u1;
        if (last || C.i + 1 == C.R.n) {
            bool whole = true;
            int slot = 0;
            if (SHARED) {
                const int ra = u - C.i, rb = ra + C.R.n;   // the units of (p, h)
                const bool starts = ra >= first;
                whole = starts && rb <= u1;
                slot = 2 * blockIdx.x + (starts ? 1 : 0);
                if (starts && tid == 0) {
                    const int b1 = (int)((rb * wgs - 1) / total);
                    W.rec[C.p * hkv + C.h] = int2{(int)blockIdx.x, b1};
                }
            }
            finish(C, whole, slot);
            if (last) break;
            begin(L);
        }
        C = L;
        L = N;
        ++u;
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
template <typename T, int D, int KIND>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(sizeof(T) * D <= 256 ? 2 : 1)))
void k_attn_tile(AttnArgs a) {
    using TL = Tile<T, D>;
    using O = Op<T>;
    constexpr int KB = ATTN_TILE_KEYS, TC = ATTN_TILE_COLS;
    constexpr int NL = KB * TL::LPR / 256;     // pieces per thread, of K and of V
    constexpr int RPL = 256 / TL::LPR;         // rows one load of the workgroup covers
    constexpr int TB = KB * TL::RB;            // bytes of a staged tile
    __shared__ __attribute__((aligned(16))) uint8_t stage[2][2][TB];
    __shared__ int sh[8];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l32 = lane & 31, h2 = lane >> 5, l16 = lane & 15, d16 = (lane >> 4) & 1;
    const int hkv = a.C.n_kv_heads;
    const AttnPart& W = a.part[KIND];
    const int n_prob = KIND == 0 ? a.B.n_seqs : a.B.n_groups;
    const float c = a.scale * kLog2e;
    const float kInf = __builtin_inff();

    auto splits_of = [&](const Prob& P, int& nct) __attribute__((always_inline)) {
        const int64_t cols = (int64_t)P.nr * a.share;
        nct = cols > ATTN_FEW_COLS ? (int)((cols + TC - 1) / TC) : 0;
        const int n = key_tiles<KB>(a, P, P.pos0, P.pos1).n;
        return n > W.spl ? (n + W.spl - 1) / W.spl : 1;
    };
    int p, base;
    if (!locate(n_prob, blockIdx.x,
                [&](int q) {
                    int nct;
                    const int ns = splits_of(load_prob<KIND>(a, q), nct);
                    return nct * ns * hkv;
                },
                tid, sh, p, base))
        return;
    const Prob P = load_prob<KIND>(a, p);
    int nct;
    const int nsplit = splits_of(P, nct);
    int rem = blockIdx.x - base;
    const int h = rem % hkv;
    rem /= hkv;
    const int split = rem / nct;
    const int ct = nct - 1 - rem % nct;
    if (rem == 0 && h == 0 && tid == 0 && W.slots) W.item[p] = int4{base, nct, nsplit, 0};

    // the workgroup's rows, its key tiles and this split's run of them
    const int j_lo = ct * TC / a.share, j_hi = min(P.nr - 1, (ct * TC + TC - 1) / a.share);
    const int wg_lo = KIND == 0 ? P.pos0 + j_lo : P.pos0, wg_hi = KIND == 0 ? P.pos0 + j_hi : P.pos1;
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
    if (there) col_pos = KIND == 0 ? P.pos0 + j : a.window > 0 ? row_position(a, row) : P.pos1;
    // least and largest position of the wave's columns
    const int wv_lo = KIND == 0 ? P.pos0 + (ct * TC + wave * 32) / a.share : P.pos0;
    const int wv_hi = KIND == 0 ? min(P.pos1, P.pos0 + (ct * TC + wave * 32 + 31) / a.share) : P.pos1;

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
    uint4 rk[NL], rv[NL];
    auto load_kv = [&](int i, int id) __attribute__((always_inline)) {
        const int base_k = R.tile(i) * KB;
        const int key = base_k + lane, at = P.key0 + key;
        const bool page_ok = id >= 0 && id < a.C.n_pages;
        bool seen = key < P.len && at <= wg_hi;
        if (a.window > 0) seen = seen && (at > wg_lo - a.window || at < a.n_sink);
        if (seen && !page_ok && a.status) flag_bad_id(a.status);
        seen = seen && page_ok;
        const uint64_t bits = __ballot(seen);
        const int page = page_ok ? id : 0;
        const int mask = (1 << a.C.page_shift) - 1;
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const int r = n * RPL + tid / TL::LPR;
            const int64_t off = (int64_t)__shfl(page, r, 64) * a.C.page_stride +
                                (int64_t)((base_k + r) & mask) * a.C.token_stride + (int64_t)h * a.C.head_stride +
                                (tid % TL::LPR) * (16 / (int)sizeof(T));
            rk[n] = *(const uint4*)((const T*)a.C.k + off);
            rv[n] = *(const uint4*)((const T*)a.C.v + off);
        }
        return bits;
    };
    auto store_kv = [&](int buf, uint64_t bits) __attribute__((always_inline)) {
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const int r = n * RPL + tid / TL::LPR, piece = tid % TL::LPR;
            *(uint4*)(stage[buf][0] + TL::k_at(r, piece)) = rk[n];
            if (bits != ~0ull && !((bits >> r) & 1)) rv[n] = uint4{0u, 0u, 0u, 0u};
            *(uint4*)(stage[buf][1] + TL::v_at(r, piece)) = rv[n];
        }
    };

    uint64_t bits = 0;
    int id = -1;
    if (i0 < i1) {
        bits = load_kv(i0, load_id(i0));
        if (i0 + 1 < i1) id = load_id(i0 + 1);
    }
    for (int i = i0; i < i1; ++i) {
        const int buf = (i - i0) & 1;
        store_kv(buf, bits);
        __syncthreads();
        const uint64_t bits_c = bits;
        if (i + 1 < i1) {
            bits = load_kv(i + 1, id);
            if (i + 2 < i1) id = load_id(i + 2);
        }
        const int lo = P.key0 + R.tile(i) * KB;
        if (!wave_there || lo > wv_hi) continue;
        const uint8_t* sk = stage[buf][0];
        const uint8_t* sv = stage[buf][1];
        // element r of s[kb]: key 32 kb + 8 (r / 4) + 4 h2 + r % 4
        f32x16_t s[2];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kb][r] = 0.f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                s[kb] = O::mma32(TL::k_frag(sk, kb * 32 + l32, ks * 16 + h2 * 8), qf[ks], s[kb]);
        }
        const bool all_see = lo + KB - 1 <= wv_lo && (a.window == 0 || lo > wv_hi - a.window);
        auto sees = [&](int k) __attribute__((always_inline)) {
            const int at = lo + k;
            return ((bits_c >> k) & 1) && at <= col_pos && (a.window == 0 || at > col_pos - a.window || at < a.n_sink);
        };
        if (bits_c != ~0ull || !all_see) {
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    if (!sees(32 * kb + 8 * (r >> 2) + 4 * h2 + (r & 3))) s[kb][r] = -kInf;
        }
        float top = s[0][0];
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, fmaxf(s[0][r], s[1][r]));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float m_new = fmaxf(m, top);
        const float mc = m_new == -kInf ? 0.f : m_new * c;
        if (__ballot(m_new != m)) {
            const float f = exp2_fast(m * c - mc);
            l *= f;
#pragma unroll
            for (int t = 0; t < D / 32; ++t) acc[t] *= f;
            m = m_new;
        }
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
        const int k4 = 4 * h2;
        if (all_see) {
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        acc[t] = O::mma32(TL::v_frag(sv, kb * 32 + x * 16 + k4, kb * 32 + x * 16 + 8 + k4,
                                                     t * 32 + d16 * 16, l16),
                                          pf[kb][x], acc[t]);
        } else {
            // a key that some columns see and others do not may hold
            // infinities or NaN: 0 times those must not reach the others
            bool odd = false;
#pragma unroll
            for (int t = 0; t < D / 32; ++t)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        typename O::frag vf = TL::v_frag(sv, kb * 32 + x * 16 + k4, kb * 32 + x * 16 + 8 + k4,
                                                         t * 32 + d16 * 16, l16);
                        odd |= O::clean(vf);
                        acc[t] = O::mma32(vf, pf[kb][x], acc[t]);
                    }
            if (__ballot(odd)) {
                for (int k = 0; k < KB; ++k) {
                    const int e = ((k >> 3) & 3) * 4 + (k & 3);
                    float w = 0.f;
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if (r == e) w = k < 32 ? s[0][r] : s[1][r];
                    w = __shfl(w, ((k >> 2) & 1) * 32 + l32, 64);
                    if (!sees(k)) continue;
#pragma unroll
                    for (int t = 0; t < D / 32; ++t)
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float x = TL::v_one(sv, k, t * 32 + 8 * (r >> 2) + k4 + (r & 3));
                            if (non_finite(x)) acc[t][r] += w * x;
                        }
                }
            }
        }
    }

    l += __shfl_xor(l, 32, 64);
    if (!there) return;
    const bool whole = nsplit == 1;
    const int64_t rh = (int64_t)row * a.n_q_heads + head;
    const int64_t sc = (int64_t)blockIdx.x * TC + wave * 32 + l32;
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

// ---------------------------------------------------------------------------
// Join
// ---------------------------------------------------------------------------

// A wave per (row, query head): adds the partial results of its own keys and
// of the shared prefix, each scaled to the largest score of all, in their
// fixed order.  Reads every partial once.
template <int D>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63;
    const int64_t rh = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const KvBatchDev& B = a.B;
    if (rh >= (int64_t)B.n_rows * a.n_q_heads) return;
    const int row = (int)(rh / a.n_q_heads), head = (int)(rh - (int64_t)row * a.n_q_heads);
    const int h = head / a.share, hkv = a.C.n_kv_heads;
    const int s = wave_find_run(B.row_off, B.n_seqs, row, lane);
    if (s >= B.n_seqs || row < B.row_off[0]) return;
    const float c = a.scale * kLog2e;
    float M = -__builtin_inff(), L = 0.f, v[N];
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = 0.f;

    // adds n partial results, the i-th at o + at(i) * D and ml[at(i)]; `most`
    // bounds the places, whatever the batch's offsets say
    auto add = [&](int n, int64_t most, const float* o, const float2* ml, auto place) __attribute__((always_inline)) {
        auto at = [&](int i) { return max((int64_t)0, min(place(i), most - 1)); };
        for (int i0 = 0; i0 < n; i0 += 64) {
            const int here = min(64, n - i0);
            const float2 x = lane < here ? ml[at(i0 + lane)] : float2{-__builtin_inff(), 0.f};
            float top = x.x;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
            const float m_new = fmaxf(M, top);
            const float mc = m_new == -__builtin_inff() ? 0.f : m_new * c;
            const float f = exp2_fast(M * c - mc);
            L *= f;
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] *= f;
            M = m_new;
            const float w = exp2_fast(x.x * c - mc);
            float sum = lane < here ? w * x.y : 0.f;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
            L += sum;
#pragma unroll 4
            for (int i = 0; i < here; ++i) {
                const float wi = __shfl(w, i, 64);
                const float* src = o + at(i0 + i) * D + lane * N;
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] += wi * src[e];
            }
        }
    };
    auto add_part = [&](const AttnPart& W, const Prob& P, int p, int col, int pos_lo, int pos_hi) __attribute__((always_inline)) {
        const bool few = (int64_t)P.nr * a.share <= ATTN_FEW_COLS;
        if (few) {
            if (P.len <= 0) return;
            if (W.few == 1) {
                add(1, rh + 1, W.row_o, W.row_ml, [&](int) { return rh; });
                return;
            }
            if (key_tiles<ATTN_FEW_KEYS>(a, P, P.pos0, P.pos1).n == 0) return;
            const int2 b = W.rec[p * hkv + h];
            if (b.x == b.y) {
                if (a.join) add(1, rh + 1, W.row_o, W.row_ml, [&](int) { return rh; });
                return;
            }
            add(min(b.y - b.x + 1, ATTN_FEW_WGS), (int64_t)2 * ATTN_FEW_WGS * 16, W.few_o, W.few_ml, [&](int i) {
                return (int64_t)(i == 0 ? 2 * b.x + 1 : 2 * (b.x + i)) * 16 + col;
            });
        } else {
            const int ct = col / ATTN_TILE_COLS;
            const int n = key_tiles<ATTN_TILE_KEYS>(a, P, pos_lo, pos_hi).n;
            const int4 it = W.slots ? W.item[p] : int4{0, 1, 1, 0};
            if (it.z == 1) {
                if (a.join) add(1, rh + 1, W.row_o, W.row_ml, [&](int) { return rh; });
                return;
            }
            const int used = max(1, (n + W.spl - 1) / W.spl);
            add(min(used, W.tile_grid), (int64_t)W.tile_grid * ATTN_TILE_COLS, W.tile_o, W.tile_ml, [&](int i) {
                return (int64_t)(it.x + (i * it.y + (it.y - 1 - ct)) * hkv + h) * ATTN_TILE_COLS + (col % ATTN_TILE_COLS);
            });
        }
    };

    const Prob P = load_prob<0>(a, s);
    const int j = row - P.r0;
    if (j < 0 || j >= P.nr) return;
    const int col = j * a.share + (head - h * a.share);
    // without a prefix, whole results are in place already
    if (!a.join) {
        const bool few = (int64_t)P.nr * a.share <= ATTN_FEW_COLS;
        if (few) {
            if (a.part[0].few == 1) return;
            if (key_tiles<ATTN_FEW_KEYS>(a, P, P.pos0, P.pos1).n > 0) {
                const int2 b = a.part[0].rec[s * hkv + h];
                if (b.x == b.y) return;
            }
        } else if (!a.part[0].slots || a.part[0].item[s].z == 1) {
            return;
        }
    }
    const bool none = P.pos0 + j < P.key0;   // more rows than tokens: this row has no place
    if (!none) {
        const int ct = col / ATTN_TILE_COLS;
        const int j_lo = ct * ATTN_TILE_COLS / a.share;
        const int j_hi = min(P.nr - 1, (ct * ATTN_TILE_COLS + ATTN_TILE_COLS - 1) / a.share);
        if (a.join && B.n_groups) {
            const int g = wave_find_run(B.group_off, B.n_groups, s, lane);
            if (g < B.n_groups) {
                const Prob G = load_prob<1>(a, g);
                const int gj = row - G.r0;
                if (gj >= 0 && gj < G.nr)
                    add_part(a.part[1], G, g, gj * a.share + (head - h * a.share), G.pos0, G.pos1);
            }
        }
        add_part(a.part[0], P, s, col, P.pos0 + j_lo, P.pos0 + j_hi);
    }
    put_out<N>(a, row, head, D, lane * N, v, L);
    if (a.lse && lane == 0) a.lse[rh] = lse_of(a, M, L);
}

template <typename T, int D, int KIND>
void launch_kind(const AttnArgs& a, hipStream_t stream) {
    const AttnPart& W = a.part[KIND];
    const int n_prob = KIND == 0 ? a.B.n_seqs : a.B.n_groups;
    if (W.few == 1)
        hipLaunchKernelGGL((k_attn_few<T, D, KIND, false>), dim3((unsigned)(n_prob * a.C.n_kv_heads)), dim3(256), 0,
                           stream, a);
    else if (W.few == 2)
        hipLaunchKernelGGL((k_attn_few<T, D, KIND, true>), dim3(ATTN_FEW_WGS), dim3(256), 0, stream, a);
    if (W.tile) hipLaunchKernelGGL((k_attn_tile<T, D, KIND>), dim3((unsigned)W.tile_grid), dim3(256), 0, stream, a);
}

template <typename T, int D>
hipError_t launch_d(const AttnArgs& a, hipStream_t stream) {
    if (a.join) launch_kind<T, D, 1>(a, stream);
    launch_kind<T, D, 0>(a, stream);
    if (a.need_join) {
        const int64_t waves = (int64_t)a.B.n_rows * a.n_q_heads;
        hipLaunchKernelGGL((k_attn_join<D>), dim3((unsigned)ceil_div(waves, 4)), dim3(256), 0, stream, a);
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
            if (W.few == 2) a.need_join = 1;
            if (ceil_div(max_len[k], ATTN_FEW_KEYS) > 2) {
                P.off[k][0] = take((size_t)n_prob[k] * hkv * sizeof(int2));
                P.off[k][1] = take((size_t)2 * ATTN_FEW_WGS * 16 * head_dim * 4);
                P.off[k][2] = take((size_t)2 * ATTN_FEW_WGS * 16 * sizeof(float2));
            }
        }
        if ((int64_t)max_rows[k] * a.share > ATTN_FEW_COLS) {
            W.tile = 1;
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
