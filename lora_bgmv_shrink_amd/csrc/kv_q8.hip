// Appending a step's keys and values to a cache in 8 bits:
//
//     e = the least power of two with max |x| <= 448 * 2^e over the block's new tokens
//         (not below the block's power so far, where it holds earlier tokens)
//     stored: e4m3(x / 2^e)
//
// x the rotated key or the value.  A number has 4 significant bits, so a
// rotation rounded before it is rounded again may end on the wrong side of a
// tie: a key's two products are made in 64 bits (of two fp32 numbers each is
// exact there), and their sum, with what 64 bits leave of it where that may
// count, is brought to fp32 by rounding to odd, which keeps what the last
// rounding has to know.  A power of two as scale costs no rounding of its own,
// keeps the earlier tokens' bits when it grows (but below 2^-6 of it), and is
// what the matrix cores' widening takes.
//
// Queries go the way of the other caches, rounded to bf16.
//
// Bytes bound it where there are many: 20304 rows of 64 heads on 8 of 128, bf16,
// 642 MB in 130 us (4.9 TB/s, nearly a plain copy's rate; keys and values alone 38 us,
// 12 of them the 64-bit rotation, which hides behind the queries' bytes).  2112
// rows of 32 heads on 8, fp32, 74 MB in 17.2 us; a decode step of 32 rows 5 us,
// the chain row -> sequence -> page -> scale -> store.
#include "kv_append.hpp"

namespace lora {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr int KQ_TOKENS = 1024;   // elements of a wave's pass: 1024 / D tokens of a head

// x in fp32, the last bit set where that is not all of x (so that a later
// rounding to fewer bits goes as it would from x); past fp32's range its largest
__device__ __forceinline__ float to_odd(double x) {
    const float f = (float)x;
    const double b = (double)f;
    int bits = __float_as_int(f);
    if (b != x && !(bits & 1)) bits += fabs(b) < fabs(x) ? 1 : -1;
    return __int_as_float(bits);
}
// Ties of two numbers, and the border of two scales, have 5 significant bits at
// the most.  Where to_odd(a + b) has no more, the sum in 64 bits is that
// number, and a + b may be next to it by less than 64 bits tell.
__device__ __forceinline__ uint32_t low_bits(float y) { return __float_as_uint(y) << 13; }
// On which side of the sum in 64 bits a + b lies: 1 the larger magnitude's, 2
// the smaller one's, 0: it is that sum.
__device__ __forceinline__ uint32_t side_of(double a, double b) {
    const double x = a + b, t = x - a, rest = (a - (x - t)) + (b - t);   // NaN where x is infinite
    return rest < 0. || rest > 0. ? ((rest > 0.) == (x > 0.) ? 1u : 2u) : 0u;
}
// y = to_odd(a + b), its last bit set for that side
__device__ __forceinline__ float to_side(float y, uint32_t side) {
    return __int_as_float(__float_as_int(y) + (low_bits(y) == 0 ? (int)(side & 1) - (int)(side >> 1 & 1) : 0));
}
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }

// the least e with top <= 448 * 2^e = 1.75 * 2^(e + 8)
__device__ __forceinline__ int power_for(float top) {
    const uint32_t b = __float_as_uint(top);
    return min(max((int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0), Q8_LEAST), Q8_MOST);
}
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// eight values times `by` as e4m3; finite ones past 448 become that
__device__ __forceinline__ uint2 narrow8(const float (&f)[8], float by) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float y = f[e] * by;
        t[e] = finite(f[e]) ? __builtin_amdgcn_fmed3f(y, -448.f, 448.f) : __builtin_nanf("");
    }
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
    return uint2{(uint32_t)lo, (uint32_t)hi};
}
__device__ __forceinline__ uint2 again8(uint2 v, float by) {   // by <= 1
    f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(v.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(v.x, true);
    f32x2_t c = __builtin_amdgcn_cvt_pk_f32_fp8(v.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(v.y, true);
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a.x * by, a.y * by, 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(b.x * by, b.y * by, lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(c.x * by, c.y * by, 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(d.x * by, d.y * by, hi, true);
    return uint2{(uint32_t)lo, (uint32_t)hi};
}

// Blocks of the step are numbered without a pass over the sequences: sequence
// s has room for its blocks from block_at(s) on, (rows before it) / block_size
// and `per` more for each sequence before it.  n rows lie in n / block_size + 2
// blocks at most, a single one in one: `per` is 2, or 1 where the batch's bound
// is a row a sequence (2 there: 256 rows 13.1 us, so 11.6).
__device__ __forceinline__ int block_at(const AppendArgs& a, int s, int first_row) {
    return (first_row >> a.S.block_shift) + a.S.per * s;
}

// NP passes of a wave hold its part of a block; WPU waves share one.
template <typename TI, int D, int NP, int WPU>
__device__ __forceinline__ void append_block(const AppendArgs& a, int64_t unit, int part, float* sh) {
    constexpr int LPT = D / 16;         // lanes of a token, 16 elements each
    constexpr int TPP = 64 / LPT;       // tokens of a pass
    const int lane = threadIdx.x & 63;
    const KvBatchDev& B = a.B;
    const int n_heads = a.S.n_kv_heads;
    const int at = (int)(unit / (2 * n_heads)), hv = (int)(unit - (int64_t)at * 2 * n_heads);
    const bool is_v = hv >= n_heads;
    const int h = is_v ? hv - n_heads : hv;

    // the sequence whose blocks `at` is among
    int s, b0, b1, len;
    if (!wave_find_seq(B, at, lane, [&](int i, int off) { return block_at(a, i, off); }, s, b0, b1, len)) return;
    const int r0 = min(max(b0, 0), B.n_rows), r1 = min(max(b1, r0), B.n_rows);
    const int first = len - (r1 - r0);   // tokens first .. len - 1 are new
    // more rows than tokens: the first ones have no place (nor any, without tokens)
    if (r1 > r0 && first < 0 && lane == 0 && part == 0 && a.status) flag_bad_id(a.status);
    const int lo0 = max(first, 0);
    const int t0 = ((lo0 >> a.S.block_shift) + (at - block_at(a, s, b0))) << a.S.block_shift;
    if (r1 == r0 || at < block_at(a, s, b0) || t0 < 0 || t0 >= len) return;
    // more rows than the bound: the last ones have no room
    if (at + 1 == block_at(a, s + 1, b1) && len - t0 > 1 << a.S.block_shift && lane == 0 && part == 0 && a.status)
        flag_bad_id(a.status);
    int before = 0;
    if (B.n_groups) {
        const int g = wave_find_run(B.group_off, B.n_groups, s, lane);
        if (g < B.n_groups) before = max(B.prefix_len[g], 0);
    }
    const int lo = max(t0, lo0), all = min(t0 + (1 << a.S.block_shift), len);
    const int hi = a.cos ? (int)min((int64_t)all, (int64_t)a.n_pos - before) : all;

    // this lane's place in every token: two pieces of 8, partners of one
    // another where heads are rotated in halves
    const int c = lane & (LPT - 1);
    const bool turn = !is_v && a.cos && c * 16 < 2 * a.half, halves = turn && !a.interleaved;
    const int e0 = halves ? c * 8 : c * 16, e1 = halves ? e0 + a.half : e0 + 8;
    const TI* from = is_v ? (const TI*)a.v + h * D : (const TI*)a.k + h * D;
    const int64_t ld = is_v ? a.ldv : a.ldk;
    const int token0 = part * NP * TPP + lane / LPT;   // of the block; a pass further on, TPP more

    // the rows are requested before the place in the cache is looked up
    Eight<TI> x0[NP], x1[NP];
    constexpr bool EARLY = NP <= 2;   // and so are their angles, where that leaves registers
    Eight<float> cs[EARLY ? NP : 1], sn[EARLY ? NP : 1];
    auto angles = [&](int t, int i) __attribute__((always_inline)) {
        cs[i].load(a.cos + (int64_t)(before + t) * a.ldr + c * 8);
        sn[i].load(a.sin + (int64_t)(before + t) * a.ldr + c * 8);
    };
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int t = t0 + token0 + p * TPP;
        if (t >= lo && t < hi) {
            const TI* src = from + (int64_t)(r0 + (t - first)) * ld;
            x0[p].load(src + e0);
            x1[p].load(src + e1);
            if (EARLY && turn) angles(t, p);
        }
    }

    const int pg = t0 >> a.C.page_shift;
    const int page = pg < B.ldp ? B.pages[(int64_t)s * B.ldp + pg] : -1;
    const bool page_ok = page >= 0 && page < a.C.n_pages;
    if ((!page_ok || hi < all) && lane == 0 && part == 0 && a.status) flag_bad_id(a.status);
    if (!page_ok || hi <= lo) return;
    const int cell = t0 & ((1 << a.C.page_shift) - 1);
    uint8_t* to = (uint8_t*)(is_v ? a.C.v : a.C.k) + (int64_t)page * a.C.page_stride + (int64_t)h * a.C.head_stride +
                  (int64_t)cell * a.C.token_stride;
    float* scale = (is_v ? a.S.v_scale : a.S.k_scale) + (int64_t)page * a.S.page_stride +
                   (int64_t)(cell >> a.S.block_shift) * a.S.block_stride + (int64_t)h * a.S.head_stride;
    const bool kept = first > t0;   // earlier tokens share the block
    const int was = kept ? min(max((int)((__float_as_uint(*scale) >> 23) & 255) - 127, Q8_LEAST), Q8_MOST) : 0;

    float y0[NP][8], y1[NP][8], top = 0.f;
    uint32_t low = ~0u;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int t = t0 + token0 + p * TPP;
        if (!(t >= lo && t < hi)) continue;
        if (turn) {
            const int i = EARLY ? p : 0;
            if (!EARLY) angles(t, 0);
            auto pair = [&](float p, float q, int e, float& u, float& w) __attribute__((always_inline)) {
                const double P = p, Q = q, C = cs[i].get(e), S = sn[i].get(e);
                u = to_odd(P * C - Q * S);
                w = to_odd(P * S + Q * C);
                low = min(low, min(low_bits(u), low_bits(w)));
            };
            if (halves) {
#pragma unroll
                for (int e = 0; e < 8; ++e) pair(x0[p].get(e), x1[p].get(e), e, y0[p][e], y1[p][e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    pair(x0[p].get(2 * e), x0[p].get(2 * e + 1), e, y0[p][2 * e], y0[p][2 * e + 1]);
                    pair(x1[p].get(2 * e), x1[p].get(2 * e + 1), e + 4, y1[p][2 * e], y1[p][2 * e + 1]);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y0[p][e] = x0[p].get(e);
                y1[p][e] = x1[p].get(e);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            top = fmaxf(top, finite(y0[p][e]) ? fabsf(y0[p][e]) : 0.f);
            top = fmaxf(top, finite(y1[p][e]) ? fabsf(y1[p][e]) : 0.f);
        }
    }
    if (low == 0) {
        // A pair at a time, from memory: nothing is held for it (with whole sums
        // in any case 2112 fp32 rows take 20.6 us, so 17.2).  top only grows:
        // for a sum just below a border the border's own scale is right too.
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int t = t0 + token0 + p * TPP;
            if (!(t >= lo && t < hi)) continue;
            const TI* src = from + (int64_t)(r0 + (t - first)) * ld;
            const int64_t angle = (int64_t)(before + t) * a.ldr + c * 8;
            uint32_t sides[2] = {0, 0};
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const int ea = halves ? e0 + k : e0 + 2 * k, eb = halves ? e1 + k : ea + 1;
                const double P = to_f32(src[ea]), Q = to_f32(src[eb]), C = a.cos[angle + k], S = a.sin[angle + k];
                sides[0] |= side_of(P * C, -(Q * S)) << (2 * k);
                sides[1] |= side_of(P * S, Q * C) << (2 * k);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                y0[p][e] = to_side(y0[p][e], halves ? sides[0] >> (2 * e) : sides[e & 1] >> (e & 6));
                y1[p][e] = to_side(y1[p][e], halves ? sides[1] >> (2 * e) : sides[e & 1] >> (8 + (e & 6)));
                if (finite(y0[p][e])) top = fmaxf(top, fabsf(y0[p][e]));
                if (finite(y1[p][e])) top = fmaxf(top, fabsf(y1[p][e]));
            }
        }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    if constexpr (WPU > 1) {   // every wave of the workgroup is here: they share the unit
        if (lane == 0) sh[part] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WPU; ++w) top = fmaxf(top, sh[w]);
    }
    int e = power_for(top);
    if (kept) e = max(e, was);
    const float by = two_to(-e);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int t = t0 + token0 + p * TPP;
        if (t >= lo && t < hi) {
            uint8_t* dst = to + (int64_t)(t - t0) * a.C.token_stride;
            *(uint2*)(dst + e0) = narrow8(y0[p], by);
            *(uint2*)(dst + e1) = narrow8(y1[p], by);
        }
    }
    if (kept && e == was) return;
    if (lane == 0 && part == 0) *scale = two_to(e);
    if (!kept) return;
    const float less = two_to(max(was - e, -60));   // far enough below for every e4m3 number to become 0
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int t = t0 + token0 + p * TPP;
        if (t < first && t < t0 + (1 << a.S.block_shift)) {
            uint2* dst = (uint2*)(to + (int64_t)(t - t0) * a.C.token_stride + c * 16);
            dst[0] = again8(dst[0], less);
            dst[1] = again8(dst[1], less);
        }
    }
}

// The blocks' workgroups, whose chains are the longer ones, then the queries'.
template <typename TI, int D, int NP, int WPU>
__global__ __launch_bounds__(KA_WAVES * 64) void k_kv_append_q8(AppendArgs a, int it, int q_runs) {
    __shared__ float sh[KA_WAVES];
    const int blocks = (int)((a.S.units * WPU + KA_WAVES - 1) / KA_WAVES);
    const int b = blockIdx.x;
    if (b >= blocks) {
        append_row<TI, bf16, D, true>(a, it, (b - blocks) / q_runs, (b - blocks) % q_runs);
        return;
    }
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (WPU == 1) {
        const int64_t unit = (int64_t)b * KA_WAVES + wave;
        if (unit < a.S.units) append_block<TI, D, NP, 1>(a, unit, 0, sh);
    } else {
        append_block<TI, D, NP, WPU>(a, b, wave, sh);
    }
}

template <typename TI, int D>
hipError_t launch_d(AppendArgs a, hipStream_t stream) {
    // whole keys and values of the heads, but for the row's part
    const int64_t q_rows = a.n_q_heads ? ceil_div(a.B.n_rows, KA_WAVES) : 0;
    const int chunks = (int)ceil_div((int64_t)a.n_q_heads * (D / 16), 64);
    const int it = (int)std::max<int64_t>(1, std::min<int64_t>(chunks, (int64_t)a.B.n_rows * chunks / 2048));
    const int q_runs = a.n_q_heads ? (int)ceil_div(chunks, it) : 1;
    // A wave takes a block of up to four passes by itself: four waves to such a
    // block have four times the lookups (2112 rows in blocks of 32 of 128: 23.5
    // us, one wave 17.3).  From eight passes on it would hold no registers for
    // others (blocks of 64: 128 us, one wave 132).
    const int passes = (int)ceil_div((int64_t)D << a.S.block_shift, KQ_TOKENS);
    const int wpu = passes <= 4 ? 1 : KA_WAVES;
    const int64_t grid = q_rows * q_runs + ceil_div(a.S.units * wpu, KA_WAVES);
    if (grid >= (int64_t)1 << 31) return hipErrorInvalidValue;
    const dim3 g((unsigned)grid), block(KA_WAVES * 64);
#define LORA_APPEND_Q8(NP, WPU) \
    hipLaunchKernelGGL((k_kv_append_q8<TI, D, NP, WPU>), g, block, 0, stream, a, it, q_runs)
    switch (passes) {
        case 1: LORA_APPEND_Q8(1, 1); break;
        case 2: LORA_APPEND_Q8(2, 1); break;
        case 4: LORA_APPEND_Q8(4, 1); break;
        case 8: LORA_APPEND_Q8(2, KA_WAVES); break;
        case 16: LORA_APPEND_Q8(4, KA_WAVES); break;
        default: LORA_APPEND_Q8(8, KA_WAVES); break;   // 128 tokens of 256
    }
#undef LORA_APPEND_Q8
    return hipGetLastError();
}

template <typename TI>
hipError_t launch_t(const AppendArgs& a, int32_t head_dim, hipStream_t stream) {
    switch (head_dim) {
        case 64: return launch_d<TI, 64>(a, stream);
        case 128: return launch_d<TI, 128>(a, stream);
        default: return launch_d<TI, 256>(a, stream);
    }
}

}  // namespace

hipError_t launch_kv_append_q8(const AppendArgs& a, lora_dtype_t in, int32_t head_dim, hipStream_t stream) {
    return in == LORA_BF16 ? launch_t<bf16>(a, head_dim, stream) : launch_t<float>(a, head_dim, stream);
}

}  // namespace lora
