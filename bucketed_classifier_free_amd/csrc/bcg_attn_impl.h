// The paged attention kernels (decode: one query a row; prompt: runs of
// queries), instantiated per storage type by bcg_attn_*.hip.
//
// Mathematics: with m the running maximum of a query's scaled scores
// s_t = scale * q . k_t, l = sum_t 2^(s_t - m) and o = sum_t 2^(s_t - m) v_t
// (scores in log2 units), one pass over the tokens keeps (m, l, o); a larger
// score multiplies l and o by 2^(m - m'), and out = o / l.  The maximum is
// moved only when a score exceeds it by more than 8: the terms are then at
// most 2^8, which fp32 sums and bf16 probabilities (a relative format) hold as
// well as terms below 1, and nearly every block skips the rescale.
//
// Matrix layout, the same for both kernels.  Both products are taken
// transposed, S^T = K Q^T and O^T = V^T P^T, so that a query is a column: in
// the 16 x 16 accumulator a lane (c = lane % 16, g = lane / 16) holds rows
// 4g..4g+3 of column c.  Then
//   - the softmax state of a query is the same in its four lanes, and a
//     rescale of o is lane-local;
//   - S^T of two 16-token tiles, rounded, is P^T as the second product wants
//     it: its k index (g, i) stands for token 4g + i of the first tile for
//     i < 4 and token 4g + i - 4 of the second, so no value changes lanes;
//   - a row of V^T is one dimension: lane c takes dimensions cE..cE+E-1 (E =
//     padded head_dim / 16) of its eight tokens with wide loads, and the
//     E products take one dimension of each lane (a 16-bit transpose in
//     registers, two byte permutes per pair); lane (c, g) ends up with 4E
//     consecutive output dimensions of query c.
// fp32 takes the same k index through 16 x 16 x 4 products, one per i.
#pragma once

#include "bcg_attn.h"
#include "bcg_device.h"

namespace bcg {
namespace attn {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x8_t __attribute__((ext_vector_type(8)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kSlack = 8.0f;

// ---------------------------------------------------------------- operands

template <typename QT> struct Op;  // compute type of a query type
template <> struct Op<bf16_t> {
    typedef u32x4_t F8;  // eight k indices of one lane
    static constexpr int dwords = 4;
    static __device__ __forceinline__ void mma(const F8& a, const F8& b, f32x4_t& c) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ F8 pack(const f32x4_t& a, const f32x4_t& b) {
        return F8{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
    }
};
template <> struct Op<float> {
    typedef f32x8_t F8;
    static constexpr int dwords = 8;
    static __device__ __forceinline__ void mma(const F8& a, const F8& b, f32x4_t& c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    }
    static __device__ __forceinline__ F8 pack(const f32x4_t& a, const f32x4_t& b) {
        return F8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
};

// N dwords in the widest loads that a 4-, 8- or 16-byte aligned address takes.
template <int N> struct Words { uint32_t w[N]; };
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
template <int N> __device__ __forceinline__ Words<N> load_words(const void* p) {
    Words<N> r;
    if constexpr (N == 1) {
        r.w[0] = *static_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const u32x2_t x = *static_cast<const u32x2_t*>(p);
        r.w[0] = x[0]; r.w[1] = x[1];
    } else {
        static_assert(N % 4 == 0, "");
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4_t x = static_cast<const u32x4_t*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) r.w[4 * i + j] = x[j];
        }
    }
    return r;
}

// Four e4m3 values (a dword) as bf16 pairs; exact.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
}

// First dimension of the eight that a lane's k indices of step s stand for.
// e4m3 takes 16 bytes (16 dimensions) a load, two steps.
template <typename KT> __device__ __forceinline__ int k_dim(int s, int g) {
    if constexpr (sizeof(KT) == 1) return (s >> 1) * 64 + g * 16 + (s & 1) * 8;
    else return s * 32 + g * 8;
}

// Keys of one 16-token tile in one lane: token c, the dimensions k_dim(s, g).
template <typename KT, int DP, bool EX> struct KTile {
    static constexpr int S = DP / 32;
    Words<S * 2 * (int)sizeof(KT)> r;  // S steps of 8 elements
    __device__ __forceinline__ void load(const KT* row, int g, int D) {
        constexpr int L = sizeof(KT) == 1 ? S / 2 : S;  // loads
        constexpr int W = sizeof(KT) == 4 ? 8 : 4;      // dwords of each
#pragma unroll
        for (int i = 0; i < L; ++i) {
            const int d = k_dim<KT>(sizeof(KT) == 1 ? 2 * i : i, g);
            const bool in = EX || d < D;
            const Words<W> x = load_words<W>(row + (in ? d : 0));
#pragma unroll
            for (int j = 0; j < W; ++j) r.w[i * W + j] = in ? x.w[j] : 0u;
        }
    }
    template <typename QT> __device__ __forceinline__ typename Op<QT>::F8 frag(int s) const {
        typename Op<QT>::F8 f;
        if constexpr (sizeof(KT) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.w[s * 8 + i]);
        } else if constexpr (sizeof(KT) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = r.w[s * 4 + i];
        } else {
            f[0] = e4m3_lo(r.w[s * 2]); f[1] = e4m3_hi(r.w[s * 2]);
            f[2] = e4m3_lo(r.w[s * 2 + 1]); f[3] = e4m3_hi(r.w[s * 2 + 1]);
        }
        return f;
    }
};

// E consecutive dimensions of one token's values in one lane.
template <typename KT, int E> using VRow = Words<E * (int)sizeof(KT) / 4>;

// Loads it: dimensions d..d+E-1 of a row of D (a multiple of 8), what lies
// beyond D (dimensions that nobody stores) replaced by the row's first ones.
template <typename KT, int E, bool EX> __device__ __forceinline__ VRow<KT, E> load_v(const KT* row, int d, int D) {
    constexpr int B = E < 8 ? E : 8, N = B * (int)sizeof(KT) / 4;
    VRow<KT, E> r;
#pragma unroll
    for (int b = 0; b < E; b += B) {
        if constexpr (EX && E * sizeof(KT) >= 16) {
            return load_words<E * (int)sizeof(KT) / 4>(row + d);
        } else {
            const Words<N> x = load_words<N>(row + (EX || d + b < D ? d + b : 0));
#pragma unroll
            for (int w = 0; w < N; ++w) r.w[b / B * N + w] = x.w[w];
        }
    }
    return r;
}

// Element j of the eight tokens' rows as the k indices of one lane.
template <typename QT, typename KT, int E>
__device__ __forceinline__ typename Op<QT>::F8 v_frag(const VRow<KT, E> (&v)[8], int j) {
    typename Op<QT>::F8 f;
    if constexpr (sizeof(KT) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i].w[j]);
    } else if constexpr (sizeof(KT) == 2) {
        const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __builtin_amdgcn_perm(v[2 * i + 1].w[j >> 1], v[2 * i].w[j >> 1], sel);
    } else {
        // gather byte j of two tokens into the low half of a dword, then widen the pair
        const uint32_t b = j & 3, sel = 0x0c0c0000u | ((4 + b) << 8) | b;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = e4m3_lo(__builtin_amdgcn_perm(v[2 * i + 1].w[j >> 2], v[2 * i].w[j >> 2], sel));
    }
    return f;
}

// The queries' fragments: eight elements at dimension d of a query (zeros beyond D).
template <typename QT> __device__ __forceinline__ typename Op<QT>::F8 load_q8(const QT* q, int d, int D, bool have) {
    typename Op<QT>::F8 f = {};
    if (have && d < D) {
        const Words<Op<QT>::dwords> x = load_words<Op<QT>::dwords>(q + d);
#pragma unroll
        for (int i = 0; i < Op<QT>::dwords; ++i) f[i] = __uint_as_float(x.w[i]);
    }
    return f;
}
template <> __device__ __forceinline__ u32x4_t load_q8<bf16_t>(const bf16_t* q, int d, int D, bool have) {
    u32x4_t f = {0, 0, 0, 0};
    if (have && d < D) f = *reinterpret_cast<const u32x4_t*>(q + d);
    return f;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum and sum over the four lanes of a column.
__device__ __forceinline__ float col_max(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
__device__ __forceinline__ float col_sum(float x) {
    x += __shfl_xor(x, 16);
    return x + __shfl_xor(x, 32);
}

// The page of the 16 tokens from t on; -1 where there is none.
__device__ __forceinline__ int page_of(const AttnParams& p, const int32_t* row_table, int t, int len) {
    if (t >= len) return -1;
    const int pg = row_table[p.shift >= 0 ? t >> p.shift : t / p.ps];
    return pg >= 0 && pg < p.np ? pg : -1;
}

template <typename QT, int E>
__device__ __forceinline__ void store_row(QT* out, const float (&x)[E], int d, int D) {
    // D is a multiple of 8 and E of 4: groups of four are stored or left out whole
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        if (d + i < D) {
            if constexpr (sizeof(QT) == 4) {
                *reinterpret_cast<f32x4_t*>(out + d + i) = f32x4_t{x[i], x[i + 1], x[i + 2], x[i + 3]};
            } else {
                *reinterpret_cast<u32x2_t*>(out + d + i) = u32x2_t{pack_bf16x2(x[i], x[i + 1]), pack_bf16x2(x[i + 2], x[i + 3])};
            }
        }
    }
}

// ---------------------------------------------------------------- decode

// One workgroup: the tokens of one split of a row for up to 16 query heads of
// one kv head.  Four waves take the split's 32-token blocks in turn, straight
// from memory into registers (each key and value is used once, so there is
// nothing for LDS to share); their states are joined in LDS at the end.
template <typename QT, typename KT, int DP, bool EX>
__global__ void __launch_bounds__(256) decode_kernel(const AttnParams p) {
    constexpr int E = DP / 16, S = DP / 32;
    typedef typename Op<QT>::F8 F8;
    __shared__ float2 ml_s[4][16];
    __shared__ __attribute__((aligned(16))) float o_s[4][16][DP];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int c = lane & 15, g = lane >> 4;
    unsigned id = blockIdx.x;
    const int tile = id % p.tiles; id /= p.tiles;
    const int h = id % p.kvh; id /= p.kvh;
    const int split = id % p.splits;
    const int row = id / p.splits;
    const int len = min(max(p.len[row], 0), p.max_len);
    const int lo = p.window > 0 ? max(0, len - p.window) : 0;
    const BlockList bl = visible_blocks(lo, len, p.sinks, 32);
    const int v0 = split * p.chunk, v1 = min(bl.nb, v0 + p.chunk);
    const int head0 = h * p.G + tile * 16, nh = min(16, p.G - tile * 16);
    const int32_t* table = p.table + (int64_t)row * p.maxb;

    F8 q[S];
    {
        const QT* qr = static_cast<const QT*>(p.q) + (int64_t)row * p.qstride + (int64_t)(head0 + c) * p.D;
#pragma unroll
        for (int s = 0; s < S; ++s) q[s] = load_q8<QT>(qr, k_dim<KT>(s, g), p.D, c < nh);
    }
    const float sc = p.kscale ? p.scale2 * p.kscale[h] : p.scale2;
    float m = kNegInf, nm = 0.0f, l = 0.0f;
    f32x4_t o[E];
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] = f32x4_t{0, 0, 0, 0};
    const KT* kc = static_cast<const KT*>(p.k) + (int64_t)h * p.ps * p.D;
    const KT* vc = static_cast<const KT*>(p.v) + (int64_t)h * p.ps * p.D;

    for (int vb = v0 + wave; vb < v1; vb += 4) {
        const int t0 = bl(vb) * 32;
        const int pg0 = page_of(p, table, t0, len), pg1 = page_of(p, table, t0 + 16, len);
        const int in0 = p.shift >= 0 ? t0 & (p.ps - 1) : t0 % p.ps;
        const int in1 = p.shift >= 0 ? (t0 + 16) & (p.ps - 1) : (t0 + 16) % p.ps;
        const int64_t a0 = max(pg0, 0), a1 = max(pg1, 0);
        KTile<KT, DP, EX> k0, k1;
        k0.load(kc + a0 * p.kps + (in0 + c) * p.D, g, p.D);
        k1.load(kc + a1 * p.kps + (in1 + c) * p.D, g, p.D);
        VRow<KT, E> v[8];
        {
            const KT* r0 = vc + a0 * p.vps + (in0 + 4 * g) * p.D;
            const KT* r1 = vc + a1 * p.vps + (in1 + 4 * g) * p.D;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = load_v<KT, E, EX>(r0 + i * p.D, c * E, p.D);
                v[4 + i] = load_v<KT, E, EX>(r1 + i * p.D, c * E, p.D);
            }
        }
        f32x4_t s0 = {0, 0, 0, 0}, s1 = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < S; ++s) {
            Op<QT>::mma(k0.template frag<QT>(s), q[s], s0);
            Op<QT>::mma(k1.template frag<QT>(s), q[s], s1);
        }
        s0 *= sc;
        s1 *= sc;
        if (!(t0 + 32 <= len && pg0 >= 0 && pg1 >= 0 && (t0 >= lo || t0 + 32 <= p.sinks))) {
            // hidden tokens: no score, and their values count as zero (0 * NaN would not)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // selects, not branches: with branches here the compiler was seen to lose the first assignment
                const int t = t0 + (i < 4 ? 0 : 16) + 4 * g + (i & 3);
                const bool seen = (t < len) & ((t >= lo) | (t < p.sinks)) & ((i < 4 ? pg0 : pg1) >= 0);
                if (i < 4) s0[i & 3] = seen ? s0[i & 3] : kNegInf;
                else s1[i & 3] = seen ? s1[i & 3] : kNegInf;
#pragma unroll
                for (int w = 0; w < E * (int)sizeof(KT) / 4; ++w) v[i].w[w] = seen ? v[i].w[w] : 0u;
            }
        }
        const float mx = fmaxf(fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3])), fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3])));
        if (__any(mx > m + kSlack)) {
            const float top = fmaxf(m, col_max(mx));
            const float f = top == kNegInf ? 1.0f : exp2_(m - top);
            m = top;
            nm = top == kNegInf ? 0.0f : -top;
            l *= f;
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] *= f;
        }
        f32x4_t p0, p1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p0[i] = exp2_(s0[i] + nm);
            p1[i] = exp2_(s1[i] + nm);
        }
        l += ((p0[0] + p0[1]) + (p0[2] + p0[3])) + ((p1[0] + p1[1]) + (p1[2] + p1[3]));
        const F8 pf = Op<QT>::pack(p0, p1);
#pragma unroll
        for (int j = 0; j < E; ++j) Op<QT>::mma(v_frag<QT, KT, E>(v, j), pf, o[j]);
    }

    // join the four waves
    l = col_sum(l);
    if (g == 0) ml_s[wave][c] = make_float2(m, l);
    __syncthreads();
    {
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, ml_s[w][c].x);
        // m = -infinity: nothing seen (l and o are 0), or nothing but NaN scores (they are NaN)
        const float f = m == kNegInf ? 1.0f : exp2_(m - top);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) o_s[wave][c][(4 * g + i) * E + j] = o[j][i] * f;
    }
    __syncthreads();
    const int hh = threadIdx.x >> 4, d = (threadIdx.x & 15) * E;
    if (hh >= nh) return;
    float top = kNegInf, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, ml_s[w][hh].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) sum += ml_s[w][hh].x == kNegInf ? ml_s[w][hh].y : ml_s[w][hh].y * exp2_(ml_s[w][hh].x - top);
    float x[E];
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = (o_s[0][hh][d + j] + o_s[1][hh][d + j]) + (o_s[2][hh][d + j] + o_s[3][hh][d + j]);
    const int64_t at = (int64_t)row * p.qh + head0 + hh;
    const float vs = p.vscale ? p.vscale[h] : 1.0f;
    if (p.splits == 1) {
        const float inv = sum == 0.0f ? 0.0f : vs / sum;
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] *= inv;
        store_row<QT, E>(static_cast<QT*>(p.out) + at * p.D, x, d, p.D);
        if (p.lse && d == 0) p.lse[at] = sum == 0.0f ? kNegInf : (top == kNegInf ? sum : (top + __log2f(sum)) * 0.69314718055994531f);
    } else {
        const int64_t ps = (int64_t)split * p.tokens * p.qh + at;
        if (v0 < v1) {
#pragma unroll
            for (int j = 0; j < E; ++j) x[j] *= vs;
            store_row<float, E>(p.part_o + ps * p.D, x, d, p.D);
        }
        if (d == 0) p.part_ml[ps] = make_float2(top, sum);
    }
}

// ---------------------------------------------------------------- prompt

// One workgroup: 64 * R columns (query, head of the kv head's group) of one
// row, four waves of R 16-column tiles each, against 64-token tiles of keys
// and values that the workgroup stages in LDS in operand order, so that every
// fragment is one conflict-free 16-byte (fp32: 32-byte) read per lane and
// serves R products.
template <typename QT, typename KT, int DP, int R, bool EX> struct Prompt {
    static constexpr int E = DP / 16, S = DP / 32, T = 64;
    static constexpr int OW = Op<QT>::dwords;                // dwords of a fragment
    typedef typename Op<QT>::F8 F8;
    static constexpr int kFrag = 64 * OW;                    // dwords of one fragment, all lanes
    static constexpr int kSide = T * DP * (int)sizeof(QT) / 4;  // dwords of one tile of keys or values
    static constexpr int CPR = DP * (int)sizeof(KT) / 16;    // 16-byte chunks of a key
    static constexpr int KL = T * CPR / 256;                 // chunks a thread stages
    static constexpr int EPC = 16 / (int)sizeof(KT);         // elements of a chunk
    static constexpr int VW = E * (int)sizeof(KT) / 4;       // dwords of a thread's part of one value

    struct Stage {
        Words<4> k[KL];
        Words<VW> v[4];
    };

    // Where element block e8 (eight dimensions) of token t lies: fragment
    // (t / 16, step), lane (c, g), its 16-byte halves rotated by the step and
    // g so that the lanes that stage one token hit different banks.
    static __device__ __forceinline__ int k_slot(int t, int e8) {
        const int s = e8 >> 2, g = e8 & 3;
        return ((t >> 4) * S + s) * kFrag + (g * 16 + ((t & 15) ^ (e8 & 7))) * OW;
    }
};

template <typename QT, typename KT, int DP, int R, bool EX>
__global__ void __launch_bounds__(256) prompt_kernel(const AttnParams p) {
    typedef Prompt<QT, KT, DP, R, EX> P;
    constexpr int E = P::E, S = P::S, T = P::T, OW = P::OW, C = 64 * R;
    typedef typename Op<QT>::F8 F8;
    extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
    uint32_t* const ks = lds;
    uint32_t* const vs = lds + P::kSide;
    int* const odd = reinterpret_cast<int*>(lds + 2 * P::kSide);  // a value that is not finite is in the tile
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;

    unsigned id = blockIdx.x;
    const int h = id % p.kvh; id /= p.kvh;
    const int split = id % p.splits; id /= p.splits;
    const int row = id % p.rows;
    const int tile = p.tiles - 1 - (int)(id / p.rows);  // the longest first
    const int q0 = min(max(p.qoff[row], 0), p.tokens);
    const int n = min(max(p.qoff[row + 1], q0), p.tokens) - q0;
    const int cols = min(n, p.max_new) * p.G, c0 = tile * C;
    if (c0 >= cols) return;
    const int len = min(max(p.len[row], 0), p.max_len);
    const int first = len - n;  // position of the row's first query
    const int32_t* table = p.table + (int64_t)row * p.maxb;

    int pos[R];
    int64_t at[R];  // (token, head) of this lane's columns, -1: none
    F8 q[R][S];
    const int cw = c0 + wave * 16 * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int col = cw + r * 16 + c, i = col / p.G;
        const bool have = col < cols;
        pos[r] = have ? first + i : -1;
        const int64_t tok = q0 + i;
        const int head = h * p.G + (col - i * p.G);
        at[r] = have ? tok * p.qh + head : -1;
        const QT* qr = static_cast<const QT*>(p.q) + (have ? tok * p.qstride + (int64_t)head * p.D : 0);
#pragma unroll
        for (int s = 0; s < S; ++s) q[r][s] = load_q8<QT>(qr, s * 32 + g * 8, p.D, have);
    }
    // positions of the workgroup's and the wave's queries
    const int pmin = first + c0 / p.G, pmax = first + (min(cols, c0 + C) - 1) / p.G;
    const bool busy = cw < cols;
    const int wmax = busy ? first + (min(cols, cw + 16 * R) - 1) / p.G : -1;
    const int lo = p.window > 0 ? max(0, pmin - p.window + 1) : 0;
    const BlockList bl = visible_blocks(lo, pmax + 1, p.sinks, T);
    const int v0 = split * p.chunk, v1 = min(bl.nb, v0 + p.chunk);

    const float sc = p.kscale ? p.scale2 * p.kscale[h] : p.scale2;
    float m[R], nm[R], l[R];
    f32x4_t o[R][E];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        m[r] = kNegInf; nm[r] = 0.0f; l[r] = 0.0f;
#pragma unroll
        for (int j = 0; j < E; ++j) o[r][j] = f32x4_t{0, 0, 0, 0};
    }
    const KT* kc = static_cast<const KT*>(p.k) + (int64_t)h * p.ps * p.D;
    const KT* vc = static_cast<const KT*>(p.v) + (int64_t)h * p.ps * p.D;

    typename P::Stage st;
    auto in_page = [&](int t) { return p.shift >= 0 ? t & (p.ps - 1) : t % p.ps; };
    // what a thread stages: keys as 16-byte chunks, row by row; values as four
    // tokens (4g'..4g'+3 of a 16-token tile) by E dimensions
    const int vh = tid >> 6;
    auto fetch = [&](int vb) {
        const int t0 = bl(vb) * T;
#pragma unroll
        for (int i = 0; i < P::KL; ++i) {
            const int ch = tid + 256 * i, t = ch / P::CPR, d = (ch % P::CPR) * P::EPC;
            const int half = t0 + (t & ~15);
            const int pg = page_of(p, table, half, len);
            const bool in = (EX || d < p.D) && pg >= 0;
            const KT* a = kc + (int64_t)max(pg, 0) * p.kps + (in_page(half) + (t & 15)) * p.D + (in ? d : 0);
            const Words<4> x = load_words<4>(a);
#pragma unroll
            for (int w = 0; w < 4; ++w) st.k[i].w[w] = EX || d < p.D ? x.w[w] : 0u;
        }
        {
            const int half = t0 + vh * 16, pg = page_of(p, table, half, len);
            const KT* a = vc + (int64_t)max(pg, 0) * p.vps + (in_page(half) + 4 * g) * p.D;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                st.v[i] = load_v<KT, E, EX>(a + i * p.D, c * E, p.D);
                const bool there = (pg >= 0) & (half + 4 * g + i < len);
#pragma unroll
                for (int w = 0; w < P::VW; ++w) st.v[i].w[w] = there ? st.v[i].w[w] : 0u;
            }
        }
    };
    // not finite: exponent bits all ones (bf16, fp32), or the one NaN code (e4m3)
    auto strange = [&](uint32_t w) -> bool {
        if constexpr (sizeof(KT) == 4) return (w & 0x7f800000u) == 0x7f800000u;
        else if constexpr (sizeof(KT) == 2) return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
        else return (w & 0x7fu) == 0x7fu || (w & 0x7f00u) == 0x7f00u || (w & 0x7f0000u) == 0x7f0000u || (w & 0x7f000000u) == 0x7f000000u;
    };
    auto store = [&](bool check) {
#pragma unroll
        for (int i = 0; i < P::KL; ++i) {
            const int ch = tid + 256 * i, t = ch / P::CPR, d = (ch % P::CPR) * P::EPC;
            const Words<4>& x = st.k[i];
            if constexpr (sizeof(KT) == 4) {
                // half of a fragment: dimensions d..d+3
                *reinterpret_cast<u32x4_t*>(ks + P::k_slot(t, d >> 3) + (d & 4)) = u32x4_t{x.w[0], x.w[1], x.w[2], x.w[3]};
            } else if constexpr (sizeof(KT) == 2) {
                *reinterpret_cast<u32x4_t*>(ks + P::k_slot(t, d >> 3)) = u32x4_t{x.w[0], x.w[1], x.w[2], x.w[3]};
            } else {
                *reinterpret_cast<u32x4_t*>(ks + P::k_slot(t, d >> 3)) =
                    u32x4_t{e4m3_lo(x.w[0]), e4m3_hi(x.w[0]), e4m3_lo(x.w[1]), e4m3_hi(x.w[1])};
                *reinterpret_cast<u32x4_t*>(ks + P::k_slot(t, (d >> 3) + 1)) =
                    u32x4_t{e4m3_lo(x.w[2]), e4m3_hi(x.w[2]), e4m3_lo(x.w[3]), e4m3_hi(x.w[3])};
            }
        }
        // fragment (two 16-token tiles, dimension j of each lane): the lane's k
        // indices 0..3 are the first tile's tokens, 4..7 the second's
#pragma unroll
        for (int j = 0; j < E; ++j) {
            uint32_t* to = vs + ((vh >> 1) * E + j) * P::kFrag + lane * OW + (vh & 1) * (OW / 2);
            if constexpr (sizeof(KT) == 4) {
                *reinterpret_cast<u32x4_t*>(to) = u32x4_t{st.v[0].w[j], st.v[1].w[j], st.v[2].w[j], st.v[3].w[j]};
            } else if constexpr (sizeof(KT) == 2) {
                const uint32_t sel = j & 1 ? 0x07060302u : 0x05040100u;
                *reinterpret_cast<u32x2_t*>(to) = u32x2_t{__builtin_amdgcn_perm(st.v[1].w[j >> 1], st.v[0].w[j >> 1], sel),
                                                          __builtin_amdgcn_perm(st.v[3].w[j >> 1], st.v[2].w[j >> 1], sel)};
            } else {
                const uint32_t b = j & 3, sel = 0x0c0c0000u | ((4 + b) << 8) | b;
                *reinterpret_cast<u32x2_t*>(to) = u32x2_t{e4m3_lo(__builtin_amdgcn_perm(st.v[1].w[j >> 2], st.v[0].w[j >> 2], sel)),
                                                          e4m3_lo(__builtin_amdgcn_perm(st.v[3].w[j >> 2], st.v[2].w[j >> 2], sel))};
            }
        }
        if (check) {
            bool any = false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < P::VW; ++w) any = any || strange(st.v[i].w[w]);
            if (any) *odd = 1;
        }
    };
    auto pages_there = [&](int t0) {
        bool ok = true;
#pragma unroll
        for (int i = 0; i < T / 16; ++i) ok = ok && page_of(p, table, t0 + 16 * i, len) >= 0;
        return ok;
    };

    if (v0 < v1) fetch(v0);
    for (int vb = v0; vb < v1; ++vb) {
        const int t0 = bl(vb) * T;
        // a tile that every query of the workgroup sees whole needs no masks
        const bool whole = t0 + T - 1 <= pmin && (p.window == 0 || t0 > pmax - p.window || t0 + T <= p.sinks) && pages_there(t0);
        __syncthreads();
        if (tid == 0) *odd = 0;
        __syncthreads();
        store(!whole);
        __syncthreads();
        if (vb + 1 < v1) fetch(vb + 1);
        if (!busy || t0 > wmax) continue;  // nothing here for this wave's queries (the barriers are met above)
        const bool slow = !whole && *odd;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            f32x4_t x[R][2];
#pragma unroll
            for (int r = 0; r < R; ++r) x[r][0] = x[r][1] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt) {
                    const F8 a = *reinterpret_cast<const F8*>(ks + ((kb * 2 + tt) * S + s) * P::kFrag + (g * 16 + (c ^ ((s * 4 + g) & 7))) * OW);
#pragma unroll
                    for (int r = 0; r < R; ++r) Op<QT>::mma(a, q[r][s], x[r][tt]);
                }
            F8 pf[R];
            bool seen[R][8];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                x[r][0] *= sc;
                x[r][1] *= sc;
                if (!whole) {
                    const int pg0 = page_of(p, table, t0 + kb * 32, len), pg1 = page_of(p, table, t0 + kb * 32 + 16, len);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int t = t0 + kb * 32 + (i < 4 ? 0 : 16) + 4 * g + (i & 3);
                        seen[r][i] = (t <= pos[r]) & ((p.window == 0) | (t > pos[r] - p.window) | (t < p.sinks)) & ((i < 4 ? pg0 : pg1) >= 0);
                        x[r][i >> 2][i & 3] = seen[r][i] ? x[r][i >> 2][i & 3] : kNegInf;
                    }
                }
                const float mx = fmaxf(fmaxf(fmaxf(x[r][0][0], x[r][0][1]), fmaxf(x[r][0][2], x[r][0][3])),
                                       fmaxf(fmaxf(x[r][1][0], x[r][1][1]), fmaxf(x[r][1][2], x[r][1][3])));
                if (__any(mx > m[r] + kSlack)) {
                    const float top = fmaxf(m[r], col_max(mx));
                    const float f = top == kNegInf ? 1.0f : exp2_(m[r] - top);
                    m[r] = top;
                    nm[r] = top == kNegInf ? 0.0f : -top;
                    l[r] *= f;
#pragma unroll
                    for (int j = 0; j < E; ++j) o[r][j] *= f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[r][i >> 2][i & 3] = exp2_(x[r][i >> 2][i & 3] + nm[r]);
                l[r] += ((x[r][0][0] + x[r][0][1]) + (x[r][0][2] + x[r][0][3])) + ((x[r][1][0] + x[r][1][1]) + (x[r][1][2] + x[r][1][3]));
                pf[r] = Op<QT>::pack(x[r][0], x[r][1]);
            }
            if (!slow) {
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    const F8 a = *reinterpret_cast<const F8*>(vs + (kb * E + j) * P::kFrag + lane * OW);
#pragma unroll
                    for (int r = 0; r < R; ++r) Op<QT>::mma(a, pf[r], o[r][j]);
                }
            } else {
                // some value of the tile is not finite: 0 * it must not reach a
                // query that does not see its token.  One token at a time, each
                // query taking the sum only if it sees the token.
                for (int k = 0; k < 32; ++k) {
                    const int kg = (k >> 2) & 3, ki = (k & 3) + (k >> 4) * 4;  // the k index (g, i) of token k
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        F8 one = pf[r];
                        bool mine = false;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const bool hit = g == kg && i == ki;
                            mine = mine || (hit && seen[r][i]);
                            if constexpr (OW == 8) { if (!hit) one[i] = 0.0f; }
                            else { if (!hit) one[i >> 1] &= i & 1 ? 0x0000ffffu : 0xffff0000u; }
                        }
                        mine = __shfl((int)mine, kg * 16 + c) != 0;
#pragma unroll
                        for (int j = 0; j < E; ++j) {
                            F8 a = *reinterpret_cast<const F8*>(vs + (kb * E + j) * P::kFrag + lane * OW);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if constexpr (OW == 8) { if (!(g == kg && i == ki)) a[i] = 0.0f; }
                                else { if (!(g == kg && i == ki)) a[i >> 1] &= i & 1 ? 0x0000ffffu : 0xffff0000u; }
                            }
                            f32x4_t y = o[r][j];
                            Op<QT>::mma(a, one, y);
#pragma unroll
                            for (int i = 0; i < 4; ++i) o[r][j][i] = mine ? y[i] : o[r][j][i];
                        }
                    }
                }
            }
        }
    }

    const float vsc = p.vscale ? p.vscale[h] : 1.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float sum = col_sum(l[r]);
        if (at[r] < 0) continue;
        const float inv = p.splits > 1 ? vsc : (sum == 0.0f ? 0.0f : vsc / sum);
        const int64_t to = p.splits > 1 ? (int64_t)split * p.tokens * p.qh + at[r] : at[r];
        float y[4 * E];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < E; ++j) y[i * E + j] = o[r][j][i] * inv;
        if (p.splits > 1) {
            if (v0 < v1) store_row<float, 4 * E>(p.part_o + to * p.D, y, 4 * g * E, p.D);
            if (g == 0) p.part_ml[to] = make_float2(m[r], sum);
        } else {
            store_row<QT, 4 * E>(static_cast<QT*>(p.out) + to * p.D, y, 4 * g * E, p.D);
            if (p.lse && g == 0)
                p.lse[to] = sum == 0.0f ? kNegInf : (m[r] == kNegInf ? sum : (m[r] + __log2f(sum)) * 0.69314718055994531f);
        }
    }
}

// ---------------------------------------------------------------- join

// One wave a (token, head): out = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
template <typename QT> __global__ void __launch_bounds__(256) join_kernel(const AttnParams p) {
    const int64_t n = (int64_t)p.tokens * p.qh, at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (at >= n) return;
    if (p.qoff) {
        // a token that no row has, or beyond max_new, was not computed
        const int tok = (int)(at / p.qh);
        bool mine = false;
        for (int r = lane; r < p.rows; r += 64) {
            const int a = min(max(p.qoff[r], 0), p.tokens), b = min(max(p.qoff[r + 1], a), p.tokens);
            mine = mine || (tok >= a && tok < b && tok - a < p.max_new);
        }
        if (!__any(mine)) return;
    }
    float top = kNegInf;
    for (int s = lane; s < p.splits; s += 64) top = fmaxf(top, p.part_ml[s * n + at].x);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) top = fmaxf(top, __shfl_xor(top, k));
    float sum = 0.0f, x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int d = lane * 4;
    for (int s = 0; s < p.splits; ++s) {
        const float2 ml = p.part_ml[s * n + at];
        if (ml.x == kNegInf && ml.y == 0.0f) continue;  // nothing seen there, its o is not written
        const float f = ml.x == kNegInf ? 1.0f : exp2_(ml.x - top);
        sum += f * ml.y;
        if (d < p.D) {
            const f32x4_t y = *reinterpret_cast<const f32x4_t*>(p.part_o + (s * n + at) * p.D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] += f * y[i];
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= inv;
    store_row<QT, 4>(static_cast<QT*>(p.out) + at * p.D, x, d, p.D);
    if (p.lse && lane == 0)
        p.lse[at] = sum == 0.0f ? kNegInf : (top == kNegInf ? sum : (top + __log2f(sum)) * 0.69314718055994531f);
}

template <typename QT> inline hipError_t launch_join(const AttnParams& p, hipStream_t st) {
    const int64_t n = (int64_t)p.tokens * p.qh;
    hipLaunchKernelGGL((join_kernel<QT>), dim3((unsigned)((n + 3) / 4)), dim3(256), 0, st, p);
    return hipGetLastError();
}

template <typename QT, typename KT, int DP>
inline hipError_t decode_dp(const AttnParams& p, hipStream_t st) {
    const dim3 grid((unsigned)((int64_t)p.rows * p.splits * p.kvh * p.tiles));
    if (p.D == DP) hipLaunchKernelGGL((decode_kernel<QT, KT, DP, true>), grid, dim3(256), 0, st, p);
    else hipLaunchKernelGGL((decode_kernel<QT, KT, DP, false>), grid, dim3(256), 0, st, p);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits == 1 ? e : launch_join<QT>(p, st);
}

// Tiles of 16 columns a wave takes: as many as the registers hold beside the
// fragments of the queries.
template <typename QT, int DP> constexpr int prompt_tiles() { return DP == 256 ? 1 : 2; }

template <typename QT, typename KT, int DP, bool EX>
inline hipError_t prompt_ex(const AttnParams& p, hipStream_t st) {
    constexpr int R = prompt_tiles<QT, DP>();
    constexpr size_t lds = (2 * Prompt<QT, KT, DP, R, EX>::kSide + 4) * sizeof(uint32_t);
    if constexpr (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(prompt_kernel<QT, KT, DP, R, EX>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)((int64_t)p.rows * p.splits * p.kvh * p.tiles));
    hipLaunchKernelGGL((prompt_kernel<QT, KT, DP, R, EX>), grid, dim3(256), lds, st, p);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || p.splits == 1 ? e : launch_join<QT>(p, st);
}
template <typename QT, typename KT, int DP>
inline hipError_t prompt_dp(const AttnParams& p, hipStream_t st) {
    return p.D == DP ? prompt_ex<QT, KT, DP, true>(p, st) : prompt_ex<QT, KT, DP, false>(p, st);
}

}  // namespace attn

template <typename QT, typename KT> hipError_t launch_decode(const AttnParams& p, hipStream_t st) {
    if (p.D <= 64) return attn::decode_dp<QT, KT, 64>(p, st);
    if (p.D <= 128) return attn::decode_dp<QT, KT, 128>(p, st);
    return attn::decode_dp<QT, KT, 256>(p, st);
}
template <typename QT, typename KT> hipError_t launch_prompt(const AttnParams& p, hipStream_t st) {
    if (p.D <= 64) return attn::prompt_dp<QT, KT, 64>(p, st);
    if (p.D <= 128) return attn::prompt_dp<QT, KT, 128>(p, st);
    return attn::prompt_dp<QT, KT, 256>(p, st);
}

}  // namespace bcg
