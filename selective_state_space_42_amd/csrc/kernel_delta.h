// kernel_delta.h -- the gated delta rule (include/ssm_delta.h): chunked
// forward kernels and the decode step.
//
// A chunk of C = 64 steps of one (batch row, value head), with S (K x V here)
// the state entering it, G_i the running sum of g inside the chunk and
// D = diag(beta):
//   A'_ij = e^{G_i - G_j} k_i.k_j  (j < i),   X = (I + A' D)^-1 A'
//   E  = V - e^G o (K S)                      each step's value less what S predicts
//   E^ = E - X (beta o E),  U = beta o E^     ... less what the chunk's earlier steps wrote
//   P_ij = scale e^{G_i - G_j} q_i.k_j  (j <= i)
//   Y  = scale e^G o (Q S) + P U
//   S' = e^{G_63} S + K^T (e^{G_63 - G} o U)
// (The inner U of the recurrence satisfies U = beta o (E - A' U); E^ solves
// (I + A' D) E^ = E, and X = (I + A' D)^-1 A' serves the gradients as well,
// since (I + D A')^-1 = I - D X: no division by beta.)
//
// Precision.  Every product runs on the bf16 matrix units (16x16x32, fp32
// accumulation).  An fp32 operand is split exactly into bf16 planes
// x = x0 + x1 + x2 (8 bits each; three planes hold all 24), and a product
// takes the plane pairs a_i b_j with i + j < 3: an fp32 product to 2^-24 at 3
// (bf16 by fp32) or 6 (fp32 by fp32) times a bf16 product's cost, against 16
// times for the fp32 matrix instruction.  bf16 inputs are one plane, exactly.
// Only y with bf16 I/O is formed from two planes (16 bits): it is rounded to 8.
//
// Data flow inside a wave.  A wave owns 16 columns v of the state and keeps
// them in accumulators through the whole sequence.  A 16x16 result leaves lane
// l with column l % 16 and rows 4 (l / 16) + r; the next product wants, as its
// right operand, k = 8 (l / 16) + j of the same column.  The order of k inside
// a product and of the rows of a tile are free as long as both operands agree,
// so row m of tile t stands for index
//     32 (t / 2) + 8 (m / 4) + 4 (t % 2) + m % 4,
// and the results of tiles 2s, 2s + 1 ARE the right operand of k step s: no
// exchange between lanes, no LDS, anywhere on the recurrence's path.
//
// Left operands are laid out once per chunk as fragments (1 KiB: 64 lanes x 16
// bytes, in lane order) by delta_pack_kernel (keys and queries, per key head)
// and delta_solve_kernel (X and P, per value head).
#pragma once

#include "device_common.h"
#include "device_math.h"

namespace ssm {
namespace delta {

constexpr int kC = 64;             // steps per chunk
constexpr int kFrag = 512;         // bf16 elements of a fragment
constexpr int kTri = 6;            // fragments of a 64 x 64 triangle: (tile, k step) pairs that are not all zero
constexpr float kClear = -10000.f; // a log decay at or below this clears the state

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct Params {
    const void *q, *k, *v, *g, *beta;
    const float* h0;
    const int32_t* lengths;
    void* y;
    float* h_last;
    uint16_t *kf, *ktf, *qf, *qtf;  // [B][Hk][nC][planes][tiles][k steps] fragments (qtf: backward only)
    uint16_t *xf, *xtf;             // [B][Hv][nC][3][6]
    uint16_t *pf, *ptf;             // [B][Hv][nC][p_planes][6]
    float* vec;                     // [B][Hv][nC][3][64]: e^G, e^{G_63 - G}, beta
    float *states, *news;           // backward: states entering each chunk (K x VP), E^ of each step (64 x VP)
    int64_t B, L, Hk, Hv, K, V, nC;
    int64_t nV, VP;                 // 16-column tiles of the state, and their columns in all
    float scale;
};

__device__ __forceinline__ int tile_row(int t, int m) { return 32 * (t >> 1) + 8 * (m >> 2) + 4 * (t & 1) + (m & 3); }
// fragment of triangle (tile t, k step s): lower triangles have s <= t / 2, upper ones s >= t / 2
__device__ __forceinline__ int tri_lower(int t, int s) { return t < 2 ? t : 2 * t - 2 + s; }
__device__ __forceinline__ int tri_upper(int t, int s) { return t < 2 ? 2 * t + s : t + 2; }

__device__ __forceinline__ int row_len(const int32_t* lengths, int64_t b, int64_t L) {
    if (!lengths) return static_cast<int>(L);
    const int64_t n = lengths[b];
    return static_cast<int>(n < 0 ? 0 : n < L ? n : L);
}

// x split into N bf16 planes, largest first
template <int N>
struct Planes {
    bf16x8 p[N];
};

template <int N>
__device__ __forceinline__ void split8(const float (&x)[8], Planes<N>& o) {
    float r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = x[j];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            o.p[n][j] = static_cast<__bf16>(r[j]);
            if (n + 1 < N) r[j] -= static_cast<float>(o.p[n][j]);
        }
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// c += a b over the plane pairs (i, j) with i + j < LIM, smallest first
template <int LIM, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Planes<NA>& a, const Planes<NB>& b, f32x4 c) {
#pragma unroll
    for (int d = LIM - 1; d >= 0; --d)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (d - i >= 0 && d - i < NB) c = mfma(a.p[i], b.p[d - i], c);
    return c;
}

// fragment f of each plane, planes `stride` fragments apart
template <int N>
__device__ __forceinline__ Planes<N> frag(const uint16_t* base, int f, int stride, int lane) {
    Planes<N> o;
#pragma unroll
    for (int n = 0; n < N; ++n)
        o.p[n] = *reinterpret_cast<const bf16x8*>(base + static_cast<int64_t>(n * stride + f) * kFrag + lane * 8);
    return o;
}

template <int N>
__device__ __forceinline__ void put_frag(uint16_t* base, int f, int stride, int lane, const float (&x)[8]) {
    Planes<N> o;
    split8<N>(x, o);
#pragma unroll
    for (int n = 0; n < N; ++n)
        *reinterpret_cast<bf16x8*>(base + static_cast<int64_t>(n * stride + f) * kFrag + lane * 8) = o.p[n];
}

__device__ __forceinline__ f32x4 zero4() { return f32x4{0.f, 0.f, 0.f, 0.f}; }

template <typename T>
struct PlanesOf {  // planes of an input, and of what y and the products behind it are formed from
    static constexpr int kIn = 1, kOut = 2;
};
template <>
struct PlanesOf<float> {
    static constexpr int kIn = 3, kOut = 3;
};

// Keys and queries of a chunk as fragments: rows = steps (kf, qf) and rows =
// key elements (ktf, qtf).  Steps behind the row's length and elements behind
// K are zeros.
template <typename T, int KS, bool BWD>
__global__ void __launch_bounds__(256) delta_pack_kernel(Params p) {
    constexpr int kN = PlanesOf<T>::kIn, kRow = 32 * KS + 2;
    __shared__ float s_x[kC][kRow];
    const int tid = threadIdx.x;
    const int64_t c = blockIdx.x % p.nC, bh = blockIdx.x / p.nC, b = bh / p.Hk, h = bh % p.Hk;
    const int64_t t0 = c * kC;
    const int64_t len = row_len(p.lengths, b, p.L);
    if (t0 >= len) return;
    const int64_t unit = static_cast<int64_t>(kN) * 4 * KS * kFrag, at = static_cast<int64_t>(blockIdx.x) * unit;
    for (int which = 0; which < 2; ++which) {
        const T* src = static_cast<const T*>(which ? p.q : p.k);
        for (int i = tid; i < kC * 32 * KS; i += 256) {
            const int t = i / (32 * KS), e = i % (32 * KS);
            const bool ok = t0 + t < len && e < p.K;
            s_x[t][e] = ok ? Elem<T>::load(src, ((b * p.L + t0 + t) * p.Hk + h) * p.K + e) : 0.f;
        }
        __syncthreads();
        uint16_t* rows = (which ? p.qf : p.kf) + at;
        uint16_t* cols = which ? (BWD ? p.qtf + at : nullptr) : p.ktf + at;
        for (int i = tid; i < 4 * KS * 64; i += 256) {
            const int lane = i & 63, f = i >> 6, t = f / KS, s = f % KS;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = s_x[tile_row(t, lane & 15)][32 * s + 8 * (lane >> 4) + j];
            put_frag<kN>(rows, f, 4 * KS, lane, x);
        }
        if (cols)
            for (int i = tid; i < 4 * KS * 64; i += 256) {
                const int lane = i & 63, f = i >> 6, t = f / 2, s = f % 2;
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = s_x[32 * s + 8 * (lane >> 4) + j][tile_row(t, lane & 15)];
                put_frag<kN>(cols, f, 4 * KS, lane, x);
            }
        __syncthreads();
    }
}

// Decays, X and P of a chunk.  The running sums of g are fp64 (their
// differences, not their size, set a decay's error).
template <typename T, int KS, bool BWD>
__global__ void __launch_bounds__(256) delta_solve_kernel(Params p) {
    constexpr int kN = PlanesOf<T>::kIn, kP = BWD ? 3 : PlanesOf<T>::kOut, kRow = kC + 4;
    __shared__ float s_a[kC][kRow], s_p[kC][kRow];
    __shared__ double s_g[kC];
    __shared__ float s_b[kC];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t c = blockIdx.x % p.nC, bh = blockIdx.x / p.nC, b = bh / p.Hv, h = bh % p.Hv;
    const int64_t t0 = c * kC;
    const int64_t len = row_len(p.lengths, b, p.L);
    if (t0 >= len) return;
    const int64_t kunit = static_cast<int64_t>(kN) * 4 * KS * kFrag;
    const int64_t kat = ((b * p.Hk + h / (p.Hv / p.Hk)) * p.nC + c) * kunit;
    if (wave == 0) {
        const bool ok = t0 + lane < len;
        const int64_t i = (b * p.L + t0 + lane) * p.Hv + h;
        const float g = ok ? Elem<T>::load(static_cast<const T*>(p.g), i) : 0.f;
        const float be = ok ? Elem<T>::load(static_cast<const T*>(p.beta), i) : 0.f;
        double G = g < kClear ? kClear : g;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const double o = __shfl_up(G, off, 64);
            if (lane >= off) G += o;
        }
        const double last = __shfl(G, 63, 64);
        s_g[lane] = G;
        s_b[lane] = be;
        float* vec = p.vec + static_cast<int64_t>(blockIdx.x) * 3 * kC;
        vec[lane] = expf(static_cast<float>(G));
        vec[kC + lane] = expf(static_cast<float>(last - G));
        vec[2 * kC + lane] = be;
    }
    __syncthreads();
    // rows of tile `wave` against the steps not behind them
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) kk[t] = qk[t] = zero4();
    const int ntile = wave < 2 ? 2 : 4;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const Planes<kN> ka = frag<kN>(p.kf + kat, wave * KS + s, 4 * KS, lane);
        const Planes<kN> qa = frag<kN>(p.qf + kat, wave * KS + s, 4 * KS, lane);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < ntile) {
                const Planes<kN> kb = frag<kN>(p.kf + kat, t * KS + s, 4 * KS, lane);
                kk[t] = mma<3>(ka, kb, kk[t]);
                qk[t] = mma<3>(qa, kb, qk[t]);
            }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int j = tile_row(t, lane & 15);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = tile_row(wave, 4 * (lane >> 4) + r);
            const float e = j <= i ? expf(static_cast<float>(s_g[i] - s_g[j])) : 0.f;
            s_a[i][j] = j < i ? kk[t][r] * e : 0.f;
            s_p[i][j] = j <= i ? qk[t][r] * e * p.scale : 0.f;
        }
    }
    __syncthreads();
    if (wave == 0) {
        // X_i = A'_i - sum_{l < i} A'_il beta_l X_l, lane j holding column j; row i of A' is
        // read whole before the lanes put X_i in its place
        float x[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) {
            float acc = s_a[i][lane];
#pragma unroll
            for (int l = 0; l < i; ++l) acc -= s_a[i][l] * s_b[l] * x[l];
            x[i] = acc;
            __builtin_amdgcn_wave_barrier();
            s_a[i][lane] = acc;
            __builtin_amdgcn_wave_barrier();
        }
    }
    __syncthreads();
    uint16_t* xf = p.xf + static_cast<int64_t>(blockIdx.x) * 3 * kTri * kFrag;
    uint16_t* pf = p.pf + static_cast<int64_t>(blockIdx.x) * kP * kTri * kFrag;
    for (int i = tid; i < 8 * 64; i += 256) {
        const int l = i & 63, t = i >> 7, s = (i >> 6) & 1;
        float x[8];
        if (s <= t / 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = s_a[tile_row(t, l & 15)][32 * s + 8 * (l >> 4) + j];
            put_frag<3>(xf, tri_lower(t, s), kTri, l, x);
            if (!BWD) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = s_p[tile_row(t, l & 15)][32 * s + 8 * (l >> 4) + j];
                put_frag<kP>(pf, tri_lower(t, s), kTri, l, x);
            }
        }
        if (BWD && s >= t / 2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = s_a[32 * s + 8 * (l >> 4) + j][tile_row(t, l & 15)];
            put_frag<3>(p.xtf + static_cast<int64_t>(blockIdx.x) * 3 * kTri * kFrag, tri_upper(t, s), kTri, l, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = s_p[32 * s + 8 * (l >> 4) + j][tile_row(t, l & 15)];
            put_frag<3>(p.ptf + static_cast<int64_t>(blockIdx.x) * 3 * kTri * kFrag, tri_upper(t, s), kTri, l, x);
        }
    }
}

// 8 consecutive floats of `base` (16-byte aligned)
__device__ __forceinline__ void load8(const float* base, float (&x)[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(base), b = *reinterpret_cast<const f32x4*>(base + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = a[j], x[4 + j] = b[j];
}

// A wave's 16 columns of the state, as accumulator tiles
template <int KS>
__device__ __forceinline__ void load_state(const float* h, int64_t K, bool ok, int lane, f32x4 (&S)[2 * KS]) {
    const int q = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int e = 32 * (t >> 1) + 8 * q + 4 * (t & 1) + r;
            S[t][r] = h && ok && e < K ? h[e] : 0.f;
        }
}

template <int KS>
__device__ __forceinline__ void store_state(float* h, int64_t K, bool ok, int lane, const f32x4 (&S)[2 * KS]) {
    const int q = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int e = 32 * (t >> 1) + 8 * q + 4 * (t & 1) + r;
            if (ok && e < K) h[e] = S[t][r];
        }
}

// The recurrence over chunks: one wave per 16 columns of a head's state.
// OUT: writes y and h_last (the forward); else the states entering each chunk
// and E^ (what the gradients read).
template <typename T, int KS, bool OUT>
__global__ void __launch_bounds__(64) delta_chunk_kernel(Params p) {
    constexpr int kN = PlanesOf<T>::kIn, kO = PlanesOf<T>::kOut;
    const int lane = threadIdx.x, q = lane >> 4;
    const int64_t VP = p.VP, vt = blockIdx.x % p.nV, bh = blockIdx.x / p.nV, b = bh / p.Hv, h = bh % p.Hv;
    const int64_t col = vt * 16 + (lane & 15);
    const bool ok = col < p.V;
    const int64_t len = row_len(p.lengths, b, p.L);
    f32x4 S[2 * KS];
    load_state<KS>(p.h0 ? p.h0 + (bh * p.V + (ok ? col : 0)) * p.K : nullptr, p.K, ok, lane, S);
    const T* v = static_cast<const T*>(p.v);
    T* y = static_cast<T*>(p.y);
    const int64_t kunit = static_cast<int64_t>(kN) * 4 * KS * kFrag;
    const int64_t kat = (b * p.Hk + h / (p.Hv / p.Hk)) * p.nC * kunit;
    for (int64_t c = 0; c * kC < len; ++c) {
        const int64_t t0 = c * kC, bhc = bh * p.nC + c;
        const uint16_t *kf = p.kf + kat + c * kunit, *ktf = p.ktf + kat + c * kunit, *qf = p.qf + kat + c * kunit;
        const uint16_t *xf = p.xf + bhc * 3 * kTri * kFrag, *pf = p.pf + bhc * kO * kTri * kFrag;
        const float* vec = p.vec + bhc * 3 * kC;
        if constexpr (!OUT) {
            float* st = p.states + bhc * (32 * KS) * VP + col;
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) st[(32 * (t >> 1) + 8 * q + 4 * (t & 1) + r) * VP] = S[t][r];
        }
        Planes<3> Sp[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = S[2 * s + (j >> 2)][j & 3];
            split8<3>(x, Sp[s]);
        }
        // E^ and U, two row tiles (32 steps) at a time: lane's steps 32 s + 8 q + 0 .. 7
        float E[2][8], be[2][8];
        Planes<3> Y[2];
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
            f32x4 ks[2] = {zero4(), zero4()};
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    ks[t] = mma<3>(frag<kN>(kf, (2 * s2 + t) * KS + s, 4 * KS, lane), Sp[s], ks[t]);
            float ga[8], x[8];
            load8(vec + 32 * s2 + 8 * q, ga);
            load8(vec + 2 * kC + 32 * s2 + 8 * q, be[s2]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t t = t0 + 32 * s2 + 8 * q + j;
                const float vv = ok && t < len ? Elem<T>::load(v, ((b * p.L + t) * p.Hv + h) * p.V + col) : 0.f;
                E[s2][j] = vv - ga[j] * ks[j >> 2][j & 3];
                x[j] = be[s2][j] * E[s2][j];
            }
            split8<3>(x, Y[s2]);
        }
        Planes<kO> U[2];
        Planes<3> W[2];
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
            float x[8], w[8];
            load8(vec + kC + 32 * s2 + 8 * q, w);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                f32x4 a = zero4();
#pragma unroll
                for (int s = 0; s <= s2; ++s)
                    a = mma<3>(frag<3>(xf, tri_lower(2 * s2 + t, s), kTri, lane), Y[s], a);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float e = E[s2][4 * t + r] - a[r];
                    if constexpr (!OUT)
                        p.news[(bhc * kC + 32 * s2 + 8 * q + 4 * t + r) * VP + col] = e;
                    x[4 * t + r] = be[s2][4 * t + r] * e;
                    w[4 * t + r] *= x[4 * t + r];
                }
            }
            split8<kO>(x, U[s2]);
            split8<3>(w, W[s2]);
        }
        if constexpr (OUT) {
#pragma unroll
            for (int s2 = 0; s2 < 2; ++s2) {
                float ga[8];
                load8(vec + 32 * s2 + 8 * q, ga);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x4 a = zero4();
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        a = mma<kO>(frag<kN>(qf, (2 * s2 + t) * KS + s, 4 * KS, lane), Sp[s], a);
#pragma unroll
                    for (int r = 0; r < 4; ++r) a[r] *= ga[4 * t + r] * p.scale;
#pragma unroll
                    for (int s = 0; s <= s2; ++s)
                        a = mma<kO>(frag<kO>(pf, tri_lower(2 * s2 + t, s), kTri, lane), U[s], a);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int64_t i = t0 + 32 * s2 + 8 * q + 4 * t + r;
                        if (ok && i < len) Elem<T>::store(y, ((b * p.L + i) * p.Hv + h) * p.V + col, a[r]);
                    }
                }
            }
        }
        const float end = vec[kC - 1];
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) {
            f32x4 a = S[t] * end;
#pragma unroll
            for (int s = 0; s < 2; ++s) a = mma<3>(frag<kN>(ktf, 2 * t + s, 4 * KS, lane), W[s], a);
            S[t] = a;
        }
    }
    if (OUT && p.h_last) store_state<KS>(p.h_last + (bh * p.V + (ok ? col : 0)) * p.K, p.K, ok, lane, S);
}

// ---- the decode step.  Eight lanes share a row v of the state, lane i of them
// holding the float4 pieces i, i + 8, ... of its K elements (VEC; single
// elements i, i + 8, ... otherwise); a workgroup has 32 rows of one head.  The
// state is read once and written once: 8 V K bytes per head, all of the cost.
struct StepParams {
    const void *q, *k, *v, *g, *beta;
    float* h;
    void* y;
    int64_t B, Hk, Hv, K, V, row_blocks;
    float scale;
};

// sum over the 8 lanes of a row
__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor(x, 1, 64);
    x += __shfl_xor(x, 2, 64);
    x += __shfl_xor(x, 4, 64);
    return x;
}

template <typename T, int NP, bool VEC>
__global__ void __launch_bounds__(256) delta_step_kernel(StepParams p) {
    const int lane = threadIdx.x & 7;
    const int64_t rb = blockIdx.x % p.row_blocks, bh = blockIdx.x / p.row_blocks, b = bh / p.Hv, h = bh % p.Hv;
    const int64_t row = rb * 32 + (threadIdx.x >> 3);
    const bool ok = row < p.V;
    float* hp = p.h + (bh * p.V + (ok ? row : 0)) * p.K;
    const int64_t kb = (b * p.Hk + h / (p.Hv / p.Hk)) * p.K;
    const T *kp = static_cast<const T*>(p.k) + kb, *qp = static_cast<const T*>(p.q) + kb;
    float s[NP][4], k[NP][4], q[NP][4];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        if constexpr (VEC) {
            const int e = 4 * (lane + 8 * n);
            const bool in = e < p.K;
            const f32x4 x = in && ok ? *reinterpret_cast<const f32x4*>(hp + e) : zero4();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[n][j] = x[j];
                k[n][j] = in ? Elem<T>::load(kp, e + j) : 0.f;
                q[n][j] = in ? Elem<T>::load(qp, e + j) : 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = lane + 8 * (4 * n + j);
                const bool in = e < p.K;
                s[n][j] = in && ok ? hp[e] : 0.f;
                k[n][j] = in ? Elem<T>::load(kp, e) : 0.f;
                q[n][j] = in ? Elem<T>::load(qp, e) : 0.f;
            }
        }
    }
    const float alpha = expf(Elem<T>::load(static_cast<const T*>(p.g), bh));
    const float beta = Elem<T>::load(static_cast<const T*>(p.beta), bh);
    const float v = Elem<T>::load(static_cast<const T*>(p.v), bh * p.V + (ok ? row : 0));
    float dot = 0.f;
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[n][j] *= alpha;
            dot += s[n][j] * k[n][j];
        }
    const float u = beta * (v - sum8(dot));
    float out = 0.f;
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[n][j] += u * k[n][j];
            out += s[n][j] * q[n][j];
        }
    out = sum8(out);
    if (!ok) return;
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        if constexpr (VEC) {
            const int e = 4 * (lane + 8 * n);
            if (e < p.K) *reinterpret_cast<f32x4*>(hp + e) = f32x4{s[n][0], s[n][1], s[n][2], s[n][3]};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int e = lane + 8 * (4 * n + j);
                if (e < p.K) hp[e] = s[n][j];
            }
        }
    }
    if (lane == 0) Elem<T>::store(static_cast<T*>(p.y), bh * p.V + row, p.scale * out);
}

}  // namespace delta
}  // namespace ssm
