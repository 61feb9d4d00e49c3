// cache_attend.cu -- exact softmax attention of a serving batch over each sequence's own cache
// (int8 or e4m3 codes with a scale per row, or bf16), all rows up to each query token's position
// or the selected ones, and the merge with the states of a shared prefix (prefix_attend.cu).
//
// "Nem Todos os Pensamentos Necessitam de HBM" (gist.science summary), Metodologia 1 (8-bit
// rows) and 3 (a row contributes the same terms wherever it is stored); "Esparsidade de
// Contexto no Tempo de Inferencia" (gist.science summary), sec. 2 (exact softmax over the
// attended rows); Adaptive DHiSparse (news page), "Metodologia" (query tokens share each
// fetched row).
//
// Mathematics.  z = scale * ks_t * (q . c_t), p = 2^(z log2 e - m), out = sum p vs_t c'_t / sum p.
// The codes enter the tensor cores as they are (int8 and e4m3 values are exact in fp16, e4m3
// scaled by 2^-8), the row scales multiply the logit and the weight in fp32.  The query row is
// scaled by a power of two to [1, 2) before it becomes fp16, which keeps 24 bits below its largest
// element.  The weight that multiplies a V row is p * vs_t, and its range is that of the scales: it is
// kept relative to a second running maximum, over z + exponent(vs_t), whose weights reach up to
// 2^15 in fp16 (so a weight 2^-39 times the largest still counts); with SD_F32 output
// as a sum of two fp16 numbers (22 bits), with SD_BF16 output as one (11 bits, below the
// output's own 8).  A bf16 cache uses bf16 operands, weights in two parts or one likewise.
//
// Bound: HBM.  So that nothing but the loads takes time, the rows go from global memory straight into
// registers in the operand layout of mma.sync m16n8k16, with no shared memory: the contraction
// over d may run in any order, so a lane takes 16 neighbouring bytes of its K rows as its elements
// of four k-steps (the query fragments are permuted alike), and the output columns may be in
// any order, so it takes 16 neighbouring columns of its four V rows.  Every load instruction then
// covers whole 64- or 128-byte lines.  S^T = K Q^T and O^T = V^T P^T put the 16 rows of a step on
// the M side and 8 query rows on the N side.  While a step is computed the next one's rows are on
// their way (2 x 2 KB a warp, 12 to 16 warps an SM).
//
// Work: units of 64 rows of one (sequence, KV head), in order, cut into equal runs, one a CTA
// (all resident at once), whatever the sequences' lengths.  A CTA's run covers one or more
// groups; a group that lies within one run is written directly, the others' states are merged
// by a second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "cache_attend.cuh"

namespace sd {
namespace {

constexpr int kCaThreads = 128;
constexpr int kCaWarps = kCaThreads / 32;

struct CaParams {
    const uint8_t* q;
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;
    const float* vs;
    const int32_t* qpos;
    const int32_t* idx;
    void* out;
    float* lse;
    int32_t* err;
    CaWorkspace ws;
    int B, V, Hq, Hkv, G, R, T, n_idx, block, n_list, P, pre_splits, out_bf16;
    float scale_log2;
};

enum { kBf16 = 0, kInt8 = 1, kE4m3 = 2 };

// ------------------------------------------------------------------ operands

// Bytes 0, 1 (hi: 2, 3) of w as two fp16: int8 from w ^ 0x80808080 (1024 + code + 128 as bits), e4m3 as
// value * 2^-8 (its exponent and mantissa bits moved into fp16's; exact, subnormals too; a NaN code
// gives 480 * 2^-8, never a NaN).
template <int KIND>
SD_DEVINL uint32_t widen(uint32_t w, bool hi) {
    if constexpr (KIND == kInt8) {
        const uint32_t t = __byte_perm(w, 0x64646464u, hi ? 0x4342 : 0x4140);
        const uint32_t c = 0x64806480u;
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&t), *reinterpret_cast<const __half2*>(&c));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        const uint32_t t = __byte_perm(w, 0u, hi ? 0x3424 : 0x1404);
        return (t & 0x80008000u) | ((t >> 1) & 0x3f803f80u);
    }
}
template <int KIND>
SD_DEVINL uint32_t biased(uint32_t w) {
    return KIND == kInt8 ? w ^ 0x80808080u : w;
}

SD_DEVINL uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A pair of weights as one 16-bit operand word, and what is left of them as another.
template <bool F16>
SD_DEVINL uint32_t weight_word(float x0, float x1, uint32_t* lo) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(x0, x1);
        if (lo != nullptr) {
            const float2 f = __half22float2(h);
            *lo = pack_f16x2(x0 - f.x, x1 - f.y);
        }
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        uint32_t hi, l;
        split_bf16x2(x0, x1, hi, l);
        if (lo != nullptr) *lo = l;
        return hi;
    }
}

template <bool F16>
SD_DEVINL void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
    else
        mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}

// 16 bytes (or 8) of a row read once: past L1, as data that nothing else wants (a verify batch
// of more than 16 query rows has two warps reading the same rows: they share them in L1).
SD_DEVINL uint4 ld_row16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
SD_DEVINL uint2 ld_row8(const uint8_t* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }

// ------------------------------------------------------------------ one step's rows

// 16 rows of K and V as this lane holds them.
template <int KIND, int D>
struct Rows {
    static constexpr int kEs = KIND == kBf16 ? 2 : 1;
    static constexpr int kKc = D * kEs / 64;  // 16-byte pieces of a K row a lane holds
    static constexpr int kVw = D * kEs / 32;  // 32-bit words of a V row a lane holds
    uint4 k[2][kKc];       // rows g8 and g8 + 8, bytes 64c + 16 t4 ..
    uint32_t v[4][kVw];    // rows 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9, columns g8 * D/8 ..
    float ks[2], vs[2];    // scales of rows g8 and g8 + 8
    int pos[2];            // their positions (INT_MAX: not attended by any query)

    SD_DEVINL void load_k(int h, const uint8_t* row, int t4) {
#pragma unroll
        for (int c = 0; c < kKc; ++c) k[h][c] = ld_row16(row + 64 * c + 16 * t4);
    }
    SD_DEVINL void load_v(int r, const uint8_t* row, int g8) {
        const uint8_t* p = row + g8 * (4 * kVw);
        if constexpr (kVw == 2) {
            const uint2 w = ld_row8(p);
            v[r][0] = w.x;
            v[r][1] = w.y;
        } else {
#pragma unroll
            for (int c = 0; c < kVw / 4; ++c) {
                const uint4 w = ld_row16(p + 16 * c);
                v[r][4 * c] = w.x;
                v[r][4 * c + 1] = w.y;
                v[r][4 * c + 2] = w.z;
                v[r][4 * c + 3] = w.w;
            }
        }
    }
};

// ------------------------------------------------------------------ a warp's state

template <int D, int NQ>
struct CaState {
    float o[D / 16][NQ][4];   // O^T: columns g8 * D/8 + 2 md (+1: entries 2, 3) of query 8nq + 2t4 + e
    float m[NQ][2], l[NQ][2]; // running max (base 2); this lane's share of the denominator
    float m2[NQ][2];          // 8-bit: running max of logit + exponent of the V scale
    SD_DEVINL void init() {
#pragma unroll
        for (int md = 0; md < D / 16; ++md)
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[md][nq][e] = 0.f;
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nq][e] = m2[nq][e] = -INFINITY;
                l[nq][e] = 0.f;
            }
    }
};

SD_DEVINL float max_over_rows(float x) {  // over the lanes of the same t4
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

// One step: S^T = K Q^T, the online softmax over the rows at or below each query's limit, then
// O^T += V^T P^T.  qs: each query's factor of the logit; lim: its last row (-1: none).
template <int KIND, int D, int NQ, bool HILO>
SD_DEVINL void ca_step(const Rows<KIND, D>& rw, const uint32_t (&qf)[D / 16][NQ][2], const float (&qs)[NQ][2],
                       const int (&lim)[NQ][2], CaState<D, NQ>& st) {
    constexpr bool F16 = KIND != kBf16;
    float s[NQ][4];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nq][e] = 0.f;
#pragma unroll
    for (int c = 0; c < Rows<KIND, D>::kKc; ++c) {
        const uint32_t w0[4] = {rw.k[0][c].x, rw.k[0][c].y, rw.k[0][c].z, rw.k[0][c].w};
        const uint32_t w1[4] = {rw.k[1][c].x, rw.k[1][c].y, rw.k[1][c].z, rw.k[1][c].w};
        if constexpr (F16) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t x0 = biased<KIND>(w0[kk]), x1 = biased<KIND>(w1[kk]);
                const uint32_t a0 = widen<KIND>(x0, false), a2 = widen<KIND>(x0, true);
                const uint32_t a1 = widen<KIND>(x1, false), a3 = widen<KIND>(x1, true);
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq)
                    mma16<F16>(s[nq], a0, a1, a2, a3, qf[4 * c + kk][nq][0], qf[4 * c + kk][nq][1]);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq)
                    mma16<F16>(s[nq], w0[2 * kk], w1[2 * kk], w0[2 * kk + 1], w1[2 * kk + 1], qf[2 * c + kk][nq][0],
                               qf[2 * c + kk][nq][1]);
        }
    }
    float ks[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f}, mant[2] = {1.f, 1.f};
    if constexpr (F16) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ks[h] = KIND == kE4m3 ? rw.ks[h] * 256.f : rw.ks[h];
            const uint32_t b = __float_as_uint(rw.vs[h]);
            const uint32_t e = (b >> 23) & 0xffu;
            ev[h] = (float)((int)e - 127);
            mant[h] = e == 0u ? 0.f : __uint_as_float((b & 0x7fffffu) | 0x3f800000u);  // scale = mant * 2^ev
        }
    }
    uint32_t ph[NQ][2], pl[NQ][2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float x[2];
            bool on[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                on[h] = rw.pos[h] <= lim[nq][e];
                const float f = F16 ? ks[h] * qs[nq][e] : qs[nq][e];
                x[h] = on[h] ? s[nq][2 * h + e] * f : -INFINITY;
            }
            const float mo = st.m[nq][e];
            const float mn = fmaxf(mo, max_over_rows(fmaxf(x[0], x[1])));
            const float ref = mn == -INFINITY ? 0.f : mn;
            const float p0 = fast_exp2(x[0] - ref), p1 = fast_exp2(x[1] - ref);
            float alpha = fast_exp2(mo - ref);
            st.m[nq][e] = mn;
            st.l[nq][e] = st.l[nq][e] * alpha + (p0 + p1);
            if constexpr (F16) {
                const float y0 = on[0] ? x[0] + ev[0] : -INFINITY, y1 = on[1] ? x[1] + ev[1] : -INFINITY;
                const float m2o = st.m2[nq][e];
                const float m2n = fmaxf(m2o, max_over_rows(fmaxf(y0, y1)));
                const float r2 = m2n == -INFINITY ? 0.f : m2n;
                alpha = fast_exp2(m2o - r2);
                st.m2[nq][e] = m2n;
                w[e] = on[0] ? fast_exp2(y0 - r2 + 14.f) * mant[0] : 0.f;
                w[2 + e] = on[1] ? fast_exp2(y1 - r2 + 14.f) * mant[1] : 0.f;
            } else {
                w[e] = p0;
                w[2 + e] = p1;
            }
            if (alpha != 1.f) {
#pragma unroll
                for (int md = 0; md < D / 16; ++md) {
                    st.o[md][nq][e] *= alpha;
                    st.o[md][nq][2 + e] *= alpha;
                }
            }
        }
        // P^T (rows by lane group) to the B operand (rows by lane pair)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t lo;
            ph[nq][h] = movmatrix_t(weight_word<F16>(w[2 * h], w[2 * h + 1], HILO ? &lo : nullptr));
            if constexpr (HILO) pl[nq][h] = movmatrix_t(lo);
        }
    }
    auto pv = [&](int md, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            mma16<F16>(st.o[md][nq], a0, a1, a2, a3, ph[nq][0], ph[nq][1]);
            if constexpr (HILO) mma16<F16>(st.o[md][nq], a0, a1, a2, a3, pl[nq][0], pl[nq][1]);
        }
    };
#pragma unroll
    for (int w = 0; w < Rows<KIND, D>::kVw; ++w) {
        const uint32_t A = rw.v[0][w], B = rw.v[1][w], C = rw.v[2][w], E = rw.v[3][w];
        if constexpr (F16) {
            const uint32_t l01 = biased<KIND>(__byte_perm(A, B, 0x5140)), l23 = biased<KIND>(__byte_perm(A, B, 0x7362));
            const uint32_t h01 = biased<KIND>(__byte_perm(C, E, 0x5140)), h23 = biased<KIND>(__byte_perm(C, E, 0x7362));
            pv(2 * w, widen<KIND>(l01, false), widen<KIND>(l01, true), widen<KIND>(h01, false), widen<KIND>(h01, true));
            pv(2 * w + 1, widen<KIND>(l23, false), widen<KIND>(l23, true), widen<KIND>(h23, false),
               widen<KIND>(h23, true));
        } else {
            pv(w, __byte_perm(A, B, 0x5410), __byte_perm(A, B, 0x7632), __byte_perm(C, E, 0x5410),
               __byte_perm(C, E, 0x7632));
        }
    }
}

// ------------------------------------------------------------------ the kernel

// Own rows sequence b has for its query tokens (up to the largest qpos).
SD_DEVINL int seq_len(const CaParams& p, int b) {
    int m = -1;
    for (int v = 0; v < p.V; ++v) m = max(m, p.qpos[(size_t)b * p.V + v]);
    return min(m, p.T - 1) + 1;
}
SD_DEVINL int tiles_of(int rows) { return max(1, (rows + kCaTile - 1) / kCaTile); }

SD_DEVINL void store_pair(void* out, bool bf16, size_t i, float x, float y) {  // elements i, i + 1 (i even)
    if (bf16)
        reinterpret_cast<uint32_t*>(out)[i / 2] = pack_bf16x2(x, y);
    else
        reinterpret_cast<float2*>(out)[i / 2] = make_float2(x, y);
}

template <int KIND, int D, int NQ, bool HILO, bool SEL, int MINB>
__global__ void __launch_bounds__(kCaThreads, MINB) cache_attend_kernel(const CaParams p) {
    constexpr bool F16 = KIND != kBf16;
    constexpr int kEs = Rows<KIND, D>::kEs;
    constexpr int kMd = D / 16;
    constexpr int kPitch = kMd * 18;  // a state row in shared memory: column g8*D/8 + 2md + j at 18 md + 2 g8 + j
    __shared__ float so[kCaWarps][8 * NQ][kPitch];
    __shared__ float2 sml[kCaWarps][8 * NQ];
    __shared__ int s_part[kCaWarps], s_b, s_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int c = (int)blockIdx.x;
    pdl_wait();  // the cache, qpos and q may be the preceding kernels' results
    pdl_launch_dependents();

    // this CTA's run of units: [w0, w1) of all groups' units in order; no CTA of the ncta that
    // take part has an empty run, so a group's runs are in consecutive slots
    long W;
    int ncta;
    int b, kvh, j, tb;
    long w0, w1;
    if constexpr (SEL) {
        tb = tiles_of(p.n_list);
        W = (long)p.B * p.Hkv * tb;
        ncta = (int)min((long)gridDim.x, W);
        if (c >= ncta) return;
        w0 = c * W / ncta;
        w1 = (c + 1) * W / ncta;
        const int g = (int)(w0 / tb);
        j = (int)(w0 - (long)g * tb);
        b = g / p.Hkv;
        kvh = g - b * p.Hkv;
    } else {
        int sum = 0;
        for (int i = tid; i < p.B; i += kCaThreads) sum += tiles_of(seq_len(p, i));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_part[warp] = sum;
        __syncthreads();
        W = ((long)s_part[0] + s_part[1] + s_part[2] + s_part[3]) * p.Hkv;
        ncta = (int)min((long)gridDim.x, W);
        if (c >= ncta) return;
        w0 = c * W / ncta;
        w1 = (c + 1) * W / ncta;
        // the sequence of unit w0: sequence i's units start at Hkv * (tiles before it)
        int run = 0;
        for (int base = 0; base < p.B; base += kCaThreads) {
            const int i = base + tid;
            const int t = i < p.B ? tiles_of(seq_len(p, i)) : 0;
            int incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            __syncthreads();
            if (lane == 31) s_part[warp] = incl;
            if (tid == 0) s_b = -1;
            __syncthreads();
            int before = run;
            for (int k = 0; k < warp; ++k) before += s_part[k];
            const long hi = (long)(before + incl) * p.Hkv, lo = hi - (long)t * p.Hkv;
            if (t > 0 && w0 >= lo && w0 < hi) {
                s_b = i;
                s_base = before + incl - t;
            }
            for (int k = 0; k < kCaWarps; ++k) run += s_part[k];
            __syncthreads();
            if (s_b >= 0) break;
        }
        b = s_b;
        tb = tiles_of(seq_len(p, b));
        const int off = (int)(w0 - (long)s_base * p.Hkv);
        kvh = off / tb;
        j = off - kvh * tb;
    }

    const int halves = p.R > 8 * NQ ? 2 : 1;  // warps 0, 1 and 2, 3 take the query rows' halves (R > 16)
    const int wh = kCaWarps / halves, half = warp / wh, w_in = warp - half * wh;
    for (long w = w0; w < w1;) {
        const int g = b * p.Hkv + kvh;
        const int len = seq_len(p, b);
        const int seg = (int)min((long)(tb - j), w1 - w);
        const int list = SEL ? p.n_list : len;
        const int j0 = j * kCaTile, j1 = len == 0 ? j0 : min(list, j0 + seg * kCaTile);

        // the query rows: 8nq + g8 of this half as B fragments
        uint32_t qf[kMd][NQ][2];
        float qs[NQ][2];
        int lim[NQ][2];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const int r = half * 8 * NQ + 8 * nq + g8;
            const bool have = r < p.R;
            const int v = have ? r / p.G : 0, gi = have ? r - v * p.G : 0;
            const uint8_t* qrow = p.q + (((size_t)b * p.V + v) * p.Hq + (size_t)kvh * p.G + gi) * (D * 2);
            if constexpr (F16) {
                uint32_t raw[kMd][2];
                uint32_t top = 0u;
#pragma unroll
                for (int cc = 0; cc < Rows<KIND, D>::kKc; ++cc)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {  // dims 64 cc + 16 t4 + 8 hh ..
                        const uint4 x = have ? ld_row16(qrow + 2 * (64 * cc + 16 * t4 + 8 * hh)) : make_uint4(0u, 0u, 0u, 0u);
                        raw[4 * cc + 2 * hh][0] = x.x;
                        raw[4 * cc + 2 * hh][1] = x.y;
                        raw[4 * cc + 2 * hh + 1][0] = x.z;
                        raw[4 * cc + 2 * hh + 1][1] = x.w;
                        top = max(top, max(max(x.x & 0x7fff0000u, (x.x << 16) & 0x7fff0000u),
                                           max(x.y & 0x7fff0000u, (x.y << 16) & 0x7fff0000u)));
                        top = max(top, max(max(x.z & 0x7fff0000u, (x.z << 16) & 0x7fff0000u),
                                           max(x.w & 0x7fff0000u, (x.w << 16) & 0x7fff0000u)));
                    }
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const uint32_t e = min(max(top >> 23, 1u), 253u);
                const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
                for (int k = 0; k < kMd; ++k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qf[k][nq][i] = pack_f16x2(bf16lo(raw[k][i]) * down, bf16hi(raw[k][i]) * down);
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2)
                    qs[nq][e2] = __shfl_sync(0xffffffffu, up * p.scale_log2, (2 * t4 + e2) * 4);
            } else {
#pragma unroll
                for (int cc = 0; cc < Rows<KIND, D>::kKc; ++cc) {  // dims 32 cc + 8 t4 ..
                    const uint4 x = have ? ld_row16(qrow + 2 * (32 * cc + 8 * t4)) : make_uint4(0u, 0u, 0u, 0u);
                    qf[2 * cc][nq][0] = x.x;
                    qf[2 * cc][nq][1] = x.y;
                    qf[2 * cc + 1][nq][0] = x.z;
                    qf[2 * cc + 1][nq][1] = x.w;
                }
                qs[nq][0] = qs[nq][1] = p.scale_log2;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int rr = half * 8 * NQ + 8 * nq + 2 * t4 + e;
                lim[nq][e] = rr < p.R ? min(p.qpos[(size_t)b * p.V + rr / p.G], p.T - 1) : -1;
            }
        }

        CaState<D, NQ> st;
        st.init();
        const uint8_t* kbase = p.kc + (size_t)g * p.T * (D * kEs);
        const uint8_t* vbase = p.vc + (size_t)g * p.T * (D * kEs);
        // lane l < 16 resolves list row l of a step (SEL): its position, or -1 (an empty slot, an
        // index outside the cache, a row no query sees)
        auto resolve = [&](int step) {
            int t = -1;
            const int i = j0 + 16 * step + (lane & 15);
            if (i < j1) {
                const int e = i / p.block;
                const long sel = p.idx[(size_t)g * p.n_idx + e];
                const long pos = sel * p.block + (i - e * p.block);
                if (sel != -1) {
                    if (sel < 0 || pos >= p.T)
                        report(p.err, SD_DEVERR_INDEX);
                    else if (pos < len)
                        t = (int)pos;
                }
            }
            return t;
        };
        auto fetch = [&](int step, int mine, Rows<KIND, D>& rw) {
            const int i0 = j0 + 16 * step;
            // list row i of the step as a position to read (always one that a query sees)
            auto at = [&](int i, int* pos) {
                if constexpr (SEL) {
                    const int t = __shfl_sync(0xffffffffu, mine, i);
                    if (pos != nullptr) *pos = t < 0 ? 0x7fffffff : t;
                    return max(t, 0);
                } else {
                    if (pos != nullptr) *pos = i0 + i;  // at or past len: above every limit
                    return min(i0 + i, len - 1);
                }
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = at(g8 + 8 * h, &rw.pos[h]);
                rw.load_k(h, kbase + (size_t)t * (D * kEs), t4);
                if constexpr (F16) {
                    rw.ks[h] = __ldg(p.ks + (size_t)g * p.T + t);
                    rw.vs[h] = __ldg(p.vs + (size_t)g * p.T + t);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = at(2 * t4 + (r & 1) + 8 * (r >> 1), nullptr);
                rw.load_v(r, vbase + (size_t)t * (D * kEs), g8);
            }
        };
        const int nsteps = (j1 - j0 + 15) / 16;
        if (w_in < nsteps) {
            Rows<KIND, D> cur, nxt;
            int mine = -1;
            if constexpr (SEL) mine = resolve(w_in);
            fetch(w_in, mine, nxt);
            if constexpr (SEL) mine = resolve(w_in + wh);
            for (int s = w_in; s < nsteps; s += wh) {
                cur = nxt;
                if (s + wh < nsteps) {
                    fetch(s + wh, mine, nxt);
                    if constexpr (SEL) mine = resolve(s + 2 * wh);
                }
                ca_step<KIND, D, NQ, HILO>(cur, qf, qs, lim, st);
            }
        }

        // the warps' states to shared memory, all relative to the softmax maximum m
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = st.l[nq][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                const int q = 8 * nq + 2 * t4 + e;
                float f = 1.f;
                if constexpr (F16)
                    f = st.m2[nq][e] == -INFINITY ? 0.f
                                                  : exp2f(st.m2[nq][e] - st.m[nq][e] - (KIND == kE4m3 ? 6.f : 14.f));
#pragma unroll
                for (int md = 0; md < kMd; ++md) {
                    so[warp][q][18 * md + 2 * g8] = st.o[md][nq][e] * f;
                    so[warp][q][18 * md + 2 * g8 + 1] = st.o[md][nq][2 + e] * f;
                }
                if (g8 == 0) sml[warp][q] = make_float2(st.m[nq][e], l);
            }
        __syncthreads();
        const bool whole = j == 0 && seg == tb && p.P == 0;
        const size_t slot = (size_t)c + g;
        for (int i = tid; i < p.R * (D / 2); i += kCaThreads) {
            const int r = i / (D / 2), d = 2 * (i - r * (D / 2));
            const int q = r % (8 * NQ), wb = r / (8 * NQ) * wh;
            const int gg = d / (D / 8), at = 18 * ((d - gg * (D / 8)) / 2) + 2 * gg;
            float M = -INFINITY;
            for (int k = 0; k < wh; ++k) M = fmaxf(M, sml[wb + k][q].x);
            float L = 0.f, x = 0.f, y = 0.f;
            if (M != -INFINITY)
                for (int k = 0; k < wh; ++k) {
                    const float2 ml = sml[wb + k][q];
                    const float f = exp2f(ml.x - M);
                    L = fmaf(ml.y, f, L);
                    x = fmaf(so[wb + k][q][at], f, x);
                    y = fmaf(so[wb + k][q][at + 1], f, y);
                }
            if (whole) {
                const int v = r / p.G;
                const size_t row = ((size_t)b * p.V + v) * p.Hq + (size_t)kvh * p.G + (r - v * p.G);
                const float inv = L > 0.f ? 1.f / L : 0.f;
                store_pair(p.out, p.out_bf16 != 0, row * D + d, x * inv, y * inv);
                if (d == 0) p.lse[row] = L > 0.f ? (M + log2f(L)) * 0.69314718055994530942f : -INFINITY;
            } else {
                reinterpret_cast<float2*>(p.ws.o)[((slot * p.R + r) * D + d) / 2] = make_float2(x, y);
                if (d == 0) p.ws.ml[slot * p.R + r] = make_float2(M, L);
            }
        }
        if (j == 0 && tid == 0) {
            // the group's last unit w + tb - 1 is of CTA ((w + tb) * ncta - 1) / W
            const int last = (int)(((w + tb) * ncta - 1) / W);
            p.ws.meta[g] = make_int2(c + g, last - c + 1);
        }
        __syncthreads();
        w += seg;
        j = 0;
        if (++kvh == p.Hkv) {
            kvh = 0;
            ++b;
            if (!SEL && w < w1) tb = tiles_of(seq_len(p, b));
        }
    }
}

// One warp a query row: the states of its group's runs and of the prefix's splits into the output.
template <int D>
__global__ void __launch_bounds__(kCaThreads) cache_merge_kernel(const CaParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long row = (long)blockIdx.x * kCaWarps + (threadIdx.x >> 5);  // (b, v, h)
    if (row >= (long)p.B * p.V * p.Hq) return;
    const int h = (int)(row % p.Hq);
    const long bv = row / p.Hq;
    const int b = (int)(bv / p.V), v = (int)(bv - (long)b * p.V);
    const int kvh = h / p.G, gi = h - kvh * p.G, r = v * p.G + gi;
    const int2 own = p.ws.meta[(size_t)b * p.Hkv + kvh];
    const int n = own.y + p.pre_splits;
    if (own.y == 1 && p.P == 0) return;  // written by the CTA that had the whole group
    const size_t M = (size_t)p.B * p.R, mrow = (size_t)bv * p.G + gi;
    auto ml_of = [&](int i) {
        return i < own.y ? p.ws.ml[(size_t)(own.x + i) * p.R + r]
                         : p.ws.pre_ml[((size_t)kvh * p.pre_splits + (i - own.y)) * M + mrow];
    };
    auto o_of = [&](int i) {
        return i < own.y ? p.ws.o + ((size_t)(own.x + i) * p.R + r) * D
                         : p.ws.pre_o + (((size_t)kvh * p.pre_splits + (i - own.y)) * M + mrow) * D;
    };
    float mx = -INFINITY;
    for (int i = lane; i < n; i += 32) mx = fmaxf(mx, ml_of(i).x);
    mx = warp_max(mx);
    const float ref = mx == -INFINITY ? 0.f : mx;
    constexpr int kE = D / 32;  // columns a lane holds
    float acc[kE] = {}, L = 0.f;
    for (int base = 0; base < n; base += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (base + lane < n) ml = ml_of(base + lane);
        const float f = exp2f(ml.x - ref);  // 0 for a state without rows
        L = fmaf(ml.y, f, L);
        const int cnt = min(32, n - base);
#pragma unroll 8
        for (int k = 0; k < cnt; ++k) {
            const float fk = __shfl_sync(0xffffffffu, f, k);
            const float* o = o_of(base + k) + kE * lane;
            if constexpr (kE == 4) {
                const float4 x = *reinterpret_cast<const float4*>(o);
                acc[0] = fmaf(x.x, fk, acc[0]);
                acc[1] = fmaf(x.y, fk, acc[1]);
                acc[2] = fmaf(x.z, fk, acc[2]);
                acc[3] = fmaf(x.w, fk, acc[3]);
            } else {
                const float2 x = *reinterpret_cast<const float2*>(o);
                acc[0] = fmaf(x.x, fk, acc[0]);
                acc[1] = fmaf(x.y, fk, acc[1]);
            }
        }
    }
    L = warp_sum(L);
    const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
    for (int e = 0; e < kE; e += 2)
        store_pair(p.out, p.out_bf16 != 0, (size_t)row * D + kE * lane + e, acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) p.lse[row] = L > 0.f ? (mx + log2f(L)) * 0.69314718055994530942f : -INFINITY;
}

// CTAs an SM holds of a variant (its __launch_bounds__): what its registers allow without spills
// (8-bit codes, d = 128: 168 and 240 registers a thread for one and two query tiles).
constexpr int ca_ctas_per_sm(int kind, int d, int nq) {
    return kind == kBf16 ? (d == 64 && nq == 1 ? 3 : 2) : (d == 64 ? 5 : 4) - nq;
}

int ca_kind(const sd_cache_attend_args* a) {
    return a->cache_dtype == SD_I8 ? kInt8 : a->cache_dtype == SD_E4M3 ? kE4m3 : kBf16;
}

CaPlan ca_plan(const sd_cache_attend_args* a) {
    CaPlan pl{};
    const long NG = (long)a->B * a->Hkv;
    const int R = (a->Hq / a->Hkv) * a->V;
    const long rows = a->idx != nullptr ? (long)a->n_idx * a->block : a->T;
    const long units = NG * std::max<long>(1, (rows + kCaTile - 1) / kCaTile);
    pl.ctas = (int)std::min<long>(units, (long)num_sms() * ca_ctas_per_sm(ca_kind(a), a->d, R <= 8 ? 1 : 2));
    pl.slots = (int)(pl.ctas + NG - 1);
    pl.pre_splits = a->P > 0 ? prefix_splits(a) : 0;
    return pl;
}

sd_status ca_validate(const sd_cache_attend_args* a, bool pointers) {
    const char* who = "sd_cache_attend";
    SD_REQUIRE(a != nullptr, "%s: null args", who);
    SD_REQUIRE(a->cache_dtype == SD_BF16 || a->cache_dtype == SD_I8 || a->cache_dtype == SD_E4M3,
               "%s: cache_dtype must be SD_BF16, SD_I8 or SD_E4M3", who);
    SD_REQUIRE(a->out_dtype == SD_F32 || a->out_dtype == SD_BF16, "%s: out_dtype must be SD_F32 or SD_BF16", who);
    SD_REQUIRE(a->B >= 0 && a->V >= 1 && a->Hkv >= 1 && a->Hq >= 1 && a->Hq % a->Hkv == 0 && a->T >= 1 && a->P >= 0,
               "%s: bad sizes (B=%d V=%d Hq=%d Hkv=%d T=%d P=%d)", who, a->B, a->V, a->Hq, a->Hkv, a->T, a->P);
    SD_REQUIRE(a->B <= 65535 && a->Hq <= 65535, "%s: B and Hq must be <= 65535", who);
    SD_REQUIRE(a->idx == nullptr || (a->n_idx >= 0 && a->block >= 1 && (long)a->n_idx * a->block < (1L << 31)),
               "%s: bad selection (n_idx=%d block=%d)", who, a->n_idx, a->block);
    if (a->d != 64 && a->d != 128) {
        set_error("%s: d must be 64 or 128 (got %d)", who, a->d);
        return SD_ERR_UNSUPPORTED;
    }
    if ((a->Hq / a->Hkv) * (long)a->V > 32) {
        set_error("%s: (Hq/Hkv)*V must be <= 32 (got %d)", who, (a->Hq / a->Hkv) * a->V);
        return SD_ERR_UNSUPPORTED;
    }
    SD_REQUIRE(a->scale > 0.f && a->scale < 1e30f, "%s: scale must be positive", who);
    SD_REQUIRE((long)a->B * a->V * a->Hq < (1L << 30) && (long)a->Hkv * a->P < (1L << 31), "%s: too many query or prefix rows",
               who);
    const long rows = a->idx != nullptr ? (long)a->n_idx * a->block : a->T;
    SD_REQUIRE((long)a->B * a->Hkv * (rows / kCaTile + 1) < (1L << 31), "%s: too many rows", who);
    if (!pointers || a->B == 0) return SD_OK;
    SD_REQUIRE(a->q && a->k_cache && a->v_cache && a->qpos && a->out && a->lse, "%s: null pointer", who);
    SD_REQUIRE(a->cache_dtype == SD_BF16 || (a->k_scale && a->v_scale), "%s: an 8-bit cache needs k_scale and v_scale",
               who);
    SD_REQUIRE(a->P == 0 || (a->k_prefix && a->v_prefix), "%s: P > 0 needs k_prefix and v_prefix", who);
    SD_REQUIRE(aligned16(a->q) && aligned16(a->k_cache) && aligned16(a->v_cache) && aligned16(a->out) &&
                   aligned16(a->k_prefix) && aligned16(a->v_prefix),
               "%s: q, cache, prefix and out must be 16-byte aligned", who);
    return SD_OK;
}

template <int KIND, int D, int NQ, bool HILO>
sd_status ca_launch(const CaParams& p, const CaPlan& pl, cudaStream_t st) {
    constexpr int kMinB = ca_ctas_per_sm(KIND, D, NQ);
    const dim3 grid((unsigned)pl.ctas), block(kCaThreads);
    cudaError_t e = p.idx != nullptr
                        ? launch_pdl(cache_attend_kernel<KIND, D, NQ, HILO, true, kMinB>, grid, block, 0, st, p)
                        : launch_pdl(cache_attend_kernel<KIND, D, NQ, HILO, false, kMinB>, grid, block, 0, st, p);
    SD_CUDA_CHECK(e, "sd_cache_attend: launch");
    return launch_status("sd_cache_attend");
}

template <int KIND, int D>
sd_status ca_dispatch(const CaParams& p, const CaPlan& pl, cudaStream_t st) {
    if (p.out_bf16)
        return p.R <= 8 ? ca_launch<KIND, D, 1, false>(p, pl, st) : ca_launch<KIND, D, 2, false>(p, pl, st);
    return p.R <= 8 ? ca_launch<KIND, D, 1, true>(p, pl, st) : ca_launch<KIND, D, 2, true>(p, pl, st);
}

}  // namespace
}  // namespace sd

using namespace sd;

extern "C" size_t sd_cache_attend_workspace_bytes(const sd_cache_attend_args* a) {
    clear_error();
    if (ca_validate(a, false) != SD_OK || a->B == 0) return 0;
    return ca_workspace(a, ca_plan(a), nullptr).bytes;
}

extern "C" sd_status sd_cache_attend(const sd_cache_attend_args* a, void* stream) {
    clear_error();
    const char* who = "sd_cache_attend";
    sd_status st = ca_validate(a, true);
    if (st != SD_OK) return st;
    if (a->B == 0) return SD_OK;
    const CaPlan pl = ca_plan(a);
    const CaWorkspace w = ca_workspace(a, pl, a->workspace);
    SD_REQUIRE(a->workspace != nullptr && a->workspace_bytes >= w.bytes, "%s: workspace of %zu bytes needed (got %zu)",
               who, w.bytes, a->workspace_bytes);
    SD_REQUIRE((reinterpret_cast<uintptr_t>(a->workspace) & 255u) == 0, "%s: the workspace must be 256-byte aligned", who);
    CaParams p{};
    p.q = static_cast<const uint8_t*>(a->q);
    p.kc = static_cast<const uint8_t*>(a->k_cache);
    p.vc = static_cast<const uint8_t*>(a->v_cache);
    p.ks = a->k_scale;
    p.vs = a->v_scale;
    p.qpos = a->qpos;
    p.idx = a->idx;
    p.out = a->out;
    p.lse = a->lse;
    p.err = a->err_word;
    p.ws = w;
    p.B = a->B;
    p.V = a->V;
    p.Hq = a->Hq;
    p.Hkv = a->Hkv;
    p.G = a->Hq / a->Hkv;
    p.R = p.G * a->V;
    p.T = a->T;
    p.n_idx = a->n_idx;
    p.block = a->block;
    p.n_list = a->idx != nullptr ? a->n_idx * a->block : 0;
    p.P = a->P;
    p.pre_splits = pl.pre_splits;
    p.out_bf16 = a->out_dtype == SD_BF16;
    p.scale_log2 = a->scale * 1.44269504088896340736f;
    cudaStream_t cs = as_stream(stream);
    if (a->P > 0) {
        st = prefix_launch(a, pl.pre_splits, w, cs);
        if (st != SD_OK) return st;
    }
    const bool d128 = a->d == 128;
    switch (ca_kind(a)) {
        case kInt8: st = d128 ? ca_dispatch<kInt8, 128>(p, pl, cs) : ca_dispatch<kInt8, 64>(p, pl, cs); break;
        case kE4m3: st = d128 ? ca_dispatch<kE4m3, 128>(p, pl, cs) : ca_dispatch<kE4m3, 64>(p, pl, cs); break;
        default: st = d128 ? ca_dispatch<kBf16, 128>(p, pl, cs) : ca_dispatch<kBf16, 64>(p, pl, cs); break;
    }
    if (st != SD_OK) return st;
    const long rows = (long)a->B * a->V * a->Hq;
    const dim3 grid((unsigned)((rows + kCaWarps - 1) / kCaWarps));
    SD_CUDA_CHECK(launch_pdl(d128 ? cache_merge_kernel<128> : cache_merge_kernel<64>, grid, dim3(kCaThreads), 0, cs, p),
                  "sd_cache_attend: merge launch");
    return launch_status(who);
}
