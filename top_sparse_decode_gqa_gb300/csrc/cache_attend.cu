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
// The codes enter the tensor cores as they are (int8 and e4m3 values are exact in fp16), the row
// scales multiply the logit and the weight in fp32.  The query row is scaled by a power of two
// to [1, 2) before it becomes fp16, which keeps 24 bits below its largest element.  The weight that
// multiplies a V row is p * vs_t, and its range is that of the scales: it is kept relative to a
// second maximum, over z + log2(vs_t), whose weights are 2^10 in fp16 (and up to 2^15, see
// below; a weight 2^-34 times the largest still counts); with SD_F32 output as a sum of two
// fp16 numbers (22 bits), with SD_BF16 output as one (11 bits, below the output's own 8).  A bf16
// cache uses bf16 operands, weights in two parts or one likewise.
// The maxima need not be exact, only near: they move when a step's weights would pass 2^4 times
// what they stand for, which one vote a step finds out; until then no value crosses lanes.
// The tensor cores cut what they add to a sum (2^-24 of it), so SD_F32 output folds the
// accumulators into fp32 sums in shared memory every 32 steps (a 131072-row cache: 1.5e-5 of
// error in the output without, 1e-6 with).
//
// Bound: HBM; for more than 16 query rows the tensor cores' mma.sync rate comes close (8 cycles an
// instruction: 174 us against 163 us of loads for 4 x 131072 int8 rows and 32 query rows in two-part
// weights; the kernel takes 421, waiting for instructions: about 500 a warp and step, 12 warps an SM).  8 ragged
// e4m3 caches of 346 MB: 59 us, 5.9 TB/s.  A warp takes 8 or 16 query rows; for 17 to 32 two warps make a team that shares the
// fetched rows.  A team copies its steps of 16 K and V rows into a ring of 2 or 3 stages of its own
// (cp.async), so loads of the next steps are in flight through this one's arithmetic and no barrier is
// wider than a team.  The contraction over d may run in any order, so a lane takes 16 neighbouring
// bytes of its K rows as its elements of four k-steps of mma.sync m16n8k16 (the query fragments are
// permuted alike), and the output columns may be in any order, so it takes neighbouring columns of
// its four V rows: whole 8- or 16-byte reads, spread over the banks by a swizzle and the order of rows.
// S^T = K Q^T and O^T = V^T P^T put the 16 rows of a step on the M side and 8 query rows on the N
// side: a row's codes are widened once for all the query rows of the warp.
//
// Work: units of 64 rows of one (sequence, KV head), in order, cut into equal runs, one a CTA
// (all resident at once), whatever the sequences' lengths.  A group counts for two units more than it has,
// which is about what its queries, its start and its end cost (without: the CTAs of the shortest of 64
// sequences of 51 to 512 rows had 8 groups each and set the kernel's time).  A CTA's run covers one or more
// groups; a group that lies within one run is written directly, the others' states are merged
// by a second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "cache_attend.cuh"
#include "tc_operands.cuh"

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
    PrefixPlan pre;
    int B, V, Hq, Hkv, G, R, T, n_idx, block, n_list, P, out_bf16;
    float scale_log2;
};

enum { kBf16 = 0, kInt8 = 1, kE4m3 = 2 };

// ------------------------------------------------------------------ operands

// Bytes 0, 1 (hi: 2, 3) of w as two fp16: int8 from w ^ 0x80808080 (1024 + code + 128 as bits),
// e4m3 by the conversion instruction.
template <int KIND>
SD_DEVINL uint32_t widen(uint32_t w, bool hi) {
    if constexpr (KIND == kInt8) {
        const uint32_t t = __byte_perm(w, 0x64646464u, hi ? 0x4342 : 0x4140);
        const uint32_t c = 0x64806480u;
        const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&t), *reinterpret_cast<const __half2*>(&c));
        return *reinterpret_cast<const uint32_t*>(&r);
    } else {
        uint32_t r;
        const uint16_t b = (uint16_t)(hi ? w >> 16 : w);
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
        return r;
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

// A pair of weights as one 16-bit operand word, and (HILO) what is left of them as another.
template <bool F16, bool HILO>
SD_DEVINL void weight_words(float x0, float x1, uint32_t& hi, uint32_t& lo) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(x0, x1);
        hi = *reinterpret_cast<const uint32_t*>(&h);
        if constexpr (HILO) {
            const float2 f = __half22float2(h);
            lo = pack_f16x2(x0 - f.x, x1 - f.y);
        }
    } else if constexpr (HILO) {
        split_bf16x2(x0, x1, hi, lo);
    } else {
        hi = pack_bf16x2(x0, x1);
    }
}

template <bool F16>
SD_DEVINL void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_f16_16816(d, a0, a1, a2, a3, b0, b1);
    else
        mma_bf16_16816(d, a0, a1, a2, a3, b0, b1);
}

// 4-byte cp.async that copies src_size (0 or 4) bytes and fills the rest with zeros.
SD_DEVINL void cp_async4_zfill(void* dst_smem, const void* src, uint32_t src_size) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst_smem)), "l"(src), "r"(src_size)
                 : "memory");
}

SD_DEVINL uint4 ld_row16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// A step's 16 rows of K and V in shared memory: 16-byte chunk c of row r of either lies at r * kRow
// + ((c ^ swizzle(r)) << 4), K first, then the rows' scales (K, V) and positions.
template <int KIND, int D>
struct Step {
    static constexpr int kEs = KIND == kBf16 ? 2 : 1;
    static constexpr int kRow = D * kEs;      // bytes of a row
    static constexpr int kChunks = kRow / 16;
    static constexpr int kKc = kRow / 64;     // 16-byte pieces of a K row a lane takes
    static constexpr int kVw = kRow / 32;     // 32-bit words of a V row a lane takes
    static constexpr int oV = 16 * kRow;
    static constexpr int oKs = 2 * oV;
    static constexpr int oVs = oKs + 64;
    static constexpr int oPos = oVs + 64;
    static constexpr int kBytes = oPos + 64;
    SD_DEVINL static int swizzle(int r) { return kChunks == 4 ? (r >> 1) & 3 : r & 7; }
    SD_DEVINL static int at(int r, int c) { return r * kRow + ((c ^ swizzle(r)) << 4); }
};

// The row (and row + 8) that stands at index i of the tensor cores' 8-row groups: with this order the
// lanes that read shared memory together, rows perm(2j), perm(2j + 1) of K and perm(0), perm(2), ..
// of V, are in different banks (128-byte rows; the order of keys does not matter otherwise).
SD_DEVINL int perm(int i) {
    constexpr uint32_t kPerm = 0x37156240u;  // 0 4 2 6 5 1 7 3
    return (int)((kPerm >> (4 * i)) & 7u);
}

// ------------------------------------------------------------------ a warp's state

constexpr float kNone = -1e30f;    // a maximum over no rows (finite: differences of it stay numbers)
constexpr int kNoPos = 0x7fffffff; // the position of a row that is none
constexpr float kGrow = 4.f;       // how far (base 2) a weight may pass its maximum before that moves
constexpr float kTopF16 = 10.f;    // log2 of the largest product weight when its maximum has just moved
constexpr float kLimF16 = 32768.f; // the product weight at which it moves

template <int D, int NQ>
struct CaState {
    float o[D / 16][NQ][4];    // O^T: columns g8 * D/8 + 2 md (+1: entries 2, 3) of query 8nq + 2t4 + e
    float m[NQ][2], l[NQ][2];  // maximum (base 2) and this lane's share of the denominator
    float c[NQ][2];            // 8-bit: the product weight is p * vs * c (c = 2^(m - m2 + kTopF16), m2 the
                               // maximum of logit + log2 vs)
    SD_DEVINL void clear() {
#pragma unroll
        for (int md = 0; md < D / 16; ++md)
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[md][nq][e] = 0.f;
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) l[nq][0] = l[nq][1] = 0.f;
    }
    SD_DEVINL void init() {
        clear();
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nq][e] = kNone;
                c[nq][e] = 0.f;
            }
    }
};

SD_DEVINL float max_over_rows(float x) {  // over the lanes of the same t4
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
SD_DEVINL float sum_over_rows(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// The B fragments of the query rows, in registers or (two tiles and more) in shared memory.
template <int D, int NQ>
struct Queries {
    static constexpr bool kShared = NQ >= 2;
    uint32_t f[kShared ? 1 : D / 16][kShared ? 1 : NQ][2];
    const uint2* sh;  // [D/16][NQ][32]
    float qs[NQ][2];  // each query's factor of the logit (with the shared prefix's base 2)
    SD_DEVINL uint2 at(int ks, int nq, int lane) const {
        if constexpr (kShared) return sh[(ks * NQ + nq) * 32 + lane];
        return make_uint2(f[ks][nq][0], f[ks][nq][1]);
    }
};

// S^T = K Q^T of the step at `st`: s[nq][2h + e] of row perm(g8) + 8h and query 8nq + 2t4 + e.
template <int KIND, int D, int NQ>
SD_DEVINL void ca_scores(const uint8_t* st, const Queries<D, NQ>& q, int lane, float (&s)[NQ][4]) {
    constexpr bool F16 = KIND != kBf16;
    using S = Step<KIND, D>;
    const int row = perm(lane >> 2), t4 = lane & 3;
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nq][e] = 0.f;
#pragma unroll
    for (int c = 0; c < S::kKc; ++c) {
        const uint4 k0 = lds128(st + S::at(row, 4 * c + t4)), k1 = lds128(st + S::at(row, 4 * c + t4) + 8 * S::kRow);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
        if constexpr (F16) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint32_t x0 = biased<KIND>(w0[kk]), x1 = biased<KIND>(w1[kk]);
                const uint32_t a0 = widen<KIND>(x0, false), a2 = widen<KIND>(x0, true);
                const uint32_t a1 = widen<KIND>(x1, false), a3 = widen<KIND>(x1, true);
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) {
                    const uint2 b = q.at(4 * c + kk, nq, lane);
                    mma16<F16>(s[nq], a0, a1, a2, a3, b.x, b.y);
                }
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) {
                    const uint2 b = q.at(2 * c + kk, nq, lane);
                    mma16<F16>(s[nq], w0[2 * kk], w1[2 * kk], w0[2 * kk + 1], w1[2 * kk + 1], b.x, b.y);
                }
        }
    }
}

// The online softmax of a step: s becomes the weights of the V rows.  Unless every query sees all
// rows of the step (all), those above a query's limit (sl[8nq + 2t4 + e]) take no part (pos(h): the
// position of row perm(g8) + 8h).
template <int KIND, int D, int NQ, class Pos>
SD_DEVINL void ca_softmax(float (&s)[NQ][4], const float (&ks)[2], const float (&vs)[2], Pos pos, bool all,
                          const int* sl, int t4, const Queries<D, NQ>& q, CaState<D, NQ>& st) {
    constexpr bool F16 = KIND != kBf16;
    float top = -INFINITY, wide = 0.f;
    float w[NQ][4], z[NQ][4];  // weights, and what makes a logit of s
    auto weights = [&]() {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float dx[2], pw[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    dx[h] = fmaf(s[nq][2 * h + e], z[nq][2 * h + e], -st.m[nq][e]);
                    w[nq][2 * h + e] = fast_exp2(dx[h]);
                    if constexpr (F16) pw[h] = w[nq][2 * h + e] * vs[h] * st.c[nq][e];
                }
                top = max3(top, dx[0], dx[1]);
                if constexpr (F16) wide = max3(wide, pw[0], pw[1]);
            }
    };
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[nq][i] = F16 ? ks[i >> 1] * q.qs[nq][i & 1] : q.qs[nq][i & 1];
    if (!all) {
        const int at[2] = {pos(0), pos(1)};
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[nq][i] = at[i >> 1] > sl[8 * nq + 2 * t4 + (i & 1)] ? -INFINITY : s[nq][i] * z[nq][i];
                z[nq][i] = 1.f;
            }
    }
    weights();
    if (__any_sync(0xffffffffu, top > kGrow || wide > kLimF16)) {
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x0 = s[nq][e] * z[nq][e], x1 = s[nq][2 + e] * z[nq][2 + e];
                const float mo = st.m[nq][e];
                const float mn = fmaxf(mo, max_over_rows(fmaxf(x0, x1)));
                const float fl = fast_exp2(mo - mn);
                float fo = fl;
                if constexpr (F16) {
                    // log2 of a zero scale is -inf: its row asks for nothing.  The product's maximum is never so
                    // far below m that c would overflow
                    float y = fmaxf(x0 + __log2f(vs[0]), x1 + __log2f(vs[1]));
                    y = max_over_rows(y);
                    const float co = st.c[nq][e];
                    const float m2o = co > 0.f ? mo + kTopF16 - __log2f(co) : kNone;
                    const float m2n = fmaxf(fmaxf(m2o, y), mn - 100.f);
                    if (mn > kNone) {
                        st.c[nq][e] = fast_exp2(mn - m2n + kTopF16);
                        fo = co > 0.f ? fl * st.c[nq][e] / co : 0.f;
                    }
                }
                st.m[nq][e] = mn;
                st.l[nq][e] *= fl;
#pragma unroll
                for (int md = 0; md < D / 16; ++md) {
                    st.o[md][nq][e] *= fo;
                    st.o[md][nq][2 + e] *= fo;
                }
            }
        weights();
    }
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = i & 1, h = i >> 1;
            st.l[nq][e] += w[nq][i];
            s[nq][i] = F16 ? w[nq][i] * vs[h] * st.c[nq][e] : w[nq][i];
        }
}

// O^T += V^T P^T of the step at `at`, P in s.
template <int KIND, int D, int NQ, bool HILO>
SD_DEVINL void ca_output(const uint8_t* at, int lane, const float (&s)[NQ][4], CaState<D, NQ>& st) {
    using S = Step<KIND, D>;
    constexpr bool F16 = KIND != kBf16;
    uint32_t ph[NQ][2], pl[NQ][2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)  // P^T (rows by lane group) to the B operand (rows by lane pair)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t hi, lo = 0u;
            weight_words<F16, HILO>(s[nq][2 * h], s[nq][2 * h + 1], hi, lo);
            ph[nq][h] = movmatrix_t(hi);
            if constexpr (HILO) pl[nq][h] = movmatrix_t(lo);
        }
    auto pv = [&](int md, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        if constexpr (HILO) {
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) mma16<F16>(st.o[md][nq], a0, a1, a2, a3, pl[nq][0], pl[nq][1]);
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) mma16<F16>(st.o[md][nq], a0, a1, a2, a3, ph[nq][0], ph[nq][1]);
    };
    // columns g8 * D/8 .. of the rows that stand at indexes 2 t4, 2 t4 + 1 and 8 further on
    const int g8 = lane >> 2, r0 = perm(2 * (lane & 3)), r1 = perm(2 * (lane & 3) + 1);
    auto words = [&](int r, int w4) {  // words 4 w4 .. of row r
        return lds128(at + S::oV + S::at(r, g8 * S::kVw / 4 + w4));
    };
    auto four = [&](int w, uint32_t A, uint32_t B, uint32_t C, uint32_t E) {
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
    };
    if constexpr (S::kVw == 2) {  // half a chunk
        const uint8_t* p0 = at + S::oV + S::at(r0, g8 >> 1) + 8 * (g8 & 1);
        const uint8_t* p1 = at + S::oV + S::at(r1, g8 >> 1) + 8 * (g8 & 1);
        const uint2 A = *reinterpret_cast<const uint2*>(p0), B = *reinterpret_cast<const uint2*>(p1);
        const uint2 C = *reinterpret_cast<const uint2*>(p0 + 8 * S::kRow), E = *reinterpret_cast<const uint2*>(p1 + 8 * S::kRow);
        four(0, A.x, B.x, C.x, E.x);
        four(1, A.y, B.y, C.y, E.y);
    } else {
#pragma unroll
        for (int w4 = 0; w4 < S::kVw / 4; ++w4) {
            const uint4 A = words(r0, w4), B = words(r1, w4), C = words(r0 + 8, w4), E = words(r1 + 8, w4);
            four(4 * w4, A.x, B.x, C.x, E.x);
            four(4 * w4 + 1, A.y, B.y, C.y, E.y);
            four(4 * w4 + 2, A.z, B.z, C.z, E.z);
            four(4 * w4 + 3, A.w, B.w, C.w, E.w);
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
SD_DEVINL unsigned tiles_of(int rows) { return (unsigned)max(1, (rows + kCaTile - 1) / kCaTile); }

SD_DEVINL void store_pair(void* out, bool bf16, size_t i, float x, float y) {  // elements i, i + 1 (i even)
    if (bf16)
        reinterpret_cast<uint32_t*>(out)[i / 2] = pack_bf16x2(x, y);
    else
        reinterpret_cast<float2*>(out)[i / 2] = make_float2(x, y);
}

// The sum of a query row's states start, start + step, ..: those of its group's runs (slots first ..
// first + runs - 1) and of the prefix's runs.  Lane l holds columns kE l ..
template <int D>
struct RowSum {
    static constexpr int kE = D / 32;
    float acc[kE], L, top;
};
template <int D>
SD_DEVINL RowSum<D> sum_states(const CaParams& p, int b, int kvh, int r, int first, int runs, int start, int step,
                               int lane) {
    constexpr int kE = RowSum<D>::kE;
    const int2 pre = p.P > 0 ? p.pre.range(kvh) : make_int2(0, 0);
    const int n = runs + pre.y;
    const unsigned M = (unsigned)p.B * p.R, mrow = (unsigned)b * p.R + r;
    auto ml_of = [&](int i) {
        return __ldcg(i < runs ? &p.ws.ml[(size_t)(first + i) * p.R + r]
                               : &p.ws.pre_ml[(size_t)(pre.x + i - runs) * M + mrow]);
    };
    auto o_of = [&](int i) {
        return i < runs ? p.ws.o + ((size_t)(first + i) * p.R + r) * D
                        : p.ws.pre_o + ((size_t)(pre.x + i - runs) * M + mrow) * D;
    };
    RowSum<D> s;
    s.L = 0.f;
    s.top = kNone;
#pragma unroll
    for (int e = 0; e < kE; ++e) s.acc[e] = 0.f;
    for (int base = start; base < n; base += 32 * step) {
        const int mine = base + step * lane, cnt = min(32, (n - base + step - 1) / step);
        const float2 ml = mine < n ? ml_of(mine) : make_float2(kNone, 0.f);
        // eight states' rows are loaded together, and the next eight before these are added
        float x[2][8][kE];
        auto load = [&](int k0, float (&to)[8][kE]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float* o = o_of(base + step * min(k0 + k, cnt - 1)) + kE * lane;
                if constexpr (kE == 4) {
                    const float4 y = __ldcg(reinterpret_cast<const float4*>(o));
                    to[k][0] = y.x, to[k][1] = y.y, to[k][2] = y.z, to[k][3] = y.w;
                } else {
                    const float2 y = __ldcg(reinterpret_cast<const float2*>(o));
                    to[k][0] = y.x, to[k][1] = y.y;
                }
            }
        };
        load(0, x[0]);
        const float was = s.top;
        s.top = fmaxf(was, warp_max(ml.x));
        const float f = exp2f(fmaxf(ml.x, kNone) - s.top), fo = exp2f(was - s.top);
        s.L = s.L * fo + ml.y * f;
#pragma unroll
        for (int e = 0; e < kE; ++e) s.acc[e] *= fo;
#pragma unroll
        for (int k0 = 0; k0 < 32; k0 += 8) {
            if (k0 >= cnt) break;
            if (k0 + 8 < cnt) load(k0 + 8, x[(k0 / 8 + 1) & 1]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k0 + k);
                if (k0 + k < cnt) {
#pragma unroll
                    for (int e = 0; e < kE; ++e) s.acc[e] = fmaf(x[(k0 / 8) & 1][k][e], fk, s.acc[e]);
                }
            }
        }
    }
    s.L = warp_sum(s.L);
    return s;
}

// TS warps make a team that shares the steps it takes (all its warps see the same rows, each for 8 NQ of
// the query rows); a team has a ring of stages of its own.
template <int KIND, int D, int NQ, int TS>
struct CaShared {
    static constexpr int kStages = KIND == kBf16 && D == 128 ? 2 : 3;
    // a state row: column g8 * D/8 + 2md + j at 18 md + 2 g8 + j
    static constexpr int kPitch = D / 16 * 18;
    alignas(128) uint8_t ring[kCaWarps / TS][kStages][Step<KIND, D>::kBytes];
    alignas(16) float o[kCaWarps][8 * NQ][kPitch];
    float2 ml[kCaWarps][8 * NQ];
    uint2 q[NQ >= 2 ? TS * D / 16 * NQ * 32 : 1];
    float qs[8 * NQ * TS];
    int lim[8 * NQ * TS];
    unsigned part[kCaWarps], base;
    int b;
};

constexpr unsigned kCaGroupCost = 2;  // (1: 55.4 us, 3: 55.2, 4: 55.5 where 2 takes 54.6)
constexpr int kFoldSteps = 32;  // steps after which SD_F32 output folds the accumulators

template <int KIND, int D, int NQ, int TS, bool HILO, bool SEL, int MINB>
__global__ void __launch_bounds__(kCaThreads, MINB) cache_attend_kernel(const CaParams p) {
    constexpr bool F16 = KIND != kBf16;
    using S = Step<KIND, D>;
    constexpr int kRow = S::kRow;
    constexpr int kMd = D / 16;
    constexpr int kTeams = kCaWarps / TS;
    using Shared = CaShared<KIND, D, NQ, TS>;
    constexpr int kStages = Shared::kStages;
    extern __shared__ __align__(128) uint8_t ca_smem[];
    auto& sh = *reinterpret_cast<Shared*>(ca_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    const int team = warp / TS, half = warp % TS;  // half: which 8 NQ of the query rows
    const unsigned c = blockIdx.x;
    // The cache, qpos and q may be the preceding kernels' results.  Behind a prefix kernel of the same
    // call, which lets this one start only after its own wait for them, they are there already: the
    // wait is then for that kernel alone, and comes before its states are read.
    if (p.P == 0) pdl_wait();
    // (No early trigger for the merge kernel, nor in that one for the next call's: CTAs that wait on an SM
    // keep others from it.  8 ragged e4m3 caches called back to back: 71 us with both, 61 without.)

    // this CTA's run of units: [w0, w1) of all groups' units in order.  A group's units are `extra` empty ones,
    // then its own; the runs that hold own units of a group are consecutive, and so are their slots.
    unsigned W, tb, j, w0;
    int b, kvh;
    const bool few = p.B <= 32;  // lane i knows sequence i: no warp needs another
    unsigned tl = 0u;
    if constexpr (SEL) {
        tb = tiles_of(p.n_list);
        W = (unsigned)p.B * p.Hkv * tb;
    } else if (few) {
        tl = lane < p.B ? tiles_of(seq_len(p, lane)) : 0u;
        W = __reduce_add_sync(0xffffffffu, tl) * p.Hkv;
    } else {
        unsigned sum = 0;
        for (int i = tid; i < p.B; i += kCaThreads) sum += tiles_of(seq_len(p, i));
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) sh.part[warp] = sum;
        __syncthreads();
        W = (sh.part[0] + sh.part[1] + sh.part[2] + sh.part[3]) * p.Hkv;
    }
    const unsigned extra = W > 2u * gridDim.x ? kCaGroupCost : 0u;  // (a unit or two a CTA: nothing to even out)
    W += (unsigned)p.B * p.Hkv * extra;
    const unsigned ncta = min(gridDim.x, W);
    if (c >= ncta) {
        if (p.P > 0) pdl_wait();  // (the merge kernel counts on the prefix being done)
        return;
    }
    const Cut cut = Cut::of(W, ncta);
    w0 = cut.start(c);
    const unsigned w1 = cut.start(c + 1);
    if constexpr (SEL) {
        tb += extra;
        const unsigned g = w0 / tb;
        j = w0 - g * tb;
        b = (int)(g / (unsigned)p.Hkv);
        kvh = (int)(g - (unsigned)b * p.Hkv);
    } else if (few) {
        if (lane < p.B) tl += extra;
        unsigned incl = tl;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        b = __ffs((int)__ballot_sync(0xffffffffu, w0 < incl * p.Hkv)) - 1;
        tb = __shfl_sync(0xffffffffu, tl, b);
        const unsigned off = w0 - (__shfl_sync(0xffffffffu, incl, b) - tb) * p.Hkv;
        kvh = (int)(off / tb);
        j = off - (unsigned)kvh * tb;
    } else {
        // the sequence of unit w0: sequence i's units start at Hkv * (units of a group before it)
        unsigned run = 0;
        for (int base = 0; base < p.B; base += kCaThreads) {
            const int i = base + tid;
            const unsigned t = i < p.B ? tiles_of(seq_len(p, i)) + extra : 0u;
            unsigned incl = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += u;
            }
            __syncthreads();
            if (lane == 31) sh.part[warp] = incl;
            if (tid == 0) sh.b = -1;
            __syncthreads();
            unsigned before = run;
            for (int k = 0; k < warp; ++k) before += sh.part[k];
            const unsigned hi = (before + incl) * p.Hkv, lo = hi - t * p.Hkv;
            if (t > 0u && w0 >= lo && w0 < hi) {
                sh.b = i;
                sh.base = lo;
            }
            for (int k = 0; k < kCaWarps; ++k) run += sh.part[k];
            __syncthreads();
            if (sh.b >= 0) break;
        }
        b = sh.b;
        tb = tiles_of(seq_len(p, b)) + extra;
        const unsigned off = w0 - sh.base;
        kvh = (int)(off / tb);
        j = off - (unsigned)kvh * tb;
    }

    for (unsigned w = w0; w < w1;) {
        if (j < extra) {
            w += extra - j;
            j = extra;
            if (w >= w1) break;
        }
        const int g = b * p.Hkv + kvh;
        const int len = seq_len(p, b);
        const unsigned seg = min(tb - j, w1 - w);
        const int list = SEL ? p.n_list : len;
        const int j0 = (int)(j - extra) * kCaTile, j1 = len == 0 ? j0 : min(list, j0 + (int)seg * kCaTile);

        const uint8_t* kbase = p.kc + (size_t)g * p.T * kRow;
        const uint8_t* vbase = p.vc + (size_t)g * p.T * kRow;
        const float* ksb = p.ks + (size_t)g * p.T;
        const float* vsb = p.vs + (size_t)g * p.T;
        const int nsteps = (j1 - j0 + 15) / 16;
        // lane l < 16 (and l + 16) resolves row l of a step: its position, or -1 (past the run's rows, an
        // empty slot, an index outside the cache, a row no query sees)
        auto resolve = [&](int step) {
            const int i = j0 + 16 * step + (lane & 15);
            int t = -1;
            if (i < j1) {
                if constexpr (SEL) {
                    const int e = (int)((unsigned)i / (unsigned)p.block);
                    const long sel = p.idx[(size_t)g * p.n_idx + e];
                    const long pos = sel * p.block + (i - e * p.block);
                    if (sel != -1) {
                        if (sel < 0 || pos >= p.T)
                            report(p.err, SD_DEVERR_INDEX);
                        else if (pos < len)
                            t = (int)pos;
                    }
                } else {
                    t = i;
                }
            }
            return t;
        };
        // Copies the team's rows of a step (resolved in `rows`) into a stage of its ring, a row that is none
        // as zeros (whatever the cache holds there, its weight of 0 must not meet a NaN or an infinity).
        // A team of two shares the copies: K, V.
        auto fetch = [&](int stage, int step, int rows) {
            uint8_t* st = sh.ring[team][stage];
            constexpr int kPer = 32 / S::kChunks > 0 ? 32 / S::kChunks : 1;  // rows an instruction copies
            const int c0 = lane % S::kChunks, r0 = lane / S::kChunks;
#pragma unroll
            for (int r = 0; r < 16; r += kPer) {
                int t;
                if constexpr (SEL) {
                    t = __shfl_sync(0xffffffffu, rows, r + r0);
                } else {
                    t = j0 + 16 * step + r + r0;
                    if (t >= j1) t = -1;
                }
                const size_t off = (size_t)max(t, 0) * kRow + 16 * c0;
                const uint32_t n = t < 0 ? 0u : 16u;
                const int to = S::at(r + r0, c0);
                if (TS == 1 || half == 0) cp_async16_zfill(st + to, kbase + off, n);
                if (TS == 1 || half == 1) cp_async16_zfill(st + S::oV + to, vbase + off, n);
            }
            if (half == 0) {
                if constexpr (F16)
                    cp_async4_zfill(st + S::oKs + 4 * lane, (lane < 16 ? ksb : vsb) + max(rows, 0), rows < 0 ? 0u : 4u);
                if (SEL && lane < 16) reinterpret_cast<int*>(st + S::oPos)[lane] = rows < 0 ? kNoPos : rows;
            }
        };
        auto team_sync = [&]() {
            if constexpr (TS == 1)
                __syncwarp();
            else
                asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TS) : "memory");
        };
        // the first steps' rows are on their way while the queries are prepared
        int early[kStages];
#pragma unroll
        for (int i = 0; i < kStages; ++i) early[i] = resolve(team + i * kTeams);
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) {
            if (team + i * kTeams < nsteps) fetch(i, team + i * kTeams, early[i]);
            cp_async_commit();
        }
        int rows = early[kStages - 1];

        // the query rows 8nq + g8 as B fragments, their limits and the smallest limit
        Queries<D, NQ> q;
        q.sh = sh.q + half * (kMd * NQ * 32);
        const int* lim = sh.lim + half * 8 * NQ;
        __syncthreads();  // (the segment before is done with the limits and the states)
        int lmin = p.T;  // rows every query sees
        if (tid < 8 * NQ * TS) sh.lim[tid] = tid < p.R ? min(p.qpos[(size_t)b * p.V + tid / p.G], p.T - 1) : -1;
        for (int v = 0; v < p.V; ++v) lmin = min(lmin, min(p.qpos[(size_t)b * p.V + v], p.T - 1) + 1);
#pragma unroll
        for (int nt = 0; nt < (Queries<D, NQ>::kShared ? TS * NQ : NQ); ++nt) {
            if (Queries<D, NQ>::kShared && warp != nt) continue;  // tile nt is warp nt's to prepare
            const int nq = Queries<D, NQ>::kShared ? 0 : nt;
            const int r = 8 * nt + g8;
            const bool have = r < p.R;
            const int v = have ? r / p.G : 0, gi = have ? r - v * p.G : 0;
            const uint8_t* qrow = p.q + (((size_t)b * p.V + v) * p.Hq + (size_t)kvh * p.G + gi) * (D * 2);
            uint32_t raw[kMd][2];
            if constexpr (F16) {
                uint32_t top = 0u;
#pragma unroll
                for (int cc = 0; cc < S::kKc; ++cc)
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
                        raw[k][i] = pack_f16x2(bf16lo(raw[k][i]) * down, bf16hi(raw[k][i]) * down);
                if (t4 == 0) sh.qs[r] = up * p.scale_log2;
            } else {
#pragma unroll
                for (int cc = 0; cc < S::kKc; ++cc) {  // dims 32 cc + 8 t4 ..
                    const uint4 x = have ? ld_row16(qrow + 2 * (32 * cc + 8 * t4)) : make_uint4(0u, 0u, 0u, 0u);
                    raw[2 * cc][0] = x.x;
                    raw[2 * cc][1] = x.y;
                    raw[2 * cc + 1][0] = x.z;
                    raw[2 * cc + 1][1] = x.w;
                }
                if (t4 == 0) sh.qs[r] = p.scale_log2;
            }
#pragma unroll
            for (int k = 0; k < kMd; ++k) {
                if constexpr (Queries<D, NQ>::kShared) {
                    sh.q[((nt / NQ * kMd + k) * NQ + nt % NQ) * 32 + lane] = make_uint2(raw[k][0], raw[k][1]);
                } else {
                    q.f[k][nq][0] = raw[k][0];
                    q.f[k][nq][1] = raw[k][1];
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const float2 f = *reinterpret_cast<const float2*>(&sh.qs[8 * (half * NQ + nq) + 2 * t4]);
            q.qs[nq][0] = f.x;
            q.qs[nq][1] = f.y;
        }

        CaState<D, NQ> st;
        st.init();
        // Folds the registers' state into the warp's in shared memory (all of it relative to the softmax
        // maximum m), and starts it anew.
        auto fold = [&](bool first) {
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int qr = 8 * nq + 2 * t4 + e;
                    const float l = sum_over_rows(st.l[nq][e]);
                    float f = 1.f;
                    if constexpr (F16) f = st.c[nq][e] > 0.f ? 1.f / st.c[nq][e] : 0.f;
                    float2 ml = make_float2(st.m[nq][e], l);
                    float old = 0.f;
                    if (!first) {
                        const float2 was = sh.ml[warp][qr];
                        ml.x = fmaxf(was.x, st.m[nq][e]);
                        old = exp2f(was.x - ml.x);
                        const float now = exp2f(st.m[nq][e] - ml.x);
                        f *= now;
                        ml.y = was.y * old + l * now;
                    }
                    float* row = sh.o[warp][qr];
#pragma unroll
                    for (int md = 0; md < kMd; ++md) {
                        float2* at = reinterpret_cast<float2*>(row + 18 * md + 2 * g8);
                        float2 x = make_float2(st.o[md][nq][e] * f, st.o[md][nq][2 + e] * f);
                        if (!first) {
                            const float2 y = *at;
                            x.x = fmaf(y.x, old, x.x);
                            x.y = fmaf(y.y, old, x.y);
                        }
                        *at = x;
                    }
                    __syncwarp();
                    if (g8 == 0) sh.ml[warp][qr] = ml;
                }
            __syncwarp();
            st.clear();
        };

        bool first = true;
        int since = 0, stage = 0;
        for (int n = team; n < nsteps || first; n += kTeams) {
            if (n < nsteps) {
                // this step has landed for every warp of the team, and all are done with the stage of the one before,
                // which takes the rows kStages - 1 steps ahead
                cp_async_wait<kStages - 2>();
                team_sync();
                if (n + (kStages - 1) * kTeams < nsteps) fetch(stage == 0 ? kStages - 1 : stage - 1, n + (kStages - 1) * kTeams, rows);
                cp_async_commit();
                rows = resolve(n + kStages * kTeams);
                const uint8_t* at = sh.ring[team][stage];
                const int row = perm(g8);
                float sc[NQ][4], ks[2], vs[2];
                ca_scores<KIND, D, NQ>(at, q, lane, sc);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ks[h] = reinterpret_cast<const float*>(at + S::oKs)[row + 8 * h];
                    vs[h] = reinterpret_cast<const float*>(at + S::oVs)[row + 8 * h];
                }
                auto pos = [&](int h) {
                    if constexpr (SEL) return reinterpret_cast<const int*>(at + S::oPos)[row + 8 * h];
                    const int i = j0 + 16 * n + row + 8 * h;
                    return i < j1 ? i : kNoPos;
                };
                const bool all = SEL ? __all_sync(0xffffffffu, max(pos(0), pos(1)) < lmin) : j0 + 16 * n + 16 <= lmin;
                ca_softmax<KIND, D, NQ>(sc, ks, vs, pos, all, lim, t4, q, st);
                ca_output<KIND, D, NQ, HILO>(at, lane, sc, st);
                stage = stage == kStages - 1 ? 0 : stage + 1;
            }
            if (n + kTeams >= nsteps || (HILO && ++since == kFoldSteps)) {
                fold(first);
                first = false;
                since = 0;
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        const bool whole = j == extra && seg == tb - extra && p.P == 0;
        const size_t slot = (size_t)c + g;
        for (int i = tid; i < p.R * (D / 2); i += kCaThreads) {
            const int r = i / (D / 2), d = 2 * (i - r * (D / 2));
            const int gg = d / (D / 8), at = 18 * ((d - gg * (D / 8)) / 2) + 2 * gg;
            const int hf = r / (8 * NQ), rr = r - hf * 8 * NQ;  // warps hf, hf + TS, .. hold this row
            float M = sh.ml[hf][rr].x;
#pragma unroll
            for (int k = 1; k < kTeams; ++k) M = fmaxf(M, sh.ml[hf + k * TS][rr].x);
            float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < kTeams; ++k) {
                const float2 ml = sh.ml[hf + k * TS][rr];
                const float2 o = *reinterpret_cast<const float2*>(&sh.o[hf + k * TS][rr][at]);
                const float f = exp2f(ml.x - M);
                L = fmaf(ml.y, f, L);
                x = fmaf(o.x, f, x);
                y = fmaf(o.y, f, y);
            }
            if (M == kNone) M = -INFINITY;
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
        if (j == extra && tid == 0)  // the runs that hold the group's units
            p.ws.meta[g] = make_int2((int)c + g, (int)(cut.run_of(w + tb - extra - 1) - c) + 1);
        w += seg;
        j = 0;
        if (++kvh == p.Hkv) {
            kvh = 0;
            ++b;
            if (!SEL && w < w1) tb = tiles_of(seq_len(p, b)) + extra;
        }
    }
    if (p.P > 0) pdl_wait();
}

// The states of every query row into the output.  kSplit: one CTA a row, whose warps take each fourth state
// and meet in shared memory in a fixed order; else one warp a row.  (The last CTA of a group merging
// it instead of a second kernel was measured: it saves a launch and loses more, since one CTA then does
// what 4 to 32 do here: 18.7 -> 22.4 us for the selected blocks, 65 -> 77 us for 64 sequences behind
// a prefix of 32768.)
template <int D, bool kSplit>
__global__ void __launch_bounds__(kCaThreads) cache_merge_kernel(const CaParams p) {
    constexpr int kE = RowSum<D>::kE;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned row = kSplit ? blockIdx.x : blockIdx.x * kCaWarps + warp;  // (b, v, h)
    const unsigned bv = row / (unsigned)p.Hq, h = row - bv * p.Hq;
    const unsigned b = bv / (unsigned)p.V, v = bv - b * p.V;
    const unsigned kvh = h / (unsigned)p.G;
    const int r = (int)(v * p.G + h - kvh * p.G);
    if (b >= (unsigned)p.B) return;
    pdl_wait();
    const int2 own = p.ws.meta[b * p.Hkv + kvh];
    if (own.y == 1 && p.P == 0) return;  // written by the CTA that had the whole group
    if constexpr (kSplit) {
        __shared__ float so[kCaWarps][D];
        __shared__ float sl[kCaWarps], sm[kCaWarps];
        const RowSum<D> s = sum_states<D>(p, (int)b, (int)kvh, r, own.x, own.y, warp, kCaWarps, lane);
#pragma unroll
        for (int e = 0; e < kE; ++e) so[warp][kE * lane + e] = s.acc[e];
        if (lane == 0) {
            sl[warp] = s.L;
            sm[warp] = s.top;
        }
        __syncthreads();
        float mx = sm[0], f[kCaWarps], L = 0.f;
#pragma unroll
        for (int k = 1; k < kCaWarps; ++k) mx = fmaxf(mx, sm[k]);
#pragma unroll
        for (int k = 0; k < kCaWarps; ++k) {
            f[k] = exp2f(sm[k] - mx);
            L = fmaf(sl[k], f[k], L);
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        if (threadIdx.x < D / 2) {
            const int d = 2 * (int)threadIdx.x;
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int k = 0; k < kCaWarps; ++k) {
                x = fmaf(so[k][d], f[k], x);
                y = fmaf(so[k][d + 1], f[k], y);
            }
            store_pair(p.out, p.out_bf16 != 0, (size_t)row * D + d, x * inv, y * inv);
        }
        if (threadIdx.x == 0) p.lse[row] = L > 0.f ? (mx + log2f(L)) * 0.69314718055994530942f : -INFINITY;
    } else {
        const RowSum<D> s = sum_states<D>(p, (int)b, (int)kvh, r, own.x, own.y, 0, 1, lane);
        const float inv = s.L > 0.f ? 1.f / s.L : 0.f;
#pragma unroll
        for (int e = 0; e < kE; e += 2)
            store_pair(p.out, p.out_bf16 != 0, (size_t)row * D + kE * lane + e, s.acc[e] * inv, s.acc[e + 1] * inv);
        if (lane == 0) p.lse[row] = s.L > 0.f ? (s.top + log2f(s.L)) * 0.69314718055994530942f : -INFINITY;
    }
}

// CTAs an SM holds of a variant (its __launch_bounds__): what its registers and rings allow.
constexpr int ca_ctas_per_sm(int kind, int d, int nq, int ts) {
    if (d == 64) return kind != kBf16 && nq == 1 ? 4 : 3;
    return kind == kBf16 || (nq == 2 && ts == 1) ? 2 : 3;
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
    pl.ctas = (int)std::min<long>(units, (long)num_sms() * ca_ctas_per_sm(ca_kind(a), a->d, R <= 8 ? 1 : 2, R <= 16 ? 1 : 2));
    pl.slots = (int)(pl.ctas + NG - 1);
    if (a->P > 0) pl.pre = prefix_plan(a);
    return pl;
}

sd_status ca_validate(const sd_cache_attend_args* a, bool pointers) {
    const char* who = "sd_cache_attend";
    SD_REQUIRE(a != nullptr, "%s: null args", who);
    SD_REQUIRE(a->cache_dtype == SD_BF16 || a->cache_dtype == SD_I8 || a->cache_dtype == SD_E4M3,
               "%s: cache_dtype must be SD_BF16, SD_I8 or SD_E4M3", who);
    SD_REQUIRE(a->out_dtype == SD_F32 || a->out_dtype == SD_BF16, "%s: out_dtype must be SD_F32 or SD_BF16", who);
    SD_REQUIRE(a->B >= 0 && a->V >= 1 && a->Hkv >= 1 && a->Hq >= 1 && a->Hq % a->Hkv == 0 && a->T >= 1 && a->P >= 0 &&
                   a->T <= (1 << 30) && a->P <= (1 << 30),
               "%s: bad sizes (B=%d V=%d Hq=%d Hkv=%d T=%d P=%d)", who, a->B, a->V, a->Hq, a->Hkv, a->T, a->P);
    SD_REQUIRE(a->B <= 65535 && a->Hq <= 65535, "%s: B and Hq must be <= 65535", who);
    SD_REQUIRE(a->idx == nullptr || (a->n_idx >= 0 && a->block >= 1 && (long)a->n_idx * a->block <= (1L << 30)),
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
    SD_REQUIRE((long)a->B * a->Hkv * (rows / kCaTile + 1 + kCaGroupCost) < (1L << 31), "%s: too many rows", who);
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

template <int KIND, int D, int NQ, int TS, bool HILO>
sd_status ca_launch(const CaParams& p, const CaPlan& pl, cudaStream_t st) {
    constexpr int kMinB = ca_ctas_per_sm(KIND, D, NQ, TS);
    constexpr int kBytes = (int)sizeof(CaShared<KIND, D, NQ, TS>);
    static_assert(kMinB * (kBytes + 1024) <= 227 * 1024, "the CTAs of an SM share its memory");
    auto kern = p.idx != nullptr ? cache_attend_kernel<KIND, D, NQ, TS, HILO, true, kMinB>
                                 : cache_attend_kernel<KIND, D, NQ, TS, HILO, false, kMinB>;
    if (kBytes > 48 * 1024)
        SD_CUDA_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes),
                      "sd_cache_attend: cudaFuncSetAttribute");
    SD_CUDA_CHECK(launch_pdl(kern, dim3((unsigned)pl.ctas), dim3(kCaThreads), (size_t)kBytes, st, p),
                  "sd_cache_attend: launch");
    return launch_status("sd_cache_attend");
}

template <int KIND, int D, bool HILO>
sd_status ca_dispatch_rows(const CaParams& p, const CaPlan& pl, cudaStream_t st) {
    return p.R <= 8    ? ca_launch<KIND, D, 1, 1, HILO>(p, pl, st)
           : p.R <= 16 ? ca_launch<KIND, D, 2, 1, HILO>(p, pl, st)
                       : ca_launch<KIND, D, 2, 2, HILO>(p, pl, st);
}
template <int KIND, int D>
sd_status ca_dispatch(const CaParams& p, const CaPlan& pl, cudaStream_t st) {
    return p.out_bf16 ? ca_dispatch_rows<KIND, D, false>(p, pl, st) : ca_dispatch_rows<KIND, D, true>(p, pl, st);
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
    p.pre = pl.pre;
    p.out_bf16 = a->out_dtype == SD_BF16;
    p.scale_log2 = a->scale * 1.44269504088896340736f;
    cudaStream_t cs = as_stream(stream);
    if (a->P > 0) {
        st = prefix_launch(a, pl.pre, w, cs);
        if (st != SD_OK) return st;
    }
    const bool d128 = a->d == 128;
    switch (ca_kind(a)) {
        case kInt8: st = d128 ? ca_dispatch<kInt8, 128>(p, pl, cs) : ca_dispatch<kInt8, 64>(p, pl, cs); break;
        case kE4m3: st = d128 ? ca_dispatch<kE4m3, 128>(p, pl, cs) : ca_dispatch<kE4m3, 64>(p, pl, cs); break;
        default: st = d128 ? ca_dispatch<kBf16, 128>(p, pl, cs) : ca_dispatch<kBf16, 64>(p, pl, cs); break;
    }
    if (st != SD_OK) return st;
    // a CTA a row while that leaves the GPU room (its states are then read four at a time), else a warp
    const unsigned rows = (unsigned)a->B * a->V * a->Hq;
    const bool split = rows <= 8u * (unsigned)num_sms();
    const auto merge = d128 ? (split ? cache_merge_kernel<128, true> : cache_merge_kernel<128, false>)
                            : (split ? cache_merge_kernel<64, true> : cache_merge_kernel<64, false>);
    SD_CUDA_CHECK(launch_pdl(merge, dim3(split ? rows : (rows + kCaWarps - 1) / kCaWarps), dim3(kCaThreads), 0, cs, p),
                  "sd_cache_attend: merge launch");
    return launch_status(who);
}
