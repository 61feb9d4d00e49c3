// prefix_attend.cu -- the prefix that a serving batch shares, attended once for all sequences on
// the 5th-generation tensor cores: the part of sd_cache_attend over k_prefix/v_prefix.
//
// "Esparsidade de Contexto no Tempo de Inferencia" (gist.science summary), sec. 2 (exact softmax);
// Adaptive DHiSparse (news page), "Metodologia" (query tokens share each fetched row: here the
// rows of all sequences' query tokens).
//
// Mathematics.  The query rows of one KV head, M = B*V*G of them, form one matrix: S = Q K^T, P =
// 2^(S c - m), O = P V with the softmax kept online per row (m, l), as in flash attention.  The
// sequences' rows are split over CTAs in pairs of 128-row tiles, the prefix into runs of key tiles; every
// (rows, run of a head) leaves its (m, l, O), which the call's merge kernel joins with the states of
// the sequences' own rows.
//
// Bound: for up to about 256 rows a KV head HBM (a key tile is read once for both row tiles),
// beyond it the tensor cores and the exponentials.  One CTA an SM; per key tile of 128 and row tile
// t = 0, 1: S_t (128 x 128 fp32 accumulators in TMEM) by d/16 MMAs, softmax by two warpgroups (two
// threads a row, 64 columns each: no shuffles, and one thread's chain of 128 exponentials was what the
// tensor cores waited for; S is read twice, 32 columns at a time, which leaves the 16 warps 96
// registers a thread), P_t back into the TMEM columns S_t held (32 keys: 16 columns of one
// bf16 part, 16 of the other), O_t += P_t V with P from TMEM and V as it lies in memory
// (MN-major).  One MMA warp alternates the tiles, so the tensor cores work on one while the other's
// softmax runs (a warp a tile lets both tiles fall into step: 153 -> 181 us).  That warp does as little else
// as it can, since what it does between MMAs the tensor cores wait for: its waits are one wait, a lane
// a barrier, and a stage is given back by the softmax threads, whose wait for the scores tells the same.
// O_t is rescaled only when a row's maximum has grown by more than 2^8 since the last time (weights stay below 2^8; the quotient O / l does not change), which is rare after the first tiles.
// The tensor cores cut what they add to a sum (2^-24 of it), so SD_F32 output starts O_t anew every
// 16 tiles and adds up in fp32 in the workspace (L2).  The softmax takes 4 to 5 instructions an
// element: products and sums two at a time (f32x2), three-way maxima.
// Several pairs of row tiles read the same key tiles side by side, from L2.  (Clusters of two CTAs that load
// half of every key tile for both were slower, 137 -> 175 us for 1024 rows a KV head: each then
// waits for the other's stages.  So was asking L2 for tiles ahead.)
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (d each).  Shared memory: 2 Q tiles, 2 stages of K
// and of V.  Every wait is bounded; a wait that runs out raises an abort flag, the copies and MMAs
// in flight land, and the kernel frees its TMEM and returns.
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "cache_attend.cuh"
#include "tc_operands.cuh"

namespace sd {
namespace {

constexpr int kPfKeys = 128;  // keys a tile
constexpr int kPfRows = 128;  // query rows a tile
// warps 0-7 and 8-15: softmax of row tiles 0 and 1 (warps 4-7 and 12-15 of keys 64-127)
constexpr int kPfProd = 16, kPfMma = 17;
constexpr int kPfThreads = 32 * 18;
constexpr int kPfStages = 2;
constexpr int kPfFold = 16;      // key tiles after which SD_F32 output folds O
constexpr float kPfGrow = 8.f;  // the growth of a row's maximum (base 2) that O is rescaled at

template <int D>
struct PfLayout {
    static constexpr int kAtoms = D / 64;
    static constexpr int kAtom = 128 * 128;           // 128 rows of 64 bf16
    static constexpr int kTile = kAtoms * kAtom;
    static constexpr int oQ = 0;
    static constexpr int oK = oQ + 2 * kTile;
    static constexpr int oV = oK + kPfStages * kTile;
    static constexpr int oBars = oV + kPfStages * kTile;
    static constexpr int oMisc = oBars + 32 * 8;
    static constexpr int oTop = oMisc + 32;           // [2][2][128] floats: the halves' maxima, then their sums
    static constexpr int kBytes = oTop + 2048 + 1024;  // slack for the 1024-byte alignment
};

struct PfParams {
    float2* ml;
    float* o;
    int32_t* err;
    PrefixPlan plan;
    int M, G, P, pairs, row_tiles, bpt;
    float scale_log2;
    unsigned long long wait_ns;
};

// A bounded wait that gives up (within its limit) and raises the abort flag for the others.  The clock
// is read once in 256 tries only: reading it takes as long as a whole step of the pipeline.
SD_DEVINL bool pf_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint64_t lim) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 0u) {
            const uint64_t now = globaltimer_ns();
            if (t0 == 0) t0 = now;
            if (*abort_flag || now - t0 > lim) {
                *abort_flag = 1;
                return false;
            }
        }
    }
}

template <int D, bool HILO, bool EVEN>
__global__ void __launch_bounds__(kPfThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const PfParams p) {
    using L = PfLayout<D>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t* sm = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint64_t* qfull = reinterpret_cast<uint64_t*>(sm + L::oBars);
    uint64_t* kfull = qfull + 1;
    uint64_t* vfull = kfull + kPfStages;
    // [2] event e, on barrier e % 2: every row tile's S(e) and O += P(e - 1) V are done, so the stages of K(e)
    // and V(e - 1) are free
    uint64_t* freed = vfull + kPfStages;
    uint64_t* sfull = freed + 2;  // [2] S_t is in TMEM (and O_t += P_t V of the tile before is done)
    uint64_t* pfull = sfull + 2;           // [2] P_t is in TMEM
    uint64_t* ofull = pfull + 2;           // [2] the last O_t is done
    uint64_t* drain = ofull + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + L::oMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::oMisc + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pair = (int)blockIdx.x % p.pairs, team = (int)blockIdx.x / p.pairs;
    const int nq = min(2, p.row_tiles - 2 * pair);  // row tiles of this CTA
    const uint64_t lim = p.wait_ns;

    if (tid == 0) {
        static_assert(kPfStages == 2, "an event's barrier follows the stage's");
        mbar_init(qfull, 1);
        for (int s = 0; s < kPfStages; ++s) {
            mbar_init(&kfull[s], 1);
            mbar_init(&vfull[s], 1);
            mbar_init(&freed[s], (uint32_t)nq);  // a stage is free once all row tiles are done with it
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sfull[t], 1);
            mbar_init(&pfull[t], 8);  // one arrival a softmax warp
            mbar_init(&ofull[t], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbarrier_init();
    }
    if (warp == kPfMma) tmem_alloc(tmem_slot, 512);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    int kvh = 0;
    auto load_tile = [&](uint8_t* dst, const CUtensorMap* map, int key, uint64_t* bar) {
        mbar_arrive_expect_tx(bar, L::kTile);
#pragma unroll
        for (int a = 0; a < L::kAtoms; ++a) tma_load_3d(dst + a * L::kAtom, map, 64 * a, key, kvh, bar);
    };
    pdl_wait();  // q and the prefix may be the preceding kernels' results
    pdl_launch_dependents();

    int issued = 0;  // key tiles whose K and V the producer asked for, twice
    int seg = 0, g0 = 0;  // segments and key tiles done before
    bool stop = false;
    for (kvh = EVEN ? p.plan.first_head(team) : team / p.plan.splits;; ++kvh) {
        // the team's key tiles of this head: n0 .. n0 + nt - 1, and the slot of their state
        int n0, nt;
        if constexpr (EVEN) {
            if (!p.plan.segment(team, kvh, n0, nt)) break;
            if (nt == 0) continue;
        } else {
            const int split = team - kvh * p.plan.splits;
            n0 = (int)p.plan.cut.start((unsigned)split);
            nt = (int)p.plan.cut.start((unsigned)split + 1u) - n0;
        }
        const int slot = EVEN ? team + kvh : team;
        if (warp == kPfProd) {
            if (lane == 0) {
                const uint32_t qbytes = (uint32_t)(p.G * p.bpt) * 128u;
                mbar_arrive_expect_tx(qfull, (uint32_t)nq * L::kAtoms * qbytes);
                for (int t = 0; t < nq; ++t)
#pragma unroll
                    for (int a = 0; a < L::kAtoms; ++a)
                        tma_load_3d(sm + L::oQ + t * L::kTile + a * L::kAtom, &qmap, 64 * a, kvh * p.G,
                                    (2 * pair + t) * p.bpt, qfull);
                auto event = [&](int e) {  // event e has happened (those before the first tile have)
                    return e < 0 || pf_wait(&freed[e & 1], (uint32_t)(e >> 1) & 1u, abort_flag, lim);
                };
                for (int n = 0; n < nt; ++n) {
                    const int g = g0 + n, s = g % kPfStages;
                    const int key = (n0 + n) * kPfKeys;
                    if (!event(g - 2)) break;
                    load_tile(sm + L::oK + s * L::kTile, &kmap, key, &kfull[s]);
                    issued = 2 * g + 1;
                    if (!event(g - 1)) break;
                    load_tile(sm + L::oV + s * L::kTile, &vmap, key, &vfull[s]);
                    issued = 2 * g + 2;
                }
            }
        } else if (warp == kPfMma) {
            // the whole warp runs along, one elected lane issues
            constexpr uint32_t kIdS = umma_idesc_bf16_f32(kPfRows, kPfKeys);
            constexpr uint32_t kIdO = umma_idesc_bf16_f32(kPfRows, D) | kUmmaBMnMajor;
            const uint32_t base = smem_addr(sm);
            const uint32_t qd = umma_lo_k(base + L::oQ), kd = umma_lo_k(base + L::oK);
            const uint32_t vd = umma_lo_mn(base + L::oV, L::kAtom);
            constexpr uint32_t kStep = L::kTile >> 4;  // a tile, in a descriptor's address field
            auto scores = [&](int t, int n) {  // S_t = Q_t K_n^T
                const uint32_t a = qd + t * kStep, b = kd + ((g0 + n) % kPfStages) * kStep;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    constexpr uint32_t kAt = L::kAtom >> 4;
                    const uint32_t off = (k >> 2) * kAt + (k & 3) * 2;
                    umma_bf16_ss(tmem + t * 128, a + off, b + off, kIdS, k > 0 ? 1u : 0u);
                }
                umma_commit(&sfull[t]);
            };
            auto output = [&](int t, int n) {  // O_t += P_t V_n
                const uint32_t b = vd + ((g0 + n) % kPfStages) * kStep;
                const uint32_t o = tmem + 256 + t * 128, a = tmem + t * 128;
                const uint32_t add = (HILO ? n % kPfFold : n) > 0 ? 1u : 0u;
#pragma unroll
                for (int k = 0; k < kPfKeys / 16; ++k) {
                    const uint32_t ak = a + 32 * (k >> 1) + 8 * (k & 1);
                    umma_bf16_ts(o, ak, b + k * (2048 >> 4), kIdO, k > 0 ? 1u : add);
                    if (HILO) umma_bf16_ts(o, ak + 16, b + k * (2048 >> 4), kIdO, 1u);
                }
            };
            // waits of the warp, lane l for the l-th barrier
            auto wait_all = [&](uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1, uint64_t* b2, uint32_t p2) {
                uint64_t* bar = lane == 0 ? b0 : lane == 1 ? b1 : b2;
                const uint32_t parity = lane == 0 ? p0 : lane == 1 ? p1 : p2;
                const bool got = __all_sync(0xffffffffu, pf_wait(bar, parity, abort_flag, lim));
                tc_fence_after_sync();
                return got;
            };
            uint64_t* k0 = &kfull[g0 % kPfStages];
            const uint32_t p0 = (uint32_t)(g0 / kPfStages) & 1u;
            bool ok = wait_all(qfull, (uint32_t)seg & 1u, k0, p0, k0, p0);
            if (ok && elect_one()) {
                scores(0, 0);
                if (nq > 1) scores(1, 0);
            }
            for (int n = 0; ok && n < nt; ++n) {
                const int g = g0 + n, last = n + 1 == nt ? g : g + 1;
                uint64_t *v = &vfull[g % kPfStages], *k = &kfull[last % kPfStages];
                const uint32_t pv = (uint32_t)(g / kPfStages) & 1u, pk = (uint32_t)(last / kPfStages) & 1u;
                for (int t = 0; t < nq; ++t) {
                    ok = wait_all(v, pv, k, pk, &pfull[t], (uint32_t)g & 1u);
                    if (!ok) break;
                    if (elect_one()) {
                        output(t, n);
                        if (n + 1 < nt) scores(t, n + 1);
                        else umma_commit(&ofull[t]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {  // let the MMAs in flight finish before their operands and TMEM go
                *abort_flag = 1;
                if (elect_one()) umma_commit(drain);
                mbar_wait(drain, 0u, lim);
            }
        } else if (warp < kPfProd && (warp >> 3) < nq) {
            const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
            constexpr int kCols = kPfKeys / 2, kOut = D / 2;  // columns of S and of O that this thread has
            const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
            const uint32_t ts = tmem + lanes + t * 128 + half * kCols, to = tmem + lanes + 256 + t * 128 + half * kOut;
            const int r = quarter * 32 + lane;  // this thread's row of the tile
            const bool mine = r < p.G * p.bpt;
            const long row = (long)(2 * pair + t) * p.G * p.bpt + r;
            const bool store = mine && row < p.M;
            const size_t at = (size_t)slot * p.M + (store ? row : 0);
            float* tops = reinterpret_cast<float*>(sm + L::oTop) + t * 256;
            // a barrier of the tile's 256 softmax threads that tells whether any of them said yes
            auto vote = [&](bool yes) {
                int any;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\t"
                    "setp.ne.s32 p, %1, 0;\n\t"
                    "barrier.cta.red.or.pred q, %2, 256, p;\n\t"
                    "selp.s32 %0, 1, 0, q;\n\t}"
                    : "=r"(any)
                    : "r"(yes ? 1 : 0), "r"(1 + t)
                    : "memory");
                return any != 0;
            };
            float m = -INFINITY, l = 0.f;
            float fm = 0.f;       // the maximum that the folded sums in the workspace are relative to
            bool folded = false;
            // this thread's columns of O_t, added to what was folded before, to the workspace
            auto write_o = [&]() {
                const float f = folded ? fast_exp2(fm - m) : 0.f;
#pragma unroll
                for (int c = 0; c < kOut / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32_nowait(to + 32 * c, o);
                    tmem_wait_ld();
                    if (store) {
                        float4* dst = reinterpret_cast<float4*>(p.o + at * D + half * kOut + 32 * c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            float4 x = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                   __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                            if (HILO && folded) {
                                const float4 y = dst[i];
                                x = make_float4(fmaf(y.x, f, x.x), fmaf(y.y, f, x.y), fmaf(y.z, f, x.z), fmaf(y.w, f, x.w));
                            }
                            dst[i] = x;
                        }
                    }
                }
                fm = m;
                folded = true;
            };
            bool ok = true;
            for (int n = 0; n < nt; ++n) {
                // every thread reaches the votes whatever its wait came to, so none waits in them for ever
                ok = pf_wait(&sfull[t], (uint32_t)(g0 + n) & 1u, abort_flag, lim);
                if (ok && (warp & 7) == 0 && lane == 0) mbar_arrive(&freed[(g0 + n) & 1]);  // this event for this row tile
                tc_fence_after_sync();
                if (HILO && n > 0 && n % kPfFold == 0) write_o();
                const int valid = p.P - (n0 + n) * kPfKeys - half * kCols;  // keys of this half within the prefix
                // 32 columns of S, the keys past the prefix as -inf
                auto load = [&](int c, uint32_t (&s)[32]) {
                    tmem_ld32_nowait(ts + 32 * c, s);
                    tmem_wait_ld();
                    if (valid < 32 * c + 32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (32 * c + i >= valid) s[i] = 0xff800000u;
                    }
                };
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    uint32_t s[32];
                    load(c, s);
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        mx[(i >> 1) & 3] = max3(mx[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                }
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                // (rows past the tile's query rows hold whatever shared memory held: they ask for nothing)
                if (vote(n == 0 || (mine && top > m + kPfGrow) || !ok)) {
                    tops[half * 128 + r] = top;
                    if (vote(*abort_flag != 0)) {  // (the vote: all of the tile's threads leave, or none)
                        ok = false;
                        break;
                    }
                    const float both = fmaxf(top, tops[(half ^ 1) * 128 + r]);
                    const float grown = n == 0 || (mine && both > m + kPfGrow) ? both : m;
                    const float f = n == 0 ? 0.f : fast_exp2(m - grown);
                    l *= f;
                    m = grown;
                    if (n > 0) {
#pragma unroll
                        for (int c = 0; c < kOut / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32_nowait(to + 32 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st16(to + 32 * c, o);
                            tmem_st16(to + 32 * c + 16, o + 16);
                        }
                    }
                    vote(false);  // the maxima are read before the next ones are written
                }
                uint64_t sum[2] = {0ull, 0ull};
                const uint64_t c2 = pack2(p.scale_log2, p.scale_log2), m2 = pack2(-m, -m);
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    uint32_t s[32], hi[16], lo[16];
                    load(c, s);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 z =
                            unpack2(fma2(pack2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, m2));
                        const float x = fast_exp2(z.x), y = fast_exp2(z.y);
                        const uint64_t xy = pack2(x, y);
                        sum[i & 1] = add2(sum[i & 1], xy);
                        hi[i] = pack_bf16x2(x, y);
                        if constexpr (HILO) {  // what is left of the weights: x - hi is exact
                            const float2 q = unpack2(fma2(pack2(bf16lo(hi[i]), bf16hi(hi[i])), pack2(-1.f, -1.f), xy));
                            lo[i] = pack_bf16x2(q.x, q.y);
                        }
                    }
                    tmem_st16(ts + 32 * c, hi);
                    if constexpr (HILO) tmem_st16(ts + 32 * c + 16, lo);
                }
                const float2 s2 = unpack2(add2(sum[0], sum[1]));
                l += s2.x + s2.y;
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[t]);
            }
            // (a tile's threads leave the loop together: by the vote, or at its end, each with its own last wait)
            if (ok) ok = pf_wait(&ofull[t], (uint32_t)seg & 1u, abort_flag, lim);
            tops[half * 128 + r] = l;
            if (!vote(!ok)) {
                tc_fence_after_sync();
                if (folded) {
                    write_o();
                } else {
                    // through the query tile's shared memory (its MMAs are done), an eighth of it a warp: a thread has
                    // a row, a store instruction whole lines of several rows
                    constexpr int kCh = D / 16;  // 16-byte chunks of a row that the warp's part holds (32 rows)
                    uint8_t* st = sm + L::oQ + t * L::kTile + (warp & 7) * (L::kTile / 8);
                    const size_t row0 = (size_t)slot * p.M + (size_t)(2 * pair + t) * p.G * p.bpt;
                    auto spot = [&](int rr, int ch) { return st + (rr * kCh + (ch ^ ((rr * kCh >> 3) & (kCh - 1)))) * 16; };
#pragma unroll
                    for (int c = 0; c < kOut / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32_nowait(to + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 8 / kCh; ++h) {
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < kCh; ++i) {
                                const int j = 4 * (h * kCh + i);
                                *reinterpret_cast<uint4*>(spot(lane, i)) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                            }
                            __syncwarp();
                            const int ch = lane & (kCh - 1);
#pragma unroll
                            for (int i = 0; i < kCh; ++i) {
                                const int rr = (32 / kCh) * i + lane / kCh, tr = quarter * 32 + rr;
                                if (tr < p.G * p.bpt && (2 * pair + t) * p.G * p.bpt + tr < p.M)
                                    *reinterpret_cast<uint4*>(p.o + (row0 + tr) * D + half * kOut + 32 * c +
                                                              4 * (h * kCh + ch)) =
                                        *reinterpret_cast<const uint4*>(spot(rr, ch));
                            }
                        }
                    }
                }
                if (store && half == 0) p.ml[at] = make_float2(m, l + tops[128 + r]);
                tc_fence_before_sync();
            }
        }
        // the next segment's queries go where this one's outputs were staged, its products where they were read
        if constexpr (EVEN) {
            fence_proxy_async_shared();
            tc_fence_before_sync();
        }
        stop = __syncthreads_or(*abort_flag) != 0;
        if (!EVEN || stop) break;
        tc_fence_after_sync();
        ++seg;
        g0 += nt;
    }
    if (stop) {
        if (tid == 32 * kPfProd) {  // let the copies in flight land
            mbar_wait(qfull, (uint32_t)seg & 1u, lim);
            for (int i = max(0, issued - 2 * kPfStages); i < issued; ++i) {
                const int n = i >> 1;
                mbar_wait((i & 1 ? vfull : kfull) + n % kPfStages, (uint32_t)(n / kPfStages) & 1u, lim);
            }
            report(p.err, SD_DEVERR_TIMEOUT);
        }
        __syncthreads();
    }
    if (warp == kPfMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
}

// 3-D tensor map of bf16 elements over [n2, n1, d] (row-major), box = 64 columns x box1 x box2,
// 128-byte swizzle, zero fill outside every dimension.
bool make_tensor_map_3d(CUtensorMap* m, const void* base, uint64_t n2, uint64_t n1, int d, int box2, int box1) {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
    auto fn = found.load(std::memory_order_relaxed);
    if (fn == nullptr) {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        found.store(fn, std::memory_order_relaxed);
    }
    cuuint64_t dims[3] = {(cuuint64_t)d, n1, n2};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, n1 * (cuuint64_t)d * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box1, (cuuint32_t)box2};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS;
}

struct PfShape {
    int bpt, row_tiles, pairs, tiles;
};
PfShape pf_shape(const sd_cache_attend_args* a) {
    PfShape s{};
    const int G = a->Hq / a->Hkv;
    s.bpt = kPfRows / G;  // (sequence, query token) entries of a row tile
    s.row_tiles = (int)(((long)a->B * a->V + s.bpt - 1) / s.bpt);
    s.pairs = (s.row_tiles + 1) / 2;
    s.tiles = (a->P + kPfKeys - 1) / kPfKeys;
    return s;
}

}  // namespace

// The plan whose slowest SM has the least to do, at kPfExtra key tiles' time for a segment's start and
// end: every head cut into so many splits, in whole waves of CTAs, or one wave of equal runs over all heads,
// some of which then hold parts of two.  (8 heads of 256 key tiles: for 1024 query rows a head 133.9 us in
// two waves of 9 splits, 123.1 in one of equal runs; for 256 rows 53.4 us in one wave of 19 splits, 54.6 in
// equal runs.)
PrefixPlan prefix_plan(const sd_cache_attend_args* a) {
    const PfShape s = pf_shape(a);
    const long units = (long)a->Hkv * s.pairs, sms = num_sms();
    PrefixPlan pl{};
    pl.tiles = s.tiles;
    pl.splits = 1;
    long cost = -1;
    for (int n = 1; n <= s.tiles && (n == 1 || units * n <= 4 * sms); ++n) {
        const long c = ((units * n + sms - 1) / sms) * ((s.tiles + n - 1) / n + kPfExtra);
        if (cost < 0 || c < cost) {
            cost = c;
            pl.splits = n;
        }
    }
    const long total = a->Hkv * ((long)s.tiles + kPfExtra), teams = std::min(sms / s.pairs, total);
    if (teams > 0 && (total + teams - 1) / teams + kPfExtra < cost) {
        pl.splits = 0;
        pl.teams = (int)teams;
        pl.slots = pl.teams + a->Hkv - 1;
        pl.cut = Cut::of((unsigned)total, (unsigned)teams);
    } else {
        pl.teams = pl.slots = a->Hkv * pl.splits;
        pl.cut = Cut::of((unsigned)s.tiles, (unsigned)pl.splits);
    }
    return pl;
}

sd_status prefix_launch(const sd_cache_attend_args* a, const PrefixPlan& plan, const CaWorkspace& w, cudaStream_t st) {
    const char* who = "sd_cache_attend";
    const PfShape s = pf_shape(a);
    CUtensorMap qmap, kmap, vmap;
    if (!make_tensor_map_3d(&qmap, a->q, (uint64_t)a->B * a->V, (uint64_t)a->Hq, a->d, s.bpt, a->Hq / a->Hkv) ||
        !make_tensor_map_3d(&kmap, a->k_prefix, (uint64_t)a->Hkv, (uint64_t)a->P, a->d, 1, kPfKeys) ||
        !make_tensor_map_3d(&vmap, a->v_prefix, (uint64_t)a->Hkv, (uint64_t)a->P, a->d, 1, kPfKeys)) {
        set_error("%s: cuTensorMapEncodeTiled failed", who);
        return SD_ERR_CUDA;
    }
    PfParams p{};
    p.ml = w.pre_ml;
    p.o = w.pre_o;
    p.err = a->err_word;
    p.G = a->Hq / a->Hkv;
    p.M = a->B * a->V * p.G;
    p.P = a->P;
    p.plan = plan;
    p.pairs = s.pairs;
    p.row_tiles = s.row_tiles;
    p.bpt = s.bpt;
    p.scale_log2 = a->scale * 1.44269504088896340736f;
    p.wait_ns = (unsigned long long)kWaitDeadlineNs;
    const bool hilo = a->out_dtype == SD_F32;
    const bool d128 = a->d == 128;
    const auto pick = [&](auto even) {
        constexpr bool E = decltype(even)::value;
        return d128 ? (hilo ? prefix_kernel<128, true, E> : prefix_kernel<128, false, E>)
                    : (hilo ? prefix_kernel<64, true, E> : prefix_kernel<64, false, E>);
    };
    const auto kern = plan.splits > 0 ? pick(std::false_type{}) : pick(std::true_type{});
    const int bytes = d128 ? PfLayout<128>::kBytes : PfLayout<64>::kBytes;
    SD_CUDA_CHECK(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes),
                  "sd_cache_attend: cudaFuncSetAttribute");
    SD_CUDA_CHECK(launch_pdl(kern, dim3((unsigned)(s.pairs * plan.teams)), dim3(kPfThreads), (size_t)bytes, st, qmap,
                             kmap, vmap, p),
                  "sd_cache_attend: prefix launch");
    return launch_status(who);
}

}  // namespace sd
