// verify_drafts.cu -- acceptance of drafted tokens and the sample that follows them.
//
// "O Fim do Gargalo de Memoria: Como o Adaptive DHiSparse Revolutiona LLMs de Contexto Longo"
// (news page), "Metodologia": a verify step checks several drafted tokens at once.  The rule is
// speculative sampling: draft i is accepted while u_i * q_i(x_i) < p_i(x_i); after a accepted
// drafts the next token is drawn from max(p_a - q_a, 0) (from p_a after the last draft) by the
// inverse of its cumulative sum: the lowest t with sum_{s<=t} r_s > u * sum r.
//
// Bound: HBM (one row of p and one of q a sequence), for few sequences the chain of dependent
// loads.  One cluster of up to 8 CTAs takes a sequence.  Every warp owns one contiguous part of the
// row and sums it; the warps' sums meet through distributed shared memory, so every CTA knows
// which warp's part holds the crossing, and the CTA of that warp reads the part again (from
// L2) to find the token.  The weights are summed as integers in units of 2^-45 (each p and q is
// rounded to the nearest such multiple): the sums do not depend on the order of additions, so neither do the
// results; a fp32 sum's rounding would move the crossing past a token of 1e-5 probability about
// once in a thousand draws, this rounding (2^-39 over a row of 131072) about once in 10^6.
// Integers by two fp32 additions of a constant, whose sum's low bits are the multiple, and integer adds: 4 to 5
// instructions at full rate for each probability, where shifting its mantissa took 14 and a fp64 sum
// runs at 1/64 of the fp32 rate.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "sd_common.cuh"
#include "sd_host.h"

namespace sd {
namespace {

constexpr int kVdThreads = 512;
constexpr int kVdWarps = kVdThreads / 32;
constexpr int kVdMaxCtas = 8;
constexpr int kVdBatch = 4;    // groups of four entries a lane loads at once
constexpr int kVdPart = 4096;  // entries of a row that make a CTA of its own worth while

struct VerifyParams {
    const void* p;        // [B, V+1, N]
    const void* q;        // [B, V, N] or null
    const int32_t* draft;
    const float* u;
    const float* u_next;
    const int32_t* count;
    int32_t* tokens;
    int32_t* accepted;
    int32_t* err;
    int V, N, ctas, vec;
};

// A probability in [0, 1] as hi * 2^-22 + lo * 2^-45: x + 3 lies in [3, 4], where a fp32 number's last
// bit is 2^-22, so its bits less those of 3.0 are hi; what is left, at most 2^-23, likewise.
struct Fixed {
    int hi, lo;
};
constexpr float kFixA = 3.f, kFixB = 3.5762786865234375e-07f;  // 3, 1.5 * 2^-22
SD_DEVINL Fixed fixed45(float x) {
    x = fminf(fmaxf(x, 0.f), 1.f);  // (a NaN becomes 0: fmaxf takes the other operand)
    const float y = __fadd_rn(x, kFixA);
    const float z = __fadd_rn(__fsub_rn(x, __fsub_rn(y, kFixA)), kFixB);
    Fixed f;
    f.hi = __float_as_int(y) - __float_as_int(kFixA);
    f.lo = __float_as_int(z) - __float_as_int(kFixB);
    return f;
}
SD_DEVINL long long joined(int hi, int lo) { return ((long long)hi << 23) + lo; }

template <int DT>
SD_DEVINL float prob_at(const void* base, size_t i) {
    if constexpr (DT == SD_F32) return reinterpret_cast<const float*>(base)[i];
    if constexpr (DT == SD_BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[i] << 16);
    return __half2float(reinterpret_cast<const __half*>(base)[i]);
}

// Four neighbouring entries of a row from index i (vec: i and the row are 4-entry aligned).
template <int DT>
SD_DEVINL void prob4(const void* base, size_t row, int i, int N, bool vec, float (&x)[4]) {
    if (vec) {
        if constexpr (DT == SD_F32) {
            const float4 f = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + row + i);
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(base) + row + i);
            if constexpr (DT == SD_BF16) {
                x[0] = bf16lo(w.x), x[1] = bf16hi(w.x), x[2] = bf16lo(w.y), x[3] = bf16hi(w.y);
            } else {
                const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
                const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
                x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = i + j < N ? prob_at<DT>(base, row + i + j) : 0.f;
    }
}

// What the next token is drawn from: entry t's weight is p[prow + t], less q[qrow + t] (mode 0,
// with q) or zero at t == skip (mode 0 without q: the draft was certain of it).
template <int DT>
struct Weights {
    const void* p;
    const void* q;  // null: no q row to take away
    size_t prow, qrow;
    int skip, N;
    bool vec;
    SD_DEVINL Fixed one(float a, float b, int i) const {
        Fixed x = fixed45(a);
        if (q != nullptr) {
            const Fixed y = fixed45(b);
            x.hi -= y.hi;
            x.lo -= y.lo;
            if (!(a > b)) x.hi = x.lo = 0;
        }
        if (i == skip) x.hi = x.lo = 0;
        return x;
    }
    SD_DEVINL void four(int i, unsigned long long (&w)[4]) const {
        float a[4], b[4] = {};
        prob4<DT>(p, prow, i, N, vec, a);
        if (q != nullptr) prob4<DT>(q, qrow, i, N, vec, b);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const Fixed f = one(a[j], b[j], i + j);
            w[j] = (unsigned long long)joined(f.hi, f.lo);
        }
    }
    // the sum of the weights of K groups of four, i, i + 128, .., all loaded before any is summed
    template <int K>
    SD_DEVINL unsigned long long sum(int i, int hi_end) const {
        float a[K][4], b[K][4];
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < 4; ++j) a[k][j] = b[k][j] = 0.f;
            if (i + 128 * k < hi_end) {
                prob4<DT>(p, prow, i + 128 * k, N, vec, a[k]);
                if (q != nullptr) prob4<DT>(q, qrow, i + 128 * k, N, vec, b[k]);
            }
        }
        int hi = 0, lo = 0;  // 4 K terms of at most 2^22 each
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const Fixed f = one(a[k][j], b[k][j], i + 128 * k + j);
                hi += f.hi;
                lo += f.lo;
            }
        return (unsigned long long)joined(hi, lo);
    }
};

SD_DEVINL unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
SD_DEVINL unsigned long long warp_scan_u64(unsigned long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

template <int DT>
__global__ void __launch_bounds__(kVdThreads, 2) verify_kernel(const VerifyParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ unsigned long long wsum[kVdWarps];                 // this CTA's warps' sums (read by the cluster)
    __shared__ unsigned long long all[kVdMaxCtas * kVdWarps];     // every warp's sum
    __shared__ unsigned long long scan[kVdWarps];
    __shared__ unsigned long long s_total, s_below, s_thr;
    __shared__ int s_accept, s_cross, s_found;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = p.ctas, rank = (int)blockIdx.x % C, b = (int)blockIdx.x / C;
    const int V = p.V, N = p.N;
    pdl_wait();  // the probabilities are the preceding kernels' results
    const int n = p.count != nullptr ? max(0, min(V, p.count[b])) : V;
    if (warp == 0) {
        // (the drafts' loads wait for nothing, n least of all: what is past it is left out)
        int a = n;
        for (int base = 0; base < V; base += 32) {
            const int i = base + lane;
            int x = -1;
            float u = 0.f, px = 0.f, qx = 1.f;
            if (i < V) {
                x = p.draft[(size_t)b * V + i];
                u = p.u[(size_t)b * V + i];
            }
            const bool in = x >= 0 && x < N;
            if (in) {
                px = prob_at<DT>(p.p, ((size_t)b * (V + 1) + i) * N + x);
                if (p.q != nullptr) qx = prob_at<DT>(p.q, ((size_t)b * V + i) * N + x);
            }
            if (i < n && !in && rank == 0) report(p.err, SD_DEVERR_INDEX);
            // products of two fp32 numbers are exact in fp64
            const bool no = i < n && !(in && (double)u * (double)qx < (double)px);
            const unsigned m = __ballot_sync(0xffffffffu, no);
            if (m != 0u) {
                a = base + __ffs(m) - 1;
                break;
            }
            if (base + 32 >= n) break;
        }
        if (lane == 0) s_accept = a;
    }
    __syncthreads();
    const int a = s_accept;
    Weights<DT> w;
    w.p = p.p;
    w.q = a < n ? p.q : nullptr;
    w.prow = ((size_t)b * (V + 1) + a) * N;
    w.qrow = ((size_t)b * V + min(a, V - 1)) * N;
    w.skip = a < n && p.q == nullptr ? p.draft[(size_t)b * V + a] : -1;
    w.N = N;
    w.vec = p.vec != 0;
    // warp (rank, warp) owns entries [k * part, (k + 1) * part), k = rank * kVdWarps + warp
    const int parts = C * kVdWarps;
    const int part = ((N + parts - 1) / parts + 3) & ~3;
    const int k = rank * kVdWarps + warp;
    for (int mode = 0;; ++mode) {
        const long lo = (long)k * part, hi = min((long)N, lo + part);
        unsigned long long sum = 0ull;
        for (long i = lo + 4 * lane; i < hi; i += 128 * kVdBatch) sum += w.template sum<kVdBatch>((int)i, (int)hi);
        sum = warp_sum_u64(sum);
        if (lane == 0) wsum[warp] = sum;
        cluster.sync();
        if (tid < parts) all[tid] = *cluster.map_shared_rank(&wsum[tid % kVdWarps], tid / kVdWarps);
        cluster.barrier_arrive();  // (waited for where this CTA would write wsum again or leave)
        __syncthreads();
        if (warp == 0) {
            constexpr int kPer = kVdMaxCtas * kVdWarps / 32;
            unsigned long long v[kPer], mine = 0ull;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                v[j] = lane * kPer + j < parts ? all[lane * kPer + j] : 0ull;
                mine += v[j];
            }
            const unsigned long long incl = warp_scan_u64(mine, lane);
            const unsigned long long total = __shfl_sync(0xffffffffu, incl, 31);
            // u * total, rounded down: an integer sum exceeds the product exactly when it
            // exceeds its floor
            const float u = fminf(fmaxf(p.u_next[b], 0.f), 0.99999994f);
            const unsigned long long thr = __umul64hi(__float2ull_rz(u * 18446744073709551616.f), total);
            const unsigned hit = __ballot_sync(0xffffffffu, incl > thr);
            if (lane == 0) {
                s_total = total;
                s_thr = thr;
            }
            if (hit != 0u && lane == __ffs(hit) - 1) {
                unsigned long long below = incl - mine;
                int j = 0;
                while (below + v[j] <= thr) below += v[j++];
                s_cross = lane * kPer + j;
                s_below = below;
            }
        }
        __syncthreads();
        if (s_total != 0ull || mode == 1) break;
        cluster.barrier_wait();
        w.q = nullptr;  // p and q are equal (no residual): the target itself
        w.skip = -1;
        __syncthreads();
    }
    int32_t* out = p.tokens + (size_t)b * (V + 1);
    if (rank == 0) {
        for (int i = tid; i <= V; i += kVdThreads)
            if (i != a) out[i] = i < a ? p.draft[(size_t)b * V + i] : -1;
        if (tid == 0) {
            p.accepted[b] = a;
            if (s_total == 0ull) out[a] = -1;  // a row of zeros: no token
        }
    }
    if (s_total == 0ull || s_cross / kVdWarps != rank) {
        cluster.barrier_wait();
        return;
    }
    // the part of warp s_cross: a scan over it, 4 entries a thread
    const int lo = s_cross * part, hi = min(N, lo + part);
    const unsigned long long thr = s_thr;
    unsigned long long below = s_below;
    if (tid == 0) s_found = 0;
    for (int base = lo; base < hi; base += 4 * kVdThreads) {
        const int i = base + 4 * tid;
        unsigned long long x[4] = {0ull, 0ull, 0ull, 0ull};
        if (i < hi) w.four(i, x);
        const unsigned long long mine = (x[0] + x[1]) + (x[2] + x[3]);
        const unsigned long long incl = warp_scan_u64(mine, lane);
        if (lane == 31) scan[warp] = incl;
        __syncthreads();
        unsigned long long before = below, whole = 0ull;
        for (int j = 0; j < kVdWarps; ++j) {
            if (j < warp) before += scan[j];
            whole += scan[j];
        }
        unsigned long long c = before + incl - mine;
        if (c <= thr && c + mine > thr) {  // the crossing is among this thread's entries
            int j = 0;
            while (c + x[j] <= thr) c += x[j++];
            out[a] = i + j;
            s_found = 1;
        }
        below += whole;
        __syncthreads();
        if (s_found) break;
    }
    cluster.barrier_wait();
}

template <int DT>
sd_status verify_launch(const VerifyParams& p, int B, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)B * p.ctas);
    cfg.blockDim = dim3(kVdThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    SD_CUDA_CHECK(cudaLaunchKernelEx(&cfg, verify_kernel<DT>, p), "sd_verify_drafts: launch");
    return launch_status("sd_verify_drafts");
}

}  // namespace
}  // namespace sd

using namespace sd;

extern "C" sd_status sd_verify_drafts(const void* p, const void* q, sd_dtype dtype, const int32_t* draft, const float* u,
                                      const float* u_next, const int32_t* count, int B, int V, int N, int32_t* tokens,
                                      int32_t* accepted, int32_t* err_word, void* stream) {
    clear_error();
    const char* who = "sd_verify_drafts";
    SD_REQUIRE(dtype == SD_F32 || dtype == SD_BF16 || dtype == SD_F16, "%s: bad dtype", who);
    SD_REQUIRE(B >= 0 && V >= 0 && V <= 1024 && N >= 1 && N <= (1 << 24), "%s: bad sizes (B=%d V=%d N=%d)", who, B, V, N);
    SD_REQUIRE((long)B * kVdMaxCtas < (1L << 31), "%s: B too large", who);
    if (B == 0) return SD_OK;
    SD_REQUIRE(p && u_next && tokens && accepted && (V == 0 || (draft && u)), "%s: null pointer", who);
    SD_REQUIRE(aligned16(p) && aligned16(q), "%s: probabilities must be 16-byte aligned", who);
    VerifyParams a{};
    a.p = p;
    a.q = q;
    a.draft = draft;
    a.u = u;
    a.u_next = u_next;
    a.count = count;
    a.tokens = tokens;
    a.accepted = accepted;
    a.err = err_word;
    a.V = V;
    a.N = N;
    a.vec = N % 4 == 0;  // then every row starts at a 4-entry boundary
    // as many CTAs a sequence as fit on the GPU at once (two an SM), each with a part worth reading
    int C = kVdMaxCtas;
    while (C > 1 && ((long)B * C > 2L * num_sms() || (N + C - 1) / C < kVdPart / 2)) C /= 2;
    a.ctas = C;
    cudaStream_t st = as_stream(stream);
    return dtype == SD_F32 ? verify_launch<SD_F32>(a, B, st)
                           : dtype == SD_BF16 ? verify_launch<SD_BF16>(a, B, st) : verify_launch<SD_F16>(a, B, st);
}
