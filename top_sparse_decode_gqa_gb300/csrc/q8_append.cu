// q8_append.cu -- new tokens' K/V rows quantised as they are written into an 8-bit cache.
//
// "Nem Todos os Pensamentos Necessitam de HBM" (gist.science summary), Metodologia 1, keeps
// rows "e.g. 8-bit"; here a whole cache is kept so from the moment a row is written.  Per row
// of d elements: a = max_j |x_j|, code_j = round(x_j * (top / a)), scale = a / top, with top =
// 127 (int8, round half to even) or 448 (e4m3, round to nearest even).  Every division and
// product is one correctly rounded fp32 operation.
//
// Bound: HBM (each row is read once and written once at half or a quarter of its size), for a
// few rows the launch.  A row is held in registers by d/8 lanes (8 elements a lane: one or two
// 16-byte loads, one 8-byte store), so the maximum is a shuffle reduction and no row is read
// twice; a warp loads kAppendRows row groups before it reduces any, which keeps 4 to 8 KB per warp in
// flight.  The row index runs over (K or V, b, h, i) with i fastest: the rows a warp writes are
// neighbours in the cache whatever the order of the source, whose rows are whole 128-byte lines.
#include <cuda_fp8.h>

#include "sd_common.cuh"
#include "sd_host.h"

namespace sd {
namespace {

constexpr int kAppendThreads = 256;
constexpr float kAppendTiny = 7.888609052210118e-31f;  // 2^-100

struct AppendParams {
    const uint8_t* src[2];      // K, V
    long long sb[2], sh[2], sn[2];  // element strides of the source
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* pos0;
    const int32_t* count;
    int32_t* err;
    int B, Hkv, n, T;
    unsigned rows;  // B * Hkv * n
};

template <int SRC>  // 8 elements of a row in fp32 (sd_dtype)
struct Eight {
    uint4 r[SRC == SD_F32 ? 2 : 1];
    SD_DEVINL void load(const uint8_t* p) {
        r[0] = __ldg(reinterpret_cast<const uint4*>(p));
        if constexpr (SRC == SD_F32) r[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    }
    SD_DEVINL void zero() {
        r[0] = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (SRC == SD_F32) r[1] = r[0];
    }
    SD_DEVINL void get(float (&x)[8]) const {
        if constexpr (SRC == SD_F32) {
            Unpack16<float>::run(r[0], x);
            Unpack16<float>::run(r[1], x + 4);
        } else if constexpr (SRC == SD_BF16) {
            Unpack16<bf16_t>::run(r[0], x);
        } else {
            const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                x[2 * j] = f.x;
                x[2 * j + 1] = f.y;
            }
        }
    }
};

SD_DEVINL uint32_t pack_int8(float a, float b, float c, float d) {
    auto q = [](float x) { return (uint32_t)max(-127, min(127, __float2int_rn(x))) & 0xffu; };
    return q(a) | (q(b) << 8) | (q(c) << 16) | (q(d) << 24);
}
SD_DEVINL uint32_t pack_e4m3(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <int SRC, bool E4M3, int D, int U>
__global__ void __launch_bounds__(kAppendThreads) q8_append_kernel(const AppendParams p) {
    constexpr int kLanes = D / 8;              // lanes of a row
    constexpr int kPerWarp = 32 / kLanes;      // rows a warp holds at once
    constexpr int kEs = SRC == SD_F32 ? 4 : 2;
    pdl_wait();  // the new rows may come from the preceding kernel
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane / kLanes, col = lane % kLanes;
    const unsigned warp = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const unsigned total = 2u * p.rows;
    Eight<SRC> x[U];
    long long dst[U];  // destination row, or -1
    int which[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned r = (warp * U + u) * kPerWarp + sub;
        dst[u] = -1;
        which[u] = 0;
        x[u].zero();
        if (r < total) {
            const int kv = r >= p.rows ? 1 : 0;
            const unsigned rr = r - (kv ? p.rows : 0u);
            const unsigned g = rr / (unsigned)p.n, i = rr - g * (unsigned)p.n;
            const unsigned b = g / (unsigned)p.Hkv, h = g - b * (unsigned)p.Hkv;
            const int cnt = p.count != nullptr ? p.count[b] : p.n;
            if ((int)i < cnt) {
                const long long pos = (long long)p.pos0[b] + i;
                if (pos < 0 || pos >= p.T) {
                    if (col == 0) report(p.err, SD_DEVERR_INDEX);
                } else {
                    dst[u] = (long long)g * p.T + pos;
                    which[u] = kv;
                    const uint8_t* s = kv ? p.src[1] : p.src[0];
                    const long long off = (long long)b * (kv ? p.sb[1] : p.sb[0]) +
                                          (long long)h * (kv ? p.sh[1] : p.sh[0]) +
                                          (long long)i * (kv ? p.sn[1] : p.sn[0]) + col * 8;
                    x[u].load(s + off * kEs);
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[8];
        x[u].get(f);
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(f[j]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (dst[u] < 0) continue;
        const float top = E4M3 ? 448.f : 127.f;
        const bool zero = a < kAppendTiny;
        const float inv = zero ? 0.f : __fdiv_rn(top, a);
        const float scale = zero ? 0.f : __fdiv_rn(a, top);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = zero ? 0.f : __fmul_rn(f[j], inv);
        uint2 c;
        if constexpr (E4M3) {
            c.x = pack_e4m3(f[0], f[1], f[2], f[3]);
            c.y = pack_e4m3(f[4], f[5], f[6], f[7]);
        } else {
            c.x = pack_int8(f[0], f[1], f[2], f[3]);
            c.y = pack_int8(f[4], f[5], f[6], f[7]);
        }
        uint8_t* out = which[u] ? p.codes[1] : p.codes[0];
        *reinterpret_cast<uint2*>(out + dst[u] * D + col * 8) = c;
        if (col == 0) (which[u] ? p.scale[1] : p.scale[0])[dst[u]] = scale;
    }
}

template <int SRC, bool E4M3, int D>
cudaError_t append_launch(const AppendParams& p, cudaStream_t st) {
    constexpr int kPerWarp = 32 / (D / 8), kWarps = kAppendThreads / 32;
    const unsigned total = 2u * p.rows;
    // Four rows a lane in flight once every SM has work at that, else one (a decode step's few
    // rows: 8192 warps hide the latency of one load, and 128 rows want 64 warps, not 16).
    const bool many = total >= (unsigned)num_sms() * kWarps * kPerWarp * 4;
    const unsigned per = kWarps * kPerWarp * (many ? 4u : 1u);
    const unsigned grid = (total + per - 1) / per;
    return many ? launch_pdl(q8_append_kernel<SRC, E4M3, D, 4>, dim3(grid), dim3(kAppendThreads), 0, st, p)
                : launch_pdl(q8_append_kernel<SRC, E4M3, D, 1>, dim3(grid), dim3(kAppendThreads), 0, st, p);
}

template <int SRC>
cudaError_t append_dispatch(const AppendParams& p, bool e4m3, int d, cudaStream_t st) {
    if (e4m3) return d == 128 ? append_launch<SRC, true, 128>(p, st) : append_launch<SRC, true, 64>(p, st);
    return d == 128 ? append_launch<SRC, false, 128>(p, st) : append_launch<SRC, false, 64>(p, st);
}

}  // namespace
}  // namespace sd

using namespace sd;

extern "C" sd_status sd_q8_append(const sd_q8_append_args* a, void* stream) {
    clear_error();
    const char* who = "sd_q8_append";
    SD_REQUIRE(a != nullptr, "%s: null args", who);
    SD_REQUIRE(a->dtype == SD_F32 || a->dtype == SD_BF16 || a->dtype == SD_F16, "%s: bad source dtype", who);
    SD_REQUIRE(a->code_dtype == SD_I8 || a->code_dtype == SD_E4M3, "%s: codes are SD_I8 or SD_E4M3", who);
    SD_REQUIRE(a->B >= 0 && a->n >= 0 && a->Hkv >= 1 && a->T >= 1, "%s: bad sizes (B=%d Hkv=%d n=%d T=%d)", who, a->B,
               a->Hkv, a->n, a->T);
    if (a->d != 64 && a->d != 128) {
        set_error("%s: d must be 64 or 128 (got %d)", who, a->d);
        return SD_ERR_UNSUPPORTED;
    }
    SD_REQUIRE((double)a->B * a->Hkv * a->n < 1073741824.0, "%s: B*Hkv*n must be below 2^30", who);
    if (a->B == 0 || a->n == 0) return SD_OK;
    SD_REQUIRE(a->k_new && a->v_new && a->k_codes && a->v_codes && a->k_scale && a->v_scale && a->pos0,
               "%s: null pointer", who);
    SD_REQUIRE(aligned16(a->k_new) && aligned16(a->v_new) && aligned16(a->k_codes) && aligned16(a->v_codes),
               "%s: rows and codes must be 16-byte aligned", who);
    const long long lines = a->dtype == SD_F32 ? 4 : 8;  // elements in 16 bytes
    const long long s[6] = {a->k_stride_b, a->k_stride_h, a->k_stride_n, a->v_stride_b, a->v_stride_h, a->v_stride_n};
    for (int i = 0; i < 6; ++i)
        SD_REQUIRE(s[i] >= 0 && s[i] % lines == 0, "%s: strides must be multiples of 16 bytes and not negative", who);
    AppendParams p{};
    p.src[0] = static_cast<const uint8_t*>(a->k_new);
    p.src[1] = static_cast<const uint8_t*>(a->v_new);
    for (int v = 0; v < 2; ++v) {
        p.sb[v] = s[3 * v];
        p.sh[v] = s[3 * v + 1];
        p.sn[v] = s[3 * v + 2];
    }
    p.codes[0] = static_cast<uint8_t*>(a->k_codes);
    p.codes[1] = static_cast<uint8_t*>(a->v_codes);
    p.scale[0] = a->k_scale;
    p.scale[1] = a->v_scale;
    p.pos0 = a->pos0;
    p.count = a->count;
    p.err = a->err_word;
    p.B = a->B;
    p.Hkv = a->Hkv;
    p.n = a->n;
    p.T = a->T;
    p.rows = (unsigned)a->B * a->Hkv * a->n;
    const bool e4m3 = a->code_dtype == SD_E4M3;
    cudaStream_t st = as_stream(stream);
    cudaError_t e = a->dtype == SD_F32   ? append_dispatch<SD_F32>(p, e4m3, a->d, st)
                    : a->dtype == SD_F16 ? append_dispatch<SD_F16>(p, e4m3, a->d, st)
                                         : append_dispatch<SD_BF16>(p, e4m3, a->d, st);
    SD_CUDA_CHECK(e, "sd_q8_append: launch");
    return launch_status(who);
}
