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
// twice.  A warp takes a block of neighbouring tokens of one head (8 at d = 128) and loads all of it before
// it reduces any row: 2 KB of 16-bit rows in flight a warp, whole kilobytes written side by side.  Blocks
// run over (sequence, tokens, K heads then V heads) with the head fastest, so that the CTAs at
// work read neighbouring memory when the source is a projection's [B, n, heads, d] output.  The
// 2 divisions of each of a block's 8 rows are one division instruction sequence, a lane each.
#include <cuda_fp8.h>

#include "sd_common.cuh"
#include "sd_host.h"

namespace sd {
namespace {

constexpr int kAppendThreads = 128;  // (a 4 x 8192-token prompt: 34.8 us, 37.3 with 256)
constexpr int kAppendLoads = 4;      // rows a lane loads together (2: 39.3 us, 8: 39.8)
constexpr float kAppendTiny = 7.888609052210118e-31f;  // 2^-100

struct AppendParams {
    const uint8_t* src[2];      // K, V
    long long sb[2], sh[2], sn[2];  // element strides of the source
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* pos0;
    const int32_t* count;
    int32_t* err;
    int Hkv, n, T;
    unsigned nb, tasks;  // token blocks of a sequence; B * nb * 2 * Hkv
};

template <int SRC>  // 8 elements of a row in fp32 (sd_dtype)
struct Eight {
    uint4 r[SRC == SD_F32 ? 2 : 1];
    SD_DEVINL void load(const uint8_t* p) {
        r[0] = *reinterpret_cast<const uint4*>(p);
        if constexpr (SRC == SD_F32) r[1] = reinterpret_cast<const uint4*>(p)[1];
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
    constexpr int kPerWarp = 32 / kLanes;      // rows a warp loads at once
    constexpr int kEs = SRC == SD_F32 ? 4 : 2;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, col = lane % kLanes;
    const unsigned task = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (task >= p.tasks) return;
    const unsigned heads = 2u * (unsigned)p.Hkv;
    const unsigned blk = task / heads, hv = task - blk * heads;
    const unsigned b = blk / p.nb, i0 = (blk - b * p.nb) * (U * kPerWarp);
    const int kv = hv >= (unsigned)p.Hkv ? 1 : 0;
    const unsigned h = hv - (kv ? (unsigned)p.Hkv : 0u);
    pdl_wait();  // the new rows may come from the preceding kernel
    const int first = p.pos0[b], cnt = min(p.n, p.count != nullptr ? p.count[b] : p.n);
    const long long sn = kv ? p.sn[1] : p.sn[0];
    const uint8_t* src = (kv ? p.src[1] : p.src[0]) +
                         ((long long)b * (kv ? p.sb[1] : p.sb[0]) + (long long)h * (kv ? p.sh[1] : p.sh[0]) + col * 8) * kEs;
    Eight<SRC> x[U];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (int)i0 + u * kPerWarp + sub;
        const long long pos = (long long)first + i;
        on[u] = i < cnt;
        if (on[u] && (pos < 0 || pos >= p.T)) {
            if (col == 0) report(p.err, SD_DEVERR_INDEX);
            on[u] = false;
        }
        if (on[u])
            x[u].load(src + i * sn * kEs);
        else
            x[u].zero();
    }
    float a[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[8];
        x[u].get(f);
        a[u] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[u] = fmaxf(a[u], fabsf(f[j]));
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) a[u] = fmaxf(a[u], __shfl_xor_sync(0xffffffffu, a[u], o));
    // lane 2u of a row's lanes divides top / a[u], lane 2u + 1 a[u] / top (a row below the smallest kept: 0)
    constexpr float top = E4M3 ? 448.f : 127.f;
    float mine = a[0];
#pragma unroll
    for (int u = 1; u < U; ++u) mine = (col >> 1) == u ? a[u] : mine;
    const bool odd = (col & 1) != 0;
    float r = __fdiv_rn(odd ? mine : top, odd ? top : mine);
    if (mine < kAppendTiny) r = 0.f;
    uint8_t* out = kv ? p.codes[1] : p.codes[0];
    float* scale = kv ? p.scale[1] : p.scale[0];
    const long long row0 = ((long long)b * p.Hkv + h) * p.T + first + (int)i0 + sub;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float inv = __shfl_sync(0xffffffffu, r, sub * kLanes + 2 * u);
        if (!on[u]) continue;
        float f[8];
        x[u].get(f);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], inv);
        uint2 c;
        if constexpr (E4M3) {
            c.x = pack_e4m3(f[0], f[1], f[2], f[3]);
            c.y = pack_e4m3(f[4], f[5], f[6], f[7]);
        } else {
            c.x = pack_int8(f[0], f[1], f[2], f[3]);
            c.y = pack_int8(f[4], f[5], f[6], f[7]);
        }
        const long long row = row0 + u * kPerWarp;
        *reinterpret_cast<uint2*>(out + row * D + col * 8) = c;
        if (col == 2 * u + 1) scale[row] = r;
    }
}

template <int SRC, bool E4M3, int D, int U>
cudaError_t append_launch_u(AppendParams p, int B, cudaStream_t st) {
    constexpr int kBlock = U * (32 / (D / 8)), kWarps = kAppendThreads / 32;
    p.nb = ((unsigned)p.n + kBlock - 1) / kBlock;
    p.tasks = (unsigned)B * p.nb * 2u * (unsigned)p.Hkv;
    return launch_pdl(q8_append_kernel<SRC, E4M3, D, U>, dim3((p.tasks + kWarps - 1) / kWarps), dim3(kAppendThreads), 0, st,
                      p);
}

template <int SRC, bool E4M3, int D>
cudaError_t append_launch(const AppendParams& p, int B, cudaStream_t st) {
    // Blocks of 4 loads a lane once every SM has two CTAs of such blocks, else of one (a decode
    // step's 128 rows are then 64 to 128 warps' work, not 16).
    constexpr int kBlock = kAppendLoads * (32 / (D / 8)), kWarps = kAppendThreads / 32;
    const long long many = (long long)B * ((p.n + kBlock - 1) / kBlock) * 2 * p.Hkv;
    return many >= 2LL * num_sms() * kWarps ? append_launch_u<SRC, E4M3, D, kAppendLoads>(p, B, st)
                                            : append_launch_u<SRC, E4M3, D, 1>(p, B, st);
}

template <int SRC>
cudaError_t append_dispatch(const AppendParams& p, int B, bool e4m3, int d, cudaStream_t st) {
    if (e4m3) return d == 128 ? append_launch<SRC, true, 128>(p, B, st) : append_launch<SRC, true, 64>(p, B, st);
    return d == 128 ? append_launch<SRC, false, 128>(p, B, st) : append_launch<SRC, false, 64>(p, B, st);
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
    SD_REQUIRE(a->Hkv <= 65535, "%s: Hkv must be <= 65535", who);
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
    p.Hkv = a->Hkv;
    p.n = a->n;
    p.T = a->T;
    const bool e4m3 = a->code_dtype == SD_E4M3;
    cudaStream_t st = as_stream(stream);
    cudaError_t e = a->dtype == SD_F32   ? append_dispatch<SD_F32>(p, a->B, e4m3, a->d, st)
                    : a->dtype == SD_F16 ? append_dispatch<SD_F16>(p, a->B, e4m3, a->d, st)
                                         : append_dispatch<SD_BF16>(p, a->B, e4m3, a->d, st);
    SD_CUDA_CHECK(e, "sd_q8_append: launch");
    return launch_status(who);
}
