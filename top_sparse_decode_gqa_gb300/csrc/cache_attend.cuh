// cache_attend.cuh -- what the kernels of sd_cache_attend share: the call's parameters on the
// device and the layout of its workspace.
#pragma once

#include <algorithm>

#include "sd_common.cuh"
#include "sd_host.h"

namespace sd {

constexpr int kCaTile = 64;  // own rows a unit of work covers

// The workspace: per group the slots its own rows' partial states are in, then those states
// (slot = CTA + group: a CTA's work is a run of neighbouring groups, so no two states share one),
// then the prefix's states [Hkv][splits][B*V*G].
struct CaWorkspace {
    int2* meta;       // [B*Hkv] (first slot, slots)
    float2* ml;       // [slots][R] running max (base 2) and denominator
    float* o;         // [slots][R][d] unnormalised output
    float2* pre_ml;   // [Hkv][splits][B*V*G]
    float* pre_o;     // [Hkv][splits][B*V*G][d]
    size_t bytes;
};

struct CaPlan {
    int ctas;         // of the own rows' kernel
    int slots;
    int pre_splits;   // of the prefix, 0 without one
};

inline CaWorkspace ca_workspace(const sd_cache_attend_args* a, const CaPlan& pl, void* base) {
    const size_t NG = (size_t)a->B * a->Hkv, R = (size_t)(a->Hq / a->Hkv) * a->V, M = (size_t)a->B * R;
    uint8_t* p = static_cast<uint8_t*>(base);
    size_t at = 0;
    auto take = [&](size_t n) {
        uint8_t* r = p + at;
        at = (at + n + 255) & ~(size_t)255;
        return r;
    };
    CaWorkspace w{};
    w.meta = reinterpret_cast<int2*>(take(NG * sizeof(int2)));
    w.ml = reinterpret_cast<float2*>(take((size_t)pl.slots * R * sizeof(float2)));
    w.o = reinterpret_cast<float*>(take((size_t)pl.slots * R * a->d * sizeof(float)));
    w.pre_ml = reinterpret_cast<float2*>(take((size_t)a->Hkv * pl.pre_splits * M * sizeof(float2)));
    w.pre_o = reinterpret_cast<float*>(take((size_t)a->Hkv * pl.pre_splits * M * a->d * sizeof(float)));
    w.bytes = at;
    return w;
}

// The prefix's part of a validated call (prefix_attend.cu): how many splits of its rows the
// plan takes, and the launch that writes their states.
int prefix_splits(const sd_cache_attend_args* a);
sd_status prefix_launch(const sd_cache_attend_args* a, int splits, const CaWorkspace& w, cudaStream_t st);

}  // namespace sd
