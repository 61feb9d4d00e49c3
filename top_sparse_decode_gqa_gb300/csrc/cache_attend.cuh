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
// then the prefix's states [slots][B*V*G] (PrefixPlan).
struct CaWorkspace {
    int2* meta;       // [B*Hkv] (first slot, slots)
    float2* ml;       // [slots][R] running max (base 2) and denominator
    float* o;         // [slots][R][d] unnormalised output
    float2* pre_ml;   // [slots][B*V*G]
    float* pre_o;     // [slots][B*V*G][d]
    size_t bytes;
};

// W units cut into n runs (n <= W): the first W % n have one more.
struct Cut {
    unsigned q, rem;
    __host__ __device__ static Cut of(unsigned W, unsigned n) { return Cut{W / n, W % n}; }
    SD_DEVINL unsigned start(unsigned c) const { return c * q + min(c, rem); }
    SD_DEVINL unsigned run_of(unsigned x) const {  // the run that holds unit x
        const unsigned big = rem * (q + 1);
        return x < big ? x / (q + 1) : rem + (x - big) / q;
    }
};

constexpr unsigned kPfExtra = 4;  // key tiles' time that a segment's start and end take

// The prefix's work: `teams` of as many CTAs as there are pairs of row tiles, each team a run of key
// tiles.  splits > 0: every KV head's tiles are cut into so many runs, and slot = team.  splits == 0: all
// heads' tiles in order (each head's behind kPfExtra empty ones) are cut into `teams` runs, and slot =
// team + head, since a run may hold parts of several heads.
struct PrefixPlan {
    int splits, teams, tiles, slots;
    Cut cut;
    SD_DEVINL unsigned units() const { return (unsigned)tiles + kPfExtra; }  // of a head (splits == 0)
    // the head's first slot and how many it has
    SD_DEVINL int2 range(int kvh) const {
        if (splits > 0) return make_int2(kvh * splits, splits);
        const unsigned first = cut.run_of((unsigned)kvh * units() + kPfExtra);
        return make_int2((int)first + kvh, (int)(cut.run_of((unsigned)(kvh + 1) * units() - 1u) - first) + 1);
    }
    // splits == 0: the head that a team starts in, and its key tiles n0 .. n0 + nt - 1 of a head (nt may be
    // 0); false when its run ends before the head
    SD_DEVINL int first_head(int team) const { return (int)(cut.start((unsigned)team) / units()); }
    SD_DEVINL bool segment(int team, int kvh, int& n0, int& nt) const {
        const unsigned w0 = cut.start((unsigned)team), w1 = cut.start((unsigned)team + 1u);
        const unsigned lo = (unsigned)kvh * units() + kPfExtra, from = max(lo, w0), to = min(lo + (unsigned)tiles, w1);
        n0 = (int)(from - lo);
        nt = to > from ? (int)(to - from) : 0;
        return w1 > lo;
    }
};

struct CaPlan {
    int ctas;         // of the own rows' kernel
    int slots;
    PrefixPlan pre;   // all 0 without a prefix
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
    w.pre_ml = reinterpret_cast<float2*>(take((size_t)pl.pre.slots * M * sizeof(float2)));
    w.pre_o = reinterpret_cast<float*>(take((size_t)pl.pre.slots * M * a->d * sizeof(float)));
    w.bytes = at;
    return w;
}

// The prefix's part of a validated call (prefix_attend.cu): its plan, and the launch that writes the
// states.
PrefixPlan prefix_plan(const sd_cache_attend_args* a);
sd_status prefix_launch(const sd_cache_attend_args* a, const PrefixPlan& plan, const CaWorkspace& w, cudaStream_t st);

}  // namespace sd
