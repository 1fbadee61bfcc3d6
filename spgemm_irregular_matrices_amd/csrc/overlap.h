// Whether strided tensors of bytes share any (host code).
#pragma once

#include <algorithm>
#include <cstdint>

namespace sg {

// Bytes [0, width) at base + sum of stride[i] * x, x in [0, count[i]). Strides of
// counts up to 1 are not used, others are not negative.
struct Places {
    int64_t base, width;
    int64_t stride[3], count[3];
};

// Whether no two of a tensor's places share a byte: in ascending order, every
// stride passes all that is reached by those below it.
inline bool places_apart(const Places& p) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return p.stride[a] < p.stride[b]; });
    __int128 span = p.width;
    for (int i : order) {
        if (p.count[i] <= 1) continue;
        if (p.stride[i] < span) return false;
        span += (__int128)p.stride[i] * (p.count[i] - 1);
    }
    return true;
}

// Whether two tensors, each with its places apart, share a byte. The difference of two
// places is a sum of strides times differences of indexes (of an index of each where
// both have that stride): the largest strides first, only those differences are looked
// at that the smaller ones can still make 0. Tensors of one allocation have the same
// large strides and take a handful of steps; strides so odd that it takes thousands
// count as meeting.
struct Meeting {
    struct Axis {
        int64_t stride, low, high;
    };
    Axis axes[6];
    int n = 0, steps = 4096;
    __int128 low[7], high[7];  // what axes from i on, and the bytes, add at least and at most

    Meeting(const Places& a, const Places& b) {
        for (int i = 0; i < 3; ++i) add(a, i, 0);
        for (int i = 0; i < 3; ++i) add(b, i, 1);
        std::sort(axes, axes + n, [](const Axis& x, const Axis& y) { return x.stride > y.stride; });
        low[n] = -(a.width - 1);
        high[n] = b.width - 1;
        for (int i = n - 1; i >= 0; --i) {
            low[i] = low[i + 1] + (__int128)axes[i].stride * axes[i].low;
            high[i] = high[i + 1] + (__int128)axes[i].stride * axes[i].high;
        }
    }
    void add(const Places& p, int i, int side) {
        if (p.count[i] <= 1) return;
        int j = 0;
        while (j < n && axes[j].stride != p.stride[i]) ++j;
        if (j == n) axes[n++] = {p.stride[i], 0, 0};
        (side ? axes[j].high : axes[j].low) += side ? p.count[i] - 1 : 1 - p.count[i];
    }
    // Whether `d` and axes from i on can make 0.
    bool from(int i, __int128 d) {
        if (d + low[i] > 0 || d + high[i] < 0) return false;
        if (i == n || --steps < 0) return true;
        const Axis& x = axes[i];
        // d + stride * k + [low, high] of the rest holds 0
        const __int128 first = -d - high[i + 1], last = -d - low[i + 1];
        const __int128 k0 = first > 0 ? (first + x.stride - 1) / x.stride : -(-first / x.stride);
        const __int128 k1 = last >= 0 ? last / x.stride : -((-last + x.stride - 1) / x.stride);
        for (__int128 k = std::max<__int128>(k0, x.low); k <= std::min<__int128>(k1, x.high); ++k)
            if (from(i + 1, d + k * x.stride)) return true;
        return false;
    }
};
inline bool places_meet(const Places& a, const Places& b) {
    return Meeting(a, b).from(0, (__int128)b.base - a.base);
}

}  // namespace sg
