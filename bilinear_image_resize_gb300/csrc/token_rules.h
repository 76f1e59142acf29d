// What the map operators work out in plain C++, on the host but for
// the waits' clock: the host tests compile this file by itself.
#pragma once

#include <cmath>
#include <vector>

#ifdef __CUDACC__
#define RZ_BOTH __host__ __device__ __forceinline__
#else
#define RZ_BOTH inline
#endif

namespace rz {
namespace rules {

// The clock of a bounded wait, in nanoseconds.  A wait looks again at least every
// millisecond while its kernel runs; what lies between two looks counts as ten at
// most, so that the time slices of other programs, in which nothing that it waits
// for can happen either, do not use up its limit.
struct WaitClock {
    unsigned long long last, waited = 0;
    RZ_BOTH explicit WaitClock(unsigned long long now) : last(now) {}
    RZ_BOTH bool over(unsigned long long now, unsigned long long limit)
    {
        const unsigned long long step = now - last, most = 10000000ull;
        last = now;
        waited += step < most ? step : most;
        return waited > limit;
    }
};

constexpr int kSms = 152;

// The shared memory that kernels have been opted into, by device; grant(bytes) asks
// for it and gives 0, or an error that is handed on.  A kernel that asks for more
// than it was given asks again.
class Granted {
    struct Entry {
        int device;
        const void *fn;
        int bytes;
    };
    std::vector<Entry> entries;

public:
    template <class F>
    int have(int device, const void *fn, int bytes, const F &grant)
    {
        Entry *found = nullptr;
        for (Entry &e : entries)
            if (e.device == device && e.fn == fn) found = &e;
        if (found && found->bytes >= bytes) return 0;
        if (const int error = grant(bytes)) return error;
        if (found) {
            found->bytes = bytes;
            return 0;
        }
        try {
            entries.push_back({device, fn, bytes});
        } catch (...) {
            // not remembered: asked for again by the next call
        }
        return 0;
    }
};

// How the norm of queries and keys cuts a token's heads, where there are few tokens:
// into more runs, down to one step a warp, until there are two CTAs' warps an SM.
// `lanes` of a warp hold a head.  Every run has heads: run i begins at i * chunk <
// heads, which the gradient's two walks rely on.
struct Runs {
    int chunks, chunk;      // runs of a token, heads of each but the last
};
inline Runs head_runs(int heads, int lanes, long long tokens, int warps)
{
    const int most = (heads * lanes + 31) / 32;
    int chunks = 1;
    while (chunks < most && tokens * chunks < 2LL * kSms * warps) chunks++;
    const int chunk = (heads + chunks - 1) / chunks;
    return {(heads + chunk - 1) / chunk, chunk};
}

// A number as the sum of two float64 that do not overlap, good to about 2^-100 of it
// (Dekker, "A floating-point technique for extending the available precision", 1971).
struct Pair {
    double hi, lo;
};
inline Pair sum_of(double big, double small)
{
    const double s = big + small;
    return {s, small - (s - big)};
}
inline Pair product_of(Pair a, Pair b)
{
    const double p = a.hi * b.hi;
    return sum_of(p, std::fma(a.hi, b.hi, -p) + (a.hi * b.lo + a.lo * b.hi));
}
// x^n 2^-e with the leading part in [1/2, 1), so that no power passes float64's range.
inline Pair power_of(Pair x, int n, int *e)
{
    Pair r{0.5, 0.0};
    int re = 1, xe = 0;
    const auto scaled = [](Pair v, int *exponent) {
        int k;
        std::frexp(v.hi, &k);
        *exponent += k;
        return Pair{std::ldexp(v.hi, -k), std::ldexp(v.lo, -k)};
    };
    x = scaled(x, &xe);
    for (; n; n >>= 1) {
        if (n & 1) {
            re += xe;
            r = scaled(product_of(r, x), &re);
        }
        xe *= 2;
        x = scaled(product_of(x, x), &xe);
    }
    *e = re;
    return r;
}

// The turns of a position step of each pair j, scale base^(-j / pairs) / (2 pi), in
// 2^-64 and without whole turns, off by less than 2^-63 of a turn plus 2^-92 of the
// step: float64's 2^-53 would leave a position of 2^31 off by 2^-22 of a turn and more.
// A pair costs a product of two numbers (64 pairs 0.7 us on the host, 13 with a root for each).
inline void turns_of(double base, double scale, int pairs, unsigned long long *out)
{
    // y = base^(-1 / pairs) from float64's: one Newton step on y^pairs base = 1, whose left side is found to 2^-96
    Pair y{std::pow(base, -1.0 / pairs), 0.0};
    if (pairs > 1 && std::isnormal(y.hi)) {
        int ey, eb;
        const Pair p = product_of(power_of(y, pairs, &ey), power_of({base, 0.0}, 1, &eb));
        const double off = (std::ldexp(p.hi, ey + eb) - 1.0) + std::ldexp(p.lo, ey + eb);   // about 2^-53 pairs
        y = sum_of(y.hi, -y.hi * off / pairs);
    }
    // modulo a turn, in two's complement
    const auto bits = [](double v) {
        v = (v - std::nearbyint(v)) * 0x1p64;
        return v < 0.0 ? 0ull - static_cast<unsigned long long>(-v) : static_cast<unsigned long long>(v);
    };
    Pair f = product_of({0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57}, {scale, 0.0});      // 1 / (2 pi) first
    for (int j = 0; j < pairs; j++, f = product_of(f, y))
        out[j] = std::isfinite(f.hi) && std::isfinite(f.lo) ? bits(f.hi) + bits(f.lo) : 0ull;
}

}  // namespace rules
}  // namespace rz
