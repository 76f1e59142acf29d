// What the operators around attention work out in plain C++, on the host but for
// the waits' clock: the host tests compile this file by itself.
#pragma once

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

}  // namespace rules
}  // namespace rz
