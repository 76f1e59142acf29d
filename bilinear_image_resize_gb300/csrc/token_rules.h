// What the operators around attention work out on the host, in plain C++: the
// host tests compile this file by itself.
#pragma once

namespace rz {
namespace rules {

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
