// kda_mla_split.h -- where the absorbed decode cuts its work, as arithmetic for the host and the device alike: `total`
// places (tiles and what each sequence costs besides) in `groups` equal ranges, range g beginning at total g / groups.
#pragma once

#if defined(__CUDACC__)
#define KDA_BOTH __host__ __device__ __forceinline__
#else
#define KDA_BOTH inline
#endif

namespace kda {
namespace mla {

// x a / b for 0 <= a, b <= 148; the 64-bit division, some 400 cycles of latency, only for what 32 bits do not hold.
KDA_BOTH long long scaled(long long x, int a, int b) {
    if (x < (1 << 24)) return static_cast<unsigned>(x) * static_cast<unsigned>(a) / static_cast<unsigned>(b);
    return x * a / b;
}
// The largest group whose range begins at or before `place` < total: (place + 1) groups - 1 over total.
KDA_BOTH int group_of(long long place, int groups, long long total) {
    const long long n = (place + 1) * groups - 1;
    if (n < (1ll << 32) && total < (1ll << 32)) return static_cast<int>(static_cast<unsigned>(n) / static_cast<unsigned>(total));
    return static_cast<int>(n / total);
}

}  // namespace mla
}  // namespace kda
