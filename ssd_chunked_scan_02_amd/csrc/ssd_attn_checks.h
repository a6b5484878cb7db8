// Argument checks that the entry points of the attention layer and of its 8-bit cache share, and how a decode step is split (host only).
#pragma once

#include <cmath>

#include "ssd_attn.h"
#include "ssd_attn_launch.h"
#include "ssd_checks.h"

namespace ssd {
namespace checks {

// A whole number (little-endian 32-bit limbs), so that bucket borders are compared without rounding.  The
// largest is 1025^32 * 32^32, under 2^481.
struct Whole {
    uint32_t limb[16] = {1};
    void times_power(uint32_t f, int n) {
        while (n-- > 0) {
            uint64_t carry = 0;
            for (uint32_t& x : limb) {
                carry += (uint64_t)x * f;
                x = (uint32_t)carry;
                carry >>= 32;
            }
        }
    }
    bool at_least(const Whole& o) const {
        for (int i = 15; i >= 0; --i)
            if (limb[i] != o.limb[i]) return limb[i] > o.limb[i];
        return true;
    }
};

// Is bucket e + k reached at distance d, (d / e)^f >= (m / e)^k, that is d^f e^k >= m^k e^f?
inline bool reached(int d, int e, int f, int m, int k) {
    Whole a, b;
    a.times_power((uint32_t)d, f);
    a.times_power((uint32_t)e, k);
    b.times_power((uint32_t)m, k);
    b.times_power((uint32_t)e, f);
    return a.at_least(b);
}

// The distances at which a direction's bucket goes up by one: e - 1 of them one apart, then f.
inline int make_buckets(ssd::AttnBuckets& out, int num_buckets, int max_distance, int both) {
    if (both != 0 && both != 1) return SSD_ERR_INVALID;
    const int n = both ? num_buckets / 2 : num_buckets;
    if (num_buckets < (both ? 4 : 2) || (both && num_buckets % 2 != 0) || n > ssd::kMaxBorders) return SSD_ERR_INVALID;
    const int e = n / 2, f = n - e;
    if (max_distance <= e) return SSD_ERR_INVALID;
    if (max_distance > ssd::kMaxDistance) return SSD_ERR_UNSUPPORTED;
    out.total = num_buckets;
    out.both = both;
    out.max_distance = max_distance;
    out.nborders = n - 1;
    int at = 0;
    for (int d = 1; d < e; ++d) out.borders[at++] = d;
    for (int k = 0; k < f; ++k) {
        // the smallest d with d >= e (m / e)^(k / f): from the power where it is clearly between two
        // whole numbers, by the exact comparison where it is next to one
        const double x = e * std::pow((double)max_distance / e, (double)k / f);
        int d = (int)std::ceil(x);
        const int near = (int)std::llround(x);
        if (std::fabs(x - near) < 1e-9 * x) d = reached(near, e, f, max_distance, k) ? near : near + 1;
        out.borders[at++] = d;
    }
    for (int d = 0, b = 0; d <= max_distance; ++d) {
        while (b < out.nborders && out.borders[b] <= d) ++b;
        out.of[d] = (uint8_t)b;
    }
    return SSD_OK;
}

inline int check_shape(int64_t H, int64_t Hk, int64_t D, int32_t dtype) {
    if (H < 1 || Hk < 1 || H > kMaxHeads || H % Hk != 0 || D < 1) return SSD_ERR_INVALID;
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_INVALID;
    if (D != 32 && D != 64 && D != 128) return SSD_ERR_UNSUPPORTED;
    if (H * D >= ((int64_t)1 << 24)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// The cap as the kernels take it, within [2^-56, 2^96], where their 1 / cap^2 and cap log2 e are finite.  Scores under a
// cap of 2^-56 are zero to the last bit of an fp32 weight, and 2^96 caps none that fp32 products of use reach.
inline float take_cap(float cap) {
    return cap > 0.f ? std::fmin(std::fmax(cap, 0x1p-56f), 0x1p96f) : 0.f;
}

inline int check_cache(const ssd_attn_cache* d) {
    if (!d) return SSD_ERR_INVALID;
    const int rc = check_shape(d->nheads, d->nkvheads, d->headdim, d->dtype);
    if (rc != SSD_OK) return rc;
    if (d->nseq < 0 || d->nseq > kMaxTokens || d->num_pages < 0 || d->num_pages >= ((int64_t)1 << 31) || d->page_size < 1 ||
        d->max_pages < 0 || d->max_pages > kMaxTokens)
        return SSD_ERR_INVALID;
    if (d->page_size % 16 != 0 || d->page_size > 65536 || d->max_pages * d->page_size > kMaxTokens) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Splits of a sequence's keys: enough workgroups for four on each of the 256 CUs, so that short and long
// sequences even out, of at least 128 keys (a block for each wave) at the longest length, and few
// enough that joining them stays small.  A short cache with a workgroup for every other CU or more is not
// split but gets eight waves a workgroup, which saves the join.  Split (with its join) against eight waves, us, 1000 keys, 32/8
// heads, 16 and 32 and 62 sequences (128, 256 and 496 workgroups):
//     bf16  32 wide 11.4/10.2  17.1/14.2  26.4/21.6      64 wide 14.6/11.8  18.9/14.6  28.5/23.5    128 wide 21.7/18.0  28.9/23.1  44.9/42.3
//     fp32  32 wide 15.4/14.1  20.6/16.6  31.8/25.6      64 wide 23.6/21.6  32.5/25.2  50.1/45.7    128 wide 39.1/46.6  64.9/55.8  139/126
// and more at 256 and 512 keys (6 to 40%).  In fp32 at 128 wide eight waves' tiles fill a CU's LDS: there below 256
// workgroups only up to 256 keys (15.4/15.3; 23.3/26.5 at 512).  One sequence: 10.8 split, 15.2 (bf16, 128 wide).
struct DecodeShape {
    int splits, wide;
};
constexpr int64_t kWideKeys = 1024, kWideKeysFullLds = 256;
inline DecodeShape split_shape(int64_t units, int64_t keys) {
    int64_t n = units > 0 ? (1024 + units - 1) / units : 1;
    const int64_t most = (keys + 127) / 128;
    if (n > most) n = most;
    if (n > 64) n = 64;
    return {n < 1 ? 1 : (int)n, 0};
}
inline int64_t decode_units(const ssd_attn_cache* d) { return d->nseq * d->nkvheads * ((d->nheads / d->nkvheads + 15) / 16); }
inline DecodeShape decode_shape(const ssd_attn_cache* d) {
    const int64_t units = decode_units(d), keys = d->max_pages * d->page_size;
    const bool full_lds = d->headdim * (d->dtype == SSD_BF16 ? 2 : 4) >= 512;
    if (keys <= (full_lds && units < 256 ? kWideKeysFullLds : kWideKeys) && units >= 128 && units < 512) return {1, 1};
    return split_shape(units, keys);
}

}  // namespace checks
}  // namespace ssd
