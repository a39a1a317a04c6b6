// rope_table.cu -- host: the frequencies of wsw_rope_kv_write in fractions of a turn.
//
// The kernel's angle is position * turns modulo 2^64, exact, so that the table alone says how good
// a far position's angle is.  In doubles a frequency is off by f 2^-53 or more, 3e-7 radians at
// position 2^31 and more than fp32's own step of the angle; so it is made from pairs of doubles (about 100 bits,
// the sums and products of Dekker, "A floating-point technique for extending the available
// precision", 1971, with a fused multiply-add for the product's error) and rounded once.  theta^(-i/n)
// is a power of the n-th root of theta, which takes two Newton steps from the double one.  Every
// operation is an IEEE one written out (no a * b + c that a compiler may or may not fuse): all hosts give the same table.
#include <cmath>
#include <cstdint>

#include "wsw.h"

namespace wsw {
namespace {

struct Pair {
    double hi, lo;  // |lo| <= half a step of hi
};

// hi + lo for |lo| not above |hi|
Pair quick(double hi, double lo) {
    const double s = hi + lo;
    return Pair{s, lo - (s - hi)};
}
Pair sum(double a, double b) {
    const double s = a + b, t = s - a;
    return Pair{s, (a - (s - t)) + (b - t)};
}
Pair add(Pair a, Pair b) {
    const Pair s = sum(a.hi, b.hi), t = sum(a.lo, b.lo);
    const Pair u = quick(s.hi, s.lo + t.hi);
    return quick(u.hi, u.lo + t.lo);
}
Pair neg(Pair a) { return Pair{-a.hi, -a.lo}; }
Pair mul(Pair a, Pair b) {
    const double p = a.hi * b.hi;
    double e = std::fma(a.hi, b.hi, -p);
    e = std::fma(a.hi, b.lo, e);
    e = std::fma(a.lo, b.hi, e);
    return quick(p, e);
}
Pair div(Pair a, Pair b) {
    const double q0 = a.hi / b.hi;
    Pair r = add(a, neg(mul(b, Pair{q0, 0})));
    const double q1 = r.hi / b.hi;
    r = add(r, neg(mul(b, Pair{q1, 0})));
    return add(quick(q0, q1), Pair{r.hi / b.hi, 0});
}
Pair power(Pair x, int64_t n) {
    Pair y{1, 0};
    for (; n > 0; n >>= 1) {
        if (n & 1) y = mul(y, x);
        if (n > 1) x = mul(x, x);
    }
    return y;
}
// x^(1 / n), x > 0
Pair root(double x, int64_t n) {
    Pair h{std::pow(x, 1.0 / static_cast<double>(n)), 0};
    for (int step = 0; step < 2; ++step) {  // h + (x / h^(n - 1) - h) / n
        const Pair d = add(div(Pair{x, 0}, power(h, n - 1)), neg(h));
        h = add(h, div(d, Pair{static_cast<double>(n), 0}));
    }
    return h;
}

constexpr Pair kTwoPi{6.283185307179586232, 2.4492935982947064e-16};

// radians per position (in [0, 2 pi)) as a whole number of 2^-64 turns
uint64_t turns_of(Pair f) {
    const Pair x = div(f, kTwoPi);
    const double hi = std::ldexp(x.hi, 64), lo = std::ldexp(x.lo, 64);
    const double whole = std::nearbyint(hi);  // hi itself from 2^53 on
    const int64_t rest = static_cast<int64_t>(std::nearbyint((hi - whole) + lo));
    // a whole turn is none
    return (whole < 18446744073709551616.0 ? static_cast<uint64_t>(whole) : 0) + static_cast<uint64_t>(rest);
}

}  // namespace
}  // namespace wsw

extern "C" int wsw_rope_table(int64_t rot_dim, double theta, int32_t scaling, double factor, int64_t original,
                              const double *freqs, uint64_t *turns, float *mscale) {
    using namespace wsw;
    if (!turns || !mscale || rot_dim < 2 || rot_dim > 256 || (rot_dim & 1)) return WSW_ERR_INVALID_ARG;
    const int64_t n = rot_dim / 2;
    if (freqs) {
        for (int64_t i = 0; i < n; ++i) {
            if (!(freqs[i] >= 0 && freqs[i] < kTwoPi.hi)) return WSW_ERR_INVALID_ARG;
            turns[i] = turns_of(Pair{freqs[i], 0});
        }
        *mscale = 1.0f;
        return WSW_OK;
    }
    if (scaling < WSW_ROPE_PLAIN || scaling > WSW_ROPE_BY_PARTS || !std::isfinite(theta) || !(theta > 1))
        return WSW_ERR_INVALID_ARG;
    if (scaling != WSW_ROPE_PLAIN && (!std::isfinite(factor) || !(factor >= 1))) return WSW_ERR_INVALID_ARG;
    if (scaling == WSW_ROPE_NTK && rot_dim <= 2) return WSW_ERR_INVALID_ARG;
    if (scaling == WSW_ROPE_BY_PARTS && original < 1) return WSW_ERR_INVALID_ARG;
    const Pair one{1, 0}, by{factor, 0};
    Pair base = root(theta, n);  // pair i turns by base^-i
    // (theta factor^(2 n / (2 n - 2)))^(-i / n) = theta^(-i / n) factor^(-i / (n - 1))
    if (scaling == WSW_ROPE_NTK) base = mul(base, root(factor, n - 1));
    for (int64_t i = 0; i < n; ++i) {
        const Pair p = power(base, i);
        Pair f = p.hi < 1e300 ? div(one, p) : Pair{0, 0};  // beyond: far below 2^-64 turns
        if (scaling == WSW_ROPE_LINEAR) f = div(f, by);
        if (scaling == WSW_ROPE_BY_PARTS) {  // turns over `original` positions: 1 .. 32
            const Pair turned = div(mul(Pair{static_cast<double>(original), 0}, f), kTwoPi);
            Pair keep = div(add(turned, neg(one)), Pair{31, 0});
            if (keep.hi < 0) keep = Pair{0, 0};
            if (keep.hi >= 1) keep = one;
            f = add(mul(keep, f), mul(add(one, neg(keep)), div(f, by)));
        }
        turns[i] = turns_of(f);
    }
    *mscale = scaling == WSW_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
    return WSW_OK;
}
