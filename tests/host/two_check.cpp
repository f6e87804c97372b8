// Host check of the two-word exp and ln of the stored-row consumers: the header is compiled as host code, with host forms of
// the device functions it uses, and compared with long double. Prints the largest errors.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include <cuda_runtime.h>

static inline float __int_as_float(int i) { float f; std::memcpy(&f, &i, 4); return f; }
static inline int __float_as_int(float f) { int i; std::memcpy(&i, &f, 4); return i; }
template <class T> static inline T __ldg(const T* p) { return *p; }
template <class T> static inline T __shfl_xor_sync(unsigned, T v, int) { return v; }

#include "tp_logits_two.cuh"

using tp::rows::Two;

static long double value(const Two& t) { return (long double)t.h + t.l; }

int main() {
    double exp_normal = 0, exp_low = 0, ln_err = 0, exp_words = 0;
    uint64_t s = 12345;
    const auto uniform = [&] {  // in [0, 1)
        s = s * 6364136223846793005ull + 1442695040888963407ull;
        return (double)(s >> 11) / 9007199254740992.0;
    };
    for (int i = 0; i < 4000000; ++i) {
        // the whole range, and near 0; with and without a second word
        const float h = (float)(i & 1 ? -87 + 175 * uniform() : (uniform() - 0.5) * 0.1);
        const Two x = {h, i & 2 ? (float)((uniform() - 0.5) * std::ldexp(std::fabs(h), -24)) : 0.f};
        const Two e = tp::rows::exp_two(x);
        const double r = (double)std::fabs(value(e) / std::exp(value(x)) - 1);
        if (h >= -70) exp_normal = std::fmax(exp_normal, r);
        else if (h >= -87) exp_low = std::fmax(exp_low, r);
        exp_words = std::fmax(exp_words, std::fabs((double)e.l) / e.h);

        const float z = (float)std::exp((i & 1 ? -85 + 170 * uniform() : (uniform() - 0.5) * 0.2));
        const Two w = {z, i & 2 ? (float)((uniform() - 0.5) * std::ldexp(z, -24)) : 0.f};
        const Two l = tp::rows::ln_two(w);
        ln_err = std::fmax(ln_err, (double)std::fabs(value(l) - std::log(value(w))));
    }
    const float inf = INFINITY;
    const auto is = [](const Two& t, float h) { return t.l == 0.f && (t.h == h || (h != h && t.h != t.h)); };
    const bool edges = is(tp::rows::exp_two(Two{-inf, 0}), 0) && is(tp::rows::exp_two(Two{-3.4e38f, 0}), 0) && is(tp::rows::exp_two(Two{-88, 0}), 0) &&
                       is(tp::rows::exp_two(Two{89, 0}), inf) && is(tp::rows::exp_two(Two{inf, 0}), inf) && is(tp::rows::exp_two(Two{NAN, 0}), NAN) &&
                       is(tp::rows::exp_two(Two{0, 0}), 1) && is(tp::rows::ln_two(Two{inf, 0}), inf) && is(tp::rows::ln_two(Two{NAN, 0}), NAN);
    std::printf("%.3e %.3e %.3e %.3e %d\n", exp_normal, exp_low, ln_err, exp_words, edges);
    return 0;
}
