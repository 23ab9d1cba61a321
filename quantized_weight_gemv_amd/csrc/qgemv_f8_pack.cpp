// Host quantizer / packer of the f8 weight layout of qgemv_f8.h.
//
// Runs once per weight matrix, off the timed path.  A block's scale comes
// from the exponent and the top of the significand of its largest magnitude,
// a code from rounding v / 2^e (exact in binary64) onto the e4m3 grid.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "qgemv_f8.h"

namespace {

constexpr int64_t kMaxK = 1 << 20;
constexpr int64_t kMaxRows = 1 << 30;

// The largest scale that a finite value needs, 2^120, and the largest code's
// value under it that fp32 still holds (the next, 256, would be 2^128).
constexpr int kMaxExponent = 120;
constexpr double kMaxOfLast = 240.0;

// The e4m3 code of v, |v| <= 448: the grid's step is 2^(x - 3) for 2^x <= |v|
// < 2^(x + 1) and 2^-9 below 2^-6.  nearbyint rounds ties to even (the
// default rounding mode), and a value that rounds up to the next power of two
// is on that binade's grid as well.
uint8_t e4m3_code(double v)
{
    const uint8_t sign = std::signbit(v) ? 0x80 : 0;
    if (!std::isfinite(v))
        return sign | 0x7f;
    double m = std::fabs(v);
    int x = -6;
    if (m >= 0x1p-6)
        x = std::ilogb(m);
    const double q = std::nearbyint(std::ldexp(m, 3 - x));   // 0..16 steps of 2^(x - 3)
    const int steps = static_cast<int>(q);
    if (steps < 8)
        return sign | static_cast<uint8_t>(steps);                         // zero or subnormal (x = -6)
    // normal: 8 + mantissa steps at exponent x; 16 steps are 8 at x + 1
    return sign | static_cast<uint8_t>(((x + 7) << 3) + (steps - 8));
}

}  // namespace

extern "C" {

size_t qpacked_bytes_f8(int64_t N, int64_t K)
{
    if (N < 1 || K < 1 || N > kMaxRows || K > kMaxK)
        return 0;
    const size_t cb = (K + 127) / 128, rt = (N + 15) / 16, rb = (N + 127) / 128;
    return (rt * cb * 2048 + rb * ((cb + 3) / 4 * 4) + 255) / 256 * 256;
}

size_t qact_bytes_f8(int64_t M, int64_t K)
{
    if (M < 1 || K < 1 || M > kMaxRows || K > kMaxK)
        return 0;
    const size_t cb = (K + 127) / 128, m = M;
    return ((m * cb * 128 + 255) / 256 * 256 + m * ((cb + 3) / 4 * 4) + 255) / 256 * 256;
}

qg_status qquantize_f8(const float *w, int64_t N, int64_t K, void *packed, size_t packed_bytes)
{
    if (!w || !packed)
        return QG_ERR_NULL;
    const size_t need = qpacked_bytes_f8(N, K);
    if (need == 0)
        return QG_ERR_SHAPE;
    if (packed_bytes < need)
        return QG_ERR_SIZE;
    auto *out = static_cast<uint8_t *>(packed);
    std::memset(out, 0, need);
    const int64_t cb = (K + 127) / 128, rt = (N + 15) / 16, ls = (cb + 3) / 4 * 4;
    uint8_t *scales = out + rt * cb * 2048;
    qg_status st = QG_OK;
    for (int64_t b = 0; b * 128 < N; ++b) {
        const int64_t n1 = N < (b + 1) * 128 ? N : (b + 1) * 128;
        for (int64_t c = 0; c < cb; ++c) {
            const int64_t k1 = K < (c + 1) * 128 ? K : (c + 1) * 128;
            float amax = 0.0f;
            for (int64_t n = b * 128; n < n1; ++n)
                for (int64_t k = c * 128; k < k1; ++k) {
                    const float a = std::fabs(w[n * K + k]);
                    if (!std::isfinite(a))
                        st = QG_ERR_RANGE;
                    else if (a > amax)
                        amax = a;
                }
            int e = 0;
            if (amax > 0.0f) {
                const float f = std::frexp(amax, &e);    // amax = f 2^e, 0.5 <= f < 1; 448 = 0.875 * 2^9
                e += f > 0.875f ? -8 : -9;
                e = e < -127 ? -127 : e;
            }
            scales[b * ls + c] = static_cast<uint8_t>(e + 127);
            for (int64_t n = b * 128; n < n1; ++n) {
                uint8_t *row = out + ((n / 16) * cb + c) * 2048 + 16 * (n % 16);
                for (int64_t k = c * 128; k < k1; ++k) {
                    double v = std::ldexp(static_cast<double>(w[n * K + k]), -e);
                    if (e == kMaxExponent && std::isfinite(v))
                        v = std::fmin(std::fmax(v, -kMaxOfLast), kMaxOfLast);
                    row[256 * (k % 128 / 16) + k % 16] = e4m3_code(v);
                }
            }
        }
    }
    return st;
}

}  // extern "C"
