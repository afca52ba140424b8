/* Exhaustive check of the token quantizer's division-free codes:
 * with s = fl32(a / 127) for a row maximum a (bf16) and y = fl32(1 / s),
 *   q0 = fl32(x y), r = fma(-q0, s, x), q1 = fma(r, y, q0)
 * must satisfy rint(q1) = rint(fl32(x / s)) for every bf16 x, |x| <= a.
 * Scaling a and x by a power of two changes nothing while s >= 2^-96, so all
 * mantissas of a at a few exponents and all x down to a 2^-11 are enough; below
 * that |q1| < 1/8 rounds to 0 on both sides. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

static float bf16(uint32_t h) {
    uint32_t u = h << 16;
    float f;
    memcpy(&f, &u, 4);
    return f;
}

int main(void) {
    long pairs = 0, bad = 0;
    /* exponents: the bottom and top of the fast range, and a spread between */
    const int exps[] = {39, 40, 41, 60, 100, 126, 127, 128, 150, 200, 240, 252, 253, 254};
    for (unsigned e = 0; e < sizeof exps / sizeof *exps; ++e)
        for (uint32_t m = 0; m < 128; ++m) {
            const uint32_t ah = ((uint32_t)exps[e] << 7) | m;
            const float a = bf16(ah);
            volatile float sv = a / 127.0f;
            const float s = sv;
            if (s < 0x1p-96f) continue;
            volatile float yv = 1.0f / s;
            const float y = yv;
            for (uint32_t xh = ah - (11u << 7); xh <= ah; ++xh) {
                const float x = bf16(xh);
                volatile float q0 = x * y;
                const float r = fmaf(-q0, s, x), q1 = fmaf(r, y, q0);
                volatile float q = x / s;
                ++pairs;
                /* round half to even is the default rounding mode of rintf */
                if (rintf(q1) != rintf(q) || fabsf(q1) > 127.5f) {
                    if (bad++ < 5) printf("a %a x %a: %a against %a\n", a, x, q1, q);
                }
            }
        }
    printf("%ld pairs, %ld wrong\n", pairs, bad);
    return bad != 0 || pairs < 1000000;
}
