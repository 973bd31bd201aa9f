// Test helper, not part of the library: the rotation's angles (ra_rotary.cuh) on the host.
#include "ra_rotary.cuh"

extern "C" void ra_test_half_turns(const float *f, const int *p, float *out, int n) {
    for (int i = 0; i < n; ++i) out[i] = ra::half_turns(p[i], ra::turn_fraction(f[i]));
}
