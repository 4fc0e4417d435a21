// Arithmetic of the gated scan (wtconv_scan.h).
#pragma once

#include "scan.h"
#include "train_device.cuh"

namespace wtconv {

// a = sigmoid(z) and b = 1 - a, both to a few units of their own last place: with e = exp(-z),
// a = 1 / (1 + e) and b = e a, or 1 - a where e > 1 (a < 1/2 there, so nothing cancels, and an e
// that overflowed gives a = 0, b = 1).  A NaN comes through.
struct Gate {
    float a, b;
};
__device__ __forceinline__ Gate gate_of(float z) {
    const float e = __expf(-z);
    Gate g;
    g.a = __frcp_rn(1.f + e);
    g.b = e > 1.f ? 1.f - g.a : e * g.a;
    return g;
}

// length of sequence b, clipped to [0, T]
__device__ __forceinline__ int scan_length(const int *lengths, int b, int T) {
    if (lengths == nullptr) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n < T ? n : T);
}

}  // namespace wtconv
