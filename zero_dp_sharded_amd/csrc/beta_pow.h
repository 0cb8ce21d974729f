// Adam's bias-correction power, shared by the shard's step and the operators' AdamW.
#pragma once

#include <stdint.h>

// beta^t as a product of t copies of (double)(float)beta, one after the other, as a
// step multiplies the power it keeps: the same bits.  Ends where a multiplication no longer
// changes the product, which is then what it stays (0, or for a beta above 1/2 a smallest
// number that rounds back to itself), so a counter of any size costs at most the
// 745 / (1 - beta) steps that the product takes down to there.
inline double beta_pow(double beta, int64_t t)
{
    const double b = (double)(float)beta;
    double p = 1.0;
    for (int64_t k = 0; k < t; ++k) {
        const double next = p * b;
        if (next == p) break;
        p = next;
    }
    return p;
}
