// tanh_poly.cuh -- tanh(y) = y q(y^2) for |y| <= 0.3: q of degree 2 interpolates tanh(y) / y at the three Chebyshev
// nodes of [0, 0.09] in y^2.  Error: below 4e-7, and below 1.2e-6 of the value (so scores far below a cap come out
// as they went in).  1 - 2 / (e^2y + 1) is as good relative to 1 only: it serves for larger |y|.
#pragma once

#define PA_TANH_RANGE 0.3f
#define PA_TANH_C0 0.99999883513f
#define PA_TANH_C1 -0.33309988804f
#define PA_TANH_C2 0.12633582392f
