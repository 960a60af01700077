// softcap.cuh -- the small-argument part of the soft cap's tanh, shared by the
// attention kernels.
#pragma once

namespace splash {

// |t| <= 0.25: tanh(t) = t (1 + u (c1 + c2 u)), u = t^2, with c1, c2 a minimax
// fit of tanh(t)/t on [0, 0.25] (Lawson-weighted least squares, q(0) = 1 held
// fixed), from the mathematics of tanh and not from any library; max relative
// error 4.8e-7, like the Maclaurin series to t^7 (3.3e-7) with one multiply-add
// less.  The error is relative to t: cap * tanh(s / cap) keeps the score's low
// bits however large the cap, where a form in e^(2t) has an absolute error
// that the cap multiplies.
constexpr float kTanhC1 = -0.33324610f;
constexpr float kTanhC2 = 0.12877172f;
constexpr float kTanhSeriesLimit = 0.25f;

}  // namespace splash
