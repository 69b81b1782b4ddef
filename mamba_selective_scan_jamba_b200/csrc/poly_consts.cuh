// Generated by gen_poly.py: minimax polynomials (Remez exchange) in float32.
#pragma once

namespace jmix {
namespace poly {

// 2^f ~ E0 + f*(E1 + f*(E2 + ...)) for f in [-1/2, 1/2]
constexpr float E0 = 1.000000000e+00f;
constexpr float E1 = 6.931471825e-01f;
constexpr float E2 = 2.402264625e-01f;
constexpr float E3 = 5.550328642e-02f;
constexpr float E4 = 9.618489072e-03f;
constexpr float E5 = 1.339993090e-03f;
constexpr float E6 = 1.534581243e-04f;

// log1p(w) ~ w*(L0 + w*(L1 + ...)) for w in [0, 1]
constexpr float L0 = 9.999999404e-01f;
constexpr float L1 = -4.999949336e-01f;
constexpr float L2 = 3.331909776e-01f;
constexpr float L3 = -2.484298199e-01f;
constexpr float L4 = 1.910600662e-01f;
constexpr float L5 = -1.366324574e-01f;
constexpr float L6 = 7.822595537e-02f;
constexpr float L7 = -2.950523980e-02f;
constexpr float L8 = 5.232694093e-03f;

// Phi(-a) exp(a^2 / 2) ~ t*(N0 + t*(N1 + ...)), t = 1 / (1 + NC a), for a in [0, 14]
constexpr float NC = 3.000000000e-01f;
constexpr float N0 = 1.196293011e-01f;
constexpr float N1 = 1.207539588e-01f;
constexpr float N2 = 9.991349280e-02f;
constexpr float N3 = 1.285616159e-01f;
constexpr float N4 = -5.368361995e-02f;
constexpr float N5 = 2.063534856e-01f;
constexpr float N6 = -1.572030634e-01f;
constexpr float N7 = 3.567476943e-02f;

// 1/x initial guess: as_float(RCP_MAGIC - bits(x)), then Newton-Raphson
constexpr int RCP_MAGIC = 0x7ef311c2;

}  // namespace poly
}  // namespace jmix
