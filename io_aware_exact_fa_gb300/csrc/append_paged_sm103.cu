// Norm, position rotation and append to a paged K/V cache for sm_103a.
//
// New token i of sequence b (n_b new tokens, length L_b with them) is at
// position p = L_b - n_b + i. For every head of q and k:
//     x' = x / sqrt(mean(x^2) + eps) * w                          (where weights are given)
//     (a, b) -> (a cos - b sin, b cos + a sin),  angle 2 pi frac(p t_j / 2^64)
// on the pairs j of its first `rot` elements: (j, j + rot / 2), or (2j, 2j + 1)
// interleaved. q' and k' are written out in bf16; k' and v go to the row of
// position p in the cache, in bf16, as e4m3 or as 4-bit codes.
//
// The frequency t_j is a fraction of a turn in 64-bit fixed point, so p t_j mod
// 2^64 is the exact angle, in turns, for any position: one integer product in
// place of a range reduction, with nothing lost at far positions and no table of
// angles to read.
//
// e4m3 pages have one scale for each K/V head, a power of two: the least 2^e with
// amax <= 448 2^e over the rows the page holds. The codes are floating point, so
// a finer scale would not make them more exact, and when a later token makes the
// scale grow, dividing the codes already held by a power of two rounds again
// only where they fall below the smallest normal code. The values are rounded
// once, from the fp32 result, not through bf16.
//
// 4-bit pages hold e2m1 codes and, for every 16 neighbours of a row, one byte of scale:
// amax / 6, rounded to three mantissa bits. Rows do not depend on one another there, so a
// K/V block takes several heads of a page and works a row's angles out once for them; the
// keys are rounded from the bf16 value that k_out gets, so the cache and a prompt's own
// attention see the same keys. A code is a step function of the key: two computations that
// round apart in the last bit of fp32 hold, now and then, values half a scale apart. So the
// way from the input to the bf16 key is fixed, operation by operation, each rounded to
// nearest in fp32 (the order of a norm's sum, no fused products, cosines and sines to
// within 2^-30 of the rounded value), and whoever computes the same steps gets the same codes.
//
// Two kinds of blocks in one launch. A K/V block takes the new rows of one page of
// one sequence and one K/V head: those rows are all that the page's scales depend
// on, so no sum or maximum goes through global atomics; it turns the keys, keeps
// them in fp32 in shared memory until the page's largest value is known, and
// writes the codes. A query block takes rows of the step and streams their query
// heads through rings of asynchronous copies, each one thread's own, so loads stay
// in flight without registers; a row's angles (with the norm's weights multiplied
// in) are computed once for all its heads.
// What bounds it: HBM for prompts (q read and written, k and v read, the cache
// written) as long as the instructions per value stay few (packed fp32
// arithmetic; with one kind of block for both 147 us in place of 132), launch and
// load latency for a step of single tokens. Measured, 32 query and 8 K/V heads,
// d = 128, e4m3: 26.7k prompt tokens with norms 115 us (5.7 TB/s, 0.85 of the copy
// rate); 256 sequences of one token 8.1 us; 4-bit: 26k prompt tokens 112 us (132 with a K/V
// block for each head, like e4m3; 106 with fused products and less exact angles).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <climits>

#include "fp4.cuh"
#include "mma_sync.cuh"
#include "paged.cuh"

namespace fa {

namespace {

constexpr int AP_THREADS = 256;        // of a block, at most
constexpr int AP_STEP_THREADS = 64;    // and at least
// Blocks of AP_THREADS that an SM should hold: four where 64 registers do without spilling (interleaved, bf16 cache:
// 32 against 34 us for 9.1k tokens of 28 heads), else three (half layout: 111 against 121 us for 26.7k prompt tokens).
constexpr int ap_ctas(int kind, bool inter) { return kind == PAGES_BF16 && inter ? 4 : 3; }
#ifndef AP_RING
#define AP_RING 3       // heads of a row whose copies a query thread has in flight
#endif
#ifndef AP_KV_RING
#define AP_KV_RING 2    // the same of a K/V block of 4-bit rows
#endif
#ifndef AP_KV_HEADS
#define AP_KV_HEADS 4   // K/V heads of such a block, at most
#endif

// A unit's 16 elements as four fp32 pairs a (first of each rotation pair) and four
// pairs b (second): elements c0 .. c0 + 7 and c1 .. c1 + 7 are a and b, or, in
// the interleaved layout, alternate. Packed fp32x2 arithmetic halves the
// instructions of the norm and the rotation.
struct Unit16 {
  uint64_t a[4], b[4];
};
template <bool INTER>
__device__ __forceinline__ Unit16 unpack16(const uint4& u0, const uint4& u1) {
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  Unit16 x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTER) {
      x.a[i] = f2pack(__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i + 1] << 16));
      x.b[i] = f2pack(__uint_as_float(w[2 * i] & 0xffff0000u), __uint_as_float(w[2 * i + 1] & 0xffff0000u));
    } else {
      x.a[i] = f2pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      x.b[i] = f2pack(__uint_as_float(w[4 + i] << 16), __uint_as_float(w[4 + i] & 0xffff0000u));
    }
  }
  return x;
}
// The 16 elements in memory order: y[0..7] at c0, y[8..15] at c1.
template <bool INTER>
__device__ __forceinline__ void in_order(const Unit16& x, float* y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0, a1, b0, b1;
    f2unpack(x.a[i], a0, a1);
    f2unpack(x.b[i], b0, b1);
    if constexpr (INTER) {
      y[4 * i] = a0, y[4 * i + 1] = b0, y[4 * i + 2] = a1, y[4 * i + 3] = b1;
    } else {
      y[2 * i] = a0, y[2 * i + 1] = a1, y[8 + 2 * i] = b0, y[9 + 2 * i] = b1;
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// sin and cos of 2 pi f for two fractions of a turn f = t / 2^32: the nearest
// quarter turn is taken off in integers (exactly), and the Taylor series on
// [-pi/4, pi/4], to x^9 and x^10, are off by less than 2e-9. Dropping the
// fraction's bits past the 32nd moves the angle by less than 2e-9 as well; fp32
// rounds by 6e-8.
__device__ __forceinline__ uint64_t dup2(float x) { return f2pack(x, x); }
// Sine and cosine q quarter turns on.
__device__ __forceinline__ void place_quarter(int q, float sn, float cn, float& so, float& co) {
  const float a = (q & 1) ? cn : sn, b = (q & 1) ? sn : cn;
  so = __uint_as_float(__float_as_uint(a) ^ ((static_cast<uint32_t>(q) & 2u) << 30));
  co = __uint_as_float(__float_as_uint(b) ^ ((static_cast<uint32_t>(q + 1) & 2u) << 30));
}
__device__ __forceinline__ void sincos_turns2(int t0, int t1, float scale, uint64_t& s2, uint64_t& c2) {
  const int q0 = static_cast<int>(static_cast<uint32_t>(t0) + 0x20000000u) >> 30;
  const int q1 = static_cast<int>(static_cast<uint32_t>(t1) + 0x20000000u) >> 30;
  const float r0 = static_cast<float>(static_cast<int>(static_cast<uint32_t>(t0) - (static_cast<uint32_t>(q0) << 30)));
  const float r1 = static_cast<float>(static_cast<int>(static_cast<uint32_t>(t1) - (static_cast<uint32_t>(q1) << 30)));
  const uint64_t x = fmul2(f2pack(r0, r1), dup2(1.4629180792671596e-9f));  // 2 pi / 2^32
  const uint64_t z = fmul2(x, x);
  uint64_t ps = ffma2(z, dup2(2.7557319e-6f), dup2(-1.9841270e-4f));
  ps = ffma2(z, ps, dup2(8.3333333e-3f));
  ps = ffma2(z, ps, dup2(-1.6666667e-1f));
  const uint64_t sx = ffma2(fmul2(x, z), ps, x);
  uint64_t pc = ffma2(z, dup2(-2.7557319e-7f), dup2(2.4801587e-5f));
  pc = ffma2(z, pc, dup2(-1.3888889e-3f));
  pc = ffma2(z, pc, dup2(4.1666667e-2f));
  pc = ffma2(z, pc, dup2(-0.5f));
  const uint64_t sc = dup2(scale);
  float s0, s1, c0, c1;
  f2unpack(fmul2(sx, sc), s0, s1);
  f2unpack(fmul2(ffma2(z, pc, dup2(1.f)), sc), c0, c1);
  float so0, so1, co0, co1;
  place_quarter(q0, s0, c0, so0, co0);
  place_quarter(q1, s1, c1, so1, co1);
  s2 = f2pack(so0, so1);
  c2 = f2pack(co0, co1);
}

// Largest magnitude among 16 values, infinities and NaN left out (they are stored as the NaN code).
__device__ __forceinline__ float finite_amax(const float* x) {
  float m = fmaxf(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
  for (int i = 2; i < 16; i += 2) m = fmax3(m, fabsf(x[i]), fabsf(x[i + 1]));  // (a NaN loses against a number)
  if (!(m <= FLT_MAX)) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m = fabsf(x[i]) <= FLT_MAX ? fmaxf(m, fabsf(x[i])) : m;
  }
  return m;
}
// The same for 16 bf16 values.
__device__ __forceinline__ float finite_amax(const uint4& u0, const uint4& u1) {
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
  __nv_bfloat162 m2 = __habs2(h[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m2 = __hmax2(m2, __habs2(h[i]));
  float m = fmaxf(__low2float(m2), __high2float(m2));
  if (!(m <= FLT_MAX)) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = fabsf(__low2float(h[i])), b = fabsf(__high2float(h[i]));
      m = a <= FLT_MAX ? fmaxf(m, a) : m;
      m = b <= FLT_MAX ? fmaxf(m, b) : m;
    }
  }
  return m;
}

// Least 2^e, e >= -40, with amax <= 448 * 2^e (448 = 1.75 * 2^8).
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, PAGED_SCALE_EXP_MIN);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The scale of a page whose new rows reach amax: that of the rows it already holds where it suffices and is one that
// append may have written (the reciprocal of a subnormal one would overflow).
__device__ __forceinline__ float merged_scale(float amax, float old, bool holds) {
  constexpr float LEAST = 1.f / static_cast<float>(1ll << -PAGED_SCALE_EXP_MIN);
  if (holds && old >= LEAST && old <= FLT_MAX && amax <= 448.f * old) return old;
  return scale_for(amax);
}

// Four values to four e4m3 codes (nearest even); infinities and NaN give the NaN
// code: y + 0 * y is y, or NaN where y is not finite.
__device__ __forceinline__ uint32_t to_codes4(float x0, float x1, float x2, float x3, float inv) {
  const uint64_t i2 = f2pack(inv, inv), z2 = 0ull;
  const uint64_t a = fmul2(f2pack(x0, x1), i2), b = fmul2(f2pack(x2, x3), i2);
  float y0, y1, y2, y3;
  f2unpack(ffma2(a, z2, a), y0, y1);
  f2unpack(ffma2(b, z2, b), y2, y3);
  return pack_e4m3x4(y0, y1, y2, y3);
}

// The unit u of a row: 8 pairs, or 16 elements that are not turned, at c0 .. c0 + 7 and c1 .. c1 + 7.
template <bool INTER>
struct UnitPlace {
  bool turned;
  int c0, c1;
  __device__ __forceinline__ UnitPlace(int u, int rot) {
    turned = u < rot / 16;
    c0 = INTER ? 16 * u : (turned ? 8 * u : rot + 16 * (u - rot / 16));
    c1 = INTER || !turned ? c0 + 8 : rot / 2 + 8 * u;
  }
};

// Cosines and sines of a unit's pairs at one position.
struct Angles {
  uint64_t c[4], s[4];
};
__device__ __forceinline__ void angles_at(Angles& f, uint32_t pos, const long long* turns8, float rot_scale) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const ulonglong2 t2 = __ldg(reinterpret_cast<const ulonglong2*>(turns8) + j);
    // p t mod 2^64, its upper half: the fraction of a turn in 2^-32
    sincos_turns2(static_cast<int>((pos * t2.x) >> 32), static_cast<int>((pos * t2.y) >> 32), rot_scale, f.s[j], f.c[j]);
  }
}
constexpr uint64_t NEG2 = 0x8000000080000000ull;  // flips both signs of a pair

// Cosine and sine of 2 pi f for two fractions of a turn f = t / 2^64, rounded to fp32 (off from the exact values by less than
// 2^-30 of them before that rounding). With x = xh + xl the angle that is left of the nearest quarter turn, in two parts:
//     sin x = xh - xh^3 / 6 + (xl + x^5 / 120 - ..),   cos x = 1 - xh^2 / 2 + (- xh xl + x^4 / 24 - ..)
// where the first two terms and their errors are kept apart and the rest, below 2^-5 of the result, is in fp32.
__device__ __forceinline__ void sincos_turns2_rounded(uint64_t t0, uint64_t t1, float scale, uint64_t& s2, uint64_t& c2) {
  auto angle = [](uint64_t t, int& q, float& a, float& b) {  // t = q 2^62 + (a + b) 2^32
    q = static_cast<int>((t + 0x2000000000000000ull) >> 62);
    const int64_t r = static_cast<int64_t>(t - (static_cast<uint64_t>(q) << 62));
    const int h = static_cast<int>(r >> 32);
    a = static_cast<float>(h);
    b = fmaf(static_cast<float>(static_cast<uint32_t>(r)), 2.3283064365386963e-10f, static_cast<float>(h - static_cast<int>(a)));
  };
  int q0, q1;
  float a0, a1, b0, b1;
  angle(t0, q0, a0, b0);
  angle(t1, q1, a1, b1);
  constexpr double UNIT = 6.283185307179586476925 / 4294967296.0;  // 2 pi / 2^32
  constexpr float UH = static_cast<float>(UNIT), UL = static_cast<float>(UNIT - static_cast<double>(UH));
  constexpr float SIXTH = 1.f / 6.f, SIXTH_L = static_cast<float>(1.0 / 6.0 - static_cast<double>(SIXTH));
  const uint64_t a = f2pack(a0, a1), b = f2pack(b0, b1);
  const uint64_t xh = fmul2(a, dup2(UH));
  const uint64_t xl = ffma2(b, dup2(UH), ffma2(a, dup2(UL), ffma2(a, dup2(UH), xh ^ NEG2)));
  const uint64_t zh = fmul2(xh, xh), zl = ffma2(xh, xh, zh ^ NEG2);           // xh^2
  const uint64_t wh = fmul2(xh, zh), wl = ffma2(xh, zl, ffma2(xh, zh, wh ^ NEG2));  // xh^3
  const uint64_t th = fmul2(wh, dup2(-SIXTH));
  const uint64_t tl = ffma2(wl, dup2(-SIXTH), ffma2(wh, dup2(-SIXTH_L), ffma2(wh, dup2(-SIXTH), th ^ NEG2)));
  uint64_t ps = ffma2(zh, dup2(-2.5052108e-8f), dup2(2.7557319e-6f));         // 1/11!, 1/9!
  ps = ffma2(zh, ps, dup2(-1.9841270e-4f));
  ps = ffma2(zh, ps, dup2(8.3333333e-3f));
  const uint64_t half_z = fmul2(zh, dup2(0.5f));
  const uint64_t turn_xl = ffma2(xl, half_z ^ NEG2, xl);                      // xl cos x
  const uint64_t rs = fadd2(tl, ffma2(fmul2(wh, zh), ps, turn_xl));
  const uint64_t s1 = fadd2(xh, th), es = fadd2(th, fadd2(s1, xh ^ NEG2) ^ NEG2);
  const uint64_t sn = fadd2(s1, fadd2(es, rs));
  uint64_t pc = ffma2(zh, dup2(-2.7557319e-7f), dup2(2.4801587e-5f));         // 1/10!, 1/8!
  pc = ffma2(zh, pc, dup2(-1.3888889e-3f));
  pc = ffma2(zh, pc, dup2(4.1666667e-2f));
  const uint64_t one = dup2(1.f);
  const uint64_t c1 = fadd2(one, half_z ^ NEG2), ec = fadd2(fadd2(one, c1 ^ NEG2), half_z ^ NEG2);
  const uint64_t rc = ffma2(fmul2(zh, zh), pc, ffma2(zl, dup2(-0.5f), fmul2(xh, xl) ^ NEG2));
  const uint64_t cn = fadd2(c1, fadd2(ec, rc));
  const uint64_t sc = dup2(scale);
  float sa, sb, ca, cb, so0, so1, co0, co1;
  f2unpack(fmul2(sn, sc), sa, sb);
  f2unpack(fmul2(cn, sc), ca, cb);
  place_quarter(q0, sa, ca, so0, co0);
  place_quarter(q1, sb, cb, so1, co1);
  s2 = f2pack(so0, so1);
  c2 = f2pack(co0, co1);
}
__device__ __forceinline__ void angles_rounded_at(Angles& f, uint32_t pos, const long long* turns8, float rot_scale) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const ulonglong2 t2 = __ldg(reinterpret_cast<const ulonglong2*>(turns8) + j);
    sincos_turns2_rounded(pos * t2.x, pos * t2.y, rot_scale, f.s[j], f.c[j]);
  }
}

// The same with a norm's weights multiplied in, for rows with many heads:
// a' = a e0 + b e1, b' = b e2 + a e3 (e1, e3 only where the unit is turned).
struct Factors {
  uint64_t e0[4], e1[4], e2[4], e3[4];
};
template <bool INTER>
__device__ __forceinline__ void factors_at(Factors& f, bool turned, uint32_t pos, const long long* turns8, float rot_scale,
                                           const uint16_t* wt, int c0, int c1) {
  Angles t;
  if (turned) {
    angles_at(t, pos, turns8, rot_scale);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) t.c[j] = f2pack(1.f, 1.f), t.s[j] = 0ull;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.e0[j] = f.e2[j] = t.c[j];
    f.e3[j] = t.s[j];
    f.e1[j] = t.s[j] ^ NEG2;
  }
  if (wt != nullptr) {
    const Unit16 w = unpack16<INTER>(__ldg(reinterpret_cast<const uint4*>(wt + c0)), __ldg(reinterpret_cast<const uint4*>(wt + c1)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.e0[i] = fmul2(f.e0[i], w.a[i]);
      f.e1[i] = fmul2(f.e1[i], w.b[i]);
      f.e2[i] = fmul2(f.e2[i], w.b[i]);
      f.e3[i] = fmul2(f.e3[i], w.a[i]);
    }
  }
}
// x / sqrt(mean(x^2) + eps) over the LPR lanes of a row; every lane of the warp takes part.
template <int D>
__device__ __forceinline__ void normalise(Unit16& x, float eps) {
  uint64_t s2 = fmul2(x.a[0], x.a[0]), s3 = fmul2(x.b[0], x.b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    s2 = ffma2(x.a[i], x.a[i], s2);
    s3 = ffma2(x.b[i], x.b[i], s3);
  }
  float q0, q1;
  f2unpack(fadd2(s2, s3), q0, q1);
  float ss = q0 + q1;
#pragma unroll
  for (int o = D / 32; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float m = fmaf(ss, 1.f / D, eps);
  float rs = rsqrtf(m);
  // one Newton step, left out where there is nothing finite to work on (m zero or infinite)
  const float nr = rs * fmaf(-0.5f * m * rs, rs, 1.5f);
  rs = nr <= FLT_MAX ? nr : rs;
  const uint64_t rs2 = f2pack(rs, rs);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x.a[i] = fmul2(x.a[i], rs2);
    x.b[i] = fmul2(x.b[i], rs2);
  }
}
__device__ __forceinline__ void turn(Unit16& x, const Factors& f, bool turned) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t ya = fmul2(x.a[i], f.e0[i]), yb = fmul2(x.b[i], f.e2[i]);
    if (turned) {  // (elsewhere a product with zero would turn an infinity into NaN)
      ya = ffma2(x.b[i], f.e1[i], ya);
      yb = ffma2(x.a[i], f.e3[i], yb);
    }
    x.a[i] = ya;
    x.b[i] = yb;
  }
}
__device__ __forceinline__ void turn(Unit16& x, const Angles& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t a = x.a[i];
    x.a[i] = ffma2(x.b[i], t.s[i] ^ NEG2, fmul2(a, t.c[i]));
    x.b[i] = ffma2(a, t.s[i], fmul2(x.b[i], t.c[i]));
  }
}

// The same with every product rounded before the sum (sums of single values, which the compiler never fuses with a product,
// as it does packed ones).
__device__ __forceinline__ uint64_t add_apart(uint64_t x, uint64_t y) {
  float x0, x1, y0, y1;
  f2unpack(x, x0, x1);
  f2unpack(y, y0, y1);
  return f2pack(__fadd_rn(x0, y0), __fadd_rn(x1, y1));
}
__device__ __forceinline__ void turn_rounded(Unit16& x, const Angles& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t a = x.a[i];
    x.a[i] = add_apart(fmul2(a, t.c[i]), fmul2(x.b[i], t.s[i] ^ NEG2));
    x.b[i] = add_apart(fmul2(x.b[i], t.c[i]), fmul2(a, t.s[i]));
  }
}

// Tokens of sequence b: first, and how many, clipped to what the call covers; `all` of them, from which positions count
// (token i is at L - all + i also where the last ones were cut off).
__device__ __forceinline__ bool tokens_of(const AppendPagedParams& p, int b, int& t0, int& n, int& all) {
  if (p.cu == nullptr) {
    n = all = p.T / p.B;
    t0 = b * n;
    return true;
  }
  t0 = __ldg(p.cu + b);
  n = all = static_cast<int>(static_cast<unsigned>(__ldg(p.cu + b + 1)) - static_cast<unsigned>(t0));
  const int most = min(p.max_new, p.T - t0);
  if (t0 >= 0 && n >= 0 && n <= most) return true;
  n = t0 < 0 ? 0 : max(0, min(n, most));
  return false;
}

// What is added to a row of sequence b to give the position that its rotation counts from.
__device__ __forceinline__ unsigned offset_of(const AppendPagedParams& p, int b) {
  return p.offsets == nullptr ? 0u : static_cast<unsigned>(__ldg(p.offsets + b));
}

// ---- query block: rows tok0 .. of the step, all heads
template <int D, bool INTER>
__device__ __forceinline__ void query_block(const AppendPagedParams& p, int block, int* s_pos, uint4* ring) {
  constexpr int LPR = D / 16;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int groups = nt / LPR;
  const int rows = groups / p.q_slots;  // rows of a block
  const int tok0 = block * rows;
  // positions of the rows: each sequence with tokens among them writes its own
  constexpr int NONE = INT_MIN;
  if (p.cu == nullptr) {
    const int n = p.T / p.B;
    for (int r = tid; r < rows; r += nt) {
      const int tok = tok0 + r, b = tok / n;
      const int L = tok < p.T ? __ldg(p.seqlens + b) : 0;
      s_pos[r] = L != 0 ? static_cast<int>(static_cast<unsigned>(L) - n + (tok - b * n) + offset_of(p, b)) : NONE;
    }
  } else {
    for (int r = tid; r < rows; r += nt) s_pos[r] = NONE;
    __syncthreads();
    for (int b = tid; b < p.B; b += nt) {
      int t0, n, all;
      if (!tokens_of(p, b, t0, n, all) && block == 0) atomicOr(p.status, FA_DEV_BAD_LENS);
      const int a = max(t0, tok0), e = min(t0 + n, tok0 + rows);
      if (a < e) {
        const int L = __ldg(p.seqlens + b);
        if (L != 0)  // (a position that wraps lies outside the cache, which the K/V blocks report)
          for (int t = a; t < e; ++t)
            s_pos[t - tok0] = static_cast<int>(static_cast<unsigned>(L) - all + (t - t0) + offset_of(p, b));
      }
    }
  }
  __syncthreads();
  const int grp = tid / LPR, u = tid % LPR;
  const int r = grp % rows, slot = grp / rows;
  const int pos = s_pos[r];
  const bool ok = pos != NONE;
  const UnitPlace<INTER> at(u, p.rot);
  const long long tok = ok ? tok0 + r : 0;
  const uint16_t* src = static_cast<const uint16_t*>(p.q) + tok * p.qst + slot * p.qsh;
  uint16_t* dst = static_cast<uint16_t*>(p.q_out) + tok * p.qost + slot * p.qosh;
  const long long sstep = p.q_slots * p.qsh, dstep = p.q_slots * p.qosh;
  const bool normed = p.q_weight != nullptr;
  // each thread's own ring of asynchronous copies: AP_RING heads in flight without a register
  const uint32_t mine = smem_u32(ring + tid);
  int h = slot, hn = slot;  // head worked on, head of the next copy
  auto fetch = [&](int i) {
    const uint32_t n = ok && hn < p.H ? 16u : 0u;
    cp_async16_ca(mine + (2 * i) * nt * 16, src + (n ? at.c0 : 0), n);
    cp_async16_ca(mine + (2 * i + 1) * nt * 16, src + (n ? at.c1 : 0), n);
    cp_async_commit();
    hn += p.q_slots;
    if (hn < p.H) src += sstep;
  };
#pragma unroll
  for (int i = 0; i < AP_RING; ++i) fetch(i);
  Factors f;
  factors_at<INTER>(f, at.turned, static_cast<uint32_t>(pos), p.turns + 8 * u, p.rot_scale,
                    static_cast<const uint16_t*>(p.q_weight), at.c0, at.c1);
  // (the same number of rounds in every thread: whole warps shuffle)
  const int rounds = (p.H + p.q_slots - 1) / p.q_slots;
  for (int it = 0; it < rounds; it += AP_RING) {
#pragma unroll
    for (int i = 0; i < AP_RING; ++i) {
      if (it + i >= rounds) break;
      cp_async_wait<AP_RING - 1>();
      Unit16 x = unpack16<INTER>(ring[2 * i * nt + tid], ring[(2 * i + 1) * nt + tid]);
      if (normed) normalise<D>(x, p.eps);
      turn(x, f, at.turned);
      fetch(i);  // (the slot has been read: x was computed from it)
      float y[16];
      in_order<INTER>(x, y);
      if (ok && h < p.H) {
        *reinterpret_cast<uint4*>(dst + at.c0) = pack8(y);
        *reinterpret_cast<uint4*>(dst + at.c1) = pack8(y + 8);
      }
      dst += dstep;
      h += p.q_slots;
    }
  }
  cp_async_wait<0>();
}

// The new rows of one page that K/V block c takes: those of sequence b, from row r0 of page `page0` of the sequence on, whose
// first position is `first`; token tok0 is the first of them. Uniform over the block; `nrows` 0: nothing to do.
struct PageRows {
  int b, page0, r0, nrows, tok0;
  long long first;
};
__device__ __forceinline__ PageRows rows_of(const AppendPagedParams& p, int c) {
  PageRows w{};
  int i;
  if (p.per_seq > 0) {
    w.b = c / p.per_seq;
    i = c - w.b * p.per_seq;
  } else {
    // Sequence b owns the blocks from cu[b] / page + 2 b on: at least as many as its tokens can touch pages. Every warp
    // finds the last b that starts at or before block c for itself, 32 candidates at a time.
    auto base = [&](int x) { return (max(__ldg(p.cu + x), 0) >> p.page_shift) + 2 * x; };
    int lo = 0, n = p.B;
    while (n > 1) {
      const int step = (n + 31) / 32, x = lo + static_cast<int>(threadIdx.x & 31) * step;
      const unsigned at_or_before = __ballot_sync(0xffffffffu, x < lo + n && base(x) <= c);
      const int skip = max(__popc(at_or_before) - 1, 0) * step;
      lo += skip;
      n = min(step, n - skip);
    }
    w.b = lo;
    i = c - base(lo);
  }
  int t0, n, all;
  (void)tokens_of(p, w.b, t0, n, all);
  const int L = __ldg(p.seqlens + w.b);
  const long long start = static_cast<long long>(L) - all, end = start + n;       // positions
  w.page0 = static_cast<int>(start >> p.page_shift) + i;                          // this block's page of the sequence
  w.first = static_cast<long long>(w.page0) << p.page_shift;
  // (blocks below the first sequence's, where tokens come before it, have i < 0)
  if (n == 0 || L == 0 || i < 0 || w.first >= end) return w;
  w.r0 = start > w.first ? static_cast<int>(start - w.first) : 0;                 // its new rows r0 .. r0 + nrows - 1
  w.nrows = static_cast<int>(end - w.first < p.page ? end - w.first : p.page) - w.r0;
  w.tok0 = t0 + static_cast<int>(w.first + w.r0 - start);                         // token of row r0
  return w;
}

// ---- K/V block of 4-bit rows: the new rows of one page, p.kv_heads K/V heads
// Rows do not depend on one another, so a block streams them, head after head, through a ring of copies, each thread's own,
// and the angles of a row are worked out once for its heads.
template <int D, bool INTER>
__device__ __forceinline__ void kv_block4(const AppendPagedParams& p, int block, uint4* ring) {
  constexpr int LPR = D / 16;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int groups = nt / LPR;
  const int parts = (p.Hkv + p.kv_heads - 1) / p.kv_heads;
  const int hk0 = block % parts * p.kv_heads, heads = min(p.kv_heads, p.Hkv - hk0);
  const PageRows w = rows_of(p, block / parts);
  if (w.nrows == 0) return;
  const bool in_table = w.page0 >= 0 && w.page0 < p.width;
  const int id = in_table ? __ldg(p.table + w.b * p.table_stride + w.page0) : -1;
  const int grp = tid / LPR, u = tid % LPR;
  const UnitPlace<INTER> at(u, p.rot);
  const int rounds = (w.nrows + groups - 1) / groups;             // (the same in every thread)
  const uint16_t* kb = static_cast<const uint16_t*>(p.k) + w.tok0 * p.kst + hk0 * p.ksh;
  const uint16_t* vb = static_cast<const uint16_t*>(p.v) + w.tok0 * p.vst + hk0 * p.vsh;
  // copies: the key's blocks of eight elements that this thread turns, the value's 16 neighbours of one scale
  int fr = 0, fh = 0;                                             // round and head of the next
  auto fetch = [&](int slot) {
    const int r = fr * groups + grp;
    const uint32_t nb = r < w.nrows ? 16u : 0u, mine = smem_u32(ring + slot * 4 * nt + tid);  // (past the last round: none)
    const uint16_t* ks = kb + (nb ? r * p.kst + fh * p.ksh : 0);
    const uint16_t* vs = vb + (nb ? r * p.vst + fh * p.vsh : 0);
    cp_async16_ca(mine, ks + at.c0, nb);
    cp_async16_ca(mine + nt * 16, ks + at.c1, nb);
    cp_async16_ca(mine + 2 * nt * 16, vs + 16 * u, nb);
    cp_async16_ca(mine + 3 * nt * 16, vs + 16 * u + 8, nb);
    cp_async_commit();
    if (++fh == heads) fh = 0, ++fr;
  };
#pragma unroll
  for (int i = 0; i < AP_KV_RING; ++i) fetch(i);
  const long long pbase = paged_row_offset(id, p.num_pages, p.Hkv, hk0, p.page, 0, 1);
  const bool store = pbase >= 0;
  if (!store && tid == 0 && hk0 == 0) atomicOr(p.status, in_table ? FA_DEV_BAD_PAGE : FA_DEV_BAD_LENS);
  const uint32_t pos0 = static_cast<uint32_t>(w.first) + w.r0 + offset_of(p, w.b);
  // A scale's 16 neighbours are blocks 2i and 2i + 1 of eight elements. This thread has blocks c0 / 8 and c1 / 8, and the
  // other one of each pair may be another thread's of the same row: lane `from` has it, as its first or its second.
  const int turned = p.rot / 16;                                  // units that are
  auto holder = [&](int k) { return INTER ? k / 2 : k < turned ? k : k < 2 * turned ? k - turned : turned + (k - 2 * turned) / 2; };
  auto piece_of = [&](int k) { return INTER ? k & 1 : k < turned ? 0 : k < 2 * turned ? 1 : k & 1; };  // first or second there
  const int k0 = (at.c0 / 8) ^ 1, k1 = (at.c1 / 8) ^ 1, from0 = holder(k0), from1 = holder(k1);
  // A norm's sum of squares: elements 32 apart in order, then neighbours in pairs, whatever the rotation's layout. This thread
  // adds up elements SPAN u .. SPAN u + SPAN - 1 and those 32, 64, .. on, which lie in pieces of the row's other threads.
  constexpr int SPAN = 32 / LPR, CHAIN = D / 32;
  int sq_at[CHAIN];
#pragma unroll
  for (int j = 0; j < CHAIN; ++j) {
    const int k = 4 * j + SPAN * u / 8;
    sq_at[j] = 16 * (piece_of(k) * nt + tid - u + holder(k)) + 2 * (SPAN * u % 8);  // (bytes)
  }
  int slot = 0;
  for (int it = 0; it < rounds; ++it) {
    const int r = it * groups + grp;
    const bool ok = r < w.nrows;
    Angles t;
    if (at.turned) angles_rounded_at(t, pos0 + r, p.turns + 8 * u, p.rot_scale);
    const long long row = pbase + w.r0 + r;
    for (int h = 0; h < heads; ++h) {
      cp_async_wait<AP_KV_RING - 1>();
      const uint4* mine = ring + slot * 4 * nt + tid;
      Unit16 x = unpack16<INTER>(mine[0], mine[nt]);
      if (p.k_weight != nullptr) {
        __syncwarp();  // the row's other threads' copies have landed
        uint64_t sq[SPAN / 2];
#pragma unroll
        for (int j = 0; j < CHAIN; ++j) {
          const uint8_t* from = reinterpret_cast<const uint8_t*>(ring + slot * 4 * nt) + sq_at[j];
          uint32_t y[SPAN / 2];
          if constexpr (SPAN == 8) {
            const uint4 z = *reinterpret_cast<const uint4*>(from);
            y[0] = z.x, y[1] = z.y, y[2] = z.z, y[3] = z.w;
          } else {
            const uint2 z = *reinterpret_cast<const uint2*>(from);
            y[0] = z.x, y[1] = z.y;
          }
#pragma unroll
          for (int i = 0; i < SPAN / 2; ++i) {  // (squares of bf16 values are exact: one rounding, that of the sum)
            const uint64_t e = f2pack(__uint_as_float(y[i] << 16), __uint_as_float(y[i] & 0xffff0000u));
            sq[i] = j == 0 ? fmul2(e, e) : ffma2(e, e, sq[i]);
          }
        }
        __syncwarp();  // (fetch may write the slot)
        float part[SPAN / 2];
#pragma unroll
        for (int i = 0; i < SPAN / 2; ++i) {
          float e0, e1;
          f2unpack(sq[i], e0, e1);
          part[i] = __fadd_rn(e0, e1);
        }
        float ss = __fadd_rn(part[0], part[1]);
        if constexpr (SPAN == 8) ss = __fadd_rn(ss, __fadd_rn(part[2], part[3]));
#pragma unroll
        for (int o = 1; o < LPR; o *= 2) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
        const float rs = rsqrtf(fmaf(ss, 1.f / D, p.eps));
        const uint64_t rs2 = f2pack(rs, rs);
        const uint16_t* wt = static_cast<const uint16_t*>(p.k_weight);
        const Unit16 f = unpack16<INTER>(__ldg(reinterpret_cast<const uint4*>(wt + at.c0)), __ldg(reinterpret_cast<const uint4*>(wt + at.c1)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x.a[j] = fmul2(fmul2(x.a[j], rs2), f.a[j]);
          x.b[j] = fmul2(fmul2(x.b[j], rs2), f.b[j]);
        }
      }
      if (at.turned) turn_rounded(x, t);
      float y[16];
      in_order<INTER>(x, y);
      const uint4 y0 = pack8(y), y1 = pack8(y + 8);
      // the key as k_out gives it, in bf16 (whole warps shuffle)
      uint32_t m0 = bf16x8_amax_bits(y0), m1 = bf16x8_amax_bits(y1);
      if (INTER || !at.turned) m0 = m1 = max(m0, m1);
      if (!INTER) {
        const uint32_t a0 = __shfl_sync(0xffffffffu, m0, from0, LPR), b0 = __shfl_sync(0xffffffffu, m1, from0, LPR);
        const uint32_t a1 = __shfl_sync(0xffffffffu, m0, from1, LPR), b1 = __shfl_sync(0xffffffffu, m1, from1, LPR);
        m0 = max(m0, k0 < turned ? a0 : b0);
        m1 = max(m1, k1 < turned ? a1 : b1);
      }
      const uint4 v0 = mine[2 * nt], v1 = mine[3 * nt];
      fetch(slot);  // (the slot has been read)
      slot = slot + 1 == AP_KV_RING ? 0 : slot + 1;
      if (!ok) continue;
      if (p.k_out != nullptr) {
        uint16_t* ko = static_cast<uint16_t*>(p.k_out) + (w.tok0 + static_cast<long long>(r)) * p.kost + (hk0 + h) * p.kosh;
        *reinterpret_cast<uint4*>(ko + at.c0) = y0;
        *reinterpret_cast<uint4*>(ko + at.c1) = y1;
      }
      if (!store) continue;
      float i0, i1, iv;
      const uint32_t s0 = fp4_scale_byte(m0, i0), s1 = fp4_scale_byte(m1, i1);
      const uint32_t sv = fp4_scale_byte(max(bf16x8_amax_bits(v0), bf16x8_amax_bits(v1)), iv);
      const long long at_row = row + static_cast<long long>(h) * p.page;
      uint8_t* kd = static_cast<uint8_t*>(p.k_pages) + at_row * (D / 2);
      uint8_t* vd = static_cast<uint8_t*>(p.v_pages) + at_row * (D / 2);
      *reinterpret_cast<uint32_t*>(kd + at.c0 / 2) = fp4_codes8(y0, i0);
      *reinterpret_cast<uint32_t*>(kd + at.c1 / 2) = fp4_codes8(y1, i1);
      *reinterpret_cast<uint2*>(vd + 8 * u) = make_uint2(fp4_codes8(v0, iv), fp4_codes8(v1, iv));
      // (both threads of a group have the same scale; the one with the even block writes it)
      if ((at.c0 & 8) == 0) p.k_scale4[at_row * (D / 16) + at.c0 / 16] = static_cast<uint8_t>(s0);
      if ((at.c1 & 8) == 0) p.k_scale4[at_row * (D / 16) + at.c1 / 16] = static_cast<uint8_t>(s1);
      p.v_scale4[at_row * (D / 16) + u] = static_cast<uint8_t>(sv);
    }
  }
  cp_async_wait<0>();
}

// ---- K/V block of bf16 or e4m3 rows: the new rows of one page, one K/V head
template <int D, int KIND, bool INTER>
__device__ __forceinline__ void kv_block(const AppendPagedParams& p, int block, unsigned int* s_amax, uint4* stash) {
  constexpr int LPR = D / 16;
  constexpr bool F8 = KIND == PAGES_E4M3;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int groups = nt / LPR;
  const int hk = block % p.Hkv;
  if constexpr (F8) {
    if (tid < 2) s_amax[tid] = 0u;
    __syncthreads();
  }
  const PageRows w = rows_of(p, block / p.Hkv);
  const int b = w.b, page0 = w.page0, r0 = w.r0, nrows = w.nrows, tok0 = w.tok0;
  const long long first = w.first;
  if (nrows == 0) return;  // (uniform over the block)

  const uint32_t offset = offset_of(p, b);

  // the table entry and the first rows are asked for together
  const bool in_table = page0 >= 0 && page0 < p.width;
  const int id = in_table ? __ldg(p.table + b * p.table_stride + page0) : -1;
  const int grp = tid / LPR, u = tid % LPR;
  const UnitPlace<INTER> at(u, p.rot);
  const uint16_t* kb = static_cast<const uint16_t*>(p.k) + tok0 * p.kst + hk * p.ksh;
  const uint16_t* vb = static_cast<const uint16_t*>(p.v) + tok0 * p.vst + hk * p.vsh;
  // every round's rows are copied to this thread's own pieces of shared memory: 0, 1 the key, 4, 5 the value
  constexpr int PIECES = F8 ? 6 : 4, VP = PIECES - 2;
  const int rounds = (nrows + groups - 1) / groups;              // (the same in every thread)
  for (int it = 0; it < rounds; ++it) {
    const int r = it * groups + grp;
    const uint32_t nb = r < nrows ? 16u : 0u, mine = smem_u32(stash + it * PIECES * nt + tid);
    const uint16_t* ks = kb + (nb ? r * p.kst : 0);
    const uint16_t* vs = vb + (nb ? r * p.vst : 0);
    cp_async16_ca(mine, ks + at.c0, nb);
    cp_async16_ca(mine + nt * 16, ks + at.c1, nb);
    cp_async16_ca(mine + VP * nt * 16, vs + at.c0, nb);
    cp_async16_ca(mine + (VP + 1) * nt * 16, vs + at.c1, nb);
  }
  cp_async_commit();
  const long long pbase = paged_row_offset(id, p.num_pages, p.Hkv, hk, p.page, 0, D);
  const bool store = pbase >= 0;
  if (!store && tid == 0 && hk == 0) atomicOr(p.status, in_table ? FA_DEV_BAD_PAGE : FA_DEV_BAD_LENS);
  float old_k = 0.f, old_v = 0.f;
  const long long sidx = static_cast<long long>(id) * p.Hkv + hk;
  if constexpr (F8) {
    if (store) {
      old_k = p.k_scale[sidx];
      old_v = p.v_scale[sidx];
    }
  }
  uint16_t* kob = p.k_out == nullptr ? nullptr : static_cast<uint16_t*>(p.k_out) + tok0 * p.kost + hk * p.kosh;
  float am_k = 0.f, am_v = 0.f;
  cp_async_wait<0>();
  for (int it = 0; it < rounds; ++it) {
    const int r = it * groups + grp;
    const bool ok = r < nrows;
    uint4* mine = stash + it * PIECES * nt + tid;
    Unit16 x = unpack16<INTER>(mine[0], mine[nt]);
    if (p.k_weight != nullptr) {
      normalise<D>(x, p.eps);
      const uint16_t* wt = static_cast<const uint16_t*>(p.k_weight);
      const Unit16 w = unpack16<INTER>(__ldg(reinterpret_cast<const uint4*>(wt + at.c0)), __ldg(reinterpret_cast<const uint4*>(wt + at.c1)));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x.a[j] = fmul2(x.a[j], w.a[j]);
        x.b[j] = fmul2(x.b[j], w.b[j]);
      }
    }
    if (!ok) continue;
    if (at.turned) {
      Angles t;
      angles_at(t, static_cast<uint32_t>(first) + r0 + r + offset, p.turns + 8 * u, p.rot_scale);
      turn(x, t);
    }
    float y[16];
    in_order<INTER>(x, y);
    const uint4 y0 = pack8(y), y1 = pack8(y + 8);
    if (kob != nullptr) {
      *reinterpret_cast<uint4*>(kob + r * p.kost + at.c0) = y0;
      *reinterpret_cast<uint4*>(kob + r * p.kost + at.c1) = y1;
    }
    if (!store) continue;
    if constexpr (F8) {
      am_k = fmaxf(am_k, finite_amax(y));
      // the turned key, in fp32, over pieces 0 .. 3
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(mine + e * nt) = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
      am_v = fmaxf(am_v, finite_amax(mine[VP * nt], mine[(VP + 1) * nt]));
    } else {
      const long long ro = pbase + (r0 + r) * D;
      uint16_t* kd = static_cast<uint16_t*>(p.k_pages) + ro;
      uint16_t* vd = static_cast<uint16_t*>(p.v_pages) + ro;
      *reinterpret_cast<uint4*>(kd + at.c0) = y0;
      *reinterpret_cast<uint4*>(kd + at.c1) = y1;
      *reinterpret_cast<uint4*>(vd + at.c0) = mine[VP * nt];
      *reinterpret_cast<uint4*>(vd + at.c1) = mine[(VP + 1) * nt];
    }
  }
  if constexpr (F8) {
    if (!store) return;  // (uniform)
    // magnitudes order as unsigned integers; a maximum does not depend on its order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      am_k = fmaxf(am_k, __shfl_xor_sync(0xffffffffu, am_k, o));
      am_v = fmaxf(am_v, __shfl_xor_sync(0xffffffffu, am_v, o));
    }
    if ((tid & 31) == 0) {
      atomicMax(&s_amax[0], __float_as_uint(am_k));
      atomicMax(&s_amax[1], __float_as_uint(am_v));
    }
    __syncthreads();
    const float sk = merged_scale(__uint_as_float(s_amax[0]), old_k, r0 > 0);
    const float sv = merged_scale(__uint_as_float(s_amax[1]), old_v, r0 > 0);
    uint8_t* kp = static_cast<uint8_t*>(p.k_pages) + pbase;
    uint8_t* vp = static_cast<uint8_t*>(p.v_pages) + pbase;
    // the codes already held, where the scale grew
    const bool rk = r0 > 0 && sk != old_k, rvv = r0 > 0 && sv != old_v;
    if (rk || rvv) {
      const float fk = old_k > 0.f && old_k <= FLT_MAX ? old_k / sk : 1.f;
      const float fv = old_v > 0.f && old_v <= FLT_MAX ? old_v / sv : 1.f;
      for (int x = tid; x < r0 * (D / 4); x += nt) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (!(w ? rvv : rk)) continue;
          uint32_t* at4 = reinterpret_cast<uint32_t*>(w ? vp : kp) + x;
          const uint32_t old = *at4;
          uint32_t h0, h1;
          e4m3x4_to_f16x2x2(old, h0, h1);
          const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
          const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
          *at4 = to_codes4(f0.x, f0.y, f1.x, f1.y, w ? fv : fk);
        }
      }
    }
    const float ik = 1.f / sk, iv = 1.f / sv;  // exact for powers of two, the scales that append writes
    for (int it = 0; it < rounds; ++it) {
      const int r = it * groups + grp;
      if (r >= nrows) break;
      const uint4* mine = stash + it * PIECES * nt + tid;
      uint32_t cw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 f = *reinterpret_cast<const float4*>(mine + e * nt);
        cw[e] = to_codes4(f.x, f.y, f.z, f.w, ik);
      }
      const int ro = (r0 + r) * D;
      *reinterpret_cast<uint2*>(kp + ro + at.c0) = make_uint2(cw[0], cw[1]);
      *reinterpret_cast<uint2*>(kp + ro + at.c1) = make_uint2(cw[2], cw[3]);
      const uint4 v0 = mine[VP * nt], v1 = mine[(VP + 1) * nt];
      const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        cw[e] = to_codes4(__uint_as_float(vw[2 * e] << 16), __uint_as_float(vw[2 * e] & 0xffff0000u),
                          __uint_as_float(vw[2 * e + 1] << 16), __uint_as_float(vw[2 * e + 1] & 0xffff0000u), iv);
      *reinterpret_cast<uint2*>(vp + ro + at.c0) = make_uint2(cw[0], cw[1]);
      *reinterpret_cast<uint2*>(vp + ro + at.c1) = make_uint2(cw[2], cw[3]);
    }
    if (tid == 0) {
      p.k_scale[sidx] = sk;
      p.v_scale[sidx] = sv;
    }
  }
}

}  // namespace

template <int D, int KIND, bool INTER>
__global__ void __launch_bounds__(AP_THREADS, ap_ctas(KIND, INTER)) fa_append_paged_kernel(const AppendPagedParams p) {
  extern __shared__ __align__(16) uint4 ap_stash[];  // 16-byte pieces, one of each thread next to one another
  __shared__ int s_pos[AP_THREADS / (D / 16)];
  __shared__ unsigned int s_amax[2];
  const int block = static_cast<int>(blockIdx.x);
  pdl_launch_dependents();  // (a read of the rows may be launched beside the last blocks; it waits for all of them)
  // The two kinds are spread evenly over the launch: a K/V block is mostly a chain of waits (which sequence, its page, its
  // rows, the page's largest value), which the query blocks beside it fill.
  const unsigned long long blocks = gridDim.x;
  const int before = static_cast<int>(static_cast<unsigned long long>(block) * p.kv_blocks / blocks);  // K/V blocks before this one
  const bool kv = static_cast<int>((block + 1ull) * p.kv_blocks / blocks) > before;
  if constexpr (KIND == PAGES_FP4) {
    if (kv) kv_block4<D, INTER>(p, before, ap_stash);
  } else {
    if (kv) kv_block<D, KIND, INTER>(p, before, s_amax, ap_stash);
  }
  if (!kv) query_block<D, INTER>(p, block - before, s_pos, ap_stash);
}

// Bytes of a block's pieces: a page's rounds of keys and values (4-bit rows: their ring), or a query block's ring.
static int ap_smem_bytes(int D, int kind, int rows, int threads) {
  const int groups = threads / (D / 16), rounds = (rows + groups - 1) / groups;
  return std::max(kind == PAGES_FP4 ? 4 * AP_KV_RING : rounds * (kind == PAGES_E4M3 ? 6 : 4), 2 * AP_RING) * threads * 16;
}
template <int D, int KIND, bool INTER>
static cudaError_t ap_attr() {
  return cudaFuncSetAttribute(fa_append_paged_kernel<D, KIND, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              ap_smem_bytes(D, KIND, 128, AP_THREADS));
}
template <int KIND>
static cudaError_t ap_attrs() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t x : {ap_attr<64, KIND, false>(), ap_attr<64, KIND, true>(), ap_attr<128, KIND, false>(),
                        ap_attr<128, KIND, true>()})
    if (x != cudaSuccess) e = x;
  return e;
}
cudaError_t append_paged_set_attributes() {
  cudaError_t e = cudaSuccess;
  for (cudaError_t x : {ap_attrs<PAGES_BF16>(), ap_attrs<PAGES_E4M3>(), ap_attrs<PAGES_FP4>()})
    if (x != cudaSuccess) e = x;
  return e;
}

template <int D, int KIND, bool INTER>
static cudaError_t ap_launch(AppendPagedParams p, cudaStream_t stream) {
  // As many threads as a page's new rows occupy, so that an SM holds many blocks of small pages or short steps (256
  // sequences of one token, 8 K/V heads: 8 us, 21 with 256 threads; 26.7k prompt tokens into pages of 16: 125 us, 170).
  int threads = AP_STEP_THREADS;
  while (threads < AP_THREADS && threads < p.max_rows * (D / 16)) threads *= 2;
  const int groups = threads / (D / 16);
  // Heads side by side in a query block: few where many rows fill the GPU anyway (a row's angles are computed once a
  // slot), many for a short step: slots are added until q_blocks_wanted blocks run. (Six an SM: 115 us for 26.7k prompt
  // tokens, 32 us for 9.1k of 28 heads; four an SM 117 and 32, eight 115 and 35.)
  int slots = 1;
  while (slots < groups && slots < p.H && static_cast<long long>(p.T) * slots < static_cast<long long>(groups) * p.q_blocks_wanted)
    slots *= 2;
  p.q_slots = slots;
  if constexpr (KIND == PAGES_FP4) {
    // K/V heads of a block, which share a row's angles: as long as a page's rows fill the block, two blocks an SM (a third of
    // the query blocks wanted) are left, and a block has no more than eight turns. 26k prompt tokens, 32/8 heads, 1, 2, 4, 8
    // heads: pages of 64 132, 114, 112, 122 us; pages of 16 149, 124, 109, 104; pages of 128 127, 121, 127, 126.
    const long long pages = p.kv_blocks / p.Hkv;
    const int rounds = (p.max_rows + groups - 1) / groups;
    p.kv_heads = 1;
    while (p.kv_heads < AP_KV_HEADS && p.kv_heads < p.Hkv && p.max_rows >= groups && 2 * p.kv_heads * rounds <= 8 &&
           pages * p.Hkv >= 2LL * p.kv_heads * (p.q_blocks_wanted / 3))
      p.kv_heads *= 2;
    p.kv_blocks = static_cast<int>(pages * ((p.Hkv + p.kv_heads - 1) / p.kv_heads));
  }
  const int rows = groups / slots;
  const long long q_blocks = (static_cast<long long>(p.T) + rows - 1) / rows;
  const size_t smem = ap_smem_bytes(D, KIND, p.max_rows, threads);
  fa_append_paged_kernel<D, KIND, INTER><<<static_cast<unsigned>(p.kv_blocks + q_blocks), threads, smem, stream>>>(p);
  return cudaGetLastError();
}
template <int D, int KIND>
static cudaError_t ap_launch_kind(const AppendPagedParams& p, cudaStream_t stream) {
  return p.interleaved ? ap_launch<D, KIND, true>(p, stream) : ap_launch<D, KIND, false>(p, stream);
}
template <int D>
static cudaError_t ap_launch_d(int kind, const AppendPagedParams& p, cudaStream_t stream) {
  if (kind == PAGES_FP4) return ap_launch_kind<D, PAGES_FP4>(p, stream);
  return kind == PAGES_E4M3 ? ap_launch_kind<D, PAGES_E4M3>(p, stream) : ap_launch_kind<D, PAGES_BF16>(p, stream);
}
cudaError_t launch_append_paged(int kind, const AppendPagedParams& p, cudaStream_t stream) {
  return p.d == 64 ? ap_launch_d<64>(kind, p, stream) : ap_launch_d<128>(kind, p, stream);
}

}  // namespace fa
