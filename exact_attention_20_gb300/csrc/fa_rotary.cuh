// Rotary positions: turning queries and keys by their positions, and appending
// new keys and values to the paged 4-bit cache with the turn on the way.
//
// The first `rot` elements of a head's d are rot / 2 pairs, (i, i + rot / 2) or,
// interleaved, (2 i, 2 i + 1).  Pair i of a token at position p turns by the
// angle 2 pi frac(p turns[i] / 2^64) and is scaled by m:
//
//     a' = m (a cos - b sin),   b' = m (a sin + b cos),
//
// and the gradient of a by that of a' is the same with -sin.  A pair's speed is
// a 64-bit fraction of a turn per position, so the angle of any 32-bit
// position is one integer product, whose wrap drops whole turns and loses
// nothing: the error is that of the speed's last bit times p, 2^-33 of a turn
// at the most (a speed cut to 64 bits), where p times an fp32 speed would be off by 2^-24 of all the
// turns made.
//
// Rotating alone rounds to bf16 once, and fp32 does (cos and sin to about
// 2^-22).  A key that is stored goes through two roundings, bf16 and then 4
// bits, and neighbouring 4-bit values are up to half apart: so that it is
// the same value whoever computes it, the key is rounded to bf16 from a sum of
// two floats that is right to about 2^-42 (Turn2 below), and the 4-bit rounding
// of a bf16 value is exact (fa_kv4.cuh).  Appending gives, bit for bit, what
// rotating (so rounded) and storing give.
#pragma once

#include "fa_kv4.cuh"

namespace fa {
namespace rotary {

constexpr int kThreads = 256;

// sin(2 pi k / 256), k = 0 .. 64, as a sum of two floats.
__device__ const float2 kSine[65] = {
    {0x0p+0f, 0x0p+0f}, {0x1.92156p-6f, -0x1.0b933p-31f}, {0x1.91f66p-5f, -0x1.de44fep-30f},
    {0x1.2d520ap-4f, -0x1.a63cc2p-29f}, {0x1.917a6cp-4f, -0x1.eb25eap-31f}, {0x1.f564e6p-4f, -0x1.2ad19ep-29f},
    {0x1.2c8106p-3f, 0x1.d1cc28p-28f}, {0x1.5e2144p-3f, 0x1.22cff2p-29f}, {0x1.8f8b84p-3f, -0x1.cb2cfap-30f},
    {0x1.c0b826p-3f, 0x1.4fc9ecp-28f}, {0x1.f19f98p-3f, -0x1.37a83ap-29f}, {0x1.111d26p-2f, 0x1.58fb3cp-29f},
    {0x1.294062p-2f, 0x1.dab3ep-27f}, {0x1.4135cap-2f, -0x1.7d134p-27f}, {0x1.58f9a8p-2f, -0x1.4a9c04p-27f},
    {0x1.708854p-2f, -0x1.e0b74cp-27f}, {0x1.87de2ap-2f, 0x1.abaa58p-28f}, {0x1.9ef794p-2f, 0x1.d476c6p-29f},
    {0x1.b5d1p-2f, 0x1.3c2b98p-27f}, {0x1.cc66eap-2f, -0x1.b38ee8p-28f}, {0x1.e2b5d4p-2f, -0x1.fe4272p-28f},
    {0x1.f8ba4ep-2f, -0x1.01d952p-28f}, {0x1.07387ap-1f, -0x1.b74004p-27f}, {0x1.11eb36p-1f, -0x1.7c969cp-26f},
    {0x1.1c73b4p-1f, -0x1.9465cep-27f}, {0x1.26d054p-1f, 0x1.9ba25cp-26f}, {0x1.30ff8p-1f, -0x1.8f47e6p-28f},
    {0x1.3affa2p-1f, 0x1.240a18p-26f}, {0x1.44cf32p-1f, 0x1.424776p-27f}, {0x1.4e6cacp-1f, -0x1.070686p-27f},
    {0x1.57d694p-1f, -0x1.6e626cp-26f}, {0x1.610b76p-1f, -0x1.5c5a64p-26f}, {0x1.6a09e6p-1f, 0x1.9fcef4p-27f},
    {0x1.72d084p-1f, -0x1.02000ep-26f}, {0x1.7b5df2p-1f, 0x1.3557d8p-28f}, {0x1.83b0ep-1f, 0x1.7ff2eep-26f},
    {0x1.8bc806p-1f, 0x1.62a2e8p-26f}, {0x1.93a224p-1f, 0x1.324c8p-26f}, {0x1.9b3e04p-1f, 0x1.fce1dp-27f},
    {0x1.a29a7ap-1f, 0x1.189e08p-31f}, {0x1.a9b662p-1f, 0x1.21d434p-26f}, {0x1.b090a6p-1f, -0x1.fabf8p-27f},
    {0x1.b72834p-1f, 0x1.465b9p-27f}, {0x1.bd7c0ap-1f, 0x1.8df2a6p-26f}, {0x1.c38b3p-1f, -0x1.cfe84ap-26f},
    {0x1.c954b2p-1f, 0x1.3411f4p-29f}, {0x1.ced7bp-1f, -0x1.786712p-26f}, {0x1.d4134ep-1f, -0x1.d646d8p-26f},
    {0x1.d906bcp-1f, 0x1.e651a8p-26f}, {0x1.ddb13cp-1f, -0x1.2667b8p-26f}, {0x1.e2121p-1f, 0x1.3da1bap-27f},
    {0x1.e6288ep-1f, 0x1.891c22p-26f}, {0x1.e9f416p-1f, -0x1.273a44p-26f}, {0x1.ed740ep-1f, 0x1.da1258p-27f},
    {0x1.f0a7fp-1f, -0x1.1b73cap-27f}, {0x1.f38f3ap-1f, 0x1.8c9cb2p-26f}, {0x1.f6297cp-1f, 0x1.feeb96p-26f},
    {0x1.f8765p-1f, -0x1.63ad16p-27f}, {0x1.fa7558p-1f, -0x1.eeb5d2p-30f}, {0x1.fc2648p-1f, -0x1.e3cc06p-26f},
    {0x1.fd88dap-1f, 0x1.e89292p-28f}, {0x1.fe9cdap-1f, 0x1.a03108p-26f}, {0x1.ff621ep-1f, 0x1.bcb6bep-28f},
    {0x1.ffd886p-1f, 0x1.099a1ap-30f}, {0x1p+0f, 0x0p+0f},
};

struct Float2 {  // hi + lo, |lo| at most half a unit of hi's last bit
  float hi, lo;
};

// a + b and the sum's rounding error, whatever the magnitudes.
__device__ __forceinline__ float two_sum(float a, float b, float& err) {
  const float s = __fadd_rn(a, b), x = __fsub_rn(s, a);
  err = __fadd_rn(__fsub_rn(a, __fsub_rn(s, x)), __fsub_rn(b, x));
  return s;
}

// The same where |a| >= |b|.
__device__ __forceinline__ Float2 quick_two_sum(float a, float b) {
  const float s = __fadd_rn(a, b);
  return Float2{s, __fsub_rn(b, __fsub_rn(s, a))};
}

// cos and sin of a turn given in 2^-64, times m, right to about 2^-44 m.
//
// The turn is the nearest 256th plus b, |b| <= 2 pi / 512.  With d = 1 - cos b
// and e = sin b, cos(a + b) = cos a - cos a d - sin a e and sin(a + b) = sin a -
// sin a d + cos a e.  e = b - b^3 / 6 + b^5 / 120 and d = b^2 / 2 - b^4 / 24: what
// is left out is below 2^-49, and only b and b^2 / 2 need a second float.
struct Turn2 {
  Float2 c, s;
  __device__ __forceinline__ Turn2(unsigned long long turn, float m) {
    const uint32_t k = static_cast<uint32_t>((turn + (1ull << 55)) >> 56);  // 256: a whole turn
    const long long rest = static_cast<long long>(turn - (static_cast<unsigned long long>(k) << 56));
    // the rest in turns as two floats: its upper 24 bits and the 32 below
    const float r1 = static_cast<float>(static_cast<int>(rest >> 32)) * 0x1p-32f;
    const float r2 = static_cast<float>(static_cast<uint32_t>(rest)) * 0x1p-64f;
    constexpr float kTurnHi = 0x1.921fb6p+2f, kTurnLo = -0x1.777a5cp-23f;  // 2 pi
    const float bh0 = r1 * kTurnHi;
    const float bl0 = fmaf(r1, kTurnHi, -bh0) + fmaf(r1, kTurnLo, r2 * kTurnHi);
    const Float2 b = quick_two_sum(bh0, bl0);
    const float b2 = b.hi * b.hi;
    const float el = fmaf(b.hi * b2, fmaf(b2, 1.f / 120.f, -1.f / 6.f), b.lo);  // e = b.hi + el
    const float half = 0.5f * b.hi;
    const float dh = half * b.hi;
    const float dl = fmaf(half, b.hi, -dh) + fmaf(b.hi, b.lo, b2 * b2 * (-1.f / 24.f));  // d = dh + dl
    // sin and cos of the 256th
    const uint32_t j = k & 63u, quarter = (k >> 6) & 3u;
    const float2 x = __ldg(kSine + j), y = __ldg(kSine + 64 - j);
    const float2 sa0 = quarter & 1u ? y : x, ca0 = quarter & 1u ? x : y;
    const float ss = quarter & 2u ? -1.f : 1.f, cs = (quarter + 1u) & 2u ? -1.f : 1.f;
    const float sh = sa0.x * ss, sl = sa0.y * ss, ch = ca0.x * cs, cl = ca0.y * cs;
    c = sum(ch, cl, sh, sl, -1.f, b.hi, el, dh, dl, m);
    s = sum(sh, sl, ch, cl, 1.f, b.hi, el, dh, dl, m);
  }
  // u - u d + sign w e, times m, for two-float u and w
  __device__ static __forceinline__ Float2 sum(float uh, float ul, float wh, float wl, float sign, float eh, float el,
                                               float dh, float dl, float m) {
    const float ws = wh * sign, wls = wl * sign;
    const float p = ws * eh, pe = fmaf(ws, eh, -p);
    const float q = -uh * dh, qe = fmaf(-uh, dh, -q);
    float r1, r2;
    const float t1 = two_sum(uh, p, r1);
    const float t2 = two_sum(t1, q, r2);
    const float low = (r1 + r2) + ((ul + pe) + (qe + fmaf(ws, el, fmaf(wls, eh, -uh * dl))));
    const Float2 v = quick_two_sum(t2, low);
    const float h = v.hi * m;
    return quick_two_sum(h, fmaf(v.hi, m, -h) + v.lo * m);
  }
};

// x c + sign y s rounded to bf16 (as the fp32 value with those bits), for
// bf16 x, y: products with their errors, a sum with its error, and, where the
// fp32 sum is exactly between two bf16 values, the side that the rest is on.
__device__ __forceinline__ float turned(float x, float y, const Float2& c, const Float2& s, float sign) {
  const float ys = y * sign;
  const float p = x * c.hi, t = ys * s.hi;
  float err;
  const float h = two_sum(p, t, err);
  const float low = ((fmaf(x, c.hi, -p) + fmaf(ys, s.hi, -t)) + fmaf(x, c.lo, ys * s.lo)) + err;
  const float v = __fadd_rn(h, low);
  const float rest = __fsub_rn(low, __fsub_rn(v, h));
  uint32_t bits = __float_as_uint(v);
  if ((bits & 0xffffu) == 0x8000u && rest != 0.f) bits += (rest > 0.f) == (v > 0.f) ? 1u : 0xffffffffu;
  // an infinite or NaN product has no error terms
  return isfinite(v) ? __uint_as_float(bits) : h;
}

// The same to fp32.
__device__ __forceinline__ float turned(float x, float y, float c, float s) { return fmaf(x, c, y * s); }

// cos and sin of a turn in 2^-64, times m: the turn is rounded to 2^-25.
__device__ __forceinline__ float2 turn1(unsigned long long turn, float m) {
  const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;  // in half turns
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * m, s * m);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// ---------------------------------------------------------------------------
// Rotating
// ---------------------------------------------------------------------------
struct View {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
  long long src_batch, src_token, src_head, dst_batch, dst_token, dst_head;  // strides in elements
};

struct RotateParams {
  View q, k;
  const int* positions;     // [B or 1][N], or null: 0 .. N - 1
  const unsigned long long* turns;  // [rot / 2]
  long long position_stride;        // of a batch entry: N, or 0
  int N, Hq, H;             // H = Hq + Hk
  int rot, interleaved, copy_rest;  // copy_rest: elements past rot are written too (not in place)
  int tokens_per_cta;
  float m, sign;            // sign: -1 for the gradient
};

constexpr int kMaxTokens = 16;  // of a CTA

// cos and sin of eight pairs, to turn sixteen elements x, y.
struct Eight {
  float c[8], s[8];
  // HALVES: pair i is element i of x and of y; else elements 2i and 2i + 1 of the two together
  template <bool HALVES>
  __device__ __forceinline__ void turn(uint4& x, uint4& y) const {
    uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const float a0 = bf16_lo(a[n]), a1 = bf16_hi(a[n]), b0 = bf16_lo(b[n]), b1 = bf16_hi(b[n]);
      if constexpr (HALVES) {
        a[n] = pack_bf16x2(turned(a0, -b0, c[2 * n], s[2 * n]), turned(a1, -b1, c[2 * n + 1], s[2 * n + 1]));
        b[n] = pack_bf16x2(turned(b0, a0, c[2 * n], s[2 * n]), turned(b1, a1, c[2 * n + 1], s[2 * n + 1]));
      } else {
        a[n] = pack_bf16x2(turned(a0, -a1, c[n], s[n]), turned(a1, a0, c[n], s[n]));
        b[n] = pack_bf16x2(turned(b0, -b1, c[4 + n], s[4 + n]), turned(b1, b0, c[4 + n], s[4 + n]));
      }
    }
    x = make_uint4(a[0], a[1], a[2], a[3]), y = make_uint4(b[0], b[1], b[2], b[3]);
  }
};

constexpr int kAhead = 4;  // heads whose loads are in flight together

// Block (x, b): tokens_per_cta tokens of batch entry b, all heads.  cos and sin
// of the tokens' pairs go to shared memory once; then a thread has the eight
// pairs of one token to itself and goes through the heads with them in registers,
// two 16-byte loads and stores each (of neighbouring elements if interleaved,
// else rot / 2 apart), four heads' loads in flight.  Bound by the bytes: q and k of
// 4 x 32 heads x 4096 tokens x 128, one direction, 84 us, 6.4 TB/s, 95 % of the
// copy rate (a thread going from head to head with cos and sin read from shared
// memory each time, four ways in conflict: 102 us).  A step of 64 tokens: 2.5 us.
template <int D>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const RotateParams p) {
  __shared__ float2 s_cs[kMaxTokens * (D / 2)];
  const int first = blockIdx.x * p.tokens_per_cta, b = blockIdx.y;
  const int count = min(p.tokens_per_cta, p.N - first);
  const int pairs = p.rot / 2;
  for (int i = threadIdx.x; i < count * pairs; i += kThreads) {
    const int t = i / pairs, pair = i - t * pairs;
    const long long pos = p.positions ? __ldg(p.positions + b * p.position_stride + first + t) : first + t;
    const float2 cs = turn1(static_cast<unsigned long long>(pos) * __ldg(p.turns + pair), p.m);
    s_cs[t * (D / 2) + pair] = make_float2(cs.x, cs.y * p.sign);
  }
  __syncthreads();
  constexpr int kUnits = D / 16;  // of a head
  const int places = p.tokens_per_cta * kUnits;  // a power of two up to kThreads
  const int place = threadIdx.x & (places - 1), group = threadIdx.x / places, groups = kThreads / places;
  const int t = place / kUnits, u = place % kUnits;
  const int rotating = p.rot / 16;
  if (t >= count || (u >= rotating && !p.copy_rest)) return;
  Eight cs;
  if (u < rotating) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = s_cs[t * (D / 2) + 8 * u + i];
      cs.c[i] = f.x, cs.s[i] = f.y;
    }
  }
  const bool halves = u < rotating && !p.interleaved;
  const int e0 = halves ? 8 * u : 16 * u, apart = halves ? pairs : 8;
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const View& v = which ? p.k : p.q;
    const int heads = which ? p.H - p.Hq : p.Hq;
    const __nv_bfloat16* src = v.src + b * v.src_batch + (first + t) * v.src_token + e0;
    __nv_bfloat16* dst = v.dst + b * v.dst_batch + (first + t) * v.dst_token + e0;
#pragma unroll 1
    for (int h = group; h < heads; h += kAhead * groups) {
      uint4 x[kAhead], y[kAhead];
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        if (h + n * groups >= heads) break;
        const __nv_bfloat16* at = src + (h + n * groups) * v.src_head;
        x[n] = *reinterpret_cast<const uint4*>(at);
        y[n] = *reinterpret_cast<const uint4*>(at + apart);
      }
#pragma unroll
      for (int n = 0; n < kAhead; ++n) {
        if (h + n * groups >= heads) break;
        if (halves) cs.turn<true>(x[n], y[n]);
        else if (u < rotating) cs.turn<false>(x[n], y[n]);
        __nv_bfloat16* at = dst + (h + n * groups) * v.dst_head;
        *reinterpret_cast<uint4*>(at) = x[n];
        *reinterpret_cast<uint4*>(at + apart) = y[n];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Appending
// ---------------------------------------------------------------------------
struct AppendParams {
  kv4::MoveParams m;        // as for storing
  const __nv_bfloat16* q;   // [T][Hq][D], token stride below; null where Hq = 0
  __nv_bfloat16* q_out;     // [T][Hq][D], contiguous
  __nv_bfloat16* k_out;     // [T][Hkv][D], contiguous; or null
  const int* positions;     // [T], or null: a token's place in its sequence
  const unsigned long long* turns;
  long long q_stride;
  int Hq, rot, interleaved;
  float scale;              // of cos and sin
};

// A turn's cos and sin in shared memory.  Lanes that read pairs 8 or 16 apart find
// them in other banks.
template <int D>
struct TurnTable {
  static constexpr int kRow = D / 2 + D / 16;
  __device__ static __forceinline__ int at(int t, int pair) { return t * kRow + pair + (pair >> 3); }
};

// Eight elements of a row, w, turned, as four words of bf16; z: their partners (w
// itself where INTERLEAVED), f: their pairs' cos and sin.  x c + sign y s in fp32
// first, which is off by less than 2^-22 m (|x| + |y|), the bound: where both ends
// of that round to the same bf16 value, so does the exact sum.  Two ends in 4000
// do not, and eight elements that have such are taken again with two floats each.
template <bool INTERLEAVED>
__device__ __forceinline__ void turned_eight(const uint32_t* w, const uint32_t* z, float sign, const float4* f, float bound,
                                             uint32_t* out) {
  uint32_t differ = 0;
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const float4 f0 = f[INTERLEAVED ? n : 2 * n], f1 = f[INTERLEAVED ? n : 2 * n + 1];
    const float x0 = bf16_lo(w[n]), x1 = bf16_hi(w[n]);
    const float y0 = INTERLEAVED ? -x1 : bf16_lo(z[n]) * sign, y1 = INTERLEAVED ? x0 : bf16_hi(z[n]) * sign;
    const float v0 = fmaf(x0, f0.x, y0 * f0.z), v1 = fmaf(x1, f1.x, y1 * f1.z);
    const float e0 = (fabsf(x0) + fabsf(y0)) * bound, e1 = (fabsf(x1) + fabsf(y1)) * bound;
    out[n] = pack_bf16x2(v0 - e0, v1 - e1);
    differ |= out[n] ^ pack_bf16x2(v0 + e0, v1 + e1);
  }
  if (differ == 0) return;
#pragma unroll 1
  for (int n = 0; n < 4; ++n) {
    const float4 f0 = f[INTERLEAVED ? n : 2 * n], f1 = f[INTERLEAVED ? n : 2 * n + 1];
    const uint32_t a = n == 0 ? w[0] : n == 1 ? w[1] : n == 2 ? w[2] : w[3];
    const uint32_t b = INTERLEAVED ? a : n == 0 ? z[0] : n == 1 ? z[1] : n == 2 ? z[2] : z[3];
    const float x0 = bf16_lo(a), x1 = bf16_hi(a);
    const float y0 = INTERLEAVED ? -x1 : bf16_lo(b) * sign, y1 = INTERLEAVED ? x0 : bf16_hi(b) * sign;
    const uint32_t r = pack_bf16x2(turned(x0, y0, Float2{f0.x, f0.y}, Float2{f0.z, f0.w}, 1.f),
                                   turned(x1, y1, Float2{f1.x, f1.y}, Float2{f1.z, f1.w}, 1.f));
    if (n == 0) out[0] = r;
    else if (n == 1) out[1] = r;
    else if (n == 2) out[2] = r;
    else out[3] = r;
  }
}

// Elements 8 e .. 8 e + 7 of a head's row `src`, turned, as four words of bf16.
template <int D>
__device__ __forceinline__ void turned_vector(const __nv_bfloat16* src, int e, const AppendParams& p, const float4* s_turn,
                                              int t, uint32_t* out) {
  const int e0 = 8 * e, half = p.rot / 2;
  const uint4 x4 = __ldg(reinterpret_cast<const uint4*>(src + e0));
  const uint32_t w[4] = {x4.x, x4.y, x4.z, x4.w};
  const float bound = p.scale * 0x1p-22f;
  if (e0 >= p.rot) {
#pragma unroll
    for (int n = 0; n < 4; ++n) out[n] = w[n];
  } else if (p.interleaved) {
    turned_eight<true>(w, w, 1.f, s_turn + TurnTable<D>::at(t, e0 / 2), bound, out);
  } else {
    const bool upper = e0 >= half;
    const uint4 y4 = __ldg(reinterpret_cast<const uint4*>(src + (upper ? e0 - half : e0 + half)));
    const uint32_t z[4] = {y4.x, y4.y, y4.z, y4.w};
    turned_eight<false>(w, z, upper ? 1.f : -1.f, s_turn + TurnTable<D>::at(t, upper ? e0 - half : e0), bound, out);
  }
}

// As storing (kv4::store_kernel), with the keys' blocks turned first, and q
// turned as by rotate_kernel before them.  79063 tokens of 32 and 8 heads, d = 128:
// 1.71 GB, 293 us, 5.8 TB/s, 86 % of the copy rate, at 59 % of the issue slots (64
// registers a thread: 293 us; 80, three CTAs an SM: 323; every key element with two
// floats each, without the bound's test: 340).
template <int D>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendParams p) {
  using kv4::kBlock;
  using kv4::kGroup;
  constexpr int kBlocks = D / kBlock;
  const kv4::MoveParams& m = p.m;
  __shared__ int s_cu[kv4::kCuCached];
  __shared__ long long s_place[kv4::kMaxTokensPerCta], s_at[kv4::kMaxTokensPerCta];
  __shared__ float4 s_turn[kv4::kMaxTokensPerCta * TurnTable<D>::kRow];
  const int first = blockIdx.x * m.tokens_per_cta;
  const int count = min(m.tokens_per_cta, m.T - first);
  const bool cached = m.n_seqs < kv4::kCuCached;
  if (cached) {
    for (int i = threadIdx.x; i <= m.n_seqs; i += kThreads) s_cu[i] = m.cu[i];
    __syncthreads();
  }
  if (threadIdx.x < count) {
    const int tok = first + threadIdx.x;
    long long at = 0;
    s_place[threadIdx.x] = cached ? kv4::place_of(tok, D, m, [&](int i) { return s_cu[i]; }, &at)
                                  : kv4::place_of(tok, D, m, [&](int i) { return __ldg(m.cu + i); }, &at);
    s_at[threadIdx.x] = p.positions ? __ldg(p.positions + tok) : at;
  }
  __syncthreads();
  const int pairs = p.rot / 2;
  for (int i = threadIdx.x; i < count * pairs; i += kThreads) {
    const int t = i / pairs, pair = i - t * pairs;
    const Turn2 turn(static_cast<unsigned long long>(s_at[t]) * __ldg(p.turns + pair), p.scale);
    s_turn[TurnTable<D>::at(t, pair)] = make_float4(turn.c.hi, turn.c.lo, turn.s.hi, turn.s.lo);
  }
  __syncthreads();
  // q: as in rotate_kernel
  if (p.Hq > 0) {
    const int places = m.tokens_per_cta * kBlocks;
    const int place = threadIdx.x & (places - 1), group = threadIdx.x / places, groups = kThreads / places;
    const int i = place / kBlocks, u = place % kBlocks;
    if (i < count && s_place[i] != -1) {
      const bool turning = 16 * u < p.rot, halves = turning && !p.interleaved;
      Eight cs;
      if (turning) {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float4 f = s_turn[TurnTable<D>::at(i, 8 * u + n)];
          cs.c[n] = f.x, cs.s[n] = f.z;
        }
      }
      const int e0 = halves ? 8 * u : 16 * u, apart = halves ? pairs : 8;
      const long long tok = first + i;
      const __nv_bfloat16* src = p.q + tok * p.q_stride + e0;
      __nv_bfloat16* dst = p.q_out + tok * p.Hq * D + e0;
#pragma unroll 1
      for (int h = group; h < p.Hq; h += kAhead * groups) {
        uint4 x[kAhead], y[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          if (h + n * groups >= p.Hq) break;
          x[n] = __ldg(reinterpret_cast<const uint4*>(src + (h + n * groups) * D));
          y[n] = __ldg(reinterpret_cast<const uint4*>(src + (h + n * groups) * D + apart));
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
          if (h + n * groups >= p.Hq) break;
          if (halves) cs.turn<true>(x[n], y[n]);
          else if (turning) cs.turn<false>(x[n], y[n]);
          *reinterpret_cast<uint4*>(dst + (h + n * groups) * D) = x[n];
          *reinterpret_cast<uint4*>(dst + (h + n * groups) * D + apart) = y[n];
        }
      }
    }
  }
  const int units = 2 * m.Hkv * count * kBlocks;  // [tensor][head][token][block]
  const int head_bytes = kv4::row_bytes(D) << m.page_shift;
  for (int u = threadIdx.x; u < units; u += kThreads) {
    const int block = u % kBlocks, rest = u / kBlocks;
    const int i = rest % count, hv = rest / count;
    const long long place = s_place[i];
    if (place == -1) continue;  // of no sequence
    const long long tok = first + i;
    const int is_v = hv >= m.Hkv;
    const int h = is_v ? hv - m.Hkv : hv;
    uint32_t w[8];
    if (is_v) {
      const uint4* src = reinterpret_cast<const uint4*>(m.v + tok * m.v_stride + static_cast<long long>(h) * D + block * kBlock);
      const uint4 a = __ldg(src), b = __ldg(src + 1);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      const __nv_bfloat16* src = m.k + tok * m.k_stride + static_cast<long long>(h) * D;
      turned_vector<D>(src, 2 * block, p, s_turn, i, w);
      turned_vector<D>(src, 2 * block + 1, p, s_turn, i, w + 4);
      if (p.k_out) {
        uint4* dst = reinterpret_cast<uint4*>(p.k_out + (tok * m.Hkv + h) * D + block * kBlock);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    if (place < 0) continue;  // refused: not stored
    const int row = static_cast<int>(place & (kGroup - 1));
    uint32_t codes[2], scale;
    kv4::quantise_block(w, is_v ? m.v_scale : m.k_scale, codes, scale);
    uint8_t* group = m.cache + (place - row) + static_cast<long long>(h) * head_bytes;
    *reinterpret_cast<uint2*>(group + kv4::codes_at(D, is_v) + row * (D / 2) + block * 8) = make_uint2(codes[0], codes[1]);
    group[kv4::scales_at(D, is_v) + row * kBlocks + block] = static_cast<uint8_t>(scale);
  }
}

}  // namespace rotary
}  // namespace fa
