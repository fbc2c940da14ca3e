// Verification of a tree of drafted tokens against the target's probabilities.
//
// One cluster of CTAs walks one sequence's tree.  At node c, with logits l over
// V tokens, M = max l and w(x) = exp((l(x) - M) / temperature), the target is p =
// w / sum w.  Child j with token x, drawn from q, is accepted where u_j q(x)
// T < a(x), a being what is left of w and T its sum: a = w at first, and after a
// child that is not accepted
//
//     a <- max(0, a - q T),   T <- sum a,
//
// which is max(r - q, 0) normalised, r = a / T.  A node's children are drawn from one
// q, so after several a = max(0, w - q S) with S the sum of their T.  A token given (no
// q) loses its w.  The next token is the first x where a(0) + ... + a(x) > u_0 T.
//
// A running sum over 10^5 tokens meets u_0 T next to some token's border all
// the time: with sums and exponentials in fp32 one call in a hundred would give
// another token than the same sums in 64 bits do.  So each w is computed as a sum
// of two floats (relative error below 2^-29: table-driven, 128 entries and a short
// polynomial) and rounded to a multiple of 2^-44; sums of those are 64-bit integers,
// exact, and the same however the row is cut.
//
// Whether a child is accepted is one comparison, for which a T right to 2^-16 is
// enough but for one child in ten thousand or so: a node's first child is judged by a
// T from one quick pass over the row, fp32 exponentials against running maxima,
// which finds M, too.  Where that child is surely accepted nothing more is asked of the
// row; where it is not sure, the exact T is.
//
// Work: a quick pass a node; where its first child is not accepted, or there is
// none, a pass for the exact T, and one more for each drawn child that is not
// accepted.  CTA r of the cluster takes the r-th part of the row's tiles of 256
// tokens, a warp a tile at a time, a lane eight tokens, and every CTA takes every
// decision from the same numbers, which the CTAs store to one another's shared memory
// once all have started.  Tiles' sums stay in shared memory, so that the
// token is found by looking at one tile again.
//
// Measured on a GB300: 48 sequences' trees of 24 drawn nodes, 128000 tokens in fp32,
// 75 to 76 us; the 96 MB of rows that are visited (3.3 a sequence, and the draft's where a
// child is refused) would take 14 at the copy rate.  A quick pass is some 15
// instructions a token, an exact one 50 with its loads and sums; a sequence's passes
// (5.6 on average, 10 at the most) follow one another, 7 of them in 30 us on an idle
// card, where each waits for its first loads, two reductions and the cluster's
// barrier.  All 48 together use 43 % of the issue slots while an SM has work.  One tree
// of 16 nodes, 32000 tokens in bf16: 12.3 us (6.0 at temperature 0).  What the steps brought at 48 sequences:
// exact weights of 60 instructions, right to 2^-40, 111 us; 30, 93; one product with
// q for all refused children, and fewer registers, 80; the quick pass's running
// maximum without a branch 75.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "sm103_ptx.cuh"

namespace fa {
namespace verify {

constexpr int kThreads = 256, kWarps = kThreads / 32;  // of a CTA, at most
constexpr int kCtasPerSm = 4;
constexpr int kMaxNodes = 64;
constexpr int kMaxVocab = 1 << 18;
constexpr int kTile = 256;                        // tokens of a warp's step
constexpr int kMaxTiles = kMaxVocab / kTile + 1;  // of a row that starts within a tile
constexpr int kMaxCluster = 16;  // (more than 8 has to be asked for)
// What the quick pass's sum may be off by, of it, twice over, where a lane takes `tiles` tiles.  A
// weight is a power of two right to 2^-22 and is brought to a later maximum by at most `tiles`
// products with such powers in the lane, each rounded to 2^-24, and three in the reductions;
// a sum has 4 additions of a tile, one a tile and 15 of the reductions; the powers' arguments are right
// to 2^-22.4 of themselves (17 where all tokens of a row lie there: 36 in 2^-24).  In 2^-24 that is
// 5 (tiles + 4) + tiles + 19 + 36.  Up to 30 tiles it is 2^-15 at the most: clusters of 16 take 17.
__host__ __device__ constexpr float quick_bound(int tiles) {
  return 6 * tiles + 75 <= 256 ? 0x1p-15f : static_cast<float>(6 * tiles + 75) * 0x1p-23f;
}
// The most tiles of a lane of `warps` warps in each of `ctas`, wherever in a tile the row starts.
__host__ __device__ constexpr int lane_tiles(int V, int ctas, int warps) {
  const int tiles = (V + 7 + kTile - 1) / kTile, per = (tiles + ctas - 1) / ctas;
  return (per + warps - 1) / warps;
}
constexpr float kSpan = 64.f;                     // powers of two below the maximum; what lies further is taken as 2^-64, which is rounded to 0
constexpr float kFar = 16384.f;                   // of the maximum's power of two: above it, differences from it are taken first

// 2^(k / 128) as a sum of two floats.
__device__ const float2 kExp2[128] = {
    {0x1p+0f, 0x0p+0f}, {0x1.0163dap+0f, 0x1.3f6666p-25f}, {0x1.02c9a4p+0f, -0x1.887fap-28f},
    {0x1.04315ep+0f, 0x1.0dcffp-25f}, {0x1.059b0ep+0f, -0x1.9d4f52p-25f}, {0x1.0706b2p+0f, 0x1.3bbedcp-25f},
    {0x1.087452p+0f, -0x1.e2990ep-26f}, {0x1.09e3ecp+0f, 0x1.58de7p-25f}, {0x1.0b5586p+0f, 0x1.9f3122p-25f},
    {0x1.0cc922p+0f, 0x1.6e48fep-25f}, {0x1.0e3ec4p+0f, -0x1.a585ccp-25f}, {0x1.0fb66ap+0f, 0x1.ffda64p-25f},
    {0x1.11301ep+0f, -0x1.fdb496p-25f}, {0x1.12abdcp+0f, 0x1.b0c73p-30f}, {0x1.1429aap+0f, 0x1.d525bcp-25f},
    {0x1.15a98cp+0f, 0x1.14b1cap-25f}, {0x1.172b84p+0f, -0x1.c15742p-27f}, {0x1.18af94p+0f, -0x1.dcdc86p-26f},
    {0x1.1a35bep+0f, 0x1.6df96ep-25f}, {0x1.1bbe08p+0f, 0x1.011734p-26f}, {0x1.1d4874p+0f, -0x1.d2e8cap-25f},
    {0x1.1ed502p+0f, 0x1.7e6c8ep-27f}, {0x1.2063b8p+0f, 0x1.0c519ap-25f}, {0x1.21f49ap+0f, -0x1.d0446ep-25f},
    {0x1.2387a6p+0f, 0x1.ceac48p-25f}, {0x1.251ce4p+0f, 0x1.f654c8p-25f}, {0x1.26b456p+0f, 0x1.789f38p-26f},
    {0x1.284dfep+0f, 0x1.f5638p-28f}, {0x1.29e9ep+0f, -0x1.5c0424p-25f}, {0x1.2b87fep+0f, -0x1.e4a4cep-25f},
    {0x1.2d285ap+0f, 0x1.b900c2p-26f}, {0x1.2ecafap+0f, 0x1.27c5eap-25f}, {0x1.306fep+0f, 0x1.4636e2p-25f},
    {0x1.32171p+0f, -0x1.d993e8p-27f}, {0x1.33c08cp+0f, -0x1.b37d2p-25f}, {0x1.356c56p+0f, -0x1.b5803cp-30f},
    {0x1.371a74p+0f, -0x1.18aac6p-25f}, {0x1.38cae6p+0f, 0x1.a0bb0cp-25f}, {0x1.3a7db4p+0f, -0x1.634c02p-25f},
    {0x1.3c32dcp+0f, 0x1.89d472p-27f}, {0x1.3dea64p+0f, 0x1.824684p-25f}, {0x1.3fa45p+0f, 0x1.2b2006p-26f},
    {0x1.4160a2p+0f, 0x1.f72e2ap-28f}, {0x1.431f5ep+0f, -0x1.abd5dap-26f}, {0x1.44e086p+0f, 0x1.8624b4p-30f},
    {0x1.46a41ep+0f, 0x1.a3a00ap-25f}, {0x1.486a2cp+0f, -0x1.47d866p-25f}, {0x1.4a32bp+0f, -0x1.e50584p-25f},
    {0x1.4bfdaep+0f, -0x1.593abcp-25f}, {0x1.4dcb2ap+0f, -0x1.8088bcp-26f}, {0x1.4f9b28p+0f, -0x1.2c5a6cp-25f},
    {0x1.516daap+0f, 0x1.67b32p-27f}, {0x1.5342b6p+0f, -0x1.2c561p-25f}, {0x1.551a4cp+0f, 0x1.4bb242p-25f},
    {0x1.56f474p+0f, -0x1.295b04p-25f}, {0x1.58d12ep+0f, -0x1.6d07p-25f}, {0x1.5ab07ep+0f, -0x1.5bd5ecp-27f},
    {0x1.5c9268p+0f, 0x1.4b28d6p-25f}, {0x1.5e76f2p+0f, -0x1.4a5bd6p-25f}, {0x1.605e1cp+0f, -0x1.a248fep-26f},
    {0x1.6247ecp+0f, -0x1.f8b55p-25f}, {0x1.643464p+0f, -0x1.66679cp-25f}, {0x1.662388p+0f, 0x1.2a9112p-27f},
    {0x1.68155ep+0f, -0x1.766ad2p-25f}, {0x1.6a09e6p+0f, 0x1.9fcef4p-26f}, {0x1.6c0128p+0f, -0x1.5e84a8p-25f},
    {0x1.6dfb24p+0f, -0x1.cd72e8p-27f}, {0x1.6ff7ep+0f, -0x1.ab9aep-26f}, {0x1.71f75ep+0f, 0x1.1d8beep-25f},
    {0x1.73f9a4p+0f, 0x1.14b02ep-25f}, {0x1.75feb6p+0f, -0x1.37b306p-25f}, {0x1.780694p+0f, 0x1.fbcba8p-25f},
    {0x1.7a1148p+0f, -0x1.829fdp-25f}, {0x1.7c1edp+0f, 0x1.30c132p-28f}, {0x1.7e2f34p+0f, -0x1.261634p-25f},
    {0x1.804276p+0f, -0x1.783cbep-25f}, {0x1.82589ap+0f, -0x1.accc7cp-26f}, {0x1.8471a4p+0f, 0x1.88f1ecp-26f},
    {0x1.868d9ap+0f, -0x1.2edb44p-26f}, {0x1.88ac7ep+0f, -0x1.9d665ap-26f}, {0x1.8ace54p+0f, 0x1.15506ep-27f},
    {0x1.8cf322p+0f, -0x1.29576ep-25f}, {0x1.8f1aeap+0f, -0x1.baa232p-26f}, {0x1.9145bp+0f, 0x1.723ff8p-25f},
    {0x1.93737cp+0f, -0x1.e64744p-25f}, {0x1.95a44cp+0f, 0x1.790a42p-25f}, {0x1.97d82ap+0f, -0x1.0d8d84p-31f},
    {0x1.9a0f18p+0f, -0x1.e6bf08p-25f}, {0x1.9c4918p+0f, 0x1.51f848p-27f}, {0x1.9e8632p+0f, -0x1.873738p-26f},
    {0x1.a0c668p+0f, -0x1.2886a6p-26f}, {0x1.a309bep+0f, 0x1.8945a6p-25f}, {0x1.a5503cp+0f, -0x1.b83b54p-25f},
    {0x1.a799e2p+0f, -0x1.99e994p-25f}, {0x1.a9e6b6p+0f, -0x1.50c048p-25f}, {0x1.ac36bcp+0f, -0x1.606432p-31f},
    {0x1.ae89fap+0f, -0x1.a94b14p-26f}, {0x1.b0e072p+0f, 0x1.31b6ccp-25f}, {0x1.b33a2cp+0f, -0x1.ec3a82p-26f},
    {0x1.b59728p+0f, 0x1.bcab28p-25f}, {0x1.b7f77p+0f, -0x1.a09438p-25f}, {0x1.ba5b04p+0f, -0x1.ebdf36p-25f},
    {0x1.bcc1eap+0f, -0x1.f687c6p-25f}, {0x1.bf2c26p+0f, -0x1.0a387ep-26f}, {0x1.c199bep+0f, -0x1.3d56b2p-27f},
    {0x1.c40ab6p+0f, -0x1.7c2c98p-39f}, {0x1.c67f12p+0f, 0x1.cafa2ap-25f}, {0x1.c8f6dap+0f, -0x1.7f230ap-25f},
    {0x1.cb720ep+0f, -0x1.8837ccp-27f}, {0x1.cdf0b6p+0f, -0x1.54478p-25f}, {0x1.d072d4p+0f, 0x1.40f13p-25f},
    {0x1.d2f87p+0f, 0x1.01b13ep-25f}, {0x1.d5818ep+0f, -0x1.822dbcp-27f}, {0x1.d80e32p+0f, -0x1.26cf8ep-25f},
    {0x1.da9e6p+0f, 0x1.ed9942p-27f}, {0x1.dd322p+0f, -0x1.9fc974p-25f}, {0x1.dfc974p+0f, -0x1.908c94p-25f},
    {0x1.e26462p+0f, -0x1.614bdap-25f}, {0x1.e502eep+0f, 0x1.e2cffep-26f}, {0x1.e7a52p+0f, -0x1.0e2cep-26f},
    {0x1.ea4afap+0f, 0x1.52486cp-27f}, {0x1.ecf482p+0f, 0x1.b1ccfep-25f}, {0x1.efa1bep+0f, 0x1.cc2b44p-25f},
    {0x1.f252b4p+0f, -0x1.1288aep-25f}, {0x1.f50766p+0f, -0x1.246ebp-26f}, {0x1.f7bfdap+0f, 0x1.b397c2p-25f},
    {0x1.fa7c18p+0f, 0x1.9e90d8p-28f}, {0x1.fd3c22p+0f, 0x1.71ee3ep-25f},
};

struct Params {
  const void* logits;
  const int* tokens;
  const int* parents;
  const float* uniforms;
  const float* draft;
  int* path;
  int* n_kept;
  int* next_token;
  int n_nodes, V;
  long long logits_stride, draft_stride;
  float c_hi, c_lo;  // log2(e) / temperature
  float span;        // kSpan of those
  float quick;       // quick_bound of the tiles that a lane takes
  int greedy;        // temperature 0
};

struct Pair {  // hi + lo
  float hi, lo;
};

__device__ __forceinline__ Pair quick_sum(float a, float b) {  // |a| >= |b|, or a = 0 = b
  const float s = __fadd_rn(a, b);
  return Pair{s, __fsub_rn(b, __fsub_rn(s, a))};
}

// What a row's weights are taken against: its maximum M.
struct Reference {
  float shift, low, top;  // tokens are taken as x - shift, from low (NaN, too) to top
  int n;                // M's power of two in 128ths: bits of n / 128 + kRound
  float rest;           // and what is left of it
};

// t + kRound is t to the nearest 128th (|t| < 2^15), which is exact.
constexpr float kRound = 98304.f;  // 1.5 * 2^16

// Far from 0 the difference to M is exact for every token that counts, near 0 it is not needed.
__device__ __forceinline__ Reference reference(float M, const Params& p) {
  Reference r;
  r.shift = fabsf(M) * p.c_hi > kFar ? M : 0.f;
  const float x = r.top = M - r.shift;
  r.low = x - p.span;
  const float t = __fmaf_rn(x, p.c_hi, kRound);
  r.n = __float_as_int(t);
  r.rest = __fmaf_rn(x, p.c_lo, __fmaf_rn(x, p.c_hi, -__fsub_rn(t, kRound)));
  return r;
}

// (x + lo) scale
struct Weight {
  float x, lo, scale;
  __device__ __forceinline__ Pair pair() const { return Pair{x * scale, lo * scale}; }
};

// exp((x - M) / temperature): with d a token's difference to the shift, d c = t + r
// for t a multiple of 1 / 128 and |r| <= 2^-8, one fused product; 2^(t - M's) from the
// table; e^(y ln 2) - 1 for y = r - M's rest by a polynomial, which leaves out less than
// 2^-45.  Off by less than 2^-29 of the weight: roundings of 2^-32 of y, of the
// polynomial's value and of its product with the table's (2^-29.7 at the most in 8
// million values against 64 bits).
__device__ __forceinline__ Weight weight(float x, const Reference& ref, const Params& p, const float2* table) {
  const float d = fminf(fmaxf(__fsub_rn(x, ref.shift), ref.low), ref.top);
  const float t = __fmaf_rn(d, p.c_hi, kRound);
  const float r = __fmaf_rn(d, p.c_hi, -__fsub_rn(t, kRound));
  const float y = __fadd_rn(r, __fmaf_rn(d, p.c_lo, -ref.rest));
  constexpr float kLn2 = 0.693147180559945f;
  const float e = __fmaf_rn(y, kLn2, __fmul_rn(__fmul_rn(y, y), __fmaf_rn(y, __fmaf_rn(y, kLn2 * kLn2 * kLn2 * kLn2 / 24,
                                                                             kLn2 * kLn2 * kLn2 / 6), kLn2 * kLn2 / 2)));
  const int k = __float_as_int(t) - ref.n;  // in 128ths: 0 down to -64 * 128
  const float2 v = table[k & 127];
  return Weight{v.x, __fmaf_rn(v.x, e, v.y), __int_as_float((k & ~127) * 65536 + 0x3f800000)};
}

// A drawn child's own, which is compared without rounding it to 2^-44: what lies further
// below M than `low` is itself, to about 2^-16, and not 2^-64; -inf (and NaN) is 0.
__device__ __forceinline__ Pair own_weight(float x, const Reference& ref, const Params& p, const float2* table) {
  const float d = __fsub_rn(fmaxf(x, -INFINITY), ref.shift);
  if (!(d < ref.low)) return weight(x, ref, p, table).pair();
  return Pair{ex2_approx(__fsub_rn(d, ref.top) * p.c_hi), 0.f};
}

// a - q S, at least 0, for S as a sum of two floats.
__device__ __forceinline__ Pair without(const Pair& a, float q, const float2& S) {
  const float h = __fmul_rn(q, S.x);
  const float more = __fmaf_rn(q, S.y, __fmaf_rn(q, S.x, -h));
  const float d = __fsub_rn(a.hi, h), err = __fsub_rn(__fsub_rn(a.hi, d), h);  // exact where something is left
  const Pair v = quick_sum(d, __fadd_rn(err, __fsub_rn(a.lo, more)));
  return v.hi > 0.f ? v : Pair{0.f, 0.f};  // not where it is NaN
}

// A value from 0 to 1 to a multiple of 2^-44: first to 2^-22, in those, then the
// rest.  256 tokens' parts can be summed in 32 bits each.
struct Fixed {
  int hi, lo;
  __device__ __forceinline__ long long value() const { return (static_cast<long long>(hi) << 22) + lo; }
};
__device__ __forceinline__ Fixed fixed44(const Weight& w) {
  constexpr float kHi = 3.f;           // sums near it are multiples of 2^-22
  constexpr float kLo = 0x1.8p-21f;    // of 2^-44
  const float h = __fmaf_rn(__fadd_rn(w.x, w.lo), w.scale, kHi);
  const float rest = __fmaf_rn(w.lo, w.scale, __fmaf_rn(w.x, w.scale, -__fsub_rn(h, kHi)));
  return Fixed{__float_as_int(h) - __float_as_int(kHi), __float_as_int(__fadd_rn(rest, kLo)) - __float_as_int(kLo)};
}
__device__ __forceinline__ Fixed fixed44(const Pair& a) { return fixed44(Weight{a.hi, a.lo, 1.f}); }

__device__ __forceinline__ float2 from_fixed44(long long T) {
  const float hi = __ll2float_rz(T);
  return make_float2(hi * 0x1p-44f, __ll2float_rn(T - static_cast<long long>(hi)) * 0x1p-44f);
}

// Of two positive sums of two floats.
__device__ __forceinline__ float2 plus(const float2& a, const float2& b) {
  const bool more = a.x >= b.x;
  const Pair s = quick_sum(more ? a.x : b.x, more ? b.x : a.x);
  const Pair v = quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.y, b.y)));
  return make_float2(v.hi, v.lo);
}

// u to 64 fractional bits, from [0, 1); anything else is taken as an end of it.
__device__ __forceinline__ unsigned long long fraction64(float u) {
  if (!(u > 0.f)) return 0ull;
  if (u >= 1.f) return ~0ull;
  return __float2ull_rd(u * 0x1p40f) << 24 | __float2ull_rd((u * 0x1p40f - __ull2float_rz(__float2ull_rd(u * 0x1p40f))) * 0x1p24f);
}

// NaN counts as -inf (a maximum takes the other operand), +inf as the largest finite value.
__device__ __forceinline__ float usable(float x) { return fminf(fmaxf(x, -INFINITY), 3.40282347e38f); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Another CTA's shared memory is there once that CTA has started, and until it ends.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  cluster_wait();
}
// A 64-bit store to the same place in CTA `rank`'s shared memory.
__device__ __forceinline__ void store_to(uint32_t rank, void* where, long long v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(where)), "r"(rank));
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// One CTA's part of one row: tokens tile * 256 - shift ..., tiles [begin, end).
// The shift puts every lane's eight tokens on a boundary for wide loads.
template <bool FP32>
struct Row {
  const __nv_bfloat16* b;
  const float* f;
  const float* q;  // the draft's row, or null
  int V, shift, begin, end, per;

  __device__ __forceinline__ Row(const Params& p, long long row, uint32_t rank, uint32_t size) {
    V = p.V;
    b = static_cast<const __nv_bfloat16*>(p.logits) + (FP32 ? 0 : row * p.logits_stride);
    f = static_cast<const float*>(p.logits) + (FP32 ? row * p.logits_stride : 0);
    q = p.draft ? p.draft + row * p.draft_stride : nullptr;
    shift = static_cast<int>(FP32 ? reinterpret_cast<uintptr_t>(f) / 4 : reinterpret_cast<uintptr_t>(b) / 2) & 7;
    const int tiles = (V + shift + kTile - 1) / kTile;
    per = (tiles + static_cast<int>(size) - 1) / static_cast<int>(size);
    begin = min(tiles, static_cast<int>(rank) * per);
    end = min(tiles, begin + per);
  }
  __device__ __forceinline__ int first(int tile) const { return tile * kTile - shift + static_cast<int>(threadIdx.x & 31) * 8; }
  __device__ __forceinline__ float at(int x) const { return FP32 ? __ldg(f + x) : __bfloat162float(b[x]); }
  // Tokens x .. x + 7, as they are; -inf outside the row.
  __device__ __forceinline__ void load(int x, float* v) const {
    if (x >= 0 && x + 8 <= V) {
      if constexpr (FP32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(f + x)), c = __ldg(reinterpret_cast<const float4*>(f + x) + 1);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = c.x, v[5] = c.y, v[6] = c.z, v[7] = c.w;
      } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(b + x));
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x + i >= 0 && x + i < V ? at(x + i) : -INFINITY;
    }
  }
  // Tokens x .. x + 3, and the draft's.
  __device__ __forceinline__ void load4(int x, float* v) const {
    if (x >= 0 && x + 4 <= V) {
      if constexpr (FP32) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(f + x));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(b + x));
        v[0] = __uint_as_float(a.x << 16), v[1] = __uint_as_float(a.x & 0xffff0000u);
        v[2] = __uint_as_float(a.y << 16), v[3] = __uint_as_float(a.y & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x + i >= 0 && x + i < V ? at(x + i) : -INFINITY;
    }
  }
  __device__ __forceinline__ void load4_draft(int x, float* v) const {
    if (x >= 0 && x + 4 <= V && (reinterpret_cast<uintptr_t>(q + x) & 15) == 0) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(q + x));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = x + i >= 0 && x + i < V ? __ldg(q + x + i) : 0.f;
    }
  }
};

// A maximum, the lowest token that has it, and the sum of weights against it.
struct Top {
  float max;
  int token;
  float sum;
};

struct Shared {
  float2 table[128];
  long long tile[kMaxTiles];       // this CTA's tiles' sums
  long long gather[2][2][kMaxCluster];  // [exchange, by turns][value]; after row_sum each CTA's sum
  long long warp[2][kWarps];       // [exchange]
  Top tops[kWarps];
  int parents[kMaxNodes], tokens[kMaxNodes], gone[kMaxNodes];
  float u[kMaxNodes], logit[kMaxNodes], draft[kMaxNodes];  // of the node's children: at their tokens
};

// Every CTA's two values to every CTA, in gather[phase]; whole CTA.  A buffer is
// written again after the barrier of the exchange between, which every CTA
// enters only when it is done reading this one.
__device__ __forceinline__ void exchange(long long v, long long w, Shared& s, int& phase, uint32_t rank, uint32_t size) {
  phase ^= 1;
  if (size == 1) {
    if (threadIdx.x < 2) s.gather[phase][threadIdx.x][0] = threadIdx.x ? w : v;
    __syncthreads();
    return;
  }
  if (threadIdx.x < 2 * size) {
    const uint32_t to = threadIdx.x >> 1, which = threadIdx.x & 1;
    store_to(to, &s.gather[phase][which][rank], which ? w : v);
  }
  cluster_sync();
}

// The lanes' Tops as one, the same in every lane (and in every warp that has the same lanes).
__device__ __forceinline__ Top join(const Top& mine, float c) {
  // the value's bits made monotonic (-0 as 0)
  const uint32_t b = __float_as_uint(mine.max + 0.f);
  const uint32_t top = __reduce_max_sync(0xffffffffu, b & 0x80000000u ? ~b : b | 0x80000000u);
  Top all;
  all.max = __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
  all.token = __reduce_min_sync(0xffffffffu, mine.max == all.max ? mine.token : 0x7fffffff);
  all.sum = mine.sum == 0.f ? 0.f : mine.sum * ex2_approx((mine.max - all.max) * c);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) all.sum += __shfl_xor_sync(0xffffffffu, all.sum, off);
  return all;
}

// The quick pass: the row's maximum, and the lowest token that has it where greedy,
// else the sum of the row's weights (quick_bound).  `first`: the kernel's first pass, whose
// exchange waits for the cluster's CTAs to have started, which the pass hides.
template <bool FP32>
__device__ __forceinline__ Top row_quick(const Row<FP32>& row, const Params& p, Shared& s, int& phase, uint32_t rank,
                                         uint32_t size, bool first) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  constexpr int kAtOnce = 2;  // tiles whose loads are in flight together
  float best = -INFINITY, sum = 0.f;  // the sum against `best`
  int where = 0x7fffffff;
#pragma unroll 1
  for (int t = row.begin + warp; t < row.end; t += kAtOnce * warps) {
    float v[kAtOnce][8];
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      if (t + n * warps < row.end) {
        row.load(row.first(t + n * warps), v[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[n][i] = usable(v[n][i]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[n][i] = -INFINITY;
      }
    }
#pragma unroll
    for (int n = 0; n < kAtOnce; ++n) {
      float top = fmax3(v[n][0], v[n][1], v[n][2]);
      top = fmax3(top, v[n][3], v[n][4]);
      top = fmax3(top, v[n][5], v[n][6]);
      top = fmaxf(top, v[n][7]);
      if (p.greedy) {
        if (top > best) {  // ascending tokens: the first of equals stays
          best = top;
          const int x = row.first(t + n * warps);
#pragma unroll
          for (int i = 7; i >= 0; --i)
            if (v[n][i] == top) where = x + i;
        }
      } else {
        // no branch: one of a warp's lanes has a new maximum nearly every time
        const float now = fmaxf(best, top), shift = now == -INFINITY ? 0.f : now;
        sum *= ex2_approx((best - shift) * p.c_hi);
        best = now;
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          a += ex2_approx((v[n][i] - shift) * p.c_hi);
          b += ex2_approx((v[n][i + 1] - shift) * p.c_hi);
        }
        sum += a + b;
      }
    }
  }
  // the warp's, the CTA's, the cluster's
  const Top none{-INFINITY, 0x7fffffff, 0.f};
  const float c = p.greedy ? 0.f : p.c_hi;
  Top top = join(Top{best, where, sum}, c);
  if (lane == 0) s.tops[warp] = top;
  __syncthreads();
  top = join(lane < warps ? s.tops[lane] : none, c);
  if (first && size > 1) cluster_wait();
  exchange(static_cast<long long>(static_cast<unsigned long long>(__float_as_uint(top.max)) << 32 | static_cast<uint32_t>(top.token)),
           __float_as_uint(top.sum), s, phase, rank, size);
  top = none;
  if (lane < size) {
    const unsigned long long v = static_cast<unsigned long long>(s.gather[phase][0][lane]);
    top = Top{__uint_as_float(static_cast<uint32_t>(v >> 32)), static_cast<int>(v & 0xffffffffu),
              __uint_as_float(static_cast<uint32_t>(s.gather[phase][1][lane]))};
  }
  return join(top, c);
}

// What is left of the weights of tokens x .. x + 3: less q S where `drawn`, less `gone` given ones.
template <bool FP32>
__device__ __forceinline__ void left4(const Row<FP32>& row, int x, const Reference& ref, bool drawn, const float2& S, int gone,
                                      const Params& p, const Shared& s, Fixed* out) {
  float v[4], q[4];
  row.load4(x, v);
  if (!drawn) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = fixed44(weight(v[i], ref, p, s.table));
  } else {
    row.load4_draft(x, q);
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = fixed44(without(weight(v[i], ref, p, s.table).pair(), q[i], S));
  }
#pragma unroll 1
  for (int n = 0; n < gone; ++n) {
    const int i = s.gone[n] - x;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i == e) out[e] = Fixed{0, 0};
  }
}

// The sums of what is left: tiles', CTAs' and, returned, the row's.
template <bool FP32>
__device__ __forceinline__ long long row_sum(const Row<FP32>& row, const Reference& ref, bool drawn, const float2& S, const Params& p, Shared& s, int& phase,
                                             uint32_t rank, uint32_t size) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  long long mine = 0;
  for (int t = row.begin + warp; t < row.end; t += warps) {
    Fixed part{0, 0};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      Fixed w[4];
      left4(row, row.first(t) + 4 * half, ref, drawn, S, 0, p, s, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) part.hi += w[i].hi, part.lo += w[i].lo;
    }
    part.hi = __reduce_add_sync(0xffffffffu, part.hi);
    part.lo = __reduce_add_sync(0xffffffffu, part.lo);
    const long long sum = part.value();
    if (lane == 0) s.tile[t - row.begin] = sum;
    mine += sum;
  }
  if (lane == 0) s.warp[phase ^ 1][warp] = mine;
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < warps; ++w) total += s.warp[phase ^ 1][w];
  exchange(total, 0, s, phase, rank, size);
  total = 0;
  for (uint32_t r = 0; r < size; ++r) total += s.gather[phase][0][r];
  return total;
}

// The first token whose running sum exceeds `target` (below the sum of all), by
// the CTA whose part it is in.
template <bool FP32>
__device__ __forceinline__ void find_token(const Row<FP32>& row, long long target, const Reference& ref, bool drawn, const float2& S, int gone, const Params& p,
                                           const Shared& s, int phase, uint32_t rank, int* where) {
  long long before = 0;
  for (uint32_t r = 0; r < rank; ++r) before += s.gather[phase][0][r];
  if (threadIdx.x >= 32 || target < before || target >= before + s.gather[phase][0][rank]) return;
  const int lane = threadIdx.x;
  auto scan = [&](long long v) {  // inclusive, over the lanes
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += y;
    }
    return v;
  };
  for (int t0 = row.begin; t0 < row.end; t0 += 32) {
    const long long v = t0 + lane < row.end ? s.tile[t0 + lane - row.begin] : 0;
    const long long c = before + scan(v);
    const uint32_t past = __ballot_sync(0xffffffffu, c > target);
    if (past == 0) {
      before = __shfl_sync(0xffffffffu, c, 31);
      continue;
    }
    const int l = __ffs(past) - 1;
    before = __shfl_sync(0xffffffffu, c - v, l);
    Fixed w[8];
    long long sum = 0;
    const int x = row.first(t0 + l);
    left4(row, x, ref, drawn, S, gone, p, s, w);
    left4(row, x + 4, ref, drawn, S, gone, p, s, w + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += w[i].value();
    long long at = before + scan(sum) - sum;
    int found = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      at += w[i].value();
      if (found < 0 && at > target) found = x + i;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, found >= 0);
    if (hit != 0 && lane == __ffs(hit) - 1) *where = found;
    return;
  }
}

template <bool FP32>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) verify_kernel(const Params p) {
  __shared__ Shared s;
  const uint32_t rank = cluster_rank(), size = cluster_size();
  const long long seq = blockIdx.x / size, node0 = seq * p.n_nodes;
  const bool writer = rank == 0 && threadIdx.x == 0;
  if (size > 1) cluster_started();
  if (threadIdx.x < 128) s.table[threadIdx.x] = kExp2[threadIdx.x];
  if (threadIdx.x < p.n_nodes) {
    s.parents[threadIdx.x] = p.parents[node0 + threadIdx.x];
    s.tokens[threadIdx.x] = p.tokens[node0 + threadIdx.x];
    s.u[threadIdx.x] = p.uniforms[node0 + threadIdx.x];
    if (rank == 0) p.path[node0 + threadIdx.x] = -1;
  }
  __syncthreads();
  int kept = 0, phase = 0, cur = s.parents[0] == -1 ? 0 : -1;
  if (writer) p.next_token[seq] = -1;
  // Every CTA takes the same way: each decision is made from s.u, s.tokens and sums that all have.
  while (cur >= 0) {
    if (writer) p.path[node0 + kept] = cur;
    ++kept;
    const Row<FP32> row(p, node0 + cur, rank, size);
    // what the children's tokens have is on its way during the pass
    float logit = -INFINITY, draft = 0.f;
    if (threadIdx.x < p.n_nodes && !p.greedy && s.parents[threadIdx.x] == cur) {
      const int x = s.tokens[threadIdx.x];
      if (x >= 0 && x < p.V) {
        logit = row.at(x);
        if (row.q) draft = __ldg(row.q + x);
      }
    }
    const Top top = row_quick(row, p, s, phase, rank, size, kept == 1);
    const float M = top.max;
    long long T = __float2ll_rn(top.sum * 0x1p44f);
    int accepted = -1;
    if (M == -INFINITY) break;
    if (p.greedy) {
      for (int j = cur + 1; j < p.n_nodes && accepted < 0; ++j)
        if (s.parents[j] == cur && s.tokens[j] == top.token) accepted = j;
      if (accepted < 0 && writer) p.next_token[seq] = top.token;
      cur = accepted;
      continue;
    }
    if (threadIdx.x < p.n_nodes) s.logit[threadIdx.x] = logit, s.draft[threadIdx.x] = draft;
    __syncthreads();
    const Reference ref = reference(M, p);
    int gone = 0;
    bool drawn = false;               // whether S is above 0
    float2 S = make_float2(0.f, 0.f);  // the T of all drawn children that were not accepted
    bool exact = false;  // T and the sums in shared memory are
    bool stale = false;  // ... but not those of S
    for (int j = cur + 1; j < p.n_nodes; ++j) {
      const int x = s.tokens[j];
      if (s.parents[j] != cur || x < 0 || x >= p.V) continue;
      if (row.q) {
        Pair a = own_weight(s.logit[j], ref, p, s.table);
        const float q = s.draft[j], u = fminf(fmaxf(s.u[j], 0.f), 1.f);  // as fraction64
        if (drawn) a = without(a, q, S);
        // u q T - a, and whether that has its sign for any T that the quick pass may stand for
        bool sure = true;
        auto excess = [&]() {
          const float2 t = from_fixed44(T);
          const float uq = u * q, uq_lo = fmaf(u, q, -uq);
          const float h = uq * t.x, l = fmaf(uq, t.x, -h) + fmaf(uq, t.y, uq_lo * t.x);
          const float d = (h - a.hi) + (l - a.lo);
          sure = exact || fabsf(d) > h * p.quick;
          return d;
        };
        float d = excess();
        if (sure && d < 0.f) {
          accepted = j;
          break;
        }
        if (!exact) {
          T = row_sum(row, ref, false, S, p, s, phase, rank, size), exact = true;
          if (!sure && (d = excess()) < 0.f) {
            accepted = j;
            break;
          }
        }
        const float2 more = plus(S, from_fixed44(T));
        const long long left = row_sum(row, ref, true, more, p, s, phase, rank, size);
        stale = left <= 0;
        if (!stale) T = left, S = more, drawn = true;
      } else {
        long long w = fixed44(weight(s.logit[j], ref, p, s.table)).value();
        for (int n = 0; n < gone; ++n)
          if (s.gone[n] == x) w = 0;
        bool sure = true;
        auto excess = [&]() {
          const long long h = static_cast<long long>(__umul64hi(fraction64(s.u[j]), static_cast<unsigned long long>(T)));
          sure = exact || llabs(h - w) > static_cast<long long>(static_cast<float>(h) * p.quick) + 1;
          return h - w;
        };
        long long d = excess();
        if (sure && d < 0) {
          accepted = j;
          break;
        }
        if (!exact) {
          T = row_sum(row, ref, false, S, p, s, phase, rank, size), exact = true;
          if (!sure && (d = excess()) < 0) {
            accepted = j;
            break;
          }
        }
        if (w == 0 || T - w <= 0) continue;
        T -= w;
        __syncthreads();
        if (threadIdx.x == 0) {
          s.gone[gone] = x;
          const int tile = (x + row.shift) / kTile;
          s.gather[phase][0][tile / row.per] -= w;
          if (tile >= row.begin && tile < row.end) s.tile[tile - row.begin] -= w;
        }
        __syncthreads();
        ++gone;
      }
    }
    if (accepted < 0) {
      if (!exact) T = row_sum(row, ref, false, S, p, s, phase, rank, size);
      if (stale) row_sum(row, ref, drawn, S, p, s, phase, rank, size);
      const long long target = static_cast<long long>(__umul64hi(fraction64(s.u[0]), static_cast<unsigned long long>(T)));
      find_token(row, target, ref, drawn, S, gone, p, s, phase, rank, p.next_token + seq);
    }
    cur = accepted;
    __syncthreads();  // shared sums have been read
  }
  if (writer) p.n_kept[seq] = kept;
  if (size > 1) {
    if (kept == 0) cluster_wait();  // no pass has
    cluster_sync();  // no CTA leaves while another may still store to it
  }
}

}  // namespace verify
}  // namespace fa
