// Rotary positions: the angle of a pair at a position, and the rows of a call
// that rotates queries and keys on their way (rope.cu's kernels and the decode
// call that writes its new rows itself).
//
// Angles.  A pair turns freqs[i] / 2^64 of a full turn per position, so the
// angle at position p is p x freqs[i] mod 2^64: one integer product, exact for
// every 32-bit p, where a float product has lost the angle's leading digits at
// far positions (2^-24 of 10^6 radians is 0.06).  Its top 32 bits give the
// nearest quarter turn and a remainder t of at most half a quarter; sine and
// cosine of t quarter turns are their Taylor series to t^9 and t^10, whose
// first left-out terms are below 2^-28, and the quarter turns swap and negate
// them.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "kv_write.cuh"

namespace tl {

// Two binary32 numbers in one 64-bit register, multiplied and added as two.
TL_DEVINLINE uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
TL_DEVINLINE float2 f2_unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
TL_DEVINLINE uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
TL_DEVINLINE uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
TL_DEVINLINE uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// (cos, sin) of n x fa / 2^64 and n x fb / 2^64 turns, all within 2^-23 of exact.
// The series of the two are evaluated in pairs of numbers.
TL_DEVINLINE void rope_turns(uint64_t fa, uint64_t fb, uint32_t n, float2& a, float2& b) {
  // the phase's top 32 bits, half a quarter turn further: the nearest quarter in
  // the top two
  const uint32_t ua = (uint32_t)((fa * n) >> 32) + 0x20000000u;
  const uint32_t ub = (uint32_t)((fb * n) >> 32) + 0x20000000u;
  auto both = [](float x) { return f2_pack(x, x); };
  const uint64_t t = f2_mul(f2_pack((float)((int32_t)(ua & 0x3fffffffu) - 0x20000000),
                                    (float)((int32_t)(ub & 0x3fffffffu) - 0x20000000)),
                            both(0x1p-30f));  // in [-1/2, 1/2]
  const uint64_t x = f2_mul(t, t);
  // (pi/2)^k / k!, alternating; pi/2 in two parts
  uint64_t s = f2_fma(x, both(1.6044118479e-4f), both(-4.6817541353e-3f));
  s = f2_fma(x, s, both(7.9692626246e-2f));
  s = f2_fma(x, s, both(-6.4596409751e-1f));
  s = f2_fma(x, s, both(-4.3711388287e-8f));
  s = f2_fma(t, both(1.5707963705f), f2_mul(t, s));
  uint64_t c = f2_fma(x, both(-2.5202042374e-5f), both(9.1926027483e-4f));
  c = f2_fma(x, c, both(-2.0863480763e-2f));
  c = f2_fma(x, c, both(2.5366950790e-1f));
  c = f2_fma(x, c, both(-1.2337005501f));
  c = f2_fma(x, c, both(1.f));
  const float2 s2 = f2_unpack(s), c2 = f2_unpack(c);
  // quarters 1 and 3 swap, 1 and 2 negate the cosine, 2 and 3 the sine
  auto place = [](float s, float c, uint32_t u) {
    const bool odd = u & 0x40000000u;
    return make_float2(
        __uint_as_float(__float_as_uint(odd ? s : c) ^ ((u + 0x40000000u) & 0x80000000u)),
        __uint_as_float(__float_as_uint(odd ? c : s) ^ (u & 0x80000000u)));
  };
  a = place(s2.x, c2.x, ua);
  b = place(s2.y, c2.y, ub);
}

// The pair (lo, hi) turned.
TL_DEVINLINE void rope_rotate(float& lo, float& hi, float c, float s) {
  const float y = fmaf(lo, c, -(hi * s));
  hi = fmaf(hi, c, lo * s);
  lo = y;
}

// ----------------------------------------------------------------- units --
//
// A row of U = d / 16 units (d a multiple of 16) is moved a unit a lane: 16
// elements with 8 whole pairs, in 16 / W words of W elements, word i of a unit
// beside word i of the next, so that a warp's access to one word of its units
// is contiguous.  Interleaved pairs: word i of unit u is the row's word i U + u.
// Halves: words go in twos, the p-th (p = i U + u, i < 8 / W) at W p in the lower
// half with its partner rot/2 further, and from p = rot / 2W on one behind the
// other behind the rotated part.  So rot is a multiple of W (interleaved) or 2W.
constexpr int kRopeMaxUnits = 16;  // of a row moved in units (d up to 256)
enum RopeElem { kElemBf16, kElemF32, kElemE4m3, kElemInt8 };

// The words' first elements (halves: the lower words, then their partners).
template <bool INTER, int W>
TL_DEVINLINE void rope_unit_words(int u, int d, int rot, int* at) {
  constexpr int NW = 16 / W;
  const int U = d >> 4;
  if (INTER) {
#pragma unroll
    for (int i = 0; i < NW; ++i) at[i] = (i * U + u) * W;
  } else {
#pragma unroll
    for (int i = 0; i < NW / 2; ++i) {
      const int e = (i * U + u) * W;
      const bool turned = 2 * e < rot;
      at[i] = turned ? e : 2 * e;  // behind: rot + 2 (e - rot/2)
      at[i + NW / 2] = turned ? e + (rot >> 1) : 2 * e + W;
    }
  }
}

// The 8 pairs of a unit: n consecutive ones a word (halves: a word of the lower half).
template <bool INTER, int W>
struct RopePairs {
  static constexpr int n = INTER ? W / 2 : W;
  // whether pair k turns (the words of a unit turn up to some, in order)
  static TL_DEVINLINE bool turn(const int* at, int k, int rot) {
    return at[k / n] < (INTER ? rot : rot >> 1);
  }
  static TL_DEVINLINE int index(const int* at, int k) {
    return (INTER ? at[k / n] >> 1 : at[k / n]) + k % n;
  }
  // whether word i is one of those
  static TL_DEVINLINE bool word(const int* at, int i, int rot) {
    return INTER ? at[i] < rot : at[i % (8 / W)] < rot >> 1;
  }
};

// A unit as it lies in memory.
template <int E, int W>
struct RopeUnit {
  static constexpr int kBytes = E == kElemF32 ? 4 : E == kElemBf16 ? 2 : 1;  // of an element
  static constexpr int NW = 16 / W;
  using Word = typename std::conditional<
      W * kBytes == 16, uint4,
      typename std::conditional<
          W * kBytes == 8, uint2,
          typename std::conditional<W * kBytes == 4, uint32_t, uint16_t>::type>::type>::type;
  alignas(16) Word w[NW];  // (read as 32-bit words too)
  TL_DEVINLINE void load(const char* row, const int* at) {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = __ldcs(reinterpret_cast<const Word*>(row + at[i] * kBytes));
  }
  TL_DEVINLINE void store(char* row, const int* at) const {
#pragma unroll
    for (int i = 0; i < NW; ++i) __stcs(reinterpret_cast<Word*>(row + at[i] * kBytes), w[i]);
  }
  // the values, word by word (int8: codes)
  TL_DEVINLINE void values(float* x) const {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(w);
    if constexpr (E == kElemF32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[i]);
    } else if constexpr (E == kElemBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
      }
    } else if constexpr (E == kElemE4m3) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t h;
        const uint16_t codes = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(codes));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    } else {
      // a code c as the float 2^23 + 128 + c, whose last byte is c + 128
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const uint32_t w4 = v[i >> 2] ^ 0x80808080u;
        const float2 f = f2_unpack(f2_add(
            f2_pack(__uint_as_float(__byte_perm(w4, 0x4b000000u, 0x7650 + (i & 3))),
                    __uint_as_float(__byte_perm(w4, 0x4b000000u, 0x7651 + (i & 3)))),
            f2_pack(-8388736.f, -8388736.f)));
        x[i] = f.x;
        x[i + 1] = f.y;
      }
    }
  }
  // values rounded to the type (not int8)
  TL_DEVINLINE void set(const float* x) {
    uint32_t* v = reinterpret_cast<uint32_t*>(w);
    if constexpr (E == kElemF32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(x[i]);
    } else if constexpr (E == kElemBf16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    } else {
      // (a sum that is a number has no NaN in it; otherwise each value is looked at)
      uint64_t sum = f2_pack(x[0], x[1]);
#pragma unroll
      for (int i = 2; i < 16; i += 2) sum = f2_add(sum, f2_pack(x[i], x[i + 1]));
      const float2 s = f2_unpack(sum);
      if (s.x + s.y == s.x + s.y) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t lo, hi;
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(x[4 * i + 1]), "f"(x[4 * i]));
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(x[4 * i + 3]), "f"(x[4 * i + 2]));
          v[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = e4m3x4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      }
    }
  }
  // int8: the codes of values x with scale sc, x / sc in binary32 rounded half
  // to even as quantize4_int8's; finite: every x is.  The quotient comes from
  // the reciprocal: with |x / sc| <= 127 it is within 3 x 2^-24 x 127 < 2^-15 of
  // the correctly rounded one, so only values that near to the middle of two
  // codes are divided.
  TL_DEVINLINE void set_codes(const float* x, float sc, bool finite) {
    constexpr float kWhole = 12582912.f;  // 1.5 x 2^23: adding it rounds to a whole number
    uint32_t* v = reinterpret_cast<uint32_t*>(w);
    const float inv = __frcp_rn(sc);
    const bool normal = finite && sc >= 1e-37f;  // so is the reciprocal
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t code[4];
      bool divide = !normal;
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const uint64_t q = f2_mul(f2_pack(x[4 * i + k], x[4 * i + k + 1]), f2_pack(inv, inv));
        const uint64_t r = f2_add(q, f2_pack(kWhole, kWhole));
        // q - (r - kWhole)
        const float2 off = f2_unpack(f2_fma(f2_add(r, f2_pack(-kWhole, -kWhole)),
                                            f2_pack(-1.f, -1.f), q));
        divide |= fmaxf(fabsf(off.x), fabsf(off.y)) > 0.5f - 0x1p-15f;
        const float2 c = f2_unpack(r);
        code[k] = __float_as_uint(c.x);
        code[k + 1] = __float_as_uint(c.y);
      }
      if (divide)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float r = 0.f;
          if (isfinite(x[4 * i + k]) && sc > 0.f)
            r = fminf(fmaxf(rintf(__fdiv_rn(x[4 * i + k], sc)), -127.f), 127.f);
          code[k] = (uint32_t)__float2int_rn(r);
        }
      v[i] = __byte_perm(__byte_perm(code[0], code[1], 0x0040),
                         __byte_perm(code[2], code[3], 0x0040), 0x5410);
    }
  }
};

// The largest finite magnitude of a unit's values; bad: one is not finite.
// (Magnitudes compare as their bits do.)
TL_DEVINLINE float rope_unit_max(const float* x, bool& bad) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  bad = top >= 0x7f800000u;
  if (!bad) return __uint_as_float(top);
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (isfinite(x[i])) m = fmaxf(m, fabsf(x[i]));
  return m;
}

// A unit's values with its pairs turned by turn(k).
template <bool INTER, int W, class Turn>
TL_DEVINLINE void rope_unit_rotate(float* x, const int* at, int rot, Turn turn) {
  using Pairs = RopePairs<INTER, W>;
#pragma unroll
  for (int g = 0; g < 8; g += Pairs::n)
    if (Pairs::turn(at, g, rot)) {
#pragma unroll
      for (int k = g; k < g + Pairs::n; ++k) {
        const float2 cs = turn(k);
        if (INTER) rope_rotate(x[2 * k], x[2 * k + 1], cs.x, cs.y);
        else rope_rotate(x[k], x[8 + k], cs.x, cs.y);
      }
    }
}

// A unit's turned values in its words; words that do not turn keep their bits.
template <bool INTER, int W, class Unit>
TL_DEVINLINE void rope_unit_set(Unit& unit, const float* x, const int* at, int rot) {
  const Unit was = unit;
  unit.set(x);
#pragma unroll
  for (int i = 0; i < Unit::NW; ++i)
    if (!RopePairs<INTER, W>::word(at, i, rot)) unit.w[i] = was.w[i];
}

// The rows of one call: h_q query heads, then h_kv key heads, then h_kv value
// heads of every token.  Without slots (slots null) there are queries alone.
struct RopeRows {
  const void *q, *k, *v;  // token t's rows at t * stride elements
  void* q_out;
  int64_t q_stride, k_stride, v_stride, out_stride;
  void *k_dst, *v_dst;        // pools (int8: codes)
  float *k_scales, *v_scales;  // int8 pools
  const int64_t* slots;
  const int32_t* positions;
  const uint64_t* freqs;
  int64_t n_slots;
  int32_t n, h_q, h_kv, d, rot, page_size;
  int32_t interleaved;
  float scale;
  uint32_t* error_word;
};

// What becomes of key and value rows: the source's type, e4m3 codes, int8
// codes and scales.
enum { kRopeSame = 0, kRopeE4m3 = 1, kRopeInt8 = 2 };

// Where the scale of head g at `slot` lies, [num_pages][h_kv][page_size] (slots
// are below 2^31: a 32-bit division).
TL_DEVINLINE int64_t rope_scale_place(const RopeRows& R, int64_t slot, int g) {
  const uint32_t page = (uint32_t)slot / (uint32_t)R.page_size;
  return ((int64_t)page * R.h_kv + g) * R.page_size + ((uint32_t)slot - page * R.page_size);
}

// A token's slot (-1: none), checked; `tell`: this thread reports.
TL_DEVINLINE int64_t rope_slot(const RopeRows& R, int64_t t, int pos, bool tell) {
  if (!R.slots) return -1;
  const int64_t slot = __ldg(R.slots + t);
  if (slot == -1) return -1;
  if (slot < 0 || slot >= R.n_slots) {
    if (tell) report(R.error_word, TL_DEVERR_SLOT_RANGE);
    return -1;
  }
  if (pos < 0) {
    if (tell) report(R.error_word, TL_DEVERR_CONTEXT_RANGE);
    return -1;
  }
  return slot;
}

// P passes over a token's heads by one warp, in rotary units: lane l takes unit
// u = l % U of head h0 + p HW + l / U in pass p, for U = d / 16 units a row and
// HW = 32 / U heads a pass.  Every load comes before the angles, which the
// warp's lanes make once for the token and every head reads (cs: 8 U float2 of
// shared memory of the warp; two pairs, 16 bytes, of each lane side by side).
template <bool F32, int KIND, bool INTER, int P, int W = F32 ? 4 : 8>
TL_DEVINLINE void rope_units(const RopeRows& R, int64_t t, int h0, int heads, int U, int HW,
                             int lane, float4* cs) {
  using Src = RopeUnit<F32 ? kElemF32 : kElemBf16, W>;
  using Pairs = RopePairs<INTER, W>;
  const int sub = lane / U, u = lane - sub * U, turned = R.h_q + R.h_kv;
  const int pos = __ldg(R.positions + t);
  int64_t slot = -1;
  if (h0 + P * HW > R.h_q) slot = rope_slot(R, t, pos, lane == 0);
  int at[16 / W];
  rope_unit_words<INTER, W>(u, R.d, R.rot, at);
  Src x[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = h0 + p * HW + sub;
    if (sub >= HW || h >= heads) continue;
    const bool is_q = h < R.h_q, is_v = h >= turned;
    // (a single pass reads rows without a slot too: it does not wait for the slot)
    if (P > 1 && !is_q && slot < 0) continue;
    const char* row = static_cast<const char*>(is_q ? R.q : is_v ? R.v : R.k) +
                      Src::kBytes * (t * (is_q ? R.q_stride : is_v ? R.v_stride : R.k_stride) +
                                     (int64_t)(is_q ? h : is_v ? h - turned : h - R.h_q) * R.d);
    x[p].load(row, at);
  }
  float2 turn[8];
  if (pos >= 0 && h0 < turned) {
    if constexpr (Pairs::n > 1) {
      // chunk c of two pairs at (c % per) * (rot/4 / per) + c / per, for the `per`
      // chunks that a lane reads one behind the other
      constexpr int per = Pairs::n / 2;
      const int step = (R.rot >> 2) / per;
      for (int c = lane; c < R.rot >> 2; c += 32) {
        float2 y, z;
        rope_turns(__ldg(R.freqs + 2 * c), __ldg(R.freqs + 2 * c + 1), (uint32_t)pos, y, z);
        cs[c % per * step + c / per] =
            make_float4(y.x * R.scale, y.y * R.scale, z.x * R.scale, z.y * R.scale);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        if (!Pairs::turn(at, k, R.rot)) continue;
        const int c = Pairs::index(at, k) >> 1;
        const float4 f = cs[c % per * step + c / per];
        turn[k] = make_float2(f.x, f.y);
        turn[k + 1] = make_float2(f.z, f.w);
      }
    } else {
      float2* one = reinterpret_cast<float2*>(cs);
      for (int c = lane; c < R.rot >> 1; c += 32) {
        const uint64_t f = __ldg(R.freqs + c);
        float2 y, same;
        rope_turns(f, f, (uint32_t)pos, y, same);
        one[c] = make_float2(y.x * R.scale, y.y * R.scale);
      }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (Pairs::turn(at, k, R.rot)) turn[k] = one[Pairs::index(at, k)];
    }
    __syncwarp();  // (cs is the warp's next item's too)
  }
  auto of = [&](int k) { return turn[k]; };
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int h = h0 + p * HW + sub;
    const bool here = sub < HW && h < heads;
    const bool is_q = h < R.h_q, is_v = h >= turned, rotates = pos >= 0 && !is_v;
    if (KIND != kRopeInt8 && (!here || (!is_q && slot < 0))) continue;
    float y[16];
    if (KIND == kRopeSame || is_q) {
      if (here) {
        if (rotates && Pairs::turn(at, 0, R.rot)) {
          x[p].values(y);
          rope_unit_rotate<INTER, W>(y, at, R.rot, of);
          rope_unit_set<INTER, W>(x[p], y, at, R.rot);
        }
        char* row =
            is_q ? static_cast<char*>(R.q_out) + Src::kBytes * (t * R.out_stride + (int64_t)h * R.d)
                 : static_cast<char*>(is_v ? R.v_dst : R.k_dst) +
                       Src::kBytes * ((slot * R.h_kv + (is_v ? h - turned : h - R.h_q)) * R.d);
        x[p].store(row, at);
      }
      if (KIND != kRopeInt8) continue;
    }
    // An int8 pass with key or value rows goes on with all of the warp's lanes, one of
    // queries alone with none: lanes behind the last whole head stand at head
    // h0 + (p + 1) HW, which may be a key's, and must not meet the shuffles alone.
    if (KIND == kRopeInt8 && h0 + (p + 1) * HW <= R.h_q) continue;
    if constexpr (KIND != kRopeSame) {
      const bool row = here && !is_q && slot >= 0;
      const int g = is_v ? h - turned : h - R.h_q;
      if (row) {
        x[p].values(y);
        if (rotates) rope_unit_rotate<INTER, W>(y, at, R.rot, of);
      }
      RopeUnit<KIND == kRopeInt8 ? kElemInt8 : kElemE4m3, W> codes;
      if constexpr (KIND == kRopeE4m3) {
        codes.set(y);
      } else {
        // the row's scale over its U lanes, in step with the warp's other lanes
        bool bad = false;
        float m = row ? rope_unit_max(y, bad) : 0.f;
        if ((U & (U - 1)) == 0) {
          for (int o = U >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        } else {
          const float own = m;
          for (int i = 0; i < U; ++i)
            m = fmaxf(m, __shfl_sync(0xffffffffu, own, (sub * U + i) & 31));
        }
        if (!row) continue;
        const float sc = __fdiv_rn(m, 127.f);
        codes.set_codes(y, sc, !bad);
        if (u == 0)
          (is_v ? R.v_scales : R.k_scales)[rope_scale_place(R, slot, g)] = sc;
        if (bad) report(R.error_word, TL_DEVERR_VALUE_RANGE);
      }
      codes.store(static_cast<char*>(is_v ? R.v_dst : R.k_dst) + (slot * R.h_kv + g) * R.d, at);
    }
  }
}

// One row (token t, head h of the h_q + 2 h_kv) by one warp, element by
// element: every size, layout and alignment.
template <bool F32, int KIND>
__device__ void rope_row(const RopeRows& R, int64_t t, int h, int lane) {
  using T = typename std::conditional<F32, float, unsigned short>::type;
  const int pos = __ldg(R.positions + t);
  const bool is_q = h < R.h_q, is_v = h >= R.h_q + R.h_kv;
  const int g = is_q ? h : is_v ? h - R.h_q - R.h_kv : h - R.h_q;
  const T* src = static_cast<const T*>(is_q ? R.q : is_v ? R.v : R.k) +
                 t * (is_q ? R.q_stride : is_v ? R.v_stride : R.k_stride) + (int64_t)g * R.d;
  int64_t slot = -1;
  if (!is_q) {
    slot = rope_slot(R, t, pos, lane == 0 && h == R.h_q);
    if (slot < 0) return;
  }
  const int rot = is_v || pos < 0 ? 0 : R.rot;  // elements that are rotated
  auto value = [&](int e) {
    return F32 ? (float)src[e] : __uint_as_float((uint32_t)src[e] << 16);
  };
  // elements of pair i, rotated
  auto pair = [&](int i, float& lo, float& hi, int& el, int& eh) {
    el = R.interleaved ? 2 * i : i;
    eh = R.interleaved ? 2 * i + 1 : i + (rot >> 1);
    lo = value(el);
    hi = value(eh);
    const uint64_t f = __ldg(R.freqs + i);
    float2 cs, same;
    rope_turns(f, f, (uint32_t)pos, cs, same);
    rope_rotate(lo, hi, cs.x * R.scale, cs.y * R.scale);
  };
  auto same = [&](T* dst) {
    for (int i = lane; i < rot >> 1; i += 32) {
      float lo, hi;
      int el, eh;
      pair(i, lo, hi, el, eh);
      if constexpr (F32) {
        dst[el] = lo;
        dst[eh] = hi;
      } else {
        const uint32_t w = pack_bf16x2(lo, hi);
        dst[el] = (T)(w & 0xffffu);
        dst[eh] = (T)(w >> 16);
      }
    }
    if (static_cast<const T*>(dst) != src)  // in place the rest is there already
      for (int e = rot + lane; e < R.d; e += 32) dst[e] = src[e];
  };
  if (is_q) {
    same(static_cast<T*>(R.q_out) + t * R.out_stride + (int64_t)h * R.d);
    return;
  }
  const int64_t at = (slot * R.h_kv + g) * R.d;
  void* pool = is_v ? R.v_dst : R.k_dst;
  if constexpr (KIND == kRopeSame) {
    same(static_cast<T*>(pool) + at);
  } else if constexpr (KIND == kRopeE4m3) {
    uint8_t* dst = static_cast<uint8_t*>(pool) + at;
    for (int i = lane; i < rot >> 1; i += 32) {
      float lo, hi;
      int el, eh;
      pair(i, lo, hi, el, eh);
      const uint32_t w = e4m3x4(lo, hi, 0.f, 0.f);
      dst[el] = (uint8_t)w;
      dst[eh] = (uint8_t)(w >> 8);
    }
    for (int e = rot + lane; e < R.d; e += 32) dst[e] = (uint8_t)e4m3x4(value(e), 0.f, 0.f, 0.f);
  } else {
    // as quantize_row_int8: the scale over the finite values, then the codes
    int8_t* dst = static_cast<int8_t*>(pool) + at;
    float m = 0.f;
    bool bad = false;
    auto see = [&](float x) {
      if (isfinite(x)) m = fmaxf(m, fabsf(x));
      else bad = true;
    };
    for (int i = lane; i < rot >> 1; i += 32) {
      float lo, hi;
      int el, eh;
      pair(i, lo, hi, el, eh);
      see(lo);
      see(hi);
    }
    for (int e = rot + lane; e < R.d; e += 32) see(value(e));
    const float sc = __fdiv_rn(warp_max(m), 127.f);
    auto code = [&](float x) {
      float r = 0.f;
      if (isfinite(x) && sc > 0.f) r = fminf(fmaxf(rintf(__fdiv_rn(x, sc)), -127.f), 127.f);
      return (int8_t)__float2int_rn(r);
    };
    for (int i = lane; i < rot >> 1; i += 32) {
      float lo, hi;
      int el, eh;
      pair(i, lo, hi, el, eh);
      dst[el] = code(lo);
      dst[eh] = code(hi);
    }
    for (int e = rot + lane; e < R.d; e += 32) dst[e] = code(value(e));
    if (lane == 0)
      (is_v ? R.v_scales : R.k_scales)[rope_scale_place(R, slot, g)] = sc;
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(R.error_word, TL_DEVERR_VALUE_RANGE);
  }
}

}  // namespace tl
