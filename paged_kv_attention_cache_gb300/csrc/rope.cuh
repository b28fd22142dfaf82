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
// them.  27 instructions a pair for both.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "kv_write.cuh"

namespace tl {

// (cos, sin) of pos x freq / 2^64 turns, both within 2^-23 of exact.
TL_DEVINLINE float2 rope_turn(uint64_t freq, int32_t pos) {
  const uint32_t turn = (uint32_t)(((uint64_t)(int64_t)pos * freq) >> 32);
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float t = (float)(int32_t)(turn - (quarter << 30)) * 0x1p-30f;  // in [-1/2, 1/2]
  const float x = t * t;
  // (pi/2)^k / k!, alternating; pi/2 in two parts
  float s = fmaf(x, 1.6044118479e-4f, -4.6817541353e-3f);
  s = fmaf(x, s, 7.9692626246e-2f);
  s = fmaf(x, s, -6.4596409751e-1f);
  s = fmaf(t, 1.5707963705f, t * fmaf(x, s, -4.3711388287e-8f));
  float c = fmaf(x, -2.5202042374e-5f, 9.1926027483e-4f);
  c = fmaf(x, c, -2.0863480763e-2f);
  c = fmaf(x, c, 2.5366950790e-1f);
  c = fmaf(x, c, -1.2337005501f);
  c = fmaf(x, c, 1.f);
  float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  if ((quarter + 1) & 2) a = -a;
  if (quarter & 2) b = -b;
  return make_float2(a, b);
}

// The pair (lo, hi) turned.
TL_DEVINLINE void rope_rotate(float& lo, float& hi, float c, float s) {
  const float y = fmaf(lo, c, -(hi * s));
  hi = fmaf(hi, c, lo * s);
  lo = y;
}

// ----------------------------------------------------------------- units --
//
// A unit is 16 elements of a row that hold 8 whole pairs: in the layout of
// halves the 8 elements from 8u and their partners from rot/2 + 8u, otherwise
// the 16 from 16u, for u < rot/16; behind the rotated part the 16 from 16u.
// Rows whose d and rot are multiples of 16 are made of such units, each two
// contiguous runs of 8 elements (16 bytes in 16 bits).
enum RopeElem { kElemBf16, kElemF32, kElemE4m3, kElemInt8 };

TL_DEVINLINE void rope_unit_offsets(int u, int rot, bool interleaved, int& a, int& b) {
  const bool halves = !interleaved && 16 * u < rot;
  a = halves ? 8 * u : 16 * u;
  b = halves ? (rot >> 1) + 8 * u : 16 * u + 8;
}

// A unit as it lies in memory: run a, then run b.
template <int E>
struct RopeUnit {
  using W = typename std::conditional<E == kElemBf16 || E == kElemF32, uint4, uint2>::type;
  static constexpr int kBytes = E == kElemF32 ? 4 : E == kElemBf16 ? 2 : 1;  // of an element
  static constexpr int kRun = E == kElemF32 ? 2 : 1;                        // words of a run
  W w[2 * kRun];
  // row: the row's first element; a, b: the runs' first elements
  TL_DEVINLINE void load(const char* row, int a, int b) {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      w[i] = __ldcg(reinterpret_cast<const W*>(row + a * kBytes) + i);
      w[kRun + i] = __ldcg(reinterpret_cast<const W*>(row + b * kBytes) + i);
    }
  }
  TL_DEVINLINE void store(char* row, int a, int b) const {
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      reinterpret_cast<W*>(row + a * kBytes)[i] = w[i];
      reinterpret_cast<W*>(row + b * kBytes)[i] = w[kRun + i];
    }
  }
  // the values, run a then run b (int8: codes)
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
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = (float)(int8_t)(v[i >> 2] >> (8 * (i & 3)));
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
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = e4m3x4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
  }
  // int8: the codes of values x with scale sc (as quantize4_int8)
  TL_DEVINLINE void set_codes(const float* x, float sc) {
    uint32_t* v = reinterpret_cast<uint32_t*>(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t word = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y = x[4 * i + k];
        float r = 0.f;
        if (isfinite(y) && sc > 0.f) r = fminf(fmaxf(rintf(__fdiv_rn(y, sc)), -127.f), 127.f);
        word |= (uint32_t)(uint8_t)(int8_t)__float2int_rn(r) << (8 * k);
      }
      v[i] = word;
    }
  }
};

// The largest finite magnitude of a unit's values; bad: one is not finite.
TL_DEVINLINE float rope_unit_max(const float* x, bool& bad) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (isfinite(x[i])) m = fmaxf(m, fabsf(x[i]));
    else bad = true;
  }
  return m;
}

// The 8 pairs of a unit's values, turned by turn(k).
template <class Turn>
TL_DEVINLINE void rope_unit_rotate(float* x, bool interleaved, Turn turn) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float2 cs = turn(k);
    if (interleaved) rope_rotate(x[2 * k], x[2 * k + 1], cs.x, cs.y);
    else rope_rotate(x[k], x[8 + k], cs.x, cs.y);
  }
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
    const float2 cs = rope_turn(__ldg(R.freqs + i), pos);
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
      (is_v ? R.v_scales : R.k_scales)[(slot / R.page_size * R.h_kv + g) * R.page_size +
                                       slot % R.page_size] = sc;
    if (__any_sync(0xffffffffu, bad) && lane == 0) report(R.error_word, TL_DEVERR_VALUE_RANGE);
  }
}

}  // namespace tl
