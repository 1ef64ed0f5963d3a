// The paged key/value cache: quantised as it is written, read back as the values it stands for.
//
// A group of 32 channels of one token and head is held as codes with one power-of-two scale:
// value = code * 2^e, e the smallest integer with max|x| <= top * 2^e (top = 448 for e4m3, 6 for
// e2m1), so that nothing saturates.  Dividing by 2^e and multiplying back are exact in f32; the only
// rounding is the code's own, to nearest, ties to even.  A value has at most 4 significant bits and an
// exponent that e's limits keep normal, so it is exact in bf16.  A group with a value that is not
// finite has the scale byte 255 and reads back as NaN.
//
// Both kernels move each byte once and compute little: HBM bounds them.  One wave holds one token at a
// time (its sequence, position and page are the wave's, found once), one lane 8 channels; four lanes
// share a group.
#pragma once

#include "serve_common.h"

namespace serve {

struct KvRows {
  const void* k;
  const void* v;
  int64_t k_token, k_head, v_token, v_head;  // strides in elements
};

// Where a new token goes: its offset inside the pool for head 0, and its slot; false where it has none.
__device__ __forceinline__ bool place_of(const Cache& c, int t, int64_t* base, int* slot, bool* bad) {
  const int b = sequence_of(c, t);
  *bad = true;
  if (b >= c.batch) return false;
  const Seq s = sequence(c, b);
  const int pos = s.len - s.n + (t - s.first);
  if (t < s.first || t >= s.first + s.n || pos < 0) return false;
  const uint32_t page = divide((uint32_t)pos, c.page);
  *base = block_of(c, b, page, 0);
  *slot = pos - (int)(page * c.page.by);
  if (*base < 0) return false;
  *bad = s.bad;
  return true;
}

template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t at, float* x) {
  if constexpr (F32) {
    const float* f = static_cast<const float*>(p) + at;
    if constexpr (VEC) {
      const f32x4 a = *reinterpret_cast<const f32x4*>(f), b = *reinterpret_cast<const f32x4*>(f + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = f[i];
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p) + at;
    if constexpr (VEC) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(h);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(a[i] << 16), x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = bf16_f32(h[i]);
    }
  }
}

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* p, int64_t at, const float* x) {
  if constexpr (F32) {
    float* f = static_cast<float*>(p) + at;
    if constexpr (VEC) {
      *reinterpret_cast<f32x4*>(f) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4*>(f + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = x[i];
    }
  } else {
    const u32x4 a = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    if constexpr (VEC) {
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + at) = a;
    } else {
      uint16_t* h = static_cast<uint16_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) h[2 * i] = (uint16_t)a[i], h[2 * i + 1] = (uint16_t)(a[i] >> 16);
    }
  }
}

template <int KIND, bool F32, bool VEC>
__global__ __launch_bounds__(256) void k_kv_write(Cache c, KvRows in, int per_wave, int items, int32_t* err) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int chunks = c.dim / 8;
  int wrong = 0;
  for (int i = 0; i < per_wave; ++i) {
    const int64_t tok = ((int64_t)blockIdx.x * 4 + wave) * per_wave + i;
    if (tok >= c.tokens) break;
    const int t = (int)tok;
    int64_t base = 0;
    int slot = 0;
    bool bad = false;
    const bool there = place_of(c, t, &base, &slot, &bad);
    if (bad && blockIdx.y == 0) ++wrong;
    if (!there) continue;
    for (int it = (int)blockIdx.y * kWave + lane; it < items; it += (int)gridDim.y * kWave) {
      const int hv = it / chunks, ch = it - hv * chunks;
      const bool is_v = hv >= c.heads;
      const int head = is_v ? hv - c.heads : hv;
      float x[8];
      load8<F32, VEC>(is_v ? in.v : in.k,
                      (int64_t)t * (is_v ? in.v_token : in.k_token) + (int64_t)head * (is_v ? in.v_head : in.k_head) + ch * 8, x);
      uint8_t* blk = c.pool + base + (int64_t)head * c.block;
      uint8_t* dst = blk + (is_v ? c.v_off : 0) + slot * c.row;
      if constexpr (KIND == LLVQ_KV_BF16) {
        store8<false, true>(dst, ch * 8, x);
      } else {
        // the group's largest magnitude over its four lanes, as bits: a NaN's and an infinity's are the
        // largest of all
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const bool nonfinite = top >= 0x7f800000u;
        // e: the exponent of max|x| less the type's, one more where the mantissa passes the type's top
        // (448 = 1.75 * 2^8, 6 = 1.5 * 2^2); a zero or subnormal maximum falls to the lower limit
        constexpr int kExp = KIND == LLVQ_KV_FP8 ? 8 : 2, kHigh = KIND == LLVQ_KV_FP8 ? 119 : 125;
        constexpr uint32_t kMant = KIND == LLVQ_KV_FP8 ? 0x600000u : 0x400000u;
        constexpr float kTop = KIND == LLVQ_KV_FP8 ? 448.0f : 6.0f;
        int e = (int)(top >> 23) - 127 - kExp + ((top & 0x7fffffu) > kMant ? 1 : 0);
        e = min(max(e, -100), kHigh);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = nonfinite ? 0.0f : fminf(fmaxf(x[j] * inv, -kTop), kTop);
        if constexpr (KIND == LLVQ_KV_FP8) {
          int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
          lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
          int hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
          hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], hi, true);
          *reinterpret_cast<u32x2*>(dst + ch * 8) = u32x2{(uint32_t)lo, (uint32_t)hi};
        } else {
          uint32_t w = 0;
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], 1.0f, 0);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], 1.0f, 1);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], 1.0f, 2);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], 1.0f, 3);
          *reinterpret_cast<uint32_t*>(dst + ch * 4) = w;
        }
        if ((ch & 3) == 0) {
          blk[(is_v ? c.vs_off : c.ks_off) + slot * c.groups + (ch >> 2)] = (uint8_t)(nonfinite ? 255 : e + 127);
          if (nonfinite && err) atomicAdd(err, 1);
        }
      }
    }
  }
  if (wrong && err && lane == 0) atomicAdd(err, wrong);
}

// 8 values of one token from its codes and scale byte.
template <int KIND>
__device__ __forceinline__ void values8(const uint8_t* codes, uint32_t scale_byte, float* x) {
  if constexpr (KIND == LLVQ_KV_BF16) {
    load8<false, true>(codes, 0, x);
  } else {
    // a byte of 255 is an infinite f32, which the conversions turn into NaN for every code
    const float scale = __uint_as_float(scale_byte << 23);
    bf16x2 p[4];
    if constexpr (KIND == LLVQ_KV_FP8) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(codes);
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, false);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[0], scale, true);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, false);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[1], scale, true);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(codes);
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t u = __builtin_bit_cast(uint32_t, p[i]);
      x[2 * i] = __uint_as_float(u << 16);
      x[2 * i + 1] = __uint_as_float(u & 0xffff0000u);
    }
  }
}

template <int KIND, bool F32, bool VEC>
__global__ __launch_bounds__(256) void k_kv_read(Cache c, KvRows out, int per_wave, int items, int32_t* err) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int chunks = c.dim / 8;
  int wrong = 0;
  for (int i = 0; i < per_wave; ++i) {
    const int64_t tok = ((int64_t)blockIdx.x * 4 + wave) * per_wave + i;
    if (tok >= c.tokens) break;
    const int t = (int)tok;
    int64_t base = 0;
    int slot = 0;
    bool bad = false;
    const bool there = place_of(c, t, &base, &slot, &bad);
    if (bad && blockIdx.y == 0) ++wrong;
    for (int it = (int)blockIdx.y * kWave + lane; it < items; it += (int)gridDim.y * kWave) {
      const int hv = it / chunks, ch = it - hv * chunks;
      const bool is_v = hv >= c.heads;
      const int head = is_v ? hv - c.heads : hv;
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (there) {
        const uint8_t* blk = c.pool + base + (int64_t)head * c.block;
        uint32_t s = 0;
        if constexpr (KIND != LLVQ_KV_BF16) s = blk[(is_v ? c.vs_off : c.ks_off) + slot * c.groups + (ch >> 2)];
        values8<KIND>(blk + (is_v ? c.v_off : 0) + slot * c.row + code_bytes(KIND, ch * 8), s, x);
      }
      store8<F32, VEC>(const_cast<void*>(is_v ? out.v : out.k),
                       (int64_t)t * (is_v ? out.v_token : out.k_token) + (int64_t)head * (is_v ? out.v_head : out.k_head) + ch * 8, x);
    }
  }
  if (wrong && err && lane == 0) atomicAdd(err, wrong);
}

}  // namespace serve
