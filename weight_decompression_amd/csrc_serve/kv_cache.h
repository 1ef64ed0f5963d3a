// The paged key/value cache: quantised as it is written, read back as the values it stands for.
//
// A group of 32 channels of one token and head is held as codes with one power-of-two scale: value = code *
// 2^e, e the smallest integer with max|x| <= top * 2^e (top = 448 for e4m3, 6 for e2m1), held within [-100, 119 or
// 125]: values saturate only within the last factor of f32's range, past top * 2^119 or 2^125.  Dividing by 2^e and
// multiplying back are exact in f32; the only rounding is the code's own, to nearest, ties to even.  A value has at most 4 significant bits and an exponent that e's limits keep
// normal, so it is exact in bf16.  A group with a value that is not finite has the scale byte 255 and reads
// back as NaN.
//
// Both kernels move each byte once and compute little: HBM bounds them.  A wave holds one token or four
// (their sequences, positions and pages are the wave's, found once), one lane 8 channels; four lanes share
// a group. Measured (medians): 12.3 k new tokens of 32 heads of 128 channels, bf16 to e2m1, written in 67 to 73 us
// (3.5 to 3.8 TB/s) and read back in 46 us (5.5); a cache of 8 heads in e4m3 read whole to bf16, 804 MB in and out, in 159 us
// (5.0 TB/s).  A large copy reaches 4.9 TB/s.  Few tokens take 3 us, a launch's least.
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

// STREAM: what is read once does not displace the cache's own lines (a prompt of 12.3 k tokens of 32 heads
// in e2m1: 69 us instead of 82).
template <bool F32, bool VEC, bool STREAM = false>
__device__ __forceinline__ void load8(const void* p, int64_t at, float* x) {
  if constexpr (F32) {
    const float* f = static_cast<const float*>(p) + at;
    if constexpr (VEC) {
      const f32x4* w = reinterpret_cast<const f32x4*>(f);
      const f32x4 a = STREAM ? __builtin_nontemporal_load(w) : w[0], b = STREAM ? __builtin_nontemporal_load(w + 1) : w[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = f[i];
    }
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p) + at;
    if constexpr (VEC) {
      const u32x4* w = reinterpret_cast<const u32x4*>(h);
      const u32x4 a = STREAM ? __builtin_nontemporal_load(w) : w[0];
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

// The places of a wave's PW tokens, and how many have none.
template <int PW>
struct Places {
  int64_t base[PW];
  int slot[PW];
  bool there[PW];
  int wrong = 0;
  __device__ __forceinline__ Places(const Cache& c, int64_t first) {
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      base[i] = 0;
      slot[i] = 0;
      there[i] = false;
      if (first + i < c.tokens) {
        bool bad;
        there[i] = place_of(c, (int)(first + i), &base[i], &slot[i], &bad);
        wrong += bad;
      }
    }
  }
};

// An item: 8 channels of one head's key or value.
struct Item {
  bool is_v;
  int head, ch;
};
__device__ __forceinline__ Item item_of(const Cache& c, int it, const Divider& chunks) {
  const int hv = (int)divide((uint32_t)it, chunks);
  const bool is_v = hv >= c.heads;
  return {is_v, is_v ? hv - c.heads : hv, it - hv * (int)chunks.by};
}

template <int KIND, bool F32, bool VEC, int PW>
__global__ __launch_bounds__(256) void k_kv_write(Cache c, KvRows in, Divider chunks, int items, int32_t* err) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * PW;
  const Places<PW> at(c, first);
  if (err && at.wrong && blockIdx.y == 0 && lane == 0) atomicAdd(err, at.wrong);
  for (int it = (int)blockIdx.y * kWave + lane; it < items; it += (int)gridDim.y * kWave) {
    const Item m = item_of(c, it, chunks);
    const int64_t from = (int64_t)m.head * (m.is_v ? in.v_head : in.k_head) + m.ch * 8;
    float x[PW][8];
#pragma unroll
    for (int i = 0; i < PW; ++i)
      if (at.there[i])
        load8<F32, VEC, true>(m.is_v ? in.v : in.k, (first + i) * (m.is_v ? in.v_token : in.k_token) + from, x[i]);
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      if (!at.there[i]) continue;
      uint8_t* blk = c.pool + at.base[i] + (int64_t)m.head * c.block;
      uint8_t* dst = blk + (m.is_v ? c.v_off : 0) + at.slot[i] * c.row;
      if constexpr (KIND == LLVQ_KV_BF16) {
        store8<false, true>(dst, m.ch * 8, x[i]);
      } else {
        // the group's largest magnitude over its four lanes, as bits: a NaN's and an infinity's are the
        // largest of all
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[i][j]) & 0x7fffffffu);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        const bool nonfinite = top >= 0x7f800000u;
        // e: the exponent of max|x| less the type's, one more where the mantissa passes the type's top
        // (448 = 1.75 * 2^8, 6 = 1.5 * 2^2); a zero or subnormal maximum falls to the lower limit
        constexpr int kExp = KIND == LLVQ_KV_FP8 ? 8 : 2, kHigh = last_scale(KIND) - 127;
        constexpr uint32_t kMant = KIND == LLVQ_KV_FP8 ? 0x600000u : 0x400000u;
        constexpr float kTop = KIND == LLVQ_KV_FP8 ? 448.0f : 6.0f;
        int e = (int)(top >> 23) - 127 - kExp + ((top & 0x7fffffu) > kMant ? 1 : 0);
        e = min(max(e, -100), kHigh);
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = nonfinite ? 0.0f : fminf(fmaxf(x[i][j] * inv, -kTop), kTop);
        if constexpr (KIND == LLVQ_KV_FP8) {
          int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
          lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
          int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
          hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
          *reinterpret_cast<u32x2*>(dst + m.ch * 8) = u32x2{(uint32_t)lo, (uint32_t)hi};
        } else {
          uint32_t w = 0;
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
          *reinterpret_cast<uint32_t*>(dst + m.ch * 4) = w;
        }
        if ((m.ch & 3) == 0) {
          blk[(m.is_v ? c.vs_off : c.ks_off) + at.slot[i] * c.groups + (m.ch >> 2)] = (uint8_t)(nonfinite ? 255 : e + 127);
          if (nonfinite && err) atomicAdd(err, 1);
        }
      }
    }
  }
}

// 8 values from their codes and scale byte.
template <int KIND>
__device__ __forceinline__ void values8(const u32x4 codes, uint32_t scale_byte, float* x) {
  // a byte of 255 (taken for every byte past the last) is an infinite f32, which the conversions turn into NaN for
  // every code
  const float scale = __uint_as_float((scale_byte > (uint32_t)last_scale(KIND) ? 255u : scale_byte) << 23);
  uint32_t u[4];
  if constexpr (KIND == LLVQ_KV_BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = codes[i];
  } else if constexpr (KIND == LLVQ_KV_FP8) {
    u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[0], scale, false));
    u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[0], scale, true));
    u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[1], scale, false));
    u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[1], scale, true));
  } else {
    u[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[0], scale, 0));
    u[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[0], scale, 1));
    u[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[0], scale, 2));
    u[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[0], scale, 3));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

template <int KIND, bool F32, bool VEC, int PW>
__global__ __launch_bounds__(256) void k_kv_read(Cache c, KvRows out, Divider chunks, int items, int32_t* err) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t first = ((int64_t)blockIdx.x * 4 + wave) * PW;
  const Places<PW> at(c, first);
  if (err && at.wrong && blockIdx.y == 0 && lane == 0) atomicAdd(err, at.wrong);
  for (int it = (int)blockIdx.y * kWave + lane; it < items; it += (int)gridDim.y * kWave) {
    const Item m = item_of(c, it, chunks);
    const int64_t to = (int64_t)m.head * (m.is_v ? out.v_head : out.k_head) + m.ch * 8;
    u32x4 codes[PW];
    uint32_t scale[PW];
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      codes[i] = u32x4{0, 0, 0, 0};  // what has no place reads as zeros
      scale[i] = 127;
      if (!at.there[i]) continue;
      const uint8_t* blk = c.pool + at.base[i] + (int64_t)m.head * c.block;
      const uint8_t* src = blk + (m.is_v ? c.v_off : 0) + at.slot[i] * c.row + code_bytes(KIND, m.ch * 8);
      if constexpr (KIND == LLVQ_KV_BF16) {
        codes[i] = *reinterpret_cast<const u32x4*>(src);
      } else {
        if constexpr (KIND == LLVQ_KV_FP8) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(src);
          codes[i][0] = w[0], codes[i][1] = w[1];
        } else {
          codes[i][0] = *reinterpret_cast<const uint32_t*>(src);
        }
        scale[i] = blk[(m.is_v ? c.vs_off : c.ks_off) + at.slot[i] * c.groups + (m.ch >> 2)];
      }
    }
#pragma unroll
    for (int i = 0; i < PW; ++i) {
      if (first + i >= c.tokens) break;
      float x[8];
      values8<KIND>(codes[i], scale[i], x);
      store8<F32, VEC>(const_cast<void*>(m.is_v ? out.v : out.k), (first + i) * (m.is_v ? out.v_token : out.k_token) + to, x);
    }
  }
}

}  // namespace serve
