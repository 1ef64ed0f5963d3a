// Attention of new tokens over the paged cache.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),
//
// over the keys j of the sequence that row i may see, in one pass over the keys: m_i is a running
// maximum, and what was summed under an older maximum is multiplied by exp(old - new).
//
// The queries that share a key head are the columns of one product: row r = t * G + g of a (sequence,
// key head) is token t's g-th query head.  Both products are taken transposed, S^T = K Q^T and
// O^T = V^T P^T, on 32x32x16 bf16 matrix instructions.  In the result layout a lane holds one column
// (lane % 32), so a row's maximum, sum and rescaling are the lane's own (and its partner's, lane ^ 32),
// and S^T's registers are, after exp and packing, P^T's operand without any exchange: a lane holds keys
// 8 * (i / 4) + 4 * (lane / 32) + i % 4, so the second product simply takes its keys in that order, and
// reads V from LDS through the transposing 64-bit load, four keys of one channel at a time.
//
// Codes become bf16 exactly (at most 4 significant bits times a power of two), so staging a tile as bf16 in LDS
// loses nothing.  Scores, maxima, sums and outputs are f32.  P is rounded to bf16 (relative 2^-8 at most, the
// same as the rounding of a bf16 output), and the sum of P is that of the rounded values, so that their
// common part cancels.  For f32 queries both Q and P are split into three bf16 terms
// (x = hi + mid + lo, what is left is below 2^-26 |x|), three matrix instructions in the place of one.
//
// A workgroup has four waves: WK of them share out the keys of a tile, 4 / WK the columns.  Few rows
// (a decode step): WK = 4.  Many rows (a chunk): WK = 1.
#pragma once

#include "kv_cache.h"
#include "serve_common.h"

namespace serve {

struct AttnArgs {
  Cache c;
  const void* q;
  void* out;
  float* part;   // [splits][tokens * heads][dim], unnormalised sums
  float* stats;  // [splits][tokens * heads][2], running maximum (in log2 units) and sum
  int64_t q_token, q_head, out_token, out_head;
  Divider share;  // query heads per key head
  int32_t row_blocks, splits, window, causal, q_vec;
  float scale_log2;
  int32_t* err;
};

constexpr float kRescaleStep = 8.0f;  // log2: how far a maximum may be passed before the sums are rescaled

// Byte offset of 16-byte chunk `ch` of key `row` in a staged tile.  Keys: 16 rows at one chunk (a
// ds_read_b128 of 16 lanes) fall on 16 different slots of 256 bytes.  Values: the four rows that one
// transposing load takes at 64 bytes of channels fall on four different 64-byte segments.
template <int DP>
__device__ __forceinline__ int k_at(int row, int ch) {
  const int sw = DP == 64 ? (row >> 1) & 7 : row & 15;
  return row * (DP * 2) + ((ch ^ sw) << 4);
}
template <int DP>
__device__ __forceinline__ int v_at(int row, int ch) {
  const int sw = DP == 64 ? (((row >> 1) & 1) << 2) | ((row >> 2) & 3) : ((row & 3) << 2) | ((row >> 2) & 3);
  return row * (DP * 2) + ((ch ^ sw) << 4);
}

__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// 16 raw bytes of codes as bf16 chunks of 8 (1, 2 or 4 of them).
template <int KIND>
__device__ __forceinline__ void expand(const u32x4 raw, uint32_t scale_byte, u32x4* o) {
  if constexpr (KIND == LLVQ_KV_BF16) {
    o[0] = raw;
  } else {
    const float scale = __uint_as_float(scale_byte << 23);
    if constexpr (KIND == LLVQ_KV_FP8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i / 2][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[i], scale, false));
        o[i / 2][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(raw[i], scale, true));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[i], scale, 0));
        o[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[i], scale, 1));
        o[i][2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[i], scale, 2));
        o[i][3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(raw[i], scale, 3));
      }
    }
  }
}

template <int NT>
__device__ __forceinline__ void split_terms(const float* x, bf16x8* o) {
  // o[0] the largest term
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r = x[i];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const __bf16 h = (__bf16)r;
      o[n][i] = h;
      if (n + 1 < NT) r -= (float)h;
    }
  }
}

// bf16 elements of four dwords that are not finite, set to zero; whether there was any.  An exponent
// of all ones is the only one that carries into the sign's place when 1 is added to it.
__device__ __forceinline__ bool drop_nonfinite(u32x4* w) {
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) any |= ((*w)[i] & 0x7f807f80u) + 0x00800080u;
  if ((any & 0x80008000u) == 0) return false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t u = (*w)[i];
    if ((u & 0x7f800000u) == 0x7f800000u) u &= 0x0000ffffu;
    if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
    (*w)[i] = u;
  }
  return true;
}

// The sum of a lane's eight p.  bf16 queries: of the rounded values, two at a time, so that what all of a
// row's roundings have in common cancels.
template <int NT>
__device__ __forceinline__ float sum_p(const float* x, const bf16x8& rounded, float l) {
  if constexpr (NT == 1) {
    const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{rounded[2 * e], rounded[2 * e + 1]}, one, l, false);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) l += x[e];
  }
  return l;
}

// Four channels of a cached value where they are not finite, zero where they are.
template <int KIND>
__device__ __forceinline__ f32x4 nonfinite4(const Cache& c, const uint8_t* blk, int slot, int ch) {
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (ch >= c.dim) return x;
  if constexpr (KIND == LLVQ_KV_BF16) {
    const uint16_t* v = reinterpret_cast<const uint16_t*>(blk + c.v_off + slot * c.row) + ch;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((v[i] & 0x7f80u) == 0x7f80u) x[i] = bf16_f32(v[i]);
  } else if (blk[c.vs_off + slot * c.groups + ch / kGroup] == 255) {
    x = f32x4{NAN, NAN, NAN, NAN};
  }
  return x;
}

// The keys of a workgroup: [first_key, last_key), those that every row of it sees, and its share of the
// tiles of `keys` keys (tile indices from key 0).
struct Span {
  int first_key, last_key, all_lo, all_hi, tile_lo, tile_hi;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int row0, int block_rows, int keys, int split) {
  const int rows = s.n * (int)a.share.by;
  const int t0 = (int)divide((uint32_t)row0, a.share);
  const int t1 = (int)divide((uint32_t)(min(row0 + block_rows, rows) - 1), a.share);
  const int p0 = s.len - s.n + t0, p1 = s.len - s.n + t1;
  Span w;
  w.last_key = a.causal ? min(max(p1 + 1, 0), s.len) : s.len;
  w.first_key = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
  w.all_hi = a.causal ? p0 + 1 : s.len;
  w.all_lo = a.window > 0 ? max(p1 - a.window + 1, 0) : 0;
  const int tile0 = w.first_key / keys;
  const int tiles = w.last_key > w.first_key ? (w.last_key + keys - 1) / keys - tile0 : 0;
  const int per = (tiles + a.splits - 1) / a.splits;
  w.tile_lo = tile0 + min(split * per, tiles);
  w.tile_hi = min(w.tile_lo + per, tile0 + tiles);
  return w;
}

// The keys that token t sees: [lo, lo + seen).
__device__ __forceinline__ void seen_of(const AttnArgs& a, const Seq& s, int t, bool live, int* lo, int* seen) {
  const int pos = s.len - s.n + t;
  const int hi = a.causal ? min(max(pos + 1, 0), s.len) : s.len;
  *lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
  *seen = live ? max(hi - *lo, 0) : 0;
}

// 8 channels of a query row as NT bf16 terms.
template <int NT>
__device__ __forceinline__ void load_query(const AttnArgs& a, int64_t at, int ch, bool live, bf16x8* terms) {
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.0f;
  if (live && ch < a.c.dim) {
    if (a.q_vec)
      load8<NT == 3, true>(a.q, at + ch, x);
    else
      load8<NT == 3, false>(a.q, at + ch, x);
  }
  split_terms<NT>(x, terms);
}

// Four channels of one row: to the workspace if the keys are split (unnormalised), else to the output.
template <int NT>
__device__ __forceinline__ void store_row4(const AttnArgs& a, int64_t row, int64_t out_at, int split, int ch, f32x4 x, float inv) {
  const Cache& c = a.c;
  if (ch >= c.dim) return;
  if (a.splits > 1) {
    const int64_t rows = (int64_t)c.tokens * c.heads * a.share.by;
    *reinterpret_cast<f32x4*>(a.part + (split * rows + row) * c.dim + ch) = x;
  } else if constexpr (NT == 1) {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + out_at + ch) =
        u32x2{pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv)};
  } else {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + out_at + ch) = x * inv;
  }
}

// Scores of keys that a row does not see do not count.
__device__ __forceinline__ float masked(float s, int j, int lo, int seen) {
  return (uint32_t)(j - lo) < (uint32_t)seen ? s : -INFINITY;
}

// Few rows: up to 64 rows of a (sequence, key head), in CT tiles of 16 columns.
//
// A decode step reads each cached byte for a handful of rows, so HBM bounds it and what counts is loads
// in flight.  Every wave therefore runs by itself: it takes every fourth 32-key piece of the workgroup's
// share, stages it in its own 64 * DP bytes of LDS (the keys, then the values in the same place) and waits for
// nothing but its own loads, which are issued a piece ahead (page numbers two pieces ahead).  With 16x16x32
// instructions a lane holds 8 scores of a piece, and a tile of outputs takes DP / 4 registers of a lane.
// In S^T's layout a lane (column lane % 16, g = lane / 16) holds keys 4 g + i and 16 + 4 g + i, which are
// taken as the eight consecutive keys of its place in the second product; the transposing load reads
// V's rows in the same order.
// Rows in LDS are padded, so that every address is one register and a constant: by 16 bytes for the keys
// (16 rows at one 16-byte chunk fall on 16 different slots of 256 bytes), by 32 for the values (the eight
// rows that half a wave takes at 32 bytes of channels fall on eight different segments).
template <int DP>
struct FewLds {
  static constexpr int kKeyRow = DP * 2 + 16, kValueRow = DP * 2 + 32;
  static constexpr int kWaveBytes = 32 * kValueRow;
};

__device__ __forceinline__ float quad_max(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quad_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// LDS that only one wave uses: its operations complete in order, so it is enough that the compiler
// keeps them in order.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Waves a SIMD that k_attn_few is compiled for: 512 registers over what it holds (queries, outputs, a piece
// in flight and what goes with it).
constexpr int few_waves(int kind, int dp, int nt, int ct) {
  const int held = nt * ct * (dp / 8 + 4) + ct * (dp / 4 + 15) + code_bytes(kind, dp) / 32 * 14 + 36;
  return held <= 128 ? 4 : held <= 168 ? 3 : held <= 256 ? 2 : 1;
}
// Two column tiles share a staged piece where two waves a SIMD still fit.
constexpr bool few_pairs(int kind, int dp, int nt) { return few_waves(kind, dp, nt, 2) >= 2; }

template <int KIND, int DP, int NT, int CT>
__global__ __launch_bounds__(256, few_waves(KIND, DP, NT, CT)) void k_attn_few(AttnArgs a) {
  constexpr int kRaw = code_bytes(KIND, DP) / 16;  // 16-byte chunks of a row of codes
  constexpr int kLoads = 32 * kRaw / kWave;        // chunks a lane loads of a piece
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;
  constexpr int kSteps = DP / 32, kOut = DP / 16;
  constexpr int32_t kNoKey = INT32_MIN;
  const Cache& c = a.c;
  using Lds = FewLds<DP>;
  __shared__ __align__(16) uint8_t lds[4 * Lds::kWaveBytes];
  __shared__ float wave_m[4][16], wave_l[4][16];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  uint8_t* mine = lds + wave * Lds::kWaveBytes;

  int id = blockIdx.x;
  const int head = id % c.heads;
  id /= c.heads;
  const int split = id % a.splits;
  id /= a.splits;
  const int rb = id % a.row_blocks;
  const int b = id / a.row_blocks;
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, rows = s.n * share;
  if (a.err && tid == 0 && head == 0 && split == 0 && rb == 0 && (s.bad || rows > a.row_blocks * 16 * CT)) atomicAdd(a.err, 1);
  const int row0 = rb * 16 * CT;
  if (row0 >= rows) return;
  const Span w = span_of(a, s, row0, 16 * CT, 128, split);

  int lo[CT], seen[CT], t[CT], qhead[CT];
  bool live[CT];
  bf16x8 q[NT][CT][kSteps];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = row0 + ct * 16 + col;
    live[ct] = row < rows;
    t[ct] = live[ct] ? (int)divide((uint32_t)row, a.share) : 0;
    qhead[ct] = head * share + (live[ct] ? row - t[ct] * share : 0);
    seen_of(a, s, t[ct], live[ct], &lo[ct], &seen[ct]);
    const int64_t at = (int64_t)(s.first + t[ct]) * a.q_token + (int64_t)qhead[ct] * a.q_head;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      bf16x8 terms[NT];
      load_query<NT>(a, at, st * 32 + g * 8, live[ct], terms);
#pragma unroll
      for (int n = 0; n < NT; ++n) q[n][ct][st] = terms[n];
    }
  }

  f32x4 acc[CT][kOut];
  float m[CT], l[CT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    m[ct] = -INFINITY;
    l[ct] = 0.0f;
#pragma unroll
    for (int d = 0; d < kOut; ++d) acc[ct][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  const int64_t head_off = (int64_t)head * c.block, page_bytes = (int64_t)c.heads * c.block;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  const int ch = lane % kRaw;  // this lane's chunk of every row that it loads
  const bool in_row = ch * 16 < c.row;
  bool lost = false;
  // the page number of this lane's key of a piece (lanes 32..63 as 0..31)
  auto page_of = [&](int tile) -> int32_t {
    const int j = (tile * 4 + wave) * 32 + (lane & 31);
    if (tile >= w.tile_hi || j < w.first_key || j >= w.last_key) return kNoKey;
    return table[divide((uint32_t)j, c.page)];
  };
  // codes and scale bytes of a piece: row i of a lane is key (i * 64 + lane) / kRaw
  int64_t base[kLoads];
  int slot[kLoads];
  bool ok[kLoads];
  u32x4 raw[2][kLoads];
  uint32_t sc[2][kLoads];
  auto locate = [&](int tile, int32_t ids) {
    lost |= ids >= c.pages || (ids < 0 && ids != kNoKey);
    const uint32_t j = (uint32_t)((tile * 4 + wave) * 32 + (lane & 31));
    const int my_slot = (int)(j - divide(j, c.page) * c.page.by);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * kWave + lane) / kRaw;
      const int32_t page = __shfl(ids, key);
      slot[i] = __shfl(my_slot, key);
      ok[i] = page >= 0 && page < c.pages && in_row;
      // a place that is not there is read from the pool's start and left out when it is staged
      if (!ok[i]) slot[i] = 0;
      base[i] = ok[i] ? (int64_t)page * page_bytes + head_off : 0;
    }
  };
  auto fetch = [&](int is_v) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint8_t* blk = c.pool + base[i];
      raw[is_v][i] = *reinterpret_cast<const u32x4*>(blk + (is_v ? c.v_off : 0) + slot[i] * c.row + (ok[i] ? ch * 16 : 0));
      if constexpr (KIND != LLVQ_KV_BF16)
        sc[is_v][i] = blk[(is_v ? c.vs_off : c.ks_off) + slot[i] * c.groups + (ok[i] ? ch * kOf / 4 : 0)];
      else
        sc[is_v][i] = 127;
    }
  };
  bool part_k = false, part_v = false;  // whether a place of the loaded piece is not there

  int32_t ids = page_of(w.tile_lo);
  bool there_k[kLoads], there_v[kLoads];
  auto note = [&](bool* there, bool* part) {
    bool all = true;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      there[i] = ok[i];
      all &= ok[i];
    }
    *part = !__all(all);
  };
  if (w.tile_lo < w.tile_hi) {
    locate(w.tile_lo, ids);
    note(there_k, &part_k);
    note(there_v, &part_v);
    fetch(0);
    fetch(1);
    ids = page_of(w.tile_lo + 1);
  }
  for (int tile = w.tile_lo; tile < w.tile_hi; ++tile) {
    const int key_base = (tile * 4 + wave) * 32;
    const bool more = tile + 1 < w.tile_hi;
    // the keys
    wave_order();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * kWave + lane) / kRaw;
      u32x4 r = raw[0][i];
      uint32_t sb = sc[0][i];
      if (part_k && !there_k[i]) r = u32x4{0, 0, 0, 0}, sb = 127;
      u32x4 o[kOf];
      expand<KIND>(r, sb, o);
#pragma unroll
      for (int n = 0; n < kOf; ++n) *reinterpret_cast<u32x4*>(mine + key * Lds::kKeyRow + (ch * kOf + n) * 16) = o[n];
    }
    wave_order();
    if (more) {
      locate(tile + 1, ids);
      ids = page_of(tile + 2);
      note(there_k, &part_k);
      fetch(0);
    }
    f32x4 score[CT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) score[ct][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(mine + (u * 16 + col) * Lds::kKeyRow + (st * 4 + g) * 16);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int n = NT - 1; n >= 0; --n) score[ct][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[n][ct][st], score[ct][u], 0, 0, 0);
      }
    }
    const bool whole = key_base >= w.all_lo && key_base + 32 <= w.all_hi && key_base + 32 <= s.len;
    bf16x8 p[NT][CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) score[ct][u][i] = masked(score[ct][u][i], key_base + u * 16 + 4 * g + i, lo[ct], seen[ct]);
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, score[ct][i / 4][i & 3]);
      top = quad_max(top) * a.scale_log2;
      if (__any(top > m[ct] + kRescaleStep)) {
        const float next = fmaxf(m[ct], top);
        const float f = m[ct] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[ct] - next);
        m[ct] = next;
        l[ct] *= f;
#pragma unroll
        for (int d = 0; d < kOut; ++d) acc[ct][d] *= f;
      }
      const float ms = m[ct] == -INFINITY ? 0.0f : m[ct];
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_exp2f(fmaf(score[ct][i / 4][i & 3], a.scale_log2, -ms));
      bf16x8 terms[NT];
      split_terms<NT>(x, terms);
      l[ct] = sum_p<NT>(x, terms[0], l[ct]);
#pragma unroll
      for (int n = 0; n < NT; ++n) p[n][ct] = terms[n];
    }
    // the values, in the keys' place
    uint32_t bad = 0;
    wave_order();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * kWave + lane) / kRaw;
      u32x4 r = raw[1][i];
      uint32_t sb = sc[1][i];
      if (part_v && !there_v[i]) r = u32x4{0, 0, 0, 0}, sb = 127;
      u32x4 o[kOf];
      bool spoilt;
      if constexpr (KIND == LLVQ_KV_BF16) {
        spoilt = drop_nonfinite(&r);
      } else {
        spoilt = sb == 255;
        if (spoilt) r = u32x4{0, 0, 0, 0}, sb = 127;
      }
      if (spoilt) bad |= 1u << key;
      expand<KIND>(r, sb, o);
#pragma unroll
      for (int n = 0; n < kOf; ++n) *reinterpret_cast<u32x4*>(mine + key * Lds::kValueRow + (ch * kOf + n) * 16) = o[n];
    }
    wave_order();
    if (more) {
      note(there_v, &part_v);
      fetch(1);
    }
#pragma unroll
    for (int d = 0; d < kOut; ++d) {
      const uint8_t* at = mine + (4 * g + ((lane & 15) >> 2)) * Lds::kValueRow + d * 32 + (lane & 3) * 8;
      union {
        s16x4 h[2];
        bf16x8 v;
      } vf;
      vf.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
      vf.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 16 * Lds::kValueRow));
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) acc[ct][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf.v, p[n][ct], acc[ct][d], 0, 0, 0);
    }
    // values that are not finite were left out (0 * NaN would spoil rows that do not see them) and are
    // added to the rows that do
    if (__any(bad != 0)) {
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) bad |= (uint32_t)__shfl_xor((int)bad, d);
      while (bad) {
        const int key = __builtin_ctz(bad), j = key_base + key;
        bad &= bad - 1;
        const uint32_t page = divide((uint32_t)j, c.page);
        const int at = j - (int)(page * c.page.by);
        const uint8_t* blk = c.pool + (int64_t)table[page] * page_bytes + head_off;
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
          const f32x4 x = nonfinite4<KIND>(c, blk, at, d * 16 + 4 * g);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct)
            if ((uint32_t)(j - lo[ct]) < (uint32_t)seen[ct]) acc[ct][d] += x;
        }
      }
    }
  }
  if (a.err && lost) atomicAdd(a.err, 1);

  // the four waves' parts are joined through LDS under their common maximum and added in the waves' order
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    l[ct] = quad_sum(l[ct]);
    __syncthreads();
    if (g == 0) wave_m[wave][col] = m[ct];
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, wave_m[i][col]);
    const float f = m[ct] == -INFINITY ? (l[ct] == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(m[ct] - top);
    if (g == 0) wave_l[wave][col] = l[ct] * f;
    float* sums = reinterpret_cast<float*>(lds);  // [wave][16 columns][DP], quads of channels swizzled by the column
#pragma unroll
    for (int d = 0; d < kOut; ++d)
      *reinterpret_cast<f32x4*>(sums + (wave * 16 + col) * DP + (((d * 4 + g) ^ (col & 7)) << 2)) = acc[ct][d] * f;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) total += wave_l[i][col];
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;  // no visible key: the row is zero
    if (live[ct]) {
      const int64_t row = (int64_t)(s.first + t[ct]) * c.heads * share + qhead[ct];
      const int64_t out_at = (int64_t)(s.first + t[ct]) * a.out_token + (int64_t)qhead[ct] * a.out_head;
      if (a.splits > 1 && wave == 0 && g == 0) {
        const int64_t all = (int64_t)c.tokens * c.heads * share;
        a.stats[(split * all + row) * 2] = top;
        a.stats[(split * all + row) * 2 + 1] = total;
      }
      if (a.splits == 1 || w.tile_lo < w.tile_hi) {
#pragma unroll
        for (int d4 = 0; d4 < kOut / 4; ++d4) {
          const int d = d4 * 4 + wave;  // each wave writes a quarter of the channels
          f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < 4; ++i) x += *reinterpret_cast<const f32x4*>(sums + (i * 16 + col) * DP + (((d * 4 + g) ^ (col & 7)) << 2));
          store_row4<NT>(a, row, out_at, split, d * 16 + g * 4, x, inv);
        }
      }
    }
  }
}

// Many rows: the tiles are shared by the workgroup's four waves, each with 32 columns of its own.
template <int KIND, int DP, int NT, int WK>
struct AttnShape {
  static constexpr int kWaveCols = 4 / WK;
  static constexpr int kRows = 32 * kWaveCols;              // rows (columns of S^T) of a workgroup
  static constexpr int kSub = WK == 1 ? 2 : 1;              // 32-key pieces of a wave in a tile
  static constexpr int kKeys = 32 * kSub * WK;              // keys of a tile
  static constexpr int kTile = kKeys * DP * 2;              // bytes of the staged keys, and of the values
  static constexpr int kRawRow = code_bytes(KIND, DP) / 16;  // 16-byte chunks of a row of codes
  static constexpr int kChunks = kKeys * kRawRow;
  static constexpr int kPer = (kChunks + 255) / 256;        // chunks a thread stages
  static constexpr int kJoin = WK > 1 ? 4 * 32 * DP * 4 : 0;  // the waves' sums, in the tiles' place
  static constexpr int kLds = 2 * kTile > kJoin ? 2 * kTile : kJoin;
};

template <int KIND, int DP, int NT, int WK>
__global__ __launch_bounds__(256) void k_attn(AttnArgs a) {
  using Sh = AttnShape<KIND, DP, NT, WK>;
  constexpr int kKeys = Sh::kKeys, kSub = Sh::kSub, kSteps = DP / 16, kOut = DP / 32;
  const Cache& c = a.c;
  __shared__ __align__(16) uint8_t lds[Sh::kLds];
  uint8_t* lds_k = lds;
  uint8_t* lds_v = lds + Sh::kTile;
  __shared__ uint32_t bad_keys[2][4];
  __shared__ __align__(16) float poison[DP];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = wave % WK, wq = wave / WK;
  const int half = lane >> 5, col = lane & 31;

  int id = blockIdx.x;
  const int head = id % c.heads;
  id /= c.heads;
  const int split = id % a.splits;
  id /= a.splits;
  const int rb = a.row_blocks - 1 - id % a.row_blocks;  // the longest rows of a causal chunk first
  const int b = id / a.row_blocks;
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, rows = s.n * share;
  if (a.err && tid == 0 && head == 0 && split == 0 && rb == 0 && (s.bad || rows > a.row_blocks * Sh::kRows))
    atomicAdd(a.err, 1);
  const int row0 = rb * Sh::kRows;
  if (row0 >= rows) return;

  // this lane's row, and the keys it sees: [lo, lo + seen)
  const int row = row0 + wq * 32 + col;
  const bool live = row < rows;
  const int t = live ? (int)divide((uint32_t)row, a.share) : 0;
  const int qhead = head * share + (live ? row - t * share : 0);
  const int pos = s.len - s.n + t;
  const int hi = a.causal ? min(max(pos + 1, 0), s.len) : s.len;
  const int lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
  const int seen = live ? max(hi - lo, 0) : 0;

  // the workgroup's keys: [first_key, last_key), and those that every row of it sees
  const int t0 = (int)divide((uint32_t)row0, a.share);
  const int t1 = (int)divide((uint32_t)(min(row0 + Sh::kRows, rows) - 1), a.share);
  const int p0 = s.len - s.n + t0, p1 = s.len - s.n + t1;
  const int last_key = a.causal ? min(max(p1 + 1, 0), s.len) : s.len;
  const int first_key = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
  const int all_hi = a.causal ? p0 + 1 : s.len;
  const int all_lo = a.window > 0 ? max(p1 - a.window + 1, 0) : 0;
  const int key0 = first_key / kKeys;
  const int tiles = last_key > first_key ? (last_key + kKeys - 1) / kKeys - key0 : 0;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int tile_lo = min(split * per, tiles), tile_hi = min(tile_lo + per, tiles);

  // the queries, as the second operand of S^T: 8 consecutive channels of the lane's column
  bf16x8 q[NT][kSteps];
  {
    const int64_t at = (int64_t)(s.first + t) * a.q_token + (int64_t)qhead * a.q_head;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      const int ch = st * 16 + half * 8;
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.0f;
      if (live && ch < c.dim) {
        if constexpr (NT == 1) {
          if (a.q_vec)
            load8<false, true>(a.q, at + ch, x);
          else
            load8<false, false>(a.q, at + ch, x);
        } else {
          if (a.q_vec)
            load8<true, true>(a.q, at + ch, x);
          else
            load8<true, false>(a.q, at + ch, x);
        }
      }
      bf16x8 terms[NT];
      split_terms<NT>(x, terms);
#pragma unroll
      for (int n = 0; n < NT; ++n) q[n][st] = terms[n];
    }
  }

  f32x16 acc[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) acc[i] = f32x16{0.0f};
  float m = -INFINITY, l = 0.0f;

  u32x4 raw_k[Sh::kPer], raw_v[Sh::kPer];
  uint32_t sc_k[Sh::kPer], sc_v[Sh::kPer];
  bool lost = false;
  auto fetch = [&](int tile) {
#pragma unroll
    for (int i = 0; i < Sh::kPer; ++i) {
      const int chunk = tid + i * 256;
      const int key = chunk / Sh::kRawRow, ch = chunk % Sh::kRawRow;
      const int j = (key0 + tile) * kKeys + key;
      raw_k[i] = raw_v[i] = u32x4{0, 0, 0, 0};
      sc_k[i] = sc_v[i] = 127;
      if (chunk < Sh::kChunks && j >= first_key && j < last_key && ch * 16 < c.row) {
        const uint32_t page = divide((uint32_t)j, c.page);
        const int slot = j - (int)(page * c.page.by);
        const int64_t base = block_of(c, b, page, head);
        if (base >= 0) {
          const uint8_t* blk = c.pool + base;
          raw_k[i] = *reinterpret_cast<const u32x4*>(blk + slot * c.row + ch * 16);
          raw_v[i] = *reinterpret_cast<const u32x4*>(blk + c.v_off + slot * c.row + ch * 16);
          if constexpr (KIND != LLVQ_KV_BF16) {
            const int g = KIND == LLVQ_KV_FP8 ? ch >> 1 : ch;
            sc_k[i] = blk[c.ks_off + slot * c.groups + g];
            sc_v[i] = blk[c.vs_off + slot * c.groups + g];
          }
        } else {
          lost = true;
        }
      }
    }
  };
  auto stage = [&](int par) {
#pragma unroll
    for (int i = 0; i < Sh::kPer; ++i) {
      const int chunk = tid + i * 256;
      if (chunk < Sh::kChunks) {
        const int key = chunk / Sh::kRawRow, ch = chunk % Sh::kRawRow;
        constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;
        u32x4 o[kOf];
        expand<KIND>(raw_k[i], sc_k[i], o);
#pragma unroll
        for (int n = 0; n < kOf; ++n) *reinterpret_cast<u32x4*>(lds_k + k_at<DP>(key, ch * kOf + n)) = o[n];
        // values that are not finite would spoil rows that do not see them (0 * NaN): they are left
        // out here and added to the rows that do see them after the tile's products
        bool bad;
        if constexpr (KIND == LLVQ_KV_BF16) {
          o[0] = raw_v[i];
          bad = drop_nonfinite(&o[0]);
        } else {
          bad = sc_v[i] == 255;
          expand<KIND>(bad ? u32x4{0, 0, 0, 0} : raw_v[i], bad ? 127 : sc_v[i], o);
        }
        if (bad) atomicOr(&bad_keys[par][key >> 5], 1u << (key & 31));
#pragma unroll
        for (int n = 0; n < kOf; ++n) *reinterpret_cast<u32x4*>(lds_v + v_at<DP>(key, ch * kOf + n)) = o[n];
      }
    }
  };

  if (tid < 8) bad_keys[tid >> 2][tid & 3] = 0;
  if (tile_lo < tile_hi) fetch(tile_lo);
  int par = 0;
  for (int tile = tile_lo; tile < tile_hi; ++tile, par ^= 1) {
    __syncthreads();  // the last tile has been read
    stage(par);
    __syncthreads();
    if (tile + 1 < tile_hi) fetch(tile + 1);

    const int key_base = (key0 + tile) * kKeys;
    const bool whole = key_base >= all_lo && key_base + kKeys <= all_hi && key_base + kKeys <= s.len;
    f32x16 sc[kSub];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const int krow = (wk * kSub + u) * 32 + col;
      sc[u] = f32x16{0.0f};
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(lds_k + k_at<DP>(krow, st * 2 + half));
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) sc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, q[n][st], sc[u], 0, 0, 0);
      }
    }
    if (!whole) {
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = key_base + (wk * kSub + u) * 32 + 8 * (i / 4) + 4 * half + (i & 3);
          sc[u][i] = (uint32_t)(j - lo) < (uint32_t)seen ? sc[u][i] : -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[u][i]);
    top = half_max(top) * a.scale_log2;
    // The maximum is raised only when it is passed by 2^8: p stays below 2^8 and its rounding is
    // relative, so the result is the same, and most tiles skip the rescaling of O.
    if (__any(top > m + kRescaleStep)) {
      const float next = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - next);
      m = next;
      l *= f;
#pragma unroll
      for (int i = 0; i < kOut; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] *= f;
    }
    const float ms = m == -INFINITY ? 0.0f : m;
    bf16x8 p[NT][kSub * 2];
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = __builtin_amdgcn_exp2f(fmaf(sc[u][h2 * 8 + e], a.scale_log2, -ms));
          if constexpr (NT > 1) l += x[e];
        }
        bf16x8 terms[NT];
        split_terms<NT>(x, terms);
        // the sum takes the rounded values, two at a time: what all of a row's roundings have in common cancels
        if constexpr (NT == 1) {
          const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{terms[0][2 * e], terms[0][2 * e + 1]}, one, l, false);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) p[n][u * 2 + h2] = terms[n];
      }
#pragma unroll
    for (int d = 0; d < kOut; ++d)
#pragma unroll
      for (int u = 0; u < kSub * 2; ++u) {
        const int vrow = wk * kSub * 32 + u * 16 + 4 * half + ((lane & 15) >> 2);
        const int ch = d * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
        const int in = (lane & 1) * 8;
        union {
          s16x4 h[2];
          bf16x8 v;
        } vf;
        vf.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lds_v + v_at<DP>(vrow, ch) + in));
        vf.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(lds_v + v_at<DP>(vrow + 8, ch) + in));
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf.v, p[n][u], acc[d], 0, 0, 0);
      }
    // values that are not finite, added to the rows that see them
    for (int w = 0; w < kKeys / 32; ++w) {
      uint32_t left = bad_keys[par][w];
      while (left) {
        const int key = w * 32 + __builtin_ctz(left);
        left &= left - 1;
        const int j = key_base + key;
        __syncthreads();
        const uint32_t page = divide((uint32_t)j, c.page);
        const int slot = j - (int)(page * c.page.by);
        const int64_t base = block_of(c, b, page, head);
        if (tid < DP) {
          float x = 0.0f;
          if (tid < c.dim && base >= 0) {
            const uint8_t* blk = c.pool + base;
            if constexpr (KIND == LLVQ_KV_BF16) {
              x = bf16_f32(reinterpret_cast<const uint16_t*>(blk + c.v_off + slot * c.row)[tid]);
              if ((__float_as_uint(x) & 0x7f800000u) != 0x7f800000u) x = 0.0f;
            } else {
              x = blk[c.vs_off + slot * c.groups + tid / kGroup] == 255 ? NAN : 0.0f;
            }
          }
          poison[tid] = x;
        }
        __syncthreads();
        if (key / (32 * kSub) == wk && (uint32_t)(j - lo) < (uint32_t)seen) {
#pragma unroll
          for (int d = 0; d < kOut; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] += poison[d * 32 + 8 * (i / 4) + 4 * half + (i & 3)];
        }
      }
    }
    if (tid < 4) bad_keys[par ^ 1][tid] = 0;
  }
  if (a.err && lost) atomicAdd(a.err, 1);

  l = half_sum(l);
  if constexpr (WK > 1) {
    // the waves that shared out the keys are joined through LDS: each brings its sums under the common
    // maximum and the sums are added in the waves' order
    __shared__ float wave_m[4][32], wave_l[4][32];
    __syncthreads();
    if (half == 0) wave_m[wave][col] = m;
    __syncthreads();
    float top = m;
#pragma unroll
    for (int w = 0; w < WK; ++w) top = fmaxf(top, wave_m[wq * WK + w][col]);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
    m = top;
    if (half == 0) wave_l[wave][col] = l * f;
    float* sums = reinterpret_cast<float*>(lds);  // [wave][32 columns][DP], quads of channels swizzled by the column
#pragma unroll
    for (int d = 0; d < kOut; ++d)
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const int quad = (d * 8 + i4 * 2 + half) ^ (col & 7);
        *reinterpret_cast<f32x4*>(sums + (wave * 32 + col) * DP + quad * 4) =
            f32x4{acc[d][i4 * 4] * f, acc[d][i4 * 4 + 1] * f, acc[d][i4 * 4 + 2] * f, acc[d][i4 * 4 + 3] * f};
      }
    __syncthreads();
    l = 0.0f;
#pragma unroll
    for (int w = 0; w < WK; ++w) l += wave_l[wq * WK + w][col];
    if (wk == 0) {
#pragma unroll
      for (int d = 0; d < kOut; ++d)
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const int quad = (d * 8 + i4 * 2 + half) ^ (col & 7);
          f32x4 x = *reinterpret_cast<const f32x4*>(sums + (wave * 32 + col) * DP + quad * 4);
#pragma unroll
          for (int w = 1; w < WK; ++w) x += *reinterpret_cast<const f32x4*>(sums + ((wave + w) * 32 + col) * DP + quad * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[d][i4 * 4 + i] = x[i];
        }
    }
    if (wk != 0) return;
  }
  if (!live) return;
  if (a.splits > 1) {
    const int64_t at = (int64_t)split * c.tokens * c.heads * share + (int64_t)(s.first + t) * c.heads * share + qhead;
    if (half == 0) {
      a.stats[at * 2] = m;
      a.stats[at * 2 + 1] = l;
    }
    if (tile_lo >= tile_hi) return;
#pragma unroll
    for (int d = 0; d < kOut; ++d)
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const int ch = d * 32 + i4 * 8 + half * 4;
        if (ch < c.dim)
          *reinterpret_cast<f32x4*>(a.part + at * c.dim + ch) =
              f32x4{acc[d][i4 * 4], acc[d][i4 * 4 + 1], acc[d][i4 * 4 + 2], acc[d][i4 * 4 + 3]};
      }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no visible key: the row is zero
  const int64_t at = (int64_t)(s.first + t) * a.out_token + (int64_t)qhead * a.out_head;
#pragma unroll
  for (int d = 0; d < kOut; ++d)
#pragma unroll
    for (int i4 = 0; i4 < 4; ++i4) {
      const int ch = d * 32 + i4 * 8 + half * 4;
      if (ch < c.dim) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = acc[d][i4 * 4 + i] * inv;
        if constexpr (NT == 1)
          *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at + ch) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
        else
          *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at + ch) = f32x4{x[0], x[1], x[2], x[3]};
      }
    }
}

// Joins the splits of a row under their common maximum.  A lane first takes the maximum and sum of two
// splits, so that the weights of all are known after one round of loads; then 64 / LANES splits of a wave
// are read side by side, four channels a lane, and what the waves of a row have is added in order through LDS.  WAVES
// waves a row: one where rows are many and splits few, four where a long axis left few rows of many splits.
constexpr int kMaxSplits = 128;

template <bool F32, int LANES, int WAVES>
__global__ __launch_bounds__(256) void k_attn_join(AttnArgs a) {
  constexpr int kSide = kWave / LANES;
  const Cache& c = a.c;
  __shared__ __align__(16) float sums[4][kSide][LANES * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int heads = c.heads * (int)a.share.by;
  const int64_t rows = (int64_t)c.tokens * heads, row = ((int64_t)blockIdx.x * 4 + wave) / WAVES;
  const bool in = row < rows;
  const int64_t t = in ? row / heads : 0, head = in ? row - t * heads : 0;
  // rows that belong to no sequence are not written
  const int b = sequence_of(c, (int)t);
  const Seq s = b < c.batch ? sequence(c, b) : Seq{0, 0, 0, true};
  const bool live = in && t >= s.first && t < s.first + s.n;

  float ms[2], ls[2], f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int sp = i * kWave + lane;
    const bool there = live && sp < a.splits;
    ms[i] = there ? a.stats[(sp * rows + row) * 2] : -INFINITY;
    ls[i] = there ? a.stats[(sp * rows + row) * 2 + 1] : 0.0f;
  }
  float top = fmaxf(ms[0], ms[1]), l = 0.0f;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // a split that a row sees nothing of wrote no sums that count: weight zero, and it is not read
    f[i] = ms[i] == -INFINITY ? (ls[i] == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(ms[i] - top);
    if (ms[i] == -INFINITY && ls[i] == 0.0f) f[i] = -1.0f;
    else l += ls[i] * f[i];
  }
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) l += __shfl_xor(l, d);

  const int side = lane / LANES, ch = (lane % LANES) * 4, part = wave % WAVES;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int i0 = part * kSide; i0 < a.splits; i0 += WAVES * kSide * 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * WAVES * kSide + side;
      const float w = __shfl(i < kWave ? f[0] : f[1], i & 63);
      if (i < a.splits && w >= 0.0f && ch < c.dim && live)
        x += *reinterpret_cast<const f32x4*>(a.part + (i * rows + row) * c.dim + ch) * w;
      else if (i < a.splits && w != w)
        x += w;
    }
  }
  if constexpr (kSide > 1 || WAVES > 1) {
    *reinterpret_cast<f32x4*>(&sums[wave][side][ch]) = x;
    __syncthreads();
    if (part != 0 || side != 0) return;
    x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < WAVES; ++i)
#pragma unroll
      for (int j = 0; j < kSide; ++j) x += *reinterpret_cast<const f32x4*>(&sums[wave + i][j][ch]);
  }
  if (!live || ch >= c.dim) return;
  x *= l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t at = t * a.out_token + head * a.out_head + ch;
  if constexpr (F32)
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at) = x;
  else
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + at) = u32x2{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3])};
}

}  // namespace serve
