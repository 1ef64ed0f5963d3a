// Attention of new tokens over the paged cache.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale q_i . k_j - m_i),
//
// over the keys j of the sequence that row i may see, in one pass over the keys: m_i is a running maximum,
// and what was summed under an older maximum is multiplied by exp(old - new).
//
// The queries that share a key head are the columns of one product: row r = t * G + g of a (sequence, key
// head) is token t's g-th query head.  Both products are taken transposed, S^T = K Q^T and O^T = V^T P^T,
// on bf16 matrix instructions (32x32x16 for many rows, 16x16x32 for few).  In the result layout of the
// first a lane holds one column (lane % 32), so a row's maximum, sum and rescaling are the lane's own (and
// its partner's, lane ^ 32), and S^T's registers are, after exp and packing, P^T's operand without any
// exchange: a lane holds keys 8 * (i / 4) + 4 * (lane / 32) + i % 4, so the second product simply takes its
// keys in that order, and reads V from LDS through the transposing 64-bit load, four keys of one channel at
// a time.
//
// Codes become bf16 exactly (at most 4 significant bits times a power of two), so staging a tile as bf16 in
// LDS loses nothing.  Scores, maxima, sums and outputs are f32.  For f32 queries both Q and P are split into three
// bf16 terms (x = hi + mid + lo, what is left is below 2^-26 |x|), three matrix instructions in the place of one.  For
// bf16 queries of few rows P is split into two (2^-17), so that the output's rounding is the only one that counts;
// that costs 1 % of a decode step in e4m3 (268 us, 271), 3 % in e2m1 (77.6, 80.2) and up to 12 % where two tiles of
// shared heads read e2m1 (4 new tokens of 64 sequences, 64 heads over 8: 71.9, 80.6).  Of many rows, where the matrix
// instructions are the bound and a second term would cost a quarter, P is rounded to bf16 (relative 2^-8 at most, as a
// bf16 output is), and the sum of P is that of the rounded values, so that their common part cancels: the error
// against 64 bits is 0.0021 of the result's norm, 0.0017 from the output's rounding alone.
//
// Two kernels share this: k_attn_few for up to 64 rows of a (sequence, key head), where a workgroup's waves
// share out the keys, and k_attn_many, where they share out the rows.
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
  int32_t row_blocks, splits, units, window, causal, q_vec;  // units: row blocks of all sequences and splits
  float scale_log2;
  int32_t* err;
  const int32_t* parents;  // kTree: [tokens]
  float* lse;              // kLse: [tokens][heads]
};

// Forms of the kernels.  kTree: a sequence's new tokens are the nodes of a tree, and a node sees the text before them
// and the nodes above it; only the pieces that hold nodes look at its set (8 trees of 64 nodes of 64 heads over up to 16384 keys in
// e2m1: 250 us, 238 for as many causal rows; 16 of up to 32 of 32 heads over up to 4096 in e4m3, f32: 100 and 99).  kLse: log sum_j
// exp(scale q_i . k_j) of every row is written as well (a decode step costs nothing more, chunks of 2 x 2048 over 8192 502 us
// instead of 480: the sum of p before it is rounded is kept beside the other).
enum { kPlain, kTree, kLse };

// What each node of a sequence's tree sees of the others, itself included: lane i holds node i's set, and its depth.
// A lane starts with its node and its parent; in each round it takes over what its 2^k-th ancestor has found, so a
// tree of depth 7 takes three rounds of shuffles, where the walk up would wait for a load a step.
struct Node {
  uint64_t above;
  int depth;
  bool bad;  // a parent that is not an earlier node (taken as none), or more nodes than a tree may have
};
__device__ __forceinline__ Node node_of(const AttnArgs& a, const Seq& s) {
  const int lane = threadIdx.x & 63;
  const bool in = lane < s.n;
  int up = in ? a.parents[s.first + lane] : -1;
  Node x;
  x.bad = up < -1 || up >= lane || s.n > LLVQ_MAX_NODES;
  if (up < -1 || up >= lane) up = -1;
  x.above = in ? 1ull << lane : 0;
  while (__any(up >= 0)) {
    const uint64_t more = (uint64_t)__shfl((unsigned long long)x.above, up & 63);
    const int next = __shfl(up, up & 63);
    if (up >= 0) x.above |= more, up = next;
  }
  x.depth = in ? __popcll(x.above) - 1 : 0;
  // parents come before their children: the nearest are the highest bits
  if (a.window > 0)
    for (int over = x.depth + 1 - a.window; over > 0; --over) x.above &= x.above - 1;
  return x;
}

__device__ __forceinline__ float log_sum(float m, float l) {  // of a maximum in log2 units and the sum under it
  return l == 0.0f ? -INFINITY : ((m == -INFINITY ? 0.0f : m) + __builtin_amdgcn_logf(l)) * 0.6931471805599453f;
}

constexpr float kRescaleStep = 8.0f;  // log2: how far a maximum may be passed before the sums are rescaled

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

// 16 bytes of value codes that are not finite by themselves: bf16 infinities and NaN, of which an exponent of all
// ones is the only one that carries into the sign's place when 1 is added to it, and the e4m3 NaN, 0x7f and 0xff,
// of which the same holds for all seven bits.  e2m1 has none.
constexpr uint32_t odd_bits(int kind) { return kind == LLVQ_KV_BF16 ? 0x80008000u : kind == LLVQ_KV_FP8 ? 0x80808080u : 0; }
template <int KIND>
__device__ __forceinline__ uint32_t odd_codes(uint32_t w) {  // odd_bits at those
  return KIND == LLVQ_KV_BF16 ? (w & 0x7f807f80u) + 0x00800080u : (w & 0x7f7f7f7fu) + 0x01010101u;
}

// Those of a wave's chunks set to zero; whether there was any (the same in every lane).  Where there is none, in
// all but damaged caches, this takes three operations a dword and one branch.
template <int KIND, int N>
__device__ __forceinline__ bool drop_odd(u32x4* raw) {
  if constexpr (KIND == LLVQ_KV_FP4) return false;
  uint32_t any = 0;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) any |= odd_codes<KIND>(raw[n][i]);
  if (!__any((any & odd_bits(KIND)) != 0)) return false;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w = raw[n][i];
      asm volatile("" : "+v"(w));  // (so that what was worked out above is not kept for here)
      constexpr int kBits = KIND == LLVQ_KV_BF16 ? 16 : 8;
      raw[n][i] = w & ~(((odd_codes<KIND>(w) & odd_bits(KIND)) >> (kBits - 1)) * ((1u << kBits) - 1));
    }
  return true;
}

// A lane's eight p, added to its four sums.  Where one term is all of P: the rounded values, two at a time, so that what
// all of a row's roundings have in common cancels.
template <int TERMS>
__device__ __forceinline__ void sum_p(const float* x, const bf16x8& rounded, float* l4) {
  if constexpr (TERMS == 1) {
    const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) l4[e] = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{rounded[2 * e], rounded[2 * e + 1]}, one, l4[e], false);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) l4[e & 3] += x[e];
  }
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
  } else {
    const bool all = blk[c.vs_off + slot * c.groups + ch / kGroup] > last_scale(KIND);
    const uint32_t codes = KIND == LLVQ_KV_FP8 ? *reinterpret_cast<const uint32_t*>(blk + c.v_off + slot * c.row + ch) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (all || (codes >> (8 * i) & 0x7fu) == 0x7fu) x[i] = NAN;
  }
  return x;
}

// The keys of a workgroup: [first_key, last_key), those that every row of it sees, and its share of the
// tiles of `keys` keys (tile indices from key 0).
struct Span {
  int first_key, last_key, all_lo, all_hi, tile_lo, tile_hi;
};
template <int MODE>
__device__ __forceinline__ Span span_of(const AttnArgs& a, const Seq& s, int row0, int block_rows, int keys, int split) {
  const int rows = s.n * (int)a.share.by;
  const int t0 = (int)divide((uint32_t)row0, a.share);
  const int t1 = (int)divide((uint32_t)(min(row0 + block_rows, rows) - 1), a.share);
  // (a node is at a depth from 0 up to its index, and sees no later one)
  const int p0 = s.len - s.n + (MODE == kTree ? 0 : t0), p1 = s.len - s.n + t1;
  Span w;
  w.last_key = a.causal ? min(max(p1 + 1, 0), s.len) : s.len;
  w.first_key = a.window > 0 ? max(p0 - a.window + 1, 0) : 0;
  w.all_hi = MODE == kTree ? p0 : a.causal ? p0 + 1 : s.len;
  w.all_lo = a.window > 0 ? max(p1 - a.window + 1, 0) : 0;
  const int tile0 = w.first_key / keys;
  const int tiles = w.last_key > w.first_key ? (w.last_key + keys - 1) / keys - tile0 : 0;
  const int per = (tiles + a.splits - 1) / a.splits;
  w.tile_lo = tile0 + min(split * per, tiles);
  w.tile_hi = min(w.tile_lo + per, tile0 + tiles);
  return w;
}

// The block that holds key j of a workgroup's, and its slot there; null if it has no such key, or no page holds it.
__device__ __forceinline__ const uint8_t* block_of_key(const Cache& c, const Span& w, const int32_t* table, int head, int j,
                                                       int* slot) {
  if (j < w.first_key || j >= w.last_key) return nullptr;
  const uint32_t page = divide((uint32_t)j, c.page);
  const int32_t id = table[page];
  *slot = j - (int)(page * c.page.by);
  return id < 0 || id >= c.pages ? nullptr : c.pool + ((int64_t)id * c.heads + head) * c.block;
}

// The keys that token t sees: [lo, lo + seen).
__device__ __forceinline__ void seen_of(const AttnArgs& a, const Seq& s, int t, bool live, int* lo, int* seen) {
  const int pos = s.len - s.n + t;
  const int hi = a.causal ? min(max(pos + 1, 0), s.len) : s.len;
  *lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
  *seen = live ? max(hi - *lo, 0) : 0;
}

// The same for a node at that depth: of the text, [lo, lo + seen); the nodes it sees are in its set.
__device__ __forceinline__ void seen_of_node(const AttnArgs& a, const Seq& s, int depth, bool live, int* lo, int* seen) {
  const int text = s.len - s.n;
  *lo = a.window > 0 ? max(text + depth - a.window + 1, 0) : 0;
  *seen = live ? max(text - *lo, 0) : 0;
}
template <int MODE>
__device__ __forceinline__ bool sees(int j, int lo, int seen, int text, uint64_t above) {
  if ((uint32_t)(j - lo) < (uint32_t)seen) return true;
  return MODE == kTree && (uint32_t)(j - text) < 64u && (above >> ((j - text) & 63) & 1) != 0;
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
template <int MODE>
__device__ __forceinline__ float masked(float s, int j, int lo, int seen, int text, uint64_t above) {
  return sees<MODE>(j, lo, seen, text, above) ? s : -INFINITY;
}

// Four scale bytes of a token (from byte 4 n on; 127, one, past the last), in loads as wide as their place
// allows.
__device__ __forceinline__ uint32_t scale_word(const uint8_t* sp, int groups, int n) {
  if (groups % 4 == 0) return 4 * n < groups ? *reinterpret_cast<const uint32_t*>(sp + 4 * n) : 0x7f7f7f7fu;
  uint32_t word = 0;
  if (groups % 2 == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      word |= (uint32_t)(4 * n + 2 * e < groups ? *reinterpret_cast<const uint16_t*>(sp + 4 * n + 2 * e) : 0x7f7f) << (16 * e);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) word |= (uint32_t)(4 * n + e < groups ? sp[4 * n + e] : 127) << (8 * e);
  }
  return word;
}
// N words of scale bytes: those that stand for NaN become 255; whether there was one.  A write leaves none past the
// type's last but 255, and few of that; whether a byte is past it is whether its complement is below 255 - last.
template <int KIND, int N>
__device__ __forceinline__ bool nan_scales(uint32_t* words) {
  if constexpr (KIND == LLVQ_KV_BF16) return false;
  constexpr uint32_t kBelow = (uint32_t)(255 - last_scale(KIND)) * 0x01010101u;
  uint32_t any = 0;
#pragma unroll
  for (int n = 0; n < N; ++n) any |= (~words[n] - kBelow) & words[n] & 0x80808080u;
  if (any != 0) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((words[n] >> (8 * e) & 255u) > (uint32_t)last_scale(KIND)) words[n] |= 255u << (8 * e);
  }
  return any != 0;
}

// Few rows: up to 64 rows of a (sequence, key head), in CT tiles of 16 columns.
//
// A decode step reads each cached byte for a handful of rows, so HBM bounds it and what counts is loads in
// flight.  Every wave therefore runs by itself: it takes every fourth (or eighth) 32-key piece of the
// workgroup's share, stages it in its own 64 * DP bytes of LDS (the keys, then the values in the same
// place) and waits for nothing but its own loads, which are issued a piece ahead (page numbers two pieces
// ahead).  With 16x16x32 instructions a lane holds 8 scores of a piece, and a tile of outputs takes DP / 4
// registers of a lane. (Tiles shared by the workgroup, with the kernel below and its barriers, took a step
// of 64 sequences of up to 16384 tokens, 64 heads over 8 key heads of 128 channels in e4m3, 837 us; this
// takes 267 us, 5.3 TB/s, where a large copy reaches 4.9.  Three sequences of up to 131000 tokens in e2m1:
// 78 us, 4.3 TB/s; 16 of up to 4096 with 8 drafts each, f32, 32 heads: 87 us, 4.2 TB/s.  One token of 32
// heads over 777 keys in bf16 takes 7.4 us and the join 4: a chain of six loads, each waiting for the one
// before.) In S^T's layout a lane (column lane % 16, g = lane / 16) holds keys 4 g + i and 16 + 4 g + i,
// which are taken as the eight consecutive keys of its place in the second product; the transposing load
// reads V's rows in the same order. Rows in LDS are padded, so that every address is one register and a
// constant: by 16 bytes for the keys (16 rows at one 16-byte chunk fall on 16 different slots of 256
// bytes), by 32 for the values (the eight rows that half a wave takes at 32 bytes of channels fall on eight
// different segments).
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

// TEAM: the waves that share out the keys of a row block.  1: a workgroup's four waves have a row block
// each, and no barrier; for so many short sequences that they fill the chip this way, where a team's start
// and its joining would take longer than the keys (57 sequences of up to 176 tokens, 32 key heads of 192
// channels in e2m1, 5 new tokens: 42 us, 54 with teams of four; 64 of up to 500, 32 heads of 128 in e4m3:
// 43 us, 4.1 TB/s).
template <int KIND, int DP, int NT, int CT, int TEAM, int MODE>
__global__ __launch_bounds__(TEAM == 8 ? 512 : 256, TEAM == 8 ? 2 : few_waves(KIND, DP, NT, CT)) void k_attn_few(AttnArgs a) {
  constexpr int kWaves = TEAM == 1 ? 4 : TEAM;
  constexpr int kRaw = code_bytes(KIND, DP) / 16;  // 16-byte chunks of a row of codes
  constexpr int kLoads = 32 * kRaw / kWave;        // chunks a lane loads of a piece
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;
  constexpr int kSteps = DP / 32, kOut = DP / 16;
  constexpr int kTerms = NT == 1 ? 2 : NT;  // of P: with one, its roundings do not average out over few keys
  const Cache& c = a.c;
  using Lds = FewLds<DP>;
  __shared__ __align__(16) uint8_t lds[kWaves * Lds::kWaveBytes];
  __shared__ float wave_m[TEAM][16], wave_l[TEAM][16];
  // the nodes' sets, looked up only at the pieces that hold nodes (the waves of a team write the same)
  __shared__ uint64_t nodes[MODE == kTree ? (TEAM == 1 ? 4 : 1) : 1][MODE == kTree ? kWave : 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave_id = __builtin_amdgcn_readfirstlane(tid >> 6), wave = TEAM == 1 ? 0 : wave_id;
  const int g = lane >> 4, col = lane & 15;
  uint8_t* mine = lds + wave_id * Lds::kWaveBytes;

  int id = TEAM == 1 ? (int)blockIdx.x * 4 + wave_id : (int)blockIdx.x;
  if (id >= a.units) return;
  const int head = id % c.heads;
  id /= c.heads;
  const int split = id % a.splits;
  id /= a.splits;
  const int rb = id % a.row_blocks;
  const int b = id / a.row_blocks;
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, rows = s.n * share;
  if (a.err && lane == 0 && wave == 0 && head == 0 && split == 0 && rb == 0 && (s.bad || rows > a.row_blocks * 16 * CT)) atomicAdd(a.err, 1);
  const int row0 = rb * 16 * CT;
  if (row0 >= rows) return;
  const Span w = span_of<MODE>(a, s, row0, 16 * CT, 32 * TEAM, split);

  const int64_t head_off = (int64_t)head * c.block, page_bytes = (int64_t)c.heads * c.block;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  const int ch = lane % kRaw;  // this lane's chunk of every row that it loads
  const bool in_row = ch * 16 < c.row;
  bool lost = false;
  // the page number of this lane's key of a piece (lanes 32..63 as 0..31)
  auto is_key = [&](int tile, int j) { return tile < w.tile_hi && j >= w.first_key && j < w.last_key; };
  auto page_of = [&](int tile) -> int32_t {
    const int j = (tile * TEAM + wave) * 32 + (lane & 31);
    return is_key(tile, j) ? table[divide((uint32_t)j, c.page)] : 0;
  };
  // A lane's key of a piece, lane % 32, tells where the piece's rows lie, and with lane / 32 whose scales it
  // holds; a lane loads chunk `ch` of keys i * 64 / kRaw + lane / kRaw.
  constexpr int kWords = KIND == LLVQ_KV_BF16 ? 1 : DP <= 128 ? 1 : 2;  // of four scale bytes
  constexpr uint32_t kOnes = 0x7f7f7f7fu;
  const uint8_t* pool = c.pool + (in_row ? ch * 16 : 0);
  const int scale_shift = KIND == LLVQ_KV_BF16 ? 0 : ch * kOf / 4 % 4 * 8, word_at = KIND == LLVQ_KV_BF16 ? 0 : ch * kOf / 16;
  const bool narrow = c.dim < DP;  // rows shorter than the tile's
  int64_t rows_at[kLoads];
  u32x4 raw_k[kLoads], raw_v[kLoads];
  uint32_t scales[kWords], next_scales[kWords], gone = 0, next_gone = 0;  // of the piece that is staged, and of the next
  auto locate = [&](int tile, int32_t ids) {
    const uint32_t j = (uint32_t)((tile * TEAM + wave) * 32 + (lane & 31));
    const bool key = is_key(tile, (int)j), ok = key && ids >= 0 && ids < c.pages;
    lost |= key && !ok;
    next_gone = (uint32_t)__ballot(!ok);
    // a place that is not there is read from the pool's start and left out when it is staged
    const int slot = ok ? (int)(j - divide(j, c.page) * c.page.by) : 0;
    const int64_t blk = ok ? (int64_t)ids * page_bytes + head_off : 0, row = blk + slot * c.row;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * kWave + lane) / kRaw;
      rows_at[i] = (int64_t)(uint32_t)__shfl((int)(uint32_t)row, key) | (int64_t)__shfl((int)(row >> 32), key) << 32;
    }
#pragma unroll
    for (int n = 0; n < kWords; ++n) {
      next_scales[n] = kOnes;
      if (KIND != LLVQ_KV_BF16 && ok)
        next_scales[n] = scale_word(c.pool + blk + (lane < 32 ? c.ks_off : c.vs_off) + slot * c.groups, c.groups, n);
    }
  };
  auto fetch_keys = [&]() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw_k[i] = *reinterpret_cast<const u32x4*>(pool + rows_at[i]);
  };
  auto fetch_values = [&]() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) raw_v[i] = *reinterpret_cast<const u32x4*>(pool + rows_at[i] + c.v_off);
  };
  // the scale byte of a chunk: of the keys (from lanes 0..31) or of the values
  auto scale_of = [&](int key, int is_v) -> uint32_t {
    if constexpr (KIND == LLVQ_KV_BF16) return 127;
    uint32_t word = (uint32_t)__shfl((int)scales[0], key + 32 * is_v);
    if constexpr (kWords == 2) {
      const uint32_t second = (uint32_t)__shfl((int)scales[kWords - 1], key + 32 * is_v);
      word = word_at ? second : word;
    }
    return word >> scale_shift & 255;
  };

  int32_t ids = page_of(w.tile_lo);
  if (w.tile_lo < w.tile_hi) {
    locate(w.tile_lo, ids);
    fetch_keys();
    fetch_values();
    ids = page_of(w.tile_lo + 1);
  }
  Node node;
  uint64_t* above = nodes[TEAM == 1 && MODE == kTree ? wave_id : 0];
  const int text = s.len - s.n;
  if constexpr (MODE == kTree) {
    node = node_of(a, s);
    above[lane] = node.above;
    wave_order();
    if (a.err && wave == 0 && head == 0 && split == 0 && rb == 0 && __any(node.bad) && lane == 0) atomicAdd(a.err, 1);
  }
  // (the queries after the first piece's loads: they are a load away, the piece two)
  int lo[CT], seen[CT], t[CT], qhead[CT];
  bool live[CT];
  bf16x8 q[NT][CT][kSteps];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int row = row0 + ct * 16 + col;
    live[ct] = row < rows;
    t[ct] = live[ct] ? (int)divide((uint32_t)row, a.share) : 0;
    qhead[ct] = head * share + (live[ct] ? row - t[ct] * share : 0);
    if constexpr (MODE == kTree) {
      const int depth = __shfl(node.depth, t[ct] & 63);
      seen_of_node(a, s, t[ct] < LLVQ_MAX_NODES ? depth : 0, live[ct], &lo[ct], &seen[ct]);
    } else {
      seen_of(a, s, t[ct], live[ct], &lo[ct], &seen[ct]);
    }
    const int64_t at = (int64_t)(s.first + t[ct]) * a.q_token + (int64_t)qhead[ct] * a.q_head;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      bf16x8 terms[NT];
      load_query<NT>(a, at, st * 32 + g * 8, live[ct], terms);
#pragma unroll
      for (int n = 0; n < NT; ++n) q[n][ct][st] = terms[n];
    }
  }

  auto above_of = [&](int ct) -> uint64_t { return MODE == kTree && live[ct] && t[ct] < LLVQ_MAX_NODES ? above[t[ct] & 63] : 0; };

  f32x4 acc[CT][kOut];
  float m[CT], l4[CT][4];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    m[ct] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) l4[ct][i] = 0.0f;
#pragma unroll
    for (int d = 0; d < kOut; ++d) acc[ct][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  int odd_lo = 0x7fffffff, odd_hi = -1;  // the first and the last tile with a value that is not finite
  for (int tile = w.tile_lo; tile < w.tile_hi; ++tile) {
    const int key_base = (tile * TEAM + wave) * 32;
    const bool more = tile + 1 < w.tile_hi;
    // the keys
    gone = next_gone;
#pragma unroll
    for (int n = 0; n < kWords; ++n) scales[n] = next_scales[n];
    const uint64_t spoilt = __ballot(nan_scales<KIND, kWords>(scales));  // keys, and from bit 32 on values
    if (gone != 0 || narrow) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        if ((gone >> ((i * kWave + lane) / kRaw) & 1) || !in_row) raw_k[i] = raw_v[i] = u32x4{0, 0, 0, 0};
    }
    wave_order();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * kWave + lane) / kRaw;
      u32x4 o[kOf];
      expand<KIND>(raw_k[i], scale_of(key, 0), o);
#pragma unroll
      for (int n = 0; n < kOf; ++n) *reinterpret_cast<u32x4*>(mine + key * Lds::kKeyRow + (ch * kOf + n) * 16) = o[n];
    }
    wave_order();
    if (more) {
      locate(tile + 1, ids);
      ids = page_of(tile + 2);
      fetch_keys();
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
    bf16x8 p[kTerms][CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (!whole) {
        const uint64_t up = above_of(ct);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            score[ct][u][i] = masked<MODE>(score[ct][u][i], key_base + u * 16 + 4 * g + i, lo[ct], seen[ct], text, up);
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, score[ct][i / 4][i & 3]);
      top = quad_max(top) * a.scale_log2;
      const bool up = top > m[ct] + kRescaleStep;
      if (__any(up)) {  // (the others' sums stay as they are: a row's roundings are its own)
        const float f = !up ? 1.0f : m[ct] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[ct] - top);
        m[ct] = up ? top : m[ct];
#pragma unroll
        for (int i = 0; i < 4; ++i) l4[ct][i] *= f;
#pragma unroll
        for (int d = 0; d < kOut; ++d) acc[ct][d] *= f;
      }
      const float ms = m[ct] == -INFINITY ? 0.0f : m[ct];
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __builtin_amdgcn_exp2f(fmaf(score[ct][i / 4][i & 3], a.scale_log2, -ms));
      bf16x8 terms[kTerms];
      split_terms<kTerms>(x, terms);
      sum_p<kTerms>(x, terms[0], l4[ct]);
#pragma unroll
      for (int n = 0; n < kTerms; ++n) p[n][ct] = terms[n];
    }
    // the values, in the keys' place.  Those that are not finite would spoil rows that do not see them (0 * NaN):
    // they are left out here and added to the rows that do see them at the end
    if (drop_odd<KIND, kLoads>(raw_v) || (spoilt >> 32) != 0) {
      odd_lo = min(odd_lo, tile);
      odd_hi = tile;
    }
    wave_order();
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int key = (i * kWave + lane) / kRaw;
      uint32_t sb = scale_of(key, 1);
      if (KIND != LLVQ_KV_BF16 && (spoilt >> 32) != 0 && sb == 255) raw_v[i] = u32x4{0, 0, 0, 0}, sb = 127;
      u32x4 o[kOf];
      expand<KIND>(raw_v[i], sb, o);
#pragma unroll
      for (int n = 0; n < kOf; ++n) *reinterpret_cast<u32x4*>(mine + key * Lds::kValueRow + (ch * kOf + n) * 16) = o[n];
    }
    wave_order();
    if (more) fetch_values();
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
        for (int n = kTerms - 1; n >= 0; --n) acc[ct][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf.v, p[n][ct], acc[ct][d], 0, 0, 0);
    }
  }
  if (a.err && lost) atomicAdd(a.err, 1);
  // what was left out: p is positive where a row sees the key, so the value itself is what the sum becomes.  The
  // keys of all tiles from the first such one to the last are looked at again, one by one: a wave keeps two numbers
  // for this through its loop, and only a damaged cache takes it
  for (int tile = odd_lo; tile <= odd_hi; ++tile)
    for (int i = 0; i < 32; ++i) {
      const int j = (tile * TEAM + wave) * 32 + i;
      int slot;
      const uint8_t* blk = block_of_key(c, w, table, head, j, &slot);
      if (!blk) continue;
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        const f32x4 x = nonfinite4<KIND>(c, blk, slot, d * 16 + 4 * g);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
          if (sees<MODE>(j, lo[ct], seen[ct], text, above_of(ct))) acc[ct][d] += x;
      }
    }

  if constexpr (TEAM == 1) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const float l = quad_sum((l4[ct][0] + l4[ct][1]) + (l4[ct][2] + l4[ct][3]));
      if (!live[ct]) continue;
      const int64_t row = (int64_t)(s.first + t[ct]) * c.heads * share + qhead[ct];
      if (MODE == kLse && g == 0) a.lse[row] = log_sum(m[ct], l);
      const int64_t out_at = (int64_t)(s.first + t[ct]) * a.out_token + (int64_t)qhead[ct] * a.out_head;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no visible key: the row is zero
#pragma unroll
      for (int d = 0; d < kOut; ++d) store_row4<NT>(a, row, out_at, 0, d * 16 + g * 4, acc[ct][d], inv);
    }
    return;
  }
  // the waves' parts are joined through LDS under their common maximum and added in the waves' order
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const float l = quad_sum((l4[ct][0] + l4[ct][1]) + (l4[ct][2] + l4[ct][3]));
    __syncthreads();
    if (g == 0) wave_m[wave][col] = m[ct];
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) top = fmaxf(top, wave_m[i][col]);
    const float f = m[ct] == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(m[ct] - top);
    if (g == 0) wave_l[wave][col] = l * f;
    float* sums = reinterpret_cast<float*>(lds);  // [wave][16 columns][DP], quads of channels swizzled by the column
#pragma unroll
    for (int d = 0; d < kOut; ++d)
      *reinterpret_cast<f32x4*>(sums + (wave * 16 + col) * DP + (((d * 4 + g) ^ (col & 7)) << 2)) = acc[ct][d] * f;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) total += wave_l[i][col];
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;  // no visible key: the row is zero
    if (live[ct]) {
      const int64_t row = (int64_t)(s.first + t[ct]) * c.heads * share + qhead[ct];
      const int64_t out_at = (int64_t)(s.first + t[ct]) * a.out_token + (int64_t)qhead[ct] * a.out_head;
      if (a.splits > 1 && wave == 0 && g == 0) {
        const int64_t all = (int64_t)c.tokens * c.heads * share;
        a.stats[(split * all + row) * 2] = top;
        a.stats[(split * all + row) * 2 + 1] = total;
      }
      if (MODE == kLse && a.splits == 1 && wave == 0 && g == 0) a.lse[row] = log_sum(top, total);
      if (a.splits == 1 || w.tile_lo < w.tile_hi) {
        for (int d = wave; d < kOut; d += TEAM) {  // the waves share out the channels
          f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < TEAM; ++i) x += *reinterpret_cast<const f32x4*>(sums + (i * 16 + col) * DP + (((d * 4 + g) ^ (col & 7)) << 2));
          store_row4<NT>(a, row, out_at, split, d * 16 + g * 4, x, inv);
        }
      }
    }
  }
}

// Many rows: 128 or 256 rows of a (sequence, key head), 32 columns a wave, tiles shared by the four or
// eight waves.
//
// A chunk of a prompt reuses every key for many rows, so the matrix instructions bound it, next to exp and
// what else the softmax costs on the vector units (a matrix instruction of 32 cycles makes 512 scores of a
// key step of 16 channels; exp alone is 8 cycles for 64 of them).  Two waves a SIMD let one's softmax run
// under the other's products.  Tiles are double-buffered in LDS: after the one barrier of a round come the
// first product and the softmax, then the next tile, whose codes were loaded a round ago, is expanded into
// the other buffer and the loads of the one after it are issued, then the second product.  Operands are
// read four instructions ahead in a pinned order.
//
// Measured at 2 x 2048 new tokens over 8192, 32 heads of 128 channels in e4m3: 480 to 513 us a call over several
// cards, 940 to 1000 TFLOP/s, about 80 % of what a large bf16 library product reaches (the kernel alone under a
// tracer, which leaves the chip idle between launches, 540).  Taken apart when it stood at 490: without the staging 80
// us less, without the softmax 65, without both 370 us, near the 290 us that the same instructions take alone (the
// clock falls under them).  64-wide heads have twice the softmax a product: 24 heads over 4 key heads in e2m1, window
// 1000, 75 us, 438 TFLOP/s.  f32 queries take three times the instructions: 1193 us at the first of these sizes.
//
// Heads of more than 128 channels are taken in two halves of the output by two workgroups, which both take
// the first product: half again the products, but what a wave holds fits two waves a SIMD (16 heads of 256
// channels in bf16, 3 x 700 over 3500: 220 us instead of 391 when this was done; 192 now with its join of 18).
template <int KIND, int DP, int NT, int WAVES>
struct ManyShape {
  static constexpr int kThreads = 64 * WAVES, kRows = 32 * WAVES;
  static constexpr int kOutDim = DP < 128 ? DP : 128;        // channels of the output that a workgroup takes
  static constexpr int kParts = DP / kOutDim;
  static constexpr int kSub = NT == 1 && DP <= 128 ? 2 : 1;  // 32-key pieces of a tile
  static constexpr int kKeys = 32 * kSub;
  // rows padded so that 16 rows at one 16-byte chunk fall on 16 slots of 256 bytes (keys), and four rows
  // at 64 bytes of channels on four segments (values)
  static constexpr int kKeyRow = DP * 2 + 16, kValueRow = kOutDim * 2 + 64;
  static constexpr int kBuffer = kKeys * (kKeyRow + kValueRow);
  // registers: queries, outputs, scores, P, operands read ahead, chunks in flight
  static constexpr int kHeld = NT * DP / 4 + kOutDim / 2 + 16 * kSub + 8 * NT * kSub + 16 + 30 +
                               5 * (kKeys * code_bytes(KIND, DP + kOutDim) / 16 / kThreads);
  // waves a SIMD; narrow heads spend their time on the softmax, not on products, and gain from a third
  // (ragged chunks of 64-wide heads: 88 us instead of 105)
  static constexpr int kWaves = DP == 64 && NT == 1 && WAVES == 4 ? 3 : kHeld <= 256 ? 2 : 1;
  static constexpr int kAhead = DP == 64 ? 2 : 4;            // operands read ahead
};

// The 16-byte chunks of codes that a thread stages of a tile: chunk `ch` of keys key0, key0 + step, ...
template <int KIND, int DIM, int KEYS, int THREADS>
struct Chunks {
  static constexpr int kRaw = code_bytes(KIND, DIM) / 16, kAll = KEYS * kRaw;
  static constexpr int kPer = (kAll + THREADS - 1) / THREADS, kStep = THREADS / kRaw;
  static_assert(THREADS % kRaw == 0 && (kPer == 1 || kAll % THREADS == 0), "a thread has one chunk place in all its rows");
  int ch, key0;
  bool any;  // (kPer is 1 where a tile has fewer chunks than threads)
  __device__ __forceinline__ explicit Chunks(int tid) : ch(tid % kRaw), key0(tid / kRaw), any(kAll >= THREADS || tid < kAll) {
    if (!any) key0 = 0;
  }
};

// Where a key lies, and its scale bytes.
template <int KIND, int DP>
struct alignas(16) Place {
  static constexpr int kWords = KIND == LLVQ_KV_BF16 ? 1 : DP <= 128 ? 1 : 2;  // of four scale bytes
  int64_t row;                        // its key codes' offset in the pool
  uint32_t scales[2][kWords];         // keys', values'
};

template <int KIND, int DP, int NT, int WAVES, int MODE>
__global__ __launch_bounds__(64 * WAVES, (ManyShape<KIND, DP, NT, WAVES>::kWaves)) void k_attn_many(AttnArgs a) {
  using Sh = ManyShape<KIND, DP, NT, WAVES>;
  constexpr int kKeys = Sh::kKeys, kSub = Sh::kSub, kSteps = DP / 16, kOut = Sh::kOutDim / 32, kRows = Sh::kRows;
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;
  using KChunks = Chunks<KIND, DP, kKeys, Sh::kThreads>;
  using VChunks = Chunks<KIND, Sh::kOutDim, kKeys, Sh::kThreads>;
  const Cache& c = a.c;
  __shared__ __align__(16) uint8_t lds[2 * Sh::kBuffer];
  __shared__ int odd_tiles[2];  // the first and the last tile with a value that is not finite
  using Where = Place<KIND, DP>;
  __shared__ Where places[2][kKeys];
  // of a tile: keys that are not there, and keys with a group of values whose scale says that they are not finite
  __shared__ uint64_t missing[2], spoilt[2];
  __shared__ uint64_t nodes[MODE == kTree ? kWave : 1];  // (the waves write the same)

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;

  int id = blockIdx.x;
  const int head = id % c.heads;
  id /= c.heads;
  const int part = id % Sh::kParts, part_dim = part * Sh::kOutDim;
  id /= Sh::kParts;
  const int split = id % a.splits;
  id /= a.splits;
  const int rb = a.row_blocks - 1 - id % a.row_blocks;  // the longest rows of a causal chunk first
  const int b = id / a.row_blocks;
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, rows = s.n * share;
  if (a.err && tid == 0 && head == 0 && split == 0 && part == 0 && rb == 0 && (s.bad || rows > a.row_blocks * kRows)) atomicAdd(a.err, 1);
  const int row0 = rb * kRows;
  if (row0 >= rows) return;
  const Span w = span_of<MODE>(a, s, row0, kRows, kKeys, split);

  const int row = row0 + wave * 32 + col;
  const bool live = row < rows;
  const int t = live ? (int)divide((uint32_t)row, a.share) : 0;
  const int qhead = head * share + (live ? row - t * share : 0);
  int lo, seen;
  const int text = s.len - s.n;
  if constexpr (MODE == kTree) {
    const Node node = node_of(a, s);
    nodes[lane] = node.above;
    wave_order();
    const int depth = __shfl(node.depth, t & 63);
    seen_of_node(a, s, t < LLVQ_MAX_NODES ? depth : 0, live, &lo, &seen);
    if (a.err && wave == 0 && head == 0 && split == 0 && part == 0 && rb == 0 && __any(node.bad) && lane == 0) atomicAdd(a.err, 1);
  } else {
    seen_of(a, s, t, live, &lo, &seen);
  }
  auto above = [&]() -> uint64_t { return MODE == kTree && live && t < LLVQ_MAX_NODES ? nodes[t & 63] : 0; };
  bf16x8 q[NT][kSteps];
#pragma unroll
  for (int st = 0; st < kSteps; ++st) {
    bf16x8 terms[NT];
    load_query<NT>(a, (int64_t)(s.first + t) * a.q_token + (int64_t)qhead * a.q_head, st * 16 + half * 8, live, terms);
#pragma unroll
    for (int n = 0; n < NT; ++n) q[n][st] = terms[n];
  }
  f32x16 acc[kOut];
#pragma unroll
  for (int i = 0; i < kOut; ++i) acc[i] = f32x16{0.0f};
  float m = -INFINITY, l4[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // (four sums: one chain of additions is slow)
  // The log-sum is that of p as it is; what divides the output is the sum of p as the second product takes it, rounded
  constexpr bool kTrue = MODE == kLse && NT == 1;
  float e4[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  const int64_t head_off = (int64_t)head * c.block, page_bytes = (int64_t)c.heads * c.block;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  // (where half of the threads have nothing of the keys, they take the values)
  const KChunks kc(tid);
  const VChunks vc(KChunks::kAll <= Sh::kThreads / 2 && VChunks::kAll <= Sh::kThreads / 2 ? tid ^ (Sh::kThreads / 2) : tid);
  const bool k_in = kc.ch * 16 < c.row, v_in = code_bytes(KIND, part_dim) + vc.ch * 16 < c.row;
  const bool narrow = c.dim < DP;  // rows shorter than the tile's
  const uint8_t* k_pool = c.pool + (k_in ? kc.ch * 16 : 0);
  const uint8_t* v_pool = c.pool + c.v_off + (v_in ? code_bytes(KIND, part_dim) + vc.ch * 16 : 0);
  // the byte of a place's scales that belongs to the thread's chunks
  const int k_shift = kc.ch * kOf / 4 % 4 * 8, v_shift = vc.ch * kOf / 4 % 4 * 8;
  const int k_word = kc.ch * kOf / 16, v_word = part_dim / 128;
  u32x4 raw_k[KChunks::kPer], raw_v[VChunks::kPer];
  uint32_t sc_k[KChunks::kPer], sc_v[VChunks::kPer];
  uint64_t gone = 0, nonfinite = 0;  // of the loaded tile
  bool lost = false;
  // Where a tile's keys lie and how they are scaled is worked out once a key, by the wave whose turn it is: the
  // page numbers are loaded five rounds ahead, the scales four, both written to LDS three and the codes loaded
  // two rounds ahead.
  int32_t ids = 0;
  Where found;
  bool found_ok = false;
  auto is_key = [&](int tile, int j) { return lane < kKeys && tile < w.tile_hi && j >= w.first_key && j < w.last_key; };
  auto load_pages = [&](int tile) {
    if (wave != (tile & (WAVES - 1))) return;
    const int j = tile * kKeys + lane;
    ids = is_key(tile, j) ? table[divide((uint32_t)j, c.page)] : 0;
  };
  auto load_scales = [&](int tile) {
    if (wave != (tile & (WAVES - 1))) return;
    const uint32_t j = (uint32_t)(tile * kKeys + lane);
    const bool key = is_key(tile, (int)j);
    found_ok = key && ids >= 0 && ids < c.pages;
    lost |= key && !found_ok;
    // a place that is not there is read from the pool's start and left out when it is staged
    const int slot = found_ok ? (int)(j - divide(j, c.page) * c.page.by) : 0;
    const int64_t blk = found_ok ? (int64_t)ids * page_bytes + head_off : 0;
    found.row = blk + slot * c.row;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < Where::kWords; ++n) found.scales[i][n] = 0x7f7f7f7fu;
    if constexpr (KIND != LLVQ_KV_BF16) {
      if (found_ok) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int n = 0; n < Where::kWords; ++n)
            found.scales[i][n] = scale_word(c.pool + blk + (i ? c.vs_off : c.ks_off) + slot * c.groups, c.groups, n);
      }
    }
  };
  auto write_places = [&](int tile) {
    if (wave != (tile & (WAVES - 1))) return;
    nan_scales<KIND, Where::kWords>(found.scales[0]);
    const bool bad = nan_scales<KIND, Where::kWords>(found.scales[1]);
    const uint64_t no = __ballot(!found_ok), spoils = __ballot(bad);
    if (lane < kKeys) places[tile & 1][lane] = found;
    if (lane == 0) {
      missing[tile & 1] = no & (kKeys == 64 ? ~0ull : (1ull << (kKeys % 64)) - 1);
      spoilt[tile & 1] = spoils & (kKeys == 64 ? ~0ull : (1ull << (kKeys % 64)) - 1);
    }
  };
  auto uniform64 = [](uint64_t x) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)x) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32;
  };
  auto fetch = [&](int tile) {
    gone = uniform64(missing[tile & 1]);
    nonfinite = uniform64(spoilt[tile & 1]);
#pragma unroll
    for (int i = 0; i < KChunks::kPer; ++i) {
      const Where* at = &places[tile & 1][kc.key0 + i * KChunks::kStep];
      raw_k[i] = *reinterpret_cast<const u32x4*>(k_pool + at->row);
      sc_k[i] = at->scales[0][Where::kWords == 1 ? 0 : k_word] >> k_shift & 255;
    }
#pragma unroll
    for (int i = 0; i < VChunks::kPer; ++i) {
      const Where* at = &places[tile & 1][vc.key0 + i * VChunks::kStep];
      raw_v[i] = *reinterpret_cast<const u32x4*>(v_pool + at->row);
      sc_v[i] = at->scales[1][Where::kWords == 1 ? 0 : v_word] >> v_shift & 255;
    }
  };
  auto stage = [&](uint8_t* buffer, int tile) {
    if (gone != 0 || narrow) {
#pragma unroll
      for (int i = 0; i < KChunks::kPer; ++i)
        if ((gone >> (kc.key0 + i * KChunks::kStep) & 1) || !k_in) raw_k[i] = u32x4{0, 0, 0, 0}, sc_k[i] = 127;
#pragma unroll
      for (int i = 0; i < VChunks::kPer; ++i)
        if ((gone >> (vc.key0 + i * VChunks::kStep) & 1) || !v_in) raw_v[i] = u32x4{0, 0, 0, 0}, sc_v[i] = 127;
    }
    // values that are not finite would spoil rows that do not see them (0 * NaN): they are left out here and
    // added to the rows that do see them at the end
    if (drop_odd<KIND, VChunks::kPer>(raw_v) || nonfinite != 0) {
      if (lane == 0) atomicMin(&odd_tiles[0], tile), atomicMax(&odd_tiles[1], tile);
    }
    if (KIND != LLVQ_KV_BF16 && nonfinite != 0) {
#pragma unroll
      for (int i = 0; i < VChunks::kPer; ++i)
        if (sc_v[i] == 255) raw_v[i] = u32x4{0, 0, 0, 0}, sc_v[i] = 127;
    }
    u32x4 o[kOf];
    if (kc.any) {
#pragma unroll
      for (int i = 0; i < KChunks::kPer; ++i) {
        expand<KIND>(raw_k[i], sc_k[i], o);
#pragma unroll
        for (int n = 0; n < kOf; ++n)
          *reinterpret_cast<u32x4*>(buffer + (kc.key0 + i * KChunks::kStep) * Sh::kKeyRow + (kc.ch * kOf + n) * 16) = o[n];
      }
    }
    if (vc.any) {
#pragma unroll
      for (int i = 0; i < VChunks::kPer; ++i) {
        expand<KIND>(raw_v[i], sc_v[i], o);
#pragma unroll
        for (int n = 0; n < kOf; ++n)
          *reinterpret_cast<u32x4*>(buffer + kKeys * Sh::kKeyRow + (vc.key0 + i * VChunks::kStep) * Sh::kValueRow +
                                    (vc.ch * kOf + n) * 16) = o[n];
      }
    }
  };

  if (tid < 2) odd_tiles[tid] = tid == 0 ? 0x7fffffff : -1;
  if (w.tile_lo < w.tile_hi) {
    // (a wave has one tile of WAVES at a time)
    for (int i = 0; i < 4; ++i) load_pages(w.tile_lo + i);
    for (int i = 0; i < 4; ++i) load_scales(w.tile_lo + i);
    write_places(w.tile_lo);
    write_places(w.tile_lo + 1);
    __syncthreads();
    fetch(w.tile_lo);
    stage(lds, w.tile_lo);
    fetch(w.tile_lo + 1);
    __syncthreads();
    write_places(w.tile_lo + 2);
    load_pages(w.tile_lo + 4);
  }
  for (int tile = w.tile_lo; tile < w.tile_hi; ++tile) {
    const int par = (tile - w.tile_lo) & 1;
    const uint8_t* buffer = lds + par * Sh::kBuffer;
    __syncthreads();  // this tile is staged, and the other buffer has been read
    const int key_base = tile * kKeys;
    // operands are read a few instructions ahead, in an order that is pinned: left to itself the compiler reads
    // each right before its use and waits for it
    constexpr int kAhead = Sh::kAhead;
    f32x16 sc[kSub];
    {
      const uint8_t* keys = buffer + col * Sh::kKeyRow + half * 16;
      auto operand = [&](int k) { return *reinterpret_cast<const bf16x8*>(keys + (k % kSub) * 32 * Sh::kKeyRow + (k / kSub) * 32); };
      bf16x8 kf[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) kf[k] = operand(k);
#pragma unroll
      for (int u = 0; u < kSub; ++u) sc[u] = f32x16{0.0f};
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < kSteps * kSub; ++k) {
#pragma unroll
        for (int n = NT - 1; n >= 0; --n)
          sc[k % kSub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[k % kAhead], q[n][k / kSub], sc[k % kSub], 0, 0, 0);
        if (k + kAhead < kSteps * kSub) kf[k % kAhead] = operand(k + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    const uint8_t* values = buffer + kKeys * Sh::kKeyRow + (4 * half + ((lane & 15) >> 2)) * Sh::kValueRow + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    auto value_operand = [&](int k) {  // k = 16-key step * kOut + output tile
      const uint8_t* at = values + (k / kOut) * 16 * Sh::kValueRow + (k % kOut) * 64;
      union {
        s16x4 h[2];
        bf16x8 v;
      } vf;
      vf.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at);
      vf.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(at + 8 * Sh::kValueRow));
      return vf.v;
    };
    if (!(key_base >= w.all_lo && key_base + kKeys <= w.all_hi && key_base + kKeys <= s.len)) {
      const uint64_t up = above();
#pragma unroll
      for (int u = 0; u < kSub; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sc[u][i] = masked<MODE>(sc[u][i], key_base + u * 32 + 8 * (i / 4) + 4 * half + (i & 3), lo, seen, text, up);
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[u][i]);
    top = half_max(top) * a.scale_log2;
    // The maximum is raised only when it is passed by 2^8: p stays below 2^8 and its rounding is
    // relative, so the result is the same, and most tiles skip the rescaling of O.  Rows that are not past it
    // keep their sums as they are: a row's roundings do not depend on keys that only its neighbours see.
    const bool up = top > m + kRescaleStep;
    if (__any(up)) {
      const float f = !up ? 1.0f : m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
      m = up ? top : m;
#pragma unroll
      for (int i = 0; i < 4; ++i) l4[i] *= f;
      if constexpr (kTrue) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e4[i] *= f;
      }
#pragma unroll
      for (int i = 0; i < kOut; ++i) acc[i] *= f;
    }
    const float ms = m == -INFINITY ? 0.0f : m;
    bf16x8 p[NT][kSub * 2];
#pragma unroll
    for (int u = 0; u < kSub; ++u)
#pragma unroll
      for (int h2 = 0; h2 < 2; ++h2) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __builtin_amdgcn_exp2f(fmaf(sc[u][h2 * 8 + e], a.scale_log2, -ms));
        bf16x8 terms[NT];
        split_terms<NT>(x, terms);
        sum_p<NT>(x, terms[0], l4);
        if constexpr (kTrue) sum_p<2>(x, terms[0], e4);
#pragma unroll
        for (int n = 0; n < NT; ++n) p[n][u * 2 + h2] = terms[n];
      }
    // (the sums are taken here and not, as the compiler would have it, at the end of the round)
    asm volatile("" : "+v"(l4[0]), "+v"(l4[1]), "+v"(l4[2]), "+v"(l4[3]));
    if (tile + 1 < w.tile_hi) {
      stage(lds + (par ^ 1) * Sh::kBuffer, tile + 1);
      fetch(tile + 2);
      write_places(tile + 3);
      load_scales(tile + 4);
      load_pages(tile + 5);
    }
    {
      bf16x8 vf[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) vf[k] = value_operand(k);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < 2 * kSub * kOut; ++k) {
#pragma unroll
        for (int n = NT - 1; n >= 0; --n)
          acc[k % kOut] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[k % kAhead], p[n][k / kOut], acc[k % kOut], 0, 0, 0);
        if (k + kAhead < 2 * kSub * kOut) vf[k % kAhead] = value_operand(k + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (w.tile_lo < w.tile_hi) {  // what was left out, as in the kernel for few rows
    __syncthreads();
    const int odd_hi = __builtin_amdgcn_readfirstlane(odd_tiles[1]);
    for (int tile = __builtin_amdgcn_readfirstlane(odd_tiles[0]); tile <= odd_hi; ++tile)
      for (int i = 0; i < kKeys; ++i) {
        const int j = tile * kKeys + i;
        int slot;
        const uint8_t* blk = block_of_key(c, w, table, head, j, &slot);
        if (!blk) continue;
        const bool seen_j = sees<MODE>(j, lo, seen, text, above());
#pragma unroll
        for (int d = 0; d < kOut; ++d)
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const f32x4 x = nonfinite4<KIND>(c, blk, slot, part_dim + d * 32 + i4 * 8 + half * 4);
#pragma unroll
            for (int n = 0; n < 4; ++n)
              if (seen_j) acc[d][i4 * 4 + n] += x[n];
          }
      }
  }
  if (a.err && lost) atomicAdd(a.err, 1);

  const float l = half_sum((l4[0] + l4[1]) + (l4[2] + l4[3]));
  const float true_l = kTrue ? half_sum((e4[0] + e4[1]) + (e4[2] + e4[3])) : l;
  if (!live) return;
  const int64_t at = (int64_t)(s.first + t) * c.heads * share + qhead;
  if (MODE == kLse && a.splits == 1 && half == 0 && part == 0) a.lse[at] = log_sum(m, true_l);
  if (a.splits > 1) {
    if (half == 0 && part == 0) {
      const int64_t all = (int64_t)c.tokens * c.heads * share;
      a.stats[(split * all + at) * 2] = m;
      a.stats[(split * all + at) * 2 + 1] = true_l;
    }
    if (w.tile_lo >= w.tile_hi) return;
    if constexpr (kTrue) {  // the split's mean is of the rounded p, its weight in the join the true sum
      const float f = l == 0.0f ? 1.0f : true_l / l;
#pragma unroll
      for (int d = 0; d < kOut; ++d) acc[d] *= f;
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // no visible key: the row is zero
  const int64_t out_at = (int64_t)(s.first + t) * a.out_token + (int64_t)qhead * a.out_head;
#pragma unroll
  for (int d = 0; d < kOut; ++d)
#pragma unroll
    for (int i4 = 0; i4 < 4; ++i4)
      store_row4<NT>(a, at, out_at, split, part_dim + d * 32 + i4 * 8 + half * 4,
                     f32x4{acc[d][i4 * 4], acc[d][i4 * 4 + 1], acc[d][i4 * 4 + 2], acc[d][i4 * 4 + 3]}, inv);
}

// Joins the splits of a row under their common maximum.  A lane first takes the maximum and sum of two
// splits, so that the weights of all are known after one round of loads; then 64 / LANES splits of a wave
// are read side by side, four channels a lane, and what the waves of a row have is added in order through
// LDS.  WAVES waves a row: one where rows are many and splits few, four where a long axis left few rows of
// many splits.
constexpr int kMaxSplits = 128;

template <bool F32, int LANES, int WAVES, int MODE>
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
  // (rows that belong to no sequence are not written)
  const bool live = in && t >= c.starts[0] && t < c.starts[c.batch];

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
  if (MODE == kLse && live && lane == 0 && wave % WAVES == 0) a.lse[row] = log_sum(top, l);

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
