// The attention weight that cached tokens have received: for every key j of a sequence and key head,
//
//   w_j (+)= sum_i exp(scale q_i . k_j - lse_i)
//
// over the rows i (new tokens and query heads of the key head) that see it, lse_i the log-sum that the attention of the same
// rows gave.  With it a weight needs no other key: keys are shared out, rows are walked, nothing is split and joined, and
// no sum depends on an order of workgroups.
//
// S = Q K^T is taken with 32x32x16 bf16 instructions, rows down and keys across: a lane holds one key and 16 rows, so a
// key's sum is the lane's own (and its partner's, lane ^ 32).  A wave keeps its keys as operands in registers for the whole
// call, straight from memory, no LDS: which channels a step of the product takes does not matter as long as both operands
// agree, so a lane's 16 raw bytes (8, 16 or 32 channels) are one, two or four steps, and the rows are read from LDS in that
// order.  Scores, exponentials and sums are f32; f32 queries are three bf16 terms, as in attention.
//
// A decode step reads each key once for a handful of rows: HBM bounds it (64 tokens of 64 heads over 8 of 128 channels, up to
// 16384 keys in e4m3: 172 us, 4.2 TB/s, a large copy 5.1; with a workgroup for 256 keys and no loads ahead 367).  A chunk of a prompt
// walks thousands of rows over each key: the matrix instructions and the exponentials, a fused multiply-add, an exp and an add a
// score, share the time (chunks of 2 x 2048 over 8192, 32 heads, e4m3: 252 us, 950 TFLOP/s of 1250 that a large library product
// reaches; 187 us of it are left without exponentials and staging, 216 without the staging, 234 without the exponentials).  One
// token of 32 heads over 777 keys in bf16: 5.5 us.  f32 queries: 188 us and 621 (three matrix instructions for one, products and
// exponentials one after the other).
//
// The log-sum is taken to log2 units before the difference: that product's rounding is |lse| 2^-24 of a weight, as much as the
// log-sum's own as f32.
#pragma once

#include <type_traits>

#include "attn.h"
#include "serve_common.h"

namespace serve {

struct WeighArgs {
  Cache c;
  const void* q;
  const float* lse;  // [tokens][heads]
  float* weights;    // [pages][heads][page]
  int64_t q_token, q_head;
  Divider share;
  int32_t tiles;     // workgroups that share out the keys of a sequence
  int32_t units;     // of all sequences and key heads
  int32_t window, causal, fresh, max_rows, q_vec;
  float scale_log2;
  int32_t* err;
};

constexpr float kLog2e = 1.4426950408889634f;

// The keys that a row at a position sees: lo, .., lo + many - 1 (none where the row is none).
struct Seen {
  int lo;
  uint32_t many;
  __device__ __forceinline__ Seen(const WeighArgs& a, int pos, bool live) {
    lo = a.window > 0 ? max(pos - a.window + 1, 0) : 0;
    const int hi = a.causal ? pos + 1 : 0x7fffffff;
    many = live ? (uint32_t)max(hi - lo, 0) : 0;
  }
  __device__ __forceinline__ Seen(int lo_, int many_) : lo(lo_), many((uint32_t)many_) {}
  __device__ __forceinline__ bool holds(int j) const { return (uint32_t)(j - lo) < many; }
};

// 8 channels of a query row as they are loaded, and as NT bf16 terms.
template <bool F32>
struct Raw8 {
  u32x4 w[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw8<F32> raw_query(const uint8_t* from, bool vec, bool live) {
  Raw8<F32> r;
  r.w[0] = u32x4{0, 0, 0, 0};
  if constexpr (F32) r.w[1] = r.w[0];
  if (!live) return r;
  if (vec) {
    r.w[0] = reinterpret_cast<const u32x4*>(from)[0];
    if constexpr (F32) r.w[1] = reinterpret_cast<const u32x4*>(from)[1];
  } else if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i / 4][i & 3] = reinterpret_cast<const uint32_t*>(from)[i];
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(from);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[0][i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
  }
  return r;
}
template <int NT>
__device__ __forceinline__ void query_terms(const Raw8<NT == 3>& r, bf16x8* terms) {
  if constexpr (NT == 1) {
    terms[0] = __builtin_bit_cast(bf16x8, r.w[0]);
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i / 4][i & 3]);
    split_terms<NT>(x, terms);
  }
}

// The channels that a lane holds in step st of a product, lanes of `part` (of 64 / width parts) side by side.  A lane's 16 raw
// bytes are 1, 2 or 4 steps of 8 channels.
template <int KIND, int PARTS>
__device__ __forceinline__ constexpr int channel_of(int st, int part) {
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;
  return ((st / kOf) * PARTS + part) * 8 * kOf + st % kOf * 8;
}

// Where a key of a sequence lies.  The page number is loaded without waiting for the sequence's length.
template <int KIND, int DP>
struct KeyPlace {
  static constexpr int kWords = KIND == LLVQ_KV_BF16 ? 1 : DP <= 128 ? 1 : 2;  // of four scale bytes
  const uint8_t* blk;  // null if it has no place
  float* weight;
  int slot;
  __device__ __forceinline__ void find(const WeighArgs& a, int j, int len, int32_t id, int head, bool* lost) {
    const Cache& c = a.c;
    const bool in = j < len, ok = in && id >= 0 && id < c.pages;
    *lost |= in && !ok;
    slot = j - (int)(divide((uint32_t)j, c.page) * c.page.by);
    const int64_t at = (int64_t)(ok ? id : 0) * c.heads + head;
    blk = ok ? c.pool + at * c.block : nullptr;
    weight = ok ? a.weights + at * c.page.by + slot : nullptr;
  }
  __device__ __forceinline__ u32x4 chunk(const Cache& c, int ch) const {
    return blk && ch * 16 < c.row ? *reinterpret_cast<const u32x4*>(blk + slot * c.row + ch * 16) : u32x4{0, 0, 0, 0};
  }
  __device__ __forceinline__ void scales(const Cache& c, uint32_t* words) const {
#pragma unroll
    for (int n = 0; n < kWords; ++n) {
      words[n] = 0x7f7f7f7fu;
      if (KIND != LLVQ_KV_BF16 && blk) words[n] = scale_word(blk + c.ks_off + slot * c.groups, c.groups, n);
    }
  }
  static __device__ __forceinline__ uint32_t scale_of(const uint32_t* words, int group) {
    if constexpr (KIND == LLVQ_KV_BF16) return 127;
    const uint32_t word = kWords == 2 && group >= 4 ? words[kWords - 1] : words[0];
    return word >> (8 * (group & 3)) & 255;
  }
};
__device__ __forceinline__ int32_t page_id(const Cache& c, const int32_t* table, int j) {
  const uint32_t page = divide((uint32_t)j, c.page);
  return page < (uint32_t)c.max_pages ? table[page] : -1;
}

// Few rows: up to 16 RT of a (sequence, key head).  Every wave runs by itself over pieces of 32 keys, the codes, scales and
// weights of the next piece and the page numbers of the one after it under way; the rows are operands in registers for the
// whole call.  16x16x32 instructions: a lane holds one key of 16 and 4 rows, four lanes of a key read 64 consecutive bytes.
template <int KIND, int DP, int NT, int RT>
__global__ __launch_bounds__(256) void k_weigh_few(WeighArgs a) {
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;  // steps of a 16-byte chunk
  constexpr int kChunks = (DP / 32 + kOf - 1) / kOf, kSteps = kChunks * kOf;   // (e2m1, 64 wide: half the lanes have zeros)
  using Key = KeyPlace<KIND, DP>;
  const Cache& c = a.c;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
  int id = blockIdx.x;
  const int head = id % c.heads;
  id /= c.heads;
  const int b = id / a.tiles, tile = id % a.tiles;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  const int stride = a.tiles * 4;
  int piece = tile * 4 + wave;
  // (a piece's keys stay below 2^31: a sequence has up to 2^30)
  int32_t ids[2], next_ids[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) ids[u] = page_id(c, table, piece * 32 + u * 16 + col);
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, tokens = min(s.n, a.max_rows), rows = tokens * share, text = s.len - s.n, heads = c.heads * share;
  if (a.err && tid == 0 && head == 0 && tile == 0 && (s.bad || s.n > a.max_rows)) atomicAdd(a.err, 1);
  if (s.n == 0) return;
  // Without a fresh start, text before every row's window stays as it is
  const int low = !a.fresh && a.window > 0 ? max(text - a.window + 1, 0) : 0;
  if (low >= 32) {
    const int skip = low / 32;
    if (piece < skip) piece += (skip - piece + stride - 1) / stride * stride;
#pragma unroll
    for (int u = 0; u < 2; ++u) ids[u] = page_id(c, table, piece * 32 + u * 16 + col);
  }
  bool lost = false;
  Key key[2];
  u32x4 raw[2][kChunks];
  uint32_t words[2][Key::kWords];
  float old[2];
  auto fetch = [&](int p) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = p * 32 + u * 16 + col;
      key[u].find(a, j, s.len, ids[u], head, &lost);
#pragma unroll
      for (int m = 0; m < kChunks; ++m) raw[u][m] = key[u].chunk(c, 4 * m + g);
      key[u].scales(c, words[u]);
      old[u] = key[u].weight && !a.fresh && j < text ? *key[u].weight : 0.0f;
    }
  };
  const int pieces = (s.len + 31) / 32;
  if (piece < pieces) {
    fetch(piece);
#pragma unroll
    for (int u = 0; u < 2; ++u) next_ids[u] = page_id(c, table, min(piece + stride, pieces) * 32 + u * 16 + col);
  }
  // the rows: as operands by lane (row col), log-sums and positions by register (row 4 g + i)
  bf16x8 q[NT][RT][kSteps];
  float lse[RT][4];
  int lo[RT][4], many[RT][4];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int row = rt * 16 + col;
    const bool live = row < rows;
    const int t = live ? (int)divide((uint32_t)row, a.share) : 0;
    const int64_t at = (int64_t)(s.first + t) * a.q_token + (int64_t)(head * share + (live ? row - t * share : 0)) * a.q_head;
#pragma unroll
    for (int st = 0; st < kSteps; ++st) {
      bf16x8 terms[NT];
      const int ch = channel_of<KIND, 4>(st, g);
      query_terms<NT>(raw_query<NT == 3>(static_cast<const uint8_t*>(a.q) + (at + ch) * (NT == 3 ? 4 : 2), a.q_vec, live && ch < c.dim), terms);
#pragma unroll
      for (int n = 0; n < NT; ++n) q[n][rt][st] = terms[n];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = rt * 16 + 4 * g + i;
      const int tt = r < rows ? (int)divide((uint32_t)r, a.share) : 0;
      lse[rt][i] = r < rows ? a.lse[(int64_t)(s.first + tt) * heads + head * share + (r - tt * share)] * kLog2e : 0.0f;
      const Seen seen(a, text + tt, r < rows);
      lo[rt][i] = seen.lo;
      many[rt][i] = (int)seen.many;
    }
  }
  const bool full = rows == 16 * RT;
  while (piece < pieces) {
    const int next = piece + stride;
    bf16x8 k[2][kSteps];
    float* to[2];
    float was[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      nan_scales<KIND, Key::kWords>(words[u]);
#pragma unroll
      for (int m = 0; m < kChunks; ++m) {
        u32x4 o[kOf];
        expand<KIND>(raw[u][m], Key::scale_of(words[u], KIND == LLVQ_KV_FP8 ? 2 * m + (g >> 1) : 4 * m + g), o);
#pragma unroll
        for (int e = 0; e < kOf; ++e)
          k[u][m * kOf + e] = __builtin_bit_cast(bf16x8, o[e]);
      }
      to[u] = key[u].weight;
      was[u] = old[u];
    }
    if (next < pieces) {
#pragma unroll
      for (int u = 0; u < 2; ++u) ids[u] = next_ids[u];
      fetch(next);
#pragma unroll
      for (int u = 0; u < 2; ++u) next_ids[u] = page_id(c, table, min(next + stride, pieces) * 32 + u * 16 + col);
    }
    // whether every row sees every key
    const bool whole = full && (!a.causal || piece * 32 + 31 <= text) && (a.window == 0 || piece * 32 > text + tokens - 1 - a.window);
    auto work = [&](auto all) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = piece * 32 + u * 16 + col;
        float sum = 0.0f;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          f32x4 sc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int st = 0; st < kSteps; ++st)
#pragma unroll
            for (int n = NT - 1; n >= 0; --n) sc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[n][rt][st], k[u][st], sc, 0, 0, 0);
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(sc[i], a.scale_log2, -lse[rt][i]));
            if (!decltype(all)::value) p[i] = Seen(lo[rt][i], many[rt][i]).holds(j) ? p[i] : 0.0f;
          }
          sum += (p[0] + p[1]) + (p[2] + p[3]);
        }
        sum = quad_sum(sum);
        if (g == 0 && to[u]) *to[u] = was[u] + sum;
      }
    };
    if (whole)
      work(std::true_type());
    else
      work(std::false_type());
    piece = next;
  }
  if (a.err && lost) atomicAdd(a.err, 1);
}

// Many rows.  A workgroup's four waves hold 64 keys each (32 of wide heads) and walk the rows that see them, in blocks that the
// workgroup stages in LDS: a block's rows are loaded while the one before is worked on, and written to the other buffer after it.
// TEAM: waves that hold the same keys and share out a block's rows, 32 each, for few keys and heads: they leave compute units
// idle, and the rows are a long way.
template <int DP, int NT, int TEAM>
struct WeighShape {
  static constexpr int kTiles = DP <= 128 ? 2 : 1;     // of 32 keys that a wave holds
  static constexpr int kKeys = 4 / TEAM * 32 * kTiles; // of a workgroup
  static constexpr int kSub = NT == 1 && TEAM == 1 ? 2 : 1;  // pieces of 32 rows of a block that a wave takes
  static constexpr int kRows = 32 * kSub * TEAM;
  static constexpr int kRow = DP * 2 + 16;             // bytes of a row in LDS, padded as attention's keys are
  static constexpr int kWaves = 4 * NT * kRows * kRow > 150 * 1024 ? 1 : 2;  // a SIMD, by two workgroups' double buffers
};

template <int KIND, int DP, int NT, int TEAM>
__global__ __launch_bounds__(256, (WeighShape<DP, NT, TEAM>::kWaves)) void k_weigh_many(WeighArgs a) {
  using Sh = WeighShape<DP, NT, TEAM>;
  using Key = KeyPlace<KIND, DP>;
  constexpr int kSteps = DP / 16, kTiles = Sh::kTiles, kSub = Sh::kSub, kRows = Sh::kRows;
  constexpr int kOf = KIND == LLVQ_KV_BF16 ? 1 : KIND == LLVQ_KV_FP8 ? 2 : 4;  // steps of a 16-byte chunk
  constexpr int kChunks = kSteps / kOf;                                        // chunks of a lane and key
  constexpr int kParts = kRows * (DP / 8) / 256;                               // 8-channel parts of a block that a thread stages
  const Cache& c = a.c;
  __shared__ __align__(16) uint8_t rows_lds[2][NT][kRows * Sh::kRow];
  // (three: the last rows of a block are weighed while the next is multiplied and the one after that written)
  __shared__ __align__(16) float lse_lds[3][kRows];
  __shared__ __align__(16) int lo_lds[3][kRows], many_lds[3][kRows];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), mate = wave % TEAM;  // (which of a team's waves)
  const int half = lane >> 5, col = lane & 31;
  int id = blockIdx.x;
  const int head = id % c.heads;
  id /= c.heads;
  const int b = id / a.tiles, tile0 = id % a.tiles;
  const Seq s = sequence(c, b);
  const int share = (int)a.share.by, tokens = min(s.n, a.max_rows), rows = tokens * share, text = s.len - s.n, heads = c.heads * share;
  if (a.err && tid == 0 && head == 0 && tile0 == 0 && (s.bad || s.n > a.max_rows)) atomicAdd(a.err, 1);
  if (s.n == 0) return;
  const int32_t* table = c.table + (int64_t)b * c.max_pages;
  __shared__ float mates[TEAM == 1 ? 1 : 4][TEAM == 1 ? 1 : 32 * kTiles];
  bool lost = false;

  for (int tile = tile0; (int64_t)tile * Sh::kKeys < s.len; tile += a.tiles) {
    const int first_key = tile * Sh::kKeys, key0 = first_key + wave / TEAM * 32 * kTiles;
    const int last_key = min(first_key + Sh::kKeys, s.len) - 1;
    // the tokens that see any key of the workgroup's: [t0, t1)
    const int t0 = a.causal ? max(first_key - text, 0) : 0;
    const int64_t reach = (int64_t)last_key - text + a.window;
    const int t1 = a.window > 0 ? (int)min((int64_t)tokens, max(reach, (int64_t)0)) : tokens;
    const int block0 = t0 * share / kRows, block1 = t1 > t0 ? (int)(((int64_t)t1 * share + kRows - 1) / kRows) : block0;
    if (block0 >= block1 && !a.fresh && last_key < text) continue;  // nothing is added

    // A thread stages the same channels of every (256 / (DP / 8))-th row, and one of the first threads a row's log-sum; from
    // block to block all of them move on by kRows rows, dt tokens and dg heads.
    constexpr int kSize = NT == 3 ? 4 : 2;
    Raw8<NT == 3> staged[kParts];
    const int ch = tid % (DP / 8) * 8;
    const int dt = (int)divide((uint32_t)kRows, a.share), dg = kRows - dt * share;
    const int64_t step = ((int64_t)dt * a.q_token + (int64_t)dg * a.q_head) * kSize, wrap = (a.q_token - (int64_t)share * a.q_head) * kSize;
    const uint8_t* part_at[kParts];
    int part_g[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const int row = block0 * kRows + (i * 256 + tid) / (DP / 8), t = (int)divide((uint32_t)row, a.share);
      part_g[i] = row - t * share;
      part_at[i] = static_cast<const uint8_t*>(a.q) +
                   ((int64_t)(s.first + t) * a.q_token + (int64_t)(head * share + part_g[i]) * a.q_head + ch) * kSize;
    }
    int row_t, row_g;
    {
      const int row = block0 * kRows + tid;
      row_t = (int)divide((uint32_t)row, a.share);
      row_g = row - row_t * share;
    }
    float staged_lse = 0.0f;
    int staged_lo = 0, staged_many = 0;
    const bool simple = a.q_vec && c.dim == DP;
    auto load = [&](int block) {
      const bool every = (block + 1) * kRows <= rows;
      if (tid < kRows) {  // (a row that is none takes the first one's: no key is seen by it)
        const bool live = every || block * kRows + tid < rows;
        staged_lse = a.lse[(int64_t)(s.first + (live ? row_t : 0)) * heads + head * share + (live ? row_g : 0)];
        const Seen seen(a, text + row_t, live);
        staged_lo = seen.lo;
        staged_many = (int)seen.many;
      }
      if (simple && every) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
#pragma unroll
          for (int n = 0; n < kSize / 2; ++n) staged[i].w[n] = reinterpret_cast<const u32x4*>(part_at[i])[n];
        }
      } else {
#pragma unroll
        for (int i = 0; i < kParts; ++i)
          staged[i] = raw_query<NT == 3>(part_at[i], a.q_vec, ch < c.dim && block * kRows + (i * 256 + tid) / (DP / 8) < rows);
      }
#pragma unroll
      for (int i = 0; i < kParts; ++i) part_at[i] += step;
      row_t += dt;
      if (dg) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          part_g[i] += dg;
          if (part_g[i] >= share) part_g[i] -= share, part_at[i] += wrap;
        }
        row_g += dg;
        if (row_g >= share) row_g -= share, ++row_t;
      }
    };
    auto write = [&](int buffer, int slot) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int r = (i * 256 + tid) / (DP / 8);
        bf16x8 terms[NT];
        query_terms<NT>(staged[i], terms);
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<bf16x8*>(&rows_lds[buffer][n][r * Sh::kRow + ch * 2]) = terms[n];
      }
      if (tid < kRows) {
        lse_lds[slot][tid] = staged_lse * kLog2e;
        lo_lds[slot][tid] = staged_lo;
        many_lds[slot][tid] = staged_many;
      }
    };

    if (block0 < block1) load(block0);
    // the keys
    float* to[kTiles];
    float old[kTiles], sum[kTiles][4];
    bf16x8 k[kTiles][kSteps];
#pragma unroll
    for (int u = 0; u < kTiles; ++u) {
      const int j = key0 + u * 32 + col;
      Key key;
      key.find(a, j, s.len, page_id(c, table, j), head, &lost);
      u32x4 raw[kChunks];
      uint32_t words[Key::kWords];
#pragma unroll
      for (int m = 0; m < kChunks; ++m) raw[m] = key.chunk(c, 2 * m + half);
      key.scales(c, words);
      to[u] = key.weight;
      old[u] = key.weight && !a.fresh && j < text ? *key.weight : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[u][i] = 0.0f;
      nan_scales<KIND, Key::kWords>(words);
#pragma unroll
      for (int m = 0; m < kChunks; ++m) {
        u32x4 o[kOf];
        expand<KIND>(raw[m], Key::scale_of(words, KIND == LLVQ_KV_FP8 ? m : 2 * m + half), o);
#pragma unroll
        for (int e = 0; e < kOf; ++e) k[u][m * kOf + e] = __builtin_bit_cast(bf16x8, o[e]);
      }
    }
    __syncthreads();  // (the tile before has been worked through)
    if (block0 < block1) write(0, 0);
    // The products of 32 rows run beside the exponentials of the 32 before them.
    f32x16 scores[2][kTiles];
    auto products = [&](int buffer, int sub, f32x16* sc) {
#pragma unroll
      for (int u = 0; u < kTiles; ++u) sc[u] = f32x16{0.0f};
#pragma unroll
      for (int st = 0; st < kSteps; ++st)
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) {
          const bf16x8 qf = *reinterpret_cast<const bf16x8*>(
              &rows_lds[buffer][n][((sub + mate) * 32 + col) * Sh::kRow + channel_of<KIND, 2>(st, half) * 2]);
#pragma unroll
          for (int u = 0; u < kTiles; ++u) sc[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf, k[u][st], sc[u], 0, 0, 0);
        }
    };
    auto weigh = [&](auto all, int slot, int sub, const f32x16* sc) {
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const int r = (sub + mate) * 32 + i4 * 8 + half * 4;
        const f32x4 l = *reinterpret_cast<const f32x4*>(&lse_lds[slot][r]);
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          const int j = key0 + u * 32 + col;
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = __builtin_amdgcn_exp2f(fmaf(sc[u][i4 * 4 + i], a.scale_log2, -l[i]));
            if (!decltype(all)::value) p[i] = Seen(lo_lds[slot][r + i], many_lds[slot][r + i]).holds(j) ? p[i] : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[u][i] += p[i];
        }
      }
    };
    // Both, for a whole block whose rows, and the 32 before it, all see all keys (its last 32 are weighed with the next):
    // after each matrix instruction a share of the exponentials, in an order that is pinned, since the two waves of a SIMD fall
    // into step and do not overlap the one's products with the other's sums (chunks of 2 x 2048 over 8192: 293 us one after
    // the other, 321 in the compiler's order, 265 so)
    auto both = [&](int buffer, int slot, int slot_before) {
      constexpr int kAhead = NT == 1 ? 3 : 2, kPer = 16 / kSteps, kAll = kSteps * kTiles, kGroup = 4 * kTiles;
      const uint8_t* from = &rows_lds[buffer][0][col * Sh::kRow];
      auto operand = [&](int i, int n) {  // of step i, counted over the block
        return *reinterpret_cast<const bf16x8*>(from + (n * kRows + i / kSteps * 32) * Sh::kRow + channel_of<KIND, 2>(i % kSteps, half) * 2);
      };
      auto sums_of = [&](int i) {  // four log-sums of the 4 i-th row on, counted over the 32 before and the block
        return *reinterpret_cast<const f32x4*>(i < 4 ? &lse_lds[slot_before][(kSub - 1) * 32 + i * 8 + half * 4]
                                                     : &lse_lds[slot][(i - 4) * 8 + half * 4]);
      };
      bf16x8 qf[kAhead][NT];
      f32x4 l[2];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) qf[i][n] = operand(i, n);
      l[0] = sums_of(0);
      float p[kPer];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int m = 0; m < kSub * kAll; ++m) {
        const int i = m / kTiles, u = m % kTiles, sub = m / kAll;
        f32x16& sc = scores[kSub == 1 ? 0 : sub & 1][u];
        if (i % kSteps == 0) sc = f32x16{0.0f};
#pragma unroll
        for (int n = NT - 1; n >= 0; --n) sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(qf[i % kAhead][n], k[u][i % kSteps], sc, 0, 0, 0);
        if (u == kTiles - 1 && i + kAhead < kSub * kSteps) {
#pragma unroll
          for (int n = 0; n < NT; ++n) qf[i % kAhead][n] = operand(i + kAhead, n);
        }
        // an element: rows by four, of each the tiles (added an instruction after their exponential)
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int e = (m - 1) * kPer + x;
          if (m > 0) sum[e % kGroup / 4][e & 3] += p[x];
        }
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          const int e = m * kPer + x, i4 = e / kGroup;
          if (e % kGroup == 0 && i4 + 1 < 4 * kSub) l[(i4 + 1) & 1] = sums_of(i4 + 1);
          const f32x16& old = scores[(sub + kSub - 1) % kSub & 1][e % kGroup / 4];
          p[x] = __builtin_amdgcn_exp2f(fmaf(old[i4 % 4 * 4 + (e & 3)], a.scale_log2, -l[i4 & 1][e & 3]));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int x = 0; x < kPer; ++x) sum[kTiles - 1][((kSub * kAll - 1) * kPer + x) & 3] += p[x];
    };
    // whether every one of 32 rows sees every key of the wave's (positions ascend with the rows)
    auto whole = [&](int r0) {
      const int p0 = text + (int)divide((uint32_t)r0, a.share), p1 = text + (int)divide((uint32_t)(r0 + 31), a.share);
      return r0 + 32 <= rows && (!a.causal || key0 + 32 * kTiles - 1 <= p0) && (a.window == 0 || key0 > p1 - a.window);
    };
    enum { kNone, kWhole, kMasked } before = kNone;
    int slot = 0, slot_before = 0;
    for (int block = block0; block < block1; ++block) {
      const int buffer = (block - block0) & 1;
      __syncthreads();
      if (block + 1 < block1) load(block + 1);
      bool fast = kSub > 1 && before == kWhole;
#pragma unroll
      for (int sub = 0; sub < kSub - 1; ++sub) fast = fast && whole(block * kRows + sub * 32);
      if (fast) {
        both(buffer, slot, slot_before);
      } else {
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          const int last = (sub + kSub - 1) % kSub;  // the 32 rows before
          if (kSub > 1 && before != kNone) weigh(std::false_type(), sub == 0 ? slot_before : slot, last, scores[last & 1]);
          products(buffer, sub, scores[kSub == 1 ? 0 : sub & 1]);
          before = kMasked;
          if (kSub == 1) {
            if (whole(block * kRows + mate * 32))
              weigh(std::true_type(), slot, 0, scores[0]);
            else
              weigh(std::false_type(), slot, 0, scores[0]);
          }
        }
      }
      before = whole(block * kRows + (kSub - 1) * 32) ? kWhole : kMasked;
      slot_before = slot;
      slot = slot == 2 ? 0 : slot + 1;
      if (block + 1 < block1) write(buffer ^ 1, slot);
    }
    if (kSub > 1 && before != kNone) weigh(std::false_type(), slot_before, kSub - 1, scores[(kSub - 1) & 1]);
    // what the new tokens' places held is of earlier tokens
    float got[kTiles];
#pragma unroll
    for (int u = 0; u < kTiles; ++u) got[u] = half_sum((sum[u][0] + sum[u][1]) + (sum[u][2] + sum[u][3]));
    if constexpr (TEAM > 1) {  // the team's sums, in the waves' order
#pragma unroll
      for (int u = 0; u < kTiles; ++u)
        if (half == 0) mates[wave][u * 32 + col] = got[u];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kTiles; ++u) {
        got[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < TEAM; ++i) got[u] += mates[wave - mate + i][u * 32 + col];
      }
    }
#pragma unroll
    for (int u = 0; u < kTiles; ++u)
      if (mate == 0 && half == 0 && to[u]) *to[u] = old[u] + got[u];
  }
  if (a.err && lost) atomicAdd(a.err, 1);
}

}  // namespace serve
