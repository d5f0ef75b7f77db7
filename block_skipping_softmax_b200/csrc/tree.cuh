// What the tree-attention kernels share: the sequences, the distribution of
// their work, and small helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.cuh"
#include "ptx.cuh"

namespace bss {

constexpr int kPage = kDecodeTile;  // 64 keys: one page, one tile
constexpr int kManyRows = 128;      // rows of a CTA of the tcgen05 kernel
constexpr unsigned kFull = 0xffffffffu;
constexpr float kRefSlack = 8.f;  // log2 units: the reference maximum lags by less, so p < 2^8

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// mbar_wait in fewer instructions, for kernels whose roles wait in many places:
// one poll, and a look at the flag and the clock every 64.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                          uint64_t limit_ns) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*abort_flag || now - t0 > limit_ns) return false;
    }
  }
}

__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u) || ((w & 0x7f800000u) == 0x7f800000u);
}

// ---- e4m3 codes in registers ------------------------------------------------

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Two codes in the upper bytes of the halfwords of w (the lower bytes may hold
// anything) to two bf16: sign, exponent and mantissa move to their bf16
// places, and 2^120 moves the exponent's bias from 7 to 127, subnormal codes
// included.  Exact.  The NaN code (0x7f) comes out as 480: the writer never
// stores it under a finite scale, and a NaN scale makes the value NaN.
__device__ __forceinline__ uint32_t e4m3_hi_to_bf16x2(uint32_t w) {
  return mul_bf16x2((w & 0x80008000u) | ((w >> 4) & 0x07f007f0u), 0x7b807b80u);
}

// Four codes (bytes of w) to two pairs of fp16, in order.  Exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Queries meet e4m3 keys as fp16, since the codes become fp16 in one
// instruction a pair.  A row is scaled by the power of two that brings its
// largest element to [2^14, 2^15): bf16's 8 bits fit in fp16's 11, so every
// element within 2^-28 of the largest is exact, and a smaller one is off by at
// most 2^-40 of the largest.  Returns the factor's exponent; 0 for a row of
// zeros or with inf or NaN.
__device__ __forceinline__ int f16_shift(uint32_t amax_bits) {
  if (amax_bits == 0 || amax_bits >= 0x7f800000u) return 0;
  return min(14 + 127 - static_cast<int>(amax_bits >> 23), 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Values of an e4m3 cache are fp16 operands too where that is exact: a code
// (a multiple of 2^-9 up to 448) times a scale from 2^-15 to 2^7 has a place in
// fp16.  A tile with a scale outside of that takes bf16 operands, at more
// instructions a code.  Probabilities carry 2^7, so that fp16 (up to 65504)
// holds them from p = 2^8 down to 2^-31 of the reference maximum.
constexpr int kPShift = 7;
// How far a scale lies above 2^-15, in steps of floats: kFitsF16 and less up to
// 2^7, more for larger, smaller, negative ones and NaN.  The maximum of several
// says whether all fit.
__device__ __forceinline__ uint32_t over_f16(float scale) { return __float_as_uint(scale) - 0x38000000u; }
constexpr uint32_t kFitsF16 = 0x43000000u - 0x38000000u;

// The exponents of two probabilities: (score - reference) * scale, in log2 units.
// minus(reference) is 0 where nothing has been seen so far: then all p are 0.
__device__ __forceinline__ float minus(float ref) { return ref == neg_inf() ? 0.f : -ref; }
template <bool SHIFT>
__device__ __forceinline__ float2 log2_p(float2 score, float2 from, float2 by) {
  const float2 x = __fadd2_rn(score, from);
  return SHIFT ? __ffma2_rn(x, by, make_float2(kPShift, kPShift)) : __fmul2_rn(x, by);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// ---- sequences and work -----------------------------------------------------

struct Seq {
  int tok0, T;      // first row of the packed batch, tokens
  int len, prefix;  // keys; keys that every token sees
};

__device__ __forceinline__ Seq seq_of(const TreeLaunch& a, int b) {
  Seq s;
  const int c0 = __ldg(a.cu_q + b), c1 = __ldg(a.cu_q + b + 1), n = __ldg(a.seq_lens + b);
  s.tok0 = min(max(c0, 0), a.total_q);
  s.T = min(min(max(c1, s.tok0), a.total_q) - s.tok0, a.max_q);
  s.len = max(0, min(min(n, a.L), a.max_pages * kPage));
  s.prefix = max(0, s.len - s.T);
  return s;
}

// The host either gives every KV head of every sequence a CTA of its own, which
// finds it without looking at other sequences (1000 sequences of 500 keys: 201 us,
// 464 by way of the line), or has the device divide the work by the lengths:
// the work of one plane (row block `plane` of every sequence that has one) is
// the line of all its tiles, sequences, KV heads and tiles in this order.  It
// is divided among the plane's CTAs in one of two ways.
//   By heads: every KV head's tiles go to `shares` CTAs of their own.
//   Equal pieces: the line is cut into pieces of the same cost, whatever the
//   sequences' lengths, so a ragged batch keeps every SM busy to the end.  A
//   piece consists of segments, runs of tiles of one KV head.
// A segment has its own start and end (queries, first copies, adding up the
// warps' sums), worth about kSegment tiles: every KV head has as many places on
// the line more than tiles, behind them, so that a piece across a head's end has
// fewer tiles.  (By tiles alone the CTAs with two segments ended 3 to 12 us behind the
// others: 64 tokens x 64 heads over 4 x 16384 keys 155 us before the merge instead of
// 147; under a load of seconds, where the power limit holds the clocks down, a pass
// 196 instead of 194.)  Heads are kept whole where their longest share is no longer
// than an equal piece.
//
// A segment that is not all of its KV head's tiles leaves a share of the result
// in one of the CTA's two places (only its first and its last segment can be
// one), which tree_merge_kernel adds up.  A sequence without keys counts as one
// tile, so that its zeros get written.
//
// Planes run side by side over the same line, so that row blocks that read the
// same pages do so at about the same time, from L2.
constexpr int kSegment = 6;

// 32 sequences of the line; a plane has fewer than 2^31 places (the host checks).
struct Line {
  int tiles;             // of this lane's sequence, at least 1; 0: it has no rows on the plane
  int incl, before;      // places of all heads up to it, and before the chunk
  unsigned active;       // lanes with rows
  int heads;             // KV heads before the chunk
  int chunk;

  // tiles of sequence b, 0 without rows on the plane
  __device__ __forceinline__ static int tiles_of(const TreeLaunch& a, int b, int first_row) {
    const Seq s = seq_of(a, b);
    return s.T * (a.Hq / a.Hkv) > first_row ? max(1, (s.len + kPage - 1) / kPage) : 0;
  }
  // Warp-collective: the sequences from `at` on.
  __device__ __forceinline__ void load(const TreeLaunch& a, int first_row, int at, int tiles_before, int heads_before) {
    const int lane = threadIdx.x & 31;
    chunk = at;
    before = tiles_before;
    heads = heads_before;
    tiles = at + lane < a.B ? tiles_of(a, at + lane, first_row) : 0;
    active = __ballot_sync(kFull, tiles > 0);
    incl = places(a);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
  }
  // of this lane's sequence: kSegment more than tiles for each KV head
  __device__ __forceinline__ int places(const TreeLaunch& a) const { return tiles ? (tiles + kSegment) * a.Hkv : 0; }
  __device__ __forceinline__ void next(const TreeLaunch& a, int first_row) {
    load(a, first_row, chunk + 32, before + total(), heads + __popc(active) * a.Hkv);
  }
  __device__ __forceinline__ int total() const { return __shfl_sync(kFull, incl, 31); }
  // KV heads before lane l's sequence
  __device__ __forceinline__ int heads_at(const TreeLaunch& a, int l) const {
    return heads + __popc(active & ((1u << l) - 1)) * a.Hkv;
  }
};

struct Division {
  int shares;            // by heads: CTAs of a head; 0: equal pieces
  int used, each, more;  // equal pieces: CTAs, the first `more` with one place more than `each`

  // Warp-collective; leaves the line at its first chunk.
  __device__ __forceinline__ Division(const TreeLaunch& a, int first_row, Line& line) {
    line.load(a, first_row, 0, 0, 0);
    int most = line.tiles, W = line.places(a), heads = line.tiles ? a.Hkv : 0;
    for (int b = 32 + (threadIdx.x & 31); b < a.B; b += 32) {
      const int tiles = line.tiles_of(a, b, first_row);
      most = max(most, tiles);
      W += tiles ? (tiles + kSegment) * a.Hkv : 0;
      heads += tiles ? a.Hkv : 0;
    }
    most = __reduce_max_sync(kFull, most);
    W = __reduce_add_sync(kFull, W);
    heads = __reduce_add_sync(kFull, heads);
    shares = used = each = more = 0;
    if (W == 0) return;
    used = max(1, min(a.ctas, (W - 1) / a.min_tiles + 1));
    each = W / used;
    more = W - each * used;
    if (heads <= a.ctas) {
      const int n = min(a.ctas / heads, (most - 1) / a.min_tiles + 1);
      if ((most - 1) / n + 1 <= each) {
        shares = n;
        used = heads * n;
      }
    }
  }
  __device__ __forceinline__ int first(int cta) const { return each * cta + min(cta, more); }
  __device__ __forceinline__ int cta_of(int place) const {
    const int split = (each + 1) * more;
    return place < split ? place / (each + 1) : more + (place - split) / each;
  }
};

struct Segment {
  int b, kv;
  int t0, nt;      // tiles [t0, t0 + nt) of the sequence
  int row0, rows;  // rows of this plane: row r is token (row0 + r) / g, head (row0 + r) % g of the group
  bool whole;      // all tiles: the result is final
  int place;       // else where the share goes: 0 (the CTA's first segment) or 1
  Seq s;
};

// The segments of this CTA, for every warp by itself (all calls warp-collective).
struct Segments {
  Line line;
  int shares, begin, pos, end;  // by heads: begin is the share, pos the KV head, end one further

  __device__ __forceinline__ void start(const TreeLaunch& a, int per) {
    const int i = blockIdx.x;
    if (a.min_tiles == 0) {  // a CTA for each KV head of each sequence
      shares = 0;
      begin = 0;
      pos = i;
      end = i + 1;
      return;
    }
    const Division d(a, blockIdx.y * per, line);
    shares = d.shares;
    begin = pos = end = 0;
    if (i >= d.used) return;
    if (shares) {
      pos = i / shares;
      begin = i - pos * shares;
      end = pos + 1;
    } else {
      begin = pos = d.first(i);
      end = d.first(i + 1);
    }
  }
  __device__ __forceinline__ bool next(const TreeLaunch& a, int per, Segment& g) {
    const int row0 = blockIdx.y * per;
    if (a.min_tiles == 0) {
      if (pos >= end) return false;
      g.b = pos / a.Hkv;
      g.kv = pos - g.b * a.Hkv;
      ++pos;
      g.s = seq_of(a, g.b);
      g.row0 = row0;
      g.rows = min(per, g.s.T * (a.Hq / a.Hkv) - row0);
      g.t0 = 0;
      g.nt = (g.s.len + kPage - 1) / kPage;
      g.whole = true;
      g.place = 0;
      return g.rows > 0;
    }
    int l, first, span;  // the lane of the sequence; its first KV head, or place of the line; places of tiles
    for (;;) {
      if (pos >= end) return false;
      if (shares) {
        while (pos >= line.heads + __popc(line.active) * a.Hkv) line.next(a, row0);
        const int lane = threadIdx.x & 31, mine = line.heads_at(a, lane);
        l = __ffs(__ballot_sync(kFull, ((line.active >> lane) & 1) && pos >= mine && pos < mine + a.Hkv)) - 1;
        first = line.heads_at(a, l);
        span = __shfl_sync(kFull, line.tiles, l);
        break;
      }
      while (pos >= line.before + line.total()) line.next(a, row0);
      l = __ffs(__ballot_sync(kFull, pos < line.before + line.incl)) - 1;
      first = line.before + __shfl_sync(kFull, line.incl - line.places(a), l);
      span = __shfl_sync(kFull, line.tiles, l);
      g.kv = (pos - first) / (span + kSegment);
      first += g.kv * (span + kSegment);
      if (pos - first < span) break;
      pos = first + span + kSegment;  // behind a head's last tile
    }
    g.b = line.chunk + l;
    g.s = seq_of(a, g.b);
    const int tiles = (g.s.len + kPage - 1) / kPage;
    g.row0 = row0;
    g.rows = min(per, g.s.T * (a.Hq / a.Hkv) - row0);
    if (shares) {
      const int share = begin;
      g.kv = pos - first;
      ++pos;
      const int from = static_cast<int>(static_cast<long long>(span) * share / shares);
      const int to = static_cast<int>(static_cast<long long>(span) * (share + 1) / shares);
      if (from == to) return false;  // fewer tiles than shares
      g.t0 = from;
      g.nt = min(to, tiles) - from;
      g.whole = to - from == span;
      g.place = 0;
      return true;
    }
    g.t0 = pos - first;
    const int n = min(span - g.t0, end - pos);
    g.nt = min(n, tiles - g.t0);
    g.whole = n == span;
    g.place = first <= begin ? 0 : 1;
    pos += g.t0 + n == span ? n + kSegment : n;
    return true;
  }
};

// Row r of a segment: its row of q and o, [total_q * Hq].
__device__ __forceinline__ size_t row_at(const TreeLaunch& a, const Segment& g, int r, int* token = nullptr) {
  const int group = a.Hq / a.Hkv;
  const int t = (g.row0 + r) / group;
  if (token) *token = t;
  return static_cast<size_t>(g.s.tok0 + t) * a.Hq + g.kv * group + (g.row0 + r) - t * group;
}
// its row of part and sums
__device__ __forceinline__ size_t share_at(const TreeLaunch& a, int per, int plane, int cta, int place, int r) {
  return ((static_cast<size_t>(plane) * a.ctas + cta) * 2 + place) * per + r;
}
// drafted keys that token t sees
__device__ __forceinline__ uint64_t bits_of(const TreeLaunch& a, const Seq& s, int t) {
  return a.mask ? a.mask[s.tok0 + t] : (t >= 63 ? ~0ull : (2ull << t) - 1);
}

// What a row without a sum gets, with these bits: 0 if it sees no key, else NaN:
// its scores are all -inf, over which softmax has no value.
__device__ __forceinline__ float without_sum(const Seq& s, uint64_t bits) {
  const bool sees = s.prefix > 0 || (bits & (s.len >= 64 ? ~0ull : (1ull << s.len) - 1)) != 0;
  return sees ? __int_as_float(0x7fffffff) : 0.f;
}

// Tensor map over a pool of e4m3 codes [groups, 64, D], d fastest: boxes of
// `keys` keys, rows swizzled as 128 bytes (D = 128) or 64 (D = 64); groups past
// the end read as zeros.
bool tma_map_codes(CUtensorMap* m, const void* base, long long groups, int D, int keys);

}  // namespace bss
