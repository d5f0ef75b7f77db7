// Tree attention for few rows a KV head (the decode of single tokens, small
// drafts): 8 NT rows a CTA on warp-level MMAs (m16n8k16).
//
// Such a call is bound by the bytes of K and V: with R rows a key's 2 d bytes
// of e4m3 (4 d of bf16) meet 4 R d flops.  So the keys take the long side of the
// MMAs and the rows the short one,
//   S^T [16 keys x 8 rows] = K Q^T,   O^T [16 of d x 8 rows] += V^T P^T,
// and a tile costs as many instructions as its bytes ask for.  A warp takes 16
// or 32 of a page's keys for all rows, with its own copies, its own ring in
// shared memory, its own running maximum and sums: nothing is exchanged between
// warps until the end of a segment, and no warp only copies.
//
// Fragments are read straight from the swizzled tiles, 16 bytes of a key row
// at a time: the order of d inside a k-step of K Q^T, of keys inside one of
// V^T P^T, and of the rows of O^T is free, and is chosen so that no operand is
// transposed in shared memory and no read of 128-byte rows meets a bank twice.
// Only P, 16-bit by then, changes its layout, by two register transposes of 8 x 8.
// e4m3 codes become fp16 in registers (or, for values of unusual scales, bf16),
// so they cross shared memory once, as bytes.
//
// Measured, 16 sequences x 16384 keys, 8 KV heads: e4m3 of 128 with 4 rows 98 us
// (5.6 TB/s of the 6.55 of a copy), with 16 rows 112 (4.9 TB/s); of 64 with 4 rows
// 58 and with 16 rows 75 (4.7 and 3.7 TB/s); bf16 of 128 166 (6.5 TB/s), of 64 90.
// 16 x 32768 e4m3 keys, 4 rows: 184 (5.9 TB/s); 250 with the rows on the MMAs' long
// side and one warp that only copied.  Heads of 64 take three quarters of the
// instructions of heads of 128 for half the bytes (scales, mask, softmax and sums
// go by the key): 12 warps an SM, half of the issue slots used, stalls of fixed
// latency.  Heads of 128 with 16 rows take 231 registers and 77 KB, two CTAs an SM
// (8 warps, 40% of the issue slots, tensor pipe 30%); with three asked for, of which
// two fitted, the third of the equal pieces came after the others, and 212 bytes
// were spilled (163 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace bss {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSmSmem = 233472;  // shared memory of an SM, of which every CTA takes 1 KB besides its own

template <int D, bool E4M3, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kKB = kRowBytes == 256 ? 1 : 2;         // blocks of 16 keys that a warp takes of a page
  static constexpr int kKeys = 16 * kKB;
  static constexpr int kShare = kPage / kKeys;                 // warps that share a page
  static constexpr int kEvery = kWarps / kShare;               // a warp takes every kEvery-th page
  static constexpr int kTile = kKeys * kRowBytes;              // a warp's keys (or values) of a page
  static constexpr int kPanels = E4M3 ? 1 : D / 64;            // swizzled panels of it
  static constexpr int kScaleBytes = E4M3 ? kKeys * 4 : 0;
  static constexpr int kStages = kRowBytes == 64 ? 4 : 2;
  static constexpr int kStageBytes = 2 * kTile;
  static constexpr int kOffScale = kWarps * kStages * kStageBytes;  // [warp][stage][K, V][keys] floats
  static constexpr int kOffRed = kOffScale + kWarps * kStages * 2 * kScaleBytes;  // rows x D floats
  static constexpr int kOffMax = kOffRed + kRows * D * 4;           // [warp][row] maxima, then sums
  static constexpr int kOffBar = kOffMax + 2 * kWarps * kRows * 4;  // [warp][stage]
  static constexpr int kOffMisc = kOffBar + kWarps * kStages * 8;   // abort
  static constexpr int kSmem = kOffMisc + 16 + 1024;
  // CTAs of an SM, which the division of the work counts on
  static constexpr int kCtas = E4M3 && D == 128 && NT == 2 ? 2 : 3;
  static_assert(kCtas * (kSmem + 1024) <= kSmSmem, "all of them resident");
};

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit values: lane (n, q) gives row n, columns 2q and
// 2q+1, and gets the same of the transposed matrix.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Lane = (n, q) = (lane / 4, lane % 4).  Row n of a block of 8 score rows is key
// key_of(n) of its 8 keys; the pair that a lane meets in V^T P^T, columns 2q and
// 2q+1, is key_of(2q) and kStep further.  With 128-byte rows the order
// 0 4 1 5 2 6 3 7 keeps the eight lanes of a 16-byte read on eight different
// banks; 64-byte rows (two a bank line) do so in their own order.
template <int D, bool E4M3>
struct Lanes {
  static constexpr bool kNarrow = E4M3 && D == 64;
  static constexpr int kStep = kNarrow ? 1 : 4;
  __device__ __forceinline__ static int key_of(int n) { return kNarrow ? n : ((n & 1) << 2) | (n >> 1); }
};

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, E4M3, NT>::kCtas)
    tree_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ TreeLaunch a) {
  using C = Cfg<D, E4M3, NT>;
  using LN = Lanes<D, E4M3>;
  constexpr int KB = C::kKB, kRows = C::kRows;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;  // the swizzle pattern repeats every 1024 B
  uint8_t* smem = smem_raw + (sbase - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bars = sbase + C::kOffBar + 8u * (warp * C::kStages);
  const uint32_t ring = sbase + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_scale = sbase + C::kOffScale + warp * C::kStages * 2 * C::kScaleBytes;
  const int part = warp % C::kShare, first_page = warp / C::kShare;  // this warp's keys of a page, its pages

  asm volatile("griddepcontrol.launch_dependents;");  // the merge may look for its shares
  if (threadIdx.x == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  Segments list;
  list.start(a, kRows);
  Segment sg{};
  __syncthreads();

  const int n = lane >> 2, q = lane & 3;
  const int key_n = LN::key_of(n);       // key of score row n; V chunk of O^T row n
  const int key_lo = LN::key_of(2 * q);  // first key of this lane's V pairs
  // byte offsets of this lane's reads, of a block of 8 keys (16-byte chunk c of
  // key row r lies at c ^ (r % 8), or at c ^ (r / 2 % 4) with 64-byte rows)
  const uint32_t k_at = LN::kNarrow ? key_n * 64 + ((q ^ ((key_n >> 1) & 3)) << 4) : key_n * 128 + ((q ^ key_n) << 4);
  uint32_t v_at[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = key_lo + e * LN::kStep;
    v_at[e] = LN::kNarrow ? r * 64 + (((n >> 1) ^ ((r >> 1) & 3)) << 4) + (n & 1) * 8 : r * 128 + ((key_n ^ r) << 4);
  }
  constexpr int kBlock = LN::kNarrow ? 8 * 64 : 8 * 128;  // bytes of 8 keys
  constexpr int kPanel = C::kKeys * 128;                  // bf16: of a panel

  float* red = reinterpret_cast<float*>(smem + C::kOffRed);   // [fragment register][lane]
  float* wmax = reinterpret_cast<float*>(smem + C::kOffMax);  // [warp][row]
  float* wsum = wmax + kWarps * kRows;
  int slot = 0;           // of the ring, and its phase
  uint32_t phase = 0;
  bool ok = true;         // after a wait gave up the warp only keeps up with the barriers

  while (list.next(a, kRows, sg)) {
    const int* table = a.block_table + static_cast<size_t>(sg.b) * a.max_pages + sg.t0;
    const int mine = sg.nt > first_page ? (sg.nt - first_page - 1) / C::kEvery + 1 : 0;  // this warp's pages
    auto page_at = [&](int i) { return i < mine ? table[i * C::kEvery + first_page] : -1; };
    // lane i: the page of tile i of the 32 tiles that are being issued, and of the next 32
    int pages = page_at(lane), pages_next = page_at(lane + 32);
    unsigned bad = 0;  // bit s: the page id of slot s was out of range
    // warp-collective: copies this warp's part of its i-th page to slot s
    auto issue = [&](int i, int s) {
      if (i >= 32 && (i & 31) == 0) {
        pages = pages_next;
        pages_next = page_at(i + 32 + lane);
      }
      const int page = __shfl_sync(kFull, pages, i & 31);
      const bool good = static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
      if constexpr (E4M3) bad = (bad & ~(1u << s)) | (good ? 0u : 1u << s);
      if (lane == 0) {
        // an id out of range reads zeros: its box lies past the pool's end
        const int grp = (good ? page : a.num_pages) * a.Hkv + sg.kv;
        const uint32_t bar = bars + 8 * s, dst = ring + s * C::kStageBytes;
        mbar_arrive_expect_tx(bar, C::kStageBytes + (good ? 2 * C::kScaleBytes : 0));
#pragma unroll
        for (int p = 0; p < C::kPanels; ++p) {
          tma_load_3d(dst + p * kPanel, &tmK, bar, p * 64, part * C::kKeys, grp);
          tma_load_3d(dst + C::kTile + p * kPanel, &tmV, bar, p * 64, part * C::kKeys, grp);
        }
        if constexpr (E4M3) {
          if (good) {
            const uint32_t to = ring_scale + s * 2 * C::kScaleBytes;
            const long long at = static_cast<long long>(grp) * kPage + part * C::kKeys;
            bulk_load(to, a.k_scales + at, C::kScaleBytes, bar);
            bulk_load(to + C::kScaleBytes, a.v_scales + at, C::kScaleBytes, bar);
          }
        }
      }
    };
    if (ok)
      for (int i = 0; i < C::kStages && i < mine; ++i) issue(i, (slot + i) % C::kStages);

    // ---- Q as the B operand: row 8 t + n, by k-step
    uint32_t qb[D / 16][NT][2];
    float mul[NT][2];      // rows 8 t + 2q, + 1: scores to log2 units
    uint64_t bits[NT][2];  // drafted keys that the row sees
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + n;
      const bool valid = r < sg.rows;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + (valid ? row_at(a, sg, r) : 0) * D;
      float m = a.scale_log2;
      if constexpr (E4M3) {
        // chunk 4j + q of 16 codes: word i feeds k-step 4j + i, codes 0, 1 as
        // k = 2q, 2q+1 and codes 2, 3 as k + 8
        uint32_t w[D / 64][8];
        uint32_t amax = 0;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint4 u = valid ? *reinterpret_cast<const uint4*>(qr + (4 * j + q) * 16 + 8 * e)
                                  : make_uint4(0, 0, 0, 0);
            w[j][4 * e] = u.x;
            w[j][4 * e + 1] = u.y;
            w[j][4 * e + 2] = u.z;
            w[j][4 * e + 3] = u.w;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            amax = max(amax, max((w[j][e] << 16) & 0x7fffffffu, w[j][e] & 0x7fff0000u));
        }
        amax = max(amax, __shfl_xor_sync(kFull, amax, 1));
        amax = max(amax, __shfl_xor_sync(kFull, amax, 2));
        const int shift = f16_shift(amax);
        const float f = pow2(shift);
        m *= pow2(-shift);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t v = w[j][2 * i + x];
              qb[4 * j + i][t][x] =
                  pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
            }
      } else {
        // chunk 4j + q of 8 values: words 2i, 2i+1 feed k-step 2j + i
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 u = valid ? *reinterpret_cast<const uint4*>(qr + (4 * j + q) * 8)
                                : make_uint4(0, 0, 0, 0);
          qb[2 * j][t][0] = u.x;
          qb[2 * j][t][1] = u.y;
          qb[2 * j + 1][t][0] = u.z;
          qb[2 * j + 1][t][1] = u.w;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        mul[t][c] = __shfl_sync(kFull, m, 4 * (2 * q + c));
        const int rr = 8 * t + 2 * q + c;
        bits[t][c] = rr < sg.rows ? bits_of(a, sg.s, (sg.row0 + rr) / (a.Hq / a.Hkv)) : 0;
      }
    }
    // O^T: rows of d by block pair and lane (see below), columns 8 t + 2q, + 1
    float o[D / 16][NT][4];
    float ref[NT][2], sum[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][t][i] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) ref[t][c] = neg_inf(), sum[t][c] = 0.f;
    }

    for (int i = 0; i < mine && ok; ++i) {
      const int s = slot;
      ok = __all_sync(kFull, mbar_poll(bars + 8 * s, phase, abort_flag, a.wait_limit_ns));
      if (!ok) {
        if (lane == 0) {
          *abort_flag = 1;
          atomicCAS(a.status, 0, ATTN_DEVICE_TIMEOUT_BASE + 30);
          // leave no copy in flight into this CTA's shared memory
          for (int x = i; x < mine && x < i + C::kStages; ++x) {
            mbar_drain(bars + 8 * slot, phase, a.wait_limit_ns);
            if (++slot == C::kStages) slot = 0, phase ^= 1;
          }
        }
        break;
      }
      if (++slot == C::kStages) slot = 0, phase ^= 1;
      const uint32_t sK = ring + s * C::kStageBytes, sV = sK + C::kTile;
      const bool bad_page = E4M3 && ((bad >> s) & 1);
      const uint32_t scales = ring_scale + s * 2 * C::kScaleBytes;

      // ---- S^T = K Q^T
      float sc[KB][NT][4];  // keys n (0, 1) and 8 + n (2, 3) of a block, rows 2q and 2q + 1
#pragma unroll
      for (int b = 0; b < KB; ++b) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[b][t][e] = 0.f;
        const uint32_t at = sK + 2 * b * kBlock + k_at;
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 u0 = lds128(j ? at ^ 64 : at), u1 = lds128(j ? (at + kBlock) ^ 64 : at + kBlock);
            const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(w0[e], a0, a2);
              e4m3x4_to_f16(w1[e], a1, a3);
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma_16816<true>(sc[b][t], a0, a1, a2, a3, qb[4 * j + e][t][0], qb[4 * j + e][t][1]);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint32_t x = at + (j >> 1) * kPanel;
            const uint4 u0 = lds128((j & 1) ? x ^ 64 : x), u1 = lds128((j & 1) ? (x + kBlock) ^ 64 : x + kBlock);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              mma_16816<false>(sc[b][t], u0.x, u1.x, u0.y, u1.y, qb[2 * j][t][0], qb[2 * j][t][1]);
              mma_16816<false>(sc[b][t], u0.z, u1.z, u0.w, u1.w, qb[2 * j + 1][t][0], qb[2 * j + 1][t][1]);
            }
          }
        }
      }
      // ---- the keys' scales, and the mask
      const int key0 = (sg.t0 + i * C::kEvery + first_page) * kPage + part * C::kKeys;
      if constexpr (E4M3) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float ks = bad_page ? 0.f : lds_f32(scales + 4 * (16 * b + 8 * h + key_n));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              sc[b][t][2 * h] *= ks;
              sc[b][t][2 * h + 1] *= ks;
            }
          }
      }
      const bool tail = key0 + C::kKeys > sg.s.prefix;
      if (tail) {
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int key = key0 + 16 * b + 8 * h + key_n;
            const int j = key - sg.s.prefix;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const bool sees = key < sg.s.prefix || (key < sg.s.len && ((bits[t][c] >> (j & 63)) & 1));
                if (!sees) sc[b][t][2 * h + c] = neg_inf();
              }
          }
      }
      // ---- running reference maximum (moved rarely)
      bool move = false;
      float mt[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float m = fmaxf(sc[0][t][c], sc[0][t][2 + c]);
          if constexpr (KB == 2) m = fmax3(m, sc[1][t][c], sc[1][t][2 + c]);
          mt[t][c] = m;
          move |= (m - ref[t][c]) * mul[t][c] > kRefSlack;  // NaN where nothing has been seen still
        }
      if (__any_sync(kFull, move)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = mt[t][c];
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, x));
            const float to = (m - ref[t][c]) * mul[t][c] > kRefSlack ? m : ref[t][c];
            const float al = to == ref[t][c] ? 1.f : ex2((ref[t][c] - to) * mul[t][c]);  // ref = -inf gives 0
            ref[t][c] = to;
            sum[t][c] *= al;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[j][t][c] *= al;
              o[j][t][2 + c] *= al;
            }
          }
        }
      }
      // ---- e4m3: V as fp16 where this warp's value scales allow (see over_f16)
      float vs[KB][4];  // scales of the keys of this lane's V rows: key_lo, + kStep, + 8 of each
      bool f16 = false;
      if constexpr (E4M3) {
        uint32_t over = 0;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            vs[b][e] = lds_f32(scales + C::kScaleBytes + 4 * (16 * b + 8 * (e >> 1) + key_lo + (e & 1) * LN::kStep));
            over = max(over, over_f16(vs[b][e]));
          }
        f16 = __all_sync(kFull, over <= kFitsF16 || bad_page);
        if (!f16 && tail) {  // what lies behind the last key does not decide
          over = 0;
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (key0 + 16 * b + 8 * (e >> 1) + key_lo + (e & 1) * LN::kStep >= sg.s.len) vs[b][e] = 1.f;
              over = max(over, over_f16(vs[b][e]));
            }
          f16 = __all_sync(kFull, over <= kFitsF16);
        }
        if (bad_page) {
#pragma unroll
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int e = 0; e < 4; ++e) vs[b][e] = 0.f;
        }
      }
      // ---- P^T as the B operand, of 2^((s - ref) scale): the difference first, which
      // keeps its bits at any size of the scores.  As bf16, the sums adding the rounded values
      // that the product meets; as fp16, whose rounding (2^-12) is below what
      // cancels there.
      uint32_t pb[KB][NT][2];  // rows 8 t + n; keys key_lo, + kStep (0) and 8 further (1)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float2 from = make_float2(minus(ref[t][0]), minus(ref[t][1])), by = make_float2(mul[t][0], mul[t][1]);
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float2 x = log2_p<E4M3>(make_float2(sc[b][t][2 * h], sc[b][t][2 * h + 1]), from, by);
            float p0 = ex2(x.x), p1 = ex2(x.y);
            uint32_t w;
            if (f16) {
              w = pack_f16x2(p0, p1);
              sum[t][0] += p0;
              sum[t][1] += p1;
            } else {
              if constexpr (E4M3) {
                // a value whose scale is NaN reaches every row that sees the key, at any p
                const float v = lds_f32(scales + C::kScaleBytes + 4 * (16 * b + 8 * h + key_n));
                if (v != v) {
                  if (sc[b][t][2 * h] != neg_inf()) p0 = v;
                  if (sc[b][t][2 * h + 1] != neg_inf()) p1 = v;
                }
              }
              w = pack_bf16x2(p0, p1);
              sum[t][0] += __uint_as_float(w << 16);
              sum[t][1] += __uint_as_float(w & 0xffff0000u);
            }
            pb[b][t][h] = transpose8(w);
          }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        const uint32_t at = sV + 2 * b * kBlock;
        // this lane's keys of the block
        auto v_key = [&](int e) { return 16 * b + 8 * (e >> 1) + key_lo + (e & 1) * LN::kStep; };
        if constexpr (E4M3) {
          uint32_t v[4][D / 32];  // codes of a key: 16 bytes, or 8 (D = 64)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (LN::kNarrow) {
              const uint2 u = lds64(at + (e >> 1) * kBlock + v_at[e & 1]);
              v[e][0] = u.x;
              v[e][1] = u.y;
            } else {
              const uint4 u = lds128(at + (e >> 1) * kBlock + v_at[e & 1]);
              v[e][0] = u.x;
              v[e][1] = u.y;
              v[e][2] = u.z;
              v[e][3] = u.w;
            }
          }
          if (f16) {
            if (tail) {  // slots past the end may hold the NaN code
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (key0 + v_key(e) >= sg.s.len) {
#pragma unroll
                  for (int x = 0; x < D / 32; ++x) v[e][x] = 0;
                }
            }
            const uint32_t s0 = pack_f16x2(vs[b][0], vs[b][1]), s1 = pack_f16x2(vs[b][2], vs[b][3]);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {  // codes 2j, 2j + 1 of two keys in one word
              const uint32_t sel = (j & 1) ? 0x7362u : 0x5140u;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16(__byte_perm(v[0][j >> 1], v[1][j >> 1], sel), a0, a1);
              e4m3x4_to_f16(__byte_perm(v[2][j >> 1], v[3][j >> 1], sel), a2, a3);
              a0 = mul_f16x2(a0, s0);
              a1 = mul_f16x2(a1, s0);
              a2 = mul_f16x2(a2, s1);
              a3 = mul_f16x2(a3, s1);
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma_16816<true>(o[j][t], a0, a1, a2, a3, pb[b][t][0], pb[b][t][1]);
            }
          } else {
            // The value scale goes to P, whose bf16 holds its exponent.  The
            // scale of a key that the row does not see may be NaN: 0 stays 0.
            uint32_t pv[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w = pb[b][t][x];
                const float p0 = __uint_as_float(w << 16), p1 = __uint_as_float(w & 0xffff0000u);
                pv[t][x] = pack_bf16x2(p0 == 0.f ? 0.f : p0 * vs[b][2 * x], p1 == 0.f ? 0.f : p1 * vs[b][2 * x + 1]);
              }
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              uint32_t f[2][2];  // [code 2j, 2j + 1][keys 0 1, 2 3]
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const int c = (2 * j + x) & 3;
                const uint32_t sel = c == 0 ? 0x4000u : c == 1 ? 0x5010u : c == 2 ? 0x6020u : 0x7030u;
                f[x][0] = e4m3_hi_to_bf16x2(__byte_perm(v[0][j >> 1], v[1][j >> 1], sel));
                f[x][1] = e4m3_hi_to_bf16x2(__byte_perm(v[2][j >> 1], v[3][j >> 1], sel));
              }
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma_16816<false>(o[j][t], f[0][0], f[1][0], f[0][1], f[1][1], pv[t][0], pv[t][1]);
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < D / 64; ++p) {  // a panel at a time: 16 registers of V
            uint32_t v[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 u = lds128(at + p * kPanel + (e >> 1) * kBlock + v_at[e & 1]);
              v[e][0] = u.x;
              v[e][1] = u.y;
              v[e][2] = u.z;
              v[e][3] = u.w;
            }
            if (tail) {
              // A key past the end contributes nothing, whatever its slot holds.
              // A drafted key with an element that is not finite must not reach
              // the rows that do not see it through 0 * inf: its value is taken
              // out of the product, and the rows that see it (their p is not 0,
              // or NaN already) become NaN.
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                bool nf = false;
#pragma unroll
                for (int x = 0; x < 4; ++x) nf |= has_nonfinite(v[e][x]);
                const int key = key0 + v_key(e);
                // the same key in all lanes of this q
                unsigned any = __ballot_sync(kFull, nf && key >= sg.s.prefix && key < sg.s.len);
                const bool drop = (any & (0x11111111u << q)) != 0;
                if (drop || key >= sg.s.len) {
#pragma unroll
                  for (int x = 0; x < 4; ++x) v[e][x] = 0;
                }
                if (drop) {
                  const int j = key - sg.s.prefix;
#pragma unroll
                  for (int t = 0; t < NT; ++t) {
                    const int rr = 8 * t + n;  // this lane's row of P^T
                    const bool sees = rr < sg.rows &&
                                      ((bits_of(a, sg.s, (sg.row0 + rr) / (a.Hq / a.Hkv)) >> (j & 63)) & 1);
                    if (sees)
                      pb[b][t][e >> 1] = (e & 1) ? (pb[b][t][e >> 1] & 0xffffu) | 0x7fc00000u
                                                 : (pb[b][t][e >> 1] & 0xffff0000u) | 0x7fc0u;
                  }
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // values 2j, 2j + 1 of two keys
              const uint32_t a0 = __byte_perm(v[0][j], v[1][j], 0x5410), a1 = __byte_perm(v[0][j], v[1][j], 0x7632);
              const uint32_t a2 = __byte_perm(v[2][j], v[3][j], 0x5410), a3 = __byte_perm(v[2][j], v[3][j], 0x7632);
#pragma unroll
              for (int t = 0; t < NT; ++t)
                mma_16816<false>(o[4 * p + j][t], a0, a1, a2, a3, pb[b][t][0], pb[b][t][1]);
            }
          }
        }
      }
      fence_proxy_async_smem();  // the reads of the slot stay before the copy that overwrites it
      __syncwarp();
      if (i + C::kStages < mine) issue(i + C::kStages, s);
    }

    // ---- add up the four warps' shares: warp 3 hands its sums to 2, 2 to 1, 1 to 0
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[t][c] += __shfl_xor_sync(kFull, sum[t][c], x);
        if (n == 0) {
          wmax[warp * kRows + 8 * t + 2 * q + c] = ref[t][c];
          wsum[warp * kRows + 8 * t + 2 * q + c] = sum[t][c];
        }
      }
    named_bar(1, kThreads);
    float M[NT][2], den[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * t + 2 * q + c;
        M[t][c] = neg_inf();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M[t][c] = fmaxf(M[t][c], wmax[w * kRows + r]);
        den[t][c] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float x = wmax[w * kRows + r];
          den[t][c] += (x == M[t][c] ? 1.f : ex2((x - M[t][c]) * mul[t][c])) * wsum[w * kRows + r];
        }
        const float f = ref[t][c] == M[t][c] ? 1.f : ex2((ref[t][c] - M[t][c]) * mul[t][c]);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          o[j][t][c] *= f;
          o[j][t][2 + c] *= f;
        }
      }
#pragma unroll 1
    for (int w = kWarps - 1; w > 0; --w) {
      if (warp == w) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float* at = red + ((j * NT + t) * 4 + e) * 32 + lane;
              *at = w == kWarps - 1 ? o[j][t][e] : *at + o[j][t][e];
            }
      }
      named_bar(1, kThreads);
    }
    if (warp == 0) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = 8 * t + 2 * q + c;
          if (r >= sg.rows) continue;
          const bool empty = den[t][c] == 0.f;  // a row that sees nothing here
          const float none = without_sum(sg.s, bits[t][c]), inv = empty ? 0.f : 1.f / den[t][c];
          const size_t share = share_at(a, kRows, blockIdx.y, blockIdx.x, sg.place, r);
          const size_t at = row_at(a, sg, r);
          if (!sg.whole && n == 0)
            a.sums[share] = make_float2(M[t][c] * mul[t][c], den[t][c] * (E4M3 ? pow2(-kPShift) : 1.f));
          // this lane's columns, in runs of 8: block pair j holds columns
          // 2j and 2j + 1 of the lane's chunk of 16 codes, or of 8 values a panel
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            const int d0 = !E4M3 ? 64 * x + 8 * key_n : LN::kNarrow ? 8 * n : 16 * key_n + 8 * x;
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int j = 4 * x + (e >> 1), k = 2 * (e & 1) + c;
              f[e] = empty ? none : (o[j][t][k] + red[((j * NT + t) * 4 + k) * 32 + lane]) * inv;
            }
            if (sg.whole) {
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o) + at * D + d0) =
                  make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                             pack_bf16x2(f[6], f[7]));
            } else {
              float4* p = reinterpret_cast<float4*>(a.part + share * D + d0);
              p[0] = make_float4(f[0], f[1], f[2], f[3]);
              p[1] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
    }
  }
}

template <int D, bool E4M3, int NT>
int launch_t(const TreeLaunch& a, Cfg<D, E4M3, NT>) {
  using C = Cfg<D, E4M3, NT>;
  auto kern = tree_few_kernel<D, E4M3, NT>;
  static uint64_t attr_done = 0;  // one bit per device ordinal
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return ATTN_ERR_CUDA;
  if (!(attr_done >> dev & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done |= uint64_t(1) << dev;
  }
  CUtensorMap mk, mv;
  const int groups = a.num_pages * a.Hkv;
  if (E4M3 ? !tma_map_codes(&mk, a.K, groups, D, C::kKeys) || !tma_map_codes(&mv, a.V, groups, D, C::kKeys)
           : !tma_map_bhnd(&mk, a.K, groups, kPage, D, C::kKeys) || !tma_map_bhnd(&mv, a.V, groups, kPage, D, C::kKeys))
    return ATTN_ERR_CUDA;
  kern<<<dim3(a.ctas, a.planes), kThreads, C::kSmem, a.stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// f of the configuration for d, the cache and the rows of a CTA
template <class F>
int with_cfg(int d, bool e4m3, int rows, F f) {
  if (!e4m3 && rows == 8) return d == 64 ? f(Cfg<64, false, 1>{}) : f(Cfg<128, false, 1>{});
  if (e4m3 && rows == 8) return d == 64 ? f(Cfg<64, true, 1>{}) : f(Cfg<128, true, 1>{});
  if (e4m3 && rows == 16) return d == 64 ? f(Cfg<64, true, 2>{}) : f(Cfg<128, true, 2>{});
  return ATTN_ERR_INVALID_ARG;
}

}  // namespace

int tree_few_ctas(int d, bool e4m3, int rows) {
  return with_cfg(d, e4m3, rows, [](auto c) { return decltype(c)::kCtas; });
}

int launch_tree_few(const TreeLaunch& a, int rows) {
  return with_cfg(a.d, a.k_scales != nullptr, rows, [&](auto c) { return launch_t(a, c); });
}

}  // namespace bss
