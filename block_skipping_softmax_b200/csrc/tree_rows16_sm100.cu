// Tree attention for few rows a KV head (decode of single tokens): 16 rows a
// CTA on warp-level MMAs (m16n8k16).
//
// Such a call is bound by the bytes of K and V: with R rows a key's 2 d bytes
// of e4m3 (4 d of bf16) meet 4 R d flops.  A CTA is one warp that issues the
// copies, a ring of tiles, and four warps that take 16 of a tile's 64 keys each
// for all 16 rows, with their own running maximum and sums, so that nothing is
// exchanged between warps until the end of a segment.  Two CTAs share an SM.
//
// Fragments are read straight from the swizzled tiles, 16 bytes of a key row
// at a time: the order of d inside a k-step of Q K^T, of keys inside one of
// P V, and of the columns of O is free, and is chosen so that no fragment is
// transposed in shared memory and no read of 128-byte rows meets a bank twice.
// e4m3 codes become fp16 (K, against fp16 queries) or bf16 (V, against bf16
// probabilities, whose exponents hold the value scales) in registers, so they
// cross shared memory once, as bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace bss {

namespace {

constexpr int kWarps = 4;  // consumers; one more warp issues the copies
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRows = kFewRows;

template <int D, bool E4M3>
struct Cfg {
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kTile = kPage * kRowBytes;
  static constexpr int kPanels = E4M3 ? 1 : D / 64;  // swizzled panels of a tile
  static constexpr int kScaleBytes = E4M3 ? kPage * 4 : 0;
  static constexpr int kStages = kRowBytes == 256 ? 3 : kRowBytes == 128 ? 5 : 6;
  static constexpr int kStageBytes = 2 * kTile;
  static constexpr int kOffScale = kStages * kStageBytes;  // [stage][K, V][64] floats
  static constexpr int kOffRed = kOffScale + kStages * 2 * kScaleBytes;  // 16 x D floats
  static constexpr int kOffMax = kOffRed + kRows * D * 4;                // [warp][row] maxima, then sums
  static constexpr int kOffBar = kOffMax + 2 * kWarps * kRows * 4;
  static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;  // abort, bad page [stage]
  static constexpr int kSmem = kOffMisc + 4 + 4 * kStages + 1024;
};

// one key row's swizzled 16-byte chunk
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  if constexpr (E4M3 && D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
  return (c >> 3) * (kPage * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&x)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(b0), "r"(b1));
}

// Lane = (n, q) = (lane / 4, lane % 4).  Of the 8 keys of a score block, B
// column n is key key_of(n), and this lane's two score columns are keys
// key_of(2q) and key_of(2q + 1).  With 128-byte rows the order 0 4 1 5 2 6 3 7
// keeps the eight lanes of a 16-byte read on eight different banks; 64-byte
// rows (two a bank line) do so in their own order.
template <int D, bool E4M3>
struct Lanes {
  static constexpr bool kNarrow = E4M3 && D == 64;
  static constexpr int kStep = kNarrow ? 1 : 4;  // key_of(2q + 1) - key_of(2q)
  __device__ __forceinline__ static int key_of(int n) { return kNarrow ? n : ((n & 1) << 2) | (n >> 1); }
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 2)
    tree_rows16_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeLaunch a) {
  using C = Cfg<D, E4M3>;
  using LN = Lanes<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;  // the swizzle pattern repeats every 1024 B
  uint8_t* smem = smem_raw + (sbase - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  volatile int* bad_page = abort_flag + 1;  // [stage]: the page id was out of range
  auto b_full = [&](int s) { return sbase + C::kOffBar + 8u * s; };
  auto b_empty = [&](int s) { return sbase + C::kOffBar + 8u * (C::kStages + s); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), kWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  Segments list;
  list.start(a, kRows);
  Segment sg{};
  __syncthreads();

  if (warp == kWarps) {
    // -------------------------------------------------------------- copies
    int issued = 0;  // tiles so far, over all segments
    bool ok = true;
    while (ok && list.next(a, kRows, sg)) {
      const int* table = a.block_table + static_cast<size_t>(sg.b) * a.max_pages + sg.t0;
      int pages = 0;  // lane i: the page of tile i + 32 n
      for (int i = 0; i < sg.nt && ok; ++i) {
        if ((i & 31) == 0) pages = i + lane < sg.nt ? table[i + lane] : -1;
        const int page = __shfl_sync(kFull, pages, i & 31);
        const int s = issued % C::kStages;
        if (lane == 0) {
          if (issued >= C::kStages)
            ok = mbar_wait(b_empty(s), ((issued / C::kStages) - 1) & 1, abort_flag, a.wait_limit_ns);
          if (ok) {
            const bool good = page >= 0 && page < a.num_pages;
            // an id out of range reads zeros: its box lies past the pool's end
            const long long grp = static_cast<long long>(good ? page : a.num_pages) * a.Hkv + sg.kv;
            bad_page[s] = good ? 0 : 1;
            mbar_arrive_expect_tx(b_full(s), C::kStageBytes + (good ? 2 * C::kScaleBytes : 0));
#pragma unroll
            for (int p = 0; p < C::kPanels; ++p) {
              const uint32_t dst = sbase + s * C::kStageBytes + p * (kPage * 128);
              tma_load_3d(dst, &tmK, b_full(s), p * 64, 0, static_cast<int>(grp));
              tma_load_3d(dst + C::kTile, &tmV, b_full(s), p * 64, 0, static_cast<int>(grp));
            }
            if constexpr (E4M3) {
              if (good) {
                const uint32_t dst = sbase + C::kOffScale + s * 2 * C::kScaleBytes;
                bulk_load(dst, a.k_scales + grp * kPage, C::kScaleBytes, b_full(s));
                bulk_load(dst + C::kScaleBytes, a.v_scales + grp * kPage, C::kScaleBytes, b_full(s));
              }
            }
          }
        }
        ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
        if (ok) ++issued;
      }
    }
    if (lane == 0) {
      if (!ok) {
        *abort_flag = 1;
        atomicCAS(a.status, 0, ATTN_DEVICE_TIMEOUT_BASE + 30);
      }
      // never leave while a copy into this CTA's shared memory is in flight
      for (int i = max(0, issued - C::kStages); i < issued; ++i)
        mbar_drain(b_full(i % C::kStages), (i / C::kStages) & 1, a.wait_limit_ns);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  const int n = lane >> 2, q = lane & 3;
  const int key_n = LN::key_of(n);      // K row of B column n; V chunk of B column n
  const int key_lo = LN::key_of(2 * q);  // this lane's keys: + 8 nb + kStep c
  const int kk0 = warp * 16 + key_lo;
  float* red = reinterpret_cast<float*>(smem + C::kOffRed);   // [fragment register][lane]
  float* wmax = reinterpret_cast<float*>(smem + C::kOffMax);  // [warp][row]
  float* wsum = wmax + kWarps * kRows;
  int done = 0;     // tiles so far
  bool ok = true;   // after a wait gave up the warp only keeps up with the barriers

  while (list.next(a, kRows, sg)) {
    // ---- Q fragments of rows n and n + 8
    uint32_t qa[D / 16][4];
    uint64_t bits[2];  // drafted keys that the row sees
    float mul[2];      // scores to log2 units
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = n + 8 * hf;
      const bool valid = r < sg.rows;
      int tok = 0;
      const size_t at = valid ? row_at(a, sg, r, &tok) : 0;
      bits[hf] = valid ? bits_of(a, sg.s, tok) : 0;
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + at * D;
      mul[hf] = a.scale_log2;
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
        mul[hf] *= pow2(-shift);
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t v = w[j][2 * i + x];
              qa[4 * j + i][2 * x + hf] =
                  pack_f16x2(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
            }
      } else {
        // chunk 4j + q of 8 values: words 2i, 2i+1 feed k-step 2j + i
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 u = valid ? *reinterpret_cast<const uint4*>(qr + (4 * j + q) * 8)
                                : make_uint4(0, 0, 0, 0);
          qa[2 * j][hf] = u.x;
          qa[2 * j][2 + hf] = u.y;
          qa[2 * j + 1][hf] = u.z;
          qa[2 * j + 1][2 + hf] = u.w;
        }
      }
    }
    float o[D / 8][4];  // column block j of O: rows n (0, 1) and n + 8 (2, 3)
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
    float ref[2] = {neg_inf(), neg_inf()}, sum[2] = {0.f, 0.f};

    for (int i = 0; i < sg.nt; ++i, ++done) {
      const int s = done % C::kStages;
      if (!ok) continue;
      ok = __all_sync(kFull, mbar_wait(b_full(s), (done / C::kStages) & 1, abort_flag, a.wait_limit_ns));
      if (!ok) {
        if (lane == 0) {
          *abort_flag = 1;
          atomicCAS(a.status, 0, ATTN_DEVICE_TIMEOUT_BASE + 31);
        }
        continue;
      }
      const uint32_t sK = sbase + s * C::kStageBytes, sV = sK + C::kTile;
      // ---- S = Q K^T for 16 keys
      float sc[2][4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nb][e] = 0.f;
        const int row = warp * 16 + nb * 8 + key_n;
        if constexpr (E4M3) {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 u = lds128(sK + chunk_at<D, E4M3>(row, 4 * j + q));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t b0, b1;
              e4m3x4_to_f16(w[e], b0, b1);
              mma_16816<true>(sc[nb], qa[4 * j + e], b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 u = lds128(sK + chunk_at<D, E4M3>(row, 4 * j + q));
            mma_16816<false>(sc[nb], qa[2 * j], u.x, u.y);
            mma_16816<false>(sc[nb], qa[2 * j + 1], u.z, u.w);
          }
        }
      }
      // ---- to log2 units, and the mask
      const int key0 = (sg.t0 + i) * kPage;
      float vs[2][2];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          vs[nb][c] = 1.f;
          if constexpr (E4M3) {
            const uint32_t at = sbase + C::kOffScale + s * 2 * C::kScaleBytes + 4 * (kk0 + nb * 8 + c * LN::kStep);
            const bool good = bad_page[s] == 0;
            const float ks = good ? lds_f32(at) : 0.f;
            vs[nb][c] = good ? lds_f32(at + C::kScaleBytes) : 0.f;
            sc[nb][c] *= ks;
            sc[nb][2 + c] *= ks;
          }
          sc[nb][c] *= mul[0];
          sc[nb][2 + c] *= mul[1];
        }
      }
      const bool tail = key0 + kPage > sg.s.prefix;
      if (tail) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int key = key0 + kk0 + nb * 8 + c * LN::kStep;
            const int j = key - sg.s.prefix;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const bool sees = key < sg.s.prefix || (key < sg.s.len && ((bits[hf] >> (j & 63)) & 1));
              if (!sees) sc[nb][2 * hf + c] = neg_inf();
            }
          }
      }
      // ---- running reference maximum (moved rarely) and probabilities
      float mt[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
        mt[hf] = fmaxf(fmaxf(sc[0][2 * hf], sc[0][2 * hf + 1]), fmaxf(sc[1][2 * hf], sc[1][2 * hf + 1]));
      if (__any_sync(kFull, mt[0] > ref[0] + kRefSlack || mt[1] > ref[1] + kRefSlack)) {
        float al[2];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float m = fmaxf(mt[hf], __shfl_xor_sync(kFull, mt[hf], 1));
          m = fmaxf(m, __shfl_xor_sync(kFull, m, 2));
          const float to = m > ref[hf] + kRefSlack ? m : ref[hf];
          al[hf] = to == ref[hf] ? 1.f : ex2(ref[hf] - to);  // ref = -inf gives 0
          ref[hf] = to;
          sum[hf] *= al[hf];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= al[0];
          o[j][1] *= al[0];
          o[j][2] *= al[1];
          o[j][3] *= al[1];
        }
      }
      // P as bf16; the sums add the rounded values that P V multiplies, before
      // the (exact, power-of-two) value scale
      float pv[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float base = ref[hf] == neg_inf() ? 0.f : ref[hf];  // nothing seen so far: all p are 0
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = sc[nb][2 * hf + c];
            const float p = __bfloat162float(__float2bfloat16_rn(ex2(x - base)));
            sum[hf] += p;
            pv[nb][2 * hf + c] = x == neg_inf() ? 0.f : p * vs[nb][c];  // an unseen key's scale may be NaN
          }
      }
      // ---- V rows of this lane's four keys: two pairs of neighbours in a k-step
      auto v_row = [&](int e) { return kk0 + (e >> 1) * 8 + (e & 1) * LN::kStep; };
      uint32_t pa[4];
      auto pack_p = [&] {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          pa[2 * x] = pack_bf16x2(pv[x][0], pv[x][1]);
          pa[2 * x + 1] = pack_bf16x2(pv[x][2], pv[x][3]);
        }
      };
      if constexpr (E4M3) {
        uint32_t v[4][D / 32];  // codes of a key: 16 bytes, or 8 (D = 64)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (LN::kNarrow) {
            const uint2 u = lds64(sV + chunk_at<D, E4M3>(v_row(e), key_n >> 1) + (key_n & 1) * 8);
            v[e][0] = u.x;
            v[e][1] = u.y;
          } else {
            const uint4 u = lds128(sV + chunk_at<D, E4M3>(v_row(e), key_n));
            v[e][0] = u.x;
            v[e][1] = u.y;
            v[e][2] = u.z;
            v[e][3] = u.w;
          }
        }
        pack_p();
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t sel = (j & 3) == 0 ? 0x4000u : (j & 3) == 1 ? 0x5010u : (j & 3) == 2 ? 0x6020u : 0x7030u;
          mma_16816<false>(o[j], pa, e4m3_hi_to_bf16x2(__byte_perm(v[0][j >> 2], v[1][j >> 2], sel)),
                           e4m3_hi_to_bf16x2(__byte_perm(v[2][j >> 2], v[3][j >> 2], sel)));
        }
      } else {
        uint32_t v[4][D / 16];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int p = 0; p < D / 64; ++p) {
            const uint4 u = lds128(sV + chunk_at<D, E4M3>(v_row(e), 8 * p + key_n));
            v[e][4 * p] = u.x;
            v[e][4 * p + 1] = u.y;
            v[e][4 * p + 2] = u.z;
            v[e][4 * p + 3] = u.w;
          }
        if (tail) {
          // A key past the end contributes nothing, whatever its slot holds.  A
          // drafted key with an element that is not finite must not reach the
          // rows that do not see it through 0 * inf: its value is taken out of
          // the product, and the rows that see it become NaN.
          unsigned nonfinite = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            bool bad = false;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) bad |= has_nonfinite(v[e][x]);
            if (bad && key0 + v_row(e) >= sg.s.prefix) nonfinite |= 1u << e;
          }
          nonfinite |= __shfl_xor_sync(kFull, nonfinite, 4);
          nonfinite |= __shfl_xor_sync(kFull, nonfinite, 8);
          nonfinite |= __shfl_xor_sync(kFull, nonfinite, 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (key0 + v_row(e) >= sg.s.len || ((nonfinite >> e) & 1)) {
#pragma unroll
              for (int x = 0; x < D / 16; ++x) v[e][x] = 0;
            }
            if ((nonfinite >> e) & 1) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (sc[e >> 1][2 * hf + (e & 1)] != neg_inf())
                  pv[e >> 1][2 * hf + (e & 1)] = __int_as_float(0x7fc00000);
            }
          }
        }
        pack_p();
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          mma_16816<false>(o[j], pa, __byte_perm(v[0][j >> 1], v[1][j >> 1], sel),
                           __byte_perm(v[2][j >> 1], v[3][j >> 1], sel));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty(s));
    }

    // ---- add up the four warps' shares: warp 3 hands its sums to 2, 2 to 1, 1 to 0
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      sum[hf] += __shfl_xor_sync(kFull, sum[hf], 1);
      sum[hf] += __shfl_xor_sync(kFull, sum[hf], 2);
      if (q == 0) {
        wmax[warp * kRows + n + 8 * hf] = ref[hf];
        wsum[warp * kRows + n + 8 * hf] = sum[hf];
      }
    }
    named_bar(1, kWarps * 32);
    float M[2], den[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      M[hf] = neg_inf();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M[hf] = fmaxf(M[hf], wmax[w * kRows + n + 8 * hf]);
      den[hf] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float x = wmax[w * kRows + n + 8 * hf];
        den[hf] += (x == M[hf] ? 1.f : ex2(x - M[hf])) * wsum[w * kRows + n + 8 * hf];
      }
      const float f = ref[hf] == M[hf] ? 1.f : ex2(ref[hf] - M[hf]);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][2 * hf] *= f;
        o[j][2 * hf + 1] *= f;
      }
    }
#pragma unroll 1
    for (int w = kWarps - 1; w > 0; --w) {
      if (warp == w) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* at = red + (4 * j + e) * 32 + lane;
            *at = w == kWarps - 1 ? o[j][e] : *at + o[j][e];
          }
      }
      named_bar(1, kWarps * 32);
    }
    if (warp == 0) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = n + 8 * hf;
        if (r >= sg.rows) continue;
        const float inv = den[hf] == 0.f ? 0.f : 1.f / den[hf];  // 0: a row that sees nothing here
        const size_t share = share_at(a, kRows, blockIdx.y, blockIdx.x, sg.place, r);
        const size_t at = row_at(a, sg, r);
        if (!sg.whole && q == 0) a.lse[share] = den[hf] == 0.f ? neg_inf() : M[hf] + __log2f(den[hf]);
        // runs of 8 neighbouring columns
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          const int c = x & 1, h = x >> 1;
          const int j0 = 8 * h;
          const int d0 = LN::kNarrow ? 16 * q + 8 * c
                         : E4M3      ? 64 * c + 16 * q + 8 * h
                                     : 64 * h + 32 * c + 8 * q;
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = 4 * (j0 + e) + 2 * hf + c;
            f[e] = den[hf] == 0.f ? 0.f : (o[j0 + e][2 * hf + c] + red[k * 32 + lane]) * inv;
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

template <int D, bool E4M3>
int launch_t(const TreeLaunch& a) {
  using C = Cfg<D, E4M3>;
  auto kern = tree_rows16_kernel<D, E4M3>;
  static uint64_t attr_done = 0;  // one bit per device ordinal
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return ATTN_ERR_CUDA;
  if (!(attr_done >> dev & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done |= uint64_t(1) << dev;
  }
  CUtensorMap mk, mv;
  if constexpr (E4M3) {
    const long long groups = static_cast<long long>(a.num_pages) * a.Hkv;
    if (!tma_map_codes(&mk, a.K, groups, D) || !tma_map_codes(&mv, a.V, groups, D)) return ATTN_ERR_CUDA;
  } else {
    const int groups = a.num_pages * a.Hkv;
    if (!tma_map_bhnd(&mk, a.K, groups, kPage, D, kPage) || !tma_map_bhnd(&mv, a.V, groups, kPage, D, kPage))
      return ATTN_ERR_CUDA;
  }
  kern<<<dim3(a.ctas, a.planes), kThreads, C::kSmem, a.stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int launch_tree_rows16(const TreeLaunch& a) {
  if (a.d == 64) return a.k_scales ? launch_t<64, true>(a) : launch_t<64, false>(a);
  return a.k_scales ? launch_t<128, true>(a) : launch_t<128, false>(a);
}

}  // namespace bss
