// Attention of drafted tokens over a paged KV cache, bf16 or e4m3.
//
// Sequence b brings T_b <= 64 drafted tokens, whose keys are already the last
// T_b of its len_b cached ones.  Token i sees the whole prefix and drafted key
// j iff bit j of its mask is set (its ancestors in the tree and itself), so
//   o_i = sum_k p_ik v_k / sum_k p_ik,  p_ik = exp(q_i k_k / sqrt(d) - m_i)
// over the keys that it sees; a token that sees none gets 0.  T_b = 1 is the
// decode of single tokens.  With e4m3 codes key k is K8_k * ks_k: ks_k scales
// a column of scores, and vs_k the column of probabilities before P V.
//
// The rows that share a KV head are the T_b * g pairs of a token and a query
// head of the group (row r: token r / g, head r % g).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace bss {

namespace {

constexpr int kPage = kDecodeTile;  // 64 keys: one page, one tile
constexpr unsigned kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Kernel for few rows: 16 rows a CTA on warp-level MMAs (m16n8k16).
//
// Decode is bound by the bytes of K and V.  A warp takes 16 of a tile's 64
// keys for all 16 rows, with its own running maximum and sums, so nothing is
// exchanged between warps until the end of the split.  The fragments are read
// straight from the swizzled tiles, 16 bytes of a key row at a time: the order
// of d inside a k-step of Q K^T, of keys inside one of P V, and of the columns
// of O is free, and is chosen so that no fragment needs a transpose in shared
// memory and no read has a bank conflict.  e4m3 codes become bf16 in
// registers (exact), so they cross shared memory once, as bytes.
constexpr int kWarps = 4;  // consumers; one more warp issues the copies
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRows = 16;
constexpr float kRefSlack = 8.f;  // log2 units: probabilities stay below 2^8

template <int D, bool E4M3>
struct Cfg {
  static constexpr int kRowBytes = E4M3 ? D : 2 * D;
  static constexpr int kTile = kPage * kRowBytes;
  static constexpr int kPanels = E4M3 ? 1 : D / 64;      // swizzled panels of a tile
  static constexpr int kScaleBytes = E4M3 ? kPage * 4 : 0;
  static constexpr int kStages = kRowBytes == 256 ? 3 : kRowBytes == 128 ? 5 : 6;
  static constexpr int kStageBytes = 2 * kTile;
  static constexpr int kOffScale = kStages * kStageBytes;  // [stage][K, V][64] floats
  static constexpr int kOffBar = kOffScale + kStages * 2 * kScaleBytes;
  static constexpr int kOffMisc = kOffBar + 2 * kStages * 8;  // abort, bad page [stage]
  static constexpr int kSmem = kOffMisc + 4 + 4 * kStages + 1024;
  static_assert(kWarps * kRows * (D + 2) * 4 <= kOffScale, "the merge reuses the ring");
};

// one key row's swizzled 16-byte chunk
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  if constexpr (E4M3 && D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
  return (c >> 3) * (kPage * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}

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

// Two e4m3 codes in the upper bytes of the halfwords of w (the lower bytes may
// hold anything) to two bf16: sign, exponent and mantissa move to their bf16
// places, and 2^120 moves the exponent's bias from 7 to 127, subnormal codes
// included.  Exact.  The NaN code (0x7f) comes out as 480: the writer never
// stores it under a finite scale, and a NaN scale makes the value NaN.
__device__ __forceinline__ uint32_t e4m3_hi_to_bf16x2(uint32_t w) {
  uint32_t x = (w & 0x80008000u) | ((w >> 4) & 0x07f007f0u);
  asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0x7b807b80u));
  return x;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ bool has_nonfinite(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u) || ((w & 0x7f800000u) == 0x7f800000u);
}

// What a CTA needs to know of its sequence.
struct Seq {
  int tok0, T;      // first token of the packed batch, tokens
  int len, prefix;  // keys; keys that every token sees
};

__device__ __forceinline__ Seq seq_of(const int* cu_q, const int* seq_lens, int b, int max_q,
                                      int total_q, int L, int max_pages) {
  Seq s;
  s.tok0 = min(max(cu_q[b], 0), total_q);
  s.T = min(min(max(cu_q[b + 1], s.tok0), total_q) - s.tok0, max_q);
  s.len = max(0, min(min(seq_lens[b], L), max_pages * kPage));
  s.prefix = max(0, s.len - s.T);
  return s;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kThreads, 2)
    tree_rows16_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const TreeLaunch a) {
  using C = Cfg<D, E4M3>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;  // the swizzle pattern repeats every 1024 B
  uint8_t* smem = smem_raw + (sbase - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  volatile int* bad_page = abort_flag + 1;  // [stage]: the page id was out of range
  auto b_full = [&](int s) { return sbase + C::kOffBar + 8u * s; };
  auto b_empty = [&](int s) { return sbase + C::kOffBar + 8u * (C::kStages + s); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x;
  const int kv = blockIdx.y % a.Hkv, rb = blockIdx.y / a.Hkv;
  const int b = blockIdx.z;
  const int g = a.Hq / a.Hkv;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const Seq sq = seq_of(a.cu_q, a.seq_lens, b, a.max_q, a.total_q, a.L, a.max_pages);
  const int rows = min(kRows, sq.T * g - rb * kRows);  // of this CTA
  if (rows <= 0) return;
  const int t_begin = split * (a.split_len / kPage);
  const int t_end = min((sq.len + kPage - 1) / kPage, t_begin + a.split_len / kPage);
  const int nt = t_end - t_begin;

  // row r of this CTA: token (row0 + r) / g of the sequence, query head kv*g + (row0 + r) % g
  const int row0 = rb * kRows;
  auto out_row = [&](int r) {  // index into [total_q * Hq]
    const int t = (row0 + r) / g;
    return static_cast<size_t>(sq.tok0 + t) * a.Hq + kv * g + (row0 + r) - t * g;
  };
  if (nt <= 0) {  // the split lies past the end of the sequence: no weight in the merge
    if (a.n_splits > 1) {
      for (int r = threadIdx.x; r < rows; r += kThreads)
        a.lse_part[out_row(r) * a.n_splits + split] = NEG_INF;
    } else {
      for (int i = threadIdx.x; i < rows * D; i += kThreads)
        static_cast<__nv_bfloat16*>(a.o)[out_row(i / D) * D + i % D] = __float2bfloat16_rn(0.f);
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), kWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();

  float o[D / 8][4];  // column block j of O: rows lane/4 and lane/4 + 8, columns by col_of
#pragma unroll
  for (int j = 0; j < D / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
  float ref[2] = {NEG_INF, NEG_INF}, sum[2] = {0.f, 0.f};

  if (warp == kWarps) {
    // -------------------------------------------------------------- producer
    const int* table = a.block_table + static_cast<size_t>(b) * a.max_pages + t_begin;
    int pages = 0;  // lane i: the page of tile (i + 32 n)
    int issued = 0;
    bool ok = true;
    for (int i = 0; i < nt && ok; ++i) {
      if ((i & 31) == 0) pages = i + lane < nt ? table[i + lane] : -1;
      const int page = __shfl_sync(kFull, pages, i & 31);
      const int s = i % C::kStages;
      if (lane == 0) {
        if (i >= C::kStages)
          ok = mbar_wait(b_empty(s), ((i / C::kStages) - 1) & 1, abort_flag, a.wait_limit_ns);
        if (ok) {
          const bool good = page >= 0 && page < a.num_pages;
          // an id out of range reads zeros: its box lies past the pool's end
          const long long grp = static_cast<long long>(good ? page : a.num_pages) * a.Hkv + kv;
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
          ++issued;
        }
      }
      ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
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
  } else {
    // -------------------------------------------------------------- consumers
    const int n = lane >> 2, q = lane & 3;
    // keys of this lane's score columns inside an 8-key block: column 2q is key
    // key_lo, column 2q+1 key key_lo + key_step; the K row of B-column n is key_n
    constexpr bool kNarrow = E4M3 && D == 64;  // 64-byte rows: two share a bank line
    const int key_n = kNarrow ? n : ((n & 1) << 2) | (n >> 1);
    const int key_lo = kNarrow ? 2 * q : q;
    constexpr int key_step = kNarrow ? 1 : 4;
    const int ch_v = kNarrow ? n : ((n & 1) << 2) | (n >> 1);  // V chunk of B-column n

    // Q fragments of rows n and n + 8
    uint32_t qa[D / 16][4];
    uint64_t bits[2];  // drafted keys that the row sees
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int r = n + 8 * hf;
      const bool valid = r < rows;
      const int t = valid ? (row0 + r) / g : 0;
      bits[hf] = 0;
      if (valid)
        bits[hf] = a.mask ? a.mask[sq.tok0 + t] : (t >= 63 ? ~0ull : (2ull << t) - 1);
      const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + (valid ? out_row(r) : 0) * D;
      if constexpr (E4M3) {
        // chunk 4j + q of 16 codes: word i feeds k-step 4j + i, codes 0, 2 as
        // k = 2q, 2q+1 and codes 1, 3 as k + 8
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint4 u[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            u[e] = valid ? *reinterpret_cast<const uint4*>(qr + (4 * j + q) * 16 + 8 * e)
                         : make_uint4(0, 0, 0, 0);
          const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            qa[4 * j + i][hf] = __byte_perm(w[2 * i], w[2 * i + 1], 0x5410);
            qa[4 * j + i][2 + hf] = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
          }
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

    bool ok = true;
    for (int i = 0; i < nt; ++i) {
      const int s = i % C::kStages;
      if (!__all_sync(kFull, mbar_wait(b_full(s), (i / C::kStages) & 1, abort_flag, a.wait_limit_ns))) {
        ok = false;
        break;
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
            for (int e = 0; e < 4; ++e)
              mma_16816(sc[nb], qa[4 * j + e][0], qa[4 * j + e][1], qa[4 * j + e][2],
                        qa[4 * j + e][3], e4m3_hi_to_bf16x2(w[e] << 8), e4m3_hi_to_bf16x2(w[e]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 u = lds128(sK + chunk_at<D, E4M3>(row, 4 * j + q));
            mma_16816(sc[nb], qa[2 * j][0], qa[2 * j][1], qa[2 * j][2], qa[2 * j][3], u.x, u.y);
            mma_16816(sc[nb], qa[2 * j + 1][0], qa[2 * j + 1][1], qa[2 * j + 1][2],
                      qa[2 * j + 1][3], u.z, u.w);
          }
        }
      }
      // ---- scale and mask; this lane's keys are kk(nb, c)
      const int key0 = (t_begin + i) * kPage;
      const int kk0 = warp * 16 + key_lo;  // + nb * 8 + c * key_step
      float vs[2][2];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float ks = a.scale_log2;
          vs[nb][c] = 1.f;
          if constexpr (E4M3) {
            const uint32_t at = sbase + C::kOffScale + s * 2 * C::kScaleBytes + 4 * (kk0 + nb * 8 + c * key_step);
            const bool good = bad_page[s] == 0;
            ks = good ? lds_f32(at) * a.scale_log2 : 0.f;
            vs[nb][c] = good ? lds_f32(at + C::kScaleBytes) : 0.f;
          }
          sc[nb][c] *= ks;
          sc[nb][2 + c] *= ks;
        }
      }
      const bool tail = key0 + kPage > sq.prefix;
      if (tail) {
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int key = key0 + kk0 + nb * 8 + c * key_step;
            const int j = key - sq.prefix;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const bool sees = key < sq.prefix || (key < sq.len && ((bits[hf] >> (j & 63)) & 1));
              if (!sees) sc[nb][2 * hf + c] = NEG_INF;
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
      uint32_t pa[4];
      float pv[2][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float base = ref[hf] == NEG_INF ? 0.f : ref[hf];  // nothing seen so far: all p are 0
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float x = sc[nb][2 * hf + c];
            const float p = __bfloat162float(__float2bfloat16_rn(ex2(x - base)));
            sum[hf] += p;
            pv[nb][2 * hf + c] = x == NEG_INF ? 0.f : p * vs[nb][c];  // an unseen key's scale may be NaN
          }
      }
      // ---- V rows of this lane's four keys: two pairs of neighbours in a k-step
      if constexpr (E4M3) {
        constexpr int kWords = D / 32;  // words of codes a key: 16 bytes, or 8 (D = 64)
        uint32_t v[4][kWords];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = kk0 + (e >> 1) * 8 + (e & 1) * key_step;
          if constexpr (kNarrow) {
            const uint2 u = lds64(sV + chunk_at<D, E4M3>(row, ch_v >> 1) + (ch_v & 1) * 8);
            v[e][0] = u.x;
            v[e][1] = u.y;
          } else {
            const uint4 u = lds128(sV + chunk_at<D, E4M3>(row, ch_v));
            v[e][0] = u.x;
            v[e][1] = u.y;
            v[e][2] = u.z;
            v[e][3] = u.w;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          pa[2 * x] = pack_bf16x2(pv[x][0], pv[x][1]);
          pa[2 * x + 1] = pack_bf16x2(pv[x][2], pv[x][3]);
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t sel = (j & 3) == 0 ? 0x4000u : (j & 3) == 1 ? 0x5010u : (j & 3) == 2 ? 0x6020u : 0x7030u;
          const uint32_t b0 = e4m3_hi_to_bf16x2(__byte_perm(v[0][j >> 2], v[1][j >> 2], sel));
          const uint32_t b1 = e4m3_hi_to_bf16x2(__byte_perm(v[2][j >> 2], v[3][j >> 2], sel));
          mma_16816(o[j], pa[0], pa[1], pa[2], pa[3], b0, b1);
        }
      } else {
        uint32_t v[4][D / 16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = kk0 + (e >> 1) * 8 + (e & 1) * key_step;
#pragma unroll
          for (int p = 0; p < D / 64; ++p) {
            const uint4 u = lds128(sV + chunk_at<D, E4M3>(row, 8 * p + ch_v));
            v[e][4 * p] = u.x;
            v[e][4 * p + 1] = u.y;
            v[e][4 * p + 2] = u.z;
            v[e][4 * p + 3] = u.w;
          }
        }
        if (tail) {
          // A key past the end contributes nothing, whatever its slot holds.  A
          // drafted key with an element that is not finite must not reach the
          // rows that do not see it through 0 * inf: its value is taken out of
          // the product, and the rows that see it become NaN.
          unsigned nonfinite = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + kk0 + (e >> 1) * 8 + (e & 1) * key_step;
            bool bad = false;
#pragma unroll
            for (int x = 0; x < D / 16; ++x) bad |= has_nonfinite(v[e][x]);
            if (bad && key >= sq.prefix) nonfinite |= 1u << e;
          }
          nonfinite |= __shfl_xor_sync(kFull, nonfinite, 4);
          nonfinite |= __shfl_xor_sync(kFull, nonfinite, 8);
          nonfinite |= __shfl_xor_sync(kFull, nonfinite, 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + kk0 + (e >> 1) * 8 + (e & 1) * key_step;
            if (key >= sq.len || ((nonfinite >> e) & 1)) {
#pragma unroll
              for (int x = 0; x < D / 16; ++x) v[e][x] = 0;
            }
            if ((nonfinite >> e) & 1) {
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                if (sc[e >> 1][2 * hf + (e & 1)] != NEG_INF)
                  pv[e >> 1][2 * hf + (e & 1)] = __int_as_float(0x7fc00000);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          pa[2 * x] = pack_bf16x2(pv[x][0], pv[x][1]);
          pa[2 * x + 1] = pack_bf16x2(pv[x][2], pv[x][3]);
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          const uint32_t b0 = __byte_perm(v[0][j >> 1], v[1][j >> 1], sel);
          const uint32_t b1 = __byte_perm(v[2][j >> 1], v[3][j >> 1], sel);
          mma_16816(o[j], pa[0], pa[1], pa[2], pa[3], b0, b1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(b_empty(s));
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicCAS(a.status, 0, ATTN_DEVICE_TIMEOUT_BASE + 31);
    }
  }
  __syncthreads();

  // ---- merge the four warps' shares of the split; the ring is free now
  const bool gave_up = *abort_flag != 0;
  float* red = reinterpret_cast<float*>(smem);        // [warp][row][D]
  float* red_m = red + kWarps * kRows * D;            // [warp][row]
  float* red_l = red_m + kWarps * kRows;
  if (warp < kWarps) {
    const int n = lane >> 2, q = lane & 3;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float l = sum[hf];
      l += __shfl_xor_sync(kFull, l, 1);
      l += __shfl_xor_sync(kFull, l, 2);
      const int r = n + 8 * hf;
      if (q == 0) {
        red_m[warp * kRows + r] = ref[hf];
        red_l[warp * kRows + r] = l;
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int x = 2 * q + c;  // column of the block
          int col;
          if constexpr (!E4M3)
            col = (j >> 3) * 64 + (((x & 1) << 2) | (x >> 1)) * 8 + (j & 7);
          else if constexpr (D == 64)
            col = x * 8 + j;
          else
            col = (((x & 1) << 2) | (x >> 1)) * 16 + j;
          red[(warp * kRows + r) * D + col] = o[j][2 * hf + c];
        }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
    const int r = i / (D / 2), c = (i % (D / 2)) * 2;
    float M = NEG_INF;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w * kRows + r]);
    float den = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = red_m[w * kRows + r] == M ? 1.f : ex2(red_m[w * kRows + r] - M);
      den += f * red_l[w * kRows + r];
      x += f * red[(w * kRows + r) * D + c];
      y += f * red[(w * kRows + r) * D + c + 1];
    }
    if (gave_up) den = 0.f;
    if (den == 0.f) x = y = 0.f;  // a row that sees nothing here
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const size_t at = out_row(r);
    if (a.n_splits > 1) {
      *reinterpret_cast<float2*>(a.o_part + (at * a.n_splits + split) * D + c) = make_float2(x * inv, y * inv);
      if (c == 0) a.lse_part[at * a.n_splits + split] = den == 0.f ? NEG_INF : M + __log2f(den);
    } else {
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o) + at * D + c) = pack_bf16x2(x * inv, y * inv);
    }
  }
}

// Exact merge of the splits: one warp a row, D/32 columns a lane.
template <int D>
__global__ void __launch_bounds__(128) tree_merge_kernel(const TreeLaunch a) {
  const int b = blockIdx.y;
  const Seq sq = seq_of(a.cu_q, a.seq_lens, b, a.max_q, a.total_q, a.L, a.max_pages);
  const int r = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= sq.T * a.Hq) return;
  const size_t at = static_cast<size_t>(sq.tok0) * a.Hq + r;
  const float* lse = a.lse_part + at * a.n_splits;
  const float* part = a.o_part + at * a.n_splits * D;
  const float NEG_INF = -__int_as_float(0x7f800000);
  float M = NEG_INF;
  for (int s = lane; s < a.n_splits; s += 32) M = fmaxf(M, lse[s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  constexpr int kC = D / 32;
  float num[kC], den = 0.f;
#pragma unroll
  for (int c = 0; c < kC; ++c) num[c] = 0.f;
  for (int s = 0; s < a.n_splits; ++s) {
    const float l = lse[s];
    if (l == NEG_INF) continue;  // an empty split: its partial sums were not written
    const float w = l == M ? 1.f : ex2(l - M);
    den += w;
#pragma unroll
    for (int c = 0; c < kC; c += 2) {
      const float2 x = *reinterpret_cast<const float2*>(part + static_cast<size_t>(s) * D + lane * kC + c);
      num[c] = fmaf(w, x.x, num[c]);
      num[c + 1] = fmaf(w, x.y, num[c + 1]);
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + at * D + lane * kC;
#pragma unroll
  for (int c = 0; c < kC; c += 2)
    *reinterpret_cast<uint32_t*>(out + c) = pack_bf16x2(num[c] * inv, num[c + 1] * inv);
}

template <int D, bool E4M3>
int launch_rows16(const TreeLaunch& a) {
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
  const int rbs = (a.max_q * (a.Hq / a.Hkv) + kRows - 1) / kRows;
  kern<<<dim3(a.n_splits, a.Hkv * rbs, a.B), kThreads, C::kSmem, a.stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D>
int launch_d(const TreeLaunch& a) {
  const int st = a.k_scales ? launch_rows16<D, true>(a) : launch_rows16<D, false>(a);
  if (st != ATTN_OK || a.n_splits == 1) return st;
  tree_merge_kernel<D><<<dim3((a.max_q * a.Hq + 3) / 4, a.B), 128, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Keys of a split: waves of the 296 resident CTAs (148 SMs x 2) times (tiles of
// a CTA + about 4 tiles' worth of start, merge and partial results).
int split_len_of(int B, int max_q, int Hq, int Hkv, int L) {
  const long long groups = static_cast<long long>(B) * Hkv * ((static_cast<long long>(max_q) * (Hq / Hkv) + kRows - 1) / kRows);
  const int n_tiles = (L + kPage - 1) / kPage;
  int best = n_tiles;
  long long best_cost = -1;
  for (int ns = 1; ns <= n_tiles && ns <= 256; ++ns) {
    const int tps = (n_tiles + ns - 1) / ns;
    const long long n = (n_tiles + tps - 1) / tps;
    const long long cost = (groups * n + 295) / 296 * (tps + 4) + (n > 1 ? 2 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = tps;
    }
  }
  return best * kPage;
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int check_sizes(int B, int max_q, int total_q, int Hq, int Hkv, int L, int d) {
  if (B <= 0 || max_q <= 0 || max_q > 64 || total_q <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || (d != 64 && d != 128)) return ATTN_ERR_INVALID_ARG;
  const long long rbs = (static_cast<long long>(max_q) * (Hq / Hkv) + kRows - 1) / kRows;
  if (B > 65535 || rbs * Hkv > 65535 || L > 0x7fffffff - kPage) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int run_tree(TreeLaunch& a, void* ws, size_t ws_bytes, void* stream) {
  if (!a.q || !a.K || !a.V || !a.o || !a.block_table || !a.seq_lens || !a.cu_q) return ATTN_ERR_INVALID_ARG;
  if (!ptr_aligned(a.q, 16) || !ptr_aligned(a.K, 16) || !ptr_aligned(a.V, 16) || !ptr_aligned(a.o, 16) ||
      !ptr_aligned(a.block_table, 4) || !ptr_aligned(a.seq_lens, 4) || !ptr_aligned(a.cu_q, 4) ||
      !ptr_aligned(a.mask, 8) || !ptr_aligned(a.k_scales, 16) || !ptr_aligned(a.v_scales, 16))
    return ATTN_ERR_INVALID_ARG;
  int st = check_sizes(a.B, a.max_q, a.total_q, a.Hq, a.Hkv, a.L, a.d);
  if (st != ATTN_OK) return st;
  if (a.num_pages <= 0 || a.max_pages <= 0) return ATTN_ERR_INVALID_ARG;
  if (a.L > static_cast<long long>(a.max_pages) * kPage) return ATTN_ERR_INVALID_ARG;
  // one group past the pool's end is addressed for a page id out of range
  if ((static_cast<long long>(a.num_pages) + 1) * a.Hkv > 0x7fffffffLL || a.max_pages > 0x7fffffff / kPage)
    return ATTN_ERR_UNSUPPORTED;
  a.split_len = split_len_of(a.B, a.max_q, a.Hq, a.Hkv, a.L);
  a.n_splits = (a.L + a.split_len - 1) / a.split_len;
  const size_t need = attn_tree_workspace_bytes(a.B, a.max_q, a.total_q, a.Hq, a.Hkv, a.L, a.d);
  if (need > 0) {
    if (!ws || !ptr_aligned(ws, 256) || ws_bytes < need) return ATTN_ERR_INVALID_ARG;
    const size_t part = align256(static_cast<size_t>(a.total_q) * a.Hq * a.n_splits * a.d * sizeof(float));
    a.o_part = static_cast<float*>(ws);
    a.lse_part = reinterpret_cast<float*>(static_cast<char*>(ws) + part);
  }
  int dev = 0;
  if ((st = device_context(&dev, &a.status)) != ATTN_OK) return st;
  a.wait_limit_ns = wait_limit_ns();
  a.scale_log2 = 1.4426950408889634f / std::sqrt(static_cast<float>(a.d));
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_tree(a);
}

}  // namespace

int launch_tree(const TreeLaunch& a) {
  if (a.d == 64) return launch_d<64>(a);
  if (a.d == 128) return launch_d<128>(a);
  return ATTN_ERR_INVALID_ARG;
}

bool tma_map_codes(CUtensorMap* m, const void* base, long long groups, int D) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(kPage), static_cast<cuuint64_t>(groups)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(kPage) * D};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(kPage), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace bss

extern "C" {

size_t attn_tree_workspace_bytes(int B, int max_q, int total_q, int Hq, int Hkv, int max_seq_len, int d) {
  using namespace bss;
  if (check_sizes(B, max_q, total_q, Hq, Hkv, max_seq_len, d) != ATTN_OK) return 0;
  const int ls = split_len_of(B, max_q, Hq, Hkv, max_seq_len);
  const size_t ns = (max_seq_len + ls - 1) / ls;
  if (ns == 1) return 0;
  const size_t rows = static_cast<size_t>(total_q) * Hq * ns;
  return align256(rows * d * sizeof(float)) + align256(rows * sizeof(float));
}

int attn_tree_paged(const void* q, const void* K_pages, const void* V_pages, const int32_t* block_table,
                    const int32_t* seq_lens, const int32_t* cu_q, const uint64_t* tree_mask, void* o, int B,
                    int max_q, int total_q, int Hq, int Hkv, int num_pages, int max_pages_per_seq,
                    int max_seq_len, int d, void* stream, void* ws, size_t ws_bytes) {
  bss::TreeLaunch a{};
  a.q = q;
  a.K = K_pages;
  a.V = V_pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q;
  a.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  a.o = o;
  a.B = B;
  a.max_q = max_q;
  a.total_q = total_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  a.L = max_seq_len;
  a.d = d;
  return bss::run_tree(a, ws, ws_bytes, stream);
}

int attn_tree_paged_e4m3(const void* q, const void* K_codes, const void* V_codes, const float* K_scales,
                         const float* V_scales, const int32_t* block_table, const int32_t* seq_lens,
                         const int32_t* cu_q, const uint64_t* tree_mask, void* o, int B, int max_q, int total_q,
                         int Hq, int Hkv, int num_pages, int max_pages_per_seq, int max_seq_len, int d,
                         void* stream, void* ws, size_t ws_bytes) {
  if (!K_scales || !V_scales) return ATTN_ERR_INVALID_ARG;
  bss::TreeLaunch a{};
  a.q = q;
  a.K = K_codes;
  a.V = V_codes;
  a.k_scales = K_scales;
  a.v_scales = V_scales;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.cu_q = cu_q;
  a.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  a.o = o;
  a.B = B;
  a.max_q = max_q;
  a.total_q = total_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.num_pages = num_pages;
  a.max_pages = max_pages_per_seq;
  a.L = max_seq_len;
  a.d = d;
  return bss::run_tree(a, ws, ws_bytes, stream);
}

}  // extern "C"
