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
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// Two e4m3 codes in the upper bytes of the halfwords of w (the lower bytes may
// hold anything) to two bf16: sign, exponent and mantissa move to their bf16
// places, and 2^120 moves the exponent's bias from 7 to 127, subnormal codes
// included.  Exact.  The NaN code (0x7f) comes out as 480: the writer never
// stores it under a finite scale, and a NaN scale makes the value NaN.
__device__ __forceinline__ uint32_t e4m3_hi_to_bf16x2(uint32_t w) {
  return mul_bf16x2((w & 0x80008000u) | ((w >> 4) & 0x07f007f0u), 0x7b807b80u);
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

// ---------------------------------------------------------------------------
// Kernel for many rows: 128 rows a CTA on tcgen05.
//
//   warp 0      copies: K and V pages, a ring in shared memory
//   warp 1      TMEM, and the one thread that issues the MMAs:
//                 S_j = Q K_j^T (two buffers), O += P_j V_j (P read from TMEM)
//   warps 2-5   softmax: a thread owns the row of TMEM lane 32 (warp % 4) + lane
//   warps 6...  tiles: e4m3 codes to bf16 (4 warps), or the check of the tiles
//               that hold drafted keys (2 warps, bf16 pool)
//
// A tile is one page of 64 keys, so that TMEM holds O and two S in 256 columns
// and two CTAs share an SM: one's softmax runs beside the other's MMAs.  The
// rows past the last one are zero queries; softmax warps without a row leave.
constexpr int kMmaRows = 128;

template <int D, bool E4M3>
struct BigCfg {
  static constexpr int kPrep = E4M3 ? 4 : 2;  // warps that convert or check tiles
  static constexpr int kThreads = (6 + kPrep) * 32;
  static constexpr int kPanels = D / 64;
  static constexpr int kQPanel = kMmaRows * 128;
  static constexpr int kTile = kPage * D * 2;  // K or V of a page as bf16
  static constexpr int kTilePanel = kPage * 128;
  static constexpr int kRaw = kPage * D;       // as codes
  static constexpr int kRing = E4M3 ? (D == 128 ? 5 : 8) : (D == 128 ? 4 : 6);  // tiles in flight
  static constexpr int kSlot = E4M3 ? kRaw : kTile;
  static constexpr int kOffQ = 0;
  static constexpr int kOffConv = kOffQ + kMmaRows * D * 2;        // e4m3: bf16 K, bf16 V
  static constexpr int kOffRing = kOffConv + (E4M3 ? 2 * kTile : 0);
  static constexpr int kOffScale = kOffRing + kRing * kSlot;       // e4m3: [slot][64] floats
  static constexpr int kOffBar = kOffScale + (E4M3 ? kRing * kPage * 4 : 0);
  // full[ring], empty[ring], q_full, s_full[2], p_full[2], pv_done, o_final,
  // checked[2]; bf16: drafted[2]; e4m3: ready[K, V], free[K, V]
  static constexpr int kBars = 2 * kRing + 13;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kSmem = kOffMisc + 64 + 1024;
  static constexpr int kTmemCols = 256;
  static_assert(D + 2 * kPage <= kTmemCols, "O and two S");
};

struct BigMisc {
  unsigned long long bad[2];  // drafted keys of a tile whose value is not finite
  uint32_t tmem_base;
  int abort;
  int bad_page[8];  // e4m3: the slot's page id was out of range
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(BigCfg<D, E4M3>::kThreads, 2)
    tree_rows128_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const TreeLaunch a) {
  using C = BigCfg<D, E4M3>;
  static_assert(sizeof(BigMisc) <= 64 && C::kRing <= 8, "misc layout");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  BigMisc* misc = reinterpret_cast<BigMisc*>(smem + C::kOffMisc);
  volatile int* abort_flag = &misc->abort;
  const uint32_t bar0 = sbase + C::kOffBar;
  auto b_full = [&](int s) { return bar0 + 8u * s; };
  auto b_empty = [&](int s) { return bar0 + 8u * (C::kRing + s); };
  const uint32_t bar1 = bar0 + 16u * C::kRing;
  const uint32_t b_q_full = bar1;
  auto b_s_full = [&](int i) { return bar1 + 8u * (1 + i); };
  auto b_p_full = [&](int i) { return bar1 + 8u * (3 + i); };
  const uint32_t b_pv_done = bar1 + 8u * 5;
  const uint32_t b_o_final = bar1 + 8u * 6;
  // V of the CTA's i-th tile with drafted keys is checked; bf16: has landed
  auto b_checked = [&](int i) { return bar1 + 8u * (7 + i); };
  auto b_drafted = [&](int i) { return bar1 + 8u * (9 + i); };
  // e4m3: K (0) or V (1) is converted, its MMAs are done
  auto b_ready = [&](int v) { return bar1 + 8u * (9 + v); };
  auto b_free = [&](int v) { return bar1 + 8u * (11 + v); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x;
  const int kv = blockIdx.y % a.Hkv, rb = blockIdx.y / a.Hkv;
  const int b = blockIdx.z;
  const int g = a.Hq / a.Hkv;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const Seq sq = seq_of(a.cu_q, a.seq_lens, b, a.max_q, a.total_q, a.L, a.max_pages);
  const int row0 = rb * kMmaRows;
  const int rows = min(kMmaRows, sq.T * g - row0);
  if (rows <= 0) return;
  const int t_begin = split * (a.split_len / kPage);
  const int t_end = min((sq.len + kPage - 1) / kPage, t_begin + a.split_len / kPage);
  const int nt = t_end - t_begin;
  auto out_row = [&](int r) {
    const int t = (row0 + r) / g;
    return static_cast<size_t>(sq.tok0 + t) * a.Hq + kv * g + (row0 + r) - t * g;
  };
  if (nt <= 0) {
    if (a.n_splits > 1) {
      for (int r = threadIdx.x; r < rows; r += C::kThreads)
        a.lse_part[out_row(r) * a.n_splits + split] = NEG_INF;
    } else {
      for (int i = threadIdx.x; i < rows * D; i += C::kThreads)
        static_cast<__nv_bfloat16*>(a.o)[out_row(i / D) * D + i % D] = __float2bfloat16_rn(0.f);
    }
    return;
  }
  // tiles from jt0 on hold drafted keys (at most two) or end past the last key
  const int jt0 = sq.prefix / kPage - t_begin;
  const int active = (rows + 31) / 32;  // softmax warps with a row

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRing; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), E4M3 ? C::kPrep : 1);
    }
    mbar_init(b_q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s_full(i), 1);
      mbar_init(b_p_full(i), active);
      mbar_init(b_checked(i), C::kPrep);
      if constexpr (E4M3) {
        mbar_init(b_ready(i), C::kPrep);
        mbar_init(b_free(i), 1);
      } else {
        mbar_init(b_drafted(i), 1);
      }
      misc->bad[i] = 0;
    }
    mbar_init(b_pv_done, 1);
    mbar_init(b_o_final, 1);
    misc->abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&misc->tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tO = misc->tmem_base;
  auto tS = [&](int i) { return tO + D + i * kPage; };
  auto give_up = [&](int site) {
    *abort_flag = 1;
    atomicCAS(a.status, 0, ATTN_DEVICE_TIMEOUT_BASE + site);
  };

  // The ring's sequence is the order of use: K_0, K_1, V_0, K_2, V_1, ...,
  // V_last.  Item i: V of tile i/2 - 1 for even i >= 2 (and for the last one),
  // else K of tile (i + 1) / 2.
  const int n_items = 2 * nt;
  auto item_of = [&](int i, int& tile) {  // returns whether it is a V tile
    if (i == n_items - 1) {
      tile = nt - 1;
      return true;
    }
    if (i == 0 || (i & 1)) {
      tile = (i + 1) / 2;
      return false;
    }
    tile = i / 2 - 1;
    return true;
  };
  auto item_k = [&](int tile) { return tile == 0 ? 0 : 2 * tile - 1; };
  auto item_v = [&](int tile) { return tile == nt - 1 ? n_items - 1 : 2 * tile + 2; };

  if (warp == 0) {
    // ------------------------------------------------ copies
    const int* table = a.block_table + static_cast<size_t>(b) * a.max_pages + t_begin;
    int pages_k = 0, pages_v = 0;  // lane i: the page of tile i + 32 n, for the K and the V stream
    int issued = 0, drafted = 0;
    bool ok = true;
    for (int i = 0; i < n_items && ok; ++i) {
      int tile;
      const bool is_v = item_of(i, tile);
      if ((tile & 31) == 0) {
        const int p = tile + lane < nt ? table[tile + lane] : -1;
        if (is_v)
          pages_v = p;
        else
          pages_k = p;
      }
      const int page = __shfl_sync(kFull, is_v ? pages_v : pages_k, tile & 31);
      const int s = i % C::kRing;
      if (lane == 0) {
        if (i >= C::kRing)
          ok = mbar_wait(b_empty(s), ((i / C::kRing) - 1) & 1, abort_flag, a.wait_limit_ns);
        if (ok) {
          const bool good = page >= 0 && page < a.num_pages;
          const long long grp = static_cast<long long>(good ? page : a.num_pages) * a.Hkv + kv;
          const uint32_t dst = sbase + C::kOffRing + s * C::kSlot;
          if constexpr (E4M3) {
            misc->bad_page[s] = good ? 0 : 1;  // reads zeros
            mbar_arrive_expect_tx(b_full(s), good ? C::kRaw + kPage * 4 : 0);
            if (good) {
              bulk_load(dst, static_cast<const uint8_t*>(is_v ? a.V : a.K) + grp * C::kRaw, C::kRaw, b_full(s));
              bulk_load(sbase + C::kOffScale + s * (kPage * 4), (is_v ? a.v_scales : a.k_scales) + grp * kPage,
                        kPage * 4, b_full(s));
            }
          } else {  // a page id out of range: the box lies past the pool's end and reads zeros
            uint32_t bar = b_full(s);
            if (is_v && tile >= jt0) {  // the MMA issuer waits for the check instead
              bar = b_drafted(tile - max(jt0, 0));
              mbar_arrive(b_full(s));
              drafted = tile - max(jt0, 0) + 1;
            }
            mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
            for (int p = 0; p < C::kPanels; ++p)
              tma_load_3d(dst + p * C::kTilePanel, is_v ? &tmV : &tmK, bar, p * 64, 0, static_cast<int>(grp));
          }
          ++issued;
        }
      }
      ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
    }
    if (lane == 0) {
      if (!ok) give_up(40);
      for (int i = max(0, issued - C::kRing); i < issued; ++i)  // no copy in flight at the end
        mbar_drain(b_full(i % C::kRing), (i / C::kRing) & 1, a.wait_limit_ns);
      for (int i = 0; i < drafted; ++i) mbar_drain(b_drafted(i), 0, a.wait_limit_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(kMmaRows, kPage, false, false);
      constexpr uint32_t idPV = idesc_bf16_f32(kMmaRows, D, false, true);
      auto wait = [&](uint32_t bar, int parity, int site) {
        if (mbar_wait(bar, parity, abort_flag, a.wait_limit_ns)) return true;
        give_up(site);
        return false;
      };
      bool ok = wait(b_q_full, 0, 41);
      for (int j = 0; ok && j <= nt; ++j) {
        if (j < nt) {
          const int i = item_k(j), s = i % C::kRing;
          const uint32_t sK = sbase + (E4M3 ? C::kOffConv : C::kOffRing + s * C::kSlot);
          if (!(ok = E4M3 ? wait(b_ready(0), j & 1, 42) : wait(b_full(s), (i / C::kRing) & 1, 42))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk & 3) * 32;  // 16 bf16 = 32 B inside a 128 B row
            mma_ss(tS(j & 1), sw128_desc(sbase + C::kOffQ + (kk >> 2) * C::kQPanel + off, 16, 1024),
                   sw128_desc(sK + (kk >> 2) * C::kTilePanel + off, 16, 1024), idS, kk > 0 ? 1u : 0u);
          }
          mma_commit(b_s_full(j & 1));
          mma_commit(E4M3 ? b_free(0) : b_empty(s));
        }
        if (j >= 1) {
          const int t = j - 1, i = item_v(t), s = i % C::kRing;
          const uint32_t sV = sbase + (E4M3 ? C::kOffConv + C::kTile : C::kOffRing + s * C::kSlot);
          if (!(ok = E4M3 ? wait(b_ready(1), t & 1, 43) : wait(b_full(s), (i / C::kRing) & 1, 43))) break;
          if (!E4M3 && t >= jt0 && !(ok = wait(b_checked(t - max(jt0, 0)), 0, 44))) break;
          if (!(ok = wait(b_p_full(t & 1), (t >> 1) & 1, 45))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kPage / 16; ++kk)
            mma_ts(tO, tS(t & 1) + kk * 8, sw128_desc(sV + kk * 16 * 128, C::kTilePanel, 1024), idPV,
                   (t > 0 || kk > 0) ? 1u : 0u);
          mma_commit(E4M3 ? b_free(1) : b_empty(s));
          mma_commit(b_pv_done);
        }
      }
      mma_commit(b_o_final);
      mbar_drain(b_o_final, 0, a.wait_limit_ns);  // MMAs finish before TMEM is released
    }
  } else if (warp < 6) {
    // ------------------------------------------------ softmax
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool valid = r < rows;
    const int tok = valid ? (row0 + r) / g : 0;
    {  // this row of Q into the swizzled operand
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                        (valid ? out_row(r) : 0) * D);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 u = valid ? src[c] : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(smem + C::kOffQ + (c >> 3) * C::kQPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = u;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(b_q_full);
    }
    uint64_t bits = 0;
    if (valid) bits = a.mask ? a.mask[sq.tok0 + tok] : (tok >= 63 ? ~0ull : (2ull << tok) - 1);
    float m_ref = NEG_INF, l_sum = 0.f;
    bool ok = true;
    if ((warp & 3) < active) {
      for (int j = 0; j < nt; ++j) {
        const int sb = j & 1;
        if (!__all_sync(kFull, mbar_wait(b_s_full(sb), (j >> 1) & 1, abort_flag, a.wait_limit_ns))) {
          if (lane == 0) give_up(46);
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t x[kPage];
        tmem_ld_row<kPage>(tS(sb) + lane_off, x);
        tmem_wait_ld();
        const bool tail = j >= jt0;
        uint64_t bad = 0;
        if (tail) {
          // which of the 64 keys this row sees
          const int key0 = (t_begin + j) * kPage;
          const int n_prefix = min(max(sq.prefix - key0, 0), kPage), n_len = min(sq.len - key0, kPage);
          uint64_t sees = n_prefix >= 64 ? ~0ull : (1ull << n_prefix) - 1;
          const int first = key0 - sq.prefix;  // drafted index of the tile's first key
          const uint64_t drafted = first >= 64 ? 0 : first >= 0 ? bits >> first : first > -64 ? bits << -first : 0;
          sees |= drafted;
          if (n_len < 64) sees &= (1ull << n_len) - 1;
#pragma unroll
          for (int c = 0; c < kPage; ++c)
            if (!((sees >> c) & 1)) x[c] = 0xff800000u;
          const int jt = j - max(jt0, 0);
          if (!__all_sync(kFull, mbar_wait(b_checked(jt), 0, abort_flag, a.wait_limit_ns))) {
            if (lane == 0) give_up(47);
            ok = false;
            break;
          }
          bad = *reinterpret_cast<volatile unsigned long long*>(&misc->bad[jt]) & sees;
        }
        float mt = NEG_INF;
#pragma unroll
        for (int c = 0; c < kPage; c += 2) mt = fmax3(mt, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
        mt *= a.scale_log2;
        const bool moved = mt > m_ref + kRefSlack;
        float alpha = 1.f;
        if (moved) {
          alpha = ex2(m_ref - mt);  // m_ref = -inf gives 0
          m_ref = mt;
        }
        const float base = m_ref == NEG_INF ? 0.f : m_ref;
        if (__any_sync(kFull, moved && j > 0)) {
          // O is read and written back: the last P V must have finished
          if (!__all_sync(kFull, mbar_wait(b_pv_done, (j - 1) & 1, abort_flag, a.wait_limit_ns))) {
            if (lane == 0) give_up(48);
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 16) {
            uint32_t o[16];
            tmem_ld16(tO + lane_off + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
            tmem_st16(tO + lane_off + c0, o);
          }
        }
        // P = 2^(x - ref) as bf16 over the scores; the sum adds the rounded values
        float rs = 0.f;
#pragma unroll
        for (int c0 = 0; c0 < kPage; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float p0 = ex2(fmaf(__uint_as_float(x[c0 + 2 * c]), a.scale_log2, -base));
            float p1 = ex2(fmaf(__uint_as_float(x[c0 + 2 * c + 1]), a.scale_log2, -base));
            const uint32_t w = pack_bf16x2(p0, p1);
            rs += __uint_as_float(w << 16) + __uint_as_float(w & 0xffff0000u);
            pk[c] = w;
          }
          if (bad) {  // a value that is not finite was taken out of V: NaN for whoever sees it
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if ((bad >> (c0 + 2 * c)) & 1) pk[c] = (pk[c] & 0xffff0000u) | 0x7fc0u;
              if ((bad >> (c0 + 2 * c + 1)) & 1) pk[c] = (pk[c] & 0xffffu) | 0x7fc00000u;
            }
          }
          tmem_st16(tS(sb) + lane_off + c0 / 2, pk);
        }
        l_sum = l_sum * alpha + rs;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p_full(sb));
      }
      // ---- O / l
      if (__all_sync(kFull, ok && mbar_wait(b_o_final, 0, abort_flag, a.wait_limit_ns) && !*abort_flag)) {
        tc_fence_after();
        const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;  // a row that sees nothing here
        const size_t at = valid ? out_row(r) : 0;
        float* part = a.o_part + (at * a.n_splits + split) * D;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.o) + at * D;
        if (valid && a.n_splits > 1)
          a.lse_part[at * a.n_splits + split] = l_sum == 0.f ? NEG_INF : m_ref + __log2f(l_sum);
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(tO + lane_off + c0, o);
          tmem_wait_ld();
          if (!valid) continue;
          float f[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] = l_sum == 0.f ? 0.f : __uint_as_float(o[c]) * inv;
          if (a.n_splits > 1) {
#pragma unroll
            for (int c = 0; c < 16; c += 4)
              *reinterpret_cast<float4*>(part + c0 + c) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
          } else {
#pragma unroll
            for (int c = 0; c < 16; c += 8)
              *reinterpret_cast<uint4*>(orow + c0 + c) =
                  make_uint4(pack_bf16x2(f[c], f[c + 1]), pack_bf16x2(f[c + 2], f[c + 3]),
                             pack_bf16x2(f[c + 4], f[c + 5]), pack_bf16x2(f[c + 6], f[c + 7]));
          }
        }
      } else if (valid) {  // a wait gave up: no weight in the merge
        const size_t at = out_row(r);
        if (a.n_splits > 1)
          a.lse_part[at * a.n_splits + split] = NEG_INF;
        else
          for (int c = 0; c < D; ++c) static_cast<__nv_bfloat16*>(a.o)[at * D + c] = __float2bfloat16_rn(0.f);
      }
    }
  } else {
    // ------------------------------------------------ tiles
    const int t = threadIdx.x - 6 * 32;
    constexpr int kN = C::kPrep * 32;
    bool ok = true;
    if constexpr (E4M3) {
      for (int i = 0; i < n_items; ++i) {
        int j;
        const int is_v = item_of(i, j) ? 1 : 0;
        const int s = i % C::kRing;
        bool got = mbar_wait(b_full(s), (i / C::kRing) & 1, abort_flag, a.wait_limit_ns);
        if (got && j > 0) got = mbar_wait(b_free(is_v), (j - 1) & 1, abort_flag, a.wait_limit_ns);
        if (!__all_sync(kFull, got)) {
          ok = false;
          break;
        }
        const uint32_t src = sbase + C::kOffRing + s * C::kSlot;
        const uint32_t scales = sbase + C::kOffScale + s * (kPage * 4);
        const uint32_t dst = sbase + C::kOffConv + is_v * C::kTile;
        const bool zero = misc->bad_page[s] != 0;
        const int key0 = (t_begin + j) * kPage;
        constexpr int kChunks = D / 16;  // 16-code chunks of a key
#pragma unroll
        for (int n = 0; n < kPage * kChunks / kN; ++n) {
          const int chunk = n * kN + t, key = chunk / kChunks, c = chunk % kChunks;
          const uint4 u = lds128(src + chunk * 16);
          const float sc = lds_f32(scales + key * 4);
          const uint32_t f = pack_bf16x2(sc, sc);  // a power of two: exact
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            o[2 * e] = mul_bf16x2(e4m3_hi_to_bf16x2(__byte_perm(w[e], 0, 0x1000)), f);
            o[2 * e + 1] = mul_bf16x2(e4m3_hi_to_bf16x2(__byte_perm(w[e], 0, 0x3020)), f);
          }
          bool clear = zero;
          if (is_v && j >= jt0) {
            clear |= key0 + key >= sq.len;
            bool nf = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) nf |= has_nonfinite(o[e]);
            if (nf && !clear && key0 + key >= sq.prefix) {
              clear = true;
              atomicOr(&misc->bad[j - max(jt0, 0)], 1ull << key);
            }
          }
          if (clear) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0;
          }
          // two 16-byte chunks of the bf16 row; the upper half of the row's
          // threads store theirs in the other order, so that eight
          // neighbours meet eight different banks
          const uint32_t row = dst + (c >> 2) * C::kTilePanel + key * 128;
          const int flip = (c >> 2) & 1, c2 = 2 * (c & 3);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int hh = h ^ flip;
            sts128(row + (((c2 + hh) ^ (key & 7)) << 4), hh ? o[4] : o[0], hh ? o[5] : o[1], hh ? o[6] : o[2],
                   hh ? o[7] : o[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(b_empty(s));
          mbar_arrive(b_ready(is_v));
          if (is_v && j >= jt0) mbar_arrive(b_checked(j - max(jt0, 0)));
        }
      }
    } else {
      // V tiles that hold drafted keys: slots past the end are cleared, and
      // values that are not finite taken out (softmax makes up for them)
      for (int j = max(jt0, 0); j < nt; ++j) {
        const int n = j - max(jt0, 0);
        if (!__all_sync(kFull, mbar_wait(b_drafted(n), 0, abort_flag, a.wait_limit_ns))) {
          ok = false;
          break;
        }
        const uint32_t tile = sbase + C::kOffRing + (item_v(j) % C::kRing) * C::kSlot;
        const int key0 = (t_begin + j) * kPage;
        for (int chunk = t; chunk < kPage * (D / 8); chunk += kN) {
          const int key = (chunk / 8) % kPage;
          const uint32_t at = tile + chunk * 16;  // panels of [64][128 B]: the swizzle stays inside a row
          const uint4 u = lds128(at);
          const bool nf = has_nonfinite(u.x) || has_nonfinite(u.y) || has_nonfinite(u.z) || has_nonfinite(u.w);
          const bool past = key0 + key >= sq.len;
          if (past || (nf && key0 + key >= sq.prefix)) {
            sts128(at, 0, 0, 0, 0);
            if (!past) atomicOr(&misc->bad[n], 1ull << key);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_checked(n));
      }
    }
    if (!ok && lane == 0) give_up(49);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tO, C::kTmemCols);
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

template <int D, bool E4M3>
int launch_rows128(const TreeLaunch& a) {
  using C = BigCfg<D, E4M3>;
  auto kern = tree_rows128_kernel<D, E4M3>;
  static uint64_t attr_done = 0;  // one bit per device ordinal
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return ATTN_ERR_CUDA;
  if (!(attr_done >> dev & 1)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done |= uint64_t(1) << dev;
  }
  CUtensorMap mk{}, mv{};  // the e4m3 pages are copied without one
  const int groups = a.num_pages * a.Hkv;
  if (!E4M3 && (!tma_map_bhnd(&mk, a.K, groups, kPage, D, kPage) || !tma_map_bhnd(&mv, a.V, groups, kPage, D, kPage)))
    return ATTN_ERR_CUDA;
  const int rbs = (a.max_q * (a.Hq / a.Hkv) + kMmaRows - 1) / kMmaRows;
  kern<<<dim3(a.n_splits, a.Hkv * rbs, a.B), C::kThreads, C::kSmem, a.stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Rows of a CTA: 16 where all rows of a KV head fit (a decode of single tokens
// with up to 16 query heads a group), else 128.
int rows_of(int max_q, int g) { return max_q * static_cast<long long>(g) <= kRows ? kRows : kMmaRows; }

template <int D>
int launch_d(const TreeLaunch& a) {
  const bool few = rows_of(a.max_q, a.Hq / a.Hkv) == kRows;
  const int st = a.k_scales ? (few ? launch_rows16<D, true>(a) : launch_rows128<D, true>(a))
                            : (few ? launch_rows16<D, false>(a) : launch_rows128<D, false>(a));
  if (st != ATTN_OK || a.n_splits == 1) return st;
  tree_merge_kernel<D><<<dim3((a.max_q * a.Hq + 3) / 4, a.B), 128, 0, a.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Keys of a split: waves of the 296 resident CTAs (148 SMs x 2) times (tiles of
// a CTA + about 4 tiles' worth of start, merge and partial results).
int split_len_of(int B, int max_q, int Hq, int Hkv, int L) {
  const int per = rows_of(max_q, Hq / Hkv);
  const long long groups = static_cast<long long>(B) * Hkv * ((static_cast<long long>(max_q) * (Hq / Hkv) + per - 1) / per);
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
