// Attention of drafted tokens over a paged KV cache, bf16 or e4m3: the C entry
// points, the choice of kernel, and the merge of shares.
//
// Sequence b brings T_b <= 64 drafted tokens, whose keys are already the last
// T_b of its len_b cached ones.  Token i sees the whole prefix and drafted key
// j iff bit j of its mask is set (its ancestors in the tree and itself), so
//   o_i = sum_k p_ik v_k / sum_k p_ik,  p_ik = exp(q_i k_k / sqrt(d) - m_i)
// over the keys that it sees; a token that sees none gets 0 (one whose scores are
// all -inf NaN).  T_b = 1 is the decode of single tokens.  With e4m3 codes key k is
// its codes times ks_k, which scales a column of scores, and value k its codes
// times vs_k.
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
#include "tree.cuh"

namespace bss {

namespace {

constexpr int kFew = 4;  // shares whose loads a warp issues at once

// The sum of the shares of a KV head's keys, exact up to fp32.  A warp takes R
// rows of a KV head, or W warps take one, each every W-th share; a lane holds D/32
// columns.  Rows that one CTA has finished are left alone.  The kernel starts
// while the one before it ends, and looks for its shares meanwhile.
template <int D, int W, int R>
__global__ void __launch_bounds__(128) tree_merge_kernel(const __grid_constant__ TreeLaunch a, int per) {
  static_assert((W == 1 || W == 4) && (W == 1 || R == 1) && 8 % R == 0, "a row's warps are in one CTA");
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
  const Seq s = seq_of(a, b);
  const int group = a.Hq / a.Hkv;
  const int units = (a.max_q * group + R - 1) / R;  // of a KV head
  const int unit = blockIdx.x * (4 / W) + warp / W, kv = unit / units, row0 = (unit - kv * units) * R;
  const int plane = row0 / per;  // of all R rows: per is a multiple of 8
  // this KV head's shares: CTAs c0 to c1, of which the first may be in the CTA's
  // second place
  Line line;
  const Division div(a, plane * per, line);
  while (b >= line.chunk + 32) line.next(a, plane * per);
  const int span = max(1, (s.len + kPage - 1) / kPage);
  const int head_at = line.heads_at(a, b - line.chunk) + kv;
  const int first = line.before + __shfl_sync(kFull, line.incl - line.places(a), b - line.chunk) +
                    kv * (span + kSegment);
  const int rows = min(s.T * group, row0 + R);
  // Every CTA waits here, those without work too: what follows in the stream may
  // count on this kernel's end alone.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kv >= a.Hkv || row0 >= rows) return;  // the same for all warps of a row
  int c0, c1, place0 = 0;
  if (div.shares) {
    c0 = head_at * div.shares;
    c1 = c0 + div.shares - 1;
  } else {
    c0 = div.cta_of(first);
    c1 = div.cta_of(first + span - 1);
    place0 = div.first(c0) >= first ? 0 : 1;
  }
  if (c0 == c1 || (div.shares && span == 1)) return;
  // with fewer tiles than shares, share i is empty unless it ends behind i's start
  auto empty = [&](int c) {
    const long long i = c - c0;
    return div.shares > span && span * i / div.shares == span * (i + 1) / div.shares;
  };
  constexpr int kC = D / 32;
  // The reference and the sum of a share go together: of shares with the same
  // reference, however large, each counts by its sum.  A share's result is its
  // mean already, so a weighted mean of them stays within their range.
  auto weight = [](float2 l, float M) { return l.y == 0.f ? 0.f : l.x == M ? l.y : l.y * ex2(l.x - M); };
  auto write = [&](int row, const float (&mean)[kC], float den) {
    const float none = den == 0.f ? without_sum(s, bits_of(a, s, row / group)) : 0.f;
    const size_t at = static_cast<size_t>(s.tok0 + row / group) * a.Hq + kv * group + row % group;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + at * D + lane * kC;
#pragma unroll
    for (int e = 0; e < kC; e += 2)
      *reinterpret_cast<uint32_t*>(out + e) = den == 0.f ? pack_bf16x2(none, none) : pack_bf16x2(mean[e], mean[e + 1]);
  };
  if (R > 1 && c1 - c0 < kFew) {  // all loads of two rows at once
#pragma unroll 2
    for (int row = row0; row < rows; ++row) {
      float2 l[kFew], v[kFew][kC / 2];
      float w[kFew], M = neg_inf(), den = 0.f, mean[kC];
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        const int c = min(c0 + i, c1);
        const size_t at = share_at(a, per, plane, c, c == c0 ? place0 : 0, row - plane * per);
        l[i] = c0 + i > c1 || empty(c) ? make_float2(neg_inf(), 0.f) : a.sums[at];
#pragma unroll
        for (int e = 0; e < kC / 2; ++e) v[i][e] = reinterpret_cast<const float2*>(a.part + at * D + lane * kC)[e];
      }
#pragma unroll
      for (int i = 0; i < kFew; ++i) M = fmaxf(M, l[i].x);
#pragma unroll
      for (int i = 0; i < kFew; ++i) den += w[i] = weight(l[i], M);
      const float inv = 1.f / den;
#pragma unroll
      for (int e = 0; e < kC; ++e) mean[e] = 0.f;
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        if (w[i] != 0.f) {  // else an empty share, perhaps: its result was not written
#pragma unroll
          for (int e = 0; e < kC / 2; ++e) {
            mean[2 * e] = fmaf(w[i] * inv, v[i][e].x, mean[2 * e]);
            mean[2 * e + 1] = fmaf(w[i] * inv, v[i][e].y, mean[2 * e + 1]);
          }
        }
      }
      write(row, mean, den);
    }
    return;
  }
#pragma unroll 1
  for (int row = row0; row < rows; ++row) {
    auto share = [&](int c) { return share_at(a, per, plane, c, c == c0 ? place0 : 0, row - plane * per); };
    auto sums = [&](int c) { return c > c1 || empty(c) ? make_float2(neg_inf(), 0.f) : a.sums[share(c)]; };
    const float2 own = sums(c0 + lane);  // the others, if there are more than 32, are read again
    float M = own.x;
    for (int c = c0 + lane + 32; c <= c1; c += 32) M = fmaxf(M, sums(c).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    const float w_own = weight(own, M);
    float mean[kC], den = w_own;
    for (int c = c0 + lane + 32; c <= c1; c += 32) den += weight(sums(c), M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
    const float inv = 1.f / den;
#pragma unroll
    for (int c = 0; c < kC; ++c) mean[c] = 0.f;
    for (int base = c0; base <= c1; base += 32) {
      const float w = base == c0 ? w_own : weight(sums(base + lane), M);  // lane i: of share base + i
      const int n = min(32, c1 - base + 1);
#pragma unroll 4
      for (int i = part; i < n; i += W) {
        const float* x = a.part + share(base + i) * D + lane * kC;
        float2 v[kC / 2];
#pragma unroll
        for (int e = 0; e < kC / 2; ++e) v[e] = reinterpret_cast<const float2*>(x)[e];
        const float wi = __shfl_sync(kFull, w, i);
        if (wi != 0.f) {
#pragma unroll
          for (int e = 0; e < kC / 2; ++e) {
            mean[2 * e] = fmaf(wi * inv, v[e].x, mean[2 * e]);
            mean[2 * e + 1] = fmaf(wi * inv, v[e].y, mean[2 * e + 1]);
          }
        }
      }
    }
    if constexpr (W > 1) {
      __shared__ float red[W][D];
#pragma unroll
      for (int e = 0; e < kC; ++e) red[part][lane * kC + e] = mean[e];
      __syncthreads();
      if (part != 0) return;
#pragma unroll
      for (int x = 1; x < W; ++x)
#pragma unroll
        for (int e = 0; e < kC; ++e) mean[e] += red[x][lane * kC + e];
    }
    write(row, mean, den);
  }
}

template <int D, int W, int R>
int launch_merge(const TreeLaunch& a, int per) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const int group = a.Hq / a.Hkv, units = (a.max_q * group + R - 1) / R * a.Hkv;
  cfg.gridDim = dim3((units + 4 / W - 1) / (4 / W), a.B);
  cfg.blockDim = dim3(128);
  cfg.stream = a.stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, W, R>, a, per) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// The launch, as far as the sizes decide it.
struct Plan {
  int per;         // rows of a CTA
  int planes, ctas;
  int min_tiles;
  bool shares;     // whether a KV head's tiles can be divided
  size_t part_bytes, bytes;
};

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

Plan plan_of(int B, int max_q, int Hq, int Hkv, int L, int d, bool e4m3) {
  Plan p{};
  const long long rows = static_cast<long long>(max_q) * (Hq / Hkv);
  // Rows of a CTA.  16 sequences x 16384 keys, 8 KV heads of 128: e4m3 with 4 rows a
  // head 98 us by 8s and 183 by 128s, with 16 rows 112 by 16s and 186 by 128s;
  // bf16 164 and 165 with 4 rows (but one sequence of 500 keys 11 and 14.4), 186 and
  // 165 with 16.
  p.per = rows <= 8 ? 8 : rows <= 16 && e4m3 ? 16 : kManyRows;
  p.planes = static_cast<int>((rows + p.per - 1) / p.per);
  const long long tiles = (L + kPage - 1) / kPage, heads = static_cast<long long>(B) * Hkv;
  const long long slots = 148 * (p.per < kManyRows ? tree_few_ctas(d, e4m3, p.per) : 2);
  const long long fit = p.planes < slots ? slots / p.planes : 1;
  // A CTA for each KV head, and no merge, where its tiles are few, or where the
  // heads are more than the CTAs that run at once and rounds of them cost less
  // than equal pieces: in tiles, rounds * (tiles + kSegment) against the equal piece
  // and its segments.  (16 x 512 e4m3 keys, 1 token: 9.4 us, 11.5 divided; 16 x 1024
  // 13.6 and 15.2, but one sequence of 1024 13.3 and 10.5; 100 x 900 keys 43 and 50.)
  // L is only a limit, and a sequence that alone comes near it would hold up its
  // few CTAs, so the rounds are for short limits (222 sequences of 500 keys but one,
  // that of 2000 keys: 67 us, 61 divided, of 4096 83 and 62, of 100000 850 and 97;
  // 222 that all have 2000 keys 154 and 157, 4096 292 and 298).
  const long long rounds = (heads + fit - 1) / fit;
  if (tiles <= 8 || (tiles <= 32 && rounds > 1 && 2 * rounds * (tiles + kSegment) <
                                                      2 * (heads * tiles / fit) + (2 * heads / fit + 3) * kSegment)) {
    p.min_tiles = 0;
    p.ctas = static_cast<int>(heads);
    return p;
  }
  // No CTA without four tiles: one token over 8192 keys 13 us, 17 from one or two
  // tiles on, where the merge has more to add up (4 tokens over 1024 keys 10.5, 10.2
  // from one tile on).
  p.min_tiles = 4;
  const long long most = (tiles * heads + p.min_tiles - 1) / p.min_tiles;
  p.ctas = static_cast<int>(most < fit ? most : fit);
  p.shares = p.ctas > 1;
  if (p.shares) {
    const size_t n = static_cast<size_t>(p.planes) * p.ctas * 2 * p.per;
    p.part_bytes = align256(n * d * sizeof(float));
    p.bytes = p.part_bytes + align256(n * sizeof(float2));
  }
  return p;
}

// Four warps a row where a KV head has many shares; four rows a warp where there are
// more than the SMs hold warps for at once (16384 rows of 3 shares each, from HBM:
// 15.4 us, 19.6 by one row a warp, whose way to its shares then costs most).
template <int D>
int merge(const TreeLaunch& a, const Plan& p) {
  if (p.ctas > 8ll * a.B * a.Hkv) return launch_merge<D, 4, 1>(a, p.per);
  if (static_cast<long long>(a.B) * a.max_q * a.Hq > 148 * 16) return launch_merge<D, 1, 4>(a, p.per);
  return launch_merge<D, 1, 1>(a, p.per);
}

int check_sizes(int B, int max_q, int total_q, int Hq, int Hkv, int L, int d) {
  if (B <= 0 || max_q <= 0 || max_q > 64 || total_q <= 0 || Hq <= 0 || Hkv <= 0 || L <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || (d != 64 && d != 128)) return ATTN_ERR_INVALID_ARG;
  if (B > 65535 || Hq > 65535 || L > 0x7fffffff - kPage) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>((L + kPage - 1) / kPage + kSegment) * B * Hkv > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
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
  const Plan p = plan_of(a.B, a.max_q, a.Hq, a.Hkv, a.L, a.d, a.k_scales != nullptr);
  if (p.shares) {
    if (!ws || !ptr_aligned(ws, 256) || ws_bytes < p.bytes) return ATTN_ERR_INVALID_ARG;
    a.part = static_cast<float*>(ws);
    a.sums = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.part_bytes);
  }
  int dev = 0;
  if ((st = device_context(&dev, &a.status)) != ATTN_OK) return st;
  a.planes = p.planes;
  a.ctas = p.ctas;
  a.min_tiles = p.min_tiles;
  a.wait_limit_ns = wait_limit_ns();
  a.scale_log2 = 1.4426950408889634f / std::sqrt(static_cast<float>(a.d));
  a.stream = static_cast<cudaStream_t>(stream);
  st = p.per < kManyRows ? launch_tree_few(a, p.per) : launch_tree_many(a);
  if (st != ATTN_OK || !p.shares) return st;
  return a.d == 64 ? merge<64>(a, p) : merge<128>(a, p);
}

}  // namespace

bool tma_map_codes(CUtensorMap* m, const void* base, long long groups, int D, int keys) {
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
  cuuint32_t box[3] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(keys), 1};
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
  // enough for either cache
  const size_t x = plan_of(B, max_q, Hq, Hkv, max_seq_len, d, false).bytes;
  const size_t y = plan_of(B, max_q, Hq, Hkv, max_seq_len, d, true).bytes;
  return x > y ? x : y;
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
