// Norms of queries and keys for each head, with the rotation by position in
// the same pass: the step between the projection and attn_prefill / the cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * w            (skipped where w is null)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * inv_freq[i]
//
// for the pairs (a, b) of the first rot elements: (i, i + rot/2), or (2i, 2i+1)
// when interleaved.  Everything is fp32 between the bf16 load and the one
// rounding at the store.  The angle is the exact product pos * inv_freq[i],
// taken in fp64 and reduced to a fraction of a turn before fp32 sees it: at
// position 2^17 an fp32 product is already off by 2^-8 rad.
//
// Bound by HBM: every element is read once and written once.  A row (one head
// of one token) is held by D/16 lanes with two chunks of 8 elements each, the
// two that meet in the rotation, so a pair needs no shuffle and the mean a
// butterfly of 2 or 3 steps.  A CTA takes several tokens; `groups` groups of
// lanes share a token's heads, so that a thread stays with one token and one
// chunk of its angles, and loads a row ahead of the one that it turns.  The
// tokens' sines and cosines are made once, into shared memory, while the first
// rows are on their way.
//
// 8192 tokens x 40 heads of 128: 28.8 us, 5.8 TB/s of the 6.55 of a copy; 30011
// x 20 heads of 64: 29.2 us, 5.3 TB/s, with a third of the issue slots idle and
// about 40 KB in flight an SM.  Two values to an fp32 instruction changed nothing.
// Ten CTAs an SM leave 48 registers, of which 24 to 32 bytes a thread are spilled.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace bss {

namespace {

constexpr int kThreads = 128;  // 256: 2% slower, by the tails of the launch
constexpr unsigned kFull = 0xffffffffu;

struct RopeArgs {
  const __nv_bfloat16* x[2];  // q, k
  __nv_bfloat16* y[2];
  const __nv_bfloat16* w[2];  // nullable
  const int* pos;
  const float* inv_freq;
  long long xs[2][3], ys[2][3];  // strides in elements: batch, token, head
  long long pos_stride_b;
  int B, N, Hq, H, rot, interleaved;  // H = Hq + Hkv
  int groups;  // groups of lanes that share a token
  int heads;   // of a token in a CTA
  float eps;
};

__device__ __forceinline__ void unpack8(const uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// CTA (x, y): kGroups / groups tokens, their heads [y * heads, ...).
template <int D, bool NORM>
__global__ void __launch_bounds__(kThreads, 10) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kLanes = D / 16;              // lanes of a row
  constexpr int kGroups = kThreads / kLanes;  // rows at a time
  extern __shared__ __align__(16) float s_angle[];  // [token][cos, sin][rot / 2]
  const int group = threadIdx.x / kLanes, l = threadIdx.x % kLanes;
  const int half = a.rot / 2;
  // this lane's chunks: i and i + rot/16 of the rotated part, or two beyond it
  const bool turned = l * 8 < half;
  const int c0 = turned ? l * 8 : 16 * l, step = turned ? half : 8;
  const int T = kGroups / a.groups, token = group / a.groups;
  const unsigned tokens = static_cast<unsigned>(a.B) * static_cast<unsigned>(a.N);
  const unsigned tok0 = blockIdx.x * T, t = tok0 + token;
  const bool live = t < tokens;
  long long xq = 0, xk = 0, yq = 0, yk = 0;
  if (live) {
    const unsigned b = a.B == 1 ? 0 : t / a.N, n = t - b * a.N;
    xq = b * a.xs[0][0] + n * a.xs[0][1] + c0;
    xk = b * a.xs[1][0] + n * a.xs[1][1] + c0 - a.Hq * a.xs[1][2];
    yq = b * a.ys[0][0] + n * a.ys[0][1] + c0;
    yk = b * a.ys[1][0] + n * a.ys[1][1] + c0 - a.Hq * a.ys[1][2];
  }
  const int end = min(a.H, static_cast<int>(blockIdx.y + 1) * a.heads);
  int h = blockIdx.y * a.heads + group - token * a.groups;
  uint4 u[2];
  auto load = [&](int head) {
    u[0] = u[1] = make_uint4(0, 0, 0, 0);
    if (live && head < end) {
      const __nv_bfloat16* x = head < a.Hq ? a.x[0] + xq + head * a.xs[0][2] : a.x[1] + xk + head * a.xs[1][2];
      u[0] = *reinterpret_cast<const uint4*>(x);
      u[1] = *reinterpret_cast<const uint4*>(x + step);
    }
  };
  load(h);
  for (int i = threadIdx.x; i < T * half; i += kThreads) {
    const unsigned ti = i / half, f = i - ti * half, tt = tok0 + ti;
    if (tt < tokens) {
      const unsigned b = a.B == 1 ? 0 : tt / a.N, n = tt - b * a.N;
      const double turns = static_cast<double>(a.pos[b * a.pos_stride_b + n]) * static_cast<double>(a.inv_freq[f]) *
                           0.15915494309189533577;
      const float part = static_cast<float>(turns - rint(turns));  // of a turn: [-1/2, 1/2]
      sincospif(2.f * part, &s_angle[ti * a.rot + half + f], &s_angle[ti * a.rot + f]);
    }
  }
  __syncthreads();
  // interleaved: the pairs lie inside a chunk, 4 angles each
  const float* angle = s_angle + token * a.rot + (a.interleaved ? c0 / 2 : c0);

  // every lane of a warp makes every round: the shuffles are warp-wide
  for (int round = blockIdx.y * a.heads; round < end; round += a.groups, h += a.groups) {
    float f[2][8];
    unpack8(u[0], f[0]);
    unpack8(u[1], f[1]);
    load(h + a.groups);
    const bool key = h >= a.Hq;
    if constexpr (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(f[0][i], f[0][i], fmaf(f[1][i], f[1][i], ss));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      const __nv_bfloat16* w = key ? a.w[1] : a.w[0];
      if (w) {
        const float rs = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float wf[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(w + c0 + x * step)), wf);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[x][i] *= rs * wf[i];
        }
      }
    }
    if (turned) {  // an element outside the rotated part stays as it is, NaN and inf among them
      if (a.interleaved) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float4 c4 = *reinterpret_cast<const float4*>(angle + x * step / 2);
          const float4 s4 = *reinterpret_cast<const float4*>(angle + half + x * step / 2);
          const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = f[x][2 * i], q = f[x][2 * i + 1];
            f[x][2 * i] = fmaf(p, cs[i], -q * sn[i]);
            f[x][2 * i + 1] = fmaf(q, cs[i], p * sn[i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 c4 = *reinterpret_cast<const float4*>(angle + i);
          const float4 s4 = *reinterpret_cast<const float4*>(angle + half + i);
          const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = f[0][i + e], q = f[1][i + e];
            f[0][i + e] = fmaf(p, cs[e], -q * sn[e]);
            f[1][i + e] = fmaf(q, cs[e], p * sn[e]);
          }
        }
      }
    }
    if (live && h < end) {
      __nv_bfloat16* y = key ? a.y[1] + yk + h * a.ys[1][2] : a.y[0] + yq + h * a.ys[0][2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *reinterpret_cast<uint4*>(y + x * step) =
            make_uint4(pack_bf16x2(f[x][0], f[x][1]), pack_bf16x2(f[x][2], f[x][3]), pack_bf16x2(f[x][4], f[x][5]),
                       pack_bf16x2(f[x][6], f[x][7]));
    }
  }
}

template <int D>
void launch_d(RopeArgs& a, cudaStream_t s) {
  constexpr int kGroups = kThreads / (D / 16);
  const unsigned tokens = static_cast<unsigned>(a.B) * static_cast<unsigned>(a.N);
  const unsigned passes = (a.H + kGroups - 1) / kGroups;
  a.groups = kGroups;
  a.heads = a.H;
  if (static_cast<long long>(tokens) * passes <= 148 * 6) {
    // all rows at once: the latency of a call is one row's (16 tokens x 40 heads of
    // 128: 3.1 us, 5.9 by the rule below)
    a.heads = kGroups;
  } else {
    // the most groups a token that leave at most a tenth of them idle (with one
    // token to a CTA of 256 threads, 8192 x 40 heads took 39.9 us instead of 29.7,
    // 30011 x 20 heads of 64 110 instead of 29.9)
    auto idle = [&](int g) { return 10 * (((a.H + g - 1) / g) * g - a.H) > ((a.H + g - 1) / g) * g; };
    while (a.groups > 1 && idle(a.groups)) a.groups /= 2;
  }
  const int T = kGroups / a.groups;
  const dim3 grid((tokens + T - 1) / T, (a.H + a.heads - 1) / a.heads);
  const size_t smem = static_cast<size_t>(T) * a.rot * sizeof(float);
  if (a.w[0] || a.w[1])
    norm_rope_kernel<D, true><<<grid, kThreads, smem, s>>>(a);
  else
    norm_rope_kernel<D, false><<<grid, kThreads, smem, s>>>(a);
}

}  // namespace

}  // namespace bss

extern "C" int attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out,
                                 const int32_t* positions, const float* inv_freq,
                                 const void* q_weight, const void* k_weight, int B, int N, int Hq,
                                 int Hkv, int d, int rot_dim, int interleaved, float eps,
                                 const long long* strides, long long pos_stride_b, void* stream) {
  using namespace bss;
  if (!q || !k || !q_out || !k_out || !strides) return ATTN_ERR_INVALID_ARG;
  if (!ptr_aligned(q, 16) || !ptr_aligned(k, 16) || !ptr_aligned(q_out, 16) ||
      !ptr_aligned(k_out, 16) || !ptr_aligned(q_weight, 16) || !ptr_aligned(k_weight, 16))
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0 || Hq <= 0 || Hkv <= 0 || (d != 64 && d != 128)) return ATTN_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0) return ATTN_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!positions || !inv_freq)) return ATTN_ERR_INVALID_ARG;
  if (!ptr_aligned(positions, 4) || !ptr_aligned(inv_freq, 4)) return ATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || eps > 3.0e38f) return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 12; ++i)
    if (strides[i] % 8 != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(Hq) + Hkv > 65535 || static_cast<long long>(B) * N > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  int dev = 0;
  int* status = nullptr;
  const int st = device_context(&dev, &status);
  if (st != ATTN_OK) return st;
  RopeArgs a{};
  a.x[0] = static_cast<const __nv_bfloat16*>(q);
  a.x[1] = static_cast<const __nv_bfloat16*>(k);
  a.y[0] = static_cast<__nv_bfloat16*>(q_out);
  a.y[1] = static_cast<__nv_bfloat16*>(k_out);
  a.w[0] = static_cast<const __nv_bfloat16*>(q_weight);
  a.w[1] = static_cast<const __nv_bfloat16*>(k_weight);
  a.pos = positions;
  a.inv_freq = inv_freq;
  for (int t = 0; t < 2; ++t)
    for (int i = 0; i < 3; ++i) {
      a.xs[t][i] = strides[3 * t + i];
      a.ys[t][i] = strides[6 + 3 * t + i];
    }
  a.pos_stride_b = pos_stride_b;
  a.N = N;
  a.Hq = Hq;
  a.H = Hq + Hkv;
  a.rot = rot_dim;
  a.interleaved = interleaved ? 1 : 0;
  a.eps = eps;
  a.B = B;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    launch_d<64>(a, s);
  else
    launch_d<128>(a, s);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
