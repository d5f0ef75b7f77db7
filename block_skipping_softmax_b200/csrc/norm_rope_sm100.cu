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
// of one token) is held by D/8 lanes of 16 bytes, so the mean is a 3- or
// 4-step butterfly and a pair (i, i + rot/2) one shuffle.  A CTA takes the
// heads of one token, which share the angles: rot/2 threads compute sines and
// cosines once into shared memory while the rows' loads are in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace bss {

namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

struct RopeArgs {
  const __nv_bfloat16* x[2];  // q, k
  __nv_bfloat16* y[2];
  const __nv_bfloat16* w[2];  // nullable
  const int* pos;
  const float* inv_freq;
  long long xs[2][3], ys[2][3];  // strides in elements: batch, token, head
  long long pos_stride_b;
  int N, Hq, H, rot, interleaved;  // H = Hq + Hkv
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

// R rows for each group of D/8 lanes, all loaded before the angles are known.
template <int D, int R>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeArgs a) {
  constexpr int kLanes = D / 8;               // lanes of a row
  constexpr int kGroups = kThreads / kLanes;  // rows at a time
  __shared__ __align__(16) float s_cos[D / 2], s_sin[D / 2];
  const int b = blockIdx.x / a.N, n = blockIdx.x % a.N;
  const int group = threadIdx.x / kLanes, c = threadIdx.x % kLanes;  // c: chunk of 8 elements
  const int head0 = blockIdx.y * (kGroups * R) + group;

  uint4 u[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int h = head0 + r * kGroups;
    const int side = h >= a.Hq;
    u[r] = make_uint4(0, 0, 0, 0);
    if (h < a.H)
      u[r] = *reinterpret_cast<const uint4*>(a.x[side] + b * a.xs[side][0] + n * a.xs[side][1] +
                                             (h - (side ? a.Hq : 0)) * a.xs[side][2] + c * 8);
  }
  const int half = a.rot / 2;
  if (threadIdx.x < half) {
    const double turns = static_cast<double>(a.pos[b * a.pos_stride_b + n]) *
                         static_cast<double>(a.inv_freq[threadIdx.x]) * 0.15915494309189533577;
    const float part = static_cast<float>(turns - rint(turns));  // a turn: [-1/2, 1/2]
    sincospif(2.f * part, &s_sin[threadIdx.x], &s_cos[threadIdx.x]);
  }
  __syncthreads();

  // this chunk's angles: 4 pairs inside the chunk, or 8 pairs with the chunk
  // rot/16 chunks away (the first half takes -sin, the second half +sin)
  const bool turned = c * 8 < a.rot;
  const bool second = c * 8 >= half;
  float cs[8], sn[8];
  int partner = threadIdx.x & 31;
  if (turned && a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[2 * i] = cs[2 * i + 1] = s_cos[c * 4 + i];
      sn[2 * i + 1] = s_sin[c * 4 + i];
      sn[2 * i] = -sn[2 * i + 1];
    }
  } else if (turned) {
    const int at = second ? c * 8 - half : c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = s_cos[at + i];
      sn[i] = second ? s_sin[at + i] : -s_sin[at + i];
    }
    partner += second ? -(half / 8) : half / 8;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = 1.f, sn[i] = 0.f;
  }

#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int h = head0 + r * kGroups;
    const int side = h >= a.Hq;
    float f[8];
    unpack8(u[r], f);
    const __nv_bfloat16* w = a.w[side];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    if (w) {
      const float rs = rsqrtf(ss * (1.f / D) + a.eps);
      float wf[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(w) + c), wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= rs * wf[i];
    }
    float g[8];
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = f[i ^ 1];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = __shfl_sync(kFull, f[i], partner);
    }
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // an element outside the rotated part stays as it is, NaN and inf among them
      const float lo = turned ? fmaf(f[2 * i], cs[2 * i], g[2 * i] * sn[2 * i]) : f[2 * i];
      const float hi =
          turned ? fmaf(f[2 * i + 1], cs[2 * i + 1], g[2 * i + 1] * sn[2 * i + 1]) : f[2 * i + 1];
      o[i] = pack_bf16x2(lo, hi);
    }
    if (h < a.H)
      *reinterpret_cast<uint4*>(a.y[side] + b * a.ys[side][0] + n * a.ys[side][1] +
                                (h - (side ? a.Hq : 0)) * a.ys[side][2] + c * 8) =
          make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int D, int R>
void launch_r(const RopeArgs& a, unsigned tokens, int ny, cudaStream_t s) {
  norm_rope_kernel<D, R><<<dim3(tokens, ny), kThreads, 0, s>>>(a);
}

template <int D>
void launch_d(const RopeArgs& a, unsigned tokens, cudaStream_t s) {
  constexpr int kGroups = kThreads / (D / 8);
  const int passes = (a.H + kGroups - 1) / kGroups;
  // Rows of a group: one where the whole launch fits the 148 SMs at once (the
  // latency of a call is then one row's), else up to four, so that a CTA's
  // loads cover the memory latency and its angles serve more heads.
  int ny = passes;
  if (static_cast<long long>(tokens) * passes > 148 * 4) ny = (passes + 3) / 4;
  switch ((a.H + kGroups * ny - 1) / (kGroups * ny)) {
    case 1: return launch_r<D, 1>(a, tokens, ny, s);
    case 2: return launch_r<D, 2>(a, tokens, ny, s);
    case 3: return launch_r<D, 3>(a, tokens, ny, s);
    default: return launch_r<D, 4>(a, tokens, ny, s);
  }
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
  const unsigned tokens = static_cast<unsigned>(B) * static_cast<unsigned>(N);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64)
    launch_d<64>(a, tokens, s);
  else
    launch_d<128>(a, tokens, s);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
