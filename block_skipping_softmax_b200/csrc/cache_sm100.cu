// Writing a paged KV cache as e4m3 codes, and reading it back as bf16.
//
// A key vector x of one head (d elements) is quantised by itself, as it is
// written: s = 2^k, k the smallest integer >= -126 with max|x| <= 448 * 2^k, and
// code = e4m3(x / s), rounded to nearest, ties to even.  That is the rule of
// attn_quantize_e4m3 with the vector as the group: a longer group would have
// to be quantised again whenever a later key is larger.  With s a power of two
// x / s and code * s are exact, so reading back is exact in bf16, and the
// attention over the codes is attention over the values read back.
//
// Both directions are bound by HBM (a token's heads: 4 d bytes of bf16 and
// 2 (d + 4) of codes and scales).  A vector is held by D/8 lanes, 16 bytes of
// bf16 and 8 of codes each, so every access is a full 128-byte line or two for
// each vector; a group of lanes takes up to four vectors, all loaded before the
// first is reduced.  What held it back beside HBM was the issue of instructions,
// so the lanes share what a vector costs once (see Row), and maxima are taken
// two to a word: 4 prompts of 4099 tokens x 8 heads of 128 are written in 18.9 us
// (5.4 TB/s; 19.6 by CTAs of 256 threads, 20.5 of 512; 27.4 when every lane found
// its vectors and reduced in fp32), and 2 x 32768 tokens read back in 71 us (5.7
// TB/s; 88 before), of 6.55 TB/s for a copy.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace bss {

namespace {

constexpr int kThreads = 128;
constexpr int kPage = kDecodeTile;  // keys of a page
constexpr unsigned kFull = 0xffffffffu;

struct CacheArgs {
  const void* x[2];  // k, v (bf16; written by the read)
  uint8_t* codes[2];
  float* scales[2];
  const long long* slots;
  long long xs[2][3];  // strides in elements: batch, token, head
  long long n_slots;   // num_pages * 64
  int B, N, Hkv;
};

// A CTA takes neighbouring tokens of one head's keys or values, which are
// neighbours in [B, H, N, d] and in a page; the CTAs of a token's other heads
// run beside it, which are neighbours in a packed [tokens, H, d].
// Finding a vector costs a dozen 64-bit operations, so lane c of a group finds
// vector c % R for the others, and reads or writes its scale.
struct Row {
  uint64_t x;    // address of the vector's first element in k or v, 0 past the last token
  long long at;  // vector index in codes and scales, -1 where the token has no slot
};

__device__ __forceinline__ Row row_of(const CacheArgs& a, unsigned t, int side, int h) {
  Row w{0, -1};
  if (t < static_cast<unsigned>(a.B) * static_cast<unsigned>(a.N)) {  // B * N < 2^31
    const unsigned b = a.B == 1 ? 0 : t / a.N, n = t - b * a.N;
    const long long slot = a.slots[t];
    const long long e = side ? b * a.xs[1][0] + n * a.xs[1][1] + h * a.xs[1][2]
                             : b * a.xs[0][0] + n * a.xs[0][1] + h * a.xs[0][2];
    w.x = reinterpret_cast<uint64_t>(side ? a.x[1] : a.x[0]) + 2 * e;
    if (slot >= 0 && slot < a.n_slots) w.at = ((slot / kPage) * a.Hkv + h) * kPage + slot % kPage;
  }
  return w;
}

template <int kLanes>
__device__ __forceinline__ Row row_from(const Row& own, int r) {
  return {__shfl_sync(kFull, own.x, r, kLanes), __shfl_sync(kFull, own.at, r, kLanes)};
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
  uint32_t m;  // a NaN stays
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(x), "r"(y));
  return m;
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  const int group = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const unsigned block = blockIdx.x / (2u * a.Hkv), head = blockIdx.x - block * (2u * a.Hkv);
  const int side = head >= static_cast<unsigned>(a.Hkv), h = side ? head - a.Hkv : head;
  uint8_t* codes = side ? a.codes[1] : a.codes[0];
  float* scales = side ? a.scales[1] : a.scales[0];
  const Row own = row_of(a, (block * R + c % R) * kGroups + group, side, h);
  long long at[R];
  uint4 u[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const Row w = row_from<kLanes>(own, r);
    at[r] = w.at;
    u[r] = make_uint4(0, 0, 0, 0);
    if (at[r] >= 0) u[r] = reinterpret_cast<const uint4*>(w.x)[c];
  }
  // max |x| of vector c % R: within the lane, then over the lanes; with four
  // vectors a word carries two of them, and a lane ends with the pair of its own
  uint32_t m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    m[r] = max_bf16x2(max_bf16x2(u[r].x & kAbs, u[r].y & kAbs), max_bf16x2(u[r].z & kAbs, u[r].w & kAbs));
  }
  uint32_t top;
  if constexpr (R == 4) {
    const uint32_t p = max_bf16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
    const uint32_t q = max_bf16x2(__byte_perm(m[2], m[3], 0x5410), __byte_perm(m[2], m[3], 0x7632));
    top = max_bf16x2(c & 2 ? q : p, __shfl_xor_sync(kFull, c & 2 ? p : q, 2));
    top = max_bf16x2(top, __shfl_xor_sync(kFull, top, 1));
  } else {
    static_assert(R == 1, "one or four vectors");
    top = max_bf16x2(m[0], __byte_perm(m[0], m[0], 0x1032));
    top = max_bf16x2(top, __shfl_xor_sync(kFull, top, 1));
    top = max_bf16x2(top, __shfl_xor_sync(kFull, top, 2));
  }
#pragma unroll
  for (int o = 4; o < kLanes; o <<= 1) top = max_bf16x2(top, __shfl_xor_sync(kFull, top, o));
  const uint32_t mx = R == 4 && !(c & 1) ? top << 16 : top & 0xffff0000u;  // as float bits
  // mx = f 2^e with f in [1, 2); 448 = 1.75 * 2^8.  max|x| <= 448 * 2^k holds
  // first at k = e - 8 when f <= 1.75, else at e - 7.  A subnormal mx (e field
  // 0) lies below 448 * 2^-126, the least scale.  1/s is then exact too:
  // |k| <= 126.
  int k = static_cast<int>(mx >> 23) - 127 - 8 + ((mx & 0x7fffffu) > 0x600000u ? 1 : 0);
  k = max(k, -126);
  float s = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
  float inv = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  if (mx == 0) s = inv = 1.f;
  if (mx >= 0x7f800000u) s = inv = __uint_as_float(0x7fc00000u);  // inf or NaN in the vector
  if (c < R && own.at >= 0) scales[own.at] = s;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float f = __shfl_sync(kFull, inv, r, kLanes);
    const uint32_t w[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint16_t lo, hi;  // cvt packs its first source into the upper byte
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(lo)
          : "f"(__uint_as_float(w[2 * i] & 0xffff0000u) * f), "f"(__uint_as_float(w[2 * i] << 16) * f));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(hi)
          : "f"(__uint_as_float(w[2 * i + 1] & 0xffff0000u) * f), "f"(__uint_as_float(w[2 * i + 1] << 16) * f));
      out[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
    }
    if (at[r] >= 0) *reinterpret_cast<uint2*>(codes + at[r] * D + c * 8) = make_uint2(out[0], out[1]);
  }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheArgs a) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  const int group = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
  const unsigned block = blockIdx.x / (2u * a.Hkv), head = blockIdx.x - block * (2u * a.Hkv);
  const int side = head >= static_cast<unsigned>(a.Hkv), h = side ? head - a.Hkv : head;
  const uint8_t* codes = side ? a.codes[1] : a.codes[0];
  const float* scales = side ? a.scales[1] : a.scales[0];
  const Row own = row_of(a, (block * R + c % R) * kGroups + group, side, h);
  const float s = own.at >= 0 ? scales[own.at] : 0.f;
  uint64_t x[R];
  uint2 u[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const Row w = row_from<kLanes>(own, r);
    x[r] = w.x;
    u[r] = make_uint2(0, 0);
    if (w.at >= 0) u[r] = *reinterpret_cast<const uint2*>(codes + w.at * D + c * 8);
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float f = __shfl_sync(kFull, s, r, kLanes);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t pair = (i & 1) ? (i < 2 ? u[r].x : u[r].y) >> 16 : (i < 2 ? u[r].x : u[r].y);
      uint32_t h2;  // two halves: every e4m3 value is exact in fp16
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(pair)));
      const __half2 h = *reinterpret_cast<const __half2*>(&h2);
      out[i] = pack_bf16x2(__low2float(h) * f, __high2float(h) * f);
    }
    if (x[r]) reinterpret_cast<uint4*>(x[r])[c] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <int D, bool WRITE, int R>
int launch_r(const CacheArgs& a, cudaStream_t s) {
  constexpr int kGroups = kThreads / (D / 8);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long grid = (tokens + kGroups * R - 1) / (kGroups * R) * 2 * a.Hkv;
  if (grid > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if constexpr (WRITE)
    cache_write_kernel<D, R><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  else
    cache_read_kernel<D, R><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Vectors of a group: one where the launch fits the 148 SMs at once, else four.
// (65536 tokens read back: 120 us by ones, 71 by fours; 4 x 4099 written: 32 and
// 19; 16 tokens of 8 heads of 128 written: 2.0 us by ones, 2.2 by fours.)
template <int D, bool WRITE>
int launch_d(const CacheArgs& a, cudaStream_t s) {
  constexpr int kGroups = kThreads / (D / 8);
  const long long rows = static_cast<long long>(a.B) * a.N * 2 * a.Hkv;
  if (rows <= 148LL * 4 * kGroups) return launch_r<D, WRITE, 1>(a, s);
  return launch_r<D, WRITE, 4>(a, s);
}

int run(const void* k, const void* v, const int64_t* slots, const void* K_codes,
        const void* V_codes, const float* K_scales, const float* V_scales, int B, int N, int Hkv,
        int num_pages, int d, const long long* strides, void* stream, bool write) {
  if (!k || !v || !slots || !K_codes || !V_codes || !K_scales || !V_scales || !strides)
    return ATTN_ERR_INVALID_ARG;
  if (!ptr_aligned(k, 16) || !ptr_aligned(v, 16) || !ptr_aligned(K_codes, 16) ||
      !ptr_aligned(V_codes, 16) || !ptr_aligned(K_scales, 16) || !ptr_aligned(V_scales, 16) ||
      !ptr_aligned(slots, 8))
    return ATTN_ERR_INVALID_ARG;
  if (B <= 0 || N <= 0 || Hkv <= 0 || num_pages <= 0 || (d != 64 && d != 128))
    return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i)
    if (strides[i] % 8 != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > 0x7fffffffLL || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  int dev = 0;
  int* status = nullptr;
  const int st = device_context(&dev, &status);
  if (st != ATTN_OK) return st;
  CacheArgs a{};
  a.x[0] = k;
  a.x[1] = v;
  a.codes[0] = static_cast<uint8_t*>(const_cast<void*>(K_codes));
  a.codes[1] = static_cast<uint8_t*>(const_cast<void*>(V_codes));
  a.scales[0] = const_cast<float*>(K_scales);
  a.scales[1] = const_cast<float*>(V_scales);
  a.slots = reinterpret_cast<const long long*>(slots);
  for (int t = 0; t < 2; ++t)
    for (int i = 0; i < 3; ++i) a.xs[t][i] = strides[3 * t + i];
  a.B = B;
  a.n_slots = static_cast<long long>(num_pages) * kPage;
  a.N = N;
  a.Hkv = Hkv;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 64) return write ? launch_d<64, true>(a, s) : launch_d<64, false>(a, s);
  return write ? launch_d<128, true>(a, s) : launch_d<128, false>(a, s);
}

}  // namespace

}  // namespace bss

extern "C" {

int attn_cache_write_e4m3(const void* k, const void* v, const int64_t* slots, void* K_codes,
                          void* V_codes, float* K_scales, float* V_scales, int B, int N, int Hkv,
                          int num_pages, int d, const long long* strides, void* stream) {
  return bss::run(k, v, slots, K_codes, V_codes, K_scales, V_scales, B, N, Hkv, num_pages, d,
                  strides, stream, true);
}

int attn_cache_read_e4m3(const void* K_codes, const void* V_codes, const float* K_scales,
                         const float* V_scales, const int64_t* slots, void* k, void* v, int B,
                         int N, int Hkv, int num_pages, int d, const long long* strides,
                         void* stream) {
  return bss::run(k, v, slots, K_codes, V_codes, K_scales, V_scales, B, N, Hkv, num_pages, d,
                  strides, stream, false);
}

}  // extern "C"
