// Tree attention for many rows a KV head: 128 rows a CTA on tcgen05.
//
//   warp 0       finds the CTA's segments and passes them on to the others
//   warp 1       bf16 pool: checks the V tiles that hold drafted keys
//   warp 2       copies: K and V pages, a ring in shared memory
//   warp 3       TMEM, and the one thread that issues the MMAs:
//                  S_j = Q K_j^T (two buffers), O += P_j V_j (P read from TMEM)
//   warps 4-7    softmax: a thread owns the row of TMEM lane 32 (warp % 4) + lane
//   warps 8-15   e4m3: 8-11 turn codes of K into an fp16 operand, 12-15 codes of
//                V into an fp16 (rarely bf16) one; the registers are divided
//                anew between the roles
//
// (The issuer and the copies are not on the schedulers of softmax warps 4 and 5,
// which are the busy ones with up to 64 rows.)
//
// A tile is one page of 64 keys, so that TMEM holds O and two S in 256 columns
// and two CTAs share an SM: one's softmax runs beside the other's MMAs.  Every
// role runs through the CTA's segments by itself; the ring, the MMAs and the
// conversion go on across their borders.  Rows past the last one are zero
// queries, and softmax warps without a row only keep step.
//
// Measured, 16 sequences x 16384 keys, 8 KV heads, with 32 / 64 / 128 rows a head:
//   bf16 of 128  171 / 176 / 196 us   of 64  100 / 116 / 141
//   e4m3 of 128  189 / 198 / 226      of 64  137 / 161 / 190
// bf16 of 128 is bound by HBM up to 64 rows (6.1 TB/s and more).  With 512 rows a head
// (64 tokens x 64 heads over 4 x 16384 keys: 158 us, 12 of them the merge; 190 to 205
// a pass under a load of seconds, which the power limit slows; heads of 64 140) the
// tensor pipe, the ex2 unit and the issue slots are each busy for 46 to 49% of the
// time: what counts is the latency of S, softmax and P, with two warps a scheduler
// to hide it.  Heads of 64 have half the bytes and MMAs behind the same chain, so it
// shows from 64 rows on (4.7 TB/s; tensor pipe and ex2 unit 30% busy, issue slots 37%).
// e4m3 adds the latency of the conversion, and more warps to the same schedulers, and
// is slower than bf16 at all of these (512 rows: 226 us, of 64 191): its cache is half
// the size, but here that is all it gains.  Its 64 registers a thread at launch cost 128
// bytes of spills (heads of 64: 120).  A segment's change costs 7 us: 3 for O, 3 for Q,
// 1 for the first S; writing Q ahead of O gained nothing.  Slower: codes of K straight
// into 8-bit MMAs, the query as two e4m3 terms (230 us against 210 then, with 64 rows);
// two softmax warps to a row, half the keys each (bf16 219 against 206 with 128 rows,
// 145 against 123 for heads of 64 with 64).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attn.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "tree.cuh"

namespace bss {

namespace {

constexpr int kRows = kManyRows;
constexpr int kSegs = 4;    // segments on their way from warp 0 to the others
constexpr int kChecks = 4;  // tiles with drafted keys on their way: see Tails

template <int D, bool E4M3>
struct Cfg {
  static constexpr int kPrep = E4M3 ? 4 : 1;  // warps that convert K, convert V or check V tiles
  static constexpr int kPrepWarp = E4M3 ? 8 : 1;
  static constexpr int kReaders = E4M3 ? 14 : 7;  // warps that follow the segments
  static constexpr int kThreads = E4M3 ? 512 : 256;
  // Registers a thread, e4m3: 64 at launch, then by warpgroup (copies and MMAs,
  // softmax, tiles, tiles), 256 in all.
  static constexpr int kRegs = 64, kRegsIssue = 40, kRegsSoftmax = 104, kRegsPrep = 56;
  static constexpr int kQPanel = kRows * 128;
  static constexpr int kTile = kPage * D * 2;  // K or V of a page as 16-bit values
  static constexpr int kTilePanel = kPage * 128;
  static constexpr int kRaw = kPage * D;       // as codes
  static constexpr int kRing = E4M3 ? (D == 128 ? 5 : 8) : (D == 128 ? 4 : 6);  // tiles in flight
  static constexpr int kSlot = E4M3 ? kRaw : kTile;
  static constexpr int kOffQ = 0;
  static constexpr int kOperands = D == 64 ? 2 : 1;                // e4m3: buffers of each operand
  static constexpr int kOffConv = kOffQ + kRows * D * 2;           // e4m3: K and V operands
  static constexpr int kOffRing = kOffConv + (E4M3 ? 2 * kOperands * kTile : 0);
  static constexpr int kScaleBytes = E4M3 ? 2 * kPage * 4 : 0;    // K, V
  static constexpr int kOffScale = kOffRing + kRing * kSlot;       // e4m3: [slot][K, V][64] floats
  static constexpr int kOffKScale = kOffScale + kRing * kScaleBytes;  // e4m3: [4][64], for softmax
  static constexpr int kOffBar = kOffKScale + (E4M3 ? 4 * kPage * 4 : 0);
  // full[ring], empty[ring], q_full, s_full[2], p_full[2], pv_done, o_final,
  // checked[4]; bf16: drafted[4]; e4m3: ready[K, V][buffers], free[K, V][buffers];
  // segment full[4], segment empty[4]
  static constexpr int kBars = 2 * kRing + 7 + 3 * kChecks + 2 * kSegs;
  static constexpr int kOffMisc = kOffBar + kBars * 8;
  static constexpr int kMiscBytes = 432;
  static constexpr int kSmem = kOffMisc + kMiscBytes + 1024;
  static constexpr int kTmemCols = 256;
  static_assert(D + 2 * kPage <= kTmemCols, "O and two S");
};

struct Misc {
  unsigned long long bad[kChecks][4];  // by tile warp: drafted keys of a tile whose value is not finite
  uint32_t tmem_base;
  int abort;
  int bad_page[8];  // e4m3: the slot's page id was out of range
  int segs[kSegs][12];
  int plain[4][2];  // e4m3, by tile: whether the scales of keys 0-31, 32-63 fit fp16 operands
};

// kind::f16 with fp16 A and B (format 0), fp32 accumulation, A K-major
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The ring's sequence within a segment of nt tiles is the order of use:
// K_0, K_1, V_0, K_2, V_1, ..., V_last.
__device__ __forceinline__ int item_k(int tile) { return tile == 0 ? 0 : 2 * tile - 1; }
__device__ __forceinline__ int item_v(int tile, int nt) { return tile == nt - 1 ? 2 * nt - 1 : 2 * tile + 2; }
__device__ __forceinline__ bool item_is_v(int i, int nt, int& tile) {
  if (i == 2 * nt - 1) {
    tile = nt - 1;
    return true;
  }
  const bool v = i >= 2 && (i & 1) == 0;
  tile = v ? i / 2 - 1 : (i + 1) / 2;
  return v;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(Cfg<D, E4M3>::kThreads, 2)
    tree_many_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeLaunch a) {
  using C = Cfg<D, E4M3>;
  static_assert(sizeof(Misc) <= C::kMiscBytes && C::kRing <= 8 && C::kPrep <= 4, "misc layout");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  Misc* misc = reinterpret_cast<Misc*>(smem + C::kOffMisc);
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
  // V tile number c with drafted keys (over the CTA's segments) is checked; bf16: has landed
  auto b_checked = [&](int c) { return bar1 + 8u * (7 + c % kChecks); };
  auto b_drafted = [&](int c) { return bar1 + 8u * (7 + kChecks + c % kChecks); };
  // e4m3: K (0) or V (1) of tile n is converted, its MMAs are done
  auto b_ready = [&](int v, int n) { return bar1 + 8u * (7 + kChecks + 2 * v + n % C::kOperands); };
  auto b_free = [&](int v, int n) { return bar1 + 8u * (11 + kChecks + 2 * v + n % C::kOperands); };

  asm volatile("griddepcontrol.launch_dependents;");  // the merge may look for its shares
  auto b_seg_full = [&](int i) { return bar1 + 8u * (7 + 3 * kChecks + i % kSegs); };
  auto b_seg_empty = [&](int i) { return bar1 + 8u * (7 + 3 * kChecks + kSegs + i % kSegs); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kRing; ++s) {
      mbar_init(b_full(s), 1);
      mbar_init(b_empty(s), E4M3 ? C::kPrep : 1);
    }
    mbar_init(b_q_full, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(b_s_full(i), 1);
      mbar_init(b_p_full(i), 4);
      if constexpr (E4M3) {
        for (int n = 0; n < C::kOperands; ++n) {
          mbar_init(b_ready(i, n), C::kPrep);
          mbar_init(b_free(i, n), 1);
        }
      }
    }
    for (int i = 0; i < kChecks; ++i) {
      mbar_init(b_checked(i), C::kPrep);
      if constexpr (!E4M3) mbar_init(b_drafted(i), 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(b_seg_full(i), 1);
      mbar_init(b_seg_empty(i), C::kReaders);
    }
    mbar_init(b_pv_done, 1);
    mbar_init(b_o_final, 1);
    misc->abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(&misc->tmem_base), C::kTmemCols);
    tmem_relinquish();
  }
  Segments list;
  if (warp == 0) list.start(a, kRows);
  Segment sg{};
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tO = misc->tmem_base;
  auto tS = [&](int i) { return tO + D + i * kPage; };
  auto give_up = [&](int site) {
    *abort_flag = 1;
    atomicCAS(a.status, 0, ATTN_DEVICE_TIMEOUT_BASE + site);
  };
  // e4m3: K and V of tile n are fp16 operands with their scales in them (known
  // once K of tile n is ready).  Else K holds the codes alone, whose scales
  // softmax applies, and V and P are bf16.
  auto plain_tile = [&](int n) {
    const volatile int* f = misc->plain[n & 3];
    return (f[0] & f[1]) != 0;
  };
  // Tiles from tail0 on hold drafted keys or end past the last key; there are at
  // most two in a segment.  They are numbered over the CTA's segments.
  auto tail0 = [&] { return max(sg.s.prefix / kPage - sg.t0, 0); };
  auto tails = [&] { return max(sg.nt - tail0(), 0); };

  // ------------------------------------------------ segments
  auto segments = [&] {
    bool more = true;
    for (int i = 0; more; ++i) {
      more = list.next(a, kRows, sg);
      if (i >= kSegs && !__all_sync(kFull, mbar_poll(b_seg_empty(i), (i / kSegs - 1) & 1, abort_flag,
                                                     a.wait_limit_ns))) {
        if (lane == 0) give_up(50);
        break;
      }
      if (lane == 0) {
        volatile int* p = misc->segs[i % kSegs];
        p[0] = more ? sg.nt : -1;
        p[1] = sg.b;
        p[2] = sg.kv;
        p[3] = sg.t0;
        p[4] = sg.rows;
        p[5] = sg.whole ? 1 : 0;
        p[6] = sg.place;
        p[7] = sg.s.tok0;
        p[8] = sg.s.len;
        p[9] = sg.s.prefix;
        mbar_arrive(b_seg_full(i));
      }
    }
  };
  auto next_segment = [&](int i) {
    if (!__all_sync(kFull, mbar_poll(b_seg_full(i), (i / kSegs) & 1, abort_flag, a.wait_limit_ns))) {
      if (lane == 0) give_up(51);
      return false;
    }
    const volatile int* p = misc->segs[i % kSegs];
    sg.nt = p[0];
    sg.b = p[1];
    sg.kv = p[2];
    sg.t0 = p[3];
    sg.rows = p[4];
    sg.whole = p[5] != 0;
    sg.place = p[6];
    sg.s.tok0 = p[7];
    sg.s.len = p[8];
    sg.s.prefix = p[9];
    sg.row0 = blockIdx.y * kRows;
    __syncwarp();
    if (lane == 0) mbar_arrive(b_seg_empty(i));
    return sg.nt >= 0;
  };

  // ------------------------------------------------ copies
  auto copies = [&] {
    int issued = 0, checks = 0, landed = 0;  // items, drafted tiles, drafted tiles issued
    bool ok = true;
    for (int seg = 0; ok && next_segment(seg); ++seg) {
      const int* table = a.block_table + static_cast<size_t>(sg.b) * a.max_pages + sg.t0;
      int pages_k = 0, pages_v = 0;  // lane i: the page of tile i + 32 n, for the K and the V stream
      const int first_tail = tail0();
      for (int i = 0; i < 2 * sg.nt && ok; ++i) {
        int tile;
        const bool is_v = item_is_v(i, sg.nt, tile);
        if ((tile & 31) == 0) {
          const int p = tile + lane < sg.nt ? table[tile + lane] : -1;
          if (is_v)
            pages_v = p;
          else
            pages_k = p;
        }
        const int page = __shfl_sync(kFull, is_v ? pages_v : pages_k, tile & 31);
        const int s = issued % C::kRing;
        if (lane == 0) {
          if (issued >= C::kRing)
            ok = mbar_poll(b_empty(s), ((issued / C::kRing) - 1) & 1, abort_flag, a.wait_limit_ns);
          if (ok) {
            const bool good = page >= 0 && page < a.num_pages;
            const long long grp = static_cast<long long>(good ? page : a.num_pages) * a.Hkv + sg.kv;
            const uint32_t dst = sbase + C::kOffRing + s * C::kSlot;
            // a page id out of range reads zeros: the box lies past the pool's end
            if constexpr (E4M3) {
              misc->bad_page[s] = good ? 0 : 1;
              mbar_arrive_expect_tx(b_full(s), C::kRaw + (good ? C::kScaleBytes : 0));
              tma_load_3d(dst, is_v ? &tmV : &tmK, b_full(s), 0, 0, static_cast<int>(grp));
              if (good) {
                // both with both, for the choice of the operands' type
                const uint32_t to = sbase + C::kOffScale + s * C::kScaleBytes;
                bulk_load(to, a.k_scales + grp * kPage, kPage * 4, b_full(s));
                bulk_load(to + kPage * 4, a.v_scales + grp * kPage, kPage * 4, b_full(s));
              }
            } else {
              uint32_t bar = b_full(s);
              if (is_v && tile >= first_tail) {  // the MMA issuer waits for the check instead
                landed = checks + tile - first_tail + 1;
                bar = b_drafted(landed - 1);
                mbar_arrive(b_full(s));
              }
              mbar_arrive_expect_tx(bar, C::kTile);
#pragma unroll
              for (int p = 0; p < D / 64; ++p)
                tma_load_3d(dst + p * C::kTilePanel, is_v ? &tmV : &tmK, bar, p * 64, 0, static_cast<int>(grp));
            }
          }
        }
        ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
        if (ok) ++issued;
      }
      checks += tails();
    }
    if (lane == 0) {
      if (!ok) give_up(40);
      // no copy in flight at the end
      for (int i = max(0, issued - C::kRing); i < issued; ++i)
        mbar_drain(b_full(i % C::kRing), (i / C::kRing) & 1, a.wait_limit_ns);
      for (int c = max(0, landed - kChecks); !E4M3 && c < landed; ++c)
        mbar_drain(b_drafted(c), (c / kChecks) & 1, a.wait_limit_ns);
    }
  };
  // ------------------------------------------------ MMA issuer
  auto issue = [&] {
    constexpr uint32_t idS = E4M3 ? idesc_f16_f32(kRows, kPage, false) : idesc_bf16_f32(kRows, kPage, false, false);
    constexpr uint32_t idPV = idesc_bf16_f32(kRows, D, false, true), idPV16 = idesc_f16_f32(kRows, D, true);
    auto wait = [&](uint32_t bar, int parity, int site) {
      if (mbar_poll(bar, parity, abort_flag, a.wait_limit_ns)) return true;
      give_up(site);
      return false;
    };
    int slot = 0, phase = 0;  // bf16: the ring's items are used in its order
    // descriptors: the high words are constants, an MMA adds offsets to the low ones
    constexpr uint32_t hi = sw128_desc_hi(1024);
    const uint32_t dQ = sw128_desc_lo(sbase + C::kOffQ, 16);
    const uint32_t dK = sw128_desc_lo(sbase + (E4M3 ? C::kOffConv : C::kOffRing), 16);
    const uint32_t dV = sw128_desc_lo(sbase + (E4M3 ? C::kOffConv + C::kOperands * C::kTile : C::kOffRing), C::kTilePanel);
    auto buffer = [&](int n) { return (E4M3 ? n % C::kOperands : slot) * ((E4M3 ? C::kTile : C::kSlot) >> 4); };
    bool ok = true;
    int seg = 0, n0 = 0, checks = 0;  // segments, tiles and drafted tiles before this one
    while (ok && next_segment(seg)) {
      if (lane == 0) {
        const int nt = sg.nt, first_tail = tail0();
        ok = wait(b_q_full, seg & 1, 41);
        for (int j = 0; ok && nt > 0 && j <= nt; ++j) {
          if (j < nt) {
            const int n = n0 + j;
            const uint32_t at = dK + buffer(n);
            if (!(ok = E4M3 ? wait(b_ready(0, n), (n / C::kOperands) & 1, 42) : wait(b_full(slot), phase, 42))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              constexpr int kStep = 32 >> 4;  // 16 values = 32 B inside a 128 B row
              mma_ss(tS(n & 1), desc_join(dQ + (kk >> 2) * (C::kQPanel >> 4) + (kk & 3) * kStep, hi),
                     desc_join(at + (kk >> 2) * (C::kTilePanel >> 4) + (kk & 3) * kStep, hi), idS, kk > 0 ? 1u : 0u);
            }
            mma_commit(b_s_full(n & 1));
            mma_commit(E4M3 ? b_free(0, n) : b_empty(slot));
            if (++slot == C::kRing) slot = 0, phase ^= 1;
          }
          if (j >= 1) {
            const int t = j - 1, n = n0 + t;
            const uint32_t at = dV + buffer(n);
            if (!(ok = E4M3 ? wait(b_ready(1, n), (n / C::kOperands) & 1, 43) : wait(b_full(slot), phase, 43))) break;
            if (!E4M3 && t >= first_tail) {
              const int c = checks + t - first_tail;
              if (!(ok = wait(b_checked(c), (c / kChecks) & 1, 44))) break;
            }
            if (!(ok = wait(b_p_full(n & 1), (n >> 1) & 1, 45))) break;
            tc_fence_after();
            const uint32_t id = E4M3 && plain_tile(n) ? idPV16 : idPV;
#pragma unroll
            for (int kk = 0; kk < kPage / 16; ++kk)
              mma_ts(tO, tS(n & 1) + kk * 8, desc_join(at + kk * (16 * 128 >> 4), hi), id, (t > 0 || kk > 0) ? 1u : 0u);
            mma_commit(E4M3 ? b_free(1, n) : b_empty(slot));
            mma_commit(b_pv_done);
            if (++slot == C::kRing) slot = 0, phase ^= 1;
          }
        }
        mma_commit(b_o_final);
      }
      ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
      n0 += sg.nt;
      checks += tails();
      ++seg;
    }
    if (lane == 0 && seg > 0) mbar_drain(b_o_final, (seg - 1) & 1, a.wait_limit_ns);  // before TMEM is released
  };
  // ------------------------------------------------ softmax
  auto softmax = [&] {
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    bool ok = true;
    int seg = 0, n0 = 0, checks = 0;
    while (ok && next_segment(seg)) {
      const bool valid = r < sg.rows;
      const bool active = (warp & 3) * 32 < sg.rows;  // some row of the warp
      int tok = 0;
      const size_t at = valid ? row_at(a, sg, r, &tok) : 0;
      float mul = a.scale_log2;
      {  // this row of Q into the swizzled operand; the last segment's MMAs are done with it
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at * D);
        float f = 1.f;
        if constexpr (E4M3) {
          uint32_t amax = 0;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 u = valid ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) amax = max(amax, max((w[e] << 16) & 0x7fffffffu, w[e] & 0x7fff0000u));
          }
          const int shift = f16_shift(amax);
          f = pow2(shift);
          mul *= pow2(-shift);
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint4 u = valid ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          uint32_t w[4] = {u.x, u.y, u.z, u.w};
          if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_f16x2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
          }
          sts128(sbase + C::kOffQ + (c >> 3) * C::kQPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4), w[0], w[1], w[2],
                 w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_q_full);
      }
      const uint64_t bits = valid ? bits_of(a, sg.s, tok) : 0;
      const int first_tail = tail0();
      float m_ref = neg_inf(), l_sum = 0.f;
      for (int j = 0; j < sg.nt; ++j) {
        const int n = n0 + j, sb = n & 1;
        if (!__all_sync(kFull, mbar_poll(b_s_full(sb), (n >> 1) & 1, abort_flag, a.wait_limit_ns))) {
          if (lane == 0) give_up(46);
          ok = false;
          break;
        }
        if (!active) {
          if (lane == 0) mbar_arrive(b_p_full(sb));
          continue;
        }
        tc_fence_after();
        // which of the 64 keys this row sees, and which of their values are not finite
        uint64_t sees = ~0ull, bad = 0;
        if (j >= first_tail) {
          const int key0 = (sg.t0 + j) * kPage;
          const int n_prefix = min(max(sg.s.prefix - key0, 0), kPage), n_len = min(sg.s.len - key0, kPage);
          sees = n_prefix >= 64 ? ~0ull : (1ull << n_prefix) - 1;
          const int first = key0 - sg.s.prefix;  // drafted index of the tile's first key
          sees |= first >= 64 ? 0 : first >= 0 ? bits >> first : first > -64 ? bits << -first : 0;
          if (n_len < 64) sees &= (1ull << n_len) - 1;
          const int c = checks + j - first_tail;
          if (!__all_sync(kFull, mbar_poll(b_checked(c), (c / kChecks) & 1, abort_flag, a.wait_limit_ns))) {
            if (lane == 0) give_up(47);
            ok = false;
            break;
          }
#pragma unroll
          for (int w = 0; w < C::kPrep; ++w)
            bad |= *reinterpret_cast<volatile unsigned long long*>(&misc->bad[c % kChecks][w]);
          bad &= sees;
        }
        const bool plain = !E4M3 || plain_tile(n);
        // the tile's maximum to the running reference; moves O along, and gives
        // the value that the exponents are relative to
        float alpha = 1.f, from = 0.f, rs = 0.f;
        auto refer = [&](float mt) {
          const bool moved = (mt - m_ref) * mul > kRefSlack;  // NaN where nothing has been seen still
          if (moved) {
            alpha = ex2((m_ref - mt) * mul);  // m_ref = -inf gives 0
            m_ref = mt;
          }
          from = minus(m_ref);
          if (__any_sync(kFull, moved && j > 0)) {
            // O is read and written back: the last P V must have finished
            if (!__all_sync(kFull, mbar_poll(b_pv_done, (n - 1) & 1, abort_flag, a.wait_limit_ns))) {
              if (lane == 0) give_up(48);
              return false;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
              uint32_t o[16];
              tmem_ld16(tO + lane_off + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
              tmem_st16(tO + lane_off + c0, o);
            }
          }
          return true;
        };
        // P = 2^((s - ref) scale), the difference first, which keeps its bits at any
        // size of the scores: as bf16, the sum adding the rounded
        // values; as fp16, whose rounding (2^-12) is below what cancels there
        if (plain) {
          uint32_t x[kPage];
          tmem_ld_row<kPage>(tS(sb) + lane_off, x);
          tmem_wait_ld();
          if (j >= first_tail) {
#pragma unroll
            for (int c = 0; c < kPage; ++c)
              if (!((sees >> c) & 1)) x[c] = 0xff800000u;
          }
          float mt[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
          for (int c = 0; c < kPage; c += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mt[e] = fmax3(mt[e], __uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
          if (!(ok = refer(fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3]))))) break;
          const float2 from2 = make_float2(from, from), mul2 = make_float2(mul, mul);
          float2 sum2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int c0 = 0; c0 < kPage; c0 += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 y = log2_p<E4M3>(
                  make_float2(__uint_as_float(x[c0 + 2 * c]), __uint_as_float(x[c0 + 2 * c + 1])), from2, mul2);
              const float p0 = ex2(y.x), p1 = ex2(y.y);
              if constexpr (E4M3) {
                pk[c] = pack_f16x2(p0, p1);
                sum2 = __fadd2_rn(sum2, make_float2(p0, p1));
              } else {
                pk[c] = pack_bf16x2(p0, p1);
                sum2 = __fadd2_rn(sum2, make_float2(__uint_as_float(pk[c] << 16), __uint_as_float(pk[c] & 0xffff0000u)));
              }
            }
            tmem_st16(tS(sb) + lane_off + c0 / 2, pk);
          }
          rs = sum2.x + sum2.y;
        } else {  // an unusual e4m3 tile: 16 columns at a time, with their scales and mask
          auto scaled16 = [&](int c0, uint32_t (&y)[16]) {
            tmem_ld16(tS(sb) + lane_off + c0, y);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float ks = lds_f32(sbase + C::kOffKScale + ((n & 3) * kPage + c0 + c) * 4);
              y[c] = __float_as_uint(__uint_as_float(y[c]) * ks);
              if (!((sees >> (c0 + c)) & 1)) y[c] = 0xff800000u;
            }
          };
          float mt = neg_inf();
#pragma unroll 1
          for (int c0 = 0; c0 < kPage; c0 += 16) {
            uint32_t y[16];
            scaled16(c0, y);
#pragma unroll
            for (int c = 0; c < 16; ++c) mt = fmaxf(mt, __uint_as_float(y[c]));
          }
          if (!(ok = refer(mt))) break;
#pragma unroll 1
          for (int c0 = 0; c0 < kPage; c0 += 16) {
            uint32_t y[16], pk[8];
            scaled16(c0, y);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const float2 z = log2_p<E4M3>(make_float2(__uint_as_float(y[2 * c]), __uint_as_float(y[2 * c + 1])),
                                            make_float2(from, from), make_float2(mul, mul));
              pk[c] = pack_bf16x2(ex2(z.x), ex2(z.y));
              rs += __uint_as_float(pk[c] << 16) + __uint_as_float(pk[c] & 0xffff0000u);
            }
            tmem_st8(tS(sb) + lane_off + c0 / 2, pk);
          }
        }
        if (__any_sync(kFull, bad != 0)) {  // a value was taken out of V: NaN for whoever sees it
          tmem_wait_st();
#pragma unroll 1
          for (int c0 = 0; c0 < kPage / 2; c0 += 16) {
            uint32_t y[16];
            tmem_ld16(tS(sb) + lane_off + c0, y);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              if ((bad >> (2 * (c0 + c))) & 1) y[c] = (y[c] & 0xffff0000u) | 0x7fc0u;
              if ((bad >> (2 * (c0 + c) + 1)) & 1) y[c] = (y[c] & 0xffffu) | 0x7fc00000u;
            }
            tmem_st16(tS(sb) + lane_off + c0, y);
          }
        }
        l_sum = l_sum * alpha + rs;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(b_p_full(sb));
      }
      // ---- O / l.  Every warp waits here: Q is free for the next segment then.
      if (!ok) break;
      ok = __all_sync(kFull, mbar_poll(b_o_final, seg & 1, abort_flag, a.wait_limit_ns) && !*abort_flag);
      if (!ok) break;
      if (active) {
        tc_fence_after();
        const bool empty = l_sum == 0.f;  // a row that sees nothing here
        const float none = without_sum(sg.s, bits), inv = empty ? 0.f : 1.f / l_sum;
        const size_t share = share_at(a, kRows, blockIdx.y, blockIdx.x, sg.place, r);
        if (valid && !sg.whole) a.sums[share] = make_float2(m_ref * mul, l_sum * (E4M3 ? pow2(-kPShift) : 1.f));
        float* part = a.part + share * D;
        __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.o) + at * D;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 16) {
          uint32_t o[16];
          tmem_ld16(tO + lane_off + c0, o);
          tmem_wait_ld();
          if (!valid) continue;
          float f[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) f[c] = empty ? none : __uint_as_float(o[c]) * inv;
          if (sg.whole) {
#pragma unroll
            for (int c = 0; c < 16; c += 8)
              *reinterpret_cast<uint4*>(orow + c0 + c) =
                  make_uint4(pack_bf16x2(f[c], f[c + 1]), pack_bf16x2(f[c + 2], f[c + 3]),
                             pack_bf16x2(f[c + 4], f[c + 5]), pack_bf16x2(f[c + 6], f[c + 7]));
          } else {
#pragma unroll
            for (int c = 0; c < 16; c += 4)
              *reinterpret_cast<float4*>(part + c0 + c) = make_float4(f[c], f[c + 1], f[c + 2], f[c + 3]);
          }
        }
        tc_fence_before();  // the next segment's first P V overwrites O
      }
      n0 += sg.nt;
      checks += tails();
      ++seg;
    }
  };
  // ------------------------------------------------ tiles
  auto tiles = [&] {
    constexpr int kN = C::kPrep * 32;
    const int t = (threadIdx.x - C::kPrepWarp * 32) % kN, w = (warp - C::kPrepWarp) % C::kPrep;
    bool ok = true;
    int n0 = 0, item0 = 0, checks = 0;
    for (int seg = 0; ok && next_segment(seg); ++seg) {
      const int first_tail = tail0();
      if constexpr (E4M3) {
        const int is_v = warp >= C::kPrepWarp + C::kPrep ? 1 : 0;
        for (int j = 0; j < sg.nt; ++j) {
          const int n = n0 + j, i = item0 + (is_v ? item_v(j, sg.nt) : item_k(j)), s = i % C::kRing;
          // The operand is free first: then the MMAs of the tiles before are
          // issued, so the slot's last item (of the other warps, perhaps) is
          // used up and b_full cannot be a phase behind.
          bool got = n < C::kOperands ||
                     mbar_poll(b_free(is_v, n), (n / C::kOperands - 1) & 1, abort_flag, a.wait_limit_ns);
          if (got) got = mbar_poll(b_full(s), (i / C::kRing) & 1, abort_flag, a.wait_limit_ns);
          if (!__all_sync(kFull, got)) {
            ok = false;
            break;
          }
          const uint32_t src = sbase + C::kOffRing + s * C::kSlot;
          const uint32_t scales = sbase + C::kOffScale + s * C::kScaleBytes;  // K, V
          const uint32_t dst = sbase + C::kOffConv + (is_v * C::kOperands + n % C::kOperands) * C::kTile;
          const bool zero = misc->bad_page[s] != 0;
          const int key0 = (sg.t0 + j) * kPage;
          // the scales of this sequence's keys decide, not what lies behind the last one
          uint32_t over = 0;
#pragma unroll
          for (int x = 0; x < 4; ++x) {  // K's, then V's
            const uint32_t o = over_f16(lds_f32(scales + (32 * x + lane) * 4));
            if (key0 + 32 * (x & 1) + lane < sg.s.len) over = max(over, o);
          }
          const bool plain = __all_sync(kFull, over <= kFitsF16 || zero);
          // A thread takes 16-code chunks, eight neighbours the same chunk of
          // eight keys: with both tiles swizzled no read or write meets a bank twice.
          constexpr int kChunks = D / 16, kM = kPage * kChunks / kN;
          const bool check = is_v && j >= first_tail;
          uint32_t bad0 = 0, bad1 = 0;  // keys 0-31 and 32-63
          auto place = [&](int m, int& key, int& c) {
            const int x = m * kN + t;
            c = (x >> 3) % kChunks;
            key = (x & 7) | (x / (8 * kChunks)) << 3;
          };
          auto load = [&](int key, int c) {
            return lds128(src + key * D + ((D == 128 ? c ^ (key & 7) : c ^ ((key >> 1) & 3)) << 4));
          };
          auto store = [&](int key, int c, const uint32_t (&o)[8]) {
            const uint32_t row = dst + (c >> 2) * C::kTilePanel + key * 128;
            const int c2 = 2 * (c & 3);
            sts128(row + ((c2 ^ (key & 7)) << 4), o[0], o[1], o[2], o[3]);
            sts128(row + (((c2 + 1) ^ (key & 7)) << 4), o[4], o[5], o[6], o[7]);
          };
          if (!is_v && t < kPage) {
            if (!plain)  // for softmax
              reinterpret_cast<float*>(smem + C::kOffKScale)[(n & 3) * kPage + t] = zero ? 0.f : lds_f32(scales + t * 4);
            if (lane == 0) misc->plain[n & 3][w] = plain ? 1 : 0;
          }
          if (plain || !is_v) {
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              int key, c;
              place(m, key, c);
              uint4 u = load(key, c);
              float sc = plain ? lds_f32(scales + (is_v * kPage + key) * 4) : 1.f;
              if (zero) sc = 0.f;
              if (check && key0 + key >= sg.s.len) {
                u = make_uint4(0, 0, 0, 0);
                sc = 0.f;  // it may be NaN
              }
              const uint32_t s2 = pack_f16x2(sc, sc), x[4] = {u.x, u.y, u.z, u.w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                e4m3x4_to_f16(x[e], o[2 * e], o[2 * e + 1]);
                o[2 * e] = mul_f16x2(o[2 * e], s2);
                o[2 * e + 1] = mul_f16x2(o[2 * e + 1], s2);
              }
              store(key, c, o);
            }
          } else {
#pragma unroll 1
            for (int m = 0; m < kM; ++m) {
              int key, c;
              place(m, key, c);
              const uint4 u = load(key, c);
              const float sc = lds_f32(scales + (kPage + key) * 4);
              const uint32_t s2 = pack_bf16x2(sc, sc), x[4] = {u.x, u.y, u.z, u.w};
              uint32_t o[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                o[2 * e] = mul_bf16x2(e4m3_hi_to_bf16x2(__byte_perm(x[e], 0, 0x1000)), s2);
                o[2 * e + 1] = mul_bf16x2(e4m3_hi_to_bf16x2(__byte_perm(x[e], 0, 0x3020)), s2);
              }
              if (check) {
                bool clear = key0 + key >= sg.s.len;
                bool nf = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) nf |= has_nonfinite(o[e]);
                if (nf && !clear && key0 + key >= sg.s.prefix) {
                  (key < 32 ? bad0 : bad1) |= 1u << (key & 31);
                  clear = true;
                }
                if (clear) {
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] = 0;
                }
              }
              store(key, c, o);
            }
            bad0 = __reduce_or_sync(kFull, bad0);
            bad1 = __reduce_or_sync(kFull, bad1);
          }
          const int c = checks + j - first_tail;
          if (check && lane == 0) misc->bad[c % kChecks][w] = static_cast<unsigned long long>(bad1) << 32 | bad0;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(b_empty(s));
            mbar_arrive(b_ready(is_v, n));
            if (check) mbar_arrive(b_checked(c));
          }
        }
      } else {
        // V tiles that hold drafted keys: slots past the end are cleared, and
        // values that are not finite taken out (softmax makes up for them)
        for (int j = first_tail; j < sg.nt; ++j) {
          const int c = checks + j - first_tail;
          if (!__all_sync(kFull, mbar_poll(b_drafted(c), (c / kChecks) & 1, abort_flag, a.wait_limit_ns))) {
            ok = false;
            break;
          }
          const uint32_t tile = sbase + C::kOffRing + ((item0 + item_v(j, sg.nt)) % C::kRing) * C::kSlot;
          const int key0 = (sg.t0 + j) * kPage;
          unsigned long long bad = 0;
          for (int base = 0; base < kPage * (D / 8); base += kN) {
            const int chunk = base + t, key = (chunk / 8) % kPage;  // panels of [64][128 B]
            const uint32_t at = tile + chunk * 16;  // the swizzle stays inside a row
            const uint4 u = lds128(at);
            const bool past = key0 + key >= sg.s.len;
            const bool nf = !past && key0 + key >= sg.s.prefix &&
                            (has_nonfinite(u.x) || has_nonfinite(u.y) || has_nonfinite(u.z) || has_nonfinite(u.w));
            if (past || nf) sts128(at, 0, 0, 0, 0);
            const unsigned vote = __ballot_sync(kFull, nf);
#pragma unroll
            for (int y = 0; y < 4; ++y)
              if ((vote >> (8 * y)) & 0xff) bad |= 1ull << (((base + w * 32) / 8 + y) % kPage);
          }
          if (lane == 0) misc->bad[c % kChecks][w] = bad;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(b_checked(c));
        }
      }
      n0 += sg.nt;
      item0 += 2 * sg.nt;
      checks += tails();
    }
    if (!ok && lane == 0) give_up(49);
  };

  if (warp < 4) {
    if constexpr (E4M3) reg_dec<C::kRegsIssue>();
    if (warp == 0)
      segments();
    else if (warp == 2)
      copies();
    else if (warp == 3)
      issue();
    else if constexpr (!E4M3)
      tiles();
  } else if (warp < 8) {
    if constexpr (E4M3) reg_inc<C::kRegsSoftmax>();
    softmax();
  } else if constexpr (E4M3) {
    reg_dec<C::kRegsPrep>();
    tiles();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tO, C::kTmemCols);
  }
}

template <int D, bool E4M3>
int launch_t(const TreeLaunch& a) {
  using C = Cfg<D, E4M3>;
  auto kern = tree_many_kernel<D, E4M3>;
  static uint64_t attr_done = 0;  // one bit per device ordinal
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return ATTN_ERR_CUDA;
  if (!(attr_done >> dev & 1)) {
    if (E4M3) {  // a warpgroup that asked for more registers than the launch left would wait for good
      static_assert(C::kRegsIssue + C::kRegsSoftmax + 2 * C::kRegsPrep <= 4 * C::kRegs, "register split");
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return ATTN_ERR_CUDA;
      if (fa.numRegs != C::kRegs) return ATTN_ERR_UNSUPPORTED;
    }
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return ATTN_ERR_CUDA;
    attr_done |= uint64_t(1) << dev;
  }
  CUtensorMap mk, mv;
  const int groups = a.num_pages * a.Hkv;
  if (E4M3 ? !tma_map_codes(&mk, a.K, groups, D, kPage) || !tma_map_codes(&mv, a.V, groups, D, kPage)
           : !tma_map_bhnd(&mk, a.K, groups, kPage, D, kPage) || !tma_map_bhnd(&mv, a.V, groups, kPage, D, kPage))
    return ATTN_ERR_CUDA;
  kern<<<dim3(a.ctas, a.planes), C::kThreads, C::kSmem, a.stream>>>(mk, mv, a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace

int launch_tree_many(const TreeLaunch& a) {
  if (a.d == 64) return a.k_scales ? launch_t<64, true>(a) : launch_t<64, false>(a);
  return a.k_scales ? launch_t<128, true>(a) : launch_t<128, false>(a);
}

}  // namespace bss
