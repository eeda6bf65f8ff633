// Selective scan over packed prompts on tcgen05, for fp16 rows, heads of 64 and states of
// 64 or 128, two heads of one group per CTA.
#pragma once

#include "mixer.cuh"
#include "tcgen05.cuh"

namespace dfssm {

// One CTA: (segment, pair of heads), the segment in chunks of Q = 128 rows.  With cs_t the
// running sum of -dt exp(A_log) in the chunk, a chunk is four products per head:
//   CB = C B^T                                       [t][s]   (once for both heads)
//   Y1 = M X,  M[t][s] = CB[t][s] exp(cs_t - cs_s) dt_s, s <= t   [t][p]
//   Y2 = C H^T, H the state that enters                [t][p]
//   S  = W B,  W[p][s] = exp(cs_Q - cs_s) dt_s x_s[p]       [p][n]
//   y_t = Y1 + exp(cs_t) Y2 + D x_t,   H <- exp(cs_Q) H + S.
// x, B and C are operands as they are (fp16 is exact); M, H and W are fp32 values and go in
// as two fp16 pieces, value = hi + lo to 2^-22, two products each, scaled by a power of two
// (per row of M, per head of H and W) so that the largest lies below 2^14: fp16 then holds
// the pieces of everything down to 2^-28 of it.  Accumulation is fp32 in tensor memory, the
// state fp32 in registers.
//   warps 0..7   arithmetic.  For M and y: warpgroup = head, thread = row t (TMEM lane);
//                for W, S and H: thread = (head, p) (TMEM lane), warpgroup = half of the
//                rows s (W) or of the state's columns (S, H; in registers throughout);
//   warp 8       TMA: B double-buffered, C and X single (each is asked for again as soon
//                as its last reader is done, a good part of a chunk before it is needed);
//   warp 9       MMA issuer;
//   warps 10, 11 a head each, one chunk ahead: step sizes, running sums (fp64) and their
//                tables.  cs is kept as two floats, hi + lo: near differences are then good to
//                2^-24 of their own size however far the sum has run (a step may be huge).
// Tensor memory (columns): CB [0,128), then Y2 of both heads; M of head 0 [128,256) as hi | lo,
// then S; M of head 1 [256,384), then W; Y1 of both heads [384,512).
// STATES: only what a segment adds to a zero state (W and S), for segments that are not
// their sequence's last; see k_scan_join.
// Every wait is bounded; one that gives up sets the status bit, the roles run through
// their loops without waiting, and the block ends as usual.
constexpr int kStQ = 128;
constexpr int kStThreads = 384;
constexpr int kStP = 64;

__host__ __device__ constexpr int st_tile_bytes(int n) { return kStQ * n * 2; }
// Tables of a chunk and head: cs log2 e as hi and lo, dt, exp(cs), W's factors, and
// exp(cs_e - cs_s) dt_s with e the last row of the 32 that s belongs to.
constexpr int kStHi = 0, kStLo = kStQ, kStDt = 2 * kStQ, kStExp = 3 * kStQ, kStW = 4 * kStQ, kStCol = 5 * kStQ,
              kStTab = 6 * kStQ;
__host__ __device__ constexpr size_t st_smem_bytes(int n, bool states) {
  return 1024 + (states ? 2 : 3) * size_t(st_tile_bytes(n)) + 2 * st_tile_bytes(kStP) +
         size_t(2) * 2 * kStP * n * 2 + size_t(4) * 4 * kStTab;
}

DFSSM_DEV uint64_t umma_desc_sw128_mn(uint32_t saddr, uint32_t lbo) {
  return uint64_t((saddr >> 4) & 0x3fffu) | (uint64_t(lbo >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
DFSSM_DEV void umma_f16_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
      :: "r"(d), "l"(ad), "l"(bd), "r"(idesc), "r"(uint32_t(acc)) : "memory");
}
DFSSM_DEV void umma_f16_ts(uint32_t d, uint32_t a, uint64_t bd, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
      :: "r"(d), "r"(a), "l"(bd), "r"(idesc), "r"(uint32_t(acc)) : "memory");
}
DFSSM_DEV float exp2_f(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
DFSSM_DEV float pow2_f(int k) { return __int_as_float((k + 127) << 23); }       // |k| <= 126
// k with v 2^k in [2^13, 2^14) (0 for v = 0, and within [-100, 100]).
DFSSM_DEV int scale_of(float v) {
  const int e = int((__float_as_uint(v) >> 23) & 0xffu) - 126;                    // v < 2^e
  return v > 0.f ? max(-100, min(100, 14 - e)) : 0;
}
// Two values as fp16 pieces: hi = their fp16 pair, lo = that of what is left.
DFSSM_DEV void split_h2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_h2(a - f.x, b - f.y);
}
DFSSM_DEV void bar_compute() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

DFSSM_DEV void bar_group(int wg) { asm volatile("bar.sync %0, 128;" :: "r"(2 + wg) : "memory"); }

struct StBars {
  uint64_t fullB[2], emptyB[2], tabA[2], tabX[2], tabE[2];
  uint64_t fullC, emptyC, fullX, emptyX, d1, mready, m2done, ydone, wready, sdone, dfree, hready, done;
};

template <typename TY, typename TS, int N, bool STATES>
__global__ void __launch_bounds__(kStThreads, 1)
    k_scan_tc(ScanArgs a, const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_c) {
  constexpr int TB = st_tile_bytes(N), TX = st_tile_bytes(kStP), HALF = st_tile_bytes(64), NH = N / 2;
  constexpr int COLS = STATES ? 256 : 512;
  constexpr uint32_t cS = STATES ? 0 : 128, cW = STATES ? 128 : 256;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) StBars bars;
  __shared__ uint32_t tmem_s;
  __shared__ int fail;
  __shared__ float scal[2][2][4];        // [buffer][head]: exp(cs_Q), max dt, 2^-k of W
  __shared__ float wmax[2][8], hinv[2][2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = smem_u32(smem_raw);
  unsigned char* base = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  unsigned char* const sB = base;                                    // [2][halves of 64][128 rows][128 B]
  unsigned char* const sX = sB + 2 * TB;                             // [2 heads][128 rows][128 B]
  unsigned char* const sC = sX + 2 * TX;
  unsigned char* const sH = sC + (STATES ? 0 : TB);                  // [2 heads][hi, lo][halves][64 rows][128 B]
  float* const tab = reinterpret_cast<float*>(sH + 2 * 2 * kStP * N * 2);   // [2][2][kStTab]

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(&tmem_s)), "n"(COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 256) {
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&tm_x)) : "memory");
    asm volatile("prefetch.tensormap [%0];" :: "l"(reinterpret_cast<uint64_t>(&tm_b)) : "memory");
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.fullB[i], 1);
      mbar_init(&bars.emptyB[i], 1);
      mbar_init(&bars.tabA[i], 2);
      mbar_init(&bars.tabX[i], 2);
      mbar_init(&bars.tabE[i], 8);
    }
    mbar_init(&bars.fullC, 1);
    mbar_init(&bars.emptyC, 1);
    mbar_init(&bars.fullX, 1);
    mbar_init(&bars.emptyX, 8);
    mbar_init(&bars.d1, 1);
    mbar_init(&bars.mready, 8);
    mbar_init(&bars.m2done, 1);
    mbar_init(&bars.ydone, 1);
    mbar_init(&bars.wready, 8);
    mbar_init(&bars.sdone, 1);
    mbar_init(&bars.dfree, 8);
    mbar_init(&bars.hready, 8);
    mbar_init(&bars.done, 1);
    fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  pdl_wait();
  pdl_release();
  auto wait = [&](uint64_t& bar, unsigned parity) { return tc_wait(&bar, parity & 1u, a.q.status, &fail, kSeqWait); };
  auto arrive = [&](uint64_t& bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar);
  };

  const int h0 = 2 * blockIdx.y, g = h0 / (a.H / a.G);
  SegWork w{};
  int slot = -1;
  bool work = seg_find(a, blockIdx.x, w) && !(STATES && w.k == w.count - 1);
  if (work && a.state) {
    slot = seq_slot(a.q, w.s, tid, kStThreads, [](bool v) { return __syncthreads_or(v) != 0; });
    work = slot >= 0;
  }
  const int chunks = work ? (w.t1 - w.t0 + kStQ - 1) / kStQ : 0;

  if (warp == 8) {
    // ---- TMA
    const bool one = elect_one();
    int issued = 0;
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, r0 = w.t0 + c * kStQ;
      bool go = c < 2 || wait(bars.emptyB[b], (c >> 1) - 1);
      if (one && go) {
        mbar_expect_tx(&bars.fullB[b], TB);
        for (int i = 0; i < N / 64; ++i)
          tma_load_2d(smem_u32(sB) + b * TB + i * HALF, &tm_b, g * N + 64 * i, r0, &bars.fullB[b]);
      }
      if (!STATES) {
        go = go && (c < 1 || wait(bars.emptyC, c - 1));
        if (one && go) {
          mbar_expect_tx(&bars.fullC, TB);
          for (int i = 0; i < N / 64; ++i) tma_load_2d(smem_u32(sC) + i * HALF, &tm_c, g * N + 64 * i, r0, &bars.fullC);
        }
      }
      go = go && (c < 1 || wait(bars.emptyX, c - 1));
      if (one && go) {
        mbar_expect_tx(&bars.fullX, 2 * TX);
        for (int i = 0; i < 2; ++i) tma_load_2d(smem_u32(sX) + i * TX, &tm_x, (h0 + i) * kStP, r0, &bars.fullX);
      }
      if (!__all_sync(0xffffffffu, go)) break;
      issued = c + 1;
    }
    // no copy may still be landing when the block ends (a load that was not issued costs
    // only time here, after a wait that gave up)
    auto landed = [&](uint64_t& bar, int parity) {
      for (long long s = 0; s < kTcSpinLimit / 16 && !mbar_try_wait(&bar, unsigned(parity) & 1u); ++s) {
      }
    };
    for (int c = max(0, issued - 2); c < chunks && c < issued + 1; ++c) landed(bars.fullB[c & 1], c >> 1);
    if (issued > 0) {
      if (!STATES) landed(bars.fullC, issued - 1);
      landed(bars.fullX, issued - 1);
    }
  } else if (warp == 9) {
    // ---- MMA
    const bool one = elect_one();
    const uint32_t i1 = umma_idesc_f16(128, 128), i2 = umma_idesc_f16(128, kStP, true), i3 = umma_idesc_f16(128, kStP),
                   i4 = umma_idesc_f16(128, N, true);
    const uint32_t aB = smem_u32(sB), aX = smem_u32(sX), aC = smem_u32(sC), aH = smem_u32(sH);
    bool go = true;
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1;
      go = wait(bars.fullB[b], c >> 1) && go;
      if (!STATES) {
        go = wait(bars.fullC, c) && go;
        if (c > 0) go = wait(bars.dfree, c - 1) && go;
        go = __all_sync(0xffffffffu, go);
        tc_fence_after();
        if (one && go) {
          for (int k = 0; k < N / 16; ++k) {
            const uint32_t at = (k >> 2) * HALF + (k & 3) * 32;
            umma_f16_ss(tmem, umma_desc_sw128(aC + at), umma_desc_sw128(aB + b * TB + at), i1, k > 0);
          }
          tc_commit(&bars.d1);
        }
        go = wait(bars.fullX, c) && go;
        go = wait(bars.mready, c) && go;
        go = __all_sync(0xffffffffu, go);
        tc_fence_after();
        if (one && go) {
          for (int h = 0; h < 2; ++h)
            for (int k = 0; k < 2 * kStQ / 16; ++k)      // hi, then lo
              umma_f16_ts(tmem + 384 + 64 * h, tmem + 128 + 128 * h + 8 * k,
                          umma_desc_sw128_mn(aX + h * TX + (k & 7) * 2048, HALF), i2, k > 0);
          tc_commit(&bars.m2done);
        }
        go = wait(bars.hready, c) && go;
        go = __all_sync(0xffffffffu, go);
        if (one && go) {
          for (int h = 0; h < 2; ++h)
            for (int j = 0; j < 2; ++j)
              for (int k = 0; k < N / 16; ++k) {
                const uint32_t ca = (k >> 2) * HALF + (k & 3) * 32, ha = (k >> 2) * 8192 + (k & 3) * 32;
                umma_f16_ss(tmem + 64 * h, umma_desc_sw128(aC + ca), umma_desc_sw128(aH + (2 * h + j) * kStP * N * 2 + ha), i3,
                            j > 0 || k > 0);
              }
          tc_commit(&bars.emptyC);
          tc_commit(&bars.ydone);
        }
      }
      go = wait(bars.wready, c) && go;
      go = __all_sync(0xffffffffu, go);
      tc_fence_after();
      if (one && go) {
        for (int k = 0; k < 2 * kStQ / 16; ++k)
          umma_f16_ts(tmem + cS, tmem + cW + 8 * k, umma_desc_sw128_mn(aB + b * TB + (k & 7) * 2048, HALF), i4, k > 0);
        tc_commit(&bars.emptyB[b]);
        tc_commit(&bars.sdone);
      }
    }
    if (!go) {        // no MMA may still run when the tensor memory is given back
      if (one) tc_commit(&bars.done);
      for (long long s = 0; s < kTcSpinLimit && !mbar_try_wait(&bars.done, 0u); ++s) {
      }
    }
  } else if (warp >= 10) {
    // ---- step sizes and tables of head h0 + hd: lane = four rows
    const int hd = warp - 10, h = h0 + hd;
    const double rate = chunks ? -exp(double(a.A_log[h])) : 0.0, log2e = 1.4426950408889634;
    const float bias = a.dt_bias[h];
    double seg = 0.0;
    float next[4];                  // raw step sizes of the chunk to come
    auto fetch = [&](int c) {
#pragma unroll
      for (int j = 0; j < 4; ++j) next[j] = scan_raw(a, min(w.t0 + c * kStQ + 4 * lane + j, w.t1 - 1), h);
    };
    if (chunks > 0) fetch(0);
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, r0 = w.t0 + c * kStQ, n = min(kStQ, w.t1 - r0);
      float dt[4];
      double cs[4], run = 0.0;
#pragma unroll
      for (int j = 0; j < 4; ++j) dt[j] = 4 * lane + j < n ? softplus_f(next[j] + bias) : 0.f;
      if (c + 1 < chunks) fetch(c + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        run += double(dt[j]) * rate;
        cs[j] = run;
      }
      double up = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      const double total = __shfl_sync(0xffffffffu, up, 31);
      float dmax = 0.f, wx[4], top = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cs[j] += up - run;
        dmax = fmaxf(dmax, dt[j]);
        wx[j] = exp2_f(float((total - cs[j]) * log2e)) * dt[j];
        top = fmaxf(top, wx[j]);
      }
      dmax = warp_max(dmax);
      top = warp_max(top);
      seg += total;
      if (c >= 2) wait(bars.tabE[b], (c >> 1) - 1);
      float* tb = tab + (2 * b + hd) * kStTab;
      if (!STATES) {
        float hi[4], lo[4], ex[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const double e = cs[j] * log2e;
          hi[j] = float(e);
          lo[j] = float(e - double(hi[j]));
          ex[j] = exp2_f(hi[j]);
        }
        *reinterpret_cast<float4*>(tb + kStHi + 4 * lane) = make_float4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<float4*>(tb + kStLo + 4 * lane) = make_float4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<float4*>(tb + kStDt + 4 * lane) = make_float4(dt[0], dt[1], dt[2], dt[3]);
        *reinterpret_cast<float4*>(tb + kStExp + 4 * lane) = make_float4(ex[0], ex[1], ex[2], ex[3]);
        const double last = __shfl_sync(0xffffffffu, cs[3], lane | 7);
        float col[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) col[j] = exp2_f(float((last - cs[j]) * log2e)) * dt[j];
        *reinterpret_cast<float4*>(tb + kStCol + 4 * lane) = make_float4(col[0], col[1], col[2], col[3]);
        if (lane == 0) scal[b][hd][1] = dmax;
      }
      if (lane == 0) scal[b][hd][0] = exp2_f(float(total * log2e));
      arrive(bars.tabA[b]);
      // the largest |x| of the chunk bounds W's values
      wait(bars.fullX, c);
      __half2 m = __floats2half2_rn(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane + 32 * i;
        if (r < n) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint4 v = *reinterpret_cast<const uint4*>(sX + hd * TX + r * 128 + 16 * j);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) m = __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&u[k])));
          }
        }
      }
      const float xmax = warp_max(fmaxf(__low2float(m), __high2float(m)));
      const int k = scale_of(xmax * top);
      const float up2 = pow2_f(k);
      *reinterpret_cast<float4*>(tb + kStW + 4 * lane) = make_float4(wx[0] * up2, wx[1] * up2, wx[2] * up2, wx[3] * up2);
      if (lane == 0) scal[b][hd][2] = pow2_f(-k);
      arrive(bars.tabX[b]);
    }
    if (STATES && work && lane == 0) a.seg_decay[size_t(blockIdx.x) * a.H + h] = exp2_f(float(seg * log2e));
  } else if (chunks > 0) {
    // ---- arithmetic
    const int wg = warp >> 2, q = warp & 3, L = 32 * q + lane;
    const uint32_t tl = tmem + (uint32_t(32 * q) << 16);
    const int hd = q >> 1, p = L & 63;                       // W, S, H: (head, p), columns NH wg ..
    const int hy = h0 + wg;                                  // M, y: head, row t = L
    const float Dh = a.D ? a.D[hy] : 0.f;
    float hs[NH];
    // the two heads' states, [128][N] in global memory, pass through shared memory (the
    // place of H) so that whole lines move: piece j of row r at j ^ (r mod 8)
    const size_t pair_at = (size_t(STATES || w.count > 1 ? blockIdx.x : slot) * a.H + h0) * kStP * N;
    auto piece = [&](int r, int j) { return reinterpret_cast<float4*>(sH) + r * (N / 4) + (j ^ (r & 7)); };
    auto load_state = [&](const auto* from) {
#pragma unroll 4
      for (int i = tid; i < 2 * kStP * N / 4; i += 256) {
        float v[4];
        ldv<4>(from + 4 * i, v);
        *piece(i / (N / 4), i % (N / 4)) = make_float4(v[0], v[1], v[2], v[3]);
      }
      bar_compute();
#pragma unroll
      for (int j = 0; j < NH / 4; ++j) {
        const float4 v = *piece(L, NH / 4 * wg + j);
        hs[4 * j] = v.x; hs[4 * j + 1] = v.y; hs[4 * j + 2] = v.z; hs[4 * j + 3] = v.w;
      }
    };
    auto store_state = [&](auto* to) {
#pragma unroll
      for (int j = 0; j < NH / 4; ++j)
        *piece(L, NH / 4 * wg + j) = make_float4(hs[4 * j], hs[4 * j + 1], hs[4 * j + 2], hs[4 * j + 3]);
      bar_compute();
#pragma unroll 4
      for (int i = tid; i < 2 * kStP * N / 4; i += 256) {
        const float4 v = *piece(i / (N / 4), i % (N / 4));
        const float f[4] = {v.x, v.y, v.z, v.w};
        stv<4>(to + 4 * i, f);
      }
    };
#pragma unroll
    for (int j = 0; j < NH; ++j) hs[j] = 0.f;
    if (!STATES) {
      if (w.count > 1) load_state(static_cast<const float*>(a.seg_state) + pair_at);
      else if (a.state && !(a.q.fresh && a.q.fresh[w.s])) load_state(static_cast<const TS*>(a.state) + pair_at);
    }
    // H into shared memory as fp16 pieces for chunk c
    auto put_h = [&](int c) {
      float m = 0.f;
#pragma unroll
      for (int j = 0; j < NH; ++j) m = fmaxf(m, fabsf(hs[j]));
      m = warp_max(m);
      if (lane == 0) wmax[c & 1][warp] = m;
      bar_compute();
      const float* wm = wmax[c & 1];
      m = fmaxf(fmaxf(wm[2 * hd], wm[2 * hd + 1]), fmaxf(wm[4 + 2 * hd], wm[5 + 2 * hd]));
      const int k = scale_of(m);
      const float up = pow2_f(k);
      if (p == 0 && wg == 0) hinv[c & 1][hd] = pow2_f(-k);
#pragma unroll
      for (int j = 0; j < NH; j += 8) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_h2(hs[j + 2 * i] * up, hs[j + 2 * i + 1] * up, hi[i], lo[i]);
        const int n = NH * wg + j;
        unsigned char* at = sH + (n >> 6) * 8192 + p * 128 + ((((n & 63) >> 3) ^ (p & 7)) << 4) + 2 * hd * kStP * N * 2;
        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + kStP * N * 2) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_async_smem();
      arrive(bars.hready);
    };
    if (!STATES) put_h(0);
    for (int c = 0; c < chunks; ++c) {
      const int b = c & 1, r0 = w.t0 + c * kStQ, n = min(kStQ, w.t1 - r0);
      const float* tb = tab + 2 * b * kStTab;
      float ytop = 1.f;                                       // 2^-k of this row of M
      if (n < kStQ) {
        // rows behind the sequence's end are another's: zero, as 0 times NaN is no 0
        wait(bars.fullX, c);
        wait(bars.fullB[b], c >> 1);
        if (L >= n) {
          const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            *reinterpret_cast<uint4*>(sX + wg * TX + L * 128 + 16 * j) = zero;
            if (N == 128 || wg == 0) *reinterpret_cast<uint4*>(sB + b * TB + wg * HALF + L * 128 + 16 * j) = zero;
          }
        }
        fence_async_smem();
        bar_compute();
      }
      if (!STATES) {
        // M
        wait(bars.tabA[b], c >> 1);
        const float* te = tb + wg * kStTab;
        const float dmax = scal[b][wg][1];
        const float thi = te[kStHi + L], tlo = te[kStLo + L];
        wait(bars.d1, c);
        tc_fence_after();
        float m = 0.f, v[32];
#pragma unroll 1
        for (int s0 = 0; s0 < 32 * q; s0 += 32) {
          tmem_ld32(tl + s0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
        }
        tmem_ld32(tl + 32 * q, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) m = fmaxf(m, i <= lane ? fabsf(v[i]) : 0.f);
        const int k = scale_of(m * dmax);
        const float up = pow2_f(k);
        ytop = pow2_f(-k);
        const uint32_t tm = tl + 128 + 128 * wg;
        uint32_t hi[16], lo[16];
        // the 32 columns of the warp's own rows
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 eh = *reinterpret_cast<const float4*>(te + kStHi + 32 * q + i);
          const float4 el = *reinterpret_cast<const float4*>(te + kStLo + 32 * q + i);
          const float4 ds = *reinterpret_cast<const float4*>(te + kStDt + 32 * q + i);
          const float e[4] = {(thi - eh.x) + (tlo - el.x), (thi - eh.y) + (tlo - el.y), (thi - eh.z) + (tlo - el.z),
                              (thi - eh.w) + (tlo - el.w)};
          const float d[4] = {ds.x, ds.y, ds.z, ds.w};
          float r[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) r[j] = i + j <= lane ? (v[i + j] * up) * (exp2_f(e[j]) * d[j]) : 0.f;
          split_h2(r[0], r[1], hi[i / 2], lo[i / 2]);
          split_h2(r[2], r[3], hi[i / 2 + 1], lo[i / 2 + 1]);
        }
        tmem_st16(tm + 16 * q, hi);
        tmem_st16(tm + 64 + 16 * q, lo);
        // earlier columns: with e the last row of their 32, exp(cs_t - cs_s) is exp(cs_t - cs_e)
        // exp(cs_e - cs_s), neither above 1: one exponential per row and 32 columns
#pragma unroll 1
        for (int s0 = 0; s0 < 32 * q; s0 += 32) {
          const float f = up * exp2_f((thi - te[kStHi + s0 + 31]) + (tlo - te[kStLo + s0 + 31]));
          tmem_ld32(tl + s0, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 cf = *reinterpret_cast<const float4*>(te + kStCol + s0 + i);
            split_h2((v[i] * f) * cf.x, (v[i + 1] * f) * cf.y, hi[i / 2], lo[i / 2]);
            split_h2((v[i + 2] * f) * cf.z, (v[i + 3] * f) * cf.w, hi[i / 2 + 1], lo[i / 2 + 1]);
          }
          tmem_st16(tm + s0 / 2, hi);
          tmem_st16(tm + 64 + s0 / 2, lo);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) hi[i] = 0u;
#pragma unroll 1
        for (int s0 = 32 * q + 32; s0 < kStQ; s0 += 32) {
          tmem_st16(tm + s0 / 2, hi);
          tmem_st16(tm + 64 + s0 / 2, hi);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bars.mready);
      }
      // W: rows s = 64 wg .. + 63 of column p of head hd
      {
        wait(bars.fullX, c);
        wait(bars.tabX[b], c >> 1);
        const float* tw = tb + hd * kStTab + kStW;
        const unsigned char* xc = sX + hd * TX + (p & 7) * 2;
        const int ch = p >> 3;
#pragma unroll 1
        for (int s0 = 64 * wg; s0 < 64 * wg + 64; s0 += 32) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(tw + s0 + i);
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[j] = __half2float(*reinterpret_cast<const __half*>(xc + (s0 + i + j) * 128 + ((ch ^ ((i + j) & 7)) << 4)));
            split_h2(x[0] * f.x, x[1] * f.y, hi[i / 2], lo[i / 2]);
            split_h2(x[2] * f.z, x[3] * f.w, hi[i / 2 + 1], lo[i / 2 + 1]);
          }
          if (!STATES && s0 == 64 * wg) {
            wait(bars.m2done, c);              // M of head 1 has been read
            tc_fence_after();
          }
          tmem_st16(tl + cW + s0 / 2, hi);
          tmem_st16(tl + cW + 64 + s0 / 2, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bars.wready);
        if (STATES) arrive(bars.emptyX);
        else bar_compute();            // X has been read: its rows take y's on the way out
      }
      if (!STATES) {
        // y: row L of head wg into its row of X, 128 bytes at a time, and from there to global
        // memory in whole lines
        constexpr int PC = 128 / int(sizeof(TY)), RD = kStP / PC;      // columns of a piece, pieces
        const float et = tb[wg * kStTab + kStExp + L];
        unsigned char* const xrow = sX + wg * TX + L * 128;
        uint4 xv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xv[j] = *reinterpret_cast<const uint4*>(xrow + ((j ^ (L & 7)) << 4));
        wait(bars.ydone, c);
        tc_fence_after();
        const float f2 = et * hinv[c & 1][wg];
        TY* const yp = static_cast<TY*>(a.y.p) + (long long)r0 * a.y.stride + hy * kStP;
#pragma unroll
        for (int rd = 0; rd < RD; ++rd) {
#pragma unroll
          for (int j = rd * PC; j < (rd + 1) * PC; j += 16) {
            float y1[16], y2[16], out[16];
            tmem_ld16(tl + 384 + 64 * wg + j, y1);
            tmem_ld16(tl + 64 * wg + j, y2);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const uint4 u = xv[(j + i) / 8];
              const uint32_t word = (i & 6) == 0 ? u.x : (i & 6) == 2 ? u.y : (i & 6) == 4 ? u.z : u.w;
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&word));
              out[i] = fmaf(Dh, f.x, fmaf(y2[i], f2, y1[i] * ytop));
              out[i + 1] = fmaf(Dh, f.y, fmaf(y2[i + 1], f2, y1[i + 1] * ytop));
            }
            constexpr int E = 16 / int(sizeof(TY));
#pragma unroll
            for (int i = 0; i < 16; i += E) {
              const int ch = (j + i) % PC / E;
              stv<E>(reinterpret_cast<TY*>(xrow + ((ch ^ (L & 7)) << 4)), reinterpret_cast<float(&)[E]>(out[i]));
            }
          }
          if (rd == RD - 1) {
            tc_fence_before();
            arrive(bars.dfree);
          }
          bar_group(wg);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 16 * i + (tid & 127) / 8, ch = tid & 7;
            const uint4 v = *reinterpret_cast<const uint4*>(sX + wg * TX + r * 128 + ((ch ^ (r & 7)) << 4));
            if (r < n) *reinterpret_cast<uint4*>(yp + (long long)r * a.y.stride + rd * PC + ch * (16 / int(sizeof(TY)))) = v;
          }
          if (rd + 1 < RD) bar_group(wg);
        }
        arrive(bars.emptyX);
      }
      // H
      const float keep = scal[b][hd][0], down = scal[b][hd][2];
      wait(bars.sdone, c);
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < NH; j += 16) {
        float v[16];
        tmem_ld16(tl + cS + NH * wg + j, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) hs[j + i] = fmaf(hs[j + i], keep, v[i] * down);
      }
      tc_fence_before();
      arrive(bars.tabE[b]);
      if (!STATES && c + 1 < chunks) put_h(c + 1);      // its barrier also keeps M's stores behind S's loads
    }
    if (STATES) store_state(a.seg_state + pair_at);
    else if (a.state && w.k == w.count - 1) store_state(static_cast<TS*>(a.state) + (size_t(slot) * a.H + h0) * kStP * N);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(COLS) : "memory");
}

}  // namespace dfssm
