// Products of matrices in microscaled 4-bit floating point on the tensor cores:
//   D = alpha A B^T + beta C,  (A B^T)[i][j] = sum_k A[i][k] B[j][k],
// sums in fp32 (tcgen05, block-scaled kinds), one rounding to D's type.
//
// A group of CG CTAs computes a tile of 128 CG rows of A and BN rows of B: each CTA stages its
// 128 rows of A and BN / CG rows of B in slices of 256 values of K (128 bytes a row, 128-byte
// swizzle) with the scales of its rows of A and of all BN rows of B, and holds its 128 x BN part of the
// accumulator in tensor memory. The scale tiles lie in memory as the copy into tensor memory wants
// them. Persistent groups walk the tiles (of a symmetric product: those on and above the diagonal).
//
// Warp roles in each CTA: 0 TMA producer; 1 TMEM allocation and, in the group's first CTA, the MMA
// issuer (a slice's scale tiles are copied into tensor memory just ahead of its four MMAs; copies and
// MMAs of one thread run in order); 4-7 epilogue, each warp 32 rows on its own: tensor memory,
// alpha, addend, rounding, a staging buffer in shared memory, TMA stores.
#include <cudaTypedefs.h>

#include <mutex>

#include "fp4.cuh"
#include "gemm.h"

namespace gns {
namespace {

constexpr int TM = 128;           // accumulator rows of a CTA
constexpr int TK = 256;           // values of K in a slice
constexpr int ROW_BYTES = TK / 2; // 128: the swizzle's span
constexpr int NUM_THREADS = 256;
constexpr int EPI_WARP = 4;
constexpr int OUT_ROW = 128;              // bytes of a row of an output chunk
constexpr int OUT_BYTES = 32 * OUT_ROW;   // one warp's chunk
constexpr int MAX_SMEM = 232448;

// Shared-memory plan.
template <int FMT, int CG, int BN>
struct Plan {
  static constexpr int KT = TK / fp4_block(FMT) / 4;  // scale tiles of a slice for 128 rows
  static constexpr int NB = BN / CG;                  // rows of B that a CTA stages
  static constexpr int BT = (BN + 127) / 128;         // row tiles of B's scales
  static constexpr int A_BYTES = TM * ROW_BYTES;
  static constexpr int B_BYTES = NB * ROW_BYTES;
  static constexpr int SFA_BYTES = KT * 512;
  static constexpr int SFB_BYTES = BT * KT * 512;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int OUT_ALL = 4 * 2 * OUT_BYTES;
  static constexpr int BAR_BYTES = 512;
  static constexpr int STAGES_MAX = (MAX_SMEM - 1024 - OUT_ALL - BAR_BYTES) / STAGE_BYTES;
  static constexpr int STAGES = STAGES_MAX < 8 ? STAGES_MAX : 8;
  static constexpr int OFF_SF = STAGES * (A_BYTES + B_BYTES);
  static constexpr int OFF_OUT = OFF_SF + STAGES * (SFA_BYTES + SFB_BYTES);
  static constexpr int OFF_BAR = OFF_OUT + OUT_ALL;
  static constexpr int SMEM_BYTES = 1024 + OFF_BAR + BAR_BYTES;
  static_assert(SMEM_BYTES <= MAX_SMEM && (A_BYTES + B_BYTES) % 1024 == 0 && OFF_OUT % 1024 == 0, "shared memory");
  // tensor memory: the accumulators, then a slice's scales
  static constexpr int SF_COLS = 4 * KT * (1 + BT);
  static constexpr int NACC = 2 * BN + SF_COLS <= 512 ? 2 : 1;
  static constexpr int USED_COLS = NACC * BN + SF_COLS;
  static constexpr int TMEM_COLS = USED_COLS <= 64 ? 64 : USED_COLS <= 128 ? 128 : USED_COLS <= 256 ? 256 : 512;
  static_assert(USED_COLS <= 512, "tensor memory");
};

struct GemmParams {
  CUtensorMap a, b, sfa, sfb, c, d, mirror;
  const float* ga;
  const float* gb;
  int M, N, kblocks;
  int tiles_m, tiles_n, tiles_per_mat, sym;
  long long total;
  int dtype;
  int has_c;
  float alpha, beta;
  int* status;
};

struct Tile {
  int b, I, J;
};

// Tiles of a matrix in bands of 8 tile rows, column by column inside a band: the groups that run at
// once share rows of both operands in L2. Symmetric: row by row above the diagonal.
GNS_DEV Tile tile_of(const GemmParams& P, long long t) {
  Tile o;
  o.b = (int)(t / P.tiles_per_mat);
  int r = (int)(t - (long long)o.b * P.tiles_per_mat);
  if (P.sym) {
    int i = 0;
    while (r >= P.tiles_m - i) r -= P.tiles_m - i++;
    o.I = i;
    o.J = i + r;
  } else {
    const int band = r / (8 * P.tiles_n);
    const int rows = min(8, P.tiles_m - 8 * band);
    r -= band * 8 * P.tiles_n;
    o.J = r / rows;
    o.I = 8 * band + r - o.J * rows;
  }
  return o;
}

// Byte of 16-byte unit u of row y of a chunk with rows of 128 bytes, 128-byte swizzle.
GNS_DEV uint32_t out_at(int y, int u) { return (uint32_t)(y * OUT_ROW + ((u ^ (y & 7)) << 4)); }

template <int DT>
GNS_DEV float2 unpack2(uint32_t w) {
  return DT == GNS_F16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                       : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <int DT>
GNS_DEV uint32_t pack2(float x, float y) {
  if (DT == GNS_F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// x 0 + sum, on two 16-bit values: NaN from the first Inf or NaN on.
template <int DT>
GNS_DEV uint32_t probe2(uint32_t x, uint32_t sum) {
  if (DT == GNS_F16) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0.f), *reinterpret_cast<const __half2*>(&sum));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __nv_bfloat162 r =
      __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), __float2bfloat162_rn(0.f), *reinterpret_cast<const __nv_bfloat162*>(&sum));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Whether one of the first `valid` of a row's stored values (128 bytes in w) is Inf or NaN.
template <int DT>
GNS_DEV bool any_nonfinite(const uint32_t (&w)[32], int valid) {
  constexpr int CW = DT == GNS_F32 ? 32 : 64;
  if (valid >= CW) {
    if (DT == GNS_F32) {
      float2 z = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        z = __ffma2_rn(make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])), make_float2(0.f, 0.f), z);
      return !(z.x == 0.f && z.y == 0.f);
    }
    uint32_t z = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) z = probe2<DT>(w[i], z);
    return (z & 0x7FFF7FFFu) != 0u;
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (DT == GNS_F32) {
      bad |= i < valid && (w[i] & 0x7F800000u) == 0x7F800000u;
    } else {
      constexpr uint32_t E = DT == GNS_F16 ? 0x7C00u : 0x7F80u;
      bad |= 2 * i < valid && (w[i] & E) == E;
      bad |= 2 * i + 1 < valid && ((w[i] >> 16) & E) == E;
    }
  }
  return bad;
}

// The sum's factor alpha g_A g_B: in fp32 where both of its products are normal numbers there, else by factor_far().
struct Factor {
  float one, two;
  bool split;
};

// The factor formed in 64 bits, which hold every product of three fp32 numbers. Where it leaves fp32's normal range the sum
// is multiplied by two numbers (.x, then .y), the second a power of two that brings the first back into it: as |sum| >=
// 2^-20 (NVFP4's smallest product) or 0, and < 2^64, neither step leaves the range unless the result does. (MXFP4 has no
// g; its alpha leaves the normal range as a subnormal only.) Out of line, and not for every tile: there it cost
// short products of several tiles a CTA 8 % (2048 x 4096 x 1024 14.7 -> 15.9 us, so 14.7).
__device__ __noinline__ float2 factor_far(float alpha, float ga, float gb) {
  constexpr double BIG = 0x1p100, MOST = 3.4028234663852886e38;
  const double f = (double)alpha * (double)ga * (double)gb, size = fabs(f);
  if (size >= 0x1p-126 && size <= MOST) return make_float2((float)f, 1.f);
  const bool low = size < 1.0;
  const double h = f * (low ? BIG : 1.0 / BIG);
  // (beyond 2^228 every sum but 0 gives Inf, and 0 stays 0)
  return make_float2((float)(fabs(h) > MOST ? copysign(MOST, h) : h), low ? (float)(1.0 / BIG) : (float)BIG);
}

GNS_DEV bool normal_f32(float v) { return fabsf(v) >= 1.17549435e-38f && fabsf(v) <= 3.402823466e38f; }

GNS_DEV Factor factor_of(const GemmParams& P, int b) {
  const float ga = P.ga ? P.ga[b] : 1.f, gb = P.gb ? P.gb[b] : 1.f;
  const float first = P.alpha * ga;
  float2 f = make_float2(first * gb, 1.f);
  if (!normal_f32(first) || !normal_f32(f.x)) f = factor_far(P.alpha, ga, gb);
  return Factor{f.x, f.y, f.y != 1.f};
}

// A warp's 32 rows of the tile, chunk by chunk (DT: the type of C and D).
template <int DT, int BN>
GNS_DEV bool epilogue_tile(const GemmParams& P, const Tile& t, uint32_t acc, int row0, int n0, uint8_t* out, uint64_t* cbar,
                           uint32_t& chunk, const Factor& f, bool mirror, int lane, volatile int* abort_flag) {
  constexpr int CW = DT == GNS_F32 ? 32 : 64;  // columns of a chunk
  bool bad = false;
  const bool rows_in = row0 < P.M;
  const int ncols = min(BN, P.N - n0);
  const int nch = rows_in ? (ncols + CW - 1) / CW : 0;
  if (nch == 0) return false;
  if (P.has_c) {
    if (lane == 0) {
      bulk_wait_read<1>();
      mbar_arrive_expect_tx(&cbar[chunk & 1], OUT_BYTES);
      tma_load_3d(out + (chunk & 1) * OUT_BYTES, &P.c, &cbar[chunk & 1], n0, row0, t.b);
    }
    __syncwarp();
  }
  uint32_t r[CW / 32][32];
#pragma unroll
  for (int h = 0; h < CW / 32; ++h) tmem_ld_32x32b_x32(acc + 32 * h, r[h]);
  for (int ch = 0; ch < nch; ++ch, ++chunk) {
    uint8_t* const buf = out + (chunk & 1) * OUT_BYTES;
    tmem_ld_wait();
    float2 v[CW / 2];
    const float2 f1 = make_float2(f.one, f.one);
#pragma unroll
    for (int i = 0; i < CW / 2; ++i)
      v[i] = __fmul2_rn(make_float2(__uint_as_float(r[i / 16][2 * i % 32]), __uint_as_float(r[i / 16][2 * i % 32 + 1])), f1);
    if (ch + 1 < nch) {  // the next chunk's values are on their way while this one is rounded and stored
#pragma unroll
      for (int h = 0; h < CW / 32; ++h) tmem_ld_32x32b_x32(acc + (ch + 1) * CW + 32 * h, r[h]);
    }
    if (f.split) {
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) v[i] = __fmul2_rn(v[i], make_float2(f.two, f.two));
    }
    if (!P.has_c) {
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
    } else {
      if (!fp4_warp_wait(&cbar[chunk & 1], (chunk >> 1) & 1u, abort_flag, P.status)) {
        // nothing is left under way: neither this load nor the next chunk's values
        if (!fp4_settle(&cbar[chunk & 1], (chunk >> 1) & 1u, global_timer_ns() + GNS_WAIT_TIMEOUT_NS))
          set_status(P.status, GNS_DEVST_TIMEOUT);
        __syncwarp();
        tmem_ld_wait();
        return bad;
      }
      const float2 b2 = make_float2(P.beta, P.beta);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint4 w = *reinterpret_cast<const uint4*>(buf + out_at(lane, u));
        if (DT == GNS_F32) {
          v[2 * u] = __ffma2_rn(b2, make_float2(__uint_as_float(w.x), __uint_as_float(w.y)), v[2 * u]);
          v[2 * u + 1] = __ffma2_rn(b2, make_float2(__uint_as_float(w.z), __uint_as_float(w.w)), v[2 * u + 1]);
        } else {
          const uint32_t e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) v[(4 * u + i) % (CW / 2)] = __ffma2_rn(b2, unpack2<DT>(e[i]), v[(4 * u + i) % (CW / 2)]);
        }
      }
    }
    uint32_t w[32];  // the row's 128 bytes
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (DT == GNS_F32)
        w[i] = __float_as_uint(i & 1 ? v[i / 2].y : v[i / 2].x);
      else
        w[i] = pack2<DT>(v[i % (CW / 2)].x, v[i % (CW / 2)].y);
    }
    // rows and columns outside the matrix hold nothing of it
    if (row0 + lane < P.M) bad |= any_nonfinite<DT>(w, ncols - ch * CW);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      *reinterpret_cast<uint4*>(buf + out_at(lane, u)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_3d(&P.d, buf, n0 + ch * CW, row0, t.b);
      bulk_commit();
    }
    if (mirror) {
      // the transpose of the chunk through the same buffer: row = column of the tile, 32 values each
      if (lane == 0) bulk_wait_read<0>();
      __syncwarp();
      if (DT == GNS_F32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) *reinterpret_cast<uint32_t*>(buf + i * 128 + lane * 4) = w[i];
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          *reinterpret_cast<uint16_t*>(buf + 2 * i * 64 + lane * 2) = (uint16_t)w[i];
          *reinterpret_cast<uint16_t*>(buf + (2 * i + 1) * 64 + lane * 2) = (uint16_t)(w[i] >> 16);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&P.mirror, buf, row0, n0 + ch * CW, t.b);
        bulk_commit();
      }
    }
    if (P.has_c && ch + 1 < nch) {
      const uint32_t q = (chunk + 1) & 1;
      if (lane == 0) {
        bulk_wait_read<1>();
        mbar_arrive_expect_tx(&cbar[q], OUT_BYTES);
        tma_load_3d(out + q * OUT_BYTES, &P.c, &cbar[q], n0 + (ch + 1) * CW, row0, t.b);
      }
    }
  }
  return bad;
}

template <int FMT, int CG, int BN>
__global__ void __launch_bounds__(NUM_THREADS, 1) fp4_gemm_kernel(const __grid_constant__ GemmParams P) {
  using L = Plan<FMT, CG, BN>;
  constexpr int STAGES = L::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* cbar = tempty + 2;  // two a warp of the epilogue
  uint64_t* mma_done = cbar + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* peer_abort = abort_flag + 1;
  uint32_t* issued = tmem_slot + 3;  // slices that each CTA of the group has begun to load (the leader's copy)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const long long group = blockIdx.x / CG, ngroups = gridDim.x / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], CG * 4);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&cbar[i], 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *peer_abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&P.a);
    tma_prefetch_desc(&P.b);
    tma_prefetch_desc(&P.sfa);
    tma_prefetch_desc(&P.sfb);
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc2(tmem_slot, L::TMEM_COLS);
      tmem_relinquish2();
    } else {
      tmem_alloc(tmem_slot, L::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = CG == 2 ? mapa_shared(smem_u32(&full[0]), 0) : smem_u32(&full[0]);
      const uint32_t base = smem_u32(smem);
      int s = 0;
      uint32_t ph = 0, begun = 0;
      bool ok = true;
      for (long long tile = group; ok && tile < P.total; tile += ngroups) {
        const Tile t = tile_of(P, tile);
        const int m0 = t.I * TM * CG + (int)rank * TM;
        const int n0 = t.J * BN;
        for (int kb = 0; kb < P.kblocks; ++kb) {
          if (!fp4_wait(&empty[s], ph ^ 1u, abort_flag, P.status)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], CG * L::STAGE_BYTES);
          const uint32_t fb = full0 + 8u * (uint32_t)s;
          const uint32_t sa = base + s * (L::A_BYTES + L::B_BYTES);
          const uint32_t sf = base + L::OFF_SF + s * (L::SFA_BYTES + L::SFB_BYTES);
          fp4_tma_load_3d<CG>(sa, &P.a, fb, kb * ROW_BYTES, m0, t.b);
          fp4_tma_load_3d<CG>(sa + L::A_BYTES, &P.b, fb, kb * ROW_BYTES, n0 + (int)rank * L::NB, t.b);
          fp4_tma_load_4d<CG>(sf, &P.sfa, fb, 0, kb * L::KT, m0 / 128, t.b);
          fp4_tma_load_4d<CG>(sf + L::SFA_BYTES, &P.sfb, fb, 0, kb * L::KT, n0 / 128, t.b);
          ++begun;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if constexpr (CG == 2)
        store_cluster(&issued[rank], 0, begun);
      else
        issued[0] = begun;
    }
  } else if (warp == 1) {
    if (rank == 0) {
      // The whole warp walks the slices, and one elected lane issues: the operands of copies and MMAs
      // then are in uniform registers. When a lane of its own issued them, in divergent code, issue and not the
      // tensor cores bounded the kernel (with that, and a slower epilogue, 16384 x 11008 x 4096 in 128 x 128 tiles
      // took 653 us, against 382).
      const uint32_t base = __shfl_sync(0xFFFFFFFFu, smem_u32(smem), 0);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const uint32_t sfa_t = tm + L::NACC * BN;
      const uint32_t sfb_t = sfa_t + 4 * L::KT;
      const bool leader = elect_one();
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int local = 0;
      for (long long tile = group; ok && tile < P.total; tile += ngroups, ++local) {
        const int acc = local % L::NACC;
        const uint32_t aph = (local / L::NACC) & 1;
        if (!(ok = fp4_warp_wait(&tempty[acc], aph ^ 1u, abort_flag, P.status))) break;
        tc_fence_after();
        const uint32_t d = tm + acc * BN;
        // B's first row in its first scale tile: 32 rows to a column
        const uint32_t sfb_0 = sfb_t + (BN % 128 ? (tile_of(P, tile).J * BN % 128) / 32 : 0);
        for (int kb = 0; kb < P.kblocks; ++kb) {
          if (!(ok = fp4_warp_wait(&full[s], ph, abort_flag, P.status))) break;
          tc_fence_after();
          const uint32_t sa = base + s * (L::A_BYTES + L::B_BYTES);
          const uint32_t sf = base + L::OFF_SF + s * (L::SFA_BYTES + L::SFB_BYTES);
          const uint64_t sfd = fp4_scale_desc(sf);
          const uint64_t ad = sdesc_sw128(sa, 16, 1024), bd = sdesc_sw128(sa + L::A_BYTES, 16, 1024);
          if (leader) {
#pragma unroll
            for (int k = 0; k < L::KT; ++k) {
              fp4_copy_scales<CG>(sfa_t + 4 * k, sfd + 32 * k);
#pragma unroll
              for (int n = 0; n < L::BT; ++n)
                fp4_copy_scales<CG>(sfb_t + 4 * (k * L::BT + n), sfd + L::SFA_BYTES / 16 + 32 * (n * L::KT + k));
            }
#pragma unroll
            for (int kk = 0; kk < TK / 64; ++kk) {
              // a scale column's word has the scales of 64 values (NVFP4) or 128 (MXFP4)
              constexpr int PER = fp4_block(FMT) / 16;
              const int k = kk / PER, id = (kk % PER) * 2;
              fp4_mma<FMT, CG>(d, ad + 2 * kk, bd + 2 * kk, fp4_idesc(FMT, TM * CG, BN, id), sfa_t + 4 * k,
                               sfb_0 + 4 * k * L::BT, (kb | kk) != 0 ? 1u : 0u);
            }
            if constexpr (CG == 2)
              umma2_commit_multicast(&empty[s], 0x3);
            else
              umma_commit(&empty[s]);
          }
          __syncwarp();
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (ok && leader) {
          if constexpr (CG == 2)
            umma2_commit_multicast(&tfull[acc], 0x3);
          else
            umma_commit(&tfull[acc]);
        }
        __syncwarp();
      }
    }
  } else if (warp >= EPI_WARP) {
    const int q = warp - EPI_WARP;  // the quarter of the lanes that this warp may read
    const uint32_t tempty0 = CG == 2 ? mapa_shared(smem_u32(&tempty[0]), 0) : smem_u32(&tempty[0]);
    uint8_t* const out = smem + L::OFF_OUT + q * 2 * OUT_BYTES;
    uint32_t chunk = 0;
    bool bad = false;
    int local = 0;
    for (long long tile = group; tile < P.total; tile += ngroups, ++local) {
      const Tile t = tile_of(P, tile);
      const int acc = local % L::NACC;
      const uint32_t aph = (local / L::NACC) & 1;
      const Factor f = factor_of(P, t.b);
      if (!fp4_warp_wait(&tfull[acc], aph, abort_flag, P.status)) break;
      tc_fence_after();
      const int row0 = t.I * TM * CG + (int)rank * TM + 32 * q;
      const uint32_t at = tmem + acc * BN + ((uint32_t)(32 * q) << 16);
      const bool mirror = P.sym && t.I != t.J;
      uint64_t* const cb = cbar + 2 * q;
      if (P.dtype == GNS_BF16)
        bad |= epilogue_tile<GNS_BF16, BN>(P, t, at, row0, t.J * BN, out, cb, chunk, f, mirror, lane, abort_flag);
      else if (P.dtype == GNS_F16)
        bad |= epilogue_tile<GNS_F16, BN>(P, t, at, row0, t.J * BN, out, cb, chunk, f, mirror, lane, abort_flag);
      else
        bad |= epilogue_tile<GNS_F32, BN>(P, t, at, row0, t.J * BN, out, cb, chunk, f, mirror, lane, abort_flag);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          mbar_arrive_cluster(tempty0 + 8u * acc);
        else
          mbar_arrive(&tempty[acc]);
      }
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
    }
    if (bad) set_status(P.status, GNS_DEVST_NONFINITE);
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) {
    if (threadIdx.x == 0 && *abort_flag) store_cluster(const_cast<int*>(peer_abort), rank ^ 1u, 1u);
    __syncwarp();
    cluster_sync_all();
  }
  if (*abort_flag || *peer_abort) {  // a wait ran out; the same answer in every thread of the group, whose roles have all ended
    const uint64_t until = global_timer_ns() + GNS_WAIT_TIMEOUT_NS;
    bool ended = true;
    if (rank == 0 && threadIdx.x == 0) {  // the operands' loads
      Fp4Ring ring{full, (uint32_t)L::STAGE_BYTES, until};
      ended = settle_ring(ring, issued[0], issued[CG - 1], (uint32_t)STAGES);
    }
    if (warp == 1 && elect_one()) {  // the MMAs, all issued by the leader's lane that is elected here
      if constexpr (CG == 2) {
        if (rank == 0) umma2_commit_multicast(mma_done, 0x3);
      } else {
        umma_commit(mma_done);
      }
      ended = fp4_settle(mma_done, 0u, until);
    }
    if (!ended) set_status(P.status, GNS_DEVST_TIMEOUT);
    __syncwarp();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync_all();  // neither CTA leaves before the other's loads have landed
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      tmem_dealloc2(tmem, L::TMEM_COLS);
    else
      tmem_dealloc(tmem, L::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------
// host side

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool encode(CUtensorMap* map, CUtensorMapDataType type, int rank, void* ptr, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  const cuuint32_t one[4] = {1u, 1u, 1u, 1u};
  return encoder()(map, type, (cuuint32_t)rank, ptr, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cuuint64_t stride_of(long long bytes) { return (cuuint64_t)(bytes < 16 ? 16 : (bytes + 15) / 16 * 16); }

bool encode_codes(CUtensorMap* map, const Fp4Ref& q, int64_t count, int box_rows) {
  const cuuint64_t dims[3] = {(cuuint64_t)(q.cols + 1) / 2, (cuuint64_t)q.rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {stride_of(q.ld), stride_of(q.stride)};
  const cuuint32_t box[3] = {ROW_BYTES, (cuuint32_t)box_rows, 1u};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, q.codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_scales(CUtensorMap* map, const Fp4Ref& q, int64_t count, int kt, int row_tiles) {
  const cuuint64_t tiles = (cuuint64_t)fp4_row_tiles(q.rows);
  const cuuint64_t dims[4] = {128u, (cuuint64_t)q.block_tiles, tiles, (cuuint64_t)count};
  const cuuint64_t strides[3] = {512u, 512u * (cuuint64_t)q.block_tiles, stride_of(q.scale_stride)};
  const cuuint32_t box[4] = {128u, (cuuint32_t)kt, (cuuint32_t)row_tiles, 1u};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, q.scales, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool encode_dense(CUtensorMap* map, const DenseRef& m, int64_t count, int64_t rows, int64_t cols, int box_cols, int box_rows,
                  CUtensorMapSwizzle swizzle) {
  const int size = m.dtype == GNS_F32 ? 4 : 2;
  const CUtensorMapDataType type = m.dtype == GNS_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : m.dtype == GNS_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
  const cuuint64_t strides[2] = {stride_of(m.ld * size), stride_of(m.stride * size)};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1u};
  return encode(map, type, 3, m.ptr, dims, strides, box, swizzle);
}

int cuda_error(std::string* err, const char* what, cudaError_t e) {
  (void)cudaGetLastError();
  *err = std::string(what) + ": " + cudaGetErrorString(e);
  return GNS_ERR_CUDA;
}

template <int FMT, int CG, int BN>
int launch(const Fp4Product& p, int32_t* status, cudaStream_t stream, std::string* err) {
  using L = Plan<FMT, CG, BN>;
  GemmParams P;
  const int cw = p.d.dtype == GNS_F32 ? 32 : 64;
  const int M = p.a.rows, N = p.b.rows;
  bool ok = encode_codes(&P.a, p.a, p.count, TM) && encode_codes(&P.b, p.b, p.count, L::NB) &&
            encode_scales(&P.sfa, p.a, p.count, L::KT, 1) && encode_scales(&P.sfb, p.b, p.count, L::KT, L::BT) &&
            encode_dense(&P.d, p.d, p.count, M, N, cw, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  P.has_c = p.c.ptr != nullptr;
  if (P.has_c)
    ok = ok && encode_dense(&P.c, p.c, p.count, M, N, cw, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  else
    P.c = P.d;
  if (p.sym)
    ok = ok && encode_dense(&P.mirror, p.d, p.count, M, N, 32, cw, CU_TENSOR_MAP_SWIZZLE_NONE);
  else
    P.mirror = P.d;
  if (!ok) {
    *err = "cuTensorMapEncodeTiled failed";
    return GNS_ERR_CUDA;
  }
  P.ga = p.fmt == GNS_NVFP4 ? p.a.tensor_scale : nullptr;
  P.gb = p.fmt == GNS_NVFP4 ? p.b.tensor_scale : nullptr;
  P.M = M;
  P.N = N;
  P.kblocks = (p.a.cols + TK - 1) / TK;
  P.tiles_m = (M + TM * CG - 1) / (TM * CG);
  P.tiles_n = (N + BN - 1) / BN;
  P.sym = p.sym;
  P.tiles_per_mat = p.sym ? P.tiles_m * (P.tiles_m + 1) / 2 : P.tiles_m * P.tiles_n;
  P.total = (long long)p.count * P.tiles_per_mat;
  P.dtype = p.d.dtype;
  P.alpha = p.alpha;
  P.beta = p.beta;
  P.status = status;

  static std::once_flag once[64];
  static cudaError_t opted[64];
  int dev = 0;
  cudaGetDevice(&dev);
  dev = dev < 0 || dev >= 64 ? 0 : dev;
  std::call_once(once[dev], [&] {
    opted[dev] = cudaFuncSetAttribute(fp4_gemm_kernel<FMT, CG, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_BYTES);
  });
  if (opted[dev] != cudaSuccess) return cuda_error(err, "cudaFuncSetAttribute", opted[dev]);
  const long long most = device_sm_count() / CG;
  const int groups = (int)(P.total < most ? P.total : most);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(groups * CG, 1, 1);
  cfg.blockDim = dim3(NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = L::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CG > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_gemm_kernel<FMT, CG, BN>, P);
  if (e != cudaSuccess) return cuda_error(err, "launch", e);
  profile_count_launch();
  return GNS_OK;
}

// 128 x 128 tiles of single CTAs, or tiles of CTA pairs: 256 x 192 (two accumulators in tensor memory) for
// A B^T, 256 x 256 (one accumulator; a symmetric product's tiles are square) for X X^T. A pair tile
// reads less per product from L2, which bounds the small one, and fills the SMs less evenly. What counts is
// the number of waves over the SMs, weighted by what one costs (a wave of 256 x 192 tiles about 1.1 to 1.2, of
// 256 x 256 tiles 1.6 to 1.9 times one of 128 x 128, for K of 4096 and more). NVFP4 with bf16 results in a captured graph,
// us, 128 x 128 against the pair's: 16384 x 11008 x 4096 382 / 277, 4096 x 11008 x 4096 103 / 79, 512 x 4096 x
// 4096 10.6 / 12.3, 16 of 1024 x 1024 x 2048 26.5 / 30.5; X X^T of 16 of 2048 x 8192 153 / 132, of 24 of
// 1024 x 4096 39 / 48. MXFP4 is within 3 % of that. Short K and fp32 results weigh the epilogue, which the rule does not:
// 2048 x 4096 x 1024 takes pairs with 14.6 / 16.8, 4096 x 4096 of X X^T in fp32 with 31.5 / 33.5.
template <int FMT>
int launch_format(const Fp4Product& p, int32_t* status, cudaStream_t stream, std::string* err) {
  const long long sms = device_sm_count(), M = p.a.rows, N = p.b.rows;
  auto up = [](long long n, long long d) { return (n + d - 1) / d; };
  auto tri = [](long long t) { return t * (t + 1) / 2; };
  const long long m1 = up(M, 128), m2 = up(M, 256);
  const long long single = up(p.count * (p.sym ? tri(m1) : m1 * up(N, 128)), sms);
  const long long pairs = up(p.count * (p.sym ? tri(m2) : m2 * up(N, 192)), sms / 2);
  if (p.sym) {
    if (1.75 * (double)pairs < (double)single) return launch<FMT, 2, 256>(p, status, stream, err);
  } else if (1.2 * (double)pairs < (double)single) {
    return launch<FMT, 2, 192>(p, status, stream, err);
  } else if (2 * p.count * m1 * up(N, 128) <= sms) {
    // half the SMs or more would be idle: tiles half as wide (1000 x 1000 x 1000 5.9 -> 5.2 us, 1 x 4096 x
    // 11008 16.4 -> 15.7)
    return launch<FMT, 1, 64>(p, status, stream, err);
  }
  return launch<FMT, 1, 128>(p, status, stream, err);
}

}  // namespace

int fp4_gemm_launch(const Fp4Product& p, int32_t* dev_status, void* stream, std::string* err) {
  if (!encoder()) {
    *err = "cuTensorMapEncodeTiled is not available from the CUDA driver";
    return GNS_ERR_CUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p.fmt == GNS_NVFP4 ? launch_format<GNS_NVFP4>(p, dev_status, s, err)
                            : launch_format<GNS_MXFP4>(p, dev_status, s, err);
}

}  // namespace gns
