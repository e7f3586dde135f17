// Device-side helpers for microscaled 4-bit floating point: the codes' and scales' conversions and
// the scales' place in memory.
#pragma once

#include "common.cuh"
#include "fp4.h"
#include "fp4_ring.h"

namespace gns {

// Byte of row r, block k in its 512-byte tile of 128 rows x 4 blocks. The four scales of a row
// are one word, and the words of rows 32 apart lie side by side: the order in which
// tcgen05.cp takes 32 rows of 16 bytes to the 32 lanes x 4 columns that the block-scaled MMA
// reads them from.
GNS_DEV int fp4_scale_at(int r, int k) { return ((r & 31) << 4) | (((r >> 5) & 3) << 2) | (k & 3); }

// 2^(e - 127) for a byte e (0: 2^-127, a subnormal), NaN for 255.
GNS_DEV float e8m0_to_f(uint32_t e) {
  return __uint_as_float(e == 0u ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23);
}

// Two e4m3 values, low byte first (every e4m3 value is an fp16 one).
GNS_DEV float2 e4m3x2_to_f2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
GNS_DEV float e4m3_to_f(uint8_t v) { return e4m3x2_to_f2(v).x; }

// Nearest e4m3, ties to even, at most 448; NaN stays NaN (0x7F).
GNS_DEV uint8_t f_to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return static_cast<uint8_t>(r);
}

// Four bytes of two codes each, from eight values: nearest, ties to even, at most 6.
GNS_DEV uint32_t f8_to_e2m1(float a, float b, float c, float d, float e, float f, float g, float h) {
  uint32_t r;
  asm("{\n\t.reg .b8 p0, p1, p2, p3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p3, %8, %7;\n\t"
      "mov.b32 %0, {p0, p1, p2, p3};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d), "f"(e), "f"(f), "f"(g), "f"(h));
  return r;
}

// The two values of one byte (every code's value is an fp16 one), as two halves.
GNS_DEV uint32_t e2m1x2_to_h2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 p0, p1, p2, p3;\n\t"
      "mov.b32 {p0, p1, p2, p3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p0;\n\t}"
      : "=r"(h)
      : "r"(byte));
  return h;
}
GNS_DEV float2 e2m1x2_to_f2(uint32_t byte) {
  const uint32_t h = e2m1x2_to_h2(byte);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <int FMT>
GNS_DEV float fp4_scale_to_f(uint8_t s) {
  return FMT == GNS_NVFP4 ? e4m3_to_f(s) : e8m0_to_f(s);
}

// The smallest power of two g with amax <= 6 * 448 * g (6 * 448 = 1.3125 * 2^11), at least
// 2^-126, from the bits of a finite amax >= 0; 0 for 0.
GNS_DEV uint32_t fp4_tensor_scale_bits(uint32_t amax_bits) {
  if (amax_bits == 0u) return 0u;
  const int e = (int)(amax_bits >> 23) - 11 + ((amax_bits & 0x7FFFFFu) > 0x280000u ? 1 : 0);
  return (uint32_t)(e < 1 ? 1 : e) << 23;
}

// 1 / g of a power of two 2^-126 <= g <= 2^126.
GNS_DEV float pow2_inverse(float g) { return __uint_as_float((254u << 23) - __float_as_uint(g)); }

// ---- block-scaled tensor-core products (tcgen05) ----

// mbar_wait without its clock read on the way: the timer is first read after 64 tries. A slice of 4-bit
// operands is a few hundred cycles of tensor-core work, and a read of the global timer costs about as much.
GNS_DEV bool fp4_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const uint32_t a = smem_u32(bar);
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(a, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, status);
}

// The same for a whole converged warp, which goes on or gives up as one: what comes next are instructions of
// all its lanes. (The clock and the flag of another role can give its lanes different answers.)
GNS_DEV bool fp4_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const uint32_t a = smem_u32(bar);
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(a, parity))) return true;
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort_flag, status));
}

// A last wait for what this CTA has under way, after a wait has run out: until the time `until` on the global timer.
GNS_DEV bool fp4_settle(uint64_t* bar, uint32_t parity, uint64_t until) {
  const uint32_t a = smem_u32(bar);
  while (!mbar_try_wait(a, parity))
    if (global_timer_ns() > until) return false;
  return true;
}

// The operand ring as settle_ring() sees it, in the group's leader: bytes: what one CTA loads of a slice.
struct Fp4Ring {
  uint64_t* full;
  uint32_t bytes;
  uint64_t until;
  GNS_DEV void forgo(uint32_t s) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[s])), "r"(bytes) : "memory");
  }
  GNS_DEV void announce(uint32_t s) { mbar_arrive_expect_tx(&full[s], bytes); }
  GNS_DEV bool wait(uint32_t s, uint32_t parity) { return fp4_settle(&full[s], parity, until); }
};

// A word of shared memory in CTA `rank` of the cluster.
GNS_DEV void store_cluster(void* at, uint32_t rank, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(at), rank)), "r"(v) : "memory");
}

// One lane of a converged warp, the same one each time.
GNS_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Instruction descriptor of kind::mxf4 / mxf4nvf4: both operands e2m1 and K-major, fp32
// accumulator, M x N x 64. Scales: e4m3 (NVFP4) or e8m0; sf_id: which byte of a scale column's words
// holds the step's first scale.
__host__ __device__ constexpr uint32_t fp4_idesc(int fmt, int M, int N, int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         ((fmt == GNS_NVFP4 ? 0u : 1u) << 23) | (static_cast<uint32_t>(M >> 4) << 24) |
         (static_cast<uint32_t>(sf_id) << 29);
}

// Shared-memory descriptor of a 512-byte scale tile for tcgen05.cp: no swizzle, 8 rows of 16 bytes
// to a core matrix, core matrices 128 bytes apart.
GNS_DEV uint64_t fp4_scale_desc(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46);
}

// One scale tile into four tensor-memory columns of all 128 lanes (32 lanes, repeated four times).
template <int CG>
GNS_DEV void fp4_copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// D[tmem] (+)= (A d_A) (B d_B)^T over 64 values of K.
template <int FMT, int CG>
GNS_DEV void fp4_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                     uint32_t accumulate) {
#define GNS_FP4_MMA(cg, kind, vec)                                                             \
  asm volatile(                                                                                \
      "{\n\t.reg .pred p;\n\t"                                                                 \
      "setp.ne.b32 p, %6, 0;\n\t"                                                              \
      "tcgen05.mma.cta_group::" cg ".kind::" kind ".block_scale.scale_vec::" vec               \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),                                       \
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                          \
      : "memory")
  if constexpr (FMT == GNS_NVFP4 && CG == 2)
    GNS_FP4_MMA("2", "mxf4nvf4", "4X");
  else if constexpr (FMT == GNS_NVFP4)
    GNS_FP4_MMA("1", "mxf4nvf4", "4X");
  else if constexpr (CG == 2)
    GNS_FP4_MMA("2", "mxf4", "2X");
  else
    GNS_FP4_MMA("1", "mxf4", "2X");
#undef GNS_FP4_MMA
}

// 4-D TMA load; completion on the mbarrier at shared::cluster address `bar` (the leader's for a
// CTA pair).
template <int CG>
GNS_DEV void fp4_tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2, int c3) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}
template <int CG>
GNS_DEV void fp4_tma_load_3d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1, int c2) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

}  // namespace gns
