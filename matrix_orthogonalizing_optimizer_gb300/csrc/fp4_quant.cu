// Conversions to and from microscaled 4-bit floating point.
//
// A block of 16 (NVFP4) or 32 (MXFP4) values along a row shares one scale d; a value x is held as
// the code nearest to x / d among +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, magnitudes
// above 6 d as 6 d.
//   NVFP4: d = g s, g = the smallest power of two with max |X| <= 6 * 448 g over the matrix,
//          s = max |block| / (6 g) rounded to e4m3
//   MXFP4: d = 2^(floor(log2(max |block|)) - 2), the exponent at least -127
// Both are formed exactly. g and MXFP4's d are powers of two. A quotient y / s is formed as
// y r + y r', r + r' = 1 / s to about 46 bits, rounded once to fp32. s (and 6) has a significand of at most
// 4 bits, so a y whose quotient is not on a border b between two codes is at least one step of y
// off b s, and the quotient more than half a step of b off b: rounding to fp32 never moves it
// onto the border, and a quotient on the border is found there. What follows is the definition to the bit.
#include <mutex>
#include <type_traits>

#include "fp4.cuh"
#include "gemm.h"

namespace gns {
namespace {

constexpr int THREADS = 256;
constexpr int TILE = 128 * 128;  // values that a block of threads works on

// N values in registers as they lie in memory, and their largest magnitude.
template <class T, int N>
struct Block {
  static constexpr int PER = 4 / sizeof(T);  // values of a word
  static constexpr int WORDS = N / PER;
  uint32_t w[WORDS];

  // p: the block's first value, 16-byte aligned; n: how many of them exist
  GNS_DEV void load(const T* p, int n) {
#pragma unroll
    for (int v = 0; v < WORDS / 4; ++v) {
      uint4 u = make_uint4(0u, 0u, 0u, 0u);
      const int left = n - v * 4 * PER;
      if (left >= 4 * PER) {
        u = __ldg(reinterpret_cast<const uint4*>(p) + v);
      } else if (left > 0) {
        uint32_t e[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 4 * PER; ++i) {
          if (i < left) {
            if (sizeof(T) == 4)
              e[i % 4] = __ldg(reinterpret_cast<const uint32_t*>(p) + v * 4 + i);
            else
              e[(i / 2) % 4] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + v * 8 + i) << (16 * (i & 1));
          }
        }
        u = make_uint4(e[0], e[1], e[2], e[3]);
      }
      w[4 * v] = u.x;
      w[4 * v + 1] = u.y;
      w[4 * v + 2] = u.z;
      w[4 * v + 3] = u.w;
    }
  }
  GNS_DEV void store(T* p) const {
#pragma unroll
    for (int v = 0; v < WORDS / 4; ++v)
      *(reinterpret_cast<uint4*>(p) + v) = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
  }
  GNS_DEV uint32_t most() const;  // bits of the largest magnitude in fp32
};

GNS_DEV float2 pair_of(uint32_t w, bf16) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
GNS_DEV float2 pair_of(uint32_t w, __half) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }
// The fp32 bits of a 16-bit magnitude (Inf and NaN stay that).
GNS_DEV uint32_t widen_bits(uint32_t h, bf16) { return h << 16; }
GNS_DEV uint32_t widen_bits(uint32_t h, __half) { return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h))); }
GNS_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

template <class T, int N>
GNS_DEV uint32_t Block<T, N>::most() const {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
    return m;
  } else {  // the bits of a magnitude grow with it, in pairs too
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < WORDS; ++i) m = max_u16x2(m, w[i] & 0x7FFF7FFFu);
    return widen_bits(max(m & 0xFFFFu, m >> 16), T());
  }
}

// The largest finite magnitude of a block whose largest is not finite.
template <class T, int N>
GNS_DEV uint32_t finite_most(const Block<T, N>& b) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < Block<T, N>::WORDS; ++i) {
    uint32_t e[2];
    if constexpr (sizeof(T) == 4) {
      e[0] = e[1] = b.w[i] & 0x7FFFFFFFu;
    } else {
      e[0] = widen_bits(b.w[i] & 0x7FFFu, T());
      e[1] = widen_bits((b.w[i] >> 16) & 0x7FFFu, T());
    }
    for (int j = 0; j < 2; ++j)
      if (e[j] < 0x7F800000u) m = max(m, e[j]);
  }
  return m;
}

// What a block's largest magnitude says: the scale's byte, and the factors of its values' quotients
// (x inv) r + (x inv) r'. A block that holds Inf or NaN: a NaN scale.
struct Scale {
  uint32_t byte;
  float inv, r, rr;
  bool huge;  // quotients beyond fp32 have to be met (a given largest magnitude that is too small)
};

template <int FMT>
GNS_DEV Scale scale_of(uint32_t most, float g) {
  Scale s;
  s.huge = false;
  if (FMT == GNS_MXFP4) {
    const uint32_t e = most >> 23;
    s.byte = e == 255u ? 255u : e < 2u ? 0u : e - 2u;
    s.inv = __uint_as_float((254u - min(s.byte, 253u)) << 23);
    s.r = s.rr = 0.f;
    return s;
  }
  s.inv = g == 0.f ? 0.f : pow2_inverse(g);
  const float top = __uint_as_float(most) * s.inv;
  s.huge = top > 1e30f;
  constexpr float SIXTH = 1.f / 6.f, REST = (float)(1.0 / 6.0 - (double)SIXTH);
  s.byte = most >= 0x7F800000u ? 0x7Fu : s.huge ? 0x7Eu : f_to_e4m3(__fmaf_rn(top, SIXTH, top * REST));
  const float d = e4m3_to_f((uint8_t)s.byte);
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(d));
  // one Newton step's residual: 1 / d = r + r (1 - d r) + O(error^2)
  const float rr = r * __fmaf_rn(-d, r, 1.f);
  const bool none = s.byte == 0u;
  s.r = none ? 0.f : r;
  s.rr = none ? 0.f : rr;
  return s;
}

template <int FMT>
GNS_DEV float2 quotients(float2 x, const Scale& s) {
  float2 y = __fmul2_rn(x, make_float2(s.inv, s.inv));
  if (FMT == GNS_MXFP4) return y;
  if (s.huge) {
    y.x = fminf(fmaxf(y.x, -1e30f), 1e30f);
    y.y = fminf(fmaxf(y.y, -1e30f), 1e30f);
  }
  return __ffma2_rn(y, make_float2(s.r, s.r), __fmul2_rn(y, make_float2(s.rr, s.rr)));
}

template <int FMT>
GNS_DEV bool nan_scale(uint32_t byte) {
  return byte == (FMT == GNS_NVFP4 ? 0x7Fu : 0xFFu);
}

// Codes of 8 values.
template <int FMT>
GNS_DEV uint32_t codes8(const float2 (&x)[4], const Scale& s) {
  const float2 a = quotients<FMT>(x[0], s), b = quotients<FMT>(x[1], s), c = quotients<FMT>(x[2], s),
               d = quotients<FMT>(x[3], s);
  const uint32_t v = f8_to_e2m1(a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y);
  return nan_scale<FMT>(s.byte) ? 0u : v;
}

struct QuantParams {
  const void* x;
  long long ld, stride;
  int rows, cols;
  int tile_rows_log2, tile_cols_log2;
  int tiles_c, tiles_per_mat;
  Fp4Ref q, qt;
  int* status;
};

// The block of values (row, k) of a tile's iteration `it`.
template <int N>
GNS_DEV void block_of(const QuantParams& P, int it, int& row, int& k) {
  const int log2 = P.tile_cols_log2 - (N == 16 ? 4 : 5);
  const int id = it * THREADS + threadIdx.x;
  row = id >> log2;
  k = id & ((1 << log2) - 1);
}

template <class T, int N, int IT>
GNS_DEV void load_tile(const QuantParams& P, int b, int r0, int c0, Block<T, N> (&v)[IT]) {
  const T* m = static_cast<const T*>(P.x) + b * P.stride;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    int row, k;
    block_of<N>(P, it, row, k);
    row += r0;
    const int c = c0 + k * N;
    v[it].load(m + (long long)row * P.ld + c, row < P.rows ? P.cols - c : 0);
  }
}

// The largest finite magnitude of the block's threads' tile, in every thread's hand (bits).
template <class T, int N, int IT>
GNS_DEV uint32_t tile_most(const Block<T, N> (&v)[IT], uint32_t* warps) {
  uint32_t m = 0u;
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    uint32_t a = v[it].most();
    if (a >= 0x7F800000u) a = finite_most(v[it]);
    m = max(m, a);
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) m = max(m, warps[i]);
  return m;
}

// scale[b] = the largest over the matrix's tiles of the tensor scale that the tile alone would
// have: the scale is a monotone function of the largest magnitude, so its maximum is the scale of
// the maximum, in whatever order the tiles arrive. scale is zero before the launch.
template <class T>
__global__ void __launch_bounds__(THREADS) amax_kernel(const __grid_constant__ QuantParams P) {
  constexpr int IT = TILE / THREADS / 16;
  __shared__ uint32_t warps[THREADS / 32];
  const long long tile = blockIdx.x;
  const int b = (int)(tile / P.tiles_per_mat);
  const int t = (int)(tile - (long long)b * P.tiles_per_mat);
  const int tr = t / P.tiles_c;
  Block<T, 16> v[IT];
  load_tile(P, b, tr << P.tile_rows_log2, (t - tr * P.tiles_c) << P.tile_cols_log2, v);
  const uint32_t most = tile_most(v, warps);
  if (threadIdx.x == 0 && most) {
    const uint32_t g = fp4_tensor_scale_bits(most);
    if (P.q.tensor_scale) atomicMax(reinterpret_cast<unsigned int*>(P.q.tensor_scale) + b, g);
    if (P.qt.tensor_scale) atomicMax(reinterpret_cast<unsigned int*>(P.qt.tensor_scale) + b, g);
  }
}

// The scales of matrices whose largest magnitude the caller gives; 1 where it is not a positive finite number.
__global__ void given_scale_kernel(const float* amax, int count, float* scale, float* scale_t) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= count) return;
  const uint32_t a = __float_as_uint(amax[b]);
  const float g = a > 0u && a < 0x7F800000u ? __uint_as_float(fp4_tensor_scale_bits(a)) : 1.f;
  if (scale) scale[b] = g;
  if (scale_t) scale_t[b] = g;
}

// Shared memory for the columns: the tile as it was read, and its transpose's codes and scales.
constexpr int CODE_PITCH = 72;  // bytes of a column's 128 codes: 64, and 8 that spread the banks
template <class T>
constexpr int column_smem() {
  return TILE * (int)sizeof(T) + 128 * CODE_PITCH + 1024;
}

// One tile. ROWS, COLS: what is wanted; with COLS the tile is 128 x 128. CLUSTER: the blocks of the
// cluster hold one whole matrix, and find its largest magnitude among themselves.
//
// Along rows a thread quantises the blocks that it has read, from registers; a row's codes leave as 8
// or 16 bytes a thread, side by side, and the four scales of a scale tile's row as one word. Along columns
// the tile goes through shared memory: a thread takes two columns (16-bit types: a word of a row has both)
// of 16 or 32 rows, and the transpose's codes and scales leave through shared memory in 16-byte pieces.
template <class T, int FMT, bool ROWS, bool COLS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS) quantize_kernel(const __grid_constant__ QuantParams P) {
  constexpr int N = FMT == GNS_NVFP4 ? 16 : 32;
  constexpr int IT = TILE / THREADS / N;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t warps[THREADS / 32];
  __shared__ uint32_t others[8];
  const int tid = threadIdx.x;
  const long long tile = blockIdx.x;
  const int b = (int)(tile / P.tiles_per_mat);
  const int t = (int)(tile - (long long)b * P.tiles_per_mat);
  const int tr = t / P.tiles_c;
  const int r0 = tr << P.tile_rows_log2, c0 = (t - tr * P.tiles_c) << P.tile_cols_log2;
  if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  Block<T, N> v[IT];
  load_tile(P, b, r0, c0, v);
  float g = 1.f;
  if constexpr (FMT == GNS_NVFP4) {
    if constexpr (CLUSTER) {
      uint32_t most = tile_most(v, warps);
      const uint32_t n = P.tiles_per_mat;
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every block of the cluster has started
      if (tid < n)  // this block's to every block of the cluster
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(smem_u32(&others[cluster_ctarank()]), tid)), "r"(most)
                     : "memory");
      cluster_sync_all();
      for (uint32_t i = 0; i < n; ++i) most = max(most, others[i]);
      g = __uint_as_float(fp4_tensor_scale_bits(most));
      if (t == 0 && tid == 0) {
        if (ROWS) P.q.tensor_scale[b] = g;
        if (COLS) P.qt.tensor_scale[b] = g;
      }
    } else {
      g = (ROWS ? P.q : P.qt).tensor_scale[b];
    }
  }
  bool bad = false;
  // a tile of at most 32 rows holds a matrix that has no more: rows 32, 64 and 96 further on are zero
  const bool few = !COLS && P.tile_rows_log2 <= 5;
  T* const xs = reinterpret_cast<T*>(smem);
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    int row, k;
    block_of<N>(P, it, row, k);
    if constexpr (COLS) v[it].store(xs + row * 128 + k * N);
    if constexpr (ROWS) {
      const Scale s = scale_of<FMT>(v[it].most(), g);
      bad |= nan_scale<FMT>(s.byte);
      uint32_t codes[N / 8];
#pragma unroll
      for (int i = 0; i < N / 8; ++i) {
        float2 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (sizeof(T) == 4)
            x[j] = make_float2(__uint_as_float(v[it].w[8 * i + 2 * j]), __uint_as_float(v[it].w[8 * i + 2 * j + 1]));
          else
            x[j] = pair_of(v[it].w[4 * i + j], T());
        }
        codes[i] = codes8<FMT>(x, s);
      }
      const int r = r0 + row, kk = (c0 / N) + k;
      if (r < P.rows && kk * N < (P.cols + 31) / 32 * 32) {  // a row's codes end at a multiple of 32
        uint8_t* o = P.q.codes + b * P.q.stride + r * P.q.ld + kk * (N / 2);
        if (N == 16)
          *reinterpret_cast<uint2*>(o) = make_uint2(codes[0], codes[1]);
        else
          *reinterpret_cast<uint4*>(o) = make_uint4(codes[0], codes[1], codes[N / 8 - 2], codes[N / 8 - 1]);
      }
      // the word of four neighbours' scales; none behind the last row or block
      uint32_t word = r < P.rows && kk * N < P.cols ? s.byte : 0u;
      word |= __shfl_down_sync(0xFFFFFFFFu, word, 1) << 8;
      word |= __shfl_down_sync(0xFFFFFFFFu, word, 2) << 16;
      if ((k & 3) == 0 && (kk >> 2) < P.q.block_tiles) {
        uint8_t* o = P.q.scales + b * P.q.scale_stride + ((long long)(r >> 7) * P.q.block_tiles + (kk >> 2)) * 512 + fp4_scale_at(r, 0);
        if (few)
          *reinterpret_cast<uint4*>(o) = make_uint4(word, 0u, 0u, 0u);
        else
          *reinterpret_cast<uint32_t*>(o) = word;
      }
    }
  }
  if constexpr (ROWS && !COLS) {
    // a scale tile has 128 rows: those behind the tile's rows (a matrix of fewer than 128) are zero
    const int rows = 1 << P.tile_rows_log2, words = (1 << P.tile_cols_log2) / (4 * N);
    const int units = few ? 32 - rows : 128 - rows;
    for (int i = tid; i < units * words; i += THREADS) {
      const int r = rows + i / words, kt = c0 / (4 * N) + i % words;
      if (kt < P.q.block_tiles) {
        uint8_t* o = P.q.scales + b * P.q.scale_stride + (long long)kt * 512 + fp4_scale_at(r, 0);
        if (few)
          *reinterpret_cast<uint4*>(o) = make_uint4(0u, 0u, 0u, 0u);
        else
          *reinterpret_cast<uint32_t*>(o) = 0u;
      }
    }
  }
  if constexpr (COLS) {
    uint8_t* const ct = smem + TILE * sizeof(T);
    uint8_t* const st = ct + 128 * CODE_PITCH;
    __syncthreads();
    constexpr int PER = 4 / sizeof(T);  // columns of a thread
    constexpr int TASKS = 128 / PER * (128 / N);
#pragma unroll 1
    for (int task = tid; task < TASKS; task += THREADS) {
      const int cw = task % (128 / PER), rb = task / (128 / PER);
      const uint32_t* p = reinterpret_cast<const uint32_t*>(xs + rb * N * 128) + cw;
      uint32_t w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = p[i * 128 / PER];
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < N; ++i) m = sizeof(T) == 4 ? max(m, w[i] & 0x7FFFFFFFu) : max_u16x2(m, w[i] & 0x7FFF7FFFu);
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        uint32_t most = m;
        if constexpr (sizeof(T) == 2) most = widen_bits(h ? m >> 16 : m & 0xFFFFu, T());
        const Scale s = scale_of<FMT>(most, g);
        bad |= nan_scale<FMT>(s.byte);
        const int c = cw * PER + h;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
          float2 x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t u = w[8 * i + 2 * j], l = w[8 * i + 2 * j + 1];
            if constexpr (sizeof(T) == 4) {
              x[j] = make_float2(__uint_as_float(u), __uint_as_float(l));
            } else {
              // this column's halves of two rows, in one word
              x[j] = pair_of(__byte_perm(u, l, h ? 0x7632 : 0x5410), T());
            }
          }
          *reinterpret_cast<uint32_t*>(ct + c * CODE_PITCH + rb * (N / 2) + i * 4) = codes8<FMT>(x, s);
        }
        const bool in = c0 + c < P.cols && r0 + rb * N < P.rows;
        st[(rb >> 2) * 512 + fp4_scale_at(c, rb)] = in ? (uint8_t)s.byte : (uint8_t)0;
      }
    }
    __syncthreads();
    // 64 bytes a column; a row of the transpose ends at a multiple of 32 codes
    const int wide = (P.rows + 31) / 32 * 32;
    for (int i = tid; i < 128 * 4; i += THREADS) {
      const int c = i >> 2, u = i & 3;
      if (c0 + c < P.cols && r0 + u * 32 < wide) {
        const uint2 a = *reinterpret_cast<const uint2*>(ct + c * CODE_PITCH + u * 16);
        const uint2 d = *reinterpret_cast<const uint2*>(ct + c * CODE_PITCH + u * 16 + 8);
        *reinterpret_cast<uint4*>(P.qt.codes + b * P.qt.stride + (long long)(c0 + c) * P.qt.ld + (r0 >> 1) + u * 16) =
            make_uint4(a.x, a.y, d.x, d.y);
      }
    }
    constexpr int ST = 128 / N / 4;  // scale tiles of 128 rows
    if (tid < ST * 32) {
      const int kt = r0 / (4 * N) + (tid >> 5);
      if (kt < P.qt.block_tiles)
        *reinterpret_cast<uint4*>(P.qt.scales + b * P.qt.scale_stride + ((long long)(c0 >> 7) * P.qt.block_tiles + kt) * 512 +
                                  (tid & 31) * 16) = *reinterpret_cast<const uint4*>(st + tid * 16);
    }
  }
  if (bad) set_status(P.status, GNS_DEVST_NONFINITE);
}

// v g cut to fp32, its last bit set where something was cut off (round to odd): rounded to a 16-bit type, that is v g
// rounded once. The rest is formed rounded up, so that it is never lost to underflow.
GNS_DEV float times_odd(float v, float g) {
  const float a = fabsf(v), h = fabsf(g), p = __fmul_rz(a, h);
  const uint32_t odd = __fmaf_ru(a, h, -p) > 0.f ? 1u : 0u;
  return copysignf(__uint_as_float(__float_as_uint(p) | odd), v) * copysignf(1.f, g);
}

// The values of a block (those `left` of them that exist). EXACT: g s is exact.
template <class T, int FMT, bool EXACT>
GNS_DEV void put_values(const uint32_t (&codes)[FMT == GNS_NVFP4 ? 2 : 4], float s, float g, T* o, int left) {
  constexpr int N = FMT == GNS_NVFP4 ? 16 : 32;
  const float d = EXACT ? g * s : s;
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __fmul2_rn(e2m1x2_to_f2(codes[i] >> (8 * j)), make_float2(d, d));
      if constexpr (!EXACT)
        v[j] = sizeof(T) == 4 ? make_float2(v[j].x * g, v[j].y * g) : make_float2(times_odd(v[j].x, g), times_odd(v[j].y, g));
    }
    uint32_t w[8];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(j & 1 ? v[j / 2].y : v[j / 2].x);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 h = __float22half2_rn(v[j]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __nv_bfloat162 h = __float22bfloat162_rn(v[j]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
    }
    if (left >= 8 * i + 8) {
      *reinterpret_cast<uint4*>(o + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
      if (sizeof(T) == 4) *(reinterpret_cast<uint4*>(o + 8 * i) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * i + j < left) {
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint32_t*>(o + 8 * i + j) = w[j];
          else
            *reinterpret_cast<uint16_t*>(o + 8 * i + j) = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
    }
  }
}

// A thread takes blocks of a row: 8 or 16 bytes of codes and a scale into 16 or 32 values.
//
// A code times s has at most 6 bits. With g a power of two (what quantisation gives), or none, g s and the values are exact
// in fp32 and the conversion to T rounds once. Another g, or one near fp32's ends, is multiplied last: rounded to
// nearest for fp32, to odd ahead of the rounding to 16 bits. The block's loads come before the question which g it
// is, so that they do not wait for g.
template <class T, int FMT>
__global__ void __launch_bounds__(THREADS) dequantize_kernel(Fp4Ref q, T* out, long long ld, long long stride, int blocks,
                                                             long long total) {
  constexpr int N = FMT == GNS_NVFP4 ? 16 : 32;
  const int b = blockIdx.y;
  const float g = FMT == GNS_NVFP4 ? q.tensor_scale[b] : 1.f;
  for (long long id = (long long)blockIdx.x * THREADS + threadIdx.x; id < total; id += (long long)gridDim.x * THREADS) {
    const int row = total < (1ll << 31) ? (int)((uint32_t)id / (uint32_t)blocks) : (int)(id / blocks);
    const int k = (int)(id - (long long)row * blocks);
    const uint8_t byte = q.scales[b * q.scale_stride + ((long long)(row >> 7) * q.block_tiles + (k >> 2)) * 512 + fp4_scale_at(row, k)];
    const uint8_t* c = q.codes + b * q.stride + row * q.ld + k * (N / 2);
    uint32_t codes[N / 8];
    if (N == 16) {
      const uint2 u = *reinterpret_cast<const uint2*>(c);
      codes[0] = u.x;
      codes[1] = u.y;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(c);
      codes[0] = u.x;
      codes[1] = u.y;
      codes[N / 8 - 2] = u.z;
      codes[N / 8 - 1] = u.w;
    }
    T* o = out + b * stride + row * ld + k * N;
    const int left = q.cols - k * N;
    const float s = fp4_scale_to_f<FMT>(byte);
    // g 0, or a power of two from 2^-126 to 2^118: g s is 0, or at least 2^-135 and below 2^127
    const uint32_t gb = __float_as_uint(g);
    if (FMT == GNS_MXFP4 || gb == 0u || ((gb & 0x7FFFFFu) == 0u && gb >= 1u << 23 && gb <= (127u + 118u) << 23))
      put_values<T, FMT, true>(codes, s, g, o, left);
    else if constexpr (FMT == GNS_NVFP4)
      put_values<T, FMT, false>(codes, s, g, o, left);
  }
}

// ---------------------------------------------------------------------------------------
// host side

int cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return GNS_OK;
  (void)cudaGetLastError();
  return set_error(GNS_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

template <class T, int FMT, bool ROWS, bool COLS, bool CLUSTER>
int launch_tiles(const QuantParams& P, long long tiles, cudaStream_t stream) {
  auto* kernel = quantize_kernel<T, FMT, ROWS, COLS, CLUSTER>;
  const int smem = COLS ? column_smem<T>() : 0;
  if (smem > 48 * 1024) {
    static std::once_flag once[64];
    static cudaError_t opted[64];
    int dev = 0;
    cudaGetDevice(&dev);
    dev = dev < 0 || dev >= 64 ? 0 : dev;
    std::call_once(once[dev], [&] { opted[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (opted[dev] != cudaSuccess) return cuda_status(opted[dev], "cudaFuncSetAttribute");
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CLUSTER ? P.tiles_per_mat : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)tiles, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTER ? 1 : 0;
  profile_count_launch();
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P), "quantize");
}

template <class T, int FMT, bool CLUSTER>
int launch_axes(const QuantParams& P, bool rows, bool cols, long long tiles, cudaStream_t stream) {
  if (rows && cols) return launch_tiles<T, FMT, true, true, CLUSTER>(P, tiles, stream);
  if (cols) return launch_tiles<T, FMT, false, true, CLUSTER>(P, tiles, stream);
  return launch_tiles<T, FMT, true, false, CLUSTER>(P, tiles, stream);
}

// The most tiles of a matrix that is done by one cluster (8 blocks: the portable size).
constexpr int CLUSTER_TILES = 8;

template <class T>
int quantize_typed(const DenseRef& x, long long count, int rows, int cols, int fmt, const Fp4Ref* q, const Fp4Ref* qt,
                   const float* amax, int32_t* status, cudaStream_t stream) {
  QuantParams P = {};
  P.x = x.ptr;
  P.ld = x.ld;
  P.stride = x.stride;
  P.rows = rows;
  P.cols = cols;
  if (q) P.q = *q;
  if (qt) P.qt = *qt;
  P.status = status;
  P.tile_rows_log2 = 7;
  // along rows alone, the tile of a matrix of few rows is as wide as it has rows to spare, up to
  // 4096 columns
  if (!qt)
    while (P.tile_rows_log2 > 2 && (1 << (P.tile_rows_log2 - 1)) >= rows) --P.tile_rows_log2;
  P.tile_cols_log2 = 14 - P.tile_rows_log2;
  P.tiles_c = (cols + (1 << P.tile_cols_log2) - 1) >> P.tile_cols_log2;
  const long long per_mat = (long long)P.tiles_c * ((rows + (1 << P.tile_rows_log2) - 1) >> P.tile_rows_log2);
  P.tiles_per_mat = (int)per_mat;
  const long long tiles = count * per_mat;
  if (tiles > 0x7FFFFFFFll) return set_error(GNS_ERR_UNSUPPORTED, "quantize: more than 2^31 - 1 tiles of 128 x 128 in a batch");
  const bool own = fmt == GNS_NVFP4 && !amax;
  if (fmt == GNS_NVFP4 && amax) {
    given_scale_kernel<<<(unsigned)((count + 127) / 128), 128, 0, stream>>>(amax, (int)count, P.q.tensor_scale, P.qt.tensor_scale);
    profile_count_launch();
    if (int rc = cuda_status(cudaGetLastError(), "quantize")) return rc;
  } else if (own && per_mat <= CLUSTER_TILES) {
    return launch_axes<T, GNS_NVFP4, true>(P, q, qt, tiles, stream);
  } else if (own) {
    // the largest magnitudes of the whole batch, then the codes: in groups of matrices that L2 still holds for the second
    // reading, launch by launch, it took longer (16 of 2048 x 8192 bf16 along both axes 420 us in groups of 48 MB, 377 of
    // 96 MB, 326 at once; 100 of 700 x 900 along rows 86, 80, 73)
    for (float* s : {P.q.tensor_scale, P.qt.tensor_scale})
      if (s)
        if (int rc = cuda_status(cudaMemsetAsync(s, 0, sizeof(float) * count, stream), "quantize")) return rc;
    amax_kernel<T><<<(unsigned)tiles, THREADS, 0, stream>>>(P);
    profile_count_launch();
    if (int rc = cuda_status(cudaGetLastError(), "quantize")) return rc;
  }
  return fmt == GNS_NVFP4 ? launch_axes<T, GNS_NVFP4, false>(P, q, qt, tiles, stream)
                          : launch_axes<T, GNS_MXFP4, false>(P, q, qt, tiles, stream);
}

template <class T>
int dequantize_typed(const Fp4Ref& q, long long count, int fmt, const DenseRef& out, cudaStream_t stream) {
  const int blocks = (q.cols + fp4_block(fmt) - 1) / fp4_block(fmt);
  const long long total = (long long)q.rows * blocks;
  const long long per = (total + THREADS - 1) / THREADS;
  const dim3 grid((unsigned)(per < (1 << 20) ? per : 1 << 20), (unsigned)count);
  T* o = static_cast<T*>(out.ptr);
  if (fmt == GNS_NVFP4)
    dequantize_kernel<T, GNS_NVFP4><<<grid, THREADS, 0, stream>>>(q, o, out.ld, out.stride, blocks, total);
  else
    dequantize_kernel<T, GNS_MXFP4><<<grid, THREADS, 0, stream>>>(q, o, out.ld, out.stride, blocks, total);
  profile_count_launch();
  return cuda_status(cudaGetLastError(), "dequantize");
}

}  // namespace

int fp4_quantize_launch(const DenseRef& x, int64_t count, int64_t rows, int64_t cols, int fmt, const Fp4Ref* q,
                        const Fp4Ref* qt, const float* amax, int32_t* dev_status, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x.dtype == GNS_F32) return quantize_typed<float>(x, count, (int)rows, (int)cols, fmt, q, qt, amax, dev_status, s);
  if (x.dtype == GNS_F16) return quantize_typed<__half>(x, count, (int)rows, (int)cols, fmt, q, qt, amax, dev_status, s);
  return quantize_typed<bf16>(x, count, (int)rows, (int)cols, fmt, q, qt, amax, dev_status, s);
}

int fp4_dequantize_launch(const Fp4Ref& q, int64_t count, int fmt, const DenseRef& out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out.dtype == GNS_F32) return dequantize_typed<float>(q, count, fmt, out, s);
  if (out.dtype == GNS_F16) return dequantize_typed<__half>(q, count, fmt, out, s);
  return dequantize_typed<bf16>(q, count, fmt, out, s);
}

}  // namespace gns
