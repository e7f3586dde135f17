// Operators over lists of tensors: the global norm of a list of gradients with the scale that
// clips them (gns_grad_norm), the clipping itself (gns_clip_grads) and the AdamW step
// (gns_adamw_step). All three stream every tensor once through the SMs and are bound by HBM
// bandwidth on long lists and by launch latency on short ones.
//
// A launch carries the descriptors of many tensors in its parameters (no descriptor table in
// device memory, so a call can be captured into a graph and needs no copy). The work is cut
// into chunks of THREADS * UNITS units of 8 consecutive elements, no chunk crossing a tensor,
// and block i takes chunks i, i + gridDim.x, ...
//
// Two layouts: a FlatList holds tensors whose elements lie without gaps in every role (a role
// is one of the buffers an operator walks in step: gradients; weights, moments, master ...);
// a RowList holds batches of rows with a pitch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>

#include "../../include/gns.h"
#include "common.cuh"
#include "gemm.h"

namespace gns {

int set_error(int code, const std::string& msg);  // sets gns_last_error(); defined with the C ABI

namespace {

constexpr int THREADS = 256;
constexpr int MAX_GRID = 1216;  // blocks of one norm launch, and its partial sums (8 for each of 152 SMs)

// ---------------------------------------------------------------------------------------
// lists as kernel parameters (at most 32,764 bytes of parameters a launch)

// start[i]: the launch's first chunk of tensor i, start[count]: all chunks. type: the GNS_ types
// of roles 0 and 1 in bits 0-1 and 2-3, bit 4 set when the tensor has every role.
template <int R, int CAP>
struct FlatList {
  static constexpr bool kRows = false;
  static constexpr int kRoles = R, kCap = CAP;
  void* ptr[R][CAP];
  long long n[CAP];
  int start[CAP + 1];
  unsigned char type[CAP];
  unsigned char align[CAP];  // what load_unit takes
  unsigned char head[CAP];   // elements before the first unit
  int count;
};

template <int R, int CAP>
struct RowList {
  static constexpr bool kRows = true;
  static constexpr int kRoles = R, kCap = CAP;
  void* ptr[R][CAP];
  long long ld[R][CAP], stride[R][CAP];
  int rows[CAP];   // of one matrix
  int nrows[CAP];  // of all matrices
  int cols[CAP];
  int start[CAP + 1];
  unsigned char type[CAP];
  unsigned char align[CAP];
  int count;
};

// ---------------------------------------------------------------------------------------
// units: 8 consecutive elements of one role, as stored

struct Unit {
  uint32_t w[8];  // 8 f32, or 8 16-bit values in w[0..3]
};

GNS_DEV void ld_v8(uint32_t (&w)[8], const void* p) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
GNS_DEV void st_v8(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
               : "memory");
}
GNS_DEV void ld_v4(uint32_t* w, const void* p) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p)
               : "memory");
}
GNS_DEV void st_v4(void* p, const uint32_t* w) {
  asm volatile("st.global.v4.b32 [%4], {%0, %1, %2, %3};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "l"(p)
               : "memory");
}

// align: 2 = every unit starts on 8 elements' bytes, 1 = on 16 bytes, 0 = on an element.
// Elements from `valid` on are neither read nor written, and read as zero.
GNS_DEV void load_unit(Unit& u, const void* base, long long off, bool f32, int align, int valid) {
  if (f32) {
    const uint32_t* p = static_cast<const uint32_t*>(base) + off;
    if (valid == 8 && align == 2) {
      ld_v8(u.w, p);
    } else if (valid == 8 && align == 1) {
      ld_v4(u.w, p);
      ld_v4(u.w + 4, p + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u.w[e] = e < valid ? p[e] : 0u;
    }
  } else {
    const unsigned short* p = static_cast<const unsigned short*>(base) + off;
    if (valid == 8 && align) {
      ld_v4(u.w, p);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = 2 * e < valid ? p[2 * e] : 0u, hi = 2 * e + 1 < valid ? p[2 * e + 1] : 0u;
        u.w[e] = lo | (hi << 16);
      }
    }
  }
}

GNS_DEV void store_unit(const Unit& u, void* base, long long off, bool f32, int align, int valid) {
  if (f32) {
    uint32_t* p = static_cast<uint32_t*>(base) + off;
    if (valid == 8 && align == 2) {
      st_v8(p, u.w);
    } else if (valid == 8 && align == 1) {
      st_v4(p, u.w);
      st_v4(p + 4, u.w + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) p[e] = u.w[e];
    }
  } else {
    unsigned short* p = static_cast<unsigned short*>(base) + off;
    if (valid == 8 && align) {
      st_v4(p, u.w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) p[e] = static_cast<unsigned short>(u.w[e / 2] >> (16 * (e & 1)));
    }
  }
}

GNS_DEV void unpack(float (&x)[8], const Unit& u, int dt) {
  if (dt == GNS_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(u.w[e]);
  } else if (dt == GNS_BF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(u.w[e] << 16);
      x[2 * e + 1] = __uint_as_float(u.w[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u.w[e]));
      x[2 * e] = f.x;
      x[2 * e + 1] = f.y;
    }
  }
}

// One rounding to the nearest value of the stored type.
GNS_DEV void pack(Unit& u, const float (&x)[8], int dt) {
  if (dt == GNS_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) u.w[e] = __float_as_uint(x[e]);
  } else if (dt == GNS_BF16) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      u.w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 h = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
      u.w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
}

// ---------------------------------------------------------------------------------------
// walking a list

// The tensor that holds a chunk: the last one that starts at or before it.
template <class L>
GNS_DEV int find_tensor(const L& l, int chunk) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.start[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Where unit j of a chunk of tensor t lies in every role; returns how many of its 8 elements
// exist (0: none).
template <int UNITS, int R, int CAP>
GNS_DEV int locate(const FlatList<R, CAP>& l, int t, int chunk, int j, long long (&off)[R]) {
  const long long o = l.head[t] + (static_cast<long long>(chunk - l.start[t]) * (THREADS * UNITS) + j) * 8;
#pragma unroll
  for (int r = 0; r < R; ++r) off[r] = o;
  const long long left = l.n[t] - o;
  return left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
}

template <int UNITS, int R, int CAP>
GNS_DEV int locate(const RowList<R, CAP>& l, int t, int chunk, int j, long long (&off)[R]) {
  const uint32_t per_row = (static_cast<uint32_t>(l.cols[t]) + 7u) >> 3;
  const long long u0 = static_cast<long long>(chunk - l.start[t]) * (THREADS * UNITS);
  const long long row0 = u0 / per_row;
  const uint32_t x = static_cast<uint32_t>(u0 - row0 * per_row) + static_cast<uint32_t>(j);
  const uint32_t q = x / per_row;
  const long long row = row0 + q;
  if (row >= l.nrows[t]) return 0;
  const uint32_t c = (x - q * per_row) * 8u;
  const uint32_t b = static_cast<uint32_t>(row) / static_cast<uint32_t>(l.rows[t]);
  const uint32_t i = static_cast<uint32_t>(row) - b * static_cast<uint32_t>(l.rows[t]);
#pragma unroll
  for (int r = 0; r < R; ++r) off[r] = b * l.stride[r][t] + i * l.ld[r][t] + c;
  return static_cast<int>(min(8u, static_cast<uint32_t>(l.cols[t]) - c));
}

// Elements before the first unit of a flat tensor: one for each of the first threads of its
// first chunk, where `head_here` is the number of them.
template <int R, int CAP>
GNS_DEV int head_here(const FlatList<R, CAP>& l, int t, int chunk) {
  return chunk == l.start[t] ? l.head[t] : 0;
}
template <int R, int CAP>
GNS_DEV int head_here(const RowList<R, CAP>&, int, int) {
  return 0;
}

// ---------------------------------------------------------------------------------------
// reductions over a block, in a fixed order; every thread gets the result

GNS_DEV double block_sum(double v) {
  __shared__ double part[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s += part[w];
  return s;
}

GNS_DEV uint32_t block_max(uint32_t v) {
  __shared__ uint32_t part[THREADS / 32];
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) m = max(m, part[w]);
  return m;
}

// ---------------------------------------------------------------------------------------
// norm: sqrt(sum x^2) over the whole list, or max |x|

constexpr int NORM_UNITS = 4;

// Calls f(unit, type) for every unit of this block's chunks.
template <int UNITS, class L, class F>
GNS_DEV void for_units(const L& l, F f) {
  const int total = l.start[l.count];
  int chunk = blockIdx.x;
  if (chunk >= total) return;
  int t = find_tensor(l, chunk);
  for (; chunk < total; chunk += gridDim.x) {
    while (l.start[t + 1] <= chunk) ++t;
    const int dt = l.type[t] & 3, align = l.align[t];
    const void* p = l.ptr[0][t];
    Unit u[UNITS];
#pragma unroll
    for (int k = 0; k < UNITS; ++k) {
      long long off[1];
      const int valid = locate<UNITS>(l, t, chunk, k * THREADS + static_cast<int>(threadIdx.x), off);
      load_unit(u[k], p, off[0], dt == GNS_F32, align, valid);
    }
#pragma unroll
    for (int k = 0; k < UNITS; ++k) f(u[k], dt);
    if (static_cast<int>(threadIdx.x) < head_here(l, t, chunk)) {
      load_unit(u[0], p, threadIdx.x, dt == GNS_F32, 0, 1);
      f(u[0], dt);
    }
  }
}

// Sum of (pre x)^2 over this block's chunks: 8 squares at a time in f32, these sums in f64.
template <class L>
GNS_DEV double sum_squares(const L& l, float pre, uint32_t* bits) {
  double s = 0.0;
  for_units<NORM_UNITS>(l, [&](const Unit& u, int dt) {
    float x[8];
    unpack(x, u, dt);
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = x[e] * pre;
      q = fmaf(v, v, q);
      *bits |= __float_as_uint(x[e]);
    }
    s += static_cast<double>(q);
  });
  return s;
}

// part[blockIdx.x] = the block's sum of squares (inf = 0) or largest magnitude (inf = 1).
//
// Squares of f32 and bf16 values leave f32's range long before the values do (above 2^64, below
// 2^-63). A block whose sum says that this has happened (it is not finite, or below 2^-80 though
// some value is not zero) sums once more with the values scaled by 2^-100 or 2^100, which is
// exact for every value that counts: the largest magnitudes become at most 2^28, and where the
// sum lies below 2^-80 none is above 2^-40, so they become at most 2^60. f64 holds the result.
template <class L>
__global__ void __launch_bounds__(THREADS) norm_part_kernel(const __grid_constant__ L l, int inf, double* part) {
  if (inf) {
    uint32_t m = 0;  // magnitudes order as their bits do, with every NaN above infinity
    for_units<NORM_UNITS>(l, [&](const Unit& u, int dt) {
      float x[8];
      unpack(x, u, dt);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
    });
    m = block_max(m);
    if (threadIdx.x == 0) part[blockIdx.x] = static_cast<double>(__uint_as_float(m));
    return;
  }
  uint32_t bits = 0;
  double s = block_sum(sum_squares(l, 1.f, &bits));
  const int any = __syncthreads_or((bits & 0x7fffffffu) != 0);
  if (!(s <= 1e38))
    s = block_sum(sum_squares(l, 0x1p-100f, &bits)) * 0x1p200;
  else if (s < 0x1p-80 && any)
    s = block_sum(sum_squares(l, 0x1p100f, &bits)) * 0x1p-200;
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// What a norm call leaves in result[0] and result[1], from its partial sums.
struct Finish {
  const double* part;
  int nparts;
  int inf;
  float max_norm;  // infinity: no clipping
  float eps;
};

GNS_DEV void finish_norm(const Finish& f, float* norm, float* scale) {
  double n = 0.0;
  if (f.inf) {
    uint32_t m = 0;
    for (int i = threadIdx.x; i < f.nparts; i += THREADS) m = max(m, __float_as_uint(static_cast<float>(f.part[i])));
    n = static_cast<double>(__uint_as_float(block_max(m)));
  } else {
    for (int i = threadIdx.x; i < f.nparts; i += THREADS) n += f.part[i];
    n = sqrt(block_sum(n));
  }
  *norm = static_cast<float>(n);
  const double c = static_cast<double>(f.max_norm) / (n + static_cast<double>(f.eps));
  *scale = isinf(f.max_norm) || c >= 1.0 ? 1.f : static_cast<float>(c);  // a NaN norm gives a NaN scale
}

__global__ void __launch_bounds__(THREADS) norm_finish_kernel(Finish f, float* result, int* status) {
  float norm, scale;
  finish_norm(f, &norm, &scale);
  if (threadIdx.x == 0) {
    result[0] = norm;
    result[1] = scale;
    if (!isfinite(norm)) set_status(status, GNS_DEVST_NONFINITE);
  }
}

// ---------------------------------------------------------------------------------------
// clipping: out = round(scale * g); roles: gradient, output (the same pointers in place)

constexpr int CLIP_UNITS = 2;

template <class L>
__global__ void __launch_bounds__(THREADS) clip_kernel(const __grid_constant__ L l, const float* result, int in_place) {
  const float scale = result[1];
  if (in_place && scale == 1.f) return;  // g * 1 is g
  const int total = l.start[l.count];
  int chunk = blockIdx.x;
  if (chunk >= total) return;
  int t = find_tensor(l, chunk);
  for (; chunk < total; chunk += gridDim.x) {
    while (l.start[t + 1] <= chunk) ++t;
    const int dt = l.type[t] & 3, align = l.align[t];
    const bool f32 = dt == GNS_F32;
    Unit u[CLIP_UNITS];
    long long off[CLIP_UNITS][2];
    int valid[CLIP_UNITS];
    float x[8];
#pragma unroll
    for (int k = 0; k < CLIP_UNITS; ++k) {
      valid[k] = locate<CLIP_UNITS>(l, t, chunk, k * THREADS + static_cast<int>(threadIdx.x), off[k]);
      load_unit(u[k], l.ptr[0][t], off[k][0], f32, align, valid[k]);
    }
#pragma unroll
    for (int k = 0; k < CLIP_UNITS; ++k) {
      unpack(x, u[k], dt);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= scale;
      pack(u[k], x, dt);
      store_unit(u[k], l.ptr[1][t], off[k][1], f32, align, valid[k]);
    }
    if (static_cast<int>(threadIdx.x) < head_here(l, t, chunk)) {
      load_unit(u[0], l.ptr[0][t], threadIdx.x, f32, 0, 1);
      unpack(x, u[0], dt);
      x[0] *= scale;
      pack(u[0], x, dt);
      store_unit(u[0], l.ptr[1][t], threadIdx.x, f32, 0, 1);
    }
  }
}

// ---------------------------------------------------------------------------------------
// AdamW; roles: W, G, M, V, master. Type bits 0-1: W, 2-3: G, 4: has a master.

struct AdamwArgs {
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float decay;  // 1 - lr weight_decay
  float lr, eps;
  float step_size;   // lr / (1 - beta1^t)
  float rsqrt_bc2;   // 1 / sqrt(1 - beta2^t)
  float log_beta1, log_beta2;
  const float* grad_scale;  // nullable
  const int* step;          // nullable: t on the device instead of step_size and rsqrt_bc2
  int* status;
};

struct AdamwStep {
  float scale, step_size, rsqrt_bc2;
};

GNS_DEV void adamw_unit(float (&w)[8], float (&g)[8], float (&m)[8], float (&v)[8], const AdamwArgs& a,
                        const AdamwStep& s, int valid, bool* bad) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float ge = g[e] * s.scale;
    m[e] = fmaf(a.beta1, m[e], a.one_minus_beta1 * ge);
    v[e] = fmaf(a.beta2, v[e], a.one_minus_beta2 * ge * ge);
    const float denom = fmaf(sqrtf(v[e]), s.rsqrt_bc2, a.eps);
    w[e] = fmaf(-s.step_size, m[e] / denom, a.decay * w[e]);
    *bad |= e < valid && !isfinite(w[e]);
  }
}

template <class L>
GNS_DEV void adamw_at(const L& l, int t, const long long (&off)[5], int align, int valid, const AdamwArgs& a,
                      const AdamwStep& s, bool* bad) {
  const int wt = l.type[t] & 3, gt = (l.type[t] >> 2) & 3;
  const bool master = l.type[t] & 16;
  Unit uw, ug, um, uv;
  if (master)
    load_unit(uw, l.ptr[4][t], off[4], true, align, valid);
  else
    load_unit(uw, l.ptr[0][t], off[0], wt == GNS_F32, align, valid);
  load_unit(ug, l.ptr[1][t], off[1], gt == GNS_F32, align, valid);
  load_unit(um, l.ptr[2][t], off[2], true, align, valid);
  load_unit(uv, l.ptr[3][t], off[3], true, align, valid);
  float w[8], g[8], m[8], v[8];
  unpack(w, uw, master ? (int)GNS_F32 : wt);
  unpack(g, ug, gt);
  unpack(m, um, GNS_F32);
  unpack(v, uv, GNS_F32);
  adamw_unit(w, g, m, v, a, s, valid, bad);
  pack(um, m, GNS_F32);
  store_unit(um, l.ptr[2][t], off[2], true, align, valid);
  pack(uv, v, GNS_F32);
  store_unit(uv, l.ptr[3][t], off[3], true, align, valid);
  if (master) {
    pack(um, w, GNS_F32);
    store_unit(um, l.ptr[4][t], off[4], true, align, valid);
  }
  pack(uw, w, wt);
  store_unit(uw, l.ptr[0][t], off[0], wt == GNS_F32, align, valid);
}

template <class L>
__global__ void __launch_bounds__(THREADS) adamw_kernel(const __grid_constant__ L l, const __grid_constant__ AdamwArgs a) {
  const int total = l.start[l.count];
  int chunk = blockIdx.x;
  if (chunk >= total) return;
  AdamwStep s;
  s.scale = a.grad_scale ? *a.grad_scale : 1.f;
  s.step_size = a.step_size;
  s.rsqrt_bc2 = a.rsqrt_bc2;
  if (a.step) {
    const float n = static_cast<float>(max(*a.step, 1));
    s.step_size = a.lr / -expm1f(n * a.log_beta1);
    s.rsqrt_bc2 = 1.f / sqrtf(-expm1f(n * a.log_beta2));
  }
  bool bad = false;
  int t = find_tensor(l, chunk);
  for (; chunk < total; chunk += gridDim.x) {
    while (l.start[t + 1] <= chunk) ++t;
    long long off[5];
    const int valid = locate<1>(l, t, chunk, threadIdx.x, off);
    if (valid) adamw_at(l, t, off, l.align[t], valid, a, s, &bad);
    if (static_cast<int>(threadIdx.x) < head_here(l, t, chunk)) {
#pragma unroll
      for (int r = 0; r < 5; ++r) off[r] = threadIdx.x;
      adamw_at(l, t, off, 0, 1, a, s, &bad);
    }
  }
  if (bad) set_status(a.status, GNS_DEVST_NONFINITE);
}

// ---------------------------------------------------------------------------------------
// host: checks and list building

int size_of(int dt) { return dt == GNS_F32 ? 4 : 2; }

int fail(int code, const char* what, int i, const char* why) {
  return set_error(code, std::string(what) + "[" + std::to_string(i) + "]: " + why);
}

bool empty(const gns_tensor& t) { return t.x.count == 0 || t.x.rows == 0 || t.x.cols == 0; }

bool flat(const gns_tensor& t) {
  const gns_batch& x = t.x;
  return (x.rows == 1 || x.ld == x.cols) && (x.count == 1 || x.stride == x.rows * x.cols);
}

int check_tensor(const gns_tensor& t, const char* what, int i) {
  const gns_batch& x = t.x;
  if (t.dtype != GNS_BF16 && t.dtype != GNS_F16 && t.dtype != GNS_F32) return fail(GNS_ERR_INVALID, what, i, "unknown dtype");
  if (x.count < 0 || x.rows < 0 || x.cols < 0) return fail(GNS_ERR_INVALID, what, i, "count, rows and cols must be >= 0");
  if (empty(t)) return GNS_OK;
  if (!x.ptr) return fail(GNS_ERR_INVALID, what, i, "null data pointer");
  if (reinterpret_cast<uintptr_t>(x.ptr) % size_of(t.dtype))
    return fail(GNS_ERR_INVALID, what, i, "pointer must be aligned to an element");
  constexpr int64_t most = int64_t(1) << 40;
  if (x.count > most || x.rows > most || x.cols > most || x.rows > most / x.count || x.cols > most / (x.count * x.rows))
    return fail(GNS_ERR_INVALID, what, i, "more than 2^40 elements");
  if (x.rows > 1 && (x.ld < x.cols || x.ld > most)) return fail(GNS_ERR_INVALID, what, i, "ld must lie in [cols, 2^40]");
  if (x.count > 1) {
    const int64_t last = x.rows > 1 ? (x.rows - 1) * x.ld : 0;
    if (x.rows > 1 && x.ld > most / x.rows) return fail(GNS_ERR_INVALID, what, i, "a matrix spans more than 2^40 elements");
    if (x.stride < last + x.cols || x.stride > most) return fail(GNS_ERR_INVALID, what, i, "stride: matrices overlap, or lie over 2^40 elements apart");
  }
  if (!flat(t) && (x.count * x.rows > 0x7fffffff || x.cols > 0x7fffffff))
    return fail(GNS_ERR_UNSUPPORTED, what, i, "rows with a pitch: at most 2^31 - 1 rows and columns");
  return GNS_OK;
}

bool same_shape(const gns_tensor& a, const gns_tensor& b) {
  return a.x.count == b.x.count && a.x.rows == b.x.rows && a.x.cols == b.x.cols;
}

// One operator's list: role r of tensor i is role[r][i]; role 4 of AdamW (the master) may be
// absent, as a whole or tensor by tensor.
struct Roles {
  const gns_tensor* role[5];
  int nroles;
  int n;
  bool has(int r, int i) const { return role[r] && !empty(role[r][i]); }
  bool is_flat(int i) const {
    for (int r = 0; r < nroles; ++r)
      if (has(r, i) && !flat(role[r][i])) return false;
    return true;
  }
  unsigned char type(int i) const {
    unsigned t = role[0][i].dtype;
    if (nroles > 1) t |= role[1][i].dtype << 2;
    if (nroles == 5 && has(4, i)) t |= 16;
    return static_cast<unsigned char>(t);
  }
};

// Whether every role of tensor i, `skip` elements in, starts on `bytes(r)`: 8 elements' bytes
// (level 2) or 16 bytes (level 1).
bool aligned(const Roles& a, int i, int skip, int level, bool rows) {
  for (int r = 0; r < a.nroles; ++r) {
    if (!a.has(r, i)) continue;
    const gns_tensor& t = a.role[r][i];
    const int es = size_of(t.dtype), need = level == 2 ? 8 * es : 16;
    if ((reinterpret_cast<uintptr_t>(t.x.ptr) + static_cast<uintptr_t>(skip) * es) % need) return false;
    if (rows && t.x.rows > 1 && (t.x.ld * es) % need) return false;
    if (rows && t.x.count > 1 && (t.x.stride * es) % need) return false;
  }
  return true;
}

// Fills entry k of a launch's list with tensor i; the number of its units of 8 elements.
template <int R, int CAP>
int64_t put(FlatList<R, CAP>* l, int k, const Roles& a, int i) {
  const gns_batch& x = a.role[0][i].x;
  const int64_t n = x.count * x.rows * x.cols;
  int head = 0, align = 0;
  for (int level = 2; level >= 1 && !align; --level)
    for (int h = 0; h < 8 && !align; ++h)
      if (aligned(a, i, h, level, false)) {
        align = level;
        head = h;
      }
  if (head > n) head = static_cast<int>(n);
  l->n[k] = n;
  l->head[k] = static_cast<unsigned char>(head);
  l->align[k] = static_cast<unsigned char>(align);
  return std::max<int64_t>(1, (n - head + 7) / 8);
}

template <int R, int CAP>
int64_t put(RowList<R, CAP>* l, int k, const Roles& a, int i) {
  const gns_batch& x = a.role[0][i].x;
  l->rows[k] = static_cast<int>(x.rows);
  l->nrows[k] = static_cast<int>(x.count * x.rows);
  l->cols[k] = static_cast<int>(x.cols);
  for (int r = 0; r < R; ++r) {
    const bool has = a.has(r, i);
    l->ld[r][k] = has && a.role[r][i].x.rows > 1 ? a.role[r][i].x.ld : 0;
    l->stride[r][k] = has && a.role[r][i].x.count > 1 ? a.role[r][i].x.stride : 0;
  }
  l->align[k] = static_cast<unsigned char>(aligned(a, i, 0, 2, true) ? 2 : aligned(a, i, 0, 1, true) ? 1 : 0);
  return x.count * x.rows * ((x.cols + 7) / 8);
}

// Collects the tensors with is_flat() == !L::kRows from `from` on, until the list is full or
// its chunks reach 2^30; returns the first tensor left over (a.n: none).
template <class L>
int fill(L* l, const Roles& a, int from, int64_t chunk_units) {
  int k = 0, i = from;
  int64_t chunks = 0;
  for (; i < a.n; ++i) {
    if (empty(a.role[0][i]) || a.is_flat(i) == L::kRows) continue;
    if (k == L::kCap) break;
    const int64_t units = put(l, k, a, i);
    const int64_t c = (units + chunk_units - 1) / chunk_units;
    if (k && chunks + c > (1 << 30)) break;
    for (int r = 0; r < L::kRoles; ++r) l->ptr[r][k] = a.has(r, i) ? a.role[r][i].x.ptr : nullptr;
    l->type[k] = a.type(i);
    l->start[k] = static_cast<int>(chunks);
    chunks += c;
    ++k;
  }
  l->start[k] = static_cast<int>(chunks);
  l->count = k;
  return i;
}

// Lists of one launch: how many tensors its parameters hold.
constexpr int NORM_FLAT = 1024, NORM_ROWS = 512, CLIP_FLAT = 768, CLIP_ROWS = 384, ADAMW_FLAT = 512, ADAMW_ROWS = 192;

static_assert(sizeof(FlatList<1, NORM_FLAT>) < 32000 && sizeof(RowList<1, NORM_ROWS>) < 32000, "kernel parameters");
static_assert(sizeof(FlatList<2, CLIP_FLAT>) < 32000 && sizeof(RowList<2, CLIP_ROWS>) < 32000, "kernel parameters");
static_assert(sizeof(FlatList<5, ADAMW_FLAT>) < 32000 && sizeof(RowList<5, ADAMW_ROWS>) < 32000, "kernel parameters");

// Launches f(list) for every launch that the tensors of one layout need.
template <class L, class F>
int each_list(const Roles& a, int64_t chunk_units, F f) {
  L l;
  for (int i = 0; i < a.n;) {
    i = fill(&l, a, i, chunk_units);
    if (!l.count) break;
    const int rc = f(l);
    if (rc) return rc;
  }
  return GNS_OK;
}

int launched(const char* what) {
  profile_count_launch();
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? GNS_OK : set_error(GNS_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

int grid_for(int chunks, int per_sm) { return std::max(1, std::min({chunks, device_sm_count() * per_sm, MAX_GRID})); }

size_t list_workspace(int n) {
  // at most one launch for every full list of each layout, and one more of each
  const size_t launches = static_cast<size_t>(n) / NORM_FLAT + static_cast<size_t>(n) / NORM_ROWS + 2;
  return launches * MAX_GRID * sizeof(double) + 256;
}

// The checks and the partial sums of a norm call; *f is ready for the kernel that finishes it.
int norm_parts(const gns_tensor* g, int n, int norm_type, float max_norm, float eps, float* result, void* ws,
               size_t ws_bytes, void* stream, Finish* f) {
  if (!g || !result) return set_error(GNS_ERR_INVALID, "null argument");
  if (n < 1) return set_error(GNS_ERR_INVALID, "need at least one tensor");
  if (norm_type != GNS_NORM_L2 && norm_type != GNS_NORM_INF) return set_error(GNS_ERR_INVALID, "unknown norm type");
  if (!(max_norm >= 0.f)) return set_error(GNS_ERR_INVALID, "max_norm must be >= 0 (infinity: no clipping)");
  if (!(eps >= 0.f) || !std::isfinite(eps)) return set_error(GNS_ERR_INVALID, "eps must be finite and >= 0");
  if (reinterpret_cast<uintptr_t>(result) % 4) return set_error(GNS_ERR_INVALID, "result: unaligned");
  for (int i = 0; i < n; ++i)
    if (int rc = check_tensor(g[i], "grads", i)) return rc;
  if (!ws) return set_error(GNS_ERR_WORKSPACE, "null workspace");
  if (reinterpret_cast<uintptr_t>(ws) % 256) return set_error(GNS_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < list_workspace(n))
    return set_error(GNS_ERR_WORKSPACE, "workspace too small: need " + std::to_string(list_workspace(n)) + " bytes");
  double* part = static_cast<double*>(ws);
  int nparts = 0;
  const int inf = norm_type == GNS_NORM_INF;
  const Roles a = {{g}, 1, n};
  auto go = [&](const auto& l) {
    const int grid = grid_for(l.start[l.count], 8);
    norm_part_kernel<<<grid, THREADS, 0, static_cast<cudaStream_t>(stream)>>>(l, inf, part + nparts);
    nparts += grid;
    return launched("grad norm");
  };
  int rc = each_list<FlatList<1, NORM_FLAT>>(a, THREADS * NORM_UNITS, go);
  if (!rc) rc = each_list<RowList<1, NORM_ROWS>>(a, THREADS * NORM_UNITS, go);
  *f = {part, nparts, inf, max_norm, eps};
  return rc;
}

int finish_launch(const Finish& f, float* result, int32_t* dev_status, void* stream) {
  norm_finish_kernel<<<1, THREADS, 0, static_cast<cudaStream_t>(stream)>>>(f, result, dev_status);
  return launched("grad norm");
}

int grad_norm(const gns_tensor* g, int n, int norm_type, float max_norm, float eps, float* result, void* ws,
              size_t ws_bytes, int32_t* dev_status, void* stream) {
  Finish f;
  if (int rc = norm_parts(g, n, norm_type, max_norm, eps, result, ws, ws_bytes, stream, &f)) return rc;
  return finish_launch(f, result, dev_status, stream);
}

int clip_grads(const gns_tensor* g, const gns_tensor* out, int n, int norm_type, float max_norm, float eps,
               float* result, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (!g) return set_error(GNS_ERR_INVALID, "null argument");
  int in_place = 1;
  for (int i = 0; out && i < n; ++i) {
    if (int rc = check_tensor(g[i], "grads", i)) return rc;
    if (int rc = check_tensor(out[i], "outs", i)) return rc;
    if (!same_shape(g[i], out[i])) return fail(GNS_ERR_INVALID, "outs", i, "must have its gradient's shape");
    if (g[i].dtype != out[i].dtype) return fail(GNS_ERR_INVALID, "outs", i, "must have its gradient's dtype");
    if (empty(g[i])) continue;
    if (g[i].x.ptr != out[i].x.ptr)
      in_place = 0;
    else if (g[i].x.rows > 1 && g[i].x.ld != out[i].x.ld || g[i].x.count > 1 && g[i].x.stride != out[i].x.stride)
      return fail(GNS_ERR_INVALID, "outs", i, "may alias its gradient only with the same layout");
  }
  Finish f;
  if (int rc = norm_parts(g, n, norm_type, max_norm, eps, result, ws, ws_bytes, stream, &f)) return rc;
  if (int rc = finish_launch(f, result, dev_status, stream)) return rc;
  const Roles a = {{g, out ? out : g}, 2, n};
  auto go = [&](const auto& l) {
    clip_kernel<<<grid_for(l.start[l.count], 8), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(l, result, in_place);
    return launched("clip");
  };
  int rc = each_list<FlatList<2, CLIP_FLAT>>(a, THREADS * CLIP_UNITS, go);
  return rc ? rc : each_list<RowList<2, CLIP_ROWS>>(a, THREADS * CLIP_UNITS, go);
}

int adamw_step(const gns_tensor* W, const gns_tensor* G, const gns_tensor* M, const gns_tensor* V,
               const gns_tensor* master, int n, const gns_adamw_params* p, const float* grad_scale,
               const int32_t* step_count, int32_t* dev_status, void* stream) {
  if (!W || !G || !M || !V || !p) return set_error(GNS_ERR_INVALID, "null argument");
  if (n < 1) return set_error(GNS_ERR_INVALID, "need at least one tensor");
  if (!std::isfinite(p->lr) || !std::isfinite(p->weight_decay)) return set_error(GNS_ERR_INVALID, "AdamW params must be finite");
  if (!(p->beta1 >= 0.0 && p->beta1 < 1.0) || !(p->beta2 >= 0.0 && p->beta2 < 1.0))
    return set_error(GNS_ERR_INVALID, "beta1 and beta2 must be in [0, 1)");
  if (!(p->eps > 0.0) || !std::isfinite(p->eps)) return set_error(GNS_ERR_INVALID, "eps must be finite and > 0");
  if (!step_count && p->step < 1) return set_error(GNS_ERR_INVALID, "step must be >= 1");
  if (reinterpret_cast<uintptr_t>(grad_scale) % 4 || reinterpret_cast<uintptr_t>(step_count) % 4)
    return set_error(GNS_ERR_INVALID, "grad_scale or step_count: unaligned");
  const gns_tensor* role[5] = {W, G, M, V, master};
  static const char* const name[5] = {"W", "G", "M", "V", "master"};
  for (int i = 0; i < n; ++i) {
    for (int r = 0; r < 5; ++r) {
      if (!role[r]) continue;
      const gns_tensor& t = role[r][i];
      if (int rc = check_tensor(t, name[r], i)) return rc;
      if (r == 4 && empty(t)) continue;  // no master for this tensor
      if (r && !same_shape(W[i], t)) return fail(GNS_ERR_INVALID, name[r], i, "must have its weight's shape");
      if (r >= 2 && t.dtype != GNS_F32) return fail(GNS_ERR_INVALID, name[r], i, "must be f32");
      if (r == 4 && W[i].dtype == GNS_F32) return fail(GNS_ERR_INVALID, name[r], i, "an f32 weight takes no master");
      if (empty(t)) continue;
      for (int q = 0; q < r; ++q)
        if (role[q] && role[q][i].x.ptr == t.x.ptr) return fail(GNS_ERR_INVALID, name[r], i, "W, G, M, V and master may not alias");
    }
  }
  AdamwArgs a;
  a.beta1 = static_cast<float>(p->beta1);
  a.one_minus_beta1 = static_cast<float>(1.0 - p->beta1);
  a.beta2 = static_cast<float>(p->beta2);
  a.one_minus_beta2 = static_cast<float>(1.0 - p->beta2);
  a.decay = static_cast<float>(1.0 - p->lr * p->weight_decay);
  a.lr = static_cast<float>(p->lr);
  a.eps = static_cast<float>(p->eps);
  const double t = std::max(p->step, 1);
  a.step_size = static_cast<float>(p->lr / (1.0 - std::pow(p->beta1, t)));
  a.rsqrt_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(p->beta2, t)));
  a.log_beta1 = static_cast<float>(std::log(p->beta1));
  a.log_beta2 = static_cast<float>(std::log(p->beta2));
  a.grad_scale = grad_scale;
  a.step = step_count;
  a.status = dev_status;
  const Roles lists = {{W, G, M, V, master}, 5, n};
  auto go = [&](const auto& l) {
    adamw_kernel<<<grid_for(l.start[l.count], 8), THREADS, 0, static_cast<cudaStream_t>(stream)>>>(l, a);
    return launched("AdamW");
  };
  int rc = each_list<FlatList<5, ADAMW_FLAT>>(lists, THREADS, go);
  return rc ? rc : each_list<RowList<5, ADAMW_ROWS>>(lists, THREADS, go);
}

// A C caller gets a status whatever happens: the only exception these calls can raise is a
// failed allocation of an error message.
template <class F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return GNS_ERR_CUDA;
  }
}

}  // namespace
}  // namespace gns

using namespace gns;

extern "C" {

GNS_API size_t gns_list_workspace_size(int n) {
  if (n < 1) {
    guarded([] { return set_error(GNS_ERR_INVALID, "need at least one tensor"); });
    return 0;
  }
  return list_workspace(n);
}

GNS_API int gns_grad_norm(const gns_tensor* grads, int n, int norm_type, float max_norm, float eps, float* result,
                          void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  return guarded([&] { return grad_norm(grads, n, norm_type, max_norm, eps, result, ws, ws_bytes, dev_status, stream); });
}

GNS_API int gns_clip_grads(const gns_tensor* grads, const gns_tensor* outs, int n, int norm_type, float max_norm,
                           float eps, float* result, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  return guarded([&] {
    return clip_grads(grads, outs, n, norm_type, max_norm, eps, result, ws, ws_bytes, dev_status, stream);
  });
}

GNS_API int gns_adamw_step(const gns_tensor* W, const gns_tensor* G, const gns_tensor* M, const gns_tensor* V,
                           const gns_tensor* master, int n, const gns_adamw_params* adamw, const float* grad_scale,
                           const int32_t* step_count, int32_t* dev_status, void* stream) {
  return guarded([&] { return adamw_step(W, G, M, V, master, n, adamw, grad_scale, step_count, dev_status, stream); });
}

}  // extern "C"
