// Operators over lists of tensors: the global norm of a list of gradients with the scale that
// clips them (gns_grad_norm), the clipping itself (gns_clip_grads) and the AdamW step
// (gns_adamw_step). They do 1 to 2 operations a byte, so HBM bounds them on long lists and the
// launch on short ones; what their kernels are about is that the loads go out early and often
// whatever the tensors' number, type, alignment and pitch.
//
// A launch carries the descriptors of many tensors in its parameters: there is no table in device
// memory to write, so a call is kernels only and can be captured. Each tensor is cut into chunks;
// blocks take chunks of the whole list and find the tensor of each in the parameters.
//
// Two layouts: a FlatList holds tensors whose elements lie without gaps in every role (a role is
// one of the buffers that an operator walks in step: gradients and outputs; weights, gradients,
// moments, masters); a RowList holds batches of rows with a pitch. One launch has one layout.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <chrono>
#include <cmath>
#include <string>
#include <type_traits>

#include "../../include/gns.h"
#include "common.cuh"
#include "gemm.h"

namespace gns {

int set_error(int code, const std::string& msg);  // sets gns_last_error(); defined with the C ABI

namespace {

constexpr int THREADS = 256;

// The threads that take a chunk together: a block of THREADS, or a warp.
struct Block {
  static constexpr int kThreads = THREADS;
  GNS_DEV static int rank() { return threadIdx.x; }
};
struct Warp {
  static constexpr int kThreads = 32;
  GNS_DEV static int rank() { return threadIdx.x & 31; }
};

constexpr int MAX_GRID = 1216;  // blocks of one launch at most

// 16-byte vectors that a thread takes at a time, and blocks of a launch on an SM. Reading goes
// fastest with 8 vectors and 4 blocks (128 KB an SM in flight: 8.6 GB at 7.3 TB/s; 4 vectors and 8
// blocks 7.1, 8 and 5 7.2). Clipping 1.2 GB, which reads and writes: 4 vectors and 3 blocks 546 us,
// 4 and 4 560, 2 and 5 550, 8 and 3 562; rows with a pitch 4 and 4 (63 us for 112 MB; 4 and 3 69, 2
// and 5 75).
constexpr int NORM_VEC = 8, NORM_BLOCKS = 4, CLIP_VEC = 4, CLIP_BLOCKS = 3, CLIP_ROW_BLOCKS = 4;
// AdamW takes one unit of 8 elements a thread, 128 threads a block. With its reads and writes mixed
// more in flight is not faster on long lists: 524 M bf16 weights with masters 2.21 ms with 4 blocks,
// 2.27 with 5, 2.30 with 6, 2.49 with 3; 66 M 277, 284, 292 and 313 us; 28 M 121, 124 and 129 us with 4,
// 5 and 6; while 10 M in 120 tensors take 45, 41 and 39 us. So a launch of 2^14 chunks (17 M elements) or
// more has 4 blocks a SM, a shorter one 6. Rows with a pitch, where more has to be worked out before
// the loads, have 7 (28 M: 129 us; 6: 141).
constexpr int ADAMW_THREADS = 128, ADAMW_BLOCKS = 6, ADAMW_LONG_BLOCKS = 4, ADAMW_ROW_BLOCKS = 7, ADAMW_LONG = 1 << 14;

// ---------------------------------------------------------------------------------------
// lists as kernel parameters (at most 32,764 bytes of parameters a launch)

// start[i]: the launch's first chunk of tensor i, start[count]: all chunks. What else is known of a
// tensor lies together, as constant memory is read by lines. type: the GNS_ types of roles 0 and 1
// in bits 0-1 and 2-3, bit 4 set when the tensor has a master (AdamW's role 4). align: 2 = every
// unit starts on 8 elements' bytes in every role, 1 = on 16 bytes, 0 = on an element.
template <int R, int CAP>
struct FlatList {
  template <int C>
  using Cap = FlatList<R, C>;
  static constexpr bool kRows = false;
  static constexpr int kRoles = R, kCap = CAP;
  struct Tensor {
    void* ptr[R];
    long long n;
    unsigned char type, align;
    unsigned char head;  // elements before the first unit
  } at[CAP];
  int start[CAP + 1];
  int count;
};

template <int R, int CAP>
struct RowList {
  template <int C>
  using Cap = RowList<R, C>;
  static constexpr bool kRows = true;
  static constexpr int kRoles = R, kCap = CAP;
  struct Tensor {
    void* ptr[R];
    long long ld[R], stride[R];
    // 2^64 / d + 1 for the units of a row and the rows of a matrix (0: d is 1)
    unsigned long long by_row, by_matrix;
    int nrows;  // of all matrices
    int rows;   // of one matrix; 0: rows lie evenly from the first matrix to the last
    int cols;
    unsigned char type, align;
    // rows on 16 bytes whose pitch is their own length up to the next unit, from the first matrix
    // to the last, in every role (as empty_padded makes them): units lie behind one another
    unsigned char tight;
  } at[CAP];
  int start[CAP + 1];
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

// The tensor that holds a chunk, the last one that starts at or before it, of tensors lo .. hi.
template <class L>
GNS_DEV int find_tensor(const L& l, int chunk, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.start[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// A unit of 2^log elements in every role: one vector of the norm and of clipping (log 2 or 3), 8
// elements of AdamW. off: its first element, step: from one element to the next. valid: how many of
// its elements exist, from the first on (0: no unit). align: as in the list. over: what lies behind
// the valid elements up to the end of a vector can be read too.
template <int R>
struct Place {
  long long off[R];
  int valid, align, step;
  bool over;
};

// A flat tensor has whole units from element `head` on; what lies before and behind them, fewer
// than 2 units, follows as units of one element. Where no head puts every role on a vector, 32 units
// share 32 << log elements, each with every 32nd of them, so that a warp's accesses to single
// elements lie side by side.
template <int R, int CAP>
GNS_DEV Place<R> place(const FlatList<R, CAP>& l, int t, long long unit, int log) {
  Place<R> p;
  long long o = unit << log;
  const long long n = l.at[t].n;
  if (l.at[t].align) {
    const int head = l.at[t].head;
    const long long whole = (n - head) >> log;
    if (unit < whole) {
      o += head;
      p.valid = 1 << log;
      p.align = l.at[t].align;
    } else {
      const long long e = unit - whole;  // of n - whole units' edge elements
      o = e < head ? e : e + (whole << log);
      p.valid = o < n;
      p.align = 0;
    }
    p.step = 1;
  } else {
    o = ((unit >> 5) << (log + 5)) + (unit & 31);
    p.valid = static_cast<int>(max(0ll, min((n - o + 31) >> 5, 1ll << log)));
    p.align = 0;
    p.step = 32;
  }
  p.over = false;
#pragma unroll
  for (int r = 0; r < R; ++r) p.off[r] = o;
  return p;
}

// x / d by a product with inv = 2^64 / d + 1 (0 for d = 1): exact for 32-bit x and d, as
// x < 2^32 times inv's error, below 1, stays under 2^64 / d. A division costs more than all else
// that is done with a vector.
GNS_DEV uint32_t quotient(uint32_t x, unsigned long long inv) {
  return inv ? static_cast<uint32_t>(__umul64hi(x, inv)) : x;
}

// A unit of a row list, and the one `step` units on.
struct Cursor {
  uint32_t per_row;    // units
  uint32_t col;        // unit of its row
  unsigned long long row;
};
template <int R, int CAP>
GNS_DEV Cursor cursor(const RowList<R, CAP>& l, int t, unsigned long long unit, int log) {
  Cursor c;
  c.per_row = (static_cast<uint32_t>(l.at[t].cols) + (1u << log) - 1u) >> log;
  // a tensor of 2^32 units or more needs the division
  c.row = (unit >> 32) == 0 ? quotient(static_cast<uint32_t>(unit), l.at[t].by_row) : unit / c.per_row;
  c.col = static_cast<uint32_t>(unit - c.row * c.per_row);
  return c;
}
template <int R, int CAP>
GNS_DEV void advance(const RowList<R, CAP>& l, int t, Cursor& c, uint32_t step) {
  const uint32_t q = step < c.per_row ? 0u : quotient(step, l.at[t].by_row);
  c.row += q;
  c.col += step - q * c.per_row;
  if (c.col >= c.per_row) {
    c.col -= c.per_row;
    ++c.row;
  }
}

template <int R, int CAP>
GNS_DEV Place<R> place(const RowList<R, CAP>& l, int t, const Cursor& c, int log) {
  Place<R> p;
  const uint32_t nrows = static_cast<uint32_t>(l.at[t].nrows), at = c.col << log;
  p.valid = c.row < nrows ? static_cast<int>(min(1u << log, static_cast<uint32_t>(l.at[t].cols) - at)) : 0;
  p.align = l.at[t].align;
  p.step = 1;
  // on 16 bytes a row's pitch holds its last vector whole; behind the last row there may be nothing
  p.over = c.row + 1 < nrows;
  const uint32_t row = static_cast<uint32_t>(c.row);
  if (l.at[t].rows) {
    const uint32_t b = quotient(row, l.at[t].by_matrix), i = row - b * static_cast<uint32_t>(l.at[t].rows);
#pragma unroll
    for (int r = 0; r < R; ++r) p.off[r] = b * l.at[t].stride[r] + i * l.at[t].ld[r] + at;
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) p.off[r] = row * l.at[t].ld[r] + at;
  }
  return p;
}
template <int R, int CAP>
GNS_DEV Place<R> place(const RowList<R, CAP>& l, int t, long long unit, int log) {
  return place(l, t, cursor(l, t, static_cast<unsigned long long>(unit), log), log);
}

// ---------------------------------------------------------------------------------------
// reductions over a block of BT threads, in a fixed order; every thread gets the result

template <int BT>
GNS_DEV float block_sum(float v) {
  __shared__ float part[BT / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < BT / 32; ++w) s += part[w];
  return s;
}

template <int BT>
GNS_DEV uint32_t block_max(uint32_t v) {
  __shared__ uint32_t part[BT / 32];
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < BT / 32; ++w) m = max(m, part[w]);
  return m;
}

// ---------------------------------------------------------------------------------------
// vectors: 16 bytes of one role, 8 values of a 16-bit type or 4 of f32

struct Vec {
  uint32_t w[4];
};

GNS_DEV int vec_log(int dt) { return dt == GNS_F32 ? 2 : 3; }

// Zeroes the elements from `valid` on.
GNS_DEV void keep(Vec& u, int valid, int log) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (log == 2)
      u.w[e] = e < valid ? u.w[e] : 0u;
    else
      u.w[e] = 2 * e + 1 < valid ? u.w[e] : 2 * e < valid ? u.w[e] & 0xffffu : 0u;
  }
}

// The elements of one role of a unit; those that do not exist read as zero.
template <int R>
GNS_DEV void load_vec(Vec& u, const void* base, const Place<R>& p, int r, int log) {
  const int valid = p.valid, step = p.step;
  if (p.align && (valid == 1 << log || (p.over && valid))) {
    ld_v4(u.w, static_cast<const char*>(base) + (p.off[r] << (4 - log)));
    if (valid != 1 << log) keep(u, valid, log);
  } else if (log == 2) {
    const uint32_t* q = static_cast<const uint32_t*>(base) + p.off[r];
#pragma unroll
    for (int e = 0; e < 4; ++e) u.w[e] = e < valid ? q[e * step] : 0u;
  } else {
    const unsigned short* q = static_cast<const unsigned short*>(base) + p.off[r];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = 2 * e < valid ? q[2 * e * step] : 0u, hi = 2 * e + 1 < valid ? q[(2 * e + 1) * step] : 0u;
      u.w[e] = lo | (hi << 16);
    }
  }
}

template <int R>
GNS_DEV void store_vec(const Vec& u, void* base, const Place<R>& p, int r, int log) {
  const int valid = p.valid, step = p.step;
  if (p.align && valid == 1 << log) {
    st_v4(static_cast<char*>(base) + (p.off[r] << (4 - log)), u.w);
  } else if (log == 2) {
    uint32_t* q = static_cast<uint32_t*>(base) + p.off[r];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < valid) q[e * step] = u.w[e];
  } else {
    unsigned short* q = static_cast<unsigned short*>(base) + p.off[r];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) q[e * step] = static_cast<unsigned short>(u.w[e / 2] >> (16 * (e & 1)));
  }
}

// The two values of a word of a 16-bit type.
template <int DT>
GNS_DEV float2 halves(uint32_t w) {
  if (DT == GNS_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// ---------------------------------------------------------------------------------------
// norm: sqrt(sum x^2) over the whole list, or max |x|

// Loads this thread's N vectors of a chunk (of a group of W threads, vector k * W + rank is its
// k-th); what does not exist reads as zero. Nearly every chunk is whole: its loads go out with
// nothing to work out for each.
template <class T, int N, int R, int CAP>
GNS_DEV void load_chunk(const FlatList<R, CAP>& l, int t, int chunk, int log, Vec (&u)[N]) {
  constexpr int W = T::kThreads;
  const long long u0 = static_cast<long long>(chunk - l.start[t]) * (W * N);
  if (R > 1 && !l.at[t].align) {
#pragma unroll
    for (int k = 0; k < N; ++k) load_vec(u[k], l.at[t].ptr[0], place(l, t, u0 + k * W + T::rank(), log), 0, log);
    return;
  }
  const char* p =
      static_cast<const char*>(l.at[t].ptr[0]) + ((l.at[t].head + (u0 << log)) << (4 - log)) + T::rank() * 16;
  const long long whole = ((l.at[t].n - l.at[t].head) >> log) - u0;
  if (whole >= W * N) {
#pragma unroll
    for (int k = 0; k < N; ++k) ld_v4(u[k].w, p + k * W * 16);
  } else {
    const int n = static_cast<int>(whole) - T::rank();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      u[k] = {};
      if (k * W < n) ld_v4(u[k].w, p + k * W * 16);
    }
  }
}

// The edge element of this thread in a chunk (a thread has one at most), of a flat tensor whose
// whole units load_chunk takes by themselves; valid = 0: none.
template <class T, int N, int R, int CAP>
GNS_DEV Place<R> edge_place(const FlatList<R, CAP>& l, int t, int chunk, int log) {
  constexpr int W = T::kThreads;
  const long long u0 = static_cast<long long>(chunk - l.start[t]) * (W * N);
  const long long whole = ((l.at[t].n - l.at[t].head) >> log) - u0;
  Place<R> p;
  p.valid = 0;
  if (whole < W * N && l.at[t].align) {
    // units whole, whole + 1, ... of this chunk: the first of them that is this thread's turn
    const int first = max(static_cast<int>(whole), 0);
    const int unit = first + ((T::rank() - first) & (W - 1));
    if (unit < W * N) p = place(l, t, u0 + unit, log);
  }
  return p;
}
template <class T, int N, int R, int CAP>
GNS_DEV Place<R> edge_place(const RowList<R, CAP>&, int, int, int) {
  Place<R> p;
  p.valid = 0;
  return p;
}

// Whether a chunk of n units from u0 on has only whole vectors to read: it ends before the last
// unit of tight rows, so that only what each row's last vector holds has to be looked at.
template <int R, int CAP>
GNS_DEV bool behind_one_another(const RowList<R, CAP>& l, int t, unsigned long long u0, int n, int log) {
  const unsigned long long per_row = (static_cast<uint32_t>(l.at[t].cols) + (1u << log) - 1u) >> log;
  return l.at[t].tight && u0 + n < per_row * static_cast<uint32_t>(l.at[t].nrows);
}

template <class T, int N, int R, int CAP>
GNS_DEV void load_chunk(const RowList<R, CAP>& l, int t, int chunk, int log, Vec (&u)[N]) {
  constexpr int W = T::kThreads;
  const unsigned long long u0 = static_cast<unsigned long long>(chunk - l.start[t]) * (W * N);
  if (behind_one_another(l, t, u0, W * N, log)) {
    const char* p = static_cast<const char*>(l.at[t].ptr[0]) + (u0 + T::rank()) * 16;
#pragma unroll
    for (int k = 0; k < N; ++k) ld_v4(u[k].w, p + k * W * 16);
    Cursor c = cursor(l, t, u0 + T::rank(), log);
    const int last = l.at[t].cols - static_cast<int>((c.per_row - 1) << log);
#pragma unroll
    for (int k = 0; k < N; ++k) {
      if (c.col == c.per_row - 1) keep(u[k], last, log);
      advance(l, t, c, W);
    }
    return;
  }
  Cursor c = cursor(l, t, u0 + T::rank(), log);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    load_vec(u[k], l.at[t].ptr[0], place(l, t, c, log), 0, log);
    advance(l, t, c, W);
  }
}

// Calls f(vectors, type) for this thread's vectors of the block's run of chunks: a run crosses few
// tensors, where a stride over the list crosses many at each step.
template <class L, class F>
GNS_DEV void for_vectors(const L& l, F f) {
  const long long total = l.start[l.count];
  const int begin = static_cast<int>(total * blockIdx.x / gridDim.x);
  const int end = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x);
  if (begin >= end) return;
  int t = find_tensor(l, begin, 0, l.count - 1);
  for (int chunk = begin; chunk < end; ++chunk) {
    while (l.start[t + 1] <= chunk) ++t;
    const int dt = l.at[t].type & 3, log = vec_log(dt);
    const auto p = edge_place<Block, NORM_VEC>(l, t, chunk, log);
    Vec u[NORM_VEC], h[1];
    if (p.valid) load_vec(h[0], l.at[t].ptr[0], p, 0, log);
    load_chunk<Block>(l, t, chunk, log, u);
    f(u, dt);
    if (p.valid) f(h, dt);
  }
}

// f32 sum of the squares of a thread's vectors of one chunk, the values scaled by `pre` first
// (SCALED).
template <int DT, bool SCALED, int N>
GNS_DEV float squares(const Vec (&u)[N], float pre) {
  float q[2] = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (DT == GNS_F32) {
        const float x = __uint_as_float(u[k].w[e]) * (SCALED ? pre : 1.f);
        q[e & 1] = fmaf(x, x, q[e & 1]);
      } else {
        float2 x = halves<DT>(u[k].w[e]);
        if (SCALED) x = make_float2(x.x * pre, x.y * pre);
        q[0] = fmaf(x.x, x.x, q[0]);
        q[1] = fmaf(x.y, x.y, q[1]);
      }
    }
  return q[0] + q[1];
}
template <bool SCALED, int N>
GNS_DEV float squares(const Vec (&u)[N], float pre, int dt) {
  return dt == GNS_F32    ? squares<GNS_F32, SCALED>(u, pre)
         : dt == GNS_BF16 ? squares<GNS_BF16, SCALED>(u, pre)
                          : squares<GNS_F16, SCALED>(u, pre);
}
template <int N>
GNS_DEV uint32_t bits_of(const Vec (&u)[N]) {
  uint32_t b = 0;
#pragma unroll
  for (int k = 0; k < N; ++k) b |= (u[k].w[0] | u[k].w[1]) | (u[k].w[2] | u[k].w[3]);
  return b;
}

// Sum of this thread's squares: up to 64 of a chunk in f32, these sums with the rounding error of
// each addition kept beside them (Knuth's two-sum), as f32 holds too little for a long list and
// f64, at 2 operations a clock and SM, took longer than the loads. In units of 2^-24 a chunk's sum is
// within 33 (two sums of 32, joined), both parts joined 1, a warp's and a block's sums 13, the slots of
// one launch 3 and 13: 63 of the sum of squares, 32 of the norm, and 2 for the root and its power of two.
template <bool SCALED, class L>
GNS_DEV float sum_squares(const L& l, float pre, uint32_t* bits) {
  float s = 0.f, lost = 0.f;
  for_vectors(l, [&](const auto& u, int dt) {
    const float q = squares<SCALED>(u, pre, dt);
    const float t = __fadd_rn(s, q), b = __fsub_rn(t, s);
    lost += __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(q, b));
    s = t;
    if (!SCALED) *bits |= bits_of(u);
  });
  return isfinite(s) ? s + lost : s;
}

// A share m 2^e of a sum of squares, e = 0, 200 or -200; or a magnitude m, e = 0.
struct Share {
  float m;
  int e;
};

// The largest magnitude of some vectors: magnitudes order as their bits do, with every NaN above
// infinity.
template <int N>
GNS_DEV uint32_t largest(const Vec (&u)[N], int dt) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = u[k].w[e];
      if (dt == GNS_F32) {
        m = max(m, w & 0x7fffffffu);
      } else {
        const float2 x = dt == GNS_BF16 ? halves<GNS_BF16>(w) : halves<GNS_F16>(w);
        m = max(m, max(__float_as_uint(x.x) & 0x7fffffffu, __float_as_uint(x.y) & 0x7fffffffu));
      }
    }
  return m;
}

// A block's share of the norm, in every thread: its sum of squares sum(pre), of the values scaled
// by pre, bits being some of theirs that are set if any is.
//
// Squares of f32 and bf16 values leave f32's range long before the values do (above 2^64, below
// 2^-63). A block whose sum says that this may have happened (it is above 2^100 or not finite, or
// below 2^-80 though some bit is set) sums once more with the values scaled by 2^-100 or 2^100,
// which is exact for every value that counts: the largest magnitudes become at most 2^28, and
// where the sum lies below 2^-80 none is above 2^-40, so they become at most 2^60.
template <int BT, class F>
GNS_DEV Share square_share(F sum, const uint32_t& bits) {
  const float s = block_sum<BT>(sum(1.f, std::false_type()));
  const int any = __syncthreads_or(bits != 0);
  if (!(s <= 0x1p100f)) return {block_sum<BT>(sum(0x1p-100f, std::true_type())), 200};
  if (s < 0x1p-80f && any) return {block_sum<BT>(sum(0x1p100f, std::true_type())), -200};
  return {s, 0};
}

// A block's share, and the number of the call that it belongs to: written and read as one 16-byte
// access, so whoever sees the number sees the share.
struct alignas(16) Slot {
  Share share;
  unsigned long long call;
};

GNS_DEV void put_slot(Slot* s, Share v, unsigned long long call) {
  asm volatile(
      "{\n\t.reg .b128 x;\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tmov.b128 x, {v, %3};\n\t"
      "st.relaxed.gpu.global.b128 [%0], x;\n\t}" ::"l"(s),
      "r"(__float_as_uint(v.m)), "r"(v.e), "l"(call)
      : "memory");
}

GNS_DEV Slot get_slot(const Slot* s) {
  uint32_t m;
  Slot r;
  asm volatile(
      "{\n\t.reg .b128 x;\n\t.reg .b64 v;\n\tld.relaxed.gpu.global.b128 x, [%3];\n\tmov.b128 {v, %2}, x;\n\t"
      "mov.b64 {%0, %1}, v;\n\t}"
      : "=r"(m), "=r"(r.share.e), "=l"(r.call)
      : "l"(s)
      : "memory");
  r.share.m = __uint_as_float(m);
  return r;
}

// Writes a slot and returns what was there, as one access.
GNS_DEV Slot exchange_slot(Slot* s, Share v, unsigned long long call) {
  uint32_t m;
  Slot r;
  asm volatile(
      "{\n\t.reg .b128 x, y;\n\t.reg .b64 v;\n\tmov.b64 v, {%4, %5};\n\tmov.b128 x, {v, %6};\n\t"
      "atom.relaxed.gpu.global.exch.b128 y, [%3], x;\n\tmov.b128 {v, %2}, y;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "=r"(m), "=r"(r.share.e), "=l"(r.call)
      : "l"(s), "r"(__float_as_uint(v.m)), "r"(v.e), "l"(call)
      : "memory");
  r.share.m = __uint_as_float(m);
  return r;
}

// Who gathers the shares and no longer waits for a slot's closes it, by this number in the call's place.
GNS_DEV unsigned long long closed(unsigned long long call) { return ~call; }

// Hands in a share that is waited for. Where its slot has been closed the share stays behind, and the
// slot is cleared: a replay of the captured call has the same number, and would take it for its own.
GNS_DEV void hand_in(Slot* s, Share v, unsigned long long call) {
  if (exchange_slot(s, v, call).call == closed(call)) put_slot(s, {0.f, 0}, 0);
}

// What a norm call leaves in result[0] and result[1], from the slots of its launches.
struct Finish {
  Slot* slots;
  unsigned long long call;
  float* result;
  int* status;
  int nslots;
  int inf;
  float max_norm;  // infinity: no clipping
  float eps;
  unsigned long long limit_ns = GNS_WAIT_TIMEOUT_NS;  // of the wait for the slots
};

// Shares are added as they are where all have e = 0, which nearly always they do. Otherwise the
// sum has the largest exponent of those that are not zero: a share with the next one is then a
// float still, one two further down is too small to count.
GNS_DEV uint32_t exponents(Share s) { return s.m == 0.f ? 0u : s.e < 0 ? 1u : s.e == 0 ? 2u : 4u; }
GNS_DEV int top_exponent(uint32_t seen) { return seen & 4u ? 200 : seen & 2u || !seen ? 0 : -200; }
GNS_DEV float scaled_share(Share s, int top) {
  return s.e == top ? s.m : s.e + 200 == top ? s.m * 0x1p-100f * 0x1p-100f : 0.f;
}

// The results from the sum of squares n 2^e, or the largest magnitude n. A NaN norm gives a NaN
// scale.
GNS_DEV void norm_and_scale(const Finish& f, float n, int e, float* norm, float* scale) {
  *norm = f.inf ? n : sqrtf(n) * (e > 0 ? 0x1p100f : e < 0 ? 0x1p-100f : 1.f);
  const float d = *norm + f.eps;
  *scale = isinf(f.max_norm) || d <= f.max_norm ? 1.f : f.max_norm / d;
}

// The norm and the scale, in every thread of the block, from slots that hold this call's shares
// (WAIT = false) or will do so (WAIT = true), added in a fixed order. Waiting ends after limit_ns
// at the latest, however many slots are still open: these are closed, the norm is NaN and the
// timeout bit is set.
template <bool WAIT>
GNS_DEV void finish_norm(const Finish& f, float* norm, float* scale) {
  uint32_t most = 0, seen = 0;
  float n = 0.f;
  uint64_t t0 = 0;
  bool late = false;  // this thread has closed a slot
  for (int i = threadIdx.x; i < f.nslots; i += THREADS) {
    Slot s = get_slot(f.slots + i);
    if (WAIT) {
      for (uint32_t k = 1; s.call != f.call; ++k) {
        if (late || (k & 63u) == 0u) {
          const uint64_t now = global_timer_ns();
          if (!t0) t0 = now;
          if (late || now - t0 > f.limit_ns) {
            const Share none = {__int_as_float(0x7fffffff), 0};
            s = exchange_slot(f.slots + i, none, closed(f.call));
            if (s.call != f.call) {
              s.share = none;
              late = true;
            } else {  // handed in meanwhile
              put_slot(f.slots + i, s.share, f.call);
            }
            break;
          }
        }
        s = get_slot(f.slots + i);
      }
    }
    most = max(most, __float_as_uint(s.share.m));
    n += s.share.m;
    seen |= exponents(s.share);
  }
  if (WAIT && late) set_status(f.status, GNS_DEVST_TIMEOUT);
  int top = 0;
  if (f.inf) {
    n = __uint_as_float(block_max<THREADS>(most));
  } else if (__syncthreads_or((seen & ~2u) != 0)) {
    seen = (__syncthreads_or((seen & 4u) != 0) ? 4u : 0u) | (__syncthreads_or((seen & 2u) != 0) ? 2u : 0u) | 1u;
    top = top_exponent(seen);
    n = 0.f;
    for (int i = threadIdx.x; i < f.nslots; i += THREADS) n += scaled_share(get_slot(f.slots + i).share, top);
    if (WAIT && late) n = __int_as_float(0x7fffffff);  // what a closed slot holds now counts for nothing
    n = block_sum<THREADS>(n);
  } else {
    n = block_sum<THREADS>(n);
  }
  if (WAIT)  // a replay of the captured call writes the same number again; a closed slot's block clears it
    for (int i = threadIdx.x; i < f.nslots; i += THREADS)
      if (!late || get_slot(f.slots + i).call != closed(f.call)) put_slot(f.slots + i, {0.f, 0}, 0);
  norm_and_scale(f, n, top, norm, scale);
}

GNS_DEV void write_result(const Finish& f, float norm, float scale) {
  if (threadIdx.x == 0) {
    f.result[0] = norm;
    f.result[1] = scale;
    if (!isfinite(norm)) set_status(f.status, GNS_DEVST_NONFINITE);
  }
}

// slots[blockIdx.x] = the block's share. Where the call needs no further launch the last block
// then gathers all slots (`finish`): no block waits for that one, so it may wait for them
// whatever the order in which they run.
template <bool INF, class L>
__global__ void __launch_bounds__(THREADS, NORM_BLOCKS) norm_kernel(const __grid_constant__ L l, Slot* slots, Finish f,
                                                                   int finish) {
  grid_dep_launch();
  Share s;
  if (INF) {
    uint32_t m = 0;
    for_vectors(l, [&](const auto& u, int dt) { m = max(m, largest(u, dt)); });
    s = {__uint_as_float(block_max<THREADS>(m)), 0};
  } else {
    uint32_t bits = 0;
    s = square_share<THREADS>([&](float pre, auto scaled) { return sum_squares<scaled.value>(l, pre, &bits); }, bits);
  }
  if (threadIdx.x == 0) {
    if (finish)
      hand_in(slots + blockIdx.x, s, f.call);
    else  // the launch that gathers begins when this one has ended
      put_slot(slots + blockIdx.x, s, f.call);
  }
  if (finish && blockIdx.x == gridDim.x - 1) {
    float norm, scale;
    finish_norm<true>(f, &norm, &scale);
    write_result(f, norm, scale);
  }
}

// Self-test of the wait: the gathering alone, timed, and the handing in of shares of 1 alone.
__global__ void __launch_bounds__(THREADS) selftest_gather_kernel(Finish f, unsigned long long* out) {
  const uint64_t t0 = global_timer_ns();
  float norm, scale;
  finish_norm<true>(f, &norm, &scale);
  write_result(f, norm, scale);
  if (out && threadIdx.x == 0) *out = global_timer_ns() - t0;
}
__global__ void __launch_bounds__(THREADS) selftest_hand_in_kernel(Slot* slots, int n, unsigned long long call) {
  for (int i = threadIdx.x; i < n; i += THREADS) hand_in(slots + i, {1.f, 0}, call);
}

// A list of empty tensors.
__global__ void __launch_bounds__(THREADS) no_norm_kernel(Finish f) {
  float norm, scale;
  finish_norm<false>(f, &norm, &scale);
  write_result(f, norm, scale);
}

// ---------------------------------------------------------------------------------------
// clipping: out = round(scale * g); roles: gradient, output (the same pointers in place)

template <int DT>
GNS_DEV void scale_vec(Vec& u, float scale) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (DT == GNS_F32) {
      u.w[e] = __float_as_uint(__uint_as_float(u.w[e]) * scale);
    } else {
      const float2 x = halves<DT>(u.w[e]);
      if (DT == GNS_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x * scale, x.y * scale);
        u.w[e] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(x.x * scale, x.y * scale);
        u.w[e] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
}

GNS_DEV void scale_vec(Vec& u, float scale, int dt) {
  if (dt == GNS_F32)
    scale_vec<GNS_F32>(u, scale);
  else if (dt == GNS_BF16)
    scale_vec<GNS_BF16>(u, scale);
  else
    scale_vec<GNS_F16>(u, scale);
}

// Stores this thread's N vectors of a chunk that load_chunk has loaded, into role 1.
template <class T, int N, int CAP>
GNS_DEV void store_chunk(const FlatList<2, CAP>& l, int t, int chunk, int log, const Vec (&u)[N]) {
  constexpr int W = T::kThreads;
  const long long u0 = static_cast<long long>(chunk - l.start[t]) * (W * N);
  if (!l.at[t].align) {
#pragma unroll
    for (int k = 0; k < N; ++k) store_vec(u[k], l.at[t].ptr[1], place(l, t, u0 + k * W + T::rank(), log), 1, log);
    return;
  }
  char* q = static_cast<char*>(l.at[t].ptr[1]) + ((l.at[t].head + (u0 << log)) << (4 - log)) + T::rank() * 16;
  const long long whole = ((l.at[t].n - l.at[t].head) >> log) - u0;
  if (whole >= W * N) {
#pragma unroll
    for (int k = 0; k < N; ++k) st_v4(q + k * W * 16, u[k].w);
  } else {
    const int n = static_cast<int>(whole) - T::rank();
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (k * W < n) st_v4(q + k * W * 16, u[k].w);
  }
}

template <class T, int N, int CAP>
GNS_DEV void store_chunk(const RowList<2, CAP>& l, int t, int chunk, int log, const Vec (&u)[N]) {
  constexpr int W = T::kThreads;
  const unsigned long long u0 = static_cast<unsigned long long>(chunk - l.start[t]) * (W * N);
  Cursor c = cursor(l, t, u0 + T::rank(), log);
  if (behind_one_another(l, t, u0, W * N, log)) {
    char* q = static_cast<char*>(l.at[t].ptr[1]) + (u0 + T::rank()) * 16;
    Place<2> e;
    e.align = e.step = 1;
    e.off[1] = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      e.valid = c.col == c.per_row - 1 ? l.at[t].cols - static_cast<int>(c.col << log) : 1 << log;
      store_vec(u[k], q + k * W * 16, e, 1, log);
      advance(l, t, c, W);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    store_vec(u[k], l.at[t].ptr[1], place(l, t, c, log), 1, log);
    advance(l, t, c, W);
  }
}

// Every block forms the norm from the slots (a few KB, in L2), which saves a launch. The chunks go
// from the list's end to its start, all blocks near one another: a block with a run of its own, as
// in norm_kernel, takes 4 % longer where memory is written too.
template <class L>
__global__ void __launch_bounds__(THREADS, L::kRows ? CLIP_ROW_BLOCKS : CLIP_BLOCKS)
    clip_kernel(const __grid_constant__ L l, Finish f, int first, int in_place) {
  grid_dep_wait();
  float norm, scale;
  finish_norm<false>(f, &norm, &scale);
  if (first && blockIdx.x == 0) write_result(f, norm, scale);
  if (in_place && scale == 1.f) return;  // g * 1 is g
  int t = l.count - 1;
  for (int chunk = l.start[l.count] - 1 - static_cast<int>(blockIdx.x); chunk >= 0; chunk -= gridDim.x) {
    if (l.start[t] > chunk) t = find_tensor(l, chunk, 0, t - 1);
    const int dt = l.at[t].type & 3, log = vec_log(dt);
    const Place<2> e = edge_place<Block, CLIP_VEC>(l, t, chunk, log);
    Vec u[CLIP_VEC], h;
    if (e.valid) load_vec(h, l.at[t].ptr[0], e, 0, log);
    load_chunk<Block>(l, t, chunk, log, u);
#pragma unroll
    for (int k = 0; k < CLIP_VEC; ++k) scale_vec(u[k], scale, dt);
    store_chunk<Block>(l, t, chunk, log, u);
    if (e.valid) {
      scale_vec(h, scale, dt);
      store_vec(h, l.at[t].ptr[1], e, 1, log);
    }
  }
}

// ---------------------------------------------------------------------------------------
// clipping a short list: the whole call in one launch of one cluster

// A chunk is 4 KB here and every chunk has a warp of its own, which keeps it in registers between
// its sum and the scaled store: the list is read once. The blocks' shares meet in shared memory.
// What this saves is a launch on the host: a call takes 6.2 us where the two kernels above take 8.4
// (4.7 and 4.9 us on the GPU, at 0.2 MB); the norm alone is one launch anyway. The sums are plain
// f32 ones in another order than norm_kernel's, so the norm's last bit may differ from grad_norm's.
constexpr int SHORT_THREADS = 512, SHORT_VEC = 8, SHORT_CLUSTER = 8;
constexpr int SHORT_CHUNKS = SHORT_CLUSTER * SHORT_THREADS / 32;

template <bool INF, class L>
__global__ void __launch_bounds__(SHORT_THREADS)
    short_clip_kernel(const __grid_constant__ L l, Finish f, int in_place) {
  __shared__ alignas(8) Share share[SHORT_CLUSTER];
  const int blocks = gridDim.x, chunk = blockIdx.x * (SHORT_THREADS / 32) + (threadIdx.x >> 5);
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const bool mine = chunk < l.start[l.count];
  const int t = mine ? find_tensor(l, chunk, 0, l.count - 1) : 0, dt = l.at[t].type & 3, log = vec_log(dt);
  Vec u[SHORT_VEC] = {}, h[1] = {};
  Place<L::kRoles> e;
  e.valid = 0;
  if (mine) {
    e = edge_place<Warp, SHORT_VEC>(l, t, chunk, log);
    if (e.valid) load_vec(h[0], l.at[t].ptr[0], e, 0, log);
    load_chunk<Warp>(l, t, chunk, log, u);
  }
  Share s;
  if (INF) {
    s = {__uint_as_float(block_max<SHORT_THREADS>(max(largest(u, dt), largest(h, dt)))), 0};
  } else {
    const uint32_t bits = bits_of(u) | bits_of(h);
    s = square_share<SHORT_THREADS>(
        [&](float pre, auto scaled) { return squares<scaled.value>(u, pre, dt) + squares<scaled.value>(h, pre, dt); },
        bits);
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every block of the cluster runs
  if (static_cast<int>(threadIdx.x) < blocks) {
    const uint32_t to = mapa_shared(smem_u32(&share[blockIdx.x]), threadIdx.x);
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(__float_as_uint(s.m)), "r"(s.e) : "memory");
  }
  cluster_sync_all();
  uint32_t most = 0, seen = 0;
  for (int b = 0; b < blocks; ++b) {
    most = max(most, __float_as_uint(share[b].m));
    seen |= exponents(share[b]);
  }
  const int top = top_exponent(seen);
  float n = 0.f, norm, scale;
  for (int b = 0; b < blocks; ++b) n += scaled_share(share[b], top);
  norm_and_scale(f, INF ? __uint_as_float(most) : n, INF ? 0 : top, &norm, &scale);
  if (blockIdx.x == 0) write_result(f, norm, scale);
  if (!mine || (in_place && scale == 1.f)) return;
#pragma unroll
  for (int k = 0; k < SHORT_VEC; ++k) scale_vec(u[k], scale, dt);
  store_chunk<Warp>(l, t, chunk, log, u);
  if (e.valid) {
    scale_vec(h[0], scale, dt);
    store_vec(h[0], l.at[t].ptr[1], e, 1, log);
  }
}

// ---------------------------------------------------------------------------------------
// AdamW; roles: W, G, M, V, master
//
// m <- beta1 m + (1 - beta1) c g;  v <- beta2 v + (1 - beta2) (c g)^2
// w <- (1 - lr wd) w - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
//
// 22 to 30 bytes an element: HBM bounds it (6.65 TB/s read and written on 524 M weights, 98 % of a
// copy's rate), with the root and the quotient hidden behind the loads of the other blocks. The
// moments and masters stay in f32: a 16-bit v loses (1 - beta2) g^2 to rounding. A 16-bit weight is
// rounded once, from f32. Types are looked at when the loads are out, so one launch takes any mix.

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

// The hardware's root and reciprocal, each within 2^-23 of the exact one (an update is then within 13
// units of 2^-24: half of v's 9, the root 2, its correction and the sum with eps 1 each, the reciprocal
// 2, the product and the step size 1 each). The correctly rounded ones
// leave their fast path for zeros and subnormals, and an embedding is full of them: rows that no
// token has touched have v = 0, and m falls below 2^-126 some 800 steps after the last gradient (66 M
// embedding weights of which 70 % get no gradient: 304 us with them, 290 with these).
GNS_DEV float approx_sqrt(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
GNS_DEV float approx_reciprocal(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

GNS_DEV void adamw_unit(float (&w)[8], float (&g)[8], float (&m)[8], float (&v)[8], const AdamwArgs& a,
                        const AdamwStep& s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float ge = g[e] * s.scale;
    m[e] = fmaf(a.beta1, m[e], a.one_minus_beta1 * ge);
    v[e] = fmaf(a.beta2, v[e], a.one_minus_beta2 * ge * ge);
    const float denom = fmaf(approx_sqrt(v[e]), s.rsqrt_bc2, a.eps);
    w[e] = fmaf(-s.step_size, m[e] * approx_reciprocal(denom), a.decay * w[e]);
  }
}

// Whether a unit holds an infinity or a NaN as stored (a 16-bit weight may become one by its rounding):
// an exponent of ones, to which one more in its lowest bit carries into the place of the sign.
GNS_DEV bool not_finite(const Unit& u, int dt, int valid) {
  uint32_t hit = 0;
  if (dt == GNS_F32) {
#pragma unroll
    for (int e = 0; e < 8; ++e) hit |= e < valid ? (u.w[e] & 0x7fffffffu) + 0x00800000u : 0u;
    return hit >> 31;
  }
  const uint32_t one = dt == GNS_BF16 ? 0x00800080u : 0x04000400u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t exist = 2 * e + 1 < valid ? 0x80008000u : 2 * e < valid ? 0x8000u : 0u;
    hit |= ((u.w[e] & 0x7fff7fffu) + one) & exist;
  }
  return hit != 0;
}

// The elements of one role of a unit; those that do not exist read as zero.
GNS_DEV void load_unit(Unit& u, const void* base, const Place<5>& p, int r, bool f32) {
  const int valid = p.valid, step = p.step;
  const bool whole = p.align && (valid == 8 || (p.over && valid));
  if (f32) {
    const uint32_t* q = static_cast<const uint32_t*>(base) + p.off[r];
    if (whole && p.align == 2) {
      ld_v8(u.w, q);
    } else if (whole) {
      ld_v4(u.w, q);
      if (valid > 4) ld_v4(u.w + 4, q + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) u.w[e] = e < valid ? q[e * step] : 0u;
    }
    if (whole && valid != 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) u.w[e] = e < valid ? u.w[e] : 0u;
    }
  } else {
    const unsigned short* q = static_cast<const unsigned short*>(base) + p.off[r];
    if (whole) {
      ld_v4(u.w, q);
      if (valid != 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) u.w[e] = 2 * e + 1 < valid ? u.w[e] : 2 * e < valid ? u.w[e] & 0xffffu : 0u;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = 2 * e < valid ? q[2 * e * step] : 0u, hi = 2 * e + 1 < valid ? q[(2 * e + 1) * step] : 0u;
        u.w[e] = lo | (hi << 16);
      }
    }
  }
}

GNS_DEV void store_unit(const Unit& u, void* base, const Place<5>& p, int r, bool f32) {
  const int valid = p.valid, step = p.step;
  if (f32) {
    uint32_t* q = static_cast<uint32_t*>(base) + p.off[r];
    if (valid == 8 && p.align == 2) {
      st_v8(q, u.w);
    } else if (valid == 8 && p.align) {
      st_v4(q, u.w);
      st_v4(q + 4, u.w + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) q[e * step] = u.w[e];
    }
  } else {
    unsigned short* q = static_cast<unsigned short*>(base) + p.off[r];
    if (valid == 8 && p.align) {
      st_v4(q, u.w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < valid) q[e * step] = static_cast<unsigned short>(u.w[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Blocks stride over the list (a run for each took 4 % longer) and find a chunk's tensor by halving:
// one step may pass a hundred tensors.
template <class L>
__global__ void __launch_bounds__(ADAMW_THREADS, L::kRows ? ADAMW_ROW_BLOCKS : ADAMW_BLOCKS)
    adamw_kernel(const __grid_constant__ L l, const __grid_constant__ AdamwArgs a) {
  const int total = l.start[l.count];
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
  int t = 0;
  for (int chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
    if (l.start[t + 1] <= chunk) t = find_tensor(l, chunk, t + 1, l.count - 1);
    const Place<5> p = place(l, t, static_cast<long long>(chunk - l.start[t]) * ADAMW_THREADS + threadIdx.x, 3);
    if (!p.valid) continue;
    const int wt = l.at[t].type & 3, gt = (l.at[t].type >> 2) & 3;
    const bool master = l.at[t].type & 16;
    Unit uw, ug, um, uv;
    if (master)
      load_unit(uw, l.at[t].ptr[4], p, 4, true);
    else
      load_unit(uw, l.at[t].ptr[0], p, 0, wt == GNS_F32);
    load_unit(ug, l.at[t].ptr[1], p, 1, gt == GNS_F32);
    load_unit(um, l.at[t].ptr[2], p, 2, true);
    load_unit(uv, l.at[t].ptr[3], p, 3, true);
    float w[8], g[8], m[8], v[8];
    unpack(w, uw, master ? (int)GNS_F32 : wt);
    unpack(g, ug, gt);
    unpack(m, um, GNS_F32);
    unpack(v, uv, GNS_F32);
    adamw_unit(w, g, m, v, a, s);
    pack(um, m, GNS_F32);
    store_unit(um, l.at[t].ptr[2], p, 2, true);
    pack(uv, v, GNS_F32);
    store_unit(uv, l.at[t].ptr[3], p, 3, true);
    if (master) {
      pack(um, w, GNS_F32);
      store_unit(um, l.at[t].ptr[4], p, 4, true);
    }
    pack(uw, w, wt);
    bad |= not_finite(uw, wt, p.valid);
    store_unit(uw, l.at[t].ptr[0], p, 0, wt == GNS_F32);
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

// Whether a b <= 2^40 (a, b > 0); no division, as there are five lists of hundreds of tensors.
bool product(int64_t a, int64_t b) {
  int64_t p;
  return !__builtin_mul_overflow(a, b, &p) && p <= int64_t(1) << 40;
}

int check_tensor(const gns_tensor& t, const char* what, int i) {
  const gns_batch& x = t.x;
  if (t.dtype != GNS_BF16 && t.dtype != GNS_F16 && t.dtype != GNS_F32)
    return fail(GNS_ERR_INVALID, what, i, "unknown dtype");
  if (x.count < 0 || x.rows < 0 || x.cols < 0)
    return fail(GNS_ERR_INVALID, what, i, "count, rows and cols must be >= 0");
  if (empty(t)) return GNS_OK;
  if (!x.ptr) return fail(GNS_ERR_INVALID, what, i, "null data pointer");
  if (reinterpret_cast<uintptr_t>(x.ptr) & (size_of(t.dtype) - 1))
    return fail(GNS_ERR_INVALID, what, i, "pointer must be aligned to an element");
  if (!product(x.count, x.rows) || !product(x.count * x.rows, x.cols))
    return fail(GNS_ERR_INVALID, what, i, "more than 2^40 elements");
  if (x.rows > 1 && (x.ld < x.cols || !product(x.ld, x.rows)))
    return fail(GNS_ERR_INVALID, what, i, "ld must be at least cols, and a matrix span at most 2^40 elements");
  if (x.count > 1) {
    const int64_t last = x.rows > 1 ? (x.rows - 1) * x.ld : 0;
    if (x.stride < last + x.cols || !product(x.stride, x.count))
      return fail(GNS_ERR_INVALID, what, i, "stride: matrices overlap, or span more than 2^40 elements");
  }
  if (!flat(t) && (x.count * x.rows > 0x7fffffff || x.cols > 0x7fffffff))
    return fail(GNS_ERR_UNSUPPORTED, what, i, "rows with a pitch: at most 2^31 - 1 rows and columns");
  return GNS_OK;
}

bool same_shape(const gns_tensor& a, const gns_tensor& b) {
  return a.x.count == b.x.count && a.x.rows == b.x.rows && a.x.cols == b.x.cols;
}

// Whether b has a's shape and steps: what holds for a's then holds for b's.
bool lies_like(const gns_tensor& a, const gns_tensor& b) {
  return ((a.x.count ^ b.x.count) | (a.x.rows ^ b.x.rows) | (a.x.cols ^ b.x.cols) | (a.x.ld ^ b.x.ld) |
          (a.x.stride ^ b.x.stride)) == 0;
}

// check_tensor for a tensor whose role 0, checked and not empty, is `first`. Five lists of hundreds of
// tensors are looked at before a launch, and nearly always all five lie alike.
int check_role(const gns_tensor& first, const gns_tensor& t, const char* what, int i) {
  if (lies_like(first, t) && t.x.ptr && (t.dtype == GNS_BF16 || t.dtype == GNS_F16 || t.dtype == GNS_F32) &&
      !(reinterpret_cast<uintptr_t>(t.x.ptr) & (size_of(t.dtype) - 1)))
    return GNS_OK;
  return check_tensor(t, what, i);
}

// One operator's list, checked: role r of tensor i is role[r][i]; role 4 of AdamW (the master) may be
// absent, as a whole or tensor by tensor. Asked only about tensors that are not empty.
struct Roles {
  const gns_tensor* role[5];
  int nroles;
  int n;
  bool has(int r, int i) const { return r < 4 || (role[4] && !empty(role[4][i])); }
  bool is_flat(int i) const {
    const gns_tensor& first = role[0][i];
    const bool f = flat(first);
    for (int r = 1; r < nroles; ++r)
      if (has(r, i) && !(lies_like(first, role[r][i]) ? f : flat(role[r][i]))) return false;
    return f;
  }
  unsigned char type(int i) const {
    unsigned t = role[0][i].dtype;
    if (nroles > 1) t |= role[1][i].dtype << 2;
    if (nroles == 5 && has(4, i)) t |= 16;
    return static_cast<unsigned char>(t);
  }
};

// Fills entry k of a launch's list with tensor i; returns the number of its units.
template <int R, int CAP>
int64_t put(FlatList<R, CAP>* l, int k, const Roles& a, int i) {
  const gns_batch& x = a.role[0][i].x;
  const int64_t n = x.count * x.rows * x.cols;
  // elements from each role's first one to the next unit boundary: `wide` counts 8 elements
  // (16-bit: 16 bytes, f32: 32), `f32_16` 16 bytes of f32
  int wide = -1, f32_16 = -1, half = -1;
  bool same_wide = true, same_16 = true;
  for (int r = 0; r < R; ++r) {
    if (!a.has(r, i)) continue;
    const gns_tensor& t = a.role[r][i];
    const uintptr_t at = reinterpret_cast<uintptr_t>(t.x.ptr);
    const bool f32 = t.dtype == GNS_F32;
    const int w = static_cast<int>((0 - (f32 ? at >> 2 : at >> 1)) & 7);
    if (wide < 0) wide = w;
    same_wide &= w == wide;
    int& seen = f32 ? f32_16 : half;
    const int v = f32 ? w & 3 : w;
    if (seen < 0) seen = v;
    same_16 &= seen == v;
  }
  const bool vectors = R < 5;
  int head = 0, align = 0;
  if (vectors) {
    head = f32_16 >= 0 ? f32_16 : half;
    align = same_16;
  } else if (same_wide) {
    head = wide;
    align = 2;
  } else if (same_16 && (half < 0 || f32_16 < 0 || (half & 3) == f32_16)) {
    head = half >= 0 ? half : f32_16;
    align = 1;
  }
  if (!align) head = 0;
  if (head > n) head = static_cast<int>(n);
  l->at[k].n = n;
  l->at[k].head = static_cast<unsigned char>(head);
  l->at[k].align = static_cast<unsigned char>(align);
  const int log = vectors && a.role[0][i].dtype == GNS_F32 ? 2 : 3;
  const int64_t whole = (n - head) >> log;
  return align ? whole + (n - (whole << log)) : (n + (32 << log) - 1) >> (log + 5) << 5;
}

uint64_t inverse(int64_t d) { return d > 1 ? ~uint64_t(0) / static_cast<uint64_t>(d) + 1 : 0; }

template <int R, int CAP>
int64_t put(RowList<R, CAP>* l, int k, const Roles& a, int i) {
  const gns_batch& x = a.role[0][i].x;
  l->at[k].nrows = static_cast<int>(x.count * x.rows);
  bool even = true;  // matrices follow one another at their rows' pitch
  l->at[k].cols = static_cast<int>(x.cols);
  uint64_t bits16 = 0, bits32 = 0;  // low bits of every address and step in bytes, 16-bit and f32
  for (int r = 0; r < R; ++r) {
    l->at[k].ld[r] = l->at[k].stride[r] = 0;
    if (!a.has(r, i)) continue;
    const gns_tensor& t = a.role[r][i];
    if (t.x.rows > 1) l->at[k].ld[r] = t.x.ld;
    if (t.x.count > 1) l->at[k].stride[r] = t.x.stride;
    even &= t.x.count == 1 || t.x.rows == 1 || t.x.stride == t.x.rows * t.x.ld;
    if (t.x.rows == 1) l->at[k].ld[r] = l->at[k].stride[r];
    const int es = size_of(t.dtype);
    (es == 4 ? bits32 : bits16) |= reinterpret_cast<uintptr_t>(t.x.ptr) | static_cast<uint64_t>(l->at[k].ld[r] * es) |
                                   static_cast<uint64_t>(l->at[k].stride[r] * es);
  }
  const bool on16 = ((bits16 | bits32) & 15) == 0;
  l->at[k].align = static_cast<unsigned char>(!on16 ? 0 : (bits32 & 31) ? 1 : 2);
  const int log = R < 5 && a.role[0][i].dtype == GNS_F32 ? 2 : 3;
  const int64_t per_row = (x.cols + (1 << log) - 1) >> log;
  l->at[k].by_row = inverse(per_row);
  l->at[k].rows = even ? 0 : static_cast<int>(x.rows);
  bool tight = even && on16;
  for (int r = 0; r < R; ++r) tight &= !a.has(r, i) || l->at[k].ld[r] == per_row << log;
  l->at[k].tight = tight;
  l->at[k].by_matrix = inverse(x.rows);
  return x.count * x.rows * per_row;
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
    for (int r = 0; r < L::kRoles; ++r) l->at[k].ptr[r] = a.has(r, i) ? a.role[r][i].x.ptr : nullptr;
    l->at[k].type = a.type(i);
    l->start[k] = static_cast<int>(chunks);
    chunks += c;
    ++k;
  }
  l->start[k] = static_cast<int>(chunks);
  l->count = k;
  return i;
}

// Lists of one launch: how many tensors its parameters hold.
constexpr int SMALL_LIST = 128;
constexpr int NORM_FLAT = 1024, NORM_ROWS = 448, CLIP_FLAT = 768, CLIP_ROWS = 320, ADAMW_FLAT = 512, ADAMW_ROWS = 176;

static_assert(sizeof(FlatList<1, NORM_FLAT>) < 32000 && sizeof(RowList<1, NORM_ROWS>) < 32000, "kernel parameters");
static_assert(sizeof(FlatList<2, CLIP_FLAT>) < 32000 && sizeof(RowList<2, CLIP_ROWS>) < 32000, "kernel parameters");
static_assert(sizeof(FlatList<5, ADAMW_FLAT>) < 32000 && sizeof(RowList<5, ADAMW_ROWS>) < 32000, "kernel parameters");

// Launches f(list) for every launch that the tensors of one layout need. A short list goes with
// short parameters (SMALL_LIST).
template <class L, class F>
int each_list(const Roles& a, int64_t chunk_units, F f) {
  if constexpr (L::kCap > SMALL_LIST) {
    if (a.n <= SMALL_LIST) return each_list<typename L::template Cap<SMALL_LIST>>(a, chunk_units, f);
  }
  L l;
  for (int i = 0; i < a.n;) {
    i = fill(&l, a, i, chunk_units);
    if (!l.count) break;
    const int rc = f(l);
    if (rc) return rc;
  }
  return GNS_OK;
}

// ALONE: an ordinary launch. BEHIND: one that may begin while the one ahead of it on the stream
// ends, and waits for it itself (grid_dep_wait) before it touches memory. CLUSTER: one cluster.
enum How { ALONE, BEHIND, CLUSTER };

template <class... P, class... A>
int launch(const char* what, void (*kernel)(P...), int grid, int threads, void* stream, How how, const A&... args) {
  static_assert((std::is_same_v<P, A> && ...), "arguments go by address");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  if (how == CLUSTER) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = grid;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  } else {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = how == ALONE ? 0 : 1;
  void* at[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  profile_count_launch();
  const cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), at);
  if (e == cudaSuccess) return GNS_OK;
  (void)cudaGetLastError();
  return set_error(GNS_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

int grid_for(int chunks, int per_sm) { return std::max(1, std::min({chunks, device_sm_count() * per_sm, MAX_GRID})); }

size_t list_workspace(int n) {
  // at most one launch for every full list of each layout, and one more of each
  const size_t launches = static_cast<size_t>(n) / NORM_FLAT + static_cast<size_t>(n) / NORM_ROWS + 2;
  return launches * MAX_GRID * sizeof(Slot) + 256;
}

// Makes the call with f(list) where the list is short: every tensor in one launch's list, of one
// layout, and few enough chunks. Returns 1 where it is not.
template <class L, class F>
int short_list(const Roles& a, int tensors, F f) {
  L l;
  fill(&l, a, 0, 32 * SHORT_VEC);
  return l.count == tensors && l.start[l.count] <= SHORT_CHUNKS ? f(l) : 1;
}

template <class F>
int short_lists(const Roles& a, int tensors, F f) {
  if (a.n > SMALL_LIST) return 1;
  int64_t total = 0;
  for (int i = 0; i < a.n; ++i) {
    const gns_tensor& t = a.role[0][i];
    total += t.x.count * t.x.rows * t.x.cols * size_of(t.dtype);
    if (total > SHORT_CHUNKS * SHORT_VEC * 512) return 1;
  }
  const int rc = short_list<FlatList<2, SMALL_LIST>>(a, tensors, f);
  return rc <= 0 ? rc : short_list<RowList<2, SMALL_LIST>>(a, tensors, f);
}

// Blocks of the cluster, a power of two: a warp for each chunk.
int short_blocks(int chunks) {
  int blocks = 1;
  while (blocks < SHORT_CLUSTER && blocks * (SHORT_THREADS / 32) < chunks) blocks *= 2;
  return blocks;
}

// A number for a norm call that no other call has, and that memory a workspace is made from does
// not hold but by a chance of 2^-64: a mix of a counter that is a bijection of 64 bits (the finalizer
// of SplitMix64, Steele, Lea and Flood 2014).
uint64_t call_number() {
  static const uint64_t seed =
      static_cast<uint64_t>(std::chrono::high_resolution_clock::now().time_since_epoch().count());
  static std::atomic<uint64_t> calls{0};
  uint64_t z = (seed << 20) + ++calls;
  z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ull;
  z = (z ^ (z >> 27)) * 0x94d049bb133111ebull;
  z ^= z >> 31;
  return z ? z : 1;
}

int check_norm(const gns_tensor* g, int n, int norm_type, float max_norm, float eps, const float* result,
               const void* ws, size_t ws_bytes) {
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
  return GNS_OK;
}

int not_empty(const gns_tensor* g, int n) {
  int k = 0;
  for (int i = 0; i < n; ++i) k += !empty(g[i]);
  return k;
}

// The launches of a norm of `left` tensors that are not empty; finish: the last of them writes
// the result.
int norm_launches(const gns_tensor* g, int n, int left, void* stream, bool finish, Finish* f) {
  const Roles a = {{g}, 1, n};
  auto go = [&](const auto& l) {
    using L = std::decay_t<decltype(l)>;
    const int grid = grid_for(l.start[l.count], NORM_BLOCKS);
    Slot* at = f->slots + f->nslots;
    f->nslots += grid;
    left -= l.count;
    return launch("grad norm", f->inf ? norm_kernel<true, L> : norm_kernel<false, L>, grid, THREADS, stream, ALONE, l,
                  at, *f, static_cast<int>(finish && !left));
  };
  const int rc = each_list<FlatList<1, NORM_FLAT>>(a, THREADS * NORM_VEC, go);
  return rc || !left ? rc : each_list<RowList<1, NORM_ROWS>>(a, THREADS * NORM_VEC, go);
}

int grad_norm(const gns_tensor* g, int n, int norm_type, float max_norm, float eps, float* result, void* ws,
              size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (int rc = check_norm(g, n, norm_type, max_norm, eps, result, ws, ws_bytes)) return rc;
  const int inf = norm_type == GNS_NORM_INF, left = not_empty(g, n);
  Finish f = {static_cast<Slot*>(ws), call_number(), result, dev_status, 0, inf, max_norm, eps};
  if (!left) return launch("grad norm", no_norm_kernel, 1, THREADS, stream, ALONE, f);
  return norm_launches(g, n, left, stream, true, &f);
}

int selftest_norm_wait(void* ws, size_t ws_bytes, int nslots, int early, int late, int norm_type, uint32_t limit_us,
                       float* result, unsigned long long* out, int32_t* dev_status, void* stream) {
  if (!ws || !result) return set_error(GNS_ERR_INVALID, "null argument");
  if (reinterpret_cast<uintptr_t>(result) % 4 || reinterpret_cast<uintptr_t>(out) % 8)
    return set_error(GNS_ERR_INVALID, "result or out: unaligned");
  if (nslots < 1 || nslots > 1 << 16 || early < 0 || late < 0 || early + late > nslots)
    return set_error(GNS_ERR_INVALID, "nslots must be in [1, 65536] and hold early + late");
  if (norm_type != GNS_NORM_L2 && norm_type != GNS_NORM_INF) return set_error(GNS_ERR_INVALID, "unknown norm type");
  if (limit_us < 1 || limit_us > 1000000) return set_error(GNS_ERR_INVALID, "limit_us must be in [1, 1000000]");
  if (reinterpret_cast<uintptr_t>(ws) % 256 || ws_bytes < nslots * sizeof(Slot))
    return set_error(GNS_ERR_WORKSPACE, "workspace unaligned or too small");
  Slot* const slots = static_cast<Slot*>(ws);
  Finish f = {slots,     call_number(), result, dev_status, nslots, norm_type == GNS_NORM_INF,
              INFINITY, 0.f,           limit_us * 1000ull};
  auto hand = [&](Slot* at, int n) {
    return launch("norm self-test", selftest_hand_in_kernel, 1, THREADS, stream, ALONE, at, n, f.call);
  };
  auto gather = [&](int k) {
    f.result = result + 2 * k;
    unsigned long long* const time = out ? out + k : nullptr;
    return launch("norm self-test", selftest_gather_kernel, 1, THREADS, stream, ALONE, f, time);
  };
  int rc;
  if ((rc = hand(slots, early)) || (rc = gather(0)) || (rc = hand(slots + early, late)) || (rc = gather(1)) ||
      (rc = hand(slots, nslots)) || (rc = hand(slots, nslots)))
    return rc;
  return gather(2);
}

int clip_grads(const gns_tensor* g, const gns_tensor* out, int n, int norm_type, float max_norm, float eps,
               float* result, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream) {
  if (int rc = check_norm(g, n, norm_type, max_norm, eps, result, ws, ws_bytes)) return rc;
  int in_place = 1;
  for (int i = 0; out && i < n; ++i) {
    if (int rc = check_tensor(out[i], "outs", i)) return rc;
    if (!same_shape(g[i], out[i])) return fail(GNS_ERR_INVALID, "outs", i, "must have its gradient's shape");
    if (g[i].dtype != out[i].dtype) return fail(GNS_ERR_INVALID, "outs", i, "must have its gradient's dtype");
    if (empty(g[i])) continue;
    if (g[i].x.ptr != out[i].x.ptr)
      in_place = 0;
    else if ((g[i].x.rows > 1 && g[i].x.ld != out[i].x.ld) || (g[i].x.count > 1 && g[i].x.stride != out[i].x.stride))
      return fail(GNS_ERR_INVALID, "outs", i, "may alias its gradient only with the same layout");
  }
  const int inf = norm_type == GNS_NORM_INF;
  int left = not_empty(g, n);
  Finish f = {static_cast<Slot*>(ws), call_number(), result, dev_status, 0, inf, max_norm, eps};
  if (!left) return launch("clip", no_norm_kernel, 1, THREADS, stream, ALONE, f);
  const Roles a = {{g, out ? out : g}, 2, n};
  int rc = short_lists(a, left, [&](const auto& l) {
    using L = std::decay_t<decltype(l)>;
    return launch("clip", inf ? short_clip_kernel<true, L> : short_clip_kernel<false, L>,
                  short_blocks(l.start[l.count]), SHORT_THREADS, stream, CLUSTER, l, f, in_place);
  });
  if (rc <= 0) return rc;
  if ((rc = norm_launches(g, n, left, stream, false, &f))) return rc;
  int first = 1;  // the launch that writes the result
  auto go = [&](const auto& l) {
    using L = std::decay_t<decltype(l)>;
    const int grid = grid_for(l.start[l.count], L::kRows ? CLIP_ROW_BLOCKS : CLIP_BLOCKS);
    const int rc = launch("clip", clip_kernel<L>, grid, THREADS, stream, BEHIND, l, f, first, in_place);
    first = 0;
    left -= l.count;
    return rc;
  };
  rc = each_list<FlatList<2, CLIP_FLAT>>(a, THREADS * CLIP_VEC, go);
  return rc || !left ? rc : each_list<RowList<2, CLIP_ROWS>>(a, THREADS * CLIP_VEC, go);
}

int adamw_step(const gns_tensor* W, const gns_tensor* G, const gns_tensor* M, const gns_tensor* V,
               const gns_tensor* master, int n, const gns_adamw_params* p, const float* grad_scale,
               const int32_t* step_count, int32_t* dev_status, void* stream) {
  if (!W || !G || !M || !V || !p) return set_error(GNS_ERR_INVALID, "null argument");
  if (n < 1) return set_error(GNS_ERR_INVALID, "need at least one tensor");
  if (!std::isfinite(p->lr) || !std::isfinite(p->weight_decay))
    return set_error(GNS_ERR_INVALID, "AdamW params must be finite");
  if (!(p->beta1 >= 0.0 && p->beta1 < 1.0) || !(p->beta2 >= 0.0 && p->beta2 < 1.0))
    return set_error(GNS_ERR_INVALID, "beta1 and beta2 must be in [0, 1)");
  if (!(p->eps > 0.0) || !std::isfinite(p->eps)) return set_error(GNS_ERR_INVALID, "eps must be finite and > 0");
  // The kernel's numbers are f32. Where one of these is infinite there, an element whose gradient and
  // state are zero becomes 0 * inf, a NaN, in place of nothing.
  const float eps = static_cast<float>(p->eps);
  if (!std::isfinite(eps) || !std::isfinite(1.f / eps))
    return set_error(GNS_ERR_INVALID, "eps and 1 / eps must be finite in fp32 (eps above 2^-128)");
  if (!std::isfinite(static_cast<float>(p->lr / (1.0 - p->beta1))))
    return set_error(GNS_ERR_INVALID, "lr / (1 - beta1) must be finite in fp32");
  if (!std::isfinite(static_cast<float>(1.0 - p->lr * p->weight_decay)))
    return set_error(GNS_ERR_INVALID, "lr weight_decay must be finite in fp32");
  if (!step_count && p->step < 1) return set_error(GNS_ERR_INVALID, "step must be >= 1");
  if (reinterpret_cast<uintptr_t>(grad_scale) % 4 || reinterpret_cast<uintptr_t>(step_count) % 4)
    return set_error(GNS_ERR_INVALID, "grad_scale or step_count: unaligned");
  const gns_tensor* role[5] = {W, G, M, V, master};
  static const char* const name[5] = {"W", "G", "M", "V", "master"};
  for (int i = 0; i < n; ++i) {
    if (int rc = check_tensor(W[i], name[0], i)) return rc;
    const bool none = empty(W[i]);
    const void* at[5] = {W[i].x.ptr};
    for (int r = 1; r < 5; ++r) {
      if (!role[r]) continue;
      const gns_tensor& t = role[r][i];
      if (int rc = none ? check_tensor(t, name[r], i) : check_role(W[i], t, name[r], i)) return rc;
      if (r == 4 && empty(t)) continue;  // no master for this tensor
      if (!same_shape(W[i], t)) return fail(GNS_ERR_INVALID, name[r], i, "must have its weight's shape");
      if (r >= 2 && t.dtype != GNS_F32) return fail(GNS_ERR_INVALID, name[r], i, "must be f32");
      if (r == 4 && W[i].dtype == GNS_F32) return fail(GNS_ERR_INVALID, name[r], i, "an f32 weight takes no master");
      if (none) continue;
      for (int q = 0; q < r; ++q)
        if (at[q] == t.x.ptr) return fail(GNS_ERR_INVALID, name[r], i, "W, G, M, V and master may not alias");
      at[r] = t.x.ptr;
    }
  }
  AdamwArgs a;
  a.beta1 = static_cast<float>(p->beta1);
  a.one_minus_beta1 = static_cast<float>(1.0 - p->beta1);
  a.beta2 = static_cast<float>(p->beta2);
  a.one_minus_beta2 = static_cast<float>(1.0 - p->beta2);
  a.decay = static_cast<float>(1.0 - p->lr * p->weight_decay);
  a.lr = static_cast<float>(p->lr);
  a.eps = eps;
  const double t = std::max(p->step, 1);
  a.step_size = static_cast<float>(p->lr / (1.0 - std::pow(p->beta1, t)));
  a.rsqrt_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(p->beta2, t)));
  a.log_beta1 = static_cast<float>(std::log(p->beta1));
  a.log_beta2 = static_cast<float>(std::log(p->beta2));
  a.grad_scale = grad_scale;
  a.step = step_count;
  a.status = dev_status;
  const Roles lists = {{W, G, M, V, master}, 5, n};
  int left = not_empty(W, n);
  auto go = [&](const auto& l) {
    using L = std::decay_t<decltype(l)>;
    const int chunks = l.start[l.count];
    const int flat_blocks = chunks < ADAMW_LONG ? ADAMW_BLOCKS : ADAMW_LONG_BLOCKS;
    const int grid = grid_for(chunks, L::kRows ? ADAMW_ROW_BLOCKS : flat_blocks);
    left -= l.count;
    return launch("AdamW", adamw_kernel<L>, grid, ADAMW_THREADS, stream, ALONE, l, a);
  };
  int rc = each_list<FlatList<5, ADAMW_FLAT>>(lists, ADAMW_THREADS, go);
  return rc || !left ? rc : each_list<RowList<5, ADAMW_ROWS>>(lists, ADAMW_THREADS, go);
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
  return guarded(
      [&] { return grad_norm(grads, n, norm_type, max_norm, eps, result, ws, ws_bytes, dev_status, stream); });
}

GNS_API int gns_selftest_norm_wait(void* ws, size_t ws_bytes, int nslots, int early, int late, int norm_type,
                                   uint32_t limit_us, float* result, uint64_t* out, int32_t* dev_status, void* stream) {
  return guarded([&] {
    return selftest_norm_wait(ws, ws_bytes, nslots, early, late, norm_type, limit_us, result,
                              reinterpret_cast<unsigned long long*>(out), dev_status, stream);
  });
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
