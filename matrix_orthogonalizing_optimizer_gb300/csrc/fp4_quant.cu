// Conversions to and from microscaled 4-bit floating point.
//
// A block of 16 (NVFP4) or 32 (MXFP4) values along a row shares one scale d; a value x is held as
// the code nearest to x / d among +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, magnitudes
// above 6 d as 6 d.
//   NVFP4: d = g s, g = the smallest power of two with max |X| <= 6 * 448 g over the matrix,
//          s = max |block| / (6 g) rounded to e4m3
//   MXFP4: d = 2^(floor(log2(max |block|)) - 2), the exponent at least -127
// Both are formed exactly: g and MXFP4's d are powers of two, and where a quotient has to be
// rounded, the divisor's significand has at most 4 bits, so that the correctly rounded fp32 quotient lies
// on a boundary between two codes only if the real one does.
#include "fp4.cuh"

namespace gns {
namespace {

template <class T>
GNS_DEV float to_f(T v);
template <>
GNS_DEV float to_f<float>(float v) {
  return v;
}
template <>
GNS_DEV float to_f<bf16>(bf16 v) {
  return __bfloat162float(v);
}
template <>
GNS_DEV float to_f<__half>(__half v) {
  return __half2float(v);
}
template <class T>
GNS_DEV T from_f(float v);
template <>
GNS_DEV float from_f<float>(float v) {
  return v;
}
template <>
GNS_DEV bf16 from_f<bf16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
GNS_DEV __half from_f<__half>(float v) {
  return __float2half_rn(v);
}

// scale[b] = the largest over the matrix's parts of the tensor scale that the part alone would
// have: the scale is a monotone function of the largest magnitude, so its maximum is the scale of
// the maximum, in whatever order the parts arrive. scale is zero before the launch.
template <class T>
__global__ void __launch_bounds__(256) amax_kernel(const T* x, long long ld, long long stride, int rows, int cols,
                                                   float* scale, float* scale_t) {
  const T* m = x + (long long)blockIdx.y * stride;
  uint32_t most = 0u;
  for (int r = blockIdx.x; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += 256) {
      const uint32_t a = __float_as_uint(to_f<T>(m[(long long)r * ld + c])) & 0x7FFFFFFFu;
      if (a < 0x7F800000u && a > most) most = a;
    }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if ((threadIdx.x & 31) == 0 && most) {
    const uint32_t g = fp4_tensor_scale_bits(most);
    if (scale) atomicMax(reinterpret_cast<unsigned int*>(scale) + blockIdx.y, g);
    if (scale_t) atomicMax(reinterpret_cast<unsigned int*>(scale_t) + blockIdx.y, g);
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

// One block of values: its scale's byte and its codes, two a byte. g: the matrix's scale (NVFP4).
// A block that holds Inf or NaN gets a NaN scale and codes of 0 (returns true).
template <int FMT, int N>
GNS_DEV bool quantize_block(const float (&x)[N], float g, uint8_t& scale, uint32_t (&codes)[N / 8]) {
  uint32_t most = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) most = max(most, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int i = 0; i < N / 8; ++i) codes[i] = 0u;
  if (most >= 0x7F800000u) {
    scale = FMT == GNS_NVFP4 ? 0x7F : 0xFF;
    return true;
  }
  float y[N];
  if (FMT == GNS_NVFP4) {
    scale = 0;
    if (g == 0.f) return false;
    const float inv = pow2_inverse(g);
    scale = f_to_e4m3(__fdiv_rn(__uint_as_float(most) * inv, 6.f));
    const float s = e4m3_to_f(scale);
    if (s == 0.f) return false;
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = __fdiv_rn(x[i] * inv, s);
  } else {
    const uint32_t e = most >> 23;
    scale = (uint8_t)(e < 2u ? 0u : e - 2u);
    const float inv = __uint_as_float((254u - scale) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = x[i] * inv;
  }
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
    codes[i] = f8_to_e2m1(y[8 * i], y[8 * i + 1], y[8 * i + 2], y[8 * i + 3], y[8 * i + 4], y[8 * i + 5], y[8 * i + 6],
                          y[8 * i + 7]);
  return false;
}

// One thread for each block of the held matrix, those of the scale tiles' padding included. Element
// (r, c) of the held matrix is x[r * step_r + c * step_c].
template <class T, int FMT>
__global__ void __launch_bounds__(128) quantize_kernel(const T* x, long long step_r, long long step_c,
                                                       long long stride, Fp4Ref q, int* status) {
  constexpr int N = FMT == GNS_NVFP4 ? 16 : 32;
  const int row = blockIdx.x * 128 + threadIdx.x;
  const int b = blockIdx.z;
  const T* m = x + b * stride + (long long)row * step_r;
  const float g = FMT == GNS_NVFP4 ? q.tensor_scale[b] : 1.f;
  for (int k = blockIdx.y; k < 4 * q.block_tiles; k += gridDim.y) {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = k * N + i;
      v[i] = row < q.rows && c < q.cols ? to_f<T>(m[c * step_c]) : 0.f;
    }
    uint8_t scale;
    uint32_t codes[N / 8];
    if (quantize_block<FMT, N>(v, g, scale, codes)) set_status(status, GNS_DEVST_NONFINITE);
    if (row >= q.rows || k * N >= q.cols) scale = 0;
    q.scales[b * q.scale_stride + ((long long)blockIdx.x * q.block_tiles + (k >> 2)) * 512 +
             fp4_scale_at(threadIdx.x, k)] = scale;
    // a row's codes end at a multiple of 32
    if (row < q.rows && k * N < (q.cols + 31) / 32 * 32) {
      uint8_t* o = q.codes + b * q.stride + row * q.ld + k * (N / 2);
#pragma unroll
      for (int i = 0; i < N / 16; ++i) *reinterpret_cast<uint2*>(o + 8 * i) = make_uint2(codes[2 * i], codes[2 * i + 1]);
    }
  }
}

template <class T, int FMT>
__global__ void __launch_bounds__(128) dequantize_kernel(Fp4Ref q, T* out, long long ld, long long stride) {
  constexpr int N = FMT == GNS_NVFP4 ? 16 : 32;
  const int blocks = (q.cols + N - 1) / N;
  const int b = blockIdx.z;
  const float g = FMT == GNS_NVFP4 ? q.tensor_scale[b] : 1.f;
  for (int row = blockIdx.y; row < q.rows; row += gridDim.y) {
    const int k = blockIdx.x * 128 + threadIdx.x;
    if (k >= blocks) continue;
    const float s = fp4_scale_to_f<FMT>(
        q.scales[b * q.scale_stride + ((long long)(row >> 7) * q.block_tiles + (k >> 2)) * 512 + fp4_scale_at(row, k)]);
    const uint8_t* c = q.codes + b * q.stride + row * q.ld + k * (N / 2);
    T* o = out + b * stride + row * ld;
    for (int i = 0; i < N; i += 2) {
      const float2 v = e2m1x2_to_f2(c[i / 2]);
      const int col = k * N + i;
      if (col < q.cols) o[col] = from_f<T>(v.x * s * g);
      if (col + 1 < q.cols) o[col + 1] = from_f<T>(v.y * s * g);
    }
  }
}

template <class T>
void quantize_typed(const DenseRef& x, int count, int rows, int cols, int fmt, const Fp4Ref* q, const Fp4Ref* qt,
                    const float* amax, int32_t* status, cudaStream_t stream) {
  const T* p = static_cast<const T*>(x.ptr);
  if (fmt == GNS_NVFP4) {
    float* s = q ? q->tensor_scale : nullptr;
    float* st = qt ? qt->tensor_scale : nullptr;
    if (amax) {
      given_scale_kernel<<<(count + 127) / 128, 128, 0, stream>>>(amax, count, s, st);
    } else {
      if (s) cudaMemsetAsync(s, 0, sizeof(float) * count, stream);
      if (st) cudaMemsetAsync(st, 0, sizeof(float) * count, stream);
      amax_kernel<T><<<dim3(rows < 1024 ? rows : 1024, count), 256, 0, stream>>>(p, x.ld, x.stride, rows, cols, s, st);
    }
    profile_count_launch();
  }
  for (int t = 0; t < 2; ++t) {
    const Fp4Ref* r = t ? qt : q;
    if (!r) continue;
    const int tiles = (r->rows + 127) / 128;
    const int nk = 4 * r->block_tiles;
    const dim3 grid(tiles, nk < 65535 ? nk : 65535, count);
    const long long sr = t ? 1 : x.ld, sc = t ? x.ld : 1;
    if (fmt == GNS_NVFP4)
      quantize_kernel<T, GNS_NVFP4><<<grid, 128, 0, stream>>>(p, sr, sc, x.stride, *r, status);
    else
      quantize_kernel<T, GNS_MXFP4><<<grid, 128, 0, stream>>>(p, sr, sc, x.stride, *r, status);
    profile_count_launch();
  }
}

template <class T>
void dequantize_typed(const Fp4Ref& q, int count, int fmt, const DenseRef& out, cudaStream_t stream) {
  const int blocks = (q.cols + fp4_block(fmt) - 1) / fp4_block(fmt);
  const dim3 grid((blocks + 127) / 128, q.rows < 65535 ? q.rows : 65535, count);
  T* o = static_cast<T*>(out.ptr);
  if (fmt == GNS_NVFP4)
    dequantize_kernel<T, GNS_NVFP4><<<grid, 128, 0, stream>>>(q, o, out.ld, out.stride);
  else
    dequantize_kernel<T, GNS_MXFP4><<<grid, 128, 0, stream>>>(q, o, out.ld, out.stride);
  profile_count_launch();
}

int launch_status(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return GNS_OK;
  return set_error(GNS_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

}  // namespace

int fp4_quantize_launch(const DenseRef& x, int64_t count, int64_t rows, int64_t cols, int fmt, const Fp4Ref* q,
                        const Fp4Ref* qt, const float* amax, int32_t* dev_status, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (x.dtype == GNS_F32)
    quantize_typed<float>(x, (int)count, (int)rows, (int)cols, fmt, q, qt, amax, dev_status, s);
  else if (x.dtype == GNS_F16)
    quantize_typed<__half>(x, (int)count, (int)rows, (int)cols, fmt, q, qt, amax, dev_status, s);
  else
    quantize_typed<bf16>(x, (int)count, (int)rows, (int)cols, fmt, q, qt, amax, dev_status, s);
  return launch_status("quantize");
}

int fp4_dequantize_launch(const Fp4Ref& q, int64_t count, int fmt, const DenseRef& out, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (out.dtype == GNS_F32)
    dequantize_typed<float>(q, (int)count, fmt, out, s);
  else if (out.dtype == GNS_F16)
    dequantize_typed<__half>(q, (int)count, fmt, out, s);
  else
    dequantize_typed<bf16>(q, (int)count, fmt, out, s);
  return launch_status("dequantize");
}

}  // namespace gns
