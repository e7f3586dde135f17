// Products of matrices in microscaled 4-bit floating point:
//   D = alpha A B^T + beta C,  (A B^T)[i][j] = sum_k A[i][k] B[j][k],
// sums in fp32, one rounding to D's type.
#include "fp4.cuh"

namespace gns {
namespace {

GNS_DEV float load_dense(const DenseRef& m, long long at) {
  if (m.dtype == GNS_F32) return static_cast<const float*>(m.ptr)[at];
  return h16_to_f(static_cast<const uint16_t*>(m.ptr)[at], m.dtype == GNS_F16);
}

// Rounds and stores; whether the stored value is finite.
GNS_DEV bool store_dense(const DenseRef& m, long long at, float v) {
  if (m.dtype == GNS_F32) {
    static_cast<float*>(m.ptr)[at] = v;
    return isfinite(v);
  }
  const uint16_t h = f_to_h16(v, m.dtype == GNS_F16);
  static_cast<uint16_t*>(m.ptr)[at] = h;
  return isfinite(h16_to_f(h, m.dtype == GNS_F16));
}

template <int FMT>
__global__ void __launch_bounds__(256) simple_kernel(Fp4Product p, int* status) {
  constexpr int N = FMT == GNS_NVFP4 ? 16 : 32;
  const int j = blockIdx.x * 16 + (threadIdx.x & 15);
  const int b = blockIdx.z;
  for (int i = blockIdx.y * 16 + (threadIdx.x >> 4); i < p.a.rows; i += gridDim.y * 16) {
    if (j >= p.b.rows || (p.sym && j < i)) continue;
    const uint8_t* ca = p.a.codes + b * p.a.stride + i * p.a.ld;
    const uint8_t* cb = p.b.codes + b * p.b.stride + j * p.b.ld;
    const uint8_t* sa = p.a.scales + b * p.a.scale_stride + (long long)(i >> 7) * p.a.block_tiles * 512;
    const uint8_t* sb = p.b.scales + b * p.b.scale_stride + (long long)(j >> 7) * p.b.block_tiles * 512;
    float sum = 0.f;
    for (int k = 0; k * N < p.a.cols; ++k) {
      float part = 0.f;
      for (int e = 0; e < N && k * N + e < p.a.cols; e += 2) {
        const float2 u = e2m1x2_to_f2(ca[(k * N + e) / 2]), v = e2m1x2_to_f2(cb[(k * N + e) / 2]);
        part += u.x * v.x + u.y * v.y;
      }
      sum += part * (fp4_scale_to_f<FMT>(sa[(k >> 2) * 512 + fp4_scale_at(i, k)]) *
                     fp4_scale_to_f<FMT>(sb[(k >> 2) * 512 + fp4_scale_at(j, k)]));
    }
    float o = sum * p.alpha;
    if (FMT == GNS_NVFP4) o = o * p.a.tensor_scale[b] * p.b.tensor_scale[b];
    const long long at = b * p.d.stride + i * p.d.ld + j;
    if (p.c.ptr) o += p.beta * load_dense(p.c, b * p.c.stride + i * p.c.ld + j);
    bool fine = store_dense(p.d, at, o);
    if (p.sym && j > i) store_dense(p.d, b * p.d.stride + j * p.d.ld + i, o);
    if (!fine) set_status(status, GNS_DEVST_NONFINITE);
  }
}

}  // namespace

int fp4_gemm_launch(const Fp4Product& p, int32_t* dev_status, void* stream, std::string* err) {
  const int ty = (p.a.rows + 15) / 16;
  const dim3 grid((p.b.rows + 15) / 16, ty < 65535 ? ty : 65535, (int)p.count);
  if (p.fmt == GNS_NVFP4)
    simple_kernel<GNS_NVFP4><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p, dev_status);
  else
    simple_kernel<GNS_MXFP4><<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p, dev_status);
  profile_count_launch();
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return GNS_OK;
  *err = std::string("launch: ") + cudaGetErrorString(e);
  return GNS_ERR_CUDA;
}

}  // namespace gns
