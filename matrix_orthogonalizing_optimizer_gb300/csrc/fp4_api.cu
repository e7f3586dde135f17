// C ABI of the operators on matrices in microscaled 4-bit floating point (include/gns.h): argument
// validation; the kernels are in fp4_quant.cu and fp4_gemm.cu.
#include <cmath>

#include "fp4.h"

namespace gns {
namespace {

int invalid(const char* name, const char* what) { return set_error(GNS_ERR_INVALID, std::string(name) + ": " + what); }

int check_fp4(const gns_fp4* q, const char* name) {
  if (!q) return invalid(name, "null descriptor");
  if (q->format != GNS_NVFP4 && q->format != GNS_MXFP4) return invalid(name, "format must be GNS_NVFP4 or GNS_MXFP4");
  const gns_batch& c = q->codes;
  // the rules of a batch of 16-bit elements hold for the codes too (shape limits, ld, stride, pointer)
  if (int rc = check_batch(&c, GNS_BF16, name)) return rc;
  if (c.ld % 32 || (c.count > 1 && c.stride % 32))
    return set_error(GNS_ERR_UNSUPPORTED, std::string(name) + ": ld and stride of codes must be multiples of 32 (16 bytes)");
  if (!q->scales) return invalid(name, "null scales");
  if (reinterpret_cast<uintptr_t>(q->scales) % 16)
    return set_error(GNS_ERR_UNSUPPORTED, std::string(name) + ": scales must be 16-byte aligned");
  if (c.count > 1) {
    if (q->scale_stride % 16) return set_error(GNS_ERR_UNSUPPORTED, std::string(name) + ": scale_stride must be a multiple of 16");
    if (q->scale_stride < 512 * fp4_row_tiles(c.rows) * fp4_block_tiles(c.cols, q->format))
      return invalid(name, "scale_stride is less than a matrix's scales");
  }
  if (q->format == GNS_NVFP4) {
    if (!q->tensor_scale) return invalid(name, "null tensor_scale");
    if (reinterpret_cast<uintptr_t>(q->tensor_scale) % 4) return invalid(name, "tensor_scale must be 4-byte aligned");
  } else if (q->tensor_scale) {
    return invalid(name, "MXFP4 has no tensor_scale");
  }
  return GNS_OK;
}

Fp4Ref ref(const gns_fp4& q) {
  Fp4Ref r;
  const gns_batch& c = q.codes;
  r.codes = static_cast<uint8_t*>(c.ptr);
  r.ld = c.ld / 2;
  r.stride = (c.count > 1 ? c.stride : c.rows * c.ld) / 2;
  r.scales = static_cast<uint8_t*>(q.scales);
  r.block_tiles = (int)fp4_block_tiles(c.cols, q.format);
  r.scale_stride = c.count > 1 ? q.scale_stride : 512 * fp4_row_tiles(c.rows) * r.block_tiles;
  r.tensor_scale = q.tensor_scale;
  r.rows = (int)c.rows;
  r.cols = (int)c.cols;
  return r;
}

DenseRef dense(const gns_batch& b, int dtype) {
  return DenseRef{b.ptr, b.ld, b.count > 1 ? b.stride : b.rows * b.ld, dtype};
}

int check_dtype(int dtype) {
  if (dtype == GNS_BF16 || dtype == GNS_F16 || dtype == GNS_F32) return GNS_OK;
  return set_error(GNS_ERR_INVALID, "dtype must be GNS_BF16, GNS_F16 or GNS_F32");
}

bool shape_is(const gns_batch& b, int64_t count, int64_t rows, int64_t cols) {
  return b.count == count && b.rows == rows && b.cols == cols;
}

int product(const gns_fp4* a, const gns_fp4* b, const gns_batch* c, const gns_batch* d, float alpha, float beta,
            gns_dtype dtype, int32_t* dev_status, void* stream, int sym) {
  int rc;
  if ((rc = check_dtype(dtype)) || (rc = check_fp4(a, sym ? "x" : "a")) || (!sym && (rc = check_fp4(b, "b"))) ||
      (rc = check_batch(d, dtype, "d")))
    return rc;
  if (a->format != b->format) return set_error(GNS_ERR_INVALID, "a and b must be of one format");
  if (a->codes.count != b->codes.count || a->codes.cols != b->codes.cols)
    return set_error(GNS_ERR_INVALID, "a and b must have equal counts and equally long rows");
  if (!shape_is(*d, a->codes.count, a->codes.rows, b->codes.rows))
    return set_error(GNS_ERR_INVALID, sym ? "d must be count x rows x rows of x" : "d must be count x rows of a x rows of b");
  if (!std::isfinite(alpha) || !std::isfinite(beta)) return set_error(GNS_ERR_INVALID, "alpha and beta must be finite");
  if (beta != 0.f) {
    if (!c) return set_error(GNS_ERR_INVALID, "c is required when beta != 0");
    if ((rc = check_batch(c, dtype, "c"))) return rc;
    if (!shape_is(*c, d->count, d->rows, d->cols)) return set_error(GNS_ERR_INVALID, "c must have the shape of d");
    if (c->ptr == d->ptr && ((c->rows > 1 && c->ld != d->ld) || (c->count > 1 && c->stride != d->stride)))
      return set_error(GNS_ERR_INVALID, "d may be c, with the same ld and stride, or lie elsewhere");
  }
  if (d->ptr == a->codes.ptr || d->ptr == b->codes.ptr || d->ptr == a->scales || d->ptr == b->scales)
    return set_error(GNS_ERR_INVALID, "d may not alias a or b");
  Fp4Product p;
  p.a = ref(*a);
  p.b = ref(*b);
  p.count = a->codes.count;
  p.fmt = a->format;
  p.sym = sym;
  p.alpha = alpha;
  p.beta = beta;
  p.c = beta != 0.f ? dense(*c, dtype) : DenseRef{nullptr, 0, 0, dtype};
  p.d = dense(*d, dtype);
  std::string err;
  rc = fp4_gemm_launch(p, dev_status, stream, &err);
  return rc ? set_error(rc, err) : GNS_OK;
}

// What an entry point allocates on the host may not be there: an exception does not cross the C ABI.
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

size_t gns_fp4_scale_bytes(int64_t rows, int64_t cols, int format) {
  const int rc = guarded([&] {
    if (format != GNS_NVFP4 && format != GNS_MXFP4) return invalid("format", "GNS_NVFP4 or GNS_MXFP4");
    if (rows < 1 || cols < 1 || rows > 65535LL * 64 || cols > 65535LL * 64)
      return invalid("rows and cols", "must be from 1 to 4194240");
    return (int)GNS_OK;
  });
  return rc ? 0 : (size_t)(512 * fp4_row_tiles(rows) * fp4_block_tiles(cols, format));
}

int gns_fp4_quantize(const gns_batch* x, gns_dtype dtype, const gns_fp4* q, const gns_fp4* qt, const float* amax,
                     int32_t* dev_status, void* stream) {
  return guarded([&] {
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_batch(x, dtype, "x"))) return rc;
    if (!q && !qt) return invalid("q and qt", "one of them is needed");
    if (q) {
      if ((rc = check_fp4(q, "q"))) return rc;
      if (!shape_is(q->codes, x->count, x->rows, x->cols)) return invalid("q", "must have the shape of x");
      if (q->codes.ptr == x->ptr) return invalid("q", "may not alias x");
    }
    if (qt) {
      if ((rc = check_fp4(qt, "qt"))) return rc;
      if (!shape_is(qt->codes, x->count, x->cols, x->rows)) return invalid("qt", "must have the shape of x's transpose");
      if (qt->codes.ptr == x->ptr) return invalid("qt", "may not alias x");
    }
    if (q && qt) {
      if (q->format != qt->format) return invalid("q and qt", "must be of one format");
      if (q->codes.ptr == qt->codes.ptr || q->scales == qt->scales ||
          (q->tensor_scale && q->tensor_scale == qt->tensor_scale))
        return invalid("q and qt", "may not share memory");
    }
    const int fmt = (q ? q : qt)->format;
    if (amax && fmt != GNS_NVFP4) return invalid("amax", "only NVFP4 has a scale of the matrix");
    Fp4Ref r, rt;
    if (q) r = ref(*q);
    if (qt) rt = ref(*qt);
    return fp4_quantize_launch(dense(*x, dtype), x->count, x->rows, x->cols, fmt, q ? &r : nullptr, qt ? &rt : nullptr, amax,
                               dev_status, stream);
  });
}

int gns_fp4_dequantize(const gns_fp4* q, const gns_batch* out, gns_dtype dtype, void* stream) {
  return guarded([&] {
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_fp4(q, "q")) || (rc = check_batch(out, dtype, "out"))) return rc;
    if (!shape_is(*out, q->codes.count, q->codes.rows, q->codes.cols)) return invalid("out", "must have the shape of q");
    if (out->ptr == q->codes.ptr || out->ptr == q->scales) return invalid("out", "may not alias q");
    return fp4_dequantize_launch(ref(*q), q->codes.count, q->format, dense(*out, dtype), stream);
  });
}

int gns_fp4_gemm(const gns_fp4* a, const gns_fp4* b, const gns_batch* c, const gns_batch* d, float alpha, float beta,
                 gns_dtype dtype, int32_t* dev_status, void* stream) {
  return guarded([&] { return product(a, b, c, d, alpha, beta, dtype, dev_status, stream, 0); });
}

int gns_fp4_sym_gemm_xxt(const gns_fp4* x, const gns_batch* c, const gns_batch* d, float alpha, float beta,
                         gns_dtype dtype, int32_t* dev_status, void* stream) {
  return guarded([&] { return product(x, x, c, d, alpha, beta, dtype, dev_status, stream, 1); });
}

}  // extern "C"
