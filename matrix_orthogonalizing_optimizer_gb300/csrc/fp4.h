// Internal interface of the operators on matrices in microscaled 4-bit floating point (not part
// of the C ABI): fp4_api.cu checks the arguments, fp4_quant.cu holds the conversions and
// fp4_gemm.cu the products.
#pragma once

#include <stdint.h>

#include <string>

#include "../../include/gns.h"

namespace gns {

// Values that share a scale.
constexpr int fp4_block(int fmt) { return fmt == GNS_NVFP4 ? 16 : 32; }
inline int64_t fp4_blocks(int64_t cols, int fmt) { return (cols + fp4_block(fmt) - 1) / fp4_block(fmt); }
// Tiles of 128 rows x 4 blocks (512 bytes) that hold a matrix's scales.
inline int64_t fp4_row_tiles(int64_t rows) { return (rows + 127) / 128; }
inline int64_t fp4_block_tiles(int64_t cols, int fmt) { return (fp4_blocks(cols, fmt) + 3) / 4; }

// A checked gns_fp4 as the kernels take it (strides in bytes).
struct Fp4Ref {
  uint8_t* codes;
  long long ld, stride;
  uint8_t* scales;
  long long scale_stride;
  float* tensor_scale;
  int rows, cols;
  int block_tiles;
};

struct DenseRef {
  void* ptr;
  long long ld, stride;  // elements
  int dtype;
};

int fp4_quantize_launch(const DenseRef& x, int64_t count, int64_t rows, int64_t cols, int fmt, const Fp4Ref* q,
                        const Fp4Ref* qt, const float* amax, int32_t* dev_status, void* stream);
int fp4_dequantize_launch(const Fp4Ref& q, int64_t count, int fmt, const DenseRef& out, void* stream);

// d = alpha a b^T + beta c; sym: b is a, and what lies below the diagonal is mirrored. c.ptr
// NULL: no addend.
struct Fp4Product {
  Fp4Ref a, b;
  int64_t count;
  int fmt;
  int sym;
  float alpha, beta;
  DenseRef c, d;
};
int fp4_gemm_launch(const Fp4Product& p, int32_t* dev_status, void* stream, std::string* err);

int set_error(int code, const std::string& msg);
int check_batch(const gns_batch* b, gns_dtype dt, const char* name);
void profile_count_launch();

}  // namespace gns
