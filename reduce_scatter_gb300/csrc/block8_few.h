// block8_few.h -- the product of few rows in 8-bit blocks (block8_few.cu).
#pragma once

#include <stdint.h>

namespace dgl {

constexpr int kFewRows = 128;  // the most rows it takes

// As dg_layer_block8_matmul, without trans_a; scale of row m, K block j:
// sa[(m >> a_shift) * sa_m + j * sa_k], of column n: sb[(n >> b_shift) * sb_n + j * sb_k].
struct FewRows {
  const void *a, *b;
  int a_type, b_type, b_mn;  // b_mn: b's rows are K's
  const float *sa, *sb;
  int64_t sa_m, sa_k, sb_n, sb_k;
  int a_shift, b_shift;
  void* D;
  int d_f32;
  int64_t M, N, K;
  void *workspace, *status;
};
int block8_few(const FewRows& f, void* stream);

}  // namespace dgl
