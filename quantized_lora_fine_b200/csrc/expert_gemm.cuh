// Host-side interface of the block-scaled and grouped GEMM engine (expert_gemm.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/qlora_b200.h"

namespace qlb {

constexpr int kMaxExperts = 1024;

enum class ExpertMode {
  Fwd,   // D = A B^T: A rows [M x K], B [E][N x K]
  Dx,    // D = A B:   A rows [M x K], B [E][K x N]
  Dw,    // D_e = A_e^T B_e over the expert's rows: A [M x Nr], B [M x N], D fp32 [E][Nr x N]
};

struct ExpertArgs {
  ExpertMode mode;
  bool f8;
  int64_t M;             // rows of all groups together
  int64_t E;             // experts (1 with offsets == nullptr: one group of all rows)
  int64_t out, in;       // weight [E][out x in]
  const int32_t* offsets;
  const void* a;         // Fwd: X; Dx, Dw: dY   (row-major; e4m3 codes or bf16)
  const void* b;         // Fwd, Dx: W; Dw: X
  const float* sa;       // f8: scales of A's rows [M][ceil(K / 128)]
  const float* sb;       // f8: scales of W [E][ceil(out / 128)][ceil(in / 128)]
  void* d;               // bf16 [M x N], Dw: fp32 [E][out x in]
  int* status;
};

qlora_status launch_expert_gemm(const ExpertArgs& a, cudaStream_t s);

// few_rows.cu: Fwd with few rows a group. With `quantize` the rows are bf16 (at most
// kFewQuantRows in all, one group) and the weight e4m3.
constexpr int64_t kFewQuantRows = 2;
bool few_rows_wanted(const ExpertArgs& a);
qlora_status launch_few_rows(const ExpertArgs& a, bool quantize, cudaStream_t s);

}  // namespace qlb
