// grouped.h -- host-side interface of the grouped GEMM (grouped_kernel.cuh):
// matrix products over ragged groups of rows, each group against its own
// matrix.  Not part of the public ABI.
#pragma once

#include "internal.h"

namespace bpt {

// NT: out[r, :] = A[r, :] W_e^T   W [groups, N, K]
// NN: out[r, :] = A[r, :] W_e     W [groups, K, N]
// TN: out_e     = A_e^T B_e       out [groups, M, N], A [rows, M], B [rows, N], K = the group's rows
enum GroupedForm { GROUPED_NT = 0, GROUPED_NN = 1, GROUPED_TN = 2 };
enum GroupedEpi {
  GROUPED_STORE = 0,    // out = acc (+ beta out), bf16 or fp32
  GROUPED_ACT = 1,      // out = act(acc); out2, out3 (optional): what the backward takes, in
                        // a layout of these kernels' own (grouped_kernel.cuh): SwiGLU (w2
                        // given) the gate and the up product, GeLU the product (out2 alone)
  GROUPED_ACT_BWD = 2,  // acc = dy W2 of a row (unweighted), w its routing weight, aux and aux2
                        // as kept: out = w acc dact/dg, out2 = w acc dact/du (SwiGLU),
                        // out3 = w act; part[2 * tile column + half][row] = sum of acc * act
};

struct GroupedOp {
  int form = GROUPED_NT;
  int epi = GROUPED_STORE;
  int64_t rows = 0, N = 0, K = 0;  // rows of A; TN: N and M = K's place is taken by M
  int64_t M = 0;                   // TN only
  int groups = 0;
  const int32_t* offsets = nullptr;  // [groups + 1] (device)
  int64_t mean_rows = 0;             // rows / groups, the variants are chosen by
  // rows operand: [a_rows, K] (TN: [a_rows, M]); a gathered one takes row
  // order[r] / k of it for the group's row r, else row r
  const void* a = nullptr;
  const void* a2 = nullptr;  // NN: a second [rows, K] whose product with w2 is added; TN: a second M columns for out2
  bool a_gather = false;
  int64_t a_rows = 0;
  const void* b = nullptr;  // TN: rows operand [b_rows, N]
  bool b_gather = false;
  int64_t b_rows = 0;
  const void* w = nullptr;   // weights
  const void* w2 = nullptr;  // NT with GROUPED_ACT: the up matrices; NN: the second product's
  const int32_t* order = nullptr;
  int top_k = 1;
  void* out = nullptr;
  void* out2 = nullptr;
  void* out3 = nullptr;
  bool out_f32 = false;
  float beta = 0.f;
  int act = 0;
  const void* aux = nullptr;
  const void* aux2 = nullptr;
  const void* row_weight = nullptr;  // [rows] by pair (order[r]), fp32 or bf16
  bool row_weight_f32 = true;
  float* part = nullptr;
  int2* span = nullptr;  // if given: the rows [x, y) that the groups hold; x = -1: some offsets are bad
};

// Returns 0 or a BPT_* status.
int grouped_gemm(const GroupedOp& op, cudaStream_t st);
// tile columns of GROUPED_ACT_BWD's part: part holds 2 * grouped_part_tiles(N) * rows floats
int64_t grouped_part_tiles(int64_t N);
constexpr int GROUPED_MAX_GROUPS = 1024;

// 3-D bf16 map over [count, rows, cols] row-major matrices, box
// {box_cols, box_rows, 1}, 128-byte swizzle: rows past a matrix's end read as
// zeros, not as the next matrix.  Returns 0 on success.
int make_map_stack(CUtensorMap* map, const void* ptr, uint64_t count, uint64_t rows, uint64_t cols, uint32_t box_cols,
                   uint32_t box_rows);

}  // namespace bpt
