// ns_q8.h -- descriptors and launch wrappers of the 8-bit linear-layer kernels
// (ns_q8.hip). Descriptors travel as kernel arguments, so a call uploads
// nothing; a longer list runs in several launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ns {

// The operand forms of the products C = A B:
//   kQ8Matmul      A = Xq  (m = tokens, k = in)   B = Wq^T (n = out)
//   kQ8GradInput   A = dY  (m = tokens, k = out)  B = Wq   (n = in)
//   kQ8GradWeight  A = dY^T (m = out, k = tokens) B = Xq   (n = in)
enum Q8Op : int { kQ8Matmul = 0, kQ8GradInput = 1, kQ8GradWeight = 2 };

// One product of a launch.
struct Q8Item {
    const void* a;        // Xq or dY
    const int8_t* b;      // Wq or Xq
    const float* sa;      // kQ8Matmul: the token scales
    const float* sb;      // kQ8Matmul: the channel scales; else B's row scales
    void* out;
    float* part;          // split sums: nsplit x m x n fp32 (kQ8Matmul: int32)
    int32_t m, n, k;
    int32_t lda, ldb, ldo;
    int32_t ntn;          // tiles along n
    int32_t nsplit;       // pieces that the k slots are cut into
    int32_t per;          // slots per piece
    int32_t begin;        // its first workgroup in the launch
};

// Items per launch: their descriptors fit the 4 KB of kernel arguments.
constexpr int kQ8Items = 40;
struct Q8Batch {
    Q8Item it[kQ8Items];
    int32_t count;
    float beta;
};
static_assert(sizeof(Q8Batch) <= 4000, "the batch travels as kernel arguments");

// One matrix of a quantise or dequantise launch.
struct Q8RowsItem {
    void* values;
    int8_t* q;
    float* scale;
    int64_t ldv, ldq;
    int32_t rows, cols;
    int32_t begin;        // its first workgroup in the launch
};
constexpr int kQ8RowsItems = 64;
struct Q8RowsBatch {
    Q8RowsItem it[kQ8RowsItems];
    int32_t count;
    int32_t mode;
};
static_assert(sizeof(Q8RowsBatch) <= 4000, "the batch travels as kernel arguments");

// Rows per workgroup of the quantise and dequantise kernels, by row length:
// short rows take a wavefront each, long ones the whole workgroup.
constexpr int kQ8WaveCols = 2048;
inline int q8_rows_per_wg(int64_t cols) { return cols <= kQ8WaveCols ? 4 : 1; }

// Tile edges: the plain kernel (any pitch and alignment) and the large one
// (operands 16-byte aligned, at pitches of a multiple of 16 bytes).
constexpr int kQ8Tile = 64, kQ8Big = 256;
// k values per slot: 64 bytes of int8, or of bf16.
inline int q8_slot_k(int op) { return op == kQ8Matmul ? 64 : 32; }

hipError_t launch_q8_quantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream);
hipError_t launch_q8_dequantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream);
// Tiles of kQ8Tile x kQ8Tile, nsplit workgroups each.
hipError_t launch_q8_tile(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream);
// Tiles of kQ8Big x kQ8Big; nsplit == 1.
hipError_t launch_q8_big(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream);
// Adds the pieces of the items with nsplit > 1 and writes their outputs;
// begin counts workgroups of kQ8JoinElems elements.
constexpr int kQ8JoinElems = 2048;
hipError_t launch_q8_join(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream);

}  // namespace ns
