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

// Items per launch: their descriptors fit the 4 KB of kernel arguments. Lists
// of up to kQ8FewItems go as fewer bytes (a launch with 3.6 KB of arguments
// takes the host 3.7 us, one with 0.5 KB 2.5 us).
constexpr int kQ8Items = 40, kQ8FewItems = 4;
template <int N>
struct Q8BatchOf {
    Q8Item it[N];
    int32_t count;
    float beta;
};
using Q8Batch = Q8BatchOf<kQ8Items>;
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
template <int N>
struct Q8RowsBatchOf {
    Q8RowsItem it[N];
    int32_t count;
    int32_t mode;
};
using Q8RowsBatch = Q8RowsBatchOf<kQ8RowsItems>;
static_assert(sizeof(Q8RowsBatch) <= 4000, "the batch travels as kernel arguments");

// Rows per workgroup of the quantise and dequantise kernels, by row length:
// short rows take a wavefront each, long ones the whole workgroup.
constexpr int kQ8WaveCols = 2048;
inline int q8_rows_per_wg(int64_t cols) { return cols <= kQ8WaveCols ? 4 : 1; }

// An operand copied to 16-byte aligned rows.
struct Q8AlignItem {
    const void* src;
    void* dst;
    int64_t pitch;        // of src, bytes
    int32_t rows, len;    // bytes of a row
    int32_t begin;        // its first workgroup in the launch
};
constexpr int kQ8AlignItems = 64;
struct Q8AlignBatch {
    Q8AlignItem it[kQ8AlignItems];
    int32_t count;
};
static_assert(sizeof(Q8AlignBatch) <= 4000, "the batch travels as kernel arguments");

// Tile edges. Both kernels load their operands 16 bytes at a time: matrices
// aligned to 16 bytes at pitches of a multiple of 16 bytes.
constexpr int kQ8Big = 256, kQ8Mid = 128;
// k values per slot: 64 bytes of int8, or of bf16.
inline int q8_slot_k(int op) { return op == kQ8Matmul ? 64 : 32; }

hipError_t launch_q8_quantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream);
hipError_t launch_q8_dequantize(const Q8RowsBatch& b, int nwg, int dtype, hipStream_t stream);
// Tiles of kQ8Big x kQ8Big, nsplit == 1: nwhole workgroups of one tile each
// (counted through the items, begin in tiles), then two for each tile left.
hipError_t launch_q8_big(int op, const Q8Batch& b, int nwg, int nwhole, int dtype, hipStream_t stream);
// Tiles of kQ8Mid x kQ8Mid, nsplit workgroups each.
hipError_t launch_q8_mid(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream);
// grad_weight of at most kQ8Thin rows, operands at any alignment and pitches of
// 16 bytes or more: tiles of kQ8Thin x kQ8Mid, nsplit workgroups each.
constexpr int kQ8Thin = 64;
hipError_t launch_q8_thin(const Q8Batch& b, int nwg, int dtype, hipStream_t stream);
// matmul of at most kQ8Few tokens, at any alignment: q8_few_channels(m)
// channels a workgroup.
constexpr int kQ8Few = 32;
__host__ __device__ inline int q8_few_channels(int m) { return m <= 16 ? 16 : 32; }
hipError_t launch_q8_few(const Q8Batch& b, int nwg, int dtype, hipStream_t stream);
// Adds the pieces of the items with nsplit != 1 (0: a sum over nothing) and
// writes their outputs;
// begin counts workgroups of kQ8JoinElems elements.
constexpr int kQ8JoinElems = 1024;
hipError_t launch_q8_join(int op, const Q8Batch& b, int nwg, int dtype, hipStream_t stream);
// begin counts workgroups of kQ8AlignChunks 16-byte chunks.
constexpr int kQ8AlignChunks = 256;
hipError_t launch_q8_align(const Q8AlignBatch& b, int nwg, hipStream_t stream);

}  // namespace ns
