// ns_f8.h -- descriptors and launch wrappers of the kernels of the layers in 8-bit
// floating point (ns_f8.hip). Descriptors travel as kernel arguments, so a call
// uploads nothing; a longer list runs in several launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ns.h"

namespace ns {

// Flags of an operand's scales.
enum F8Flags : int32_t {
    kF8PowA = 1,      // one-byte scales
    kF8PowB = 2,
    kF8SquareA = 4,   // a scale for 128 rows
    kF8SquareB = 8,
};

// One product C = beta C + A B^T of a launch.
struct F8Item {
    const char* a;        // m x k
    const char* b;        // n x k
    const char* sa;       // scales, block by block
    const char* sb;
    void* out;
    float* part;          // split sums: nsplit x m x n
    int32_t m, n, k;
    int32_t lda, ldb, ldo;
    int32_t ldsa, ldsb;   // pitches of the scales
    int32_t flags;
    int32_t ntn;          // tiles along n
    int32_t nsplit;       // pieces that the blocks of k are cut into
    int32_t per;          // blocks per piece
    int32_t begin;        // its first workgroup in the launch
    int32_t pad;
};

// Items per launch: their descriptors fit the 4 KB of kernel arguments. Lists of
// up to kF8FewItems go as fewer bytes.
constexpr int kF8Items = 36, kF8FewItems = 4;
template <int N>
struct F8BatchOf {
    F8Item it[N];
    int32_t count;
    float beta;
};
using F8Batch = F8BatchOf<kF8Items>;
static_assert(sizeof(F8Batch) <= 4000, "the batch travels as kernel arguments");

// One matrix of a quantise launch: tiles of 128 x 128 values.
struct F8RowsItem {
    const char* values;
    char *q, *scale, *qt, *scale_t;
    int64_t ldv, ldq, ldqt;
    int32_t lds, ldst;    // pitches of the scales
    int32_t rows, cols;
    int32_t ntn;          // tiles along a row
    int32_t begin;        // its first workgroup in the launch
};
constexpr int kF8RowsItems = 40;
template <int N>
struct F8RowsBatchOf {
    F8RowsItem it[N];
    int32_t count;
    int32_t square;
};
using F8RowsBatch = F8RowsBatchOf<kF8RowsItems>;
static_assert(sizeof(F8RowsBatch) <= 4000, "the batch travels as kernel arguments");

// One matrix of a dequantise launch.
struct F8ValuesItem {
    const char *q, *scale;
    char* values;
    int64_t ldq, ldv;
    int32_t lds;
    int32_t rows, cols;
    int32_t kind;         // format | scale type << 1 | square << 2
    int32_t begin;        // its first workgroup in the launch
    int32_t pad;
};
constexpr int kF8ValuesItems = 48;
template <int N>
struct F8ValuesBatchOf {
    F8ValuesItem it[N];
    int32_t count;
};
using F8ValuesBatch = F8ValuesBatchOf<kF8ValuesItems>;
static_assert(sizeof(F8ValuesBatch) <= 4000, "the batch travels as kernel arguments");

// Dequantise: a workgroup takes this many pieces of 16 bytes of values, of several rows
// where they are short, else of one row.
constexpr int kF8ValuesPieces = 1024;
inline int64_t f8_values_wgs(int64_t rows, int64_t cols, int64_t elt)
{
    const int64_t n = kF8ValuesPieces, g = (cols * elt + 15) / 16;
    return g <= n ? (rows + n / g - 1) / (n / g) : rows * ((g + n - 1) / n);
}

// format: of every matrix (quantise), of the products' A. any: 0 where all scales are of
// one byte, else 1, or 2 where all of B's are for squares.
hipError_t launch_f8_quantize(const F8RowsBatch& b, int nwg, int format, int pow2, int dtype, hipStream_t stream);
hipError_t launch_f8_dequantize(const F8ValuesBatch& b, int nwg, int dtype, hipStream_t stream);
constexpr int kF8Block = 128;   // values of a block, and bytes of a slot of k
// Tiles of kF8MidM x kF8MidN or kF8SmallM x kF8SmallN, nsplit workgroups each.
constexpr int kF8MidM = 128, kF8MidN = 256, kF8SmallM = 128, kF8SmallN = 128;
hipError_t launch_f8_small(const F8Batch& b, int nwg, int format, int any, int dtype, hipStream_t stream);
// (mid tiles: of the products that has_mid names)
constexpr bool has_mid(int any, int dtype) { return (any != 0) == (dtype == NS_FP32); }
hipError_t launch_f8_mid(const F8Batch& b, int nwg, int format, int any, int dtype, hipStream_t stream);
// Tiles of kF8Big x kF8Big, one-byte scales, nsplit == 1.
constexpr int kF8Big = 256;
hipError_t launch_f8_big(const F8Batch& b, int nwg, int format, int dtype, hipStream_t stream);
// Products of at most kF8Few rows of A: `rows` rows of B a workgroup, 16 or 32.
constexpr int kF8Few = 32;
hipError_t launch_f8_few(const F8Batch& b, int nwg, int rows, int format, int any, int dtype, hipStream_t stream);
// Adds the pieces of the items with nsplit != 1 (0: a sum over nothing) and writes
// their outputs; begin counts workgroups of kF8JoinElems elements.
constexpr int kF8JoinElems = 1024;
hipError_t launch_f8_join(const F8Batch& b, int nwg, int dtype, hipStream_t stream);

}  // namespace ns
