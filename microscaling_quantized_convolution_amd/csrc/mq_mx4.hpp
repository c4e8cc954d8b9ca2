// mq_mx4.hpp -- what the microscaled 4-bit linear layers share (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mq.h"

namespace mq {

constexpr int kMxBlock = MQ_MX4_BLOCK; // elements per scale
constexpr int kMxPiece = MQ_MX4_PIECE; // columns that lie together
constexpr int kMxScaleMin = 2;         // smallest scale byte written: the step of the smallest
                                       // codes, 2^-1 * 2^(2-127), is the smallest normal fp32
constexpr int kMxScaleMax = 252;       // largest: its code 6 is 1.5 * 2^127

// A quantized matrix (mq_mx4): piece p of row r at codes + (p * rows + r) * 128 and
// scales + (p * rows + r) * 8.
struct Mx4View {
    uint8_t *codes, *scales;
    int rows, cols;
    __host__ __device__ int pieces() const { return (cols + kMxPiece - 1) / kMxPiece; }
};

struct MatView {
    void *p;
    int64_t stride; // elements
    int dtype;
};

// What is quantized: a matrix, or one of the gradients of h = silu(g) u for dh (row- and
// column-wise; `col` is its transpose along its rows). rows, cols: the matrix's.
struct Mx4QuantArgs {
    MatView x;       // or dh
    MatView g, u;    // gradients only
    int rows, cols;
    Mx4View row, col;   // codes null: not wanted
    Mx4View row2, col2; // gradients: of u (row, col: of g)
    int sr;
    uint32_t seed_lo, seed_hi;
};

// y_j = sum over s of a[j][s] b[j][s]^T for j < jobs (the same M x N each); s = 1 only where
// pieces[1] > 0. Gated: job 0's b[0] and b[1] are the two weights, of the one operand a[0], and y[0]
// receives silu(G) U, g and u (null: not wanted) the products themselves.
struct Mx4MatmulArgs {
    Mx4View a[2][2], b[2][2];
    MatView y[2], g, u;
    int jobs, m, n;
    int pieces[2];
    bool gated;
    bool through;   // set by the launch: outputs are written past the caches
    MatView x;      // null, or a[0][0] still dense (mx4_quantizes_rows): m rows of `cols`
    int cols;
};

hipError_t launch_mx4_quantize(const Mx4QuantArgs &a, hipStream_t st);
hipError_t launch_mx4_gradients(const Mx4QuantArgs &a, hipStream_t st);
hipError_t launch_mx4_dequantize(const Mx4View &q, const MatView &out, hipStream_t st);
hipError_t launch_mx4_matmul(const Mx4MatmulArgs &a, hipStream_t st);
// Up to 16 rows, a workgroup takes 16 columns and its waves share the sum, while all of the launch's are there
// at once, two to a CU (n <= 8192; behind that, tiles of 64 columns, which read the weight in larger pieces).
// 4096 columns, us: 16 rows on 8192 7.1 (tiles 7.5), on 10240 9.0 (7.5); gated, with the quantization, 4 rows on
// 8192 11.5 (12.4), on 9216 13.9 (12.5). Plain products of up to 4 rows keep up with a third workgroup: 1 row on
// 12288 7.3 (7.5), of 16384 columns 20.6 (22.0), 4 rows 21.7 (22.0); on 16384 9.3 (8.0).
inline bool mx4_takes_rows(int m, int64_t n, bool gated) { return m <= 16 && n <= (m <= 4 && !gated ? 12288 : 8192); }
// whether launch_mx4_matmul takes these m rows dense, and quantizes them itself (where it takes rows)
bool mx4_quantizes_rows(int m, int n, int k);
hipError_t launch_mx4_rows(const Mx4MatmulArgs &a, hipStream_t st); // m <= 16

// The rules of the launches, which tests hold their sizes against: the kernel that products of these
// sizes take (pieces: of both sums) ...
enum Mx4Kind { kMx4Rows, kMx4Tile64, kMx4Tile128Deep, kMx4Tile128, kMx4Tile256 };
int mx4_matmul_kind(int jobs, int m, int n, int pieces, bool gated);
// ... and the rows to a lane of a quantization along the columns (32: the packed kernel)
int mx4_quantize_height(int rows, int cols, int dtype, bool sr, bool gradients);

} // namespace mq
