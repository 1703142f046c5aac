// Rows as sums of MXFP4 rows, for the block-scaled tensor cores.
//
// An element of a block of 32 becomes a whole number of 22 bits and a sign, in units of 2^-21 of the
// power of two below the block's largest; its eight octal digits, from -4 to 3, are E2M1 values,
// and digit i's MXFP4 row has the block's scale times 8^i.  So a row is the sum of eight MXFP4 rows,
// within 2^-22 of each block's largest: E4M3 elements and bf16 elements down to 2^-14 of it are exact.
// The product kernel (mxfp4_product.cu) takes them as columns, eight for one row of x, and adds each eight in its
// epilogue, the smallest first: while weights stream from HBM the tensor cores have room for 192 columns
// (743 cycles a SM for a stage's bytes, 375 for its MMAs at 192).
//
// Measured (896 experts of 1024 x 3584, 4096 rows): split 26 us (67 MB of pieces to L2), product 255 us, the weights
// at 6.8 TB/s; together 290 to 296, where the rows in registers (mxfp4_stream.cuh) take 403.  Experts of 256 tokens:
// split 31, gate and up 450 (6.7 TB/s), SiTU-GLU 21, down 256 (5.8 TB/s, with 59 MB of fp32 rows written), combine 11 to 20.
#pragma once

#include "mxfp4.cuh"

namespace qbh {

constexpr int kPieces = 8;

// Whether pieces pay: by the elements of weights that products of eight rows at a time would read, n matrices
// of `elements` each and once more per eight rows.  GPU time in us (a replayed graph, cold caches) as it is and in
// pieces: one row by 6144 x K = 7168 (44 M) 24 and 22, by 12288 (88 M) 30 and 24; 64 rows by 896 x 7168 (58 M) 26
// and 20; 128 rows over 24 matrices of 512 x 1024 (21 M) 18 and 16; the experts (3584 x 1024, three matrices) of a
// token's 4 routes (44 M) 42 and 40, of 6 (66 M) 52 and 44, of 8 (99 M) 50 and 46, of 256 tokens' 16 (15 G) 1439 and 789.
// Below the bound pieces would save about 2 us of GPU time for one or two launches and a scratch tensor more.
inline bool pieces_pay(long long n, long long rows, long long elements) { return (n + rows / 8) * elements >= 1LL << 26; }
inline bool pieces_ok(int K) { return K % 256 == 0; }   // whole words of scales for a warp
inline size_t piece_code_bytes(long long rows, int K) { return align_up((size_t)rows * kPieces * (K / 2), 256); }
inline size_t piece_bytes(long long rows, int K) {
    return piece_code_bytes(rows, K) + align_up((size_t)rows * kPieces * (K / 32), 256);
}

// The rows that pieces are made of: x [., K], bf16 or MXFP8, row r of the product from row map[r] / div (map NULL: r).
struct PieceSource {
    int x_type;
    const void* x;
    long long ldx;
    const uint8_t* x_scales;
    const int32_t* map;
    int div;
    const uint8_t* odd;   // [rows][32]: a byte for each 256 elements, not 0 where pieces do not stand for them; NULL: they do
};

// y [R, N] (with a second tensor [R, 2 N]: its products behind the first's), rows moved by row_map, from the
// pieces of R rows; offsets [E + 1] count pieces.  The product of a row with an odd byte is formed from x itself.
struct PieceProduct {
    int R, E, N, K;
    const uint8_t *x_codes, *x_scales;
    const uint8_t *w_codes, *w_scales, *w2_codes, *w2_scales;
    const int32_t* offsets;
    const int32_t* row_map;
    void* y;
    int y_type;
    long long ldy;
    PieceSource x;
    bool followed;   // the next kernel is one that waits for this one before it reads anything: it may be launched early
};
int piece_product(const PieceProduct& p, cudaStream_t s);

constexpr int kOddBytes = 32;
// The pieces of x's R rows, those that an expert owns, and their odd bytes (infinities, magnitudes below 2^-100 or
// out of the scales' range); offsets become those of pieces.
int split_rows(int R, int E, int K, const PieceSource& x, const int32_t* offsets, uint8_t* pieces, int32_t* piece_offsets,
               uint8_t* odd, cudaStream_t s);
// The same for the tokens' routes idx [T k] in expert order; row_map: the route at each place.
int split_routes(int T, int k, int E, int K, const PieceSource& x, const int32_t* idx, uint8_t* pieces, int32_t* piece_offsets,
                 int32_t* row_map, uint8_t* odd, cudaStream_t s);
// The pieces of SiTU-GLU(h[:, :M], h[:, M:]), h [R, 2 M] fp32, for the rows that piece_offsets count.
int split_glu(int R, int E, int M, const float* h, float beta1, float beta2, const int32_t* piece_offsets, uint8_t* pieces,
              cudaStream_t s);
int pieces_init();

}  // namespace qbh
