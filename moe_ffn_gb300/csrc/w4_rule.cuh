// w4_rule.cuh — which of the 4-bit products' two kernels takes a call.  Compiled for the
// host as well, so that the rule can be checked on a CPU.
#pragma once
#include <cmath>
#include <cstdint>

namespace qmoe {
namespace w4 {

// Whether the kernel for many rows takes a call of M rows of x and E matrices of N x K
// (f32: of an f32 x).  That kernel starts slowly, about 10 us, and then reads each weight
// once for 64 rows.  The one for few starts in 4, but reads the weights again for every 16
// rows (5 of f32), has its own cost for each tile of outputs, as if K were 768 longer, and
// loses more than in proportion with a long K, whose x does not stay in shared memory.  So
// the rows of a matrix count times N (K + 768)^1.5, over the matrices that have rows; how
// the rows spread over them is known on the device only, so the average stands for it.
//
// The constants are fitted to 882 cases timed with both kernels
// (profiles/w4_kernel_times.json), over which the choice loses 1.0% a case with one matrix
// (f32 0.4%), 1.2% with groups (f32 2.4%).  us, few / many: one matrix, 4096 x 4096, 16 / 24 / 48 rows 11.1 / 14.0 /
// 28.1 against 14.2 / 15.2 / 16.5; 14336 x 4096, 8 / 12 / 24 rows 14.6 / 18.2 / 30.5 against
// 21.1 / 21.9 / 23.0; 768 x 2048, 128 / 384 rows 9.2 / 17.1 against 12.8 / 13.7; 16384 x 128, 32 / 64
// rows 4.7 / 8.3 against 6.9 / 7.2; 64 groups, 1024 x 2048, 2 / 8 rows each 27.7 / 39.5 against
// 32.8 / 32.9.  f32: 14336 x 4096, 4 / 16 rows 16.6 / 51.1 against 32.6 / 35.9; 64 groups, 5 / 8
// rows each 46.1 / 79.2 against 56.1 / 56.3.
// It takes the slower one by more than a fifth in 13 of the cases: with few k-blocks, where
// either kernel's last round is nearly empty (16384 x 128, 48 rows 8.8 against 7.0, with 32
// columns a scale 11.1 against 7.5; 1024 x 256, 1024 rows 15.1, many, against 10.8; 4096 x
// 512, 192 and 256 rows 15.5 and 15.8, many, against 12.2 and 12.0), at 4096 x 2048, 40 rows
// (16.0 against 13.2), and for 64 groups, 2048 x 768 (5 rows 33.6, many, against 27.5; f32, 8
// rows 97.7, many, against 61.1).
inline bool many_rows(int64_t M, int E, int64_t N, int64_t K, bool f32) {
    const double groups = static_cast<double>(M < E ? M : E);
    const double rows = static_cast<double>(M) / groups;
    const double k = (K + 768) / 4096.0;
    const double weights = groups * static_cast<double>(N) / 4096.0 * k * std::sqrt(k);
    if (E > 1) return f32 ? (rows - 4.5) * weights > 12.5 : rows * weights > 33.0;
    return f32 ? (rows - 5.0) * weights > 17.0 : (rows - 7.0) * weights > 23.0;
}

}  // namespace w4
}  // namespace qmoe
