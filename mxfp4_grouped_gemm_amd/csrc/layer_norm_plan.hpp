// How the backward pass of the layer norm is launched: which kernel, and how many
// workgroups (host code alone).
#pragma once

#include <stdint.h>

namespace moe {

// Columns of a row in registers with the sums of its columns (4000 rows of 12288 in
// 16 waves 145 us, read twice 119), and without them, for few rows.
constexpr int kHeldColumns = 8192, kFewColumns = 16384;

// Whether the sums over the rows are taken in the launch of the rows (us, bf16 stream,
// here and in two launches, of more than 8192 columns in three: 3584 columns: 1024
// rows 13.4, 1025 17.7 (not here), 2048 21.2 and 18.3; 256 columns: 2048 rows 12.9 and
// 17.5; 8200: 600 rows 19.6 and 22.9, 1000 27.0 and 28.6; 12288: 64 rows 10.2 and 17.7,
// 1000 31.9 and 34.4; 16384: 1000 rows 38.9 and 43.0; dx alone, which the same kernel
// makes so that its bits do not depend on what else is asked for: 1000 rows of 8200 12.5
// and 11.0, of 16384 17.3 and 18.9).
inline bool layer_norm_few_rows(int T, int H) { return H <= kFewColumns && T <= (H <= 512 ? 2048 : 1024); }

// Workgroups that go through the rows, where a row (of up to 512 columns: four rows)
// is in a workgroup's registers. sums: beside workgroups that take the columns' sums.
inline int layer_norm_row_groups(int T, int H, bool sums) {
    const int rows = H <= 512 ? 4 : 1;
    const int64_t groups = ((int64_t)T + rows - 1) / rows;
    // As many as the registers of their waves leave room for, but not so many that
    // their partial sums count (16384 rows of 3584: 512 workgroups 89 us, 768 96, 1024
    // 104; 513 to 1024 columns, with 1024, 1280 and 2048 workgroups: 30000 rows of 640
    // 45.3, 42.1 and 38.5, 32768 of 1024 55.0, 55.2 and 59.4, with an fp32 stream 102,
    // 110 and 111; 7000 of 8192: 256 workgroups 90.5, 512 96; 1500 of 8192: 26.6 and
    // 34.3). Few rows of more than 8192 columns: beside the sums, which want the room
    // as well, 64 and 128 workgroups: 400 rows of 12288 16.0 and 19.4, 512 18.7 and 21.1,
    // 600 22.5 and 23.6, 1000 of 8200 32.5 and 27.0; of an odd width, whose loads are at
    // 2-byte addresses, 300 of 10001 19.6 and 18.8, 512 29.3 and 23.8, but 487 of 10158
    // 19.5 and 21.0 (256 workgroups: 400 of 12288 20.0, 1000 of 8200 30.8); dx alone, 64,
    // 128 and 256: 400 of 12288 14.7, 10.6 and 8.8, 600 19.9, 13.1 and 10.6, 1000 of 8200
    // 28.9, 16.8 and 12.4 (512: 12.8).
    const int wide = !sums ? 256 : T <= (H % 2 ? 320 : 512) ? 64 : 128;
    const int most = H <= 512 ? 1024 : H <= 1024 ? 1280 : H <= 2048 ? 1024 : H <= 4096 ? 512 : H <= kHeldColumns ? 256 : wide;
    return (int)(groups < most ? groups : most);
}

// Parts of the sums over the rows that a second launch joins (0: none, few rows). Of
// rows that are read again for them: 64 runs of rows (us with 32, 64, 128 and 256: 4000
// rows of 12288 138, 120, 119 and 125; 16000 of 10001 625, 555, 524 and 515; 1100 of
// 16384 59.1, 57.7, 62.4 and 72.4; 300 of 65536 86, 95, 116 and 155).
inline int layer_norm_parts(int T, int H) {
    if (T <= 0 || layer_norm_few_rows(T, H)) return 0;
    if (H <= kHeldColumns) return layer_norm_row_groups(T, H, true);
    return T < 64 ? T : 64;
}

}  // namespace moe
