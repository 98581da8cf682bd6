/* Every offset that a tile's loads of the 4-bit product form, over the range of a
 * row's blocks, rows left and blocks left: no sum leaves its type (the build's
 * sanitizers watch), pieces past a row's end lie beyond the buffer in every round,
 * and all others that the buffer lets through lie in the operand. */
#include <stdint.h>
#include <stdio.h>

#include "mx4_index.h"

template <int T, int ROW>
static long tile() {
  using L = sbp::Mx4Loads<ROW>;
  const int kbs[] = {1, 2, 3, 4, 5, 7, 8, 15, 16, 17, 65, 4096 + 3, (1 << 18) - 1, 1 << 18};
  const int haves[] = {1, 2, 31, T / 2 + 1, T - 1, T};
  const int rounds = T * ROW / 4096;
  long seen = 0;
  for (int kb : kbs)
    for (int have : haves) {
      const int64_t operand = int64_t{have} * kb * 16;
      const int step = kb > 4200 ? kb / 13 : 1;  // slices: all, or some and the last ones
      for (int first = 0; first < kb;
           first += first + (ROW / 16) * (step + 1) < kb ? (ROW / 16) * step : ROW / 16) {
        // the buffer begins at the slice and ends with the operand's rows
        const uint32_t length = static_cast<uint32_t>(operand - int64_t{first} * 16);
        for (int wave = 0; wave < 4; ++wave)
          for (int lane = 0; lane < 64; ++lane)
            for (int piece = 0; piece < L::kLanes; ++piece) {
              const int row = L::row(wave, lane);
              const bool past = first + piece >= kb;
              const sbp::Mx4Offset voff =
                  past ? sbp::kMx4Past : L::first(row, kb, piece);
              for (int r = 0; r < rounds; ++r) {
                const uint32_t off =
                    static_cast<uint32_t>(L::at(voff, L::round_bytes(kb), r));
                const int of = row + r * L::kRows;  // the row of the tile
                if (of >= T) return printf("row %d of %d\n", of, T), -1;
                // the bound check takes 16 bytes from off on, in 32 bits
                if (off > 0xFFFFFFF0u - 16) return printf("wraps: %u\n", off), -1;
                const bool read = off < length;
                const int64_t want = int64_t{of} * kb * 16 + piece * 16;
                if (read != (!past && of < have) || (read && off != want) ||
                    (read && off + int64_t{16} > length))
                  return printf("kb %d have %d first %d row %d piece %d: %u of %u\n", kb, have,
                                first, of, piece, off, length), -1;
                ++seen;
              }
            }
      }
    }
  return seen;
}

int main() {
  const long a = tile<256, 64>(), b = tile<128, 64>(), c = tile<64, 128>();
  if (a < 0 || b < 0 || c < 0) return 1;
  printf("%ld offsets ok\n", a + b + c);
  return 0;
}
