// Offsets of the product's loads (mx4_matmul.hip), for the device and for tests
// on the host: a tile's slice is T rows of so many bytes, 16 a lane.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define SBP_MX_HD __host__ __device__ __forceinline__
#else
#define SBP_MX_HD inline
#endif

namespace sbp {

using Mx4Offset = uint32_t;  // kMx4Past and the last round's bytes are past 2^31
constexpr Mx4Offset kMx4Past = 0x7FFFFFF0;  // beyond every buffer

template <int ROW>  // bytes of a row in a slice
struct Mx4Loads {
  static constexpr int kLanes = ROW / 16;     // that load a row
  static constexpr int kRows = 256 / kLanes;  // that a block of 256 loads at a time
  // The row of the tile that a lane loads a piece of in round 0, and kRows further on in
  // each round after.
  static SBP_MX_HD int row(int wave, int lane) { return wave * (64 / kLanes) + lane / kLanes; }
  // Of the piece in round 0, in an operand of kb blocks a row.
  static SBP_MX_HD Mx4Offset first(int row, int kb, int piece) {
    return static_cast<Mx4Offset>(row) * kb * 16 + piece * 16;
  }
  static SBP_MX_HD Mx4Offset round_bytes(int kb) {
    return static_cast<Mx4Offset>(kRows) * kb * 16;
  }
  // In round r: voff is first()'s, or kMx4Past where the piece lies past its row's end.
  static SBP_MX_HD Mx4Offset at(Mx4Offset voff, Mx4Offset round_bytes, int r) {
    return voff + r * round_bytes;
  }
};

}  // namespace sbp
