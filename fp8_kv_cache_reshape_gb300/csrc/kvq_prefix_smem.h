// Shared-memory map of the shared-prefix kernel (plain C++: its byte ranges
// are also checked on the host).
#pragma once

namespace kvq {

constexpr int kTileRows = 128;  // query rows per tile: a tile per stream, a quarter of it per softmax warp
constexpr int kTileKeys = 128;  // keys per tile
constexpr int kSoftWarps = 8;

template <int D>
struct PrefixSmem {
  static constexpr int NST = D == 128 ? 3 : 6;      // K stages, V stages
  static constexpr int TILE = kTileKeys * D;        // bytes of a K or V tile
  static constexpr int PAGE = 16 * D;
  static constexpr int QT = kTileRows * D;          // one term of a query tile
  static constexpr int OFF_Q = 0;                   // [stream][term]
  static constexpr int OFF_K = OFF_Q + 4 * QT;
  static constexpr int OFF_V = OFF_K + NST * TILE;
  static constexpr int OFF_VH = OFF_V + NST * TILE;  // two f16 V tiles
  static constexpr int OFF_VH_END = OFF_VH + 2 * 2 * TILE;
  // The D bytes of a query row (of a stream's tile) in one of its two terms.
  static constexpr int q_row(int stream, int term, int row) { return OFF_Q + (2 * stream + term) * QT + row * D; }
  // Output staging: 32 rows of 32 floats per softmax warp, rows 16 bytes off
  // each other's banks.  Head dim 128: in the bytes of the warp's own query
  // rows (16 rows in each term), because nothing keeps a stream's other warps
  // from writing the next segment's queries while this one stages; the MMAs
  // that read its queries are done by then.  Head dim 64, whose rows are half
  // that: an area of its own.
  static constexpr int PITCH = 36;
  static constexpr int STAGE_HALF = 16 * PITCH * 4;
  static constexpr int STAGE_BYTES = D == 128 ? 0 : kSoftWarps * 2 * STAGE_HALF;
  static constexpr int stage_row(int stream, int quarter, int row) {
    return (D == 128 ? q_row(stream, row / 16, quarter * 32) : OFF_VH_END + ((4 * stream + quarter) * 2 + row / 16) * STAGE_HALF) +
           row % 16 * PITCH * 4;
  }
  static constexpr int OFF_BAR = OFF_VH_END + STAGE_BYTES;
  static constexpr int BAR_BYTES = 1024;
  static constexpr int SMEM = OFF_BAR + BAR_BYTES + 1024;  // + alignment slack
  static_assert(D != 128 || STAGE_HALF <= 32 * D, "staging within the warp's own query rows");
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

}  // namespace kvq
