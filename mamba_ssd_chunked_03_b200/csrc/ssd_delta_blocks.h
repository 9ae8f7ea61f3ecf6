// Which 16 x 16 blocks of a 64-token piece's P and Z (ssd_delta_grads.cuh) have
// tokens.  A piece is one or two chunks of 32 tokens, two blocks each; a piece
// of 32 tokens or fewer has no second chunk, and what the preparation leaves
// for a chunk (decays, factors, tiles) does not exist for it: the last piece's
// would lie behind its part of the workspace.  Plain C++, so that the rule can
// be checked on the host.
#pragma once

namespace ssd {
namespace delta {

// Block of rows mt and columns sb, `chunks` of the piece's two exist: on or
// below the diagonal, its rows (and so its columns) in a chunk that exists.
constexpr bool block_exists(int mt, int sb, int chunks) { return sb <= mt && mt < 2 * chunks; }

}  // namespace delta
}  // namespace ssd
