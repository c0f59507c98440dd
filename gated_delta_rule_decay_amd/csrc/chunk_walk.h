// chunk_walk.h -- a sweep's walk over the chunks of a segment, in 32-bit
// positions.  Plain C++: the host tests compile it too.
#pragma once

namespace gdn2 {

// Whether tokens remain behind the chunk of C positions at p0, of `len` > 0
// in all.  A segment may have up to 2^31 - 1 tokens: p0 + C of its last chunk
// is past what an int holds, so it is never formed.
constexpr bool chunk_follows(int p0, int len, int C) { return p0 < len - C; }

}  // namespace gdn2
