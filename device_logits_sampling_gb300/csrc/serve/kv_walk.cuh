// Which tokens the steps of an item are, and which pages its copies look up: the rules of first tokens that stay visible
// outside a window, plain integers that the host can go through too.
#pragma once

#ifdef __CUDACC__
#define ARC_WALK __host__ __device__ __forceinline__
#else
#define ARC_WALK inline
#endif

namespace arcs {

// First token of an item's step s of 2^shift tokens: `sinks` steps of first tokens, then those from step0 on.
ARC_WALK int sinks_token(int s, int sinks, int step0, int shift) { return (s < sinks ? s : step0 + (s - sinks)) << shift; }

// Whether no row of a tile, whose rows see `first` .. `last` at most and the tokens below `front`, sees any of the 16 tokens
// from tok on.
ARC_WALK bool sinks_unseen(int tok, int first, int last, int front) { return tok > last || (tok + 15 < first && tok >= front); }

// Whether the entry of the page that begins with token `next` may be loaded ahead from the page of the tokens from tok on,
// which some row sees.  From a window's page on, the window sees the next; from the last page of first tokens on, there
// may be pages between.
ARC_WALK bool sinks_ahead(int tok, int next, int last, int front) { return next <= last && (next < front || tok >= front); }

}  // namespace arcs
