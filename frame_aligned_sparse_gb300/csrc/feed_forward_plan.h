// How the feed-forward products are spread over the GPU, and the workspace they
// need.  Host code only: the same for every launch, the workspace's size and the
// tests.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace fas {
namespace feed_forward {

constexpr int kBlock = 64;  // elements of a TMA block's side: a 128-byte swizzled row

enum Epilogue { kPlain = 0, kGateUp = 1, kInner = 2 };

// Few tokens take one pass over the weights (feed_forward_few): up to 8 at any
// size, more where what each further 8 tokens cost is less than what the pass
// saves.  Of the gate-up product that grows with the inner features, its CTAs; of
// the product onto the width with the inner features too, its sums, and it is
// most where few columns make few CTAs, or so many that they fill the GPU
// twice.  In us, that way and with the tiles, weights in HBM: 2048 x 5504, one
// token 15.8 and 29.0, 16 tokens 19.5 and 26.1, 24 tokens 27.7 and 25.9;
// 256 x 1024, 24 tokens 6.7 and 12.8.  The product onto the width alone, 12
// tokens, longer than the tiles by: 1024 x 16384 2.3, 1024 x 8192 -2.1, 4096 x
// 16384 -3.0.  What is left: the 512 CTAs of the gate-up product of 8192 x 8192
// just miss one round (12 tokens 92 and 82).
constexpr int kFewTokens = 31;  // at most
inline bool few_gate_up(int64_t tokens, int64_t inner) {
  return tokens <= 16 || (tokens <= kFewTokens && inner <= 4096);
}
inline bool few_out(int64_t tokens, int64_t width, int64_t inner) {
  if (tokens <= 16) return tokens <= 8 || inner <= 8192 || width >= 2048;
  return tokens <= kFewTokens && width <= 4096 && inner <= (width < 1024 ? 4096 : 6144);
}

// What runs at once: CTAs, one an SM, and pairs of CTAs (an SM may be left
// without a partner).
struct Machine {
  int ctas = 1, pairs = 0;
  int units(int G) const { return G == 1 ? ctas : pairs; }
};

// The forms of a tile, and what they take in nanoseconds (measured on long
// products): a step of 64 along k, what of a tile does not run beside another's
// products, and writing and adding up a tile of fp32 parts.
struct Form {
  int G, cols, step, tile, part;
  constexpr int rows() const { return 128 * G; }
  int64_t tiles(int64_t m, int64_t n) const { return (m + rows() - 1) / rows() * ((n + cols - 1) / cols); }
};
constexpr Form kForms[3] = {{1, 128, 315, 0, 25}, {2, 256, 358, 0, 100}, {2, 512, 632, 2000, 200}};
constexpr int64_t kJoinNs = 4000;  // the launch that adds up the parts
// What each epilogue adds to a tile's steps, and what a tile takes at least
// (20,000 rows with 2 to 32 steps).
constexpr struct {
  int more, least;
} kEpilogues[3][3] = {{{0, 1000}, {0, 2000}, {0, 4000}}, {{1200, 2000}, {600, 3600}, {}}, {{2000, 5800}, {5300, 11600}, {}}};

// How a launch's tiles are spread.
struct Spread {
  int form = 0, splits = 1;
  int64_t whole = 0;     // tiles done whole
  int64_t parts = 0;     // of the others, together
  int64_t ns = INT64_MAX;
  int64_t bytes() const { return parts * kForms[form].rows() * kForms[form].cols * 4; }
};
// The form that is done first.  Whole rounds of tiles, one for every CTA or
// pair, are done whole; what is left over would keep only some of them busy,
// and few tiles altogether most of them idle, so those are split along k where
// that is sooner done.  The products with an epilogue of their own have no
// parts, and no tiles of 512 columns, whose epilogue the next tile waits for.
template <class Tiles>
Spread spread(Epilogue e, const Tiles& tiles, int64_t k, const Machine& machine) {
  const int64_t ksteps = (k + kBlock - 1) / kBlock;
  Spread best;
  for (int i = 0; i < (e == kPlain ? 3 : 2); ++i) {
    const Form& f = kForms[i];
    const int64_t n = tiles(f), units = machine.units(f.G);
    if (units < 1) continue;
    const int64_t rest = n % units;
    auto tile = [&](int64_t steps) { return std::max<int64_t>(steps * f.step + kEpilogues[e][i].more, kEpilogues[e][i].least) + f.tile; };
    auto offer = [&](int64_t whole, int64_t splits, int64_t parts, int64_t ns) {
      if (ns < best.ns) best = {i, (int)splits, whole, parts, ns};
    };
    offer(n, 1, 0, (n + units - 1) / units * tile(ksteps));
    if (e != kPlain || rest == 0) continue;
    const int64_t base = n / units * tile(ksteps) + kJoinNs;
    for (int64_t s = 2; s <= 32 && s * 4 <= ksteps; ++s) {
      const int64_t per = (ksteps + s - 1) / s;
      if ((ksteps + per - 1) / per != s) continue;  // a part without a step
      offer(n - rest, s, rest * s, base + (rest * s + units - 1) / units * tile(per) + rest * s * f.part);
    }
  }
  return best;
}
inline Spread spread(Epilogue e, int64_t m, int64_t n, int64_t k, const Machine& machine) {
  return spread(e, [=](const Form& f) { return f.tiles(m, n); }, k, machine);
}
// Both weights' gradients, [2 inner, width] and [width, inner].
inline Spread spread_weights(int64_t tokens, int64_t width, int64_t inner, const Machine& machine) {
  return spread(kPlain, [=](const Form& f) { return f.tiles(2 * inner, width) + f.tiles(width, inner); }, tokens, machine);
}

constexpr int64_t align_up(int64_t n) { return (n + 255) / 256 * 256; }

// The workspace: h [tokens, inner]; in the backward pass also (dg, du)
// [tokens, 2 inner] and, where they were not kept, (g, u) and their low parts
// [tokens, inner]; then the fp32 parts of one launch at a time.
struct Workspace {
  int64_t h = 0, dgu = 0, gu = 0, low = 0, parts = 0, bytes = 0;
  Workspace(int64_t tokens, int width, int inner, bool backward, bool kept, const Machine& machine) {
    int64_t at = align_up(tokens * inner * 2);
    int64_t most = 0;
    if (backward) {
      dgu = at;
      at += align_up(tokens * inner * 4);
      gu = at;
      if (!kept) at += align_up(tokens * inner * 4);
      low = at;
      if (!kept) at += align_up(tokens * inner * 2);
      most = std::max(spread(kPlain, tokens, width, 2 * (int64_t)inner, machine).bytes(),
                      spread_weights(tokens, width, inner, machine).bytes());
    } else {
      most = few_out(tokens, width, inner) ? 0 : spread(kPlain, tokens, width, inner, machine).bytes();
    }
    parts = at;
    bytes = at + align_up(most);
  }
};

}  // namespace feed_forward
}  // namespace fas
