// Host plan of a chunk's attention (rule documented on mla_chunk_plan in include/mla_decode.h).
//
// A unit of work is up to 512 queries of one request and head against a range of KV tiles of 128 rows, run by one pair of
// SMs. Units are handed out head by head, the longest of a head first, each to the pair that is free earliest: the units
// that run at once then read the same heads' K and V through L2, and the last ones are short. Where there are too few of
// them, long units are cut over the KV tiles and their pieces merged.
#include <algorithm>
#include <cstdint>
#include <queue>
#include <vector>

#include "mla_kernels.h"

namespace mla {
namespace {

// Costs in tenths of what two sub-tiles (of 256 queries) take for a KV tile, measured in SM cycles: two sub-tiles whose products
// and softmax run under each other take 3090, one alone 2780. What a unit costs besides (loads of Q, the first scores, the
// epilogue), and what a merge has to save to be worth its launch and its partial results.
constexpr int64_t kBoth = 10, kAlone = 9;
constexpr int64_t kUnitCost = 25;
constexpr int64_t kMergeCost = 50;
constexpr int kMinTiles = 4;  // of a piece

struct QueryTile {
  int32_t req, q0, rows;  // rows: queries, up to 512
  int32_t tiles[2];  // KV tiles of the sub-tiles
};

int64_t tiles_cost(const QueryTile& q, int begin, int end) {
  const int lo = std::min(q.tiles[0], q.tiles[1]), hi = std::max(q.tiles[0], q.tiles[1]);
  const int64_t both = std::max(0, std::min(lo, end) - begin);
  const int64_t alone = std::max(0, std::min(hi, end) - std::max(lo, begin));
  return both * kBoth + alone * kAlone;
}

}  // namespace

ChunkPlan make_chunk_plan(const int32_t* q_lens, const int32_t* kv_lens, int batch, int heads, bool causal, int group,
                          int num_sms) {
  ChunkPlan p;
  const int pairs = std::max(1, num_sms / 2);
  p.requests.resize(4 * static_cast<size_t>(batch));
  int32_t q_start = 0, kv_start = 0;
  std::vector<QueryTile> tiles;
  for (int b = 0; b < batch; ++b) {
    const int32_t n = q_lens[b], len = kv_lens[b];
    const int32_t r[4] = {q_start, n, kv_start, len};
    std::copy(r, r + 4, p.requests.begin() + 4 * b);
    const int32_t blocks = (len + 127) / 128;
    p.tile_req.insert(p.tile_req.end(), blocks, b);
    for (int32_t q0 = 0; q0 < n; q0 += 512) {
      QueryTile q = {b, q0, std::min(512, n - q0), {0, 0}};
      for (int s = 0; s < 2; ++s) {
        const int64_t last = std::min<int64_t>(static_cast<int64_t>(q0) + 256 * (s + 1), n) - 1;
        if (q0 + 256 * static_cast<int64_t>(s) >= n) continue;
        const int64_t lim = causal ? std::min<int64_t>(len, static_cast<int64_t>(len) - n + last + 1) : len;
        q.tiles[s] = lim <= 0 ? 0 : static_cast<int32_t>((lim + 127) / 128);
      }
      tiles.push_back(q);
    }
    q_start += n;
    kv_start += blocks * 128;
  }
  // the longest first; a head's units stay together
  std::stable_sort(tiles.begin(), tiles.end(), [](const QueryTile& a, const QueryTile& b) {
    return std::max(a.tiles[0], a.tiles[1]) > std::max(b.tiles[0], b.tiles[1]);
  });
  int64_t total = 0, longest = 0;
  for (const QueryTile& q : tiles) {
    const int n = std::max(q.tiles[0], q.tiles[1]);
    const int64_t c = tiles_cost(q, 0, n);
    total += (c + kUnitCost) * group;
    longest = std::max(longest, c);
  }
  // The cut: pieces of at most `cap`. Returns the pieces of a query tile.
  auto pieces_of = [&](const QueryTile& q, int64_t cap) -> int {
    const int n = std::max(q.tiles[0], q.tiles[1]);
    const int64_t c = tiles_cost(q, 0, n);
    if (cap <= 0 || c <= cap) return 1;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((c + cap - 1) / cap, n / kMinTiles)));
  };
  typedef std::pair<int64_t, int> Free;  // (time, pair)
  auto run = [&](int64_t cap, std::vector<std::vector<int32_t>>* lists) -> int64_t {
    std::priority_queue<Free, std::vector<Free>, std::greater<Free>> free;
    for (int i = 0; i < pairs; ++i) free.push(Free(0, i));
    int64_t end = 0;
    bool cut = false;
    int64_t slot = 0;  // rows of partial results
    for (int h = 0; h < group; ++h)
      for (const QueryTile& q : tiles) {
        const int n = std::max(q.tiles[0], q.tiles[1]);
        const int pieces = pieces_of(q, cap);
        cut |= pieces > 1;
        for (int i = 0; i < pieces; ++i) {
          const int t0 = static_cast<int>(static_cast<int64_t>(n) * i / pieces);
          const int t1 = static_cast<int>(static_cast<int64_t>(n) * (i + 1) / pieces);
          Free f = free.top();
          free.pop();
          if (lists) {
            const int32_t item[8] = {q.req, q.q0, h, t0, t1, pieces > 1 ? static_cast<int32_t>(slot + static_cast<int64_t>(i) * q.rows) : -1, 0, 0};
            (*lists)[f.second].insert((*lists)[f.second].end(), item, item + 8);
          }
          f.first += tiles_cost(q, t0, t1) + kUnitCost;
          end = std::max(end, f.first);
          free.push(f);
        }
        if (pieces > 1) {
          if (lists) {
            const int32_t merge[8] = {q.req, q.q0, h, static_cast<int32_t>(slot), pieces, 0, 0, 0};
            p.merges.insert(p.merges.end(), merge, merge + 8);
          }
          slot += static_cast<int64_t>(pieces) * q.rows;
        }
      }
    if (lists) p.slots = static_cast<int32_t>(slot);
    return slot >= (1ll << 31) ? INT64_MAX : end + (cut ? kMergeCost : 0);
  };
  // no cut, or the one that ends first among pieces of a pair's whole share and of parts of it
  int64_t best_cap = 0;
  if (!tiles.empty()) {
    const int64_t share = std::max<int64_t>(1, total / pairs);
    if (longest > share / 4) {
      int64_t best = run(0, nullptr);
      for (int k = 1; k <= 24; ++k) {
        const int64_t cap = std::max<int64_t>(1, share * 6 / (4 + k));  // 1.2 shares down to a fifth of one
        const int64_t end = run(cap, nullptr);
        if (end < best) {
          best = end;
          best_cap = cap;
        }
      }
    }
  }
  std::vector<std::vector<int32_t>> lists(pairs);
  run(best_cap, &lists);
  p.pair_items.push_back(0);
  for (const std::vector<int32_t>& l : lists) {
    if (l.empty()) continue;  // (a pair without work is not launched)
    p.items.insert(p.items.end(), l.begin(), l.end());
    p.pair_items.push_back(static_cast<int32_t>(p.items.size() / 8));
  }
  return p;
}

}  // namespace mla
