// Host plan of a chunk's attention (rule documented on mla_chunk_plan in include/mla_decode.h).
//
// A unit of work is up to 512 queries of one request and head against a range of KV tiles of 128 rows, run by one pair of
// SMs. Whole units are handed out head by head, the longest of a head first, each to the pair that is free earliest: the units
// that run at once then read the same heads' K and V through L2, and the last ones are short. Where that leaves pairs idle for
// longer than a merge takes, the units are laid end to end in the same order and cut into equal shares, a pair each.
#include <algorithm>
#include <cstdint>
#include <queue>
#include <vector>

#include "mla_kernels.h"

namespace mla {
namespace {

// Costs in tenths of what two sub-tiles (of 256 queries) take for a KV tile, measured in SM cycles: two sub-tiles whose products
// and softmax run under each other take 3250 (1.7 us), one alone 2880. What a unit costs besides (loads of Q, the first scores,
// the epilogue; about 5 us). What a merge costs, and one more for so many rows of partial results (516 bytes, written and read).
constexpr int64_t kBoth = 10, kAlone = 9;
constexpr int64_t kUnitCost = 30;
constexpr int64_t kMergeCost = 25, kMergeRows = 1200;
constexpr int kMinTiles = 4;  // of a piece

struct QueryTile {
  int32_t request[4];  // q_start, q_len, kv_start, kv_len
  int32_t q0, rows;    // rows: queries, up to 512
  int32_t tiles[2];  // KV tiles of the sub-tiles
  int longest() const { return std::max(tiles[0], tiles[1]); }
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
  int32_t q_start = 0, kv_start = 0;
  std::vector<QueryTile> tiles;
  for (int b = 0; b < batch; ++b) {
    const int32_t n = q_lens[b], len = kv_lens[b];
    const int32_t blocks = n > 0 ? static_cast<int32_t>((static_cast<int64_t>(len) + 127) / 128) : 0;
    for (int32_t k = 0; k < blocks; ++k) {
      const int32_t tile[4] = {b, 128 * k, len, 0};
      p.kv_tiles.insert(p.kv_tiles.end(), tile, tile + 4);
    }
    for (int32_t q0 = 0; q0 < n; q0 += 512) {
      QueryTile q = {{q_start, n, kv_start, len}, q0, std::min(512, n - q0), {0, 0}};
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
    return a.longest() > b.longest();
  });
  int64_t total = 0;
  for (const QueryTile& q : tiles) {
    total += (tiles_cost(q, 0, q.longest()) + kUnitCost) * group;
  }
  typedef std::pair<int64_t, int> Free;  // (time, pair)
  struct Piece {
    int pair, head, tile, begin, end;  // tile: of `tiles`
  };
  std::vector<Piece> pieces;
  // Whole units; returns when the last pair ends.
  int64_t end = 0;
  {
    std::priority_queue<Free, std::vector<Free>, std::greater<Free>> free;
    for (int i = 0; i < pairs; ++i) free.push(Free(0, i));
    pieces.reserve(tiles.size() * static_cast<size_t>(group));
    for (int h = 0; h < group; ++h)
      for (int i = 0; i < static_cast<int>(tiles.size()); ++i) {
        const QueryTile& q = tiles[i];
        Free f = free.top();
        free.pop();
        pieces.push_back({f.second, h, i, 0, q.longest()});
        f.first += tiles_cost(q, 0, q.longest()) + kUnitCost;
        end = std::max(end, f.first);
        free.push(f);
      }
  }
  // Shares of at most `share`; returns false if the pairs do not suffice.
  auto cut = [&](int64_t share, std::vector<Piece>* out) -> bool {
    out->clear();
    int pair = 0;
    int64_t left = share;
    for (int h = 0; h < group; ++h)
      for (int i = 0; i < static_cast<int>(tiles.size()); ++i) {
        const QueryTile& q = tiles[i];
        const int n = q.longest();
        for (int t = 0, done = 0; !done;) {
          int t1 = n;
          if (tiles_cost(q, t, n) + kUnitCost > left) {
            // as many KV tiles as the share has room for, no piece below kMinTiles
            t1 = t + static_cast<int>(std::max<int64_t>(0, left - kUnitCost) / kBoth);
            while (t1 < n && tiles_cost(q, t, t1 + 1) + kUnitCost <= left) ++t1;
            t1 = std::min(t1, n - kMinTiles);
            if (t1 - t < kMinTiles) {
              if (left == share) t1 = n;  // (a unit that does not fit a whole share, nor can be cut)
              else {
                if (++pair == pairs) return false;
                left = share;
                continue;
              }
            }
          }
          out->push_back({pair, h, i, t, t1});
          left -= tiles_cost(q, t, t1) + kUnitCost;
          t = t1;
          done = t1 == n;
        }
      }
    return true;
  };
  // rows of partial results of a cut (units in order, a unit's pieces together)
  auto partial_rows = [&](const std::vector<Piece>& v) {
    int64_t rows = 0;
    for (const Piece& x : v)
      if (x.begin > 0 || x.end < tiles[x.tile].longest()) rows += tiles[x.tile].rows;
    return rows;
  };
  // Equal shares set all heads going at once: query tiles of one head no longer meet at its K and V in L2 (2048 queries after
  // 32768 rows at 128 heads, 512 units: 4451 us against 4260), so with many units they are for requests of one query tile, or
  // K and V that L2 holds (420 queries and three short requests at 128 heads: 180 us against 198).
  bool alone = true;
  for (int b = 0; b < batch; ++b) alone &= q_lens[b] <= 512;
  const int64_t units = static_cast<int64_t>(tiles.size()) * group;
  const bool may_cut = units <= 3 * pairs || (units <= 8 * pairs && (alone || static_cast<int64_t>(kv_start) * group * 512 <= (96 << 20)));
  if (units > 0 && may_cut && end > total / pairs + kMergeCost) {
    std::vector<Piece> shares;
    for (int64_t share = std::max<int64_t>(total / pairs, kUnitCost + 2 * kMinTiles * kBoth); share < end; share += share / 64 + 1) {
      if (!cut(share, &shares)) continue;
      const int64_t rows = partial_rows(shares);
      if (rows < (1ll << 31) && share + kMergeCost + rows / kMergeRows < end) pieces = shares;
      break;
    }
  }
  std::vector<std::vector<int32_t>> lists(pairs);
  int64_t slot = 0;
  for (size_t i = 0; i < pieces.size();) {
    const Piece& x = pieces[i];
    const QueryTile& q = tiles[x.tile];
    size_t n = 1;
    while (pieces[i + n - 1].end < q.longest()) ++n;  // a unit's pieces follow one another
    for (size_t k = 0; k < n; ++k) {
      const Piece& y = pieces[i + k];
      const int32_t at = n > 1 ? static_cast<int32_t>(slot + static_cast<int64_t>(k) * q.rows) : -1;
      const int32_t item[12] = {q.request[0], q.request[1], q.request[2], q.request[3], q.q0, x.head, y.begin, y.end, at, 0, 0, 0};
      lists[y.pair].insert(lists[y.pair].end(), item, item + 12);
    }
    if (n > 1) {
      const int32_t merge[8] = {q.request[0] + q.q0, q.rows, x.head, static_cast<int32_t>(slot), static_cast<int32_t>(n), 0, 0, 0};
      p.merges.insert(p.merges.end(), merge, merge + 8);
      slot += static_cast<int64_t>(n) * q.rows;
    }
    i += n;
  }
  p.slots = static_cast<int32_t>(slot);
  p.pair_items.push_back(0);
  for (const std::vector<int32_t>& l : lists) {
    if (l.empty()) continue;  // (a pair without work is not launched)
    p.items.insert(p.items.end(), l.begin(), l.end());
    p.pair_items.push_back(static_cast<int32_t>(p.items.size() / 12));
  }
  return p;
}

}  // namespace mla
