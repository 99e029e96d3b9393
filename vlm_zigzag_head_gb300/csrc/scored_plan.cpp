// Host planner of attention with modified scores.
#include "scored_plan.h"

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <vector>

namespace cpattn {

namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

// Calls f(first row, rows, prefix) for the parts of sample i that are tiled
// separately: a prefix that sees itself in both directions, and the rest.
template <typename F>
void parts(const int32_t* cu, const int32_t* prefix_lens, bool bidirectional, int i, F f) {
  const int64_t len = (int64_t)cu[i + 1] - cu[i];
  const int64_t pre = bidirectional && prefix_lens ? prefix_lens[i] : 0;
  if (pre > 0) f((int64_t)0, pre, true);
  if (len > pre) f(pre, len - pre, false);
}

// Costs beside a unit's tiles, in half tiles (about 1.1 us each): its loads and
// epilogue, what a part adds to them (fp32 results that are read again, or sums in
// memory), and the join (or the clearing and rounding of the sums).
constexpr int64_t kUnitCost = 7, kPartCost = 3, kJoinCost = 4;

// Time of the launch with parts of at most `limit` tiles (0: none cut): longest
// first onto the SM that is free first.  runs[n]: runs of n tiles over all heads.
int64_t makespan(const std::vector<int64_t>& runs, int64_t limit, int sms) {
  std::vector<int64_t> units(runs.size(), 0);   // by tiles
  std::vector<int64_t> cut(runs.size(), 0);
  bool any = false;
  for (size_t n = 1; n < runs.size(); ++n) {
    if (runs[n] == 0) continue;
    const int64_t np = limit > 0 ? cdiv((int64_t)n, limit) : 1;
    any = any || np > 1;
    for (int64_t x = 0; x < np; ++x) {
      const int64_t tiles = n * (x + 1) / np - n * x / np;
      (np > 1 ? cut : units)[tiles] += runs[n];
    }
  }
  std::vector<int64_t> free_at(sms, 0);
  int64_t last = 0;
  for (size_t n = runs.size(); n-- > 1;)
    for (int64_t x = 0; x < units[n] + cut[n]; ++x) {
      const int64_t t = free_at[0] + 2 * (int64_t)n + kUnitCost + (x < cut[n] ? kPartCost : 0);
      replace_least(free_at, t);
      last = std::max(last, t);
    }
  return last + (any ? kJoinCost : 0);
}

// Tiles of the longest part of a run, 0 to cut none: the limit with the shortest
// launch, where that saves an eighth.  No search where the longest run is within
// an SM's share (what follows it fills the SMs) or units are many (the search
// would cost the host milliseconds).  Forward / backward, parts against whole, us:
// 2048 tokens x 1 head 51 -> 40 / 62 -> 28, 4096 x 4 82 -> 54 / 105 -> 84, 12 000 x 1
// 233 -> 66 / 202 -> 95; where the rule cuts nothing, parts of 16 tiles: 4096 x 16
// 104 -> 144, 8192 x 8 138 -> 188.
int64_t part_limit(const std::vector<int64_t>& runs, int sms) {
  const int64_t longest = (int64_t)runs.size() - 1;
  int64_t total = 0, units = 0;
  for (int64_t n = 1; n <= longest; ++n) {
    total += runs[n] * n;
    units += runs[n];
  }
  if (longest <= std::max<int64_t>(cdiv(total, sms), 3) || !item_major(units, sms)) return 0;
  const int64_t whole = makespan(runs, 0, sms);
  int64_t best = whole - whole / 8, limit = 0, last = longest;
  for (int64_t np : {2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64}) {
    const int64_t l = cdiv(longest, np);
    if (l == last || l < 2) continue;
    last = l;
    const int64_t t = makespan(runs, l, sms);
    if (t < best) {
      best = t;
      limit = l;
    }
  }
  return limit;
}
int64_t n_parts(int64_t tiles, int64_t limit) { return limit > 0 ? cdiv(tiles, limit) : 1; }

int64_t fwd_tiles(int64_t t0, int64_t rows_left, int64_t part_rows, bool both) {
  return cdiv(both ? part_rows : t0 + std::min<int64_t>(kFwdPairQ, rows_left), kFwdTileK);
}

// h's part limits.
void choose_parts(const int32_t* cu, int n_seqs, const int32_t* prefix_lens, bool bidirectional,
                  int H, ScorePlanHeader* h) {
  std::vector<int64_t> runs[2];
  for (int i = 0; i < n_seqs; ++i) {
    const int64_t len = (int64_t)cu[i + 1] - cu[i];
    parts(cu, prefix_lens, bidirectional, i, [&](int64_t first, int64_t rows, bool both) {
      auto add = [&](int x, int64_t n) {
        if ((int64_t)runs[x].size() <= n) runs[x].resize(n + 1, 0);
        runs[x][n] += H;
      };
      for (int64_t t = 0; t < rows; t += kFwdPairQ)
        add(0, fwd_tiles(first + t, rows - t, rows, both));
      for (int64_t t = 0; t < rows; t += kBwdTileK)
        add(1, cdiv(both ? len : len - first - t, 128));
    });
  }
  h->fwd_part = (int32_t)part_limit(runs[0], h->n_sms);
  h->bwd_part = (int32_t)part_limit(runs[1], h->n_sms);
}

}  // namespace

std::string score_plan_layout(const int32_t* cu, int n_seqs, const int32_t* prefix_lens,
                              bool bidirectional, int H, int sms, const int32_t* buckets,
                              int n_dist, ScorePlanHeader* h) {
  char buf[160];
  if (!cu) return "cu_seqlens is NULL";
  if (n_seqs < 1) return "n_seqs must be >= 1";
  if (H < 1 || H > 65535) return "H must be in [1, 65535]";
  if (sms < 1 || sms > 4096) return "n_sms must be in [1, 4096]";
  if (cu[0] != 0) return "cu_seqlens[0] must be 0";
  if (n_dist < 0 || n_dist > kMaxDist) return "n_dist must be in [0, 65536]";
  if (n_dist > 0 && !buckets) return "buckets is NULL";
  int64_t fwd = 0, bwd = 0, tiles = 0, walk = 0, joins = 0, run_rows = 0, key_tiles = 0;
  int64_t n_short = 0;
  for (int i = 0; i < n_seqs; ++i) {
    const int64_t len = (int64_t)cu[i + 1] - cu[i];
    if (len < 0) {
      snprintf(buf, sizeof buf, "cu_seqlens falls at sample %d", i);
      return buf;
    }
    if (prefix_lens && (prefix_lens[i] < 0 || prefix_lens[i] > len)) {
      snprintf(buf, sizeof buf, "prefix of sample %d (%d tokens) is not in [0, %lld]", i,
               prefix_lens[i], (long long)len);
      return buf;
    }
    tiles += cdiv(len, kTile32);
    if (len <= kF16Tokens) n_short += cdiv(len, kTile32);
    walk = std::max(walk, cdiv(len, kTile32));
  }
  ScorePlanHeader p{};
  p.n_sms = sms;
  choose_parts(cu, n_seqs, prefix_lens, bidirectional, H, &p);
  for (int i = 0; i < n_seqs; ++i)
    parts(cu, prefix_lens, bidirectional, i, [&](int64_t first, int64_t rows, bool both) {
      for (int64_t t = 0; t < rows; t += kFwdPairQ) {
        const int64_t n = n_parts(fwd_tiles(first + t, rows - t, rows, both), p.fwd_part);
        fwd += n;
        joins += n > 1;
        run_rows += n > 1 ? n * std::min<int64_t>(kFwdPairQ, rows - t) : 0;
      }
      for (int64_t t = 0; t < rows; t += kBwdTileK) {
        const int64_t len = (int64_t)cu[i + 1] - cu[i];
        bwd += n_parts(cdiv(both ? len : len - first - t, 128), p.bwd_part);
        ++key_tiles;
      }
    });
  int nb = 0;
  for (int i = 0; i < n_dist; ++i) {
    if (buckets[i] < 0 || buckets[i] >= kMaxDist) return "a bucket is not in [0, 65536)";
    nb = std::max(nb, buckets[i] + 1);
  }
  if (fwd * H > 0x7fffffffLL || bwd > 0x7fffffffLL || run_rows > 0x7fffffffLL)
    return "too many work units";
  p.magic = kScorePlanMagic;
  p.T = cu[n_seqs];
  p.H = H;
  p.n_seqs = n_seqs;
  p.bidirectional = bidirectional ? 1 : 0;
  p.n_dist = n_dist;
  p.n_buckets = nb;
  p.n_fwd = (int32_t)fwd;
  p.n_bwd = (int32_t)bwd;
  p.n_tiles = (int32_t)tiles;
  p.n_joins = (int32_t)joins;
  p.run_rows = (int32_t)run_rows;
  p.bwd_cut = bwd > key_tiles ? 1 : 0;
  p.max_walk = (int32_t)walk;
  p.n_short = (int32_t)n_short;
  p.n_units = (int32_t)(fwd * H);
  p.grid = std::min<int32_t>(p.n_units, sms);
  p.item_major = item_major(p.n_units, sms) ? 1 : 0;
  uint64_t o = up256(sizeof(ScorePlanHeader));
  p.fwd = o; o = up256(o + fwd * sizeof(FwdItem));
  p.bwd = o; o = up256(o + bwd * sizeof(BwdItem));
  p.runs = o; o = up256(o + bwd * sizeof(Seg));
  p.units = o;
  o = up256(o + ((uint64_t)p.n_units + p.grid + 1) * sizeof(int32_t));
  p.buckets = o; o = up256(o + (uint64_t)n_dist * sizeof(int32_t));
  p.tiles = o; o = up256(o + tiles * sizeof(Tile32));
  p.joins = o; o = up256(o + joins * sizeof(Join));
  p.total = o;
  *h = p;
  return "";
}

void score_plan_build(const ScorePlanHeader& h, const int32_t* cu, const int32_t* prefix_lens,
                      const int32_t* buckets, void* block) {
  char* b = static_cast<char*>(block);
  memset(b, 0, h.total);
  memcpy(b, &h, sizeof h);
  const bool bidir = h.bidirectional != 0;
  std::vector<FwdItem> fwd;
  std::vector<BwdItem> bwd;
  std::vector<Tile32> tiles;
  std::vector<Join> joins;
  int32_t run_rows = 0;
  for (int i = 0; i < h.n_seqs; ++i) {
    const int64_t s0 = cu[i], len = (int64_t)cu[i + 1] - s0;
    parts(cu, prefix_lens, bidir, i, [&](int64_t first, int64_t rows, bool both) {
      for (int64_t t0 = first; t0 < first + rows; t0 += kFwdPairQ) {
        // queries t0 .. of the sample against its keys from 0 on: a both-way
        // prefix sees `rows` keys, the other rows keys up to their own
        FwdItem it{};
        it.q_row0 = it.out_row0 = (int32_t)(s0 + t0);
        it.q_len = (int32_t)std::min<int64_t>(kFwdPairQ, first + rows - t0);
        it.q_src = SRC_NAT;
        it.nseg = 1;
        it.run_row0 = -1;
        it.flags = F_FIRST | F_FINAL;
        Seg& s = it.seg[0];
        s.row0 = (int32_t)s0;
        s.len = (int32_t)(both ? rows : len);
        s.src = SRC_NAT;
        s.causal = both ? 0 : 1;
        s.delta = s.rel = (int32_t)t0;
        const int64_t nt = fwd_tiles(t0, first + rows - t0, rows, both);
        const int64_t np = n_parts(nt, h.fwd_part);
        if (np > 1) {   // parts leave fp32 results
          joins.push_back({it.out_row0, it.q_len, run_rows, (int32_t)np});
          it.flags = F_FIRST;
        }
        const Seg whole = s;
        for (int64_t x = 0; x < np; ++x) {
          const int64_t from = nt * x / np, to = nt * (x + 1) / np;
          s = whole;
          s.row0 += (int32_t)(from * kFwdTileK);
          s.len = (int32_t)((x + 1 < np ? to * kFwdTileK : whole.len) - from * kFwdTileK);
          s.delta = s.rel = (int32_t)(t0 - from * kFwdTileK);
          it.n_tiles = (int32_t)(to - from);
          if (np > 1) {
            it.run_row0 = run_rows;
            run_rows += it.q_len;
          }
          fwd.push_back(it);
        }
      }
      for (int64_t u0 = first; u0 < first + rows; u0 += kBwdTileK) {
        // keys u0 .. of the sample against the queries that see them: every
        // row of the sample for a both-way prefix, else rows from u0 on
        BwdItem it{};
        it.k_row0 = it.dk_row0 = (int32_t)(s0 + u0);
        it.k_len = (int32_t)std::min<int64_t>(kBwdTileK, first + rows - u0);
        it.nseg = 1;
        it.dk_mode = DK_TEXT;
        it.slot = i;
        it.flags = F_FIRST;
        Seg& s = it.seg[0];
        const int64_t q0 = both ? 0 : u0;
        s.row0 = (int32_t)(s0 + q0);
        s.len = (int32_t)(len - q0);
        s.src = SRC_NAT;
        s.causal = both ? 0 : 1;
        const Seg whole = s;
        const int64_t nt = cdiv(whole.len, 128), np = n_parts(nt, h.bwd_part);
        for (int64_t x = 0; x < np; ++x) {
          const int64_t from = nt * x / np, to = nt * (x + 1) / np;
          s = whole;
          s.row0 += (int32_t)(from * 128);
          s.len = (int32_t)((x + 1 < np ? to * 128 : whole.len) - from * 128);
          s.delta = both ? 0 : (int32_t)(from * 128);
          s.rel = (int32_t)(q0 - u0 + from * 128);
          it.n_tiles = (int32_t)(to - from);
          bwd.push_back(it);
        }
      }
    });
    for (int64_t t0 = 0; t0 < len; t0 += kTile32) {
      Tile32 t{};
      t.row0 = (int32_t)(s0 + t0);
      t.len = (int32_t)std::min<int64_t>(kTile32, len - t0);
      t.seq0 = (int32_t)s0;
      t.seq_len = (int32_t)len;
      t.sample = i;
      t.prefix = bidir && prefix_lens ? prefix_lens[i] : 0;
      tiles.push_back(t);
    }
  }
  // heaviest first, as every work list of the library
  std::stable_sort(fwd.begin(), fwd.end(),
                   [](const FwdItem& x, const FwdItem& y) { return x.n_tiles > y.n_tiles; });
  std::stable_sort(bwd.begin(), bwd.end(),
                   [](const BwdItem& x, const BwdItem& y) { return x.n_tiles > y.n_tiles; });
  Seg* runs = reinterpret_cast<Seg*>(b + h.runs);
  for (size_t i = 0; i < bwd.size(); ++i) {
    bwd[i].run0 = (int32_t)i;
    runs[i] = bwd[i].seg[0];
    bwd[i].seg[0] = Seg{};
  }
  if (!fwd.empty()) memcpy(b + h.fwd, fwd.data(), fwd.size() * sizeof(FwdItem));
  if (!bwd.empty()) memcpy(b + h.bwd, bwd.data(), bwd.size() * sizeof(BwdItem));
  if (!tiles.empty()) memcpy(b + h.tiles, tiles.data(), tiles.size() * sizeof(Tile32));
  if (!joins.empty()) memcpy(b + h.joins, joins.data(), joins.size() * sizeof(Join));
  if (h.n_dist > 0) memcpy(b + h.buckets, buckets, h.n_dist * sizeof(int32_t));
  if (h.n_units > 0) {
    std::vector<int32_t> units, off;
    plan_unit_lists(fwd, h.H, h.grid, &units, &off, h.item_major != 0);
    memcpy(b + h.units, units.data(), units.size() * sizeof(int32_t));
    memcpy(b + h.units + units.size() * sizeof(int32_t), off.data(), off.size() * sizeof(int32_t));
  }
}

}  // namespace cpattn
