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

}  // namespace

std::string score_plan_layout(const int32_t* cu, int n_seqs, const int32_t* prefix_lens,
                              bool bidirectional, int H, int sms, const int32_t* buckets,
                              int n_dist, ScorePlanHeader* h) {
  char buf[160];
  if (!cu) return "cu_seqlens is NULL";
  if (n_seqs < 1) return "n_seqs must be >= 1";
  if (H < 1 || H > 65535) return "H must be in [1, 65535]";
  if (sms < 1) return "n_sms must be >= 1";
  if (cu[0] != 0) return "cu_seqlens[0] must be 0";
  if (n_dist < 0 || n_dist > kMaxDist) return "n_dist must be in [0, 65536]";
  if (n_dist > 0 && !buckets) return "buckets is NULL";
  int64_t fwd = 0, bwd = 0, tiles = 0, walk = 0;
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
    parts(cu, prefix_lens, bidirectional, i, [&](int64_t, int64_t rows, bool) {
      fwd += cdiv(rows, kFwdPairQ);
      bwd += cdiv(rows, kBwdTileK);
    });
    tiles += cdiv(len, kTile32);
    walk = std::max(walk, cdiv(len, kTile32));
  }
  int nb = 0;
  for (int i = 0; i < n_dist; ++i) {
    if (buckets[i] < 0 || buckets[i] >= kMaxDist) return "a bucket is not in [0, 65536)";
    nb = std::max(nb, buckets[i] + 1);
  }
  if (fwd * H > 0x7fffffffLL) return "too many work units";
  ScorePlanHeader p{};
  p.magic = kScorePlanMagic;
  p.T = cu[n_seqs];
  p.H = H;
  p.n_seqs = n_seqs;
  p.n_sms = sms;
  p.bidirectional = bidirectional ? 1 : 0;
  p.n_dist = n_dist;
  p.n_buckets = nb;
  p.n_fwd = (int32_t)fwd;
  p.n_bwd = (int32_t)bwd;
  p.n_tiles = (int32_t)tiles;
  p.max_walk = (int32_t)walk;
  p.n_units = (int32_t)(fwd * H);
  p.grid = std::min<int32_t>(p.n_units, sms);
  p.item_major = item_major(p.n_units, sms) ? 1 : 0;
  uint64_t o = up256(sizeof(ScorePlanHeader));
  p.fwd = o; o = up256(o + fwd * sizeof(FwdItem));
  p.bwd = o; o = up256(o + bwd * sizeof(BwdItem));
  p.runs = o; o = up256(o + bwd * sizeof(Seg));
  p.units = o;
  o = up256(o + (uint64_t)(p.n_units + p.grid + 1) * sizeof(int32_t));
  p.buckets = o; o = up256(o + (uint64_t)n_dist * sizeof(int32_t));
  p.tiles = o; o = up256(o + tiles * sizeof(Tile32));
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
        it.n_tiles = (int32_t)cdiv(both ? rows : std::min<int64_t>(len, t0 + it.q_len), kFwdTileK);
        fwd.push_back(it);
      }
      for (int64_t u0 = first; u0 < first + rows; u0 += kBwdTileK) {
        // keys u0 .. of the sample against the queries that see them: every
        // row of the sample for a both-way prefix, else rows from u0 on
        BwdItem it{};
        it.k_row0 = it.dk_row0 = (int32_t)(s0 + u0);
        it.k_len = (int32_t)std::min<int64_t>(kBwdTileK, first + rows - u0);
        it.nseg = 1;
        it.dk_mode = DK_TEXT;
        it.flags = F_FIRST;
        Seg& s = it.seg[0];
        const int64_t q0 = both ? 0 : u0;
        s.row0 = (int32_t)(s0 + q0);
        s.len = (int32_t)(len - q0);
        s.src = SRC_NAT;
        s.causal = both ? 0 : 1;
        s.delta = 0;
        s.rel = (int32_t)(q0 - u0);
        it.n_tiles = (int32_t)cdiv(s.len, 128);
        bwd.push_back(it);
      }
    });
    for (int64_t t0 = 0; t0 < len; t0 += kTile32) {
      Tile32 t{};
      t.row0 = (int32_t)(s0 + t0);
      t.len = (int32_t)std::min<int64_t>(kTile32, len - t0);
      t.seq0 = (int32_t)s0;
      t.seq_len = (int32_t)len;
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
  if (h.n_dist > 0) memcpy(b + h.buckets, buckets, h.n_dist * sizeof(int32_t));
  if (h.n_units > 0) {
    std::vector<int32_t> units, off;
    plan_unit_lists(fwd, h.H, h.grid, &units, &off, h.item_major != 0);
    memcpy(b + h.units, units.data(), units.size() * sizeof(int32_t));
    memcpy(b + h.units + units.size() * sizeof(int32_t), off.data(), off.size() * sizeof(int32_t));
  }
}

}  // namespace cpattn
