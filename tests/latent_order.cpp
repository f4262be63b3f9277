// Host program for tests/test_latent_order.py: the waits and arrivals of the latent kernels' warps, as
// straight programs over the kernels' own rings (spa_latent_ring.h), walked through every interleaving.
//
// A wait for phase n of a barrier by its parity is sound where the barrier has completed n phases (the
// wait holds) or n + 1 (it passes).  With fewer it passes although the phase is to come, with more it
// holds although the phase is over.  The program looks at every warp that stands before a wait, in
// every state that can be reached, and prints the first wait that is neither, or a state in which all
// are stuck.
//
//   latent_order decode FP8 BOXED PRING GROW TILES...   tiles of each token; GROW: bit k set where the
//       maximum moves at tile k; PRING: slots of the P-ready and PV-done barriers where they are a ring
//       of their own (0: the kernel's, at the tile's slot of the ring of rows)
//   latent_order prefill CHUNKS VORDER S0,S1,RAGGED...  key steps of both query tiles of each item, and
//       whether the last step ends inside a tile; VORDER: the loader waits for V as the kernel does
// prints "ok STATES" or "WHAT AT ..."
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>
#include <unordered_set>
#include <vector>

#include "spa_latent_ring.h"

namespace {

struct Op {
  enum Kind { kWait, kArrive, kIssue } kind;
  int bar;      // wait, arrive: the barrier.  issue: the queue (< 0: a copy, which lands in any order)
  int phase;    // wait
  std::vector<int> bars;   // issue: one arrival after the other
};
struct Warp {
  std::string name;
  std::vector<Op> ops;
};

struct Model {
  std::vector<std::string> bar_name;
  std::vector<int> bar_count;
  std::map<std::string, int> bars;
  std::vector<Warp> warps;
  int queues = 0;

  int bar(const std::string& kind, int slot, int count = 1) {
    const std::string n = kind + "[" + std::to_string(slot) + "]";
    const auto it = bars.find(n);
    if (it != bars.end()) return it->second;
    bars[n] = (int)bar_name.size();
    bar_name.push_back(n);
    bar_count.push_back(count);
    return bars[n];
  }
  // phase: the one waited for; parity: what the kernel passes for it
  void wait(Warp& w, int b, int phase, uint32_t parity) {
    if (((uint32_t)phase & 1u) != (parity & 1u)) {
      std::printf("parity of another phase at %s, %s phase %d\n", w.name.c_str(), bar_name[b].c_str(), phase);
      std::exit(0);
    }
    w.ops.push_back({Op::kWait, b, phase, {}});
  }
  void arrive(Warp& w, int b) { w.ops.push_back({Op::kArrive, b, 0, {}}); }
  void issue(Warp& w, int queue, std::vector<int> to) { w.ops.push_back({Op::kIssue, queue, 0, to}); }

  void run() const;
};

// A state: a program counter a warp, arrivals a barrier, entries done a queue, copies in flight.
void Model::run() const {
  // what the queues and copies do is known from the programs: entry i of a queue, copy i of a warp
  struct Async {
    int warp, pc, at;   // issued once the warp is past pc; its arrival
    int queue;          // (copies: -1)
  };
  std::vector<std::vector<Async>> q(queues);
  std::vector<Async> copies;
  for (int w = 0; w < (int)warps.size(); ++w)
    for (int i = 0; i < (int)warps[w].ops.size(); ++i) {
      const Op& o = warps[w].ops[i];
      if (o.kind != Op::kIssue) continue;
      for (const int b : o.bars) {
        if (o.bar < 0) copies.push_back({w, i, b, -1});
        else q[o.bar].push_back({w, i, b, o.bar});
      }
    }
  const size_t nw = warps.size(), nb = bar_name.size();
  const size_t len = nw + nb + queues + copies.size();
  std::unordered_set<std::string> seen;
  std::vector<std::string> todo;
  std::string s(len, '\0');
  seen.insert(s);
  todo.push_back(s);
  auto phases = [&](const std::string& x, int b) { return (unsigned char)x[nw + b] / bar_count[b]; };
  while (!todo.empty()) {
    const std::string x = todo.back();
    todo.pop_back();
    bool moved = false, finished = true;
    auto go = [&](const std::string& y) {
      moved = true;
      if (seen.insert(y).second) todo.push_back(y);
    };
    for (size_t w = 0; w < nw; ++w) {
      const int pc = (unsigned char)x[w];
      if (pc == (int)warps[w].ops.size()) continue;
      finished = false;
      const Op& o = warps[w].ops[pc];
      std::string y = x;
      y[w] = (char)(pc + 1);
      if (o.kind == Op::kWait) {
        const int c = phases(x, o.bar);
        if (c != o.phase && c != o.phase + 1) {
          std::printf("%s at %s, %s phase %d of %d\n", c < o.phase ? "early" : "late", warps[w].name.c_str(),
                      bar_name[o.bar].c_str(), o.phase, c);
          return;
        }
        if (c == o.phase + 1) go(y);
      } else {
        if (o.kind == Op::kArrive) ++y[nw + o.bar];
        go(y);
      }
    }
    for (int i = 0; i < queues; ++i) {
      const int d = (unsigned char)x[nw + nb + i];
      if (d == (int)q[i].size() || (unsigned char)x[q[i][d].warp] <= q[i][d].pc) continue;
      std::string y = x;
      ++y[nw + nb + i];
      ++y[nw + q[i][d].at];
      go(y);
    }
    for (size_t i = 0; i < copies.size(); ++i) {
      const size_t at = nw + nb + queues + i;
      if (x[at] || (unsigned char)x[copies[i].warp] <= copies[i].pc) continue;
      std::string y = x;
      y[at] = 1;
      ++y[nw + copies[i].at];
      go(y);
    }
    if (!moved && !finished) {
      std::printf("stuck at");
      for (size_t w = 0; w < nw; ++w) std::printf(" %s:%d", warps[w].name.c_str(), (int)(unsigned char)x[w]);
      std::printf("\n");
      return;
    }
  }
  std::printf("ok %zu\n", seen.size());
}

using spa::LatentTileRing;

void decode(bool fp8, bool boxed, int pring, unsigned grow, const std::vector<int>& tokens) {
  constexpr int kInfos = 4;
  const int sbufs = fp8 ? 2 : 1;
  Model m;
  m.queues = 2;
  Warp load{"loader", {}}, s{"S", {}}, o{"O", {}}, soft{"softmax", {}}, q{"q", {}};
  struct Tile { int token; bool first, last; };
  std::vector<Tile> tiles;
  for (int t = 0; t < (int)tokens.size(); ++t)
    for (int j = 0; j < tokens[t]; ++j) tiles.push_back({t, j == 0, j == tokens[t] - 1});
  const int n = (int)tiles.size();
  auto full = [&](int i) { return m.bar("FULL", i); };
  auto empty = [&](int i) { return m.bar("EMPTY", i); };
  auto info_full = [&](int k) { return m.bar("INFO_FULL", k % kInfos); };
  auto info_empty = [&](int k) { return m.bar("INFO_EMPTY", k % kInfos, 4); };
  auto s_full = [&](int k) { return m.bar("S_FULL", k % sbufs); };
  auto s_empty = [&](int k) { return m.bar("S_EMPTY", k % sbufs); };
  // P ready, and MMAs of O done, of tile k at position `at` of the ring of rows
  auto p_full = [&](int k, const LatentTileRing& at) { return m.bar("P_FULL", pring ? k % pring : at.slot); };
  auto wait_pv = [&](int k, const LatentTileRing& at) {
    if (pring) m.wait(soft, m.bar("PV_DONE", k % pring), k / pring, (uint32_t)(k / pring));
    else m.wait(soft, empty(at.slot), k / LatentTileRing::kSlots, at.parity);
  };
  auto put_q = [&](int token) {
    m.wait(q, m.bar("Q_EMPTY", 0), token - 1, (uint32_t)(token - 1) & 1);
    m.arrive(q, m.bar("Q_FULL", 0));
  };
  if (boxed) {
    m.arrive(load, m.bar("TOKEN", 0));
    m.wait(q, m.bar("TOKEN", 0), 0, 0);
    put_q(0);
  }
  m.wait(o, info_full(0), 0, 0);
  m.wait(soft, info_full(0), 0, 0);
  LatentTileRing at, at1, at2;
  for (int k = 0; k < n; ++k) {
    const Tile& t = tiles[k];
    const int use = k / LatentTileRing::kSlots;
    const int ip = k / kInfos, sp = k / sbufs;
    if (k > 0) {
      at2 = at1;
      at1 = at;
      at.next();
    }
    auto copy = [&](Warp& w) {
      m.wait(w, empty(at.slot), use - 1, at.parity ^ 1);
      m.issue(w, -1, {full(at.slot)});
    };
    // loader
    if (boxed) copy(load);
    m.wait(load, info_empty(k), ip - 1, (uint32_t)(ip & 1) ^ 1);
    m.arrive(load, info_full(k));
    // queries (and rows by cp.async)
    m.wait(q, info_full(k), ip, ip & 1);
    if (!boxed) copy(q);
    m.arrive(q, info_empty(k));
    if (t.first && !(boxed && k == 0)) put_q(t.token);
    // S
    m.wait(s, info_full(k), ip, ip & 1);
    m.arrive(s, info_empty(k));
    if (t.first) m.wait(s, m.bar("Q_FULL", 0), t.token, t.token & 1);
    m.wait(s, full(at.slot), use, at.parity);
    m.wait(s, s_empty(k), sp - 1, (uint32_t)(sp & 1) ^ 1);
    m.issue(s, 0, {s_full(k)});
    if (t.last) m.issue(s, 0, {m.bar("Q_EMPTY", 0)});
    // softmax
    m.wait(soft, s_full(k), sp, sp & 1);
    m.arrive(soft, s_empty(k));
    if (pring && fp8 && k >= 2) wait_pv(k - 2, at2);   // (its P had two places of its own then)
    if ((grow >> k & 1) && !t.first) wait_pv(k - 1, at1);
    m.arrive(soft, p_full(k, at));
    m.arrive(soft, info_empty(k));
    if (t.last) {
      wait_pv(k, at);
      m.arrive(soft, m.bar("O_FREE", 0));
    }
    // O
    if (pring) m.wait(o, p_full(k, at), k / pring, (uint32_t)(k / pring));
    else m.wait(o, p_full(k, at), use, at.parity);
    m.arrive(o, info_empty(k));
    if (t.first) m.wait(o, m.bar("O_FREE", 0), t.token - 1, (uint32_t)(t.token - 1) & 1);
    m.issue(o, 1, {empty(at.slot)});
    if (pring) m.issue(o, 1, {m.bar("PV_DONE", k % pring)});
  }
  m.warps = {load, s, o, soft, q};
  m.run();
}

struct Item { int steps[2]; bool ragged; };

void prefill(int chunks, bool vorder, const std::vector<Item>& items) {
  constexpr int kKs = 4, kVs = 2, kItems = 2;
  Model m;
  m.queues = 2;
  Warp load{"loader", {}}, s{"S", {}}, o{"O", {}}, soft[2] = {{"softmax 0", {}}, {"softmax 1", {}}};
  auto next_item = [&](Warp& w, int n) {
    m.wait(w, m.bar("I_FULL", n % kItems), n / kItems, (n / kItems) & 1);
    m.arrive(w, m.bar("I_EMPTY", n % kItems, 4));
  };
  auto bar = [&](const char* kind, int slot) { return m.bar(kind, slot); };
  int kc = 0, vc = 0, issued = 0, l_qs[2] = {}, s_qs[2] = {}, done[2] = {}, opened[2] = {};
  for (int n = 0; n <= (int)items.size(); ++n) {
    m.wait(load, m.bar("I_EMPTY", n % kItems, 4), n / kItems - 1, (uint32_t)((n / kItems) & 1) ^ 1);
    m.arrive(load, bar("I_FULL", n % kItems));
    next_item(s, n);
    next_item(o, n);
    next_item(soft[0], n);
    next_item(soft[1], n);
    if (n == (int)items.size()) break;
    const Item& it = items[n];
    const int steps = it.steps[0] > it.steps[1] ? it.steps[0] : it.steps[1];
    for (int t = 0; t < 2; ++t) {
      if (it.steps[t] == 0) continue;
      m.wait(load, bar("Q_EMPTY", t), l_qs[t] - 1, (uint32_t)(l_qs[t] & 1) ^ 1);
      ++l_qs[t];
      m.issue(load, -1, {bar("Q_FULL", t)});
    }
    int sdone[2] = {done[0], done[1]};
    for (int j = 0; j < steps; ++j, kc += chunks, ++vc) {
      const bool ends = it.ragged && j == steps - 1;
      // loader
      if (vorder && ends && vc >= kVs)
        m.wait(load, bar("V_FULL", vc % kVs), vc / kVs - 1, (uint32_t)(vc / kVs - 1) & 1);
      for (int c = 0; c < chunks; ++c) {
        const int f = kc + c;
        m.wait(load, bar("K_EMPTY", f % kKs), f / kKs - 1, (uint32_t)((f / kKs) & 1) ^ 1);
        m.issue(load, -1, {bar("K_FULL", f % kKs)});
      }
      m.wait(load, bar("V_EMPTY", vc % kVs), vc / kVs - 1, (uint32_t)((vc / kVs) & 1) ^ 1);
      m.issue(load, -1, {bar("V_FULL", vc % kVs)});
      // S
      for (int t = 0; t < 2; ++t) {
        if (j >= it.steps[t]) continue;
        const bool last = t == 1 || j >= it.steps[1];
        if (t == 0 || it.steps[0] <= j)
          for (int c = 0; c < chunks; ++c)
            m.wait(s, bar("K_FULL", (kc + c) % kKs), (kc + c) / kKs, ((kc + c) / kKs) & 1);
        if (j == 0) {
          m.wait(s, bar("Q_FULL", t), s_qs[t], s_qs[t] & 1);
          ++s_qs[t];
        }
        if (issued > 0) m.wait(s, bar("S_EMPTY", 0), issued - 1, (issued - 1) & 1);
        ++issued;
        if (last)
          for (int c = 0; c < chunks; ++c) m.issue(s, 0, {bar("K_EMPTY", (kc + c) % kKs)});
        m.issue(s, 0, {bar("S_FULL", t)});
        if (j == it.steps[t] - 1) m.issue(s, 0, {bar("Q_EMPTY", t)});
      }
      // O
      m.wait(o, bar("V_FULL", vc % kVs), vc / kVs, (vc / kVs) & 1);
      for (int t = 0; t < 2; ++t) {
        if (j >= it.steps[t]) continue;
        m.wait(o, bar("P_READY", t), done[t], done[t] & 1);
        if (j == 0) {
          m.wait(o, bar("O_FREE", t), opened[t] - 1, (uint32_t)(opened[t] & 1) ^ 1);
          ++opened[t];
        }
        m.wait(o, bar("P_READY", 2 + t), done[t], done[t] & 1);
        ++done[t];
        m.issue(o, 1, {bar("PV_DONE", t)});
      }
      m.issue(o, 1, {bar("V_EMPTY", vc % kVs)});
      // softmax
      for (int t = 0; t < 2; ++t) {
        if (j >= it.steps[t]) continue;
        Warp& w = soft[t];
        m.wait(w, bar("S_FULL", t), sdone[t], sdone[t] & 1);
        m.arrive(w, bar("S_EMPTY", 0));
        if (j > 0) m.wait(w, bar("PV_DONE", t), sdone[t] - 1, (uint32_t)(sdone[t] - 1) & 1);
        if (ends) m.wait(w, bar("V_FULL", vc % kVs), vc / kVs, (vc / kVs) & 1);
        m.arrive(w, bar("P_READY", t));
        m.arrive(w, bar("P_READY", 2 + t));
        ++sdone[t];
      }
    }
    for (int t = 0; t < 2; ++t) {
      if (it.steps[t] == 0) continue;
      m.wait(soft[t], bar("PV_DONE", t), sdone[t] - 1, (uint32_t)(sdone[t] - 1) & 1);
      m.arrive(soft[t], bar("O_FREE", t));
    }
  }
  m.warps = {load, s, o, soft[0], soft[1]};
  m.run();
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 6 && !std::strcmp(argv[1], "decode")) {
    std::vector<int> tokens;
    for (int i = 6; i < argc; ++i) tokens.push_back(std::atoi(argv[i]));
    decode(std::atoi(argv[2]), std::atoi(argv[3]), std::atoi(argv[4]), (unsigned)std::atoi(argv[5]), tokens);
  } else if (argc > 4 && !std::strcmp(argv[1], "prefill")) {
    std::vector<Item> items;
    for (int i = 4; i < argc; ++i) {
      Item it;
      int r = 0;
      if (std::sscanf(argv[i], "%d,%d,%d", &it.steps[0], &it.steps[1], &r) != 3) return 2;
      it.ragged = r;
      items.push_back(it);
    }
    prefill(std::atoi(argv[2]), std::atoi(argv[3]), items);
  } else {
    return 2;
  }
  return 0;
}
