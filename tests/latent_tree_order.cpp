// Host program for tests/test_latent_tree_order.py: the waits and arrivals of the tree decode kernel's warps
// (csrc/spa_latent_tree.cu), walked through every interleaving by the model of latent_order.cpp.  The pair of
// CTAs is walked as one.
//
//   latent_tree_order BOX QTMA EARLY GROW KF KS VF VS SOFT TILES...   boxes or cp.async; q by tensor maps or by all loading
//       warps; maxima a tile ahead of the weights: as the kernel has them (1), always (2); bit k of GROW: a maximum
//       moves at tile k; fills of a tile and slots of K, and of V; softmax warps; tiles of each unit
// prints "ok STATES" or "WHAT AT ..."
#define main latent_order_main
#include "latent_order.cpp"
#undef main

int main(int argc, char** argv) {
  if (argc < 11) return 1;
  const bool box = std::atoi(argv[1]), qtma = std::atoi(argv[2]);
  const int early = std::atoi(argv[3]), grow = std::atoi(argv[4]), kf = std::atoi(argv[5]), ks = std::atoi(argv[6]),
            vf = std::atoi(argv[7]), vs = std::atoi(argv[8]), kSoft = std::atoi(argv[9]);
  struct Tile {
    bool first, last;
    int unit;
  };
  std::vector<Tile> tiles;
  for (int a = 10; a < argc; ++a)
    for (int i = 0, n = std::atoi(argv[a]); i < n; ++i) tiles.push_back({i == 0, i == n - 1, a - 10});
  const int n_tiles = (int)tiles.size(), kInfos = 4, kS = 4;
  Model m;
  m.queues = 2;                              // commits of the MMAs of S and of O
  const int loaders = box ? 2 : 1;
  const auto info_full = [&](int k) { return m.bar("INFO_FULL", k % kInfos); };
  const auto info_empty = [&](int k) { return m.bar("INFO_EMPTY", k % kInfos, kSoft + loaders + 3); };
  const auto max_bar = [&](int k) { return m.bar("MAX", k & 1, kSoft); };
  const auto p_ready = [&](int k) { return m.bar("P_READY", k & 1, kSoft); };
  const auto pv_done = [&](int k) { return m.bar("PV_DONE", k & 1); };
  const auto s_empty = [&](int k) { return m.bar("S_EMPTY", k % kS, kSoft); };
  const int q_full = m.bar("Q_FULL", 0, box && !qtma ? 2 : 1), q_empty = m.bar("Q_EMPTY", 0), q_local = m.bar("Q_LOCAL", 0);
  const int o_free = m.bar("O_FREE", 0, kSoft), l_full = m.bar("L_FULL", 0, kSoft), l_empty = m.bar("L_EMPTY", 0, kSoft);
  const auto wait_info = [&](Warp& w, int k) { m.wait(w, info_full(k), k / kInfos, (uint32_t)(k / kInfos)); };
  // use i of a ring of n slots: free again, as the kernel asks for it (a fresh barrier lets the first n through)
  const auto wait_free = [&](Warp& w, const char* kind, int i, int n) {
    if (i >= n) m.wait(w, m.bar(kind, i % n), i / n - 1, (uint32_t)((i / n) & 1) ^ 1u);
  };
  const auto wait_use = [&](Warp& w, const char* kind, int i, int n) {
    m.wait(w, m.bar(kind, i % n), i / n, (uint32_t)(i / n));
  };

  Warp sched{"schedule", {}}, kload{"K loader", {}}, vload{"V loader", {}}, clean{"cleaner", {}}, smma{"S", {}}, omma{"O", {}};
  const auto k_part = [&](Warp& w, int k) {
    for (int f = 0; f < kf; ++f) {
      const int i = k * kf + f;
      wait_free(w, "K_EMPTY", i, ks);
      m.issue(w, -1, {m.bar(box ? "K_READY" : "K_FULL", i % ks)});
    }
  };
  const auto v_part = [&](Warp& w, int k) {
    for (int f = 0; f < vf; ++f) {
      const int i = k * vf + f;
      wait_free(w, "V_EMPTY", i, vs);
      m.issue(w, -1, {m.bar("V_FULL", i % vs)});
    }
  };
  const auto q_part = [&](Warp& w, int k, bool copy) {
    const int u = tiles[k].unit;
    if (u > 0) m.wait(w, q_empty, u - 1, (uint32_t)(u & 1) ^ 1u);
    if (copy) {
      m.issue(w, -1, {q_local});
      m.wait(w, q_local, u, (uint32_t)u);
    }
    m.arrive(w, q_full);
  };
  for (int k = 0; k < n_tiles; ++k) {
    const Tile& t = tiles[k];
    if (k >= kInfos) m.wait(sched, info_empty(k), k / kInfos - 1, (uint32_t)((k / kInfos) & 1) ^ 1u);
    m.arrive(sched, info_full(k));
    // loaders
    if (box) {
      wait_info(kload, k);
      k_part(kload, k);
      if (t.first && !qtma) q_part(kload, k, false);
      m.arrive(kload, info_empty(k));
      wait_info(vload, k);
      if (t.first) q_part(vload, k, qtma);
      v_part(vload, k);
      m.arrive(vload, info_empty(k));
    } else {
      wait_info(vload, k);
      k_part(vload, k);
      if (t.first) q_part(vload, k, qtma);
      v_part(vload, k);
      m.arrive(vload, info_empty(k));
    }
    // cleaner
    wait_info(clean, k);
    if (!box)
      for (int f = 0; f < kf; ++f) {
        wait_use(clean, "K_FULL", k * kf + f, ks);
        m.arrive(clean, m.bar("K_READY", (k * kf + f) % ks));
      }
    for (int f = 0; f < vf; ++f) {
      wait_use(clean, "V_FULL", k * vf + f, vs);
      m.arrive(clean, m.bar("V_READY", (k * vf + f) % vs));
    }
    m.arrive(clean, info_empty(k));
    // MMAs
    wait_info(smma, k);
    m.arrive(smma, info_empty(k));
    if (t.first) m.wait(smma, q_full, t.unit, (uint32_t)t.unit);
    if (k >= kS) m.wait(smma, s_empty(k), k / kS - 1, (uint32_t)((k / kS) & 1) ^ 1u);
    for (int f = 0; f < kf; ++f) {
      const int i = k * kf + f;
      wait_use(smma, "K_READY", i, ks);
      std::vector<int> to{m.bar("K_EMPTY", i % ks)};
      if (f == kf - 1) {
        to.push_back(m.bar("S_FULL", k % kS));
        if (t.last) to.push_back(q_empty);
      }
      m.issue(smma, 0, to);
    }
    wait_info(omma, k);
    m.arrive(omma, info_empty(k));
    m.wait(omma, p_ready(k), k >> 1, (uint32_t)(k >> 1));
    if (t.first && t.unit > 0) m.wait(omma, o_free, t.unit - 1, (uint32_t)(t.unit - 1));
    for (int f = 0; f < vf; ++f) {
      const int i = k * vf + f;
      wait_use(omma, "V_READY", i, vs);
      std::vector<int> to{m.bar("V_EMPTY", i % vs)};
      if (f == vf - 1) to.push_back(pv_done(k));
      m.issue(omma, 1, to);
    }
  }
  m.warps = {sched, vload, clean, smma, omma};
  if (box) m.warps.push_back(kload);
  for (int s = 0; s < kSoft; ++s) {
    Warp w{"softmax " + std::to_string(s), {}};
    int k = 0, n = 0;
    while (k < n_tiles) {
      if (n < n_tiles) {
        wait_info(w, n);
        if (n == k || early == 2 || (box && !tiles[n].first)) {
          m.wait(w, m.bar("S_FULL", n % kS), n / kS, (uint32_t)(n / kS));
          m.arrive(w, max_bar(n));
          if (++n == k + 1) continue;
        }
      }
      m.wait(w, max_bar(k), k >> 1, (uint32_t)(k >> 1));
      m.arrive(w, s_empty(k));
      if (k > 1) m.wait(w, pv_done(k), (k >> 1) - 1, (uint32_t)((k >> 1) & 1) ^ 1u);
      if ((grow >> k & 1) && !tiles[k].first) m.wait(w, pv_done(k - 1), (k - 1) >> 1, (uint32_t)((k - 1) >> 1));
      m.arrive(w, p_ready(k));
      m.arrive(w, info_empty(k));
      if (tiles[k].last) {
        const int u = tiles[k].unit;
        m.wait(w, pv_done(k), k >> 1, (uint32_t)(k >> 1));
        m.arrive(w, l_full);
        m.wait(w, l_full, u, (uint32_t)u);
        m.arrive(w, l_empty);
        m.arrive(w, o_free);
        m.wait(w, l_empty, u, (uint32_t)u);
      }
      ++k;
    }
    m.warps.push_back(w);
  }
  m.run();
  return 0;
}
