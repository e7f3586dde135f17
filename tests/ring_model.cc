// settle_ring() against a model of mbarriers: groups of one or two CTAs load slices into a ring, an MMA issuer uses them, every
// role stops at a random point (its wait ran out), and loads land whenever they like. Prints "ok <runs>" or what went wrong.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "fp4_ring.h"

struct Barrier {  // one arrival a phase
  int pending = 1, phase = 0;
  long tx = 0;
  void check() {
    if (pending == 0 && tx == 0) {
      ++phase;
      pending = 1;
    }
  }
  void expect(long n) { tx += n; }
  void land(long n) {
    tx -= n;
    check();
  }
  bool arrive() {
    if (pending != 1) return false;
    pending = 0;
    check();
    return true;
  }
  bool done(unsigned parity) const { return (unsigned)(phase & 1) != parity; }
};

struct Load {
  unsigned s;
};

static std::mt19937 rng(7);
static unsigned pick(unsigned n) { return rng() % n; }

struct Group {
  unsigned cg, stages;
  std::vector<Barrier> full;
  std::vector<unsigned> used;      // how often the stage's contents have been used: what `empty` tells every CTA
  std::vector<Load> flying;
  unsigned issued[2] = {0, 0}, consumed = 0;
  bool wrong = false;

  Group(unsigned cg_, unsigned stages_) : cg(cg_), stages(stages_), full(stages_), used(stages_, 0) {}
  bool can_issue(unsigned r) const { return used[issued[r] % stages] >= issued[r] / stages; }
  void issue(unsigned r) {
    const unsigned s = issued[r]++ % stages;
    if (r == 0) {
      full[s].expect(cg);
      wrong |= !full[s].arrive();
    }
    flying.push_back({s});
  }
  void land() {
    if (flying.empty()) return;
    const unsigned i = pick((unsigned)flying.size());
    const unsigned s = flying[i].s;
    flying.erase(flying.begin() + i);
    full[s].land(1);
  }
  void consume() {
    const unsigned s = consumed % stages;
    if (!full[s].done((consumed / stages) & 1u)) return;
    ++used[s];
    ++consumed;
  }
  // what settle_ring() asks of the leader
  void forgo(unsigned s) { full[s].land(1); }
  void announce(unsigned s) {
    full[s].expect(1);
    wrong |= !full[s].arrive();
  }
  bool wait(unsigned s, unsigned parity) {
    while (!full[s].done(parity) && !flying.empty()) land();
    return full[s].done(parity);
  }
};

int main(int argc, char** argv) {
  const bool settle = argc < 2 || atoi(argv[1]) != 0;
  const int runs = 20000;
  for (int run = 0; run < runs; ++run) {
    Group g(1 + pick(2), 2 + pick(7));
    bool alive[3] = {true, g.cg == 2, true};  // the producers, the MMA issuer
    const unsigned slices = 1 + pick(40);
    for (int step = 0; step < 400; ++step) {
      const unsigned what = pick(40);
      if (what < 3 && pick(8) == 0) alive[what] = false;
      if (what >= 3 && what < 20) {
        const unsigned r = pick(g.cg);
        if (alive[r] && g.issued[r] < slices && g.can_issue(r)) g.issue(r);
      } else if (what < 30) {
        if (alive[2]) g.consume();
      } else {
        g.land();
      }
    }
    const bool ok = !settle || gns::settle_ring(g, g.issued[0], g.cg == 2 ? g.issued[1] : g.issued[0], g.stages);
    bool clean = true;
    for (const Barrier& b : g.full) clean &= b.pending == 1 && b.tx == 0;
    if (!ok || g.wrong || !g.flying.empty() || !clean) {
      printf("run %d: cg %u stages %u issued %u %u consumed %u: waits %s, %zu loads in flight, barriers %s%s\n", run, g.cg, g.stages,
             g.issued[0], g.issued[1], g.consumed, ok ? "end" : "run out", g.flying.size(), clean ? "clean" : "half done",
             g.wrong ? ", an arrival too many" : "");
      return 1;
    }
  }
  printf("ok %d\n", runs);
  return 0;
}
