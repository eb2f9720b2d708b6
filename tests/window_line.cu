// The division of windowed attention's work (pa_window_split.cuh) on the host, for random batches: every unit of
// every row tile is some worker's exactly once, in order, its chunks are those that a row of the tile attends, and
// partial results, their slots and notes fit together. argv: seed, batches. Prints the batches, row tiles and
// divided ones looked at; what is wrong goes to stderr with exit code 1.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "pa_window_split.cuh"

using namespace pa;

static std::mt19937_64 rng;
static long batches = 0, seen_tiles = 0, divided = 0;
static int64_t pick(int64_t lo, int64_t hi) { return lo + int64_t(rng() % uint64_t(hi - lo + 1)); }

static void check(bool ok, const char* what, long a = 0, long b = 0) {
  if (ok) return;
  fprintf(stderr, "batch %ld: %s (%ld, %ld)\n", batches, what, a, b);
  exit(1);
}

struct Piece {
  int worker, s0, s1, slot, parts;
};

template <int UNIT, int CHUNK, int NR, int LEAD>
static void run(bool huge) {
  using Walk = WindowWalk<UNIT, CHUNK, NR, LEAD>;
  using Line = typename Walk::Line;
  ++batches;
  TreeParams P{};
  P.batch = int(pick(0, 3) ? pick(1, 40) : 1);
  P.kv_heads = int(pick(1, 4));
  P.group = int(pick(0, 5) ? pick(1, 12) : pick(1, 3 * NR));
  P.num_heads = P.kv_heads * P.group;
  P.max_q = int(pick(0, 2) ? pick(1, 40) : pick(1, 700));
  P.max_keys = huge ? 2147483647 - 4095 : int(pick(1, 4000));
  P.window = int(pick(0, 3) ? pick(1, huge ? 2147483647 : 600) : 2147483647);
  P.sinks = int(pick(0, 1) ? 0 : pick(0, 5) ? pick(0, 300) : 2147483647);
  std::vector<int> q(P.batch), L(P.batch);
  const bool lengths = pick(0, 3) != 0;
  int64_t tokens = 0;
  for (int b = 0; b < P.batch; ++b) {
    q[b] = !lengths ? 1 : pick(0, 5) ? int(pick(1, P.max_q)) : 0;
    L[b] = int(pick(0, 9) ? pick(std::min(q[b], P.max_keys), P.max_keys) : std::min(q[b], P.max_keys));
    if (!pick(0, 15)) L[b] = q[b] - 1;             // broken, or padding
    if (lengths && !pick(0, 15)) q[b] = -2;
    tokens += std::max(q[b], 0);
  }
  P.tokens = tokens + pick(0, 3);
  if (P.tokens < P.max_q) P.tokens = P.max_q;      // (a sequence of more than all tokens is broken)
  P.context_lens = L.data();
  P.q_seqlens = lengths ? q.data() : nullptr;
  TreeSplit S{};
  S.workers = int(pick(0, 1) ? pick(1, 40) : pick(1, 1300));
  S.min_units = (LEAD + 1) * UNIT;
  S.tile_tokens = std::max(NR / P.group, 1);
  S.tile_parts = (P.group - 1) / NR + 1;
  const Line line(S);

  int64_t total = 0;
  for (int b = 0; b < P.batch; ++b) total += line.total(P, line.load(P, b));

  // the row tile that comes next, in the order of the line
  int b = 0, head = 0, tile = 0;
  int64_t q_start = 0;
  const auto good = [&] {
    const int n = lengths ? q[b] : 1;
    return n > 0 && n <= P.max_q && n <= P.tokens && L[b] >= n && L[b] <= P.max_keys;
  };
  const auto skip = [&] {  // sequences without tiles
    while (b < P.batch && !good()) {
      q_start = std::min<int64_t>(q_start + std::max(lengths ? q[b] : 1, 0), P.tokens);
      ++b;
    }
  };
  skip();
  std::vector<Piece> pieces;  // of it so far

  for (int w = 0; w < S.workers; ++w) {
    Walk walk{};
    walk.worker = w;
    walk.total = total;
    if (!walk.share(S)) continue;
    check(walk.u1 - walk.u0 >= (total >= S.min_units ? S.min_units : total), "a small piece", w);
    bool found = false;
    int64_t before = 0;
    for (int k = 0; k < P.batch && walk.u0 < walk.u1; ++k) {
      const auto s = line.load(P, k);
      const int64_t places = line.total(P, s);
      if (walk.u0 - before < places) {
        walk.seq = s;
        walk.b = k;
        walk.enter(P, line, before);
        found = true;
        break;
      }
      before += places;
      walk.q_start = tree_tokens(P, walk.q_start, s.q);
    }
    check(found || walk.u0 >= walk.u1, "no sequence", w);
    if (!found) continue;
    int used = 0;  // slots of this worker
    WindowTile t;
    bool noted = false;
    while (walk.next(P, S, t)) {
      check(b < P.batch, "more row tiles than there are", w);
      const int n = lengths ? q[b] : 1, pre = L[b] - n;
      const int i0 = tile * S.tile_tokens, i1 = std::min(i0 + S.tile_tokens, n) - 1;
      const int64_t p0 = int64_t(pre) + i0, p1 = int64_t(pre) + i1;
      check(t.b == b && t.kvh == head / S.tile_parts && t.token0 == i0, "another row tile", t.b, t.token0);
      check(t.r0 == i0 * P.group + head % S.tile_parts * NR && t.q == i1 + 1 && t.L == p1 + 1 && t.q_start == q_start,
            "another tile's rows", t.r0, t.q_start);
      const int64_t lo = std::max<int64_t>(p0 - P.window + 1, 0), lo1 = std::max<int64_t>(p1 - P.window + 1, 0);
      check(t.lo == lo && t.lo1 == lo1 && t.first() == p0, "another window", t.lo, t.lo1);
      // the chunks that a row attends: those of the sinks before the window, and of the window
      const int64_t near = lo / CHUNK, last = p1 / CHUNK;
      const int64_t far = std::min<int64_t>((int64_t(P.sinks) + CHUNK - 1) / CHUNK, near);
      const int64_t chunks = far + last - near + 1, units = (chunks + UNIT / CHUNK - 1) / (UNIT / CHUNK);
      check(t.s0 >= 0 && t.s0 < t.s1 && t.s1 <= units, "units", t.s0, t.s1);
      if (!huge) {
        std::vector<int64_t> want;
        for (int64_t c = 0; c <= last; ++c) {
          bool any = false;
          for (int64_t key = c * CHUNK; key < (c + 1) * CHUNK && !any; ++key)
            any = key <= p1 && (key >= lo || key < P.sinks);
          if (any) want.push_back(c);
        }
        check(int64_t(want.size()) == chunks, "number of chunks", long(want.size()), long(chunks));
        for (int64_t c = 0; c < chunks; ++c) check(t.chunk(int(c)) == want[c], "a chunk", long(c), t.chunk(int(c)));
      } else {
        check(t.chunk(0) == (far ? 0 : near) && t.chunk(int(chunks) - 1) == last, "chunks", t.chunk(0));
      }
      check(t.s0 == (pieces.empty() ? 0 : pieces.back().s1), "units left out or done twice", t.s0);
      check(t.slot == -1 || t.slot / 2 == w, "another worker's slot", t.slot, w);
      if (t.slot >= 0) {
        check(!(used >> (t.slot & 1) & 1), "a slot twice", t.slot);
        used |= 1 << (t.slot & 1);
      }
      check(!(t.parts && noted), "two notes", w);
      noted |= t.parts != 0;
      pieces.push_back({w, t.s0, t.s1, t.slot, t.parts});
      if (t.s1 < units) continue;
      ++seen_tiles;
      if (pieces.size() == 1) {
        check(t.slot == -1 && t.parts == 0, "a whole tile with a slot", t.slot, t.parts);
      } else {
        ++divided;
        check(pieces[0].parts == int(pieces.size()), "parts noted", pieces[0].parts, long(pieces.size()));
        check(pieces[0].slot >= 0, "a part without a slot");
        for (size_t k = 1; k < pieces.size(); ++k)
          check(pieces[k].worker == pieces[0].worker + int(k) && pieces[k].slot == 2 * pieces[k].worker &&
                    pieces[k].parts == 0,
                "where the join looks for a part", pieces[k].worker, pieces[k].slot);
      }
      pieces.clear();
      if (++tile * int64_t(S.tile_tokens) >= n) {
        tile = 0;
        if (++head == P.kv_heads * S.tile_parts) {
          head = 0;
          q_start = std::min<int64_t>(q_start + n, P.tokens);
          ++b;
          skip();
        }
      }
    }
  }
  check(b == P.batch && pieces.empty(), "row tiles left out", b, P.batch);
}

int main(int argc, char** argv) {
  rng.seed(argc > 1 ? strtoull(argv[1], nullptr, 10) : 0);
  const int n = argc > 2 ? atoi(argv[2]) : 100;
  // as the kernels divide: the units, chunks, rows and leads of the tcgen05 and of the warp-level ones
  for (int k = 0; k < n; ++k) {
    const bool huge = k % 8 == 7;
    run<128, 64, 128, 3>(huge);
    run<128, 64, 256, 3>(huge);
    run<128, 64, 256, 5>(huge);
    run<32, 32, 8, 3>(huge);
    run<32, 32, 16, 4>(huge);
    run<16, 16, 8, 3>(huge);
    run<16, 16, 16, 4>(huge);
  }
  printf("%ld batches, %ld row tiles, %ld divided\n", batches, seen_tiles, divided);
  return 0;
}
