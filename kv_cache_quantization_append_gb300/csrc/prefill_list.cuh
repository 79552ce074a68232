// The list of a prefill chunk's work over 8-bit blocks, and how CTAs share it: arithmetic only, host and device.
//
// A row tile is ROWS (query, head) rows of one (layer, sequence, kv-head).  Either the row tiles' costs form one line that is cut
// into equal parts, one per CTA (a row tile that a cut divides is joined by a second launch), or CTAs take row tiles whole, one
// after the other.  Sequences that are not part of the call are in neither.
#pragma once

namespace kvq {
namespace prefill_list {

#define KVQ_HD __host__ __device__ __forceinline__

constexpr int ROWS = 128;     // rows of a row tile = MMA M = lanes of tensor memory
constexpr int NT = 64;        // recorded positions of a tile = a page
constexpr int FULL_NT = 32;   // positions of a raw tile with hi and lo planes
// A row tile's fixed cost in positions, KF of it before its first tile (queries, the start of the products), the rest for raw
// tiles and the output; and the positions that a CTA takes at least.  A prompt of 2048 tokens and 32 heads, cut: 518 us at a cost of
// 32, 345 at 128, 240 at 448, 208 at 1024, 213 at 1536; at 15001 positions it hardly matters.  Three turns of 37 tokens at 1000
// positions: 55 us with shares of 512, 49 of 256, 38 of 128, 33 with raw tiles' cost at their end.
constexpr long long K0 = 1024, KF = 512, MIN_SHARE = 128;

template <typename T>
KVQ_HD T least(T a, T b) { return a < b ? a : b; }
template <typename T>
KVQ_HD T most(T a, T b) { return a < b ? b : a; }

struct Unit {
  int b, x, hl;           // sequence, row tile, (layer, kv-head)
  long long start, cost;  // on the cost line
};

// A row tile: its queries' positions, the recorded positions [0, qend) that any of them reads, the raw ones from rlo.  Raw tiles
// have hi and lo planes of FULL_NT positions, but those of a bf16 cache's own call one plane of raw_nt: first n_full of the former,
// for tokens of earlier calls, whose copies are floats.
struct Tiles {
  int t0, nq, Pmin, Pmax, qend, nqt, rlo, n_full, n;
  Tiles() = default;
  KVQ_HD Tiles(int p0, int T, int qpt, int x, int W, int raw_nt) {
    t0 = x * qpt;
    nq = least(qpt, T - t0);
    Pmin = p0 + t0;
    Pmax = Pmin + nq - 1;
    qend = most(0, Pmax - W + 1);
    nqt = (qend + NT - 1) / NT;
    rlo = most(0, Pmin - W + 1);
    n_full = raw_nt == FULL_NT ? 0 : most(0, p0 - rlo + FULL_NT - 1) / FULL_NT;
    n = nqt + n_full + most(0, Pmax - rlo - n_full * FULL_NT + raw_nt) / raw_nt;
  }
  // the first position of raw tile r
  KVQ_HD int raw_at(int r, int raw_nt) const { return rlo + least(r, n_full) * FULL_NT + most(0, r - n_full) * raw_nt; }
  // tiles before offset `off` of the row tile's stretch of the cost line, `cost` long: what is fixed, recorded tiles of
  // their positions, raw ones of equal shares of the rest
  KVQ_HD int before(long long off, long long cost) const {
    const int o = (int)(off - KF), rest = o - nqt * NT;
    if (o <= 0) return 0;
    if (rest <= 0) return least(n, (o + NT - 1) / NT);
    return least(n, nqt + rest * (n - nqt) / most(1, (int)(cost - KF) - nqt * NT));
  }
};

// Tiles ta .. tb - 1 of a row tile (tb -1: nothing)
struct Part {
  int b, x, hl;
  int ta, tb;
  Tiles tl;
  long long next;  // where on the cost line the CTA goes on
};

// Costs in positions: row tile x of a sequence at p0 counts p0 + (x + 1) qpt + K0, about the positions it visits.  The line
// goes through sequences, row tiles, (layer, kv-head) pairs.
struct List {
  int B, T, qpt, nx, HL, W, raw_nt;
  int n_act;                     // sequences of the call
  const int* p0;                 // per sequence; -1: not part of the call
  const long long* pre;          // cost before each sequence, [B + 1]
  const unsigned short* act;     // which are part of it, in order
  List() = default;
  KVQ_HD List(int B, int T, int g, int HL, int W, int raw_nt, const int* p0, const long long* pre, const unsigned short* act, int n_act)
      : B(B), T(T), qpt(ROWS / g), nx((T + ROWS / g - 1) / (ROWS / g)), HL(HL), W(W), raw_nt(raw_nt), n_act(n_act), p0(p0), pre(pre), act(act) {}
  KVQ_HD long long cost(int b, int x) const { return p0[b] + (long long)(x + 1) * qpt + K0; }
  KVQ_HD long long upto(int b, int x) const { return (x * (p0[b] + K0) + (long long)qpt * x * (x + 1) / 2) * HL; }
  KVQ_HD long long total() const { return pre[B]; }
  // part c of n, [lo, hi): the parts' costs differ by 1 at most
  KVQ_HD void cut(int c, int n, long long& lo, long long& hi) const {
    const long long share = total() / n, rest = total() - share * n;
    lo = share * c + least((long long)c, rest);
    hi = lo + share + (c < rest);
  }
  KVQ_HD Tiles tiles(int b, int x) const { return Tiles(p0[b], T, qpt, x, W, raw_nt); }
  KVQ_HD Unit find(long long y) const {
    Unit u;
    int lo = 0, hi = B - 1;
    while (lo < hi) {  // the last sequence that starts at or before y (those without work start where the next does)
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= y) lo = mid;
      else hi = mid - 1;
    }
    u.b = lo;
    const long long r = y - pre[lo];
    int xl = 0, xh = nx - 1;
    while (xl < xh) {
      const int mid = (xl + xh + 1) >> 1;
      if (upto(lo, mid) <= r) xl = mid;
      else xh = mid - 1;
    }
    u.x = xl;
    u.cost = cost(lo, xl);
    const long long r2 = r - upto(lo, xl);
    u.hl = (int)(r2 / u.cost);
    u.start = y - r2 % u.cost;
    return u;
  }
  // a row tile's tiles from ta on, as far as a part of the line that ends at hi goes; false: there are none
  KVQ_HD bool take(const Unit& u, int ta, long long hi, Part& p) const {
    const Tiles tl = tiles(u.b, u.x);
    if (ta < 0) ta = tl.before(-1 - ta, u.cost);  // (-1 - offset within the row tile)
    const int tb = hi >= u.start + u.cost ? tl.n : tl.before(hi - u.start, u.cost);
    p.b = u.b;
    p.x = u.x;
    p.hl = u.hl;
    p.ta = ta;
    p.tl = tl;
    p.next = u.start + u.cost;
    p.tb = ta < tb ? tb : -1;
    return ta < tb;
  }
  // the first tiles of the line from lo on, up to hi; whether the part begins with them
  KVQ_HD bool first(long long lo, long long hi, Part& p) const {
    const Unit u = find(lo);
    if (take(u, (int)(u.start - lo) - 1, hi, p)) return true;
    follow(p, hi, p);
    return false;
  }
  // the tiles after those of `from` (may be p)
  KVQ_HD void follow(const Part& from, long long hi, Part& p) const {
    int b = from.b, x = from.x, hl = from.hl;
    long long y = from.next;
    p.tb = -1;
    while (y < hi) {
      if (++hl == HL) {
        hl = 0;
        if (++x == nx) {
          x = 0;
          do ++b;
          while (p0[b] < 0);  // (there is one: the line goes on)
        }
      }
      Unit n;
      n.b = b;
      n.x = x;
      n.hl = hl;
      n.start = y;
      n.cost = cost(b, x);
      if (take(n, 0, hi, p)) return;
      y += n.cost;
    }
  }
  // row tiles to be taken whole, those at the chunk's end (the longest of a sequence) first
  KVQ_HD long long units() const { return (long long)nx * n_act * HL; }
  KVQ_HD bool whole(long long i, Part& p) const {
    p.tb = -1;
    if (i >= units()) return false;
    const int per = n_act * HL, j = (int)(i % per);
    Unit n;
    n.x = nx - 1 - (int)(i / per);
    n.b = act[j / HL];
    n.hl = j % HL;
    n.start = 0;
    n.cost = 1;
    return take(n, 0, 1, p);
  }
  // Whether CTAs take row tiles whole instead of equal stretches of the line, whose cuts cost most CTAs a row tile's fixed cost
  // more: when the sum of the longest of each round is below 1.15 of a share with that cost; where they are 16 a CTA or more, when
  // the longest of all (it may be taken last) is not above a share.  (far: the largest position.)
  // Whole against cut: a prompt of 2048 tokens of 32 heads 160 against 219 us, 4096 tokens 411 / 550, 1024 tokens 89 / 102, 1500 of
  // 24 heads 110 / 129; 2048 of 16 heads at position 6000 (256 long row tiles) 322 / 304, not taken.  64 prompts of 256 tokens 585 /
  // 737, one of them at position 20000 1012 / 1057, at 60000 1701 / 1495 and at 100000 2380 / 1766, not taken.
  KVQ_HD bool take_whole(int ctas, int far) const {
    const long long n = units(), each = (long long)n_act * HL, share = total() / ctas;
    if (n >= 16LL * ctas) return far + (long long)nx * qpt + K0 <= share;
    long long rounds = 0;
    for (long long i = 0; i < n; i += ctas) rounds += far + (nx - i / each) * qpt + K0;
    return n > 0 && 20 * rounds <= 23 * (share + K0);
  }
  // how many CTAs have work: parts of the line, or row tiles
  KVQ_HD int parts(int ctas, bool whole_tiles) const {
    if (total() == 0) return 0;
    return (int)most(1LL, least((long long)ctas, whole_tiles ? units() : total() / MIN_SHARE));
  }
};

#undef KVQ_HD

}  // namespace prefill_list
}  // namespace kvq
