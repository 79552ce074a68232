// Test helper: the arithmetic by which CTAs share a prefill chunk over 8-bit blocks, walked through on the host.
#include <cuda_runtime.h>

#include <vector>

#include "../../kv_cache_quantization_append_gb300/csrc/prefill_list.cuh"

using namespace kvq::prefill_list;

// Every stretch that any CTA works on, five ints each: (layer, kv-head), sequence, row tile, first tile, tile after the last;
// then (tiles of the row tile, CTA, slot of its partial result or -1).  Returns how many, or -1 where `room` is too little.
// info: whether row tiles are taken whole, CTAs with work.
extern "C" int walk(const int* pos, int B, int T, int g, int HL, int W, int raw_nt, int max_seq_len, int ctas, int* out, int room,
                    int* info) {
  std::vector<int> p0(B);
  std::vector<long long> pre(B + 1);
  std::vector<unsigned short> act;
  List l(B, T, g, HL, W, raw_nt, p0.data(), pre.data(), nullptr, 0);
  int far = -1;
  pre[0] = 0;
  for (int b = 0; b < B; ++b) {
    p0[b] = pos[b] >= 0 && (long long)pos[b] + T <= max_seq_len ? pos[b] : -1;
    pre[b + 1] = pre[b];
    far = most(far, p0[b]);
    if (p0[b] < 0) continue;
    pre[b + 1] += l.upto(b, l.nx);
    act.push_back((unsigned short)b);
  }
  l.act = act.data();
  l.n_act = (int)act.size();
  const bool whole = l.take_whole(ctas, far);
  const int parts = l.parts(ctas, whole);
  info[0] = whole;
  info[1] = parts;
  int n = 0;
  auto put = [&](const Part& p, int cta, int slot) {
    if (n < room) {
      int* o = out + 8 * n;
      o[0] = p.hl;
      o[1] = p.b;
      o[2] = p.x;
      o[3] = p.ta;
      o[4] = p.tb;
      o[5] = p.tl.n;
      o[6] = cta;
      o[7] = p.ta == 0 && p.tb == p.tl.n ? -1 : slot;
    }
    ++n;
  };
  int taken = 0;
  for (int c = 0; c < parts; ++c) {
    Part p;
    if (whole) {
      if (l.whole(c, p)) put(p, c, 0);
      continue;
    }
    long long lo, hi;
    l.cut(c, parts, lo, hi);
    int slot = l.first(lo, hi, p) ? 0 : 1;
    while (p.tb >= 0) {
      put(p, c, slot);
      l.follow(p, hi, p);
      slot = 1;
    }
  }
  // the rest, to whichever CTA is free
  if (whole)
    for (Part p; l.whole(ctas + taken, p); ++taken) put(p, taken % ctas, 0);
  return n <= room ? n : -1;
}
