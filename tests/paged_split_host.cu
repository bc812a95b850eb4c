// The integer logic of the paged attention kernels on the host: which part of
// which unit each CTA takes, and where a position lies in the cache.
#include <cstring>

#include "paged.cuh"

using namespace mha;

namespace {
PagedProblem problem(const int32_t *starts, const int32_t *lens, const int32_t *table, int B, int T,
                     int H, int Hkv, int hpu, int tb, int causal, int pages, int page_shift,
                     int max_pages, int layout, int which = 1) {
  const PagedSplit splits[3] = {kSplitSimt, kSplitFew, kSplitMany};
  PagedProblem p;
  std::memset(&p, 0, sizeof p);
  p.batch = PagedBatch{starts, lens, table, B, T, pages, 1 << page_shift, page_shift, max_pages,
                       layout};
  p.H = H;
  p.Hkv = Hkv;
  p.group = H / Hkv;
  p.hpu = hpu;
  p.hblocks = (p.group + hpu - 1) / hpu;
  p.tb = tb;
  p.causal = causal;
  p.rows = hpu * tb;
  p.split = splits[which];
  return p;
}
}  // namespace

// What paged_span finds, by a plain search.
static PagedSpan span_of(const PagedProblem &p, int cta, int grid) {
  long long one = 0, units = 0;
  for (int b = 0; b < p.batch.B; ++b) {
    const PagedSeq s = paged_seq(p.batch, b);
    for (int u = 0; u < paged_blocks(p, s); ++u, ++units)
      one += paged_unit_cost(p, s, paged_blocks(p, s), u);
  }
  const int hbs = p.Hkv * p.hblocks;
  PagedSpan sp = paged_stretch(one * hbs, units * hbs, cta, grid, p.split.stretches);
  long long s = 0;
  for (int hb = 0; hb < hbs; ++hb)
    for (int b = 0; b < p.batch.B; ++b) {
      const PagedSeq q = paged_seq(p.batch, b);
      const int blocks = paged_blocks(p, q);
      for (int u = 0; u < blocks; ++u) {
        const long long cost = paged_unit_cost(p, q, blocks, u);
        if (sp.lo >= s && sp.lo < s + cost) {
          sp.at = s;
          sp.hb = hb;
          sp.b = b;
          sp.u = u;
          return sp;
        }
        s += cost;
      }
    }
  return sp;
}

// Rows of (cta, b, i0, i1, h0, heads, kv, nt, t0, t1, slot or -1); returns their number.
extern "C" int parts(const int32_t *starts, const int32_t *lens, int B, int T, int H, int Hkv,
                     int hpu, int tb, int causal, int page_shift, int max_pages, int grid,
                     int which, int32_t *out, int most) {
  const PagedProblem p =
      problem(starts, lens, nullptr, B, T, H, Hkv, hpu, tb, causal, 0, page_shift, max_pages, 0, which);
  int n = 0;
  for (int c = 0; c < grid; ++c) {
    PagedWalk w;
    w.begin(p, span_of(p, c, grid));
    PagedPart part;
    while (w.next(p, part)) {
      if (n == most) return -1;
      const int32_t row[11] = {c,       part.b,  part.i0, part.i1,
                               part.h0, part.heads, part.kv, part.nt,
                               part.t0, part.t1, paged_split(part) ? paged_slot(part) : -1};
      std::memcpy(out + 11 * n++, row, sizeof row);
    }
  }
  return n;
}

extern "C" long long cell(const int32_t *table, int pages, int page_shift, int max_pages,
                          int layout, int b, int pos, int head, int heads) {
  const PagedProblem p =
      problem(nullptr, nullptr, table, 0, 0, 1, 1, 1, 1, 1, pages, page_shift, max_pages, layout);
  return paged_cell(p.batch, b, pos, head, heads);
}

extern "C" void seq(const int32_t *starts, const int32_t *lens, int T, int page_shift,
                    int max_pages, int b, int32_t *out) {
  const PagedProblem p =
      problem(starts, lens, nullptr, 1, T, 1, 1, 1, 1, 1, 0, page_shift, max_pages, 0);
  const PagedSeq s = paged_seq(p.batch, b);
  out[0] = s.q0;
  out[1] = s.n;
  out[2] = s.len;
  out[3] = s.base;
}

// Units of a sequence: their lengths' prefix sums by the closed form, and the unit
// at each boundary; returns 0 when they agree with sums and a plain search.
extern "C" int unit_sums(const int32_t *starts, const int32_t *lens, int T, int tb, int causal,
                         int page_shift, int max_pages, int which) {
  const PagedProblem p =
      problem(starts, lens, nullptr, 1, T, 1, 1, 1, tb, causal, 0, page_shift, max_pages, 0, which);
  const PagedSeq s = paged_seq(p.batch, 0);
  const int blocks = paged_blocks(p, s);
  long long sum = 0;
  for (int u = 0; u < blocks; ++u) {
    const long long cost = paged_unit_cost(p, s, blocks, u);
    if (paged_cost_before(p, s, blocks, u) != sum) return 1 + u;
    if (cost < p.split.unit_cost) return -1;
    long long first = -1, last = -1;
    if (paged_unit_at(p, s, blocks, sum, first) != u ||
        paged_unit_at(p, s, blocks, sum + cost - 1, last) != u || first != sum || last != sum)
      return -2 - u;
    sum += cost;
  }
  return paged_cost_before(p, s, blocks, blocks) == sum ? 0 : -100;
}

extern "C" long long slot_floats(int rows, int d) {
  return static_cast<long long>(paged_slot_floats(rows, d));
}
