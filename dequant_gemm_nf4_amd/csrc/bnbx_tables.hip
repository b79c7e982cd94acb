// The one-time host tables of the two 4-bit quant types (levels, encode
// tables), shared by the C entry points of both libraries.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "bnbx_internal.hpp"

namespace bnbx {
namespace {

// Standard normal CDF and density in binary64 (C library erfc / exp).
double normal_cdf(double x) { return 0.5 * erfc(-x * 0.70710678118654752440); }
double normal_pdf(double x) { return exp(-0.5 * x * x) * 0.39894228040143267794; }

// Upper-half standard normal quantile by Newton's method on the CDF from 0.
// The CDF is concave on [0, inf), so from the left every Newton step stays at
// or below the root and the iterates rise monotonically to it; stop when a
// step no longer moves x up.
double normal_quantile_upper(double p) {
  double x = 0.0;
  for (int it = 0; it < 200; ++it) {
    const double nx = x - (normal_cdf(x) - p) / normal_pdf(x);
    if (!(nx > x)) break;
    x = nx;
  }
  return x;
}

struct Tables {
  float levels[16];   // level of each code
  EncodeTable enc;
  LevelTable lv;
};

// NF4 codebook (mlqm.cn bitsandbytes article, sec. 3.2: 16 levels laid out
// by the normal density, dense near 0, with exact 0 and ends at +-1): 8
// positive quantiles of probabilities evenly spaced from the offset toward
// 1/2, 7 mirrored negative ones over the same span, and 0, all divided by the
// outermost quantile.  The offset averages the 1/30 and 1/32 tail masses.
// Codes are in ascending level order.
void nf4_levels(float* levels) {
  const double off = 1.0 - 0.5 * (1.0 / 30.0 + 1.0 / 32.0);
  const double top = normal_quantile_upper(off);
  double v[16];
  int k = 0;
  for (int i = 0; i < 7; ++i) v[k++] = -normal_quantile_upper(off + i * (0.5 - off) / 7.0);
  v[k++] = 0.0;
  for (int i = 0; i < 8; ++i) v[k++] = normal_quantile_upper(off + i * (0.5 - off) / 8.0);
  std::sort(v, v + 16);
  for (int i = 0; i < 16; ++i) levels[i] = (float)(v[i] / top);   // ends: +-top/top = +-1
}

// FP4 (mlqm.cn article, sec. 4: the plain 4-bit float quant type; the pages
// give no layout, E2M1 is taken): code bit 3 is the sign, bits 2-1 the
// exponent e, bit 0 the mantissa m; magnitude m/2 for e = 0, else
// 2^(e-1) (1 + m/2), i.e. 0, 0.5, 1, 1.5, 2, 3, 4, 6 for codes 0-7, divided by
// 6 so the block absmax maps to +-1.
void fp4_levels(float* levels) {
  for (int c = 0; c < 16; ++c) {
    const int e = (c >> 1) & 3, m = c & 1;
    const double mag = e == 0 ? 0.5 * m : ldexp(1.0 + 0.5 * m, e - 1);
    levels[c] = (float)((c & 8 ? -mag : mag) / 6.0);
  }
}

// Encode tables of a codebook.  `order` lists the codes of the distinct
// levels by ascending value (count of them in `nl`; FP4 leaves out -0, code
// 8, which the encoder never emits).  Thresholds: the smallest float strictly
// above each midpoint of neighbouring levels, so the nearest level wins and
// an exact tie takes the lower one.  Returns false if the codebook does not
// fit the bucket scheme (never for the two fixed codebooks; checked anyway,
// and reported by every call as BNBX_E_INTERNAL).
bool build_encode(const float* levels, const int* order, int nl, bool in_order, EncodeTable& enc) {
  float thr[15];
  for (int i = 0; i + 1 < nl; ++i) {
    const double mid = ((double)levels[order[i]] + (double)levels[order[i + 1]]) * 0.5;
    float th = (float)mid;
    if ((double)th <= mid) th = nextafterf(th, INFINITY);
    thr[i] = th;
  }
  // Encode buckets: bucket b holds x with round-half-even(16x + 16) == b,
  // i.e. x in [(b - 1/2)/16 - 1, (b + 1/2)/16 - 1].  Each bucket must hold at
  // most one threshold and no threshold may sit near a bucket edge (the
  // rounding of 16x + 16 moves an edge by far less than the margin checked).
  for (int b = 0; b < kBuckets; ++b) {
    const double lo = (b - 0.5) / 16.0 - 1.0, hi = (b + 0.5) / 16.0 - 1.0;
    uint32_t below = 0;
    float inside = INFINITY;
    int count = 0;
    for (int i = 0; i + 1 < nl; ++i) {
      const double th = thr[i];
      if (fabs(th - lo) < 1e-4 || fabs(th - hi) < 1e-4) return false;   // too near an edge
      if (th < lo) ++below;
      else if (th < hi) { inside = thr[i]; ++count; }
    }
    if (count > 1) return false;   // two thresholds in one bucket
    enc.thr[b] = inside;
    if (in_order) {
      enc.base[b] = below;
    } else {
      const uint32_t c0 = (uint32_t)order[below];
      const uint32_t c1 = count ? (uint32_t)order[below + 1] : c0;
      enc.base[b] = c0 | (c1 << 4);
    }
  }
  return true;
}

bool build_tables(int quant_type, Tables& t) {
  int order[16];
  int nl = 0;
  if (quant_type == kQuantNF4) {
    nf4_levels(t.levels);
    for (int c = 0; c < 16; ++c) order[nl++] = c;
  } else {
    fp4_levels(t.levels);
    for (int c = 0; c < 16; ++c)
      if (c != 8) order[nl++] = c;
    std::sort(order, order + nl, [&](int a, int b) { return t.levels[a] < t.levels[b]; });
  }
  for (int i = 0; i < 16; ++i) t.lv.level[i] = t.levels[i];
  return build_encode(t.levels, order, nl, quant_type == kQuantNF4, t.enc);
}

struct AllTables {
  Tables t[2];
  bool ok;
};

const AllTables& all_tables() {
  static AllTables a;
  static std::once_flag once;
  std::call_once(once, [] {
    const bool nf4 = build_tables(kQuantNF4, a.t[0]);
    const bool fp4 = build_tables(kQuantFP4, a.t[1]);
    a.ok = nf4 && fp4;
  });
  return a;
}

const Tables& tables(int quant_type) { return all_tables().t[quant_type == kQuantFP4 ? 1 : 0]; }

}  // namespace

bool tables_ok() { return all_tables().ok; }
const float* levels_f32(int quant_type) { return tables(quant_type).levels; }
const EncodeTable& encode_table(int quant_type) { return tables(quant_type).enc; }
const LevelTable& level_table(int quant_type) { return tables(quant_type).lv; }

}  // namespace bnbx
