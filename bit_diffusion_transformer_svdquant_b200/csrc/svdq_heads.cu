// C ABI of the rotary positions (svdq_rotary) and the quantized key/value cache (svdq_kv_*): argument checks and
// launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "svdq.h"
#include "svdq_heads.cuh"
#include "svdq_host.h"

using namespace svdq::host;

namespace {

constexpr int kMaxHeads = 4096;
constexpr long long kMaxStride = 1ll << 38;

bool at16(const void* p) { return aligned16(p); }

// Bytes of a head in a cache.
int code_bytes(int D, int format) { return format == SVDQ_KV_MXFP4 ? D / 2 : D; }
int scale_bytes(int D, int format) { return format == SVDQ_KV_MXFP4 ? (D + 31) / 32 : 1; }

// The bytes of a strided tensor: runs of `width` bytes at base + sum of i_d stride_d, 0 <= i_d < n_d (strides in bytes,
// not negative).
struct Grid {
  struct Dim {
    long long stride, n;
  };
  uintptr_t base, end;  // [base, end) holds all of them (end at most the largest address)
  long long width;
  int dims;             // those of more than one index
  Dim dim[3];
  Grid() {}
  Grid(const void* p, long long bytes) : base(reinterpret_cast<uintptr_t>(p)), end(base + bytes), width(bytes), dims(0) {}
  Grid(const void* p, long long esize, long long run, Dim a, Dim b = {0, 1}, Dim c = {0, 1}) : Grid(p, esize * run) {
    unsigned __int128 last = end;
    for (const Dim& d : {a, b, c})
      if (d.n > 1) {
        dim[dims++] = {d.stride * esize, d.n};
        last += static_cast<unsigned __int128>(d.n - 1) * (d.stride * esize);
      }
    end = last > UINTPTR_MAX ? UINTPTR_MAX : static_cast<uintptr_t>(last);
  }
  // Each dimension steps over all that those of smaller strides span: no two places share a byte.
  bool nested() const {
    Dim d[3];
    std::copy(dim, dim + dims, d);
    std::sort(d, d + dims, [](const Dim& l, const Dim& r) { return l.stride < r.stride; });
    __int128 extent = width;
    for (int i = 0; i < dims; ++i) {
      if (d[i].stride < extent) return false;
      extent += static_cast<__int128>(d[i].n - 1) * d[i].stride;
    }
    return true;
  }
};

// Whether two grids share a byte: whether integers k_u, one for each different stride u, make base' - base + sum of k_u u lie
// within the runs' widths; k_u is the difference of the grids' indices along the dimensions of that stride. Strides are
// taken from the largest down, and of each only the k_u that what lies below can still make up for: one to three
// where strides nest, as a tensor's do. A search past kMost steps counts as shared.
class Overlap {
 public:
  bool shared(const Grid& a, const Grid& b) {
    add(a, -1);
    add(b, 1);
    before_ = a.width, after_ = b.width;
    return search(static_cast<wide>(b.base) - static_cast<wide>(a.base), 0, false);
  }
  // whether two places of one grid do
  bool itself(const Grid& g) {
    for (int i = 0; i < g.dims; ++i) {
      if (g.dim[i].stride < g.width) return true;
      for (int j = 0; j < i; ++j)
        if (g.dim[i].stride == g.dim[j].stride) return true;
    }
    add(g, -1);
    add(g, 1);
    before_ = after_ = g.width;
    different_ = true;
    return search(0, 0, false);
  }

 private:
  using wide = __int128;  // strides below 2^40 bytes times indices below 2^31
  static constexpr int kMost = 1 << 16;
  struct Term {
    long long stride, lo, hi;  // lo <= k <= hi
    wide low, high;            // of the sum of this term and those below it
  } term_[6];
  int terms_ = 0, steps_ = 0;
  long long before_, after_;
  bool different_ = false;  // at least one k is not 0

  void add(const Grid& g, int sign) {
    for (int at = 0; at < g.dims; ++at) {
      const Grid::Dim& d = g.dim[at];
      if (d.stride == 0) continue;
      int i = 0;
      while (i < terms_ && term_[i].stride > d.stride) ++i;
      if (i == terms_ || term_[i].stride != d.stride) {
        std::copy_backward(term_ + i, term_ + terms_, term_ + terms_ + 1);
        term_[i] = {d.stride, 0, 0, 0, 0};
        ++terms_;
      }
      (sign > 0 ? term_[i].hi : term_[i].lo) += sign * (d.n - 1);
    }
    for (int i = terms_ - 1; i >= 0; --i) {
      const wide below_low = i + 1 < terms_ ? term_[i + 1].low : 0, below_high = i + 1 < terms_ ? term_[i + 1].high : 0;
      term_[i].low = below_low + static_cast<wide>(term_[i].lo) * term_[i].stride;
      term_[i].high = below_high + static_cast<wide>(term_[i].hi) * term_[i].stride;
    }
  }
  static wide floor_div(wide x, wide d) { return x / d - (x % d < 0 ? 1 : 0); }
  // `at`: base' - base and the terms above `level`
  bool search(wide at, int level, bool moved) {
    if (level == terms_) return at > -after_ && at < before_ && (moved || !different_);
    const Term& t = term_[level];
    const wide low = level + 1 < terms_ ? term_[level + 1].low : 0, high = level + 1 < terms_ ? term_[level + 1].high : 0;
    const wide first = std::max<wide>(t.lo, floor_div(-after_ - at - high, t.stride) + 1);
    const wide last = std::min<wide>(t.hi, floor_div(before_ - 1 - at - low, t.stride));
    for (wide k = first; k <= last; ++k) {
      if (++steps_ > kMost) return true;
      if (search(at + k * t.stride, level + 1, moved || k != 0)) return true;
    }
    return false;
  }
};
bool meet(const Grid& a, const Grid& b) { return a.base < b.end && b.base < a.end && Overlap().shared(a, b); }

svdq_status check_norm(const svdq_norm& n, const char* what, int D) {
  if (n.kind < SVDQ_NORM_NONE || n.kind > SVDQ_NORM_LAYER || (n.f32 != 0 && n.f32 != 1) ||
      (n.kind != SVDQ_NORM_NONE && !(n.eps >= 0.0f)))
    return fail(SVDQ_ERR_INVALID_ARG, "norm of %s: kind %d, eps %g, f32 %d", what, n.kind, n.eps, n.f32);
  const uintptr_t mask = n.f32 ? 3u : 1u;
  if (n.kind != SVDQ_NORM_NONE && ((reinterpret_cast<uintptr_t>(n.weight) | reinterpret_cast<uintptr_t>(n.bias)) & mask))
    return fail(SVDQ_ERR_UNSUPPORTED, "norm of %s: vectors of %d off their element size", what, D);
  return SVDQ_OK;
}

svdq_status check_heads(const svdq_heads& h, const char* what, const svdq_heads_args& a, bool stored) {
  if (h.heads < 1 || h.heads > kMaxHeads) return fail(SVDQ_ERR_INVALID_ARG, "%s: %d heads", what, h.heads);
  if (h.x == nullptr || (stored && h.out == nullptr)) return fail(SVDQ_ERR_INVALID_ARG, "%s: null pointer", what);
  auto bad = [&](long long sb, long long st, long long sh) {
    return sb < 0 || st < 0 || sh < 0 || sb >= kMaxStride || st >= kMaxStride || sh >= kMaxStride;
  };
  if (bad(h.sb, h.st, h.sh) || (stored && bad(h.ob, h.ot, h.oh)))
    return fail(SVDQ_ERR_INVALID_ARG, "%s: a stride is negative or above 2^38", what);
  const int xe = a.x_f32 ? 4 : 2, oe = a.out_f32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(h.x) & (xe - 1)) || (stored && (reinterpret_cast<uintptr_t>(h.out) & (oe - 1))))
    return fail(SVDQ_ERR_UNSUPPORTED, "%s: off its element size", what);
  return check_norm(h.norm, what, a.D);
}

svdq_status check_rope(const svdq_rope& r, int D) {
  if (r.dim == 0) return SVDQ_OK;
  if (r.dim < 0 || r.dim % 2 != 0 || r.dim > D)
    return fail(SVDQ_ERR_INVALID_ARG, "rotated values: %d of heads of %d", r.dim, D);
  if ((r.half != 0 && r.half != 1) || (r.inverse != 0 && r.inverse != 1) || (r.positions_i64 != 0 && r.positions_i64 != 1))
    return fail(SVDQ_ERR_INVALID_ARG, "rotary flags: half %d, inverse %d, positions_i64 %d", r.half, r.inverse,
                r.positions_i64);
  if (r.axes < 1 || r.axes > svdq::heads::kMaxAxes) return fail(SVDQ_ERR_INVALID_ARG, "%d position axes: 1 to 4", r.axes);
  int pairs = 0;
  for (int i = 0; i < r.axes; ++i) {
    if (r.axis_pairs[i] < 1 || r.axis_pairs[i] > r.dim / 2)
      return fail(SVDQ_ERR_INVALID_ARG, "axis %d: %d pairs", i, r.axis_pairs[i]);
    pairs += r.axis_pairs[i];
  }
  if (pairs != r.dim / 2) return fail(SVDQ_ERR_INVALID_ARG, "axes of %d pairs for %d rotated values", pairs, r.dim);
  if (r.turns == nullptr || r.positions == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "rotary: null pointer");
  const uintptr_t mask = r.positions_i64 ? 7u : 3u;
  if ((reinterpret_cast<uintptr_t>(r.turns) & 7u) || (reinterpret_cast<uintptr_t>(r.positions) & mask))
    return fail(SVDQ_ERR_UNSUPPORTED, "rotary: turns or positions off their element size");
  if (r.pb < 0 || r.pt < 0 || r.pb >= kMaxStride || r.pt >= kMaxStride)
    return fail(SVDQ_ERR_INVALID_ARG, "rotary: a position stride is negative or above 2^38");
  return SVDQ_OK;
}

svdq_status check_sizes(const svdq_heads_args& a) {
  if (a.samples < 0 || a.rows_per_sample < 0 ||
      static_cast<long long>(a.samples) * a.rows_per_sample > 0x7FFFFFFFll / 2)
    return fail(SVDQ_ERR_INVALID_ARG, "%d samples of %d rows", a.samples, a.rows_per_sample);
  if (a.D < 2 || a.D % 2 != 0 || a.D > svdq::heads::kMaxD)
    return fail(SVDQ_ERR_UNSUPPORTED, "heads of %d values: an even number up to %d", a.D, svdq::heads::kMaxD);
  if ((a.x_f32 != 0 && a.x_f32 != 1) || (a.out_f32 != 0 && a.out_f32 != 1))
    return fail(SVDQ_ERR_INVALID_ARG, "x_f32 %d, out_f32 %d", a.x_f32, a.out_f32);
  return SVDQ_OK;
}

bool same_view(const Grid& a, const Grid& b) {
  return a.base == b.base && a.width == b.width && a.dims == b.dims &&
         std::equal(a.dim, a.dim + a.dims, b.dim, [](const auto& l, const auto& r) { return l.stride == r.stride && l.n == r.n; });
}

// What a call reads, or what it writes.
struct Touched {
  Grid at;
  const char* name;
  const svdq_heads* of;  // whose heads: an output of heads may be their own input
};
struct TouchedList {
  Touched item[16];
  int n = 0;
  void add(const Grid& g, const char* name, const svdq_heads* of = nullptr) { item[n++] = {g, name, of}; }
  // a tensor's heads and the vectors of their norm
  void add_input(const svdq_heads& h, const char* name, const svdq_heads_args& a) {
    add(Grid(h.x, a.x_f32 ? 4 : 2, a.D, {h.sb, a.samples}, {h.st, a.rows_per_sample}, {h.sh, h.heads}), name, &h);
    if (h.norm.kind == SVDQ_NORM_NONE) return;
    if (h.norm.weight != nullptr) add(Grid(h.norm.weight, (h.norm.f32 ? 4 : 2) * a.D), "a norm's weight");
    if (h.norm.bias != nullptr) add(Grid(h.norm.bias, (h.norm.f32 ? 4 : 2) * a.D), "a norm's bias");
  }
  void add_output(const svdq_heads& h, const char* name, const svdq_heads_args& a) {
    add(Grid(h.out, a.out_f32 ? 4 : 2, a.D, {h.ob, a.samples}, {h.ot, a.rows_per_sample}, {h.oh, h.heads}), name, &h);
  }
  void add_rope(const svdq_rope& r, const svdq_heads_args& a) {
    if (r.dim == 0) return;
    add(Grid(r.turns, 4 * r.dim), "the turns");
    add(Grid(r.positions, r.positions_i64 ? 8 : 4, r.axes, {r.pb, a.samples}, {r.pt, a.rows_per_sample}), "the positions");
  }
  void add_cache(const svdq_kv_cache& c) {
    const long long heads = static_cast<long long>(c.pages) * c.page_size * c.heads;
    for (int i = 0; i < 2; ++i) {
      add(Grid(c.codes[i], heads * code_bytes(c.D, c.format)), "the cache's codes");
      add(Grid(c.scales[i], heads * scale_bytes(c.D, c.format)), "the cache's scales");
    }
  }
};

// Every output shares no byte with another place of its own, with what the call reads or with another output, but an output
// of heads may be their input (the same view, of one type).
svdq_status check_overlap(const TouchedList& out, const TouchedList& in) {
  for (int o = 0; o < out.n; ++o) {
    const Touched& y = out.item[o];
    if (!y.at.nested() && Overlap().itself(y.at)) return fail(SVDQ_ERR_INVALID_ARG, "%s: places of the output overlap", y.name);
    for (int i = 0; i < in.n; ++i) {
      const Touched& x = in.item[i];
      if (!(x.of != nullptr && x.of == y.of && same_view(x.at, y.at)) && meet(y.at, x.at))
        return fail(SVDQ_ERR_INVALID_ARG, "%s: the output overlaps %s", y.name, x.name);
    }
    for (int p = 0; p < o; ++p)
      if (meet(y.at, out.item[p].at))
        return fail(SVDQ_ERR_INVALID_ARG, "%s: the output overlaps %s", y.name, out.item[p].name);
  }
  return SVDQ_OK;
}

svdq_status check_cache(const svdq_kv_cache& c) {
  if (c.pages < 1 || c.page_size < 1 || c.heads < 1 || c.heads > kMaxHeads ||
      static_cast<long long>(c.pages) * c.page_size > (1ll << 40))
    return fail(SVDQ_ERR_INVALID_ARG, "cache of %d pages of %d, %d heads", c.pages, c.page_size, c.heads);
  if (c.D < 8 || c.D % 8 != 0 || c.D > svdq::heads::kMaxD)
    return fail(SVDQ_ERR_UNSUPPORTED, "cache heads of %d values: a multiple of 8 up to %d", c.D, svdq::heads::kMaxD);
  if (c.format != SVDQ_KV_FP8 && c.format != SVDQ_KV_MXFP4) return fail(SVDQ_ERR_INVALID_ARG, "cache format %d", c.format);
  for (int i = 0; i < 2; ++i) {
    if (c.codes[i] == nullptr || c.scales[i] == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "cache has a null buffer");
    if (!at16(c.codes[i])) return fail(SVDQ_ERR_UNSUPPORTED, "cache codes must be 16-byte aligned");
  }
  return SVDQ_OK;
}

unsigned magic(int d) { return d == 1 ? 0u : static_cast<unsigned>((0x100000000ull + d - 1) / d); }

svdq::heads::Cache device_cache(const svdq_kv_cache& c) {
  svdq::heads::Cache d{};
  d.page_size = c.page_size;
  d.heads = c.heads;
  d.D = c.D;
  d.mx = c.format == SVDQ_KV_MXFP4 ? 1 : 0;
  d.code_bytes = code_bytes(c.D, c.format);
  d.scale_bytes = scale_bytes(c.D, c.format);
  d.slots = static_cast<long long>(c.pages) * c.page_size;
  return d;
}

// Whether every access of 8 values (4 in the half layout) lies on its own size.
bool vector_ok(const svdq_heads_args& a, const svdq::heads::Args& k) {
  if (a.D % 8 != 0 || a.rope.dim % 8 != 0) return false;
  for (int i = 0; i < k.parts; ++i) {
    const auto& p = k.part[i];
    if (!at16(p.x) || (p.sb | p.st | p.sh) % 8 != 0) return false;
    if (!p.quant && (!at16(p.out) || (p.ob | p.ot | p.oh) % 8 != 0)) return false;
    if (p.norm && ((p.weight && !at16(p.weight)) || (p.bias && !at16(p.bias)))) return false;
  }
  return true;
}

void add_part(svdq::heads::Args& k, const svdq_heads& h, bool rotate) {
  auto& p = k.part[k.parts++];
  p.x = h.x;
  p.sb = h.sb;
  p.st = h.st;
  p.sh = h.sh;
  p.out = h.out;
  p.ob = h.ob;
  p.ot = h.ot;
  p.oh = h.oh;
  p.norm = h.norm.kind;
  if (p.norm != 0) {
    p.weight = h.norm.weight;
    p.bias = h.norm.bias;
    p.nf32 = h.norm.f32;
    p.eps = h.norm.eps;
  }
  p.heads = h.heads;
  p.rotate = rotate ? 1 : 0;
}

// KG: lanes per head fixed at compile time (16: heads of 72 to 128 values), or 0
using Kernel = void (*)(svdq::heads::Args, int);
template <class T, bool HALF, int KG>
Kernel heads_kernel(int cache) {
  using namespace svdq::heads;
  return cache == kFp8 ? svdq::heads::heads_kernel<T, HALF, KG, kFp8>
         : cache == kMx ? svdq::heads::heads_kernel<T, HALF, KG, kMx>
                        : svdq::heads::heads_kernel<T, HALF, KG, kBf16>;
}
template <class T>
Kernel heads_kernel(bool half, int G, int cache) {
  if (G == 16) return half ? heads_kernel<T, true, 16>(cache) : heads_kernel<T, false, 16>(cache);
  return half ? heads_kernel<T, true, 0>(cache) : heads_kernel<T, false, 0>(cache);
}

// Samples whose rows follow each other in every tensor are one sample.
void join_samples(svdq::heads::Args& k, const svdq_rope& rope) {
  const int T = k.rows_per_sample;
  if (k.samples == 1) return;
  auto even = [&](long long sb, long long st) { return T == 1 || sb == T * st; };
  for (int i = 0; i < k.parts; ++i) {
    const auto& p = k.part[i];
    if (!even(p.sb, p.st) || (!p.quant && !even(p.ob, p.ot))) return;
  }
  if (rope.dim > 0 && !even(rope.pb, rope.pt)) return;
  for (int i = 0; T == 1 && i < k.parts; ++i) k.part[i].st = k.part[i].sb, k.part[i].ot = k.part[i].ob;
  if (T == 1) k.rope.pt = rope.pb;
  k.rows_per_sample = T * k.samples;
  k.samples = 1;
}

svdq_status run_heads(const svdq_heads_args& a, svdq::heads::Args& k, svdq_stream_t stream) {
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  k.samples = a.samples;
  k.rows_per_sample = a.rows_per_sample;
  k.D = a.D;
  k.out_f32 = a.out_f32;
  if (a.rope.dim > 0) {
    k.rope.turns = reinterpret_cast<const unsigned long long*>(a.rope.turns);
    k.rope.pos = a.rope.positions;
    k.rope.pb = a.rope.pb;
    k.rope.pt = a.rope.pt;
    k.rope.dim = a.rope.dim;
    k.rope.half = a.rope.half;
    k.rope.pos_i64 = a.rope.positions_i64;
    k.rope.inverse = a.rope.inverse;
    k.rope.amplitude = a.rope.amplitude;
    int end = 0;
    for (int i = 0; i < svdq::heads::kMaxAxes; ++i) {
      if (i < a.rope.axes) end += a.rope.axis_pairs[i];
      k.rope.axis_end[i] = end;
    }
  }
  join_samples(k, a.rope);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int most = 0;
  for (int i = 0; i < k.parts; ++i) most = k.part[i].heads > most ? k.part[i].heads : most;
  constexpr int kWarps = svdq::heads::kThreads / 32;
  cudaError_t e;
  if (vector_ok(a, k) && k.samples <= 65535) {
    int G = 4;
    while (8 * G < a.D) G *= 2;
    const int per_warp = 32 / G;
    int units = 0;  // warps' worth of heads
    bool even = true;
    for (int i = 0; i < k.parts; ++i) {
      units += (k.part[i].heads + per_warp - 1) / per_warp;
      even = even && k.part[i].rotate == k.part[0].rotate;
    }
    // warps per block: 8, or fewer where that leaves fewer of them without a head
    int block = 8;
    for (int w = 7; w >= 4; --w)
      if (round_up(units, w) < round_up(units, block)) block = w;
    if (units < block) block = units;
    const int columns = (units + block - 1) / block;
    // Rows per block: as many blocks as make 32 warps an SM, which registers allow, so that their start and end are paid
    // once. (Blocks of one or two warps, of one to four heads, do not all fit: their tables let 11 blocks on an SM, and the
    // grid takes 1.5 to 3 rounds. With 11 blocks counted in their place, us here / there: 4608 rows of 1 head 7.3 / 4.6, of 4
    // 7.1 / 5.2; 16896 rows of 1 12.0 / 11.8, of 4 12.8 / 14.8; 65536 rows of 1 34.5 / 36.6, of 4 43.4 / 40.4: better for some,
    // worse for others, as strips are whole batches.) Where some parts cost more than others (rotation, norm) three rounds of blocks even that out, if strips stay
    // long (16384 tokens written, 72 heads of 128: 115, 110, 104 and 105 us at 1 to 4 rounds; q and k of 16896 rows, all
    // alike: 70, 73, 75 us at 1 to 3).
    const long long columns_all = static_cast<long long>(columns) * k.samples;
    auto strip_of = [&](int rounds) {
      const long long strips = std::max(1ll, rounds * (32 / block) * static_cast<long long>(sms) / columns_all);
      const long long n = (k.rows_per_sample + strips - 1) / strips;
      return n > svdq::heads::kBatch ? (n + svdq::heads::kBatch - 1) / svdq::heads::kBatch * svdq::heads::kBatch : n;
    };
    long long strip = strip_of(even ? 1 : 3);
    if (strip < 4 * svdq::heads::kBatch) strip = strip_of(1);
    k.strip = static_cast<int>(strip);
    const dim3 grid(static_cast<unsigned>((k.rows_per_sample + strip - 1) / strip), columns, k.samples);
    const bool half = a.rope.dim > 0 && a.rope.half != 0;
    const int cache = !k.part[k.parts - 1].quant ? svdq::heads::kBf16 : k.cache.mx ? svdq::heads::kMx : svdq::heads::kFp8;
    const Kernel kern = a.x_f32 ? heads_kernel<float>(half, G, cache) : heads_kernel<__nv_bfloat16>(half, G, cache);
    e = launch(kern, grid, 32 * block, 0, 0, st, k, G);
  } else {
    const int split = (most + kWarps - 1) / kWarps;
    const dim3 grid(k.samples * k.rows_per_sample, split < 8 ? split : 8, 1);
    e = a.x_f32 ? launch(svdq::heads::heads_any_kernel<float>, grid, svdq::heads::kThreads, 0, 0, st, k)
                : launch(svdq::heads::heads_any_kernel<__nv_bfloat16>, grid, svdq::heads::kThreads, 0, 0, st, k);
  }
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of heads::heads_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("heads::heads_kernel");
}

}  // namespace

extern "C" {

svdq_status svdq_rotary(const svdq_heads_args* a, svdq_stream_t stream) {
  if (a == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_sizes(*a); s != SVDQ_OK) return s;
  if (a->rope.dim == 0) return fail(SVDQ_ERR_INVALID_ARG, "no value is rotated");
  if (svdq_status s = check_rope(a->rope, a->D); s != SVDQ_OK) return s;
  const bool two = a->k.heads != 0;
  if (a->v.heads != 0) return fail(SVDQ_ERR_INVALID_ARG, "v belongs to svdq_kv_write");
  if (a->samples == 0 || a->rows_per_sample == 0) return SVDQ_OK;  // no row: empty tensors have no address
  if (svdq_status s = check_heads(a->q, "q", *a, true); s != SVDQ_OK) return s;
  if (two)
    if (svdq_status s = check_heads(a->k, "k", *a, true); s != SVDQ_OK) return s;
  TouchedList in, out;
  in.add_input(a->q, "q", *a);
  out.add_output(a->q, "q", *a);
  if (two) in.add_input(a->k, "k", *a), out.add_output(a->k, "k", *a);
  in.add_rope(a->rope, *a);
  if (svdq_status s = check_overlap(out, in); s != SVDQ_OK) return s;
  svdq::heads::Args k{};
  add_part(k, a->q, true);
  if (two) add_part(k, a->k, true);
  return run_heads(*a, k, stream);
}

size_t svdq_kv_code_bytes(int pages, int page_size, int heads, int D, svdq_kv_format format) {
  if (pages < 1 || page_size < 1 || heads < 1 || heads > kMaxHeads || D < 8 || D % 8 != 0 || D > svdq::heads::kMaxD ||
      (format != SVDQ_KV_FP8 && format != SVDQ_KV_MXFP4) || static_cast<long long>(pages) * page_size > (1ll << 40))
    return 0;
  return static_cast<size_t>(pages) * page_size * heads * code_bytes(D, format);
}

size_t svdq_kv_scale_bytes(int pages, int page_size, int heads, int D, svdq_kv_format format) {
  if (svdq_kv_code_bytes(pages, page_size, heads, D, format) == 0) return 0;
  return static_cast<size_t>(pages) * page_size * heads * scale_bytes(D, format);
}

svdq_status svdq_kv_write(const svdq_kv_cache* c, const svdq_heads_args* a, const void* slots, int slots_i64,
                          svdq_stream_t stream) {
  if (c == nullptr || a == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_cache(*c); s != SVDQ_OK) return s;
  if (svdq_status s = check_sizes(*a); s != SVDQ_OK) return s;
  if (svdq_status s = check_rope(a->rope, a->D); s != SVDQ_OK) return s;
  if (a->D != c->D) return fail(SVDQ_ERR_INVALID_ARG, "heads of %d values for a cache of %d", a->D, c->D);
  if (slots_i64 != 0 && slots_i64 != 1) return fail(SVDQ_ERR_INVALID_ARG, "slots_i64 %d", slots_i64);
  const bool q = a->q.heads != 0;
  if (a->v.norm.kind != SVDQ_NORM_NONE) return fail(SVDQ_ERR_INVALID_ARG, "v has no norm");
  if (a->samples == 0 || a->rows_per_sample == 0) return SVDQ_OK;
  if (slots == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (reinterpret_cast<uintptr_t>(slots) & (slots_i64 ? 7u : 3u))
    return fail(SVDQ_ERR_UNSUPPORTED, "slots off their element size");
  if (q)
    if (svdq_status s = check_heads(a->q, "q", *a, true); s != SVDQ_OK) return s;
  if (svdq_status s = check_heads(a->k, "k", *a, false); s != SVDQ_OK) return s;
  if (svdq_status s = check_heads(a->v, "v", *a, false); s != SVDQ_OK) return s;
  if (a->k.heads != c->heads || a->v.heads != c->heads)
    return fail(SVDQ_ERR_INVALID_ARG, "k of %d heads, v of %d, for a cache of %d", a->k.heads, a->v.heads, c->heads);
  TouchedList in, out;
  if (q) in.add_input(a->q, "q", *a), out.add_output(a->q, "q", *a);
  in.add_input(a->k, "k", *a);
  in.add_input(a->v, "v", *a);
  in.add_rope(a->rope, *a);
  in.add(Grid(slots, (slots_i64 ? 8ll : 4ll) * a->samples * a->rows_per_sample), "the slots");
  out.add_cache(*c);
  if (svdq_status s = check_overlap(out, in); s != SVDQ_OK) return s;
  svdq::heads::Args k{};
  k.cache = device_cache(*c);
  k.slots = slots;
  k.slots_i64 = slots_i64;
  if (q) add_part(k, a->q, a->rope.dim > 0);
  for (int i = 0; i < 2; ++i) {
    add_part(k, i ? a->v : a->k, i == 0 && a->rope.dim > 0);
    auto& p = k.part[k.parts - 1];
    p.quant = 1;
    p.codes = static_cast<uint8_t*>(c->codes[i]);
    p.scales = static_cast<uint8_t*>(c->scales[i]);
  }
  return run_heads(*a, k, stream);
}

svdq_status svdq_kv_read(const svdq_kv_cache* c, const int32_t* table, long long ld_table, int width,
                         const int32_t* offsets, int samples, int rows, void* k_out, long long k_row, long long k_head,
                         void* v_out, long long v_row, long long v_head, svdq_out_dtype out_dtype, svdq_stream_t stream) {
  if (c == nullptr || offsets == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_cache(*c); s != SVDQ_OK) return s;
  if (out_dtype != SVDQ_OUT_BF16 && out_dtype != SVDQ_OUT_F32) return fail(SVDQ_ERR_INVALID_ARG, "bad out dtype");
  if (samples < 1 || rows < 0 || rows > 0x7FFFFFFF / 2 || width < 0 || ld_table < (samples > 1 ? width : 0) ||
      ld_table >= kMaxStride)
    return fail(SVDQ_ERR_INVALID_ARG, "%d samples, %d rows, a table of %d columns and stride %lld", samples, rows, width,
                ld_table);
  if (rows == 0) return SVDQ_OK;
  if (k_out == nullptr || v_out == nullptr || (width > 0 && table == nullptr))
    return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const int esize = out_dtype == SVDQ_OUT_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(table) & 3u) || (reinterpret_cast<uintptr_t>(offsets) & 3u) ||
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & (esize - 1)))
    return fail(SVDQ_ERR_UNSUPPORTED, "table, offsets or outputs off their element size");
  svdq_heads_args o{};
  o.samples = 1;
  o.rows_per_sample = rows;
  o.D = c->D;
  o.out_f32 = o.x_f32 = out_dtype == SVDQ_OUT_F32 ? 1 : 0;
  o.k.heads = o.v.heads = c->heads;
  o.k.out = k_out, o.k.ot = k_row, o.k.oh = k_head;
  o.v.out = v_out, o.v.ot = v_row, o.v.oh = v_head;
  if (k_row < 0 || k_head < 0 || v_row < 0 || v_head < 0 || k_row >= kMaxStride || k_head >= kMaxStride ||
      v_row >= kMaxStride || v_head >= kMaxStride)
    return fail(SVDQ_ERR_INVALID_ARG, "an output stride is negative or above 2^38");
  TouchedList in, out;
  out.add_output(o.k, "keys", o);
  out.add_output(o.v, "values", o);
  in.add_cache(*c);
  in.add(Grid(offsets, 4 * (samples + 1ll)), "the offsets");
  if (width > 0) in.add(Grid(table, 4, width, {ld_table, samples}), "the table");
  if (svdq_status s = check_overlap(out, in); s != SVDQ_OK) return s;
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  svdq::heads::ReadArgs r{};
  for (int i = 0; i < 2; ++i) {
    r.codes[i] = static_cast<const uint8_t*>(c->codes[i]);
    r.scales[i] = static_cast<const uint8_t*>(c->scales[i]);
    const svdq_heads& h = i ? o.v : o.k;
    r.out[i] = h.out;
    r.ot[i] = h.ot;
    r.oh[i] = h.oh;
  }
  r.cache = device_cache(*c);
  r.table = table;
  r.offsets = offsets;
  r.ld_table = ld_table;
  r.width = width;
  r.samples = samples;
  r.rows = rows;
  const long long strides = k_row | k_head | v_row | v_head;
  const bool vec = at16(k_out) && at16(v_out) && strides % 8 == 0;
  const bool wide = c->D % 16 == 0 && ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0 &&
                    strides % 16 == 0;
  r.per_head = c->D / (wide ? 16 : 8);
  r.chunks = c->heads * r.per_head;
  r.magic = magic(r.per_head);
  r.magic_row = magic(r.chunks);
  // rows per block: as many as fill its loads in flight, fewer where that leaves SMs without a block
  const int fill = std::max(1, svdq::heads::kThreads * (wide ? 4 : 8) / r.chunks);
  const int spread = std::max(1, rows / sms);
  r.block_rows = std::min(std::min(fill, spread), svdq::heads::kReadRows);
  using namespace svdq::heads;
  auto* kern = o.out_f32 ? (wide ? kv_read_kernel<true, 16, true> : vec ? kv_read_kernel<true, 8, true> : kv_read_kernel<true, 8, false>)
                         : (wide  ? kv_read_kernel<false, 16, true>
                            : vec ? kv_read_kernel<false, 8, true>
                                  : kv_read_kernel<false, 8, false>);
  const cudaError_t e = launch(kern, dim3((rows + r.block_rows - 1) / r.block_rows, 2),
                               svdq::heads::kThreads, 0, 0, static_cast<cudaStream_t>(stream), r);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of heads::kv_read_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("heads::kv_read_kernel");
}

}  // extern "C"
