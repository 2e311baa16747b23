// api_linear.cu -- the C ABI of the operators on BF16 layers (sgemm_linear.h): argument checks, workspace and launches.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>
#include <iterator>

#include "linear_internal.h"
#include "sgemm_internal.h"
#include "sgemm_linear.h"

using namespace sgemm_impl;

namespace {

constexpr int64_t kMaxDim = INT_MAX - 1024;  // indices of the kernels' last tiles stay below 2^31

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// The row stride of copies and of what lies in the workspace: whole lines of 128 bytes (rows of 4112 bytes, which the tensor
// cores' copies can read too, cost a fifth more per K tile, as each 128 bytes of them lie in two lines).
int64_t whole_lines(int64_t n) { return ceil_div(n, 64) * 64; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int type_size(int type) { return type == SGEMM_BF16 ? 2 : 4; }
bool known_type(int type) { return type == SGEMM_F32 || type == SGEMM_BF16; }
bool known_act(int act) { return act >= SGEMM_ACT_NONE && act <= SGEMM_ACT_GELU_TANH; }

// Whether rows of elements of `size` bytes start at multiples of `n` bytes.
bool rows_at(const void* p, int64_t ld, int size, int n) { return aligned(p, n) && ld * size % n == 0; }

// A matrix argument: its memory is there (where it is used), aligned to its type, and its rows do not overlap.
bool usable(const void* p, int size, bool used) { return !used || (p && aligned(p, size)); }
bool wide_enough(int64_t ld, int64_t cols) { return ld >= std::max<int64_t>(1, cols); }
// A kept matrix (checked as a whole: one argument).
bool usable_kept(const sgemm_kept_t* k, int64_t cols, bool work) {
  if (!k) return true;
  if (!wide_enough(k->ld, cols) || !usable(k->data, k->scale ? 1 : 2, work)) return false;
  return !k->scale || (aligned(k->scale, 4) && wide_enough(k->lds, ceil_div(cols, 128)));
}

// ---------------------------------------------------------------- the choice of kernel

std::atomic<int> g_force_variant{SGEMM_VARIANT_AUTO}, g_force_tile{0}, g_force_split{0};

// K tiles that a BF16 output's sum has in one accumulator of the pair kernel, at most.  The tensor cores truncate what they add:
// the more, the larger the accumulator is against it, and where the terms have one sign all in one direction.  At this length
// such a sum is 7.5e-5 too small, a twenty-sixth of a BF16 value's smallest half step; accumulators of 1024 K tiles were 3.8e-4 off
// and whole sums of 16384 of them 6.6e-3, three half steps (measured; where signs are random 6.1e-8 per K tile).
constexpr int kWholeMost = 256;

// A product: M x N over `segments` times K.
struct Shape {
  int64_t M = 0, N = 0, K = 0;
  int segments = 1;
  bool gated = false, kept8 = false;
  int64_t k_tiles() const { return ceil_div(K, 64) * segments; }
  bool long_sum() const { return k_tiles() > kWholeMost; }
  int64_t pair_tiles(int tile) const { return ceil_div(M, 256) * ceil_div(N, gated ? tile / 2 : tile); }
};

// Times in ns that the choice of kernel goes by, fitted to 640 launches of 54 products (1 to 4096 tokens, gradients and gated ones
// among them) forced to each kernel, tile and split on a GB300.  Against 1249 launches of these and 15 more products with long sums
// they are off by 10 to 13% (20% where units of the pair kernel share K), and the launch they choose takes 2.5% longer than the
// fastest on average, 29% at worst.  In the pair kernel, by tile width: a K tile of 64, and the rest of a tile,
// and the rate at which few clusters read.  On the short side: a K tile in a CTA that has its SM to itself, the rest of a tile, and
// what joining a tile's shares adds.
struct PairCost {
  int tile, k_ns, tile_ns;
};
constexpr PairCost kPairCost[] = {{256, 294, 2020}, {128, 215, 1060}, {64, 209, 740}};
struct ShortCost {
  int tile, k_ns, tile_ns, join_ns;
};
constexpr ShortCost kShortCost[] = {{16, 267, 2730, 570}, {32, 298, 3580, 85}, {64, 328, 4530, 5}, {128, 154, 6330, 0}};
constexpr double kPairLaunchNs = 3000, kShortLaunchNs = 790;
constexpr double kPairBytesPerNs = 3490;
constexpr int kLeastShare = 8;  // K tiles of a unit that shares a tile
constexpr double kJoinNs = 4000, kJoinBytesPerNs = 4000;
constexpr double kSharedSm = 0.34;       // a K tile takes this much longer with a second CTA on the SM
constexpr double kGatedK = 1.19, kGatedTile = 1.36;  // a gated tile's K tiles and rest against a plain one's
constexpr double kSmBytesPerNs = 89.0;   // an SM's largest share of the memory bandwidth

// CTAs that run at a time in clusters of `split` with `per_sm` to an SM: groups of 4 or 8 do not fill every part of the chip.
int64_t cluster_ctas(int sm_count, int split, int per_sm) {
  const int of19 = split <= 2 ? 19 : split == 4 ? 18 : per_sm > 1 ? 17 : 15;
  return std::max<int64_t>(split, (int64_t)sm_count * per_sm * of19 / 19);
}

bool short_alone(int tile, bool gated) { return gated || tile == 128; }  // one CTA per SM
int64_t short_ring(int tile, bool gated) { return (short_alone(tile, gated) ? 2 : 1) * 98 * 1024; }

bool pair_tile_fits(int tile, const Shape& s) {
  return s.gated ? tile >= (s.kept8 || s.long_sum() ? 256 : 128) : tile >= (s.kept8 ? 128 : 64);
}

struct Choice {
  int variant = 0, tile = 0, split = 1;            // split: of the short-side kernel
  int splits[kLinearJobs] = {1, 1, 1};             // of each product in the pair kernel
  double ns = 1e30;
};

// The pair kernel's time for up to three products in one launch, the K tiles of each tile of product i shared by splits[i] units:
// that of the cluster with the most work (units are dealt round robin; a cluster has one more of a product's where the deal of
// its last round starts, so one of these has the most), and of joining the shares.
double pair_ns(const Shape* s, int n, const PairCost& c, int64_t clusters, const int* splits) {
  double most = 0.0, bytes = 0.0, joined = 0.0;
  int64_t units[kLinearJobs];
  for (int i = 0; i < n; ++i) {
    units[i] = s[i].pair_tiles(c.tile) * splits[i];
    bytes += 2.0 * ((double)s[i].M * s[i].K * s[i].segments + (double)s[i].N * s[i].K * s[i].segments * (s[i].gated ? 2 : 1) + (double)s[i].M * s[i].N);
    if (splits[i] > 1) joined += 4.0 * s[i].M * s[i].N * (2 * splits[i] + 1);
  }
  int64_t start = 0;
  for (int i = 0; i < n; start += units[i++]) {
    const int64_t at = (start + units[i] / clusters * clusters) % clusters;
    double ns = 0.0;
    int64_t first = 0;
    for (int k = 0; k < n; first += units[k++]) {
      // units of product k that cluster `at` gets: those in [first, first + units) that are `at` modulo the clusters
      const int64_t skip = ((at - first) % clusters + clusters) % clusters;
      const int64_t mine = units[k] > skip ? (units[k] - skip - 1) / clusters + 1 : 0;
      ns += (double)mine * (ceil_div(s[k].k_tiles(), splits[k]) * c.k_ns + c.tile_ns);
    }
    most = std::max(most, ns);
  }
  return kPairLaunchNs + std::max(most, bytes / kPairBytesPerNs) + (joined > 0.0 ? kJoinNs + joined / kJoinBytesPerNs : 0.0);
}

// The pair kernel's launch with K shared where that is worth it: units of about equal length, as many as clusters or twice that.
void offer_pair(const Shape* s, int n, const PairCost& c, int64_t clusters, int forced, Choice* best) {
  const auto offer = [&](const int* splits) {
    const double ns = pair_ns(s, n, c, clusters, splits);
    if (ns >= best->ns) return;
    *best = Choice{SGEMM_VARIANT_LINEAR_PAIR, c.tile, 1, {1, 1, 1}, ns};
    std::copy(splits, splits + n, best->splits);
  };
  int splits[kLinearJobs] = {1, 1, 1};
  int64_t tiles = 0, steps = 0, longest = 0;
  for (int i = 0; i < n; ++i) {
    tiles += s[i].pair_tiles(c.tile);
    steps += s[i].pair_tiles(c.tile) * s[i].k_tiles();
    longest = std::max(longest, s[i].k_tiles());
  }
  const bool can = !s[0].gated && !s[0].kept8;  // (the joining kernel has no second product and no groups)
  if (forced > 0 && can) {
    for (int i = 0; i < n; ++i) splits[i] = (int)std::min<int64_t>(forced, s[i].k_tiles());
    return offer(splits);
  }
  offer(splits);
  if (!can || forced > 0 || tiles >= 2 * clusters || longest < 2 * kLeastShare) return;
  for (int rounds = 1; rounds <= 2; ++rounds) {
    const double length = std::max((double)kLeastShare, (double)steps / (double)(rounds * clusters));
    bool any = false;
    for (int i = 0; i < n; ++i) {
      splits[i] = (int)std::max<int64_t>(1, std::min<int64_t>(kLinearMostShares, (int64_t)((double)s[i].k_tiles() / length + 0.25)));
      any |= splits[i] > 1;
    }
    if (any) offer(splits);
  }
}

// The cheapest launch of one product (several: in one launch of the pair kernel), among the variant, tile and split that are
// forced (0: any); clusters: CTA pairs that run at a time, 0 on a device without clusters, where only unshared tiles can run.
Choice choose(const Shape* s, int n, int64_t clusters, int sm_count, int variant, int tile, int split) {
  Choice best;
  const auto offer = [&](int v, int t, int k, double ns) {
    if (ns < best.ns) best = Choice{v, t, k, {1, 1, 1}, ns};
  };
  const auto forced_here = [&](const auto& tiles, const auto& fits) {
    return std::any_of(std::begin(tiles), std::end(tiles), [&](int t) { return t == tile && fits(t); });
  };
  if (variant != SGEMM_VARIANT_LINEAR_SHORT && clusters > 0) {
    const bool only = forced_here(kLinearPairTiles, [&](int t) { return pair_tile_fits(t, s[0]); });
    for (const PairCost& c : kPairCost)
      if (pair_tile_fits(c.tile, s[0]) && (!only || c.tile == tile)) offer_pair(s, n, c, clusters, variant == SGEMM_VARIANT_LINEAR_PAIR ? split : 0, &best);
  }
  if (variant != SGEMM_VARIANT_LINEAR_PAIR && n == 1) {
    const int64_t kt = s->k_tiles();
    const bool gated = s->gated;
    const auto fits = [&](int t) { return !gated || t < 128; };
    const bool only = forced_here(kLinearShortTiles, fits);
    for (const ShortCost& c : kShortCost) {
      if (!fits(c.tile) || (only ? c.tile != tile : c.tile > 16 && c.tile >= 2 * s->M)) continue;
      const int64_t tiles = ceil_div(s->N, 128) * ceil_div(s->M, c.tile);
      if (tiles * 8 > INT_MAX) continue;
      const int wide = gated ? 2 : 1;
      for (int k = 1; k <= 8; k *= 2) {
        if (clusters == 0 && k > 1) break;
        if (split != 0 ? split != k : k > 1 && kt < 2 * k) continue;  // two K tiles per CTA at least
        const int per_sm = short_alone(c.tile, gated) ? 1 : 2;
        const double on_sm = std::min((double)per_sm, std::max(1.0, (double)tiles * k / sm_count));
        const double one = std::max(c.k_ns * (gated ? kGatedK : 1.0) * (1.0 + kSharedSm * (on_sm - 1.0)), on_sm * (16384 * wide + 64 * c.tile) / kSmBytesPerNs);
        const double rounds = (double)ceil_div(tiles * k, cluster_ctas(sm_count, k, per_sm));
        offer(SGEMM_VARIANT_LINEAR_SHORT, c.tile, k,
              kShortLaunchNs + rounds * (ceil_div(kt, k) * one + c.tile_ns * (gated ? kGatedTile : 1.0) + (k > 1 ? c.join_ns : 0)));
      }
    }
  }
  return best;
}

Choice choose(const Shape* s, int n, int sm_count, int pair_clusters) {
  const int64_t clusters = pair_clusters >= 0 ? pair_clusters : std::max(1, sm_count / 2);
  return choose(s, n, clusters, sm_count, g_force_variant.load(), g_force_tile.load(), g_force_split.load());
}

int64_t short_stage(int tile, bool gated, bool s_mn) { return (gated ? 2 : 1) * 16384 + (s_mn ? std::max(1, tile / 64) * 8192 : tile * 128); }
int short_stages(int tile, bool gated, bool s_mn) {
  return (int)std::min<int64_t>(kLinearShortMaxStages, short_ring(tile, gated) / short_stage(tile, gated, s_mn));
}

// ---------------------------------------------------------------- operands and workspace

// Pieces of one workspace, 256 bytes apart (counted first, then placed).
struct Pieces {
  uint8_t* base = nullptr;
  int64_t at = 0;
  template <typename T>
  T* take(int64_t n) {
    T* r = base ? reinterpret_cast<T*>(base + at) : nullptr;
    at += round256(n * (int64_t)sizeof(T));
    return r;
  }
};

// A stored matrix of a product.  TMA reads BF16 rows that start at multiples of 16 bytes; others are copied first.
struct Operand {
  LinearKeptIn m;
  int64_t rows = 0, cols = 0;  // stored
  void* copy = nullptr;
  bool copied = false;

  Operand() = default;
  Operand(const void* p, int64_t ld, const float* scale, int64_t lds, int64_t rows_, int64_t cols_) : rows(rows_), cols(cols_) {
    m.data = p;
    m.ld = ld;
    m.scale = scale;
    m.lds = lds;
    copied = scale || !aligned(p, 16) || (ld % 8 != 0 && rows > 1);
  }
  void place(Pieces* w) {
    if (copied) copy = w->take<uint16_t>(rows * whole_lines(cols));
  }
  cudaError_t map(int box_rows, CUtensorMap* out) const {
    const int64_t ld = copied || rows == 1 ? whole_lines(cols) : m.ld;  // (a map wants a stride even where it steps over nothing)
    return encode_linear_map(copied ? copy : m.data, cols, rows, ld, box_rows, out);
  }
};

// Makes the copies that operands (up to three of them) need, in one launch.
cudaError_t make_copies(std::initializer_list<const Operand*> list, const Guard& g, cudaStream_t stream) {
  LinearExpandParams p;
  p.guard = g;
  int n = 0;
  for (const Operand* o : list) {
    if (!o || !o->copied) continue;
    LinearExpand& e = p.part[n++];
    e.m = o->m;
    e.rows = o->rows;
    e.cols = (int)o->cols;
    e.dst = o->copy;
    e.ldd = whole_lines(o->cols);
  }
  return n ? launch_linear_expand(p, stream) : cudaSuccess;
}

// Tensor-core instruction descriptor, kind::f16: FP32 accumulator, BF16 operands, their orders (1: MN-major), N and M.
uint32_t instruction(int a_mn, int b_mn, int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}

// A product with its operands and output.  mn: an operand's stored rows run along the output, not along k.
struct Product {
  Shape shape;
  const Operand *a[2] = {nullptr, nullptr}, *b[2] = {nullptr, nullptr};
  int a_mn = 0, b_mn = 0;
  void* d = nullptr;
  int64_t ldd = 0;
  bool f32 = false;
};

// K tiles of 64 that the pair kernel sums in one accumulator where FP32 values leave it (an FP32 output, scales): 8, but for the
// first, which takes more the longer the sum is: the epilogue of the tile before has the first one's time, 294 ns per K tile of a
// 256-wide tile, before the folding starts again.  An accumulator of n K tiles is off by 6.1e-8 n of its own sum (measured over 1 to
// 256 of them), in that sum's direction.  The sums of several are independent and go by the square roots of their lengths n_i, so
// together they are off by 6.1e-8 sqrt(sum(n_i^3) / sum(n_i)) of the whole.  The first is the longest that keeps this root at 13
// (8e-7): n^3 - 64 n <= 105 K tiles.  (A first of 16 whatever the length, and of 24 for 8-bit values
// of longer sums, were off by 1e-6 at some lengths.  Sums of terms of one sign come out 7.3e-7 too small at most, by 1 to 1024 K tiles.)
constexpr int kFold = 8, kFoldMost = 32;
int first_fold(int64_t k_tiles) {
  int n = kFold;
  while (n < kFoldMost && (int64_t)(n + 1) * ((n + 1) * (n + 1) - 64) <= 105 * k_tiles) ++n;
  return n;
}

// One launch of the products: of one with a choice of either kernel, of several with the pair kernel.
struct Launch {
  Product pr[kLinearJobs];
  int n = 0;
  LinearOut out;

  Product& add() { return pr[n++]; }

  // How it runs: all in one launch of the pair kernel; or the first by itself, where that is cheaper (a product of few rows
  // beside long ones), and the others in one; or (no clusters) each by itself.
  struct Group {
    int first, count;
    Choice choice;
  };
  Group group[kLinearJobs];
  int groups = 0;
  float* sums[kLinearJobs] = {nullptr, nullptr, nullptr};  // of products whose K is shared

  void plan(const CallDevice& dev) {
    Shape s[kLinearJobs];
    for (int i = 0; i < n; ++i) s[i] = pr[i].shape;
    const auto of = [&](int first, int count) { return Group{first, count, choose(s + first, count, dev.sm_count, dev.pair_clusters)}; };
    group[0] = of(0, n);
    groups = 1;
    if (n == 1) return;
    const Group one = of(0, 1), rest = of(1, n - 1);
    if (rest.choice.variant == 0) {
      for (groups = 0; groups < n; ++groups) group[groups] = of(groups, 1);
    } else if (one.choice.ns + rest.choice.ns < group[0].choice.ns) {
      group[0] = one;
      group[1] = rest;
      groups = 2;
    }
  }
  bool by_pairs() const { return n == 1 && group[0].choice.variant == SGEMM_VARIANT_LINEAR_PAIR; }
  bool shares_k() const { return group[0].choice.splits[0] > 1; }

  static int64_t sums_ld(const Shape& s) { return ceil_div(s.N, 32) * 32; }
  static int64_t rows_apart(const Shape& s) { return ceil_div(s.M, 256) * 256; }
  void place(Pieces* w) {
    for (int g = 0; g < groups; ++g)
      for (int i = 0; i < group[g].count; ++i) {
        const int split = group[g].choice.splits[i], at = group[g].first + i;
        if (split > 1) sums[at] = w->take<float>(split * rows_apart(pr[at].shape) * sums_ld(pr[at].shape));
      }
  }

  int run(const CallDevice& dev, cudaStream_t stream, cudaError_t* e) {
    int st = SGEMM_OK;
    for (int g = 0; g < groups && st == SGEMM_OK && *e == cudaSuccess; ++g) st = launch(group[g].first, group[g].count, group[g].choice, dev, stream, e);
    return st;
  }

 private:
  int launch(int first, int count, const Choice& c, const CallDevice& dev, cudaStream_t stream, cudaError_t* e) {
    const Product* list = pr + first;
    if (c.variant == 0) return SGEMM_ERR_UNSUPPORTED;  // forced to what needs clusters
    const bool pair = c.variant == SGEMM_VARIANT_LINEAR_PAIR, gated = list[0].shape.gated;
    out.guard = {dev.fault, dev.bounds};
    out.bias_vec = aligned(out.bias, 16);
    out.r_vec = rows_at(out.residual, out.ldr, 2, 16);
    LinearMaps maps;
    LinearPairParams p;
    LinearJoinParams join;
    bool joins = false;
    const Operand* known[6];
    int box[6], maps_used = 0;
    const auto map_of = [&](const Operand* o, int rows) {  // an operand's map, made once
      for (int i = 0; i < maps_used; ++i)
        if (known[i] == o && box[i] == rows) return i;
      known[maps_used] = o;
      box[maps_used] = rows;
      if (*e == cudaSuccess) *e = o->map(rows, &maps.op[maps_used]);
      return maps_used++;
    };
    int64_t tiles = 0, steps = 0;
    bool fold = out.keep == 2;
    for (int i = 0; i < count; ++i) fold |= list[i].f32 || c.splits[i] > 1 || list[i].shape.long_sum();
    for (int i = 0; i < count; ++i) {
      const Product& r = list[i];
      LinearJob& j = p.job[i];
      const int size = r.f32 ? 4 : 2;
      j.M = (int)r.shape.M;
      j.N = (int)r.shape.N;
      j.d = r.d;
      j.ldd = r.ldd;
      j.f32 = r.f32;
      j.d_tma = tma_writes(r.d, r.ldd, r.shape.N, size);
      j.d_vec = rows_at(r.d, r.ldd, size, 4 * size);
      j.k_tiles = (int)ceil_div(r.shape.K, 64);
      j.segments = r.shape.segments;
      const bool wide = r.f32 || out.keep == 2;  // FP32 values leave the kernel
      j.fold0 = wide ? first_fold(r.shape.k_tiles()) : kWholeMost;
      j.fold = wide ? kFold : kWholeMost;
      j.a_mn = r.a_mn;
      j.b_mn = r.b_mn;
      if (pair) {
        j.tiles_m = (int)ceil_div(r.shape.M, 256);
        j.tiles_n = (int)ceil_div(r.shape.N, gated ? c.tile / 2 : c.tile);
        j.idesc = instruction(r.a_mn, r.b_mn, 256, c.tile);
        if (c.splits[i] > 1) {  // the units' sums are what the kernel writes
          LinearJoin& t = join.part[i];
          t.sums = sums[first + i];
          t.ld = sums_ld(r.shape);
          t.split = c.splits[i];
          t.rows_apart = (int)rows_apart(r.shape);
          t.job = j;
          joins = true;
          if ((int64_t)t.split * t.rows_apart > kMaxDim) return SGEMM_ERR_UNSUPPORTED;
          j.split = t.split;
          j.rows_apart = t.rows_apart;
          j.M = t.split * t.rows_apart;
          j.N = (int)t.ld;
          j.d = sums[first + i];
          j.ldd = t.ld;
          j.f32 = j.d_tma = 1;
          j.fold0 = first_fold(ceil_div(r.shape.k_tiles(), t.split));
          j.fold = kFold;
          if (*e == cudaSuccess) *e = encode_linear_out_map(j.d, t.ld, j.M, t.ld, false, 32, &maps.d[i]);
        } else if (j.d_tma && *e == cudaSuccess) *e = encode_linear_out_map(r.d, r.shape.N / (16 / size) * (16 / size), r.shape.M, r.ldd, !r.f32, r.f32 ? 32 : linear_pair_box(c.tile, gated, fold), &maps.d[i]);
      } else {
        j.tiles_m = (int)ceil_div(r.shape.M, c.tile);
        j.tiles_n = (int)ceil_div(r.shape.N, 128);
        j.idesc = instruction(r.b_mn, r.a_mn, 128, c.tile);
      }
      for (int k = 0; k < 2; ++k) {
        if (r.a[k]) j.a[k] = map_of(r.a[k], r.a_mn || pair ? 64 : std::min(64, c.tile));
        if (r.b[k]) j.b[k] = map_of(r.b[k], r.b_mn || !pair ? 64 : std::min(64, c.tile / 2));
      }
      tiles += (int64_t)j.tiles_m * j.tiles_n * j.split;
      steps += (int64_t)j.tiles_m * j.tiles_n * r.shape.k_tiles();
    }
    for (int i = 0; i < 2; ++i) {
      LinearKept& k = out.kept[i];
      if (!k.data) continue;
      k.vec = out.keep == 2 ? rows_at(k.data, k.ld, 1, 16) : tma_writes(k.data, k.ld, list[0].shape.N, 2);
      out.kept_vec8[i] = rows_at(k.data, k.ld, 2, 8);
      if (pair && out.keep == 1 && k.vec && *e == cudaSuccess)
        *e = encode_linear_out_map(k.data, list[0].shape.N / 8 * 8, list[0].shape.M, k.ld, true, linear_pair_box(c.tile, gated, fold), &maps.kept[i]);
    }
    if (*e != cudaSuccess) return SGEMM_OK;
    if (pair) {
      const int64_t clusters = std::min<int64_t>(tiles, dev.pair_clusters);
      if (tiles > INT_MAX || steps / clusters > INT_MAX / 2) return SGEMM_ERR_UNSUPPORTED;
      p.out = out;
      if (joins && count == 1) {  // the epilogue is the joining kernel's
        p.out.bias = p.out.residual = nullptr;
        p.out.act = p.out.keep = 0;
      }
      p.jobs = count;
      p.clusters = (int)clusters;
      p.timeout_ns = wait_timeout_ns();
      p.fault = dev.fault;
      *e = launch_linear_pair(c.tile, gated, joins ? LinearPairForm::kShared : fold ? LinearPairForm::kFold : LinearPairForm::kWhole, maps, p, stream);
      if (joins && *e == cudaSuccess) {
        join.out = out;
        *e = launch_linear_join(join, stream);
      }
      return SGEMM_OK;
    }
    LinearShortParams q;
    q.out = out;
    q.job = p.job[0];
    q.tile_s = c.tile;
    q.split = c.split;
    q.stages = short_stages(c.tile, gated, list[0].a_mn != 0);
    q.stage_bytes = (int)short_stage(c.tile, gated, list[0].a_mn != 0);
    q.timeout_ns = wait_timeout_ns();
    q.fault = dev.fault;
    if (tiles * c.split > INT_MAX) return SGEMM_ERR_UNSUPPORTED;
    *e = launch_linear_short(gated, maps, q, stream);
    return SGEMM_OK;
  }

  static bool tma_writes(const void* p, int64_t ld, int64_t cols, int size) { return rows_at(p, ld, size, 16) && cols * size >= 16; }
};

// What is kept, as the kernels take it: 0 nothing, 1 BF16, 2 8-bit.
int keep_of(const sgemm_kept_t* k, LinearKept* out) {
  if (!k) return 0;
  out->data = k->data;
  out->ld = k->ld;
  out->scale = k->scale;
  out->lds = k->lds;
  return k->scale ? 2 : 1;
}
LinearKeptIn kept_in(const sgemm_kept_t* k) {
  LinearKeptIn m;
  if (!k) return m;
  m.data = k->data;
  m.ld = k->ld;
  m.scale = k->scale;
  m.lds = k->lds;
  m.vec = k->scale ? rows_at(k->data, k->ld, 1, 8) : rows_at(k->data, k->ld, 2, 16);
  return m;
}

int no_memory(cudaError_t e) {
  record_cuda_failure(e);
  return e == cudaErrorMemoryAllocation ? SGEMM_ERR_NOMEM : SGEMM_ERR_CUDA;
}
int launch_status(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : record_cuda_failure(e); }

// Allocates the workspace that `place` lays out, runs `work` (a status; CUDA's error in its argument) and frees it.
template <typename Place, typename Work>
int with_workspace(const CallDevice& dev, cudaStream_t stream, const Place& place, const Work& work) {
  Pieces w;
  place(&w);
  void* ws = nullptr;
  if (w.at > 0) {
    const cudaError_t e = cudaMallocFromPoolAsync(&ws, (size_t)w.at, dev.pool, stream);
    if (e != cudaSuccess) return no_memory(e);
    w = Pieces{static_cast<uint8_t*>(ws), 0};
    place(&w);
  }
  cudaError_t e = cudaSuccess;
  const int s = work(&e);
  if (ws) {
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = ef;
  }
  return s != SGEMM_OK ? s : launch_status(e);
}

cudaError_t zero_rows(void* p, int64_t ld, int64_t rows, int64_t cols, int size, cudaStream_t stream) {
  return cudaMemset2DAsync(p, (size_t)ld * size, 0, (size_t)cols * size, (size_t)rows, stream);
}

bool too_large(std::initializer_list<int64_t> v) {
  return std::any_of(v.begin(), v.end(), [](int64_t x) { return x > kMaxDim; });
}

// The forward products: X (W0, gated: W1)^T with their epilogue.
int forward(int64_t tokens, int64_t inputs, int64_t outputs, const void* X, int64_t ldx, const void* W0, int64_t ldw0, const void* W1,
            int64_t ldw1, Launch& launch, cudaStream_t stream) {
  Product& pr = launch.pr[0];
  CallDevice dev;
  const int s = linear_device(&dev);
  if (s != SGEMM_OK) return s;
  const bool gated = pr.shape.gated;
  const bool empty = inputs == 0;  // a sum of nothing: 8 zeros per row instead
  const int64_t K = empty ? 8 : inputs;
  void* zeros = nullptr;
  Operand x(X, ldx, nullptr, 0, tokens, K), w0(W0, ldw0, nullptr, 0, outputs, K), w1(W1, ldw1, nullptr, 0, outputs, K);
  if (empty) x.copied = w0.copied = w1.copied = false;
  pr.shape.M = tokens;
  pr.shape.N = outputs;
  pr.shape.K = K;
  pr.shape.kept8 = launch.out.keep == 2;
  pr.a[0] = &x;
  pr.b[0] = &w0;
  if (gated) pr.b[1] = &w1;
  // the pair kernel's lanes read a row of the residual each, 16 bytes at a time; rows that lie anywhere are copied first
  // (reading them along the rows in its epilogue took longer than the copy and the epilogue together)
  launch.plan(dev);
  LinearOut& out = launch.out;
  Operand r(out.residual, out.ldr, nullptr, 0, tokens, outputs);
  r.copied = out.residual && launch.by_pairs() && !launch.shares_k() && !rows_at(out.residual, out.ldr, 2, 16);
  return with_workspace(
      dev, stream,
      [&](Pieces* w) {
        if (empty) zeros = w->take<uint16_t>(8 * std::max(tokens, outputs));
        x.place(w);
        w0.place(w);
        if (gated) w1.place(w);
        r.place(w);
        launch.place(w);
      },
      [&](cudaError_t* e) {
        const Guard g{dev.fault, dev.bounds};
        if (empty) {
          for (Operand* o : {&x, &w0, &w1}) o->m.data = zeros, o->m.ld = 8;
          *e = cudaMemsetAsync(zeros, 0, (size_t)std::max(tokens, outputs) * 16, stream);
        }
        if (*e == cudaSuccess) *e = make_copies({&x, &w0, gated ? &w1 : nullptr, &r}, g, stream);
        if (r.copied) out.residual = r.copy, out.ldr = whole_lines(outputs);
        return *e == cudaSuccess ? launch.run(dev, stream, e) : SGEMM_OK;
      });
}

// tokens x inputs over the outputs (twice them with two gradients and weights).
Product input_gradient(int64_t tokens, int64_t inputs, int64_t outputs, const Operand* d0, const Operand* d1, const Operand* w0, const Operand* w1,
                       void* dX, int64_t lddx) {
  Product r;
  r.shape.M = tokens;
  r.shape.N = inputs;
  r.shape.K = outputs;
  r.shape.segments = d1 ? 2 : 1;
  r.a[0] = d0;
  r.a[1] = d1;
  r.b[0] = w0;
  r.b[1] = w1;
  r.b_mn = 1;
  r.d = dX;
  r.ldd = lddx;
  return r;
}
// outputs x inputs over the tokens.
Product weight_gradient(int64_t tokens, int64_t inputs, int64_t outputs, const Operand* d, const Operand* x, void* dW, int64_t lddw, int type) {
  Product r;
  r.shape.M = outputs;
  r.shape.N = inputs;
  r.shape.K = tokens;
  r.a[0] = d;
  r.b[0] = x;
  r.a_mn = r.b_mn = 1;
  r.d = dW;
  r.ldd = lddw;
  r.f32 = type == SGEMM_F32;
  return r;
}

}  // namespace

extern "C" {

int sgemm_linear(int64_t tokens, int64_t inputs, int64_t outputs, const void* X, int64_t ldx, const void* W, int64_t ldw, const void* bias,
                 int activation, const void* R, int64_t ldr, const sgemm_kept_t* kept, void* Y, int64_t ldy, int type,
                 struct CUstream_st* stream) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool work = tokens > 0 && outputs > 0, read = work && inputs > 0;
  if (!usable(X, 2, read)) return -4;
  if (!wide_enough(ldx, inputs)) return -5;
  if (!usable(W, 2, read)) return -6;
  if (!wide_enough(ldw, inputs)) return -7;
  if (!usable(bias, 2, work && bias)) return -8;
  if (!known_act(activation)) return -9;
  if (!usable(R, 2, work && R)) return -10;
  if (R && !wide_enough(ldr, outputs)) return -11;
  if (!usable_kept(kept, outputs, work)) return -12;
  if (!known_type(type)) return -15;
  if (!usable(Y, type_size(type), work) || (work && Y == R && type != SGEMM_BF16)) return -13;
  if (!wide_enough(ldy, outputs) || (work && Y == R && tokens > 1 && ldy != ldr)) return -14;
  if (!work) return SGEMM_OK;
  if (too_large({tokens, inputs, outputs, ldx, ldw, ldy, R ? ldr : 0, kept ? kept->ld : 0})) return SGEMM_ERR_UNSUPPORTED;
  Launch launch;
  Product& pr = launch.add();
  pr.d = Y;
  pr.ldd = ldy;
  pr.f32 = type == SGEMM_F32;
  LinearOut& o = launch.out;
  o.bias = bias;
  o.residual = R;
  o.ldr = ldr;
  o.act = activation;
  o.keep = keep_of(kept, &o.kept[0]);
  return forward(tokens, inputs, outputs, X, ldx, W, ldw, nullptr, 0, launch, reinterpret_cast<cudaStream_t>(stream));
}

int sgemm_gated(int64_t tokens, int64_t inputs, int64_t outputs, const void* X, int64_t ldx, const void* gate, int64_t ldg, const void* up,
                int64_t ldu, int activation, const sgemm_kept_t* kept_gate, const sgemm_kept_t* kept_up, void* H, int64_t ldh,
                struct CUstream_st* stream) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool work = tokens > 0 && outputs > 0, read = work && inputs > 0;
  if (!usable(X, 2, read)) return -4;
  if (!wide_enough(ldx, inputs)) return -5;
  if (!usable(gate, 2, read)) return -6;
  if (!wide_enough(ldg, inputs)) return -7;
  if (!usable(up, 2, read)) return -8;
  if (!wide_enough(ldu, inputs)) return -9;
  if (!known_act(activation)) return -10;
  if (!usable_kept(kept_gate, outputs, work)) return -11;
  if (!usable_kept(kept_up, outputs, work) || !kept_gate != !kept_up || (kept_up && !kept_gate->scale != !kept_up->scale)) return -12;
  if (!usable(H, 2, work)) return -13;
  if (!wide_enough(ldh, outputs)) return -14;
  if (!work) return SGEMM_OK;
  if (too_large({tokens, inputs, outputs, ldx, ldg, ldu, ldh, kept_gate ? kept_gate->ld : 0, kept_up ? kept_up->ld : 0})) return SGEMM_ERR_UNSUPPORTED;
  Launch launch;
  Product& pr = launch.add();
  pr.shape.gated = true;
  pr.d = H;
  pr.ldd = ldh;
  LinearOut& o = launch.out;
  o.act = activation;
  o.keep = keep_of(kept_gate, &o.kept[0]);
  keep_of(kept_up, &o.kept[1]);
  return forward(tokens, inputs, outputs, X, ldx, gate, ldg, up, ldu, launch, reinterpret_cast<cudaStream_t>(stream));
}

int sgemm_linear_backward(int64_t tokens, int64_t inputs, int64_t outputs, const void* dY, int64_t lddy, const sgemm_kept_t* X,
                          const void* W, int64_t ldw, int activation, const sgemm_kept_t* kept, void* dX, int64_t lddx, void* dW,
                          int64_t lddw, int dw_type, float* dbias, struct CUstream_st* stream_) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool read = tokens > 0 && outputs > 0, work = read && inputs > 0;
  if (!known_type(dw_type)) return -15;
  if (!known_act(activation)) return -9;
  if (!usable(dY, 2, read && (dX || dW || dbias))) return -4;
  if (!wide_enough(lddy, outputs)) return -5;
  if (dW && (!X || !usable_kept(X, inputs, work))) return -6;
  if (dX && !usable(W, 2, work)) return -7;
  if (dX && !wide_enough(ldw, inputs)) return -8;
  if (activation != SGEMM_ACT_NONE && (!kept || !usable_kept(kept, outputs, read))) return -10;
  if (!usable(dX, 2, dX != nullptr)) return -11;
  if (dX && !wide_enough(lddx, inputs)) return -12;
  if (!usable(dW, type_size(dw_type), dW != nullptr)) return -13;
  if (dW && !wide_enough(lddw, inputs)) return -14;
  if (!usable(dbias, 4, dbias != nullptr)) return -16;
  if (too_large({tokens, inputs, outputs, lddy, dX ? ldw : 0, dX ? lddx : 0, dW ? lddw : 0, dW ? X->ld : 0, activation != SGEMM_ACT_NONE ? kept->ld : 0}))
    return SGEMM_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (tokens == 0 || inputs == 0 || outputs == 0) {  // nothing, or sums of nothing
    if (tokens == 0) {
      cudaError_t e = cudaSuccess;
      if (dW && inputs > 0 && outputs > 0) e = zero_rows(dW, lddw, outputs, inputs, type_size(dw_type), stream);
      if (e == cudaSuccess && dbias && outputs > 0) e = cudaMemsetAsync(dbias, 0, (size_t)outputs * 4, stream);
      return launch_status(e);
    }
    if (outputs == 0) return dX && inputs > 0 ? launch_status(zero_rows(dX, lddx, tokens, inputs, 2, stream)) : SGEMM_OK;
    dX = dW = nullptr;  // (no inputs: dbias alone)
  }
  if (!dX && !dW && !dbias) return SGEMM_OK;
  CallDevice dev;
  const int s = linear_device(&dev);
  if (s != SGEMM_OK) return s;
  const bool act = activation != SGEMM_ACT_NONE, products = dX || dW;
  LinearGradParams g;
  g.rows = tokens;
  g.cols = (int)outputs;
  g.dy = dY;
  g.lddy = lddy;
  if (act) g.a = kept_in(kept);
  g.act = activation;
  g.dbias = dbias;
  g.guard = {dev.fault, dev.bounds};
  shape_linear_grad(&g, dev.pair_clusters > 0, dev.sm_count);
  g.vec = rows_at(dY, lddy, 2, 16) && (!act || g.a.vec);
  // dA: dY itself where it can be read as it is and there is no activation
  Operand d(dY, lddy, nullptr, 0, tokens, outputs);
  const bool write = products && (act || d.copied);
  Operand w(W, ldw, nullptr, 0, outputs, inputs);
  Operand x(X ? X->data : nullptr, X ? X->ld : 1, X ? X->scale : nullptr, X ? X->lds : 1, tokens, inputs);
  const int64_t ldd = whole_lines(outputs);
  Launch launch;
  if (dX) launch.add() = input_gradient(tokens, inputs, outputs, &d, nullptr, &w, nullptr, dX, lddx);
  if (dW) launch.add() = weight_gradient(tokens, inputs, outputs, &d, &x, dW, lddw, dw_type);
  if (launch.n) launch.plan(dev);
  return with_workspace(
      dev, stream,
      [&](Pieces* p) {
        g.da = write ? p->take<uint16_t>(tokens * ldd) : nullptr;
        g.partial = dbias && !g.joined ? p->take<float>((int64_t)g.row_blocks * outputs) : nullptr;
        if (dX) w.place(p);
        if (dW) x.place(p);
        launch.place(p);
      },
      [&](cudaError_t* e) {
        g.ldd = ldd;
        if (write || dbias) *e = launch_linear_grad(g, stream);
        if (*e == cudaSuccess) *e = make_copies({dX ? &w : nullptr, dW ? &x : nullptr}, g.guard, stream);
        if (*e != cudaSuccess) return (int)SGEMM_OK;
        if (write) d = Operand(g.da, ldd, nullptr, 0, tokens, outputs);
        return launch.n ? launch.run(dev, stream, e) : (int)SGEMM_OK;
      });
}

int sgemm_gated_backward(int64_t tokens, int64_t inputs, int64_t outputs, const void* dH, int64_t lddh, const sgemm_kept_t* X,
                         const void* gate, int64_t ldg, const void* up, int64_t ldu, int activation, const sgemm_kept_t* kept_gate,
                         const sgemm_kept_t* kept_up, void* dX, int64_t lddx, void* dG, int64_t lddg, void* dU, int64_t lddu, int dw_type,
                         void* H, int64_t ldh, struct CUstream_st* stream_) {
  if (tokens < 0) return -1;
  if (inputs < 0) return -2;
  if (outputs < 0) return -3;
  const bool read = tokens > 0 && outputs > 0, work = read && inputs > 0;
  if (!usable(dH, 2, read && (dX || dG || dU || H))) return -4;
  if (!wide_enough(lddh, outputs)) return -5;
  if (dG && (!X || !usable_kept(X, inputs, work))) return -6;
  if (dX && !usable(gate, 2, work)) return -7;
  if (dX && !wide_enough(ldg, inputs)) return -8;
  if (dX && !usable(up, 2, work)) return -9;
  if (dX && !wide_enough(ldu, inputs)) return -10;
  if (!known_act(activation)) return -11;
  if (!kept_gate || !usable_kept(kept_gate, outputs, read)) return -12;
  if (!kept_up || !usable_kept(kept_up, outputs, read) || !kept_gate->scale != !kept_up->scale) return -13;
  if (!usable(dX, 2, dX != nullptr)) return -14;
  if (dX && !wide_enough(lddx, inputs)) return -15;
  if (!known_type(dw_type)) return -20;
  if (!usable(dG, type_size(dw_type), dG != nullptr)) return -16;
  if (dG && !wide_enough(lddg, inputs)) return -17;
  if (!usable(dU, type_size(dw_type), dU != nullptr) || !dG != !dU) return -18;
  if (dU && !wide_enough(lddu, inputs)) return -19;
  if (!usable(H, 2, H != nullptr)) return -21;
  if (H && !wide_enough(ldh, outputs)) return -22;
  if (too_large({tokens, inputs, outputs, lddh, dX ? ldg : 0, dX ? ldu : 0, dX ? lddx : 0, dG ? lddg : 0, dU ? lddu : 0, H ? ldh : 0, dG ? X->ld : 0,
                 kept_gate->ld, kept_up->ld}))
    return SGEMM_ERR_UNSUPPORTED;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (tokens == 0 || inputs == 0 || outputs == 0) {  // nothing, or sums of nothing
    if (tokens == 0) {
      cudaError_t e = cudaSuccess;
      if (dG && inputs > 0 && outputs > 0) e = zero_rows(dG, lddg, outputs, inputs, type_size(dw_type), stream);
      if (dG && inputs > 0 && outputs > 0 && e == cudaSuccess) e = zero_rows(dU, lddu, outputs, inputs, type_size(dw_type), stream);
      return launch_status(e);
    }
    if (outputs == 0) return dX && inputs > 0 ? launch_status(zero_rows(dX, lddx, tokens, inputs, 2, stream)) : SGEMM_OK;
    dX = dG = dU = nullptr;  // (no inputs: H alone)
  }
  if (!dX && !dG && !H) return SGEMM_OK;
  CallDevice dev;
  const int s = linear_device(&dev);
  if (s != SGEMM_OK) return s;
  LinearGradParams g;
  g.rows = tokens;
  g.cols = (int)outputs;
  g.dy = dH;
  g.lddy = lddh;
  g.a = kept_in(kept_gate);
  g.b = kept_in(kept_up);
  g.act = activation;
  g.h = H;
  g.ldh = ldh;
  g.guard = {dev.fault, dev.bounds};
  shape_linear_grad(&g, dev.pair_clusters > 0, dev.sm_count);
  g.vec = rows_at(dH, lddh, 2, 16) && g.a.vec && g.b.vec && (!H || rows_at(H, ldh, 2, 16));
  Operand wg(gate, ldg, nullptr, 0, outputs, inputs), wu(up, ldu, nullptr, 0, outputs, inputs);
  Operand x(X ? X->data : nullptr, X ? X->ld : 1, X ? X->scale : nullptr, X ? X->lds : 1, tokens, inputs);
  const int64_t ldd = whole_lines(outputs);
  Operand da, db;
  Launch launch;
  if (dX) launch.add() = input_gradient(tokens, inputs, outputs, &da, &db, &wg, &wu, dX, lddx);
  if (dG) launch.add() = weight_gradient(tokens, inputs, outputs, &da, &x, dG, lddg, dw_type);
  if (dG) launch.add() = weight_gradient(tokens, inputs, outputs, &db, &x, dU, lddu, dw_type);
  if (launch.n) launch.plan(dev);
  return with_workspace(
      dev, stream,
      [&](Pieces* p) {
        g.da = dX || dG ? p->take<uint16_t>(tokens * ldd) : nullptr;
        g.db = dX || dG ? p->take<uint16_t>(tokens * ldd) : nullptr;
        if (dX) {
          wg.place(p);
          wu.place(p);
        }
        if (dG) x.place(p);
        launch.place(p);
      },
      [&](cudaError_t* e) {
        g.ldd = ldd;
        *e = launch_linear_grad(g, stream);
        if (*e == cudaSuccess) *e = make_copies({dX ? &wg : nullptr, dX ? &wu : nullptr, dG ? &x : nullptr}, g.guard, stream);
        if (*e != cudaSuccess) return (int)SGEMM_OK;
        da = Operand(g.da, ldd, nullptr, 0, tokens, outputs);
        db = Operand(g.db, ldd, nullptr, 0, tokens, outputs);
        return launch.n ? launch.run(dev, stream, e) : (int)SGEMM_OK;
      });
}

int sgemm_linear_plan(int64_t rows, int64_t cols, int64_t K, int gated, int kept8, int sm_count, sgemm_plan_t* plan) {
  if (rows < 1) return -1;
  if (cols < 1) return -2;
  if (K < 1) return -3;
  if (!plan) return -7;
  if (too_large({rows, cols, K})) return SGEMM_ERR_UNSUPPORTED;
  CallDevice dev;
  dev.sm_count = sm_count;
  dev.pair_clusters = -1;
  if (sm_count <= 0) {
    const int s = linear_device(&dev);
    if (s != SGEMM_OK) return s;
  }
  Shape s;
  s.M = rows;
  s.N = cols;
  s.K = K;
  s.gated = gated != 0;
  s.kept8 = kept8 != 0;
  const Choice c = choose(&s, 1, dev.sm_count, dev.pair_clusters);
  if (c.variant == 0) return SGEMM_ERR_UNSUPPORTED;
  const bool pair = c.variant == SGEMM_VARIANT_LINEAR_PAIR;
  *plan = sgemm_plan_t{};
  plan->variant = c.variant;
  plan->tile_m = pair ? 256 : 128;
  plan->tile_n = c.tile;
  plan->tile_k = 64;
  plan->stages = pair ? linear_pair_stages(c.tile) : short_stages(c.tile, s.gated, false);
  plan->threads = pair ? kLinearPairThreads : kLinearShortThreads;
  plan->split_k = pair ? c.splits[0] : c.split;
  plan->kernel_launches = plan->split_k > 1 && pair ? 2 : 1;
  plan->dp_tiles = pair ? s.pair_tiles(c.tile) : ceil_div(cols, 128) * ceil_div(rows, c.tile);
  const int64_t clusters = dev.pair_clusters >= 0 ? dev.pair_clusters : std::max(1, dev.sm_count / 2);
  plan->grid_x = pair ? 2 * std::min(plan->dp_tiles * plan->split_k, clusters) : plan->dp_tiles * c.split;
  plan->workspace_bytes = pair && plan->split_k > 1 ? round256(4 * plan->split_k * Launch::rows_apart(s) * Launch::sums_ld(s)) : 0;
  plan->grid_y = 1;
  plan->smem_bytes = pair ? linear_pair_smem(c.tile) : linear_short_smem(c.tile, s.gated, plan->stages, (int)short_stage(c.tile, s.gated, false));
  return SGEMM_OK;
}

int sgemm_linear_set_override(int variant, int tile_n, int split) {
  if (variant != SGEMM_VARIANT_AUTO && variant != SGEMM_VARIANT_LINEAR_PAIR && variant != SGEMM_VARIANT_LINEAR_SHORT) return -1;
  const bool is_short = variant == SGEMM_VARIANT_LINEAR_SHORT;
  const auto is_in = [&](const auto& tiles) { return std::find(std::begin(tiles), std::end(tiles), tile_n) != std::end(tiles); };
  const bool known = is_short ? is_in(kLinearShortTiles) : variant == SGEMM_VARIANT_LINEAR_PAIR && is_in(kLinearPairTiles);
  if (tile_n != 0 && !known) return -2;
  if (variant == SGEMM_VARIANT_AUTO ? split != 0 : is_short ? split != 0 && split != 1 && split != 2 && split != 4 && split != 8 : split < 0 || split > kLinearMostShares)
    return -3;
  g_force_variant.store(variant);
  g_force_tile.store(tile_n);
  g_force_split.store(split);
  return SGEMM_OK;
}

}  // extern "C"
