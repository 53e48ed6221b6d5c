// Entry points of the layers in front of the head (include/cce_layers.h and include/cce_layers_ex.h):
// argument checks, workspace layout, the choice of tiles, launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/cce_layers_ex.h"
#include "internal.h"
#include "linear.h"

namespace cce {
namespace {

constexpr int64_t LIMIT = (int64_t(1) << 31) - 512;
constexpr int64_t WIDTH = int64_t(1) << 30;   // of a row
constexpr int64_t MATRIX = int64_t(1) << 45;  // elements of one

constexpr size_t NO_WORKSPACE = 16;           // what the queries give where none is needed

bool multiple(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(bytes) == 0; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t type_bytes(int t) { return t == CCE_F32 ? 4 : 2; }
bool type_ok(int t) { return t == CCE_F32 || t == CCE_F16 || t == CCE_BF16; }
bool operand_type(int t) { return t == CCE_F16 || t == CCE_BF16; }
// How pre-activations are kept.
bool kept_type(int z, int type) { return z == type || (z == CCE_KEPT16 && type == CCE_BF16); }
bool act_ok(int act) { return act >= CCE_ACT_NONE && act <= CCE_ACT_SILU; }
bool sizes_ok(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && M < LIMIT && N >= 1 && N < WIDTH && K >= 1 && K < WIDTH && M * N < MATRIX && M * K < MATRIX &&
         N * K < MATRIX;
}
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// ----------------------------------------------------------------- tiles
// What decides over the tiles of a product: sizes alone, so that a workspace can be
// sized without a device.
struct Shape {
  int I, J;
  int K, parts;  // `parts` sums of K
  bool b_mn;     // B comes in groups of 64 j
};
struct Choice {
  int jt, splits, kb_split;
  int64_t items;
  double item_cycles;
};
struct Plan {
  bool pair;
  Choice c[LIN_MAX_PROBLEMS];
  double cycles;
};

constexpr int UNITS = LIN_SMS;
constexpr int64_t MAX_PART_BYTES = 256ll << 20;  // of a product's partial sums

int64_t i_tiles(const Shape& s, bool pair, bool gated) { return cdiv(s.I, (pair ? 2 : 1) * (gated ? LIN_BI / 2 : LIN_BI)); }
int k_blocks(const Shape& s, bool pair) { return static_cast<int>(s.parts * cdiv(s.K, lin_bk(pair))); }

// Cycles of one work item: its blocks of K at the slower of the tensor core (8,192
// flops a cycle and SM) and the loads (56 bytes a cycle and SM from L2), and what a
// tile costs beside them.  (Measured: 16,384 x 2,048 x 4,096 takes 152 us as pairs with 256
// columns, 159 with 224, 215 with 128, and 184 as single CTAs with 256; 64 x 4,096 x
// 4,096 18.5 us in one piece and 11.0 with K in four; dW of 4,096 x 896 x 896 18.9 and 14.0.)
double item_cycles(int jt, int kb, bool pair, bool b_mn) {
  const double mma = 2.0 * jt;
  const double load = (LIN_BI + lin_b_rows(jt, pair, b_mn)) * 128.0 / 56.0;
  return kb * std::max(mma, load) * (lin_bk(pair) / 64) + 500.0;
}

// The longest of the units' shares: unit u takes items u, u + units, ... of the
// problems one after another.
double makespan(const Choice* c, int n, int units) {
  int64_t ends[LIN_MAX_PROBLEMS], at = 0;
  for (int q = 0; q < n; ++q) ends[q] = at += c[q].items;
  const auto count = [&](int64_t end, int64_t u) { return end > u ? (end - u - 1) / units + 1 : 0; };
  double worst = 0.0;
  const auto share = [&](int64_t u) {
    double t = 0.0;
    int64_t before = 0;
    for (int q = 0; q < n; ++q) {
      const int64_t to = count(ends[q], u);
      t += static_cast<double>(to - before) * c[q].item_cycles;
      before = to;
    }
    worst = std::max(worst, t);
  };
  share(0);
  for (int q = 0; q < n; ++q) share(ends[q] % units);  // a count changes at these units only
  return worst;
}

double join_cycles(const Shape& s, const Choice& c, bool gated) {
  if (c.splits == 1) return 0.0;
  return 4000.0 + (c.splits * (gated ? 2.0 : 1.0) + 1.0) * s.I * s.J * 4.0 / 2500.0;
}

// Tries the widths and splits of problem q with the others as they are.
void choose(const Shape* s, int n, int q, bool pair, bool gated, Plan* best) {
  const int units = pair ? UNITS / 2 : UNITS;
  const int mats = gated ? 2 : 1;
  const int kb = k_blocks(s[q], pair);
  constexpr int step = 32;
  Plan p = *best;
  for (int jt = step; jt <= 256; jt += step) {
    if (jt > step && jt - step >= s[q].J) break;  // a narrower one holds all rows
    const int64_t tiles = i_tiles(s[q], pair, gated) * cdiv(s[q].J, jt);
    for (int splits = 1; splits <= std::min(kb, 64); splits = splits < 8 ? splits + 1 : splits + 4) {
      if (splits > 1 && (tiles * (splits - 1) > 2 * units ||
                         int64_t(splits) * mats * s[q].I * s[q].J * 4 > MAX_PART_BYTES))
        break;
      Choice& c = p.c[q];
      c.jt = jt;
      c.kb_split = static_cast<int>(cdiv(kb, splits));
      c.splits = static_cast<int>(cdiv(kb, c.kb_split));
      if (c.splits != splits) continue;  // the same as fewer splits
      c.items = tiles * splits;
      c.item_cycles = item_cycles(jt, c.kb_split, pair, s[q].b_mn);
      p.cycles = makespan(p.c, n, units);
      for (int r = 0; r < n; ++r) p.cycles += join_cycles(s[r], p.c[r], gated);
      if (best->cycles < 0.0 || p.cycles < best->cycles) *best = p;
    }
  }
}

Plan plan_tiles(const Shape* s, int n, bool gated) {
  Plan best{};
  best.cycles = -1.0;
  for (const bool pair : {true, false}) {
    Plan p{};
    p.pair = pair;
    p.cycles = -1.0;
    for (int q = 0; q < n; ++q) {  // each alone, then each with the others
      Plan one{};
      one.pair = pair;
      one.cycles = -1.0;
      choose(s + q, 1, 0, pair, gated, &one);
      p.c[q] = one.c[0];
    }
    for (int q = 0; q < n; ++q) {
      p.cycles = -1.0;
      choose(s, n, q, pair, gated, &p);
    }
    if (best.cycles < 0.0 || p.cycles < best.cycles) best = p;
  }
  return best;
}

// Plans are functions of sizes alone, and searching one takes up to some 20 us: the last ones are kept, for all threads.  A set
// has room for sixteen, so that a model's layers, a few hundred plans, do not push each other out.
class Plans {
 public:
  Plan of(const Shape* s, int n, bool gated) {
    uint64_t h = static_cast<uint64_t>(n * 2 + gated);
    for (int q = 0; q < n; ++q) {
      for (const int v : {s[q].I, s[q].J, s[q].K, s[q].parts, static_cast<int>(s[q].b_mn)})
        h = (h ^ static_cast<uint64_t>(v)) * 0x9e3779b97f4a7c15ull;
    }
    Set& set = sets_[h >> 58];
    {
      const std::lock_guard<std::mutex> lock(mutex_);
      for (int w = 0; w < WAYS; ++w) {
        if (set.hash[w] == h && same(set.kept[w], s, n, gated)) return set.kept[w].plan;
      }
    }
    ++searches_;
    Planned made;
    std::copy(s, s + n, made.s);
    made.n = n;
    made.gated = gated;
    made.plan = plan_tiles(s, n, gated);
    const std::lock_guard<std::mutex> lock(mutex_);
    set.hash[set.oldest] = h;
    set.kept[set.oldest] = made;
    set.oldest = (set.oldest + 1) % WAYS;
    return made.plan;
  }
  uint64_t searches() const { return searches_; }

 private:
  static constexpr int WAYS = 16;
  struct Planned {
    Shape s[LIN_MAX_PROBLEMS];
    int n;  // 0: none
    bool gated;
    Plan plan;
  };
  struct Set {
    uint64_t hash[WAYS];
    Planned kept[WAYS];
    int oldest;
  };
  static bool same(const Planned& k, const Shape* s, int n, bool gated) {
    if (k.n != n || k.gated != gated) return false;
    for (int q = 0; q < n; ++q) {
      const Shape &a = k.s[q], &b = s[q];
      if (a.I != b.I || a.J != b.J || a.K != b.K || a.parts != b.parts || a.b_mn != b.b_mn) return false;
    }
    return true;
  }

  std::mutex mutex_;
  std::atomic<uint64_t> searches_{0};
  Set sets_[64] = {};
};

Plans g_plans;

Plan plan_of(const Shape* s, int n, bool gated) { return g_plans.of(s, n, gated); }

size_t part_bytes(const Shape& s, const Choice& c, bool gated) {
  return c.splits == 1 ? 0 : round256(size_t(4) * c.splits * (gated ? 2 : 1) * s.I * s.J);
}

size_t parts_bytes(const Shape* s, int n, bool gated) {
  const Plan p = plan_of(s, n, gated);
  size_t b = 0;
  for (int q = 0; q < n; ++q) b += part_bytes(s[q], p.c[q], gated);
  return b;
}

// ---------------------------------------------------------------- products
struct Device {
  int sms = 0, pairs = 0;
  int32_t* error = nullptr;

  cce_status ready() { return static_cast<cce_status>(layers_device_ready(&sms, &pairs, &error)); }
};

struct Operand {
  const void* p;
  int64_t pitch;
};

// One product: out[J][I] over `parts` pairs of operands.
struct Product {
  Shape s;
  Operand a[2], b[2];  // gated: both weights, and x
  bool a_mn;
  LinEpilogue e;
};

Shape shape_of(int64_t I, int64_t J, int64_t K, int parts, bool b_mn) {
  return Shape{static_cast<int>(I), static_cast<int>(J), static_cast<int>(K), parts, b_mn};
}

// The map of an operand with `rows` of its own index in a tile: boxes of 64 contiguous
// elements, in 3 dimensions all of a stage's.
bool encode(CUtensorMap* m, bool bf16, const Operand& o, int K, int own, bool mn, bool whole, uint32_t bk, int rows) {
  const uint64_t inner = mn ? own : K, outer = mn ? K : own;
  const uint32_t box_rows = mn ? bk : static_cast<uint32_t>(rows), groups = (mn ? rows : static_cast<int>(bk)) / 64;
  return whole ? encode_groups(m, bf16, o.p, inner, outer, o.pitch, box_rows, groups)
               : encode_operand(m, bf16, o.p, inner, outer, o.pitch, 64, box_rows);
}

// The products in one launch (at least one, with a sum of parts beside them), and the joins of those whose K is split.  `part`:
// room for their partial sums.
cce_status run_products(const Product* in, int n, bool gated, bool bf16, const LinSum& sum, void* part, const Device& on,
                        cudaStream_t s, int* launches) {
  Shape shapes[LIN_MAX_PROBLEMS];
  for (int q = 0; q < n; ++q) shapes[q] = in[q].s;
  const Plan plan = plan_of(shapes, n, gated);
  if (plan.pair && on.pairs < 1) return CCE_ERR_CUDA;
  // the tensor maps are made by the driver, which wants this thread to have a context
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess || cudaSetDevice(device) != cudaSuccess) return CCE_ERR_CUDA;
  const uint32_t bk = static_cast<uint32_t>(lin_bk(plan.pair));
  LinArgs a{};
  a.problems = n;
  a.bf16 = bf16;
  a.error = on.error;
  a.sum = sum;
  char* at = static_cast<char*>(part);
  int64_t items = 0;
  int widest = 0;
  for (int q = 0; q < n; ++q) {
    const Product& f = in[q];
    const Choice& c = plan.c[q];
    const int parts = f.s.parts;
    LinProblem& p = a.p[q];
    p.I = f.s.I;
    p.J = f.s.J;
    p.klen[0] = f.s.K;
    p.klen[1] = parts > 1 ? f.s.K : 0;
    p.kb_first = static_cast<int>(cdiv(f.s.K, bk));
    p.kb_all = k_blocks(f.s, plan.pair);
    p.a_mn = f.a_mn;
    p.b_mn = f.s.b_mn;
    // a third dimension of groups of 64 would reach past the row's end otherwise
    p.a_3d = !gated && (f.a_mn ? p.I : f.s.K) % 64 == 0;
    const int own_rows = plan.pair ? c.jt / 2 : c.jt, b_rows = lin_b_rows(c.jt, plan.pair, f.s.b_mn);
    p.b_3d = f.s.b_mn ? p.J % 64 == 0 && own_rows % 64 == 0 : f.s.K % 64 == 0;
    p.jt = c.jt;
    p.i_tiles = static_cast<int>(i_tiles(f.s, plan.pair, gated));
    p.j_tiles = static_cast<int>(cdiv(f.s.J, c.jt));
    p.splits = c.splits;
    p.kb_split = c.kb_split;
    p.group = std::min(p.i_tiles, 8);
    if (c.items >= LIMIT) return CCE_ERR_SHAPE;
    p.items = static_cast<int>(c.items);
    items += c.items;
    p.part = reinterpret_cast<float*>(at);
    at += part_bytes(f.s, c, gated);
    p.e = f.e;
    const bool rows_16 = f.e.y_type != CCE_F32 && multiple(f.e.y, 16) && f.e.y_pitch % 8 == 0;
    const bool z_16 = !f.e.z[0] || (multiple(f.e.z[0], 16) && multiple(f.e.z[1], 16) && f.e.z_pitch % 8 == 0);
    p.wide = c.splits == 1 && rows_16 && z_16 && p.I % 8 == 0;
    widest = std::max(widest, b_rows);
    if (gated) {
      const uintptr_t g = reinterpret_cast<uintptr_t>(f.a[0].p), u = reinterpret_cast<uintptr_t>(f.a[1].p);
      p.up_first = u < g;
      // one map over both weights, if their distance is one that a stride can have
      p.a_4d = f.a[0].pitch == f.a[1].pitch && p.I % LIN_TURN == 0 && u != g && (u < g ? g - u : u - g) < (uint64_t(1) << 40) &&
               encode_turns(&p.a[0], bf16, f.a[p.up_first].p, f.s.K, p.I, f.a[0].pitch, u < g ? g - u : u - g);
      if (!p.a_4d) p.up_first = 0;
    }
    for (int m = 0; m < (gated ? 2 : parts) && !p.a_4d; ++m) {
      if (!encode(&p.a[m], bf16, f.a[m], f.s.K, p.I, f.a_mn, p.a_3d, bk, gated ? LIN_TURN : LIN_BI)) return CCE_ERR_CUDA;
    }
    for (int m = 0; m < parts; ++m) {
      if (!encode(&p.b[m], bf16, f.b[m], f.s.K, p.J, f.s.b_mn, p.b_3d, bk, b_rows)) return CCE_ERR_CUDA;
    }
  }
  if (items >= LIMIT) return CCE_ERR_SHAPE;
  a.items = static_cast<int>(items);
  a.stage_bytes = (LIN_BI + widest) * static_cast<int>(bk) * 2;
  if (n == 1 && !gated && in[0].e.y_type == CCE_F32 && plan.c[0].kb_split > LIN_CHUNK_K / static_cast<int>(bk))
    a.chunk = LIN_CHUNK_K / static_cast<int>(bk);
  a.stages = std::min(LIN_MAX_STAGES, LIN_RING_BYTES / a.stage_bytes);
  const int units = static_cast<int>(std::min<int64_t>(plan.pair ? on.pairs : on.sms, items));
  cudaError_t e = launch_linear_gemm(a, plan.pair, gated, units, s);
  ++*launches;
  for (int q = 0; q < n && e == cudaSuccess; ++q) {
    if (a.p[q].splits == 1) continue;
    e = launch_linear_join(a.p[q], gated, bf16, on.sms, s);
    ++*launches;
  }
  return e == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

// ------------------------------------------------------------------ checks
struct Matrix {
  const void* p;
  int64_t pitch;
  int type;
  int64_t rows, cols;
};

// An operand of a product: on 16 bytes, whole vectors a row.
cce_status check_operand(const Matrix& m) {
  if (m.rows > 0 && !m.p) return CCE_ERR_NULL;
  if (m.pitch < m.cols || m.pitch >= (int64_t(1) << 31)) return CCE_ERR_SHAPE;
  if (!multiple(m.p, 16) || m.pitch % 8 != 0) return CCE_ERR_ALIGN;
  return CCE_OK;
}
cce_status check_matrix(const Matrix& m, bool optional = false) {
  if (!m.p) return optional || m.rows == 0 ? CCE_OK : CCE_ERR_NULL;
  if (m.pitch < m.cols || m.pitch >= (int64_t(1) << 30)) return CCE_ERR_SHAPE;
  return multiple(m.p, type_bytes(m.type)) ? CCE_OK : CCE_ERR_ALIGN;
}
// Rows that are only read, in runs (include/cce_ops.h, "Rows").
cce_status check_rows(const Matrix& m, int64_t inner, int64_t outer_stride) {
  if (!m.p) return CCE_OK;
  if (inner < 1 || m.pitch < 0 || m.pitch >= (int64_t(1) << 30) || outer_stride < 0 || outer_stride >= MATRIX)
    return CCE_ERR_SHAPE;
  return multiple(m.p, type_bytes(m.type)) ? CCE_OK : CCE_ERR_ALIGN;
}
cce_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need <= NO_WORKSPACE) return CCE_OK;
  if (!ws) return CCE_ERR_NULL;
  if (!multiple(ws, 256)) return CCE_ERR_ALIGN;
  return have < need ? CCE_ERR_WORKSPACE : CCE_OK;
}
template <typename... S>
cce_status first_of(S... s) {
  cce_status r = CCE_OK;
  ((r = r == CCE_OK ? s : r), ...);
  return r;
}

size_t forward_bytes(int64_t M, int64_t N, int64_t K, bool gated) {
  if (!sizes_ok(M, N, K)) return 0;
  if (M <= LIN_FEW_ROWS) return NO_WORKSPACE;
  const Shape s = shape_of(N, M, K, 1, false);
  return std::max<size_t>(NO_WORKSPACE, parts_bytes(&s, 1, gated));
}

cce_status forward(const Matrix& x, const Matrix* w, bool gated, int64_t M, int64_t N, int64_t K, const LinEpilogue& e,
                   void* ws, cudaStream_t stream) {
  Device on;
  int launches = 0;
  cce_status st = on.ready();
  if (st != CCE_OK || M == 0) return st;
  const bool bf16 = x.type == CCE_BF16;
  if (M <= LIN_FEW_ROWS) {
    const LinFew f{{w[0].p, w[gated ? 1 : 0].p}, {w[0].pitch, w[gated ? 1 : 0].pitch}, x.p, x.pitch, static_cast<int>(N),
                   static_cast<int>(M), static_cast<int>(K), e};
    st = launch_linear_few(f, gated, bf16, stream) == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
    ++launches;
  } else {
    Product p{};
    p.s = shape_of(N, M, K, 1, false);
    for (int m = 0; m < (gated ? 2 : 1); ++m) p.a[m] = Operand{w[m].p, w[m].pitch};
    p.b[0] = Operand{x.p, x.pitch};
    p.e = e;
    st = run_products(&p, 1, gated, bf16, LinSum{}, ws, on, stream, &launches);
  }
  count_launches(launches);
  return st;
}

// ---------------------------------------------------------------- backward
struct BackwardShapes {
  Shape dx, dw;
};
BackwardShapes backward_shapes(int64_t M, int64_t N, int64_t K, int mats) {
  return {shape_of(K, M, N, mats, false), shape_of(K, N, M, 1, true)};
}

// What a backward call computes, and whether dz is written for its products.
struct Wanted {
  bool dx, dw[2], db, staged;

  static Wanted of(int flags) {
    return {(flags & CCE_WANT_DX) != 0, {(flags & CCE_WANT_DW) != 0, (flags & CCE_WANT_DW_UP) != 0}, (flags & CCE_WANT_DB) != 0,
            (flags & CCE_WANT_DZ) != 0};
  }
};

// dz for the products, the row sums' parts, and the products' partial sums, in this order.
struct BackwardLayout {
  size_t dz, sums, parts;
  int64_t pitch;
  size_t total() const { return std::max<size_t>(NO_WORKSPACE, dz + sums + parts); }
};

BackwardLayout backward_layout(int64_t M, int64_t N, int64_t K, int mats, const Wanted& want) {
  BackwardLayout l{};
  l.pitch = cdiv(N, 8) * 8;
  if (M == 0) return l;
  if (want.staged) l.dz = round256(size_t(2) * mats * M * l.pitch);
  if (want.db) l.sums = round256(size_t(4) * linear_grad_parts(M, N) * N);
  const BackwardShapes b = backward_shapes(M, N, K, mats);
  Shape all[LIN_MAX_PROBLEMS];
  int n = 0;
  for (int m = 0; m < mats; ++m) {
    if (want.dw[m]) all[n++] = b.dw;
  }
  if (want.dx) all[n++] = b.dx;
  if (n > 0) l.parts = parts_bytes(all, n, false);
  return l;
}

// Enough for any call of these sizes.
size_t any_backward_bytes(int64_t M, int64_t N, int64_t K, int mats) {
  if (!sizes_ok(M, N, K)) return 0;
  size_t most = 0;
  for (int products = 0; products < (mats == 2 ? 8 : 4); ++products) {  // which of dx, dW and the up projection's dW
    const Wanted want{(products & 1) != 0, {(products & 2) != 0, (products & 4) != 0}, mats == 1, true};
    most = std::max(most, backward_layout(M, N, K, mats, want).total());
  }
  return most;
}

LinEpilogue dense_out(void* y, int64_t pitch, int type) {
  LinEpilogue e{};
  e.y = y;
  e.y_pitch = pitch;
  e.y_type = type;
  return e;
}

// From the parts of dz to the gradients asked for.  weights, grad_w: mats of them.
cce_status backward_products(const Operand* dz, const Matrix& x, const Matrix* w, int mats, int64_t M, int64_t N,
                             int64_t K, void* grad_x, void* const* grad_w, const LinSum& sum, void* parts,
                             const Device& on, cudaStream_t s, int* launches) {
  const BackwardShapes b = backward_shapes(M, N, K, mats);
  const int type = x.type;
  Product p[LIN_MAX_PROBLEMS]{};
  int n = 0;
  for (int m = 0; m < mats; ++m) {
    if (!grad_w[m]) continue;
    p[n].s = b.dw;
    p[n].a[0] = Operand{x.p, x.pitch};
    p[n].b[0] = dz[m];
    p[n].a_mn = true;
    p[n++].e = dense_out(grad_w[m], K, type);
  }
  if (grad_x) {
    p[n].s = b.dx;
    for (int m = 0; m < mats; ++m) {
      p[n].a[m] = Operand{w[m].p, w[m].pitch};
      p[n].b[m] = dz[m];
    }
    p[n].a_mn = true;
    p[n++].e = dense_out(grad_x, K, type);
  }
  if (n > 0) return run_products(p, n, false, type == CCE_BF16, sum, parts, on, s, launches);
  if (sum.parts == 0) return CCE_OK;
  ++*launches;
  return launch_linear_sum(sum, s) == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

cce_status zero(void* p, size_t bytes, cudaStream_t s) {
  return !p || cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

}  // namespace
}  // namespace cce

using namespace cce;

extern "C" {

int cce_layers_abi_version(void) { return 100; }
uint64_t cce_layers_plan_searches(void) { return g_plans.searches(); }

size_t cce_linear_forward_workspace_bytes(int64_t M, int64_t N, int64_t K) { return forward_bytes(M, N, K, false); }
size_t cce_gated_linear_forward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return forward_bytes(M, N, K, true);
}
size_t cce_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) { return any_backward_bytes(M, N, K, 1); }
size_t cce_gated_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return any_backward_bytes(M, N, K, 2);
}
size_t cce_linear_backward_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int want) {
  if (!sizes_ok(M, N, K) || (want & ~(CCE_WANT_DX | CCE_WANT_DW | CCE_WANT_DB | CCE_WANT_DZ))) return 0;
  return backward_layout(M, N, K, 1, Wanted::of(want)).total();
}
size_t cce_gated_linear_backward_workspace_bytes_ex(int64_t M, int64_t N, int64_t K, int want) {
  if (!sizes_ok(M, N, K) || (want & ~(CCE_WANT_DX | CCE_WANT_DW | CCE_WANT_DW_UP))) return 0;
  return backward_layout(M, N, K, 2, Wanted::of(want == 0 ? 0 : want | CCE_WANT_DZ)).total();
}

cce_status cce_linear_forward(const void* x, int64_t x_pitch, const void* weight, int64_t w_pitch, int type,
                              const void* bias, int bias_type, const void* residual, int64_t r_inner, int64_t r_row_stride,
                              int64_t r_outer_stride, int act, int64_t M, int64_t N, int64_t K, void* y,
                              int64_t y_pitch, int y_type, void* z, int64_t z_pitch, int z_type, void* workspace,
                              size_t ws_bytes, void* stream) {
  if (!operand_type(type) || !type_ok(bias_type) || (y_type != type && y_type != CCE_F32) || !act_ok(act) ||
      !kept_type(z_type, type))
    return CCE_ERR_ARG;
  if (!sizes_ok(M, N, K)) return CCE_ERR_SHAPE;
  const Matrix xm{x, x_pitch, type, M, K}, wm{weight, w_pitch, type, N, K};
  const cce_status st =
      first_of(check_operand(xm), check_operand(wm), check_matrix({bias, N, bias_type, 1, N}, true),
               check_rows({residual, r_row_stride, y_type, M, N}, r_inner, r_outer_stride),
               check_matrix({y, y_pitch, y_type, M, N}),
               check_matrix({z, z_pitch, type, M, N}, true),
               check_workspace(workspace, ws_bytes, forward_bytes(M, N, K, false)));
  if (st != CCE_OK) return st;
  const bool runs = residual && r_inner < M;
  const LinEpilogue e{y, y_pitch, bias, residual, r_row_stride, runs ? r_outer_stride : 0, runs ? static_cast<int>(r_inner) : 0,
                      {z, nullptr}, z_pitch, y_type, bias_type, act, z_type};
  return forward(xm, &wm, false, M, N, K, e, workspace, static_cast<cudaStream_t>(stream));
}

cce_status cce_gated_linear_forward(const void* x, int64_t x_pitch, const void* gate_weight, int64_t gw_pitch,
                                    const void* up_weight, int64_t uw_pitch, int type, int act, int64_t M, int64_t N,
                                    int64_t K, void* y, int64_t y_pitch, void* gate, void* up, int64_t z_pitch,
                                    int z_type, void* workspace, size_t ws_bytes, void* stream) {
  if (!operand_type(type) || !act_ok(act) || !kept_type(z_type, type)) return CCE_ERR_ARG;
  if (!sizes_ok(M, N, K)) return CCE_ERR_SHAPE;
  if (!gate != !up) return CCE_ERR_NULL;
  const Matrix xm{x, x_pitch, type, M, K};
  const Matrix wm[2] = {{gate_weight, gw_pitch, type, N, K}, {up_weight, uw_pitch, type, N, K}};
  const cce_status st = first_of(check_operand(xm), check_operand(wm[0]), check_operand(wm[1]),
                                 check_matrix({y, y_pitch, type, M, N}), check_matrix({gate, z_pitch, type, M, N}, true),
                                 check_matrix({up, z_pitch, type, M, N}, true),
                                 check_workspace(workspace, ws_bytes, forward_bytes(M, N, K, true)));
  if (st != CCE_OK) return st;
  const LinEpilogue e{y, y_pitch, nullptr, nullptr, 0, 0, 0, {gate, up}, z_pitch, type, type, act, z_type};
  return forward(xm, wm, true, M, N, K, e, workspace, static_cast<cudaStream_t>(stream));
}

cce_status cce_linear_backward(const void* grad_y, int64_t g_pitch, int y_type, const void* x, int64_t x_pitch,
                               const void* weight, int64_t w_pitch, int type, const void* z, int64_t z_pitch,
                               int z_type, int act, int64_t M, int64_t N, int64_t K, void* grad_x,
                               void* grad_weight, void* grad_bias, int bias_type, void* workspace, size_t ws_bytes,
                               void* stream) {
  if (!operand_type(type) || !type_ok(bias_type) || (y_type != type && y_type != CCE_F32) || !act_ok(act) ||
      !kept_type(z_type, type))
    return CCE_ERR_ARG;
  if (!sizes_ok(M, N, K)) return CCE_ERR_SHAPE;
  const Matrix xm{x, x_pitch, type, M, K}, wm{weight, w_pitch, type, N, K};
  cce_status st = first_of(
      check_matrix({grad_y, g_pitch, y_type, M, N}), check_operand(xm), check_operand(wm),
      check_matrix({z, z_pitch, type, M, N}, act == CCE_ACT_NONE), check_matrix({grad_x, K, type, M, K}, true),
      check_matrix({grad_weight, K, type, N, K}, true), check_matrix({grad_bias, N, bias_type, 1, N}, true));
  if (st != CCE_OK) return st;
  // without an activation the products read grad_y itself where they can
  const bool direct = act == CCE_ACT_NONE && y_type == type && multiple(grad_y, 16) && g_pitch % 8 == 0;
  const bool staged = !direct && (grad_x || grad_weight);
  const BackwardLayout l = backward_layout(M, N, K, 1, Wanted{grad_x != nullptr, {grad_weight != nullptr}, grad_bias != nullptr, staged});
  st = check_workspace(workspace, ws_bytes, l.total());
  if (st != CCE_OK) return st;
  Device on;
  int launches = 0;
  st = on.ready();
  if (st != CCE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0)
    return first_of(zero(grad_weight, size_t(2) * N * K, s), zero(grad_bias, size_t(type_bytes(bias_type)) * N, s));
  char* ws = static_cast<char*>(workspace);
  Operand dz{grad_y, g_pitch};
  if (staged) dz = Operand{ws, l.pitch};
  LinSum sum{};
  if (staged || grad_bias) {
    LinGrad g{};
    g.dy = grad_y;
    g.dy_pitch = g_pitch;
    g.dy_type = y_type;
    g.z[0] = act == CCE_ACT_NONE ? nullptr : z;
    g.z_pitch[0] = z_pitch;
    g.kept = z_type == CCE_KEPT16;
    g.dz[0] = staged ? ws : nullptr;
    g.dz_pitch = l.pitch;
    g.part = grad_bias ? reinterpret_cast<float*>(ws + l.dz) : nullptr;
    g.M = static_cast<int>(M);
    g.N = static_cast<int>(N);
    g.act = act;
    int parts = 0;
    if (launch_linear_grad(g, false, type == CCE_BF16, s, &parts) != cudaSuccess) st = CCE_ERR_CUDA;
    ++launches;
    if (grad_bias) sum = LinSum{g.part, grad_bias, parts, g.N, bias_type};
  }
  if (st == CCE_OK)
    st = backward_products(&dz, xm, &wm, 1, M, N, K, grad_x, &grad_weight, sum, ws + l.dz + l.sums, on, s,
                           &launches);
  count_launches(launches);
  return st;
}

cce_status cce_gated_linear_backward(const void* grad_y, int64_t g_pitch, const void* x, int64_t x_pitch,
                                     const void* gate_weight, int64_t gw_pitch, const void* up_weight,
                                     int64_t uw_pitch, int type, const void* gate, int64_t gate_pitch, const void* up,
                                     int64_t up_pitch, int z_type, int act, int64_t M, int64_t N, int64_t K,
                                     void* grad_x, void* grad_gate_weight, void* grad_up_weight, void* workspace, size_t ws_bytes,
                                     void* stream) {
  if (!operand_type(type) || !act_ok(act) || !kept_type(z_type, type)) return CCE_ERR_ARG;
  if (!sizes_ok(M, N, K)) return CCE_ERR_SHAPE;
  const Matrix xm{x, x_pitch, type, M, K};
  const Matrix wm[2] = {{gate_weight, gw_pitch, type, N, K}, {up_weight, uw_pitch, type, N, K}};
  cce_status st = first_of(
      check_matrix({grad_y, g_pitch, type, M, N}), check_operand(xm), check_operand(wm[0]), check_operand(wm[1]),
      check_matrix({gate, gate_pitch, type, M, N}), check_matrix({up, up_pitch, type, M, N}),
      check_matrix({grad_x, K, type, M, K}, true), check_matrix({grad_gate_weight, K, type, N, K}, true),
      check_matrix({grad_up_weight, K, type, N, K}, true));
  if (st != CCE_OK) return st;
  const bool any = grad_x || grad_gate_weight || grad_up_weight;
  const BackwardLayout l = backward_layout(
      M, N, K, 2, Wanted{grad_x != nullptr, {grad_gate_weight != nullptr, grad_up_weight != nullptr}, false, any});
  st = check_workspace(workspace, ws_bytes, l.total());
  if (st != CCE_OK) return st;
  Device on;
  int launches = 0;
  st = on.ready();
  if (st != CCE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0)
    return first_of(zero(grad_gate_weight, size_t(2) * N * K, s), zero(grad_up_weight, size_t(2) * N * K, s));
  if (!any) return CCE_OK;
  char* ws = static_cast<char*>(workspace);
  LinGrad g{};
  g.dy = grad_y;
  g.dy_pitch = g_pitch;
  g.dy_type = type;
  g.z[0] = gate;
  g.z[1] = up;
  g.z_pitch[0] = gate_pitch;
  g.z_pitch[1] = up_pitch;
  g.kept = z_type == CCE_KEPT16;
  // one matrix after the other: rows of each start on 16 bytes
  g.dz[0] = ws;
  g.dz[1] = ws + size_t(2) * M * l.pitch;
  g.dz_pitch = l.pitch;
  g.M = static_cast<int>(M);
  g.N = static_cast<int>(N);
  g.act = act;
  int rows = 0;
  if (launch_linear_grad(g, true, type == CCE_BF16, s, &rows) != cudaSuccess) st = CCE_ERR_CUDA;
  ++launches;
  const Operand dz[2] = {{g.dz[0], l.pitch}, {g.dz[1], l.pitch}};
  void* grad_w[2] = {grad_gate_weight, grad_up_weight};
  if (st == CCE_OK)
    st = backward_products(dz, xm, wm, 2, M, N, K, grad_x, grad_w, LinSum{}, ws + l.dz, on, s, &launches);
  count_launches(launches);
  return st;
}

cce_status cce_copy_rows(const cce_row_copy* copies, int n, void* stream) {
  if (n < 0 || n > CCE_MAX_ROW_COPIES) return CCE_ERR_ARG;
  if (n > 0 && !copies) return CCE_ERR_NULL;
  LinCopies a{};
  for (int i = 0; i < n; ++i) {
    const cce_row_copy& c = copies[i];
    if (c.bytes != 2 && c.bytes != 4) return CCE_ERR_ARG;
    if (c.rows < 0 || c.cols < 0 || c.rows >= LIMIT || c.cols >= LIMIT || c.inner < 1 || c.row_stride < 0 ||
        c.outer_stride < 0 || c.pitch < c.cols)
      return CCE_ERR_SHAPE;
    if (c.rows == 0 || c.cols == 0) continue;
    if (!c.src || !c.dst) return CCE_ERR_NULL;
    if (!multiple(c.src, c.bytes) || !multiple(c.dst, 16) || c.pitch * c.bytes % 16 != 0) return CCE_ERR_ALIGN;
    a.first[a.n] = a.rows;
    a.c[a.n++] = c;
    a.rows += c.rows;
  }
  int sms = 0;
  const cce_status st = static_cast<cce_status>(device_ready(&sms));
  if (st != CCE_OK || a.n == 0) return st;
  count_launches(1);
  return launch_linear_copies(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

cce_status cce_layers_take_error(int32_t* word, void* stream) {
  if (!word) return CCE_ERR_NULL;
  int sms = 0;
  const cce_status st = static_cast<cce_status>(device_ready(&sms));
  if (st != CCE_OK) return st;
  return take_linear_error(word, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CCE_OK : CCE_ERR_CUDA;
}

cce_status cce_selftest_layers_wait_timeout(uint32_t timeout_us, void* stream) {
  if (timeout_us == 0 || timeout_us > 10000000u) return CCE_ERR_ARG;
  Device on;
  const cce_status st = on.ready();
  if (st != CCE_OK) return st;
  count_launches(1);
  return launch_linear_wait_timeout(on.error, uint64_t(timeout_us) * 1000u, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? CCE_OK
             : CCE_ERR_CUDA;
}

}  // extern "C"
