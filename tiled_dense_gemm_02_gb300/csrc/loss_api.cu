// C ABI of the vocabulary-head losses (include/tgemm_loss.h): argument checks,
// workspace layout, the pieces of the vocabulary and the order of launches.
//
// Forward:  [teacher lists]  gather  STATS (one launch over the vocabulary)  combine
// Backward: [teacher lists]  gather  { DZ  DH  DW } per piece  last step of dH
// (loss_rows.cu and loss_gemm.cuh hold the kernels.)  A weight whose rows are
// not 16-byte aligned is copied to an aligned pitch piece by piece, and an fp32
// weight to its three bf16 planes.  Forward calls skip the gather where it
// saves nothing: up to one tile of rows that can be read in place, and the few
// rows of loss_few.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/tgemm_loss.h"
#include "loss_internal.h"

namespace tgemm {

cudaError_t launch_repack(const void* src, int64_t ld_src, void* dst, int64_t ld_dst, int rows, int cols,
                          int src_granule, int sms, cudaStream_t stream);

namespace {

constexpr double kLog2e = 1.4426950408889634;
constexpr int64_t kMaxExtent = int64_t(1) << 31;
// CTA pairs the layout is planned for (a GB300's 152 SMs); the layout must not
// depend on the device, so that its size can be asked for without one.
constexpr int kPlanPairs = 76;
// Bytes of one piece of dz, and of a piece of W that is copied.  Pieces of twice
// the size of L2 run tens of rounds of tiles per product, so the rounds left
// partly empty cost little; larger ones gain nothing.  A piece has 2048 entries at
// least, and W copied for one row of tiles whole rounds of them (plan_layout), at
// least 19456 entries: 117 KB per column of W in fp32, 39 KB in 16 bits.
constexpr int64_t kPieceBytes = int64_t(256) << 20;
// Stages of a k axis (64 deep, four steps of the adder each) summed in tensor
// memory before they are added in fp32 (loss_gemm.cuh).  Every step truncates, by
// less than 2^-23 of the sum: 64 steps by less than 7.6e-6 however long the axis,
// and by an eighth of that where the products' signs are mixed.  Logits of 16-bit
// operands, 2048 x 131072 x 4096 forward, chunks of 8 / 16 / 24 / 32 / 64 stages:
// 1326 / 1270 / 1210 / 1200 / 1176 us; error of lse (9.0), 300 x 4096 x 4096, by the
// first four: 0.6 / 1.0 / 1.4 / 2.0 e-6, against a last bit of 0.95e-6.  fp32: half,
// as gradients and logits are fp32 alike: 4 to 7 e-7 of their norm.  16-bit
// gradients, whose outputs keep 8 or 11 bits: 256 steps stay below 2^-15 (whole sums
// of 65536 terms of one sign were 1.7e-4 off); backward calls of 2048 x 131072 x 4096
// and of 8192 x 131072 x 1024, chunks of 32 / 64 stages / whole: 4085 / 4020 / 3980
// and 5345 / 5312 / 5212 us.
constexpr int kLogitChunk = 16, kPlaneChunk = 8, kGradientChunk = 64;
// 16-bit forward calls: k-stages of a tile up to which its statistics, not its
// product, bound the call, and eight epilogue warps beat four.  Measured at 4096 x
// 32768: D = 64 75 -> 64 us, 256 79 -> 70 us with eight; 512 104 -> 97 us, 1024 177 ->
// 168 us with four.  (Several chunks take eight, for the registers.)
constexpr int64_t kShortStages = 6;
// 16-bit backward calls: rows up to which dz is kept in two planes.  They go by the
// rows passed: the host does not know how many count.  With one plane dH and dW
// are 1.2 to 1.5 times as far off, in the norm, as their own last rounding makes
// them, from 33 rows to 1024 alike (bf16 2.2e-3 against 1.65e-3); with two rows that
// count, one row of dH was up to 1.6 times.  Two planes leave 1.00 times, and double
// the gradient products' stages.  Backward calls with one and two planes, 8192 x
// 512: 33 rows 33.7 and 36.0 us, 256 rows 33.0 and 39.8 us; 32768 x 2048: 33 rows 100
// and 123 us, 256 rows 123 and 159 us.
constexpr int64_t kTwoPlaneRows = 32;
// dH and dW share a launch while together they are at most this many stages of
// work a pair (an epilogue counts as eight).  Measured, backward calls in two
// launches and in one: bf16 300 x 10000 x 512 40.6 and 35.4 us, 512 x 8192 x 1024
// 51.7 and 45.5 us; fp32 900 x 2600 x 128 74.9 and 60.2 us; above the bound,
// where the fixed shares of the pairs end unevenly, bf16 128 x 32768 x 1024 66.4
// and 77.4 us.
constexpr int64_t kBothStages = 96, kEpilogueStages = 8;
constexpr float kRangeF16 = 16384.0f;  // |dz| <= 2: fp16's largest value is 65504, its small normals reach 2^-14

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Call {
  bool backward = false, distill = false;
  int64_t T = 0, V = 0, D = 0, K = 1;
  const void* H = nullptr;
  int64_t ldh = 0;
  const void* W = nullptr;
  int64_t ldw = 0;
  const int64_t* ids = nullptr;  // targets, or the teacher's entries
  int64_t ld_ids = 1;
  const float* logits = nullptr;
  int64_t ld_logits = 0;
  int dtype = 0;
  const tgemm_loss_options* opts = nullptr;
  float* loss = nullptr;
  float* lse_out = nullptr;
  const float* lse = nullptr;
  const float* grad = nullptr;
  void* dH = nullptr;
  int64_t lddh = 0;
  void* dW = nullptr;
  int64_t lddw = 0;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
  cudaStream_t stream = nullptr;
};

// Byte offsets into the workspace; every part starts on a 256-byte boundary.
struct Layout {
  int planes = 1;              // of H and W
  int dz_planes = 1;
  int z_planes = 1;            // planes of dz in memory: dz_planes, fp16 twice as many (kSpread)
  bool few = false;            // a few rows, on the CUDA cores
  bool simt = false;           // forward of 9 to 32 fp32 rows, on the CUDA cores
  bool direct = false;         // H is read in place
  bool pack = false;           // W is copied to an aligned pitch or to planes, piece by piece
  int64_t piece = 0, pieces = 1;
  int64_t ldh = 0, ldw_p = 0, ldz = 0, ld_acc = 0;
  int splits = 1, k_per_split = 0;
  int64_t count = 0, source = 0, place = 0, target = 0, ids = 0, q = 0, own = 0, flags = 0, coef = 0, h = 0;
  int64_t ms = 0, dot = 0, z = 0, w = 0, acc = 0;
  int64_t parts = 0;           // statistics per row
  int stats_warps = 1;         // STATS: epilogue warps per quarter of the rows
  int64_t total = 0;
};

// dH: its k axis (the piece's entries) is long and its tiles may be few, so
// each tile's k range is cut into `splits` until the rounds of the persistent
// grid balance.  The splits are joined in order by the last step, which reads
// them all: in stages of 0.27 us (a pair's 256 x 256 x 64 at 1.7 PFLOP/s)
// against 4 bytes an element at 5 TB/s, once.
void plan_dh(int64_t T, int64_t D, int64_t kb, int terms, Layout& l) {
  const int64_t tiles = ceil_div(T, kHeadTile) * ceil_div(D, kHeadTile);
  double best_us = 1e300;
  int64_t best = 1;
  for (int64_t s = 1; s <= std::max<int64_t>(1, std::min<int64_t>(64, kb / 4)); ++s) {
    if (s > 1 && s * T * l.ld_acc * 4 > kPieceBytes) break;
    const double us = 0.27 * static_cast<double>(l.pieces * ceil_div(tiles * s, kPlanPairs) * terms * ceil_div(kb, s)) +
                      static_cast<double>(s * T * l.ld_acc) * 4 / 5e6;
    if (us < 0.97 * best_us) {
      best = s;
      best_us = us;
    }
  }
  l.k_per_split = static_cast<int>(ceil_div(kb, best));
  l.splits = static_cast<int>(ceil_div(kb, l.k_per_split));
}

Layout plan_layout(bool backward, int64_t T, int64_t V, int64_t D, int64_t K, bool distill, const void* W, int64_t ldw,
                   int dtype, int64_t piece_opt) {
  Layout l;
  l.few = few_rows(backward, T, V, D, dtype == TGEMM_F32, host_granule(W, ldw, dtype == TGEMM_F32 ? 4 : 2) == 16);
  l.planes = dtype == TGEMM_F32 ? kPlanes : 1;
  l.dz_planes = l.planes > 1 ? l.planes : T <= kTwoPlaneRows ? 2 : 1;
  l.z_planes = l.dz_planes * (dtype == TGEMM_F16 ? 2 : 1);
  l.ldh = l.ldw_p = round_up(D, 8);
  l.simt = !backward && !l.few && l.planes > 1 && T <= kHeadSimtRows;
  l.pack = !l.few && !l.simt && (l.planes > 1 || host_granule(W, ldw, 2) < 16);
  l.ld_acc = round_up(D, 4);
  const int64_t whole = round_up(V, kHeadTile);
  if (piece_opt > 0) {
    l.piece = std::min(piece_opt, whole);
  } else if (!backward && !l.pack) {
    l.piece = whole;
  } else {
    const int64_t per = 2 * std::max<int64_t>(backward ? l.z_planes * T : 0, l.pack ? l.planes * l.ldw_p : 0);  // bytes per entry
    const int64_t fit = std::max<int64_t>(2048, kPieceBytes / per / kHeadTile * kHeadTile);
    if (l.pack && T <= kHeadTile) {
      // one row of tiles: whole rounds of the grid, though the copy be larger (33
      // fp32 rows of 131072 x 4096: 43 tiles for 76 pairs were 2414 + 4355 us,
      // forward and backward, 76 are 1940 + 3417)
      l.piece = std::min(round_up(fit, kPlanPairs * kHeadTile), whole);
    } else {
      l.piece = std::min(fit, whole);
      l.piece = round_up(ceil_div(V, ceil_div(V, l.piece)), kHeadTile);
    }
  }
  l.pieces = ceil_div(V, l.piece);
  l.ldz = l.piece;
  int64_t at = 0;
  const auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += round_up(std::max<int64_t>(bytes, 1), 256);
    return here;
  };
  l.count = take(256);
  l.source = take(T * 4);
  l.place = take(T * 4);
  l.target = take(distill ? 0 : T * 8);
  l.ids = take(distill ? T * K * 4 : 0);
  l.q = take(distill ? T * K * 4 : 0);
  l.own = take(distill ? T * 4 : 0);
  l.flags = take(distill ? T : 0);
  l.coef = take(backward ? T * 16 : 0);
  l.h = take(T * l.ldh * 2 * l.planes);
  if (l.pack) l.w = take(l.piece * l.ldw_p * 2 * l.planes);
  if (backward && l.few) {
    l.splits = few_shares(V, D, dtype == TGEMM_F32);
    l.z = take(V * few_held(T) * 4);
    l.acc = take(l.splits * T * l.ld_acc * 4);
  } else if (backward) {
    l.z = take(T * l.ldz * 2 * l.z_planes);
    plan_dh(T, D, ceil_div(std::min(l.piece, V), kTileK), l.planes > 1 ? 6 : l.dz_planes, l);
    l.acc = take(l.splits * T * l.ld_acc * 4);
  } else {
    const int64_t k_blocks = ceil_div(D, kTileK);
    l.stats_warps = k_blocks > kShortStages && k_blocks <= kLogitChunk ? 1 : 2;
    l.parts = l.few    ? few_blocks(T, V)
              : l.simt ? ceil_div(V, head_simt_tile(T))
                       : ceil_div(V, kHeadTile);
    l.ms = take(l.parts * T * 8);
    l.dot = take(l.parts * T * 4);
  }
  l.total = at;
  return l;
}

int check_options(const tgemm_loss_options* o, bool distill) {
  if (!o) return TGEMM_OK;
  if (!std::isfinite(o->scale) || o->scale < 0.0f) return TGEMM_ERR_INVALID_VALUE;
  if (!(o->label_smoothing >= 0.0f && o->label_smoothing <= 1.0f)) return TGEMM_ERR_INVALID_VALUE;
  if (!std::isfinite(o->z_loss) || o->z_loss < 0.0f) return TGEMM_ERR_INVALID_VALUE;
  if (distill && (o->label_smoothing != 0.0f || o->z_loss != 0.0f)) return TGEMM_ERR_INVALID_VALUE;
  if (o->piece < 0 || o->piece % kHeadTile != 0 || o->wait_timeout_us < 0) return TGEMM_ERR_INVALID_VALUE;
  for (int r : o->reserved)
    if (r != 0) return TGEMM_ERR_INVALID_VALUE;
  return TGEMM_OK;
}

int check_shape(int64_t T, int64_t V, int64_t D, int64_t K, bool distill, int dtype, const tgemm_loss_options* opts) {
  if (T < 0 || V < 1 || D < 1 || (distill && K < 1)) return TGEMM_ERR_INVALID_VALUE;
  if (dtype != TGEMM_F32 && dtype != TGEMM_F16 && dtype != TGEMM_BF16) return TGEMM_ERR_UNSUPPORTED_DTYPE;
  const int st = check_options(opts, distill);
  if (st != TGEMM_OK) return st;
  // the last tile's end and a row's bytes must stay ints
  if (T >= kMaxExtent - kHeadTile || V >= kMaxExtent - kHeadTile || D >= kMaxExtent / 8 ||
      (distill && K > TGEMM_DISTILL_MAX_K))
    return TGEMM_ERR_TOO_LARGE;
  return TGEMM_OK;
}

struct Span {
  const void* p;
  uint64_t bytes;
  int align;
};
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
  return {p, rows > 0 ? static_cast<uint64_t>((rows - 1) * ld + cols) * es : 0, es};
}

int check_call(const Call& c) {
  int st = check_shape(c.T, c.V, c.D, c.K, c.distill, c.dtype, c.opts);
  if (st != TGEMM_OK) return st;
  if (c.ldh < c.D || c.ldw < c.D || c.ld_ids < c.K || (c.distill && c.ld_logits < c.K) || (c.dH && c.lddh < c.D) ||
      (c.dW && c.lddw < c.D))
    return TGEMM_ERR_INVALID_VALUE;
  for (int64_t ld : {c.ldh, c.ldw, c.ld_ids, c.ld_logits, c.lddh, c.lddw})
    if (ld >= kMaxExtent) return TGEMM_ERR_TOO_LARGE;
  if (c.backward && !c.dH && !c.dW) return TGEMM_OK;
  const int es = c.dtype == TGEMM_F32 ? 4 : 2;
  if (c.T > 0) {
    if (!c.H || !c.W || !c.ids || (c.distill && !c.logits)) return TGEMM_ERR_INVALID_VALUE;
    if (c.backward ? (!c.lse || !c.grad) : (!c.loss || !c.lse_out)) return TGEMM_ERR_INVALID_VALUE;
  }
  const Span in[] = {span(c.H, c.T, c.D, c.ldh, es),       span(c.W, c.T > 0 ? c.V : 0, c.D, c.ldw, es),
                     span(c.ids, c.T, c.K, c.ld_ids, 8),   span(c.logits, c.distill ? c.T : 0, c.K, c.ld_logits, 4),
                     span(c.lse, c.T, 1, 1, 4),            span(c.grad, c.T, 1, 1, 4)};
  const Span out[] = {span(c.loss, c.T, 1, 1, 4), span(c.lse_out, c.T, 1, 1, 4),
                      span(c.dH, c.dH ? c.T : 0, c.D, c.lddh, es), span(c.dW, c.dW ? c.V : 0, c.D, c.lddw, es),
                      Span{c.workspace, c.workspace_bytes, 1}};
  for (const Span& s : in)
    if (s.p && s.bytes && reinterpret_cast<uint64_t>(s.p) % s.align) return TGEMM_ERR_MISALIGNED;
  for (const Span& s : out)
    if (s.p && s.bytes && reinterpret_cast<uint64_t>(s.p) % s.align) return TGEMM_ERR_MISALIGNED;
  const auto meet = [](const Span& a, const Span& b) {
    const uint64_t x = reinterpret_cast<uint64_t>(a.p), y = reinterpret_cast<uint64_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && host_ranges_overlap(x, x + a.bytes, y, y + b.bytes);
  };
  constexpr int n_out = sizeof out / sizeof out[0];
  for (int i = 0; i < n_out; ++i) {
    for (const Span& s : in)
      if (meet(out[i], s)) return TGEMM_ERR_ALIAS;
    for (int j = i + 1; j < n_out; ++j)
      if (meet(out[i], out[j])) return TGEMM_ERR_ALIAS;
  }
  return TGEMM_OK;
}

#define TGEMM_TRY(expr)                        \
  do {                                         \
    const int st_ = (expr);                    \
    if (st_ != TGEMM_OK) return st_;           \
  } while (0)
#define TGEMM_CUDA(expr, what)                              \
  do {                                                      \
    const cudaError_t e_ = (expr);                          \
    if (e_ != cudaSuccess) return host_cuda_fail(e_, what); \
  } while (0)

// The products of one call, launched piece by piece.
class Products {
 public:
  Products(const Call& c, const Layout& l, const HeadRows& rows, char* ws, float scale, float flat, int sms, int pairs,
           unsigned int* status)
      : c_(c), l_(l), rows_(rows), ws_(ws), sms_(sms), pairs_(pairs), type_(c.dtype == TGEMM_F16 ? 1 : 0) {
    std::memset(&a_, 0, sizeof a_);
    a_.count = rows.count;
    a_.T = static_cast<int>(c.T);
    a_.V = static_cast<int>(c.V);
    a_.K = static_cast<int>(c.K);
    a_.D = static_cast<int>(c.D);
    a_.bf16 = type_ == 0;  // fp32's planes are bf16
    a_.k2 = static_cast<float>(scale * kLog2e);
    a_.flat = flat;
    a_.target = c.distill ? nullptr : l.direct ? c.ids : rows.target;
    a_.mass = 1.0f - (c.opts ? c.opts->label_smoothing : 0.0f);
    a_.source = rows.source;
    a_.ids = rows.ids;
    a_.q = rows.q;
    a_.ms = reinterpret_cast<float2*>(ws + l.ms);
    a_.dot = reinterpret_cast<float*>(ws + l.dot);
    a_.coef = rows.coef;
    a_.spread = rows.spread;
    a_.factor = rows.factor;
    a_.splits = 1;
    a_.parts = l.stats_warps;
    a_.chunk = l.planes > 1 ? kPlaneChunk : kLogitChunk;
    const int to_us = (c.opts && c.opts->wait_timeout_us) ? c.opts->wait_timeout_us : 2000000;
    a_.timeout_ns = static_cast<unsigned long long>(to_us) * 1000ull;
    a_.status = status;
  }

  int run() {
    for (int64_t i = 0; i < l_.pieces; ++i) {
      v0_ = i * l_.piece;
      n_ = std::min(l_.piece, c_.V - v0_);
      a_.cols = static_cast<int>(n_);
      a_.col0 = static_cast<int>(v0_);
      a_.b_row0 = l_.pack ? 0 : a_.col0;
      a_.tile0 = static_cast<int>(v0_ / kHeadTile);
      a_.reduce = i > 0;
      TGEMM_TRY(copy_weight());
      TGEMM_TRY(logits());
      if (c_.backward) TGEMM_TRY(gradients());
    }
    return TGEMM_OK;
  }

 private:
  int64_t w_plane() const { return l_.piece * l_.ldw_p; }

  // A weight that cannot be read in place: this piece's copy.
  int copy_weight() {
    if (!l_.pack) return TGEMM_OK;
    const int n = static_cast<int>(n_);
    if (l_.planes > 1) {
      const float* src = static_cast<const float*>(c_.W) + v0_ * c_.ldw;
      TGEMM_CUDA(launch_split(src, c_.ldw, ws_ + l_.w, l_.ldw_p, w_plane(), n, a_.D, host_granule(src, c_.ldw, 4) == 16,
                              c_.stream),
                 "split launch");
    } else {
      const char* src = static_cast<const char*>(c_.W) + v0_ * c_.ldw * 2;
      TGEMM_CUDA(launch_repack(src, c_.ldw, ws_ + l_.w, l_.ldw_p, n, a_.D, host_granule(src, c_.ldw, 2), sms_, c_.stream),
                 "repack launch");
    }
    return TGEMM_OK;
  }

  int map_weight(CUtensorMap* m, uint32_t box_cols, uint32_t box_rows) {
    if (!l_.pack) return host_map_3d(m, type_, c_.W, c_.D, c_.V, 1, c_.ldw * 2, 0, box_cols, box_rows);
    // the copy's rows past the piece hold an earlier piece: the map ends before them
    return host_map_3d(m, type_, ws_ + l_.w, c_.D, n_, l_.planes, l_.ldw_p * 2, w_plane() * 2, box_cols, box_rows);
  }
  int map_hidden(CUtensorMap* m, uint32_t box_cols, uint32_t box_rows) {
    if (l_.direct) return host_map_3d(m, type_, c_.H, c_.D, c_.T, 1, c_.ldh * 2, 0, box_cols, box_rows);
    return host_map_3d(m, type_, rows_.h, c_.D, c_.T, l_.planes, l_.ldh * 2, rows_.plane * 2, box_cols, box_rows);
  }
  int map_dz(CUtensorMap* m, uint32_t box_cols, uint32_t box_rows) {
    return host_map_3d(m, type_, ws_ + l_.z, l_.ldz, c_.T, l_.z_planes, l_.ldz * 2, c_.T * l_.ldz * 2, box_cols,
                       box_rows);
  }

  // `units`: tiles, were every row to count
  template <typename Launch>
  int launch(Launch function, int planes, const CUtensorMap& ma, const CUtensorMap& mb, const CUtensorMap& mc,
             const HeadArgs& a, int64_t units) {
    const int pairs = static_cast<int>(std::min<int64_t>(pairs_, units));
    TGEMM_CUDA(function(planes, ma, mb, mc, a, pairs, c_.stream), "head launch");
    host_count_launches(1);
    return TGEMM_OK;
  }

  int logits() {
    if (l_.simt) {
      HeadSimtArgs s;
      s.head = a_;
      s.head.tile0 = static_cast<int>(v0_ / head_simt_tile(c_.T));
      s.H = static_cast<const float*>(c_.H);
      s.ldh = c_.ldh;
      s.W = static_cast<const float*>(c_.W) + v0_ * c_.ldw;
      s.ldw = c_.ldw;
      const bool aligned = host_granule(s.W, s.ldw, 4) == 16 && host_granule(s.H, s.ldh, 4) == 16;
      TGEMM_CUDA(launch_head_simt(s, aligned, c_.stream), "logits launch");
      return TGEMM_OK;
    }
    CUtensorMap mh, mw, mz;
    TGEMM_TRY(map_hidden(&mh, kTileK, kTileM));
    TGEMM_TRY(map_weight(&mw, kTileK, kTileM));
    if (c_.backward) TGEMM_TRY(map_dz(&mz, 64, 32));
    a_.k_blocks = static_cast<int>(ceil_div(c_.D, kTileK));
    const int64_t units = ceil_div(c_.T, kHeadTile) * ceil_div(n_, kHeadTile);
    return c_.backward ? launch(launch_head_dz, l_.dz_planes, mh, mw, mz, a_, units)
                       : launch(launch_head_stats, l_.planes, mh, mw, mw, a_, units);
  }

  int gradients() {
    HeadLaunch dh, dw;
    if (c_.dH) TGEMM_TRY(hidden_gradient(dh));
    if (c_.dW) TGEMM_TRY(weight_gradient(dw));
    const int64_t m_tiles = ceil_div(c_.T, kHeadTile), d_tiles = ceil_div(c_.D, kHeadTile);
    const int64_t dh_units = m_tiles * d_tiles * l_.splits, dw_units = ceil_div(n_, kHeadTile) * d_tiles;
    if (c_.dH && c_.dW && l_.pieces == 1) {
      // a unit's stages and its epilogue, in stages
      const int64_t terms = l_.planes > 1 ? 6 : l_.dz_planes;
      const int64_t dh_work = dh_units * (terms * l_.k_per_split + kEpilogueStages);
      const int64_t dw_work = dw_units * (terms * ceil_div(c_.T, kTileK) + kEpilogueStages);
      if (dh_work + dw_work <= kBothStages * pairs_ && pairs_ >= 2) {
        const int64_t share = std::max<int64_t>(1, std::min<int64_t>(pairs_ - 1, pairs_ * dh_work / (dh_work + dw_work)));
        TGEMM_CUDA(launch_head_both(l_.dz_planes, dh, static_cast<int>(std::min(share, dh_units)), dw,
                                    static_cast<int>(std::min(pairs_ - share, dw_units)), c_.stream),
                   "head launch");
        host_count_launches(1);
        return TGEMM_OK;
      }
    }
    if (c_.dH) TGEMM_TRY(launch(launch_head_dh, l_.dz_planes, dh.a, dh.b, dh.c, dh.args, dh_units));
    if (c_.dW) TGEMM_TRY(launch(launch_head_dw, l_.dz_planes, dw.a, dw.b, dw.c, dw.args, dw_units));
    return TGEMM_OK;
  }

  int hidden_gradient(HeadLaunch& out) {
    HeadArgs& b = out.args;
    b = a_;
    b.k_blocks = static_cast<int>(ceil_div(n_, kTileK));
    b.splits = l_.splits;
    b.k_per_split = l_.k_per_split;
    b.chunk = l_.planes > 1 ? kPlaneChunk : kGradientChunk;
    TGEMM_TRY(map_dz(&out.a, kTileK, kTileM));
    TGEMM_TRY(map_weight(&out.b, 64, kTileK));
    return host_map_3d(&out.c, 2, ws_ + l_.acc, c_.D, c_.T, l_.splits, l_.ld_acc * 4, c_.T * l_.ld_acc * 4, 32, 32);
  }

  int weight_gradient(HeadLaunch& out) {
    HeadArgs& b = out.args;
    b = a_;
    b.out = c_.dW;
    b.ld_out = c_.lddw;
    b.out_row0 = static_cast<int>(v0_);
    b.reduce = 0;
    const bool f32 = l_.planes > 1;
    b.chunk = f32 ? kPlaneChunk : kGradientChunk;
    b.k_blocks = static_cast<int>(ceil_div(c_.T, kTileK));  // at most: the count is the device's
    b.store_granule = host_granule(c_.dW, c_.lddw, f32 ? 4 : 2);
    TGEMM_TRY(map_dz(&out.a, 64, kTileK));
    TGEMM_TRY(map_hidden(&out.b, 64, kTileK));
    if (b.store_granule == 16) {
      b.store_granule = 0;
      return host_map_3d(&out.c, f32 ? 2 : type_, c_.dW, c_.D, c_.V, 1, c_.lddw * (f32 ? 4 : 2), 0, f32 ? 32 : 64, 32);
    }
    out.c = out.b;  // not used
    return TGEMM_OK;
  }

  const Call& c_;
  const Layout& l_;
  const HeadRows& rows_;
  char* ws_;
  int sms_, pairs_, type_;
  int64_t v0_ = 0, n_ = 0;  // this piece's first entry and width
  HeadArgs a_;
};

int run_loss(const Call& c) {
  TGEMM_TRY(check_call(c));
  if (c.backward ? (!c.dH && !c.dW) : c.T == 0) return TGEMM_OK;
  const int es = c.dtype == TGEMM_F32 ? 4 : 2;
  const float scale = c.opts && c.opts->scale != 0.0f ? c.opts->scale : 1.0f;
  const float smoothing = c.opts ? c.opts->label_smoothing : 0.0f;
  const float z_loss = c.opts ? c.opts->z_loss : 0.0f;
  const float flat = smoothing / static_cast<float>(c.V);
  Layout l;
  if (c.T > 0) {
    l = plan_layout(c.backward, c.T, c.V, c.D, c.K, c.distill, c.W, c.ldw, c.dtype, c.opts ? c.opts->piece : 0);
    if (!c.workspace || reinterpret_cast<uint64_t>(c.workspace) % 256 ||
        c.workspace_bytes < static_cast<size_t>(l.total))
      return TGEMM_ERR_INVALID_VALUE;
  }
  int sms = 0, pairs = 0;
  unsigned int* status = nullptr;
  TGEMM_TRY(host_device(&sms, &pairs, &status));
  if (c.T == 0) {
    if (c.dW) TGEMM_CUDA(launch_zero_fill(c.dW, c.V, c.D, c.lddw, es, c.stream), "zero-fill launch");
    return TGEMM_OK;
  }
  // the gather drops the rows that do not count and aligns the others: one tile
  // of aligned rows needs neither (its ignored rows touch no other row's sums)
  const int granule = host_granule(c.H, c.ldh, es);
  l.direct = l.few || l.simt || (!c.backward && l.planes == 1 && c.T <= kHeadTile && granule == 16);
  char* ws = static_cast<char*>(c.workspace);
  GatherArgs g;
  std::memset(&g, 0, sizeof g);
  HeadRows& rows = g.rows;
  if (!l.direct) {
    rows.count = reinterpret_cast<int*>(ws + l.count);
    rows.factor = reinterpret_cast<float*>(ws + l.count) + 1;
    rows.source = reinterpret_cast<int*>(ws + l.source);
    rows.place = reinterpret_cast<int*>(ws + l.place);
    if (!c.distill) rows.target = reinterpret_cast<int64_t*>(ws + l.target);
    rows.h = ws + l.h;
    rows.ldh = l.ldh;
    rows.plane = c.T * l.ldh;
  }
  if (c.distill) {
    rows.ids = reinterpret_cast<int*>(ws + l.ids);
    rows.q = reinterpret_cast<float*>(ws + l.q);
    rows.own = reinterpret_cast<float*>(ws + l.own);
    rows.flags = reinterpret_cast<unsigned char*>(ws + l.flags);
  }
  if (c.backward && !l.few) {
    rows.coef = reinterpret_cast<float4*>(ws + l.coef);
    if (c.dtype == TGEMM_F16) rows.spread = rows.count + 2;
  }
  g.T = static_cast<int>(c.T);
  g.D = static_cast<int>(c.D);
  g.es = es;
  g.H = c.H;
  g.ldh = c.ldh;
  g.granule = granule;
  g.rule.targets = c.distill ? nullptr : c.ids;
  g.rule.ignore_index = c.opts ? c.opts->ignore_index : -100;
  g.rule.flags = rows.flags;
  g.rule.V = static_cast<int>(c.V);
  g.z_loss = z_loss;
  g.scale = scale;
  g.range = c.dtype == TGEMM_F16 ? kRangeF16 : 1.0f;
  g.lse = c.lse;
  g.grad = c.grad;
  g.loss_out = c.loss;
  g.lse_out = c.lse_out;
  if (c.distill)
    TGEMM_CUDA(launch_distill_lists(c.ids, c.ld_ids, c.logits, c.ld_logits, g.T, g.rule.V, static_cast<int>(c.K), scale,
                                    rows, c.stream),
               "teacher list launch");
  if (!l.direct) TGEMM_CUDA(launch_gather(g, sms, c.stream), "gather launch");
  const int out_type = c.dtype == TGEMM_F32 ? 2 : c.dtype == TGEMM_F16 ? 1 : 0;
  float2* ms = reinterpret_cast<float2*>(ws + l.ms);
  float* dot = reinterpret_cast<float*>(ws + l.dot);
  if (l.few) {
    FewArgs f;
    std::memset(&f, 0, sizeof f);
    f.T = g.T;
    f.V = g.rule.V;
    f.D = g.D;
    f.K = static_cast<int>(c.K);
    f.H = c.H;
    f.ldh = c.ldh;
    f.W = c.W;
    f.ldw = c.ldw;
    f.k2 = static_cast<float>(scale * kLog2e);
    f.flat = flat;
    f.targets = g.rule.targets;
    f.mass = 1.0f - smoothing;
    f.ids = rows.ids;
    f.q = rows.q;
    f.ms = ms;
    f.dot = dot;
    f.ld_stats = c.T;
    const int w_granule = host_granule(c.W, c.ldw, es), blocks = few_blocks(c.T, c.V);
    if (c.backward) {
      f.rule = g.rule;
      f.scale = scale;
      f.z_loss = z_loss;
      f.lse = c.lse;
      f.grad = c.grad;
      f.dz = reinterpret_cast<float*>(ws + l.z);
      FewGradArgs d;
      std::memset(&d, 0, sizeof d);
      d.T = f.T;
      d.V = f.V;
      d.D = f.D;
      d.H = c.H;
      d.ldh = c.ldh;
      d.W = c.W;
      d.ldw = c.ldw;
      d.dz = f.dz;
      d.rule = g.rule;
      d.dW = c.dW;
      d.lddw = c.lddw;
      d.store_granule = c.dW ? host_granule(c.dW, c.lddw, es) : 0;
      d.acc = c.dH ? reinterpret_cast<float*>(ws + l.acc) : nullptr;
      d.ld_acc = l.ld_acc;
      d.shares = l.splits;
      TGEMM_CUDA(launch_few_grad(f, d, out_type, w_granule == 16, blocks, c.stream), "few-rows launch");
    } else {
      TGEMM_CUDA(launch_few_stats(f, out_type, w_granule, blocks, c.stream), "few-rows launch");
    }
  } else {
    if (pairs < 1) return host_cuda_fail(cudaErrorLaunchOutOfResources, "CTA pairs");
    Products products(c, l, rows, ws, scale, flat, sms, pairs, status);
    TGEMM_TRY(products.run());
  }
  if (!c.backward)
    TGEMM_CUDA(launch_combine(ms, dot, static_cast<int>(l.parts), g.T, scale, z_loss, rows, g.rule, c.loss,
                              c.lse_out, c.stream),
               "combine launch");
  else if (c.dH)
    TGEMM_CUDA(launch_finish_dh(reinterpret_cast<float*>(ws + l.acc), l.ld_acc, c.T * l.ld_acc, l.splits, g.T, g.D, rows,
                                g.rule, out_type, c.dH, c.lddh, c.stream),
               "dH launch");
  return TGEMM_OK;
}

}  // namespace
}  // namespace tgemm

extern "C" {

int tgemm_loss_workspace_size(int backward, int64_t T, int64_t V, int64_t D, int64_t K, const void* W, int64_t ldw,
                              int dtype, const tgemm_loss_options* opts, size_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1) || K < 0) return TGEMM_ERR_INVALID_VALUE;
  const bool distill = K > 0;
  const int st = tgemm::check_shape(T, V, D, distill ? K : 1, distill, dtype, opts);
  if (st != TGEMM_OK) return st;
  if (ldw < D) return TGEMM_ERR_INVALID_VALUE;
  if (ldw >= tgemm::kMaxExtent) return TGEMM_ERR_TOO_LARGE;
  *bytes = T == 0 ? 0
                  : static_cast<size_t>(tgemm::plan_layout(backward != 0, T, V, D, distill ? K : 1, distill, W, ldw,
                                                           dtype, opts ? opts->piece : 0)
                                            .total);
  return TGEMM_OK;
}

int tgemm_xent_forward(int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh, const void* W, int64_t ldw,
                       const int64_t* targets, int dtype, const tgemm_loss_options* opts, float* loss, float* lse,
                       void* workspace, size_t workspace_bytes, void* stream) {
  tgemm::Call c;
  c.T = T;
  c.V = V;
  c.D = D;
  c.H = H;
  c.ldh = ldh;
  c.W = W;
  c.ldw = ldw;
  c.ids = targets;
  c.dtype = dtype;
  c.opts = opts;
  c.loss = loss;
  c.lse_out = lse;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_loss(c);
}

int tgemm_xent_backward(int64_t T, int64_t V, int64_t D, const void* H, int64_t ldh, const void* W, int64_t ldw,
                        const int64_t* targets, const float* lse, const float* grad, int dtype,
                        const tgemm_loss_options* opts, void* dH, int64_t lddh, void* dW, int64_t lddw, void* workspace,
                        size_t workspace_bytes, void* stream) {
  tgemm::Call c;
  c.backward = true;
  c.T = T;
  c.V = V;
  c.D = D;
  c.H = H;
  c.ldh = ldh;
  c.W = W;
  c.ldw = ldw;
  c.ids = targets;
  c.lse = lse;
  c.grad = grad;
  c.dtype = dtype;
  c.opts = opts;
  c.dH = dH;
  c.lddh = lddh;
  c.dW = dW;
  c.lddw = lddw;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_loss(c);
}

int tgemm_distill_forward(int64_t T, int64_t V, int64_t D, int64_t K, const void* H, int64_t ldh, const void* W,
                          int64_t ldw, const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits,
                          int dtype, const tgemm_loss_options* opts, float* loss, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  tgemm::Call c;
  c.distill = true;
  c.T = T;
  c.V = V;
  c.D = D;
  c.K = K;
  c.H = H;
  c.ldh = ldh;
  c.W = W;
  c.ldw = ldw;
  c.ids = ids;
  c.ld_ids = ld_ids;
  c.logits = logits;
  c.ld_logits = ld_logits;
  c.dtype = dtype;
  c.opts = opts;
  c.loss = loss;
  c.lse_out = lse;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_loss(c);
}

int tgemm_distill_backward(int64_t T, int64_t V, int64_t D, int64_t K, const void* H, int64_t ldh, const void* W,
                           int64_t ldw, const int64_t* ids, int64_t ld_ids, const float* logits, int64_t ld_logits,
                           const float* lse, const float* grad, int dtype, const tgemm_loss_options* opts, void* dH,
                           int64_t lddh, void* dW, int64_t lddw, void* workspace, size_t workspace_bytes,
                           void* stream) {
  tgemm::Call c;
  c.backward = true;
  c.distill = true;
  c.T = T;
  c.V = V;
  c.D = D;
  c.K = K;
  c.H = H;
  c.ldh = ldh;
  c.W = W;
  c.ldw = ldw;
  c.ids = ids;
  c.ld_ids = ld_ids;
  c.logits = logits;
  c.ld_logits = ld_logits;
  c.lse = lse;
  c.grad = grad;
  c.dtype = dtype;
  c.opts = opts;
  c.dH = dH;
  c.lddh = lddh;
  c.dW = dW;
  c.lddw = lddw;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_loss(c);
}

}  // extern "C"
