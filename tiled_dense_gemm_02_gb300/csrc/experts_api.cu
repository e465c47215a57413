// C ABI of the experts' products (include/tgemm_experts.h): argument checks, the
// layout of the workspace and of what is kept for the backward call, and the
// order of launches.
//
// Forward:  sort of the places  [gather of x]  UP  DOWN  join
// Backward: gather of grad  DH  [fp16: rounding of dg, du and w h]  DOUT  DX  join  DIN
// A few places forward: UP and DOWN on the CUDA cores (experts_few.cu).
// (experts_rows.cu and experts_gemm.cuh hold the other kernels.)  Weights whose rows are
// not 16-byte aligned are copied to an aligned pitch first.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "../../include/tgemm_experts.h"
#include "experts_internal.h"

namespace tgemm {

namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 31;
// Stages of a k axis (64 deep, four steps of the adder each) summed in tensor memory
// before they are added in fp32.  Every step truncates, by less than 2^-23 of
// the sum, an eighth of that on average where signs are mixed; every chunk's addition rounds,
// by 2^-24.  16-bit results: 256 steps stay below 2^-15 (and 2^-24 for every 4096 terms).  g, u and
// d_out W_out, whose product is the fp32 gradient of the weights: 16 steps, below 2^-19 (and 2^-24
// for every 256 terms).  Chunks of 2 / 4 / 8 / 16 stages, 8192 x 4
// rows of 2048 x 1408 in bf16: that gradient is 3.7e-7 / 6.6e-7 / 1.4e-6 / 2.9e-6 of its norm
// off (the plain fp32 form 7.3e-7); UP and DH take 332 + 294 us at 4, 263 + 201 us whole.  fp16's
// products have 22 bits where bf16's have 16 and lose more: up to 9.8e-7 at 4 stages over drawn
// sizes (bf16 7.5e-7), 7.6e-7 at 3.
constexpr int kChunk = 64, kExactChunk = 4, kExactChunkF16 = 3;
// Places up to which UP gathers x's rows by itself: a launch less where tiles have few rows
// (64 tokens, 128 experts of 2048 x 768: 204 us, and bound by the weights' bytes); many rows
// a tile are bound by the gathering copies (experts_gemm.cuh).
constexpr int64_t kGatherPlaces = kPlaceBlock;
// Whether a forward call reads the weights place by place on the CUDA cores: two launches
// that stream p experts' weights at about 4.5 TB/s, or five that read those of the d
// different ones among them (on average) at about 5.2 TB/s and start 12 us later.
// Measured, p places, this way and the tensor cores: 2048 x 1024, 64 experts, p = 8 / 16 / 32 / 64
// 27 / 41 / 72 / 130 and 39 / 60 / 82 / 116 us; 4096 x 4096, 8 experts, p = 2 / 4 / 8 / 16
// 46 / 79 / 137 / 246 and 64 / 80 / 140 / 142 us; 512 x 256, 8 experts, p = 16 6 and 19 us.
constexpr int64_t kFewPlaces = 32;
bool few_places(int64_t places, int64_t E, int64_t D, int64_t F) {
  if (places > kFewPlaces) return false;
  const double mb = 6e-6 * static_cast<double>(D) * static_cast<double>(F), p = static_cast<double>(places);
  const double different = E * (1.0 - std::pow(1.0 - 1.0 / static_cast<double>(E), p));
  return p * mb / 4.5 <= different * mb / 5.2 + 12.0;
}

int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Call {
  bool backward = false;
  int64_t T = 0, E = 0, k = 0, D = 0, F = 0;
  const void* x = nullptr;
  int64_t ldx = 0;
  const void* w_in = nullptr;
  int64_t ld_in = 0;
  const void* w_out = nullptr;
  int64_t ld_out = 0;
  const int64_t* ids = nullptr;
  const float* weights = nullptr;
  int dtype = 0;
  const tgemm_experts_options* opts = nullptr;
  void* out = nullptr;
  int64_t ldo = 0;
  void* saved = nullptr;
  size_t saved_bytes = 0;
  const void* grad = nullptr;
  int64_t ldg = 0;
  void* dx = nullptr;
  int64_t lddx = 0;
  void* dw_in = nullptr;
  int64_t ldd_in = 0;
  void* dw_out = nullptr;
  int64_t ldd_out = 0;
  float* d_weights = nullptr;
  void* workspace = nullptr;
  size_t workspace_bytes = 0;
  cudaStream_t stream = nullptr;
};

// Rows with the filling, and token tiles, at most.
int64_t most_rows(int64_t places, int64_t E) { return round_up(places + (kRowPad - 1) * std::min(E, places), kRowPad); }
int64_t most_tiles(int64_t places, int64_t E) { return most_rows(places, E) / kTokenTile + std::min(E, places); }

// Byte offsets; every part starts on a 256-byte boundary.
struct Taker {
  int64_t at = 0;
  int64_t operator()(int64_t bytes) {
    const int64_t here = at;
    at += round_up(std::max<int64_t>(bytes, 1), 256);
    return here;
  }
};

struct RowsLayout {
  int64_t head, count, first, tiles, token, place, row;
};
RowsLayout plan_rows(Taker& take, int64_t places, int64_t E) {
  RowsLayout l;
  const int64_t rows = most_rows(places, E);
  l.head = take(8);
  l.count = take(4 * E);
  l.first = take(4 * (E + 1));
  l.tiles = take(16 * most_tiles(places, E));
  l.token = take(4 * rows);
  l.place = take(4 * rows);
  l.row = take(4 * places);
  return l;
}
ExpertRows rows_at(char* base, const RowsLayout& l) {
  ExpertRows r = {};
  r.head = reinterpret_cast<int*>(base + l.head);
  r.count = reinterpret_cast<int*>(base + l.count);
  r.first = reinterpret_cast<int*>(base + l.first);
  r.tiles = reinterpret_cast<int4*>(base + l.tiles);
  r.token = reinterpret_cast<int*>(base + l.token);
  r.place = reinterpret_cast<int*>(base + l.place);
  r.row = reinterpret_cast<int*>(base + l.row);
  return r;
}

// Kept for the backward call: the sorted places, the sorted rows of x, g and u.
struct SavedLayout {
  RowsLayout rows;
  int64_t x, gu, ldg, total;
};
SavedLayout plan_saved(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F) {
  SavedLayout l;
  Taker take;
  l.rows = plan_rows(take, T * k, E);
  l.ldg = round_up(F, 4);
  l.x = take(most_rows(T * k, E) * round_up(D, 64) * 2);
  l.gu = take(most_rows(T * k, E) * 2 * l.ldg * 4);
  l.total = take.at;
  return l;
}

struct Layout {
  bool copy_in, copy_out;  // weights off the 16-byte grid
  RowsLayout rows;
  int64_t partial, x, w_in, w_out, h, dgu, y, y_exponent, dots, v, largest;
  int64_t ldx, ldh, ld_dgu, ldy, ld_in, ld_out;
  int parts;               // DH: dots of a row
  int64_t total;
};
Layout plan_layout(bool backward, int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, const void* w_in,
                   int64_t ld_in, const void* w_out, int64_t ld_out, int dtype) {
  Layout l = {};
  Taker take;
  const int64_t places = T * k, rows = most_rows(places, E);
  l.copy_in = host_granule(w_in, ld_in, 2) < 16;
  l.copy_out = host_granule(w_out, ld_out, 2) < 16;
  // sorted matrices: whole blocks of 64 columns, which the weights' gradients copy
  l.ldx = round_up(D, 64);
  l.ldh = round_up(F, 64);
  l.ld_dgu = round_up(2 * F, 64);
  l.ldy = round_up(D, 64);
  l.ld_in = round_up(D, 8);
  l.ld_out = round_up(F, 8);
  l.parts = static_cast<int>(ceil_div(F, 256) * 8);
  l.x = take(rows * l.ldx * 2);
  l.w_in = take(l.copy_in ? E * 2 * F * l.ld_in * 2 : 0);
  l.w_out = take(l.copy_out ? E * D * l.ld_out * 2 : 0);
  l.h = take(rows * l.ldh * 2);  // 32 rows at least; a few places' h in fp32 is at most half as many
  l.y = take(rows * l.ldy * (dtype == TGEMM_BF16 ? 2 : 4));
  l.y_exponent = take(dtype == TGEMM_BF16 ? rows * (l.ldy / 32) : 0);
  if (backward) {
    l.dgu = take(rows * l.ld_dgu * 2);
    l.dots = take(rows * l.parts * 4);
    if (dtype == TGEMM_F16) {
      l.v = take(rows * round_up(F, 4) * 4);
      l.largest = take(E * 2 * 4);
    }
  } else {
    l.rows = plan_rows(take, places, E);
    l.partial = take(order_blocks(places) * E * 4);
  }
  l.total = take.at;
  return l;
}

int check_shape(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, int dtype) {
  if (T < 0 || E < 1 || k < 1 || D < 1 || F < 1) return TGEMM_ERR_INVALID_VALUE;
  if (dtype != TGEMM_F16 && dtype != TGEMM_BF16) return TGEMM_ERR_UNSUPPORTED_DTYPE;
  // row numbers, tile numbers, a row's bytes and a weight's rows stay ints
  if (E > kMaxExperts || k >= 1 << 16 || D >= 1 << 24 || F >= 1 << 24 || T >= kMaxExtent - 256 ||
      T * k + kRowPad * E >= kMaxExtent - 512 || E * 2 * F >= kMaxExtent || E * D >= kMaxExtent)
    return TGEMM_ERR_TOO_LARGE;
  const int64_t blocks = ceil_div(D, 256) + ceil_div(F, 128);
  if (most_tiles(std::max<int64_t>(1, T * k), E) * blocks >= kMaxExtent / 2 ||
      E * ceil_div(2 * F, 256) * ceil_div(D, 256) >= kMaxExtent / 2)
    return TGEMM_ERR_TOO_LARGE;
  return TGEMM_OK;
}

int check_options(const tgemm_experts_options* o) {
  if (!o) return TGEMM_OK;
  if (o->wait_timeout_us < 0) return TGEMM_ERR_INVALID_VALUE;
  for (int r : o->reserved)
    if (r != 0) return TGEMM_ERR_INVALID_VALUE;
  return TGEMM_OK;
}

struct Span {
  const void* p;
  uint64_t bytes;
  int align;
};
Span span(const void* p, int64_t rows, int64_t cols, int64_t ld, int es) {
  return Span{p, p && rows > 0 ? static_cast<uint64_t>((rows - 1) * ld + cols) * es : 0, es};
}

int check_call(const Call& c) {
  int st = check_shape(c.T, c.E, c.k, c.D, c.F, c.dtype);
  if (st != TGEMM_OK) return st;
  if ((st = check_options(c.opts)) != TGEMM_OK) return st;
  if (c.ldx < c.D || c.ld_in < c.D || c.ld_out < c.F) return TGEMM_ERR_INVALID_VALUE;
  if (c.backward ? (c.ldg < c.D || (c.dx && c.lddx < c.D) || (c.dw_in && c.ldd_in < c.D) ||
                    (c.dw_out && c.ldd_out < c.F))
                 : c.ldo < c.D)
    return TGEMM_ERR_INVALID_VALUE;
  for (int64_t ld : {c.ldx, c.ld_in, c.ld_out, c.ldo, c.ldg, c.lddx, c.ldd_in, c.ldd_out})
    if (ld >= kMaxExtent) return TGEMM_ERR_TOO_LARGE;
  if (c.T > 0) {
    if (!c.x || !c.w_in || !c.w_out || !c.weights) return TGEMM_ERR_INVALID_VALUE;
    if (c.backward ? (!c.saved || !c.grad) : (!c.ids || !c.out)) return TGEMM_ERR_INVALID_VALUE;
    if (c.saved && (reinterpret_cast<uint64_t>(c.saved) % 256 ||
                    c.saved_bytes < static_cast<size_t>(plan_saved(c.T, c.E, c.k, c.D, c.F).total)))
      return TGEMM_ERR_INVALID_VALUE;
    const Layout l = plan_layout(c.backward, c.T, c.E, c.k, c.D, c.F, c.w_in, c.ld_in, c.w_out, c.ld_out,
                                 c.dtype);
    if (!c.workspace || reinterpret_cast<uint64_t>(c.workspace) % 256 ||
        c.workspace_bytes < static_cast<size_t>(l.total))
      return TGEMM_ERR_INVALID_VALUE;
  }
  const int64_t n = c.T > 0 ? 1 : 0;
  constexpr int kIn = 6, kOut = 7;
  Span in[kIn], out[kOut];
  in[0] = span(c.x, c.T, c.D, c.ldx, 2);
  in[1] = span(c.w_in, n * c.E * 2 * c.F, c.D, c.ld_in, 2);
  in[2] = span(c.w_out, n * c.E * c.D, c.F, c.ld_out, 2);
  in[3] = span(c.ids, c.T, c.k, c.k, 8);
  in[4] = span(c.weights, c.T, c.k, c.k, 4);
  in[5] = span(c.grad, c.T, c.D, c.ldg, 2);
  out[0] = span(c.out, c.T, c.D, c.ldo, 2);
  out[1] = span(c.dx, c.T, c.D, c.lddx, 2);
  out[2] = span(c.dw_in, c.E * 2 * c.F, c.D, c.ldd_in, 2);
  out[3] = span(c.dw_out, c.E * c.D, c.F, c.ldd_out, 2);
  out[4] = span(c.d_weights, c.T, c.k, c.k, 4);
  out[5] = Span{c.workspace, n ? c.workspace_bytes : 0, 1};
  out[6] = Span{c.saved, n ? c.saved_bytes : 0, 1};
  for (const Span& s : in)
    if (s.p && s.bytes && reinterpret_cast<uint64_t>(s.p) % s.align) return TGEMM_ERR_MISALIGNED;
  for (const Span& s : out)
    if (s.p && s.bytes && reinterpret_cast<uint64_t>(s.p) % s.align) return TGEMM_ERR_MISALIGNED;
  const auto meet = [](const Span& a, const Span& b) {
    const uint64_t x = reinterpret_cast<uint64_t>(a.p), y = reinterpret_cast<uint64_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && host_ranges_overlap(x, x + a.bytes, y, y + b.bytes);
  };
  for (int i = 0; i < kOut; ++i) {
    for (const Span& s : in)
      if (meet(out[i], s)) return TGEMM_ERR_ALIAS;
    for (int j = i + 1; j < kOut; ++j)
      if (meet(out[i], out[j])) return TGEMM_ERR_ALIAS;
  }
  return TGEMM_OK;
}

#define TGEMM_TRY(expr)              \
  do {                               \
    const int st_ = (expr);          \
    if (st_ != TGEMM_OK) return st_; \
  } while (0)
#define TGEMM_CUDA(expr, what)                              \
  do {                                                      \
    const cudaError_t e_ = (expr);                          \
    if (e_ != cudaSuccess) return host_cuda_fail(e_, what); \
  } while (0)

// A matrix as the products read it: where it lies, or its copy.
struct Operand {
  const void* p;
  int64_t ld;
};

class Experts {
 public:
  Experts(const Call& c, int sms, int pairs, unsigned int* status)
      : c_(c),
        l_(plan_layout(c.backward, c.T, c.E, c.k, c.D, c.F, c.w_in, c.ld_in, c.w_out, c.ld_out, c.dtype)),
        s_(plan_saved(c.T, c.E, c.k, c.D, c.F)),
        ws_(static_cast<char*>(c.workspace)),
        saved_(static_cast<char*>(c.saved)),
        sms_(sms),
        pairs_(pairs),
        type_(c.dtype == TGEMM_F16 ? 1 : 0),
        rows_max_(most_rows(c.T * c.k, c.E)) {
    std::memset(&a_, 0, sizeof a_);
    a_.E = static_cast<int>(c.E);
    a_.D = static_cast<int>(c.D);
    a_.F = static_cast<int>(c.F);
    a_.T = static_cast<int>(c.T);
    a_.bf16 = type_ == 0;
    a_.rows = saved_ ? rows_at(saved_, s_.rows) : rows_at(ws_, l_.rows);
    a_.h = ws_ + l_.h;
    a_.ldh = l_.ldh;
    a_.gu = saved_ ? reinterpret_cast<float*>(saved_ + s_.gu) : nullptr;
    a_.ldg = s_.ldg;
    a_.dgu = ws_ + l_.dgu;
    a_.ld_dgu = l_.ld_dgu;
    a_.dots = reinterpret_cast<float*>(ws_ + l_.dots);
    a_.weights = c.weights;
    a_.y = ws_ + l_.y;
    a_.y_exponent = reinterpret_cast<uint8_t*>(ws_ + l_.y_exponent);
    a_.ldy = l_.ldy;
    const int to_us = (c.opts && c.opts->wait_timeout_us) ? c.opts->wait_timeout_us : 2000000;
    a_.timeout_ns = static_cast<unsigned long long>(to_us) * 1000ull;
    a_.status = status;
  }

  int forward() {
    if (few()) return forward_few();
    OrderArgs o = {};
    o.ids = c_.ids;
    o.places = c_.T * c_.k;
    o.T = a_.T;
    o.E = a_.E;
    o.k = static_cast<int>(c_.k);
    o.rows = a_.rows;
    o.rows.partial = reinterpret_cast<int*>(ws_ + l_.partial);
    TGEMM_CUDA(launch_order(o, c_.stream), "order launch");
    TGEMM_TRY(weights(true, true));
    ExpertMaps m;
    {
      ExpertArgs a = a_;
      TGEMM_TRY(map_gates(m, a));
      a.gather = !saved_ && o.places <= kGatherPlaces && host_granule(c_.x, c_.ldx, 2) == 16;
      if (a.gather) {
        TGEMM_TRY(host_map_2d(&m.b, type_, c_.x, c_.D, c_.T, c_.ldx * 2, 64, 1));
        m.b32 = m.b16 = m.b;
      } else {
        char* rows = saved_ ? saved_ + s_.x : ws_ + l_.x;
        TGEMM_TRY(gather(c_.x, c_.ldx, rows));
        TGEMM_TRY(token_maps(m, rows, c_.D, l_.ldx));
      }
      TGEMM_TRY(map_rows(&m.c, a.h, c_.F, a.ldh, 16));
      a.m_blocks = static_cast<int>(ceil_div(c_.F, 128));
      a.k_blocks = static_cast<int>(ceil_div(c_.D, kTileK));
      a.chunk = saved_ ? exact_chunk() : kChunk;
      TGEMM_TRY(launch(launch_expert_up, m, a, tokens(a)));
    }
    {
      ExpertArgs a = a_;
      TGEMM_TRY(host_map_3d(&m.a, type_, w_out_.p, c_.F, c_.D, c_.E, w_out_.ld * 2, c_.D * w_out_.ld * 2, kTileK, kTileM));
      TGEMM_TRY(token_maps(m, a.h, c_.F, a.ldh));
      TGEMM_TRY(map_joined(m, a));
      a.m_blocks = static_cast<int>(ceil_div(c_.D, 256));
      a.k_blocks = static_cast<int>(ceil_div(c_.F, kTileK));
      a.chunk = kChunk;
      TGEMM_TRY(launch(launch_expert_down, m, a, tokens(a)));
    }
    JoinArgs j = {};
    j.weights = c_.weights;
    j.out = c_.out;
    j.ld_out = c_.ldo;
    return join(j);
  }

  int backward() {
    TGEMM_TRY(weights(c_.dx != nullptr, true));
    ExpertMaps m;
    if (type_ == 1) {
      a_.v = reinterpret_cast<float*>(ws_ + l_.v);
      a_.largest = reinterpret_cast<unsigned int*>(ws_ + l_.largest);
    }
    TGEMM_TRY(gather(c_.grad, c_.ldg, ws_ + l_.x, a_.largest, 2 * a_.E));
    {
      ExpertArgs a = a_;
      TGEMM_TRY(map_transposed(m, a, w_out_, c_.F, c_.D));
      TGEMM_TRY(token_maps(m, ws_ + l_.x, c_.D, l_.ldx));
      m.c = m.b;
      a.m_blocks = static_cast<int>(ceil_div(c_.F, 256));
      a.k_blocks = static_cast<int>(ceil_div(c_.D, kTileK));
      a.chunk = exact_chunk();  // whichever gradients are wanted: the others' bits stay
      TGEMM_TRY(launch(launch_expert_dh, m, a, tokens(a)));
    }
    if (type_ == 1 && (c_.dx || c_.dw_in || c_.dw_out)) TGEMM_TRY(round_gradients());
    if (c_.dw_out) {
      ExpertArgs a = a_;
      TGEMM_TRY(map_blocks(&m.a, ws_ + l_.x, c_.D, l_.ldx));
      TGEMM_TRY(map_blocks(&m.b, a.h, c_.F, a.ldh));
      TGEMM_TRY(gradient_out(a, m, c_.dw_out, c_.ldd_out, c_.D, c_.F));
      TGEMM_TRY(launch(launch_expert_dout, m, a, int64_t(a.E) * a.m_blocks * a.n_blocks));
    }
    JoinArgs j = {};
    if (c_.d_weights) {
      j.dots = a_.dots;
      j.parts = l_.parts;
      j.d_weights = c_.d_weights;
    }
    if (c_.dx) {
      ExpertArgs a = a_;
      TGEMM_TRY(map_transposed(m, a, w_in_, c_.D, 2 * c_.F));
      TGEMM_TRY(token_maps(m, a.dgu, 2 * c_.F, a.ld_dgu));
      TGEMM_TRY(map_joined(m, a));
      a.m_blocks = static_cast<int>(ceil_div(c_.D, 256));
      a.k_blocks = static_cast<int>(ceil_div(2 * c_.F, kTileK));
      a.chunk = kChunk;
      TGEMM_TRY(launch(launch_expert_dx, m, a, tokens(a)));
      j.out = c_.dx;
      j.ld_out = c_.lddx;
    }
    if (c_.dx || c_.d_weights) TGEMM_TRY(join(j));
    if (c_.dw_in) {
      ExpertArgs a = a_;
      TGEMM_TRY(map_blocks(&m.a, a.dgu, 2 * c_.F, a.ld_dgu));
      TGEMM_TRY(map_blocks(&m.b, saved_ + s_.x, c_.D, l_.ldx));
      TGEMM_TRY(gradient_out(a, m, c_.dw_in, c_.ldd_in, 2 * c_.F, c_.D));
      TGEMM_TRY(launch(launch_expert_din, m, a, int64_t(a.E) * a.m_blocks * a.n_blocks));
    }
    return TGEMM_OK;
  }

 private:
  bool few() const {
    return !saved_ && few_places(c_.T * c_.k, c_.E, c_.D, c_.F) && host_granule(c_.x, c_.ldx, 2) == 16 && !l_.copy_in && !l_.copy_out;
  }
  int forward_few() {
    ExpertFewArgs a = {};
    a.T = a_.T;
    a.E = a_.E;
    a.k = static_cast<int>(c_.k);
    a.D = a_.D;
    a.F = a_.F;
    a.x = c_.x;
    a.ldx = c_.ldx;
    a.w_in = c_.w_in;
    a.ld_in = c_.ld_in;
    a.w_out = c_.w_out;
    a.ld_out = c_.ld_out;
    a.ids = c_.ids;
    a.weights = c_.weights;
    a.h = reinterpret_cast<float*>(ws_ + l_.h);
    a.ldh = round_up(c_.F, 4);
    a.out = c_.out;
    a.ldo = c_.ldo;
    TGEMM_CUDA(launch_experts_few(a, type_ == 0, c_.stream), "few places launch");
    return TGEMM_OK;
  }

  int exact_chunk() const { return type_ == 1 ? kExactChunkF16 : kExactChunk; }
  int64_t tokens(const ExpertArgs& a) const { return most_tiles(c_.T * c_.k, c_.E) * a.m_blocks; }

  template <typename Launch>
  int launch(Launch function, const ExpertMaps& m, const ExpertArgs& args, int64_t units) {
    const int pairs = static_cast<int>(std::min<int64_t>(pairs_, units));
    TGEMM_CUDA(function(m, args, pairs, c_.stream), "expert launch");
    host_count_launches(1);
    return TGEMM_OK;
  }

  // W_in's rows in steps of 16 gates and their 16 ups, 64 features a box, where the
  // features are whole steps.
  int map_gates(ExpertMaps& m, ExpertArgs& a) {
    const uint64_t ld = w_in_.ld * 2, F = c_.F;
    a.split = F % 16 != 0;
    if (a.split) return host_map_3d(&m.a, type_, w_in_.p, c_.D, F, 2 * c_.E, ld, F * ld, kTileK, 16, 2);
    const uint64_t dims[5] = {static_cast<uint64_t>(c_.D), 16, 2, F / 16, static_cast<uint64_t>(c_.E)};
    const uint64_t strides[4] = {ld, F * ld, 16 * ld, 2 * F * ld};
    const uint32_t box[5] = {kTileK, 16, 2, 4, 1};
    return host_map(&m.a, type_, w_in_.p, 5, dims, strides, box);
  }
  // A weight's columns as M, 64 of its rows and 128 columns a box, where the columns
  // are whole blocks of 64 (the box's last columns would else lie past the weight's end).
  int map_transposed(ExpertMaps& m, ExpertArgs& a, const Operand& w, int64_t cols, int64_t rows) {
    a.split = cols % 64 != 0;
    if (a.split) return host_map_3d(&m.a, type_, w.p, cols, rows, c_.E, w.ld * 2, rows * w.ld * 2, 64, kTileK);
    const uint64_t ld = w.ld * 2, R = rows;
    const uint64_t dims[4] = {64, R, static_cast<uint64_t>(cols / 64), static_cast<uint64_t>(c_.E)};
    const uint64_t strides[3] = {ld, 128, R * ld};
    const uint32_t box[4] = {64, kTileK, 2, 1};
    return host_map(&m.a, type_, w.p, 4, dims, strides, box);
  }
  // A sorted matrix: boxes of 64 columns, of 64 rows and 128 columns (the pitch is whole
  // blocks of 64; what lies past cols is in rows of M or columns of N that are not stored).
  int map_rows(CUtensorMap* m, const void* p, int64_t cols, int64_t ld, uint32_t box_rows) {
    return host_map_3d(m, type_, p, cols, rows_max_, 1, ld * 2, 0, 64, box_rows);
  }
  // Where DOWN and DX store: halves (type 1) for bf16; fp16's fp32 rows are stored by the threads.
  int map_joined(ExpertMaps& m, const ExpertArgs& a) {
    m.c = m.b;
    return type_ == 0 ? host_map_3d(&m.c, 1, a.y, c_.D, rows_max_, 1, a.ldy * 2, 0, 64, 16) : TGEMM_OK;
  }
  int map_blocks(CUtensorMap* m, const void* p, int64_t cols, int64_t ld) {
    return host_map_3d(m, type_, p, 64, rows_max_, ceil_div(cols, 64), ld * 2, 128, 64, kTileK, 2);
  }
  int token_maps(ExpertMaps& m, const void* p, int64_t cols, int64_t ld) {
    TGEMM_TRY(map_rows(&m.b, p, cols, ld, 64));
    TGEMM_TRY(map_rows(&m.b32, p, cols, ld, 32));
    return map_rows(&m.b16, p, cols, ld, 16);
  }
  int gather(const void* x, int64_t ld, void* rows, unsigned int* zeros = nullptr, int words = 0) {
    TGEMM_CUDA(launch_gather_rows(a_.rows, rows_max_, x, ld, host_granule(x, ld, 2), a_.D, rows, l_.ldx, zeros, words, sms_,
                                  c_.stream),
               "gather launch");
    return TGEMM_OK;
  }

  int round_gradients() {
    RoundArgs r = {};
    r.E = a_.E;
    r.F = a_.F;
    r.rows = a_.rows;
    r.weights = a_.weights;
    r.gu = a_.gu;
    r.v = a_.v;
    r.ldg = a_.ldg;
    r.largest = a_.largest;
    r.dgu = a_.dgu;
    r.ld_dgu = a_.ld_dgu;
    r.h = a_.h;
    r.ldh = a_.ldh;
    TGEMM_CUDA(launch_round_gradients(r, rows_max_, c_.stream), "rounding launch");
    return TGEMM_OK;
  }

  int join(JoinArgs& j) {
    j.rows = &a_.rows;
    j.T = c_.T;
    j.k = static_cast<int>(c_.k);
    j.D = a_.D;
    j.y = a_.y;
    j.y_exponent = a_.y_exponent;
    j.ldy = a_.ldy;
    j.type = type_;
    TGEMM_CUDA(launch_join(j, c_.stream), "join launch");
    return TGEMM_OK;
  }

  int gradient_out(ExpertArgs& a, ExpertMaps& m, void* out, int64_t ld, int64_t M, int64_t N) {
    a.m_blocks = static_cast<int>(ceil_div(M, 256));
    a.n_blocks = static_cast<int>(ceil_div(N, 256));
    a.chunk = kChunk;
    a.out = out;
    a.ld_out = ld;
    a.store_granule = host_granule(out, ld, 2);
    m.b32 = m.b16 = m.c = m.a;  // not used, unless c is set here
    if (a.store_granule < 16) return TGEMM_OK;
    a.store_granule = 0;
    return host_map_3d(&m.c, type_, out, N, M, c_.E, ld * 2, M * ld * 2, 64, 32);
  }

  // The weights that a call reads, copied where they lie off the 16-byte grid.
  int weights(bool in, bool out) {
    in = in && l_.copy_in;
    out = out && l_.copy_out;
    w_in_ = in ? Operand{ws_ + l_.w_in, l_.ld_in} : Operand{c_.w_in, c_.ld_in};
    w_out_ = out ? Operand{ws_ + l_.w_out, l_.ld_out} : Operand{c_.w_out, c_.ld_out};
    if (!in && !out) return TGEMM_OK;
    WeightCopy first = {}, second = {};
    if (in) first = WeightCopy{c_.w_in, ws_ + l_.w_in, c_.ld_in, l_.ld_in, static_cast<int>(2 * c_.F), a_.D};
    if (out) second = WeightCopy{c_.w_out, ws_ + l_.w_out, c_.ld_out, l_.ld_out, a_.D, a_.F};
    TGEMM_CUDA(launch_copy_weights(a_.rows.count, a_.E, std::min(c_.E, c_.T * c_.k), first, second, sms_, c_.stream),
               "copy of the weights");
    return TGEMM_OK;
  }

  const Call& c_;
  Layout l_;
  SavedLayout s_;
  char* ws_;
  char* saved_;
  int sms_, pairs_, type_;
  int64_t rows_max_;
  ExpertArgs a_;
  Operand w_in_, w_out_;
};

int run_experts(const Call& c) {
  TGEMM_TRY(check_call(c));
  if (c.backward ? (!c.dx && !c.dw_in && !c.dw_out && !c.d_weights) : c.T == 0) return TGEMM_OK;
  int sms = 0, pairs = 0;
  unsigned int* status = nullptr;
  TGEMM_TRY(host_device(&sms, &pairs, &status));
  if (c.T == 0) {
    if (c.dw_in) TGEMM_CUDA(launch_zero_fill(c.dw_in, c.E * 2 * c.F, c.D, c.ldd_in, 2, c.stream), "zero-fill launch");
    if (c.dw_out) TGEMM_CUDA(launch_zero_fill(c.dw_out, c.E * c.D, c.F, c.ldd_out, 2, c.stream), "zero-fill launch");
    return TGEMM_OK;
  }
  if (pairs < 1) return host_cuda_fail(cudaErrorLaunchOutOfResources, "CTA pairs");
  Experts run(c, sms, pairs, status);
  return c.backward ? run.backward() : run.forward();
}

}  // namespace
}  // namespace tgemm

extern "C" {

int tgemm_experts_workspace_size(int backward, int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, const void* W_in,
                                 int64_t ld_in, const void* W_out, int64_t ld_out, int dtype, size_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1)) return TGEMM_ERR_INVALID_VALUE;
  const int st = tgemm::check_shape(T, E, k, D, F, dtype);
  if (st != TGEMM_OK) return st;
  if (ld_in < D || ld_out < F) return TGEMM_ERR_INVALID_VALUE;
  if (ld_in >= tgemm::kMaxExtent || ld_out >= tgemm::kMaxExtent) return TGEMM_ERR_TOO_LARGE;
  *bytes = T == 0 ? 0
                  : static_cast<size_t>(
                        tgemm::plan_layout(backward != 0, T, E, k, D, F, W_in, ld_in, W_out, ld_out, dtype).total);
  return TGEMM_OK;
}

int tgemm_experts_saved_size(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, int dtype, size_t* bytes) {
  if (!bytes) return TGEMM_ERR_INVALID_VALUE;
  const int st = tgemm::check_shape(T, E, k, D, F, dtype);
  if (st != TGEMM_OK) return st;
  *bytes = T == 0 ? 0 : static_cast<size_t>(tgemm::plan_saved(T, E, k, D, F).total);
  return TGEMM_OK;
}

int tgemm_experts_forward(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, const void* x, int64_t ldx,
                          const void* W_in, int64_t ld_in, const void* W_out, int64_t ld_out, const int64_t* ids,
                          const float* weights, int dtype, const tgemm_experts_options* opts, void* out, int64_t ldo,
                          void* saved, size_t saved_bytes, void* workspace, size_t workspace_bytes, void* stream) {
  tgemm::Call c;
  c.T = T;
  c.E = E;
  c.k = k;
  c.D = D;
  c.F = F;
  c.x = x;
  c.ldx = ldx;
  c.w_in = W_in;
  c.ld_in = ld_in;
  c.w_out = W_out;
  c.ld_out = ld_out;
  c.ids = ids;
  c.weights = weights;
  c.dtype = dtype;
  c.opts = opts;
  c.out = out;
  c.ldo = ldo;
  c.saved = saved;
  c.saved_bytes = saved_bytes;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_experts(c);
}

int tgemm_experts_backward(int64_t T, int64_t E, int64_t k, int64_t D, int64_t F, const void* x, int64_t ldx,
                           const void* W_in, int64_t ld_in, const void* W_out, int64_t ld_out, const float* weights,
                           const void* saved, size_t saved_bytes, const void* grad, int64_t ldg, int dtype,
                           const tgemm_experts_options* opts, void* dx, int64_t lddx, void* dW_in, int64_t ldd_in,
                           void* dW_out, int64_t ldd_out, float* d_weights, void* workspace, size_t workspace_bytes,
                           void* stream) {
  tgemm::Call c;
  c.backward = true;
  c.T = T;
  c.E = E;
  c.k = k;
  c.D = D;
  c.F = F;
  c.x = x;
  c.ldx = ldx;
  c.w_in = W_in;
  c.ld_in = ld_in;
  c.w_out = W_out;
  c.ld_out = ld_out;
  c.weights = weights;
  c.saved = const_cast<void*>(saved);
  c.saved_bytes = saved_bytes;
  c.grad = grad;
  c.ldg = ldg;
  c.dtype = dtype;
  c.opts = opts;
  c.dx = dx;
  c.lddx = lddx;
  c.dw_in = dW_in;
  c.ldd_in = ldd_in;
  c.dw_out = dW_out;
  c.ldd_out = ldd_out;
  c.d_weights = d_weights;
  c.workspace = workspace;
  c.workspace_bytes = workspace_bytes;
  c.stream = static_cast<cudaStream_t>(stream);
  return tgemm::run_experts(c);
}

}  // extern "C"
