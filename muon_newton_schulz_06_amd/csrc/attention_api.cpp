// C ABI of the attention half of a block (include/muon_attention.h): argument
// checks, workspace layout and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/muon_attention.h"
#include "attention.hpp"
#include "call.hpp"

namespace muon {
namespace {

constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxHeads = int64_t(1) << 16;

// Sizes and strides of a tensor of heads, {batch, tokens, heads}.
struct Heads {
  int64_t n[3], s[3], dim;
  int64_t count() const { return n[0] * n[1] * n[2]; }
  int64_t last() const {  // elements from the first to behind the last
    int64_t e = dim;
    for (int i = 0; i < 3; ++i) e += (n[i] - 1) * s[i];
    return e;
  }
  bool same(const Heads& o) const {
    for (int i = 0; i < 3; ++i)
      if (n[i] != o.n[i] || (n[i] > 1 && s[i] != o.s[i])) return false;
    return dim == o.dim;
  }
};

// Args for tensors of heads: ranges, and token strides that keep interleaved
// tensors apart.
struct HeadArgs : Args {
  struct Tensor {
    Range r;
    Heads h;
    int64_t esz;
  };
  std::vector<Tensor> tensors;

  void heads(const char* name, const void* p, const Heads& h, size_t esz, bool written) {
    if (!ok() || h.count() == 0) return;
    if (!p) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if ((uintptr_t)p % esz) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is not aligned to its type");
    for (int i = 0; i < 3; ++i) {
      if (h.n[i] <= 1) continue;
      if (h.s[i] < 0) return fail(MUON_ERR_INVALID_ARG, std::string(name) + ": negative stride");
      if (h.s[i] > kMaxStride) return fail(MUON_ERR_UNSUPPORTED, std::string(name) + ": stride above 2^40");
    }
    if (written) {  // from the smallest stride up, each must clear what lies below it
      int64_t order[3] = {0, 1, 2}, extent = h.dim;
      std::sort(order, order + 3, [&](int64_t a, int64_t b) { return h.s[a] < h.s[b]; });
      for (int64_t i : order) {
        if (h.n[i] <= 1) continue;
        if (h.s[i] < extent) return fail(MUON_ERR_ALIAS, std::string(name) + ": its own elements overlap");
        extent += (h.n[i] - 1) * h.s[i];
      }
    }
    Heads k = h;
    for (int i = 0; i < 3; ++i)
      if (k.n[i] <= 1) k.s[i] = 0;
    const uintptr_t lo = (uintptr_t)p;
    tensors.push_back({{lo, lo + (uintptr_t)k.last() * esz, name, 0, written}, k, (int64_t)esz});
  }

  // Tokens (or, of one token, batch entries) of both lie whole multiples of one
  // stride apart, and what one holds of a token ends before the other's begins.
  static bool apart(const Tensor& a, const Tensor& b) {
    if (a.esz != b.esz) return false;
    const Tensor* t[2] = {&a, &b};
    int64_t s = 0, ext[2];
    for (int i = 1; i >= 0; --i)
      for (const Tensor* x : t)
        if (s == 0 && x->h.n[i] > 1) s = x->h.s[i] * a.esz;
    if (s == 0) return false;
    for (int i = 0; i < 2; ++i) {
      const Heads& h = t[i]->h;
      for (int j = 0; j < 2; ++j)
        if (h.n[j] > 1 && h.s[j] * a.esz % s) return false;
      ext[i] = ((h.n[2] - 1) * h.s[2] + h.dim) * a.esz;
    }
    const int64_t d = (((int64_t)(b.r.lo - a.r.lo)) % s + s) % s;
    return d >= ext[0] && d + ext[1] <= s;
  }

  // Written tensors overlap nothing, but for the pairs `same` allows.
  template <typename F>
  void all_aliases(F&& same) {
    aliases();
    for (size_t i = 0; ok() && i < tensors.size(); ++i) {
      const Tensor& a = tensors[i];
      for (size_t j = 0; ok() && j < tensors.size(); ++j) {
        const Tensor& b = tensors[j];
        if (i == j || !a.r.written || !(a.r.lo < b.r.hi && b.r.lo < a.r.hi)) continue;
        if (!b.r.written && a.r.lo == b.r.lo && a.h.same(b.h) && same(a.r.name, b.r.name)) continue;
        if (!apart(a, b)) fail(MUON_ERR_ALIAS, std::string(a.r.name) + " overlaps " + b.r.name);
      }
      for (size_t j = 0; ok() && j < ranges.size(); ++j) {
        const Range& b = ranges[j];
        if ((a.r.written || b.written) && a.r.lo < b.hi && b.lo < a.r.hi)
          fail(MUON_ERR_ALIAS, std::string(a.r.name) + " overlaps " + b.name);
      }
    }
  }
};

Heads heads_of(int64_t batch, int64_t tokens, int64_t heads, int64_t dim, const int64_t s[3]) {
  return Heads{{batch, tokens, heads}, {s[0], s[1], s[2]}, dim};
}

// ----- rotary ------------------------------------------------------------------
muon_status_t rotary(const muon_rotary_t* r, const muon_rotary_heads_t* tensors, int32_t count, bool inverse,
                     void* stream) {
  HeadArgs a;
  if (!r || !tensors) {
    a.fail(MUON_ERR_INVALID_ARG, "rotary or tensors is NULL");
    return a.report();
  }
  if (count != 1 && count != 2) a.fail(MUON_ERR_INVALID_ARG, "count must be 1 or 2");
  a.size("batch", r->batch, 0, kMaxTokens);
  a.size("tokens", r->tokens, 0, kMaxTokens);
  if (a.ok()) a.size("batch * tokens", r->batch * r->tokens, 0, kMaxTokens);
  a.size("dim", r->dim, 1, 1024);
  a.dtype("dtype", r->dtype);
  if (a.ok() && (r->rotated < 2 || r->rotated % 2 || r->rotated > r->dim))
    a.fail(MUON_ERR_INVALID_ARG, "rotated must be even, at least 2 and at most dim");
  if (!std::isfinite(r->scale)) a.fail(MUON_ERR_INVALID_ARG, "scale not finite");
  if (!a.ok()) return a.report();
  const int64_t total = r->batch * r->tokens;
  const size_t e = esize(r->dtype);
  static const char* const names[2][2] = {{"in", "out"}, {"in of the second tensor", "out of the second tensor"}};
  int64_t all = 0;
  for (int i = 0; i < count; ++i) {
    const muon_rotary_heads_t& t = tensors[i];
    a.size("heads", t.heads, 0, kMaxHeads);
    if (!a.ok()) break;
    all += t.heads;
    a.heads(names[i][0], t.in, heads_of(r->batch, r->tokens, t.heads, r->dim, t.in_strides), e, false);
    a.heads(names[i][1], t.out, heads_of(r->batch, r->tokens, t.heads, r->dim, t.out_strides), e, true);
  }
  if (a.ok() && total > 0 && all > 0) {
    a.matrix("freqs", r->freqs, 1, r->rotated / 2, r->rotated / 2, 8, false);
    if (r->positions) {
      if (r->position_bytes != 4 && r->position_bytes != 8)
        a.fail(MUON_ERR_INVALID_ARG, "position_bytes must be 4 or 8");
      else if (r->batch > 1 && r->position_stride != 0)
        a.matrix("positions", r->positions, r->batch, r->tokens, r->position_stride, r->position_bytes, false);
      else
        a.matrix("positions", r->positions, 1, r->tokens, r->tokens, r->position_bytes, false);
    }
  }
  a.all_aliases([](const char* out, const char* in) {  // a tensor's own out and in
    return (out == names[0][1] && in == names[0][0]) || (out == names[1][1] && in == names[1][0]);
  });
  if (!a.ok()) return a.report();
  if (total == 0 || all == 0) return MUON_OK;
  const muon_status_t s = check_device();
  if (s != MUON_OK) return s;
  RotaryLaunch L{};
  bool inPlace = true;
  const int64_t unit = r->interleaved ? r->rotated : r->rotated / 2;
  int n = 0;
  for (int i = 0; i < count; ++i) {
    const muon_rotary_heads_t& t = tensors[i];
    if (t.heads == 0) continue;
    RotarySide& S = L.side[n++];
    S.in = t.in;
    S.out = t.out;
    S.heads = (int32_t)t.heads;
    const int64_t sizes[3] = {r->batch, r->tokens, t.heads};
    for (int j = 0; j < 3; ++j) {  // a size of one makes its stride meaningless
      S.in_s[j] = sizes[j] > 1 ? t.in_strides[j] : 0;
      S.out_s[j] = sizes[j] > 1 ? t.out_strides[j] : 0;
      if (S.in_s[j] != S.out_s[j]) inPlace = false;
    }
    if (t.in != t.out) inPlace = false;
  }
  L.heads = (int32_t)all;
  L.batch = r->batch;
  L.tokens = r->tokens;
  L.dim = (int32_t)r->dim;
  L.rot = (int32_t)r->rotated;
  L.freqs = r->freqs;
  L.pos = r->positions;
  L.pos64 = r->position_bytes == 8;
  L.posBatch = r->batch > 1 ? r->position_stride : 0;
  L.start = r->start;
  L.scale = r->scale;
  L.inverse = inverse;
  L.interleaved = r->interleaved != 0;
  L.copyRest = !inPlace;
  L.bf16 = r->dtype == MUON_DTYPE_BF16;
  // accesses of up to 16 bytes, whatever their alignment, of whole groups of pairs
  L.vec = (int)(16 / e);
  while (unit % L.vec) L.vec /= 2;
  return launched("rotary positions", launch_rotary(L, (hipStream_t)stream), (hipStream_t)stream);
}

// ----- dropout -----------------------------------------------------------------
muon_status_t dropout(const char* xn, const void* x, int64_t ldx, const void* res, int64_t ldr, double p, uint64_t seed,
                      uint64_t offset, const uint64_t* offsetDev, const char* yn, void* y, int64_t ldy, int64_t rows,
                      int64_t cols, int32_t dtype, void* stream) {
  Args a;
  a.size("rows", rows, 0, kMaxTokens);
  a.size("cols", cols, 1, kMaxWidth);
  a.dtype("dtype", dtype);
  if (!(p >= 0.0 && p <= 1.0)) a.fail(MUON_ERR_INVALID_ARG, "p must be in [0, 1]");
  const size_t e = esize(dtype);
  if (a.ok()) {
    a.matrix(xn, x, rows, cols, ldx, e, false);
    if (res) a.matrix("residual", res, rows, cols, ldr, e, false);
    a.matrix(yn, y, rows, cols, ldy, e, true);
    if (offsetDev) a.matrix("offset_device", offsetDev, rows > 0, 1, 1, 8, false);
  }
  a.aliases([&](const char* out, const char* in) { return out == yn && std::string(in) != "offset_device"; });
  if (!a.ok()) return a.report();
  if (rows == 0) return MUON_OK;
  const muon_status_t s = check_device();
  if (s != MUON_OK) return s;
  DropoutLaunch L{};
  L.x = x;
  L.res = res;
  L.y = y;
  L.ldx = ldx;
  L.ldr = ldr;
  L.ldy = ldy;
  L.rows = rows;
  L.cols = cols;
  L.key[0] = (uint32_t)seed;
  L.key[1] = (uint32_t)(seed >> 32);
  L.offset = offset;
  L.offsetDev = offsetDev;
  const double word = std::nearbyint(p * 4294967296.0);
  L.none = word >= 4294967296.0;
  L.threshold = L.none ? 0xffffffffu : (uint32_t)word;
  L.mult = L.none ? 0.f : (float)(1.0 / (1.0 - p));
  L.bf16 = dtype == MUON_DTYPE_BF16;
  // rows that follow one another without gaps are one row
  if (rows == 1 || (ldx == cols && ldy == cols && (!res || ldr == cols))) {
    L.cols = rows * cols;
    L.rows = 1;
    L.ldx = L.ldy = L.ldr = L.cols;
  }
  L.vec = L.rows == 1 && whole_chunks(x, L.ldx, L.cols, e) && whole_chunks(y, L.ldy, L.cols, e) &&
          (!res || whole_chunks(res, L.ldr, L.cols, e));
  return launched("dropout", launch_dropout(L, (hipStream_t)stream), (hipStream_t)stream);
}

// ----- differential attention ----------------------------------------------------
int64_t blocks_of(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Whether the 16-byte loads into LDS can read the tensor: aligned heads of
// whole chunks, a tile's tokens within the loads' 31-bit offsets.
bool direct(const void* p, const Heads& h, size_t e) {
  const int64_t v = 16 / (int64_t)e;
  if ((uintptr_t)p % 16 || h.dim % v) return false;
  for (int i = 0; i < 3; ++i)
    if (h.n[i] > 1 && h.s[i] % v) return false;
  return h.n[1] <= 1 || h.s[1] < (int64_t(1) << 24);
}

struct AttnTensors {
  Heads q, k, v, out;
};
AttnTensors attn_tensors(const muon_diff_attention_t& f) {
  const int64_t none[3] = {0, 0, 0};
  return {heads_of(f.batch, f.queries, 2 * f.heads, f.dim, f.q_strides),
          heads_of(f.batch, f.keys, 2 * f.kv_heads, f.dim, f.k_strides),
          heads_of(f.batch, f.keys, f.kv_heads, 2 * f.dim, f.v_strides),
          heads_of(f.batch, f.queries, f.heads, 2 * f.dim, none)};
}

// A dense copy's strides: heads of `pitch` values one after another.
int64_t pitch_of(int64_t dim, size_t e) { return (dim * (int64_t)e + 15) / 16 * (16 / (int64_t)e); }
size_t copy_bytes(const Heads& h, size_t e) { return (size_t)h.count() * pitch_of(h.dim, e) * e; }
void dense(int64_t s[3], const Heads& h, int64_t pitch) {
  s[2] = pitch;
  s[1] = pitch * h.n[2];
  s[0] = s[1] * h.n[1];
}

struct AttnLayout {
  size_t stat, unit, kept, saved;  // in `saved`
  size_t list, q, k, v, part, partStat, total;
  int64_t rows;            // of a combo
  int64_t combos, pitch;
  int dp;
  // forward: the few-row kernel, row blocks, splits of the keys
  bool few;
  int64_t rowBlocks;
  int splits, splitKeys;
};

// Splits of a forward pass over the keys: with fewer than two workgroups per CU
// the keys are cut so that there are about that many.
void plan_splits(AttnLayout& l, bool bf16, int64_t nk) {
  const int64_t base = l.combos * l.rowBlocks, bn = attn_fwd_keys(bf16, l.dp);
  l.splits = 1;
  l.splitKeys = (int)((nk + bn - 1) / bn * bn);
  if (base == 0 || base >= 256 || nk < 4 * bn) return;  // (0: no queries or no batch)
  const int64_t want = std::min<int64_t>(std::max<int64_t>(1, kMaxSplits / base), blocks_of(nk, 2 * bn));
  const int64_t keys = blocks_of(blocks_of(nk, want), bn) * bn;
  l.splits = (int)blocks_of(nk, keys);
  l.splitKeys = (int)keys;
}

AttnLayout attn_layout(const muon_diff_attention_t& f) {
  AttnLayout l{};
  const bool bf16 = f.dtype == MUON_DTYPE_BF16;
  const size_t e = esize(f.dtype);
  const AttnTensors t = attn_tensors(f);
  const int64_t group = f.heads / f.kv_heads;
  l.rows = f.queries * group;
  l.combos = f.batch * f.kv_heads;
  l.dp = f.dim <= 64 ? 64 : 128;
  l.pitch = pitch_of(2 * f.dim, e);
  l.stat = 0;
  l.unit = align256((size_t)l.combos * 2 * l.rows * 4);
  l.kept = l.unit + (bf16 ? l.unit : 0);
  l.saved = l.kept + align256((size_t)l.combos * (bf16 ? 2 : 1) * l.rows * l.pitch * e);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  l.few = l.rows <= attn_fwd_rows(bf16, l.dp, true);
  const int64_t per = attn_fwd_rows(bf16, l.dp, l.few);
  l.rowBlocks = blocks_of(l.rows, per);
  if (f.sequences > 0) {
    l.rowBlocks = l.rows / per + f.sequences + 2;
    l.list = take(256 + (size_t)l.rowBlocks * sizeof(AttnBlock));
  }
  l.q = take(direct(f.q, t.q, e) ? 0 : copy_bytes(t.q, e));
  l.k = take(direct(f.k, t.k, e) ? 0 : copy_bytes(t.k, e));
  l.v = take(direct(f.v, t.v, e) ? 0 : copy_bytes(t.v, e));
  l.splits = 1;
  l.splitKeys = (int)f.keys;
  if (f.sequences == 0) plan_splits(l, bf16, f.keys);
  if (l.splits > 1) {
    const size_t n = (size_t)l.splits * l.combos * l.rows * 2;
    l.part = take(n * 2 * l.dp * 4);
    l.partStat = take(n * 4);
  }
  l.total = at;
  return l;
}

// How the blocks of a pass are dealt out (see AttnRuns), and where its list lies.
struct RunsPlan {
  int64_t blocks;
  int streams, least;
  size_t list, cum;
};

struct AttnGradLayout {
  size_t q, k, v, dout, rec, recL, recD, rowLam, oddKeys, part, rowPart, total;
  RunsPlan keys, rows;
};

AttnGradLayout attn_grad_layout(const muon_diff_attention_t& f, const AttnLayout& l, const void* dout,
                                const int64_t ds[3]) {
  AttnGradLayout g{};
  const bool bf16 = f.dtype == MUON_DTYPE_BF16;
  const size_t e = esize(f.dtype);
  AttnTensors t = attn_tensors(f);
  for (int i = 0; i < 3; ++i) t.out.s[i] = ds[i];
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  // A workgroup per block where these fill the CUs' places twice (the longer
  // ones first, so that the sums of two come out alike); else equal stretches of
  // all tiles, one per place, or fewer of `least` tiles.  The sums of a block that
  // stretches share are written and read once more.  Blocks of keys of a packed
  // batch go in stretches too: one of a long sequence is seen by the group's whole
  // rows, many times the mean (8192 tokens in 11 documents, 28 heads of 64: 744 µs
  // by blocks, 483 in stretches); blocks of rows are smaller (232 / 349 µs).
  const bool packed = f.sequences > 0, light = bf16 && l.dp == 64;
  auto runs = [&](RunsPlan& r, bool unequal, int64_t n, int per, double tilesOfBlock, int places, int least) {
    r.blocks = blocks_of(n, per);
    r.least = least;
    if (l.combos > 0 && n > 0 && (unequal || l.combos * r.blocks < 2 * places)) {
      const double tiles = (double)l.combos * r.blocks * tilesOfBlock;
      r.streams = (int)std::min<double>(places, std::max(8.0, std::ceil(tiles / least / 8) * 8));
    }
    if (packed) r.blocks = n / per + f.sequences + 2;
    if (packed || r.streams) r.list = take(256 + (size_t)r.blocks * sizeof(AttnBlock));
    if (r.streams) r.cum = take((size_t)(r.blocks + 1) * sizeof(int64_t));
  };
  runs(g.keys, packed, f.keys, kDkvKeys, (double)(f.heads / f.kv_heads) * blocks_of(f.queries, 32), 256, light ? 6 : 3);
  runs(g.rows, false, l.rows, kDqRows, blocks_of(f.keys, attn_dq_keys(bf16, l.dp)), light ? 512 : 256, 2);
  g.q = take(direct(f.q, t.q, e) ? 0 : copy_bytes(t.q, e));
  g.k = take(direct(f.k, t.k, e) ? 0 : copy_bytes(t.k, e));
  g.v = take(direct(f.v, t.v, e) ? 0 : copy_bytes(t.v, e));
  g.dout = take(direct(dout, t.out, e) ? 0 : copy_bytes(t.out, e));
  const size_t rows = (size_t)t.out.count();
  g.rec = take(rows * 16);
  g.recL = take(bf16 ? rows * 16 : 0);
  g.recD = take(bf16 ? rows * 16 : 0);
  g.rowLam = take(rows * 4);
  g.oddKeys = take((size_t)(l.combos * f.keys));  // (causal or not: the size queries do not ask)
  g.part = take((size_t)g.keys.streams * 2 * kDkvKeys * 4 * l.dp * 4);
  g.rowPart = take((size_t)g.rows.streams * 2 * kDqRows * (2 * l.dp + 4) * 4);
  g.total = at;
  return g;
}

void attn_sizes(Args& a, const muon_diff_attention_t* f) {
  if (!f) return a.fail(MUON_ERR_INVALID_ARG, "attention is NULL");
  a.size("batch", f->batch, 0, kMaxTokens);
  a.size("queries", f->queries, 0, kMaxTokens);
  a.size("keys", f->keys, 0, kMaxTokens);
  a.size("heads", f->heads, 1, kMaxHeads);
  a.size("kv_heads", f->kv_heads, 1, kMaxHeads);
  a.size("dim", f->dim, 1, 128);
  a.size("sequences", f->sequences, 0, kMaxTokens);
  a.dtype("dtype", f->dtype);
  if (!a.ok()) return;
  if (f->heads % f->kv_heads) return a.fail(MUON_ERR_INVALID_ARG, "kv_heads does not divide heads");
  a.size("batch * queries", f->batch * f->queries, 0, kMaxTokens);
  a.size("batch * keys", f->batch * f->keys, 0, kMaxTokens);
  a.size("queries * group", f->queries * (f->heads / f->kv_heads), 0, (int64_t(1) << 30) - 1);
  a.size("batch * queries * heads", f->batch * f->queries * f->heads, 0, int64_t(1) << 28);
  if (f->sequences > 0 && (f->batch != 1 || f->queries != f->keys))
    a.fail(MUON_ERR_INVALID_ARG, "a packed batch needs batch = 1 and queries = keys");
}

// Workgroups of a launch, as one grid dimension of 256 threads holds them.
constexpr int64_t kMaxBlocks = (int64_t(1) << 23);

// A call's tensors, in place or as aligned copies.
struct AttnCall {
  const muon_diff_attention_t& f;
  char* ws;
  hipStream_t st;
  AttnCopies copies{};
  bool bf16() const { return f.dtype == MUON_DTYPE_BF16; }
  const void* operand(const void* p, const Heads& h, size_t at, int64_t s[3]) {
    const size_t e = esize(f.dtype);
    if (direct(p, h, e)) {
      for (int i = 0; i < 3; ++i) s[i] = h.n[i] > 1 ? h.s[i] : 0;
      return p;
    }
    const int64_t pitch = pitch_of(h.dim, e);
    dense(s, h, pitch);
    if (h.count() == 0) return p;
    AttnCopy& c = copies.c[copies.n++];
    c.src = p;
    c.dst = ws + at;
    for (int i = 0; i < 3; ++i) c.s[i] = h.n[i] > 1 ? h.s[i] : 0;
    c.batch = h.n[0];
    c.tokens = h.n[1];
    c.heads = (int32_t)h.n[2];
    c.dim = (int32_t)h.dim;
    c.pitch = (int32_t)pitch;
    return ws + at;
  }
  // Adds a list to the launch that makes them.
  AttnList list(AttnPrepLaunch& P, size_t at, int32_t tokens, int32_t units, int32_t per) const {
    auto& l = P.list[P.lists++];
    l.count = (int32_t*)(ws + at);
    l.blocks = (AttnBlock*)(ws + at + 256);
    l.tokens = tokens;
    l.units = units;
    l.per = per;
    return {l.blocks, l.count};
  }
  muon_status_t copy() const {
    return copies.n ? launched("aligned copies", launch_attn_copy(bf16(), copies, st), st) : MUON_OK;
  }
};

AttnPrepLaunch prep_of(const muon_diff_attention_t& f) {
  AttnPrepLaunch P{};
  P.offsets = f.offsets;
  P.sequences = (int32_t)f.sequences;
  P.group = (int32_t)(f.heads / f.kv_heads);
  P.causal = f.causal != 0;
  P.queries = f.queries;
  P.keys = f.keys;
  return P;
}

// Strides of an output, and whether it takes 16-byte stores.
bool output_strides(int64_t s[3], const void* p, const Heads& h, size_t e) {
  const int64_t v = 16 / (int64_t)e;
  bool vec = (uintptr_t)p % 16 == 0 && h.dim % v == 0;
  for (int i = 0; i < 3; ++i) {
    s[i] = h.n[i] > 1 ? h.s[i] : 0;
    vec = vec && s[i] % v == 0;
  }
  return vec;
}

AttnShape shape_of(const muon_diff_attention_t& f, const AttnLayout& l) {
  AttnShape s{};
  s.combos = (int32_t)l.combos;
  s.kv = (int32_t)f.kv_heads;
  s.group = (int32_t)(f.heads / f.kv_heads);
  s.nq = f.queries;
  s.nk = f.keys;
  s.dim = (int32_t)f.dim;
  s.c = (float)((double)f.scale * 1.44269504088896340736);  // log2 e
  s.causal = f.causal != 0;
  s.lam = f.lambda;
  s.pitch = l.pitch;
  return s;
}

void attn_inputs(HeadArgs& a, const muon_diff_attention_t& f, const AttnTensors& t) {
  const size_t e = esize(f.dtype);
  // the backward pass holds log-sums divided by scale·log2 e
  if (!(f.scale >= 0x1p-60f && f.scale <= 0x1p60f)) a.fail(MUON_ERR_INVALID_ARG, "scale must be 2^-60 to 2^60");
  a.heads("q", f.q, t.q, e, false);
  a.heads("k", f.k, t.k, e, false);
  a.heads("v", f.v, t.v, e, false);
  if (f.batch * f.queries > 0) a.matrix("lambda", f.lambda, 1, f.heads, f.heads, 4, false);
  if (f.sequences > 0) a.matrix("offsets", f.offsets, 1, f.sequences + 1, f.sequences + 1, 4, false);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_rotary(const muon_rotary_t* r, const muon_rotary_heads_t* tensors, int32_t count, void* stream) {
  return guarded([&]() -> muon_status_t { return rotary(r, tensors, count, false, stream); });
}

muon_status_t muon_rotary_grad(const muon_rotary_t* r, const muon_rotary_heads_t* tensors, int32_t count, void* stream) {
  return guarded([&]() -> muon_status_t { return rotary(r, tensors, count, true, stream); });
}

muon_status_t muon_dropout(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual, double p,
                           uint64_t seed, uint64_t offset, const uint64_t* offset_device, void* y, int64_t ld_y,
                           int64_t rows, int64_t cols, muon_dtype_t dtype, void* stream) {
  return guarded([&]() -> muon_status_t {
    return dropout("x", x, ld_x, residual, ld_residual, p, seed, offset, offset_device, "y", y, ld_y, rows, cols, dtype,
                   stream);
  });
}

muon_status_t muon_dropout_grad(const void* dy, int64_t ld_dy, double p, uint64_t seed, uint64_t offset,
                                const uint64_t* offset_device, void* dx, int64_t ld_dx, int64_t rows, int64_t cols,
                                muon_dtype_t dtype, void* stream) {
  return guarded([&]() -> muon_status_t {
    return dropout("dy", dy, ld_dy, nullptr, 0, p, seed, offset, offset_device, "dx", dx, ld_dx, rows, cols, dtype,
                   stream);
  });
}

muon_status_t muon_diff_attention_saved_size(const muon_diff_attention_t* f, size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    Args a;
    attn_sizes(a, f);
    if (!bytes) a.fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    if (!a.ok()) return a.report();
    *bytes = attn_layout(*f).saved;
    return MUON_OK;
  });
}

muon_status_t muon_diff_attention_workspace_size(const muon_diff_attention_t* f, const void* dout,
                                                 const int64_t dout_strides[3], size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    Args a;
    attn_sizes(a, f);
    if (!bytes) a.fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    if (a.ok() && dout && !dout_strides) a.fail(MUON_ERR_INVALID_ARG, "dout_strides is NULL");
    if (!a.ok()) return a.report();
    const AttnLayout l = attn_layout(*f);
    *bytes = dout ? attn_grad_layout(*f, l, dout, dout_strides).total : l.total;
    return MUON_OK;
  });
}

muon_status_t muon_diff_attention(const muon_diff_attention_t* f, void* out, const int64_t out_strides[3], void* saved,
                                  size_t saved_bytes, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    HeadArgs a;
    attn_sizes(a, f);
    if (a.ok() && !out_strides) a.fail(MUON_ERR_INVALID_ARG, "out_strides is NULL");
    if (!a.ok()) return a.report();
    const AttnLayout l = attn_layout(*f);
    AttnTensors t = attn_tensors(*f);
    for (int i = 0; i < 3; ++i) t.out.s[i] = out_strides[i];
    const size_t e = esize(f->dtype);
    attn_inputs(a, *f, t);
    a.heads("out", out, t.out, e, true);
    if (saved) a.buffer("saved", saved, saved_bytes, l.saved, true);
    a.buffer("workspace", workspace, workspace_bytes, l.total, true);
    a.size("workgroups", l.combos * l.rowBlocks * l.splits, 0, kMaxBlocks);
    a.all_aliases([](const char*, const char*) { return false; });
    if (!a.ok()) return a.report();
    if (f->batch * f->queries == 0) return MUON_OK;
    muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    AttnCall call{*f, (char*)workspace, st};
    AttnFwdLaunch L{};
    L.s = shape_of(*f, l);
    L.s.q = call.operand(f->q, t.q, l.q, L.s.qs);
    L.s.k = call.operand(f->k, t.k, l.k, L.s.ks);
    L.s.v = call.operand(f->v, t.v, l.v, L.s.vs);
    s = call.copy();
    if (s != MUON_OK) return s;
    const bool bf16 = call.bf16();
    if (f->sequences > 0) {
      AttnPrepLaunch P = prep_of(*f);
      L.list = call.list(P, l.list, (int32_t)f->queries, L.s.group, attn_fwd_rows(bf16, l.dp, l.few));
      s = launched("blocks of the batch", launch_attn_prep(P, st), st);
      if (s != MUON_OK) return s;
    }
    if (saved) {
      L.s.stat = (float*)((char*)saved + l.stat);
      L.s.unit = (float*)((char*)saved + l.unit);
      L.s.kept = (char*)saved + l.kept;
    }
    L.out = out;
    L.vec = output_strides(L.os, out, t.out, e);
    L.rowBlocks = (int32_t)l.rowBlocks;
    L.splits = l.splits;
    L.splitKeys = l.splitKeys;
    L.part = (float*)((char*)workspace + l.part);
    L.partStat = (float*)((char*)workspace + l.partStat);
    s = launched("differential attention", launch_attn_fwd(bf16, l.dp, l.few, L, st), st);
    if (s != MUON_OK || l.splits == 1) return s;
    return launched("sum of the key splits", launch_attn_join(bf16, l.dp, L, st), st);
  });
}

muon_status_t muon_diff_attention_grad(const muon_diff_attention_t* f, const void* dout, const int64_t dout_strides[3],
                                       const void* out, const int64_t out_strides[3], const void* saved,
                                       size_t saved_bytes, const muon_diff_attention_grads_t* grads, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    HeadArgs a;
    attn_sizes(a, f);
    if (!grads) a.fail(MUON_ERR_INVALID_ARG, "grads is NULL");
    if (a.ok() && (!dout_strides || !out_strides)) a.fail(MUON_ERR_INVALID_ARG, "dout_strides or out_strides is NULL");
    if (!a.ok()) return a.report();
    const AttnLayout l = attn_layout(*f);
    const AttnGradLayout w = attn_grad_layout(*f, l, dout, dout_strides);
    const AttnTensors t = attn_tensors(*f);
    const size_t e = esize(f->dtype);
    const Heads hd = heads_of(f->batch, f->queries, f->heads, 2 * f->dim, dout_strides);
    const Heads ho = heads_of(f->batch, f->queries, f->heads, 2 * f->dim, out_strides);
    Heads gq = t.q, gk = t.k, gv = t.v;
    for (int i = 0; i < 3; ++i) {
      gq.s[i] = grads->dq_strides[i];
      gk.s[i] = grads->dk_strides[i];
      gv.s[i] = grads->dv_strides[i];
    }
    attn_inputs(a, *f, t);
    a.heads("dout", dout, hd, e, false);
    a.heads("out", out, ho, e, false);
    a.buffer("saved", saved, saved_bytes, l.saved, false);
    if (grads->dq) a.heads("dq", grads->dq, gq, e, true);
    if (!grads->dk != !grads->dv && t.k.count()) a.fail(MUON_ERR_INVALID_ARG, "dk and dv go together");
    if (grads->dk) a.heads("dk", grads->dk, gk, e, true);
    if (grads->dv) a.heads("dv", grads->dv, gv, e, true);
    if (grads->dlambda) a.matrix("dlambda", grads->dlambda, 1, f->heads, f->heads, 4, true);
    a.buffer("workspace", workspace, workspace_bytes, w.total, true);
    a.size("workgroups", l.combos * std::max(w.keys.blocks, w.rows.blocks), 0, kMaxBlocks);
    a.all_aliases([](const char*, const char*) { return false; });
    if (!a.ok()) return a.report();
    const bool wantK = grads->dk && t.k.count() > 0, wantQ = (grads->dq || grads->dlambda) && t.q.count() > 0;
    if (!wantK && !wantQ && !grads->dlambda) return MUON_OK;
    muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    char* ws = (char*)workspace;
    AttnCall call{*f, ws, st};
    const bool bf16 = call.bf16();
    AttnGradLaunch L{};
    L.s = shape_of(*f, l);
    L.s.q = call.operand(f->q, t.q, w.q, L.s.qs);
    L.s.k = call.operand(f->k, t.k, w.k, L.s.ks);
    L.s.v = call.operand(f->v, t.v, w.v, L.s.vs);
    L.dout = call.operand(dout, hd, w.dout, L.gs);
    s = call.copy();
    if (s != MUON_OK) return s;
    AttnPrepLaunch P = prep_of(*f);
    auto runs = [&](const RunsPlan& r, int32_t tokens, int32_t units, int32_t per, int32_t tile) {
      AttnRuns R{};
      R.blocks = (int32_t)r.blocks;
      R.streams = r.streams;
      R.least = r.least;
      if (r.streams || f->sequences > 0) R.list = call.list(P, r.list, tokens, units, per);
      if (r.streams) {
        P.list[P.lists - 1].tile = tile;
        P.list[P.lists - 1].cum = (int64_t*)(ws + r.cum);
        R.cum = P.list[P.lists - 1].cum;
      }
      return R;
    };
    L.keyRuns = runs(w.keys, (int32_t)f->keys, 1, kDkvKeys, 0);
    L.rowRuns = runs(w.rows, (int32_t)f->queries, L.s.group, kDqRows, attn_dq_keys(bf16, l.dp));
    L.s.stat = (float*)((char*)saved + l.stat);
    L.s.unit = (float*)((char*)saved + l.unit);
    L.s.kept = (char*)saved + l.kept;
    L.out = out;
    L.outVec = output_strides(L.os, out, ho, e);
    L.rec = (lf4*)(ws + w.rec);
    L.recL = (lu4*)(ws + w.recL);
    L.recD = (lu4*)(ws + w.recD);
    L.rowLam = (float*)(ws + w.rowLam);
    if (wantQ && f->causal) L.oddKeys = (uint8_t*)(ws + w.oddKeys);
    L.dq = grads->dq;
    L.dqVec = output_strides(L.dqs, grads->dq, gq, e);
    L.dk = grads->dk;
    output_strides(L.dks, grads->dk, gk, e);
    L.dv = grads->dv;
    output_strides(L.dvs, grads->dv, gv, e);
    L.dlam = grads->dlambda;
    L.scale = f->scale;
    L.batch = (int32_t)f->batch;
    L.heads = (int32_t)f->heads;
    L.packed = f->sequences > 0;
    L.part = (float*)(ws + w.part);
    L.rowPart = (float*)(ws + w.rowPart);
    L.joinKeys = wantK && w.keys.streams;
    L.joinRows = wantQ && w.rows.streams;
    if (hd.count() > 0 || P.lists) {
      s = launched("row sums of the gradient", launch_attn_rows(bf16, L, P, st), st);
      if (s != MUON_OK) return s;
    }
    if (wantK) {
      s = launched("gradients of keys and values", launch_attn_dkv(bf16, l.dp, L, st), st);
      if (s != MUON_OK) return s;
    }
    if (wantQ) {
      s = launched("gradient of the queries", launch_attn_dq(bf16, l.dp, L, st), st);
      if (s != MUON_OK) return s;
    }
    if (L.joinKeys || L.joinRows) {
      s = launched("sums of shared blocks", launch_attn_grad_join(bf16, l.dp, L, st), st);
      if (s != MUON_OK) return s;
    }
    if (!grads->dlambda) return MUON_OK;
    return launched("gradient of lambda", launch_attn_dlam(L, st), st);
  });
}

}  // extern "C"
