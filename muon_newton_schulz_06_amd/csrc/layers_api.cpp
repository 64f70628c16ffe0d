// C ABI of the layer operators (include/muon_layers.h): argument checks,
// workspace layout and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <string>
#include <vector>

#include "../../include/muon_layers.h"
#include "launch.hpp"
#include "layers.hpp"

namespace muon {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 24;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int64_t kMaxLd = int64_t(1) << 32;

// Collects a call's argument errors and address ranges; the first error is
// kept.  Everything here runs before any HIP call.
struct Args {
  struct Range {
    uintptr_t lo, hi;
    const char* name;
    int64_t ld;
    bool written;
  };
  muon_status_t status = MUON_OK;
  std::string msg;
  std::vector<Range> ranges;

  bool ok() const { return status == MUON_OK; }
  void fail(muon_status_t s, const std::string& m) {
    if (ok()) {
      status = s;
      msg = m;
    }
  }
  void size(const char* name, int64_t v, int64_t lo, int64_t hi) {
    if (v < lo) fail(MUON_ERR_INVALID_ARG, std::string(name) + " below " + std::to_string(lo));
    else if (v > hi) fail(MUON_ERR_UNSUPPORTED, std::string(name) + " above " + std::to_string(hi));
  }
  void dtype(const char* name, int32_t d) {
    if (d != MUON_DTYPE_F32 && d != MUON_DTYPE_BF16)
      fail(MUON_ERR_INVALID_ARG, std::string("unknown ") + name);
  }
  // rows × cols of esz-byte elements; a matrix without rows may be NULL
  void matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t esz,
              bool written) {
    if (!ok() || rows == 0) return;
    if (!p) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is NULL");
    if ((uintptr_t)p % esz) return fail(MUON_ERR_INVALID_ARG, std::string(name) + " is not aligned to its type");
    if (ld < cols) return fail(MUON_ERR_INVALID_ARG, std::string(name) + ": row stride below the row length");
    if (ld > kMaxLd) return fail(MUON_ERR_UNSUPPORTED, std::string(name) + ": row stride above 2^32");
    const uintptr_t lo = (uintptr_t)p;
    ranges.push_back({lo, lo + (uintptr_t)(((rows - 1) * ld + cols) * (int64_t)esz), name, ld, written});
  }
  void buffer(const char* name, const void* p, size_t have, size_t need, bool written) {
    if (!ok() || need == 0) return;
    if (!p) return fail(MUON_ERR_WORKSPACE, std::string(name) + " is NULL");
    if ((uintptr_t)p & 255) return fail(MUON_ERR_WORKSPACE, std::string(name) + " not 256-byte aligned");
    if (have < need)
      return fail(MUON_ERR_WORKSPACE, std::string(name) + " too small: need " + std::to_string(need) +
                                          " bytes, got " + std::to_string(have));
    const uintptr_t lo = (uintptr_t)p;
    ranges.push_back({lo, lo + need, name, 0, written});
  }
  // Written ranges overlap nothing, but for the pairs `same` allows (an
  // output that is the same matrix as an input).
  template <typename F>
  void aliases(F&& same) {
    for (size_t i = 0; ok() && i < ranges.size(); ++i)
      for (size_t j = 0; ok() && j < ranges.size(); ++j) {
        const Range &a = ranges[i], &b = ranges[j];
        if (i == j || !a.written || !(a.lo < b.hi && b.lo < a.hi)) continue;
        if (!b.written && a.lo == b.lo && a.hi == b.hi && a.ld == b.ld && same(a.name, b.name)) continue;
        fail(MUON_ERR_ALIAS, std::string(a.name) + " overlaps " + b.name);
      }
  }
  void aliases() {
    aliases([](const char*, const char*) { return false; });
  }
  muon_status_t report() const {
    if (!ok()) set_last_error(msg);
    return status;
  }
};

muon_status_t check_device() {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) {
    set_last_error("no HIP device visible");
    return MUON_ERR_NO_DEVICE;
  }
  return MUON_OK;
}

// Status of a launch; with MUON_DEBUG_SYNC=1 (and no capture) it waits for
// the stream, so that a failing kernel is named.
muon_status_t launched(const char* what, hipError_t e, hipStream_t st) {
  if (e == hipSuccess) {
    const char* dbg = std::getenv("MUON_DEBUG_SYNC");
    if (dbg && dbg[0] == '1') {
      hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
      if (hipStreamIsCapturing(st, &cs) == hipSuccess && cs == hipStreamCaptureStatusNone) {
        e = hipStreamSynchronize(st);
        if (e == hipSuccess) e = hipGetLastError();
      }
    }
  }
  if (e == hipSuccess) return MUON_OK;
  set_last_error(std::string(what) + ": " + hipGetErrorString(e));
  return MUON_ERR_HIP;
}

// No exception leaves an entry point.
template <typename F>
muon_status_t guarded(F&& f) {
  try {
    set_last_error("");
    return f();
  } catch (const std::exception& e) {
    try {
      set_last_error(e.what());
    } catch (...) {
    }
    return MUON_ERR_INVALID_ARG;
  } catch (...) {
    return MUON_ERR_INVALID_ARG;
  }
}

size_t esize(int32_t dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

// Rows of whole 16-byte chunks at 16-byte aligned addresses.
bool whole_chunks(const void* p, int64_t ld, int64_t cols, size_t esz) {
  const int64_t v = 16 / (int64_t)esz;
  return ((uintptr_t)p & 15) == 0 && ld % v == 0 && cols % v == 0;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// ----- embedding gradient's workspace ----------------------------------------
struct EmbedLayout {
  size_t key[2], idx[2], counts, pieces, total;
};
EmbedLayout embed_layout(int64_t tokens, int64_t dim) {
  EmbedLayout l{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  const bool small = tokens <= kEmbedSmallSort;
  for (int i = 0; i < 2; ++i) {
    const size_t n = i && small ? 0 : (size_t)tokens * 4;
    l.key[i] = take(n);
    l.idx[i] = take(n);
  }
  const int64_t blocks = (tokens + kEmbedSortBlock - 1) / kEmbedSortBlock;
  l.counts = take(small ? 0 : (size_t)(blocks << kEmbedSortBits) * 4);
  l.pieces = take((size_t)(tokens / kEmbedPiece) * dim * 4);
  l.total = at;
  return l;
}

// ----- gated feed-forward block ----------------------------------------------
int64_t tiles_of(int64_t n, int64_t t) { return (n + t - 1) / t; }
int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }

// Whether a bf16 operand can be read by the 16-byte buffer loads: aligned
// rows of whole chunks, and a tile's rows within the loads' 31-bit offsets.
bool direct16(const void* p, int64_t ld, int64_t cols) {
  return whole_chunks(p, ld, cols, 2) && ld < (int64_t(1) << 22) - 64;
}

// How a product runs: the tile (rows × columns; tm = 0: the few-token kernel)
// and its k splits.
struct TilePlan {
  int tm, tn, splits, per;  // per: k-tiles of 32 in a split
};

// Estimated time of n workgroups of `per` k-tiles, in µs, fitted to measured
// products (bf16 tiles 256² run one to a CU, 128² two; the fp32 tiles are
// bound by the matrix pipe or, alone on a CU, by a step's latency, and the
// stores of a 128-row one overlap less: 38 tokens, 2944×6681, the weights'
// gradients 158 µs with 128 rows, 131 with 64; 1024 tokens, 2048×8192, y 309 /
// 344).
double tile_time(bool bf16, int tm, int64_t n, int64_t per) {
  const double cu = std::ceil(n / 256.0);  // workgroups on the busiest CU
  if (bf16) return tm == 256 ? cu * (per * 0.77 + 14) : std::ceil(n / 512.0) * (per * (n <= 256 ? 0.40 : 0.62) + 10);
  if (tm == 128) return 10 + 8.5 * cu + per * std::max(2.75, 2.2 * cu);
  return 10 + 3 * cu + per * std::max(1.65, 1.2 * cu);
}

// Tile and splits of a product of M × N results (all problems of a launch
// together) over KT k-tiles.
TilePlan plan_tiles(bool bf16, int64_t M, int64_t N, int64_t KT) {
  static const int k16[2][2] = {{256, 256}, {128, 128}}, k32[2][2] = {{128, 128}, {64, 128}};
  const int unit = bf16 ? 4 : 1;  // the bf16 loop runs whole groups of four k-tiles
  TilePlan best{};
  double bestT = 0;
  for (int i = 0; i < 2; ++i) {
    const int tm = bf16 ? k16[i][0] : k32[i][0], tn = bf16 ? k16[i][1] : k32[i][1];
    const int64_t tiles = tiles_of(M, tm) * tiles_of(N, tn);
    for (int s = 1; s <= 32; ++s) {
      const int64_t per = std::max<int64_t>(unit, tiles_of(tiles_of(KT, s), unit) * unit);
      if (s > 1 && (tiles_of(KT, per) != s || per < 8)) continue;
      double t = tile_time(bf16, tm, tiles * s, per);
      if (s > 1) t += 5.0 + 8.0 * s * M * N / 4e6;  // the splits' sums written and read
      if (!best.tm || t < bestT) {
        best = {tm, tn, s, (int)per};
        bestT = t;
      }
    }
  }
  return best;
}

// Whether the forward pass of T tokens takes the few-token kernel.  It reads
// every weight once at HBM's rate, but its workgroups each read the tokens
// again, so its time grows with tokens × weights.  Measured (µs, few-token
// kernel against tiles): bf16 3584×18944 T 1: 85 / 113, 12: 109 / 103, 64: 216 /
// 130; bf16 1024×4096 T 64: 25 / 28; fp32 (blocks of 16 tokens, so whole blocks
// count) 3584×18944 T 16: 231 / 331, 32: 311 / 329, 48: 302 / 301; 2944×6681
// T 32: 89 / 106, 38: 121 / 113; 1024×4096 T 40: 35 / 46, 64: 43 / 47.
bool few_tokens(bool bf16, int64_t T, int64_t weights) {
  if (bf16) return T <= kFfnFew && (double)T * weights <= 2e9;
  return T <= 32 || (T <= kFfnFew && (double)tiles_of(T, 16) * weights <= 1.5e8);
}

// The few-token kernel: about 1024 workgroups of 16 weight rows, each split at
// least 16 k-tiles long: a step of four waves × four loads.  With one block of
// tokens a wave takes eight loads, so that a split of 16 k-tiles leaves two of
// its waves without work (measured with this step length only).
TilePlan plan_few(int64_t N, int64_t K) {
  constexpr int64_t step = 16;  // k-tiles
  const int64_t KT = tiles_of(K, 32), want = std::max<int64_t>(1, tiles_of(1024, tiles_of(N, 16)));
  const int64_t per = std::max(step, tiles_of(tiles_of(KT, want), step) * step);
  return {0, 16, (int)tiles_of(KT, per), (int)per};
}

struct FfnLayout {
  int64_t ldh;               // hidden rounded up to 8
  size_t ab, savedH, saved;  // in `saved`
  // workspace: what the call computes (h, or dg and du), aligned copies, and
  // the splits' sums
  size_t mid, x, dy, gate, up, down, part, total;
  bool few;
  // forward: the gated projections and y; backward: dh, dx and the weights'
  TilePlan first, second, third;
};

int64_t round4(int64_t n) { return (n + 3) / 4 * 4; }

// Layout for the forward (grad = 0) or the backward pass.
FfnLayout ffn_layout(const muon_ffn_t& f, bool grad) {
  FfnLayout l{};
  const size_t e = esize(f.dtype);
  const bool bf16 = f.dtype == MUON_DTYPE_BF16;
  const int64_t T = f.tokens, D = f.model, F = f.hidden, D8 = round8(D);
  l.ldh = round8(F);
  const size_t rows = (size_t)T * l.ldh * e;
  l.ab = 0;
  l.savedH = align256((size_t)T * l.ldh * (bf16 ? 6 : 8));  // a and b: 24 bits each, or fp32
  l.saved = l.savedH + align256(rows);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align256(n);
    return o;
  };
  l.mid = take(grad ? 2 * rows : rows);
  if (T == 0) {
    l.third = plan_tiles(bf16, 3 * F, D, 0);
    l.total = at;
    return l;
  }
  l.few = !grad && few_tokens(bf16, T, 3 * D * F);
  if (bf16 && !l.few) {
    l.x = take((size_t)T * D8 * 2);
    l.dy = take(grad ? (size_t)T * D8 * 2 : 0);
    l.gate = take(direct16(f.w_gate, f.ld_gate, D) ? 0 : (size_t)F * D8 * 2);
    l.up = take(direct16(f.w_up, f.ld_up, D) ? 0 : (size_t)F * D8 * 2);
    l.down = take(direct16(f.w_down, f.ld_down, F) ? 0 : (size_t)D * l.ldh * 2);
  }
  size_t part = 0;  // floats
  auto splits = [&](const TilePlan& p, int64_t n) {
    if (p.splits > 1) part = std::max(part, (size_t)p.splits * n);
  };
  if (l.few) {
    l.first = plan_few(F, D);
    l.second = plan_few(D, F);
    splits(l.first, T * 2 * round4(F));
    splits(l.second, T * round4(D));
  } else if (!grad) {
    l.first = plan_tiles(bf16, T, 2 * F, tiles_of(D, 32));
    l.second = plan_tiles(bf16, T, D, tiles_of(F, 32));
    splits(l.first, T * 2 * round4(F));
    splits(l.second, T * round4(D));
  } else {
    l.first = plan_tiles(bf16, T, F, tiles_of(D, 32));
    l.second = plan_tiles(bf16, T, D, 2 * tiles_of(F, 32));
    l.third = plan_tiles(bf16, 3 * F, D, tiles_of(T, 32));
    splits(l.first, T * round4(F));
    splits(l.second, T * round4(D));
    splits(l.third, 2 * F * round4(D) + D * round4(F));
  }
  l.part = take(part * 4);
  l.total = at;
  return l;
}

void ffn_sizes(Args& a, const muon_ffn_t* f) {
  if (!f) return a.fail(MUON_ERR_INVALID_ARG, "ffn is NULL");
  a.size("tokens", f->tokens, 0, kMaxTokens);
  a.size("model", f->model, 1, kMaxWidth);
  a.size("hidden", f->hidden, 1, kMaxWidth);
  a.dtype("dtype", f->dtype);
}

void ffn_weights(Args& a, const muon_ffn_t& f) {
  const size_t e = esize(f.dtype);
  a.matrix("w_gate", f.w_gate, f.hidden, f.model, f.ld_gate, e, false);
  a.matrix("w_up", f.w_up, f.hidden, f.model, f.ld_up, e, false);
  a.matrix("w_down", f.w_down, f.model, f.hidden, f.ld_down, e, false);
}

void set_out(FfnProb& p, void* C, int64_t ldc, bool bf16) {
  p.C = C;
  p.ldc = ldc;
  p.vecC = ldc % 4 == 0 && (uintptr_t)C % (bf16 ? 8 : 16) == 0;
}

struct Op {
  const void* p;
  int64_t ld;
  int64_t ext;  // elements of a row, a multiple of 8 on the bf16 path
};

// A call of the block: its layout, stream and (bf16) aligned operands.
struct FfnCall {
  const muon_ffn_t& f;
  const FfnLayout& l;
  char* ws;
  hipStream_t st;
  FfnPacks packs{};
  bool bf16() const { return f.dtype == MUON_DTYPE_BF16; }

  // The operand itself, or its aligned copy at `at` in the workspace, which
  // copies() then makes.
  Op operand(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t at) {
    if (!bf16() || l.few || direct16(p, ld, cols)) return {p, ld, cols};
    const int64_t ldo = round8(cols);
    packs.p[packs.n++] = {p, ld, rows, cols, ws + at, ldo};
    return {ws + at, ldo, ldo};
  }
  muon_status_t copies() const {
    return packs.n ? launched("aligned copies", launch_ffn_pack(packs, st), st) : MUON_OK;
  }

  // The launch's products by plan g, and the sums of their splits.
  muon_status_t run(const char* what, int epi, bool ar, bool br, const TilePlan& g, FfnLaunch& L, int nprob) const {
    L.ldh = l.ldh;
    L.nprob = nprob;
    L.splitTiles = g.per;
    float* part = (float*)(ws + l.part);
    for (int q = 0; q < nprob; ++q) {
      FfnProb& p = L.prob[q];
      const int64_t tn = epi == FFN_GLU ? g.tn / 2 : g.tn;  // a tile holds both projections' columns
      if (g.tm) L.tiles[q + 1] = L.tiles[q] + (int32_t)(tiles_of(p.M, g.tm) * tiles_of(p.N, tn) * g.splits);
      p.partN = round4(p.N) * (epi == FFN_GLU ? 2 : 1);
      p.part = g.splits > 1 ? part : nullptr;
      part += (size_t)g.splits * p.M * p.partN;
    }
    hipError_t e;
    if (!g.tm) e = launch_ffn_few(epi, bf16(), g.splits, L, st);
    else if (!bf16()) e = launch_ffn_tile32(epi, g.tm, ar, br, L, st);
    else if (epi == FFN_GLU) e = launch_ffn16_glu(g.tm, L, st);
    else if (epi == FFN_BACK) e = launch_ffn16_back(g.tm, L, st);
    else e = launch_ffn16_store(g.tm, ar, br, L, st);
    const muon_status_t s = launched(what, e, st);
    if (s != MUON_OK || g.splits == 1) return s;
    return launched("sum of the k splits", launch_ffn_join(epi, bf16(), g.splits, L, st), st);
  }
};

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status_t muon_embedding(const void* ids, int32_t id_bytes, int64_t tokens, const void* weight,
                             int64_t ld_weight, int64_t vocab, int64_t dim, float scale, void* out,
                             int64_t ld_out, muon_dtype_t dtype, void* stream) {
  return guarded([&]() -> muon_status_t {
    Args a;
    a.size("tokens", tokens, 0, kMaxTokens);
    a.size("vocab", vocab, 1, kMaxVocab);
    a.size("dim", dim, 1, kMaxWidth);
    a.dtype("dtype", dtype);
    if (id_bytes != 4 && id_bytes != 8) a.fail(MUON_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
    if (!std::isfinite(scale)) a.fail(MUON_ERR_INVALID_ARG, "scale not finite");
    if (a.ok()) {
      const size_t e = esize(dtype);
      a.matrix("ids", ids, tokens > 0, tokens, tokens, id_bytes, false);
      a.matrix("weight", weight, tokens > 0 ? vocab : 0, dim, ld_weight, e, false);
      a.matrix("out", out, tokens, dim, ld_out, e, true);
    }
    a.aliases();
    if (!a.ok()) return a.report();
    if (tokens == 0) return MUON_OK;
    const muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    const size_t e = esize(dtype);
    EmbedLaunch L{ids, id_bytes == 8, dtype == MUON_DTYPE_BF16, tokens, vocab, dim, weight, ld_weight,
                  out, ld_out, scale,
                  whole_chunks(weight, ld_weight, dim, e) && whole_chunks(out, ld_out, dim, e)};
    return launched("embedding", launch_embedding(L, (hipStream_t)stream), (hipStream_t)stream);
  });
}

muon_status_t muon_embedding_grad_workspace_size(int64_t tokens, int64_t vocab, int64_t dim,
                                                 size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    Args a;
    a.size("tokens", tokens, 0, kMaxTokens);
    a.size("vocab", vocab, 1, kMaxVocab);
    a.size("dim", dim, 1, kMaxWidth);
    if (!bytes) a.fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    if (!a.ok()) return a.report();
    *bytes = embed_layout(tokens, dim).total;
    return MUON_OK;
  });
}

muon_status_t muon_embedding_grad(const void* dy, int64_t ld_dy, const void* ids, int32_t id_bytes,
                                  int64_t tokens, int64_t vocab, int64_t dim, float scale,
                                  void* dweight, int64_t ld_dweight, muon_dtype_t dtype,
                                  muon_dtype_t dweight_dtype, int32_t accumulate, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    Args a;
    a.size("tokens", tokens, 0, kMaxTokens);
    a.size("vocab", vocab, 1, kMaxVocab);
    a.size("dim", dim, 1, kMaxWidth);
    a.dtype("dtype", dtype);
    a.dtype("dweight_dtype", dweight_dtype);
    if (id_bytes != 4 && id_bytes != 8) a.fail(MUON_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
    if (!std::isfinite(scale)) a.fail(MUON_ERR_INVALID_ARG, "scale not finite");
    EmbedLayout lay{};
    if (a.ok()) {
      lay = embed_layout(tokens, dim);
      a.matrix("ids", ids, tokens > 0, tokens, tokens, id_bytes, false);
      a.matrix("dy", dy, tokens, dim, ld_dy, esize(dtype), false);
      a.matrix("dweight", dweight, vocab, dim, ld_dweight, esize(dweight_dtype), true);
      a.buffer("workspace", workspace, workspace_bytes, lay.total, true);
    }
    a.aliases();
    if (!a.ok()) return a.report();
    if (tokens == 0 && accumulate) return MUON_OK;
    const muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    char* ws = (char*)workspace;
    EmbedGradLaunch L{};
    L.ids = ids;
    L.id64 = id_bytes == 8;
    L.dyBf16 = dtype == MUON_DTYPE_BF16;
    L.dwBf16 = dweight_dtype == MUON_DTYPE_BF16;
    L.accumulate = accumulate != 0;
    L.tokens = tokens;
    L.vocab = vocab;
    L.dim = dim;
    L.dy = dy;
    L.ldy = ld_dy;
    L.dw = dweight;
    L.ldw = ld_dweight;
    L.scale = scale;
    L.vec = whole_chunks(dy, ld_dy, dim, esize(dtype));
    L.vecw = whole_chunks(dweight, ld_dweight, dim, esize(dweight_dtype));
    for (int i = 0; i < 2; ++i) {
      L.key[i] = (uint32_t*)(ws + lay.key[i]);
      L.idx[i] = (uint32_t*)(ws + lay.idx[i]);
    }
    L.counts = (uint32_t*)(ws + lay.counts);
    L.pieces = (float*)(ws + lay.pieces);
    return launched("embedding gradient", launch_embedding_grad(L, (hipStream_t)stream), (hipStream_t)stream);
  });
}

muon_status_t muon_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                            const void* weight, muon_dtype_t weight_dtype, float eps, void* y,
                            int64_t ld_y, void* sum, int64_t ld_sum, float* rstd, int64_t tokens,
                            int64_t dim, muon_dtype_t dtype, void* stream) {
  return guarded([&]() -> muon_status_t {
    Args a;
    a.size("tokens", tokens, 0, kMaxTokens);
    a.size("dim", dim, 1, kMaxWidth);
    a.dtype("dtype", dtype);
    a.dtype("weight_dtype", weight_dtype);
    if (!std::isfinite(eps) || eps < 0) a.fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (sum && !residual && tokens > 0) a.fail(MUON_ERR_INVALID_ARG, "sum without residual");
    const size_t e = esize(dtype);
    if (a.ok()) {
      a.matrix("x", x, tokens, dim, ld_x, e, false);
      if (residual) a.matrix("residual", residual, tokens, dim, ld_residual, e, false);
      a.matrix("weight", weight, tokens > 0, dim, dim, esize(weight_dtype), false);
      a.matrix("y", y, tokens, dim, ld_y, e, true);
      if (sum) a.matrix("sum", sum, tokens, dim, ld_sum, e, true);
      if (rstd) a.matrix("rstd", rstd, tokens > 0, tokens, tokens, 4, true);
    }
    a.aliases([](const char* out, const char* in) {
      return (out[0] == 'y' || out[0] == 's') && (in[0] == 'x' || std::string(in) == "residual");
    });
    if (!a.ok()) return a.report();
    if (tokens == 0) return MUON_OK;
    const muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    NormFwdLaunch L{x, residual, weight, y, sum, rstd, ld_x, ld_residual, ld_y, ld_sum, tokens, dim, eps,
                    dtype == MUON_DTYPE_BF16, weight_dtype == MUON_DTYPE_BF16,
                    whole_chunks(x, ld_x, dim, e) && whole_chunks(y, ld_y, dim, e) &&
                        (!residual || whole_chunks(residual, ld_residual, dim, e)) &&
                        (!sum || whole_chunks(sum, ld_sum, dim, e))};
    return launched("rms norm", launch_rms_norm(L, (hipStream_t)stream), (hipStream_t)stream);
  });
}

muon_status_t muon_rms_norm_grad_workspace_size(int64_t tokens, int64_t dim, size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    Args a;
    a.size("tokens", tokens, 0, kMaxTokens);
    a.size("dim", dim, 1, kMaxWidth);
    if (!bytes) a.fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    if (!a.ok()) return a.report();
    *bytes = tokens == 0 ? 0 : align256((size_t)rms_norm_grad_blocks(tokens) * dim * 4);
    return MUON_OK;
  });
}

muon_status_t muon_rms_norm_grad(const void* dy, int64_t ld_dy, const void* s, int64_t ld_s,
                                 const void* weight, muon_dtype_t weight_dtype, const float* rstd,
                                 const void* dsum, int64_t ld_dsum, void* dx, int64_t ld_dx,
                                 void* dweight, int32_t accumulate, int64_t tokens, int64_t dim,
                                 muon_dtype_t dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  return guarded([&]() -> muon_status_t {
    Args a;
    a.size("tokens", tokens, 0, kMaxTokens);
    a.size("dim", dim, 1, kMaxWidth);
    a.dtype("dtype", dtype);
    a.dtype("weight_dtype", weight_dtype);
    const size_t e = esize(dtype);
    size_t need = 0;
    if (a.ok()) {
      if (dweight && tokens > 0) need = align256((size_t)rms_norm_grad_blocks(tokens) * dim * 4);
      a.matrix("dy", dy, tokens, dim, ld_dy, e, false);
      a.matrix("s", s, tokens, dim, ld_s, e, false);
      a.matrix("weight", weight, tokens > 0, dim, dim, esize(weight_dtype), false);
      a.matrix("rstd", rstd, tokens > 0, tokens, tokens, 4, false);
      if (dsum) a.matrix("dsum", dsum, tokens, dim, ld_dsum, e, false);
      a.matrix("dx", dx, tokens, dim, ld_dx, e, true);
      if (dweight) a.matrix("dweight", dweight, 1, dim, dim, esize(weight_dtype), true);
      a.buffer("workspace", workspace, workspace_bytes, need, true);
    }
    a.aliases([](const char* out, const char* in) {
      return std::string(out) == "dx" && (std::string(in) == "dy" || std::string(in) == "dsum");
    });
    if (!a.ok()) return a.report();
    if (tokens == 0 && (!dweight || accumulate)) return MUON_OK;
    const muon_status_t st = check_device();
    if (st != MUON_OK) return st;
    NormGradLaunch L{};
    L.dy = dy;
    L.s = s;
    L.w = weight;
    L.dsum = dsum;
    L.rstd = rstd;
    L.dx = dx;
    L.dw = dweight;
    L.part = (float*)workspace;
    L.ldy = ld_dy;
    L.lds = ld_s;
    L.ldd = ld_dsum;
    L.ldx = ld_dx;
    L.tokens = tokens;
    L.dim = dim;
    L.blocks = tokens > 0 ? rms_norm_grad_blocks(tokens) : 0;
    L.bf16 = dtype == MUON_DTYPE_BF16;
    L.wBf16 = weight_dtype == MUON_DTYPE_BF16;
    L.vec = whole_chunks(dy, ld_dy, dim, e) && whole_chunks(s, ld_s, dim, e) && whole_chunks(dx, ld_dx, dim, e) &&
            (!dsum || whole_chunks(dsum, ld_dsum, dim, e));
    L.accumulate = accumulate != 0;
    return launched("rms norm gradient", launch_rms_norm_grad(L, (hipStream_t)stream), (hipStream_t)stream);
  });
}

muon_status_t muon_gated_ffn_saved_size(const muon_ffn_t* ffn, size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    Args a;
    ffn_sizes(a, ffn);
    if (!bytes) a.fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    if (!a.ok()) return a.report();
    *bytes = ffn_layout(*ffn, false).saved;
    return MUON_OK;
  });
}

muon_status_t muon_gated_ffn_workspace_size(const muon_ffn_t* ffn, int32_t grad, size_t* bytes) {
  return guarded([&]() -> muon_status_t {
    Args a;
    ffn_sizes(a, ffn);
    if (!bytes) a.fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    if (!a.ok()) return a.report();
    *bytes = ffn_layout(*ffn, grad != 0).total;
    return MUON_OK;
  });
}

muon_status_t muon_gated_ffn(const muon_ffn_t* ffn, const void* x, int64_t ld_x, void* y,
                             int64_t ld_y, void* saved, size_t saved_bytes, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    Args a;
    ffn_sizes(a, ffn);
    FfnLayout l{};
    if (a.ok()) {
      if (ffn->activation < MUON_ACT_SILU || ffn->activation > MUON_ACT_GELU_TANH)
        a.fail(MUON_ERR_INVALID_ARG, "unknown activation");
      l = ffn_layout(*ffn, false);
      const size_t e = esize(ffn->dtype);
      ffn_weights(a, *ffn);
      a.matrix("x", x, ffn->tokens, ffn->model, ld_x, e, false);
      a.matrix("y", y, ffn->tokens, ffn->model, ld_y, e, true);
      if (saved) a.buffer("saved", saved, saved_bytes, l.saved, true);
      a.buffer("workspace", workspace, workspace_bytes, l.total, true);
    }
    a.aliases();
    if (!a.ok()) return a.report();
    if (ffn->tokens == 0) return MUON_OK;
    muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    FfnCall call{*ffn, l, (char*)workspace, st};
    const bool bf16 = call.bf16();
    const int64_t T = ffn->tokens, D = ffn->model, F = ffn->hidden;
    const Op ox = call.operand(x, ld_x, T, D, l.x);
    const Op og = call.operand(ffn->w_gate, ffn->ld_gate, F, D, l.gate);
    const Op ou = call.operand(ffn->w_up, ffn->ld_up, F, D, l.up);
    const Op od = call.operand(ffn->w_down, ffn->ld_down, D, F, l.down);
    s = call.copies();
    if (s != MUON_OK) return s;
    void* h = saved ? (char*)saved + l.savedH : (char*)workspace + l.mid;
    FfnLaunch L{};
    L.act = ffn->activation;
    L.ab = saved ? (char*)saved + l.ab : nullptr;
    FfnProb& p = L.prob[0];
    p.A[0] = ox.p;
    p.lda = ox.ld;
    p.B[0] = og.p;
    p.B[1] = ou.p;
    p.ldb[0] = og.ld;
    p.ldb[1] = ou.ld;
    p.M = (int32_t)T;
    p.N = (int32_t)F;
    p.K[0] = (int32_t)ox.ext;
    set_out(p, h, l.ldh, bf16);
    s = call.run("gated projections", FFN_GLU, false, false, l.first, L, 1);
    if (s != MUON_OK) return s;
    FfnLaunch Y{};
    Y.outBf16 = bf16;
    FfnProb& d = Y.prob[0];
    d.A[0] = h;
    d.lda = l.ldh;
    d.B[0] = od.p;
    d.ldb[0] = od.ld;
    d.M = (int32_t)T;
    d.N = (int32_t)D;
    d.K[0] = (int32_t)od.ext;
    set_out(d, y, ld_y, bf16);
    return call.run("down projection", FFN_STORE, false, false, l.second, Y, 1);
  });
}

muon_status_t muon_gated_ffn_grad(const muon_ffn_t* ffn, const void* x, int64_t ld_x,
                                  const void* dy, int64_t ld_dy, const void* saved,
                                  size_t saved_bytes, const muon_ffn_grads_t* grads,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> muon_status_t {
    Args a;
    ffn_sizes(a, ffn);
    if (!grads) a.fail(MUON_ERR_INVALID_ARG, "grads is NULL");
    FfnLayout l{};
    bool wantW = false;
    if (a.ok()) {
      l = ffn_layout(*ffn, true);
      const size_t e = esize(ffn->dtype);
      wantW = grads->dw_gate || grads->dw_up || grads->dw_down;
      if (wantW) a.dtype("grad_dtype", grads->grad_dtype);
      const size_t eg = esize(grads->grad_dtype);
      ffn_weights(a, *ffn);
      a.matrix("x", x, ffn->tokens, ffn->model, ld_x, e, false);
      a.matrix("dy", dy, ffn->tokens, ffn->model, ld_dy, e, false);
      a.buffer("saved", saved, saved_bytes, l.saved, false);
      if (grads->dx) a.matrix("dx", grads->dx, ffn->tokens, ffn->model, grads->ld_dx, e, true);
      if (wantW) {
        a.matrix("dw_gate", grads->dw_gate, ffn->hidden, ffn->model, grads->ld_gate, eg, true);
        a.matrix("dw_up", grads->dw_up, ffn->hidden, ffn->model, grads->ld_up, eg, true);
        a.matrix("dw_down", grads->dw_down, ffn->model, ffn->hidden, grads->ld_down, eg, true);
      }
      a.buffer("workspace", workspace, workspace_bytes, l.total, true);
    }
    a.aliases();
    if (!a.ok()) return a.report();
    if (!wantW && (!grads->dx || ffn->tokens == 0)) return MUON_OK;
    if (ffn->tokens == 0 && grads->accumulate) return MUON_OK;
    muon_status_t s = check_device();
    if (s != MUON_OK) return s;
    const hipStream_t st = (hipStream_t)stream;
    FfnCall call{*ffn, l, (char*)workspace, st};
    const bool bf16 = call.bf16();
    const size_t e = esize(ffn->dtype);
    const char* sv = (const char*)saved;
    char* dgu = (char*)workspace + l.mid;
    const int32_t T = (int32_t)ffn->tokens, D = (int32_t)ffn->model, F = (int32_t)ffn->hidden;
    Op ox{x, ld_x, D}, oy{dy, ld_dy, D}, og{}, ou{}, od{};
    if (T > 0) {
      oy = call.operand(dy, ld_dy, T, D, l.dy);
      od = call.operand(ffn->w_down, ffn->ld_down, D, F, l.down);
      if (wantW) ox = call.operand(x, ld_x, T, D, l.x);
      if (grads->dx) {
        og = call.operand(ffn->w_gate, ffn->ld_gate, F, D, l.gate);
        ou = call.operand(ffn->w_up, ffn->ld_up, F, D, l.up);
      }
      s = call.copies();
      if (s != MUON_OK) return s;
      FfnLaunch L{};
      L.ab = (void*)(sv + l.ab);
      FfnProb& p = L.prob[0];
      p.A[0] = oy.p;
      p.lda = oy.ld;
      p.B[0] = od.p;
      p.ldb[0] = od.ld;
      p.extB = (int32_t)od.ext;
      p.M = T;
      p.N = F;
      p.K[0] = D;
      set_out(p, dgu, 2 * l.ldh, bf16);
      s = call.run("gradient of the gated product", FFN_BACK, false, true, l.first, L, 1);
      if (s != MUON_OK) return s;
    }
    if (T > 0 && grads->dx) {
      FfnLaunch L{};
      L.outBf16 = bf16;
      FfnProb& p = L.prob[0];
      p.A[0] = dgu;
      p.A[1] = dgu + l.ldh * e;
      p.lda = 2 * l.ldh;
      p.B[0] = og.p;
      p.B[1] = ou.p;
      p.ldb[0] = og.ld;
      p.ldb[1] = ou.ld;
      p.extB = (int32_t)og.ext;
      p.M = T;
      p.N = D;
      p.K[0] = p.K[1] = F;
      set_out(p, grads->dx, grads->ld_dx, bf16);
      s = call.run("gradient of the input", FFN_STORE, false, true, l.second, L, 1);
      if (s != MUON_OK) return s;
    }
    if (!wantW) return MUON_OK;
    FfnLaunch L{};
    L.outBf16 = grads->grad_dtype == MUON_DTYPE_BF16;
    L.accumulate = grads->accumulate != 0;
    // three products over the tokens in one launch
    for (int q = 0; q < 3; ++q) {
      FfnProb& p = L.prob[q];
      p.A[0] = q < 2 ? (const void*)(dgu + q * l.ldh * e) : oy.p;
      p.lda = q < 2 ? 2 * l.ldh : oy.ld;
      p.extA = (int32_t)(q < 2 ? l.ldh : oy.ext);
      p.B[0] = q < 2 ? ox.p : (const void*)(sv + l.savedH);
      p.ldb[0] = q < 2 ? ox.ld : l.ldh;
      p.extB = (int32_t)(q < 2 ? ox.ext : l.ldh);
      p.M = q < 2 ? F : D;
      p.N = q < 2 ? D : F;
      p.K[0] = T;
      set_out(p, q == 0 ? grads->dw_gate : q == 1 ? grads->dw_up : grads->dw_down,
              q == 0 ? grads->ld_gate : q == 1 ? grads->ld_up : grads->ld_down, L.outBf16);
    }
    return call.run("gradients of the weights", FFN_STORE, true, true, l.third, L, 3);
  });
}

}  // extern "C"
