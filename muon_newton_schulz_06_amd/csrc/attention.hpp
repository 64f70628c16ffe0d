// Launch descriptors of the attention half of a block (rotary positions,
// differential attention, dropout).  Descriptors are passed by value.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace muon {

struct lf4 {
  float v[4];
};
struct lu4 {
  uint32_t v[4];
};

// ----- rotary positions ------------------------------------------------------
struct RotarySide {
  const void* in;
  void* out;
  int64_t in_s[3], out_s[3];  // batch, token, head
  int32_t heads;
};
struct RotaryLaunch {
  RotarySide side[2];
  int32_t heads;  // of both sides
  int64_t batch, tokens;
  int32_t dim, rot;
  const double* freqs;
  const void* pos;  // null: start + token
  int32_t pos64;
  int64_t posBatch;  // stride between the rows of pos
  int64_t start;
  float scale;
  int32_t inverse, interleaved, copyRest;  // copyRest: values past `rot` are not in place already
  int32_t bf16, vec;                       // vec: elements per access
};
hipError_t launch_rotary(const RotaryLaunch& L, hipStream_t st);

// ----- dropout ---------------------------------------------------------------
struct DropoutLaunch {
  const void* x;
  const void* res;
  void* y;
  int64_t ldx, ldr, ldy;
  int64_t rows, cols;
  uint32_t key[2];
  uint64_t offset;
  const uint64_t* offsetDev;  // null, or added to offset
  uint32_t threshold;         // words below it drop
  int32_t none;               // nothing is kept
  float mult;
  int32_t bf16, vec;  // vec: one row of whole aligned 16-byte chunks
};
hipError_t launch_dropout(const DropoutLaunch& L, hipStream_t st);

// ----- differential attention ------------------------------------------------
// Rows of a (batch, key/value head) pair: row t·G + g is token t's query of
// head g of the pair's group of G heads, so a tile of rows shares its keys and
// values whatever the group, and one token's G heads fill a tile together.
// "Combo" numbers such a pair: batch·kv + head.

// Rows or keys of a workgroup of a packed batch: row (or key) `at` and the
// following ones of the sequence of n tokens that begins at token `tok`, with
// nk keys (n, or 0 outside every sequence).
struct AttnBlock {
  int32_t tok, n, nk, at;
};
struct AttnList {
  const AttnBlock* blocks;  // null: a dense batch
  const int32_t* count;
};

struct AttnShape {
  int32_t combos, kv, group;  // combos = batch · kv heads
  int64_t nq, nk;             // tokens of a batch's queries and keys
  int32_t dim;
  float c;  // scale · log2 e
  int32_t causal;
  const void *q, *k, *v;
  int64_t qs[3], ks[3], vs[3];  // batch, token, head strides, elements
  const float* lam;             // per head
  // saved: log2 of the maps' sums, [combo][map][row], and their results P_m·V
  // for the row sums of the backward pass (see attn_rows): fp32 the second map's,
  // [combo][row][pitch]; bf16 both, [combo][map][row][pitch], 16-bit whole
  // multiples of the row's unit, [combo][map][row]
  float* stat;
  float* unit;
  void* kept;
  int64_t pitch;
};

struct AttnFwdLaunch {
  AttnShape s;  // kept, stat null: not wanted
  void* out;
  int64_t os[3];
  int32_t vec;  // out rows take aligned 16-byte stores
  AttnList list;
  int32_t rowBlocks;  // per combo (packed: an upper bound)
  int32_t splits, splitKeys;
  // splits > 1: normalised results [split][combo][row][map][2·DP] and the
  // logarithms of their sums [split][combo][row][map]
  float *part, *partStat;
};
constexpr int kMaxSplits = 512;
// Rows of a workgroup, keys of its tiles.
int attn_fwd_rows(bool bf16, int dp, bool few);
int attn_fwd_keys(bool bf16, int dp);
hipError_t launch_attn_fwd(bool bf16, int dp, bool few, const AttnFwdLaunch& L, hipStream_t st);
hipError_t launch_attn_join(bool bf16, int dp, const AttnFwdLaunch& L, hipStream_t st);

// How the blocks (of rows or keys) of all combos are dealt out: a workgroup per
// block (streams = 0), or equal stretches of the tiles of all blocks, at least
// `least` tiles each.
struct AttnRuns {
  AttnList list;
  const int64_t* cum;  // tiles of the list's blocks before each, of all at [count]
  int32_t blocks;      // of a combo, without a list or as an upper bound
  int32_t streams, least;
};

struct AttnGradLaunch {
  AttnShape s;
  const void* dout;  // whole aligned chunks
  int64_t gs[3];
  const void* out;  // any alignment; read for fp32 only
  int64_t os[3];
  int32_t outVec;  // out is whole aligned chunks too
  // What the products need of a row, [batch][head][token]: {L1, L2, δ1, δ2}, and
  // for bf16 the same as operands of a product (see attn_dkv), two 16-byte records.
  lf4* rec;
  lu4 *recL, *recD;
  uint8_t* oddKeys;  // [combo][key]: whether a key holds an infinity or NaN; null: of no matter
  float* rowLam;     // per row δ2 as the products give it, [batch][head][token]
  void *dq, *dk, *dv;
  int64_t dqs[3], dks[3], dvs[3];
  int32_t dqVec;
  float* dlam;  // null: not wanted
  float scale;
  int32_t batch, heads;
  AttnRuns keyRuns, rowRuns;  // of attn_dkv, attn_dq
  int32_t packed;
  // sums of blocks that stretches share: attn_dkv [2·stretch][128 keys][4·DP] of
  // dk1, dk2, dv; attn_dq [2·stretch][128 rows][2·DP + 4] of dq1, dq2 and λ's
  float *part, *rowPart;
  int32_t joinKeys, joinRows;  // which of them there are
};
constexpr int kDkvKeys = 128, kDqRows = 128;
hipError_t launch_attn_dkv(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st);
int attn_dq_keys(bool bf16, int dp);  // of a tile
hipError_t launch_attn_dq(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st);
hipError_t launch_attn_grad_join(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st);
hipError_t launch_attn_dlam(const AttnGradLaunch& L, hipStream_t st);

// Block lists: units·n rows of a sequence of n tokens are cut into blocks of
// `per`.  Without offsets the tokens are one sequence.
struct AttnPrepLaunch {
  const int32_t* offsets;
  int32_t sequences;
  struct {
    AttnBlock* blocks;
    int32_t* count;
    int32_t tokens, units, per;
    // null, or tiles (one at least) of the blocks before each, of all at [count]:
    // of blocks of keys (units 1) tiles of 32 rows, of blocks of rows tiles of
    // `tile` keys
    int64_t* cum;
    int32_t tile;
  } list[2];
  int32_t group, causal;
  int64_t queries, keys;  // of the one sequence
  int32_t lists;
};
hipError_t launch_attn_prep(const AttnPrepLaunch& L, hipStream_t st);
// The row sums of the backward pass, and its lists beside them.
hipError_t launch_attn_rows(bool bf16, const AttnGradLaunch& L, const AttnPrepLaunch& P, hipStream_t st);

// Aligned copies [batch][token][head][pitch] of tensors whose rows are not
// whole aligned 16-byte chunks.
struct AttnCopy {
  const void* src;
  void* dst;
  int64_t s[3];
  int64_t batch, tokens;
  int32_t heads, dim, pitch;
};
struct AttnCopies {
  AttnCopy c[5];
  int32_t n;
};
hipError_t launch_attn_copy(bool bf16, const AttnCopies& K, hipStream_t st);

}  // namespace muon
