// Differential attention, forward: with S_m = scale·Q_m·K_mᵀ for the two maps
// of a head, P_m = softmax(S_m) over the keys a row sees,
//   out = (P_1 − λ·P_2)·V = P_1·V − λ·(P_2·V).
//
// One pass over the keys with each map's running maximum and sum: the two
// products P_m·V are accumulated apart, since A = P_1 − λ·P_2 needs the final
// sums.  (Two passes, the first for the sums alone, would take as many
// products and twice the exponentials.)
//
// A wave has one map of 32·RS rows; RG groups of rows times two maps make a
// workgroup, whose waves share the tiles of K_1, K_2 and V in LDS (two
// buffers, loaded without passing through registers).  It forms the transposed
// scores K·Qᵀ, so that a lane holds scores of one row only: the maximum and
// sum run within the lane and one exchange between its two halves, and the
// probabilities are the next product's operand as they lie (Vᵀ·Pᵀ).  At the
// end the second map's wave hands λ·P_2·V over through LDS.
//
// Rounding: scores, maxima, sums and results are fp32; for bf16 tensors the
// probabilities are rounded to bf16 as operands of the second product.  Two sums
// of them run along: of the unrounded ones, for the log-sums that the backward
// pass recomputes probabilities from, and of the rounded ones, by which a result
// is divided.  Where one key has most of a row, the rounding of its probability
// then drops out; divided by the other sum, it would be an error of the whole
// result, much larger than the gradients of such a row's scores,
// P·(dA − δ), that the backward pass takes from it.  (With few rows they are not
// rounded but split in two, and the first sum serves for both.)
//
// Bound by the matrix unit and the exponentials beside it: a wave issues 24
// products of 32×32×16 for 2048 probabilities, two waves per SIMD.  4 × 4096
// tokens, 28 heads of 64 on 4, bf16, causal: 700 to 720 µs (1000 TFLOP/s of the
// four products) without the second sum and with the second map's result kept
// alone, 770 to 790 with both; comparing every maximum: 800 and more.  One token of
// 16384 keys, split over 512 workgroups: 12.3 µs (2.7 TB/s; 11.2 with rounded
// probabilities, an error of 2.2·10^-3 to 2.9·10^-3 instead of the output's own
// 1.7·10^-3; three tiles on their way at once instead of one: no faster), and 6 for the join.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attention.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

// Row blocks and tiles of a kernel: RS·32 rows per wave, RG groups of waves,
// BN keys per tile.
template <typename T, int DP, bool FEW> struct Fwd {
  static constexpr int kRS = !FEW && AT<T>::kBytes == 2 && DP == 64 ? 2 : 1;
  static constexpr int kRG = FEW ? 1 : 2;
  static constexpr int kBM = 32 * kRS * kRG;
  static constexpr int kWaves = 2 * kRG, kThreads = 64 * kWaves;
  static constexpr int kBN = AT<T>::kBytes == 2 && DP == 64 ? 64 : 32;
  static constexpr int kK = DP * AT<T>::kBytes, kV = 2 * kK;  // bytes of a row
  static constexpr int kStage = kBN * (2 * kK + kV);
};

template <typename T, int DP, bool FEW>
__global__ __launch_bounds__((Fwd<T, DP, FEW>::kThreads), 2) void attn_fwd(const AttnFwdLaunch L) {
  using F = Fwd<T, DP, FEW>;
  constexpr int RS = F::kRS, BN = F::kBN, E = AT<T>::kBytes;
  constexpr int NC = DP / AT<T>::kStep;   // steps over a head's values
  constexpr int NV = 2 * DP / 32;         // 32-column groups of V
  constexpr int SP = AT<T>::kSteps32;     // steps over 32 keys
  // With few rows the matrix unit waits for the loads anyway: a bf16 probability
  // is two operands, its rounding and what that leaves (16 bits of it).
  constexpr bool TWO = FEW && E == 2;
  __shared__ __attribute__((aligned(1024))) char lds[2 * F::kStage];
  __shared__ int odd[F::kWaves];

  const AttnShape& S = L.s;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int map = wave & 1, rg = wave >> 1;

  // this workgroup's combo, rows and split
  int id = blockIdx.x;
  const int combo = id % S.combos;
  id /= S.combos;
  const int split = id % L.splits;
  id /= L.splits;
  int tok0 = 0, nq = (int)S.nq, nk = (int)S.nk, at = 0;
  if (L.list.blocks) {
    const int n = *L.list.count;
    if (id >= n) return;
    const AttnBlock B = L.list.blocks[n - 1 - id];
    tok0 = B.tok;
    nq = B.n;
    nk = B.nk;
    at = B.at;
  } else {  // the rows that see most keys first
    at = (L.rowBlocks - 1 - id) * F::kBM;
  }
  const int batch = combo / S.kv, hk = combo % S.kv, G = S.group;
  const int rows = nq * G;  // of this sequence
  const int shift = nk - nq + 1;

  // each lane's rows: their token and head, and how many keys they see
  int64_t qoff[RS];
  int lim[RS], head[RS];
  bool valid[RS];
  int tok[RS];
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    const int row = at + (rg * RS + r) * 32 + (lane & 31);
    valid[r] = row < rows;
    tok[r] = row / G;
    const int g = row - tok[r] * G;
    head[r] = hk * G + g;
    lim[r] = !valid[r] ? 0 : S.causal ? min(max(tok[r] + shift, 0), nk) : nk;
    tok[r] += tok0;
    qoff[r] = batch * S.qs[0] + tok[r] * S.qs[1] + (2 * head[r] + map) * S.qs[2];
  }
  // keys any row of the workgroup sees, and those all of them see
  const int last = min(at + F::kBM, rows) - 1;
  const int most = S.causal ? min(max(last / G + shift, 0), nk) : nk;
  const int least = S.causal ? min(max(at / G + shift, 0), nk) : nk;
  int kBegin = 0, kEnd = most;
  if (L.splits > 1) {
    kBegin = split * L.splitKeys;
    kEnd = min(most, kBegin + L.splitKeys);
  }

  lu32x4 q[RS][NC];
#pragma unroll
  for (int r = 0; r < RS; ++r)
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      q[r][c] = lu32x4{0, 0, 0, 0};
      if (valid[r] && (2 * c + half) * 16 < S.dim * E)
        q[r][c] = *(const lu32x4*)((const char*)S.q + qoff[r] * E + (2 * c + half) * 16);
    }

  TileLoader<F::kK, BN, F::kWaves> ldk;
  TileLoader<F::kV, BN, F::kWaves> ldv;
  ldk.init(lane, wave, S.ks[1] * E, S.dim * E);
  ldv.init(lane, wave, S.vs[1] * E, 2 * S.dim * E);
  const char* k1 = (const char*)S.k + (batch * S.ks[0] + tok0 * S.ks[1] + 2 * hk * S.ks[2]) * E;
  const char* v0 = (const char*)S.v + (batch * S.vs[0] + tok0 * S.vs[1] + hk * S.vs[2]) * E;
  const uint32_t base = a_lds(lds);
  auto issue = [&](int key, uint32_t buf) __attribute__((always_inline)) {
    const char* k = k1 + (int64_t)key * S.ks[1] * E;
    ldk.issue(k, most - key, buf);
    ldk.issue(k + S.ks[2] * E, most - key, buf + BN * F::kK);
    ldv.issue(v0 + (int64_t)key * S.vs[1] * E, most - key, buf + 2 * BN * F::kK);
  };
  const RowReader<F::kK> rd(lane, map * (BN * F::kK));  // in the map's own keys
  const ColReader<T, F::kV> cd(lane);

  af32x16 o[RS][NV];
  float m[RS], l[RS], lr[RS], lag[RS];
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    m[r] = l[r] = lr[r] = 0.f;
    lag[r] = -1.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) o[r][n] = af32x16{};
  }

  // 32 keys of a tile.  Exponents refer to m, a maximum of keys gone by that may
  // lag behind the true one: as long as no 16 probabilities of a lane sum to more
  // than kLag, nothing is compared and nothing rescaled.
  constexpr float kLag = 1024.f;
  auto step = [&](uint32_t kt, uint32_t vt, int key, bool masked) __attribute__((always_inline)) {
    af32x16 s[RS];
#pragma unroll
    for (int r = 0; r < RS; ++r) s[r] = af32x16{};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const lu32x4 a = rd.get(kt, c);
#pragma unroll
      for (int r = 0; r < RS; ++r) s[r] = a_mma<T>(a, q[r][c], s[r]);
    }
    lu32x4 p[RS][SP], rest[TWO ? RS : 1][SP];
#pragma unroll
    for (int r = 0; r < RS; ++r) {
      __builtin_amdgcn_sched_barrier(0);  // (the rows' exponentials in turn: 2% of a packed batch's time)
      if (masked) {
        const int n = lim[r] - key - 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[r][i] = 8 * (i >> 2) + (i & 3) < n ? s[r][i] : kNegInf;
      }
      float e[16], sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        e[i] = a_exp2(s[r][i] * S.c - m[r]);
        sum += e[i];
      }
      if (__any(sum > lag[r])) {
        float mx = s[r][0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[r][i]);
        mx = a_half_max(mx) * S.c;
        // a row that has seen no key has m = 0, sums of 0 and no lag allowed
        const float mn = lag[r] < 0.f ? mx : fmaxf(m[r], mx);
        const bool seen = mn != kNegInf;
        const float f = lag[r] < 0.f ? 0.f : a_exp2(m[r] - mn);
        m[r] = seen ? mn : 0.f;
        lag[r] = seen ? kLag : -1.f;
        l[r] *= f;
        lr[r] *= f;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[r][n][i] *= f;
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          e[i] = a_exp2(s[r][i] * S.c - m[r]);
          sum += e[i];
        }
      }
      l[r] += sum;
#pragma unroll
      for (int t = 0; t < SP; ++t) {
        p[r][t] = a_operand<T>(e, t);
        if constexpr (TWO) {
          float d[16] = {};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t two = p[r][t][i / 2];
            d[8 * t + i] = e[8 * t + i] - __uint_as_float(i % 2 ? two & 0xffff0000u : two << 16);
          }
          rest[r][t] = a_operand<T>(d, t);
        } else if constexpr (E == 2) {
          lr[r] = a_operand_sum(p[r][t], lr[r]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < SP; ++t)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const lu32x4 a = cd.get(vt, t, n);
#pragma unroll
        for (int r = 0; r < RS; ++r) {
          o[r][n] = a_mma<T>(a, p[r][t], o[r][n]);
          if constexpr (TWO) o[r][n] = a_mma<T>(a, rest[r][t], o[r][n]);
        }
      }
  };

  // A tile of values of which some rows see only a part: an infinity or NaN is
  // added to the sums of the rows that see its key, and leaves the tile, where a
  // probability of 0 times it would reach the others.  Without one the look at the
  // tile is all (a block has one or two such tiles: 4 × 4096 tokens 755 µs without
  // the look, 751 to 773 with it; packed 218 and 221).
  auto part = [&](uint32_t vt, int key) __attribute__((always_inline)) {
    typedef __attribute__((address_space(3))) lu32x4* Chunk;
    constexpr int kPer = BN * F::kV / 16 / F::kThreads;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) top = a_top<T>(*(Chunk)(uintptr_t)(vt + (tid + i * F::kThreads) * 16), top);
    const bool any = __any(a_odd<T>(top));
    if (lane == 0) odd[wave] = any;
    a_meet();
    int all = 0;
#pragma unroll
    for (int w = 0; w < F::kWaves; ++w) all |= odd[w];
    if (__builtin_expect(!__builtin_amdgcn_readfirstlane(all), 1)) return;
    // as products that overflow, so that they take the sums' own place: of +-2^100
    // where an infinity of that sign (or a NaN: both) stands, and of 2^100 where seen
#pragma clang loop unroll(disable)
    for (int t = 0; t < BN / AT<T>::kStep; ++t) {
      lu32x4 seen[RS];
#pragma unroll
      for (int r = 0; r < RS; ++r) seen[r] = a_below<T>(lim[r] - key - AT<T>::kStep * t - 4 * half);
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const lu32x4 v = cd.get(vt, t, n);
#pragma unroll
        for (int sign = 0; sign < 2; ++sign) {
          const lu32x4 a = a_odd_of<T>(v, sign);
#pragma unroll
          for (int r = 0; r < RS; ++r) o[r][n] = a_mma<T>(a, seen[r], o[r][n]);
        }
      }
    }
    a_meet();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const Chunk c = (Chunk)(uintptr_t)(vt + (tid + i * F::kThreads) * 16);
      *c = a_finite<T>(*c);
    }
    a_meet();
  };

  if (kBegin < kEnd) issue(kBegin, base);
  // The two buffers by turns, their addresses constants: pairs of tiles that all rows
  // see whole, then the others.
  int key = kBegin;
  for (const int whole = min(least, kEnd); key + 2 * BN <= whole; key += 2 * BN) {
    a_for<0, 2>([&](auto bc) __attribute__((always_inline)) {
      constexpr int b = decltype(bc)::value;
      const uint32_t buf = base + b * F::kStage;
      a_landed();  // this tile; the other buffer is free
      if (b == 0 || key + 2 * BN < kEnd) issue(key + (b + 1) * BN, base + (1 - b) * F::kStage);
#pragma unroll
      for (int j = 0; j < BN; j += 32) step(buf + j * F::kK, buf + 2 * BN * F::kK + j * F::kV, key + b * BN + j, false);
    });
  }
  for (; key < kEnd; key += 2 * BN) {
    a_for<0, 2>([&](auto bc) __attribute__((always_inline)) {
      constexpr int b = decltype(bc)::value;
      const uint32_t buf = base + b * F::kStage;
      const int k0 = key + b * BN;
      if (k0 >= kEnd) return;
      a_landed();
      if (k0 + BN < kEnd) issue(k0 + BN, base + (1 - b) * F::kStage);
      if (least < most && k0 + BN > least) part(buf + 2 * BN * F::kK, k0);
#pragma unroll
      for (int j = 0; j < BN; j += 32) {
        if (k0 + j >= kEnd) break;
        step(buf + j * F::kK, buf + 2 * BN * F::kK + j * F::kV, k0 + j, k0 + j + 32 > least);
      }
    });
  }
  __syncthreads();

#pragma unroll
  for (int r = 0; r < RS; ++r) {
    l[r] = a_half_sum(l[r]);
    const float sum = E == 2 && !TWO ? a_half_sum(lr[r]) : l[r];
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;  // a row that sees no key: zeros
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[r][n][i] *= inv;
  }
  if (L.splits > 1) {
#pragma unroll
    for (int r = 0; r < RS; ++r) {
      if (!valid[r]) continue;
      const int64_t row = (int64_t)(tok[r]) * G + head[r] - hk * G;
      const int64_t slot = (((int64_t)split * S.combos + combo) * (S.nq * G) + row) * 2 + map;
      if (half == 0) L.partStat[slot] = l[r] == 0.f ? kNegInf : m[r] + a_log2(l[r]);
      float* d = L.part + slot * (2 * DP);
#pragma unroll
      for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(lf32x4*)(d + n * 32 + 8 * g + 4 * half) =
              lf32x4{o[r][n][4 * g], o[r][n][4 * g + 1], o[r][n][4 * g + 2], o[r][n][4 * g + 3]};
    }
    return;
  }

  // the second map's results pass to the wave of the first, λ times, register
  // by register
  constexpr int kWaveX = RS * NV * 4 * 1024;
  static_assert(F::kRG * kWaveX <= 2 * F::kStage, "exchange fits");
  lf32x4* x = (lf32x4*)(lds + rg * kWaveX) + lane;
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    const int64_t row = (int64_t)tok[r] * G + head[r] - hk * G, rowsAll = S.nq * G;
    if (S.stat && half == 0 && valid[r])  // a row that sees no key: +∞, so that its probabilities are 0
      S.stat[((int64_t)combo * 2 + map) * rowsAll + row] = l[r] == 0.f ? -kNegInf : m[r] + a_log2(l[r]);
    if (S.kept && (E == 2 || map == 1)) {
      const int64_t at = ((int64_t)combo * (E == 2 ? 2 : 1) + (E == 2 ? map : 0)) * rowsAll + row;
      float inv = 1.f;
      if constexpr (E == 2) {
        uint32_t top = 0;  // as whole numbers infinities and NaN are above all else
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) top = max(top, __float_as_uint(o[r][n][i]) & 0x7fffffffu);
        const Whole w(a_half_max(top));
        inv = w.inv;
        if (half == 0 && valid[r]) S.unit[at] = w.unit;
      }
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = E == 2 ? o[r][n][i] * inv : o[r][n][i];
        a_store_row<T, true>((char*)S.kept + at * S.pitch * E, v, n * 32, 2 * S.dim, true, valid[r], half);
      }
    }
    if (map == 1) {
      const float lam = valid[r] ? S.lam[head[r]] : 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          x[((r * NV + n) * 4 + g) * 64] = lf32x4{o[r][n][4 * g] * lam, o[r][n][4 * g + 1] * lam,
                                                  o[r][n][4 * g + 2] * lam, o[r][n][4 * g + 3] * lam};
      }
    }
  }
  __syncthreads();
  if (map == 1) return;
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    char* d = (char*)L.out + (batch * L.os[0] + tok[r] * L.os[1] + head[r] * L.os[2]) * E;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      float v[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const lf32x4 y = x[((r * NV + n) * 4 + g) * 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * g + i] = o[r][n][4 * g + i] - y[i];
      }
      a_store_row<T>(d, v, n * 32, 2 * S.dim, L.vec, valid[r], half);
    }
  }
}

// The splits' results of a row joined, a workgroup per row: the splits' weights
// from the logarithms of their sums, then both maps' columns, four a thread,
// the splits dealt out to as many groups of threads as there are and the groups
// added in order.
template <typename T, int DP, int THREADS> __global__ __launch_bounds__(THREADS) void attn_join(const AttnFwdLaunch L) {
  constexpr int E = AT<T>::kBytes, COLS = DP, GROUPS = THREADS / COLS;  // threads for 2 · 2·DP columns
  __shared__ float weight[2][kMaxSplits], top[2], sums[2];
  __shared__ uint32_t most[2];  // the largest magnitude of a map's results
  __shared__ lf32x4 part[GROUPS][COLS];
  const AttnShape& S = L.s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t rows = S.nq * S.group, all = rows * S.combos, id = blockIdx.x;
  const int combo = (int)(id / rows);
  const int64_t row = id - combo * rows;
  const int64_t tok = row / S.group;
  const int batch = combo / S.kv, head = (combo % S.kv) * S.group + (int)(row - tok * S.group);
  if (tid < 2) most[tid] = 0;
  if (wave < 2) {  // a wave per map
    float m = kNegInf, l = 0.f;
    for (int s = lane; s < L.splits; s += 64) {
      const float v = L.partStat[(s * all + id) * 2 + wave];
      weight[wave][s] = v;
      m = v != v || v > m ? v : m;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float v = __shfl_xor(m, o, 64);
      m = v != v || v > m ? v : m;
    }
    for (int s = lane; s < L.splits; s += 64) {
      const float w = m == kNegInf ? 0.f : a_exp2(weight[wave][s] - m);
      weight[wave][s] = w;
      l += w;
    }
    l = l_wave_sum(l);
    if (lane == 0) {
      top[wave] = m;
      sums[wave] = l;
      if (S.stat) S.stat[((int64_t)combo * 2 + wave) * rows + row] = m == kNegInf ? -kNegInf : m + a_log2(l);
    }
  }
  __syncthreads();
  const int col = tid % COLS, group = tid / COLS, map = col / (COLS / 2);
  const float* d = L.part + id * (4 * DP) + col * 4;
  lf32x4 res = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = group; s < L.splits; s += GROUPS) {
    const float w = weight[map][s];
    const lf32x4 v = *(const lf32x4*)(d + s * all * (4 * DP));
    // a split whose keys the row does not see left zeros
#pragma unroll
    for (int i = 0; i < 4; ++i) res[i] += w * v[i];
  }
  part[group][col] = res;
  __syncthreads();
  const bool mine = tid < COLS / 2;
  lf32x4 r[2];
  if (mine) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      lf32x4 s = part[0][m * (COLS / 2) + tid];
      for (int g = 1; g < GROUPS; ++g) s += part[g][m * (COLS / 2) + tid];
      const float inv = top[m] == kNegInf ? 0.f : 1.f / sums[m];
      uint32_t largest = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[m][i] = s[i] * inv;
        largest = max(largest, __float_as_uint(r[m][i]) & 0x7fffffffu);
      }
      if (E == 2 && S.kept) atomicMax(&most[m], largest);  // (a maximum: in any order)
    }
    const float lam = S.lam[head];
    char* o = (char*)L.out + (batch * L.os[0] + tok * L.os[1] + head * L.os[2]) * E;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (tid * 4 + i < 2 * S.dim) LType<T>::put(o, tid * 4 + i, r[0][i] - lam * r[1][i]);
  }
  if (!S.kept) return;
  __syncthreads();
  if (!mine || tid * 4 >= S.pitch) return;
  if constexpr (E == 2) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int64_t at = ((int64_t)combo * 2 + m) * rows + row;
      const Whole w(most[m]);
      if (tid == 0) S.unit[at] = w.unit;
      *(lu32x2*)((char*)S.kept + (at * S.pitch + tid * 4) * E) =
          lu32x2{a_pair_whole(r[m][0] * w.inv, r[m][1] * w.inv), a_pair_whole(r[m][2] * w.inv, r[m][3] * w.inv)};
    }
  } else {
    *(lf32x4*)((char*)S.kept + (id * S.pitch + tid * 4) * E) = r[1];
  }
}

template <typename T, int DP, bool FEW> hipError_t run(const AttnFwdLaunch& L, hipStream_t st) {
  attn_fwd<T, DP, FEW><<<dim3((unsigned)(L.s.combos * L.rowBlocks * L.splits)), Fwd<T, DP, FEW>::kThreads, 0, st>>>(L);
  return hipGetLastError();
}
template <typename T, int DP> hipError_t join(const AttnFwdLaunch& L, hipStream_t st) {
  const int64_t rows = L.s.nq * L.s.group * L.s.combos;
  // a row's reads all in flight where there are many splits, and so few rows (one
  // token, 128 splits: 7.6 µs by four waves a row, 6.0 by sixteen)
  if (L.splits >= 32) attn_join<T, DP, 1024><<<dim3((unsigned)rows), 1024, 0, st>>>(L);
  else attn_join<T, DP, 256><<<dim3((unsigned)rows), 256, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace

int attn_fwd_rows(bool bf16, int dp, bool few) { return few ? 32 : bf16 && dp == 64 ? 128 : 64; }
int attn_fwd_keys(bool bf16, int dp) { return bf16 && dp == 64 ? 64 : 32; }
static_assert(Fwd<Bf16, 64, false>::kBM == 128 && Fwd<Bf16, 128, false>::kBM == 64 && Fwd<float, 64, false>::kBM == 64 &&
                  Fwd<float, 128, false>::kBM == 64 && Fwd<float, 128, true>::kBM == 32 && Fwd<Bf16, 64, true>::kBM == 32,
              "attn_fwd_rows");
static_assert(Fwd<Bf16, 64, false>::kBN == 64 && Fwd<Bf16, 128, false>::kBN == 32 && Fwd<float, 64, true>::kBN == 32,
              "attn_fwd_keys");

hipError_t launch_attn_fwd(bool bf16, int dp, bool few, const AttnFwdLaunch& L, hipStream_t st) {
  if (bf16) {
    if (dp == 64) return few ? run<Bf16, 64, true>(L, st) : run<Bf16, 64, false>(L, st);
    return few ? run<Bf16, 128, true>(L, st) : run<Bf16, 128, false>(L, st);
  }
  if (dp == 64) return few ? run<float, 64, true>(L, st) : run<float, 64, false>(L, st);
  return few ? run<float, 128, true>(L, st) : run<float, 128, false>(L, st);
}

hipError_t launch_attn_join(bool bf16, int dp, const AttnFwdLaunch& L, hipStream_t st) {
  if (bf16) return dp == 64 ? join<Bf16, 64>(L, st) : join<Bf16, 128>(L, st);
  return dp == 64 ? join<float, 64>(L, st) : join<float, 128>(L, st);
}

}  // namespace muon
