// Differential attention, gradient of the queries: for a row
//   dS_1 = P_1·(dA − δ_1),  dS_2 = −λ·P_2·(dA − δ_2),  dA = dO·Vᵀ,
//   dQ_m = scale·dS_m·K_m,
// with P_m = exp2(c·S_m − L_m) recomputed from the saved log-sums.
//
// A wave has 32 rows (Q of both maps and dO in registers as operands) and runs
// over the tiles of K_1, K_2 and V in LDS.  Everything is formed transposed, a
// lane holding values of one row only: S_mᵀ = K_m·Q_mᵀ, dAᵀ = V·dOᵀ, and dS_mᵀ
// serves as it lies in dQ_mᵀ = K_mᵀ·dS_mᵀ.  dA is formed once for both maps,
// and −λ·scale is applied to the sums.
//
// λ's gradient is −Σ P_2·dA = −Σ_rows (δ_2 + Σ_j P_2·(dA − δ_2)): the second
// sum, of the unrounded terms, takes out what δ_2 lacks (it came from rounded
// probabilities), so the result is accurate to fp32.
//
// Bound by the matrix unit, as attn_dkv: 24 products a tile of 32 keys beside
// some 130 operations and 32 exponentials, two waves per SIMD (64-wide bf16).
// 4 × 4096 tokens, 28 heads of 64 on 4: 800 µs, 900 TFLOP/s.  Where there are
// fewer blocks than twice the CUs' places, equal stretches of tiles as in
// attn_dkv (333 tokens, fp32: 78 µs by blocks, 28 + 10 in stretches).  A packed
// batch of more blocks keeps them whole, unlike there (8192 tokens in 11
// documents: 232 µs, in stretches 349).  dS between the products instead of all
// at once: 793 µs, the same.
#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

template <typename T, int DP> struct Dq {
  static constexpr int kWaves = 4, kThreads = 256;
  static constexpr int kBN = 32;
  static constexpr int kK = DP * AT<T>::kBytes, kV = 2 * kK;
  static constexpr int kStage = kBN * (2 * kK + kV);
  // 64-wide bf16: dO is an operand in LDS, not in registers, which leaves room
  // for operands read ahead at two waves per SIMD
  static constexpr bool kInLds = AT<T>::kBytes == 2 && DP == 64;
  static constexpr int kWavesPerSimd = kInLds ? 2 : 1;
  static constexpr int kAhead = 8;
  static constexpr int kOut = kInLds ? kDqRows * kV : 0;  // bytes of dO
};

// MAPS: bit 0 the first map, bit 1 the second (and λ's gradient).
template <typename T, int DP, int MAPS>
__global__ __launch_bounds__(256, (Dq<T, DP>::kWavesPerSimd)) void attn_dq(const AttnGradLaunch L) {
  using F = Dq<T, DP>;
  constexpr bool k1st = MAPS & 1, k2nd = MAPS & 2;
  constexpr int BN = F::kBN, E = AT<T>::kBytes;
  constexpr int NC = DP / AT<T>::kStep, ND = DP / 32, SP = AT<T>::kSteps32;
  __shared__ __attribute__((aligned(1024))) char lds[2 * F::kStage + F::kOut];
  const AttnShape& S = L.s;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // one block of rows, all its key tiles, or an equal stretch of the tiles of
  // all blocks (dense: the rows that see most keys first)
  Stretch W(L.rowRuns, S.combos, blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8);  // neighbours on one XCD
  Piece P;
  while (W.next(L.rowRuns, S.combos, (L.rowRuns.blocks - 1 - (int)blockIdx.x / S.combos) * kDqRows, P)) {
  const int tok0 = P.tok, at = P.at;
  const int nq = L.packed ? P.n : (int)S.nq, nk = L.packed ? (P.inside ? P.n : 0) : (int)S.nk;
  const int batch = P.combo / S.kv, hk = P.combo % S.kv, G = S.group;
  const int rows = nq * G, shift = nk - nq + 1;
  const int row = at + wave * 32 + (lane & 31);
  const bool valid = row < rows;
  const int t = row / G, g = row - t * G, head = hk * G + g;
  const int lim = !valid ? 0 : S.causal ? min(max(t + shift, 0), nk) : nk;
  const int64_t tok = tok0 + t;
  const int last = min(at + kDqRows, rows) - 1;
  const int kSee = S.causal ? min(max(last / G + shift, 0), nk) : nk;
  const int kBegin = (int)P.begin * BN, kEnd = (int)min(P.end * BN, (int64_t)kSee);
  const int least = S.causal ? min(max(at / G + shift, 0), nk) : nk;

  lu32x4 q[2][NC], d[F::kInLds ? 1 : 2 * NC];
  {
    const char* p = (const char*)S.q + (batch * S.qs[0] + tok * S.qs[1] + 2 * head * S.qs[2]) * E;
    const char* o = (const char*)L.dout + (batch * L.gs[0] + tok * L.gs[1] + head * L.gs[2]) * E;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        q[m][c] = lu32x4{0, 0, 0, 0};
        if (valid && (2 * c + half) * 16 < S.dim * E)
          q[m][c] = *(const lu32x4*)(p + m * S.qs[2] * E + (2 * c + half) * 16);
      }
    if constexpr (!F::kInLds) {
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) {
        d[c] = lu32x4{0, 0, 0, 0};
        if (valid && (2 * c + half) * 16 < 2 * S.dim * E) d[c] = *(const lu32x4*)(o + (2 * c + half) * 16);
      }
    } else {  // this wave's rows of dO, into its own part of LDS
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) {
        lu32x4 x = {0, 0, 0, 0};
        if (valid && (2 * c + half) * 16 < 2 * S.dim * E) x = *(const lu32x4*)(o + (2 * c + half) * 16);
        RowReader<F::kV>(lane).put(a_lds(lds) + 2 * F::kStage + wave * 32 * F::kV, c, x);
      }
    }
  }
  const int64_t recAt = ((int64_t)batch * L.heads + head) * S.nq + tok;
  float l1 = -kNegInf, l2 = -kNegInf, d1 = 0.f, d2 = 0.f;
  if (valid) {
    const lf4 r = L.rec[recAt];
    l1 = r.v[0];
    l2 = r.v[1];
    d1 = r.v[2];
    d2 = r.v[3];
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
    ldk.issue(k, kSee - key, buf);
    ldk.issue(k + S.ks[2] * E, kSee - key, buf + BN * F::kK);
    ldv.issue(v0 + (int64_t)key * S.vs[1] * E, kSee - key, buf + 2 * BN * F::kK);
  };
  const RowReader<F::kK> rk(lane);
  const RowReader<F::kV> rv(lane);
  const ColReader<T, F::kK> ck(lane);

  af32x16 acc[2][ND];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < ND; ++n) acc[m][n] = af32x16{};
  float sum = 0.f;

  // The products of 32 keys in the order they run, each with the LDS operand it
  // reads: dA, S_1, S_2, dQ_1, dQ_2.  Operands are read AHEAD products ahead, past
  // the end those of the next 32 keys.
  // (where dO lies in LDS, its operand before each of V's)
  constexpr int AHEAD = F::kAhead, bS1 = (F::kInLds ? 4 : 2) * NC, bS2 = bS1 + (k1st ? NC : 0), bQ1 = bS2 + (k2nd ? NC : 0);
  constexpr int bQ2 = bQ1 + (k1st ? SP * ND : 0), ALL = bQ2 + (k2nd ? SP * ND : 0);
  static_assert(ALL % AHEAD == 0, "a step takes whole rounds of the ring");
  lu32x4 ring[AHEAD];
  auto read = [&](auto bc, auto stepc, auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value, at0 = decltype(bc)::value * F::kStage, s0 = decltype(stepc)::value * 32;
    const uint32_t kt = base + at0 + s0 * F::kK, vt = base + at0 + 2 * BN * F::kK + s0 * F::kV;
    if constexpr (F::kInLds && j < bS1) return rv.get(j % 2 ? vt : base + 2 * F::kStage + wave * 32 * F::kV, j / 2);
    else if constexpr (j < bS1) return rv.get(vt, j);
    else if constexpr (j < bS2) return rk.get(kt, j - bS1);
    else if constexpr (j < bQ1) return rk.get(kt + BN * F::kK, j - bS2);
    else if constexpr (j < bQ2) return ck.get(kt, (j - bQ1) / ND, (j - bQ1) % ND);
    else return ck.get(kt + BN * F::kK, (j - bQ2) / ND, (j - bQ2) % ND);
  };
  constexpr int STEPS = BN / 32;
  // step s of the tile in buffer b; `between` runs before the next tile's first read
  auto step = [&](auto bc, auto stepc, int key, bool masked, auto&& between) __attribute__((always_inline)) {
    constexpr int s = decltype(stepc)::value, b = decltype(bc)::value;
    constexpr auto nextB = std::integral_constant<int, s + 1 < STEPS ? b : 1 - b>{};
    constexpr auto nextS = std::integral_constant<int, (s + 1) % STEPS>{};
    af32x16 a{}, v{};
    lu32x4 op[2][SP], cur{};
    float e[16];
    const int on = lim - key - 4 * half;
    a_for<0, ALL>([&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
      if constexpr (j == ALL - AHEAD) between();
      const lu32x4 r = ring[j % AHEAD];
      if constexpr (j + AHEAD < ALL) ring[j % AHEAD] = read(bc, stepc, std::integral_constant<int, j + AHEAD>{});
      else ring[j % AHEAD] = read(nextB, nextS, std::integral_constant<int, j + AHEAD - ALL>{});
      if constexpr (j < bS1) {
        if constexpr (!F::kInLds) a = a_mma<T>(r, d[j], a);
        else if constexpr (j % 2) a = a_mma<T>(r, cur, a);
        else cur = r;
      } else if constexpr (j < bQ1) {
        constexpr int m = j >= bS2, c = j - (m ? bS2 : bS1);
        if constexpr (c == 0) v = af32x16{};
        v = a_mma<T>(r, q[m][c], v);
        if constexpr (c == NC - 1) {
          const float l = m ? l2 : l1, dd = m ? d2 : d1;
#pragma unroll
          for (int i = 0; i < 16; ++i) e[i] = a_exp2(v[i] * S.c - l) * (a[i] - dd);
          if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = 8 * (i >> 2) + (i & 3) < on ? e[i] : 0.f;
          }
          if constexpr (m) {
#pragma unroll
            for (int i = 0; i < 16; ++i) sum += e[i];
          }
#pragma unroll
          for (int u = 0; u < SP; ++u) op[m][u] = a_operand<T>(e, u);
        }
      } else {
        constexpr int m = j >= bQ2, i = j - (m ? bQ2 : bQ1), u = i / ND, n = i % ND;
        acc[m][n] = a_mma<T>(r, op[m][u], acc[m][n]);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  // Infinities and NaN of keys: of one that a row does not see dS is 0, but 0 times
  // them is not.  Where there are any among the keys that only some of the rows see,
  // this goes through those tiles: rows that see such a key become NaN (as their
  // log-sums are, but for scores of −∞), and its values leave the tile.
  uint32_t flag = 0;
  if (const int from = max(least, kBegin); from < kEnd && S.causal) {
    const uint8_t* o = L.oddKeys + (int64_t)P.combo * S.nk + tok0;
    if (from + lane < kEnd) flag = o[from + lane];
    for (int j = from + 64; j < kEnd; j += 64)
      if (j + lane < kEnd) flag |= o[j + lane];
  }
  auto clean = [&](uint32_t buf, int key) __attribute__((always_inline)) {
    static_assert(BN == 32, "a lane per key and map");
    typedef __attribute__((address_space(3))) lu32x4* Chunk;
    uint32_t top = 0;
#pragma clang loop unroll(disable)
    for (int c = 0; c < F::kK / 16; ++c) top = a_top<T>(*(Chunk)(uintptr_t)(buf + lane * F::kK + c * 16), top);
    const uint64_t bad = __ballot(a_odd<T>(top));
    const int n = lim - key;
    const uint32_t seen = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1;
    if ((uint32_t)bad & seen) l1 = __builtin_nanf("");
    if ((uint32_t)(bad >> 32) & seen) l2 = __builtin_nanf("");
    a_meet();
#pragma clang loop unroll(disable)
    for (int i = tid; i < 2 * BN * F::kK / 16; i += F::kThreads) {
      const Chunk c = (Chunk)(uintptr_t)(buf + i * 16);
      *c = a_finite<T>(*c);
    }
    a_meet();
  };

  __syncthreads();  // every wave has left the LDS of the piece before
  if (kBegin < kEnd) {
    issue(kBegin, base);
    a_landed();
    const bool look = kBegin + BN > least && __any(flag);
    if (kBegin + BN < kEnd) issue(kBegin + BN, base + F::kStage);
    if (__builtin_expect(look, 0)) clean(base, kBegin);
    a_for<0, AHEAD>([&](auto jc) __attribute__((always_inline)) {
      ring[decltype(jc)::value] = read(std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{}, jc);
    });
  }
  // the two buffers by turns, their addresses constants
  for (int key = kBegin; key < kEnd; key += 2 * BN) {
    a_for<0, 2>([&](auto bc) __attribute__((always_inline)) {
      constexpr int b = decltype(bc)::value;
      const int k0 = key + b * BN;
      if (k0 >= kEnd) return;
      a_for<0, STEPS>([&](auto sc) __attribute__((always_inline)) {
        constexpr int s = decltype(sc)::value;
        step(bc, sc, k0 + 32 * s, k0 + 32 * s + 32 > least, [&]() __attribute__((always_inline)) {
          if constexpr (s == STEPS - 1) {
            a_landed();  // the next tile is there, this one has been read by every wave
            const bool look = k0 + BN < kEnd && k0 + 2 * BN > least && __any(flag);
            if (k0 + 2 * BN < kEnd) issue(k0 + 2 * BN, base + b * F::kStage);
            if (__builtin_expect(look, 0)) clean(base + (1 - b) * F::kStage, k0 + BN);
          }
        });
      });
    });
  }
  if constexpr (k2nd) sum = a_half_sum(sum);
  if (P.slot >= 0) {
    float* o = L.rowPart + (P.slot * kDqRows + wave * 32 + (lane & 31)) * (2 * DP + 4);
    if (k2nd && valid && half == 0) o[2 * DP] = sum;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (!(MAPS >> m & 1)) continue;
#pragma unroll
      for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)  // rows that do not exist have a place too
          *(lf32x4*)(o + m * DP + n * 32 + 8 * i + 4 * half) =
              lf32x4{acc[m][n][4 * i], acc[m][n][4 * i + 1], acc[m][n][4 * i + 2], acc[m][n][4 * i + 3]};
    }
    continue;
  }
  if (k2nd && valid && half == 0) L.rowLam[recAt] = d2 + sum;
  if (!L.dq) continue;
  // of a row that sees one key alone P = 1 whatever the scores: no gradient
  const float f[2] = {L.scale, valid ? -S.lam[head] * L.scale : 0.f};
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    if (!(MAPS >> m & 1)) continue;
    char* o = (char*)L.dq + (batch * L.dqs[0] + tok * L.dqs[1] + (2 * head + m) * L.dqs[2]) * E;
#pragma unroll
    for (int n = 0; n < ND; ++n) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = lim > 1 ? acc[m][n][i] * f[m] : 0.f;
      a_store_row<T>(o, v, n * 32, S.dim, L.dqVec, valid, half);
    }
  }
  }
}

template <typename T, int DP, int MAPS> hipError_t run(const AttnGradLaunch& L, hipStream_t st) {
  attn_dq<T, DP, MAPS><<<dim3((unsigned)(L.rowRuns.streams ? L.rowRuns.streams : L.s.combos * L.rowRuns.blocks)), 256, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace

int attn_dq_keys(bool, int) { return 32; }
static_assert(Dq<Bf16, 64>::kBN == 32 && Dq<Bf16, 128>::kBN == 32 && Dq<float, 64>::kBN == 32 && Dq<float, 128>::kBN == 32,
              "attn_dq_keys");

hipError_t launch_attn_dq(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st) {
  if (bf16) return dp == 64 ? run<Bf16, 64, 3>(L, st) : run<Bf16, 128, 3>(L, st);
  if (dp == 64) return run<float, 64, 3>(L, st);
  // operands and sums of both maps are more than a wave's registers: a pass each
  const hipError_t e = run<float, 128, 1>(L, st);
  return e != hipSuccess ? e : run<float, 128, 2>(L, st);
}

}  // namespace muon
