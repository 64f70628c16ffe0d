// Differential attention, gradients of the keys and values: over all rows that
// see a key, of all heads of its group,
//   dV = Σ (P_1 − λ·P_2)ᵀ·dO,   dK_m = scale·Σ dS_mᵀ·Q_m
// with dS as in attn_dq.hip.
//
// A wave has 32 keys: K_1, K_2, V as operands and the sums of dK_1, dK_2, dV
// in registers.  It runs over tiles of 32 tokens of one head (head by head, so
// λ is one number), Q_1, Q_2 and dO in LDS.  A lane holds values of one key,
// the registers run over rows: S_m = Q_m·K_mᵀ, dA = dO·Vᵀ, and the results serve
// as they lie in dV = Aᵀ·dO, dK_m = dS_mᵀ·Q_m.
//
// A row's statistics are then needed register by register.  For bf16 they
// enter through the matrix unit: −L_m/c, −δ_1 and −δ_2 are one more step of the
// products each, whose row operand holds the value as three bf16 (24 bits) and
// whose column operand is 1 there.
// That is 4 steps beside 32, instead of 16 reads of four values from LDS
// beside 32 and 48 subtractions.  fp32 does the same with products of 2.
//
// No atomics: a workgroup owns its keys.  Where there are few of them or they are
// seen by unequal numbers of rows (a packed batch), every workgroup takes an
// equal stretch of tiles instead, and the sums of blocks that stretches share are
// joined in order (8192 tokens in 11 documents, 28 heads of 64: 744 µs by blocks,
// 484 in stretches and 22 for the joins).
//
// Bound by the matrix unit and what shares the wave's time with it.  One wave per
// SIMD (K_m, V, the sums and a ring of operands read ahead fill its registers)
// issues 36 products of 32×32×16 a tile beside some 200 other operations and 32
// exponentials.  4 × 4096 tokens, 28 heads of 64 on 4, bf16: 1240 to 1380 µs, 700
// to 770 TFLOP/s of the five products (8192³ by the library: 1374).  Measured and
// not taken: two waves per SIMD with half the sums each (1384 to 1427 µs, the
// scores formed twice), the next tile's scores beside this tile's element-wise
// work (1304).  Without its loads it would take 190 µs less, without the
// exponentials 180, with a third of the LDS reads 150: no one of them bounds it.
#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

// What a pass makes (PART): bit 0 dV, bit 1 dK.
template <typename T, int DP> struct Dkv {
  static constexpr int kWaves = 4, kThreads = 256, kRows = 32;
  static constexpr int kK = DP * AT<T>::kBytes, kVB = 2 * kK;
  static constexpr int kStage = kRows * (2 * kK + kVB) + (AT<T>::kBytes == 2 ? 2048 : 1024);
  // Tiles come in groups with one wait and barrier each: three groups in LDS,
  // one in use, one there, one on its way; two single tiles where there is no
  // room for three.
  static constexpr int kGroup = 6 * kStage <= 160 * 1024 ? 2 : 1;
  static constexpr int kStages = 3 * kGroup * kStage <= 160 * 1024 ? 3 * kGroup : 2;
  // operands read ahead of their product, as registers allow
  static constexpr int kAhead = AT<T>::kBytes == 2 ? 6 : 2;
};

template <typename T, int DP, int PART>
__global__ __launch_bounds__(256, 1) void attn_dkv(const AttnGradLaunch L) {
  using F = Dkv<T, DP>;
  constexpr bool kV = PART & 1, kK = PART & 2;
  constexpr int kRecs = AT<T>::kBytes == 2 ? 2 : 1;  // loads of the records
  constexpr int E = AT<T>::kBytes, NC = DP / AT<T>::kStep, ND = DP / 32, SP = AT<T>::kSteps32;
  constexpr int RQ = F::kRows * F::kK, RECS = 2 * RQ + F::kRows * F::kVB;  // bytes of a Q tile; where the records lie
  __shared__ __attribute__((aligned(1024))) char lds[F::kStages * F::kStage];
  const AttnShape& S = L.s;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // What this workgroup makes: one block of keys, all its row tiles; or, where
  // the blocks are few or unequal, an equal stretch of all tiles of all blocks
  // one after another, which may begin or end inside a block.
  Stretch W(L.keyRuns, S.combos, blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8);  // neighbours on one XCD
  Piece P;
  // (dense: the keys that most rows see first)
  while (W.next(L.keyRuns, S.combos, blockIdx.x / S.combos * kDkvKeys, P)) {
  const int tok0 = P.tok, nq = L.packed ? P.n : (int)S.nq, nk = L.packed ? P.n : (int)S.nk, at = P.at;
  const int batch = P.combo / S.kv, hk = P.combo % S.kv, G = S.group;
  const int shift = nk - nq + 1;
  const int key0 = at + wave * 32, key = key0 + (lane & 31);
  const bool valid = key < nk;

  lu32x4 k[2][NC], v[2 * NC];
  {
    const char* p = (const char*)S.k + (batch * S.ks[0] + (int64_t)(tok0 + key) * S.ks[1] + 2 * hk * S.ks[2]) * E;
    const char* o = (const char*)S.v + (batch * S.vs[0] + (int64_t)(tok0 + key) * S.vs[1] + hk * S.vs[2]) * E;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        k[m][c] = lu32x4{0, 0, 0, 0};
        if (valid && (2 * c + half) * 16 < S.dim * E)
          k[m][c] = *(const lu32x4*)(p + m * S.ks[2] * E + (2 * c + half) * 16);
      }
    if constexpr (kK) {
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) {
        v[c] = lu32x4{0, 0, 0, 0};
        if (valid && (2 * c + half) * 16 < 2 * S.dim * E) v[c] = *(const lu32x4*)(o + (2 * c + half) * 16);
      }
    }
  }

  // row tiles: tokens from the first that sees a key of the workgroup
  const int first = S.causal ? max(at - shift + 1, 0) & ~31 : 0;
  const int perHead = P.inside && nq > first ? (nq - first + 31) / 32 : 0;
  const int begin = (int)P.begin, end = (int)min(P.end, (int64_t)perHead * G);

  TileLoader<F::kK, F::kRows, F::kWaves> ldq;
  TileLoader<F::kVB, F::kRows, F::kWaves> ldd;
  ldq.init(lane, wave, S.qs[1] * E, S.dim * E);
  ldd.init(lane, wave, L.gs[1] * E, 2 * S.dim * E);
  const char* q0 = (const char*)S.q + (batch * S.qs[0] + tok0 * S.qs[1] + 2 * hk * G * S.qs[2]) * E;
  const char* d0 = (const char*)L.dout + (batch * L.gs[0] + tok0 * L.gs[1] + hk * G * L.gs[2]) * E;
  const int64_t rec0 = ((int64_t)batch * L.heads + hk * G) * S.nq + tok0;
  const uint32_t base = a_lds(lds);
  // The next tile to load: head g, tokens from t.  Past the last tile the loads
  // deliver zeros.
  struct Place {
    int g, t;
  };
  auto next = [&](Place& p) __attribute__((always_inline)) {
    p.t += 32;
    if (p.t >= nq) {
      p.t = first;
      ++p.g;
    }
  };
  Place now{0, first};
  if (begin < end) now = Place{begin / perHead, first + 32 * (begin % perHead)};
  Place load = now;
  int filled = begin;
  const int64_t qStep = 32 * S.qs[1] * E, dStep = 32 * L.gs[1] * E;
  const char *q, *d, *rec;
  auto locate = [&]() __attribute__((always_inline)) {
    q = q0 + (load.t * S.qs[1] + 2 * load.g * S.qs[2]) * E;
    d = d0 + (load.t * L.gs[1] + load.g * L.gs[2]) * E;
    rec = (const char*)(E == 4 ? (const void*)L.rec : wave == 0 ? (const void*)L.recL : (const void*)L.recD) +
          (rec0 + load.g * S.nq + load.t) * 16;
  };
  locate();
  auto issue = [&](uint32_t buf) __attribute__((always_inline)) {
    const int left = filled < end ? nq - load.t : 0;
    if (left >= 32) {
      ldq.issue(q, buf);
      ldq.issue(q + S.qs[2] * E, buf + RQ);
      ldd.issue(d, buf + 2 * RQ);
    } else {
      ldq.issue(q, left, buf);
      ldq.issue(q + S.qs[2] * E, left, buf + RQ);
      ldd.issue(d, left, buf + 2 * RQ);
    }
    // the records: bf16 recL by wave 0, recD by wave 1; fp32 rec by wave 0
    // (lanes past 31 deliver zeros behind the 32 records)
    if (wave < kRecs)
      f_dma16(__builtin_amdgcn_readfirstlane(buf + RECS + wave * 1024),
              lane < 32 && lane < left ? (uint32_t)lane * 16 : kFfnNowhere, f_buffer((uint64_t)rec));
    ++filled;
    const int g = load.g;
    next(load);
    if (load.g != g) {
      locate();
    } else {
      q += qStep;
      d += dStep;
      rec += 512;
    }
  };
  const RowReader<F::kK> rq(lane);
  const RowReader<F::kVB> rd(lane);
  const ColReader<T, F::kK> cq(lane);
  const ColReader<T, F::kVB> cd(lane);

  // column operands of the statistics' steps: which of a record's values count
  lu32x4 one0 = {0, 0, 0, 0}, one3 = {0, 0, 0, 0};
  if (half == 0) {
    one0 = lu32x4{0x3f803f80u, 0x00003f80u, 0u, 0u};
    one3 = lu32x4{0u, 0x3f800000u, 0x3f803f80u, 0u};
  }
  const float invc = -1.f / S.c;

  af32x16 dk[2][ND], dv[2 * ND];
#pragma unroll
  for (int n = 0; n < ND; ++n) dk[0][n] = dk[1][n] = dv[n] = dv[ND + n] = af32x16{};

  // A tile's products in the order they run, each with the LDS operand it
  // reads: S_1, S_2 (their statistics last), dA and its statistics, dV, dK_1 and
  // dK_2.  Operands are read kAhead products ahead, past the tile's end those
  // of the next tile; element-wise work stands between the products, where it
  // runs beside them.
  constexpr int nS = NC + 1, nA = kK ? 2 * NC + 1 : 0, nV = kV ? SP * 2 * ND : 0, nK = kK ? SP * ND : 0;
  constexpr int bS2 = nS, bA = bS2 + nS, bV = bA + nA, bK1 = bV + nV, bK2 = bK1 + nK;
  constexpr int ALL = bK2 + nK, AHEAD = F::kAhead;
  constexpr int PERIOD = (ALL + AHEAD - 1) / AHEAD * AHEAD;  // a tile's places in the ring of operands, some idle
  constexpr bool kAcross = F::kStages >= 3;  // the next tile is there before this one ends
  auto read = [&](auto stage, auto jc) __attribute__((always_inline)) {
    constexpr int j = decltype(jc)::value;
    const uint32_t buf = base + decltype(stage)::value * F::kStage;
    const uint32_t rec = buf + RECS + (lane & 31) * 16;
    if constexpr (j < bS2) {
      if constexpr (j < NC) return rq.get(buf, j);
      else return *(a_lds_u4)(uintptr_t)rec;
    } else if constexpr (j < bA) {
      if constexpr (j - bS2 < NC) return rq.get(buf + RQ, j - bS2);
      else return *(a_lds_u4)(uintptr_t)rec;
    } else if constexpr (j < bV) {
      if constexpr (j - bA < 2 * NC) return rd.get(buf + 2 * RQ, j - bA);
      else return *(a_lds_u4)(uintptr_t)(E == 2 ? rec + 1024 : rec);
    } else if constexpr (j < bK1) {
      constexpr int u = (j - bV) / (2 * ND), n = (j - bV) % (2 * ND);
      return cd.get(buf + 2 * RQ, u, n);
    } else {
      constexpr int m = j >= bK2, i = j - (m ? bK2 : bK1), u = i / ND, n = i % ND;
      return cq.get(buf + m * RQ, u, n);
    }
  };
  // Rows with an infinity or NaN: for the keys that a row does not see its
  // probabilities and dS are 0, but 0 times these is not.  So the odd values leave a
  // row of dO (dS is NaN by δ; dV follows behind the tiles), and a row of Q leaves the
  // tile where its log-sum is not finite (P is NaN, ∞ or 0 by that), once every wave has
  // its scores.  All waves do so alike, before their products over the rows.
  bool odd = false;
  constexpr int kLook = kK ? bA - 1 : NC;  // a product that reads the records
  static_assert((kV ? bV : bK1) - AHEAD > kLook, "rows are clean before they are read as columns");
  auto clean = [&](uint32_t buf, uint32_t bad) __attribute__((always_inline)) {
    odd = true;
    if constexpr (kK) a_meet();
#pragma clang loop unroll(disable)
    for (int c = 0; c < 2 * NC; ++c) {
      if (kK && c < NC && (bad & 1)) rq.put(buf, c, lu32x4{0, 0, 0, 0});
      if (kK && c < NC && (bad & 2)) rq.put(buf + RQ, c, lu32x4{0, 0, 0, 0});
      if (kV && bad) rd.put(buf + 2 * RQ, c, a_finite<T>(rd.get(buf + 2 * RQ, c)));
    }
  };
  auto look = [&](uint32_t buf, lu32x4 rec) __attribute__((always_inline)) {
    uint32_t bad = rec[3];
    if constexpr (E == 4)
      bad = a_bad_row(__uint_as_float(rec[0]), __uint_as_float(rec[1]), __uint_as_float(rec[2]), __uint_as_float(rec[3]));
    if (__builtin_expect(__any(bad), 0)) clean(buf, bad);
  };
  lu32x4 ring[AHEAD];
  // −L/c is finite, since an infinity would meet zeros in the product; a NaN stays
  auto bounded = [](float x) __attribute__((always_inline)) { return x < -1e30f ? -1e30f : x; };
  const float unit = half ? 0.f : 1.f;
  // one statistics step: record values 0, 1, 2 (first) or 3, 4, 5 as three bf16, or fp32 value `at` times f
  auto stat = [&](lu32x4 r, auto first, float value, af32x16 c) __attribute__((always_inline)) {
    if constexpr (E == 2) return a_mma<T>(r, decltype(first)::value ? one0 : one3, c);
    else return __builtin_amdgcn_mfma_f32_32x32x2f32(value, unit, c, 0, 0, 0);
  };
  auto tile = [&](auto stage, float lam, int t, int rows, bool masked, auto&& between) __attribute__((always_inline)) {
    constexpr auto after = std::integral_constant<int, (decltype(stage)::value + 1) % F::kStages>{};

    af32x16 s1{}, s2{}, a1{}, a2{};
    float p1[16], p2[16], p[16];
    lu32x4 op{};
    // elements [16·i/n, 16·(i+1)/n) of an element-wise step spread over n products
    auto spread = [&](auto ic, auto nc, auto&& f) __attribute__((always_inline)) {
      constexpr int i = decltype(ic)::value, n = decltype(nc)::value;
      if constexpr (i >= 0 && i < n) {
#pragma unroll
        for (int e = 16 * i / n; e < 16 * (i + 1) / n; ++e) f(e);
      }
    };
    auto first = [&](int e) __attribute__((always_inline)) { p1[e] = a_exp2(s1[e] * S.c); };
    auto second = [&](int e) __attribute__((always_inline)) { p2[e] = -lam * a_exp2(s2[e] * S.c); };
    auto grads = [&](int e) __attribute__((always_inline)) {
      p1[e] *= a1[e];
      p2[e] *= a2[e];
    };
    // row t + i sees this lane's key if key < t + i + shift; of a row that sees
    // one key alone P = 1 whatever the scores, and dS = 0
    const int n0 = S.causal ? key - shift - t - 4 * half : -1;
    const int lone = (S.causal ? 1 - shift - t : -1) - 4 * half;
    a_for<0, PERIOD>([&](auto jc) __attribute__((always_inline)) {
      constexpr int j = decltype(jc)::value;
      if constexpr (j == PERIOD - AHEAD) between();
      const lu32x4 r = ring[j % AHEAD];
      if constexpr (j + AHEAD < ALL) ring[j % AHEAD] = read(stage, std::integral_constant<int, j + AHEAD>{});
      else if constexpr (kAcross && j + AHEAD >= PERIOD)
        ring[j % AHEAD] = read(after, std::integral_constant<int, j + AHEAD - PERIOD>{});
      if constexpr (j >= ALL) return;
      if constexpr (j < bS2) {
        if constexpr (j < NC) s1 = a_mma<T>(r, k[0][j], s1);
        else s1 = stat(r, std::true_type{}, bounded(__uint_as_float(r[0]) * invc), s1);
        if constexpr (j == kLook) look(base + decltype(stage)::value * F::kStage, r);
      } else if constexpr (j < bA) {
        if constexpr (j - bS2 < NC) s2 = a_mma<T>(r, k[1][j - bS2], s2);
        else s2 = stat(r, std::false_type{}, bounded(__uint_as_float(r[1]) * invc), s2);
        if constexpr (j == kLook) look(base + decltype(stage)::value * F::kStage, r);
      } else if constexpr (j < bV) {
        if constexpr (j - bA < 2 * NC) {
          a1 = a_mma<T>(r, v[j - bA], a1);
        } else {
          a2 = stat(r, std::false_type{}, -__uint_as_float(r[3]), a1);
          a1 = stat(r, std::true_type{}, -__uint_as_float(r[2]), a1);
        }
      } else if constexpr (j < bK1) {
        constexpr int u = (j - bV) / (2 * ND), n = (j - bV) % (2 * ND);
        if constexpr (n == 0) op = a_operand<T>(p, u);
        dv[n] = a_mma<T>(op, r, dv[n]);
      } else {
        constexpr int m = j >= bK2, i = j - (m ? bK2 : bK1), u = i / ND, n = i % ND;
        if constexpr (n == 0) op = m ? a_operand<T>(p2, u) : a_operand<T>(p1, u);
        dk[m][n] = a_mma<T>(op, r, dk[m][n]);
      }
      // probabilities of the first map beside the second's scores, of the second
      // beside dA
      spread(std::integral_constant<int, j - bS2 - 1>{}, std::integral_constant<int, nS>{}, first);
      if constexpr (kK) {
        spread(std::integral_constant<int, j - bA - 1>{}, std::integral_constant<int, nA - 1>{}, second);
      } else if constexpr (j == bA - 1) {
        spread(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, first);
        spread(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, second);
      }
      if constexpr (j == bV - 1) {
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = 8 * (i >> 2) + (i & 3);
            const bool on = (row > n0) & (row < rows);
            p1[i] = on ? p1[i] : 0.f;
            p2[i] = on ? p2[i] : 0.f;
            if constexpr (kK) {
              const bool grad = on & (nk > 1) & (row != lone);
              a1[i] = grad ? a1[i] : 0.f;
              a2[i] = grad ? a2[i] : 0.f;
            }
          }
        }
        if constexpr (kV) {
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = p1[i] + p2[i];
        } else {
          spread(std::integral_constant<int, 0>{}, std::integral_constant<int, 1>{}, grads);
        }
      }
      if constexpr (kV && kK) spread(std::integral_constant<int, j - bV>{}, std::integral_constant<int, nV>{}, grads);
      __builtin_amdgcn_sched_barrier(0);
    });
  };

  auto prologue = [&](auto stage) __attribute__((always_inline)) {
    a_for<0, AHEAD>([&](auto jc) __attribute__((always_inline)) { ring[decltype(jc)::value] = read(stage, jc); });
  };
  // read when the head changes and waited for there: a wait where it is used
  // would be one for the loads into LDS too
  auto lambda = [&](int g) __attribute__((always_inline)) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(S.lam[hk * G + g])));
  };
  float lam = begin < end ? lambda(now.g) : 0.f;
  constexpr int NS = F::kStages;
  __syncthreads();  // every wave has left the LDS of the piece before
  if (begin < end) {
    for (int i = 0; i < (kAcross ? 2 * F::kGroup : 1); ++i) issue(base + i * F::kStage);
    a_landed();
    prologue(std::integral_constant<int, 0>{});
  }
  // whole rounds of the stages: tiles past the last add nothing
  for (int i = begin; i < end; i += NS) {
    a_for<0, NS>([&](auto sc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value, U = F::kGroup;
      const int rows = i + s < end ? nq - now.t - 4 * half : 0;
      const bool masked = nk == 1 || (S.causal && now.t + shift < key0 + 32) || i + s >= end || nq - now.t < 32;
      if constexpr (kAcross) {
        tile(sc, lam, now.t, rows, masked, [&]() __attribute__((always_inline)) {
          if constexpr (s % U == U - 1) {
            // the next group is there, and the one before this is free
            asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
            a_for<0, U>([&](auto uc) __attribute__((always_inline)) {
              issue(base + (s + U + 1 + decltype(uc)::value) % NS * F::kStage);
            });
          }
        });
      } else {
        issue(base + (s + 1) % NS * F::kStage);
        tile(sc, lam, now.t, rows, masked, [] {});
        a_landed();
        prologue(std::integral_constant<int, (s + 1) % NS>{});
      }
      const int g = now.g;
      next(now);
      if (now.g != g) lam = lambda(min(now.g, G - 1));
    });
  }
  // no load may still be on its way into LDS when the workgroup ends
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

  // the odd values of dO, for the keys that their rows see
  if (kV && odd) {
    for (int i = begin; i < end; ++i) {
      const int g = i / perHead, t0 = first + 32 * (i % perHead), t1 = t0 + (lane & 31);
      uint32_t bad = 0;
      if (t1 < nq) {
        const lf4 r = L.rec[rec0 + (int64_t)g * S.nq + t1];
        bad = a_bad_row(r.v[0], r.v[1], r.v[2], r.v[3]);
      }
      for (uint32_t rows = (uint32_t)__ballot(bad != 0); rows; rows &= rows - 1) {
        const int t = t0 + __builtin_ctz(rows);
        const char* o = d0 + (t * L.gs[1] + g * L.gs[2]) * E;
#pragma unroll
        for (int n = 0; n < 2 * ND; ++n) {
          const int c = n * 32 + (lane & 31);
          const float x = c < 2 * S.dim ? LType<T>::get(o, c) : 0.f, nan = x - x;  // (0 where x is finite)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int kk = key0 + 8 * (e >> 2) + 4 * half + (e & 3);
            dv[n][e] += !S.causal || kk < t + shift ? nan : 0.f;
          }
        }
      }
    }
  }

  // registers run over keys here: lane l has column l % 32 of every sum
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int kk = key0 + 8 * (r >> 2) + 4 * half + (r & 3);
    if (kk >= nk) continue;
    const int64_t tok = tok0 + kk;
    if (P.slot >= 0) {
      float* o = L.part + (P.slot * kDkvKeys + kk - at) * (4 * DP) + (lane & 31);
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        if constexpr (kK) {
          o[n * 32] = dk[0][n][r];
          o[DP + n * 32] = dk[1][n][r];
        }
        if constexpr (kV) {
          o[2 * DP + n * 32] = dv[n][r];
          o[2 * DP + (ND + n) * 32] = dv[ND + n][r];
        }
      }
      continue;
    }
    char* ok = (char*)L.dk + (batch * L.dks[0] + tok * L.dks[1] + 2 * hk * L.dks[2]) * E;
    char* ov = (char*)L.dv + (batch * L.dvs[0] + tok * L.dvs[1] + hk * L.dvs[2]) * E;
#pragma unroll
    for (int n = 0; n < ND; ++n) {
      const int c = n * 32 + (lane & 31);
      if (kK && c < S.dim) {
        LType<T>::put(ok, c, dk[0][n][r] * L.scale);
        LType<T>::put(ok + L.dks[2] * E, c, dk[1][n][r] * L.scale);
      }
      if constexpr (kV) {
        if (c < 2 * S.dim) LType<T>::put(ov, c, dv[n][r]);
        if (DP + c < 2 * S.dim) LType<T>::put(ov, DP + c, dv[ND + n][r]);
      }
    }
  }
  }
}

template <typename T, int DP, int PART, int... REST> hipError_t run(const AttnGradLaunch& L, hipStream_t st) {
  attn_dkv<T, DP, PART><<<dim3((unsigned)(L.keyRuns.streams ? L.keyRuns.streams : L.s.combos * L.keyRuns.blocks)), 256, 0, st>>>(L);
  const hipError_t e = hipGetLastError();
  if constexpr (sizeof...(REST) > 0) return e != hipSuccess ? e : run<T, DP, REST...>(L, st);
  else return e;
}

}  // namespace

hipError_t launch_attn_dkv(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st) {
  // operands and sums of 32 wide keys are more than a wave's registers: more passes
  if (bf16) return dp == 64 ? run<Bf16, 64, 3>(L, st) : run<Bf16, 128, 1, 2>(L, st);
  return dp == 64 ? run<float, 64, 3>(L, st) : run<float, 128, 1, 2>(L, st);
}

}  // namespace muon
