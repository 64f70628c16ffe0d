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
// No atomics: a workgroup owns its keys.  Where there are few, the row tiles
// are split, and the splits' sums are joined in order.
#include <hip/hip_runtime.h>

#include "attention.hpp"
#include "attn_tile.hpp"

namespace muon {
namespace {

// What a pass makes (PART): bit 0 dV, bit 1 dK_1, bit 2 dK_2.
template <typename T, int DP> struct Dkv {
  static constexpr int kWaves = 4, kThreads = 256, kRows = 32;
  static constexpr int kK = DP * AT<T>::kBytes, kVB = 2 * kK;
  static constexpr int kStage = kRows * (2 * kK + kVB) + (AT<T>::kBytes == 2 ? 2048 : 1024);
};

template <typename T, int DP, int PART>
__global__ __launch_bounds__(256, 1) void attn_dkv(const AttnGradLaunch L) {
  using F = Dkv<T, DP>;
  constexpr bool kV = PART & 1, kK1 = PART & 2, kK2 = PART & 4;  // what is made,
  constexpr bool kS1 = kV || kK1, kS2 = kV || kK2;               // and from which scores
  constexpr int E = AT<T>::kBytes, NC = DP / AT<T>::kStep, ND = DP / 32, SP = AT<T>::kSteps32;
  constexpr int RQ = F::kRows * F::kK, RECS = 2 * RQ + F::kRows * F::kVB;  // bytes of a Q tile; where the records lie
  __shared__ __attribute__((aligned(1024))) char lds[2 * F::kStage];
  const AttnShape& S = L.s;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  int id = blockIdx.x;
  const int combo = id % S.combos;
  id /= S.combos;
  const int split = id % L.splits;
  id /= L.splits;
  int tok0 = 0, nq = (int)S.nq, nk = (int)S.nk, inside = 1, at = 0;
  if (L.keyList.blocks) {
    if (id >= *L.keyList.count) return;
    const AttnBlock B = L.keyList.blocks[id];
    tok0 = B.tok;
    nq = nk = B.n;
    inside = B.nk > 0;
    at = B.at;
  } else {  // the keys that most rows see first
    at = id * kDkvKeys;
  }
  const int batch = combo / S.kv, hk = combo % S.kv, G = S.group;
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
    if constexpr (PART & 6) {
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) {
        v[c] = lu32x4{0, 0, 0, 0};
        if (valid && (2 * c + half) * 16 < 2 * S.dim * E) v[c] = *(const lu32x4*)(o + (2 * c + half) * 16);
      }
    }
  }

  // row tiles: tokens from the first that sees a key of the workgroup
  const int first = S.causal ? max(at - shift + 1, 0) & ~31 : 0;
  const int perHead = inside && nq > first ? (nq - first + 31) / 32 : 0;
  const int tiles = perHead * G;
  const int share = (tiles + L.splits - 1) / L.splits;
  const int begin = min(split * share, tiles), end = min(begin + share, tiles);

  TileLoader<F::kK, F::kRows, F::kWaves> ldq;
  TileLoader<F::kVB, F::kRows, F::kWaves> ldd;
  ldq.init(lane, wave, S.qs[1] * E, S.dim * E);
  ldd.init(lane, wave, L.gs[1] * E, 2 * S.dim * E);
  const char* q0 = (const char*)S.q + (batch * S.qs[0] + tok0 * S.qs[1] + 2 * hk * G * S.qs[2]) * E;
  const char* d0 = (const char*)L.dout + (batch * L.gs[0] + tok0 * L.gs[1] + hk * G * L.gs[2]) * E;
  const int64_t rec0 = ((int64_t)batch * L.heads + hk * G) * S.nq + tok0;
  const uint32_t base = a_lds(lds);
  // tile i: head i / perHead, tokens from first + 32·(i % perHead)
  auto issue = [&](int g, int t, uint32_t buf) __attribute__((always_inline)) {
    const char* q = q0 + (t * S.qs[1] + 2 * g * S.qs[2]) * E;
    ldq.issue(q, nq - t, buf);
    ldq.issue(q + S.qs[2] * E, nq - t, buf + RQ);
    ldd.issue(d0 + (t * L.gs[1] + g * L.gs[2]) * E, nq - t, buf + 2 * RQ);
    // the records: bf16 recL by wave 0, recD by wave 1; fp32 rec
    const int64_t r = rec0 + g * S.nq + t;
    if (wave < 2) {
      const int i = lane & 31;
      if constexpr (E == 2) {
        // lanes past 31 deliver zeros behind the 32 records
        if (wave == 0 || (PART & 6))
          f_dma16(__builtin_amdgcn_readfirstlane(buf + RECS + wave * 1024), lane < 32 && i < nq - t ? (uint32_t)i * 16 : kFfnNowhere,
                  f_buffer((uint64_t)((wave == 0 ? L.recL : L.recD) + r)));
      } else if (wave == 0) {
        f_dma16(__builtin_amdgcn_readfirstlane(buf + RECS), lane < 32 && i < nq - t ? (uint32_t)i * 16 : kFfnNowhere,
                f_buffer((uint64_t)(L.rec + r)));
      }
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

  auto step = [&](uint32_t buf, float lam, int t, bool masked) __attribute__((always_inline)) {
    const uint32_t rec = buf + RECS + (lane & 31) * 16;
    af32x16 s1{}, s2{}, a1{}, a2{};
    const lu32x4 r = *(a_lds_u4)(uintptr_t)rec;
    [[maybe_unused]] const float u = half ? 0.f : 1.f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if constexpr (kS1) s1 = a_mma<T>(rq.get(buf, c), k[0][c], s1);
      if constexpr (kS2) s2 = a_mma<T>(rq.get(buf + RQ, c), k[1][c], s2);
    }
    // the statistics' steps come last: added first, each later sum would be
    // rounded at their size
    if constexpr (E == 2) {
      if constexpr (kS1) s1 = a_mma<T>(r, one0, s1);
      if constexpr (kS2) s2 = a_mma<T>(r, one3, s2);
    } else {
      if constexpr (kS1)
        s1 = __builtin_amdgcn_mfma_f32_32x32x2f32(fmaxf(__uint_as_float(r[0]) * invc, -1e30f), u, s1, 0, 0, 0);
      if constexpr (kS2)
        s2 = __builtin_amdgcn_mfma_f32_32x32x2f32(fmaxf(__uint_as_float(r[1]) * invc, -1e30f), u, s2, 0, 0, 0);
    }
    if constexpr (PART & 6) {  // a1 becomes dA − δ_1, a2 dA − δ_2
#pragma unroll
      for (int c = 0; c < 2 * NC; ++c) a1 = a_mma<T>(rd.get(buf + 2 * RQ, c), v[c], a1);
      if constexpr (E == 2) {
        const lu32x4 d = *(a_lds_u4)(uintptr_t)(rec + 1024);
        if constexpr (kK2) a2 = a_mma<T>(d, one3, a1);
        if constexpr (kK1) a1 = a_mma<T>(d, one0, a1);
      } else {
        if constexpr (kK2) a2 = __builtin_amdgcn_mfma_f32_32x32x2f32(-__uint_as_float(r[3]), u, a1, 0, 0, 0);
        if constexpr (kK1) a1 = __builtin_amdgcn_mfma_f32_32x32x2f32(-__uint_as_float(r[2]), u, a1, 0, 0, 0);
      }
    }
    // row t + i sees this lane's key if key < t + i + shift; of a row that sees
    // one key alone P = 1 whatever the scores, and dS = 0
    if (masked) {
      const int n = S.causal ? key - shift - t - 4 * half : -1;
      const int lone = (S.causal ? 1 - shift - t : -1) - 4 * half;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool on = 8 * (i >> 2) + (i & 3) > n;
        const bool grad = on && nk > 1 && 8 * (i >> 2) + (i & 3) != lone;
        if constexpr (kS1) s1[i] = on ? s1[i] : kNegInf;
        if constexpr (kS2) s2[i] = on ? s2[i] : kNegInf;
        if constexpr (kK1) a1[i] = grad ? a1[i] : 0.f;
        if constexpr (kK2) a2[i] = grad ? a2[i] : 0.f;
      }
    }
    float p1[16], p2[16], p[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if constexpr (kS1) p1[i] = a_exp2(s1[i] * S.c);
      if constexpr (kS2) p2[i] = -lam * a_exp2(s2[i] * S.c);
      if constexpr (kV) p[i] = p1[i] + p2[i];
      if constexpr (kK1) p1[i] *= a1[i];
      if constexpr (kK2) p2[i] *= a2[i];
    }
#pragma unroll
    for (int u = 0; u < SP; ++u) {
      if constexpr (kV) {
        const lu32x4 a = a_operand<T>(p, u);
#pragma unroll
        for (int n = 0; n < 2 * ND; ++n)
          dv[n] = a_mma<T>(a, cd.get(buf + 2 * RQ + u * AT<T>::kStep * F::kVB, n), dv[n]);
      }
      if constexpr (kK1) {
        const lu32x4 a = a_operand<T>(p1, u);
#pragma unroll
        for (int n = 0; n < ND; ++n) dk[0][n] = a_mma<T>(a, cq.get(buf + u * AT<T>::kStep * F::kK, n), dk[0][n]);
      }
      if constexpr (kK2) {
        const lu32x4 a = a_operand<T>(p2, u);
#pragma unroll
        for (int n = 0; n < ND; ++n) dk[1][n] = a_mma<T>(a, cq.get(buf + RQ + u * AT<T>::kStep * F::kK, n), dk[1][n]);
      }
    }
  };

  uint32_t buf = base;
  int g = perHead ? begin / perHead : 0, i = begin - g * perHead;
  if (begin < end) issue(g, first + 32 * i, base);
  for (int tile = begin; tile < end; ++tile) {
    a_landed();
    const uint32_t other = 2 * base + F::kStage - buf;
    const int t = first + 32 * i;
    const float lam = S.lam[hk * G + g];
    if (++i == perHead) {
      i = 0;
      ++g;
    }
    if (tile + 1 < end) issue(g, first + 32 * i, other);
    // no row of the tile sees a key of this wave: nothing to add
    if (!S.causal || t + 31 + shift > key0) step(buf, lam, t, nk == 1 || (S.causal && t + shift < key0 + 32));
    buf = other;
  }

  // registers run over keys here: lane l has column l % 32 of every sum
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int kk = key0 + 8 * (r >> 2) + 4 * half + (r & 3);
    if (kk >= nk) continue;
    const int64_t tok = tok0 + kk;
    if (L.splits > 1) {
      float* o = L.part + (((int64_t)split * S.combos + combo) * S.nk + tok) * (4 * DP) + (lane & 31);
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        if constexpr (kK1) o[n * 32] = dk[0][n][r];
        if constexpr (kK2) o[DP + n * 32] = dk[1][n][r];
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
      if (c < S.dim) {
        if constexpr (kK1) LType<T>::put(ok, c, dk[0][n][r] * L.scale);
        if constexpr (kK2) LType<T>::put(ok + L.dks[2] * E, c, dk[1][n][r] * L.scale);
      }
      if constexpr (kV) {
        if (c < 2 * S.dim) LType<T>::put(ov, c, dv[n][r]);
        if (DP + c < 2 * S.dim) LType<T>::put(ov, DP + c, dv[ND + n][r]);
      }
    }
  }
}

// The splits' sums added in order: a workgroup per key of a combo, four
// columns a thread.
template <typename T, int DP> __global__ __launch_bounds__(DP) void attn_dkv_join(const AttnGradLaunch L) {
  constexpr int E = AT<T>::kBytes;
  const AttnShape& S = L.s;
  const int64_t combo = blockIdx.x / S.nk, key = blockIdx.x - combo * S.nk;
  const int c0 = threadIdx.x * 4;
  const int64_t all = S.combos * S.nk * (4 * DP);
  const float* p = L.part + (combo * S.nk + key) * (4 * DP) + c0;
  lf32x4 s = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < L.splits; ++i) s += *(const lf32x4*)(p + i * all);
  const int64_t batch = combo / S.kv, hk = combo % S.kv;
  if (c0 < 2 * DP) {
    const int m = c0 >= DP, c = c0 - m * DP;
    char* o = (char*)L.dk + (batch * L.dks[0] + key * L.dks[1] + (2 * hk + m) * L.dks[2]) * E;
    for (int i = 0; i < 4; ++i)
      if (c + i < S.dim) LType<T>::put(o, c + i, s[i] * L.scale);
  } else {
    const int c = c0 - 2 * DP;
    char* o = (char*)L.dv + (batch * L.dvs[0] + key * L.dvs[1] + hk * L.dvs[2]) * E;
    for (int i = 0; i < 4; ++i)
      if (c + i < 2 * S.dim) LType<T>::put(o, c + i, s[i]);
  }
}

template <typename T, int DP, int PART, int... REST> hipError_t run(const AttnGradLaunch& L, hipStream_t st) {
  attn_dkv<T, DP, PART><<<dim3((unsigned)(L.s.combos * L.keyBlocks * L.splits)), 256, 0, st>>>(L);
  const hipError_t e = hipGetLastError();
  if constexpr (sizeof...(REST) > 0) return e != hipSuccess ? e : run<T, DP, REST...>(L, st);
  else return e;
}
template <typename T, int DP> hipError_t join(const AttnGradLaunch& L, hipStream_t st) {
  attn_dkv_join<T, DP><<<dim3((unsigned)(L.s.combos * L.s.nk)), DP, 0, st>>>(L);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_dkv(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st) {
  // operands and sums of 32 wide keys are more than a wave's registers: more passes
  if (bf16) return dp == 64 ? run<Bf16, 64, 7>(L, st) : run<Bf16, 128, 1, 6>(L, st);
  return dp == 64 ? run<float, 64, 7>(L, st) : run<float, 128, 1, 2, 4>(L, st);
}
hipError_t launch_attn_dkv_join(bool bf16, int dp, const AttnGradLaunch& L, hipStream_t st) {
  if (bf16) return dp == 64 ? join<Bf16, 64>(L, st) : join<Bf16, 128>(L, st);
  return dp == 64 ? join<float, 64>(L, st) : join<float, 128>(L, st);
}

}  // namespace muon
