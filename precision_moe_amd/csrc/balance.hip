// Training side of the router front: expert counts, the balance loss and the
// z-loss of each sequence, and the gradient of the logits.
//
// Notation: l the FP32 logits of a token, m = max_e l_e, lse = m + log sum_e
// exp(l_e - m), p_e = exp(l_e - lse). A token is active when one of its ids is
// in [0, E) and one of its logits is not -inf; other tokens (the padding of a
// batch) count nowhere and get a zero gradient. For sequence s, n_s is its
// number of active tokens, c_se its routes to expert e, f_se = c_se / (n_s K)
// and P_se = sum_t p_te:
//   balance_s = E sum_e f_se P_se / n_s,     z_s = sum_t lse_t^2 / n_s,
// both 0 when n_s = 0. f is a count and has no gradient, so
//   d balance_s / d l_te = (E / n_s) p_te (f_se - sum_e' f_se' p_te')
//   d z_s / d l_te       = (2 / n_s) lse_t p_te,
// and with d w_j the gradient of the top-k weight w_j = p_{id_j}
//   d l_e += p_e (sum_{j: id_j = e} d w_j - sum_j d w_j p_{id_j}),
// or, for the renormalized weights q_j = p_{id_j} / sum_k p_{id_k},
//   d l_{id_j} += q_j (d w_j - sum_k d w_k q_k).
//
// L = 16 lanes hold one token up to E = 128 and L = 64 above: lane i the logits of
// experts i, i + L, ..., or, where E fills them exactly, 4 i .. 4 i + 3, 4 L further,
// ... (16 bytes a load). With 16 a wavefront works on four tokens, and what is done
// once for a token costs a quarter of an instruction: the gradient of T = 65521
// tokens, E = 64, takes 14.7 us a call (64 lanes: 19.8). With many experts the
// registers of 16 lanes would leave too few wavefronts: T = 8192, E = 1024, 39 us
// against 18.8.
// The sums over tokens are taken in a fixed order without atomics on floats,
// so results do not vary between runs.
#include <algorithm>

#include "device.h"
#include "kernels.h"

namespace pmoe {

typedef float floatx4_t __attribute__((ext_vector_type(4)));
constexpr float kNegInf = -__builtin_inff();

// Moves between lanes without LDS traffic (data-parallel primitives): rotations within
// rows of 16 lanes, and, for sums over the wave, the last lanes of rows into the rows above.
template <int kCtrl, int kRows>
__device__ __forceinline__ float lane_move(float old, float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(old), __float_as_uint(v), kCtrl, kRows, 0xf, false));
}
template <int kBy>
__device__ __forceinline__ float turn16(float v) {
  return __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(v), 0x120 + kBy, 0xf, 0xf, true));
}
// Sum and maximum over 16 lanes, in all of them (the partial sums are the same in the lanes
// that hold them, since an addition does not depend on its operands' order).
__device__ __forceinline__ float sum16(float v) {
  v += turn16<8>(v);
  v += turn16<4>(v);
  v += turn16<2>(v);
  return v + turn16<1>(v);
}
__device__ __forceinline__ float max16(float v) {
  v = __builtin_fmaxf(v, turn16<8>(v));
  v = __builtin_fmaxf(v, turn16<4>(v));
  v = __builtin_fmaxf(v, turn16<2>(v));
  return __builtin_fmaxf(v, turn16<1>(v));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum_f(float v) {
  v = sum16(v);
  v += lane_move<0x142, 0xa>(0.0f, v);
  v += lane_move<0x143, 0xc>(0.0f, v);
  return last_lane(v);
}
__device__ __forceinline__ float wave_max_f(float v) {
  v = max16(v);
  v = __builtin_fmaxf(v, lane_move<0x142, 0xa>(v, v));
  v = __builtin_fmaxf(v, lane_move<0x143, 0xc>(v, v));
  return last_lane(v);
}
// Over the L lanes of a token, in all of them.
template <int L>
__device__ __forceinline__ float token_sum(float v) {
  return L == 16 ? sum16(v) : wave_sum_f(v);
}
template <int L>
__device__ __forceinline__ float token_max(float v) {
  return L == 16 ? max16(v) : wave_max_f(v);
}
template <int L>
__device__ __forceinline__ uint64_t token_ballot(bool on, int group) {
  return L == 16 ? (__ballot(on) >> (16 * group)) & 0xFFFFull : __ballot(on);
}

// exp(x) for x <= 0 as 2^(x log2 e): the product is carried with its rounding
// error, which scales the hardware's 2^t. Below -200 (and at -inf) the result
// is 0; NaN stays NaN.
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -200.0f ? -200.0f : x;
  constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float t = x * kLog2e;
  const float e = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -t));
  const float r = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(r, e * kLn2, r);
}

// 1 / x to about half a step: one Newton step on the hardware's reciprocal.
__device__ __forceinline__ float recip(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  return __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
}

__device__ __forceinline__ int expert_id(const void* ids, int ids64, long i, int E) {
  const long long id = ids64 ? static_cast<const long long*>(ids)[i] : static_cast<const int*>(ids)[i];
  return id >= 0 && id < E ? (int)id : -1;
}

// The sequence of token t (the same in L lanes): the last s with offsets[s] <= t, -1 before
// the first and S behind the last. Every round the L lanes probe L places of the range.
template <int L>
__device__ __forceinline__ int sequence_of(const int* offsets, int S, int t, int group, int i) {
  if (offsets == nullptr) return 0;
  int lo = 0, n = S + 1;  // offsets[0 .. lo) <= t, offsets[lo + n ..) > t
  while (n > 0) {
    const int step = (n + L - 1) / L;
    const int at = i * step;
    const int passed = __popcll(token_ballot<L>(at < n && offsets[lo + min(at, n - 1)] <= t, group));
    if (passed == 0) return lo - 1;
    const int base = (passed - 1) * step;  // this place is <= t, the next probe is not
    const int next = min(passed * step, n);
    lo += base + 1;
    n = next - base - 1;
  }
  return lo - 1;
}

// The expert of a lane's c-th logit. kFull: E is L NPL, and rows are aligned to 16 bytes.
template <int L, bool kFull>
__device__ __forceinline__ int expert_of(int i, int c) {
  return kFull ? 4 * L * (c >> 2) + 4 * i + (c & 3) : i + L * c;
}

// What L lanes read of a token: its logits, and in lane j the ids of the slots j and j + L.
// `first` is a token that is the same in all lanes, `by` the lane's distance to it.
template <int L, int NPL, bool kFull>
struct Token {
  static constexpr int kSlots = 32 / L > 0 ? 32 / L : 1;  // K <= 32
  float v[NPL];
  int id[kSlots];
  __device__ __forceinline__ void load(const float* logits, const void* ids, int ids64, long first, int by, int E,
                                       int K, int i) {
    const float* rows = logits + first * E;
    const uint32_t at = (uint32_t)by * E;
    if constexpr (kFull) {
#pragma unroll
      for (int c = 0; c < NPL; c += 4) {
        const floatx4_t u = *reinterpret_cast<const floatx4_t*>(rows + (at + expert_of<L, kFull>(i, c)));
        v[c] = u[0], v[c + 1] = u[1], v[c + 2] = u[2], v[c + 3] = u[3];
      }
    } else {
#pragma unroll
      for (int c = 0; c < NPL; ++c) v[c] = i + L * c < E ? rows[at + i + L * c] : kNegInf;
    }
#pragma unroll
    for (int y = 0; y < kSlots; ++y) {
      const int j = i + L * y;
      id[y] = j < K ? expert_id(ids, ids64, (first + by) * K + j, E) : -1;
    }
  }
  __device__ __forceinline__ bool any_id(int group) const {
    bool on = false;
#pragma unroll
    for (int y = 0; y < kSlots; ++y) on |= id[y] >= 0;
    return token_ballot<L>(on, group) != 0;
  }
};

// The softmax of a token.
template <int NPL>
struct Row {
  float ex[NPL];  // exp(l - m); 0 behind E
  float m, sum, inv;
  bool active;
  __device__ __forceinline__ float lse() const { return m + logf(sum); }
};

template <int L, int NPL>
__device__ __forceinline__ Row<NPL> softmax_row(const float (&v)[NPL], bool any_id, int group) {
  Row<NPL> r;
  float m = v[0];
#pragma unroll
  for (int c = 1; c < NPL; ++c) m = __builtin_fmaxf(m, v[c]);
  r.m = token_max<L>(m);
  r.active = any_id && r.m > kNegInf;
  if (__ballot(any_id && !r.active)) {  // rare: all -inf, or NaN among them, which has to come out as NaN
    bool nan = false;
#pragma unroll
    for (int c = 0; c < NPL; ++c) nan |= v[c] != v[c];
    r.active = any_id && (r.m > kNegInf || token_ballot<L>(nan, group) != 0);
  }
  if (!r.active) r.m = 0.0f;
  float part = 0.0f;
#pragma unroll
  for (int c = 0; c < NPL; ++c) {
    r.ex[c] = exp_neg(v[c] - r.m);
    part += r.ex[c];
  }
  r.sum = token_sum<L>(part);
  r.inv = recip(r.sum);
  if (__ballot(!r.active)) {  // whatever stands in a padding token stays out of every sum
#pragma unroll
    for (int c = 0; c < NPL; ++c) r.ex[c] = r.active ? r.ex[c] : 0.0f;
    r.inv = r.active ? r.inv : 0.0f;
  }
  return r;
}

// ---------------------------------------------------------------- forward
// A slot holds the sums of some tokens of one sequence: probability sums [E4],
// route counts [E4], the sum of lse^2 and the number of active tokens (E4: E
// rounded up to 4, so that slots are read 16 bytes at a time).
__host__ __device__ inline int balance_e4(int E) { return (E + 3) & ~3; }
__host__ __device__ inline long balance_slot_words(int E) { return 2L * balance_e4(E) + 4; }

// The losses of a sequence from its sums in LDS; all threads of the workgroup.
__device__ __forceinline__ void write_sequence(const BalanceParams& p, int s, const float* prob,
                                               const int* count, float zsum, int n, float* wave_part) {
  const int tid = threadIdx.x, lane = tid & 63;
  float term = 0.0f;
  for (int e = tid; e < p.E; e += blockDim.x) {
    p.counts[(long)s * p.E + e] = count[e];
    p.prob[(long)s * p.E + e] = prob[e];
    term += (float)count[e] * prob[e];
  }
  term = wave_sum_f(term);
  if (lane == 0) wave_part[tid >> 6] = term;
  __syncthreads();
  if (tid == 0) {
    float sum = 0.0f;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) sum += wave_part[w];
    const float d = (float)max(n, 1);
    p.tokens[s] = n;
    p.balance[s] = (float)p.E / (float)p.K * (sum / d) / d;
    p.z[s] = zsum / d;
  }
}

// Workgroup c (8 waves, 8 or 32 tokens at a time) takes the tokens [c * rows,
// (c + 1) * rows) and writes, for every sequence s that has tokens there, the
// slot c + s. Along the tokens either c or s grows from one (c, s) to the
// next, so the slot numbers differ; there are chunks + S of them at most. With
// kDirect there is one workgroup and one sequence, and it writes the results.
// Bound by latency more than by bytes: T = 32749, E = 96, K = 6, S = 61 reads 13.4 MB in 21 us a
// call, most of it the two launches; T = 65536, E = 256, S = 200 reads 69 MB in 26.
constexpr int kRowWaves = 8;
template <int L, int NPL, bool kFull, bool kDirect>
__global__ __launch_bounds__(64 * kRowWaves) void balance_rows_kernel(BalanceParams p, int rows) {
  constexpr int kThreads = 64 * kRowWaves, G = 64 / L;  // G tokens to a wave
  __shared__ float prob[kRowWaves][L * NPL];
  __shared__ int count[L * NPL];
  __shared__ float zsum[16];  // also write_sequence's
  __shared__ int nact[kRowWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = lane / L, i = lane % L;
  const int T = p.T, E = p.E, K = p.K;
  const int* offsets = p.offsets;
  const int begin = blockIdx.x * rows, end = min(T, begin + rows);
  int t0 = begin;
  if (kDirect && offsets) t0 = min(max(offsets[0], 0), end);
  while (kDirect || t0 < end) {  // uniform: every lane sees the same offsets
    int s = 0, t1 = end;
    if (kDirect) {
      if (offsets) t1 = min(max(offsets[1], t0), end);
    } else {
      s = sequence_of<L>(offsets, p.S, t0, group, i);
      if (s >= p.S) break;
      if (s < 0) {
        t0 = min(end, max(offsets[0], t0 + 1));
        continue;
      }
      if (offsets) t1 = min(end, max(offsets[s + 1], t0 + 1));
    }
    for (int e = threadIdx.x; e < L * NPL; e += kThreads) count[e] = 0;
    __syncthreads();
    float sum[NPL];
#pragma unroll
    for (int c = 0; c < NPL; ++c) sum[c] = 0.0f;
    float z = 0.0f;
    int n = 0;
    for (int t = t0 + G * wave; t < t1; t += G * kRowWaves) {
      const bool on = t + group < t1;
      Token<L, NPL, kFull> now;
      now.load(p.logits, p.ids, p.ids64, t, on ? group : 0, E, K, i);
      const Row<NPL> r = softmax_row<L, NPL>(now.v, now.any_id(group) && on, group);
      if (r.active) {
#pragma unroll
        for (int y = 0; y < now.kSlots; ++y)
          if (now.id[y] >= 0) atomicAdd(&count[now.id[y]], 1);
        const float lse = r.lse();
        n += 1;
        z += lse * lse;
      }
#pragma unroll
      for (int c = 0; c < NPL; ++c) sum[c] = __builtin_fmaf(r.ex[c], r.inv, sum[c]);
    }
    // the tokens of a wave, then the waves in order
    const auto over_tokens = [](auto v) {
#pragma unroll
      for (int d = L; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
      return v;
    };
#pragma unroll
    for (int c = 0; c < NPL; ++c) {
      const float v = over_tokens(sum[c]);
      if (group == 0) prob[wave][expert_of<L, kFull>(i, c)] = v;
    }
    z = over_tokens(z);
    n = over_tokens(n);
    if (lane == 0) {
      zsum[wave] = z;
      nact[wave] = n;
    }
    __syncthreads();
    const int used = min(kRowWaves, (t1 - t0 + G - 1) / G);  // waves that had a token
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float q = prob[0][e];
      for (int w = 1; w < used; ++w) q += prob[w][e];
      prob[0][e] = q;
    }
    float zs = 0.0f;
    int ns = 0;
    for (int w = 0; w < kRowWaves; ++w) {
      zs += zsum[w];
      ns += nact[w];
    }
    __syncthreads();
    if (kDirect) {
      write_sequence(p, 0, prob[0], count, zs, ns, zsum);
      return;
    }
    const int E4 = balance_e4(E);
    float* slot = static_cast<float*>(p.ws) + (blockIdx.x + s) * balance_slot_words(E);
    for (int e = threadIdx.x; e < E; e += kThreads) {
      slot[e] = prob[0][e];
      reinterpret_cast<int*>(slot)[E4 + e] = count[e];
    }
    if (threadIdx.x == 0) {
      slot[2 * E4] = zs;
      reinterpret_cast<int*>(slot)[2 * E4 + 1] = ns;
    }
    __syncthreads();
    t0 = t1;
  }
}

// One workgroup per sequence adds its slots: quad q of four columns (of the
// probability sums, behind them of the counts) in blockDim / quads groups of
// threads, group g every groups-th slot; then the groups in order.
__global__ __launch_bounds__(1024) void balance_sum_kernel(BalanceParams p, int rows, int quads) {
  __shared__ uint4 part[1024];
  __shared__ __align__(16) float prob[kMaxExperts];
  __shared__ __align__(16) int count[kMaxExperts];
  __shared__ float zsh[16];
  __shared__ int nsh[16];
  static_assert(__alignof__(part) % 16 == 0 && __alignof__(prob) % 16 == 0 && __alignof__(count) % 16 == 0,
                "written 16 bytes at a time");
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E4 = balance_e4(p.E);
  const int a = p.offsets ? min(max(p.offsets[s], 0), p.T) : 0;
  const int b = p.offsets ? min(max(p.offsets[s + 1], 0), p.T) : p.T;
  const int c0 = a / rows, c1 = a < b ? (b - 1) / rows + 1 : c0;
  const long words = balance_slot_words(p.E);
  const float* slots = static_cast<const float*>(p.ws) + s * words;
  float zs = 0.0f;
  int ns = 0;
  for (int c = c0 + tid; c < c1; c += blockDim.x) {
    const float* slot = slots + c * words;
    zs += slot[2 * E4];
    ns += reinterpret_cast<const int*>(slot)[2 * E4 + 1];
  }
  zs = wave_sum_f(zs);
  ns = wave_sum(ns);
  if (lane == 0) {
    zsh[wave] = zs;
    nsh[wave] = ns;
  }
  const int groups = blockDim.x / quads, grp = tid / quads, q = tid % quads;
  const bool is_prob = q < E4 / 4, is_count = !is_prob && q < E4 / 2;
  floatx4_t ps = {0.0f, 0.0f, 0.0f, 0.0f};
  int4 cs = make_int4(0, 0, 0, 0);
  if (is_prob) {
#pragma unroll 4
    for (int c = c0 + grp; c < c1; c += groups) ps += *reinterpret_cast<const floatx4_t*>(slots + c * words + 4 * q);
    part[tid] = __builtin_bit_cast(uint4, ps);
  } else if (is_count) {
#pragma unroll 4
    for (int c = c0 + grp; c < c1; c += groups) {
      const int4 u = *reinterpret_cast<const int4*>(slots + c * words + 4 * q);
      cs.x += u.x, cs.y += u.y, cs.z += u.z, cs.w += u.w;
    }
    part[tid] = __builtin_bit_cast(uint4, cs);
  }
  __syncthreads();
  if (grp == 0 && is_prob) {
    for (int g = 1; g < groups; ++g) ps += __builtin_bit_cast(floatx4_t, part[g * quads + q]);
    *reinterpret_cast<floatx4_t*>(prob + 4 * q) = ps;
  } else if (grp == 0 && is_count) {
    for (int g = 1; g < groups; ++g) {
      const int4 u = __builtin_bit_cast(int4, part[g * quads + q]);
      cs.x += u.x, cs.y += u.y, cs.z += u.z, cs.w += u.w;
    }
    *reinterpret_cast<int4*>(count + 4 * q - E4) = cs;
  }
  zs = 0.0f;
  ns = 0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) {
    zs += zsh[w];
    ns += nsh[w];
  }
  __syncthreads();
  write_sequence(p, s, prob, count, zs, ns, zsh);
}

// Up to this many tokens of one sequence go through one workgroup, in one launch: 16 times as
// many as it works on at a time. T = 512, E = 64 takes 16.2 us a call so and 18.3 in two launches,
// T = 256, E = 256 21.7 and 18.3.
static int direct_tokens(int E) { return E <= 128 ? 512 : 128; }

// Tokens of one workgroup: the square root of a sequence's mean length, so that the tokens of a
// workgroup and the slots of a sequence grow alike; with short sequences more, up to what the
// workgroup's waves take at a time, as long as that stays within half the mean length (T = 65536,
// E = 64, S = 2000: 41.9 us a call, without 65; with all of the mean length T = 4096, S = 200
// takes 22.1 instead of 18.9, for then most workgroups walk through two sequences).
constexpr int kMostGroups = 1 << 22;  // a launch has less than 2^32 threads
int balance_rows(int T, int E, int S) {
  const int wide = kRowWaves * (E <= 128 ? 4 : 1);
  int rows = 4;
  while ((long)rows * rows * S < T || (rows < wide && 2l * rows * S < T) || T / rows >= kMostGroups) rows *= 2;
  return rows;
}

size_t balance_ws_bytes(int T, int E, int S) {
  const int rows = balance_rows(T, E, S);
  return ((size_t)(T + rows - 1) / rows + S) * balance_slot_words(E) * 4;
}

#define PMOE_BY_LOGITS2(E, l, npl, call)    \
  do {                                      \
    constexpr int L = l, NPL = npl;         \
    if ((E) == L * NPL && aligned) {        \
      constexpr bool kFull = true;          \
      call;                                 \
    } else {                                \
      constexpr bool kFull = false;         \
      call;                                 \
    }                                       \
  } while (0)
#define PMOE_BY_LOGITS(E, call)             \
  do {                                      \
    if ((E) <= 64)                          \
      PMOE_BY_LOGITS2(E, 16, 4, call);      \
    else if ((E) <= 128)                    \
      PMOE_BY_LOGITS2(E, 16, 8, call);      \
    else if ((E) <= 256)                    \
      PMOE_BY_LOGITS2(E, 64, 4, call);      \
    else if ((E) <= 512)                    \
      PMOE_BY_LOGITS2(E, 64, 8, call);      \
    else                                    \
      PMOE_BY_LOGITS2(E, 64, 16, call);     \
  } while (0)

static bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

hipError_t launch_router_balance(const BalanceParams& p, hipStream_t s) {
  const bool aligned = aligned16(p.logits);
  if (p.S == 1 && p.T <= direct_tokens(p.E)) {
    PMOE_BY_LOGITS(p.E, (balance_rows_kernel<L, NPL, kFull, true><<<1, 64 * kRowWaves, 0, s>>>(p, p.T)));
    return hipGetLastError();
  }
  const int rows = balance_rows(p.T, p.E, p.S);
  if (p.T > 0) {
    const int chunks = (p.T + rows - 1) / rows;
    PMOE_BY_LOGITS(p.E, (balance_rows_kernel<L, NPL, kFull, false><<<chunks, 64 * kRowWaves, 0, s>>>(p, rows)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // With more sequences than CUs, small workgroups: T = 65536, E = 64, S = 2000 took 65 us a call
  // so and 75 with 1024 threads, with S = 200, E = 256 25.9 with 1024 and 27.3 with 256.
  int quads = 16;
  while (quads < balance_e4(p.E) / 2) quads *= 2;
  const int threads = p.S <= 256 ? 1024 : (quads < 256 ? 256 : quads);
  balance_sum_kernel<<<p.S, threads, 0, s>>>(p, rows, quads);
  return hipGetLastError();
}

// ---------------------------------------------------------------- backward
// A wave takes `rows` tokens for each of its G = 64 / L groups of lanes, G at a time, and the
// groups keep the expert shares f of their sequence in registers while it stays the same. The
// next token is asked for before one is worked on, but Token::load checks the range of its ids, which
// waits for them and for the logits asked for before: only other waves' work hides that time.
// With u_e = d_balance E / n_s f_se and a_j what the slots add at their experts,
//   d l_e = p_e (u_e - mean + 2 d_z / n_s lse) + sum_{j: id_j = e} a_j,
//   mean = sum_e u_e p_e + sum_j d w_j p_{id_j},  a_j = p_{id_j} d w_j,
// or for renormalized weights mean = sum_e u_e p_e, a_j = q_j (d w_j - sum_k d w_k q_k).
// The slots' logits are read once more, by the lanes of the slots; the a_j reach the lanes of
// their experts through a row of LDS that is zero between tokens.
// The logits are read once and the gradient written once, which bounds it for long batches:
// T = 65521, E = 256, K = 8 takes 37 us a call, 138 MB at 3.7 TB/s (a large copy: 5.1). Two
// tokens asked for ahead, or eight rows to a wave, took 42, with the same wait in them.
template <int L, int NPL, bool kFull>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradParams p, int rows) {
  constexpr int G = 64 / L, kSlots = Token<L, NPL, kFull>::kSlots;
  __shared__ float add_sh[4 * G][L * NPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = lane / L, i = lane % L;
  const int E = p.E, K = p.K;
  const long first = (long)(blockIdx.x * 4 + wave) * G * rows;  // the wave's tokens
  const int n = (int)max(0l, min((long)G * rows, p.T - first));
  float* add = add_sh[wave * G + group];  // these L lanes' alone: a wave's LDS operations stay in order
#pragma unroll
  for (int c = 0; c < NPL; ++c) add[i + L * c] = 0.0f;
  float share[NPL];  // d_balance E / n_s f_se
  float cz = 0.0f;   // 2 d_z / n_s
#pragma unroll
  for (int c = 0; c < NPL; ++c) share[c] = 0.0f;
  const bool losses = p.tokens != nullptr;
  long seq_end = 0;  // the sequence in `share` holds the tokens up to here
  Token<L, NPL, kFull> next;
  // lanes without a token look at group 0's
  if (n > 0) next.load(p.logits, p.ids, p.ids64, first, group < n ? group : 0, E, K, i);
  for (int y = 0; y < n; y += G) {
    const bool on = y + group < n;
    const int by = on ? y + group : y;
    const long t = first + by;
    const Token<L, NPL, kFull> now = next;
    if (y + G < n) next.load(p.logits, p.ids, p.ids64, first, y + G + group < n ? y + G + group : y + G, E, K, i);
    float dw[kSlots] = {}, slot[kSlots] = {};  // of the lane's slots: gradient, logit
    if (p.d_topk_w) {
#pragma unroll
      for (int h = 0; h < kSlots; ++h)
        if (now.id[h] >= 0) {
          dw[h] = p.d_topk_w[t * K + i + L * h];
          slot[h] = p.logits[t * E + now.id[h]];
        }
    }
    if (losses && on && t >= seq_end) {
      const int s = sequence_of<L>(p.offsets, p.S, (int)t, group, i);
      const bool in = s >= 0 && s < p.S;  // else the losses do not see the token
      seq_end = p.offsets ? (in ? max((long)p.offsets[s + 1], t + 1) : t + 1) : p.T;
      const float n_s = in ? (float)max(p.tokens[s], 1) : 1.0f;
      cz = in && p.d_z ? 2.0f * p.d_z[s] / n_s : 0.0f;
      const float cb = in && p.d_balance ? p.d_balance[s] * ((float)E / (n_s * n_s * (float)K)) : 0.0f;
#pragma unroll
      for (int c = 0; c < NPL; ++c) {
        const int e = expert_of<L, kFull>(i, c);
        share[c] = in && p.d_balance && (kFull || e < E) ? cb * (float)p.counts[(long)s * E + e] : 0.0f;
      }
    }
    const Row<NPL> r = softmax_row<L, NPL>(now.v, now.any_id(group), group);
    float mean = 0.0f;
#pragma unroll
    for (int c = 0; c < NPL; ++c) mean = __builtin_fmaf(share[c], r.ex[c], mean);
    mean = token_sum<L>(mean) * r.inv;
    if (p.d_topk_w) {
      float ps[kSlots], weight = 0.0f, dot = 0.0f;
#pragma unroll
      for (int h = 0; h < kSlots; ++h) {
        ps[h] = now.id[h] >= 0 ? exp_neg(slot[h] - r.m) : 0.0f;
        weight += ps[h];
        dot = __builtin_fmaf(ps[h], dw[h], dot);
      }
      float inv = r.inv;
      if (p.renorm) {
        const float den = token_sum<L>(weight);
        inv = den < 1e-37f ? 0.0f : recip(den);  // NaN stays
      }
      dot = token_sum<L>(dot) * inv;
      if (!p.renorm) mean += dot;
      const float minus = p.renorm ? dot : 0.0f;
#pragma unroll
      for (int h = 0; h < kSlots; ++h)
        if (r.active && now.id[h] >= 0) atomicAdd(&add[now.id[h]], ps[h] * inv * (dw[h] - minus));
      __builtin_amdgcn_wave_barrier();
    }
    const float shift = losses && p.d_z ? (r.active ? cz * r.lse() : 0.0f) - mean : -mean;
    if (on) {
      float* rows_out = p.d_logits + first * E;
      const uint32_t at = (uint32_t)by * E;
      float out[NPL];
#pragma unroll
      for (int c = 0; c < NPL; ++c) {
        const float a = p.d_topk_w ? add[expert_of<L, kFull>(i, c)] : 0.0f;
        const float v = __builtin_fmaf(r.ex[c] * r.inv, share[c] + shift, a);
        out[c] = r.active ? v : 0.0f;
      }
      if constexpr (kFull) {
#pragma unroll
        for (int c = 0; c < NPL; c += 4)
          *reinterpret_cast<floatx4_t*>(rows_out + (at + expert_of<L, kFull>(i, c))) =
              floatx4_t{out[c], out[c + 1], out[c + 2], out[c + 3]};
      } else {
#pragma unroll
        for (int c = 0; c < NPL; ++c)
          if (i + L * c < E) rows_out[at + i + L * c] = out[c];
      }
    }
    if (p.d_topk_w) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int h = 0; h < kSlots; ++h)
        if (now.id[h] >= 0) add[now.id[h]] = 0.0f;
    }
  }
}

hipError_t launch_router_backward(const RouterGradParams& p, hipStream_t s) {
  // Up to four tokens to a group of lanes, which pays for its start, where that still leaves
  // sixteen waves for each CU.
  const int tokens = 4 * (p.E <= 128 ? 4 : 1);  // of a workgroup at a time
  const int rows = std::max({1, std::min(4, p.T / (1024 * tokens)), p.T / tokens / kMostGroups + 1});
  const int grid = (p.T + tokens * rows - 1) / (tokens * rows);
  const bool aligned = aligned16(p.logits) && aligned16(p.d_logits);
  PMOE_BY_LOGITS(p.E, (router_grad_kernel<L, NPL, kFull><<<grid, 256, 0, s>>>(p, rows)));
  return hipGetLastError();
}

}  // namespace pmoe
