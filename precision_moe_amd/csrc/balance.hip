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
// One wavefront holds one row: lane i the logits of experts i, i + 64, ... .
// The sums over tokens are taken in a fixed order without atomics on floats,
// so results do not vary between runs.
#include "device.h"
#include "kernels.h"

namespace pmoe {

typedef float floatx4_t __attribute__((ext_vector_type(4)));
constexpr float kNegInf = -__builtin_inff();

// Wave-wide sum and maximum by data-parallel-primitive moves (no LDS traffic): 1, 2, 4
// and 8 lanes up within rows of 16, then row 0 into 1 and 2 into 3, then 1 into 3; lane
// 63 ends with the result. A fixed order, so a fixed rounding.
template <int kCtrl, int kRows>
__device__ __forceinline__ float lane_move(float old, float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(__float_as_uint(old), __float_as_uint(v), kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum_f(float v) {
  v += lane_move<0x111, 0xf>(0.0f, v);
  v += lane_move<0x112, 0xf>(0.0f, v);
  v += lane_move<0x114, 0xf>(0.0f, v);
  v += lane_move<0x118, 0xf>(0.0f, v);
  v += lane_move<0x142, 0xa>(0.0f, v);
  v += lane_move<0x143, 0xc>(0.0f, v);
  return last_lane(v);
}
__device__ __forceinline__ float wave_max_f(float v) {
  v = __builtin_fmaxf(v, lane_move<0x111, 0xf>(v, v));
  v = __builtin_fmaxf(v, lane_move<0x112, 0xf>(v, v));
  v = __builtin_fmaxf(v, lane_move<0x114, 0xf>(v, v));
  v = __builtin_fmaxf(v, lane_move<0x118, 0xf>(v, v));
  v = __builtin_fmaxf(v, lane_move<0x142, 0xa>(v, v));
  v = __builtin_fmaxf(v, lane_move<0x143, 0xc>(v, v));
  return last_lane(v);
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

// The sequence of token t: the last s with offsets[s] <= t, -1 before the first
// and S behind the last. Every round the 64 lanes probe 64 places of the range.
__device__ __forceinline__ int sequence_of(const int* offsets, int S, int t, int lane) {
  if (offsets == nullptr) return 0;
  int lo = 0, n = S + 1;  // offsets[0 .. lo) <= t, offsets[lo + n ..) > t
  while (n > 0) {
    const int step = (n + 63) >> 6;
    const int at = lane * step;
    const int passed = __popcll(__ballot(at < n && offsets[lo + min(at, n - 1)] <= t));
    if (passed == 0) return lo - 1;
    const int base = (passed - 1) * step;  // this place is <= t, the next probe is not
    const int next = min(passed * step, n);
    lo += base + 1;
    n = next - base - 1;
  }
  return lo - 1;
}

// One row of logits in registers and what its softmax needs.
template <int NPL>
struct Row {
  float ex[NPL];  // exp(l - m); 0 behind E
  float m, sum, inv;
  bool active;
  __device__ __forceinline__ float lse() const { return m + logf(sum); }
};

template <int NPL>
__device__ __forceinline__ void load_logits(const float* row, int E, int lane, float (&v)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < E ? row[e] : kNegInf;
  }
}

template <int NPL>
__device__ __forceinline__ Row<NPL> softmax_row(const float (&v)[NPL], bool any_id) {
  Row<NPL> r;
  float m = v[0];
  bool some = !(v[0] == kNegInf);  // NaN counts: it has to come out as NaN
#pragma unroll
  for (int i = 1; i < NPL; ++i) {
    some |= !(v[i] == kNegInf);
    m = __builtin_fmaxf(m, v[i]);
  }
  r.m = wave_max_f(m);
  r.active = any_id && __ballot(some) != 0;
  if (!r.active) r.m = 0.0f;
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    r.ex[i] = exp_neg(v[i] - r.m);
    part += r.ex[i];
  }
  r.sum = wave_sum_f(part);
  r.inv = r.active ? recip(r.sum) : 0.0f;
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

// Workgroup c (16 waves, a row per wave at a time) takes the tokens [c * rows,
// (c + 1) * rows) and writes, for every sequence s that has tokens there, the
// slot c + s. Along the tokens either c or s grows from one (c, s) to the
// next, so the slot numbers differ; there are chunks + S of them at most. With
// kDirect there is one workgroup and one sequence, and it writes the results.
template <int NPL, bool kDirect>
__global__ __launch_bounds__(1024) void balance_rows_kernel(BalanceParams p, int rows) {
  __shared__ float prob[16][64 * NPL];
  __shared__ int count[64 * NPL];
  __shared__ float zsum[16];
  __shared__ int nact[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int T = p.T, E = p.E, K = p.K;
  const int* offsets = p.offsets;
  const int begin = blockIdx.x * rows, end = min(T, begin + rows);
  int t0 = begin;
  if (kDirect && offsets) t0 = min(max(offsets[0], 0), end);
  while (kDirect || t0 < end) {  // uniform: every wave sees the same offsets
    int s = 0, t1 = end;
    if (kDirect) {
      if (offsets) t1 = min(max(offsets[1], t0), end);
    } else {
      s = sequence_of(offsets, p.S, t0, lane);
      if (s >= p.S) break;
      if (s < 0) {
        t0 = min(end, max(offsets[0], t0 + 1));
        continue;
      }
      if (offsets) t1 = min(end, max(offsets[s + 1], t0 + 1));
    }
    for (int e = threadIdx.x; e < 64 * NPL; e += 1024) count[e] = 0;
    __syncthreads();
    float sum[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum[i] = 0.0f;
    float z = 0.0f;
    int n = 0;
    for (int t = t0 + wave; t < t1; t += 16) {
      float v[NPL];
      load_logits<NPL>(p.logits + (long)t * E, E, lane, v);
      const int id = lane < K ? expert_id(p.ids, p.ids64, (long)t * K + lane, E) : -1;
      const Row<NPL> r = softmax_row<NPL>(v, __ballot(id >= 0) != 0);
      if (r.active) {
        if (id >= 0) atomicAdd(&count[id], 1);
        const float lse = r.lse();
        n += 1;
        z += lse * lse;
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) sum[i] = __builtin_fmaf(r.ex[i], r.inv, sum[i]);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) prob[wave][lane + 64 * i] = sum[i];
    if (lane == 0) {
      zsum[wave] = z;
      nact[wave] = n;
    }
    __syncthreads();
    const int used = min(16, t1 - t0);  // waves that had a row, in wave order
    for (int e = threadIdx.x; e < E; e += 1024) {
      float q = prob[0][e];
      for (int w = 1; w < used; ++w) q += prob[w][e];
      prob[0][e] = q;
    }
    float zs = 0.0f;
    int ns = 0;
    for (int w = 0; w < 16; ++w) {
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
    for (int e = threadIdx.x; e < E; e += 1024) {
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
  __shared__ float prob[kMaxExperts];
  __shared__ int count[kMaxExperts];
  __shared__ float zsh[16];
  __shared__ int nsh[16];
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

// Up to this many tokens of one sequence go through one workgroup, in one launch.
constexpr int kDirectTokens = 128;

// Tokens of one workgroup: the square root of a sequence's mean length, so
// that the tokens of a workgroup and the slots of a sequence grow alike.
int balance_rows(int T, int S) {
  int rows = 4;
  while ((long)rows * rows * S < T) rows *= 2;
  return rows;
}

size_t balance_ws_bytes(int T, int E, int S) {
  const int rows = balance_rows(T, S);
  return ((size_t)(T + rows - 1) / rows + S) * balance_slot_words(E) * 4;
}

#define PMOE_BY_LOGITS(E, call)          \
  do {                                   \
    if ((E) <= 64) {                     \
      constexpr int NPL = 1;             \
      call;                              \
    } else if ((E) <= 128) {             \
      constexpr int NPL = 2;             \
      call;                              \
    } else if ((E) <= 256) {             \
      constexpr int NPL = 4;             \
      call;                              \
    } else if ((E) <= 512) {             \
      constexpr int NPL = 8;             \
      call;                              \
    } else {                             \
      constexpr int NPL = 16;            \
      call;                              \
    }                                    \
  } while (0)

hipError_t launch_router_balance(const BalanceParams& p, hipStream_t s) {
  if (p.S == 1 && p.T <= kDirectTokens) {
    PMOE_BY_LOGITS(p.E, (balance_rows_kernel<NPL, true><<<1, 1024, 0, s>>>(p, p.T)));
    return hipGetLastError();
  }
  const int rows = balance_rows(p.T, p.S);
  if (p.T > 0) {
    const int chunks = (p.T + rows - 1) / rows;
    PMOE_BY_LOGITS(p.E, (balance_rows_kernel<NPL, false><<<chunks, 1024, 0, s>>>(p, rows)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  int quads = 16;
  while (quads < balance_e4(p.E) / 2) quads *= 2;
  const int threads = p.S <= 256 ? 1024 : (quads < 256 ? 256 : quads);
  balance_sum_kernel<<<p.S, threads, 0, s>>>(p, rows, quads);
  return hipGetLastError();
}

// ---------------------------------------------------------------- backward
// A wave takes `rows` consecutive tokens and keeps the expert shares f of their
// sequence in registers while it stays the same; the next row's logits are on
// their way while one is worked on. With
//   u_e = d_balance E / n_s f_se + sum_{j: id_j = e} d w_j
// the terms that are not renormalized are p_e (u_e - sum p u + 2 d_z / n_s lse).
// The d w_j reach the lanes of their experts through a row of LDS that is zero
// between tokens.
template <int NPL>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradParams p, int rows) {
  __shared__ float direct_sh[4][64 * NPL];
  __shared__ float times_sh[4][64 * NPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int t0 = (blockIdx.x * 4 + wave) * rows, t1 = min(p.T, t0 + rows);
  const int E = p.E, K = p.K;
  float* direct = direct_sh[wave];  // used by this wave alone: its LDS operations stay in order
  float* times = times_sh[wave];
#pragma unroll
  for (int i = 0; i < NPL; ++i) direct[lane + 64 * i] = times[lane + 64 * i] = 0.0f;
  float share[NPL];  // d_balance E / n_s f_se
  float cz = 0.0f;   // 2 d_z / n_s
#pragma unroll
  for (int i = 0; i < NPL; ++i) share[i] = 0.0f;
  float next[NPL];
  if (t0 < t1) load_logits<NPL>(p.logits + (long)t0 * E, E, lane, next);
  const bool losses = p.tokens != nullptr;
  int seq_end = t0;  // the sequence in `share` holds the tokens up to here
  for (int t = t0; t < t1; ++t) {
    float v[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = next[i];
    const int id = lane < K ? expert_id(p.ids, p.ids64, (long)t * K + lane, E) : -1;
    const float dw = p.d_topk_w && id >= 0 ? p.d_topk_w[(long)t * K + lane] : 0.0f;
    if (t + 1 < t1) load_logits<NPL>(p.logits + (long)(t + 1) * E, E, lane, next);
    if (losses && t >= seq_end) {
      const int s = sequence_of(p.offsets, p.S, t, lane);
      const bool in = s >= 0 && s < p.S;  // else the losses do not see the token
      seq_end = in && p.offsets ? max(p.offsets[s + 1], t + 1) : (p.offsets ? t + 1 : p.T);
      const float n = in ? (float)max(p.tokens[s], 1) : 1.0f;
      cz = in && p.d_z ? 2.0f * p.d_z[s] / n : 0.0f;
      const float cb = in && p.d_balance ? p.d_balance[s] * ((float)E / (n * n * (float)K)) : 0.0f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 64 * i;
        share[i] = in && p.d_balance && e < E ? cb * (float)p.counts[(long)s * E + e] : 0.0f;
      }
    }
    const Row<NPL> r = softmax_row<NPL>(v, __ballot(id >= 0) != 0);
    float* out = p.d_logits + (long)t * E;
    if (!r.active) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (lane + 64 * i < E) out[lane + 64 * i] = 0.0f;
      continue;
    }
    float u[NPL], top[NPL];  // top: the renormalized part of the gradient
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      u[i] = share[i];
      top[i] = 0.0f;
    }
    if (p.d_topk_w) {
      if (id >= 0) atomicAdd(&direct[id], dw);
      if (id >= 0 && p.renorm) atomicAdd(&times[id], 1.0f);  // slots of the expert
      __builtin_amdgcn_wave_barrier();
      if (p.renorm) {
        float den = 0.0f, num = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          den = __builtin_fmaf(times[lane + 64 * i], r.ex[i], den);
          num = __builtin_fmaf(direct[lane + 64 * i], r.ex[i], num);
        }
        den = wave_sum_f(den);
        num = wave_sum_f(num);
        const float inv = den > 0.0f ? recip(den) : 0.0f;
        const float mean = num * inv;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          top[i] = r.ex[i] * inv * (direct[lane + 64 * i] - times[lane + 64 * i] * mean);
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) u[i] += direct[lane + 64 * i];
      }
      __builtin_amdgcn_wave_barrier();
      if (id >= 0) direct[id] = times[id] = 0.0f;
    }
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) mean = __builtin_fmaf(u[i], r.ex[i], mean);
    mean = wave_sum_f(mean) * r.inv;
    const float zt = losses && p.d_z ? cz * r.lse() : 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane + 64 * i < E)
        out[lane + 64 * i] = __builtin_fmaf(r.ex[i] * r.inv, (u[i] - mean) + zt, top[i]);
  }
}

hipError_t launch_router_backward(const RouterGradParams& p, hipStream_t s) {
  const int rows = p.T >= 32768 ? 4 : 1;
  const int grid = (p.T + 4 * rows - 1) / (4 * rows);
  PMOE_BY_LOGITS(p.E, (router_grad_kernel<NPL><<<grid, 256, 0, s>>>(p, rows)));
  return hipGetLastError();
}

}  // namespace pmoe
