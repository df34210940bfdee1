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

constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float wave_sum_f(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
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
  float ex[NPL];  // exp(l - m)
  float inv;      // 1 / sum of ex
  float lse;
  bool active;
};

template <int NPL>
__device__ __forceinline__ Row<NPL> load_row(const float* row, int E, int lane, bool any_id) {
  Row<NPL> r;
  float m = kNegInf;
  bool some = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 64 * i;
    r.ex[i] = e < E ? row[e] : kNegInf;
    some |= !(r.ex[i] == kNegInf);  // NaN counts: it has to come out as NaN
    m = __builtin_fmaxf(m, r.ex[i]);
  }
  m = wave_max(m);
  r.active = any_id && __ballot(some) != 0;
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    r.ex[i] = r.active && lane + 64 * i < E ? expf(r.ex[i] - m) : 0.0f;
    part += r.ex[i];
  }
  part = wave_sum_f(part);
  r.inv = r.active ? 1.0f / part : 0.0f;
  r.lse = r.active ? m + logf(part) : 0.0f;
  return r;
}

// ---------------------------------------------------------------- forward
// Workgroup c takes the tokens [c * rows, (c + 1) * rows) and writes, for every
// sequence s that has tokens there, the slot c + s: probability sums [E], route
// counts [E], the sum of lse^2 and the number of active tokens. Along the
// tokens either c or s grows from one (c, s) to the next, so the slot numbers
// differ; there are chunks + S of them at most.
__host__ __device__ inline long balance_slot_words(int E) { return 2L * E + 2; }

template <int NPL>
__global__ __launch_bounds__(256) void balance_rows_kernel(
    const float* __restrict__ logits, const void* __restrict__ ids, int ids64, int T, int E, int K,
    const int* __restrict__ offsets, int S, int rows, float* __restrict__ slots) {
  __shared__ float prob[4][64 * NPL];
  __shared__ int count[64 * NPL];
  __shared__ float zsum[4];
  __shared__ int nact[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int begin = blockIdx.x * rows, end = min(T, begin + rows);
  int t0 = begin;
  while (t0 < end) {  // uniform: every wave sees the same offsets
    const int s = sequence_of(offsets, S, t0, lane);
    if (s >= S) break;
    if (s < 0) {
      t0 = min(end, max(offsets[0], t0 + 1));
      continue;
    }
    const int t1 = offsets ? min(end, max(offsets[s + 1], t0 + 1)) : end;
    for (int e = threadIdx.x; e < E; e += 256) count[e] = 0;
    __syncthreads();
    float sum[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) sum[i] = 0.0f;
    float z = 0.0f;
    int n = 0;
    for (int t = t0 + wave; t < t1; t += 4) {
      const int id = lane < K ? expert_id(ids, ids64, (long)t * K + lane, E) : -1;
      const Row<NPL> r = load_row<NPL>(logits + (long)t * E, E, lane, __ballot(id >= 0) != 0);
      if (r.active) {
        if (id >= 0) atomicAdd(&count[id], 1);
        n += 1;
        z += r.lse * r.lse;
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) sum[i] += r.ex[i] * r.inv;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) prob[wave][lane + 64 * i] = sum[i];
    if (lane == 0) {
      zsum[wave] = z;
      nact[wave] = n;
    }
    __syncthreads();
    float* slot = slots + (blockIdx.x + s) * balance_slot_words(E);
    for (int e = threadIdx.x; e < E; e += 256) {
      slot[e] = ((prob[0][e] + prob[1][e]) + prob[2][e]) + prob[3][e];
      reinterpret_cast<int*>(slot)[E + e] = count[e];
    }
    if (threadIdx.x == 0) {
      slot[2 * E] = ((zsum[0] + zsum[1]) + zsum[2]) + zsum[3];
      reinterpret_cast<int*>(slot)[2 * E + 1] = nact[0] + nact[1] + nact[2] + nact[3];
    }
    __syncthreads();
    t0 = t1;
  }
}

// One workgroup of 1024 threads per sequence adds its slots: 1024 / cols groups
// of threads take every (1024 / cols)-th slot, a thread one column.
__global__ __launch_bounds__(1024) void balance_sum_kernel(
    const float* __restrict__ slots, int T, int E, int K, const int* __restrict__ offsets, int rows,
    int cols, int* __restrict__ counts, int* __restrict__ tokens, float* __restrict__ prob,
    float* __restrict__ balance, float* __restrict__ z) {
  __shared__ float psh[1024];
  __shared__ int csh[1024];
  __shared__ float zsh[16];
  __shared__ int nsh[16];
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int a = offsets ? min(max(offsets[s], 0), T) : 0;
  const int b = offsets ? min(max(offsets[s + 1], 0), T) : T;
  const int c0 = a / rows, c1 = a < b ? (b - 1) / rows + 1 : c0;
  const long words = balance_slot_words(E);
  const int groups = 1024 / cols, grp = tid / cols, col = tid % cols;
  // the number of active tokens and the sum of lse^2
  float zs = 0.0f;
  int ns = 0;
  for (int c = c0 + tid; c < c1; c += 1024) {
    const float* slot = slots + (c + s) * words;
    zs += slot[2 * E];
    ns += reinterpret_cast<const int*>(slot)[2 * E + 1];
  }
  zs = wave_sum_f(zs);
  ns = wave_sum(ns);
  if (lane == 0) {
    zsh[wave] = zs;
    nsh[wave] = ns;
  }
  float ps = 0.0f;
  int cs = 0;
  if (col < E)
    for (int c = c0 + grp; c < c1; c += groups) {
      const float* slot = slots + (c + s) * words;
      ps += slot[col];
      cs += reinterpret_cast<const int*>(slot)[E + col];
    }
  psh[tid] = ps;
  csh[tid] = cs;
  __syncthreads();
  zs = 0.0f;
  ns = 0;
  for (int w = 0; w < 16; ++w) {
    zs += zsh[w];
    ns += nsh[w];
  }
  float term = 0.0f;
  if (tid < E) {  // E <= cols, so group 0 holds every column
    ps = psh[tid];
    cs = csh[tid];
    for (int g = 1; g < groups; ++g) {
      ps += psh[g * cols + tid];
      cs += csh[g * cols + tid];
    }
    counts[(long)s * E + tid] = cs;
    prob[(long)s * E + tid] = ps;
    term = (float)cs * ps;
  }
  term = wave_sum_f(term);
  __syncthreads();
  if (lane == 0) zsh[wave] = term;
  __syncthreads();
  if (tid == 0) {
    float sum = 0.0f;
    for (int w = 0; w < 16; ++w) sum += zsh[w];
    const float n = (float)max(ns, 1);
    tokens[s] = ns;
    balance[s] = (float)E / (float)K * (sum / n) / n;
    z[s] = zs / n;
  }
}

// Rows of one workgroup: enough workgroups to fill the GPU, few enough slots
// for the second kernel.
int balance_rows(int T) {
  int rows = 16;
  while (rows < 1024 && (long)rows * 512 < T) rows *= 2;
  return rows;
}

size_t balance_ws_bytes(int T, int E, int S) {
  const int rows = balance_rows(T);
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
  const int rows = balance_rows(p.T);
  float* slots = static_cast<float*>(p.ws);
  if (p.T > 0) {
    const int chunks = (p.T + rows - 1) / rows;
    PMOE_BY_LOGITS(p.E, (balance_rows_kernel<NPL><<<chunks, 256, 0, s>>>(
                            p.logits, p.ids, p.ids64, p.T, p.E, p.K, p.offsets, p.S, rows, slots)));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  int cols = 64;
  while (cols < p.E) cols *= 2;
  balance_sum_kernel<<<p.S, 1024, 0, s>>>(slots, p.T, p.E, p.K, p.offsets, rows, cols, p.counts,
                                          p.tokens, p.prob, p.balance, p.z);
  return hipGetLastError();
}

// ---------------------------------------------------------------- backward
// A wave takes `rows` consecutive tokens and keeps the expert shares f of their
// sequence in registers while it stays the same. With
//   u_e = d_balance E / n_s f_se + sum_{j: id_j = e} d w_j
// the terms that are not renormalized are p_e (u_e - sum p u + 2 d_z / n_s lse).
template <int NPL>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradParams p, int rows) {
  const int lane = threadIdx.x & 63;
  const int t0 = (blockIdx.x * 4 + (threadIdx.x >> 6)) * rows;
  const int E = p.E, K = p.K;
  float share[NPL];  // d_balance E / n_s f_se
  float cz = 0.0f;   // 2 d_z / n_s
#pragma unroll
  for (int i = 0; i < NPL; ++i) share[i] = 0.0f;
  int have = -2;
  for (int t = t0; t < min(p.T, t0 + rows); ++t) {
    const int s = sequence_of(p.offsets, p.S, t, lane);
    if (s != have) {
      have = s;
      const bool in = p.tokens && s >= 0 && s < p.S;  // else the losses do not see the token
      const float n = in ? (float)max(p.tokens[s], 1) : 1.0f;
      cz = in && p.d_z ? 2.0f * p.d_z[s] / n : 0.0f;
      const float cb = in && p.d_balance ? p.d_balance[s] * ((float)E / (n * n * (float)K)) : 0.0f;
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = lane + 64 * i;
        share[i] = in && p.d_balance && e < E ? cb * (float)p.counts[(long)s * E + e] : 0.0f;
      }
    }
    const int id = lane < K ? expert_id(p.ids, p.ids64, (long)t * K + lane, E) : -1;
    const Row<NPL> r = load_row<NPL>(p.logits + (long)t * E, E, lane, __ballot(id >= 0) != 0);
    float* out = p.d_logits + (long)t * E;
    if (!r.active) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (lane + 64 * i < E) out[lane + 64 * i] = 0.0f;
      continue;
    }
    float u[NPL], prob[NPL], top[NPL];  // top: the renormalized part of the gradient
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      u[i] = share[i];
      prob[i] = r.ex[i] * r.inv;
      top[i] = 0.0f;
    }
    if (p.d_topk_w) {
      const float dw = id >= 0 ? p.d_topk_w[(long)t * K + lane] : 0.0f;
      float direct[NPL], times[NPL];  // sum of d w_j and number of slots of each expert
#pragma unroll
      for (int i = 0; i < NPL; ++i) direct[i] = times[i] = 0.0f;
      for (int j = 0; j < K; ++j) {
        const int ej = __shfl(id, j, 64);
        const float dj = __shfl(dw, j, 64);
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (ej == lane + 64 * i) {
            direct[i] += dj;
            times[i] += 1.0f;
          }
      }
      if (p.renorm) {
        float den = 0.0f, num = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          den += times[i] * r.ex[i];
          num += direct[i] * r.ex[i];
        }
        den = wave_sum_f(den);
        num = wave_sum_f(num);
        const float inv = den > 0.0f ? 1.0f / den : 0.0f;
        const float mean = num * inv;
#pragma unroll
        for (int i = 0; i < NPL; ++i) top[i] = r.ex[i] * inv * (direct[i] - times[i] * mean);
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) u[i] += direct[i];
      }
    }
    float mean = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) mean += u[i] * prob[i];
    mean = wave_sum_f(mean);
    const float zt = cz * r.lse;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (lane + 64 * i < E) out[lane + 64 * i] = prob[i] * ((u[i] - mean) + zt) + top[i];
  }
}

hipError_t launch_router_backward(const RouterGradParams& p, hipStream_t s) {
  const int rows = p.T >= 32768 ? 4 : 1;
  const int grid = (p.T + 4 * rows - 1) / (4 * rows);
  PMOE_BY_LOGITS(p.E, (router_grad_kernel<NPL><<<grid, 256, 0, s>>>(p, rows)));
  return hipGetLastError();
}

}  // namespace pmoe
