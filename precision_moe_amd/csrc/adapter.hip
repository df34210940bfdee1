// Low-rank adapters of many requests beside one shared projection. Token t uses
// adapter a = ids[t] (none if outside [0, n)), with down matrix A_a [R, H], up
// matrix B_a [N, R] and scale s_a:
//   v_t = A_a x_t  (FP32),        out_t = bf16(base_t + s_a B_a v_t),
// and for the gradient dy of out
//   du_t = s_a B_a^T dy_t,        dx_t = bf16(base_t + A_a^T du_t),
//   dA_a = sum_t du_t x_t^T,      dB_a = s_a sum_t dy_t v_t^T.
// R is small (8 .. 128), so x, dy, base and the outputs are what has to move;
// the matrices of one adapter stay in the caches while its tokens pass.
//
// Grouping. Tokens need not be sorted. A workgroup owns 64 consecutive tokens;
// every wave finds by ballots which of them share an adapter and works on one
// such group after the other, its rows gathered into blocks of 16 (the width of
// one MFMA). No plan is built and nothing is kept between calls. In a prompt
// the 64 tokens are one or two groups; in a decode step they may be 64, and
// then gridDim.z workgroups share the groups of one block of tokens.
//
// Bits of a token do not depend on the other tokens of the call: a column of an
// MFMA depends on its own operand column only, and how a sum over H (or N) is
// cut into parts follows from H (or N) alone.
//
// All products run on v_mfma_f32_16x16x32_bf16 (lane l holds row or column
// l % 16 and the eight k of group l / 16; the result lane holds column l % 16
// and rows 4 (l / 16) + 0..3). FP32 factors (v, du) enter as sums of BF16
// values: two (16 significant bits) where the result is rounded to BF16 (8
// bits), three (24 bits, all of FP32) where it stays FP32.
#include "device.h"
#include "kernels.h"

namespace pmoe {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int kTok = 64;  // tokens of one workgroup

__device__ __forceinline__ floatx4 mfma16(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ bf16x8_t as_bf16x8(uint4 u) { return __builtin_bit_cast(bf16x8_t, u); }

__device__ __forceinline__ int adapter_of(const void* ids, int ids64, long t, int n) {
  const long long id = ids64 ? static_cast<const long long*>(ids)[t] : static_cast<const int*>(ids)[t];
  return id >= 0 && id < n ? (int)id : -1;
}

// The groups of a block of 64 tokens, one after the other, the same in every
// wave. After next(): `adapter` and `count` of the group; lane m of `member`
// holds the place (0..63) of the group's m-th token for m < count.
struct Groups {
  int id;          // of this lane's token; -1: none, -2: behind the last token
  uint64_t left;   // tokens not yet handled
  int adapter, count, member;
  __device__ __forceinline__ Groups(const void* ids, int ids64, long t0, int T, int n, bool with_none,
                                    int lane) {
    id = t0 + lane < T ? adapter_of(ids, ids64, t0 + lane, n) : -2;
    left = __ballot(id >= (with_none ? -1 : 0));
  }
  __device__ __forceinline__ bool next(int lane) {
    if (left == 0) return false;
    adapter = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t match = __ballot(id == adapter);
    left &= ~match;
    count = __popcll(match);
    const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
    // members to the front, the others behind them: every lane sends its place
    const int in = __popcll(match & below);
    const int to = (match >> lane) & 1 ? in : count + (lane - in);
    member = __builtin_amdgcn_ds_permute(to * 4, lane);
    return true;
  }
};

// ---------------------------------------------------------------- reduction over H (or N)
// Parts of the sum over a row of D elements: gridDim.y workgroups of four waves
// each take a span of `span` elements (a multiple of 64) per wave. Chosen from
// D alone.
int adapter_parts(int D) {
  const int p = (D + 1023) / 1024;
  return p < 8 ? p : 8;
}
static int adapter_span(int D) { return ((D + adapter_parts(D) * 4 - 1) / (adapter_parts(D) * 4) + 63) / 64 * 64; }

// 16 elements of column r of W [D][R] from row k on, as the two operands that
// belong to 16 consecutive elements of a row.
__device__ __forceinline__ void load_column16(const uint16_t* w, int R, uint4& lo, uint4& hi) {
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (uint32_t)w[(long)(2 * i) * R] | ((uint32_t)w[(long)(2 * i + 1) * R] << 16);
  lo = make_uint4(v[0], v[1], v[2], v[3]);
  hi = make_uint4(v[4], v[5], v[6], v[7]);
}

// part[y][t][r] = sum over the y-th part of in[t][k] * W_a[r][k] (kTrans: W_a[k][r]).
template <int NR, bool kTrans>
__global__ __launch_bounds__(256) void adapter_reduce_kernel(
    const uint16_t* __restrict__ in, const void* __restrict__ ids, int ids64, int T, int n, int D, int R,
    const uint16_t* __restrict__ W, int span, float* __restrict__ part) {
  __shared__ floatx4 red[4][NR][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, g = lane >> 4;
  const long t0 = (long)blockIdx.x * kTok;
  const int k_begin = (blockIdx.y * 4 + wave) * span, k_end = min(D, k_begin + span);
  float* dst = part + (long)blockIdx.y * T * R;
  Groups grp(ids, ids64, t0, T, n, false, lane);
  for (int gi = 0; grp.next(lane); ++gi) {
    if (gi % gridDim.z != blockIdx.z) continue;
    const int nf = (grp.count + 15) >> 4;
    const uint16_t* x[4];
    bool on[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int m = 16 * f + col;
      on[f] = m < grp.count;
      x[f] = in + (t0 + __shfl(grp.member, on[f] ? m : 0, 64)) * D;
    }
    const uint16_t* w = W + (long)grp.adapter * R * D;
    floatx4 acc[4][NR];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int c = 0; c < NR; ++c) acc[f][c] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = k_begin; k0 < k_end; k0 += 64) {
      const int k = k0 + 16 * g;  // D is a multiple of 16: these 16 elements are in or out together
      const bool in_row = k < k_end;
      uint4 wl[NR], wh[NR];
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        const int r = 16 * c + col;
        wl[c] = wh[c] = make_uint4(0, 0, 0, 0);
        if (in_row && r < R) {
          if (kTrans) {
            load_column16(w + (long)k * R + r, R, wl[c], wh[c]);
          } else {
            wl[c] = *reinterpret_cast<const uint4*>(w + (long)r * D + k);
            wh[c] = *reinterpret_cast<const uint4*>(w + (long)r * D + k + 8);
          }
        }
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (f >= nf) continue;
        uint4 xl = make_uint4(0, 0, 0, 0), xh = xl;
        if (in_row && on[f]) {
          xl = *reinterpret_cast<const uint4*>(x[f] + k);
          xh = *reinterpret_cast<const uint4*>(x[f] + k + 8);
        }
#pragma unroll
        for (int c = 0; c < NR; ++c) {
          acc[f][c] = mfma16(as_bf16x8(wl[c]), as_bf16x8(xl), acc[f][c]);
          acc[f][c] = mfma16(as_bf16x8(wh[c]), as_bf16x8(xh), acc[f][c]);
        }
      }
    }
    // the four waves' sums, in wave order
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      if (f >= nf) continue;
#pragma unroll
      for (int c = 0; c < NR; ++c) red[wave][c][lane] = acc[f][c];
      __syncthreads();
      const int m = 16 * f + col;
      const long t = t0 + __shfl(grp.member, m, 64);
      for (int c = wave; c < NR; c += 4) {
        const floatx4 s = ((red[0][c][lane] + red[1][c][lane]) + red[2][c][lane]) + red[3][c][lane];
        const int r = 16 * c + 4 * g;
        if (m < grp.count && r < R) *reinterpret_cast<floatx4*>(dst + t * R + r) = s;
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- expansion to N (or H)
// x = hi + lo in BF16, 16 significant bits. An infinite x has lo = 0.
__device__ __forceinline__ void split2(float x, uint16_t& hi, uint16_t& lo) {
  hi = (uint16_t)f32_to_bf16(x);
  const float rest = x - bf16_to_f32(hi);
  lo = (uint16_t)f32_to_bf16(__builtin_fabsf(x) == __builtin_inff() ? 0.0f : rest);
}

// Rows of the low-rank vectors of a group in LDS: the sum of the parts (in
// order) times the adapter's scale, as hi and lo. With R <= 16 one row holds
// hi[16] lo[16], which fill the 32 k of one MFMA; with more, hi[] and lo[] are
// planes of whole steps of 32 that meet the same operand of the matrix.
template <int NR>
struct LowRows {
  static constexpr int kSteps = NR == 1 ? 1 : NR / 2;
  static constexpr int kWidth = NR == 1 ? 32 : 2 * 32 * kSteps;  // BF16 values of a row
  static constexpr int kStride = kWidth + 8;
  uint16_t v[kTok][kStride];
};

// out[t][c] = bf16(base[t][c] + sum_r low[t][r] W_a[c][r]) (kTrans: W_a[r][c]),
// low = scale * (sum of the parts). Workgroups with blockIdx.y == 0 also write the sum
// of the parts to `sums` (times the scale if scale_sums), 0 without an adapter.
template <int NR, bool kTrans>
__global__ __launch_bounds__(256) void adapter_expand_kernel(
    const float* __restrict__ part, int parts, const void* __restrict__ ids, int ids64, int T, int n,
    int D, int R, const uint16_t* __restrict__ W, const float* __restrict__ scale,
    const uint16_t* base, uint16_t* out, float* __restrict__ sums, int scale_sums, int chunk) {
  using Low = LowRows<NR>;
  __shared__ __align__(16) Low low;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  const long t0 = (long)blockIdx.x * kTok;
  const int c_begin = blockIdx.y * chunk, c_end = min(D, c_begin + chunk);
  // tokens without an adapter: base, or zeros
  const bool fill = out != nullptr && base != out;
  Groups grp(ids, ids64, t0, T, n, true, lane);
  for (int gi = 0; grp.next(lane); ++gi) {
    if (gi % gridDim.z != blockIdx.z) continue;
    if (grp.adapter < 0) {
      for (int m = 0; m < grp.count; ++m) {
        const long t = t0 + __builtin_amdgcn_readlane(grp.member, m);
        if (fill)
          for (int c = c_begin + tid * 8; c < c_end; c += 2048)
            *reinterpret_cast<uint4*>(out + t * D + c) =
                base ? *reinterpret_cast<const uint4*>(base + t * D + c) : make_uint4(0, 0, 0, 0);
        if (blockIdx.y == 0 && sums != nullptr)
          for (int r = tid; r < R; r += 256) sums[t * R + r] = 0.0f;
      }
      continue;
    }
    const int nf = (grp.count + 15) >> 4;
    const float s = scale[grp.adapter];
    __syncthreads();  // the rows of the group before are no longer read
    for (int i = tid; i < nf * 16 * (16 * NR / 4); i += 256) {
      const int m = i / (16 * NR / 4), r = i % (16 * NR / 4) * 4;
      const long t = t0 + __shfl(grp.member, m, 64);  // whole waves come here
      floatx4 v = {0.0f, 0.0f, 0.0f, 0.0f};
      if (m < grp.count && r < R) {
        for (int p = 0; p < parts; ++p)
          v += *reinterpret_cast<const floatx4*>(part + ((long)p * T + t) * R + r);
        if (blockIdx.y == 0 && sums != nullptr)
          *reinterpret_cast<floatx4*>(sums + t * R + r) = scale_sums ? v * s : v;
      }
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) split2(v[j] * s, hi[j], lo[j]);
      const int lo_at = NR == 1 ? 16 : Low::kWidth / 2;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        low.v[m][r + j] = hi[j];
        low.v[m][lo_at + r + j] = lo[j];
      }
    }
    __syncthreads();
    if (out == nullptr) continue;
    const uint16_t* w = W + (long)grp.adapter * R * D;
    if (!kTrans) {
      // 64 columns at a time: operand row i of block b is column 16 (i / 4) + 4 b + i % 4, so
      // that a lane's four blocks end as 16 consecutive columns of one token.
      for (int c0 = c_begin + 64 * wave; c0 < c_end; c0 += 256) {
        uint4 wop[Low::kSteps][4];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int c = c0 + 16 * (col >> 2) + 4 * b + (col & 3);
#pragma unroll
          for (int q = 0; q < Low::kSteps; ++q) {
            const int r = NR == 1 ? 8 * (g & 1) : 32 * q + 8 * g;
            wop[q][b] = make_uint4(0, 0, 0, 0);
            if (c < D && r < R) wop[q][b] = *reinterpret_cast<const uint4*>(w + (long)c * R + r);
          }
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          if (f >= nf) continue;
          floatx4 acc[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) acc[b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
          const uint16_t* row = low.v[16 * f + col];
#pragma unroll
          for (int q = 0; q < Low::kSteps; ++q) {
            const uint4 vh = *reinterpret_cast<const uint4*>(row + 32 * q + 8 * g);
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[b] = mfma16(as_bf16x8(wop[q][b]), as_bf16x8(vh), acc[b]);
            if (NR > 1) {
              const uint4 vl = *reinterpret_cast<const uint4*>(row + Low::kWidth / 2 + 32 * q + 8 * g);
#pragma unroll
              for (int b = 0; b < 4; ++b) acc[b] = mfma16(as_bf16x8(wop[q][b]), as_bf16x8(vl), acc[b]);
            }
          }
          const int m = 16 * f + col, c = c0 + 16 * g;
          const long at = (t0 + __shfl(grp.member, m, 64)) * D + c;
          if (m < grp.count && c < D) {
            uint32_t o[8];
            uint32_t bv[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (base) {
              const uint4 b0 = *reinterpret_cast<const uint4*>(base + at);
              const uint4 b1 = *reinterpret_cast<const uint4*>(base + at + 8);
              bv[0] = b0.x, bv[1] = b0.y, bv[2] = b0.z, bv[3] = b0.w;
              bv[4] = b1.x, bv[5] = b1.y, bv[6] = b1.z, bv[7] = b1.w;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              o[j] = f32x2_to_bf16x2(bf16_to_f32(bv[j] & 0xFFFFu) + acc[j / 2][2 * (j & 1)],
                                     bf16_to_f32(bv[j] >> 16) + acc[j / 2][2 * (j & 1) + 1]);
            *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(out + at + 8) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        }
      }
    } else {
      // 128 columns at a time. W_a has its columns contiguous, an operand wants eight r of one
      // column: lane (col, g) loads eight rows r of the columns 8 col .. 8 col + 7 and turns
      // that 8 x 8 block in registers; operand row i of block b is column 8 i + b, so a lane
      // ends with the 32 consecutive columns 32 g + 8 i + b of one token.
      for (int c0 = c_begin + 128 * wave; c0 < c_end; c0 += 512) {
        floatx4 acc[4][8];
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
          for (int b = 0; b < 8; ++b) acc[f][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        const int c = c0 + 8 * col;
#pragma unroll
        for (int q = 0; q < Low::kSteps; ++q) {
          const int r0 = NR == 1 ? 8 * (g & 1) : 32 * q + 8 * g;
          uint32_t in[8][4];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (c < D && r0 < R) u = *reinterpret_cast<const uint4*>(w + (long)(r0 + j) * D + c);
            in[j][0] = u.x, in[j][1] = u.y, in[j][2] = u.z, in[j][3] = u.w;
          }
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const uint32_t sel = b & 1 ? 0x07060302u : 0x05040100u;
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(in[2 * j + 1][b / 2], in[2 * j][b / 2], sel);
            const bf16x8_t wop = as_bf16x8(make_uint4(o[0], o[1], o[2], o[3]));
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              if (f >= nf) continue;
              const uint16_t* row = low.v[16 * f + col];
              acc[f][b] = mfma16(wop, as_bf16x8(*reinterpret_cast<const uint4*>(row + 32 * q + 8 * g)), acc[f][b]);
              if (NR > 1)
                acc[f][b] = mfma16(wop, as_bf16x8(*reinterpret_cast<const uint4*>(
                                            row + Low::kWidth / 2 + 32 * q + 8 * g)), acc[f][b]);
            }
          }
        }
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          if (f >= nf) continue;
          const int m = 16 * f + col;
          const long t = t0 + __shfl(grp.member, m, 64);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int cc = c0 + 32 * g + 8 * i;
            if (m < grp.count && cc < D) {
              const long at = t * D + cc;
              uint4 bb = make_uint4(0, 0, 0, 0);
              if (base) bb = *reinterpret_cast<const uint4*>(base + at);
              const uint32_t bv[4] = {bb.x, bb.y, bb.z, bb.w};
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                o[j] = f32x2_to_bf16x2(bf16_to_f32(bv[j] & 0xFFFFu) + acc[f][2 * j][i],
                                       bf16_to_f32(bv[j] >> 16) + acc[f][2 * j + 1][i]);
              *reinterpret_cast<uint4*>(out + at) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- gradients of the matrices
// x = h + m + l in BF16: all 24 bits of an FP32 value (in range; an infinite x has m = l = 0).
__device__ __forceinline__ void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
  h = f32_to_bf16(x);
  const float r1 = __builtin_fabsf(x) == __builtin_inff() ? 0.0f : x - bf16_to_f32(h);
  m = f32_to_bf16(r1);
  l = f32_to_bf16(r1 - bf16_to_f32(m));
}

constexpr int kSegMax = 4096;  // tokens of one segment, whose list of one adapter is kept in LDS
constexpr int kGradCols = 128;

struct GradParams {
  const uint16_t* x;    // [T][H]
  const uint16_t* dy;   // [T][N]
  const float* du;      // [T][R], scaled
  const float* v;       // [T][R]
  const float* scale;   // [n]
  const void* ids;
  int ids64, T, n, H, N, R, seg;
  float* d_down;        // [n][R][H], or with several segments the partial sums [segments][n][R][H]
  float* d_up;          // [n][N][R], likewise
};

// One workgroup: adapter blockIdx.y, segment blockIdx.z, 128 columns of x (dA)
// or, behind those, of dy (dB), and 16 NR values of r (with R > 64 there are two
// such halves: more than 4 x 8 accumulators of 4 do not fit the registers). The adapter's tokens of the segment are listed
// in LDS, the waves take every fourth step of 32 of them. k is the token here,
// so both operands are wanted with eight tokens of one column: x (dy) is turned
// in registers as in the expansion, du (s v) is read column by column.
template <int NR>
__global__ __launch_bounds__(256) void adapter_grad_kernel(GradParams p) {
  __shared__ int list[kSegMax + 32];
  __shared__ int wave_count[4];
  __shared__ floatx4 red[4][8][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  const int a = blockIdx.y, seg0 = blockIdx.z * p.seg;
  const int seg1 = min(p.T, seg0 + p.seg);
  const int down_chunks = (p.H + kGradCols - 1) / kGradCols;
  const int chunks = down_chunks + (p.N + kGradCols - 1) / kGradCols;
  const int chunk = blockIdx.x % chunks, r_begin = blockIdx.x / chunks * (16 * NR);
  const bool down = chunk < down_chunks;
  const int c0 = (down ? chunk : chunk - down_chunks) * kGradCols;
  const int D = down ? p.H : p.N, R = p.R;
  const uint16_t* in = down ? p.x : p.dy;
  const float* low = down ? p.du : p.v;
  const float s = down ? 1.0f : p.scale[a];
  // the adapter's tokens, in order
  int have = 0;
  for (int b = seg0; b < seg1; b += 256) {
    const int t = b + tid;
    const bool mine = t < seg1 && adapter_of(p.ids, p.ids64, t, p.n) == a;
    const uint64_t match = __ballot(mine);
    if (lane == 0) wave_count[wave] = __popcll(match);
    __syncthreads();
    int at = have;
    for (int w = 0; w < 4; ++w) {
      if (w < wave) at += wave_count[w];
      have += wave_count[w];
    }
    const uint64_t below = lane == 0 ? 0ull : (~0ull >> (64 - lane));
    if (mine) list[at + __popcll(match & below)] = t;
    __syncthreads();
  }
  if (tid < 32) list[have + tid] = -1;
  __syncthreads();
  floatx4 acc[NR][8];
#pragma unroll
  for (int c = 0; c < NR; ++c)
#pragma unroll
    for (int b = 0; b < 8; ++b) acc[c][b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
  const int cc = c0 + 8 * col;
  for (int k0 = 32 * wave; k0 < have; k0 += 128) {
    int tok[8];
    uint32_t q[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      tok[j] = list[k0 + 8 * g + j];
      uint4 u = make_uint4(0, 0, 0, 0);
      if (tok[j] >= 0 && cc < D) u = *reinterpret_cast<const uint4*>(in + (long)tok[j] * D + cc);
      q[j][0] = u.x, q[j][1] = u.y, q[j][2] = u.z, q[j][3] = u.w;
    }
    bf16x8_t op[8];
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t sel = b & 1 ? 0x07060302u : 0x05040100u;
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = __builtin_amdgcn_perm(q[2 * j + 1][b / 2], q[2 * j][b / 2], sel);
      op[b] = as_bf16x8(make_uint4(o[0], o[1], o[2], o[3]));
    }
#pragma unroll
    for (int c = 0; c < NR; ++c) {
      const int r = r_begin + 16 * c + col;
      uint32_t h[8], m[8], l[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = tok[j] >= 0 && r < R ? low[(long)tok[j] * R + r] * s : 0.0f;
        split3(f, h[j], m[j], l[j]);
      }
      uint4 ho, mo, lo;
      ho = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
      mo = make_uint4(m[0] | m[1] << 16, m[2] | m[3] << 16, m[4] | m[5] << 16, m[6] | m[7] << 16);
      lo = make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16, l[4] | l[5] << 16, l[6] | l[7] << 16);
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (down) {  // rows: columns of x, columns: r
          acc[c][b] = mfma16(op[b], as_bf16x8(lo), acc[c][b]);
          acc[c][b] = mfma16(op[b], as_bf16x8(mo), acc[c][b]);
          acc[c][b] = mfma16(op[b], as_bf16x8(ho), acc[c][b]);
        } else {     // rows: r, columns: columns of dy
          acc[c][b] = mfma16(as_bf16x8(lo), op[b], acc[c][b]);
          acc[c][b] = mfma16(as_bf16x8(mo), op[b], acc[c][b]);
          acc[c][b] = mfma16(as_bf16x8(ho), op[b], acc[c][b]);
        }
      }
    }
  }
  // the waves' sums in wave order, 16 values of r at a time
  const long slot = (long)blockIdx.z * p.n + a;
#pragma unroll
  for (int c = 0; c < NR; ++c) {
#pragma unroll
    for (int b = 0; b < 8; ++b) red[wave][b][lane] = acc[c][b];
    __syncthreads();
    if (down) {
      // value (b, lane (col, g), i) is row r = r_begin + 16 c + col, column c0 + 32 g + 8 i + b
      const int r16 = tid >> 4, gg = (tid & 15) >> 2, i = tid & 3;
      const int r = r_begin + 16 * c + r16, h = c0 + 32 * gg + 8 * i;
      float v[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int ln = gg * 16 + r16;
        v[b] = ((red[0][b][ln][i] + red[1][b][ln][i]) + red[2][b][ln][i]) + red[3][b][ln][i];
      }
      if (r < R && h < D) {
        float* dst = p.d_down + (slot * R + r) * D + h;
        *reinterpret_cast<floatx4*>(dst) = floatx4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<floatx4*>(dst + 4) = floatx4{v[4], v[5], v[6], v[7]};
      }
    } else {
      // value (b, lane (col, g), i) is row c0 + 8 col + b, column r = r_begin + 16 c + 4 g + i
      const int row = tid >> 1, b = row & 7, cl = row >> 3;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int gg = 2 * (tid & 1) + k, ln = gg * 16 + cl;
        const floatx4 v = ((red[0][b][ln] + red[1][b][ln]) + red[2][b][ln]) + red[3][b][ln];
        const int r = r_begin + 16 * c + 4 * gg;
        if (r < R && c0 + row < D) *reinterpret_cast<floatx4*>(p.d_up + (slot * D + c0 + row) * R + r) = v;
      }
    }
    __syncthreads();
  }
}

// out[i] = sum over the segments, in order.
__global__ __launch_bounds__(256) void adapter_sum_kernel(const floatx4* __restrict__ part, int segments,
                                                          long n4, floatx4* __restrict__ out) {
  for (long i = blockIdx.x * 256L + threadIdx.x; i < n4; i += (long)gridDim.x * 256) {
    floatx4 v = part[i];
    for (int s = 1; s < segments; ++s) v += part[s * n4 + i];
    out[i] = v;
  }
}

// ---------------------------------------------------------------- launches
#define PMOE_BY_RANK(R, call)   \
  do {                          \
    if ((R) <= 16) {            \
      constexpr int NR = 1;     \
      call;                     \
    } else if ((R) <= 32) {     \
      constexpr int NR = 2;     \
      call;                     \
    } else if ((R) <= 64) {     \
      constexpr int NR = 4;     \
      call;                     \
    } else {                    \
      constexpr int NR = 8;     \
      call;                     \
    }                           \
  } while (0)

static int blocks_of(int T) { return (T + kTok - 1) / kTok; }

// Workgroups that share the groups of a block of tokens: as many as there can
// be groups while the launch stays within some thousand workgroups.
static int group_split(int T, int n, int others) {
  int most = T < kTok ? T : kTok;
  if (n + 1 < most) most = n + 1;
  const int room = 4096 / (blocks_of(T) * others);
  return room < 1 ? 1 : (room < most ? room : most);
}

// Columns of one expanding workgroup.
static int expand_chunk(int T, int D) {
  int chunk = 2048;
  while (chunk > 512 && (long)blocks_of(T) * ((D + chunk - 1) / chunk) < 512) chunk /= 2;
  return chunk;
}

static hipError_t reduce(bool trans, const void* in, const AdapterParams& p, int D, const void* W,
                         float* part, hipStream_t s) {
  const int parts = adapter_parts(D);
  const dim3 grid(blocks_of(p.T), parts, group_split(p.T, p.n, parts));
  const int span = adapter_span(D);
  const uint16_t* x = static_cast<const uint16_t*>(in);
  const uint16_t* w = static_cast<const uint16_t*>(W);
  if (trans)
    PMOE_BY_RANK(p.R, (adapter_reduce_kernel<NR, true><<<grid, 256, 0, s>>>(x, p.ids, p.ids64, p.T, p.n, D,
                                                                            p.R, w, span, part)));
  else
    PMOE_BY_RANK(p.R, (adapter_reduce_kernel<NR, false><<<grid, 256, 0, s>>>(x, p.ids, p.ids64, p.T, p.n, D,
                                                                             p.R, w, span, part)));
  return hipGetLastError();
}

static hipError_t expand(bool trans, const float* part, int parts, const AdapterParams& p, int D,
                         const void* W, const void* base, void* out, float* sums, int scale_sums,
                         hipStream_t s) {
  const int chunk = expand_chunk(p.T, D);
  const int chunks = out ? (D + chunk - 1) / chunk : 1;
  const dim3 grid(blocks_of(p.T), chunks, group_split(p.T, p.n, chunks));
  const uint16_t* w = static_cast<const uint16_t*>(W);
  const uint16_t* b = static_cast<const uint16_t*>(base);
  uint16_t* o = static_cast<uint16_t*>(out);
  if (trans)
    PMOE_BY_RANK(p.R, (adapter_expand_kernel<NR, true><<<grid, 256, 0, s>>>(
                          part, parts, p.ids, p.ids64, p.T, p.n, D, p.R, w, p.scale, b, o, sums, scale_sums, chunk)));
  else
    PMOE_BY_RANK(p.R, (adapter_expand_kernel<NR, false><<<grid, 256, 0, s>>>(
                          part, parts, p.ids, p.ids64, p.T, p.n, D, p.R, w, p.scale, b, o, sums, scale_sums, chunk)));
  return hipGetLastError();
}

// Segments of the tokens for the gradients of the matrices: more than the list
// in LDS allows, and enough workgroups when there are few adapters.
static int grad_segment(int T, int n, int H, int N) {
  const long per_segment = (long)n * ((H + kGradCols - 1) / kGradCols + (N + kGradCols - 1) / kGradCols);
  int seg = kSegMax;
  while (seg > 512 && per_segment * ((T + seg - 1) / seg) < 512) seg /= 2;
  return seg;
}

namespace {
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
}  // namespace

size_t adapter_forward_ws_bytes(int T, int H, int R) {
  return up256((size_t)adapter_parts(H) * T * R * 4);
}

size_t adapter_backward_ws_bytes(int T, int n, int H, int N, int R) {
  const int seg = grad_segment(T, n, H, N), segments = (T + seg - 1) / seg;
  size_t b = up256((size_t)adapter_parts(N) * T * R * 4) + up256((size_t)T * R * 4);
  if (segments > 1) b += up256((size_t)segments * n * R * H * 4) + up256((size_t)segments * n * R * N * 4);
  return b;
}

hipError_t launch_adapter_forward(const AdapterParams& p, hipStream_t s) {
  float* part = static_cast<float*>(p.ws);
  const hipError_t e = reduce(false, p.x, p, p.H, p.down, part, s);
  if (e != hipSuccess) return e;
  return expand(false, part, adapter_parts(p.H), p, p.N, p.up, p.base, p.out, p.v_out, 0, s);
}

hipError_t launch_adapter_backward(const AdapterParams& p, hipStream_t s) {
  char* at = static_cast<char*>(p.ws);
  float* part = reinterpret_cast<float*>(at);
  at += up256((size_t)adapter_parts(p.N) * p.T * p.R * 4);
  float* du = reinterpret_cast<float*>(at);
  at += up256((size_t)p.T * p.R * 4);
  if (p.T > 0) {
    hipError_t e = reduce(true, p.dy, p, p.N, p.up, part, s);
    if (e != hipSuccess) return e;
    e = expand(true, part, adapter_parts(p.N), p, p.H, p.down, p.base, p.out, du, 1, s);
    if (e != hipSuccess) return e;
  }
  if (!p.d_down) return hipSuccess;
  const int seg = grad_segment(p.T, p.n, p.H, p.N);
  const int segments = p.T > 0 ? (p.T + seg - 1) / seg : 1;
  const size_t na = (size_t)p.n * p.R * p.H, nb = (size_t)p.n * p.R * p.N;
  GradParams q;
  q.x = static_cast<const uint16_t*>(p.x);
  q.dy = static_cast<const uint16_t*>(p.dy);
  q.du = du;
  q.v = p.v_in;
  q.scale = p.scale;
  q.ids = p.ids;
  q.ids64 = p.ids64;
  q.T = p.T, q.n = p.n, q.H = p.H, q.N = p.N, q.R = p.R, q.seg = seg;
  q.d_down = segments > 1 ? reinterpret_cast<float*>(at) : p.d_down;
  q.d_up = segments > 1 ? reinterpret_cast<float*>(at + up256(segments * na * 4)) : p.d_up;
  const int chunks = (p.H + kGradCols - 1) / kGradCols + (p.N + kGradCols - 1) / kGradCols;
  const dim3 grid(chunks * (p.R > 64 ? 2 : 1), p.n, segments);
  PMOE_BY_RANK(p.R, (adapter_grad_kernel<(NR < 4 ? NR : 4)><<<grid, 256, 0, s>>>(q)));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || segments == 1) return e;
  const auto add = [&](const float* from, size_t count, float* to) {
    const long n4 = (long)(count / 4);
    const long blocks = (n4 + 255) / 256;
    adapter_sum_kernel<<<(int)(blocks < 4096 ? blocks : 4096), 256, 0, s>>>(
        reinterpret_cast<const floatx4*>(from), segments, n4, reinterpret_cast<floatx4*>(to));
    return hipGetLastError();
  };
  e = add(q.d_down, na, p.d_down);
  return e != hipSuccess ? e : add(q.d_up, nb, p.d_up);
}

}  // namespace pmoe
