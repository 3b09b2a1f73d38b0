// Short causal depthwise convolution on gfx950: forward, backward and the
// single-token step.
//     p_t = bias + sum_j w_j x_{t-(W-1)+j},  y = p or p sigmoid(p)
// A few multiply-adds a value, so every pass is HBM-bound: each thread owns a
// vector of channels and walks a run of tokens with the last W - 1 rows in
// registers; the rows of the run are loaded together.  A run that crosses from one
// packed sequence into the next starts again from the next one's state.
#include <hip/hip_runtime.h>

#include "gdn_layer.h"
#include "gdn_layer_device.h"

namespace gdn {
namespace {

using namespace layer;

template <typename E>
constexpr int kVec = 16 / static_cast<int>(sizeof(E));
// Channels of a thread in the forward: eight-byte bf16 loads leave registers for more
// waves (runs of eight rows of 4 x 4096 x 2048 bf16, 134 MB: 29 us, 4.6 TB/s; 33 us
// with eight channels).  The rows two runs share cost 25 MB more reads; neighbouring runs
// on one XCD take most of that back but no time (29 us in groups of up to 32, 34 us with
// a contiguous eighth of the rows on each XCD).
constexpr int kWalkV = 4;

// One thread's channels: weights, bias, and the reading of input and state rows.
template <typename E, int W, int V>
struct Chan {
  float w[W][V], b[V];
  __device__ __forceinline__ void load(const ConvParams& p, int c0) {
    Raw<float, V * W> rw;
    Raw<float, V> rb;
    rw.load(p.weight + static_cast<int64_t>(c0) * W);
    rb.zero();
    if (p.bias) rb.load(p.bias + c0);
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = rw.get(e * W + j);
      b[e] = rb.get(e);
    }
  }
  // rows pos - (W-1) .. pos - 1 of the line (state, sequence) of sequence n at bos
  __device__ __forceinline__ void window(const ConvParams& p, int c0, int n, int64_t bos, int64_t pos,
                                         float (&win)[W - 1][V]) const {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t at = pos - (W - 1) + j;
      Raw<E, V> r;
      if (at >= 0)
        r.load(static_cast<const E*>(p.x) + (bos + at) * p.C + c0);
      else if (p.state0)
        r.load(static_cast<const E*>(p.state0) + (static_cast<int64_t>(n) * (W - 1) + at + W - 1) * p.C + c0);
      else
        r.zero();
#pragma unroll
      for (int e = 0; e < V; ++e) win[j][e] = r.get(e);
    }
  }
  __device__ __forceinline__ void pre(const float (&win)[W - 1][V], const float (&x)[V], float (&out)[V]) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = b[e];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][e], win[j][e], s);
      out[e] = fmaf(w[W - 1][e], x[e], s);
    }
  }
  static __device__ __forceinline__ void shift(float (&win)[W - 1][V], const float (&x)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
      win[W - 2][e] = x[e];
    }
  }
};

// Row r of the kept rows of sequence n (position len - (W-1) + r of its line).
template <typename E, int W>
__device__ __forceinline__ void final_row(const ConvParams& p, int64_t item) {
  constexpr int V = kVec<E>;
  const int nv = p.C / V;
  const int c0 = static_cast<int>(item % nv) * V;
  const int64_t nr = item / nv;
  const int r = static_cast<int>(nr % (W - 1)), n = static_cast<int>(nr / (W - 1));
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  const int64_t at = len - (W - 1) + r;
  Raw<E, V> v;
  if (at >= 0)
    v.load(static_cast<const E*>(p.x) + (bos + at) * p.C + c0);
  else if (p.state0)
    v.load(static_cast<const E*>(p.state0) + (static_cast<int64_t>(n) * (W - 1) + at + W - 1) * p.C + c0);
  else
    v.zero();
  *reinterpret_cast<u32x4_t*>(static_cast<E*>(p.state_final) + nr * p.C + c0) = v.w[0];
}

// Threads 0 .. runs * nv - 1 walk runs of RT rows; the ones behind them copy the
// kept rows.
template <typename E, int W, int RT>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvParams p, int64_t walkers, int64_t items) {
  constexpr int V = kWalkV;
  int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= walkers) {
    id -= walkers;
    if (id < items) final_row<E, W>(p, id);
    return;
  }
  const int nv = p.C / V;
  const int c0 = static_cast<int>(id % nv) * V;
  const int64_t t0 = id / nv * RT;
  const E* const x = static_cast<const E*>(p.x) + c0;
  Raw<E, V> raw[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) raw[i].load(x + min(t0 + i, p.rows - 1) * p.C);
  Chan<E, W, V> ch;
  ch.load(p, c0);
  int n = seq_of_row(p.seq, p.N, t0);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  float win[W - 1][V];
  ch.window(p, c0, n, bos, t0 - bos, win);
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t t = t0 + i;
    if (t >= p.rows) break;
    if (t == bos + len) {
      do chunk::seq_range(p.seq, ++n, bos, len);
      while (len == 0);
      ch.window(p, c0, n, bos, 0, win);
    }
    float xf[V], y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) xf[e] = raw[i].get(e);
    ch.pre(win, xf, y);
    if (p.silu) {
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] *= sigmoid_(y[e]);
    }
    store_vec<E, V>(static_cast<E*>(p.y) + t * p.C + c0, y);
    ch.shift(win, xf);
  }
}

template <typename E, int W>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvParams p, int64_t items) {
  constexpr int V = kVec<E>;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= items) return;
  const int nv = p.C / V;
  const int c0 = static_cast<int>(id % nv) * V;
  const int64_t n = id / nv;
  E* const state = static_cast<E*>(p.state_final) + n * (W - 1) * p.C + c0;
  Raw<E, V> rows[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].load(state + static_cast<int64_t>(j) * p.C);
  rows[W - 1].load(static_cast<const E*>(p.x) + n * p.C + c0);
  Chan<E, W, V> ch;
  ch.load(p, c0);
  float win[W - 1][V], xf[V], y[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j][e] = rows[j].get(e);
    xf[e] = rows[W - 1].get(e);
  }
  ch.pre(win, xf, y);
  if (p.silu) {
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] *= sigmoid_(y[e]);
  }
  store_vec<E, V>(static_cast<E*>(p.y) + n * p.C + c0, y);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) *reinterpret_cast<u32x4_t*>(state + static_cast<int64_t>(j) * p.C) = rows[j + 1].w[0];
}

// dp = dy d(p sigmoid(p))/dp
__device__ __forceinline__ float silu_grad(float p, float dy) {
  const float s = sigmoid_(p);
  return dy * s * fmaf(p, 1.f - s, 1.f);
}

// Backward.  dx_s = sum_k w_{W-1-k} dp_{s+k} over the tokens s + k of s's sequence
// (a row still open at token t is held in `open`), plus dstate_final on kept rows.
// A thread walks a run of 32 rows of four channels (and W - 1 rows of the next run for
// their dp alone), two rows at a time with the next two in flight; four channels
// rather than eight halve the registers of the weights and their gradients, for four
// waves a SIMD (4 x 4096 x 2048 bf16, 201 MB: 51 us, 3.9 TB/s; with eight channels and two
// waves 80 us, with four rows ahead and three waves 61 us).  At width 4 those waves leave 4
// (bf16) and 6 (fp32, three waves) registers too few, which the compiler keeps in scratch.  A
// thread has 32 rows however few there are: 512 x 512 bf16, eight workgroups, takes 26 us
// forward and backward.  A workgroup covers 512 rows
// of 64 channels: its sums of dp x and dp are reduced over the runs (lanes, then waves)
// and written once, and a second kernel adds the workgroups' sums in order.
constexpr int kBwdV = 4, kBwdRun = 32, kBwdLanes = 16, kBwdAhead = 2;
static_assert(256 / kBwdLanes * kBwdRun == kConvBwdRows, "rows of a workgroup");

template <typename E, int W>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 4 : 3) void conv_bwd_kernel(ConvParams p) {
  constexpr int V = kBwdV;
  const int tid = threadIdx.x, lane = tid % kBwdLanes, wave = tid >> 6;
  const int nv = p.C / V;
  const int vec = blockIdx.y * kBwdLanes + lane;
  const int c0 = min(vec, nv - 1) * V;
  const bool live = vec < nv;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kConvBwdRows + tid / kBwdLanes * kBwdRun;
  float dw[W][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    db[e] = 0.f;
  }
  if (live && t0 < p.rows) {
    const E* const x = static_cast<const E*>(p.x) + c0;
    const E* const dy = static_cast<const E*>(p.dy) + c0;
    E* const dx = static_cast<E*>(p.dx) + c0;
    const int64_t own_end = min(t0 + kBwdRun, p.rows), last = min(t0 + kBwdRun + W - 1, p.rows);
    Raw<E, V> rx[kBwdAhead], rd[kBwdAhead];
    auto fetch = [&](int64_t t) {
#pragma unroll
      for (int i = 0; i < kBwdAhead; ++i) {
        const int64_t at = min(t + i, last - 1) * p.C;
        rx[i].load(x + at);
        rd[i].load(dy + at);
      }
    };
    fetch(t0);
    Chan<E, W, V> ch;
    ch.load(p, c0);
    int n = seq_of_row(p.seq, p.N, t0);
    int64_t bos, len;
    chunk::seq_range(p.seq, n, bos, len);
    float win[W - 1][V], open[W - 1][V];  // open[k]: dx of row t - 1 - k so far
    ch.window(p, c0, n, bos, t0 - bos, win);
    auto reset = [&] {
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) open[k][e] = 0.f;
    };
    reset();
    // rows end - 1 - k of a sequence that ends before row `end`
    auto flush = [&](int64_t end) {
#pragma unroll
      for (int k = 0; k < W - 1; ++k) {
        const int64_t s = end - 1 - k;
        if (s < t0 || s >= own_end || s < bos) continue;
        if (p.dstate_final) {
          Raw<E, V> r;
          r.load(static_cast<const E*>(p.dstate_final) + (static_cast<int64_t>(n) * (W - 1) + W - 2 - k) * p.C + c0);
#pragma unroll
          for (int e = 0; e < V; ++e) open[k][e] += r.get(e);
        }
        store_vec<E, V>(dx + s * p.C, open[k]);
      }
    };
    bool done = false;
#pragma unroll 1
    for (int64_t tb = t0; tb < last && !done; tb += kBwdAhead) {
      Raw<E, V> cx[kBwdAhead], cd[kBwdAhead];
#pragma unroll
      for (int i = 0; i < kBwdAhead; ++i) {
        cx[i] = rx[i];
        cd[i] = rd[i];
      }
      if (tb + kBwdAhead < last) fetch(tb + kBwdAhead);
#pragma unroll
      for (int i = 0; i < kBwdAhead; ++i) {
        const int64_t t = tb + i;
        if (t >= last) break;
        if (t == bos + len) {
          flush(t);
          if (t >= own_end) {
            done = true;
            break;
          }
          do chunk::seq_range(p.seq, ++n, bos, len);
          while (len == 0);
          ch.window(p, c0, n, bos, 0, win);
          reset();
        }
        float xf[V], pre[V], dp[V], out[V];
#pragma unroll
        for (int e = 0; e < V; ++e) xf[e] = cx[i].get(e);
        ch.pre(win, xf, pre);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dp[e] = p.silu ? silu_grad(pre[e], cd[i].get(e)) : cd[i].get(e);
          out[e] = fmaf(ch.w[0][e], dp[e], open[W - 2][e]);
#pragma unroll
          for (int k = W - 2; k > 0; --k) open[k][e] = fmaf(ch.w[W - 1 - k][e], dp[e], open[k - 1][e]);
          open[0][e] = ch.w[W - 1][e] * dp[e];
        }
        const int64_t s = t - (W - 1);
        if (s >= t0 && s >= bos) store_vec<E, V>(dx + s * p.C, out);
        if (t < own_end) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(dp[e], win[j][e], dw[j][e]);
            dw[W - 1][e] = fmaf(dp[e], xf[e], dw[W - 1][e]);
            db[e] += dp[e];
          }
        }
        ch.shift(win, xf);
      }
    }
    if (!done && last == bos + len) flush(last);
  }
  __shared__ float red[4][kBwdLanes][(W + 1) * V];
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = j < W ? dw[j < W ? j : 0][e] : db[e];
#pragma unroll
      for (int m = kBwdLanes; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
      if ((tid & 63) < kBwdLanes) red[wave][lane][j * V + e] = s;
    }
  __syncthreads();
  for (int i = tid; i < kBwdLanes * (W + 1) * V; i += 256) {
    const int l = i / V % kBwdLanes, e = i % V, j = i / (V * kBwdLanes), je = j * V + e;
    const int c = (blockIdx.y * kBwdLanes + l) * V + e;
    if (c < p.C)
      p.ws[(static_cast<int64_t>(blockIdx.x) * (W + 1) + j) * p.C + c] =
          (red[0][l][je] + red[1][l][je]) + (red[2][l][je] + red[3][l][je]);
  }
}

// dstate0: row r of the state (position r - (W-1)) meets weight j at token r - j.
template <typename E, int W>
__device__ __forceinline__ void dstate0_rows(const ConvParams& p, int64_t item) {
  constexpr int V = kVec<E>;
  const int nv = p.C / V;
  const int c0 = static_cast<int>(item % nv) * V;
  const int n = static_cast<int>(item / nv);
  int64_t bos, len;
  chunk::seq_range(p.seq, n, bos, len);
  Chan<E, W, V> ch;
  ch.load(p, c0);
  float win[W - 1][V], g[W - 1][V];
  ch.window(p, c0, n, bos, 0, win);
#pragma unroll
  for (int r = 0; r < W - 1; ++r)
#pragma unroll
    for (int e = 0; e < V; ++e) g[r][e] = 0.f;
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    if (t >= len) break;
    Raw<E, V> rx, rd;
    rx.load(static_cast<const E*>(p.x) + (bos + t) * p.C + c0);
    rd.load(static_cast<const E*>(p.dy) + (bos + t) * p.C + c0);
    float xf[V], pre[V];
#pragma unroll
    for (int e = 0; e < V; ++e) xf[e] = rx.get(e);
    ch.pre(win, xf, pre);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float dp = p.silu ? silu_grad(pre[e], rd.get(e)) : rd.get(e);
#pragma unroll
      for (int j = 0; t + j < W - 1; ++j) g[t + j][e] = fmaf(ch.w[j][e], dp, g[t + j][e]);
    }
    ch.shift(win, xf);
  }
  // a sequence shorter than the state keeps the state's last rows
  if (p.dstate_final) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      if (r < len) continue;
      Raw<E, V> rd;
      rd.load(static_cast<const E*>(p.dstate_final) + (static_cast<int64_t>(n) * (W - 1) + r - len) * p.C + c0);
#pragma unroll
      for (int e = 0; e < V; ++e) g[r][e] += rd.get(e);
    }
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r)
    store_vec<E, V>(static_cast<E*>(p.dstate0) + (static_cast<int64_t>(n) * (W - 1) + r) * p.C + c0, g[r]);
}

// dweight and dbias from the workgroups' sums, eight of them in flight; the threads
// behind the first `sums` form dstate0.
template <typename E, int W>
__global__ __launch_bounds__(256) void conv_bwd_finish_kernel(ConvParams p, int64_t blocks, int64_t sums, int64_t items) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= sums) {
    if (i - sums < items) dstate0_rows<E, W>(p, i - sums);
    return;
  }
  const int64_t n = static_cast<int64_t>(W + 1) * p.C;
  if (i >= n) return;
  float part[8] = {};
  int64_t b = 0;
  for (; b + 8 <= blocks; b += 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) part[k] += p.ws[(b + k) * n + i];
  }
  for (; b < blocks; ++b) part[0] += p.ws[b * n + i];
  const float s = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
  const int j = static_cast<int>(i / p.C), c = static_cast<int>(i % p.C);
  if (j < W)
    p.dweight[static_cast<int64_t>(c) * W + j] = s;
  else if (p.dbias)
    p.dbias[c] = s;
}

unsigned blocks_of(int64_t threads) { return static_cast<unsigned>((threads + 255) / 256); }

template <typename E, int W, int RT>
hipError_t fwd_t(const ConvParams& p, hipStream_t s) {
  const int64_t walkers = (p.rows + RT - 1) / RT * (p.C / kWalkV);
  const int64_t items = p.state_final ? static_cast<int64_t>(p.N) * (W - 1) * (p.C / kVec<E>) : 0;
  if (walkers + items == 0) return hipSuccess;
  hipLaunchKernelGGL((conv_fwd_kernel<E, W, RT>), dim3(blocks_of(walkers + items)), dim3(256), 0, s, p, walkers, items);
  return hipGetLastError();
}

template <typename E, int W>
hipError_t fwd_w(const ConvParams& p, hipStream_t s) {
  // runs of eight rows read each row 1 + (W-1)/8 times, from the cache where two runs
  // meet; below one wave a SIMD that way, runs of two spread a short prompt over more
  // of the chip
  if (p.rows * (p.C / kWalkV) / 8 < 1024 * 64) return fwd_t<E, W, 2>(p, s);
  return fwd_t<E, W, 8>(p, s);
}

template <typename E, int W>
hipError_t bwd_w(const ConvParams& p, hipStream_t s) {
  const int64_t blocks = conv_bwd_blocks(p.rows);
  if (blocks > 0)
    hipLaunchKernelGGL((conv_bwd_kernel<E, W>),
                       dim3(static_cast<unsigned>(blocks), (p.C / kBwdV + kBwdLanes - 1) / kBwdLanes), dim3(256), 0, s, p);
  const int64_t sums = static_cast<int64_t>(blocks_of(static_cast<int64_t>(W + 1) * p.C)) * 256;
  const int64_t items = p.dstate0 ? static_cast<int64_t>(p.N) * (p.C / kVec<E>) : 0;
  hipLaunchKernelGGL((conv_bwd_finish_kernel<E, W>), dim3(blocks_of(sums + items)), dim3(256), 0, s, p, blocks, sums, items);
  return hipGetLastError();
}

template <typename E, int W>
hipError_t step_w(const ConvParams& p, hipStream_t s) {
  const int64_t items = static_cast<int64_t>(p.N) * (p.C / kVec<E>);
  hipLaunchKernelGGL((conv_step_kernel<E, W>), dim3(blocks_of(items)), dim3(256), 0, s, p, items);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_fwd(const ConvParams& p, int W, bool bf16, hipStream_t s) {
  switch (W) {
    case 2: return bf16 ? fwd_w<uint16_t, 2>(p, s) : fwd_w<float, 2>(p, s);
    case 3: return bf16 ? fwd_w<uint16_t, 3>(p, s) : fwd_w<float, 3>(p, s);
    default: return bf16 ? fwd_w<uint16_t, 4>(p, s) : fwd_w<float, 4>(p, s);
  }
}

hipError_t launch_conv_bwd(const ConvParams& p, int W, bool bf16, hipStream_t s) {
  switch (W) {
    case 2: return bf16 ? bwd_w<uint16_t, 2>(p, s) : bwd_w<float, 2>(p, s);
    case 3: return bf16 ? bwd_w<uint16_t, 3>(p, s) : bwd_w<float, 3>(p, s);
    default: return bf16 ? bwd_w<uint16_t, 4>(p, s) : bwd_w<float, 4>(p, s);
  }
}

hipError_t launch_conv_step(const ConvParams& p, int W, bool bf16, hipStream_t s) {
  switch (W) {
    case 2: return bf16 ? step_w<uint16_t, 2>(p, s) : step_w<float, 2>(p, s);
    case 3: return bf16 ? step_w<uint16_t, 3>(p, s) : step_w<float, 3>(p, s);
    default: return bf16 ? step_w<uint16_t, 4>(p, s) : step_w<float, 4>(p, s);
  }
}

}  // namespace gdn
