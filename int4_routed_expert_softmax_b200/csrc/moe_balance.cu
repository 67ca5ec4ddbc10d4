// moe_balance.cu -- the router's balance loss over packed sequences: counts of
// kept pairs per expert, mean probabilities, loss, and the gradient of the
// logits (with the gradient of the kept softmax weights).
//
// Forward, per segment s with n counted tokens and p_t = softmax(logits_t):
//   counts_e = kept pairs on e,  P_e = sum_t p_t[e] / n,
//   loss = sum_e f_e P_e,        f_e = counts_e E / (k n).
// Backward (counts are constants of the loss):
//   dlogits_t[e] = dloss / n * p_e (f_e - sum_j f_j p_j)  +  kept part,
//   kept part: for slot i, w_i (dw_i - sum_j w_j dw_j) at e = idx[t][i]
//   (w = softmax over the kept logits).
//
// Both directions read each logit once and are bound by that traffic: a warp
// holds one row in registers (lane = a few experts), two shuffle trees give
// its maximum and its sum, and the next row's loads are in flight meanwhile.
// The backward recomputes p, which costs less than reading T * E saved values.
#include <cfloat>

#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kBalThreads = 512;
constexpr int kBalWarps = kBalThreads / 32;

// Expert of a lane's i-th value.  VEC = 4: 16-byte loads (E % 4 == 0 and a
// 16-byte aligned base); VEC = 1: any E.
template <int VEC>
__device__ __forceinline__ int expert_of(int i, int lane) {
  return VEC == 4 ? (i >> 2) * 128 + lane * 4 + (i & 3) : i * 32 + lane;
}

template <int NI, int VEC>
__device__ __forceinline__ void load_row(const float *row, int E, int lane, float (&v)[NI]) {
  if (VEC == 4) {
#pragma unroll
    for (int j = 0; j < NI / 4; ++j) {
      const int e = j * 128 + lane * 4;
      const float4 q = e < E ? __ldcs(reinterpret_cast<const float4 *>(row + e))
                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = i * 32 + lane;
      v[i] = e < E ? __ldcs(row + e) : -INFINITY;
    }
  }
}

// v -> softmax of the row (a row of -inf alone, which leaves no expert, gives
// 0 everywhere; NaN and +inf give NaN).
template <int NI>
__device__ __forceinline__ void softmax_row(float (&v)[NI]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < NI; ++i) m = fmaxf(m, v[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.0f;  // every term is then exp(-inf) = 0 (or NaN for a NaN)
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    v[i] = expf(v[i] - m);
    s += v[i];
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const float inv = s == 0.0f ? 0.0f : __fdiv_rn(1.0f, s);
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] *= inv;
}

// Segment bounds, clamped so that no offset, however wrong, leaves [0, T].  Up
// to kSegTab of them are copied to shared memory first: a search then waits for
// global memory once.
constexpr int kSegTab = 256;
struct Segments {
  const int32_t *seg;  // the table in shared memory, or the caller's, or null
  int S, T;
  __device__ __forceinline__ int at(int s) const {
    if (seg == nullptr) return s == 0 ? 0 : T;
    return min(max(seg[s], 0), T);
  }
  // First segment that ends behind t (S if none): the offsets do not decrease.
  __device__ __forceinline__ int of(int t) const {
    if (seg == nullptr) return 0;
    int lo = 0, hi = S;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid + 1) > t) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  }
};
// Synchronises the CTA.
__device__ __forceinline__ Segments load_segments(const BalanceArgs &a, int32_t *tab) {
  Segments sg{a.seg, a.S, a.T};
  if (a.seg != nullptr && a.S < kSegTab) {
    for (int i = threadIdx.x; i <= a.S; i += blockDim.x) tab[i] = a.seg[i];
    sg.seg = tab;
  }
  __syncthreads();
  return sg;
}

// pmean, counts, ntok and this thread's share of the loss for expert e.
__device__ __forceinline__ float finish_expert(const BalanceArgs &a, int s, int e, double p, int c, int n) {
  const float pm = n > 0 ? (float)(p / n) : 0.0f;
  a.counts[(size_t)s * a.E + e] = c;
  a.pmean[(size_t)s * a.E + e] = pm;
  return n > 0 ? (float)((double)c * a.E / ((double)a.k * n)) * pm : 0.0f;
}

// A CTA takes `chunk` consecutive tokens and leaves, for every segment that
// they touch, the sums of p, the counts and the counted tokens in slot
// blockIdx.x + s of the workspace: (CTA, segment) pairs follow each other with
// both indexes never falling, so their sum is a slot of its own.  A call of one
// CTA finishes the segments itself.  A warp takes U rows at a time (two of up to
// 256 experts; more do not fit its registers) while the next U, and what the
// counts need of them, are on their way: one row at a time ran at 3.4 TB/s.
template <int NI, int VEC>
__global__ void __launch_bounds__(kBalThreads) k_balance_fwd(const BalanceArgs a) {
  extern __shared__ float bsm[];
  constexpr int U = NI <= 8 ? 2 : 1;
  const int E = a.E;
  float *sp = bsm;                                     // [kBalWarps][E] sums of p per warp
  int *sc = reinterpret_cast<int *>(sp + kBalWarps * E);  // [E] counts
  __shared__ int32_t tab[kSegTab];
  __shared__ int sn[2];                                // counted tokens, two segments in turn
  __shared__ float sl[kBalWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool alone = gridDim.x == 1;
  pdl_launch_dependents();
  const int t0 = min((int)((int64_t)blockIdx.x * a.chunk), a.T), t1 = min(t0 + a.chunk, a.T);
  if (blockIdx.x == 0 && !alone)
    for (int s = tid; s < a.S; s += kBalThreads) a.ticket[s] = 0u;
  for (int e = tid; e < E; e += kBalThreads) sc[e] = 0;
  if (tid < 2) sn[tid] = 0;
  const Segments sg = load_segments(a, tab);
  const int s0 = alone ? 0 : sg.of(t0);
  int par = 0;
  for (int s = s0; s < a.S; ++s) {
    const int b0 = max(sg.at(s), t0), b1 = min(sg.at(s + 1), t1);
    if (!alone) {
      if (sg.at(s) >= t1) break;
      if (b0 >= b1) continue;  // empty, or none of its tokens here: its slot is never read
    }
    float acc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.0f;
    int n = 0;
    float nx[U][NI];
    int ne[U];   // this lane's expert of each row, -1: none
    bool nv[U];  // the row counts
    auto load = [&](int t) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tu = t + u * kBalWarps;
        nv[u] = tu < b1 && (a.valid == nullptr || a.valid[tu] != 0);
        ne[u] = tu < b1 && lane < a.k ? a.idx[(size_t)tu * a.k + lane] : -1;
        if (tu < b1) load_row<NI, VEC>(a.logits + (size_t)tu * E, E, lane, nx[u]);
      }
    };
    int t = b0 + warp;
    load(t);
    while (t < b1) {
      float v[U][NI];
      int e[U];
      bool ok[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        e[u] = ne[u];
        ok[u] = nv[u];
#pragma unroll
        for (int i = 0; i < NI; ++i) v[u][i] = nx[u][i];
      }
      t += U * kBalWarps;
      if (t < b1) load(t);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!ok[u]) continue;
        if (e[u] >= 0 && e[u] < E) atomicAdd(sc + e[u], 1);
        softmax_row<NI>(v[u]);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] += v[u][i];
        ++n;
      }
    }
    if (lane == 0 && n) atomicAdd(sn + par, n);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = expert_of<VEC>(i, lane);
      if (e < E) sp[warp * E + e] = acc[i];
    }
    __syncthreads();
    n = sn[par];
    float lsum = 0.0f;
    for (int e = tid; e < E; e += kBalThreads) {
      float p = 0.0f;
#pragma unroll
      for (int w = 0; w < kBalWarps; ++w) p += sp[w * E + e];
      if (alone) {
        lsum += finish_expert(a, s, e, p, sc[e], n);
      } else {
        const size_t at = (size_t)(blockIdx.x + s) * E + e;
        a.part_p[at] = p;
        a.part_c[at] = sc[e];
      }
      sc[e] = 0;
    }
    if (tid == 0) {
      sn[par ^ 1] = 0;
      if (alone) a.ntok[s] = n;
      else a.part_n[blockIdx.x + s] = n;
    }
    if (alone) {
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
      if (lane == 0) sl[warp] = lsum;
    }
    __syncthreads();
    if (alone && tid == 0) {
      float l = 0.0f;
      for (int w = 0; w < kBalWarps; ++w) l += sl[w];
      a.loss[s] = l;
    }
    par ^= 1;
  }
}

// Joins the CTAs' sums: block (x, s) takes 32 experts of segment s, lane =
// expert, the warps every 32nd slot, five of them at once; sums in 64 bits,
// always in the same order.  The last block of a segment adds the blocks'
// shares of the loss.
__global__ void __launch_bounds__(1024) k_balance_join(const BalanceArgs a) {
  __shared__ double rp[32][32];
  __shared__ int rc[32][32], rn[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  const Segments sg{a.seg, a.S, a.T};
  const int b0 = sg.at(s), b1 = sg.at(s + 1);
  pdl_wait();
  double p = 0.0;
  int c = 0, n = 0;
  if (b0 < b1) {
    const int c1 = (b1 - 1) / a.chunk;
    for (int q0 = b0 / a.chunk + warp; q0 <= c1; q0 += 5 * 32) {
      float pv[5];
      int cv[5], nv[5];
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        const int q = q0 + 32 * u;
        const size_t slot = (size_t)(q + s);
        const bool in = q <= c1;
        pv[u] = in && e < a.E ? a.part_p[slot * a.E + e] : 0.0f;
        cv[u] = in && e < a.E ? a.part_c[slot * a.E + e] : 0;
        nv[u] = in ? a.part_n[slot] : 0;
      }
#pragma unroll
      for (int u = 0; u < 5; ++u) {
        p += (double)pv[u];
        c += cv[u];
        n += nv[u];
      }
    }
  }
  rp[warp][lane] = p;
  rc[warp][lane] = c;
  if (lane == 0) rn[warp] = n;
  __syncthreads();
  if (warp != 0) return;
  p = 0.0, c = 0, n = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    p += rp[w][lane];
    c += rc[w][lane];
    n += rn[w];
  }
  float l = e < a.E ? finish_expert(a, s, e, p, c, n) : 0.0f;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  if (lane == 0) {
    if (blockIdx.x == 0) a.ntok[s] = n;
    a.part_l[(size_t)s * gridDim.x + blockIdx.x] = l;
    __threadfence();
    if (atomicAdd(a.ticket + s, 1u) == gridDim.x - 1) {
      __threadfence();
      float sum = 0.0f;
      for (unsigned i = 0; i < gridDim.x; ++i) sum += __ldcg(a.part_l + (size_t)s * gridDim.x + i);
      a.loss[s] = sum;
    }
  }
}

// Warps take runs of consecutive tokens, so that f of the segment stays in
// registers.  The kept part goes through a row of shared memory per warp that
// is zero between tokens.
template <int NI, int VEC>
__global__ void __launch_bounds__(256) k_balance_bwd(const BalanceArgs a) {
  extern __shared__ float bsm[];
  const int E = a.E;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ int32_t tab[kSegTab];
  float *kept = bsm + (size_t)warp * ((E + 3) & ~3);
  if (a.dw != nullptr)
    for (int e = lane; e < E; e += 32) kept[e] = 0.0f;
  const Segments sg = load_segments(a, tab);
  const int64_t w = (int64_t)blockIdx.x * 8 + warp;
  const int t0 = (int)min((int64_t)a.T, w * a.chunk), t1 = min(t0 + a.chunk, a.T);
  if (t0 >= t1) return;
  int s = -1, s_end = t0, s_begin = t0;  // the segment whose f is held; tokens s_begin .. s_end
  float f[NI], cs = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) f[i] = 0.0f;
  // the next row and its pairs are on their way while a row is worked on
  float nx[NI], nw = 0.0f, nd = 0.0f;
  int ne = -1;
  bool nv = true;
  auto load = [&](int t) {
    load_row<NI, VEC>(a.logits + (size_t)t * E, E, lane, nx);
    if (a.valid != nullptr) nv = a.valid[t] != 0;
    if (a.dw != nullptr && lane < a.k) {
      const size_t at = (size_t)t * a.k + lane;
      ne = a.idx[at];
      nw = a.w[at];
      nd = a.dw[at];
    }
  };
  load(t0);
  for (int t = t0; t < t1; ++t) {
    float v[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) v[i] = nx[i];
    const int e = ne;
    const float wi = nw, di = nd;
    const bool valid = nv;
    if (t + 1 < t1) load(t + 1);
    if (t >= s_end) {
      s = sg.of(t);
      s_begin = s < a.S ? sg.at(s) : a.T;
      s_end = s < a.S ? sg.at(s + 1) : a.T;
      const int n = s < a.S ? a.ntok[s] : 0;
      cs = n > 0 ? __fdiv_rn(a.dloss[s], (float)n) : 0.0f;
      const float fs = n > 0 ? (float)((double)E / ((double)a.k * n)) : 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int e = expert_of<VEC>(i, lane);
        f[i] = n > 0 && e < E ? (float)a.counts[(size_t)s * E + e] * fs : 0.0f;
      }
    }
    const bool counted = t >= s_begin && s < a.S && valid;
    if (counted) {
      softmax_row<NI>(v);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) dot = ffma(f[i], v[i], dot);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = cs * v[i] * (f[i] - dot);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) v[i] = 0.0f;
    }
    if (a.dw != nullptr) {
      float wd = wi * di;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) wd += __shfl_xor_sync(0xffffffffu, wd, off);
      const bool live = e >= 0 && e < E;
      const float g = wi * (di - wd);
      const unsigned same = __match_any_sync(0xffffffffu, live ? e : -1 - lane);
      if (__any_sync(0xffffffffu, same & (same - 1))) {
        // an expert listed twice: its terms one after the other, by slot
        for (int i = 0; i < a.k; ++i) {
          if (lane == i && live) kept[e] += g;
          __syncwarp();
        }
      } else if (live) {
        kept[e] = g;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int x = expert_of<VEC>(i, lane);
        if (x < E) v[i] += kept[x];
      }
      __syncwarp();
      if (live) kept[e] = 0.0f;
      __syncwarp();
    }
    float *row = a.dlogits + (size_t)t * E;
    if (VEC == 4) {
#pragma unroll
      for (int j = 0; j < NI / 4; ++j) {
        const int e = j * 128 + lane * 4;
        if (e < E)
          __stcs(reinterpret_cast<float4 *>(row + e), make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int e = i * 32 + lane;
        if (e < E) __stcs(row + e, v[i]);
      }
    }
  }
}

bool vec4(const BalanceArgs &a) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits);
  return a.E % 4 == 0 && (p & 15) == 0;
}

template <int NI, int VEC>
cudaError_t fwd(const BalanceArgs &a, int grid, cudaStream_t s) {
  const size_t smem = (size_t)(kBalWarps + 1) * a.E * 4;
  static int smem_set[64] = {0};
  cudaError_t err = ensure_smem(k_balance_fwd<NI, VEC>, smem, smem_set);
  if (err != cudaSuccess) return err;
  k_balance_fwd<NI, VEC><<<grid, kBalThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int NI, int VEC>
cudaError_t bwd(const BalanceArgs &a, int grid, cudaStream_t s) {
  const size_t smem = a.dw != nullptr ? (size_t)8 * ((a.E + 3) & ~3) * 4 : 0;
  k_balance_bwd<NI, VEC><<<grid, 256, smem, s>>>(a);
  return cudaGetLastError();
}

// Values per lane: the smallest instance that holds the row.
#define MOE_BALANCE_DISPATCH(fn)                                              \
  if (vec4(a)) {                                                             \
    if (a.E <= 128) return fn<4, 4>(a, grid, s);                             \
    if (a.E <= 256) return fn<8, 4>(a, grid, s);                             \
    if (a.E <= 512) return fn<16, 4>(a, grid, s);                            \
    return fn<32, 4>(a, grid, s);                                            \
  }                                                                          \
  if (a.E <= 128) return fn<4, 1>(a, grid, s);                               \
  if (a.E <= 256) return fn<8, 1>(a, grid, s);                               \
  if (a.E <= 512) return fn<16, 1>(a, grid, s);                              \
  return fn<32, 1>(a, grid, s);

cudaError_t dispatch_fwd(const BalanceArgs &a, int grid, cudaStream_t s) { MOE_BALANCE_DISPATCH(fwd) }
cudaError_t dispatch_bwd(const BalanceArgs &a, int grid, cudaStream_t s) { MOE_BALANCE_DISPATCH(bwd) }

}  // namespace

// Up to 64 tokens stay in one CTA (four rows a warp, one launch); beyond, up
// to two CTAs per SM of 32 tokens at least.
BalancePlan balance_plan(int T, int sms) {
  BalancePlan p;
  if (T <= 64) {
    p.grid = 1;
    p.chunk = T > 0 ? T : 1;
    return p;
  }
  const int most = kBalanceCtas * sms;
  p.chunk = (T + most - 1) / most;
  if (p.chunk < kBalanceChunkMin) p.chunk = kBalanceChunkMin;
  p.grid = (T + p.chunk - 1) / p.chunk;
  return p;
}

cudaError_t launch_balance_fwd(const BalanceArgs &a, int grid, cudaStream_t s) {
  cudaError_t err = dispatch_fwd(a, grid, s);
  if (err != cudaSuccess || grid == 1) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.E + 31) / 32), (unsigned)a.S);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_balance_join, a);
}

cudaError_t launch_balance_bwd(const BalanceArgs &a, int sms, cudaStream_t s) {
  // eight CTAs of eight warps fill an SM; a warp's run of tokens is what is left
  BalanceArgs b = a;
  const int64_t warps = (int64_t)sms * 64;
  b.chunk = (int)((a.T + warps - 1) / warps);
  if (b.chunk < 1) b.chunk = 1;
  const int nw = (a.T + b.chunk - 1) / b.chunk;
  return dispatch_bwd(b, (nw + 7) / 8, s);
}

}  // namespace moe
