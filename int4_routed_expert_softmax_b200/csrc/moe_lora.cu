// moe_lora.cu -- the int4 gs64 x Q8_0 projection with low-rank adapters of many
// requests beside it:
//
//   out_t = W^ x^_t + scale_a B_a u_t,   u_t = A_a x_t,   a = adapter[t].
//
// The base product is the layer's own definition: with exact integer block
// sums S_b(n, t) over 32 elements,
//   out(n, t) = sum over groups g of s(n, g) (S_2g d(t, 2g) + S_2g+1 d(t, 2g+1)).
// One mma.sync m16n8k32 with unsigned weight nibbles and signed codes gives
// sixteen by eight block sums at once, already in the registers that scale
// them.  The fifth-generation tensor cores would leave them in tensor memory:
// a block sum ends every 32 elements, so each would be read back through
// tcgen05.ld before its scaling, and the scaling sets the pace on either
// route.  The alternative without block sums, tcgen05 on fp16 hi / lo
// operands, costs three MMAs per product for the same 22 bits.  Rate of the
// integer mma.sync on this part: 1.12 POP/s (two per product).
//
// A nibble u is w + 8; the accumulator therefore starts at -8 times the sum
// of the block's codes (kept beside the block's scale), and at the bits of
// 1.5 * 2^23, which makes the sum a float for one subtraction.  The scaling
// runs in packed pairs of columns: per 64-group and pair two subtractions, a
// product and two fused multiply-adds.
//
// Small batches (at most kLoraSmallT tokens): two launches in token order.
//   k_lora_in    : Q8_0 of x, and partial sums of A x per slice of the inputs;
//   k_lora_proj  : 16 rows of W per CTA, its eight warps splitting the inputs;
//                  the weights are loaded into registers before the wait for
//                  k_lora_in, so that the two overlap.
// Larger ones: tokens sorted by adapter.
//   k_lora_sort  : counting sort of the tokens by adapter;
//   k_lora_quant : Q8_0 of x by sorted position;
//   k_lora_shrink: scale A x, 16 tokens of one adapter per CTA (tf32 hi + lo);
//   k_lora_gemm  : tiles of W rows by sorted tokens; the adapters of the
//                  tile's tokens are added in its epilogue by tf32 MMAs on the
//                  same accumulators.
#include "moe_lora.cuh"

namespace moe {
namespace {

// Scales and code sums of positions 2i and 2i + 1 for group g, at
// xs + (i * G + g) * 8: d of block 0, d of block 1, then the MMA's starting
// values of block 0 and block 1, each for the two positions.
__device__ __forceinline__ float *xs_at(float *xs, int64_t pos, int G, int g, int what) {
  return xs + ((pos >> 1) * G + g) * 8 + 2 * what + (pos & 1);
}

// Q8_0 of four elements (8 lanes share a 32-block): the codes packed, and for
// the block's first lane its scale and starting value.  The scale is the
// product with fp32's 1/127, as tensor libraries evaluate a division by a
// constant: at most a unit in the last place from amax / 127.
__device__ __forceinline__ uint32_t quant4(const float4 v, float &d, int &c) {
  float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  d = fmul(m, 1.0f / 127.0f);
  const int q0 = q8_code(v.x, d), q1 = q8_code(v.y, d), q2 = q8_code(v.z, d), q3 = q8_code(v.w, d);
  int s = q0 + q1 + q2 + q3;
#pragma unroll
  for (int off = 4; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  c = kMagicBits - 8 * s;
  return (uint32_t)(q0 & 255) | ((uint32_t)(q1 & 255) << 8) | ((uint32_t)(q2 & 255) << 16) | ((uint32_t)q3 << 24);
}

// ===========================================================================
// small batches
// ===========================================================================
template <bool BF16>
__global__ void __launch_bounds__(128) k_lora_in(const LoraArgs a) {
  __shared__ float xsm[kLoraSlice];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.y, k0 = blockIdx.x * kLoraSlice;
  const int G = a.K / 64, r = a.r;
  pdl_launch_dependents();
  const int k = k0 + 4 * tid;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (k < a.K) v = *reinterpret_cast<const float4 *>(a.x + (size_t)t * a.K + k);
  const int id = adapter_of(a, t);
  float d;
  int c;
  const uint32_t q = quant4(v, d, c);
  if (k < a.K) {
    *reinterpret_cast<uint32_t *>(a.xq + (size_t)t * a.K + k) = q;
    if ((tid & 7) == 0) {
      const int b = (k >> 5) & 1;
      *xs_at(a.xs, t, G, k >> 6, b) = d;
      *xs_at(a.xs, t, G, k >> 6, 2 + b) = __int_as_float(c);
    }
  }
  if (id == a.n) return;
  *reinterpret_cast<float4 *>(xsm + 4 * tid) = v;
  __syncthreads();
  // rows j = warp, warp + 4, ..: lane = 16 of the slice's inputs (8 + 8)
  const uint16_t *A = static_cast<const uint16_t *>(a.A) + (size_t)id * r * a.K + k0;
  float *dst = a.upart + ((size_t)blockIdx.x * a.T + t) * r;
  for (int j = warp; j < r; j += 4) {
    float s = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = h * 256 + lane * 8;
      if (k0 + i < a.K) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(A + (size_t)j * a.K + i));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 f = half2_values<BF16>(ww[m]);
          s = ffma(f.x, xsm[i + 2 * m], s);
          s = ffma(f.y, xsm[i + 2 * m + 1], s);
        }
      }
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) dst[j] = s;
  }
}

constexpr int kProjPre = 12;  // groups a warp holds in registers (12 * 8 warps * 64 = 6144 inputs)

// Accumulates one 64-group of a 16-row tile against eight columns.
// wl, wh: 8 packed bytes of rows g and g + 8; b0, b1: the columns' codes.
__device__ __forceinline__ void group_mma(f32x2 (&acc)[2], const uint2 wl, const uint2 wh, const uint2 b0,
                                          const uint2 b1, const float4 d, const float4 c, f32x2 s0, f32x2 s1) {
  constexpr uint32_t kLow = 0x0F0F0F0Fu;
  int p[4], q[4];
  mma_u8s8(p, wl.x & kLow, wh.x & kLow, wl.y & kLow, wh.y & kLow, b0.x, b0.y, __float_as_int(c.x),
           __float_as_int(c.y));
  mma_u8s8(q, (wl.x >> 4) & kLow, (wh.x >> 4) & kLow, (wl.y >> 4) & kLow, (wh.y >> 4) & kLow, b1.x, b1.y,
           __float_as_int(c.z), __float_as_int(c.w));
  const f32x2 m = pack2(-kMagic, -kMagic);
  const f32x2 d0 = pack2(d.x, d.y), d1 = pack2(d.z, d.w);
  const f32x2 tl = fma2(add2(pack2i(q[0], q[1]), m), d1, mul2(add2(pack2i(p[0], p[1]), m), d0));
  const f32x2 th = fma2(add2(pack2i(q[2], q[3]), m), d1, mul2(add2(pack2i(p[2], p[3]), m), d0));
  acc[0] = fma2(tl, s0, acc[0]);
  acc[1] = fma2(th, s1, acc[1]);
}

template <int NT, bool BF16>
__global__ void __launch_bounds__(256) k_lora_proj(const LoraArgs a) {
  extern __shared__ __align__(16) float psm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, q4 = lane & 3;
  const int G = a.K / 64, N = a.N, r = a.r, T = a.T;
  const int Gp = G + 2;
  float *red = psm;                                            // [8][16][NT * 8]
  float *us = red + 8 * 16 * NT * 8;                           // [NT * 8][r]
  __half *ssc = reinterpret_cast<__half *>(us + NT * 8 * r);   // [16][Gp]
  const int n0 = blockIdx.x * 16;
  const int rl = min(n0 + gq, N - 1), rh = min(n0 + gq + 8, N - 1);  // N may end inside the tile
  const unsigned char *Wl = a.W + (size_t)rl * (a.K / 2) + q4 * 8;
  const unsigned char *Wh = a.W + (size_t)rh * (a.K / 2) + q4 * 8;
  const __half *sc = reinterpret_cast<const __half *>(a.W + (size_t)N * (a.K / 2));
  uint2 wl[kProjPre], wh[kProjPre];
  auto load_w = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kProjPre; ++i) {
      const int g = warp + 8 * (i0 + i);
      if (g < G) {
        wl[i] = __ldg(reinterpret_cast<const uint2 *>(Wl + (size_t)g * 32));
        wh[i] = __ldg(reinterpret_cast<const uint2 *>(Wh + (size_t)g * 32));
      }
    }
  };
  load_w(0);
  for (int i = tid; i < 16 * G; i += 256) {
    const int row = i / G, g = i - row * G;
    ssc[row * Gp + g] = sc[(size_t)min(n0 + row, N - 1) * G + g];
  }
  pdl_wait();
  __syncthreads();
  f32x2 acc[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = 0ull;
  for (int i0 = 0; warp + 8 * i0 < G; i0 += kProjPre) {
    if (i0 > 0) load_w(i0);
#pragma unroll
    for (int i = 0; i < kProjPre; ++i) {
      const int g = warp + 8 * (i0 + i);
      if (g < G) {
        const float s0 = __half2float(ssc[gq * Gp + g]), s1 = __half2float(ssc[(gq + 8) * Gp + g]);
        const f32x2 p0 = pack2(s0, s0), p1 = pack2(s1, s1);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int8_t *cq = a.xq + (size_t)(j * 8 + gq) * a.K + (size_t)g * 64 + q4 * 8;
          const uint2 b0 = *reinterpret_cast<const uint2 *>(cq), b1 = *reinterpret_cast<const uint2 *>(cq + 32);
          const float4 *x4 = reinterpret_cast<const float4 *>(a.xs + ((size_t)(j * 4 + q4) * G + g) * 8);
          group_mma(acc[j], wl[i], wh[i], b0, b1, x4[0], x4[1], p0, p1);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float *o = red + (warp * 16 + gq) * (NT * 8) + j * 8 + 2 * q4;
    *reinterpret_cast<float2 *>(o) = unpack2(acc[j][0]);
    *reinterpret_cast<float2 *>(o + 8 * NT * 8) = unpack2(acc[j][1]);
  }
  // A x of the tokens, the slices in order
  const int slices = (a.K + kLoraSlice - 1) / kLoraSlice;
  for (int i = tid; i < T * r; i += 256) {
    const int t = i / r, id = adapter_of(a, t);
    float u = 0.0f;
    if (id < a.n)
      for (int s = 0; s < slices; ++s) u += a.upart[(size_t)s * T * r + i];
    if (blockIdx.x == 0 && a.u != nullptr) a.u[i] = u;
    us[i] = id < a.n ? a.scale[id] * u : 0.0f;
  }
  __syncthreads();
  for (int i = tid; i < 16 * T; i += 256) {
    const int row = i & 15, t = i >> 4;
    if (n0 + row >= N) continue;
    float o = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) o += red[(w * 16 + row) * (NT * 8) + t];
    const int id = adapter_of(a, t);
    if (id < a.n) {
      const uint4 *B = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.B) + ((size_t)id * N + n0 + row) * r);
      const float *ut = us + t * r;
      float l = 0.0f;
      for (int j = 0; j < r / 8; ++j) {
        const uint4 w = __ldg(B + j);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 f = half2_values<BF16>(ww[m]);
          l = ffma(f.x, ut[8 * j + 2 * m], l);
          l = ffma(f.y, ut[8 * j + 2 * m + 1], l);
        }
      }
      o += l;
    }
    a.out[(size_t)t * N + n0 + row] = o;
  }
}

// ===========================================================================
// sorted batches
// ===========================================================================
// One CTA.  off[a]: first sorted position of adapter a (a = n: the tokens
// without one), off[n + 1] = T; tile[a]: first kLoraSeg-token tile of adapter
// a, tile[n + 1] the number of tiles.  The sort is stable, so that every sum
// over an adapter's tokens has one order.  The placing pass runs in one warp,
// 32 tokens at a time.
__global__ void __launch_bounds__(1024) k_lora_sort(const LoraArgs a) {
  extern __shared__ int cnt[];  // [n + 1]
  __shared__ int wsum[2][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bins = a.n + 1;
  if (tid < 4 && a.status != nullptr) a.status[tid] = 0;
  for (int i = tid; i < bins; i += 1024) cnt[i] = 0;
  __syncthreads();
  for (int t = tid; t < a.T; t += 1024) atomicAdd(cnt + adapter_of(a, t), 1);
  __syncthreads();
  int base = 0, tbase = 0;
  for (int i0 = 0; i0 < bins; i0 += 1024) {
    const int i = i0 + tid;
    const int c = i < bins ? cnt[i] : 0, tc = (c + kLoraSeg - 1) / kLoraSeg;
    int x = c, y = tc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int vx = __shfl_up_sync(0xffffffffu, x, o), vy = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += vx, y += vy;
    }
    if (lane == 31) wsum[0][warp] = x, wsum[1][warp] = y;
    __syncthreads();
    int px = base, py = tbase, ax = 0, ay = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) px += wsum[0][w], py += wsum[1][w];
      ax += wsum[0][w], ay += wsum[1][w];
    }
    if (i < bins) {
      cnt[i] = px + x - c;
      a.off[i] = px + x - c;
      a.tile[i] = py + y - tc;
    }
    base += ax, tbase += ay;
    __syncthreads();
  }
  if (tid == 0) {
    a.off[bins] = a.T;
    a.tile[bins] = tbase;
  }
  if (warp != 0) return;
  int nx = lane < a.T ? adapter_of(a, lane) : -1;
  for (int t0 = 0; t0 < a.T; t0 += 32) {
    const int t = t0 + lane, id = nx;
    if (t + 32 < a.T) nx = adapter_of(a, t + 32);
    else nx = -1;
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (t < a.T) a.perm[cnt[id] + rank] = t;
    __syncwarp();
    if (t < a.T && rank == 0) cnt[id] += __popc(same);
    __syncwarp();
  }
}

// A warp takes 128 inputs of one position.
__global__ void __launch_bounds__(256) k_lora_quant(const LoraArgs a) {
  const int lane = threadIdx.x & 31;
  const int per = (a.K + 127) / 128, G = a.K / 64;
  const int64_t n = (int64_t)a.T * per;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < n; i += (int64_t)gridDim.x * 8) {
    const int pos = (int)(i / per), k = (int)(i - (int64_t)pos * per) * 128 + lane * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (k < a.K) v = *reinterpret_cast<const float4 *>(a.x + (size_t)a.perm[pos] * a.K + k);
    float d;
    int c;
    const uint32_t q = quant4(v, d, c);
    if (k < a.K) {
      *reinterpret_cast<uint32_t *>(a.xq + (size_t)pos * a.K + k) = q;
      if ((lane & 7) == 0) {
        const int b = (k >> 5) & 1;
        *xs_at(a.xs, pos, G, k >> 6, b) = d;
        *xs_at(a.xs, pos, G, k >> 6, 2 + b) = __int_as_float(c);
      }
    }
  }
}

// dst[p][j] = scale_a sum_k src[token][k] M_a(j, k): a CTA takes one tile of
// up to 16 tokens of one adapter, its eight warps splitting k in steps of 16;
// a lane's four consecutive k of a step serve two MMAs (their order inside a
// sum is free, as long as both operands agree).
template <int RT, bool BF16, bool TR>
__global__ void __launch_bounds__(256) k_lora_shrink(const LoraArgs a, const float *src, int L, const void *M,
                                                     float *dst, float *user) {
  extern __shared__ __align__(16) float red[];  // [8][16][RT * 8]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int r = a.r;
  const int id = adapter_at(a.tile, a.n, blockIdx.x);
  if ((int)blockIdx.x >= a.tile[a.n + 1]) return;
  const int p0 = a.off[id] + ((int)blockIdx.x - a.tile[id]) * kLoraSeg;
  const int np = min(kLoraSeg, a.off[id + 1] - p0);
  if (id == a.n) {
    if (user != nullptr)
      for (int i = tid; i < np * r; i += 256) user[(size_t)a.perm[p0 + i / r] * r + i % r] = 0.0f;
    return;
  }
  const uint16_t *Ma = static_cast<const uint16_t *>(M) + (size_t)id * r * L;
  const float *x0 = g < np ? src + (size_t)a.perm[p0 + g] * L : nullptr;
  const float *x1 = g + 8 < np ? src + (size_t)a.perm[p0 + g + 8] * L : nullptr;
  float acc[RT][4];
#pragma unroll
  for (int j = 0; j < RT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  const int steps = (L + 15) / 16;
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
  for (int st = warp; st < steps; st += 8) {
    const int k = st * 16 + 4 * q;
    const bool in = k < L;  // L is a multiple of 8: a lane's four are all in or out
    const float4 v0 = x0 != nullptr && in ? *reinterpret_cast<const float4 *>(x0 + k) : zero;
    const float4 v1 = x1 != nullptr && in ? *reinterpret_cast<const float4 *>(x1 + k) : zero;
    const float f0[4] = {v0.x, v0.y, v0.z, v0.w}, f1[4] = {v1.x, v1.y, v1.z, v1.w};
    uint32_t hi[2][4], lo[2][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const Tf32Pair s0 = split_tf32(f0[2 * m + h]), s1 = split_tf32(f1[2 * m + h]);
        hi[m][2 * h] = s0.hi, lo[m][2 * h] = s0.lo;
        hi[m][2 * h + 1] = s1.hi, lo[m][2 * h + 1] = s1.lo;
      }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if (j * 8 < r) {
        float b[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (in) {
          if (TR) {
#pragma unroll
            for (int m = 0; m < 4; ++m) b[m] = half_value<BF16>(__ldg(Ma + (size_t)(k + m) * r + j * 8 + g));
          } else {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(Ma + (size_t)(j * 8 + g) * L + k));
            const float2 e = half2_values<BF16>(w.x), f = half2_values<BF16>(w.y);
            b[0] = e.x, b[1] = e.y, b[2] = f.x, b[3] = f.y;
          }
        }
        float t[4];
        mma_tf32_zero(t, lo[0], __float_as_uint(b[0]), __float_as_uint(b[1]));
        mma_tf32(t, lo[1], __float_as_uint(b[2]), __float_as_uint(b[3]));
        mma_tf32(t, hi[0], __float_as_uint(b[0]), __float_as_uint(b[1]));
        mma_tf32(t, hi[1], __float_as_uint(b[2]), __float_as_uint(b[3]));
        add4(acc[j], t);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    float *o = red + (warp * 16 + g) * (RT * 8) + j * 8 + 2 * q;
    *reinterpret_cast<float2 *>(o) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2 *>(o + 8 * RT * 8) = make_float2(acc[j][2], acc[j][3]);
  }
  __syncthreads();
  const float sc = a.scale[id];
  for (int i = tid; i < np * r; i += 256) {
    const int p = i / r, j = i - p * r;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += red[(w * 16 + p) * (RT * 8) + j];
    dst[(size_t)(p0 + p) * r + j] = sc * s;
    if (user != nullptr) user[(size_t)a.perm[p0 + p] * r + j] = s;
  }
}

// Tiles of BM rows of W by BN sorted positions.  Stages of two 64-groups come
// through shared memory by cp.async; with KW = 2 one half of the warps takes
// the first group of a stage and the other half the second, joined at the end.
// Row strides of 96 (weights) and 160 (codes) bytes keep the fragments' 8-byte
// reads free of bank conflicts.
template <int WM_, int WN_, int KW_, int MT_, int NT_, int STG_>
struct GemmCfg {
  static constexpr int WM = WM_, WN = WN_, KW = KW_, MT = MT_, NT = NT_, STG = STG_;
  static constexpr int BM = WM * MT * 16, BN = WN * NT * 8, THREADS = WM * WN * KW * 32;
  static constexpr int WB = BM * 96, CB = BN * 160, XB = BN * 32, STAGE = WB + CB + XB;
  static size_t smem(int G) {
    const size_t main = (size_t)STG * STAGE + (size_t)BM * (G + 2) * 2;
    const size_t join = KW > 1 ? (size_t)(KW - 1) * BM * BN * 4 : 0;
    return main > join ? main : join;
  }
};

template <typename C, bool BF16>
__global__ void __launch_bounds__(C::THREADS) k_lora_gemm(const LoraArgs a) {
  extern __shared__ __align__(128) unsigned char gsm[];
  constexpr int BM = C::BM, BN = C::BN, MT = C::MT, NT = C::NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, q4 = lane & 3;
  const int G = a.K / 64, N = a.N, T = a.T, r = a.r, Gp = G + 2;
  const int wm = warp % C::WM, wn = warp / C::WM % C::WN, kw = warp / (C::WM * C::WN);
  const int n0 = blockIdx.x * BM, p0 = blockIdx.y * BN;
  __half *ssc = reinterpret_cast<__half *>(gsm + C::STG * C::STAGE);
  const int S = (G + 1) / 2;
  auto load_stage = [&](int st) {
    unsigned char *b = gsm + (st % C::STG) * C::STAGE;
    const int g0 = 2 * st, ng = min(2, G - g0);
    for (int i = tid; i < BM * 4; i += C::THREADS) {
      const int row = i >> 2, c = i & 3;
      if (c < 2 * ng)
        cp_async16(b + row * 96 + c * 16, a.W + (size_t)min(n0 + row, N - 1) * (a.K / 2) + (size_t)g0 * 32 + c * 16);
    }
    for (int i = tid; i < BN * 8; i += C::THREADS) {
      const int row = i >> 3, c = i & 7;
      if (c < 4 * ng)
        cp_async16(b + C::WB + row * 160 + c * 16, a.xq + (size_t)(p0 + row) * a.K + (size_t)g0 * 64 + c * 16);
    }
    for (int i = tid; i < BN * 2; i += C::THREADS) {
      const int pr = i >> 2, gg = (i >> 1) & 1, c = i & 1;
      if (gg < ng)
        cp_async16(b + C::WB + C::CB + gg * (BN * 16) + pr * 32 + c * 16,
                   a.xs + ((size_t)(p0 / 2 + pr) * G + g0 + gg) * 8 + c * 4);
    }
  };
  const __half *sc = reinterpret_cast<const __half *>(a.W + (size_t)N * (a.K / 2));
  for (int i = tid; i < BM * G; i += C::THREADS) {
    const int row = i / G, g = i - row * G;
    ssc[row * Gp + g] = sc[(size_t)min(n0 + row, N - 1) * G + g];
  }
#pragma unroll
  for (int st = 0; st < C::STG - 1; ++st) {
    if (st < S) load_stage(st);
    cp_async_commit();
  }
  f32x2 acc[MT][NT][2];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j][0] = acc[i][j][1] = 0ull;

  for (int st = 0; st < S; ++st) {
    cp_async_wait<C::STG - 2>();
    __syncthreads();
    if (st + C::STG - 1 < S) load_stage(st + C::STG - 1);
    cp_async_commit();
    const unsigned char *b = gsm + (st % C::STG) * C::STAGE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (C::KW == 2 && h != kw) continue;
      const int g = 2 * st + h;
      if (g >= G) break;
      uint2 wl[MT], wh[MT];
      f32x2 s0[MT], s1[MT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int row = (wm * MT + i) * 16 + gq;
        wl[i] = *reinterpret_cast<const uint2 *>(b + row * 96 + h * 32 + q4 * 8);
        wh[i] = *reinterpret_cast<const uint2 *>(b + (row + 8) * 96 + h * 32 + q4 * 8);
        const float e = __half2float(ssc[row * Gp + g]), f = __half2float(ssc[(row + 8) * Gp + g]);
        s0[i] = pack2(e, e);
        s1[i] = pack2(f, f);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int col = (wn * NT + j) * 8;
        const unsigned char *cb = b + C::WB + (col + gq) * 160 + h * 64 + q4 * 8;
        const uint2 b0 = *reinterpret_cast<const uint2 *>(cb), b1 = *reinterpret_cast<const uint2 *>(cb + 32);
        const float4 *x4 = reinterpret_cast<const float4 *>(b + C::WB + C::CB + h * (BN * 16) + (col / 2 + q4) * 32);
        const float4 d = x4[0], c = x4[1];
#pragma unroll
        for (int i = 0; i < MT; ++i) group_mma(acc[i][j], wl[i], wh[i], b0, b1, d, c, s0[i], s1[i]);
      }
    }
  }
  cp_async_wait<0>();
  if (C::KW == 2) {
    // the second half's sums go to the first through shared memory
    __syncthreads();
    f32x2 *join = reinterpret_cast<f32x2 *>(gsm) + (size_t)(warp % (C::WM * C::WN)) * (MT * NT * 2 * 32) + lane;
    if (kw == 1) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          join[((i * NT + j) * 2) * 32] = acc[i][j][0];
          join[((i * NT + j) * 2 + 1) * 32] = acc[i][j][1];
        }
    }
    __syncthreads();
    if (kw == 1) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        acc[i][j][0] = add2(acc[i][j][0], join[((i * NT + j) * 2) * 32]);
        acc[i][j][1] = add2(acc[i][j][1], join[((i * NT + j) * 2 + 1) * 32]);
      }
  }
  float o[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float2 x = unpack2(acc[i][j][0]), y = unpack2(acc[i][j][1]);
      o[i][j][0] = x.x, o[i][j][1] = x.y, o[i][j][2] = y.x, o[i][j][3] = y.y;
    }
  // the adapters of this warp's positions, one after the other
  const int pw = p0 + wn * NT * 8, pe = min(pw + NT * 8, T);
  const int nw = n0 + wm * MT * 16;
  if (pw < pe && pw < a.off[a.n]) {
    for (int id = adapter_at(a.off, a.n, pw); id < a.n && a.off[id] < pe; ++id) {
      const int b0 = max(a.off[id], pw), b1 = min(a.off[id + 1], pe);
      if (b0 >= b1) continue;
      const uint16_t *B = static_cast<const uint16_t *>(a.B) + (size_t)id * N * r;
      for (int k = 0; k < r; k += 8) {
        uint32_t af[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int row = nw + i * 16 + gq;
          const uint32_t w0 = __ldg(reinterpret_cast<const uint32_t *>(B + (size_t)min(row, N - 1) * r + k) + q4);
          const uint32_t w1 = __ldg(reinterpret_cast<const uint32_t *>(B + (size_t)min(row + 8, N - 1) * r + k) + q4);
          const float2 v0 = half2_values<BF16>(w0), v1 = half2_values<BF16>(w1);
          af[i][0] = __float_as_uint(v0.x), af[i][1] = __float_as_uint(v1.x);
          af[i][2] = __float_as_uint(v0.y), af[i][3] = __float_as_uint(v1.y);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int p = pw + j * 8 + gq;
          float2 u = make_float2(0.0f, 0.0f);
          if (p >= b0 && p < b1) u = *reinterpret_cast<const float2 *>(a.us + (size_t)p * r + k + 2 * q4);
          const Tf32Pair x = split_tf32(u.x), y = split_tf32(u.y);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            float t[4];
            mma_tf32_zero(t, af[i], x.lo, y.lo);
            mma_tf32(t, af[i], x.hi, y.hi);
            add4(o[i][j], t);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int p = pw + j * 8 + 2 * q4 + c;
      if (p < T) {
        float *row = a.out + (size_t)a.perm[p] * N;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          const int n = nw + i * 16 + gq;
          if (n < N) row[n] = o[i][j][c];
          if (n + 8 < N) row[n + 8] = o[i][j][2 + c];
        }
      }
    }
  }
}

template <int RT, bool BF16, bool TR>
cudaError_t shrink(const LoraArgs &a, const float *src, int L, const void *M, float *dst, float *user,
                   cudaStream_t s) {
  const size_t smem = (size_t)8 * 16 * RT * 8 * 4;
  static int smem_set[64] = {0};
  cudaError_t err = ensure_smem(k_lora_shrink<RT, BF16, TR>, smem, smem_set);
  if (err != cudaSuccess) return err;
  const int tiles = (a.T + kLoraSeg - 1) / kLoraSeg + a.n;  // at most: each adapter's last tile may be short
  k_lora_shrink<RT, BF16, TR><<<tiles, 256, smem, s>>>(a, src, L, M, dst, user);
  return cudaGetLastError();
}

template <bool BF16, bool TR>
cudaError_t shrink_rank(const LoraArgs &a, const float *src, int L, const void *M, float *dst, float *user,
                        cudaStream_t s) {
  if (a.r <= 16) return shrink<2, BF16, TR>(a, src, L, M, dst, user, s);
  if (a.r <= 32) return shrink<4, BF16, TR>(a, src, L, M, dst, user, s);
  if (a.r <= 64) return shrink<8, BF16, TR>(a, src, L, M, dst, user, s);
  return shrink<16, BF16, TR>(a, src, L, M, dst, user, s);
}

template <int NT, bool BF16>
cudaError_t proj(const LoraArgs &a, cudaStream_t s) {
  const size_t smem = (size_t)(8 * 16 * NT * 8 + NT * 8 * a.r) * 4 + (size_t)16 * (a.K / 64 + 2) * 2;
  static int smem_set[64] = {0};
  cudaError_t err = ensure_smem(k_lora_proj<NT, BF16>, smem, smem_set);
  if (err != cudaSuccess) return err;
  return launch_pdl(k_lora_proj<NT, BF16>, dim3((unsigned)((a.N + 15) / 16)), dim3(256), smem, s, a);
}

template <bool BF16>
cudaError_t small(const LoraArgs &a, cudaStream_t s) {
  k_lora_in<BF16><<<dim3((unsigned)((a.K + kLoraSlice - 1) / kLoraSlice), (unsigned)a.T), 128, 0, s>>>(a);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  if (a.T <= 8) return proj<1, BF16>(a, s);
  if (a.T <= 16) return proj<2, BF16>(a, s);
  return proj<4, BF16>(a, s);
}

template <typename C, bool BF16>
cudaError_t gemm(const LoraArgs &a, cudaStream_t s) {
  const size_t smem = C::smem(a.K / 64);
  static int smem_set[64] = {0};
  cudaError_t err = ensure_smem(k_lora_gemm<C, BF16>, smem, smem_set);
  if (err != cudaSuccess) return err;
  const dim3 grid((unsigned)((a.N + C::BM - 1) / C::BM), (unsigned)((a.T + C::BN - 1) / C::BN));
  k_lora_gemm<C, BF16><<<grid, C::THREADS, smem, s>>>(a);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t large(const LoraArgs &a, int sms, cudaStream_t s) {
  using Big = GemmCfg<2, 4, 1, 4, 4, 3>;    // 128 x 128
  using Small = GemmCfg<2, 2, 2, 2, 4, 3>;  // 64 x 64, two halves of K
  const int64_t tiles = (int64_t)((a.N + 127) / 128) * ((a.T + 127) / 128);
  return tiles >= sms ? gemm<Big, BF16>(a, s) : gemm<Small, BF16>(a, s);
}

}  // namespace

cudaError_t launch_lora_sort(const LoraArgs &a, cudaStream_t s) {
  k_lora_sort<<<1, 1024, (size_t)(a.n + 1) * 4, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_lora_shrink(const LoraArgs &a, const float *src, int L, const void *M, bool transposed, float *dst,
                               float *user, cudaStream_t s) {
  if (transposed)
    return a.bf16 ? shrink_rank<true, true>(a, src, L, M, dst, user, s)
                  : shrink_rank<false, true>(a, src, L, M, dst, user, s);
  return a.bf16 ? shrink_rank<true, false>(a, src, L, M, dst, user, s)
                : shrink_rank<false, false>(a, src, L, M, dst, user, s);
}

cudaError_t launch_lora_small(const LoraArgs &a, cudaStream_t s) {
  return a.bf16 ? small<true>(a, s) : small<false>(a, s);
}

cudaError_t launch_lora_large(const LoraArgs &a, int sms, cudaStream_t s) {
  cudaError_t err = launch_lora_sort(a, s);
  if (err != cudaSuccess) return err;
  const int64_t warps = (int64_t)a.T * ((a.K + 127) / 128);
  const int64_t most = (int64_t)sms * 8;
  const int64_t ctas = (warps + 7) / 8;
  k_lora_quant<<<(unsigned)(ctas < most ? ctas : most), 256, 0, s>>>(a);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  err = launch_lora_shrink(a, a.x, a.K, a.A, false, a.us, a.u, s);
  if (err != cudaSuccess) return err;
  return a.bf16 ? large<true>(a, sms, s) : large<false>(a, sms, s);
}

}  // namespace moe
