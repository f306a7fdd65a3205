// The two ends of the training form around the transformer's layers: RMSNorm with its gradient,
// and the embedding lookup with the gradient of its table.  Both move bytes: what bounds them is
// HBM, so every row is read once, held in registers and written once; for few rows it is the
// launches.
#include "ends.h"

#include <algorithm>

namespace smdm {

namespace {

SMDM_DEV void load4(const float* p, float* v) {
  const float4 u = *reinterpret_cast<const float4*>(p);
  v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
}
SMDM_DEV void load4(const __nv_bfloat16* p, float* v) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
SMDM_DEV uint32_t bf2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
SMDM_DEV void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
SMDM_DEV void store4(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(bf2(v[0], v[1]), bf2(v[2], v[3]));
}
template <int VEC, typename T>
SMDM_DEV void load_v(const T* p, float* v) {
  if constexpr (VEC == 4) load4(p, v);
  else v[0] = to_f<T>(*p);
}
template <int VEC, typename T>
SMDM_DEV void store_v(T* p, const float* v) {
  if constexpr (VEC == 4) store4(p, v);
  else *p = from_f<T>(v[0]);
}

// N elements as loaded, in as few instructions as their bytes allow (16 each),
// widened when they are used: a conversion next to its load would make the thread wait for each
// load before it issues the next.
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  SMDM_DEV void load(const T* p) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(p + k * 4 / (int)sizeof(T));
        w[k] = u.x; w[k + 1] = u.y; w[k + 2] = u.z; w[k + 3] = u.w;
      }
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x; w[1] = u.y;
    }
  }
  SMDM_DEV void get(float* v) const {
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
      if constexpr (sizeof(T) == 4) {
        v[k] = __uint_as_float(w[k]);
      } else {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T x;
  SMDM_DEV void load(const T* p) { x = *p; }
  SMDM_DEV void get(float* v) const { v[0] = to_f<T>(x); }
};

template <int N>
SMDM_DEV void store_n(float* p, const float* v) {
#pragma unroll
  for (int k = 0; k < N; k += 4) store4(p + k, v + k);
}
template <int N>
SMDM_DEV void store_n(__nv_bfloat16* p, const float* v) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(bf2(v[0], v[1]), bf2(v[2], v[3]), bf2(v[4], v[5]),
                                              bf2(v[6], v[7]));
  else
    store4(p, v);
}

int device_sms() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Sum over the TPR threads of a row (a warp, or the whole CTA).
template <int TPR>
SMDM_DEV float row_sum(float s, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();                  // the previous row's sums have been read
    if ((threadIdx.x & 31) == 0) red[warp] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) s += red[i];
  }
  return s;
}

constexpr int kNormThreads = 256;

// y = x r gain, r = (mean x^2 + eps)^-1/2.  TPR threads per row, NU units of VEC elements each: a
// warp up to 1024 elements (no barrier in the row's sum), a CTA above.  66 rows of 4096: 2.5 us,
// a launch's time; 12544 rows (fp32 to bf16) of 4096: 48 us, 6.4 TB/s, of 1024: 17.6 us, 4.4 TB/s.
template <typename X, typename T, int TPR, int VEC, int NU>
__global__ void __launch_bounds__(kNormThreads) train_rms_kernel(RmsArgs a) {
  griddep_launch();
  griddep_wait();
  __shared__ float red[32];
  constexpr int RPC = kNormThreads / TPR;
  const int tid = threadIdx.x % TPR;
  const int row = blockIdx.x * RPC + threadIdx.x / TPR;
  if (RPC > 1 && row >= a.rows) return;
  const int units = a.d / VEC;
  const X* x = static_cast<const X*>(a.x) + (size_t)row * a.ld_x;
  Raw<X, VEC> rx[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u)
    if (tid + u * TPR < units) rx[u].load(x + (size_t)(tid + u * TPR) * VEC);
  float v[NU * VEC];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    if (tid + u * TPR < units) {
      rx[u].get(v + u * VEC);
#pragma unroll
      for (int k = 0; k < VEC; ++k) ss += v[u * VEC + k] * v[u * VEC + k];
    }
  }
  ss = row_sum<TPR>(ss, red);
  const float r = 1.f / sqrtf(ss / (float)a.d + a.eps);
  if (a.rstd_out && tid == 0) a.rstd_out[row] = r;
  T* y = static_cast<T*>(a.y) + (size_t)row * a.ld_y;
  const T* gain = static_cast<const T*>(a.gain);
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int i = tid + u * TPR;
    if (i < units) {
      float g[VEC];
      load_v<VEC>(gain + (size_t)i * VEC, g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) g[k] *= v[u * VEC + k] * r;
      store_v<VEC>(y + (size_t)i * VEC, g);
    }
  }
}

// u = gy gain;  gx = r (u - x r^2 mean(u x)) + add;  ggain = sum over rows of gy x r.
// Persistent CTAs: the gain and this CTA's share of its gradient stay in registers over all the
// CTA's rows; the shares go to ws[CTA][d] and are added up in order by rms_gain_kernel.  12544 rows of
// 1024 (fp32 x and add, bf16 grad_y): 37.6 us, 4.8 TB/s.
template <typename X, typename T, int TPR, int VEC, int NU>
__global__ void __launch_bounds__(kNormThreads) train_rms_grad_kernel(RmsArgs a) {
  griddep_launch();
  griddep_wait();
  __shared__ float red[32];
  constexpr int RPC = kNormThreads / TPR;
  const int tid = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int units = a.d / VEC;
  float gain[NU * VEC], acc[NU * VEC];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int i = tid + u * TPR;
#pragma unroll
    for (int k = 0; k < VEC; ++k) gain[u * VEC + k] = acc[u * VEC + k] = 0.f;
    if (i < units) load_v<VEC>(static_cast<const T*>(a.gain) + (size_t)i * VEC, gain + u * VEC);
  }
  for (int row = blockIdx.x * RPC + sub; row < a.rows; row += gridDim.x * RPC) {
    const X* x = static_cast<const X*>(a.x) + (size_t)row * a.ld_x;
    const T* gy = static_cast<const T*>(a.grad_y) + (size_t)row * a.ld_y;
    const X* ad = a.add ? static_cast<const X*>(a.add) + (size_t)row * a.d : nullptr;
    const float r = a.rstd[row];
    Raw<X, VEC> rx[NU], ra[NU];
    Raw<T, VEC> rg[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + u * TPR;
      if (i < units) {
        rx[u].load(x + (size_t)i * VEC);
        rg[u].load(gy + (size_t)i * VEC);
        if (ad) ra[u].load(ad + (size_t)i * VEC);
      }
    }
    float v[NU * VEC], g[NU * VEC];
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if (tid + u * TPR < units) {
        rx[u].get(v + u * VEC);
        rg[u].get(g + u * VEC);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const int e = u * VEC + k;
          acc[e] += g[e] * (v[e] * r);
          g[e] *= gain[e];
          dot += g[e] * v[e];
        }
      }
    }
    dot = row_sum<TPR>(dot, red);
    const float c = dot / (float)a.d * r * r;
    X* gx = static_cast<X*>(a.grad_x) + (size_t)row * a.d;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + u * TPR;
      if (i < units) {
        float o[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] = r * (g[u * VEC + k] - v[u * VEC + k] * c);
        if (ad) {
          float w[VEC];
          ra[u].get(w);
#pragma unroll
          for (int k = 0; k < VEC; ++k) o[k] += w[k];
        }
        store_v<VEC>(gx + (size_t)i * VEC, o);
      }
    }
  }
  // (a single CTA's share is the gradient)
  float* ws = a.ws + (size_t)blockIdx.x * a.d;
  T* gg = static_cast<T*>(a.grad_gain);
  if constexpr (RPC == 1) {
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + u * TPR;
      if (i >= units) continue;
      if (gridDim.x == 1) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) gg[i * VEC + k] = from_f<T>(acc[u * VEC + k]);
      } else {
        store_v<VEC>(ws + (size_t)i * VEC, acc + u * VEC);
      }
    }
  } else {
    // the warps' shares side by side in shared memory, added in order
    extern __shared__ float sh[];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + u * TPR;
      if (i < units) store_v<VEC>(sh + (size_t)sub * a.d + (size_t)i * VEC, acc + u * VEC);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.d; i += kNormThreads) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < RPC; ++w) t += sh[(size_t)w * a.d + i];
      if (gridDim.x == 1) gg[i] = from_f<T>(t);
      else ws[i] = t;
    }
  }
}

// The gradient for wide rows on 16-byte boundaries: the same sums, with the rows' loads taken off
// the threads.  Bulk copies bring x, grad_y and add of the CTA's next rows into a ring of shared
// memory stages while the threads work on the current one, so that HBM stays busy through the
// row's reduction and its stores.  One row per turn and CTA of TH threads.  12544 rows of 4096
// (fp32 x and add, bf16 grad_y): 111 us, 6.5 TB/s, with the kernel that adds up the gain's
// gradient; with the rows loaded by the threads, next to the reduction that waits for them, 236.
struct RmsRing {
  int stages, stage_bytes, gy_off, add_off;   // offsets within a stage
};

template <typename X, typename T, int TH>
__global__ void __launch_bounds__(TH, 512 / TH) train_rms_grad_ring_kernel(RmsArgs a, RmsRing q) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[32];
  __shared__ __align__(8) uint64_t full[8];
  __shared__ int s_abort;
  constexpr int NU = 4;
  const int tid = threadIdx.x;
  const int units = a.d >> 2;
  if (tid == 0) {
    for (int i = 0; i < q.stages; ++i) mbar_init(&full[i], 1);
    s_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch();
  griddep_wait();
  volatile int* abort_flag = &s_abort;
  const uint32_t xb = a.d * sizeof(X), gb = a.d * sizeof(T);
  auto fetch = [&](int row, int st) {
    uint8_t* p = ring + (size_t)st * q.stage_bytes;
    mbar_arrive_expect_tx(&full[st], xb + gb + (a.add ? xb : 0u));
    bulk_load(p, static_cast<const X*>(a.x) + (size_t)row * a.ld_x, xb, &full[st]);
    bulk_load(p + q.gy_off, static_cast<const T*>(a.grad_y) + (size_t)row * a.ld_y, gb, &full[st]);
    if (a.add)
      bulk_load(p + q.add_off, static_cast<const X*>(a.add) + (size_t)row * a.d, xb, &full[st]);
  };
  if (tid == 0)
    for (int i = 0; i < q.stages; ++i) {
      const long long row = blockIdx.x + (long long)i * gridDim.x;
      if (row < a.rows) fetch((int)row, i);
    }
  float gain[NU * 4], acc[NU * 4];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int i = tid + u * TH;
#pragma unroll
    for (int k = 0; k < 4; ++k) gain[u * 4 + k] = acc[u * 4 + k] = 0.f;
    if (i < units) load4(static_cast<const T*>(a.gain) + (size_t)i * 4, gain + u * 4);
  }
  int st = 0, turn = 0;
  uint32_t phase = 0;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
    float r = a.rstd[row];
    // (rows that did not arrive give NaN, not what the stage held before)
    if (!mbar_wait(&full[st], phase, abort_flag, nullptr)) r = __int_as_float(0x7fffffff);
    const uint8_t* p = ring + (size_t)st * q.stage_bytes;
    const X* x = reinterpret_cast<const X*>(p);
    const T* gy = reinterpret_cast<const T*>(p + q.gy_off);
    const X* ad = reinterpret_cast<const X*>(p + q.add_off);
    float v[NU * 4], g[NU * 4], w[NU * 4];
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + u * TH;
      if (i < units) {
        load4(x + i * 4, v + u * 4);
        load4(gy + i * 4, g + u * 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[u * 4 + k] = 0.f;
        if (a.add) load4(ad + i * 4, w + u * 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = u * 4 + k;
          acc[e] += g[e] * (v[e] * r);
          g[e] *= gain[e];
          dot += g[e] * v[e];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    // two sets of partial sums in turn: the next row's do not overwrite the ones being read
    float* rd = red + (turn & 1) * 16;
    if ((tid & 31) == 0) rd[tid >> 5] = dot;
    __syncthreads();                        // the stage has been read, too
    const long long next = row + (long long)q.stages * gridDim.x;
    // (after a wait that gave up the stage's copies may still be on their way, and its barrier still
    // waits for them: nothing more is fetched, and the waits for it give up at once)
    if (tid == 0 && next < a.rows && !*abort_flag) fetch((int)next, st);
    dot = 0.f;
#pragma unroll
    for (int i = 0; i < TH / 32; ++i) dot += rd[i];
    const float c = dot / (float)a.d * r * r;
    X* gx = static_cast<X*>(a.grad_x) + (size_t)row * a.d;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int i = tid + u * TH;
      if (i < units) {
        float o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = r * (g[u * 4 + k] - v[u * 4 + k] * c) + w[u * 4 + k];
        store4(gx + (size_t)i * 4, o);
      }
    }
    if (++st == q.stages) { st = 0; phase ^= 1; }
  }
  if (*abort_flag) let_land();
  float* ws = a.ws + (size_t)blockIdx.x * a.d;
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const int i = tid + u * TH;
    if (i >= units) continue;
    if (gridDim.x == 1) store4(static_cast<T*>(a.grad_gain) + (size_t)i * 4, acc + u * 4);
    else store4(ws + (size_t)i * 4, acc + u * 4);
  }
}

// Columns of ws[parts][d] added up: 32 columns and 32 part groups per CTA.
template <typename T>
__global__ void __launch_bounds__(1024) rms_gain_kernel(const float* ws, int parts, int d, T* out) {
  griddep_launch();
  griddep_wait();
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int p = g; p < parts; p += 32) s += ws[(size_t)p * d + c];
  sh[g][lane] = s;
  __syncthreads();
  // warp g adds up column g
  s = sh[lane][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + g < d) out[blockIdx.x * 32 + g] = from_f<T>(s);
}

// ------------------------------------------------------------------------------------------
// Embedding
// ------------------------------------------------------------------------------------------
// One warp per row.  A lane takes as many elements as fill 16 bytes of the wider of the two types,
// so that every store instruction of a warp writes whole 32-byte sectors in a row.  A negative id
// gives a row of zeros.  12544 rows of 4096, bf16 to fp32: 41 us, 5.7 TB/s of rows written
// and of the about 3340 different ones read; 65 with each lane's 32 bytes written in two halves, 48
// with loads between the stores.
template <typename T, typename O, bool VECT>
__global__ void __launch_bounds__(256) embed_kernel(EmbedArgs a) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  const int id = a.ids[row];
  const bool on = id >= 0 && id < a.n_emb;
  if (id >= a.n_emb && a.status && lane == 0) atomicOr(a.status, kStatusBounds);
  const T* t = static_cast<const T*>(a.table) + (size_t)(on ? id : 0) * a.ld_table;
  O* o = static_cast<O*>(a.out) + (size_t)row * a.d;
  if constexpr (VECT) {
    constexpr int N = sizeof(T) == 4 || sizeof(O) == 4 ? 4 : 8;
    constexpr int B = 8;               // loads in flight; stores follow them
    for (int c0 = lane * N; c0 < a.d; c0 += B * 32 * N) {
      Raw<T, N> raw[B];
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (c0 + b * 32 * N < a.d) raw[b].load(t + c0 + b * 32 * N);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int c = c0 + b * 32 * N;
        if (c < a.d) {
          float v[N];
          raw[b].get(v);
#pragma unroll
          for (int k = 0; k < N; ++k) v[k] = on ? v[k] * a.scale : 0.f;
          store_n<N>(o + c, v);
        }
      }
    }
  } else {
    for (int c = lane; c < a.d; c += 32) o[c] = from_f<O>(on ? to_f<T>(t[c]) * a.scale : 0.f);
  }
}

// Sorting (id, row) pairs as 64-bit words: all different, so any sorting method is a stable one
// and the sums below always add a token's rows in the same order.
constexpr int kChunk = kSortChunk;

// Each of the first `chunks` CTAs sorts one chunk of `size` words (a power of two, up to kChunk): a
// bitonic network, two words per thread.  Exchanges over distances below 64 stay within a warp
// (shuffles; the last one within a thread), 51 of the 66 steps of 2048 words; only the other 15
// go through shared memory.  Thread t holds words 2t and 2t + 1.
// The other CTAs clear the table's gradient meanwhile.  The sort keeps few SMs busy, so the rows
// of tokens that do occur cost nothing visible although they are written again (looking every
// row up in the sorted list instead, in the next kernel: 24.2 us instead of 17.1 for 512 rows
// and a table of 32066).
// W: 32-bit words (id, place in the chunk) where the ids leave room for the place's 11 bits.
template <typename W>
__global__ void __launch_bounds__(1024) embed_sort_kernel(const int* ids, int n, int n_emb, int size,
                                                          int chunks, unsigned long long* out,
                                                          uint8_t* table, size_t table_bytes,
                                                          uint32_t* status) {
  griddep_launch();
  griddep_wait();
  if ((int)blockIdx.x >= chunks) {
    // bytes before the first 16-byte boundary, whole 16-byte words, bytes behind the last
    const size_t head = min(table_bytes, (size_t)(-reinterpret_cast<uintptr_t>(table) & 15));
    const size_t words = (table_bytes - head) / 16;
    uint4* w = reinterpret_cast<uint4*>(table + head);
    const size_t step = (size_t)(gridDim.x - chunks) * blockDim.x;
    const size_t at = (size_t)(blockIdx.x - chunks) * blockDim.x + threadIdx.x;
    for (size_t i = at; i < words; i += step) w[i] = make_uint4(0, 0, 0, 0);
    if (at < head) table[at] = 0;
    if (at < table_bytes - head - words * 16) table[head + words * 16 + at] = 0;
    return;
  }
  __shared__ __align__(16) W s[kChunk];
  constexpr bool k32 = sizeof(W) == 4;
  const int base = blockIdx.x * size, t = threadIdx.x;
  auto word = [&](int i) {
    const int r = base + i;
    unsigned key = k32 ? (1u << 21) - 1 : 0xffffffffu;   // behind every id
    if (r < n) {
      const int id = ids[r];
      if (id >= 0 && id < n_emb) key = (unsigned)id;
      else {
        key = (unsigned)n_emb;             // takes no part
        if (id >= n_emb && status) atomicOr(status, kStatusBounds);
      }
    }
    return k32 ? (W)((key << 11) | (unsigned)i) : (W)(((unsigned long long)key << 32) | (unsigned)r);
  };
  auto order = [](W& x, W& y, bool up) {
    if ((x > y) == up) {
      const W z = x;
      x = y;
      y = z;
    }
  };
  W x = word(2 * t), y = word(2 * t + 1);
  for (int k = 2; k <= size; k <<= 1) {
    const bool up = ((2 * t) & k) == 0;
    if (k >= 128) {
      // distances 64 and more: word pairs of the whole chunk in shared memory
      s[2 * t] = x;
      s[2 * t + 1] = y;
      __syncthreads();
      for (int j = k >> 1; j >= 64; j >>= 1) {
        const int i = ((t & ~(j - 1)) << 1) | (t & (j - 1)), l = i | j;
        W p = s[i], q = s[l];
        order(p, q, (i & k) == 0);
        s[i] = p;
        s[l] = q;
        __syncthreads();
      }
      x = s[2 * t];
      y = s[2 * t + 1];
      __syncthreads();
    }
    for (int j = min(k >> 1, 32); j >= 2; j >>= 1) {
      // partner thread t ^ (j / 2): the lower one keeps the smaller word of an ascending pair
      const bool keep_min = ((t & (j >> 1)) == 0) == up;
      const W px = __shfl_xor_sync(0xffffffffu, x, j >> 1);
      const W py = __shfl_xor_sync(0xffffffffu, y, j >> 1);
      x = (px < x) == keep_min ? px : x;
      y = (py < y) == keep_min ? py : y;
    }
    order(x, y, up);
  }
  auto wide = [&](W w) {
    return k32 ? ((unsigned long long)(w >> 11) << 32) | (unsigned)(base + (int)(w & (kChunk - 1)))
               : (unsigned long long)w;
  };
  if (base + 2 * t < n) out[base + 2 * t] = wide(x);
  if (base + 2 * t + 1 < n) out[base + 2 * t + 1] = wide(y);
}

// Merge groups of `ways` (a power of two, at most 32) sorted runs of `run` words: a word's place is its place in its own run
// plus the number of smaller words in each of the others, found by one lane per run.
__global__ void __launch_bounds__(256) embed_merge_kernel(const unsigned long long* in, int n,
                                                          int run, int ways,
                                                          unsigned long long* out) {
  griddep_launch();
  griddep_wait();
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  const int way = (int)(t & (ways - 1));
  const long long i = t / ways;
  const bool in_range = i < n;
  const unsigned long long x = in_range ? in[i] : 0;
  const long long group = i / ((long long)run * ways) * run * ways;
  const long long lo0 = group + (long long)way * run;
  int rank = 0;
  if (in_range && lo0 < n) {
    if (i >= lo0 && i < lo0 + run) {
      rank = (int)(i - lo0);
    } else {
      const unsigned long long* b = in + lo0;
      int lo = 0, hi = (int)min((long long)run, n - lo0);
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (b[mid] < x) lo = mid + 1;
        else hi = mid;
      }
      rank = lo;
    }
  }
  for (int o = ways / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (in_range && way == 0) out[group + rank] = x;
}

struct EmbedGradArgs {
  EmbedArgs e;
  const unsigned long long* list;   // sorted (id, row); id n_emb: takes no part
  float* part;                      // [pieces][2][d]
  int per, pieces, slabs;           // list entries per piece; 256-column slabs
};

SMDM_DEV int key_of(unsigned long long w) { return (int)(w >> 32); }

// First entry of list[from, to) whose id is not `key` (to if there is none); a warp's search.
SMDM_DEV int run_end(const unsigned long long* list, int from, int to, int key, int lane) {
  for (int i = from; i < to; i += 32) {
    const unsigned m = __ballot_sync(0xffffffffu, i + lane < to && key_of(list[i + lane]) != key);
    if (m) return i + __ffs(m) - 1;
  }
  return to;
}

// Sum the rows of every token.  One warp takes a piece of `per` sorted entries and 256 columns.  A
// run of one token that starts in a piece and ends within the next one is summed by the warp
// where it starts and written at once, rounded from its fp32 sum.  A longer one ([MASK]) leaves
// its part in slot 1 of the piece where it starts and in slot 0 of every later one
// (embed_join_kernel adds them up in order).
// Eight rows are in flight per warp.  (Four, loaded while the four before are added: 32 -> 41 us
// for 12544 rows of 4096 bf16; the wait for memory then covers half as many bytes.)
template <typename T, typename O, bool VECT>
__global__ void __launch_bounds__(256) embed_sum_kernel(EmbedGradArgs a) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = a.e.rows, d = a.e.d, none = a.e.n_emb;   // (id n_emb: takes no part)
  T* table = static_cast<T*>(a.e.grad_table);
  const int job = blockIdx.x * 8 + warp;
  const int piece = job / a.slabs, slab = job % a.slabs;
  if (piece >= a.pieces) return;
  // this lane's columns: 8 in a row (bf16 rows), 4 and 4 that lie 128 apart (fp32), or 8 that
  // lie 32 apart (rows off their 16-byte boundaries)
  constexpr int N = !VECT ? 1 : sizeof(O) == 2 ? 8 : 4;
  auto col = [&](int j) { return slab * 256 + (j / N) * 32 * N + lane * N + j % N; };
  const O* g = static_cast<const O*>(a.e.grad_out);

  // the entries to take: the piece, without a run that the piece before takes whole, and with
  // the rest of its own last run when that ends within the next piece
  const int i0 = piece * a.per, i1 = min(n, i0 + a.per);
  const int first_key = key_of(a.list[i0]), last_key = key_of(a.list[i1 - 1]);
  const int prev_key = i0 > 0 ? key_of(a.list[i0 - 1]) : -1;
  int begin = i0, end = i1;
  if (first_key == prev_key && last_key != prev_key &&
      (i0 == a.per || key_of(a.list[i0 - a.per - 1]) != prev_key))
    begin = run_end(a.list, i0, i1, prev_key, lane);
  const bool starts_here = !(first_key == last_key && prev_key == last_key);
  if (i1 < n && starts_here && last_key < none && key_of(a.list[i1]) == last_key) {
    const int next = min(n, i1 + a.per);
    if (key_of(a.list[next - 1]) != last_key) end = run_end(a.list, i1, next, last_key, lane);
  }
  const int after = end < n ? key_of(a.list[end]) : -1;    // the id behind the entries

  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  int base = begin;        // entries base .. base + 63 are in cur and nxt, one per lane
  int cur_key, cur_row, nxt_key, nxt_row;
  auto fetch = [&](int at, int& key, int& row) {
    const unsigned long long w = at + lane < end ? a.list[at + lane] : 0;
    key = at + lane < end ? key_of(w) : none;
    row = (int)(unsigned)w;                       // (row 0 where there is no entry)
  };
  fetch(base, cur_key, cur_row);
  fetch(base + 32, nxt_key, nxt_row);
  constexpr int kAhead = 8;
  Raw<O, N> v[kAhead][8 / N];
  bool first_run = true;
  for (int e = begin; e < end; e += kAhead) {
    // (rows that take no part are read and left out)
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const O* r = g + (size_t)__shfl_sync(0xffffffffu, cur_row, e - base + k) * a.e.ld_grad;
#pragma unroll
      for (int j = 0; j < 8; j += N) v[k][j / N].load(r + min(col(j), d - N));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int at = e - base + k;
      const int key = __shfl_sync(0xffffffffu, cur_key, at & 31);
      const int follow = __shfl_sync(0xffffffffu, at == 31 ? nxt_key : cur_key, (at + 1) & 31);
      if (e + k >= end || key >= none) continue;             // uniform over the warp
#pragma unroll
      for (int j = 0; j < 8; j += N) {
        float w[N];
        v[k][j / N].get(w);
#pragma unroll
        for (int x = 0; x < N; ++x) acc[j + x] += w[x];
      }
      const bool last = e + k + 1 >= end;
      if (!last && follow == key) continue;                  // the run goes on
      const bool from_before = first_run && key == prev_key;
      const bool goes_on = last && after == key;
      if (from_before || goes_on) {
        float* p = a.part + ((size_t)piece * 2 + (from_before ? 0 : 1)) * d;
#pragma unroll
        for (int j = 0; j < 8; j += N)
          if (col(j) < d) {
            if constexpr (VECT) store_n<N>(p + col(j), acc + j);
            else p[col(j)] = acc[j];
          }
      } else {
        T* o = table + (size_t)key * d;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] *= a.e.scale;
#pragma unroll
        for (int j = 0; j < 8; j += N)
          if (col(j) < d) {
            if constexpr (VECT) store_n<N>(o + col(j), acc + j);
            else o[col(j)] = from_f<T>(acc[j]);
          }
      }
      first_run = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    }
    if (e + kAhead - base == 32) {
      base += 32;
      cur_key = nxt_key;
      cur_row = nxt_row;
      fetch(base + 32, nxt_key, nxt_row);
    }
  }
}

constexpr int kJoinThreads = 512;

// Add up the parts of every run that starts in one piece and goes on in the next: 16 warps
// take every 16th part in order, then the warps' sums are added in order.  The CTAs with one
// blockIdx.x look at the same 256 pieces, find the runs that start there and share their (run,
// column block) pairs; a CTA per piece would mostly start CTAs that have nothing to do.
// VECT: a lane's four columns lie together, else 32 apart.
template <typename T, bool VECT>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(EmbedGradArgs a) {
  griddep_launch();
  griddep_wait();
  constexpr int VEC = 4, kCols = 32 * VEC;
  __shared__ int s_run[256];
  constexpr int kGroups = kJoinThreads / 32;
  __shared__ int s_warp[kGroups];
  __shared__ float sh[kGroups][kCols];
  const int d = a.e.d, n = a.e.rows;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int blocks = (d + kCols - 1) / kCols;
  T* table = static_cast<T*>(a.e.grad_table);
  const int p = blockIdx.x * 256 + threadIdx.x;
  bool starts = false;
  if (threadIdx.x < 256 && p + 1 < a.pieces) {
    const int i0 = p * a.per, i1 = i0 + a.per;
    const int key = key_of(a.list[i1 - 1]);
    // it goes on, through the whole next piece, and did not come in
    starts = key < a.e.n_emb && key_of(a.list[min(n, i1 + a.per) - 1]) == key &&
             !(i0 > 0 && key_of(a.list[i0]) == key && key_of(a.list[i0 - 1]) == key);
  }
  const unsigned m = __ballot_sync(0xffffffffu, starts);
  if (lane == 0) s_warp[grp] = __popc(m);
  __syncthreads();
  int at = 0, runs = 0;
  for (int w = 0; w < kGroups; ++w) {
    if (w < grp) at += s_warp[w];
    runs += s_warp[w];
  }
  if (starts) s_run[at + __popc(m & ((1u << lane) - 1u))] = p;
  __syncthreads();
  const long long jobs = (long long)runs * blocks;
  for (long long j = blockIdx.y; j < jobs; j += gridDim.y) {
    const int first = s_run[j / blocks];
    const int c0 = (int)(j % blocks) * kCols;
    auto col = [&](int e) { return VECT ? lane * VEC + e : e * 32 + lane; };
    const int key = key_of(a.list[(size_t)(first + 1) * a.per]);
    // part 0: slot 1 of the first piece; part k: slot 0 of the k-th piece after it, as long as
    // that piece begins with this token (its list entry is read along with the part)
    float s[VEC];
#pragma unroll
    for (int k = 0; k < VEC; ++k) s[k] = 0.f;
    bool more = true;
    for (int k0 = grp; more && first + k0 < a.pieces; k0 += kGroups * 4) {
      float v[4][VEC];
      bool in[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + kGroups * u, q = min(first + k, a.pieces - 1);
        in[u] = first + k < a.pieces && (k == 0 || key_of(a.list[(size_t)q * a.per]) == key);
        const float* p = a.part + ((size_t)q * 2 + (k == 0 ? 1 : 0)) * d;
        if constexpr (VECT) {
          load4(p + min(c0 + col(0), d - VEC), v[u]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v[u][e] = p[min(c0 + col(e), d - 1)];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        more = more && in[u];
        if (more)
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[e] += v[u][e];
      }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) sh[grp][col(e)] = s[e];
    __syncthreads();
    if (threadIdx.x < kCols) {
      const int cc = c0 + threadIdx.x;
      float t = 0.f;
      for (int g = 0; g < kGroups; ++g) t += sh[g][threadIdx.x];
      if (cc < d) table[(size_t)key * d + cc] = from_f<T>(t * a.e.scale);
    }
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) gather_f32_kernel(const float* x, const int* index, int rows,
                                                         int n, int d, float* out,
                                                         uint32_t* status) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  int r = index[row];
  if (r < 0 || r >= n) {
    if (lane == 0 && status) atomicOr(status, kStatusBounds);
    r = 0;
  }
  for (int c = lane * 4; c < d; c += 128)
    *reinterpret_cast<float4*>(out + (size_t)row * d + c) =
        *reinterpret_cast<const float4*>(x + (size_t)r * d + c);
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
size_t up_to(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Threads per row: a warp up to 1024 elements (32 per lane), then the whole CTA.
int norm_tpr(int d) { return d <= 1024 ? 32 : 256; }

int norm_grad_ctas(int rows, int d) {
  const int tpr = norm_tpr(d), rpc = std::max(1, 256 / tpr);
  if (tpr > 32 && rows <= 4) return 1;
  return std::min((rows + rpc - 1) / rpc, device_sms() * (tpr == 32 ? 4 : 2));
}

// Wide rows whose every copy starts on 16 bytes: two CTAs of 256 threads per SM, or one of 512
// above 4096 elements, with as many stages as their share of shared memory holds.
template <typename X, typename T, int TH>
cudaError_t rms_ring(const RmsArgs& a, int* ctas, cudaStream_t st) {
  RmsRing q{};
  const int xb = (int)up_to(a.d * sizeof(X), 128), gb = (int)up_to(a.d * sizeof(T), 128);
  q.gy_off = xb;
  q.add_off = xb + gb;
  q.stage_bytes = xb + gb + (a.add ? xb : 0);
  const int budget = (TH == 256 ? 110 : 220) * 1024;
  q.stages = std::min(8, budget / q.stage_bytes);
  auto kern = train_rms_grad_ring_kernel<X, T, TH>;
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, budget);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  // (four rows one after the other cost less than a second launch)
  *ctas = a.rows <= 4 ? 1 : std::min(a.rows, device_sms() * (512 / TH));
  return launch_pdl(kern, dim3(*ctas), dim3(TH), (size_t)q.stages * q.stage_bytes, st, 1, a, q);
}

template <typename X, typename T, int TPR, int VEC, int NU>
cudaError_t rms_one(const RmsArgs& a, int* grad_ctas, cudaStream_t st) {
  constexpr int B = kNormThreads, RPC = B / TPR;
  if (!grad_ctas)
    return launch_pdl(train_rms_kernel<X, T, TPR, VEC, NU>, dim3((a.rows + RPC - 1) / RPC),
                      dim3(B), 0, st, 1, a);
  *grad_ctas = norm_grad_ctas(a.rows, a.d);
  return launch_pdl(train_rms_grad_kernel<X, T, TPR, VEC, NU>, dim3(*grad_ctas), dim3(B),
                    RPC > 1 ? (size_t)a.d * RPC * 4 : 0, st, 1, a);
}

template <typename X, typename T>
cudaError_t rms_types(const RmsArgs& a, int* grad, cudaStream_t st) {
  // four elements at a time where every row starts on their alignment
  bool v4 = a.d % 4 == 0 && a.ld_x % 4 == 0 && a.ld_y % 4 == 0 && aligned(a.x, 4 * sizeof(X)) &&
            aligned(a.gain, 4 * sizeof(T));
  if (!grad) v4 = v4 && aligned(a.y, 4 * sizeof(T));
  else
    v4 = v4 && aligned(a.grad_y, 4 * sizeof(T)) && aligned(a.grad_x, 4 * sizeof(X)) &&
         aligned(a.add, 4 * sizeof(X));
  const int tpr = norm_tpr(a.d);
  if (v4) {
    const bool ring = grad && tpr > 32 && a.d * sizeof(X) % 16 == 0 && a.d * sizeof(T) % 16 == 0 &&
                      a.ld_x * sizeof(X) % 16 == 0 && a.ld_y * sizeof(T) % 16 == 0 &&
                      aligned(a.x, 16) && aligned(a.grad_y, 16) && aligned(a.add, 16) &&
                      aligned(a.grad_gain, 4 * sizeof(T));
    if (ring)
      return a.d <= 4096 ? rms_ring<X, T, 256>(a, grad, st) : rms_ring<X, T, 512>(a, grad, st);
    if (tpr == 32) {
      return a.d <= 512 ? rms_one<X, T, 32, 4, 4>(a, grad, st) : rms_one<X, T, 32, 4, 8>(a, grad, st);
    }
    return a.d <= 4096 ? rms_one<X, T, 256, 4, 4>(a, grad, st)
                       : rms_one<X, T, 256, 4, 8>(a, grad, st);
  }
  if (tpr == 32)
    return a.d <= 256 ? rms_one<X, T, 32, 1, 8>(a, grad, st) : rms_one<X, T, 32, 1, 32>(a, grad, st);
  return rms_one<X, T, 256, 1, 32>(a, grad, st);
}

cudaError_t rms_any(const RmsArgs& a, int* grad, cudaStream_t st) {
  if (a.x_f32) return a.f32 ? rms_types<float, float>(a, grad, st)
                            : rms_types<float, __nv_bfloat16>(a, grad, st);
  return a.f32 ? rms_types<__nv_bfloat16, float>(a, grad, st)
               : rms_types<__nv_bfloat16, __nv_bfloat16>(a, grad, st);
}

struct EmbedPlan {
  int chunks, per, pieces, slabs;
  size_t list[2], part, total;
};

EmbedPlan embed_plan(int rows, int d) {
  EmbedPlan p{};
  p.chunks = (rows + kChunk - 1) / kChunk;
  p.slabs = (d + 255) / 256;
  // Entries of one warp: enough warps to fill the device (16 per SM), few enough runs cut.  For
  // 12544 rows of 4096 this gives 64 entries, 56 us; 32 entries 64 us, 128 entries 71.
  const long long warps = (long long)device_sms() * 16;
  p.per = rows <= 32 ? 32 : 8;       // (one piece needs no joining)
  while (p.per < 128 && (long long)rows * p.slabs / (2 * p.per) >= warps) p.per *= 2;
  p.pieces = (rows + p.per - 1) / p.per;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off = up_to(off + b, 256);
    return o;
  };
  p.list[0] = take((size_t)rows * 8);
  p.list[1] = take(p.chunks > 1 ? (size_t)rows * 8 : 0);
  p.part = take((size_t)p.pieces * 2 * d * 4);
  p.total = off;
  return p;
}

template <typename T, typename O>
cudaError_t embed_types(const EmbedArgs& a, cudaStream_t st) {
  const bool v = a.d % 8 == 0 && a.ld_table % 8 == 0 && aligned(a.table, 16) && aligned(a.out, 16);
  const dim3 grid((a.rows + 7) / 8);
  return v ? launch_pdl(embed_kernel<T, O, true>, grid, dim3(256), 0, st, 1, a)
           : launch_pdl(embed_kernel<T, O, false>, grid, dim3(256), 0, st, 1, a);
}

template <typename T, typename O>
cudaError_t embed_grad_types(const EmbedGradArgs& g, cudaStream_t st) {
  const EmbedArgs& a = g.e;
  const bool v = a.d % 8 == 0 && a.ld_grad % 8 == 0 && aligned(a.grad_out, 16) &&
                 aligned(a.grad_table, 16);
  const dim3 grid((unsigned)(((long long)g.pieces * g.slabs + 7) / 8));
  const cudaError_t e = v ? launch_pdl(embed_sum_kernel<T, O, true>, grid, dim3(256), 0, st, 1, g)
                          : launch_pdl(embed_sum_kernel<T, O, false>, grid, dim3(256), 0, st, 1, g);
  if (e != cudaSuccess || g.pieces < 2) return e;
  const int batches = (g.pieces - 1 + 255) / 256;
  const dim3 jgrid(batches, std::max(1, std::min(65535, device_sms() * 4 / batches)));
  return a.d % 4 == 0 ? launch_pdl(embed_join_kernel<T, true>, jgrid, dim3(kJoinThreads), 0, st, 1, g)
                      : launch_pdl(embed_join_kernel<T, false>, jgrid, dim3(kJoinThreads), 0, st, 1, g);
}

}  // namespace

cudaError_t launch_train_rmsnorm(const RmsArgs& a, cudaStream_t st) { return rms_any(a, nullptr, st); }

size_t rmsnorm_grad_bytes(int rows, int d) {
  return std::max<size_t>(256, up_to((size_t)norm_grad_ctas(rows, d) * d * 4, 256));
}

int rmsnorm_grad_launches(int rows, int d) { return norm_grad_ctas(rows, d) > 1 ? 2 : 1; }

cudaError_t launch_train_rmsnorm_grad(const RmsArgs& a, cudaStream_t st) {
  int parts = 0;
  const cudaError_t e = rms_any(a, &parts, st);
  if (e != cudaSuccess || parts == 1) return e;
  const dim3 grid((a.d + 31) / 32);
  return a.f32 ? launch_pdl(rms_gain_kernel<float>, grid, dim3(1024), 0, st, 1,
                            (const float*)a.ws, parts, a.d, static_cast<float*>(a.grad_gain))
               : launch_pdl(rms_gain_kernel<__nv_bfloat16>, grid, dim3(1024), 0, st, 1,
                            (const float*)a.ws, parts, a.d,
                            static_cast<__nv_bfloat16*>(a.grad_gain));
}

cudaError_t launch_embed(const EmbedArgs& a, cudaStream_t st) {
  if (a.f32) return a.out_f32 ? embed_types<float, float>(a, st)
                              : embed_types<float, __nv_bfloat16>(a, st);
  return a.out_f32 ? embed_types<__nv_bfloat16, float>(a, st)
                   : embed_types<__nv_bfloat16, __nv_bfloat16>(a, st);
}

size_t embed_grad_bytes(int rows, int d, int n_emb) {
  (void)n_emb;
  return std::max<size_t>(256, embed_plan(rows, d).total);
}

// Runs merged per level: as few as one level takes, up to 32 (every search reads the list from L2).
static int merge_ways(int n) {
  const int chunks = (n + kChunk - 1) / kChunk;
  return chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
}

int sort_ids_launches(int n) {
  int k = 1;
  for (long long run = kChunk; run < n; run *= merge_ways(n)) ++k;
  return k;
}

cudaError_t launch_sort_ids(const int* ids, int n, int n_ids, unsigned long long* a,
                            unsigned long long* b, void* clear, size_t clear_bytes,
                            uint32_t* status, cudaStream_t st, const unsigned long long** sorted) {
  static_assert(kChunk == 1 << 11, "the 32-bit words hold a place of 11 bits");
  auto sort = n_ids < (1 << 21) - 1 ? embed_sort_kernel<unsigned>
                                    : embed_sort_kernel<unsigned long long>;
  const int chunks = (n + kChunk - 1) / kChunk;
  int size = 256;
  while (size < kChunk && size < n) size *= 2;
  const int threads = size / 2;
  const int clears = (int)std::min<size_t>((size_t)device_sms() * (2048 / threads),
                                           (clear_bytes + 16 * threads - 1) / (16 * threads));
  cudaError_t e = launch_pdl(sort, dim3(chunks + clears), dim3(threads), 0, st, 1, ids, n, n_ids,
                             size, chunks, a, static_cast<uint8_t*>(clear), clear_bytes, status);
  if (e != cudaSuccess) return e;
  const int ways = merge_ways(n);
  for (long long run = kChunk; run < n; run *= ways) {
    const long long searches = (long long)n * ways;
    e = launch_pdl(embed_merge_kernel, dim3((unsigned)((searches + 255) / 256)), dim3(256), 0, st, 1,
                   (const unsigned long long*)a, n, (int)run, ways, b);
    if (e != cudaSuccess) return e;
    std::swap(a, b);
  }
  *sorted = a;
  return cudaSuccess;
}

cudaError_t launch_embed_grad(const EmbedArgs& a, cudaStream_t st) {
  const EmbedPlan p = embed_plan(a.rows, a.d);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  EmbedGradArgs g{};
  g.e = a;
  const cudaError_t e = launch_sort_ids(
      a.ids, a.rows, a.n_emb, reinterpret_cast<unsigned long long*>(ws + p.list[0]),
      reinterpret_cast<unsigned long long*>(ws + p.list[1]), a.grad_table,
      (size_t)a.n_emb * a.d * (a.f32 ? 4 : 2), a.status, st, &g.list);
  if (e != cudaSuccess) return e;
  g.part = reinterpret_cast<float*>(ws + p.part);
  g.per = p.per;
  g.pieces = p.pieces;
  g.slabs = p.slabs;
  if (a.f32) return a.out_f32 ? embed_grad_types<float, float>(g, st)
                              : embed_grad_types<float, __nv_bfloat16>(g, st);
  return a.out_f32 ? embed_grad_types<__nv_bfloat16, float>(g, st)
                   : embed_grad_types<__nv_bfloat16, __nv_bfloat16>(g, st);
}

cudaError_t launch_gather_f32(const float* x, const int* index, int rows, int n, int d, float* out,
                              uint32_t* status, cudaStream_t st) {
  return launch_pdl(gather_f32_kernel, dim3((rows + 7) / 8), dim3(256), 0, st, 1, x, index, rows, n,
                    d, out, status);
}

}  // namespace smdm
