// The LM head's loss and gradient for a handful of rows (kFewRows or fewer), on the CUDA cores.
//
// With so few rows the work is to pass the weights by once (and, for the gradient, to write
// theirs): 2 V d operations per row against the 4 or 2 bytes of a weight.  The matrix unit would
// pad the rows to 128, and fp32 weights would first be written out as bf16 parts, three times
// the bytes.  Here a warp takes four weight rows at a time, all of the hidden rows stay in
// shared memory, and each weight is read once, where it lies, in the type it has.
//
// It takes the calls whose weights would have to be written out (fp32 ones, and bf16 ones whose rows
// do not start on 16-byte boundaries).  fp32, 1024 x 32000: loss of 4 / 16 rows 36 / 70 us against
// 112 / 112 through the parts, gradient 103 / 151 us against 205 / 206.  What bounds it: up to eight
// rows the loads in flight (36 us are 3.6 TB/s, 0.56 of the measured peak: registers leave room for
// one to three blocks per SM), then the multiply-adds and the loads that feed them.
#include <algorithm>

#include "head.h"

namespace smdm {

namespace {

constexpr int kFewThreads = 256;
constexpr int kGradThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

SMDM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct FewDev {
  int rows, d, d_pad, vocab;     // d_pad: d rounded up to 256
  int row0;                      // logits: first row of the launch's group
  long long ld_hidden, ld_head;
  const void* hidden;
  const void* head;
  const int* target;
  // loss
  float2* part;                  // [16][CTAs]
  float* tlogit;                 // [16]
  // gradient
  const float* lse;
  const float* grad_nll;
  float* dlog;                   // [16][ld_dlog]
  int ld_dlog;
  float* acc;                    // [chunks][RM][d_pad]
  int chunk;                     // vocabulary rows of one gradient CTA
  void* grad_hidden;
  void* grad_head;
  uint32_t* status;
};

SMDM_DEV bool takes_part(const FewDev& a, int r) {
  return r < a.rows && a.target[r] >= 0 && a.target[r] < a.vocab;
}

// E elements as loaded (16 bytes of them, or one).
template <typename T, int E>
struct Piece {
  uint32_t w[4];
  SMDM_DEV void load(const T* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  }
  SMDM_DEV void zero() { w[0] = w[1] = w[2] = w[3] = 0; }
  SMDM_DEV float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
template <>
struct Piece<__nv_bfloat16, 2> {
  uint32_t w;
  SMDM_DEV void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint32_t*>(p); }
  SMDM_DEV void zero() { w = 0; }
  SMDM_DEV float get(int i) const { return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16); }
};
template <typename T>
struct Piece<T, 1> {
  T x;
  SMDM_DEV void load(const T* p) { x = *p; }
  SMDM_DEV void zero() { x = T(0.f); }
  SMDM_DEV float get(int) const { return to_f<T>(x); }
};

// Logits of RM rows: a warp and four vocabulary rows per turn.  GRAD: their gradient into dlog;
// else the running (maximum, sum) of every row.
// E: elements per load (16 bytes; 4 or one element for rows off those boundaries).
template <typename T, int E, int RM, bool GRAD>
__global__ void __launch_bounds__(kFewThreads) few_logits_kernel(FewDev a) {
  griddep_launch();
  griddep_wait();
  extern __shared__ __align__(16) float sh[];       // [RM][d_pad]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = warp; i < RM; i += kFewThreads / 32) {
    // (a row that takes no part counts as zeros: what it holds reaches nothing)
    const int r = a.row0 + i;
    const bool on = takes_part(a, r);
    const T* h = static_cast<const T*>(a.hidden) + (size_t)r * a.ld_hidden;
    for (int c = lane; c < a.d_pad; c += 32)
      sh[(size_t)i * a.d_pad + c] = on && c < a.d ? to_f<T>(h[c]) : 0.f;
    if (blockIdx.x == 0 && lane == 0 && r < a.rows && a.target[r] >= a.vocab && a.status)
      atomicOr(a.status, kStatusBounds);
  }
  __syncthreads();
  constexpr int NV = 4, N = NV * RM;                // sums of a turn, index r * NV + v
  constexpr int U = E * sizeof(T) < 16 ? 8 : 2;     // K steps whose loads are in flight together
  constexpr int KEEP = N >= 32 ? N / 32 : 1;        // sums a lane ends up with
  constexpr int EH = E < 4 ? E : 4;                 // hidden values per shared load
  constexpr int DUP = N < 32 ? 32 / N : 1;          // lanes that end up with the same sum
  // the lane's sums: index first + 0 .. KEEP - 1
  const int first = lane / DUP * KEEP;
  const int my_r = a.row0 + first / NV;
  const int tgt = takes_part(a, my_r) ? a.target[my_r] : -1;
  float lse = 0.f, g = 0.f;
  if (GRAD && tgt >= 0) {
    lse = a.lse[my_r];
    g = a.grad_nll[my_r];
  }
  float m = -INFINITY, s = 0.f;
  const int step = gridDim.x * (kFewThreads / 32) * NV;
  for (int v0 = (blockIdx.x * (kFewThreads / 32) + warp) * NV; v0 < a.vocab; v0 += step) {
    const T* w[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
      w[i] = static_cast<const T*>(a.head) + (size_t)min(v0 + i, a.vocab - 1) * a.ld_head;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int k0 = lane * E; k0 < a.d; k0 += 32 * E * U) {
      Piece<T, E> p[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = k0 + u * 32 * E;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (k < a.d) p[u][i].load(w[i] + k);
          else p[u][i].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        // (past d the weights are zero and the copy of the row is, too: d_pad covers it)
        const int k = min(k0 + u * 32 * E, a.d_pad - E);
#pragma unroll
        for (int e0 = 0; e0 < E; e0 += EH) {
#pragma unroll
          for (int r = 0; r < RM; ++r) {
            float h[4];
            if constexpr (EH == 4) {
              const float4 f = *reinterpret_cast<const float4*>(sh + (size_t)r * a.d_pad + k + e0);
              h[0] = f.x; h[1] = f.y; h[2] = f.z; h[3] = f.w;
            } else if constexpr (EH == 2) {
              const float2 f = *reinterpret_cast<const float2*>(sh + (size_t)r * a.d_pad + k);
              h[0] = f.x; h[1] = f.y;
            } else {
              h[0] = sh[(size_t)r * a.d_pad + k];
            }
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int e = 0; e < EH; ++e)
                acc[r * NV + i] = fmaf(p[u][i].get(e0 + e), h[e], acc[r * NV + i]);
          }
        }
      }
    }
    // sums over the lanes: each step halves the sums a lane is left with
    int cnt = N;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (cnt > 1) {
        cnt >>= 1;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
          if (i < cnt) {
            const float keep = (lane & o) ? acc[i + cnt] : acc[i];
            const float send = (lane & o) ? acc[i] : acc[i + cnt];
            acc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
      } else {
        acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], o);
      }
    }
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
      const int v = v0 + (first + i) % NV;
      const float z = acc[i];
      if (v >= a.vocab) continue;
      if constexpr (GRAD) {
        float q = ex2((z - lse) * kLog2e);
        if (v == tgt) q -= 1.f;
        if (lane % DUP == 0)
          a.dlog[(size_t)my_r * a.ld_dlog + v] = tgt >= 0 ? q * g : 0.f;
      } else {
        if (v == tgt) a.tlogit[my_r] = z;
        const float mn = fmaxf(m, z), ref = mn == -INFINITY ? 0.f : mn;
        s = s * (s == 0.f ? 0.f : ex2((m - ref) * kLog2e)) + ex2((z - ref) * kLog2e);
        m = mn;
      }
    }
  }
  if constexpr (!GRAD) {
    // (lanes that hold copies of one sum, N < 32, count once)
    if (lane % DUP != 0) s = 0.f;
    __shared__ float2 red[kFewThreads];
    red[threadIdx.x] = make_float2(m, s);
    __syncthreads();
    // row r: lanes whose my_r is r, of every warp
    constexpr int LPR = 32 / RM;                    // lanes of a row in a warp
    for (int r = warp; r < RM; r += kFewThreads / 32) {
      float2 p = make_float2(-INFINITY, 0.f);
      // 8 warps x LPR lanes entries, spread over the lanes
      for (int i = lane; i < kFewThreads / 32 * LPR; i += 32) {
        const float2 q = red[(i / LPR) * 32 + r * LPR + i % LPR];
        if (q.y != 0.f) {
          const float mn = fmaxf(p.x, q.x);
          p.y = p.y * (p.y == 0.f ? 0.f : ex2((p.x - mn) * kLog2e)) + q.y * ex2((q.x - mn) * kLog2e);
          p.x = mn;
        }
      }
      float mx = p.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      float t = p.y == 0.f ? 0.f : p.y * ex2((p.x - mx) * kLog2e);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
      if (lane == 0) a.part[(size_t)(a.row0 + r) * gridDim.x + blockIdx.x] = make_float2(mx, t);
    }
  }
}

// nll and lse from the CTAs' pairs: one warp per row.
__global__ void __launch_bounds__(512) few_finish_kernel(FewDev a, int ctas, float* nll, float* lse) {
  griddep_launch();
  griddep_wait();
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
  if (r >= a.rows) return;
  float m = -INFINITY;
  for (int i = lane; i < ctas; i += 32) {
    const float2 p = a.part[(size_t)r * ctas + i];
    if (p.y != 0.f) m = fmaxf(m, p.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float s = 0.f;
  for (int i = lane; i < ctas; i += 32) {
    const float2 p = a.part[(size_t)r * ctas + i];
    if (p.y != 0.f) s += p.y * ex2((p.x - m) * kLog2e);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
    const bool on = takes_part(a, r);
    const float l = logf(s);
    lse[r] = on ? m + l : 0.f;
    nll[r] = on ? (m - a.tlogit[r]) + l : 0.f;
  }
}

// Both products of the logits' gradient D in one pass over the weights: a thread owns NC columns,
// its hidden values and its sums of dH stay in registers; for every vocabulary row it reads the
// weights once (dH += D w) and writes their gradient (dW = sum over rows of D h).
// NC: 4 columns in a row, or 1.
template <typename T, int NC, int RM>
__global__ void __launch_bounds__(kGradThreads) few_grad_kernel(FewDev a) {
  griddep_launch();
  griddep_wait();
  constexpr int kSub = 64;                          // vocabulary rows whose D is staged at once
  __shared__ __align__(16) float dl[kSub][RM];
  const int c = (blockIdx.x * kGradThreads + threadIdx.x) * NC;
  const bool in = c < a.d;
  float h[RM][NC], acc[RM][NC];
#pragma unroll
  for (int r = 0; r < RM; ++r) {
    const bool on = takes_part(a, r) && in;
    const T* p = static_cast<const T*>(a.hidden) + (size_t)r * a.ld_hidden + c;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      h[r][k] = on ? to_f<T>(p[k]) : 0.f;
      acc[r][k] = 0.f;
    }
  }
  const int v_begin = blockIdx.y * a.chunk, v_end = min(a.vocab, v_begin + a.chunk);
  const T* w = static_cast<const T*>(a.head) + c;
  T* gw = a.grad_head ? static_cast<T*>(a.grad_head) + c : nullptr;
  const bool need_w = a.grad_hidden != nullptr;
  for (int vb = v_begin; vb < v_end; vb += kSub) {
    const int nv = min(kSub, v_end - vb);
    __syncthreads();
    for (int i = threadIdx.x; i < kSub * RM; i += kGradThreads) {
      const int v = i % kSub, r = i / kSub;
      dl[v][r] = v < nv && r < a.rows ? a.dlog[(size_t)r * a.ld_dlog + vb + v] : 0.f;
    }
    __syncthreads();
    if (!in) continue;
    constexpr int U = 4;                            // weight rows in flight
    for (int v = 0; v < nv; v += U) {
      float x[U][NC];
      if constexpr (NC == 4) {
        uint4 raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const T* p = w + (size_t)(vb + min(v + u, nv - 1)) * a.ld_head;
          if (!need_w) raw[u] = make_uint4(0, 0, 0, 0);
          else if constexpr (sizeof(T) == 4) raw[u] = *reinterpret_cast<const uint4*>(p);
          else {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            raw[u] = make_uint4(q.x, q.y, 0, 0);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if constexpr (sizeof(T) == 4) {
            x[u][0] = __uint_as_float(raw[u].x); x[u][1] = __uint_as_float(raw[u].y);
            x[u][2] = __uint_as_float(raw[u].z); x[u][3] = __uint_as_float(raw[u].w);
          } else {
            x[u][0] = __uint_as_float(raw[u].x << 16);
            x[u][1] = __uint_as_float(raw[u].x & 0xffff0000u);
            x[u][2] = __uint_as_float(raw[u].y << 16);
            x[u][3] = __uint_as_float(raw[u].y & 0xffff0000u);
          }
        }
      } else {
        T raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          raw[u] = need_w ? w[(size_t)(vb + min(v + u, nv - 1)) * a.ld_head] : T(0.f);
#pragma unroll
        for (int u = 0; u < U; ++u) x[u][0] = to_f<T>(raw[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (v + u >= nv) break;
        float o[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) o[k] = 0.f;
#pragma unroll
        for (int r = 0; r < RM; ++r) {
          const float q = dl[v + u][r];
#pragma unroll
          for (int k = 0; k < NC; ++k) {
            o[k] = fmaf(q, h[r][k], o[k]);
            acc[r][k] = fmaf(q, x[u][k], acc[r][k]);
          }
        }
        if (gw) {
          T* p = gw + (size_t)(vb + v + u) * a.d;
          if constexpr (NC == 4) {
            if constexpr (sizeof(T) == 4) {
              __stcs(reinterpret_cast<float4*>(p), make_float4(o[0], o[1], o[2], o[3]));
            } else {
              const __nv_bfloat162 lo = __floats2bfloat162_rn(o[0], o[1]),
                                   hi = __floats2bfloat162_rn(o[2], o[3]);
              __stcs(reinterpret_cast<uint2*>(p),
                     make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                *reinterpret_cast<const uint32_t*>(&hi)));
            }
          } else {
            *p = from_f<T>(o[0]);
          }
        }
      }
    }
  }
  if (in && need_w)
#pragma unroll
    for (int r = 0; r < RM; ++r)
#pragma unroll
      for (int k = 0; k < NC; ++k)
        a.acc[((size_t)blockIdx.y * RM + r) * a.d_pad + c + k] = acc[r][k];
}

// dH: the vocabulary chunks' sums, 32 columns and 32 chunk groups per CTA; zeros for a row that
// takes no part, whatever the weights hold.
template <typename T, int RM>
__global__ void __launch_bounds__(1024) few_sum_kernel(FewDev a, int chunks) {
  griddep_launch();
  griddep_wait();
  __shared__ float sh[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int r = blockIdx.y, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < a.d)
#pragma unroll 8
    for (int k = g; k < chunks; k += 32) s += a.acc[((size_t)k * RM + r) * a.d_pad + c];
  sh[g][lane] = s;
  __syncthreads();
  s = sh[lane][g];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int cc = blockIdx.x * 32 + g;
  if (lane == 0 && cc < a.d)
    static_cast<T*>(a.grad_hidden)[(size_t)r * a.d + cc] = from_f<T>(takes_part(a, r) ? s : 0.f);
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int few_rm(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }
// Rows of one logits launch: as many as fit shared memory (0: not even four).
int few_group(int rows, int d) {
  int g = few_rm(rows);
  while (g >= 4 && (size_t)g * up(d, 256) * 4 > (size_t)kFewSmem) g /= 2;
  return g < 4 ? 0 : g;
}
size_t few_smem(int rows, int d) { return (size_t)few_group(rows, d) * up(d, 256) * 4; }

struct FewPlan {
  int rm, group, ctas, slabs, chunk, chunks;
  size_t part, tlogit, dlog, acc, total;
};

// wide: four columns per gradient thread.  (The workspace is sized for both.)
FewPlan few_plan(int rows, int d, int vocab, int sms, bool wide) {
  FewPlan p{};
  p.rm = few_rm(rows);
  p.group = few_group(rows, d);
  const int per_sm = few_smem(rows, d) <= 56 * 1024 ? 4 : few_smem(rows, d) <= 110 * 1024 ? 2 : 1;
  p.ctas = std::min((vocab + 31) / 32, sms * per_sm);
  const int cols = kGradThreads * (wide ? 4 : 1);
  p.slabs = (d + cols - 1) / cols;
  // about three CTAs per SM
  const int want = std::max(1, sms * 3 / p.slabs);
  p.chunk = std::max(16, (vocab + want - 1) / want);
  p.chunks = (vocab + p.chunk - 1) / p.chunk;
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off = up(off + b, 1024);
    return o;
  };
  p.part = take((size_t)p.rm * p.ctas * 8);
  p.tlogit = take((size_t)p.rm * 4);
  p.dlog = take((size_t)p.rm * up(vocab, 64) * 4);
  p.acc = take((size_t)p.chunks * p.rm * up(d, 256) * 4);
  p.total = off;
  return p;
}

template <typename K>
cudaError_t opt_in(K kern, bool* ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
  if (e == cudaSuccess) ready[dev] = true;
  return e;
}

template <typename T, int E, int RM, bool GRAD>
cudaError_t logits_one(const FewDev& a, int ctas, cudaStream_t st) {
  static bool ready[64];
  auto kern = few_logits_kernel<T, E, RM, GRAD>;
  const cudaError_t e = opt_in(kern, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kFewThreads), (size_t)RM * a.d_pad * 4, st, 1, a);
}

template <typename T, int E, bool GRAD>
cudaError_t logits_rm(FewDev a, const FewPlan& p, cudaStream_t st) {
  for (a.row0 = 0; a.row0 < a.rows; a.row0 += p.group) {
    const cudaError_t e = p.group == 4   ? logits_one<T, E, 4, GRAD>(a, p.ctas, st)
                          : p.group == 8 ? logits_one<T, E, 8, GRAD>(a, p.ctas, st)
                                         : logits_one<T, E, 16, GRAD>(a, p.ctas, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool GRAD>
cudaError_t logits_any(const HeadArgs& h, const FewDev& a, const FewPlan& p, cudaStream_t st) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(h.head);
  const int es = h.f32 ? 4 : 2;
  const bool words = base % 16 == 0 && (long long)h.d * es % 16 == 0 && h.ld_head * es % 16 == 0;
  if (h.f32)
    return words ? logits_rm<float, 4, GRAD>(a, p, st) : logits_rm<float, 1, GRAD>(a, p, st);
  if (words) return logits_rm<__nv_bfloat16, 8, GRAD>(a, p, st);
  return base % 4 == 0 && h.d % 2 == 0 && h.ld_head % 2 == 0
             ? logits_rm<__nv_bfloat16, 2, GRAD>(a, p, st)
             : logits_rm<__nv_bfloat16, 1, GRAD>(a, p, st);
}

template <typename T, int RM>
cudaError_t grad_rm(const FewDev& a, const FewPlan& p, bool wide, cudaStream_t st) {
  const dim3 grid(p.slabs, p.chunks);
  const cudaError_t e =
      wide ? launch_pdl(few_grad_kernel<T, 4, RM>, grid, dim3(kGradThreads), 0, st, 1, a)
           : launch_pdl(few_grad_kernel<T, 1, RM>, grid, dim3(kGradThreads), 0, st, 1, a);
  if (e != cudaSuccess || !a.grad_hidden) return e;
  return launch_pdl(few_sum_kernel<T, RM>, dim3((a.d + 31) / 32, a.rows), dim3(1024), 0, st, 1, a,
                    p.chunks);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

FewDev few_dev(const HeadArgs& h, const FewPlan& p) {
  FewDev a{};
  uint8_t* ws = static_cast<uint8_t*>(h.ws);
  a.rows = h.rows;
  a.d = h.d;
  a.d_pad = (int)up(h.d, 256);
  a.vocab = h.vocab;
  a.ld_hidden = h.ld_hidden;
  a.ld_head = h.ld_head;
  a.hidden = h.hidden;
  a.head = h.head;
  a.target = h.target;
  a.part = reinterpret_cast<float2*>(ws + p.part);
  a.tlogit = reinterpret_cast<float*>(ws + p.tlogit);
  a.lse = h.lse;
  a.grad_nll = h.grad_nll;
  a.dlog = reinterpret_cast<float*>(ws + p.dlog);
  a.ld_dlog = (int)up(h.vocab, 64);
  a.acc = reinterpret_cast<float*>(ws + p.acc);
  a.chunk = p.chunk;
  a.grad_hidden = h.grad_hidden;
  a.grad_head = h.grad_head;
  a.status = h.status;
  return a;
}

bool weight_words(const HeadArgs& h) {
  const int es = h.f32 ? 4 : 2;
  return on16(h.head) && (long long)h.d * es % 16 == 0 && h.ld_head * es % 16 == 0;
}

}  // namespace

bool head_few_fits(int rows, int d) { return rows <= kFewRows && few_group(rows, d) > 0; }

int head_few_groups(int rows, int d) {
  const int g = few_group(rows, d);
  return (rows + g - 1) / g;
}

size_t head_few_bytes(int rows, int d, int vocab, int sms) {
  return std::max(few_plan(rows, d, vocab, sms, true).total,
                  few_plan(rows, d, vocab, sms, false).total);
}

cudaError_t launch_head_few_loss(const HeadArgs& h, int sms, cudaStream_t st) {
  const FewPlan p = few_plan(h.rows, h.d, h.vocab, sms, true);
  const FewDev a = few_dev(h, p);
  const cudaError_t e = logits_any<false>(h, a, p, st);
  if (e != cudaSuccess) return e;
  return launch_pdl(few_finish_kernel, dim3(1), dim3(32 * p.rm), 0, st, 1, a, p.ctas, h.nll,
                    h.lse_out);
}

cudaError_t launch_head_few_grad(const HeadArgs& h, int sms, cudaStream_t st) {
  const bool vec = weight_words(h);
  const bool wide = vec && (!h.grad_head || on16(h.grad_head));
  const FewPlan p = few_plan(h.rows, h.d, h.vocab, sms, wide);
  const FewDev a = few_dev(h, p);
  const cudaError_t e = logits_any<true>(h, a, p, st);
  if (e != cudaSuccess) return e;
  switch (p.rm) {
    case 4: return h.f32 ? grad_rm<float, 4>(a, p, wide, st) : grad_rm<__nv_bfloat16, 4>(a, p, wide, st);
    case 8: return h.f32 ? grad_rm<float, 8>(a, p, wide, st) : grad_rm<__nv_bfloat16, 8>(a, p, wide, st);
    default: return h.f32 ? grad_rm<float, 16>(a, p, wide, st) : grad_rm<__nv_bfloat16, 16>(a, p, wide, st);
  }
}

}  // namespace smdm
