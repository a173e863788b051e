// rmsnorm.cuh -- K16: RMSNorm on its own (the model's final norm in training) and its gradients.
//
//   forward   rho = (mean(x^2) + eps)^(-1/2),  y = x rho w
//   backward  u = dy w,  dx = rho u - x rho (rho (rho mean(u x))),  dw[c] = sum_r dy[r][c] x[r][c] rho_r
//
// Bound by HBM: one read of x (and dy), one write of y (dx). A CTA takes R rows at a time with every
// thread holding the same 8-column chunks of each row in registers, so a row is read once, one block
// reduction serves R rows, and in the backward the thread's share of dw stays in registers over all
// rows of the CTA (written once as a partial row, added up in a fixed order by a second kernel). Rows
// that 16-byte accesses do not fit (an odd width, an unaligned base) go through kernels that hold single
// columns in registers instead, up to 11 * 256 of them, and are read twice beyond that or beyond 16384.
// Sums are float32; y, dx are rounded once to their type. 16384 x 1024 bf16: forward 13.2 us (5.1 TB/s),
// backward 21 + 3.5 us (4.8 TB/s; 39.5 us before the next rows' loads were issued ahead of the block
// reduction), together 37.5 us of device time against a floor of 25.6. Forward + backward in the same way:
// 8192 x 2560 bf16 52 us (floor 32), 5001 x 2048 float32 41 (31), 16384 x 2053 bf16 146 (51).
#pragma once

#include "common.cuh"

namespace mmf {
namespace rms {

constexpr int kMaxThreads = 512;
constexpr int kMaxChunks = 4;    // 8-column chunks per thread: rows of up to 16384
constexpr int kGenThreads = 256;

struct Args {
  const void* x;        // [m][d]
  const void* dy;       // backward [m][d]
  const float* w;       // [d] or nullptr (1)
  void* out;            // forward y, backward dx
  float* part;          // backward [gridDim.x][d] partial dw, or nullptr
  int64_t m;
  int32_t d;
  float eps;
};

// These kernels launch as programmatic dependents: set-up overlaps the end of the kernel before, nothing
// is read or written before the wait.
__device__ __forceinline__ void dependent() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <mmf_dtype DT>
__device__ __forceinline__ void load8(const void* p, int64_t idx, float (&v)[8]) {
  if (DT == MMF_F32) {
    const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + idx);
    const float4 a = s[0], b = s[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + idx);
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(u[q] << 16);
      v[2 * q + 1] = __uint_as_float(u[q] & 0xffff0000u);
    }
  }
}
template <mmf_dtype DT>
__device__ __forceinline__ void store8(void* p, int64_t idx, const float (&v)[8]) {
  if (DT == MMF_F32) {
    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + idx);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * q], v[2 * q + 1]);
      u[q] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p) + idx) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// dx = rho u - k xh with xh = x rho and k = rho (rho mean(u x)), which is of dx's size: rho^3 alone leaves
// float32's range for rows of 1e15, or of 1e-13 without eps. The roundings are spelled out, so that dx does not
// depend on what the compiler fuses where dw is asked for.
__device__ __forceinline__ float grad(float rho, float u, float k, float xh) { return fmaf(-k, xh, __fmul_rn(rho, u)); }

// Block sums of V values at once; red has V * 16 floats. One barrier before the result; the caller
// alternates between two red arrays, so that the next call's writes cannot meet this call's reads.
template <int V>
__device__ __forceinline__ void block_sums(float (&v)[V], float (*red)[16]) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = warp_sum(v[i]);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) red[i][wid] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += red[i][w];
    v[i] = s;
  }
}

// d % 8 == 0, 16-byte aligned rows; chunk j of thread t is j * blockDim.x + t.
template <mmf_dtype XT, mmf_dtype YT, int NC, int R>
__global__ void __launch_bounds__(kMaxThreads) rms_fwd_kernel(const Args a) {
  dependent();
  __shared__ float red[2][R][16];
  const int nck = a.d >> 3, T = blockDim.x;
  const float inv_d = 1.0f / (float)a.d;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.m; r0 += (int64_t)gridDim.x * R, turn ^= 1) {
    float x[R][NC][8], ss[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = j * T + (int)threadIdx.x;
        if (r0 + r < a.m && c < nck) {
          load8<XT>(a.x, (r0 + r) * a.d + 8 * c, x[r][j]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[r][j][e] = 0.0f;
        }
      }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ss[r] = 0.0f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[r] = fmaf(x[r][j][e], x[r][j][e], ss[r]);
    }
    block_sums<R>(ss, red[turn]);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = j * T + (int)threadIdx.x;
      if (c >= nck) continue;
      float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (a.w) load8<MMF_F32>(a.w, 8 * c, w);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r0 + r >= a.m) continue;
        const float rho = rsqrtf(ss[r] * inv_d + a.eps);
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = x[r][j][e] * rho * w[e];
        store8<YT>(a.out, (r0 + r) * a.d + 8 * c, y);
      }
    }
  }
}

// Eight values as loaded: 16 bytes of bf16 or 32 of float32.
template <mmf_dtype DT> struct Raw8 { uint4 v[DT == MMF_F32 ? 2 : 1]; };
template <mmf_dtype DT>
__device__ __forceinline__ void load_raw(const void* p, int64_t idx, Raw8<DT>& r) {
  const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const typename Elem<DT>::T*>(p) + idx);
  r.v[0] = s[0];
  if (DT == MMF_F32) r.v[DT == MMF_F32 ? 1 : 0] = s[1];
}
template <mmf_dtype DT>
__device__ __forceinline__ float raw_at(const Raw8<DT>& r, int e) {
  if (DT == MMF_F32) {
    const uint4& q = r.v[DT == MMF_F32 ? e >> 2 : 0];
    const uint32_t w = (e & 3) == 0 ? q.x : (e & 3) == 1 ? q.y : (e & 3) == 2 ? q.z : q.w;
    return __uint_as_float(w);
  }
  const uint4& q = r.v[0];
  const uint32_t w = (e >> 1) == 0 ? q.x : (e >> 1) == 1 ? q.y : (e >> 1) == 2 ? q.z : q.w;
  return __uint_as_float(e & 1 ? w & 0xffff0000u : w << 16);
}

// The next turn's rows are loaded before this turn's block reduction, so that loads are in flight
// across its barrier.
template <mmf_dtype XT, mmf_dtype GT, int NC, int R>
__global__ void __launch_bounds__(kMaxThreads) rms_bwd_kernel(const Args a) {
  dependent();
  __shared__ float red[2][2 * R][16];
  const int nck = a.d >> 3, T = blockDim.x;
  const float inv_d = 1.0f / (float)a.d;
  float w[NC][8], dw[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = j * T + (int)threadIdx.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) { w[j][e] = 1.0f; dw[j][e] = 0.0f; }
    if (a.w && c < nck) load8<MMF_F32>(a.w, 8 * c, w[j]);
  }
  Raw8<XT> x[R][NC], xn[R][NC];
  Raw8<GT> g[R][NC], gn[R][NC];
  const auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = j * T + (int)threadIdx.x;
        xn[r][j] = Raw8<XT>{};
        gn[r][j] = Raw8<GT>{};
        if (r0 + r < a.m && c < nck) {
          load_raw<XT>(a.x, (r0 + r) * a.d + 8 * c, xn[r][j]);
          load_raw<GT>(a.dy, (r0 + r) * a.d + 8 * c, gn[r][j]);
        }
      }
  };
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * R;
  fetch((int64_t)blockIdx.x * R);
  for (int64_t r0 = (int64_t)blockIdx.x * R; r0 < a.m; r0 += step, turn ^= 1) {
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = s[R + r] = 0.0f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        x[r][j] = xn[r][j];
        g[r][j] = gn[r][j];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xv = raw_at<XT>(x[r][j], e);
          s[r] = fmaf(xv, xv, s[r]);
          s[R + r] = fmaf(raw_at<GT>(g[r][j], e) * w[j][e], xv, s[R + r]);
        }
      }
    }
    fetch(r0 + step);
    block_sums<2 * R>(s, red[turn]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r0 + r >= a.m) continue;
      const float rho = rsqrtf(s[r] * inv_d + a.eps);
      const float k = rho * (rho * (s[R + r] * inv_d));
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int c = j * T + (int)threadIdx.x;
        if (c >= nck) continue;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = __fmul_rn(raw_at<XT>(x[r][j], e), rho), gv = raw_at<GT>(g[r][j], e);
          dw[j][e] = fmaf(gv, xh, dw[j][e]);
          o[e] = grad(rho, gv * w[j][e], k, xh);
        }
        store8<XT>(a.out, (r0 + r) * a.d + 8 * c, o);
      }
    }
  }
  if (a.part) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = j * T + (int)threadIdx.x;
      if (c < nck) store8<MMF_F32>(a.part, (int64_t)blockIdx.x * a.d + 8 * c, dw[j]);
    }
  }
}

// Any width and alignment: single columns, thread t's at t + j * kGenThreads. NC > 0: rows of up to NC *
// kGenThreads columns, a thread's columns of a row (and its share of dw) in registers, one row at a time
// so that four to six CTAs share an SM (16384 x 2053 bf16, forward + backward: 146 us against 190 for the
// form that reads twice); NC = 0: wider rows, read twice, dw in the thread's columns of the partial row.
template <mmf_dtype DT>
__device__ __forceinline__ float at(const void* p, int64_t i) {
  return Elem<DT>::load(reinterpret_cast<const typename Elem<DT>::T*>(p) + i);
}
template <mmf_dtype DT>
__device__ __forceinline__ void put(void* p, int64_t i, float v) {
  Elem<DT>::store(reinterpret_cast<typename Elem<DT>::T*>(p) + i, v);
}
template <mmf_dtype XT, mmf_dtype YT, int NC>
__global__ void __launch_bounds__(kGenThreads, NC > 0 ? 6 : 1) rms_fwd_any_kernel(const Args a) {
  dependent();
  __shared__ float red[2][1][16];
  const int tid = threadIdx.x;
  const float inv_d = 1.0f / (float)a.d;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x, turn ^= 1) {
    float ss[1] = {0.0f}, x[NC > 0 ? NC : 1];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = tid + j * kGenThreads;
      x[j] = c < a.d ? at<XT>(a.x, r * a.d + c) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) ss[0] = fmaf(x[j], x[j], ss[0]);
    if (NC == 0)
      for (int c = tid; c < a.d; c += kGenThreads) {
        const float v = at<XT>(a.x, r * a.d + c);
        ss[0] = fmaf(v, v, ss[0]);
      }
    block_sums<1>(ss, red[turn]);
    const float rho = rsqrtf(ss[0] * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = tid + j * kGenThreads;
      if (c < a.d) put<YT>(a.out, r * a.d + c, x[j] * rho * (a.w ? a.w[c] : 1.0f));
    }
    if (NC == 0)
      for (int c = tid; c < a.d; c += kGenThreads)
        put<YT>(a.out, r * a.d + c, at<XT>(a.x, r * a.d + c) * rho * (a.w ? a.w[c] : 1.0f));
  }
}
template <mmf_dtype XT, mmf_dtype GT, int NC>
__global__ void __launch_bounds__(kGenThreads, NC > 9 ? 4 : NC > 0 ? 5 : 1) rms_bwd_any_kernel(const Args a) {
  dependent();
  __shared__ float red[2][2][16];
  const int tid = threadIdx.x;
  float* part = a.part ? a.part + (int64_t)blockIdx.x * a.d : nullptr;
  float dw[NC > 0 ? NC : 1];
#pragma unroll
  for (int j = 0; j < NC; ++j) dw[j] = 0.0f;
  if (NC == 0 && part)
    for (int c = tid; c < a.d; c += kGenThreads) part[c] = 0.0f;  // each thread only touches its own columns
  const float inv_d = 1.0f / (float)a.d;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x, turn ^= 1) {
    float s[2] = {0.0f, 0.0f}, x[NC > 0 ? NC : 1], g[NC > 0 ? NC : 1];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = tid + j * kGenThreads;
      x[j] = c < a.d ? at<XT>(a.x, r * a.d + c) : 0.0f;
      g[j] = c < a.d ? at<GT>(a.dy, r * a.d + c) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = tid + j * kGenThreads;
      s[0] = fmaf(x[j], x[j], s[0]);
      s[1] = fmaf(g[j] * (a.w && c < a.d ? a.w[c] : 1.0f), x[j], s[1]);
    }
    if (NC == 0)
      for (int c = tid; c < a.d; c += kGenThreads) {
        const float v = at<XT>(a.x, r * a.d + c);
        const float u = at<GT>(a.dy, r * a.d + c) * (a.w ? a.w[c] : 1.0f);
        s[0] = fmaf(v, v, s[0]);
        s[1] = fmaf(u, v, s[1]);
      }
    block_sums<2>(s, red[turn]);
    const float rho = rsqrtf(s[0] * inv_d + a.eps);
    const float k = rho * (rho * (s[1] * inv_d));
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = tid + j * kGenThreads;
      const float xh = __fmul_rn(x[j], rho);
      dw[j] = fmaf(g[j], xh, dw[j]);
      if (c < a.d) put<XT>(a.out, r * a.d + c, grad(rho, g[j] * (a.w ? a.w[c] : 1.0f), k, xh));
    }
    if (NC == 0)
      for (int c = tid; c < a.d; c += kGenThreads) {
        const float xh = __fmul_rn(at<XT>(a.x, r * a.d + c), rho), gv = at<GT>(a.dy, r * a.d + c);
        if (part) part[c] = fmaf(gv, xh, part[c]);
        put<XT>(a.out, r * a.d + c, grad(rho, gv * (a.w ? a.w[c] : 1.0f), k, xh));
      }
  }
  if (part) {
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (tid + j * kGenThreads < a.d) part[tid + j * kGenThreads] = dw[j];
  }
}

// dw[c] = sum over the partial rows, in a fixed order: 32 columns x 32 lanes per CTA.
__global__ void __launch_bounds__(1024) rms_dw_kernel(const float* __restrict__ part, int rows, int d, float* __restrict__ dw) {
  dependent();
  __shared__ float red[32][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, c = blockIdx.x * 32 + tx;
  float s = 0.0f;
  if (c < d)
    for (int r = ty; r < rows; r += 32) s += part[(int64_t)r * d + c];
  red[ty][tx] = s;
  __syncthreads();
  const float v = warp_sum(red[tx][ty]);
  if (tx == 0 && blockIdx.x * 32 + ty < d) dw[blockIdx.x * 32 + ty] = v;
}

}  // namespace rms
}  // namespace mmf
