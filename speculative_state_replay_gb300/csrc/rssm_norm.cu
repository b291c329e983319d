// rssm_norm.cu -- the norms around a block: the mixer's output norm with its
// silu gate, and the residual add between the norm after a block and the one
// before the next.
#include "rssm_device.cuh"

namespace rssm {
namespace {

template <typename E>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
  static __device__ __forceinline__ uint32_t from2(float, float) { return 0u; }  // (4-byte values are stored as they are)
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
  static __device__ __forceinline__ float2 to2(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }
  static __device__ __forceinline__ uint32_t from2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float to(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
  static __device__ __forceinline__ float2 to2(uint32_t w) { return h2f2(w); }
  static __device__ __forceinline__ uint32_t from2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

using pair = unsigned long long;
__device__ __forceinline__ uint32_t low(pair d) { return static_cast<uint32_t>(d); }
__device__ __forceinline__ uint32_t high(pair d) { return static_cast<uint32_t>(d >> 32); }

// VEC elements of type E, in 16-byte pieces (one element where VEC is 1): as
// they come, as floats, and back.  Activations are read once (no L1 line is
// kept for them: the weights' stay).
template <typename E, int VEC>
struct Raw {
  static constexpr int W = VEC == 1 ? 1 : VEC * static_cast<int>(sizeof(E)) / 16;
  uint4 w[W];
  // wide: p is on 32 bytes, and they are read by one instruction (lanes that
  // read 16 bytes 32 apart pass the L1 in twice as many)
  __device__ __forceinline__ void load(const E* p, bool wide = false) {
    if constexpr (VEC == 1) {
      *reinterpret_cast<E*>(w) = *p;
    } else if (W == 2 && wide) {
      pair d[4];
      asm volatile("ld.global.cs.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(d[0]), "=l"(d[1]), "=l"(d[2]), "=l"(d[3]) : "l"(p));
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = make_uint4(low(d[2 * i]), high(d[2 * i]), low(d[2 * i + 1]), high(d[2 * i + 1]));
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void floats(float (&f)[VEC]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (VEC == 1) {
      f[0] = Elem<E>::to(*reinterpret_cast<const E*>(w));
    } else if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 d = Elem<E>::to2(u[i]);
        f[2 * i] = d.x;
        f[2 * i + 1] = d.y;
      }
    }
  }
};
template <typename E, int VEC>
__device__ __forceinline__ void load_vec(const E* p, float (&f)[VEC]) {
  Raw<E, VEC> r;
  r.load(p);
  r.floats(f);
}
// weights: read by every row
template <int VEC>
__device__ __forceinline__ void load_weight(const float* p, float (&f)[VEC], bool wide = false) {
  if constexpr (VEC == 1) {
    f[0] = __ldg(p);
  } else if (VEC == 8 && wide) {
    pair d[4];
    asm("ld.global.nc.v4.b64 {%0, %1, %2, %3}, [%4];" : "=l"(d[0]), "=l"(d[1]), "=l"(d[2]), "=l"(d[3]) : "l"(p));
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = __uint_as_float(i & 1 ? high(d[i / 2 % 4]) : low(d[i / 2 % 4]));
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = w.x;
      f[i + 1] = w.y;
      f[i + 2] = w.z;
      f[i + 3] = w.w;
    }
  }
}
template <typename E, int VEC>
__device__ __forceinline__ void store_vec(E* p, const float (&f)[VEC], bool wide = false) {
  if constexpr (VEC == 1) {
    *p = Elem<E>::from(f[0]);
  } else if (VEC * sizeof(E) == 32 && wide) {
    pair d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] = static_cast<pair>(__float_as_uint(f[(2 * i + 1) % VEC])) << 32 | __float_as_uint(f[2 * i % VEC]);
    asm volatile("st.global.cs.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(d[0]), "l"(d[1]), "l"(d[2]), "l"(d[3]) : "memory");
  } else {
    constexpr int N = 16 / sizeof(E);
#pragma unroll
    for (int w = 0; w < VEC / N; ++w) {
      uint4 raw;
      uint32_t* u = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = sizeof(E) == 4 ? __float_as_uint(f[w * N + i]) : Elem<E>::from2(f[(w * N + 2 * i) % VEC], f[(w * N + 2 * i + 1) % VEC]);
      __stcs(reinterpret_cast<uint4*>(p) + w, raw);
    }
  }
}

// z / (1 + e^-z), the reciprocal by the hardware's, 2^-23 off.  2-byte values
// take its power of two as well, |z| 2^-24 and 2^-22 off: 2^-18 at z = -85, and
// below -87 it is 0, against 2^-9 or 2^-12 of the output's rounding.  fp32
// values: e^-|z| by expf, exact to 2 units whatever z, on the side where it is
// at most 1, so that gates below -87 are what they are too.
template <typename E>
__device__ __forceinline__ float silu(float z) {
  float e, r;
  if constexpr (sizeof(E) == 4) {
    e = expf(-fabsf(z));
    z = z < 0.0f ? z * e : z;
  } else {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
  }
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return z * r;
}

// Sum over a team of TEAM lanes of a warp, or over the block (TEAM 0; `sh`: 32
// floats that no earlier sum of the kernel used).
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* sh) {
  constexpr int W = TEAM == 0 ? 32 : TEAM;
#pragma unroll
  for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TEAM == 0) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < warps; ++w) v += sh[w];
  }
  return v;
}

struct GatedNormArgs {
  const void* x;
  const void* z;
  const float* w;
  void* out;
  long long x_stride, z_stride, out_stride;
  unsigned items, groups;  // groups of all rows (below 2^30), and of one
  int group, w_group;  // w_group: weights between groups (0: one set for all)
  float eps;
  int norm_first;
};

// A team of lanes (TEAM of a warp, or a block) per (row, group), the group's
// values in NV vectors a lane; IT groups one after another, their loads first
// (short groups: a lane would have two loads on their way otherwise).  NV 0:
// groups too long for that, read twice.  Where a lane has four vectors at a time
// registers are for four blocks of 256: groups of 1000 (bf16, 46 M values) take
// 44 us, 54 with two blocks.
template <typename E, int VEC, int TEAM, int NV, int IT>
__global__ void __launch_bounds__(TEAM == 0 ? 1024 : 256, NV * IT == 4 && TEAM != 0 ? 4 : 1) gated_norm_kernel(const GatedNormArgs a) {
  __shared__ float sh[32];
  pdl_wait();
  pdl_trigger();
  const int width = TEAM == 0 ? static_cast<int>(blockDim.x) : TEAM;
  constexpr int kTeams = TEAM == 0 ? 1 : 256 / TEAM;
  const unsigned first = blockIdx.x * (kTeams * IT) + (TEAM == 0 ? 0 : threadIdx.x / (TEAM ? TEAM : 1));
  const int lane = TEAM == 0 ? threadIdx.x : threadIdx.x % (TEAM ? TEAM : 1);
  const auto row_of = [&](unsigned item, unsigned& grp) {
    const unsigned row = item / a.groups;
    grp = item - row * a.groups;
    return row;
  };
  if constexpr (NV > 0) {
    Raw<E, VEC> rx[IT][NV], rz[IT][NV];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const unsigned item = first + it * kTeams;
      unsigned grp;
      const unsigned row = row_of(item < a.items ? item : 0, grp);
      const E* x = static_cast<const E*>(a.x) + row * a.x_stride + grp * a.group;
      const E* z = static_cast<const E*>(a.z) + row * a.z_stride + grp * a.group;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = (v * width + lane) * VEC;
        if (item < a.items && i < a.group) {
          rx[it][v].load(x + i);
          rz[it][v].load(z + i);
        } else {
          rx[it][v].zero();
          rz[it][v].zero();
        }
      }
    }
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const unsigned item = first + it * kTeams;
      unsigned grp;
      const unsigned row = row_of(item < a.items ? item : 0, grp);
      E* out = static_cast<E*>(a.out) + row * a.out_stride + grp * a.group;
      const float* w = a.w + grp * a.w_group;
      float fx[NV][VEC], sum = 0.0f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        rx[it][v].floats(fx[v]);
        if (!a.norm_first) {
          float fz[VEC];
          rz[it][v].floats(fz);
#pragma unroll
          for (int e = 0; e < VEC; ++e) fx[v][e] *= silu<E>(fz[e]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum = fmaf(fx[v][e], fx[v][e], sum);
      }
      sum = team_sum<TEAM>(sum, sh);
      const float r = rsqrtf(sum / a.group + a.eps);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = (v * width + lane) * VEC;
        if (item < a.items && i < a.group) {
          float fw[VEC];
          load_weight<VEC>(w + i, fw);
#pragma unroll
          for (int e = 0; e < VEC; ++e) fw[e] *= fx[v][e] * r;
          if (a.norm_first) {
            float fz[VEC];
            rz[it][v].floats(fz);
#pragma unroll
            for (int e = 0; e < VEC; ++e) fw[e] *= silu<E>(fz[e]);
          }
          store_vec<E, VEC>(out + i, fw);
        }
      }
    }
  } else {
    unsigned grp;
    const unsigned row = row_of(first, grp);
    const E* x = static_cast<const E*>(a.x) + row * a.x_stride + grp * a.group;
    const E* z = static_cast<const E*>(a.z) + row * a.z_stride + grp * a.group;
    E* out = static_cast<E*>(a.out) + row * a.out_stride + grp * a.group;
    const float* w = a.w + grp * a.w_group;
    float sum = 0.0f;
    for (int i = lane * VEC; i < a.group; i += width * VEC) {
      float fx[VEC], fz[VEC];
      load_vec<E, VEC>(x + i, fx);
      if (!a.norm_first) load_vec<E, VEC>(z + i, fz);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (!a.norm_first) fx[e] *= silu<E>(fz[e]);
        sum = fmaf(fx[e], fx[e], sum);
      }
    }
    sum = team_sum<TEAM>(sum, sh);
    const float r = rsqrtf(sum / a.group + a.eps);
    for (int i = lane * VEC; i < a.group; i += width * VEC) {
      float fx[VEC], fz[VEC], fw[VEC];
      load_vec<E, VEC>(x + i, fx);
      load_vec<E, VEC>(z + i, fz);
      load_weight<VEC>(w + i, fw);
#pragma unroll
      for (int e = 0; e < VEC; ++e) fw[e] = a.norm_first ? fx[e] * r * fw[e] * silu<E>(fz[e]) : fx[e] * silu<E>(fz[e]) * r * fw[e];
      store_vec<E, VEC>(out + i, fw);
    }
  }
}

struct ResidualNormArgs {
  const void* x;
  const void* residual;
  const float* post;
  const float* scale;
  const float* w;
  void* residual_out;
  void* out;
  long long x_stride, residual_stride, residual_out_stride, out_stride;
  unsigned rows;
  int dim;
  float alpha, eps;
  bool wide;  // fp32 rows and weights are on 32 bytes
};

// A block per row, the row's values in NV vectors a thread; NV 0: rows too long
// for that, read once per sum and once more to write.  Several small blocks an
// SM keep loads on their way while others wait for their two sums: rows of 8192
// (bf16, fp32 residual, 42 M values) take 78 us with 256 threads of 4 vectors,
// 83 with 512 of 2 and 102 with 1024 of one; 80 registers a thread are for three
// blocks of 256 (83 us with 88).  fp32 rows and weights on 32 bytes are read and
// written 32 bytes a lane, 76 us (with a post norm and a scale, 8192 rows of
// 5120, 84 us where 16 bytes a lane take 88).  Blocks that go through rows with the next
// one's loads on their way took 103 us.
constexpr int residual_regs(int vec, int nv) { return nv == 1 ? 32 : nv == 4 && vec == 8 ? 80 : 64; }
template <typename E, typename R, int VEC, int NV>
__global__ void __maxnreg__(residual_regs(VEC, NV)) residual_norm_kernel(const ResidualNormArgs a) {
  __shared__ float sh[64];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, width = blockDim.x;
  if constexpr (NV > 0) {
    const long long row = blockIdx.x;
    const E* x = static_cast<const E*>(a.x) + row * a.x_stride;
    const R* res = static_cast<const R*>(a.residual) + row * a.residual_stride;
    R* res_out = static_cast<R*>(a.residual_out) + row * a.residual_out_stride;
    E* out = static_cast<E*>(a.out) + row * a.out_stride;
    Raw<E, VEC> rx[NV];
    Raw<R, VEC> rr[NV];
    float h[NV][VEC], sum = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * width + tid) * VEC;
      if (i < a.dim) {
        rx[v].load(x + i);
        rr[v].load(res + i, a.wide);
      } else {
        rx[v].zero();
        rr[v].zero();
      }
    }
    float r = a.alpha;
    if (a.post) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float f[VEC];
        rx[v].floats(f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum = fmaf(f[e], f[e], sum);
      }
      sum = team_sum<0>(sum, sh);
      r *= rsqrtf(sum / a.dim + a.eps);
      sum = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * width + tid) * VEC;
      if (i < a.dim) {
        float f[VEC], fw[VEC];
        rx[v].floats(f);
        rr[v].floats(h[v]);
        if (a.post) {
          load_weight<VEC>(a.post + i, fw, a.wide);
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[e] *= fw[e];
        }
        if (a.scale) {
          load_weight<VEC>(a.scale + i, fw, a.wide);
#pragma unroll
          for (int e = 0; e < VEC; ++e) f[e] *= fw[e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          h[v][e] = fmaf(r, f[e], h[v][e]);
          sum = fmaf(h[v][e], h[v][e], sum);
        }
        store_vec<R, VEC>(res_out + i, h[v], a.wide);
      }
    }
    sum = team_sum<0>(sum, sh + 32);
    const float s = rsqrtf(sum / a.dim + a.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * width + tid) * VEC;
      if (i < a.dim) {
        float fw[VEC];
        load_weight<VEC>(a.w + i, fw, a.wide);
#pragma unroll
        for (int e = 0; e < VEC; ++e) fw[e] *= h[v][e] * s;
        store_vec<E, VEC>(out + i, fw);
      }
    }
  } else {
    const unsigned row = blockIdx.x;
    const E* x = static_cast<const E*>(a.x) + row * a.x_stride;
    const R* res = static_cast<const R*>(a.residual) + row * a.residual_stride;
    R* res_out = static_cast<R*>(a.residual_out) + row * a.residual_out_stride;
    E* out = static_cast<E*>(a.out) + row * a.out_stride;
    float r = a.alpha, sum = 0.0f;
    if (a.post) {
      for (int i = tid * VEC; i < a.dim; i += width * VEC) {
        float f[VEC];
        load_vec<E, VEC>(x + i, f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum = fmaf(f[e], f[e], sum);
      }
      sum = team_sum<0>(sum, sh);
      r *= rsqrtf(sum / a.dim + a.eps);
      sum = 0.0f;
    }
    const auto stream = [&](int i, float (&h)[VEC]) {
      float f[VEC], fw[VEC];
      load_vec<E, VEC>(x + i, f);
      load_vec<R, VEC>(res + i, h);
      if (a.post) {
        load_weight<VEC>(a.post + i, fw);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] *= fw[e];
      }
      if (a.scale) {
        load_weight<VEC>(a.scale + i, fw);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] *= fw[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = fmaf(r, f[e], h[e]);
    };
    for (int i = tid * VEC; i < a.dim; i += width * VEC) {
      float h[VEC];
      stream(i, h);
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum = fmaf(h[e], h[e], sum);
    }
    sum = team_sum<0>(sum, sh + 32);
    const float s = rsqrtf(sum / a.dim + a.eps);
    for (int i = tid * VEC; i < a.dim; i += width * VEC) {
      float h[VEC], fw[VEC];
      stream(i, h);
      load_weight<VEC>(a.w + i, fw);
#pragma unroll
      for (int e = 0; e < VEC; ++e) fw[e] *= h[e] * s;
      store_vec<R, VEC>(res_out + i, h);
      store_vec<E, VEC>(out + i, fw);
    }
  }
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

template <typename E, int VEC, int TEAM, int NV>
cudaError_t launch_teams(const GatedNormArgs& a, cudaStream_t st) {
  constexpr int teams = 256 / TEAM;
  // Two groups a team once one would make over three waves of blocks: 64 us
  // where one takes 71, and three 64 (524288 groups of 128, bf16).
  if (NV <= 2 && a.items >= (1u << 20) / TEAM)
    return launch_pdl(gated_norm_kernel<E, VEC, TEAM, NV, NV <= 2 ? 2 : 1>, dim3((a.items + 2 * teams - 1) / (2 * teams)), dim3(256), 0, st, a);
  return launch_pdl(gated_norm_kernel<E, VEC, TEAM, NV, 1>, dim3((a.items + teams - 1) / teams), dim3(256), 0, st, a);
}

template <typename E, int VEC>
cudaError_t launch_gated(const GatedNormArgs& a, cudaStream_t st) {
  const int vecs = (a.group + VEC - 1) / VEC;
  if (vecs <= 8) return launch_teams<E, VEC, 8, 1>(a, st);
  if (vecs <= 16) return launch_teams<E, VEC, 16, 1>(a, st);
  if (vecs <= 32) return launch_teams<E, VEC, 32, 1>(a, st);
  if (vecs <= 64) return launch_teams<E, VEC, 32, 2>(a, st);
  if (vecs <= 128) return launch_teams<E, VEC, 32, 4>(a, st);
  const dim3 grid(a.items);
  // as few threads as hold the group in 4 vectors: several blocks an SM have
  // loads on their way while one sums (5784 groups of 8192, bf16: 45 us with
  // 256 threads, 58 with 512 of 2 vectors, 97 with 1024 of one)
  if (vecs <= 4096) return launch_pdl(gated_norm_kernel<E, VEC, 0, 4, 1>, grid, dim3((vecs + 127) / 128 * 32), 0, st, a);
  return launch_pdl(gated_norm_kernel<E, VEC, 0, 0, 1>, grid, dim3(1024), 0, st, a);
}

template <typename E, typename R, int VEC>
cudaError_t launch_residual(const ResidualNormArgs& a, cudaStream_t st) {
  const int vecs = (a.dim + VEC - 1) / VEC;
  const dim3 grid(a.rows);
  // blocks of 256 threads at most, where 4 vectors a thread hold the row
  if (vecs <= 256) return launch_pdl(residual_norm_kernel<E, R, VEC, 1>, grid, dim3((vecs + 31) / 32 * 32), 0, st, a);
  if (vecs <= 512) return launch_pdl(residual_norm_kernel<E, R, VEC, 2>, grid, dim3((vecs + 63) / 64 * 32), 0, st, a);
  if (vecs <= (VEC == 8 ? 2048 : 4096))
    return launch_pdl(residual_norm_kernel<E, R, VEC, 4>, grid, dim3((vecs + 127) / 128 * 32), 0, st, a);
  return launch_pdl(residual_norm_kernel<E, R, VEC, 0>, grid, dim3(1024), 0, st, a);
}

template <typename E>
cudaError_t residual_of(const ResidualNormArgs& a, bool f32, bool vec, cudaStream_t st) {
  constexpr int V = 16 / static_cast<int>(sizeof(E));
  if (f32) return vec ? launch_residual<E, float, V>(a, st) : launch_residual<E, float, 1>(a, st);
  return vec ? launch_residual<E, E, V>(a, st) : launch_residual<E, E, 1>(a, st);
}

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" rssm_status rssm_gated_norm(const void* x, int64_t x_stride, const void* z, int64_t z_stride, int32_t dtype,
                                       const float* weight, int32_t shared_weight, int64_t rows, int32_t dim,
                                       int32_t group, float eps, int32_t norm_first, void* out, int64_t out_stride,
                                       void* stream) {
  if (rows < 0 || dim < 1 || group < 1 || dim % group || !(eps >= 0.0f)) return RSSM_ERR_INVALID_ARGUMENT;
  if ((shared_weight != 0 && shared_weight != 1) || (norm_first != 0 && norm_first != 1)) return RSSM_ERR_INVALID_ARGUMENT;
  if (dtype != RSSM_F32 && dtype != RSSM_BF16 && dtype != RSSM_F16) return RSSM_ERR_INVALID_ARGUMENT;
  if (x_stride < dim || z_stride < dim || out_stride < dim) return RSSM_ERR_INVALID_ARGUMENT;
  if (rows == 0) return RSSM_OK;
  const int esz = dtype == RSSM_F32 ? 4 : 2, V = 16 / esz;
  if (!x || !z || !out || !weight || !on4(weight) || reinterpret_cast<uintptr_t>(x) % esz ||
      reinterpret_cast<uintptr_t>(z) % esz || reinterpret_cast<uintptr_t>(out) % esz)
    return RSSM_ERR_INVALID_ARGUMENT;
  const int groups = dim / group;
  if (rows > (1ll << 30) / groups) return RSSM_ERR_UNSUPPORTED;
  GatedNormArgs a = {x, z, weight, out, x_stride, z_stride, out_stride, static_cast<unsigned>(rows * groups), static_cast<unsigned>(groups),
                     group, shared_weight ? 0 : group, eps, norm_first};
  const bool vec = on16(x) && on16(z) && on16(out) && on16(weight) && x_stride % V == 0 && z_stride % V == 0 &&
                   out_stride % V == 0 && group % V == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == RSSM_F32)
    e = vec ? launch_gated<float, 4>(a, st) : launch_gated<float, 1>(a, st);
  else if (dtype == RSSM_BF16)
    e = vec ? launch_gated<__nv_bfloat16, 8>(a, st) : launch_gated<__nv_bfloat16, 1>(a, st);
  else
    e = vec ? launch_gated<__half, 8>(a, st) : launch_gated<__half, 1>(a, st);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

extern "C" rssm_status rssm_residual_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                                          int32_t dtype, int32_t residual_dtype, const float* post_weight,
                                          const float* scale, float alpha, const float* weight, int64_t rows,
                                          int32_t dim, float eps, void* residual_out, int64_t residual_out_stride,
                                          void* out, int64_t out_stride, void* stream) {
  if (rows < 0 || dim < 1 || !(eps >= 0.0f)) return RSSM_ERR_INVALID_ARGUMENT;
  if (dtype != RSSM_F32 && dtype != RSSM_BF16 && dtype != RSSM_F16) return RSSM_ERR_INVALID_ARGUMENT;
  if (residual_dtype != RSSM_F32 && residual_dtype != dtype) return RSSM_ERR_INVALID_ARGUMENT;
  if (x_stride < dim || residual_stride < dim || residual_out_stride < dim || out_stride < dim) return RSSM_ERR_INVALID_ARGUMENT;
  if (rows == 0) return RSSM_OK;
  const int esz = dtype == RSSM_F32 ? 4 : 2, rsz = residual_dtype == RSSM_F32 ? 4 : 2, V = 16 / esz;
  if (!x || !residual || !residual_out || !out || !weight || !on4(weight) || !on4(post_weight) || !on4(scale) ||
      reinterpret_cast<uintptr_t>(x) % esz || reinterpret_cast<uintptr_t>(out) % esz ||
      reinterpret_cast<uintptr_t>(residual) % rsz || reinterpret_cast<uintptr_t>(residual_out) % rsz)
    return RSSM_ERR_INVALID_ARGUMENT;
  if (rows > 0x7fffffffll) return RSSM_ERR_UNSUPPORTED;
  ResidualNormArgs a = {x, residual, post_weight, scale, weight, residual_out, out, x_stride, residual_stride,
                        residual_out_stride, out_stride, static_cast<unsigned>(rows), dim, alpha, eps, false};
  const bool vec = on16(x) && on16(residual) && on16(residual_out) && on16(out) && on16(weight) && on16(post_weight) &&
                   on16(scale) && dim % V == 0 && x_stride % V == 0 && out_stride % V == 0 && residual_stride % V == 0 &&
                   residual_out_stride % V == 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = residual_dtype == RSSM_F32;
  a.wide = vec && on32(weight) && on32(post_weight) && on32(scale) &&
           (!f32 || (on32(residual) && on32(residual_out) && residual_stride % 8 == 0 && residual_out_stride % 8 == 0));
  const cudaError_t e = dtype == RSSM_F32    ? residual_of<float>(a, true, vec, st)
                        : dtype == RSSM_BF16 ? residual_of<__nv_bfloat16>(a, f32, vec, st)
                                             : residual_of<__half>(a, f32, vec, st);
  return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}
