// tg_qk_norm_rope: RMS norm of every query and key head and the rotary embedding in
// one pass, and its backward. Per token t and head (x is one head's dh elements, w the
// norm's weight for queries or for keys):
//     r = 1 / sqrt(mean(x^2) + eps),   n = w * x * r,   y = R(pos[t]) n,
// R the rotation of the pairs (i, i + rot/2), i < rot/2, by pos * theta_i,
// theta_i = base^(-2i/rot); elements from rot on are not rotated. Backward, from dy:
//     g = R(-pos) dy,   dw = sum_{t,h} g x r,   dx = r (w g - x r^2 mean(w g x)).
//
// Both are bound by memory: each element is read and written once (16-bit: 4 bytes
// forward, 6 backward). A warp takes a token (or, for few tokens, part of its heads),
// so the angles are formed once per token, a part by each of the heads that are side by side,
// and serve every head: lane c of a head holds E pairs from E c on (elements E c .. and
// rot/2 + E c ..; E = 8 or 4), so a rotation needs no exchange between lanes, and the mean
// is a few shuffles. 16384 tokens of 24 bf16 heads of 128 take 39.7 us (5.1 TB/s, 77% of a
// plain copy's rate), backward over 10721 tokens 46.8 us (4.2 TB/s): what is left is
// latency at 20 and 12 warps an SM (issue slots 47% and 39% busy, DRAM 48% and 44%). fp32:
// 8192 tokens 36.2 us (5.6 TB/s), backward over 5000 tokens 40.0 us (4.6 TB/s).
//
// The weight gradients are summed in fp32: a lane's chain is its warp's tokens times the
// heads that its lane group takes (10721 tokens of 16 heads of 128: 24 to 28 terms), then come
// lane groups, warps and blocks, so the error grows with tokens x heads / 1776 warps.
//
// The angle of position p and frequency i is taken in turns, p * F_i mod 1 with F_i =
// theta_i / (2 pi) as a 64-bit fixed-point fraction (an integer product, exact modulo
// one turn). The nearest quarter turn is split off in integers, which leaves an angle
// of at most an eighth of a turn: as a float it is off by 2^-24 relatively, so by at
// most 2^-24 * pi/4 in radians, and the quarter turns are exact sign changes.
#include "common.cuh"

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxDh = 256;

struct NormRopeArgs {
  const void *q, *k;              // inputs
  const void *gq, *gk;            // backward: upstream gradients
  void *oq, *ok;                  // outputs (forward) or input gradients (backward)
  int64_t q_st, k_st, gq_st, gk_st, oq_st, ok_st;   // elements from token to token
  const float *wq, *wk;
  const int32_t* pos;
  int64_t n_tokens;
  int n_hq, n_hkv, dh, rot;
  float eps;
  double ratio;                   // base^(-2/rot)
  int parts;                      // warps that share one token
  float* partial;                 // backward: [gridDim.x][2][dh] sums of g x r
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// N elements of type T as N / 2 pairs of floats.
template <typename T, int N>
struct Io;
template <>
struct Io<__nv_bfloat16, 8> {
  using Vec = uint4;
  static __device__ __forceinline__ void unpack(const Vec& v, float2* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ Vec pack(const float2* f) {
    return make_uint4(tg::pack_bf16x2(f[0].x, f[0].y), tg::pack_bf16x2(f[1].x, f[1].y),
                      tg::pack_bf16x2(f[2].x, f[2].y), tg::pack_bf16x2(f[3].x, f[3].y));
  }
};
template <>
struct Io<__nv_bfloat16, 4> {
  using Vec = uint2;
  static __device__ __forceinline__ void unpack(const Vec& v, float2* f) {
    f[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
    f[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
  }
  static __device__ __forceinline__ Vec pack(const float2* f) {
    return make_uint2(tg::pack_bf16x2(f[0].x, f[0].y), tg::pack_bf16x2(f[1].x, f[1].y));
  }
};
template <>
struct Io<float, 4> {
  using Vec = float4;
  static __device__ __forceinline__ void unpack(const Vec& v, float2* f) {
    f[0] = make_float2(v.x, v.y);
    f[1] = make_float2(v.z, v.w);
  }
  static __device__ __forceinline__ Vec pack(const float2* f) { return make_float4(f[0].x, f[0].y, f[1].x, f[1].y); }
};

// Frequencies F_i = ratio^i / (2 pi) in turns, 0.64 fixed point, i = i0 .. i0 + N - 1 (i0 < 128).
template <int N>
__device__ __forceinline__ void turns_from(double ratio, int i0, uint64_t* f) {
  double t = 0.15915494309189535, p = ratio;
#pragma unroll
  for (int b = 0; b < 7; ++b) {
    if ((i0 >> b) & 1) t *= p;
    p *= p;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    f[j] = __double2ull_rn(t * 18446744073709551616.0);
    t *= ratio;
  }
}

// Sine and cosine of position pos times a turn fraction. kFull: to fp32; otherwise by MUFU,
// off by about 2^-21, which moves a rotated element by 2^-20 of its pair's size at most: far
// below half a bf16 step of the larger one, more than that of one that nearly cancels.
template <bool kFull>
__device__ __forceinline__ void angle(int64_t pos, uint64_t turn, float* sn, float* cs) {
  const uint64_t fx = static_cast<uint64_t>(pos) * turn;
  const uint32_t hi = static_cast<uint32_t>((fx + (1ull << 31)) >> 32);   // 2^-32 of a turn
  const uint32_t quarter = (hi + (1u << 29)) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) * 0x1p-31f;   // half turns
  float s, c;
  if constexpr (kFull) sincospif(x, &s, &c);
  else __sincosf(x * 3.14159265358979f, &s, &c);
  const bool odd = quarter & 1;
  const float a = odd ? c : s, b = odd ? s : c;
  *sn = (quarter & 2) ? -a : a;
  *cs = ((quarter + 1) & 2) ? -b : b;
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// E: elements of a lane in either half of its pairs, LPH lanes per head (at least dh / (2 E)).
// kU heads of each lane group are in flight at once.
template <typename T, int E, int LPH, bool kBwd>
__global__ void __launch_bounds__(kThreads, kBwd ? 3 : 5) norm_rope_kernel(const NormRopeArgs A) {
  using IO = Io<T, E>;
  using Vec = typename IO::Vec;
  constexpr int kP = E / 2;
  constexpr int kHpw = 32 / LPH;   // heads a warp handles side by side
  constexpr int kU = 2;
  constexpr int kNa = E / kHpw;    // angles that a lane forms
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane % LPH, sub = lane / LPH;
  const int nc = A.dh / (2 * E), nr = A.rot / (2 * E);
  const bool active = c < nc, turns = c < nr;
  const int offa = !active ? 0 : turns ? E * c : A.rot + 2 * E * (c - nr);
  const int offb = !active ? 0 : turns ? A.rot / 2 + E * c : offa + E;
  uint64_t freq[kNa];
  turns_from<kNa>(A.ratio, turns ? E * c + kNa * sub : 0, freq);
  tg::pdl_launch_dependents();
  tg::pdl_wait();   // global memory only from here on

  // the weights, [0] queries, [1] keys; zeros for lanes without elements
  __shared__ __align__(16) float sw[2][kMaxDh];
  for (int i = tid; i < 2 * kMaxDh; i += kThreads) {
    const int d = i & (kMaxDh - 1);
    sw[i / kMaxDh][d] = d < A.dh ? (i < kMaxDh ? A.wq : A.wk)[d] : 0.f;
  }
  __syncthreads();
  float2 dwa[2][kBwd ? kP : 1] = {}, dwb[2][kBwd ? kP : 1] = {};
  const float inv_dh = 1.f / static_cast<float>(A.dh);
  const int64_t n_work = A.n_tokens * A.parts;
#pragma unroll 1
  for (int64_t wk = static_cast<int64_t>(blockIdx.x) * kWarps + warp; wk < n_work;
       wk += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t t = A.parts == 1 ? wk : wk / A.parts;
    const int part = static_cast<int>(wk - t * A.parts);
    const int64_t p = A.pos[t];
    // The heads side by side need the same angles: each forms a part of them.
    float s_own[kNa], c_own[kNa];
#pragma unroll
    for (int j = 0; j < kNa; ++j) {
      s_own[j] = 0.f, c_own[j] = 1.f;
      if (turns) angle<sizeof(T) == 4>(p, freq[j], &s_own[j], &c_own[j]);
    }
    __syncwarp();
    float2 sn[kP], cs[kP];
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float s = __shfl_sync(0xFFFFFFFFu, s_own[j % kNa], c + LPH * (j / kNa));
      const float k = __shfl_sync(0xFFFFFFFFu, c_own[j % kNa], c + LPH * (j / kNa));
      if (j & 1) sn[j / 2].y = s, cs[j / 2].y = k;
      else sn[j / 2].x = s, cs[j / 2].x = k;
    }
#pragma unroll
    for (int key = 0; key < 2; ++key) {   // queries, then keys
      const int heads = key ? A.n_hkv : A.n_hq;
      const T* x0 = static_cast<const T*>(key ? A.k : A.q) + t * (key ? A.k_st : A.q_st);
      const T* g0 = static_cast<const T*>(key ? A.gk : A.gq) + t * (key ? A.gk_st : A.gq_st);
      T* y0 = static_cast<T*>(key ? A.ok : A.oq) + t * (key ? A.ok_st : A.oq_st);
      // forward: y_a = r (x_a w_a cos - x_b w_b sin), y_b = r (x_b w_b cos + x_a w_a sin), with
      // the products of weight and angle formed once for all heads
      float2 wa[kP], wb[kP];
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        wa[j] = *reinterpret_cast<const float2*>(&sw[key][offa + 2 * j]);
        wb[j] = *reinterpret_cast<const float2*>(&sw[key][offb + 2 * j]);
      }
      float2 ca[kP], sb[kP], cb[kP], sa[kP];
      if constexpr (!kBwd) {
#pragma unroll
        for (int j = 0; j < kP; ++j) {
          ca[j] = mul2(wa[j], cs[j]);
          sa[j] = mul2(wa[j], sn[j]);
          cb[j] = mul2(wb[j], cs[j]);
          sb[j] = mul2(wb[j], make_float2(-sn[j].x, -sn[j].y));
        }
      }
      // heads part*kHpw + sub, then every parts*kHpw-th
      const int step = A.parts * kHpw;
#pragma unroll 1
      for (int h0 = part * kHpw + sub; h0 - sub < heads; h0 += kU * step) {
        Vec va[kU], vb[kU], ga[kBwd ? kU : 1], gb[kBwd ? kU : 1];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int h = h0 + u * step;
          va[u] = vb[u] = Vec{};
          if constexpr (kBwd) ga[u] = gb[u] = Vec{};
          if (h < heads && active) {
            va[u] = *reinterpret_cast<const Vec*>(x0 + h * A.dh + offa);
            vb[u] = *reinterpret_cast<const Vec*>(x0 + h * A.dh + offb);
            if constexpr (kBwd) {
              ga[u] = *reinterpret_cast<const Vec*>(g0 + h * A.dh + offa);
              gb[u] = *reinterpret_cast<const Vec*>(g0 + h * A.dh + offb);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int h = h0 + u * step;
          float2 xa[kP], xb[kP], ya[kP], yb[kP], ss = {};
          IO::unpack(va[u], xa);
          IO::unpack(vb[u], xb);
#pragma unroll
          for (int j = 0; j < kP; ++j) ss = fma2(xa[j], xa[j], fma2(xb[j], xb[j], ss));
          float r = __frsqrt_rn(fmaf(head_sum<LPH>(ss.x + ss.y), inv_dh, A.eps));
          // A head that is not there has r = 0, not 1 / sqrt(eps): infinite without an epsilon, that
          // times its zeros would be NaN in the weight gradients' sums.
          if (kBwd && h >= heads) r = 0.f;
          if constexpr (!kBwd) {
#pragma unroll
            for (int j = 0; j < kP; ++j) {
              ya[j] = mul2(both(r), fma2(xb[j], sb[j], mul2(xa[j], ca[j])));
              yb[j] = mul2(both(r), fma2(xa[j], sa[j], mul2(xb[j], cb[j])));
            }
          } else {
            float2 da[kP], db[kP], m2 = {};
            IO::unpack(ga[u], da);
            IO::unpack(gb[u], db);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
              const float2 ua = fma2(da[j], cs[j], mul2(db[j], sn[j]));
              const float2 ub = fma2(db[j], cs[j], mul2(da[j], make_float2(-sn[j].x, -sn[j].y)));
              xa[j] = mul2(xa[j], both(r));
              xb[j] = mul2(xb[j], both(r));
              dwa[key][j] = fma2(ua, xa[j], dwa[key][j]);
              dwb[key][j] = fma2(ub, xb[j], dwb[key][j]);
              da[j] = mul2(ua, wa[j]);
              db[j] = mul2(ub, wb[j]);
              m2 = fma2(da[j], xa[j], fma2(db[j], xb[j], m2));
            }
            const float m = head_sum<LPH>(m2.x + m2.y) * -inv_dh;
#pragma unroll
            for (int j = 0; j < kP; ++j) {
              ya[j] = mul2(both(r), fma2(xa[j], both(m), da[j]));
              yb[j] = mul2(both(r), fma2(xb[j], both(m), db[j]));
            }
          }
          if (h < heads && active) {
            *reinterpret_cast<Vec*>(y0 + h * A.dh + offa) = IO::pack(ya);
            *reinterpret_cast<Vec*>(y0 + h * A.dh + offb) = IO::pack(yb);
          }
        }
      }
    }
  }
  if constexpr (kBwd) {
    // the block's sums, added in a fixed order: lane groups, then warps
    __shared__ float sums[kWarps][2][kMaxDh];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int j = 0; j < kP; ++j) {
        float v[4] = {dwa[e][j].x, dwa[e][j].y, dwb[e][j].x, dwb[e][j].y};
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int o = LPH; o < 32; o <<= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
        if (sub == 0 && active) {
          sums[warp][e][offa + 2 * j] = v[0];
          sums[warp][e][offa + 2 * j + 1] = v[1];
          sums[warp][e][offb + 2 * j] = v[2];
          sums[warp][e][offb + 2 * j + 1] = v[3];
        }
      }
    __syncthreads();
    for (int i = tid; i < 2 * A.dh; i += kThreads) {
      const int e = i / A.dh, d = i - e * A.dh;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += sums[w][e][d];
      A.partial[static_cast<int64_t>(blockIdx.x) * 2 * A.dh + i] = s;
    }
  }
}

// dw[i] = sum over the blocks' partials, in a fixed order: 32 columns a block, 32 rows
// of threads over the partials, then a tree over those.
__global__ void __launch_bounds__(1024)
    norm_dw_kernel(const float* __restrict__ partial, int n_part, int dh, float* __restrict__ dwq,
                   float* __restrict__ dwk) {
  __shared__ float acc[32][33];
  tg::pdl_launch_dependents();
  tg::pdl_wait();
  const int col = blockIdx.x * 32 + threadIdx.x, n = 2 * dh;
  float s = 0.f;
  if (col < n)
    for (int r = threadIdx.y; r < n_part; r += 32) s += partial[static_cast<int64_t>(r) * n + col];
  acc[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = acc[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < n) (out < dh ? dwq[out] : dwk[out - dh]) = s;
}

// Blocks of a launch: as many as the SMs hold, walking the tokens: forward five (two heads in
// flight; 16384 tokens of 24 heads of 128: 40.0 us, 41.4 with four blocks, 41.8 with six, 44.3
// with three heads in flight), backward three (10721 tokens: 46.8 us, 49.9 with four), whose
// sums then are few.
int most_blocks(bool bwd) { return 148 * (bwd ? 3 : 5); }

// Whether lanes take eight elements of either half (16-byte loads of bf16): the halves of
// the rotated part and the rest must be made of whole such pieces. 16384 tokens of 24 heads
// of 128: 56 us with four, 42 us with eight (backward, 10721 tokens: 69 and 49 us; both
// before the angles were shared).
bool wide_lanes(tg_dtype dtype, int dh, int rot) { return dtype == TG_BF16 && dh % 16 == 0 && rot % 16 == 0; }

// Warps per token: one, unless there are too few tokens to fill the machine.
int warps_per_token(int64_t n_tokens, int heads, int lanes, bool bwd) {
  const int hpw = 32 / lanes, most = (heads + hpw - 1) / hpw;
  int64_t p = most_blocks(bwd) * static_cast<int64_t>(kWarps) / (n_tokens > 0 ? n_tokens : 1);
  if (p < 1) p = 1;
  return static_cast<int>(p < most ? p : most);
}
int lanes_of(int dh, int e) {
  int lanes = 8;
  while (lanes * 2 * e < dh) lanes *= 2;
  return lanes;
}
int n_blocks(int64_t n_tokens, int parts, bool bwd) {
  const int64_t b = (n_tokens * parts + kWarps - 1) / kWarps, most = most_blocks(bwd);
  return static_cast<int>(b < most ? b : most);
}

template <typename T, int E, bool kBwd>
tg_status launch_lanes(const NormRopeArgs& a, int lanes, int blocks, cudaStream_t st) {
  const dim3 g(blocks), b(kThreads);
  if (lanes == 8) return tg::launch(norm_rope_kernel<T, E, 8, kBwd>, g, b, 0, st, 0, a);
  if (lanes == 16) return tg::launch(norm_rope_kernel<T, E, 16, kBwd>, g, b, 0, st, 0, a);
  if constexpr (E == 4) return tg::launch(norm_rope_kernel<T, E, 32, kBwd>, g, b, 0, st, 0, a);
  return TG_ERR_UNSUPPORTED;   // not reached: 16 lanes of 16 elements hold the widest head
}

// Fills in what follows from the sizes and launches.
template <bool kBwd>
tg_status launch_norm(NormRopeArgs a, tg_dtype dtype, float rope_base, int* blocks, cudaStream_t st) {
  const bool wide = wide_lanes(dtype, a.dh, a.rot);
  const int lanes = lanes_of(a.dh, wide ? 8 : 4);
  a.ratio = a.rot ? exp(-2.0 / a.rot * log(static_cast<double>(rope_base))) : 0.0;
  a.parts = warps_per_token(a.n_tokens, a.n_hq, lanes, kBwd);
  *blocks = n_blocks(a.n_tokens, a.parts, kBwd);
  if (dtype == TG_F32) return launch_lanes<float, 4, kBwd>(a, lanes, *blocks, st);
  return wide ? launch_lanes<__nv_bfloat16, 8, kBwd>(a, lanes, *blocks, st)
              : launch_lanes<__nv_bfloat16, 4, kBwd>(a, lanes, *blocks, st);
}

// What both directions ask of their arguments; es is the element size.
tg_status check_norm(tg_dtype dtype, int64_t n_tokens, int n_hq, int n_hkv, int head_dim,
                     int rot_dim, float eps, float rope_base, int* es) {
  if (n_tokens < 0 || n_hq <= 0 || n_hkv <= 0 || head_dim <= 0 || rot_dim < 0 ||
      rot_dim > head_dim || !(eps >= 0.f) || !(rope_base > 1.f) || !(rope_base < 3.4e38f))
    return TG_ERR_INVALID_ARG;
  if (dtype != TG_BF16 && dtype != TG_F32) return TG_ERR_UNSUPPORTED;
  if (head_dim % 8 || head_dim < 8 || head_dim > kMaxDh || rot_dim % 8 || n_hq > 4096 || n_hkv > 4096)
    return TG_ERR_UNSUPPORTED;
  *es = dtype == TG_BF16 ? 2 : 4;
  return TG_OK;
}

bool bad_stride(int64_t st, int heads, int dh) { return st < static_cast<int64_t>(heads) * dh; }

}  // namespace

extern "C" tg_status tg_qk_norm_rope(const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, tg_dtype dtype, int64_t n_tokens, int n_hq,
                                     int n_hkv, int head_dim, int rot_dim, const float* q_weight,
                                     const float* k_weight, float eps, float rope_base,
                                     const int32_t* pos, void* q_out, int64_t q_out_stride,
                                     void* k_out, int64_t k_out_stride, tg_stream_t stream) {
  tg::NvtxRange nvtx_range("tg_qk_norm_rope");
  int es = 0;
  const tg_status bad = check_norm(dtype, n_tokens, n_hq, n_hkv, head_dim, rot_dim, eps, rope_base, &es);
  if (bad != TG_OK) return bad;
  if (n_tokens == 0) return TG_OK;
  if (!q || !k || !q_weight || !k_weight || !pos || !q_out || !k_out) return TG_ERR_INVALID_ARG;
  if (bad_stride(q_stride, n_hq, head_dim) || bad_stride(k_stride, n_hkv, head_dim) ||
      bad_stride(q_out_stride, n_hq, head_dim) || bad_stride(k_out_stride, n_hkv, head_dim))
    return TG_ERR_INVALID_ARG;
  if (!tg::aligned16(q) || !tg::aligned16(k) || !tg::aligned16(q_out) || !tg::aligned16(k_out) ||
      ((q_stride | k_stride | q_out_stride | k_out_stride) * es) % 16)
    return TG_ERR_MISALIGNED;
  NormRopeArgs a = {};
  a.q = q, a.k = k, a.oq = q_out, a.ok = k_out;
  a.q_st = q_stride, a.k_st = k_stride, a.oq_st = q_out_stride, a.ok_st = k_out_stride;
  a.wq = q_weight, a.wk = k_weight, a.pos = pos;
  a.n_tokens = n_tokens, a.n_hq = n_hq, a.n_hkv = n_hkv, a.dh = head_dim, a.rot = rot_dim;
  a.eps = eps;
  int blocks;
  return launch_norm<false>(a, dtype, rope_base, &blocks, stream);
}

extern "C" size_t tg_qk_norm_rope_bwd_workspace_size(int64_t n_tokens, int n_hq, int n_hkv,
                                                     int head_dim) {
  if (n_tokens <= 0 || n_hq <= 0 || n_hkv <= 0 || head_dim <= 0 || head_dim > kMaxDh) return 0;
  // the most blocks that either type and any rotation takes
  const int64_t warps = n_tokens * (static_cast<int64_t>(n_hq) + n_hkv);
  const int64_t b = (warps + kWarps - 1) / kWarps, most = most_blocks(true);
  return static_cast<size_t>(b < most ? b : most) * 2 * head_dim * sizeof(float);
}

extern "C" tg_status tg_qk_norm_rope_bwd(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* dq_out,
    int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride, tg_dtype dtype,
    int64_t n_tokens, int n_hq, int n_hkv, int head_dim, int rot_dim, const float* q_weight,
    const float* k_weight, float eps, float rope_base, const int32_t* pos, void* dq,
    int64_t dq_stride, void* dk, int64_t dk_stride, float* dq_weight, float* dk_weight,
    void* workspace, size_t workspace_bytes, tg_stream_t stream) {
  tg::NvtxRange nvtx_range("tg_qk_norm_rope_bwd");
  int es = 0;
  const tg_status bad = check_norm(dtype, n_tokens, n_hq, n_hkv, head_dim, rot_dim, eps, rope_base, &es);
  if (bad != TG_OK) return bad;
  if (!dq_weight || !dk_weight) return TG_ERR_INVALID_ARG;
  if (n_tokens > 0) {
    if (!q || !k || !dq_out || !dk_out || !q_weight || !k_weight || !pos || !dq || !dk)
      return TG_ERR_INVALID_ARG;
    if (bad_stride(q_stride, n_hq, head_dim) || bad_stride(k_stride, n_hkv, head_dim) ||
        bad_stride(dq_out_stride, n_hq, head_dim) || bad_stride(dk_out_stride, n_hkv, head_dim) ||
        bad_stride(dq_stride, n_hq, head_dim) || bad_stride(dk_stride, n_hkv, head_dim))
      return TG_ERR_INVALID_ARG;
    if (!tg::aligned16(q) || !tg::aligned16(k) || !tg::aligned16(dq_out) || !tg::aligned16(dk_out) ||
        !tg::aligned16(dq) || !tg::aligned16(dk) ||
        ((q_stride | k_stride | dq_out_stride | dk_out_stride | dq_stride | dk_stride) * es) % 16)
      return TG_ERR_MISALIGNED;
  }
  const size_t need = tg_qk_norm_rope_bwd_workspace_size(n_tokens, n_hq, n_hkv, head_dim);
  if (need && (!workspace || workspace_bytes < need)) return TG_ERR_WORKSPACE;
  if (need && !tg::aligned16(workspace)) return TG_ERR_MISALIGNED;
  NormRopeArgs a = {};
  a.q = q, a.k = k, a.gq = dq_out, a.gk = dk_out, a.oq = dq, a.ok = dk;
  a.q_st = q_stride, a.k_st = k_stride, a.gq_st = dq_out_stride, a.gk_st = dk_out_stride;
  a.oq_st = dq_stride, a.ok_st = dk_stride;
  a.wq = q_weight, a.wk = k_weight, a.pos = pos;
  a.n_tokens = n_tokens, a.n_hq = n_hq, a.n_hkv = n_hkv, a.dh = head_dim, a.rot = rot_dim;
  a.eps = eps;
  a.partial = static_cast<float*>(workspace);
  int blocks = 0;
  if (n_tokens > 0) {
    const tg_status r = launch_norm<true>(a, dtype, rope_base, &blocks, stream);
    if (r != TG_OK) return r;
  }
  return tg::launch(norm_dw_kernel, dim3((2 * head_dim + 31) / 32), dim3(32, 32), 0, stream, 0,
                    static_cast<const float*>(a.partial), blocks, head_dim, dq_weight, dk_weight);
}
