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
// so the angles are formed once per token and serve every head: lane c of the dh/8
// lanes of a head holds the four pairs 4c .. 4c+3 (elements 4c.. and rot/2 + 4c..), so
// a rotation needs no exchange between lanes, and the mean is log2(dh/8) shuffles.
//
// The angle of position p and frequency i is taken in turns, p * F_i mod 1 with F_i =
// theta_i / (2 pi) as a 64-bit fixed-point fraction (an integer product, exact modulo
// one turn). The nearest quarter turn is split off in integers, which leaves an angle
// of at most an eighth of a turn: as a float it is off by 2^-24 relatively, so by at
// most 2^-24 * pi/4 in radians, and the quarter turns are exact sign changes.
#include "common.cuh"

namespace {

constexpr int kWarps = 8;
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

template <typename T>
struct Io;
template <>
struct Io<__nv_bfloat16> {
  using Vec = uint2;   // four elements
  static __device__ __forceinline__ void unpack(const Vec& v, float* f) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ Vec pack(const float* f) {
    return make_uint2(tg::pack_bf16x2(f[0], f[1]), tg::pack_bf16x2(f[2], f[3]));
  }
  // absolute error about 2^-21, far below half a bf16 step of the result
  static __device__ __forceinline__ void sincos(float half_turns, float* s, float* c) {
    __sincosf(half_turns * 3.14159265358979f, s, c);
  }
};
template <>
struct Io<float> {
  using Vec = float4;
  static __device__ __forceinline__ void unpack(const Vec& v, float* f) {
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
  static __device__ __forceinline__ Vec pack(const float* f) {
    return make_float4(f[0], f[1], f[2], f[3]);
  }
  static __device__ __forceinline__ void sincos(float half_turns, float* s, float* c) {
    sincospif(half_turns, s, c);
  }
};

// The lane's frequencies F_i = ratio^i / (2 pi) in turns, 0.64 fixed point, i = 4c + j.
__device__ __forceinline__ void lane_turns(double ratio, int c, uint64_t* f) {
  double t = 0.15915494309189535, p = (ratio * ratio) * (ratio * ratio);
#pragma unroll
  for (int b = 0; b < 5; ++b) {
    if ((c >> b) & 1) t *= p;
    p *= p;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = __double2ull_rn(t * 18446744073709551616.0);
    t *= ratio;
  }
}

template <typename T>
__device__ __forceinline__ void angle(int64_t pos, uint64_t turn, float* sn, float* cs) {
  const uint64_t fx = static_cast<uint64_t>(pos) * turn;
  const uint32_t hi = static_cast<uint32_t>((fx + (1ull << 31)) >> 32);   // 2^-32 of a turn
  const uint32_t quarter = (hi + (1u << 29)) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(hi - (quarter << 30))) * 0x1p-31f;
  float s, c;
  Io<T>::sincos(x, &s, &c);
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

// LPH lanes per head (8, 16 or 32: dh up to 64, 128 or 256); kU heads of each lane
// group are in flight at once.
template <typename T, int LPH, bool kBwd>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs A) {
  using Vec = typename Io<T>::Vec;
  constexpr int kHpw = 32 / LPH;   // heads a warp handles side by side
  constexpr int kU = kBwd ? 2 : 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = lane % LPH, sub = lane / LPH;
  const int nc = A.dh / 8, nr = A.rot / 8;
  const bool active = c < nc, turns = c < nr;
  const int offa = turns ? 4 * c : A.rot + 8 * (c - nr);
  const int offb = turns ? A.rot / 2 + 4 * c : offa + 4;
  uint64_t freq[4];
  lane_turns(A.ratio, turns ? c : 0, freq);
  tg::pdl_launch_dependents();
  tg::pdl_wait();   // global memory only from here on

  float wa[2][4], wb[2][4];   // this lane's weights, [0] queries, [1] keys
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float* w = e ? A.wk : A.wq;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      wa[e][j] = active ? w[offa + j] : 0.f;
      wb[e][j] = active ? w[offb + j] : 0.f;
    }
  }
  float dwa[2][4] = {}, dwb[2][4] = {};
  const float inv_dh = 1.f / static_cast<float>(A.dh);
  const int heads = A.n_hq + A.n_hkv;
  const int64_t n_work = A.n_tokens * A.parts;
  for (int64_t wk = static_cast<int64_t>(blockIdx.x) * kWarps + warp; wk < n_work;
       wk += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t t = wk / A.parts;
    const int part = static_cast<int>(wk - t * A.parts);
    const int64_t p = A.pos[t];
    float sn[4], cs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (turns) angle<T>(p, freq[j], &sn[j], &cs[j]);
      else sn[j] = 0.f, cs[j] = 1.f;
    }
    // heads part*kHpw + sub, then every parts*kHpw-th
    const int step = A.parts * kHpw;
    for (int h0 = part * kHpw + sub; h0 - sub < heads; h0 += kU * step) {
      Vec va[kU], vb[kU], ga[kBwd ? kU : 1], gb[kBwd ? kU : 1];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step;
        if (h < heads && active) {
          const bool key = h >= A.n_hq;
          const T* x = key ? static_cast<const T*>(A.k) + t * A.k_st + (h - A.n_hq) * A.dh
                           : static_cast<const T*>(A.q) + t * A.q_st + h * A.dh;
          va[u] = *reinterpret_cast<const Vec*>(x + offa);
          vb[u] = *reinterpret_cast<const Vec*>(x + offb);
          if constexpr (kBwd) {
            const T* g = key ? static_cast<const T*>(A.gk) + t * A.gk_st + (h - A.n_hq) * A.dh
                             : static_cast<const T*>(A.gq) + t * A.gq_st + h * A.dh;
            ga[u] = *reinterpret_cast<const Vec*>(g + offa);
            gb[u] = *reinterpret_cast<const Vec*>(g + offb);
          }
        } else {
          va[u] = Vec{}, vb[u] = Vec{};
          if constexpr (kBwd) ga[u] = Vec{}, gb[u] = Vec{};
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step;
        const bool key = h >= A.n_hq;
        float xa[4], xb[4], ya[4], yb[4];
        Io<T>::unpack(va[u], xa);
        Io<T>::unpack(vb[u], xb);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], ss));
        const float r = __frsqrt_rn(fmaf(head_sum<LPH>(ss), inv_dh, A.eps));
        if constexpr (!kBwd) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float na = xa[j] * r * (key ? wa[1][j] : wa[0][j]);
            const float nb = xb[j] * r * (key ? wb[1][j] : wb[0][j]);
            ya[j] = fmaf(na, cs[j], -nb * sn[j]);
            yb[j] = fmaf(nb, cs[j], na * sn[j]);
          }
        } else {
          float da[4], db[4], m = 0.f;
          Io<T>::unpack(ga[u], da);
          Io<T>::unpack(gb[u], db);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float ua = fmaf(da[j], cs[j], db[j] * sn[j]);
            const float ub = fmaf(db[j], cs[j], -da[j] * sn[j]);
            xa[j] *= r;
            xb[j] *= r;
            if (key) {
              dwa[1][j] = fmaf(ua, xa[j], dwa[1][j]);
              dwb[1][j] = fmaf(ub, xb[j], dwb[1][j]);
            } else {
              dwa[0][j] = fmaf(ua, xa[j], dwa[0][j]);
              dwb[0][j] = fmaf(ub, xb[j], dwb[0][j]);
            }
            da[j] = ua * (key ? wa[1][j] : wa[0][j]);
            db[j] = ub * (key ? wb[1][j] : wb[0][j]);
            m = fmaf(da[j], xa[j], fmaf(db[j], xb[j], m));
          }
          m = head_sum<LPH>(m) * inv_dh;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            ya[j] = r * fmaf(-xa[j], m, da[j]);
            yb[j] = r * fmaf(-xb[j], m, db[j]);
          }
        }
        if (h < heads && active) {
          T* y = key ? static_cast<T*>(A.ok) + t * A.ok_st + (h - A.n_hq) * A.dh
                     : static_cast<T*>(A.oq) + t * A.oq_st + h * A.dh;
          *reinterpret_cast<Vec*>(y + offa) = Io<T>::pack(ya);
          *reinterpret_cast<Vec*>(y + offb) = Io<T>::pack(yb);
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
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int o = LPH; o < 32; o <<= 1) {
          dwa[e][j] += __shfl_xor_sync(0xFFFFFFFFu, dwa[e][j], o);
          dwb[e][j] += __shfl_xor_sync(0xFFFFFFFFu, dwb[e][j], o);
        }
        if (sub == 0 && active) {
          sums[warp][e][offa + j] = dwa[e][j];
          sums[warp][e][offb + j] = dwb[e][j];
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

constexpr int kMaxBlocks = 148 * 4;   // blocks of a launch: four per SM

int n_blocks(int64_t n_tokens, int parts) {
  const int64_t b = (n_tokens * parts + kWarps - 1) / kWarps;
  return static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
}

// Warps per token: one, unless there are too few tokens to fill the machine.
int warps_per_token(int64_t n_tokens, int heads, int dh) {
  const int hpw = dh <= 64 ? 4 : dh <= 128 ? 2 : 1;
  const int most = (heads + hpw - 1) / hpw;
  int64_t p = kMaxBlocks * static_cast<int64_t>(kWarps) / (n_tokens > 0 ? n_tokens : 1);
  if (p < 1) p = 1;
  return static_cast<int>(p < most ? p : most);
}

template <typename T, bool kBwd>
tg_status launch_norm(const NormRopeArgs& a, int blocks, cudaStream_t st) {
  if (a.dh <= 64)
    return tg::launch(norm_rope_kernel<T, 8, kBwd>, dim3(blocks), dim3(kThreads), 0, st, 0, a);
  if (a.dh <= 128)
    return tg::launch(norm_rope_kernel<T, 16, kBwd>, dim3(blocks), dim3(kThreads), 0, st, 0, a);
  return tg::launch(norm_rope_kernel<T, 32, kBwd>, dim3(blocks), dim3(kThreads), 0, st, 0, a);
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
  a.ratio = rot_dim ? exp(-2.0 / rot_dim * log(static_cast<double>(rope_base))) : 0.0;
  a.parts = warps_per_token(n_tokens, n_hq + n_hkv, head_dim);
  const int blocks = n_blocks(n_tokens, a.parts);
  return dtype == TG_BF16 ? launch_norm<__nv_bfloat16, false>(a, blocks, stream)
                          : launch_norm<float, false>(a, blocks, stream);
}

extern "C" size_t tg_qk_norm_rope_bwd_workspace_size(int64_t n_tokens, int n_hq, int n_hkv,
                                                     int head_dim) {
  if (n_tokens <= 0 || n_hq <= 0 || n_hkv <= 0 || head_dim <= 0 || head_dim > kMaxDh) return 0;
  return static_cast<size_t>(n_blocks(n_tokens, warps_per_token(n_tokens, n_hq + n_hkv, head_dim))) *
         2 * head_dim * sizeof(float);
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
  a.ratio = rot_dim ? exp(-2.0 / rot_dim * log(static_cast<double>(rope_base))) : 0.0;
  a.parts = warps_per_token(n_tokens, n_hq + n_hkv, head_dim);
  a.partial = static_cast<float*>(workspace);
  int blocks = 0;
  if (n_tokens > 0) {
    blocks = n_blocks(n_tokens, a.parts);
    const tg_status r = dtype == TG_BF16 ? launch_norm<__nv_bfloat16, true>(a, blocks, stream)
                                         : launch_norm<float, true>(a, blocks, stream);
    if (r != TG_OK) return r;
  }
  return tg::launch(norm_dw_kernel, dim3((2 * head_dim + 31) / 32), dim3(32, 32), 0, stream, 0,
                    static_cast<const float*>(a.partial), blocks, head_dim, dq_weight, dk_weight);
}
