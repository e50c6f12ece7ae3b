// tg_tree_attention: a tree of drafted tokens attends over the compacted cache
// (MarkTechPost page on TokenGate, section "Comment déployer TokenGate ?": generation
// runs on the cache that the pruned prefill leaves; section "Qu'est-ce que l'attention
// gérée par des tokens ?": key-score bias and per-head temperature). Drafted token t
// of sequence b sees every cache row j < cache_len[b] and the drafted tokens whose bit
// is set in tree_mask[b][t]:
//     z_j = q . k_j / (sqrt(dh) tau_h) + g_h s_j,   O = sum_j softmax_j(z) v_j.
#include <cuda_fp16.h>

#include "common.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kMaxDraft = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct TreeArgs {
  const __nv_bfloat16 *q, *kd, *vd;
  const float* sd;
  const int64_t* mask;
  const int32_t* draft_len;
  const uint8_t *kc, *vc;
  const float *ks, *vs, *sc;
  const int32_t* cache_len;
  const float *gain, *tau;
  __nv_bfloat16* out;
  int batch, n_draft, cap, max_len, n_hq, n_hkv;
  int* status;
};

template <int DH, int kType>
__device__ __forceinline__ float cache_value(const uint8_t* p, int64_t i) {
  if constexpr (kType == TG_BF16) {
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  } else if constexpr (kType == TG_I8) {
    return static_cast<float>(static_cast<int8_t>(p[i]));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(p[i])));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
  }
}

// One warp per (sequence, drafted token, query head), one key at a time.
template <int DH, int kType>
__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const TreeArgs A) {
  constexpr int kE = DH / 32;
  tg::pdl_launch_dependents();
  tg::pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(A.batch) * A.n_draft * A.n_hq) return;
  const int hq = static_cast<int>(w % A.n_hq);
  const int64_t bt = w / A.n_hq;
  const int t = static_cast<int>(bt % A.n_draft), b = static_cast<int>(bt / A.n_draft);
  const int kvh = hq / (A.n_hq / A.n_hkv);
  const int len = A.cache_len[b], dl = A.draft_len ? A.draft_len[b] : A.n_draft;
  if (len < 0 || len > A.cap || len > A.max_len || dl < 0 || dl > A.n_draft) {
    if (lane == 0) tg::set_status(A.status, TG_ERR_DEVICE_CHECK);
    return;
  }
  if (t >= dl) return;
  float q[kE], o[kE];
  const float c = kLog2e / (sqrtf(static_cast<float>(DH)) * A.tau[hq]);
  const float g = A.gain[hq] * kLog2e;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = __bfloat162float(A.q[w * DH + lane * kE + e]);
    o[e] = 0.f;
  }
  const uint64_t mask = static_cast<uint64_t>(A.mask[bt]);
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < len + dl; ++j) {
    float k[kE], v[kE], ksc = 1.f, vsc = 1.f, s;
    if (j < len) {
      const int64_t row = static_cast<int64_t>(b) * A.cap + j, hr = row * A.n_hkv + kvh;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        k[e] = cache_value<DH, kType>(A.kc, hr * DH + lane * kE + e);
        v[e] = cache_value<DH, kType>(A.vc, hr * DH + lane * kE + e);
      }
      if constexpr (kType != TG_BF16) ksc = A.ks[hr], vsc = A.vs[hr];
      s = A.sc[row];
    } else {
      const int i = j - len;
      if (!((mask >> i) & 1)) continue;
      const int64_t row = static_cast<int64_t>(b) * A.n_draft + i, hr = row * A.n_hkv + kvh;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        k[e] = __bfloat162float(A.kd[hr * DH + lane * kE + e]);
        v[e] = __bfloat162float(A.vd[hr * DH + lane * kE + e]);
      }
      s = A.sd[row];
    }
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) z = fmaf(q[e], k[e], z);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, off);
    z = fmaf(z * ksc, c, g * s);
    if (z == -INFINITY) continue;   // a weight of zero
    const float mn = fmaxf(m, z);
    const float a = exp2f(m - mn), p = exp2f(z - mn);
    l = fmaf(l, a, p);
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = fmaf(o[e], a, p * vsc * v[e]);
    m = mn;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;   // nothing visible: zeros
#pragma unroll
  for (int e = 0; e < kE; ++e) A.out[w * DH + lane * kE + e] = __float2bfloat16_rn(o[e] * inv);
}

template <int DH, int kType>
tg_status launch_tree(const TreeArgs& a, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(a.batch) * a.n_draft * a.n_hq;
  return tg::launch(tree_attn_kernel<DH, kType>, dim3(static_cast<unsigned>((warps + 3) / 4)),
                    dim3(kThreads), 0, st, 0, a);
}

}  // namespace

extern "C" size_t tg_tree_attention_workspace_size(int batch, int n_draft, int max_len, int n_hq,
                                                   int n_hkv, int head_dim) {
  if (batch <= 0 || n_draft <= 0 || max_len < 0 || n_hq <= 0 || n_hkv <= 0 || head_dim <= 0) return 0;
  return 16;
}

extern "C" tg_status tg_tree_attention(
    const void* q, const void* k_draft, const void* v_draft, const float* s_draft,
    const int64_t* tree_mask, const int32_t* draft_len, int batch, int n_draft,
    const void* k_cache, const void* v_cache, tg_dtype cache_dtype, const float* k_scale,
    const float* v_scale, const float* s_cache, const int32_t* cache_len, int cap, int max_len,
    int n_hq, int n_hkv, int head_dim, const float* gain, const float* tau, void* out,
    void* workspace, size_t workspace_bytes, tg_stream_t stream) {
  tg::NvtxRange nvtx_range("tg_tree_attention");
  if (batch < 0 || n_draft < 0 || cap <= 0 || max_len < 0 || n_hq <= 0 || n_hkv <= 0 ||
      head_dim <= 0 || max_len > cap || n_hq % n_hkv != 0)
    return TG_ERR_INVALID_ARG;
  if (cache_dtype != TG_BF16 && cache_dtype != TG_I8 && cache_dtype != TG_E4M3)
    return TG_ERR_UNSUPPORTED;
  if (batch == 0 || n_draft == 0) return TG_OK;
  if (!q || !k_draft || !v_draft || !s_draft || !tree_mask || !k_cache || !v_cache || !s_cache ||
      !cache_len || !gain || !tau || !out)
    return TG_ERR_INVALID_ARG;
  const bool quantised = cache_dtype != TG_BF16;
  if (quantised ? !k_scale || !v_scale : k_scale || v_scale) return TG_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || n_draft > kMaxDraft || n_hq / n_hkv > 128 ||
      batch > 1024 || n_hkv > 1024 || static_cast<int64_t>(batch) * cap > INT32_MAX - 128)
    return TG_ERR_UNSUPPORTED;
  if (!tg::aligned16(q) || !tg::aligned16(k_draft) || !tg::aligned16(v_draft) ||
      !tg::aligned16(k_cache) || !tg::aligned16(v_cache) || !tg::aligned16(out))
    return TG_ERR_MISALIGNED;
  const size_t need = tg_tree_attention_workspace_size(batch, n_draft, max_len, n_hq, n_hkv, head_dim);
  if (!workspace || workspace_bytes < need) return TG_ERR_WORKSPACE;
  if (!tg::aligned16(workspace)) return TG_ERR_MISALIGNED;
  TreeArgs a = {};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.kd = static_cast<const __nv_bfloat16*>(k_draft), a.vd = static_cast<const __nv_bfloat16*>(v_draft);
  a.sd = s_draft, a.mask = tree_mask, a.draft_len = draft_len;
  a.kc = static_cast<const uint8_t*>(k_cache), a.vc = static_cast<const uint8_t*>(v_cache);
  a.ks = k_scale, a.vs = v_scale, a.sc = s_cache, a.cache_len = cache_len;
  a.gain = gain, a.tau = tau, a.out = static_cast<__nv_bfloat16*>(out);
  a.batch = batch, a.n_draft = n_draft, a.cap = cap, a.max_len = max_len, a.n_hq = n_hq, a.n_hkv = n_hkv;
  a.status = tg::status_word();
  if (!a.status) return TG_ERR_CUDA;
  if (head_dim == 128) {
    if (cache_dtype == TG_BF16) return launch_tree<128, TG_BF16>(a, stream);
    return cache_dtype == TG_I8 ? launch_tree<128, TG_I8>(a, stream) : launch_tree<128, TG_E4M3>(a, stream);
  }
  if (cache_dtype == TG_BF16) return launch_tree<64, TG_BF16>(a, stream);
  return cache_dtype == TG_I8 ? launch_tree<64, TG_I8>(a, stream) : launch_tree<64, TG_E4M3>(a, stream);
}
