// The quantised KV cache: rows are stored as 8-bit codes with one fp32 scale per row
// and KV head (MarkTechPost page on TokenGate, section "Comment déployer TokenGate ?":
// the cache of kept tokens is what generation holds in memory; codes halve it again).
//
// tg_quant_cache_append writes rows: for one row's head x (dh bf16 values)
//     scale = fl32(max|x| / qmax), qmax = 127 (int8) or 448 (e4m3),
//     code  = x / scale rounded to the nearest code, ties to even.
// The code is that of the exact quotient x / scale, without a division. Let X and A be the
// 8-bit significands of x and the maximum, B = 2n + 1 that of a border between two codes (at
// most 8 bits for int8, 5 for e4m3), Q = 127 or 7 the odd part of qmax: up to powers of two
// x qmax / max over the border is Q X / (B A), which is 1 or differs from it by at least
// 1 / (253 * 255) > 2^-16. So only an exact tie comes near a border, and there the rounding of
// the scale decides: a scale above max / qmax makes the quotient less than the border, one
// below it more. Its sign is that of scale * qmax - max (one exact fused product); x is
// multiplied by 1 / scale (off by 2^-22 with all roundings) times 1 -+ 2^-18, and the product
// rounded to 20 bits, which gives a tie back where the scale is exact and moves nothing else
// over a border.
// A scale below 2^-60 is stored as 0 with codes 0; a row that holds an infinity or a
// NaN gets a NaN scale and codes 0, so it reads back as NaN.
//
// tg_quant_cache_read gives rows back: code * scale in fp32, rounded once.
//
// Both are bound by memory (append: 2 bytes in and 1 out per value; read: 1 in and 2
// or 4 out): 12220 rows of eight heads of 128 in eight sequences are appended in 17.9 us (e4m3,
// 4.2 TB/s, 65% of issue slots busy) and 18.6 us (int8), 34446 int8 rows in four sequences read
// back as bf16 in 39.1 us (5.5 TB/s, 84% of a plain copy's rate) and as f32 in 76.5 us (4.6 TB/s).
// A warp takes one row (for few rows: part of its heads); a head's lanes hold 16
// values each to write (so that the scale is formed by few) and 8 to read.
#include <cuda_fp16.h>

#include "common.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxBlocks = 148 * 8;
constexpr float kMinScale = 0x1p-60f;
constexpr int kMaxBatch = 65535;

struct QuantArgs {
  const void *k, *v;              // append: new rows
  const float* s_new;
  const int32_t *cu, *src_idx, *start, *cache_len;
  uint8_t *kc, *vc;
  float *ks, *vs, *s_cache;
  int32_t* new_len;               // append: written with start + rows, or null
  void *ko, *vo;                  // read: outputs
  float* so;
  int64_t n_rows, n_src;
  int batch, cap, n_hkv, parts;
  int* status;
};

// Sequence of packed row r: the last b with cu[b] <= r, by a 32-way search (one load
// and a vote a level). -1 for rows before the first or behind the last sequence.
__device__ __forceinline__ int find_seq(const int32_t* cu, int batch, int64_t r, int lane) {
  int lo = 0, n = batch + 1;   // the answer lies in [lo, lo + n)
  if (static_cast<int64_t>(cu[0]) > r) return -1;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + min(lane * step, n - 1);
    const unsigned below = __ballot_sync(0xFFFFFFFFu, static_cast<int64_t>(cu[i]) <= r);
    const int last = 31 - __clz(below);   // cu ascends, and cu[lo] <= r
    const int at = min(last * step, n - 1);
    n = min(step, n - at);
    lo += at;
  }
  return lo < batch ? lo : -1;
}

// Whether the search above gives sequence b for all of its rows c0 .. c1 - 1 (one or more). Where the
// offsets ascend it does. Where they do not, two sequences may claim the same rows; the
// search still gives a row to one sequence at most, and since every level's choice grows
// with r, rows between two that go to b go to b too: it is enough to look at the ends.
// Not inlined, so that the row loops keep the registers for their loads (34446 int8 rows
// read to bf16 through the binding: 40.0 us, inlined 41.0).
__device__ __noinline__ bool owns(const int32_t* cu, int batch, int b, int64_t c0, int64_t c1, int lane) {
  int lo = 0, n = batch + 1;
  if (static_cast<int64_t>(cu[0]) > c0) return false;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int64_t c = cu[lo + min(lane * step, n - 1)];
    const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, c <= c0));
    if (last != 31 - __clz(__ballot_sync(0xFFFFFFFFu, c < c1))) return false;
    const int at = min(last * step, n - 1);
    n = min(step, n - at);
    lo += at;
  }
  return lo == b;
}

// The offsets of up to kSmemBatch sequences and the rows they start at are read once a
// block: every row then finds its sequence without a load from global memory.
constexpr int kSmemBatch = 1024;
struct SeqSmem {
  int32_t cu[kSmemBatch + 1], start[kSmemBatch];
};
struct SeqTable {
  const int32_t *cu, *start;   // start: null for 0
  bool ascends;                // the offsets are known to ascend
};
__device__ __forceinline__ SeqTable seq_table(const QuantArgs& A, SeqSmem& S) {
  if (A.batch > kSmemBatch) return SeqTable{A.cu, A.start, false};
  bool ok = true;
  for (int b = threadIdx.x; b <= A.batch; b += kThreads) {
    const int32_t c = A.cu[b], before = A.cu[b > 0 ? b - 1 : 0];
    if (b < A.batch) S.start[b] = A.start ? A.start[b] : 0;
    S.cu[b] = c;
    ok = ok && before <= c;
  }
  ok = __syncthreads_and(ok);
  return SeqTable{S.cu, S.start, ok};
}

// A sequence's rows as the call describes them, and whether they fit.
struct SeqRows {
  int64_t first;   // its first packed row
  int64_t n;       // rows
  int64_t start;   // cache row of the first
  bool ok;
};
__device__ __forceinline__ SeqRows seq_rows(const QuantArgs& A, const SeqTable& Q, int b, bool reading) {
  SeqRows s;
  const int64_t c0 = Q.cu[b], c1 = Q.cu[b + 1];
  s.first = c0;
  s.n = c1 - c0;
  s.start = Q.start ? Q.start[b] : 0;
  int64_t top = A.cap;
  if (reading) {
    const int64_t len = A.cache_len[b];
    top = len < top ? len : top;
  }
  s.ok = c0 >= 0 && s.n >= 0 && c1 <= A.n_rows && s.start >= 0 && s.start + s.n <= top;
  return s;
}

// ---- codes ----

// Two quotients to two codes, as the low and high byte of 16 bits.
template <bool kE4m3>
__device__ __forceinline__ uint32_t codes_of(float y0, float y1) {
  if constexpr (kE4m3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y1), "f"(y0));
    return r;
  } else {   // 1.5 * 2^23 + y has round(y) in its last bits (|y| <= 127), ties to even
    const uint32_t a = __float_as_uint(y0 + 12582912.f), b = __float_as_uint(y1 + 12582912.f);
    return __byte_perm(a, b, 0x0040) & 0xFFFFu;
  }
}
// A quotient to 20 bits.
__device__ __forceinline__ float to_20_bits(float y) {
  return __uint_as_float((__float_as_uint(y) + 4) & ~7u);
}
// The codes of bf16 pairs; inv is 1 / scale with the nudge.
template <bool kE4m3>
__device__ __forceinline__ uint32_t encode2(uint32_t u, float inv) {
  return codes_of<kE4m3>(to_20_bits(__uint_as_float(u << 16) * inv),
                         to_20_bits(__uint_as_float(u & 0xFFFF0000u) * inv));
}
template <bool kE4m3>
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  return make_uint2(encode2<kE4m3>(x.x, inv) | encode2<kE4m3>(x.y, inv) << 16,
                    encode2<kE4m3>(x.z, inv) | encode2<kE4m3>(x.w, inv) << 16);
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <int DH, bool kE4m3>
__global__ void __launch_bounds__(kThreads) quant_append_kernel(const QuantArgs A) {
  constexpr int kLph = DH / 16;         // lanes of a head
  constexpr int kHpw = 32 / kLph;       // heads side by side
  constexpr int kU = 2;                 // of them in flight
  __shared__ SeqSmem S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % kLph, sub = lane / kLph;
  tg::pdl_launch_dependents();
  tg::pdl_wait();
  const SeqTable Q = seq_table(A, S);
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  // the record of sequences that do not fit (offsets that do not ascend have one whose end is
  // before its start), and lengths of those without rows
  for (int64_t b = gw * 32 + lane; b < A.batch; b += n_warps * 32) {
    const SeqRows s = seq_rows(A, Q, static_cast<int>(b), false);
    if (!s.ok) tg::set_status(A.status, TG_ERR_DEVICE_CHECK);
    else if (A.new_len && s.n == 0) A.new_len[b] = static_cast<int32_t>(s.start);
  }
  const int heads = 2 * A.n_hkv;        // of K, then of V
  const int64_t n_work = A.n_rows * A.parts;
#pragma unroll 1
  for (int64_t w = gw; w < n_work; w += n_warps) {
    const int64_t r = A.parts == 1 ? w : w / A.parts;
    const int part = static_cast<int>(w - r * A.parts);
    const int64_t src = A.src_idx ? A.src_idx[r] : r;
    const bool have = src >= 0 && src < A.n_src;   // a row that is not there is stored as zeros
    const int b = find_seq(Q.cu, A.batch, r, lane);
    if (b < 0) continue;
    const SeqRows s = seq_rows(A, Q, b, false);
    if (!s.ok || r - s.first >= s.n) continue;
    if (!Q.ascends && s.n > 1 && !owns(Q.cu, A.batch, b, s.first, s.first + s.n, lane)) continue;
    const int64_t row = static_cast<int64_t>(b) * A.cap + s.start + (r - s.first);
    if (!tg::in_bounds(row, static_cast<int64_t>(A.batch) * A.cap, A.status)) continue;
    if (part == 0 && lane == 0) {
      if (!have) tg::set_status(A.status, TG_ERR_DEVICE_CHECK);
      if (A.new_len && r == s.first) A.new_len[b] = static_cast<int32_t>(s.start + s.n);
      A.s_cache[row] = have ? A.s_new[src] : 0.f;
    }
    // heads part*kHpw + sub, then every parts*kHpw-th
    const int step = A.parts * kHpw;
#pragma unroll 1
    for (int h0 = part * kHpw; h0 < heads; h0 += kU * step) {
      uint4 x[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step + sub;
        const bool val = h >= A.n_hkv;
        x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
        if (h < heads && have) {
          const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(val ? A.v : A.k) +
                                                          (src * A.n_hkv + (val ? h - A.n_hkv : h)) * DH + 16 * c);
          x[u][0] = p[0];
          x[u][1] = p[1];
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * step + sub;
        const bool val = h >= A.n_hkv;
        // bf16 magnitudes order as their bits do, infinities and NaN on top
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          m = max_u16x2(m, max_u16x2(max_u16x2(x[u][i].x & 0x7FFF7FFFu, x[u][i].y & 0x7FFF7FFFu),
                                     max_u16x2(x[u][i].z & 0x7FFF7FFFu, x[u][i].w & 0x7FFF7FFFu)));
#pragma unroll
        for (int o = kLph / 2; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        m = max(m >> 16, m & 0xFFFFu);
        const bool finite = m < 0x7F80u;
        // max / qmax rounded once to fp32: the quotient of eight bits by qmax lies far more than
        // a 64-bit product's 2^-52 from any border between two fp32 values
        float scale = static_cast<float>(static_cast<double>(__uint_as_float(m << 16)) * (1.0 / (kE4m3 ? 448.0 : 127.0)));
        if (scale < kMinScale) scale = 0.f;
        uint2 a = make_uint2(0, 0), b2 = a;
        if (finite && scale > 0.f) {
          float inv;
          asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
          const float over = fmaf(scale, kE4m3 ? 448.f : 127.f, -__uint_as_float(m << 16));
          if (over != 0.f) inv *= over > 0.f ? 1.f - 0x1p-18f : 1.f + 0x1p-18f;
          a = encode8<kE4m3>(x[u][0], inv);
          b2 = encode8<kE4m3>(x[u][1], inv);
        }
        if (h < heads) {
          const int64_t hr = row * A.n_hkv + (val ? h - A.n_hkv : h);
          *reinterpret_cast<uint4*>((val ? A.vc : A.kc) + hr * DH + 16 * c) = make_uint4(a.x, a.y, b2.x, b2.y);
          if (c == 0) (val ? A.vs : A.ks)[hr] = finite ? scale : __uint_as_float(0x7FC00000u);
        }
      }
    }
  }
}

// The lengths of an append in place: cache_len is also where the rows start, so it
// moves only once the copy kernel has read it. Every block looks at all offsets; the
// sequences' rows are searched for only where those do not ascend.
__global__ void __launch_bounds__(kThreads) quant_len_kernel(const QuantArgs A, int32_t* len) {
  tg::pdl_launch_dependents();
  tg::pdl_wait();
  const int b = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
  SeqRows s = {};
  if (b < A.batch) s = seq_rows(A, SeqTable{A.cu, A.start, false}, b, false);
  bool down = false;
#pragma unroll 8
  for (int i = threadIdx.x; i < A.batch; i += kThreads) down |= A.cu[i] > A.cu[i + 1];
  down = __syncthreads_or(down);
  for (unsigned left = __ballot_sync(0xFFFFFFFFu, down && s.ok && s.n > 0); left; left &= left - 1) {
    const int l = __ffs(left) - 1;
    const int64_t c0 = __shfl_sync(0xFFFFFFFFu, s.first, l), n = __shfl_sync(0xFFFFFFFFu, s.n, l);
    const bool all = owns(A.cu, A.batch, b - lane + l, c0, c0 + n, lane);
    if (lane == l) s.ok = all;
  }
  if (s.ok) len[b] = static_cast<int32_t>(s.start + s.n);
}

template <bool kE4m3>
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
  if constexpr (kE4m3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  }
}

template <int DH, bool kE4m3, bool kF32>
__global__ void __launch_bounds__(kThreads) quant_read_kernel(const QuantArgs A) {
  constexpr int kLph = DH / 8;
  constexpr int kHpw = 32 / kLph;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = lane % kLph, sub = lane / kLph;
  __shared__ SeqSmem S;
  tg::pdl_launch_dependents();
  tg::pdl_wait();
  const SeqTable Q = seq_table(A, S);
  const int64_t gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t b = gw * 32 + lane; b < A.batch; b += n_warps * 32)
    if (!seq_rows(A, Q, static_cast<int>(b), true).ok) tg::set_status(A.status, TG_ERR_DEVICE_CHECK);
  const int64_t n_work = A.n_rows * A.parts;
  for (int64_t w = gw; w < n_work; w += n_warps) {
    const int64_t r = A.parts == 1 ? w : w / A.parts;
    const int part = static_cast<int>(w - r * A.parts);
    const int b = find_seq(Q.cu, A.batch, r, lane);
    if (b < 0) continue;
    const SeqRows s = seq_rows(A, Q, b, true);
    if (!s.ok || r - s.first >= s.n) continue;
    if (!Q.ascends && s.n > 1 && !owns(Q.cu, A.batch, b, s.first, s.first + s.n, lane)) continue;
    const int64_t row = static_cast<int64_t>(b) * A.cap + s.start + (r - s.first);
    if (!tg::in_bounds(row, static_cast<int64_t>(A.batch) * A.cap, A.status)) continue;
    if (part == 0 && lane == 0) A.so[r] = A.s_cache[row];
    constexpr int kU = 4;
    for (int h0 = part * kHpw; h0 < 2 * A.n_hkv; h0 += kU * A.parts * kHpw) {
      uint2 x[kU];
      float sc[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * A.parts * kHpw + sub;
        const bool val = h >= A.n_hkv;
        const int64_t hr = row * A.n_hkv + (val ? h - A.n_hkv : h);
        if (h < 2 * A.n_hkv) {
          x[u] = *reinterpret_cast<const uint2*>((val ? A.vc : A.kc) + hr * DH + 8 * c);
          sc[u] = (val ? A.vs : A.ks)[hr];
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + u * A.parts * kHpw + sub;
        if (h >= 2 * A.n_hkv) continue;
        const bool val = h >= A.n_hkv;
        const int64_t at = (r * A.n_hkv + (val ? h - A.n_hkv : h)) * DH + 8 * c;
        float f[8];
        decode4<kE4m3>(x[u].x, f);
        decode4<kE4m3>(x[u].y, f + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= sc[u];
        if constexpr (kF32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(val ? A.vo : A.ko) + at);
          o[0] = make_float4(f[0], f[1], f[2], f[3]);
          o[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(val ? A.vo : A.ko) + at) =
              make_uint4(tg::pack_bf16x2(f[0], f[1]), tg::pack_bf16x2(f[2], f[3]),
                         tg::pack_bf16x2(f[4], f[5]), tg::pack_bf16x2(f[6], f[7]));
        }
      }
    }
  }
}

// Warps per row: one, unless there are too few rows to give every warp of the machine one.
// Appending 12220 rows of eight e4m3 heads of 128: 17.9 us with one, 20.3 us with two; 51 rows:
// 4.3 us with one, 3.3 us with two, 3.1 us with the four (of four heads each) that this gives.
int warps_per_row(int64_t n_rows, int n_hkv, int dh, int per_lane) {
  const int hpw = 32 / (dh / per_lane);
  const int most = (2 * n_hkv + hpw - 1) / hpw;
  const int64_t p = n_rows > 0 ? (148 * 4 * kWarps + n_rows - 1) / n_rows : 1;
  return static_cast<int>(p < most ? p : most);
}

int n_blocks(int64_t n_rows, int parts) {
  int64_t b = (n_rows * parts + kWarps - 1) / kWarps;
  if (b < 1) b = 1;
  return static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
}

tg_status check_quant(tg_dtype cache_dtype, int64_t n_rows, int batch, int cap, int n_hkv,
                      int head_dim) {
  if (batch < 0 || cap <= 0 || n_hkv <= 0 || head_dim <= 0 || n_rows < 0) return TG_ERR_INVALID_ARG;
  if (cache_dtype != TG_I8 && cache_dtype != TG_E4M3) return TG_ERR_UNSUPPORTED;
  if ((head_dim != 64 && head_dim != 128) || batch > kMaxBatch || n_hkv > 4096 || n_rows > INT32_MAX)
    return TG_ERR_UNSUPPORTED;
  return TG_OK;
}

}  // namespace

extern "C" tg_status tg_quant_cache_append(
    const void* k_new, const void* v_new, const float* s_new, int64_t n_src,
    const int32_t* src_idx, int64_t n_new, const int32_t* cu_new, const int32_t* start, int batch,
    int cap, int n_hkv, int head_dim, tg_dtype cache_dtype, void* k_cache, void* v_cache,
    float* k_scale, float* v_scale, float* s_cache, int32_t* cache_len, tg_stream_t stream) {
  tg::NvtxRange nvtx_range("tg_quant_cache_append");
  const tg_status bad = check_quant(cache_dtype, n_new, batch, cap, n_hkv, head_dim);
  if (bad != TG_OK) return bad;
  if (n_src < 0 || (!src_idx && n_new != n_src)) return TG_ERR_INVALID_ARG;
  if (batch == 0) return TG_OK;
  if (!cu_new || !k_cache || !v_cache || !k_scale || !v_scale || !s_cache || !cache_len)
    return TG_ERR_INVALID_ARG;
  if (n_new > 0 && (!k_new || !v_new || !s_new)) return TG_ERR_INVALID_ARG;
  // start and cache_len are one array (an append in place) or two that do not overlap
  const int32_t* from = start ? start : cache_len;
  const bool in_place = from == cache_len;
  if (!in_place && from < cache_len + batch && cache_len < from + batch) return TG_ERR_INVALID_ARG;
  if (!tg::aligned16(k_new) || !tg::aligned16(v_new) || !tg::aligned16(k_cache) ||
      !tg::aligned16(v_cache))
    return TG_ERR_MISALIGNED;
  QuantArgs a = {};
  a.k = k_new, a.v = v_new, a.s_new = s_new;
  a.cu = cu_new, a.src_idx = src_idx, a.start = from;
  a.kc = static_cast<uint8_t*>(k_cache), a.vc = static_cast<uint8_t*>(v_cache);
  a.ks = k_scale, a.vs = v_scale, a.s_cache = s_cache;
  a.new_len = in_place ? nullptr : cache_len;
  a.n_rows = n_new, a.n_src = n_src, a.batch = batch, a.cap = cap, a.n_hkv = n_hkv;
  a.parts = warps_per_row(n_new, n_hkv, head_dim, 16);
  a.status = tg::status_word();
  if (!a.status) return TG_ERR_CUDA;
  const dim3 grid(n_blocks(n_new, a.parts)), block(kThreads);
  tg_status r;
  if (head_dim == 128)
    r = cache_dtype == TG_E4M3 ? tg::launch(quant_append_kernel<128, true>, grid, block, 0, stream, 0, a)
                               : tg::launch(quant_append_kernel<128, false>, grid, block, 0, stream, 0, a);
  else
    r = cache_dtype == TG_E4M3 ? tg::launch(quant_append_kernel<64, true>, grid, block, 0, stream, 0, a)
                               : tg::launch(quant_append_kernel<64, false>, grid, block, 0, stream, 0, a);
  if (r != TG_OK || !in_place) return r;
  return tg::launch(quant_len_kernel, dim3((batch + kThreads - 1) / kThreads), block, 0, stream, 0, a,
                    cache_len);
}

extern "C" tg_status tg_quant_cache_read(const void* k_cache, const void* v_cache,
                                         const float* k_scale, const float* v_scale,
                                         const float* s_cache, const int32_t* cache_len,
                                         const int32_t* start, const int32_t* cu_rows,
                                         int64_t n_rows, int batch, int cap, int n_hkv,
                                         int head_dim, tg_dtype cache_dtype, tg_dtype out_dtype,
                                         void* k, void* v, float* s, tg_stream_t stream) {
  tg::NvtxRange nvtx_range("tg_quant_cache_read");
  const tg_status bad = check_quant(cache_dtype, n_rows, batch, cap, n_hkv, head_dim);
  if (bad != TG_OK) return bad;
  if (out_dtype != TG_F32 && out_dtype != TG_BF16) return TG_ERR_UNSUPPORTED;
  if (batch == 0 || n_rows == 0) return TG_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !s_cache || !cache_len || !cu_rows || !k ||
      !v || !s)
    return TG_ERR_INVALID_ARG;
  if (!tg::aligned16(k_cache) || !tg::aligned16(v_cache) || !tg::aligned16(k) || !tg::aligned16(v))
    return TG_ERR_MISALIGNED;
  QuantArgs a = {};
  a.cu = cu_rows, a.start = start, a.cache_len = cache_len;
  a.kc = static_cast<uint8_t*>(const_cast<void*>(k_cache));
  a.vc = static_cast<uint8_t*>(const_cast<void*>(v_cache));
  a.ks = const_cast<float*>(k_scale), a.vs = const_cast<float*>(v_scale);
  a.s_cache = const_cast<float*>(s_cache);
  a.ko = k, a.vo = v, a.so = s;
  a.n_rows = n_rows, a.batch = batch, a.cap = cap, a.n_hkv = n_hkv;
  a.parts = warps_per_row(n_rows, n_hkv, head_dim, 8);
  a.status = tg::status_word();
  if (!a.status) return TG_ERR_CUDA;
  const dim3 grid(n_blocks(n_rows, a.parts)), block(kThreads);
  const int pick = (head_dim == 128 ? 4 : 0) + (cache_dtype == TG_E4M3 ? 2 : 0) + (out_dtype == TG_F32);
  switch (pick) {
    case 0: return tg::launch(quant_read_kernel<64, false, false>, grid, block, 0, stream, 0, a);
    case 1: return tg::launch(quant_read_kernel<64, false, true>, grid, block, 0, stream, 0, a);
    case 2: return tg::launch(quant_read_kernel<64, true, false>, grid, block, 0, stream, 0, a);
    case 3: return tg::launch(quant_read_kernel<64, true, true>, grid, block, 0, stream, 0, a);
    case 4: return tg::launch(quant_read_kernel<128, false, false>, grid, block, 0, stream, 0, a);
    case 5: return tg::launch(quant_read_kernel<128, false, true>, grid, block, 0, stream, 0, a);
    case 6: return tg::launch(quant_read_kernel<128, true, false>, grid, block, 0, stream, 0, a);
    default: return tg::launch(quant_read_kernel<128, true, true>, grid, block, 0, stream, 0, a);
  }
}
