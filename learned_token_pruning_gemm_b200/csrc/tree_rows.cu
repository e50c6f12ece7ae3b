// tg_tree_attention for few rows (drafted tokens x query heads of a KV head, up to 16) over a
// cache of codes: the part over the cache. There is little to multiply per byte of cache then,
// and tree_attn_kernel, which widens every code to an operand tile for 128 rows, takes longer
// over the widening than this kernel over everything. Here all warps run the same code, straight
// from a TMA ring into the register fragments of m16n8k16 products, each with its own running
// reference, sums and O, so nothing joins them but the ring.
//
// A unit is 16 keys a warp: the warps share hw KV heads of the same cache rows (all of them
// up to four or eight, so that a tile is one contiguous piece of the cache or nearly) and, where
// there are fewer heads, split the keys in kw parts. Every warp leaves a partial (max, sum, O)
// per item, and the second kernel adds those up and brings in the drafted rows.
//
// Products are taken as S^T = K Q^T (16 keys x 8 rows at a time) and O^T = V^T P^T: rows
// are the short side of a product, so eight rows cost half of sixteen. The weights change
// from one product's result to the other's operand by a transpose of 8 x 8 in the warp.
// Any dim may take any place of an inner index or of the 16-high side, as long as both
// operands agree, so that every thread (g = lane / 4, i = lane % 4) reads 16-byte pieces:
//   S^T: dims 32 i .. 32 i + 31 of keys g and g + 8;
//   O^T: dims 16 g .. 16 g + 15 of keys 2 i, 2 i + 1, 2 i + 8 and 2 i + 9: product t holds the
//        dims at places 2 t and 2 t + 1 of these
// (head dim 64: half of these, and 8-byte pieces of V).
// What bounds it is the instructions, about 480 a unit, and their latency at 12 to 16 warps an SM
// (43% of issue slots busy). 32 sequences of 1868 e4m3 rows of eight heads, a token of 16 heads:
// 37.4 us with the combining kernel (33 without; 19.4 us is the read at a plain copy's
// rate), int8 40.5 us; eight tokens over 8 x 10721 rows: 71 us (27.9). Head dim 64: 32 us (10.0) and
// 59 us (14.4).
//
// Codes are widened to fp16, which holds them exactly at half the instructions that bf16
// takes; the queries are then fp16 too, after their largest value is brought near 2^8.
#include "tree.cuh"

namespace {

using tg::TreeArgs;
using tg::bf16x2_to_f16x2;
using tg::max_u16x2;
using tg::pack_f16x2;
using tg::wait;
using tg::widen4;

// NT tiles of eight rows. Several CTAs share an SM, so that one's start and end of an item
// pass under the others' work; registers say how many, and the ring takes the rest of the
// shared memory. Single tokens as above: 37.6 us with 2 CTAs of 8 warps, 39.0 with 4 of 4
// (a ring of 5), 43.8 with 3 of 4 (a ring of 8), 61.9 with 5 of 4 (registers spill).
template <int DH, int NT>
struct Cfg {
  static constexpr int kWarps = NT == 1 ? 8 : 4;   // of a CTA
  static constexpr int kCtas = NT == 1 ? 2 : 3;    // an SM
  static constexpr int kRing = (NT == 1 ? 5 : 7) * (128 / DH);   // tiles
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTile = 16 * kWarps * DH;   // bytes of a K or V tile, at most
  static_assert(kRing >= 4, "a unit's tiles are asked for while the one before is in use");
};

// Places in the walk over a CTA's units.
struct Cursor {
  int u, u1, b, group, j, nt, len;
  __device__ __forceinline__ void start(const TreeArgs& A, const tg::TreeSeqs& s, int first, int n) {
    u = first;
    u1 = first + n;
    b = tg::sequence_of(A, s, u);
    len = s.len[b];
    nt = tg::key_units(A, len);
    group = (u - s.base[b]) / nt;
    j = u - s.base[b] - group * nt;
  }
  __device__ __forceinline__ void advance(const TreeArgs& A, const tg::TreeSeqs& s) {
    ++u;
    if (++j < nt || u >= u1) return;
    j = 0;
    if (++group < tg::head_groups(A)) return;
    group = 0;
    do ++b;
    while (s.base[b + 1] == s.base[b]);   // sequences without units
    len = s.len[b];
    nt = tg::key_units(A, len);
  }
};

template <int DH, int NT>
struct RowSmem {
  using C = Cfg<DH, NT>;
  uint8_t tile[C::kRing][C::kTile];
  uint2 q[C::kWarps][NT][DH / 16][32];       // B fragments of each warp's queries
  float2 cg[C::kWarps][8 * NT];        // each row's logit factor and gain, log2 domain
  uint64_t full[C::kRing], empty[C::kRing];
  Cursor next;                      // the unit that is loaded next, and
  int issued;                       // the tiles that are on their way or here
  int abort_flag;
  // behind it, by the batch: first units, cache lengths, drafted tokens
  __device__ __forceinline__ tg::TreeSeqs seqs(int batch) {
    int* p = reinterpret_cast<int*>(this + 1);
    return tg::TreeSeqs{p, p + batch + 1, reinterpret_cast<uint8_t*>(p + 2 * batch + 1)};
  }
};

// Loads tiles as far as the ring reaches (K at even places, V at odd ones): tile t needs
// tile t - kRing to be consumed by every warp, which is waited for, and all before
// `consumed` are by this one. One thread.
template <int DH, int NT>
__device__ __noinline__ void row_loads(const TreeArgs& A, RowSmem<DH, NT>& S, const CUtensorMap* tm_k,
                                       const CUtensorMap* tm_v, int consumed) {
  using C = Cfg<DH, NT>;
  const tg::TreeSeqs Q = S.seqs(A.batch);
  int t = S.issued;
  Cursor c = S.next;
  while (t < consumed + C::kRing && c.u < c.u1) {
    const int s = t % C::kRing;
    if (t >= C::kRing && !wait(&S.empty[s], ((t / C::kRing) - 1) & 1, A.status, &S.abort_flag)) break;
    tg::mbar_arrive_expect_tx(&S.full[s], A.hw * A.unit * DH);
    tg::tma_load_3d(S.tile[s], t & 1 ? tm_v : tm_k, &S.full[s], 0, c.b * A.cap + c.j * A.unit, c.group * A.hw);
    if (t & 1) c.advance(A, Q);
    ++t;
  }
  S.issued = t;
  S.next = c;
}

// One 16 x 8 x 16 product, fp16 operands, fp32 sums. volatile: it stays before the arrival that
// gives its tile back, so that the tile's loads are over by then.
__device__ __forceinline__ void mma_16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
               "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values held as product fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// 8 bytes global -> shared, asynchronously
__device__ __forceinline__ void cp8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tg::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

template <int kType, int DH, int NT>
__global__ void __launch_bounds__(Cfg<DH, NT>::kThreads, Cfg<DH, NT>::kCtas)
    tree_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ TreeArgs A) {
  constexpr bool kE4m3 = kType == TG_E4M3;
  constexpr uint32_t kFlip = kType == TG_I8 ? 0x80808080u : 0u;
  using C = Cfg<DH, NT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (tg::smem_u32(smem_raw) & 1023u)) & 1023u;
  RowSmem<DH, NT>& S = *reinterpret_cast<RowSmem<DH, NT>*>(smem_raw + pad);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, i4 = lane & 3;
  if (tid == 0) {
    for (int s = 0; s < C::kRing; ++s) {
      tg::mbar_init(&S.full[s], 1);
      tg::mbar_init(&S.empty[s], C::kWarps);
    }
    S.abort_flag = 0;
    tg::fence_barrier_init();
    tg::tma_prefetch_desc(&tm_k);
    tg::tma_prefetch_desc(&tm_v);
  }
  tg::pdl_launch_dependents();
  tg::pdl_wait();   // global memory only from here on
  const tg::TreeSeqs Q = S.seqs(A.batch);
  const tg::Shares share(A, tg::count_units<C::kThreads>(A, Q));
  const int n = share.size(blockIdx.x);
  if (n == 0) return;   // uniform: nothing to do here
  Cursor c;
  c.start(A, Q, share.first(blockIdx.x), n);
  const bool loader = tid == C::kThreads - 1;   // the last warp's last thread
  if (loader) {
    S.issued = 0;
    S.next = c;
    row_loads<DH, NT>(A, S, &tm_k, &tm_v, 0);
  }
  __syncwarp();

  // A wait that runs out records itself and sets the abort flag, after which every wait
  // returns at once: the loops below take the same steps either way.
  const int rows = A.group * A.n_draft;
  const int hd = warp / A.kw, k0 = 16 * (warp - hd * A.kw);   // head of the item, first key of the unit
  constexpr int kT = DH / 16;         // products of a unit, of either kind
  float o[NT][kT][4];                  // product t: dims at places 2t, 2t + 1 x rows 2 i4, 2 i4 + 1
  float m[NT][2], l[NT][2];           // of rows 2 i4 and 2 i4 + 1 of every tile
  bool first = true;
  int r = 0;
#pragma unroll 1
  for (int u = 0; u < n; ++u) {
    const int kvh = c.group * A.hw + hd;
    const bool head = hd < A.hw && kvh < A.n_hkv;   // else this warp only keeps the ring going
    const int nv = min(A.unit, c.len - c.j * A.unit);
    const bool any = head && k0 < nv;
    // What the thread's keys g and g + 8 bring besides K and V. Keys behind the last one read its
    // place and are masked below.
    float sk[2] = {}, ks[2] = {}, vs[2] = {};
    if (any) {
      const int row0 = c.b * A.cap + c.j * A.unit;   // batch * cap is below 2^31
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = row0 + min(k0 + g + 8 * x, nv - 1);
        if (!tg::in_bounds(row, static_cast<int64_t>(A.batch) * A.cap, A.status)) continue;
        const int64_t at = static_cast<int64_t>(row) * A.n_hkv + kvh;
        sk[x] = A.sc[row];
        ks[x] = A.ks[at];
        vs[x] = A.vs[at];
      }
    }
    if (first && head) {   // a new item: its queries, and nothing seen yet
      __syncwarp();
      const int64_t row_q = static_cast<int64_t>(c.b) * A.n_draft * A.n_hq + kvh * A.group;
#pragma unroll 1
      for (int nt = 0; nt < NT; ++nt) {   // rows behind the last: any row that is there
        const int row = min(8 * nt + g, rows - 1), tok = tg::token_of(A, row);
        const __nv_bfloat16* p = A.q + (row_q + tok * A.n_hq + row - tok * A.group) * DH;
#pragma unroll
        for (int t = 0; t < kT; ++t)   // dims as the keys' below
          cp8(&S.q[warp][nt][t][lane],
              p + DH / 4 * i4 + 4 * t);
      }
      if (lane < 8 * NT) {
        const int row = min(lane, rows - 1), hq = kvh * A.group + row - tg::token_of(A, row) * A.group;
        S.cg[warp][lane] = make_float2(tg::kLog2e / (sqrtf(static_cast<float>(DH)) * A.tau[hq]), A.gain[hq] * tg::kLog2e);
      }
      cp_wait_all();
      __syncwarp();
      // to fp16: the row is multiplied by the power of two that brings its largest value
      // (exponent field e) to [2^8, 2^9), so that values down to 2^-22 of it stay exact
#pragma unroll 1
      for (int nt = 0; nt < NT; ++nt) {
        uint2 x[kT];
        uint32_t mx = 0;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          x[t] = S.q[warp][nt][t][lane];
          mx = max_u16x2(mx, max_u16x2(x[t].x & 0x7FFF7FFFu, x[t].y & 0x7FFF7FFFu));
        }
        mx = max_u16x2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = max_u16x2(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const int e = max(static_cast<int>(max(mx >> 16, mx & 0xFFFFu) >> 7), 9);
        const float down = __int_as_float((262 - e) << 23);
#pragma unroll
        for (int t = 0; t < kT; ++t)
          S.q[warp][nt][t][lane] = make_uint2(bf16x2_to_f16x2(x[t].x, down), bf16x2_to_f16x2(x[t].y, down));
        if (i4 == 0) S.cg[warp][8 * nt + g].x *= __int_as_float((e - 8) << 23);
      }
      __syncwarp();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][t][e] = 0.f;
      }
    }
    // ---- S^T = K Q^T ----
    float z[NT][4];   // key g: rows 2 i4, 2 i4 + 1; key g + 8: the same
    const int s = r % C::kRing, sv = (r + 1) % C::kRing;
    wait(&S.full[s], (r / C::kRing) & 1, A.status, &S.abort_flag);
    __syncwarp();
    if (any) {
      // a head's rows of the tile follow each other; the places of both keys among eight are g
      const uint8_t* p = S.tile[s] + (hd * A.unit + k0 + g) * DH;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[nt][e] = 0.f;
      float z2[NT][4] = {};   // every other product's sums: two chains are half as long
#pragma unroll
      for (int i = 0; i < DH / 64; ++i) {
        const uint8_t* at = p + ((DH == 128 ? (2 * i4 + i) ^ g : i4 ^ (g >> 1)) << 4);
        const uint4 x0 = *reinterpret_cast<const uint4*>(at), x1 = *reinterpret_cast<const uint4*>(at + 8 * DH);
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // product t: four dims of the thread's part
          const int t = 4 * i + e;
          uint32_t a0, a1, a2, a3;
          widen4<kE4m3>(word_of(x0, e) ^ kFlip, a0, a2);
          widen4<kE4m3>(word_of(x1, e) ^ kFlip, a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 b = S.q[warp][nt][t][lane];
            mma_16816(e & 1 ? z2[nt] : z[nt], a0, a1, a2, a3, b.x, b.y);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[nt][e] += z2[nt][e];
    }
    __syncwarp();
    if (lane == 0) tg::mbar_arrive(&S.empty[s]);
    // the ring goes on where every warp is through with the unit before
    if (loader) row_loads<DH, NT>(A, S, &tm_k, &tm_v, r);
    __syncwarp();
    uint32_t b[NT][2];   // the weights as fragments
    if (any) {
      // ---- weights ----
      // The value scale v joins the logit, z + log2 v, so that the fp16 weights
      // 2^(z + log2 v - m) are what the codes are multiplied by and m follows their largest;
      // the row sum takes them in fp32, divided by v. Where v is 0 all codes are, and any v
      // small enough not to lead will do.
      float lv[2], iv[2];
      if (fmaxf(fabsf(sk[0]), fabsf(sk[1])) > tg::kMostScore) sk[0] = tg::held(sk[0]), sk[1] = tg::held(sk[1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (vs[x] == 0.f) vs[x] = 0x1p-40f;
        lv[x] = __log2f(vs[x]);
        iv[x] = __frcp_rn(vs[x]);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float4 cg = *reinterpret_cast<const float4*>(&S.cg[warp][8 * nt + 2 * i4]);   // two rows
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float &y0 = z[nt][2 * x], &y1 = z[nt][2 * x + 1];
          y0 = fmaf(y0 * ks[x], cg.x, fmaf(cg.y, sk[x], lv[x]));
          y1 = fmaf(y1 * ks[x], cg.z, fmaf(cg.w, sk[x], lv[x]));
          if (k0 + g + 8 * x >= nv) y0 = y1 = -INFINITY;   // a key that is not there
        }
        // A row's reference is a whole number 6 below its largest logit or less (which keeps small
        // fp16 weights exact) when it is set, and moves when a logit exceeds it by more than 14, so
        // that the weights are 2^14 at most, in fp16's range. The difference is compared, as the
        // weights take it: a sum m + 14 of large numbers is rounded to their last place, and
        // weights of 2^16 passed under it.
        constexpr float kLift = 6.f, kMost = kLift + tg::kRescaleThreshold;
        const float m0 = fmaxf(z[nt][0], z[nt][2]), m1 = fmaxf(z[nt][1], z[nt][3]);
        if (__any_sync(0xFFFFFFFFu, m0 - m[nt][0] > kMost || m1 - m[nt][1] > kMost)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = e ? m1 : m0;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, x));
            t = t - m[nt][e] > kMost ? ceilf(t) - kLift : m[nt][e];
            const float alpha = t == m[nt][e] ? 1.f : tg::exp2_approx(m[nt][e] - t);
            m[nt][e] = t;
            l[nt][e] *= alpha;
#pragma unroll
            for (int k = 0; k < kT; ++k) {
              o[nt][k][e] *= alpha;
              o[nt][k][2 + e] *= alpha;
            }
          }
        }
        const float n0 = m[nt][0] == -INFINITY ? 0.f : -m[nt][0], n1 = m[nt][1] == -INFINITY ? 0.f : -m[nt][1];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float p0 = tg::exp2_approx(z[nt][2 * x] + n0), p1 = tg::exp2_approx(z[nt][2 * x + 1] + n1);
          const uint32_t w = pack_f16x2(p0, p1);
          l[nt][0] = fmaf(p0, iv[x], l[nt][0]);
          l[nt][1] = fmaf(p1, iv[x], l[nt][1]);
          b[nt][x] = transpose8(w);
        }
      }
    }
    wait(&S.full[sv], ((r + 1) / C::kRing) & 1, A.status, &S.abort_flag);
    __syncwarp();
    if (any) {
      // ---- O^T += V^T P^T ----
      uint32_t xv[4][DH / 32];   // keys 2 i4 + {0, 1, 8, 9}
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int key = k0 + 2 * i4 + (y & 1) + 8 * (y >> 1);
        const uint8_t* p = S.tile[sv] + (hd * A.unit + key) * DH;
        const bool ok = nv - k0 >= 16 || key < nv;   // rows behind the end weigh 0
        if constexpr (DH == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(p + ((g ^ (key & 7)) << 4));
          xv[y][0] = ok ? x.x : 0u, xv[y][1] = ok ? x.y : 0u, xv[y][2] = ok ? x.z : 0u, xv[y][3] = ok ? x.w : 0u;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(p + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + 8 * (g & 1));
          xv[y][0] = ok ? x.x : 0u, xv[y][1] = ok ? x.y : 0u;
        }
      }
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        uint32_t a[4];   // [key half][place]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t x = xv[2 * h][t >> 1], y = xv[2 * h + 1][t >> 1];
          widen4<kE4m3>(__byte_perm(x, y, t & 1 ? 0x7362 : 0x5140) ^ kFlip, a[2 * h], a[2 * h + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816(o[nt][t], a[0], a[1], a[2], a[3], b[nt][0], b[nt][1]);
      }
    }
    __syncwarp();
    if (lane == 0) tg::mbar_arrive(&S.empty[sv]);
    r += 2;
    first = c.j + 1 == c.nt || u + 1 == n;   // the last unit of its item here
    if (first && head) {
      // CTA c and item i (numbered over all sequences): slot c + i grows along the units
      const int64_t slot = (static_cast<int64_t>(blockIdx.x + c.b * tg::head_groups(A) + c.group) * A.hw * A.kw + warp) * rows;
      float* pl = tg::part_ml(A, rows, DH) + slot * 2;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = l[nt][e];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
          const int row = 8 * nt + 2 * i4 + e;
          if (row >= rows) continue;
          float* p = A.part + (slot + row) * DH + DH / 8 * g;   // the thread's dims
#pragma unroll
          for (int h = 0; h < kT / 2; ++h)
            *reinterpret_cast<float4*>(p + 4 * h) =
                make_float4(o[nt][2 * h][e], o[nt][2 * h][2 + e], o[nt][2 * h + 1][e], o[nt][2 * h + 1][2 + e]);
          if (g == 0) *reinterpret_cast<float2*>(pl + 2 * row) = make_float2(m[nt][e], sum);
        }
    }
    c.advance(A, Q);
  }
  if (loader && S.abort_flag)   // let copies in flight land before the CTA exits
    for (int i = S.issued > C::kRing ? S.issued - C::kRing : 0; i < S.issued; ++i)
      wait(&S.full[i % C::kRing], (i / C::kRing) & 1, A.status, nullptr);
}

template <int kType, int DH, int NT>
tg_status launch(const TreeArgs& a, cudaStream_t st) {
  using C = Cfg<DH, NT>;
  CUtensorMap tk, tv;
  if (!tg::tree_cache_map(a, a.kc, DH, true, a.unit, a.hw, &tk) ||
      !tg::tree_cache_map(a, a.vc, DH, true, a.unit, a.hw, &tv))
    return TG_ERR_CUDA;
  constexpr int fixed = sizeof(RowSmem<DH, NT>) + 1024;
  static_assert((fixed + 1024 + 512) * C::kCtas <= 233472, "an SM's shared memory");
  auto with_seqs = [](int batch) { return fixed + 9 * batch + 8; };
  const int smem = with_seqs(a.batch);
  // the limit that the largest batch needs, so that batches that grow do not raise it step by step
  if (!tg::ensure_smem(reinterpret_cast<const void*>(tree_rows_kernel<kType, DH, NT>), with_seqs(tg::kTreeMaxBatch)))
    return TG_ERR_CUDA;
  return tg::launch(tree_rows_kernel<kType, DH, NT>, dim3(a.n_cta), dim3(C::kThreads), smem, st, 0, tk, tv, a);
}

template <int kType>
tg_status launch_type(const TreeArgs& a, int head_dim, cudaStream_t st) {
  const bool one = a.group * a.n_draft <= 8;
  if (head_dim == 128) return one ? launch<kType, 128, 1>(a, st) : launch<kType, 128, 2>(a, st);
  return one ? launch<kType, 64, 1>(a, st) : launch<kType, 64, 2>(a, st);
}

}  // namespace

int tg::tree_rows_ctas(int rows) { return 148 * (rows <= 8 ? Cfg<128, 1>::kCtas : Cfg<128, 2>::kCtas); }
int tg::tree_rows_warps(int rows) { return rows <= 8 ? Cfg<128, 1>::kWarps : Cfg<128, 2>::kWarps; }

tg_status tg::launch_tree_rows(const TreeArgs& a, int head_dim, tg_dtype cache_dtype, cudaStream_t stream) {
  return cache_dtype == TG_I8 ? launch_type<TG_I8>(a, head_dim, stream) : launch_type<TG_E4M3>(a, head_dim, stream);
}
