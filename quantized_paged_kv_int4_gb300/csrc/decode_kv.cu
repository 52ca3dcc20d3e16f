// kvq_decode_kv: split paged decode attention of one query token per sequence over a 16-bit or FP8
// (E4M3FN) paged cache.
//
// Mathematics: for sequence b, query head hq and its kv head, S_n = scale q . k_n over the sequence's
// keys, one pass with a running reference m: l = sum 2^(S - m), acc = sum 2^(S - m) v_n, both in fp32;
// o = acc / l and lse = m + log2 l hold for any m, so m moves (and rescales) only when a score passes
// m + kSlack. Pieces of a sequence are joined by their log-sum-exps (merge_kernel, decode_common.cuh).
//
// What bounds it: HBM. A key and a value of D elements serve the Hq / Hk query heads of their kv head
// with 4 D Hq / Hk operations, two orders of magnitude below the tensor rate.
//
// One warp serves one (kv head, block of 8 NT query heads) over a run of 16-token tiles, with nothing
// shared between warps. Both products are mma.m16n8k16 with the 16 tokens of a tile as rows of the
// scores (S^T = K Q^T) and as the depth of the output (O^T = V^T P^T): the operand rows come straight
// from global memory into registers, 16 bytes a lane, because the order of the head dimension inside a
// k-step and of the output rows inside an m-tile is free as long as both operands agree:
//   K: lane (g, t) reads rows g and g + 8, chunk c = dims 32 c + 8 t .. + 7 (FP8: 64 c + 16 t .. + 15);
//      the query fragments are read with the same order;
//   V: lane (g, t) reads tokens 2t, 2t + 1, 2t + 8, 2t + 9 at the dims of chunk g; a byte permute of two
//      tokens' words gives the operand's token pairs.
// P goes from the score layout to the operand layout by a transposing warp move (movmatrix).
//
// Operands. 16-bit caches enter as they are. FP8 codes become fp16, exactly; q becomes fp16 times 2^-k, k
// for each query head from its largest element, which keeps every bf16 element within 2^-29 of the
// largest exactly (query_shift, decode_common.cuh). P is fp16 for fp16 and FP8 caches (relative 2^-11 a
// weight). For bf16 caches it would be bf16 (2^-8), as large as the rounding of the output itself: there P
// enters as bf16 hi + lo, relative 2^-16, in two products, which for Hq / Hk <= 4 are the two halves of
// one product's columns.

#include "decode_common.cuh"
#include "kvq_host.h"

namespace kvq {

__device__ unsigned g_flags_decode_kv = 0;

constexpr float kSlack = 8.f;  // a weight is at most 2^8: fp16 keeps 2^-14 .. 2^8 at full precision

struct KvParams {
  SplitArgs s;  // max_blocks in 16-token pages
  const void *q;
  const uint8_t *k, *v;
  long long k_block, k_token, k_head, v_block, v_token, v_head;  // bytes
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  int32_t bt_stride, bs;
  long long num_blocks;
  int32_t q_f16;       // q is fp16 (else bf16)
  int32_t col_blocks;  // blocks of 8 NT query heads per kv head
  float sc_log2;       // softmax_scale * log2(e)
  float cap2, inv_cap2;  // soft cap in base 2
  const float *alibi;
};

enum : int { KV_BF16 = 0, KV_F16 = 1, KV_E4M3 = 2 };

template <int D, int CT, int NT>
struct KvGeom {
  static constexpr int ES = CT == KV_E4M3 ? 1 : 2;
  static constexpr int ROW = D * ES;               // bytes of a row
  static constexpr int KC = ROW / 64;              // 16-byte chunks per lane of a K row
  static constexpr int VB = ROW / 8 < 16 ? ROW / 8 : 16;  // bytes of a lane's V chunk
  static constexpr int VC = ROW / (8 * VB);        // chunks per lane of a V row
  static constexpr int MT = D / 16;                // output m-tiles
  static constexpr int KS = D / 16;                // k-steps
  // tiles in flight: 8 KB of K and V for each warp
  static constexpr int U = ROW >= 256 ? 1 : (ROW == 128 ? 2 : 4);
};

__device__ __forceinline__ uint4 ldg_stream16(const uint8_t *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ldg_stream8(const uint8_t *p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return static_cast<uint32_t>(r.x) | (static_cast<uint32_t>(r.y) << 16);
}
template <int CT>
__device__ __forceinline__ void mma_kv(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  if constexpr (CT == KV_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    mma_f16_16816(c, a0, a1, a2, a3, b0, b1);
}
__device__ __forceinline__ uint32_t bf2_as_u32(__nv_bfloat162 b) { return *reinterpret_cast<uint32_t *>(&b); }
__device__ __forceinline__ uint32_t word(const uint4 &r, int i) { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }

// One warp, one piece [t0, t1) of sequence b: kv head h, query heads h G + 8 NT cb .. of it; the warp takes
// every warps_per_head-th tile. FOLD (bf16, G <= 4): columns 4 .. 7 repeat the heads of columns 0 .. 3 and
// take the low parts of P.
template <int D, int CT, int NT, bool FOLD, bool MODS>
__device__ __forceinline__ void kv_piece(const KvParams &p, int b, int h, int cb, int sub, int t0, int t1, int L,
                                         long long slot) {
  using Gm = KvGeom<D, CT, NT>;
  constexpr int U = Gm::U;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int G = p.s.G, WPH = p.s.warps_per_head, c0 = cb * 8 * NT;  // first query head of the block

  const int first = t0 / kPage + sub, last = (t1 - 1) / kPage;
  const int n_my = first <= last ? (last - first) / WPH + 1 : 0;
  const int32_t *bt = p.block_table + static_cast<long long>(b) * p.bt_stride;
  const int tpb = p.bs / kPage;  // tiles of a block
  auto load_ids = [&](int batch) -> int {
    const int i = batch * 32 + lane;
    return i < n_my ? __ldg(bt + (first + i * WPH) / tpb) : -1;
  };
  int ids = load_ids(0), ids_next = load_ids(1), batch = 0;

  // the query fragments, b0 / b1 of k-step ks
  uint32_t qf[NT][Gm::KS][2];
  float sc[NT][2];   // score scale of columns 2t, 2t + 1
  float slope[NT][2];
  const float k_scale = CT == KV_E4M3 && p.k_scale != nullptr ? __ldg(p.k_scale + h) : 1.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int col = FOLD ? (g & 3) : c0 + 8 * nt + g;
    const bool live = col < G;
    const uint8_t *qr = static_cast<const uint8_t *>(p.q) +
                        (static_cast<long long>(b) * p.s.Hq + static_cast<long long>(h) * G + (live ? col : 0)) * D * 2;
    if constexpr (CT != KV_E4M3) {
#pragma unroll
      for (int c = 0; c < Gm::KC; ++c) {
        const uint4 r = live ? __ldg(reinterpret_cast<const uint4 *>(qr + 64 * c + 16 * t)) : make_uint4(0, 0, 0, 0);
        qf[nt][2 * c][0] = r.x;
        qf[nt][2 * c][1] = r.y;
        qf[nt][2 * c + 1][0] = r.z;
        qf[nt][2 * c + 1][1] = r.w;
      }
      sc[nt][0] = sc[nt][1] = p.sc_log2;
    } else {
      uint32_t w[2 * Gm::KS];  // element pairs: chunk c's 16 dims are words 8 c .. 8 c + 7
      float big = 0.f;
#pragma unroll
      for (int c = 0; c < Gm::KC; ++c) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint4 r = live ? __ldg(reinterpret_cast<const uint4 *>(qr + 128 * c + 32 * t + 16 * hf)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[8 * c + 4 * hf + i] = word(r, i);
        }
      }
      auto pair = [&](uint32_t x) {
        return p.q_f16 ? __half22float2(u32_as_h2(x))
                       : make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
      };
#pragma unroll
      for (int i = 0; i < 2 * Gm::KS; ++i) {
        const float2 f = pair(w[i]);
        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      big = fmaxf(big, __shfl_xor_sync(FULL, big, 1));
      big = fmaxf(big, __shfl_xor_sync(FULL, big, 2));
      const int k = query_shift(big, 0, live ? &g_flags_decode_kv : nullptr);
      const float down = pow2i(-k), up = pow2i(k) * p.sc_log2 * k_scale;
#pragma unroll
      for (int ks = 0; ks < Gm::KS; ++ks) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 f = pair(w[2 * ks + i]);
          qf[nt][ks][i] = h2_as_u32(__floats2half2_rn(f.x * down, f.y * down));
        }
      }
      sc[nt][0] = __shfl_sync(FULL, up, 8 * t);  // column 2t is lane g = 2t's
      sc[nt][1] = __shfl_sync(FULL, up, 8 * t + 4);
    }
    if constexpr (MODS) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int cc = FOLD ? ((2 * t + i) & 3) : c0 + 8 * nt + 2 * t + i;
        slope[nt][i] = p.alibi != nullptr && cc < G ? __ldg(p.alibi + h * G + cc) * 1.4426950408889634f : 0.f;
      }
    }
  }

  float m[NT][2], l[NT][2], acc[NT][Gm::MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = -INFINITY;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < Gm::MT; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
  }

  const uint8_t *kh = p.k + h * p.k_head + g * p.k_token + 16 * t;
  const uint8_t *vh = p.v + h * p.v_head + 2 * t * p.v_token + Gm::VB * g;
  // Tile i of the warp: its block and its place in it. A tile past the end or in a bad block gives an
  // offset inside the pool (block 0) and no live tokens.
  struct Tile {
    long long blk;
    int row, pos, lo, hi;  // live tokens [lo, hi) of the tile
  };
  auto tile_of = [&](int i) -> Tile {
    if (i < n_my && (i >> 5) != batch) {  // warp-uniform
      batch = i >> 5;
      ids = ids_next;
      ids_next = load_ids(batch + 1);
    }
    const int id = __shfl_sync(FULL, ids, i & 31);
    Tile x;
    const int page = first + i * WPH;
    x.pos = page * kPage;
    const bool in = i < n_my, ok = in && id >= 0 && id < p.num_blocks;
    if (in && !ok && lane == 0) atomicOr(&g_flags_decode_kv, ERR_BLOCK);
    x.blk = ok ? id : 0;
    x.row = ok ? (page % tpb) * kPage : 0;
    x.lo = ok ? max(t0 - x.pos, 0) : 0;
    x.hi = ok ? min(t1 - x.pos, kPage) : 0;
    return x;
  };
  uint4 kr[U][2][Gm::KC];
  Tile tile[U], next[U];
  auto load_k = [&](const Tile &x, uint4 (&r)[2][Gm::KC]) {
    const uint8_t *src = kh + x.blk * p.k_block + x.row * p.k_token;
#pragma unroll
    for (int c = 0; c < Gm::KC; ++c) {
      r[0][c] = ldg_stream16(src + 64 * c);
      r[1][c] = ldg_stream16(src + 8 * p.k_token + 64 * c);
    }
  };
  if (n_my > 0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      tile[u] = tile_of(u);
      load_k(tile[u], kr[u]);
    }
  }

  for (int i0 = 0; i0 < n_my; i0 += U) {
    // ---- values of this step on their way
    uint32_t vr[U][4][Gm::VC * Gm::VB / 4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t *src = vh + tile[u].blk * p.v_block + tile[u].row * p.v_token;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint8_t *r = src + ((j & 1) + 8 * (j >> 1)) * p.v_token;
#pragma unroll
        for (int c = 0; c < Gm::VC; ++c) {
          if constexpr (Gm::VB == 16) {
            const uint4 x = ldg_stream16(r + 128 * c);
            vr[u][j][4 * c] = x.x;
            vr[u][j][4 * c + 1] = x.y;
            vr[u][j][4 * c + 2] = x.z;
            vr[u][j][4 * c + 3] = x.w;
          } else {
            const uint2 x = ldg_stream8(r);
            vr[u][j][0] = x.x;
            vr[u][j][1] = x.y;
          }
        }
      }
    }
    // ---- scores: rows are tokens g, g + 8, columns 2t, 2t + 1
    float S[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[u][nt][0] = S[u][nt][1] = S[u][nt][2] = S[u][nt][3] = 0.f;
#pragma unroll
      for (int c = 0; c < Gm::KC; ++c) {
        if constexpr (CT != KV_E4M3) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_kv<CT>(S[u][nt], word(kr[u][0][c], 2 * hf), word(kr[u][1][c], 2 * hf), word(kr[u][0][c], 2 * hf + 1),
                         word(kr[u][1][c], 2 * hf + 1), qf[nt][2 * c + hf][0], qf[nt][2 * c + hf][1]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = word(kr[u][0][c], w), y = word(kr[u][1][c], w);
            const uint32_t a0 = e4m3x2_f16x2(x & 0xffffu), a2 = e4m3x2_f16x2(x >> 16);
            const uint32_t a1 = e4m3x2_f16x2(y & 0xffffu), a3 = e4m3x2_f16x2(y >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_kv<CT>(S[u][nt], a0, a1, a2, a3, qf[nt][4 * c + w][0], qf[nt][4 * c + w][1]);
          }
        }
      }
    }
    // ---- keys of the next step on their way
    const bool more = i0 + U < n_my;
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        next[u] = tile_of(i0 + U + u);
        load_k(next[u], kr[u]);
      }
    }
    // ---- weights
    bool above = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = S[u][nt][e] * sc[nt][e & 1];
          if constexpr (MODS) {
            if (p.cap2 > 0.f) x = p.cap2 * tanhf(x * p.inv_cap2);
            x = fmaf(slope[nt][e & 1], static_cast<float>(tile[u].pos + g + 8 * (e >> 1) - (L - 1)), x);
          }
          const int row = g + 8 * (e >> 1);
          x = row >= tile[u].lo && row < tile[u].hi ? x : -INFINITY;
          S[u][nt][e] = x;
          above |= x > m[nt][e & 1] + kSlack;
        }
      }
    }
    if (__any_sync(FULL, above)) {  // the references move up to the step's largest scores
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float top = m[nt][i];
#pragma unroll
          for (int u = 0; u < U; ++u) top = fmaxf(top, fmaxf(S[u][nt][i], S[u][nt][i + 2]));
          top = warp_max_g(top);
          const float al = m[nt][i] == top ? 1.f : fast_exp2(m[nt][i] - top);
          m[nt][i] = top;
          l[nt][i] *= al;
#pragma unroll
          for (int k = 0; k < Gm::MT; ++k) {
            acc[nt][k][i] *= al;
            acc[nt][k][i + 2] *= al;
          }
        }
      }
    }
    // ---- P in operand order: b0 tokens 2t, 2t + 1, b1 tokens 2t + 8, 2t + 9 of column g
    uint32_t ph[U][NT][2], pl[U][NT][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float ref = m[nt][e & 1];
          w[e] = fast_exp2(S[u][nt][e] - (ref == -INFINITY ? 0.f : ref));
          l[nt][e & 1] += w[e];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (CT == KV_BF16) {
            const __nv_bfloat162 hi = __floats2bfloat162_rn(w[2 * r], w[2 * r + 1]);
            const __nv_bfloat162 lo = __floats2bfloat162_rn(w[2 * r] - __low2float(hi), w[2 * r + 1] - __high2float(hi));
            if constexpr (FOLD) {
              ph[u][nt][r] = movmatrix_trans(t < 2 ? bf2_as_u32(hi) : bf2_as_u32(lo));
            } else {
              ph[u][nt][r] = movmatrix_trans(bf2_as_u32(hi));
              pl[u][nt][r] = movmatrix_trans(bf2_as_u32(lo));
            }
          } else {
            ph[u][nt][r] = movmatrix_trans(h2_as_u32(__floats2half2_rn(w[2 * r], w[2 * r + 1])));
          }
        }
      }
    }
    // ---- values of dead tokens may be anything: zero them (0 * NaN is NaN)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (tile[u].lo > 0 || tile[u].hi < kPage) {  // warp-uniform
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = 2 * t + (j & 1) + 8 * (j >> 1);
          if (row < tile[u].lo || row >= tile[u].hi) {
#pragma unroll
            for (int c = 0; c < Gm::VC * Gm::VB / 4; ++c) vr[u][j][c] = 0;
          }
        }
      }
    }
    // ---- O^T += V^T P^T
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int c = 0; c < Gm::VC * Gm::VB / 4; ++c) {
        const uint32_t va = vr[u][0][c], vb = vr[u][1][c], vc = vr[u][2][c], vd = vr[u][3][c];
        if constexpr (CT != KV_E4M3) {
          const uint32_t a0 = __byte_perm(va, vb, 0x5410), a1 = __byte_perm(va, vb, 0x7632);
          const uint32_t a2 = __byte_perm(vc, vd, 0x5410), a3 = __byte_perm(vc, vd, 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_kv<CT>(acc[nt][c], a0, a1, a2, a3, ph[u][nt][0], ph[u][nt][1]);
            if constexpr (CT == KV_BF16 && !FOLD) mma_kv<CT>(acc[nt][c], a0, a1, a2, a3, pl[u][nt][0], pl[u][nt][1]);
          }
        } else {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {  // dims 4 c + 2 hf, + 1 of the lane's chunk: one m-tile
            const uint32_t sel = hf ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(va, vb, sel), y = __byte_perm(vc, vd, sel);
            const uint32_t a0 = e4m3x2_f16x2(x & 0xffffu), a1 = e4m3x2_f16x2(x >> 16);
            const uint32_t a2 = e4m3x2_f16x2(y & 0xffffu), a3 = e4m3x2_f16x2(y >> 16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_kv<CT>(acc[nt][2 * c + hf], a0, a1, a2, a3, ph[u][nt][0], ph[u][nt][1]);
          }
        }
      }
    }
    if (more) {
#pragma unroll
      for (int u = 0; u < U; ++u) tile[u] = next[u];
    }
  }

  // ---- the piece's partial: column n, dims EPC g' .. of the lane's chunks (two for each m-tile)
  constexpr int DPL = Gm::VC * Gm::VB / Gm::ES / Gm::VC;  // dims of a chunk
  const long long row0 = (slot * WPH + sub) * p.s.Hq + static_cast<long long>(h) * G;
  const float v_scale = CT == KV_E4M3 && p.v_scale != nullptr ? __ldg(p.v_scale + h) : 1.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float sum = warp_sum_g(l[nt][i]);
      const float inv = sum > 0.f ? v_scale / sum : (sum == 0.f ? 0.f : sum);  // NaN stays
      float o[2 * Gm::MT];
#pragma unroll
      for (int k = 0; k < Gm::MT; ++k) {
        float x = acc[nt][k][i], y = acc[nt][k][i + 2];
        if constexpr (FOLD) {
          x += __shfl_xor_sync(FULL, x, 2);
          y += __shfl_xor_sync(FULL, y, 2);
        }
        o[2 * k] = x * inv;
        o[2 * k + 1] = y * inv;
      }
      const int col = c0 + 8 * nt + 2 * t + i;
      if (col < G && (!FOLD || t < 2)) {
        float *dst = p.s.part_o + (row0 + col) * D + DPL * g;
#pragma unroll
        for (int k = 0; k < 2 * Gm::MT; k += 4)
          *reinterpret_cast<float4 *>(dst + (k / DPL) * 8 * DPL + k % DPL) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        if (g == 0) p.s.part_lse[row0 + col] = sum == 0.f ? -INFINITY : m[nt][i] + log2f(sum);
      }
    }
  }
}

// Calls seg(b, t0, t1, L, slot) for every sequence piece of this CTA, on the partition that merge_kernel
// recomputes (decode_common.cuh): fixed splits of the keys that the window leaves, or runs of the
// concatenated pages.
template <int THREADS, typename SegFn>
__device__ __forceinline__ void kv_pieces(const SplitArgs &a, unsigned *flags, SegFn &&seg) {
  if (a.num_splits > 0) {
    const int b = blockIdx.x / a.num_splits, s = blockIdx.x % a.num_splits;
    const SeqSpan sp = seq_span(a, b, threadIdx.x == 0 && s == 0 && blockIdx.y == 0 ? flags : nullptr);
    const int span = (sp.L - sp.lo + a.num_splits - 1) / a.num_splits;
    const long long t0 = sp.lo + static_cast<long long>(s) * span;
    const int t1 = static_cast<int>(min(t0 + span, static_cast<long long>(sp.L)));
    if (t0 < t1) seg(b, static_cast<int>(t0), t1, sp.L, static_cast<long long>(blockIdx.x));
    return;
  }
  __shared__ long long s_scan[THREADS / 32];
  __shared__ long long s_first_p;
  __shared__ int s_first_b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](long long v, long long *total) -> long long {  // inclusive, over the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(FULL, v, o);
      if (lane >= o) v += n;
    }
    if (lane == 31) s_scan[warp] = v;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const long long x = s_scan[w];
      if (w < warp) before += x;
      all += x;
    }
    __syncthreads();
    *total = all;
    return v + before;
  };
  const bool report = blockIdx.x == 0 && blockIdx.y == 0;
  const long long C = gridDim.x, c = blockIdx.x;
  long long pages = 0;
  long long keep_np = 0, keep_incl = 0;  // this thread's sequence, when one round covers the batch
  for (int base = 0; base < a.B; base += THREADS) {
    const int b = base + threadIdx.x;
    const long long np = b < a.B ? seq_span(a, b, report ? flags : nullptr).np : 0;
    long long chunk;
    const long long incl = scan(np, &chunk);
    keep_np = np;
    keep_incl = incl;
    pages += chunk;
  }
  const long long q = pages / C, r = pages % C;
  const long long pb = c * q + min(c, r), pe = pb + q + (c < r ? 1 : 0);
  if (pb >= pe) return;
  if (threadIdx.x == 0) s_first_b = -1;
  __syncthreads();
  long long running = 0;
  for (int base = 0; base < a.B; base += THREADS) {
    const int b = base + threadIdx.x;
    long long np = keep_np, incl = keep_incl;
    if (a.B > THREADS) {
      np = b < a.B ? seq_span(a, b, nullptr).np : 0;
      long long chunk;
      incl = scan(np, &chunk) + running;
      running += chunk;
    }
    const long long excl = incl - np;
    if (np > 0 && excl <= pb && pb < incl) {
      s_first_b = b;
      s_first_p = excl;
    }
    __syncthreads();
    if (s_first_b >= 0) break;  // uniform: written before the barrier, at most once
    __syncthreads();
  }
  int b = s_first_b;
  long long P = s_first_p;
  while (P < pe && b >= 0 && b < a.B) {
    const SeqSpan sp = seq_span(a, b, nullptr);
    if (sp.np > 0) {
      const long long lo = max(pb, P) - P, hi = min(pe, P + sp.np) - P;
      const int t0 = max(static_cast<int>((sp.f + lo) * kPage), sp.lo);
      const int t1 = static_cast<int>(min((sp.f + hi) * kPage, static_cast<long long>(sp.L)));
      if (threadIdx.x == 0 && blockIdx.y == 0) {
        if (P >= pb) a.seg_first[b] = static_cast<int>(c);
        if (P + sp.np <= pe) a.seg_last[b] = static_cast<int>(c);
      }
      seg(b, t0, t1, sp.L, c + b);
    }
    P += sp.np;
    ++b;
  }
}

constexpr int kKvWarps = 4;
constexpr int kKvMaxResident = 3;  // CTAs of an SM, by registers: 3 at up to 168, else 2
template <int D, int CT, int NT>
constexpr int kv_resident() { return NT == 1 && D < 256 && CT != KV_E4M3 ? 3 : 2; }

template <int D, int CT, int NT, bool FOLD, bool MODS>
__global__ void __launch_bounds__(32 * kKvWarps, kv_resident<D, CT, NT>()) decode_kv_kernel(const __grid_constant__ KvParams p) {
  asm volatile("griddepcontrol.launch_dependents;");  // let the merge kernel's launch begin early
  const int warp = threadIdx.x >> 5;
  const int hv = blockIdx.y * p.s.heads_per_cta + warp % p.s.heads_per_cta;  // (kv head, block of query heads)
  const int h = hv / p.col_blocks, cb = hv % p.col_blocks, sub = warp / p.s.heads_per_cta;
  kv_pieces<32 * kKvWarps>(p.s, &g_flags_decode_kv, [&](int b, int t0, int t1, int L, long long slot) {
    kv_piece<D, CT, NT, FOLD, MODS>(p, b, h, cb, sub, t0, t1, L, slot);
  });
}

bool take_flags_decode_kv(cudaStream_t stream, unsigned *host_word) {
  static const unsigned zero = 0;
  if (cudaMemcpyFromSymbolAsync(host_word, g_flags_decode_kv, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream) !=
      cudaSuccess)
    return false;
  return cudaMemcpyToSymbolAsync(g_flags_decode_kv, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream) ==
         cudaSuccess;
}

// Blocks of query heads: 8 columns when a kv head has at most 8 of them, else 16 (D = 256: 8, the
// accumulators of 16 would not fit the registers).
static int kv_tiles(int G, int D) { return G <= 8 || D == 256 ? 1 : 2; }

static bool kv_plan(int B, int Hq, int Hk, int D, int num_splits, SplitPlan *plan) {
  const int G = Hq / Hk, cols = 8 * kv_tiles(G, D);
  const long long units = static_cast<long long>(Hk) * ((G + cols - 1) / cols);
  int hpc = kKvWarps;
  while (units % hpc) hpc /= 2;
  plan->heads_per_cta = hpc;
  plan->head_groups = static_cast<int>(units / hpc);
  plan->warps_per_head = kKvWarps / hpc;
  if (units / hpc > 65535) return false;
  if (num_splits > 0) {
    const long long ctas = static_cast<long long>(B) * num_splits;
    if (ctas > 0x7fffffffLL) return false;
    plan->seg_ctas = static_cast<int>(ctas);
    plan->slots = ctas;
  } else {
    const int sms = sm_count();
    if (sms <= 0) return false;
    plan->seg_ctas = (kKvMaxResident * sms + plan->head_groups - 1) / plan->head_groups;
    plan->slots = static_cast<long long>(plan->seg_ctas) + B;
  }
  return true;
}

template <int D, int CT, int NT, bool FOLD>
static kvq_status launch_kv(KvParams &p, const SplitPlan &plan, bool mods, cudaStream_t s) {
  if (p.s.num_splits == 0)  // one wave: the workspace has room for kKvMaxResident CTAs of an SM
    p.s.seg_ctas = (kv_resident<D, CT, NT>() * sm_count() + plan.head_groups - 1) / plan.head_groups;
  const dim3 grid(p.s.seg_ctas, plan.head_groups);
  if (mods)
    decode_kv_kernel<D, CT, NT, FOLD, true><<<grid, 32 * kKvWarps, 0, s>>>(p);
  else
    decode_kv_kernel<D, CT, NT, FOLD, false><<<grid, 32 * kKvWarps, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return KVQ_ERR_CUDA;
  const long long rows = static_cast<long long>(p.s.B) * p.s.Hq;
  if (launch_dependent(merge_kernel<D, true>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), s, p.s) != cudaSuccess)
    return KVQ_ERR_CUDA;
  return launch_status();
}

template <int D, int CT>
static kvq_status launch_kv_tiles(KvParams &p, const SplitPlan &plan, bool mods, cudaStream_t s) {
  if constexpr (D < 256) {
    if (kv_tiles(p.s.G, D) == 2) return launch_kv<D, CT, 2, false>(p, plan, mods, s);
  }
  if constexpr (CT == KV_BF16) {
    if (p.s.G <= 4) return launch_kv<D, CT, 1, true>(p, plan, mods, s);
  }
  return launch_kv<D, CT, 1, false>(p, plan, mods, s);
}

template <int D>
static kvq_status launch_kv_type(KvParams &p, const SplitPlan &plan, kvq_dtype dtype, bool mods, cudaStream_t s) {
  switch (dtype) {
    case KVQ_BF16: return launch_kv_tiles<D, KV_BF16>(p, plan, mods, s);
    case KVQ_F16: return launch_kv_tiles<D, KV_F16>(p, plan, mods, s);
    default: return launch_kv_tiles<D, KV_E4M3>(p, plan, mods, s);
  }
}

}  // namespace kvq

using namespace kvq;

extern "C" size_t kvq_decode_kv_workspace_bytes(int32_t B, int32_t Hq, int32_t Hk, int32_t D, int32_t num_splits) {
  if (B < 0 || Hq < 1 || Hk < 1 || Hq % Hk || num_splits < 0 || (D != 64 && D != 128 && D != 256)) return 0;
  SplitPlan plan;
  if (!kv_plan(B, Hq, Hk, D, num_splits, &plan)) return 0;
  return workspace_bytes(B, Hq, D, plan);
}

extern "C" kvq_status kvq_decode_kv(const void *q, kvq_dtype q_dtype, const kvq_paged_kv *cache,
                                    const int32_t *block_table, int32_t max_blocks, const int32_t *seq_lens,
                                    float softmax_scale, int32_t num_splits, void *workspace,
                                    size_t workspace_bytes, void *out, kvq_dtype out_dtype, int32_t B,
                                    int32_t Hq, int32_t Hk, int32_t D, const kvq_score_mods *mods,
                                    kvq_stream_t stream) {
  if (B < 0 || Hq < 1 || Hk < 1 || max_blocks < 0 || num_splits < 0 || cache == nullptr) return KVQ_ERR_INVALID_ARG;
  if (mods && (mods->sliding_window < 0 || !(mods->softcap >= 0.f) || !(mods->softcap < INFINITY) ||
               !aligned(mods->sinks, 4) || !aligned(mods->alibi_slopes, 4) || mods->q_len < 0 ||
               !aligned(mods->lse_out, 4)))
    return KVQ_ERR_INVALID_ARG;
  if (Hq % Hk != 0) return KVQ_ERR_INVALID_ARG;
  if (q_dtype != KVQ_BF16 && q_dtype != KVQ_F16) return KVQ_ERR_INVALID_ARG;
  if (out_dtype != KVQ_BF16 && out_dtype != KVQ_F16 && out_dtype != KVQ_F32) return KVQ_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return KVQ_ERR_UNSUPPORTED;
  if (mods && (mods->q_len > 1 || mods->query_start_loc != nullptr)) return KVQ_ERR_UNSUPPORTED;
  const kvq_status sc = check_paged_kv(cache, q_dtype);
  if (sc != KVQ_OK) return sc;
  if (cache->block_size % kPage) return KVQ_ERR_UNSUPPORTED;
  if (!(softmax_scale > 0.f) || !(softmax_scale < INFINITY)) return KVQ_ERR_INVALID_ARG;
  if (static_cast<long long>(max_blocks) * cache->block_size > 0x7fffffffLL - kPage) return KVQ_ERR_UNSUPPORTED;
  SplitPlan plan;
  if (!kv_plan(B, Hq, Hk, D, num_splits, &plan)) return KVQ_ERR_UNSUPPORTED;
  if (B == 0) return KVQ_OK;
  if (!q || !block_table || !seq_lens || !out || !workspace || max_blocks < 1) return KVQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(out, 16) ||
      !aligned(workspace, 16))
    return KVQ_ERR_INVALID_ARG;
  if (workspace_bytes < kvq::workspace_bytes(B, Hq, D, plan)) return KVQ_ERR_WORKSPACE;

  KvParams p = {};
  SplitArgs &sa = p.s;
  sa.seq_lens = seq_lens;
  sa.max_blocks = max_blocks * (cache->block_size / kPage);
  sa.num_splits = num_splits;
  sa.B = B;
  sa.Hq = Hq;
  sa.Hk = Hk;
  sa.G = Hq / Hk;
  sa.Q = 1;
  sa.heads_per_cta = plan.heads_per_cta;
  sa.warps_per_head = plan.warps_per_head;
  sa.seg_ctas = plan.seg_ctas;
  sa.slots = plan.slots;
  workspace_carve(workspace, B, Hq, D, plan, &sa.part_o, &sa.part_lse, &sa.seg_first, &sa.seg_last);
  sa.out = out;
  sa.out_dtype = out_dtype;
  sa.window = mods ? mods->sliding_window : 0;
  sa.sinks = mods ? mods->sinks : nullptr;
  sa.lse_out = mods ? mods->lse_out : nullptr;
  const long long es = cache->dtype == KVQ_E4M3 ? 1 : 2;
  p.q = q;
  p.q_f16 = q_dtype == KVQ_F16;
  p.k = static_cast<const uint8_t *>(cache->k);
  p.v = static_cast<const uint8_t *>(cache->v);
  p.k_block = cache->k_stride_block * es;
  p.k_token = cache->k_stride_token * es;
  p.k_head = cache->k_stride_head * es;
  p.v_block = cache->v_stride_block * es;
  p.v_token = cache->v_stride_token * es;
  p.v_head = cache->v_stride_head * es;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.block_table = block_table;
  p.bt_stride = max_blocks;
  p.bs = cache->block_size;
  p.num_blocks = cache->num_blocks;
  const int cols = 8 * kv_tiles(sa.G, D);
  p.col_blocks = (sa.G + cols - 1) / cols;
  p.sc_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  const double cap2 = mods ? static_cast<double>(mods->softcap) * 1.4426950408889634 : 0.0;
  p.cap2 = static_cast<float>(cap2);
  p.inv_cap2 = cap2 > 0.0 ? static_cast<float>(1.0 / cap2) : 0.f;
  p.alibi = mods ? mods->alibi_slopes : nullptr;
  const bool scored = p.cap2 > 0.f || p.alibi != nullptr;  // the window and the sinks need no kernel of their own
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 64) return launch_kv_type<64>(p, plan, cache->dtype, scored, s);
  if (D == 128) return launch_kv_type<128>(p, plan, cache->dtype, scored, s);
  return launch_kv_type<256>(p, plan, cache->dtype, scored, s);
}
