// kvq_rope and kvq_write_kv: rotary positions, and the write of new keys and values into a 16-bit or
// FP8 paged cache with the rotation in the same pass.
//
// Mathematics: pair i of a head turns by the angle positions[t] * f_i. f_i is a 64-bit fraction of a
// turn, so positions[t] * f_i mod 2^64 is the angle modulo a turn, exactly; its top 32 bits, signed,
// times 2^-31 are the angle in units of pi in [-1, 1), which sincospif takes as it is: no range
// reduction, and the same accuracy (2^-25 turns) at any position. cos and sin belong to the token,
// not to the head: a CTA computes them once into shared memory, and all heads of q and k use them.
//
// What bounds it: HBM. Every element is read once and written once. A thread moves 16-byte chunks:
// the two chunks of eight elements whose pairs belong together (half layout), or one (interleaved
// pairs, elements that pass, values). Products and sums are fp32 and rounded once, to the output's or
// the cache's type.
//
// Heads whose pairs do not keep to such chunks (rotary_dim / 2 not a multiple of 8, odd strides) take
// the element path: a thread owns a pair (or one element that passes), so that q_out == q stays safe.

#include "kvq_device.cuh"
#include "kvq_host.h"

namespace kvq {

__device__ unsigned g_flags_write_kv = 0;

struct RowSet {  // [T, heads, D] rows and where they go
  const void *src;
  void *dst;
  long long src_t, src_h, dst_t, dst_h;
  int32_t heads;
};

struct WriteKvParams {
  RowSet q, k, v;              // k.dst / v.dst: the pools when slots != null (dst_t unused)
  const int64_t *slots;
  long long k_block, k_token, v_block, v_token;  // pool strides in elements
  const float *k_scale, *v_scale;
  int32_t bs;
  long long num_blocks;
  const int32_t *positions;    // null: no rotation
  const uint64_t *freqs;
  int32_t half;                // rotary_dim / 2
  int32_t interleaved;
  float factor;
  int32_t T, D;
};

enum : int { kFp8Dst = 3 };  // destination type of the pools beside KVQ_BF16 / KVQ_F16 / KVQ_F32

template <int T>
__device__ __forceinline__ float load1(const void *p, long long i) {
  if constexpr (T == KVQ_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
  else if constexpr (T == KVQ_F16) return __half2float(static_cast<const __half *>(p)[i]);
  else return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ uint8_t to_fp8(float x, float scale) {
  const float y = __fdiv_rn(x, scale);  // the conversion itself saturates at 448 and keeps a NaN
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3));
}
template <int T>
__device__ __forceinline__ void store1(void *p, long long i, float x, float scale) {
  if constexpr (T == KVQ_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
  else if constexpr (T == KVQ_F16) static_cast<__half *>(p)[i] = __float2half_rn(x);
  else if constexpr (T == KVQ_F32) static_cast<float *>(p)[i] = x;
  else static_cast<uint8_t *>(p)[i] = to_fp8(x, scale);
}

template <int T>
__device__ __forceinline__ void load8(const void *p, long long i, float (&x)[8]) {
  if constexpr (T == KVQ_F32) {
    const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    const float4 a = s[0], b = s[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    const uint4 r = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (T == KVQ_BF16) {
        x[2 * j] = __uint_as_float(w[j] << 16);
        x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(u32_as_h2(w[j]));
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
      }
    }
  }
}
template <int T>
__device__ __forceinline__ void store8(void *p, long long i, const float (&x)[8], float scale) {
  if constexpr (T == KVQ_F32) {
    float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else if constexpr (T == kFp8Dst) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[j] |= static_cast<uint32_t>(to_fp8(x[4 * j + e], scale)) << (8 * e);
    }
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p) + i) = make_uint2(w[0], w[1]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (T == KVQ_BF16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
      } else {
        w[j] = h2_as_u32(__floats2half2_rn(x[2 * j], x[2 * j + 1]));
      }
    }
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// cos and sin of the token's pairs, times the factor, into shared memory
__device__ __forceinline__ void fill_angles(const WriteKvParams &p, int pos, float2 *cs) {
  for (int i = threadIdx.x; i < p.half; i += blockDim.x) {
    const uint64_t turn = static_cast<uint64_t>(static_cast<uint32_t>(pos)) * __ldg(p.freqs + i);  // mod 2^64: mod a turn
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31: units of pi
    float s, c;
    sincospif(x, &s, &c);
    cs[i] = make_float2(c * p.factor, s * p.factor);
  }
}

// IN: type of q, k, v and q_out / k_out. POOL: type of the pools (IN, or FP8), or -1: k_out, no cache.
template <int IN, int POOL, bool VEC>
__global__ void __launch_bounds__(256) write_kv_kernel(const WriteKvParams p) {
  extern __shared__ __align__(16) float2 kvq_angles[];
  const int t = blockIdx.x;
  const int pos = p.positions != nullptr ? __ldg(p.positions + t) : 0;
  if (pos < 0) return;  // padding
  long long slot = -1;
  if constexpr (POOL >= 0) {
    slot = __ldg(p.slots + t);
    if (slot >= p.num_blocks * p.bs) {
      if (threadIdx.x == 0) atomicOr(&g_flags_write_kv, ERR_SLOT);
      slot = -1;
    }
  }
  const bool rot = p.positions != nullptr;
  if (rot) {
    fill_angles(p, pos, kvq_angles);
    __syncthreads();
  }
  long long kd = 0, vd = 0;  // element offsets of the token in the pools
  if (POOL >= 0 && slot >= 0) {
    const long long blk = slot / p.bs, row = slot - blk * p.bs;
    kd = blk * p.k_block + row * p.k_token;
    vd = blk * p.v_block + row * p.v_token;
  }
  const bool kv = POOL < 0 || slot >= 0;
  const int half = rot ? p.half : 0, R = 2 * half;
  // items: a row's pairs (VEC: chunks of 8 pairs, or of 4 interleaved) and the elements that pass
  const int pass = VEC ? (p.D - R) / 8 : p.D - R;
  const int pairs = VEC ? (p.interleaved ? R / 8 : half / 8) : half;
  const int per = pairs + pass, rows = p.q.heads + (kv ? p.k.heads : 0);
  const int vper = VEC ? p.D / 8 : p.D, items = rows * per + (kv && POOL >= 0 ? p.v.heads * vper : 0);
  for (int i = threadIdx.x; i < items; i += blockDim.x) {
    int row, j, which;
    if (i < rows * per) {
      row = i / per;
      j = i - row * per;
      which = row < p.q.heads ? 0 : 1;
      if (which) row -= p.q.heads;
    } else {
      row = (i - rows * per) / vper;
      j = (i - rows * per) - row * vper + pairs;  // past the pairs: passes
      which = 2;
    }
    const RowSet &rs = which == 0 ? p.q : which == 1 ? p.k : p.v;
    const long long so = t * rs.src_t + row * rs.src_h;
    const bool pool = POOL >= 0 && which != 0;
    const long long dd = (pool ? (which == 1 ? kd : vd) : t * rs.dst_t) + row * rs.dst_h;
    float scale = 1.f;
    if constexpr (POOL == kFp8Dst) {
      const float *sc = which == 1 ? p.k_scale : p.v_scale;
      if (pool && sc != nullptr) scale = __ldg(sc + row);
    }
    const int d0 = which == 2 ? 0 : R;  // first element that passes
    if constexpr (VEC) {
      auto put = [&](long long d, const float (&x)[8]) {
        if constexpr (POOL >= 0) {
          if (pool) {
            store8<POOL>(rs.dst, dd + d, x, scale);
            return;
          }
        }
        store8<IN>(rs.dst, dd + d, x, scale);
      };
      float x[8];
      if (j >= pairs) {
        const int d = d0 + 8 * (j - pairs);
        load8<IN>(rs.src, so + d, x);
        put(d, x);
      } else if (p.interleaved) {
        load8<IN>(rs.src, so + 8 * j, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 cs = kvq_angles[4 * j + e];
          const float a = x[2 * e], b = x[2 * e + 1];
          x[2 * e] = a * cs.x - b * cs.y;
          x[2 * e + 1] = b * cs.x + a * cs.y;
        }
        put(8 * j, x);
      } else {
        float y[8];
        load8<IN>(rs.src, so + 8 * j, x);
        load8<IN>(rs.src, so + half + 8 * j, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 cs = kvq_angles[8 * j + e];
          const float a = x[e], b = y[e];
          x[e] = a * cs.x - b * cs.y;
          y[e] = b * cs.x + a * cs.y;
        }
        put(8 * j, x);
        put(half + 8 * j, y);
      }
    } else {
      auto put = [&](long long d, float x) {
        if constexpr (POOL >= 0) {
          if (pool) {
            store1<POOL>(rs.dst, dd + d, x, scale);
            return;
          }
        }
        store1<IN>(rs.dst, dd + d, x, scale);
      };
      if (j >= pairs) {
        const int d = d0 + j - pairs;
        put(d, load1<IN>(rs.src, so + d));
      } else {
        const int da = p.interleaved ? 2 * j : j, db = p.interleaved ? 2 * j + 1 : j + half;
        const float2 cs = kvq_angles[j];
        const float a = load1<IN>(rs.src, so + da), b = load1<IN>(rs.src, so + db);
        put(da, a * cs.x - b * cs.y);
        put(db, b * cs.x + a * cs.y);
      }
    }
  }
}

bool take_flags_write_kv(cudaStream_t stream, unsigned *host_word) {
  static const unsigned zero = 0;
  if (cudaMemcpyFromSymbolAsync(host_word, g_flags_write_kv, sizeof(unsigned), 0, cudaMemcpyDeviceToHost, stream) !=
      cudaSuccess)
    return false;
  return cudaMemcpyToSymbolAsync(g_flags_write_kv, &zero, sizeof(unsigned), 0, cudaMemcpyHostToDevice, stream) ==
         cudaSuccess;
}

// The chunk path's conditions on one row set.
static bool chunked(const RowSet &r) {
  return r.heads == 0 || (aligned(r.src, 16) && aligned(r.dst, 16) && r.src_t % 8 == 0 && r.src_h % 8 == 0 &&
                          r.dst_t % 8 == 0 && r.dst_h % 8 == 0);
}
static bool chunked_pairs(const WriteKvParams &p) {
  return p.D % 8 == 0 && (p.positions == nullptr || (p.interleaved ? p.half % 4 == 0 : p.half % 8 == 0));
}

template <int IN, int POOL>
static kvq_status launch_write_kv(const WriteKvParams &p, bool vec, cudaStream_t s) {
  const size_t smem = p.positions != nullptr ? static_cast<size_t>(p.half) * sizeof(float2) : 0;
  if (vec)
    write_kv_kernel<IN, POOL, true><<<p.T, 256, smem, s>>>(p);
  else
    write_kv_kernel<IN, POOL, false><<<p.T, 256, smem, s>>>(p);
  return launch_status();
}

static kvq_status check_rotary(const kvq_rotary *r, int D, WriteKvParams *p) {
  p->positions = nullptr;
  p->freqs = nullptr;
  p->half = 0;
  p->interleaved = 0;
  p->factor = 1.f;
  if (r == nullptr) return KVQ_OK;
  if (r->rotary_dim < 2 || r->rotary_dim % 2 || r->rotary_dim > D) return KVQ_ERR_INVALID_ARG;
  if (!(r->attn_factor > -INFINITY) || !(r->attn_factor < INFINITY)) return KVQ_ERR_INVALID_ARG;
  if (!r->positions || !r->freqs || !aligned(r->positions, 4) || !aligned(r->freqs, 8)) return KVQ_ERR_INVALID_ARG;
  p->positions = r->positions;
  p->freqs = r->freqs;
  p->half = r->rotary_dim / 2;
  p->interleaved = r->interleaved != 0;
  p->factor = r->attn_factor;
  return KVQ_OK;
}

}  // namespace kvq

using namespace kvq;

extern "C" kvq_status kvq_rope_frequencies(int32_t rotary_dim, double base, const kvq_rope_scaling *scaling,
                                           uint64_t *freqs, float *attn_factor) {
  if (rotary_dim < 2 || rotary_dim % 2 || !(base > 1.0) || !(base < INFINITY) || !freqs || !attn_factor)
    return KVQ_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  kvq_rope_kind kind = scaling ? scaling->kind : KVQ_ROPE_NONE;
  double factor = 1.0, n = 1.0, low = 0.0, high = 0.0;
  if (kind != KVQ_ROPE_NONE) {
    if (kind != KVQ_ROPE_LINEAR && kind != KVQ_ROPE_BANDS && kind != KVQ_ROPE_YARN) return KVQ_ERR_INVALID_ARG;
    factor = scaling->factor;
    if (!(factor >= 1.0) || !(factor < INFINITY)) return KVQ_ERR_INVALID_ARG;
    if (kind != KVQ_ROPE_LINEAR) {
      n = scaling->original;
      low = scaling->low;
      high = scaling->high;
      if (low == 0.0 && high == 0.0) {
        low = 1.0;
        high = kind == KVQ_ROPE_BANDS ? 4.0 : 32.0;
      }
      if (!(n > 0.0) || !(n < INFINITY) || !(low >= 0.0) || !(high > low) || !(high < INFINITY) ||
          (kind == KVQ_ROPE_YARN && !(low > 0.0)))
        return KVQ_ERR_INVALID_ARG;
    }
  }
  double i_high = 0.0, i_low = 0.0;
  if (kind == KVQ_ROPE_YARN) {  // the pair that makes x turns over the original context
    auto pair_of = [&](double x) { return rotary_dim * log(n / (two_pi * x)) / (2.0 * log(base)); };
    i_high = fmax(floor(pair_of(high)), 0.0);
    i_low = fmin(ceil(pair_of(low)), rotary_dim - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    const double f = pow(base, -2.0 * i / rotary_dim);
    double g = f;
    if (kind == KVQ_ROPE_LINEAR) {
      g = f / factor;
    } else if (kind == KVQ_ROPE_BANDS) {
      const double r = fmin(fmax((n * f / two_pi - low) / (high - low), 0.0), 1.0);
      g = f * (r + (1.0 - r) / factor);
    } else if (kind == KVQ_ROPE_YARN) {
      const double r = fmin(fmax((i - i_high) / fmax(i_low - i_high, 0.001), 0.0), 1.0);
      g = f * ((1.0 - r) + r / factor);
    }
    freqs[i] = static_cast<uint64_t>(g / two_pi * 18446744073709551616.0);  // 0 < g <= 1 rad: below a turn
  }
  *attn_factor = kind == KVQ_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
  return KVQ_OK;
}

extern "C" kvq_status kvq_rope(const void *q, int64_t q_stride_t, int64_t q_stride_h, void *q_out,
                               int64_t qo_stride_t, int64_t qo_stride_h, int32_t Hq, const void *k,
                               int64_t k_stride_t, int64_t k_stride_h, void *k_out, int64_t ko_stride_t,
                               int64_t ko_stride_h, int32_t Hk, const kvq_rotary *rotary, kvq_dtype dtype,
                               int32_t T, int32_t D, kvq_stream_t stream) {
  if (T < 0 || Hq < 0 || Hk < 0 || D < 1) return KVQ_ERR_INVALID_ARG;
  if (dtype != KVQ_BF16 && dtype != KVQ_F16 && dtype != KVQ_F32) return KVQ_ERR_INVALID_ARG;
  if (D > 1024 || static_cast<long long>(Hq) + Hk > 65536) return KVQ_ERR_UNSUPPORTED;
  if (rotary == nullptr) return KVQ_ERR_INVALID_ARG;
  WriteKvParams p = {};
  if (T == 0 || Hq + Hk == 0) return KVQ_OK;
  const kvq_status st = check_rotary(rotary, D, &p);
  if (st != KVQ_OK) return st;
  const uintptr_t es = dtype == KVQ_F32 ? 4 : 2;
  if ((Hq > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)) || !aligned(q, es) || !aligned(q_out, es) ||
      !aligned(k, es) || !aligned(k_out, es))
    return KVQ_ERR_INVALID_ARG;
  if ((Hq > 0 && q == q_out && (q_stride_t != qo_stride_t || q_stride_h != qo_stride_h)) ||
      (Hk > 0 && k == k_out && (k_stride_t != ko_stride_t || k_stride_h != ko_stride_h)))
    return KVQ_ERR_INVALID_ARG;
  p.q = {q, q_out, q_stride_t, q_stride_h, qo_stride_t, qo_stride_h, Hq};
  p.k = {k, k_out, k_stride_t, k_stride_h, ko_stride_t, ko_stride_h, Hk};
  p.T = T;
  p.D = D;
  p.bs = 1;
  const bool vec = chunked(p.q) && chunked(p.k) && chunked_pairs(p);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == KVQ_BF16) return launch_write_kv<KVQ_BF16, -1>(p, vec, s);
  if (dtype == KVQ_F16) return launch_write_kv<KVQ_F16, -1>(p, vec, s);
  return launch_write_kv<KVQ_F32, -1>(p, vec, s);
}

extern "C" kvq_status kvq_write_kv(const void *key, int64_t k_stride_t, int64_t k_stride_h, const void *value,
                                   int64_t v_stride_t, int64_t v_stride_h, const kvq_paged_kv *cache,
                                   const int64_t *slot_mapping, const void *q, int64_t q_stride_t,
                                   int64_t q_stride_h, void *q_out, int64_t qo_stride_t, int64_t qo_stride_h,
                                   int32_t Hq, const kvq_rotary *rotary, kvq_dtype dtype, int32_t T, int32_t Hk,
                                   int32_t D, kvq_stream_t stream) {
  if (T < 0 || Hq < 0 || Hk < 1 || D < 1 || cache == nullptr) return KVQ_ERR_INVALID_ARG;
  if (dtype != KVQ_BF16 && dtype != KVQ_F16) return KVQ_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 256 || static_cast<long long>(Hq) + Hk > 65536) return KVQ_ERR_UNSUPPORTED;
  const kvq_status sc = check_paged_kv(cache, dtype);
  if (sc != KVQ_OK) return sc;
  if ((Hq > 0) != (q != nullptr) || (Hq > 0) != (q_out != nullptr) || (Hq > 0 && rotary == nullptr))
    return KVQ_ERR_INVALID_ARG;
  WriteKvParams p = {};
  if (T == 0) return KVQ_OK;
  const kvq_status st = check_rotary(rotary, D, &p);
  if (st != KVQ_OK) return st;
  if (!key || !value || !slot_mapping || !aligned(slot_mapping, 8)) return KVQ_ERR_INVALID_ARG;
  if (Hq > 0 && q == q_out && (q_stride_t != qo_stride_t || q_stride_h != qo_stride_h)) return KVQ_ERR_INVALID_ARG;
  p.q = {q, q_out, q_stride_t, q_stride_h, qo_stride_t, qo_stride_h, Hq};
  p.k = {key, cache->k, k_stride_t, k_stride_h, 0, cache->k_stride_head, Hk};
  p.v = {value, cache->v, v_stride_t, v_stride_h, 0, cache->v_stride_head, Hk};
  if (!chunked(p.q) || !chunked(p.k) || !chunked(p.v)) return KVQ_ERR_INVALID_ARG;
  p.slots = slot_mapping;
  p.k_block = cache->k_stride_block;
  p.k_token = cache->k_stride_token;
  p.v_block = cache->v_stride_block;
  p.v_token = cache->v_stride_token;
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.bs = cache->block_size;
  p.num_blocks = cache->num_blocks;
  p.T = T;
  p.D = D;
  const bool vec = chunked_pairs(p);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cache->dtype == KVQ_E4M3)
    return dtype == KVQ_BF16 ? launch_write_kv<KVQ_BF16, kFp8Dst>(p, vec, s)
                             : launch_write_kv<KVQ_F16, kFp8Dst>(p, vec, s);
  return dtype == KVQ_BF16 ? launch_write_kv<KVQ_BF16, KVQ_BF16>(p, vec, s)
                           : launch_write_kv<KVQ_F16, KVQ_F16>(p, vec, s);
}
