// rows.cuh — what the row-wise kernels (norm.cuh, rope.cuh) share: loads and
// stores of V elements with their conversion to fp32, and reductions over a
// team, a group of whole warps that works on one row together.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace solattn {

enum : int { kDtypeBf16 = 0, kDtypeFp16 = 1, kDtypeFp32 = 2 };

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }

// V elements as they lie in memory: V = 8 moves 16-byte vectors (32-byte ones
// for fp32), V = 1 single elements, for rows whose address or width is odd.
template <typename T, int V>
struct Raw;
template <typename T>
struct Raw<T, 8> {
  static constexpr int kVecs = sizeof(T) / 2;   // 16-byte vectors
  uint4 r[kVecs];
};
template <typename T>
struct Raw<T, 1> {
  T r;
};

// Streaming load: each input element is read once, so it does not displace
// the modulation vectors in L1.  Not the non-coherent path: a row may be
// written in place by the thread that read it.
__device__ __forceinline__ uint4 ld_row_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
// Eight fp32 in one 32-byte load (p 32-byte aligned): as two 16-byte loads each
// of the warp's would fetch every 32-byte sector that it touches half of.
__device__ __forceinline__ void ld_row_v8(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_row_v8(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void load_raw(Raw<T, 8>& v, const T* p) {
  if constexpr (sizeof(T) == 4) ld_row_v8(p, v.r[0], v.r[1]);
  else v.r[0] = ld_row_v4(p);
}
template <typename T>
__device__ __forceinline__ void load_raw(Raw<T, 1>& v, const T* p) {
  v.r = *p;
}

// Asynchronous copies of 16 bytes into shared memory.  The kernels' warps bring
// vectors of 8 elements by such pieces in address order; a lane of fp32 finds its
// 32 bytes in pieces that two other lanes have copied, so it reads behind a
// __syncwarp and the warp refills behind another.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int D>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(D) : "memory"); }

template <typename T>
__device__ __forceinline__ void widen2(uint32_t w, float& a, float& b);
template <>
__device__ __forceinline__ void widen2<__nv_bfloat16>(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void widen2<__half>(uint32_t w, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
template <typename T>
__device__ __forceinline__ uint32_t narrow2(float a, float b);
template <>
__device__ __forceinline__ uint32_t narrow2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void widen(const Raw<T, 8>& v, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(v.r[i].x);
      f[4 * i + 1] = __uint_as_float(v.r[i].y);
      f[4 * i + 2] = __uint_as_float(v.r[i].z);
      f[4 * i + 3] = __uint_as_float(v.r[i].w);
    }
  } else {
    widen2<T>(v.r[0].x, f[0], f[1]);
    widen2<T>(v.r[0].y, f[2], f[3]);
    widen2<T>(v.r[0].z, f[4], f[5]);
    widen2<T>(v.r[0].w, f[6], f[7]);
  }
}
// Vector `vec` of a stage that asynchronous copies have filled.
template <typename T>
__device__ __forceinline__ void take_staged(const uint8_t* stage, int vec, float (&f)[8]) {
  Raw<T, 8> r;
#pragma unroll
  for (int h = 0; h < Raw<T, 8>::kVecs; ++h)
    r.r[h] = *reinterpret_cast<const uint4*>(stage + vec * 8 * static_cast<int>(sizeof(T)) + 16 * h);
  widen(r, f);
}
template <typename T>
__device__ __forceinline__ void widen(const Raw<T, 1>& v, float (&f)[1]) {
  f[0] = to_f32<T>(v.r);
}

template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    st_row_v8(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])),
              make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7])));
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(narrow2<T>(f[0], f[1]), narrow2<T>(f[2], f[3]), narrow2<T>(f[4], f[5]), narrow2<T>(f[6], f[7]));
  }
}
template <typename T>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, 8>& v) {
  if constexpr (sizeof(T) == 4) st_row_v8(p, v.r[0], v.r[1]);
  else *reinterpret_cast<uint4*>(p) = v.r[0];
}
template <typename T>
__device__ __forceinline__ void store_row(T* p, const float (&f)[1]) {
  *p = from_f32<T>(f[0]);
}

// ------------------------------------------------------------------ arithmetic on V values
// Two fp32 operations an instruction where V is even.
template <int V>
__device__ __forceinline__ void fma_v(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 r = __ffma2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), make_float2(c[j], c[j + 1]));
      d[j] = r.x, d[j + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = fmaf(a[j], b[j], c[j]);
  }
}
template <int V>
__device__ __forceinline__ void fma_s(float (&d)[V], const float (&a)[V], float b, const float (&c)[V]) {
  float t[V];
#pragma unroll
  for (int j = 0; j < V; ++j) t[j] = b;
  fma_v<V>(d, a, t, c);
}
template <int V>
__device__ __forceinline__ void mul_v(float (&d)[V], const float (&a)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 r = __fmul2_rn(make_float2(d[j], d[j + 1]), make_float2(a[j], a[j + 1]));
      d[j] = r.x, d[j + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = __fmul_rn(d[j], a[j]);
  }
}
template <int V>
__device__ __forceinline__ void mul_s(float (&d)[V], float a) {
  float t[V];
#pragma unroll
  for (int j = 0; j < V; ++j) t[j] = a;
  mul_v<V>(d, t);
}
template <int V>
__device__ __forceinline__ void add_s(float (&d)[V], float a) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 r = __fadd2_rn(make_float2(d[j], d[j + 1]), make_float2(a, a));
      d[j] = r.x, d[j + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] += a;
  }
}
// Adds the values, or their squares, to two partial sums.
template <int V>
__device__ __forceinline__ void sum_v(float2& s, const float (&a)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) s = __fadd2_rn(s, make_float2(a[j], a[j + 1]));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) s.x += a[j];
  }
}
template <int V>
__device__ __forceinline__ void sum_sq(float2& s, const float (&a)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) s = __ffma2_rn(make_float2(a[j], a[j + 1]), make_float2(a[j], a[j + 1]), s);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) s.x = fmaf(a[j], a[j], s.x);
  }
}

// Largest absolute value of two and of what was largest; a NaN comes through.
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// The factor 127 / amax of a row's 8-bit values in two terms, hi rounded and lo
// what that left out (the residual of a quotient is exact), by 2^-20 too small;
// amax between 2^-100 and 2^100.
struct Up8 {
  float hi, lo;
};
__device__ __forceinline__ Up8 up_s8(float amax) {
  const float hi = 127.f / amax;
  return Up8{hi, fmaf(-hi, amax, 127.f) * (hi * static_cast<float>((1.0 - 0x1p-20) / 127.0))};
}
// v * up to the nearest whole numbers, ties to even, as the low bytes of k: adding
// 1.5 * 2^23 leaves the whole number there.  hi alone would not do: where
// 127 v / amax is a half, which is common in rows of 16-bit values (0.2% of normal
// bf16 ones), v * hi lies beside it, on the same side for a whole row.  So
//   y = fl(v * hi),  z = fl(y + v * lo).
// Beside a half h, v * hi = h + E with |E| at most a unit of h, and y = h + R, R
// being E to the nearest unit (h has few bits, so a tie there falls to h).
// y + v * lo = h + R - E lies within half a unit of h, and z = h: lo, a little too
// small, does not carry it beyond.  Values of 11 bits or fewer, bf16 and fp16, thus
// give the exact result (tried out for every ratio of two of them): no other
// quotient of theirs is nearer to h = c / 2 than 2^-18 of it, as 254 v - c amax is
// two units of v's last place at least.  Of other fp32 values one whose quotient is
// within a unit of a half, 2^-23 of it, may be taken for that half.
template <int V>
__device__ __forceinline__ void whole_s8(const float (&v)[V], const Up8& up, uint32_t (&k)[V]) {
  float lo[V], z[V];
#pragma unroll
  for (int j = 0; j < V; ++j) lo[j] = up.lo, z[j] = v[j];
  mul_s<V>(z, up.hi);
  fma_v<V>(z, v, lo, z);
  add_s<V>(z, 12582912.f);
#pragma unroll
  for (int j = 0; j < V; ++j) k[j] = __float_as_uint(z[j]);
}
__device__ __forceinline__ uint2 pack_s8(const float (&v)[8], const Up8& up) {
  uint32_t k[8];
  whole_s8<8>(v, up, k);
  return make_uint2(__byte_perm(__byte_perm(k[0], k[1], 0x0040), __byte_perm(k[2], k[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(k[4], k[5], 0x0040), __byte_perm(k[6], k[7], 0x0040), 0x5410));
}
template <int V>
__device__ __forceinline__ void store_s8(int8_t* p, const float (&v)[V], const Up8& up) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint2*>(p) = pack_s8(v, up);
  } else {
    uint32_t k[1];
    whole_s8<1>(v, up, k);
    *p = static_cast<int8_t>(k[0]);
  }
}

// N vectors of V consecutive parameters, `step` elements apart, whose type is
// only known at run time: one branch for all of them, so that the loads are
// under way together.  Those at or past `end` are left as they are.
template <int V, int N>
__device__ __forceinline__ void load_params(const void* p, int dtype, long long at, int c, int step, int end,
                                            float (&f)[N][V]) {
  if (dtype == kDtypeFp32) {
    const float* q = static_cast<const float*>(p) + at;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c + i * step >= end) continue;
      if constexpr (V == 8) {
        const float4 a = *reinterpret_cast<const float4*>(q + c + i * step);
        const float4 b = *reinterpret_cast<const float4*>(q + c + i * step + 4);
        f[i][0] = a.x, f[i][1] = a.y, f[i][2] = a.z, f[i][3] = a.w;
        f[i][4] = b.x, f[i][5] = b.y, f[i][6] = b.z, f[i][7] = b.w;
      } else {
        f[i][0] = q[c + i * step];
      }
    }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + at;
    const bool bf = dtype == kDtypeBf16;
    uint4 w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c + i * step >= end) continue;
      if constexpr (V == 8) w[i] = *reinterpret_cast<const uint4*>(q + c + i * step);
      else w[i].x = q[c + i * step];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (c + i * step >= end) continue;
      if constexpr (V == 8) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (bf) widen2<__nv_bfloat16>(u[j], f[i][2 * j], f[i][2 * j + 1]);
          else widen2<__half>(u[j], f[i][2 * j], f[i][2 * j + 1]);
        }
      } else {
        f[i][0] = bf ? __uint_as_float(w[i].x << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(w[i].x)));
      }
    }
  }
}

// ------------------------------------------------------------------ teams
// A team is WARPS whole warps of a block at most, numbered from 0 (WARPS = 1:
// one); a block holds up to 15 teams of more than one warp (each has a named
// barrier of its own, barrier 0 being the block's).  Every warp of a team takes
// the same calls.  Its warps meet in two rows of kSlots slots of W floats,
// which alternate: one barrier a reduction is enough then, as a warp that is
// one reduction ahead writes the other row, and it cannot be two ahead.  Slots
// past the last warp's stay zero, so that all are read without a count.
template <int WARPS, int W>
struct Team {
  static constexpr int kSlots = (WARPS + 3) / 4 * 4;
  int warps;      // warps of a team
  int index;      // this team's number in the block
  int warp;       // this warp's number in the team
  float* slots;   // the row that the next reduction writes
  float* other;

  // Shared floats (16-byte aligned) of a block of `threads` threads whose teams
  // have more than WARPS / 2 warps, or more than `least`.
  static constexpr int shared(int threads, int least) {
    return WARPS == 1 ? 4 : 2 * W * kSlots * (threads / 32 / (least + 1) + 1);
  }
  // The slots are cleared here: the caller has the block synchronise before
  // the first reduction.
  __device__ __forceinline__ void make(int warps_, float* all, int count) {
    warps = WARPS == 1 ? 1 : warps_;
    index = (threadIdx.x / 32) / warps;
    warp = (threadIdx.x / 32) % warps;
    if constexpr (WARPS > 1) {
      slots = all + 2 * W * kSlots * index;
      other = slots + W * kSlots;
      for (int i = threadIdx.x; i < count; i += blockDim.x) all[i] = 0.f;
    }
  }
  __device__ __forceinline__ void sync() const {
    if (WARPS == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
  }
  __device__ __forceinline__ float* turn() {
    float* s = slots;
    slots = other;
    other = s;
    return s;
  }

  // Sums over the team, the same bits in every thread and on every run: lanes
  // by a butterfly, warps in a fixed order.  What a warp of the team wrote to
  // shared memory before, all of them can read behind it.
  template <int R>
  __device__ __forceinline__ void sum(float (&x)[R]) {
    static_assert(R <= W, "slots");
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] += __shfl_xor_sync(0xFFFFFFFFu, x[r], o);
    if constexpr (WARPS == 1) {
      __syncwarp();
      return;
    } else {
      float* s = turn();
      if ((threadIdx.x & 31) == 0) {
        if constexpr (R == 2) *reinterpret_cast<float2*>(s + 2 * warp) = make_float2(x[0], x[1]);
        else s[warp] = x[0];
      }
      sync();
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = 0.f;
#pragma unroll
      for (int i = 0; i < kSlots; i += 4 / R) {
        const float4 f = *reinterpret_cast<const float4*>(s + R * i);
        if constexpr (R == 2) x[0] += f.x + f.z, x[1] += f.y + f.w;
        else x[0] += (f.x + f.y) + (f.z + f.w);
      }
    }
  }
  // Largest of absolute values; their bit patterns compare as they do, with a
  // NaN's above infinity's, so that a NaN anywhere comes through.
  template <int R>
  __device__ __forceinline__ void max(float (&x)[R]) {
    static_assert(R <= W, "slots");
#pragma unroll
    for (int r = 0; r < R; ++r)
      x[r] = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x[r]) & 0x7FFFFFFFu));
    if constexpr (WARPS > 1) {
      float* s = turn();
      if ((threadIdx.x & 31) == 0) {
        if constexpr (R == 2) *reinterpret_cast<float2*>(s + 2 * warp) = make_float2(x[0], x[1]);
        else s[warp] = x[0];
      }
      sync();
      uint32_t m[R];
#pragma unroll
      for (int r = 0; r < R; ++r) m[r] = 0;
#pragma unroll
      for (int i = 0; i < kSlots; i += 4 / R) {
        const uint4 f = *reinterpret_cast<const uint4*>(s + R * i);
        if constexpr (R == 2) m[0] = ::max(m[0], ::max(f.x, f.z)), m[1] = ::max(m[1], ::max(f.y, f.w));
        else m[0] = ::max(::max(m[0], ::max(f.x, f.y)), ::max(f.z, f.w));
      }
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = __uint_as_float(m[r]);
    }
  }
};

// x / n for n = 1 / inv: a product and a correction of its error, so that the
// mean of equal values is that value.
__device__ __forceinline__ float divide_by(float x, float n, float inv) {
  const float q = x * inv;
  const float better = fmaf(fmaf(-q, n, x), inv, q);
  return fabsf(q) <= 3.402823466e38f ? better : q;
}

}  // namespace solattn
