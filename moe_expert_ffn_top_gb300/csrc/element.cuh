// Element types of the training-step operators: fp32, bf16 and fp16 values in memory,
// fp32 in registers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "../../include/moe_lora.h"

namespace moelora {

inline bool dtype_ok(int32_t t) { return t == MOE_LORA_F32 || t == MOE_LORA_BF16 || t == MOE_LORA_F16; }
inline int dtype_bytes(int32_t t) { return t == MOE_LORA_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// ------------------------------------------------------------------ pairs of fp32
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ------------------------------------------------------------------ vectors
// Two neighbouring elements of type T in a register pair: from memory words and back.
template <class T>
struct Two;
template <>
struct Two<float> {
  static constexpr int kWords = 2;
  static __device__ __forceinline__ float2 get(const uint32_t* w) {
    return make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
  }
  static __device__ __forceinline__ void put(uint32_t* w, float2 v) {
    w[0] = __float_as_uint(v.x);
    w[1] = __float_as_uint(v.y);
  }
};
template <>
struct Two<__nv_bfloat16> {
  static constexpr int kWords = 1;
  static __device__ __forceinline__ float2 get(const uint32_t* w) {
    return make_float2(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void put(uint32_t* w, float2 v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    w[0] = reinterpret_cast<const uint32_t&>(h);
  }
};
template <>
struct Two<__half> {
  static constexpr int kWords = 1;
  static __device__ __forceinline__ float2 get(const uint32_t* w) {
    return __half22float2(reinterpret_cast<const __half2&>(w[0]));
  }
  static __device__ __forceinline__ void put(uint32_t* w, float2 v) {
    const __half2 h = __floats2half2_rn(v.x, v.y);
    w[0] = reinterpret_cast<const uint32_t&>(h);
  }
};

// What a thread holds of a row at one place, as loaded: VL elements in 16 bytes, or, for
// rows without 16-byte alignment (VL = 1), two single elements `hop` columns apart (hop
// 0: the second is past the row's end and reads as 0).
template <class T, int VL>
struct Vec {
  static constexpr int kPairs = VL / 2;
  uint32_t w[4];
  __device__ __forceinline__ void clear() { w[0] = w[1] = w[2] = w[3] = 0; }
  // data that passes once: kept out of L1, so that what is reused stays there (not the
  // read-only path: an operator may run in place)
  __device__ __forceinline__ void load(const T* p, int) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
  }
  __device__ __forceinline__ void from_smem(const uint4* p) {
    const uint4 u = *p;
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  }
  __device__ __forceinline__ void store(T* p, int) const {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ float2 get(int i) const { return Two<T>::get(w + i * Two<T>::kWords); }
  __device__ __forceinline__ void put(int i, float2 v) { Two<T>::put(w + i * Two<T>::kWords, v); }
};
template <class T>
struct Vec<T, 1> {
  static constexpr int kPairs = 1;
  T a, b;
  __device__ __forceinline__ void clear() { a = b = from_f32<T>(0.f); }
  __device__ __forceinline__ void load(const T* p, int hop) {
    a = *p;
    b = hop ? p[hop] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void store(T* p, int hop) const {
    *p = a;
    if (hop) p[hop] = b;
  }
  __device__ __forceinline__ float2 get(int) const { return make_float2(to_f32(a), to_f32(b)); }
  __device__ __forceinline__ void put(int, float2 v) {
    a = from_f32<T>(v.x);
    b = from_f32<T>(v.y);
  }
};

__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// Asynchronous copies of 16 (or 4) bytes into shared memory.  A thread that reads only what it
// copied itself needs no barrier: waiting for its own groups is enough.
__device__ __forceinline__ void async_copy16(void* dst_smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_address(dst_smem)), "l"(src) : "memory");
}
// the first `bytes` of 16, the rest as zeros
__device__ __forceinline__ void async_copy16_part(void* dst_smem, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(shared_address(dst_smem)), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void async_copy8(void* dst_smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(shared_address(dst_smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_copy4(void* dst_smem, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(shared_address(dst_smem)), "l"(src) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// waits until at most N of this thread's groups are incomplete
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Column and second-element distance of a thread's slot i in a row of n, shared by tpr threads.
template <int VL>
struct SlotAt {
  int c, hop;
  bool in;
  __device__ __forceinline__ SlotAt(int lane, int i, int tpr, int n) {
    c = VL == 1 ? lane + 2 * i * tpr : (lane + i * tpr) * VL;
    in = c < n;
    hop = VL == 1 && c + tpr < n ? tpr : 0;
  }
  // the same slot of a slice that starts at column `first`
  __device__ __forceinline__ SlotAt shifted(int first) const {
    SlotAt s = *this;
    s.c += first;
    return s;
  }
  // v for both elements of a pair, 0 for the second where that is past the end
  __device__ __forceinline__ float2 pair(float v) const { return make_float2(v, VL == 1 && !hop ? 0.f : v); }
};

// A thread's ring: kStages stages of kSlots 16-byte slots, those of a warp side by side.
template <int kStages, int kSlots>
struct Ring {
  uint4* base;
  __device__ __forceinline__ explicit Ring(void* sm)
      : base(static_cast<uint4*>(sm) + (threadIdx.x >> 5) * (kStages * kSlots * 32) + (threadIdx.x & 31)) {}
  __device__ __forceinline__ uint4* slot(int stage, int i) const { return base + (stage * kSlots + i) * 32; }
};
template <int kStages, int kSlots>
constexpr size_t ring_bytes(int threads) {
  return (size_t)threads * kStages * kSlots * 16;
}

// The elements of a slot in a weight vector, widened.
template <class W, int VL, int kPairs>
__device__ __forceinline__ void ld_pairs(const W* p, int hop, float2 (&f)[kPairs]) {
  if constexpr (VL == 1) {
    const float a = to_f32(*p), b = to_f32(p[hop]);  // hop 0: the same element again, and no branch
    f[0] = make_float2(a, hop ? b : 0.f);
  } else if constexpr (sizeof(W) == 4) {
#pragma unroll
    for (int i = 0; i < kPairs; i += 2) {
      const float4 u = *reinterpret_cast<const float4*>(p + 2 * i);
      f[i] = make_float2(u.x, u.y);
      f[i + 1] = make_float2(u.z, u.w);
    }
  } else {  // 16-bit weights: VL elements in 2 * VL bytes
    uint32_t w[kPairs];
    if constexpr (kPairs == 4)
      reinterpret_cast<uint4&>(w[0]) = *reinterpret_cast<const uint4*>(p);
    else
      reinterpret_cast<uint2&>(w[0]) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) f[i] = Two<W>::get(w + i);
  }
}

}  // namespace moelora
