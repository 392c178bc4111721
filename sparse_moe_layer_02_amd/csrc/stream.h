// Values of sweeps that read and write each once: past the caches, in pieces of
// 8 values, or of 4 where fp32 is among the types, so that each load and store of
// a wave has whole lines.  (Streams of 192 MB and more: 6.2 to 6.7 TB/s so, 5.5
// to 5.9 with the default policy; norm backward of 8192 rows of 6144 from 8-bit
// rows 58 us against 72; with half lines a load it gains nothing.)
#pragma once

#include <type_traits>

#include "mx8.h"

namespace moe {
namespace stream {

// VEC values as they are kept: loaded early as Raw, taken apart later.
// arrived: a point that the load is waited for at, before any that follow it.
typedef __attribute__((__vector_size__(4 * sizeof(__bf16)))) __bf16 bf16x4;
template <typename T, int VEC> struct Source;
template <int VEC> struct Source<bf16, VEC> {
  typedef __attribute__((__vector_size__(VEC * sizeof(__bf16)))) __bf16 Raw;
  const bf16* p;
  static __device__ __forceinline__ void arrived(Raw& r) { asm volatile("" : "+v"(r)); }
  __device__ __forceinline__ Raw load(size_t at) const {
    return __builtin_nontemporal_load((const Raw*)(p + at));
  }
  static __device__ __forceinline__ void values(const Raw& r, float* v) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = (float)r[i];
  }
};
template <> struct Source<float, 4> {
  typedef f32x4 Raw;
  const float* p;
  static __device__ __forceinline__ void arrived(Raw& r) { asm volatile("" : "+v"(r)); }
  __device__ __forceinline__ Raw load(size_t at) const {
    return __builtin_nontemporal_load((const f32x4*)(p + at));
  }
  static __device__ __forceinline__ void values(const Raw& r, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r[i];
  }
};
struct Mx8;
template <int VEC> struct Source<Mx8, VEC> {
  typedef mx8::Codes<VEC> Codes;
  struct Raw {
    Codes codes;
    unsigned scale;
  };
  const uint8_t* codes;
  const uint8_t* scales;
  static __device__ __forceinline__ void arrived(Raw& r) {
    asm volatile("" : "+v"(r.codes), "+v"(r.scale));
  }
  __device__ __forceinline__ Raw load(size_t at) const {
    return Raw{__builtin_nontemporal_load((const Codes*)(codes + at)), scales[at / 32]};
  }
  static __device__ __forceinline__ void values(const Raw& r, float* v) {
    mx8::decode<VEC>(r.codes, r.scale, v);
  }
};

template <int VEC> __device__ __forceinline__ void load_floats(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < VEC; i += 4) *(f32x4*)(v + i) = *(const f32x4*)(p + i);
}
template <int VEC> __device__ __forceinline__ void store_floats(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < VEC; i += 4) *(f32x4*)(p + i) = *(const f32x4*)(v + i);
}
// VEC values past the caches.
template <int VEC> __device__ __forceinline__ void store_past(bf16* p, const float* o) {
  typename Source<bf16, VEC>::Raw v;
#pragma unroll
  for (int i = 0; i < VEC; ++i) v[i] = (bf16)o[i];
  __builtin_nontemporal_store(v, (typename Source<bf16, VEC>::Raw*)p);
}
template <int VEC> __device__ __forceinline__ void store_past(float* p, const float* o) {
  __builtin_nontemporal_store(f32x4{o[0], o[1], o[2], o[3]}, (f32x4*)p);
}

// Values of a piece for these types.
template <typename... T> constexpr int piece_of() {
  return (std::is_same<T, float>::value || ...) ? 4 : 8;
}

}  // namespace stream
}  // namespace moe
