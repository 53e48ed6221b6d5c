// Element types of the bandwidth-bound operators: vectors of VEC elements
// loaded and stored in accesses of up to 16 bytes, converted to and from fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "../../include/cce_ops.h"

namespace cce {

template <typename T>
struct ElemType;
template <>
struct ElemType<float> {
  static constexpr int id = CCE_F32;
};
template <>
struct ElemType<__half> {
  static constexpr int id = CCE_F16;
};
template <>
struct ElemType<__nv_bfloat16> {
  static constexpr int id = CCE_BF16;
};

// VEC consecutive elements as raw words.  The access width is the vector's
// size, 16 bytes at most (a wider vector takes several accesses).
template <typename T, int VEC>
struct Vec {
  static constexpr int BYTES = static_cast<int>(sizeof(T)) * VEC;
  static constexpr int WORDS = (BYTES + 3) / 4;
  alignas(BYTES >= 16 ? 16 : 4 * WORDS) uint32_t w[WORDS];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  // Ordinary loads: a kernel started by launch_after() reads what the kernel before it was still writing when it
  // started, and only these are ordered behind wait_for_previous().
  __device__ __forceinline__ void load(const T* p) { load_as<false>(p); }
  // From memory that nothing writes from the kernel's start to its end: not in a kernel started by launch_after().
  // These may be moved across the kernel's own stores.
  __device__ __forceinline__ void load_constant(const T* p) { load_as<true>(p); }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
    }
  }
  // Elements lo .. hi - 1 alone, the others 0.
  __device__ __forceinline__ void load_some(const T* p, int lo, int hi) {
    zero();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (e >= lo && e < hi) {
        if constexpr (sizeof(T) == 4) {
          w[e] = reinterpret_cast<const uint32_t*>(p)[e];
        } else {
          w[e / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[e]) << (16 * (e & 1));
        }
      }
    }
  }
  __device__ __forceinline__ void store_some(T* p, int lo, int hi) const {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (e >= lo && e < hi) {
        if constexpr (sizeof(T) == 4) {
          reinterpret_cast<uint32_t*>(p)[e] = w[e];
        } else {
          reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
        }
      }
    }
  }
  __device__ __forceinline__ void keep(int lo, int hi) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (e < lo || e >= hi) {
        if constexpr (sizeof(T) == 4) {
          w[e] = 0u;
        } else {
          w[e / 2] &= e & 1 ? 0x0000ffffu : 0xffff0000u;
        }
      }
    }
  }
  // Becomes the elements shift .. shift + VEC - 1 of lo and hi in a row, 0 <= shift < VEC.
  __device__ __forceinline__ void join(const Vec& lo, const Vec& hi, int shift) {
    uint32_t a[2 * WORDS];
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
      a[i] = lo.w[i];
      a[WORDS + i] = hi.w[i];
    }
    const int bytes = shift * static_cast<int>(sizeof(T));
#pragma unroll
    for (int step = WORDS / 2; step > 0; step /= 2) {
#pragma unroll
      for (int i = 0; i + step < 2 * WORDS; ++i) a[i] = bytes & 4 * step ? a[i + step] : a[i];
    }
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = sizeof(T) == 4 ? a[i] : __funnelshift_r(a[i], a[i + 1], 8 * (bytes & 3));
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(w[i]);
    } else {
      const uint16_t h = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
      if constexpr (ElemType<T>::id == CCE_BF16) {
        return __uint_as_float(static_cast<uint32_t>(h) << 16);
      } else {
        return __half2float(__ushort_as_half(h));
      }
    }
  }
  // All VEC elements from fp32, rounded to nearest even.
  __device__ __forceinline__ void set(const float (&f)[VEC]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (VEC == 1) {
      w[0] = half_bits(f[0]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        if constexpr (ElemType<T>::id == CCE_BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
          std::memcpy(&w[i], &h, 4);
        } else {
          const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
          std::memcpy(&w[i], &h, 4);
        }
      }
    }
  }

 private:
  template <bool CONSTANT, typename W>
  __device__ __forceinline__ static W word(const W* p) {
    if constexpr (CONSTANT) {
      return __ldg(p);
    } else {
      return *p;
    }
  }
  template <bool CONSTANT>
  __device__ __forceinline__ void load_as(const T* p) {
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) words4(i, word<CONSTANT>(reinterpret_cast<const uint4*>(p) + i));
    } else if constexpr (BYTES == 8) {
      words2(word<CONSTANT>(reinterpret_cast<const uint2*>(p)));
    } else if constexpr (BYTES == 4) {
      w[0] = word<CONSTANT>(reinterpret_cast<const uint32_t*>(p));
    } else {
      static_assert(BYTES == 2, "one 16-bit element");
      w[0] = word<CONSTANT>(reinterpret_cast<const uint16_t*>(p));
    }
  }
  __device__ __forceinline__ void words4(int i, const uint4& v) {
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
  __device__ __forceinline__ void words2(const uint2& v) {
    w[0] = v.x;
    w[1] = v.y;
  }
  __device__ __forceinline__ static uint32_t half_bits(float f) {
    if constexpr (ElemType<T>::id == CCE_BF16) {
      return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    } else {
      return __half_as_ushort(__float2half_rn(f));
    }
  }
};

// Copies that pass the registers by: a thread's own 4, 8 or 16 bytes from global
// to shared memory, in groups that it waits for (all but the newest N of them).
template <int BYTES>
__device__ __forceinline__ void copy_async(void* shared, const void* global) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(shared));
  if constexpr (BYTES == 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(global) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(global), "n"(BYTES) : "memory");
  }
}
__device__ __forceinline__ void end_copy_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copy_groups() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two fp32 values in a register pair, for the packed fp32 instructions (one issue slot for two results).
struct Pair {
  unsigned long long v;

  __device__ __forceinline__ static Pair of(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(lo), "f"(hi));
    return p;
  }
  __device__ __forceinline__ static Pair both(float f) { return of(f, f); }
  __device__ __forceinline__ float2 get() const {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
  }
  __device__ __forceinline__ float sum() const {
    const float2 f = get();
    return f.x + f.y;
  }
};

__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__device__ __forceinline__ Pair fma_down(Pair a, Pair b, Pair c) {  // rounded towards minus infinity
  Pair r;
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

template <typename T, int VEC, bool SOME, bool CONSTANT>
__device__ __forceinline__ void load_param_as(const T* p, int n, float (&out)[VEC]) {
  static_assert(!SOME || !CONSTANT, "load_some is ordinary");
  Vec<T, VEC> v;
  if constexpr (SOME) {
    v.load_some(p, 0, n);
  } else if constexpr (CONSTANT) {
    v.load_constant(p);
  } else {
    v.load(p);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) out[e] = v.get(e);
}

// VEC parameters of a run-time type as fp32 (the type is uniform over a launch).
// SOME: the first n alone, the others 0, at any element's alignment.  CONSTANT: by load_constant().
template <int VEC, bool SOME = false, bool CONSTANT = false>
__device__ __forceinline__ void load_param(const void* p, int type, int64_t i, float (&out)[VEC], int n = VEC) {
  if (type == CCE_F32) {
    load_param_as<float, VEC, SOME, CONSTANT>(static_cast<const float*>(p) + i, n, out);
  } else if (type == CCE_BF16) {
    load_param_as<__nv_bfloat16, VEC, SOME, CONSTANT>(static_cast<const __nv_bfloat16*>(p) + i, n, out);
  } else {
    load_param_as<__half, VEC, SOME, CONSTANT>(static_cast<const __half*>(p) + i, n, out);
  }
}

__device__ __forceinline__ void store_param(void* p, int type, int64_t i, float f) {
  if (type == CCE_F32) {
    static_cast<float*>(p)[i] = f;
  } else if (type == CCE_BF16) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(f);
  } else {
    static_cast<__half*>(p)[i] = __float2half_rn(f);
  }
}

// A kernel launched by launch_after() may start while the kernel before it in
// the stream ends: it calls wait_for_previous() before it touches memory, and a
// kernel calls let_next_start() once it needs no more blocks.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// cluster: blocks of a cluster (1: none).
template <typename... Params, typename... Args>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, unsigned cluster,
                         cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace cce
