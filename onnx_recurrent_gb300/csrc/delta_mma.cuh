// Matrix products of the gated delta rule on the tensor cores: operands in
// fp16 parts, tensor memory, and waits that end.
//
// An fp32 operand x is taken as two fp16 parts, hi = fp16(x / s) and lo = fp16(x / s - hi), with s
// a power of two that brings the largest |x| of its row to between 2^14 and 2^15: nearly all of fp16's exponents then lie
// below it.  hi + lo has 22 bits (off by 2^-23 of x at most) of every value down to 2^-17 of the row's power of two, and what a smaller one
// loses is below 2^-40 of that.  (With the largest at 1, that floor was 2^-25: a step whose slopes are a millionth of its
// neighbours' kept five bits of them.)  A product of two such operands is
// hi lo + lo hi + hi hi (what is left out is below 2^-22 of it), summed in fp32 in this order: every instruction of 16
// products rounds its sum towards zero, so the large ones come last (first, results were off by twice as much).  Scales are applied
// exactly, to a row of the result or, along the sum, to the other operand.  16-bit inputs are one part:
// bf16 values down to 2^-32 of their row's power of two have no second, nor have fp16 values, but for subnormal ones beside
// 2^15 or more.
#pragma once

#include <type_traits>

#include "delta_tile.cuh"
#include "tma.cuh"

namespace rnngb {
namespace delta {

constexpr unsigned kBlock = 8192;            // 64 rows of 64 fp16 values, 128-byte swizzle

// Byte of element c of row r in a 64-row block (c < 64).
__device__ __forceinline__ unsigned swizzled(int r, int c) { return (unsigned)(r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2); }

// The power of two s of a row whose largest is m, |m| / s below 2^15, and one over it; 1 for 0, and both stay ordinary numbers.
struct Scale {
    float up, down;
};
constexpr int kTop = 15;
__device__ __forceinline__ Scale scale_of(float m)
{
    int e = (int)((__float_as_uint(m) >> 23) & 255u) + 1 - kTop;        // biased exponent of s
    e = m == 0.f ? 127 : e < 2 ? 2 : e;                                  // (at most 241)
    return Scale{__uint_as_float((unsigned)e << 23), __uint_as_float((unsigned)(254 - e) << 23)};
}

// Two neighbouring values (the first in the low half) as parts.
__device__ __forceinline__ unsigned half_pair(float a, float b)
{
    unsigned v;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(v) : "f"(b), "f"(a));
    return v;
}
__device__ __forceinline__ float2 pair_value(unsigned v)
{
    const __half2 h = *reinterpret_cast<const __half2*>(&v);
    return __half22float2(h);
}
__device__ __forceinline__ void split_pair(float a, float b, unsigned& hi, unsigned& lo)
{
    hi = half_pair(a, b);
    const float2 h = pair_value(hi);
    lo = half_pair(a - h.x, b - h.y);
}

// Shared-memory descriptors of blocks: rows along N (or M) with the sum along the row ("K-major"),
// 1024 bytes from 8 rows to the next 8; or the sum along the rows ("MN-major"), with
// `apart` bytes from 64 values of N to the next 64.
__device__ __forceinline__ uint64_t desc_rows(unsigned saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)1u << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
__device__ __forceinline__ uint64_t desc_columns(unsigned saddr, unsigned apart)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)(apart >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 | (uint64_t)1u << 46 | (uint64_t)2u << 61;
}
// Instruction descriptor: fp16 operands, fp32 sums, M = 128; `columns`: B's sum runs along its rows.
__host__ __device__ constexpr uint32_t instr(int n, bool columns) { return (1u << 4) | (columns ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }

// Asks for memory to be brought into L2 (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void prefetch(const void* at, unsigned bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}
// One lane of a converged warp.  Products are issued by a whole warp of which one lane acts: operands
// then stay in uniform registers (33 clocks a product of 128 x 64 x 16; by a lone lane, 45).
__device__ __forceinline__ bool elected()
{
    unsigned v;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(v));
    return v != 0;
}
// D[128][n] (+)= A[128][16] B[n][16]^T, A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// The same with A in shared memory (K-major).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// What threads wrote to shared memory is read by products and copies after this and a barrier.
__device__ __forceinline__ void fence_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, unsigned columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, unsigned columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

// 32 columns of this thread's lane, and 16 and 32 of them written.
__device__ __forceinline__ void tmem_ld(uint32_t at, f2 (&v)[16])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = pack2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16])
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const unsigned* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 values of a row over its scale as parts: 16 columns of hi at `hi`, 16 of lo at `lo`.
__device__ __forceinline__ void put_parts(uint32_t hi, uint32_t lo, const f2* v, float down)
{
    unsigned h[16], l[16];
    const f2 d = dup2(down), minus = dup2(-1.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const f2 a = mul2(v[i], d);
        float x, y;
        unpack2(a, x, y);
        h[i] = half_pair(x, y);
        const float2 b = pair_value(h[i]);
        unpack2(fma2(pack2(b.x, b.y), minus, a), x, y);
        l[i] = half_pair(x, y);
    }
    tmem_st16(hi, h);
    tmem_st16(lo, l);
}

// Waits end after this long; a kernel whose wait gave up says so in its status and returns.
constexpr long long kWaitNs = 2000000000ll;
__device__ __forceinline__ bool wait(uint64_t* bar, unsigned parity, volatile int* given_up)
{
    if (mbar_test(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    unsigned it = 0;
    while (!mbar_test(bar, parity)) {
        if ((++it & 255u) == 0u) {
            if (*given_up) return false;
            if ((long long)(globaltimer_ns() - t0) > kWaitNs) {
                *given_up = 1;
                return false;
            }
        }
    }
    return true;
}

// Meets `threads` threads at barrier `id` and says whether all of them came with ok.
__device__ __forceinline__ bool meet(int id, int threads, bool ok)
{
    int all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, %2, %3, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((int)ok), "r"(id), "r"(threads)
        : "memory");
    return all != 0;
}

// A fragment of four 8 x 8 matrices from swizzled rows.
__device__ __forceinline__ void ld_matrix(unsigned (&r)[4], unsigned saddr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(saddr)
                 : "memory");
}
__device__ __forceinline__ void mma_sync(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}


// What the first launch leaves for the second, as it will lie in shared memory: K and Q of a chunk and key
// head in KP parts of DKB blocks (64 steps by 64 values each; a block of Q follows its block of K), T
// and P of a chunk and head in two parts each, and the factors of its steps.
template <int DKB, int KP>
struct Images {
    static constexpr unsigned keys = 2 * KP * DKB * kBlock, mats = kDeltaMats;
};
// Factors: of V and of K S0 in b (V - e^G K S0), of U's columns, of U's rows for the state, of Q S0 and of P U
// in Y (kWhole: e^G_last).  The scales of the rows of K, Q, T and P are in them; those of K and Q also stand alone.
enum Factor { kBeta = 0, kDecayed = 64, kT = 128, kLast = 192, kQuery = 256, kP = 320, kKeyScale = 384, kQueryScale = 448, kWhole = 512 };

// Four neighbouring values of rows of T: N rows at once, their loads together (a branch between them would make each wait
// for the one before).  Row a is at `row + a * apart`, lanes have the values 4 l .. 4 l + 3 of `left`; rows of which
// in(a) is false, and values past `left`, are 0.
template <typename T>
struct alignas(4 * sizeof(T)) Four {
    T v[4];
};
template <int N, typename T, typename In>
__device__ __forceinline__ void load_fours(const T* row, int64_t apart, int left, bool wide, In in, float (&x)[N][4])
{
    const int c = threadIdx.x % 32 * 4;
    if (wide) {
        Four<T> q[N] = {};
#pragma unroll
        for (int a = 0; a < N; ++a)
            if (in(a) && c < left) q[a] = *reinterpret_cast<const Four<T>*>(row + a * apart + c);
#pragma unroll
        for (int a = 0; a < N; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[a][e] = to_f(q[a].v[e]);
    } else {
        T q[N][4];
#pragma unroll
        for (int a = 0; a < N; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) q[a][e] = in(a) && c + e < left ? row[a * apart + c + e] : from_f<T>(0.f);
#pragma unroll
        for (int a = 0; a < N; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[a][e] = to_f(q[a][e]);
    }
}
// The largest of a row of 128 values, four a lane.
__device__ __forceinline__ float row_most(const float (&x)[4])
{
    float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));      // not negative: its bits sort as it does
}
// A row over its scale into blocks `apart` bytes from one another (the second part after the first's BLOCKS).
template <int BLOCKS, int PARTS>
__device__ __forceinline__ void put_row(unsigned char* img, unsigned apart, int r, const float (&x)[4], float down)
{
    const int c = threadIdx.x % 32 * 4;
    if (c < BLOCKS * 64) {
        uint2 hi, lo;
        split_pair(x[0] * down, x[1] * down, hi.x, lo.x);
        split_pair(x[2] * down, x[3] * down, hi.y, lo.y);
        unsigned char* at = img + c / 64 * apart + swizzled(r, c % 64);
        *reinterpret_cast<uint2*>(at) = hi;
        if (PARTS == 2) *reinterpret_cast<uint2*>(at + BLOCKS * apart) = lo;
    }
}
// Whether rows of d values start on multiples of four of them.
template <typename T>
__device__ __forceinline__ bool fours(const View& v, int d)
{
    return (uintptr_t)v.data % (4 * sizeof(T)) == 0 && (v.ss | v.bs | d) % 4 == 0;
}

// V and Y of a chunk by columns: 64 steps of 16 bits and 16 bytes more, so that threads' 16-byte accesses spread over all banks.
constexpr int kPitch = 144;
constexpr unsigned kSheet = 128 * kPitch;

// A 64-step chunk of rows of 16-bit values to columns in shared memory (and back): thread t of 64 has step t; 16 bytes at
// a time where the rows are aligned.  Rows have `cols` (at most 128) values; out of range they are 0.  (Short loops: what a chain's
// warps run each chunk has to stay in the instruction cache.)
template <typename T>
__device__ __forceinline__ void rows_to_sheet(unsigned char* sheet_at, const T* row, bool in, bool wide, int cols, int t)
{
    unsigned short* sheet = reinterpret_cast<unsigned short*>(sheet_at) + t;
    const unsigned short* from = reinterpret_cast<const unsigned short*>(row);
    if (wide && cols % 8 == 0) {
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 64) {
            uint4 x[8];         // all on their way at once
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                x[q] = make_uint4(0, 0, 0, 0);
                if (in && c0 + 8 * q < cols) x[q] = *reinterpret_cast<const uint4*>(from + c0 + 8 * q);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const unsigned pairs[4] = {x[q].x, x[q].y, x[q].z, x[q].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) sheet[(c0 + 8 * q + e) * (kPitch / 2)] = (unsigned short)(pairs[e / 2] >> (e % 2 * 16));
            }
        }
    } else {
#pragma unroll 1
        for (int c0 = 0; c0 < 128; c0 += 16) {
            unsigned short x[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = in && c0 + e < cols ? from[c0 + e] : (unsigned short)0;
#pragma unroll
            for (int e = 0; e < 16; ++e) sheet[(c0 + e) * (kPitch / 2)] = x[e];
        }
    }
}
template <typename T>
__device__ __forceinline__ void sheet_to_rows(const unsigned char* sheet_at, T* row_at, bool wide, int cols, int t)
{
    const unsigned short* sheet = reinterpret_cast<const unsigned short*>(sheet_at) + t;
    unsigned short* row = reinterpret_cast<unsigned short*>(row_at);
    if (wide && cols % 8 == 0) {
#pragma unroll 2
        for (int c = 0; c < cols; c += 8) {
            unsigned short x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = sheet[(c + e) * (kPitch / 2)];
            *reinterpret_cast<uint4*>(row + c) = make_uint4(x[0] | (unsigned)x[1] << 16, x[2] | (unsigned)x[3] << 16,
                                                            x[4] | (unsigned)x[5] << 16, x[6] | (unsigned)x[7] << 16);
        }
    } else {
#pragma unroll 4
        for (int c = 0; c < cols; ++c) row[c] = sheet[c * (kPitch / 2)];
    }
}

constexpr unsigned kTmem = 512;             // a block takes all of it
constexpr int kChainThreads = 384;

template <typename T>
__device__ __forceinline__ f2 pair_of(unsigned raw);
template <>
__device__ __forceinline__ f2 pair_of<__nv_bfloat16>(unsigned raw) { return pack2(__uint_as_float(raw << 16), __uint_as_float(raw & 0xffff0000u)); }
template <>
__device__ __forceinline__ f2 pair_of<__half>(unsigned raw)
{
    const float2 v = pair_value(raw);
    return pack2(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ unsigned raw_pair(f2 v)
{
    float a, b;
    unpack2(v, a, b);
    if (sizeof(T) == 4) return 0;
    unsigned r;
    if constexpr (std::is_same_v<T, __nv_bfloat16>) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else r = half_pair(a, b);
    return r;
}
__device__ __forceinline__ float most_of(float m, f2 v)
{
    float a, b;
    unpack2(v, a, b);
    return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
}

template <typename T, int DKB, int KP>
struct ChainSmem {
    static constexpr bool staged = sizeof(T) == 2;
    static constexpr unsigned stage = Images<DKB, KP>::keys + Images<DKB, KP>::mats;
    static constexpr int stages = 2;
    static constexpr size_t bytes = stages * (size_t)stage + (staged ? 3 * kSheet : 0) + 1024;
};

// Rows and heads over y and z of a grid.
inline dim3 heads_grid(int64_t x, int64_t nh)
{
    const int64_t y = nh < 65535 ? nh : 65535;
    return dim3((unsigned)x, (unsigned)y, (unsigned)((nh + y - 1) / y));
}


// What a chain keeps of a chunk for the gradient's second launch, for each tile of 128 values: matrices [value][step or key] in two
// parts under one scale a tile (the products' sums run over the values).  They lie without a swizzle, eight steps or keys (16
// bytes) of all 128 values one after another, so that the 32 lanes of a chain's warp, a value each, write 512 bytes together
// (rows of 128 bytes, swizzled, took a store 32 lines: 4600 clocks a chunk instead of 800).
constexpr unsigned kSheetImage = 128 * 128;     // 128 values of 64 steps or keys
constexpr unsigned kPiece = 128 * 16;
template <int N>
__device__ __forceinline__ void keep_parts(unsigned char* image, unsigned second, int r, int piece, const f2* v, float down)
{
    const f2 d = dup2(down);
    unsigned char* at = image + piece * kPiece + r * 16;
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        unsigned hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x, y;
            unpack2(mul2(v[4 * i + e], d), x, y);
            split_pair(x, y, hi[e], lo[e]);
        }
        *reinterpret_cast<uint4*>(at + i * kPiece) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(at + i * kPiece + second) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}
// Descriptor of such a matrix, the sum along the values, from value 16 ks on: 128 bytes from 8 values to the next, kPiece
// from 8 steps or keys to the next.
__device__ __forceinline__ uint64_t desc_kept(unsigned saddr, int ks)
{
    return (uint64_t)(((saddr + ks * 256) >> 4) & 0x3FFFu) | (uint64_t)(128u >> 4) << 16 | (uint64_t)(kPiece >> 4) << 32 | (uint64_t)1u << 46;
}
// The largest of a block's 256 threads' values, which their warps have left in `most`.
__device__ __forceinline__ float most_of_warps(const float (&most)[8])
{
    float m = most[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, most[i]);
    return m;
}
__device__ __forceinline__ float warp_most(float m) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))); }

}  // namespace delta
}  // namespace rnngb
