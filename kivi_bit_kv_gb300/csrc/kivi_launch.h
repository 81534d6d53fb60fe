// kivi_launch.h -- host-side launchers behind the C ABI (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kivi.h"

namespace kivi {

// Streaming multiprocessors of the current device (cached per device).
int sm_count();

// Lets `kern` use `bytes` of dynamic shared memory; asks the runtime once per
// device (`done`: a static of the launcher).  `bytes` is a constant of the
// kernel, so that host threads that race ask for the same.
template <class Kern>
inline cudaError_t allow_smem(Kern kern, int bytes, int (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && __atomic_load_n(&done[dev], __ATOMIC_RELAXED))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64)
        __atomic_store_n(&done[dev], 1, __ATOMIC_RELAXED);
    return e;
}

// Number of decode chunks (one CTA per KV head and chunk) that cover Tmax.
int pv_chunks(const kivi_cache& c, int Hq);

cudaError_t launch_quant_keys(const kivi_cache& c, const uint16_t* K, int T,
                              const int32_t* seq_lens, cudaStream_t s);
cudaError_t launch_quant_values(const kivi_cache& c, const uint16_t* V, int T,
                                const int32_t* seq_lens, cudaStream_t s);
cudaError_t launch_dequant(const kivi_cache& c, int which, uint16_t* out, int T_out,
                           cudaStream_t s);
cudaError_t launch_append(const kivi_cache& c, const uint16_t* k, const uint16_t* v,
                          int32_t* status, cudaStream_t s);
cudaError_t launch_append_path(const kivi_cache& c, const uint16_t* k, const uint16_t* v, int N,
                               const int32_t* path, int P, const int32_t* counts, int32_t* status,
                               cudaStream_t s);
// Scores of the quantized groups and the n_keep best of each (b, h).
cudaError_t launch_block_select(const kivi_cache& c, const uint16_t* q, int Hq, int32_t* blocks, int n_keep,
                                float* scores, cudaStream_t s);
// Attention of N query tokens per sequence over the cache: all of it and the
// drafted tokens (blocks NULL), or the listed key groups and the residual
// (N = 1, k NULL).
struct AttendArgs {
    const uint16_t* q;       // [B][Hq][N][D]
    const uint16_t* k;       // [B][H][N][D] or NULL
    const uint16_t* v;
    const uint64_t* mask;    // [B][N][ceil(N/64)]
    const int32_t* n_draft;  // [B] or NULL
    const int32_t* blocks;   // [B][H][n_keep] or NULL
    float* out;              // [B][Hq][N][D]
    float sm_scale;
    int32_t Hq, N, n_keep;
};
cudaError_t launch_attend(const kivi_cache& c, const AttendArgs& a, void* ws, cudaStream_t s);
// The same for one head dimension and code width (0: keys and values differ);
// instantiated in attend_d<D>_*.cu.
template <int D, int B>
cudaError_t launch_attend_b(const kivi_cache& c, const AttendArgs& a, float* ws, cudaStream_t s);
// Workspace bytes of a call with N drafted tokens, and of any with up to N.
size_t attend_ws_bytes(const kivi_cache& c, int Hq, int N);
size_t attend_ws_bytes_upto(const kivi_cache& c, int Hq, int N);
cudaError_t launch_decode_qk(const kivi_cache& c, const uint16_t* q, int Hq, float sm_scale,
                             float* logits, int ld_logits, cudaStream_t s);
// ws_o: [B*Hq][nchunks][D], ws_m / ws_l: [B*Hq][nchunks] (fp32).
cudaError_t launch_decode_pv(const kivi_cache& c, const float* logits, int ld_logits, int Hq,
                             float* out, float* ws_o, float* ws_m, float* ws_l,
                             cudaStream_t s);

// q . K, softmax and p . V in one persistent pipelined kernel (one CTA per
// SM) plus a combine kernel for rows that CTA ranges cut; any bits_k, bits_v.
// ws: stream_ws_bytes(c, Hq) bytes.
cudaError_t launch_decode_attention(const kivi_cache& c, const uint16_t* q, int Hq, float sm_scale,
                                    float* out, float* ws, cudaStream_t s);
// Workspace bytes of launch_decode_attention (grid bounded by kMaxStreamCTAs).
size_t stream_ws_bytes(const kivi_cache& c, int Hq);

// The decode kernels of one head dimension D (64, 128, 256), without the
// combine step; instantiated in decode_d<D>.cu.
template <int D>
cudaError_t launch_decode_qk_d(const kivi_cache& c, const uint16_t* q, int Hq, float sm_scale, float* logits,
                               int ld_logits, cudaStream_t s);
template <int D>
cudaError_t launch_decode_pv_d(const kivi_cache& c, const float* logits, int ld_logits, int Hq, float* ws_o,
                               float* ws_m, float* ws_l, cudaStream_t s);
// The streamed fused decode of one head dimension D and key width BK (all
// value widths and query heads per pass), instantiated in
// decode_stream_d<D>_k<BK>.cu.
template <int D, int BK>
cudaError_t launch_decode_stream(const kivi_cache& c, const uint16_t* q, int Hq, float sm_scale, float* out,
                                 float* ws, cudaStream_t s);

// Compact payload (include/kivi.h): its size for host lengths lens[B], and
// the export / import kernels (header checks and size limits on the device).
size_t payload_bytes(const kivi_cache& c, const int32_t* lens);
cudaError_t launch_export(const kivi_cache& c, void* dst, size_t dst_bytes, uint64_t fingerprint,
                          int32_t* status, cudaStream_t s);
cudaError_t launch_import(const kivi_cache& c, const void* src, size_t src_bytes, uint64_t fingerprint,
                          int32_t* status, cudaStream_t s);

// The argument checks kivi_decode_pv makes before it looks at its workspace
// (cache, Hq, logits, out); KIVI_OK or the status it would return.
int32_t check_decode_pv_args(const kivi_cache* c, const float* logits, int32_t ld_logits, int32_t Hq,
                             const float* out);

#ifdef KIVI_CHECKS
// Read and clear the check word of each translation unit with checked kernels.
int32_t check_word_quant();
int32_t check_word_dequant();
int32_t check_word_append();
int32_t check_word_payload();
int32_t check_word_decode();
int32_t check_word_decode_d64();
int32_t check_word_decode_d128();
int32_t check_word_decode_d256();
int32_t check_word_select();
template <int D, int B>
int32_t check_word_attend_b();
int32_t check_word_attend();
#endif

// Sets the message kivi_last_error() returns on this host thread; returns status.
int32_t record_error(int32_t status, const char* message);

}  // namespace kivi
