/*
 * A plain C caller of the operators around the experts' products: only include/mxq_moe.h and
 * the HIP runtime. It reads router logits (fp32 [tokens, experts]) and token rows (bf16
 * [tokens, width]) from files, chooses top_k experts, sorts, sends the rows to them in MXFP4,
 * widens them to fp32, combines them, and takes the gradients of rows, weights and logits for a
 * gradient equal to the combined result; it also keeps the widened rows in FP8 and takes the
 * gradient of SiLU from them. Every output goes to <prefix>.<name>.
 *
 * usage: mxq_moe_caller tokens experts top_k width logits.bin x.bin prefix   (width % 32 == 0)
 * Exit status: 0 on success, 1 on a usage or I/O error, 2 on a library or HIP error.
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <hip/hip_runtime_api.h>

#include "mxq_moe.h"

typedef struct {
  const char* name;
  void* at; /* on the device */
  size_t bytes;
} buffer;

enum { LOGITS, X, WEIGHTS, EXPERTS, OFFSETS, POSITIONS, ORDER, SORT_WS, CODES, SCALES, ROWS, OUT, DY, DW, DLOGITS, Q8, S8,
       DZ, DB, H, GRAD_WS, BUFFERS };

static int fail(const char* what) {
  fprintf(stderr, "%s failed\n", what);
  return 2;
}

static int read_file(const char* path, buffer* b) {
  FILE* f = fopen(path, "rb");
  void* host = malloc(b->bytes);
  const int ok = f && host && fread(host, 1, b->bytes, f) == b->bytes &&
                 hipMemcpy(b->at, host, b->bytes, hipMemcpyHostToDevice) == hipSuccess;
  if (f) fclose(f);
  free(host);
  return ok;
}

static int write_file(const char* prefix, const buffer* b) {
  char path[4096];
  snprintf(path, sizeof path, "%s.%s", prefix, b->name);
  FILE* f = fopen(path, "wb");
  void* host = malloc(b->bytes);
  const int ok = f && host && hipMemcpy(host, b->at, b->bytes, hipMemcpyDeviceToHost) == hipSuccess &&
                 fwrite(host, 1, b->bytes, f) == b->bytes;
  if (f) fclose(f);
  free(host);
  return ok;
}

int main(int argc, char** argv) {
  if (argc != 8) {
    fprintf(stderr, "usage: %s tokens experts top_k width logits.bin x.bin prefix\n", argv[0]);
    return 1;
  }
  const int64_t T = atoll(argv[1]), E = atoll(argv[2]), k = atoll(argv[3]), W = atoll(argv[4]), R = T * k;
  if (T <= 0 || E <= 0 || k <= 0 || W <= 0 || W % 32) return 1;
  const int64_t groups = (W + 127) / 128;
  const int64_t sort_ws = mxq_expert_sort_workspace(R, E), grad_ws = mxq_act_grad_workspace(R, W, E);
  buffer b[BUFFERS] = {
      {"logits", 0, (size_t)(T * E * 4)}, {"x", 0, (size_t)(T * W * 2)}, {"weights", 0, (size_t)(R * 4)},
      {"experts", 0, (size_t)(R * 4)}, {"offsets", 0, (size_t)(E + 1) * 8}, {"positions", 0, (size_t)(R * 4)},
      {"order", 0, (size_t)(R * 4)}, {"sort_ws", 0, (size_t)(sort_ws + 16)}, {"codes", 0, (size_t)(R * W / 2)},
      {"scales", 0, (size_t)(R * W / 32)}, {"rows", 0, (size_t)(R * W * 4)}, {"out", 0, (size_t)(T * W * 4)},
      {"dy", 0, (size_t)(R * W * 4)}, {"dw", 0, (size_t)(R * 4)}, {"dlogits", 0, (size_t)(T * E * 4)},
      {"q8", 0, (size_t)(R * W)}, {"s8", 0, (size_t)(R * groups * 4)}, {"dz", 0, (size_t)(R * W * 4)},
      {"db", 0, (size_t)(E * W * 4)}, {"h", 0, (size_t)(R * W * 4)}, {"grad_ws", 0, (size_t)(grad_ws + 16)}};
  int i, rc = 0;
  for (i = 0; i < BUFFERS; ++i)
    if (hipMalloc(&b[i].at, b[i].bytes) != hipSuccess) rc = fail("hipMalloc");
  if (!rc && (!read_file(argv[5], &b[LOGITS]) || !read_file(argv[6], &b[X]))) rc = 1;
  int32_t *experts = (int32_t*)b[EXPERTS].at, *pos = (int32_t*)b[POSITIONS].at;
  float *weights = (float*)b[WEIGHTS].at, *dw = (float*)b[DW].at;
  int64_t* offsets = (int64_t*)b[OFFSETS].at;
  if (!rc && mxq_route(b[LOGITS].at, MXQ_F32, T, E, E, k, 1, weights, experts, 0)) rc = fail("mxq_route");
  if (!rc && mxq_expert_sort(experts, R, E, offsets, pos, (int32_t*)b[ORDER].at, b[SORT_WS].at, 0)) rc = fail("mxq_expert_sort");
  if (!rc && mxq_dispatch(b[X].at, MXQ_BF16, T, W, W, pos, k, R, MXQ_ROWS_MXFP4, b[CODES].at, b[SCALES].at, 0))
    rc = fail("mxq_dispatch");
  if (!rc && mxq_dequantize((const uint8_t*)b[CODES].at, (const uint8_t*)b[SCALES].at, MXQ_MXFP4, R, W, 0, b[ROWS].at, MXQ_F32, 0))
    rc = fail("mxq_dequantize");
  if (!rc && mxq_combine(b[ROWS].at, MXQ_F32, R, W, pos, weights, T, k, 0, b[OUT].at, MXQ_F32, 0)) rc = fail("mxq_combine");
  if (!rc && mxq_combine_grad(b[OUT].at, MXQ_F32, b[ROWS].at, MXQ_F32, R, W, pos, weights, T, k, b[DY].at, dw, 0))
    rc = fail("mxq_combine_grad");
  if (!rc && mxq_route_grad(dw, weights, experts, b[LOGITS].at, MXQ_F32, T, E, E, k, 1, b[DLOGITS].at, 0))
    rc = fail("mxq_route_grad");
  if (!rc && mxq_fp8_quantize(b[ROWS].at, MXQ_F32, R, W, W, (uint8_t*)b[Q8].at, (float*)b[S8].at, 0)) rc = fail("mxq_fp8_quantize");
  if (!rc && mxq_fp8_act_grad(b[DY].at, MXQ_F32, (const uint8_t*)b[Q8].at, (const float*)b[S8].at, R, W, MXQ_ACT_SILU,
                              offsets, E, b[DZ].at, (float*)b[DB].at, b[H].at, b[GRAD_WS].at, 0))
    rc = fail("mxq_fp8_act_grad");
  if (!rc && hipDeviceSynchronize() != hipSuccess) rc = fail("hipDeviceSynchronize");
  for (i = WEIGHTS; !rc && i < BUFFERS; ++i)
    if (i != SORT_WS && i != GRAD_WS && !write_file(argv[7], &b[i])) rc = 1;
  for (i = 0; i < BUFFERS; ++i) (void)hipFree(b[i].at);
  return rc;
}
