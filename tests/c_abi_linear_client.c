/* A plain C11 client of liblmc's linear attention and rotation: one request's
 * prompt, its last token as a step, and the queries turned in place, through
 * the C ABI on the default stream with device memory from the CUDA runtime's C
 * API.
 *
 * usage: c_abi_linear_client DIR
 *   DIR/case.txt   "block_size heads dim tokens"
 *   DIR/q.bin, k.bin, v.bin (bfloat16 [tokens][heads][dim]), DIR/decay.bin
 *   (float [tokens][heads]), DIR/frequencies.bin (float [dim / 2])
 * writes DIR/out.out, DIR/turned.out and DIR/status.out */
#include <cuda_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "lmc.h"

#define CHECK(cond, what)                          \
    do {                                           \
        if (!(cond)) {                             \
            fprintf(stderr, "failed: %s\n", what); \
            return 1;                              \
        }                                          \
    } while (0)

static char path[4096];
static const char *in_dir(const char *dir, const char *name) {
    snprintf(path, sizeof path, "%s/%s", dir, name);
    return path;
}

static void *device(const void *host, size_t n) {
    void *d = NULL;
    if (cudaMalloc(&d, n) != cudaSuccess)
        return NULL;
    if (host ? cudaMemcpy(d, host, n, cudaMemcpyHostToDevice) != cudaSuccess : cudaMemset(d, 0, n) != cudaSuccess)
        return NULL;
    return d;
}

static void *from_file(const char *dir, const char *name, size_t n) {
    void *buf = malloc(n), *d = NULL;
    FILE *f = fopen(in_dir(dir, name), "rb");
    if (buf && f && fread(buf, 1, n, f) == n)
        d = device(buf, n);
    if (f)
        fclose(f);
    free(buf);
    return d;
}

static int to_file(const char *dir, const char *name, const void *dev, size_t n) {
    void *buf = malloc(n);
    FILE *f = fopen(in_dir(dir, name), "wb");
    const int ok = buf && f && cudaMemcpy(buf, dev, n, cudaMemcpyDeviceToHost) == cudaSuccess && fwrite(buf, 1, n, f) == n;
    if (f)
        fclose(f);
    free(buf);
    return ok;
}

int main(int argc, char **argv) {
    CHECK(argc == 2, "usage: c_abi_linear_client DIR");
    const char *dir = argv[1];
    int N, H, d, n;
    FILE *f = fopen(in_dir(dir, "case.txt"), "r");
    CHECK(f && fscanf(f, "%d %d %d %d", &N, &H, &d, &n) == 4, "case.txt");
    fclose(f);
    const int cols = (n + N - 1) / N;

    lmc_layer_spec layer;
    memset(&layer, 0, sizeof layer);
    layer.kind = LMC_LAYER_KDA;
    layer.conv_bytes = 64;
    layer.rec_bytes = (int64_t)H * d * d * 4;
    lmc_layout_params params;
    memset(&params, 0, sizeof params);
    params.num_layers = 1;
    params.mode = LMC_LAYOUT_PADDED;
    params.grouping = LMC_GROUP_SPLIT;
    params.block_size = N;
    params.mem_bytes = cols * (layer.conv_bytes + layer.rec_bytes);
    params.layers = &layer;
    lmc_layout *L = NULL;
    CHECK(lmc_layout_build(&params, &L) == LMC_OK, "lmc_layout_build");

    int32_t *ids = malloc(sizeof(int32_t) * (size_t)(n > cols ? n : cols));
    CHECK(ids, "malloc");
    for (int i = 0; i < cols; i++)
        ids[i] = cols - 1 - i;
    int32_t *table = device(ids, sizeof(int32_t) * (size_t)cols);
    for (int i = 0; i < n; i++)
        ids[i] = i;
    int32_t *positions = device(ids, sizeof(int32_t) * (size_t)n);
    const int32_t most[2] = {0, n - 1}, before[2] = {0, n - 1};
    int32_t *starts = device(most, sizeof most), *lengths = device(before, sizeof before);
    const size_t row = (size_t)H * (size_t)d, bytes = (size_t)n * row * 2;
    uint8_t *q = from_file(dir, "q.bin", bytes), *k = from_file(dir, "k.bin", bytes), *v = from_file(dir, "v.bin", bytes);
    float *decay = from_file(dir, "decay.bin", (size_t)n * (size_t)H * 4);
    float *frequencies = from_file(dir, "frequencies.bin", (size_t)d / 2 * 4);
    uint8_t *out = device(NULL, bytes), *pool = device(NULL, (size_t)params.mem_bytes);
    uint32_t *status = device(NULL, 4);
    CHECK(table && positions && starts && lengths && q && k && v && decay && frequencies && out && pool && status,
          "device memory");

    lmc_linear a;
    memset(&a, 0, sizeof a);
    a.dtype = LMC_E_BF16;
    a.num_requests = 1;
    a.num_heads = a.num_key_heads = H;
    a.key_dim = a.value_dim = d;
    a.scale = 0.125f;
    a.table.table = table;
    a.table.row_stride = a.table.num_cols = cols;
    a.lengths = lengths;
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.decay = decay;
    a.q_row_stride = a.k_row_stride = a.v_row_stride = a.out_row_stride = (int64_t)row;
    a.q_head_stride = a.k_head_stride = a.v_head_stride = a.out_head_stride = d;
    a.decay_row_stride = H;
    a.decay_head_stride = 1;
    int64_t need = 0;
    CHECK(lmc_linear_scan_workspace(L, 0, 1, n - 1, H, &need) == LMC_OK, "lmc_linear_scan_workspace");
    void *workspace = device(NULL, (size_t)need);
    CHECK(workspace, "workspace");
    CHECK(lmc_linear_scan(L, &a, starts, n - 1, pool, workspace, need - 1, status, NULL) == LMC_ERR_INVALID_ARG,
          "a short workspace is refused");
    CHECK(lmc_linear_scan(L, &a, starts, n - 1, pool, workspace, need, status, NULL) == LMC_OK, "lmc_linear_scan");
    const size_t last = (size_t)(n - 1) * row * 2;
    a.q = q + last;
    a.k = k + last;
    a.v = v + last;
    a.out = out + last;
    a.decay = decay + (size_t)(n - 1) * (size_t)H;
    a.lengths = lengths + 1;
    CHECK(lmc_linear_step(L, &a, pool, status, NULL) == LMC_OK, "lmc_linear_step");

    lmc_rotation turn;
    memset(&turn, 0, sizeof turn);
    turn.num_heads = H;
    turn.head_dim = turn.rot_dim = d;
    turn.rot_mode = LMC_ROT_HALVES;
    turn.mscale = 1.0f;
    turn.frequencies = frequencies;
    turn.positions = positions;
    CHECK(lmc_rotate(&turn, LMC_E_BF16, q, (int64_t)row, d, q, (int64_t)row, d, n, NULL) == LMC_OK, "lmc_rotate");
    CHECK(cudaDeviceSynchronize() == cudaSuccess, "synchronize");

    uint32_t st = 0;
    CHECK(to_file(dir, "out.out", out, bytes) && to_file(dir, "turned.out", q, bytes) &&
              cudaMemcpy(&st, status, 4, cudaMemcpyDeviceToHost) == cudaSuccess,
          "outputs");
    f = fopen(in_dir(dir, "status.out"), "w");
    CHECK(f && fprintf(f, "%u\n", st) > 0 && fclose(f) == 0, "status.out");
    lmc_layout_free(L);
    free(ids);
    puts("done");
    return 0;
}
