/* A plain C11 client of liblmc's token operators: one request's entries are
 * appended to an MLA layer, attended with their weights, the heaviest selected
 * and moved into other blocks, through the C ABI on the default stream with
 * device memory from the CUDA runtime's C API.
 *
 * usage: c_abi_tokens_client DIR
 *   DIR/case.txt   "N entry_dim value_dim heads tokens budget recent"
 *   DIR/rows.bin (bfloat16 [tokens][entry_dim]), DIR/q.bin (bfloat16 [heads][entry_dim])
 * writes DIR/out.out, DIR/lse.out, DIR/weights.out, DIR/kept.out,
 * DIR/scores.out, DIR/moved.out (the kept entries, read back from the pool)
 * and DIR/status.out ("status kept_length") */
#include <cuda_runtime.h>
#include <math.h>
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
    CHECK(argc == 2, "usage: c_abi_tokens_client DIR");
    const char *dir = argv[1];
    int N, E, V, H, n, budget, recent;
    FILE *f = fopen(in_dir(dir, "case.txt"), "r");
    CHECK(f && fscanf(f, "%d %d %d %d %d %d %d", &N, &E, &V, &H, &n, &budget, &recent) == 7, "case.txt");
    fclose(f);
    const int cols = (n + N - 1) / N, fresh = (budget + N - 1) / N, blocks = cols + fresh;

    lmc_layer_spec layer;
    memset(&layer, 0, sizeof layer);
    layer.kind = LMC_LAYER_MLA;
    layer.token_bytes = 2 * (int64_t)E;
    lmc_layout_params params;
    memset(&params, 0, sizeof params);
    params.num_layers = 1;
    params.mode = LMC_LAYOUT_PADDED;
    params.grouping = LMC_GROUP_SPLIT;
    params.block_size = N;
    params.mem_bytes = (int64_t)blocks * N * 2 * E;
    params.layers = &layer;
    lmc_layout *L = NULL;
    CHECK(lmc_layout_build(&params, &L) == LMC_OK, "lmc_layout_build");
    lmc_layout_info info;
    CHECK(lmc_layout_query(L, &info) == LMC_OK && info.num_blocks == blocks, "lmc_layout_query");
    const lmc_layer_desc desc = info.layers[0];

    int32_t *ids = malloc(sizeof(int32_t) * (size_t)(n > blocks ? n : blocks));
    CHECK(ids, "malloc");
    for (int i = 0; i < blocks; i++)
        ids[i] = i;
    int32_t *src = device(ids, sizeof(int32_t) * (size_t)blocks), *dst = src + cols;
    for (int i = 0; i < n; i++)
        ids[i] = i;
    int32_t *positions = device(ids, sizeof(int32_t) * (size_t)n), *requests = device(NULL, sizeof(int32_t) * (size_t)n);
    int32_t *lengths = device(&n, sizeof n);
    const size_t row_bytes = (size_t)E * 2;
    void *rows = from_file(dir, "rows.bin", (size_t)n * row_bytes), *q = from_file(dir, "q.bin", (size_t)H * row_bytes);
    uint8_t *pool = device(NULL, (size_t)params.mem_bytes);
    uint32_t *status = device(NULL, 4);
    void *out = device(NULL, (size_t)H * (size_t)V * 2);
    float *lse = device(NULL, (size_t)H * 4), *weights = device(NULL, (size_t)n * 4);
    int32_t *kept = device(NULL, (size_t)budget * 4), *kept_length = device(NULL, 4);
    float *scores = device(NULL, (size_t)budget * 4);
    CHECK(src && positions && requests && lengths && rows && q && pool && status && out && lse && weights && kept &&
              kept_length && scores,
          "device memory");

    lmc_entries entries;
    memset(&entries, 0, sizeof entries);
    entries.layer = 0;
    entries.dtype = LMC_E_BF16;
    entries.entry_dim = E;
    entries.num_requests = 1;
    entries.scale = 1.0f;
    entries.table.table = src;
    entries.table.row_stride = cols;
    entries.table.num_cols = cols;
    CHECK(lmc_append(L, &entries, pool, requests, positions, rows, LMC_E_BF16, E, n, status, NULL) == LMC_OK,
          "lmc_append");

    int64_t bytes = 0;
    CHECK(lmc_attend_workspace(L, 0, 1, H, V, n, 1, &bytes) == LMC_OK, "lmc_attend_workspace");
    void *workspace = device(NULL, (size_t)bytes);
    CHECK(workspace, "workspace");
    lmc_attention a;
    memset(&a, 0, sizeof a);
    a.lengths = lengths;
    a.max_length = n;
    a.q = q;
    a.q_request_stride = (int64_t)H * E;
    a.q_head_stride = E;
    a.out = out;
    a.out_request_stride = (int64_t)H * V;
    a.out_head_stride = V;
    a.lse = lse;
    a.lse_request_stride = H;
    a.weights = weights;
    a.weights_request_stride = n;
    a.q_dtype = LMC_E_BF16;
    a.num_heads = H;
    a.value_dim = V;
    a.softmax_scale = 1.0f / sqrtf((float)E);
    CHECK(lmc_attend(L, &entries, pool, &a, workspace, bytes - 1, status, NULL) == LMC_ERR_INVALID_ARG,
          "a short workspace is refused");
    CHECK(lmc_attend(L, &entries, pool, &a, workspace, bytes, status, NULL) == LMC_OK, "lmc_attend");

    CHECK(lmc_select_tokens(weights, n, n, 1, 1, lengths, n, budget, recent, kept, scores, kept_length, status, NULL) ==
              LMC_OK,
          "lmc_select_tokens");
    lmc_block_table to = entries.table;
    to.table = dst;
    to.row_stride = to.num_cols = fresh;
    CHECK(lmc_move_tokens(L, desc.kv_group, pool, 1, &entries.table, &to, kept, 1, budget, budget, kept_length, budget,
                          status, NULL) == LMC_OK,
          "lmc_move_tokens");
    CHECK(cudaDeviceSynchronize() == cudaSuccess, "synchronize");

    CHECK(to_file(dir, "out.out", out, (size_t)H * (size_t)V * 2) && to_file(dir, "lse.out", lse, (size_t)H * 4) &&
              to_file(dir, "weights.out", weights, (size_t)n * 4) && to_file(dir, "kept.out", kept, (size_t)budget * 4) &&
              to_file(dir, "scores.out", scores, (size_t)budget * 4) &&
              to_file(dir, "moved.out", pool + desc.base + (int64_t)cols * desc.stride, (size_t)budget * row_bytes),
          "outputs");
    uint32_t st = 0;
    int32_t kl = 0;
    CHECK(cudaMemcpy(&st, status, 4, cudaMemcpyDeviceToHost) == cudaSuccess &&
              cudaMemcpy(&kl, kept_length, 4, cudaMemcpyDeviceToHost) == cudaSuccess,
          "status");
    f = fopen(in_dir(dir, "status.out"), "w");
    CHECK(f && fprintf(f, "%u %d\n", st, kl) > 0 && fclose(f) == 0, "status.out");
    lmc_layout_free(L);
    free(ids);
    puts("done");
    return 0;
}
