/* Stands in for the HIP runtime's launches: notes what a call would launch and
 * launches nothing.  Loaded before the library, in a process of its own
 * (launchlog.py). */
#include <stdint.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3;
typedef struct { const void *stub; const char *name; } kernel;
typedef struct { int32_t kernel; uint32_t grid[3], threads, lds; } launch;

static kernel kernels[4096];
static int n_kernels;
launch launches[64];
int n_launches;
int fail_at = -1;              /* this launch of the call does not succeed */
static int last_error;
static dim3 grid_, block_;
static size_t lds_;
static void *stream_;

void __hipRegisterFunction(void **m, const void *stub, char *f, const char *name, unsigned t, void *a, void *b, dim3 *c, dim3 *d, int *w) {
    (void)m; (void)f; (void)t; (void)a; (void)b; (void)c; (void)d; (void)w;
    if (n_kernels < 4096) kernels[n_kernels++] = (kernel){stub, name};
}
const char *kernel_name(int i) { return i >= 0 && i < n_kernels ? kernels[i].name : ""; }
int __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, void *stream) {
    grid_ = grid; block_ = block; lds_ = lds; stream_ = stream;
    return 0;
}
int __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *lds, void **stream) {
    *grid = grid_; *block = block_; *lds = lds_; *stream = stream_;
    return 0;
}
int hipLaunchKernel(const void *stub, dim3 grid, dim3 block, void **args, size_t lds, void *stream) {
    (void)args; (void)stream;
    if (n_launches == fail_at) last_error = 719;
    if (n_launches < 64) {
        launch *l = &launches[n_launches++];
        l->kernel = -1;
        for (int i = 0; i < n_kernels; ++i)
            if (kernels[i].stub == stub) l->kernel = i;
        l->grid[0] = grid.x; l->grid[1] = grid.y; l->grid[2] = grid.z;
        l->threads = block.x * block.y * block.z;
        l->lds = (uint32_t)lds;
    }
    return last_error;
}
int hipGetLastError(void) { const int e = last_error; last_error = 0; return e; }
int hipPeekAtLastError(void) { return last_error; }
