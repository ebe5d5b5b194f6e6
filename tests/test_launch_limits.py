"""What the host keeps about kernels and the device from one launch to the next, on a stand-in for the CUDA runtime (no GPU): a kernel's
shared-memory limit never ends up below what a launch asked for, whichever threads and records raise it, and a query that failed is
not taken for an answer."""
import os
import shutil
import subprocess

import pytest

import dense_gemm_blackwell_gb300 as dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_blackwell_gb300", "csrc")


def nvcc():
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    return None


def compiled(path, name, source):
    """{first word: the others} of what the host program prints."""
    cc = nvcc()
    if cc is None:
        pytest.skip("nvcc not available")
    src, exe = path / (name + ".cu"), path / name
    src.write_text(source)
    done = subprocess.run([cc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                          capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout
    return {line.split()[0]: [int(v) for v in line.split()[1:]] for line in out.splitlines()}


# The runtime's calls that set and read a kernel's limit.  A device's blocks may have 227 KB, of which the kernels here hold 512 bytes.
RUNTIME = r'''
#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <functional>
#include <map>
#include <mutex>
#include <thread>
#include <cuda_runtime.h>

namespace fake {
constexpr int kOptin = 232448, kStatic = 512;
std::mutex mutex;
std::map<const void*, int> limit;
cudaError_t last_error = cudaSuccess;
std::function<void()> on_set = [] {};
template <typename K>
cudaError_t set_attribute(K kern, cudaFuncAttribute, int value) {
    on_set();
    std::lock_guard<std::mutex> hold(mutex);
    if (value > kOptin - kStatic) {
        last_error = cudaErrorInvalidValue;
        return cudaErrorInvalidValue;
    }
    limit[(const void*)kern] = value;
    return cudaSuccess;
}
template <typename K>
cudaError_t get_attributes(cudaFuncAttributes* a, K) {
    *a = cudaFuncAttributes{};
    a->sharedSizeBytes = kStatic;
    return cudaSuccess;
}
inline cudaError_t get_device(int* device) {
    *device = 0;
    return cudaSuccess;
}
inline cudaError_t device_attribute(int* value, cudaDeviceAttr attr, int) {
    if (attr != cudaDevAttrMaxSharedMemoryPerBlockOptin) return cudaErrorInvalidValue;
    *value = kOptin;
    return cudaSuccess;
}
}  // namespace fake
#define cudaFuncSetAttribute fake::set_attribute
#define cudaFuncGetAttributes fake::get_attributes
#define cudaGetDevice fake::get_device
#define cudaDeviceGetAttribute fake::device_attribute
'''


def test_shared_memory_limits(tmp_path):
    """Two threads that ask for two sizes of one kernel at once; two records of one kernel; more than a block may have."""
    got = compiled(tmp_path, "limits", RUNTIME + r'''
#include "common.cuh"
__global__ void one(int) {}
__global__ void two(int) {}
__global__ void three(int) {}

int main() {
    using dgb::ensure_smem_limit;
    static std::atomic<int> set_one[dgb::kMaxDevices], set_two[2][dgb::kMaxDevices], set_three[dgb::kMaxDevices];
    {
        // the first thread's call is held up on its way into the driver until the other thread is done (or cannot get on)
        std::mutex m;
        std::condition_variable cv;
        bool held = false, done = false;
        fake::on_set = [&] {
            std::unique_lock<std::mutex> l(m);
            if (held) return;
            held = true;
            cv.notify_all();
            cv.wait_for(l, std::chrono::seconds(1), [&] { return done; });
        };
        std::thread small([&] { ensure_smem_limit(one, 60000, set_one); });
        {
            std::unique_lock<std::mutex> l(m);
            cv.wait_for(l, std::chrono::seconds(10), [&] { return held; });
        }
        std::thread large([&] {
            ensure_smem_limit(one, 150000, set_one);
            std::lock_guard<std::mutex> l(m);
            done = true;
            cv.notify_all();
        });
        small.join();
        large.join();
        fake::on_set = [] {};
        const int status = ensure_smem_limit(one, 100000, set_one);
        std::printf("threads %d %d\n", status, fake::limit[(const void*)one]);
    }
    ensure_smem_limit(two, 150000, set_two[0]);
    ensure_smem_limit(two, 60000, set_two[1]);
    std::printf("records %d %d\n", (int)ensure_smem_limit(two, 150000, set_two[0]), fake::limit[(const void*)two]);
    int over = ensure_smem_limit(three, fake::kOptin, set_three);
    std::printf("over %d %d %d\n", over, (int)fake::last_error, (int)ensure_smem_limit(three, fake::kOptin - fake::kStatic, set_three));
    std::printf("all %d\n", fake::limit[(const void*)three]);
    return 0;
}
''')
    for name in ("threads", "records"):
        status, limit = got[name]
        assert status == 0 and limit >= 150000, (name, got[name])
    assert got["over"][0] == got["over"][1] != 0 and got["over"][2] == 0 and got["all"] == [232448 - 512]


def test_a_failed_query_of_resident_clusters_is_not_kept(tmp_path):
    """16 tokens of 28672 columns fit a cluster's shared memory only: the call whose query fails says so, and the next one has the
    device's answer, which is asked for once."""
    got = compiled(tmp_path, "resident", RUNTIME + r'''
#include "int4_matmul.cu"

static bool fails = true;
static int queries = 0, launches = 0, grid = 0, split = 0;
namespace dgb {
gemm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA; }
gemm_status_t device_facts(DeviceFacts* out) {
    out->device = 0;
    out->sms = 152;
    out->smem_optin = fake::kOptin;
    return GEMM_OK;
}
int int4_resident(int k_split_log, int per_sm) {
    ++queries;
    return fails ? 0 : (per_sm * 152 * 9 / 10) >> k_split_log;
}
cudaError_t int4_resident(int k_split_log, int per_sm, int* clusters) {
    if ((*clusters = int4_resident(k_split_log, per_sm)) == 0) return cudaErrorInvalidValue;
    return cudaSuccess;
}
cudaError_t launch_int4_bf16(const Int4Params& p, bool, cudaStream_t) {
    ++launches;
    grid = p.grid;
    split = 1 << p.k_split_log;
    return cudaSuccess;
}
cudaError_t launch_int4_f16(const Int4Params& p, bool gated, cudaStream_t stream) { return launch_int4_bf16(p, gated, stream); }
}  // namespace dgb

int main() {
    int4_matmul_args_t a = {};
    a.tokens = 16;
    a.n = 8192;
    a.k = 28672;
    a.group = 128;
    a.dtype = GEMM_BF16;
    a.activation = GATED_NONE;
    a.x = a.codes = a.scales = (void*)4096;
    a.y = (void*)4096;
    std::printf("failed %d %d\n", (int)int4_matmul_run(&a, nullptr), launches);
    fails = false;
    const int status = (int)int4_matmul_run(&a, nullptr);
    std::printf("next %d %d %d %d\n", status, launches, grid, split);
    queries = 0;
    std::printf("again %d %d %d\n", (int)int4_matmul_run(&a, nullptr), grid, queries);
    return 0;
}
''')
    assert got["failed"] == [dg.GEMM_ERR_CUDA, 0]
    status, launches, grid, split = got["next"]
    assert status == 0 and launches == 1 and split >= 4 and grid > 100, got["next"]
    assert got["again"] == [0, grid, 0]


# gated.cu's plans on stand-ins for the products that they are made of
GATED = RUNTIME + r'''
#include "gated.cu"
#include <vector>

struct gemm_plan_s {};
static std::vector<gemm_desc_t> made;
static bool fails = false;
namespace dgb {
gemm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? GEMM_OK : GEMM_ERR_CUDA; }
gemm_status_t device_facts(DeviceFacts* out) {
    out->device = 0;
    out->sms = 152;
    out->smem_optin = fake::kOptin;
    return GEMM_OK;
}
int gated_few_max_clusters(int, int k_split, const DeviceFacts& dev) { return fails && k_split > 1 ? 0 : dev.sms / k_split; }
cudaError_t gated_few_max_clusters(int dtype, int k_split, const DeviceFacts& dev, int* clusters) {
    *clusters = gated_few_max_clusters(dtype, k_split, dev);
    return *clusters > 0 ? cudaSuccess : cudaErrorInvalidValue;
}
cudaError_t launch_gated_few(const GatedFewParams&, int, dim3, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_gated(const PersistentParams&, const GatedTail&, int, int, int, size_t, cudaStream_t) { return cudaSuccess; }
gemm_status_t product_params(gemm_plan_t, const void*, const void*, void*, PersistentParams*) { return GEMM_OK; }
gemm_status_t encode_rows_map(CUtensorMap*, int, const void*, int64_t, int64_t, int64_t, int) { return GEMM_OK; }
gemm_device_error_t* device_record(gemm_plan_t) { return nullptr; }
}  // namespace dgb
extern "C" {
gemm_status_t gemm_plan_create(gemm_plan_t* plan, const gemm_desc_t* d) {
    made.push_back(*d);
    *plan = new gemm_plan_s;
    return GEMM_OK;
}
gemm_status_t gemm_plan_info(gemm_plan_t, gemm_plan_info_t* info) {
    *info = gemm_plan_info_t{};
    return GEMM_OK;
}
gemm_status_t gemm_plan_destroy(gemm_plan_t plan) {
    delete plan;
    return GEMM_OK;
}
gemm_status_t gemm_run(gemm_plan_t, const void*, const void*, void*, const float*, const float*, gemm_stream_t) { return GEMM_OK; }
gemm_status_t gemm_sync_status(gemm_plan_t, gemm_stream_t, gemm_device_error_t*) { return GEMM_OK; }
}

// One word of the name, then status, whether the kernel for few tokens is taken and its split.
static void plan(const char* name, int64_t tokens, int64_t features, int64_t k, int gradients = 0) {
    made.clear();
    gated_desc_t d = {};
    d.tokens = tokens;
    d.features = features;
    d.k = k;
    d.dtype = d.dtype_dw = GEMM_BF16;
    d.gradients = gradients;
    gated_plan_t p = nullptr;
    gated_plan_info_t info = {};
    const int status = (int)gated_plan_create(&p, &d);
    if (p) gated_plan_info(p, &info);
    std::printf("%s %d %d %d", name, status, info.few_tiles, info.k_split);
    for (const gemm_desc_t& g : made) std::printf(" %d", g.tile_n);
    std::printf("\n");
    gated_plan_destroy(p);
}
'''


def test_a_failed_query_is_the_error_of_a_gated_plan(tmp_path):
    """Where the clusters of a split cannot be asked for, the plan says so instead of quietly going without them."""
    got = compiled(tmp_path, "plans", GATED + r'''
int main() {
    plan("whole", 4, 1024, 8192);
    fails = true;
    plan("failed", 4, 1024, 8192);
    plan("pipeline", 4096, 1024, 8192);
    return 0;
}
''')
    assert got["whole"][:2] == [0, 1] and got["whole"][2] > 1       # K is shared where it can be
    assert got["failed"][:2] == [dg.GEMM_ERR_CUDA, 0]
    assert got["pipeline"][:2] == [0, 0]


def test_wide_tiles_of_the_gradients_products(tmp_path):
    """512 columns a tile where tiles of SM pairs fill their waves; the planner's own where 128 rows or fewer are lone CTAs' tiles."""
    got = compiled(tmp_path, "plans", GATED + r'''
int main() {
    plan("batch", 4096, 8192, 4096, 1);
    plan("ragged", 4096, 8192, 4104, 1);
    plan("few", 64, 8192, 32768, 1);
    plan("narrow", 16384, 64, 32768, 1);
    return 0;
}
''')
    # of the forward product, of the rows' gradients, of the weights' gradients
    assert got["batch"][0] == 0 and got["batch"][4:] == [512, 512]
    assert got["ragged"][4:] == [0, 0]
    assert got["few"][4:] == [0, 0]
    assert got["narrow"][4:][1] == 0


def test_few_tiles_of_a_long_k_share_it(tmp_path):
    """The pipeline's tiles may be split along K where most of the device would have none and K is long."""
    got = compiled(tmp_path, "plans", GATED + r'''
static void flags(const char* name, int64_t tokens, int64_t features, int64_t k) {
    plan("-", tokens, features, k);
    std::printf("%s %d\n", name, (made[0].flags & GEMM_FLAG_NO_STREAM_K) != 0);
}
int main() {
    flags("long", 130, 512, 28672);
    flags("longer", 256, 1024, 28672);
    flags("short", 130, 1024, 4096);
    flags("medium", 130, 1024, 6144);
    flags("many", 256, 4096, 14336);
    return 0;
}
''')
    whole = {name: flag[0] for name, flag in got.items() if name != "-"}
    assert whole == {"long": 0, "longer": 0, "short": 1, "medium": 1, "many": 1}
