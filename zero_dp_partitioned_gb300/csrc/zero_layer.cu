// zero_layer.cu -- host checks shared by the layer operators.
#include <map>
#include <mutex>
#include <utility>

#include "zero_layer.cuh"

namespace zdp {

int refuse(int code, const char* call, const char* what, const char* why) {
    set_error(std::string(call) + ": " + what + why);
    return code;
}

int check_mat(const zero_mat* m, int64_t rows, int64_t cols, unsigned types, const char* call, const char* what) {
    if (!m) return refuse(ZERO_EINVAL, call, what, " is NULL");
    if (m->dtype < 0 || m->dtype > 31 || !(types >> m->dtype & 1u))
        return refuse(ZERO_EINVAL, call, what, ": unknown or unsupported dtype");
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!m->data) return refuse(ZERO_EINVAL, call, what, ": NULL data");
    if (rows > 1 && m->ld < cols) return refuse(ZERO_EINVAL, call, what, ": rows closer than their columns");
    if (!aligned(m->data, (size_t)elem_size(m->dtype)))
        return refuse(ZERO_EALIGN, call, what, ": not aligned to its element");
    return ZERO_OK;
}

int raise_smem(const void* f, size_t smem, const char* who) {
    static std::mutex mu;
    static std::map<std::pair<int, const void*>, size_t> raised;     // (device, kernel) -> its limit
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, who);
    std::lock_guard<std::mutex> g(mu);
    size_t& had = raised[{dev, f}];
    if (smem <= (had ? had : 40 * 1024)) return ZERO_OK;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) had = smem;
    return cuda_fail(e, who);
}

int sm_count() {
    static std::mutex mu;
    static std::map<int, int> known;                 // device -> SM count
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> g(mu);
        const auto it = known.find(dev);
        if (it != known.end()) return it->second;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) known[dev] = n;
    }
    if (e != cudaSuccess) {
        cuda_fail(e, "device query");
        return 0;
    }
    return n;
}

}  // namespace zdp
