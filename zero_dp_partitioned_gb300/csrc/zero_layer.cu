// zero_layer.cu -- host checks shared by the layer operators.
#include <map>
#include <mutex>

#include "zero_layer.cuh"

namespace zdp {

int check_mat(const zero_mat* m, int64_t rows, int64_t cols, unsigned types, const char* what) {
    const std::string w(what);
    if (!m) return fail(ZERO_EINVAL, (w + " is NULL").c_str());
    if (m->dtype < 0 || m->dtype > 31 || !(types >> m->dtype & 1u))
        return fail(ZERO_EINVAL, (w + ": unknown or unsupported dtype").c_str());
    if (rows == 0 || cols == 0) return ZERO_OK;
    if (!m->data) return fail(ZERO_EINVAL, (w + ": NULL data").c_str());
    if (rows > 1 && m->ld < cols) return fail(ZERO_EINVAL, (w + ": rows closer than their columns").c_str());
    if (!aligned(m->data, (size_t)elem_size(m->dtype)))
        return fail(ZERO_EALIGN, (w + ": not aligned to its element").c_str());
    return ZERO_OK;
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
