// The attention's launches against a CUDA runtime of this file's own, in which a kernel's attributes belong to
// the device that is current when they are set, as they do in CUDA's: three devices, of which the third refuses
// the first attribute that is set on it. Prints what went wrong; exits 0 if nothing did.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <map>
#include <utility>

#include "hc_spec.h"

namespace {

int device = 0, refusals = 0, launches = 0, grid = 0, wrong = 0;
std::map<std::pair<int, const void *>, int> limits;  // of dynamic shared memory, where one was set
constexpr int kPerSm[3] = {2, 3, 1}, kSms[3] = {152, 100, 152};

void expect(bool ok, const char *what, int line)
{
    if (!ok) {
        std::printf("line %d: %s\n", line, what);
        ++wrong;
    }
}
#define EXPECT(x) expect(x, #x, __LINE__)

CUresult encode(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    return CUDA_SUCCESS;
}

}  // namespace

extern "C" {

void **__cudaRegisterFatBinary(void *)
{
    static void *handle;
    return &handle;
}
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void **, const char *, char *, const char *, int, uint3 *, uint3 *, dim3 *, dim3 *, int *) {}
cudaError_t __cudaPopCallConfiguration(dim3 *, dim3 *, size_t *, void *) { return cudaErrorUnknown; }
cudaError_t __cudaGetKernel(cudaKernel_t *, const void *) { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void **, size_t, cudaStream_t) { return cudaErrorUnknown; }

cudaError_t cudaGetDevice(int *d)
{
    *d = device;
    return cudaSuccess;
}

cudaError_t cudaFuncSetAttribute(const void *f, cudaFuncAttribute a, int value)
{
    if (device == 2 && refusals == 0) {
        ++refusals;
        return cudaErrorNotReady;
    }
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize)
        limits[{device, f}] = value;
    return cudaSuccess;
}

cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int threads, size_t)
{
    *n = threads > 128 ? 1 : kPerSm[device];  // the wide kernel's blocks take an SM's shared memory
    return cudaSuccess;
}

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *c, const void *f, void **)
{
    ++launches;
    if (c->dynamicSmemBytes == 0)
        return cudaSuccess;  // a join
    const auto at = limits.find({device, f});
    grid = (int)c->gridDim.x;
    return (int)c->dynamicSmemBytes <= (at == limits.end() ? 48 * 1024 : at->second) ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t cudaGetDriverEntryPointByVersion(const char *, void **f, unsigned, unsigned long long, cudaDriverEntryPointQueryResult *r)
{
    *f = reinterpret_cast<void *>(&encode);
    if (r)
        *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}

}  // extern "C"

static cudaError_t attend(int type, int group, int D, int T, int G)
{
    tshc::AttnParams p{};
    p.c.type = type;
    p.c.group = group;
    p.c.page_shift = 4;
    p.c.heads = 2;
    p.c.D = D;
    p.c.max_pages = 10;
    p.c.n_pages = 100;
    p.c.k = p.c.v = reinterpret_cast<uint8_t *>(0x10000);
    p.B = 3;
    p.T = T;
    p.G = G;
    p.q_heads = 2 * G;
    p.rows = T * G;
    tshc::LaunchCfg cfg;
    cfg.sm_count = kSms[device];
    cfg.pdl = true;
    return tshc::launch_tree_attention(p, cfg, nullptr);
}

int main()
{
    const int kinds[5][2] = {{0, 0}, {1, 0}, {2, 32}, {2, 64}, {2, 128}};
    bool first = true;
    for (int d : {0, 1, 2, 0})
        for (auto &kind : kinds)
            for (int D : {64, 128, 256})
                for (int T : {1, 20, 40, 70, 150}) {
                    if (kind[1] > D)
                        continue;
                    device = d;
                    if (d == 2 && first) {  // the refusal is this call's alone
                        first = false;
                        EXPECT(attend(kind[0], kind[1], D, T, 1) == cudaErrorNotReady);
                    }
                    launches = 0;
                    EXPECT(attend(kind[0], kind[1], D, T, 1) == cudaSuccess);
                    EXPECT(launches == 2);
                    const bool wide = D <= 128 && T > (kind[0] == 2 ? 64 : 32);
                    EXPECT(grid == (wide ? 1 : kPerSm[d]) * kSms[d]);
                }
    return wrong ? 1 : 0;
}
