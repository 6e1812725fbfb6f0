// Host driver of allow_lds (csrc/internal.h), for test_step_abi.py: the HIP
// calls that it makes are replaced by ones that keep a limit per device, as the
// runtime does. Prints "ok" where every launch would be within its limit.
#include <cstdio>
#include <map>
#include <thread>
#include <utility>
#include <vector>

#include "internal.h"

namespace {
std::mutex g_lock;
std::map<std::pair<const void*, int>, int> g_limit;
int g_sets = 0;
thread_local int t_device = 0;
void first_kernel() {}
void second_kernel() {}

bool fits(const void* kernel, int bytes) {
    std::lock_guard<std::mutex> lock(g_lock);
    const auto it = g_limit.find({kernel, t_device});
    return bytes <= (it == g_limit.end() ? 64 * 1024 : it->second);
}
template <auto Kernel>
bool launch(int device, int kilobytes) {
    t_device = device;
    return w4a16::allow_lds<Kernel>((size_t)kilobytes * 1024) == hipSuccess && fits(reinterpret_cast<const void*>(Kernel), kilobytes * 1024);
}
}  // namespace

extern "C" hipError_t hipGetDevice(int* device) {
    *device = t_device;
    return hipSuccess;
}
extern "C" hipError_t hipFuncSetAttribute(const void* kernel, hipFuncAttribute, int value) {
    std::lock_guard<std::mutex> lock(g_lock);
    g_limit[{kernel, t_device}] = value;
    ++g_sets;
    return hipSuccess;
}

int main() {
    int failures = 0;
    auto check = [&](bool ok, const char* what) {
        if (!ok) std::printf("FAIL %s\n", what), ++failures;
    };
    check(launch<first_kernel>(0, 64) && g_sets == 0, "within every device's limit");
    check(launch<first_kernel>(0, 80), "device 0");
    check(launch<first_kernel>(1, 80), "device 1");
    check(launch<second_kernel>(1, 100) && launch<second_kernel>(0, 90), "another kernel");
    check(launch<first_kernel>(0, 120) && launch<first_kernel>(0, 80) && launch<first_kernel>(0, 120), "never lowered");
    check(launch<first_kernel>(1, 80) && g_sets == 5, "asked for once");
    std::vector<std::thread> threads;
    std::atomic<int> bad{0};
    for (int t = 0; t < 8; ++t)
        threads.emplace_back([&, t] {
            for (int i = 0; i < 200; ++i) bad += !launch<second_kernel>(2 + i % 5, 65 + (t * 37 + i * 11) % 90);
        });
    for (auto& t : threads) t.join();
    check(bad == 0, "calls at once");
    if (failures == 0) std::printf("ok\n");
    return failures != 0;
}
