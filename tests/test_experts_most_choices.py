"""Routing and the exchange with the most choices that 31 bits count, for numbers of choices a token that do not divide 2^31, over the fake
CUDA runtime of test_experts_fake_runtime: every launch is one that the device takes."""
import os
import shutil
import subprocess

import pytest

from test_experts_fake_runtime import CSRC, DRIVER, ROOT

MAIN = r"""
int main()
{
    char *const B = reinterpret_cast<char *>(1 << 20);
    float *const F = reinterpret_cast<float *>(B);
    int32_t *const I = reinterpret_cast<int32_t *>(B);
    for (int32_t k : {1, 2, 3, 5, 7, 31, 32}) {
        const int64_t T = ((int64_t{1} << 31) - 1) / k;
        for (mlp_dtype dt : {MLP_DT_BF16, MLP_DT_F32}) {
            for (int64_t E : {k, 33, 300, 1024}) {
                every_failure("route", 1, [&] { return mlp_route_forward(T, E, k, B, E, dt, nullptr, 0, F, I, I, I, I, F, B, nullptr); });
                every_failure("route backward", 1, [&] { return mlp_route_backward(T, E, k, B, E, dt, 1, I, I, F, F, B, E, nullptr); });
            }
            // the widest rows of as many tokens: pieces of 128 bytes a token below 2^31
            const int64_t pieces = ((int64_t{1} << 31) - 1) / T, most = pieces * (dt == MLP_DT_F32 ? 32 : 64);
            for (int64_t C : {int64_t{1}, most / 2 + 1, most - 1, most})
                for (int64_t shift : {0, 4}) {
                    char *A = B + shift;
                    const int64_t R = (int64_t{1} << 31) - 1;
                    every_failure("dispatch", 1, [&] { return mlp_dispatch_forward(T, C, k, A, C, dt, I, R, A, C, nullptr); });
                    every_failure("dispatch backward", 1, [&] { return mlp_dispatch_backward(T, C, k, A, C, dt, I, R, A, C, A, C, nullptr); });
                    every_failure("combine", 1, [&] { return mlp_combine_forward(T, C, k, A, C, dt, F, I, R, A, C, A, C, nullptr); });
                    every_failure("combine backward", 1, [&] { return mlp_combine_backward(T, C, k, A, C, A, C, dt, F, I, R, A, C, F, nullptr); });
                }
        }
    }
    std::printf("%d wrong\n", bad);
    return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("nvcc") is None, reason="no nvcc")
def test_the_most_choices_over_a_fake_runtime(tmp_path):
    driver = tmp_path / "driver.cpp"
    driver.write_text(DRIVER[:DRIVER.index("int main()")] + MAIN)
    common = ["nvcc", "-std=c++17", "-Xcicc", "-O0", "-gencode", "arch=compute_103a,code=compute_103a", "-I", os.path.join(ROOT, "include")]
    compilers = [subprocess.Popen([*common, "-c", "-o", str(tmp_path / f"{n}.o"), os.path.join(CSRC, f"{n}.cu")]) for n in ("route", "exchange")]
    compilers.append(subprocess.Popen([*common, "-c", "-o", str(tmp_path / "driver.o"), str(driver)]))
    assert [c.wait() for c in compilers] == [0] * 3
    exe = str(tmp_path / "driver")
    subprocess.run(["g++", "-o", exe, *(str(tmp_path / f"{n}.o") for n in ("driver", "route", "exchange"))], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip().endswith("0 wrong"), run.stdout[-3000:]
