"""CPU checks of how the adapters cut a call: the chunk count over the whole range of rows that a call may have, at compile time on
the kernel's own function, and the choice of the launch form with its workspace."""
import os
import random
import subprocess

import w4a4_mxfp4_quantized_b200 as mq
from w4a4_mxfp4_quantized_b200 import build as mq_build

CHECKS = """
#include <stdint.h>
#include "lora.cuh"
constexpr bool all(int32_t most) {
    for (int64_t rows : {int64_t{0}, int64_t{1}, int64_t{15}, int64_t{16}, int64_t{17}, int64_t{63}, int64_t{64}, int64_t{65},
                         (int64_t{1} << 30) + 1, (int64_t{1} << 31) - 65, (int64_t{1} << 31) - 64, (int64_t{1} << 31) - 17,
                         (int64_t{1} << 31) - 15, (int64_t{1} << 31) - 1})
        if (macaq::lora_chunk_count(static_cast<int32_t>(rows), most) != (rows + most - 1) / most) return false;
    return true;
}
static_assert(all(16) && all(64), "chunks of an adapter's rows");
"""


def test_chunk_count_over_all_row_counts(tmp_path):
    src = tmp_path / "chunks.cu"
    src.write_text(CHECKS)
    flags = [f for f in mq_build.NVCC_FLAGS if f != "-shared"]
    subprocess.run([mq_build.nvcc(), *flags, f"-I{mq_build.INCLUDE}", f"-I{mq_build.CSRC}", "-c", "-o", os.fspath(tmp_path / "chunks.o"),
                    os.fspath(src)], check=True)


def test_workspace_without_widths_is_enough_for_every_width():
    mq_build.build()
    rng = random.Random(1)
    sizes = [8, 64, 328, 1024, 4096, 14336, 1 << 20, 1 << 24]
    for _ in range(3000):
        M, r, L = int(2 ** rng.uniform(0, 20)), 8 * rng.randint(1, 16), rng.choice([1, 2, 4, 16, 32, 33, 100, 1024])
        K, N, dtype = rng.choice(sizes), rng.choice(sizes), rng.choice([mq.OUT_BF16, mq.OUT_F32])
        need = mq.lora_workspace_bytes(M, r, L, dtype, K, N)
        for k, n in ((0, 0), (K, 0), (0, N)):
            assert mq.lora_workspace_bytes(M, r, L, dtype, k, n) >= need, (M, r, L, dtype, K, N)


def test_the_bank_does_not_decide_the_launch_form():
    """2048 rows on 4096 -> 14336 take the two launches however many adapters are loaded; a decode batch of 64 takes one."""
    mq_build.build()
    for L in (1, 4, 32, 33, 64, 65, 128, 129, 256, 1024):
        assert mq.lora_workspace_bytes(2048, 64, L, mq.OUT_BF16, 4096, 14336) > 0, L
        assert mq.lora_workspace_bytes(2048, 16, L, mq.OUT_BF16, 4096, 14336) > 0, L
    for L in (32, 33, 64, 1024):
        assert mq.lora_workspace_bytes(64, 16, L, mq.OUT_BF16, 4096, 14336) == 0, L
