"""CPU check of the adapters' chunk count over the whole range of rows that a call may have, at compile time on the kernel's own function."""
import os
import subprocess

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
