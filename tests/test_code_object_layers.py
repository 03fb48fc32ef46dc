"""The scratch check of the product kernels, for the code objects of every source in the library (no GPU needed)."""
import os
import re
import subprocess

import pytest

import dense_tiled_gemm_amd as gb

LLVM = "/opt/rocm/llvm/bin"
TOOLS = [os.path.join(LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf")]
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def test_no_kernel_of_any_source_uses_scratch(tmp_path):
    if not os.path.exists(gb.LIB_PATH):
        pytest.skip("library not built")
    if not all(os.path.exists(t) for t in TOOLS):
        pytest.skip("LLVM tools of the ROCm install not found")
    fat = str(tmp_path / "fat.bin")
    subprocess.run([TOOLS[0], "--dump-section=.hip_fatbin=" + fat, gb.LIB_PATH, os.devnull], check=True)
    data = open(fat, "rb").read()
    starts = [m.start() for m in re.finditer(MAGIC, data)]
    assert len(starts) == 4, starts  # one bundle per source
    seen = []
    for i, (at, end) in enumerate(zip(starts, starts[1:] + [len(data)])):
        part, co = str(tmp_path / ("part%d.bin" % i)), str(tmp_path / ("part%d.co" % i))
        open(part, "wb").write(data[at:end])
        subprocess.run([TOOLS[1], "--unbundle", "--type=o", "--input=" + part,
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", "--output=" + co], check=True)
        notes = subprocess.run([TOOLS[2], "--notes", co], check=True, capture_output=True, text=True).stdout
        for block in notes.split("  - .agpr_count")[1:]:
            field = lambda key: int(re.search(r"\." + key + r":\s+(\d+)", block).group(1))
            name = re.search(r"\.name:\s+(\S+)", block).group(1)
            assert field("private_segment_fixed_size") == 0, name
            assert field("vgpr_spill_count") == 0 and field("sgpr_spill_count") == 0, name
            assert field("vgpr_count") <= 256, name
            seen.append(name)
    for kernel in ("norm_kernel", "norm_back_kernel", "norm_long_kernel", "act_back_kernel", "fold_kernel", "skinny_epi_kernel",
                   "epi_fill_kernel", "linear_back_kernel", "slices_kernel", "pad_rows_kernel", "dma_kernel", "trans_kernel"):
        assert any(kernel in n for n in seen), kernel
