"""The streaming kernels' main loops in the built library (no GPU needed): a step overwrites the stage that the step before
it read, by loads that go to LDS past the registers, so the loop waits for every LDS read before its first such load."""
import os
import re
import subprocess

import pytest

import dense_tiled_gemm_amd as gb

LLVM = "/opt/rocm/llvm/bin"
OBJCOPY, BUNDLER, READELF, OBJDUMP = TOOLS = [os.path.join(LLVM, t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf",
                                                                             "llvm-objdump")]
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def code_objects(tmp_path):
    """Paths of the gfx950 code objects, one per source."""
    if not os.path.exists(gb.LIB_PATH):
        pytest.skip("library not built")
    if not all(os.path.exists(t) for t in TOOLS):
        pytest.skip("LLVM tools of the ROCm install not found")
    fat = str(tmp_path / "fat.bin")
    subprocess.run([OBJCOPY, "--dump-section=.hip_fatbin=" + fat, gb.LIB_PATH, os.devnull], check=True)
    data = open(fat, "rb").read()
    starts = [m.start() for m in re.finditer(MAGIC, data)]
    for i, (at, end) in enumerate(zip(starts, starts[1:] + [len(data)])):
        part, co = str(tmp_path / ("part%d.bin" % i)), str(tmp_path / ("part%d.co" % i))
        open(part, "wb").write(data[at:end])
        subprocess.run([BUNDLER, "--unbundle", "--type=o", "--input=" + part, "--targets=hipv4-amdgcn-amd-amdhsa--gfx950",
                        "--output=" + co], check=True)
        yield co


def main_loop(lines):
    """The instructions of one kernel's innermost loop that multiplies and loads to LDS, from behind its last LDS read on: the
    order in which they run, wherever the loop was rotated to; None without such a loop."""
    code = []
    for line in lines:
        m = re.match(r"\s+(.*?)\s*// ([0-9A-F]+): ", line)
        if m:
            code.append((int(m.group(2), 16), m.group(1)))
    at = {address: i for i, (address, _) in enumerate(code)}
    best = None
    for i, (address, text) in enumerate(code):
        m = re.match(r"s_c?branch\S*\s+(\d+)", text)
        if not m:
            continue
        words = int(m.group(1))
        first = at.get(address + 4 + 4 * (words - 65536 if words >= 32768 else words))
        if first is not None and first < i and (best is None or i + 1 - first < len(best)):
            body = [t for _, t in code[first:i + 1]]
            if all(any(f(t) for t in body) for f in (is_stage_load, is_read, lambda t: "mfma" in t)):
                best = body
    if best is None:
        return None
    last = max(i for i, t in enumerate(best) if is_read(t))
    return best[last + 1:] + best[:last + 1]


def is_read(text):
    return text.startswith("ds_read")


def is_stage_load(text):
    return text.startswith("buffer_load") and text.split()[-1] == "lds"


def test_reads_are_waited_for_before_their_stage_is_overwritten(tmp_path):
    seen = 0
    for co in code_objects(tmp_path):
        symbols = subprocess.run([READELF, "-sW", co], check=True, capture_output=True, text=True).stdout
        names = sorted({n for n in re.findall(r"FUNC\s+\S+\s+\S+\s+\S+\s+(\S+)", symbols) if "skinny" in n})
        if not names:
            continue
        text = subprocess.run([OBJDUMP, "-d", "--disassemble-symbols=" + ",".join(names), co], check=True, capture_output=True,
                              text=True).stdout
        for part in re.split(r"\n(?=[0-9a-f]+ <)", text):
            name = re.search(r"<(\S+)>:", part)
            body = main_loop(part.split("\n")) if name else None
            if body is None:
                continue
            waits = [t for t in body[:next(i for i, t in enumerate(body) if is_stage_load(t))] if t.startswith("s_waitcnt")]
            # with the wait for the step's own stage, or behind it: every read of the step before
            stage = next(i for i, t in enumerate(waits) if "vmcnt" in t)
            assert any("lgkmcnt(0)" in t for t in waits[stage:]), name.group(1)
            seen += 1
    assert seen >= 32, seen  # 12 of scales per block, 15 gated, 5 with an epilogue, and the plain ones
