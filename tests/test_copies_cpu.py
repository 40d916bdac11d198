"""The copies straight into LDS that are written as instructions of their own (grouped products in large tiles) leave m0, which
the compiler keeps for itself, as they found it: read from the disassembly of the built library.  CPU only."""
import os
import re
import subprocess

import pytest

import submanifold_sparse_convolution_submconv3d_amd as sc

BIN = "/opt/rocm/llvm/bin"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{kernel: its instructions} of the large tiles."""
    tools = [os.path.join(BIN, t) for t in ("llvm-objdump", "clang-offload-bundler", "llvm-objcopy")]
    if not all(os.path.exists(t) for t in tools):
        pytest.skip("no LLVM tools")
    sc.load_library()
    d = tmp_path_factory.mktemp("code")
    fat = str(d / "fat")
    subprocess.check_call([tools[2], "--dump-section", ".hip_fatbin=" + fat, sc._LIB_PATH, os.devnull])
    # one bundle for each source file, at 4 KB boundaries
    blob, magic, found = open(fat, "rb").read(), b"__CLANG_OFFLOAD_BUNDLE__", {}
    starts = [m.start() for m in re.finditer(magic, blob)] + [len(blob)]
    for i, (a, b) in enumerate(zip(starts, starts[1:])):
        if b"k_linear_big" not in blob[a:b]:
            continue
        bundle, code = str(d / ("b%d" % i)), str(d / ("c%d" % i))
        with open(bundle, "wb") as f:
            f.write(blob[a:b])
        subprocess.check_call([tools[1], "--unbundle", "--type=o", "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", "--input=" + bundle, "--output=" + code])
        name = None
        for line in subprocess.check_output([tools[0], "-d", "--no-show-raw-insn", "--no-leading-addr", code], text=True).splitlines():
            m = re.match(r"(?:[0-9a-f]+ )?<(\S+)>:", line)
            if m:
                name = m.group(1) if "k_linear_big" in m.group(1) else None
            elif name and line.strip():
                found.setdefault(name, []).append(re.sub(r"\s*//.*", "", line).strip())
    return found


def test_copies_leave_m0_alone(kernels):
    assert len(kernels) >= 14
    for name, code in kernels.items():
        copies = [i for i, line in enumerate(code) if line.startswith("global_load_lds")]
        assert copies, name
        ours = set()
        for i in copies:
            save, to, wait, back = code[i - 3], code[i - 2], code[i - 1], code[i + 1]
            m = re.fullmatch(r"s_mov_b32 (\S+), m0", save)
            assert m and re.fullmatch(r"s_mov_b32 m0, \S+", to) and wait.startswith("s_nop") and back == "s_mov_b32 m0, %s" % m.group(1), (
                name, code[i - 3:i + 2])
            assert to != "s_mov_b32 m0, %s" % m.group(1)
            ours.update((i - 3, i - 2, i + 1))
        assert len(ours) == 3 * len(copies)
